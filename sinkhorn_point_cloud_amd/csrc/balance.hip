// balance.hip -- an expert router's balance loss, its counts and its gradient.
//
// For a group of rows (one packed sequence, or the whole batch) with chosen
// experts [T][K], p = softmax of a row of router logits, n = the rows of the
// group that chose anything:
//     counts_e = how often expert e was chosen,   f_e = E counts_e / (K n),
//     balance  = (1/n) sum_t sum_e f_e p_te       (1 when all are equal),
//     zloss    = (1/n) sum_t LSE_t^2,
//     d(alpha balance + zeta zloss)/dz_te
//              = p_te (alpha (f_e - sum_j f_j p_tj) + 2 zeta LSE_t) / n.
// The counts come from the choices alone, so the logits are read once: the
// pass that knows f writes the gradient, and a row's sum f . p, which the
// gradient needs anyway, is also all that the loss needs.  Since sum_e p = 1,
// f - 1 stands for f in those differences: near balance nothing cancels.
//
// Three launches: counts per chunk of rows; gradient, each work-group summing
// its group's counts first; sums per group.  Chunks lie within one group and
// the sums are taken in a fixed order: no atomics in memory, the same result
// every time.
//
// What bounds it: HBM for large batches, the launches for small ones.
#include "rows.h"
#include "token_loss.h"

namespace sk {
namespace {

using rows::Pack;
using rows::kInf;
using rows::shift_of;
using rows::grid_of;
using rows::group_index;

constexpr int kThreads = 256;

// Where a chunk of `size` rows lies: its group, its rows, and the group's chunks.
struct Place {
    int group;            // -1: no such chunk
    long first, last;     // rows of the chunk
    long chunk0, chunks;  // the group's first chunk and how many it has
};

__device__ __forceinline__ long clamp_row(long v, long T) { return min(max(v, 0l), T); }

// Every lane of the calling wave gets the answer.
__device__ Place place_of(const BalanceArgs &a, long chunk, long size)
{
    const long T = a.T;
    Place r{-1, 0, 0, 0, 0};
    if (!a.offsets) {
        r.chunks = (T + size - 1) / size;
        if (chunk < r.chunks)
            r.group = 0;
        r.first = chunk * size;
        r.last = min(r.first + size, T);
        return r;
    }
    long before = 0;
    for (int base = 0; base < a.G; base += kWave) {
        const int g = base + lane_id();
        long b = 0, e = 0;
        if (g < a.G) {
            b = clamp_row(a.offsets[g], T);
            e = max(clamp_row(a.offsets[g + 1], T), b);
        }
        const long n = (e - b + size - 1) / size;
        long upto = n;   // inclusive sum over the lanes
#pragma unroll
        for (int d = 1; d < kWave; d <<= 1) {
            const long o = __shfl_up(upto, d, kWave);
            if (lane_id() >= d)
                upto += o;
        }
        const unsigned long long hit = __ballot(chunk < before + upto);
        if (hit) {
            const int at = __ffsll(hit) - 1;
            r.group = base + at;
            r.chunks = __shfl(n, at, kWave);
            r.chunk0 = before + __shfl(upto, at, kWave) - r.chunks;
            r.first = __shfl(b, at, kWave) + (chunk - r.chunk0) * size;
            r.last = min(r.first + size, __shfl(e, at, kWave));
            return r;
        }
        before += __shfl(upto, kWave - 1, kWave);
    }
    return r;
}

// Tokens per expert, rows with a choice and bad indices of one chunk of rows.
__global__ __launch_bounds__(kThreads) void count_kernel(BalanceArgs a, BalanceWs w, long size)
{
    extern __shared__ int hist[];   // [E + 2]
    const long chunk = group_index();
    const Place at = place_of(a, chunk, size);
    if (at.group < 0)
        return;
    for (int e = threadIdx.x; e < a.E + 2; e += kThreads)
        hist[e] = 0;
    __syncthreads();
    int rows = 0, bad = 0;
    for (long t = at.first + threadIdx.x; t < at.last; t += kThreads) {
        const int32_t *idx = a.index + t * a.K;
        bool any = false;
        for (int k = 0; k < a.K; ++k) {
            const int e = idx[k];
            if (e >= a.E)
                ++bad;
            else if (e >= 0) {
                any = true;
                atomicAdd(&hist[e], 1);
            }
        }
        rows += any;
    }
    rows = wave_sum(rows);
    bad = wave_sum(bad);
    if (lane_id() == 0) {
        atomicAdd(&hist[a.E], rows);
        atomicAdd(&hist[a.E + 1], bad);
    }
    __syncthreads();
    int32_t *out = w.count_part + chunk * (a.E + 2);
    for (int e = threadIdx.x; e < a.E + 2; e += kThreads)
        out[e] = hist[e];
}

// Reductions over the L lanes of a row.
template <int L> __device__ __forceinline__ float lanes_sum(float v)
{
#pragma unroll
    for (int o = L / 2; o > 0; o >>= 1)
        v += __shfl_xor(v, o, kWave);
    return v;
}
template <int L> __device__ __forceinline__ float lanes_max(float v)
{
#pragma unroll
    for (int o = L / 2; o > 0; o >>= 1)
        v = fmaxf(v, __shfl_xor(v, o, kWave));
    return v;
}

// One chunk of rows, L lanes to a row and R values to a lane.
template <typename T, int L, int R>
__global__ __launch_bounds__(kThreads) void balance_kernel(BalanceArgs a, BalanceWs w, long size,
                                                           long count_size)
{
    extern __shared__ float f1[];   // [E]: f - 1
    __shared__ double room[2 * kThreads / kWave];
    const long chunk = group_index();
    const Place at = place_of(a, chunk, size);
    if (at.group < 0)
        return;
    const int E = a.E, K = a.K;
    // the group's counts, from its chunks of the first pass
    long c0 = 0, cn = (a.T + count_size - 1) / count_size;
    if (a.offsets) {
        // chunks of the groups before this one
        for (int g = threadIdx.x % kWave; g < at.group; g += kWave) {
            const long b = clamp_row(a.offsets[g], a.T);
            c0 += (max(clamp_row(a.offsets[g + 1], a.T), b) - b + count_size - 1) / count_size;
        }
        c0 = wave_sum(c0);
        const long b = clamp_row(a.offsets[at.group], a.T);
        cn = (max(clamp_row(a.offsets[at.group + 1], a.T), b) - b + count_size - 1) / count_size;
        cn = min(cn, w.count_chunks - c0);
    }
    const int32_t *part = w.count_part + c0 * (E + 2);
    int n = 0, bad = 0;
    for (long i = lane_id(); i < cn; i += kWave) {
        n += part[i * (E + 2) + E];
        bad += part[i * (E + 2) + E + 1];
    }
    n = wave_sum(n);
    bad = wave_sum(bad);
    const double per = n ? (double)E / ((double)K * (double)n) : 0.0;
    for (int e = threadIdx.x; e < E; e += kThreads) {
        int c = 0;
        for (long i = 0; i < cn; ++i)
            c += part[i * (E + 2) + e];
        f1[e] = bad ? __builtin_nanf("") : (float)((double)c * per - 1.0);
        if (chunk == at.chunk0)
            a.counts[(long)at.group * E + e] = c;
    }
    __syncthreads();

    const int lane = threadIdx.x % L, slot = threadIdx.x / L;
    float f[R];
#pragma unroll
    for (int r = 0; r < R; ++r)
        f[r] = lane + r * L < E ? f1[lane + r * L] : 0.f;
    const float over = n ? 1.f / (float)n : 0.f;
    const float alpha = (float)a.balance * over, zeta = (float)(2.0 * a.z) * over;
    double dots = 0.0, squares = 0.0;
    for (long t = at.first + slot; t < at.last; t += kThreads / L) {
        const T *row = (const T *)a.logits + t * a.ld;
        T *out = a.dlogits ? (T *)a.dlogits + t * a.dld : nullptr;
        int chose = 0;
        for (int k = lane; k < K; k += L) {
            const int e = a.index[t * K + k];
            chose |= e >= 0;
        }
        float x[R], m = -kInf, s = 0.f, dot = 0.f;
#pragma unroll
        for (int r = 0; r < R; ++r) {
            x[r] = lane + r * L < E ? Pack<T>::get(row + lane + r * L) : -kInf;
            m = fmaxf(m, x[r]);
        }
        chose = lanes_max<L>((float)chose) > 0.f;
        m = lanes_max<L>(m);
        const float shift = shift_of(m);
#pragma unroll
        for (int r = 0; r < R; ++r) {
            x[r] = ex2((x[r] - shift) * kLog2e);
            s += x[r];
            dot = fmaf(x[r], f[r], dot);
        }
        s = lanes_sum<L>(s);
        dot = lanes_sum<L>(dot);
        const bool used = chose && s != 0.f;
        const float inv = used ? 1.f / s : 0.f, lse = used ? m + logf(s) : 0.f;
        dot *= inv;
        if (used && lane == 0) {
            dots += 1.0 + (double)dot;
            squares += (double)lse * (double)lse;
        }
        if (out) {
            const float base = fmaf(zeta, lse, -alpha * dot);
#pragma unroll
            for (int r = 0; r < R; ++r)
                if (lane + r * L < E)
                    Pack<T>::put(out + lane + r * L,
                                 used ? x[r] * inv * fmaf(alpha, f[r], base) : 0.f);
        }
    }
    dots = wave_sum(dots);
    squares = wave_sum(squares);
    if (lane_id() == 0) {
        room[threadIdx.x / kWave] = dots;
        room[kThreads / kWave + threadIdx.x / kWave] = squares;
    }
    __syncthreads();
    if (threadIdx.x < 2) {
        double v = 0.0;
        for (int i = 0; i < kThreads / kWave; ++i)
            v += room[threadIdx.x * (kThreads / kWave) + i];
        w.sum_part[2 * chunk + threadIdx.x] = v;
    }
}

// The losses of one group; the counts of a group without rows; with `fill`,
// zeros over the rows outside every group (by the groups before and behind).
__global__ __launch_bounds__(kThreads) void balance_sum_kernel(BalanceArgs a, BalanceWs w,
                                                               long size, long count_size)
{
    __shared__ double room[kThreads / kWave][2];
    __shared__ long seen[kThreads / kWave][2];
    const int g = blockIdx.x, E = a.E;
    const long T = a.T;
    long b = 0, e = T, c0 = 0, k0 = 0;
    if (a.offsets) {
        for (int i = threadIdx.x; i < g; i += kThreads) {
            const long bi = clamp_row(a.offsets[i], T);
            const long len = max(clamp_row(a.offsets[i + 1], T), bi) - bi;
            c0 += (len + size - 1) / size;
            k0 += (len + count_size - 1) / count_size;
        }
        c0 = wave_sum(c0);
        k0 = wave_sum(k0);
        if (lane_id() == 0) {
            seen[threadIdx.x / kWave][0] = c0;
            seen[threadIdx.x / kWave][1] = k0;
        }
        __syncthreads();
        c0 = k0 = 0;
        for (int i = 0; i < kThreads / kWave; ++i) {
            c0 += seen[i][0];
            k0 += seen[i][1];
        }
        b = clamp_row(a.offsets[g], T);
        e = max(clamp_row(a.offsets[g + 1], T), b);
    }
    // the caps hold for offsets in order; out of order they keep the reads in bounds
    const long cn = min((e - b + size - 1) / size, w.grad_chunks - c0);
    const long kn = min((e - b + count_size - 1) / count_size, w.count_chunks - k0);
    double v[2] = {0.0, 0.0};
    for (long i = threadIdx.x; i < cn; i += kThreads) {
        v[0] += w.sum_part[2 * (c0 + i)];
        v[1] += w.sum_part[2 * (c0 + i) + 1];
    }
    int n = 0;
    for (long i = 0; i < kn; ++i)
        n += w.count_part[(k0 + i) * (E + 2) + E];
    v[0] = wave_sum(v[0]);
    v[1] = wave_sum(v[1]);
    if (lane_id() == 0) {
        room[threadIdx.x / kWave][0] = v[0];
        room[threadIdx.x / kWave][1] = v[1];
    }
    __syncthreads();
    if (threadIdx.x < 2) {
        double s = 0.0;
        for (int i = 0; i < kThreads / kWave; ++i)
            s += room[i][threadIdx.x];
        (threadIdx.x ? a.zloss : a.loss)[g] = n ? (float)(s / (double)n) : 0.f;
    }
    if (cn <= 0)
        for (int i = threadIdx.x; i < E; i += kThreads)
            a.counts[(long)g * E + i] = 0;
}

template <typename T> __global__ void fill_kernel(BalanceArgs a)
{
    const long t = group_index();
    if (t >= a.T)
        return;
    const long first = clamp_row(a.offsets[0], a.T), last = clamp_row(a.offsets[a.G], a.T);
    if (t >= first && t < last)
        return;
    T *out = (T *)a.dlogits + t * a.dld;
    for (int e = threadIdx.x; e < a.E; e += kWave)
        Pack<T>::put(out + e, 0.f);
}

// Rows of a chunk: about 64 chunks to count, about 1024 work-groups for the rest.
long count_size(int T) { return std::max(256l, ((long)T + 63) / 64); }
int lanes_of(int E) { return E <= 8 ? 8 : E <= 16 ? 16 : E <= 32 ? 32 : 64; }
long grad_size(int T, int E)
{
    const long pass = kThreads / lanes_of(E);   // rows a work-group takes at once
    const long want = ((long)T + 1023) / 1024;
    return (want + pass - 1) / pass * pass;
}

template <typename T, int L, int R>
void run(const BalanceArgs &a, const BalanceWs &w, hipStream_t st)
{
    hipLaunchKernelGGL((balance_kernel<T, L, R>), grid_of(balance_grad_chunks(a.T, a.E, a.G)),
                       dim3(kThreads), (size_t)a.E * 4, st, a, w, grad_size(a.T, a.E),
                       count_size(a.T));
}

template <typename T> void run_rows(const BalanceArgs &a, const BalanceWs &w, hipStream_t st)
{
    if (a.E <= 8)
        run<T, 8, 1>(a, w, st);
    else if (a.E <= 16)
        run<T, 16, 1>(a, w, st);
    else if (a.E <= 32)
        run<T, 32, 1>(a, w, st);
    else if (a.E <= 64)
        run<T, 64, 1>(a, w, st);
    else if (a.E <= 128)
        run<T, 64, 2>(a, w, st);
    else if (a.E <= 256)
        run<T, 64, 4>(a, w, st);
    else if (a.E <= 512)
        run<T, 64, 8>(a, w, st);
    else
        run<T, 64, 16>(a, w, st);
    if (a.fill && a.offsets && a.dlogits)
        hipLaunchKernelGGL((fill_kernel<T>), grid_of(a.T), dim3(kWave), 0, st, a);
}

}  // namespace

long balance_count_chunks(int T, int G) { return T / count_size(T) + G; }
long balance_grad_chunks(int T, int E, int G) { return T / std::max(1l, grad_size(T, E)) + G; }

hipError_t launch_balance(const BalanceArgs &a, const BalanceWs &w, hipStream_t st)
{
    if (a.T > 0) {
        hipLaunchKernelGGL(count_kernel, grid_of(balance_count_chunks(a.T, a.G)), dim3(kThreads),
                           (size_t)(a.E + 2) * 4, st, a, w, count_size(a.T));
        if (a.dtype == 1)
            run_rows<uint16_t>(a, w, st);
        else
            run_rows<float>(a, w, st);
    }
    hipLaunchKernelGGL(balance_sum_kernel, dim3(a.G), dim3(kThreads), 0, st, a, w,
                       std::max(1l, grad_size(a.T, a.E)), count_size(a.T));
    return hipGetLastError();
}

}  // namespace sk
