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
// Large batches take three launches: counts per chunk of rows; gradient, each
// work-group summing its group's counts first; sums per group.  Small ones take
// one, a work-group per group doing all of it: 512 rows of 8 experts take 12.7 us a
// call against 18.3, for the host has two launches fewer (of kernels 10.4 against
// 9.7).  Chunks lie within one group and the sums are taken in a fixed order: no
// atomics in memory, the same result every time.
//
// Within a row everything is fp32, with one rounding of each exponent: a row has at
// most 1024 terms, 64 to a lane, and nothing is taken from the softmax but products
// that are rounded to the outputs' 24 or 8 bits.  Gradients are off by 1e-7 to 2e-7
// of themselves that way, losses by less (fp64 from the row on).
//
// A row is 16 lanes' (reductions are lane moves within a row of the wave), four
// rows to a wave, the next row loaded while one is worked on.
//
// What bounds it: for large batches one launch waiting for the other and, in each
// work-group, the group's counts before the first row (65536 x 256 bf16: 6, 20 and 4
// us, 3.3 TB/s in the second); for small ones the rounds of a single work-group
// (512 x 8) and the call.  More than 512 experts: 64 values a lane, which spill
// beside the row that is asked for ahead (64 x 1024 33 us).
#include "rows.h"
#include "token_loss.h"

namespace sk {
namespace {

using rows::Pack;
using rows::kInf;
using rows::shift_of;
using rows::grid_of;
using rows::group_index;

constexpr int kThreads = 256;    // a chunk's work-group
constexpr int kCounters = 512;   // a counting work-group
constexpr int kSmall = 1024;     // a small group's
constexpr int kLanes = 16;       // lanes of a row
constexpr int kBatch = 16;       // partial counts a thread asks for at once
constexpr int kFillers = 64;     // work-groups that zero the rows outside every group

// How rows are cut into chunks: 2^count_bits of them to count, 2^grad_bits for the
// gradient.  Row numbers and chunks fit 32 bits (2^24 rows, 2^20 groups).
struct Sizes {
    int count_bits, grad_bits;
};
__device__ __forceinline__ int chunks_of(int rows, int bits)
{
    return (rows + (1 << bits) - 1) >> bits;
}
// Chunk numbers of group g, which begins at row b: from g + floor(b / size) on.  A
// group of b to e has floor(e / size) - floor(b / size) + 1 numbers that way, at
// least as many as it needs, and no sum over the groups before it is formed.
// Numbers left over are work-groups that end at once.
__device__ __forceinline__ int chunk0_of(int g, int b, int bits) { return g + (b >> bits); }

// Where a chunk lies: its group and rows, and the group's chunks of either kind.
struct Place {
    int group;                  // -1: no such chunk
    int first, last;            // rows of the chunk
    int count0, counts;         // the group's first counting chunk and how many it has
    bool leads;                 // the group's first chunk
};

__device__ __forceinline__ int clamp_row(int64_t v, int T)
{
    return (int)min(max(v, (int64_t)0), (int64_t)T);
}

// The place of chunk number `chunk` of the one kind or the other; every lane of
// the calling wave gets the answer.  The group is the last that begins at or
// before the chunk: each round of the search asks for 64 groups at equal
// distances, so 64 groups take one and 2^20 four.
template <bool Grad> __device__ Place place_of(const BalanceArgs &a, const Sizes &z, int chunk)
{
    const int T = a.T, bits = Grad ? z.grad_bits : z.count_bits;
    Place r{-1, 0, 0, 0, 0, false};
    int g = 0, b = 0, e = T;
    if (a.offsets) {
        for (int count = a.G;;) {
            const int step = (count + kWave - 1) / kWave, at = g + lane_id() * step;
            const int row = clamp_row(a.offsets[min(at, a.G)], T);
            const bool begun = at < g + count && chunk0_of(at, row, bits) <= chunk;
            const int lane = max((int)__popcll(__ballot(begun)) - 1, 0);
            g += lane * step;
            if (step == 1) {
                b = __shfl(row, lane, kWave);
                e = lane + 1 < kWave ? __shfl(row, lane + 1, kWave)
                                     : clamp_row(a.offsets[g + 1], T);
                e = max(e, b);
                break;
            }
            count = min(step, count - lane * step);
        }
    }
    const int i = chunk - chunk0_of(g, b, bits);
    // (negative: offsets out of order)
    if (i < 0 || i >= chunks_of(e - b, bits))
        return r;
    r.group = g;
    r.first = b + (i << bits);
    r.last = min(r.first + (1 << bits), e);
    r.count0 = chunk0_of(g, b, z.count_bits);
    r.counts = chunks_of(e - b, z.count_bits);
    r.leads = i == 0;
    return r;
}

// Adds the choices of rows [first, last) to hist [E + 2]: tokens per expert,
// rows with a choice, indices out of range.
template <int NT>
__device__ __forceinline__ void count_rows(const BalanceArgs &a, int first, int last, int *hist)
{
    int rows = 0, bad = 0;
    for (int t = first + threadIdx.x; t < last; t += NT) {
        const int32_t *idx = a.index + (long)t * a.K;
        bool any = false;
        for (int k = 0; k < a.K; k += 8) {
            int e[8];
#pragma unroll
            for (int j = 0; j < 8; ++j)
                e[j] = k + j < a.K ? idx[k + j] : -1;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                any |= e[j] >= 0;
                bad += e[j] >= a.E;
                if (e[j] >= 0 && e[j] < a.E)
                    atomicAdd(&hist[e[j]], 1);
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
}

__global__ __launch_bounds__(kCounters) void count_kernel(BalanceArgs a, BalanceWs w, Sizes z)
{
    extern __shared__ int hist[];   // [E + 2]
    const long chunk = group_index();
    if (chunk >= w.count_chunks)
        return;
    const Place at = place_of<false>(a, z, (int)chunk);
    if (at.group < 0)
        return;
    for (int e = threadIdx.x; e < a.E + 2; e += kCounters)
        hist[e] = 0;
    __syncthreads();
    count_rows<kCounters>(a, at.first, at.last, hist);
    __syncthreads();
    int32_t *out = w.count_part + chunk * (a.E + 2);
    for (int e = threadIdx.x; e < a.E + 2; e += kCounters)
        out[e] = hist[e];
}

__device__ __forceinline__ float lanes_max(float v)
{
    v = fmaxf(v, dpp_move<kDppXor1>(v));
    v = fmaxf(v, dpp_move<kDppXor2>(v));
    v = fmaxf(v, dpp_move<kDppHalfMirror>(v));
    return fmaxf(v, dpp_move<kDppMirror>(v));
}

// R values a lane, W of them side by side; Wide: in one load or store, where
// every row starts on such a boundary and E is a multiple of W.  A lane's columns
// are the same either way, and with them the order of every sum.
template <typename T, int R, bool Wide> struct Values {
    static constexpr int W = R < 4 ? R : 4;
    struct alignas(W * sizeof(T)) Word {
        T v[W];
    };
    Word w[R / W];
    int first;   // the row's first index

    __device__ __forceinline__ static int column(int r, int lane)
    {
        return (r / W * kLanes + lane) * W + r % W;
    }
    __device__ __forceinline__ void load(const BalanceArgs &a, int t, int lane)
    {
        const T *row = (const T *)a.logits + t * a.ld;
#pragma unroll
        for (int i = 0; i < R / W; ++i) {
            const int c = column(i * W, lane);
            if constexpr (Wide) {
                if (c < a.E)
                    w[i] = *reinterpret_cast<const Word *>(row + c);
            } else {
#pragma unroll
                for (int j = 0; j < W; ++j)
                    if (c + j < a.E)
                        w[i].v[j] = row[c + j];
            }
        }
        int any = -1;
        for (int k = lane; k < a.K; k += kLanes)
            any = max(any, a.index[(long)t * a.K + k]);
        first = any;
    }
};

// The rows [first, last) of one group, NT threads: gradients, and this thread's
// part of the sums.  The first rows are asked for before the group's counts are
// known.
template <typename T, int NT, int R, bool Wide> struct GroupRows {
    using V = Values<T, R, Wide>;
    static constexpr int W = V::W, slots = NT / kLanes;
    const BalanceArgs &a;
    const int first, last, lane, t0;
    V next;

    __device__ __forceinline__ GroupRows(const BalanceArgs &args, int first, int last)
        : a(args), first(first), last(last), lane(threadIdx.x % kLanes),
          t0(first + threadIdx.x / kLanes)
    {
        if (t0 < last)
            next.load(a, t0, lane);
    }
    // f1 [E]: f - 1
    __device__ __forceinline__ void run(const float *f1, int n, double &dots, double &squares)
    {
        const int E = a.E;
        float f[R];
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const int c = V::column(r, lane);
            f[r] = c < E ? f1[c] : 0.f;
        }
        const float over = n ? 1.f / (float)n : 0.f;
        const float alpha = (float)a.balance * over, zeta = (float)(2.0 * a.z) * over;
        // all lanes of a wave stay together: the lane moves need them
        const int rounds = (last - first + slots - 1) / slots;
        for (int i = 0; i < rounds; ++i) {
            const int t = t0 + i * slots;
            const V now = next;
            if (t + slots < last)
                next.load(a, t + slots, lane);
            const bool row = t < last;
            float x[R], m = -kInf, s = 0.f, dot = 0.f;
#pragma unroll
            for (int r = 0; r < R; ++r) {
                x[r] = row && V::column(r, lane) < E ? Pack<T>::get(&now.w[r / W].v[r % W]) : -kInf;
                m = fmaxf(m, x[r]);
            }
            const bool chose = lanes_max(row && now.first >= 0 ? 1.f : 0.f) > 0.f;
            m = lanes_max(m);
            const float shift = shift_of(m);
#pragma unroll
            for (int r = 0; r < R; ++r) {
                x[r] = ex2((x[r] - shift) * kLog2e);
                s += x[r];
                dot = fmaf(x[r], f[r], dot);
            }
            s = row16_sum(s);
            dot = row16_sum(dot);
            const bool used = chose && s != 0.f;
            const float inv = used ? 1.f / s : 0.f, lse = used ? m + logf(s) : 0.f;
            dot *= inv;
            if (used && lane == 0) {
                dots += 1.0 + (double)dot;
                squares += (double)lse * (double)lse;
            }
            if (a.dlogits && row) {
                T *out = (T *)a.dlogits + t * a.dld;
                const float base = fmaf(zeta, lse, -alpha * dot);
#pragma unroll
                for (int i = 0; i < R / W; ++i) {
                    const int c = V::column(i * W, lane);
                    typename V::Word y;
#pragma unroll
                    for (int j = 0; j < W; ++j)
                        Pack<T>::put(&y.v[j], used ? x[i * W + j] * inv *
                                                         fmaf(alpha, f[i * W + j], base)
                                                   : 0.f);
                    if constexpr (Wide) {
                        if (c < E)
                            *reinterpret_cast<typename V::Word *>(out + c) = y;
                    } else {
#pragma unroll
                        for (int j = 0; j < W; ++j)
                            if (c + j < E)
                                out[c + j] = y.v[j];
                    }
                }
            }
        }
    }
};

// The two sums over the work-group, in a fixed order; thread 0 and 1 get them.
template <int NT>
__device__ __forceinline__ double group_sums(double dots, double squares, double *room)
{
    constexpr int waves = NT / kWave;
    dots = rows::sum_wave(dots);
    squares = rows::sum_wave(squares);
    if (lane_id() == 0) {
        room[threadIdx.x / kWave] = dots;
        room[waves + threadIdx.x / kWave] = squares;
    }
    __syncthreads();
    double v = 0.0;
    if (threadIdx.x < 2)
        for (int i = 0; i < waves; ++i)
            v += room[threadIdx.x * waves + i];
    return v;
}

// Zeros over the rows outside every group, one of kFillers work-groups.
template <typename T, int NT> __device__ void fill_rows(const BalanceArgs &a, int filler)
{
    const int first = clamp_row(a.offsets[0], a.T);
    const int last = max(clamp_row(a.offsets[a.G], a.T), first);
    const int count = first + a.T - last;
    for (int i = filler * (NT / kWave) + threadIdx.x / kWave; i < count;
         i += kFillers * (NT / kWave)) {
        T *out = (T *)a.dlogits + (long)(i < first ? i : last + i - first) * a.dld;
        for (int e = lane_id(); e < a.E; e += kWave)
            Pack<T>::put(out + e, 0.f);
    }
}

// One chunk of rows.
template <typename T, int R, bool Wide>
__global__ __launch_bounds__(kThreads) void balance_kernel(BalanceArgs a, BalanceWs w, Sizes z)
{
    extern __shared__ int dyn[];   // [E + 2] counts, [E] f - 1
    __shared__ double room[2 * kThreads / kWave];
    const long chunk = group_index();
    if (chunk >= w.grad_chunks) {
        if (a.fill && a.offsets && a.dlogits && chunk < w.grad_chunks + kFillers)
            fill_rows<T, kThreads>(a, (int)(chunk - w.grad_chunks));
        return;
    }
    const Place at = place_of<true>(a, z, (int)chunk);
    if (at.group < 0)
        return;
    GroupRows<T, kThreads, R, Wide> rows(a, at.first, at.last);
    const int E = a.E, K = a.K;
    int *count = dyn;
    float *f1 = (float *)(dyn + E + 2);
    for (int e = threadIdx.x; e < E + 2; e += kThreads)
        count[e] = 0;
    // the group's counts, from its chunks of the first pass (the cap holds for
    // offsets in order; out of order it keeps the reads in bounds)
    const int c0 = at.count0, cn = min(at.counts, (int)w.count_chunks - c0);
    __syncthreads();
    const int32_t *part = w.count_part + (long)c0 * (E + 2);
    const int total = cn * (E + 2);
    if (total <= kBatch * kThreads) {
        // few: as one run, all of a thread's loads in flight together (256 experts, 65536
        // rows in 24 groups: 22.1 -> 20.5 us; 8192 rows in 4: 9.1 -> 7.0)
        int c[kBatch], e = threadIdx.x % (E + 2);
        const int turn = kThreads % (E + 2);
#pragma unroll
        for (int j = 0; j < kBatch; ++j) {
            const int i = threadIdx.x + j * kThreads;
            c[j] = 0;
            if (j * kThreads < total && i < total)   // the first the same for all: a branch
                c[j] = part[i];
        }
#pragma unroll
        for (int j = 0; j < kBatch; ++j)
            if (j * kThreads < total) {
                if (c[j])
                    atomicAdd(&count[e], c[j]);
                e += turn;
                e -= e >= E + 2 ? E + 2 : 0;
            }
    } else {
        // many: a column of a wave's chunks to a lane (one group of 64 experts, 64
        // chunks: 6.4 us, as one run 7.4)
        for (int e = lane_id(); e < E + 2; e += kWave) {
            int c = 0;
#pragma unroll 8
            for (int i = threadIdx.x / kWave; i < cn; i += kThreads / kWave)
                c += part[(long)i * (E + 2) + e];
            atomicAdd(&count[e], c);
        }
    }
    __syncthreads();
    const int n = count[E], bad = count[E + 1];
    const double per = n ? (double)E / ((double)K * (double)n) : 0.0;
    for (int e = threadIdx.x; e < E; e += kThreads) {
        f1[e] = bad ? __builtin_nanf("") : (float)((double)count[e] * per - 1.0);
        if (at.leads)
            a.counts[(long)at.group * E + e] = count[e];
    }
    if (at.leads && threadIdx.x == 0)
        w.rows[at.group] = n;
    __syncthreads();
    double dots = 0.0, squares = 0.0;
    rows.run(f1, n, dots, squares);
    const double v = group_sums<kThreads>(dots, squares, room);
    if (threadIdx.x < 2)
        w.sum_part[2 * chunk + threadIdx.x] = v;
}

// The losses of one group; the counts of a group without rows.
__global__ __launch_bounds__(kThreads) void balance_sum_kernel(BalanceArgs a, BalanceWs w, Sizes z)
{
    __shared__ double room[2 * kThreads / kWave];
    const int g = blockIdx.x, E = a.E, T = a.T;
    int b = 0, e = T;
    if (a.offsets) {
        b = clamp_row(a.offsets[g], T);
        e = max(clamp_row(a.offsets[g + 1], T), b);
    }
    const int c0 = chunk0_of(g, b, z.grad_bits);
    // the cap holds for offsets in order; out of order it keeps the reads in bounds
    const int cn = min(chunks_of(e - b, z.grad_bits), (int)w.grad_chunks - c0);
    double dots = 0.0, squares = 0.0;
    for (int i = threadIdx.x; i < cn; i += kThreads) {
        dots += w.sum_part[2l * (c0 + i)];
        squares += w.sum_part[2l * (c0 + i) + 1];
    }
    const double v = group_sums<kThreads>(dots, squares, room);
    if (threadIdx.x < 2) {
        const int n = cn > 0 ? w.rows[g] : 0;
        (threadIdx.x ? a.zloss : a.loss)[g] = n ? (float)(v / (double)n) : 0.f;
    }
    if (cn <= 0)
        for (int i = threadIdx.x; i < E; i += kThreads)
            a.counts[(long)g * E + i] = 0;
}

// A small group as a whole.
template <typename T, int R, bool Wide>
__global__ __launch_bounds__(kSmall) void balance_small_kernel(BalanceArgs a)
{
    extern __shared__ int dyn[];   // [E + 2] counts, [E] f - 1
    __shared__ double room[2 * kSmall / kWave];
    const int g = blockIdx.x, E = a.E;
    if (g >= a.G) {
        fill_rows<T, kSmall>(a, g - a.G);
        return;
    }
    const int first = a.offsets ? clamp_row(a.offsets[g], a.T) : 0;
    const int last = a.offsets ? max(clamp_row(a.offsets[g + 1], a.T), first) : a.T;
    GroupRows<T, kSmall, R, Wide> rows(a, first, last);
    int *count = dyn;
    float *f1 = (float *)(dyn + E + 2);
    for (int e = threadIdx.x; e < E + 2; e += kSmall)
        count[e] = 0;
    __syncthreads();
    count_rows<kSmall>(a, first, last, count);
    __syncthreads();
    const int n = count[E], bad = count[E + 1];
    const double per = n ? (double)E / ((double)a.K * (double)n) : 0.0;
    for (int e = threadIdx.x; e < E; e += kSmall) {
        f1[e] = bad ? __builtin_nanf("") : (float)((double)count[e] * per - 1.0);
        a.counts[(long)g * E + e] = count[e];
    }
    __syncthreads();
    double dots = 0.0, squares = 0.0;
    rows.run(f1, n, dots, squares);
    const double v = group_sums<kSmall>(dots, squares, room);
    if (threadIdx.x < 2)
        (threadIdx.x ? a.zloss : a.loss)[g] = n ? (float)(v / (double)n) : 0.f;
}

// 128 to 256 chunks to count (64 to 128 of twice the threads took 7.0 us for 65536 x 8
// choices, these 5.3) and 1024 to 2048 for the rest, where there are rows enough for
// at least 256 and 16 a chunk.
Sizes sizes_of(int T)
{
    auto bits = [](int v) { return 31 - __builtin_clz((unsigned)v); };
    return Sizes{std::max(8, bits(T / 128 + 1)), std::max(4, bits(T / 1024 + 1))};
}

// One work-group per group where that is little work even if a single group
// holds every row.
bool small(int T, int E) { return T <= 1024 && (long)T * E <= 65536; }

template <typename T, int R, bool Wide>
void run(const BalanceArgs &a, const BalanceWs &w, hipStream_t st)
{
    const int fillers = a.fill && a.offsets && a.dlogits ? kFillers : 0;
    const size_t room = (size_t)(2 * a.E + 2) * 4;
    if (small(a.T, a.E))
        hipLaunchKernelGGL((balance_small_kernel<T, R, Wide>), dim3(a.G + fillers), dim3(kSmall),
                           room, st, a);
    else
        hipLaunchKernelGGL((balance_kernel<T, R, Wide>), grid_of(w.grad_chunks + fillers),
                           dim3(kThreads), room, st, a, w, sizes_of(a.T));
}

template <typename T, int R>
void run_width(const BalanceArgs &a, const BalanceWs &w, hipStream_t st)
{
    constexpr int W = Values<T, R, true>::W;
    const bool wide = a.E % W == 0 && a.ld % W == 0 && (!a.dlogits || a.dld % W == 0) &&
                      ((uintptr_t)a.logits | (uintptr_t)a.dlogits) % (W * sizeof(T)) == 0;
    if (wide)
        run<T, R, true>(a, w, st);
    else
        run<T, R, false>(a, w, st);
}

template <typename T> void run_rows(const BalanceArgs &a, const BalanceWs &w, hipStream_t st)
{
    if (a.E <= kLanes)
        run_width<T, 1>(a, w, st);
    else if (a.E <= 2 * kLanes)
        run_width<T, 2>(a, w, st);
    else if (a.E <= 4 * kLanes)
        run_width<T, 4>(a, w, st);
    else if (a.E <= 8 * kLanes)
        run_width<T, 8>(a, w, st);
    else if (a.E <= 16 * kLanes)
        run_width<T, 16>(a, w, st);
    else if (a.E <= 32 * kLanes)
        run_width<T, 32>(a, w, st);
    else
        run_width<T, 64>(a, w, st);
}

}  // namespace

// chunk numbers go up to the last group's: G - 1 + floor(T / size)
long balance_count_chunks(int T, int G) { return (T >> sizes_of(T).count_bits) + (long)G; }
long balance_grad_chunks(int T, int G) { return (T >> sizes_of(T).grad_bits) + (long)G; }

hipError_t launch_balance(const BalanceArgs &a, const BalanceWs &w, hipStream_t st)
{
    const bool one = small(a.T, a.E);
    if (!one)
        hipLaunchKernelGGL(count_kernel, grid_of(w.count_chunks), dim3(kCounters),
                           (size_t)(a.E + 2) * 4, st, a, w, sizes_of(a.T));
    if (a.dtype == 1)
        run_rows<uint16_t>(a, w, st);
    else
        run_rows<float>(a, w, st);
    if (!one)
        hipLaunchKernelGGL(balance_sum_kernel, dim3(a.G), dim3(kThreads), 0, st, a, w,
                           sizes_of(a.T));
    return hipGetLastError();
}

}  // namespace sk
