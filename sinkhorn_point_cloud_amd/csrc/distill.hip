// distill.hip -- distillation from a teacher's top logits: the divergence of a
// student's softmax from a teacher's distribution on K tokens, and its gradient.
//
// Per row, at temperature tau, with the teacher's logits u_k at tokens i_k, the
// student's softmax q over the whole row and a row weight w:
//     p_k  = exp(u_k / tau - U),    U = LSE_k(u_k / tau), or the teacher's own
//                                   log-sum-exp over its whole vocabulary,
//     loss = w tau^2 sum_k p_k (log p_k - log q_{i_k}),
//     dloss/dz_v = w tau (C q_v - sum_{k: i_k = v} p_k),   C = sum_k p_k.
// A token may stand in the list twice; its terms add.  The gradient is a
// multiple of the row's exponentials with K elements written again, so the
// plan of the row kernels holds: one read of the row, one write of its
// gradient.  The teacher's side (K values) is worked out by one wave while the
// row's loads are in flight.
//
// What bounds it: HBM.
#include "rows.h"
#include "token_loss.h"

namespace sk {
namespace {

using namespace rows;

constexpr int kSplit = 256;

struct Args {
    LogitRows r;
    DistillArgs d;
    TokenWs w;
    int parts;
    Scale c;
};

// The list of a row in shared memory: entry k's token, probability and the
// student's logit there, and the entries of each owner thread as a linked list.
struct List {
    int *head;   // [NT] first entry whose element the thread owns, or -1
    int *mark;   // [NT] bit i: an entry lies in the thread's i-th chunk (modulo 32)
    int *next;   // [K]
    int *token;  // [K]
    float *p;    // [K]
    float *take; // [K] what the gradient takes away for entry k, see link()
    float *z;    // [K]
    __device__ __forceinline__ List(int *room, int NT, int K)
        : head(room), mark(room + NT), next(mark + NT), token(next + K), p((float *)(token + K)),
          take(p + K), z(take + K)
    {
    }
};
size_t list_bytes(int NT, int K) { return (size_t)(2 * NT + 5 * K) * 4; }

struct Teacher {
    double C, U;   // sum of p, log-sum-exp
    bool any, bad;
};

// The first entries of a row's list, asked for ahead of the row itself: loads
// return in order, so the list's work can begin while the row is on its way.
struct Ahead {
    static constexpr int n = 4;   // 256 entries
    int v[n];
    float u[n];
    __device__ __forceinline__ void load(const Args &a, long t)
    {
        const int K = a.d.K;
#pragma unroll
        for (int j = 0; j < n; ++j) {
            const int k = lane_id() + j * kWave;
            v[j] = -1;
            u[j] = 0.f;
            if (j * kWave < K && k < K) {
                v[j] = a.d.index[t * K + k];
                u[j] = a.d.teacher[t * K + k];
            }
        }
    }
    // f(k, token, logit) for every entry of this lane
    template <typename F> __device__ __forceinline__ void each(const Args &a, long t, F &&f) const
    {
        const int K = a.d.K;
#pragma unroll
        for (int j = 0; j < n; ++j) {
            const int k = lane_id() + j * kWave;
            if (j * kWave < K && k < K)   // the first the same for the wave: a branch
                f(k, v[j], u[j]);
        }
        for (int k = lane_id() + n * kWave; k < K; k += kWave)
            f(k, a.d.index[t * K + k], a.d.teacher[t * K + k]);
    }
};

// One wave: the teacher's probabilities into the list, as fp32 exponentials of
// the differences to the largest logit, or to the given log-sum-exp (fp64: the
// two may be far from 0 and near each other).
__device__ __forceinline__ Teacher teacher_side(const Args &a, long t, const Ahead &in,
                                                const List &l)
{
    const int V = a.r.V;
    float top = -kInf;
    int bad = 0;
    in.each(a, t, [&](int k, int v, float u) {
        l.token[k] = v;
        if (v >= 0) {
            bad |= v >= V || u != u;
            top = fmaxf(top, u);
        }
    });
    top = max_wave(top);
    Teacher r;
    r.bad = __any(bad);
    r.any = top != -kInf;
    float C = 0.f;
    if (a.d.teacher_lse) {
        const double c = a.r.scale * kLog2eD;   // log2(e) / tau
        r.U = (double)a.d.teacher_lse[t];
        const double less = r.U * kLog2eD;
        in.each(a, t, [&](int k, int v, float u) {
            const float p = r.any && v >= 0 ? ex2((float)((double)u * c - less)) : 0.f;
            l.p[k] = p;
            C += p;
        });
    } else {
        float s = 0.f;
        in.each(a, t, [&](int k, int v, float u) {
            const float e = r.any && v >= 0 ? a.c.pow(u - top) : 0.f;
            l.p[k] = e;
            s += e;
        });
        s = sum_wave(s);
        r.U = (double)top * a.r.scale + ln_of(s);
        const float over = 1.f / s;
        in.each(a, t, [&](int k, int, float) {
            const float p = r.any ? l.p[k] * over : 0.f;
            l.p[k] = p;
            C += p;
        });
    }
    r.C = (double)sum_wave(C);
    return r;
}

struct RowScalars {
    float A, M, sub;   // out_v = A 2^((z_v - M) c) - sub sum_{k: i_k = v} p_k
    int zero;
};

// One wave, once the row's (M, S) and the list are there: loss and coefficients.
__device__ __forceinline__ RowScalars student_side(const Args &a, long t, const Ahead &in,
                                                   const List &l, const Teacher &r, float M,
                                                   float S, bool writes)
{
    const int lane = lane_id();
    const double inv = a.r.scale, tau = 1.0 / inv;
    const double w = a.d.weights ? (double)a.d.weights[t] : 1.0;
    // log p_k - log q_k = (u_k - (z_k - M)) / tau - (U - ln S): fp64, for it is
    // small where the two agree
    const double apart = r.U - ln_of(S);
    double sum = 0.0;
    in.each(a, t, [&](int k, int, float u) {
        const double p = (double)l.p[k];
        if (p != 0.0)
            sum += p * (((double)u - ((double)l.z[k] - (double)M)) * inv - apart);
    });
    sum = sum_wave(sum);
    const bool none = S == 0.f || (!r.any && !r.bad);
    const double nan = __builtin_nan("");
    if (writes && lane == 0)
        a.d.loss[t] = none ? 0.f : (float)(r.bad ? nan : w * tau * tau * sum);
    const double add = w * tau;
    return RowScalars{(float)(r.bad ? nan : add * r.C / (double)S), M, (float)add, none};
}

// One wave: hands the entries to the threads that own their elements.  Of a
// token's several entries the first takes away all of it, summed in list order,
// whatever order the linked list has.
template <int NT, typename Src>
__device__ __forceinline__ void link(const List &l, const Src &src, int K)
{
    bool twice = false;
    for (int k = lane_id(); k < K; k += kWave) {
        const int v = l.token[k];
        const int who = src.owner(v);
        l.take[k] = l.p[k];
        if (who >= 0) {
            const int before = atomicExch(&l.head[who], k);
            l.next[k] = before;
            atomicOr(&l.mark[who], 1 << (src.turn(v) & 31));
            // every pair of a list's entries is met once
            for (int j = before; j >= 0; j = l.next[j])
                twice |= l.token[j] == v;
        }
    }
    if (__any(twice))
        for (int k = lane_id(); k < K; k += kWave) {
            const int v = l.token[k];
            float sum = 0.f;
            bool first = true;
            for (int j = 0; j < K; ++j)
                if (l.token[j] == v) {
                    first &= j >= k;
                    sum += l.p[j];
                }
            l.take[k] = first ? sum : 0.f;
        }
}

// The entries that this thread owns, as terms of its gradient values.
struct ListTerms {
    const List &l;
    int first;    // the thread's first entry
    int mark;
    float sub;    // -sub take_k at token k

    __device__ __forceinline__ ListTerms(const List &list, float sub)
        : l(list), first(list.head[threadIdx.x]), mark(list.mark[threadIdx.x]), sub(sub)
    {
    }
    template <int n> __device__ __forceinline__ void chunk(int i, int at, float (&x)[n]) const
    {
        if (mark >> (i & 31) & 1)
            for (int k = first; k >= 0; k = l.next[k]) {
                const int off = l.token[k] - at;
                const float s = sub * l.take[k];
#pragma unroll
                for (int j = 0; j < n; ++j)
                    x[j] -= j == off ? s : 0.f;
            }
    }
    __device__ __forceinline__ float edge(int v) const
    {
        float s = 0.f;
        for (int k = first; k >= 0; k = l.next[k])
            s -= l.token[k] == v ? sub * l.take[k] : 0.f;
        return s;
    }
};

__device__ __forceinline__ bool dropped(const Args &a, long t)
{
    return a.d.weights && a.d.weights[t] == 0.f;
}

template <typename T, int NT, typename Src>
__global__ __launch_bounds__(NT) void distill_kernel(Args a)
{
    extern __shared__ u32x4 chunks[];   // [Src::lds_chunks], then the list
    __shared__ float2 room[NT / kWave];
    __shared__ RowScalars scal;
    const long t = group_index();
    if (t >= a.r.T)
        return;
    int *dyn = (int *)(chunks + Src::lds_chunks);
    const int V = a.r.V, K = a.d.K;
    T *out = (T *)a.r.dlogits + t * a.r.dld;
    const bool grad = a.r.dlogits;
    if (dropped(a, t)) {
        if (threadIdx.x == 0)
            a.d.loss[t] = 0.f;
        if (grad)
            zero_row<T, NT>(out, V, 0, 1);
        return;
    }
    const List l(dyn, NT, K);
    l.head[threadIdx.x] = -1;
    l.mark[threadIdx.x] = 0;
    __syncthreads();
    const T *row = (const T *)a.r.logits + t * a.r.ld;
    Src src(row, V, 0, 1, chunks);
    Teacher r{};
    Ahead ahead;
    if (threadIdx.x < kWave)
        ahead.load(a, t);
    src.load();
    if (threadIdx.x < kWave) {
        ahead.each(a, t, [&](int k, int v, float) {
            l.z[k] = v >= 0 && v < V ? Pack<T>::get(row + v) : 0.f;
        });
        r = teacher_side(a, t, ahead, l);
        if (grad)
            link<NT>(l, src, K);
    }
    float M = -kInf, S = 0.f;
    src.stats(a.c, M, S);
    merge_group<NT>(M, S, a.c, room);
    if (threadIdx.x < kWave) {
        const RowScalars k = student_side(a, t, ahead, l, r, M, S, true);
        if (threadIdx.x == 0)
            scal = k;
    }
    if (!grad)
        return;
    __syncthreads();
    const RowScalars k = scal;
    if (k.zero) {
        zero_row<T, NT>(out, V, 0, 1);
        return;
    }
    src.dense(out, Dense{k.A, k.M, a.c.hi}, ListTerms(l, k.sub));
}

// Few rows: partial statistics, and the student's logits at the list's tokens
// (the second launch may write its gradient over the logits).
template <typename T> __global__ __launch_bounds__(kSplit) void distill_part_kernel(Args a)
{
    __shared__ float2 room[kSplit / kWave];
    const long t = group_index() / a.parts;
    const int part = (int)(group_index() % a.parts), K = a.d.K, V = a.r.V;
    if (t >= a.r.T || dropped(a, t))
        return;
    const T *row = (const T *)a.r.logits + t * a.r.ld;
    if (part == a.parts - 1)
        for (int k = threadIdx.x; k < K; k += kSplit) {
            const int v = a.d.index[t * K + k];
            a.d.zk[t * K + k] = v >= 0 && v < V ? Pack<T>::get(row + v) : 0.f;
        }
    Streamed<T, kSplit> src(row, V, part, a.parts);
    float m = -kInf, s = 0.f;
    src.stats(a.c, m, s);
    merge_group<kSplit>(m, s, a.c, room);
    if (threadIdx.x == 0)
        a.w.part[t * a.parts + part] = make_float2(m, s);
}

template <typename T> __global__ __launch_bounds__(kSplit) void distill_join_kernel(Args a, int run)
{
    extern __shared__ int dyn[];
    __shared__ RowScalars scal;
    const long t = group_index() / run;
    const int part = (int)(group_index() % run), V = a.r.V, K = a.d.K;
    if (t >= a.r.T)
        return;
    T *out = (T *)a.r.dlogits + t * a.r.dld;
    const bool grad = a.r.dlogits;
    if (dropped(a, t)) {
        if (threadIdx.x == 0 && part == 0)
            a.d.loss[t] = 0.f;
        if (grad)
            zero_row<T, kSplit>(out, V, part, run);
        return;
    }
    const List l(dyn, kSplit, K);
    l.head[threadIdx.x] = -1;
    l.mark[threadIdx.x] = 0;
    __syncthreads();
    const Streamed<T, kSplit> src((const T *)a.r.logits + t * a.r.ld, V, part, run);
    if (threadIdx.x < kWave) {
        Ahead ahead;
        ahead.load(a, t);
        const Teacher r = teacher_side(a, t, ahead, l);
        for (int k = lane_id(); k < K; k += kWave)
            l.z[k] = a.d.zk[t * K + k];
        if (grad)
            link<kSplit>(l, src, K);
        float M = -kInf, S = 0.f;
        const float2 *p = a.w.part + t * a.parts;
        for (int i = lane_id(); i < a.parts; i += kWave) {
            const float mn = fmaxf(M, p[i].x), at = shift_of(mn);
            S = S * a.c.pow(M - at) + p[i].y * a.c.pow(p[i].x - at);
            M = mn;
        }
        merge_wave(M, S, a.c);
        const RowScalars k = student_side(a, t, ahead, l, r, M, S, part == 0);
        if (threadIdx.x == 0)
            scal = k;
    }
    if (!grad)
        return;
    __syncthreads();
    const RowScalars k = scal;
    if (k.zero) {
        zero_row<T, kSplit>(out, V, part, run);
        return;
    }
    src.dense(out, Dense{k.A, k.M, a.c.hi}, ListTerms(l, k.sub));
}

template <typename T> struct RunRows {
    const Args &a;
    hipStream_t st;
    template <int NT, typename Src> void operator()() const
    {
        hipLaunchKernelGGL((distill_kernel<T, NT, Src>), grid_of(a.r.T), dim3(NT),
                           (size_t)Src::lds_chunks * 16 + list_bytes(NT, a.d.K), st, a);
    }
};

template <typename T> void launch_rows(const Args &a, hipStream_t st)
{
    if (a.parts > 1) {
        hipLaunchKernelGGL((distill_part_kernel<T>), grid_of((long)a.r.T * a.parts), dim3(kSplit),
                           0, st, a);
        const int run = a.r.dlogits ? a.parts : 1;
        hipLaunchKernelGGL((distill_join_kernel<T>), grid_of((long)a.r.T * run), dim3(kSplit),
                           list_bytes(kSplit, a.d.K), st, a, run);
        return;
    }
    const RunRows<T> run{a, st};
    // without a gradient too: the loss is then the same to the bit
    with_source<T>(a.r.V, list_bytes(1024, a.d.K), run);
}

}  // namespace

hipError_t launch_distill(const LogitRows &r, const DistillArgs &d, const TokenWs &w,
                          hipStream_t st)
{
    Args a{r, d, w, token_parts(r.T, r.V, r.dtype), scale_of_row(r.scale)};
    if (r.dtype == 1)
        launch_rows<uint16_t>(a, st);
    else
        launch_rows<float>(a, st);
    return hipGetLastError();
}

}  // namespace sk
