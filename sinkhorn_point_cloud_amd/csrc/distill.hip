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
// The teacher's probabilities are fp64 numbers from fp32 exponentials (off by 2^-23
// and 2^-24 of the exponent): fp64 ones for K entries lengthen the one wave's work
// that the row's others wait for.
//
// What bounds it: HBM.  A list of 275 entries or more leaves no room for 9 chunks a
// thread in LDS, and a row of more than 256 KB is then read twice (2048 x 151936 bf16
// with 512 entries: 312 us).
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
    double *p;    // [K]
    int *head;    // [NT] first entry whose element the thread owns, or -1
    int *mark;    // [NT] bit i: an entry lies in the thread's i-th chunk (modulo 32)
    int *next;    // [K]
    int *token;   // [K]
    float *u;     // [K] the teacher's logit
    float *own;   // [K] the gradient at entry k's token
    float *z;     // [K]
    __device__ __forceinline__ List(void *room, int NT, int K)
        : p((double *)room), head((int *)(p + K)), mark(head + NT), next(mark + NT),
          token(next + K), u((float *)(token + K)), own(u + K), z(own + K)
    {
    }
};
size_t list_bytes(int NT, int K) { return (size_t)(2 * NT + 7 * K) * 4; }

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
    // one wave
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
    // the whole list into shared memory; z(k, token): the student's logit there
    template <typename Z>
    __device__ __forceinline__ void list(const Args &a, long t, const List &l, Z &&z) const
    {
        const int K = a.d.K;
        auto put = [&](int k, int token, float logit) {
            l.token[k] = token;
            l.u[k] = logit;
            l.z[k] = z(k, token);
        };
#pragma unroll
        for (int j = 0; j < n; ++j) {
            const int k = lane_id() + j * kWave;
            if (j * kWave < K && k < K)   // the first the same for the wave: a branch
                put(k, v[j], u[j]);
        }
        for (int k = lane_id() + n * kWave; k < K; k += kWave)
            put(k, a.d.index[t * K + k], a.d.teacher[t * K + k]);
    }
};

// f(k, token, logit) for every entry of this lane
template <typename F> __device__ __forceinline__ void each(const List &l, int K, F &&f)
{
    for (int k = lane_id(); k < K; k += kWave)
        f(k, l.token[k], l.u[k]);
}

// One wave: the teacher's probabilities into the list, in fp64 from fp32
// exponentials e_k of the differences to the largest logit: e_k / (1 + rest), the
// rest without one maximum, so that a probability near 1 is as near to it as it
// should be.  Against a given log-sum-exp they are 1 + expm1.
__device__ __forceinline__ Teacher teacher_side(const Args &a, long t, const List &l)
{
    const int V = a.r.V, K = a.d.K;
    float top = -kInf;
    int bad = 0;
    each(l, K, [&](int, int v, float u) {
        if (v >= 0) {
            bad |= v >= V || !(u < kInf);
            top = fmaxf(top, u);
        }
    });
    top = max_wave(top);
    Teacher r;
    r.bad = __any(bad);
    r.any = top != -kInf;
    if (a.d.teacher_lse) {
        r.U = (double)a.d.teacher_lse[t];
        double C = 0.0;
        each(l, K, [&](int k, int v, float u) {
            const float g = (float)((double)u * a.r.scale - r.U);
            const double p = !r.any || v < 0   ? 0.0
                             : fabsf(g) < 1.f ? 1.0 + (double)expm1_of(g)
                                              : (double)ex2(g * kLog2e);
            l.p[k] = p;
            C += p;
        });
        r.C = sum_wave(C);
    } else {
        float rest = 0.f;
        int tops = 0;
        each(l, K, [&](int k, int v, float u) {
            const float e = r.any && v >= 0 ? a.c.pow(u - top) : 0.f;
            l.p[k] = (double)e;
            if (r.any && v >= 0 && u == top)
                ++tops;
            else
                rest += e;
        });
        const double others = sum_wave((double)rest) + (double)(wave_sum(tops) - 1);
        r.U = (double)top * a.r.scale + ln_sum(others);
        const double over = r.any ? 1.0 / (1.0 + others) : 0.0;
        each(l, K, [&](int k, int, float) { l.p[k] *= over; });
        r.C = r.any ? 1.0 : 0.0;
    }
    return r;
}

struct RowScalars {
    Coefficient a;
    float M;   // out_v = a 2^((z_v - M) c) for tokens that are not in the list
    int zero;
};

// One wave: hands the entries to the threads that own their elements.  Returns
// whether a token stands in the list more than once.
template <typename Src>
__device__ __forceinline__ bool link(const List &l, const Src &src, int K)
{
    bool twice = false;
    for (int first = 0; first < K; first += kWave) {
        const int k = first + lane_id();
        int v = -1, before = -1;
        if (k < K) {
            v = l.token[k];
            // without probability: the dense value is the entry's own (a list padded with
            // one token and -inf is no list of duplicates)
            const int who = l.p[k] != 0.0 ? src.owner(v) : -1;
            if (who >= 0) {
                before = atomicExch(&l.head[who], k);
                l.next[k] = before;
                atomicOr(&l.mark[who], 1 << (src.turn(v) & 31));
            }
        }
        // the walk, and what follows it, reads other lanes' entries
        rows::wave_fence();
        // every pair of a linked list's entries is met once
        for (int j = before; j >= 0; j = l.next[j])
            twice |= l.token[j] == v;
    }
    return __any(twice);
}

// One wave, once the row's (M, R) and the list are there: loss, coefficients and
// the gradient at the list's tokens, add (C q - p).
__device__ __forceinline__ RowScalars student_side(const Args &a, long t, const List &l,
                                                   const Teacher &r, bool twice,
                                                   float M, double R, bool writes)
{
    const int lane = lane_id(), K = a.d.K;
    const double inv = a.r.scale, tau = 1.0 / inv;
    const double w = a.d.weights ? (double)a.d.weights[t] : 1.0;
    const double nan = __builtin_nan("");
    const double add = w * tau, over = r.bad ? nan : r.C / row_sum(M, R);
    // log p_k - log q_k = (u_k - (z_k - M)) / tau - (U - ln(1 + R)): fp64, for it
    // is small where the two agree
    const double apart = r.U - row_ln(M, R);
    double sum = 0.0;
    each(l, K, [&](int k, int, float u) {
        const double p = l.p[k];
        if (p != 0.0)
            sum += p * (((double)u - ((double)l.z[k] - (double)M)) * inv - apart);
        double P = p;
        if (twice) {
            // all of the token's entries, in list order: the same for each of them
            P = 0.0;
            for (int j = 0; j < K; ++j)
                P += l.token[j] == l.token[k] ? l.p[j] : 0.0;
        }
        l.own[k] = (float)(add * (over * (double)a.c.pow(l.z[k] - M) - P));
    });
    sum = sum_wave(sum);
    const bool none = row_empty(M, R) || (!r.any && !r.bad);
    if (writes && lane == 0)
        a.d.loss[t] = none ? 0.f : (float)(r.bad ? nan : w * tau * tau * sum);
    return RowScalars{coefficient(add * over), M, none};
}

// The entries that this thread owns, as values of its gradient.
struct ListTerms {
    const List &l;
    int first;    // the thread's first entry
    int mark;

    __device__ __forceinline__ explicit ListTerms(const List &list)
        : l(list), first(list.head[threadIdx.x]), mark(list.mark[threadIdx.x])
    {
    }
    template <int n> __device__ __forceinline__ void chunk(int i, int at, float (&x)[n]) const
    {
        if (mark >> (i & 31) & 1)
            for (int k = first; k >= 0; k = l.next[k]) {
                const int off = l.token[k] - at;
                const float own = l.own[k];
#pragma unroll
                for (int j = 0; j < n; ++j)
                    x[j] = j == off ? own : x[j];
            }
    }
    __device__ __forceinline__ float edge(int v, float y) const
    {
        for (int k = first; k >= 0; k = l.next[k])
            y = l.token[k] == v ? l.own[k] : y;
        return y;
    }
};

__device__ __forceinline__ bool dropped(const Args &a, long t)
{
    return a.d.weights && a.d.weights[t] == 0.f;
}

template <typename T, int NT, typename Src>
__global__ __launch_bounds__(NT, Src::waves) void distill_kernel(Args a)
{
    extern __shared__ u32x4 chunks[];   // [Src::lds_chunks], then the list
    __shared__ RowPart room[NT / kWave];
    __shared__ RowScalars scal;
    const long t = group_index();
    if (t >= a.r.T)
        return;
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
    const List l(chunks + Src::lds_chunks, NT, K);
    l.head[threadIdx.x] = -1;
    l.mark[threadIdx.x] = 0;
    __syncthreads();
    const T *row = (const T *)a.r.logits + t * a.r.ld;
    Src src(row, V, 0, 1, chunks);
    Teacher r{};
    bool twice = false;
    Ahead ahead;
    if (threadIdx.x < kWave)
        ahead.load(a, t);
    src.load();
    if (threadIdx.x < kWave) {
        ahead.list(a, t, l, [&](int, int v) {
            return v >= 0 && v < V ? Pack<T>::get(row + v) : 0.f;
        });
        r = teacher_side(a, t, l);
        if (grad)
            twice = link(l, src, K);
    }
    float M = -kInf, rest = 0.f;
    src.stats(a.c, M, rest);
    const double R = merge_group<NT>(M, rest, a.c, room);
    if (threadIdx.x < kWave) {
        const RowScalars k = student_side(a, t, l, r, twice, M, R, true);
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
    src.dense(out, Dense{k.a.A, k.M, a.c.near, k.a.up}, ListTerms(l));
}

// Few rows: partial statistics, and the student's logits at the list's tokens
// (the second launch may write its gradient over the logits).
template <typename T> __global__ __launch_bounds__(kSplit) void distill_part_kernel(Args a)
{
    __shared__ RowPart room[kSplit / kWave];
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
    const double R = merge_group<kSplit>(m, s, a.c, room);
    if (threadIdx.x == 0)
        a.w.part[t * a.parts + part] = RowPart{R, m};
}

template <typename T> __global__ __launch_bounds__(kSplit) void distill_join_kernel(Args a, int run)
{
    extern __shared__ u32x4 chunks[];   // the list
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
    const List l(chunks, kSplit, K);
    l.head[threadIdx.x] = -1;
    l.mark[threadIdx.x] = 0;
    __syncthreads();
    const Streamed<T, kSplit> src((const T *)a.r.logits + t * a.r.ld, V, part, run);
    if (threadIdx.x < kWave) {
        Ahead ahead;
        ahead.load(a, t);
        ahead.list(a, t, l, [&](int k, int) { return a.d.zk[t * K + k]; });
        const Teacher r = teacher_side(a, t, l);
        const bool twice = grad && link(l, src, K);
        float M;
        const double R = merge_parts(a.w.part + t * a.parts, a.parts, a.c, M);
        const RowScalars k = student_side(a, t, l, r, twice, M, R, part == 0);
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
    src.dense(out, Dense{k.a.A, k.M, a.c.near, k.a.up}, ListTerms(l));
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
    // up to 256 rows have a compute unit each (128 of 64 KB with 20 entries: 10.8 us at
    // 64 registers a thread, 9.0 at 128)
    with_source<T>(a.r.V, list_bytes(1024, a.d.K), a.r.T <= 256, run);
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
