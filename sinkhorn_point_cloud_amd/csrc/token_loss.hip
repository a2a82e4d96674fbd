// token_loss.hip -- log-probabilities of tokens and the losses on them: one
// log-sum-exp per row of logits and the gradient coefficient x (1[label] - softmax).
//
// With q = softmax(s z) of a row, y its label, M the row maximum and R the sum
// of e_v = 2^((z_v - M) c), c = s log2(e), but for one maximum:
//     logp = s (z_y - M) - ln(1 + R),        lse = s M + ln(1 + R),
//     d logp / d z_v = -s q_v = -s e_v / (1 + R)  for v other than y,
//                      -s expm1(logp)             for y.
// Exponentials, maxima and a thread's sums are fp32, the sums' joins fp64.  The
// log-probability is put together in fp64 (off by about 1e-8) and so are its
// differences to given ones: a ratio is clipped by the same decision as in 64 bits
// unless it is that near the border.  Ratio and KL term are short fp64 series of
// those differences; the library's double-precision exponential and logarithm,
// several hundred instructions in one wave with the others waiting, cost 2 us a row.
// What the gradient pass takes up for every value (coefficient, maximum) is fp32.
//
// What bounds it: HBM.  A row is read once and its gradient written once.
#include "rows.h"
#include "token_loss.h"

namespace sk {
namespace {

using namespace rows;

constexpr int kSplit = 256;   // threads of a work-group that shares its row with others

// What the scalar phase of a row leaves for its gradient pass.
struct RowScalars {
    Coefficient a;
    float M, own;   // out_v = a 2^((z_v - M) c), `own` for the label
    int zero;       // the row's gradient is zero
};

enum RowState { kOutside, kZeroRow, kUsed };

// The part a row plays: outside every sequence, without a label (or a gradient), or used.
__device__ __forceinline__ RowState row_state(const Packed &p, long t, long T, int label)
{
    if (p.offsets) {
        const long first = min(max((long)p.offsets[0], 0l), T);
        const long last = min(max((long)p.offsets[p.n], 0l), T);
        if (t < first || t >= last)
            return p.fill ? kZeroRow : kOutside;
    }
    return label < 0 ? kZeroRow : kUsed;
}

struct LabelArgs {
    LogitRows r;
    const int32_t *labels;
    Packed p;
    TokenWs w;
    int parts;
    Scale c;
    LogpOut out;
    PolicyArgs pol;
    const float *G;   // dL/dlogp of a row; a row of 0 is not read
    int fold;         // the policy loss finds a row's weight in the row's own work-group
};

struct SeqRange {
    long first, last;
};
__device__ __forceinline__ SeqRange seq_range(const Packed &p, int i, long T)
{
    SeqRange r;
    r.first = min(max((long)p.offsets[i], 0l), T);
    r.last = min(max((long)p.offsets[i + 1], r.first), T);
    return r;
}

// The sequence of a row, of at most kWave of them: as many as end at or before it.
__device__ __forceinline__ int seq_of(const Packed &p, long t)
{
    const bool ends = lane_id() < p.n && (long)p.offsets[lane_id() + 1] <= t;
    return min((int)__popcll(__ballot(ends)), p.n - 1);
}

__device__ __forceinline__ RowState row_state(const LabelArgs &a, long t, int label)
{
    const RowState r = row_state(a.p, t, a.r.T, label);
    return r == kUsed && a.G && a.G[t] == 0.f ? kZeroRow : r;
}

// --- the scalar phase: fp64, one wave, the same in every lane

// add (1[v = label] - q_v).  A NaN log-probability (a label beyond the row)
// makes the whole row NaN.
__device__ __forceinline__ RowScalars coefficients(double add, double logp, float M, double R)
{
    const float own = (float)(-add * (double)expm1_of((float)logp));
    const double a = logp == logp ? -add / row_sum(M, R) : __builtin_nan("");
    return RowScalars{coefficient(a), M, own, row_empty(M, R)};
}

struct LogpMode {
    static constexpr bool kGradient = false;
    struct Row {};
    template <int NT>
    __device__ __forceinline__ static Row begin(const LabelArgs &, long, int *)
    {
        return Row{};
    }
    __device__ __forceinline__ static RowScalars row(const LabelArgs &a, long t, const Row &,
                                                     float M, double R, float zy, bool writes)
    {
        const double lnS = row_ln(M, R), s = a.r.scale;
        const bool none = row_empty(M, R);
        if (writes && lane_id() == 0) {
            if (a.out.logp)
                a.out.logp[t] = none ? 0.f : (float)(((double)zy - (double)M) * s - lnS);
            if (a.out.lse)
                a.out.lse[t] = none ? -kInf : (float)((double)M * s + lnS);
            if (a.out.stat)
                a.out.stat[t] = RowStat{M, (float)R, none ? 0.0 : ((double)zy - (double)M) * s - lnS};
        }
        return RowScalars{{0.f, 0.f}, 0.f, 0.f, 1};
    }
    __device__ __forceinline__ static void unused(const LabelArgs &a, long t)
    {
        if (a.out.logp)
            a.out.logp[t] = 0.f;
        if (a.out.lse)
            a.out.lse[t] = 0.f;
        if (a.out.stat)
            a.out.stat[t] = RowStat{-kInf, 0.f, 0.0};
    }
};

// The gradient alone, of given dL/dlogp.
struct BackwardMode {
    static constexpr bool kGradient = true;
    struct Row {};
    template <int NT>
    __device__ __forceinline__ static Row begin(const LabelArgs &, long, int *)
    {
        return Row{};
    }
    __device__ __forceinline__ static RowScalars row(const LabelArgs &a, long t, const Row &,
                                                     float M, double R, float zy, bool)
    {
        const double logp = ((double)zy - (double)M) * a.r.scale - row_ln(M, R);
        return coefficients((double)a.G[t] * a.r.scale, logp, M, R);
    }
    __device__ __forceinline__ static void unused(const LabelArgs &, long) {}
};

// The KL term e^g - 1 - g and its slope e^g - 1 from g and e = e^g, in fp64 and its
// range: the term is a multiple of e^g for a label that the reference finds likely,
// and after weights it may be an ordinary number where e^g is beyond fp32.  Near 0
// the series, where the difference would cancel (|g| < 0.35: the first term left out,
// 2 g^7/9!, is below 2^-27 of the value, as is beyond it what e, off by 3e-10, leaves).
struct KlTerm {
    double over, slope;
};
__device__ __forceinline__ KlTerm kl_term(double g, double e)
{
    double r = 1.0 / 40320;
    r = fma(r, g, 1.0 / 5040);
    r = fma(r, g, 1.0 / 720);
    r = fma(r, g, 1.0 / 120);
    r = fma(r, g, 1.0 / 24);
    r = fma(r, g, 1.0 / 6);
    r = fma(r, g, 0.5);
    const double near = r * g * g;
    const double far = e == (double)kInf ? e : e - 1.0 - g;   // infinite: a label of probability 0
    return fabs(g) < 0.35 ? KlTerm{near, near + g} : KlTerm{far, e - 1.0};
}

struct PolicyMode {
    static constexpr bool kGradient = true;
    struct Row {
        double w;              // row weight
        float adv, old, ref;   // advantage, given log-probabilities
    };
    // Every thread of the work-group, while the row's loads are in flight: what the
    // scalar phase needs is there when it begins.
    template <int NT>
    __device__ __forceinline__ static Row begin(const LabelArgs &a, long t, int *room)
    {
        const PolicyArgs &q = a.pol;
        const float old = q.old[t], ref = q.ref ? q.ref[t] : 0.f;
        if (!a.fold) {
            const PolicyRow info = q.info[t];
            return Row{info.w, info.adv, old, ref};
        }
        const int lane = lane_id(), i = seq_of(a.p, t);
        double w = q.weights ? (double)q.weights[i] : 1.0;
        if (q.mean) {
            const SeqRange r = seq_range(a.p, i, a.r.T);
            int n = 0;
            for (long k = r.first + threadIdx.x; k < r.last; k += NT)
                n += a.labels[k] >= 0;
            n = wave_sum(n);
            if constexpr (NT > kWave) {
                if (lane == 0)
                    room[threadIdx.x / kWave] = n;
                __syncthreads();
                n = wave_sum(lane < NT / kWave ? room[lane] : 0);
            }
            w = n ? w / (double)n : 0.0;
        }
        return Row{w, q.adv[q.adv_per_token ? t : i], old, ref};
    }
    __device__ __forceinline__ static RowScalars row(const LabelArgs &a, long t, const Row &info,
                                                     float M, double R, float zy, bool writes)
    {
        const PolicyArgs &q = a.pol;
        // without a distribution, or weighted out: no part, whatever the row holds
        const bool empty = row_empty(M, R), none = empty || info.w == 0.0;
        const double s = a.r.scale, w = info.w;
        const float adv = info.adv;
        const double logp = ((double)zy - (double)M) * s - row_ln(M, R);
        // the clipping decision is taken on the log-ratio, in fp64
        const double change = logp - (double)info.old;
        const double gap = (double)info.ref - logp;
        // the ratio's exponential in one half of the lanes, the KL term's in the other
        const double e = exp2_fine((lane_id() < kWave / 2 ? change : gap) * kLog2eD);
        const double ratio = read_lane(e, 0);
        const bool above = adv > 0.f && change > q.log_hi;
        const bool below = adv < 0.f && change < q.log_lo;
        const double gain = (above ? q.hi : below ? q.lo : ratio) * (double)adv;
        double slope = above || below ? 0.0 : -ratio * (double)adv;   // d(-gain)/d logp
        double kl = 0.0, cost = 0.0;
        if (q.ref) {
            const KlTerm k = kl_term(gap, read_lane(e, kWave - 1));
            kl = k.over;
            if (q.kl != 0.0) {   // only reported else, and it may be infinite
                cost = q.kl * kl;
                slope -= q.kl * k.slope;
            }
        }
        if (writes && lane_id() == 0) {
            if (q.logp)
                q.logp[t] = empty ? 0.f : (float)logp;
            q.term[t] = none ? make_double2(0.0, 0.0) : make_double2(w * (cost - gain), w * kl);
        }
        RowScalars k = coefficients(slope * w * s, logp, M, R);
        k.zero = none;
        return k;
    }
    __device__ __forceinline__ static void unused(const LabelArgs &a, long t)
    {
        if (a.pol.logp)
            a.pol.logp[t] = 0.f;
        a.pol.term[t] = make_double2(0.0, 0.0);
    }
};

// A work-group per row: statistics, scalars and gradient in one launch.
template <typename T, int NT, typename Src, typename Mode>
__global__ __launch_bounds__(NT, Src::waves) void row_kernel(LabelArgs a)
{
    extern __shared__ u32x4 chunks[];   // [Src::lds_chunks]
    __shared__ RowPart room[NT / kWave];
    __shared__ int count[NT / kWave];
    __shared__ RowScalars scal;
    const long t = group_index();
    if (t >= a.r.T)
        return;
    const int V = a.r.V;
    T *out = (T *)a.r.dlogits + t * a.r.dld;
    const bool grad = Mode::kGradient && a.r.dlogits;
    const int label = a.labels[t];
    const RowState state = row_state(a, t, label);
    if (state == kOutside)
        return;
    if (state == kZeroRow) {
        if (threadIdx.x == 0)
            Mode::unused(a, t);
        if (grad)
            zero_row<T, NT>(out, V, 0, 1);
        return;
    }
    const T *row = (const T *)a.r.logits + t * a.r.ld;
    Src src(row, V, 0, 1, chunks);
    const float zy = label < V ? Pack<T>::get(row + label) : __builtin_nanf("");
    src.load();
    const typename Mode::Row info = Mode::template begin<NT>(a, t, count);
    float M = -kInf, r = 0.f;
    src.stats(a.c, M, r);
    const double R = merge_group<NT>(M, r, a.c, room);
    if (threadIdx.x < kWave) {
        const RowScalars k = Mode::row(a, t, info, M, R, zy, true);
        if (threadIdx.x == 0)
            scal = k;
    }
    if (!grad)
        return;
    __syncthreads();
    const RowScalars k = scal;
    if (k.zero)
        zero_row<T, NT>(out, V, 0, 1);
    else
        src.dense(out, Dense{k.a.A, k.M, a.c.near, k.a.up}, OneTerm{label, k.own});
}

// Few rows: each over `parts` work-groups.  First launch: partial statistics.
template <typename T> __global__ __launch_bounds__(kSplit) void part_kernel(LabelArgs a)
{
    __shared__ RowPart room[kSplit / kWave];
    const long t = group_index() / a.parts;
    const int part = (int)(group_index() % a.parts);
    if (t >= a.r.T)
        return;
    const int label = a.labels[t];
    if (row_state(a, t, label) != kUsed)
        return;
    const T *row = (const T *)a.r.logits + t * a.r.ld;
    Streamed<T, kSplit> src(row, a.r.V, part, a.parts);
    float m = -kInf, s = 0.f;
    src.stats(a.c, m, s);
    const double R = merge_group<kSplit>(m, s, a.c, room);
    if (threadIdx.x == 0) {
        a.w.part[t * a.parts + part] = RowPart{R, m};
        if (part == 0)
            a.w.zlab[t] = label < a.r.V ? Pack<T>::get(row + label) : __builtin_nanf("");
    }
}

// Second launch: the merged statistics, the scalars (by every part for itself)
// and the part's share of the gradient.  Without a gradient one part is run.
template <typename T, typename Mode>
__global__ __launch_bounds__(kSplit) void join_kernel(LabelArgs a, int run)
{
    __shared__ int count[kSplit / kWave];
    __shared__ RowScalars scal;
    const long t = group_index() / run;
    const int part = (int)(group_index() % run), V = a.r.V;
    if (t >= a.r.T)
        return;
    T *out = (T *)a.r.dlogits + t * a.r.dld;
    const bool grad = Mode::kGradient && a.r.dlogits;
    const int label = a.labels[t];
    const RowState state = row_state(a, t, label);
    if (state == kOutside)
        return;
    if (state == kZeroRow) {
        if (threadIdx.x == 0 && part == 0)
            Mode::unused(a, t);
        if (grad)
            zero_row<T, kSplit>(out, V, part, run);
        return;
    }
    const float zy = a.w.zlab[t];
    const typename Mode::Row info = Mode::template begin<kSplit>(a, t, count);
    if (threadIdx.x < kWave) {
        float M;
        const double R = merge_parts(a.w.part + t * a.parts, a.parts, a.c, M);
        const RowScalars k = Mode::row(a, t, info, M, R, zy, part == 0);
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
    const Streamed<T, kSplit> src((const T *)a.r.logits + t * a.r.ld, V, part, run);
    src.dense(out, Dense{k.a.A, k.M, a.c.near, k.a.up}, OneTerm{label, k.own});
}

// --- per sequence

constexpr int kSeqThreads = 1024;

// Sums of up to three fp64 values over the work-group, in a fixed order.
template <int K> __device__ __forceinline__ void group_sum(double (&v)[K], double *room)
{
    constexpr int waves = kSeqThreads / kWave;
#pragma unroll
    for (int k = 0; k < K; ++k) {
        const double w = sum_wave(v[k]);
        if (lane_id() == 0)
            room[k * waves + threadIdx.x / kWave] = w;
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < K; ++k)
        v[k] = sum_wave(lane_id() < waves ? room[k * waves + lane_id()] : 0.0);
    __syncthreads();
}

// Row weight (the sequence's, over its labels if the mean is asked for) and advantage.
__global__ __launch_bounds__(kSeqThreads) void policy_rows_kernel(const int32_t *labels, Packed p,
                                                                  long T, PolicyArgs a)
{
    __shared__ double room[kSeqThreads / kWave];
    const int i = blockIdx.x;
    const SeqRange r = seq_range(p, i, T);
    double w = a.weights ? (double)a.weights[i] : 1.0;
    if (a.mean) {
        double n[1] = {0.0};
        for (long t = r.first + threadIdx.x; t < r.last; t += kSeqThreads)
            n[0] += labels[t] >= 0 ? 1.0 : 0.0;
        group_sum<1>(n, room);
        w = n[0] > 0.0 ? w / n[0] : 0.0;
    }
    for (long t = r.first + threadIdx.x; t < r.last; t += kSeqThreads)
        a.info[t] = PolicyRow{w, a.adv[a.adv_per_token ? t : i]};
}

__global__ __launch_bounds__(kSeqThreads) void policy_sum_kernel(Packed p, long T, PolicyArgs a)
{
    __shared__ double room[2 * kSeqThreads / kWave];
    const int i = blockIdx.x;
    const SeqRange r = seq_range(p, i, T);
    double v[2] = {0.0, 0.0};
    for (long t = r.first + threadIdx.x; t < r.last; t += kSeqThreads) {
        const double2 k = a.term[t];
        v[0] += k.x;
        v[1] += k.y;
    }
    group_sum<2>(v, room);
    if (threadIdx.x == 0) {
        a.loss[i] = (float)v[0];
        a.kl_out[i] = (float)v[1];
    }
}

// One pair, by a work-group of NT threads: the two sequences' summed log-ratios
// (half of the threads each), the loss (written where asked for) and, left in
// slopes, its derivative by a log-probability of either sequence.  One barrier
// inside; `slopes` is there for every thread behind another.
template <int NT>
__device__ __forceinline__ void pair_slopes(const int32_t *labels, const Packed &p, long T,
                                            const PreferenceArgs &a, int i, bool writes,
                                            double (&room)[2][2][NT / 2 / kWave],
                                            float (&slopes)[2])
{
    constexpr int half = NT / 2, waves = half / kWave;
    const int h = threadIdx.x / half;
    const SeqRange r = seq_range(p, 2 * i + h, T);
    double sum = 0.0;
    int n = 0;
    for (long t = r.first + threadIdx.x % half; t < r.last; t += half)
        // a row without any finite logit drops out like one without a label
        if (labels[t] >= 0 && !row_empty(a.stat[t].M, a.stat[t].R)) {
            sum += a.stat[t].logp - (a.ref ? (double)a.ref[t] : 0.0);
            ++n;
        }
    sum = sum_wave(sum);
    n = wave_sum(n);
    if (lane_id() == 0) {
        room[h][0][threadIdx.x % half / kWave] = sum;
        room[h][1][threadIdx.x % half / kWave] = (double)n;
    }
    __syncthreads();
    if (threadIdx.x >= kWave)
        return;
    double ratio[2], share[2];
    for (int k = 0; k < 2; ++k) {
        const double v = sum_wave(lane_id() < waves ? room[k][0][lane_id()] : 0.0);
        const double c = sum_wave(lane_id() < waves ? room[k][1][lane_id()] : 0.0);
        share[k] = a.mean ? (c > 0.0 ? 1.0 / c : 0.0) : 1.0;
        ratio[k] = v * share[k];
    }
    const double beta = a.beta, gap = ratio[0] - ratio[1];
    const double w = a.weights ? (double)a.weights[i] : 1.0;
    double loss, slope;
    if (a.kind == 0) {
        // -(1 - eps) log sigma(h) - eps log sigma(-h), h = beta gap
        const double x = beta * gap, eps = a.smoothing;
        const double e = exp(-fabs(x)), far = log1p(e);
        // (a side without weight has no part, though it may be infinite)
        loss = eps < 1.0 ? (1.0 - eps) * (far + fmax(-x, 0.0)) : 0.0;
        loss += eps > 0.0 ? eps * (far + fmax(x, 0.0)) : 0.0;
        loss = x != x ? x : loss;
        // sigma(-x)
        slope = beta * (eps - (x > 0.0 ? e : 1.0) / (1.0 + e));
    } else {
        const double d = gap - 0.5 / beta;
        loss = d * d;
        slope = 2.0 * d;
    }
    if (w == 0.0)   // weighted out, whatever its rows hold
        loss = slope = 0.0;
    if (threadIdx.x == 0) {
        if (writes) {
            a.loss[i] = (float)(w * loss);
            a.reward[2 * i] = (float)(beta * ratio[0]);
            a.reward[2 * i + 1] = (float)(beta * ratio[1]);
        }
        slopes[0] = (float)(slope * w * share[0]);
        slopes[1] = (float)(-slope * w * share[1]);
    }
}

__global__ __launch_bounds__(kSeqThreads) void preference_kernel(const int32_t *labels, Packed p,
                                                                 long T, PreferenceArgs a)
{
    constexpr int half = kSeqThreads / 2;
    __shared__ double room[2][2][half / kWave];
    __shared__ float slopes[2];
    const int i = blockIdx.x, h = threadIdx.x / half;
    pair_slopes<kSeqThreads>(labels, p, T, a, i, true, room, slopes);
    __syncthreads();
    const SeqRange r = seq_range(p, 2 * i + h, T);
    const float k = slopes[h];
    for (long t = r.first + threadIdx.x % half; t < r.last; t += half)
        a.coef[t] = labels[t] >= 0 ? k : 0.f;
}

struct GradArgs {
    LogitRows r;
    const int32_t *labels;
    Packed p;
    PreferenceArgs q;
    int parts;
    Scale c;
};

// The gradient of a preference loss's rows, whose statistics are known.  Fold:
// each work-group sums its own row's pair, and as many more work-groups as there
// are pairs write the losses; else their slopes are in q.coef.
template <typename T, bool Fold> __global__ __launch_bounds__(kSplit) void pair_grad_kernel(GradArgs a)
{
    __shared__ double room[2][2][kSplit / 2 / kWave];
    __shared__ float slopes[2];
    // last rows first: they are the ones that the statistics' pass read last, and
    // up to 256 MB of them are still in the last-level cache (8192 x 65536 bf16,
    // half of them scored: 402 -> 394 us for the two passes)
    const long rows = a.r.dlogits ? a.r.T : 0;
    const long t = rows - 1 - group_index() / a.parts;
    const int part = (int)(group_index() % a.parts), V = a.r.V;
    if (t < 0) {
        const long i = group_index() - rows * a.parts;
        if (Fold && i < a.p.n / 2)
            pair_slopes<kSplit>(a.labels, a.p, a.r.T, a.q, (int)i, true, room, slopes);
        return;
    }
    T *out = (T *)a.r.dlogits + t * a.r.dld;
    const int label = a.labels[t];
    const RowState state = row_state(a.p, t, a.r.T, label);
    if (state == kOutside)
        return;
    const RowStat stat = state == kUsed ? a.q.stat[t] : RowStat{-kInf, 0.f, 0.0};
    if (row_empty(stat.M, stat.R)) {
        zero_row<T, kSplit>(out, V, part, a.parts);
        return;
    }
    float G;
    if constexpr (Fold) {
        const int i = seq_of(a.p, t);
        pair_slopes<kSplit>(a.labels, a.p, a.r.T, a.q, i / 2, false, room, slopes);
        __syncthreads();
        G = slopes[i % 2];
    } else {
        G = a.q.coef[t];
    }
    if (G == 0.f) {
        zero_row<T, kSplit>(out, V, part, a.parts);
        return;
    }
    const RowScalars k = coefficients((double)G * a.r.scale, stat.logp, stat.M, stat.R);
    const Streamed<T, kSplit> src((const T *)a.r.logits + t * a.r.ld, V, part, a.parts);
    src.dense(out, Dense{k.a.A, k.M, a.c.near, k.a.up}, OneTerm{label, k.own});
}

}  // namespace

// ------------------------------------------------------------------ launches

namespace {

template <typename T, typename Mode> struct RunRows {
    const LabelArgs &a;
    hipStream_t st;
    template <int NT, typename Src> void operator()() const
    {
        hipLaunchKernelGGL((row_kernel<T, NT, Src, Mode>), grid_of(a.r.T), dim3(NT),
                           (size_t)Src::lds_chunks * 16, st, a);
    }
};

template <typename T, typename Mode> void launch_rows(const LabelArgs &a, hipStream_t st)
{
    if (a.parts > 1) {
        hipLaunchKernelGGL((part_kernel<T>), grid_of((long)a.r.T * a.parts), dim3(kSplit), 0, st,
                           a);
        const int run = Mode::kGradient && a.r.dlogits ? a.parts : 1;
        hipLaunchKernelGGL((join_kernel<T, Mode>), grid_of((long)a.r.T * run), dim3(kSplit), 0,
                           st, a, run);
        return;
    }
    const RunRows<T, Mode> run{a, st};
    // a loss keeps its launch shape without a gradient: the same to the bit
    if constexpr (Mode::kGradient)
        with_source<T>(a.r.V, 0, false, run);
    else
        with_stream<T>(a.r.V, a.r.T, run);
}

template <typename Mode> hipError_t dispatch_rows(const LabelArgs &a, hipStream_t st)
{
    if (a.r.dtype == 1)
        launch_rows<uint16_t, Mode>(a, st);
    else
        launch_rows<float, Mode>(a, st);
    return hipGetLastError();
}

}  // namespace

// What a row needs of its sequence or pair (a count of labels, two sums) is found
// in its own work-group where that is cheap: the sequences are one to a lane, and
// a sequence's rows a few to a thread.  It saves a launch.
static int fold_rows(int T, int n) { return n <= kWave && T <= 2048; }

// Work-groups per row.  A row of up to 128 KB is one work-group's (one launch):
// with few such rows the split saves at most 4 us of the kernels' time (1 row of
// 128 KB: 10.7 against 6.9 us) and costs another launch.  Longer rows are split
// while there are too few to keep the compute units loading (1 row of 256 KB:
// 17.8 against 6.9 us, 64 rows 20.8 against 13.0, 128 rows 23.2 against 20.3, 200
// rows 25.3 against 30.2), into about 1024 work-groups of at least two chunks a
// thread.
int token_parts(int T, int V, int dtype)
{
    const long bytes = (long)V * (dtype == 1 ? 2 : 4), chunks = bytes / 16;
    if (T < 1 || T > 128 || bytes <= 128 << 10)
        return 1;
    return (int)std::min({1024l / T, chunks / (2 * kSplit), 64l});
}

int grad_parts(int T, int V, int dtype)
{
    const long chunks = (long)V * (dtype == 1 ? 2 : 4) / 16;
    return (int)std::max(1l, std::min(chunks / (8 * kSplit), 64l));
}

hipError_t launch_logp(const LogitRows &r, const int32_t *labels, const Packed &p,
                       const TokenWs &w, const LogpOut &out, hipStream_t st)
{
    LabelArgs a{};
    a.r = r;
    a.r.dlogits = nullptr;
    a.labels = labels;
    a.p = p;
    a.w = w;
    a.parts = token_parts(r.T, r.V, r.dtype);
    a.c = scale_of_row(r.scale);
    a.out = out;
    return dispatch_rows<LogpMode>(a, st);
}

hipError_t launch_logp_backward(const LogitRows &r, const int32_t *labels, const float *G,
                                const TokenWs &w, hipStream_t st)
{
    LabelArgs a{};
    a.r = r;
    a.labels = labels;
    a.w = w;
    a.parts = token_parts(r.T, r.V, r.dtype);
    a.c = scale_of_row(r.scale);
    a.G = G;
    return dispatch_rows<BackwardMode>(a, st);
}

hipError_t launch_policy(const LogitRows &r, const int32_t *labels, const Packed &p,
                         const PolicyArgs &q, const TokenWs &w, hipStream_t st)
{
    if (r.T > 0) {
        LabelArgs a{};
        a.fold = fold_rows(r.T, p.n);
        if (!a.fold)
            hipLaunchKernelGGL(policy_rows_kernel, dim3(p.n), dim3(kSeqThreads), 0, st, labels, p,
                               (long)r.T, q);
        a.r = r;
        a.labels = labels;
        a.p = p;
        a.w = w;
        a.parts = token_parts(r.T, r.V, r.dtype);
        a.c = scale_of_row(r.scale);
        a.pol = q;
        const hipError_t e = dispatch_rows<PolicyMode>(a, st);
        if (e)
            return e;
    }
    hipLaunchKernelGGL(policy_sum_kernel, dim3(p.n), dim3(kSeqThreads), 0, st, p, (long)r.T, q);
    return hipGetLastError();
}

template <bool Fold> static void run_pairs(const GradArgs &a, hipStream_t st)
{
    const dim3 grid = grid_of((a.r.dlogits ? (long)a.r.T * a.parts : 0) + (Fold ? a.p.n / 2 : 0));
    if (a.r.dtype == 1)
        hipLaunchKernelGGL((pair_grad_kernel<uint16_t, Fold>), grid, dim3(kSplit), 0, st, a);
    else
        hipLaunchKernelGGL((pair_grad_kernel<float, Fold>), grid, dim3(kSplit), 0, st, a);
}

hipError_t launch_preference(const LogitRows &r, const int32_t *labels, const Packed &p,
                             const PreferenceArgs &q, const TokenWs &w, hipStream_t st)
{
    if (r.T > 0) {
        const hipError_t e =
            launch_logp(r, labels, p, w, LogpOut{q.logp, nullptr, q.stat}, st);
        if (e)
            return e;
    }
    const GradArgs a{r, labels, p, q, grad_parts(r.T, r.V, r.dtype), scale_of_row(r.scale)};
    if (fold_rows(r.T, p.n)) {
        run_pairs<true>(a, st);
    } else {
        hipLaunchKernelGGL(preference_kernel, dim3(p.n / 2), dim3(kSeqThreads), 0, st, labels, p,
                           (long)r.T, q);
        if (r.dlogits && r.T > 0)   // without rows there is no grid to launch
            run_pairs<false>(a, st);
    }
    return hipGetLastError();
}

}  // namespace sk
