// token_loss.hip -- log-probabilities of tokens and the losses on them: one
// log-sum-exp per row of logits and the gradient coefficient x (1[label] - softmax).
//
// With q = softmax(s z) of a row, y its label and M, S the row maximum and the
// sum of 2^((z_v - M) c), c = s log2(e):
//     logp = s (z_y - M) - ln S,        lse = s M + ln S,
//     d logp / d z_v = s (1[v = y] - q_v),   q_v = 2^((z_v - M) c) / S.
// Sums and maxima are fp32 over non-negative terms; the logarithm and every
// per-row scalar behind it (ratios, clipping decisions, KL terms) are fp64 in
// one wave, so a ratio is clipped by the same decision as in 64 bits unless it
// is within a few 1e-7 of the border.
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
    float A, M, add;   // out_v = A 2^((z_v - M) c) + add [v = label]
    int zero;          // the row's gradient is zero
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
    float c;
    LogpOut out;
    PolicyArgs pol;
    const float *G;   // dL/dlogp of a row; a row of 0 is not read
};

__device__ __forceinline__ RowState row_state(const LabelArgs &a, long t, int label)
{
    const RowState r = row_state(a.p, t, a.r.T, label);
    return r == kUsed && a.G && a.G[t] == 0.f ? kZeroRow : r;
}

// --- the scalar phase: fp64, one wave, the same in every lane

struct LogpMode {
    static constexpr bool kGradient = false;
    __device__ __forceinline__ static RowScalars row(const LabelArgs &a, long t, float M, float S,
                                                     float zy, bool writes)
    {
        const double lnS = log((double)S), s = a.r.scale;
        const bool none = S == 0.f;
        if (writes && lane_id() == 0) {
            if (a.out.logp)
                a.out.logp[t] = none ? 0.f : (float)(((double)zy - (double)M) * s - lnS);
            if (a.out.lse)
                a.out.lse[t] = none ? -kInf : (float)((double)M * s + lnS);
            if (a.out.stat)
                a.out.stat[t] = make_float2(M, S);
        }
        return RowScalars{0.f, 0.f, 0.f, 1};
    }
    __device__ __forceinline__ static void unused(const LabelArgs &a, long t)
    {
        if (a.out.logp)
            a.out.logp[t] = 0.f;
        if (a.out.lse)
            a.out.lse[t] = 0.f;
        if (a.out.stat)
            a.out.stat[t] = make_float2(0.f, 0.f);
    }
};

// The gradient alone, of given dL/dlogp.
struct BackwardMode {
    static constexpr bool kGradient = true;
    __device__ __forceinline__ static RowScalars row(const LabelArgs &a, long t, float M, float S,
                                                     float zy, bool)
    {
        const double add = (double)a.G[t] * a.r.scale;
        const bool none = S == 0.f;
        // a label beyond the row has no log-probability: NaN, like its loss
        const float A = zy == zy ? (float)(-add / (double)S) : __builtin_nanf("");
        return RowScalars{A, M, (float)add, none};
    }
    __device__ __forceinline__ static void unused(const LabelArgs &, long) {}
};

struct PolicyMode {
    static constexpr bool kGradient = true;
    __device__ __forceinline__ static RowScalars row(const LabelArgs &a, long t, float M, float S,
                                                     float zy, bool writes)
    {
        const PolicyArgs &q = a.pol;
        const float2 info = q.info[t];
        const bool none = S == 0.f;
        const double s = a.r.scale, w = info.x, adv = info.y;
        const double logp = ((double)zy - (double)M) * s - log((double)S);
        const double ratio = exp(logp - (double)q.old[t]);
        const bool above = adv > 0.0 && ratio > q.hi;
        const bool below = adv < 0.0 && ratio < q.lo;
        const double gain = (above ? q.hi : below ? q.lo : ratio) * adv;
        double slope = above || below ? 0.0 : -ratio * adv;   // d(-gain)/d logp
        double kl = 0.0;
        if (q.ref) {
            const double gap = (double)q.ref[t] - logp, em = expm1(gap);
            kl = isinf(em) ? em : em - gap;   // a label of probability 0: infinite
            slope -= q.kl * em;
        }
        if (writes && lane_id() == 0) {
            if (q.logp)
                q.logp[t] = none ? 0.f : (float)logp;
            q.term[t] = none ? make_float2(0.f, 0.f)
                             : make_float2((float)(w * (q.kl * kl - gain)),
                                           (float)(w * kl));
        }
        const double add = slope * w * s;
        return RowScalars{(float)(-add / (double)S), M, (float)add, none};
    }
    __device__ __forceinline__ static void unused(const LabelArgs &a, long t)
    {
        if (a.pol.logp)
            a.pol.logp[t] = 0.f;
        a.pol.term[t] = make_float2(0.f, 0.f);
    }
};

// The row's gradient from its scalars; `zy` is the label's logit.
template <typename T, typename Src>
__device__ __forceinline__ void write_gradient(const Src &src, T *out, int label, float zy,
                                               const RowScalars &k, float c)
{
    const Dense d{k.A, k.M, c};
    src.dense(out, d);
    if (src.owner(label) == (int)threadIdx.x)
        Pack<T>::put(out + label, d.at(zy) + k.add);
}

// A work-group per row: statistics, scalars and gradient in one launch.
template <typename T, int NT, typename Src, typename Mode>
__global__ __launch_bounds__(NT) void row_kernel(LabelArgs a)
{
    __shared__ float2 room[NT / kWave];
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
    Src src(row, V, 0, 1);
    const float zy = label < V ? Pack<T>::get(row + label) : __builtin_nanf("");
    src.load();
    float M = -kInf, S = 0.f;
    src.stats(a.c, M, S);
    merge_group<NT>(M, S, a.c, room);
    if (threadIdx.x < kWave) {
        const RowScalars k = Mode::row(a, t, M, S, zy, true);
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
        write_gradient<T>(src, out, label, zy, k, a.c);
}

// Few rows: each over `parts` work-groups.  First launch: partial statistics.
template <typename T> __global__ __launch_bounds__(kSplit) void part_kernel(LabelArgs a)
{
    __shared__ float2 room[kSplit / kWave];
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
    merge_group<kSplit>(m, s, a.c, room);
    if (threadIdx.x == 0) {
        a.w.part[t * a.parts + part] = make_float2(m, s);
        if (part == 0)
            a.w.zlab[t] = label < a.r.V ? Pack<T>::get(row + label) : __builtin_nanf("");
    }
}

// (M, S) of a row from its partial ones, in every lane of the calling wave.
__device__ __forceinline__ void merge_parts(const float2 *part, int parts, float c, float &M,
                                            float &S)
{
    M = -kInf;
    S = 0.f;
    for (int i = lane_id(); i < parts; i += kWave) {
        const float2 p = part[i];
        const float mn = fmaxf(M, p.x), at = shift_of(mn);
        S = S * ex2((M - at) * c) + p.y * ex2((p.x - at) * c);
        M = mn;
    }
    merge_wave(M, S, c);
}

// Second launch: the merged statistics, the scalars (by every part for itself)
// and the part's share of the gradient.  Without a gradient one part is run.
template <typename T, typename Mode>
__global__ __launch_bounds__(kSplit) void join_kernel(LabelArgs a, int run)
{
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
    if (threadIdx.x < kWave) {
        float M, S;
        merge_parts(a.w.part + t * a.parts, a.parts, a.c, M, S);
        const RowScalars k = Mode::row(a, t, M, S, zy, part == 0);
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
    write_gradient<T>(src, out, label, zy, k, a.c);
}

struct GradArgs {
    LogitRows r;
    const int32_t *labels;
    Packed p;
    const float2 *stat;
    const float *G;
    int parts;
    float c;
};

// The gradient of rows whose statistics are known.
template <typename T> __global__ __launch_bounds__(kSplit) void label_grad_kernel(GradArgs a)
{
    const long t = group_index() / a.parts;
    const int part = (int)(group_index() % a.parts), V = a.r.V;
    if (t >= a.r.T)
        return;
    T *out = (T *)a.r.dlogits + t * a.r.dld;
    const int label = a.labels[t];
    const RowState state = row_state(a.p, t, a.r.T, label);
    if (state == kOutside)
        return;
    const float2 k0 = state == kUsed ? a.stat[t] : make_float2(0.f, 0.f);
    const float M = k0.x;
    const double shrink = 1.0 / (double)k0.y;   // softmax = 2^((z - M) c) * shrink
    const bool none = k0.y == 0.f;
    const double add = (state == kUsed ? (double)a.G[t] : 0.0) * a.r.scale;
    if (state == kZeroRow || none) {
        zero_row<T, kSplit>(out, V, part, a.parts);
        return;
    }
    const T *row = (const T *)a.r.logits + t * a.r.ld;
    const Streamed<T, kSplit> src(row, V, part, a.parts);
    const bool mine = src.owner(label) == (int)threadIdx.x;
    const float zy = mine ? Pack<T>::get(row + label) : 0.f;
    // a label beyond the row has no log-probability: NaN, like its loss
    const RowScalars k{label < V ? (float)(-add * shrink) : __builtin_nanf(""), M, (float)add, 0};
    const Dense d{k.A, k.M, a.c};
    src.dense(out, d);
    if (mine)
        Pack<T>::put(out + label, d.at(zy) + k.add);
}

// --- per sequence

constexpr int kSeqThreads = 1024;

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

// Sums of up to three fp64 values over the work-group, in a fixed order.
template <int K> __device__ __forceinline__ void group_sum(double (&v)[K], double *room)
{
    constexpr int waves = kSeqThreads / kWave;
#pragma unroll
    for (int k = 0; k < K; ++k) {
        const double w = wave_sum(v[k]);
        if (lane_id() == 0)
            room[k * waves + threadIdx.x / kWave] = w;
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < K; ++k)
        v[k] = wave_sum(lane_id() < waves ? room[k * waves + lane_id()] : 0.0);
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
        a.info[t] = make_float2((float)w, a.adv[a.adv_per_token ? t : i]);
}

__global__ __launch_bounds__(kSeqThreads) void policy_sum_kernel(Packed p, long T, PolicyArgs a)
{
    __shared__ double room[2 * kSeqThreads / kWave];
    const int i = blockIdx.x;
    const SeqRange r = seq_range(p, i, T);
    double v[2] = {0.0, 0.0};
    for (long t = r.first + threadIdx.x; t < r.last; t += kSeqThreads) {
        const float2 k = a.term[t];
        v[0] += (double)k.x;
        v[1] += (double)k.y;
    }
    group_sum<2>(v, room);
    if (threadIdx.x == 0) {
        a.loss[i] = (float)v[0];
        a.kl_out[i] = (float)v[1];
    }
}

// One pair: the two sequences' summed log-ratios, the loss and its slope.
__global__ __launch_bounds__(kSeqThreads) void preference_kernel(const int32_t *labels, Packed p,
                                                                 long T, PreferenceArgs a)
{
    __shared__ double room[2 * kSeqThreads / kWave];
    const int i = blockIdx.x;
    double ratio[2], share[2];
    for (int h = 0; h < 2; ++h) {
        const SeqRange r = seq_range(p, 2 * i + h, T);
        double v[2] = {0.0, 0.0};
        for (long t = r.first + threadIdx.x; t < r.last; t += kSeqThreads)
            // a row without any finite logit drops out like one without a label
            if (labels[t] >= 0 && a.stat[t].y != 0.f) {
                v[0] += (double)a.logp[t] - (a.ref ? (double)a.ref[t] : 0.0);
                v[1] += 1.0;
            }
        group_sum<2>(v, room);
        share[h] = a.mean ? (v[1] > 0.0 ? 1.0 / v[1] : 0.0) : 1.0;
        ratio[h] = v[0] * share[h];
    }
    const double beta = a.beta, gap = ratio[0] - ratio[1];
    const double w = a.weights ? (double)a.weights[i] : 1.0;
    double loss, slope;
    if (a.kind == 0) {
        // -(1 - eps) log sigma(h) - eps log sigma(-h), h = beta gap
        const double h = beta * gap, eps = a.smoothing;
        const double far = log1p(exp(-fabs(h)));
        loss = (1.0 - eps) * (far + fmax(-h, 0.0)) + eps * (far + fmax(h, 0.0));
        if (h != h)
            loss = h;
        slope = beta * (eps - 1.0 / (1.0 + exp(h)));
    } else {
        const double d = gap - 0.5 / beta;
        loss = d * d;
        slope = 2.0 * d;
    }
    if (threadIdx.x == 0) {
        a.loss[i] = (float)(w * loss);
        a.reward[2 * i] = (float)(beta * ratio[0]);
        a.reward[2 * i + 1] = (float)(beta * ratio[1]);
    }
    for (int h = 0; h < 2; ++h) {
        const SeqRange r = seq_range(p, 2 * i + h, T);
        const float k = (float)((h ? -slope : slope) * w * share[h]);
        for (long t = r.first + threadIdx.x; t < r.last; t += kSeqThreads)
            a.coef[t] = labels[t] >= 0 ? k : 0.f;
    }
}

}  // namespace

// ------------------------------------------------------------------ launches

namespace {

float scale2(double scale) { return (float)(scale * kLog2eD); }

template <typename T, int NT, typename Src, typename Mode>
void run_rows(const LabelArgs &a, hipStream_t st)
{
    hipLaunchKernelGGL((row_kernel<T, NT, Src, Mode>), grid_of(a.r.T), dim3(NT), 0, st, a);
}

template <typename T, typename Mode> void launch_rows(const LabelArgs &a, hipStream_t st)
{
    if (a.parts > 1) {
        hipLaunchKernelGGL((part_kernel<T>), grid_of((long)a.r.T * a.parts), dim3(kSplit), 0, st, a);
        const int run = Mode::kGradient && a.r.dlogits ? a.parts : 1;
        hipLaunchKernelGGL((join_kernel<T, Mode>), grid_of((long)a.r.T * run), dim3(kSplit), 0, st, a, run);
        return;
    }
    run_rows<T, 1024, Streamed<T, 1024>, Mode>(a, st);
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

int token_parts(int T, int V, int dtype)
{
    const long chunks = (long)V * (dtype == 1 ? 2 : 4) / 16;
    // enough work-groups to fill the device, none with less than two chunks a thread
    const long want = T > 0 ? (512 + T - 1) / T : 1, most = chunks / (2 * kSplit);
    return (int)std::max(1l, std::min({want, most, 64l}));
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
    a.c = scale2(r.scale);
    a.out = out;
    return dispatch_rows<LogpMode>(a, st);
}

hipError_t launch_label_grad(const LogitRows &r, const int32_t *labels, const Packed &p,
                             const float2 *stat, const float *G, hipStream_t st)
{
    GradArgs a{r, labels, p, stat, G, grad_parts(r.T, r.V, r.dtype), scale2(r.scale)};
    const dim3 grid = grid_of((long)r.T * a.parts);
    if (r.dtype == 1)
        hipLaunchKernelGGL((label_grad_kernel<uint16_t>), grid, dim3(kSplit), 0, st, a);
    else
        hipLaunchKernelGGL((label_grad_kernel<float>), grid, dim3(kSplit), 0, st, a);
    return hipGetLastError();
}

hipError_t launch_logp_backward(const LogitRows &r, const int32_t *labels, const float *G,
                                const TokenWs &w, hipStream_t st)
{
    LabelArgs a{};
    a.r = r;
    a.labels = labels;
    a.w = w;
    a.parts = token_parts(r.T, r.V, r.dtype);
    a.c = scale2(r.scale);
    a.G = G;
    return dispatch_rows<BackwardMode>(a, st);
}

hipError_t launch_policy(const LogitRows &r, const int32_t *labels, const Packed &p,
                         const PolicyArgs &q, const TokenWs &w, hipStream_t st)
{
    if (r.T > 0) {
        hipLaunchKernelGGL(policy_rows_kernel, dim3(p.n), dim3(kSeqThreads), 0, st, labels, p,
                           (long)r.T, q);
        LabelArgs a{};
        a.r = r;
        a.labels = labels;
        a.p = p;
        a.w = w;
        a.parts = token_parts(r.T, r.V, r.dtype);
        a.c = scale2(r.scale);
        a.pol = q;
        const hipError_t e = dispatch_rows<PolicyMode>(a, st);
        if (e)
            return e;
    }
    hipLaunchKernelGGL(policy_sum_kernel, dim3(p.n), dim3(kSeqThreads), 0, st, p, (long)r.T, q);
    return hipGetLastError();
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
    hipLaunchKernelGGL(preference_kernel, dim3(p.n / 2), dim3(kSeqThreads), 0, st, labels, p,
                       (long)r.T, q);
    if (r.T > 0 && r.dlogits)
        return launch_label_grad(r, labels, p, q.stat, q.coef, st);
    return hipGetLastError();
}

}  // namespace sk
