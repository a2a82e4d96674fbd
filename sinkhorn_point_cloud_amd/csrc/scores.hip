// scores.hip -- log-probability of a row's label, entropy and top alternatives of
// rows of logits, and the gradient of the first two.
//
// With M the row maximum, e_v = 2^-y_v, y_v = (M - z_v) c, c = s log2(e), R the sum
// of e_v but for one maximum and W the sum of e_v y_v:
//     lse = s M + ln(1 + R),   logp = s (z_y - M) - ln(1 + R),
//     H = ln(1 + R) + D,       D = ln 2 W / (1 + R), the mean of s (M - z),
//     dH/dz_v = s q_v (s (M - z_v) - D),   q_v = e_v / (1 + R).
// W is a sum of terms that are not negative, carried with the running maximum: when
// it rises by g / c, W becomes 2^-g (W + g (R + 1)).  Both parts of H keep their
// relative precision where one token has nearly all of the probability.
//
// The alternatives: of the threads' own maxima, joined to G = 64 for up to 16
// alternatives and to 256 for more, the `top`-th largest is a lower bound of the row's
// `top`-th largest value.  In random order about -G ln(1 - top / G) values lie above
// it: 18 for 16 alternatives, 177 for 128 (and those that differ from it in the lower 16
// bits of their keys alone).  They are listed in shared memory and ranked there by value
// and index, so the order in which they were listed does not matter.  Each thread keeps
// the maxima of up to 8 groups of its chunks, and only groups that reach the bound are
// read again.  A row of which more do not fit (many equal values, or the large ones all
// in one thread's chunks) has its `top`-th entry found by bisection first (4096 rows of
// 131072 bf16 values, each of one value: 940 us).
//
// What bounds it: HBM.  (A row kept in registers for the second look leaves a compute
// unit no other row to load meanwhile: 4096 rows of 131072 bf16 values with 64
// alternatives took 477 us that way, 201 to 216 this way, 4.6 TB/s.)
#include "head.h"
#include "rows.h"

namespace sk {
namespace {

using namespace rows;

constexpr int kSplit = 256;      // threads of a work-group that shares its row with others
constexpr float kFar = 1000.f;   // 2^-kFar is 0: stands for the distance of what has no probability

// --- maximum, rest and weighted distance

struct Stats {
    float m = -kInf, r = 0.f, w = 0.f;
};

// (d c, clipped) for a difference d <= 0, negated
__device__ __forceinline__ float distance(float d, const Scale &c)
{
    return min_of(-fmaf(d, c.hi, d * c.lo), kFar);   // NaN stays
}

// Takes K values in, as absorb() of the losses, with the weighted distance.  Returns
// the largest of them.
template <int K>
__device__ __forceinline__ float absorb(const float (&x)[K], const Scale &c, Stats &s)
{
    float low[K], top = x[0];
#pragma unroll
    for (int i = 1; i < K; ++i) {
        low[i] = min_of(top, x[i]);
        top = max_of(top, x[i]);
    }
    const float mn = max_of(s.m, top), at = shift_of(mn);
    const float g = distance(min_of(s.m, top) - at, c), f = ex2(-g);
    float sum = f, far = f * g;
#pragma unroll
    for (int i = 1; i < K; ++i) {
        const float y = distance(low[i] - at, c), e = ex2(-y);
        sum += e;
        far = fmaf(e, y, far);
    }
    const bool rises = top > s.m;
    s.w = rises ? fmaf(f, fmaf(g, s.r, s.w), far) : s.w + far;
    s.r = fmaf(s.r, rises ? f : 1.f, sum);
    s.m = mn;
    return top;
}

// A part's (r, w) from its own maximum to the common one `top`.
template <typename F>
__device__ __forceinline__ void shift(F &r, F &w, F f, F g, bool holds)
{
    // its own maximum becomes an ordinary term, but for the one that is left out
    w = holds ? w : f * fma(g, r + (F)1, w);
    r = holds ? r : fma(r, f, f);
}

__device__ __forceinline__ ScorePart merge_lanes(float m, double r, double w, const Scale &c)
{
    const float top = max_wave(m);
    const float d = m - shift_of(top);
    const double y = -(double)d * ((double)c.hi + (double)c.lo);
    const bool far = y >= (double)kFar;   // its 2^-y counts as 0, as an fp32 one is
    const double g = far ? (double)kFar : y;
    const bool holds = __ffsll(__ballot(m == top)) - 1 == lane_id();
    shift(r, w, far ? 0.0 : exp2_fine(-g), g, holds);
    return ScorePart{sum_wave(r), sum_wave(w), top};
}

// Of the whole work-group, in its first wave.  `room`: one entry per wave.  One barrier.
template <int NT>
__device__ __forceinline__ ScorePart merge_group(const Stats &s, const Scale &c, ScorePart *room)
{
    const float top = max_wave(s.m);
    const float g = distance(s.m - shift_of(top), c), f = ex2(-g);
    const bool holds = __ffsll(__ballot(s.m == top)) - 1 == lane_id();
    float r = s.r, w = s.w;
    shift(r, w, f, g, holds);
    ScorePart p{sum_wave((double)r), sum_wave((double)w), top};
    if constexpr (NT > kWave) {
        constexpr int waves = NT / kWave;
        if (lane_id() == 0)
            room[threadIdx.x / kWave] = p;
        __syncthreads();
        if (threadIdx.x < kWave) {
            const ScorePart v = lane_id() < waves ? room[lane_id()] : ScorePart{0.0, 0.0, -kInf};
            p = merge_lanes(v.m, v.r, v.w, c);
        }
    }
    return p;
}

__device__ __forceinline__ ScorePart merge_parts(const ScorePart *part, int parts, const Scale &c)
{
    const ScorePart v = lane_id() < parts ? part[lane_id()] : ScorePart{0.0, 0.0, -kInf};
    return merge_lanes(v.m, v.r, v.w, c);
}

// --- the alternatives

// Keys in the order of the values: -0 as 0, NaN above +inf.
__device__ __forceinline__ uint32_t key_of(float x)
{
    const uint32_t b = __float_as_uint(x + 0.f);
    return x != x ? 0xFFFFFFFFu : b & 0x80000000u ? ~b : b | 0x80000000u;
}
constexpr uint32_t kNoKey = 0x007FFFFFu;   // of -inf, which is no alternative
__device__ __forceinline__ float value_of(uint32_t key)
{
    return key == 0xFFFFFFFFu ? __builtin_nanf("")
                              : __uint_as_float(key & 0x80000000u ? key ^ 0x80000000u : ~key);
}
// Value and index in one: the order of alternatives.  0: none.  (Values that stand for
// none, behind a row's end, may come with an index beyond its bits.)
constexpr int kIndexBits = 24;
constexpr uint32_t kIndexMask = (1u << kIndexBits) - 1;
__device__ __forceinline__ uint64_t entry_of(uint32_t key, int v)
{
    return (uint64_t)key << kIndexBits | ((kIndexMask - (uint32_t)v) & kIndexMask);
}
__device__ __forceinline__ uint32_t key_in(uint64_t entry) { return (uint32_t)(entry >> kIndexBits); }
__device__ __forceinline__ int index_in(uint64_t entry)
{
    return (int)(kIndexMask - ((uint32_t)entry & kIndexMask));
}

template <int NT> struct ListRoom {
    static constexpr int room = NT == kWave ? 256 : 1024;   // values that can be listed
    uint32_t keys[NT], border;
    uint64_t entry[room + 8];
    int count, wave[NT / kWave];
    unsigned long long any, all;
    uint16_t flag[room];   // groups of values that reach the border
    int flags;
};

// The lower 16 bits cleared of the `top`-th largest of P x 64 maxima, each over some of
// the NT threads' keys (0 if there are not as many): by bisection, two bits at a time, in
// one wave; every lane of it has the result.
template <int NT, int P> __device__ __forceinline__ uint32_t nth_key(const uint32_t *keys, int top)
{
    uint32_t k[P], found = 0;
#pragma unroll
    for (int i = 0; i < P; ++i) {
        k[i] = keys[i * kWave + lane_id()];
#pragma unroll
        for (int j = P; j < NT / kWave; j += P)
            k[i] = max(k[i], keys[(i + j) * kWave + lane_id()]);
    }
#pragma unroll
    for (int bit = 30; bit >= 16; bit -= 2) {
        int n[3] = {0, 0, 0};
#pragma unroll
        for (int q = 0; q < 3; ++q)
#pragma unroll
            for (int i = 0; i < P; ++i)
                n[q] += __popcll(__ballot(k[i] >= (found | (uint32_t)(q + 1) << bit)));
        found |= (uint32_t)((n[0] >= top) + (n[1] >= top) + (n[2] >= top)) << bit;
    }
    return found;
}

// Sum of a count over the work-group, in every thread.  Two barriers.
template <int NT> __device__ __forceinline__ int group_count(int n, int *wave)
{
    n = wave_sum(n);
    if constexpr (NT == kWave)
        return n;
    __syncthreads();
    if (lane_id() == 0)
        wave[threadIdx.x / kWave] = n;
    __syncthreads();
    n = 0;
#pragma unroll
    for (int i = 0; i < NT / kWave; ++i)
        n += wave[i];
    return n;
}

// Places in a list of `count` for the lanes of a wave that want one: one atomic a wave.
// (One a lane, in a loop over the values of a group: 8192 rows of 8192 bf16 values with
// 20 alternatives 53 us, of which the list 18.)
__device__ __forceinline__ int take_place(int &count, bool wanted)
{
    const uint64_t mask = __ballot(wanted);
    if (!mask)
        return 0;
    const int first = __builtin_ctzll(mask);
    int at = 0;
    if (lane_id() == first)
        at = atomicAdd(&count, (int)__popcll(mask));
    at = __builtin_amdgcn_readlane(at, first);
    return at + (int)__builtin_amdgcn_mbcnt_hi((uint32_t)(mask >> 32),
                                               __builtin_amdgcn_mbcnt_lo((uint32_t)mask, 0));
}
// Appends what is wanted to the list; nothing is written beyond its room.
template <int NT>
__device__ __forceinline__ void append(ListRoom<NT> &room, bool wanted, uint64_t entry)
{
    const int at = take_place(room.count, wanted);
    if (wanted && at < ListRoom<NT>::room)
        room.entry[at] = entry;
}

// This thread's largest key; then, behind a barrier, the border of the list, by one wave.
// 64 maxima for up to 16 alternatives, 256 for more: at 128 alternatives some 177 values
// are listed, with the maxima of 1024 threads it would be 137, and the bisection is as
// much shorter.
template <int NT> __device__ __forceinline__ void set_key(ListRoom<NT> &room, uint32_t most)
{
    room.keys[threadIdx.x] = most;
    if (threadIdx.x == 0)
        room.count = room.flags = 0;
}
template <int NT> __device__ __forceinline__ void set_border(ListRoom<NT> &room, int top)
{
    constexpr int P = NT < 256 ? NT / kWave : 4;
    uint32_t k = 0;
    if (top <= 16)
        k = nth_key<NT, 1>(room.keys, top);
    else if (top <= P * kWave)
        k = nth_key<NT, P>(room.keys, top);
    if (lane_id() == 0)
        room.border = max(k, kNoKey + 1);
}

// Lists the alternatives of a source: `list(border)` appends the values of this thread at
// or above the border, `scan(most, f)` calls f(key, index) for every value of this thread
// in the first `most` of `batches` pieces, which come in the order of indices.  set_key()
// came before, a barrier, set_border() and another.  Leaves at most its room's entries in
// room.entry, the `top` largest among them (fewer where there are fewer).
// Returns how many; the list is there for every thread.
template <int NT, typename List, typename Scan>
__device__ __forceinline__ int list_top(ListRoom<NT> &room, int top, int batches, List &&list, Scan &&scan)
{
    const uint32_t border = room.border;
    list(border);
    __syncthreads();
    const int n = room.count;
    if (n <= ListRoom<NT>::room)
        return n;
    // more than fit: the `top`-th entry itself, a bit at a time (entries differ), from the
    // first bit on in which any two at or above the border do
    if (threadIdx.x == 0) {
        room.any = 0;
        room.all = ~0ull;
    }
    __syncthreads();
    unsigned long long any = 0, all = ~0ull;
    scan(batches, [&](uint32_t key, int v) {
        if (key >= border) {
            any |= entry_of(key, v);
            all &= entry_of(key, v);
        }
    });
    atomicOr(&room.any, any);
    atomicAnd(&room.all, all);
    __syncthreads();
    const uint64_t differ = room.any ^ room.all;
    const int first = differ ? 63 - __builtin_clzll(differ) : -1;
    // where all have one value, the first `top` of them will do
    int most = batches;
    if (first < kIndexBits)
        for (most = 1; most < batches; most *= 2) {
            int c = 0;
            scan(most, [&](uint32_t key, int) { c += key >= border; });
            if (group_count<NT>(c, room.wave) >= top)
                break;
        }
    most = min(most, batches);
    uint64_t least = first < 0 ? room.all : room.all >> first >> 1 << first << 1;
#pragma unroll 1
    for (int bit = first; bit >= 0; --bit) {
        const uint64_t with = least | 1ull << bit;
        int c = 0;
        scan(most, [&](uint32_t key, int v) { c += entry_of(key, v) >= with; });
        if (group_count<NT>(c, room.wave) >= top)
            least = with;
    }
    __syncthreads();
    if (threadIdx.x == 0)
        room.count = 0;
    __syncthreads();
    scan(most, [&](uint32_t key, int v) {
        const uint64_t e = entry_of(key, v);
        append(room, e >= least, e);
    });
    __syncthreads();
    return room.count;
}

// Calls put(place, entry) for the largest `top` of the n listed ones, each by the
// thread that has counted how many are larger.  One barrier.
template <int NT, typename Put>
__device__ __forceinline__ void rank_list(ListRoom<NT> &room, int n, int top, Put &&put)
{
    // zeros behind the list, which count for none: eight at a time
    if (threadIdx.x < 8)
        room.entry[n + threadIdx.x] = 0;
    __syncthreads();
    for (int i = threadIdx.x; i < n; i += NT) {
        const uint64_t e = room.entry[i];
        int place = 0;
        for (int j = 0; j < n; j += 8) {
#pragma unroll
            for (int k = 0; k < 8; ++k)
                place += room.entry[j + k] > e;
        }
        if (place < top)
            put(place, e);
    }
}

constexpr int kBatch = 4;    // chunks that a thread asks for together
constexpr int kGroups = 8;   // of batches, a maximum of each

// A row, or a part of one, read from memory: its statistics, and the maxima of groups
// of each thread's chunks.
template <typename T, int NT> struct Reader : Slice<T, NT> {
    using S = Slice<T, NT>;
    static constexpr int n = S::n;
    int batches, per;    // of the longest thread, and in a group
    int turns;           // chunks of a thread in a group: a short row's groups are chunks
    float edge, most[kGroups];

    __device__ __forceinline__ Reader(const T *p, int len, int part, int parts) : S(p, len, part, parts)
    {
        batches = (S::c1 - S::c0 + NT * kBatch - 1) / (NT * kBatch);
        per = (batches + kGroups - 1) / kGroups;
        turns = batches * kBatch <= kGroups ? 1 : per * kBatch;
        edge = S::has_edge(threadIdx.x) ? Pack<T>::get(S::row + S::edge_at(threadIdx.x)) : -kInf;
    }
    // f(first element, values) for the chunks of batch b
    template <typename F> __device__ __forceinline__ void batch(int b, F &&f) const
    {
        const int at = S::c0 + b * NT * kBatch + (int)threadIdx.x;
        u32x4 v[kBatch];
        if (S::c0 + (b + 1) * NT * kBatch <= S::c1) {
#pragma unroll
            for (int j = 0; j < kBatch; ++j)
                v[j] = *S::chunk(at + j * NT);
        } else {
#pragma unroll
            for (int j = 0; j < kBatch; ++j) {
                v[j] = u32x4{Pack<T>::kNone, Pack<T>::kNone, Pack<T>::kNone, Pack<T>::kNone};
                if (at + j * NT < S::c1)
                    v[j] = *S::chunk(at + j * NT);
            }
        }
#pragma unroll
        for (int j = 0; j < kBatch; ++j) {
            float x[n];
            Pack<T>::open(v[j], x);
            f(S::cut.head + (at + j * NT) * n, x);
        }
    }
    __device__ __forceinline__ void stats(const Scale &c, Stats &s)
    {
        if (turns == 1) {
#pragma unroll
            for (int b = 0; b < kGroups / kBatch; ++b) {
                int j = b * kBatch;
                if (b < batches) {
                    batch(b, [&](int, const float (&x)[n]) { most[j++] = absorb<n>(x, c, s); });
                } else {
#pragma unroll
                    for (int k = 0; k < kBatch; ++k)
                        most[j++] = -kInf;
                }
            }
        } else {
#pragma unroll
            for (int g = 0; g < kGroups; ++g) {
                float m = -kInf;
                for (int b = g * per; b < min((g + 1) * per, batches); ++b)
                    batch(b, [&](int, const float (&x)[n]) { m = max_of(m, absorb<n>(x, c, s)); });
                most[g] = m;
            }
        }
        const float x[1] = {edge};
        absorb<1>(x, c, s);
    }
    // f(key, index) for every value of this thread in the first `most` batches, which come
    // in the order of their indices; values of -inf, or none, among them
    template <typename F> __device__ __forceinline__ void scan(int most, F &&f) const
    {
        if (most >= batches || (int)threadIdx.x < S::cut.head)
            f(key_of(edge), S::edge_at(threadIdx.x));
        const int end = (int)min((long)S::c1, S::c0 + (long)most * (NT * kBatch));
#pragma unroll 1
        for (int i = S::c0 + (int)threadIdx.x; i < end; i += NT) {
            float x[n];
            Pack<T>::open(*S::chunk(i), x);
#pragma unroll
            for (int k = 0; k < n; ++k)
                f(key_of(x[k]), S::cut.head + i * n + k);
        }
    }
    // Appends the values at or above the border: first the groups that have any, then
    // their values, dealt to all threads.  More groups than fit count as more values than
    // fit.  For the whole work-group; one barrier.
    __device__ __forceinline__ void list(uint32_t border, ListRoom<NT> &room) const
    {
        append(room, key_of(edge) >= border, entry_of(key_of(edge), S::edge_at(threadIdx.x)));
#pragma unroll
        for (int g = 0; g < kGroups; ++g)
            if (g * turns < batches * kBatch) {
                const bool has = key_of(most[g]) >= border;
                const int at = take_place(room.flags, has);
                if (has && at < ListRoom<NT>::room)
                    room.flag[at] = (uint16_t)(g << 10 | threadIdx.x);
            }
        __syncthreads();
        const int flags = room.flags;
        if (flags > ListRoom<NT>::room) {
            if (threadIdx.x == 0)
                room.count = ListRoom<NT>::room + 1;
            return;
        }
        for (int turn = 0; turn < turns; ++turn)
            for (int i = threadIdx.x; i < flags * n; i += NT) {
                const int f = room.flag[i / n], chunk = S::c0 + ((f >> 10) * turns + turn) * NT + (f & 1023);
                const int v = S::cut.head + chunk * n + i % n;
                const uint32_t key = chunk < S::c1 ? key_of(Pack<T>::get(S::row + v)) : 0u;
                append(room, key >= border, entry_of(key, v));
            }
    }
};

// --- a row's outputs

struct Args {
    ScoreArgs a;
    int parts;
    Scale c;
};

__device__ __forceinline__ bool row_used(const ScoreArgs &a, long t)
{
    return !a.labels || a.labels[t] >= 0;
}

// Writes an alternative, or what marks an empty place.
__device__ __forceinline__ void put_best(const ScoreArgs &a, long t, int place, uint64_t e, double lse)
{
    const int v = index_in(e);
    const float x = value_of(key_in(e));
    a.index[t * a.top + place] = v;
    a.best[t * a.top + place] = (float)((double)x * a.scale - lse);
}
template <int NT> __device__ __forceinline__ void put_empty(const ScoreArgs &a, long t, int from)
{
    for (int i = from + (int)threadIdx.x; i < a.top; i += NT) {
        a.index[t * a.top + i] = -1;
        a.best[t * a.top + i] = -kInf;
    }
}
template <int NT> __device__ __forceinline__ void put_unused(const ScoreArgs &a, long t)
{
    if (threadIdx.x == 0) {
        if (a.logp)
            a.logp[t] = 0.f;
        if (a.lse)
            a.lse[t] = 0.f;
        if (a.entropy)
            a.entropy[t] = 0.f;
    }
    put_empty<NT>(a, t, 0);
}

// One wave, the same in every lane; returns the log-sum-exp.
__device__ __forceinline__ double put_scores(const ScoreArgs &a, long t, const ScorePart &p, float zy)
{
    const bool none = row_empty(p.m, p.r);
    const double ln = row_ln(p.m, p.r), s = a.scale;
    const double lse = (double)p.m * s + ln;
    if (lane_id() == 0) {
        if (a.logp)
            a.logp[t] = none ? 0.f : (float)(((double)zy - (double)p.m) * s - ln);
        if (a.lse)
            a.lse[t] = none ? -kInf : (float)lse;
        if (a.entropy)
            a.entropy[t] = none ? 0.f : (float)(ln + kLn2D * p.w / row_sum(p.m, p.r));
    }
    return lse;
}

template <typename T> __device__ __forceinline__ float logit_at(const ScoreArgs &a, const T *row, long t)
{
    if (!a.labels)
        return 0.f;
    const int y = a.labels[t];
    return y < a.V ? Pack<T>::get(row + y) : __builtin_nanf("");
}

// A work-group per row.
template <typename T, int NT, bool Top> __global__ __launch_bounds__(NT, 8) void score_kernel(Args g)
{
    __shared__ ScorePart room[NT / kWave];
    __shared__ double row_lse;
    const ScoreArgs &a = g.a;
    const long t = group_index();
    if (t >= a.T)
        return;
    if (!row_used(a, t)) {
        put_unused<NT>(a, t);
        return;
    }
    const T *row = (const T *)a.logits + t * a.ld;
    Reader<T, NT> src(row, a.V, 0, 1);
    const float zy = logit_at(a, row, t);
    Stats s;
    src.stats(g.c, s);
    __shared__ typename std::conditional<Top, ListRoom<NT>, int>::type list;
    if constexpr (Top)
        set_key<NT>(list, key_of(s.m));
    const ScorePart p = merge_group<NT>(s, g.c, room);   // a barrier, of more than a wave
    if (threadIdx.x < kWave) {
        const double lse = put_scores(a, t, p, zy);
        if (threadIdx.x == 0)
            row_lse = lse;
    }
    if constexpr (Top) {
        // by the second wave, while the first has the row's statistics to do
        if (NT == kWave || threadIdx.x / kWave == 1)
            set_border<NT>(list, a.top);
        __syncthreads();
        const int n = list_top<NT>(
            list, a.top, src.batches, [&](uint32_t border) { src.list(border, list); },
            [&](int most, auto &&f) { src.scan(most, f); });
        const double lse = row_lse;
        rank_list<NT>(list, n, a.top, [&](int place, uint64_t e) { put_best(a, t, place, e, lse); });
        put_empty<NT>(a, t, n);
    }
}

// Few rows: each over `parts` work-groups.
template <typename T, bool Top> __global__ __launch_bounds__(kSplit, 8) void part_kernel(Args g)
{
    __shared__ ScorePart room[kSplit / kWave];
    const ScoreArgs &a = g.a;
    const long t = group_index() / g.parts;
    const int part = (int)(group_index() % g.parts);
    if (t >= a.T || !row_used(a, t))
        return;
    if (a.dlogits && !(a.grad && a.grad[t] != 0.f) && !(a.grad_entropy && a.grad_entropy[t] != 0.f))
        return;
    const T *row = (const T *)a.logits + t * a.ld;
    Reader<T, kSplit> src(row, a.V, part, g.parts);
    Stats s;
    src.stats(g.c, s);
    __shared__ typename std::conditional<Top, ListRoom<kSplit>, int>::type list;
    if constexpr (Top)
        set_key<kSplit>(list, key_of(s.m));
    const ScorePart p = merge_group<kSplit>(s, g.c, room);
    if (threadIdx.x == 0) {
        a.part[t * g.parts + part] = p;
        if (part == 0)
            a.zlab[t] = logit_at(a, row, t);
    }
    if constexpr (Top) {
        if (threadIdx.x / kWave == 1)
            set_border<kSplit>(list, a.top);
        __syncthreads();
        const int n = list_top<kSplit>(
            list, a.top, src.batches, [&](uint32_t border) { src.list(border, list); },
            [&](int most, auto &&f) { src.scan(most, f); });
        uint64_t *out = a.list + (t * g.parts + part) * a.top;
        rank_list<kSplit>(list, n, a.top, [&](int place, uint64_t e) { out[place] = e; });
        for (int i = n + (int)threadIdx.x; i < a.top; i += kSplit)
            out[i] = 0;
    }
}

// Second launch: outputs from the merged parts.
template <bool Top> __global__ __launch_bounds__(kSplit) void join_kernel(Args g)
{
    __shared__ double row_lse;
    const ScoreArgs &a = g.a;
    const long t = group_index();
    if (t >= a.T)
        return;
    if (!row_used(a, t)) {
        put_unused<kSplit>(a, t);
        return;
    }
    __shared__ typename std::conditional<Top, ListRoom<kSplit>, int>::type list;
    // the parts' alternatives, in the form of values and indices
    const uint64_t *in = Top ? a.list + t * g.parts * a.top : nullptr;
    const int all = g.parts * a.top;
    auto scan = [&](int, auto &&f) {   // one piece
        for (int i = threadIdx.x; i < all; i += kSplit) {
            const uint64_t e = in[i];
            f(key_in(e), index_in(e));
        }
    };
    if constexpr (Top) {
        uint32_t most = 0;
        scan(1, [&](uint32_t key, int) { most = max(most, key); });
        set_key<kSplit>(list, most);
        __syncthreads();
        if (threadIdx.x / kWave == 1)
            set_border<kSplit>(list, a.top);
    }
    if (threadIdx.x < kWave) {
        const double lse = put_scores(a, t, merge_parts(a.part + t * g.parts, g.parts, g.c), a.zlab[t]);
        if (threadIdx.x == 0)
            row_lse = lse;
    }
    if constexpr (Top) {
        __syncthreads();
        const int n = list_top<kSplit>(
            list, a.top, 1,
            [&](uint32_t border) {
                scan(1, [&](uint32_t key, int v) { append(list, key >= border, entry_of(key, v)); });
            },
            scan);
        const double lse = row_lse;
        rank_list<kSplit>(list, n, a.top, [&](int place, uint64_t e) { put_best(a, t, place, e, lse); });
        put_empty<kSplit>(a, t, n);
    }
}

// --- the gradient

// out_v = 2^(up - y_v) (A + B y_v): A = -s (grad + grad_entropy D) / (1 + R) and B =
// s ln 2 grad_entropy / (1 + R), divided by 2^up where they come near fp32's end.
struct DenseScores {
    float A, B, M, c, up;
    __device__ __forceinline__ float at(float x) const
    {
        const float y = fminf((M - x) * c, kFar);
        return ex2(up - y) * fmaf(B, y, A);
    }
};
struct GradScalars {
    DenseScores d;
    float own;   // the label's value
    int zero;
};

__device__ __forceinline__ GradScalars grad_scalars(const Args &g, long t, const ScorePart &p, float zy)
{
    const ScoreArgs &a = g.a;
    const double s = a.scale, S = row_sum(p.m, p.r), D = kLn2D * p.w / S;
    const double gl = a.grad ? (double)a.grad[t] : 0.0;
    const double ge = a.grad_entropy ? (double)a.grad_entropy[t] : 0.0;
    const double away = ((double)p.m - (double)zy) * s;   // the label's distance
    const double logp = -away - row_ln(p.m, p.r);
    double A = -s * (gl + ge * D) / S, B = s * kLn2D * ge / S;
    // a label beyond the row makes its gradient NaN, if there is one
    double own = -s * gl * (double)expm1_of((float)logp);
    if (gl != 0.0 && logp != logp)
        A = __builtin_nan("");
    if (ge != 0.0 && zy != -kInf)
        own += s * ge * exp2_fine(logp * kLog2eD) * (away - D);
    const double most = fmax(fabs(A), fabs(B));
    float up = 0.f;
    if (most > 0x1p64 && most < __builtin_inf()) {
        // what is left stays finite times any distance, and 2^up while the value does
        const int e = __builtin_amdgcn_frexp_exp(most) - 64;
        A = __builtin_amdgcn_ldexp(A, -e);
        B = __builtin_amdgcn_ldexp(B, -e);
        up = (float)e;
    }
    return GradScalars{{(float)A, (float)B, p.m, g.c.near, up}, (float)own, row_empty(p.m, p.r)};
}

__device__ __forceinline__ bool grad_used(const ScoreArgs &a, long t)
{
    return row_used(a, t) &&
           ((a.grad && a.grad[t] != 0.f) || (a.grad_entropy && a.grad_entropy[t] != 0.f));
}
// the label where it has a value of its own
__device__ __forceinline__ OneTerm own_term(const ScoreArgs &a, long t, float own)
{
    return OneTerm{a.grad && a.grad[t] != 0.f ? a.labels[t] : -1, own};
}

template <typename T, int NT, typename Src>
__global__ __launch_bounds__(NT, Src::waves) void score_grad_kernel(Args g)
{
    extern __shared__ u32x4 chunks[];   // [Src::lds_chunks]
    __shared__ ScorePart room[NT / kWave];
    __shared__ GradScalars scal;
    const ScoreArgs &a = g.a;
    const long t = group_index();
    if (t >= a.T)
        return;
    T *out = (T *)a.dlogits + t * a.dld;
    if (!grad_used(a, t)) {
        zero_row<T, NT>(out, a.V, 0, 1);
        return;
    }
    const T *row = (const T *)a.logits + t * a.ld;
    Src src(row, a.V, 0, 1, chunks);
    const float zy = logit_at(a, row, t);
    src.load();
    Stats s;
    const float edge[1] = {src.edge_value()};
    src.template each<true>([&](int, int, const float (&x)[Pack<T>::n]) { absorb<Pack<T>::n>(x, g.c, s); });
    absorb<1>(edge, g.c, s);
    const ScorePart p = merge_group<NT>(s, g.c, room);
    if (threadIdx.x < kWave) {
        const GradScalars k = grad_scalars(g, t, p, zy);
        if (threadIdx.x == 0)
            scal = k;
    }
    __syncthreads();
    const GradScalars k = scal;
    if (k.zero)
        zero_row<T, NT>(out, a.V, 0, 1);
    else
        src.dense(out, k.d, own_term(a, t, k.own));
}

template <typename T> __global__ __launch_bounds__(kSplit) void grad_join_kernel(Args g)
{
    __shared__ GradScalars scal;
    const ScoreArgs &a = g.a;
    const long t = group_index() / g.parts;
    const int part = (int)(group_index() % g.parts);
    if (t >= a.T)
        return;
    T *out = (T *)a.dlogits + t * a.dld;
    if (!grad_used(a, t)) {
        zero_row<T, kSplit>(out, a.V, part, g.parts);
        return;
    }
    if (threadIdx.x < kWave) {
        const GradScalars k =
            grad_scalars(g, t, merge_parts(a.part + t * g.parts, g.parts, g.c), a.zlab[t]);
        if (threadIdx.x == 0)
            scal = k;
    }
    __syncthreads();
    const GradScalars k = scal;
    if (k.zero) {
        zero_row<T, kSplit>(out, a.V, part, g.parts);
        return;
    }
    const Streamed<T, kSplit> src((const T *)a.logits + t * a.ld, a.V, part, g.parts);
    src.dense(out, k.d, own_term(a, t, k.own));
}

// ------------------------------------------------------------------ launches

template <typename T, int NT> void run_rows(const Args &g, hipStream_t st)
{
    if (g.a.top)
        hipLaunchKernelGGL((score_kernel<T, NT, true>), grid_of(g.a.T), dim3(NT), 0, st, g);
    else
        hipLaunchKernelGGL((score_kernel<T, NT, false>), grid_of(g.a.T), dim3(NT), 0, st, g);
}
template <typename T> struct RunScoreGrad {
    const Args &g;
    hipStream_t st;
    template <int NT, typename Src> void operator()() const
    {
        hipLaunchKernelGGL((score_grad_kernel<T, NT, Src>), grid_of(g.a.T), dim3(NT),
                           (size_t)Src::lds_chunks * 16, st, g);
    }
};

template <typename T> hipError_t run_scores(const Args &g, hipStream_t st)
{
    const ScoreArgs &a = g.a;
    if (g.parts > 1) {
        const dim3 all = grid_of((long)a.T * g.parts), rows = grid_of(a.T);
        if (a.top) {
            hipLaunchKernelGGL((part_kernel<T, true>), all, dim3(kSplit), 0, st, g);
            hipLaunchKernelGGL((join_kernel<true>), rows, dim3(kSplit), 0, st, g);
        } else {
            hipLaunchKernelGGL((part_kernel<T, false>), all, dim3(kSplit), 0, st, g);
            hipLaunchKernelGGL((join_kernel<false>), rows, dim3(kSplit), 0, st, g);
        }
    } else {
        // Few rows take more threads each; up to 256 KB, more rows at once on a compute unit
        // load more evenly (8192 rows of 131072 bf16 values with 20 alternatives: 256, 512
        // and 1024 threads 412, 429 and 444 us; longer ones less so: 3000 of 100003 fp32
        // 233, 218 and 203).  Many alternatives need threads for their bound.
        const long bytes = (long)a.V * (long)sizeof(T), few = a.T <= 256 ? 4 : 1;
        if (few * bytes <= 8 << 10 && a.top <= 32)
            run_rows<T, 64>(g, st);
        else if (few * bytes <= 64 << 10)
            run_rows<T, 256>(g, st);
        else if (few * bytes <= 256 << 10)
            run_rows<T, 512>(g, st);
        else
            run_rows<T, 1024>(g, st);
    }
    return hipGetLastError();
}

template <typename T> hipError_t run_scores_backward(const Args &g, hipStream_t st)
{
    const ScoreArgs &a = g.a;
    if (g.parts > 1) {
        const dim3 all = grid_of((long)a.T * g.parts);
        hipLaunchKernelGGL((part_kernel<T, false>), all, dim3(kSplit), 0, st, g);
        hipLaunchKernelGGL((grad_join_kernel<T>), all, dim3(kSplit), 0, st, g);
    } else {
        with_source<T>(a.V, 0, false, RunScoreGrad<T>{g, st});
    }
    return hipGetLastError();
}

}  // namespace

// A row of up to 128 KB is one work-group's; longer ones are split while there are too
// few rows to keep the compute units loading, as for the losses.
int score_parts(int T, int V, int dtype)
{
    const long bytes = (long)V * (dtype == 1 ? 2 : 4), chunks = bytes / 16;
    if (T < 1 || T > 128 || bytes <= 128 << 10)
        return 1;
    return (int)std::min({1024l / T, chunks / (2 * kSplit), 64l});
}

hipError_t launch_scores(const ScoreArgs &a, hipStream_t st)
{
    const Args g{a, score_parts(a.T, a.V, a.dtype), scale_of_row(a.scale)};
    return a.dtype == 1 ? run_scores<uint16_t>(g, st) : run_scores<float>(g, st);
}

hipError_t launch_scores_backward(const ScoreArgs &a, hipStream_t st)
{
    const Args g{a, score_parts(a.T, a.V, a.dtype), scale_of_row(a.scale)};
    return a.dtype == 1 ? run_scores_backward<uint16_t>(g, st) : run_scores_backward<float>(g, st);
}

}  // namespace sk
