// rows.h -- one row of logits as a work-group sees it: 16-byte chunks dealt to
// the threads, the running (maximum, sum) of its exponentials, and the pass
// that writes coefficient x exponential.
//
// A row starts at any address that suits its type.  It is cut into 16-byte
// chunks (4 fp32 or 8 bf16 values), the first on a multiple of 128 bytes (64 for
// a work-group of one wave), and the values before the first and behind the last
// of them, the edge, dealt one to a thread.  A wave's loads and stores then cover
// whole lines: with chunks on multiples of 16 bytes alone, rows of 100003 fp32
// values moved 4% more bytes and took 10% longer (2048 of them 321 against 292
// us).  Chunk c0 + i * threads + t belongs to
// thread t, so that a wave's loads are 1 KB in a run and the thread that owns
// an element is known from its index alone: that thread puts an element's own
// value into the chunk before it stores it.  (Written again behind the dense store,
// each such element is a 2- or 4-byte write to a line on its way to memory: 16384
// rows of 32000 bf16 values with 64 terms took 398 us that way, 367 this way.)
//
// The exponentials are taken in base 2: with c = scale log2(e) and the row
// maximum M, e_v = 2^((x_v - M) c).  The difference is formed first, so a row
// of the type's lowest finite values is an ordinary row.  What is summed is the
// rest R = sum_v e_v - 1, every term but one that is 1: where one value has
// nearly all of the probability, ln(1 + R) and 1 - q keep their relative
// precision.  Values of -inf take no part; a row of nothing else has M = -inf
// and R = 0.  NaN gives a NaN rest.
#pragma once

#include "common.h"
#include "token_loss.h"

#include <algorithm>
#include <math.h>

namespace sk {
namespace rows {

// Four 32-bit words: a chunk as it is loaded and stored.
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef float f32x2 __attribute__((ext_vector_type(2)));

constexpr float kInf = __builtin_inff();

// A grid of `count` work-groups in two dimensions: threads along one dimension
// of a launch have to stay below 2^32, and rows x threads may not.
inline dim3 grid_of(long count)
{
    const long x = std::min(count, 1l << 20);
    return dim3((unsigned)x, (unsigned)((count + x - 1) / x));
}
__device__ __forceinline__ long group_index() { return (long)blockIdx.y * gridDim.x + blockIdx.x; }

template <typename T> struct Pack;
template <> struct Pack<float> {
    static constexpr int n = 4;
    static constexpr uint32_t kNone = 0xFF800000u;   // -inf
    __device__ __forceinline__ static void open(u32x4 v, float (&x)[n])
    {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            x[i] = __uint_as_float(v[i]);
    }
    __device__ __forceinline__ static u32x4 close(const float (&x)[n])
    {
        u32x4 v;
#pragma unroll
        for (int i = 0; i < 4; ++i)
            v[i] = __float_as_uint(x[i]);
        return v;
    }
    __device__ __forceinline__ static float get(const float *p) { return *p; }
    __device__ __forceinline__ static void put(float *p, float x) { *p = x; }
};
template <> struct Pack<uint16_t> {
    static constexpr int n = 8;
    static constexpr uint32_t kNone = 0xFF80FF80u;
    __device__ __forceinline__ static void open(u32x4 v, float (&x)[n])
    {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            x[2 * i] = __uint_as_float(v[i] << 16);
            x[2 * i + 1] = __uint_as_float(v[i] & 0xFFFF0000u);
        }
    }
    // fp32 to bf16, round to nearest even: the gradient's one rounding
    __device__ __forceinline__ static u32x4 close(const float (&x)[n])
    {
        u32x4 v;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const f32x2 two = {x[2 * i], x[2 * i + 1]};
            v[i] = __builtin_bit_cast(uint32_t, __builtin_convertvector(two, bf16x2));
        }
        return v;
    }
    __device__ __forceinline__ static float get(const uint16_t *p) { return bf16_to_float(*p); }
    __device__ __forceinline__ static void put(uint16_t *p, float x)
    {
        *p = __builtin_bit_cast(uint16_t, (__bf16)x);
    }
};

// How one row is cut: `head` values, `chunks` aligned chunks, then the rest;
// `edge` = values before and behind.
struct Cut {
    int head, chunks, edge;
};

// Line: the chunks begin on a multiple of so many bytes.
template <typename T, int Line> __device__ __forceinline__ Cut cut_of(const T *p, int len)
{
    constexpr int n = Pack<T>::n, per = Line / (int)sizeof(T);
    const int off = (int)(((uintptr_t)p & (Line - 1)) / sizeof(T));
    Cut c;
    c.head = off ? min(len, per - off) : 0;
    c.chunks = (len - c.head) / n;
    c.edge = len - c.chunks * n;
    return c;
}

// The part of a row that one work-group of NT threads handles: chunks
// [c0, c1), and the edge if it is the first part.
template <typename T, int NT> struct Slice {
    static constexpr int n = Pack<T>::n;
    // at most kLine - 1 bytes and less than a chunk are edge: NT values at most
    static constexpr int kLine = NT >= 128 ? 128 : 64;
    const T *row;
    Cut cut;
    int c0, c1;
    bool edges;

    __device__ __forceinline__ Slice(const T *p, int len, int part, int parts) : row(p)
    {
        cut = cut_of<T, kLine>(p, len);
        const int per = (cut.chunks + parts - 1) / parts;
        c0 = min(part * per, cut.chunks);
        c1 = min(c0 + per, cut.chunks);
        edges = part == 0;
    }
    __device__ __forceinline__ bool has_edge(int t) const { return edges && t < cut.edge; }
    // element of edge value t
    __device__ __forceinline__ int edge_at(int t) const
    {
        return t < cut.head ? t : t + cut.chunks * n;
    }
    __device__ __forceinline__ const u32x4 *chunk(int c) const
    {
        return reinterpret_cast<const u32x4 *>(row + cut.head) + c;
    }
    // thread that owns element v, or -1 where another part does or the row has no such element
    __device__ __forceinline__ int owner(int v) const
    {
        const int behind = cut.head + cut.chunks * n;
        if (v < 0 || v >= behind + cut.edge - cut.head)
            return -1;
        if (v < cut.head)
            return edges ? v : -1;
        if (v >= behind)
            return edges ? v - cut.chunks * n : -1;
        const int c = (v - cut.head) / n;
        return c >= c0 && c < c1 ? (c - c0) % NT : -1;
    }
    // which of its owner's chunks an owned element of a chunk is in
    __device__ __forceinline__ int turn(int v) const { return ((v - cut.head) / n - c0) / NT; }
};

// What the lanes of a wave wrote to memory before it, all of them see behind it.  (A
// wave's accesses to LDS stay in order; this keeps the compiler from moving them.)
__device__ __forceinline__ void wave_fence()
{
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
}

// Reductions over a wave without LDS: over each row of 16 lanes by lane moves,
// then the four rows through scalar registers, in a fixed order.  All lanes
// active; every lane gets the result.
__device__ __forceinline__ float read_lane(float v, int lane)
{
    return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), lane));
}
__device__ __forceinline__ float sum_wave(float v)
{
    v = row16_sum(v);
    return (read_lane(v, 0) + read_lane(v, 16)) + (read_lane(v, 32) + read_lane(v, 48));
}
__device__ __forceinline__ float max_wave(float v)
{
    v = fmaxf(v, dpp_move<kDppXor1>(v));
    v = fmaxf(v, dpp_move<kDppXor2>(v));
    v = fmaxf(v, dpp_move<kDppHalfMirror>(v));
    v = fmaxf(v, dpp_move<kDppMirror>(v));
    return fmaxf(fmaxf(read_lane(v, 0), read_lane(v, 16)),
                 fmaxf(read_lane(v, 32), read_lane(v, 48)));
}
template <int Ctrl> __device__ __forceinline__ double dpp_move(double v)
{
    return __hiloint2double(
        __builtin_amdgcn_mov_dpp(__double2hiint(v), Ctrl, 0xF, 0xF, true),
        __builtin_amdgcn_mov_dpp(__double2loint(v), Ctrl, 0xF, 0xF, true));
}
__device__ __forceinline__ double read_lane(double v, int lane)
{
    return __hiloint2double(__builtin_amdgcn_readlane(__double2hiint(v), lane),
                            __builtin_amdgcn_readlane(__double2loint(v), lane));
}
__device__ __forceinline__ double sum_wave(double v)
{
    v += dpp_move<kDppXor1>(v);
    v += dpp_move<kDppXor2>(v);
    v += dpp_move<kDppHalfMirror>(v);
    v += dpp_move<kDppMirror>(v);
    return (read_lane(v, 0) + read_lane(v, 16)) + (read_lane(v, 32) + read_lane(v, 48));
}

// c = scale log2(e) in two pieces.  With one, every exponent of a row's sum would
// be off by the same relative 2^-25: an error of one sign, about 1e-7 in each
// log-probability, which adds up over a sequence.  hi lies below c, so that lo is
// positive and a difference of -inf gives -inf in both terms.
struct Scale {
    float hi, lo, near;   // near: c rounded, for what no sum takes up
    __device__ __forceinline__ float pow(float d) const { return ex2(fmaf(d, hi, d * lo)); }
};
inline Scale scale_of_row(double scale)
{
    const double c = scale * kLog2eD;
    float hi = (float)c;
    if ((double)hi >= c)
        hi = nextafterf(hi, 0.f);
    return Scale{hi, (float)(c - (double)hi), (float)c};
}

// Running maximum and rest.  The shift of an empty state is 0, so that no
// difference of two infinities is formed.
__device__ __forceinline__ float shift_of(float m) { return m == -kInf ? 0.f : m; }

// Minimum and maximum that keep a NaN.
__device__ __forceinline__ float min_of(float a, float b)
{
    return __builtin_elementwise_minimum(a, b);
}
__device__ __forceinline__ float max_of(float a, float b)
{
    return __builtin_elementwise_maximum(a, b);
}

// Takes K values into (m, r).  A chain of exchanges leaves the largest in `top`
// and all the others, each once, in `low`.
template <int K>
__device__ __forceinline__ void absorb(const float (&x)[K], const Scale &k, float &m, float &r)
{
    float low[K], top = x[0];
#pragma unroll
    for (int i = 1; i < K; ++i) {
        low[i] = min_of(top, x[i]);
        top = max_of(top, x[i]);
    }
    const float mn = max_of(m, top), at = shift_of(mn);
    const float f = k.pow(min_of(m, top) - at);   // the smaller of the two maxima
    float sum = f;
#pragma unroll
    for (int i = 1; i < K; ++i)
        sum += k.pow(low[i] - at);
    r = fmaf(r, top > m ? f : 1.f, sum);
    m = mn;
}

// (M, R) of a wave from its lanes' own, the same in all of them.  Where many waves
// share a row, sums of 16 lanes are fp32, whose roundings average out; the last
// joins, whose would not, are fp64 here and below.
template <bool Alone>
__device__ __forceinline__ double merge_wave(float &m, float r, const Scale &c)
{
    const float top = max_wave(m), at = shift_of(top);
    const float f = c.pow(m - at);
    // the first lane that has the maximum leaves its 1 out, every other counts
    const bool holds = __ffsll(__ballot(m == top)) - 1 == lane_id();
    m = top;
    r = holds ? r : fmaf(r, f, f);
    if constexpr (Alone)
        return sum_wave((double)r);
    r = row16_sum(r);
    return ((double)read_lane(r, 0) + (double)read_lane(r, 16)) +
           ((double)read_lane(r, 32) + (double)read_lane(r, 48));
}

// 2^y in the range of fp64, off by less than 3e-10 of itself (the first term left
// out, g^9/9!); NaN stays.
__device__ __forceinline__ double exp2_fine(double y)
{
    y = y < -1100.0 ? -1100.0 : y > 1100.0 ? 1100.0 : y;
    const double whole = __builtin_rint(y), g = (y - whole) * kLn2D;   // |g| <= 0.347
    double p = 1.0 / 40320;
    p = fma(p, g, 1.0 / 5040);
    p = fma(p, g, 1.0 / 720);
    p = fma(p, g, 1.0 / 120);
    p = fma(p, g, 1.0 / 24);
    p = fma(p, g, 1.0 / 6);
    p = fma(p, g, 0.5);
    p = fma(p, g, 1.0);
    return __builtin_amdgcn_ldexp(fma(p, g, 1.0), y == y ? (int)whole : 0);
}

// 2^((m - M) c) in fp64: the hardware's exponential, off by up to 2^-23, would be
// most of the error of a sum of few parts.
__device__ __forceinline__ double pow_fine(float d, const Scale &c)
{
    return exp2_fine((double)d * ((double)c.hi + (double)c.lo));
}

// (M, R) from those of up to 64 parts, one to a lane (Lanes: 16, where there are no
// more, in the first lanes).  One wave; every lane gets the result.  (With fp32
// exponentials and sums here a log-probability was off by 5e-8 to 1e-7, the square
// loss of a pair, a small difference of sums, by up to 1e-6 of itself.)
template <int Lanes> __device__ __forceinline__ double merge_parts(float &m, double r, const Scale &c)
{
    const float top = max_wave(m), at = shift_of(top);
    const double f = pow_fine(m - at, c);
    const bool holds = __ffsll(__ballot(m == top)) - 1 == lane_id();
    m = top;
    r = holds ? r : fma(r, f, f);
    if constexpr (Lanes > 16)
        return sum_wave(r);
    r += dpp_move<kDppXor1>(r);
    r += dpp_move<kDppXor2>(r);
    r += dpp_move<kDppHalfMirror>(r);
    r += dpp_move<kDppMirror>(r);
    return read_lane(r, 0);
}
__device__ __forceinline__ double merge_parts(const RowPart *part, int parts, const Scale &c, float &M)
{
    const RowPart p = lane_id() < parts ? part[lane_id()] : RowPart{0.0, -kInf};
    M = p.m;
    return merge_parts<kWave>(M, p.r, c);
}

// (M, R) of the whole work-group, in its first wave.  `room`: one entry per wave.
// One barrier; `room` may be written again only behind another one.
template <int NT>
__device__ __forceinline__ double merge_group(float &m, float r, const Scale &c, RowPart *room)
{
    double R = merge_wave<NT == kWave>(m, r, c);
    if constexpr (NT > kWave) {
        constexpr int waves = NT / kWave;
        static_assert(waves <= 16);
        if (lane_id() == 0)
            room[threadIdx.x / kWave] = RowPart{R, m};
        __syncthreads();
        if (threadIdx.x < kWave) {
            const RowPart v = lane_id() < waves ? room[lane_id()] : RowPart{0.0, -kInf};
            m = v.m;
            R = merge_parts<16>(m, v.r, c);
        }
    }
    return R;
}

// A row without any probability, and the sum 1 + R in fp64: NaN for a maximum of
// +inf, whose terms would be differences of infinities.
__device__ __forceinline__ bool row_empty(float M, double R) { return M == -kInf && R == 0.0; }
__device__ __forceinline__ double row_sum(float M, double R)
{
    return M == kInf ? __builtin_nan("") : 1.0 + R;
}
__device__ __forceinline__ double ln_sum(double R);
__device__ __forceinline__ double row_ln(float M, double R)
{
    return M == kInf ? __builtin_nan("") : ln_sum(R);
}

// ln(1 + R) to 2^-44 of itself: 2 artanh(t), t = R / (2 + R), or for larger R the
// same for the sum's mantissa m between sqrt(1/2) and sqrt(2), t = (m - 1) /
// (m + 1).  |t| <= 0.172: the first term left out, t^17/17, is below 2^-44 t.
// (The library's logarithm, with its tables of extra precision, took several
// times as long while the row's other waves waited.)
__device__ __forceinline__ double ln_sum(double R)
{
    double e = 0.0, a = R, b = 2.0 + a;
    if (R >= 0.4140625) {
        const double s = 1.0 + a;
        double m = __builtin_amdgcn_frexp_mant(s);
        int k = __builtin_amdgcn_frexp_exp(s);
        if (m < 0.7071067811865476) {
            m *= 2.0;
            --k;
        }
        e = (double)k;
        a = m - 1.0;
        b = m + 1.0;
    }
    const double t = a / b, q = t * t;
    double p = 1.0 / 15;
    p = fma(p, q, 1.0 / 13);
    p = fma(p, q, 1.0 / 11);
    p = fma(p, q, 1.0 / 9);
    p = fma(p, q, 1.0 / 7);
    p = fma(p, q, 1.0 / 5);
    p = fma(p, q, 1.0 / 3);
    return fma(e, kLn2D, 2.0 * fma(p * q, t, t));
}

// e^g - 1 to fp32 precision, relative also near 0 (|g| < 1: the first term left
// out, g^12/12!, is below 2^-27 of the value)
__device__ __forceinline__ float expm1_of(float g)
{
    if (!(fabsf(g) < 1.f))
        return ex2(g * kLog2e) - 1.f;
    float r = 1.f / 39916800.f;
    r = fmaf(r, g, 1.f / 3628800.f);
    r = fmaf(r, g, 1.f / 362880.f);
    r = fmaf(r, g, 1.f / 40320.f);
    r = fmaf(r, g, 1.f / 5040.f);
    r = fmaf(r, g, 1.f / 720.f);
    r = fmaf(r, g, 1.f / 120.f);
    r = fmaf(r, g, 1.f / 24.f);
    r = fmaf(r, g, 1.f / 6.f);
    r = fmaf(r, g, 0.5f);
    return fmaf(r * g, g, g);
}

// coefficient x exponential of one row, out_v = A 2^((x_v - M) c + up) (or another
// at(x) of a caller's), but for the elements that have a value of their own.  Those
// are a `Terms` with
//     chunk(i, first, x): sets them in a thread's i-th chunk, whose first element is `first`,
//     edge(v, y):         the value of element v of the edge, y if it has none.
// `up` is 0 but for a coefficient beyond fp32, of which A is then the mantissa: the
// coefficient is no output, and times a probability of 0 it is 0.
struct Coefficient {
    float A, up;
};
__device__ __forceinline__ Coefficient coefficient(double a)
{
    if (fabs(a) > 3.4028234663852886e38 && fabs(a) < __builtin_inf())
        return Coefficient{(float)__builtin_amdgcn_frexp_mant(a),
                           (float)__builtin_amdgcn_frexp_exp(a)};
    return Coefficient{(float)a, 0.f};
}
struct Dense {
    float A, M, c, up;
    __device__ __forceinline__ float at(float x) const { return A * ex2(fmaf(x - M, c, up)); }
};

// One element.
struct OneTerm {
    int v;
    float value;
    template <int n> __device__ __forceinline__ void chunk(int, int first, float (&x)[n]) const
    {
        const int at = v - first;
        if (at >= 0 && at < n) {
#pragma unroll
            for (int k = 0; k < n; ++k)
                x[k] = k == at ? value : x[k];
        }
    }
    __device__ __forceinline__ float edge(int u, float y) const { return u == v ? value : y; }
};

template <typename T>
__device__ __forceinline__ void store_chunk(T *out, const float (&y)[Pack<T>::n], bool aligned)
{
    if (aligned) {
        // not read again here: kept out of the way of what other rows read
        __builtin_nontemporal_store(Pack<T>::close(y), reinterpret_cast<u32x4 *>(out));
    } else {
#pragma unroll
        for (int i = 0; i < Pack<T>::n; ++i)
            Pack<T>::put(out + i, y[i]);
    }
}

// The row read from memory in each pass.
template <typename T, int NT> struct Streamed : Slice<T, NT> {
    using S = Slice<T, NT>;
    static constexpr int n = S::n;
    static constexpr int lds_chunks = 0, waves = 8;
    static constexpr int kUnroll = 4;
    __device__ __forceinline__ Streamed(const T *p, int len, int part, int parts,
                                        u32x4 * = nullptr)
        : S(p, len, part, parts)
    {
    }

    __device__ __forceinline__ void load() {}

    // f(this thread's i-th, chunk, values) for each chunk, read from memory
    template <bool First, typename F> __device__ __forceinline__ void each(F &&f) const
    {
        int i = S::c0 + (int)threadIdx.x, k = 0;
        for (; i + (kUnroll - 1) * NT < S::c1; i += kUnroll * NT, k += kUnroll) {
            u32x4 v[kUnroll];
#pragma unroll
            for (int j = 0; j < kUnroll; ++j)
                v[j] = *S::chunk(i + j * NT);
#pragma unroll
            for (int j = 0; j < kUnroll; ++j) {
                float x[n];
                Pack<T>::open(v[j], x);
                f(k + j, i + j * NT, x);
            }
        }
        for (; i < S::c1; i += NT, ++k) {
            float x[n];
            Pack<T>::open(*S::chunk(i), x);
            f(k, i, x);
        }
    }
    // the thread's value of the edge, -inf without one
    __device__ __forceinline__ float edge_value() const
    {
        const int t = threadIdx.x;
        return S::has_edge(t) ? Pack<T>::get(S::row + S::edge_at(t)) : -kInf;
    }

    __device__ __forceinline__ void stats(const Scale &c, float &m, float &s) const
    {
        const int t = threadIdx.x;
        if (S::has_edge(t)) {
            const float x[1] = {Pack<T>::get(S::row + S::edge_at(t))};
            absorb<1>(x, c, m, s);
        }
        int i = S::c0 + t;
        for (; i + (kUnroll - 1) * NT < S::c1; i += kUnroll * NT) {
            u32x4 v[kUnroll];
#pragma unroll
            for (int j = 0; j < kUnroll; ++j)
                v[j] = *S::chunk(i + j * NT);
#pragma unroll
            for (int j = 0; j < kUnroll; ++j) {
                float x[n];
                Pack<T>::open(v[j], x);
                absorb<n>(x, c, m, s);
            }
        }
        for (; i < S::c1; i += NT) {
            float x[n];
            Pack<T>::open(*S::chunk(i), x);
            absorb<n>(x, c, m, s);
        }
    }

    template <typename D, typename Terms>
    __device__ __forceinline__ void dense(T *out, const D &d, const Terms &terms) const
    {
        const int t = threadIdx.x;
        const bool aligned = (((uintptr_t)(out + S::cut.head)) & 15) == 0;
        if (S::has_edge(t)) {
            const int v = S::edge_at(t);
            Pack<T>::put(out + v, terms.edge(v, d.at(Pack<T>::get(S::row + v))));
        }
        auto put = [&](int i, u32x4 v) {
            float x[n];
            Pack<T>::open(v, x);
#pragma unroll
            for (int k = 0; k < n; ++k)
                x[k] = d.at(x[k]);
            const int first = S::cut.head + i * n;
            terms.chunk((i - S::c0) / NT, first, x);
            store_chunk<T>(out + first, x, aligned);
        };
        int i = S::c0 + t;
        for (; i + (kUnroll - 1) * NT < S::c1; i += kUnroll * NT) {
            u32x4 v[kUnroll];
#pragma unroll
            for (int j = 0; j < kUnroll; ++j)
                v[j] = *S::chunk(i + j * NT);
#pragma unroll
            for (int j = 0; j < kUnroll; ++j)
                put(i + j * NT, v[j]);
        }
        for (; i < S::c1; i += NT)
            put(i, *S::chunk(i));
    }
};

// Chunks on their way into shared memory: 16 bytes a lane, a wave's chunk in a
// run from `to` on (the same in all its lanes).
__device__ __forceinline__ void load_to_lds(const u32x4 *from, u32x4 *to)
{
    __builtin_amdgcn_global_load_lds(
        (const __attribute__((address_space(1))) void *)from,
        (__attribute__((address_space(3))) void *)to, 16, 0, 0);
}

// The row read once and kept between the passes: N chunks a thread in
// registers, L more in shared memory; what is beyond (N + L) * NT chunks is
// read in both passes.  Every thread reads its own chunks only, so the shared
// memory needs a wait for its loads and no barrier.
template <typename T, int NT, int N, int L = 0> struct Held : Slice<T, NT> {
    using S = Slice<T, NT>;
    static constexpr int n = S::n;
    static constexpr int lds_chunks = L * NT;
    // waves per SIMD: with up to 8 chunks a thread all of a compute unit's 2048
    // threads fit (64 registers each), so that rows overlap
    static constexpr int waves = N <= 8 ? 8 : 4;
    static constexpr int kUnroll = 2;   // registers are taken
    u32x4 v[N];
    float e;
    u32x4 *lds;   // [L][NT]

    __device__ __forceinline__ Held(const T *p, int len, int part, int parts, u32x4 *room)
        : S(p, len, part, parts), lds(room)
    {
    }
    __device__ __forceinline__ void load()
    {
        const int t = threadIdx.x;
        e = S::has_edge(t) ? Pack<T>::get(S::row + S::edge_at(t)) : -kInf;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            v[i] = u32x4{Pack<T>::kNone, Pack<T>::kNone, Pack<T>::kNone, Pack<T>::kNone};
            const int at = S::c0 + i * NT + t;
            // read once: kept out of the caches (2048 to 16384 rows of 64 to 256 KB:
            // 2 to 7% faster, rows of just 128 KB 5% slower)
            if (at < S::c1)
                v[i] = __builtin_nontemporal_load(S::chunk(at));
        }
        if constexpr (L > 0) {
            u32x4 *wave = lds + wave_id_uniform() * kWave;
#pragma unroll
            for (int i = 0; i < L; ++i) {
                const int at = S::c0 + (N + i) * NT + t;
                if (at < S::c1)
                    load_to_lds(S::chunk(at), wave + i * NT);
            }
        }
    }
    __device__ __forceinline__ float edge_value() const { return e; }
    // f(this thread's i-th, chunk, values) for each held chunk, then for those beyond
    template <bool First, typename F> __device__ __forceinline__ void each(F &&f) const
    {
        const int t = threadIdx.x;
#pragma unroll
        for (int i = 0; i < N; ++i)
            if (S::c0 + i * NT < S::c1) {
                float x[n];
                Pack<T>::open(v[i], x);
                f(i, S::c0 + i * NT + t, x);
            }
        if constexpr (L > 0) {
            // the loads into shared memory are this wave's own; the first pass waits for them
            if constexpr (First)
                asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
#pragma unroll
            for (int i = 0; i < L; ++i) {
                const int at = S::c0 + (N + i) * NT + t;
                if (at < S::c1) {
                    float x[n];
                    Pack<T>::open(lds[i * NT + t], x);
                    f(N + i, at, x);
                }
            }
            int i = S::c0 + (N + L) * NT + t;
            for (; i + (kUnroll - 1) * NT < S::c1; i += kUnroll * NT) {
                u32x4 w[kUnroll];
#pragma unroll
                for (int j = 0; j < kUnroll; ++j)
                    w[j] = *S::chunk(i + j * NT);
#pragma unroll
                for (int j = 0; j < kUnroll; ++j) {
                    float x[n];
                    Pack<T>::open(w[j], x);
                    f((i - S::c0) / NT + j, i + j * NT, x);
                }
            }
            for (; i < S::c1; i += NT) {
                float x[n];
                Pack<T>::open(*S::chunk(i), x);
                f((i - S::c0) / NT, i, x);
            }
        }
    }
    __device__ __forceinline__ void stats(const Scale &c, float &m, float &s) const
    {
        each<true>([&](int, int, const float (&x)[n]) { absorb<n>(x, c, m, s); });
        const float x[1] = {e};
        absorb<1>(x, c, m, s);
    }
    template <typename D, typename Terms>
    __device__ __forceinline__ void dense(T *out, const D &d, const Terms &terms) const
    {
        const int t = threadIdx.x;
        const bool aligned = (((uintptr_t)(out + S::cut.head)) & 15) == 0;
        if (S::has_edge(t)) {
            const int u = S::edge_at(t);
            Pack<T>::put(out + u, terms.edge(u, d.at(e)));
        }
        each<false>([&](int i, int at, float (&x)[n]) {
            if (at < S::c1) {
#pragma unroll
                for (int k = 0; k < n; ++k)
                    x[k] = d.at(x[k]);
                const int first = S::cut.head + at * n;
                terms.chunk(i, first, x);
                store_chunk<T>(out + first, x, aligned);
            }
        });
    }
};

// Calls f with the row source that fits rows of `len` values.  A work-group of
// 1024 threads has 128 registers a thread and 160 KB of shared memory: it holds
// 16 chunks a thread (256 KB) in registers, up to 400 KB with 9 chunks in shared
// memory, and 464 KB with 20 and 9; longer rows are read twice beyond that.
// `taken`: bytes of shared memory that the caller needs itself; where they leave
// no room for chunks, a long row is read twice as a whole.
// `alone`: no two rows will share a compute unit, and the caller's own work would
// spill registers beside 8 chunks a thread at 64.
template <typename T, typename F> void with_source(int len, size_t taken, bool alone, F &&f)
{
    const long chunks = (long)len * (long)sizeof(T) / 16;
    const bool room = taken + 9 * 1024 * 16 <= (160u << 10) - 512;
    if (chunks <= 256)
        f.template operator()<64, Held<T, 64, 4>>();
    else if (chunks <= 512)
        f.template operator()<64, Held<T, 64, 8>>();
    else if (chunks <= 1024)
        f.template operator()<256, Held<T, 256, 4>>();
    else if (chunks <= 2048)
        f.template operator()<256, Held<T, 256, 8>>();
    else if (chunks <= 4096 && !alone)
        f.template operator()<512, Held<T, 512, 8>>();
    else if (chunks <= 8192 && !alone)
        f.template operator()<1024, Held<T, 1024, 8>>();
    else if (chunks <= 16384)
        f.template operator()<1024, Held<T, 1024, 16>>();
    else if (!room)
        f.template operator()<1024, Streamed<T, 1024>>();
    else if (chunks <= 25600)
        f.template operator()<1024, Held<T, 1024, 16, 9>>();
    else
        f.template operator()<1024, Held<T, 1024, 20, 9>>();
}

// The same for a pass that reads the row once.  Few rows take more threads each
// (4 rows of 64 KB: 5.1 us with 256 threads a row, 4.2 with 1024).
template <typename T, typename F> void with_stream(int len, int rows, F &&f)
{
    const long chunks = (long)len * (long)sizeof(T) / 16 / (rows <= 256 ? 1 : 4);
    if (chunks <= 128)
        f.template operator()<64, Streamed<T, 64>>();
    else if (chunks <= 1024)
        f.template operator()<256, Streamed<T, 256>>();
    else
        f.template operator()<1024, Streamed<T, 1024>>();
}

// Zeros over the slice's elements of an output row (cut by the output's own
// alignment: nothing is read).
template <typename T, int NT> __device__ __forceinline__ void zero_row(T *out, int len, int part, int parts)
{
    const Slice<T, NT> z(out, len, part, parts);
    const int t = threadIdx.x;
    if (z.has_edge(t))
        Pack<T>::put(out + z.edge_at(t), 0.f);
    u32x4 *base = reinterpret_cast<u32x4 *>(out + z.cut.head);
    for (int i = z.c0 + t; i < z.c1; i += NT)
        base[i] = u32x4{0u, 0u, 0u, 0u};
}

}  // namespace rows
}  // namespace sk
