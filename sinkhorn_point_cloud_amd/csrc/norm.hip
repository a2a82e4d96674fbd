// norm.hip -- root-mean-square norm of rows with the residual's addition, in the
// stream's type or in 8 bits, and its gradient.
//
//     h = round(x + residual),  r = 1 / sqrt(sum h^2 / d + eps),  y = h w r;
//     8 bits: p = h w, a = max |p|,  q = rint(127 p / a),  scale = a r / 127;
//     backward, u = dy w, n = h r:  dx = r (u - n (r sum u h) / d) + dh,
//                                   dweight_j = sum over rows of dy_j n_j.
// What bounds it: HBM.  A row is read once and kept in registers as 16-byte chunks,
// chunk i + j NT with thread i of the row's NT.  Rows at any address: the hardware loads
// and stores 16 bytes at any multiple of the type's size.  A row that ends inside a
// chunk has its last one begin earlier, and what the chunk before it holds already
// counts as zeros; so do the chunks of threads beyond the row, which read its last one
// again.  The loads are then the same for all threads and asked for together.  (With a
// path for the end of its own, value by value, 777 rows of 2501 fp32 values took 9.8 us,
// the gradient 16.3.)  A thread writes only values that no other counts, behind its own
// reads of them, so an output may be an input itself.
// Sums within a row are fp64: squares of any finite input stay in range, and the
// row's factor is off by no more than its own rounding.
#include "head.h"
#include "rows.h"

namespace sk {
namespace {

using namespace rows;

enum Mode { kTyped, kEight, kEightPlain };

// 16 bytes at any address that suits the type.
template <typename T> struct Any;
template <> struct Any<float> {
    typedef u32x4 __attribute__((aligned(4))) chunk;
};
template <> struct Any<uint16_t> {
    typedef u32x4 __attribute__((aligned(2))) chunk;
};

// Where a chunk of a row begins, and how many of its values count as zeros.
template <typename T> struct Place {
    static constexpr int n = Pack<T>::n;
    int first, skip;
    __device__ __forceinline__ Place(int c, int chunks, int d)
    {
        first = max(min(c * n, d - n), 0);
        skip = c < chunks ? c * n - first : n;
    }
};

// Rows shorter than a chunk are read value by value.
template <typename T> __device__ __forceinline__ u32x4 load_chunk(const T *row, int first, int d)
{
    constexpr int n = Pack<T>::n;
    if (d >= n)
        return *reinterpret_cast<const typename Any<T>::chunk *>(row + first);
    float x[n];
#pragma unroll
    for (int i = 0; i < n; ++i)
        x[i] = i < d ? Pack<T>::get(row + i) : 0.f;
    return Pack<T>::close(x);
}
template <typename T> __device__ __forceinline__ u32x4 ones()
{
    constexpr uint32_t one = sizeof(T) == 2 ? 0x3F803F80u : 0x3F800000u;
    return u32x4{one, one, one, one};
}
// Zeros for the first `skip` values.
template <typename T> __device__ __forceinline__ u32x4 clear(u32x4 v, int skip)
{
    constexpr int n = Pack<T>::n;
    if (skip > 0) {
        float x[n];
        Pack<T>::open(v, x);
#pragma unroll
        for (int i = 0; i < n; ++i)
            x[i] = i < skip ? 0.f : x[i];
        v = Pack<T>::close(x);
    }
    return v;
}
template <typename T> __device__ __forceinline__ void put_chunk(T *row, const Place<T> &at, int d, u32x4 v)
{
    constexpr int n = Pack<T>::n;
    if (at.skip == 0 && d >= n) {
        *reinterpret_cast<typename Any<T>::chunk *>(row + at.first) = v;
    } else if (at.skip < n) {
        float x[n];
        Pack<T>::open(v, x);
#pragma unroll
        for (int i = 0; i < n; ++i)
            if (i >= at.skip && i < d)
                Pack<T>::put(row + at.first + i, x[i]);
    }
}
template <typename T>
__device__ __forceinline__ void put_bytes(int8_t *row, const Place<T> &at, int d, const int (&q)[Pack<T>::n])
{
    constexpr int n = Pack<T>::n;
    int8_t *p = row + at.first;
    if (at.skip == 0 && d >= n) {
        typedef uint32_t __attribute__((aligned(1))) word;
#pragma unroll
        for (int i = 0; i < n; i += 4)
            reinterpret_cast<word *>(p)[i / 4] =
                (uint32_t)(q[i] & 255) | (uint32_t)(q[i + 1] & 255) << 8 |
                (uint32_t)(q[i + 2] & 255) << 16 | (uint32_t)q[i + 3] << 24;
    } else if (at.skip < n) {
#pragma unroll
        for (int i = 0; i < n; ++i)
            if (i >= at.skip && i < d)
                p[i] = (int8_t)q[i];
    }
}

// Keeps a chunk in its registers: without it the compiler holds the opened values of a
// row from one use to the next, twice the registers for bf16.
__device__ __forceinline__ void packed(u32x4 &v) { asm volatile("" : "+v"(v)); }
__device__ __forceinline__ int fresh(int v)
{
    asm volatile("" : "+v"(v));
    return v;
}

// A row's threads: a wave, four rows to a work-group, or a whole work-group.
template <bool Alone> struct Team {
    int size, i0;
    long row;   // of the launch
    __device__ __forceinline__ Team()
        : size(Alone ? kWave : (int)blockDim.x), i0(Alone ? lane_id() : (int)threadIdx.x),
          row(Alone ? group_index() * 4 + threadIdx.x / kWave : group_index())
    {
    }
};

// Sum, or maximum, of up to 16 waves' values, from `room`, the same in every lane: a lane
// takes one of them, and lane moves do the rest.
template <typename P> __device__ __forceinline__ P of_waves(const P *room, bool sum)
{
    const int lane = lane_id() & 15;
    P v = lane < (int)blockDim.x / kWave ? room[lane] : (P)0;   // the maxima are of magnitudes
    auto join = [&](P other) { v = sum ? v + other : other > v ? other : v; };
    join(dpp_move<kDppXor1>(v));
    join(dpp_move<kDppXor2>(v));
    join(dpp_move<kDppHalfMirror>(v));
    join(dpp_move<kDppMirror>(v));
    return v;
}
// Over a row's threads.  One barrier for rows of more than a wave; `room`, an entry a
// wave, may be written again behind another.
template <bool Alone> __device__ __forceinline__ double row_total(double v, double *room)
{
    v = sum_wave(v);
    if constexpr (!Alone) {
        if (lane_id() == 0)
            room[threadIdx.x / kWave] = v;
        __syncthreads();
        v = of_waves(room, true);
    }
    return v;
}
template <bool Alone, typename P> __device__ __forceinline__ P row_most(P v, P *room)
{
    v = wave_max(v);
    if constexpr (!Alone) {
        if (lane_id() == 0)
            room[threadIdx.x / kWave] = v;
        __syncthreads();
        v = of_waves(room, false);
    }
    return v;
}

// 127 p / a to the nearest whole number, ties to even, where a = m 2^e with m in
// [1/2, 1): from the fp32 quotient, off by less than 1e-4, unless that is nearer to
// the middle of two; there the sign of 127 p - (k + 1/2) a decides.  127 p of a fp32
// product (48 bits) has up to 55 bits: its rounding and what that left out.  Both, and
// the difference so near the middle (of at most 43 bits), are exact in fp64.
__device__ __forceinline__ float quotient(double p, int e, float inv)
{
    return (float)__builtin_amdgcn_ldexp(p, -e) * inv;
}
__device__ __forceinline__ float quotient(float p, int e, float inv)
{
    return __builtin_amdgcn_ldexpf(p, -e) * inv;
}
__device__ __forceinline__ bool near_middle(float t)
{
    return fabsf(fabsf(t - __builtin_rintf(t)) - 0.5f) < 1e-4f;
}
__device__ __forceinline__ int step_exact(double p, double a, float t)
{
    const double k = __builtin_floor((double)t);
    const double much = 127.0 * p, rest = fma(127.0, p, -much);
    const double gap = fma(-(k + 0.5), a, much) + rest;
    const int low = (int)k;
    return gap > 0.0 || (gap == 0.0 && (low & 1)) ? low + 1 : low;
}

template <typename T, bool Alone, int NV, int M>
__global__ __launch_bounds__(NV == 1 || Alone ? 256 : NV == 2 ? 512 : 1024) void norm_kernel(NormArgs a)
{
    constexpr int n = Pack<T>::n;
    using P = typename std::conditional<sizeof(T) == 2, float, double>::type;
    __shared__ double room[16];
    __shared__ P most_room[16];
    const Team<Alone> team;
    const long t = team.row;
    if (t >= a.T)
        return;
    const int d = a.d, chunks = (d + n - 1) / n;
    const T *x = (const T *)a.x + t * a.ldx;
    constexpr bool kNorm = M != kEightPlain;
    const bool has_res = kNorm && a.residual, has_weight = kNorm && a.weight;
    u32x4 h[NV], r[NV], w[NV];
    // all that the row needs is asked for before any of it is used
#define SK_PLACE(j) const Place<T> at(team.i0 + (j) * team.size, chunks, d)
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        SK_PLACE(j);
        h[j] = load_chunk(x, at.first, d);
    }
    if (has_res) {
        const T *res = (const T *)a.residual + t * a.ldr;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            SK_PLACE(j);
            r[j] = load_chunk(res, at.first, d);
        }
    }
    // (but for the longest rows' weights, whose registers are taken)
    auto weight = [&](int j) {
        SK_PLACE(j);
        return load_chunk((const T *)a.weight, at.first, d);
    };
    if (NV < 8 && has_weight) {
#pragma unroll
        for (int j = 0; j < NV; ++j)
            w[j] = weight(j);
    }
    T *hout = kNorm && a.h ? (T *)a.h + t * a.ldh : nullptr;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        SK_PLACE(j);
        if (has_res) {
            float u[n], v[n];
            Pack<T>::open(h[j], u);
            Pack<T>::open(r[j], v);
#pragma unroll
            for (int k = 0; k < n; ++k)
                u[k] += v[k];
            h[j] = Pack<T>::close(u);
        }
        h[j] = clear<T>(h[j], at.skip);
        if (NV < 8 && has_weight)
            w[j] = clear<T>(w[j], at.skip);   // 0 times what may be infinite is none
        if (hout)
            put_chunk(hout, at, d, h[j]);
    }
    double factor = 1.0;
    if constexpr (M != kEightPlain) {
        double ss = 0.0;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            float u[n];
            Pack<T>::open(h[j], u);
#pragma unroll
            for (int k = 0; k < n; ++k)
                ss = fma((double)u[k], (double)u[k], ss);
        }
        ss = row_total<Alone>(ss, room);
#pragma unroll
        for (int j = 0; j < NV; ++j)
            packed(h[j]);
        factor = 1.0 / sqrt(ss / d + a.eps);
    }
    if constexpr (M == kTyped) {
        T *y = (T *)a.y + t * a.ldy;
        const float rf = (float)factor;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            SK_PLACE(j);
            float u[n];
            Pack<T>::open(h[j], u);
#pragma unroll
            for (int k = 0; k < n; ++k)
                u[k] *= rf;
            if (has_weight) {
                float v[n];
                Pack<T>::open(NV < 8 ? w[j] : clear<T>(weight(j), Place<T>(team.i0 + j * team.size, chunks, d).skip), v);
#pragma unroll
                for (int k = 0; k < n; ++k)
                    u[k] *= v[k];
            }
            put_chunk(y, at, d, Pack<T>::close(u));
        }
    } else {
        auto product = [&](int j, P (&p)[n]) {
            float u[n];
            Pack<T>::open(h[j], u);
            if (has_weight) {
                float v[n];
                Pack<T>::open(NV < 8 ? w[j] : clear<T>(weight(j), Place<T>(team.i0 + j * team.size, chunks, d).skip), v);
#pragma unroll
                for (int k = 0; k < n; ++k)
                    p[k] = (P)u[k] * (P)v[k];
            } else {
#pragma unroll
                for (int k = 0; k < n; ++k)
                    p[k] = (P)u[k];
            }
        };
        const P inf = (P)__builtin_inf();
        P most = 0;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            P p[n];
            product(j, p);
#pragma unroll
            for (int k = 0; k < n; ++k) {
                const P b = p[k] < 0 ? -p[k] : p[k];
                most = b <= most ? most : b == b ? b : inf;   // a NaN counts as infinite
            }
            __builtin_amdgcn_sched_barrier(0);   // one chunk's values at a time in registers
        }
        most = row_most<Alone>(most, most_room);
#pragma unroll
        for (int j = 0; j < NV; ++j)
            packed(h[j]);
        int8_t *q = a.q + t * a.ldq;
        const bool sound = most < inf;
        if (team.i0 == 0)
            a.scale[t] = sound ? (float)((double)most * factor / 127.0) : __builtin_nanf("");
        const int e = sound ? __builtin_amdgcn_frexp_exp(most) : 0;
        const double mant = __builtin_amdgcn_ldexp((double)most, -e);
        const float inv = sound && most > 0 ? (float)(127.0 / mant) : 0.f;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            SK_PLACE(j);
            P p[n];
            product(j, p);
            int s[n];
            bool middle = false;
            float v[n];
#pragma unroll
            for (int k = 0; k < n; ++k) {
                v[k] = sound ? quotient(p[k], e, inv) : 0.f;
                s[k] = (int)__builtin_rintf(v[k]);
                middle |= near_middle(v[k]);
            }
            if (middle) {
#pragma unroll
                for (int k = 0; k < n; ++k)
                    if (near_middle(v[k]))
                        s[k] = step_exact((double)p[k], (double)most, v[k]);
            }
            put_bytes<T>(q, at, d, s);
            __builtin_amdgcn_sched_barrier(0);
        }
    }
}

// The gradient.  A worker (the NT threads of a row) takes rows g, g + G, ... and
// keeps its share of dweight in registers.
template <typename T, bool Alone, int NV>
__global__ __launch_bounds__(NV == 1 || Alone ? 256 : NV == 2 ? 512 : 1024) void
norm_grad_kernel(NormGradArgs a, int G)
{
    constexpr int n = Pack<T>::n;
    __shared__ double room[2][32];
    const Team<Alone> team;
    const long g = team.row;
    if (g >= G)
        return;
    const int d = a.d, chunks = (d + n - 1) / n;
    float acc[NV][n];
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int k = 0; k < n; ++k)
            acc[j][k] = 0.f;
    int turn = 0;
    for (long t = g; t < a.T; t += G, turn ^= 1) {
        // found again for each row: the compiler would keep a mask for each value instead
        const int i0 = fresh(team.i0);
#undef SK_PLACE
#define SK_PLACE(j) const Place<T> at(i0 + (j) * team.size, chunks, d)
        const T *h = (const T *)a.h + t * a.ldh, *dy = (const T *)a.dy + t * a.lddy;
        const T *dh = a.dh ? (const T *)a.dh + t * a.lddh : nullptr;
        u32x4 hv[NV], gv[NV], ev[NV], wv[NV];
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            SK_PLACE(j);
            hv[j] = load_chunk(h, at.first, d);
            gv[j] = load_chunk(dy, at.first, d);
        }
        // without a weight ones, without dh zeros: the same arithmetic for all
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            SK_PLACE(j);
            wv[j] = ones<T>();
            if (a.weight)
                wv[j] = load_chunk((const T *)a.weight, at.first, d);
        }
        // longer rows' registers are taken: theirs is asked for behind the sums
        auto beside = [&](int j) {
            SK_PLACE(j);
            u32x4 v = {0u, 0u, 0u, 0u};
            if (dh)
                v = load_chunk(dh, at.first, d);
            return v;
        };
        if constexpr (NV <= 2) {
#pragma unroll
            for (int j = 0; j < NV; ++j)
                ev[j] = beside(j);
        }
        double ss = 0.0, uh = 0.0;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            SK_PLACE(j);
            hv[j] = clear<T>(hv[j], at.skip);
            gv[j] = clear<T>(gv[j], at.skip);
            wv[j] = clear<T>(wv[j], at.skip);   // 0 times what may be infinite is none
            float x[n], y[n], w[n];
            Pack<T>::open(hv[j], x);
            Pack<T>::open(gv[j], y);
            Pack<T>::open(wv[j], w);
#pragma unroll
            for (int k = 0; k < n; ++k) {
                const float u = y[k] * w[k];
                ss = fma((double)x[k], (double)x[k], ss);
                uh = fma((double)u, (double)x[k], uh);
            }
        }
        ss = sum_wave(ss);
        uh = sum_wave(uh);
        if constexpr (!Alone) {
            // two rooms in turn: one barrier a row
            double *to = room[turn];
            if (lane_id() == 0) {
                to[threadIdx.x / kWave] = ss;
                to[16 + threadIdx.x / kWave] = uh;
            }
            __syncthreads();
            ss = of_waves(to, true);
            uh = of_waves(to + 16, true);
        }
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            packed(hv[j]);
            packed(gv[j]);
            packed(wv[j]);
        }
        // n is at most sqrt(d) and the mean of u n at most u's: factors that leave fp32 in no row
        // whose gradient does not (r^3 (sum u h) / d and dy r are 0 for rows of 1e20 and small dy)
        const double r = 1.0 / sqrt(ss / d + a.eps);
        const float rf = (float)r, mean = (float)(r * (uh / d));
        T *dx = (T *)a.dx + t * a.lddx;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            SK_PLACE(j);
            float x[n], y[n], w[n], e[n];
            Pack<T>::open(hv[j], x);
            Pack<T>::open(gv[j], y);
            Pack<T>::open(wv[j], w);
            Pack<T>::open(NV <= 2 ? ev[j] : beside(j), e);
#pragma unroll
            for (int k = 0; k < n; ++k) {
                const float norm = x[k] * rf;
                acc[j][k] = fmaf(y[k], norm, acc[j][k]);
                y[k] = fmaf(rf, fmaf(-norm, mean, y[k] * w[k]), e[k]);
            }
            put_chunk(dx, at, d, Pack<T>::close(y));
        }
    }
    if (!a.dweight)
        return;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        const Place<T> at(team.i0 + j * team.size, chunks, d);
#pragma unroll
        for (int k = 0; k < n; ++k)
            if (k >= at.skip && k < d)
                a.part[g * d + at.first + k] = acc[j][k];
    }
}
#undef SK_PLACE

// dweight from the workers' shares: C columns a work-group, 1024 / C threads a column,
// eight shares asked for together.
template <int C>
__global__ __launch_bounds__(1024) void norm_join_kernel(const float *part, int G, int d, float *dweight)
{
    constexpr int slices = 1024 / C;
    __shared__ double room[slices][C];
    const int column = threadIdx.x % C, at = blockIdx.x * C + column, slice = threadIdx.x / C;
    double v = 0.0;
    if (at < d) {
        int g = slice;
        for (; g + 7 * slices < G; g += 8 * slices) {
            float x[8];
#pragma unroll
            for (int i = 0; i < 8; ++i)
                x[i] = part[(long)(g + i * slices) * d + at];
#pragma unroll
            for (int i = 0; i < 8; ++i)
                v += (double)x[i];
        }
        for (; g < G; g += slices)
            v += (double)part[(long)g * d + at];
    }
    room[slice][column] = v;
    __syncthreads();
    if (slice == 0 && at < d) {
#pragma unroll
        for (int i = 1; i < slices; ++i)
            v += room[i][column];
        dweight[at] = (float)v;
    }
}

// Threads and chunks a thread for rows of `chunks` 16-byte chunks: as many waves as the
// row fills.  (Rows of more than 16384 fp32 values take eight chunks a thread of the largest
// work-group, whose 128 registers the gradient exceeds by 70: 2000 x 32768 428 us, 2.5 TB/s.)
int threads_of(int chunks, int nv) { return (chunks + nv * kWave - 1) / (nv * kWave) * kWave; }
template <typename T, typename F> void with_shape(int chunks, F &&f)
{
    if (chunks <= 64)
        f.template operator()<true, 1>(256);
    else if (chunks <= 128)
        f.template operator()<true, 2>(256);
    else if (chunks <= 256)
        f.template operator()<false, 1>(threads_of(chunks, 1));
    else if (chunks <= 1024)
        f.template operator()<false, 2>(threads_of(chunks, 2));
    else if (sizeof(T) == 2 || chunks <= 4096)
        f.template operator()<false, 4>(threads_of(chunks, 4));
    else if constexpr (sizeof(T) == 4)
        f.template operator()<false, 8>(threads_of(chunks, 8));
}

int chunks_of(int d, int dtype)
{
    const int n = dtype == 1 ? 8 : 4;
    return (d + n - 1) / n;
}
int rows_per_group(int chunks) { return chunks <= 128 ? 4 : 1; }

template <typename T, int M> struct RunNorm {
    const NormArgs &a;
    hipStream_t st;
    template <bool Alone, int NV> void operator()(int threads) const
    {
        hipLaunchKernelGGL((norm_kernel<T, Alone, NV, M>), grid_of(Alone ? ((long)a.T + 3) / 4 : a.T),
                           dim3(threads), 0, st, a);
    }
};
template <typename T> struct RunGrad {
    const NormGradArgs &a;
    int G;
    hipStream_t st;
    template <bool Alone, int NV> void operator()(int threads) const
    {
        hipLaunchKernelGGL((norm_grad_kernel<T, Alone, NV>), grid_of(Alone ? (G + 3) / 4 : G), dim3(threads),
                           0, st, a, G);
    }
};

template <typename T> void run_norm(const NormArgs &a, hipStream_t st)
{
    const int chunks = chunks_of(a.d, a.dtype);
    if (!a.q)
        with_shape<T>(chunks, RunNorm<T, kTyped>{a, st});
    else if (a.norm)
        with_shape<T>(chunks, RunNorm<T, kEight>{a, st});
    else
        with_shape<T>(chunks, RunNorm<T, kEightPlain>{a, st});
}

}  // namespace

hipError_t launch_norm(const NormArgs &a, hipStream_t st)
{
    if (a.dtype == 1)
        run_norm<uint16_t>(a, st);
    else
        run_norm<float>(a, st);
    return hipGetLastError();
}

int norm_groups(int T, int d, int dtype)
{
    // workers of a wave are more, where they still have eight rows each (65536 x 512 bf16: with
    // 1024, 2048 and 4096 of them 69, 50 and 44 us, the join 5, 6 and 10)
    const int per = rows_per_group(chunks_of(d, dtype));
    const int most = per > 1 ? std::clamp(T / 8 / per * per, 1024, 2048) : 1024;
    return std::min((T + per - 1) / per * per, most);
}

hipError_t launch_norm_backward(const NormGradArgs &a, hipStream_t st)
{
    const int G = norm_groups(a.T, a.d, a.dtype), chunks = chunks_of(a.d, a.dtype);
    if (G > 0) {
        if (a.dtype == 1)
            with_shape<uint16_t>(chunks, RunGrad<uint16_t>{a, G, st});
        else
            with_shape<float>(chunks, RunGrad<float>{a, G, st});
    }
    if (a.dweight && a.d <= 1024)
        hipLaunchKernelGGL((norm_join_kernel<16>), dim3((a.d + 15) / 16), dim3(1024), 0, st, a.part, G, a.d,
                           a.dweight);
    else if (a.dweight)
        hipLaunchKernelGGL((norm_join_kernel<64>), dim3((a.d + 63) / 64), dim3(1024), 0, st, a.part, G, a.d,
                           a.dweight);
    return hipGetLastError();
}

}  // namespace sk
