// norm.hip -- root-mean-square norm of rows with the residual's addition, in the
// stream's type or in 8 bits, and its gradient.
//
//     h = round(x + residual),  r = 1 / sqrt(sum h^2 / d + eps),  y = h w r;
//     8 bits: p = h w, a = max |p|,  q = rint(127 p / a),  scale = a r / 127;
//     backward, u = dy w:  dx = r (u - h r^2 (sum u h) / d) + dh,
//                          dweight_j = sum over rows of dy_j h_j r.
// What bounds it: HBM.  A row is read once and kept in registers as 16-byte
// chunks, chunk i + j NT with thread i of the row's NT; a thread reads and writes
// the same elements, so an output may be an input itself.  Rows at any address:
// the hardware loads and stores 16 bytes at any multiple of the type's size.
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

template <typename T> __device__ __forceinline__ u32x4 load_chunk(const T *row, int c, int d)
{
    constexpr int n = Pack<T>::n;
    const T *p = row + c * n;
    if ((c + 1) * n <= d)
        return *reinterpret_cast<const typename Any<T>::chunk *>(p);
    float x[n];
#pragma unroll
    for (int i = 0; i < n; ++i)
        x[i] = c * n + i < d ? Pack<T>::get(p + i) : 0.f;
    return Pack<T>::close(x);
}
template <typename T> __device__ __forceinline__ void put_chunk(T *row, int c, int d, u32x4 v)
{
    constexpr int n = Pack<T>::n;
    T *p = row + c * n;
    if ((c + 1) * n <= d) {
        *reinterpret_cast<typename Any<T>::chunk *>(p) = v;
        return;
    }
    float x[n];
    Pack<T>::open(v, x);
#pragma unroll
    for (int i = 0; i < n; ++i)
        if (c * n + i < d)
            Pack<T>::put(p + i, x[i]);
}
template <int n> __device__ __forceinline__ void put_bytes(int8_t *row, int c, int d, const int (&q)[n])
{
    int8_t *p = row + c * n;
    if ((c + 1) * n <= d) {
        typedef uint32_t __attribute__((aligned(1))) word;
#pragma unroll
        for (int i = 0; i < n; i += 4)
            reinterpret_cast<word *>(p)[i / 4] =
                (uint32_t)(q[i] & 255) | (uint32_t)(q[i + 1] & 255) << 8 |
                (uint32_t)(q[i + 2] & 255) << 16 | (uint32_t)q[i + 3] << 24;
        return;
    }
#pragma unroll
    for (int i = 0; i < n; ++i)
        if (c * n + i < d)
            p[i] = (int8_t)q[i];
}

// Sum, or maximum, over the NT threads of a row, the same in all of them.  One
// barrier for rows of more than a wave; `room` may be written again behind another.
template <int NT> __device__ __forceinline__ double row_total(double v, double *room)
{
    v = sum_wave(v);
    if constexpr (NT > kWave) {
        if (lane_id() == 0)
            room[threadIdx.x / kWave] = v;
        __syncthreads();
        v = room[0];
#pragma unroll
        for (int i = 1; i < NT / kWave; ++i)
            v += room[i];
    }
    return v;
}
template <int NT, typename P> __device__ __forceinline__ P row_most(P v, P *room)
{
    v = wave_max(v);
    if constexpr (NT > kWave) {
        if (lane_id() == 0)
            room[threadIdx.x / kWave] = v;
        __syncthreads();
        v = room[0];
#pragma unroll
        for (int i = 1; i < NT / kWave; ++i)
            v = room[i] > v ? room[i] : v;
    }
    return v;
}

// 127 p / a to the nearest whole number, ties to even, where a = m 2^e with m in
// [1/2, 1): from the fp32 quotient, off by less than 1e-4, unless that is nearer to
// the middle of two; there the sign of 127 p - (k + 1/2) a decides, which is exact
// in fp64 for bf16 products (and off by 2^-53 for fp32 ones).
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
    const double gap = fma(-(k + 0.5), a, 127.0 * p);
    const int low = (int)k;
    return gap > 0.0 || (gap == 0.0 && (low & 1)) ? low + 1 : low;
}

template <typename T, int NT, int NV, int M>
__global__ __launch_bounds__(NT < 256 ? 256 : NT) void norm_kernel(NormArgs a)
{
    constexpr int n = Pack<T>::n, per = NT < 256 ? 256 / NT : 1;
    using P = typename std::conditional<sizeof(T) == 2, float, double>::type;
    __shared__ double room[NT / kWave];
    __shared__ P most_room[NT / kWave];
    const long t = group_index() * per + (per > 1 ? threadIdx.x / NT : 0);
    if (t >= a.T)
        return;
    const int i0 = threadIdx.x % NT, d = a.d, chunks = (d + n - 1) / n;
    const T *x = (const T *)a.x + t * a.ldx;
    u32x4 h[NV], w[NV];
#pragma unroll
    for (int j = 0; j < NV; ++j)
        if (i0 + j * NT < chunks)
            h[j] = load_chunk(x, i0 + j * NT, d);
    if (a.residual) {
        const T *res = (const T *)a.residual + t * a.ldr;
        u32x4 r[NV];
#pragma unroll
        for (int j = 0; j < NV; ++j)
            if (i0 + j * NT < chunks)
                r[j] = load_chunk(res, i0 + j * NT, d);
#pragma unroll
        for (int j = 0; j < NV; ++j)
            if (i0 + j * NT < chunks) {
                float u[n], v[n];
                Pack<T>::open(h[j], u);
                Pack<T>::open(r[j], v);
#pragma unroll
                for (int k = 0; k < n; ++k)
                    u[k] += v[k];
                h[j] = Pack<T>::close(u);
            }
    }
    if (a.weight) {
#pragma unroll
        for (int j = 0; j < NV; ++j)
            if (i0 + j * NT < chunks)
                w[j] = load_chunk((const T *)a.weight, i0 + j * NT, d);
    }
    if (a.h) {
        T *out = (T *)a.h + t * a.ldh;
#pragma unroll
        for (int j = 0; j < NV; ++j)
            if (i0 + j * NT < chunks)
                put_chunk(out, i0 + j * NT, d, h[j]);
    }
    double r = 1.0;
    if constexpr (M != kEightPlain) {
        double ss = 0.0;
#pragma unroll
        for (int j = 0; j < NV; ++j)
            if (i0 + j * NT < chunks) {
                float u[n];
                Pack<T>::open(h[j], u);
#pragma unroll
                for (int k = 0; k < n; ++k)
                    ss = fma((double)u[k], (double)u[k], ss);
            }
        ss = row_total<NT>(ss, room);
        r = 1.0 / sqrt(ss / d + a.eps);
    }
    if constexpr (M == kTyped) {
        T *y = (T *)a.y + t * a.ldy;
        const float rf = (float)r;
#pragma unroll
        for (int j = 0; j < NV; ++j)
            if (i0 + j * NT < chunks) {
                float u[n];
                Pack<T>::open(h[j], u);
                if (a.weight) {
                    float v[n];
                    Pack<T>::open(w[j], v);
#pragma unroll
                    for (int k = 0; k < n; ++k)
                        u[k] = u[k] * rf * v[k];
                } else {
#pragma unroll
                    for (int k = 0; k < n; ++k)
                        u[k] *= rf;
                }
                put_chunk(y, i0 + j * NT, d, Pack<T>::close(u));
            }
    } else {
        // the products, and whether all of them are finite: a maximum passes a NaN over
        auto product = [&](int j, P (&p)[n]) {
            float u[n];
            Pack<T>::open(h[j], u);
            if (a.weight) {
                float v[n];
                Pack<T>::open(w[j], v);
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
        for (int j = 0; j < NV; ++j)
            if (i0 + j * NT < chunks) {
                P p[n];
                product(j, p);
#pragma unroll
                for (int k = 0; k < n; ++k) {
                    const P b = p[k] < 0 ? -p[k] : p[k];
                    most = b <= most ? most : b == b ? b : inf;
                }
            }
        most = row_most<NT>(most, most_room);
        int8_t *q = a.q + t * a.ldq;
        const bool sound = most < inf;
        if (i0 == 0)
            a.scale[t] = sound ? (float)((double)most * r / 127.0) : __builtin_nanf("");
        const int e = sound ? __builtin_amdgcn_frexp_exp(most) : 0;
        const double mant = __builtin_amdgcn_ldexp((double)most, -e);
        const float inv = sound && most > 0 ? (float)(127.0 / mant) : 0.f;
#pragma unroll
        for (int j = 0; j < NV; ++j)
            if (i0 + j * NT < chunks) {
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
                put_bytes<n>(q, i0 + j * NT, d, s);
            }
    }
}

// The gradient.  A worker (the NT threads of a row) takes rows g, g + G, ... and
// keeps its share of dweight in registers.
template <typename T, int NT, int NV>
__global__ __launch_bounds__(NT < 256 ? 256 : NT) void norm_grad_kernel(NormGradArgs a, int G)
{
    constexpr int n = Pack<T>::n, per = NT < 256 ? 256 / NT : 1;
    __shared__ double room[2][2 * NT / kWave];
    const int g = (int)(group_index() * per) + (per > 1 ? (int)threadIdx.x / NT : 0);
    if (g >= G)
        return;
    const int i0 = threadIdx.x % NT, d = a.d, chunks = (d + n - 1) / n;
    float acc[NV][n];
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int k = 0; k < n; ++k)
            acc[j][k] = 0.f;
    int turn = 0;
    for (long t = g; t < a.T; t += G, turn ^= 1) {
        const T *h = (const T *)a.h + t * a.ldh, *dy = (const T *)a.dy + t * a.lddy;
        u32x4 hv[NV], gv[NV];
#pragma unroll
        for (int j = 0; j < NV; ++j)
            if (i0 + j * NT < chunks) {
                hv[j] = load_chunk(h, i0 + j * NT, d);
                gv[j] = load_chunk(dy, i0 + j * NT, d);
            }
        double ss = 0.0, uh = 0.0;
#pragma unroll
        for (int j = 0; j < NV; ++j)
            if (i0 + j * NT < chunks) {
                float x[n], y[n], w[n];
                Pack<T>::open(hv[j], x);
                Pack<T>::open(gv[j], y);
                if (a.weight)
                    Pack<T>::open(load_chunk((const T *)a.weight, i0 + j * NT, d), w);
#pragma unroll
                for (int k = 0; k < n; ++k) {
                    const float u = a.weight ? y[k] * w[k] : y[k];
                    ss = fma((double)x[k], (double)x[k], ss);
                    uh = fma((double)u, (double)x[k], uh);
                }
            }
        ss = sum_wave(ss);
        uh = sum_wave(uh);
        if constexpr (NT > kWave) {
            // two rooms in turn: one barrier a row
            double *at = room[turn];
            if (lane_id() == 0) {
                at[2 * (threadIdx.x / kWave)] = ss;
                at[2 * (threadIdx.x / kWave) + 1] = uh;
            }
            __syncthreads();
            ss = uh = 0.0;
#pragma unroll
            for (int i = 0; i < NT / kWave; ++i) {
                ss += at[2 * i];
                uh += at[2 * i + 1];
            }
        }
        const double r = 1.0 / sqrt(ss / d + a.eps);
        const float rf = (float)r, c = (float)(r * r * r * (uh / d));
        T *dx = (T *)a.dx + t * a.lddx;
        const T *dh = a.dh ? (const T *)a.dh + t * a.lddh : nullptr;
#pragma unroll
        for (int j = 0; j < NV; ++j)
            if (i0 + j * NT < chunks) {
                float x[n], y[n], w[n], e[n];
                Pack<T>::open(hv[j], x);
                Pack<T>::open(gv[j], y);
                if (a.weight)
                    Pack<T>::open(load_chunk((const T *)a.weight, i0 + j * NT, d), w);
                if (dh)
                    Pack<T>::open(load_chunk(dh, i0 + j * NT, d), e);
#pragma unroll
                for (int k = 0; k < n; ++k) {
                    const float yr = y[k] * rf;
                    acc[j][k] = fmaf(yr, x[k], acc[j][k]);
                    const float v = fmaf(-c, x[k], a.weight ? yr * w[k] : yr);
                    y[k] = dh ? v + e[k] : v;
                }
                put_chunk(dx, i0 + j * NT, d, Pack<T>::close(y));
            }
    }
    if (!a.dweight)
        return;
#pragma unroll
    for (int j = 0; j < NV; ++j)
        if (i0 + j * NT < chunks)
#pragma unroll
            for (int k = 0; k < n; ++k)
                if ((i0 + j * NT) * n + k < d)
                    a.part[(long)g * d + (i0 + j * NT) * n + k] = acc[j][k];
}

// dweight from the workers' shares: 64 columns a work-group, 16 threads a column.
__global__ __launch_bounds__(1024) void norm_join_kernel(const float *part, int G, int d, float *dweight)
{
    __shared__ double room[16][kWave];
    const int at = blockIdx.x * kWave + lane_id(), slice = threadIdx.x / kWave;
    double v = 0.0;
    if (at < d)
        for (int g = slice; g < G; g += 16)
            v += (double)part[(long)g * d + at];
    room[slice][lane_id()] = v;
    __syncthreads();
    if (slice == 0 && at < d) {
#pragma unroll
        for (int i = 1; i < 16; ++i)
            v += room[i][lane_id()];
        dweight[at] = (float)v;
    }
}

// Threads and chunks a thread for rows of `chunks` 16-byte chunks.
template <typename F> void with_shape(int chunks, F &&f)
{
    if (chunks <= 64)
        f.template operator()<64, 1>();
    else if (chunks <= 128)
        f.template operator()<64, 2>();
    else if (chunks <= 256)
        f.template operator()<256, 1>();
    else if (chunks <= 512)
        f.template operator()<256, 2>();
    else if (chunks <= 1024)
        f.template operator()<256, 4>();
    else if (chunks <= 2048)
        f.template operator()<512, 4>();
    else if (chunks <= 4096)
        f.template operator()<1024, 4>();
    else
        f.template operator()<1024, 8>();
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
    template <int NT, int NV> void operator()() const
    {
        const int per = NT < 256 ? 256 / NT : 1;
        hipLaunchKernelGGL((norm_kernel<T, NT, NV, M>), grid_of(((long)a.T + per - 1) / per),
                           dim3(NT * per), 0, st, a);
    }
};
template <typename T> struct RunGrad {
    const NormGradArgs &a;
    int G;
    hipStream_t st;
    template <int NT, int NV> void operator()() const
    {
        const int per = NT < 256 ? 256 / NT : 1;
        hipLaunchKernelGGL((norm_grad_kernel<T, NT, NV>), grid_of(((long)G + per - 1) / per),
                           dim3(NT * per), 0, st, a, G);
    }
};

template <typename T> void run_norm(const NormArgs &a, hipStream_t st)
{
    const int chunks = chunks_of(a.d, a.dtype);
    if (!a.q)
        with_shape(chunks, RunNorm<T, kTyped>{a, st});
    else if (a.norm)
        with_shape(chunks, RunNorm<T, kEight>{a, st});
    else
        with_shape(chunks, RunNorm<T, kEightPlain>{a, st});
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
    const int per = rows_per_group(chunks_of(d, dtype));
    return std::min((T + per - 1) / per * per, 1024);
}

hipError_t launch_norm_backward(const NormGradArgs &a, hipStream_t st)
{
    const int G = norm_groups(a.T, a.d, a.dtype), chunks = chunks_of(a.d, a.dtype);
    if (G > 0) {
        if (a.dtype == 1)
            with_shape(chunks, RunGrad<uint16_t>{a, G, st});
        else
            with_shape(chunks, RunGrad<float>{a, G, st});
    }
    if (a.dweight)
        hipLaunchKernelGGL(norm_join_kernel, dim3((a.d + kWave - 1) / kWave), dim3(1024), 0, st,
                           a.part, G, a.d, a.dweight);
    return hipGetLastError();
}

}  // namespace sk
