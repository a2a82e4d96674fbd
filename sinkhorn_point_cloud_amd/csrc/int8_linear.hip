// int8_linear.hip -- product of 8-bit integers with a scale for each token and each
// channel: out[t][n] = xscale[t] wscale[n] sum_k x[t][k] w[n][k] + bias[n].
//
// The sums are exact 32-bit integers, so any split of the K axis gives the same
// result.  Matrix instructions take both operands with K along a row, 16 bytes a
// lane.  Channels are the rows of an instruction's result and tokens its columns:
// a lane then holds four channels of one token side by side.
//
// Two kernels.  Up to 64 tokens the weights are what is read: each wave streams its
// own rows of them from memory to registers.  Beyond, tiles of both operands go
// through shared memory, 64 bytes of K at a time, four stages deep.
#include "head.h"

#include <algorithm>
#include <type_traits>

namespace sk {
namespace {

typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef int i32x16 __attribute__((ext_vector_type(16)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));

struct Args {
    ProductArgs a;
    int parts;   // of the K axis, over work-groups
};

// 16 bytes of zeros: what is behind a row's end.
__device__ const uint4 kZeros[1] = {{0u, 0u, 0u, 0u}};

__device__ __forceinline__ i32x4 load16(const int8_t *p) { return *reinterpret_cast<const i32x4 *>(p); }

// Mask of 16 bytes of which the first `live` count (any number).
__device__ __forceinline__ i32x4 byte_mask(int live)
{
    i32x4 m;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int n = min(max(live - 4 * i, 0), 4);
        m[i] = n == 4 ? -1 : (int)((1u << 8 * n) - 1u);
    }
    return m;
}

// Four channels n .. n + 3 of token t, of which `live` are there.
template <typename O>
__device__ __forceinline__ void put4(const ProductArgs &a, long t, int n, i32x4 sum, float xs, bool whole)
{
    const int live = min(4, a.N - n);
    if (live <= 0)
        return;
    O *out = (O *)a.out + t * a.ldo + n;
    float v[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int at = min(n + i, a.N - 1);
        v[i] = (float)sum[i] * (xs * a.wscale[at]);
        if (a.bias)
            v[i] += a.bias[at];
    }
    if (whole && live == 4) {
        if constexpr (sizeof(O) == 4)
            *reinterpret_cast<f32x4 *>(out) = f32x4{v[0], v[1], v[2], v[3]};
        else
            *reinterpret_cast<bf16x4 *>(out) =
                bf16x4{(__bf16)v[0], (__bf16)v[1], (__bf16)v[2], (__bf16)v[3]};
        return;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
        if (i < live)
            out[i] = (O)v[i];
}
// whether four channels are one aligned store
template <typename O> __device__ __forceinline__ bool whole_stores(const ProductArgs &a)
{
    return (((uintptr_t)a.out | (uintptr_t)(a.ldo * (int64_t)sizeof(O))) & (4 * sizeof(O) - 1)) == 0;
}

// --- few tokens: weights from memory to registers

constexpr int kDeep = 4;   // steps of 64 bytes that are asked for together

// RT x 16 channels and TT x 16 tokens a work-group; its 4 waves take every fourth
// piece of kDeep steps along K and their sums are joined in shared memory.
template <typename O, int RT, int TT>
__global__ __launch_bounds__(256) void stream_kernel(Args g)
{
    const ProductArgs &a = g.a;
    __shared__ i32x4 room[3][RT * TT][kWave];
    const int lane = lane_id(), wave = wave_id_uniform(), row = lane & 15, quad = lane >> 4;
    const int n0 = blockIdx.x * RT * 16, t0 = blockIdx.y * TT * 16;
    const int8_t *w[RT], *x[TT];
#pragma unroll
    for (int i = 0; i < RT; ++i)
        w[i] = a.w + (long)min(n0 + i * 16 + row, a.N - 1) * a.ldw + quad * 16;
#pragma unroll
    for (int i = 0; i < TT; ++i)
        x[i] = a.x + (long)min(t0 + i * 16 + row, a.T - 1) * a.ldx + quad * 16;
    i32x4 acc[RT][TT];
#pragma unroll
    for (int i = 0; i < RT; ++i)
#pragma unroll
        for (int j = 0; j < TT; ++j)
            acc[i][j] = i32x4{0, 0, 0, 0};
    const int whole = a.K / 64;   // steps without an end of a row
    int s = wave * kDeep;
    for (; s + kDeep <= whole; s += 4 * kDeep) {
        i32x4 wv[kDeep][RT], xv[kDeep][TT];
#pragma unroll
        for (int k = 0; k < kDeep; ++k) {
#pragma unroll
            for (int i = 0; i < RT; ++i)
                wv[k][i] = __builtin_nontemporal_load(reinterpret_cast<const i32x4 *>(w[i] + (long)(s + k) * 64));
#pragma unroll
            for (int j = 0; j < TT; ++j)
                xv[k][j] = load16(x[j] + (long)(s + k) * 64);
        }
#pragma unroll
        for (int k = 0; k < kDeep; ++k)
#pragma unroll
            for (int i = 0; i < RT; ++i)
#pragma unroll
                for (int j = 0; j < TT; ++j)
                    acc[i][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(wv[k][i], xv[k][j], acc[i][j], 0, 0, 0);
    }
    // the wave whose piece holds the end: its steps one by one
    for (const int last = min(s + kDeep, (a.K + 63) / 64); s < last; ++s) {
        const int live = a.K - s * 64 - quad * 16;   // bytes of this lane's 16
        const i32x4 mask = byte_mask(live);
        i32x4 wv[RT], xv[TT];
#pragma unroll
        for (int i = 0; i < RT; ++i)
            wv[i] = live > 0 ? load16(w[i] + (long)s * 64) : i32x4{0, 0, 0, 0};
#pragma unroll
        for (int j = 0; j < TT; ++j)
            xv[j] = live > 0 ? load16(x[j] + (long)s * 64) & mask : i32x4{0, 0, 0, 0};
#pragma unroll
        for (int i = 0; i < RT; ++i)
#pragma unroll
            for (int j = 0; j < TT; ++j)
                acc[i][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(wv[i], xv[j], acc[i][j], 0, 0, 0);
    }
    if (wave > 0) {
#pragma unroll
        for (int i = 0; i < RT; ++i)
#pragma unroll
            for (int j = 0; j < TT; ++j)
                room[wave - 1][i * TT + j][lane] = acc[i][j];
    }
    __syncthreads();
    if (wave > 0)
        return;
    const bool even = whole_stores<O>(a);
#pragma unroll
    for (int j = 0; j < TT; ++j) {
        const int t = t0 + j * 16 + row;
        if (t >= a.T)
            continue;
        const float xs = a.xscale[t];
#pragma unroll
        for (int i = 0; i < RT; ++i) {
            i32x4 sum = acc[i][j];
#pragma unroll
            for (int k = 0; k < 3; ++k)
                sum += room[k][i * TT + j][lane];
            put4<O>(a, t, n0 + i * 16 + quad * 4, sum, xs, even);
        }
    }
}

// --- many tokens: tiles in shared memory

constexpr int kStages = 4, kBytes = 64;   // stages, and bytes of K in one

// 16 bytes a lane into shared memory, a wave's KB in a run from `to` on.  In asm, so
// that reads of other stages do not wait for it; the waits are in wait_stage().  (A
// write of m0 needs a wait state before the load that reads it; nothing else here uses m0.)
__device__ __forceinline__ void copy16(const int8_t *from, uint32_t to)
{
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, off" ::"s"(to), "v"(from)
                 : "memory");
}
// Waits until all but `Left` of this wave's copies are there and its reads of shared
// memory are done, then for the other waves.
template <int Left> __device__ __forceinline__ void wait_stage()
{
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(Left) : "memory");
}

// What the lanes of a wave wrote to shared memory before it, all of them see behind it.
__device__ __forceinline__ void wave_fence()
{
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
}

// 16 bytes at any address that suits the type.
template <typename O, int n> struct alignas(sizeof(O)) Run {
    O v[n];
};

// 32 tokens' sums of Cols channels from a wave's room, scaled, to the result.
template <typename O, int Cols>
__device__ __forceinline__ void put_rows(const ProductArgs &a, const int32_t *room, int pitch, int t0, int n0,
                                         O *out, int64_t ldo)
{
    constexpr int n = 16 / (int)sizeof(O), lanes = Cols / n, rows = kWave / lanes;
    const int at = lane_id() % lanes * n, live = a.N - n0 - at;
    if (live <= 0)
        return;
    float ws[n], bias[n];
#pragma unroll
    for (int k = 0; k < n; ++k) {
        const int c = n0 + at + min(k, live - 1);
        ws[k] = a.wscale[c];
        bias[k] = a.bias ? a.bias[c] : 0.f;
    }
#pragma unroll
    for (int r = lane_id() / lanes; r < 32; r += rows) {
        const int t = t0 + r;
        if (t >= a.T)
            break;
        const float xs = a.xscale[t];
        Run<O, n> v;
#pragma unroll
        for (int k = 0; k < n; k += 4) {
            const i32x4 sum = *reinterpret_cast<const i32x4 *>(room + r * pitch + at + k);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float y = (float)sum[e] * (xs * ws[k + e]);
                v.v[k + e] = (O)(a.bias ? y + bias[k + e] : y);
            }
        }
        O *p = out + t * ldo + n0 + at;
        if (live >= n) {
            *reinterpret_cast<Run<O, n> *>(p) = v;
        } else {
#pragma unroll
            for (int k = 0; k < n; ++k)
                if (k < live)
                    p[k] = v.v[k];
        }
    }
}
// The same sums as they are, for the join of parts.
template <int Cols>
__device__ __forceinline__ void put_sums(const ProductArgs &a, const int32_t *room, int pitch, int t0, int n0,
                                         int32_t *out)
{
    for (int i = lane_id(); i < 32 * Cols; i += kWave) {
        const int t = t0 + i / Cols, n = n0 + i % Cols;
        if (t < a.T && n < a.N)
            out[(long)t * a.N + n] = room[i / Cols * pitch + i % Cols];
    }
}

template <typename O, int BT, int BN>
__global__ __launch_bounds__(256, BT *BN >= 256 * 256 ? 1 : 2) void tile_kernel(Args g)
{
    // a row of a stage is 64 bytes; chunk c of 16 bytes lies at c ^ (row / 4 & 3), so
    // that 16 rows' chunks c cover all 64 banks
    constexpr int rows = BT + BN, stage = rows * kBytes, loads = rows / 64;
    constexpr int TT = BT / 64, TN = BN / 64;   // 32 x 32 results of a wave (half of the tile each way)
    extern __shared__ char lds[];               // [kStages][stage]
    const ProductArgs &a = g.a;
    const int lane = lane_id(), wave = wave_id_uniform();
    // tiles in bands of 8 along the tokens, channels across; a run of them to each XCD
    const int tiles_t = (a.T + BT - 1) / BT, tiles_n = (a.N + BN - 1) / BN;
    const long all = (long)tiles_t * tiles_n, per = (all + 7) / 8;
    const long b = blockIdx.x % 8 * per + blockIdx.x / 8;
    if (blockIdx.x / 8 >= per || b >= all)
        return;
    const long band = b / (8l * tiles_n), in = b - band * 8l * tiles_n;
    const int high = min(8, tiles_t - (int)band * 8);
    const int t0 = ((int)band * 8 + (int)(in % high)) * BT, n0 = (int)(in / high) * BN;
    // this part's stages along K
    const int chunks = (a.K + 15) / 16, steps = (a.K + kBytes - 1) / kBytes;
    const int each = (steps + g.parts - 1) / g.parts;
    const int first = min((int)blockIdx.y * each, steps), count = min(each, steps - first);

    const int8_t *from[loads];
    const int sub = lane >> 2, chunk = (lane & 3) ^ (lane >> 4 & 3);
#pragma unroll
    for (int i = 0; i < loads; ++i) {
        const int r = (i * 4 + wave) * 16 + sub;   // of the stage: tokens, then channels
        from[i] = r < BT ? a.x + (long)min(t0 + r, a.T - 1) * a.ldx
                         : a.w + (long)min(n0 + r - BT, a.N - 1) * a.ldw;
        from[i] += (long)first * kBytes + chunk * 16;
    }
    const uint32_t base = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) char *)lds;
    // a stage of whole chunks, and any stage of this part
    auto issue_whole = [&](int k) {
        const uint32_t to = base + (k % kStages) * stage + wave * 1024;
#pragma unroll
        for (int i = 0; i < loads; ++i) {
            copy16(from[i], to + i * 4096);
            from[i] += kBytes;
        }
    };
    auto issue = [&](int k) {
        if (first + k + 1 < steps || chunks % 4 == 0) {
            issue_whole(k);
            return;
        }
        // chunks behind the rows' end: zeros
        const uint32_t to = base + (k % kStages) * stage + wave * 1024;
        const bool there = (first + k) * 4 + chunk < chunks;
#pragma unroll
        for (int i = 0; i < loads; ++i)
            copy16(there ? from[i] : (const int8_t *)kZeros, to + i * 4096);
    };
    i32x16 acc[TN][TT];
#pragma unroll
    for (int i = 0; i < TN; ++i)
#pragma unroll
        for (int j = 0; j < TT; ++j)
#pragma unroll
            for (int k = 0; k < 16; ++k)
                acc[i][j][k] = 0;
    const int wt = wave & 1, wn = wave >> 1, r32 = lane & 31, half = lane >> 5;
    int at[2];   // of this lane's 16 bytes, for either half of a stage
#pragma unroll
    for (int s = 0; s < 2; ++s)
        at[s] = r32 * kBytes + ((2 * s + half) ^ (r32 >> 2 & 3)) * 16;
    const int xrow = wt * (BT / 2) * kBytes, wrow = (BT + wn * (BN / 2)) * kBytes;
    i32x4 wf[2][TN], xf[2][TT];
    auto fetch = [&](int k, int s) {
        const char *p = lds + (k % kStages) * stage + at[s];
#pragma unroll
        for (int i = 0; i < TN; ++i)
            wf[s][i] = *reinterpret_cast<const i32x4 *>(p + wrow + i * 32 * kBytes);
#pragma unroll
        for (int j = 0; j < TT; ++j)
            xf[s][j] = *reinterpret_cast<const i32x4 *>(p + xrow + j * 32 * kBytes);
    };
    auto multiply = [&](int s) {
#pragma unroll
        for (int i = 0; i < TN; ++i)
#pragma unroll
            for (int j = 0; j < TT; ++j)
                acc[i][j] = __builtin_amdgcn_mfma_i32_32x32x32_i8(wf[s][i], xf[s][j], acc[i][j], 0, 0, 0);
    };
    if (count > 0) {
#pragma unroll
        for (int k = 0; k < kStages - 1; ++k)
            if (k < count)
                issue(k);
        if (count > 2)
            wait_stage<2 * loads>();
        else
            wait_stage<0>();
        fetch(0, 0);
        // behind each wait, stage k + 1 is there for all and nobody reads stage k - 1 any more
        int k = 0;
        for (; k + 4 < count; ++k) {
            wait_stage<loads>();
            issue_whole(k + 3);
            fetch(k, 1);
            multiply(0);
            fetch(k + 1, 0);
            multiply(1);
        }
#pragma unroll 1
        for (; k + 1 < count; ++k) {
            if (k + 2 < count)
                wait_stage<loads>();
            else
                wait_stage<0>();
            if (k + 3 < count)
                issue(k + 3);
            fetch(k, 1);
            multiply(0);
            fetch(k + 1, 0);
            multiply(1);
        }
        // the last stage: what lies behind the rows' end counts as zeros
        fetch(count - 1, 1);
        if (a.K % 16 && first + count == steps) {
#pragma unroll
            for (int s = 0; s < 2; ++s) {
                const i32x4 mask = byte_mask(a.K - (steps - 1) * kBytes - (2 * s + half) * 16);
#pragma unroll
                for (int j = 0; j < TT; ++j)
                    xf[s][j] &= mask;
            }
        }
        multiply(0);
        multiply(1);
    }
    // A lane holds four channels of a token, and 32 tokens' rows of 16 bytes would be
    // written at once: the sums go through shared memory, 32 tokens at a time and each
    // wave in its own room, and leave in runs of a wave's BN / 2 channels.  (4096 x 4096
    // to 131072 in bf16: 3.69 ms without it.)
    constexpr int cols = BN / 2, pitch = cols + 4;   // 16 tokens' stores cover all banks
    static_assert(4 * 32 * pitch * 4 <= kStages * stage);
    __syncthreads();
    int32_t *room = reinterpret_cast<int32_t *>(lds) + wave * 32 * pitch;
    const int nw = n0 + wn * cols;
#pragma unroll
    for (int j = 0; j < TT; ++j) {
#pragma unroll
        for (int i = 0; i < TN; ++i)
#pragma unroll
            for (int q = 0; q < 4; ++q)
                *reinterpret_cast<i32x4 *>(room + r32 * pitch + i * 32 + q * 8 + half * 4) =
                    i32x4{acc[i][j][4 * q], acc[i][j][4 * q + 1], acc[i][j][4 * q + 2], acc[i][j][4 * q + 3]};
        wave_fence();
        const int tw = t0 + wt * (BT / 2) + j * 32;
        if (g.parts == 1)
            put_rows<O, cols>(a, room, pitch, tw, nw, (O *)a.out, a.ldo);
        else
            put_sums<cols>(a, room, pitch, tw, nw, a.part + (long)blockIdx.y * a.T * a.N);
        wave_fence();
    }
}

// Sums of the parts of the K axis.
template <typename O> __global__ __launch_bounds__(256) void join_kernel(Args g)
{
    const ProductArgs &a = g.a;
    const long t = blockIdx.y, step = (long)a.T * a.N;
    const int n = blockIdx.x * 256 + threadIdx.x;
    for (long row = t; row < a.T; row += gridDim.y) {
        if (n >= a.N)
            continue;
        int sum = 0;
        for (int p = 0; p < g.parts; ++p)
            sum += a.part[p * step + row * a.N + n];
        float v = (float)sum * (a.xscale[row] * a.wscale[n]);
        if (a.bias)
            v += a.bias[n];
        ((O *)a.out)[row * a.ldo + n] = (O)v;
    }
}

constexpr int kStreamTokens = 64;

template <typename O, int RT, int TT> void run_stream(const Args &g, hipStream_t st)
{
    const dim3 grid((g.a.N + RT * 16 - 1) / (RT * 16), (g.a.T + TT * 16 - 1) / (TT * 16));
    hipLaunchKernelGGL((stream_kernel<O, RT, TT>), grid, dim3(256), 0, st, g);
}
template <typename O, int BT, int BN> void run_tiles(const Args &g, hipStream_t st)
{
    const long all = ((long)g.a.T + BT - 1) / BT * (((long)g.a.N + BN - 1) / BN);
    const size_t room = (size_t)kStages * (BT + BN) * kBytes;
    hipLaunchKernelGGL((tile_kernel<O, BT, BN>), dim3((unsigned)((all + 7) / 8 * 8), g.parts), dim3(256),
                       room, st, g);
    if (g.parts > 1)
        hipLaunchKernelGGL((join_kernel<O>), dim3((g.a.N + 255) / 256, std::min(g.a.T, 32768)), dim3(256), 0,
                           st, g);
}

// Tiles of 256 x 256 where they fill the compute units, else of 128 x 128.
bool large_tiles(int T, int N)
{
    return ((long)T + 255) / 256 * (((long)N + 255) / 256) >= 256;
}

template <typename O> void run_product(const Args &g, hipStream_t st)
{
    const int T = g.a.T;
    if (T <= 16)
        run_stream<O, 1, 1>(g, st);
    else if (T <= 32)
        run_stream<O, 2, 2>(g, st);
    else if (T <= kStreamTokens)
        run_stream<O, 2, 4>(g, st);
    else if (large_tiles(T, g.a.N))
        run_tiles<O, 256, 256>(g, st);
    else
        run_tiles<O, 128, 128>(g, st);
}

}  // namespace

// Work-groups that share a tile along K, where there are too few tiles for the
// compute units.
int product_parts(int T, int K, int N)
{
    if (T <= kStreamTokens || large_tiles(T, N))
        return 1;
    const long tiles = ((long)T + 127) / 128 * (((long)N + 127) / 128);
    return (int)std::max(1l, std::min({256 / tiles, (long)K / (8 * kBytes), 16l}));
}

hipError_t launch_product(const ProductArgs &a, hipStream_t st)
{
    const Args g{a, product_parts(a.T, a.K, a.N)};
    if (a.dtype == 1)
        run_product<__bf16>(g, st);
    else
        run_product<float>(g, st);
    return hipGetLastError();
}

}  // namespace sk
