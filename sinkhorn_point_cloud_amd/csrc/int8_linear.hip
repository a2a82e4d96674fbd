// int8_linear.hip -- product of 8-bit integers with a scale for each token and each
// channel: out[t][n] = xscale[t] wscale[n] sum_k x[t][k] w[n][k] + bias[n].
//
// The sums are exact 32-bit integers, so any split of the K axis gives the same
// result.  Matrix instructions take both operands with K along a row, 16 bytes a
// lane.  Channels are the rows of an instruction's result and tokens its columns:
// a lane then holds four channels of one token side by side.
//
// Tiles of both operands go through shared memory, some stages of K ahead of the
// products, also for a few tokens: the copies keep more bytes on their way than loads
// to registers do (4 x 4096 to 131072: 106 us against 140 of a kernel that streams
// weights to registers with a wave's 16 rows, 110 with 32 rows).  A few tokens and a
// few channels leave too few tiles to fill the device; there four waves share 16
// channels along K.
#include "head.h"

#include <algorithm>

namespace sk {
namespace {

typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef i32x4 __attribute__((aligned(2))) i32x4_a2;
typedef i32x4 __attribute__((aligned(4))) i32x4_a4;
typedef int i32x16 __attribute__((ext_vector_type(16)));

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

// --- few tokens and channels: weights from memory to registers

constexpr int kDeep = 4;   // steps of 64 bytes that are asked for together

// 16 channels and 16 tokens a work-group; its 4 waves take every fourth piece of kDeep
// steps along K and their sums are joined in shared memory.
template <typename O> __global__ __launch_bounds__(256) void stream_kernel(Args g)
{
    const ProductArgs &a = g.a;
    __shared__ i32x4 room[3][kWave];
    const int lane = lane_id(), wave = wave_id_uniform(), row = lane & 15, quad = lane >> 4;
    const int n0 = blockIdx.x * 16;
    const int8_t *w = a.w + (long)min(n0 + row, a.N - 1) * a.ldw + quad * 16;
    const int8_t *x = a.x + (long)min(row, a.T - 1) * a.ldx + quad * 16;
    i32x4 acc = {0, 0, 0, 0};
    const int whole = a.K / 64;   // steps without an end of a row
    int s = wave * kDeep;
    for (; s + kDeep <= whole; s += 4 * kDeep) {
        i32x4 wv[kDeep], xv[kDeep];
#pragma unroll
        for (int k = 0; k < kDeep; ++k) {
            wv[k] = __builtin_nontemporal_load(reinterpret_cast<const i32x4 *>(w + (long)(s + k) * 64));
            xv[k] = load16(x + (long)(s + k) * 64);
        }
#pragma unroll
        for (int k = 0; k < kDeep; ++k)
            acc = __builtin_amdgcn_mfma_i32_16x16x64_i8(wv[k], xv[k], acc, 0, 0, 0);
    }
    // the wave whose piece holds the end: its steps one by one
    for (const int last = min(s + kDeep, (a.K + 63) / 64); s < last; ++s) {
        const int live = a.K - s * 64 - quad * 16;   // bytes of this lane's 16
        const i32x4 none = {0, 0, 0, 0};
        const i32x4 wv = live > 0 ? load16(w + (long)s * 64) : none;
        const i32x4 xv = live > 0 ? load16(x + (long)s * 64) & byte_mask(live) : none;
        acc = __builtin_amdgcn_mfma_i32_16x16x64_i8(wv, xv, acc, 0, 0, 0);
    }
    if (wave > 0)
        room[wave - 1][lane] = acc;
    __syncthreads();
    if (wave > 0 || row >= a.T)
        return;
#pragma unroll
    for (int k = 0; k < 3; ++k)
        acc += room[k][lane];
    O *out = (O *)a.out + row * a.ldo;
    const float xs = a.xscale[row];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const int n = n0 + quad * 4 + k;
        if (n < a.N) {
            const float y = (float)acc[k] * (xs * a.wscale[n]);
            out[n] = (O)(a.bias ? y + a.bias[n] : y);
        }
    }
}

// --- tiles in shared memory

// 16 bytes a lane into shared memory, a wave's KB in a run from `to` on.  In asm, so
// that reads of other stages do not wait for it; the waits are in wait_stage().  (A
// write of m0 needs a wait state before the load that reads it.)
__device__ __forceinline__ void copy16(const int8_t *from, uint32_t to)
{
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, off" ::"s"(to), "v"(from)
                 : "memory", "m0");
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

// 16 bytes of results.
template <typename O, int n> struct Run {
    O v[n];
};
// To any address that suits their type, past the caches that hold the operands (333 x
// 1500 to 50001 fp32 77 us through them, 51 past them; 4096 x 256 to 64000 bf16 251 and
// 191).
__device__ __forceinline__ void put_run(float *p, i32x4 v)
{
    __builtin_nontemporal_store(v, reinterpret_cast<i32x4_a4 *>(p));
}
__device__ __forceinline__ void put_run(__bf16 *p, i32x4 v)
{
    __builtin_nontemporal_store(v, reinterpret_cast<i32x4_a2 *>(p));
}

// The channels of a run that a lane writes: n0 + at on, of `live`.
template <typename O, int Cols> struct Channels {
    static constexpr int n = 16 / (int)sizeof(O), lanes = Cols / n;
    float ws[n], bias[n];
    int at, live;
    __device__ __forceinline__ Channels(const ProductArgs &a, int n0)
        : at(lane_id() % lanes * n), live(a.N - n0 - at)
    {
#pragma unroll
        for (int k = 0; k < n; ++k) {
            const int c = min(n0 + at + k, a.N - 1);
            ws[k] = a.wscale[c];
            bias[k] = a.bias ? a.bias[c] : 0.f;
        }
    }
};

// 32 tokens' sums from a wave's room, scaled, to the result; a token's scale lies behind
// its sums.
template <typename O, int Cols>
__device__ __forceinline__ void put_rows(const ProductArgs &a, const Channels<O, Cols> &c, const int32_t *room,
                                         int pitch, int t0, int n0)
{
    constexpr int n = Channels<O, Cols>::n, lanes = Channels<O, Cols>::lanes, rows = kWave / lanes;
    if (c.live <= 0)
        return;
    O *out = (O *)a.out + n0 + c.at;
    const bool bias = a.bias != nullptr;
#pragma unroll
    for (int i = 0; i < 32 / rows; ++i) {
        const int r = i * rows + lane_id() / lanes, t = t0 + r;
        if (t < a.T) {
            const float xs = __int_as_float(room[r * pitch + Cols]);
            Run<O, n> v;
#pragma unroll
            for (int k = 0; k < n; k += 4) {
                const i32x4 sum = *reinterpret_cast<const i32x4 *>(room + r * pitch + c.at + k);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float y = (float)sum[e] * (xs * c.ws[k + e]);
                    v.v[k + e] = (O)(bias ? y + c.bias[k + e] : y);
                }
            }
            O *p = out + t * a.ldo;
            if (c.live >= n) {
                put_run(p, __builtin_bit_cast(i32x4, v));
            } else {
#pragma unroll
                for (int k = 0; k < n; ++k)
                    if (k < c.live)
                        p[k] = v.v[k];
            }
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

// A tile of BT tokens and BN channels, a quarter for each wave; `Stages` stages of
// `Bytes` bytes of K in shared memory.
template <typename O, int BT, int BN, int Bytes, int Stages, int Occ>
__global__ __launch_bounds__(256, Occ) void tile_kernel(Args g)
{
    // a stage's rows are Bytes apart; chunk c of 16 bytes lies at c ^ turn(row), so that
    // 16 rows' chunks c cover all 64 banks
    constexpr int rows = BT + BN, stage = rows * Bytes, per_row = Bytes / 16;
    constexpr int loads = rows * per_row / 256, subs = Bytes / 32;
    constexpr int TT = BT / 64, TN = BN / 64;   // 32 x 32 results of a wave
    auto turn = [](int row) { return Bytes == 64 ? row >> 2 & 3 : row >> 1 & 7; };
    extern __shared__ char lds[];               // [Stages][stage]
    const ProductArgs &a = g.a;
    const int lane = lane_id(), wave = wave_id_uniform();
    // tiles in bands of 4 along the tokens, channels across; a run of them to each XCD.
    // (4096 x 4096 to 131072: 2.31 ms, bands of 1, 2, 8 and 16 2.56, 2.35, 2.39, 2.53: work-groups
    // that run at once share tiles of both operands, and write beside one another rather
    // than below, in rows a power of two apart.)
    const int tiles_t = (a.T + BT - 1) / BT, tiles_n = (a.N + BN - 1) / BN;
    const long all = (long)tiles_t * tiles_n, per = (all + 7) / 8;
    const long b = blockIdx.x % 8 * per + blockIdx.x / 8;
    if (blockIdx.x / 8 >= per || b >= all)
        return;
    constexpr int kBand = 4;
    const long band = b / ((long)kBand * tiles_n), in = b - band * kBand * tiles_n;
    const int high = min(kBand, tiles_t - (int)band * kBand);
    const int t0 = ((int)band * kBand + (int)(in % high)) * BT, n0 = (int)(in / high) * BN;
    // this part's stages along K
    const int chunks = (a.K + 15) / 16, steps = (a.K + Bytes - 1) / Bytes;
    const int each = (steps + g.parts - 1) / g.parts;
    const int first = min((int)blockIdx.y * each, steps), count = min(each, steps - first);

    const int8_t *from[loads];
    const int sub = lane / per_row, chunk = lane % per_row ^ turn(sub);
    static_assert(64 / per_row % (Bytes == 64 ? 16 : 8) == 0);   // turn(row) is that of sub, or
    const int odd = Bytes == 64 ? 0 : 4;                          // of 8 rows more: ^ 4
#pragma unroll
    for (int i = 0; i < loads; ++i) {
        const int r = (i * 4 + wave) * (64 / per_row) + sub;   // of the stage: tokens, then channels
        from[i] = r < BT ? a.x + (long)min(t0 + r, a.T - 1) * a.ldx
                         : a.w + (long)min(n0 + r - BT, a.N - 1) * a.ldw;
        from[i] += (long)first * Bytes + (chunk ^ (wave & 1 ? odd : 0)) * 16;
    }
    const int mine = chunk ^ (wave & 1 ? odd : 0);
    const uint32_t base = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) char *)lds;
    // Piece p of `subs` of the copies of stage k: of whole chunks, or any stage's.
    auto copy = [&](int k, int i) {
        copy16(from[i], base + (k % Stages) * stage + wave * 1024 + i * 4096);
        from[i] += Bytes;
    };
    auto issue = [&](int k, int p0, int p1) {
        if (k >= count)
            return;
        const bool there = (first + k) * per_row + mine < chunks;   // else behind the rows' end: zeros
#pragma unroll
        for (int i = 0; i < loads; ++i)
            if (i >= p0 * loads / subs && i < p1 * loads / subs) {
                copy16(there ? from[i] : (const int8_t *)kZeros,
                       base + (k % Stages) * stage + wave * 1024 + i * 4096);
                from[i] += Bytes;
            }
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
    int at[subs];   // of this lane's 16 bytes, for each 32 bytes of a stage
#pragma unroll
    for (int s = 0; s < subs; ++s)
        at[s] = r32 * Bytes + ((2 * s + half) ^ turn(r32)) * 16;
    // the scales that the results will need
    constexpr int cols = BN / 2, pitch = cols + 4;   // 16 tokens' stores cover all banks
    const int nw = n0 + wn * cols;
    const Channels<O, cols> channels(a, nw);
    float xs[TT];
#pragma unroll
    for (int j = 0; j < TT; ++j)
        xs[j] = a.xscale[min(t0 + wt * (BT / 2) + j * 32 + r32, a.T - 1)];
    const int xrow = wt * (BT / 2) * Bytes, wrow = (BT + wn * (BN / 2)) * Bytes;
    i32x4 wf[2][TN], xf[2][TT];
    // Operand r of the TN + TT of piece s of stage k.
    auto fetch = [&](int k, int s, int r) {
        const char *p = lds + (k % Stages) * stage + at[s];
        if (r < TN)
            wf[s & 1][r] = *reinterpret_cast<const i32x4 *>(p + wrow + r * 32 * Bytes);
        else
            xf[s & 1][r - TN] = *reinterpret_cast<const i32x4 *>(p + xrow + (r - TN) * 32 * Bytes);
    };
    auto fetch_all = [&](int k, int s) {
#pragma unroll
        for (int r = 0; r < TN + TT; ++r)
            fetch(k, s, r);
    };
    auto multiply = [&](int s, int m) {
        const int i = m / TT, j = m % TT;
        acc[i][j] = __builtin_amdgcn_mfma_i32_32x32x32_i8(wf[s & 1][i], xf[s & 1][j], acc[i][j], 0, 0, 0);
    };
    auto multiply_all = [&](int s) {
#pragma unroll
        for (int m = 0; m < TN * TT; ++m)
            multiply(s, m);
    };
    // Piece s multiplied, with the reads of the next piece (n of stage kn) and piece p of
    // the copies of stage kc between the products: the matrix cores never wait for the
    // issue of either.
    auto step = [&](int s, int kn, int n, int kc, int p) {
        constexpr int M = TN * TT, R = TN + TT;
#pragma unroll
        for (int m = 0; m < M; ++m) {
#pragma unroll
            for (int r = 0; r < R; ++r)
                if (r * (M / 2) / R == m)
                    fetch(kn, n, r);
            const int c0 = p * loads / subs, c = (p + 1) * loads / subs - c0;
#pragma unroll
            for (int i = 0; i < loads; ++i)
                if (i >= c0 && i < c0 + c && M / 2 + (i - c0) * (M / 2) / c == m)
                    copy(kc, i);
            multiply(s, m);
            __builtin_amdgcn_sched_barrier(0);
        }
    };
    // what lies behind the rows' end in their last chunk counts as zeros
    auto mask = [&](int s) {
        const i32x4 m = byte_mask(a.K - (steps - 1) * Bytes - (2 * s + half) * 16);
#pragma unroll
        for (int j = 0; j < TT; ++j)
            xf[s & 1][j] &= m;
    };
    if (count > 0) {
        // all stages but the last whole, of that the first piece
#pragma unroll
        for (int k = 0; k < Stages; ++k)
            issue(k, 0, k + 1 < Stages ? subs : 1);
        if (count >= Stages)
            wait_stage<(Stages - 2) * loads + loads / subs>();
        else
            wait_stage<0>();
        fetch_all(0, 0);
        int k = 0;
        for (; k + Stages + 1 < count; ++k) {
#pragma unroll
            for (int s = 0; s + 1 < subs; ++s)
                step(s, k, s + 1, k + Stages - 1, s + 1);
            // stage k + 1 is there for all, and nobody reads stage k any more
            wait_stage<(Stages - 2) * loads>();
            step(subs - 1, k + 1, 0, k + Stages, 0);
        }
#pragma unroll 1
        for (; k < count; ++k) {
            const bool end = k + 1 == count && a.K % 16 && first + count == steps;
#pragma unroll
            for (int s = 0; s + 1 < subs; ++s) {
                issue(k + Stages - 1, s + 1, s + 2);
                fetch_all(k, s + 1);
                if (end)
                    mask(s);
                multiply_all(s);
            }
            if (end)
                mask(subs - 1);
            if (k + 1 < count) {
                if (k + Stages <= count)
                    wait_stage<(Stages - 2) * loads>();
                else
                    wait_stage<0>();
            }
            issue(k + Stages, 0, 1);
            multiply_all(subs - 1);
            fetch_all(k + 1, 0);   // behind the last stage: an older one, for nothing
        }
    }
    // A lane holds four channels of a token, and 32 tokens' rows of 16 bytes would be
    // written at once: the sums go through shared memory, 32 tokens at a time and each
    // wave in its own room, and leave in runs of a wave's BN / 2 channels.  (4096 x 4096
    // to 131072 in bf16: 3.69 ms without it.)
    __syncthreads();
    int32_t *room = reinterpret_cast<int32_t *>(lds) + wave * 32 * pitch;
#pragma unroll
    for (int j = 0; j < TT; ++j) {
        if (half == 0)
            room[r32 * pitch + cols] = __float_as_int(xs[j]);
#pragma unroll
        for (int i = 0; i < TN; ++i)
#pragma unroll
            for (int q = 0; q < 4; ++q)
                *reinterpret_cast<i32x4 *>(room + r32 * pitch + i * 32 + q * 8 + half * 4) =
                    i32x4{acc[i][j][4 * q], acc[i][j][4 * q + 1], acc[i][j][4 * q + 2], acc[i][j][4 * q + 3]};
        wave_fence();
        const int tw = t0 + wt * (BT / 2) + j * 32;
        if (g.parts == 1)
            put_rows<O, cols>(a, channels, room, pitch, tw, nw);
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

// Which kernel, and the tile.  256 x 256 where such tiles fill the compute units and K is
// long enough for what surrounds the products to be small: 8192 x 8192 to 8192 475 us
// against 677 with 128 x 128.  Else work-groups that share a compute unit hide it: 256 x
// 128, two of them, where the tokens fill such tiles (4096 x 1024 to 131072 844 us against
// 937 with 128 x 128 and 892 with 256 x 256, 1000 x 1000 to 30000 52 against 59 and 55), or
// 128 x 128, three of them (333 x 1500 to 50001 51 us against 64 and 67).  For up to 64
// tokens, whose tiles are read for the weights' sake, 64 x 128, or 64 x 64 split along K
// where the channels are few (with weights that no cache holds, 64 x 64 and 64 x 128:
// 64 x 14336 to 4096 26 and 75 us, 40 x 8192 to 32000 64 and 61, to 50000 116 and 97).
enum Shape { kStream, kTiles64, kTiles64x128, kTiles128, kTiles256x128, kTiles256 };
long tiles_of(int T, int N, int BT, int BN) { return ((long)T + BT - 1) / BT * (((long)N + BN - 1) / BN); }
Shape shape_of(int T, int K, int N)
{
    if (T <= 16 && N <= 8192)
        return kStream;
    if (T <= 64)
        return N < 32768 ? kTiles64 : kTiles64x128;
    if (T > 128 && K >= 2048 && tiles_of(T, N, 256, 256) >= 192)
        return kTiles256;
    const long padded = ((long)T + 255) / 256 * 256;
    return K < 2048 && padded <= T * 1.15 && tiles_of(T, N, 256, 128) >= 384 ? kTiles256x128 : kTiles128;
}

template <typename O, int BT, int BN, int Bytes, int Stages, int Occ>
void run_tiles(const Args &g, hipStream_t st)
{
    const long all = tiles_of(g.a.T, g.a.N, BT, BN);
    const size_t stages = (size_t)Stages * (BT + BN) * Bytes, sums = (size_t)4 * 32 * (BN / 2 + 4) * 4;
    hipLaunchKernelGGL((tile_kernel<O, BT, BN, Bytes, Stages, Occ>),
                       dim3((unsigned)((all + 7) / 8 * 8), g.parts), dim3(256), std::max(stages, sums), st, g);
    if (g.parts > 1)
        hipLaunchKernelGGL((join_kernel<O>), dim3((g.a.N + 255) / 256, std::min(g.a.T, 32768)), dim3(256), 0,
                           st, g);
}

template <typename O> void run_product(const Args &g, hipStream_t st)
{
    switch (shape_of(g.a.T, g.a.K, g.a.N)) {
    case kStream:
        hipLaunchKernelGGL((stream_kernel<O>), dim3((g.a.N + 15) / 16), dim3(256), 0, st, g);
        break;
    case kTiles64: run_tiles<O, 64, 64, 64, 4, 4>(g, st); break;
    case kTiles64x128: run_tiles<O, 64, 128, 64, 4, 3>(g, st); break;
    case kTiles128: run_tiles<O, 128, 128, 64, 3, 3>(g, st); break;
    case kTiles256x128: run_tiles<O, 256, 128, 64, 3, 2>(g, st); break;
    case kTiles256: run_tiles<O, 256, 256, 128, 2, 1>(g, st); break;
    }
}

}  // namespace

// Work-groups that share a tile along K, where there are too few tiles for the
// compute units.
int product_parts(int T, int K, int N)
{
    const Shape shape = shape_of(T, K, N);
    if (shape != kTiles64 && shape != kTiles128)
        return 1;
    const int side = shape == kTiles64 ? 64 : 128;
    const long tiles = tiles_of(T, N, side, side);
    return (int)std::max(1l, std::min({256 / std::max(tiles, 1l), (long)K / 512, 16l}));
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
