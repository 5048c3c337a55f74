// MXFP4 (OCP microscaling, 4-bit floating point): row codes, and the LM head on them.
//
// A row of d elements is cut into blocks of 32 (the last one filled up with zeros).  With amax
// the largest magnitude of a block,
//   e = clamp(floor(log2(amax)) - 2, -127, 127),  scale byte = e + 127 (E8M0),
//   code_k = the E2M1 value nearest to x_k 2^-e (ties to the even code, at most 6),
// so a code's value is 0, 0.5, 1, 1.5, 2, 3, 4 or 6 with a sign, and amax 2^-e lies in [4, 8): what
// is above 6 there is taken to 6, the rule of the format's specification.  x 2^-e is
// exact.  A block of zeros has scale byte 0; a block holding a NaN or an infinity has scale byte
// 255 (NaN) and codes 0.  Two codes make a byte, the even element in its low half.
//
// The product is out[i, v] = sum_b 2^(eh + ew) sum_{k in b} h_k w_k.  v_mfma_scale_f32_16x16x128
// multiplies four blocks a time: of each eight in turn, lanes (r, g) of the first instruction hold
// the 16 bytes of row r's block 2 g and their scale byte, those of the second block 2 g + 1.
// Products of codes are exact and sums are fp32; every form below adds the blocks in this order
// and so gives the same bits.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <type_traits>
#include <utility>

#include "launch.h"
#include "launch_head.h"
#include "row_ops.h"

namespace mosaic {
namespace {

using namespace rows;

typedef int i32x4_t __attribute__((ext_vector_type(4)));
typedef int i32x8_t __attribute__((ext_vector_type(8)));
typedef uint16_t u16x2_t __attribute__((ext_vector_type(2)));

// Eight consecutive elements of a row.
template <bool BF16>
struct Eight {
    Raw<BF16> r[8 / kChunk<BF16>];

    __device__ __forceinline__ void load(const void *row, int k, int d)
    {
        constexpr int N = kChunk<BF16>;
#pragma unroll
        for (int i = 0; i < 8 / N; ++i) {
            const int at = k + i * N;
            if (at + N <= d) {
                r[i].load(row, at);
            } else {
                r[i].fill(0.0f);
                if (at < d)
                    r[i].load_part(row, at, d - at);
            }
        }
    }
    __device__ __forceinline__ void get(float (&x)[8]) const
    {
        constexpr int N = kChunk<BF16>;
#pragma unroll
        for (int i = 0; i < 8 / N; ++i) {
            float y[N];
            r[i].get(y);
#pragma unroll
            for (int e = 0; e < N; ++e)
                x[i * N + e] = y[e];
        }
    }
};

// 2^lpr threads (4 to 256) take a row, eight elements a thread and turn and four threads a block,
// and a workgroup 256 >> lpr rows.  `values` may be X: each element is read and written by the same thread.
template <bool BF16>
__global__ __launch_bounds__(256) void quantize_mxfp4_kernel(const void *X, int64_t nsrc, int32_t d, int32_t blocks, int lpr,
                                                             const int32_t *__restrict__ row_idx, int64_t rows,
                                                             uint8_t *__restrict__ q, uint8_t *__restrict__ scale,
                                                             void *values)
{
    constexpr int ES = BF16 ? 2 : 4, UN = 2;
    const int t = threadIdx.x & ((1 << lpr) - 1), each = 256 >> lpr, chunks = blocks * 4;
    for (int64_t row = (int64_t)blockIdx.x * each + (threadIdx.x >> lpr); row < rows; row += (int64_t)gridDim.x * each) {
        const int64_t src = row_idx ? (int64_t)row_idx[row] : row;
        const bool inside = src >= 0 && src < nsrc;   // a row id outside gives a row of NaN
        const char *from = (const char *)X + (inside ? src : 0) * d * ES;
        for (int c0 = t; c0 < chunks; c0 += UN << lpr) {
            Eight<BF16> in[UN];
#pragma unroll
            for (int u = 0; u < UN; ++u)
                if (c0 + (u << lpr) < chunks)
                    in[u].load(from, (c0 + (u << lpr)) * 8, d);
#pragma unroll
            for (int u = 0; u < UN; ++u) {
                const int c = c0 + (u << lpr);
                if (c >= chunks)   // (the four threads of a block alike)
                    continue;
                float x[8];
                in[u].get(x);
                uint32_t top = 0;
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    top = max(top, __builtin_bit_cast(uint32_t, x[e]) & 0x7fffffffu);
                top = max(top, (uint32_t)__shfl_xor((int)top, 1, 64));
                top = max(top, (uint32_t)__shfl_xor((int)top, 2, 64));
                const int field = (int)(top >> 23);   // of the exponent: amax lies in [2^(field - 127), twice that)
                const bool fine = field != 255 && inside;
                const int byte = fine ? max(field - 2, 0) : 255;
                const float down = __builtin_bit_cast(float, (uint32_t)(254 - byte) << 23);
                uint32_t w = 0;
                if (fine) {
                    float y[8];
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        y[e] = __builtin_amdgcn_fmed3f(x[e] * down, -6.0f, 6.0f);
                    // v_cvt_scalef32_pk_fp4_f32 rounds to nearest even
                    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(0u, y[0], y[1], 1.0f, 0);
                    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, y[2], y[3], 1.0f, 1);
                    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, y[4], y[5], 1.0f, 2);
                    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, y[6], y[7], 1.0f, 3);
                }
                if (q)
                    *(uint32_t *)(q + (row * blocks + (c >> 2)) * 16 + (c & 3) * 4) = w;
                if (scale && (c & 3) == 0)
                    scale[row * blocks + (c >> 2)] = (uint8_t)byte;
                if (values) {
                    const float up = !fine ? __builtin_nanf("")
                                           : (byte ? __builtin_bit_cast(float, (uint32_t)byte << 23) : 0x1p-127f);
                    float v[8];
                    auto pair = [&](auto i) __attribute__((always_inline)) {
                        const auto p = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, decltype(i)::value);
                        v[2 * i] = p[0] * up;
                        v[2 * i + 1] = p[1] * up;
                    };
                    pair(std::integral_constant<int, 0>{});
                    pair(std::integral_constant<int, 1>{});
                    pair(std::integral_constant<int, 2>{});
                    pair(std::integral_constant<int, 3>{});
                    constexpr int N = kChunk<BF16>;
                    char *to = (char *)values + row * d * ES;
#pragma unroll
                    for (int i = 0; i < 8 / N; ++i)
                        if (c * 8 + i * N < d)
                            store_upto<BF16>(to, c * 8 + i * N, *(float(*)[N])&v[i * N], d - c * 8 - i * N);
                }
            }
        }
    }
}

// c + a b of four blocks, with the scale bytes sa of a's register and sb of b's.
template <int SA, int SB>
__device__ __forceinline__ f32x4_t mfma_fp4(const i32x4_t &a, const i32x4_t &b, const f32x4_t &c, int scale_a, int scale_b)
{
    const i32x8_t x = __builtin_shufflevector(a, a, 0, 1, 2, 3, -1, -1, -1, -1);
    const i32x8_t y = __builtin_shufflevector(b, b, 0, 1, 2, 3, -1, -1, -1, -1);
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(x, y, c, 4, 4, SA, scale_a, SB, scale_b);
}

// s_waitcnt vmcnt(N) lgkmcnt(0)
template <int N>
__device__ __forceinline__ void wait_vm()
{
    static_assert(N >= 0 && N < 64, "vmcnt range");
    __builtin_amdgcn_s_waitcnt((N & 0xF) | (0x7 << 4) | (0x0 << 8) | ((N >> 4) << 14));
}

// Workgroup barrier without the fence of __syncthreads(), which would wait for the requests
// in flight.
__device__ __forceinline__ void bar()
{
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
}

typedef __attribute__((address_space(3))) void lds_void_t;

// Requests straight to LDS: 16 bytes per lane, lane i's to lds + 16 i (STREAM: streaming cache
// policy).
template <bool STREAM>
__device__ __forceinline__ void request(const void *src, void *lds)
{
    __builtin_amdgcn_global_load_lds(src, (lds_void_t *)lds, 16, 0, STREAM ? 2 : 0);
}

// Where the eight 16-byte blocks of a row's K tile lie in its 128 bytes of LDS: block 2 g + s, which
// lanes (r, g) read for sub-step s, at place (4 s + g) ^ swizzle(r).  A 16-byte read goes through
// the LDS in groups of 16 lanes that mix neighbouring g; the sub-step in the place's high bit and the
// row's swizzle keep each group on 64 different banks (with 2 g + s as the place, 44% of the LDS'
// cycles were conflicts).
__device__ __forceinline__ int swizzle(int row) { return (row >> 1) & 7; }
// the block at place `place` of a row
__device__ __forceinline__ int block_at(int place, int row)
{
    const int x = place ^ swizzle(row);
    return 2 * (x & 3) + (x >> 2);
}

// What a request past the end of a row reads: codes and scale bytes of zero.
__device__ __attribute__((aligned(16))) const uint8_t kZeroCodes[16] = {};

// Four consecutive vocabulary entries v .. v + 3 of one row; vec: the address is a multiple of
// the four values' size.
template <bool OUT_BF16>
__device__ __forceinline__ void store4(void *out, int64_t off, const f32x4_t &x, int v, int V, bool vec)
{
    if (vec && v + 3 < V) {
        if constexpr (OUT_BF16)
            *(u32x2_t *)((uint16_t *)out + off) = u32x2_t{pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3])};
        else
            *(f32x4_t *)((float *)out + off) = x;
        return;
    }
#pragma unroll
    for (int e = 0; e < 4; ++e)
        if (v + e < V)
            store1<OUT_BF16>(out, off + e, x[e]);
}

// The two scale bytes of a row's blocks b, b + 1 (b even), zeros behind the row's end, in the low
// half of a register.  WORDS: the row's bytes are whole aligned words, one of which is loaded; else,
// for rows of two blocks and more at any address, both bytes.  The loads have no branch: a row's end
// moves them back, and `get` leaves out what they read too early.  They are relaxed atomics of the
// wave's own scope, which are plain loads that the compiler leaves in their place and order: the
// kernel counts them among its requests.
template <bool WORDS>
struct ScalePair {
    int x;
    uint8_t lo, hi;

    __device__ __forceinline__ void load(const uint8_t *row, int b, int blocks)
    {
        if constexpr (WORDS) {
            x = __hip_atomic_load((const int *)(row + min(b & ~3, blocks - 4)), __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_WAVEFRONT);
        } else {
            const uint8_t *p = row + min(b, blocks - 2);
            lo = __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_WAVEFRONT);
            hi = __hip_atomic_load(p + 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_WAVEFRONT);
        }
    }
    // after the wait for the K tile
    __device__ __forceinline__ int get(int b, int blocks) const
    {
        if constexpr (WORDS) {
            int w = x;
            asm volatile("" : "+v"(w));   // or the compiler shifts before the wait, and waits for that
            return b < blocks ? w >> (8 * (b & 2)) : 0;
        }
        return (int)(lo | (uint32_t)hi << 8) >> min(8 * max(b - (blocks - 2), 0), 16);
    }
};

// Rows of a single block (d <= 32): a wave for 16 x 16 outputs, its operands straight from memory.
template <bool OUT_BF16>
__global__ __launch_bounds__(256) void gemm_mxfp4_block_kernel(const uint8_t *__restrict__ Hq,
                                                               const uint8_t *__restrict__ hs,
                                                               const int32_t *__restrict__ count, int32_t max_rows,
                                                               const uint8_t *__restrict__ Wq,
                                                               const uint8_t *__restrict__ ws, int32_t V,
                                                               void *__restrict__ out)
{
    const int rows = (int)row_count(count, max_rows);
    const int lane = threadIdx.x & 63, r = lane & 15, g = lane >> 4;
    const int64_t row_tiles = (rows + 15) / 16, tiles = row_tiles * ((V + 15) / 16);
    for (int64_t t = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6); t < tiles; t += (int64_t)gridDim.x * 4) {
        const int v0 = (int)(t / row_tiles) * 16, m0 = (int)(t % row_tiles) * 16;
        i32x4_t w = {0, 0, 0, 0}, h = w;
        int sw = 0, sh = 0;
        if (g == 0) {
            const int64_t wrow = min(v0 + r, V - 1), hrow = min(m0 + r, rows - 1);
            w = *(const i32x4_t *)(Wq + wrow * 16);
            h = *(const i32x4_t *)(Hq + hrow * 16);
            sw = ws[wrow];
            sh = hs[hrow];
        }
        const f32x4_t acc = mfma_fp4<0, 0>(w, h, f32x4_t{0.0f, 0.0f, 0.0f, 0.0f}, sw, sh);
        // lane (r, g) holds entries 4 g .. 4 g + 3 of the tile for its row r
        if (m0 + r < rows)
            store4<OUT_BF16>(out, (int64_t)(m0 + r) * V + v0 + 4 * g, acc, v0 + 4 * g, V, false);
    }
}

// Small tiles: few rows, too few 256 x 256 tiles to fill the chip, or scale rows at any address.
// BM x BV outputs per workgroup of NW waves, WGM of them side by side along the rows; K tiles of
// 128 bytes (eight blocks) a row requested straight to LDS, NSTAGE - 1 of them ahead, in a ring with
// one barrier per step, the rows' 16-byte blocks XOR-swizzled.  The scale bytes of a wave's rows come
// straight to registers, with the K tile's requests.  Several workgroups share a CU, and each goes
// from tile to tile without letting its requests run dry (4096 x 126464 x 4000, 128 x 128 tiles: 3.5 ms,
// 4.4 with a workgroup per tile).  STREAM: W is read once (one row tile): its requests take the streaming
// cache policy.
//
// 20 x 152064 x 3584: 65 us, 4.6 TB/s of codes and scales; one row 52 us, 5.5 TB/s.  Between the two
// lies the H tile, which every workgroup requests again with each W tile; tiles of 256 entries (62 us, one
// row 55; 8 x 65536 x 8192: 66 us for 59) and K tiles of 64 bytes (99 us) gain nothing over these sizes.
template <int BM, int BV, int WGM, int NSTAGE, bool STREAM, bool WORDS, bool OUT_BF16>
__global__ __launch_bounds__(256) void gemm_mxfp4_small_kernel(const uint8_t *__restrict__ Hq,
                                                               const uint8_t *__restrict__ hs,
                                                               const int32_t *__restrict__ rows_dev, int32_t max_rows,
                                                               const uint8_t *__restrict__ Wq,
                                                               const uint8_t *__restrict__ ws, int32_t V, int32_t blocks,
                                                               void *__restrict__ out, int32_t group_m)
{
    constexpr int BK = 128, CHUNKS = BK / 16, RPI = 64 / CHUNKS;
    constexpr int WGV = 4 / WGM, WM = BM / WGM, WV = BV / WGV, AM = WM / 16, AV = WV / 16;
    constexpr int W_TILE = BV * BK, STAGE = W_TILE + BM * BK;
    constexpr int LW = BV / RPI / 4, LH = BM / RPI / 4, T = LW + LH;   // requests per wave and K tile
    constexpr int TS = T + (AV + AM) * (WORDS ? 1 : 2);                 // and loads
    static_assert(LW >= 1 && LH >= 1 && NSTAGE >= 3 && (NSTAGE - 2) * TS < 64, "requests");
    __shared__ __attribute__((aligned(1024))) char smem[NSTAGE * STAGE];

    const int rows = (int)row_count(rows_dev, max_rows);
    const int nvt = (V + BV - 1) / BV, nmt = (rows + BM - 1) / BM, nblk = nvt * nmt;
    if ((int)blockIdx.x >= nblk)
        return;
    // Tile i of this workgroup: the workgroups of one XCD (the grid is a multiple of eight, or holds
    // every tile) take a contiguous run of tiles, of group_m row tiles the row tiles of a vocabulary
    // tile one after another, so that they share its W rows in that XCD's L2.
    auto tile_coords = [&](int i, int &m0, int &v0) __attribute__((always_inline)) {
        const int b = min((int)blockIdx.x + i * (int)gridDim.x, nblk - 1);
        const int q8 = nblk >> 3, rem = nblk & 7, xcd = b & 7, slot = b >> 3;
        const int t = (xcd < rem ? xcd * (q8 + 1) : rem * (q8 + 1) + (xcd - rem) * q8) + slot;
        const int first_m = t / (group_m * nvt) * group_m, gsz = min(nmt - first_m, group_m);
        const int local = t - first_m * nvt;
        m0 = (first_m + local % gsz) * BM;
        v0 = local / gsz * BV;
    };
    const int n_my = (nblk - (int)blockIdx.x + (int)gridDim.x - 1) / (int)gridDim.x;
    const int nk = (blocks + CHUNKS - 1) / CHUNKS, d = blocks * 16;

    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wv = wave % WGV, wm = wave / WGV;
    const int r16 = lane & 15, qd = lane >> 4;
    int chunk[T];
#pragma unroll
    for (int j = 0; j < T; ++j)
        chunk[j] = block_at(lane % CHUNKS, (j < LW ? wave * LW + j : wave * LH + j - LW) * RPI + lane / CHUNKS) * 16;
    // where the requests have got to: an output tile's rows, and the K tile
    const uint8_t *src[T], *scale_of[AV + AM];
    int f_tile = 0, f_kt = 0;
    auto sources = [&](int i) __attribute__((always_inline)) {
        int m0, v0;
        tile_coords(i, m0, v0);
#pragma unroll
        for (int j = 0; j < T; ++j) {
            const int r = (j < LW ? wave * LW + j : wave * LH + j - LW) * RPI + lane / CHUNKS;
            src[j] = j < LW ? Wq + (int64_t)min(v0 + r, V - 1) * d : Hq + (int64_t)min(m0 + r, rows - 1) * d;
            src[j] += chunk[j];
        }
#pragma unroll
        for (int j = 0; j < AV + AM; ++j)
            scale_of[j] = j < AV ? ws + (int64_t)min(v0 + wv * WV + j * 16 + r16, V - 1) * blocks
                                 : hs + (int64_t)min(m0 + wm * WM + (j - AV) * 16 + r16, rows - 1) * blocks;
    };
    ScalePair<WORDS> sc[NSTAGE][AV + AM];   // scale bytes of the K tiles under way: stage kt % NSTAGE
    // the next K tile into a stage (past the last one: the last tile's again, unused, so that the waits
    // need not know the end)
    auto issue = [&](int stage, ScalePair<WORDS> (&s)[AV + AM]) __attribute__((always_inline)) {
        const int kb = f_kt * BK;
#pragma unroll
        for (int j = 0; j < AV + AM; ++j)
            s[j].load(scale_of[j], f_kt * CHUNKS + 2 * qd, blocks);
#pragma unroll
        for (int j = 0; j < T; ++j) {
            const uint8_t *p = kb + chunk[j] < d && f_tile < n_my ? src[j] + kb : kZeroCodes;
            char *at = smem + stage * STAGE + (j < LW ? (wave * LW + j) * 1024 : W_TILE + (wave * LH + j - LW) * 1024);
            if (j < LW)
                request<STREAM>(p, at);
            else
                request<false>(p, at);
        }
        if (++f_kt == nk) {
            f_kt = 0;
            sources(++f_tile);
        }
    };
    f32x4_t acc[AV][AM];
#pragma unroll
    for (int a = 0; a < AV; ++a)
#pragma unroll
        for (int m = 0; m < AM; ++m)
            acc[a][m] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
    const int lane_chunk = (qd ^ swizzle(r16)) * 16;
    const int a_addr = (wv * WV + r16) * BK + lane_chunk, b_addr = W_TILE + (wm * WM + r16) * BK + lane_chunk;

    const bool vec = ((uintptr_t)out & 15) == 0 && (V & 3) == 0;
    int tile = 0, kt = 0;
    sources(0);
#pragma unroll
    for (int s = 0; s < NSTAGE - 1; ++s)
        issue(s, sc[s]);
    // K tile kt of an output tile, of stage P
    auto step = [&](auto stage) __attribute__((always_inline)) {
        constexpr int P = decltype(stage)::value, NEXT = (P + NSTAGE - 1) % NSTAGE;
        wait_vm<(NSTAGE - 2) * TS>();   // K tile kt has landed; the younger ones may not have
        bar();   // every wave's part of it, and every wave is done with the stage read before
        issue(NEXT, sc[NEXT]);
        int s[AV + AM];
#pragma unroll
        for (int j = 0; j < AV + AM; ++j)
            s[j] = sc[P][j].get(kt * CHUNKS + 2 * qd, blocks);
        auto half = [&](auto h) __attribute__((always_inline)) {
            constexpr int S = decltype(h)::value;
            i32x4_t af[AV], bf[AM];
#pragma unroll
            for (int a = 0; a < AV; ++a)
                af[a] = *(const i32x4_t *)(smem + P * STAGE + ((a_addr + a * 16 * BK) ^ (64 * S)));
#pragma unroll
            for (int m = 0; m < AM; ++m)
                bf[m] = *(const i32x4_t *)(smem + P * STAGE + ((b_addr + m * 16 * BK) ^ (64 * S)));
#pragma unroll
            for (int a = 0; a < AV; ++a)
#pragma unroll
                for (int m = 0; m < AM; ++m)
                    acc[a][m] = mfma_fp4<S, S>(af[a], bf[m], acc[a][m], s[a], s[AV + m]);
        };
        half(std::integral_constant<int, 0>{});
        half(std::integral_constant<int, 1>{});
        if (++kt < nk)
            return;
        int m0, v0;
        tile_coords(tile, m0, v0);
#pragma unroll
        for (int a = 0; a < AV; ++a) {
            const int v = v0 + wv * WV + a * 16 + qd * 4;
#pragma unroll
            for (int m = 0; m < AM; ++m) {
                const int row = m0 + wm * WM + m * 16 + r16;
                if (tile < n_my && row < rows && v < V)
                    store4<OUT_BF16>(out, (int64_t)row * V + v, acc[a][m], v, V, vec);
                acc[a][m] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
            }
        }
        kt = 0;
        ++tile;
    };
    // (steps past the last tile of a round are computed and not stored)
    while (tile < n_my)
        [&]<int... P>(std::integer_sequence<int, P...>) __attribute__((always_inline)) {
            (step(std::integral_constant<int, P>{}), ...);
        }(std::make_integer_sequence<int, NSTAGE>{});
    wait_vm<0>();   // no request into the workgroup's LDS may be left when it ends
}

__device__ __forceinline__ void request4(const void *src, void *lds)
{
    __builtin_amdgcn_global_load_lds(src, (lds_void_t *)lds, 4, 0, 0);
}

// BM x 256 outputs per workgroup of eight waves, BM = 128 or 256, walked persistently.  A K tile is
// 128 bytes (eight blocks) of each row.  Waves 0-3 (one per SIMD) request it straight to LDS, into two
// stages: as soon as every wave has a tile's last fragments in registers, its stage takes the tile
// after next.  16-byte blocks are XOR-swizzled, the A fragments single-buffered, the B fragments
// double-buffered.  The tile order keeps the XCDs side by side on the vocabulary.
//  * Scales: eight bytes a row and K tile.  GROUPED (the rows' blocks are a multiple of 16): those of
//    four K tiles are requested together, 32 bytes a row, a quarter of the rows with each of the four K
//    tiles before; else the K tile's own two words of each row, with the tile.  What a request costs is
//    the lines that it touches: the words of a K tile touch 512 lines for their 4 KB, beside the codes'
//    512 for 64 KB.
//  * Lanes trade words in the epilogue so that each store instruction writes whole 128-byte lines.
//  * Not GROUPED: the rows' blocks are a multiple of four only; what lies behind a row's end is read
//    from kZeroCodes.
//  * STREAM: W is read once (one row tile): its requests take the streaming cache policy.
template <int BM, bool STREAM, bool OUT_BF16, bool GROUPED>
__global__ __attribute__((amdgpu_flat_work_group_size(512, 512), amdgpu_waves_per_eu(2, 2))) void
gemm_mxfp4_kernel(const uint8_t *__restrict__ Hq, const uint8_t *__restrict__ hs, const int32_t *__restrict__ rows_dev,
                  int32_t max_rows, const uint8_t *__restrict__ Wq, const uint8_t *__restrict__ ws, int32_t V,
                  int32_t blocks, void *__restrict__ out, int32_t group_m)
{
    constexpr int NW = 8, NWV = BM == 128 ? 4 : 2, DMAW = 4, BV = 256, BK = 128;
    constexpr int CHUNKS = BK / 16, RPI = 64 / CHUNKS;          // rows per request instruction
    constexpr int W_TILE = BV * BK, H_TILE = BM * BK, S_TILE = GROUPED ? 512 * 32 : (BV + BM) * 8, S_ST = GROUPED ? 2 : 4;
    constexpr int H_BASE = 2 * W_TILE, S_BASE = H_BASE + 2 * H_TILE;
    constexpr int WV = BV / NWV, WM = BM / (NW / NWV), AV = WV / 16, AM = WM / 16;
    constexpr int LW = BV / RPI / DMAW, LH = BM / RPI / DMAW;   // requests per requesting wave
    constexpr int SW = BV * 2 / 64 / DMAW, SH = BM * 2 / 64 / DMAW;
    constexpr int LT = LW + LH + (GROUPED ? 1 : SW + SH);       // and with the scales
    static_assert(S_BASE + S_ST * S_TILE <= 160 * 1024, "LDS");
    __shared__ __attribute__((aligned(1024))) char smem[S_BASE + S_ST * S_TILE];

    const int rows = (int)row_count(rows_dev, max_rows), d = blocks * 16;
    const int nvt = (V + BV - 1) / BV, nmt = (rows + BM - 1) / BM, ntiles = nvt * nmt;
    const int nk = (blocks + CHUNKS - 1) / CHUNKS;

    // Tile list of this workgroup: in a full super-group of 8 * group_m row tiles, XCD x takes
    // row tiles x, x + 8, ... of every vocabulary tile; the rest goes to the XCDs in eight
    // contiguous runs.
    const int per_xcd = gridDim.x >> 3, xcd = blockIdx.x & 7, slot = blockIdx.x >> 3;
    const int per_group = group_m * nvt, sg = 8 * group_m, nfull = nmt / sg;
    const int full_tiles = nfull * per_group;
    const int rtiles = ntiles - 8 * full_tiles, q8 = rtiles >> 3, rem = rtiles & 7;
    const int start = xcd < rem ? xcd * (q8 + 1) : rem * (q8 + 1) + (xcd - rem) * q8;
    const int count = full_tiles + q8 + (xcd < rem ? 1 : 0);
    const int n_my = slot < count ? (count - slot + per_xcd - 1) / per_xcd : 0;
    if (n_my == 0)
        return;
    auto tile_coords = [&](int i, int &m0, int &v0) __attribute__((always_inline)) {
        const int tx = slot + i * per_xcd;
        if (tx < full_tiles) {
            const int s = tx / per_group, t = 8 * (tx - s * per_group) + xcd;
            m0 = (s * sg + t % sg) * BM;
            v0 = (t / sg) * BV;
            return;
        }
        const int t = start + tx - full_tiles, g = t / per_group;
        const int first_m = nfull * sg + g * group_m, gsz = min(nmt - first_m, group_m);
        const int local = t - g * per_group;
        m0 = (first_m + local % gsz) * BM;
        v0 = (local / gsz) * BV;
    };

    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wv = wave % NWV, wm = wave / NWV, dwave = wave % DMAW;

    // Requests: lane i of instruction j fills place i % CHUNKS of tile row (dwave * L + j) * RPI + i /
    // CHUNKS.  Scale words: lane i
    // of instruction j takes half i % 2 of row (dwave * S + j) * 32 + i / 2.  Rows past V / rows
    // re-read the last valid row; their results are never stored.
    // Offsets are made anew for each request, from a few registers: kept, they would take twenty.
    const uint32_t wrow0 = (uint32_t)(dwave * LW * RPI + lane / CHUNKS) * (uint32_t)d;
    const uint32_t hrow0 = (uint32_t)(dwave * LH * RPI + lane / CHUNKS) * (uint32_t)d;
    const uint32_t wsrow0 = (uint32_t)(dwave * SW * 32 + lane / 2) * (uint32_t)blocks;
    const uint32_t hsrow0 = (uint32_t)(dwave * SH * 32 + lane / 2) * (uint32_t)blocks;
    static_assert(LW % 2 == 0 && LH % 2 == 0 && RPI == 8, "requests of one parity swizzle alike");
    const uint32_t chunk[2] = {(uint32_t)block_at(lane % CHUNKS, lane / CHUNKS) * 16,
                               (uint32_t)block_at(lane % CHUNKS, lane / CHUNKS + RPI) * 16};
    const uint32_t half = lane % 2 * 4;
    const uint8_t *wbase, *hbase, *wsbase, *hsbase;
    uint32_t wlast, hlast;   // the last valid row of the tile
    auto make_src = [&](int m0, int v0) __attribute__((always_inline)) {
        wbase = Wq + (int64_t)v0 * d;
        hbase = Hq + (int64_t)m0 * d;
        wsbase = ws + (int64_t)v0 * blocks;
        hsbase = hs + (int64_t)m0 * blocks;
        wlast = (uint32_t)min(BV, V - v0) - 1;
        hlast = (uint32_t)min(BM, rows - m0) - 1;
    };
    // Quarter t % 4 of the scales of group t / 4 + 1 (128 of the 512 rows: W's, then H's; with 128 of H the
    // last quarter repeats them, unused), two lanes a row, into the group's half of the stages.  Group g is
    // requested at t = 4 g - 4 .. 4 g - 1, with K tiles t, when the group before the last has been
    // read; zeros behind the rows' ends.
    auto issue_group = [&](int t) __attribute__((always_inline)) {
        const int g = (t >> 2) + 1, q = t & 3;
        uint32_t r = dwave * 32 + lane / 2 + (q & 1) * 128;
        asm volatile("" : "+v"(r));
        const uint32_t k = g * 32 + lane % 2 * 16, off = min(r, q < 2 ? wlast : hlast) * (uint32_t)blocks + k;
        const uint64_t src = (uint64_t)(q < 2 ? wsbase : hsbase) + off, in = k < (uint32_t)blocks ? ~(uint64_t)0 : 0;
        request<false>((const void *)((src & in) | ((uint64_t)kZeroCodes & ~in)),
                       smem + S_BASE + (g & 1) * S_TILE + (q * 128 + dwave * 32) * 32);
    };
    const uint32_t d32 = (uint32_t)d, b32 = (uint32_t)blocks;
    // the words of K tile kt's scales
    auto issue_words = [&](int kt) __attribute__((always_inline)) {
        uint32_t wsr = wsrow0, hsr = hsrow0;
        asm volatile("" : "+v"(wsr), "+v"(hsr));   // (or the offsets are kept after all)
        auto from = [&](const uint8_t *base, uint32_t row0, uint32_t last, int j) __attribute__((always_inline)) {
            const uint32_t off = min(row0 + (uint32_t)(j * 32) * b32, last * b32) + half;
            return kt * CHUNKS + half < b32 ? base + kt * CHUNKS + off : kZeroCodes;
        };
        char *at = smem + S_BASE + (kt & 3) * S_TILE;
#pragma unroll
        for (int j = 0; j < SW; ++j)
            request4(from(wsbase, wsr, wlast, j), at + (dwave * SW + j) * 256);
#pragma unroll
        for (int j = 0; j < SH; ++j)
            request4(from(hsbase, hsr, hlast, j), at + BV * 8 + (dwave * SH + j) * 256);
    };
    // K tile kt's codes into stage p
    auto issue_codes = [&](int p, int kt) __attribute__((always_inline)) {
        uint32_t wr = wrow0, hr = hrow0;
        asm volatile("" : "+v"(wr), "+v"(hr));
        auto from = [&](const uint8_t *base, uint32_t row0, uint32_t last, int j) __attribute__((always_inline)) {
            const uint32_t off = min(row0 + (uint32_t)(j * RPI) * d32, last * d32) + chunk[j & 1];
            return GROUPED || kt * BK + chunk[j & 1] < d32 ? base + kt * BK + off : kZeroCodes;
        };
#pragma unroll
        for (int j = 0; j < LW; ++j)
            request<STREAM>(from(wbase, wr, wlast, j), smem + p * W_TILE + (dwave * LW + j) * 1024);
#pragma unroll
        for (int j = 0; j < LH; ++j)
            request<false>(from(hbase, hr, hlast, j), smem + H_BASE + p * H_TILE + (dwave * LH + j) * 1024);
    };
    // what goes out in step kt, into stage p
    auto issue = [&](int p, int kt) __attribute__((always_inline)) {
        if constexpr (GROUPED)
            issue_group(kt + 2);
        else
            issue_words(kt + 3);
        issue_codes(p, kt + 2);
    };

    f32x4_t acc[AV][AM];
    auto zero_acc = [&]() __attribute__((always_inline)) {
#pragma unroll
        for (int a = 0; a < AV; ++a)
#pragma unroll
            for (int b = 0; b < AM; ++b)
                acc[a][b] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
    };
    zero_acc();

    // Fragments: lane (r16, qd) reads row r16 of a 16-row block, its blocks 2 qd and 2 qd + 1 in the
    // two sub-steps; 16-row blocks start at multiples of 16, so a row's swizzle is the lane's.
    const int r16 = lane & 15, qd = lane >> 4;
    const int lane_chunk = (qd ^ swizzle(r16)) * 16;
    const int a_addr = (wv * WV + r16) * BK + lane_chunk, b_addr = H_BASE + (wm * WM + r16) * BK + lane_chunk;
    constexpr int S_ROW = GROUPED ? 32 : 8;
    const int sa_addr = S_BASE + (wv * WV + r16) * S_ROW + 2 * qd;
    const int sb_addr = S_BASE + (BV + wm * WM + r16) * S_ROW + 2 * qd;
    // where K tile kt's scales lie behind these
    auto scales_at = [&](int kt) { return GROUPED ? (kt >> 2 & 1) * S_TILE + (kt & 3) * 8 : (kt & 3) * S_TILE; };
    i32x4_t af[AV], bf[2][AM];
    // scale bytes of the K tile, two 16-row blocks to a register: byte 2 (a % 2) + s for sub-step s
    u16x2_t sa[AV / 2], sb[AM / 2];
    auto read_a = [&](int p, int s, int a) __attribute__((always_inline)) {
        return *(const i32x4_t *)(smem + ((a_addr + p * W_TILE) ^ (64 * s)) + a * 16 * BK);
    };
    auto read_b = [&](int p, int s, int b) __attribute__((always_inline)) {
        return *(const i32x4_t *)(smem + ((b_addr + p * H_TILE) ^ (64 * s)) + b * 16 * BK);
    };
    auto read_scales = [&](int at, u16x2_t (&x)[AV / 2], u16x2_t (&y)[AM / 2]) __attribute__((always_inline)) {
#pragma unroll
        for (int a = 0; a < AV; ++a)
            x[a / 2][a % 2] = *(const uint16_t *)(smem + sa_addr + at + a * 16 * S_ROW);
#pragma unroll
        for (int b = 0; b < AM; ++b)
            y[b / 2][b % 2] = *(const uint16_t *)(smem + sb_addr + at + b * 16 * S_ROW);
    };
    // MFMAs of sub-step S of a K tile, while the next sub-step's fragments are read: sub-step 1 of
    // the same stage p, or sub-step 0 of the next K tile's stage p.  The B fragments go first, each A
    // fragment after its row's MFMAs, the last one before them, so that the wave's last read is not
    // followed by the step's wait.  Odd rows take the B blocks in reverse: consecutive MFMAs share an
    // operand, which takes less power.  Sub-step 0 also reads the next K tile's scales (at `at`).
    uint16_t ra[AV], rb[AM];
    auto mma_load = [&](auto sub, int p, int at) __attribute__((always_inline)) {
        constexpr int S = decltype(sub)::value;
#pragma unroll
        for (int b = 0; b < AM; ++b) {
            bf[S ^ 1][b] = read_b(p, S ^ 1, b);
            if (S == 0)
                rb[b] = *(const uint16_t *)(smem + sb_addr + at + b * 16 * S_ROW);
        }
#pragma unroll
        for (int a = 0; a < AV; ++a) {
            const i32x4_t x = af[a];
            if (a == AV - 1)
                af[a] = read_a(p, S ^ 1, a);
            if (S == 0)
                ra[a] = *(const uint16_t *)(smem + sa_addr + at + a * 16 * S_ROW);
#pragma unroll
            for (int c = 0; c < AM; ++c) {
                const int b = (a & 1) ? AM - 1 - c : c;
                const int wsc = __builtin_bit_cast(int, sa[a / 2]), hsc = __builtin_bit_cast(int, sb[b / 2]);
                if (a % 2 == 0)
                    acc[a][b] = b % 2 == 0 ? mfma_fp4<S, S>(x, bf[S][b], acc[a][b], wsc, hsc)
                                           : mfma_fp4<S, 2 + S>(x, bf[S][b], acc[a][b], wsc, hsc);
                else
                    acc[a][b] = b % 2 == 0 ? mfma_fp4<2 + S, S>(x, bf[S][b], acc[a][b], wsc, hsc)
                                           : mfma_fp4<2 + S, 2 + S>(x, bf[S][b], acc[a][b], wsc, hsc);
            }
            if (a < AV - 1)
                af[a] = read_a(p, S ^ 1, a);
        }
        // here, not later: behind a branch the compiler would gather two sub-steps' MFMAs
#pragma unroll
        for (int a = 0; a < AV; ++a)
#pragma unroll
            for (int b = 0; b < AM; ++b)
                asm volatile("" : "+v"(acc[a][b]));
    };
    // Instruction order of a sub-step: the B fragments beside the first row's MFMAs, each A fragment after
    // its row's, and between them a scale (sub-step 0) or a request (sub-step 1) beside an MFMA.
    auto interleave = [&](int nreq, bool scales) __attribute__((always_inline)) {
        int left = nreq;
#pragma unroll
        for (int a = 0; a < AV; ++a) {
            if (a > 0)
                __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
            if (a == AV - 1)
                __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
#pragma unroll
            for (int c = 0; c < AM; ++c) {
                __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
                if (a == 0)
                    __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
                if (scales && a > 0 && a <= 6 && c % 2 == 0)
                    __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
                if (left > 0) {
                    __builtin_amdgcn_sched_group_barrier(0x020, 1, 0);
                    --left;
                }
            }
        }
    };

    // a tile's first two K tiles
    auto prologue = [&]() __attribute__((always_inline)) {
        if constexpr (GROUPED) {
#pragma unroll
            for (int t = -4; t < 2; ++t)   // the first group, and half of the second
                issue_group(t);
        } else {
#pragma unroll
            for (int t = 0; t < 3; ++t)
                issue_words(t);
        }
        issue_codes(0, 0);
        if (nk > 1)
            issue_codes(1, 1);
    };

    const bool vec_ok = ((uintptr_t)out & 15) == 0 && V % (OUT_BF16 ? 8 : 4) == 0;
    // Rows of whole 128-byte lines are stored with the streaming cache policy, which leaves the
    // caches to the codes.
    const bool lines = vec_ok && ((uintptr_t)out & 127) == 0 && V % (OUT_BF16 ? 64 : 32) == 0;
    // one lane's N = 8 (bf16) or 4 (fp32) results of row `row` from vocabulary entry v on
    auto store_words = [&](int row, int v, const uint32_t (&w)[4]) __attribute__((always_inline)) {
        constexpr int N = OUT_BF16 ? 8 : 4;
        if (row >= rows)
            return;
        char *o = (char *)out + ((int64_t)row * V + v) * (OUT_BF16 ? 2 : 4);
        if (vec_ok && v + N <= V) {
            const i32x4_t x = {(int)w[0], (int)w[1], (int)w[2], (int)w[3]};
            if (lines) {
                // (between the fences, or the two stores are made one, without the policy)
                asm volatile("" ::: "memory");
                __builtin_nontemporal_store(x, (i32x4_t *)o);
                asm volatile("" ::: "memory");
            } else {
                *(i32x4_t *)o = x;
            }
            return;
        }
#pragma unroll
        for (int e = 0; e < N; ++e) {
            if (v + e < V) {
                if constexpr (OUT_BF16)
                    ((uint16_t *)o)[e] = (uint16_t)(w[e >> 1] >> (16 * (e & 1)));
                else
                    ((uint32_t *)o)[e] = w[e];
            }
        }
    };
    // Lanes r16 and r16 ^ 8 trade words (row rotate by 8, the bank mask picks the receiving
    // half), so that x holds rows 0-7 of both operands and y rows 8-15.
    auto trade = [&](uint32_t (&x)[4], uint32_t (&y)[4]) __attribute__((always_inline)) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int a = (int)x[e], b = (int)y[e];
            x[e] = (uint32_t)__builtin_amdgcn_update_dpp(a, b, 0x128, 0xf, 0xc, false);
            y[e] = (uint32_t)__builtin_amdgcn_update_dpp(b, a, 0x128, 0xf, 0x3, false);
        }
    };
    // Lane (r16, qd) holds entries 4 qd .. 4 qd + 3 of each 16-entry block for row r16 of each
    // 16-row block.
    auto epilogue = [&](int m0, int v0) __attribute__((always_inline)) {
#pragma unroll
        for (int q = 0; q < AV / 4; ++q) {
#pragma unroll
            for (int b = 0; b < AM; ++b) {
                const int row = m0 + wm * WM + b * 16 + (r16 & 7);
                if constexpr (OUT_BF16) {
                    // neighbouring blocks: permlane16_swap gives a lane eight entries of one
                    uint32_t p[2][4];
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const f32x4_t &lo = acc[4 * q + 2 * i][b], &hi = acc[4 * q + 2 * i + 1][b];
                        const auto s0 = __builtin_amdgcn_permlane16_swap(pack_bf16(lo[0], lo[1]), pack_bf16(hi[0], hi[1]),
                                                                         false, false);
                        const auto s1 = __builtin_amdgcn_permlane16_swap(pack_bf16(lo[2], lo[3]), pack_bf16(hi[2], hi[3]),
                                                                         false, false);
                        p[i][0] = s0[0];
                        p[i][1] = s1[0];
                        p[i][2] = s0[1];
                        p[i][3] = s1[1];
                    }
                    trade(p[0], p[1]);
                    const int v = v0 + wv * WV + (4 * q + 2 * (r16 >> 3) + (qd & 1)) * 16 + 4 * (qd & 2);
                    store_words(row, v, p[0]);
                    store_words(row + 8, v, p[1]);
                } else {
#pragma unroll
                    for (int i = 0; i < 4; i += 2) {
                        uint32_t p[2][4];
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            p[0][e] = __builtin_bit_cast(uint32_t, (float)acc[4 * q + i][b][e]);
                            p[1][e] = __builtin_bit_cast(uint32_t, (float)acc[4 * q + i + 1][b][e]);
                        }
                        trade(p[0], p[1]);
                        const int v = v0 + wv * WV + (4 * q + i + (r16 >> 3)) * 16 + 4 * qd;
                        store_words(row, v, p[0]);
                        store_words(row + 8, v, p[1]);
                    }
                }
            }
        }
    };

    auto main_loop = [&](auto dma_tag) __attribute__((always_inline)) {
        constexpr bool DMA_ON = decltype(dma_tag)::value;
        constexpr std::integral_constant<int, 0> first{};
        constexpr std::integral_constant<int, 1> second{};
        int m0, v0;
        tile_coords(0, m0, v0);
        if constexpr (DMA_ON) {
            make_src(m0, v0);
            prologue();
        }
        for (int i = 0; i < n_my; ++i) {
            // K tile 0 has landed; K tile 1 may still be in flight
            if (nk > 1)
                wait_vm<LW + LH>();
            else
                wait_vm<0>();
            bar();
#pragma unroll
            for (int a = 0; a < AV; ++a)
                af[a] = read_a(0, 0, a);
#pragma unroll
            for (int b = 0; b < AM; ++b)
                bf[0][b] = read_b(0, 0, b);
            read_scales(0, sa, sb);
            // the scales that sub-step 0 has read, for the next K tile
            auto next_scales = [&]() __attribute__((always_inline)) {
#pragma unroll
                for (int a = 0; a < AV; ++a)
                    sa[a / 2][a % 2] = ra[a];
#pragma unroll
                for (int b = 0; b < AM; ++b)
                    sb[b / 2][b % 2] = rb[b];
            };
            int kt = 0, p = 0;
            for (; kt + 2 < nk; ++kt) {
                mma_load(first, p, scales_at(kt + 1));
                interleave(0, true);
                __builtin_amdgcn_sched_barrier(0);
                wait_vm<0>();   // K tile kt + 1, and this wave's last fragments of this one
                bar();
                __builtin_amdgcn_sched_barrier(0);
                if constexpr (DMA_ON)
                    issue(p, kt);
                p ^= 1;
                mma_load(second, p, 0);
                interleave(DMA_ON ? LT : 0, false);
                __builtin_amdgcn_sched_barrier(0);
                next_scales();
            }
            for (; kt < nk; ++kt) {
                mma_load(first, p, scales_at(kt + 1));
                if (kt + 1 < nk) {
                    wait_vm<0>();
                    bar();
                }
                p ^= 1;
                mma_load(second, p, 0);   // after the last K tile its reads are unused
                next_scales();
            }
            // Every wave's last fragments are in registers.  The stores go first, then the next
            // tile's requests: its first wait then leaves its second K tile in flight instead of
            // waiting for it behind these stores.
            wait_vm<0>();
            bar();
            epilogue(m0, v0);
            zero_acc();
            if (i + 1 < n_my) {
                tile_coords(i + 1, m0, v0);
                if constexpr (DMA_ON) {
                    make_src(m0, v0);
                    prologue();
                }
            }
        }
    };
    if (wave < DMAW)
        main_loop(std::true_type{});
    else
        main_loop(std::false_type{});
}

// The forms of the small kernel.  BYTES: taken only where the scale rows are no whole words.
template <int BM_, int BV_, int WGM_, int NSTAGE_, bool STREAM_, bool BYTES_ = false>
struct Small {
    static constexpr int BM = BM_, BV = BV_, WGM = WGM_, NSTAGE = NSTAGE_;
    static constexpr bool STREAM = STREAM_, BYTES = BYTES_;
    static constexpr int PER_CU = 163840 / (NSTAGE_ * (BM_ + BV_) * 128);   // workgroups that the LDS holds
};

}  // namespace

hipError_t launch_quantize_rows_mxfp4(const void *X, bool in_bf16, int64_t nsrc, int64_t d, const int32_t *row_idx,
                                      int64_t rows, uint8_t *q, uint8_t *scale, void *values, hipStream_t stream)
{
    const int64_t blocks = mxfp4_blocks(d);
    // the most threads of which four fifths have work over all turns (65536 x 1040 bf16, 132 chunks: 32 threads)
    const int64_t chunks = blocks * 4;
    int lpr = 8;
    while (lpr > 2 && chunks * 5 < ((chunks + (1 << lpr) - 1) >> lpr << lpr) * 4)
        --lpr;
    const int64_t each = 256 >> lpr;
    const dim3 grid((unsigned)std::min<int64_t>((rows + each - 1) / each, 1 << 20));
    auto go = [&](auto kernel) {
        hipLaunchKernelGGL(kernel, grid, dim3(256), 0, stream, X, nsrc, (int32_t)d, (int32_t)blocks, lpr, row_idx, rows, q,
                           scale, values);
    };
    in_bf16 ? go(quantize_mxfp4_kernel<true>) : go(quantize_mxfp4_kernel<false>);
    return hipGetLastError();
}

hipError_t launch_gemm_mxfp4(const uint8_t *Hq, const uint8_t *hs, const int32_t *count, int64_t rows,
                             const uint8_t *Wq, const uint8_t *ws, int64_t V, int64_t blocks, void *out, bool out_bf16,
                             hipStream_t stream)
{
    int dev = 0, cus = 256;
    if (hipGetDevice(&dev) == hipSuccess)
        (void)hipDeviceGetAttribute(&cus, hipDeviceAttributeMultiprocessorCount, dev);
    auto tiles = [&](int64_t bm, int64_t bv) { return ((V + bv - 1) / bv) * ((rows + bm - 1) / bm); };
    auto go = [&](auto kernel, int64_t grid, int threads) {
        hipLaunchKernelGGL(kernel, dim3((unsigned)grid), dim3(threads), 0, stream, Hq, hs, count, (int32_t)rows, Wq, ws,
                           (int32_t)V, (int32_t)blocks, out, kDefaultGroupM);
    };
    auto pick = [&](auto bf16_tag) {
        constexpr bool B = decltype(bf16_tag)::value;
        if (blocks == 1) {
            const dim3 grid((unsigned)std::min<int64_t>((tiles(16, 16) + 3) / 4, 1 << 20));
            hipLaunchKernelGGL((gemm_mxfp4_block_kernel<B>), grid, dim3(256), 0, stream, Hq, hs, count, (int32_t)rows, Wq,
                               ws, (int32_t)V, out);
            return;
        }
        const bool words = blocks % 4 == 0 && (((uintptr_t)hs | (uintptr_t)ws) & 3) == 0;
        auto small = [&](auto form) {
            using F = decltype(form);
            const int64_t slots = std::max(8, cus / 8 * 8) * F::PER_CU;
            const int64_t grid = std::min(tiles(F::BM, F::BV), slots);
            if constexpr (!F::BYTES)
                if (words)
                    return go(gemm_mxfp4_small_kernel<F::BM, F::BV, F::WGM, F::NSTAGE, F::STREAM, true, B>, grid, 256);
            go(gemm_mxfp4_small_kernel<F::BM, F::BV, F::WGM, F::NSTAGE, F::STREAM, false, B>, grid, 256);
        };
        // Latency counts: eight stages, and a tile for each CU at most.
        if (tiles(32, 32) <= cus)
            return small(Small<32, 32, 2, 8, false>{});
        if (rows <= 32 && tiles(32, 128) >= cus)
            return small(Small<32, 128, 1, 4, true>{});
        if (rows <= 32)
            return small(Small<32, 64, 1, 4, true>{});
        // 33 to 64 rows over many entries take the large kernel's 128-row tiles, half empty or more,
        // for its longer requests (64 x 126464 x 4096: 58 us, tiles of 64 x 128 77; 48 x 65536 x 4096: 30 us,
        // 39; 33 x 152064 x 3584: 73 us, 70), if the scale rows are whole words.
        if (rows <= 64 && !words && tiles(64, 128) >= cus)
            return small(Small<64, 128, 1, 3, true, true>{});
        if (rows <= 64 && (!words || tiles(64, 128) < cus))
            return small(Small<64, 64, 2, 4, true>{});
        if (tiles(128, 128) < cus)
            return small(Small<64, 64, 2, 4, false>{});
        if (!words)
            return small(Small<128, 128, 2, 3, false, true>{});
        auto large = [&](auto bm_tag) {
            constexpr int BM = decltype(bm_tag)::value;
            const int64_t n = tiles(BM, 256);
            // one persistent workgroup per CU, a multiple of the eight XCDs
            const int64_t grid = std::min<int64_t>(std::max(8, cus / 8 * 8), (n + 7) / 8 * 8);
            const bool grouped = blocks % 16 == 0 && (((uintptr_t)hs | (uintptr_t)ws) & 15) == 0;
            if (!grouped)
                go(gemm_mxfp4_kernel<BM, false, B, false>, grid, 512);
            else if (rows <= BM)
                go(gemm_mxfp4_kernel<BM, true, B, true>, grid, 512);
            else
                go(gemm_mxfp4_kernel<BM, false, B, true>, grid, 512);
        };
        auto rounds = [&](int64_t n) { return (n + cus - 1) / cus; };
        // A round of 128-row tiles takes two thirds of one of 256-row tiles (1229 x 126464 x 4096: 457 us in
        // 20 rounds, 357 in 10; 384 rows: 150 in 6, 143 in 4; 128 x 152064 x 3584: 79, 91, in 3 each; 512 x
        // 8192 x 4096: 18, 26, in one; 4096 x 126464 x 4096: 1.48 ms, 1.07, 4.0 PFLOP/s).
        if (rounds(tiles(128, 256)) * 2 < rounds(tiles(256, 256)) * 3)
            large(std::integral_constant<int, 128>{});
        else
            large(std::integral_constant<int, 256>{});
    };
    if (out_bf16)
        pick(std::true_type{});
    else
        pick(std::false_type{});
    return hipGetLastError();
}

}  // namespace mosaic
