// INT8 LM head: products of 8-bit integer codes with a scale per row (token) and per
// vocabulary entry (channel),
//   out[i, v] = (sum_k Hq[i, k] Wq[v, k]) * hs[i] * ws[v].
// The sums are exact in int32 (d <= 131071, codes of magnitude 128 at most), so every form
// below gives the same bits, whatever its order: the sum is converted to fp32 (one rounding
// above 2^24), multiplied by hs[i], then by ws[v], and rounded to bf16 where that is the
// output's type.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <type_traits>

#include "launch.h"
#include "launch_ops.h"
#include "row_ops.h"

namespace mosaic {
namespace {

typedef int i32x4_t __attribute__((ext_vector_type(4)));
typedef float f32x4_t __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2_t __attribute__((ext_vector_type(2)));

// Four consecutive vocabulary entries v .. v + 3 of one row; vec: the address is a multiple of
// the four values' size.
template <bool OUT_BF16>
__device__ __forceinline__ void store4(void *out, int64_t off, const float (&x)[4], int v, int V, bool vec)
{
    if (vec && v + 3 < V) {
        if constexpr (OUT_BF16)
            *(u32x2_t *)((uint16_t *)out + off) = u32x2_t{rows::pack_bf16(x[0], x[1]), rows::pack_bf16(x[2], x[3])};
        else
            *(f32x4_t *)((float *)out + off) = f32x4_t{x[0], x[1], x[2], x[3]};
        return;
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        if (v + e < V) {
            if constexpr (OUT_BF16)
                ((__bf16 *)out)[off + e] = static_cast<__bf16>(x[e]);
            else
                ((float *)out)[off + e] = x[e];
        }
    }
}

// s_waitcnt vmcnt(N) lgkmcnt(0)
template <int N>
__device__ __forceinline__ void wait_vm()
{
    static_assert(N >= 0 && N < 64, "vmcnt range");   // 63: no wait for loads
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

// The 16 codes of a row p of d codes from k on, k a multiple of 16, zeros behind the row's end;
// the row may start at any byte.  A chunk that the end cuts is read as the row's last 16 codes
// and shifted, so that nothing outside the row is read.
__device__ __forceinline__ i32x4_t row_chunk(const int8_t *p, int k, int d)
{
    i32x4_t r = {0, 0, 0, 0};
    if (k >= d)
        return r;
    if (k + 16 <= d) {
        __builtin_memcpy(&r, p + k, 16);
        return r;
    }
    uint64_t w[2] = {0, 0};
    if (d >= 16) {
        __builtin_memcpy(w, p + d - 16, 16);
        const int shift = 8 * (k + 16 - d);   // 8 .. 120 bits
        w[0] = shift < 64 ? (w[0] >> shift) | (w[1] << (64 - shift)) : w[1] >> (shift - 64);
        w[1] = shift < 64 ? w[1] >> shift : 0;
    } else {
#pragma unroll 1
        for (int b = 0; b < d; ++b) {
            const uint64_t c = (uint64_t)(uint8_t)p[b] << (8 * (b & 7));
            w[0] |= b < 8 ? c : 0;
            w[1] |= b < 8 ? 0 : c;
        }
    }
    __builtin_memcpy(&r, w, 16);
    return r;
}

// Any shape and alignment.  BM x BV outputs per workgroup of NW waves, NWV of them side by side
// along the vocabulary; K in steps of 128 codes, fetched SETS steps ahead into registers with
// 16-byte loads at any byte address and staged into LDS (rows of 128 + 16 bytes, which spreads
// the 16-byte fragment reads over the banks).  Rows past V / rows re-read the last valid row.
// SETS: 4 for the small tiles (2 x 13433 x 5656: 20 us, 25 with 2), 2 where registers are short.
// 3000 x 32000 x 4095 takes 726 to 777 us (1.05 POP/s; L1 busy 77% of the time, matrix pipes
// 23%), x 4100: 604 us, x 4096 in this form 578 us, in the aligned forms 350 us.  So most of what
// is lost to those is the form, whose smaller tiles go through registers; the rest is the L1,
// which takes a 16-byte load at an odd address in four parts.
template <int BM, int BV, int NW, int NWV, int SETS, bool OUT_BF16>
__global__ __launch_bounds__(64 * NW) void gemm_int8_any_kernel(const int8_t *__restrict__ Hq,
                                                                const float *__restrict__ hs,
                                                                const int32_t *__restrict__ count, int32_t max_rows,
                                                                const int8_t *__restrict__ Wq,
                                                                const float *__restrict__ ws, int32_t V, int32_t d,
                                                                void *__restrict__ out, int64_t ldo, int32_t group_m)
{
    constexpr int BK = 128, CHUNKS = BK / 16, PITCH = BK + 16, STAGE = (BV + BM) * PITCH;
    constexpr int WV = BV / NWV, WM = BM / (NW / NWV), AV = WV / 16, AM = WM / 16;
    constexpr int RPT = 64 * NW / CHUNKS, LW = BV / RPT, LH = BM / RPT, T = LW + LH;   // rows, chunks at a time
    __shared__ __attribute__((aligned(16))) char smem[2 * STAGE];
    const int rows = (int)rows::row_count(count, max_rows);
    const int nvt = (V + BV - 1) / BV, nmt = (rows + BM - 1) / BM, nblk = nvt * nmt;
    const int blk = blockIdx.x;
    if (blk >= nblk)
        return;
    // the workgroups of one XCD take a contiguous run of tiles: of group_m row tiles, the row
    // tiles of a vocabulary tile one after another
    const int q8 = nblk >> 3, rem = nblk & 7, xcd = blk & 7;
    const int t = (xcd < rem ? xcd * (q8 + 1) : rem * (q8 + 1) + (xcd - rem) * q8) + (blk >> 3);
    const int first_m = t / (group_m * nvt) * group_m, gsz = min(nmt - first_m, group_m);
    const int local = t - first_m * nvt;
    const int m0 = (first_m + local % gsz) * BM, v0 = local / gsz * BV;

    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int sr = tid / CHUNKS, sk = tid % CHUNKS * 16;   // thread's row (+ RPT j) and chunk
    const int8_t *wbase = Wq + (int64_t)v0 * d, *hbase = Hq + (int64_t)m0 * d;
    uint32_t off[T];
#pragma unroll
    for (int j = 0; j < T; ++j)
        off[j] = (uint32_t)(j < LW ? min(sr + j * RPT, V - 1 - v0) : min(sr + (j - LW) * RPT, rows - 1 - m0)) * (uint32_t)d;
    static_assert(SETS % 2 == 0, "a set of registers meets one LDS stage");
    i32x4_t x[SETS][T];   // K tiles under way
    auto fetch_tile = [&](int set, int kt, auto whole) __attribute__((always_inline)) {
#pragma unroll
        for (int j = 0; j < T; ++j) {
            const int8_t *p = (j < LW ? wbase : hbase) + off[j];
            if constexpr (decltype(whole)::value)
                __builtin_memcpy(&x[set][j], p + kt * BK + sk, 16);
            else
                x[set][j] = row_chunk(p, kt * BK + sk, d);
        }
    };
    auto put_tile = [&](int set, int stage) __attribute__((always_inline)) {
#pragma unroll
        for (int j = 0; j < T; ++j)
            *(i32x4_t *)(smem + stage * STAGE + (sr + j * RPT) * PITCH + sk) = x[set][j];
    };
    const int wv = wave % NWV * WV, wm = wave / NWV * WM;
    const int fr = lane & 15, kg = lane >> 4;
    i32x4_t acc[AV][AM];
#pragma unroll
    for (int a = 0; a < AV; ++a)
#pragma unroll
        for (int b = 0; b < AM; ++b)
            acc[a][b] = i32x4_t{0, 0, 0, 0};
    const int nk = (d + BK - 1) / BK;
    // K tile kt (kt % SETS = P) from stage kt % 2; kt + SETS is fetched meanwhile (whole: it ends
    // inside the row; past the row's end: zeros, unused)
    auto step = [&](auto set, int kt, auto whole) __attribute__((always_inline)) {
        constexpr int P = decltype(set)::value;
        fetch_tile(P, kt + SETS, whole);
        const char *s = smem + P % 2 * STAGE;
#pragma unroll
        for (int q = 0; q < BK / 64; ++q) {
            i32x4_t af[AV], bf[AM];
#pragma unroll
            for (int a = 0; a < AV; ++a)
                af[a] = *(const i32x4_t *)(s + (wv + a * 16 + fr) * PITCH + q * 64 + kg * 16);
#pragma unroll
            for (int b = 0; b < AM; ++b)
                bf[b] = *(const i32x4_t *)(s + (BV + wm + b * 16 + fr) * PITCH + q * 64 + kg * 16);
#pragma unroll
            for (int a = 0; a < AV; ++a)
#pragma unroll
                for (int b = 0; b < AM; ++b)
                    acc[a][b] = __builtin_amdgcn_mfma_i32_16x16x64_i8(af[a], bf[b], acc[a][b], 0, 0, 0);
        }
        put_tile((P + 1) % SETS, 1 - P % 2);   // last read in the step before, a barrier in between
        wait_vm<63>();   // (the LDS accesses; the K tiles under way stay so)
        bar();
    };
    // calls f with 0 .. SETS - 1 as constants
    auto each_set = [&](auto f) __attribute__((always_inline)) {
        f(std::integral_constant<int, 0>{});
        f(std::integral_constant<int, 1>{});
        if constexpr (SETS == 4) {
            f(std::integral_constant<int, 2>{});
            f(std::integral_constant<int, 3>{});
        }
    };
    each_set([&](auto set) __attribute__((always_inline)) {
        if ((set + 1) * BK <= d)
            fetch_tile(set, set, std::true_type{});
        else
            fetch_tile(set, set, std::false_type{});
    });
    put_tile(0, 0);
    wait_vm<63>();
    bar();
    int kt = 0;
    for (; (kt + 2 * SETS) * BK <= d; kt += SETS)
        each_set([&](auto set) __attribute__((always_inline)) { step(set, kt + set, std::true_type{}); });
    for (; kt < nk; kt += SETS)
        each_set([&](auto set) __attribute__((always_inline)) {
            if (kt + set < nk)
                step(set, kt + set, std::false_type{});
        });
    // lane (fr, kg) holds entries 4 kg .. 4 kg + 3 of a 16-entry block for row fr of a 16-row block
    const bool vec = OUT_BF16 ? ((uintptr_t)out & 7) == 0 && (ldo & 3) == 0
                              : ((uintptr_t)out & 15) == 0 && (ldo & 3) == 0;
#pragma unroll
    for (int b = 0; b < AM; ++b) {
        const int row = m0 + wm + b * 16 + fr;
        if (row >= rows)
            continue;
        const float hsc = hs[row];
#pragma unroll
        for (int a = 0; a < AV; ++a) {
            const int v = v0 + wv + a * 16 + kg * 4;
            if (v >= V)
                continue;
            float y[4];
#pragma unroll
            for (int e = 0; e < 4; ++e)
                y[e] = (float)acc[a][b][e] * hsc * ws[min(v + e, V - 1)];
            store4<OUT_BF16>(out, (int64_t)row * ldo + v, y, v, V, vec);
        }
    }
}

typedef __attribute__((address_space(3))) void lds_void_t;

// Requests straight to LDS: 16 bytes per lane, lane i's to lds + 16 i (STREAM: streaming cache
// policy), or 4.
template <bool STREAM>
__device__ __forceinline__ void request(const void *src, void *lds)
{
    __builtin_amdgcn_global_load_lds(src, (lds_void_t *)lds, 16, 0, STREAM ? 2 : 0);
}
__device__ __forceinline__ void request4(const void *src, void *lds)
{
    __builtin_amdgcn_global_load_lds(src, (lds_void_t *)lds, 4, 0, 0);
}

// What a request past the end of a row reads (rows whose d is no multiple of the K tile).
__device__ __attribute__((aligned(16))) const int8_t kZeroCodes[16] = {};

// BM x 256 outputs per workgroup of eight waves, BM = 128 or 256, walked persistently.  K tiles of 128 codes
// are rows of 128 bytes, as the bf16 kernel's K tiles of 64 elements are, and
// v_mfma_i32_16x16x64_i8 takes the 16 bytes per lane and the cycles of
// v_mfma_f32_16x16x32_bf16 at twice the products, so the pipeline is that kernel's: requests
// straight to LDS by waves 0-3 (one per SIMD), three W stages and two H stages (160 KiB),
// XOR-swizzled 16-byte chunks, the A fragments single-buffered, the tile order that keeps the
// XCDs side by side on the vocabulary.
//  * The tile's row scales (256 of W, 256 of H) are requested into the W stage that the K
//    loop's last step but one frees, one step ahead of their use; the ring of W stages starts
//    behind that stage in the next tile, whose third K tile is the first to reach it.
//  * Epilogue: int32 -> fp32, times both scales, rounded; lanes trade words so that each
//    store instruction writes whole 128-byte lines.
//  * TAIL: d is a multiple of 16 only; chunks past the row's end are read from kZeroCodes.
//  * STREAM: W is read once (one row tile): its requests take the streaming cache policy.
// Bound by power: 4096 x 126464 x 4096 takes 1.54 to 1.66 ms, box to box (2.6 to 2.7 POP/s), at 1.72
// to 1.75 GHz with the matrix pipes busy 73 to 75% of the cycles.
template <int BM, bool STREAM, bool OUT_BF16, bool TAIL>
__global__ __attribute__((amdgpu_flat_work_group_size(512, 512), amdgpu_waves_per_eu(2, 2))) void
gemm_int8_kernel(const int8_t *__restrict__ Hq, const float *__restrict__ hs, const int32_t *__restrict__ rows_dev,
                 int32_t max_rows, const int8_t *__restrict__ Wq, const float *__restrict__ ws, int32_t V, int32_t d,
                 void *__restrict__ out, int64_t ldo, int32_t group_m)
{
    constexpr int NW = 8, NWV = BM == 128 ? 4 : 2, DMAW = 4, BV = 256, BK = 128, WST = 3, HST = 2;
    constexpr int CHUNKS = BK / 16, RPI = 64 / CHUNKS;          // rows per request instruction
    constexpr int W_TILE = BV * BK, H_TILE = BM * BK, H_BASE = WST * W_TILE;
    constexpr int WV = BV / NWV, WM = BM / (NW / NWV), AV = WV / 16, AM = WM / 16;
    constexpr int LW = BV / RPI / DMAW, LH = BM / RPI / DMAW;   // requests per requesting wave
    static_assert(H_BASE + HST * H_TILE <= 160 * 1024, "LDS");
    __shared__ __attribute__((aligned(1024))) char smem[H_BASE + HST * H_TILE];

    const int rows = (int)rows::row_count(rows_dev, max_rows);
    const int nvt = (V + BV - 1) / BV, nmt = (rows + BM - 1) / BM, ntiles = nvt * nmt;
    const int nk = (d + BK - 1) / BK;

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
    auto swz = [](int r) { return (r >> 1) & 7; };

    // Requests: lane i of instruction j fills tile row (dwave * L + j) * RPI + i / CHUNKS, whose
    // logical chunk (i % CHUNKS) ^ swz(row) goes to physical chunk i % CHUNKS.  Rows past V /
    // rows re-read the last valid row; their results are never stored.
    auto tile_row = [&](int j, int per_wave) { return (dwave * per_wave + j) * RPI + lane / CHUNKS; };
    auto chunk_of = [&](int j) { return ((lane % CHUNKS) ^ swz(tile_row(j, LW))) * 16; };
    static_assert(LW % 2 == 0 && LH % 2 == 0, "rows of W and of H that one lane requests swizzle alike");
    const int8_t *wbase, *hbase;
    uint32_t woff[LW], hoff[LH];
    auto make_src = [&](int m0, int v0) __attribute__((always_inline)) {
        wbase = Wq + (int64_t)v0 * d;
        hbase = Hq + (int64_t)m0 * d;
#pragma unroll
        for (int j = 0; j < LW; ++j)
            woff[j] = (uint32_t)min(tile_row(j, LW), V - 1 - v0) * (uint32_t)d + (uint32_t)chunk_of(j);
#pragma unroll
        for (int j = 0; j < LH; ++j)
            hoff[j] = (uint32_t)min(tile_row(j, LH), rows - 1 - m0) * (uint32_t)d + (uint32_t)chunk_of(j);
    };
    auto source = [&](const int8_t *base, uint32_t off, int kb, int j) __attribute__((always_inline)) {
        const int8_t *src = base + kb + off;
        if constexpr (TAIL)
            src = kb + chunk_of(j) < d ? src : kZeroCodes;
        return src;
    };
    auto issue_w = [&](int rw, int kt) __attribute__((always_inline)) {
#pragma unroll
        for (int j = 0; j < LW; ++j)
            request<STREAM>(source(wbase, woff[j], kt * BK, j), smem + rw + (dwave * LW + j) * 1024);
    };
    auto issue_h = [&](int rh, int kt) __attribute__((always_inline)) {
#pragma unroll
        for (int j = 0; j < LH; ++j)
            request<false>(source(hbase, hoff[j], kt * BK, j), smem + rh + (dwave * LH + j) * 1024);
    };
    // row scales: 256 of W, then 256 of H, indices clamped to the last valid row
    auto issue_scales = [&](int at, int m0, int v0) __attribute__((always_inline)) {
        const int r = dwave * 64 + lane;
        request4(ws + min(v0 + r, V - 1), smem + at + dwave * 256);
        request4(hs + min(m0 + r, rows - 1), smem + at + BV * 4 + dwave * 256);
    };
    auto next_w = [](int rw) { return rw + W_TILE == H_BASE ? 0 : rw + W_TILE; };
    auto next_h = [](int rh) { return rh + H_TILE == H_BASE + HST * H_TILE ? H_BASE : rh + H_TILE; };

    i32x4_t acc[AV][AM];
    auto zero_acc = [&]() __attribute__((always_inline)) {
#pragma unroll
        for (int a = 0; a < AV; ++a)
#pragma unroll
            for (int b = 0; b < AM; ++b)
                acc[a][b] = i32x4_t{0, 0, 0, 0};
    };
    zero_acc();

    // Fragments: lane (r16, qd) reads row r16 of a 16-row block, logical chunk 4 s + qd of
    // sub-step s; blocks start at multiples of 16 rows, so a row's swizzle is the lane's.
    const int r16 = lane & 15, qd = lane >> 4;
    const int lane_chunk = (qd ^ swz(r16)) * 16;
    const int a_addr = (wv * WV + r16) * BK + lane_chunk, b_addr = (wm * WM + r16) * BK + lane_chunk;
    i32x4_t af[AV], bf[2][AM];
    // MFMAs on B buffer `cur` while sub-step s of the stages at rw (W) and rh (H) is read: the B
    // fragments first, each A fragment after its row's MFMAs, the last one before them, so
    // that the wave's last read is not followed by the step's wait.  Odd rows take the B
    // blocks in reverse: consecutive MFMAs share an operand, which takes less power.
    auto mma_load = [&](int rw, int rh, int s, int cur) __attribute__((always_inline)) {
        const int ab = (a_addr + rw) ^ (64 * s), bb = (b_addr + rh) ^ (64 * s);
#pragma unroll
        for (int b = 0; b < AM; ++b)
            bf[cur ^ 1][b] = *(const i32x4_t *)(smem + bb + b * 16 * BK);
#pragma unroll
        for (int a = 0; a < AV; ++a) {
            i32x4_t nxt;
            if (a == AV - 1)
                nxt = *(const i32x4_t *)(smem + ab + a * 16 * BK);
#pragma unroll
            for (int c = 0; c < AM; ++c) {
                const int b = (a & 1) ? AM - 1 - c : c;
                acc[a][b] = __builtin_amdgcn_mfma_i32_16x16x64_i8(af[a], bf[cur][b], acc[a][b], 0, 0, 0);
            }
            af[a] = a == AV - 1 ? nxt : *(const i32x4_t *)(smem + ab + a * 16 * BK);
        }
    };
    // Instruction order of a sub-step: each request beside an MFMA, then the fragment reads
    // spread over the MFMAs.
    auto interleave = [&](int nreq) __attribute__((always_inline)) {
#pragma unroll
        for (int i = 0; i < LW; ++i) {
            if (i < nreq) {
                __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
                __builtin_amdgcn_sched_group_barrier(0x020, 1, 0);
            }
        }
#pragma unroll
        for (int b = 0; b < AM; ++b) {
            __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
            __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
        }
        const int used = nreq + AM;
#pragma unroll
        for (int a = 0; a < AV; ++a) {
            if (a == AV - 1)
                __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
#pragma unroll
            for (int c = 0; c < AM; ++c)
                if (a * AM + c >= used)
                    __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
            if (a < AV - 1)
                __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
        }
    };

    int w0 = 0;   // W stage of the current tile's K tile 0
    // a tile's first two K tiles, in the order the waits count on
    auto prologue = [&]() __attribute__((always_inline)) {
        issue_h(H_BASE, 0);
        issue_w(w0 * W_TILE, 0);
        if (nk > 1) {
            issue_h(H_BASE + H_TILE, 1);
            issue_w((w0 + 1) % WST * W_TILE, 1);
        }
    };

    const bool vec_ok = ((uintptr_t)out & 15) == 0 && ldo % (OUT_BF16 ? 8 : 4) == 0;
    // Rows of whole 128-byte lines are stored with the streaming cache policy, which leaves the
    // caches to the codes: 256 x 152064 x 3584: 148 against 158 us, 4096 x 126464 x 2048: 866
    // against 910 us (on another MI355X, at a lower clock, both alike); with rows that start
    // inside a line, 2048 x 50000 x 8192, it costs: 686 against 663 us.
    const bool lines = vec_ok && ((uintptr_t)out & 127) == 0 && ldo % (OUT_BF16 ? 64 : 32) == 0;
    // one lane's N = 8 (bf16) or 4 (fp32) results of row `row` from vocabulary entry v on
    auto store_words = [&](int row, int v, const uint32_t (&w)[4]) __attribute__((always_inline)) {
        constexpr int N = OUT_BF16 ? 8 : 4;
        if (row >= rows)
            return;
        char *o = (char *)out + ((int64_t)row * ldo + v) * (OUT_BF16 ? 2 : 4);
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
    auto epilogue = [&](const float *sc, int m0, int v0) __attribute__((always_inline)) {
        float h[AM];
#pragma unroll
        for (int b = 0; b < AM; ++b)
            h[b] = sc[BV + wm * WM + b * 16 + r16];
#pragma unroll
        for (int q = 0; q < AV / 4; ++q) {
            f32x4_t w[4];
#pragma unroll
            for (int i = 0; i < 4; ++i)
                w[i] = *(const f32x4_t *)(sc + wv * WV + (4 * q + i) * 16 + 4 * qd);
#pragma unroll
            for (int b = 0; b < AM; ++b) {
                const int row = m0 + wm * WM + b * 16 + (r16 & 7);
                float x[4][4];
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        x[i][e] = (float)acc[4 * q + i][b][e] * h[b] * w[i][e];
                if constexpr (OUT_BF16) {
                    // neighbouring blocks: permlane16_swap gives a lane eight entries of one
                    uint32_t p[2][4];
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const auto s0 = __builtin_amdgcn_permlane16_swap(rows::pack_bf16(x[2 * i][0], x[2 * i][1]),
                                                                         rows::pack_bf16(x[2 * i + 1][0], x[2 * i + 1][1]),
                                                                         false, false);
                        const auto s1 = __builtin_amdgcn_permlane16_swap(rows::pack_bf16(x[2 * i][2], x[2 * i][3]),
                                                                         rows::pack_bf16(x[2 * i + 1][2], x[2 * i + 1][3]),
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
                            p[0][e] = __builtin_bit_cast(uint32_t, x[i][e]);
                            p[1][e] = __builtin_bit_cast(uint32_t, x[i + 1][e]);
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
            int rw = w0 * W_TILE, rh = H_BASE, kt = 0;
            int sc_at = next_w(next_w(rw));   // one K tile: the stage it does not use
            if constexpr (DMA_ON) {
                if (nk == 1)
                    issue_scales(sc_at, m0, v0);
            }
#pragma unroll
            for (int a = 0; a < AV; ++a)
                af[a] = *(const i32x4_t *)(smem + a_addr + rw + a * 16 * BK);
#pragma unroll
            for (int b = 0; b < AM; ++b)
                bf[0][b] = *(const i32x4_t *)(smem + b_addr + rh + b * 16 * BK);
            for (; kt + 2 < nk; ++kt) {
                // W's rows of K tile kt + 2 go to the stage the last barrier freed; the wait
                // leaves them in flight and needs the rest, K tile kt + 1
                if constexpr (DMA_ON)
                    issue_w(next_w(next_w(rw)), kt + 2);
                mma_load(rw, rh, 1, 0);
                interleave(DMA_ON ? LW : 0);
                __builtin_amdgcn_sched_barrier(0);
                wait_vm<LW>();
                bar();
                __builtin_amdgcn_sched_barrier(0);
                if constexpr (DMA_ON)
                    issue_h(rh, kt + 2);
                rw = next_w(rw);
                rh = next_h(rh);
                mma_load(rw, rh, 0, 1);
                interleave(DMA_ON ? LH : 0);
                __builtin_amdgcn_sched_barrier(0);
            }
            for (; kt < nk; ++kt) {
                mma_load(rw, rh, 1, 0);
                if (kt + 1 < nk) {
                    wait_vm<0>();
                    bar();
                    sc_at = rw;   // K tile nk - 2: its stage is free
                    if constexpr (DMA_ON)
                        issue_scales(sc_at, m0, v0);
                    rw = next_w(rw);
                    rh = next_h(rh);
                }
                mma_load(rw, rh, 0, 1);   // after the last K tile its reads are unused
            }
            // The scales have landed, and every wave's last fragments are in registers.  The
            // stores go first, then the next tile's requests: its first wait then leaves its
            // second K tile in flight instead of waiting for it behind these stores.
            wait_vm<0>();
            bar();
            epilogue((const float *)(smem + sc_at), m0, v0);
            zero_acc();
            w0 = (sc_at / W_TILE + 1) % WST;
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

// Small tiles: few rows, or too few 256 x 256 tiles to fill the chip.  BM x BV outputs per
// workgroup of four waves, WGM of them side by side along the rows; K tiles of 128 codes
// requested straight to LDS, NSTAGE - 1 of them ahead, in a ring with one barrier per step.
// Several workgroups share a CU, so one's start and end lie under the others' streams.
// STREAM: W is read once (one row tile): its requests take the streaming cache policy.
template <int BM, int BV, int WGM, int NSTAGE, bool STREAM, bool OUT_BF16>
__global__ __launch_bounds__(256) void gemm_int8_small_kernel(const int8_t *__restrict__ Hq,
                                                              const float *__restrict__ hs,
                                                              const int32_t *__restrict__ rows_dev, int32_t max_rows,
                                                              const int8_t *__restrict__ Wq,
                                                              const float *__restrict__ ws, int32_t V, int32_t d,
                                                              void *__restrict__ out, int64_t ldo)
{
    constexpr int BK = 128, CHUNKS = BK / 16, RPI = 64 / CHUNKS;
    constexpr int WGV = 4 / WGM, WM = BM / WGM, WV = BV / WGV, AM = WM / 16, AV = WV / 16;
    constexpr int W_TILE = BV * BK, STAGE = W_TILE + BM * BK;
    constexpr int LW = BV / RPI / 4, LH = BM / RPI / 4, T = LW + LH;   // requests per wave and K tile
    static_assert(LW >= 1 && LH >= 1 && NSTAGE >= 3 && (NSTAGE - 2) * T < 64, "requests");
    __shared__ __attribute__((aligned(1024))) char smem[NSTAGE * STAGE];

    const int rows = (int)rows::row_count(rows_dev, max_rows);
    const int nvt = (V + BV - 1) / BV, nmt = (rows + BM - 1) / BM, nblk = nvt * nmt;
    const int b = blockIdx.x;
    if (b >= nblk)
        return;
    // the workgroups of one XCD take a contiguous run of tiles, the row tiles of a vocabulary
    // tile one after another, so that they share its W rows in that XCD's L2
    const int q8 = nblk >> 3, rem = nblk & 7, xcd = b & 7, slot = b >> 3;
    const int t = (xcd < rem ? xcd * (q8 + 1) : rem * (q8 + 1) + (xcd - rem) * q8) + slot;
    const int m0 = t % nmt * BM, v0 = t / nmt * BV;
    const int nk = (d + BK - 1) / BK;

    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wv = wave % WGV, wm = wave / WGV;
    auto swz = [](int r) { return (r >> 1) & 7; };
    const int8_t *src[T];
    int chunk[T];
#pragma unroll
    for (int j = 0; j < T; ++j) {
        const int r = (j < LW ? wave * LW + j : wave * LH + j - LW) * RPI + lane / CHUNKS;
        chunk[j] = ((lane % CHUNKS) ^ swz(r)) * 16;
        src[j] = j < LW ? Wq + (int64_t)min(v0 + r, V - 1) * d : Hq + (int64_t)min(m0 + r, rows - 1) * d;
        src[j] += chunk[j];
    }
    auto issue = [&](int stage, int kt) __attribute__((always_inline)) {
        const int kb = kt * BK;
#pragma unroll
        for (int j = 0; j < T; ++j) {
            const int8_t *p = kb + chunk[j] < d ? src[j] + kb : kZeroCodes;
            char *at = smem + stage * STAGE + (j < LW ? (wave * LW + j) * 1024 : W_TILE + (wave * LH + j - LW) * 1024);
            if (j < LW)
                request<STREAM>(p, at);
            else
                request<false>(p, at);
        }
    };
    i32x4_t acc[AV][AM];
#pragma unroll
    for (int a = 0; a < AV; ++a)
#pragma unroll
        for (int m = 0; m < AM; ++m)
            acc[a][m] = i32x4_t{0, 0, 0, 0};
    const int r16 = lane & 15, qd = lane >> 4;
    const int lane_chunk = (qd ^ swz(r16)) * 16;
    const int a_addr = (wv * WV + r16) * BK + lane_chunk, b_addr = W_TILE + (wm * WM + r16) * BK + lane_chunk;

#pragma unroll
    for (int s = 0; s < NSTAGE - 1; ++s)
        if (s < nk)
            issue(s, s);
    int rd = 0;
    for (int kt = 0; kt < nk; ++kt) {
        // K tile kt has landed; the younger ones (NSTAGE - 2, fewer at the end) may not have
        if (kt + NSTAGE - 1 <= nk)
            wait_vm<(NSTAGE - 2) * T>();
        else
            wait_vm<0>();
        bar();   // every wave's part of it, and every wave is done with the stage read before
        if (kt + NSTAGE - 1 < nk)
            issue(rd == 0 ? NSTAGE - 1 : rd - 1, kt + NSTAGE - 1);
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            i32x4_t af[AV], bf[AM];
#pragma unroll
            for (int a = 0; a < AV; ++a)
                af[a] = *(const i32x4_t *)(smem + rd * STAGE + ((a_addr + a * 16 * BK) ^ (64 * s)));
#pragma unroll
            for (int m = 0; m < AM; ++m)
                bf[m] = *(const i32x4_t *)(smem + rd * STAGE + ((b_addr + m * 16 * BK) ^ (64 * s)));
#pragma unroll
            for (int a = 0; a < AV; ++a)
#pragma unroll
                for (int m = 0; m < AM; ++m)
                    acc[a][m] = __builtin_amdgcn_mfma_i32_16x16x64_i8(af[a], bf[m], acc[a][m], 0, 0, 0);
        }
        rd = rd + 1 == NSTAGE ? 0 : rd + 1;
    }
    const bool vec = ((uintptr_t)out & 15) == 0 && (ldo & 3) == 0;
#pragma unroll
    for (int a = 0; a < AV; ++a) {
        const int v = v0 + wv * WV + a * 16 + qd * 4;
        if (v >= V)
            continue;
        float w[4];
#pragma unroll
        for (int e = 0; e < 4; ++e)
            w[e] = ws[min(v + e, V - 1)];
#pragma unroll
        for (int m = 0; m < AM; ++m) {
            const int row = m0 + wm * WM + m * 16 + r16;
            if (row >= rows)
                continue;
            const float h = hs[row];
            float x[4];
#pragma unroll
            for (int e = 0; e < 4; ++e)
                x[e] = (float)acc[a][m][e] * h * w[e];
            store4<OUT_BF16>(out, (int64_t)row * ldo + v, x, v, V, vec);
        }
    }
}

}  // namespace

// Which form runs, from the sizes and the alignment alone (times of one launch on an MI355X,
// bf16 output; the forms give the same bits):
//  * codes that are not 16-byte aligned rows (d % 16 != 0): gemm_int8_any_kernel, in tiles of
//    32 x 128 (20 x 152064 x 3583: 141 us, 153 in tiles of 32 x 64, 189 of 64 x 64), 64 x 128 (64 x
//    152064 x 3585: 163 us, 188 of 64 x 64, 192 of 128 x 128), or 128 x 128 where these fill more
//    than half of the chip (1000 x 50000 x 2001: 241 us, 347 of 64 x 64; 200 x 8192 x 4095, 128
//    tiles: 45 against 39 us).
//  * so few outputs that 32 x 32 tiles fit on the chip at once, one on a CU: these, with more K
//    tiles under way (100 x 700 x 8192: 16 against 24 us; unaligned, d = 8001: 23 against 41 us;
//    20 x 4096 x 4096, 128 tiles: 9.6 against 12 us; 256 x 4096 x 4096, 1024 tiles: 23 against 15).
//  * at most 32 rows, at most 64 rows: W is streamed once past a row tile of 32 or 64 rows.
//    d = 3584, V = 152064, 20 rows: 86 us (6.4 TB/s), 106 us with tiles of 128 rows; 64 rows:
//    109 against 108 us, but 48 rows 104 against 105, 33 rows 96 against 108.  Vocabulary tiles
//    of 128 entries, or of 64 where that gives less than one workgroup per CU (64 x 30000 x 4096:
//    29 against 33 us).
//  * more rows, but too few 128 x 256 tiles to fill three eighths of the chip: 64 x 64 tiles.
//    200 x 8192 x 4096 (64 tiles of 128 x 256): 18 against 23 us; 512 x 8192 x 4096 (128 tiles):
//    33 against 24 us.
//  * else tiles of 128 or 256 rows, by the rounds that the CUs need for either, a tile of 128
//    rows at three fifths of one of 256 (it halves the products, but not the codes of W):
//    128 x 152064 x 3584: 111 against 147 us; 384 x 126464 x 4096: 208 against 223; 192 x 152064 x
//    3584: 161 against 148; 1229 x 126464 x 4096: 624 against 530.
//  * one row tile reads W once, with the streaming cache policy: 128 x 152064 x 3584: 111 against
//    119 us, 256 x 100000 x 2048: 69 against 75.  It holds for a smaller W too where other work
//    has been through the caches since the last call (20 x 50000 x 4096: 42 against 48 us; right
//    after a call that left W there, 39 against 32).  Rows of 128 or 256 whose d is no multiple of
//    128 go without it: 128 x 126464 x 4112: 130 us, 112 us for d = 4096 with it.
//  * a device-side count does not choose: `rows` does, the capacity.  Capacity 1229, V = 126464, d =
//    4096: 20 counted rows 136 us, 92 us in a call of 20; 128 rows 124 against 108.
hipError_t launch_gemm_int8(const int8_t *Hq, const float *hs, const int32_t *count, int64_t rows, const int8_t *Wq,
                            const float *ws, int64_t V, int64_t d, void *out, bool out_bf16, int64_t ldo,
                            hipStream_t stream)
{
    int dev = 0, cus = 256;
    if (hipGetDevice(&dev) == hipSuccess)
        (void)hipDeviceGetAttribute(&cus, hipDeviceAttributeMultiprocessorCount, dev);
    auto tiles = [&](int64_t bm, int64_t bv) { return ((V + bv - 1) / bv) * ((rows + bm - 1) / bm); };
    auto go = [&](auto kernel, int64_t grid, int threads, auto... more) {
        hipLaunchKernelGGL(kernel, dim3((unsigned)grid), dim3(threads), 0, stream, Hq, hs, count, (int32_t)rows, Wq,
                           ws, (int32_t)V, (int32_t)d, out, ldo, more...);
    };
    auto pick = [&](auto bf16_tag) {
        constexpr bool B = decltype(bf16_tag)::value;
        if (d % 16 != 0 || ((uintptr_t)Hq & 15) || ((uintptr_t)Wq & 15))
        {
            if (tiles(32, 32) <= cus)
                return go(gemm_int8_any_kernel<32, 32, 4, 2, 4, B>, tiles(32, 32), 256, kDefaultGroupM);
            if (rows <= 32 && tiles(32, 128) >= cus)
                return go(gemm_int8_any_kernel<32, 128, 4, 4, 4, B>, tiles(32, 128), 256, kDefaultGroupM);
            if (rows <= 32)
                return go(gemm_int8_any_kernel<32, 64, 4, 4, 4, B>, tiles(32, 64), 256, kDefaultGroupM);
            if (rows <= 64 && tiles(64, 128) >= cus)
                return go(gemm_int8_any_kernel<64, 128, 4, 4, 4, B>, tiles(64, 128), 256, kDefaultGroupM);
            if (rows <= 64 || tiles(128, 128) * 8 < cus * 5)
                return go(gemm_int8_any_kernel<64, 64, 4, 2, 4, B>, tiles(64, 64), 256, kDefaultGroupM);
            return go(gemm_int8_any_kernel<128, 128, 8, 4, 2, B>, tiles(128, 128), 512, kDefaultGroupM);
        }
        if (tiles(32, 32) <= cus)
            return go(gemm_int8_small_kernel<32, 32, 2, 8, false, B>, tiles(32, 32), 256);
        if (rows <= 32 && tiles(32, 128) >= cus)
            return go(gemm_int8_small_kernel<32, 128, 1, 4, true, B>, tiles(32, 128), 256);
        if (rows <= 32)
            return go(gemm_int8_small_kernel<32, 64, 1, 4, true, B>, tiles(32, 64), 256);
        if (rows <= 64 && tiles(64, 128) >= cus)
            return go(gemm_int8_small_kernel<64, 128, 1, 3, true, B>, tiles(64, 128), 256);
        if (rows <= 64)
            return go(gemm_int8_small_kernel<64, 64, 2, 4, true, B>, tiles(64, 64), 256);
        if (tiles(128, 256) * 8 < cus * 3)
            return go(gemm_int8_small_kernel<64, 64, 2, 4, false, B>, tiles(64, 64), 256);
        auto large = [&](auto bm_tag) {
            constexpr int BM = decltype(bm_tag)::value;
            const int64_t n = tiles(BM, 256);
            // one persistent workgroup per CU, a multiple of the eight XCDs
            const int64_t grid = std::min<int64_t>(std::max(8, cus / 8 * 8), (n + 7) / 8 * 8);
            if (d % 128 != 0)
                go(gemm_int8_kernel<BM, false, B, true>, grid, 512, kDefaultGroupM);
            else if (rows <= BM)
                go(gemm_int8_kernel<BM, true, B, false>, grid, 512, kDefaultGroupM);
            else
                go(gemm_int8_kernel<BM, false, B, false>, grid, 512, kDefaultGroupM);
        };
        auto rounds = [&](int64_t n) { return (n + cus - 1) / cus; };
        if (rounds(tiles(128, 256)) * 3 < rounds(tiles(256, 256)) * 5)
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
