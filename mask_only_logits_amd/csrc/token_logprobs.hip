// Log-probabilities of given tokens over rows of logits, the rows' entropies and top
// alternatives, and the gradient of log-probability and entropy.
//
// For a row of logits z_v (v < V), a given token t and a temperature T, with
//   m = max_v z_v,  x_v = (z_v - m) / T,  l = log sum_v exp(x_v),  p_v = exp(x_v - l):
//   logprob = x_t - l
//   H = -sum_v p_v log p_v = l - sum_v p_v x_v
//   alternatives: the largest z_v > -inf, the lower index first among equals, with x_v - l
//   d(g logprob + h H) / dz_v = (g ([v = t] - p_v) - h p_v (x_v - l + H)) / T.
// A token outside [0, V) is none: logprob 0, and no gradient from it.  A row with a NaN or
// +inf, or with nothing above -inf, has NaN everywhere and no alternatives.  m and l are kept
// apart, as their sum would lose bits of l.  All arithmetic is fp32; the gradient is rounded once.
#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>

#include <algorithm>

#include "launch_head.h"
#include "row_ops.h"

namespace mosaic {
namespace {

using namespace rows;

constexpr float kLog2e = 1.44269504088896340736f, kLn2 = 0.69314718055994530942f;
constexpr float kInf = __builtin_inff();
constexpr float kFar = -1000.0f;   // 2^kFar is 0

__device__ __forceinline__ float fast_exp2(float x) { return __builtin_amdgcn_exp2f(x); }

// Exponents of logits against their maximum m in powers of two, (z - m) c0 with c0 = log2(e) / T,
// taken as z c - k with one rounding; k = m c rounded, and what it lost, m c - k, is `off`.
// Where |m| c0 reaches 2^30 every logit counts as m or as nothing, and c is a power of two with
// which m c is exact and no product overflows.  An empty set (m = -inf) takes k = 0.
struct Ref {
    float c, k, off;

    __device__ __forceinline__ Ref(float m, float c0)
    {
        c = c0;
        k = m * c0;
        off = __builtin_fmaf(m, c0, -k);
        if (!(fabsf(k) < 0x1p30f)) {
            const int e = (int)((__builtin_bit_cast(uint32_t, m) >> 23) & 255u);
            if (m == -kInf) {
                k = off = 0.0f;
            } else if (e < 255) {
                c = __builtin_bit_cast(float, (uint32_t)(294 - e) << 23);   // m c in [2^40, 2^41)
                k = m * c;
                off = 0.0f;
            }
        }
    }
    __device__ __forceinline__ float at(float z) const { return __builtin_fmaf(z, c, -k); }
};

// (z - m) / T, with the difference in halves so that it stays inside fp32
__device__ __forceinline__ float exponent(float z, float m, float T) { return 2.0f * ((0.5f * z - 0.5f * m) / T); }

// Of a set of logits: the maximum m, s = sum of 2^y and u = sum of 2^y y, y = (z - m) c0.
struct Sums {
    float m = -kInf, s = 0.0f, u = 0.0f;

    __device__ __forceinline__ void join(float m2, float s2, float u2, float c0)
    {
        const float mx = fmaxf(m, m2);
        raise(mx, c0);
        Sums o;
        o.m = m2;
        o.s = s2;
        o.u = u2;
        o.raise(mx, c0);
        s += o.s;
        u += o.u;
    }
    // the same set against a larger maximum
    __device__ __forceinline__ void raise(float mx, float c0)
    {
        const float y = m == -kInf ? kFar : fmaxf((m - mx) * c0, kFar), f = fast_exp2(y);
        u = f * (u + y * s);   // (2^y y of the set's maximum counts too)
        s = f * s;
        m = mx;
    }
    __device__ __forceinline__ void join_wave(float c0)
    {
#pragma unroll
        for (int o = 32; o >= 1; o >>= 1)
            join(__shfl_xor(m, o, 64), __shfl_xor(s, o, 64), __shfl_xor(u, o, 64), c0);
    }
};

// The sums over a stream of logits.
template <bool ENT>
struct RunningSums {
    float m = -kInf, s = 0.0f, u = 0.0f, c0;   // s and u of y + off
    Ref ref;

    __device__ __forceinline__ RunningSums(float c) : c0(c), ref(-kInf, c) {}
    __device__ __forceinline__ Sums done() const
    {
        const float f = fast_exp2(-ref.off);
        Sums x;
        x.m = m;
        x.s = f * s;
        x.u = f * (u - ref.off * s);
        return x;
    }
    __device__ __forceinline__ void raise(float mx)
    {
        Sums x = done();
        x.raise(mx, c0);
        m = mx;
        ref = Ref(mx, c0);
        const float f = fast_exp2(ref.off);
        s = f * x.s;
        u = f * (x.u + ref.off * x.s);
    }
    template <int N>
    __device__ __forceinline__ void add(const float (&z)[N])
    {
        float mx = fmaxf(fmaxf(z[0], z[1]), fmaxf(z[2], z[3]));
        if constexpr (N == 8)
            mx = fmaxf(mx, fmaxf(fmaxf(z[4], z[5]), fmaxf(z[6], z[7])));
        if (mx > m)
            raise(mx);
        float e[N], w[N];
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const float y = ref.at(z[i]);
            e[i] = fast_exp2(y);
            if constexpr (ENT)
                w[i] = fmaxf(y, kFar);   // (2^y y is 0 for z = -inf)
        }
        float a = (e[0] + e[1]) + (e[2] + e[3]);
        if constexpr (N == 8)
            a += (e[4] + e[5]) + (e[6] + e[7]);
        s += a;
        if constexpr (ENT) {
            float b = 0.0f;
#pragma unroll
            for (int i = 0; i < N; ++i)
                b = __builtin_fmaf(e[i], w[i], b);
            u += b;
        }
    }
};

// What the threads of a workgroup know of a row after the sums.
struct Row {
    float m, l, H;
    bool fine;   // a maximum, and sums that are numbers

    __device__ __forceinline__ Row(const Sums &x)
    {
        m = x.m;
        fine = x.m != -kInf && x.s >= 1.0f - 0x1p-8f && x.s < kInf;
        // (the maximum's own term is 1, so what lies below 1, or H below 0, is rounding)
        l = fine ? logf(fmaxf(x.s, 1.0f)) : __builtin_nanf("");
        H = fine ? fmaxf(l - kLn2 * (x.u / x.s), 0.0f) : __builtin_nanf("");
    }
};

// Chunks of N logits of [lo, hi), lo a multiple of N: chunk i of this thread's is
// lo / N + threadIdx.x + i * NT.  UN loads are issued before their values are used.  The chunk
// that hi cuts is filled up with -inf.
template <bool BF16, int NT, int UN, bool STREAM, typename F>
__device__ __forceinline__ void for_chunks(const TokenLogprobs &a, int64_t row, int lo, int hi, F f)
{
    constexpr int N = kChunk<BF16>;
    const int64_t base = row * a.ldz;
    const int full = lo + (hi - lo) / N * N;
    for (int v = lo + threadIdx.x * N; v < full; v += UN * NT * N) {
        Raw<BF16> r[UN];
#pragma unroll
        for (int i = 0; i < UN; ++i)
            if (v + i * NT * N < full)
                r[i].template load<STREAM>(a.Z, base + v + i * NT * N);
#pragma unroll
        for (int i = 0; i < UN; ++i) {
            if (v + i * NT * N < full) {
                float z[N];
                r[i].get(z);
                f(z, v + i * NT * N, N);
            }
        }
    }
    if (full < hi && threadIdx.x == NT - 1) {
        Raw<BF16> r;
        r.fill(-kInf);
        r.load_part(a.Z, base + full, hi - full);
        float z[N];
        r.get(z);
        f(z, full, hi - full);
    }
}

// Keys that order logits, the lower index first among equals (+0 and -0 are equal); 0 is none.
__device__ __forceinline__ uint32_t order_of(float z)
{
    const uint32_t b = __builtin_bit_cast(uint32_t, z + 0.0f);
    return b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ uint64_t key_of(float z, int v) { return (uint64_t)order_of(z) << 32 | (uint32_t)~v; }
__device__ __forceinline__ int index_of(uint64_t key) { return (int)~(uint32_t)key; }
__device__ __forceinline__ float value_of(uint64_t key)
{
    const uint32_t o = (uint32_t)(key >> 32);
    return __builtin_bit_cast(float, o & 0x80000000u ? o & 0x7fffffffu : ~o);
}
constexpr uint32_t kOrderOfMinusInf = 0x007fffffu;   // keys above this value's are logits that count

// Words of LDS that select_top takes beside its list.
constexpr int kSelectWords = 256 + 4;

// The keys of the row's n largest logits above -inf into list[0 .. return value), in any order; NT
// threads.  Digits of the n-th largest key are found one after another, eight bits a pass over
// the row, so this takes up to nine passes, whatever the logits.
template <bool BF16, int NT>
__device__ int select_top(const TokenLogprobs &a, int64_t row, int n, uint64_t *list, int32_t *lds)
{
    int32_t *hist = lds, *found = lds + 256;   // found: digit, still needed, all taken, entries listed
    uint64_t prefix = 0;
    int need = n;
    bool all = false;
    for (int shift = 56; shift >= 0 && !all; shift -= 8) {
        for (int i = threadIdx.x; i < 256; i += NT)
            hist[i] = 0;
        __syncthreads();
        for_chunks<BF16, NT, 4, false>(a, row, 0, a.V, [&](auto &z, int v, int cnt) {
#pragma unroll
            for (int i = 0; i < kChunk<BF16>; ++i) {
                const uint64_t key = key_of(z[i], v + i);
                if (i < cnt && (uint32_t)(key >> 32) > kOrderOfMinusInf && (shift == 56 || key >> (shift + 8) == prefix))
                    atomicAdd(&hist[(int)(key >> shift) & 255], 1);
            }
        });
        __syncthreads();
        if (threadIdx.x < 64) {
            // lane i: digits 255 - 4 i and the three below; how many lie above them
            const int lane = threadIdx.x;
            int h[4], sum = 0;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                h[j] = hist[255 - 4 * lane - j];
                sum += h[j];
            }
            int upto = sum;
#pragma unroll
            for (int o = 1; o < 64; o <<= 1) {
                const int x = __shfl_up(upto, o, 64);
                upto += lane >= o ? x : 0;
            }
            int above = upto - sum;
            const int total = __shfl(upto, 63, 64);
            if (lane == 0 && total <= need) {   // fewer than asked for: all of them
                found[0] = 0;
                found[1] = 0;
                found[2] = 1;
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                if (total > need && above < need && above + h[j] >= need) {
                    found[0] = 255 - 4 * lane - j;
                    found[1] = need - above;
                    found[2] = above + h[j] == need;
                }
                above += h[j];
            }
        }
        __syncthreads();
        if (found[1] == 0) {   // (in the first pass only: later ones have `need` keys at least)
            prefix = 0;
        } else {
            prefix = prefix << 8 | (uint32_t)found[0];
            need = found[1];
        }
        all = found[2] != 0;
        if (all)
            prefix = found[1] == 0 ? 0 : prefix << shift;   // its keys with any digits after
        __syncthreads();
    }
    if (threadIdx.x == 0)
        found[3] = 0;
    __syncthreads();
    for_chunks<BF16, NT, 4, false>(a, row, 0, a.V, [&](auto &z, int v, int cnt) {
#pragma unroll
        for (int i = 0; i < kChunk<BF16>; ++i) {
            const uint64_t key = key_of(z[i], v + i);
            if (i < cnt && (uint32_t)(key >> 32) > kOrderOfMinusInf && key >= prefix) {
                const int at = atomicAdd(&found[3], 1);
                if (at < kTopMax)   // (n at most)
                    list[at] = key;
            }
        }
    });
    __syncthreads();
    return min(found[3], n);
}

// Writes the row's alternatives from a list of `listed` keys that holds the n largest: each
// thread counts the keys above its own.  Places without one take -1 and -inf.
template <int NT>
__device__ __forceinline__ void write_top(const TokenLogprobs &a, int64_t row, const Row &x, const uint64_t *list,
                                          int listed)
{
    for (int i = threadIdx.x; i < listed; i += NT) {
        const uint64_t key = list[i];
        int place = 0;
        for (int j = 0; j < listed; ++j)
            place += list[j] > key;
        if (place < a.top_n) {
            a.top_ids[row * a.top_n + place] = index_of(key);
            a.top_logprobs[row * a.top_n + place] = exponent(value_of(key), x.m, a.temperature) - x.l;
        }
    }
    for (int i = listed + threadIdx.x; i < a.top_n; i += NT) {
        a.top_ids[row * a.top_n + i] = -1;
        a.top_logprobs[row * a.top_n + i] = x.fine ? -kInf : x.l;
    }
}

// Everything but the alternatives, by one thread.
__device__ __forceinline__ void write_row(const TokenLogprobs &a, int64_t row, const Row &x, float z_token, bool token)
{
    a.stats[2 * row] = x.m;
    a.stats[2 * row + 1] = x.l;
    if (a.logprob)
        a.logprob[row] = token ? exponent(z_token, x.m, a.temperature) - x.l : 0.0f;
    if (a.entropy)
        a.entropy[row] = x.H;
}

// One row per workgroup.
template <bool BF16, int NT, bool ENT>
__global__ __launch_bounds__(NT) void token_logprobs_row_kernel(const TokenLogprobs a)
{
    constexpr int NW = NT / 64;
    __shared__ float part[3 * NW];
    __shared__ int32_t words[kSelectWords];
    __shared__ uint64_t list[kTopMax];
    const float c0 = kLog2e / a.temperature;
    const int64_t n = row_count(a.count, a.rows);
    for (int64_t row = blockIdx.x; row < n; row += gridDim.x) {
        RunningSums<ENT> run(c0);
        for_chunks<BF16, NT, 4, false>(a, row, 0, a.V, [&](auto &z, int, int) { run.add(z); });
        Sums x = run.done();
        x.join_wave(c0);
        if ((threadIdx.x & 63) == 0) {
            part[threadIdx.x >> 6] = x.m;
            part[NW + (threadIdx.x >> 6)] = x.s;
            part[2 * NW + (threadIdx.x >> 6)] = x.u;
        }
        __syncthreads();
        x = Sums();
        for (int w = 0; w < NW; ++w)
            x.join(part[w], part[NW + w], part[2 * NW + w], c0);
        const Row r(x);
        if (threadIdx.x == 0) {
            const int32_t t = a.tokens ? a.tokens[row] : -1;
            const bool token = t >= 0 && t < a.V;
            write_row(a, row, r, token ? load1(a.Z, row * a.ldz + t, BF16) : 0.0f, token);
        }
        if (a.top_n > 0) {
            const int listed = r.fine ? select_top<BF16, NT>(a, row, a.top_n, list, words) : 0;
            write_top<NT>(a, row, r, list, listed);
        }
        __syncthreads();   // the LDS is taken again for the next row
    }
}

// The gradient of a stretch of a row, element by element: it may be written over the logits.
template <bool BF16, int NT>
__global__ __launch_bounds__(NT) void token_logprobs_grad_kernel(const TokenLogprobs a, int cuts)
{
    constexpr int N = kChunk<BF16>;
    const int64_t n = row_count(a.count, a.rows);
    for (int64_t b = blockIdx.x; b < n * cuts; b += gridDim.x) {
        const int64_t row = b / cuts;
        const int s = (int)(b % cuts), chunks = (a.V + 7) / 8, each = (chunks + cuts - 1) / cuts;
        const int lo = min(s * each, chunks) * 8, hi = min(min((s + 1) * each, chunks) * 8, a.V);
        const float m = a.stats[2 * row], l = a.stats[2 * row + 1], inv = 1.0f / a.temperature;
        const int32_t t = a.tokens ? a.tokens[row] : -1;
        const bool token = t >= 0 && t < a.V && a.grad_logprob;
        const float g = token ? a.grad_logprob[row] * inv : 0.0f;
        const float h = a.grad_entropy ? a.grad_entropy[row] * inv : 0.0f;
        const float H = a.grad_entropy ? a.entropy[row] : 0.0f;
        const Ref ref(m, kLog2e / a.temperature);
        const float scale = fast_exp2(-ref.off) / expf(l);
        // log p + H = y ln 2 + this
        const float add = H - l - ref.off * kLn2;
        for_chunks<BF16, NT, 4, false>(a, row, min(lo, hi), hi, [&](auto &z, int v, int cnt) {
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const float y = ref.at(z[i]), p = scale * fast_exp2(y);
                const float w = -__builtin_fmaf(h, __builtin_fmaf(fmaxf(y, kFar), kLn2, add), g);
                z[i] = __builtin_fmaf(p, w, v + i == t ? g : 0.0f);
            }
            store_upto<BF16>(a.grad, row * a.ldg + v, z, cnt);
        });
    }
}

template <bool BF16>
hipError_t run(const TokenLogprobs &a, hipStream_t stream)
{
    const dim3 grid((unsigned)std::min<int64_t>(a.rows, 1 << 20));
    if (a.entropy)
        hipLaunchKernelGGL((token_logprobs_row_kernel<BF16, 1024, true>), grid, dim3(1024), 0, stream, a);
    else
        hipLaunchKernelGGL((token_logprobs_row_kernel<BF16, 1024, false>), grid, dim3(1024), 0, stream, a);
    return hipGetLastError();
}

template <bool BF16>
hipError_t run_grad(const TokenLogprobs &a, hipStream_t stream)
{
    const int cuts = std::max(1, a.V / 16384);
    hipLaunchKernelGGL((token_logprobs_grad_kernel<BF16, 256>), dim3((unsigned)std::min<int64_t>(a.rows * cuts, 1 << 20)),
                       dim3(256), 0, stream, a, cuts);
    return hipGetLastError();
}

}  // namespace

int64_t token_logprobs_workspace_bytes(int64_t, int64_t, int64_t) { return 0; }

hipError_t launch_token_logprobs(const TokenLogprobs &a, bool z_bf16, hipStream_t stream)
{
    return z_bf16 ? run<true>(a, stream) : run<false>(a, stream);
}

hipError_t launch_token_logprobs_grad(const TokenLogprobs &a, bool z_bf16, hipStream_t stream)
{
    return z_bf16 ? run_grad<true>(a, stream) : run_grad<false>(a, stream);
}

}  // namespace mosaic
