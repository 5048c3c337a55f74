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
#include <type_traits>

#include "launch_head.h"
#include "row_ops.h"

namespace mosaic {
namespace {

using namespace rows;

constexpr float kLog2e = 1.44269504088896340736f, kLn2 = 0.69314718055994530942f;
constexpr float kInf = __builtin_inff();
constexpr float kFar = -1000.0f;   // 2^kFar is 0
// Chunks of 16 bytes that a thread requests together (1229 x 126464 bf16 with two alternatives: 60 us,
// with four 64 us; short rows gain by four what long ones lose).
constexpr int kAhead = 8;
constexpr int64_t kLaunchRows = (int64_t)1 << 23;   // rows of a launch
// Rows are split for kPartTarget workgroups, four on each of 256 CUs, into parts of kPartMin logits or
// more (20 x 152064 with 20 alternatives: 14.8 us, parts of 4096 or 8192 15.4, whole 25.9; 4 x
// 32000 with 64: whole 15.7, in parts of 8192 21.7, as the join has more keys to look at).
constexpr int kPartsMax = 64, kPartTarget = 1024, kPartMin = 16384;

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
    // of the wave's lanes (lane 0's, as joins that round differently leave the lanes bits apart)
    __device__ __forceinline__ void join_wave(float c0)
    {
#pragma unroll
        for (int o = 32; o >= 1; o >>= 1)
            join(__shfl_xor(m, o, 64), __shfl_xor(s, o, 64), __shfl_xor(u, o, 64), c0);
        m = __shfl(m, 0, 64);
        s = __shfl(s, 0, 64);
        u = __shfl(u, 0, 64);
    }
};

template <int N>
__device__ __forceinline__ float max_of(const float (&z)[N])
{
    float a = fmaxf(fmaxf(z[0], z[1]), fmaxf(z[2], z[3]));
    if constexpr (N == 8)
        a = fmaxf(a, fmaxf(fmaxf(z[4], z[5]), fmaxf(z[6], z[7])));
    return a;
}

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
    __device__ __forceinline__ void add(const float (&z)[N], float mx)   // mx: the largest
    {
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

// Calls f(z, v, count, round) for this thread's chunks z of N logits of [lo, hi), lo a multiple of N:
// in round c the one at v = lo + (c NT + threadIdx.x) N.  UN loads are issued before their values are
// used.  The chunk that hi cuts is filled up with -inf.  (Rounds that all threads take are counted
// in scalar registers, and their loads have a scalar base.)
template <bool BF16, int NT, int UN, bool STREAM, typename F>
__device__ __forceinline__ void for_chunks(const TokenLogprobs &a, int64_t row, int lo, int hi, F f)
{
    constexpr int N = kChunk<BF16>;
    const int t = threadIdx.x, rounds = (hi - lo) / (NT * N);
    const char *from = (const char *)a.Z + (row * a.ldz + lo) * (16 / N);
    auto some = [&](int c, auto whole) __attribute__((always_inline)) {
        constexpr bool W = decltype(whole)::value;
        Raw<BF16> r[UN];
#pragma unroll
        for (int i = 0; i < UN; ++i)
            if (W || c + i < rounds)
                r[i].template load<STREAM>(from + (int64_t)(c + i) * (NT * 16) + t * 16u, 0);
#pragma unroll
        for (int i = 0; i < UN; ++i) {
            if (W || c + i < rounds) {
                float z[N];
                r[i].get(z);
                f(z, lo + ((c + i) * NT + t) * N, N, c + i);
            }
        }
    };
    int c = 0;
    for (; c + UN <= rounds; c += UN)
        some(c, std::true_type{});
    const int v = lo + (rounds * NT + t) * N;
    Raw<BF16> r;
    if (v + N <= hi) {
        r.template load<STREAM>(from + (int64_t)rounds * (NT * 16) + t * 16u, 0);
    } else {
        r.fill(-kInf);
        if (v < hi)
            r.load_part(a.Z, row * a.ldz + v, hi - v);
    }
    if (c < rounds)
        some(c, std::false_type{});
    if (v < hi) {
        float z[N];
        r.get(z);
        f(z, v, min(N, hi - v), rounds);
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
constexpr int kListMax = 512;

// The keys of the n largest logits of [lo, hi) above -inf into list[0 .. return value), in any order; NT
// threads.  Digits of the n-th largest key are found one after another, eight bits a pass over
// the row, so this takes up to nine passes, whatever the logits; they are written for few registers.
template <bool BF16, int NT>
__device__ int select_top(const TokenLogprobs &a, int64_t row, int lo, int hi, int n, uint64_t *list, int32_t *lds)
{
    int32_t *hist = lds, *found = lds + 256;   // found: digit, still needed, all taken, entries listed
    uint64_t prefix = 0;
    int need = n;
    bool all = false;
#pragma unroll 1
    for (int shift = 56; shift >= 0 && !all; shift -= 8) {
        for (int i = threadIdx.x; i < 256; i += NT)
            hist[i] = 0;
        __syncthreads();
#pragma unroll 1
        for (int v = lo + threadIdx.x; v < hi; v += NT) {
            const uint64_t key = key_of(load1(a.Z, row * a.ldz + v, BF16), v);
            if ((uint32_t)(key >> 32) > kOrderOfMinusInf && (shift == 56 || key >> (shift + 8) == prefix))
                atomicAdd(&hist[(int)(key >> shift) & 255], 1);
        }
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
#pragma unroll 1
    for (int v = lo + threadIdx.x; v < hi; v += NT) {
        const uint64_t key = key_of(load1(a.Z, row * a.ldz + v, BF16), v);
        if ((uint32_t)(key >> 32) > kOrderOfMinusInf && key >= prefix) {
            const int at = atomicAdd(&found[3], 1);
            if (at < kTopMax)   // (n at most)
                list[at] = key;
        }
    }
    __syncthreads();
    return min(found[3], n);
}

// A thread's largest logit and the round of the chunk that holds it, and the largest maximum of its other chunks.
struct Best {
    float m = -kInf, m2 = -kInf;
    int at = 0;

    __device__ __forceinline__ void add(float mx, int round)
    {
        m2 = fmaxf(m2, fminf(mx, m));
        at = mx > m ? round : at;
        m = fmaxf(m, mx);
    }
};

// LDS of the search for the top n.
struct TopLds {
    uint64_t key[256];
    uint64_t list[kListMax];
    uint64_t least;
    int32_t listed;
    int32_t words[kSelectWords];
};

// A key that n of the workgroup's logits reach, from one key of a logit (or 0) of each of its 256
// threads: the n-th largest of the keys, of groups of four threads for small n.  The lowest key that
// counts where there are fewer.
__device__ __forceinline__ uint64_t least_key(uint64_t mine, int n, TopLds &lds)
{
    const int t = threadIdx.x;
    int groups = 256;
    if (n <= 32) {
        groups = 64;
#pragma unroll
        for (int o = 32; o >= 16; o >>= 1)
            mine = max(mine, (uint64_t)__shfl_xor((unsigned long long)mine, o, 64));
        if ((t & 63) < 16)
            lds.key[(t >> 6) * 16 + (t & 15)] = mine;
    } else {
        lds.key[t] = mine;
    }
    if (t == 0) {
        lds.least = (uint64_t)(kOrderOfMinusInf + 1) << 32;
        lds.listed = 0;
    }
    __syncthreads();
    if (t < groups) {
        const uint64_t k = lds.key[t];
        int above = 0;
#pragma unroll 16
        for (int j = 0; j < groups; ++j)
            above += lds.key[j] > k;
        if (k != 0 && above == n - 1)   // (keys of logits are distinct)
            lds.least = k;
    }
    __syncthreads();
    return lds.least;
}

__device__ __forceinline__ void list_key(uint64_t key, TopLds &lds)
{
    const int at = atomicAdd(&lds.listed, 1);
    if (at < kListMax)
        lds.list[at] = key;
}

// The keys of [lo, hi)'s n largest logits, and of some below, into lds.list; how many.  256 threads,
// each with the `best` of its chunks.  Chunks with a logit that may count are read again: of a
// thread the one with its maximum, and where another may hold one all of them.
template <bool BF16>
__device__ int list_top(const TokenLogprobs &a, int64_t row, int lo, int hi, const Best &best, TopLds &lds)
{
    constexpr int N = kChunk<BF16>, NT = 256;
    auto chunk = [&](int64_t round, int t) { return lo + (round * NT + t) * N; };
    // (of the maximum's chunk the last entry, as the place of the maximum in it is not known)
    const uint64_t least =
        least_key(best.m > -kInf ? key_of(best.m, (int)chunk(best.at, threadIdx.x) + N - 1) : 0, a.top_n, lds);
    auto look = [&](int v) __attribute__((always_inline)) {
        Raw<BF16> r;
        if (v + N <= hi) {
            r.load(a.Z, row * a.ldz + v);
        } else {
            r.fill(-kInf);
            r.load_part(a.Z, row * a.ldz + v, hi - v);
        }
        float z[N];
        r.get(z);
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const uint64_t key = key_of(z[i], v + i);
            if (key >= least)   // (what fills a chunk up is -inf)
                list_key(key, lds);
        }
    };
    auto counts = [&](float z) { return z > -kInf && order_of(z) >= (uint32_t)(least >> 32); };
    if (counts(best.m))
        look((int)chunk(best.at, threadIdx.x));
    for (uint64_t more = __ballot(counts(best.m2)); more != 0; more &= more - 1) {
        const int from = __builtin_ctzll(more), t = (int)(threadIdx.x & ~63u) + from;
        const int seen = __shfl(best.at, from, 64);
        for (int c = threadIdx.x & 63; chunk(c, t) < hi; c += 64)
            if (c != seen)
                look((int)chunk(c, t));
    }
    __syncthreads();
    int listed = lds.listed;
    if (listed > kListMax)
        listed = select_top<BF16, NT>(a, row, lo, hi, a.top_n, lds.list, lds.words);
    return listed;
}

// Calls put(place, key) for the n largest keys other than 0 of a list: each thread counts the keys
// above its own.
template <typename F>
__device__ __forceinline__ void place_top(const uint64_t *list, int listed, int n, F put)
{
    for (int i = threadIdx.x; i < listed; i += 256) {
        const uint64_t key = list[i];
        int place = 0;
#pragma unroll 8
        for (int j = 0; j < listed; ++j)
            place += list[j] > key;
        if (place < n && key != 0)
            put(place, key);
    }
}

// Writes the row's alternatives from a list with its n largest keys, all there are if those are
// fewer.  Places without one take -1 and -inf.
__device__ __forceinline__ void write_top(const TokenLogprobs &a, int64_t row, const Row &x, const uint64_t *list,
                                          int listed)
{
    place_top(list, listed, a.top_n, [&](int place, uint64_t key) {
        a.top_ids[row * a.top_n + place] = index_of(key);
        a.top_logprobs[row * a.top_n + place] = exponent(value_of(key), x.m, a.temperature) - x.l;
    });
    for (int i = listed + threadIdx.x; i < a.top_n; i += 256) {
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

// The token of a row, and its logit.
struct Token {
    bool given = false;
    float z = 0.0f;

    template <bool BF16>
    __device__ __forceinline__ void load(const TokenLogprobs &a, int64_t row)
    {
        const int32_t t = a.tokens ? a.tokens[row] : -1;
        given = t >= 0 && t < a.V;
        if (given)
            z = load1(a.Z, row * a.ldz + t, BF16);
    }
};

// The sums of [lo, hi) of a row in every thread of 256, and the thread's own best.  A thread's sums
// start anew every 512 chunks, so that their rounding does not grow with the row.
template <bool BF16, bool ENT, bool TOP>
__device__ __forceinline__ Sums scan(const TokenLogprobs &a, int64_t row, int lo, int hi, Best &best, float *part)
{
    constexpr int NT = 256, NW = NT / 64, ROUNDS = 512, RUN = ROUNDS * NT * kChunk<BF16>;
    const float c0 = kLog2e / a.temperature;
    Sums x;
    for (int at = lo, before = 0; at < hi; at += RUN, before += ROUNDS) {
        RunningSums<ENT> run(c0);
        for_chunks<BF16, NT, kAhead, true>(a, row, at, min(hi, at + RUN), [&](auto &z, int, int, int round) {
            const float mx = max_of(z);
            if constexpr (TOP)
                best.add(mx, before + round);
            run.add(z, mx);
        });
        const Sums y = run.done();
        x.join(y.m, y.s, y.u, c0);
    }
    x.join_wave(c0);
    if ((threadIdx.x & 63) == 0) {
        part[threadIdx.x >> 6] = x.m;
        part[NW + (threadIdx.x >> 6)] = x.s;
        part[2 * NW + (threadIdx.x >> 6)] = x.u;
    }
    __syncthreads();
    x = Sums();
#pragma unroll
    for (int w = 0; w < NW; ++w)
        x.join(part[w], part[NW + w], part[2 * NW + w], c0);
    return x;
}

// One row per workgroup, from row `from` on.
template <bool BF16, bool ENT, bool TOP>
__global__ __launch_bounds__(256) void token_logprobs_row_kernel(const TokenLogprobs a, int64_t from)
{
    __shared__ float part[12];
    __shared__ TopLds lds;
    const int64_t n = row_count(a.count, a.rows);
    const int64_t row = from + blockIdx.x;
    if (row >= n)
        return;
    Token token;
    if (threadIdx.x == 0)
        token.load<BF16>(a, row);
    Best best;
    const Row r(scan<BF16, ENT, TOP>(a, row, 0, a.V, best, part));
    if (threadIdx.x == 0)
        write_row(a, row, r, token.z, token.given);
    if constexpr (TOP) {
        const int listed = r.fine ? list_top<BF16>(a, row, 0, a.V, best, lds) : 0;
        write_top(a, row, r, lds.list, listed);
    }
}

// What a split row's parts leave in the workspace: each part's largest key, each one's second and so
// on, 0 without a logit, so that the join's threads get keys of all sizes; then m, s and u of each.
struct Parts {
    uint64_t *keys;
    float *sums;
    int parts;

    __host__ __device__ Parts(const TokenLogprobs &a, int parts_) : parts(parts_)
    {
        keys = (uint64_t *)a.workspace;
        sums = (float *)(keys + a.rows * parts * a.top_n);
    }
};

// A part of a row per workgroup.
template <bool BF16, bool ENT, bool TOP>
__global__ __launch_bounds__(256) void token_logprobs_part_kernel(const TokenLogprobs a, const Parts out)
{
    __shared__ float part[12];
    __shared__ TopLds lds;
    const int64_t n = row_count(a.count, a.rows);
    const int parts = out.parts, chunks = (a.V + 7) / 8, each = (chunks + parts - 1) / parts;
    const int64_t b = blockIdx.x;
    if (b >= n * parts)
        return;
    const int64_t row = b / parts;
    const int s = (int)(b % parts);
    const int lo = min(s * each, chunks) * 8, hi = max(lo, min(min((s + 1) * each, chunks) * 8, a.V));
    Best best;
    const Sums x = scan<BF16, ENT, TOP>(a, row, min(lo, hi), hi, best, part);
    if (threadIdx.x == 0) {
        out.sums[3 * b] = x.m;
        out.sums[3 * b + 1] = x.s;
        out.sums[3 * b + 2] = x.u;
    }
    if constexpr (TOP) {
        const int listed = list_top<BF16>(a, row, lo, hi, best, lds);
        uint64_t *keys = out.keys + row * a.top_n * parts + s;
        place_top(lds.list, listed, a.top_n, [&](int place, uint64_t key) { keys[place * parts] = key; });
        for (int i = listed + threadIdx.x; i < a.top_n; i += 256)
            keys[i * parts] = 0;
    }
}

// Joins the parts of a row, kPartsMax at most.
template <bool BF16, bool TOP>
__global__ __launch_bounds__(256) void token_logprobs_join_kernel(const TokenLogprobs a, const Parts in)
{
    __shared__ uint64_t all[TOP ? kPartsMax * kTopMax : 1];
    __shared__ TopLds lds;
    const int64_t n = row_count(a.count, a.rows);
    const float c0 = kLog2e / a.temperature;
    const int64_t row = blockIdx.x;
    if (row >= n)
        return;
    Token token;
    if (threadIdx.x == 0)
        token.load<BF16>(a, row);
    Sums x;
    const int lane = threadIdx.x & 63;
    if (lane < in.parts) {
        const float *p = in.sums + 3 * (row * in.parts + lane);
        x.m = p[0];
        x.s = p[1];
        x.u = p[2];
    }
    x.join_wave(c0);
    const Row r(x);
    if (threadIdx.x == 0)
        write_row(a, row, r, token.z, token.given);
    if constexpr (TOP) {
        const int total = r.fine ? in.parts * a.top_n : 0;
        uint64_t mine = 0;
        for (int i = threadIdx.x; i < total; i += 256) {
            all[i] = in.keys[row * in.parts * a.top_n + i];
            mine = max(mine, all[i]);
        }
        const uint64_t least = least_key(mine, a.top_n, lds);
        for (int i = threadIdx.x; i < total; i += 256)
            if (all[i] >= least)
                list_key(all[i], lds);
        __syncthreads();
        const int listed = lds.listed;
        write_top(a, row, r, listed > kListMax ? all : lds.list, listed > kListMax ? total : listed);
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
        for_chunks<BF16, NT, 4, false>(a, row, min(lo, hi), hi, [&](auto &z, int v, int cnt, int) {
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

// Parts of a row: few rows are split so that the chip is filled.  (The workspace's size is the same
// on every device, so this counts with 256 CUs.)
int parts_of(int64_t rows, int64_t V)
{
    const int64_t n = std::min<int64_t>({kPartsMax, kPartTarget / std::max<int64_t>(rows, 1), V / kPartMin});
    return (int)std::max<int64_t>(n, 1);
}

template <bool BF16>
hipError_t run(const TokenLogprobs &a, hipStream_t stream)
{
    const int parts = parts_of(a.rows, a.V);
    const Parts p(a, parts);
    auto go = [&](auto ent, auto top) {
        constexpr bool E = decltype(ent)::value, T = decltype(top)::value;
        if (parts == 1) {
            // (a launch holds fewer than 2^32 threads)
            for (int64_t from = 0; from < a.rows; from += kLaunchRows)
                hipLaunchKernelGGL((token_logprobs_row_kernel<BF16, E, T>),
                                   dim3((unsigned)std::min(a.rows - from, kLaunchRows)), dim3(256), 0, stream, a, from);
            return;
        }
        hipLaunchKernelGGL((token_logprobs_part_kernel<BF16, E, T>), dim3((unsigned)(a.rows * parts)), dim3(256), 0,
                           stream, a, p);
        hipLaunchKernelGGL((token_logprobs_join_kernel<BF16, T>), dim3((unsigned)a.rows), dim3(256), 0, stream, a, p);
    };
    auto with = [&](auto ent) { a.top_n > 0 ? go(ent, std::true_type{}) : go(ent, std::false_type{}); };
    a.entropy ? with(std::true_type{}) : with(std::false_type{});
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

int64_t token_logprobs_workspace_bytes(int64_t rows, int64_t V, int64_t top_n)
{
    const int64_t parts = parts_of(rows, V);
    return parts == 1 || rows == 0 ? 0 : rows * parts * (8 * top_n + 12);
}

hipError_t launch_token_logprobs(const TokenLogprobs &a, bool z_bf16, hipStream_t stream)
{
    return z_bf16 ? run<true>(a, stream) : run<false>(a, stream);
}

hipError_t launch_token_logprobs_grad(const TokenLogprobs &a, bool z_bf16, hipStream_t stream)
{
    return z_bf16 ? run_grad<true>(a, stream) : run_grad<false>(a, stream);
}

}  // namespace mosaic
