// Distillation of the masked rows' logits from a teacher's top logits.
//
// A row has student logits z_v (v < V) and the teacher's K top logits t_j at vocabulary
// entries c_j.  An entry with c_j outside [0, V) or t_j = -inf is absent.  With the
// temperature T,
//   p_j   = exp((t_j - max t) / T) / sum_j exp((t_j - max t) / T)   over the present entries
//   m     = max_v z_v,   l = log sum_v exp((z_v - m) / T)
//   log q_v = (z_v - m) / T - l
//   loss  = T^2 sum_j p_j (log p_j - log q_{c_j})
//   dloss/dz_v = T (q_v - sum_{j: c_j = v} p_j)
// and a row without a present entry has loss 0 and gradient 0.  Terms with p_j = 0 count
// 0.  The statistics kept for a later gradient are m and l, apart: their sum as one fp32
// number would lose bits of l when m is large.  All arithmetic is fp32; the gradient is
// rounded once, to the logits' type.
//
// The loss reads the logits once, the gradient reads and writes them.  4096 x 126464 bf16, the
// gradient alone: 369 us (5.6 TB/s, what HBM bounds); the loss alone: 167 us (6.2 TB/s).  1229 x
// 126464, loss and gradient: 131 us (4.75 TB/s), where the gradient alone moves the same bytes in
// 110: between a row's reads and its writes its CU goes over the registers twice with little
// under way, and 1229 rows take five turns of 256 CUs for 4.8.
//  * distill_row_kernel: a workgroup per row.  Loss and gradient together keep the row in
//    registers between the two, so the logits are read once.
//  * distill_part_kernel, distill_split_kernel: rows split over several workgroups, for few
//    rows; the first leaves a maximum and a sum of each part, the second joins them.  The
//    second also computes the gradient alone, from the kept statistics.
// The gradient's bulk T g q_v is written first, without regard to the teacher; then the few
// entries that the teacher names are written again with their p taken off.
#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>

#include <algorithm>

#include "launch_ops.h"
#include "row_ops.h"

namespace mosaic {
namespace {

using namespace rows;

constexpr float kLog2e = 1.44269504088896340736f;
constexpr float kInf = __builtin_inff();

__device__ __forceinline__ float fast_exp2(float x) { return __builtin_amdgcn_exp2f(x); }

// Exponents of a set of logits against its maximum m: (z - m) / T in powers of two is taken as
// z * c - k with one rounding, k = m * c rounded, and what k lost, m * c - k, is known
// exactly (`off`) and put right once per sum: a third fewer operations than subtracting
// first.  Where |m| c reaches 2^30 (logits of the type's lowest value, say) what k loses could
// pass exp's range, but then the next lower fp32 number is 64 powers of two away from m: every
// logit counts as m or as nothing, so c is replaced by a power of two with which m * c is exact
// and no product overflows.  An empty set (m = -inf) takes k = 0.
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
                c = __builtin_bit_cast(float, (uint32_t)(294 - e) << 23);   // m * c in [2^40, 2^41)
                k = m * c;
                off = 0.0f;
            }
        }
    }
    __device__ __forceinline__ float exp(float z) const { return fast_exp2(__builtin_fmaf(z, c, -k)); }
};

// Factor that takes a sum of exp((z - from) / T) to one of exp((z - to) / T).
__device__ __forceinline__ float rescale(float from, float to, float c)
{
    return from == -kInf ? 0.0f : fast_exp2((from - to) * c);
}

// Maximum and sum of exp((z - max) / T) of a set of logits; c = log2(e) / T.
struct MaxSum {
    float m = -kInf, s = 0.0f;

    __device__ __forceinline__ void join(float m2, float s2, float c)
    {
        const float mx = fmaxf(m, m2);
        s = s * rescale(m, mx, c) + s2 * rescale(m2, mx, c);
        m = mx;
    }
    __device__ __forceinline__ void join_wave(float c)
    {
#pragma unroll
        for (int o = 32; o >= 1; o >>= 1)
            join(__shfl_xor(m, o, 64), __shfl_xor(s, o, 64), c);
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

template <int N>
__device__ __forceinline__ float sum_of(const float (&z)[N], const Ref &ref)
{
    float e[N];
#pragma unroll
    for (int i = 0; i < N; ++i)
        e[i] = ref.exp(z[i]);
    float a = (e[0] + e[1]) + (e[2] + e[3]);
    if constexpr (N == 8)
        a += (e[4] + e[5]) + (e[6] + e[7]);
    return a;
}

// The same over a stream of logits.
struct RunningMaxSum {
    float m = -kInf, s = 0.0f, c0;
    Ref ref;

    __device__ __forceinline__ RunningMaxSum(float c) : c0(c), ref(-kInf, c) {}
    template <int N>
    __device__ __forceinline__ void add(const float (&z)[N])
    {
        const float mx = max_of(z);
        if (mx > m) {
            s = s * fast_exp2(-ref.off) * rescale(m, mx, c0);
            m = mx;
            ref = Ref(m, c0);
            s *= fast_exp2(ref.off);
        }
        s += sum_of(z, ref);
    }
    __device__ __forceinline__ MaxSum done() const { return MaxSum{m, s * fast_exp2(-ref.off)}; }
};

// What turns a row's logits into gradients: g q_v = scale * exp2(z_v * c - k), with g = T times
// the upstream gradient.
struct RowGrad {
    Ref ref;
    float scale, g;

    // s = exp(l) = sum_v exp((z_v - m) / T)
    __device__ __forceinline__ RowGrad(const Distill &a, int64_t row, const MaxSum &x)
        : ref(x.m, kLog2e / a.temperature), g(a.temperature * (a.grad_loss ? a.grad_loss[row] : 1.0f))
    {
        scale = g * fast_exp2(-ref.off) / x.s;
    }
    template <int N>
    __device__ __forceinline__ void apply(float (&z)[N]) const
    {
#pragma unroll
        for (int i = 0; i < N; ++i)
            z[i] = scale * ref.exp(z[i]);
    }
};

// The teacher's side of one row, in LDS (dynamic: 32 + 3 K + table words).
struct Teacher {
    float *part;        // [2][16] maxima and sums of the waves
    float *p;           // [K], 0 for an absent entry
    float *z;           // [K] the student's logits at the entries
    int32_t *id;        // [K], -1 for an absent entry
    int32_t *table;     // set of the ids: open addressing, a power of two >= 2 K slots
    int slots;
    int32_t *flags;     // present, repeated
    float *entropy;     // sum_j p_j log p_j

    __device__ __forceinline__ Teacher(int32_t *lds, int K, int n_slots)
    {
        part = (float *)lds;
        flags = lds + 32;
        entropy = (float *)(lds + 34);
        p = (float *)(lds + 36);
        z = p + K;
        id = (int32_t *)(z + K);
        table = id + K;
        slots = n_slots;
    }
};

// Slots of the id set, and the LDS bytes of a Teacher.
int table_slots(int K)
{
    int n = 64;
    while (n < 2 * K)
        n *= 2;
    return n;
}
size_t teacher_bytes(int K) { return (size_t)(36 + 3 * K + table_slots(K)) * 4; }

// Fills t from the row's K entries; run by one wave, visible to the others after a barrier.
// The student's logits at the entries come from z_at (in the order of the entries) where it
// is given, else from the logits of the row, those with lo <= c_j < hi only.
template <bool BF16>
__device__ __forceinline__ void load_teacher(const Distill &a, int64_t row, const Teacher &t, const float *z_at, int lo,
                                             int hi)
{
    const int lane = threadIdx.x & 63;
    const float c = kLog2e / a.temperature;
    if (a.grad)   // only the gradient asks for repeated entries
        for (int i = lane; i < t.slots; i += 64)
            t.table[i] = -1;
    float mx = -kInf;
    bool any = false;
    for (int j = lane; j < a.K; j += 64) {
        const int32_t id = a.ids[row * a.K + j];
        const float x = load1(a.top, row * a.K + j, a.top_bf16);
        const bool here = id >= 0 && id < a.V && x != -kInf;
        float z = 0.0f;
        if (z_at)
            z = z_at[j];
        else if (here && id >= lo && id < hi)
            z = load1(a.Z, row * a.ldz + id, BF16);
        t.id[j] = here ? id : -1;
        t.p[j] = x;
        t.z[j] = z;
        mx = here ? fmaxf(mx, x) : mx;
        any = any || here;
    }
    mx = wave_reduce(mx, MaxOp{});
    const bool present = __any(any);
    float sum = 0.0f;
    for (int j = lane; j < a.K; j += 64) {
        const float e = t.id[j] >= 0 ? fast_exp2((t.p[j] - mx) * c) : 0.0f;
        t.p[j] = e;
        sum += e;
    }
    sum = wave_reduce(sum, AddOp{});
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "workgroup");   // the cleared table, before other lanes' entries
    __builtin_amdgcn_wave_barrier();
    float h = 0.0f;
    bool repeated = false;
    for (int j = lane; j < a.K; j += 64) {
        const float p = present ? t.p[j] / sum : 0.0f;
        t.p[j] = p;
        h += p != 0.0f ? p * logf(p) : 0.0f;
        const int32_t id = t.id[j];
        if (id < 0 || !a.grad)
            continue;
        // at most K of >= 2 K slots are taken, so a free one is found
        int s = (int)(((uint32_t)id * 2654435761u) >> 16) & (t.slots - 1);
        for (;;) {
            const int32_t old = atomicCAS(&t.table[s], -1, id);
            if (old == -1 || old == id) {
                repeated = repeated || old == id;
                break;
            }
            s = (s + 1) & (t.slots - 1);
        }
    }
    h = wave_reduce(h, AddOp{});
    repeated = __any(repeated);
    if (lane == 0) {
        t.flags[0] = present;
        t.flags[1] = repeated;
        *t.entropy = h;
    }
}

// The row's loss from its statistics, in every lane of the calling wave.
__device__ __forceinline__ float row_loss(const Distill &a, const Teacher &t, float m, float l)
{
    const float T = a.temperature, inv = 1.0f / T;
    float x = 0.0f;
    for (int j = threadIdx.x & 63; j < a.K; j += 64)
        x += t.p[j] != 0.0f ? t.p[j] * ((t.z[j] - m) * inv - l) : 0.0f;
    const float loss = T * T * (*t.entropy - wave_reduce(x, AddOp{}));
    if (loss != kInf)
        return loss;
    // The teacher has mass where z is -inf, or so low (a mask of the type's lowest value) that
    // z - m or its quotient by T passed fp32's range.  T times the difference need not, so it is
    // taken in halves, with T beside p; what is infinite stays so.
    x = 0.0f;
    for (int j = threadIdx.x & 63; j < a.K; j += 64)
        x += t.p[j] != 0.0f ? t.p[j] * T * (0.5f * m - 0.5f * t.z[j]) : 0.0f;
    return T * T * (*t.entropy + l) + 2.0f * wave_reduce(x, AddOp{});
}

// The gradient of a row without teacher entries.
template <bool BF16, int NT>
__device__ __forceinline__ void zero_grad(const Distill &a, int64_t row, int lo, int hi)
{
    constexpr int N = kChunk<BF16>;
    for (int v = lo + threadIdx.x * N; v < hi; v += NT * N) {
        const float z[N] = {};
        store_upto<BF16>(a.grad, row * a.ldg + v, z, hi - v);
    }
}

// Writes the gradient at the teacher's entries with lo <= c_j < hi again, with p taken off; the
// bulk has been written before the last barrier.
template <bool BF16, int NT>
__device__ __forceinline__ void fix_entries(const Distill &a, const Teacher &t, int64_t row, int lo, int hi,
                                            const RowGrad &f)
{
    const bool repeated = t.flags[1];
    for (int j = threadIdx.x; j < a.K; j += NT) {
        const int32_t id = t.id[j];
        if (id < lo || id >= hi)   // absent ones are -1
            continue;
        float p = t.p[j];
        if (repeated) {            // an entry named again is written once, by the first, with all shares
            bool first = true;
            p = 0.0f;
            for (int i = 0; i < a.K; ++i) {
                if (t.id[i] == id) {
                    first = first && i >= j;
                    p += t.p[i];
                }
            }
            if (!first)
                continue;
        }
        store1<BF16>(a.grad, row * a.ldg + id, f.scale * f.ref.exp(t.z[j]) - f.g * p);
    }
}

// Maximum and sum over chunks held in registers, the first `live` of R (the others lie behind
// the row's end for every thread).  The fences keep the compiler from unpacking many chunks at
// once, for which there are no registers.
template <bool BF16, int R>
__device__ __forceinline__ float held_max(Raw<BF16> (&r)[R], int live, float mx)
{
#pragma unroll
    for (int i = 0; i < R; ++i) {
        if (i < live) {
            float z[kChunk<BF16>];
            r[i].opaque();
            r[i].get(z);
            mx = fmaxf(mx, max_of(z));
        }
        if (i % 2)
            __builtin_amdgcn_sched_barrier(0);
    }
    return mx;
}

template <bool BF16, int R>
__device__ __forceinline__ float held_sum(Raw<BF16> (&r)[R], int live, const Ref &ref)
{
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < R; ++i) {
        if (i < live) {
            float z[kChunk<BF16>];
            r[i].opaque();
            r[i].get(z);
            s += sum_of(z, ref);
        }
        if (i % 2)
            __builtin_amdgcn_sched_barrier(0);
    }
    return s;
}

// Chunks of N logits of [lo, hi), lo a multiple of N: chunk i of this thread's is
// lo / N + threadIdx.x + i * NT.  UN loads are issued before their values are used.
template <bool BF16, int NT, bool STREAM, typename F>
__device__ __forceinline__ void for_chunks(const Distill &a, int64_t row, int lo, int hi, F f)
{
    constexpr int UN = 4, N = kChunk<BF16>;
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

// Maximum and sum of this thread's logits of [lo, hi), chunked as by for_chunks.  RUNS: runs of 2^9
// chunks of a thread are added one after another, then the runs: 2^13 chunks in one sum, whose
// additions of equal terms all round the same way, took l off by 1227 half steps (a row of 2^30
// bf16 logits).  Without it for rows of one run, which these steps would slow down (20 x 152064
// bf16: 13.9 against 13.6 us).
template <int NT, int N>
constexpr int kRun = 512 * NT * N;

template <bool BF16, int NT, bool STREAM, bool RUNS>
__device__ __forceinline__ MaxSum max_sum_of(const Distill &a, int64_t row, int lo, int hi, float c)
{
    auto run_of = [&](int from, int to) __attribute__((always_inline)) {
        RunningMaxSum run(c);
        for_chunks<BF16, NT, STREAM>(a, row, from, to, [&](auto &z, int, int) { run.add(z); });
        return run.done();
    };
    if constexpr (!RUNS)
        return run_of(lo, hi);
    constexpr int RUN = kRun<NT, kChunk<BF16>>;
    MaxSum x;
    for (int v = lo; v < hi; v += RUN) {
        const MaxSum y = run_of(v, min(v + RUN, hi));
        x.join(y.m, y.s, c);
    }
    return x;
}

// Barrier between the gradient's bulk and the entries written again: every wave's stores have
// been acknowledged before any wave passes it.
__device__ __forceinline__ void barrier_after_stores()
{
    __builtin_amdgcn_s_waitcnt(0x0f70);   // vmcnt(0)
    __syncthreads();
}

// Gradient bulk of the part [lo, hi) of a row, then the teacher's entries in it.
template <bool BF16, int NT, bool STREAM>
__device__ __forceinline__ void part_grad(const Distill &a, const Teacher &t, int64_t row, int lo, int hi,
                                          const MaxSum &x)
{
    const RowGrad f(a, row, x);
    if (t.flags[0])
        for_chunks<BF16, NT, STREAM>(a, row, lo, hi, [&](auto &z, int v, int n) {
            f.apply(z);
            store_upto<BF16, STREAM>(a.grad, row * a.ldg + v, z, n);
        });
    else
        zero_grad<BF16, NT>(a, row, lo, hi);
    barrier_after_stores();
    fix_entries<BF16, NT>(a, t, row, lo, hi, f);
}

// (m, s) of NW waves from the teacher's part array.
template <int NW>
__device__ __forceinline__ MaxSum join_parts(const Teacher &t, float c)
{
    MaxSum x;
#pragma unroll
    for (int w = 0; w < NW; ++w)
        x.m = fmaxf(x.m, t.part[w]);
#pragma unroll
    for (int w = 0; w < NW; ++w)
        x.s += t.part[16 + w] * rescale(t.part[w], x.m, c);
    return x;
}

// Joins the (m, s) of a workgroup's waves, the result in every thread.  Its barrier also
// publishes the teacher.
template <int NT>
__device__ __forceinline__ MaxSum join_block(const MaxSum &x, const Teacher &t, float c)
{
    if constexpr (NT == 64) {
        __syncthreads();
        return x;
    }
    if ((threadIdx.x & 63) == 0) {
        t.part[threadIdx.x >> 6] = x.m;
        t.part[16 + (threadIdx.x >> 6)] = x.s;
    }
    __syncthreads();
    return join_parts<NT / 64>(t, c);
}

// One row per workgroup.  R > 0: the row stays in registers, R chunks of N logits per
// thread (V <= N NT R), and is read once; R = 0: a gradient reads it again (RUNS: as above).
template <bool BF16, int NT, int R, bool RUNS = false>
__global__ __launch_bounds__(NT) void distill_row_kernel(const Distill a, int slots)
{
    extern __shared__ int32_t lds[];
    const Teacher t(lds, a.K, slots);
    const float c = kLog2e / a.temperature;
    const int64_t n = row_count(a.count, a.rows);
    constexpr int N = kChunk<BF16>;
    const int V = a.V, full = V / N * N;
    const int live = (full + NT * N - 1) / (NT * N);
    uint32_t d0 = threadIdx.x * N;   // a chunk's place: a uniform pointer and this offset
    constexpr int64_t ES = BF16 ? 2 : 4;
    for (int64_t row = blockIdx.x; row < n; row += gridDim.x) {
        asm volatile("" : "+v"(d0));   // or the places of all chunks stay in registers between rows
        MaxSum x;
        Raw<BF16> r[R > 0 ? R : 1], rest;   // whole chunks, and the last, shorter one
        const bool has_rest = full < V && threadIdx.x == NT - 1;
        if (threadIdx.x < 64)
            load_teacher<BF16>(a, row, t, nullptr, 0, V);
        if constexpr (R > 0) {
#pragma unroll
            for (int i = 0; i < R; ++i) {
                r[i].fill(-kInf);
                if (i * NT * N + (int)d0 < full)
                    r[i].load((const char *)a.Z + (row * a.ldz + i * NT * N) * ES, d0);
            }
            rest.fill(-kInf);
            if (has_rest)
                rest.load_part(a.Z, row * a.ldz + full, V - full);
            float z[kChunk<BF16>];
            rest.get(z);
            x.m = wave_reduce(held_max(r, live, has_rest ? max_of(z) : -kInf), MaxOp{});
            const Ref ref(x.m, c);
            x.s = wave_reduce(held_sum(r, live, ref) + (has_rest ? sum_of(z, ref) : 0.0f), AddOp{}) * fast_exp2(-ref.off);
        } else {
            if (a.grad)   // it will be read again
                x = max_sum_of<BF16, NT, false, RUNS>(a, row, 0, V, c);
            else
                x = max_sum_of<BF16, NT, true, RUNS>(a, row, 0, V, c);
            x.join_wave(c);
        }
        x = join_block<NT>(x, t, c);
        const float m = x.m, l = logf(x.s);
        const bool present = t.flags[0];
        if (threadIdx.x < 64) {
            const float loss = row_loss(a, t, m, l);
            if (threadIdx.x == 0) {
                a.loss[row] = present ? loss : 0.0f;
                a.stats[2 * row] = m;
                a.stats[2 * row + 1] = l;
            }
        }
        if (a.grad) {
            if constexpr (R > 0) {
                const RowGrad f(a, row, x);
                if (!present) {
                    zero_grad<BF16, NT>(a, row, 0, V);
                } else {
#pragma unroll
                    for (int i = 0; i < R; ++i) {
                        if (i * NT * N + (int)d0 < full) {
                            float z[kChunk<BF16>];
                            r[i].opaque();
                            r[i].get(z);
                            f.apply(z);
                            store<BF16>((char *)a.grad + (row * a.ldg + i * NT * N) * ES, d0, z);
                        }
                        __builtin_amdgcn_sched_barrier(0);
                    }
                    if (has_rest) {
                        float z[kChunk<BF16>];
                        rest.get(z);
                        f.apply(z);
                        store_upto<BF16>(a.grad, row * a.ldg + full, z, V - full);
                    }
                }
                barrier_after_stores();
                fix_entries<BF16, NT>(a, t, row, 0, V, f);
            } else {
                // the row's second and last read, out of the Infinity Cache: with the streaming
                // policy, reads and stores leave it to the rows under way
                part_grad<BF16, NT, true>(a, t, row, 0, V, x);
            }
        }
        __syncthreads();   // the teacher's arrays are refilled for the next row
    }
}

// Loss and gradient of long rows.  A workgroup of 16 waves has a CU to itself and walks its
// rows: 15 waves hold the row in registers, R chunks of N logits per thread (V <= 960 N R),
// and wave 0 takes the logits behind the last whole chunk, prepares the next row's teacher,
// writes the loss and mends the entries of the row before.  As soon as a chunk's gradient is
// stored, its registers take the next row's logits, so that reads and writes run side by side.
// The one barrier of a row publishes the waves' sums and the teacher, and finds the stores of
// the row before complete, behind the loads that it waits for anyway.
// STREAM: streaming cache policy.
template <bool BF16, int R, bool STREAM>
__global__ __launch_bounds__(1024) void distill_stream_kernel(const Distill a, int slots, int teacher_words)
{
    extern __shared__ int32_t lds[];
    constexpr int ND = 960, N = kChunk<BF16>;
    const Teacher t0(lds, a.K, slots), t1(lds + teacher_words, a.K, slots);
    const float c = kLog2e / a.temperature;
    const int64_t n = row_count(a.count, a.rows);
    const int V = a.V, full = V / N * N;
    int64_t row = blockIdx.x;
    if (row >= n)
        return;
    // (m, s) of a wave for the join
    auto leave = [&](const Teacher &t, float m, float s) __attribute__((always_inline)) {
        if ((threadIdx.x & 63) == 0) {
            t.part[threadIdx.x >> 6] = m;
            t.part[16 + (threadIdx.x >> 6)] = s;
        }
    };
    if (threadIdx.x < 64) {
        const int v = full + threadIdx.x;   // this lane's logit behind the last whole chunk
        float z = -kInf;
        auto prepare = [&](int64_t r, const Teacher &t) __attribute__((always_inline)) {
            if (v < V)
                z = load1(a.Z, r * a.ldz + v, BF16);
            load_teacher<BF16>(a, r, t, nullptr, 0, V);
            const float m = wave_reduce(z, MaxOp{});
            const Ref ref(m, c);
            leave(t, m, wave_reduce(ref.exp(z), AddOp{}) * fast_exp2(-ref.off));
        };
        prepare(row, t0);
        __syncthreads();
        MaxSum before;
        for (bool odd = false, first = true;; odd = !odd, first = false) {
            const Teacher &t = odd ? t1 : t0, &other = odd ? t0 : t1;
            const MaxSum x = join_parts<16>(t, c);
            const float l = logf(x.s), loss = row_loss(a, t, x.m, l);
            if (threadIdx.x == 0) {
                a.loss[row] = t.flags[0] ? loss : 0.0f;
                a.stats[2 * row] = x.m;
                a.stats[2 * row + 1] = l;
            }
            const RowGrad f(a, row, x);
            if (v < V)
                store1<BF16>(a.grad, row * a.ldg + v, t.flags[0] ? f.scale * f.ref.exp(z) : 0.0f);
            if (!first)
                fix_entries<BF16, 64>(a, other, row - gridDim.x, 0, V, RowGrad(a, row - gridDim.x, before));
            before = x;
            const int64_t next = row + gridDim.x;
            if (next < n)
                prepare(next, other);
            barrier_after_stores();
            if (next >= n) {
                fix_entries<BF16, 64>(a, t, row, 0, V, f);
                return;
            }
            row = next;
        }
    }
    // Chunk i's place: a uniform pointer and the lane's offset.  The offset is hidden from the
    // compiler once per row, or it keeps the sums of all chunks in registers between rows.
    const int live = (full + ND * N - 1) / (ND * N);
    uint32_t d0 = (threadIdx.x - 64) * N;
    Raw<BF16> r[R];
    constexpr int64_t ES = BF16 ? 2 : 4;
    auto fetch = [&](int i, int64_t from) __attribute__((always_inline)) {
        if (i * ND * N + (int)d0 < full)
            r[i].template load<STREAM>((const char *)a.Z + (from * a.ldz + i * ND * N) * ES, d0);
    };
#pragma unroll
    for (int i = 0; i < R; ++i) {
        r[i].fill(-kInf);
        fetch(i, row);
    }
    for (bool odd = false;; odd = !odd) {
        const Teacher &t = odd ? t1 : t0;
        asm volatile("" : "+v"(d0));
        const float m = wave_reduce(held_max(r, live, -kInf), MaxOp{});
        const Ref ref(m, c);
        leave(t, m, wave_reduce(held_sum(r, live, ref), AddOp{}) * fast_exp2(-ref.off));
        barrier_after_stores();   // of the row before, which wave 0 mends after it
        const RowGrad f(a, row, join_parts<16>(t, c));
        const int64_t next = row + gridDim.x;
        const bool present = t.flags[0];
#pragma unroll
        for (int i = 0; i < R; ++i) {
            if (i * ND * N + (int)d0 < full) {
                float z[kChunk<BF16>] = {};
                if (present) {
                    r[i].opaque();
                    r[i].get(z);
                    f.apply(z);
                }
                store<BF16, STREAM>((char *)a.grad + (row * a.ldg + i * ND * N) * ES, d0, z);
                if (next < n)
                    fetch(i, next);
            }
            __builtin_amdgcn_sched_barrier(0);
        }
        if (next >= n) {
            barrier_after_stores();
            return;
        }
        row = next;
    }
}

// Part s of a row's `parts`: logits [lo, hi), multiples of eight but for the last.
__device__ __forceinline__ void part_range(int V, int parts, int s, int &lo, int &hi)
{
    const int chunks = (V + 7) / 8, each = (chunks + parts - 1) / parts;
    lo = min(s * each, chunks) * 8;
    hi = min(min((s + 1) * each, chunks) * 8, V);
    lo = min(lo, hi);
}

constexpr int kPartThreads = 256;

// (maximum, sum) of each part of each row into partials[row][part][2], and the student's
// logits at the teacher's entries into z_at[row][K] (the gradient may overwrite them).
template <bool BF16, bool RUNS>
__global__ __launch_bounds__(kPartThreads) void distill_part_kernel(const Distill a, int parts,
                                                                     float *__restrict__ z_at)
{
    __shared__ float red[8];
    const float c = kLog2e / a.temperature;
    const int64_t row = blockIdx.x / parts;
    const int s = blockIdx.x % parts;
    if (row >= row_count(a.count, a.rows))
        return;
    int lo, hi;
    part_range(a.V, parts, s, lo, hi);
    MaxSum x = max_sum_of<BF16, kPartThreads, false, RUNS>(a, row, lo, hi, c);
    x.join_wave(c);
    if ((threadIdx.x & 63) == 0) {
        red[threadIdx.x >> 6] = x.m;
        red[4 + (threadIdx.x >> 6)] = x.s;
    }
    __syncthreads();
    if (threadIdx.x == 0) {
        for (int w = 1; w < 4; ++w)
            x.join(red[w], red[4 + w], c);
        a.partials[2 * blockIdx.x] = x.m;
        a.partials[2 * blockIdx.x + 1] = x.s;
    }
    if (s == parts - 1)
        for (int j = threadIdx.x; j < a.K; j += kPartThreads) {
            const int32_t id = a.ids[row * a.K + j];
            z_at[row * a.K + j] = id >= 0 && id < a.V ? load1(a.Z, row * a.ldz + id, BF16) : 0.0f;
        }
}

// Gradient of part blockIdx.x % cuts of a row.  parts > 0: the statistics are joined from the
// row's partials, and the workgroup of the first part writes them and the loss; parts = 0:
// they are given.
template <bool BF16, int NT, bool STREAM>
__global__ __launch_bounds__(NT) void distill_split_kernel(const Distill a, int slots, int parts, int cuts,
                                                                      const float *__restrict__ z_at)
{
    extern __shared__ int32_t lds[];
    const Teacher t(lds, a.K, slots);
    const float c = kLog2e / a.temperature;
    const int64_t n = row_count(a.count, a.rows);
    for (int64_t b = blockIdx.x; b < n * cuts; b += gridDim.x) {
        const int64_t row = b / cuts;
        const int s = (int)(b % cuts);
        int lo, hi;
        part_range(a.V, cuts, s, lo, hi);
        if (threadIdx.x < 64)
            load_teacher<BF16>(a, row, t, z_at ? z_at + row * a.K : nullptr, z_at ? 0 : lo, z_at ? a.V : hi);
        MaxSum x;
        if (parts > 0) {
            const int i = threadIdx.x & 63;   // parts <= 64
            if (i < parts)
                x = MaxSum{a.partials[2 * (row * parts + i)], a.partials[2 * (row * parts + i) + 1]};
            x.join_wave(c);
        } else {
            x = MaxSum{a.stats[2 * row], expf(a.stats[2 * row + 1])};
        }
        __syncthreads();   // the teacher is there
        if (parts > 0 && s == 0 && threadIdx.x < 64) {
            const float l = logf(x.s), loss = row_loss(a, t, x.m, l);
            if (threadIdx.x == 0) {
                a.loss[row] = t.flags[0] ? loss : 0.0f;
                a.stats[2 * row] = x.m;
                a.stats[2 * row + 1] = l;
            }
        }
        if (a.grad)
            part_grad<BF16, NT, STREAM>(a, t, row, lo, hi, x);
        __syncthreads();   // the teacher's arrays are refilled for the next row
    }
}

// Parts of a row in the split form: about 2048 workgroups, of 4096 logits at least each.
int parts_of(int64_t rows, int64_t V)
{
    return (int)std::max<int64_t>(1, std::min<int64_t>({64, 2048 / std::max<int64_t>(rows, 1), V / 4096}));
}

// Few rows of many logits go over several workgroups each: for the gradient from 16384 logits
// on (129 x 126464, loss and gradient: as fast either way), for the loss alone, two launches
// against one, where a row passes 400 KB
// (20 x 524288 bf16: 16 against 39 us; 20 x 152064: 16.0 against 15.7 us, 20 x 100000 fp32: 15.4
// against 14.0; 256 x 262144: 34 against 29).  These are calls with their launches.  Replayed in a
// graph, where a second launch costs less, two would be faster for fewer rows or shorter ones too:
// 20 x 152064: 8.8 against 13.6 us, 64 x 126464: 11.5 against 13.4, 20 x 32000: 8.2 against 9.7;
// but 128 x 126464: 14.5 against 14.1.  A captured call takes the eager call's form all the same,
// so that both give the same bits.
bool is_split(int64_t rows, int64_t V, bool bf16, bool grad)
{
    return rows <= 128 && (grad ? V >= 16384 : V * (bf16 ? 2 : 4) > 409600);
}

// Logits that cannot stay in the 256 MB Infinity Cache are read and written with the streaming
// cache policy: 4096 x 126464 bf16, loss and gradient: 435 against 463 us, the gradient alone
// 410 against 468 us; but 512 x 126464: 54 against 46 us for the gradient.  The loss alone reads
// each logit once and always takes it (4096 x 126464: 169 against 189 us, 512: 33 against 35).
template <bool BF16>
bool is_large(const Distill &a)
{
    return a.rows * a.V >= ((int64_t)256 << 20) / (BF16 ? 2 : 4);
}

// Chunks per thread of the stream form: 20 fill its registers.
template <bool BF16>
constexpr int kStreamChunks[3] = {BF16 ? 13 : 10, BF16 ? 17 : 15, 20};

// Which form a row takes, by its length (bf16; fp32 chunks take twice the registers):
//  * up to 2048 logits: a wave per row.  Up to 8192: a wave per row where there are rows enough
//    for several waves per SIMD, else four waves (8000 x 8000, loss and gradient: 56 against
//    60 us; the loss alone 31 against 46 us).
//  * the loss alone of longer rows: 4 waves per row, 8 up to three rows per CU, 16 up to one
//    (126464 logits: 256 rows 16 us with 16 waves, 18 with 8, 27 with 4; 512 rows 30, 26, 31; 850
//    rows 53, 44, 42).
//  * up to 65536: 4 or 8 waves per row, several rows on a CU.  4000 x 20000: 72 us with 4 waves,
//    88 us with 8, 105 us through the stream form; 2000 x 50000: 90 us with 8, 97 us there.
//  * longer: the stream form, a row at a time on each CU, up to what its registers hold, 153600
//    bf16 logits (4096 x 126464: 419 us; without the reads of the next row beside the writes of
//    this one 475 us).
//  * longer still: the row is read twice (2000 x 200000: 338 us, 375 us without the streaming
//    policy in the second pass).
template <bool BF16>
hipError_t run(const Distill &a, hipStream_t stream)
{
    const int slots = table_slots(a.K);
    const size_t lds = teacher_bytes(a.K);
    if (is_split(a.rows, a.V, BF16, a.grad)) {
        const int parts = parts_of(a.rows, a.V), cuts = a.grad ? parts : 1;
        float *z_at = a.partials + 2 * a.rows * parts;
        const bool runs = a.V / parts > kRun<kPartThreads, kChunk<BF16>>;
        hipLaunchKernelGGL((runs ? distill_part_kernel<BF16, true> : distill_part_kernel<BF16, false>),
                           dim3((unsigned)(a.rows * parts)), dim3(kPartThreads), 0, stream, a, parts, z_at);
        hipLaunchKernelGGL((distill_split_kernel<BF16, 256, false>), dim3((unsigned)(a.rows * cuts)), dim3(256), lds,
                           stream, a, slots, parts, cuts, z_at);
        return hipGetLastError();
    }
    auto rows = [&](auto kernel, int threads) {
        hipLaunchKernelGGL(kernel, dim3((unsigned)std::min<int64_t>(a.rows, 1 << 20)), dim3(threads), lds, stream, a,
                           slots);
    };
    auto in_runs = [&](auto kernel, auto kernel_runs, int threads) {
        rows(a.V > kRun<1, kChunk<BF16>> * threads ? kernel_runs : kernel, threads);
    };
    int dev = 0, cus = 256;
    if (hipGetDevice(&dev) == hipSuccess)
        (void)hipDeviceGetAttribute(&cus, hipDeviceAttributeMultiprocessorCount, dev);
    auto rows_per_cu = [&](auto kernel, auto kernel_large) {
        const dim3 grid((unsigned)std::min<int64_t>(a.rows, cus));
        if (is_large<BF16>(a))
            hipLaunchKernelGGL(kernel_large, grid, dim3(1024), 2 * lds, stream, a, slots, (int)(lds / 4));
        else
            hipLaunchKernelGGL(kernel, grid, dim3(1024), 2 * lds, stream, a, slots, (int)(lds / 4));
    };
    const bool many = a.rows >= 2048;
    constexpr int N = kChunk<BF16>, B = 8 / N;   // B: chunks of the type that eight logits take
    if (a.V <= 2048)
        rows(distill_row_kernel<BF16, 64, 4 * B>, 64);
    else if (!a.grad && many && a.V <= 16384)
        rows(distill_row_kernel<BF16, 64, 0>, 64);
    else if (!a.grad && (a.rows > 3 * cus || a.V <= 32768))
        in_runs(distill_row_kernel<BF16, 256, 0>, distill_row_kernel<BF16, 256, 0, true>, 256);
    else if (!a.grad && a.rows > cus)
        in_runs(distill_row_kernel<BF16, 512, 0>, distill_row_kernel<BF16, 512, 0, true>, 512);
    else if (!a.grad)
        in_runs(distill_row_kernel<BF16, 1024, 0>, distill_row_kernel<BF16, 1024, 0, true>, 1024);
    else if (BF16 && many && a.V <= 8192)
        rows(distill_row_kernel<BF16, 64, BF16 ? 16 : 4 * B>, 64);
    else if (a.V <= 8192)
        rows(distill_row_kernel<BF16, 256, 4 * B>, 256);
    else if (a.V <= 16384)
        rows(distill_row_kernel<BF16, 256, 8 * B>, 256);
    else if (BF16 && a.V <= 32768)
        rows(distill_row_kernel<BF16, 256, 16>, 256);
    else if (a.V <= (BF16 ? 65536 : 32768))
        rows(distill_row_kernel<BF16, 512, 16>, 512);
    else if (a.V <= 960 * N * kStreamChunks<BF16>[0])
        rows_per_cu(distill_stream_kernel<BF16, kStreamChunks<BF16>[0], false>,
                    distill_stream_kernel<BF16, kStreamChunks<BF16>[0], true>);
    else if (a.V <= 960 * N * kStreamChunks<BF16>[1])
        rows_per_cu(distill_stream_kernel<BF16, kStreamChunks<BF16>[1], false>,
                    distill_stream_kernel<BF16, kStreamChunks<BF16>[1], true>);
    else if (a.V <= 960 * N * kStreamChunks<BF16>[2])
        rows_per_cu(distill_stream_kernel<BF16, kStreamChunks<BF16>[2], false>,
                    distill_stream_kernel<BF16, kStreamChunks<BF16>[2], true>);
    else
        in_runs(distill_row_kernel<BF16, 1024, 0>, distill_row_kernel<BF16, 1024, 0, true>, 1024);
    return hipGetLastError();
}

// Parts of a row for the gradient alone: 12288 to 32768 logits each, so that the workgroups under
// way cover a compact stretch of memory (4096 x 126464 bf16: 367 us in 4 parts per row, 410 us
// in one, 423 us in 16, where the teacher is prepared too often).  Of these numbers of parts
// the one that best fills the last round of workgroups, counted as 8 on a CU, and the last turn of
// their loops, 4 chunks per thread (1229 rows: 109 us in 8 parts, 117 us in 4, 121 us in 5).  The
// kernel's registers let 7 on a CU.  Neither count is the better model: with 7 in the rule 4096 x
// 126464 takes 349 us instead of 375 and 1000 rows 100 instead of 106, but 1229 rows 119 instead of
// 111 and 1600 rows 151 instead of 140; with the kernel held to 8, 0 to 3% slower (300 rows: 9%).
int cuts_of(int64_t rows, int64_t V, int chunk)
{
    int dev = 0, cus = 256;
    if (hipGetDevice(&dev) == hipSuccess)
        (void)hipDeviceGetAttribute(&cus, hipDeviceAttributeMultiprocessorCount, dev);
    const double slots = 8.0 * cus, chunks = (double)V / (chunk * 256);
    int best = 1;
    double most = 0.0;
    const int64_t lo = std::max<int64_t>(1, (V + 32767) / 32768), hi = std::min<int64_t>(std::max(lo, V / 12288), lo + 63);
    for (int64_t n = lo; n <= hi; ++n) {
        const double groups = (double)rows * n / slots, turns = chunks / n / 4.0;
        const double full = groups / ceil(groups) * (turns / ceil(turns)) - 0.005 * n;
        if (full > most) {
            most = full;
            best = (int)n;
        }
    }
    return std::max((int)lo, best);
}

template <bool BF16>
hipError_t run_grad(const Distill &a, hipStream_t stream)
{
    const int cuts = std::max(parts_of(a.rows, a.V), cuts_of(a.rows, a.V, kChunk<BF16>));
    auto go = [&](auto kernel, int threads) {
        hipLaunchKernelGGL(kernel, dim3((unsigned)std::min<int64_t>(a.rows * cuts, 1 << 20)), dim3(threads),
                           teacher_bytes(a.K), stream, a, table_slots(a.K), 0, cuts, (const float *)nullptr);
    };
    if (a.V <= 4096 && a.rows >= 2048)   // a wave per row: enough rows, of few chunks each
        go(distill_split_kernel<BF16, 64, false>, 64);
    else if (is_large<BF16>(a))
        go(distill_split_kernel<BF16, 256, true>, 256);
    else
        go(distill_split_kernel<BF16, 256, false>, 256);
    return hipGetLastError();
}

}  // namespace

int64_t distill_workspace_bytes(int64_t rows, int64_t V, int64_t K)
{
    // whichever type and direction the call has: what is split as bf16 is split as fp32
    const bool split = is_split(rows, V, false, false) || is_split(rows, V, false, true);
    return split ? 4 * rows * (2 * parts_of(rows, V) + K) : 0;
}

hipError_t launch_distill(const Distill &a, bool z_bf16, hipStream_t stream)
{
    return z_bf16 ? run<true>(a, stream) : run<false>(a, stream);
}

hipError_t launch_distill_grad(const Distill &a, bool z_bf16, hipStream_t stream)
{
    return z_bf16 ? run_grad<true>(a, stream) : run_grad<false>(a, stream);
}

}  // namespace mosaic
