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
// HBM bounds both directions: the loss reads the logits once, the gradient reads and writes
// them.
//  * distill_row_kernel: a workgroup per row.  Loss and gradient together keep the row in
//    registers between the two, so the logits are read once.
//  * distill_part_kernel, distill_split_kernel: rows split over several workgroups, for few
//    rows; the first leaves a maximum and a sum of each part, the second joins them.  The
//    second also computes the gradient alone, from the kept statistics.
// The gradient's bulk T g q_v is written first, without regard to the teacher; then the few
// entries that the teacher names are written again with their p taken off.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "launch.h"
#include "row_ops.h"

namespace mosaic {
namespace {

using namespace rows;

constexpr float kLog2e = 1.44269504088896340736f;
constexpr float kInf = __builtin_inff();

__device__ __forceinline__ float fast_exp2(float x) { return __builtin_amdgcn_exp2f(x); }

// -inf stands for nothing seen yet, and (-inf) - (-inf) would be NaN
__device__ __forceinline__ float ref_of(float m) { return m == -kInf ? 0.0f : m; }

// Running maximum and sum of exp((z - max) / T) of a set of logits; c = log2(e) / T.
struct MaxSum {
    float m = -kInf, s = 0.0f;

    __device__ __forceinline__ void add(const float (&z)[8], float c)
    {
        float mx = fmaxf(fmaxf(fmaxf(z[0], z[1]), fmaxf(z[2], z[3])), fmaxf(fmaxf(z[4], z[5]), fmaxf(z[6], z[7])));
        if (mx > m) {
            s *= fast_exp2((m - mx) * c);
            m = mx;
        }
        const float r = ref_of(m);
        float e[8];
#pragma unroll
        for (int i = 0; i < 8; ++i)
            e[i] = fast_exp2((z[i] - r) * c);
        s += ((e[0] + e[1]) + (e[2] + e[3])) + ((e[4] + e[5]) + (e[6] + e[7]));
    }
    __device__ __forceinline__ void join(float m2, float s2, float c)
    {
        const float mx = fmaxf(m, m2), r = ref_of(mx);
        s = s * fast_exp2((m - r) * c) + s2 * fast_exp2((m2 - r) * c);
        m = mx;
    }
    __device__ __forceinline__ void join_wave(float c)
    {
#pragma unroll
        for (int o = 32; o >= 1; o >>= 1)
            join(__shfl_xor(m, o, 64), __shfl_xor(s, o, 64), c);
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
    for (int i = lane; i < t.slots; i += 64)
        t.table[i] = -1;
    float mx = -kInf;
    bool any = false;
    for (int j = lane; j < a.K; j += 64) {
        const int32_t id = a.ids[row * a.K + j];
        const float x = load1(a.top, row * a.K + j, a.top_bf16);
        const bool here = id >= 0 && id < a.V && x != -kInf;
        float z = 0.0f;
        if (here && id >= lo && id < hi)
            z = z_at ? z_at[j] : load1(a.Z, row * a.ldz + id, BF16);
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
        if (id < 0)
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
    return T * T * (*t.entropy - wave_reduce(x, AddOp{}));
}

// Writes the gradient at the teacher's entries with lo <= c_j < hi again, with p taken off; the
// bulk has been written before the last barrier.  g: T times the row's upstream gradient.
template <bool BF16, int NT>
__device__ __forceinline__ void fix_entries(const Distill &a, const Teacher &t, int64_t row, int lo, int hi, float g,
                                            float m, float l)
{
    const float c = kLog2e / a.temperature, l2 = l * kLog2e;
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
        store1<BF16>(a.grad, row * a.ldg + id, g * (fast_exp2((t.z[j] - m) * c - l2) - p));
    }
}

// eight logits to eight gradients T g q_v (0 in a row without teacher entries)
__device__ __forceinline__ void grad8(float (&z)[8], float g, float m, float c, float l2, bool present = true)
{
#pragma unroll
    for (int i = 0; i < 8; ++i)
        z[i] = present ? g * fast_exp2((z[i] - m) * c - l2) : 0.0f;
}

// running maxima and sums over chunks held in registers
template <bool BF16>
__device__ __forceinline__ void max8(Raw8<BF16> &r, float (&mx)[2])
{
    float z[8];
    r.opaque();
    r.get(z);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        mx[0] = fmaxf(mx[0], z[2 * e]);
        mx[1] = fmaxf(mx[1], z[2 * e + 1]);
    }
}

template <bool BF16>
__device__ __forceinline__ void sum8(Raw8<BF16> &r, float ref, float c, float (&s)[2])
{
    float z[8];
    r.opaque();
    r.get(z);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        s[0] += fast_exp2((z[2 * e] - ref) * c);
        s[1] += fast_exp2((z[2 * e + 1] - ref) * c);
    }
}

__device__ __forceinline__ float upstream(const Distill &a, int64_t row)
{
    return a.temperature * (a.grad_loss ? a.grad_loss[row] : 1.0f);
}

// Chunks of eight logits of [lo, hi), lo a multiple of eight: chunk i of this thread's is
// lo / 8 + threadIdx.x + i * NT.  UN loads are issued before their values are used.
template <bool BF16, int NT, typename F>
__device__ __forceinline__ void for_chunks(const Distill &a, int64_t row, int lo, int hi, F f)
{
    constexpr int UN = BF16 ? 4 : 2;
    const int64_t base = row * a.ldz;
    const int full = lo + ((hi - lo) & ~7);
    for (int v = lo + threadIdx.x * 8; v < full; v += UN * NT * 8) {
        Raw8<BF16> r[UN];
#pragma unroll
        for (int i = 0; i < UN; ++i)
            if (v + i * NT * 8 < full)
                r[i].load(a.Z, base + v + i * NT * 8);
#pragma unroll
        for (int i = 0; i < UN; ++i) {
            if (v + i * NT * 8 < full) {
                float z[8];
                r[i].get(z);
                f(z, v + i * NT * 8, 8);
            }
        }
    }
    if (full < hi && threadIdx.x == NT - 1) {
        Raw8<BF16> r;
        r.fill(-kInf);
        r.load_part(a.Z, base + full, hi - full);
        float z[8];
        r.get(z);
        f(z, full, hi - full);
    }
}

// Gradient bulk of the part [lo, hi) of a row, then the teacher's entries in it.
template <bool BF16, int NT>
__device__ __forceinline__ void part_grad(const Distill &a, const Teacher &t, int64_t row, int lo, int hi, float m,
                                          float l)
{
    const float c = kLog2e / a.temperature, l2 = l * kLog2e, g = upstream(a, row);
    if (t.flags[0])
        for_chunks<BF16, NT>(a, row, lo, hi, [&](float (&z)[8], int v, int n) {
            grad8(z, g, m, c, l2);
            store_upto<BF16>(a.grad, row * a.ldg + v, z, n);
        });
    else
        for (int v = lo + threadIdx.x * 8; v < hi; v += NT * 8) {
            const float z[8] = {};
            store_upto<BF16>(a.grad, row * a.ldg + v, z, hi - v);
        }
    __syncthreads();   // orders the two writes of an entry
    fix_entries<BF16, NT>(a, t, row, lo, hi, g, m, l);
}

// (m, s) of NW waves from the teacher's part array.
template <int NW>
__device__ __forceinline__ MaxSum join_parts(const Teacher &t, float c)
{
    MaxSum x;
#pragma unroll
    for (int w = 0; w < NW; ++w)
        x.m = fmaxf(x.m, t.part[w]);
    const float ref = ref_of(x.m);
#pragma unroll
    for (int w = 0; w < NW; ++w)
        x.s += t.part[16 + w] * fast_exp2((t.part[w] - ref) * c);
    return x;
}

// Joins the waves' (m, s) of a workgroup: m and l of the row in every thread.  Its barrier also
// publishes the teacher.
template <int NT>
__device__ __forceinline__ void join_block(MaxSum x, const Teacher &t, float c, float &m, float &l)
{
    x.join_wave(c);
    if constexpr (NT == 64) {
        __syncthreads();
    } else {
        const int wave = threadIdx.x >> 6;
        if ((threadIdx.x & 63) == 0) {
            t.part[wave] = x.m;
            t.part[16 + wave] = x.s;
        }
        __syncthreads();
        x = join_parts<NT / 64>(t, c);
    }
    m = x.m;
    l = logf(x.s);
}

// One row per workgroup.  R > 0: the row stays in registers, R chunks of eight logits per
// thread (V <= 8 NT R), and is read once; R = 0: a gradient reads it again.
template <bool BF16, int NT, int R>
__global__ __launch_bounds__(NT) void distill_row_kernel(const Distill a, int slots)
{
    extern __shared__ int32_t lds[];
    const Teacher t(lds, a.K, slots);
    const float c = kLog2e / a.temperature;
    const int64_t n = row_count(a.count, a.rows);
    const int V = a.V, full = V & ~7;
    for (int64_t row = blockIdx.x; row < n; row += gridDim.x) {
        MaxSum x;
        Raw8<BF16> r[R > 0 ? R : 1], rest;   // whole chunks, and the last, shorter one
        if (threadIdx.x < 64)
            load_teacher<BF16>(a, row, t, nullptr, 0, V);
        if constexpr (R > 0) {
#pragma unroll
            for (int i = 0; i < R; ++i) {
                const int v = (i * NT + threadIdx.x) * 8;
                r[i].fill(-kInf);
                if (v < full)
                    r[i].load(a.Z, row * a.ldz + v);
            }
            rest.fill(-kInf);
            if (full < V && threadIdx.x == NT - 1)
                rest.load_part(a.Z, row * a.ldz + full, V - full);
            float mx[2] = {-kInf, -kInf};
#pragma unroll
            for (int i = 0; i < R; ++i)
                max8(r[i], mx);
            max8(rest, mx);
            x.m = fmaxf(mx[0], mx[1]);
            const float ref = ref_of(x.m);
            float s[2] = {0.0f, 0.0f};
#pragma unroll
            for (int i = 0; i < R; ++i)
                sum8(r[i], ref, c, s);
            if (full < V)
                sum8(rest, ref, c, s);
            x.s = s[0] + s[1];
        } else {
            for_chunks<BF16, NT>(a, row, 0, V, [&](float (&z)[8], int, int) { x.add(z, c); });
        }
        float m, l;
        join_block<NT>(x, t, c, m, l);
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
                const float l2 = l * kLog2e, g = upstream(a, row);
#pragma unroll
                for (int i = 0; i < R; ++i) {
                    const int v = (i * NT + threadIdx.x) * 8;
                    if (v < full) {
                        float z[8];
                        r[i].opaque();
                        r[i].get(z);
                        grad8(z, g, m, c, l2, present);
                        store8<BF16>(a.grad, row * a.ldg + v, z);
                    }
                }
                if (full < V && threadIdx.x == NT - 1) {
                    float z[8];
                    rest.get(z);
                    grad8(z, g, m, c, l2, present);
                    store_upto<BF16>(a.grad, row * a.ldg + full, z, V - full);
                }
                __syncthreads();   // orders the two writes of an entry
                fix_entries<BF16, NT>(a, t, row, 0, V, g, m, l);
            } else {
                part_grad<BF16, NT>(a, t, row, 0, V, m, l);
            }
        }
        __syncthreads();   // the teacher's arrays are refilled for the next row
    }
}

// Loss and gradient of long rows.  A workgroup of 16 waves has a CU to itself and walks its
// rows: 15 waves hold the row in registers, R chunks of eight logits per thread (V <= 7680 R),
// and wave 0 prepares the next row's teacher, writes the loss and mends the entries of the row
// before.  As soon as a chunk's gradient is stored, its registers take the next row's logits,
// so that reads and writes run side by side; the one barrier of a row publishes the waves'
// sums and the teacher, and finds the stores of the row before complete, behind the loads
// that it waits for anyway.
template <bool BF16, int R>
__global__ __launch_bounds__(1024) void distill_stream_kernel(const Distill a, int slots, int teacher_words)
{
    extern __shared__ int32_t lds[];
    constexpr int ND = 960;
    const Teacher t0(lds, a.K, slots), t1(lds + teacher_words, a.K, slots);
    const float c = kLog2e / a.temperature;
    const int64_t n = row_count(a.count, a.rows);
    const int V = a.V, full = V & ~7;
    int64_t row = blockIdx.x;
    if (row >= n)
        return;
    if (threadIdx.x < 64) {
        load_teacher<BF16>(a, row, t0, nullptr, 0, V);
        __syncthreads();
        float pm = 0.0f, pl = 0.0f;
        for (bool odd = false, first = true;; odd = !odd, first = false) {
            const Teacher &t = odd ? t1 : t0, &other = odd ? t0 : t1;
            const MaxSum x = join_parts<15>(t, c);
            const float m = x.m, l = logf(x.s), loss = row_loss(a, t, m, l);
            if (threadIdx.x == 0) {
                a.loss[row] = t.flags[0] ? loss : 0.0f;
                a.stats[2 * row] = m;
                a.stats[2 * row + 1] = l;
            }
            if (!first)
                fix_entries<BF16, 64>(a, other, row - gridDim.x, 0, V, upstream(a, row - gridDim.x), pm, pl);
            pm = m;
            pl = l;
            const int64_t next = row + gridDim.x;
            if (next < n)
                load_teacher<BF16>(a, next, other, nullptr, 0, V);
            __syncthreads();
            if (next >= n) {
                fix_entries<BF16, 64>(a, t, row, 0, V, upstream(a, row), m, l);
                return;
            }
            row = next;
        }
    }
    const int d = threadIdx.x - 64;
    const bool has_rest = full < V && d == ND - 1;
    Raw8<BF16> r[R], rest;   // whole chunks, and the last, shorter one
    rest.fill(-kInf);
#pragma unroll
    for (int i = 0; i < R; ++i) {
        r[i].fill(-kInf);
        if ((i * ND + d) * 8 < full)
            r[i].load(a.Z, row * a.ldz + (i * ND + d) * 8);
    }
    if (has_rest)
        rest.load_part(a.Z, row * a.ldz + full, V - full);
    for (bool odd = false;; odd = !odd) {
        const Teacher &t = odd ? t1 : t0;
        float mx[2] = {-kInf, -kInf};
#pragma unroll
        for (int i = 0; i < R; ++i)
            max8(r[i], mx);
        if (full < V)
            max8(rest, mx);
        const float wm = wave_reduce(fmaxf(mx[0], mx[1]), MaxOp{}), ref = ref_of(wm);
        float s[2] = {0.0f, 0.0f};
#pragma unroll
        for (int i = 0; i < R; ++i)
            sum8(r[i], ref, c, s);
        if (full < V)
            sum8(rest, ref, c, s);
        const float ws = wave_reduce(s[0] + s[1], AddOp{});
        if ((threadIdx.x & 63) == 0) {
            t.part[(threadIdx.x >> 6) - 1] = wm;
            t.part[15 + (threadIdx.x >> 6)] = ws;
        }
        __syncthreads();
        const MaxSum x = join_parts<15>(t, c);
        const float m = x.m, l2 = logf(x.s) * kLog2e, g = upstream(a, row);
        const bool present = t.flags[0];
        const int64_t next = row + gridDim.x;
#pragma unroll
        for (int i = 0; i < R; ++i) {
            const int v = (i * ND + d) * 8;
            if (v < full) {
                float z[8];
                r[i].opaque();
                r[i].get(z);
                grad8(z, g, m, c, l2, present);
                store8<BF16>(a.grad, row * a.ldg + v, z);
                if (next < n)
                    r[i].load(a.Z, next * a.ldz + v);
            }
        }
        if (has_rest) {
            float z[8];
            rest.get(z);
            grad8(z, g, m, c, l2, present);
            store_upto<BF16>(a.grad, row * a.ldg + full, z, V - full);
            if (next < n)
                rest.load_part(a.Z, next * a.ldz + full, V - full);
        }
        if (next >= n) {
            __syncthreads();   // the last row's stores, before its entries are mended
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

constexpr int kSplitThreads = 256;

// (maximum, sum) of each part of each row into partials[row][part][2], and the student's
// logits at the teacher's entries into z_at[row][K] (the gradient may overwrite them).
template <bool BF16>
__global__ __launch_bounds__(kSplitThreads) void distill_part_kernel(const Distill a, int parts,
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
    MaxSum x;
    for_chunks<BF16, kSplitThreads>(a, row, lo, hi, [&](float (&z)[8], int, int) { x.add(z, c); });
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
        for (int j = threadIdx.x; j < a.K; j += kSplitThreads) {
            const int32_t id = a.ids[row * a.K + j];
            z_at[row * a.K + j] = id >= 0 && id < a.V ? load1(a.Z, row * a.ldz + id, BF16) : 0.0f;
        }
}

// Gradient of part blockIdx.x % cuts of a row.  parts > 0: the statistics are joined from the
// row's partials, and the workgroup of the first part writes them and the loss; parts = 0:
// they are given.
template <bool BF16>
__global__ __launch_bounds__(kSplitThreads) void distill_split_kernel(const Distill a, int slots, int parts, int cuts,
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
        float m, l;
        if (parts > 0) {
            MaxSum x;
            const int i = threadIdx.x & 63;   // parts <= 64
            if (i < parts)
                x = MaxSum{a.partials[2 * (row * parts + i)], a.partials[2 * (row * parts + i) + 1]};
            x.join_wave(c);
            m = x.m;
            l = logf(x.s);
        } else {
            m = a.stats[2 * row];
            l = a.stats[2 * row + 1];
        }
        __syncthreads();   // the teacher is there
        if (parts > 0 && s == 0 && threadIdx.x < 64) {
            const float loss = row_loss(a, t, m, l);
            if (threadIdx.x == 0) {
                a.loss[row] = t.flags[0] ? loss : 0.0f;
                a.stats[2 * row] = m;
                a.stats[2 * row + 1] = l;
            }
        }
        if (a.grad)
            part_grad<BF16, kSplitThreads>(a, t, row, lo, hi, m, l);
        __syncthreads();   // the teacher's arrays are refilled for the next row
    }
}

// Parts of a row in the split form: about 2048 workgroups, of 4096 logits at least each.
int parts_of(int64_t rows, int64_t V)
{
    return (int)std::max<int64_t>(1, std::min<int64_t>({64, 2048 / std::max<int64_t>(rows, 1), V / 4096}));
}

// Few rows of many logits go over several workgroups each.
bool is_split(int64_t rows, int64_t V, bool grad) { return rows <= (grad ? 128 : 1024) && V >= 16384; }

template <bool BF16>
hipError_t run(const Distill &a, hipStream_t stream)
{
    const int slots = table_slots(a.K);
    const size_t lds = teacher_bytes(a.K);
    if (is_split(a.rows, a.V, a.grad)) {
        const int parts = parts_of(a.rows, a.V), cuts = a.grad ? parts : 1;
        float *z_at = a.partials + 2 * a.rows * parts;
        hipLaunchKernelGGL(distill_part_kernel<BF16>, dim3((unsigned)(a.rows * parts)), dim3(kSplitThreads), 0,
                           stream, a, parts, z_at);
        hipLaunchKernelGGL(distill_split_kernel<BF16>, dim3((unsigned)(a.rows * cuts)), dim3(kSplitThreads), lds,
                           stream, a, slots, parts, cuts, z_at);
        return hipGetLastError();
    }
    const dim3 grid((unsigned)std::min<int64_t>(a.rows, 1 << 20));
    auto go = [&](auto kernel, int threads) {
        hipLaunchKernelGGL(kernel, grid, dim3(threads), lds, stream, a, slots);
    };
    auto stream_rows = [&](auto kernel) {
        int dev = 0, cus = 256;
        if (hipGetDevice(&dev) == hipSuccess)
            (void)hipDeviceGetAttribute(&cus, hipDeviceAttributeMultiprocessorCount, dev);
        hipLaunchKernelGGL(kernel, dim3((unsigned)std::min<int64_t>(a.rows, cus)), dim3(1024), 2 * lds, stream, a,
                           slots, (int)(lds / 4));
    };
    if (a.V <= 64 * 8 * 4)
        go(distill_row_kernel<BF16, 64, 4>, 64);
    else if (a.V <= 256 * 8 * 8)
        go(distill_row_kernel<BF16, 256, 8>, 256);
    else if (!a.grad)
        go(distill_row_kernel<BF16, 256, 0>, 256);
    else if (a.V <= 7680 * 5)
        stream_rows(distill_stream_kernel<BF16, 5>);
    else if (a.V <= 7680 * 9)
        stream_rows(distill_stream_kernel<BF16, 9>);
    else if (BF16 && a.V <= 7680 * 13)
        stream_rows(distill_stream_kernel<BF16, BF16 ? 13 : 9>);
    else if (BF16 && a.V <= 7680 * 17)
        stream_rows(distill_stream_kernel<BF16, BF16 ? 17 : 9>);
    else if (BF16 && a.V <= 7680 * 20)
        stream_rows(distill_stream_kernel<BF16, BF16 ? 20 : 9>);
    else
        go(distill_row_kernel<BF16, 1024, 0>, 1024);
    return hipGetLastError();
}

template <bool BF16>
hipError_t run_grad(const Distill &a, hipStream_t stream)
{
    const int cuts = parts_of(a.rows, a.V);
    hipLaunchKernelGGL(distill_split_kernel<BF16>, dim3((unsigned)std::min<int64_t>(a.rows * cuts, 1 << 20)),
                       dim3(kSplitThreads), teacher_bytes(a.K), stream, a, table_slots(a.K), 0, cuts,
                       (const float *)nullptr);
    return hipGetLastError();
}

}  // namespace

int64_t distill_workspace_bytes(int64_t rows, int64_t V, int64_t K)
{
    return is_split(rows, V, false) ? 4 * rows * (2 * parts_of(rows, V) + K) : 0;
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
