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
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "launch.h"
#include "row_ops.h"

namespace mosaic {
namespace {

using namespace rows;

constexpr float kLog2e = 1.44269504088896340736f;

// Running maximum and sum of exp((z - max) / T) of a set of logits; c = log2(e) / T.
struct MaxSum {
    float m = -__builtin_inff(), s = 0.0f;

    // -inf stands for nothing seen yet, and (-inf) - (-inf) would be NaN
    __device__ __forceinline__ static float ref(float m) { return m == -__builtin_inff() ? 0.0f : m; }

    template <int N>
    __device__ __forceinline__ void add(const float (&z)[N], float c)
    {
        float mx = z[0];
#pragma unroll
        for (int i = 1; i < N; ++i)
            mx = fmaxf(mx, z[i]);
        if (mx > m) {
            s *= exp2f((m - mx) * c);
            m = mx;
        }
        const float r = ref(m);
#pragma unroll
        for (int i = 0; i < N; ++i)
            s += exp2f((z[i] - r) * c);
    }

    __device__ __forceinline__ void join(float m2, float s2, float c)
    {
        const float mx = fmaxf(m, m2), r = ref(mx);
        s = s * exp2f((m - r) * c) + s2 * exp2f((m2 - r) * c);
        m = mx;
    }
};

// The teacher's side of one row, in LDS.
struct Teacher {
    int32_t id[kDistillMaxK];
    float p[kDistillMaxK];      // 0 for an absent entry
    float z[kDistillMaxK];      // the student's logit at the entry
    float red[16];
};

// Fills t from the row's K entries (every thread takes part; ends with a barrier).  Returns
// sum_j p_j log p_j, and whether any entry is present.
template <bool BF16, int NW>
__device__ __forceinline__ float load_teacher(const Distill &a, int64_t row, Teacher &t, bool &present)
{
    const float c = kLog2e / a.temperature;
    float mx = -__builtin_inff();
    int any = 0;
    for (int j = threadIdx.x; j < a.K; j += 64 * NW) {
        const int32_t id = a.ids[row * a.K + j];
        float x[1];
        if (a.top_bf16)
            load<true, 1>(a.top, row * a.K + j, x);
        else
            load<false, 1>(a.top, row * a.K + j, x);
        const bool here = id >= 0 && id < a.V && x[0] != -__builtin_inff();
        float z[1] = {0.0f};
        if (here)
            load<BF16, 1>(a.Z, row * a.ldz + id, z);
        t.id[j] = here ? id : -1;
        t.p[j] = x[0];
        t.z[j] = z[0];
        mx = here ? fmaxf(mx, x[0]) : mx;
        any |= here;
    }
    mx = block_reduce<NW>(mx, MaxOp{}, t.red);
    present = __syncthreads_or(any);
    float sum = 0.0f;
    for (int j = threadIdx.x; j < a.K; j += 64 * NW) {
        const float e = t.id[j] >= 0 ? exp2f((t.p[j] - mx) * c) : 0.0f;
        t.p[j] = e;
        sum += e;
    }
    sum = block_reduce<NW>(sum, AddOp{}, t.red);
    float h = 0.0f;
    for (int j = threadIdx.x; j < a.K; j += 64 * NW) {
        const float p = present ? t.p[j] / sum : 0.0f;
        t.p[j] = p;
        h += p != 0.0f ? p * logf(p) : 0.0f;
    }
    return block_reduce<NW>(h, AddOp{}, t.red);
}

// The row's loss from its statistics, in every thread.
template <int NW>
__device__ __forceinline__ float row_loss(const Distill &a, Teacher &t, float entropy, float m, float l)
{
    const float T = a.temperature, inv = 1.0f / T;
    float x = 0.0f;
    for (int j = threadIdx.x; j < a.K; j += 64 * NW)
        x += t.p[j] != 0.0f ? t.p[j] * ((t.z[j] - m) * inv - l) : 0.0f;
    x = block_reduce<NW>(x, AddOp{}, t.red);
    return T * T * (entropy - x);
}

// Gradient of one row from its statistics.  The bulk is written first, T g q_v everywhere;
// then the entries the teacher names are written again with their p taken off.
template <bool BF16, int VEC, int NW>
__device__ __forceinline__ void row_grad(const Distill &a, Teacher &t, int64_t row, bool present, float m, float l)
{
    const float c = kLog2e / a.temperature, l2 = l * kLog2e;
    const float g = a.temperature * (a.grad_loss ? a.grad_loss[row] : 1.0f);
    for (int64_t v = threadIdx.x * VEC; v < a.V; v += 64 * NW * VEC) {
        float z[VEC];
        if (present) {
            load<BF16, VEC>(a.Z, row * a.ldz + v, z);
#pragma unroll
            for (int i = 0; i < VEC; ++i)
                z[i] = g * exp2f((z[i] - m) * c - l2);
        } else {
#pragma unroll
            for (int i = 0; i < VEC; ++i)
                z[i] = 0.0f;
        }
        store<BF16, VEC>(a.grad, row * a.ldg + v, z);
    }
    // every wave's stores have reached memory before any is overwritten
    __builtin_amdgcn_s_waitcnt(0);
    __syncthreads();
    for (int j = threadIdx.x; j < a.K; j += 64 * NW) {
        const int32_t id = t.id[j];
        if (id < 0)
            continue;
        float p = 0.0f;
        bool first = true;
        for (int i = 0; i < a.K; ++i) {
            if (t.id[i] == id) {
                first = first && i >= j;
                p += t.p[i];
            }
        }
        if (first) {   // an entry named twice is written once, with both shares
            const float x[1] = {g * (exp2f((t.z[j] - m) * c - l2) - p)};
            store<BF16, 1>(a.grad, row * a.ldg + id, x);
        }
    }
    __syncthreads();   // the teacher's arrays are refilled for the next row
}

// One row per workgroup.
template <bool BF16, int VEC, int NW, bool LOSS>
__global__ __launch_bounds__(64 * NW) void distill_row_kernel(const Distill a)
{
    __shared__ Teacher t;
    const float c = kLog2e / a.temperature;
    const int64_t n = row_count(a.count, a.rows);
    for (int64_t row = blockIdx.x; row < n; row += gridDim.x) {
        bool present;
        const float entropy = load_teacher<BF16, NW>(a, row, t, present);
        float m, l;
        if constexpr (LOSS) {
            MaxSum x;
            for (int64_t v = threadIdx.x * VEC; v < a.V; v += 64 * NW * VEC) {
                float z[VEC];
                load<BF16, VEC>(a.Z, row * a.ldz + v, z);
                x.add(z, c);
            }
            m = block_reduce<NW>(x.m, MaxOp{}, t.red);
            l = logf(block_reduce<NW>(x.s * exp2f((x.m - MaxSum::ref(m)) * c), AddOp{}, t.red));
            const float loss = row_loss<NW>(a, t, entropy, m, l);
            if (threadIdx.x == 0) {
                a.loss[row] = present ? loss : 0.0f;
                a.stats[2 * row] = m;
                a.stats[2 * row + 1] = l;
            }
        } else {
            m = a.stats[2 * row];
            l = a.stats[2 * row + 1];
        }
        if (a.grad)
            row_grad<BF16, VEC, NW>(a, t, row, present, m, l);
        else
            __syncthreads();
    }
}

template <bool BF16, bool LOSS>
hipError_t run(const Distill &a, hipStream_t stream)
{
    const int64_t es = BF16 ? 2 : 4;
    auto ok = [&](const void *p, int64_t ld) { return !p || (((uintptr_t)p & 15) == 0 && ld * es % 16 == 0); };
    const bool vec = a.V % 8 == 0 && ok(a.Z, a.ldz) && ok(a.grad, a.ldg);
    const dim3 grid((unsigned)std::min<int64_t>(a.rows, 1 << 20));
    if (vec)
        hipLaunchKernelGGL((distill_row_kernel<BF16, 8, 16, LOSS>), grid, dim3(1024), 0, stream, a);
    else
        hipLaunchKernelGGL((distill_row_kernel<BF16, 1, 16, LOSS>), grid, dim3(1024), 0, stream, a);
    return hipGetLastError();
}

}  // namespace

int64_t distill_workspace_bytes(int64_t, int64_t) { return 0; }

hipError_t launch_distill(const Distill &a, bool z_bf16, hipStream_t stream)
{
    return z_bf16 ? run<true, true>(a, stream) : run<false, true>(a, stream);
}

hipError_t launch_distill_grad(const Distill &a, bool z_bf16, hipStream_t stream)
{
    return z_bf16 ? run<true, false>(a, stream) : run<false, false>(a, stream);
}

}  // namespace mosaic
