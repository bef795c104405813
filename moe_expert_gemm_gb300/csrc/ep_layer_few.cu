// A whole MoE layer for a few tokens: the up/gate products with the activation, then the down
// products with the gates, a kernel each. Bound by the weights of the experts that have tokens.
// This is the plain form: a warp takes one value of one token's activation, or of its output.
#include "ep_internal.h"
#include "ep_ptx.cuh"
#include "ep_rows.cuh"

namespace ep {

namespace {

constexpr int kFewThreads = 256;

__device__ __forceinline__ float value(const uint8_t *base, int64_t i, bool fp8)
{
    if (fp8)
        return __half2float(__nv_cvt_fp8_to_halfraw(base[i], __NV_E4M3));
    return __bfloat162float(reinterpret_cast<const __nv_bfloat16 *>(base)[i]);
}

__device__ __forceinline__ float warp_sum(float v)
{
#pragma unroll
    for (int o = 16; o; o >>= 1)
        v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// The local expert of a slot; -1 if it lives elsewhere, -2 if nowhere.
__device__ __forceinline__ int local_expert(const FewParams &p, int slot)
{
    const int id = __ldg(p.topk_ids + slot);
    if (id < 0 || id >= p.n_ranks * p.El)
        return -2;
    return id / p.El == p.my_rank ? id % p.El : -1;
}

}  // namespace

// a[slot][i] in fp32.
__global__ void __launch_bounds__(kFewThreads) few_up_kernel(const FewParams p)
{
    griddep_wait();
    griddep_launch_dependents();
    float *a = reinterpret_cast<float *>(p.workspace);
    const int lane = threadIdx.x & 31;
    const int64_t warps = static_cast<int64_t>(gridDim.x) * (kFewThreads / 32);
    const int64_t all = static_cast<int64_t>(p.T) * p.top_k * p.I;
    for (int64_t w = static_cast<int64_t>(blockIdx.x) * (kFewThreads / 32) + threadIdx.x / 32; w < all; w += warps) {
        const int slot = static_cast<int>(w / p.I), i = static_cast<int>(w % p.I), t = slot / p.top_k;
        const int e = local_expert(p, slot);
        if (e < 0) {
            if (e == -2 && i == 0 && lane == 0)
                atomicOr(p.status, EP_STATUS_ROUTING);
            continue;
        }
        const int64_t gate_row = static_cast<int64_t>(e) * 2 * p.I + i, up_row = gate_row + p.I;
        float gate = 0.f, up = 0.f;
        for (int k = lane; k < p.H; k += 32) {
            const float x = value(p.x, static_cast<int64_t>(t) * p.H + k, p.fp8);
            float wg = value(p.W1, gate_row * p.H + k, p.fp8), wu = value(p.W1, up_row * p.H + k, p.fp8);
            if (p.fp8) {
                const float s = p.x_scales[static_cast<int64_t>(t) * (p.H / 128) + k / 128];
                wg *= s * p.w1_scales[gate_row / 128 * (p.H / 128) + k / 128];
                wu *= s * p.w1_scales[up_row / 128 * (p.H / 128) + k / 128];
            }
            gate = fmaf(wg, x, gate);
            up = fmaf(wu, x, up);
        }
        gate = warp_sum(gate);
        up = warp_sum(up);
        if (lane == 0)
            a[w] = silu_f32(gate) * up;
    }
}

__global__ void __launch_bounds__(kFewThreads) few_down_kernel(const FewParams p)
{
    griddep_wait();
    griddep_launch_dependents();
    const float *a = reinterpret_cast<const float *>(p.workspace);
    const int lane = threadIdx.x & 31;
    const int64_t warps = static_cast<int64_t>(gridDim.x) * (kFewThreads / 32);
    const int64_t all = static_cast<int64_t>(p.T) * p.H;
    for (int64_t w = static_cast<int64_t>(blockIdx.x) * (kFewThreads / 32) + threadIdx.x / 32; w < all; w += warps) {
        const int t = static_cast<int>(w / p.H), n = static_cast<int>(w % p.H);
        float out = 0.f;
        for (int j = 0; j < p.top_k; ++j) {
            const int slot = t * p.top_k + j, e = local_expert(p, slot);
            if (e < 0)
                continue;
            const int64_t row = static_cast<int64_t>(e) * p.H + n;
            float y = 0.f;
            for (int k0 = 0; k0 < p.I; k0 += 128) {
                float v[4];
                uint32_t bits = 0;
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    const int k = k0 + 32 * u + lane;
                    v[u] = k < p.I ? a[static_cast<int64_t>(slot) * p.I + k] : 0.f;
                    bits = max(bits, rows::size_bits(v[u]));
                }
                const float s = rows::scale_of(__reduce_max_sync(0xffffffffu, bits));
                float part = 0.f;
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    const int k = k0 + 32 * u + lane;
                    if (k >= p.I)
                        continue;
                    if (p.fp8) {
                        const __nv_fp8_storage_t q = __nv_cvt_float_to_fp8(v[u] * (1.f / s), __NV_SATFINITE, __NV_E4M3);
                        v[u] = __half2float(__nv_cvt_fp8_to_halfraw(q, __NV_E4M3));
                    } else {
                        v[u] = __bfloat162float(__float2bfloat16_rn(v[u]));
                    }
                    part = fmaf(value(p.W2, row * p.I + k, p.fp8), v[u], part);
                }
                y = p.fp8 ? fmaf(s * p.w2_scales[row / 128 * (p.I / 128) + k0 / 128], part, y) : y + part;
            }
            out = fmaf(__ldg(p.gates + slot), warp_sum(y), out);
        }
        if (lane == 0)
            reinterpret_cast<__nv_bfloat16 *>(p.out)[w] = __float2bfloat16_rn(out);
    }
}

int64_t few_workspace_bytes(const FewParams &p)
{
    return static_cast<int64_t>(p.T) * p.top_k * p.I * 4 + 16;
}

cudaError_t launch_layer_few(const FewParams &p, int num_sms, cudaStream_t s)
{
    const cudaError_t e = launch_behind(few_up_kernel, 8 * num_sms, kFewThreads, 0, s, p);
    return e != cudaSuccess ? e : launch_behind(few_down_kernel, 8 * num_sms, kFewThreads, 0, s, p);
}

}  // namespace ep
