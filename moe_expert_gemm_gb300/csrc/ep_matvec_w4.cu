// Expert products of a few rows on 4-bit weights: C[m][n] = sum_k W_e[n][k] a[m][k].
//
// One warp forms one output element: its lanes walk the weight row 8 codes at a time.
#include <cuda_bf16.h>

#include "ep_internal.h"
#include "ep_ptx.cuh"

namespace ep {

constexpr int kW4Threads = 256;

__device__ __forceinline__ float e2m1_value(uint32_t code)
{
    const float mag = code & 6 ? static_cast<float>(2 + (code & 1)) * static_cast<float>(1 << ((code >> 1 & 3) - 1)) * 0.5f
                               : 0.5f * (code & 1);
    return code & 8 ? -mag : mag;
}

__device__ float w4_dot(const W4Params &p, int e, int64_t n, const uint8_t *a, int lane)
{
    const int64_t row = static_cast<int64_t>(e) * p.N + n;
    const uint32_t *w = reinterpret_cast<const uint32_t *>(p.W + row * (p.K / 2));
    const int groups = p.K / p.group;
    float sum = 0.f;
    for (int c = lane; c < p.K / 8; c += 32) {
        const uint32_t codes = __ldg(w + c);
        const uint4 av = __ldg(reinterpret_cast<const uint4 *>(a) + c);
        const uint32_t x[4] = {av.x, av.y, av.z, av.w};
        const int64_t g = row * groups + c * 8 / p.group;
        float scale, zero = 8.f;
        if (p.format == EP_W4_E2M1) {
            const uint32_t b = __ldg(static_cast<const uint8_t *>(p.scales) + g);
            scale = b == 255 ? NAN : b ? __uint_as_float(b << 23) : 0x1p-127f;
        } else {
            scale = __uint_as_float(static_cast<uint32_t>(__ldg(static_cast<const unsigned short *>(p.scales) + g)) << 16);
            if (p.zeros)
                zero = __ldg(p.zeros + g);
        }
        float part = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const uint32_t q = codes >> 4 * i & 15;
            const float v = p.format == EP_W4_E2M1 ? e2m1_value(q) : static_cast<float>(q) - zero;
            part = fmaf(v, __uint_as_float(i & 1 ? x[i / 2] & 0xFFFF0000u : x[i / 2] << 16), part);
        }
        sum = fmaf(scale, part, sum);
    }
#pragma unroll
    for (int o = 16; o; o >>= 1)
        sum += __shfl_xor_sync(0xffffffffu, sum, o);
    return sum;
}

__global__ void __launch_bounds__(kW4Threads) matvec_w4_kernel(const W4Params p)
{
    const int lane = threadIdx.x & 31;
    const int64_t warp = (static_cast<int64_t>(blockIdx.x) * kW4Threads + threadIdx.x) >> 5;
    const int64_t warps = static_cast<int64_t>(gridDim.x) * kW4Threads / 32;
    const int64_t m_total = __ldg(p.expert_offsets + p.El);
    bool bad = false;
    for (int e = lane; e <= p.El; e += 32) {
        const int lo = e ? __ldg(p.expert_offsets + e - 1) : 0, hi = __ldg(p.expert_offsets + e);
        bad |= hi < lo || hi > p.max_rows;
    }
    if (__any_sync(0xffffffffu, bad)) {
        if (warp == 0 && lane == 0)
            atomicOr(p.status, EP_STATUS_BOUNDS);
        return;
    }
    const int cols = p.swiglu ? p.N / 2 : p.N;
    for (int64_t u = warp; u < m_total * cols; u += warps) {
        const int64_t m = u / cols;
        const int n = static_cast<int>(u - m * cols);
        int e = 0;
        while (e + 1 < p.El && __ldg(p.expert_offsets + e + 1) <= m)
            ++e;
        const uint8_t *a;
        if (p.A) {
            a = p.A + m * p.K * 2;
        } else {
            const int64_t gi = __ldg(p.gather_idx + m);
            const int64_t Tk = static_cast<int64_t>(p.T) * p.top_k;
            const int64_t rk = gi / Tk, t = (gi - rk * Tk) / p.top_k;
            if (gi < 0 || rk >= p.n_ranks) {
                if (lane == 0)
                    atomicOr(p.status, EP_STATUS_BOUNDS);
                continue;
            }
            a = p.x[rk] + t * p.K * 2;
        }
        float y = w4_dot(p, e, n, a, lane);
        if (p.swiglu)
            y = silu_f32(y) * w4_dot(p, e, n + p.N / 2, a, lane);
        if (lane == 0)
            reinterpret_cast<__nv_bfloat16 *>(p.C)[m * cols + n] = __float2bfloat16_rn(y);
    }
}

int64_t w4_workspace_bytes()
{
    return 16;
}

cudaError_t launch_matvec_w4(const W4Params &p, int num_sms, cudaStream_t s)
{
    matvec_w4_kernel<<<8 * num_sms, kW4Threads, 0, s>>>(p);
    return cudaGetLastError();
}

}  // namespace ep
