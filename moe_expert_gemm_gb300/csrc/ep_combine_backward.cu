// Gradient of the gate-weighted combine out[t] = sum_j g[t, j] * row(t, j):
//   dgates[t, j] = <dout[t], row(t, j)>,   drow(t, j) = g[t, j] * dout[t].
// HBM-bound: the rows are read once, their gradient written once. One block takes one
// token.
#include <cuda_bf16.h>

#include "ep_internal.h"

namespace ep {

constexpr int kCombineBwdThreads = 256;

__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi)
{
    const __nv_bfloat162 b = __float22bfloat162_rn(make_float2(lo, hi));
    return *reinterpret_cast<const uint32_t *>(&b);
}

__global__ void __launch_bounds__(kCombineBwdThreads)
    combine_backward_kernel(const CombineBackwardParams p)
{
    __shared__ float part[kCombineBwdThreads / 32];
    const int64_t t = blockIdx.x;
    const int vecs = p.N / 8;
    const uint4 *dout = reinterpret_cast<const uint4 *>(p.dout + t * p.N * 2);
    for (int j = 0; j < p.top_k; ++j) {
        const int64_t row = (t * p.top_k + j) * p.N * 2;
        const float g = p.drows ? __ldg(p.gates + t * p.top_k + j) : 0.f;
        float sum = 0.f;
        for (int v = threadIdx.x; v < vecs; v += kCombineBwdThreads) {
            const uint4 dv = __ldg(dout + v);
            const uint32_t d[4] = {dv.x, dv.y, dv.z, dv.w};
            if (p.dgates) {
                const uint4 rv = *(reinterpret_cast<const uint4 *>(p.recv_buf + row) + v);
                const uint32_t r[4] = {rv.x, rv.y, rv.z, rv.w};
#pragma unroll
                for (int h = 0; h < 4; ++h) {
                    sum = fmaf(bf16_lo(d[h]), bf16_lo(r[h]), sum);
                    sum = fmaf(bf16_hi(d[h]), bf16_hi(r[h]), sum);
                }
            }
            if (p.drows) {
                uint32_t o[4];
#pragma unroll
                for (int h = 0; h < 4; ++h)
                    o[h] = pack_bf16(g * bf16_lo(d[h]), g * bf16_hi(d[h]));
                *(reinterpret_cast<uint4 *>(p.drows + row) + v) = make_uint4(o[0], o[1], o[2], o[3]);
            }
        }
        if (!p.dgates)
            continue;
#pragma unroll
        for (int o = 16; o; o >>= 1)
            sum += __shfl_xor_sync(0xffffffffu, sum, o);
        if (threadIdx.x % 32 == 0)
            part[threadIdx.x / 32] = sum;
        __syncthreads();
        if (threadIdx.x == 0) {
            float all = 0.f;
            for (int w = 0; w < kCombineBwdThreads / 32; ++w)
                all += part[w];
            p.dgates[t * p.top_k + j] = all;
        }
        __syncthreads();
    }
}

cudaError_t launch_combine_backward(const CombineBackwardParams &p, int num_sms, cudaStream_t s)
{
    (void)num_sms;
    combine_backward_kernel<<<p.T, kCombineBwdThreads, 0, s>>>(p);
    return cudaGetLastError();
}

}  // namespace ep
