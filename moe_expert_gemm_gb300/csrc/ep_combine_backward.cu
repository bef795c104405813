// Gradient of the gate-weighted combine out[t] = sum_j g[t, j] * row(t, j):
//   dgates[t, j] = <dout[t], row(t, j)>,   drow(t, j) = g[t, j] * dout[t].
// HBM-bound: every row is read once and its gradient written once; a token's dout comes
// from HBM once and from the L1 for its other rows, which are handled side by side. Measured:
// 8192 tokens of 8 rows of 7168, both gradients, 292 us, 6.84 TB/s.
// A warp takes a row; kUnroll 16-byte pieces of the row and of dout a lane are under way at
// once. Where there are fewer rows than warps to keep the memory busy, a block of eight
// warps takes a row and joins their sums in warp order.
#include <cuda_bf16.h>

#include "ep_internal.h"
#include "ep_ptx.cuh"

namespace ep {

constexpr int kCombineBwdWarps = 8;
constexpr int kUnroll = 4;

__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi)
{
    const __nv_bfloat162 b = __float22bfloat162_rn(make_float2(lo, hi));
    return *reinterpret_cast<const uint32_t *>(&b);
}

// Pieces first, first + step, ... of one row; returns the lane's part of <dout, row>.
template <bool DGATES, bool DROWS>
__device__ __forceinline__ float row_pieces(const uint4 *dout, const uint4 *row, uint4 *drow, float g,
                                            int first, int step, int pieces)
{
    float sum = 0.f;
    for (int v0 = first; v0 < pieces; v0 += kUnroll * step) {
        uint4 d[kUnroll], r[kUnroll];
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            const int v = v0 + u * step;
            if (v < pieces) {
                d[u] = dout[v];
                if (DGATES)
                    r[u] = __ldcs(row + v);
            }
        }
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            const int v = v0 + u * step;
            if (v >= pieces)
                break;
            const uint32_t dw[4] = {d[u].x, d[u].y, d[u].z, d[u].w};
            if (DGATES) {
                const uint32_t rw[4] = {r[u].x, r[u].y, r[u].z, r[u].w};
#pragma unroll
                for (int h = 0; h < 4; ++h) {
                    sum = fmaf(bf16_lo(dw[h]), bf16_lo(rw[h]), sum);
                    sum = fmaf(bf16_hi(dw[h]), bf16_hi(rw[h]), sum);
                }
            }
            if (DROWS) {
                uint32_t o[4];
#pragma unroll
                for (int h = 0; h < 4; ++h)
                    o[h] = pack_bf16(g * bf16_lo(dw[h]), g * bf16_hi(dw[h]));
                __stcs(drow + v, make_uint4(o[0], o[1], o[2], o[3]));
            }
        }
    }
    return sum;
}

// WPR: warps of a row, 1 or all of the block.
template <bool DGATES, bool DROWS, int WPR>
__global__ void __launch_bounds__(32 * kCombineBwdWarps)
    combine_backward_kernel(const CombineBackwardParams p)
{
    griddep_wait();
    griddep_launch_dependents();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int pieces = p.N / 8;
    const int64_t rows = static_cast<int64_t>(p.T) * p.top_k;
    const int64_t stride = static_cast<int64_t>(gridDim.x) * (kCombineBwdWarps / WPR);
    for (int64_t row = static_cast<int64_t>(blockIdx.x) * (kCombineBwdWarps / WPR) + (WPR == 1 ? warp : 0);
         row < rows; row += stride) {
        const int64_t t = row / p.top_k;
        const float g = DROWS ? p.gates[row] : 0.f;
        float sum = row_pieces<DGATES, DROWS>(
            reinterpret_cast<const uint4 *>(p.dout) + t * pieces,
            reinterpret_cast<const uint4 *>(p.recv_buf) + row * pieces,
            reinterpret_cast<uint4 *>(p.drows) + row * pieces, g, WPR == 1 ? lane : threadIdx.x,
            32 * WPR, pieces);
        if constexpr (DGATES) {
#pragma unroll
            for (int o = 16; o; o >>= 1)
                sum += __shfl_xor_sync(0xffffffffu, sum, o);
            if constexpr (WPR == 1) {
                if (lane == 0)
                    p.dgates[row] = sum;
            } else {
                __shared__ float part[WPR];
                if (lane == 0)
                    part[warp] = sum;
                __syncthreads();
                if (threadIdx.x == 0) {
                    float all = 0.f;
                    for (int w = 0; w < WPR; ++w)
                        all += part[w];
                    p.dgates[row] = all;
                }
                __syncthreads();
            }
        }
    }
}

template <bool DGATES, bool DROWS>
static cudaError_t launch_form(const CombineBackwardParams &p, int num_sms, cudaStream_t s)
{
    const int64_t rows = static_cast<int64_t>(p.T) * p.top_k;
    // A block to a row while the rows are few and its threads find work: at N = 7168 and
    // 1024 / 2048 / 4096 rows 6.2 / 11.2 / 21.5 us against 8.9 / 12.8 / 21.4 of a warp to a
    // row, at N = 2048 and 512 / 1024 rows 2.3 / 3.4 against 2.7 / 2.7.
    const int pieces = p.N / 8, threads = 32 * kCombineBwdWarps;
    if ((rows <= 16 * num_sms && pieces >= 2 * threads) || (rows <= 2 * num_sms && pieces >= threads)) {
        return launch_behind(combine_backward_kernel<DGATES, DROWS, kCombineBwdWarps>,
                             static_cast<unsigned>(rows), 32 * kCombineBwdWarps, 0, s, p);
    } else {
        const int64_t blocks = (rows + kCombineBwdWarps - 1) / kCombineBwdWarps;
        const int64_t most = static_cast<int64_t>(num_sms) * 1024;
        return launch_behind(combine_backward_kernel<DGATES, DROWS, 1>,
                             static_cast<unsigned>(blocks < most ? blocks : most),
                             32 * kCombineBwdWarps, 0, s, p);
    }
}

cudaError_t launch_combine_backward(const CombineBackwardParams &p, int num_sms, cudaStream_t s)
{
    if (p.dgates && p.drows)
        return launch_form<true, true>(p, num_sms, s);
    return p.dgates ? launch_form<true, false>(p, num_sms, s) : launch_form<false, true>(p, num_sms, s);
}

}  // namespace ep
