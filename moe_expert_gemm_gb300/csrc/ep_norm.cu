// The residual's addition and the root-mean-square norm in front of a layer, and its gradient.
//
//   h = x + residual,  r = 1 / sqrt(mean(h^2) + eps),  v = h * r * weight
//   g = dy * weight,   dh = r * (g - h * r^2 * mean(g * h)) + dsum,   dweight = sum_t dy * h * r
//
// Both are bound by their rows' bytes. A row stays in the registers of one thread block (or of
// one warp, where it is short) from its load to its stores: it is read once, and may be
// overwritten in place.
#include "ep_internal.h"
#include "ep_ptx.cuh"
#include "ep_rows.cuh"

namespace ep {

using namespace rows;

namespace {

constexpr int kPieces = 2;      // of a thread
constexpr int kMaxWarps = 32;   // 2 pieces of 8 by 1024 threads: EP_MAX_NORM_HIDDEN values
static_assert(kPieces * kPiece * 32 * kMaxWarps == EP_MAX_NORM_HIDDEN, "a row in a block");
constexpr int kPartBlocks = 320;  // that leave partial sums of dweight, at most

// Sum over the block of two values, the same order for every thread.
__device__ __forceinline__ float2 block_sum(float a, float b, float2 *part)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
#pragma unroll
    for (int o = 16; o; o >>= 1) {
        a += __shfl_xor_sync(0xffffffffu, a, o);
        b += __shfl_xor_sync(0xffffffffu, b, o);
    }
    if (lane == 0)
        part[warp] = make_float2(a, b);
    __syncthreads();
    float2 v = lane < warps ? part[lane] : make_float2(0.f, 0.f);
#pragma unroll
    for (int o = 16; o; o >>= 1) {
        v.x += __shfl_xor_sync(0xffffffffu, v.x, o);
        v.y += __shfl_xor_sync(0xffffffffu, v.y, o);
    }
    __syncthreads();
    return v;
}

}  // namespace

template <bool VEC>
__global__ void __launch_bounds__(32 * kMaxWarps) norm_kernel(const NormParams p)
{
    __shared__ float2 part[kMaxWarps];
    griddep_wait();
    griddep_launch_dependents();
    const int n = p.hidden;
    for (int64_t t = blockIdx.x; t < p.T; t += gridDim.x) {
        float h[kPieces][kPiece];
        float squares = 0.f;
#pragma unroll
        for (int i = 0; i < kPieces; ++i) {
            const int c = (i * blockDim.x + threadIdx.x) * kPiece;
#pragma unroll
            for (int j = 0; j < kPiece; ++j)
                h[i][j] = 0.f;
            if (c < n) {
                load_piece<VEC>(p.x + t * p.x_stride * 2, true, c, n, h[i]);
                if (p.residual) {
                    float res[kPiece];
                    load_piece<VEC>(p.residual + t * p.residual_stride * (p.residual_bf16 ? 2 : 4),
                                    p.residual_bf16, c, n, res);
#pragma unroll
                    for (int j = 0; j < kPiece; ++j)
                        h[i][j] += res[j];
                }
            }
#pragma unroll
            for (int j = 0; j < kPiece; ++j)
                squares = fmaf(h[i][j], h[i][j], squares);
        }
        // (the barriers in here also stand between the row's loads and its stores in place)
        const float r = rsqrtf(block_sum(squares, 0.f, part).x / n + p.eps);
#pragma unroll
        for (int i = 0; i < kPieces; ++i) {
            const int c = (i * blockDim.x + threadIdx.x) * kPiece;
            if (c < n && p.sum)
                store_piece<VEC>(p.sum + t * p.sum_stride * (p.residual_bf16 ? 2 : 4), p.residual_bf16, c,
                                 n, h[i]);
            float w[kPiece], v[kPiece] = {};
            if (c < n) {
                load_piece<VEC>(p.weight, p.weight_bf16, c, n, w);
#pragma unroll
                for (int j = 0; j < kPiece; ++j)
                    v[j] = h[i][j] * r * w[j];
                if (p.y)
                    store_piece<VEC>(p.y + t * p.y_stride * 2, true, c, n, v);
            }
            if (p.q)
                store_e4m3<VEC>(p.q + t * n, p.q_scales + t * ((n + 127) / 128), c, n, v);
        }
    }
}

template <bool VEC>
__global__ void __launch_bounds__(32 * kMaxWarps) norm_backward_kernel(const NormBackwardParams p)
{
    __shared__ float2 part[kMaxWarps];
    griddep_wait();
    griddep_launch_dependents();
    const int n = p.hidden, hb = p.h_bf16 ? 2 : 4;
    float dw[kPieces][kPiece] = {};
    for (int64_t t = blockIdx.x; t < p.T; t += gridDim.x) {
        float h[kPieces][kPiece] = {}, dy[kPieces][kPiece] = {}, g[kPieces][kPiece] = {};
        float squares = 0.f, dot = 0.f;
#pragma unroll
        for (int i = 0; i < kPieces; ++i) {
            const int c = (i * blockDim.x + threadIdx.x) * kPiece;
            if (c < n) {
                load_piece<VEC>(p.h + t * p.h_stride * hb, p.h_bf16, c, n, h[i]);
                load_piece<VEC>(p.dy + t * p.dy_stride * 2, true, c, n, dy[i]);
                load_piece<VEC>(p.weight, p.weight_bf16, c, n, g[i]);
            }
#pragma unroll
            for (int j = 0; j < kPiece; ++j) {
                g[i][j] *= dy[i][j];
                squares = fmaf(h[i][j], h[i][j], squares);
                dot = fmaf(g[i][j], h[i][j], dot);
            }
        }
        const float2 sums = block_sum(squares, dot, part);
        const float r = rsqrtf(sums.x / n + p.eps), back = r * r * (sums.y / n);
#pragma unroll
        for (int i = 0; i < kPieces; ++i) {
            const int c = (i * blockDim.x + threadIdx.x) * kPiece;
            float d[kPiece], ds[kPiece] = {};
            if (c < n && p.dsum)
                load_piece<VEC>(p.dsum + t * p.dsum_stride * hb, p.h_bf16, c, n, ds);
#pragma unroll
            for (int j = 0; j < kPiece; ++j) {
                d[j] = fmaf(r, g[i][j] - h[i][j] * back, ds[j]);
                dw[i][j] = fmaf(dy[i][j], h[i][j] * r, dw[i][j]);
            }
            if (c < n && p.dh)
                store_piece<VEC>(p.dh + t * p.dh_stride * hb, p.h_bf16, c, n, d);
            if (c < n && p.dx)
                store_piece<VEC>(p.dx + t * p.dx_stride * 2, true, c, n, d);
        }
    }
    if (p.dweight) {
        float *mine = p.parts + static_cast<int64_t>(blockIdx.x) * n;
#pragma unroll
        for (int i = 0; i < kPieces; ++i)
#pragma unroll
            for (int j = 0; j < kPiece; ++j) {
                const int c = (i * blockDim.x + threadIdx.x) * kPiece + j;
                if (c < n)
                    mine[c] = dw[i][j];
            }
    }
}

// dweight from the blocks' sums, in block order.
__global__ void __launch_bounds__(128) norm_weight_kernel(const NormBackwardParams p, int blocks)
{
    griddep_wait();
    griddep_launch_dependents();
    const int c = blockIdx.x * blockDim.x + threadIdx.x;
    if (c >= p.hidden)
        return;
    float sum = 0.f;
    for (int b = 0; b < blocks; ++b)
        sum += p.parts[static_cast<int64_t>(b) * p.hidden + c];
    p.dweight[c] = sum;
}

namespace {

// Rows of a stride that start and go on in whole pieces of `bytes`-byte values.
bool whole_pieces(const void *base, int64_t stride, int bytes)
{
    return !base || (reinterpret_cast<uintptr_t>(base) % 16 == 0 && stride * bytes % 16 == 0);
}

int threads_for(int hidden)
{
    const int per_thread = kPieces * kPiece;
    return ((hidden + per_thread - 1) / per_thread + 31) / 32 * 32;
}

}  // namespace

cudaError_t launch_norm(const NormParams &p, int num_sms, cudaStream_t s)
{
    const int rb = p.residual_bf16 ? 2 : 4;
    const bool vec = p.hidden % kPiece == 0 && whole_pieces(p.x, p.x_stride, 2) &&
                     whole_pieces(p.residual, p.residual_stride, rb) && whole_pieces(p.sum, p.sum_stride, rb) &&
                     whole_pieces(p.y, p.y_stride, 2) && whole_pieces(p.weight, 0, 4) &&
                     reinterpret_cast<uintptr_t>(p.q) % 8 == 0;
    const int most = 16 * num_sms;
    const unsigned grid = p.T < most ? p.T : most;
    return launch_behind(vec ? norm_kernel<true> : norm_kernel<false>, grid, threads_for(p.hidden), 0, s, p);
}

int64_t norm_backward_workspace_bytes(int T, int hidden)
{
    return static_cast<int64_t>(T < kPartBlocks ? T : kPartBlocks) * hidden * 4;
}

cudaError_t launch_norm_backward(const NormBackwardParams &p, int num_sms, cudaStream_t s)
{
    const int hb = p.h_bf16 ? 2 : 4;
    const bool vec = p.hidden % kPiece == 0 && whole_pieces(p.h, p.h_stride, hb) &&
                     whole_pieces(p.dy, p.dy_stride, 2) && whole_pieces(p.dsum, p.dsum_stride, hb) &&
                     whole_pieces(p.dh, p.dh_stride, hb) && whole_pieces(p.dx, p.dx_stride, 2) &&
                     whole_pieces(p.weight, 0, 4);
    const int most = 2 * num_sms < kPartBlocks ? 2 * num_sms : kPartBlocks;
    const int grid = p.T < most ? p.T : most;
    cudaError_t e = launch_behind(vec ? norm_backward_kernel<true> : norm_backward_kernel<false>, grid,
                                  threads_for(p.hidden), 0, s, p);
    if (e == cudaSuccess && p.dweight)
        e = launch_behind(norm_weight_kernel, (p.hidden + 127) / 128, 128, 0, s, p, grid);
    return e;
}

}  // namespace ep
