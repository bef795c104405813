// The gated activation between two blockwise fp8 products: SiLU(gate) * up as e4m3 rows with a
// scale for each 128 columns. Bound by its rows' bytes, 4 read and 1 written a value. A thread
// takes eight columns, a half warp a scale's 128, whose largest magnitude it finds by shuffles.
#include "ep_internal.h"
#include "ep_ptx.cuh"
#include "ep_rows.cuh"

namespace ep {

using namespace rows;

constexpr int kSwigluE4m3Threads = 256;

__global__ void __launch_bounds__(kSwigluE4m3Threads) swiglu_e4m3_kernel(const SwigluE4m3Params p)
{
    griddep_wait();
    griddep_launch_dependents();
    int64_t m_total = __ldg(p.expert_offsets + p.El);
    m_total = m_total < 0 ? 0 : (m_total > p.max_rows ? p.max_rows : m_total);
    const int pieces = p.inter / kPiece, groups = (pieces + kGroupPieces - 1) / kGroupPieces;
    // half warps count through all rows' groups
    const int64_t all = m_total * groups;
    const int lane = threadIdx.x % kGroupPieces;
    const int64_t step = static_cast<int64_t>(gridDim.x) * (kSwigluE4m3Threads / kGroupPieces);
    int64_t at = static_cast<int64_t>(blockIdx.x) * (kSwigluE4m3Threads / kGroupPieces) + threadIdx.x / kGroupPieces;
    // (both halves of a warp stay for its shuffles)
    for (; at - at % 2 < all; at += step) {
        const int64_t m = at / groups;
        const int c = (static_cast<int>(at - m * groups) * kGroupPieces + lane) * kPiece;
        const bool there = at < all && c < p.inter;
        float v[kPiece] = {};
        if (there) {
            float gate[kPiece], up[kPiece];
            load_piece<true>(p.G + m * p.inter * 4, true, c, p.inter, gate);
            load_piece<true>(p.G + (m * 2 + 1) * p.inter * 2, true, c, p.inter, up);
#pragma unroll
            for (int j = 0; j < kPiece; ++j)
                v[j] = silu_f32(gate[j]) * up[j];
        }
        store_e4m3<true>(p.q + m * p.inter, p.q_scales + m * groups, there ? c : p.inter, p.inter, v);
    }
}

cudaError_t launch_swiglu_e4m3(const SwigluE4m3Params &p, int num_sms, cudaStream_t s)
{
    const int64_t groups = (p.inter + 127) / 128;
    const int64_t blocks = (p.max_rows * groups * kGroupPieces + kSwigluE4m3Threads - 1) / kSwigluE4m3Threads;
    const int64_t most = 8ll * num_sms;
    return launch_behind(swiglu_e4m3_kernel, static_cast<unsigned>(blocks < most ? blocks : most),
                         kSwigluE4m3Threads, 0, s, p);
}

}  // namespace ep
