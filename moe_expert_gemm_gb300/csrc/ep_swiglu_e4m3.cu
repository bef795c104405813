// The gated activation between two blockwise fp8 products: SiLU(gate) * up as e4m3 rows with a
// scale for each 128 columns. Bound by its rows' bytes, 4 read and 1 written a value. A thread
// takes eight columns, a half warp a scale's 128, whose largest magnitude it finds by shuffles.
#include "ep_internal.h"
#include "ep_ptx.cuh"
#include "ep_rows.cuh"

namespace ep {

using namespace rows;

namespace {

constexpr int kThreads = 256;
constexpr int kRowsAhead = 4;  // of a thread, under way at once

}  // namespace

// A block takes tiles of kRowsAhead * (256 / width) rows, `width` threads (whole half warps) to a
// row.
__global__ void __launch_bounds__(kThreads) swiglu_e4m3_kernel(const SwigluE4m3Params p, int width)
{
    griddep_wait();
    griddep_launch_dependents();
    int64_t m_total = __ldg(p.expert_offsets + p.El);
    m_total = m_total < 0 ? 0 : (m_total > p.max_rows ? p.max_rows : m_total);
    const int pieces = p.inter / kPiece, groups = (pieces + kGroupPieces - 1) / kGroupPieces;
    const int x = threadIdx.x % width, y = threadIdx.x / width, rows_at_once = kThreads / width;
    const int rows = rows_at_once * kRowsAhead;
    for (int64_t m0 = static_cast<int64_t>(blockIdx.x) * rows; m0 < m_total; m0 += static_cast<int64_t>(gridDim.x) * rows) {
        for (int c0 = 0; c0 < pieces; c0 += width) {
            const int c = (c0 + x) * kPiece;
            uint4 gate[kRowsAhead], up[kRowsAhead];
#pragma unroll
            for (int i = 0; i < kRowsAhead; ++i) {
                const int64_t m = m0 + i * rows_at_once + y;
                gate[i] = up[i] = make_uint4(0, 0, 0, 0);
                if (m < m_total && c < p.inter) {
                    const uint8_t *row = p.G + m * p.inter * 4 + c * 2;
                    gate[i] = __ldcs(reinterpret_cast<const uint4 *>(row));
                    up[i] = __ldcs(reinterpret_cast<const uint4 *>(row + p.inter * 2));
                }
            }
#pragma unroll
            for (int i = 0; i < kRowsAhead; ++i) {
                const int64_t m = m0 + i * rows_at_once + y;
                float v[kPiece], u[kPiece];
                unpack(gate[i], v);
                unpack(up[i], u);
#pragma unroll
                for (int j = 0; j < kPiece; ++j)
                    v[j] = silu_times(v[j], u[j]);
                store_e4m3<true>(p.q + m * p.inter, p.q_scales + m * groups, m < m_total ? c : p.inter, p.inter, v);
            }
        }
    }
}

cudaError_t launch_swiglu_e4m3(const SwigluE4m3Params &p, int num_sms, cudaStream_t s)
{
    int width = kGroupPieces;
    while (width < kThreads && width * kPiece < p.inter)
        width *= 2;
    const int64_t rows = kThreads / width * kRowsAhead;
    const int64_t blocks = (p.max_rows + rows - 1) / rows, most = 6ll * num_sms;
    return launch_behind(swiglu_e4m3_kernel, static_cast<unsigned>(blocks < most ? blocks : most), kThreads, 0, s, p,
                         width);
}

}  // namespace ep
