// The gated activation between two blockwise fp8 products: SiLU(gate) * up as e4m3 rows with a
// scale for each 128 columns. Bound by its rows' bytes, 4 read and 1 written a value. A thread
// takes eight columns, a half warp a scale's 128, whose largest magnitude it finds by shuffles.
// Measured: 65536 x 2048 107 us, 6.3 TB/s, 93 % of the copy bandwidth.
#include <climits>

#include "ep_internal.h"
#include "ep_ptx.cuh"
#include "ep_rows.cuh"

namespace ep {

using namespace rows;

namespace {

constexpr int kThreads = 256;
constexpr int kRowsAhead = 4;  // of a thread, under way at once (65536 x 2048: 106 us; 2: 139)

// x / (1 + e^-x) of two bf16 values. e^-x = 2^t * 2^d with t + d = -x log2 e: t is -x times
// the first 16 bits of log2 e, exact as x has 8, and 2^d = 1 + d ln 2 to within (88 * 2^-17 ln 2)^2 / 2
// = 1.1e-7. With the errors of ex2 (2^-22) and rcp (2^-23) and three roundings a value is off by at
// most 12 half steps. The quotient is of quarters: 1 + e^-x may pass 2^126, where rcp gives 0. (0 where
// e^-x leaves fp32, for gates of -89 and less, where the value is under 2^-121.)
__device__ __forceinline__ Two silu2(Two x)
{
    constexpr float first = 1.44268798828125f, rest_ln2 = 4.8884952e-6f;
    const Two quarter = two(0.25f, 0.25f);
    float t0, t1, e0, e1;
    split(mul2(x, two(-first, -first)), t0, t1);
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e0) : "f"(t0));
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e1) : "f"(t1));
    const Two to_d = fma2(x, two(-0.25f * rest_ln2, -0.25f * rest_ln2), quarter);  // 2^d / 4
    float s0, s1;
    split(fma2(two(e0, e1), to_d, quarter), s0, s1);
    asm("rcp.approx.ftz.f32 %0, %0;" : "+f"(s0));
    asm("rcp.approx.ftz.f32 %0, %0;" : "+f"(s1));
    return mul2(mul2(x, quarter), two(s0, s1));
}

}  // namespace

// A block takes tiles of kRowsAhead * (256 / width) rows by the pieces of `width` threads (whole half
// warps), which take turns through a row's chunks. ONE: there is one (65536 x 2048 107 us, in the other
// form 108).
template <bool ONE>
__global__ void __launch_bounds__(kThreads) swiglu_e4m3_kernel(const SwigluE4m3Params p, int width)
{
    griddep_wait();
    griddep_launch_dependents();
    // (an ordinary load: the kernel before may write the offsets while this one is already there, and a load
    // through the read-only path need not stay behind the wait)
    int64_t m_total = p.expert_offsets[p.El];
    m_total = m_total < 0 ? 0 : (m_total > p.max_rows ? p.max_rows : m_total);
    const int pieces = p.inter / kPiece, groups = (pieces + kGroupPieces - 1) / kGroupPieces;
    const int x = threadIdx.x % width, y = threadIdx.x / width, rows_at_once = kThreads / width;
    const int rows = rows_at_once * kRowsAhead;
    const int chunks = ONE ? 1 : (pieces + width - 1) / width;
    const int64_t row_step = static_cast<int64_t>(gridDim.x / chunks) * rows;
    const int chunk_step = gridDim.x % chunks;
    int chunk = blockIdx.x % chunks;
    for (int64_t m0 = static_cast<int64_t>(blockIdx.x / chunks) * rows; m0 < m_total;) {
        const int c = (chunk * width + x) * kPiece;
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
            const Piece g = unpack(gate[i]), u = unpack(up[i]);
            Piece v;
#pragma unroll
            for (int j = 0; j < 4; ++j)
                v.v[j] = mul2(silu2(g.v[j]), u.v[j]);
            const int at = m < m_total ? c : p.inter;
            const uint2 codes = quantise(v, p.q_scales + m * groups, at, p.inter);
            if (at < p.inter)
                *reinterpret_cast<uint2 *>(p.q + m * p.inter + c) = codes;
        }
        m0 += row_step;
        chunk += chunk_step;
        if (chunk >= chunks) {
            chunk -= chunks;
            m0 += rows;
        }
    }
}

cudaError_t launch_swiglu_e4m3(const SwigluE4m3Params &p, int num_sms, cudaStream_t s)
{
    // Threads to a row: of 16, 32 .. 256 those of which a row leaves the fewest idle, the most of them
    // (30000 x 1032: 16 threads 29.6 us, 64 34.7, 256 42.9; 65536 x 2048: 256 threads 108, 16 111).
    const int pieces = p.inter / kPiece;
    int width = kGroupPieces, slots = INT_MAX;
    for (int w = kGroupPieces; w <= kThreads; w *= 2)
        if (const int all = (pieces + w - 1) / w * w; all <= slots)
            width = w, slots = all;
    const int64_t rows = kThreads / width * kRowsAhead;
    // (as many blocks as are resident: with 6 an SM 65536 x 2048 took 118 us)
    const int64_t tiles = (p.max_rows + rows - 1) / rows * (slots / width), most = 4ll * num_sms;
    const unsigned blocks = static_cast<unsigned>(tiles < most ? tiles : most);
    return launch_behind(slots == width ? swiglu_e4m3_kernel<true> : swiglu_e4m3_kernel<false>, blocks, kThreads, 0, s, p, width);
}

}  // namespace ep
