// The residual's addition and the root-mean-square norm in front of a layer, and its gradient.
//
//   h = x + residual,  r = 1 / sqrt(mean(h^2) + eps),  v = h * r * weight
//   g = dy * weight,   dh = r * (g - h * r^2 * mean(g * h)) + dsum,   dweight = sum_t dy * h * r
//
// Both are bound by their rows' bytes. A row stays in one thread block from its load to its
// stores: it is read once, and may be overwritten in place. Rows of whole 16-byte pieces are
// copied to shared memory some rows ahead (cp.async), every thread the pieces that it will use
// itself, so that nobody waits for anybody but in the row's sums; the weight stays in
// registers. Rows of any other alignment go to shared memory and back in the widest pieces
// that they allow, consecutive threads consecutive pieces.
#include "ep_internal.h"
#include "ep_ptx.cuh"
#include "ep_rows.cuh"

namespace ep {

using namespace rows;

namespace {

constexpr int kPieces = 2;      // of a thread, at most
constexpr int kMaxWarps = 32;   // 2 pieces of 8 by 1024 threads: EP_MAX_NORM_HIDDEN values
static_assert(kPieces * kPiece * 32 * kMaxWarps == EP_MAX_NORM_HIDDEN, "a row in a block");
constexpr int kPartBlocks = 640;       // that leave partial sums of dweight, at most
constexpr int kSmemOfSm = 216 * 1024;  // for rows under way
constexpr int kMaxPerSm = 8;           // blocks

// The widest pieces that the rows of a call's tensors allow.
struct RowUnits {
    int of[5];
};

// Sum over the block of two values, the same order for every thread. `part` is not used again
// before another barrier of the block (two buffers that take turns).
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
    return v;
}

__device__ __forceinline__ void copy_async(uint32_t smem, const void *src)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem), "l"(src) : "memory");
}

__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }

template <int N>
__device__ __forceinline__ void copy_wait()
{
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// A thread's pieces of one row of a tensor: 16 bytes of a piece lie blockDim.x apart.
__device__ __forceinline__ void copy_piece(uint8_t *to, const uint8_t *row, bool bf16, int c)
{
    const uint32_t dst = smem_u32(to) + threadIdx.x * 16;
    if (bf16) {
        copy_async(dst, row + c * 2);
    } else {
        copy_async(dst, row + c * 4);
        copy_async(dst + blockDim.x * 16, row + c * 4 + 16);
    }
}

__device__ __forceinline__ void read_piece(const uint8_t *from, bool bf16, float (&f)[kPiece])
{
    const uint4 *p = reinterpret_cast<const uint4 *>(from) + threadIdx.x;
    if (bf16) {
        unpack(*p, f);
    } else {
        const float4 a = *reinterpret_cast<const float4 *>(p);
        const float4 b = *reinterpret_cast<const float4 *>(p + blockDim.x);
        f[0] = a.x, f[1] = a.y, f[2] = a.z, f[3] = a.w;
        f[4] = b.x, f[5] = b.y, f[6] = b.z, f[7] = b.w;
    }
}

}  // namespace

// `bytes` of a row between global and shared memory, in units of `unit` bytes that both are
// aligned to (a divisor of 16); what is left over byte by byte. ASYNC: to shared memory by
// cp.async, which takes units of 4 and more.
template <bool ASYNC, typename U>
__device__ __forceinline__ void copy_units(uint8_t *to, const uint8_t *from, int bytes)
{
    constexpr int kUnit = sizeof(U);
#pragma unroll 4
    for (int i = threadIdx.x; i < bytes / kUnit; i += blockDim.x) {
        if constexpr (ASYNC && kUnit >= 4)
            asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(smem_u32(to) + i * kUnit),
                         "l"(from + i * kUnit), "n"(kUnit)
                         : "memory");
        else
            reinterpret_cast<U *>(to)[i] = reinterpret_cast<const U *>(from)[i];
    }
}

template <bool ASYNC>
__device__ __forceinline__ void copy_row(uint8_t *to, const uint8_t *from, int bytes, int unit)
{
    switch (unit) {
    case 16:
        copy_units<ASYNC, uint4>(to, from, bytes);
        break;
    case 8:
        copy_units<ASYNC, uint2>(to, from, bytes);
        break;
    case 4:
        copy_units<ASYNC, uint32_t>(to, from, bytes);
        break;
    case 2:
        copy_units<ASYNC, uint16_t>(to, from, bytes);
        break;
    default:
        copy_units<ASYNC, uint8_t>(to, from, bytes);
    }
    for (int i = bytes / unit * unit + threadIdx.x; i < bytes; i += blockDim.x)
        to[i] = from[i];
}

// Rows of any alignment, by way of shared memory: x (then y) and the residual (then sum), each
// padded to whole pieces, in two buffers that take turns where they fit; q. A thread overwrites
// only the pieces that it alone has read.
__global__ void __launch_bounds__(32 * kMaxWarps) norm_any_kernel(const NormParams p, const RowUnits units,
                                                                 int buffers)
{
    extern __shared__ __align__(16) uint8_t row[];
    __shared__ float2 part[2][kMaxWarps];
    int turn = 0;
    const int n = p.hidden, rb = p.residual_bf16 ? 2 : 4, padded = (n + kPiece - 1) / kPiece * kPiece;
    const int bytes = padded * (p.residual || p.sum ? 2 + rb : 2);
    uint8_t *const q = row + buffers * bytes;
    griddep_wait();
    griddep_launch_dependents();
    auto ask = [&](int64_t t, int buffer) {
        if (t < p.T) {
            uint8_t *const x = row + buffer * bytes;
            copy_row<true>(x, p.x + t * p.x_stride * 2, n * 2, units.of[0]);
            if (p.residual)
                copy_row<true>(x + padded * 2, p.residual + t * p.residual_stride * rb, n * rb, units.of[1]);
        }
        copy_commit();
    };
    if (buffers > 1)
        ask(blockIdx.x, 0);
    int buffer = 0;
    for (int64_t t = blockIdx.x; t < p.T; t += gridDim.x) {
        uint8_t *const x = row + buffer * bytes, *const res = x + padded * 2;
        if (buffers > 1) {
            ask(t + gridDim.x, buffer ^ 1);
            copy_wait<1>();
            buffer ^= 1;
        } else {
            ask(t, 0);
            copy_wait<0>();
        }
        __syncthreads();
        float h[kPieces][kPiece] = {};
        float squares = 0.f;
#pragma unroll
        for (int i = 0; i < kPieces; ++i) {
            const int c = (i * blockDim.x + threadIdx.x) * kPiece;
            if (c < n) {
                load_piece<true>(x, true, c, n, h[i]);
                float r[kPiece] = {};
                if (p.residual)
                    load_piece<true>(res, p.residual_bf16, c, n, r);
#pragma unroll
                for (int j = 0; j < kPiece; ++j)
                    h[i][j] = c + j < n ? h[i][j] + r[j] : 0.f;
            }
#pragma unroll
            for (int j = 0; j < kPiece; ++j)
                squares = fmaf(h[i][j], h[i][j], squares);
        }
        const float r = rsqrtf(block_sum(squares, 0.f, part[turn ^= 1]).x / n + p.eps);
#pragma unroll
        for (int i = 0; i < kPieces; ++i) {
            const int c = (i * blockDim.x + threadIdx.x) * kPiece;
            float v[kPiece] = {};
            if (c < n) {
                if (p.sum)
                    store_piece<true>(res, p.residual_bf16, c, n, h[i]);
                load_piece<false>(p.weight, p.weight_bf16, c, n, v);
#pragma unroll
                for (int j = 0; j < kPiece; ++j)
                    v[j] = h[i][j] * r * v[j];
                if (p.y)
                    store_piece<true>(x, true, c, n, v);
            }
            if (p.q)
                store_e4m3<true>(q, p.q_scales + t * ((n + 127) / 128), c, n, v);
        }
        __syncthreads();
        if (p.sum)
            copy_row<false>(p.sum + t * p.sum_stride * rb, res, n * rb, units.of[2]);
        if (p.y)
            copy_row<false>(p.y + t * p.y_stride * 2, x, n * 2, units.of[3]);
        if (p.q)
            copy_row<false>(p.q + t * n, q, n, units.of[4]);
        __syncthreads();
    }
}

// The same for the gradient: h (then dh), dy (then dx), dsum.
__global__ void __launch_bounds__(32 * kMaxWarps) norm_backward_any_kernel(const NormBackwardParams p,
                                                                            const RowUnits units, int buffers)
{
    extern __shared__ __align__(16) uint8_t row[];
    __shared__ float2 part[2][kMaxWarps];
    int turn = 0;
    const int n = p.hidden, hb = p.h_bf16 ? 2 : 4, padded = (n + kPiece - 1) / kPiece * kPiece;
    const int bytes = padded * (2 + hb * (p.dsum ? 2 : 1));
    griddep_wait();
    griddep_launch_dependents();
    auto ask = [&](int64_t t, int buffer) {
        if (t < p.T) {
            uint8_t *const to = row + buffer * bytes;
            copy_row<true>(to, p.h + t * p.h_stride * hb, n * hb, units.of[0]);
            copy_row<true>(to + padded * hb, p.dy + t * p.dy_stride * 2, n * 2, units.of[1]);
            if (p.dsum)
                copy_row<true>(to + padded * (hb + 2), p.dsum + t * p.dsum_stride * hb, n * hb, units.of[2]);
        }
        copy_commit();
    };
    if (buffers > 1)
        ask(blockIdx.x, 0);
    int buffer = 0;
    float dw[kPieces][kPiece] = {};
    for (int64_t t = blockIdx.x; t < p.T; t += gridDim.x) {
        uint8_t *const h_row = row + buffer * bytes, *const dy_row = h_row + padded * hb;
        uint8_t *const dsum_row = dy_row + padded * 2;
        if (buffers > 1) {
            ask(t + gridDim.x, buffer ^ 1);
            copy_wait<1>();
            buffer ^= 1;
        } else {
            ask(t, 0);
            copy_wait<0>();
        }
        __syncthreads();
        float squares = 0.f, dot = 0.f;
#pragma unroll
        for (int i = 0; i < kPieces; ++i) {
            const int c = (i * blockDim.x + threadIdx.x) * kPiece;
            if (c >= n)
                break;
            float h[kPiece], dy[kPiece], w[kPiece];
            load_piece<true>(h_row, p.h_bf16, c, n, h);
            load_piece<true>(dy_row, true, c, n, dy);
            load_piece<false>(p.weight, p.weight_bf16, c, n, w);
#pragma unroll
            for (int j = 0; j < kPiece; ++j)
                if (c + j < n) {
                    squares = fmaf(h[j], h[j], squares);
                    dot = fmaf(dy[j] * w[j], h[j], dot);
                }
        }
        const float2 sums = block_sum(squares, dot, part[turn ^= 1]);
        const float r = rsqrtf(sums.x / n + p.eps), back = r * r * (sums.y / n);
#pragma unroll
        for (int i = 0; i < kPieces; ++i) {
            const int c = (i * blockDim.x + threadIdx.x) * kPiece;
            if (c >= n)
                break;
            float h[kPiece], dy[kPiece], w[kPiece], d[kPiece] = {};
            load_piece<true>(h_row, p.h_bf16, c, n, h);
            load_piece<true>(dy_row, true, c, n, dy);
            load_piece<false>(p.weight, p.weight_bf16, c, n, w);
            if (p.dsum)
                load_piece<true>(dsum_row, p.h_bf16, c, n, d);
#pragma unroll
            for (int j = 0; j < kPiece; ++j) {
                d[j] = fmaf(r, dy[j] * w[j] - h[j] * back, d[j]);
                if (c + j < n)
                    dw[i][j] = fmaf(dy[j], h[j] * r, dw[i][j]);
            }
            if (p.dh)
                store_piece<true>(h_row, p.h_bf16, c, n, d);
            if (p.dx)
                store_piece<true>(dy_row, true, c, n, d);
        }
        __syncthreads();
        if (p.dh)
            copy_row<false>(p.dh + t * p.dh_stride * hb, h_row, n * hb, units.of[3]);
        if (p.dx)
            copy_row<false>(p.dx + t * p.dx_stride * 2, dy_row, n * 2, units.of[4]);
        __syncthreads();
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

// Rows of whole aligned pieces. P: pieces of a thread, S: rows under way.
template <int P, int S>
__global__ void __launch_bounds__(32 * kMaxWarps) norm_kernel(const NormParams p)
{
    extern __shared__ __align__(16) uint8_t ring[];
    __shared__ float2 part[2][kMaxWarps];
    const int n = p.hidden, rb = p.residual_bf16 ? 2 : 4;
    // of a thread's piece: x, then the residual
    const int x_bytes = blockDim.x * 16, piece_bytes = x_bytes * (p.residual ? 1 + rb / 2 : 1);
    griddep_wait();
    griddep_launch_dependents();
    auto ask = [&](int64_t t, int stage) {
        if (t < p.T) {
#pragma unroll
            for (int i = 0; i < P; ++i) {
                const int c = (i * blockDim.x + threadIdx.x) * kPiece;
                if (c >= n)
                    break;
                uint8_t *to = ring + (stage * P + i) * piece_bytes;
                copy_piece(to, p.x + t * p.x_stride * 2, true, c);
                if (p.residual)
                    copy_piece(to + x_bytes, p.residual + t * p.residual_stride * rb, p.residual_bf16, c);
            }
        }
        copy_commit();
    };
#pragma unroll
    for (int i = 0; i < S - 1; ++i)
        ask(blockIdx.x + static_cast<int64_t>(i) * gridDim.x, i);
    float w[P][kPiece] = {};
#pragma unroll
    for (int i = 0; i < P; ++i) {
        const int c = (i * blockDim.x + threadIdx.x) * kPiece;
        if (c < n)
            load_piece<true>(p.weight, p.weight_bf16, c, n, w[i]);
    }
    int stage = 0, turn = 0;
    for (int64_t t = blockIdx.x; t < p.T; t += gridDim.x) {
        ask(t + static_cast<int64_t>(S - 1) * gridDim.x, stage == 0 ? S - 1 : stage - 1);
        copy_wait<S - 1>();
        float h[P][kPiece] = {};
        float squares = 0.f;
#pragma unroll
        for (int i = 0; i < P; ++i) {
            const int c = (i * blockDim.x + threadIdx.x) * kPiece;
            const uint8_t *from = ring + (stage * P + i) * piece_bytes;
            if (c < n) {
                read_piece(from, true, h[i]);
                if (p.residual) {
                    float res[kPiece];
                    read_piece(from + x_bytes, p.residual_bf16, res);
#pragma unroll
                    for (int j = 0; j < kPiece; ++j)
                        h[i][j] += res[j];
                }
            }
#pragma unroll
            for (int j = 0; j < kPiece; ++j)
                squares = fmaf(h[i][j], h[i][j], squares);
        }
        const float r = rsqrtf(block_sum(squares, 0.f, part[turn ^= 1]).x / n + p.eps);
#pragma unroll
        for (int i = 0; i < P; ++i) {
            const int c = (i * blockDim.x + threadIdx.x) * kPiece;
            if (c < n && p.sum)
                store_piece<true>(p.sum + t * p.sum_stride * rb, p.residual_bf16, c, n, h[i]);
#pragma unroll
            for (int j = 0; j < kPiece; ++j)
                h[i][j] = h[i][j] * r * w[i][j];
            if (c < n && p.y)
                store_piece<true>(p.y + t * p.y_stride * 2, true, c, n, h[i]);
            if (p.q)
                store_e4m3<true>(p.q + t * n, p.q_scales + t * ((n + 127) / 128), c, n, h[i]);
        }
        stage = stage == S - 1 ? 0 : stage + 1;
    }
}

template <int P, int S>
__global__ void __launch_bounds__(32 * kMaxWarps) norm_backward_kernel(const NormBackwardParams p)
{
    extern __shared__ __align__(16) uint8_t ring[];
    __shared__ float2 part[2][kMaxWarps];
    const int n = p.hidden, hb = p.h_bf16 ? 2 : 4;
    // of a thread's piece: h, dy, then dsum
    const int dy_bytes = blockDim.x * 16, h_bytes = dy_bytes * (hb / 2);
    const int piece_bytes = dy_bytes + h_bytes * (p.dsum ? 2 : 1);
    griddep_wait();
    griddep_launch_dependents();
    auto ask = [&](int64_t t, int stage) {
        if (t < p.T) {
#pragma unroll
            for (int i = 0; i < P; ++i) {
                const int c = (i * blockDim.x + threadIdx.x) * kPiece;
                if (c >= n)
                    break;
                uint8_t *to = ring + (stage * P + i) * piece_bytes;
                copy_piece(to, p.h + t * p.h_stride * hb, p.h_bf16, c);
                copy_piece(to + h_bytes, p.dy + t * p.dy_stride * 2, true, c);
                if (p.dsum)
                    copy_piece(to + h_bytes + dy_bytes, p.dsum + t * p.dsum_stride * hb, p.h_bf16, c);
            }
        }
        copy_commit();
    };
#pragma unroll
    for (int i = 0; i < S - 1; ++i)
        ask(blockIdx.x + static_cast<int64_t>(i) * gridDim.x, i);
    float w[P][kPiece] = {}, dw[P][kPiece] = {};
#pragma unroll
    for (int i = 0; i < P; ++i) {
        const int c = (i * blockDim.x + threadIdx.x) * kPiece;
        if (c < n)
            load_piece<true>(p.weight, p.weight_bf16, c, n, w[i]);
    }
    int stage = 0, turn = 0;
    for (int64_t t = blockIdx.x; t < p.T; t += gridDim.x) {
        ask(t + static_cast<int64_t>(S - 1) * gridDim.x, stage == 0 ? S - 1 : stage - 1);
        copy_wait<S - 1>();
        float squares = 0.f, dot = 0.f;
#pragma unroll
        for (int i = 0; i < P; ++i) {
            const int c = (i * blockDim.x + threadIdx.x) * kPiece;
            const uint8_t *from = ring + (stage * P + i) * piece_bytes;
            if (c >= n)
                break;
            float h[kPiece], dy[kPiece];
            read_piece(from, p.h_bf16, h);
            read_piece(from + h_bytes, true, dy);
#pragma unroll
            for (int j = 0; j < kPiece; ++j) {
                squares = fmaf(h[j], h[j], squares);
                dot = fmaf(dy[j] * w[i][j], h[j], dot);
            }
        }
        const float2 sums = block_sum(squares, dot, part[turn ^= 1]);
        const float r = rsqrtf(sums.x / n + p.eps), back = r * r * (sums.y / n);
#pragma unroll
        for (int i = 0; i < P; ++i) {
            const int c = (i * blockDim.x + threadIdx.x) * kPiece;
            const uint8_t *from = ring + (stage * P + i) * piece_bytes;
            if (c >= n)
                break;
            float h[kPiece], dy[kPiece], d[kPiece] = {};
            read_piece(from, p.h_bf16, h);
            read_piece(from + h_bytes, true, dy);
            if (p.dsum)
                read_piece(from + h_bytes + dy_bytes, p.h_bf16, d);
#pragma unroll
            for (int j = 0; j < kPiece; ++j) {
                d[j] = fmaf(r, dy[j] * w[i][j] - h[j] * back, d[j]);
                dw[i][j] = fmaf(dy[j], h[j] * r, dw[i][j]);
            }
            if (p.dh)
                store_piece<true>(p.dh + t * p.dh_stride * hb, p.h_bf16, c, n, d);
            if (p.dx)
                store_piece<true>(p.dx + t * p.dx_stride * 2, true, c, n, d);
        }
        stage = stage == S - 1 ? 0 : stage + 1;
    }
    if (p.dweight) {
        uint8_t *mine = reinterpret_cast<uint8_t *>(p.parts + static_cast<int64_t>(blockIdx.x) * n);
#pragma unroll
        for (int i = 0; i < P; ++i) {
            const int c = (i * blockDim.x + threadIdx.x) * kPiece;
            if (c < n)
                store_piece<true>(mine, false, c, n, dw[i]);
        }
    }
}

// dweight from the blocks' sums: 32 threads to a column, each every 32nd block in turn, then
// the 32 in order.
__global__ void __launch_bounds__(1024) norm_weight_kernel(const NormBackwardParams p, int blocks)
{
    __shared__ float part[32][33];
    griddep_wait();
    griddep_launch_dependents();
    const int x = threadIdx.x & 31, y = threadIdx.x >> 5, c = blockIdx.x * 32 + x;
    float sum = 0.f;
    if (c < p.hidden) {
#pragma unroll 4
        for (int b = y; b < blocks; b += 32)
            sum += __ldcg(p.parts + static_cast<int64_t>(b) * p.hidden + c);
    }
    part[y][x] = sum;
    __syncthreads();
    // (a warp to a column now)
    sum = part[x][y];
#pragma unroll
    for (int o = 16; o; o >>= 1)
        sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if (x == 0 && blockIdx.x * 32 + y < p.hidden)
        p.dweight[blockIdx.x * 32 + y] = sum;
}

namespace {

// Rows of a stride that start and go on in whole pieces of `bytes`-byte values.
bool whole_pieces(const void *base, int64_t stride, int bytes)
{
    return !base || (reinterpret_cast<uintptr_t>(base) % 16 == 0 && stride * bytes % 16 == 0);
}

// The widest unit that all rows of a tensor start and go on in.
int unit_of(const void *base, int64_t stride, int bytes)
{
    const uint64_t all = reinterpret_cast<uintptr_t>(base) | static_cast<uint64_t>(stride) * bytes | 16;
    return static_cast<int>(all & (~all + 1));
}

int threads_for(int hidden, int pieces)
{
    const int per_thread = pieces * kPiece;
    return ((hidden + per_thread - 1) / per_thread + 31) / 32 * 32;
}

// How a row of a launch is laid out: threads, pieces of each, rows under way (0: more than
// shared memory holds) and blocks of an SM.
struct Form {
    int threads, pieces, stages, per_sm, smem;
};

Form form_for(int hidden, int value_bytes)
{
    Form f;
    f.pieces = hidden > kPiece * 512 ? 2 : 1;
    f.threads = threads_for(hidden, f.pieces);
    const int row = f.threads * f.pieces * kPiece * value_bytes;
    f.per_sm = 1024 / f.threads < 1 ? 1 : 1024 / f.threads;
    f.per_sm = f.per_sm > kMaxPerSm ? kMaxPerSm : f.per_sm;
    while (f.per_sm > 1 && 2 * row * f.per_sm > kSmemOfSm)
        --f.per_sm;
    f.stages = kSmemOfSm / (row * f.per_sm);
    f.stages = f.stages > 4 ? 4 : f.stages < 2 ? 0 : f.stages;
    f.smem = f.stages * row;
    return f;
}

template <typename Kern, typename... Args>
cudaError_t launch_rows(Kern kern, int threads, int smem, unsigned grid, cudaStream_t s, const Args &...args)
{
    if (smem > 48 * 1024) {
        const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
        if (e != cudaSuccess)
            return e;
    }
    return launch_behind(kern, grid, threads, smem, s, args...);
}

int padded(int hidden) { return (hidden + kPiece - 1) / kPiece * kPiece; }

}  // namespace

cudaError_t launch_norm(const NormParams &p, int num_sms, cudaStream_t s)
{
    const int rb = p.residual_bf16 ? 2 : 4;
    const bool vec = p.hidden % kPiece == 0 && whole_pieces(p.x, p.x_stride, 2) &&
                     whole_pieces(p.residual, p.residual_stride, rb) && whole_pieces(p.sum, p.sum_stride, rb) &&
                     whole_pieces(p.y, p.y_stride, 2) && whole_pieces(p.weight, 0, 4) &&
                     reinterpret_cast<uintptr_t>(p.q) % 8 == 0;
    const Form f = form_for(p.hidden, 2 + (p.residual ? rb : 0));
    if (!vec || !f.stages) {
        const int most = 16 * num_sms;
        const int row = padded(p.hidden) * (2 + (p.residual || p.sum ? rb : 0)), q = p.q ? padded(p.hidden) : 0;
        const int buffers = 2 * row + q <= kSmemOfSm ? 2 : 1;
        const RowUnits units = {{unit_of(p.x, p.x_stride, 2), unit_of(p.residual, p.residual_stride, rb),
                                 unit_of(p.sum, p.sum_stride, rb), unit_of(p.y, p.y_stride, 2),
                                 unit_of(p.q, p.hidden, 1)}};
        return launch_rows(norm_any_kernel, threads_for(p.hidden, kPieces), buffers * row + q,
                           p.T < most ? p.T : most, s, p, units, buffers);
    }
    const int most = f.per_sm * num_sms;
    const unsigned grid = p.T < most ? p.T : most;
    auto go = [&](auto two, auto three, auto four) {
        return launch_rows(f.stages == 2 ? two : f.stages == 3 ? three : four, f.threads, f.smem, grid, s, p);
    };
    return f.pieces == 1 ? go(norm_kernel<1, 2>, norm_kernel<1, 3>, norm_kernel<1, 4>)
                         : go(norm_kernel<2, 2>, norm_kernel<2, 3>, norm_kernel<2, 4>);
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
    const Form f = form_for(p.hidden, 2 + hb * 2);  // (without dsum, too: the same order of dweight's sum)
    int most = f.per_sm * num_sms;
    most = most < kPartBlocks ? most : kPartBlocks;
    const unsigned grid = p.T < most ? p.T : most;
    cudaError_t e;
    if (!vec || !f.stages) {
        const RowUnits units = {{unit_of(p.h, p.h_stride, hb), unit_of(p.dy, p.dy_stride, 2),
                                 unit_of(p.dsum, p.dsum_stride, hb), unit_of(p.dh, p.dh_stride, hb),
                                 unit_of(p.dx, p.dx_stride, 2)}};
        const int row = padded(p.hidden) * (2 + hb * (p.dsum ? 2 : 1)), buffers = 2 * row <= kSmemOfSm ? 2 : 1;
        e = launch_rows(norm_backward_any_kernel, threads_for(p.hidden, kPieces), buffers * row, grid, s, p, units,
                        buffers);
    } else {
        auto go = [&](auto two, auto three, auto four) {
            return launch_rows(f.stages == 2 ? two : f.stages == 3 ? three : four, f.threads, f.smem, grid, s, p);
        };
        e = f.pieces == 1 ? go(norm_backward_kernel<1, 2>, norm_backward_kernel<1, 3>, norm_backward_kernel<1, 4>)
                          : go(norm_backward_kernel<2, 2>, norm_backward_kernel<2, 3>, norm_backward_kernel<2, 4>);
    }
    if (e == cudaSuccess && p.dweight)
        e = launch_behind(norm_weight_kernel, (p.hidden + 31) / 32, 1024, 0, s, p, static_cast<int>(grid));
    return e;
}

}  // namespace ep
