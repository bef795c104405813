// The residual's addition and the root-mean-square norm in front of a layer, and its gradient.
//
//   h = x + residual,  r = 1 / sqrt(mean(h^2) + eps),  v = h * r * weight
//   g = dy * weight,   dh = r * (g - h * r^2 * mean(g * h)) + dsum,   dweight = sum_t dy * h * r
//
// Both are bound by their rows' bytes. A row stays in one thread block from its load to its
// stores: it is read once, and may be overwritten in place.
//  * Rows come to shared memory a row or two ahead (cp.async). Rows of whole 16-byte pieces: every
//    warp copies the pieces that it will use itself, so that nobody waits for anybody but in
//    the row's sums, and stores them from its registers. Any other rows lie in shared memory as
//    far from a 16-byte boundary as in memory, so that all but their ends still moves in
//    aligned pieces, in and out; threads shift the words that they read.
//  * Instructions come next to bytes here (a gradient of 43 a value took as long as its bytes):
//    hence arithmetic on two values at a time, the weight in registers, addresses that go on from
//    row to row, and up to four pieces of eight values a thread, which share the row's sums.
//  * dweight: a block adds its rows' terms in registers and leaves them in the workspace; a second
//    kernel adds the blocks'.
//
// Measured at 8192 x 7168 (GB300, of the copy bandwidth of 6.77 TB/s): beside a bf16 residual to e4m3
// 63 us, 97 %; to bf16 73 us, 95 %; the gradient in bf16 with the residual's 74 us, 93 %, in fp32
// 122 us, 99 %. Rows of other alignments, 4096 x 3675: 32 us, 55 %, the gradient 48 us, 37 %.
#include <type_traits>

#include "ep_internal.h"
#include "ep_ptx.cuh"
#include "ep_rows.cuh"

namespace ep {

using namespace rows;

namespace {

constexpr int kMaxThreads = 512;
static_assert(4 * kPiece * kMaxThreads == EP_MAX_NORM_HIDDEN, "a row in a block");
constexpr int kSmemOfSm = 216 * 1024;  // for rows under way
constexpr int kMaxPerSm = 16;          // blocks

// Blocks that leave partial sums of dweight, at most. (Short rows want many: 8192 x 256 8.8 us, with 640
// 12.5; 8192 x 2048 26.9, with 640 29.6.)
__host__ __device__ constexpr int part_blocks(int hidden) { return hidden <= 2048 ? 1280 : 640; }

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
    // (at most 16 warps: both halves of a warp do the same)
    float2 v = lane % 16 < warps ? part[lane % 16] : make_float2(0.f, 0.f);
#pragma unroll
    for (int o = 8; o; o >>= 1) {
        v.x += __shfl_xor_sync(0xffffffffu, v.x, o);
        v.y += __shfl_xor_sync(0xffffffffu, v.y, o);
    }
    return v;
}

// The same of one value.
__device__ __forceinline__ float block_sum(float a, float2 *part)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
#pragma unroll
    for (int o = 16; o; o >>= 1)
        a += __shfl_xor_sync(0xffffffffu, a, o);
    if (lane == 0)
        part[warp].x = a;
    __syncthreads();
    a = lane % 16 < warps ? part[lane % 16].x : 0.f;
#pragma unroll
    for (int o = 8; o; o >>= 1)
        a += __shfl_xor_sync(0xffffffffu, a, o);
    return a;
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

// The column of this lane's piece i of P: a warp's pieces lie behind one another, 32 at a time.
template <int P>
__device__ __forceinline__ int column(int warp, int i)
{
    return ((warp * P + i) * 32 + static_cast<int>(threadIdx.x & 31)) * kPiece;
}

// Bytes of 32 pieces.
__host__ __device__ constexpr int warp_bytes(bool bf16) { return 32 * kPiece * (bf16 ? 2 : 4); }

// A warp's part of a row of n values to shared memory, 16 bytes a lane at a time, so that every request is
// of whole sectors.
template <int P>
__device__ __forceinline__ void copy_part(uint8_t *to, const uint8_t *row, bool bf16, int warp, int n)
{
    const int begin = warp * P * warp_bytes(bf16), left = n * (bf16 ? 2 : 4) - begin;
    const uint32_t dst = smem_u32(to);
    row += begin;
#pragma unroll
    for (int i = 0; i < P * warp_bytes(bf16); i += 512) {
        const int at = i + static_cast<int>(threadIdx.x & 31) * 16;
        if (at < left)
            copy_async(dst + at, row + at);
    }
}

// This lane's piece of 32 that are there.
__device__ __forceinline__ Piece read_piece(const uint8_t *from, bool bf16)
{
    const int lane = threadIdx.x & 31;
    if (bf16)
        return unpack(reinterpret_cast<const uint4 *>(from)[lane]);
    const float4 *p = reinterpret_cast<const float4 *>(from) + lane * 2;
    return piece_of(p[0], p[1]);
}

// How far a row begins behind a 16-byte boundary.
__device__ __forceinline__ int skew_of(const void *row) { return static_cast<int>(reinterpret_cast<uintptr_t>(row) & 15); }

// Of `bytes` behind a skew, those that whole 16-byte pieces leave out are at most 15 at either end: a
// thread of the first warp each. This thread's, or -1.
__device__ __forceinline__ int end_of(int skew, int bytes)
{
    const int end = skew + bytes, head = min(skew ? 16 : 0, end), i = threadIdx.x % 16;
    const int at = threadIdx.x < 16 ? skew + i : max(end & ~15, head) + i;
    return threadIdx.x < 32 && at < (threadIdx.x < 16 ? head : end) ? at : -1;
}

// `bytes` of a row to shared memory, to skew_of(from) behind a 16-byte boundary: asynchronously but
// for the ends, of which this thread's byte is returned (put_end brings it to its place when the
// copies have arrived, so that nobody waits for the one before the others).
__device__ __forceinline__ uint8_t copy_in(uint8_t *to, const uint8_t *from, int bytes)
{
    const int skew = skew_of(from), at = end_of(skew, bytes);
    from -= skew;  // (whole 16 bytes from the first to the last lie inside the row)
    const int last = (skew + bytes) & ~15;
    for (int i = (skew ? 16 : 0) + threadIdx.x * 16; i < last; i += blockDim.x * 16)
        copy_async(smem_u32(to) + i, from + i);
    return at >= 0 ? from[at] : 0;
}

__device__ __forceinline__ void put_end(uint8_t *to, int skew, int bytes, uint8_t end)
{
    const int at = end_of(skew, bytes);
    if (at >= 0)
        to[at] = end;
}

// The same back, from skew_of(to) behind a 16-byte boundary of shared memory.
__device__ __forceinline__ void copy_out(uint8_t *to, const uint8_t *from, int bytes)
{
    const int skew = skew_of(to), at = end_of(skew, bytes), last = (skew + bytes) & ~15;
    to -= skew;
    for (int i = (skew ? 16 : 0) + threadIdx.x * 16; i < last; i += blockDim.x * 16)
        *reinterpret_cast<uint4 *>(to + i) = *reinterpret_cast<const uint4 *>(from + i);
    if (at >= 0)
        to[at] = from[at];
}

// The N words that begin `skew` bytes behind a 16-byte boundary of shared memory (of which N + 4 are
// there to be read).
template <int N>
__device__ __forceinline__ void read_skewed(const uint8_t *from, int skew, uint32_t (&out)[N])
{
    uint32_t w[N + 4];
#pragma unroll
    for (int i = 0; i < N + 4; i += 4) {
        const uint4 v = *reinterpret_cast<const uint4 *>(from + i * 4);
        w[i] = v.x, w[i + 1] = v.y, w[i + 2] = v.z, w[i + 3] = v.w;
    }
    const int shift = (skew & 3) * 8;
    auto take = [&](int first) {
#pragma unroll
        for (int i = 0; i < N; ++i)
            out[i] = __funnelshift_r(w[first + i], first + i + 1 < N + 4 ? w[first + i + 1] : 0, shift);
    };
    switch (skew >> 2) {  // (the same for the whole block)
    case 0:
        take(0);
        break;
    case 1:
        take(1);
        break;
    case 2:
        take(2);
        break;
    default:
        take(3);
    }
}

// Values c .. c+7 of a row of n that copy_in brought, 0 past its end.
__device__ __forceinline__ Piece read_any(const uint8_t *from, int skew, bool bf16, int c, int n)
{
    Piece p;
    if (bf16) {
        uint32_t w[4];
        read_skewed(from + c * 2, skew, w);
        p = unpack(make_uint4(w[0], w[1], w[2], w[3]));
    } else {
        uint32_t w[8];
        read_skewed(from + c * 4, skew, w);
#pragma unroll
        for (int i = 0; i < 4; ++i)
            p.v[i] = two(__uint_as_float(w[2 * i]), __uint_as_float(w[2 * i + 1]));
    }
    if (c + kPiece > n) {
        float f[kPiece];
        values_of(p, f);
#pragma unroll
        for (int i = 0; i < kPiece; ++i)
            f[i] = c + i < n ? f[i] : 0.f;
#pragma unroll
        for (int i = 0; i < 4; ++i)
            p.v[i] = two(f[2 * i], f[2 * i + 1]);
    }
    return p;
}

// And to where copy_out takes them from.
__device__ __forceinline__ void write_any(uint8_t *to, int skew, bool bf16, int c, int n, const Piece &p)
{
    float f[kPiece];
    values_of(p, f);
    if (bf16) {
        uint16_t *at = reinterpret_cast<uint16_t *>(to + skew) + c;
        const uint4 v = pack(p);
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
        if (skew % 4 == 0 && c + kPiece <= n) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                reinterpret_cast<uint32_t *>(at)[i] = w[i];
        } else {
#pragma unroll
            for (int i = 0; i < kPiece; ++i)
                if (c + i < n)
                    at[i] = static_cast<uint16_t>(w[i / 2] >> (i % 2 * 16));
        }
    } else {
        float *at = reinterpret_cast<float *>(to + skew) + c;
#pragma unroll
        for (int i = 0; i < kPiece; ++i)
            if (c + i < n)
                at[i] = f[i];
    }
}

__device__ __forceinline__ void write_any(uint8_t *to, int skew, int c, int n, uint2 codes)
{
    uint8_t *at = to + skew + c;
    if (skew % 4 == 0 && c + kPiece <= n) {
        reinterpret_cast<uint32_t *>(at)[0] = codes.x;
        reinterpret_cast<uint32_t *>(at)[1] = codes.y;
    } else {
#pragma unroll
        for (int i = 0; i < kPiece; ++i)
            if (c + i < n)
                at[i] = static_cast<uint8_t>((i < 4 ? codes.x : codes.y) >> (8 * (i & 3)));
    }
}

// Bytes in shared memory of a row of n values: whole pieces, and 16 bytes for the skew.
__host__ __device__ constexpr int room_of(int n, int value_bytes)
{
    return (n + kPiece - 1) / kPiece * kPiece * value_bytes / 16 * 16 + 32;
}

// This thread's pieces of the weight.
template <int P>
__device__ __forceinline__ void load_weight(const uint8_t *weight, bool bf16, int warp, int n, Piece (&w)[P])
{
    const bool aligned = reinterpret_cast<uintptr_t>(weight) % 16 == 0;
#pragma unroll
    for (int i = 0; i < P; ++i) {
        const int c = column<P>(warp, i);
        w[i] = zeros();
        if (c >= n)
            continue;
        if (!aligned || c + kPiece > n)
            w[i] = load_any(weight, bf16, c, n);
        else if (bf16)
            w[i] = unpack(*reinterpret_cast<const uint4 *>(weight + c * 2));
        else
            w[i] = piece_of(*reinterpret_cast<const float4 *>(weight + c * 4),
                            *reinterpret_cast<const float4 *>(weight + c * 4 + 16));
    }
}

__device__ __forceinline__ Piece scaled(const Piece &h, float r, const Piece &w)
{
    const Two rr = two(r, r);
    Piece v;
#pragma unroll
    for (int j = 0; j < 4; ++j)
        v.v[j] = mul2(mul2(h.v[j], rr), w.v[j]);
    return v;
}

// The gradient's terms of a piece: d += r (dy w - h back), dw += dy (h r). (back is r (r mean(g h)), in this
// order: r^2 alone leaves fp32 for rows of 2^-64 and less, r mean(g h) only where r g, the gradient, does.)
__device__ __forceinline__ void gradient(const Piece &h, const Piece &dy, const Piece &w, float r, float back, Piece &d,
                                         Piece &dw)
{
    const Two rr = two(r, r), minus_back = two(-back, -back);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        d.v[j] = fma2(rr, fma2(h.v[j], minus_back, mul2(dy.v[j], w.v[j])), d.v[j]);
        dw.v[j] = fma2(dy.v[j], mul2(h.v[j], rr), dw.v[j]);
    }
}

// And those of its sums.
__device__ __forceinline__ void gradient_sums(const Piece &h, const Piece &dy, const Piece &w, Two &squares, Two &dot)
{
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        squares = fma2(h.v[j], h.v[j], squares);
        dot = fma2(mul2(dy.v[j], w.v[j]), h.v[j], dot);
    }
}

}  // namespace

// Rows of whole aligned pieces. BF16: the residual stream's type; P: pieces of a thread, S: rows under
// way.
template <bool BF16, int P, int S>
__global__ void __launch_bounds__(P == 1 ? 128 : 512, P == 1 ? 8 : P == 2 ? 2 : 1) norm_kernel(const NormParams p)
{
    extern __shared__ __align__(16) uint8_t ring[];
    __shared__ float2 part[2][kMaxThreads / 32];
    constexpr int rb = BF16 ? 2 : 4;
    const int n = p.hidden, warps = blockDim.x >> 5;
    const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0);  // (for the compiler to see that its lanes agree)
    // of a warp: x, then the residual
    constexpr int x_bytes = P * warp_bytes(true);
    const int bytes = x_bytes + (p.residual ? P * warp_bytes(BF16) : 0);
    const float over_n = 1.f / n;
    griddep_wait();
    griddep_launch_dependents();
    // this block's rows and the way from one to the next
    int64_t t = blockIdx.x;
    const uint8_t *x = p.x + t * p.x_stride * 2, *res = p.residual + t * p.residual_stride * rb;
    uint8_t *sum = p.sum + t * p.sum_stride * rb, *y = p.y + t * p.y_stride * 2, *q = p.q + t * n;
    float *scales = p.q_scales + t * ((n + 127) / 128);
    const int64_t blocks = gridDim.x, x_step = blocks * p.x_stride * 2, res_step = blocks * p.residual_stride * rb;
    auto ask = [&](int ahead, int stage) {
        if (t + ahead * blocks < p.T) {
            const uint8_t *const from = x + ahead * x_step, *const res_from = res + ahead * res_step;
            uint8_t *const to = ring + (stage * warps + warp) * bytes;
            copy_part<P>(to, from, true, warp, n);
            if (p.residual)
                copy_part<P>(to + x_bytes, res_from, BF16, warp, n);
        }
        copy_commit();
    };
#pragma unroll
    for (int i = 0; i < S - 1; ++i)
        ask(i, i);
    Piece w[P];
    load_weight(p.weight, p.weight_bf16, warp, n, w);
    int stage = 0, turn = 0;
    for (; t < p.T; t += blocks) {
        uint8_t *const mine = ring + (stage * warps + warp) * bytes;
        if (!BF16)
            __syncwarp();  // (pieces are copied by the warp's other lanes)
        ask(S - 1, stage == 0 ? S - 1 : stage - 1);
        copy_wait<S - 1>();
        if (!BF16)
            __syncwarp();
        Piece h[P];
        Two squares = 0;
#pragma unroll
        for (int i = 0; i < P; ++i) {
            const int c = column<P>(warp, i);
            h[i] = c < n ? read_piece(mine + i * warp_bytes(true), true) : zeros();
            if (p.residual) {
                const Piece r = c >= n ? zeros() : read_piece(mine + x_bytes + i * warp_bytes(BF16), BF16);
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    h[i].v[j] = add2(h[i].v[j], r.v[j]);
            }
#pragma unroll
            for (int j = 0; j < 4; ++j)
                squares = fma2(h[i].v[j], h[i].v[j], squares);
        }
        const float r = rsqrtf(block_sum(sum_of(squares), part[turn ^= 1]) * over_n + p.eps);
#pragma unroll
        for (int i = 0; i < P; ++i) {
            const int c = column<P>(warp, i);
            if (c < n && p.sum)
                store_piece(sum, BF16, c, h[i]);
            const Piece v = scaled(h[i], r, w[i]);
            if (c < n && p.y)
                store_piece(y, true, c, v);
            if (p.q) {
                const uint2 codes = quantise(v, scales, c, n);
                if (c < n)
                    *reinterpret_cast<uint2 *>(q + c) = codes;
            }
        }
        stage = stage == S - 1 ? 0 : stage + 1;
        x += x_step;
        res += res_step;
        sum += blocks * p.sum_stride * rb;
        y += blocks * p.y_stride * 2;
        q += blocks * n;
        scales += blocks * ((n + 127) / 128);
    }
}

template <bool BF16, int P, int S>
__global__ void __launch_bounds__(P == 1 ? 128 : P == 2 ? 256 : 512, P == 1 ? 8 : P == 2 ? 3 : 1)
    norm_backward_kernel(const NormBackwardParams p)
{
    extern __shared__ __align__(16) uint8_t ring[];
    __shared__ float2 part[2][kMaxThreads / 32];
    constexpr int hb = BF16 ? 2 : 4;
    const int n = p.hidden, warps = blockDim.x >> 5;
    const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0);  // (for the compiler to see that its lanes agree)
    // of a warp: h, dy, then dsum
    constexpr int h_bytes = P * warp_bytes(BF16), dy_bytes = P * warp_bytes(true);
    const int bytes = dy_bytes + h_bytes * (p.dsum ? 2 : 1);
    const float over_n = 1.f / n;
    griddep_wait();
    griddep_launch_dependents();
    int64_t t = blockIdx.x;
    const uint8_t *h = p.h + t * p.h_stride * hb, *dy = p.dy + t * p.dy_stride * 2, *dsum = p.dsum + t * p.dsum_stride * hb;
    uint8_t *dh = p.dh + t * p.dh_stride * hb, *dx = p.dx + t * p.dx_stride * 2;
    const int64_t blocks = gridDim.x;
    const int64_t h_step = blocks * p.h_stride * hb, dy_step = blocks * p.dy_stride * 2, dsum_step = blocks * p.dsum_stride * hb;
    auto ask = [&](int ahead, int stage) {
        if (t + ahead * blocks < p.T) {
            const uint8_t *const h_from = h + ahead * h_step, *const dy_from = dy + ahead * dy_step;
            const uint8_t *const dsum_from = dsum + ahead * dsum_step;
            uint8_t *const to = ring + (stage * warps + warp) * bytes;
            copy_part<P>(to, h_from, BF16, warp, n);
            copy_part<P>(to + h_bytes, dy_from, true, warp, n);
            if (p.dsum)
                copy_part<P>(to + h_bytes + dy_bytes, dsum_from, BF16, warp, n);
        }
        copy_commit();
    };
#pragma unroll
    for (int i = 0; i < S - 1; ++i)
        ask(i, i);
    Piece w[P], dw[P];
    load_weight(p.weight, p.weight_bf16, warp, n, w);
#pragma unroll
    for (int i = 0; i < P; ++i)
        dw[i] = zeros();
    int stage = 0, turn = 0;
    for (; t < p.T; t += blocks) {
        uint8_t *const mine = ring + (stage * warps + warp) * bytes;
        if (!BF16)
            __syncwarp();  // (pieces are copied by the warp's other lanes)
        ask(S - 1, stage == 0 ? S - 1 : stage - 1);
        copy_wait<S - 1>();
        if (!BF16)
            __syncwarp();
        Two squares = 0, dot = 0;
#pragma unroll
        for (int i = 0; i < P; ++i) {
            const int c = column<P>(warp, i);
            const uint8_t *const h_at = mine + i * warp_bytes(BF16), *const dy_at = mine + h_bytes + i * warp_bytes(true);
            if (c < n)
                gradient_sums(read_piece(h_at, BF16), read_piece(dy_at, true), w[i], squares,
                              dot);
        }
        const float2 sums = block_sum(sum_of(squares), sum_of(dot), part[turn ^= 1]);
        const float r = rsqrtf(sums.x * over_n + p.eps), back = r * (r * (sums.y * over_n));
#pragma unroll
        for (int i = 0; i < P; ++i) {
            const int c = column<P>(warp, i);
            const uint8_t *const h_at = mine + i * warp_bytes(BF16), *const dy_at = mine + h_bytes + i * warp_bytes(true);
            if (c >= n)
                break;
            Piece d = p.dsum ? read_piece(h_at + h_bytes + dy_bytes, BF16) : zeros();
            gradient(read_piece(h_at, BF16), read_piece(dy_at, true), w[i], r, back, d, dw[i]);
            if (p.dh)
                store_piece(dh, BF16, c, d);
            if (p.dx)
                store_piece(dx, true, c, d);
        }
        stage = stage == S - 1 ? 0 : stage + 1;
        h += h_step;
        dy += dy_step;
        dsum += dsum_step;
        dh += blocks * p.dh_stride * hb;
        dx += blocks * p.dx_stride * 2;
    }
    if (p.dweight) {
        uint8_t *const to = reinterpret_cast<uint8_t *>(p.parts + static_cast<int64_t>(blockIdx.x) * n);
#pragma unroll
        for (int i = 0; i < P; ++i)
            if (const int c = column<P>(warp, i); c < n)
                store_piece(to, false, c, dw[i]);
    }
}

// Rows of any alignment: x (then y) and the residual (then sum) in two buffers that take turns; q. (What
// is written has the skew of where it goes, so that it may overlap what other threads read: between the
// two lies a barrier.)
template <bool BF16, int P>
__global__ void __launch_bounds__(P == 1 ? 128 : 512, P == 1 ? 8 : P == 2 ? 2 : 1) norm_any_kernel(const NormParams p)
{
    extern __shared__ __align__(16) uint8_t row[];
    __shared__ float2 part[2][kMaxThreads / 32];
    constexpr int rb = BF16 ? 2 : 4;
    const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0);
    const float over_n = 1.f / p.hidden;
    const int n = p.hidden, x_room = room_of(n, 2);
    const int room = x_room + (p.residual || p.sum ? room_of(n, rb) : 0);
    uint8_t *const q_row = row + 2 * room;
    griddep_wait();
    griddep_launch_dependents();
    uint8_t x_end = 0, res_end = 0;  // of the row asked for
    auto ask = [&](int64_t t, int buffer) {
        if (t < p.T) {
            x_end = copy_in(row + buffer * room, p.x + t * p.x_stride * 2, n * 2);
            if (p.residual)
                res_end = copy_in(row + buffer * room + x_room, p.residual + t * p.residual_stride * rb, n * rb);
        }
        copy_commit();
    };
    ask(blockIdx.x, 0);
    Piece w[P];
    load_weight(p.weight, p.weight_bf16, warp, n, w);
    int buffer = 0, turn = 0;
    for (int64_t t = blockIdx.x; t < p.T; t += gridDim.x) {
        uint8_t *const x = row + buffer * room, *const res = x + x_room;
        const int x_skew = skew_of(p.x + t * p.x_stride * 2);
        const int res_skew = skew_of(p.residual + t * p.residual_stride * rb);
        copy_wait<0>();
        put_end(x, x_skew, n * 2, x_end);
        if (p.residual)
            put_end(res, res_skew, n * rb, res_end);
        __syncthreads();
        ask(t + gridDim.x, buffer ^= 1);  // (where the row before this one has left by now)
        Piece h[P];
        Two squares = 0;
#pragma unroll
        for (int i = 0; i < P; ++i) {
            const int c = column<P>(warp, i);
            h[i] = zeros();
            if (c < n) {
                h[i] = read_any(x, x_skew, true, c, n);
                if (p.residual) {
                    const Piece r = read_any(res, res_skew, BF16, c, n);
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        h[i].v[j] = add2(h[i].v[j], r.v[j]);
                }
            }
#pragma unroll
            for (int j = 0; j < 4; ++j)
                squares = fma2(h[i].v[j], h[i].v[j], squares);
        }
        const float r = rsqrtf(block_sum(sum_of(squares), part[turn ^= 1]) * over_n + p.eps);
        uint8_t *const sum = p.sum + t * p.sum_stride * rb, *const y = p.y + t * p.y_stride * 2, *const q = p.q + t * n;
#pragma unroll
        for (int i = 0; i < P; ++i) {
            const int c = column<P>(warp, i);
            if (c < n && p.sum)
                write_any(res, skew_of(sum), BF16, c, n, h[i]);
            const Piece v = scaled(h[i], r, w[i]);
            if (c < n && p.y)
                write_any(x, skew_of(y), true, c, n, v);
            if (p.q) {
                const uint2 codes = quantise(v, p.q_scales + t * ((n + 127) / 128), c, n);
                if (c < n)
                    write_any(q_row, skew_of(q), c, n, codes);
            }
        }
        __syncthreads();
        if (p.sum)
            copy_out(sum, res, n * rb);
        if (p.y)
            copy_out(y, x, n * 2);
        if (p.q)
            copy_out(q, q_row, n);
    }
}

// The same for the gradient: h (then dh), dy (then dx), dsum, in one buffer where two do not fit.
template <bool BF16, int P>
__global__ void __launch_bounds__(P == 1 ? 128 : P == 2 ? 256 : 512, P == 1 ? 8 : P == 2 ? 3 : 1)
    norm_backward_any_kernel(const NormBackwardParams p, int buffers)
{
    extern __shared__ __align__(16) uint8_t row[];
    __shared__ float2 part[2][kMaxThreads / 32];
    constexpr int hb = BF16 ? 2 : 4;
    const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0);
    const float over_n = 1.f / p.hidden;
    const int n = p.hidden, h_room = room_of(n, hb), dy_room = room_of(n, 2);
    const int room = dy_room + h_room * (p.dsum ? 2 : 1);
    griddep_wait();
    griddep_launch_dependents();
    uint8_t h_end = 0, dy_end = 0, dsum_end = 0;  // of the row asked for
    auto ask = [&](int64_t t, int buffer) {
        if (t < p.T) {
            uint8_t *const to = row + buffer * room;
            h_end = copy_in(to, p.h + t * p.h_stride * hb, n * hb);
            dy_end = copy_in(to + h_room, p.dy + t * p.dy_stride * 2, n * 2);
            if (p.dsum)
                dsum_end = copy_in(to + h_room + dy_room, p.dsum + t * p.dsum_stride * hb, n * hb);
        }
        copy_commit();
    };
    if (buffers > 1)
        ask(blockIdx.x, 0);
    Piece w[P], dw[P];
    load_weight(p.weight, p.weight_bf16, warp, n, w);
#pragma unroll
    for (int i = 0; i < P; ++i)
        dw[i] = zeros();
    int buffer = 0, turn = 0;
    for (int64_t t = blockIdx.x; t < p.T; t += gridDim.x) {
        uint8_t *const h_row = row + buffer * room, *const dy_row = h_row + h_room, *const dsum_row = dy_row + dy_room;
        const int h_skew = skew_of(p.h + t * p.h_stride * hb), dy_skew = skew_of(p.dy + t * p.dy_stride * 2);
        const int dsum_skew = skew_of(p.dsum + t * p.dsum_stride * hb);
        if (buffers == 1)
            ask(t, 0);
        copy_wait<0>();
        put_end(h_row, h_skew, n * hb, h_end);
        put_end(dy_row, dy_skew, n * 2, dy_end);
        if (p.dsum)
            put_end(dsum_row, dsum_skew, n * hb, dsum_end);
        __syncthreads();
        if (buffers > 1)  // (where the row before this one has left by now)
            ask(t + gridDim.x, buffer ^= 1);
        Two squares = 0, dot = 0;
#pragma unroll
        for (int i = 0; i < P; ++i) {
            const int c = column<P>(warp, i);
            if (c < n)
                gradient_sums(read_any(h_row, h_skew, BF16, c, n), read_any(dy_row, dy_skew, true, c, n), w[i],
                              squares, dot);
        }
        const float2 sums = block_sum(sum_of(squares), sum_of(dot), part[turn ^= 1]);
        const float r = rsqrtf(sums.x * over_n + p.eps), back = r * (r * (sums.y * over_n));
        uint8_t *const dh = p.dh + t * p.dh_stride * hb, *const dx = p.dx + t * p.dx_stride * 2;
        Piece d[P];
#pragma unroll
        for (int i = 0; i < P; ++i) {
            const int c = column<P>(warp, i);
            d[i] = zeros();
            if (c >= n)
                continue;
            if (p.dsum)
                d[i] = read_any(dsum_row, dsum_skew, BF16, c, n);
            gradient(read_any(h_row, h_skew, BF16, c, n), read_any(dy_row, dy_skew, true, c, n), w[i], r, back,
                     d[i], dw[i]);
        }
        // what goes where it came from, byte by byte, overwrites nothing that another thread still reads
        if ((p.dh && skew_of(dh) != h_skew) || (p.dx && skew_of(dx) != dy_skew))
            __syncthreads();
#pragma unroll
        for (int i = 0; i < P; ++i) {
            const int c = column<P>(warp, i);
            if (c < n && p.dh)
                write_any(h_row, skew_of(dh), BF16, c, n, d[i]);
            if (c < n && p.dx)
                write_any(dy_row, skew_of(dx), true, c, n, d[i]);
        }
        __syncthreads();
        if (p.dh)
            copy_out(dh, h_row, n * hb);
        if (p.dx)
            copy_out(dx, dy_row, n * 2);
        if (buffers == 1)
            __syncthreads();
    }
    if (p.dweight) {
        float *mine = p.parts + static_cast<int64_t>(blockIdx.x) * n;
#pragma unroll
        for (int i = 0; i < P; ++i) {
            float f[kPiece];
            values_of(dw[i], f);
#pragma unroll
            for (int j = 0; j < kPiece; ++j) {
                const int c = column<P>(warp, i) + j;
                if (c < n)
                    mine[c] = f[j];
            }
        }
    }
}

// dweight from the blocks' sums, C columns a thread block: 1024 / C threads to a column, which take the
// blocks in turn, then theirs in order.
template <int C>
__global__ void __launch_bounds__(1024) norm_weight_kernel(const NormBackwardParams p, int blocks)
{
    __shared__ float part[32][C + 1];
    griddep_wait();
    griddep_launch_dependents();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int x = threadIdx.x % C, y = threadIdx.x / C, c0 = blockIdx.x * C;
    float sum = 0.f;
    if (c0 + x < p.hidden) {
#pragma unroll 8
        for (int b = y; b < blocks; b += 1024 / C)
            sum += __ldcg(p.parts + static_cast<int64_t>(b) * p.hidden + c0 + x);
    }
#pragma unroll
    for (int o = 16; o >= C; o >>= 1)
        sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if (lane < C)
        part[warp][lane] = sum;
    __syncthreads();
    // (a warp to a column now)
    if (warp < C) {
        sum = part[lane][warp];
#pragma unroll
        for (int o = 16; o; o >>= 1)
            sum += __shfl_xor_sync(0xffffffffu, sum, o);
        if (lane == 0 && c0 + warp < p.hidden)
            p.dweight[c0 + warp] = sum;
    }
}

namespace {

// Rows of a stride that start and go on in whole pieces of `bytes`-byte values.
bool whole_pieces(const void *base, int64_t stride, int bytes)
{
    return !base || (reinterpret_cast<uintptr_t>(base) % 16 == 0 && stride * bytes % 16 == 0);
}

// How a row of a launch is laid out: threads, pieces of each, rows under way and blocks of an SM.
struct Form {
    int threads, pieces, stages, per_sm;
};

// `two_upto`: the longest rows of two pieces a thread.
// Blocks of an SM go by the registers that the kernels' launch bounds allow a thread, 64 or (`regs`
// for two pieces, 128 for four) more: blocks past what is resident would begin when the others end.
constexpr Form form_for(int hidden, int value_bytes, int two_upto, int regs, int stages)
{
    Form f{};
    f.pieces = hidden <= 1024 ? 1 : hidden <= two_upto ? 2 : 4;
    const int per_thread = f.pieces * kPiece;
    f.threads = ((hidden + per_thread - 1) / per_thread + 31) / 32 * 32;
    const int row = f.threads * per_thread * value_bytes;
    const int most = 65536 / (f.pieces == 1 ? 64 : f.pieces == 2 ? regs : 128) / f.threads;
    f.per_sm = most < 1 ? 1 : most > kMaxPerSm ? kMaxPerSm : most;
    while (f.per_sm > 1 && 2 * row * f.per_sm > kSmemOfSm)
        --f.per_sm;
    f.stages = kSmemOfSm / (row * f.per_sm);
    f.stages = f.stages > stages ? stages : f.stages;
    return f;
}

// The forms of both calls' whole rows, and the rows that their kernels keep under way: as many as fit, but
// for the longest rows three (the gradient: two).
constexpr Form norm_form(int hidden, int value_bytes) { return form_for(hidden, value_bytes, 8192, 64, 3); }
constexpr int norm_stages(const Form &f, bool bf16) { return f.pieces == 1 || bf16 || f.stages > 2 ? 3 : 2; }

// (the bytes as with dsum, where there is none, too: the same order of dweight's sum)
// Two rows under way: three took 8192 x 7168 in fp32 from 123 to 138 us, 8192 x 4096 in bf16 from 46 to 51.
constexpr Form backward_form(int hidden, int h_bytes) { return form_for(hidden, 2 + h_bytes * 2, 4096, 85, 2); }
constexpr int backward_stages(const Form &f, bool bf16) { return f.pieces <= 2 || bf16 || f.stages > 1 ? 2 : 1; }

// Every row that a kernel keeps under way has its place in shared memory.
constexpr bool rows_fit()
{
    for (int hidden = kPiece; hidden <= EP_MAX_NORM_HIDDEN; hidden += kPiece)
        for (int bytes = 2; bytes <= 4; bytes += 2) {  // of the residual stream's values
            const Form alone = norm_form(hidden, 2), beside = norm_form(hidden, 2 + bytes);
            const Form back = backward_form(hidden, bytes);
            const bool bf16 = bytes == 2;
            if (alone.stages < norm_stages(alone, bf16) || beside.stages < norm_stages(beside, bf16) ||
                back.stages < backward_stages(back, bf16))
                return false;
        }
    return true;
}
static_assert(rows_fit(), "the rows under way");

template <typename Kern, typename... Args>
cudaError_t launch_rows(Kern kern, int threads, int smem, unsigned grid, cudaStream_t s, const Args &...args)
{
    if (smem > 47 * 1024) {  // (48 KB with the kernel's own)
        // (the attribute is the kernel's, not the call's: one value for all calls, as other threads set it, too)
        const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemOfSm);
        if (e != cudaSuccess)
            return e;
    }
    return launch_behind(kern, grid, threads, smem, s, args...);
}

}  // namespace

cudaError_t launch_norm(const NormParams &p, int num_sms, cudaStream_t s)
{
    const int rb = p.residual_bf16 ? 2 : 4;
    const bool whole = p.hidden % kPiece == 0 && whole_pieces(p.x, p.x_stride, 2) &&
                       whole_pieces(p.residual, p.residual_stride, rb) && whole_pieces(p.sum, p.sum_stride, rb) &&
                       whole_pieces(p.y, p.y_stride, 2) && reinterpret_cast<uintptr_t>(p.q) % 8 == 0;
    const int bytes = 2 + (p.residual ? rb : 0);
    const Form f = norm_form(p.hidden, bytes);
    // Of rows with a residual a block takes about 6 (fp32: 3), as the SMs' shares of the bandwidth are
    // not equal and new blocks go to those that are ahead: 8192 x 7168 beside a bf16 residual 65 us in
    // 4 waves of blocks (71.6 in one, 77 in 16), an fp32 one 96 in 8 (112 in one), 4096 wide 38.6 in
    // 2 (41.9 in one). Without a residual one wave is best (7168 wide 38.4, two 40.2).
    const int resident = f.per_sm * num_sms, rows = resident * (p.residual_bf16 ? 6 : 3);
    const int waves = !p.residual || p.T < rows ? 1 : static_cast<int>((int64_t{p.T} + rows / 2) / rows);
    const int most = resident * waves;
    const unsigned grid = p.T < most ? p.T : most;
    if (whole) {
        // (one row a block needs no second: no attribute to set, a tenth of a small call's host time)
        const int stages = norm_stages(f, p.residual_bf16);
        const int smem = (p.T == static_cast<int>(grid) ? 1 : stages) * f.threads * f.pieces * kPiece * bytes;
        auto go = [&](auto bf16) {
            constexpr bool B = decltype(bf16)::value;
            constexpr int two = B ? 3 : 2;  // (norm_stages)
            const auto kern = f.pieces == 1   ? norm_kernel<B, 1, 3>
                              : f.pieces == 2 ? (stages == 2 ? norm_kernel<B, 2, two> : norm_kernel<B, 2, 3>)
                                              : (stages == 2 ? norm_kernel<B, 4, two> : norm_kernel<B, 4, 3>);
            return launch_rows(kern, f.threads, smem, grid, s, p);
        };
        return p.residual_bf16 ? go(std::true_type()) : go(std::false_type());
    }
    const int room = room_of(p.hidden, 2) + (p.residual || p.sum ? room_of(p.hidden, rb) : 0);
    const int q_room = p.q ? room_of(p.hidden, 1) : 0;
    static_assert(2 * (room_of(EP_MAX_NORM_HIDDEN, 2) + room_of(EP_MAX_NORM_HIDDEN, 4)) +
                      room_of(EP_MAX_NORM_HIDDEN, 1) <= kSmemOfSm, "two rows and the codes");
    auto go = [&](auto bf16) {
        constexpr bool B = decltype(bf16)::value;
        return launch_rows(f.pieces == 1   ? norm_any_kernel<B, 1>
                           : f.pieces == 2 ? norm_any_kernel<B, 2>
                                           : norm_any_kernel<B, 4>,
                           f.threads, 2 * room + q_room, grid, s, p);
    };
    return p.residual_bf16 ? go(std::true_type()) : go(std::false_type());
}

int64_t norm_backward_workspace_bytes(int T, int hidden)
{
    return static_cast<int64_t>(T < part_blocks(hidden) ? T : part_blocks(hidden)) * hidden * 4;
}

cudaError_t launch_norm_backward(const NormBackwardParams &p, int num_sms, cudaStream_t s)
{
    const int hb = p.h_bf16 ? 2 : 4;
    const bool whole = p.hidden % kPiece == 0 && whole_pieces(p.h, p.h_stride, hb) &&
                       whole_pieces(p.dy, p.dy_stride, 2) && whole_pieces(p.dsum, p.dsum_stride, hb) &&
                       whole_pieces(p.dh, p.dh_stride, hb) && whole_pieces(p.dx, p.dx_stride, 2);
    const Form f = backward_form(p.hidden, hb);
    int most = f.per_sm * num_sms;
    if (p.dweight && most > part_blocks(p.hidden))  // (rows alone: 8192 x 512 12.1 us with this limit, 8.2 without)
        most = part_blocks(p.hidden);
    const unsigned grid = p.T < most ? p.T : most;
    cudaError_t e;
    if (whole) {
        const int stages = backward_stages(f, p.h_bf16);
        const int smem = (p.T == static_cast<int>(grid) ? 1 : stages) * f.threads * f.pieces * kPiece *
                         (2 + hb * (p.dsum ? 2 : 1));
        auto go = [&](auto bf16) {
            constexpr bool B = decltype(bf16)::value;
            constexpr int one = B ? 2 : 1;  // (backward_stages)
            const auto kern = f.pieces == 1   ? norm_backward_kernel<B, 1, 2>
                              : f.pieces == 2 ? norm_backward_kernel<B, 2, 2>
                              : stages == 1   ? norm_backward_kernel<B, 4, one>
                                              : norm_backward_kernel<B, 4, 2>;
            return launch_rows(kern, f.threads, smem, grid, s, p);
        };
        e = p.h_bf16 ? go(std::true_type()) : go(std::false_type());
    } else {
        const int room = room_of(p.hidden, 2) + room_of(p.hidden, hb) * (p.dsum ? 2 : 1);
        const int buffers = 2 * room <= kSmemOfSm ? 2 : 1;
        auto go = [&](auto bf16) {
            constexpr bool B = decltype(bf16)::value;
            return launch_rows(f.pieces == 1   ? norm_backward_any_kernel<B, 1>
                               : f.pieces == 2 ? norm_backward_any_kernel<B, 2>
                                               : norm_backward_any_kernel<B, 4>,
                               f.threads, buffers * room, grid, s, p, buffers);
        };
        e = p.h_bf16 ? go(std::true_type()) : go(std::false_type());
    }
    if (e == cudaSuccess && p.dweight) {
        // Many blocks, of short rows: more and narrower blocks here (8192 x 256 beside bf16 8.8 us, with 32
        // columns 9.9, 8192 x 1024 16.4 and 18.3; 8192 x 7168 77.1 us, with 32 columns 74.3).
        const bool narrow = grid > 640;
        const int columns = narrow ? 8 : 32;
        e = launch_behind(narrow ? norm_weight_kernel<8> : norm_weight_kernel<32>, (p.hidden + columns - 1) / columns,
                          1024, 0, s, p, static_cast<int>(grid));
    }
    return e;
}

}  // namespace ep
