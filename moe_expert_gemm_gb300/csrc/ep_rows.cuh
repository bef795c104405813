// Rows in pieces of eight values: loads and stores in fp32 and bf16, and the quantisation of
// 128 columns to e4m3 with one scale.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp8.h>

#include <cstdint>

namespace ep {
namespace rows {

constexpr int kPiece = 8;         // values of a piece
constexpr int kGroupPieces = 16;  // pieces of a scale's 128 columns: half a warp

__device__ __forceinline__ float lo_of(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float hi_of(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

__device__ __forceinline__ uint32_t pack(float lo, float hi)
{
    const __nv_bfloat162 b = __float22bfloat162_rn(make_float2(lo, hi));
    return *reinterpret_cast<const uint32_t *>(&b);
}

__device__ __forceinline__ void unpack(const uint4 &v, float (&f)[kPiece])
{
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i)
        f[2 * i] = lo_of(w[i]), f[2 * i + 1] = hi_of(w[i]);
}

__device__ __forceinline__ uint4 pack(const float (&f)[kPiece])
{
    return make_uint4(pack(f[0], f[1]), pack(f[2], f[3]), pack(f[4], f[5]), pack(f[6], f[7]));
}

// Values c .. c+7 of a row at `base` (of n values; 0 past its end). VEC: whole, aligned pieces.
template <bool VEC>
__device__ __forceinline__ void load_piece(const uint8_t *base, bool bf16, int c, int n, float (&f)[kPiece])
{
    if (bf16) {
        const __nv_bfloat16 *r = reinterpret_cast<const __nv_bfloat16 *>(base) + c;
        if (VEC) {
            unpack(*reinterpret_cast<const uint4 *>(r), f);
        } else {
#pragma unroll
            for (int i = 0; i < kPiece; ++i)
                f[i] = c + i < n ? __bfloat162float(r[i]) : 0.f;
        }
    } else {
        const float *r = reinterpret_cast<const float *>(base) + c;
        if (VEC) {
            const float4 a = *reinterpret_cast<const float4 *>(r);
            const float4 b = *reinterpret_cast<const float4 *>(r + 4);
            f[0] = a.x, f[1] = a.y, f[2] = a.z, f[3] = a.w;
            f[4] = b.x, f[5] = b.y, f[6] = b.z, f[7] = b.w;
        } else {
#pragma unroll
            for (int i = 0; i < kPiece; ++i)
                f[i] = c + i < n ? r[i] : 0.f;
        }
    }
}

template <bool VEC>
__device__ __forceinline__ void store_piece(uint8_t *base, bool bf16, int c, int n, const float (&f)[kPiece])
{
    if (bf16) {
        __nv_bfloat16 *r = reinterpret_cast<__nv_bfloat16 *>(base) + c;
        if (VEC) {
            *reinterpret_cast<uint4 *>(r) = pack(f);
        } else {
#pragma unroll
            for (int i = 0; i < kPiece; ++i)
                if (c + i < n)
                    r[i] = __float2bfloat16_rn(f[i]);
        }
    } else {
        float *r = reinterpret_cast<float *>(base) + c;
        if (VEC) {
            *reinterpret_cast<float4 *>(r) = make_float4(f[0], f[1], f[2], f[3]);
            *reinterpret_cast<float4 *>(r + 4) = make_float4(f[4], f[5], f[6], f[7]);
        } else {
#pragma unroll
            for (int i = 0; i < kPiece; ++i)
                if (c + i < n)
                    r[i] = f[i];
        }
    }
}

// SiLU(x) * u. The quotient by the fast division (error 2 units in the last place; 0 where e^-x
// passes 2^126, where the true value is below 2^-119).
__device__ __forceinline__ float silu_times(float x, float u)
{
    return __fdividef(x, 1.f + expf(-x)) * u;
}

// The bits of |v|: as integers they order finite values, infinities and NaN in that order.
__device__ __forceinline__ uint32_t size_bits(float v) { return __float_as_uint(v) & 0x7FFFFFFFu; }

__device__ __forceinline__ uint32_t size_bits(const float (&f)[kPiece])
{
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < kPiece; ++i)
        m = max(m, size_bits(f[i]));
    return m;
}

// Scale of a group whose largest magnitude has these bits: max(a / 448, 2^-126) to within two
// half steps; NaN where the group holds an infinity or NaN, so that the group is NaN as a whole.
__device__ __forceinline__ float scale_of(uint32_t bits)
{
    return bits >= 0x7F800000u ? __uint_as_float(0x7FC00000u)
                               : fmaxf(__uint_as_float(bits) * (1.f / 448.f), 1.17549435e-38f);
}

// Its reciprocal (2^-120 .. 2^126) to within two half steps.
__device__ __forceinline__ float inverse_of(float scale) { return __fdividef(1.f, scale); }

// e4m3 of v * inv, to nearest even. (v / scale passes 448 by fp32 roundings at most, which the
// saturating conversion takes back; NaN gives NaN.)
__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d)
{
    const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
    const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(c, d), __NV_SATFINITE, __NV_E4M3);
    return lo | hi << 16;
}

__device__ __forceinline__ uint2 e4m3x8(const float (&f)[kPiece], float inv)
{
    return make_uint2(e4m3x4(f[0] * inv, f[1] * inv, f[2] * inv, f[3] * inv),
                      e4m3x4(f[4] * inv, f[5] * inv, f[6] * inv, f[7] * inv));
}

// Largest of the values of a half warp (all of its lanes take part).
__device__ __forceinline__ uint32_t half_warp_max(uint32_t v)
{
#pragma unroll
    for (int o = 8; o; o >>= 1)
        v = max(v, __shfl_xor_sync(0xffffffffu, v, o));
    return v;
}

// Codes of piece c of a row's n columns, of a group that lies in this half warp (a piece past
// the row's end counts as zeros), and by the group's first lane its scale.
template <bool VEC>
__device__ __forceinline__ void store_e4m3(uint8_t *q, float *scales, int c, int n, const float (&f)[kPiece])
{
    const float s = scale_of(half_warp_max(size_bits(f)));
    if (c >= n)
        return;
    const uint2 codes = e4m3x8(f, inverse_of(s));
    if (VEC) {
        *reinterpret_cast<uint2 *>(q + c) = codes;
    } else {
#pragma unroll
        for (int i = 0; i < kPiece; ++i)
            if (c + i < n)
                q[c + i] = static_cast<uint8_t>((i < 4 ? codes.x : codes.y) >> (8 * (i & 3)));
    }
    if (c % (kPiece * kGroupPieces) == 0)
        scales[c / (kPiece * kGroupPieces)] = s;
}

}  // namespace rows
}  // namespace ep
