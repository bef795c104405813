// Rows in pieces of eight values: loads and stores in fp32 and bf16, arithmetic two values at a
// time, and the quantisation of 128 columns to e4m3 with one scale.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp8.h>

#include <cstdint>

namespace ep {
namespace rows {

constexpr int kPiece = 8;         // values of a piece
constexpr int kGroupPieces = 16;  // pieces of a scale's 128 columns: half a warp

// Two fp32 values, as the packed instructions take them; each is rounded on its own.
using Two = uint64_t;

__device__ __forceinline__ Two two(float lo, float hi)
{
    Two t;
    asm("mov.b64 %0, {%1, %2};" : "=l"(t) : "f"(lo), "f"(hi));
    return t;
}

__device__ __forceinline__ void split(Two t, float &lo, float &hi)
{
    asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(t));
}

__device__ __forceinline__ float sum_of(Two t)
{
    float lo, hi;
    split(t, lo, hi);
    return lo + hi;
}

__device__ __forceinline__ Two add2(Two a, Two b)
{
    Two d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}

__device__ __forceinline__ Two mul2(Two a, Two b)
{
    Two d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}

__device__ __forceinline__ Two fma2(Two a, Two b, Two c)
{
    Two d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
}

// A piece's values.
struct Piece {
    Two v[4];
};

__device__ __forceinline__ Piece zeros()
{
    return Piece{{0, 0, 0, 0}};
}

__device__ __forceinline__ Two two_of(uint32_t bf16x2)
{
    return two(__uint_as_float(bf16x2 << 16), __uint_as_float(bf16x2 & 0xFFFF0000u));
}

__device__ __forceinline__ Piece unpack(const uint4 &v)
{
    return Piece{{two_of(v.x), two_of(v.y), two_of(v.z), two_of(v.w)}};
}

__device__ __forceinline__ uint32_t pack(float lo, float hi)
{
    const __nv_bfloat162 b = __float22bfloat162_rn(make_float2(lo, hi));
    return *reinterpret_cast<const uint32_t *>(&b);
}

__device__ __forceinline__ uint32_t pack(Two t)
{
    float lo, hi;
    split(t, lo, hi);
    return pack(lo, hi);
}

__device__ __forceinline__ uint4 pack(const Piece &p)
{
    return make_uint4(pack(p.v[0]), pack(p.v[1]), pack(p.v[2]), pack(p.v[3]));
}

__device__ __forceinline__ Piece piece_of(const float4 &a, const float4 &b)
{
    return Piece{{two(a.x, a.y), two(a.z, a.w), two(b.x, b.y), two(b.z, b.w)}};
}

__device__ __forceinline__ void values_of(const Piece &p, float (&f)[kPiece])
{
#pragma unroll
    for (int i = 0; i < 4; ++i)
        split(p.v[i], f[2 * i], f[2 * i + 1]);
}

// Values c .. c+7 of a row of n at `base`, of any alignment (0 past the row's end).
__device__ __forceinline__ Piece load_any(const uint8_t *base, bool bf16, int c, int n)
{
    float f[kPiece];
#pragma unroll
    for (int i = 0; i < kPiece; ++i) {
        f[i] = 0.f;
        if (c + i < n)
            f[i] = bf16 ? __bfloat162float(reinterpret_cast<const __nv_bfloat16 *>(base)[c + i])
                        : reinterpret_cast<const float *>(base)[c + i];
    }
    return Piece{{two(f[0], f[1]), two(f[2], f[3]), two(f[4], f[5]), two(f[6], f[7])}};
}

// Whole pieces, 16-byte aligned, of global memory.
__device__ __forceinline__ void store_piece(uint8_t *base, bool bf16, int c, const Piece &p)
{
    if (bf16) {
        *reinterpret_cast<uint4 *>(base + c * 2) = pack(p);
    } else {
        float f[kPiece];
        values_of(p, f);
        uint8_t *const to = base + c * 4;
        if ((reinterpret_cast<uintptr_t>(base) & 31) == 0) {  // a whole sector at once
            asm volatile("st.global.v8.f32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(to), "f"(f[0]), "f"(f[1]),
                         "f"(f[2]), "f"(f[3]), "f"(f[4]), "f"(f[5]), "f"(f[6]), "f"(f[7]));
        } else {
            *reinterpret_cast<float4 *>(to) = make_float4(f[0], f[1], f[2], f[3]);
            *reinterpret_cast<float4 *>(to + 16) = make_float4(f[4], f[5], f[6], f[7]);
        }
    }
}

// SiLU(x) * u. The quotient by the fast division (error 2 units in the last place), of quarters, as it gives
// 0 where the divisor passes 2^126. (0 where e^-x leaves fp32, below -88.7, where the value is under 2^-121.)
__device__ __forceinline__ float silu_times(float x, float u)
{
    return __fdividef(0.25f * x, fmaf(0.25f, expf(-x), 0.25f)) * u;
}

// The bits of |v|: as integers they order finite values, infinities and NaN in that order.
__device__ __forceinline__ uint32_t size_bits(float v) { return __float_as_uint(v) & 0x7FFFFFFFu; }

// max(|a|, |b|, |c|), NaN if one of them is.
__device__ __forceinline__ float max_size(float a, float b, float c)
{
    float d;
    asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}

__device__ __forceinline__ uint32_t size_bits(const Piece &p)
{
    float f[kPiece], m = 0.f;
    values_of(p, f);
#pragma unroll
    for (int i = 0; i < kPiece; i += 2)
        m = max_size(m, f[i], f[i + 1]);
    return size_bits(m);
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

__device__ __forceinline__ uint2 e4m3x8(const Piece &p, float inv)
{
    const Two i = two(inv, inv);
    float f[kPiece];
    values_of(Piece{{mul2(p.v[0], i), mul2(p.v[1], i), mul2(p.v[2], i), mul2(p.v[3], i)}}, f);
    return make_uint2(e4m3x4(f[0], f[1], f[2], f[3]), e4m3x4(f[4], f[5], f[6], f[7]));
}

// Largest of the values of a half warp (all of its lanes take part).
__device__ __forceinline__ uint32_t half_warp_max(uint32_t v)
{
#pragma unroll
    for (int o = 8; o; o >>= 1)
        v = max(v, __shfl_xor_sync(0xffffffffu, v, o));
    return v;
}

// Codes of piece c of a row's n columns, of a group that lies in this half warp (values past the
// row's end are zeros), and by the group's first lane its scale.
__device__ __forceinline__ uint2 quantise(const Piece &p, float *scales, int c, int n)
{
    const float s = scale_of(half_warp_max(size_bits(p)));
    if (c < n && c % (kPiece * kGroupPieces) == 0)
        scales[c / (kPiece * kGroupPieces)] = s;
    return e4m3x8(p, inverse_of(s));
}

}  // namespace rows
}  // namespace ep
