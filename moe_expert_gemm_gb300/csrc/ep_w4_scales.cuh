// Scales and zero points of the 4-bit expert products on their way from global memory, as
// they lie there, to a stage of shared memory, as bf16 numbers.
#pragma once

#include "ep_w4.cuh"

namespace ep {
namespace w4 {

// N 32-bit words at once (N = 1, 2 or 4), to or from shared memory.
template <int N>
__device__ __forceinline__ void copy_words(void *dst, const void *src)
{
    if constexpr (N == 1)
        *static_cast<uint32_t *>(dst) = *static_cast<const uint32_t *>(src);
    else if constexpr (N == 2)
        *static_cast<uint2 *>(dst) = *static_cast<const uint2 *>(src);
    else
        *static_cast<uint4 *>(dst) = *static_cast<const uint4 *>(src);
}

// GS bytes or halves from global memory as they lie there: one aligned load, or (VEC
// false) by words of which each holds at least one of the `have` that exist; what stands
// past those is anything.
template <int BYTES, bool VEC>
struct Piece {
    static constexpr int kWords = (BYTES + 3) / 4;
    uint32_t w[kWords];

    template <typename T>
    __device__ __forceinline__ void load(const T *from, int have)
    {
        if constexpr (VEC && BYTES == 16)
            *this = from_uint4(__ldg(reinterpret_cast<const uint4 *>(from)));
        else if constexpr (VEC && BYTES == 8) {
            const uint2 v = __ldg(reinterpret_cast<const uint2 *>(from));
            w[0] = v.x, w[1] = v.y;
        } else if constexpr (VEC && BYTES == 4)
            w[0] = __ldg(reinterpret_cast<const uint32_t *>(from));
        else if constexpr (VEC)
            w[0] = __ldg(reinterpret_cast<const unsigned short *>(from));
        else {  // the aligned words that hold some of it, shifted into place
            const uint64_t at = reinterpret_cast<uint64_t>(from);
            const uint32_t *word = reinterpret_cast<const uint32_t *>(at & ~3ull);
            const int skip = static_cast<int>(at & 3), end = skip + static_cast<int>(sizeof(T)) * have;
            uint32_t in[kWords + 1];
#pragma unroll
            for (int i = 0; i <= kWords; ++i) {
                in[i] = 0;
                if (4 * i < end && (i < kWords || skip > 0))
                    in[i] = __ldg(word + i);
            }
#pragma unroll
            for (int i = 0; i < kWords; ++i)
                w[i] = __funnelshift_r(in[i], in[i + 1], 8 * skip);
        }
    }

    static __device__ __forceinline__ Piece from_uint4(uint4 v)
    {
        Piece r;
        r.w[0] = v.x, r.w[1] = v.y, r.w[2] = v.z, r.w[3] = v.w;
        return r;
    }
};

// A weight row's scales and zero points of one step, on their way to shared memory as GS
// bf16 numbers each. Nothing is done with them between load and store, so that the loads
// of several rows are under way at once.
template <int GS, bool E2M1, bool VEC>
struct Scales {
    Piece<E2M1 ? GS : 2 * GS, VEC> scale;
    Piece<GS, VEC> zero;

    // `have` of the step's groups exist, from index `at` on.
    __device__ __forceinline__ void load(const W4Params &p, int64_t at, int have)
    {
        if constexpr (E2M1) {
            scale.load(static_cast<const uint8_t *>(p.scales) + at, have);
            if (!VEC) {  // (none past the last group, as large() looks at all)
#pragma unroll
                for (int i = 0; i < scale.kWords; ++i)
                    scale.w[i] &= have >= 4 * i + 4 ? ~0u : have <= 4 * i ? 0u : ~(~0u << 8 * (have - 4 * i));
            }
        } else {
            scale.load(static_cast<const unsigned short *>(p.scales) + at, have);
            if (p.zeros)
                zero.load(p.zeros + at, have);
            else
#pragma unroll
                for (int i = 0; i < zero.kWords; ++i)
                    zero.w[i] = 0x08080808u;
        }
    }

    // e2m1: whether a scale is too large for the codes to take on.
    __device__ __forceinline__ bool large() const
    {
        uint32_t most = 0;
        if constexpr (E2M1) {
#pragma unroll
            for (int i = 0; i < GS; ++i)
                most = max(most, scale.w[i / 4] >> (8 * (i % 4)) & 255);
        }
        return most > 128;
    }

    __device__ __forceinline__ void store(uint8_t *to_scale, uint8_t *to_zero, bool apart) const
    {
        alignas(16) uint32_t out[GS / 2];
        if constexpr (E2M1) {
            // 2^(e - 1), the factor of a code as unpack_e2m1 forms it, or apart from the
            // codes 2^(e - 127) (bf16: the exponent bits; 2^-127 is subnormal)
            if (!apart) {  // two at a time: e + 126 has eight bits
#pragma unroll
                for (int i = 0; i < GS / 2; ++i)
                    out[i] = (__byte_perm(scale.w[i / 2], 0, i % 2 ? 0x4342 : 0x4140) + 0x007E007Eu) << 7;
            } else {
#pragma unroll
                for (int i = 0; i < GS; ++i) {
                    const uint32_t e = scale.w[i / 4] >> (8 * (i % 4)) & 255;
                    const uint32_t h = e == 255 ? 0x7FC0u : e == 0 ? 0x0040u : e << 7;
                    out[i / 2] = i % 2 ? out[i / 2] | h << 16 : h;
                }
            }
            copy_words<GS / 2>(to_scale, out);
        } else {
#pragma unroll
            for (int i = 0; i < GS / 2; ++i)
                out[i] = scale.w[i];
            copy_words<GS / 2>(to_scale, out);
#pragma unroll
            for (int i = 0; i < GS; ++i) {  // -zero / 64: small integers, exact
                const float z = static_cast<float>(zero.w[i / 4] >> (8 * (i % 4)) & 15) * -0.015625f;
                const uint32_t h = __float_as_uint(z) >> 16;
                out[i / 2] = i % 2 ? out[i / 2] | h << 16 : h;
            }
            copy_words<GS / 2>(to_zero, out);
        }
    }
};

}  // namespace w4
}  // namespace ep
