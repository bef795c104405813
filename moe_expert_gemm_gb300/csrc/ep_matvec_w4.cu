// Expert products of a few rows on 4-bit weights: C[m][n] = sum_k W_e[n][k] a[m][k].
//
// Every weight of an expert that has rows is read once and meets a handful of activation
// rows, so the call is bound by the weights' bytes, N*K/2 per expert, as long as the codes
// become multiplicands fast enough. The weights are therefore the 16-row operand of the
// warp's 16x8x16 bf16 matrix instruction and the activation rows its 8 columns: 8 rows
// cost the same unpacking as one.
//
//  * A code becomes an exact bf16 multiple of (q - zero), or of its e2m1 value, in a mask
//    and a fused multiply-add (unpack_int, unpack_e2m1). The sum over a group of k runs in
//    fp32 on these numbers; the group's scale multiplies that sum in fp32, so no weight is
//    ever rounded.
//  * e2m1 scales are powers of two, which the codes can take on exactly in bf16: there a
//    group needs no sum of its own (as long as the scale is at most 2; else it gets one).
//  * The order of k inside a matrix instruction is free. A thread's words of a weight row
//    (as many at once as a scale group of k feeds the four threads of a row) hold 8
//    consecutive codes each, whose halves are the pairs (0,4) (1,5) (2,6) (3,7). Up to 16
//    rows a pass the activations are laid into shared memory in that order, past that the
//    weights' pairs are put in order.
//  * Work is counted in steps of 256 k by 128 * R weight rows (16 KB * R), ordered by
//    expert, column tile, chunk of 8 * NT rows and k, and cut into equal runs, one per
//    thread block, of whole tiles or wherever the cuts fall (Runs). A tile cut between
//    blocks is joined through the workspace: every block leaves its fp32 partial sums
//    there, the last one to arrive adds them in block order.
//  * Thread block: a producer warp streams the weights (TMA, 128-byte swizzle) into a ring
//    of stages; staging warps bring the scales and the activation rows (past 16 rows the
//    producer brings those, by a bulk copy each); eight consumer warps for each of the
//    tile's R parts own 16 weight rows each (8 of the part's first half and 8 of its
//    second: with SwiGLU the gate and the up row of the same output).
#include <cuda_bf16.h>

#include <type_traits>

#include "ep_internal.h"
#include "ep_ptx.cuh"

namespace ep {

namespace {

constexpr int kPartRows = 128;                   // weight rows of a part of a tile
constexpr int kStepK = 256;                      // k of a step: 128 bytes of codes a row
constexpr int kPartBytes = kPartRows * kStepK / 2;
constexpr int kXPitch = kStepK * 2 + 64;         // bytes of an activation row of a step that
                                                 // lies as it is; the padding spreads 8 rows
                                                 // over the banks
constexpr int kPartWarps = 8;                    // consumer warps of a part
constexpr int kMaxStages = 5;
constexpr int kW4MaxBlocks = 320;                // at two blocks an SM
constexpr int kMaxAccs = 16;                     // NT * R at one block an SM
constexpr uint64_t kW4TimeoutNs = 2000000000ull;

// One block's share of one tile: steps [s0, s1).
struct Segment {
    int e, m0, m1, n0;  // expert, its rows [m0, m1), first column
    int s0, s1;
    int first;          // number of the tile's first step
};

// How the steps are cut into the blocks' runs. A tile's steps are kept together as long
// as that costs less than the joining of cut tiles, which takes about as long as
// kJoinSteps steps (1-token down projection of 8 experts, 4096 x 1536 each: 256 whole
// tiles on 256 blocks).
constexpr int kJoinSteps = 3;

struct Runs {
    int per, rest;  // pieces of every run; the first `rest` runs have one more
    int piece;      // steps of a piece: 1, or a tile's

    // The block whose run holds step i (of runs cut at any step).
    __device__ int owner(int i) const
    {
        return i < rest * (per + 1) ? i / (per + 1) : rest + (i - rest * (per + 1)) / per;
    }
};

// Where a block's run begins: the tile (expert, number among its units), its step, and
// the steps to go.
struct Start {
    int e, u, s0, first, todo;
};

struct Shared {
    uint64_t full[kMaxStages], empty[kMaxStages];
    int sums_apart[kMaxStages];  // e2m1: the stage's scales need sums by group
    int skips;                   // rows with a bad gather index were met
    int offsets[EP_MAX_LOCAL_EXPERTS + 1];
    int bad;
    int abort;
    Runs runs;
    Start start;
    Segment cut[2];  // the tiles the block's run begins and ends inside
    int last[2];
};

// The activations of up to 16 rows are laid out by the staging warps.
constexpr bool x_staged(int NT)
{
    return NT <= 2;
}

constexpr int stagers_of(int NT)
{
    return x_staged(NT) ? 3 : 2;
}

constexpr int threads_of(int NT, int R)
{
    return 32 * (1 + stagers_of(NT) + R * kPartWarps);
}

// Blocks of an SM: the widest form needs an SM's registers and shared memory.
constexpr int blocks_per_sm(int R)
{
    return R == 1 ? 2 : 1;
}

// Weights, activations, scales and zero points (both bf16) of a step; a multiple of the
// 1 KB the swizzled weight tiles start on.
constexpr int stage_bytes(int NT, int R, int GS, bool E2M1)
{
    return (R * kPartBytes + NT * 8 * (x_staged(NT) ? kStepK * 2 : kXPitch) +
            R * kPartRows * GS * (E2M1 ? 2 : 4) + 1023) / 1024 * 1024;
}

constexpr int stages_of(int NT, int R, int GS, bool E2M1)
{
    const int n = (226 / blocks_per_sm(R) * 1024 - 1024 - static_cast<int>(sizeof(Shared))) /
                  stage_bytes(NT, R, GS, E2M1);
    return n > kMaxStages ? kMaxStages : n;
}

constexpr int smem_bytes(int NT, int R, int GS, bool E2M1)
{
    return 1024 + stages_of(NT, R, GS, E2M1) * stage_bytes(NT, R, GS, E2M1) +
           static_cast<int>(sizeof(Shared));
}

// The segments of this block's run, one after the other.
template <int CHUNK>
struct Walk {
    int e, u, s0, first, todo;  // the next segment's expert, unit in it, step, ...
    int tile, chunk, chunks;    // of that unit; chunks 0: not yet known
    int steps, tiles;

    __device__ Walk(const W4Params &p, const Shared &sh, int tiles_)
        : e(sh.start.e), u(sh.start.u), s0(sh.start.s0), first(sh.start.first),
          todo(sh.start.todo), tile(0), chunk(0), chunks(0), steps(p.steps), tiles(tiles_)
    {
    }

    __device__ __forceinline__ bool next(const Shared &sh, int tile_cols, Segment &s)
    {
        if (todo <= 0)
            return false;
        if (chunks == 0) {  // the run's first segment
            chunks = static_cast<int>(
                (static_cast<unsigned>(sh.offsets[e + 1] - sh.offsets[e]) + CHUNK - 1) / CHUNK);
            tile = chunks == 1 ? u : u / chunks;
            chunk = u - tile * chunks;
        }
        const int r0 = sh.offsets[e], r1 = sh.offsets[e + 1];
        s.e = e;
        s.m0 = r0 + chunk * CHUNK;
        s.m1 = r1 - s.m0 < CHUNK ? r1 : s.m0 + CHUNK;
        s.n0 = tile * tile_cols;
        s.first = first;
        s.s0 = s0;
        s.s1 = todo < steps - s0 ? s0 + todo : steps;
        todo -= s.s1 - s.s0;
        s0 = 0;
        first += steps;
        if (++chunk == chunks) {
            chunk = 0;
            if (++tile == tiles && todo > 0) {
                tile = 0;
                do {  // the next expert with rows: there is one, as there are steps to go
                    ++e;
                    chunks = static_cast<int>(
                        (static_cast<unsigned>(sh.offsets[e + 1] - sh.offsets[e]) + CHUNK - 1) / CHUNK);
                } while (chunks == 0);
            }
        }
        return true;
    }
};

// Activation row m: in A, or the token the plan names; NULL for a bad gather index.
__device__ __forceinline__ const uint8_t *row_of(const W4Params &p, int m)
{
    if (p.A)
        return p.A + static_cast<int64_t>(m) * p.K * 2;
    // (tokens * top_k of all ranks fit 31 bits)
    const uint32_t gi = static_cast<uint32_t>(__ldg(p.gather_idx + m));
    const uint32_t Tk = static_cast<uint32_t>(p.T) * p.top_k;
    if (gi >= Tk * p.n_ranks)
        return nullptr;
    const uint32_t rk = gi / Tk;
    return p.x[rk] + static_cast<int64_t>((gi - rk * Tk) / p.top_k) * p.K * 2;
}

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
// false) one by one, the ones past `have` left out.
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
        else {
            constexpr int kPer = 4 / sizeof(T);
#pragma unroll
            for (int i = 0; i < kWords; ++i)
                w[i] = 0;
#pragma unroll
            for (int i = 0; i < BYTES / static_cast<int>(sizeof(T)); ++i)
                if (i < have)
                    w[i / kPer] |= static_cast<uint32_t>(__ldg(from + i)) << (8 * sizeof(T) * (i % kPer));
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
#pragma unroll
            for (int i = 0; i < GS; ++i) {
                const uint32_t e = scale.w[i / 4] >> (8 * (i % 4)) & 255;
                // 2^(e - 1), the factor of a code as unpack_e2m1 forms it, or apart from
                // the codes 2^(e - 127) (bf16: the exponent bits; 2^-127 is subnormal)
                const uint32_t h = !apart ? (e + 126) << 7 : e == 255 ? 0x7FC0u : e == 0 ? 0x0040u : e << 7;
                out[i / 2] = i % 2 ? out[i / 2] | h << 16 : h;
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

__device__ __forceinline__ uint32_t bf16x2_mul(uint32_t a, uint32_t b)
{
    uint32_t d;
    asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}

__device__ __forceinline__ uint32_t bf16x2_fma(uint32_t a, uint32_t b, uint32_t c)
{
    uint32_t d;
    asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
    return d;
}

// Halves of words with the codes 0 and 4, and 1 and 5, of eight -> the pairs (0,1), (4,5).
__device__ __forceinline__ void in_order(uint32_t &v04, uint32_t &v15)
{
    const uint32_t v = __byte_perm(v04, v15, 0x5410);
    v15 = __byte_perm(v04, v15, 0x7632);
    v04 = v;
}

// 8 codes -> bf16 pairs, each (code - zero) / 64: (0,4) (1,5) (2,6) (3,7), or IN_ORDER (0,1)
// (2,3) (4,5) (6,7). The low four bits of a bf16 number alone are the subnormal code *
// 2^-133; its bits 4..7 alone are code * 2^-129, subnormal or in the first binade, where
// the spacing is the same. So a mask and one fused multiply-add do it, exactly;
// `minus_zero` is -zero / 64.
template <bool IN_ORDER>
__device__ __forceinline__ void unpack_int(uint32_t w, uint32_t minus_zero, uint32_t (&v)[4])
{
    constexpr uint32_t two127 = 0x7F00u, two123 = 0x7D00u;
    const uint32_t h = w >> 8;
    uint32_t a = w & 0x000F000Fu, b = w & 0x00F000F0u, c = h & 0x000F000Fu, d = h & 0x00F000F0u;
    if (IN_ORDER) {
        in_order(a, b);
        in_order(c, d);
        constexpr uint32_t up = two123 << 16 | two127;
        v[0] = bf16x2_fma(a, up, minus_zero);
        v[1] = bf16x2_fma(c, up, minus_zero);
        v[2] = bf16x2_fma(b, up, minus_zero);
        v[3] = bf16x2_fma(d, up, minus_zero);
    } else {
        v[0] = bf16x2_fma(a, two127 * 0x10001u, minus_zero);
        v[1] = bf16x2_fma(b, two123 * 0x10001u, minus_zero);
        v[2] = bf16x2_fma(c, two127 * 0x10001u, minus_zero);
        v[3] = bf16x2_fma(d, two123 * 0x10001u, minus_zero);
    }
}
constexpr float kIntScale = 64.f;
constexpr uint32_t kTwo126 = 0x7E807E80u;

// e2m1: a code's four bits go to bits 15..12 (for the sign) and 9..6 (exponent and
// mantissa) of its half at once by a multiplication; the number so formed is 2^-126 times
// the code's value. `factor`, in both halves, is 2^126 or that times the scale: with two
// significant bits the product is exact down to the smallest scale.
template <bool IN_ORDER>
__device__ __forceinline__ void unpack_e2m1(uint32_t w, uint32_t factor, uint32_t (&v)[4])
{
    const uint32_t h = w >> 8;
    uint32_t a = (w & 0x000F000Fu) * 0x1040u, b = (w & 0x00F000F0u) * 0x0104u;
    uint32_t c = (h & 0x000F000Fu) * 0x1040u, d = (h & 0x00F000F0u) * 0x0104u;
    if (IN_ORDER) {
        in_order(a, b);
        in_order(c, d);
    }
    v[0] = bf16x2_mul(a & 0x81C081C0u, factor);
    v[IN_ORDER ? 2 : 1] = bf16x2_mul(b & 0x81C081C0u, factor);
    v[IN_ORDER ? 1 : 2] = bf16x2_mul(c & 0x81C081C0u, factor);
    v[3] = bf16x2_mul(d & 0x81C081C0u, factor);
}

__device__ __forceinline__ void mma_bf16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1,
                                         const float (&c)[4])
{
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%10,%11,%12,%13};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(c[0]), "f"(c[1]), "f"(c[2]),
          "f"(c[3]));
}

__device__ __forceinline__ void give_up(const W4Params &p, Shared &sh)
{
    atomicOr(p.status, EP_STATUS_TIMEOUT);
    *reinterpret_cast<volatile int *>(&sh.abort) = 1;
}

// Stores a thread's sums of a whole tile: acc[nt][0..1] are rows 8nt+2q, +1 of its first
// weight row, column n of the tile's results, acc[nt][2..3] of its second.
template <int NT>
__device__ __forceinline__ void store_tile(const W4Params &p, const Segment &s,
                                           const float (&acc)[NT][4], int n, int q, bool skips)
{
    const int cols = p.swiglu ? p.N / 2 : p.N;
    const float back = p.format == EP_W4_INT ? kIntScale : 1.f;
    __nv_bfloat16 *C = reinterpret_cast<__nv_bfloat16 *>(p.C);
    n += s.n0;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int m = s.m0 + 8 * nt + 2 * q + h;
            if (m >= s.m1 || (skips && !row_of(p, m)))
                continue;
            __nv_bfloat16 *out = C + static_cast<int64_t>(m) * cols;
            const float a = acc[nt][h] * back, b = acc[nt][2 + h] * back;
            if (p.swiglu) {
                if (n < cols)
                    out[n] = __float2bfloat16_rn(silu_f32(a) * b);
            } else {
                if (n < cols)
                    out[n] = __float2bfloat16_rn(a);
                if (n + 64 < cols)
                    out[n + 64] = __float2bfloat16_rn(b);
            }
        }
}

}  // namespace

// NT: groups of 8 activation rows a pass over the weights serves. R: parts of a tile. GS:
// scale groups of a step (256 / group size). VEC: K is whole steps, a step's scales one
// aligned piece (W4Params::scale_vec).
template <int NT, int R, int GS, bool E2M1, bool VEC>
__global__ void __launch_bounds__(threads_of(NT, R), blocks_per_sm(R))
    matvec_w4_kernel(const __grid_constant__ CUtensorMap tw, const W4Params p)
{
    constexpr int kConsumers = R * kPartWarps, kStagers = stagers_of(NT);
    constexpr bool kStageX = x_staged(NT);
    constexpr int kStages = stages_of(NT, R, GS, E2M1);
    constexpr int kStage = stage_bytes(NT, R, GS, E2M1);
    constexpr int kXOff = R * kPartBytes;
    constexpr int kScaleOff = kXOff + NT * 8 * (kStageX ? kStepK * 2 : kXPitch);
    constexpr int kZeroOff = kScaleOff + R * kPartRows * GS * 2;
    // Staging warps take turns. One may look at a stage's barrier only when at most one of
    // its phases is open (a wait knows a phase's parity alone), so no more of them take part
    // than there are stages.
    constexpr int kTurns = kStagers < kStages ? kStagers : kStages;
    // Words of a weight row a thread of the row's four takes at once: their 32 * kWords
    // codes belong to one scale group.
    constexpr int kWords = !kStageX || GS == 8 ? 1 : 8 / GS;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *ring = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
    Shared &sh = *reinterpret_cast<Shared *>(ring + kStages * kStage);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

    const int part_cols = p.swiglu ? 64 : kPartRows, tile_cols = R * part_cols;
    const int cols = p.swiglu ? p.N / 2 : p.N;
    if (warp == 1 && lane == 0) {
        tma_prefetch_map(&tw);
        for (int i = 0; i < kStages; ++i) {
            mbar_init(&sh.full[i], 2);  // the producer, a staging warp
            mbar_init(&sh.empty[i], kConsumers);
        }
        fence_mbar_init();
        sh.abort = 0;
        sh.skips = 0;
        sh.cut[0].e = sh.cut[1].e = -1;
    }
    const int tiles = (cols + tile_cols - 1) / tile_cols;
    griddep_launch_dependents();
    griddep_wait();
    if (warp == 0) {
        // units of every expert (chunks of its rows x column tiles), their sums, and from
        // them where this block's run begins
        constexpr int kSets = EP_MAX_LOCAL_EXPERTS / 32;
        int lo[kSets], hi[kSets], upto[kSets];
#pragma unroll
        for (int i = 0; i < kSets; ++i) {
            const int e = 32 * i + lane;
            lo[i] = e < p.El ? __ldg(p.expert_offsets + e) : 0;
            hi[i] = e < p.El ? __ldg(p.expert_offsets + e + 1) : 0;
        }
        int units = 0;
        bool bad = false;
#pragma unroll
        for (int i = 0; i < kSets; ++i) {
            upto[i] = 0;
            if (32 * i >= p.El)
                break;
            bad |= lo[i] < 0 || hi[i] < lo[i] || hi[i] > p.max_rows;
            int sum = static_cast<int>((static_cast<unsigned>(hi[i] - lo[i]) + 8 * NT - 1) / (8 * NT)) * tiles;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int v = __shfl_up_sync(0xffffffffu, sum, o);
                if (lane >= o)
                    sum += v;
            }
            upto[i] = units + sum;
            units = __shfl_sync(0xffffffffu, upto[i], 31);
        }
        bad = __any_sync(0xffffffffu, bad);
        const int grid = static_cast<int>(gridDim.x), block = static_cast<int>(blockIdx.x);
        const int total = units * p.steps;
        const bool whole = (units + grid - 1) / grid * p.steps <= (total + grid - 1) / grid + kJoinSteps;
        Runs runs;
        runs.piece = whole ? p.steps : 1;
        runs.per = (whole ? units : total) / grid;
        runs.rest = (whole ? units : total) - runs.per * grid;
        const int at = (block * runs.per + (block < runs.rest ? block : runs.rest)) * runs.piece;
        const int todo = (runs.per + (block < runs.rest)) * runs.piece;
        const int unit = at / p.steps;
#pragma unroll
        for (int i = 0; i < kSets; ++i) {
            if (32 * i >= p.El)
                break;
            const int e = 32 * i + lane;
            if (e < p.El) {
                sh.offsets[e] = lo[i];
                if (e == p.El - 1)
                    sh.offsets[p.El] = hi[i];
            }
        }
        if (lane == 0) {
            sh.bad = bad;
            sh.runs = runs;
            if (bad && block == 0)
                atomicOr(p.status, EP_STATUS_BOUNDS);
        }
        // the expert whose units hold `unit`
        int base = 0;
#pragma unroll
        for (int i = 0; i < kSets; ++i) {
            if (32 * i >= p.El)
                break;
            const int up = __shfl_up_sync(0xffffffffu, upto[i], 1);
            const int from = lane == 0 ? base : up;
            if (from <= unit && unit < upto[i])
                sh.start = Start{32 * i + lane, unit - from, at - unit * p.steps, unit * p.steps, todo};
            base = __shfl_sync(0xffffffffu, upto[i], 31);
        }
        if (lane == 0 && unit >= units)
            sh.start.todo = 0;
    }
    __syncthreads();
    if (sh.bad)
        return;

    volatile int *abort_flag = &sh.abort;
    Walk<8 * NT> walk(p, sh, tiles);
    Segment seg;
    int stage = 0;
    uint32_t phase = 0;
    auto advance = [&] {
        if (++stage == kStages) {
            stage = 0;
            phase ^= 1;
        }
    };

    if (warp == 0) {
        // --------------------- producer: weights (and, where not staged, activation rows)
        constexpr int kSets = kStageX ? 0 : (NT + 3) / 4;
        int issued = 0;
        bool ok = true;
        while (ok && walk.next(sh, tile_cols, seg)) {
            const int rows = seg.m1 - seg.m0;
            const uint8_t *mine[kSets + 1];  // rows lane, lane + 32 of the segment
            int found = 0;
#pragma unroll
            for (int i = 0; i < kSets; ++i) {
                mine[i] = 32 * i + lane < rows ? row_of(p, seg.m0 + 32 * i + lane) : nullptr;
                if (32 * i + lane < rows && !mine[i]) {
                    atomicOr(p.status, EP_STATUS_BOUNDS);
                    sh.skips = 1;
                }
                found += __popc(__ballot_sync(0xffffffffu, mine[i] != nullptr));
            }
            __syncwarp();
            const int y0 = seg.e * p.N + seg.n0;
            const int to_up = p.swiglu ? cols : 64;
            for (int k = seg.s0; k < seg.s1; ++k) {
                ok = __all_sync(0xffffffffu, mbar_wait(&sh.empty[stage], phase ^ 1, kW4TimeoutNs,
                                                       abort_flag));
                if (!ok)
                    break;
                uint8_t *dst = ring + stage * kStage;
                const uint32_t x_bytes =
                    VEC || k * kStepK + kStepK <= p.K ? kStepK * 2 : (p.K - k * kStepK) * 2;
                if (lane == 0) {
                    mbar_arrive_expect_tx(&sh.full[stage], R * kPartBytes + found * x_bytes);
#pragma unroll
                    for (int r = 0; r < R; ++r) {
                        tma_load_2d(dst + r * kPartBytes, &tw, &sh.full[stage], k * (kStepK / 2),
                                    y0 + r * part_cols);
                        tma_load_2d(dst + r * kPartBytes + kPartBytes / 2, &tw, &sh.full[stage],
                                    k * (kStepK / 2), y0 + r * part_cols + to_up);
                    }
                }
                __syncwarp();
#pragma unroll
                for (int i = 0; i < kSets; ++i)
                    if (mine[i])
                        bulk_load(dst + kXOff + (32 * i + lane) * kXPitch, mine[i] + k * (kStepK * 2),
                                  x_bytes, &sh.full[stage]);
                ++issued;
                advance();
            }
        }
        if (!ok && lane == 0) {
            give_up(p, sh);
            // the copies in flight land before the block's shared memory goes away
            volatile int no_abort = 0;
            for (int i = issued > kStages ? issued - kStages : 0; i < issued; ++i)
                mbar_wait(&sh.full[i % kStages], (i / kStages) & 1, 1000000, &no_abort);
        }
        return;
    }

    if (warp <= kStagers) {
        // -------------- staging: scales and zero points, up to 16 rows' activations
        if (warp > kTurns)
            return;
        int turn = warp - 1;  // steps until this warp's next
        constexpr int kRowSets = R * kPartRows / 32;
        constexpr int kBatch = kStageX ? 4 : 1;  // activation rows under way at once
        const int groups = p.K / (kStepK / GS);
        // where a lane's piece (8 activations, in pair order) of a row goes: the place of the
        // thread (row, q) that takes word w of its codes of block b
        const int b = lane / (4 * kWords) * kWords + lane % kWords, q = lane / kWords % 4;
        bool ok = true;
        while (ok && walk.next(sh, tile_cols, seg)) {
            const int rows = seg.m1 - seg.m0;
            unsigned long long mine = 0;  // lane i: where the segment's row i lies
            if (kStageX && lane < rows) {
                mine = reinterpret_cast<unsigned long long>(row_of(p, seg.m0 + lane));
                if (!mine) {
                    atomicOr(p.status, EP_STATUS_BOUNDS);
                    sh.skips = 1;
                }
            }
            // where this lane's weight rows have their scales (rows past the last column
            // take the last one's: nobody stores what comes of them)
            int64_t scale_at[kRowSets];
#pragma unroll
            for (int i = 0; i < kRowSets; ++i) {
                const int r = 32 * i + lane, part = r / kPartRows, in = r % kPartRows;
                int n = seg.n0 + part * part_cols + (p.swiglu ? in % 64 : in);
                n = n < cols ? n : cols - 1;
                scale_at[i] = (static_cast<int64_t>(seg.e) * p.N + n +
                               (p.swiglu && in >= 64 ? cols : 0)) * groups;
            }
            for (int k = seg.s0; k < seg.s1; ++k, turn = turn == 0 ? kTurns - 1 : turn - 1) {
                if (turn != 0) {
                    advance();
                    continue;
                }
                // all loads first, then the wait for the stage, then the stores
                Scales<GS, E2M1, VEC> sc[kRowSets];
#pragma unroll
                for (int i = 0; i < kRowSets; ++i)
                    sc[i].load(p, scale_at[i] + k * GS, groups - k * GS);
                const int k0 = k * kStepK + lane * 8;
                uint4 v[kBatch];
                auto load_rows = [&](int r0) {
#pragma unroll
                    for (int i = 0; i < kBatch; ++i) {
                        if (r0 + i >= rows)
                            break;
                        const uint4 *from = reinterpret_cast<const uint4 *>(
                            __shfl_sync(0xffffffffu, mine, r0 + i));
                        v[i] = make_uint4(0, 0, 0, 0);
                        if (from && (VEC || k0 < p.K))
                            v[i] = __ldg(from + k0 / 8);
                    }
                };
                if (kStageX)
                    load_rows(0);
                ok = __all_sync(0xffffffffu, mbar_wait(&sh.empty[stage], phase ^ 1, kW4TimeoutNs,
                                                       abort_flag));
                if (!ok)
                    break;
                uint8_t *dst = ring + stage * kStage;
                // (columns of the matrix instruction past the last row hold whatever they held:
                // they only reach results that nobody stores)
                for (int r0 = 0; kStageX && r0 < rows; r0 += kBatch) {
                    if (r0)
                        load_rows(r0);
#pragma unroll
                    for (int i = 0; i < kBatch; ++i) {
                        if (r0 + i >= rows)
                            break;
                        const int row = r0 + i, to = (b * NT + row / 8) * 32 + row % 8 * 4 + q;
                        *reinterpret_cast<uint4 *>(dst + kXOff + to * 16) = make_uint4(
                            __byte_perm(v[i].x, v[i].z, 0x5410), __byte_perm(v[i].x, v[i].z, 0x7632),
                            __byte_perm(v[i].y, v[i].w, 0x5410), __byte_perm(v[i].y, v[i].w, 0x7632));
                    }
                }
                bool apart = false;
                if (E2M1) {
#pragma unroll
                    for (int i = 0; i < kRowSets; ++i)
                        apart |= sc[i].large();
                    apart = __any_sync(0xffffffffu, apart);
                    if (lane == 0)
                        sh.sums_apart[stage] = apart;
                }
#pragma unroll
                for (int i = 0; i < kRowSets; ++i) {
                    const int r = 32 * i + lane;
                    sc[i].store(dst + kScaleOff + r * GS * 2, dst + kZeroOff + r * GS * 2, apart);
                }
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(&sh.full[stage]);
                advance();
            }
        }
        if (!ok && lane == 0)
            give_up(p, sh);
        return;
    }

    // ------------------------------------------------------------------ consumers
    const int cw = warp - 1 - kStagers, g = lane >> 2, q = lane & 3;
    const int part_of = cw / kPartWarps, row = 8 * (cw % kPartWarps) + g;  // in each half of it
    const int ctid = cw * 32 + lane;
    // this thread's first words of a weight row, in the 128-byte swizzle (the 16-byte piece i
    // of row r is at i ^ r % 8)
    const int at0 = part_of * kPartBytes + row * 128 + ((q * kWords / 4 ^ g) << 4) + q * kWords % 4 * 4;
    const int scale0 = kScaleOff + (part_of * kPartRows + row) * GS * 2;
    const int zero0 = scale0 + kZeroOff - kScaleOff;
    float *partial = reinterpret_cast<float *>(p.workspace + kW4MaxBlocks * 16);
    constexpr int64_t kSlot = kConsumers * 32 * NT * 4;  // floats of one partial tile
    int *counters = reinterpret_cast<int *>(p.workspace);
    bool ok = true;
    while (walk.next(sh, tile_cols, seg)) {
        const int nts = (seg.m1 - seg.m0 + 7) / 8;
        float acc[NT][4];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int i = 0; i < 4; ++i)
                acc[nt][i] = 0.f;
        for (int k = seg.s0; k < seg.s1; ++k) {
            ok = __all_sync(0xffffffffu,
                            mbar_wait(&sh.full[stage], phase, kW4TimeoutNs, abort_flag));
            if (!ok)
                break;
            const uint8_t *src = ring + stage * kStage;
            const int blocks = VEC || (k + 1) * kStepK <= p.K ? 8 : (p.K - k * kStepK) / 32;
            // a row's scales and zero points as words of two; where registers are short
            // (NT = 8) they are fetched one by one instead
            constexpr bool kScalesAtOnce = NT < 8;
            alignas(16) uint32_t scale[2][GS / 2], zero[2][GS / 2] = {};
            if constexpr (kScalesAtOnce) {
                copy_words<GS / 2>(scale[0], src + scale0);
                copy_words<GS / 2>(scale[1], src + scale0 + 64 * GS * 2);
                if constexpr (!E2M1) {
                    copy_words<GS / 2>(zero[0], src + zero0);
                    copy_words<GS / 2>(zero[1], src + zero0 + 64 * GS * 2);
                }
            }
            auto scale_of = [&](int h, int gr) {
                if constexpr (kScalesAtOnce)
                    return __uint_as_float(gr & 1 ? scale[h][gr / 2] & 0xFFFF0000u : scale[h][gr / 2] << 16);
                else
                    return __uint_as_float(static_cast<uint32_t>(*reinterpret_cast<const uint16_t *>(
                                               src + scale0 + (h * 64 * GS + gr) * 2)) << 16);
            };
            // in both halves of a word
            auto twice = [&](const uint32_t (&words)[2][GS / 2], int at, int h, int gr) {
                if constexpr (kScalesAtOnce)
                    return __byte_perm(words[h][gr / 2], 0u, gr & 1 ? 0x3232u : 0x1010u);
                else
                    return *reinterpret_cast<const uint16_t *>(src + at + (h * 64 * GS + gr) * 2) * 0x10001u;
            };
            // The step's 8 blocks of 32 k. APART: a group's sum is formed on its own and
            // scaled after; else the codes take on their scales.
            auto step = [&](auto apart_) {
                constexpr bool APART = decltype(apart_)::value;
                float part[NT][4];
#pragma unroll
                for (int b0 = 0; b0 < 8; b0 += kWords) {
                    if (!VEC && b0 >= blocks)
                        break;
                    alignas(16) uint32_t w[2][kWords];
#pragma unroll
                    for (int h = 0; h < 2; ++h)
                        copy_words<kWords>(w[h], src + h * (kPartBytes / 2) + (at0 ^ (b0 << 4)));
#pragma unroll
                    for (int j = 0; j < kWords; ++j) {
                        const int b = b0 + j, gr = b * GS / 8;
                        const bool first = APART && (b * GS % 8 == 0 || GS == 8);
                        const bool last = APART && ((b + 1) * GS % 8 == 0 || GS == 8);
                        uint32_t a[2][4];
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            if constexpr (E2M1)
                                unpack_e2m1<!kStageX>(w[h][j], APART ? kTwo126 : twice(scale, scale0, h, gr),
                                                      a[h]);
                            else
                                unpack_int<!kStageX>(w[h][j], twice(zero, zero0, h, gr), a[h]);
                        }
                        const float s0 = last ? scale_of(0, gr) : 0.f, s1 = last ? scale_of(1, gr) : 0.f;
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) {
                            // (two at a time: an odd last one costs less than a check each)
                            if (nt > 0 && nt % 2 == 0 && nt >= nts)
                                break;
                            const uint4 x = *reinterpret_cast<const uint4 *>(
                                kStageX ? src + kXOff + ((b * NT + nt) * 32 + lane) * 16
                                        : src + kXOff + (nt * 8 + g) * kXPitch + b * 64 + q * 16);
                            float(&d)[4] = APART ? part[nt] : acc[nt];
                            const float none[4] = {0.f, 0.f, 0.f, 0.f};
                            if (first)
                                mma_bf16(d, a[0][0], a[1][0], a[0][1], a[1][1], x.x, x.y, none);
                            else
                                mma_bf16(d, a[0][0], a[1][0], a[0][1], a[1][1], x.x, x.y, d);
                            mma_bf16(d, a[0][2], a[1][2], a[0][3], a[1][3], x.z, x.w, d);
                            if (last) {
                                acc[nt][0] = fmaf(s0, part[nt][0], acc[nt][0]);
                                acc[nt][1] = fmaf(s0, part[nt][1], acc[nt][1]);
                                acc[nt][2] = fmaf(s1, part[nt][2], acc[nt][2]);
                                acc[nt][3] = fmaf(s1, part[nt][3], acc[nt][3]);
                            }
                        }
                    }
                }
            };
            if (!E2M1 || sh.sums_apart[stage])
                step(std::true_type{});
            else
                step(std::false_type{});
            // the copy that refills the stage goes through the async proxy: without this
            // fence reads of the stage may still be under way when it lands
            fence_proxy_async_shared();
            __syncwarp();
            if (lane == 0)
                mbar_arrive(&sh.empty[stage]);
            advance();
        }
        if (!ok)
            break;
        if (seg.s0 == 0 && seg.s1 == walk.steps) {
            store_tile<NT>(p, seg, acc, part_of * part_cols + row, q, sh.skips);
            continue;
        }
        // a cut tile: leave the sums in the block's slot for the tile its run begins
        // inside (0) or ends inside (1)
        const int slot = seg.s0 == 0 ? 1 : 0;
        float4 *mine = reinterpret_cast<float4 *>(partial + (blockIdx.x * 2 + slot) * kSlot);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
            if (nt < nts)
                __stcg(mine + nt * kConsumers * 32 + ctid,
                       make_float4(acc[nt][0], acc[nt][1], acc[nt][2], acc[nt][3]));
        if (ctid == 0)
            sh.cut[slot] = seg;
    }
    // The cut tiles, after all else: of a tile's blocks the last one to come here adds
    // the sums of all of them, in block order. A warp that gave up takes all consumers
    // with it here, where they meet first.
    if (!ok && lane == 0)
        give_up(p, sh);
    if (sh.runs.piece > 1)
        return;  // runs of whole tiles
    // (the barrier orders the block's partial sums before the release of one thread)
    if (!named_bar_and(1, kConsumers * 32, ok))
        return;
    if (cw < 2 && lane == 0) {
        const Segment &cut = sh.cut[cw];
        int last = 0;
        if (cut.e >= 0) {
            const int c0 = sh.runs.owner(cut.first), c1 = sh.runs.owner(cut.first + walk.steps - 1);
            last = atom_add_acq_rel_gpu(counters + c0, 1) == c1 - c0;
            if (last)
                counters[c0] = 0;  // ready for the next call
        }
        sh.last[cw] = last;
    }
    named_bar_sync(1, kConsumers * 32);
    for (int slot = 0; slot < 2; ++slot) {
        if (!sh.last[slot])
            continue;
        seg = sh.cut[slot];
        const int nts = (seg.m1 - seg.m0 + 7) / 8;
        const int c0 = sh.runs.owner(seg.first), c1 = sh.runs.owner(seg.first + walk.steps - 1);
        float acc[NT][4] = {};
        for (int c = c0; c <= c1; ++c) {
            const float4 *theirs =
                reinterpret_cast<const float4 *>(partial + (c * 2 + (c == c0 ? 1 : 0)) * kSlot);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
                if (nt < nts) {
                    const float4 v = __ldcg(theirs + nt * kConsumers * 32 + ctid);
                    acc[nt][0] += v.x;
                    acc[nt][1] += v.y;
                    acc[nt][2] += v.z;
                    acc[nt][3] += v.w;
                }
        }
        store_tile<NT>(p, seg, acc, part_of * part_cols + row, q, sh.skips);
    }
}

int64_t w4_workspace_bytes()
{
    // counters, and two partial tiles a block: NT <= 4 at two blocks an SM, or
    // NT * R <= kMaxAccs at one
    return kW4MaxBlocks * 16 + kW4MaxBlocks / 2 * 2ll * kPartWarps * 32 * kMaxAccs * 16;
}

template <int NT, int R, int GS, bool E2M1, bool VEC>
static cudaError_t launch_w4(const CUtensorMap &tw, const W4Params &p, int num_sms, cudaStream_t s)
{
    static_assert(NT * R * blocks_per_sm(R) <= kMaxAccs, "the workspace is too small");
    const auto kern = matvec_w4_kernel<NT, R, GS, E2M1, VEC>;
    constexpr int smem = smem_bytes(NT, R, GS, E2M1), most = kW4MaxBlocks / 2 * blocks_per_sm(R);
    const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess)
        return e;
    const int grid = blocks_per_sm(R) * num_sms;
    return launch_behind(kern, grid < most ? grid : most, threads_of(NT, R), smem, s, tw, p);
}

template <int NT, int R, bool VEC>
static cudaError_t launch_nt(const CUtensorMap &tw, const W4Params &p, int num_sms, cudaStream_t s)
{
    if (p.format == EP_W4_E2M1)
        return launch_w4<NT, R, 8, true, VEC>(tw, p, num_sms, s);
    switch (p.group) {
    case 32:
        return launch_w4<NT, R, 8, false, VEC>(tw, p, num_sms, s);
    case 64:
        return launch_w4<NT, R, 4, false, VEC>(tw, p, num_sms, s);
    default:
        return launch_w4<NT, R, 2, false, VEC>(tw, p, num_sms, s);
    }
}

template <bool VEC>
static cudaError_t launch_vec(const CUtensorMap &tw, const W4Params &p, int num_sms, cudaStream_t s)
{
    // rows a pass serves: what an expert is expected to get, at most what it can get
    const int64_t tokens = static_cast<int64_t>(p.T) * p.n_ranks;
    int64_t rows = (tokens * p.top_k + static_cast<int64_t>(p.n_ranks) * p.El - 1) /
                   (static_cast<int64_t>(p.n_ranks) * p.El);
    rows = rows < p.max_rows ? rows : p.max_rows;
    if (rows <= 8)
        return launch_nt<1, 1, VEC>(tw, p, num_sms, s);
    if (rows <= 16)
        return launch_nt<2, 1, VEC>(tw, p, num_sms, s);
    return launch_nt<8, 2, VEC>(tw, p, num_sms, s);
}

cudaError_t launch_matvec_w4(const CUtensorMap &tw, const W4Params &p, int num_sms, cudaStream_t s)
{
    return p.scale_vec ? launch_vec<true>(tw, p, num_sms, s) : launch_vec<false>(tw, p, num_sms, s);
}

}  // namespace ep
