// What the two kernels of the 4-bit expert products share: how the work is cut into the
// thread blocks' runs, how codes become multiplicands, how a tile's sums are stored and
// tiles cut between blocks joined.
//
// Work is counted in steps of 256 k by a tile of weight rows, ordered by expert, column
// tile, chunk of activation rows and k, and cut into equal runs, one per thread block, of
// whole tiles or wherever the cuts fall (Runs). A tile cut between blocks is joined through
// the workspace: every block leaves its fp32 partial sums there, the last one to arrive
// adds them in block order.
#pragma once

#include <cuda_bf16.h>

#include "ep_internal.h"
#include "ep_ptx.cuh"

namespace ep {
namespace w4 {

constexpr int kPartRows = 128;     // weight rows of a part of a tile
constexpr int kStepK = 256;        // k of a step: 128 bytes of codes a row
constexpr int kMaxBlocks = 320;    // at two blocks an SM
constexpr int kPartThreads = 256;  // that hold the sums of a part

// One block's share of one tile: steps [s0, s1).
struct Segment {
    int e, m0, m1, n0;  // expert, its rows [m0, m1), first column
    int s0, s1;
    int first;          // number of the tile's first step
};

// How the steps are cut into the blocks' runs. A tile's steps are kept together as long
// as that costs less than the joining of cut tiles, which takes about as long as
// kJoinSteps steps. Measured, whole tiles against cut ones (steps of the longest run):
//   one token, 8 experts of 4096 x 1536:      11.9 us (6)  against 14.5 (5.1)
//   11 tokens, 32 experts of 4096 x 2048:     29.9 us (32) against 32.3 (27)
//   one token, 8 experts of 4096 x 7168:      31.7 us (56) against 32.8 (47)
//   5 tokens, one matrix of 4096 x 14336:     60.8 us (56) against 17.3 (5.9)
constexpr int kJoinSteps = 9;

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

// What a block knows of its run, in shared memory.
struct RunInfo {
    int offsets[EP_MAX_LOCAL_EXPERTS + 1];
    int bad;
    int skips;  // rows with a bad gather index were met
    Runs runs;
    Start start;
    Segment cut[2];  // the tiles the block's run begins and ends inside
    int last[2];
};

// Cuts the work and finds where this block's run begins; by one warp, before a block
// barrier. CHUNK: activation rows a pass over the weights serves.
template <int CHUNK>
__device__ __forceinline__ void plan_run(const W4Params &p, RunInfo &sh, int tiles, int lane)
{
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
        int sum = static_cast<int>((static_cast<unsigned>(hi[i] - lo[i]) + CHUNK - 1) / CHUNK) * tiles;
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
    if (lane == 0) {
        sh.skips = 0;
        sh.cut[0].e = sh.cut[1].e = -1;
    }
}

// The segments of this block's run, one after the other.
template <int CHUNK>
struct Walk {
    int e, u, s0, first, todo;  // the next segment's expert, unit in it, step, ...
    int tile, chunk, chunks;    // of that unit; chunks 0: not yet known
    int steps, tiles;

    __device__ Walk(const W4Params &p, const RunInfo &sh, int tiles_)
        : e(sh.start.e), u(sh.start.u), s0(sh.start.s0), first(sh.start.first),
          todo(sh.start.todo), tile(0), chunk(0), chunks(0), steps(p.steps), tiles(tiles_)
    {
    }

    __device__ __forceinline__ bool next(const RunInfo &sh, int tile_cols, Segment &s)
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

// 8 codes -> the bf16 pairs (0,4) (1,5) (2,6) (3,7), each (code - zero) / 64. The low four
// bits of a bf16 number alone are the subnormal code * 2^-133; its bits 4..7 alone are
// code * 2^-129, subnormal or in the first binade, where the spacing is the same. So a
// mask and one fused multiply-add do it, exactly; `minus_zero` is -zero / 64.
__device__ __forceinline__ void unpack_int(uint32_t w, uint32_t minus_zero, uint32_t (&v)[4])
{
    constexpr uint32_t two127 = 0x7F007F00u, two123 = 0x7D007D00u;
    const uint32_t h = w >> 8;
    v[0] = bf16x2_fma(w & 0x000F000Fu, two127, minus_zero);
    v[1] = bf16x2_fma(w & 0x00F000F0u, two123, minus_zero);
    v[2] = bf16x2_fma(h & 0x000F000Fu, two127, minus_zero);
    v[3] = bf16x2_fma(h & 0x00F000F0u, two123, minus_zero);
}
constexpr float kIntScale = 64.f;

// e2m1: a code's four bits go to bits 15..12 (for the sign) and 9..6 (exponent and
// mantissa) of its half at once by a multiplication; the number so formed is 2^-126 times
// the code's value. `factor`, in both halves, is 2^126 or that times the scale: with two
// significant bits the product is exact down to the smallest scale.
__device__ __forceinline__ void unpack_e2m1(uint32_t w, uint32_t factor, uint32_t (&v)[4])
{
    const uint32_t h = w >> 8;
    v[0] = bf16x2_mul(((w & 0x000F000Fu) * 0x1040u) & 0x81C081C0u, factor);
    v[1] = bf16x2_mul(((w & 0x00F000F0u) * 0x0104u) & 0x81C081C0u, factor);
    v[2] = bf16x2_mul(((h & 0x000F000Fu) * 0x1040u) & 0x81C081C0u, factor);
    v[3] = bf16x2_mul(((h & 0x00F000F0u) * 0x0104u) & 0x81C081C0u, factor);
}
constexpr uint32_t kTwo126 = 0x7E807E80u;

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

// The block's cut tiles, after all else: of a tile's blocks the last one to come here calls
// add(segment, c0, c1), which is to add what blocks c0 .. c1 left and to store it. The THREADS
// threads that left sums meet at named barrier 1 (which orders the block's sums before the
// release of one thread). A warp that gave up (`ok` false) takes all with it.
template <int THREADS, typename Add>
__device__ __forceinline__ void join_cut_tiles(const W4Params &p, RunInfo &sh, int tid, bool ok, Add add)
{
    if (sh.runs.piece > 1)
        return;  // runs of whole tiles
    if (!named_bar_and(1, THREADS, ok))
        return;
    int *counters = reinterpret_cast<int *>(p.workspace);
    if (tid == 0 || tid == 32) {
        const int slot = tid / 32;
        const Segment &cut = sh.cut[slot];
        int last = 0;
        if (cut.e >= 0) {
            const int c0 = sh.runs.owner(cut.first), c1 = sh.runs.owner(cut.first + p.steps - 1);
            last = atom_add_acq_rel_gpu(counters + c0, 1) == c1 - c0;
            if (last)
                counters[c0] = 0;  // ready for the next call
        }
        sh.last[slot] = last;
    }
    named_bar_sync(1, THREADS);
    for (int slot = 0; slot < 2; ++slot)
        if (sh.last[slot]) {
            const Segment s = sh.cut[slot];
            add(s, sh.runs.owner(s.first), sh.runs.owner(s.first + p.steps - 1));
        }
}

}  // namespace w4
}  // namespace ep
