// Expert products of a few rows on 4-bit weights: C[m][n] = sum_k W_e[n][k] a[m][k].
//
// Every weight of an expert that has rows is read once and meets a handful of activation
// rows, so the call is bound by the weights' bytes, N*K/2 per expert, as long as the codes
// become multiplicands fast enough. The weights are therefore the 16-row operand of the
// warp's 16x8x16 bf16 matrix instruction and the activation rows its 8 columns: 8 rows
// cost the same unpacking as one. Past 16 rows a pass ep_matvec_w4_wide.cu takes over.
//
//  * A code becomes an exact bf16 multiple of (q - zero), or of its e2m1 value, in a mask
//    and a fused multiply-add (unpack_int, unpack_e2m1). The sum over a group of k runs in
//    fp32 on these numbers; the group's scale multiplies that sum in fp32, so no weight is
//    ever rounded.
//  * e2m1 scales are powers of two, which the codes can take on exactly in bf16: there a
//    group needs no sum of its own (as long as the scale is at most 2; else it gets one).
//  * The order of k inside a matrix instruction is free. A thread's words of a weight row
//    (as many at once as a scale group of k feeds the four threads of a row) hold 8
//    consecutive codes each, whose halves are the pairs (0,4) (1,5) (2,6) (3,7); the
//    activations are laid into shared memory in that order.
//  * A tile is 128 weight rows (with SwiGLU 64 gate rows and their up rows), a step of it
//    16 KB. Thread block: one thread streams the weights (TMA, 128-byte swizzle) into a ring
//    of stages; three warps stage activations and scales; eight consumer warps own 16
//    weight rows each, 8 of the tile's first half and 8 of its second: with SwiGLU the gate
//    and the up row of the same output meet in one thread.
//  * Measured: one token, 8 experts of 4096 x 7168 (integer codes, SwiGLU), 32 us a call for
//    121 MB of codes and scales, 3.8 TB/s; 8 of 4096 x 1536 (e2m1) 11.9 us, of which the
//    host's call is 6.5. Eight consumer warps take 290 instructions each a step of 16 KB:
//    with consumers that only wait the first takes 26 us.
#include <type_traits>

#include "ep_w4.cuh"
#include "ep_w4_scales.cuh"

namespace ep {

using namespace w4;

namespace {

constexpr int kStepBytes = kPartRows * kStepK / 2;
constexpr int kConsumers = 8, kStagers = 3;  // warps
constexpr int kThreads = 32 * (1 + kStagers + kConsumers);
constexpr int kMaxStages = 5;
constexpr int kSmem = 113 * 1024;            // two blocks an SM
constexpr uint64_t kTimeoutNs = 2000000000ull;

struct Shared {
    uint64_t full[kMaxStages], empty[kMaxStages];
    int sums_apart[kMaxStages];  // e2m1: the stage's scales need sums by group
    int abort;
    RunInfo run;
};

// Weights, activations, scales and zero points (both bf16) of a step; a multiple of the
// 1 KB the swizzled weight tiles start on.
constexpr int stage_bytes(int NT, int GS, bool E2M1)
{
    return (kStepBytes + NT * 8 * kStepK * 2 + kPartRows * GS * (E2M1 ? 2 : 4) + 1023) / 1024 * 1024;
}

constexpr int stages_of(int NT, int GS, bool E2M1)
{
    const int n = (kSmem - 1024 - static_cast<int>(sizeof(Shared))) / stage_bytes(NT, GS, E2M1);
    return n > kMaxStages ? kMaxStages : n;
}

constexpr int smem_bytes(int NT, int GS, bool E2M1)
{
    return 1024 + stages_of(NT, GS, E2M1) * stage_bytes(NT, GS, E2M1) + static_cast<int>(sizeof(Shared));
}

__device__ __forceinline__ void give_up(const W4Params &p, Shared &sh)
{
    atomicOr(p.status, EP_STATUS_TIMEOUT);
    *reinterpret_cast<volatile int *>(&sh.abort) = 1;
}

}  // namespace

// NT: groups of 8 activation rows a pass over the weights serves. GS: scale groups of a
// step (256 / group size). VEC: K is whole steps, a step's scales one aligned piece
// (W4Params::scale_vec).
template <int NT, int GS, bool E2M1, bool VEC>
__global__ void __launch_bounds__(kThreads, 2)
    matvec_w4_kernel(const __grid_constant__ CUtensorMap tw, const __grid_constant__ W4Params p)
{
    constexpr int kStages = stages_of(NT, GS, E2M1);
    constexpr int kStage = stage_bytes(NT, GS, E2M1);
    constexpr int kXOff = kStepBytes, kScaleOff = kXOff + NT * 8 * kStepK * 2;
    constexpr int kZeroOff = kScaleOff + kPartRows * GS * 2;
    // Staging warps take turns. One may look at a stage's barrier only when at most one of
    // its phases is open (a wait knows a phase's parity alone), so no more of them take part
    // than there are stages.
    constexpr int kTurns = kStagers < kStages ? kStagers : kStages;
    // Words of a weight row a thread of the row's four takes at once: their 32 * kWords
    // codes belong to one scale group.
    constexpr int kWords = 8 / GS;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *ring = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
    Shared &sh = *reinterpret_cast<Shared *>(ring + kStages * kStage);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

    const int tile_cols = p.swiglu ? 64 : kPartRows;
    const int cols = p.swiglu ? p.N / 2 : p.N;
    if (warp == 1 && lane == 0) {
        tma_prefetch_map(&tw);
        for (int i = 0; i < kStages; ++i) {
            mbar_init(&sh.full[i], 2);  // the producer, a staging warp
            mbar_init(&sh.empty[i], kConsumers);
        }
        fence_mbar_init();
        sh.abort = 0;
    }
    const int tiles = (cols + tile_cols - 1) / tile_cols;
    griddep_wait();
    griddep_launch_dependents();
    if (warp == 0)
        plan_run<8 * NT>(p, sh.run, tiles, lane);
    __syncthreads();
    if (sh.run.bad)
        return;

    volatile int *abort_flag = &sh.abort;
    Walk<8 * NT> walk(p, sh.run, tiles);
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
        // ------------------------------------------------------- producer: weights
        if (lane != 0)
            return;
        int issued = 0;
        bool ok = true;
        while (ok && walk.next(sh.run, tile_cols, seg)) {
            const int y0 = seg.e * p.N + seg.n0, y1 = y0 + (p.swiglu ? cols : 64);
            for (int k = seg.s0; k < seg.s1; ++k) {
                if (!mbar_wait(&sh.empty[stage], phase ^ 1, kTimeoutNs, abort_flag)) {
                    ok = false;
                    break;
                }
                uint8_t *dst = ring + stage * kStage;
                mbar_arrive_expect_tx(&sh.full[stage], kStepBytes);
                tma_load_2d(dst, &tw, &sh.full[stage], k * (kStepK / 2), y0);
                tma_load_2d(dst + kStepBytes / 2, &tw, &sh.full[stage], k * (kStepK / 2), y1);
                ++issued;
                advance();
            }
        }
        if (!ok) {
            give_up(p, sh);
            // the copies in flight land before the block's shared memory goes away
            volatile int no_abort = 0;
            for (int i = issued > kStages ? issued - kStages : 0; i < issued; ++i)
                mbar_wait(&sh.full[i % kStages], (i / kStages) & 1, 1000000, &no_abort);
        }
        return;
    }

    if (warp <= kStagers) {
        // ------------------------- staging: activations, scales and zero points
        if (warp > kTurns)
            return;
        int turn = warp - 1;  // steps until this warp's next
        constexpr int kRowSets = kPartRows / 32;
        constexpr int kBatch = 4;  // activation rows under way at once
        const int groups = p.K / (kStepK / GS);
        // where a lane's piece (8 activations, in pair order) of a row goes: the place of the
        // thread (row, q) that takes word w of its codes of block b
        const int b = lane / (4 * kWords) * kWords + lane % kWords, q = lane / kWords % 4;
        bool ok = true;
        while (ok && walk.next(sh.run, tile_cols, seg)) {
            const int rows = seg.m1 - seg.m0;
            unsigned long long mine = 0;  // lane i: where the segment's row i lies
            if (lane < rows) {
                mine = reinterpret_cast<unsigned long long>(row_of(p, seg.m0 + lane));
                if (!mine) {
                    atomicOr(p.status, EP_STATUS_BOUNDS);
                    sh.run.skips = 1;
                }
            }
            // where this lane's weight rows have their scales (rows past the last column
            // take the last one's: nobody stores what comes of them)
            int64_t scale_at[kRowSets];
#pragma unroll
            for (int i = 0; i < kRowSets; ++i) {
                const int r = 32 * i + lane;
                int n = seg.n0 + (p.swiglu ? r % 64 : r);
                n = n < cols ? n : cols - 1;
                scale_at[i] = (static_cast<int64_t>(seg.e) * p.N + n + (p.swiglu && r >= 64 ? cols : 0)) * groups;
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
                load_rows(0);
                ok = __all_sync(0xffffffffu, mbar_wait(&sh.empty[stage], phase ^ 1, kTimeoutNs,
                                                       abort_flag));
                if (!ok)
                    break;
                uint8_t *dst = ring + stage * kStage;
                // (columns of the matrix instruction past the last row hold whatever they held:
                // they only reach results that nobody stores)
                for (int r0 = 0; r0 < rows; r0 += kBatch) {
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
    const int row = 8 * cw + g;  // in each half of a tile
    const int ctid = cw * 32 + lane;
    // this thread's first words of a weight row, in the 128-byte swizzle (the 16-byte piece i
    // of row r is at i ^ r % 8)
    const int at0 = row * 128 + ((q * kWords / 4 ^ g) << 4) + q * kWords % 4 * 4;
    const int scale0 = kScaleOff + row * GS * 2;
    const int zero0 = scale0 + kZeroOff - kScaleOff;
    float4 *const sums = reinterpret_cast<float4 *>(p.workspace + kMaxBlocks * 16);
    constexpr int64_t kSlot = 32 * kConsumers * NT;  // fours of a partial tile
    bool ok = true;
    while (walk.next(sh.run, tile_cols, seg)) {
        const int nts = (seg.m1 - seg.m0 + 7) / 8;
        float acc[NT][4];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int i = 0; i < 4; ++i)
                acc[nt][i] = 0.f;
        for (int k = seg.s0; k < seg.s1; ++k) {
            ok = __all_sync(0xffffffffu,
                            mbar_wait(&sh.full[stage], phase, kTimeoutNs, abort_flag));
            if (!ok)
                break;
            const uint8_t *src = ring + stage * kStage;
            const int blocks = VEC || (k + 1) * kStepK <= p.K ? 8 : (p.K - k * kStepK) / 32;
            // a row's scales and zero points, two a word
            alignas(16) uint32_t scale[2][GS / 2], zero[2][GS / 2] = {};
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                copy_words<GS / 2>(scale[h], src + scale0 + h * 64 * GS * 2);
                if constexpr (!E2M1)
                    copy_words<GS / 2>(zero[h], src + zero0 + h * 64 * GS * 2);
            }
            auto scale_of = [&](int h, int gr) {
                return __uint_as_float(gr & 1 ? scale[h][gr / 2] & 0xFFFF0000u : scale[h][gr / 2] << 16);
            };
            auto twice = [&](uint32_t two, int gr) {  // one of them in both halves
                return __byte_perm(two, 0u, gr & 1 ? 0x3232u : 0x1010u);
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
                        copy_words<kWords>(w[h], src + h * (kStepBytes / 2) + (at0 ^ (b0 << 4)));
#pragma unroll
                    for (int j = 0; j < kWords; ++j) {
                        const int b = b0 + j, gr = b * GS / 8;
                        const bool first = APART && (b * GS % 8 == 0 || GS == 8);
                        const bool last = APART && ((b + 1) * GS % 8 == 0 || GS == 8);
                        uint32_t a[2][4];
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            if constexpr (E2M1)
                                unpack_e2m1(w[h][j], APART ? kTwo126 : twice(scale[h][gr / 2], gr), a[h]);
                            else
                                unpack_int(w[h][j], twice(zero[h][gr / 2], gr), a[h]);
                        }
                        const float s0 = last ? scale_of(0, gr) : 0.f, s1 = last ? scale_of(1, gr) : 0.f;
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) {
                            const uint4 x = *reinterpret_cast<const uint4 *>(
                                src + kXOff + ((b * NT + nt) * 32 + lane) * 16);
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
        if (seg.s0 == 0 && seg.s1 == walk.steps)
            store_tile<NT>(p, seg, acc, row, q, sh.run.skips);
        else {
            // a cut tile: leave the sums in the block's slot for the tile its run begins inside
            // (0) or ends inside (1)
            const int slot = seg.s0 == 0 ? 1 : 0;
            float4 *to = sums + (blockIdx.x * 2 + slot) * kSlot + ctid;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
                if (nt < nts)
                    __stcg(to + nt * 32 * kConsumers,
                           make_float4(acc[nt][0], acc[nt][1], acc[nt][2], acc[nt][3]));
            if (ctid == 0)
                sh.run.cut[slot] = seg;
        }
    }
    if (!ok && lane == 0)
        give_up(p, sh);
    join_cut_tiles<32 * kConsumers>(p, sh.run, ctid, ok, [&](const Segment &s, int from, int to) {
        const int nts = (s.m1 - s.m0 + 7) / 8;
        float acc[NT][4] = {};
        // (four blocks' sums under way at once: a tile of a long K has ten and more)
        constexpr int kAhead = 4;
        for (int b0 = from; b0 <= to; b0 += kAhead) {
            float4 v[kAhead][NT];
#pragma unroll
            for (int i = 0; i < kAhead; ++i)
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    const int b = b0 + i;
                    v[i][nt] = make_float4(0.f, 0.f, 0.f, 0.f);
                    if (b <= to && nt < nts)
                        v[i][nt] = __ldcg(sums + (b * 2 + (b == from ? 1 : 0)) * kSlot + ctid + nt * 32 * kConsumers);
                }
#pragma unroll
            for (int i = 0; i < kAhead; ++i)
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    acc[nt][0] += v[i][nt].x;
                    acc[nt][1] += v[i][nt].y;
                    acc[nt][2] += v[i][nt].z;
                    acc[nt][3] += v[i][nt].w;
                }
        }
        store_tile<NT>(p, s, acc, row, q, sh.run.skips);
    });
}

int64_t w4_workspace_bytes()
{
    // counters, and two partial tiles a block: 128 rows by 64 columns at most
    return kMaxBlocks * (16 + 2ll * kPartRows * 64 * 4);
}

template <int NT, int GS, bool E2M1, bool VEC>
static cudaError_t launch_w4(const CUtensorMap &tw, const W4Params &p, int num_sms, cudaStream_t s)
{
    const auto kern = matvec_w4_kernel<NT, GS, E2M1, VEC>;
    constexpr int smem = smem_bytes(NT, GS, E2M1);
    const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess)
        return e;
    const int grid = 2 * num_sms;
    return launch_behind(kern, grid < kMaxBlocks ? grid : kMaxBlocks, kThreads, smem, s, tw, p);
}

template <int NT, bool VEC>
static cudaError_t launch_nt(const CUtensorMap &tw, const W4Params &p, int num_sms, cudaStream_t s)
{
    if (p.format == EP_W4_E2M1)
        return launch_w4<NT, 8, true, VEC>(tw, p, num_sms, s);
    switch (p.group) {
    case 32:
        return launch_w4<NT, 8, false, VEC>(tw, p, num_sms, s);
    case 64:
        return launch_w4<NT, 4, false, VEC>(tw, p, num_sms, s);
    default:
        return launch_w4<NT, 2, false, VEC>(tw, p, num_sms, s);
    }
}

cudaError_t launch_matvec_w4(const CUtensorMap &tw, const W4Params &p, int num_sms, cudaStream_t s)
{
    // Rows a pass serves, by the rows that an expert is expected to get (some get more and
    // take another pass). Measured with 32 experts of 7168 x 2048, us a call, e2m1 / int:
    //   rows  4:   8 a pass  74 /  57, 16 a pass  80 /  70
    //   rows  6:   8 a pass  83 /  65, 16 a pass  84 /  72
    //   rows  8:   8 a pass 107 /  81, 16 a pass  86 /  74
    //   rows 12:  16 a pass 103 /  89, 64 a pass 102 / 144
    //   rows 16:  16 a pass 129 / 111, 64 a pass 103 / 144
    //   rows 24:  16 a pass 178 / 152, 64 a pass 107 / 148
    //   rows 64:  16 a pass 387 / 329, 64 a pass 167 / 230
    // (64 a pass is the form of ep_matvec_w4_wide.cu, which takes integer weights as two
    // numbers each.) A batch that fits one pass of the smaller form whole stays there.
    const int64_t tokens = static_cast<int64_t>(p.T) * p.n_ranks;
    int64_t rows = (tokens * p.top_k + static_cast<int64_t>(p.n_ranks) * p.El - 1) /
                   (static_cast<int64_t>(p.n_ranks) * p.El);
    rows = rows < p.max_rows ? rows : p.max_rows;
    if (p.max_rows > 16 && rows > (p.format == EP_W4_E2M1 ? 12 : 23))
        return launch_matvec_w4_wide(tw, p, num_sms, s);
    if (p.max_rows > 8 && rows > 6)
        return p.scale_vec ? launch_nt<2, true>(tw, p, num_sms, s) : launch_nt<2, false>(tw, p, num_sms, s);
    return p.scale_vec ? launch_nt<1, true>(tw, p, num_sms, s) : launch_nt<1, false>(tw, p, num_sms, s);
}

}  // namespace ep
