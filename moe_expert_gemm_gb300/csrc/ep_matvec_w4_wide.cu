// Expert products on 4-bit weights for up to 64 activation rows a pass: ep_matvec_w4.cu
// with the matrix work on the tensor memory's engine.
//
// With some tens of rows an expert the warp-wide matrix instructions take longer than the
// weights' bytes (a step of 128 x 256 weights and 32 rows is 1024 cycles of them, the bytes
// 720). Here the warps only unpack: a thread owns a weight row, turns its codes into bf16
// and stores them into tensor memory, where a row is a lane and two k a column; one thread
// issues tcgen05.mma with that as the first operand, the activations (in shared memory)
// as the second and the fp32 sums of the tile in tensor memory, 128 weight rows by up to 64
// activation rows.
//
//  * The scales go onto the codes, as the sums run over all of K. e2m1 codes take on a
//    power of two exactly (one of 2^128 or more counts as infinite). An integer code times
//    its scale has up to 12 significant bits: it is split into two bf16 numbers, a product a
//    little short of it and what that leaves (at most 8 bits: a fused multiply-add gives
//    it exactly), and both are multiplied.
//  * k comes in the order in which a word's halves give it, (0,4) (1,5) (2,6) (3,7) of
//    eight; the staging warps lay the activations out in that order too, in the 128-byte
//    swizzle that the matrix engine reads.
//  * Thread block: warp 0 streams the weights (TMA), warp 1 issues the products, warps 2
//    and 3 stage activations and scales, warps 4 to 11 unpack (warp i the tensor memory
//    lanes 32 (i % 4) on, the k's first half or second) and store the results.
#include "ep_w4.cuh"
#include "ep_w4_scales.cuh"

namespace ep {

using namespace w4;

namespace {

constexpr int kRows = 64;                        // activation rows of a pass
constexpr int kWeightBytes = kPartRows * kStepK / 2;
constexpr int kAtomBytes = kRows * 128;          // 64 k of the activations
constexpr int kXBytes = kAtomBytes * kStepK / 64;
constexpr int kStages = 2;
constexpr int kStagers = 2;
constexpr int kUnpackers = 8;
constexpr int kThreads = 32 * (2 + kStagers + kUnpackers);
constexpr int kSums = 32;                        // a thread's sums of a tile
constexpr uint32_t kTmemCols = 256;              // of a block: two blocks an SM
constexpr uint32_t kACols = 64;                  // of a buffer of unpacked weights
constexpr uint64_t kTimeoutNs = 2000000000ull;

struct Shared {
    uint64_t full[kStages], empty[kStages];
    uint64_t a_full[2], a_empty[2];
    uint64_t sums_full, drained;
    uint32_t tmem;
    int large[kStages];  // e2m1: the stage holds scales past 2
    int abort;
    RunInfo run;
    float up[16 * 64];   // SwiGLU: 16 columns of the up rows' sums
};

constexpr int stage_bytes(int GS, bool E2M1)
{
    return (kWeightBytes + kXBytes + kPartRows * GS * (E2M1 ? 2 : 4) + 1023) / 1024 * 1024;
}

constexpr int smem_bytes(int GS, bool E2M1)
{
    return 1024 + kStages * stage_bytes(GS, E2M1) + static_cast<int>(sizeof(Shared));
}

__device__ __forceinline__ void give_up(const W4Params &p, Shared &sh)
{
    atomicOr(p.status, EP_STATUS_TIMEOUT);
    *reinterpret_cast<volatile int *>(&sh.abort) = 1;
}

// D(tmem) (+)= A(tmem) * B(smem desc)^T, bf16 inputs.
__device__ __forceinline__ void mma_f16_tmem(uint32_t d, uint32_t a, uint64_t b_desc, uint32_t idesc,
                                             uint32_t accumulate)
{
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
        "r"(a), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}

// Thread i's N registers into lane (base + i), N consecutive columns.
__device__ __forceinline__ void tmem_store(uint32_t taddr, const uint32_t (&r)[32])
{
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
        "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, "
        "%17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};" ::"r"(taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
        "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]),
        "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]),
        "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]), "r"(r[29]),
        "r"(r[30]), "r"(r[31])
        : "memory");
}

__device__ __forceinline__ void tmem_store(uint32_t taddr, const uint32_t (&r)[16])
{
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
        "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
        "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
}

__device__ __forceinline__ void tmem_store_wait()
{
    asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}

// Stores a thread's sums of a whole tile: row `row` of it, columns 32 * half + c.
__device__ __forceinline__ void store_sums(const W4Params &p, Shared &sh, const Segment &s,
                                           const float (&v)[kSums], int row, int half)
{
    const int cols = p.swiglu ? p.N / 2 : p.N;
    const float back = p.format == EP_W4_INT ? kIntScale : 1.f;
    __nv_bfloat16 *C = reinterpret_cast<__nv_bfloat16 *>(p.C);
    const bool skips = sh.run.skips;
    auto put = [&](int m, int n, float y) {
        if (m < s.m1 && n < cols && !(skips && !row_of(p, m)))
            C[static_cast<int64_t>(m) * cols + n] = __float2bfloat16_rn(y);
    };
    const int m0 = s.m0 + 32 * half;
    if (!p.swiglu) {
#pragma unroll
        for (int c = 0; c < kSums; ++c)
            put(m0 + c, s.n0 + row, v[c] * back);
        return;
    }
    // rows 64 on are the up rows of rows 0 on
#pragma unroll
    for (int c0 = 0; c0 < kSums; c0 += 8) {
        if (row >= 64)
#pragma unroll
            for (int c = 0; c < 8; ++c)
                sh.up[(8 * half + c) * 64 + row - 64] = v[c0 + c];
        named_bar_sync(1, 32 * kUnpackers);
        if (row < 64)
#pragma unroll
            for (int c = 0; c < 8; ++c)
                put(m0 + c0 + c, s.n0 + row,
                    silu_f32(v[c0 + c] * back) * (sh.up[(8 * half + c) * 64 + row] * back));
        named_bar_sync(1, 32 * kUnpackers);
    }
}

}  // namespace

template <int GS, bool E2M1, bool VEC>
__global__ void __launch_bounds__(kThreads, 2)
    matvec_w4_wide_kernel(const __grid_constant__ CUtensorMap tw, const __grid_constant__ W4Params p)
{
    constexpr int kStage = stage_bytes(GS, E2M1);
    constexpr int kXOff = kWeightBytes, kScaleOff = kXOff + kXBytes;
    constexpr int kZeroOff = kScaleOff + kPartRows * GS * 2;
    // k of a buffer of unpacked weights: 64 columns of one number a weight or of two
    constexpr int kBatchK = E2M1 ? 128 : 64, kBatches = kStepK / kBatchK;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *ring = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
    Shared &sh = *reinterpret_cast<Shared *>(ring + kStages * kStage);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int tile_cols = p.swiglu ? 64 : kPartRows;
    const int cols = p.swiglu ? p.N / 2 : p.N;
    const int tiles = (cols + tile_cols - 1) / tile_cols;
    if (tid == 64) {
        tma_prefetch_map(&tw);
        for (int i = 0; i < kStages; ++i) {
            mbar_init(&sh.full[i], 2);                // the producer, a staging warp
            mbar_init(&sh.empty[i], kUnpackers + 1);  // the unpacking warps, the products
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&sh.a_full[i], kUnpackers);
            mbar_init(&sh.a_empty[i], 1);
        }
        mbar_init(&sh.sums_full, 1);
        mbar_init(&sh.drained, 1);
        fence_mbar_init();
        sh.abort = 0;
    }
    griddep_launch_dependents();
    griddep_wait();
    // (tensor memory only now: the previous kernel may still have wanted it)
    if (warp == 1) {
        tmem_alloc(&sh.tmem, kTmemCols);
        tmem_relinquish();
    }
    if (warp == 0)
        plan_run<kRows>(p, sh.run, tiles, lane);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = sh.tmem;
    volatile int *abort_flag = &sh.abort;
    Walk<kRows> walk(p, sh.run, tiles);
    if (sh.run.bad)
        walk.todo = 0;
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
        if (lane == 0) {
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
                    mbar_arrive_expect_tx(&sh.full[stage], kWeightBytes);
                    tma_load_2d(dst, &tw, &sh.full[stage], k * (kStepK / 2), y0);
                    tma_load_2d(dst + kWeightBytes / 2, &tw, &sh.full[stage], k * (kStepK / 2), y1);
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
        }
        __syncwarp();
    } else if (warp == 1) {
        // ---------------------------------------------------------------- products
        if (lane == 0) {
            int batch = 0;  // of all: buffer batch % 2
            bool ok = true;
            while (ok && walk.next(sh.run, tile_cols, seg)) {
                const uint32_t idesc = make_idesc(1u, 128, (seg.m1 - seg.m0 + 15) / 16 * 16);
                for (int k = seg.s0; ok && k < seg.s1; ++k) {
                    ok = mbar_wait(&sh.full[stage], phase, kTimeoutNs, abort_flag);
                    const uint32_t x = smem_u32(ring + stage * kStage + kXOff);
                    const int here = VEC || (k + 1) * kStepK <= p.K ? kStepK : p.K - k * kStepK;
                    for (int i = 0; ok && i < kBatches; ++i, ++batch) {
                        const int buf = batch & 1;
                        ok = mbar_wait(&sh.a_full[buf], (batch >> 1) & 1, kTimeoutNs, abort_flag);
                        if (!ok)
                            break;
                        tc_fence_after();
                        const uint32_t a = tmem + kRows + buf * kACols;
#pragma unroll
                        for (int j = 0; j < kBatchK / 16; ++j) {
                            const int at = i * kBatchK + j * 16;
                            if (!VEC && at >= here)
                                break;
                            const uint64_t b =
                                desc_kmajor_sw128(x + at / 64 * kAtomBytes + at % 64 * 2);
                            mma_f16_tmem(tmem, a + j * 8, b, idesc, k > seg.s0 || i > 0 || j > 0);
                            if (!E2M1)
                                mma_f16_tmem(tmem, a + kACols / 2 + j * 8, b, idesc, 1);
                        }
                        mma_commit(&sh.a_empty[buf]);
                    }
                    if (!ok)
                        break;
                    mma_commit(&sh.empty[stage]);
                    advance();
                }
                if (ok)
                    mma_commit(&sh.sums_full);
            }
            if (!ok)
                give_up(p, sh);
            // every product issued has ended once this arrives
            mma_commit(&sh.drained);
            volatile int no_abort = 0;
            mbar_wait(&sh.drained, 0, kTimeoutNs, &no_abort);
        }
        __syncwarp();
    } else if (warp < 2 + kStagers) {
        // ----------------------------------------- staging: activations and scales
        bool turn = warp == 2;  // this warp's step, the other's, ... (as many as stages: a
                                // wait knows a phase's parity alone)
        constexpr int kRowSets = kPartRows / 32, kBatch = 8;
        const int groups = p.K / (kStepK / GS);
        bool ok = true;
        while (ok && walk.next(sh.run, tile_cols, seg)) {
            const int rows = seg.m1 - seg.m0;
            unsigned long long mine[2];  // where the segment's rows lane, lane + 32 lie
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const bool there = 32 * i + lane < rows;
                mine[i] = there ? reinterpret_cast<unsigned long long>(row_of(p, seg.m0 + 32 * i + lane)) : 0;
                if (there && !mine[i]) {
                    atomicOr(p.status, EP_STATUS_BOUNDS);
                    sh.run.skips = 1;
                }
            }
            int64_t scale_at[kRowSets];
#pragma unroll
            for (int i = 0; i < kRowSets; ++i) {
                const int r = 32 * i + lane;
                int n = seg.n0 + (p.swiglu ? r % 64 : r);
                n = n < cols ? n : cols - 1;  // (rows past the last column: nobody stores them)
                scale_at[i] = (static_cast<int64_t>(seg.e) * p.N + n + (p.swiglu && r >= 64 ? cols : 0)) * groups;
            }
            for (int k = seg.s0; k < seg.s1; ++k, turn = !turn) {
                if (!turn) {
                    advance();
                    continue;
                }
                Scales<GS, E2M1, VEC> sc[kRowSets];
#pragma unroll
                for (int i = 0; i < kRowSets; ++i)
                    sc[i].load(p, scale_at[i] + k * GS, groups - k * GS);
                const int k0 = k * kStepK + lane * 8;  // this lane's piece of a row
                uint4 v[kBatch];
                auto load_rows = [&](int r0) {
#pragma unroll
                    for (int i = 0; i < kBatch; ++i) {
                        if (r0 + i >= rows)
                            break;
                        const uint4 *from = reinterpret_cast<const uint4 *>(
                            __shfl_sync(0xffffffffu, r0 < 32 ? mine[0] : mine[1], (r0 + i) & 31));
                        v[i] = make_uint4(0, 0, 0, 0);
                        if (from && (VEC || k0 < p.K))
                            v[i] = __ldg(from + k0 / 8);
                    }
                };
                load_rows(0);
                ok = __all_sync(0xffffffffu,
                                mbar_wait(&sh.empty[stage], phase ^ 1, kTimeoutNs, abort_flag));
                if (!ok)
                    break;
                uint8_t *dst = ring + stage * kStage;
                uint8_t *x = dst + kXOff + lane / 8 * kAtomBytes;
                for (int r0 = 0; r0 < rows; r0 += kBatch) {
                    if (r0)
                        load_rows(r0);
#pragma unroll
                    for (int i = 0; i < kBatch; ++i) {
                        if (r0 + i >= rows)
                            break;
                        const int r = r0 + i;
                        *reinterpret_cast<uint4 *>(x + r * 128 + ((lane % 8 ^ r % 8) << 4)) = make_uint4(
                            __byte_perm(v[i].x, v[i].z, 0x5410), __byte_perm(v[i].x, v[i].z, 0x7632),
                            __byte_perm(v[i].y, v[i].w, 0x5410), __byte_perm(v[i].y, v[i].w, 0x7632));
                    }
                }
                bool large = false;
                if (E2M1) {
#pragma unroll
                    for (int i = 0; i < kRowSets; ++i)
                        large |= sc[i].large();
                    large = __any_sync(0xffffffffu, large);
                    if (lane == 0)
                        sh.large[stage] = large;
                }
#pragma unroll
                for (int i = 0; i < kRowSets; ++i) {
                    const int r = 32 * i + lane;
                    sc[i].store(dst + kScaleOff + r * GS * 2, dst + kZeroOff + r * GS * 2, large);
                }
                fence_proxy_async_shared();  // the products read the activations
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(&sh.full[stage]);
                advance();
            }
        }
        if (!ok && lane == 0)
            give_up(p, sh);
    } else {
        // ------------------------------------------------------ unpacking, results
        const int quarter = warp & 3, half = (warp - 2 - kStagers) >> 2;
        const int row = 32 * quarter + lane, utid = tid - 32 * (2 + kStagers);
        const uint32_t my_lanes = tmem + (static_cast<uint32_t>(32 * quarter) << 16);
        const uint8_t *const scale0 = ring + kScaleOff + row * GS * 2;
        // fours of this thread's sums that belong to rows of the segment
        auto used = [&](const Segment &s) {
            const int n = (s.m1 - s.m0 - 32 * half + 3) / 4;
            return n < 0 ? 0 : n > kSums / 4 ? kSums / 4 : n;
        };
        int batch = 0, segments = 0;
        bool ok = true;
        while (walk.next(sh.run, tile_cols, seg)) {
            for (int k = seg.s0; ok && k < seg.s1; ++k) {
                ok = __all_sync(0xffffffffu,
                                mbar_wait(&sh.full[stage], phase, kTimeoutNs, abort_flag));
                if (!ok)
                    break;
                const uint8_t *src = ring + stage * kStage;
                const bool large = E2M1 && sh.large[stage];
                for (int i = 0; i < kBatches; ++i, ++batch) {
                    const int buf = batch & 1;
                    // chunks of 32 k: two of four, or one of two
                    constexpr int kChunks = kBatchK / 64;
                    uint4 codes[kChunks];
                    uint32_t scale[kChunks], zero[kChunks];
#pragma unroll
                    for (int j = 0; j < kChunks; ++j) {
                        const int c = (2 * i + half) * kChunks + j, gr = c * GS / 8;
                        codes[j] = *reinterpret_cast<const uint4 *>(src + row * 128 + ((c ^ row % 8) << 4));
                        scale[j] = *reinterpret_cast<const uint16_t *>(scale0 + stage * kStage + gr * 2) * 0x10001u;
                        if (!E2M1)
                            zero[j] = *reinterpret_cast<const uint16_t *>(scale0 + stage * kStage + kZeroOff -
                                                                          kScaleOff + gr * 2) * 0x10001u;
                    }
                    ok = __all_sync(0xffffffffu, mbar_wait(&sh.a_empty[buf], (batch >> 1 & 1) ^ 1, kTimeoutNs,
                                                           abort_flag));
                    if (!ok)
                        break;
                    tc_fence_after();
                    const uint32_t a = my_lanes + kRows + buf * kACols + half * (16 * kChunks);
                    if constexpr (E2M1) {
                        uint32_t w[32];
#pragma unroll
                        for (int j = 0; j < 2; ++j) {
                            const uint32_t c[4] = {codes[j].x, codes[j].y, codes[j].z, codes[j].w};
#pragma unroll
                            for (int b = 0; b < 4; ++b) {
                                uint32_t t[4];
                                unpack_e2m1(c[b], large ? kTwo126 : scale[j], t);
#pragma unroll
                                for (int h = 0; h < 4; ++h)
                                    w[16 * j + 4 * b + h] = large ? bf16x2_mul(t[h], scale[j]) : t[h];
                            }
                        }
                        tmem_store(a, w);
                    } else {
                        uint32_t hi[16], lo[16];
                        const uint32_t c[4] = {codes[0].x, codes[0].y, codes[0].z, codes[0].w};
                        // the first part with a scale two steps short: it stays short of the
                        // product, and the second part has its sign (so that an infinite
                        // activation meets no 0 that the product is not)
                        const uint32_t less = (scale[0] & 0x7FFFu) > 1 ? 0x00020002u : 0u;
                        const uint32_t minus = (scale[0] - less) ^ 0x80008000u;
#pragma unroll
                        for (int b = 0; b < 4; ++b) {
                            uint32_t t[4];
                            unpack_int(c[b], zero[0], t);
#pragma unroll
                            for (int h = 0; h < 4; ++h) {
                                const uint32_t n = bf16x2_mul(t[h], minus);
                                lo[4 * b + h] = bf16x2_fma(t[h], scale[0], n);
                                hi[4 * b + h] = n ^ 0x80008000u;
                            }
                        }
                        tmem_store(a, hi);
                        tmem_store(a + kACols / 2, lo);
                    }
                    tmem_store_wait();
                    tc_fence_before();
                    if (i == kBatches - 1)
                        fence_proxy_async_shared();  // before the next copy into the stage
                    __syncwarp();
                    if (lane == 0) {
                        mbar_arrive(&sh.a_full[buf]);
                        if (i == kBatches - 1)
                            mbar_arrive(&sh.empty[stage]);
                    }
                }
                if (!ok)
                    break;
                advance();
            }
            if (ok)
                ok = __all_sync(0xffffffffu,
                                mbar_wait(&sh.sums_full, segments & 1, kTimeoutNs, abort_flag));
            ++segments;
            // (all of the unpacking warps leave together: they meet at barriers below)
            if (!ok && lane == 0)
                give_up(p, sh);
            if (!named_bar_and(1, 32 * kUnpackers, ok)) {
                ok = false;
                break;
            }
            tc_fence_after();
            uint32_t r[32];
            tmem_ld_32x32b_x32(my_lanes + 32 * half, r);
            tmem_ld_wait();
            tmem_regs_ready(r);
            tc_fence_before();
            float v[kSums];
#pragma unroll
            for (int c = 0; c < kSums; ++c)
                v[c] = __uint_as_float(r[c]);
            if (seg.s0 == 0 && seg.s1 == walk.steps)
                store_sums(p, sh, seg, v, row, half);
            else
                leave_sums<kSums / 4, 32 * kUnpackers>(
                    p, sh.run, seg, *reinterpret_cast<float(*)[kSums / 4][4]>(v), used(seg), utid);
        }
        join_cut_tiles<kSums / 4, 32 * kUnpackers>(
            p, sh.run, utid, ok, used, [&](const Segment &s, const float(&v)[kSums / 4][4]) {
                store_sums(p, sh, s, *reinterpret_cast<const float(*)[kSums]>(v), row, half);
            });
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 1)
        tmem_dealloc(tmem, kTmemCols);
}

template <int GS, bool E2M1, bool VEC>
static cudaError_t launch_wide(const CUtensorMap &tw, const W4Params &p, int num_sms, cudaStream_t s)
{
    const auto kern = matvec_w4_wide_kernel<GS, E2M1, VEC>;
    constexpr int smem = smem_bytes(GS, E2M1);
    static_assert(smem <= 113 * 1024, "two blocks an SM");
    const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess)
        return e;
    const int grid = 2 * num_sms;
    return launch_behind(kern, grid < kMaxBlocks ? grid : kMaxBlocks, kThreads, smem, s, tw, p);
}

template <bool VEC>
static cudaError_t launch_form(const CUtensorMap &tw, const W4Params &p, int num_sms, cudaStream_t s)
{
    if (p.format == EP_W4_E2M1)
        return launch_wide<8, true, VEC>(tw, p, num_sms, s);
    switch (p.group) {
    case 32:
        return launch_wide<8, false, VEC>(tw, p, num_sms, s);
    case 64:
        return launch_wide<4, false, VEC>(tw, p, num_sms, s);
    default:
        return launch_wide<2, false, VEC>(tw, p, num_sms, s);
    }
}

cudaError_t launch_matvec_w4_wide(const CUtensorMap &tw, const W4Params &p, int num_sms, cudaStream_t s)
{
    return p.scale_vec ? launch_form<true>(tw, p, num_sms, s) : launch_form<false>(tw, p, num_sms, s);
}

}  // namespace ep
