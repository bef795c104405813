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
//    it exactly, down to scales of 2^-120; below, bf16's own spacing cuts it), and both
//    are multiplied.
//  * k comes in the order in which a word's halves give it, (0,4) (1,5) (2,6) (3,7) of
//    eight; the staging warps lay the activations out in that order too, in the 128-byte
//    swizzle that the matrix engine reads.
//  * Thread block: warp 0 streams the weights (TMA), warp 1 issues the products, warps 2
//    to 5 stage activations and scales, warps 6 to 9 unpack (warp i the tensor memory
//    lanes 32 (i % 4) on) and store the results. Codes, activations and unpacked weights
//    have a ring each, so that nobody waits for more than what it reads.
//  * What bounds it is the issue of instructions, 17 for a word of eight codes before all
//    else; hence straight code for the staging warps, which have a row's piece in ten.
//  * Measured: 128 tokens, 8 of 32 experts, 7168 x 2048 in e2m1: 110 us a call for 267 MB,
//    2.4 TB/s, 270 TFLOP/s, the schedulers and the integer pipe 57 % busy; 92 us with codes
//    that are not unpacked. The warp-wide matrix instructions took 167 us.
#include "ep_w4.cuh"
#include "ep_w4_scales.cuh"

namespace ep {

using namespace w4;

namespace {

constexpr int kRows = 64;                        // activation rows of a pass
constexpr int kWeightBytes = kPartRows * kStepK / 2;
constexpr int kAtomBytes = kRows * 128;          // 64 k of the activations
constexpr int kXK = 128;                         // k of a stage of activations: half a step
constexpr int kXBytes = kAtomBytes * kXK / 64;
constexpr int kStages = 3, kXStages = 3, kBuffers = 3;
constexpr int kStagers = 4;
constexpr int kUnpackers = 4;
constexpr int kThreads = 32 * (2 + kStagers + kUnpackers);
constexpr uint32_t kTmemCols = 256;              // of a block: two blocks an SM
constexpr uint32_t kACols = 64;                  // of a buffer of unpacked weights
constexpr uint64_t kTimeoutNs = 2000000000ull;

struct Shared {
    uint64_t full[kStages], empty[kStages];       // codes and scales
    uint64_t x_full[kXStages], x_empty[kXStages];  // activations
    uint64_t a_full[kBuffers], a_empty[kBuffers];  // unpacked weights
    uint64_t sums_full, drained;
    uint32_t tmem;
    int large[kStages][kStagers];  // e2m1: the stage holds scales past 2, of 32 weight rows
    int abort;
    RunInfo run;
    float up[4 * 64];  // SwiGLU: 4 columns of the up rows' sums
};

constexpr int stage_bytes(int GS, bool E2M1)
{
    return (kWeightBytes + kPartRows * GS * (E2M1 ? 2 : 4) + 1023) / 1024 * 1024;
}

constexpr int smem_bytes(int GS, bool E2M1)
{
    return 1024 + kStages * stage_bytes(GS, E2M1) + kXStages * kXBytes + static_cast<int>(sizeof(Shared));
}

// The place of a block's sums of a cut tile: 64 columns of 128 rows, 4 columns by a row at a
// time.
__device__ __forceinline__ float4 *sums_of(const W4Params &p, int slot)
{
    return reinterpret_cast<float4 *>(p.workspace + kMaxBlocks * 16) +
           static_cast<int64_t>(slot) * (kRows / 4 * kPartRows);
}

// mbar_wait with less code at each of the many waits of this kernel and a longer suspension
// (128 tokens as above: 110 us, with mbar_wait 118).
__device__ __forceinline__ bool wait_long(uint64_t *bar, uint32_t parity, uint64_t timeout_ns,
                                          volatile int *abort)
{
    auto probe = [&] {
        uint32_t ok;
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\t"
            "selp.u32 %0, 1, 0, p;\n\t}"
            : "=r"(ok)
            : "r"(smem_u32(bar)), "r"(parity), "r"(10000u)
            : "memory");
        return ok != 0;
    };
    if (probe())
        return true;
    const uint64_t t0 = globaltimer_ns();
    while (!probe())
        if (*abort || globaltimer_ns() - t0 > timeout_ns)
            return false;
    return true;
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

// Thread i's registers into lane (base + i), consecutive columns.
__device__ __forceinline__ void tmem_store(uint32_t taddr, const uint32_t (&r)[16])
{
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
        "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
        "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
}

// 8 consecutive columns of lane (base + i) to thread i, when they are there.
__device__ __forceinline__ void tmem_load(uint32_t taddr, float (&v)[8])
{
    uint32_t r[8];
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
                   "=r"(r[7])
                 : "r"(taddr)
                 : "memory");
    tmem_ld_wait();
    tmem_regs_ready(r);
#pragma unroll
    for (int c = 0; c < 8; ++c)
        v[c] = __uint_as_float(r[c]);
}

__device__ __forceinline__ void tmem_store_wait()
{
    asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}

// Stores a thread's sums of a whole tile, row `row` of it and the segment's rows c0 .. c0 + 7.
__device__ __forceinline__ void store_sums(const W4Params &p, Shared &sh, const Segment &s,
                                           const float (&v)[8], int row, int c0)
{
    const int cols = p.swiglu ? p.N / 2 : p.N;
    const float back = p.format == EP_W4_INT ? kIntScale : 1.f;
    float up[8];
    if (p.swiglu) {  // tile rows 64 on are the up rows of rows 0 on
        float *const mine = sh.up + row % 64;
#pragma unroll
        for (int h = 0; h < 8; h += 4) {
            if (row >= 64)
#pragma unroll
                for (int c = 0; c < 4; ++c)
                    mine[c * 64] = v[h + c] * back;
            named_bar_sync(1, 32 * kUnpackers);
#pragma unroll
            for (int c = 0; c < 4; ++c)
                up[h + c] = mine[c * 64];
            named_bar_sync(1, 32 * kUnpackers);
        }
        if (row >= 64)
            return;
    }
    const int n = s.n0 + row;
    if (n >= cols)
        return;
    __nv_bfloat16 *C = reinterpret_cast<__nv_bfloat16 *>(p.C) + static_cast<int64_t>(s.m0 + c0) * cols + n;
    if (!sh.run.skips) {
        const int end = s.m1 - s.m0 - c0;
#pragma unroll
        for (int c = 0; c < 8; ++c, C += cols) {
            const float y = v[c] * back;
            if (c < end)
                *C = __float2bfloat16_rn(p.swiglu ? silu_f32(y) * up[c] : y);
        }
    } else {
        float y[8];
#pragma unroll
        for (int c = 0; c < 8; ++c)
            y[c] = p.swiglu ? silu_f32(v[c] * back) * up[c] : v[c] * back;
#pragma unroll 1
        for (int m = s.m0 + c0; m < s.m1 && m < s.m0 + c0 + 8; ++m, C += cols) {
            if (row_of(p, m))
                *C = __float2bfloat16_rn(y[0]);
#pragma unroll
            for (int c = 0; c < 7; ++c)
                y[c] = y[c + 1];
        }
    }
}

}  // namespace

template <int GS, bool E2M1, bool VEC>
__global__ void __launch_bounds__(kThreads, 2)
    matvec_w4_wide_kernel(const __grid_constant__ CUtensorMap tw, const __grid_constant__ W4Params p)
{
    constexpr int kStage = stage_bytes(GS, E2M1);
    constexpr int kScaleOff = kWeightBytes, kZeroOff = kScaleOff + kPartRows * GS * 2;
    // k of a buffer of unpacked weights: 64 columns of one number a weight or of two
    constexpr int kBatchK = E2M1 ? 128 : 64, kBatches = kStepK / kBatchK;
    constexpr int kChunks = kBatchK / 32;  // of 32 k, of a buffer
    extern __shared__ uint8_t smem_raw[];
    uint8_t *ring = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
    uint8_t *x_ring = ring + kStages * kStage;
    Shared &sh = *reinterpret_cast<Shared *>(x_ring + kXStages * kXBytes);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int tile_cols = p.swiglu ? 64 : kPartRows;
    const int cols = p.swiglu ? p.N / 2 : p.N;
    const int tiles = (cols + tile_cols - 1) / tile_cols;
    if (tid == 64) {
        tma_prefetch_map(&tw);
        for (int i = 0; i < kStages; ++i) {
            mbar_init(&sh.full[i], kStagers + 1);     // the staging warps, the producer
            mbar_init(&sh.empty[i], kUnpackers);
        }
        for (int i = 0; i < kXStages; ++i) {
            mbar_init(&sh.x_full[i], kStagers);
            mbar_init(&sh.x_empty[i], 1);
        }
        for (int i = 0; i < kBuffers; ++i) {
            mbar_init(&sh.a_full[i], kUnpackers);
            mbar_init(&sh.a_empty[i], 1);
        }
        mbar_init(&sh.sums_full, 1);
        mbar_init(&sh.drained, 1);
        fence_mbar_init();
        sh.abort = 0;
    }
    griddep_wait();
    griddep_launch_dependents();
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
    int stage = 0, xs = 0, buf = 0;
    uint32_t phase = 0, x_phase = 0, buf_phase = 0;
    auto advance = [](int &i, uint32_t &ph, int n) {
        if (++i == n) {
            i = 0;
            ph ^= 1;
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
                    if (!wait_long(&sh.empty[stage], phase ^ 1, kTimeoutNs, abort_flag)) {
                        ok = false;
                        break;
                    }
                    uint8_t *dst = ring + stage * kStage;
                    mbar_arrive_expect_tx(&sh.full[stage], kWeightBytes);
                    tma_load_2d(dst, &tw, &sh.full[stage], k * (kStepK / 2), y0);
                    tma_load_2d(dst + kWeightBytes / 2, &tw, &sh.full[stage], k * (kStepK / 2), y1);
                    ++issued;
                    advance(stage, phase, kStages);
                }
            }
            if (!ok) {
                give_up(p, sh);
                // the copies in flight land before the block's shared memory goes away
                volatile int no_abort = 0;
                for (int i = issued > kStages ? issued - kStages : 0; i < issued; ++i)
                    wait_long(&sh.full[i % kStages], (i / kStages) & 1, 1000000, &no_abort);
            }
        }
        __syncwarp();
    } else if (warp == 1) {
        // ---------------------------------------------------------------- products
        if (lane == 0) {
            bool ok = true;
            while (ok && walk.next(sh.run, tile_cols, seg)) {
                const uint32_t idesc = make_idesc(1u, 128, (seg.m1 - seg.m0 + 15) / 16 * 16);
                for (int k = seg.s0; ok && k < seg.s1; ++k) {
                    const int here = VEC || (k + 1) * kStepK <= p.K ? kStepK : p.K - k * kStepK;
#pragma unroll 1
                    for (int i = 0; i < kBatches; ++i) {
                        constexpr int kPer = kXK / kBatchK;  // batches of a stage of activations
                        ok = (i % kPer || wait_long(&sh.x_full[xs], x_phase, kTimeoutNs, abort_flag)) &&
                             wait_long(&sh.a_full[buf], buf_phase, kTimeoutNs, abort_flag);
                        if (!ok)
                            break;
                        tc_fence_after();
                        const uint32_t a = tmem + kRows + buf * kACols;
                        const uint32_t x = smem_u32(x_ring + xs * kXBytes) + i % kPer * kAtomBytes;
#pragma unroll
                        for (int j = 0; j < kBatchK / 16; ++j) {
                            if (!VEC && i * kBatchK + j * 16 >= here)
                                break;
                            const uint64_t b = desc_kmajor_sw128(x + j / 4 * kAtomBytes + j % 4 * 32);
                            mma_f16_tmem(tmem, a + j * 8, b, idesc, k > seg.s0 || i > 0 || j > 0);
                            if (!E2M1)
                                mma_f16_tmem(tmem, a + kACols / 2 + j * 8, b, idesc, 1);
                        }
                        mma_commit(&sh.a_empty[buf]);
                        advance(buf, buf_phase, kBuffers);
                        if (i % kPer == kPer - 1) {
                            mma_commit(&sh.x_empty[xs]);
                            advance(xs, x_phase, kXStages);
                        }
                    }
                }
                if (ok)
                    mma_commit(&sh.sums_full);
            }
            if (!ok)
                give_up(p, sh);
            // every product issued has ended once this arrives
            mma_commit(&sh.drained);
            volatile int no_abort = 0;
            wait_long(&sh.drained, 0, kTimeoutNs, &no_abort);
        }
        __syncwarp();
    } else if (warp < 2 + kStagers) {
        // ----------------------------------------- staging: activations and scales
        const int part = warp - 2;  // of every eight rows two, and the scales of 32 weight rows
        constexpr int kLoads = kRows / 8;
        const int groups = p.K / (kStepK / GS);
        bool ok = true;
        while (ok && walk.next(sh.run, tile_cols, seg)) {
            const int rows = seg.m1 - seg.m0;
            // the segment's rows 8 i + 2 part and the next, half a warp each (rows that are not
            // there are left as they are: nobody stores their sums)
            const uint4 *from[kLoads];
#pragma unroll
            for (int i = 0; i < kLoads; ++i) {
                const int m = seg.m0 + 8 * i + 2 * part + lane / 16;
                from[i] = m < seg.m1 ? reinterpret_cast<const uint4 *>(row_of(p, m)) : nullptr;
                if (m < seg.m1 && !from[i]) {
                    atomicOr(p.status, EP_STATUS_BOUNDS);
                    sh.run.skips = 1;
                }
                from[i] = from[i] ? from[i] + lane % 16 : nullptr;
            }
            const int scale_row = 32 * part + lane;
            int n = seg.n0 + (p.swiglu ? scale_row % 64 : scale_row);
            n = n < cols ? n : cols - 1;  // (rows past the last column: nobody stores them)
            const int64_t scale_at =
                (static_cast<int64_t>(seg.e) * p.N + n + (p.swiglu && scale_row >= 64 ? cols : 0)) * groups;
            Scales<GS, E2M1, VEC> sc;
            uint4 v[kLoads] = {};
            auto load_rows = [&](int k, int h) {  // k half h of step k
                const int at = k * (kStepK / 8) + h * (kXK / 8);
                const bool there = VEC || (at + lane % 16) * 8 < p.K;  // (no product reads the rest)
                // (two blocks of straight code: a branch a row would take longer than the row)
                auto load = [&](int i0) {
#pragma unroll
                    for (int i = i0; i < i0 + kLoads / 2; ++i)
                        if (from[i] && there)
                            v[i] = __ldg(from[i] + at);
                };
                load(0);
                if (rows > kRows / 2)
                    load(kLoads / 2);
            };
            auto store_rows = [&] {
                ok = __all_sync(0xffffffffu,
                                wait_long(&sh.x_empty[xs], x_phase ^ 1, kTimeoutNs, abort_flag));
                if (!ok)
                    return;
                const int r = 2 * part + lane / 16;  // (of eight: a swizzled row of 128 bytes)
                uint8_t *x = x_ring + xs * kXBytes + lane % 16 / 8 * kAtomBytes + r * 128 + ((lane % 8 ^ r) << 4);
                auto store = [&](int i0) {
#pragma unroll
                    for (int i = i0; i < i0 + kLoads / 2; ++i)
                        *reinterpret_cast<uint4 *>(x + i * 1024) = make_uint4(
                            __byte_perm(v[i].x, v[i].z, 0x5410), __byte_perm(v[i].x, v[i].z, 0x7632),
                            __byte_perm(v[i].y, v[i].w, 0x5410), __byte_perm(v[i].y, v[i].w, 0x7632));
                };
                store(0);
                if (rows > kRows / 2)
                    store(kLoads / 2);
                fence_proxy_async_shared();  // the products read them
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(&sh.x_full[xs]);
                advance(xs, x_phase, kXStages);
            };
            sc.load(p, scale_at + seg.s0 * GS, groups - seg.s0 * GS);
            load_rows(seg.s0, 0);
            for (int k = seg.s0; k < seg.s1; ++k) {
                ok = __all_sync(0xffffffffu,
                                wait_long(&sh.empty[stage], phase ^ 1, kTimeoutNs, abort_flag));
                if (!ok)
                    break;
                uint8_t *dst = ring + stage * kStage;
                const bool large = E2M1 && __any_sync(0xffffffffu, sc.large());
                if (E2M1 && lane == 0)
                    sh.large[stage][part] = large;
                sc.store(dst + kScaleOff + scale_row * GS * 2, dst + kZeroOff + scale_row * GS * 2, large);
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(&sh.full[stage]);
                advance(stage, phase, kStages);
                store_rows();
                if (!ok)
                    break;
                load_rows(k, 1);
                const bool more = k + 1 < seg.s1;
                if (more)
                    sc.load(p, scale_at + (k + 1) * GS, groups - (k + 1) * GS);
                store_rows();
                if (!ok)
                    break;
                if (more)
                    load_rows(k + 1, 0);
            }
        }
        if (!ok && lane == 0)
            give_up(p, sh);
    } else {
        // ------------------------------------------------------ unpacking, results
        const int quarter = warp & 3;
        const int row = 32 * quarter + lane, utid = tid - 32 * (2 + kStagers);
        const uint32_t my_lanes = tmem + (static_cast<uint32_t>(32 * quarter) << 16);
        const uint8_t *const scale0 = ring + kScaleOff + row * GS * 2;
        int segments = 0;
        bool ok = true;
        while (walk.next(sh.run, tile_cols, seg)) {
            for (int k = seg.s0; ok && k < seg.s1; ++k) {
                ok = __all_sync(0xffffffffu,
                                wait_long(&sh.full[stage], phase, kTimeoutNs, abort_flag));
                if (!ok)
                    break;
                const uint8_t *src = ring + stage * kStage;
                const bool large = E2M1 && sh.large[stage][quarter];
                for (int i = 0; i < kBatches; ++i) {
                    // (one after the other, the code has to stay small)
                    uint32_t a = my_lanes + kRows + buf * kACols;
                    ok = __all_sync(0xffffffffu, wait_long(&sh.a_empty[buf], buf_phase ^ 1, kTimeoutNs,
                                                           abort_flag));
                    if (!ok)
                        break;
                    tc_fence_after();
#pragma unroll 1
                    for (int j = 0; j < kChunks; ++j, a += 16) {
                        const int c = i * kChunks + j;
                        const uint8_t *at = scale0 + stage * kStage + c * GS / 8 * 2;
                        const uint4 codes =
                            *reinterpret_cast<const uint4 *>(src + row * 128 + ((c ^ row % 8) << 4));
                        const uint32_t w[4] = {codes.x, codes.y, codes.z, codes.w};
                        const uint32_t scale = *reinterpret_cast<const uint16_t *>(at) * 0x10001u;
                        uint32_t v[16];
                        if constexpr (E2M1) {
                            const uint32_t factor = large ? kTwo126 : scale;
#pragma unroll
                            for (int b = 0; b < 4; ++b)
                                unpack_e2m1(w[b], factor, *reinterpret_cast<uint32_t(*)[4]>(v + 4 * b));
                            if (large) {
#pragma unroll
                                for (int h = 0; h < 16; ++h)
                                    v[h] = bf16x2_mul(v[h], scale);
                            }
                            tmem_store(a, v);
                        } else {
                            const uint32_t zero = *reinterpret_cast<const uint16_t *>(at + kZeroOff - kScaleOff) * 0x10001u;
                            // the first part with a scale two steps short: it stays short of the
                            // product, and the second part has its sign (so that an infinite
                            // activation meets no 0 that the product is not)
                            const uint32_t less = (scale & 0x7FFFu) > 1 ? 0x00020002u : 0u;
                            const uint32_t minus = (scale - less) ^ 0x80008000u;
                            uint32_t lo[16];
#pragma unroll
                            for (int b = 0; b < 4; ++b) {
                                uint32_t t[4];
                                unpack_int(w[b], zero, t);
#pragma unroll
                                for (int h = 0; h < 4; ++h) {
                                    const uint32_t n = bf16x2_mul(t[h], minus);
                                    lo[4 * b + h] = bf16x2_fma(t[h], scale, n);
                                    v[4 * b + h] = n ^ 0x80008000u;
                                }
                            }
                            tmem_store(a, v);
                            tmem_store(a + kACols / 2, lo);
                        }
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
                    advance(buf, buf_phase, kBuffers);
                }
                if (!ok)
                    break;
                advance(stage, phase, kStages);
            }
            if (ok)
                ok = __all_sync(0xffffffffu,
                                wait_long(&sh.sums_full, segments & 1, kTimeoutNs, abort_flag));
            ++segments;
            // (all of the unpacking warps leave together: they meet at barriers below)
            if (!ok && lane == 0)
                give_up(p, sh);
            if (!named_bar_and(1, 32 * kUnpackers, ok)) {
                ok = false;
                break;
            }
            tc_fence_after();
            const bool whole = seg.s0 == 0 && seg.s1 == walk.steps;
            const int rows = seg.m1 - seg.m0, slot = seg.s0 == 0 ? 1 : 0;
#pragma unroll 1
            for (int c = 0; c < rows; c += 8) {
                float v[8];
                tmem_load(my_lanes + c, v);
                if (whole) {
                    store_sums(p, sh, seg, v, row, c);
                } else {
                    float4 *to = sums_of(p, blockIdx.x * 2 + slot) + c / 4 * kPartRows + row;
                    __stcg(to, make_float4(v[0], v[1], v[2], v[3]));
                    __stcg(to + kPartRows, make_float4(v[4], v[5], v[6], v[7]));
                }
            }
            if (!whole && utid == 0)
                sh.run.cut[slot] = seg;
            tc_fence_before();
        }
        join_cut_tiles<32 * kUnpackers>(p, sh.run, utid, ok, [&](const Segment &s, int from, int to) {
            const int rows = s.m1 - s.m0;
#pragma unroll 1
            for (int c = 0; c < rows; c += 8) {
                float v[8] = {};
                constexpr int kAhead = 4;  // blocks' sums under way at once
                for (int b0 = from; b0 <= to; b0 += kAhead) {
                    float4 x[kAhead], y[kAhead];
#pragma unroll
                    for (int i = 0; i < kAhead; ++i) {
                        const int b = b0 + i;
                        x[i] = y[i] = make_float4(0.f, 0.f, 0.f, 0.f);
                        if (b <= to) {
                            const float4 *theirs =
                                sums_of(p, b * 2 + (b == from ? 1 : 0)) + c / 4 * kPartRows + row;
                            x[i] = __ldcg(theirs), y[i] = __ldcg(theirs + kPartRows);
                        }
                    }
#pragma unroll
                    for (int i = 0; i < kAhead; ++i) {
                        v[0] += x[i].x, v[1] += x[i].y, v[2] += x[i].z, v[3] += x[i].w;
                        v[4] += y[i].x, v[5] += y[i].y, v[6] += y[i].z, v[7] += y[i].w;
                    }
                }
                store_sums(p, sh, s, v, row, c);
            }
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
