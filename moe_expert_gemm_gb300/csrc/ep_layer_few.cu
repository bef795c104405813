// A whole MoE layer for a few tokens, in two kernels: the up/gate products with the activation,
// and the down products with the gates.
//
//   h[row(t, e)] = SiLU(Wgate_e x_t) * (Wup_e x_t),   out[t] = sum_e g(t, e) W2_e h[row(t, e)]
//
// Every weight of an expert that has tokens is read once and meets at most 64 of them, so the
// call is bound by the weights' bytes. They stream through shared memory (TMA, 128-byte swizzle)
// into tcgen05.mma as its 128-row operand, straight from where they land; the tokens are the
// product's columns, 16 at least: no instruction of any warp touches a weight.
//
//  * A step is two tiles of 128 weight rows by 128 bytes of k. Up/gate: the gate rows of 128
//    intermediate indices and their up rows, whose sums meet in the same lane of tensor memory.
//    Down: twice as much k of 128 rows of the output, so that few blocks share a row's sum. The
//    tokens' pieces come along, from the L2.
//  * Work is a list of units of equal numbers of steps: up/gate, an expert's 128 indices; down,
//    128 rows of the output with all experts one after the other, so that a token's sum over
//    its experts never leaves the block. The list is cut into one run a block, of whole units or,
//    where that balances better, anywhere (Runs); units that are cut are joined through the
//    workspace by the last of their blocks, in block order.
//  * Sums are taken out of tensor memory into registers (fp32), a thread to a weight row: e4m3, of
//    each 128 k, with their scales; down, at an expert's end with the gates.
//    Tensor memory holds two periods' sums, so that the products go on meanwhile. Two groups
//    of four warps do that: one for the gate and one for the up rows, or (down) for half of
//    the tokens each.
//  * The plan (who has which expert) is made by every block for itself from the ids, with a
//    64-bit mask of tokens for each expert.
//  * The second kernel starts while the first one's last blocks finish: a block makes its plan
//    and fills its ring with weights before it waits for the activations.
//
// Measured (several GB300s; weights' bytes of the copy bandwidth of 6.77 TB/s): a token with 2 of 8
// experts of 4096 x 14336 113 to 116 us, 90 to 92 %; 16 tokens, 8 of 32 of 7168 x 2048 in e4m3 210 to 222 us,
// 93 to 98 %; 64 tokens, 8 of 16 of 4096 x 2048 142 to 145 us, 82 to 84 %; 5 tokens, 3 of 12 of 1496 x 1000
// 23 to 25 us, of which the bytes are 8.
#include <type_traits>

#include "ep_internal.h"
#include "ep_ptx.cuh"
#include "ep_rows.cuh"

namespace ep {

namespace {

constexpr int kTile = 128;                     // weight rows of one product
constexpr int kWeightBytes = 2 * kTile * 128;  // of a step
constexpr int kMaxBlocks = 160;
constexpr int kMaxRows = EP_MAX_FEW_TOKENS * 32;
constexpr int kEpilogueWarps = 8;  // two groups of four
constexpr int kThreads = 32 * (4 + kEpilogueWarps);
constexpr int kEpilogueThreads = 32 * kEpilogueWarps;
constexpr int kPartBase = EP_FEW_COUNTER_BYTES;  // of the workspace; counters before it
static_assert(kMaxBlocks * 4 <= kPartBase, "counters");

// How the list is cut. Steps that the joining of cut units is worth, and the fewest steps that a cut
// leaves a block: the last block of a unit adds a part of its tokens' sums for each of them. A
// compromise, which the times do not single out: over 90 shapes of 1 to 64 tokens the geometric mean lies
// 0.8 % under that of half of sqrt(steps) for any number of tokens, 0.6 % under that of a joining worth 3
// steps, 0.4 % under that of 0.1 + tokens / 64 below the root, while a single shape moves by up to 20 %
// either way, and shapes that neither touches by some per cent from run to run.
constexpr int kJoinSteps = 4;

__device__ __forceinline__ int min_steps(int steps, int tokens)
{
    const int s = static_cast<int>(ceilf(sqrtf((0.1f + tokens * 0.01f) * steps)));
    return s < 2 ? 2 : s > 64 ? 64 : s;
}

struct Segment {
    int unit, s0, s1;  // steps [s0, s1) of the unit
};

// How the units' steps are cut into the blocks' runs.
struct Runs {
    int per, rest;  // pieces of every run; the first `rest` runs have one more
    int piece;      // steps of a piece: 1, or a unit's

    // The block whose run holds step i (of runs cut at any step).
    __device__ int owner(int i) const
    {
        return i < rest * (per + 1) ? i / (per + 1) : rest + (i - rest * (per + 1)) / per;
    }
};

template <bool DOWN, int NT>
constexpr int stage_bytes()
{
    return kWeightBytes + (DOWN ? 2 : 1) * NT * 128;
}

template <bool DOWN, int NT>
constexpr int stages()
{
    return !DOWN && NT == 16 ? 6 : DOWN && NT == 64 ? 4 : 5;
}

// Exchange of up to 16 tokens' sums: 128 gate rows, their 128 up rows.
constexpr int kWindow = 16;
struct Exchange {
    alignas(16) float sums[kWindow][2 * kTile];  // (read in pieces of four)
};

// e4m3: the scales of some periods ahead, of the tokens (up/gate) or of the expert's rows (down),
// and of the weights: gate and up rows, or two blocks of k.
constexpr int kScaleStages = 8;
template <int NT>
struct Scales {
    uint64_t full[kScaleStages], empty[kScaleStages];
    float token[kScaleStages][2][NT], weight[kScaleStages][2];
};
struct Nothing {};

// Gates of each slot, of each row, and the slots' local experts (-1: not here).
struct Gates {
    float of_slot[kMaxRows], of_row[kMaxRows];
    int16_t expert[kMaxRows];
};

template <bool DOWN, bool FP8, int NT>
struct Shared {
    uint64_t full[6], empty[6];
    uint64_t sums_full[2], sums_empty[2];
    uint64_t drained;
    uint32_t mask[EP_MAX_LOCAL_EXPERTS][2];  // tokens of each local expert
    uint32_t tmem;
    int abort;
    int n_active, rows, start, todo;  // active experts, their tokens; the run
    Runs runs;
    Segment cut[2];  // the units the block's run begins and ends inside
    int last[2];
    uint16_t active[EP_MAX_LOCAL_EXPERTS];  // experts that have tokens, ascending
    uint16_t place[EP_MAX_LOCAL_EXPERTS];   // of an expert among them
    int16_t first[EP_MAX_LOCAL_EXPERTS];    // first row of the place's tokens
    std::conditional_t<DOWN, Gates, Exchange> x;
    std::conditional_t<FP8, Scales<NT>, Nothing> scales;

    __device__ uint64_t tokens(int e) const { return mask[e][0] | static_cast<uint64_t>(mask[e][1]) << 32; }
};

template <bool DOWN, bool FP8, int NT>
constexpr int smem_bytes()
{
    return 1024 + stages<DOWN, NT>() * stage_bytes<DOWN, NT>() + static_cast<int>(sizeof(Shared<DOWN, FP8, NT>));
}

template <typename S>
__device__ __forceinline__ void give_up(const FewParams &p, S &sh)
{
    atomicOr(p.status, EP_STATUS_TIMEOUT);
    *reinterpret_cast<volatile int *>(&sh.abort) = 1;
}

// Which tokens each local expert has, the experts that have some, the first row of each, and
// (down) every row's gate. All threads, the masks zero; the gates are there after another barrier.
// (Past the first level of cache: the second kernel reads ids and gates before it waits.)
template <bool DOWN, typename S>
__device__ __forceinline__ void make_plan(const FewParams &p, S &sh)
{
    const int tid = threadIdx.x, slots = p.T * p.top_k, first = p.my_rank * p.El;
    bool bad = false;
    for (int s = tid; s < slots; s += kThreads) {
        const int id = __ldcg(p.topk_ids + s), t = s / p.top_k;
        const bool here = id >= first && id < first + p.El;
        const int e = here ? id - first : -1;
        bad |= id < 0 || id >= p.n_ranks * p.El;
        if (here)
            atomicOr(&sh.mask[e][t / 32], 1u << t % 32);
        if constexpr (DOWN) {
            sh.x.expert[s] = static_cast<int16_t>(e);
            sh.x.of_slot[s] = __ldcg(p.gates + s);
        }
    }
    if (!DOWN && bad && blockIdx.x == 0)
        atomicOr(p.status, EP_STATUS_ROUTING);
    __syncthreads();
    if (tid < 32) {
        int places = 0, rows = 0;
        for (int e0 = 0; e0 < p.El; e0 += 32) {
            const int e = e0 + tid, n = e < p.El ? __popcll(sh.tokens(e)) : 0;
            const uint32_t has = __ballot_sync(0xffffffffu, n > 0);
            int upto = n;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int v = __shfl_up_sync(0xffffffffu, upto, o);
                if (tid >= o)
                    upto += v;
            }
            if (n > 0) {
                const int place = places + __popc(has & ((1u << tid) - 1));
                sh.active[place] = static_cast<uint16_t>(e);
                sh.place[e] = static_cast<uint16_t>(place);
                sh.first[place] = static_cast<int16_t>(rows + upto - n);
            }
            places += __popc(has);
            rows += __shfl_sync(0xffffffffu, upto, 31);
        }
        if (tid == 0) {
            sh.n_active = places;
            sh.rows = rows;
        }
    }
    __syncthreads();
    if constexpr (DOWN) {
        for (int s = tid; s < slots; s += kThreads) {
            const int t = s / p.top_k, s0 = t * p.top_k, e = sh.x.expert[s];
            if (e < 0)
                continue;
            // an expert named twice: the first slot has the sum of the gates
            bool again = false;
            for (int i = s0; i < s; ++i)
                again |= sh.x.expert[i] == e;
            if (again)
                continue;
            float g = sh.x.of_slot[s];
            for (int i = s + 1; i < s0 + p.top_k; ++i)
                if (sh.x.expert[i] == e)
                    g += sh.x.of_slot[i];
            sh.x.of_row[sh.first[sh.place[e]] + __popcll(sh.tokens(e) & ((1ull << t) - 1))] = g;
        }
    }
}

// The segments of a block's run, one after the other.
struct Walk {
    int unit, s0, todo, steps;

    template <typename S>
    __device__ Walk(const S &sh, int steps_)
        : unit(steps_ ? sh.start / steps_ : 0), s0(steps_ ? sh.start - unit * steps_ : 0), todo(sh.todo), steps(steps_)
    {
    }

    __device__ __forceinline__ bool next(Segment &s)
    {
        if (todo <= 0)
            return false;
        s.unit = unit++;
        s.s0 = s0;
        s.s1 = todo < steps - s0 ? s0 + todo : steps;
        todo -= s.s1 - s.s0;
        s0 = 0;
        return true;
    }
};

// Four bytes to shared memory behind the thread's back, and its arrival at a barrier once all
// that it has asked for is there.
__device__ __forceinline__ void copy_word(float *to, const float *from)
{
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(smem_u32(to)), "l"(from) : "memory");
}

__device__ __forceinline__ void copy_arrive(uint64_t *bar)
{
    asm volatile("cp.async.mbarrier.arrive.noinc.shared.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}

template <typename T>
__device__ __forceinline__ void advance(int &i, T &phase, int n)
{
    if (++i == n) {
        i = 0;
        phase ^= 1;
    }
}

}  // namespace

int few_columns(int T) { return T <= 16 ? 16 : T <= 32 ? 32 : 64; }

int64_t few_workspace_rows(int T)
{
    return kPartBase + static_cast<int64_t>(kMaxBlocks) * 2 * few_columns(T) * 2 * kTile * 4;
}

// In the workspace: counters, partial sums, the activation's rows, and (e4m3) their scales.
static int64_t few_workspace_scales(const FewParams &p)
{
    const int64_t rows = static_cast<int64_t>(p.T) * p.top_k;
    return few_workspace_rows(p.T) + (rows * p.I * (p.fp8 ? 1 : 2) + 127) / 128 * 128;
}

int64_t few_workspace_bytes(const FewParams &p)
{
    return few_workspace_scales(p) + (p.fp8 ? static_cast<int64_t>(p.T) * p.top_k * (p.I / 128) * 4 : 0);
}

// NT: columns of a product at most, 16, 32 or 64.
template <bool DOWN, bool FP8, int NT>
__global__ void __launch_bounds__(kThreads, 1)
    few_kernel(const __grid_constant__ CUtensorMap tw, const __grid_constant__ CUtensorMap tx,
               const __grid_constant__ FewParams p, uint8_t *h_rows, float *h_scales)
{
    constexpr int kStages = stages<DOWN, NT>();
    constexpr int kStage = stage_bytes<DOWN, NT>();
    constexpr int kBlockK = FP8 ? 128 : 64;            // k of 128 bytes
    constexpr int kStepK = DOWN ? 2 * kBlockK : kBlockK;
    constexpr int kUnitRows = kTile;                   // (of the gate, too, of the up matrix)
    // two periods of two products' sums; e4m3, down: and NT columns of scratch
    constexpr uint32_t kTmemCols = (DOWN && FP8 ? 8 : 4) * NT;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *ring = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
    using Sh = Shared<DOWN, FP8, NT>;
    Sh &sh = *reinterpret_cast<Sh *>(ring + kStages * kStage);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    if (tid == 64) {
        tma_prefetch_map(&tw);
        tma_prefetch_map(&tx);
        for (int i = 0; i < kStages; ++i) {
            mbar_init(&sh.full[i], 1);
            mbar_init(&sh.empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&sh.sums_full[i], 1);
            mbar_init(&sh.sums_empty[i], kEpilogueWarps);
        }
        mbar_init(&sh.drained, 1);
        if constexpr (FP8)
            for (int i = 0; i < kScaleStages; ++i) {
                mbar_init(&sh.scales.full[i], 32);
                mbar_init(&sh.scales.empty[i], kEpilogueWarps);
            }
        fence_mbar_init();
        sh.abort = 0;
        sh.cut[0].unit = sh.cut[1].unit = -1;
        sh.last[0] = sh.last[1] = 0;
    }
    for (int e = tid; e < p.El; e += kThreads)
        sh.mask[e][0] = sh.mask[e][1] = 0;
    __syncthreads();
    if (!DOWN) {
        griddep_wait();
        griddep_launch_dependents();
    }
    // (tensor memory only now: the previous kernel may still have wanted it. The second kernel's block
    // finds its SM left by the first one's, which held as much shared memory)
    if (warp == kThreads / 32 - 1) {
        tmem_alloc(&sh.tmem, kTmemCols);
        tmem_relinquish();
    }
    // (the first kernel waited for all that came before it ahead of letting the second one start:
    // ids, gates and weights are there; only what the first kernel writes is waited for below)
    make_plan<DOWN>(p, sh);
    const int tiles = ((DOWN ? p.H : p.I) + kUnitRows - 1) / kUnitRows;
    const int expert_steps = ((DOWN ? p.I : p.H) + kStepK - 1) / kStepK;
    const int units = DOWN ? tiles : tiles * sh.n_active;
    const int steps = DOWN ? expert_steps * sh.n_active : expert_steps;
    if (tid == 0) {
        const int grid = static_cast<int>(gridDim.x), block = static_cast<int>(blockIdx.x);
        const int total = units * steps;
        const int least = min_steps(steps, DOWN ? p.T : sh.n_active ? sh.rows / sh.n_active : 0);
        int cut = (total + grid - 1) / grid;
        cut = cut < least ? least : cut;
        const bool whole = (units + grid - 1) / grid * steps <= cut + kJoinSteps;
        const int blocks = whole || total / grid >= least ? grid : (total + least - 1) / least;
        Runs runs;
        runs.piece = whole ? steps : 1;
        runs.per = (whole ? units : total) / blocks;
        runs.rest = (whole ? units : total) - runs.per * blocks;
        sh.runs = runs;
        sh.start = (block * runs.per + (block < runs.rest ? block : runs.rest)) * runs.piece;
        sh.todo = block < blocks ? (runs.per + (block < runs.rest)) * runs.piece : 0;
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = sh.tmem;
    volatile int *abort_flag = &sh.abort;
    Walk walk(sh, steps);
    Segment seg;
    int stage = 0;
    uint32_t phase = 0;

    if (warp == 0) {
        // ------------------------------------------- producer: weights and columns
        if (lane == 0) {
            // one step's place, coordinates and columns
            struct At {
                int unit, place, k;
            };
            auto start_of = [&](const Segment &s) {
                return DOWN ? At{s.unit, s.s0 / expert_steps, s.s0 % expert_steps}
                            : At{s.unit % tiles, s.unit / tiles, s.s0};
            };
            auto columns = [&](const At &at) {  // (in 16s)
                return DOWN ? (__popcll(sh.tokens(sh.active[at.place])) + 15) / 16 : NT / 16;
            };
            // (the L2 keeps tokens, activations and partial sums rather: 64 tokens, 8 of 16 experts
            // of 4096 x 2048, 156 us a call, without 162)
            const uint64_t once = policy_evict_first();
            auto load_weights = [&](const At &at, int i) {
                const int e = sh.active[at.place], y = at.unit * kUnitRows, x = at.k * kStepK;
                uint8_t *dst = ring + i * kStage;
                mbar_arrive_expect_tx(&sh.full[i], kWeightBytes + columns(at) * (DOWN ? 4096 : 2048));
                tma_load_3d_once(dst, &tw, &sh.full[i], x, y, e, once);
                tma_load_3d_once(dst + kTile * 128, &tw, &sh.full[i], DOWN ? x + kBlockK : x, DOWN ? y : y + p.I,
                                 e, once);
            };
            auto load_columns = [&](const At &at, int i) {
                uint8_t *dst = ring + i * kStage + kWeightBytes;
                if (DOWN) {
                    const int n = columns(at), row = sh.first[at.place], x = at.k * kStepK;
                    for (int c = 0; c < n; ++c) {
                        tma_load_2d(dst + c * 2048, &tx, &sh.full[i], x, row + 16 * c);
                        tma_load_2d(dst + NT * 128 + c * 2048, &tx, &sh.full[i], x + kBlockK, row + 16 * c);
                    }
                } else {
                    tma_load_2d(dst, &tx, &sh.full[i], at.k * kStepK, 0);
                }
            };
            int issued = 0;
            bool ok = true;
            if (DOWN) {
                // a ring full of weights, then, once they are there, its columns
                for (int pass = 0; pass < 2; ++pass) {
                    Walk ahead = walk;
                    int n = 0;
                    if (pass == 1)
                        griddep_wait();
                    while (n < kStages && ahead.next(seg)) {
                        At at = start_of(seg);
                        for (int s = seg.s0; s < seg.s1 && n < kStages; ++s, ++n) {
                            if (pass == 0)
                                load_weights(at, n);
                            else
                                load_columns(at, n);
                            if (++at.k == expert_steps)
                                at.k = 0, ++at.place;
                        }
                    }
                    issued = n;
                }
            }
            int skip = issued;
            while (ok && walk.next(seg)) {
                At at = start_of(seg);
                for (int s = seg.s0; s < seg.s1; ++s) {
                    if (skip > 0) {
                        --skip;
                    } else {
                        if (!mbar_wait(&sh.empty[stage], phase ^ 1, p.timeout_ns, abort_flag)) {
                            ok = false;
                            break;
                        }
                        load_weights(at, stage);
                        load_columns(at, stage);
                        ++issued;
                    }
                    advance(stage, phase, kStages);
                    if (DOWN && ++at.k == expert_steps)
                        at.k = 0, ++at.place;
                    else if (!DOWN)
                        ++at.k;
                }
            }
            if (!ok)
                give_up(p, sh);
            wait_for_copies<kStages>(sh.full, issued, kEndNs);
        }
        __syncwarp();
    } else if (warp == 1) {
        // ---------------------------------------------------------------- products
        if (lane == 0) {
            // (the columns come after the first kernel: the waits' limits do not count its time)
            if (DOWN)
                griddep_wait();
            bool ok = true;
            int buf = 0;
            uint32_t buf_phase = 0;
            while (ok && walk.next(seg)) {
                int place = DOWN ? seg.s0 / expert_steps : 0, k = DOWN ? seg.s0 % expert_steps : seg.s0;
                bool fresh = true;  // a period begins
                uint32_t idesc = 0;
                for (int s = seg.s0; s < seg.s1; ++s) {
                    if (fresh) {
                        const int n = DOWN ? __popcll(sh.tokens(sh.active[place])) : p.T;
                        idesc = make_idesc(FP8 ? 0u : 1u, kTile, (n + 15) / 16 * 16);
                        ok = mbar_wait(&sh.sums_empty[buf], buf_phase ^ 1, p.timeout_ns, abort_flag);
                    }
                    ok = ok && mbar_wait(&sh.full[stage], phase, p.timeout_ns, abort_flag);
                    if (!ok)
                        break;
                    tc_fence_after();
                    const uint32_t w = smem_u32(ring + stage * kStage), x = w + kWeightBytes;
                    // the step's two tiles: other rows (up/gate) or k (down) of their own, or, bf16,
                    // more of the same sum
                    const uint32_t d = tmem + buf * 2 * NT;
                    constexpr bool one_sum = DOWN && !FP8;
#pragma unroll
                    for (int i = 0; i < 2; ++i)
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            const uint64_t a = desc_kmajor_sw128(w + i * kTile * 128 + j * 32);
                            const uint64_t b = desc_kmajor_sw128(x + (DOWN ? i * NT * 128 : 0) + j * 32);
                            const uint32_t more = !fresh || j > 0 || (one_sum && i > 0);
                            if (FP8)
                                mma_f8(d + i * NT, a, b, idesc, more);
                            else
                                mma_f16(one_sum ? d : d + i * NT, a, b, idesc, more);
                        }
                    mma_commit(&sh.empty[stage]);
                    advance(stage, phase, kStages);
                    const bool expert_ends = ++k == expert_steps;
                    fresh = FP8 || s + 1 == seg.s1 || (DOWN && expert_ends);
                    if (fresh) {
                        mma_commit(&sh.sums_full[buf]);
                        advance(buf, buf_phase, 2);
                    }
                    if (expert_ends)
                        k = 0, ++place;
                }
            }
            if (!ok)
                give_up(p, sh);
            // every product issued has ended once this arrives
            mma_commit(&sh.drained);
            volatile int no_abort = 0;
            mbar_wait(&sh.drained, 0, kEndNs, &no_abort);
        }
        __syncwarp();
    } else if (warp >= 4) {
        // ------------------------------------------------------------ sums, results
        if (DOWN)
            griddep_wait();
        const int group = (warp - 4) / 4, quarter = warp & 3, row = 32 * quarter + lane;
        const int etid = tid - 32 * 4;
        // this thread's row of `tokens` sums: of the gate or the up rows, or of half of the tokens
        constexpr int kTokens = DOWN ? NT / 2 : NT;
        const int base = DOWN ? group * kTokens : 0;
        const uint32_t my_sums = tmem + (DOWN ? 0 : group * NT) + (static_cast<uint32_t>(32 * quarter) << 16);
        float *const parts = reinterpret_cast<float *>(p.workspace + kPartBase);
        constexpr int kPartRows = DOWN ? kTile : 2 * kTile;  // of a part, by NT tokens
        auto part_of = [&](int slot) {
            return parts + (static_cast<int64_t>(slot) * NT + base) * kPartRows + (DOWN ? 0 : group * kTile) + row;
        };
        static_assert(kPartBase % 16 == 0, "sums are read in pieces of four");
        // (bit t: token base + t)
        auto mine = [&](uint64_t mask) {
            return DOWN ? (mask >> base) & ((1ull << kTokens) - 1) : mask;
        };
        const uint64_t all_tokens = mine(p.T == 64 ? ~0ull : (1ull << p.T) - 1);
        float acc[kTokens];

        // Up/gate: a warp's row of the activation, 4 of the unit's 128 indices a lane, from the sums.
        auto store_activation = [&](int unit, int64_t r, const float4 &g, const float4 &u) {
            const int i = unit % tiles * kUnitRows + 4 * lane;
            const float v[4] = {rows::silu_times(g.x, u.x), rows::silu_times(g.y, u.y),
                                rows::silu_times(g.z, u.z), rows::silu_times(g.w, u.w)};
            if constexpr (FP8) {
                uint32_t m = 0;
#pragma unroll
                for (int c = 0; c < 4; ++c)
                    m = max(m, rows::size_bits(v[c]));
                const float scale = rows::scale_of(__reduce_max_sync(0xffffffffu, m)), inv = rows::inverse_of(scale);
                *reinterpret_cast<uint32_t *>(h_rows + r * p.I + i) =
                    rows::e4m3x4(v[0] * inv, v[1] * inv, v[2] * inv, v[3] * inv);
                if (lane == 0)
                    h_scales[r * (p.I / 128) + i / 128] = scale;
            } else if (i < p.I) {  // (a multiple of 8)
                *reinterpret_cast<uint2 *>(h_rows + (r * p.I + i) * 2) =
                    make_uint2(rows::pack(v[0], v[1]), rows::pack(v[2], v[3]));
            }
        };

        // A whole unit's sums in acc: the activation's rows, or the output's.
        auto finish = [&](int unit) {
            if constexpr (DOWN) {
                const int n = unit * kUnitRows + row;
                if (n < p.H) {
                    __nv_bfloat16 *out = reinterpret_cast<__nv_bfloat16 *>(p.out) + static_cast<int64_t>(base) * p.H + n;
#pragma unroll
                    for (int t = 0; t < kTokens; ++t)
                        if (all_tokens >> t & 1)
                            out[static_cast<int64_t>(t) * p.H] = __float2bfloat16_rn(acc[t]);
                }
            } else {
                const int place = unit / tiles;
                const uint64_t mask = sh.tokens(sh.active[place]);
                int at = sh.first[place];  // the next token's row
#pragma unroll
                for (int t0 = 0; t0 < NT; t0 += kWindow) {
                    const uint32_t here = static_cast<uint32_t>(mask >> t0) & 0xFFFF;
                    if (!here)
                        continue;
                    int n = 0;
#pragma unroll
                    for (int c = 0; c < kWindow; ++c)
                        if (here >> c & 1)
                            sh.x.sums[n++][group * kTile + row] = acc[t0 + c];
                    named_bar_sync(1, kEpilogueThreads);
                    for (int j = warp - 4; j < n; j += kEpilogueWarps) {
                        const float4 *sums = reinterpret_cast<const float4 *>(sh.x.sums[j]);
                        store_activation(unit, at + j, sums[lane], sums[32 + lane]);
                    }
                    at += n;
                    named_bar_sync(1, kEpilogueThreads);
                }
            }
        };

        // e4m3, down: the sums of the expert under way, its tokens without gaps.
        float own[DOWN && FP8 ? kTokens : 1];
        const uint32_t my_scratch = tmem + 4 * NT + group * kTokens + (static_cast<uint32_t>(32 * quarter) << 16);
        // The block's sums of a cut unit are stored: counts it in. The part that a run begins with is
        // counted long before the block before ends its own, the unit's first, which so is the
        // one that joins: a block seldom has two units to join.
        auto count_in = [&](int slot, bool ok) {
            if (!named_bar_and(1, kEpilogueThreads, ok))
                return false;
            if (etid == 0) {
                int *counters = reinterpret_cast<int *>(p.workspace);
                const int unit = sh.cut[slot].unit;
                const int c0 = sh.runs.owner(unit * steps), c1 = sh.runs.owner(unit * steps + steps - 1);
                const int last = atom_add_acq_rel_gpu(counters + c0, 1) == c1 - c0;
                if (last)
                    counters[c0] = 0;  // ready for the next call
                sh.last[slot] = last;
            }
            return true;
        };

        bool ok = true;
        int buf = 0;
        uint32_t buf_phase = 0;
        int sc = 0;
        uint32_t sc_phase = 0;
        while (walk.next(seg)) {
#pragma unroll
            for (int t = 0; t < kTokens; ++t)
                acc[t] = 0.f;
            if constexpr (DOWN && FP8)
#pragma unroll
                for (int t = 0; t < kTokens; ++t)
                    own[t] = 0.f;
            int place = DOWN ? seg.s0 / expert_steps : seg.unit / tiles;
            int k = DOWN ? seg.s0 % expert_steps : seg.s0;
            for (int s = seg.s0; ok && s < seg.s1;) {
                // one period: its steps, tokens and factors
                const uint64_t mask = sh.tokens(sh.active[place]), here = mine(mask);
                int n = FP8 ? 1 : (DOWN ? expert_steps - k : seg.s1 - s);
                n = n < seg.s1 - s ? n : seg.s1 - s;
                int next_place = place, next_k = k + n;
                if (next_k == expert_steps)
                    next_k = 0, ++next_place;
                // lane i's factors: up/gate, of tokens i and i + 32; down, of the expert's i-th token of
                // this half, two blocks of k
                const int first = DOWN ? __popcll(mask & ((1ull << base) - 1)) : 0, count = __popcll(here);
                float factor[2];
                if constexpr (FP8) {
                    ok = __all_sync(0xffffffffu,
                                    mbar_wait(&sh.scales.full[sc], sc_phase, p.timeout_ns, abort_flag));
                    if (!ok)
                        break;
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        // (a block past the end of k has no scales; its sums are 0)
                        const bool there = DOWN ? lane < count && 2 * k + i < p.I / 128
                                                : 32 * i + lane < NT && (mask >> (32 * i + lane) & 1);
                        factor[i] = !there ? 0.f
                                    : DOWN ? sh.scales.token[sc][i][first + lane] * sh.scales.weight[sc][i]
                                           : sh.scales.token[sc][0][32 * i + lane] * sh.scales.weight[sc][group];
                    }
                    __syncwarp();
                    if (lane == 0)
                        mbar_arrive(&sh.scales.empty[sc]);
                    advance(sc, sc_phase, kScaleStages);
                }
                ok = __all_sync(0xffffffffu,
                                mbar_wait(&sh.sums_full[buf], buf_phase, p.timeout_ns, abort_flag));
                if (!ok)
                    break;
                tc_fence_after();
                const uint32_t from = my_sums + buf * 2 * NT + first;
                if constexpr (!DOWN) {
                    // columns: the tokens (nobody uses the sums of those that are not the expert's)
#pragma unroll
                    for (int t0 = 0; t0 < kTokens; t0 += 16) {
                        if (!(here >> t0 & 0xFFFF))
                            continue;
                        uint32_t v[16];
                        tmem_ld_32x32b_x16(from + t0, v);
                        tmem_ld_wait();
                        tmem_regs_ready(v);
#pragma unroll
                        for (int c = 0; c < 16; ++c) {
                            if (FP8) {
                                const float f = __shfl_sync(0xffffffffu, factor[t0 / 32], (t0 + c) % 32);
                                acc[t0 + c] = fmaf(f, __uint_as_float(v[c]), acc[t0 + c]);
                            } else {
                                acc[t0 + c] = __uint_as_float(v[c]);
                            }
                        }
                    }
                } else {
                    // columns: the expert's tokens without gaps
                    if constexpr (FP8) {
#pragma unroll
                        for (int c0 = 0; c0 < kTokens; c0 += 8) {
                            if (c0 >= count)
                                continue;
                            uint32_t v[2][8];
                            tmem_ld_32x32b_x8(from + c0, v[0]);
                            tmem_ld_32x32b_x8(from + NT + c0, v[1]);
                            tmem_ld_wait();
                            tmem_regs_ready(v[0]);
                            tmem_regs_ready(v[1]);
#pragma unroll
                            for (int c = 0; c < 8; ++c)
#pragma unroll
                                for (int i = 0; i < 2; ++i) {
                                    const float f = __shfl_sync(0xffffffffu, factor[i], c0 + c);
                                    own[c0 + c] = fmaf(f, __uint_as_float(v[i][c]), own[c0 + c]);
                                }
                        }
                    }
                    if (next_k == 0 || s + n == seg.s1) {
                        // the expert's sums, each to its token's place in acc, by way of tensor memory
                        // (whose columns can be chosen at run time), with the gates
                        uint32_t at = from;
                        if constexpr (FP8) {
                            at = my_scratch;
#pragma unroll
                            for (int c0 = 0; c0 < kTokens; c0 += 8) {
                                uint32_t v[8];
#pragma unroll
                                for (int c = 0; c < 8; ++c) {
                                    v[c] = __float_as_uint(own[c0 + c]);
                                    own[c0 + c] = 0.f;
                                }
                                if (c0 < count)
                                    tmem_st_32x32b_x8(at + c0, v);
                            }
                            tmem_st_wait();
                        }
                        float gate = 0.f;
                        if (lane < kTokens && (here >> lane & 1))
                            gate = sh.x.of_row[sh.first[place] + first + __popcll(here & ((1ull << lane) - 1))];
                        constexpr int kAtOnce = kTokens < 16 ? 8 : 16;
#pragma unroll
                        for (int t0 = 0; t0 < kTokens; t0 += kAtOnce) {
                            const uint32_t now = static_cast<uint32_t>(here >> t0) & ((1u << kAtOnce) - 1);
                            if (!now)
                                continue;
                            uint32_t v[kAtOnce];
#pragma unroll
                            for (int c = 0; c < kAtOnce; ++c) {
                                v[c] = 0;
                                if (now >> c & 1)
                                    v[c] = tmem_ld_32x32b_x1(at++);
                            }
                            tmem_ld_wait();
                            tmem_regs_ready(v);
#pragma unroll
                            for (int c = 0; c < kAtOnce; ++c)
                                if (now >> c & 1) {
                                    const float g = __shfl_sync(0xffffffffu, gate, t0 + c);
                                    acc[t0 + c] = fmaf(g, __uint_as_float(v[c]), acc[t0 + c]);
                                }
                        }
                    }
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(&sh.sums_empty[buf]);
                advance(buf, buf_phase, 2);
                s += n;
                place = next_place, k = next_k;
            }
            // (all of these warps leave together: they meet at barriers below)
            if (!ok && lane == 0)
                give_up(p, sh);
            if (!named_bar_and(1, kEpilogueThreads, ok)) {
                ok = false;
                break;
            }
            if (seg.s0 == 0 && seg.s1 == steps) {
                finish(seg.unit);
            } else {
                const int slot = seg.s0 == 0 ? 1 : 0;
                const uint64_t tokens = DOWN ? all_tokens : sh.tokens(sh.active[seg.unit / tiles]);
                float *to = part_of(blockIdx.x * 2 + slot);
#pragma unroll
                for (int t = 0; t < kTokens; ++t)
                    if (tokens >> t & 1)
                        __stcg(to + t * kPartRows, acc[t]);
                if (etid == 0)
                    sh.cut[slot] = seg;
                ok = count_in(slot, ok);
                if (!ok)
                    break;
            }
        }
        // the block's cut units, after all else: the last of a unit's blocks to count itself in adds
        // what they left, in block order
        if (sh.runs.piece == 1 && named_bar_and(1, kEpilogueThreads, ok)) {
            for (int slot = 0; slot < 2; ++slot) {
                if (!sh.last[slot])
                    continue;
                const int unit = sh.cut[slot].unit;
                const int c0 = sh.runs.owner(unit * steps), c1 = sh.runs.owner(unit * steps + steps - 1);
                const int place = DOWN ? 0 : unit / tiles, i0 = (unit - place * tiles) * kUnitRows + 4 * lane;
                const uint64_t tokens = DOWN ? (p.T == 64 ? ~0ull : (1ull << p.T) - 1) : sh.tokens(sh.active[place]);
                const int count = __popcll(tokens);
                // A warp takes a token's 128 rows (gate and up, each), a lane four of them; kAtATime
                // tokens' and kAhead blocks' sums are under way at once.
                constexpr int kAtATime = NT == 16 ? 1 : DOWN ? NT / kEpilogueWarps : NT / 16;
                constexpr int kAhead = (DOWN ? 16 : 8) / kAtATime;
                uint64_t left = tokens;  // from this warp's next token on
                auto skip = [&](int n) {
                    for (int i = 0; i < n; ++i)
                        left &= left - 1;
                };
                skip(warp - 4);
                for (int j0 = warp - 4; j0 < count; j0 += kEpilogueWarps * kAtATime) {
                    int token[kAtATime];
                    float4 sum[kAtATime][DOWN ? 1 : 2];
#pragma unroll
                    for (int a = 0; a < kAtATime; ++a) {
                        token[a] = __ffsll(static_cast<long long>(left)) - 1;  // (-1: none)
                        skip(kEpilogueWarps);
                        for (int g = 0; g < (DOWN ? 1 : 2); ++g)
                            sum[a][g] = make_float4(0.f, 0.f, 0.f, 0.f);
                    }
                    for (int b0 = c0; b0 <= c1; b0 += kAhead) {
                        float4 v[kAhead][kAtATime][DOWN ? 1 : 2];
#pragma unroll
                        for (int h = 0; h < kAhead; ++h) {
                            const int b = b0 + h, from = b * 2 + (b == c0 ? 1 : 0);
#pragma unroll
                            for (int a = 0; a < kAtATime; ++a)
#pragma unroll
                                for (int g = 0; g < (DOWN ? 1 : 2); ++g) {
                                    v[h][a][g] = make_float4(0.f, 0.f, 0.f, 0.f);
                                    if (b <= c1 && token[a] >= 0)
                                        v[h][a][g] = __ldcg(reinterpret_cast<const float4 *>(
                                            parts + (static_cast<int64_t>(from) * NT + token[a]) * kPartRows + g * kTile + 4 * lane));
                                }
                        }
#pragma unroll
                        for (int h = 0; h < kAhead; ++h)
#pragma unroll
                            for (int a = 0; a < kAtATime; ++a)
#pragma unroll
                                for (int g = 0; g < (DOWN ? 1 : 2); ++g) {
                                    sum[a][g].x += v[h][a][g].x, sum[a][g].y += v[h][a][g].y;
                                    sum[a][g].z += v[h][a][g].z, sum[a][g].w += v[h][a][g].w;
                                }
                    }
#pragma unroll
                    for (int a = 0; a < kAtATime; ++a) {
                        if (token[a] < 0)
                            continue;
                        const float4 g = sum[a][0];
                        if constexpr (DOWN) {
                            const float v[4] = {g.x, g.y, g.z, g.w};
                            __nv_bfloat16 *out = reinterpret_cast<__nv_bfloat16 *>(p.out) + static_cast<int64_t>(token[a]) * p.H + i0;
#pragma unroll
                            for (int c = 0; c < 4; ++c)
                                if (i0 + c < p.H)
                                    out[c] = __float2bfloat16_rn(v[c]);
                        } else {
                            store_activation(unit, sh.first[place] + j0 + a * kEpilogueWarps, g, sum[a][1]);
                        }
                    }
                }
            }
        }
    } else if (FP8 && warp == 3) {
        // ------------------------------------------------------------ scales, ahead
        if constexpr (FP8) {
            if (DOWN)
                griddep_wait();
            bool ok = true;
            int sc = 0;
            uint32_t sc_phase = 0;
            const int groups = (DOWN ? p.I : p.H) / 128;
            while (ok && walk.next(seg)) {
                int place = DOWN ? seg.s0 / expert_steps : seg.unit / tiles;
                int k = DOWN ? seg.s0 % expert_steps : seg.s0;
                const int tile = DOWN ? seg.unit : seg.unit % tiles;
                for (int s = seg.s0; s < seg.s1; ++s) {
                    ok = __all_sync(0xffffffffu,
                                    mbar_wait(&sh.scales.empty[sc], sc_phase ^ 1, p.timeout_ns, abort_flag));
                    if (!ok)
                        break;
                    const int64_t e = sh.active[place];
                    if constexpr (DOWN) {
                        const int n = __popcll(sh.tokens(sh.active[place])), first = sh.first[place];
                        for (int b = 0; b < 2 && 2 * k + b < groups; ++b) {
                            for (int i = lane; i < n; i += 32)
                                copy_word(&sh.scales.token[sc][b][i], h_scales + static_cast<int64_t>(first + i) * groups + 2 * k + b);
                            if (lane == 0)
                                copy_word(&sh.scales.weight[sc][b], p.w2_scales + (e * (p.H / 128) + tile) * groups + 2 * k + b);
                        }
                    } else {
                        for (int t = lane; t < p.T; t += 32)
                            copy_word(&sh.scales.token[sc][0][t], p.x_scales + static_cast<int64_t>(t) * groups + k);
                        if (lane < 2)
                            copy_word(&sh.scales.weight[sc][lane], p.w1_scales + (e * (p.I / 64) + lane * (p.I / 128) + tile) * groups + k);
                    }
                    copy_arrive(&sh.scales.full[sc]);
                    advance(sc, sc_phase, kScaleStages);
                    if (++k == expert_steps)
                        k = 0, ++place;
                }
            }
            if (!ok && lane == 0)
                give_up(p, sh);
            asm volatile("cp.async.wait_all;" ::: "memory");
        }
    } else if (DOWN && warp == 2) {
        griddep_wait();
        griddep_launch_dependents();
        // no token has an expert here
        if (sh.n_active == 0) {
            const int64_t all = static_cast<int64_t>(p.T) * p.H;
            for (int64_t i = static_cast<int64_t>(blockIdx.x) * 32 + lane; i < all; i += static_cast<int64_t>(gridDim.x) * 32)
                reinterpret_cast<__nv_bfloat16 *>(p.out)[i] = __float2bfloat16_rn(0.f);
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == kThreads / 32 - 1)
        tmem_dealloc(tmem, kTmemCols);
}

template <bool FP8, int NT>
static cudaError_t launch_form(const FewMaps &maps, const FewParams &p, int num_sms, cudaStream_t s)
{
    const auto up = few_kernel<false, FP8, NT>, down = few_kernel<true, FP8, NT>;
    constexpr int up_smem = smem_bytes<false, FP8, NT>(), down_smem = smem_bytes<true, FP8, NT>();
    static_assert(up_smem <= 227 * 1024 && down_smem <= 227 * 1024, "shared memory of a block");
    cudaError_t e = cudaFuncSetAttribute(up, cudaFuncAttributeMaxDynamicSharedMemorySize, up_smem);
    if (e == cudaSuccess)
        e = cudaFuncSetAttribute(down, cudaFuncAttributeMaxDynamicSharedMemorySize, down_smem);
    if (e != cudaSuccess)
        return e;
    const int grid = num_sms < kMaxBlocks ? num_sms : kMaxBlocks;
    uint8_t *h_rows = p.workspace + few_workspace_rows(p.T);
    float *h_scales = reinterpret_cast<float *>(p.workspace + few_workspace_scales(p));
    e = launch_behind(up, grid, kThreads, up_smem, s, maps.w1, maps.x, p, h_rows, h_scales);
    return e != cudaSuccess ? e
                            : launch_behind(down, grid, kThreads, down_smem, s, maps.w2, maps.h, p, h_rows, h_scales);
}

cudaError_t launch_layer_few(const FewMaps &maps, const FewParams &p, int num_sms, cudaStream_t s)
{
    switch (few_columns(p.T)) {
    case 16:
        return p.fp8 ? launch_form<true, 16>(maps, p, num_sms, s) : launch_form<false, 16>(maps, p, num_sms, s);
    case 32:
        return p.fp8 ? launch_form<true, 32>(maps, p, num_sms, s) : launch_form<false, 32>(maps, p, num_sms, s);
    default:
        return p.fp8 ? launch_form<true, 64>(maps, p, num_sms, s) : launch_form<false, 64>(maps, p, num_sms, s);
    }
}

}  // namespace ep
