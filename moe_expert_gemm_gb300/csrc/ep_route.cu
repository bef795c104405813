// The router's decision (ep_route) and the gradient of its gates (ep_route_backward).
//
// Scores s_i of a token's E logits l_i: the softmax, or s_i = 1 / (1 + e^-l_i). The
// experts are chosen by v_i = s_i + bias_i, or by l_i itself without a bias (s grows
// with l), inside the best groups; gates are the chosen experts' scores, optionally over
// their sum. With c = sum_j dg_j a_j over the chosen, a_j = s_j / sum, the gradient is
//   renormalised: softmax dl_j = a_j (dg_j - c)   (what falls on other experts cancels),
//                 sigmoid dl_j = a_j (1 - s_j) (dg_j - c);
//   plain:        softmax dl_i = s_i ([i chosen] dg_i - sum_j dg_j s_j),
//                 sigmoid dl_j = s_j (1 - s_j) dg_j;
// each times `scale`.
//
// The bytes are one pass over the logits; what has to be kept down is the instructions
// for a token. Forms, by the number of experts:
//  * route_thread_kernel, E <= 16: a thread takes a token, its experts in registers.
//  * route_warp_kernel, E <= 256 (groups: a power of two): a warp takes a token, 8 values
//    a lane. A choice value that needs an exponential and a division is first taken
//    approximately; the k-th largest of the lanes' maxima bounds the k-th choice from
//    below, which leaves hardly more than k candidates. Those go to one lane each, get
//    their exact fp32 value there, and are ranked by counting. Where the approximation
//    cannot decide (groups closer than its error, NaN, too few unmasked experts, more than
//    32 candidates) the token is done over by route_token. So is every token where fewer than
//    top_k lanes hold experts of the kept groups: topk_groups * 32 / n_groups lanes, fewer
//    if groups are small or their pieces leave lanes empty. 65536 tokens of 256 experts by
//    sigmoid and bias, top 8, us: 8 groups keep 4 / 2 / 1: 45 / 59 / 187, 16 keep 3: 152,
//    32 keep 4: 139 (252 experts in 9 groups, by the form below alone: 169).
//  * route_token_kernel: everything else, by scanning shared memory.
// The gradient likewise: a warp to a token with its values in registers up to 256 experts,
// past that in shared memory.
// Measured, us for 65536 tokens: 8 or 16 experts, bf16, 7 a thread to a token (the host's
// time of a call), 21 a warp to a token; 32 / 256 experts 24 / 30 a warp to a token, 46 / 74
// by scanning; 256 experts in 8 groups by sigmoid and bias 46 and 155 (67 MB of logits take
// 10: 660 instructions a token bound it, of them a quarter the groups' two best, a third
// the candidates' exact values and order). Gradient, softmax of 64 / 256 experts: 13 / 25 in
// registers (256: 80 % of the copy rate), 29 / 46 in shared memory.
#include <cuda_bf16.h>

#include <cfloat>

#include "ep_internal.h"
#include "ep_ptx.cuh"

namespace ep {

constexpr int kRouteThreads = 128;
constexpr unsigned kFull = 0xffffffffu;

// Order of choice values as unsigned integers: 0 out of the running, 1 masked, above
// that the value's order (-0 and +0 alike).
__device__ __forceinline__ uint32_t choice_key(float v)
{
    const uint32_t b = __float_as_uint(v + 0.f);
    return b >> 31 ? ~b : b | 0x80000000u;
}
constexpr uint32_t kKeyOut = 0, kKeyMasked = 1;

__device__ __forceinline__ float key_value(uint32_t key)
{
    return __uint_as_float(key >> 31 ? key ^ 0x80000000u : ~key);
}

template <int W>
__device__ __forceinline__ void store_vec(float *p, const float *v)
{
    if constexpr (W == 4)
        *reinterpret_cast<float4 *>(p) = make_float4(v[0], v[1], v[2], v[3]);
    else if constexpr (W == 2)
        *reinterpret_cast<float2 *>(p) = make_float2(v[0], v[1]);
    else
        *p = v[0];
}

template <int W>
__device__ __forceinline__ void store_vec(__nv_bfloat16 *p, const float *v)
{
    if constexpr (W == 1) {
        *p = __float2bfloat16_rn(v[0]);
    } else {
        uint32_t w[W / 2];
#pragma unroll
        for (int i = 0; i < W / 2; ++i) {
            const __nv_bfloat162 b = __float22bfloat162_rn(make_float2(v[2 * i], v[2 * i + 1]));
            w[i] = *reinterpret_cast<const uint32_t *>(&b);
        }
        if constexpr (W == 8)
            *reinterpret_cast<uint4 *>(p) = make_uint4(w[0], w[1], w[2], w[3]);
        else if constexpr (W == 4)
            *reinterpret_cast<uint2 *>(p) = make_uint2(w[0], w[1]);
        else
            *reinterpret_cast<uint32_t *>(p) = w[0];
    }
}

// (Plain loads: a gradient may be written over its logits.)
template <typename T>
struct Logit;
template <>
struct Logit<float> {
    static constexpr float lowest = -FLT_MAX;
    static __device__ __forceinline__ float load(const float *p) { return *p; }
    static __device__ __forceinline__ void store(float *p, float v) { *p = v; }
};
template <>
struct Logit<__nv_bfloat16> {
    static constexpr float lowest = -3.3895313892515355e38f;  // -(2 - 2^-7) * 2^127
    static __device__ __forceinline__ float load(const __nv_bfloat16 *p)
    {
        return __uint_as_float(static_cast<uint32_t>(*reinterpret_cast<const unsigned short *>(p)) << 16);
    }
    static __device__ __forceinline__ void store(__nv_bfloat16 *p, float v)
    {
        *p = __float2bfloat16_rn(v);
    }
};

__device__ __forceinline__ float sigmoid_f32(float x)
{
    return 1.f / (1.f + expf(-x));
}

// Whether a logit makes all of its token's gates NaN, whichever experts are chosen.
__device__ __forceinline__ bool makes_nan(float x, bool sigmoid)
{
    return isnan(x) || (!sigmoid && x == INFINITY);
}

// Approximations (errors: choice_error). e^x by 2^(x log2 e).
__device__ __forceinline__ float fast_exp(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x * 1.44269504f));
    return y;
}

__device__ __forceinline__ float fast_sigmoid(float x)
{
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(1.f + fast_exp(-x)));
    return y;
}

__device__ __forceinline__ float warp_sum(float x)
{
#pragma unroll
    for (int o = 16; o; o >>= 1)
        x += __shfl_xor_sync(kFull, x, o);
    return x;
}

__device__ __forceinline__ float warp_max(float x)
{
#pragma unroll
    for (int o = 16; o; o >>= 1)
        x = fmaxf(x, __shfl_xor_sync(kFull, x, o));
    return x;
}

// One token by one warp, whatever its logits; `key` points to kTokenWords * E words: choice
// keys, scores, groups' worths.
constexpr int kTokenWords = 3;

template <typename T>
__device__ __noinline__ void route_token(const RouteParams &p, int64_t t, uint32_t *key)
{
    const int lane = threadIdx.x & 31;
    const int E = p.E, k = p.top_k;
    float *score = reinterpret_cast<float *>(key + E);
    const T *l = static_cast<const T *>(p.logits) + t * p.stride;
    __syncwarp();  // the caller's use of the memory is over

    float top = -INFINITY;
    bool nan = false;
    for (int i = lane; i < E; i += 32) {
        const float x = Logit<T>::load(l + i);
        nan |= makes_nan(x, p.score == EP_SCORE_SIGMOID);
        if (x > Logit<T>::lowest)  // neither masked nor NaN
            top = fmaxf(top, x);
    }
    nan = __any_sync(kFull, nan);
    top = warp_max(top);
    float total = 0.f;
    for (int i = lane; i < E; i += 32) {
        const float x = Logit<T>::load(l + i);
        float s = 0.f;
        if (x > Logit<T>::lowest)
            s = p.score == EP_SCORE_SIGMOID ? sigmoid_f32(x) : expf(x - top);
        score[i] = s;
        total += s;
    }
    total = warp_sum(total);
    for (int i = lane; i < E; i += 32) {
        const float x = Logit<T>::load(l + i);
        float v = x;
        if (p.bias)
            v = (p.score == EP_SCORE_SIGMOID ? score[i] : score[i] / total) + __ldg(p.bias + i);
        key[i] = x > Logit<T>::lowest ? choice_key(v) : kKeyMasked;
    }
    __syncwarp();

    if (p.topk_groups < p.n_groups) {
        const int per = E / p.n_groups;
        uint32_t *worth = key + 2 * E;
        for (int g = lane; g < p.n_groups; g += 32) {
            uint32_t best = kKeyMasked, second = kKeyMasked;
            float s_best = 0.f, s_second = 0.f;
            for (int i = g * per; i < (g + 1) * per; ++i) {
                if (key[i] > best) {
                    second = best, s_second = s_best;
                    best = key[i], s_best = score[i];
                } else if (key[i] > second) {
                    second = key[i], s_second = score[i];
                }
            }
            if (p.group_top == 2 && best != kKeyMasked) {
                if (p.bias) {
                    s_best = key_value(best);
                    s_second = second == kKeyMasked ? 0.f : key_value(second);
                }
                best = choice_key(s_best + s_second);
            }
            worth[g] = best;
        }
        __syncwarp();
        for (int g = lane; g < p.n_groups; g += 32) {
            const uint32_t w = worth[g];
            int better = 0;
            for (int h = 0; h < p.n_groups; ++h)
                better += worth[h] > w || (worth[h] == w && h < g);
            if (better >= p.topk_groups)
                for (int i = g * per; i < (g + 1) * per; ++i)
                    key[i] = kKeyOut;
        }
        __syncwarp();
    }

    int id = 0;  // lane j: the j-th chosen expert
    for (int j = 0; j < k; ++j) {
        uint32_t best = 0;
        int at = 0;
        for (int i = lane; i < E; i += 32)
            if (key[i] > best) {
                best = key[i];
                at = i;
            }
        const uint32_t top_key = __reduce_max_sync(kFull, best);
        const unsigned first = __reduce_min_sync(kFull, best == top_key ? at : E);
        if (lane == j)
            id = static_cast<int>(first);
        if (lane == first % 32)
            key[first] = kKeyOut;
        __syncwarp();
    }

    const float x = lane < k ? Logit<T>::load(l + id) : -INFINITY;
    const bool live = lane < k && x > Logit<T>::lowest;
    float a = 0.f;
    if (p.score == EP_SCORE_SOFTMAX && p.renormalize) {
        const float m = warp_max(live ? x : -INFINITY);
        a = live ? expf(x - m) : 0.f;
    } else if (live) {
        a = p.score == EP_SCORE_SIGMOID ? sigmoid_f32(x) : expf(x - top) / total;
    }
    if (p.renormalize) {
        const float sum = warp_sum(a);
        a = sum == 0.f ? 0.f : a / sum;
    }
    if (nan)
        a = NAN;
    if (lane < k) {
        p.topk_ids[t * k + lane] = id;
        if (p.gates)
            p.gates[t * k + lane] = a * p.scale;
    }
}

template <typename T>
__global__ void __launch_bounds__(kRouteThreads) route_token_kernel(const __grid_constant__ RouteParams p)
{
    griddep_wait();
    griddep_launch_dependents();
    extern __shared__ uint32_t smem[];
    const int warp = threadIdx.x >> 5;
    const int64_t t = static_cast<int64_t>(blockIdx.x) * (kRouteThreads / 32) + warp;
    if (t < p.T)
        route_token<T>(p, t, smem + static_cast<int64_t>(warp) * kTokenWords * p.E);
}

// A lane's experts in route_warp_kernel: group lane / lanes (of 32 / n_groups lanes each),
// members i * lanes + lane % lanes, or, W at a time, pieces of W consecutive members.
template <int VPL, int W>
struct LaneExperts {
    int first, per, lanes_log2, sub;

    __device__ __forceinline__ LaneExperts(const RouteParams &p, int lane)
    {
        per = p.per;
        lanes_log2 = p.lanes_log2;
        sub = lane & ((1 << lanes_log2) - 1);
        first = (lane >> lanes_log2) * per;
    }
    __device__ __forceinline__ int member(int i) const
    {
        return ((i / W) << lanes_log2) * W + sub * W + i % W;
    }
};

// W values at once (as many as their bytes allow), W * sizeof(T) aligned.
template <int W>
__device__ __forceinline__ void load_vec(const float *p, float *out)
{
    if constexpr (W == 4) {
        const float4 v = *reinterpret_cast<const float4 *>(p);
        out[0] = v.x, out[1] = v.y, out[2] = v.z, out[3] = v.w;
    } else if constexpr (W == 2) {
        const float2 v = *reinterpret_cast<const float2 *>(p);
        out[0] = v.x, out[1] = v.y;
    } else {
        out[0] = *p;
    }
}

template <int W>
__device__ __forceinline__ void load_vec(const __nv_bfloat16 *p, float *out)
{
    if constexpr (W == 1) {
        out[0] = Logit<__nv_bfloat16>::load(p);
    } else {
        uint32_t w[W / 2];
        if constexpr (W == 8) {
            const uint4 v = *reinterpret_cast<const uint4 *>(p);
            w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
        } else if constexpr (W == 4) {
            const uint2 v = *reinterpret_cast<const uint2 *>(p);
            w[0] = v.x, w[1] = v.y;
        } else {
            w[0] = *reinterpret_cast<const uint32_t *>(p);
        }
#pragma unroll
        for (int i = 0; i < W / 2; ++i) {
            out[2 * i] = __uint_as_float(w[i] << 16);
            out[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
        }
    }
}

// How far a choice value taken with the fast exponential and reciprocal may lie from the fp32
// formula's: e^-x is off by a few units in 2^-22 relative plus |x| 2^-23, which the
// sigmoid's slope turns into less than 2^-21 absolute; a softmax score is off by less; the
// addition of the bias rounds once on either side, to within 2^-23 of the value, so that half
// of the second term is left for a rounding of what is made of it. The largest (or second
// largest) of some values is off by no more than a value of its size.
__device__ __forceinline__ float choice_error(float v)
{
    return 0x1p-20f + 0x1p-22f * fabsf(v);
}

constexpr int kRouteWarps = 8;  // of a block of route_warp_kernel

// What the experts are chosen by: the logit, or sigmoid or softmax score plus bias.
enum Choice { kByLogit, kBySigmoid, kBySoftmax };

// VEC: a lane's members come in pieces of W, loaded at once.
template <typename T, int VPL, bool VEC, Choice BY>
__global__ void __launch_bounds__(32 * kRouteWarps) route_warp_kernel(const __grid_constant__ RouteParams p)
{
    griddep_wait();
    griddep_launch_dependents();
    constexpr int kMost = 16 / static_cast<int>(sizeof(T));
    constexpr int W = VEC ? (VPL < kMost ? VPL : kMost) : 1;
    constexpr int WB = VEC ? (VPL < 4 ? VPL : 4) : 1;  // of the bias
    extern __shared__ uint32_t smem[];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t t = static_cast<int64_t>(blockIdx.x) * kRouteWarps + warp;
    if (t >= p.T)
        return;
    uint32_t *own = smem + static_cast<int64_t>(warp) * p.warp_words;
    const int k = p.top_k;
    const bool sigmoid = p.score == EP_SCORE_SIGMOID;
    const LaneExperts<VPL, W> at(p, lane);
    const T *row = static_cast<const T *>(p.logits) + t * p.stride + at.first;
    float x[VPL], v[VPL];
#pragma unroll
    for (int i = 0; i < VPL; i += W) {
#pragma unroll
        for (int j = 0; j < W; ++j)
            x[i + j] = -INFINITY;
        if (at.member(i) < at.per)  // a piece is whole or missing
            load_vec<W>(row + at.member(i), x + i);
    }
    if constexpr (BY != kByLogit) {
        const float *b = p.bias + at.first;
#pragma unroll
        for (int i = 0; i < VPL; i += WB) {
#pragma unroll
            for (int j = 0; j < WB; ++j)
                v[i + j] = 0.f;
            if (at.member(i) < at.per)
                load_vec<WB>(b + at.member(i), v + i);
        }
    }
    bool odd = false, usual = true;
#pragma unroll
    for (int i = 0; i < VPL; ++i)
        usual &= x[i] > Logit<T>::lowest;
    usual = __all_sync(kFull, usual);  // no expert masked, missing or NaN
    if (!usual) {
#pragma unroll
        for (int i = 0; i < VPL; ++i) {
            odd |= isnan(x[i]);
            if (!(x[i] > Logit<T>::lowest))
                x[i] = -INFINITY;
        }
    }
    // of the whole row, for the scores of the softmax
    float top = 0.f, total = 1.f;
    if (BY == kBySoftmax || (BY == kByLogit && !sigmoid && (!p.renormalize || p.two_of_group))) {
        top = x[0];
#pragma unroll
        for (int i = 1; i < VPL; ++i)
            top = fmaxf(top, x[i]);
        top = warp_max(top);
        odd |= !(fabsf(top) < INFINITY);
        total = 0.f;
#pragma unroll
        for (int i = 0; i < VPL; ++i)
            total += expf(x[i] - top);
        total = warp_sum(total);
    }
    if constexpr (BY != kByLogit) {
        const float rtotal = 1.f / total;
#pragma unroll
        for (int i = 0; i < VPL; ++i)
            v[i] += BY == kBySigmoid ? fast_sigmoid(x[i]) : fast_exp(x[i] - top) * rtotal;
        if (!usual) {
#pragma unroll
            for (int i = 0; i < VPL; ++i)
                v[i] = x[i] == -INFINITY ? -INFINITY : v[i];
        }
    } else {
#pragma unroll
        for (int i = 0; i < VPL; ++i)
            v[i] = x[i];
    }

    if (p.topk_groups < p.n_groups) {
        // the two best of the group, over its lanes
        float a = -INFINITY, b = -INFINITY;
        if (BY == kByLogit && p.two_of_group) {
#pragma unroll
            for (int i = 0; i < VPL; ++i) {
                const float w = x[i] == -INFINITY ? -INFINITY
                                : sigmoid         ? fast_sigmoid(x[i])
                                                  : fast_exp(x[i] - top);
                b = fmaxf(b, fminf(a, w));
                a = fmaxf(a, w);
            }
        } else {
#pragma unroll
            for (int i = 0; i < VPL; ++i) {
                b = fmaxf(b, fminf(a, v[i]));
                a = fmaxf(a, v[i]);
            }
        }
        for (int o = 1; o < 1 << p.lanes_log2; o <<= 1) {
            const float a2 = __shfl_xor_sync(kFull, a, o), b2 = __shfl_xor_sync(kFull, b, o);
            b = fmaxf(fminf(a, a2), fmaxf(b, b2));
            a = fmaxf(a, a2);
        }
        const float worth = !p.two_of_group || b == -INFINITY ? a : a + b;
        bool keep;
        if (BY == kByLogit && !p.two_of_group) {  // the worth is a logit: exact, ties to the lower group
            const int mine = lane >> p.lanes_log2;
            int better = 0;
            for (int g = 0; g < p.n_groups; ++g) {
                const float w = __shfl_sync(kFull, worth, g << p.lanes_log2);
                better += w > worth || (w == worth && g < mine);
            }
            keep = better < p.topk_groups;
        } else {
            // The groups with the topk_groups largest worths. The members of a sum are each off
            // by their own size's error, which may be far above the sum's: where the least that a
            // kept worth may be does not pass the most that another may be (or worths are
            // equal), the fp32 formula has to tell.
            const uint32_t mine = choice_key(worth);
            uint32_t left = mine, last = 0;
            for (int g = 0; g < p.topk_groups; ++g) {
                last = __reduce_max_sync(kFull, left);
                left = left == last ? 0 : left;
            }
            keep = mine >= last;
            const bool any = a > -INFINITY;  // (else nothing of the group is left)
            const float off = !any ? 0.f
                              : choice_error(a) + 0x1p-23f * fabsf(worth) +
                                    (p.two_of_group && b > -INFINITY ? choice_error(b) : 0.f);
            const uint32_t least = __reduce_min_sync(kFull, keep ? choice_key(worth - off) : ~0u);
            const uint32_t most_other = __reduce_max_sync(kFull, keep ? 0 : choice_key(worth + off));
            const unsigned kept = __ballot_sync(kFull, keep);
            odd |= least <= most_other || least <= choice_key(-INFINITY) ||
                   __popc(kept) != p.topk_groups << p.lanes_log2;
        }
        if (!keep) {
#pragma unroll
            for (int i = 0; i < VPL; ++i)
                v[i] = -INFINITY;
        }
    }

    // the k-th largest of the lanes' maxima is at most the k-th largest of all
    float most = v[0];
#pragma unroll
    for (int i = 1; i < VPL; ++i)
        most = fmaxf(most, v[i]);
    uint32_t key = choice_key(most), kth = 0;
    for (int j = 0; j < k; ++j) {
        kth = __reduce_max_sync(kFull, key);
        key = key == kth ? 0 : key;
    }
    float bar = key_value(kth);
    odd |= kth <= choice_key(-INFINITY);
    if (BY != kByLogit)
        bar -= 2.f * choice_error(bar);
    uint32_t mine = 0;  // this lane's candidates
#pragma unroll
    for (int i = 0; i < VPL; ++i)
        mine |= v[i] >= bar ? 1u << i : 0u;
    int n = 0;  // candidates in all
    if (!__any_sync(kFull, odd)) {
        unsigned who;
        while ((who = __ballot_sync(kFull, mine != 0)) != 0 && n <= 32) {
            const int to = n + __popc(who & ((1u << lane) - 1));
            if (mine && to < 32)
                own[to] = at.first + at.member(__ffs(mine) - 1);
            mine &= mine - 1;
            n += __popc(who);
        }
    }
    if (n < k || n > 32) {
        route_token<T>(p, t, own);
        return;
    }
    __syncwarp();
    // a candidate a lane, with its value as the fp32 formula has it; in the order (value,
    // lower id first) as one number
    float cx = -INFINITY, s = 0.f;
    int id = p.E;
    uint64_t order = 0;
    if (lane < n) {
        id = own[lane];
        cx = Logit<T>::load(static_cast<const T *>(p.logits) + t * p.stride + id);
        float cv = cx;
        if (sigmoid)
            s = sigmoid_f32(cx);
        else if (BY == kBySoftmax || !p.renormalize)
            s = expf(cx - top) / total;
        if (BY != kByLogit)
            cv = s + __ldg(p.bias + id);
        order = static_cast<uint64_t>(choice_key(cv)) << 32 | ~static_cast<uint32_t>(id);
    }
    __syncwarp();
    uint64_t *orders = reinterpret_cast<uint64_t *>(own);
    orders[lane] = order;
    __syncwarp();
    int rank = 0;
    for (int c = 0; c < n; c += 4) {  // (past n they are 0)
        const ulonglong2 u = *reinterpret_cast<const ulonglong2 *>(orders + c);
        const ulonglong2 w = *reinterpret_cast<const ulonglong2 *>(orders + c + 2);
        rank += (u.x > order) + (u.y > order) + (w.x > order) + (w.y > order);
    }
    const bool chosen = lane < n && rank < k;
    if (!sigmoid && p.renormalize) {
        const float m = warp_max(chosen ? cx : -INFINITY);
        s = expf(cx - m);
    }
    s = chosen ? s : 0.f;
    if (p.renormalize) {
        const float sum = warp_sum(s);
        s = sum == 0.f ? 0.f : s / sum;
    }
    if (!chosen)
        return;
    p.topk_ids[t * k + rank] = id;
    if (p.gates)
        p.gates[t * k + rank] = s * p.scale;
}

// A thread a token, E <= EP.
template <typename T, int EP>
__global__ void __launch_bounds__(128) route_thread_kernel(const __grid_constant__ RouteParams p)
{
    griddep_wait();
    griddep_launch_dependents();
    const int64_t t = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x;
    if (t >= p.T)
        return;
    const int E = p.E, k = p.top_k;
    const bool sigmoid = p.score == EP_SCORE_SIGMOID;
    const T *l = static_cast<const T *>(p.logits) + t * p.stride;
    constexpr int W = 16 / sizeof(T) < EP ? 16 / sizeof(T) : EP;
    float x[EP];
    if (p.vec && E == EP) {
#pragma unroll
        for (int i = 0; i < EP; i += W)
            load_vec<W>(l + i, x + i);
    } else {
#pragma unroll
        for (int i = 0; i < EP; ++i)
            x[i] = i < E ? Logit<T>::load(l + i) : -INFINITY;
    }
    bool nan = false;
    float top = -INFINITY, total = 0.f;
#pragma unroll
    for (int i = 0; i < EP; ++i) {
        nan |= makes_nan(x[i], sigmoid);
        if (!(x[i] > Logit<T>::lowest))
            x[i] = -INFINITY;
        top = fmaxf(top, x[i]);
    }
    if (!sigmoid && (p.bias || !p.renormalize)) {
#pragma unroll
        for (int i = 0; i < EP; ++i)
            total += x[i] == -INFINITY ? 0.f : expf(x[i] - top);
    }
    auto score = [&](float y) {
        return y == -INFINITY ? 0.f : sigmoid ? sigmoid_f32(y) : expf(y - top) / total;
    };
    uint32_t key[EP];
#pragma unroll
    for (int i = 0; i < EP; ++i) {
        const float v = p.bias && i < E ? score(x[i]) + __ldg(p.bias + i) : x[i];
        key[i] = i >= E ? kKeyOut : x[i] == -INFINITY ? kKeyMasked : choice_key(v);
    }
    float sx[EP], m = -INFINITY;  // logits of the chosen
#pragma unroll
    for (int j = 0; j < EP; ++j) {
        if (j >= k)
            break;
        uint32_t best = kKeyOut;
        int id = 0;
        sx[j] = -INFINITY;
#pragma unroll
        for (int i = 0; i < EP; ++i)
            if (key[i] > best) {
                best = key[i];
                id = i;
                sx[j] = x[i];
            }
#pragma unroll
        for (int i = 0; i < EP; ++i)
            key[i] = i == id ? kKeyOut : key[i];
        m = fmaxf(m, sx[j]);
        p.topk_ids[t * k + j] = id;
    }
    if (!p.gates)
        return;
    float sum = 0.f;
#pragma unroll
    for (int j = 0; j < EP; ++j) {
        if (j >= k)
            break;
        sx[j] = !sigmoid && p.renormalize ? (sx[j] == -INFINITY ? 0.f : expf(sx[j] - m)) : score(sx[j]);
        sum += sx[j];
    }
#pragma unroll
    for (int j = 0; j < EP; ++j) {
        if (j >= k)
            break;
        float a = sx[j];
        if (p.renormalize)
            a = sum == 0.f ? 0.f : a / sum;
        p.gates[t * k + j] = nan ? NAN : a * p.scale;
    }
}

// The gradient of a token by a warp, VPL values a lane in pieces of W. The dense value
// (0, or -s_i c of the plain softmax) goes to every logit first, the chosen ones' over it:
// a warp's later stores follow its earlier ones.
template <typename T, int VPL, bool VEC>
__global__ void __launch_bounds__(32 * kRouteWarps)
    route_backward_warp_kernel(const __grid_constant__ RouteBackwardParams p)
{
    griddep_wait();
    griddep_launch_dependents();
    constexpr int kMost = 16 / static_cast<int>(sizeof(T));
    constexpr int W = VEC ? (VPL < kMost ? VPL : kMost) : 1;
    const int lane = threadIdx.x & 31;
    const int64_t t = static_cast<int64_t>(blockIdx.x) * kRouteWarps + (threadIdx.x >> 5);
    if (t >= p.T)
        return;
    const int E = p.E, k = p.top_k;
    const T *l = static_cast<const T *>(p.logits) + t * p.stride;
    T *out = static_cast<T *>(p.dlogits) + t * p.dstride;
    auto expert = [&](int i) { return (i / W) * 32 * W + lane * W + i % W; };
    const bool dense = p.score == EP_SCORE_SOFTMAX && !p.renormalize;
    float y[VPL];
    if (dense) {
#pragma unroll
        for (int i = 0; i < VPL; i += W) {
#pragma unroll
            for (int j = 0; j < W; ++j)
                y[i + j] = -INFINITY;
            if (expert(i) < E)
                load_vec<W>(l + expert(i), y + i);
        }
    }
    int id = lane < k ? __ldg(p.topk_ids + t * k + lane) : -1;
    float dg = lane < k ? __ldg(p.dgates + t * k + lane) : 0.f;
    if (lane < k && (id < 0 || id >= E)) {
        atomicOr(p.status, EP_STATUS_ROUTING);
        id = -1;
    }
    const float x = id >= 0 ? Logit<T>::load(l + id) : -INFINITY;
    const bool live = id >= 0 && !(x <= Logit<T>::lowest);
    if (!live)
        dg = 0.f;
    float dl;
    if (dense) {
        float top = -INFINITY, total = 0.f;
#pragma unroll
        for (int i = 0; i < VPL; ++i)
            top = fmaxf(top, y[i]);
        top = warp_max(top);
#pragma unroll
        for (int i = 0; i < VPL; ++i) {
            y[i] = y[i] <= Logit<T>::lowest ? 0.f : expf(y[i] - top);
            total += y[i];
        }
        total = warp_sum(total);
        const float rtotal = 1.f / total;
        const float s = live ? expf(x - top) * rtotal : 0.f;
        const float part = live ? dg * s : 0.f;
        const float c = warp_sum(part);
        dl = part - s * c;
        const float cr = c * rtotal * p.scale;
#pragma unroll
        for (int i = 0; i < VPL; ++i)
            y[i] = y[i] == 0.f ? 0.f : -y[i] * cr;
    } else {
        float a = 0.f, slope = 1.f;
        if (p.score == EP_SCORE_SOFTMAX) {
            const float m = warp_max(live ? x : -INFINITY);
            a = live ? expf(x - m) : 0.f;
        } else if (live) {
            a = sigmoid_f32(x);
            slope = sigmoid_f32(-x);
        }
        if (p.renormalize) {
            const float sum = warp_sum(a);
            a = sum == 0.f ? 0.f : a / sum;
            dg -= warp_sum(dg * a);
        }
        dl = a == 0.f ? 0.f : a * slope * dg;
#pragma unroll
        for (int i = 0; i < VPL; ++i)
            y[i] = 0.f;
    }
    __syncwarp();  // every lane has read its logits (they may be what is written)
#pragma unroll
    for (int i = 0; i < VPL; i += W)
        if (expert(i) < E)
            store_vec<W>(out + expert(i), y + i);
    __syncwarp();
    if (live)
        Logit<T>::store(out + id, dl * p.scale);
}

// Shared memory of a warp: the E gradients of its token.
template <typename T>
__global__ void __launch_bounds__(kRouteThreads) route_backward_kernel(const __grid_constant__ RouteBackwardParams p)
{
    griddep_wait();
    griddep_launch_dependents();
    extern __shared__ uint32_t smem[];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int E = p.E, k = p.top_k;
    float *d = reinterpret_cast<float *>(smem) + static_cast<int64_t>(warp) * E;
    const int64_t t = static_cast<int64_t>(blockIdx.x) * (kRouteThreads / 32) + warp;
    if (t >= p.T)
        return;
    const T *l = static_cast<const T *>(p.logits) + t * p.stride;
    int id = lane < k ? __ldg(p.topk_ids + t * k + lane) : -1;
    float dg = lane < k ? __ldg(p.dgates + t * k + lane) : 0.f;
    if (lane < k && (id < 0 || id >= E)) {
        atomicOr(p.status, EP_STATUS_ROUTING);
        id = -1;
    }
    const float x = id >= 0 ? Logit<T>::load(l + id) : -INFINITY;
    const bool live = id >= 0 && !(x <= Logit<T>::lowest);
    if (!live)
        dg = 0.f;
    const bool dense = p.score == EP_SCORE_SOFTMAX && !p.renormalize;
    float dl;
    if (dense) {
        float top = -INFINITY, total = 0.f;
        for (int i = lane; i < E; i += 32)
            top = fmaxf(top, Logit<T>::load(l + i));
        top = warp_max(top);
        auto e = [&](float y) { return y <= Logit<T>::lowest ? 0.f : expf(y - top); };
        for (int i = lane; i < E; i += 32)
            total += e(Logit<T>::load(l + i));
        total = warp_sum(total);
        dl = live ? dg * (e(x) / total) : 0.f;
        const float c = warp_sum(dl);
        for (int i = lane; i < E; i += 32) {
            const float y = Logit<T>::load(l + i);
            d[i] = y <= Logit<T>::lowest ? 0.f : -(e(y) / total) * c;
        }
    } else {
        float a = 0.f, slope = 1.f;
        if (p.score == EP_SCORE_SOFTMAX) {
            const float m = warp_max(live ? x : -INFINITY);
            a = live ? expf(x - m) : 0.f;
        } else if (live) {
            a = sigmoid_f32(x);
            slope = sigmoid_f32(-x);
        }
        if (p.renormalize) {
            const float sum = warp_sum(a);
            a = sum == 0.f ? 0.f : a / sum;
            dg -= warp_sum(dg * a);
        }
        dl = a == 0.f ? 0.f : a * slope * dg;
        for (int i = lane; i < E; i += 32)
            d[i] = 0.f;
    }
    for (int j = 0; j < k; ++j) {
        __syncwarp();
        if (lane == j && live)
            d[id] += dl;
    }
    __syncwarp();
    T *out = static_cast<T *>(p.dlogits) + t * p.dstride;
    for (int i = lane; i < E; i += 32)
        Logit<T>::store(out + i, d[i] * p.scale);
}

template <typename Kern, typename Params>
static cudaError_t launch_rows(Kern kern, const Params &p, int warps, int64_t warp_bytes,
                               cudaStream_t s)
{
    const int smem = static_cast<int>(warps * warp_bytes);
    if (smem > 48 * 1024) {
        const cudaError_t e =
            cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
        if (e != cudaSuccess)
            return e;
    }
    return launch_behind(kern, static_cast<unsigned>((static_cast<int64_t>(p.T) + warps - 1) / warps),
                         32 * warps, smem, s, p);
}

static bool aligned(const void *p, int64_t bytes)
{
    return reinterpret_cast<uintptr_t>(p) % static_cast<uintptr_t>(bytes) == 0;
}

// Values a lane takes of each: 1, 2, 4 or 8.
static int lane_values(int per_lane)
{
    return per_lane <= 1 ? 1 : per_lane <= 2 ? 2 : per_lane <= 4 ? 4 : 8;
}

template <typename T, int VPL>
static cudaError_t launch_route_vpl(const RouteParams &p, cudaStream_t s)
{
    const int64_t bytes = 4 * p.warp_words;
    if (!p.bias)
        return p.vec ? launch_rows(route_warp_kernel<T, VPL, true, kByLogit>, p, kRouteWarps, bytes, s)
                     : launch_rows(route_warp_kernel<T, VPL, false, kByLogit>, p, kRouteWarps, bytes, s);
    if (p.score == EP_SCORE_SIGMOID)
        return p.vec ? launch_rows(route_warp_kernel<T, VPL, true, kBySigmoid>, p, kRouteWarps, bytes, s)
                     : launch_rows(route_warp_kernel<T, VPL, false, kBySigmoid>, p, kRouteWarps, bytes, s);
    return p.vec ? launch_rows(route_warp_kernel<T, VPL, true, kBySoftmax>, p, kRouteWarps, bytes, s)
                 : launch_rows(route_warp_kernel<T, VPL, false, kBySoftmax>, p, kRouteWarps, bytes, s);
}

template <typename T>
static cudaError_t launch_route_type(RouteParams p, cudaStream_t s)
{
    constexpr int most = 16 / sizeof(T);
    const int groups = p.topk_groups < p.n_groups ? p.n_groups : 1;  // that matter
    p.n_groups = groups;
    if (groups == 1)
        p.topk_groups = 1;
    p.two_of_group = groups > 1 && p.group_top == 2;
    if (p.E <= 16 && groups == 1) {
        const int ep = p.E <= 8 ? 8 : 16;
        p.vec = aligned(p.logits, 16) && p.stride % most == 0;
        const unsigned blocks = static_cast<unsigned>((static_cast<int64_t>(p.T) + 127) / 128);
        return ep == 8 ? launch_behind(route_thread_kernel<T, 8>, blocks, 128, 0, s, p)
                       : launch_behind(route_thread_kernel<T, 16>, blocks, 128, 0, s, p);
    }
    int lanes_log2 = 5;
    while (lanes_log2 > 0 && 32 >> lanes_log2 < groups)
        --lanes_log2;
    p.per = p.E / groups;
    p.lanes_log2 = lanes_log2;
    const int per_lane = (p.per + (1 << lanes_log2) - 1) >> lanes_log2;
    if (32 >> lanes_log2 != groups || per_lane > 8)
        return launch_rows(route_token_kernel<T>, p, kRouteThreads / 32, 4ll * kTokenWords * p.E, s);
    // 32 candidates' orders, or a token done over; 16-byte pieces
    p.warp_words = ((kTokenWords * p.E > 64 ? kTokenWords * p.E : 64) + 3) / 4 * 4;
    const int vpl = lane_values(per_lane), w = vpl < most ? vpl : most, wb = vpl < 4 ? vpl : 4;
    p.vec = p.per % w == 0 && p.per % wb == 0 && p.stride % w == 0 &&
            aligned(p.logits, w * static_cast<int>(sizeof(T))) && aligned(p.bias, 4 * wb);
    switch (vpl) {
    case 1:
        return launch_route_vpl<T, 1>(p, s);
    case 2:
        return launch_route_vpl<T, 2>(p, s);
    case 4:
        return launch_route_vpl<T, 4>(p, s);
    default:
        return launch_route_vpl<T, 8>(p, s);
    }
}

cudaError_t launch_route(const RouteParams &p, int num_sms, cudaStream_t s)
{
    (void)num_sms;
    return p.bf16 ? launch_route_type<__nv_bfloat16>(p, s) : launch_route_type<float>(p, s);
}

template <typename T, int VPL>
static cudaError_t launch_backward_vpl(const RouteBackwardParams &p, cudaStream_t s)
{
    constexpr int most = 16 / sizeof(T), w = VPL < most ? VPL : most;
    const bool vec = p.E % w == 0 && p.stride % w == 0 && p.dstride % w == 0 &&
                     aligned(p.logits, w * sizeof(T)) && aligned(p.dlogits, w * sizeof(T));
    return vec ? launch_rows(route_backward_warp_kernel<T, VPL, true>, p, kRouteWarps, 0, s)
               : launch_rows(route_backward_warp_kernel<T, VPL, false>, p, kRouteWarps, 0, s);
}

template <typename T>
static cudaError_t launch_backward_type(const RouteBackwardParams &p, cudaStream_t s)
{
    if (p.E > 256)
        return launch_rows(route_backward_kernel<T>, p, kRouteThreads / 32, 4ll * p.E, s);
    switch (lane_values((p.E + 31) / 32)) {
    case 1:
        return launch_backward_vpl<T, 1>(p, s);
    case 2:
        return launch_backward_vpl<T, 2>(p, s);
    case 4:
        return launch_backward_vpl<T, 4>(p, s);
    default:
        return launch_backward_vpl<T, 8>(p, s);
    }
}

cudaError_t launch_route_backward(const RouteBackwardParams &p, int num_sms, cudaStream_t s)
{
    (void)num_sms;
    return p.bf16 ? launch_backward_type<__nv_bfloat16>(p, s) : launch_backward_type<float>(p, s);
}

}  // namespace ep
