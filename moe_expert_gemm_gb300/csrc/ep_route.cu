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
// each times `scale`. One warp takes one token.
#include <cuda_bf16.h>

#include <cfloat>

#include "ep_internal.h"

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

template <typename T>
struct Logit;
template <>
struct Logit<float> {
    static constexpr float lowest = -FLT_MAX;
    static __device__ __forceinline__ float load(const float *p) { return __ldg(p); }
    static __device__ __forceinline__ void store(float *p, float v) { *p = v; }
};
template <>
struct Logit<__nv_bfloat16> {
    static constexpr float lowest = -3.3895313892515355e38f;  // -(2 - 2^-7) * 2^127
    static __device__ __forceinline__ float load(const __nv_bfloat16 *p)
    {
        return __uint_as_float(
            static_cast<uint32_t>(__ldg(reinterpret_cast<const unsigned short *>(p))) << 16);
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

// Shared memory of a warp: E choice keys and E scores.
template <typename T>
__global__ void __launch_bounds__(kRouteThreads) route_kernel(const RouteParams p)
{
    extern __shared__ uint32_t smem[];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int E = p.E, k = p.top_k;
    uint32_t *key = smem + static_cast<int64_t>(warp) * 2 * E;
    float *score = reinterpret_cast<float *>(key + E);
    const int64_t t = static_cast<int64_t>(blockIdx.x) * (kRouteThreads / 32) + warp;
    if (t >= p.T)
        return;
    const T *l = static_cast<const T *>(p.logits) + t * p.stride;

    float top = -INFINITY;
    bool nan = false;
    for (int i = lane; i < E; i += 32) {
        const float x = Logit<T>::load(l + i);
        nan |= isnan(x);
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
        // every lane ranks its groups against all others
        const int per = E / p.n_groups;
        auto worth = [&](int g) -> uint32_t {
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
            if (p.group_top == 1 || best == kKeyMasked)
                return best;
            if (p.bias) {
                const uint32_t a = best >> 31 ? best ^ 0x80000000u : ~best;
                const uint32_t b = second >> 31 ? second ^ 0x80000000u : ~second;
                s_best = __uint_as_float(a);
                s_second = second == kKeyMasked ? 0.f : __uint_as_float(b);
            }
            return choice_key(s_best + s_second);
        };
        uint64_t out = 0;  // this lane's groups that are not among the best
        for (int g = lane, n = 0; g < p.n_groups; g += 32, ++n) {
            const uint32_t w = worth(g);
            int better = 0;
            for (int h = 0; h < p.n_groups; ++h) {
                const uint32_t o = worth(h);
                better += o > w || (o == w && h < g);
            }
            if (better >= p.topk_groups)
                out |= 1ull << n;
        }
        __syncwarp();
        for (int g = lane, n = 0; g < p.n_groups; g += 32, ++n)
            if (out >> n & 1)
                for (int i = g * per; i < (g + 1) * per; ++i)
                    key[i] = kKeyOut;
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

// Shared memory of a warp: the E gradients of its token.
template <typename T>
__global__ void __launch_bounds__(kRouteThreads) route_backward_kernel(const RouteBackwardParams p)
{
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
static cudaError_t launch_rows(Kern kern, const Params &p, int64_t warp_bytes, cudaStream_t s)
{
    const int warps = kRouteThreads / 32;
    const int smem = static_cast<int>(warps * warp_bytes);
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess)
        return e;
    kern<<<static_cast<unsigned>((p.T + warps - 1) / warps), kRouteThreads, smem, s>>>(p);
    return cudaGetLastError();
}

cudaError_t launch_route(const RouteParams &p, int num_sms, cudaStream_t s)
{
    (void)num_sms;
    return p.bf16 ? launch_rows(route_kernel<__nv_bfloat16>, p, 8ll * p.E, s)
                  : launch_rows(route_kernel<float>, p, 8ll * p.E, s);
}

cudaError_t launch_route_backward(const RouteBackwardParams &p, int num_sms, cudaStream_t s)
{
    (void)num_sms;
    return p.bf16 ? launch_rows(route_backward_kernel<__nv_bfloat16>, p, 4ll * p.E, s)
                  : launch_rows(route_backward_kernel<float>, p, 4ll * p.E, s);
}

}  // namespace ep
