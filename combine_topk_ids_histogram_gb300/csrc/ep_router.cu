// ep_router.cu -- the router in front of the dispatch: each token's K experts and their
// probabilities from its logits, and the gradient of the logits from the gradient of the
// probabilities (what ep_combine_bwd returns).
//
// One warp per token; every lane holds E/32 of the row's selection scores as order-preserving
// integer keys.
#include "ep_host.h"
#include "ep_types.cuh"

namespace ep {
namespace {

constexpr int kRouterThreads = 256;
constexpr int kRouterWarps = kRouterThreads / 32;

// Keys compare as unsigned integers the way the scores compare as numbers; +0 and -0 are equal,
// a NaN is above everything, and 0 stands for "not selectable" (-inf, or taken already).
__device__ __forceinline__ unsigned score_key(float s) {
    if (s != s) return 0xffffffffu;
    const unsigned u = __float_as_uint(s + 0.0f);
    const unsigned k = (u & 0x80000000u) ? ~u : u | 0x80000000u;
    return k == 0x007fffffu ? 0u : k;   // the key of -inf
}

struct RouterScore {
    int sigmoid, renorm;
    float scale;
};

// Probabilities of the selected logits, lane k holding slot k (used: the slot has an expert).
// `row` gives the logits of all experts to a softmax over all of them.  Renormalised scores are
// divided through by the largest of them first, exp(min(max l, 0)) for sigmoids, so that rows
// of very negative logits keep their ratios.
template <typename T, int NVAL>
__device__ __forceinline__ float slot_prob(float l, bool used, const T *row, int E, int lane, RouterScore sc) {
    const float neg_inf = __int_as_float(0xff800000);
    if (sc.sigmoid) {
        if (!sc.renorm) return used ? sc.scale / (1.0f + expf(-l)) : 0.0f;
        const float m = fminf(warp_max(used ? l : neg_inf), 0.0f);
        const float s = !used ? 0.0f : l >= 0.0f ? 1.0f / (1.0f + expf(-l)) : expf(l - m) / (1.0f + expf(l));
        const float total = warp_sum(s);
        return used ? sc.scale * (s / total) : 0.0f;
    }
    if (sc.renorm) {
        const float m = warp_max(used ? l : neg_inf);
        const float e = used ? expf(l - m) : 0.0f;
        const float total = warp_sum(e);
        return used ? sc.scale * (e / total) : 0.0f;
    }
    float m = neg_inf;
#pragma unroll
    for (int i = 0; i < NVAL; ++i) {
        const int e = i * 32 + lane;
        if (e < E) m = fmaxf(m, to_f32(row[e]));
    }
    m = warp_max(m);
    if (m == neg_inf) return 0.0f;
    float total = 0.0f;
#pragma unroll
    for (int i = 0; i < NVAL; ++i) {
        const int e = i * 32 + lane;
        if (e < E) total += expf(to_f32(row[e]) - m);
    }
    total = warp_sum(total);
    return used ? sc.scale * (expf(l - m) / total) : 0.0f;
}

template <typename T, int NVAL>
__global__ void __launch_bounds__(kRouterThreads)
ep_router_topk_kernel(const T *__restrict__ logits, long long ld, const float *__restrict__ bias, int tokens, int E,
                      int K, RouterScore sc, int one_wave, int32_t *__restrict__ ids, float *__restrict__ probs) {
    pdl_begin_if(one_wave);
    const int lane = threadIdx.x & 31;
    const int t = blockIdx.x * kRouterWarps + (threadIdx.x >> 5);
    if (t >= tokens) return;
    const T *row = logits + (size_t)t * ld;
    unsigned key[NVAL];
#pragma unroll
    for (int i = 0; i < NVAL; ++i) {
        const int e = i * 32 + lane;
        key[i] = 0u;
        if (e < E) {
            float s = to_f32(row[e]);
            if (bias) s += bias[e];
            key[i] = score_key(s);
        }
    }
    int my_id = -1;   // lane k: the expert of slot k
    for (int k = 0; k < K; ++k) {
        unsigned best = 0u;
#pragma unroll
        for (int i = 0; i < NVAL; ++i) best = max(best, key[i]);
        const unsigned top = __reduce_max_sync(kFullMask, best);
        if (top == 0u) break;   // nothing selectable is left
        int e = E;
#pragma unroll
        for (int i = NVAL - 1; i >= 0; --i)
            if (key[i] == top) e = i * 32 + lane;
        const int first = __reduce_min_sync(kFullMask, e);   // ties to the lower id
#pragma unroll
        for (int i = 0; i < NVAL; ++i)
            if (first == i * 32 + lane) key[i] = 0u;
        if (lane == k) my_id = first;
    }
    const bool used = my_id >= 0;
    const float l = used ? to_f32(row[my_id]) : 0.0f;
    const float p = slot_prob<T, NVAL>(l, used, row, E, lane, sc);
    if (lane < K) {
        ids[(size_t)t * K + lane] = my_id;
        probs[(size_t)t * K + lane] = p;
    }
}

// d logits of one token.  With p the slots' probabilities and G = sum over slots of g*p / scale:
//   softmax over the selected:   dl[id_k] = p_k (g_k - G)
//   sigmoid over the selected:   the same, times 1 - sigmoid(l)
//   sigmoid:                     dl[id_k] = g_k p_k (1 - sigmoid(l))
//   softmax over all:            dl[e] = -P_e * scale * G, and + g_k p_k at e = id_k
// Slots that name the same expert add up in slot order.
template <typename T, int NVAL>
__global__ void __launch_bounds__(kRouterThreads)
ep_router_topk_bwd_kernel(const float *__restrict__ grad_p, const T *__restrict__ logits, long long ld,
                          const int32_t *__restrict__ ids, int tokens, int E, int K, RouterScore sc, int one_wave,
                          T *__restrict__ grad) {
    pdl_begin_if(one_wave);
    const int lane = threadIdx.x & 31;
    const int t = blockIdx.x * kRouterWarps + (threadIdx.x >> 5);
    if (t >= tokens) return;
    const T *row = logits + (size_t)t * ld;
    T *out = grad + (size_t)t * E;
    int id = -1;
    float g = 0.0f;
    if (lane < K) {
        id = ids[(size_t)t * K + lane];
        g = grad_p[(size_t)t * K + lane];
    }
    const bool used = id >= 0 && id < E;
    if (!used) g = 0.0f;
    const float l = used ? to_f32(row[id]) : 0.0f;
    const float p = slot_prob<T, NVAL>(l, used, row, E, lane, sc);
    const float G = warp_sum(g * p) / sc.scale;
    float d;
    if (sc.sigmoid) d = p * (sc.renorm ? g - G : g) / (1.0f + expf(l));
    else d = sc.renorm ? p * (g - G) : p * g;
    if (!used) d = 0.0f;
    float sum = 0.0f;
    for (int k = 0; k < K; ++k) {
        const int ik = __shfl_sync(kFullMask, id, k);
        const float dk = __shfl_sync(kFullMask, d, k);
        if (ik == id) sum += dk;
    }
    if (!sc.sigmoid && !sc.renorm) {
        const float neg_inf = __int_as_float(0xff800000);
        float m = neg_inf, total = 0.0f;
        float v[NVAL];
#pragma unroll
        for (int i = 0; i < NVAL; ++i) {
            const int e = i * 32 + lane;
            v[i] = e < E ? to_f32(row[e]) : neg_inf;
            m = fmaxf(m, v[i]);
        }
        m = warp_max(m);
        if (m == neg_inf) m = 0.0f;
#pragma unroll
        for (int i = 0; i < NVAL; ++i) total += v[i] = expf(v[i] - m);
        total = warp_sum(total);
        const float f = total > 0.0f ? -sc.scale * G / total : 0.0f;
#pragma unroll
        for (int i = 0; i < NVAL; ++i) {
            const int e = i * 32 + lane;
            if (e < E) out[e] = from_f32<T>(f * v[i]);
        }
        sum += f * expf(l - m);
    } else {
        for (int e = lane; e < E; e += 32) out[e] = from_f32<T>(0.0f);
    }
    __syncwarp();   // the row is written before its selected entries are
    if (used) out[id] = from_f32<T>(sum);
}

bool router_args_ok(int T, int E, int K, int dtype, long long ld, int score, int renorm, float scale) {
    if (!sizes_ok(T, K, E, 0) || K > E) return false;
    if (dtype < EP_BF16 || dtype > EP_F32 || ld < E) return false;
    if ((score != EP_SCORE_SOFTMAX && score != EP_SCORE_SIGMOID) || (renorm != 0 && renorm != 1)) return false;
    return scale > 0.0f && scale <= FLT_MAX;
}

bool element_aligned(const void *p, int dtype) {
    return (reinterpret_cast<uintptr_t>(p) & (dtype == EP_F32 ? 3u : 1u)) == 0;
}

template <typename F>
int by_width(int E, F f) {
    if (E <= 32) return f(std::integral_constant<int, 1>());
    if (E <= 64) return f(std::integral_constant<int, 2>());
    if (E <= 128) return f(std::integral_constant<int, 4>());
    if (E <= 256) return f(std::integral_constant<int, 8>());
    if (E <= 512) return f(std::integral_constant<int, 16>());
    return f(std::integral_constant<int, 32>());
}

template <typename F>
int by_type(int dtype, F f) {
    if (dtype == EP_BF16) return f((const __nv_bfloat16 *)nullptr);
    if (dtype == EP_F16) return f((const __half *)nullptr);
    return f((const float *)nullptr);
}

}  // namespace
}  // namespace ep

using namespace ep;

extern "C" int ep_router_topk(const void *logits, long long stride, int dtype, const float *bias, int T,
                              int n_experts, int K, int score, int renormalize, float scale, int32_t *topk_ids,
                              float *topk_probs, void *stream) {
    EP_NVTX_RANGE("ep_router_topk");
    if (!router_args_ok(T, n_experts, K, dtype, stride, score, renormalize, scale)) return EP_ERR_INVALID_ARG;
    if (!element_aligned(logits, dtype) || !element_aligned(bias, EP_F32) || !aligned16(topk_ids) ||
        !aligned16(topk_probs))
        return EP_ERR_INVALID_ARG;
    if (T == 0) return EP_OK;
    if (!logits || !topk_ids || !topk_probs) return EP_ERR_INVALID_ARG;
    const RouterScore sc{score == EP_SCORE_SIGMOID, renormalize, scale};
    const int grid = (T + kRouterWarps - 1) / kRouterWarps;
    return by_type(dtype, [&](auto *tp) {
        using P = decltype(tp);
        return by_width(n_experts, [&](auto nval) {
            using E = std::remove_const_t<std::remove_pointer_t<P>>;
            return launch_pdl(ep_router_topk_kernel<E, decltype(nval)::value>, dim3(grid), dim3(kRouterThreads), 0,
                              as_stream(stream), (P)logits, stride, bias, T, n_experts, K, sc, one_wave(grid),
                              topk_ids, topk_probs);
        });
    });
}

extern "C" int ep_router_topk_bwd(const float *grad_probs, const void *logits, long long stride, int dtype,
                                  const int32_t *topk_ids, int T, int n_experts, int K, int score, int renormalize,
                                  float scale, void *grad_logits, void *stream) {
    EP_NVTX_RANGE("ep_router_topk_bwd");
    if (!router_args_ok(T, n_experts, K, dtype, stride, score, renormalize, scale)) return EP_ERR_INVALID_ARG;
    if (!element_aligned(logits, dtype) || !aligned16(grad_logits) || !aligned16(topk_ids) || !aligned16(grad_probs))
        return EP_ERR_INVALID_ARG;
    if (T == 0) return EP_OK;
    if (!grad_probs || !logits || !topk_ids || !grad_logits) return EP_ERR_INVALID_ARG;
    const RouterScore sc{score == EP_SCORE_SIGMOID, renormalize, scale};
    const int grid = (T + kRouterWarps - 1) / kRouterWarps;
    return by_type(dtype, [&](auto *tp) {
        using P = decltype(tp);
        return by_width(n_experts, [&](auto nval) {
            using E = std::remove_const_t<std::remove_pointer_t<P>>;
            return launch_pdl(ep_router_topk_bwd_kernel<E, decltype(nval)::value>, dim3(grid), dim3(kRouterThreads), 0,
                              as_stream(stream), grad_probs, (P)logits, stride, topk_ids, T, n_experts, K, sc,
                              one_wave(grid), (E *)grad_logits);
        });
    });
}
