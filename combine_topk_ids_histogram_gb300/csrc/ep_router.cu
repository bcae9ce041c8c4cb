// ep_router.cu -- the router in front of the dispatch: each token's K experts and their
// probabilities from its logits, and the gradient of the logits from the gradient of the
// probabilities (what ep_combine_bwd returns).
//
// One warp per token.  Lane l holds the scores of experts V * l to V * l + V - 1 as order-preserving integer keys.  The K-th largest
// of the lanes' largest keys bounds the K-th largest key from below; the few keys at or above it (about K + 2 for
// independent scores) are gathered and ranked against one another.  Against K rounds of finding and
// striking out the largest of all keys this takes half of the instructions, whose issue bounds the call: 32768 tokens of 256
// fp32 sigmoid scores with a bias, top-8, take 15.2 us (32.6 with rounds) at 425 instructions per token, issue slots 74 % busy;
// 16 tokens of 128 take 2.1 us.
#include "ep_host.h"
#include "ep_types.cuh"

namespace ep {
namespace {

constexpr int kRouterThreads = 256;
constexpr int kRouterWarps = kRouterThreads / 32;

// Keys compare as unsigned integers the way the scores compare as numbers: adding +0 makes one zero of the two and one
// NaN of all, whose key is above every other.
__device__ __forceinline__ unsigned score_key(float s) {
    const unsigned u = __float_as_uint(s + 0.0f);
    return u ^ ((unsigned)((int)u >> 31) | 0x80000000u);
}
constexpr unsigned kNoKey = 0x007fffffu;   // the key of -inf: not selectable, like every smaller one

// V consecutive elements of a row from e0 on, `fill` past its end.  vec: rows lie on boundaries of 16 bytes.
template <typename T, int V>
__device__ __forceinline__ void load_row(const T *row, int e0, int E, bool vec, float fill, float (&f)[V]) {
    constexpr int VL = V * sizeof(T) > 16 ? 16 / sizeof(T) : V;
#pragma unroll
    for (int j = 0; j < V; j += VL) {
        if (vec && e0 + j + VL <= E) {
            float g[VL];
            ld_pack<T, VL>(row + e0 + j).unpack(g);
#pragma unroll
            for (int i = 0; i < VL; ++i) f[j + i] = g[i];
        } else {
#pragma unroll
            for (int i = 0; i < VL; ++i) f[j + i] = e0 + j + i < E ? to_f32(row[e0 + j + i]) : fill;
        }
    }
}

struct RouterScore {
    int sigmoid, renorm;
    float scale;
};

// Probabilities of the selected logits, lane k holding slot k (used: the slot has an expert).  `row` gives the logits of all experts to a softmax over all of them.  Renormalised scores are
// divided through by the largest of them first, exp(min(max l, 0)) for sigmoids, so that rows
// of very negative logits keep their ratios.
template <typename T, int V>
__device__ __forceinline__ float slot_prob(float l, bool used, const T *row, int E, bool vec, int lane, RouterScore sc) {
    const float neg_inf = __int_as_float(0xff800000);
    if (sc.sigmoid) {
        if (!sc.renorm) return used ? sc.scale / (1.0f + expf(-l)) : 0.0f;
        const float m = fminf(warp_max(used ? l : neg_inf), 0.0f);
        // exp(l - m) / (1 + exp(l)) below 0 and 1 / (1 + exp(-l)) from there on (then m = 0)
        const float e = expf(-fabsf(l)), top = l >= 0.0f ? 1.0f : m == 0.0f ? e : expf(l - m);
        const float s = used ? top / (1.0f + e) : 0.0f;
        const float total = warp_sum(s);
        return used ? sc.scale * (s / total) : 0.0f;
    }
    if (sc.renorm) {
        const float m = warp_max(used ? l : neg_inf);
        const float e = used ? expf(l - m) : 0.0f;
        const float total = warp_sum(e);
        return used ? sc.scale * (e / total) : 0.0f;
    }
    float v[V];
    load_row<T, V>(row, lane * V, E, vec, neg_inf, v);
    float m = neg_inf;
#pragma unroll
    for (int i = 0; i < V; ++i) m = fmaxf(m, v[i]);
    m = warp_max(m);
    if (m == neg_inf) m = 0.0f;                                     // all masked, or NaN (which the maximum passes over)
    float total = 0.0f;
#pragma unroll
    for (int i = 0; i < V; ++i) total += expf(v[i] - m);
    total = warp_sum(total);
    return used ? sc.scale * (expf(l - m) / total) : 0.0f;
}

template <typename T, int V>
__global__ void __launch_bounds__(kRouterThreads)
ep_router_topk_kernel(const T *__restrict__ logits, long long ld, const float *__restrict__ bias, int tokens, int E,
                      int K, RouterScore sc, int vec, int one_wave, int32_t *__restrict__ ids,
                      float *__restrict__ probs) {
    __shared__ __align__(16) unsigned long long s_cand[kRouterWarps][32];
    __shared__ int s_slot[kRouterWarps][32];
    pdl_begin_if(one_wave);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int t = blockIdx.x * kRouterWarps + warp;
    if (t >= tokens) return;
    const T *row = logits + (size_t)t * ld;
    const float neg_inf = __int_as_float(0xff800000);
    const int e0 = lane * V;
    float f[V];
    load_row<T, V>(row, e0, E, vec & 1, neg_inf, f);
    if (bias) {
        float b[V];
        load_row<float, V>(bias, e0, E, vec & 2, 0.0f, b);
#pragma unroll
        for (int i = 0; i < V; ++i) f[i] += b[i];
    }
    unsigned key[V];
#pragma unroll
    for (int i = 0; i < V; ++i) key[i] = score_key(f[i]);
    unsigned best = 0u, top = 0u;
#pragma unroll
    for (int i = 0; i < V; ++i) best = max(best, key[i]);
    // a lower bound of the K-th largest key; lanes with equal maxima are struck out together, which only lowers it
#pragma unroll 4
    for (int k = 0; k < K; ++k) {
        top = __reduce_max_sync(kFullMask, best);
        if (best == top) best = 0u;
    }
    const unsigned bound = max(top, kNoKey + 1);
    unsigned mask = 0u;                                             // this lane's candidates
#pragma unroll
    for (int i = 0; i < V; ++i) mask |= key[i] >= bound ? 1u << i : 0u;
    int at = __popc(mask);
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(kFullMask, at, o);
        if (lane >= o) at += v;
    }
    const int n = __shfl_sync(kFullMask, at, 31);
    int my_id = -1;                                                 // lane k: the expert of slot k
    if (n <= 32) {
        // the larger key, then the lower id, is the larger 64-bit number
        s_cand[warp][lane] = 0ull;
        __syncwarp();
        unsigned long long *to = &s_cand[warp][at - __popc(mask)];
#pragma unroll
        for (int i = 0; i < V; ++i)
            if (mask >> i & 1u) *to++ = (unsigned long long)key[i] << 32 | (unsigned)~(e0 + i);
        __syncwarp();
        const unsigned long long own = s_cand[warp][lane];
        int rank = 0;
        for (int j = 0; j < n; j += 2) {                            // past the last candidate is 0
            const ulonglong2 o = *reinterpret_cast<const ulonglong2 *>(&s_cand[warp][j]);
            rank += (o.x > own) + (o.y > own);
        }
        if (lane < n && rank < K) s_slot[warp][rank] = ~(int)(unsigned)own;
        __syncwarp();
        if (lane < min(n, K)) my_id = s_slot[warp][lane];
    } else {                                                        // many equal keys: K rounds of the largest key
        for (int k = 0; k < K; ++k) {
            unsigned m = 0u;
#pragma unroll
            for (int i = 0; i < V; ++i) m = max(m, key[i]);
            const unsigned largest = __reduce_max_sync(kFullMask, m);
            if (largest <= kNoKey) break;
            int e = E;
#pragma unroll
            for (int i = V - 1; i >= 0; --i)
                if (key[i] == largest) e = e0 + i;
            const int first = __reduce_min_sync(kFullMask, e);
#pragma unroll
            for (int i = 0; i < V; ++i)
                if (first == e0 + i) key[i] = 0u;
            if (lane == k) my_id = first;
        }
    }
    const bool used = my_id >= 0;
    const float l = used ? to_f32(row[my_id]) : 0.0f;
    const float p = slot_prob<T, V>(l, used, row, E, vec & 1, lane, sc);
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
template <typename T, int V>
__global__ void __launch_bounds__(kRouterThreads)
ep_router_topk_bwd_kernel(const float *__restrict__ grad_p, const T *__restrict__ logits, long long ld,
                          const int32_t *__restrict__ ids, int tokens, int E, int K, RouterScore sc, int vec,
                          int vec_out, int one_wave, T *__restrict__ grad) {
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
    const float p = slot_prob<T, V>(l, used, row, E, vec, lane, sc);
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
    float v[V];
#pragma unroll
    for (int i = 0; i < V; ++i) v[i] = 0.0f;
    if (!sc.sigmoid && !sc.renorm) {
        const float neg_inf = __int_as_float(0xff800000);
        load_row<T, V>(row, lane * V, E, vec, neg_inf, v);
        float m = neg_inf, total = 0.0f;
#pragma unroll
        for (int i = 0; i < V; ++i) m = fmaxf(m, v[i]);
        m = warp_max(m);
        if (m == neg_inf) m = 0.0f;
#pragma unroll
        for (int i = 0; i < V; ++i) total += v[i] = expf(v[i] - m);
        total = warp_sum(total);
        const float f = total > 0.0f ? -sc.scale * G / total : 0.0f;
#pragma unroll
        for (int i = 0; i < V; ++i) v[i] *= f;
        sum += f * expf(l - m);
    }
    constexpr int VL = V * sizeof(T) > 16 ? 16 / sizeof(T) : V;
#pragma unroll
    for (int j = 0; j < V; j += VL) {
        const int e = lane * V + j;
        if (vec_out && e + VL <= E) {
            float g[VL];
#pragma unroll
            for (int i = 0; i < VL; ++i) g[i] = v[j + i];
            Pack<T, VL> o;
            o.pack(g);
            *reinterpret_cast<Pack<T, VL> *>(out + e) = o;
        } else {
#pragma unroll
            for (int i = 0; i < VL; ++i)
                if (e + i < E) out[e + i] = from_f32<T>(v[j + i]);
        }
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

// Whether rows can be read (or written) 16 bytes at a time: a lane's run of experts starts on a boundary of its own size.
bool rows_aligned(const void *p, long long stride, int dtype) {
    return aligned16(p) && stride * (dtype == EP_F32 ? 4 : 2) % 16 == 0;
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
        return by_width(n_experts, [&](auto v) {
            using E = std::remove_const_t<std::remove_pointer_t<P>>;
            return launch_pdl(ep_router_topk_kernel<E, decltype(v)::value>, dim3(grid), dim3(kRouterThreads), 0,
                              as_stream(stream), (P)logits, stride, bias, T, n_experts, K, sc,
                              (int)rows_aligned(logits, stride, dtype) | (aligned16(bias) ? 2 : 0), one_wave(grid), topk_ids,
                              topk_probs);
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
        return by_width(n_experts, [&](auto v) {
            using E = std::remove_const_t<std::remove_pointer_t<P>>;
            return launch_pdl(ep_router_topk_bwd_kernel<E, decltype(v)::value>, dim3(grid), dim3(kRouterThreads), 0,
                              as_stream(stream), grad_probs, (P)logits, stride, topk_ids, T, n_experts, K, sc,
                              (int)rows_aligned(logits, stride, dtype), (int)rows_aligned(grad_logits, n_experts, dtype),
                              one_wave(grid), (E *)grad_logits);
        });
    });
}
