// ep_experts.cu -- products of the experts' 4-bit weights with the rows of a dispatch layout, for
// batches of few tokens (decode), optionally with the gated activation silu(gate) * up.
//
// Weights are in the format the NVFP4 dispatch writes: E2M1 codes, two per byte, with an E4M3 scale
// per 16 elements, and an fp32 scale per output row.
#include "ep_host.h"
#include "ep_types.cuh"

namespace ep {
namespace {

constexpr int kExpertThreads = 256;

__device__ __forceinline__ float e2m1_value(unsigned c) {
    const float mag = (c & 4u) ? (float)((2u | (c & 1u)) << ((c >> 1) & 1u)) : 0.5f * (float)(c & 3u);
    return (c & 8u) ? -mag : mag;
}
__device__ __forceinline__ float e4m3_value(unsigned c) {
    const unsigned e = (c >> 3) & 15u, m = c & 7u;
    const float mag = e == 0u ? (float)m * 0x1p-9f : __uint_as_float(((e + 120u) << 23) | (m << 20));
    return (c & 0x80u) ? -mag : mag;
}

struct ExpertArgs {
    const uint16_t *x;
    const uint8_t *codes, *scales;
    const float *row_scale;
    int H, N, by_token, swiglu, T, G, R_max;
    const int32_t *row_offsets, *src_info, *status;
    uint16_t *out;
};

// Product of weight row n of group g with the row x (one warp; the same value in every lane).
__device__ __forceinline__ float row_product(const ExpertArgs &a, int g, int n, const uint16_t *x, int lane) {
    const size_t r = (size_t)g * a.N + n;
    const uint8_t *c = a.codes + r * (a.H / 2), *s = a.scales + r * (a.H / 16);
    float sum = 0.0f;
    for (int k = lane; k < a.H / 2; k += 32) {
        const unsigned b = c[k];
        const float sc = e4m3_value(s[k / 8]);
        sum = fmaf(e2m1_value(b & 15u) * sc, bf16_lo(x[2 * k]), sum);
        sum = fmaf(e2m1_value(b >> 4) * sc, bf16_lo(x[2 * k + 1]), sum);
    }
    return warp_sum(sum) * a.row_scale[r];
}

// One warp per output element.
__global__ void __launch_bounds__(kExpertThreads)
ep_expert_matvec_kernel(ExpertArgs a) {
    pdl_wait();
    if (cta_status(a.status)) return;
    const int lane = threadIdx.x & 31;
    const int n_out = a.swiglu ? a.N / 2 : a.N;
    const int n = blockIdx.x * (kExpertThreads / 32) + (threadIdx.x >> 5);
    if (n >= n_out) return;
    int g = 0;
    const int R = a.row_offsets[a.G];
    for (int row = blockIdx.y; row < R && row < a.R_max; row += gridDim.y) {
        while (g < a.G && a.row_offsets[g + 1] <= row) ++g;
        const int src = a.by_token ? a.src_info[2 * (size_t)row] : row;
        float v = 0.0f;
        if (src >= 0 && src < (a.by_token ? a.T : a.R_max)) {
            const uint16_t *x = a.x + (size_t)src * a.H;
            v = row_product(a, g, n, x, lane);
            if (a.swiglu) {
                const float up = row_product(a, g, n_out + n, x, lane);
                v = v / (1.0f + expf(-v)) * up;
            }
        } else if (src != -1) {
            bounds_fail(a.status);
        }
        if (lane == 0) a.out[(size_t)row * n_out + n] = __bfloat16_as_ushort(__float2bfloat16_rn(v));
    }
}

}  // namespace
}  // namespace ep

using namespace ep;

extern "C" int ep_expert_matvec(const uint16_t *x, int x_by_token, const uint8_t *codes, const uint8_t *scales,
                                const float *row_scale, int hidden_size, int out_rows, int swiglu,
                                const ep_layout_t *L, uint16_t *out, void *stream) {
    EP_NVTX_RANGE("ep_expert_matvec");
    const int H = hidden_size, N = out_rows;
    if (!layout_ok(L) || !hidden_ok(H) || N < 1 || N > kMaxN || (swiglu != 0 && swiglu != 1)) return EP_ERR_INVALID_ARG;
    if ((x_by_token != 0 && x_by_token != 1) || (swiglu && N % 2 != 0)) return EP_ERR_INVALID_ARG;
    const void *ptrs[] = {x, codes, scales, row_scale, out};
    for (const void *p : ptrs)
        if (!aligned16(p)) return EP_ERR_INVALID_ARG;
    if (L->T == 0) return EP_OK;
    for (const void *p : ptrs)
        if (!p) return EP_ERR_INVALID_ARG;
    if (x_by_token && !L->src_info) return EP_ERR_INVALID_ARG;
    ExpertArgs a = {x, codes, scales, row_scale, H, N, x_by_token, swiglu, L->T, L->E + L->fused_shared,
                    layout_rows(L), L->row_offsets, L->src_info, L->status, out};
    const int n_out = swiglu ? N / 2 : N;
    const int warps = kExpertThreads / 32;
    const int rows = a.R_max < 256 ? a.R_max : 256;
    return launch_pdl(ep_expert_matvec_kernel, dim3((n_out + warps - 1) / warps, rows), dim3(kExpertThreads), 0,
                      as_stream(stream), a);
}
