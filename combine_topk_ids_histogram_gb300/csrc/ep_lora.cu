// ep_lora.cu -- low-rank adapters of many requests at once beside a shared projection: tokens are grouped by adapter with a
// dispatch layout, and
//
//   out[t, :] = y[t, :] + scale[g] * B[g] (A[g] x[t, :])         for the adapter g of token t,
//
// out[t] = y[t] for a token without one.  A [G, r, H] and B [G, N, r] are read once per tile of rows, x and y once: HBM bounds
// prompts, latency decode steps, so both products are one kernel.  A cluster of C CTAs takes a tile of rows.  Its warps split H
// and add up A x with mma.sync (rows as M, r as N; the tensor cores are far from their rate at r <= 128), the partial sums are
// added in a fixed order, first a CTA's warps through shared memory, then the CTAs through each other's, and the warps then
// split N for the second product, which takes y along.  The contraction may take its k in any order as long as both
// operands take the same one: a thread reads 8 consecutive elements of a row, and columns of the second product
// are permuted so that a thread's sums are 8 consecutive outputs.
#include <algorithm>

#include "ep_host.h"
#include "ep_tensor.cuh"
#include "ep_types.cuh"

namespace ep {
namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kMaxRank = 128;
constexpr int kMaxCluster = 8;

struct LoraArgs {
    const uint16_t *y, *x, *a, *b;
    const float *scale;
    long long ldy, ldx, ldo;
    int H, N, r, T, G, R_max, by_token;
    int rows;                            // of the layout in a tile
    int tiles, C;                        // tiles of rows, and CTAs on each
    const int32_t *row_offsets, *expert_ids, *src_info, *row_of, *status;
    uint16_t *out;
};

template <typename T>
__device__ __forceinline__ void mma16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
    if constexpr (std::is_same_v<T, __half>)
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
                     : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3]) : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
    else
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
                     : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3]) : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ float ld_cluster_f32(uint32_t addr) {
    float v;
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
    return v;
}

// A sum v of A x as two 16-bit numbers, hi + lo: their products with B are exact in fp32, and v keeps 16 bits (bf16) or 22 (fp16).
template <typename T> __device__ __forceinline__ void split2(float v0, float v1, uint32_t &hi, uint32_t &lo) {
    hi = f32_to_word(v0, v1, T());
    const float2 h = word_to_f32(hi, T());
    lo = f32_to_word(v0 - h.x, v1 - h.y, T());
}

// Rows without an adapter, to another buffer.
__device__ void copy_rows(const LoraArgs &a, int cta, int ctas) {
    for (int t = cta * kWarps + (threadIdx.x >> 5); t < a.T; t += ctas * kWarps) {
        const int row = a.row_of[t];
        if (row >= 0 && row < a.R_max) continue;
        for (int n = (threadIdx.x & 31) * 8; n < a.N; n += 256)
            *reinterpret_cast<uint4 *>(a.out + t * a.ldo + n) = *reinterpret_cast<const uint4 *>(a.y + t * a.ldy + n);
    }
}

// RN: r / 8 rounded up to 2, 4, 8 or 16; MM: 16 rows each.
template <typename T, int RN, int MM>
__global__ void __launch_bounds__(kThreads) ep_lora_kernel(const LoraArgs a, int one_wave) {
    constexpr int kR = 8 * RN, kRows = 16 * MM, kCells = kRows * kR;
    constexpr int kSteps = RN <= 2 ? 4 : RN <= 4 ? 2 : 1;    // of 32 k in flight per warp
    extern __shared__ float s_part[];                        // [kWarps][kRows][kR], then this CTA's sums, then all CTAs'
    float *const s_mine = s_part + kWarps * kCells, *const s_all = s_mine + kCells;
    __shared__ float s_scale[kRows];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, c = lane >> 2, q = lane & 3;
    pdl_begin_if(one_wave);
    const int tile = blockIdx.x / a.C, rank = blockIdx.x % a.C;
    if constexpr (kBoundsCheck) {                            // another CTA may set a bit meanwhile: the cluster acts on one reading
        __shared__ int s_status;
        if (tid == 0) s_status = load_status(a.status);
        cluster_sync_all();
        const uint32_t first = at_rank(smem_u32(&s_status), 0);
        int st;
        asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(st) : "r"(first) : "memory");
        cluster_sync_all();
        if (st) return;
    } else if (load_status(a.status)) {
        return;
    }
    if (tile >= a.tiles) {
        copy_rows(a, blockIdx.x - a.tiles * a.C, gridDim.x - a.tiles * a.C);
        return;
    }
    const int R = min(a.row_offsets[a.G], a.R_max), end = min(R, (tile + 1) * a.rows);
    int next;
    for (int row = tile * a.rows; row < end; row = next) {
        const int g = a.expert_ids[row];
        next = row + 1;
        if (g < 0 || g >= a.G) {
            bounds_fail(a.status);
            continue;
        }
        next = max(min(end, a.row_offsets[g + 1]), next);    // the tile's rows of this adapter
        const int rows = next - row;
        int at[2 * MM];                                      // the row of x, y and out; -1: none
#pragma unroll
        for (int i = 0; i < 2 * MM; ++i) {
            const int j = c + 8 * i;
            at[i] = j < rows ? (a.by_token ? a.src_info[2 * (size_t)(row + j)] : row + j) : -1;
            if (a.by_token && at[i] >= a.T) {
                bounds_fail(a.status);
                at[i] = -1;
            }
        }
        float acc[MM][RN][4] = {};
        for (int st = rank * kWarps + warp; st * 32 < a.H; st += kSteps * a.C * kWarps) {
            uint4 xv[kSteps][2 * MM], wv[kSteps][RN];
            const uint4 zero = make_uint4(0, 0, 0, 0);
#pragma unroll
            for (int u = 0; u < kSteps; ++u) {
                const int k = (st + u * a.C * kWarps) * 32 + 8 * q;
#pragma unroll
                for (int j = 0; j < RN; ++j)
                    wv[u][j] = k < a.H && 8 * j + c < a.r ? *reinterpret_cast<const uint4 *>(a.a + ((size_t)g * a.r + 8 * j + c) * a.H + k) : zero;
#pragma unroll
                for (int i = 0; i < 2 * MM; ++i)
                    xv[u][i] = k < a.H && at[i] >= 0 ? *reinterpret_cast<const uint4 *>(a.x + at[i] * a.ldx + k) : zero;
            }
#pragma unroll
            for (int u = 0; u < kSteps; ++u)
#pragma unroll
                for (int j = 0; j < RN; ++j)
#pragma unroll
                    for (int m = 0; m < MM; ++m) {
                        mma16<T>(acc[m][j], xv[u][2 * m].x, xv[u][2 * m + 1].x, xv[u][2 * m].y, xv[u][2 * m + 1].y, wv[u][j].x, wv[u][j].y);
                        mma16<T>(acc[m][j], xv[u][2 * m].z, xv[u][2 * m + 1].z, xv[u][2 * m].w, xv[u][2 * m + 1].w, wv[u][j].z, wv[u][j].w);
                    }
        }
#pragma unroll
        for (int m = 0; m < MM; ++m)
#pragma unroll
            for (int j = 0; j < RN; ++j) {
                float *const p = s_part + warp * kCells + (16 * m + c) * kR + 8 * j + 2 * q;
                *reinterpret_cast<float2 *>(p) = make_float2(acc[m][j][0], acc[m][j][1]);
                *reinterpret_cast<float2 *>(p + 8 * kR) = make_float2(acc[m][j][2], acc[m][j][3]);
            }
        __syncthreads();
        for (int i = tid; i < kCells; i += kThreads) {
            float v = 0.0f;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) v += s_part[w * kCells + i];
            s_mine[i] = v;
        }
        cluster_sync_all();
        for (int i = tid; i < kCells; i += kThreads) {
            float v = 0.0f;
            for (int k = 0; k < a.C; ++k) v += ld_cluster_f32(at_rank(smem_u32(s_mine + i), k));
            s_all[i] = v;
        }
        __syncthreads();
        if constexpr (std::is_same_v<T, __half>) {           // a power of two per row keeps the sums in fp16's range
            for (int i = warp; i < kRows; i += kWarps) {
                float v = 0.0f;
                for (int k = lane; k < kR; k += 32) v = fmaxf(v, fabsf(s_all[i * kR + k]));
                v = warp_max(v);
                if (lane == 0) s_scale[i] = v > 0.0f && v < 3.4e38f ? exp2f((float)min(14 - ilogbf(v), 126)) : 1.0f;
            }
            __syncthreads();
        }
        constexpr int kK = RN / 2;                           // steps of 16 of the second product
        uint32_t hi[MM][kK][4], lo[MM][kK][4];
        float back[2 * MM];                                  // adapter's scale, over the row's
        const float scale = a.scale ? a.scale[g] : 1.0f;
#pragma unroll
        for (int i = 0; i < 2 * MM; ++i) {
            const int j = c + 8 * i;
            float f = 1.0f;
            if constexpr (std::is_same_v<T, __half>) f = s_scale[j];
            back[i] = scale / f;
#pragma unroll
            for (int s = 0; s < kK; ++s)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int k = RN == 2 ? 4 * q + 2 * h : s / 2 * 32 + 8 * q + s % 2 * 4 + 2 * h;
                    const float2 v = *reinterpret_cast<const float2 *>(s_all + j * kR + k);
                    split2<T>(v.x * f, v.y * f, hi[i / 2][s][i % 2 + 2 * h], lo[i / 2][s][i % 2 + 2 * h]);
                }
        }
        for (int blk = rank * kWarps + warp; blk * 32 < a.N; blk += a.C * kWarps) {
            const int n = blk * 32 + 8 * q;
            uint4 yv[2 * MM];
#pragma unroll
            for (int i = 0; i < 2 * MM; ++i)
                if (n < a.N && at[i] >= 0) yv[i] = *reinterpret_cast<const uint4 *>(a.y + at[i] * a.ldy + n);
            float sum[MM][4][4] = {};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int nb = blk * 32 + 8 * (c >> 1) + 2 * j + (c & 1);
                const uint16_t *const bp = a.b + ((size_t)g * a.N + nb) * a.r;
                uint32_t bv[2 * kK];
                if constexpr (RN == 2) {
                    uint2 v = make_uint2(0, 0);
                    if (nb < a.N && 4 * q < a.r) v = *reinterpret_cast<const uint2 *>(bp + 4 * q);
                    bv[0] = v.x;
                    bv[1] = v.y;
                } else {
#pragma unroll
                    for (int s = 0; s < kK / 2; ++s) {
                        uint4 v = make_uint4(0, 0, 0, 0);
                        if (nb < a.N && 32 * s + 8 * q < a.r) v = *reinterpret_cast<const uint4 *>(bp + 32 * s + 8 * q);
                        bv[4 * s] = v.x;
                        bv[4 * s + 1] = v.y;
                        bv[4 * s + 2] = v.z;
                        bv[4 * s + 3] = v.w;
                    }
                }
#pragma unroll
                for (int s = 0; s < kK; ++s)
#pragma unroll
                    for (int m = 0; m < MM; ++m) {
                        mma16<T>(sum[m][j], lo[m][s][0], lo[m][s][1], lo[m][s][2], lo[m][s][3], bv[2 * s], bv[2 * s + 1]);
                        mma16<T>(sum[m][j], hi[m][s][0], hi[m][s][1], hi[m][s][2], hi[m][s][3], bv[2 * s], bv[2 * s + 1]);
                    }
            }
            if (n < a.N) {
#pragma unroll
                for (int i = 0; i < 2 * MM; ++i)
                    if (at[i] >= 0) {
                        const uint32_t w[4] = {yv[i].x, yv[i].y, yv[i].z, yv[i].w};
                        uint32_t o[4];
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            const float2 v = word_to_f32(w[j], T());
                            o[j] = f32_to_word(fmaf(back[i], sum[i / 2][j][i % 2 * 2], v.x), fmaf(back[i], sum[i / 2][j][i % 2 * 2 + 1], v.y), T());
                        }
                        *reinterpret_cast<uint4 *>(a.out + at[i] * a.ldo + n) = make_uint4(o[0], o[1], o[2], o[3]);
                    }
            }
        }
        cluster_sync_all();                                  // the sums have been read everywhere
    }
}

template <typename T, int RN, int MM> int launch_lora(const LoraArgs &a, int copy, cudaStream_t st) {
    constexpr auto kern = ep_lora_kernel<T, RN, MM>;
    constexpr size_t smem = (size_t)(kWarps + 2) * 16 * MM * 8 * RN * sizeof(float);
    const int rc = allow_smem<kern>(smem);
    if (rc != EP_OK) return rc;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(a.tiles * a.C + copy));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = a.C;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return launch_result(cudaLaunchKernelEx(&cfg, kern, a, one_wave((int)cfg.gridDim.x)));
}

template <typename T> int launch_rank(const LoraArgs &a, int copy, cudaStream_t st) {
    const bool wide = a.rows > 16;
    if (a.r <= 16) return wide ? launch_lora<T, 2, 2>(a, copy, st) : launch_lora<T, 2, 1>(a, copy, st);
    if (a.r <= 32) return wide ? launch_lora<T, 4, 2>(a, copy, st) : launch_lora<T, 4, 1>(a, copy, st);
    if (a.r <= 64) return wide ? launch_lora<T, 8, 2>(a, copy, st) : launch_lora<T, 8, 1>(a, copy, st);
    return launch_lora<T, 16, 1>(a, copy, st);
}

bool lora_stride_ok(long long ld, int cols) { return ld >= cols && ld % 8 == 0; }

}  // namespace
}  // namespace ep

using namespace ep;

extern "C" int ep_lora_add(const void *y, long long y_stride, const void *x, long long x_stride, const void *a, const void *b,
                           const float *scale, int in_features, int out_features, int rank, int dtype, int by_token,
                           const ep_layout_t *L, void *out, long long out_stride, void *stream) {
    EP_NVTX_RANGE("ep_lora_add");
    const int H = in_features, N = out_features;
    if (!layout_ok(L) || !hidden_ok(H) || N < 16 || N > kMaxN || N % 16 != 0 || rank < 8 || rank > kMaxRank || rank % 8 != 0)
        return EP_ERR_INVALID_ARG;
    if ((dtype != EP_BF16 && dtype != EP_F16) || (by_token != 0 && by_token != 1)) return EP_ERR_INVALID_ARG;
    if (!lora_stride_ok(y_stride, N) || !lora_stride_ok(x_stride, H) || !lora_stride_ok(out_stride, N)) return EP_ERR_INVALID_ARG;
    // one adapter per token, so that no two rows name the same output
    if (by_token && (L->K != 1 || L->fused_shared)) return EP_ERR_INVALID_ARG;
    if (out == y && out_stride != y_stride) return EP_ERR_INVALID_ARG;
    for (const void *p : {y, x, a, b, (const void *)scale, (const void *)out})
        if (!aligned16(p)) return EP_ERR_INVALID_ARG;
    if (L->T == 0) return EP_OK;
    if (!y || !x || !a || !b || !out || !L->expert_ids || (by_token && !L->src_info)) return EP_ERR_INVALID_ARG;
    LoraArgs p = {};
    p.y = (const uint16_t *)y; p.x = (const uint16_t *)x; p.a = (const uint16_t *)a; p.b = (const uint16_t *)b;
    p.scale = scale; p.ldy = y_stride; p.ldx = x_stride; p.ldo = out_stride;
    p.H = H; p.N = N; p.r = rank; p.T = L->T; p.G = L->E + L->fused_shared; p.R_max = layout_rows(L); p.by_token = by_token;
    p.row_offsets = L->row_offsets; p.expert_ids = L->expert_ids; p.src_info = L->src_info; p.row_of = L->row_of; p.status = L->status;
    p.out = (uint16_t *)out;
    if (p.R_max == 0) p.R_max = 1;
    // a tile's rows: about as many as an adapter has
    const long long per = (long long)L->T * L->K / p.G;
    const int most = rank > 64 ? 16 : 32;
    p.rows = 1;
    while (p.rows < most && p.rows < per) p.rows *= 2;
    p.tiles = (p.R_max + p.rows - 1) / p.rows;
    p.C = 1;
    const int sms = std::max(device_sm_count(), 1);
    while (p.C < kMaxCluster && (long long)p.tiles * p.C < 2 * sms && p.C * kWarps * 32 < std::max(H, N)) p.C *= 2;
    int copy = by_token && out != y ? std::min((L->T + kWarps - 1) / kWarps, 2 * sms) : 0;
    copy = (copy + p.C - 1) / p.C * p.C;
    cudaStream_t st = as_stream(stream);
    return dtype == EP_F16 ? launch_rank<__half>(p, copy, st) : launch_rank<__nv_bfloat16>(p, copy, st);
}
