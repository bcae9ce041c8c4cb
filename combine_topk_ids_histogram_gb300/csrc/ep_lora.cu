// ep_lora.cu -- low-rank adapters of many requests at once beside a shared projection: tokens are grouped by adapter with a
// dispatch layout, and
//
//   out[t, :] = y[t, :] + scale[g] * B[g] (A[g] x[t, :])         for the adapter g of token t,
//
// out[t] = y[t] for a token without one.  A [G, r, H] and B [G, N, r] are read once per tile of rows, x and y once.  A cluster of
// C CTAs takes a tile of rows, all of one adapter, and both products of it, so that the r sums per row never leave the SMs:
//   few rows    up to 16, on mma.sync (rows as M, r as N).  The warps of the cluster split H, add the sums up in a fixed order, first a
//               CTA's through shared memory, then the CTAs' through each other's, and split N for the second product,
//               which takes y along.  The contraction may take its k in any order as long as both operands take the same one: a thread reads
//               8 consecutive elements of a row, and the second product's columns are permuted so that a thread's sums are
//               8 consecutive outputs.  One token, rank 16, 2048 -> 2048: 3.7 us; 64 tokens, 48 adapters of rank 32, 7168 -> 4096:
//               9.5 us (floor 3.9).  Latency bounds it: the ids, A and x, the exchange, one after another.
//   many rows   128, on tcgen05.  8192 tokens, 5 adapters of rank 64, 4096 -> 4096: 57 us (floor 29).  HBM bounds the second half
//               (5 TB/s), the copies' latency and the exchange of the sums between the CTAs the first.
#include <stddef.h>

#include <algorithm>
#include <type_traits>

#include "ep_async.cuh"
#include "ep_host.h"
#include "ep_ring.h"
#include "ep_tensor.cuh"
#include "ep_types.cuh"

namespace ep {
namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kMaxRank = 128;
constexpr int kMaxCluster = 8;
// The tensor cores' adder cuts off what it adds, to one side: sums of A x leave it after so many products and go on in fp32, rounded to
// nearest.  (Of 32768 fp16 products of one sign 2e-4 would be lost, of 512 3e-6.  The second product has 128 at most.)
constexpr int kLongest = 512;

struct LoraArgs {
    const uint16_t *y, *x, *a, *b;
    const float *scale;
    long long ldy, ldx, ldo;
    int H, N, r, T, G, R_max, by_token;
    int rows;                            // of the layout in a tile
    int tiles, heads, C;                 // tiles of rows; adapters' first rows apart (0 or G); CTAs on each
    int copy;                            // whether rows without an adapter have to be copied
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
__device__ __forceinline__ int ld_cluster_s32(uint32_t addr) {
    int v;
    asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
    return v;
}
__device__ __forceinline__ float ld_cluster_f32(uint32_t addr) {
    float v;
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
    return v;
}

__device__ __forceinline__ void st_cluster_x4(uint32_t addr, const uint32_t (&v)[4]) {
    asm volatile("st.shared::cluster.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]) : "memory");
}
__device__ __forceinline__ float4 ld_cluster_f32x4(uint32_t addr) {
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(addr) : "memory");
    return v;
}

// The magnitude that counts for a row's scale: infinities are theirs whatever it is.
__device__ __forceinline__ float finite_abs(float v) { return fabsf(v) <= FLT_MAX ? fabsf(v) : 0.0f; }
// The power of two that brings a largest magnitude to [2^14, 2^15), in fp16's range: from its exponent (1 for 0).
__device__ __forceinline__ float fp16_scale(float most) {
    const int e = (int)(__float_as_uint(most) >> 23) - 127;
    return most > 0.0f ? __uint_as_float((uint32_t)(min(14 - e, 126) + 127) << 23) : 1.0f;
}

// A sum v of A x as two 16-bit numbers, hi + lo: their products with B are exact in fp32, and v keeps 16 bits (bf16) or 22 (fp16).
// Where v, hi or an element of B is infinite, those products may cancel to NaN: sums that are not finite are added up anew from v.
template <typename T> __device__ __forceinline__ void split2(float v0, float v1, uint32_t &hi, uint32_t &lo) {
    hi = f32_to_word(v0, v1, T());
    const float2 h = word_to_f32(hi, T());
    lo = f32_to_word(v0 - h.x, v1 - h.y, T());
}
// The same where v has to be found again in hi + lo: an infinite one has no lo, and a finite one whose hi is infinite (above bf16's largest
// number) the largest number as hi.
template <typename T> __device__ __forceinline__ void split2_whole(float v0, float v1, uint32_t &hi, uint32_t &lo) {
    split2<T>(v0, v1, hi, lo);
    const float2 h = word_to_f32(hi, T());
    if (fmaxf(fabsf(h.x), fabsf(h.y)) <= FLT_MAX) return;
    constexpr uint32_t kInf = std::is_same_v<T, __half> ? 0x7c00u : 0x7f80u;
    const float v[2] = {v0, v1};
    uint32_t w[2] = {hi & 0xffffu, hi >> 16}, l[2] = {lo & 0xffffu, lo >> 16};
#pragma unroll
    for (int i = 0; i < 2; ++i)
        if ((w[i] & 0x7fffu) == kInf) {
            if (fabsf(v[i]) <= FLT_MAX) {
                w[i] -= 1;
                l[i] = f32_to_word(v[i] - word_to_f32(w[i], T()).x, 0.0f, T()) & 0xffffu;
            } else {
                l[i] = 0;
            }
        }
    hi = w[0] | w[1] << 16;
    lo = l[0] | l[1] << 16;
}
// Whether one of these is NaN or infinite.
template <typename... Vs> __device__ __forceinline__ bool not_finite(Vs... v) {
    float z = 0.0f;
    ((z = fmaf(v, 0.0f, z)), ...);
    return !(z == 0.0f);
}

// The rows of a cluster, all of one adapter: of tile t those from its first row to the end of that row's adapter, and of tile
// `tiles` + g the first rows of adapter g, up to where a tile begins.  (Tiles of several adapters would take as often as long.)
struct Rows {
    int g, first, end;                   // end <= first: none
    __device__ __forceinline__ Rows(const LoraArgs &a, int tile) {
        if (tile < a.tiles) {
            first = tile * a.rows;
            g = a.expert_ids[first];     // these loads go out together
            const int R = min(a.row_offsets[a.G], a.R_max);
            end = min(R, first + a.rows);
            if (first >= R) return;
            if (g < 0 || g >= a.G) {
                if (kBoundsCheck && load_status(a.status) == 0) bounds_fail(a.status);
                end = first;
            } else if (a.rows > 1) {
                end = min(end, a.row_offsets[g + 1]);
            }
        } else {
            g = tile - a.tiles;
            first = min(max(a.row_offsets[g], 0), a.R_max);
            end = min(min(a.row_offsets[g + 1], a.R_max), (first + a.rows - 1) / a.rows * a.rows);
        }
    }
};

// Rows without an adapter, to another buffer: the first eight warps of every CTA take some, eight 16-byte pieces per lane at a time.
__device__ __forceinline__ void copy_rows(const LoraArgs &a) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    for (int t = blockIdx.x * kWarps + warp; warp < kWarps && t < a.T; t += gridDim.x * kWarps) {
        const int row = a.row_of[t];
        if (row >= 0 && row < a.R_max) continue;
        for (int n0 = lane * 8; n0 < a.N; n0 += 8 * 256) {
            uint4 v[8];
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (n0 + i * 256 < a.N) v[i] = *reinterpret_cast<const uint4 *>(a.y + t * a.ldy + n0 + i * 256);
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (n0 + i * 256 < a.N) *reinterpret_cast<uint4 *>(a.out + t * a.ldo + n0 + i * 256) = v[i];
        }
    }
}

// What a thread needs of 32 columns of B and y: rows c and c + 8 of its 16.
template <int RN> struct Block {
    uint4 y[2];
    uint32_t b[4][RN];                                       // r in the order of the sums' fragments
    __device__ __forceinline__ void load(const LoraArgs &a, int g, int n0, const int (&at)[2], int c, int q) {
        const int n = n0 + 8 * q;
#pragma unroll
        for (int i = 0; i < 2; ++i)
            if (n < a.N && at[i] >= 0) y[i] = *reinterpret_cast<const uint4 *>(a.y + at[i] * a.ldy + n);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int nb = n0 + 8 * (c >> 1) + 2 * j + (c & 1);
            const uint16_t *const bp = a.b + ((size_t)g * a.N + nb) * a.r;
            if constexpr (RN == 2) {
                uint2 v = make_uint2(0, 0);
                if (nb < a.N && 4 * q < a.r) v = *reinterpret_cast<const uint2 *>(bp + 4 * q);
                b[j][0] = v.x;
                b[j][1] = v.y;
            } else {
#pragma unroll
                for (int s = 0; s < RN / 4; ++s) {
                    uint4 v = make_uint4(0, 0, 0, 0);
                    if (nb < a.N && 32 * s + 8 * q < a.r) v = *reinterpret_cast<const uint4 *>(bp + 32 * s + 8 * q);
                    b[j][4 * s] = v.x;
                    b[j][4 * s + 1] = v.y;
                    b[j][4 * s + 2] = v.z;
                    b[j][4 * s + 3] = v.w;
                }
            }
        }
    }
};

// Up to 16 rows to a tile; the warps split H and N.  RN: r / 8 rounded up to 2, 4, 8 or 16.
template <typename T, int RN>
__global__ void __launch_bounds__(kThreads, 2) ep_lora_kernel(const LoraArgs a, int one_wave) {
    constexpr int kR = 8 * RN, kRows = 16, kCells = kRows * kR;
    constexpr int kSteps = RN <= 2 ? 4 : 2;                  // of 32 k in flight per warp, one behind the other in a row
    constexpr bool kAhead = RN <= 8;                         // the first block of B and y comes along with A and x
    extern __shared__ float s_part[];                        // [kWarps][kRows][kR], then this CTA's sums, then all CTAs'
    float *const s_mine = s_part + kWarps * kCells, *const s_all = a.C > 1 ? s_mine + kCells : s_mine;
    __shared__ float s_scale[kRows];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, c = lane >> 2, q = lane & 3;
    pdl_begin_if(one_wave);
    const int tile = blockIdx.x / a.C, rank = blockIdx.x % a.C, part = rank * kWarps + warp, parts = a.C * kWarps;
    int token[2] = {};                                       // comes along with the loads of Rows
    if (a.by_token && tile < a.tiles) {
#pragma unroll
        for (int i = 0; i < 2; ++i) token[i] = a.src_info[2 * (size_t)min(tile * a.rows + c + 8 * i, a.R_max - 1)];
    }
    const Rows rows(a, tile);
    // Another kernel that uses the layout may set a bit meanwhile, and so may this one: the cluster acts on one reading, the first
    // CTA's, once it meets.  Until then nothing is written, and whatever a layout with a status holds is checked like any other.
    __shared__ int s_status;
    const int status = load_status(a.status);
    if (rows.end <= rows.first) {
        if (a.copy && status == 0) copy_rows(a);
        return;
    }
    const int g = rows.g, cells = (rows.end - rows.first) * kR;
    const float scale = a.scale ? a.scale[g] : 1.0f;
    int at[2];                                               // the row of x, y and out; -1: none
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int j = rows.first + c + 8 * i;
        at[i] = j >= rows.end ? -1 : !a.by_token ? j : tile < a.tiles ? token[i] : a.src_info[2 * (size_t)j];
        if (a.by_token && at[i] >= a.T) {
            if (status == 0) bounds_fail(a.status);
            at[i] = -1;
        }
    }
    Block<RN> ahead;
    if (kAhead) ahead.load(a, g, part * 32, at, c, q);
    float acc[RN][4] = {};
    const uint4 zero = make_uint4(0, 0, 0, 0);
    // The warp's sums so far, to the thread's own places in shared memory.
    auto put = [&](bool first) {
#pragma unroll
        for (int j = 0; j < RN; ++j)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                if (i == 1 && cells <= 8 * kR) break;
                float2 *const p = reinterpret_cast<float2 *>(s_part + warp * kCells + (c + 8 * i) * kR + 8 * j + 2 * q);
                float2 v = make_float2(acc[j][2 * i], acc[j][2 * i + 1]);
                if (!first) v = make_float2(p->x + v.x, p->y + v.y);
                *p = v;
                acc[j][2 * i] = acc[j][2 * i + 1] = 0.0f;
            }
    };
    int until = kLongest / (kSteps * 32);                    // turns until the sums leave the tensor cores
    bool first = true;
    for (int k0 = part * kSteps * 32; k0 < a.H; k0 += parts * kSteps * 32) {
        if (until-- == 0) {
            put(first);
            first = false;
            until = kLongest / (kSteps * 32) - 1;
        }
        uint4 xv[kSteps][2];
#pragma unroll
        for (int u = 0; u < kSteps; ++u)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int k = k0 + 32 * u + 8 * q;
                xv[u][i] = k < a.H && at[i] >= 0 ? *reinterpret_cast<const uint4 *>(a.x + at[i] * a.ldx + k) : zero;
            }
#pragma unroll
        for (int u = 0; u < kSteps; ++u) {
            const int k = k0 + 32 * u + 8 * q;
            const uint16_t *const ap = a.a + ((size_t)g * a.r + c) * a.H + k;
#pragma unroll
            for (int j0 = 0; j0 < RN; j0 += 8) {
                uint4 wv[RN < 8 ? RN : 8];
#pragma unroll
                for (int j = j0; j < RN && j < j0 + 8; ++j)
                    wv[j - j0] = k < a.H && 8 * j + c < a.r ? *reinterpret_cast<const uint4 *>(ap + (size_t)8 * j * a.H) : zero;
#pragma unroll
                for (int j = j0; j < RN && j < j0 + 8; ++j) {
                    mma16<T>(acc[j], xv[u][0].x, xv[u][1].x, xv[u][0].y, xv[u][1].y, wv[j - j0].x, wv[j - j0].y);
                    mma16<T>(acc[j], xv[u][0].z, xv[u][1].z, xv[u][0].w, xv[u][1].w, wv[j - j0].z, wv[j - j0].w);
                }
            }
        }
    }
    put(first);
    if (tid == 0) s_status = status;
    __syncthreads();
    for (int i = tid; i < cells; i += kThreads) {            // (rows without a token stay undefined, and go into no other)
        float v = 0.0f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) v += s_part[w * kCells + i];
        s_mine[i] = (i & (kR - 1)) < a.r ? v : 0.0f;         // (an infinite x times the zeros behind A's rows is NaN)
    }
    int one_status = s_status;
    if (a.C > 1) {
        cluster_sync_all();
        one_status = ld_cluster_s32(at_rank(smem_u32(&s_status), 0));
        for (int i = tid; i < cells; i += kThreads) {
            float u[kMaxCluster], v = 0.0f;                  // loads on their way together: each takes some 700 cycles
#pragma unroll
            for (int k = 0; k < kMaxCluster; ++k)
                if (k < a.C) u[k] = ld_cluster_f32(at_rank(smem_u32(s_mine + i), k));
#pragma unroll
            for (int k = 0; k < kMaxCluster; ++k)
                if (k < a.C) v += u[k];
            s_all[i] = v;
        }
    }
    if (one_status) {
        if (a.C > 1) cluster_sync_all();                     // (read everywhere)
        return;
    }
    __syncthreads();
    if constexpr (std::is_same_v<T, __half>) {           // a power of two per row keeps the sums in fp16's range
        for (int i = warp; i * kR < cells; i += kWarps) {
            float v = 0.0f;
            for (int k = lane; k < kR; k += 32) v = fmaxf(v, finite_abs(s_all[i * kR + k]));
            v = warp_max(v);
            if (lane == 0) s_scale[i] = fp16_scale(v);
        }
        __syncthreads();
    }
    constexpr int kK = RN / 2;                       // steps of 16 of the second product
    uint32_t hi[kK][4], lo[kK][4];
    float back[2];                                           // adapter's scale, over the row's
#pragma unroll
    for (int i = 0; i < 2; ++i) {
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
                split2<T>(v.x * f, v.y * f, hi[s][i + 2 * h], lo[s][i + 2 * h]);
            }
    }
    // The second product from column n0 on.  The first time up to a block with a sum that is not finite (nearly never), of which it
    // writes nothing, and then with care: such outputs are added up from A x, B and y in memory.
    auto second = [&](auto with_care, int n0) {
        constexpr bool careful = decltype(with_care)::value;
        for (; n0 < a.N; n0 += parts * 32) {
            if (careful) __syncwarp();
            Block<RN> now;
            if (kAhead && !careful && n0 == part * 32) now = ahead;
            else now.load(a, g, n0, at, c, q);
            float sum[4][4] = {};
#pragma unroll
            for (int j = 0; j < 4; ++j)
#pragma unroll
                for (int s = 0; s < kK; ++s) {
                    mma16<T>(sum[j], lo[s][0], lo[s][1], lo[s][2], lo[s][3], now.b[j][2 * s], now.b[j][2 * s + 1]);
                    mma16<T>(sum[j], hi[s][0], hi[s][1], hi[s][2], hi[s][3], now.b[j][2 * s], now.b[j][2 * s + 1]);
                }
            bool odd[2];
#pragma unroll
            for (int i = 0; i < 2; ++i)
                odd[i] = at[i] >= 0 && not_finite(sum[0][2 * i], sum[0][2 * i + 1], sum[1][2 * i], sum[1][2 * i + 1], sum[2][2 * i], sum[2][2 * i + 1],
                                                  sum[3][2 * i], sum[3][2 * i + 1]);
            if (!careful && __any_sync(kFullMask, odd[0] || odd[1])) break;
            const int n = n0 + 8 * q;
            if (n >= a.N) continue;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                if (at[i] < 0) continue;
                uint16_t *const out = a.out + at[i] * a.ldo + n;
                if (careful && odd[i]) {
                    const float *const t = s_all + (c + 8 * i) * kR;
                    const uint16_t *bp = a.b + ((size_t)g * a.N + n) * a.r;
#pragma unroll 1
                    for (int e = 0; e < 8; ++e) {
                        float v = 0.0f;
#pragma unroll 1
                        for (int k = 0; k < a.r; ++k) v = fmaf(t[k], word_to_f32(*bp++, T()).x, v);
                        out[e] = (uint16_t)f32_to_word(fmaf(scale, v, word_to_f32(a.y[at[i] * a.ldy + n + e], T()).x), 0.0f, T());
                    }
                    continue;
                }
                const uint32_t w[4] = {now.y[i].x, now.y[i].y, now.y[i].z, now.y[i].w};
                uint32_t o[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float2 v = word_to_f32(w[j], T());
                    o[j] = f32_to_word(fmaf(back[i], sum[j][2 * i], v.x), fmaf(back[i], sum[j][2 * i + 1], v.y), T());
                }
                *reinterpret_cast<uint4 *>(out) = make_uint4(o[0], o[1], o[2], o[3]);
            }
        }
        return n0;
    };
    const int rest = second(std::false_type{}, part * 32);
    if (rest < a.N) second(std::true_type{}, rest);
    if (a.copy) copy_rows(a);
    if (a.C > 1) cluster_sync_all();                         // the sums have been read everywhere
}

// ------------------------------------------------------------------------------------------------------------ many rows
// The same for tiles of 128 rows on tcgen05, where the bytes of x, y and out are what counts.  The rows are M; both products stream
// through a ring in shared memory that cp.async fills ahead: 64 columns of x with 64 of A (N is r), then 64 of y with 64 rows of B
// (K is r).  The CTAs of a cluster split H, add up A x through each other's shared memory, and split N.  (With mma.sync from
// shared memory its products took half of the time: 71 us with 8192 tokens, 5 adapters of rank 64, 4096 -> 4096, where this takes 57.)
constexpr int kTileRows = 128, kTileThreads = kThreads + 32;           // the last warp issues the products

__device__ __forceinline__ void cp_async16_or_zero(uint32_t smem, const void *gmem, bool valid) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem), "l"(gmem), "r"(valid ? 16 : 0) : "memory");
}
// An arrival once this thread's copies so far have landed (counted in the barrier's total).
__device__ __forceinline__ void cp_async_arrive(uint32_t bar) {
    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
}

// Where 16-byte piece p (of 8) of a row is in a tile of 128-byte rows, in the swizzle that tcgen05.mma reads.
__device__ __forceinline__ uint32_t swizzled(int row, int p) { return row * 128 + ((p ^ (row & 7)) << 4); }

// RB: blocks of 64 that r fills at most (1: r <= 64, 2: r <= 128).
template <int RB> struct TileSmem {
    static constexpr int kPitch = 64 * RB + 4;               // of the exchanged sums, in fp32: 16 bytes of each row in banks of their own
    static constexpr int kLeft = kTileRows * 128, kRight = RB * 8192, kStage = kLeft + kRight;
    static constexpr int kLow = RB * kTileRows * 128;        // A x as 16-bit operand: high parts, then low parts
    static constexpr int kBytes = kRing * kStage + 2 * kLow + 1024;
    static_assert(kTileRows * kPitch * 4 <= kRing * kStage, "the exchanged sums take the place of the ring");
};

// Eight warps copy, add up and write; the ninth waits for what they copied and issues the products.  It fences as well: the
// fence between copies and tensor cores waits for all copies of the thread that issues it, those of later stages too.
template <typename T, int RB>
__global__ void __launch_bounds__(kTileThreads, RB == 1 ? 2 : 1) ep_lora_tile_kernel(const LoraArgs a, int one_wave) {
    using S = TileSmem<RB>;
    constexpr uint32_t kTmem = 128 * RB;                     // columns: twice the sums of A x, then of 64 outputs
    extern __shared__ __align__(16) uint8_t s_raw[];
    uint8_t *const smem = s_raw + (1024 - (smem_u32(s_raw) & 1023)) % 1024;
    __shared__ __align__(8) uint64_t s_full[kRing], s_free[kRing], s_done[kRing], s_taken[2];
    __shared__ uint32_t s_tmem;
    __shared__ float s_scale[kTileRows];
    __shared__ int s_at[kTileRows];
    const int tid = threadIdx.x, warp = __shfl_sync(kFullMask, tid >> 5, 0), lane = tid & 31;
    pdl_begin_if(one_wave);
    const int tile = blockIdx.x / a.C, rank = blockIdx.x % a.C;
    const Rows rows(a, tile);
    __shared__ int s_status;                                 // as above
    const int status = load_status(a.status);
    if (rows.end <= rows.first) {
        if (a.copy && status == 0) copy_rows(a);
        return;
    }
    if (tid == 0) s_status = status;
    const int g = rows.g;
    if (tid < kTileRows) {
        const int row = rows.first + tid;
        int at = row < rows.end ? (a.by_token ? a.src_info[2 * (size_t)row] : row) : -1;
        if (a.by_token && at >= a.T) {
            if (status == 0) bounds_fail(a.status);
            at = -1;
        }
        s_at[tid] = at;
    }
    if (warp == 4) tmem_alloc<1>(smem_u32(&s_tmem), kTmem);
    if (tid == 0) {
        for (int i = 0; i < kRing; ++i) {
            mbar_init(smem_u32(&s_full[i]), kThreads);
            mbar_init(smem_u32(&s_free[i]), kWarps);
            mbar_init(smem_u32(&s_done[i]), 1);
        }
        for (int i = 0; i < 2; ++i) mbar_init(smem_u32(&s_taken[i]), kWarps);
        mbar_init_done();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = s_tmem, ring = smem_u32(smem), low = ring + kRing * S::kStage;
    const bool f16 = std::is_same_v<T, __half>;
    const int n1 = (a.r + 15) & ~15;                         // r in steps of the tensor cores
    bool ok = true;                                          // false: a wait ran out, and the warp does no more of the loop it is in, nor of the next
    // This thread copies a 16-byte piece of rows tid / 8 + 32 i of both tiles.
    const int piece = tid & 7, r0 = (tid & (kThreads - 1)) >> 3;
    const uint32_t to = swizzled(r0, piece);
    const uint16_t *left[4];
    bool has[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int at = s_at[r0 + 32 * i];
        has[i] = at >= 0;
        left[i] = a.x + (has[i] ? at * a.ldx : 0) + 8 * piece;
    }
    const uint16_t *right = a.a + (size_t)g * a.r * a.H + 8 * piece;
    const int first1 = (a.H + 63) / 64 * rank / a.C;
    auto fill_first = [&](int i, int slot) {
        const int col = (first1 + i) * 64;
        if (col < a.H) {
            const uint32_t st = ring + slot * S::kStage + to;
            const bool in = col + 8 * piece < a.H;
#pragma unroll
            for (int j = 0; j < 4; ++j) cp_async16_or_zero(st + j * 4096, in ? left[j] + col : a.x, in && has[j]);
#pragma unroll
            for (int j = 0; j < 2 * RB; ++j) {
                const int r = r0 + 32 * j;
                const bool valid = in && r < a.r;
                if (r < n1) cp_async16_or_zero(st + S::kLeft + j * 4096, valid ? right + (size_t)r * a.H + col : a.a, valid);
            }
        }
        cp_async_arrive(smem_u32(&s_full[slot]));
    };
    // ---- A x: every CTA sums its stages of H.  Barriers' phases count on through both parts.
    const int first2 = (a.N + 63) / 64 * rank / a.C, stages1 = (a.H + 63) / 64 * (rank + 1) / a.C - first1, stages2 = (a.N + 63) / 64 * (rank + 1) / a.C - first2;
    auto wait = [&](uint64_t &bar, int phase) {
        if (ok) ok = __all_sync(kFullMask, mbar_wait(smem_u32(&bar), phase & 1));
        return ok;
    };
    const bool issuer = warp == kWarps;
    // Sums: rows q * 32 + lane, 32 * RB columns.  They leave tensor memory after every chunk of stages.
    const int q = warp & 3, half = (warp >> 2) & 1, row = q * 32 + lane;
    const uint32_t lanes = tmem + ((uint32_t)(q * 32) << 16);
    float total[RB][32] = {};
    auto take = [&](int chunk) {
        tc_fence_after();
#pragma unroll
        for (int b = 0; b < RB; ++b) {
            const int k0 = (half * RB + b) * 32;
            if (k0 >= n1) continue;
            float v[32];
            tmem_ld32(lanes + chunk_buffer(chunk) * 64 * RB + k0, v);
            tmem_wait_ld();
#pragma unroll
            for (int j = 0; j < 32; ++j) total[b][j] += v[j];
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(at_rank(smem_u32(&s_taken[chunk_buffer(chunk)]), cluster_rank()));
    };
    if (issuer) {
        const uint32_t id1 = mma_desc(f16, 128, n1, false, false);
        for (int i = 0; i < stages1; ++i) {
            const int slot = ring_slot(i);
            if (!wait(s_full[slot], ring_phase(i))) break;
            const int chunk = stage_chunk(i);
            if (chunk_begins(i) && chunk >= 2 && !wait(s_taken[chunk_buffer(chunk)], chunk_phase(chunk - 2))) break;
            fence_proxy_async_smem();
            if (elect_one()) {
                tc_fence_after();
                const uint64_t da = smem_desc(ring + slot * S::kStage, 0), db = smem_desc(ring + slot * S::kStage + S::kLeft, 0);
                const int steps = min(4, (a.H - (first1 + i) * 64 + 15) / 16);
                for (int k = 0; k < steps; ++k) tc_mma<1>(tmem + chunk_buffer(chunk) * 64 * RB, da + 2 * k, db + 2 * k, id1, !chunk_begins(i) || k > 0);
                tc_commit<1>(smem_u32(&s_done[slot]));
            }
            __syncwarp();
        }
    } else {
        for (int i = 0; i < kRing - 1 && i < stages1; ++i) fill_first(i, i);
        if (a.copy && s_status == 0) copy_rows(a);           // while they are on their way
        for (int i = 0; i < stages1; ++i) {
            if (i > 0 && !wait(s_done[ring_slot(i - 1)], ring_phase(i - 1))) break;      // the products of stage i - 1 have read its slot
            if (i + kRing - 1 < stages1) fill_first(i + kRing - 1, ring_slot(i + kRing - 1));
            if (i > 0 && chunk_begins(i)) take(stage_chunk(i - 1));
        }
        if (stages1 > 0 && wait(s_done[ring_slot(stages1 - 1)], ring_phase(stages1 - 1))) take(stage_chunk(stages1 - 1));
    }
    __syncthreads();
    // ---- the cluster's sums, as 16-bit operand
    float *const mine = reinterpret_cast<float *>(smem) + row * S::kPitch;
#pragma unroll
    for (int b = 0; b < RB; ++b) {
        const int k0 = (half * RB + b) * 32;
        if (issuer || k0 >= n1) continue;
        const float(&v)[32] = total[b];
#pragma unroll
        for (int j = 0; j < 8; ++j) *reinterpret_cast<float4 *>(mine + k0 + 4 * j) = make_float4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
    }
    cluster_sync_all();                                      // (a barrier of the CTA where it is alone)
    if (ld_cluster_s32(at_rank(smem_u32(&s_status), 0))) {
        tc_fence_before();
        cluster_sync_all();                                  // (read everywhere)
        tc_fence_after();
        if (warp == 4) tmem_free<1>(tmem, kTmem);
        return;
    }
    // Every CTA adds up its share of the rows and hands them to all.  8 * RB lanes side by side read a row side by side (16-byte
    // reads of 32 different rows took 60,000 cycles for what takes a few thousand so), 8 columns each.
    const int share = (kTileRows + a.C - 1) / a.C, last = min(kTileRows, (rank + 1) * share);
    for (int i = tid; !issuer && rank * share + i / (8 * RB) < last; i += kThreads) {
        const int r = rank * share + i / (8 * RB), k = i % (8 * RB);
        const uint32_t from = smem_u32(reinterpret_cast<float *>(smem) + r * S::kPitch + 8 * k);
        float t[8] = {};
        if (8 * k < a.r)                                     // (an infinite x times the zeros behind A's rows is NaN)
            for (int o = 0; o < a.C; o += 4) {               // loads on their way together: each takes some 700 cycles
                float4 u[4][2];
#pragma unroll
                for (int h = 0; h < 8; ++h) u[h >> 1][h & 1] = ld_cluster_f32x4(at_rank(from + (h & 1) * 16, min(o + (h >> 1), a.C - 1)));
#pragma unroll
                for (int h = 0; h < 8; ++h)
                    if (o + (h >> 1) < a.C) {
                        const float4 v = u[h >> 1][h & 1];
                        float *const p = t + 4 * (h & 1);
                        p[0] += v.x;
                        p[1] += v.y;
                        p[2] += v.z;
                        p[3] += v.w;
                    }
            }
        float f = 1.0f;                                      // a power of two per row keeps the sums in fp16's range
        if (f16) {
            float most = 0.0f;
#pragma unroll
            for (int j = 0; j < 8; ++j) most = fmaxf(most, finite_abs(t[j]));
            const uint32_t mates = (RB == 1 ? 0xffu : 0xffffu) << (lane & ~(8 * RB - 1));
#pragma unroll
            for (int o = 4 * RB; o > 0; o >>= 1) most = fmaxf(most, __shfl_xor_sync(mates, most, o));
            f = fp16_scale(most);
        }
        uint32_t hi[4], lo[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) split2_whole<T>(t[2 * j] * f, t[2 * j + 1] * f, hi[j], lo[j]);
        const uint32_t to_op = low + (k >> 3) * kTileRows * 128 + swizzled(r, k & 7), to_f = smem_u32(s_scale + r);
        for (int o = 0; o < a.C; ++o) {
            st_cluster_x4(at_rank(to_op, o), hi);
            st_cluster_x4(at_rank(to_op + S::kLow, o), lo);
            if (k == 0) st_cluster(at_rank(to_f, o), __float_as_uint(f));
        }
    }
    fence_proxy_async_smem();
    tc_fence_before();
    cluster_sync_all();                                      // the operand is complete everywhere, and the ring has the sums' place again
    const float back = (a.scale ? a.scale[g] : 1.0f) / s_scale[row];
    // ---- out = y + B (A x): every CTA its stages of N
#pragma unroll
    for (int i = 0; i < 4; ++i) left[i] = a.y + (has[i] ? s_at[r0 + 32 * i] * a.ldy : 0) + 8 * piece;
    right = a.b + (size_t)g * a.N * a.r + 8 * piece;
    auto fill_second = [&](int i, int slot) {
        const int col = (first2 + i) * 64;
        if (col < a.N) {
            const uint32_t st = ring + slot * S::kStage + to;
            const bool in = col + 8 * piece < a.N;
#pragma unroll
            for (int j = 0; j < 4; ++j) cp_async16_or_zero(st + j * 4096, in ? left[j] + col : a.y, in && has[j]);
#pragma unroll
            for (int j = 0; j < 2; ++j)
#pragma unroll
                for (int b = 0; b < RB; ++b) {
                    const int n = col + r0 + 32 * j;
                    const bool valid = n < a.N && 64 * b + 8 * piece < a.r;
                    if (64 * b + 8 * piece < n1)
                        cp_async16_or_zero(st + S::kLeft + b * 8192 + j * 4096, valid ? right + (size_t)n * a.r + 64 * b : a.b, valid);
                }
        }
        cp_async_arrive(smem_u32(&s_full[slot]));
    };
    tc_fence_after();
    if (issuer) {
        const uint32_t id2 = mma_desc(f16, 128, 64, false, false);
        for (int i = 0; ok && i < stages2; ++i) {
            const int slot = ring_slot(i);
            if (!wait(s_full[slot], ring_phase(i, stages1))) break;
            // (twice 64 columns of sums: those of stage i - 2 have been read when its slot's successor is filled)
            if (i >= 2 && !wait(s_free[ring_slot(i - 2)], ring_phase(i - 2))) break;
            fence_proxy_async_smem();
            if (elect_one()) {
                tc_fence_after();
                const uint64_t da = smem_desc(low, 0), db = smem_desc(ring + slot * S::kStage + S::kLeft, 0);
                for (int k = 0; k < n1 / 16; ++k) {
                    const uint64_t ka = (k >> 2) * (kTileRows * 128 / 16) + 2 * (k & 3), kb = (k >> 2) * (8192 / 16) + 2 * (k & 3);
                    tc_mma<1>(tmem + (i & 1) * 64, da + S::kLow / 16 + ka, db + kb, id2, k > 0);
                    tc_mma<1>(tmem + (i & 1) * 64, da + ka, db + kb, id2, true);
                }
                tc_commit<1>(smem_u32(&s_done[slot]));
            }
            __syncwarp();
        }
    } else {
        for (int i = 0; ok && i < kRing - 1 && i < stages2; ++i) fill_second(i, i);
        for (int i = 0; ok && i < stages2; ++i) {
            const int slot = ring_slot(i), col = (first2 + i) * 64;
            if (i > 0 && !wait(s_free[ring_slot(i - 1)], ring_phase(i - 1))) break;      // every warp has written stage i - 1
            if (i + kRing - 1 < stages2) fill_second(i + kRing - 1, ring_slot(i + kRing - 1));
            if (!wait(s_full[slot], ring_phase(i, stages1)) || !wait(s_done[slot], ring_phase(i, stages1))) break;
            __syncwarp();
            tc_fence_after();
            uint8_t *const st = smem + slot * S::kStage;
            float v[32];
            tmem_ld32(lanes + (i & 1) * 64 + half * 32, v);
            tmem_wait_ld();
            tc_fence_before();
            bool odd = false;
#pragma unroll
            for (int j = 0; j < 32; j += 8) odd |= not_finite(v[j], v[j + 1], v[j + 2], v[j + 3], v[j + 4], v[j + 5], v[j + 6], v[j + 7]);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                uint4 *const p = reinterpret_cast<uint4 *>(st + swizzled(row, half * 4 + j));
                const uint4 y = *p;
                const uint32_t w[4] = {y.x, y.y, y.z, y.w};
                uint32_t o[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const float2 yv = word_to_f32(w[k], T());
                    o[k] = f32_to_word(fmaf(back, v[8 * j + 2 * k], yv.x), fmaf(back, v[8 * j + 2 * k + 1], yv.y), T());
                }
                *p = make_uint4(o[0], o[1], o[2], o[3]);
            }
            if (odd) {                                       // nearly never: outputs that are NaN, from the parts of A x, B and y in memory
                const auto number = [&](uint32_t tile, int r, int k) {       // k of row r of an operand's blocks of 64 columns
                    return word_to_f32(*reinterpret_cast<const uint16_t *>(smem + tile + swizzled(r, k >> 3 & 7) + (k & 7) * 2), T()).x;
                };
                const int at = s_at[row];
#pragma unroll 1
                for (int n = half * 32; at >= 0 && n < half * 32 + 32 && col + n < a.N; ++n) {
                    uint16_t *const out = reinterpret_cast<uint16_t *>(st + swizzled(row, n >> 3) + (n & 7) * 2);
                    const float was = word_to_f32(*out, T()).x;
                    if (was == was) continue;
                    float sum = 0.0f;
#pragma unroll 1
                    for (int k = 0; k < a.r; ++k) {
                        const uint32_t t = kRing * S::kStage + (k >> 6) * kTileRows * 128;
                        sum = fmaf(number(t, row, k & 63) + number(t + S::kLow, row, k & 63),
                                   number(slot * S::kStage + S::kLeft + (k >> 6) * 8192, n, k & 63), sum);
                    }
                    *out = (uint16_t)f32_to_word(fmaf(back, sum, word_to_f32(a.y[at * a.ldy + col + n], T()).x), 0.0f, T());
                }
            }
            __syncwarp();
            // this warp's 32 rows and 32 columns, four lanes to a row
            const int n = col + half * 32 + (lane & 3) * 8;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int r = q * 32 + j * 8 + (lane >> 2), at = s_at[r];
                if (at >= 0 && n < a.N) *reinterpret_cast<uint4 *>(a.out + at * a.ldo + n) = *reinterpret_cast<const uint4 *>(st + swizzled(r, half * 4 + (lane & 3)));
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(at_rank(smem_u32(&s_free[slot]), cluster_rank()));
        }
    }
    if (!ok) {                                               // copies and products that are still on their way get the time to arrive
        atomicOr(const_cast<int32_t *>(a.status), EP_STATUS_TIMEOUT);
        asm volatile("cp.async.wait_all;" ::: "memory");
        const unsigned long long t = global_ns();
        while (global_ns() - t < 1000000ull) {}
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 4) tmem_free<1>(tmem, kTmem);
}

template <auto kern> int launch_lora(const LoraArgs &a, int threads, size_t smem, cudaStream_t st) {
    const int rc = allow_smem<kern>(smem);
    if (rc != EP_OK) return rc;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((a.tiles + a.heads) * a.C));
    cfg.blockDim = dim3(threads);
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

template <typename T> int launch_type(const LoraArgs &a, cudaStream_t st) {
    if (a.rows == kTileRows)
        return a.r <= 64 ? launch_lora<ep_lora_tile_kernel<T, 1>>(a, kTileThreads, TileSmem<1>::kBytes, st)
                         : launch_lora<ep_lora_tile_kernel<T, 2>>(a, kTileThreads, TileSmem<2>::kBytes, st);
    const auto smem = [](int RN) { return (size_t)(kWarps + 2) * 16 * 8 * RN * sizeof(float); };
    if (a.r <= 16) return launch_lora<ep_lora_kernel<T, 2>>(a, kThreads, smem(2), st);
    if (a.r <= 32) return launch_lora<ep_lora_kernel<T, 4>>(a, kThreads, smem(4), st);
    return a.r <= 64 ? launch_lora<ep_lora_kernel<T, 8>>(a, kThreads, smem(8), st) : launch_lora<ep_lora_kernel<T, 16>>(a, kThreads, smem(16), st);
}

// Tiles of 128 rows begin slowly (19 us at least, of which their sums' way across the cluster is some) and then read A and B an
// eighth as often as tiles of 16 rows, whose time is about 3.2e-7 us per 16 rows, column of x or y, and (r + 25).  The border is at 50 us
// of that.  16 / 128 rows, every token with an adapter, in a CUDA graph: 1024 tokens, 4 adapters of rank 16, 4096 -> 4096: 8.2 / 21 us; 2048, 16 of rank 64, 2048 -> 2048: 17 / 43;
// 8192, 1 of rank 16, 4096 -> 4096: 55 / 47; 4096, 32 of rank 128: 91 / 74; 8192, 5 of rank 64: 119 / 54; 16384, 8 of rank 16,
// 2048 -> 6144: 133 / 94.
bool takes_tiles(long long rows, int H, int N, int rank) { return rows * (H + N) * (rank + 25) >= 2500000000ll; }

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
    // a tile's rows: about as many as an adapter has; then as many CTAs to a tile as two to an SM allow
    const long long all = rows_max(L->T, L->K, L->fused_shared), per = all / p.G;
    const int sms = std::max(device_sm_count(), 1);
    p.rows = 1;
    while (p.rows < 16 && p.rows < per) p.rows *= 2;
    if (per >= kTileRows && takes_tiles(all, H, N, rank)) p.rows = kTileRows;
    p.tiles = (p.R_max + p.rows - 1) / p.rows;
    p.heads = p.rows > 1 ? p.G : 0;
    const long long groups = (long long)p.tiles + p.heads, stages = (std::max(H, N) + 63) / 64;
    p.C = (int)std::max(1ll, std::min({(long long)kMaxCluster, 2 * sms / groups, p.rows == kTileRows ? stages : (stages + 3) / 4}));
    p.copy = by_token && out != y;
    cudaStream_t st = as_stream(stream);
    return dtype == EP_F16 ? launch_type<__half>(p, st) : launch_type<__nv_bfloat16>(p, st);
}
