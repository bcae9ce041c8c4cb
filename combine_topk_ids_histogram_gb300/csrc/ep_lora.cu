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
#include <stddef.h>

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
    int tiles, heads, C;                 // tiles of rows; adapters' first rows apart (0 or G); CTAs on each
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

__device__ __forceinline__ float4 ld_cluster_f32x4(uint32_t addr) {
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(addr) : "memory");
    return v;
}

// The power of two that brings a largest magnitude to [2^14, 2^15), in fp16's range: from its exponent (1 for 0, infinities and NaN).
__device__ __forceinline__ float fp16_scale(float most) {
    const int e = (int)(__float_as_uint(most) >> 23) - 127;
    return most > 0.0f && e < 128 ? __uint_as_float((uint32_t)(min(14 - e, 126) + 127) << 23) : 1.0f;
}

// A sum v of A x as two 16-bit numbers, hi + lo: their products with B are exact in fp32, and v keeps 16 bits (bf16) or 22 (fp16).
template <typename T> __device__ __forceinline__ void split2(float v0, float v1, uint32_t &hi, uint32_t &lo) {
    hi = f32_to_word(v0, v1, T());
    const float2 h = word_to_f32(hi, T());
    lo = f32_to_word(v0 - h.x, v1 - h.y, T());
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
                bounds_fail(a.status);
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

// Rows without an adapter, to another buffer.
__device__ void copy_rows(const LoraArgs &a, int cta, int ctas) {
    for (int t = cta * kWarps + (threadIdx.x >> 5); t < a.T; t += ctas * kWarps) {
        const int row = a.row_of[t];
        if (row >= 0 && row < a.R_max) continue;
        for (int n = (threadIdx.x & 31) * 8; n < a.N; n += 256)
            *reinterpret_cast<uint4 *>(a.out + t * a.ldo + n) = *reinterpret_cast<const uint4 *>(a.y + t * a.ldy + n);
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
    const bool copies = tile >= a.tiles + a.heads;
    const Rows rows(a, copies ? 0 : tile);
    if constexpr (kBoundsCheck) {                            // another CTA may set a bit meanwhile: the cluster acts on one reading
        __shared__ int s_status;
        if (tid == 0) s_status = load_status(a.status);
        cluster_sync_all();
        int st;
        asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(st) : "r"(at_rank(smem_u32(&s_status), 0)) : "memory");
        cluster_sync_all();
        if (st) return;
    } else if (load_status(a.status)) {
        return;
    }
    if (copies) {
        copy_rows(a, blockIdx.x - (a.tiles + a.heads) * a.C, gridDim.x - (a.tiles + a.heads) * a.C);
        return;
    }
    if (rows.end <= rows.first) return;
    const int g = rows.g;
    int at[2];                                           // the row of x, y and out; -1: none
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int j = rows.first + c + 8 * i;
        at[i] = j < rows.end ? (a.by_token ? a.src_info[2 * (size_t)j] : j) : -1;
        if (a.by_token && at[i] >= a.T) {
            bounds_fail(a.status);
            at[i] = -1;
        }
    }
    Block<RN> ahead;
    if (kAhead) ahead.load(a, g, part * 32, at, c, q);
    float acc[RN][4] = {};
    const uint4 zero = make_uint4(0, 0, 0, 0);
    for (int k0 = part * kSteps * 32; k0 < a.H; k0 += parts * kSteps * 32) {
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
#pragma unroll
    for (int j = 0; j < RN; ++j) {
        float *const p = s_part + warp * kCells + c * kR + 8 * j + 2 * q;
        *reinterpret_cast<float2 *>(p) = make_float2(acc[j][0], acc[j][1]);
        *reinterpret_cast<float2 *>(p + 8 * kR) = make_float2(acc[j][2], acc[j][3]);
    }
    __syncthreads();
    for (int i = tid; i < kCells; i += kThreads) {
        float v = 0.0f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) v += s_part[w * kCells + i];
        s_mine[i] = v;
    }
    if (a.C > 1) {
        cluster_sync_all();
        for (int i = tid; i < kCells; i += kThreads) {
            float v = 0.0f;
            for (int k = 0; k < a.C; ++k) v += ld_cluster_f32(at_rank(smem_u32(s_mine + i), k));
            s_all[i] = v;
        }
    }
    __syncthreads();
    if constexpr (std::is_same_v<T, __half>) {           // a power of two per row keeps the sums in fp16's range
        for (int i = warp; i < kRows; i += kWarps) {
            float v = 0.0f;
            for (int k = lane; k < kR; k += 32) v = fmaxf(v, fabsf(s_all[i * kR + k]));
            v = warp_max(v);
            if (lane == 0) s_scale[i] = fp16_scale(v);
        }
        __syncthreads();
    }
    constexpr int kK = RN / 2;                       // steps of 16 of the second product
    uint32_t hi[kK][4], lo[kK][4];
    float back[2];                                   // adapter's scale, over the row's
    const float scale = a.scale ? a.scale[g] : 1.0f;
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
    for (int n0 = part * 32; n0 < a.N; n0 += parts * 32) {
        Block<RN> now;
        if (kAhead && n0 == part * 32) now = ahead;
        else now.load(a, g, n0, at, c, q);
        float sum[4][4] = {};
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int s = 0; s < kK; ++s) {
                mma16<T>(sum[j], lo[s][0], lo[s][1], lo[s][2], lo[s][3], now.b[j][2 * s], now.b[j][2 * s + 1]);
                mma16<T>(sum[j], hi[s][0], hi[s][1], hi[s][2], hi[s][3], now.b[j][2 * s], now.b[j][2 * s + 1]);
            }
        const int n = n0 + 8 * q;
        if (n >= a.N) continue;
#pragma unroll
        for (int i = 0; i < 2; ++i)
            if (at[i] >= 0) {
                const uint32_t w[4] = {now.y[i].x, now.y[i].y, now.y[i].z, now.y[i].w};
                uint32_t o[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float2 v = word_to_f32(w[j], T());
                    o[j] = f32_to_word(fmaf(back[i], sum[j][2 * i], v.x), fmaf(back[i], sum[j][2 * i + 1], v.y), T());
                }
                *reinterpret_cast<uint4 *>(a.out + at[i] * a.ldo + n) = make_uint4(o[0], o[1], o[2], o[3]);
            }
    }
    if (a.C > 1) cluster_sync_all();                         // the sums have been read everywhere
}

// ------------------------------------------------------------------------------------------------------------ many rows
// The same for tiles of 64 rows, where the bytes of x, y and out are what counts: both products stream through a ring in shared
// memory that cp.async fills ahead of them, 64 columns of x with 64 of A, then 64 of y with 64 rows of B, and four warps'
// 16 rows share each of them.
constexpr int kTileRows = 64;
constexpr int ring_stages(int RN) { return RN == 16 ? 4 : RN == 8 ? 6 : 8; }     // in up to 96 KB, for two CTAs to an SM

__device__ __forceinline__ void cp_async16_or_zero(uint32_t smem, const void *gmem, bool valid) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem), "l"(gmem), "r"(valid ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N> __device__ __forceinline__ void cp_async_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

// Rows of `pitch` 16-byte pieces.  A quarter of a warp reads four pieces of two neighbouring rows: with 8 pieces or more to a row the
// odd ones are exchanged in fours, so that the two do not meet in the same banks.
template <int PITCH> __device__ __forceinline__ int piece_at(int row, int piece) {
    return row * PITCH + (PITCH >= 8 ? piece ^ ((row & 1) << 2) : piece);
}

template <int RN> struct Ring {
    static constexpr int kRank = 8 * RN;                     // rows of A, and columns of B
    uint4 left[kTileRows * 8];                               // 64 rows x 64 columns of x, then of y
    uint4 right[kRank * 8];                                  // rank x 64 columns of A, then 64 rows x rank of B
};

template <typename T, int RN>
__global__ void __launch_bounds__(kThreads, 2) ep_lora_rows_kernel(const LoraArgs a, int one_wave) {
    constexpr int kR = 8 * RN, kK = RN / 2, kRing = RN == 16 ? 4 : RN == 8 ? 6 : 8;
    // Sums of A x: two warps' parts, in rows that begin 8 banks apart, then all of them in the second's place, 2 banks apart, which is
    // what their writers and readers meet least in.  They lie in the ring's first kHeld slots.
    constexpr int kPitch = kR + 8, kPart = kTileRows * kPitch, kPitchAll = kR + 2;
    constexpr int kHeld = (2 * kPart * (int)sizeof(float) + (int)sizeof(Ring<RN>) - 1) / (int)sizeof(Ring<RN>);
    static_assert(kHeld < kRing, "room for the sums");
    extern __shared__ __align__(16) uint8_t s_raw[];
    Ring<RN> *const ring = reinterpret_cast<Ring<RN> *>(s_raw);
    float *const s_part = reinterpret_cast<float *>(s_raw), *const s_all = s_part + kPart;
    __shared__ float s_scale[kTileRows];
    __shared__ int s_at[kTileRows];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, c = lane >> 2, q = lane & 3, rg = warp & 3, split = warp >> 2;
    pdl_begin_if(one_wave);
    const int tile = blockIdx.x / a.C, rank = blockIdx.x % a.C;
    const bool copies = tile >= a.tiles + a.heads;
    const Rows rows(a, copies ? 0 : tile);
    if constexpr (kBoundsCheck) {
        __shared__ int s_status;
        if (tid == 0) s_status = load_status(a.status);
        cluster_sync_all();
        int st;
        asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(st) : "r"(at_rank(smem_u32(&s_status), 0)) : "memory");
        cluster_sync_all();
        if (st) return;
    } else if (load_status(a.status)) {
        return;
    }
    if (copies) {
        copy_rows(a, blockIdx.x - (a.tiles + a.heads) * a.C, gridDim.x - (a.tiles + a.heads) * a.C);
        return;
    }
    if (rows.end <= rows.first) return;
    const int g = rows.g;
    if (tid < kTileRows) {
        const int row = rows.first + tid;
        int at = row < rows.end ? (a.by_token ? a.src_info[2 * (size_t)row] : row) : -1;
        if (a.by_token && at >= a.T) {
            bounds_fail(a.status);
            at = -1;
        }
        s_at[tid] = at;
    }
    __syncthreads();
    const bool busy = rows.first + 16 * rg < rows.end;
    // What this thread copies: a 16-byte piece of rows tid / 8 and 32 + tid / 8 of x or y, and of kMine rows of A or B.
    constexpr int kMine = RN >= 4 ? RN / 4 : 1;
    const bool right = RN >= 4 || tid < 128;
    const int piece = tid & 7, at0 = s_at[tid >> 3], at1 = s_at[32 + (tid >> 3)];
    const uint32_t base = smem_u32(s_raw), to0 = base + piece_at<8>(tid >> 3, piece) * 16, to1 = to0 + 32 * 8 * 16;
    auto fill = [&](int slot, int col, int cols, const uint16_t *p0, const uint16_t *p1, const uint16_t *const (&pr)[kMine], size_t step,
                    const uint32_t (&tor)[kMine], const bool (&okr)[kMine]) {
        if (col < cols) {
            const uint32_t st = slot * (uint32_t)sizeof(Ring<RN>);
            const bool in = col + 8 * piece < cols;
            cp_async16_or_zero(to0 + st, in ? p0 + col : a.x, in && at0 >= 0);
            cp_async16_or_zero(to1 + st, in ? p1 + col : a.x, in && at1 >= 0);
#pragma unroll
            for (int j = 0; j < kMine; ++j)
                if (right) cp_async16_or_zero(tor[j] + st, okr[j] ? pr[j] + col * step : a.a, okr[j]);
        }
        cp_async_commit();
    };
    float acc[RN][4] = {};
    const uint16_t *p0 = a.x + (at0 >= 0 ? at0 * a.ldx : 0) + 8 * piece, *p1 = a.x + (at1 >= 0 ? at1 * a.ldx : 0) + 8 * piece, *pr[kMine];
    uint32_t tor[kMine];
    bool okr[kMine];
#pragma unroll
    for (int j = 0; j < kMine; ++j) {
        const int r = 32 * j + (tid >> 3);
        okr[j] = r < a.r;
        pr[j] = a.a + ((size_t)g * a.r + (okr[j] ? r : 0)) * a.H + 8 * piece;
        tor[j] = base + (uint32_t)(offsetof(Ring<RN>, right) + piece_at<8>(r, piece) * 16);
    }
    auto fill_first = [&](int i, int slot) {                 // stage i of this CTA
        const int col = (rank + i * a.C) * 64;
        const bool in = col + 8 * piece < a.H;
        bool ok[kMine];
#pragma unroll
        for (int j = 0; j < kMine; ++j) ok[j] = okr[j] && in;
        fill(slot, col, a.H, p0, p1, pr, 1, tor, ok);
    };
    for (int i = 0; i < kRing - 1; ++i) fill_first(i, i);
    int now = 0, then = kRing - 1;                           // the slot in use, and the one to fill
    for (int i = 0; (rank + i * a.C) * 64 < a.H; ++i, now = now == kRing - 1 ? 0 : now + 1, then = then == kRing - 1 ? 0 : then + 1) {
        cp_async_wait<kRing - 2>();
        __syncthreads();
        fill_first(i + kRing - 1, then);
        if (!busy) continue;
        const Ring<RN> &st = ring[now];
        const uint4 x0 = st.left[piece_at<8>(16 * rg + c, 4 * split + q)], x1 = st.left[piece_at<8>(16 * rg + c + 8, 4 * split + q)];
#pragma unroll
        for (int j = 0; j < RN; ++j) {
            const uint4 w = st.right[piece_at<8>(8 * j + c, 4 * split + q)];
            mma16<T>(acc[j], x0.x, x1.x, x0.y, x1.y, w.x, w.y);
            mma16<T>(acc[j], x0.z, x1.z, x0.w, x1.w, w.z, w.w);
        }
    }
    cp_async_wait<0>();
    __syncthreads();
    p0 = a.y + (at0 >= 0 ? at0 * a.ldy : 0) + 8 * piece;
    p1 = a.y + (at1 >= 0 ? at1 * a.ldy : 0) + 8 * piece;
    int rows_b[kMine];
#pragma unroll
    for (int j = 0; j < kMine; ++j) {
        const int p = j * kThreads + tid, n = p / RN, k = p % RN;
        rows_b[j] = n;
        okr[j] = 8 * k < a.r;
        pr[j] = a.b + ((size_t)g * a.N + n) * a.r + (okr[j] ? 8 * k : 0);
        tor[j] = base + (uint32_t)(offsetof(Ring<RN>, right) + piece_at<RN>(n, k) * 16);
    }
    auto fill_second = [&](int i, int slot) {
        const int col = (rank + i * a.C) * 64;
        bool ok[kMine];
#pragma unroll
        for (int j = 0; j < kMine; ++j) ok[j] = okr[j] && col + rows_b[j] < a.N;
        fill(slot, col, a.N, p0, p1, pr, a.r, tor, ok);
    };
    for (int i = 0; i < kRing - kHeld; ++i) fill_second(i, kHeld + i);          // what the sums leave room for comes meanwhile
#pragma unroll
    for (int j = 0; j < RN; ++j) {
        float *const p = s_part + split * kPart + (16 * rg + c) * kPitch + 8 * j + 2 * q;
        *reinterpret_cast<float2 *>(p) = make_float2(acc[j][0], acc[j][1]);
        *reinterpret_cast<float2 *>(p + 8 * kPitch) = make_float2(acc[j][2], acc[j][3]);
    }
    __syncthreads();
    for (int i = tid; i < kTileRows * kR / 4; i += kThreads) {
        float4 *const p = reinterpret_cast<float4 *>(s_part + i / (kR / 4) * kPitch + i % (kR / 4) * 4);
        const float4 u = p[0], v = p[kPart / 4];
        p[0] = make_float4(u.x + v.x, u.y + v.y, u.z + v.z, u.w + v.w);
    }
    cluster_sync_all();                                      // (a barrier of the CTA where it is alone)
    for (int i = tid; i < kTileRows * kR / 4; i += kThreads) {
        const int r = i / (kR / 4), k4 = i % (kR / 4) * 4;
        const uint32_t at = smem_u32(s_part + r * kPitch + k4);
        float4 v = ld_cluster_f32x4(at_rank(at, 0));
        for (int k = 1; k < a.C; ++k) {
            const float4 u = ld_cluster_f32x4(at_rank(at, k));
            v = make_float4(v.x + u.x, v.y + u.y, v.z + u.z, v.w + u.w);
        }
        float2 *const to = reinterpret_cast<float2 *>(s_all + r * kPitchAll + k4);
        to[0] = make_float2(v.x, v.y);
        to[1] = make_float2(v.z, v.w);
        if constexpr (std::is_same_v<T, __half>) {           // kR / 4 lanes hold a row
            float m = fmaxf(fmaxf(fabsf(v.x), fabsf(v.y)), fmaxf(fabsf(v.z), fabsf(v.w)));
#pragma unroll
            for (int o = kR / 8; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(kFullMask, m, o));
            if (k4 == 0) s_scale[r] = fp16_scale(m);
        }
    }
    __syncthreads();
    uint32_t hi[kK][4], lo[kK][4];
    float back[2];                                           // adapter's scale, over the row's
    int at[2];
    const float scale = a.scale ? a.scale[g] : 1.0f;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int j = 16 * rg + c + 8 * i;
        at[i] = s_at[j];
        float f = 1.0f;
        if constexpr (std::is_same_v<T, __half>) f = s_scale[j];
        back[i] = scale / f;
#pragma unroll
        for (int s = 0; s < kK; ++s)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int k = RN == 2 ? 4 * q + 2 * h : s / 2 * 32 + 8 * q + s % 2 * 4 + 2 * h;
                const float2 v = *reinterpret_cast<const float2 *>(s_all + j * kPitchAll + k);
                split2<T>(v.x * f, v.y * f, hi[s][i + 2 * h], lo[s][i + 2 * h]);
            }
    }
    cluster_sync_all();                                      // the sums have been read everywhere: the ring has their place again
    for (int i = kRing - kHeld; i < kRing - 1; ++i) fill_second(i, i - (kRing - kHeld));
    now = kHeld;
    then = kHeld - 1;
    for (int i = 0; (rank + i * a.C) * 64 < a.N; ++i, now = now == kRing - 1 ? 0 : now + 1, then = then == kRing - 1 ? 0 : then + 1) {
        cp_async_wait<kRing - 2>();
        __syncthreads();
        fill_second(i + kRing - 1, then);
        const int n = (rank + i * a.C) * 64 + 32 * split + 8 * q;
        if (!busy || n - 8 * q >= a.N) continue;
        const Ring<RN> &st = ring[now];
        float sum[4][4] = {};
        const int nb = 32 * split + 8 * (c >> 1) + (c & 1);  // + 2j
        if constexpr (RN == 2) {
            uint2 w[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) w[j] = *(reinterpret_cast<const uint2 *>(st.right + (nb + 2 * j) * 2) + q);
#pragma unroll
            for (int j = 0; j < 4; ++j) mma16<T>(sum[j], lo[0][0], lo[0][1], lo[0][2], lo[0][3], w[j].x, w[j].y);
#pragma unroll
            for (int j = 0; j < 4; ++j) mma16<T>(sum[j], hi[0][0], hi[0][1], hi[0][2], hi[0][3], w[j].x, w[j].y);
        } else {
#pragma unroll
            for (int s = 0; s < RN / 4; ++s) {               // four sums side by side: each product waits for the one before in its sum
                uint4 w[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) w[j] = st.right[piece_at<RN>(nb + 2 * j, 4 * s + q)];
#pragma unroll
                for (int h = 0; h < 4; ++h) {
                    const uint32_t *const f = h & 1 ? hi[2 * s + (h >> 1)] : lo[2 * s + (h >> 1)];
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        mma16<T>(sum[j], f[0], f[1], f[2], f[3], h < 2 ? w[j].x : w[j].z, h < 2 ? w[j].y : w[j].w);
                }
            }
        }
        if (n >= a.N) continue;
#pragma unroll
        for (int i2 = 0; i2 < 2; ++i2)
            if (at[i2] >= 0) {
                const uint4 y = st.left[piece_at<8>(16 * rg + c + 8 * i2, 4 * split + q)];
                const uint32_t w[4] = {y.x, y.y, y.z, y.w};
                uint32_t o[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float2 v = word_to_f32(w[j], T());
                    o[j] = f32_to_word(fmaf(back[i2], sum[j][2 * i2], v.x), fmaf(back[i2], sum[j][2 * i2 + 1], v.y), T());
                }
                *reinterpret_cast<uint4 *>(a.out + at[i2] * a.ldo + n) = make_uint4(o[0], o[1], o[2], o[3]);
            }
    }
}

template <auto kern> int launch_lora(const LoraArgs &a, size_t smem, int copy, cudaStream_t st) {
    const int rc = allow_smem<kern>(smem);
    if (rc != EP_OK) return rc;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((a.tiles + a.heads) * a.C + copy));
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

template <typename T, int RN> int launch_rank(const LoraArgs &a, int copy, cudaStream_t st) {
    if (a.rows == kTileRows) return launch_lora<ep_lora_rows_kernel<T, RN>>(a, sizeof(Ring<RN>) * ring_stages(RN), copy, st);
    return launch_lora<ep_lora_kernel<T, RN>>(a, (size_t)(kWarps + 2) * 16 * 8 * RN * sizeof(float), copy, st);
}
template <typename T> int launch_type(const LoraArgs &a, int copy, cudaStream_t st) {
    if (a.r <= 16) return launch_rank<T, 2>(a, copy, st);
    if (a.r <= 32) return launch_rank<T, 4>(a, copy, st);
    return a.r <= 64 ? launch_rank<T, 8>(a, copy, st) : launch_rank<T, 16>(a, copy, st);
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
    // a tile's rows: about as many as an adapter has; then as many CTAs to a tile as two to an SM allow
    const long long per = (long long)L->T * L->K / p.G;
    const int sms = std::max(device_sm_count(), 1);
    p.rows = 1;
    while (p.rows < 16 && p.rows < per) p.rows *= 2;
    if (per >= kTileRows) p.rows = kTileRows;
    p.tiles = (p.R_max + p.rows - 1) / p.rows;
    p.heads = p.rows > 1 ? p.G : 0;
    p.C = 1;
    while (p.C < kMaxCluster && ((long long)p.tiles + p.heads) * p.C * 2 <= 2 * sms && p.C * kWarps * 32 < std::max(H, N)) p.C *= 2;
    int copy = by_token && out != y ? std::min((L->T + kWarps - 1) / kWarps, 2 * sms) : 0;
    copy = (copy + p.C - 1) / p.C * p.C;
    cudaStream_t st = as_stream(stream);
    return dtype == EP_F16 ? launch_type<__half>(p, copy, st) : launch_type<__nv_bfloat16>(p, copy, st);
}
