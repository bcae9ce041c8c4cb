// ep_experts.cu -- products of the experts' 4-bit weights with the rows of a dispatch layout, for
// batches of few tokens (decode), optionally with the gated activation silu(gate) * up.
//
//   out[r, n] = row_scale[n] * sum over k of E2M1(code[n, k]) * E4M3(scale[n, k/16]) * x[r, k]
//
// Weights are in the format the NVFP4 dispatch writes.  A group's weights are read from HBM once for
// all of its rows, so HBM bounds the call while an expert has few rows: 9/16 byte per weight.  16 tokens, top-8 of 256 and a
// shared expert, 7168 -> 2 x 2048 gated: 268 us, 0.80 of the measured copy bandwidth (0.94 while all SMs work); 1 token, top-8 of
// 128, 2048 -> 2 x 768: 6.4 us.  From about 16 rows per expert on the conversion and the products bound it: 64 tokens, top-2 of
// 8, 14336 -> 4096: 102 us.
//
// The products run on mma.sync.m16n8k16 with weight rows as M and layout rows as N: at 8 rows
// or fewer per expert the tensor cores are far from their rate, and operands that a thread builds in
// its own registers need no pass through shared memory, which would carry four times the
// weights' bytes.  An E2M1 value times an E4M3 scale has 6 significant bits and lies in
// [2^-10, 2688], so it is exact in fp16; a row of x is scaled by the power of two that puts its
// largest magnitude in [2^14, 2^15), where a bf16 is exact in fp16 too unless it is below 2^-32 of
// that magnitude.  The contraction may take its k in any order as long as both operands take the same
// one: a thread reads 64 consecutive codes of a weight row (32 bytes) and feeds them to 16 steps of the
// tensor cores, and a first kernel writes x as fp16 in that order.
#include <math.h>

#include <algorithm>

#include "ep_host.h"
#include "ep_types.cuh"

namespace ep {
namespace {

constexpr int kStepK = 256;              // k per warp step: 64 per thread of a quad
constexpr int kPackThreads = 1024;       // at most; a thread takes 8 values at a time

struct ExpertArgs {
    const uint16_t *x;
    const uint8_t *codes, *scales;
    const float *row_scale;
    int H, N, by_token, swiglu, T, G, R_max;
    int KS;                              // warps that share a tile and split its k: 1, 2 or 4
    const int32_t *row_offsets, *expert_ids, *src_info, *status;
    uint4 *xw;                           // [R_max][step][word][quad thread] x as fp16, 16-byte pieces
    uint32_t *xs;                        // [R_max] what a row's sums are multiplied by: two powers of two as bf16
    int draw;                            // CTAs draw their items; needs two steps or more of every warp in an item
    unsigned *drawn;                     // items drawn beyond the first two of every CTA
    uint16_t *out;
};

__device__ __forceinline__ void cp_async4(void *smem, const void *gmem) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"((unsigned)__cvta_generic_to_shared(smem)), "l"(gmem) : "memory");
}

inline int pack_steps(int H) { return (H + kStepK - 1) / kStepK; }

__device__ __forceinline__ void cp_async16(void *smem, const void *gmem) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"((unsigned)__cvta_generic_to_shared(smem)), "l"(gmem) : "memory");
}

// Eight codes of a word to four fp16 pairs (consecutive codes), times the scale of their block.
__device__ __forceinline__ void codes_to_f16(uint32_t w, uint32_t scale2, uint32_t (&o)[4]) {
    asm("{.reg .b8 b0, b1, b2, b3;\n"
        " mov.b32 {b0, b1, b2, b3}, %4;\n"
        " cvt.rn.f16x2.e2m1x2 %0, b0;\n"
        " cvt.rn.f16x2.e2m1x2 %1, b1;\n"
        " cvt.rn.f16x2.e2m1x2 %2, b2;\n"
        " cvt.rn.f16x2.e2m1x2 %3, b3;}"
        : "=r"(o[0]), "=r"(o[1]), "=r"(o[2]), "=r"(o[3])
        : "r"(w));
#pragma unroll
    for (int i = 0; i < 4; ++i) asm("mul.rn.f16x2 %0, %0, %1;" : "+r"(o[i]) : "r"(scale2));
}

// Four E4M3 scales to fp16.
__device__ __forceinline__ void scales_to_f16(uint32_t w, uint32_t (&s)[2]) {
    asm("{.reg .b16 h0, h1;\n mov.b32 {h0, h1}, %2;\n cvt.rn.f16x2.e4m3x2 %0, h0;\n cvt.rn.f16x2.e4m3x2 %1, h1;}"
        : "=r"(s[0]), "=r"(s[1])
        : "r"(w));
}
// Scale i of them in both halves of a word.
__device__ __forceinline__ uint32_t scale_pair(const uint32_t (&s)[2], int i) {
    return __byte_perm(s[i >> 1], 0, i & 1 ? 0x3232 : 0x1010);
}

__device__ __forceinline__ void mma_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
                 "{%0, %1, %2, %3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// What a thread holds of one step: for each of its 2 * MT weight rows 64 consecutive codes and their scales.  ALIGN is the
// number of bytes that every weight row begins on a multiple of: 32, 16 or 8.
template <int MT, int ALIGN> struct Weights {
    uint32_t w[2 * MT][8];
    uint32_t s[2 * MT][ALIGN == 32 ? 1 : 2];
    uint32_t at;                         // ALIGN 8: bits 2r, 2r + 1: the byte of s[r] that is the first scale; from bit 8: a mask's shift
};

// k of word wi (8 codes) of quad thread q within a step.
__device__ __forceinline__ int word_k(int q, int wi) { return q * 64 + wi * 8; }

template <int ALIGN, int MT>
__device__ __forceinline__ void load_weights(Weights<MT, ALIGN> &d, const uint8_t *codes, const uint8_t *scales,
                                             const uint8_t *scales_end, const unsigned (&row)[2 * MT], int step, int q, int H) {
    const int k = step * kStepK + q * 64;
#pragma unroll
    for (int r = 0; r < 2 * MT; ++r) {
#pragma unroll
        for (int i = 0; i < 8; ++i) d.w[r][i] = 0u;
        d.s[r][0] = 0u;
        if constexpr (ALIGN != 32) d.s[r][1] = 0u;
    }
    if constexpr (ALIGN == 8) d.at = 0u;
    if (k >= H) return;
    if constexpr (ALIGN == 8) d.at = (unsigned)max(0, 64 - (H - k)) << 7;   // 8 * scales past the row's end, at bit 8
#pragma unroll
    for (int r = 0; r < 2 * MT; ++r) {
        const unsigned long long at = (unsigned long long)row[r] * ((unsigned)H >> 1) + (unsigned)(k >> 1);
        const uint8_t *c = codes + at, *s = scales + (at >> 3);
        if constexpr (ALIGN == 32) {
            asm volatile("ld.global.nc.L1::no_allocate.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                         : "=r"(d.w[r][0]), "=r"(d.w[r][1]), "=r"(d.w[r][2]), "=r"(d.w[r][3]), "=r"(d.w[r][4]),
                           "=r"(d.w[r][5]), "=r"(d.w[r][6]), "=r"(d.w[r][7])
                         : "l"(c));
            d.s[r][0] = __ldg(reinterpret_cast<const uint32_t *>(s));
        } else if constexpr (ALIGN == 16) {
#pragma unroll
            for (int j = 0; j < 2; ++j)
                if (k + 32 * j < H) {
                    const uint4 v = __ldg(reinterpret_cast<const uint4 *>(c + 16 * j));
                    d.w[r][4 * j] = v.x; d.w[r][4 * j + 1] = v.y; d.w[r][4 * j + 2] = v.z; d.w[r][4 * j + 3] = v.w;
                    d.s[r][j] = __ldg(reinterpret_cast<const uint16_t *>(s + 2 * j));
                }
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (k + 16 * j < H) {
                    const uint2 v = __ldg(reinterpret_cast<const uint2 *>(c + 8 * j));
                    d.w[r][2 * j] = v.x; d.w[r][2 * j + 1] = v.y;
                }
            // the scales begin at any byte: the two aligned words around them, bytes where the scales' own end cuts one off
            const unsigned off = (unsigned)(at >> 3) & 3u;
            d.at |= off << (2 * r);
            s -= off;
            if (s + 8 <= scales_end) {
                d.s[r][0] = __ldg(reinterpret_cast<const uint32_t *>(s));
                d.s[r][1] = __ldg(reinterpret_cast<const uint32_t *>(s + 4));
            } else {
                for (int i = 0; i < 8; ++i)
                    if (s + i < scales_end) d.s[r][i >> 2] |= (uint32_t)s[i] << (8 * (i & 3));
            }
        }
    }
}

// The four scales of row r, one per byte; zero past the row's end.
template <int ALIGN, int MT> __device__ __forceinline__ uint32_t row_scales(const Weights<MT, ALIGN> &d, int r) {
    if constexpr (ALIGN == 32) return d.s[r][0];
    else if constexpr (ALIGN == 16) return __byte_perm(d.s[r][0], d.s[r][1], 0x5410);
    else return __funnelshift_r(d.s[r][0], d.s[r][1], 8 * (d.at >> (2 * r) & 3u)) & (~0u >> (d.at >> 8));
}

// One step of a warp: MT * 16 weight rows x 256 k x the first USE of NT blocks of 8 layout rows.  x: the step's pieces of this thread's
// layout row in shared memory, xo: how far on its row of the second block of 8 is.
template <int USE, int ALIGN, int MT, int NT>
__device__ __forceinline__ void mma_step(const Weights<MT, ALIGN> &d, const uint4 *x, const int (&xo)[NT],
                                         float (&acc)[MT][NT][4]) {
    uint32_t sc[2 * MT][2];
#pragma unroll
    for (int r = 0; r < 2 * MT; ++r) scales_to_f16(row_scales(d, r), sc[r]);
#pragma unroll
    for (int wi = 0; wi < 8; ++wi) {
        uint4 b[USE];
#pragma unroll
        for (int t = 0; t < USE; ++t) b[t] = x[xo[t] + wi * 4];
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
            uint32_t lo[4], hi[4];   // weight rows g and g + 8 of the tile
            codes_to_f16(d.w[2 * mt][wi], scale_pair(sc[2 * mt], wi >> 1), lo);
            codes_to_f16(d.w[2 * mt + 1][wi], scale_pair(sc[2 * mt + 1], wi >> 1), hi);
#pragma unroll
            for (int t = 0; t < USE; ++t) {
                mma_f16(acc[mt][t], lo[0], hi[0], lo[1], hi[1], b[t].x, b[t].y);
                mma_f16(acc[mt][t], lo[2], hi[2], lo[3], hi[3], b[t].z, b[t].w);
            }
        }
    }
}

// A row of x (null: no token) as fp16 in the order that the products take, and what its sums are multiplied by, as a pair
// of bf16: all threads of a CTA together.
__device__ __forceinline__ uint32_t pack_row(const uint4 *x, int H, uint4 *dst) {
    __shared__ unsigned s_top[kPackThreads / 32];
    const int tid = threadIdx.x;
    unsigned top = 0u;                                              // largest finite magnitude, as bf16 bits
    for (int p = tid; x && p < H / 8; p += blockDim.x) {
        const uint4 v = __ldg(x + p);
        const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const unsigned mag = u[i] & 0x7fff7fffu;
            top = __vmaxu2(top, mag & ~__vcmpgeu2(mag, 0x7f807f80u));
        }
    }
    top = __reduce_max_sync(kFullMask, max(top & 0xffffu, top >> 16));
    if ((tid & 31) == 0) s_top[tid >> 5] = top;
    __syncthreads();
    for (int w = 0; w < (int)blockDim.x / 32; ++w) top = max(top, s_top[w]);
    const int e = max((int)(top >> 7), 15);                         // biased exponent; both powers stay normal
    const float up = __uint_as_float((unsigned)(268 - e) << 23);    // 2^(141 - e)
    const int pieces = (H + kStepK - 1) / kStepK * 32;
    for (int p = tid; p < pieces; p += blockDim.x) {
        const int k = (p >> 5) * kStepK + word_k(p & 3, (p >> 2) & 7);
        uint4 v = make_uint4(0u, 0u, 0u, 0u);
        if (x && k < H) {
            float f[8];
            unpack8(__ldg(x + (k >> 3)), f);
            __half2 h[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) h[i] = __floats2half2_rn(f[2 * i] * up, f[2 * i + 1] * up);
            __builtin_memcpy(&v, h, 16);
        }
        dst[p] = v;
    }
    const unsigned both = (unsigned)(e - 14) + 127u, half = both >> 1;          // 2^(e - 141) in biased exponents, and halved
    return half << 23 | (both - half) << 7;
}

// A sum of products times the scales of its row of W and its row of x.  The latter, a power of two, is multiplied in two
// halves around the former: no product on the way leaves fp32's range unless the result does (row scales of W of 2^-86 to 2^86).
__device__ __forceinline__ float scaled(float sum, float rs, uint32_t xs) { return sum * bf16_hi(xs) * rs * bf16_lo(xs); }

// The row of x that a layout row takes, null for a row without a token.
__device__ __forceinline__ const uint4 *source_row(const ExpertArgs &a, int src) {
    const bool real = src >= 0 && src < (a.by_token ? a.T : a.R_max);
    if (!real && src != -1) bounds_fail(a.status);
    return real ? reinterpret_cast<const uint4 *>(a.x + (size_t)src * a.H) : nullptr;
}

// One CTA per row.
__global__ void __launch_bounds__(kPackThreads)
ep_expert_pack_kernel(const ExpertArgs a) {
    pdl_begin();
    const int row = blockIdx.x, tid = threadIdx.x;
    if (row == 0 && tid == 0) *a.drawn = 0u;
    const int R = a.row_offsets[a.G];                               // these three loads go out together
    const int src = a.by_token ? a.src_info[2 * (size_t)row] : row;
    if (cta_status(a.status) || row >= R) return;
    const int pieces = (a.H + kStepK - 1) / kStepK * 32;
    const uint32_t xs = pack_row(source_row(a, src), a.H, a.xw + (size_t)row * pieces);
    if (tid == 0) a.xs[row] = xs;
}

// Sums of products leave the tensor cores after every part of x, because their adder truncates: a chain over all of k would
// lose up to an ulp of the running sum in each of H / 16 additions.  A thread keeps the parts' sum in its own places of
// shared memory, [register][lane] of its warp, which costs no registers; their address is made anew from the thread's index
// for the same reason.  64 tokens, top-2 of 8, 14336 -> 4096: 99.6 us without this, 101.1 with it; 104 to 112 with the
// address held, with 16-byte places, with the sum in registers, or at the part's end.
template <int N> __device__ __forceinline__ unsigned own_places(const void *sums) {
    unsigned tid;
    asm volatile("mov.u32 %0, %%tid.x;" : "=r"(tid));
    return (unsigned)__cvta_generic_to_shared(sums) + (tid >> 5) * (N * 128) + (tid & 31) * 4;
}
__device__ __forceinline__ float ld_shared(unsigned at) {
    float v;
    asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(at));
    return v;
}
template <int MT, int NT> __device__ __forceinline__ void put_sums(const void *sums, float (&acc)[MT][NT][4], bool first) {
    const unsigned at = own_places<4 * MT * NT>(sums);
#pragma unroll
    for (int u = 0; u < 4 * MT * NT; ++u) {
        float &v = acc[u / (4 * NT)][u / 4 % NT][u & 3];
        float before = 0.0f;
        if (!first) before = ld_shared(at + u * 128);
        asm volatile("st.shared.f32 [%0], %1;" ::"r"(at + u * 128), "f"(before + v) : "memory");
        v = 0.0f;
    }
}
template <int MT, int NT> __device__ __forceinline__ void take_sums(const void *sums, float (&acc)[MT][NT][4]) {
    const unsigned at = own_places<4 * MT * NT>(sums);
#pragma unroll
    for (int u = 0; u < 4 * MT * NT; ++u) acc[u / (4 * NT)][u / 4 % NT][u & 3] += ld_shared(at + u * 128);
}

// How a kernel is built: MT m16 tiles of weight rows per warp and NT blocks of 8 layout rows per pass, for THREADS threads
// and CTAS CTAs per SM; P steps of x fill one of the two shared-memory buffers, in rows PITCH pieces apart, half a
// 128-byte line beyond whole lines so that two rows' reads miss each other's banks.
template <int MT_, int NT_, int THREADS_, int CTAS_, int P_> struct Shape {
    static constexpr int MT = MT_, NT = NT_, THREADS = THREADS_, CTAS = CTAS_, P = P_;
    static constexpr int WARPS = THREADS / 32, ROWS = 8 * NT, PITCH = P * 32 + 4;
    static constexpr size_t SMEM = (size_t)2 * ROWS * PITCH * sizeof(uint4);
};

// Work is cut into items: a tile of weight rows of a group and a chunk of up to 8 * NT of the group's rows, chunks of
// a tile next to each other so that L2 serves the second reading of its weights.  A CTA begins with two
// items and draws the others from a counter, each while it works on the one before the last, because SMs
// differ in speed by a sixth while HBM is busy (items in turn / drawn: 271 / 265 us for 16 tokens, top-8 of 256, 7168 -> 2 x
// 2048 gated; 116 / 106 us for 64 tokens, top-4 of 64, 4096 -> 2 x 2048).  Sums do not depend on who draws what.
// KS of a CTA's warps share each 32-row tile and split its k; their sums meet in shared memory in a fixed
// order.  Nothing drains at an item's end: x of the next part of P steps, of the next item too, is copied to
// shared memory while the present one is computed, and a warp has its next step's weights on their way to
// registers.  The first weights start before x is there, because the weights, like every argument, were
// complete before the first kernel started.
template <int ALIGN, typename S>
__global__ void __launch_bounds__(S::THREADS, S::CTAS)
ep_expert_matvec_kernel(const ExpertArgs a) {
    constexpr int kChunkRows = S::ROWS, P = S::P, PITCH = S::PITCH, MT = S::MT, NT = S::NT;
    constexpr int kExpertThreads = S::THREADS, kExpertWarps = S::WARPS, kTileRows = 16 * MT;
    extern __shared__ uint4 s_x[];                                  // [2][8 * NT][PITCH]
    __shared__ float s_red[kExpertWarps][4 * MT * NT][32];          // partial sums, [warp][register][lane]
    __shared__ uint32_t s_xs[2][kChunkRows];                        // scales of an item's rows of x
    __shared__ float s_rs[2][kExpertThreads];                       // and of W (the up rows last)
    __shared__ int s_first[kMaxE + 2];                              // chunks before each group
    __shared__ int s_row[kMaxE + 2];                                // first row of each group
    __shared__ int s_warp[kExpertWarps];
    __shared__ int s_next[2];                                       // the item after the present one, by its parity
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, gl = lane >> 2, q = lane & 3;

    // chunks before each group: thread i scans a run of groups
    for (int g = tid; g <= a.G; g += kExpertThreads) s_row[g] = min(max(a.row_offsets[g], 0), a.R_max);
    __syncthreads();
    {
        const int per = (a.G + kExpertThreads - 1) / kExpertThreads;
        const int g0 = min(tid * per, a.G), g1 = min(g0 + per, a.G);
        int n = 0, prev = s_row[g0];
        for (int g = g0; g < g1; ++g) {
            const int next = s_row[g + 1];
            s_first[g] = n;                                         // within the thread's run
            n += next > prev ? (next - prev + kChunkRows - 1) / kChunkRows : 0;
            prev = next;
        }
        int incl = n;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int v = __shfl_up_sync(kFullMask, incl, o);
            if (lane >= o) incl += v;
        }
        if (lane == 31) s_warp[warp] = incl;
        __syncthreads();
        int base = incl - n;
        for (int w = 0; w < warp; ++w) base += s_warp[w];
        for (int g = g0; g < g1; ++g) s_first[g] += base;
        if (tid == kExpertThreads - 1) s_first[a.G] = base + n;
        __syncthreads();
    }
    const int KS = a.KS, NS = kExpertWarps / KS;
    const int kw = warp & (KS - 1), nw = warp / KS;
    const int n_out = a.swiglu ? a.N >> 1 : a.N;
    const int per_warp = a.swiglu ? kTileRows / 2 : kTileRows;
    const int rows_out = per_warp * NS;                             // output columns of an item
    const int blocks = (n_out + rows_out - 1) / rows_out;
    // fits an int: an item has 32 columns or more, a chunk 8 rows but for a group's last, and the output fits the device
    const int items = s_first[a.G] * blocks;
    const int steps = (a.H + kStepK - 1) / kStepK;

    struct Cursor {
        int item, g, chunk, block;                                  // chunk: of the group
    };
    const auto locate = [&](Cursor &c) {                            // from c.item: the last group that begins at or before it
        int lo = 0, hi = a.G;
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (s_first[mid] * blocks <= c.item) lo = mid;
            else hi = mid;
        }
        const int of_group = c.item - s_first[lo] * blocks, n = s_first[lo + 1] - s_first[lo];
        c.g = lo;
        c.block = n == 1 ? of_group : of_group / n;
        c.chunk = of_group - c.block * n;
    };
    // the weight rows of this thread in an item, clamped to the matrix (the excess is not stored).  Rows g and g + 8 of a
    // tile are output columns 8 apart, or a gate row and its up row.
    const auto weight_rows = [&](const Cursor &c, unsigned (&row)[2 * MT]) {
        const unsigned base = (unsigned)c.g * (unsigned)a.N;
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
            const int n = c.block * rows_out + nw * per_warp + mt * (a.swiglu ? 8 : 16) + gl;
            row[2 * mt] = base + (unsigned)min(n, n_out - 1);
            row[2 * mt + 1] = base + (unsigned)(a.swiglu ? n_out + min(n, n_out - 1) : min(n + 8, n_out - 1));
        }
    };
    Cursor cur = {(int)blockIdx.x, 0, 0, 0};
    if (cur.item >= items) {                                        // this kernel must not end before the first one has
        pdl_wait();
        return;
    }
    locate(cur);
    Cursor pf = cur;
    unsigned pf_row[2 * MT];
    weight_rows(pf, pf_row);
    int pf_step = kw, parity = 0;
    if (tid == 0) s_next[0] = cur.item + (int)gridDim.x;
    Weights<MT, ALIGN> nxt;
    const uint8_t *const scales_end = a.scales + (size_t)a.G * a.N * (a.H >> 4);
    // past the last item this loads the last step once more: no branch around the loads
    const auto prefetch = [&]() {
        load_weights<ALIGN, MT>(nxt, a.codes, a.scales, scales_end, pf_row, pf_step, q, a.H);
        if (pf_step + KS < steps) {
            pf_step += KS;
        } else {
            const int n = a.draw ? s_next[parity] : pf.item + (int)gridDim.x;
            if (n < items) {
                pf_step = kw;
                pf.item = n;
                locate(pf);
                weight_rows(pf, pf_row);
            }
        }
    };
    const auto row_of_chunk = [&](const Cursor &c) { return s_row[c.g] + c.chunk * kChunkRows; };
    const auto rows_of_chunk = [&](const Cursor &c) { return min(s_row[c.g + 1] - row_of_chunk(c), kChunkRows); };
    // starts the copy of x for steps [from, from + P) of an item, a warp taking a step of a row at a time, and with the
    // first ones that of what the item's sums are multiplied by
    const auto copy_x = [&](const Cursor &c, int from, uint4 *buf, int parity) {
        const int n = min(P, steps - from), m = rows_of_chunk(c);
        const uint4 *src = a.xw + ((size_t)row_of_chunk(c) * steps + from) * 32 + lane;
        for (int u = warp; u < m * n; u += kExpertWarps) {
            const int r = u / n, st = u - r * n;
            cp_async16(buf + r * PITCH + st * 32 + lane, src + ((size_t)r * steps + st) * 32);
        }
        if (from == 0) {
            if (tid < m) cp_async4(&s_xs[parity][tid], a.xs + row_of_chunk(c) + tid);
            if (tid < kTileRows * NS) {
                const int up = a.swiglu && tid >= rows_out, n = min(c.block * rows_out + tid - (up ? rows_out : 0), n_out - 1);
                cp_async4(&s_rs[parity][tid], a.row_scale + (size_t)c.g * a.N + (up ? n_out : 0) + n);
            }
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    prefetch();
    pdl_begin();                                                    // x is there
    copy_x(cur, 0, s_x, 0);
    if (cta_status(a.status)) {
        asm volatile("cp.async.wait_group 0;" ::: "memory");
        return;
    }

    int buf = 0;
    for (; cur.item < items; parity ^= 1) {
        const int row0 = row_of_chunk(cur), m = rows_of_chunk(cur);
        Cursor nx = cur;
        unsigned drawn = 0u;
        float acc[MT][NT][4];
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
                for (int i = 0; i < 4; ++i) acc[mt][t][i] = 0.0f;
        // columns past the chunk's rows repeat its last row; their sums are not stored
        const int x_at = min(gl, m - 1) * PITCH + q;
        int xo[NT];
#pragma unroll
        for (int t = 0; t < NT; ++t) xo[t] = (min(t * 8 + gl, m - 1) - min(gl, m - 1)) * PITCH;
        for (int from = 0; from < steps; from += P, buf ^= 1) {
            asm volatile("cp.async.wait_group 0;" ::: "memory");
            __syncthreads();                                        // this part is there, and every warp is done with the other
            if (from == 0) {
                nx.item = a.draw ? s_next[parity] : cur.item + (int)gridDim.x;
                if (nx.item < items) locate(nx);
                if (a.draw && tid == 0) drawn = atomicAdd(a.drawn, 1u);
            }
            uint4 *other = s_x + (buf ^ 1) * kChunkRows * PITCH;
            if (from + P < steps) copy_x(cur, from + P, other, parity);
            else if (nx.item < items) copy_x(nx, 0, other, parity ^ 1);
            if (from > 0) put_sums(s_red, acc, from == P);
            const int to = min(P, steps - from);
            const uint4 *x = s_x + buf * kChunkRows * PITCH + x_at;
            for (int st = kw; st < to; st += KS) {
                const Weights<MT, ALIGN> w = nxt;
                prefetch();
                if (NT > 1 && m <= 8) mma_step<1>(w, x + st * 32, xo, acc);
                else mma_step<NT>(w, x + st * 32, xo, acc);
            }
        }

        if (steps > P) take_sums(s_red, acc);
        if (a.draw && tid == 0) s_next[parity ^ 1] = (int)(drawn + 2 * gridDim.x);   // not before: the answer takes a microsecond

        // join the KS partial sums; the warps of a tile share the (row of x, weight row) pairs
        if (KS > 1) {
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                for (int t = 0; t < NT; ++t)
#pragma unroll
                    for (int i = 0; i < 4; ++i) s_red[warp][mt * 4 * NT + t * 4 + i][lane] = acc[mt][t][i];
            __syncthreads();
        }
#pragma unroll
        for (int u = 0; u < 2 * MT * NT; ++u) {                     // u = (mt, t, column of the pair)
            if ((u & (KS - 1)) != kw) continue;
            const int mt = u / (2 * NT), t = u / 2 % NT, i = u & 1;
            const int r = t * 8 + q * 2 + i;
            if (r >= m) continue;
            float v[2] = {acc[mt][t][i], acc[mt][t][2 + i]};        // weight rows g and g + 8
            if (KS > 1) {
                v[0] = v[1] = 0.0f;
                for (int w = 0; w < KS; ++w) {
                    v[0] += s_red[nw * KS + w][mt * 4 * NT + t * 4 + i][lane];
                    v[1] += s_red[nw * KS + w][mt * 4 * NT + t * 4 + 2 + i][lane];
                }
            }
            const int at = nw * per_warp + mt * (a.swiglu ? 8 : 16) + gl, n = cur.block * rows_out + at;
            const uint32_t xs = s_xs[parity][r];
            const float *rs = s_rs[parity] + at;
            uint16_t *out = a.out + (size_t)(row0 + r) * n_out;
            if (a.swiglu) {
                if (n < n_out) {
                    const float gate = scaled(v[0], rs[0], xs), up = scaled(v[1], rs[rows_out], xs);
                    out[n] = __bfloat16_as_ushort(__float2bfloat16_rn(gate / (1.0f + expf(-gate)) * up));
                }
            } else {
                if (n < n_out) out[n] = __bfloat16_as_ushort(__float2bfloat16_rn(scaled(v[0], rs[0], xs)));
                if (n + 8 < n_out) out[n + 8] = __bfloat16_as_ushort(__float2bfloat16_rn(scaled(v[1], rs[8], xs)));
            }
        }
        cur = nx;
    }
}

// One token: every row is its expert's only one, so rows are items of their own and a layout of K (+1) rows needs no scan.  A
// CTA packs the row for itself while its first weights are on their way, which saves the kernels above a launch and its
// dependency.  Taken while one wave of CTAs covers the rows, with items of at most 8 steps or split ones (1 token, us against
// the kernels above: top-8 of 128, 2048 -> 2 x 768 gated 6.4 against 8.2, 768 -> 2048 4.3 against 6.7; top-2 of 8, 14336 -> 4096
// 24.0 against 32.6; 4096 -> 2 x 7168 gated 18.7 against 22.1, where KS = 2 just fits, and 4096 -> 2 x 14336, where it does not,
// 31.3 by both).
constexpr int kRowThreads = 256, kRowCtas = 2;                      // per SM

template <int ALIGN>
__global__ void __launch_bounds__(kRowThreads, kRowCtas)
ep_expert_row_kernel(const ExpertArgs a, int one_wave) {
    constexpr int MT = 2, kWarps = kRowThreads / 32;
    extern __shared__ uint4 s_x[];                                  // [step][word][quad thread]
    __shared__ float s_sum[kWarps][2 * MT][8];                      // of each warp's rows g and g + 8 of its tiles
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, gl = lane >> 2, q = lane & 3;
    const int row = blockIdx.y, KS = a.KS, kw = warp & (KS - 1), nw = warp / KS;
    pdl_begin_if(one_wave);
    const int R = a.row_offsets[a.G], g = a.expert_ids[row];        // these loads go out together
    const int src = a.by_token ? a.src_info[2 * (size_t)row] : row;
    if (cta_status(a.status) || row >= R) return;
    if (g < 0 || g >= a.G) {
        bounds_fail(a.status);
        return;
    }
    const int n_out = a.swiglu ? a.N >> 1 : a.N, per_warp = a.swiglu ? 8 * MT : 16 * MT, rows_out = per_warp * (kWarps / KS);
    const int steps = (a.H + kStepK - 1) / kStepK;
    const uint8_t *const scales_end = a.scales + (size_t)a.G * a.N * (a.H >> 4);
    unsigned w_row[2 * MT];                                         // as in the kernel above
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
        const int n = blockIdx.x * rows_out + nw * per_warp + mt * (a.swiglu ? 8 : 16) + gl;
        const unsigned base = (unsigned)g * (unsigned)a.N;
        w_row[2 * mt] = base + (unsigned)min(n, n_out - 1);
        w_row[2 * mt + 1] = base + (unsigned)(a.swiglu ? n_out + min(n, n_out - 1) : min(n + 8, n_out - 1));
    }
    Weights<MT, ALIGN> nxt;
    load_weights<ALIGN, MT>(nxt, a.codes, a.scales, scales_end, w_row, kw, q, a.H);
    const int n = blockIdx.x * rows_out + tid;                      // the output of this thread
    const bool mine = tid < rows_out && n < n_out;
    float rs = 0.0f, rs_up = 0.0f;
    if (mine) {
        rs = a.row_scale[(size_t)g * a.N + n];
        if (a.swiglu) rs_up = a.row_scale[(size_t)g * a.N + n_out + n];
    }
    const uint32_t xs = pack_row(source_row(a, src), a.H, s_x);
    __syncthreads();
    float sum[2 * MT] = {};                                         // of weight rows g and g + 8 of each tile, over the steps
    const int xo[1] = {0};
    for (int st = kw; st < steps; st += KS) {
        const Weights<MT, ALIGN> w = nxt;
        // past the last step this loads it once more: no branch around the loads
        load_weights<ALIGN, MT>(nxt, a.codes, a.scales, scales_end, w_row, st + KS < steps ? st + KS : st, q, a.H);
        float acc[MT][1][4] = {};
        mma_step<1>(w, s_x + st * 32 + q, xo, acc);                 // all 8 columns are the row; the first is kept
#pragma unroll
        for (int i = 0; i < 2 * MT; ++i) sum[i] += acc[i >> 1][0][2 * (i & 1)];
    }
    if (q == 0) {
#pragma unroll
        for (int i = 0; i < 2 * MT; ++i) s_sum[warp][i][gl] = sum[i];
    }
    __syncthreads();
    if (!mine) return;
    const int tw = tid / per_warp * KS, j = tid % per_warp;
    float v = 0.0f, up = 0.0f;
    for (int w = tw; w < tw + KS; ++w) {
        if (a.swiglu) {
            v += s_sum[w][j >> 3 << 1][j & 7];
            up += s_sum[w][(j >> 3 << 1) + 1][j & 7];
        } else {
            v += s_sum[w][j >> 3][j & 7];
        }
    }
    v = scaled(v, rs, xs);
    if (a.swiglu) v = v / (1.0f + expf(-v)) * scaled(up, rs_up, xs);
    a.out[(size_t)row * n_out + n] = __bfloat16_as_ushort(__float2bfloat16_rn(v));
}

// Up to 8 rows per expert: two steps of weights in 128 registers, 16 warps per SM, passes of 8 rows.  More: a pass serves 16
// rows and 12 warps have 168 registers each, since spilled prefetches would be waited for.  8 experts, top-2, 4096 -> 2 x 2048
// gated, with 4 / 6 / 8 / 10 rows per expert: 23 / 28 / 33 / 37 us with passes of 8 rows, 31 / 32 / 34 / 36 us with 16; 64
// experts with 4 / 8: 106 / 157 against 116 / 159; 8 experts with 16 rows, 14336 -> 4096: 141 and 102 us.  Of the shapes for 16
// rows this one is best there: 10 % more with two CTAs of 6 warps, 18 % with 8 warps, 31 % with passes of 32 rows.
using FewRows = Shape<2, 1, 256, 2, 8>;
using MoreRows = Shape<2, 2, 384, 1, 8>;

// Rows on 8-byte boundaries only need more registers for their scales.  16 tokens, 64 experts, top-4, 2064 -> 2 x 2048 gated /
// 7184 -> the same: 58 / 164 us with FewRows, which spills, 55 / 155 us with this.  On 16-byte boundaries FewRows holds: 53 us
// at 2080, 60 with this.  (2048 takes 37 us: its rows fill whole steps of 256 k and one load brings each thread's 64 codes.)
using FewUnaligned = Shape<2, 1, 384, 1, 8>;

// KS: the split that ends soonest.  x is the number of items per CTA, and an item lasts its warps' steps and about one more to
// begin and end it, a little longer where sums are joined.  Passes of 8 rows are bound by HBM, so CTAs that work alone on an SM
// are faster, and the last drawn items end within about 0.6 of an item's time of x; passes of 16 rows are bound by their own
// instructions and take whole rounds.  KS 1 / 2 / 4: 16 tokens, top-8 of 256, 7168 -> 2 x 2048 gated 269 / 266 / 283 us; 64
// tokens, top-4 of 64, 4096 -> 2 x 2048 106 / 117 / 132; 4 tokens, top-8 of 128, 2048 -> 2 x 768 20 / 17 / 18; 64 tokens,
// top-2 of 8, 14336 -> 4096 102 / 112 / 131.
template <typename S>
int choose_split(const ExpertArgs &a, int steps, float chunks) {
    const int n_out = a.swiglu ? a.N / 2 : a.N, per_warp = S::MT * (a.swiglu ? 8 : 16);
    int best = 1;
    float best_time = 0.0f;
    const float sms = (float)std::max(device_sm_count(), 1);
    for (int ks = 1; ks <= 4 && ks <= steps; ks *= 2) {
        const int rows = per_warp * (S::WARPS / ks);
        const float items = chunks * (float)((n_out + rows - 1) / rows);
        const float x = items / (sms * S::CTAS);
        const float begin_end = ks == 1 ? 1.0f : ks == 2 ? 1.25f : 1.4f;
        const float time = (S::NT > 1 ? ceilf(x) : fmaxf(x, 1.0f) + 0.6f) * ((float)((steps + ks - 1) / ks) + begin_end);
        if (ks == 1 || time < best_time) {
            best = ks;
            best_time = time;
        }
    }
    return best;
}

template <int ALIGN, typename S>
int launch_expert_matvec(ExpertArgs a, float chunks, cudaStream_t st) {
    constexpr auto kern = ep_expert_matvec_kernel<ALIGN, S>;
    a.KS = choose_split<S>(a, pack_steps(a.H), chunks);
    a.draw = pack_steps(a.H) >= 2 * a.KS;
    int rc = allow_smem<kern>(S::SMEM);
    if (rc != EP_OK) return rc;
    const int pack = std::min(std::max((a.H / 8 + 31) / 32 * 32, 128), kPackThreads);
    rc = launch_pdl(ep_expert_pack_kernel, dim3(a.R_max), dim3(pack), 0, st, a);
    if (rc != EP_OK) return rc;
    const int grid = resident_blocks(kern, S::THREADS, S::SMEM);
    if (grid <= 0) return EP_ERR_CUDA;
    return launch_pdl(kern, dim3(grid), dim3(S::THREADS), S::SMEM, st, a);
}

// CTAs of the row kernel when KS of a CTA's warps share a tile.
int row_blocks(const ExpertArgs &a, int KS) {
    const int n_out = a.swiglu ? a.N / 2 : a.N, rows_out = FewRows::MT * (a.swiglu ? 8 : 16) * (kRowThreads / 32 / KS);
    return (n_out + rows_out - 1) / rows_out;
}

// And how many of them are resident at once.
int row_wave() { return kRowCtas * device_sm_count(); }

template <int ALIGN>
int launch_expert_row(ExpertArgs a, cudaStream_t st) {
    constexpr auto kern = ep_expert_row_kernel<ALIGN>;
    const int rc = allow_smem<kern>((size_t)pack_steps(kMaxH) * 512);
    if (rc != EP_OK) return rc;
    a.KS = 1;                                                       // the most that one wave of CTAs has room for
    while (a.KS < 4 && 2 * a.KS <= pack_steps(a.H) && row_blocks(a, 2 * a.KS) * a.R_max <= row_wave()) a.KS *= 2;
    const dim3 grid(row_blocks(a, a.KS), a.R_max);
    return launch_pdl(kern, grid, dim3(kRowThreads), (size_t)pack_steps(a.H) * 512, st, a, one_wave(grid.x * grid.y));
}

}  // namespace
}  // namespace ep

using namespace ep;

extern "C" size_t ep_expert_matvec_workspace_bytes(const ep_layout_t *L, int hidden_size) {
    if (!layout_ok(L) || !hidden_ok(hidden_size)) return 0;
    const size_t R = layout_rows(L);
    return R * pack_steps(hidden_size) * 512 + 16 + R * sizeof(uint32_t);
}

extern "C" int ep_expert_matvec(const uint16_t *x, int x_by_token, const uint8_t *codes, const uint8_t *scales,
                                const float *row_scale, int hidden_size, int out_rows, int swiglu,
                                const ep_layout_t *L, uint16_t *out, void *workspace, size_t workspace_bytes,
                                void *stream) {
    EP_NVTX_RANGE("ep_expert_matvec");
    const int H = hidden_size, N = out_rows;
    if (!layout_ok(L) || !hidden_ok(H) || N < 1 || N > kMaxN || (swiglu != 0 && swiglu != 1)) return EP_ERR_INVALID_ARG;
    if ((x_by_token != 0 && x_by_token != 1) || (swiglu && N % 2 != 0)) return EP_ERR_INVALID_ARG;
    const void *ptrs[] = {x, codes, scales, row_scale, out, workspace};
    for (const void *p : ptrs)
        if (!aligned16(p)) return EP_ERR_INVALID_ARG;
    if (L->T == 0) return EP_OK;
    for (const void *p : ptrs)
        if (!p) return EP_ERR_INVALID_ARG;
    if (x_by_token && !L->src_info) return EP_ERR_INVALID_ARG;
    if (workspace_bytes < ep_expert_matvec_workspace_bytes(L, H)) return EP_ERR_INVALID_ARG;
    ExpertArgs a = {};
    a.x = x; a.codes = codes; a.scales = scales; a.row_scale = row_scale;
    a.H = H; a.N = N; a.by_token = x_by_token; a.swiglu = swiglu;
    a.T = L->T; a.G = L->E + L->fused_shared; a.R_max = layout_rows(L);
    a.row_offsets = L->row_offsets; a.expert_ids = L->expert_ids; a.src_info = L->src_info; a.status = L->status;
    const int steps = pack_steps(H);
    a.xw = (uint4 *)workspace;
    a.drawn = (unsigned *)(a.xw + (size_t)a.R_max * steps * 32);
    a.xs = (uint32_t *)(a.drawn + 4);
    a.out = out;
    const float per_expert = (float)L->T * L->K / L->E;
    const bool few = per_expert <= 8.0f;
    // chunks that a layout of this many rows has, if the router spreads them evenly
    const float active = L->E * (1.0f - powf(fmaxf(1.0f - (float)L->K / L->E, 0.0f), (float)L->T));
    const float rows = few ? 8.0f : 16.0f;
    const float chunks = active * fmaxf(1.0f, per_expert / rows + 0.5f) + (L->fused_shared ? ceilf(L->T / rows) : 0.0f);
    cudaStream_t st = as_stream(stream);
    const bool by64 = H % 64 == 0 && (reinterpret_cast<uintptr_t>(codes) & 31u) == 0;
    if (L->T == 1 && a.R_max <= L->K + 1 && L->expert_ids && row_blocks(a, steps > 8 ? 2 : 1) * a.R_max <= row_wave()) {
        if (by64) return launch_expert_row<32>(a, st);
        return H % 32 == 0 ? launch_expert_row<16>(a, st) : launch_expert_row<8>(a, st);
    }
    if (few) {
        if (by64) return launch_expert_matvec<32, FewRows>(a, chunks, st);
        return H % 32 == 0 ? launch_expert_matvec<16, FewRows>(a, chunks, st) : launch_expert_matvec<8, FewUnaligned>(a, chunks, st);
    }
    if (by64) return launch_expert_matvec<32, MoreRows>(a, chunks, st);
    return H % 32 == 0 ? launch_expert_matvec<16, MoreRows>(a, chunks, st) : launch_expert_matvec<8, MoreRows>(a, chunks, st);
}
