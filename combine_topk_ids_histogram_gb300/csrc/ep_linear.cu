// ep_linear.cu -- grouped products of the rows of a dispatch layout with their group's 16-bit weights, optionally with the gated
// activation silu(gate) * up, and their gradients.
//
//   forward     out[r, n] = sum over k of x[r, k] w[g, n, k]                 (gated: w holds F gate rows, then F up rows)
//   grad_x      out[r, k] = sum over n of grad[r, n] w[g, n, k]              (or, through the gate, that of gate and up)
//   grad_w      out[g, n, k] = sum over the rows r of g of grad[r, n] x[r, k]
//
// One kernel, templated on the form, of CTA pairs that stay: a pair takes the places of pairs that have not begun until none is left,
// so that pairs which drew long tiles take fewer.  The weights' rows (or columns) are M of the tensor cores' product and the
// layout's rows are N, in steps of 32: a group of any number of rows then costs about what its rows cost, and weights, which have
// hundreds of rows or more, fill M.  A pair shares a product of 256 x 256: each CTA loads 128 of M and half of N by TMA, one copy for
// an operand, and keeps the sums of its 128 of M in tensor memory, twice, so that one chunk's sums leave while the next one's are
// added up.  Warp 0 loads, warp 1 of the first CTA issues the products, warp 3 looks tiles up ahead of the others, warps 4 to 11 take
// results out, four at a time 32 columns, with registers that the others hand over; warp 2 (grad_w) clears the rows behind a group's last one in shared memory, since
// there they are summed over.  No atomics: the order of every sum is fixed.
//
// 4864 rows of one group, 4096 -> 4096: 84 us, 1940 TFLOP/s (0.97 of the measured cuBLAS burst), and so the gated form and grad_x; K = 16384:
// 332 to 340 us, where the power limit lowers the clock.  Many groups of few rows are bound by HBM (256 tokens, top-8 of 64 and a shared
// expert, 7168 -> 2 x 2048 gated: 576 us, 6.7 TB/s), those between by the way from L2, which has to bring 32 KB for 512 cycles of
// products at 256 rows and as much for half the work at 128, while outputs leave: 65536 rows, drawn log-normally over 128 groups, 2048 ->
// 2 x 768 gated with gate and up saved 294 us (floor 205), the down product 148 (115), grad_x through the gate 200 (160), grad_w 178
// (115), each kernel by itself on inputs that stay the same; calls on changing inputs take 342, 171 and, both gradients, 406.
// Without its loads / its outputs the first of them took 207 / 276 us of 324 in an earlier form; fetching the next tile's operands into
// L2 ahead (by TMA, in bulk, or by lines) gained nothing in grad_w and cost up to 150 % elsewhere, eviction hints changed nothing,
// and taking several groups at a time, less read at the same moment by several pairs, cost 4 to 60 %.
#include <limits.h>
#include <math.h>

#include <algorithm>

#include "ep_async.cuh"
#include "ep_host.h"
#include "ep_tensor.cuh"
#include "ep_types.cuh"

namespace ep {
namespace {

enum Form { kPlain, kGlu, kGradX, kGradGate, kGradW };

constexpr int kPair = 2;                      // CTAs that work on one product
constexpr int kThreads = 384;
constexpr int kOutGroups = 2;                // of four warps that take results out
constexpr int kFewRegs = 48, kManyRegs = 208;   // of a thread of the first four warps, and of the others (launched with 168 each)
constexpr int kBlockK = 64;                  // of the summed dimension in a stage: 128 bytes, one swizzle row
constexpr int kTileA = 128 * kBlockK * 2;    // bytes a CTA loads of each operand per stage
constexpr int kTileB = 128 * kBlockK * 2;
constexpr int kStageBytes = kTileA + kTileB;
constexpr int kCols = 256;                   // columns of tensor memory per tile's sums
constexpr int kMaxGroups = kMaxE + 1;
// As many stages as fit.  What they hide is the way from L2: in an earlier form, with 3 / 4 / 5 of them the gated products of 65536 rows
// in 128 groups, 2048 -> 2 x 768 took 327 / 294 / 272 us, the down products 188 / 172 / 156.
constexpr int kStages = 6;
constexpr int kStaging = 16384;              // bytes in which a group of four warps turns its results into rows
constexpr int kSuper = 8;                    // grad_w: tiles of N that go through all of K before the next
// The tensor cores' adder cuts off what it adds, all to one side: terms of one sign lose 2^-22 of the running sum with every 16 products
// (fp16; a third of that in bf16, whose products have fewer digits).  So sums leave them every 8 blocks, 512 products, and are added up in
// registers, rounded to nearest.  Whatever the number of products, sums of normal ones lose 4.7e-7 of their norm then (fp16 6.5e-7) and of one
// sign 9e-7 (2.8e-6); fp16 sums that stayed for 32768 / 65536 products lost 2e-4 / 4e-4, half an ulp and more.  With 256 products
// bf16 lost 2.3e-7, and fp32 gradients of 8192 rows took 1506 us (8 x 28672 x 4096) where they take 1320.  For rows the first two chunks are
// longer, so that products get further ahead while a tile's results leave: 65536 rows in 128 groups, 2048 -> 2 x 768 with gate and up kept
// take 330 us with chunks of 8 blocks, 294 so, and 285 with sums that stay; grad_x through the gate 230, 200 and 182.
constexpr int kChunk = 8, kFirstChunk = 12;

// A tile: rows or features, and what is summed over.
struct Work {
    int g, m, row, n;                        // group (-1: no more tiles); first of M of the pair; first row; valid of N
    int col;                                 // grad_w: first column
    int kb, last;                            // blocks of 64 to sum over, and the valid of the last
    int half;                                // of N, what each CTA loads
};

constexpr int kSlots = 3;                    // tiles that the roles may be apart, and be taken ahead

struct Control {
    uint64_t full[kStages], empty[kStages], landed[kStages];
    uint64_t sums_full[2], sums_empty[2], work_full[kSlots], work_empty[kSlots];
    uint64_t drawn, read;                    // the answer to a request for the next tile: arrived, and read by both CTAs
    uint4 answer;
    Work work[kSlots];
    uint32_t tmem, skip;
    int part[kThreads / 32];
    int start[(kMaxGroups + 1) / 2 + 1];     // first tile of every other group
};
constexpr size_t kSmem = (size_t)kStages * kStageBytes + kOutGroups * kStaging + sizeof(Control);
static_assert(kSmem <= 227 * 1024, "shared memory of a CTA");

struct LinearArgs {
    const int32_t *row_offsets;
    int32_t *status;
    int G, R_max;
    int M;                                   // of the output: features of a row (gated: F), rows of a weight gradient
    int sum;                                 // length of the sums (forms that sum over rows: columns of the output)
    int f16, wide, add;                      // operands fp16; grad_w: fp32 output, added to what is there
    int beside;                              // grad_w behind grad_x in the same call
    int whole_a, whole_b;                    // whether the operand's map has the blocks of 64 as a dimension
    uint16_t *out, *gate_up;                 // gate_up: saved by kGlu, read by kGradGate
};

// What tile number `tile` is.
template <Form FORM> struct Tiles {
    static constexpr int kM = FORM == kGlu ? 64 * kPair : 128 * kPair, kN = 128 * kPair;
    static constexpr int kUnit = 16 * kPair;    // of N in a product
    static constexpr int kFirst = FORM == kGradW ? kChunk : kFirstChunk;
    // Blocks of the chunk that begins at block b.
    static __device__ __forceinline__ int chunk_blocks(int b) { return b < 2 * kFirst ? kFirst : kChunk; }
    const LinearArgs &a;
    const Control &c;

    // A group's first row, inside the buffers whatever the layout says.
    __device__ int off(int g) const { return min(max(a.row_offsets[g], 0), a.R_max); }
    __device__ int parts(int rows) const { return (max(rows, 0) + kN - 1) / kN; }
    // False behind the last one.
    __device__ bool look_up(int tile, Work &w) const {
        const int m_tiles = (a.M + kM - 1) / kM;
        if constexpr (FORM == kGradW) {
            const int n_tiles = (a.sum + kN - 1) / kN, in = tile % (m_tiles * n_tiles);
            w.g = tile / (m_tiles * n_tiles);
            if (w.g >= a.G) return false;
            const int first = in / (kSuper * n_tiles) * kSuper, wide = min(kSuper, m_tiles - first), at = in - first * n_tiles;
            w.m = (first + at % wide) * kM;
            w.col = at / wide * kN;
            w.n = min(kN, a.sum - w.col);
            w.row = off(w.g);
            sum_over(w, max(off(w.g + 1) - w.row, 0));
        } else {
            int p = 0, hi = (a.G + 1) / 2;   // the last two groups that begin at or before the tile
            if (tile >= c.start[hi]) return false;
            while (hi - p > 1) {
                const int mid = (p + hi) >> 1;
                if (c.start[mid] <= tile) p = mid;
                else hi = mid;
            }
            int g = 2 * p, begin = off(g), end = off(g + 1), in = tile - c.start[p];
            const int behind = off(min(g + 2, a.G)), tiles = parts(end - begin) * m_tiles;
            if (in >= tiles) {
                in -= tiles;
                begin = end;
                end = behind;
                ++g;
            }
            // the group's rows in equal parts: a part of few rows would load the weights for little work
            const int rows = end - begin, n = parts(rows), part = ((rows + n - 1) / n + kUnit - 1) / kUnit * kUnit, at = in % n * part;
            w.g = g;
            w.m = in / n * kM;
            w.row = begin + at;
            w.n = min(part, rows - at);
            sum_over(w, a.sum);
        }
        // whole blocks of 64 where one copy brings them
        const int unit = FORM == kGradW && a.whole_b ? 64 : kUnit / kPair;
        w.half = (w.n + unit * kPair - 1) / (unit * kPair) * unit;
        return true;
    }
    __device__ void sum_over(Work &w, int n) const {
        w.kb = (n + kBlockK - 1) / kBlockK;
        w.last = n - (w.kb - 1) * kBlockK;
    }
};

// A role's view of them: one warp looks tiles up ahead of the others and hands them over in shared memory, since the look-up takes
// some 700 cycles, in which no copy or product would be issued.
struct Feed {
    Control &c;
    int i;
    // Called by a whole warp, or by one lane alone.
    template <bool kWarp> __device__ bool next(Work &w, uint32_t rank, bool &ok) {
        const int s = i % kSlots;
        ok = mbar_wait(smem_u32(&c.work_full[s]), i / kSlots & 1);
        if constexpr (kWarp) ok = __all_sync(kFullMask, ok);
        if (!ok) return false;
        w = c.work[s];
        ++i;
        if constexpr (kWarp) __syncwarp();
        if (!kWarp || (threadIdx.x & 31) == 0) mbar_arrive(at_rank(smem_u32(&c.work_empty[s]), rank));
        return w.g >= 0;
    }
};

__device__ __forceinline__ uint32_t pack16(float lo, float hi, int f16) {
    return f16 ? f32_to_word(lo, hi, __half()) : f32_to_word(lo, hi, __nv_bfloat16());
}
__device__ __forceinline__ float wide16(uint16_t v, int f16) {
    return f16 ? __half2float(__ushort_as_half(v)) : __uint_as_float((uint32_t)v << 16);
}
// Of all warps of a group of four.
template <int N> __device__ __forceinline__ void regs_down() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N)); }
template <int N> __device__ __forceinline__ void regs_up() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N)); }
__device__ __forceinline__ void bar_sync(int id, int threads) { asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory"); }
// And whether `v` holds for all of them.
__device__ __forceinline__ bool bar_all(int id, int threads, bool v) {
    uint32_t r;
    asm volatile("{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %3, 0;\n\tbarrier.cta.red.and.pred q, %1, %2, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
                 : "=r"(r) : "r"(id), "r"(threads), "r"((uint32_t)v) : "memory");
    return r != 0;
}
__device__ __forceinline__ void cp_async16(void *smem, const void *gmem) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(smem)), "l"(gmem) : "memory");
}

// s = 1 / (1 + exp(-v)), and 1 - s without cancellation, from e = exp(-|v|): no exponential overflows, small ones keep their digits
// down to the subnormal numbers, and the divisor lies in [1, 2], where the fast division is within 2 ulp.
struct Sigmoid {
    float s, rest;
    __device__ explicit Sigmoid(float v) {
        const float e = expf(-fabsf(v)), r = __fdividef(1.0f, 1.0f + e);
        s = v < 0.0f ? e * r : r;
        rest = v < 0.0f ? r : e * r;
    }
};

// The copies of block b of a tile, whose m and n begin at these for the CTA, into a stage.  One for an operand where its map allows it: each
// takes the issuing thread some 50 cycles of the 512 that the products of a block last.
template <Form FORM> struct Copies {
    const CUtensorMap &map_a, &map_b, &map_c;
    const LinearArgs &a;
    uint32_t stage, bar;
    template <int DIMS> __device__ __forceinline__ void load(int at, const CUtensorMap &m, const int (&c)[DIMS]) const {
        tma_load<DIMS>(stage + at, &m, c, bar);
    }
    __device__ __forceinline__ void block(const Work &w, int b, int m, int n, int half) const {
        const int k = b * kBlockK;
        if constexpr (FORM == kGradW) {
            if (a.whole_a) {
                load(0, map_a, {0, w.row + k, m >> 6});
            } else {
                load(0, map_a, {m, w.row + k});
                load(8192, map_a, {m + 64, w.row + k});
            }
        } else if constexpr (FORM == kPlain) {
            load(0, map_a, {k, m, w.g});
        } else if constexpr (FORM == kGlu) {
            load(0, map_a, {k, 0, 0, m >> 4, w.g});
        } else if (a.whole_a) {
            load(0, map_a, {0, k, m >> 6, w.g});
        } else {
            load(0, map_a, {m, k, w.g});
            load(8192, map_a, {m + 64, k, w.g});
        }
        if constexpr (FORM == kGradW) {
            if (a.whole_b) {
                load(kTileA, map_b, {0, w.row + k, n >> 6});
            } else {
                load(kTileA, map_b, {n, w.row + k});
                load(kTileA + 8192, map_b, {n + 64, w.row + k});
            }
        } else if (half > 96) {
            load(kTileA, map_b, {k, n});
        } else {
            for (int i = 0; i < half; i += 32) load(kTileA + i * 128, map_c, {k, n + i});
        }
    }
};

template <Form FORM>
__global__ void __launch_bounds__(kThreads, 1)
ep_linear_kernel(const __grid_constant__ CUtensorMap map_a, const __grid_constant__ CUtensorMap map_b,
                 const __grid_constant__ CUtensorMap map_c, const LinearArgs a) {
    constexpr bool kAmn = FORM == kGradX || FORM == kGradGate || FORM == kGradW, kBmn = FORM == kGradW;
    extern __shared__ __align__(1024) uint8_t smem[];    // nothing else is in shared memory, so that it begins on such a boundary
    uint8_t *const staging = smem + kStages * kStageBytes;
    Control &c = *reinterpret_cast<Control *>(staging + kOutGroups * kStaging);
    const int tid = threadIdx.x, warp = __shfl_sync(kFullMask, tid >> 5, 0), lane = tid & 31;
    const uint32_t rank = cluster_rank();

    cluster_arrive();
    if (tid == 0) {
        tma_prefetch_map(&map_a);
        tma_prefetch_map(&map_b);
        for (int s = 0; s < kStages; ++s) {
            mbar_init(smem_u32(&c.full[s]), kPair);         // each CTA's loader (or its clearing warp)
            mbar_init(smem_u32(&c.empty[s]), 1);
            mbar_init(smem_u32(&c.landed[s]), 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(smem_u32(&c.sums_full[b]), 1);
            mbar_init(smem_u32(&c.sums_empty[b]), 4 * kOutGroups * kPair);
        }
        mbar_init(smem_u32(&c.drawn), 1);
        mbar_init(smem_u32(&c.read), kPair);
        for (int s = 0; s < kSlots; ++s) {
            mbar_init(smem_u32(&c.work_full[s]), 1);
            // loads, results, products in the first CTA, rows to clear
            mbar_init(smem_u32(&c.work_empty[s]), 1 + 4 * kOutGroups + (rank == 0) + (FORM == kGradW));
        }
        mbar_init_done();
    }
    if (warp == 2) tmem_alloc<kPair>(smem_u32(&c.tmem), 2 * kCols);
    // The weights' gradient needs nothing of the rows' in front of it: it begins as that one's CTAs leave, and waits for its end at its
    // own.  What came before both was complete when the CTAs in front let this launch begin.
    if (a.beside) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    else pdl_begin();
    cluster_wait();                                      // the other CTA has begun
    if (tid == 0 && rank == 0) {                         // the pair acts on one reading of the status
        const uint32_t st = (uint32_t)load_status(a.status);
        c.skip = st;
        st_cluster(at_rank(smem_u32(&c.skip), 1), st);
    }
    const Tiles<FORM> tiles{a, c};
    if (kBoundsCheck) {
        for (int i = tid; i <= a.G; i += kThreads)
            if (a.row_offsets[i] != tiles.off(i)) bounds_fail(a.status);
    }
    if (FORM != kGradW) {                                // a running count of the groups' tiles
        constexpr int kPer = ((kMaxGroups + 1) / 2 + kThreads - 1) / kThreads;
        const int m_tiles = (a.M + tiles.kM - 1) / tiles.kM, n = (a.G + 1) / 2, per = (n + kThreads - 1) / kThreads;
        int mine[kPer], sum = 0;
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            mine[i] = 0;
            const int g = 2 * (tid * per + i);
            if (i < per && g < a.G) {
                const int b0 = tiles.off(g), b1 = tiles.off(g + 1), b2 = tiles.off(min(g + 2, a.G));
                mine[i] = (tiles.parts(b1 - b0) + tiles.parts(b2 - b1)) * m_tiles;
            }
            sum += mine[i];
        }
        int run = sum;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int up = __shfl_up_sync(kFullMask, run, o);
            if (lane >= o) run += up;
        }
        if (lane == 31) c.part[warp] = run;
        __syncthreads();
        run -= sum;
        for (int w = 0; w < warp; ++w) run += c.part[w];
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            if (i < per && tid * per + i < n) c.start[tid * per + i] = run;
            run += mine[i];
        }
        if (tid == kThreads - 1) c.start[n] = run;
    }
    tc_fence_before();
    __syncthreads();
    cluster_sync_all();
    tc_fence_after();
    const uint32_t tmem = c.tmem;
    bool ok = true;                                      // false: a wait ran out
    if (c.skip == 0) {
        Feed feed{c, 0};
        Work w = {};
        if (warp >= 4) {                                 // ------------------------------------------------ results
            regs_up<kManyRegs>();
            const int q = warp & 3, part = (warp - 4) >> 2, et = tid & 127, bar = 1 + part;
            const uint32_t lanes = tmem + ((uint32_t)(q * 32) << 16);
            int buf = 0;
            uint32_t done = 0;
            uint8_t *const own = staging + part * kStaging;
            uint16_t *const st16 = reinterpret_cast<uint16_t *>(own);
            constexpr int kOwn = kCols / 32 / kOutGroups;
            float total[kOwn][32];                       // this thread's sums over the chunks so far, in blocks of 32 columns (rows of the output)
            // A block's first column: the two groups take turns, by 64 where the output has 16 bits and lines of 64 columns.
            auto column = [&](int i) {
                return FORM == kGradW && !a.wide ? ((i >> 1) * kOutGroups + part) * 64 + (i & 1) * 32 : (i * kOutGroups + part) * 32;
            };
            auto load = [&](int i, float(&v)[32]) {
                tmem_ld32(lanes + buf * kCols + column(i), v);
                tmem_wait_ld();
            };
            auto take = [&](int i, bool add) {
                float v[32];
                load(i, v);
#pragma unroll
                for (int j = 0; j < 32; ++j) {
                    total[i][j] = add ? total[i][j] + v[j] : v[j];
                    asm volatile("" : "+f"(total[i][j]));        // before the next reading begins, which needs the registers of v
                }
            };
            auto taken = [&]() {                         // the products may have the buffer again
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(at_rank(smem_u32(&c.sums_empty[buf]), 0));
                buf ^= 1;
                ++done;
            };
            while (ok && feed.next<true>(w, rank, ok)) {
                if (FORM == kGradW && w.kb == 0 && a.add) continue;      // nothing to add
                const int m0 = w.m + (int)rank * (Tiles<FORM>::kM / kPair);          // first feature of this CTA
                const bool one = w.kb <= Tiles<FORM>::kFirst;        // the only chunk stays in tensor memory until the output needs it
                auto prefetch = [&](int s) {             // kGradGate: the saved gate and up of 16 rows, half of a block
                    uint16_t *const st = st16 + (s & 1) * 4096;
                    for (int i = et; i < 256; i += 128) {
                        const int t = column(s >> 1) + (s & 1) * 16 + (i >> 4), f = m0 + (i & 15) * 8;
                        if (t < w.n && f < a.M) {
                            const uint16_t *src = a.gate_up + (size_t)(w.row + t) * 2 * a.M + f;
                            cp_async16(st + i * 8, src);
                            cp_async16(st + 2048 + i * 8, src + a.M);
                        }
                    }
                    asm volatile("cp.async.commit_group;" ::: "memory");
                };
                if constexpr (FORM != kGradW) bar_sync(bar, 128);        // the last tile has left the staging buffers
                if constexpr (FORM == kGradGate) prefetch(0);
                auto arrived = [&]() {
                    ok = __all_sync(kFullMask, mbar_wait(smem_u32(&c.sums_full[buf]), (done >> 1) & 1));
                    tc_fence_after();
                };
                if (w.kb > 0) arrived();
                if (!one) {
#pragma unroll
                    for (int i = 0; i < kOwn; ++i) take(i, false);
                    taken();
                    for (int b = Tiles<FORM>::kFirst; ok && b < w.kb; b += Tiles<FORM>::chunk_blocks(b)) {
                        arrived();
#pragma unroll
                        for (int i = 0; i < kOwn; ++i)
                            if (column(i) < w.n) take(i, true);
                        taken();
                    }
                }
                if constexpr (FORM == kGradW) {
                    if (!ok) break;
                    // 32 rows of 128 bytes per warp at a time, swizzled as TMA reads them: 32 columns of fp32 or 64 of 16 bits
                    uint8_t *const line = own + q * 4096 + lane * 128;
                    auto store = [&](int col) {
                        fence_proxy_async_smem();
                        __syncwarp();
                        if (lane == 0 && m0 + q * 32 < a.M) {
                            const uint32_t src = smem_u32(own + q * 4096);
                            if (a.wide && a.add) tma_add_3d(&map_c, src, w.col + col, m0 + q * 32, w.g);
                            else tma_store_3d(&map_c, src, w.col + col, m0 + q * 32, w.g);
                        }
                        if (lane == 0) bulk_commit();
                    };
                    auto left = [&]() {                  // the rows before have been read
                        if (lane == 0) bulk_wait_read_all();
                        __syncwarp();
                    };
                    auto wide_out = [&](int i, const float(&v)[32]) {
                        left();
#pragma unroll
                        for (int j = 0; j < 8; ++j)
                            *reinterpret_cast<float4 *>(line + ((j ^ (lane & 7)) << 4)) = make_float4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
                        store(column(i));
                    };
                    auto half_out = [&](int i, const float(&v)[32]) {
                        const int h = i & 1;             // half of a line
                        if (h == 0) left();
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            *reinterpret_cast<uint4 *>(line + (((4 * h + j) ^ (lane & 7)) << 4)) =
                                make_uint4(pack16(v[8 * j], v[8 * j + 1], a.f16), pack16(v[8 * j + 2], v[8 * j + 3], a.f16),
                                           pack16(v[8 * j + 4], v[8 * j + 5], a.f16), pack16(v[8 * j + 6], v[8 * j + 7], a.f16));
                        if (h == 1) store(column(i & ~1));
                    };
                    auto more = [&](int i) { return column(a.wide ? i : i & ~1) < w.n; };
                    if (one && !a.wide) {
#pragma unroll
                        for (int i = 0; i < kOwn; ++i)
                            if (more(i)) {
                                float v[32] = {};
                                if (w.kb > 0) load(i, v);
                                half_out(i, v);
                            }
                    } else if (one) {
                        for (int i = 0; i < kOwn && more(i); ++i) {
                            float v[32] = {};
                            if (w.kb > 0) load(i, v);
                            wide_out(i, v);
                        }
                    } else if (a.wide) {
#pragma unroll
                        for (int i = 0; i < kOwn; ++i)
                            if (more(i)) wide_out(i, total[i]);
                    } else {
#pragma unroll
                        for (int i = 0; i < kOwn; ++i)
                            if (more(i)) half_out(i, total[i]);
                    }
                    if (one && w.kb > 0) taken();
                } else {
                    const int F = a.M;
                    if (!(ok = bar_all(bar, 128, ok))) break;
                    auto rows_out = [&](int i, const float(&v)[32]) {
                        const int at = i & 1;            // of the two staging buffers
                        const size_t row0 = (size_t)w.row + column(i);
                        const int rows = min(32, w.n - column(i));
                        if constexpr (FORM == kPlain || FORM == kGradX) {
                            uint16_t *const st = st16 + at * 4096;
#pragma unroll
                            for (int j = 0; j < 32; j += 2) {
                                const uint32_t p = pack16(v[j], v[j + 1], a.f16);
                                st[j * 128 + et] = (uint16_t)p;
                                st[(j + 1) * 128 + et] = (uint16_t)(p >> 16);
                            }
                            bar_sync(bar, 128);
                            for (int i = et; i < rows * 16; i += 128) {
                                const int f = m0 + (i & 15) * 8;
                                if (f < F) *reinterpret_cast<uint4 *>(a.out + (row0 + (i >> 4)) * F + f) = *reinterpret_cast<const uint4 *>(st + i * 8);
                            }
                        } else if constexpr (FORM == kGradGate) {
#pragma unroll
                            for (int h = 0; h < 2; ++h) {
                                if (h * 16 >= rows) break;
                                asm volatile("cp.async.wait_group 0;" ::: "memory");
                                bar_sync(bar, 128);        // everyone's pieces of these rows; the other buffer is free
                                if (h == 0 ? 16 < rows : column(i + 1) < w.n) prefetch(2 * i + h + 1);
                                uint16_t *const st = st16 + h * 4096;
                                uint16_t gs[16], us[16];                 // all read before the first is needed
#pragma unroll
                                for (int j = 0; j < 16; ++j) gs[j] = st[j * 128 + et], us[j] = st[2048 + j * 128 + et];
#pragma unroll
                                for (int j = 0; j < 16; ++j) {
                                    const float gate = wide16(gs[j], a.f16), up = wide16(us[j], a.f16), d = v[16 * h + j];
                                    const Sigmoid sig(gate);
                                    const uint32_t p = pack16(d * up * (sig.s * (1.0f + gate * sig.rest)), d * (gate * sig.s), a.f16);
                                    st[j * 128 + et] = (uint16_t)p;
                                    st[2048 + j * 128 + et] = (uint16_t)(p >> 16);
                                }
                                bar_sync(bar, 128);
                                for (int i = et; i < min(16, rows - 16 * h) * 16; i += 128) {
                                    const int f = m0 + (i & 15) * 8;
                                    if (f < F) {
                                        uint16_t *const dst = a.out + (row0 + 16 * h + (i >> 4)) * 2 * F + f;
                                        *reinterpret_cast<uint4 *>(dst) = *reinterpret_cast<const uint4 *>(st + i * 8);
                                        *reinterpret_cast<uint4 *>(dst + F) = *reinterpret_cast<const uint4 *>(st + 2048 + i * 8);
                                    }
                                }
                            }
                        } else {
                            // The lower 16 lanes hold gates, the upper ones the ups of the same features: each takes half of the rows.
                            const bool up = lane >= 16;
                            const int f = q * 16 + (lane & 15);
                            uint16_t *const act = st16 + at * 2048, *const gu = st16 + 4096;
                            if (a.gate_up) {
                                if (i > 0) bar_sync(bar, 128);           // the rows before have left
#pragma unroll
                                for (int j = 0; j < 32; j += 2) {
                                    const uint32_t p = pack16(v[j], v[j + 1], a.f16);
                                    gu[j * 128 + up * 64 + f] = (uint16_t)p;
                                    gu[(j + 1) * 128 + up * 64 + f] = (uint16_t)(p >> 16);
                                }
                            }
#pragma unroll
                            for (int j = 0; j < 16; j += 2) {
                                float y[2];
#pragma unroll
                                for (int k = 0; k < 2; ++k) {
                                    const float other = __shfl_xor_sync(kFullMask, up ? v[j + k] : v[16 + j + k], 16), own = up ? v[16 + j + k] : v[j + k];
                                    const float gate = up ? other : own;
                                    y[k] = gate * Sigmoid(gate).s * (up ? own : other);
                                }
                                const uint32_t p = pack16(y[0], y[1], a.f16);
                                act[(up * 16 + j) * 64 + f] = (uint16_t)p;
                                act[(up * 16 + j + 1) * 64 + f] = (uint16_t)(p >> 16);
                            }
                            bar_sync(bar, 128);
                            for (int i = et; i < rows * 8; i += 128) {
                                const int f8 = m0 + (i & 7) * 8;
                                if (f8 < F) *reinterpret_cast<uint4 *>(a.out + (row0 + (i >> 3)) * F + f8) = *reinterpret_cast<const uint4 *>(act + i * 8);
                            }
                            if (a.gate_up) {
                                for (int i = et; i < rows * 16; i += 128) {
                                    const int f8 = m0 + (i & 7) * 8;
                                    if (f8 < F) *reinterpret_cast<uint4 *>(a.gate_up + (row0 + (i >> 4)) * 2 * F + (i & 8 ? F : 0) + f8) =
                                                    *reinterpret_cast<const uint4 *>(gu + i * 8);
                                }
                            }
                        }
                    };
                    if (FORM != kGradGate && one) {
                        for (int i = 0; column(i) < w.n; ++i) {
                            float v[32];
                            load(i, v);
                            rows_out(i, v);
                        }
                    } else if constexpr (FORM == kGradGate) {
                        // One copy of the code for all blocks, whose sums move up instead: four of them would have to be fetched at every launch
                        // (a call of 1332 rows took 47 us with them, and 39 so).
#pragma unroll 1
                        for (int i = 0; column(i) < w.n; ++i) {
                            if (one) load(i, total[0]);
                            rows_out(i, total[0]);
#pragma unroll
                            for (int k = 0; k + 1 < kOwn; ++k)
#pragma unroll
                                for (int j = 0; j < 32; ++j) total[k][j] = total[k + 1][j];
                        }
                    } else {
#pragma unroll
                        for (int i = 0; i < kOwn; ++i)
                            if (column(i) < w.n) rows_out(i, total[i]);
                    }
                    if (one) taken();
                }
            }
            if (FORM == kGradW && lane == 0) bulk_wait_all();
        } else {
            regs_down<kFewRegs>();
            if (warp == 0) {                                 // ------------------------------------------------ loads
                if (elect_one()) {
                    int s = 0, used = 0;
                    uint32_t round = 0;
                    while (ok && feed.next<false>(w, rank, ok)) {
                        const int half = w.half, m = w.m + (int)rank * (Tiles<FORM>::kM / kPair);
                        const int n = (FORM == kGradW ? w.col : w.row) + (int)rank * half;
                        const uint32_t bytes = kTileA + (FORM == kGradW || half > 96 ? kTileB : ((half + 31) >> 5) * 4096);
                        for (int b = 0; b < w.kb; ++b) {
                            if (used == kStages && !(ok = mbar_wait(smem_u32(&c.empty[s]), (round & 1) ^ 1))) break;
                            // a block that ends inside 16 rows lands here first and is cleared behind its end
                            const bool clear = FORM == kGradW && b == w.kb - 1 && (w.last & 15) != 0;
                            const uint32_t bar = clear ? smem_u32(&c.landed[s]) : at_rank(smem_u32(&c.full[s]), 0);
                            mbar_arrive_expect(clear ? at_rank(bar, rank) : bar, bytes);
                            Copies<FORM>{map_a, map_b, map_c, a, smem_u32(smem + s * kStageBytes), bar}.block(w, b, m, n, half);
                            if (++s == kStages) s = 0, ++round;
                            used = min(used + 1, kStages);
                        }
                    }
                    // Nothing of the pair may still be on its way to this CTA when it ends.
                    for (int i = 0; ok && i < used; ++i) {
                        s = s == 0 ? kStages - 1 : s - 1;
                        if (s == kStages - 1) --round;
                        ok = mbar_wait(smem_u32(&c.empty[s]), round & 1);
                    }
                    if (!ok) {
                        const unsigned long long t = global_ns();
                        while (global_ns() - t < 1000000ull) {}
                    }
                }
            } else if (warp == 1) {                          // ------------------------------------------------ products
                if (rank == 0) {                             // the whole warp keeps step, one lane issues
                    int s = 0, buf = 0;
                    uint32_t round = 0, done = 0;
                    const uint32_t idesc = mma_desc(a.f16 != 0, 128 * kPair, 0, kAmn, kBmn);
                    const uint64_t desc = smem_desc(smem_u32(smem), 8192);
                    while (ok && feed.next<true>(w, rank, ok)) {
                        const uint32_t id = idesc | (uint32_t)(w.half * kPair >> 4) << 18;
                        for (int b = 0, first = 0, next = 0; b < w.kb; ++b) {
                            if (b == next) {                 // a chunk begins
                                first = b;
                                next = b + Tiles<FORM>::chunk_blocks(b);
                                if (!(ok = __all_sync(kFullMask, mbar_wait(smem_u32(&c.sums_empty[buf]), ((done >> 1) & 1) ^ 1)))) break;
                                tc_fence_after();
                            }
                            const uint32_t d = tmem + buf * kCols;
                            const bool last = b == w.kb - 1, ends = last || b + 1 == next, cleared = FORM == kGradW && last && (w.last & 15) != 0;
                            const uint32_t full = smem_u32(&c.full[s]);
                            if (!(ok = __all_sync(kFullMask, cleared ? mbar_wait<true>(full, round & 1) : mbar_wait(full, round & 1)))) break;
                            tc_fence_after();
                            const uint64_t da = desc + s * (kStageBytes >> 4), db = da + (kTileA >> 4);
                            if (elect_one()) {
                                const int steps = last ? (w.last + 15) >> 4 : kBlockK / 16;
#pragma unroll
                                for (int i = 0; i < kBlockK / 16; ++i)
                                    if (i < steps) tc_mma<kPair>(d, da + i * (kAmn ? 128 : 2), db + i * (kBmn ? 128 : 2), id, b > first || i > 0);
                                tc_commit<kPair>(smem_u32(&c.empty[s]));
                                if (ends) tc_commit<kPair>(smem_u32(&c.sums_full[buf]));
                            }
                            __syncwarp();
                            if (ends) buf ^= 1, ++done;
                            if (++s == kStages) s = 0, ++round;
                        }
                    }
                }
            } else if (warp == 2) {                          // ------------------------------------------------ rows to clear
                if constexpr (FORM == kGradW) {
                    int s = 0;
                    uint32_t seen = 0;                       // parity of landed[s]
                    while (ok && feed.next<true>(w, rank, ok)) {
                        s = (s + max(w.kb - 1, 0)) % kStages;
                        if (w.kb == 0) continue;
                        if (w.last & 15) {
                            if (!(ok = __all_sync(kFullMask, mbar_wait(smem_u32(&c.landed[s]), seen >> s & 1)))) break;
                            seen ^= 1u << s;
                            // rows last to the next multiple of 16, of two blocks of 64 columns of each operand
                            uint8_t *const st = smem + s * kStageBytes + w.last * 128;
                            const int rows = 16 - (w.last & 15);
                            for (int i = lane; i < 4 * rows * 8; i += 32)
                                *reinterpret_cast<uint4 *>(st + i / (rows * 8) * 8192 + i % (rows * 8) * 16) = make_uint4(0, 0, 0, 0);
                            asm volatile("fence.proxy.async;" ::: "memory");
                            __syncwarp();
                            if (lane == 0) mbar_arrive_release(at_rank(smem_u32(&c.full[s]), 0));
                        }
                        if (++s == kStages) s = 0;
                    }
                }
            } else if (warp == 3) {                          // ------------------------------------------------ tiles
                if (elect_one()) {
                    const uint32_t read = at_rank(smem_u32(&c.read), 0);
                    int tile = blockIdx.x / kPair, slot = 0;
                    uint32_t round = 0;
                    auto hand_over = [&]() {
                        if (round > 0 && !(ok = mbar_wait(smem_u32(&c.work_empty[slot]), (round & 1) ^ 1))) return;
                        c.work[slot] = w;
                        mbar_arrive(at_rank(smem_u32(&c.work_full[slot]), rank));
                        if (++slot == kSlots) slot = 0, ++round;
                    };
                    for (uint32_t i = 0; ok; ++i) {
                        const bool some = tile >= 0 && tiles.look_up(tile, w);
                        if (tile >= 0) {                     // ask for the next one, once both CTAs have read the last answer
                            mbar_arrive_expect(at_rank(smem_u32(&c.drawn), rank), 16);
                            if (rank == 0) {
                                if (i > 0 && !(ok = mbar_wait(smem_u32(&c.read), (i & 1) ^ 1))) break;
                                next_cluster_request(smem_u32(&c.answer), smem_u32(&c.drawn));
                            }
                        }
                        if (some) hand_over();
                        if (!ok || tile < 0) break;
                        if (!(ok = mbar_wait(smem_u32(&c.drawn), i & 1))) break;
                        tile = next_cluster_block(smem_u32(&c.answer));
                        if (tile >= 0) tile /= kPair;
                        fence_proxy_async_smem();
                        mbar_arrive(read);
                    }
                    w.g = -1;
                    if (ok) hand_over();
                }
            }
        }
    }
    if (!ok) atomicOr(a.status, EP_STATUS_TIMEOUT);
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    cluster_sync_all();
    tc_fence_after();
    if (warp == 2) tmem_free<kPair>(tmem, 2 * kCols);
    if (a.beside) pdl_wait();
}

// ------------------------------------------------------------------------------------------------------------ host
using Encode = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *, const cuuint64_t *,
                            const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave, CUtensorMapSwizzle,
                            CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
Encode encoder() {
    static const Encode fn = [] {
        void *p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) != cudaSuccess ||
            q != cudaDriverEntryPointSuccess)
            p = nullptr;
        return reinterpret_cast<Encode>(p);
    }();
    return fn;
}

struct Dim {
    uint64_t size, stride;                       // elements
    uint32_t box;
};
// A map over these dimensions, the innermost first (stride 1), in boxes that are 128 bytes wide.
template <int N> bool encode(CUtensorMap *m, const void *p, int bytes, const Dim (&d)[N]) {
    const Encode fn = encoder();
    if (!fn) return false;
    cuuint64_t sizes[N], strides[N];
    cuuint32_t box[N], one[N];
    for (int i = 0; i < N; ++i) {
        sizes[i] = d[i].size;
        if (i) strides[i - 1] = d[i].stride * bytes;
        box[i] = d[i].box;
        one[i] = 1;
    }
    return fn(m, bytes == 4 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_UINT16, N, const_cast<void *>(p), sizes, strides,
              box, one, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}
// Rows of `cols`, of which the sums run along a row (boxes of `box` rows), or down the rows (two blocks of 64 columns by 64
// rows; one box where blocks are whole, which a last one that is not would read beyond the matrix).
bool encode_rows(CUtensorMap *m, const void *p, uint64_t cols, uint64_t rows, uint64_t ld, uint32_t box) {
    return encode(m, p, 2, {{cols, 1, kBlockK}, {rows, ld, box}});
}
bool encode_columns(CUtensorMap *m, const void *p, uint64_t cols, uint64_t rows, uint64_t ld, bool whole) {
    return whole ? encode(m, p, 2, {{64, 1, 64}, {rows, ld, kBlockK}, {cols / 64, 64, 2}}) : encode(m, p, 2, {{cols, 1, 64}, {rows, ld, kBlockK}});
}

template <Form FORM>
int launch_form(const CUtensorMap &ma, const CUtensorMap &mb, const CUtensorMap &mc, const LinearArgs &a, cudaStream_t st) {
    constexpr auto kern = ep_linear_kernel<FORM>;
    const int rc = allow_smem<kern>(kSmem);
    if (rc != EP_OK) return rc;
    static const bool has_regs = [] {                // what the warps take over from one another has to be there, or they would wait for it
        cudaFuncAttributes f;
        return cudaFuncGetAttributes(&f, kern) == cudaSuccess && f.numRegs * kThreads >= kFewRegs * 128 + kManyRegs * kOutGroups * 128;
    }();
    if (!has_regs) return EP_ERR_CUDA;
    constexpr int kM = Tiles<FORM>::kM, kN = Tiles<FORM>::kN;
    const long long m_tiles = (a.M + kM - 1) / kM;
    const long long tiles = m_tiles * (FORM == kGradW ? (long long)a.G * ((a.sum + kN - 1) / kN) : (long long)a.R_max / kN + std::min(a.G, a.R_max));
    cudaLaunchConfig_t cfg = {};
    if (tiles > INT_MAX / kPair) return EP_ERR_INVALID_ARG;
    cfg.gridDim = dim3((unsigned)std::max(1ll, tiles) * kPair);        // the most there can be; clusters that run take them in turn
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = kSmem;
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = kPair;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return launch_result(cudaLaunchKernelEx(&cfg, kern, ma, mb, mc, a));
}

// Sizes and pointers common to both calls.
bool linear_ok(const ep_layout_t *L, int K, int N, int dtype) {
    return layout_ok(L) && hidden_ok(K) && N >= 16 && N <= kMaxN && N % 16 == 0 && (dtype == EP_BF16 || dtype == EP_F16);
}
bool stride_ok(long long ld, int cols) { return ld >= cols && ld % 8 == 0 && ld < (1ll << 31); }

LinearArgs linear_args(const ep_layout_t *L, int dtype) {
    LinearArgs a = {};
    a.row_offsets = L->row_offsets;
    a.status = L->status;
    a.G = L->E + L->fused_shared;
    a.R_max = layout_rows(L);
    a.f16 = dtype == EP_F16;
    return a;
}

}  // namespace
}  // namespace ep

using namespace ep;

extern "C" int ep_expert_linear(const void *x, long long x_stride, const void *w, int in_features, int out_rows, int dtype, int swiglu,
                                const ep_layout_t *L, void *out, void *gate_up, void *stream) {
    EP_NVTX_RANGE("ep_expert_linear");
    const int K = in_features, N = out_rows;
    if (!linear_ok(L, K, N, dtype) || !stride_ok(x_stride, K) || (swiglu != 0 && swiglu != 1)) return EP_ERR_INVALID_ARG;
    if (swiglu ? N % 32 != 0 : gate_up != nullptr) return EP_ERR_INVALID_ARG;
    for (const void *p : {x, w, (const void *)out, (const void *)gate_up})
        if (!aligned16(p)) return EP_ERR_INVALID_ARG;
    if (L->T == 0) return EP_OK;
    if (!x || !w || !out) return EP_ERR_INVALID_ARG;
    LinearArgs a = linear_args(L, dtype);
    a.M = swiglu ? N / 2 : N;
    a.sum = K;
    a.out = (uint16_t *)out;
    a.gate_up = (uint16_t *)gate_up;
    const uint64_t k = K, f = a.M, g = a.G, each = (uint64_t)N * K;
    CUtensorMap ma, mb, mc;
    bool ok = encode_rows(&mb, x, K, a.R_max, x_stride, 128) && encode_rows(&mc, x, K, a.R_max, x_stride, 32);
    if (!swiglu) ok = ok && encode(&ma, w, 2, {{k, 1, kBlockK}, {(uint64_t)N, k, 128}, {g, each, 1}});
    else ok = ok && encode(&ma, w, 2, {{k, 1, kBlockK}, {16, k, 16}, {2, f * k, 2}, {f / 16, 16 * k, 4}, {g, each, 1}});     // 16 gates, their 16 ups
    if (!ok) return EP_ERR_CUDA;
    cudaStream_t st = as_stream(stream);
    return swiglu ? launch_form<kGlu>(ma, mb, mc, a, st) : launch_form<kPlain>(ma, mb, mc, a, st);
}

extern "C" int ep_expert_linear_bwd(const void *grad, long long grad_stride, const void *x, long long x_stride, const void *w,
                                    int in_features, int out_rows, int dtype, const void *gate_up, const ep_layout_t *L, void *grad_x,
                                    void *grad_w, int grad_w_dtype, int accumulate, void *stream) {
    EP_NVTX_RANGE("ep_expert_linear_bwd");
    const int K = in_features, N = out_rows;
    if (!linear_ok(L, K, N, dtype) || !stride_ok(grad_stride, N) || (!grad_x && !grad_w)) return EP_ERR_INVALID_ARG;
    if (gate_up && !grad_x) return EP_ERR_INVALID_ARG;
    if (grad_w) {
        if (!stride_ok(x_stride, K) || (accumulate != 0 && accumulate != 1)) return EP_ERR_INVALID_ARG;
        if (grad_w_dtype != dtype && grad_w_dtype != EP_F32) return EP_ERR_INVALID_ARG;
        if (accumulate && grad_w_dtype != EP_F32) return EP_ERR_INVALID_ARG;
    }
    for (const void *p : {grad, x, w, gate_up, (const void *)grad_x, (const void *)grad_w})
        if (!aligned16(p)) return EP_ERR_INVALID_ARG;
    if (L->T > 0 && (!grad || (grad_x && !w) || (grad_w && !x))) return EP_ERR_INVALID_ARG;
    LinearArgs a = linear_args(L, dtype);
    cudaStream_t st = as_stream(stream);
    CUtensorMap ma, mb, mc;
    const uint64_t k = K, n = N, g = a.G, each = n * k;
    if (grad_x && L->T > 0) {
        a.M = K;
        a.sum = N;
        a.out = (uint16_t *)grad_x;
        a.gate_up = (uint16_t *)const_cast<void *>(gate_up);
        a.whole_a = K % 64 == 0;
        const bool ok = a.whole_a ? encode(&ma, w, 2, {{64, 1, 64}, {n, k, kBlockK}, {k / 64, 64, 2}, {g, each, 1}})
                                  : encode(&ma, w, 2, {{k, 1, 64}, {n, k, kBlockK}, {g, each, 1}});
        if (!ok || !encode_rows(&mb, grad, N, a.R_max, grad_stride, 128) || !encode_rows(&mc, grad, N, a.R_max, grad_stride, 32)) return EP_ERR_CUDA;
        const int rc = gate_up ? launch_form<kGradGate>(ma, mb, mc, a, st) : launch_form<kGradX>(ma, mb, mc, a, st);
        if (rc != EP_OK) return rc;
    }
    if (!grad_w) return EP_OK;
    a.beside = grad_x && L->T > 0;
    a.M = N;
    a.sum = K;
    a.wide = grad_w_dtype == EP_F32;
    a.add = accumulate;
    a.whole_a = N % 64 == 0;
    a.whole_b = K % 64 == 0;
    // without a token there is nothing to load, and the maps only need a valid address
    const bool none = L->T == 0;
    const uint64_t rows = none ? 1 : a.R_max;
    if (!encode_columns(&ma, none ? grad_w : grad, n, rows, none ? n : grad_stride, a.whole_a) ||
        !encode_columns(&mb, none ? grad_w : x, k, rows, none ? k : x_stride, a.whole_b) ||
        !encode(&mc, grad_w, a.wide ? 4 : 2, {{k, 1, a.wide ? 32u : 64u}, {n, k, 32}, {g, each, 1}}))
        return EP_ERR_CUDA;
    return launch_form<kGradW>(ma, mb, mc, a, st);
}
