// ep_norm.cu -- layer norm and RMS norm over the rows of a token matrix, in front of the router
// and the dispatch, and their backward pass with the reduction of the parameters' gradients.
//
//   forward   xh = (x - mean) * rstd, y = xh * w + b; mean = sum(x)/H,
//             rstd = 1/sqrt(sum((x - mean)^2)/H + eps)  (RMS: mean = 0)
//   backward  a = g * w, dx = rstd * (a - mean(a) - xh * mean(a * xh))  (RMS: no mean(a)),
//             dw = sum over rows of g * xh, db = sum over rows of g
//
// Statistics and sums are fp32.  The variance is summed over (x - mean) in a second pass over
// registers, which also corrects the mean, so rows with a large mean lose nothing.  HBM is the floor of both passes: each row is
// read once and written once.  4096 x 7168 bf16 forward: RMS 21.5 us, 0.82 of the measured copy bandwidth with the launch, layer
// norm 28.1 us, 0.63 (the corrected mean is another pass over registers and a second sum);
// 32768 x 7168 bf16 backward: 292 us, 0.72, where issue and the row sums at 14 warps per SM bound it; single rows: 2.0 us.
//
// Many rows: one CTA per SM whose threads form groups, a group holding 32 elements of a row per thread, and
// looping over rows.  Rows arrive in a ring of shared-memory stages by asynchronous copies, so that the
// bytes in flight (about 170 KB per SM) do not depend on registers, and each group's barriers leave the
// other groups running.
#include "ep_host.h"
#include "ep_types.cuh"

namespace ep {
namespace {

constexpr int kFwdEpt = 32, kBwdEpt = 32;     // elements of a row per thread in the pipelined kernels
constexpr int kFwdThreads = 672, kBwdThreads = 512;
constexpr int kBwdStages = 3;
template <typename T> constexpr int kFwdStages = sizeof(T) == 4 ? 3 : 4;
constexpr int kSharedBytes = 226 * 1024; // shared memory for stages and parameters
constexpr int kBwdMaxH = 8192;
constexpr int kPartials = 304;           // rows of partial column sums a workspace has room for
// Few rows.  Forward: one CTA per row while the rows have at most kResidentPerSm threads per SM.  us against the pipelined
// kernel, bf16, layer norm / RMS: H = 256, T = 8000 5.9 / 5.7 against 7.7 / 5.6, T = 9500 6.5 / 6.5 against 7.7 / 5.7; H = 2048,
// T = 1000 4.6 / 3.4 against 5.0 / 4.3, T = 1216 5.3 / 3.8 against 4.9 / 4.3; H = 7168, T = 152 3.5 / 2.4 against 5.3 / 4.4,
// T = 304 6.2 / 4.1 against 5.5 / 4.4, T = 347 8.2 / 5.5 against 5.5 / 4.5; H = 16384, four vectors per thread, T = 300
// 5.6 / 4.3 against 7.7 / 5.9 (eight, which spill: 9.1 / 6.7).
// Backward: one launch that reads x and g twice, up to few_bwd_rows rows.  us against the pipelined kernel, bf16: H = 256, T = 400
// 5.6 against 6.2, T = 456 6.8 against 6.2; H = 2048, T = 800 11.3 against 11.6, T = 1000 13.7 against 11.7; H = 8192, T = 800
// 21.4 against 25.2, T = 1500 37.4 against 31.5.  fp32: H = 2048, T = 300 6.8 against 7.8, T = 400 8.8 against 7.9; H = 4096,
// T = 456 12.4 against 13.4; H = 8192, T = 456 22.6 against 24.6, T = 600 28.2 against 27.2.
constexpr int kResidentPerSm = 1696;
constexpr int few_bwd_rows(int H, int element) {
    return element == 2 ? (H > 256 ? 800 : 400) : (H >= 4096 ? 456 : 340);
}

constexpr int round_up(int n, int to) { return (n + to - 1) / to * to; }

// Sum of one or two values over the threads of a group of G threads (a whole number of warps); ty is the
// group's index in its CTA and names its barrier (1 to 15: a CTA has at most 15 groups of several warps).  `red` has
// room for 32 values, zero past the group's warps, and is not written again before the next barrier of the group.
__device__ __forceinline__ void group_barrier(int G, int ty) {
    if (G == 32) __syncwarp();
    else asm volatile("bar.sync %0, %1;" ::"r"(ty + 1), "r"(G) : "memory");
}
__device__ __forceinline__ float group_sum(float a, float *red, int G, int ty) {
    a = warp_sum(a);
    if (G == 32) return a;
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = a;
    group_barrier(G, ty);
    float s = 0.0f;
    for (int i = 0; i < (G >> 5); i += 4) {
        const float4 v = *reinterpret_cast<const float4 *>(red + i);
        s += (v.x + v.y) + (v.z + v.w);
    }
    return s;
}
__device__ __forceinline__ float2 group_sum2(f32x2 a, f32x2 *red, int G, int ty) {
    // the lower half of a warp adds up the first values, the upper half the second ones
    const int lane = threadIdx.x & 31, upper = lane >> 4;
    const float2 p = f2_get(a);
    float v = upper ? p.y : p.x;
    v += __shfl_xor_sync(kFullMask, upper ? p.x : p.y, 16);
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) v += __shfl_xor_sync(kFullMask, v, o);
    if (G == 32) {
        const float other = __shfl_xor_sync(kFullMask, v, 16);
        return upper ? make_float2(other, v) : make_float2(v, other);
    }
    if ((lane & 15) == 0) reinterpret_cast<float *>(red + (threadIdx.x >> 5))[upper] = v;
    group_barrier(G, ty);
    f32x2 s = f2(0.0f, 0.0f);
    for (int i = 0; i < (G >> 5); i += 2) {
        const ulonglong2 v = *reinterpret_cast<const ulonglong2 *>(red + i);
        s = f2_add(s, f2_add(v.x, v.y));
    }
    return f2_get(s);
}

// How the rows of all matrices of a call lie.
//   kAligned  on 16-byte boundaries;
//   kShifted  off them, row for row by the same amount in every matrix (dense matrices of any width): work is by the
//             aligned 16-byte pieces that cover a row, the first and last of them in part.  The amount repeats every
//             `period` rows, and a group takes rows that share one, so its columns stay the same;
//   kAny      anything else: element by element.
enum Lay { kAligned, kShifted, kAny };

// How a thread of a pipelined kernel holds its EPT elements of a row: in units of E elements as E/2 pairs.  Unit i is
// piece tid + i * G of 16 bytes (kAny: the elements tid + (i * E + j) * G).  Units past the row's end read its last piece or
// element instead, which costs no branch (another thread may still be copying it: any value does); what lies outside the
// row is left out of sums (add) and not stored.
template <typename T, int EPT, int LAY> struct Units {
    static constexpr int VEC = 16 / (int)sizeof(T), E = LAY == kAny ? 4 : VEC, N = EPT / E;
    int tid, G, H, shift;                // shift: elements by which rows follow a 16-byte boundary
    __device__ __forceinline__ int first(int i) const { return (tid + i * G) * VEC - shift; }   // column of the unit's first element
    __device__ __forceinline__ int col(int i, int j) const { return LAY == kAny ? tid + (i * E + j) * G : first(i) + j; }
    __device__ __forceinline__ bool has(int i, int j) const {
        const int c = col(i, LAY == kAligned ? 0 : j);
        return c < H && (LAY != kShifted || c >= 0);
    }
    __device__ __forceinline__ bool whole(int i) const {            // not for kAny
        return LAY == kAligned ? has(i, 0) : first(i) >= 0 && first(i) + VEC <= H;
    }
    // row: where column 0 is (kAny), or the piece that column 0 is in
    template <typename P> __device__ __forceinline__ void load(const P *row, int i, f32x2 (&v)[E / 2]) const {
        float f[E];
        if constexpr (LAY != kAny) {
            ld_pack<P, VEC>(row + min(tid + i * G, (H + shift - 1) / VEC) * VEC).unpack(f);
        } else {
#pragma unroll
            for (int j = 0; j < E; ++j) f[j] = to_f32(row[min(col(i, j), H - 1)]);
        }
#pragma unroll
        for (int j = 0; j < E / 2; ++j) v[j] = f2(f[2 * j], f[2 * j + 1]);
    }
    __device__ __forceinline__ void store(T *row, int i, const f32x2 (&v)[E / 2]) const {      // row: where column 0 is
        float f[E];
#pragma unroll
        for (int j = 0; j < E / 2; ++j) {
            const float2 p = f2_get(v[j]);
            f[2 * j] = p.x;
            f[2 * j + 1] = p.y;
        }
        bool vector = false;
        if constexpr (LAY != kAny) {
            vector = whole(i);
            if (vector) st_pack_stream<T, VEC>(row + first(i), f);
        }
        if constexpr (LAY != kAligned) {
#pragma unroll
            for (int j = 0; j < E; ++j)
                if (!vector && has(i, j)) row[col(i, j)] = from_f32<T>(f[j]);
        }
    }
    __device__ __forceinline__ void store_sums(float *row, int i, const f32x2 (&v)[E / 2]) const {
#pragma unroll
        for (int j = 0; j < E / 2; ++j) {
            const float2 p = f2_get(v[j]);
            if (has(i, 2 * j)) row[col(i, 2 * j)] = p.x;
            if (has(i, 2 * j + 1)) row[col(i, 2 * j + 1)] = p.y;
        }
    }
    // sum + the squares of the unit's values that are in the row
    __device__ __forceinline__ f32x2 add_squares(f32x2 sum, int i, const f32x2 (&v)[E / 2]) const {
        bool done = false;
        if constexpr (LAY != kAny) {
            done = whole(i);
            if (done) {
                f32x2 s = f2_mul(v[0], v[0]);
#pragma unroll
                for (int j = 1; j < E / 2; ++j) s = f2_fma(v[j], v[j], s);
                sum = f2_add(sum, s);
            }
        }
        if constexpr (LAY != kAligned) {
            if (!done)
#pragma unroll
                for (int j = 0; j < E / 2; ++j) {
                    const float2 p = f2_get(f2_mul(v[j], v[j]));
                    sum = f2_add(sum, f2(has(i, 2 * j) ? p.x : 0.0f, has(i, 2 * j + 1) ? p.y : 0.0f));
                }
        }
        return sum;
    }
    // sum + the unit's values that are in the row
    __device__ __forceinline__ f32x2 add(f32x2 sum, int i, const f32x2 (&v)[E / 2]) const {
        bool done = false;
        if constexpr (LAY != kAny) {
            done = whole(i);
            if (done) {
                f32x2 s = v[0];
#pragma unroll
                for (int j = 1; j < E / 2; ++j) s = f2_add(s, v[j]);
                sum = f2_add(sum, s);
            }
        }
        if constexpr (LAY != kAligned) {
            if (!done)
#pragma unroll
                for (int j = 0; j < E / 2; ++j) {
                    const float2 p = f2_get(v[j]);
                    sum = f2_add(sum, f2(has(i, 2 * j) ? p.x : 0.0f, has(i, 2 * j + 1) ? p.y : 0.0f));
                }
        }
        return sum;
    }
};

// The rows of a group: gi-th of n groups.
struct Rows {
    int first, step;
    __device__ __forceinline__ Rows(int gi, int n, int period) {
        const int kind = gi % period, k = gi / period;              // groups of a kind take the rows of that kind in turn
        first = kind + k * period;
        step = (n - kind + period - 1) / period * period;
    }
};

// A matrix whose rows a group copies to shared memory as the aligned 16-byte pieces that cover them; a piece that would
// reach outside the matrix, before its first or after its last row, is copied by elements.  A thread copies pieces tid,
// tid + G, ...: those it will read itself, so that it has only its own copies to wait for (kAny: the group meets at a
// barrier).
template <typename T, int EPT, int LAY> struct RowSource {
    static constexpr int VEC = 16 / (int)sizeof(T);
    const T *base, *end;                 // the matrix: end is past the last row's last element
    long long ld;
    int H;
    __device__ __forceinline__ RowSource(const T *m, long long ld_, int rows, int H_)
        : base(m), end(m + (size_t)(rows - 1) * ld_ + H_), ld(ld_), H(H_) {}
    static __host__ __device__ __forceinline__ int stage_bytes(int H) { return ((int)sizeof(T) * H + 15) / 16 * 16 + (LAY == kAligned ? 0 : 16); }
    __device__ __forceinline__ int shift(int row) const {            // elements by which a row follows a 16-byte boundary
        return LAY == kAligned ? 0 : (int)(reinterpret_cast<uintptr_t>(base + (size_t)row * ld) & 15u) / (int)sizeof(T);
    }
    __device__ __forceinline__ void copy(int row, char *stage, int tid, int G) const {
        const unsigned to = (unsigned)__cvta_generic_to_shared(stage) + tid * 16;
        const int before = shift(row);
        const T *from = base + (size_t)row * ld - before + tid * VEC;
        if constexpr (LAY == kAligned) {
#pragma unroll
            for (int i = 0; i < EPT / VEC; ++i)
                if ((tid + i * G) * VEC < H)
                    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to + i * G * 16), "l"(from + i * G * VEC) : "memory");
        } else {
            const int pieces = (before + H + VEC - 1) / VEC;
            for (int i = 0; tid + i * G < pieces; ++i, from += G * VEC) {
                if (from >= base && from + VEC <= end) {
                    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to + i * G * 16), "l"(from) : "memory");
                } else {
                    for (int j = 0; j < VEC; ++j)
                        if (from + j >= base && from + j < end) reinterpret_cast<T *>(stage)[(tid + i * G) * VEC + j] = from[j];
                }
            }
        }
    }
};

// Shared memory of a parameter.
template <typename W> constexpr __host__ __device__ int param_bytes(int H) { return ((int)sizeof(W) * H + 15) / 16 * 16; }
// Copies of the parameters: one for all groups, or one behind each group's own boundary.
constexpr __host__ __device__ int param_copies(int lay, int R) { return lay == kShifted ? R : 1; }

__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N> __device__ __forceinline__ void copies_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

// ---------------------------------------------------------------------------------------
// forward
// ---------------------------------------------------------------------------------------
// The mean that the first pass over a row gives is off by the rounding of its sum.  The second pass also sums d = x - mean,
// whose own mean delta is what the first one missed, and the roundings of the d's, up to 2^-24 of their mean magnitude (all
// to one side where x has few digits).  The variance is corrected by it; the mean and d are too where delta is more than those
// can be, twice that of the root mean square of d.  A constant row has d = delta exactly, and so y = bias.
__device__ __forceinline__ bool mean_missed(float delta, float mean_square) { return delta * delta > 0x1p-46f * mean_square; }

// The variance about the corrected mean from the mean square about the first one; NaN stays NaN.
__device__ __forceinline__ float centred_var(float mean_square, float delta) {
    const float v = fmaf(-delta, delta, mean_square);
    return v < 0.0f ? 0.0f : v;
}

template <typename T, typename W, int LAY>
__global__ void __launch_bounds__(kFwdThreads, 1)
ep_norm_kernel(const T *__restrict__ x, long long ldx, const W *__restrict__ w, const W *__restrict__ b,
               int rows, int H, float eps, int rms, int period, T *__restrict__ y, float *__restrict__ mean_out,
               float *__restrict__ rstd_out) {
    constexpr int D = kFwdStages<T>;
    using U = Units<T, kFwdEpt, LAY>;
    extern __shared__ __align__(16) char smem[];                    // [copy][weight, bias], [group][stage]
    __shared__ __align__(16) float s_red[2][32][4];                 // a group's values, or pairs of values, lie in whole rows
    const int G = blockDim.x, R = blockDim.y, tid = threadIdx.x, ty = threadIdx.y;
    if (ty * G + tid < 128) s_red[0][0][ty * G + tid] = s_red[1][0][ty * G + tid] = 0.0f;
    pdl_begin();
    const RowSource<T, kFwdEpt, LAY> src(x, ldx, rows, H);
    const Rows mine(blockIdx.x * R + ty, gridDim.x * R, period);
    const int step = mine.step, shift = LAY == kShifted && mine.first < rows ? src.shift(mine.first) : 0;
    const U un{tid, G, H, shift};
    const int bytes = src.stage_bytes(H), params = param_bytes<W>(H + 2 * U::VEC);
    char *stages = smem + param_copies(LAY, R) * 2 * params + (size_t)ty * D * bytes;
    int row = mine.first;
#pragma unroll
    for (int i = 0; i < D - 1; ++i) {
        if (row + i * step < rows) src.copy(row + i * step, stages + i * bytes, tid, G);
        copies_commit();
    }
    const float h = (float)H, inv_h = 1.0f / h;
    // the parameters, as far behind a 16-byte boundary as the group's rows (L1 is too small beside the stages to keep them)
    W *s_w = reinterpret_cast<W *>(smem + (LAY == kShifted ? ty : 0) * 2 * params), *s_b = s_w + params / sizeof(W);
#pragma unroll 8
    for (int c = LAY == kShifted ? tid : ty * G + tid; c < H; c += LAY == kShifted ? G : R * G) {
        s_w[c + shift] = w[c];
        if (b) s_b[c + shift] = b[c];
    }
    const int red_rows = ((G >> 5) + 3) / 4;
    float *red0 = &s_red[0][ty * red_rows][0], *red1 = &s_red[1][ty * red_rows][0];
    f32x2 *red2 = reinterpret_cast<f32x2 *>(&s_red[1][ty * (((G >> 5) + 1) / 2)][0]);   // red1's place, for a layer norm
    __syncthreads();
    for (int at = 0, buf = 0; row < rows; row += step, at = at + 1 == D ? 0 : at + 1, buf ^= 1) {
        copies_wait<D - 2>();
        if (LAY == kAny) group_barrier(G, ty);
        // the stage before this one was read before the group's last barrier (or by this thread alone)
        if (row + (D - 1) * step < rows) src.copy(row + (D - 1) * step, stages + (at == 0 ? D - 1 : at - 1) * bytes, tid, G);
        copies_commit();
        const T *s_row = reinterpret_cast<const T *>(stages + at * bytes) + (LAY == kAny ? src.shift(row) : 0);
        f32x2 d[U::N][U::E / 2];
#pragma unroll
        for (int i = 0; i < U::N; ++i) un.load(s_row, i, d[i]);
        float mean = 0.0f, rstd;
        if (!rms) {
            f32x2 s = f2(0.0f, 0.0f);
#pragma unroll
            for (int i = 0; i < U::N; ++i) s = un.add(s, i, d[i]);
            const float2 p = f2_get(s);
            mean = group_sum(p.x + p.y, red0, G, ty) / h;
            const f32x2 neg = f2(-mean, -mean);
#pragma unroll
            for (int i = 0; i < U::N; ++i)
#pragma unroll
                for (int j = 0; j < U::E / 2; ++j) d[i][j] = f2_add(d[i][j], neg);
        }
        f32x2 q = f2(0.0f, 0.0f);
#pragma unroll
        for (int i = 0; i < U::N; ++i) q = un.add_squares(q, i, d[i]);
        const float2 p = f2_get(q);
        if (rms) {
            rstd = __frsqrt_rn(group_sum(p.x + p.y, buf ? red0 : red1, G, ty) / h + eps);
        } else {
            f32x2 s = f2(0.0f, 0.0f);
#pragma unroll
            for (int i = 0; i < U::N; ++i) s = un.add(s, i, d[i]);
            const float2 r = f2_get(s), t = group_sum2(f2(r.x + r.y, p.x + p.y), red2, G, ty);
            float delta = t.x * inv_h;
            const float mean_square = t.y / h;
            rstd = __frsqrt_rn(centred_var(mean_square, delta) + eps);
            if (mean_missed(delta, mean_square)) {
                delta = t.x / h;
                const f32x2 neg = f2(-delta, -delta);
#pragma unroll
                for (int i = 0; i < U::N; ++i)
#pragma unroll
                    for (int j = 0; j < U::E / 2; ++j) d[i][j] = f2_add(d[i][j], neg);
                mean += delta;
            }
        }
        if (tid == 0) {
            if (!rms) mean_out[row] = mean;
            rstd_out[row] = rstd;
        }
        const f32x2 r2 = f2(rstd, rstd);
        T *yr = y + (size_t)row * H;
#pragma unroll
        for (int i = 0; i < U::N; ++i) {
            f32x2 u[U::E / 2];
            un.load(s_w, i, u);
#pragma unroll
            for (int j = 0; j < U::E / 2; ++j) d[i][j] = f2_mul(d[i][j], r2);
            if (b) {
                f32x2 c[U::E / 2];
                un.load(s_b, i, c);
#pragma unroll
                for (int j = 0; j < U::E / 2; ++j) d[i][j] = f2_fma(d[i][j], u[j], c[j]);
            } else {
#pragma unroll
                for (int j = 0; j < U::E / 2; ++j) d[i][j] = f2_mul(d[i][j], u[j]);
            }
            un.store(yr, i, d[i]);
        }
    }
}

// Few rows, or rows wider than the pipelined kernel's: one CTA per row, NV vectors per thread straight from memory.
template <typename T, typename W, int VEC, int NV>
__global__ void __launch_bounds__(1024, 1)
ep_norm_row_kernel(const T *__restrict__ x, long long ldx, const W *__restrict__ w, const W *__restrict__ b,
                   int H, float eps, int rms, int one_wave, T *__restrict__ y, float *__restrict__ mean_out,
                   float *__restrict__ rstd_out) {
    __shared__ __align__(16) float s_red[32];
    __shared__ __align__(16) f32x2 s_red2[32];
    if (threadIdx.x < 32) {
        s_red[threadIdx.x] = 0.0f;
        s_red2[threadIdx.x] = f2(0.0f, 0.0f);
    }
    __syncthreads();
    pdl_begin_if(one_wave);
    const int G = blockDim.x, tid = threadIdx.x, row = blockIdx.x, nv = H / VEC;
    const float h = (float)H, inv_h = 1.0f / h;
    const T *xr = x + (size_t)row * ldx;
    float d[NV][VEC];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int v = tid + i * G;
        if (v < nv) {
            ld_pack_stream<T, VEC>(xr + (size_t)v * VEC).unpack(d[i]);
        } else {
#pragma unroll
            for (int j = 0; j < VEC; ++j) d[i][j] = 0.0f;
        }
    }
    Pack<W, VEC> w0, b0;                 // one vector per thread: the parameters are on their way while the row is reduced
    if (NV == 1 && tid < nv) {
        w0 = ld_pack<W, VEC>(w + (size_t)tid * VEC);
        if (b) b0 = ld_pack<W, VEC>(b + (size_t)tid * VEC);
    }
    float mean = 0.0f;
    if (!rms) {
        float s = 0.0f;
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int j = 0; j < VEC; ++j) s += d[i][j];
        mean = group_sum(s, s_red, G, 0) / h;
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int j = 0; j < VEC; ++j) d[i][j] = tid + i * G < nv ? d[i][j] - mean : 0.0f;
    }
    float q = 0.0f, sd = 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
            q = fmaf(d[i][j], d[i][j], q);
            sd += d[i][j];
        }
    float rstd, delta = 0.0f;
    if (rms) {
        rstd = __frsqrt_rn(group_sum(q, s_red, G, 0) / h + eps);
    } else {
        const float2 t = group_sum2(f2(sd, q), s_red2, G, 0);
        delta = t.x * inv_h;
        const float mean_square = t.y / h;
        rstd = __frsqrt_rn(centred_var(mean_square, delta) + eps);
        delta = mean_missed(delta, mean_square) ? t.x / h : 0.0f;
        mean += delta;
    }
    if (tid == 0) {
        if (!rms) mean_out[row] = mean;
        rstd_out[row] = rstd;
    }
    T *yr = y + (size_t)row * H;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int v = tid + i * G;
        if (v < nv) {
            float o[VEC];
            if (NV > 1) w0 = ld_pack<W, VEC>(w + (size_t)v * VEC);
            w0.unpack(o);
            float c[VEC];
            if (b) {
                if (NV > 1) b0 = ld_pack<W, VEC>(b + (size_t)v * VEC);
                b0.unpack(c);
            }
#pragma unroll
            for (int j = 0; j < VEC; ++j) {
                const float n = (d[i][j] - delta) * rstd;
                o[j] = b ? fmaf(n, o[j], c[j]) : n * o[j];
            }
            st_pack_stream<T, VEC>(yr + (size_t)v * VEC, o);
        }
    }
}

// ---------------------------------------------------------------------------------------
// backward, rows of up to kBwdMaxH elements: x and g are read once for dx, dw and db.  A thread keeps the sums of
// its columns over all the group's rows in registers; groups are joined per CTA in shared memory, CTAs by
// ep_norm_cols_kernel, both in a fixed order.
// ---------------------------------------------------------------------------------------
template <typename T, typename W, int LAY>
__global__ void __launch_bounds__(kBwdThreads, 1)
ep_norm_bwd_kernel(const T *__restrict__ g, long long ldg, const T *__restrict__ x, long long ldx,
                   const W *__restrict__ w, const float *__restrict__ mean_in,
                   const float *__restrict__ rstd_in, int rows, int H, int rms, int want_db, int period,
                   T *__restrict__ dx, float *__restrict__ part) {
    constexpr int D = kBwdStages;
    using U = Units<T, kBwdEpt, LAY>;
    extern __shared__ __align__(16) char smem[];                    // [copy] weight, [group][stage][x, g]; at the end [group][2][H] sums
    __shared__ __align__(16) f32x2 s_red[2][32][2];                 // a group's values lie in whole rows of 2
    const int G = blockDim.x, R = blockDim.y, tid = threadIdx.x, ty = threadIdx.y;
    if (ty * G + tid < 64) s_red[0][0][ty * G + tid] = s_red[1][0][ty * G + tid] = f2(0.0f, 0.0f);
    pdl_begin();
    const RowSource<T, kBwdEpt, LAY> sx(x, ldx, rows, H), sg(g, ldg, rows, H);
    const Rows mine(blockIdx.x * R + ty, gridDim.x * R, period);
    const int step = mine.step, shift = LAY == kShifted && mine.first < rows ? sx.shift(mine.first) : 0;
    const U un{tid, G, H, shift};
    const int bytes = sx.stage_bytes(H), params = param_bytes<W>(H + 2 * U::VEC);
    char *stages = smem + param_copies(LAY, R) * params + (size_t)ty * D * 2 * bytes;
    W *s_w = reinterpret_cast<W *>(smem + (LAY == kShifted ? ty : 0) * params);
    int row = mine.first;
#pragma unroll
    for (int i = 0; i < D - 1; ++i) {
        if (row + i * step < rows) {
            sx.copy(row + i * step, stages + 2 * i * bytes, tid, G);
            sg.copy(row + i * step, stages + (2 * i + 1) * bytes, tid, G);
        }
        copies_commit();
    }
#pragma unroll 8
    for (int c = LAY == kShifted ? tid : ty * G + tid; c < H; c += LAY == kShifted ? G : R * G) s_w[c + shift] = w[c];
    f32x2 dw[U::N][U::E / 2], db[U::N][U::E / 2];
#pragma unroll
    for (int i = 0; i < U::N; ++i)
#pragma unroll
        for (int j = 0; j < U::E / 2; ++j) dw[i][j] = db[i][j] = f2(0.0f, 0.0f);
    const float h = (float)H;
    float next_mean = 0.0f, next_rstd = 0.0f;                       // a row ahead
    if (row < rows) {
        if (!rms) next_mean = mean_in[row];
        next_rstd = rstd_in[row];
    }
    f32x2 *red[2] = {&s_red[0][ty * (((G >> 5) + 1) / 2)][0], &s_red[1][ty * (((G >> 5) + 1) / 2)][0]};
    __syncthreads();
    for (int at = 0, buf = 0; row < rows; row += step, at = at + 1 == D ? 0 : at + 1, buf ^= 1) {
        const float mean = next_mean, rstd = next_rstd;
        if (row + step < rows) {
            if (!rms) next_mean = mean_in[row + step];
            next_rstd = rstd_in[row + step];
        }
        copies_wait<D - 2>();
        if (LAY == kAny) group_barrier(G, ty);
        // the stage before this one was read to the end before (kAny: before the barrier just passed)
        if (row + (D - 1) * step < rows) {
            char *to = stages + 2 * (at == 0 ? D - 1 : at - 1) * bytes;
            sx.copy(row + (D - 1) * step, to, tid, G);
            sg.copy(row + (D - 1) * step, to + bytes, tid, G);
        }
        copies_commit();
        const T *xr = reinterpret_cast<const T *>(stages + 2 * at * bytes) + (LAY == kAny ? sx.shift(row) : 0);
        const T *gr = reinterpret_cast<const T *>(stages + (2 * at + 1) * bytes) + (LAY == kAny ? sg.shift(row) : 0);
        const f32x2 neg_mean = f2(-mean, -mean), r2 = f2(rstd, rstd);
        f32x2 sa = f2(0.0f, 0.0f), sax = sa;
#pragma unroll
        for (int i = 0; i < U::N; ++i) {
            f32x2 xe[U::E / 2], ge[U::E / 2], u[U::E / 2];
            un.load(xr, i, xe);
            un.load(gr, i, ge);
            un.load(s_w, i, u);
#pragma unroll
            for (int j = 0; j < U::E / 2; ++j) {
                const f32x2 xh = f2_mul(f2_add(xe[j], neg_mean), r2);
                dw[i][j] = f2_fma(ge[j], xh, dw[i][j]);
                if (want_db) db[i][j] = f2_add(db[i][j], ge[j]);
                u[j] = f2_mul(ge[j], u[j]);
                xe[j] = f2_mul(u[j], xh);
            }
            sa = un.add(sa, i, u);
            sax = un.add(sax, i, xe);
        }
        const float2 pa = f2_get(sa), px = f2_get(sax);
        const float2 s = group_sum2(f2(pa.x + pa.y, px.x + px.y), red[buf], G, ty);
        const float ma = rms ? 0.0f : s.x / h, max_ = s.y / h;
        const f32x2 neg_ma = f2(-ma, -ma), neg_max = f2(-max_, -max_);
        T *out = dx + (size_t)row * H;
#pragma unroll
        for (int i = 0; i < U::N; ++i) {
            f32x2 xe[U::E / 2], ge[U::E / 2], u[U::E / 2];
            un.load(xr, i, xe);
            un.load(gr, i, ge);
            un.load(s_w, i, u);
#pragma unroll
            for (int j = 0; j < U::E / 2; ++j) {
                const f32x2 xh = f2_mul(f2_add(xe[j], neg_mean), r2);
                xe[j] = f2_mul(f2_fma(xh, neg_max, f2_fma(ge[j], u[j], neg_ma)), r2);
            }
            un.store(out, i, xe);
        }
    }
    // the CTA's column sums
    copies_wait<0>();
    __syncthreads();
    float *sums = reinterpret_cast<float *>(smem) + (size_t)ty * 2 * H;
#pragma unroll
    for (int i = 0; i < U::N; ++i) {
        un.store_sums(sums, i, dw[i]);
        un.store_sums(sums + H, i, db[i]);
    }
    sums = reinterpret_cast<float *>(smem);
    __syncthreads();
    const int n = want_db ? 2 * H : H;
    for (int c = ty * G + tid; c < n; c += R * G) {
        float s = 0.0f;
        for (int r = 0; r < R; ++r) s += sums[(size_t)r * 2 * H + c];
        part[(size_t)blockIdx.x * 2 * H + c] = s;
    }
}

// ---------------------------------------------------------------------------------------
// backward, few rows: one launch, whose first `rows` CTAs make dx (a row each, read again from L1 for the second pass) and
// whose other CTAs make dw and db of 32 columns each (mean and rstd are inputs, so columns need no row sums).  x and g
// are read twice, the second time from L2; no partial sums and no second kernel.
// ---------------------------------------------------------------------------------------
constexpr int kFewThreads = 1024, kColRows = kFewThreads / 32;

template <typename T, typename W, int VEC>
__global__ void __launch_bounds__(kFewThreads)
ep_norm_bwd_few_kernel(const T *__restrict__ g, long long ldg, const T *__restrict__ x, long long ldx,
                       const W *__restrict__ w, const float *__restrict__ mean_in, const float *__restrict__ rstd_in,
                       int rows, int H, int rms, T *__restrict__ dx, float *__restrict__ dw, float *__restrict__ db) {
    __shared__ __align__(16) f32x2 s_red[32];
    __shared__ float s_col[2][kColRows][33];
    pdl_wait();
    const int tid = threadIdx.x;
    if ((int)blockIdx.x < rows) {
        if (tid < 32) s_red[tid] = f2(0.0f, 0.0f);
        const int row = blockIdx.x;
        const T *xr = x + (size_t)row * ldx, *gr = g + (size_t)row * ldg;
        const float mean = rms ? 0.0f : mean_in[row], rstd = rstd_in[row];
        float sa = 0.0f, sax = 0.0f;
        for (int c = tid * VEC; c < H; c += kFewThreads * VEC) {
            float xf[VEC], gf[VEC], wf[VEC];
            ld_pack<T, VEC>(xr + c).unpack(xf);
            ld_pack<T, VEC>(gr + c).unpack(gf);
            ld_pack<W, VEC>(w + c).unpack(wf);
#pragma unroll
            for (int j = 0; j < VEC; ++j) {
                const float a = gf[j] * wf[j];
                sa += a;
                sax = fmaf(a, (xf[j] - mean) * rstd, sax);
            }
        }
        __syncthreads();
        const float2 s = group_sum2(f2(sa, sax), s_red, kFewThreads, 0);
        const float ma = rms ? 0.0f : s.x / (float)H, max_ = s.y / (float)H;
        for (int c = tid * VEC; c < H; c += kFewThreads * VEC) {
            float xf[VEC], gf[VEC], wf[VEC], o[VEC];
            ld_pack<T, VEC>(xr + c).unpack(xf);
            ld_pack<T, VEC>(gr + c).unpack(gf);
            ld_pack<W, VEC>(w + c).unpack(wf);
#pragma unroll
            for (int j = 0; j < VEC; ++j) o[j] = rstd * (fmaf(gf[j], wf[j], -ma) - (xf[j] - mean) * rstd * max_);
            st_pack_stream<T, VEC>(dx + (size_t)row * H + c, o);
        }
        return;
    }
    const int lane = tid & 31, part = tid >> 5, c = (blockIdx.x - rows) * 32 + lane;
    float sw = 0.0f, sb = 0.0f;
    if (c < H) {
#pragma unroll 4
        for (int row = part; row < rows; row += kColRows) {
            const float gj = to_f32(g[(size_t)row * ldg + c]);
            sw = fmaf(gj, (to_f32(x[(size_t)row * ldx + c]) - (rms ? 0.0f : mean_in[row])) * rstd_in[row], sw);
            sb += gj;
        }
    }
    s_col[0][part][lane] = sw;
    s_col[1][part][lane] = sb;
    __syncthreads();
    // warp i joins column i: lane r holds part r
    const int col = (blockIdx.x - rows) * 32 + part;
    const float tw = warp_sum(s_col[0][lane][part]), tb = warp_sum(s_col[1][lane][part]);
    if (lane == 0 && col < H) {
        dw[col] = tw;
        if (db) db[col] = tb;
    }
}

// ---------------------------------------------------------------------------------------
// backward, wider rows: dx with one CTA per row that reads the row twice (the second time from
// L2), and the column sums, which need no row sums because mean and rstd are inputs, by a
// kernel of their own.
// ---------------------------------------------------------------------------------------
template <typename T, typename W>
__global__ void __launch_bounds__(1024, 1)
ep_norm_bwd_wide_kernel(const T *__restrict__ g, long long ldg, const T *__restrict__ x, long long ldx,
                        const W *__restrict__ w, const float *__restrict__ mean_in,
                        const float *__restrict__ rstd_in, int H, int rms, T *__restrict__ dx) {
    __shared__ __align__(16) f32x2 s_red[32];
    pdl_wait();
    const int row = blockIdx.x;
    const T *xr = x + (size_t)row * ldx, *gr = g + (size_t)row * ldg;
    const float mean = rms ? 0.0f : mean_in[row], rstd = rstd_in[row];
    float sa = 0.0f, sax = 0.0f;
    for (int c = threadIdx.x; c < H; c += blockDim.x) {
        const float a = to_f32(gr[c]) * to_f32(w[c]);
        sa += a;
        sax = fmaf(a, (to_f32(xr[c]) - mean) * rstd, sax);
    }
    const float2 s = group_sum2(f2(sa, sax), s_red, blockDim.x, 0);
    const float ma = rms ? 0.0f : s.x / (float)H, max_ = s.y / (float)H;
    for (int c = threadIdx.x; c < H; c += blockDim.x) {
        const float xh = (to_f32(xr[c]) - mean) * rstd;
        dx[(size_t)row * H + c] = from_f32<T>(rstd * (to_f32(gr[c]) * to_f32(w[c]) - ma - xh * max_));
    }
}

template <typename T>
__global__ void __launch_bounds__(256)
ep_norm_bwd_wide_cols_kernel(const T *__restrict__ g, long long ldg, const T *__restrict__ x, long long ldx,
                             const float *__restrict__ mean_in, const float *__restrict__ rstd_in, int rows,
                             int H, int rms, float *__restrict__ part) {
    pdl_wait();
    const int c = blockIdx.x * blockDim.x + threadIdx.x;
    if (c >= H) return;
    float dw = 0.0f, db = 0.0f;
    for (int row = blockIdx.y; row < rows; row += gridDim.y) {
        const float gj = to_f32(g[(size_t)row * ldg + c]);
        const float xh = (to_f32(x[(size_t)row * ldx + c]) - (rms ? 0.0f : mean_in[row])) * rstd_in[row];
        dw = fmaf(gj, xh, dw);
        db += gj;
    }
    part[(size_t)blockIdx.y * 2 * H + c] = dw;
    part[(size_t)blockIdx.y * 2 * H + H + c] = db;
}

// Column sums of the partial rows: 32 columns per CTA, kColRows partial rows at a time, joined
// in shared memory in a fixed order.  blockIdx.y: 0 for dw, 1 for db.
__global__ void __launch_bounds__(32 * kColRows)
ep_norm_cols_kernel(const float *__restrict__ part, int nparts, int H, float *__restrict__ dw,
                    float *__restrict__ db) {
    __shared__ float s[kColRows][33];
    pdl_wait();
    const int c = blockIdx.x * 32 + threadIdx.x;
    float v = 0.0f;
    if (c < H)
        for (int p = threadIdx.y; p < nparts; p += kColRows) v += part[(size_t)p * 2 * H + (size_t)blockIdx.y * H + c];
    s[threadIdx.y][threadIdx.x] = v;
    __syncthreads();
    // warp i sums column i: lane r holds partial row r
    const float t = warp_sum(s[threadIdx.x][threadIdx.y]);
    const int col = blockIdx.x * 32 + threadIdx.y;
    if (threadIdx.x == 0 && col < H) (blockIdx.y ? db : dw)[col] = t;
}

// ---------------------------------------------------------------------------------------
// launches
// ---------------------------------------------------------------------------------------
struct NormArgs {
    const void *g;
    long long ldg;
    const void *x;
    long long ldx;
    const void *w, *b;
    const float *mean_in, *rstd_in;
    int rows, H, rms, period;
    float eps;
    void *out;
    float *mean_out, *rstd_out, *part, *dw, *db;
    cudaStream_t st;
};

template <typename T, typename W, int VEC, int NV>
int launch_fwd_rows(const NormArgs &a) {
    return launch_pdl(ep_norm_row_kernel<T, W, VEC, NV>, dim3(a.rows), dim3(round_up((a.H / VEC + NV - 1) / NV, 32)), 0,
                      a.st, (const T *)a.x, a.ldx, (const W *)a.w, (const W *)a.b, a.H, a.eps, a.rms, one_wave(a.rows),
                      (T *)a.out, a.mean_out, a.rstd_out);
}

// A pipelined kernel's CTA: groups of G threads that hold a row, as many as `threads` and the shared memory have room for
// with row_bytes for each and params bytes per copy of the parameters; no groups (y = 0) where not even one fits.
dim3 group_shape(int H, int ept, int threads, int lay, int params, int row_bytes) {
    const int G = round_up((H + ept - 1) / ept, 32);
    const int fit = lay == kShifted ? kSharedBytes / (row_bytes + params) : (kSharedBytes - params) / row_bytes;
    return dim3(G, min(min(threads / G, fit), G == 32 ? 32 : 15));
}
// CTAs for a pipelined kernel: one per SM, or as many as the rows fill.
int group_grid(int rows, int R) {
    const int sms = device_sm_count(), full = (rows + R - 1) / R;
    return sms > 0 && sms < full ? sms : full;
}

// A piece more than the elements fill, for rows that begin and end inside one.
constexpr int laid(int H, int lay, int vec) { return lay == kShifted ? H + 2 * (vec - 1) : H; }

template <typename T, typename W, int LAY>
int launch_fwd(const NormArgs &a) {
    constexpr int VEC = 16 / sizeof(T), RV = LAY == kAligned ? VEC : 1;   // the one-row kernel's vectors
    constexpr int NV = RV == 8 ? 4 : 8;                                  // of them per thread in rows of more than 1024
    const int nv = a.H / RV;
    if ((long long)a.rows * round_up(nv <= 1024 ? nv : (nv + NV - 1) / NV, 32) <= (long long)device_sm_count() * kResidentPerSm) {
        if (nv <= 1024) return launch_fwd_rows<T, W, RV, 1>(a);
        if (nv <= 1024 * NV) return launch_fwd_rows<T, W, RV, NV>(a);
    }
    const int row_bytes = kFwdStages<T> * RowSource<T, kFwdEpt, LAY>::stage_bytes(a.H), params = 2 * param_bytes<W>(a.H + 2 * VEC);
    const dim3 block = group_shape(laid(a.H, LAY, VEC), kFwdEpt, kFwdThreads, LAY, params, row_bytes);
    if (block.y < 1) return launch_fwd_rows<T, W, RV, (RV == 1 ? 32 : NV)>(a);
    constexpr auto kern = ep_norm_kernel<T, W, LAY>;
    const int rc = allow_smem<kern>(kSharedBytes);
    if (rc != EP_OK) return rc;
    const size_t smem = param_copies(LAY, block.y) * params + (size_t)block.y * row_bytes;
    return launch_pdl(kern, dim3(group_grid(a.rows, block.y)), block, smem, a.st, (const T *)a.x, a.ldx, (const W *)a.w,
                      (const W *)a.b, a.rows, a.H, a.eps, a.rms, a.period, (T *)a.out, a.mean_out, a.rstd_out);
}

int launch_cols(const NormArgs &a, int nparts) {
    return launch_pdl(ep_norm_cols_kernel, dim3((a.H + 31) / 32, a.db ? 2 : 1), dim3(32, kColRows), 0, a.st,
                      (const float *)a.part, nparts, a.H, a.dw, a.db);
}

template <typename T, typename W, int LAY>
int launch_bwd(const NormArgs &a) {
    if (a.rows <= few_bwd_rows(a.H, sizeof(T))) {
        constexpr int VEC = LAY == kAligned ? 16 / sizeof(T) : 1;
        return launch_pdl(ep_norm_bwd_few_kernel<T, W, VEC>, dim3(a.rows + (a.H + 31) / 32), dim3(kFewThreads), 0, a.st,
                          (const T *)a.g, a.ldg, (const T *)a.x, a.ldx, (const W *)a.w, a.mean_in, a.rstd_in, a.rows, a.H,
                          a.rms, (T *)a.out, a.dw, a.db);
    }
    if (a.H <= kBwdMaxH) {
        constexpr int VEC = 16 / sizeof(T);
        const int row_bytes = kBwdStages * 2 * RowSource<T, kBwdEpt, LAY>::stage_bytes(a.H), params = param_bytes<W>(a.H + 2 * VEC);
        const dim3 block = group_shape(laid(a.H, LAY, VEC), kBwdEpt, kBwdThreads, LAY, params, row_bytes);
        constexpr auto kern = ep_norm_bwd_kernel<T, W, LAY>;
        const size_t stages = param_copies(LAY, block.y) * params + (size_t)block.y * row_bytes;
        const size_t sums = (size_t)block.y * 2 * a.H * sizeof(float);
        const int rc = allow_smem<kern>(kSharedBytes);
        if (rc != EP_OK) return rc;
        const int grid = min(group_grid(a.rows, block.y), kPartials);
        const int e = launch_pdl(kern, dim3(grid), block, stages > sums ? stages : sums, a.st, (const T *)a.g, a.ldg,
                                 (const T *)a.x, a.ldx, (const W *)a.w, a.mean_in, a.rstd_in, a.rows, a.H, a.rms,
                                 a.db ? 1 : 0, a.period, (T *)a.out, a.part);
        return e != EP_OK ? e : launch_cols(a, grid);
    }
    int rc = launch_pdl(ep_norm_bwd_wide_kernel<T, W>, dim3(a.rows), dim3(1024), 0, a.st, (const T *)a.g, a.ldg,
                        (const T *)a.x, a.ldx, (const W *)a.w, a.mean_in, a.rstd_in, a.H, a.rms, (T *)a.out);
    if (rc != EP_OK) return rc;
    const int parts = min(a.rows, 16);
    rc = launch_pdl(ep_norm_bwd_wide_cols_kernel<T>, dim3((a.H + 255) / 256, parts), dim3(256), 0, a.st,
                    (const T *)a.g, a.ldg, (const T *)a.x, a.ldx, a.mean_in, a.rstd_in, a.rows, a.H, a.rms, a.part);
    return rc != EP_OK ? rc : launch_cols(a, parts);
}

// How the rows lie: x, y and, going backward, g.
template <typename T>
int lay_of(const NormArgs &a, int &period) {
    constexpr int VEC = 16 / sizeof(T);
    const auto off = [](const void *p) { return (int)(reinterpret_cast<uintptr_t>(p) & 15u); };
    period = 1;
    if (off(a.x) != off(a.out) || a.ldx % VEC != a.H % VEC) return kAny;
    if (a.g && (off(a.g) != off(a.x) || a.ldg % VEC != a.H % VEC)) return kAny;
    if (off(a.x) == 0 && a.H % VEC == 0) return aligned16(a.w) && aligned16(a.b) ? kAligned : kShifted;
    while (period * a.H % VEC) period *= 2;
    return kShifted;
}

template <typename T, typename W>
int launch_norm(NormArgs a) {
    const int lay = lay_of<T>(a, a.period);
    if (lay == kAny) a.period = 1;
    if (a.g) return lay == kAligned ? launch_bwd<T, W, kAligned>(a) : lay == kShifted ? launch_bwd<T, W, kShifted>(a) : launch_bwd<T, W, kAny>(a);
    return lay == kAligned ? launch_fwd<T, W, kAligned>(a) : lay == kShifted ? launch_fwd<T, W, kShifted>(a) : launch_fwd<T, W, kAny>(a);
}

int launch_norm(const NormArgs &a, int dtype, int wdtype) {
    if (dtype == EP_F32) return launch_norm<float, float>(a);
    if (dtype == EP_BF16)
        return wdtype == EP_F32 ? launch_norm<__nv_bfloat16, float>(a) : launch_norm<__nv_bfloat16, __nv_bfloat16>(a);
    return wdtype == EP_F32 ? launch_norm<__half, float>(a) : launch_norm<__half, __half>(a);
}

bool norm_sizes_ok(int T, int H) { return T >= 0 && T <= kMaxT && H >= 1 && H <= kMaxH; }

// Element types: x in {bf16, fp16, fp32}, parameters in x's type or fp32.
bool norm_types_ok(int dtype, int wdtype) {
    return dtype >= EP_BF16 && dtype <= EP_F32 && (wdtype == dtype || wdtype == EP_F32);
}

bool aligned_to(const void *p, int dtype) {
    return (reinterpret_cast<uintptr_t>(p) & (dtype == EP_F32 ? 3u : 1u)) == 0;
}

}  // namespace
}  // namespace ep

using namespace ep;

extern "C" size_t ep_layer_norm_bwd_workspace_bytes(int T, int hidden_size) {
    if (!norm_sizes_ok(T, hidden_size)) return 0;
    const size_t parts = T < 1 ? 1 : T < kPartials ? T : kPartials;
    return (parts * 2 * hidden_size * sizeof(float) + 15) / 16 * 16;
}

extern "C" int ep_layer_norm(const void *x, long long x_stride, int dtype, const void *weight, const void *bias,
                             int param_dtype, int T, int hidden_size, float eps, int rms, void *y, float *mean,
                             float *rstd, void *stream) {
    EP_NVTX_RANGE("ep_layer_norm");
    const int H = hidden_size;
    if (!norm_sizes_ok(T, H) || !norm_types_ok(dtype, param_dtype) || (rms != 0 && rms != 1)) return EP_ERR_INVALID_ARG;
    if (!(eps >= 0.0f) || x_stride < H) return EP_ERR_INVALID_ARG;
    if (!aligned_to(x, dtype) || !aligned_to(y, dtype) || !aligned_to(weight, param_dtype) ||
        !aligned_to(bias, param_dtype) || !aligned_to(mean, EP_F32) || !aligned_to(rstd, EP_F32))
        return EP_ERR_INVALID_ARG;
    if (T == 0) return EP_OK;
    if (!x || !weight || !y || !rstd || (!rms && !mean)) return EP_ERR_INVALID_ARG;
    NormArgs a = {};
    a.x = x; a.ldx = x_stride; a.w = weight; a.b = bias;
    a.rows = T; a.H = H; a.rms = rms; a.eps = eps;
    a.out = y; a.mean_out = mean; a.rstd_out = rstd; a.st = as_stream(stream);
    return launch_norm(a, dtype, param_dtype);
}

extern "C" int ep_layer_norm_bwd(const void *grad_y, long long grad_stride, const void *x, long long x_stride,
                                 int dtype, const void *weight, int param_dtype, const float *mean, const float *rstd,
                                 int T, int hidden_size, int rms, void *grad_x, float *grad_weight, float *grad_bias,
                                 void *workspace, size_t workspace_bytes, void *stream) {
    EP_NVTX_RANGE("ep_layer_norm_bwd");
    const int H = hidden_size;
    if (!norm_sizes_ok(T, H) || !norm_types_ok(dtype, param_dtype) || (rms != 0 && rms != 1)) return EP_ERR_INVALID_ARG;
    if (x_stride < H || grad_stride < H || !grad_weight || !workspace) return EP_ERR_INVALID_ARG;
    if (workspace_bytes < ep_layer_norm_bwd_workspace_bytes(T, H) || !aligned16(workspace)) return EP_ERR_INVALID_ARG;
    if (!aligned_to(x, dtype) || !aligned_to(grad_y, dtype) || !aligned_to(grad_x, dtype) ||
        !aligned_to(weight, param_dtype) || !aligned_to(mean, EP_F32) || !aligned_to(rstd, EP_F32) ||
        !aligned_to(grad_weight, EP_F32) || !aligned_to(grad_bias, EP_F32))
        return EP_ERR_INVALID_ARG;
    if (T > 0 && (!grad_y || !x || !weight || !rstd || !grad_x || (!rms && !mean))) return EP_ERR_INVALID_ARG;
    NormArgs a = {};
    a.g = grad_y; a.ldg = grad_stride; a.x = x; a.ldx = x_stride; a.w = weight;
    a.mean_in = mean; a.rstd_in = rstd; a.rows = T; a.H = H; a.rms = rms;
    a.out = grad_x; a.part = (float *)workspace; a.dw = grad_weight; a.db = grad_bias; a.st = as_stream(stream);
    if (T == 0) return launch_cols(a, 0);
    return launch_norm(a, dtype, param_dtype);
}
