// ep_norm.cu -- layer norm and RMS norm over the rows of a token matrix, in front of the router
// and the dispatch, and their backward pass with the reduction of the parameters' gradients.
//
//   forward   xh = (x - mean) * rstd, y = xh * w + b; mean = sum(x)/H,
//             rstd = 1/sqrt(sum((x - mean)^2)/H + eps)  (RMS: mean = 0)
//   backward  a = g * w, dx = rstd * (a - mean(a) - xh * mean(a * xh))  (RMS: no mean(a)),
//             dw = sum over rows of g * xh, db = sum over rows of g
//
// Statistics and sums are fp32.  The variance is summed over (x - mean) in a second pass over
// registers, so rows with a large mean lose nothing.  Both passes are bound by HBM: each row is
// read once, kept in registers, and written once.
#include "ep_host.h"
#include "ep_types.cuh"

namespace ep {
namespace {

// ---------------------------------------------------------------------------------------
// forward
// ---------------------------------------------------------------------------------------
// Sum over the threads of one row: a warp (WARP) or the whole CTA.  `red` holds one float per
// warp; two calls in a row use different halves, so one barrier each is enough.
template <bool WARP>
__device__ __forceinline__ float row_sum(float v, float *red) {
    v = warp_sum(v);
    if (WARP) return v;
    const int nw = blockDim.x >> 5;
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
    __syncthreads();
    float s = 0.0f;
    for (int i = 0; i < nw; ++i) s += red[i];
    return s;
}

// NV vectors of VEC elements per thread, one row per warp or per CTA.
template <typename T, typename W, int VEC, int NV, bool WARP>
__global__ void __launch_bounds__(1024)
ep_norm_kernel(const T *__restrict__ x, long long ldx, const W *__restrict__ w, const W *__restrict__ b,
               int rows, int H, float eps, int rms, int one_wave, T *__restrict__ y,
               float *__restrict__ mean_out, float *__restrict__ rstd_out) {
    __shared__ float red[2][32];
    pdl_begin_if(one_wave);
    const int group = WARP ? 32 : blockDim.x;
    const int tid = WARP ? threadIdx.x & 31 : threadIdx.x;
    const int row = WARP ? blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5) : blockIdx.x;
    if (WARP && row >= rows) return;
    const int nv = H / VEC;
    const T *xr = x + (size_t)row * ldx;
    Pack<T, VEC> d[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int v = tid + i * group;
        if (v < nv) d[i] = ld_pack_stream<T, VEC>(xr + (size_t)v * VEC);
    }
    float mean = 0.0f;
    if (!rms) {
        float s = 0.0f;
#pragma unroll
        for (int i = 0; i < NV; ++i)
            if (tid + i * group < nv)
#pragma unroll
                for (int j = 0; j < VEC; ++j) s += d[i].f(j);
        mean = row_sum<WARP>(s, red[0]) / (float)H;
    }
    float q = 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i)
        if (tid + i * group < nv)
#pragma unroll
            for (int j = 0; j < VEC; ++j) {
                const float c = d[i].f(j) - mean;
                q = fmaf(c, c, q);
            }
    const float rstd = 1.0f / sqrtf(row_sum<WARP>(q, red[1]) / (float)H + eps);
    if (tid == 0) {
        if (!rms) mean_out[row] = mean;
        rstd_out[row] = rstd;
    }
    T *yr = y + (size_t)row * H;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int v = tid + i * group;
        if (v >= nv) break;
        const Pack<W, VEC> wv = ld_pack<W, VEC>(w + (size_t)v * VEC);
        float o[VEC];
#pragma unroll
        for (int j = 0; j < VEC; ++j) o[j] = (d[i].f(j) - mean) * rstd * wv.f(j);
        if (b) {
            const Pack<W, VEC> bv = ld_pack<W, VEC>(b + (size_t)v * VEC);
#pragma unroll
            for (int j = 0; j < VEC; ++j) o[j] += bv.f(j);
        }
        st_pack_stream<T, VEC>(yr + (size_t)v * VEC, o);
    }
}

// ---------------------------------------------------------------------------------------
// backward, rows of up to kFusedH elements: a group of threads keeps one row of x and g in
// registers and the sums of its columns over all its rows beside them, so x and g are read once
// for dx, dw and db.  Group sums are joined per CTA in shared memory, CTA sums by
// ep_norm_cols_kernel, both in a fixed order.
// ---------------------------------------------------------------------------------------
constexpr int kFusedH = 8192;
constexpr int kFusedThreads = 512;
constexpr int kPartials = 304;   // rows of partial column sums: two CTAs on each of 152 SMs

// Sum of two values over the threads of a group of G threads (ty: the group's index in the CTA).
__device__ __forceinline__ float2 group_sum2(float a, float b, float2 *red, int G, int ty) {
    a = warp_sum(a);
    b = warp_sum(b);
    if (G == 32) return make_float2(a, b);
    const int nw = G >> 5;
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = make_float2(a, b);
    asm volatile("bar.sync %0, %1;" ::"r"(ty + 1), "r"(G) : "memory");
    float2 s = make_float2(0.0f, 0.0f);
    for (int i = 0; i < nw; ++i) {
        s.x += red[i].x;
        s.y += red[i].y;
    }
    return s;
}

template <typename T, typename W, int VEC, int NV>
__global__ void __launch_bounds__(kFusedThreads)
ep_norm_bwd_kernel(const T *__restrict__ g, long long ldg, const T *__restrict__ x, long long ldx,
                   const W *__restrict__ w, const float *__restrict__ mean_in,
                   const float *__restrict__ rstd_in, int rows, int H, int rms, int want_db,
                   T *__restrict__ dx, float *__restrict__ part) {
    extern __shared__ float s_cols[];   // [2][H], with more than one group per CTA
    __shared__ float2 s_red[2][kFusedThreads / 32];
    pdl_begin();
    const int G = blockDim.x, R = blockDim.y, tid = threadIdx.x, ty = threadIdx.y;
    const int nv = H / VEC;
    float dw[NV][VEC], db[NV][VEC];
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int j = 0; j < VEC; ++j) dw[i][j] = db[i][j] = 0.0f;
    int buf = 0;
    for (int row = blockIdx.x * R + ty; row < rows; row += gridDim.x * R, buf ^= 1) {
        Pack<T, VEC> xv[NV], gv[NV];
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int v = tid + i * G;
            if (v < nv) {
                xv[i] = ld_pack_stream<T, VEC>(x + (size_t)row * ldx + (size_t)v * VEC);
                gv[i] = ld_pack_stream<T, VEC>(g + (size_t)row * ldg + (size_t)v * VEC);
            }
        }
        const float mean = rms ? 0.0f : mean_in[row], rstd = rstd_in[row];
        float sa = 0.0f, sax = 0.0f;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int v = tid + i * G;
            if (v < nv) {
                const Pack<W, VEC> wv = ld_pack<W, VEC>(w + (size_t)v * VEC);
#pragma unroll
                for (int j = 0; j < VEC; ++j) {
                    const float gj = gv[i].f(j), xh = (xv[i].f(j) - mean) * rstd, a = gj * wv.f(j);
                    sa += a;
                    sax = fmaf(a, xh, sax);
                    dw[i][j] = fmaf(gj, xh, dw[i][j]);
                    db[i][j] += gj;
                }
            }
        }
        const float2 s = group_sum2(sa, sax, s_red[buf] + ty * (G >> 5), G, ty);
        const float ma = rms ? 0.0f : s.x / (float)H, max_ = s.y / (float)H;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int v = tid + i * G;
            if (v < nv) {
                const Pack<W, VEC> wv = ld_pack<W, VEC>(w + (size_t)v * VEC);
                float o[VEC];
#pragma unroll
                for (int j = 0; j < VEC; ++j) {
                    const float xh = (xv[i].f(j) - mean) * rstd;
                    o[j] = rstd * (gv[i].f(j) * wv.f(j) - ma - xh * max_);
                }
                st_pack_stream<T, VEC>(dx + (size_t)row * H + (size_t)v * VEC, o);
            }
        }
    }
    // the CTA's column sums: group 0 in registers, the other groups' added in order
    for (int r = 1; r < R; ++r) {
        __syncthreads();
        if (ty == r) {
#pragma unroll
            for (int i = 0; i < NV; ++i)
                if (tid + i * G < nv)
#pragma unroll
                    for (int j = 0; j < VEC; ++j) {
                        s_cols[(tid + i * G) * VEC + j] = dw[i][j];
                        s_cols[H + (tid + i * G) * VEC + j] = db[i][j];
                    }
        }
        __syncthreads();
        if (ty == 0) {
#pragma unroll
            for (int i = 0; i < NV; ++i)
                if (tid + i * G < nv)
#pragma unroll
                    for (int j = 0; j < VEC; ++j) {
                        dw[i][j] += s_cols[(tid + i * G) * VEC + j];
                        db[i][j] += s_cols[H + (tid + i * G) * VEC + j];
                    }
        }
    }
    if (ty != 0) return;
    float *pw = part + (size_t)blockIdx.x * 2 * H, *pb = pw + H;
#pragma unroll
    for (int i = 0; i < NV; ++i)
        if (tid + i * G < nv)
#pragma unroll
            for (int j = 0; j < VEC; ++j) {
                pw[(tid + i * G) * VEC + j] = dw[i][j];
                if (want_db) pb[(tid + i * G) * VEC + j] = db[i][j];
            }
}

// ---------------------------------------------------------------------------------------
// backward, wider rows: dx with one CTA per row that reads the row twice (the second time from
// L2), and the column sums, which need no row sums because mean and rstd are inputs, by a
// kernel of their own.
// ---------------------------------------------------------------------------------------
template <typename T, typename W>
__global__ void __launch_bounds__(1024)
ep_norm_bwd_wide_kernel(const T *__restrict__ g, long long ldg, const T *__restrict__ x, long long ldx,
                        const W *__restrict__ w, const float *__restrict__ mean_in,
                        const float *__restrict__ rstd_in, int H, int rms, T *__restrict__ dx) {
    __shared__ float2 s_red[32];
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
    const float2 s = group_sum2(sa, sax, s_red, blockDim.x, 0);
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
constexpr int kColRows = 32;
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
    int rows, H, rms;
    float eps;
    void *out;
    float *mean_out, *rstd_out, *part, *dw, *db;
    cudaStream_t st;
};

constexpr int round_up32(int n) { return (n + 31) / 32 * 32; }

template <typename T, typename W, int VEC, int NV>
int launch_fwd_nv(const NormArgs &a, int group) {
    const auto launch = [&](auto kern, int grid, int threads) {
        return launch_pdl(kern, dim3(grid), dim3(threads), 0, a.st, (const T *)a.x, a.ldx, (const W *)a.w,
                          (const W *)a.b, a.rows, a.H, a.eps, a.rms, one_wave(grid), (T *)a.out, a.mean_out,
                          a.rstd_out);
    };
    if (group == 32) return launch(ep_norm_kernel<T, W, VEC, NV, true>, (a.rows + 3) / 4, 128);
    return launch(ep_norm_kernel<T, W, VEC, NV, false>, a.rows, group);
}

template <typename T, typename W, int VEC>
int launch_fwd(const NormArgs &a) {
    const int nv = a.H / VEC;
    // few rows: as many threads per row as it has vectors; many rows: a warp for up to 8 vectors
    // per lane, then as few warps as hold the row
    if (a.rows <= 2 * 152 && nv <= 1024) return launch_fwd_nv<T, W, VEC, 1>(a, round_up32(nv));
    if (nv <= 32) return launch_fwd_nv<T, W, VEC, 1>(a, 32);
    if (nv <= 64) return launch_fwd_nv<T, W, VEC, 2>(a, 32);
    if (nv <= 128) return launch_fwd_nv<T, W, VEC, 4>(a, 32);
    if (nv <= 8 * 1024) return launch_fwd_nv<T, W, VEC, 8>(a, round_up32((nv + 7) / 8));
    return launch_fwd_nv<T, W, VEC, 32>(a, round_up32((nv + 31) / 32));
}

int launch_cols(const NormArgs &a, int nparts) {
    return launch_pdl(ep_norm_cols_kernel, dim3((a.H + 31) / 32, a.db ? 2 : 1), dim3(32, kColRows), 0, a.st,
                      (const float *)a.part, nparts, a.H, a.dw, a.db);
}

template <typename T, typename W, int VEC, int NV>
int launch_bwd_nv(const NormArgs &a) {
    const int G = round_up32((a.H / VEC + NV - 1) / NV);
    const int R = G == 32 ? 16 : G < kFusedThreads ? kFusedThreads / G : 1;
    const size_t smem = R > 1 ? (size_t)2 * a.H * sizeof(float) : 0;
    const int grid = min((a.rows + R - 1) / R, kPartials);
    const int rc = launch_pdl(ep_norm_bwd_kernel<T, W, VEC, NV>, dim3(grid), dim3(G, R), smem, a.st, (const T *)a.g,
                              a.ldg, (const T *)a.x, a.ldx, (const W *)a.w, a.mean_in, a.rstd_in, a.rows, a.H, a.rms,
                              a.db ? 1 : 0, (T *)a.out, a.part);
    return rc != EP_OK ? rc : launch_cols(a, grid);
}

template <typename T, typename W, int VEC>
int launch_bwd(const NormArgs &a) {
    if (a.rows == 0) return launch_cols(a, 0);
    if (a.H <= kFusedH / 2) return launch_bwd_nv<T, W, VEC, 8 / VEC>(a);
    if (a.H <= kFusedH) return launch_bwd_nv<T, W, VEC, 16 / VEC>(a);
    int rc = launch_pdl(ep_norm_bwd_wide_kernel<T, W>, dim3(a.rows), dim3(1024), 0, a.st, (const T *)a.g, a.ldg,
                        (const T *)a.x, a.ldx, (const W *)a.w, a.mean_in, a.rstd_in, a.H, a.rms, (T *)a.out);
    if (rc != EP_OK) return rc;
    const int parts = min(a.rows, 16);
    rc = launch_pdl(ep_norm_bwd_wide_cols_kernel<T>, dim3((a.H + 255) / 256, parts), dim3(256), 0, a.st,
                    (const T *)a.g, a.ldg, (const T *)a.x, a.ldx, a.mean_in, a.rstd_in, a.rows, a.H, a.rms, a.part);
    return rc != EP_OK ? rc : launch_cols(a, parts);
}

// Vectors of 16 bytes need every row and parameter on a 16-byte boundary.
template <typename T, typename W>
int launch_norm(const NormArgs &a) {
    constexpr int VEC = 16 / sizeof(T);
    const bool vec = a.H % VEC == 0 && a.ldx % VEC == 0 && (!a.g || a.ldg % VEC == 0) && aligned16(a.x) &&
                     aligned16(a.g) && aligned16(a.w) && aligned16(a.b) && aligned16(a.out);
    if (a.g) return vec ? launch_bwd<T, W, VEC>(a) : launch_bwd<T, W, 1>(a);
    return vec ? launch_fwd<T, W, VEC>(a) : launch_fwd<T, W, 1>(a);
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
