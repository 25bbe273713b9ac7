// layer_norm.hip - layer norm forward and backward over rows of any width.
//
// Both passes read and write each value once at best and do about ten
// operations on it: HBM bounds them.
#include <math.h>

#include "common.hpp"
#include "dense_ops.h"
#include "dense.hpp"

namespace spopt {

// Sum over the 256 threads of a block; every thread gets it.  `lds` holds one
// float per wave; a barrier before the next use is inside.
__device__ __forceinline__ float block_sum(float v, float* lds) {
#pragma unroll
    for (int off = kWave / 2; off; off >>= 1) v += __shfl_xor(v, off, kWave);
    __syncthreads();
    if (lane_id() == 0) lds[threadIdx.x >> 6] = v;
    __syncthreads();
    float s = 0.f;
    for (int i = 0; i < (int)(blockDim.x >> 6); ++i) s += lds[i];
    return s;
}

// One block per row, any width: the row is read once for the mean, again for
// the centred squares and again for the output (the later reads from cache).
template <class T, class W>
__global__ __launch_bounds__(256) void k_ln_fwd_any(const T* x, int64_t xs, int64_t rows,
                                                    int64_t cols, const W* w, const W* b,
                                                    float eps, T* y, int64_t ys, float* mean,
                                                    float* rstd) {
    __shared__ float lds[4];
    for (int64_t r = blockIdx.x; r < rows; r += gridDim.x) {
        const T* xr = x + r * xs;
        float s = 0.f;
        for (int64_t c = threadIdx.x; c < cols; c += 256) s += (float)xr[c];
        const float mu = block_sum(s, lds) / (float)cols;
        float q = 0.f;
        for (int64_t c = threadIdx.x; c < cols; c += 256) {
            const float d = (float)xr[c] - mu;
            q += d * d;
        }
        const float rs = 1.0f / sqrtf(block_sum(q, lds) / (float)cols + eps);
        if (threadIdx.x == 0) {
            if (mean) mean[r] = mu;
            if (rstd) rstd[r] = rs;
        }
        for (int64_t c = threadIdx.x; c < cols; c += 256) {
            float v = ((float)xr[c] - mu) * rs;
            if (w) v *= (float)w[c];
            if (b) v += (float)b[c];
            y[r * ys + c] = (T)v;
        }
    }
}

// dx of one row per block, any width.
template <class T, class W>
__global__ __launch_bounds__(256) void k_ln_dx_any(const T* dy, int64_t ds, const T* x,
                                                   int64_t xs, int64_t rows, int64_t cols,
                                                   const float* mean, const float* rstd,
                                                   const W* w, T* dx, int64_t os) {
    __shared__ float lds[4];
    for (int64_t r = blockIdx.x; r < rows; r += gridDim.x) {
        const T *xr = x + r * xs, *dr = dy + r * ds;
        const float mu = mean[r], rs = rstd[r];
        float s1 = 0.f, s2 = 0.f;
        for (int64_t c = threadIdx.x; c < cols; c += 256) {
            const float z = (float)dr[c] * (w ? (float)w[c] : 1.f);
            s1 += z;
            s2 += z * (((float)xr[c] - mu) * rs);
        }
        const float m1 = block_sum(s1, lds) / (float)cols;
        const float m2 = block_sum(s2, lds) / (float)cols;
        for (int64_t c = threadIdx.x; c < cols; c += 256) {
            const float z = (float)dr[c] * (w ? (float)w[c] : 1.f);
            const float h = ((float)xr[c] - mu) * rs;
            dx[r * os + c] = (T)(rs * (z - m1 - h * m2));
        }
    }
}

// Sums of dy * xhat and dy over one slice of rows (blockIdx.y) for 64 columns:
// four rows at a time, joined in LDS.  part: [slices][2][cols].
template <class T>
__global__ __launch_bounds__(256) void k_ln_cols_any(const T* dy, int64_t ds, const T* x,
                                                     int64_t xs, int64_t rows, int64_t cols,
                                                     const float* mean, const float* rstd,
                                                     int64_t per, float* part) {
    __shared__ float lw[4][64], lb[4][64];
    const int lane = lane_id(), k = threadIdx.x >> 6;
    const int64_t c = (int64_t)blockIdx.x * 64 + lane;
    const int64_t r0 = blockIdx.y * per, r1 = r0 + per < rows ? r0 + per : rows;
    float sw = 0.f, sb = 0.f;
    if (c < cols)
        for (int64_t r = r0 + k; r < r1; r += 4) {
            const float g = (float)dy[r * ds + c];
            sw += g * (((float)x[r * xs + c] - mean[r]) * rstd[r]);
            sb += g;
        }
    lw[k][lane] = sw;
    lb[k][lane] = sb;
    __syncthreads();
    if (k == 0 && c < cols) {
        float* p = part + (int64_t)blockIdx.y * 2 * cols + c;
        p[0] = (lw[0][lane] + lw[1][lane]) + (lw[2][lane] + lw[3][lane]);
        p[cols] = (lb[0][lane] + lb[1][lane]) + (lb[2][lane] + lb[3][lane]);
    }
}

// dweight and dbias from the slices' sums: a block takes 64 columns, its four
// waves a quarter of the slices each; joined in double.
template <class W>
__global__ __launch_bounds__(256) void k_ln_join(const float* part, int64_t slices, int64_t cols,
                                                 W* dw, W* db) {
    __shared__ double lw[4][64], lb[4][64];
    const int lane = lane_id(), k = threadIdx.x >> 6;
    const int64_t c = (int64_t)blockIdx.x * 64 + lane;
    double sw = 0., sb = 0.;
    if (c < cols)
        for (int64_t i = k; i < slices; i += 4) {
            sw += (double)part[i * 2 * cols + c];
            sb += (double)part[(i * 2 + 1) * cols + c];
        }
    lw[k][lane] = sw;
    lb[k][lane] = sb;
    __syncthreads();
    if (k == 0 && c < cols) {
        if (dw) dw[c] = (W)(float)((lw[0][lane] + lw[1][lane]) + (lw[2][lane] + lw[3][lane]));
        if (db) db[c] = (W)(float)((lb[0][lane] + lb[1][lane]) + (lb[2][lane] + lb[3][lane]));
    }
}

// Row slices of the column sums: enough blocks to fill the card, and partial
// sums of no more than about 1/32 of the inputs.
static int64_t ln_slices(int64_t rows) {
    const int64_t s = ceil_div(rows, 64);
    return s < 1 ? 1 : s > 256 ? 256 : s;
}

static int ln_check(const char* what, int64_t rows, int64_t cols, int32_t dtype, int32_t wdtype) {
    if (rows < 0 || cols < 1 || rows > INT64_MAX / 8 / cols)
        return fail(SPOPT_EINVAL, "%s: bad size %lld x %lld", what, (long long)rows,
                    (long long)cols);
    if (dtype < SPOPT_DTYPE_F32 || dtype > SPOPT_DTYPE_F16)
        return fail(SPOPT_EINVAL, "%s: unknown type %d", what, dtype);
    if (wdtype != SPOPT_DTYPE_F32 && wdtype != dtype)
        return fail(SPOPT_EINVAL, "%s: weight type %d is neither float32 nor that of x", what,
                    wdtype);
    return SPOPT_OK;
}

static bool bad_stride(int64_t stride, int64_t rows, int64_t cols) {
    return rows > 1 && (stride < cols || stride > INT64_MAX / 8 / rows);
}

// Calls f(T{}, W{}) for the element type of x and of the weight.
template <class F>
static void ln_types(int32_t dtype, int32_t wdtype, F&& f) {
    if (dtype == SPOPT_DTYPE_F32)
        f(float{}, float{});
    else if (dtype == SPOPT_DTYPE_BF16)
        wdtype == SPOPT_DTYPE_F32 ? f(__bf16{}, float{}) : f(__bf16{}, __bf16{});
    else
        wdtype == SPOPT_DTYPE_F32 ? f(_Float16{}, float{}) : f(_Float16{}, _Float16{});
}

static unsigned row_grid(int64_t rows) { return (unsigned)(rows < 65536 ? rows : 65536); }

}  // namespace spopt

using namespace spopt;

extern "C" int layer_norm_forward(const void* x, int64_t x_stride, int64_t rows, int64_t cols,
                                  int32_t dtype, const void* weight, const void* bias,
                                  int32_t wdtype, double eps, void* y, int64_t y_stride,
                                  float* mean, float* rstd, void* stream, uint32_t flags) {
    hipStream_t s = (hipStream_t)stream;
    int rc = ln_check("layer_norm_forward", rows, cols, dtype, wdtype);
    if (rc) return rc;
    if (!(eps > 0.0) || !isfinite(eps))
        return fail(SPOPT_EINVAL, "layer_norm_forward: eps must be finite and > 0");
    if (rows == 0) return SPOPT_OK;
    if (x == nullptr || y == nullptr) return fail(SPOPT_EINVAL, "layer_norm_forward: NULL x or y");
    if (bad_stride(x_stride, rows, cols) || bad_stride(y_stride, rows, cols))
        return fail(SPOPT_EINVAL, "layer_norm_forward: a row stride below cols");
    if (flags & SPOPT_VALIDATE) {
        rc = validate_on_device(s, false, "layer_norm_forward", [&](uint32_t* status) {
            return launch_check_finite(x, dtype, rows, cols, x_stride, status, s);
        });
        if (rc) return rc;
    }
    ln_types(dtype, wdtype, [&](auto t, auto wt) {
        using T = decltype(t);
        using W = decltype(wt);
        k_ln_fwd_any<T, W><<<row_grid(rows), 256, 0, s>>>(
            (const T*)x, x_stride, rows, cols, (const W*)weight, (const W*)bias, (float)eps,
            (T*)y, y_stride, mean, rstd);
    });
    SPOPT_LAUNCHED();
    return SPOPT_OK;
}

extern "C" int layer_norm_backward_workspace_size(int64_t rows, int64_t cols, size_t* bytes) {
    if (bytes == nullptr || rows < 0 || cols < 1 || rows > INT64_MAX / 8 / cols ||
        cols > INT64_MAX / 8192)
        return fail(SPOPT_EINVAL, "layer_norm_backward_workspace_size: bad size %lld x %lld",
                    (long long)rows, (long long)cols);
    *bytes = (size_t)ln_slices(rows) * 2 * (size_t)cols * sizeof(float);
    return SPOPT_OK;
}

extern "C" int layer_norm_backward(const void* dy, int64_t dy_stride, const void* x,
                                   int64_t x_stride, int64_t rows, int64_t cols, int32_t dtype,
                                   const float* mean, const float* rstd, const void* weight,
                                   int32_t wdtype, void* dx, int64_t dx_stride, void* dweight,
                                   void* dbias, void* workspace, size_t workspace_bytes,
                                   void* stream, uint32_t flags) {
    hipStream_t s = (hipStream_t)stream;
    int rc = ln_check("layer_norm_backward", rows, cols, dtype, wdtype);
    if (rc) return rc;
    if (rows > 0 && (dy == nullptr || x == nullptr || mean == nullptr || rstd == nullptr))
        return fail(SPOPT_EINVAL, "layer_norm_backward: NULL dy, x, mean or rstd");
    if (bad_stride(dy_stride, rows, cols) || bad_stride(x_stride, rows, cols) ||
        (dx != nullptr && bad_stride(dx_stride, rows, cols)))
        return fail(SPOPT_EINVAL, "layer_norm_backward: a row stride below cols");
    size_t need = 0;
    rc = layer_norm_backward_workspace_size(rows, cols, &need);
    if (rc) return rc;
    const bool sums = dweight != nullptr || dbias != nullptr;
    if (sums && (workspace == nullptr || !aligned16(workspace) || workspace_bytes < need))
        return fail(SPOPT_EWORKSPACE, "layer_norm_backward: workspace of %zu bytes, needs %zu",
                    workspace_bytes, need);
    if ((flags & SPOPT_VALIDATE) && rows > 0) {
        rc = validate_on_device(s, false, "layer_norm_backward", [&](uint32_t* status) {
            const int e = launch_check_finite(dy, dtype, rows, cols, dy_stride, status, s);
            return e ? e : launch_check_finite(x, dtype, rows, cols, x_stride, status, s);
        });
        if (rc) return rc;
    }
    const int64_t slices = rows == 0 ? 0 : ln_slices(rows);
    ln_types(dtype, wdtype, [&](auto t, auto wt) {
        using T = decltype(t);
        using W = decltype(wt);
        float* part = (float*)workspace;
        const unsigned cb = (unsigned)ceil_div(cols, 64);
        // The column sums first: dx may lie over dy or x.
        if (sums && rows > 0)
            k_ln_cols_any<T><<<dim3(cb, (unsigned)slices), 256, 0, s>>>(
                (const T*)dy, dy_stride, (const T*)x, x_stride, rows, cols, mean, rstd,
                ceil_div(rows, slices), part);
        if (dx != nullptr && rows > 0)
            k_ln_dx_any<T, W><<<row_grid(rows), 256, 0, s>>>(
                (const T*)dy, dy_stride, (const T*)x, x_stride, rows, cols, mean, rstd,
                (const W*)weight, (T*)dx, dx_stride);
        if (sums)
            k_ln_join<W><<<cb, 256, 0, s>>>(part, slices, cols, (W*)dweight, (W*)dbias);
    });
    SPOPT_LAUNCHED();
    return SPOPT_OK;
}
