// layer_norm.hip - layer norm forward and backward over rows of any width.
//
// Both passes read and write each value once at best and do about ten
// operations on it: HBM bounds them (a 1 GiB copy reaches 5.1 TB/s here), and
// the time to launch where there are few rows.
#include <math.h>

#include <type_traits>

#include "common.hpp"
#include "dense_ops.h"
#include "dense.hpp"

namespace spopt {

// Sum over the G lanes of a group that share a row (G = 4 to 64): every
// lane gets it.  The first four exchanges stay in the vector unit: quads, then
// mirrors of 8 and 16 lanes, which join sums that are already alike within
// each half.
template <int G>
__device__ __forceinline__ float lane_sum(float v) {
    auto dpp = [](float x, auto ctrl) {
        return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(
            0, __builtin_bit_cast(int, x), decltype(ctrl)::value, 0xf, 0xf, true));
    };
    v += dpp(v, std::integral_constant<int, 0xB1>{});   // quad_perm 1,0,3,2
    v += dpp(v, std::integral_constant<int, 0x4E>{});   // quad_perm 2,3,0,1
    if (G >= 8) v += dpp(v, std::integral_constant<int, 0x141>{});   // row_half_mirror
    if (G >= 16) v += dpp(v, std::integral_constant<int, 0x140>{});  // row_mirror
    if (G >= 32) v += __shfl_xor(v, 16, kWave);
    if (G >= 64) v += __shfl_xor(v, 32, kWave);
    return v;
}

// Sum over a block of `waves` waves; every thread gets it.  A barrier is
// passed before `lds` is written, so it can be used again at once.
__device__ __forceinline__ float block_sum(float v, float* lds, int waves = 4) {
    v = lane_sum<64>(v);
    __syncthreads();
    if (lane_id() == 0) lds[threadIdx.x >> 6] = v;
    __syncthreads();
    float s = 0.f;
    for (int i = 0; i < waves; ++i) s += lds[i];
    return s;
}

// Where chunk `ch` of V columns lies in a row of `cols` >= V: the last one is
// moved back to end with the row, its first `skip` columns being the chunk
// before's (they count in no sum; stores write them twice, the same value).  A
// chunk past the row counts nothing (skip = V) and reads column 0.
template <int V>
struct Chunk {
    int at, skip;
    bool in;
    __device__ __forceinline__ Chunk(int ch, int cols) {
        const int c = ch * V;
        in = c < cols;
        at = in ? (c < cols - V ? c : cols - V) : 0;
        skip = in ? c - at : V;
    }
};

// A row in the registers of G lanes, NV chunks of V values each: read once,
// the mean and then the centred squares summed from registers, written once.
// G <= 64: 256 / G rows a block; above: a block of G threads per row.  The
// variance is of the differences from the mean, so a far mean costs no digits.
// Measured: 65536 x 128 float32 14.2 us (4.7 TB/s), 16384 x 4096 bfloat16 54 us
// (4.9 TB/s), 4099 x 1001 float16 (rows at odd addresses) 6.7 us, 4 x 1024
// 3.3 us; three passes over a row with single loads took 85 us for the first.
template <class T, class W, int V, int NV, int G>
__global__ __launch_bounds__(G < 256 ? 256 : G) void k_ln_fwd(const T* x, int64_t xs,
                                                             int64_t rows, int cols, const W* w,
                                                             const W* b, float eps, T* y,
                                                             int64_t ys, float* mean,
                                                             float* rstd) {
    constexpr int RPB = G < 256 ? 256 / G : 1;
    __shared__ float lds[G < 256 ? 1 : G / 64];
    const int gl = G < 256 ? threadIdx.x % G : threadIdx.x;
    const int64_t step = (int64_t)gridDim.x * RPB;
    const float n = (float)cols;  // divided by: a constant row has exactly its value as mean
    for (int64_t r0 = (int64_t)blockIdx.x * RPB; r0 < rows; r0 += step) {
        const int64_t rr = r0 + (G < 256 ? threadIdx.x / G : 0);
        const int64_t r = rr < rows ? rr : rows - 1;  // spare groups redo the last row, unwritten
        float v[NV][V];
#pragma unroll
        for (int k = 0; k < NV; ++k) load_v<T, V>(x + r * xs + Chunk<V>(k * G + gl, cols).at, v[k]);
        float s = 0.f;
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const Chunk<V> c(k * G + gl, cols);
#pragma unroll
            for (int e = 0; e < V; ++e) s += e >= c.skip ? v[k][e] : 0.f;
        }
        const float mu = (G < 256 ? lane_sum<G>(s) : block_sum(s, lds, G / 64)) / n;
        float q = 0.f;
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const Chunk<V> c(k * G + gl, cols);
#pragma unroll
            for (int e = 0; e < V; ++e) {
                v[k][e] -= mu;
                q += e >= c.skip ? v[k][e] * v[k][e] : 0.f;
            }
        }
        const float rs =
            1.0f / sqrtf((G < 256 ? lane_sum<G>(q) : block_sum(q, lds, G / 64)) / n + eps);
        if (gl == 0 && rr < rows) {
            if (mean) mean[r] = mu;
            if (rstd) rstd[r] = rs;
        }
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const Chunk<V> c(k * G + gl, cols);
            float wv[V], bv[V];
            if (w) load_v<W, V>(w + c.at, wv);
            if (b) load_v<W, V>(b + c.at, bv);
#pragma unroll
            for (int e = 0; e < V; ++e) {
                float o = v[k][e] * rs;
                if (w) o *= wv[e];
                if (b) o += bv[e];
                v[k][e] = o;
            }
            if (c.in && rr < rows) store_v<T, V>(y + r * ys + c.at, v[k]);
        }
    }
}

// Rows too wide for registers (over 32768 columns of 16 bits, 16384 of 32; backward
// over 16384).  One block per row, any width: the row is read once for the mean, again for
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

// dx of one row per block, any width: two passes over the row, the second mostly
// from cache.  2000 x 20000 bfloat16: 77 us, and 56 us for the column sums.
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

// The whole backward pass of the rows of one slice (blockIdx.x): each group of
// G lanes takes every (groups)th row of it, with the row's dy and x read once
// into registers, the next row's asked for before this one is worked on, and
// the lane's columns' sums of dy * xhat and dy kept in registers over all its
// rows.  At the end the block's groups are joined in LDS and written to
// part[slice][2][cols].  One pass: dx and the column sums from separate kernels
// read dy and x twice (119 us against 22 at 65536 x 128, 290 against 86 at
// 16384 x 4096).  Measured: 65536 x 128 float32 17.3 us (5.8 TB/s with what the
// last-level cache holds), 16384 x 4096 bfloat16 82 us (4.9 TB/s), 777 x 5003
// 14 us (195 blocks of 4 rows: the latency of each row's loads).  From 8193
// columns on (G = 1024) a row with its two sums a column is more than 128
// registers hold: 29 to 57 of a lane go to scratch and back; 2048 x 16384
// bfloat16 65 us and 7 for the join, for 39 at the copy's rate.
template <class T, class W, int V, int NV, int G>
__global__ __launch_bounds__(G < 256 ? 256 : G) void k_ln_bwd(
    const T* dy, int64_t ds, const T* x, int64_t xs, int64_t rows, int cols, const float* mean,
    const float* rstd, const W* w, T* dx, int64_t os, int64_t per, float* part, W* dwo,
    W* dbo) {
    constexpr int RPB = G < 256 ? 256 / G : 1;
    // 1024 threads have 128 registers each: no room for a row ahead.
    constexpr bool kAhead = G < 1024;
    __shared__ float lds[G < 256 ? 1 : 4 * (G / 64)];
    typedef typename Pack<T, V>::type P;
    const int gl = G < 256 ? threadIdx.x % G : threadIdx.x;
    const int grp = G < 256 ? threadIdx.x / G : 0;
    const float inv = 1.0f / (float)cols;
    const int64_t r0 = (int64_t)blockIdx.x * per, r1 = r0 + per < rows ? r0 + per : rows;
    float dw[NV][V] = {}, db[NV][V] = {};
    float wv[NV][V];
#pragma unroll
    for (int k = 0; k < NV; ++k) {
        if (w)
            load_v<W, V>(w + Chunk<V>(k * G + gl, cols).at, wv[k]);
        else
            for (int e = 0; e < V; ++e) wv[k][e] = 1.f;
    }
    P nd[NV], nx[NV];
    float nmu = 0.f, nrs = 0.f;
    auto fetch = [&](int64_t q) {
        const int64_t r = q < rows ? q : rows - 1;
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const int at = Chunk<V>(k * G + gl, cols).at;
            nd[k] = *reinterpret_cast<const P*>(dy + r * ds + at);
            nx[k] = *reinterpret_cast<const P*>(x + r * xs + at);
        }
        nmu = mean[r];
        nrs = rstd[r];
    };
    if (kAhead) fetch(r0 + grp);
    int parity = 0;
    for (int64_t rb = r0; rb < r1; rb += RPB) {
        const int64_t r = rb + grp;
        const bool live = r < r1;
        P d[NV], h[NV];
        if (!kAhead) fetch(r);
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            d[k] = nd[k];
            h[k] = nx[k];
        }
        const float mu = nmu, rs = live ? nrs : 0.f;
        if (kAhead && rb + RPB < r1) fetch(r + RPB);
        float s1 = 0.f, s2 = 0.f;
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const Chunk<V> c(k * G + gl, cols);
#pragma unroll
            for (int e = 0; e < V; ++e) {
                const bool on = live && e >= c.skip;
                float g, xv;
                if constexpr (V == 1) {
                    g = (float)d[k];
                    xv = (float)h[k];
                } else {
                    g = (float)d[k][e];
                    xv = (float)h[k][e];
                }
                const float hat = (xv - mu) * rs;
                const float z = g * wv[k][e];
                s1 += on ? z : 0.f;
                s2 += on ? z * hat : 0.f;
                dw[k][e] += on ? g * hat : 0.f;
                db[k][e] += on ? g : 0.f;
            }
        }
        if constexpr (G < 256) {
            s1 = lane_sum<G>(s1);
            s2 = lane_sum<G>(s2);
        } else {
            // One barrier a row: the two halves of lds take turns.
            s1 = lane_sum<64>(s1);
            s2 = lane_sum<64>(s2);
            float* l = lds + parity * 2 * (G / 64);
            parity ^= 1;
            if (lane_id() == 0) {
                l[2 * (threadIdx.x >> 6)] = s1;
                l[2 * (threadIdx.x >> 6) + 1] = s2;
            }
            __syncthreads();
            s1 = s2 = 0.f;
#pragma unroll
            for (int i = 0; i < G / 64; ++i) {
                s1 += l[2 * i];
                s2 += l[2 * i + 1];
            }
        }
        if (dx != nullptr) {
            const float m1 = s1 * inv, m2 = s2 * inv;
#pragma unroll
            for (int k = 0; k < NV; ++k) {
                const Chunk<V> c(k * G + gl, cols);
                float o[V];
#pragma unroll
                for (int e = 0; e < V; ++e) {
                    float g, xv;
                    if constexpr (V == 1) {
                        g = (float)d[k];
                        xv = (float)h[k];
                    } else {
                        g = (float)d[k][e];
                        xv = (float)h[k][e];
                    }
                    o[e] = rs * (g * wv[k][e] - m1 - (xv - mu) * rs * m2);
                }
                if (live && c.in) store_v<T, V>(dx + r * os + c.at, o);
            }
        }
    }
    if (part == nullptr) return;
    float* p = part + (int64_t)blockIdx.x * 2 * cols;
    // A single slice's sums are the gradients.
    auto put = [&](int col, float sw, float sb) {
        if (gridDim.x > 1) {
            p[col] = sw;
            p[cols + col] = sb;
            return;
        }
        if (dwo) dwo[col] = (W)sw;
        if (dbo) dbo[col] = (W)sb;
    };
    if constexpr (G < 256) {
        // Lane gl of every group holds the same columns: join the groups.
        __shared__ float jw[RPB][G * NV * V], jb[RPB][G * NV * V];
#pragma unroll
        for (int k = 0; k < NV; ++k)
#pragma unroll
            for (int e = 0; e < V; ++e) {
                jw[grp][(k * G + gl) * V + e] = dw[k][e];
                jb[grp][(k * G + gl) * V + e] = db[k][e];
            }
        __syncthreads();
        for (int i = threadIdx.x; i < G * NV * V; i += 256) {
            const Chunk<V> c(i / V, cols);
            if (i % V < c.skip) continue;
            float sw = 0.f, sb = 0.f;
#pragma unroll
            for (int q = 0; q < RPB; ++q) {
                sw += jw[q][i];
                sb += jb[q][i];
            }
            put(c.at + i % V, sw, sb);
        }
    } else {
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const Chunk<V> c(k * G + gl, cols);
            if (c.skip == 0 && gridDim.x > 1) {
                store_v<float, V>(p + c.at, dw[k]);
                store_v<float, V>(p + cols + c.at, db[k]);
                continue;
            }
#pragma unroll
            for (int e = 0; e < V; ++e)
                if (e >= c.skip) put(c.at + e, dw[k][e], db[k][e]);
        }
    }
}

// Sums of dy * xhat and dy over one slice of rows (blockIdx.y) for 64 columns
// from c0 on: four rows at a time, joined in LDS.  part: [slices][2][cols].
template <class T>
__global__ __launch_bounds__(256) void k_ln_cols_any(const T* dy, int64_t ds, const T* x,
                                                     int64_t xs, int64_t rows, int64_t cols,
                                                     const float* mean, const float* rstd,
                                                     int64_t per, float* part, int64_t c0) {
    __shared__ float lw[4][64], lb[4][64];
    const int lane = lane_id(), k = threadIdx.x >> 6;
    const int64_t c = c0 + (int64_t)blockIdx.x * 64 + lane;
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

// dweight and dbias from the slices' sums: a block takes 32 columns of one of
// the two, 16 threads on each column's slices, joined in double in a fixed
// order.  Latency bounds it: 4 to 7 us up to 256 slices of 16384 columns, 12 us
// for 250 of 20000, with eight loads in flight (23 us for 512 slices of 16384
// columns with one).
template <class W>
__global__ __launch_bounds__(512) void k_ln_join(const float* part, int64_t slices, int64_t cols,
                                                 W* dw, W* db, int64_t c0) {
    __shared__ double l[16][33];
    const int q = threadIdx.x & 31, k = threadIdx.x >> 5;
    const int64_t c = c0 + (int64_t)blockIdx.x * 32 + q;
    W* out = blockIdx.y ? db : dw;
    if (out == nullptr) return;
    double s = 0.;
    if (c < cols) {
        const float* p = part + blockIdx.y * cols + c;
        int64_t i = k;
        for (; i + 112 < slices; i += 128) {  // eight loads at once
            float v[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] = p[(i + 16 * e) * 2 * cols];
#pragma unroll
            for (int e = 0; e < 8; ++e) s += (double)v[e];
        }
        for (; i < slices; i += 16) s += (double)p[i * 2 * cols];
    }
    l[k][q] = s;
    __syncthreads();
    if (k != 0 || c >= cols) return;
    s = 0.;
#pragma unroll
    for (int e = 0; e < 16; ++e) s += l[e][q];
    out[c] = (W)(float)s;
}

// How a row is shared out: G lanes of NV chunks of V values hold it.
struct RowPlan {
    int g, nv;     // 0: no kernel holds a row this wide
    bool one;      // fewer columns than a vector: single values, 16 lanes
};

// 16-byte chunks.  Few lanes on narrow rows, so that every lane loads; a wave
// up to 32 values a lane forward (16 backward, which keeps dy, x and two sums
// of each), a block beyond, as then several rows' loads still fit a CU.
static RowPlan ln_plan(int64_t cols, int v, bool backward) {
    static const RowPlan fwd[] = {{4, 1}, {8, 1}, {16, 1}, {32, 1}, {64, 1}, {64, 2}, {64, 4}, {256, 2}, {256, 4},
                                  {256, 8}, {1024, 4}};
    static const RowPlan bwd[] = {{4, 1}, {8, 1}, {16, 1}, {32, 1}, {64, 1}, {64, 2}, {256, 1}, {256, 2}, {512, 2},
                                  {1024, 2}, {1024, 4}};
    if (cols < v) return {16, 1, true};
    if (backward) {
        for (const RowPlan& p : bwd)
            if (cols <= (int64_t)p.g * p.nv * v && p.nv * v <= 16) return p;
    } else {
        for (const RowPlan& p : fwd)
            if (cols <= (int64_t)p.g * p.nv * v) return p;
    }
    return {0, 0, false};
}

// Row slices of the column sums, one block each.  Of narrow rows a block takes
// several at a time: slices of 16 rows and more, 1024 at most.  Of wide ones a
// slice's sums are as long as a row, 8 bytes a column against 6 or 12 that a
// row reads and writes: 256 slices fill the card, more only while their sums
// stay below an eighth of the rows' traffic (2048 x 16384 bfloat16, 512 slices:
// half of it), 512 at most.  Rows that one block is through with in four rounds
// are one slice, whose sums need no second launch (4 x 1024: 3.5 us of kernels
// for 6.4, 12 us for 16 on the host).
static int64_t ln_slices(int64_t rows, int64_t cols, int64_t bytes, int64_t* per) {
    const RowPlan p = ln_plan(cols, (int)(16 / bytes), true);
    if (p.g != 0 && rows <= 4 * (p.g < 256 ? 256 / p.g : 1)) {
        *per = rows < 1 ? 1 : rows;
        return 1;
    }
    int64_t s = cols <= 1024 ? ceil_div(rows, 16) : rows * 3 * bytes / 64;
    if (cols > 1024 && s < 256) s = 256;
    const int64_t most = cols <= 1024 ? 1024 : 512;
    if (s > most) s = most;
    *per = s < 1 ? 1 : ceil_div(rows, s);
    if (*per < 1) *per = 1;
    s = ceil_div(rows, *per);  // no empty slice
    return s < 1 ? 1 : s;
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

template <int N>
using Int = std::integral_constant<int, N>;

// Calls launch(c0, blocks) for ranges of the columns, `per` a block: HIP takes
// fewer than 2^32 threads along an axis.  (Further columns in turn by each block
// instead made k_ln_cols_any 62 us for 56 at 2000 x 20000.)
template <class F>
static void by_columns(int64_t cols, int per, F&& launch) {
    const int64_t range = (int64_t)per << 20;
    for (int64_t c0 = 0; c0 < cols; c0 += range)
        launch(c0, (unsigned)ceil_div(cols - c0 < range ? cols - c0 : range, per));
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
    // The kernels add it in float32: one that becomes 0 there would divide a constant row by 0.
    if (!((float)eps > 0.f) || !isfinite((float)eps))
        return fail(SPOPT_EINVAL, "layer_norm_forward: eps must be finite and > 0 in float32");
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
        constexpr int V = 16 / sizeof(T);
        const RowPlan p = ln_plan(cols, V, false);
        auto go = [&](auto v, auto nv, auto g) {
            constexpr int G = decltype(g)::value;
            const unsigned grid = row_grid(ceil_div(rows, G < 256 ? 256 / G : 1));
            k_ln_fwd<T, W, decltype(v)::value, decltype(nv)::value, G>
                <<<grid, G < 256 ? 256 : G, 0, s>>>((const T*)x, x_stride, rows, (int)cols,
                                                    (const W*)weight, (const W*)bias, (float)eps,
                                                    (T*)y, y_stride, mean, rstd);
        };
        auto at = [&](auto nv, auto g) { go(Int<V>{}, nv, g); };
        if (p.one) go(Int<1>{}, Int<1>{}, Int<16>{});
        else if (p.g == 4) at(Int<1>{}, Int<4>{});
        else if (p.g == 8) at(Int<1>{}, Int<8>{});
        else if (p.g == 16) at(Int<1>{}, Int<16>{});
        else if (p.g == 32) at(Int<1>{}, Int<32>{});
        else if (p.g == 64 && p.nv == 1) at(Int<1>{}, Int<64>{});
        else if (p.g == 64 && p.nv == 2) at(Int<2>{}, Int<64>{});
        else if (p.g == 64) at(Int<4>{}, Int<64>{});
        else if (p.g == 256 && p.nv == 2) at(Int<2>{}, Int<256>{});
        else if (p.g == 256 && p.nv == 4) at(Int<4>{}, Int<256>{});
        else if (p.g == 256) at(Int<8>{}, Int<256>{});
        else if (p.g == 1024) at(Int<4>{}, Int<1024>{});
        else
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
    int64_t per;
    const int64_t two = ln_slices(rows, cols, 2, &per), four = ln_slices(rows, cols, 4, &per);
    *bytes = (size_t)(two > four ? two : four) * 2 * (size_t)cols * sizeof(float);
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
    int64_t per;
    int64_t slices = ln_slices(rows, cols, (int64_t)dtype_bytes(dtype), &per);
    if (rows == 0) slices = 0;
    ln_types(dtype, wdtype, [&](auto t, auto wt) {
        using T = decltype(t);
        using W = decltype(wt);
        constexpr int V = 16 / sizeof(T);
        float* part = sums ? (float*)workspace : nullptr;
        const RowPlan p = ln_plan(cols, V, true);
        auto go = [&](auto v, auto nv, auto g) {
            constexpr int G = decltype(g)::value;
            k_ln_bwd<T, W, decltype(v)::value, decltype(nv)::value, G>
                <<<(unsigned)slices, G < 256 ? 256 : G, 0, s>>>(
                    (const T*)dy, dy_stride, (const T*)x, x_stride, rows, (int)cols, mean, rstd,
                    (const W*)weight, (T*)dx, dx_stride, per, part, (W*)dweight, (W*)dbias);
        };
        auto at = [&](auto nv, auto g) { go(Int<V>{}, nv, g); };
        if (rows == 0 || (!sums && dx == nullptr)) {
        } else if (p.one) go(Int<1>{}, Int<1>{}, Int<16>{});
        else if (p.g == 4) at(Int<1>{}, Int<4>{});
        else if (p.g == 8) at(Int<1>{}, Int<8>{});
        else if (p.g == 16) at(Int<1>{}, Int<16>{});
        else if (p.g == 32) at(Int<1>{}, Int<32>{});
        else if (p.g == 64 && p.nv == 1) at(Int<1>{}, Int<64>{});
        else if (p.g == 64) at(Int<2>{}, Int<64>{});
        else if (p.g == 256 && p.nv == 1) at(Int<1>{}, Int<256>{});
        else if (p.g == 256 && p.nv == 2) at(Int<2>{}, Int<256>{});
        else if (p.g == 512) at(Int<2>{}, Int<512>{});
        else if (p.g == 1024 && p.nv == 2) at(Int<2>{}, Int<1024>{});
        else if (p.g == 1024) {
            if constexpr (sizeof(T) == 4) at(Int<4>{}, Int<1024>{});
        } else {
            // Wider rows: the column sums first, as dx may lie over dy or x.
            if (sums)
                by_columns(cols, 64, [&](int64_t c0, unsigned blocks) {
                    k_ln_cols_any<T><<<dim3(blocks, (unsigned)slices), 256, 0, s>>>(
                        (const T*)dy, dy_stride, (const T*)x, x_stride, rows, cols, mean, rstd,
                        per, part, c0);
                });
            if (dx != nullptr)
                k_ln_dx_any<T, W><<<row_grid(rows), 256, 0, s>>>(
                    (const T*)dy, dy_stride, (const T*)x, x_stride, rows, cols, mean, rstd,
                    (const W*)weight, (T*)dx, dx_stride);
        }
        const bool direct = p.g != 0 && slices == 1;
        if (sums && !direct)
            by_columns(cols, 32, [&](int64_t c0, unsigned blocks) {
                k_ln_join<W><<<dim3(blocks, 2), 512, 0, s>>>(part, slices, cols, (W*)dweight,
                                                             (W*)dbias, c0);
            });
    });
    SPOPT_LAUNCHED();
    return SPOPT_OK;
}
