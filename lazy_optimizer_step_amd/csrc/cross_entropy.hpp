// cross_entropy.hpp - what the loss's two sets of kernels share: those of packed
// operands (cross_entropy.hip) and those that read theirs as they are
// (cross_entropy_direct.hip).
#pragma once

#include <math.h>

#include <type_traits>

#include "dense.hpp"
#include "matrix.hpp"

namespace spopt {

typedef __bf16 bhalf8 __attribute__((ext_vector_type(8)));

__device__ __forceinline__ float4v matrix_16x16x32(half8 a, half8 b, float4v c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
}
__device__ __forceinline__ float4v matrix_16x16x32(bhalf8 a, bhalf8 b, float4v c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}

// What a call's kernels hand on to the next ones.
struct CeScalars {
    int ex, ew;  // powers of two in front of the operands x and W (float32)
    int ek;      // g is times 2^ek / mu
    float mu;
};

// What is done with a tile of the logits.
struct CeLogits {
    const CeScalars* scalars;
    const int64_t* targets;
    int64_t first;       // class of the piece's first column
    int64_t classes;     // of all pieces
    float smoothing;
    // forward
    float2* parts;       // [tile of classes][row]: maximum, sum of exponentials
    float* sums;         // [tile of classes][row]: sum of the logits (smoothing only)
    float* at_target;    // [row]
    int64_t first_tile;
    // backward
    const float* lse;
    const float* coef;   // [row] c_i 2^ek / mu
    void* g;             // [row][ldg]
    int64_t ldg, rows_p, cols_p;  // g's extent, zeros beyond the matrix
};

enum : int { kCeLoss = 0, kCeGrad = 1, kCeDx = 2, kCeDw = 3 };

// Tile `t` of a product, four rows of tiles at a time, column by column.
__device__ __forceinline__ void ce_place(int64_t t, int64_t tm, int64_t tn, int64_t* ti,
                                         int64_t* tj) {
    const int64_t band = t / (4 * tn), in = t % (4 * tn);
    const int64_t rows = tm - 4 * band < 4 ? tm - 4 * band : 4;
    *ti = 4 * band + in % rows;
    *tj = in / rows;
}

// The column of class `target` in a tile whose first is `first`; -1 where it lies
// far from it.
__device__ __forceinline__ int ce_column(int64_t target, int64_t first) {
    const uint64_t j = (uint64_t)target - (uint64_t)first;
    return j < 4096 ? (int)j : -1;
}

constexpr float kLog2e = 1.44269504088896340736f;

// exp(z - b), the difference formed before it is scaled.
__device__ __forceinline__ float exp_less(float z, float b) {
    return __builtin_amdgcn_exp2f((z - b) * kLog2e);
}

// A tile of the logits, one of `tn` in a row of the piece's, in the lanes of a
// block's WGN columns of waves: each row's maximum, its sum of exponentials and of
// logits into the tile's places, and the target's logit into its own.  `red`:
// 3 BM WGN floats of LDS that no wave reads or awaits any more.
template <int BM, int BN, int WGN, class Tile, class S>
__device__ __forceinline__ void ce_loss_tile(Tile& tile, float* red, int64_t i0, int64_t j0,
                                             int64_t tj, int64_t m, int64_t n, const CeLogits& w,
                                             S scale) {
    const bool whole = j0 + BN <= n;
    const int wn = tile.wv % WGN;
    __syncthreads();
#pragma unroll
    for (int x = 0; x < Tile::FM; ++x) {
        const int r = tile.row_of(x);
        const int64_t i = i0 + r;
        const int t = i < m ? ce_column(w.targets[i], w.first + j0) : -1;
        float top = -INFINITY, z = 0.f, s = 0.f;
#pragma unroll
        for (int y = 0; y < Tile::FN; ++y)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                float v = scale(tile.acc[x][y][e]);
                const int j = tile.col_of(y) + e;
                if (whole || j0 + j < n) {
                    z += v;
                    if (j == t) w.at_target[i] = v;
                } else {
                    v = -INFINITY;
                }
                tile.acc[x][y][e] = v;
                top = fmaxf(top, v);
            }
        top = fmaxf(top, __shfl_xor(top, 16, kWave));
        top = fmaxf(top, __shfl_xor(top, 32, kWave));
        const float base = top == -INFINITY ? 0.f : top;
#pragma unroll
        for (int y = 0; y < Tile::FN; ++y)
#pragma unroll
            for (int e = 0; e < 4; ++e) s += exp_less(tile.acc[x][y][e], base);
        s += __shfl_xor(s, 16, kWave);
        s += __shfl_xor(s, 32, kWave);
        z += __shfl_xor(z, 16, kWave);
        z += __shfl_xor(z, 32, kWave);
        if (tile.lane < 16) {
            red[(wn * 3 + 0) * BM + r] = top;
            red[(wn * 3 + 1) * BM + r] = s;
            red[(wn * 3 + 2) * BM + r] = z;
        }
    }
    __syncthreads();
    for (int r = threadIdx.x; r < BM; r += blockDim.x) {
        if (i0 + r >= m) break;
        float top = -INFINITY, s = 0.f, z = 0.f;
#pragma unroll
        for (int k = 0; k < WGN; ++k) top = fmaxf(top, red[k * 3 * BM + r]);
        const float base = top == -INFINITY ? 0.f : top;
#pragma unroll
        for (int k = 0; k < WGN; ++k) {
            s += red[(k * 3 + 1) * BM + r] * exp_less(red[k * 3 * BM + r], base);
            z += red[(k * 3 + 2) * BM + r];
        }
        const int64_t at = (w.first_tile + tj) * m + i0 + r;
        w.parts[at] = make_float2(top, s);
        if (w.sums) w.sums[at] = z;
    }
}

// g of a tile of the logits, coef(i) the factor of row i.  Split: hi and lo.
template <class T, bool SPLIT, int BN, class Tile, class S, class C>
__device__ __forceinline__ void ce_grad_tile(const Tile& tile, int64_t i0, int64_t j0, int64_t m,
                                             int64_t n, const CeLogits& w, S scale, C coef_of) {
    constexpr int V = Tile::kRow;  // adjacent columns of a lane
    T* const g = (T*)w.g;
    const bool whole = j0 + BN <= n;
    const float off = w.smoothing / (float)w.classes, on = 1.f - w.smoothing;
#pragma unroll
    for (int x = 0; x < Tile::FM; ++x) {
        const int64_t i = i0 + tile.row_of(x);
        if (i >= w.rows_p) continue;
        const bool row = i < m;
        const int t = row ? ce_column(w.targets[i], w.first + j0) : -1;
        const float coef = row ? coef_of(i) : 0.f, lse = row ? w.lse[i] : 0.f;
#pragma unroll
        for (int y = 0; y < Tile::FN; y += V / 4) {
            const int j = tile.col_of(y);
            if (j0 + j >= w.cols_p) continue;
            float v[V];
#pragma unroll
            for (int e = 0; e < V; ++e) {
                float p = exp_less(scale(tile.acc[x][y + e / 4][e & 3]), lse) - off;
                if (j + e == t) p -= on;
                p *= coef;
                // Rows that do not count may hold anything.
                v[e] = coef == 0.f || (!whole && j0 + j + e >= n) ? 0.f : p;
            }
            if constexpr (SPLIT) {
                float lo[V];
#pragma unroll
                for (int e = 0; e < V; ++e) lo[e] = v[e] - (float)(T)v[e];
                T* to = g + i * w.ldg + (j0 + j) / 32 * 64 + (j0 + j) % 32;
                store_v<T, V>(to, v);
                store_v<T, V>(to + 32, lo);
            } else {
                store_v<T, V>(g + i * w.ldg + j0 + j, v);
            }
        }
    }
}

// Where a product's result goes: sums in float32, [row][ld], added to what is
// there or not; or (parts NULL) scaled and rounded to where it belongs.
struct CeResult {
    float* parts;
    int64_t ld;
    int add;
    void* out;
    int64_t out_ld;
};

template <class O, class Tile, class S>
__device__ __forceinline__ void ce_store_tile(const Tile& tile, int64_t i0, int64_t j0, int64_t m,
                                              int64_t n, const CeResult& w, float* parts,
                                              S scale) {
#pragma unroll
    for (int x = 0; x < Tile::FM; ++x) {
        const int64_t i = i0 + tile.row_of(x);
        if (i >= m) continue;
#pragma unroll
        for (int y = 0; y < Tile::FN; ++y) {
            const int64_t j = j0 + tile.col_of(y);
            if (parts != nullptr) {
                if (j >= w.ld) continue;
                float4v* const to = (float4v*)(parts + i * w.ld + j);
                *to = w.add ? *to + tile.acc[x][y] : tile.acc[x][y];
                continue;
            }
            float v[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) v[e] = scale(tile.acc[x][y][e]);
            O* const to = (O*)w.out + i * w.out_ld + j;
            if (j + 4 <= n) {
                store_v<O, 4>(to, v);
            } else {
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (j + e < n) to[e] = (O)v[e];
            }
        }
    }
}

__device__ __forceinline__ double ce_block_sum(double v, double* lds) {
#pragma unroll
    for (int off = kWave / 2; off; off >>= 1) v += __shfl_xor(v, off, kWave);
    __syncthreads();
    if (lane_id() == 0) lds[threadIdx.x >> 6] = v;
    __syncthreads();
    double s = 0.;
    for (int i = 0; i < (int)(blockDim.x >> 6); ++i) s += lds[i];
    return s;
}

enum : int {
    kCeNone = SPOPT_REDUCE_NONE,
    kCeSum = SPOPT_REDUCE_SUM,
    kCeMean = SPOPT_REDUCE_MEAN
};

// What a row's factor c_i is made of.
struct CeRows {
    const float* dloss;
    const int64_t* targets;
    int64_t ignored, rows, classes;
    int reduction;
    float on;  // 1 - smoothing
};

// c_i times the number that brings the largest gradient that is to be expected,
// (1 - smoothing) max |c| at a target of no probability, to 2^13.  float16 then
// holds small probabilities; and of a call whose rows count alike the gradients
// at the targets, the largest by far, lie just below a power of two, where
// rounding takes least of them (with 2^13 times a mantissa that may lie
// anywhere, gradients of bfloat16 and float16 were off by 1.2 to 1.48 times what
// the rounding of the results alone does; now by ... ).
struct CeFactor {
    float one, inv;
    int ek;
    float mu;
    // By all threads of a block.  `plain`: the factors as they are, for a float32 g.
    __device__ __forceinline__ void init(const CeRows& a, bool plain, double* lds,
                                         float* top_of) {
        double n = 0.;
        float top = 0.f;
        for (int64_t i = threadIdx.x; i < a.rows; i += blockDim.x) {
            if (a.targets[i] == a.ignored) continue;
            n += 1.;
            if (!plain && a.reduction == kCeNone && finite_f(a.dloss[i]))
                top = fmaxf(top, fabsf(a.dloss[i]));
        }
        one = 0.f;
        if (a.reduction == kCeNone) {
            if (!plain) {
#pragma unroll
                for (int off = kWave / 2; off; off >>= 1)
                    top = fmaxf(top, __shfl_xor(top, off, kWave));
                if (lane_id() == 0) top_of[threadIdx.x >> 6] = top;
                __syncthreads();
                for (int k = 0; k < (int)(blockDim.x >> 6); ++k) top = fmaxf(top, top_of[k]);
            }
        } else {
            one = a.dloss[0];
            if (a.reduction == kCeMean)
                one = (float)((double)one / fmax(ce_block_sum(n, lds), 1.));
            top = fabsf(one);
        }
        ek = 0;
        mu = inv = 1.f;
        if (!plain && top > 0.f && finite_f(top)) {
            // Where 1 - smoothing is small, what is expected is not the largest.
            mu = frexpf(top * fmaxf(a.on, 0.5f), &ek);
            inv = 1.f / mu;
            ek = 13 - ek;
        }
    }
    __device__ __forceinline__ float of(const CeRows& a, int64_t i) const {
        const int64_t t = a.targets[i];
        if (t == a.ignored) return 0.f;
        if (t < 0 || t >= a.classes) return NAN;
        return ldexpf((a.reduction == kCeNone ? a.dloss[i] : one) * inv, ek);
    }
};

// What brings a sum of products with g back.
__device__ __forceinline__ float ce_unscale(float v, float mu, int e) { return ldexpf(v * mu, -e); }

// ------------------------------------------------------------- direct ---

// An operand as the caller laid it out, or g in the workspace: rows of `cols`
// values, those whose target is `ignored` taken as zeros.
struct CeSide {
    const void* base;
    int64_t ld, rows, cols;
    const int64_t* targets;  // or NULL
    int64_t ignored;
};

// The two products of the gradients: tiles of dx come first, then those of dW.
struct CeBoth {
    CeSide g, w, x;
    CeResult dx, dw;
    int64_t rows, cols, classes;
    int64_t dx_tiles, dw_tiles;  // 0 where not wanted
    int dx_tile, dw_tile;        // rows of a tile
    int dx_splits, dw_splits;
    const CeScalars* scalars;
};

// `tile`: rows of a tile, 16 or 64.
int ce_direct_loss(int32_t dtype, int tile, const CeSide& x, const CeSide& w, const CeLogits& l,
                   hipStream_t s);
int ce_direct_grad(int32_t dtype, int tile, const CeSide& x, const CeSide& w, const CeLogits& l,
                   const CeRows& rows, CeScalars* scalars, hipStream_t s);
int ce_direct_products(int32_t dtype, const CeBoth& b, hipStream_t s);

}  // namespace spopt
