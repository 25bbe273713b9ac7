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

typedef float float16v __attribute__((ext_vector_type(16)));

__device__ __forceinline__ float16v matrix_32x32x16(half8 a, half8 b, float16v c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(a, b, c, 0, 0, 0);
}
__device__ __forceinline__ float16v matrix_32x32x16(bhalf8 a, bhalf8 b, float16v c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
}

// What a call's kernels hand on to the next ones.
struct CeScalars {
    int ex, ew;  // powers of two in front of the operands x and W (float32)
    int ed;      // and of x as dW's operand
    int ek;      // g is times 2^ek / mu, and a power of two of each row (CeRows::powers)
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
    float2* parts;       // [part of the classes][row]: maximum, sum of exponentials
    float* sums;         // [part][row]: sum of the logits (smoothing only)
    float* at_target;    // [row]
    int64_t first_part;
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

constexpr float kLog2e = 1.44269504088896340736f;

// exp(z - b), the difference formed before it is scaled.
__device__ __forceinline__ float exp_less(float z, float b) {
    return __builtin_amdgcn_exp2f((z - b) * kLog2e);
}

// A tile's struct says where its result lies: row_of(x), x < FM, is the row of a
// lane's values of row x, which kRowLanes lanes apart others share; col_of(y), y <
// FN, the first of the four adjacent columns of at(x, y, 0 .. 3).

// 2^exponent, within [2^-120, 2^120]: sums of products of split operands lie in
// [2^-48, 2^50], so that beyond it logits are infinite, or zero beside any exponential.
__device__ __forceinline__ float ce_logit_scale(int exponent) {
    return ldexpf(1.f, exponent < -120 ? -120 : exponent > 120 ? 120 : exponent);
}

// The rows of a lane while the classes' tiles go by: a base, the sum of exponentials
// under it and the sum of the logits, over this lane's columns.  A part may be a
// whole table of classes, thousands of tiles: a tile's few values are added up in
// float32, and tiles in double.  (In float32 a class of probability near 1 early in
// the table leaves the later ones' shares no bits: with 0.999 there and 131072
// classes in one part, the loss came out 6% low.  Double costs 4% of 8192 x 128 x
// 50021 float32.)  The base is the largest logit so far or less than a factor of 2
// below it: so the sum is scaled anew only where it at least doubles, and the factors'
// roundings do not add up either.  Bases are of z / scale, scale a power of two.
template <class Tile>
struct CeRowSums {
    float top[Tile::FM];
    double s[Tile::FM], z[Tile::FM];
    int target[Tile::FM];  // its column in the piece; -1 where that lies elsewhere
    float scale, to_bits;  // scale * log2 e
    float step;            // a factor of 2, in z / scale

    __device__ __forceinline__ void init(const Tile& tile, const CeLogits& w, int64_t i0,
                                         int64_t m, int64_t n, int exponent) {
        scale = ce_logit_scale(exponent);
        to_bits = scale * kLog2e;
        step = ce_logit_scale(-exponent) / kLog2e;
#pragma unroll
        for (int x = 0; x < Tile::FM; ++x) {
            const int64_t i = i0 + tile.row_of(x);
            const int64_t t = i < m ? w.targets[i] - w.first : -1;
            target[x] = t >= 0 && t < n ? (int)t : -1;
            top[x] = -INFINITY;
            s[x] = z[x] = 0.;
        }
    }

    // A tile's logits, from column j0 of the piece's n on.
    template <int BN, int WGN>
    __device__ __forceinline__ void add(const Tile& tile, const CeLogits& w, int64_t i0, int64_t j0,
                                        int64_t n) {
        const bool whole = j0 + BN <= n;
        const int left = whole ? BN : (int)(n - j0);
#pragma unroll
        for (int x = 0; x < Tile::FM; ++x) {
            // Columns past the last weigh nothing.
            auto value = [&](int y, int e) {
                return whole || tile.col_of(y) + e < left ? tile.at(x, y, e) : -INFINITY;
            };
            float m = top[x];
#pragma unroll
            for (int y = 0; y < Tile::FN; ++y)
#pragma unroll
                for (int e = 0; e < 4; ++e) m = fmaxf(m, value(y, e));
            m = m > top[x] + step ? m : top[x];
            const float base = m == -INFINITY ? 0.f : m;
            float sum = 0.f;
#pragma unroll
            for (int y = 0; y < Tile::FN; ++y)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    sum += __builtin_amdgcn_exp2f((value(y, e) - base) * to_bits);
            s[x] = s[x] * (double)__builtin_amdgcn_exp2f((top[x] - base) * to_bits) + (double)sum;
            top[x] = m;
            if (w.sums) {
                float add = 0.f;
#pragma unroll
                for (int y = 0; y < Tile::FN; ++y)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        if (whole || tile.col_of(y) + e < left) add += tile.at(x, y, e);
                z[x] += (double)add;
            }
            // Few waves hold the target of one of their rows.
            const int t = target[x] - (int)j0;
            if (ballot(target[x] >= 0 && t >= tile.wj && t < tile.wj + BN / WGN)) {
                float hit = 0.f;
                bool found = false;
#pragma unroll
                for (int y = 0; y < Tile::FN; ++y)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        if (tile.col_of(y) + e == t) {
                            hit = tile.at(x, y, e);
                            found = target[x] >= 0;
                        }
                if (found) w.at_target[i0 + tile.row_of(x)] = hit * scale;
            }
        }
    }

    // The lanes' and waves' sums as one, into the place of part `part`.  `red`: 3 BM
    // WGN floats of LDS that no wave reads or awaits any more.
    template <int BM, int WGN>
    __device__ __forceinline__ void store(const Tile& tile, const CeLogits& w, float* red,
                                          int64_t i0, int64_t m, int64_t part) {
        __syncthreads();
        const int wn = tile.wv % WGN;
#pragma unroll
        for (int x = 0; x < Tile::FM; ++x) {
            float t = top[x], v = (float)s[x], u = (float)z[x];
#pragma unroll
            for (int off = Tile::kRowLanes; off < kWave; off <<= 1)
                t = fmaxf(t, __shfl_xor(t, off, kWave));
            v *= __builtin_amdgcn_exp2f((top[x] - (t == -INFINITY ? 0.f : t)) * to_bits);
#pragma unroll
            for (int off = Tile::kRowLanes; off < kWave; off <<= 1) {
                v += __shfl_xor(v, off, kWave);
                u += __shfl_xor(u, off, kWave);
            }
            if (tile.lane < Tile::kRowLanes) {
                const int r = tile.row_of(x);
                red[(wn * 3 + 0) * BM + r] = t;
                red[(wn * 3 + 1) * BM + r] = v;
                red[(wn * 3 + 2) * BM + r] = u;
            }
        }
        __syncthreads();
        for (int r = threadIdx.x; r < BM; r += blockDim.x) {
            if (i0 + r >= m) break;
            float t = -INFINITY, v = 0.f, u = 0.f;
#pragma unroll
            for (int k = 0; k < WGN; ++k) t = fmaxf(t, red[k * 3 * BM + r]);
            const float base = t == -INFINITY ? 0.f : t;
#pragma unroll
            for (int k = 0; k < WGN; ++k) {
                v += red[(k * 3 + 1) * BM + r] *
                     __builtin_amdgcn_exp2f((red[k * 3 * BM + r] - base) * to_bits);
                u += red[(k * 3 + 2) * BM + r];
            }
            w.parts[part * m + i0 + r] = make_float2(t * scale, v);
            if (w.sums) w.sums[part * m + i0 + r] = u * scale;
        }
    }
};

// The rows of a lane while g is formed tile by tile: with c = log2 e, 2^(c z - bits),
// bits = c lse rounded, times a factor that takes the rounding back.  A value costs
// a fused multiply-add, an exponential (at a quarter of the rate), a product and a
// select.
template <class Tile>
struct CeRowGrads {
    float coef[Tile::FM], bits[Tile::FM], factor[Tile::FM];
    int target[Tile::FM];
    float to_bits;

    template <class C>
    __device__ __forceinline__ void init(const Tile& tile, const CeLogits& w, int64_t i0,
                                         int64_t m, int64_t n, int exponent, C coef_of) {
        to_bits = ce_logit_scale(exponent) * kLog2e;
#pragma unroll
        for (int x = 0; x < Tile::FM; ++x) {
            const int64_t i = i0 + tile.row_of(x);
            const bool row = i < m;
            const int64_t t = row ? w.targets[i] - w.first : -1;
            const float lse = row ? w.lse[i] : 0.f;
            target[x] = t >= 0 && t < n ? (int)t : -1;
            coef[x] = row ? coef_of(i) : 0.f;
            bits[x] = lse * kLog2e;
            factor[x] = coef[x] * __builtin_amdgcn_exp2f(-__builtin_fmaf(lse, kLog2e, -bits[x]));
            // Rows that do not count may have any lse.
            if (coef[x] == 0.f) factor[x] = 0.f;
        }
    }

    // g of a tile; split: hi and lo.
    template <class T, bool SPLIT, int BN, int WGN>
    __device__ __forceinline__ void store(const Tile& tile, const CeLogits& w, int64_t i0,
                                          int64_t j0, int64_t n) const {
        constexpr int V = Tile::kRow;  // adjacent columns of a lane
        T* const g = (T*)w.g;
        const bool whole = j0 + BN <= n;
        const float off = w.smoothing / (float)w.classes, on = 1.f - w.smoothing;
#pragma unroll
        for (int x = 0; x < Tile::FM; ++x) {
            const int64_t i = i0 + tile.row_of(x);
            if (i >= w.rows_p) continue;
            const int t = target[x] < 0 ? -1 : target[x] - (int)j0;
            const float less = off * coef[x], once = on * coef[x];
            // Few waves hold the target of one of their rows.
            const bool hit = ballot(t >= tile.wj && t < tile.wj + BN / WGN) != 0;
#pragma unroll
            for (int y = 0; y < Tile::FN; y += V / 4) {
                const int j = tile.col_of(y);
                if (j0 + j >= w.cols_p) continue;
                float v[V];
#pragma unroll
                for (int e = 0; e < V; ++e) {
                    const float p = __builtin_amdgcn_exp2f(
                        __builtin_fmaf(tile.at(x, y + e / 4, e & 3), to_bits, -bits[x]));
                    // Rows that do not count may hold anything.
                    v[e] = factor[x] == 0.f ? 0.f : factor[x] * p;
                }
                if (w.smoothing != 0.f) {
#pragma unroll
                    for (int e = 0; e < V; ++e) v[e] -= less;
                }
                if (hit) {
#pragma unroll
                    for (int e = 0; e < V; ++e)
                        if (j + e == t) v[e] -= once;
                }
                if (!whole) {
#pragma unroll
                    for (int e = 0; e < V; ++e)
                        if (j0 + j + e >= n) v[e] = 0.f;
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
};

// Where a product's result goes: sums in float32, [row][ld], added to what is
// there or not; or (parts NULL) scaled and rounded to where it belongs.
struct CeResult {
    float* parts;
    int64_t ld;
    int add;
    void* out;
    int64_t out_ld;
    const int* powers;  // of each row, or NULL
};

template <class O, class Tile, class S>
__device__ __forceinline__ void ce_store_tile(Tile& tile, int64_t i0, int64_t j0, int64_t m,
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
                const float4v v = tile.four(x, y);
                *to = w.add ? *to + v : v;
                continue;
            }
            float v[4];
            const int power = w.powers ? w.powers[i] : 0;
#pragma unroll
            for (int e = 0; e < 4; ++e) v[e] = scale(tile.at(x, y, e), power);
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

// What a block of k_ce_scan found in its share of the rows.
struct CeScan {
    double n;   // rows that count
    float top;  // the largest finite |dloss| (kCeNone)
};
constexpr int kCeScans = 256;

// What a row's factor c_i is made of.
struct CeRows {
    const float* dloss;
    const int64_t* targets;
    int64_t ignored, rows, classes;
    int reduction;
    float on;  // 1 - smoothing
    const CeScan* scans;  // or NULL: each block goes over the rows itself
    int n_scans;
    bool powers;  // each row of g is brought to the largest's binade by a power of its own
};

// Rows [first, end) in steps, as one thread's share.
__device__ __forceinline__ CeScan ce_scan_rows(const CeRows& a, int64_t first, int64_t end,
                                               int64_t step) {
    CeScan s{0., 0.f};
    for (int64_t i = first; i < end; i += step) {
        if (a.targets[i] == a.ignored) continue;
        s.n += 1.;
        if (a.reduction == kCeNone && finite_f(a.dloss[i])) s.top = fmaxf(s.top, fabsf(a.dloss[i]));
    }
    return s;
}

// c_i times the number that brings the largest gradient that is to be expected,
// (1 - smoothing) max |c| at a target of no probability, to 2^13.  float16 then
// holds small probabilities; and of a call whose rows count alike the gradients
// at the targets, the largest by far, lie at a power of two or just below, where
// rounding takes least of them.  8192 x 4096 x 131072 bfloat16, errors of dx and dW
// (norm of the difference over norm): 1.7e-3, which is the results' own rounding;
// with a power of two in front 1.8e-3 to 2.5e-3, by where c's mantissa lies, and where
// each row has a factor of its own 2.2e-3.  (Two bfloat16 for each of g, as in small
// calls, would take that off and two thirds more time: 10 n V d operations in place of 6.)
//
// Where every row has a factor of its own and g is held in float16 (one or two), a row
// whose factor is small beside the largest would lose what its classes of small
// probability add up to.  So its g has a power of two more, which its row of dx is
// brought back by; dW sums over rows, so that there x's rows have the opposite power.
// (Direct: g is float32, and gets the power on its way into dx's product alone.)
struct CeFactor {
    float one, inv;
    int ek, e0;  // |c| < 2^e0
    float mu;
    // By all threads of a block.  `plain`: the factors as they are, for a float32 g.
    __device__ __forceinline__ void init(const CeRows& a, bool plain, double* lds,
                                         float* top_of) {
        double n = 0.;
        float top = 0.f;
        // A sum's factors, and those of a float32 g, take nothing from the other rows.
        if (a.reduction == kCeMean || (a.reduction == kCeNone && !plain)) {
            if (a.scans == nullptr) {
                const CeScan s = ce_scan_rows(a, threadIdx.x, a.rows, blockDim.x);
                n = s.n;
                top = s.top;
            } else if ((int)threadIdx.x < a.n_scans) {
                n = a.scans[threadIdx.x].n;
                top = a.scans[threadIdx.x].top;
            }
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
        ek = e0 = 0;
        mu = inv = 1.f;
        if (!plain && top > 0.f && finite_f(top)) {
            // Where 1 - smoothing is small, what is expected is not the largest.
            mu = frexpf(top * fmaxf(a.on, 0.5f), &ek);
            inv = 1.f / mu;
            ek = 13 - ek;
            frexpf(top, &e0);
        }
    }
    // The power of two of row i beyond 2^ek.
    __device__ __forceinline__ int power(const CeRows& a, int64_t i) const {
        if (!a.powers || a.targets[i] == a.ignored) return 0;
        const float c = a.dloss[i];
        if (c == 0.f || !finite_f(c)) return 0;
        int e;
        frexpf(c, &e);
        return e0 - e;
    }
    // c_i 2^ek / mu.
    __device__ __forceinline__ float of(const CeRows& a, int64_t i, int power = 0) const {
        const int64_t t = a.targets[i];
        if (t == a.ignored) return 0.f;
        if (t < 0 || t >= a.classes) return NAN;
        return ldexpf(a.reduction == kCeNone ? a.dloss[i] : one, ek + power) * inv;
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
    const int* powers;       // of each row, or NULL
};

// The two products of the gradients: tiles of dx come first, then those of dW.
struct CeBoth {
    CeSide g, w, x;
    CeResult dx, dw;
    int64_t rows, cols, classes;
    int64_t dx_blocks, dw_blocks;  // of each split; 0 where not wanted
    int dw_group;                // tiles of dW that a block goes through
    int dx_tile, dw_tile;        // rows of a tile
    int dx_splits, dw_splits;
    const CeScalars* scalars;
};

// `tile`: rows of a tile, 16 or 64.
int ce_direct_loss(int32_t dtype, int tile, const CeSide& x, const CeSide& w, const CeLogits& l,
                   hipStream_t s);
int ce_direct_grad(int32_t dtype, int tile, const CeSide& x, const CeSide& w, const CeLogits& l,
                   const CeRows& rows, CeScalars* scalars, int* powers, hipStream_t s);
int ce_direct_products(int32_t dtype, const CeBoth& b, hipStream_t s);

}  // namespace spopt
