// cross_entropy.hip - softmax cross entropy of hidden states against every row
// of a table of classes, forward and backward, without keeping the logits.
//
// With z = x W^T (rows x classes):
//   forward   lse_i = log sum_j exp z_ij,  loss_i = lse_i - (1 - e) z_it - e mean_j z_ij
//   backward  g_ij = c_i (exp(z_ij - lse_i) - (1 - e) [j = t] - e / classes),
//             dx = g W,  dW = g^T x
// Matrix products bound both: 2 and 6 operations for each row, class and
// column.  The forward pass keeps each row's maximum and sum of exponentials in
// registers while tiles of z go by; a small kernel joins the parts.  The backward
// pass goes over the classes in pieces: z of a piece once more, g of it in 16
// bits into the workspace, and from there the piece's rows of dW and its share of
// dx.  Nothing of rows x classes outlives a piece.  (z held from the forward pass
// would spare a quarter of both passes' products, for 2 bytes a row and class.)
//
// Types.  16-bit operands go to the matrix cores as they are, sums are float32,
// and g is rounded to the operands' type (cross_entropy.hpp's CeFactor says with
// what in front; small calls hold it in float32).  A float32 operand a becomes two float16, hi = a 2^e rounded and
// lo = a 2^e - hi rounded, e one for the whole operand that brings its largest
// value to 2^14: 22 bits of each value (fewer of those below 2^-18 of the largest:
// off by 2^-39 of it at most).  A product is hi hi + hi lo + lo hi, three matrix
// instructions in place of one; errors are float32's (8192 x 128 x 50021: 3.8e-7 of
// dx, float32 products 3.6e-6).
//
// Measured on one MI355X (cards differ by 7%): 4096 x 2048 x 131072 bfloat16 forward
// 1.79 to 1.94 ms (1.13 to 1.23 PFLOP/s), 8192 x 4096 x 131072 backward 20.7 to 21.9
// ms (1.20 to 1.28 PFLOP/s; a library product of these sizes 1.31 to 1.50), 8192 x 128
// x 50021 float32 0.36 to 0.37 and 1.46 to 1.54 ms, bfloat16 0.18 to 0.19 and 0.70.
#include "cross_entropy.hpp"

namespace spopt {

// An operand of a product: rows of 16-bit values.  Where the inner axis runs
// along the rows, `last` is the last row; where it runs from row to row, the
// last row and `cols` the columns that each row holds (a multiple of 8).  Split
// rows hold 32 hi values, then their 32 lo, and so on.
struct CeOperand {
    const void* base;
    int64_t ld, last, cols;
};

struct CeProduct {
    CeOperand p, q;
    int64_t m, n;     // the result's rows and columns
    int64_t steps;    // of the inner axis, 64 values each (32 split)
    int splits;       // parts of the inner axis, or (logits) of the tiles of classes
    int64_t tiles_m, tiles_n;
};

// Products of tiles of 64 and 128: operands go through LDS 64 values of the inner axis at a time, loaded straight into it
// while earlier stages are multiplied.  Operands whose inner axis lies along
// their rows are laid out with chunk c of 8 values at c ^ (row & 7); the others
// are turned as they are read.  Split operands bring 32 values of the inner
// axis a stage, hi in its first half and lo in its second.
template <class T, bool SPLIT, bool TP, bool TQ, class TL>
struct CeTile {
    static constexpr int BM = TL::BM, BN = TL::BN, WM = BM / TL::WGM, WN = BN / TL::WGN;
    static constexpr int FM = WM / 16, FN = WN / 16, kWaves = TL::WGM * TL::WGN;
    static constexpr int kRow = TQ ? 4 : 8;  // adjacent columns of a lane
    static constexpr int kLoadsP = BM / 8 / kWaves, kLoadsQ = BN / 8 / kWaves;
    static constexpr int kInner = SPLIT ? 32 : 64;
    typedef T vec8 __attribute__((ext_vector_type(8)));
    typedef T vec4 __attribute__((ext_vector_type(4)));
    static_assert(BM % (8 * kWaves) == 0 && BN % (8 * kWaves) == 0, "rows share out evenly");
    static_assert(TQ || FN % 2 == 0, "eight adjacent columns take two parts");

    // A side's loads: a lane's places in the operand.
    template <bool TURN, int B, int LOADS>
    struct Feed {
        const T* src[LOADS];
        int row[TURN ? LOADS : 1];
        int64_t ld, last;
        __device__ __forceinline__ void init(const CeOperand& o, int64_t first, int lane, int wv,
                                             bool pair) {
            const T* base = (const T*)o.base;
            ld = o.ld;
            last = o.last;
#pragma unroll
            for (int l = 0; l < LOADS; ++l) {
                if constexpr (TURN) {
                    const int at = (l * kWaves + wv) * 64 + lane;
                    const int v = at / (B / 8), slot = at % (B / 8);
                    int64_t c = first + (((slot >> 1) ^ turn_q<B>(v)) * 2 + (slot & 1)) * 8;
                    if (c > o.cols - 8) c = o.cols - 8;
                    if (SPLIT) c = (c / 32) * 64 + c % 32 + (v >> 5) * 32;
                    row[l] = SPLIT ? v & 31 : v;
                    src[l] = base + c;
                } else {
                    const int at = (l * kWaves + wv) * 8 + (lane >> 3);
                    int64_t r = first + at;
                    if (pair) {
                        const int in = at & 31;
                        r = first + at - in + ((in & 12) >> 2) * 8 + (in >> 4) * 4 + (in & 3);
                    }
                    if (r > last) r = last;
                    src[l] = base + r * ld + ((lane & 7) ^ (lane >> 3)) * 8;
                }
            }
        }
        __device__ __forceinline__ void bring(int64_t k, T* to, int wv) const {
#pragma unroll
            for (int l = 0; l < LOADS; ++l) {
                const T* from;
                if constexpr (TURN) {
                    int64_t r = k * kInner + row[l];
                    if (r > last) r = last;
                    from = src[l] + r * ld;
                } else {
                    from = src[l] + k * 64;
                }
                load_lds16(from, to + (l * kWaves + wv) * 512);
            }
        }
    };

    int lane, wv, wi, wj;
    float4v acc[FM][FN];

    // Operand `f` of half kk from a side's stage in LDS.
    template <bool TURN, int B>
    __device__ __forceinline__ vec8 operand(const T* l, int first, int kk) const {
        if constexpr (TURN) {
            const int row = (lane >> 4) * 8 + ((lane & 15) >> 2);
            const T* a = l + (kk * 32 + row) * B + ((first / 16) ^ turn_q<B>(row)) * 16 +
                         (lane & 3) * 4;
            const vec4 lo = __builtin_bit_cast(vec4, read_turned((const _Float16*)a));
            const vec4 hi = __builtin_bit_cast(vec4, read_turned((const _Float16*)(a + 4 * B)));
            return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
        } else {
            return *(const vec8*)(l + (first + (lane & 15)) * kTile +
                                  ((kk * 4 + (lane >> 4)) ^ (lane & 7)) * 8);
        }
    }

    __device__ __forceinline__ void multiply(const vec8 (&fa)[FM], const vec8 (&fb)[FN]) {
#pragma unroll
        for (int x = 0; x < FM; ++x)
#pragma unroll
            for (int y = 0; y < FN; ++y) acc[x][y] = matrix_16x16x32(fb[y], fa[x], acc[x][y]);
    }

    __device__ __forceinline__ void init() {
        lane = lane_id();
        wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
        wi = (wv / TL::WGN) * WM;
        wj = (wv % TL::WGN) * WN;
    }

    __device__ __forceinline__ void clear() {
#pragma unroll
        for (int x = 0; x < FM; ++x)
#pragma unroll
            for (int y = 0; y < FN; ++y) acc[x][y] = float4v{0.f, 0.f, 0.f, 0.f};
    }

    // Tiles [t0, t1) of a row of tiles, steps [k0, k1) of the inner axis for each (one
    // at least): `done(t)` where a tile's sums are there.  The loads run on from
    // tile to tile: the next one's are on their way while this one's sums are dealt
    // with.
    template <class F>
    __device__ __forceinline__ void run(T* lds, const CeProduct& c, int64_t i0, int64_t t0,
                                        int64_t t1, int64_t k0, int64_t k1, F done) {
        Feed<TP, BM, kLoadsP> fp;
        Feed<TQ, BN, kLoadsQ> fq;
        fp.init(c.p, i0, lane, wv, false);
        fq.init(c.q, t0 * BN, lane, wv, !TQ);
        constexpr int kLoads = kLoadsP + kLoadsQ;
        int64_t bt = t0, bk = k0;
        // Past the end the last step is brought again, so that every wait counts
        // the same loads; nothing reads it.
        auto stage = [&](int buf) {
            T* const to = lds + buf * TL::kStage;
            fp.bring(bk, to, wv);
            fq.bring(bk, to + BM * kTile, wv);
            if (bk + 1 < k1) {
                ++bk;
            } else if (bt + 1 < t1) {
                ++bt;
                bk = k0;
                fq.init(c.q, bt * BN, lane, wv, !TQ);
            }
        };
        vec8 fa0[FM], fb0[FN], fa1[FM], fb1[FN];
        auto operands = [&](int buf, int kk, vec8 (&fa)[FM], vec8 (&fb)[FN]) {
            const T* lp = lds + buf * TL::kStage;
            const T* lq = lp + BM * kTile;
#pragma unroll
            for (int y = 0; y < FN; ++y) fb[y] = operand<TQ, BN>(lq, wj + y * 16, kk);
#pragma unroll
            for (int x = 0; x < FM; ++x) fa[x] = operand<TP, BM>(lp, wi + x * 16, kk);
        };
        int buf = 0;
#pragma unroll
        for (int k = 0; k < TL::STAGES - 1; ++k) stage(k);
        for (int64_t t = t0; t < t1; ++t) {
            clear();
            for (int64_t k = k0; k < k1; ++k) {
                // This stage's loads have landed in every wave, and every wave has
                // read the stage before, whose place the next loads take.
                wait_stage<(TL::STAGES - 2) * kLoads>();
                stage(buf == 0 ? TL::STAGES - 1 : buf - 1);
                operands(buf, 0, fa0, fb0);
                multiply(fa0, fb0);
                operands(buf, 1, fa1, fb1);
                if constexpr (SPLIT) {
                    multiply(fa0, fb1);
                    multiply(fa1, fb0);
                } else {
                    multiply(fa1, fb1);
                }
                buf = buf + 1 == TL::STAGES ? 0 : buf + 1;
            }
            done(t);
        }
        wait_loads<0>();
    }

    static constexpr int kRowLanes = 16;
    __device__ __forceinline__ float at(int x, int y, int e) const { return acc[x][y][e]; }
    __device__ __forceinline__ float4v four(int x, int y) const { return acc[x][y]; }
    // Row x and column (y, e) of this lane, within the tile.
    __device__ __forceinline__ int row_of(int x) const { return wi + x * 16 + (lane & 15); }
    __device__ __forceinline__ int col_of(int y) const {
        return wj + (lane >> 4) * kRow + (kRow == 8 ? (y & ~1) * 16 + (y & 1) * 4 : y * 16);
    }
};

// A tile of 256 x 256 by four waves, 128 x 128 each, which read two thirds of what
// eight would from LDS.  A wave is alone on its SIMD, so that what it waits for
// is laid between its products (of 32 x 32, whose issue leaves it room): while
// one half of a stage is multiplied, the other's operands are read, and the loads
// of the stage after next go out, P's in the first half and Q's in the second.  LDS
// (all 160 KB) has three places for P and two for Q, so that P's go to one that is
// free already, and Q's to what this step's first half has emptied.  One barrier a
// stage, of 64 matrix instructions a wave.  8192 x 4096 x 32768 bfloat16, random
// values: matrix instructions are busy 66 to 70% of the cycles at 1.7 to 1.8 GHz, of
// the card's 2.4: what bounds it is the power they take (of zeros the same kernel
// takes 1.34 in place of 1.77 ms).  Eight waves of 128 x 64 in turns of the same
// stages, or two stages of each side: 53 to 58% at 2.0 GHz, 4 to 8% slower.
template <class T, bool TP, bool TQ>
struct CeWide {
    static constexpr int BM = 256, BN = 256, WGN = 2, FM = 4, FN = 16, kRowLanes = 32;
    static constexpr int kRow = TQ ? 4 : 8;
    static constexpr int kSide = 256 * kTile;  // values of a side's stage
    typedef T vec8 __attribute__((ext_vector_type(8)));
    typedef T vec4 __attribute__((ext_vector_type(4)));

    // Where row v of a turned side has its 16 columns from 16 u on: at u ^ turn(v).
    // Two such parts of four rows then lie in different eighths of 256 bytes.
    static __device__ __forceinline__ int turn(int v) { return (v & 3) << 1; }

    // Chunk c of row r of the other sides lies at c ^ turn_row(r): LDS gives the same
    // chunk of rows r .. r + 7 and r + 16 .. r + 23 at once.
    static __device__ __forceinline__ int turn_row(int r) { return (r & 7) ^ (r >> 4 & 1); }

    // A side's eight loads a stage: each lane's distance from a base that is the
    // same for the wave.
    template <bool TURN>
    struct Feed {
        const char* base;
        int64_t ld, last;
        uint32_t off[8];
        __device__ __forceinline__ void init(const CeOperand& o, int64_t first, int lane, int wv,
                                             bool pair) {
            ld = o.ld * 2;
            last = o.last;
            base = (const char*)o.base + (TURN ? 0 : first * ld);
#pragma unroll
            for (int l = 0; l < 8; ++l) {
                if constexpr (TURN) {
                    const int v = (l * 4 + wv) * 2 + (lane >> 5), slot = lane & 31;
                    int64_t c = first + (((slot >> 1) ^ turn(v)) * 2 + (slot & 1)) * 8;
                    if (c > o.cols - 8) c = o.cols - 8;
                    off[l] = (uint32_t)(v * ld + c * 2);
                } else {
                    const int at = (l * 4 + wv) * 8 + (lane >> 3), in = at & 31;
                    int64_t r = pair ? at - in + (in >> 4) * 16 + (in >> 2 & 1) * 8 +
                                           (in >> 3 & 1) * 4 + (in & 3)
                                     : at;
                    if (r > last - first) r = last - first;
                    off[l] = (uint32_t)(r * ld + ((lane & 7) ^ turn_row(at)) * 16);
                }
            }
        }
        // Load l of step k.
        __device__ __forceinline__ void bring(int l, int64_t k, T* to, int lane, int wv) const {
            const char* from = base + (TURN ? k * 64 * ld : k * 128);
            uint32_t o = off[l];
            if constexpr (TURN) {
                // Rows past the last bring that one: g's zeros meet it.
                const int v = (l * 4 + wv) * 2 + (lane >> 5);
                const int over = v + (int)(k * 64 - last);
                o -= (uint32_t)(over > 0 ? over : 0) * (uint32_t)ld;
            }
            load_lds16_from(from, o, to + (l * 4 + wv) * 512);
        }
    };

    int lane, wv, wi, wj;
    float16v acc[4][4];

    __device__ __forceinline__ void init() {
        lane = lane_id();
        wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
        wi = (wv >> 1) * 128;
        wj = (wv & 1) * 128;
    }
    __device__ __forceinline__ void clear() {
#pragma unroll
        for (int x = 0; x < 4; ++x)
#pragma unroll
            for (int y = 0; y < 4; ++y)
#pragma unroll
                for (int e = 0; e < 16; ++e) acc[x][y][e] = 0.f;
    }

    // The operand of 32 rows (or columns) from `first` on, 16 values of the inner
    // axis: the kk-th of a stage's four.
    template <bool TURN>
    __device__ __forceinline__ vec8 operand(const T* l, int first, int kk) const {
        if constexpr (TURN) {
            const int row = (lane >> 5) * 8 + ((lane & 15) >> 2);
            const T* a = l + (kk * 16 + row) * 256 +
                         ((first / 16 + (lane >> 4 & 1)) ^ turn(row)) * 16 + (lane & 3) * 4;
            const vec4 lo = __builtin_bit_cast(vec4, read_turned((const _Float16*)a));
            const vec4 hi = __builtin_bit_cast(vec4, read_turned((const _Float16*)(a + 4 * 256)));
            return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
        } else {
            return *(const vec8*)(l + (first + (lane & 31)) * kTile +
                                  ((kk * 2 + (lane >> 5)) ^ turn_row(lane & 31)) * 8);
        }
    }

    // Tile t0 alone: a loop over tiles around it would take registers that it lacks.
    template <class F>
    __device__ __forceinline__ void run(T* lds, const CeProduct& c, int64_t i0, int64_t t0, int64_t,
                                        int64_t k0, int64_t k1, F done) {
        const int64_t j0 = t0 * 256;
        clear();
        Feed<TP> fp;
        Feed<TQ> fq;
        fp.init(c.p, i0, lane, wv, false);
        fq.init(c.q, j0, lane, wv, !TQ);
        // Past the end the last step is brought again; nothing reads it.
        auto bring_p = [&](int l, int slot, int64_t k) {
            if (k >= k1) k = k1 - 1;
            fp.bring(l, k, lds + slot * kSide, lane, wv);
        };
        auto bring_q = [&](int l, int slot, int64_t k) {
            if (k >= k1) k = k1 - 1;
            fq.bring(l, k, lds + (3 + slot) * kSide, lane, wv);
        };
        vec8 a[4][4], b[4][4];
        // Operand g of half h: in the order in which they are met.
        auto read = [&](int g, int ps, int qs, int h) {
            const int kk = 2 * h + g / 8, i = g % 8;
            if (i < 4)
                b[kk][i] = operand<TQ>(lds + (3 + qs) * kSide, wj + i * 32, kk);
            else
                a[kk][i - 4] = operand<TP>(lds + ps * kSide, wi + (i - 4) * 32, kk);
        };
        // 32 products of half h, and between them the other half's operands (in
        // slots ps and qs) and eight loads of step k.
        auto half = [&](auto h_, int ps, int qs, int slot, int64_t k) {
            constexpr int h = decltype(h_)::value;
#pragma unroll
            for (int g = 0; g < 16; ++g) {
                if (h == 0 && g % 2 == 0) bring_p(g / 2, slot, k);
                if (h == 1 && g < 8) bring_q(g, slot, k);
                if (g < 4) {
                    read(2 * g, ps, qs, 1 - h);
                    read(2 * g + 1, ps, qs, 1 - h);
                } else if (g < 12) {
                    read(g + 4, ps, qs, 1 - h);
                }
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    const int kk = 2 * h + g / 8, x = g % 8 / 2, y = g % 2 * 2 + u;
                    acc[x][y] = matrix_32x32x16(b[kk][y], a[kk][x], acc[x][y]);
                }
                __builtin_amdgcn_sched_barrier(0);
            }
        };
        typedef std::integral_constant<int, 0> First;
        typedef std::integral_constant<int, 1> Second;
#pragma unroll
        for (int k = 0; k < 2; ++k)
#pragma unroll
            for (int l = 0; l < 8; ++l) {
                bring_p(l, k, k0 + k);
                bring_q(l, k, k0 + k);
            }
        wait_stage<16>();
#pragma unroll
        for (int g = 0; g < 16; ++g) read(g, 0, 0, 0);
        int ps = 0, qs = 0;
        for (int64_t k = k0; k < k1; ++k) {
            const int p1 = ps == 2 ? 0 : ps + 1, p2 = ps == 0 ? 2 : ps - 1;
            // P's rows of the step after next go to where the step before had its own.
            half(First{}, ps, qs, p2, k + 2);
            // All but those have landed in every wave, and every wave has read this step.
            wait_stage<8>();
            half(Second{}, p1, qs ^ 1, qs, k + 2);
            ps = p1;
            qs ^= 1;
        }
        wait_stage<0>();
        done(t0);
    }

    __device__ __forceinline__ float at(int x, int y, int e) const {
        return acc[x][y / 4][y % 4 * 4 + e];
    }
    __device__ __forceinline__ float4v four(int x, int y) const {
        return float4v{at(x, y, 0), at(x, y, 1), at(x, y, 2), at(x, y, 3)};
    }
    __device__ __forceinline__ int row_of(int x) const { return wi + x * 32 + (lane & 31); }
    __device__ __forceinline__ int col_of(int y) const {
        const int g = y % 4, h = lane >> 5;
        return wj + y / 4 * 32 + (kRow == 8 ? (g >> 1) * 16 + h * 8 + (g & 1) * 4 : g * 8 + h * 4);
    }
};

// The tile's struct: four waves of 128 x 128 where it is 256 wide.
template <class T, bool SPLIT, bool TP, bool TQ, class TL>
using CeTileOf = std::conditional_t<TL::BM == 256, CeWide<T, TP, TQ>, CeTile<T, SPLIT, TP, TQ, TL>>;

// A block takes one of `parts` parts of the piece's tiles of classes, for one tile
// of rows: their maxima and sums stay in registers from tile to tile (8192 x 128 x
// 50021 float32: 360 us; sums in float32 345, and then 446 with a block and a place in
// the workspace for each tile).  Blocks of the same part follow one another, so that an XCD's L2 sees W's
// rows once.
template <class T, bool SPLIT, int MODE, class TL>
__global__ __launch_bounds__(TL::kThreads)
    __attribute__((amdgpu_waves_per_eu(TL::BM == 256 ? 1 : 2))) void k_ce_logits(CeProduct c,
                                                                                 CeLogits w) {
    extern __shared__ __align__(16) char lds_raw[];
    typedef CeTileOf<T, SPLIT, false, false, TL> Tile;
    constexpr int BM = TL::BM, BN = TL::BN;
    const int64_t b = xcd_order(blockIdx.x, gridDim.x);
    int64_t part = b / c.tiles_m, ti = b % c.tiles_m;
    if (BM == 256) ce_place(b, c.tiles_m, c.tiles_n, &ti, &part);
    const int64_t i0 = ti * BM;
    const int64_t t0 = part * c.tiles_n / c.splits, t1 = (part + 1) * c.tiles_n / c.splits;
    Tile tile;
    tile.init();
    const int e = SPLIT ? -(w.scalars->ex + w.scalars->ew) : 0;
    if constexpr (MODE == kCeLoss) {
        CeRowSums<Tile> sums;
        sums.init(tile, w, i0, c.m, c.n, e);
        tile.run((T*)lds_raw, c, i0, t0, t1, 0, c.steps, [&](int64_t t) {
            sums.template add<BN, TL::WGN>(tile, w, i0, t * BN, c.n);
        });
        sums.template store<BM, TL::WGN>(tile, w, (float*)lds_raw, i0, c.m, w.first_part + part);
    } else {
        CeRowGrads<Tile> grads;
        grads.init(tile, w, i0, c.m, c.n, e, [&](int64_t i) { return w.coef[i]; });
        tile.run((T*)lds_raw, c, i0, t0, t1, 0, c.steps, [&](int64_t t) {
            grads.template store<T, SPLIT, BN, TL::WGN>(tile, w, i0, t * BN, c.n);
        });
    }
}

template <class T, bool SPLIT, int MODE, class TL>
__global__ __launch_bounds__(TL::kThreads)
    __attribute__((amdgpu_waves_per_eu(TL::BM == 256 ? 1 : 2))) void k_ce_product(
        CeProduct c, CeResult w, const CeScalars* sc) {
    extern __shared__ __align__(16) char lds_raw[];
    typedef CeTileOf<T, SPLIT, MODE == kCeDw, true, TL> Tile;
    typedef std::conditional_t<SPLIT, float, T> O;
    const int64_t tiles = c.tiles_m * c.tiles_n;
    const int64_t b = xcd_order(blockIdx.x, gridDim.x);
    const int64_t split = b / tiles;
    int64_t ti, tj;
    ce_place(b % tiles, c.tiles_m, c.tiles_n, &ti, &tj);
    const int64_t i0 = ti * TL::BM;
    const int64_t k0 = split * c.steps / c.splits, k1 = (split + 1) * c.steps / c.splits;
    Tile tile;
    tile.init();
    // A last, shorter piece of the classes may leave a split nothing to add.
    if (k0 == k1) return;
    tile.run((T*)lds_raw, c, i0, tj, tj + 1, k0, k1, [](int64_t) {});
    const int e = sc->ek + (MODE == kCeDw ? sc->ed : SPLIT ? sc->ew : 0);
    const float mu = sc->mu;
    ce_store_tile<O>(tile, i0, tj * TL::BN, c.m, c.n, w,
                     w.parts == nullptr ? nullptr : w.parts + split * c.m * w.ld,
                     [&](float v, int power) { return ce_unscale(v, mu, e + power); });
}

// out = the splits' sums (zeros where there are none), scaled and rounded.  HBM
// bounds it.
template <class O>
__global__ __launch_bounds__(256) void k_ce_gather(const float* parts, int splits, int64_t rows,
                                                   int64_t ld, int64_t cols, const CeScalars* sc,
                                                   int use_w, int use_d, const int* powers, O* out,
                                                   int64_t out_ld) {
    const int64_t quads = ld / 4, all = rows * quads;
    const float mu = splits == 0 ? 0.f : sc->mu;
    const int scale = splits == 0 ? 0 : sc->ek + (use_w ? sc->ew : 0) + (use_d ? sc->ed : 0);
    for (int64_t q = (int64_t)blockIdx.x * 256 + threadIdx.x; q < all;
         q += (int64_t)gridDim.x * 256) {
        const int64_t i = q / quads, j = q % quads * 4;
        if (j >= cols) continue;
        double s[4] = {};
        const float* from = parts + i * ld + j;
        // Eight loads on their way at once.
        for (int k0 = 0; k0 < splits; k0 += 8) {
            float4v p[8];
#pragma unroll
            for (int k = 0; k < 8; ++k)
                p[k] = k0 + k < splits ? *(const float4v*)(from + (k0 + k) * rows * ld)
                                       : float4v{0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int k = 0; k < 8; ++k)
#pragma unroll
                for (int e = 0; e < 4; ++e) s[e] += (double)p[k][e];
        }
        float v[4];
        const int by = scale + (powers ? powers[i] : 0);
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = ce_unscale((float)s[e], mu, by);
        O* const to = out + i * out_ld + j;
        if (j + 4 <= cols) {
            store_v<O, 4>(to, v);
        } else {
            for (int e = 0; j + e < cols; ++e) to[e] = (O)v[e];
        }
    }
}

// ------------------------------------------------------------- operands ---

constexpr int kAmaxParts = 512;

// The largest finite magnitude that each block meets, as its bits in float32.  Row 0 of
// the grid takes x, but for the rows that are ignored, row 1 W.
template <class S>
__global__ __launch_bounds__(256) void k_ce_amax(const S* x, int64_t x_ld, int64_t rows,
                                                 const int64_t* targets, int64_t ignored,
                                                 const S* w, int64_t w_ld, int64_t classes,
                                                 int64_t cols, uint32_t* parts) {
    __shared__ uint32_t lds[4];
    const bool of_w = blockIdx.y == 1;
    const S* a = of_w ? w : x;
    const int64_t ld = of_w ? w_ld : x_ld, n = of_w ? classes : rows;
    uint32_t top = 0;
    auto take = [&](float v) {
        const uint32_t u = __builtin_bit_cast(uint32_t, v) & 0x7fffffffu;
        if (u < 0x7f800000u && u > top) top = u;
    };
    const int64_t chunks = (cols + 3) / 4, all = n * chunks;
    for (int64_t q = (int64_t)blockIdx.x * 256 + threadIdx.x; q < all;
         q += (int64_t)gridDim.x * 256) {
        const int64_t r = q / chunks, j = q % chunks * 4;
        if (!of_w && targets[r] == ignored) continue;
        const S* p = a + r * ld + j;
        if (j + 4 <= cols) {
            float v[4];
            load_v<S, 4>(p, v);
#pragma unroll
            for (int e = 0; e < 4; ++e) take(v[e]);
        } else {
            for (int e = 0; j + e < cols; ++e) take((float)p[e]);
        }
    }
#pragma unroll
    for (int off = kWave / 2; off; off >>= 1) {
        const uint32_t o = (uint32_t)__shfl_xor((int)top, off, kWave);
        top = o > top ? o : top;
    }
    if (lane_id() == 0) lds[threadIdx.x >> 6] = top;
    __syncthreads();
    if (threadIdx.x == 0) {
        for (int k = 1; k < 4; ++k) top = lds[k] > top ? lds[k] : top;
        parts[blockIdx.y * kAmaxParts + blockIdx.x] = top;
    }
}

// A copy of an operand as the products take it: rows_p rows of cols_p columns
// (a multiple of 64), zeros beyond the matrix and in rows that do not count.
// float32: scaled by 2^e and split; `amax` holds the blocks' shares of the
// largest value, and block 0 leaves e in *exponent.  With `powers`, a second copy as
// dW's operand, row i times 2^(e - powers[i]): what float16 takes of it is off by
// 2^-39 of x's largest value at most, whatever the rows' factors.
template <class S, class T>
__global__ __launch_bounds__(256) void k_ce_pack(const S* a, int64_t ld, int64_t rows,
                                                 int64_t cols, int64_t rows_p, int64_t cols_p,
                                                 const int64_t* targets, int64_t ignored,
                                                 const uint32_t* amax, int n_amax, int* exponent,
                                                 T* out, const int* powers, int* exponent2,
                                                 T* out2) {
    constexpr bool kSplit = std::is_same_v<S, float>;
    int ex = 0;
    if (kSplit || powers != nullptr) {
        __shared__ uint32_t lds[4];
        uint32_t top = 0;
        for (int k = threadIdx.x; k < n_amax; k += 256) top = amax[k] > top ? amax[k] : top;
#pragma unroll
        for (int off = kWave / 2; off; off >>= 1) {
            const uint32_t o = (uint32_t)__shfl_xor((int)top, off, kWave);
            top = o > top ? o : top;
        }
        if (lane_id() == 0) lds[threadIdx.x >> 6] = top;
        __syncthreads();
        for (int k = 0; k < 4; ++k) top = lds[k] > top ? lds[k] : top;
        if (top != 0) {
            frexpf(__builtin_bit_cast(float, top), &ex);  // |a| < 2^ex
            ex = 15 - ex;
        }
        if (blockIdx.x == 0 && threadIdx.x == 0) {
            if (kSplit) *exponent = ex;
            if (exponent2 != nullptr) *exponent2 = ex;
        }
    }
    const int64_t chunks = cols_p / 8, all = rows_p * chunks;
    for (int64_t q = (int64_t)blockIdx.x * 256 + threadIdx.x; q < all;
         q += (int64_t)gridDim.x * 256) {
        const int64_t r = q / chunks, j = q % chunks * 8;
        float v[8] = {};
        if (r < rows && j < cols && (targets == nullptr || targets[r] != ignored)) {
            const S* p = a + r * ld + j;
            if (j + 8 <= cols) {
                load_v<S, 8>(p, v);
            } else {
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    if (j + e < cols) v[e] = (float)p[e];
            }
        }
        if (kSplit && powers == nullptr) {
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] = ldexpf(v[e], ex);
        }
        auto put = [&](T* to, const float (&u)[8]) {
            if constexpr (kSplit) {
                float lo[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) lo[e] = u[e] - (float)(T)u[e];
                to += r * 2 * cols_p + j / 32 * 64 + j % 32;
                store_v<T, 8>(to, u);
                store_v<T, 8>(to + 32, lo);
            } else {
                store_v<T, 8>(to + r * cols_p + j, u);
            }
        };
        if (powers != nullptr) {
            const int by = ex - powers[r];
            float u[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                u[e] = ldexpf(v[e], by);
                if (kSplit) v[e] = ldexpf(v[e], ex);
            }
            put(out2, u);
        }
        put(out, v);
    }
}

// ------------------------------------------------------ joins and sums ---

// lse and loss of each row from its tiles' pairs: `per` rows (a power of two, up
// to 64, or 1024) at a time by a block's 1024 threads, the tiles shared out to
// 1024 / per of them.  A block alone sums the rows' losses itself.
__global__ __launch_bounds__(1024) void k_ce_join(const float2* parts, const float* sums,
                                                  const float* at_target, const int64_t* targets,
                                                  int64_t ignored, int64_t rows, int64_t tiles,
                                                  int64_t classes, float smoothing, int per,
                                                  int reduction, float* row_loss, float* loss,
                                                  float* lse) {
    __shared__ float tops[16][64];
    __shared__ double both[2][16][64];
    const int t = threadIdx.x, slices = 1024 / per, lane = lane_id(), wv = t >> 6;
    double total = 0., count = 0.;
    for (int64_t first = (int64_t)blockIdx.x * per; first < rows; first += (int64_t)gridDim.x * per) {
        const int64_t i = first + t % per;
        float top = -INFINITY;
        double s = 0., z = 0.;
        auto add = [&](float m, double v) {
            const float next = fmaxf(top, m);
            if (top != next) s *= (double)exp_less(top, next);
            s += m == next ? v : v * (double)exp_less(m, next);
            top = next;
        };
        if (i < rows) {
            int64_t k = t / per;
            for (; k + 3 * slices < tiles; k += 4 * slices) {
                float2 p[4];
#pragma unroll
                for (int u = 0; u < 4; ++u) p[u] = parts[(k + u * slices) * rows + i];
#pragma unroll
                for (int u = 0; u < 4; ++u) add(p[u].x, p[u].y);
            }
            for (; k < tiles; k += slices) {
                const float2 p = parts[k * rows + i];
                add(p.x, p.y);
            }
            if (sums)
                for (k = t / per; k < tiles; k += slices) z += (double)sums[k * rows + i];
        }
        for (int off = per; off < kWave; off <<= 1) {
            const float m = __shfl_xor(top, off, kWave);
            const double v = __shfl_xor(s, off, kWave);
            add(m, v);
            z += __shfl_xor(z, off, kWave);
        }
        if (per != 1024) __syncthreads();
        if (lane < per && per != 1024) {
            tops[wv][lane] = top;
            both[0][wv][lane] = s;
            both[1][wv][lane] = z;
        }
        if (per != 1024) __syncthreads();
        if (t >= per || i >= rows) continue;
        for (int k = 1; k < 16 && per != 1024; ++k) {
            add(tops[k][t], both[0][k][t]);
            z += both[1][k][t];
        }
        const int64_t goal = targets[i];
        const bool valid = goal != ignored;
        const double l = (double)top + log(s);
        double own = 0.;
        if (valid) {
            own = goal < 0 || goal >= classes
                      ? (double)NAN
                      : l - (1. - (double)smoothing) * (double)at_target[i] -
                            (double)smoothing * (z / (double)classes);
            total += own;
            count += 1.;
        }
        lse[i] = valid ? (float)l : 0.f;
        if (reduction == kCeNone)
            loss[i] = (float)own;
        else if (gridDim.x != 1)
            row_loss[i] = (float)own;
    }
    if (reduction == kCeNone || gridDim.x != 1) return;
    total = ce_block_sum(total, both[0][0]);
    count = ce_block_sum(count, both[1][0]);
    if (t == 0) *loss = (float)(reduction == kCeMean ? total / fmax(count, 1.) : total);
}

// The rows' losses as one, by one block.
__global__ __launch_bounds__(1024) void k_ce_reduce(const float* row_loss, const int64_t* targets,
                                                    int64_t ignored, int64_t rows, int reduction,
                                                    float* loss) {
    __shared__ double lds[16];
    double s = 0., n = 0.;
    for (int64_t i = threadIdx.x; i < rows; i += 1024) {
        s += (double)row_loss[i];
        n += targets[i] != ignored ? 1. : 0.;
    }
    s = ce_block_sum(s, lds);
    n = ce_block_sum(n, lds);
    if (threadIdx.x == 0) *loss = (float)(reduction == kCeMean ? s / fmax(n, 1.) : s);
}

// What CeFactor takes from all rows, each block's share.
__global__ __launch_bounds__(256) void k_ce_scan(CeRows rows, CeScan* scans) {
    __shared__ double lds[4];
    __shared__ float tops[4];
    CeScan s = ce_scan_rows(rows, (int64_t)blockIdx.x * 256 + threadIdx.x, rows.rows,
                            (int64_t)gridDim.x * 256);
    s.n = ce_block_sum(s.n, lds);
#pragma unroll
    for (int off = kWave / 2; off; off >>= 1) s.top = fmaxf(s.top, __shfl_xor(s.top, off, kWave));
    if (lane_id() == 0) tops[threadIdx.x >> 6] = s.top;
    __syncthreads();
    if (threadIdx.x != 0) return;
    for (int k = 0; k < 4; ++k) s.top = fmaxf(s.top, tops[k]);
    scans[blockIdx.x] = s;
}

// Each row's factor and power, 0 beyond the last.  One block, or more where the rows have been
// scanned.
__global__ __launch_bounds__(1024) void k_ce_coef(CeRows rows, int64_t rows_p, float* coef,
                                                  int* powers, CeScalars* scalars) {
    __shared__ double lds[16];
    __shared__ float top_of[16];
    CeFactor f;
    f.init(rows, false, lds, top_of);
    if (blockIdx.x == 0 && threadIdx.x == 0) {
        scalars->ek = f.ek;
        scalars->mu = f.mu;
        scalars->ed = 0;
    }
    for (int64_t i = (int64_t)blockIdx.x * 1024 + threadIdx.x; i < rows_p; i += gridDim.x * 1024) {
        const int power = i < rows.rows ? f.power(rows, i) : 0;
        coef[i] = i < rows.rows ? f.of(rows, i, power) : 0.f;
        if (rows.powers) powers[i] = power;
    }
}

// Sets kStatusRange for a target that is neither ignored nor a class, and
// kStatusNonFinite where a row that counts holds a NaN or an infinity.
template <class T>
__global__ __launch_bounds__(256) void k_ce_check(const T* x, int64_t ld, int64_t rows,
                                                  int64_t cols, const int64_t* targets,
                                                  int64_t ignored, int64_t classes,
                                                  uint32_t* status) {
    for (int64_t r = blockIdx.x; r < rows; r += gridDim.x) {
        const int64_t t = targets[r];
        if (t == ignored) continue;
        uint32_t bad = t < 0 || t >= classes ? kStatusRange : 0u;
        for (int64_t c = threadIdx.x; c < cols; c += 256)
            if (!finite_f((float)x[r * ld + c])) bad |= kStatusNonFinite;
        if (bad) atomicOr(status, bad);
    }
}

// ------------------------------------------------------------------ host ---

typedef Tiling<64, 64, 2, 2, 2> CeS;
typedef Tiling<128, 128, 2, 4, 2> CeM;
typedef Tiling<256, 256, 2, 2, 2> CeL;

// Into how many parts the tiles of classes are shared out for each of tiles_m tiles
// of rows: as many blocks as the card holds at once (two of 128 a CU, four of 64),
// and parts alike; each by itself of the largest.
static int ce_parts(int64_t tiles_m, int64_t tiles_n, int tile) {
    if (tile == 256) return (int)tiles_n;
    const int64_t room = tile == 128 ? 512 : 1024, fewest = ceil_div(tiles_m, room);
    int64_t best = 1, least = INT64_MAX;
    // By how many times the blocks fill the card: the tiles that a place goes
    // through one after another.
    for (int64_t rounds = fewest; rounds < fewest + 8; ++rounds) {
        int64_t p = rounds * room / tiles_m;
        if (p > tiles_n) p = tiles_n;
        const int64_t cost = rounds * ceil_div(tiles_n, p);
        if (cost < least) {
            least = cost;
            best = p;
        }
    }
    return (int)best;
}

// How a product is tiled, and into how many parts its inner axis is cut.
struct CePlan {
    int tile;    // its rows: 64, 128 or 256; 16 or 64 of the direct kernels
    int splits;
    double us;   // what it is expected to take
};

// An inner step takes a tile of 64, 128 and 256 about 0.22, 0.45 and 1.6 us of its
// CU, and what comes before and after two steps more, six of 256's, which is alone
// on its CU; split operands half as much again.  Cut products write and read
// their parts once more, 5 bytes a picosecond.  Measured, bfloat16, forward, by
// tile: 8192 x 512 x 50000 898, 466 and 567 us, 1000 x 2048 x 32000 207, 139 and
// 133, 4000 x 128 x 10000 40, 37 and 60.
static CePlan ce_plan(int64_t m, int64_t n, int64_t steps, bool cut, bool split) {
    CePlan best{64, 1, INFINITY};
    const struct { int b; double us, more; } kind[3] = {
        {64, 0.22, 2}, {128, 0.45, 2}, {256, 1.6, 6}};
    for (const auto& k : kind) {
        if (split && k.b == 256) break;
        const int64_t tiles = ceil_div(m, k.b) * ceil_div(n, k.b);
        for (int s = 1; s <= (cut ? 32 : 1); s *= 2) {
            if (s > 1 && steps < 4 * s) break;
            if (tiles * s > (1 << 22) && !(k.b == (split ? 128 : 256) && s == 1)) continue;
            const double us = (double)ceil_div(tiles * s, 256) * ((double)ceil_div(steps, s) + k.more) *
                                  k.us * (split ? 1.5 : 1.) +
                              (s > 1 ? 3. + (double)s * (double)m * (double)n * 8. / 5e6 : 0.);
            if (us < best.us) best = CePlan{k.b, s, us};
        }
    }
    return best;
}

struct CeShape {
    int64_t rows, cols, classes;
    int32_t dtype;
    bool split;
    int64_t cols_p;     // columns of a packed operand
    int64_t rows_p;     // rows of g and of x's copy
    int64_t value;      // 16-bit values that a value takes in a packed operand
};

static CeShape ce_shape(int64_t rows, int64_t cols, int64_t classes, int32_t dtype) {
    CeShape s{rows, cols, classes, dtype, dtype == SPOPT_DTYPE_F32, 0, 0, 1};
    s.cols_p = ceil_div(cols, 64) * 64;
    s.rows_p = ceil_div(rows, 64) * 64;
    s.value = s.split ? 2 : 1;
    return s;
}

// Classes at a time.  Forward: copies of W's rows of up to 256 MiB, and grids of
// up to 2^22 tiles.  Backward: g of up to 512 MiB, or 256 where rows are short and
// g's traffic bounds the pass, as the last-level cache then keeps much of it (512
// against 256: 8192 x 128 x 50021 float32 1735 and 1552 us, bfloat16 820 and 709; 2000 x 64
// x 100000 bfloat16 408 and 290; 8192 x 256 x 50021 bfloat16 1130 and 1103; 384 to 640
// columns within 6% either way; 2000 x 1024 x 100000 bfloat16 1404 and 1642, 4096 x 1024 x
// 131072 3692 and 4363); for at least 2048 classes.
static int64_t ce_piece(const CeShape& s, bool backward) {
    int64_t most = ((int64_t)1 << 28) / (s.cols_p * s.value * 2);
    if (backward) {
        const int64_t g = ((int64_t)1 << (s.cols <= 512 ? 28 : 29)) / (s.rows_p * s.value * 2);
        most = most < g ? most : g;
    }
    if (most < 2048) most = 2048;
    const int64_t tiles = ((int64_t)1 << 22) / ceil_div(s.rows, 256);
    if (most > tiles * 256) most = tiles * 256;
    most = most / 256 * 256;
    const int64_t all = ceil_div(s.classes, 256) * 256;
    if (most >= all) return all;
    return ceil_div(ceil_div(all, ceil_div(all, most)), 256) * 256;  // pieces alike
}

struct CeBuffers {
    CeScalars* scalars;
    CeScan* scans;
    uint32_t* amax;
    void* x;            // x's copy
    void* x2;           // and the one that dW takes where rows have powers
    void* w;            // a piece of W's copy
    // forward
    float2* parts;
    float* sums;
    float* at_target;
    float* row_loss;
    // backward
    float* coef;
    int* powers;
    void* g;
    float* dx_parts;
    float* dw_parts;
};

struct CeRun {
    CeShape s;
    bool direct;         // the kernels of cross_entropy_direct.hip
    int64_t piece;
    CePlan logits, dx, dw;
    int64_t parts;       // of the classes, in the forward pass
};

// As ce_plan, for the direct kernels: an inner step takes a tile of 16 and 64
// rows about 0.25 and 0.3 us, of float32 0.4 and 0.7, and joining the parts of a
// cut axis a launch.
static CePlan ce_direct_plan(const CeShape& s, int64_t m, int64_t n, int64_t k, bool cut) {
    const int64_t steps = ceil_div(k, s.split ? 32 : 64);
    CePlan best{64, 1, INFINITY};
    for (int tile = 16; tile <= 64; tile += 48)
        for (int splits = 1; splits <= (cut ? 32 : 1); splits *= 2) {
            const int64_t blocks = ceil_div(m, tile) * ceil_div(n, 64) * splits;
            // Each part has a step at least.
            if (splits > 1 && (blocks > 1024 || splits > steps)) break;
            const double step = s.split ? tile == 16 ? 0.4 : 0.7 : tile == 16 ? 0.25 : 0.3;
            const double us = (double)ceil_div(blocks, 256) *
                                  ((double)ceil_div(steps, splits) * step + 1.) +
                              (splits > 1 ? 5. : 0.);
            if (us < best.us) best = CePlan{tile, splits, us};
        }
    return best;
}

// Which kernels, and their tiles.  Packed operands cost a launch for each copy and
// each thing found out about them, 3.3 us each, and the copies' traffic (x's in
// any backward pass; both operands' of float32, 12 bytes a value with the pass that
// finds the largest; of 16 bits, 4 bytes a value of rows that have a remainder);
// the direct kernels multiply more slowly, those of float32 far more.  Both sides
// measured at 136 sizes, forward and backward: the estimates choose the slower one
// at 30 of 272, by 1.03 to 1.3 times, and 1.5 to 1.7 backward at 200000 rows and more of 10
// classes, where a block's time is not what its steps take.  4 x 256 x 1000 float32: 20.7
// against 31.8 us forward and 24.4 against 43.3 backward; 500 x 256 x 100000 float32: 323
// against 153 and 1007 against 416.
static CeRun ce_run(const CeShape& s, bool backward) {
    CeRun d{}, p{};
    d.s = p.s = s;
    d.direct = true;
    d.piece = ceil_div(s.classes, 64) * 64;
    d.parts = ceil_div(s.classes, 64);
    d.logits = ce_direct_plan(s, s.rows, s.classes, s.cols, false);
    p.piece = ce_piece(s, backward);
    const int64_t inner = s.split ? 32 : 64;
    const int64_t first = s.classes < p.piece ? s.classes : p.piece;
    const double pieces = (double)ceil_div(s.classes, p.piece);
    p.logits = ce_plan(s.rows, first, s.cols_p / inner, false, s.split);
    const bool copies = s.split || s.cols % 64 != 0;
    double us_d = d.logits.us, us_p = p.logits.us * pieces;
    us_p += copies ? (double)((s.rows + s.classes) * s.cols) * (s.split ? 12. : 4.) / 4.2e6 : 0.;
    if (!backward) {
        us_p += s.split ? 10. : copies ? 6.6 : 0.;
    } else {
        d.dx = ce_direct_plan(s, s.rows, s.cols, s.classes, true);
        d.dw = ce_direct_plan(s, s.classes, s.cols, s.rows, true);
        p.dx = ce_plan(s.rows, s.cols, ceil_div(first, inner), true, s.split);
        p.dw = ce_plan(first, s.cols, ceil_div(s.rows, inner), true, s.split);
        us_d += d.dx.us + d.dw.us;
        us_p += (p.dx.us + p.dw.us) * pieces + (s.split ? 16. : copies ? 13. : 10.);
        us_p += copies ? 0. : (double)(s.rows * s.cols) * 4. / 4.2e6;
    }
    // Grids and g have to fit at once.
    const int64_t blocks = ceil_div(s.rows, 16) * ceil_div(s.classes, 64) +
                           (ceil_div(s.rows, 16) + ceil_div(s.classes, 16)) * ceil_div(s.cols, 64);
    const bool fits = blocks < (1 << 22) && s.rows_p <= ((int64_t)1 << 29) / (d.piece * 4);
    if (fits && us_d <= 1.1 * us_p) return d;
    for (int64_t v = 0; v < s.classes; v += p.piece) {
        const int64_t n = s.classes - v < p.piece ? s.classes - v : p.piece;
        p.parts += ce_parts(ceil_div(s.rows, p.logits.tile), ceil_div(n, p.logits.tile),
                            p.logits.tile);
    }
    return p;
}

static size_t ce_layout(const CeRun& r, bool backward, char* base, CeBuffers* b) {
    const CeShape& s = r.s;
    size_t at = 0;
    auto take = [&](size_t bytes) {
        char* p = base + at;
        at += align_up(bytes, 256);
        return (void*)p;
    };
    b->scalars = (CeScalars*)take(sizeof(CeScalars));
    b->scans = (CeScan*)take(backward ? kCeScans * sizeof(CeScan) : 0);
    if (!r.direct) {
        b->amax = (uint32_t*)take(2 * kAmaxParts * 4);
        b->x = take((size_t)(s.rows_p * s.cols_p * s.value) * 2);
        b->w = take((size_t)(r.piece * s.cols_p * s.value) * 2);
    }
    if (!backward) {
        b->parts = (float2*)take((size_t)(r.parts * s.rows) * 8);
        b->sums = (float*)take((size_t)(r.parts * s.rows) * 4);
        b->at_target = (float*)take((size_t)s.rows * 4);
        b->row_loss = (float*)take((size_t)s.rows * 4);
        return at;
    }
    // The reduction, which decides whether rows have powers, does not change the size.
    if (!r.direct) b->coef = (float*)take((size_t)s.rows_p * 4);
    if (s.dtype != SPOPT_DTYPE_BF16 && !(r.direct && s.split)) {
        b->powers = (int*)take((size_t)s.rows_p * 4);
        if (!r.direct) b->x2 = take((size_t)(s.rows_p * s.cols_p * s.value) * 2);
    }
    b->g = take((size_t)(s.rows_p * r.piece) * (r.direct ? 4 : 2 * s.value));
    b->dx_parts = (float*)take((size_t)(r.dx.splits * s.rows * s.cols_p) * 4);
    b->dw_parts = (float*)take(
        r.dw.splits > 1 ? (size_t)(r.dw.splits * r.piece * s.cols_p) * 4 : 0);
    return at;
}

static int ce_check_size(const char* what, int64_t rows, int64_t cols, int64_t classes,
                         int32_t dtype) {
    if (dtype != SPOPT_DTYPE_F32 && dtype != SPOPT_DTYPE_BF16 && dtype != SPOPT_DTYPE_F16)
        return fail(SPOPT_EINVAL, "%s: unknown element type %d", what, dtype);
    constexpr int64_t kMost = (int64_t)1 << 36;
    if (rows < 0 || cols < 1 || classes < 1 || rows > (1 << 27) || cols > (1 << 20) ||
        classes > (1 << 30) || rows > kMost / cols || classes > kMost / cols)
        return fail(SPOPT_EINVAL, "%s: bad size %lld x %lld for %lld classes", what,
                    (long long)rows, (long long)cols, (long long)classes);
    return SPOPT_OK;
}

template <class F>
static void ce_types(int32_t dtype, F&& f) {
    if (dtype == SPOPT_DTYPE_F32)
        f(_Float16{}, std::true_type{});
    else if (dtype == SPOPT_DTYPE_F16)
        f(_Float16{}, std::false_type{});
    else
        f(__bf16{}, std::false_type{});
}

template <bool SPLIT, class F>
static void ce_tilings(int tile, F&& f) {
    if (tile == 64) {
        f(CeS{});
    } else if (SPLIT || tile == 128) {
        f(CeM{});
    } else {
        if constexpr (!SPLIT) f(CeL{});
    }
}

template <class K, class TL, class... A>
static int ce_launch(K kernel, TL, int64_t blocks, hipStream_t s, const A&... a) {
    // The 256 tile holds three stages of one side and two of the other.
    constexpr int bytes = TL::BM == 256 ? 160 * 1024 : TL::STAGES * TL::kStage * 2;
    if constexpr (bytes > 64 * 1024) {
        SPOPT_HIP(hipFuncSetAttribute((const void*)kernel,
                                      hipFuncAttributeMaxDynamicSharedMemorySize, bytes));
    }
    kernel<<<(unsigned)blocks, TL::kThreads, bytes, s>>>(a...);
    SPOPT_LAUNCHED();
    return SPOPT_OK;
}

template <int MODE>
static int ce_logits(const CeRun& r, CeProduct c, const CeLogits& w, hipStream_t s) {
    int rc = SPOPT_OK;
    c.tiles_m = ceil_div(c.m, r.logits.tile);
    // g's columns beyond the piece's last class are written too, as zeros.
    c.tiles_n = ceil_div(MODE == kCeGrad ? w.cols_p : c.n, r.logits.tile);
    c.splits = ce_parts(c.tiles_m, c.tiles_n, r.logits.tile);
    ce_types(r.s.dtype, [&](auto t, auto split) {
        ce_tilings<decltype(split)::value>(r.logits.tile, [&](auto tl) {
            rc = ce_launch(k_ce_logits<decltype(t), decltype(split)::value, MODE, decltype(tl)>,
                           tl, c.tiles_m * c.splits, s, c, w);
        });
    });
    return rc;
}

template <int MODE>
static int ce_product(const CeRun& r, const CePlan& plan, CeProduct c, const CeResult& w,
                      const CeScalars* sc, hipStream_t s) {
    int rc = SPOPT_OK;
    c.splits = plan.splits;
    c.tiles_m = ceil_div(c.m, plan.tile);
    c.tiles_n = ceil_div(c.n, plan.tile);
    ce_types(r.s.dtype, [&](auto t, auto split) {
        ce_tilings<decltype(split)::value>(plan.tile, [&](auto tl) {
            rc = ce_launch(k_ce_product<decltype(t), decltype(split)::value, MODE, decltype(tl)>,
                           tl, c.tiles_m * c.tiles_n * c.splits, s, c, w, sc);
        });
    });
    return rc;
}

static unsigned ce_grid(int64_t items) {
    const int64_t b = ceil_div(items, 256);
    return (unsigned)(b < 1 ? 1 : b < 8192 ? b : 8192);
}

// An operand as the products take it: in place where it can be read 16 bytes at
// a time without a remainder, else a copy in `to`.
static int ce_operand(const CeShape& s, const void* a, int64_t ld, int64_t rows, int64_t rows_p,
                      bool copy, const int64_t* targets, int64_t ignored, const uint32_t* amax,
                      int n_amax, int* exponent, void* to, CeOperand* o, hipStream_t stream,
                      const int* powers = nullptr, int* exponent2 = nullptr, void* to2 = nullptr) {
    if (!copy && !s.split && s.cols % 64 == 0 && ld % 8 == 0 && ld <= (1 << 21) && aligned16(a)) {
        *o = CeOperand{a, ld, rows - 1, s.cols_p};
        return SPOPT_OK;
    }
    const unsigned grid = ce_grid(rows_p * s.cols_p / 8);
    if (s.split)
        k_ce_pack<float, _Float16><<<grid, 256, 0, stream>>>(
            (const float*)a, ld, rows, s.cols, rows_p, s.cols_p, targets, ignored, amax, n_amax,
            exponent, (_Float16*)to, powers, exponent2, (_Float16*)to2);
    else if (s.dtype == SPOPT_DTYPE_F16)
        k_ce_pack<_Float16, _Float16><<<grid, 256, 0, stream>>>(
            (const _Float16*)a, ld, rows, s.cols, rows_p, s.cols_p, targets, ignored, amax, n_amax,
            nullptr, (_Float16*)to, powers, exponent2, (_Float16*)to2);
    else
        k_ce_pack<__bf16, __bf16><<<grid, 256, 0, stream>>>(
            (const __bf16*)a, ld, rows, s.cols, rows_p, s.cols_p, targets, ignored, nullptr, 0,
            nullptr, (__bf16*)to, nullptr, nullptr, nullptr);
    SPOPT_LAUNCHED();
    *o = CeOperand{to, s.cols_p * s.value, rows_p - 1, s.cols_p};
    return SPOPT_OK;
}

// Both operands' largest values where they are split; x's where its rows get powers.
static int ce_amax(const CeShape& s, const void* x, int64_t x_ld, const int64_t* targets,
                   int64_t ignored, const void* w, int64_t w_ld, bool powers, const CeBuffers& b,
                   int* parts, hipStream_t stream) {
    *parts = 0;
    if (!s.split && !powers) return SPOPT_OK;
    const int64_t most = s.split && s.classes > s.rows ? s.classes : s.rows;
    int64_t n = ceil_div(most * s.cols, 256 * 16);
    if (n > kAmaxParts) n = kAmaxParts;
    if (s.split)
        k_ce_amax<<<dim3((unsigned)n, 2), 256, 0, stream>>>(
            (const float*)x, x_ld, s.rows, targets, ignored, (const float*)w, w_ld, s.classes,
            s.cols, b.amax);
    else
        k_ce_amax<<<dim3((unsigned)n, 1), 256, 0, stream>>>(
            (const _Float16*)x, x_ld, s.rows, targets, ignored, (const _Float16*)nullptr, 0, 0,
            s.cols, b.amax);
    SPOPT_LAUNCHED();
    *parts = (int)n;
    return SPOPT_OK;
}

// What both passes check alike.
static int ce_enter(const char* what, const CeShape& s, const void* x, int64_t x_ld,
                    const void* w, int64_t w_ld, const int64_t* targets, double smoothing,
                    int32_t reduction) {
    if (!(smoothing >= 0.0 && smoothing <= 1.0))
        return fail(SPOPT_EINVAL, "%s: label smoothing must lie in [0, 1]", what);
    if (reduction != SPOPT_REDUCE_NONE && reduction != SPOPT_REDUCE_SUM &&
        reduction != SPOPT_REDUCE_MEAN)
        return fail(SPOPT_EINVAL, "%s: unknown reduction %d", what, reduction);
    if (s.rows > 0 && (x == nullptr || targets == nullptr))
        return fail(SPOPT_EINVAL, "%s: NULL x or targets", what);
    if (w == nullptr) return fail(SPOPT_EINVAL, "%s: NULL weight", what);
    if ((s.rows > 1 && x_ld < s.cols) || (s.classes > 1 && w_ld < s.cols))
        return fail(SPOPT_EINVAL, "%s: a row stride below cols", what);
    return SPOPT_OK;
}

static int ce_validate(const char* what, const CeShape& s, const void* x, int64_t x_ld,
                       const void* w, int64_t w_ld, const int64_t* targets, int64_t ignored,
                       hipStream_t stream) {
    return validate_on_device(stream, false, what, [&](uint32_t* status) {
        const unsigned grid = (unsigned)(s.rows < 4096 ? s.rows : 4096);
        auto check = [&](auto t) {
            using S = decltype(t);
            k_ce_check<S><<<grid, 256, 0, stream>>>((const S*)x, x_ld, s.rows, s.cols, targets,
                                                    ignored, s.classes, status);
        };
        if (s.dtype == SPOPT_DTYPE_F32)
            check(float{});
        else if (s.dtype == SPOPT_DTYPE_F16)
            check(_Float16{});
        else
            check(__bf16{});
        SPOPT_LAUNCHED();
        return launch_check_finite(w, s.dtype, s.classes, s.cols, w_ld, status, stream);
    });
}

// Scans the rows once where every block of g's kernel (direct), or the one of
// k_ce_coef, would take longer over them than a launch does.  Backward, in the blocks
// against once: 64 columns and 10 classes float32, 4000 rows 26 against 28 us, 16384 rows
// 50 against 47, 1000000 rows 23500 against 2180; 256 x 1000 bfloat16 with a factor for each
// row, 2000 rows 45.7 against 48, 4000 rows 73 against 67; packed, 256 x 1000 float32, 8192
// rows 104.6 against 106.2, 16384 rows 153 against 151, 65536 rows 500 against 473.
static int ce_scan(CeRows* rows, const CeRun& r, const CeBuffers& b, hipStream_t s) {
    if (rows->reduction == SPOPT_REDUCE_SUM ||
        (rows->reduction == SPOPT_REDUCE_NONE && r.direct && r.s.split))
        return SPOPT_OK;
    const int64_t readers =
        r.direct ? ceil_div(rows->rows, r.logits.tile) * ceil_div(rows->classes, 64) : 256;
    if (rows->rows <= ((int64_t)1 << 21) / readers) return SPOPT_OK;
    const int64_t blocks = ceil_div(rows->rows, 1024);
    rows->n_scans = (int)(blocks < kCeScans ? blocks : kCeScans);
    k_ce_scan<<<(unsigned)rows->n_scans, 256, 0, s>>>(*rows, b.scans);
    SPOPT_LAUNCHED();
    rows->scans = b.scans;
    return SPOPT_OK;
}

static int ce_workspace(const char* what, const void* workspace, size_t have, size_t need) {
    if (need != 0 && (workspace == nullptr || !aligned16(workspace) || have < need))
        return fail(SPOPT_EWORKSPACE, "%s: workspace of %zu bytes, needs %zu", what, have, need);
    return SPOPT_OK;
}

}  // namespace spopt

using namespace spopt;

extern "C" int linear_cross_entropy_workspace_size(int64_t rows, int64_t cols, int64_t classes,
                                                   int32_t dtype, int32_t backward,
                                                   size_t* bytes) {
    const char* what = "linear_cross_entropy_workspace_size";
    if (bytes == nullptr) return fail(SPOPT_EINVAL, "%s: NULL output", what);
    int rc = ce_check_size(what, rows, cols, classes, dtype);
    if (rc) return rc;
    *bytes = 0;
    if (rows == 0) return SPOPT_OK;
    CeBuffers b;
    *bytes = ce_layout(ce_run(ce_shape(rows, cols, classes, dtype), backward != 0), backward != 0,
                       nullptr, &b);
    return SPOPT_OK;
}

extern "C" int linear_cross_entropy_plan(int64_t rows, int64_t cols, int64_t classes, int32_t dtype,
                                         int32_t backward, spopt_ce_plan* plan) {
    const char* what = "linear_cross_entropy_plan";
    if (plan == nullptr) return fail(SPOPT_EINVAL, "%s: NULL output", what);
    const int rc = ce_check_size(what, rows, cols, classes, dtype);
    if (rc) return rc;
    if (rows == 0) return fail(SPOPT_EINVAL, "%s: no rows", what);
    const CeRun r = ce_run(ce_shape(rows, cols, classes, dtype), backward != 0);
    *plan = spopt_ce_plan{r.direct, r.logits.tile, r.dx.tile, r.dw.tile,
                          r.dx.splits, r.dw.splits, r.piece};
    return SPOPT_OK;
}

extern "C" int linear_cross_entropy_forward(const void* x, int64_t x_stride, const void* weight,
                                            int64_t weight_stride, int64_t rows, int64_t cols,
                                            int64_t classes, int32_t dtype,
                                            const int64_t* targets, int64_t ignore_index,
                                            double label_smoothing, int32_t reduction, float* loss,
                                            float* lse, void* workspace, size_t workspace_bytes,
                                            void* stream, uint32_t flags) {
    const char* what = "linear_cross_entropy_forward";
    hipStream_t s = (hipStream_t)stream;
    int rc = ce_check_size(what, rows, cols, classes, dtype);
    if (rc) return rc;
    const CeShape sh = ce_shape(rows, cols, classes, dtype);
    rc = ce_enter(what, sh, x, x_stride, weight, weight_stride, targets, label_smoothing,
                  reduction);
    if (rc) return rc;
    if ((loss == nullptr && (rows > 0 || reduction != SPOPT_REDUCE_NONE)) ||
        (lse == nullptr && rows > 0))
        return fail(SPOPT_EINVAL, "%s: NULL loss or lse", what);
    if (rows == 0) {
        if (reduction == SPOPT_REDUCE_NONE) return SPOPT_OK;
        k_ce_reduce<<<1, 1024, 0, s>>>(nullptr, nullptr, ignore_index, 0, reduction, loss);
        SPOPT_LAUNCHED();
        return SPOPT_OK;
    }
    const CeRun r = ce_run(sh, false);
    CeBuffers b;
    rc = ce_workspace(what, workspace, workspace_bytes, ce_layout(r, false, (char*)workspace, &b));
    if (rc) return rc;
    if (flags & SPOPT_VALIDATE) {
        rc = ce_validate(what, sh, x, x_stride, weight, weight_stride, targets, ignore_index, s);
        if (rc) return rc;
    }
    CeLogits w{};
    w.scalars = b.scalars;
    w.targets = targets;
    w.classes = classes;
    w.smoothing = (float)label_smoothing;
    w.parts = b.parts;
    w.sums = label_smoothing != 0.0 ? b.sums : nullptr;
    w.at_target = b.at_target;
    CeProduct c{};
    int amax = 0;
    if (r.direct) {
        rc = ce_direct_loss(dtype, r.logits.tile, CeSide{x, x_stride, rows, cols, targets, ignore_index, nullptr},
                            CeSide{weight, weight_stride, classes, cols, nullptr, 0, nullptr}, w, s);
    } else {
        rc = ce_amax(sh, x, x_stride, targets, ignore_index, weight, weight_stride, false, b, &amax,
                     s);
        c.m = rows;
        c.steps = sh.cols_p / (sh.split ? 32 : 64);
        if (!rc)
            rc = ce_operand(sh, x, x_stride, rows, rows, false, targets, ignore_index, b.amax,
                            amax, &b.scalars->ex, b.x, &c.p, s);
    }
    if (rc) return rc;
    for (int64_t v = 0; v < classes && !r.direct; v += r.piece) {
        c.n = classes - v < r.piece ? classes - v : r.piece;
        w.first = v;
        rc = ce_operand(sh, (const char*)weight + (size_t)(v * weight_stride) * dtype_bytes(dtype),
                        weight_stride, c.n, c.n, false, nullptr, 0, b.amax + kAmaxParts, amax,
                        &b.scalars->ew, b.w, &c.q, s);
        if (!rc) rc = ce_logits<kCeLoss>(r, c, w, s);
        if (rc) return rc;
        w.first_part += ce_parts(ceil_div(rows, r.logits.tile), ceil_div(c.n, r.logits.tile),
                                 r.logits.tile);
    }
    // Rows of few tiles one a thread; and where one block is enough (for up to
    // 128 rows, or 2048 of few tiles), it spares the launch that sums the rows.
    int per = rows > 64 && r.parts <= 16 ? 1024 : 64;
    while (per <= 64 && per > 1 && rows <= per / 2) per /= 2;
    int64_t blocks = ceil_div(rows, per);
    if (reduction != SPOPT_REDUCE_NONE && blocks == 2) blocks = 1;
    k_ce_join<<<(unsigned)blocks, 1024, 0, s>>>(
        b.parts, w.sums, b.at_target, targets, ignore_index, rows, r.parts, classes,
        w.smoothing, per, reduction, b.row_loss, loss, lse);
    SPOPT_LAUNCHED();
    if (reduction != SPOPT_REDUCE_NONE && blocks > 1) {
        k_ce_reduce<<<1, 1024, 0, s>>>(b.row_loss, targets, ignore_index, rows, reduction, loss);
        SPOPT_LAUNCHED();
    }
    return SPOPT_OK;
}

extern "C" int linear_cross_entropy_backward(
    const float* dloss, const void* x, int64_t x_stride, const void* weight, int64_t weight_stride,
    int64_t rows, int64_t cols, int64_t classes, int32_t dtype, const int64_t* targets,
    int64_t ignore_index, double label_smoothing, int32_t reduction, const float* lse, void* dx,
    int64_t dx_stride, void* dweight, int64_t dweight_stride, void* workspace,
    size_t workspace_bytes, void* stream, uint32_t flags) {
    const char* what = "linear_cross_entropy_backward";
    hipStream_t s = (hipStream_t)stream;
    int rc = ce_check_size(what, rows, cols, classes, dtype);
    if (rc) return rc;
    const CeShape sh = ce_shape(rows, cols, classes, dtype);
    rc = ce_enter(what, sh, x, x_stride, weight, weight_stride, targets, label_smoothing,
                  reduction);
    if (rc) return rc;
    if (rows > 0 && (dloss == nullptr || lse == nullptr))
        return fail(SPOPT_EINVAL, "%s: NULL dloss or lse", what);
    if ((dx != nullptr && rows > 1 && dx_stride < cols) ||
        (dweight != nullptr && classes > 1 && dweight_stride < cols))
        return fail(SPOPT_EINVAL, "%s: a row stride below cols", what);
    if (dx == nullptr && dweight == nullptr) return SPOPT_OK;
    // The splits' sums of an operand's gradient, to where it belongs.
    auto gather = [&](const float* parts, const CeScalars* sc, int splits, int64_t n, int uw,
                      int ud, const int* powers, void* out, int64_t ld) {
        const unsigned grid = ce_grid(n * (sh.cols_p / 4));
        if (dtype == SPOPT_DTYPE_F32)
            k_ce_gather<<<grid, 256, 0, s>>>(parts, splits, n, sh.cols_p, cols, sc, uw, ud, powers,
                                             (float*)out, ld);
        else if (dtype == SPOPT_DTYPE_F16)
            k_ce_gather<<<grid, 256, 0, s>>>(parts, splits, n, sh.cols_p, cols, sc, uw, ud, powers,
                                             (_Float16*)out, ld);
        else
            k_ce_gather<<<grid, 256, 0, s>>>(parts, splits, n, sh.cols_p, cols, sc, uw, ud, powers,
                                             (__bf16*)out, ld);
    };
    if (rows == 0) {
        if (dweight == nullptr) return SPOPT_OK;
        gather(nullptr, nullptr, 0, classes, 0, 0, nullptr, dweight, dweight_stride);
        SPOPT_LAUNCHED();
        return SPOPT_OK;
    }
    const CeRun r = ce_run(sh, true);
    CeBuffers b{};
    rc = ce_workspace(what, workspace, workspace_bytes, ce_layout(r, true, (char*)workspace, &b));
    if (rc) return rc;
    if (flags & SPOPT_VALIDATE) {
        rc = ce_validate(what, sh, x, x_stride, weight, weight_stride, targets, ignore_index, s);
        if (rc) return rc;
    }
    CeRows factors{dloss, targets, ignore_index, rows, classes, reduction,
                   (float)(1.0 - label_smoothing), nullptr, 0,
                   reduction == SPOPT_REDUCE_NONE && b.powers != nullptr};
    const int* const powers = factors.powers ? b.powers : nullptr;
    rc = ce_scan(&factors, r, b, s);
    if (rc) return rc;
    CeLogits w{};
    w.scalars = b.scalars;
    w.targets = targets;
    w.classes = classes;
    w.smoothing = (float)label_smoothing;
    w.lse = lse;
    w.coef = b.coef;
    w.g = b.g;
    w.rows_p = sh.rows_p;
    if (r.direct) {
        w.ldg = w.cols_p = r.piece;
        w.rows_p = rows;
        const CeSide xs{x, x_stride, rows, cols, targets, ignore_index, nullptr};
        const CeSide ws{weight, weight_stride, classes, cols, nullptr, 0, nullptr};
        rc = ce_direct_grad(dtype, r.logits.tile, xs, ws, w, factors, b.scalars, b.powers, s);
        if (rc) return rc;
        CeBoth both{};
        both.g = CeSide{b.g, r.piece, rows, r.piece, nullptr, 0, powers};
        both.w = ws;
        both.x = xs;
        both.rows = rows;
        both.cols = cols;
        both.classes = classes;
        both.dx_tile = r.dx.tile;
        both.dw_tile = r.dw.tile;
        both.dx_splits = r.dx.splits;
        both.dw_splits = r.dw.splits;
        both.scalars = b.scalars;
        if (dx != nullptr)
            both.dx_blocks = ceil_div(rows, r.dx.tile) * ceil_div(cols, 64);
        // Tiles of few inner steps are mostly waits for loads and stores: a block goes
        // through as many as leave the card full, the loads running on.
        const int64_t tiles = ceil_div(classes, r.dw.tile), across = ceil_div(cols, 64);
        const int64_t most = tiles * across * r.dw.splits / 2048;
        both.dw_group = (int)(most < 1 ? 1 : most > tiles ? tiles : most);
        if (dweight != nullptr) both.dw_blocks = ceil_div(tiles, both.dw_group) * across;
        both.dx = CeResult{r.dx.splits > 1 ? b.dx_parts : nullptr, sh.cols_p, 0, dx, dx_stride,
                           powers};
        both.dw = CeResult{r.dw.splits > 1 ? b.dw_parts : nullptr, sh.cols_p, 0, dweight,
                           dweight_stride, nullptr};
        rc = ce_direct_products(dtype, both, s);
        if (rc) return rc;
        if (dx != nullptr && r.dx.splits > 1)
            gather(b.dx_parts, b.scalars, r.dx.splits, rows, 0, 0, powers, dx, dx_stride);
        if (dweight != nullptr && r.dw.splits > 1)
            gather(b.dw_parts, b.scalars, r.dw.splits, classes, 0, 0, nullptr, dweight,
                   dweight_stride);
        SPOPT_LAUNCHED();
        return SPOPT_OK;
    }
    int amax = 0;
    rc = ce_amax(sh, x, x_stride, targets, ignore_index, weight, weight_stride, powers != nullptr, b,
                 &amax, s);
    if (rc) return rc;
    const int64_t coefs = factors.scans == nullptr ? 1 : ceil_div(sh.rows_p, 4096);
    k_ce_coef<<<(unsigned)(coefs < 1024 ? coefs : 1024), 1024, 0, s>>>(factors, sh.rows_p, b.coef,
                                                                       b.powers, b.scalars);
    SPOPT_LAUNCHED();
    // x is copied for its rows that are ignored: they may hold anything, and meet
    // g's zeros in dW.
    CeOperand xo{}, wo{}, g{};
    rc = ce_operand(sh, x, x_stride, rows, sh.rows_p, true, targets, ignore_index, b.amax, amax,
                    &b.scalars->ex, b.x, &xo, s, powers, &b.scalars->ed, b.x2);
    if (rc) return rc;
    CeOperand xd = xo;
    if (powers != nullptr) xd.base = b.x2;
    const int64_t inner = sh.split ? 32 : 64;
    for (int64_t v = 0; v < classes; v += r.piece) {
        const int64_t n = classes - v < r.piece ? classes - v : r.piece;
        const int64_t n_p = ceil_div(n, 64) * 64, ldg = n_p * sh.value;
        rc = ce_operand(sh, (const char*)weight + (size_t)(v * weight_stride) * dtype_bytes(dtype),
                        weight_stride, n, n, false, nullptr, 0, b.amax + kAmaxParts, amax,
                        &b.scalars->ew, b.w, &wo, s);
        if (rc) return rc;
        CeProduct c{};
        c.p = xo;
        c.q = wo;
        c.m = rows;
        c.n = n;
        c.steps = sh.cols_p / inner;
        w.first = v;
        w.ldg = ldg;
        w.cols_p = n_p;
        rc = ce_logits<kCeGrad>(r, c, w, s);
        if (rc) return rc;
        g = CeOperand{b.g, ldg, sh.rows_p - 1, n_p};
        CeResult o{};
        if (dx != nullptr) {
            c.p = g;
            c.q = wo;
            c.m = rows;
            c.n = cols;
            c.steps = n_p / inner;
            o.out = dx;
            o.out_ld = dx_stride;
            o.ld = sh.cols_p;
            o.add = v > 0;
            o.powers = powers;
            o.parts = r.dx.splits == 1 && r.piece >= classes ? nullptr : b.dx_parts;
            rc = ce_product<kCeDx>(r, r.dx, c, o, b.scalars, s);
            if (rc) return rc;
        }
        if (dweight != nullptr) {
            c.p = g;
            c.q = xd;
            c.m = n;
            c.n = cols;
            c.steps = sh.rows_p / inner;
            o.out = (char*)dweight + (size_t)(v * dweight_stride) * dtype_bytes(dtype);
            o.out_ld = dweight_stride;
            o.ld = sh.cols_p;
            o.add = 0;
            o.powers = nullptr;
            o.parts = r.dw.splits == 1 ? nullptr : b.dw_parts;
            rc = ce_product<kCeDw>(r, r.dw, c, o, b.scalars, s);
            if (rc) return rc;
            if (r.dw.splits > 1) {
                gather(b.dw_parts, b.scalars, r.dw.splits, n, 0, 1, nullptr, o.out,
                       dweight_stride);
                SPOPT_LAUNCHED();
            }
        }
    }
    if (dx != nullptr && (r.dx.splits > 1 || r.piece < classes)) {
        gather(b.dx_parts, b.scalars, r.dx.splits, rows, sh.split, 0, powers, dx, dx_stride);
        SPOPT_LAUNCHED();
    }
    return SPOPT_OK;
}
