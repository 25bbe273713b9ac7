// cross_entropy_direct.hip - the loss's kernels for small calls, which read the
// caller's operands as they lie: any stride and alignment, float32 on the float32
// matrix instructions.
//
// A launch costs the host 3.5 us, which is all that a small call takes.  These
// take two launches forward (the logits' tiles, the join) and two backward (g;
// both products, and a third where an inner axis is cut), where packed operands
// take up to five and nine.  Operands go through registers into LDS, three to six
// stages on their way, in tiles of 64 x 64 or, of few rows, 16 x 64, laid out in LDS
// as cross_entropy.hip's.  4 x 256 x 1000 float32: 20.7 us forward and 24.4 backward a
// call, packed 31.8 and 43.3; of the 20.7 the host takes about 13.  6 x 966 x 67682
// float16 backward 155 us, where one pass over W takes 26: rows at odd addresses, and
// W read twice.
#include "cross_entropy.hpp"

namespace spopt {

typedef uint32_t uint4v __attribute__((ext_vector_type(4)));

// PAIR: P is g in float32, which is taken as two of T, the rounded value and what that
// leaves, and multiplied twice: what rounds the gradients is then their own type
// alone.  Of few rows or classes g rounded once is off by as much again (bfloat16, 2.4e-3
// against 1.6e-3), and what a row's classes have in common does not leave dx.  Small calls
// have the time: 300 x 100 x 3001 bfloat16 30.5 -> 31.2 us, 2000 x 256 x 1000 44 -> 47.5,
// 6 x 966 x 67682 float16 148 -> 155.
template <class T, bool TP, bool TQ, int BM_, bool PAIR = false>
struct CeDirect {
    static constexpr int BM = BM_, BN = 64, WGN = BM == 64 ? 2 : 4;  // four waves
    static constexpr int FM = BM / 16 * WGN / 4, FN = 4 / WGN;
    static constexpr int kAhead = BM == 64 ? PAIR ? 3 : 4 : 6;  // stages on their way in registers
    static constexpr int kRow = TQ || FN % 2 ? 4 : 8;     // adjacent columns of a lane
    static constexpr int E = 16 / (int)sizeof(T);         // values of a chunk
    static constexpr int kInner = 128 / (int)sizeof(T);   // values of the inner axis a stage
    static constexpr int kPlane = BM * 128;               // bytes of a stage
    static constexpr int kSideP = kPlane * (PAIR ? 2 : 1), kSideQ = BN * 128;
    static constexpr int kBytes = 2 * (kSideP + kSideQ);  // of LDS
    typedef T chunk __attribute__((ext_vector_type(E)));
    typedef float wide __attribute__((ext_vector_type(E)));
    static_assert(BM == 64 || BM == 16, "two tiles");
    static_assert(!PAIR || sizeof(T) == 2, "float32 holds g");

    // Row v of a turned side has its 16 columns from 16 u on at u ^ turn(v).
    template <int B>
    static __device__ __forceinline__ int turn(int v) {
        return B == 16 ? 0 : sizeof(T) == 4 ? v >> 2 & 3 : turn_q<64>(v);
    }

    // A side's loads: 8 B chunks a stage.
    template <bool TURN, int B, bool WIDE = false>
    struct Feed {
        static constexpr int kLoads = B == 64 ? 2 : 1;
        typedef std::conditional_t<WIDE, float, T> S;
        typedef std::conditional_t<WIDE, wide, chunk> loaded;
        const S* base;
        int up[WIDE && !TURN ? kLoads : 1];  // the row's power of two
        const int64_t* targets;
        int64_t ld, rows, cols, ignored, row[kLoads], col;
        int place[kLoads];
        __device__ __forceinline__ void init(const CeSide& s, int64_t first, bool pair) {
            base = (const S*)s.base;
            targets = s.targets;
            ld = s.ld;
            rows = s.rows;
            cols = s.cols;
            ignored = s.ignored;
            constexpr int kWide = 16 / E;  // chunks of 16 columns
#pragma unroll
            for (int l = 0; l < kLoads; ++l) {
                const int at = ((int)threadIdx.x + 256 * l) % (8 * B);
                if constexpr (TURN) {
                    const int v = at / (B / E), c = at % (B / E);
                    row[l] = v;
                    col = first + c * E;
                    place[l] = (v * (B / E) + ((c / kWide) ^ turn<B>(v)) * kWide + c % kWide) * 16;
                } else {
                    const int v = at / 8, c = at % 8, in = v & 31;
                    row[l] = first + (pair ? v - in + ((in & 12) >> 2) * 8 + (in >> 4) * 4 + (in & 3)
                                           : v);
                    if (row[l] >= rows || (targets && targets[row[l]] == ignored)) row[l] = -1;
                    if constexpr (WIDE)
                        up[l] = s.powers && row[l] >= 0 ? s.powers[row[l]] : 0;
                    col = c * E;
                    place[l] = (v * 8 + (c ^ (v & 7))) * 16;
                }
            }
        }
        // Chunk l of step k, `shift` columns on (of a turned side).
        __device__ __forceinline__ loaded load(int64_t k, int l, int64_t shift) const {
            int64_t r = row[l], c = TURN ? col + shift : col;
            bool in;
            if constexpr (TURN) {
                r += k * kInner;
                in = r < rows && !(targets && targets[r] == ignored);
            } else {
                c += k * kInner;
                in = r >= 0;
            }
            loaded v = {};
            if (!in || c >= cols) return v;
            const S* p = base + r * ld;
            if constexpr (WIDE) {
                return *(const loaded*)(p + c);  // g's rows are padded to whole chunks
            } else {
                if (cols < E) {
#pragma unroll
                    for (int e = 0; e < E; ++e)
                        if (c + e < cols) v[e] = p[c + e];
                    return v;
                }
                // The chunk at a row's end is moved back to end with it, and its values
                // forward again: loads of single values would keep the whole wave.
                const int64_t at = c + E <= cols ? c : cols - E;
                v = *(const typename Pack<T, E>::type*)(p + at);
                const int skip = (int)(c - at);
                if (skip != 0) {
                    uint4v q = __builtin_bit_cast(uint4v, v);
                    if (skip & E / 2) q = uint4v{q[2], q[3], 0, 0};
                    if (skip & E / 4) q = uint4v{q[1], q[2], q[3], 0};
                    if (E == 8 && skip & 1)
                        q = uint4v{q[0] >> 16 | q[1] << 16, q[1] >> 16 | q[2] << 16,
                                   q[2] >> 16 | q[3] << 16, q[3] >> 16};
                    v = __builtin_bit_cast(chunk, q);
                }
                return v;
            }
        }
        // Chunk l into a stage in LDS.
        __device__ __forceinline__ void put(char* to, int l, const loaded& v) const {
            if constexpr (WIDE) {
                chunk hi, lo;
#pragma unroll
                for (int e = 0; e < E; ++e) {
                    const float u = TURN ? v[e] : ldexpf(v[e], up[l]);
                    hi[e] = (T)u;
                    lo[e] = (T)(u - (float)hi[e]);
                }
                *(chunk*)(to + place[l]) = hi;
                *(chunk*)(to + kPlane + place[l]) = lo;
            } else {
                *(chunk*)(to + place[l]) = v;
            }
        }
    };

    int lane, wv, wi, wj;
    float4v acc[FM][FN];

    __device__ __forceinline__ void init() {
        lane = lane_id();
        wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
        wi = wv / WGN * FM * 16;
        wj = wv % WGN * FN * 16;
    }
    __device__ __forceinline__ void clear() {
#pragma unroll
        for (int x = 0; x < FM; ++x)
#pragma unroll
            for (int y = 0; y < FN; ++y) acc[x][y] = float4v{0.f, 0.f, 0.f, 0.f};
    }

    // The operand of 16 rows (or columns) from `first` on: half kk of a stage.
    template <bool TURN, int B>
    __device__ __forceinline__ auto operand(const char* l, int first, int kk) const {
        typedef T vec __attribute__((ext_vector_type(E)));
        if constexpr (TURN && sizeof(T) == 4) {
            const int v = (kk * 4 + (lane >> 4)) * 4;
            const T* a = (const T*)l + v * B + ((first >> 4) ^ turn<B>(v)) * 16 + (lane & 15);
            return vec{a[0], a[B], a[2 * B], a[3 * B]};
        } else if constexpr (TURN) {
            typedef T half __attribute__((ext_vector_type(4)));
            const int v = (lane >> 4) * 8 + ((lane & 15) >> 2);
            const T* a = (const T*)l + (kk * 32 + v) * B + ((first >> 4) ^ turn<B>(v)) * 16 +
                         (lane & 3) * 4;
            const half lo = __builtin_bit_cast(half, read_turned((const _Float16*)a));
            const half hi = __builtin_bit_cast(half, read_turned((const _Float16*)(a + 4 * B)));
            return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
        } else {
            const int v = first + (lane & 15);
            return *(const vec*)(l + (v * 8 + ((kk * 4 + (lane >> 4)) ^ (v & 7))) * 16);
        }
    }

    // `tiles` tiles one below the other (one, but for a turned P), steps [k0, k1) of
    // the inner axis for each, one at least: `done(t)` where tile t's sums are there.  The loads run
    // on from tile to tile.
    template <class F>
    __device__ __forceinline__ void run(char* lds, const CeSide& p, const CeSide& q, int64_t i0,
                                        int tiles, int64_t j0, int64_t k0, int64_t k1, F done) {
        typedef Feed<TP, BM, PAIR> FeedP;
        typedef Feed<TQ, BN> FeedQ;
        FeedP fp;
        FeedQ fq;
        fp.init(p, i0, false);
        fq.init(q, j0, kRow == 8);
        const bool with_p = BM == 64 || threadIdx.x < 8 * BM;
        typename FeedP::loaded cp[kAhead][FeedP::kLoads];
        chunk cq[kAhead][FeedQ::kLoads];
        int64_t bk = k0, shift = 0, left = tiles * (k1 - k0);
        if (left <= 0) return;  // the host cuts no axis into more parts than it has steps
        auto bring = [&](int u) {
            if (left == 0) return;
#pragma unroll
            for (int l = 0; l < FeedP::kLoads; ++l)
                if (with_p) cp[u][l] = fp.load(bk, l, shift);
#pragma unroll
            for (int l = 0; l < FeedQ::kLoads; ++l) cq[u][l] = fq.load(bk, l, 0);
            --left;
            if (++bk == k1) {
                bk = k0;
                shift += BM;
            }
        };
#pragma unroll
        for (int u = 0; u < kAhead; ++u) bring(u);
        clear();
        int buf = 0, t = 0;
        int64_t k = k0;
        while (t < tiles) {
#pragma unroll
            for (int u = 0; u < kAhead; ++u) {
                if (t == tiles) break;
                char* const to = lds + buf * (kSideP + kSideQ);
#pragma unroll
                for (int l = 0; l < FeedP::kLoads; ++l)
                    if (with_p) fp.put(to, l, cp[u][l]);
#pragma unroll
                for (int l = 0; l < FeedQ::kLoads; ++l) fq.put(to + kSideP, l, cq[u][l]);
                bring(u);
                // One barrier a stage: whoever writes this place next has passed
                // the other one's, after all reads of this.
                __syncthreads();
#pragma unroll
                for (int kk = 0; kk < 2; ++kk) {
                    chunk a[FM], b[FN], less[PAIR ? FM : 1];
#pragma unroll
                    for (int x = 0; x < FM; ++x) a[x] = operand<TP, BM>(to, wi + x * 16, kk);
                    if constexpr (PAIR) {
#pragma unroll
                        for (int x = 0; x < FM; ++x)
                            less[x] = operand<TP, BM>(to + kPlane, wi + x * 16, kk);
                    }
#pragma unroll
                    for (int y = 0; y < FN; ++y) b[y] = operand<TQ, BN>(to + kSideP, wj + y * 16, kk);
#pragma unroll
                    for (int x = 0; x < FM; ++x)
#pragma unroll
                        for (int y = 0; y < FN; ++y) {
                            if constexpr (sizeof(T) == 4) {
#pragma unroll
                                for (int e = 0; e < 4; ++e)
                                    acc[x][y] = __builtin_amdgcn_mfma_f32_16x16x4f32(
                                        b[y][e], a[x][e], acc[x][y], 0, 0, 0);
                            } else {
                                acc[x][y] = matrix_16x16x32(b[y], a[x], acc[x][y]);
                                if constexpr (PAIR)
                                    acc[x][y] = matrix_16x16x32(b[y], less[x], acc[x][y]);
                            }
                        }
                }
                buf ^= 1;
                if (++k == k1) {
                    done(t);
                    k = k0;
                    if (++t < tiles) clear();
                }
            }
        }
        __syncthreads();
    }

    static constexpr int kRowLanes = 16;
    __device__ __forceinline__ float at(int x, int y, int e) const { return acc[x][y][e]; }
    __device__ __forceinline__ float4v four(int x, int y) const { return acc[x][y]; }
    __device__ __forceinline__ int row_of(int x) const { return wi + x * 16 + (lane & 15); }
    __device__ __forceinline__ int col_of(int y) const {
        return wj + (lane >> 4) * kRow + (kRow == 8 ? y * 4 : y * 16);
    }
};

template <class T, int MODE, int BM>
__global__ __launch_bounds__(256) void k_ced_logits(CeSide x, CeSide w, CeLogits l, int64_t tn,
                                                    int64_t tm, CeRows rows, CeScalars* scalars,
                                                    int* powers) {
    typedef CeDirect<T, false, false, BM> Tile;
    __shared__ __align__(16) char lds[Tile::kBytes];
    int64_t ti, tj;
    ce_place(xcd_order(blockIdx.x, gridDim.x), tm, tn, &ti, &tj);
    const int64_t i0 = ti * BM, j0 = tj * 64;
    Tile tile;
    tile.init();
    tile.run(lds, x, w, i0, 1, j0, 0, (x.cols + Tile::kInner - 1) / Tile::kInner, [](int) {});
    if constexpr (MODE == kCeLoss) {
        CeRowSums<Tile> sums;
        sums.init(tile, l, i0, x.rows, w.rows, 0);
        sums.template add<64, Tile::WGN>(tile, l, i0, j0, w.rows);
        sums.template store<BM, Tile::WGN>(tile, l, (float*)lds, i0, x.rows, tj);
    } else {
        CeFactor f;
        f.init(rows, sizeof(T) == 4, (double*)lds, (float*)lds + 64);
        if (blockIdx.x == 0 && threadIdx.x == 0) {
            scalars->ek = f.ek;
            scalars->mu = f.mu;
        }
        // Its rows' powers are the next launch's.
        const int64_t i = i0 + threadIdx.x;
        if (rows.powers && tj == 0 && threadIdx.x < BM && i < x.rows) powers[i] = f.power(rows, i);
        CeRowGrads<Tile> grads;
        grads.init(tile, l, i0, x.rows, w.rows, 0, [&](int64_t i) { return f.of(rows, i); });
        grads.template store<float, false, 64, Tile::WGN>(tile, l, i0, j0, w.rows);
    }
}

// Block `at` of a product of m rows, the inner axis of k values cut into `splits`:
// `group` tiles one below the other.
template <class T, bool TP, int BM>
__device__ __forceinline__ void ced_product(char* lds, const CeSide& p, const CeSide& q,
                                            const CeResult& w, int64_t at, int64_t blocks,
                                            int group, int splits, int64_t m, int64_t n, int64_t k,
                                            const CeScalars* sc) {
    CeDirect<T, TP, true, BM, sizeof(T) == 2> tile;
    const int64_t split = at / blocks, t = at % blocks, tn = (n + 63) / 64;
    const int64_t steps = (k + tile.kInner - 1) / tile.kInner;
    const int64_t i0 = t / tn * group * BM, j0 = t % tn * 64;
    const int64_t left = (m - i0 + BM - 1) / BM;
    const int e = sc->ek;
    const float mu = sc->mu;
    tile.init();
    tile.run(lds, p, q, i0, left < group ? (int)left : group, j0, split * steps / splits,
             (split + 1) * steps / splits, [&](int g) {
                 ce_store_tile<T>(tile, i0 + g * BM, j0, m, n, w,
                                  w.parts ? w.parts + split * m * w.ld : nullptr,
                                  [&](float v, int power) { return ce_unscale(v, mu, e + power); });
             });
}

// Three blocks a CU: 6 x 966 x 67682 float16 155 us, with two 188.
template <class T, int BM_DX, int BM_DW>
__global__ __launch_bounds__(256, 3) void k_ced_products(CeBoth b) {
    __shared__ __align__(16) char lds[CeDirect<T, true, true, 64, sizeof(T) == 2>::kBytes];
    // The product whose blocks take longer begins.
    const int64_t dx = b.dx_blocks * b.dx_splits, dw = b.dw_blocks * b.dw_splits;
    const bool dw_first = b.rows / b.dw_splits > b.classes / b.dx_splits;
    const int64_t at = blockIdx.x, first = dw_first ? dw : dx;
    if ((at < first) != dw_first)
        ced_product<T, false, BM_DX>(lds, b.g, b.w, b.dx, dw_first ? at - dw : at, b.dx_blocks,
                                     1, b.dx_splits, b.rows, b.cols, b.classes, b.scalars);
    else
        ced_product<T, true, BM_DW>(lds, b.g, b.x, b.dw, dw_first ? at : at - dx, b.dw_blocks,
                                    b.dw_group, b.dw_splits, b.classes, b.cols, b.rows, b.scalars);
}

template <class F>
static int ced_types(int32_t dtype, F&& f) {
    if (dtype == SPOPT_DTYPE_F32)
        f(float{});
    else if (dtype == SPOPT_DTYPE_F16)
        f(_Float16{});
    else
        f(__bf16{});
    SPOPT_LAUNCHED();
    return SPOPT_OK;
}

typedef std::integral_constant<int, 16> Rows16;
typedef std::integral_constant<int, 64> Rows64;

template <class F>
static void ced_rows(int tile, F&& f) {
    if (tile == 16)
        f(Rows16{});
    else
        f(Rows64{});
}

int ce_direct_loss(int32_t dtype, int tile, const CeSide& x, const CeSide& w, const CeLogits& l,
                   hipStream_t s) {
    return ced_types(dtype, [&](auto t) {
        ced_rows(tile, [&](auto bm) {
            const int64_t tm = ceil_div(x.rows, bm.value), tn = ceil_div(w.rows, 64);
            k_ced_logits<decltype(t), kCeLoss, bm.value>
                <<<(unsigned)(tm * tn), 256, 0, s>>>(x, w, l, tn, tm, CeRows{}, nullptr, nullptr);
        });
    });
}

int ce_direct_grad(int32_t dtype, int tile, const CeSide& x, const CeSide& w,
                   const CeLogits& l, const CeRows& rows, CeScalars* scalars, int* powers,
                   hipStream_t s) {
    return ced_types(dtype, [&](auto t) {
        ced_rows(tile, [&](auto bm) {
            const int64_t tm = ceil_div(x.rows, bm.value), tn = ceil_div(w.rows, 64);
            k_ced_logits<decltype(t), kCeGrad, bm.value>
                <<<(unsigned)(tm * tn), 256, 0, s>>>(x, w, l, tn, tm, rows, scalars, powers);
        });
    });
}

int ce_direct_products(int32_t dtype, const CeBoth& b, hipStream_t s) {
    const int64_t blocks = b.dx_blocks * b.dx_splits + b.dw_blocks * b.dw_splits;
    return ced_types(dtype, [&](auto t) {
        ced_rows(b.dx_tile, [&](auto bx) {
            ced_rows(b.dw_tile, [&](auto bw) {
                k_ced_products<decltype(t), bx.value, bw.value>
                    <<<(unsigned)blocks, 256, 0, s>>>(b);
            });
        });
    });
}

}  // namespace spopt
