// muon.hip - Newton-Schulz orthogonalisation of matrices and the Muon step.
//
// With X the r x c iterate (r <= c, the input transposed where it is taller
// than wide), one step is three products:
//   A = X X^T,   B = b A + c A A,   X <- a X + B X.
// The first two are P P^T with the inner axis adjacent in memory, which is what
// the matrix cores' operands take (A is symmetric); of their symmetric results
// the lower tiles are computed and mirrored.  For B X the inner axis runs along
// X's columns: its operand is turned as it is read from LDS.
//
// Types.  The operands are float16 and the sums float32.  float16 carries 11
// bits against bfloat16's 8 at the same rate; its range is met by X * 2^6, of
// which A * 2^12 follows without a factor, and B as it is: entries of B below
// float16's normal range are off by 2^-25 at most, which a X is not changed by
// (entries are bounded by the largest singular value, which the host checks).
// X is also carried in float32, for the a X term: in the directions of small
// singular values B is near zero, so that rounding errors of X come in through
// a X alone there, and grow by a factor of a in every step.  B's diagonal keeps
// float32's digits: as X's rows become orthonormal it nears b + c while the
// rest of B vanishes, and float16 alone would round it to 5e-4.
//
// Which X the diagonal meets.  With E the rounding of X to float16, B (X + E)
// is off by B E, which lies in B's range, that is in directions that X has.
// The diagonal times X in float32 in place of X + E takes diag E out of that:
// what is left is smaller where B is nearly diagonal, but of a matrix of low
// rank or with few rows that are not zero it lies in directions that X lacks,
// and each later step multiplies it by a.  So while steps follow that would,
// the diagonal's float16 part stays in the product and its remainder joins
// a X; in the last two steps (and of a single row, which lacks no direction)
// all of it joins a X.  Errors against 64 bits, relative to the result's norm,
// by 5 steps in an emulation of these roundings: rank 1 of 64 x 64 7e-4, 4 rows
// of 512 that are not zero 1.6e-3, Gaussian 128 x 128 1.2e-3.  With all of the
// diagonal beside a X throughout 9e-3, 3.8e-2 and 1.0e-3, only its remainder
// throughout 7e-4, 1.7e-3 and 1.5e-3.  The largest met are of matrices with 2
// or 3 rows (6e-3) and of constant ones, whose values all round alike (5e-3).
#include <math.h>

#include <type_traits>

#include "dense.hpp"

namespace spopt {

typedef _Float16 half4 __attribute__((ext_vector_type(4)));
typedef _Float16 half8 __attribute__((ext_vector_type(8)));
typedef float float4v __attribute__((ext_vector_type(4)));

constexpr int kTile = 64;                    // rows, columns and inner axis are padded to it
constexpr int kXExp = 6;
constexpr float kXScale = 1 << kXExp;
constexpr float kAScale = kXScale * kXScale; // 2^12
constexpr int kNormParts = 1024;             // partial sums of a matrix's norm, at most

// The matrix U that a call orthogonalises, formed as it is read.
template <class G>
struct Source {
    const G* g;
    const float* buf;  // the momentum after this step's update
    float mu;
    int kind;          // 0: g, 1: buf, 2: g + mu * buf
    __device__ __forceinline__ float at(int64_t i) const {
        if (kind == 0) return (float)g[i];
        if (kind == 1) return buf[i];
        return (float)g[i] + mu * buf[i];
    }
};

__device__ __forceinline__ double block_sum_d(double v, double* lds) {
#pragma unroll
    for (int off = kWave / 2; off; off >>= 1) v += __shfl_xor(v, off, kWave);
    if (lane_id() == 0) lds[threadIdx.x >> 6] = v;
    __syncthreads();
    double s = 0.;
    for (int i = 0; i < (int)(blockDim.x >> 6); ++i) s += lds[i];
    return s;
}

// buf <- mu * buf + g where the step keeps a momentum, and each block's share
// of sum(U^2), in double.  Block (x, y): slice x of matrix y, 8 values a
// thread at a time (matrices of odd sizes start anywhere).  HBM bounds it:
// 4096 x 4096 float32 13 us (5.0 TB/s), 2048 x 8192 with a momentum 30 us.
template <class G>
__global__ __launch_bounds__(256) void k_ns_norm(Source<G> u, float* buf, int64_t numel,
                                                 double* part) {
    __shared__ double lds[4];
    const int64_t base = (int64_t)blockIdx.y * numel;
    const G* g = u.g + base;
    double s = 0.;
    const int64_t whole = numel / 8 * 8;
    for (int64_t i = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 8; i < whole;
         i += (int64_t)gridDim.x * 256 * 8) {
        float v[8];
        load_v<G, 8>(g + i, v);
        if (u.kind != 0) {
            float b[8];
            load_v<float, 8>(buf + base + i, b);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                b[e] = u.mu * b[e] + v[e];
                v[e] = u.kind == 1 ? b[e] : v[e] + u.mu * b[e];
            }
            store_v<float, 8>(buf + base + i, b);
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) s += (double)v[e] * (double)v[e];
    }
    const int64_t i = whole + threadIdx.x;
    if (blockIdx.x == 0 && i < numel) {
        if (u.kind != 0) buf[base + i] = u.mu * buf[base + i] + (float)g[i];
        const double v = (double)u.at(base + i);
        s += v * v;
    }
    s = block_sum_d(s, lds);
    if (threadIdx.x == 0) part[(int64_t)blockIdx.y * kNormParts + blockIdx.x] = s;
}

// x * 2^6 / (norm + eps) for the norm's square: the scale as a power of two and
// a factor in (1, 2], as float32 alone would not hold every norm's reciprocal,
// nor float64 that of the smallest eps.
struct NormScale {
    int ex;
    float f;
    __device__ __forceinline__ NormScale(double sq, double eps) {
        f = (float)(1.0 / frexp(sqrt(sq) + eps, &ex));
        ex = kXExp - ex;
    }
    __device__ __forceinline__ float operator()(float x) const { return ldexpf(x, ex) * f; }
};

struct NsBuffers {
    _Float16* x[2];  // [batch][rp * cp]   X * 2^6, one step's and the next's
    float* x32;      // [batch][rp * cp]   X * 2^6
    _Float16* a16;   // [batch][rp * rp]   A * 2^12
    _Float16* b16;   // [batch][rp * rp]   B, its diagonal as ns_split says
    float* diag;     // [batch][rp]        B's diagonal but for what b16 holds of it
    double* part;    // [batch][kNormParts]
};

struct NsShape {
    int64_t batch, m, n;
    int r, c, rp, cp;
    bool flip;       // X is the input's transpose
};

// X0 = U / (|U| + eps) into the padded buffers, rows and columns beyond the
// matrix as zeros.  One 64 x 64 tile of X per block, through LDS where X is the
// input's transpose.  HBM bounds it: 4096 x 4096 float32 31 us (5.4 TB/s, part of
// it in the last-level cache); single values in place of fours took 36 us, and
// 12.8 in place of 8.6 us at 1024 x 1024.
template <class G>
__global__ __launch_bounds__(256) void k_ns_init(Source<G> u, NsBuffers w, NsShape sh, int parts,
                                                 double eps) {
    __shared__ double lds[4];
    __shared__ float tile[kTile][kTile + 1];
    const int64_t z = blockIdx.z;
    const int i0 = blockIdx.y * kTile, j0 = blockIdx.x * kTile;
    const int q = (threadIdx.x & 15) * 4, k = threadIdx.x >> 4;
    const int64_t base = z * sh.m * sh.n;
    // Four adjacent values of four of the input's rows (those of X, or X's
    // columns) are asked for before anything is waited for.
    const int lines = sh.flip ? sh.c : sh.r, width = sh.flip ? sh.r : sh.c;
    const int line0 = sh.flip ? j0 : i0, first = (sh.flip ? i0 : j0) + q;
    const bool quad = first + 4 <= width;
    float v[4][4] = {}, b[4][4];
    auto read = [&](const auto* from, float (&x)[4][4]) {
        typedef std::remove_cv_t<std::remove_reference_t<decltype(*from)>> E;
#pragma unroll
        for (int t = 0; t < 4; ++t) {
            const int line = line0 + 16 * t + k;
            // Lines past the matrix read its last one, and count as zeros below.
            const E* p = from + base + (int64_t)(line < lines ? line : lines - 1) * width;
            if (quad) {
                load_v<E, 4>(p + first, x[t]);
            } else {
#pragma unroll
                for (int e = 0; e < 4; ++e) x[t][e] = (float)p[first + e < width ? first + e : 0];
            }
        }
    };
    if (u.kind != 1) read(u.g, v);
    if (u.kind != 0) {
        read(u.buf, b);
#pragma unroll
        for (int t = 0; t < 4; ++t)
#pragma unroll
            for (int e = 0; e < 4; ++e)
                v[t][e] = u.kind == 1 ? b[t][e] : v[t][e] + u.mu * b[t][e];
    }
    double sq = 0.;
    for (int t = threadIdx.x; t < parts; t += 256) sq += w.part[z * kNormParts + t];
    const NormScale scale(block_sum_d(sq, lds), eps);
#pragma unroll
    for (int t = 0; t < 4; ++t)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const bool in = line0 + 16 * t + k < lines && first + e < width;
            v[t][e] = in ? scale(v[t][e]) : 0.f;
            if (sh.flip) tile[q + e][16 * t + k] = v[t][e];
        }
    if (sh.flip) {
        __syncthreads();
#pragma unroll
        for (int t = 0; t < 4; ++t)
#pragma unroll
            for (int e = 0; e < 4; ++e) v[t][e] = tile[16 * t + k][q + e];
    }
    const int64_t xb = z * sh.rp * sh.cp;
#pragma unroll
    for (int t = 0; t < 4; ++t) {
        const int64_t o = xb + (int64_t)(i0 + 16 * t + k) * sh.cp + j0 + q;
        store_v<_Float16, 4>(w.x[0] + o, v[t]);
        store_v<float, 4>(w.x32 + o, v[t]);
    }
}

enum : int { kGram = 0, kPoly = 1, kNext = 2, kOut = 3, kParam32 = 4, kParam16 = 5 };

// Whether it does, `left` steps before the last, for X of `rows` rows.
__host__ __device__ __forceinline__ int ns_split(int left, int rows) {
    return left >= 2 && rows > 1;
}

struct NsStep {
    float a, b, c;
    int split;       // whether the product holds the float16 part of B's diagonal
    void* out;       // kOut: bfloat16; kParam*: the weight
    float keep, move;  // kParam*: p <- keep * p - move * X
};

// Waits until at most N of this wave's loads (into LDS too) are on their way;
// wait_stage also for its reads of LDS, and for the block's other waves.
template <int N>
__device__ __forceinline__ void wait_loads() {
    asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
}
template <int N>
__device__ __forceinline__ void wait_stage() {
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(N) : "memory");
}

// 16 bytes a lane straight into LDS, the wave's 64 at adjacent places from `to`
// (the same for the whole wave).  In assembly, as the compiler would wait for
// every load that writes LDS before each transposing read of it, also of
// another stage; wait_stage counts them instead.  No register is written but
// m0: reserved, so that the compiler allocates nothing to it (and warns where it
// is listed as clobbered), and no instruction that it makes of this file reads
// it.
__device__ __forceinline__ void load_lds16(const _Float16* from, _Float16* to) {
    const uint32_t m0 = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) void*)to;
    asm volatile("s_mov_b32 m0, %1\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, off" ::"v"(from),
                 "s"(m0)
                 : "memory");
}

__device__ __forceinline__ half4 read_turned(const _Float16* p) {
    typedef short short4v __attribute__((ext_vector_type(4)));
    return __builtin_bit_cast(half4, __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                                         (__attribute__((address_space(3))) short4v*)p));
}

// Where row `row` of BN values has its 32-byte part u in LDS: at u ^ turn_q(row).
// Rows r .. r + 3 and r + 8 .. r + 11 (or r + 16 .. r + 19) then lie in different
// eighths of the 256 bytes that LDS gives a cycle.
template <int BN>
__device__ __forceinline__ int turn_q(int row) {
    const int far = (row >> 3 ^ row >> 4) & 1;
    return BN % 128 == 0 ? (row & 3) | far << 2 : (row >> 1 & 1) | far << 1;
}

template <int MODE>
struct OutType {
    typedef __bf16 type;
};
template <>
struct OutType<kParam32> {
    typedef float type;
};

// The last step's values to where they go: the result, or the weight's update.
template <int MODE, int V>
__device__ __forceinline__ void write_out(typename OutType<MODE>::type* d, const float (&v)[V],
                                          const NsStep& st) {
    typedef typename OutType<MODE>::type O;
    if constexpr (MODE == kOut) {
        store_v<O, V>(d, v);
    } else {
        float p[V];
        load_v<O, V>(d, p);
#pragma unroll
        for (int e = 0; e < V; ++e) p[e] = st.keep * p[e] - st.move * v[e];
        store_v<O, V>(d, p);
    }
}

// A block's tile of BM x BN values, shared out to WGM x WGN waves, and how many
// stages of the inner axis LDS holds.
template <int BM_, int BN_, int WGM_, int WGN_, int STAGES_>
struct Tiling {
    static constexpr int BM = BM_, BN = BN_, WGM = WGM_, WGN = WGN_, STAGES = STAGES_;
    static constexpr int kThreads = WGM * WGN * 64;
    static constexpr int kStage = (BM + BN) * kTile;  // float16 values of one inner step
};

// Order of the tiles: blocks go to the 8 XCDs in turn, so block b takes place
// b / 8 of the (b % 8)th eighth, and each XCD's L2 sees neighbouring tiles.
__device__ __forceinline__ int64_t xcd_order(int64_t b, int64_t n) {
    const int64_t q = n / 8, rem = n % 8, x = b % 8;
    return x * q + (x < rem ? x : rem) + b / 8;
}

// One product P Q^T, tile by tile, and what its result is for:
//   kGram  A = X X^T           kPoly  B = b A + c A A     (lower tiles, mirrored)
//   kNext  X <- a X + B X      kOut / kParam*  the last step's X, written out
//
// The inner axis goes through LDS 64 values at a time: the next stages' rows
// are on their way straight into LDS while this one is multiplied.  Two stages
// are enough where several blocks share a CU or the tile is large; a block
// alone on its CU takes four, as operands that the launch before wrote come
// from beyond the XCD's own L2.  A row's eight 16-byte chunks lie in an order turned by the row
// (chunk c at c ^ (row & 7)): the 16 rows that a matrix instruction's operand
// takes then meet every bank equally, without padding, which the loads into
// LDS could not leave.
//
// Which of the tile's rows lies in which row of LDS is chosen for the end: with
// Q's rows as the matrix instruction's first operand, lane l holds, of rows
// FM (l % 16) .. + FM - 1 of its wave's part (FM adjacent ones, from FM
// instructions), 8 adjacent columns of every 32 (4 of every 16 where a wave has
// an odd number of 16-column parts).  Rows of the result are written 16 bytes
// of float16 at a time and columns (the mirrored half, X^T) up to 8 values at a
// time, with no exchange between lanes.
//
// Measured at 4096 x 4096 (what the product alone is worth at the 1.1 PFLOP/s
// that the library's float16 product of this size reaches): A 72 to 81 us and
// A A 75 to 85 us in 253 tiles of 192 (62 us), B X 131 to 147 us in 256 tiles of
// 256 (125 us; the 10 bytes a value of its epilogue are another 33 us of HBM
// time).  LDS reads meet no bank conflict; matrix instructions are issued 45%
// of the time.  The 256 tile's accumulators leave its epilogues short of
// registers: 45 of a lane go to scratch and back in kPoly, 10 to 16 in the last
// step's forms, none in kNext.
template <int MODE, class T>
__global__ __launch_bounds__(T::kThreads) void k_ns_gemm(NsBuffers w, NsShape sh, NsStep st,
                                                         int from, int tiles) {
    constexpr int BM = T::BM, BN = T::BN, WM = BM / T::WGM, WN = BN / T::WGN;
    constexpr int FM = WM / 16, FN = WN / 16, kWaves = T::WGM * T::WGN;
    constexpr int kRow = MODE >= kNext || FN % 2 ? 4 : 8;        // columns of a row's store
    constexpr int kCol = FM % 8 == 0 ? 8 : FM % 4 == 0 ? 4 : FM % 2 ? 1 : 2;  // rows of a column's store
    extern __shared__ __align__(16) char lds_raw[];
    _Float16* const lds = (_Float16*)lds_raw;
    const int64_t t = xcd_order(blockIdx.x, gridDim.x);
    const int64_t z = t / tiles;
    const int tile = (int)(t % tiles);
    const int64_t nx = (int64_t)sh.rp * sh.cp, na = (int64_t)sh.rp * sh.rp;
    constexpr bool kTurn = MODE >= kNext;  // Q's inner axis runs along its rows
    const _Float16 *p, *q;
    int k_len = sh.rp, j_len = sh.rp, ti, tj;
    if (MODE == kGram) {
        p = q = w.x[from] + z * nx;
        k_len = sh.cp;
    } else if (MODE == kPoly) {
        p = q = w.a16 + z * na;
    } else {
        p = w.b16 + z * na;
        q = w.x[from] + z * nx;
        j_len = sh.cp;
    }
    if (MODE <= kPoly) {
        // Row ti holds tiles 0 .. ti of the lower triangle.
        ti = (int)((sqrtf(8.f * (float)tile + 1.f) - 1.f) * 0.5f);
        while ((int64_t)(ti + 1) * (ti + 2) / 2 <= tile) ++ti;
        while ((int64_t)ti * (ti + 1) / 2 > tile) --ti;
        tj = tile - (int)((int64_t)ti * (ti + 1) / 2);
    } else {
        // Four rows of tiles at a time, column by column.
        const int tr = (sh.rp + BM - 1) / BM, tc = (sh.cp + BN - 1) / BN;
        const int band = tile / (4 * tc), in = tile % (4 * tc);
        const int rows = tr - 4 * band < 4 ? tr - 4 * band : 4;
        ti = 4 * band + in % rows;
        tj = in / rows;
    }
    const int i0 = ti * BM, j0 = tj * BN;
    const int lane = lane_id(), wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wi = (wv / T::WGN) * WM, wj = (wv % T::WGN) * WN;

    // A wave's load brings 64 chunks of 16 bytes to adjacent places in LDS.  Of
    // an operand with its inner axis adjacent these are 8 rows of 8 chunks; rows
    // past its end repeat the last one, and their products are not written.
    constexpr int kLoadsP = BM / 8 / kWaves, kLoadsQ = BN / 8 / kWaves;
    constexpr int kLoads = kLoadsP + kLoadsQ;
    static_assert(BM % (8 * kWaves) == 0 && BN % (8 * kWaves) == 0, "rows share out evenly");
    const _Float16 *src_p[kLoadsP], *src_q[kLoadsQ];
    const int ch8 = ((lane & 7) ^ (lane >> 3)) * 8;
#pragma unroll
    for (int l = 0; l < kLoadsP; ++l) {
        const int row = (l * kWaves + wv) * 8 + (lane >> 3), in = row % WM;
        const int r = i0 + row - in + (in & 15) * FM + (in >> 4);
        src_p[l] = p + (int64_t)(r < sh.rp ? r : sh.rp - 1) * k_len + ch8;
    }
#pragma unroll
    for (int l = 0; l < kLoadsQ; ++l) {
        if (kTurn) {
            // 64 rows (the inner axis) of BN / 8 chunks, those of 16 columns
            // at place u ^ turn_q(row): see turned() below.
            const int at = (l * kWaves + wv) * 64 + lane;
            const int row = at / (BN / 8), slot = at % (BN / 8);
            const int j = j0 + (((slot >> 1) ^ turn_q<BN>(row)) * 2 + (slot & 1)) * 8;
            src_q[l] = q + (int64_t)row * sh.cp + (j < sh.cp ? j : sh.cp - 8);
        } else {
            const int at = (l * kWaves + wv) * 8 + (lane >> 3), in = at & (4 * kRow - 1);
            const int r = j0 + at - in + ((in & 12) >> 2) * kRow + (in >> 4) * 4 + (in & 3);
            src_q[l] = q + (int64_t)(r < j_len ? r : j_len - 1) * k_len + ch8;
        }
    }
    const int64_t step_q = kTurn ? (int64_t)sh.cp : 1;
    auto stage = [&](int buf, int k0) {
        _Float16* const to = lds + buf * T::kStage;
#pragma unroll
        for (int l = 0; l < kLoadsP; ++l) load_lds16(src_p[l] + k0, to + (l * kWaves + wv) * 512);
#pragma unroll
        for (int l = 0; l < kLoadsQ; ++l)
            load_lds16(src_q[l] + k0 * step_q, to + BM * kTile + (l * kWaves + wv) * 512);
    };
    // Q's operand where it has to be turned: a transposing read gives each of 16
    // lanes one column's values of 4 rows, lane i naming 4 columns of row i / 4.
    // The rows' 32-byte parts are laid out so that the 8 rows of 32 lanes meet
    // different banks of the 64.
    int turn[FN];
#pragma unroll
    for (int y = 0; y < FN; ++y) {
        const int row = (lane >> 4) * 8 + ((lane & 15) >> 2);  // and 4, 32, 36 on: turned alike
        turn[y] = row * BN + ((wj / 16 + y) ^ turn_q<BN>(row)) * 16 + (lane & 3) * 4;
    }
    auto turned = [&](const _Float16* lq, int kk, int y) {
        const half4 a = read_turned(lq + turn[y] + kk * 32 * BN);
        const half4 b = read_turned(lq + turn[y] + (kk * 32 + 4) * BN);
        return __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7);
    };

    float4v acc[FM][FN] = {};
    const int steps = k_len / kTile;
    // Past the end the last step is brought again, so that every wait counts
    // the same loads; nothing reads it.
    auto at = [&](int k) { return (k < steps ? k : steps - 1) * kTile; };
    half8 fa0[FM], fb0[FN], fa1[FM], fb1[FN];
    // Half kk of a stage's operands into registers.
    auto operands = [&](int buf, int kk, half8 (&fa)[FM], half8 (&fb)[FN]) {
        const _Float16* lp = lds + buf * T::kStage + (wi + (lane & 15)) * kTile;
        const _Float16* lq = lds + buf * T::kStage + BM * kTile;
        const int ch = ((kk * 4 + (lane >> 4)) ^ (lane & 7)) * 8;
#pragma unroll
        for (int y = 0; y < FN; ++y)
            fb[y] = kTurn ? turned(lq, kk, y)
                              : *(const half8*)(lq + (wj + y * 16 + (lane & 15)) * kTile + ch);
#pragma unroll
        for (int x = 0; x < FM; ++x) fa[x] = *(const half8*)(lp + x * 16 * kTile + ch);
    };
    auto multiply = [&](half8 (&fa)[FM], half8 (&fb)[FN]) {
#pragma unroll
        for (int x = 0; x < FM; ++x)
#pragma unroll
            for (int y = 0; y < FN; ++y)
                acc[x][y] = __builtin_amdgcn_mfma_f32_16x16x32_f16(fb[y], fa[x],
                                                                   acc[x][y], 0, 0, 0);
    };
    int buf = 0;
    if constexpr (BM < 192) {
#pragma unroll
        for (int k = 0; k < T::STAGES - 1; ++k) stage(k, at(k));
        for (int k = 0; k < steps; ++k) {
            // This stage's loads have landed in every wave, and every wave has
            // read the stage before, whose place the next loads take.
            wait_stage<(T::STAGES - 2) * kLoads>();
            stage(buf == 0 ? T::STAGES - 1 : buf - 1, at(k + T::STAGES - 1));
            operands(buf, 0, fa0, fb0);
            multiply(fa0, fb0);
            operands(buf, 1, fa1, fb1);
            multiply(fa1, fb1);
            buf = buf + 1 == T::STAGES ? 0 : buf + 1;
        }
    } else {
        // Large tiles read each half's operands while the half before is
        // multiplied, a read every few products: 4096 x 4096 1420 against 1457
        // us, timed in turn.  Small ones lose by the longer start: 1024 x 512 by 16 267 to 257.
        constexpr int kReads = FM + (kTurn ? 2 : 1) * FN, kPer = FM * FN / kReads;
        auto weave = [&] {
#pragma unroll
            for (int g = 0; g < kReads; ++g) {
                __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);     // a read of LDS
                __builtin_amdgcn_sched_group_barrier(0x008, kPer, 0);  // matrix instructions
            }
            __builtin_amdgcn_sched_group_barrier(0x008, FM * FN - kPer * kReads, 0);
        };
#pragma unroll
        for (int k = 0; k < T::STAGES; ++k) stage(k, at(k));
        wait_stage<(T::STAGES - 1) * kLoads>();
        operands(0, 0, fa0, fb0);
        for (int k = 0; k < steps; ++k) {
            operands(buf, 1, fa1, fb1);
            multiply(fa0, fb0);
            weave();
            // The next stage's loads have landed in every wave, and every wave
            // has read this one, whose place the loads after them take.
            wait_stage<(T::STAGES - 2) * kLoads>();
            stage(buf, at(k + T::STAGES));
            buf = buf + 1 == T::STAGES ? 0 : buf + 1;
            operands(buf, 0, fa0, fb0);
            multiply(fa1, fb1);
            weave();
        }
    }
    wait_loads<0>();
    // The tile's results, row by row and then, from the same registers, column
    // by column.  `whole`: no part of the tile lies past the matrix.
    const int ib = i0 + wi + (lane & 15) * FM, jb = j0 + wj + (lane >> 4) * kRow;
    auto finish = [&](auto whole) {
        constexpr bool kWhole = decltype(whole)::value;
        const int i_end = MODE >= kOut ? sh.r : sh.rp;
        const int j_end = MODE >= kOut ? sh.c : j_len;
        const int64_t ob = z * sh.m * sh.n;
        typedef typename OutType<MODE>::type O;
        O* const out = (O*)st.out + ob;
#pragma unroll
        for (int x = 0; x < FM; ++x)
#pragma unroll
            for (int y = 0; y < FN; y += kRow / 4) {
                const int i = ib + x, j = jb + y * 16;
                if (!kWhole && (i >= sh.rp || j >= j_len)) continue;
                float v[kRow];
#pragma unroll
                for (int e = 0; e < kRow; ++e) v[e] = acc[x][y + e / 4][e & 3];
                if (MODE == kGram || MODE == kPoly) {
                    const int64_t o = z * na + (int64_t)i * sh.rp + j;
                    float a8[kRow];
                    if (MODE == kPoly) load_v<_Float16, kRow>(w.a16 + o, a8);
#pragma unroll
                    for (int e = 0; e < kRow; ++e)
                        if (MODE == kPoly) {
                            v[e] = st.b / kAScale * a8[e] + st.c / (kAScale * kAScale) * v[e];
                            if (ti == tj && i == j + e) {
                                const float in = st.split ? (float)(_Float16)v[e] : 0.f;
                                w.diag[z * sh.rp + i] = v[e] - in;
                                v[e] = in;
                            }
                        }
                    store_v<_Float16, kRow>((MODE == kGram ? w.a16 : w.b16) + o, v);
                } else {
                    const int64_t o = z * nx + (int64_t)i * sh.cp + j;
                    float x0[kRow];
                    load_v<float, kRow>(w.x32 + o, x0);
                    const float a = st.a + w.diag[z * sh.rp + i];
                    // X * 2^6 of the next step
#pragma unroll
                    for (int e = 0; e < kRow; ++e) v[e] = a * x0[e] + v[e];
                    if (MODE == kNext) {
                        store_v<float, kRow>(w.x32 + o, v);
                        store_v<_Float16, kRow>(w.x[from ^ 1] + o, v);
                        continue;
                    }
#pragma unroll
                    for (int e = 0; e < kRow; ++e) v[e] /= kXScale;
                    if (!sh.flip) {
                        O* d = out + (int64_t)i * sh.c + j;
                        if (kWhole || (i < i_end && j + kRow <= j_end)) {
                            write_out<MODE, kRow>(d, v, st);
                        } else if (i < i_end) {
                            for (int e = 0; e < kRow; ++e)
                                if (j + e < j_end) {
                                    const float one[1] = {v[e]};
                                    write_out<MODE, 1>(d + e, one, st);
                                }
                        }
                    }
                }
#pragma unroll
                for (int e = 0; e < kRow; ++e) acc[x][y + e / 4][e & 3] = v[e];
                // Loads of at most four such parts at once: all of them would spill.
                if ((x * FN + y) % (4 * kRow / 4) == 0) __builtin_amdgcn_sched_barrier(0);
            }
        if ((MODE <= kPoly && ti == tj) || MODE == kNext || (MODE >= kOut && !sh.flip)) return;
#pragma unroll
        for (int y = 0; y < FN; ++y)
#pragma unroll
            for (int e = 0; e < 4; ++e)
#pragma unroll
                for (int x = 0; x < FM; x += kCol) {
                    const int i = ib + x;
                    const int j = kRow == 8 ? jb + (y & ~1) * 16 + (y & 1) * 4 + e
                                            : jb + y * 16 + e;
                    if (!kWhole && (i >= sh.rp || j >= j_end)) continue;
                    float v[kCol];
#pragma unroll
                    for (int f = 0; f < kCol; ++f) v[f] = acc[x + f][y][e];
                    if (MODE <= kPoly)
                        store_v<_Float16, kCol>(
                            (MODE == kGram ? w.a16 : w.b16) + z * na + (int64_t)j * sh.rp + i, v);
                    else if (kWhole || i + kCol <= i_end)
                        write_out<MODE, kCol>(out + (int64_t)j * sh.r + i, v, st);
                    else
                        for (int f = 0; f < kCol; ++f)
                            if (i + f < i_end) {
                                const float one[1] = {v[f]};
                                write_out<MODE, 1>(out + (int64_t)j * sh.r + i + f, one, st);
                            }
                }
    };
    if (i0 + BM <= (MODE >= kOut ? sh.r : sh.rp) && j0 + BN <= (MODE >= kOut ? sh.c : j_len))
        finish(std::true_type{});
    else
        finish(std::false_type{});
}

// -------------------------------------- matrices of up to 128 rows or columns ---

// Up to 16 R rows (R = 4 or 8) and 16 W FN adjacent columns of X, held by a
// block of W waves: in registers in float32 (wave v has all rows of 16 FN
// columns) and in LDS in float16, with an R x R square (A, then B) beside it.
//
// LDS rows (X's of 16 W FN values, the square's of 128) are laid out with chunk
// c of 8 values of row i at c ^ turn_of(i): the 8 rows of two chunks that LDS
// gives in a cycle, and the 8 rows of a transposing read, lie in different
// parts of its 256 bytes.
__device__ __forceinline__ int turn_of(int row) {
    return (((row & 7) ^ ((row >> 1) & 4)) << 1) | ((row >> 3) & 1);  // of row % 16
}

template <int R, int FN, int W>
struct Panel {
    static constexpr int kX = 16 * W * FN, kA = 128;
    static constexpr int FA = R / 4, FB = 4 * R / W;  // a wave's part of the square
    static constexpr int kBytes = 16 * R * ((kX + kA) * 2 + 4);
    // Of 16 waves' square parts the 6 above the diagonal are mirrored ones.
    static constexpr bool kMirror = W == 16;
    _Float16 *lx, *la;
    float* diag;          // B's diagonal but for what `la` holds of it
    int lane, l15, g4, ft, wj, wr, wc;
    uint32_t di, dj;      // strides of X's rows and columns in the input
    int rows, cols;       // of the input's, from this panel's first column on
    bool by_four;         // four adjacent columns lie together in the input

    __device__ __forceinline__ Panel(char* lds, const NsShape& sh, int first_col)
        : lx((_Float16*)lds),
          la((_Float16*)lds + 16 * R * kX),
          diag((float*)(lds + 16 * R * (kX + kA) * 2)) {
        const int wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
        wj = wv * 16 * FN;
        wr = wv / (W / 4);
        wc = wv % (W / 4);
        set_lane(lane_id());
        di = sh.flip ? 1 : sh.c;
        dj = sh.flip ? sh.r : 1;
        rows = sh.r;
        cols = sh.c - first_col;
        by_four = !sh.flip && sh.c % 4 == 0;
    }
    __device__ __forceinline__ void set_lane(int l) {
        lane = l;
        l15 = l & 15;
        g4 = l >> 4;
        ft = turn_of(l15);
    }
    // Has the places in LDS worked out anew from here on: kept over a loop they
    // would not fit the registers.
    __device__ __forceinline__ void forget_places() {
        int l = lane;
        asm volatile("" : "+v"(l));
        set_lane(l);
    }
    __device__ __forceinline__ bool in_square() const { return !kMirror || wc <= wr; }

    // Value e of part (x, y): row 16 x + l15, column wj + 16 y + 4 g4 + e; where
    // it lies in the input (within 2^32 values of the panel's first).
    __device__ __forceinline__ uint32_t index(int x, int y, int e, bool* in) const {
        const int i = 16 * x + l15, j = wj + 16 * y + 4 * g4 + e;
        *in = i < rows && j < cols;
        return *in ? (uint32_t)i * di + (uint32_t)j * dj : 0u;
    }
    template <bool FOUR, class E>
    __device__ __forceinline__ void read_row(const E* from, int x, float4v (&v)[FN]) const {
        bool in;
#pragma unroll
        for (int y = 0; y < FN; ++y) {
            if constexpr (FOUR) {
                float q[4];
                load_v<E, 4>(from + index(x, y, 0, &in), q);
#pragma unroll
                for (int e = 0; e < 4; ++e) v[y][e] = in ? q[e] : 0.f;
            } else {
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float q = (float)from[index(x, y, e, &in)];
                    v[y][e] = in ? q : 0.f;
                }
            }
        }
    }
    // U of the panel into `xv`: g, buf or g + mu * buf (kind 0, 1, 2), where
    // `move` is set with buf <- mu * buf + g before.
    template <bool FOUR, class E>
    __device__ __forceinline__ void read_u(const E* g, float* buf, float mu, int kind, bool move,
                                           float4v (&xv)[R][FN]) const {
        // One row of parts at a time: all in flight would need too many registers.
#pragma unroll
        for (int x = 0; x < R; ++x) {
            read_row<FOUR>(g, x, xv[x]);
            __builtin_amdgcn_sched_barrier(0);
        }
        if (kind == 0) return;
#pragma unroll
        for (int x = 0; x < R; ++x) {
            float4v b[FN];
            read_row<FOUR>(buf, x, b);
#pragma unroll
            for (int y = 0; y < FN; ++y) {
                if (move) b[y] = mu * b[y] + xv[x][y];
                xv[x][y] = kind == 1 ? b[y] : xv[x][y] + mu * b[y];
                if (!move) continue;
                bool in;
                if constexpr (FOUR) {
                    const uint32_t o = index(x, y, 0, &in);
                    const float q[4] = {b[y][0], b[y][1], b[y][2], b[y][3]};
                    if (in) store_v<float, 4>(buf + o, q);
                } else {
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const uint32_t o = index(x, y, e, &in);
                        if (in) buf[o] = b[y][e];
                    }
                }
            }
        }
    }
    __device__ __forceinline__ void read_u(const void* g, bool bf16, int64_t base, float* buf,
                                           float mu, int kind, bool move,
                                           float4v (&xv)[R][FN]) const {
        float* const b = kind ? buf + base : nullptr;
        if (by_four) {
            if (bf16)
                read_u<true>((const __bf16*)g + base, b, mu, kind, move, xv);
            else
                read_u<true>((const float*)g + base, b, mu, kind, move, xv);
        } else {
            if (bf16)
                read_u<false>((const __bf16*)g + base, b, mu, kind, move, xv);
            else
                read_u<false>((const float*)g + base, b, mu, kind, move, xv);
        }
    }
    __device__ __forceinline__ void normalise(double sq, double eps, float4v (&xv)[R][FN]) const {
        const NormScale scale(sq, eps);
#pragma unroll
        for (int x = 0; x < R; ++x)
#pragma unroll
            for (int y = 0; y < FN; ++y)
#pragma unroll
                for (int e = 0; e < 4; ++e) xv[x][y][e] = scale(xv[x][y][e]);
    }
    // 4 adjacent values of row i (i % 16 == l15) from column j on.
    __device__ __forceinline__ void put(_Float16* l, int width, int i, int j, float4v v) const {
        half4 h;
#pragma unroll
        for (int e = 0; e < 4; ++e) h[e] = (_Float16)v[e];
        *(half4*)(l + i * width + (((j >> 3) ^ ft) << 3) + (j & 7)) = h;
    }
    __device__ __forceinline__ void put_x(const float4v (&xv)[R][FN]) const {
#pragma unroll
        for (int x = 0; x < R; ++x)
#pragma unroll
            for (int y = 0; y < FN; ++y) put(lx, kX, 16 * x + l15, wj + 16 * y + 4 * g4, xv[x][y]);
    }
    __device__ __forceinline__ void put_square(const float4v (&v)[FA][FB]) const {
#pragma unroll
        for (int x = 0; x < FA; ++x)
#pragma unroll
            for (int y = 0; y < FB; ++y) {
                const int i = 16 * (FA * wr + x) + l15, j = 16 * (FB * wc + y) + 4 * g4;
                put(la, kA, i, j, v[x][y]);
                if (kMirror && wc < wr)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        la[(j + e) * kA + (((i >> 3) ^ turn_of(j + e)) << 3) + (i & 7)] =
                            (_Float16)v[x][y][e];
            }
    }
    // Values 8 chunk .. + 7 of row i (i % 16 == l15).
    __device__ __forceinline__ half8 rows8(const _Float16* l, int width, int i, int chunk) const {
        return *(const half8*)(l + i * width + ((chunk ^ ft) << 3));
    }
    // acc += the wave's part of P P^T, P the rows of `l`, over 32 k32 columns.
    __device__ __forceinline__ void square(const _Float16* l, int width, int k32,
                                           float4v (&acc)[FA][FB]) const {
        half8 fa[2][FA], fb[2][FB];
        auto operands = [&](int k, int q) {
#pragma unroll
            for (int x = 0; x < FA; ++x)
                fa[q][x] = rows8(l, width, 16 * (FA * wr + x) + l15, 4 * k + g4);
#pragma unroll
            for (int y = 0; y < FB; ++y)
                fb[q][y] = rows8(l, width, 16 * (FB * wc + y) + l15, 4 * k + g4);
        };
        auto multiply = [&](int q) {
#pragma unroll
            for (int x = 0; x < FA; ++x)
#pragma unroll
                for (int y = 0; y < FB; ++y)
                    acc[x][y] = __builtin_amdgcn_mfma_f32_16x16x32_f16(fb[q][y], fa[q][x],
                                                                       acc[x][y], 0, 0, 0);
        };
        if constexpr (W == 8) {
            // The next operands are asked for before these are used (k32 is
            // even); 16 waves have no registers for it, but each other.
            operands(0, 0);
            for (int k = 0; k < k32; k += 2) {
                operands(k + 1, 1);
                multiply(0);
                operands(k + 2 < k32 ? k + 2 : 0, 0);
                multiply(1);
            }
        } else {
            for (int k = 0; k < k32; ++k) {
                operands(k, 0);
                multiply(0);
            }
        }
    }
    // From A * 2^12 in `ga` and, as float16, in LDS: B into LDS, its diagonal as
    // `split` (ns_split) says.
    __device__ __forceinline__ void polynomial(const float4v (&ga)[FA][FB], const NsStep& st,
                                               bool split) const {
        float4v gb[FA][FB] = {};
        if (in_square()) {
            square(la, kA, R / 2, gb);
#pragma unroll
            for (int x = 0; x < FA; ++x)
#pragma unroll
                for (int y = 0; y < FB; ++y)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        // A as the square was taken of it: its rounding then moves
                        // both terms, which nearly cancel.
                        gb[x][y][e] = (float)(_Float16)ga[x][y][e] * (st.b / kAScale) +
                                      gb[x][y][e] * (st.c / (kAScale * kAScale));
                    }
#pragma unroll
            for (int x = 0; x < FA; ++x)
#pragma unroll
                for (int y = 0; y < FB; ++y) {
                    if (FA * wr + x != FB * wc + y) continue;
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        if (l15 == 4 * g4 + e) {
                            const float in = split ? (float)(_Float16)gb[x][y][e] : 0.f;
                            diag[16 * (FA * wr + x) + l15] = gb[x][y][e] - in;
                            gb[x][y][e] = in;
                        }
                }
        }
        __syncthreads();
        if (in_square()) put_square(gb);
        __syncthreads();
    }
    // X <- a X + B X: the accumulators start at a X and `diag` X.
    __device__ __forceinline__ void next(float a, float4v (&xv)[R][FN]) const {
#pragma unroll
        for (int x = 0; x < R; ++x) {
            const float f = a + diag[16 * x + l15];
#pragma unroll
            for (int y = 0; y < FN; ++y) xv[x][y] *= f;
        }
#pragma unroll
        for (int kk = 0; kk < R / 2; ++kk) {
            half8 fa[R], fb[FN];
#pragma unroll
            for (int y = 0; y < FN; ++y) {
                const int j = wj + 16 * y + 4 * (lane & 3), i = kk * 32 + g4 * 8 + (l15 >> 2);
                half4 h[2];
#pragma unroll
                for (int q = 0; q < 2; ++q)
                    h[q] = read_turned(lx + (i + 4 * q) * kX +
                                       (((j >> 3) ^ turn_of(i + 4 * q)) << 3) + (j & 7));
                fb[y] = __builtin_shufflevector(h[0], h[1], 0, 1, 2, 3, 4, 5, 6, 7);
            }
#pragma unroll
            for (int x = 0; x < R; ++x) fa[x] = rows8(la, kA, 16 * x + l15, 4 * kk + g4);
#pragma unroll
            for (int x = 0; x < R; ++x)
#pragma unroll
                for (int y = 0; y < FN; ++y)
                    xv[x][y] = __builtin_amdgcn_mfma_f32_16x16x32_f16(fb[y], fa[x], xv[x][y], 0, 0,
                                                                      0);
        }
    }
    template <int MODE, bool FOUR>
    __device__ __forceinline__ void write_as(int64_t base, const NsStep& st,
                                             float4v (&xv)[R][FN]) const {
        typedef typename OutType<MODE>::type O;
        O* const out = (O*)st.out + base;
#pragma unroll
        for (int x = 0; x < R; ++x) {
#pragma unroll
            for (int y = 0; y < FN; ++y) {
                bool in;
                xv[x][y] *= 1.f / kXScale;
                if constexpr (FOUR) {
                    const uint32_t o = index(x, y, 0, &in);
                    const float q[4] = {xv[x][y][0], xv[x][y][1], xv[x][y][2], xv[x][y][3]};
                    if (in) write_out<MODE, 4>(out + o, q, st);
                } else {
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const uint32_t o = index(x, y, e, &in);
                        const float q[1] = {xv[x][y][e]};
                        if (in) write_out<MODE, 1>(out + o, q, st);
                    }
                }
            }
            __builtin_amdgcn_sched_barrier(0);
        }
    }
    template <int MODE>
    __device__ __forceinline__ void write_as(int64_t base, const NsStep& st,
                                             float4v (&xv)[R][FN]) const {
        if (by_four)
            write_as<MODE, true>(base, st, xv);
        else
            write_as<MODE, false>(base, st, xv);
    }
    __device__ __forceinline__ void write(int mode, int64_t base, const NsStep& st,
                                          float4v (&xv)[R][FN]) const {
        if (mode == kOut)
            write_as<kOut>(base, st, xv);
        else if (mode == kParam32)
            write_as<kParam32>(base, st, xv);
        else
            write_as<kParam16>(base, st, xv);
    }
};

struct PanelRun {
    int kind;          // as Source
    int gbf16, mode;   // the gradient's type; kOut, kParam32 or kParam16
    const void* g;
    float* buf;
    float mu;
    double eps;
    int steps;
    // Wide matrices only: panels of a matrix, slices of its norm, and buffers
    int panels, parts;
    const double* part;  // [batch][kNormParts]
    float* x32;          // [batch][panels][16 R * 16 W FN], as the lanes hold them
    float* gram;         // [batch][panels][256 R^2], likewise: a panel's share of A * 2^12
    _Float16* a16;       // [batch][256 R^2], likewise: A * 2^12
};

// A matrix that one panel holds, from the gradient to the result in one launch,
// one block each: the norm is summed, and the momentum moved, as the values are
// first read.  A step of 128 x 128 takes 3.3 us, about evenly of LDS reads, matrix
// instructions and conversions; the whole iteration 24 us (17 launches of the
// tiled products: 65 us), 26 us for 256 matrices.  64 rows of 513 to 1024
// columns (R, FN, W = 4, 4, 16) are more than the registers of 16 waves hold:
// 128 of a lane go to scratch and back; 64 x 1024 44 us.
template <int R, int FN, int W>
__global__ __launch_bounds__(64 * W) void k_ns_small(PanelRun u, NsShape sh, NsStep st) {
    extern __shared__ __align__(16) char lds_raw[];
    typedef Panel<R, FN, W> P;
    P p(lds_raw, sh, 0);
    const int64_t base = (int64_t)blockIdx.x * sh.m * sh.n;
    float4v xv[R][FN];
    p.read_u(u.g, u.gbf16, base, u.buf, u.mu, u.kind, true, xv);
    double sq = 0.;
#pragma unroll
    for (int x = 0; x < R; ++x)
#pragma unroll
        for (int y = 0; y < FN; ++y)
#pragma unroll
            for (int e = 0; e < 4; ++e) sq += (double)xv[x][y][e] * (double)xv[x][y][e];
    p.normalise(block_sum_d(sq, (double*)p.la), u.eps, xv);
    const int c32 = (sh.c + 63) / 64 * 2;  // inner steps of A: columns past them are zero
    for (int k = 0; k < u.steps; ++k) {
        p.forget_places();
        __syncthreads();  // the norm's sums, or B and the old X, have been read
        p.put_x(xv);
        __syncthreads();
        float4v ga[P::FA][P::FB] = {};
        if (p.in_square()) {
            p.square(p.lx, P::kX, c32, ga);
            p.put_square(ga);
        }
        __syncthreads();
        p.polynomial(ga, st, ns_split(u.steps - 1 - k, sh.r));
        p.next(st.a, xv);
    }
    p.write(u.mode, base, st, xv);
}

// A wide matrix, panel by panel, one block each.  STEP false: U becomes X0.
// STEP true: with A, which every block turns into B for itself (128^3 products:
// about a microsecond), X becomes the next X, and with no step left the
// result.  Either leaves the panel's share of the next A.  Latency bounds both:
// 8 us a step for 8 panels (1001 x 128) or 32 (4096 x 128); in tiled products A's
// long sum ran in three blocks and the same matrices took 80 and 139 us in all,
// against 57 and 62.
template <int R, int FN, bool STEP>
__global__ __launch_bounds__(512) void k_ns_panel(PanelRun u, NsShape sh, NsStep st, int left) {
    extern __shared__ __align__(16) char lds_raw[];
    typedef Panel<R, FN, 8> P;
    const int z = blockIdx.x / u.panels, panel = blockIdx.x % u.panels;
    P p(lds_raw, sh, panel * P::kX);
    const int64_t base =
        (int64_t)z * sh.m * sh.n + (int64_t)panel * P::kX * (sh.flip ? sh.r : 1);
    float4v xv[R][FN];
    float4v* const mine = (float4v*)u.x32 +
                          ((int64_t)blockIdx.x * 8 + (threadIdx.x >> 6)) * R * FN * 64 + p.lane;
    if constexpr (STEP) {
        const half4* a =
            (const half4*)u.a16 + ((int64_t)z * 8 + (threadIdx.x >> 6)) * P::FA * P::FB * 64 + p.lane;
        half4 h[P::FA][P::FB];
#pragma unroll
        for (int x = 0; x < P::FA; ++x)
#pragma unroll
            for (int y = 0; y < P::FB; ++y) h[x][y] = a[(x * P::FB + y) * 64];
#pragma unroll
        for (int x = 0; x < R; ++x)
#pragma unroll
            for (int y = 0; y < FN; ++y) xv[x][y] = mine[(x * FN + y) * 64];
        float4v ga[P::FA][P::FB];
#pragma unroll
        for (int x = 0; x < P::FA; ++x)
#pragma unroll
            for (int y = 0; y < P::FB; ++y)
#pragma unroll
                for (int e = 0; e < 4; ++e) ga[x][y][e] = (float)h[x][y][e];
        p.put_square(ga);
        p.put_x(xv);
        __syncthreads();
        p.polynomial(ga, st, ns_split(left, sh.r));
        p.next(st.a, xv);
        if (left == 0) {
            p.write(u.mode, base, st, xv);
            return;
        }
        __syncthreads();  // the old X has been read
    } else {
        p.read_u(u.g, u.gbf16, base, u.buf, u.mu, u.kind, false, xv);
        double sq = 0.;
        for (int t = threadIdx.x; t < u.parts; t += 512) sq += u.part[(int64_t)z * kNormParts + t];
        p.normalise(block_sum_d(sq, (double*)p.la), u.eps, xv);
    }
#pragma unroll
    for (int x = 0; x < R; ++x)
#pragma unroll
        for (int y = 0; y < FN; ++y) mine[(x * FN + y) * 64] = xv[x][y];
    p.put_x(xv);
    __syncthreads();
    float4v ga[P::FA][P::FB] = {};
    p.square(p.lx, P::kX, P::kX / 32, ga);
    float4v* const share = (float4v*)u.gram +
                           ((int64_t)blockIdx.x * 8 + (threadIdx.x >> 6)) * P::FA * P::FB * 64 +
                           p.lane;
#pragma unroll
    for (int x = 0; x < P::FA; ++x)
#pragma unroll
        for (int y = 0; y < P::FB; ++y) share[(x * P::FB + y) * 64] = ga[x][y];
}

// A of each matrix from its panels' shares, in a fixed order: a block takes 64
// groups of four values, each wave a quarter of the panels.  3 us.
__global__ __launch_bounds__(256) void k_ns_panel_sum(PanelRun u, int quads) {
    __shared__ float4v l[4][64];
    const int lane = lane_id(), k = threadIdx.x >> 6;
    const int per = quads / 64;  // blocks of a matrix
    const int64_t z = blockIdx.x / per;
    const int at = (int)(blockIdx.x % per) * 64 + lane;
    const float4v* from = (const float4v*)u.gram + z * u.panels * quads + at;
    float4v s = {};
    int i = k;
    for (; i + 12 < u.panels; i += 16) {
        const float4v a = from[(int64_t)i * quads], b = from[(int64_t)(i + 4) * quads],
                      c = from[(int64_t)(i + 8) * quads], d = from[(int64_t)(i + 12) * quads];
        s += (a + b) + (c + d);
    }
    for (; i < u.panels; i += 4) s += from[(int64_t)i * quads];
    l[k][lane] = s;
    __syncthreads();
    if (k != 0) return;
    s = (l[0][lane] + l[1][lane]) + (l[2][lane] + l[3][lane]);
    half4 h;
#pragma unroll
    for (int e = 0; e < 4; ++e) h[e] = (_Float16)s[e];
    ((half4*)u.a16)[z * quads + at] = h;
}

// ------------------------------------------------------------------ host ---

static NsShape ns_shape(int64_t batch, int64_t m, int64_t n) {
    NsShape s;
    s.batch = batch;
    s.m = m;
    s.n = n;
    s.flip = m > n;
    s.r = (int)(s.flip ? n : m);
    s.c = (int)(s.flip ? m : n);
    s.rp = (int)align_up((size_t)s.r, kTile);
    s.cp = (int)align_up((size_t)s.c, kTile);
    return s;
}

// Matrices of up to 128 rows or columns: in one launch where a panel holds them,
// in panels else.
static bool ns_is_narrow(const NsShape& sh) { return sh.r <= 128; }
static bool ns_is_small(const NsShape& sh) {
    return sh.r <= 64 ? sh.c <= 1024 : sh.r <= 128 && sh.c <= 256;
}
// Columns of a wide matrix's panel.
static int ns_panel_cols(const NsShape& sh) { return sh.r <= 64 ? 256 : 128; }

// Lays the buffers of `batch` wide matrices out from `base` (NULL to count).
static size_t ns_panel_layout(const NsShape& s, int64_t batch, char* base, PanelRun* u) {
    size_t at = 0;
    auto take = [&](size_t bytes) {
        char* p = base ? base + at : nullptr;
        at += align_up(bytes, 256);
        return p;
    };
    const int cols = ns_panel_cols(s), r = s.r <= 64 ? 64 : 128;
    u->panels = (int)ceil_div(s.c, cols);
    const size_t n = (size_t)batch * u->panels;
    u->part = (const double*)take((size_t)batch * kNormParts * sizeof(double));
    u->x32 = (float*)take(n * r * cols * 4);
    u->gram = (float*)take(n * r * r * 4);
    u->a16 = (_Float16*)take((size_t)batch * r * r * 2);
    return at;
}

// Lays the buffers out from `base` (NULL to count only); returns the bytes.
static size_t ns_layout(const NsShape& s, char* base, NsBuffers* w) {
    size_t at = 0;
    if (ns_is_small(s)) return 256;  // unused: every call takes a workspace
    if (ns_is_narrow(s)) {
        PanelRun u;
        return ns_panel_layout(s, s.batch, nullptr, &u);
    }
    auto take = [&](size_t bytes) {
        char* p = base ? base + at : nullptr;
        at += align_up(bytes, 256);
        return p;
    };
    const size_t nx = (size_t)s.batch * s.rp * s.cp, na = (size_t)s.batch * s.rp * s.rp;
    w->part = (double*)take((size_t)s.batch * kNormParts * sizeof(double));
    w->x[0] = (_Float16*)take(nx * 2);
    w->x[1] = (_Float16*)take(nx * 2);
    w->x32 = (float*)take(nx * 4);
    w->a16 = (_Float16*)take(na * 2);
    w->b16 = (_Float16*)take(na * 2);
    w->diag = (float*)take((size_t)s.batch * s.rp * 4);
    return at;
}

static int ns_check_size(const char* what, int64_t batch, int64_t m, int64_t n) {
    if (batch < 0 || m < 1 || n < 1 || m > (1 << 20) || n > (1 << 20) ||
        (batch > 0 && m * n > ((int64_t)1 << 40) / batch))
        return fail(SPOPT_EINVAL, "%s: bad size %lld x %lld x %lld", what, (long long)batch,
                    (long long)m, (long long)n);
    return SPOPT_OK;
}

// Whether the iteration stays where float16 holds it: from singular values in
// [0, 1] (and a little, for rounding), the largest that each step reaches, by
// the critical points of a s + b s^3 + c s^5.
static int ns_check_config(const char* what, const spopt_ns_config& c) {
    if (c.steps < 1 || c.steps > 64) return fail(SPOPT_EINVAL, "%s: steps must lie in [1, 64]", what);
    if (!(c.eps > 0.0) || !isfinite(c.eps))
        return fail(SPOPT_EINVAL, "%s: eps must be finite and > 0", what);
    const double a = c.coef[0], b = c.coef[1], d = c.coef[2];
    if (!isfinite(a) || !isfinite(b) || !isfinite(d))
        return fail(SPOPT_EINVAL, "%s: coefficients must be finite", what);
    double hi = 1.0;
    for (int k = 0; k < c.steps; ++k) {
        hi *= 1.01;
        const double top = hi * hi;  // in t = s^2
        double poly = fabs(b * top + d * top * top);
        if (d != 0.0 && -b / (2 * d) > 0.0 && -b / (2 * d) < top)
            poly = fmax(poly, fabs(b * b / (4 * d)));
        auto f = [&](double t) { return fabs(sqrt(t) * (a + b * t + d * t * t)); };
        double next = f(top);
        // d/ds = a + 3 b t + 5 d t^2
        if (d != 0.0) {
            const double disc = 9 * b * b - 20 * a * d;
            if (disc >= 0.0)
                for (int sg = -1; sg <= 1; sg += 2) {
                    const double t = (-3 * b + sg * sqrt(disc)) / (10 * d);
                    if (t > 0.0 && t < top) next = fmax(next, f(t));
                }
        } else if (b != 0.0) {
            const double t = -a / (3 * b);
            if (t > 0.0 && t < top) next = fmax(next, f(t));
        }
        if (!(poly <= 8.0) || !(next <= 2.0))
            return fail(SPOPT_EINVAL,
                        "%s: coefficients %g, %g, %g take a singular value beyond 2 (or their "
                        "polynomial beyond 8) in step %d",
                        what, a, b, d, k + 1);
        hi = next;
    }
    return SPOPT_OK;
}

typedef Tiling<64, 64, 2, 2, 4> TileS4;
typedef Tiling<64, 64, 2, 2, 2> TileS;
typedef Tiling<96, 96, 2, 2, 4> TileN;
typedef Tiling<128, 128, 2, 4, 4> TileM4;
typedef Tiling<128, 128, 2, 4, 2> TileM;
typedef Tiling<192, 192, 2, 4, 3> TileT;
typedef Tiling<256, 256, 2, 4, 2> TileL;

template <int MODE, class T>
static int64_t ns_tiles(const NsShape& sh) {
    const int64_t tr = ceil_div(sh.rp, T::BM), tc = ceil_div(sh.cp, T::BN);
    return MODE <= kPoly ? tr * (tr + 1) / 2 : tr * tc;
}

template <int MODE, class T>
static int ns_launch(const NsBuffers& w, const NsShape& sh, const NsStep& st, int from,
                     unsigned nb, hipStream_t s) {
    const int64_t tiles = ns_tiles<MODE, T>(sh);
    constexpr int bytes = T::STAGES * T::kStage * (int)sizeof(_Float16);
    if constexpr (bytes > 64 * 1024) {
        SPOPT_HIP(hipFuncSetAttribute((const void*)k_ns_gemm<MODE, T>,
                                      hipFuncAttributeMaxDynamicSharedMemorySize, bytes));
    }
    k_ns_gemm<MODE, T><<<(unsigned)(tiles * nb), T::kThreads, bytes, s>>>(w, sh, st, from,
                                                                        (int)tiles);
    SPOPT_LAUNCHED();
    return SPOPT_OK;
}

// The tiling whose rounds over the 256 CUs take least.  An inner step of 64
// takes a tile of 64, 96, 128, 192 and 256 about 0.2, 0.45, 0.5, 1.1 and 1.8 us
// of its CU (measured on products that fill the card).  Large tiles read less
// for each product, small ones leave fewer CUs idle: for the lower triangles of
// 2048 and 4096 rows, 96 and 192 are 253 tiles where 128 is 136 or 528 and 256
// is 136 (2048 x 8192: 820 us for the iteration by 96, 864 by 128; 4096 x 4096:
// 1463 by 192, 1674 by 256).  Where each CU has one block, four stages in LDS
// beat two: 1024 x 1024 by 64 tiles 150 against 184 us, 2048 x 2048 by 128
// tiles 382 against 417 us; with several blocks a CU they lose (4096 x 4096 by
// 128: 2083 against 1872 us).
template <int MODE>
static int ns_product(const NsBuffers& w, const NsShape& sh, const NsStep& st, int from,
                      unsigned nb, hipStream_t s) {
    auto rounds = [&](int64_t tiles) { return (double)ceil_div(tiles * nb, 256); };
    const double ts = rounds(ns_tiles<MODE, TileS>(sh)), tm = rounds(ns_tiles<MODE, TileM>(sh));
    const double cs = 0.2 * ts, cm = 0.5 * tm, ct = 1.1 * rounds(ns_tiles<MODE, TileT>(sh)),
                 cl = 1.8 * rounds(ns_tiles<MODE, TileL>(sh));
    const double best = fmin(fmin(cs, cm), fmin(ct, cl));
    if constexpr (MODE <= kPoly)
        if (0.45 * rounds(ns_tiles<MODE, TileN>(sh)) < best)
            return ns_launch<MODE, TileN>(w, sh, st, from, nb, s);
    if (cs <= best)
        return ts <= 2 ? ns_launch<MODE, TileS4>(w, sh, st, from, nb, s)
                       : ns_launch<MODE, TileS>(w, sh, st, from, nb, s);
    if (cm <= best)
        return tm <= 1 ? ns_launch<MODE, TileM4>(w, sh, st, from, nb, s)
                       : ns_launch<MODE, TileM>(w, sh, st, from, nb, s);
    if (ct <= best) return ns_launch<MODE, TileT>(w, sh, st, from, nb, s);
    return ns_launch<MODE, TileL>(w, sh, st, from, nb, s);
}

template <int R, int FN, int W>
static int ns_small_launch(const PanelRun& u, const NsShape& sh, const NsStep& st, hipStream_t s) {
    constexpr int bytes = Panel<R, FN, W>::kBytes;
    if constexpr (bytes > 64 * 1024) {
        SPOPT_HIP(hipFuncSetAttribute((const void*)k_ns_small<R, FN, W>,
                                      hipFuncAttributeMaxDynamicSharedMemorySize, bytes));
    }
    // Blocks of a grid: HIP takes fewer than 2^32 threads along an axis.
    constexpr int64_t chunk = ((int64_t)1 << 30) / (64 * W);
    for (int64_t z = 0; z < sh.batch; z += chunk) {
        const int64_t nb = sh.batch - z < chunk ? sh.batch - z : chunk, at = z * sh.m * sh.n;
        PanelRun v = u;
        NsStep sz = st;
        v.g = (const char*)u.g + at * (u.gbf16 ? 2 : 4);
        if (u.buf) v.buf += at;
        sz.out = (char*)st.out + at * (u.mode == kParam32 ? 4 : 2);
        k_ns_small<R, FN, W><<<(unsigned)nb, 64 * W, bytes, s>>>(v, sh, sz);
        SPOPT_LAUNCHED();
    }
    return SPOPT_OK;
}

static int ns_small(const PanelRun& u, const NsShape& sh, const NsStep& st, hipStream_t s) {
    const int64_t fn = ceil_div(sh.c, 128);
    if (sh.r <= 64)
        return fn <= 1   ? ns_small_launch<4, 1, 8>(u, sh, st, s)
               : fn <= 2 ? ns_small_launch<4, 1, 16>(u, sh, st, s)
               : fn <= 4 ? ns_small_launch<4, 2, 16>(u, sh, st, s)
                         : ns_small_launch<4, 4, 16>(u, sh, st, s);
    return fn <= 1 ? ns_small_launch<8, 1, 8>(u, sh, st, s)
                   : ns_small_launch<8, 1, 16>(u, sh, st, s);
}

// Wide matrices: the norm's slices, X0, and two launches a step.
template <class G, int R, int FN>
static int ns_panels(PanelRun r, Source<G> u, const NsShape& sh, const NsStep& st,
                     void* workspace, hipStream_t s) {
    const int64_t numel = sh.m * sh.n;
    constexpr int bytes = Panel<R, FN, 8>::kBytes, quads = 64 * R * R;
    SPOPT_HIP(hipFuncSetAttribute((const void*)k_ns_panel<R, FN, false>,
                                  hipFuncAttributeMaxDynamicSharedMemorySize, bytes));
    SPOPT_HIP(hipFuncSetAttribute((const void*)k_ns_panel<R, FN, true>,
                                  hipFuncAttributeMaxDynamicSharedMemorySize, bytes));
    PanelRun all = r;
    ns_panel_layout(sh, sh.batch, (char*)workspace, &all);
    // As many matrices at a time as keep the grids below 2^22 blocks.
    int64_t chunk = ((int64_t)1 << 22) / all.panels;
    if (chunk > 4096) chunk = 4096;
    for (int64_t z0 = 0; z0 < sh.batch; z0 += chunk) {
        const unsigned nb = (unsigned)(sh.batch - z0 < chunk ? sh.batch - z0 : chunk);
        PanelRun v = all;
        Source<G> uz = u;
        NsStep sz = st;
        uz.g += z0 * numel;
        if (u.buf) uz.buf += z0 * numel;
        v.g = uz.g;
        if (r.buf) v.buf += z0 * numel;
        sz.out = (char*)st.out + z0 * numel * (r.mode == kParam32 ? 4 : 2);
        v.part += z0 * kNormParts;
        v.x32 += z0 * v.panels * 16 * R * Panel<R, FN, 8>::kX;
        v.gram += z0 * v.panels * quads * 4;
        v.a16 += z0 * quads * 4;
        k_ns_norm<G><<<dim3((unsigned)r.parts, nb), 256, 0, s>>>(uz, v.buf, numel, (double*)v.part);
        const unsigned grid = nb * (unsigned)v.panels;
        k_ns_panel<R, FN, false><<<grid, 512, bytes, s>>>(v, sh, sz, 0);
        for (int k = 0; k < r.steps; ++k) {
            k_ns_panel_sum<<<nb * (quads / 64), 256, 0, s>>>(v, quads);
            k_ns_panel<R, FN, true><<<grid, 512, bytes, s>>>(v, sh, sz, r.steps - 1 - k);
        }
        SPOPT_LAUNCHED();
    }
    return SPOPT_OK;
}

template <class G>
static int ns_run(const NsShape& sh, Source<G> u, float* buf, const spopt_ns_config& c,
                  void* workspace, int last, NsStep st, hipStream_t s) {
    const int64_t numel = sh.m * sh.n;
    int64_t parts = ceil_div(numel, 256 * 16);
    if (parts > kNormParts) parts = kNormParts;
    st.a = (float)c.coef[0];
    st.b = (float)c.coef[1];
    st.c = (float)c.coef[2];
    PanelRun pr{};
    pr.kind = u.kind;
    pr.gbf16 = sizeof(G) == 2;
    pr.mode = last;
    pr.g = u.g;
    pr.buf = buf;
    pr.mu = u.mu;
    pr.eps = c.eps;
    pr.steps = c.steps;
    pr.parts = (int)parts;
    if (ns_is_small(sh)) return ns_small(pr, sh, st, s);
    if (ns_is_narrow(sh))
        return sh.r <= 64 ? ns_panels<G, 4, 2>(pr, u, sh, st, workspace, s)
                          : ns_panels<G, 8, 1>(pr, u, sh, st, workspace, s);
    NsBuffers w;
    ns_layout(sh, (char*)workspace, &w);
    const int tr = sh.rp / kTile, tc = sh.cp / kTile;
    // The batch in the grids' last axis: at most so many matrices at a time.
    const int64_t chunk = 32768;
    for (int64_t z0 = 0; z0 < sh.batch; z0 += chunk) {
        const unsigned nb = (unsigned)(sh.batch - z0 < chunk ? sh.batch - z0 : chunk);
        const int64_t nx = (int64_t)sh.rp * sh.cp, na = (int64_t)sh.rp * sh.rp;
        NsBuffers v = w;
        v.part += z0 * kNormParts;
        v.x[0] += z0 * nx;
        v.x[1] += z0 * nx;
        v.x32 += z0 * nx;
        v.a16 += z0 * na;
        v.b16 += z0 * na;
        v.diag += z0 * sh.rp;
        Source<G> uz = u;
        uz.g += z0 * numel;
        if (u.buf) uz.buf += z0 * numel;
        NsStep sz = st;
        sz.out = (char*)st.out + z0 * numel * (last == kParam32 ? 4 : 2);
        k_ns_norm<G><<<dim3((unsigned)parts, nb), 256, 0, s>>>(uz, buf ? buf + z0 * numel : buf,
                                                             numel, v.part);
        SPOPT_LAUNCHED();
        k_ns_init<G><<<dim3(tc, tr, nb), 256, 0, s>>>(uz, v, sh, (int)parts, c.eps);
        SPOPT_LAUNCHED();
        for (int k = 0; k < c.steps; ++k) {
            const int from = k & 1;
            sz.split = ns_split(c.steps - 1 - k, sh.r);
            int rc = ns_product<kGram>(v, sh, sz, from, nb, s);
            if (!rc) rc = ns_product<kPoly>(v, sh, sz, from, nb, s);
            if (!rc)
                rc = k + 1 < c.steps    ? ns_product<kNext>(v, sh, sz, from, nb, s)
                     : last == kOut     ? ns_product<kOut>(v, sh, sz, from, nb, s)
                     : last == kParam32 ? ns_product<kParam32>(v, sh, sz, from, nb, s)
                                        : ns_product<kParam16>(v, sh, sz, from, nb, s);
            if (rc) return rc;
        }
    }
    return SPOPT_OK;
}

static bool is_matrix_type(int32_t t) { return t == SPOPT_DTYPE_F32 || t == SPOPT_DTYPE_BF16; }

// What newton_schulz and muon_step check alike.
static int ns_enter(const char* what, const void* g, int32_t gdtype, const void* out,
                    const NsShape& sh, const spopt_ns_config& c, const void* workspace,
                    size_t workspace_bytes, hipStream_t s, uint32_t flags) {
    if (!is_matrix_type(gdtype))
        return fail(SPOPT_EINVAL, "%s: gradient type %d is neither float32 nor bfloat16", what,
                    gdtype);
    int rc = ns_check_config(what, c);
    if (rc) return rc;
    if (sh.batch > 0 && (g == nullptr || out == nullptr))
        return fail(SPOPT_EINVAL, "%s: NULL matrix", what);
    NsBuffers w;
    const size_t need = ns_layout(sh, nullptr, &w);
    if (sh.batch > 0 && (workspace == nullptr || !aligned16(workspace) || workspace_bytes < need))
        return fail(SPOPT_EWORKSPACE, "%s: workspace of %zu bytes, needs %zu", what,
                    workspace_bytes, need);
    if ((flags & SPOPT_VALIDATE) && sh.batch > 0)
        return validate_on_device(s, false, what, [&](uint32_t* status) {
            return launch_check_finite(g, gdtype, sh.batch * sh.m, sh.n, sh.n, status, s);
        });
    return SPOPT_OK;
}

}  // namespace spopt

using namespace spopt;

extern "C" int newton_schulz_workspace_size(int64_t batch, int64_t m, int64_t n, size_t* bytes) {
    if (bytes == nullptr) return fail(SPOPT_EINVAL, "newton_schulz_workspace_size: NULL output");
    int rc = ns_check_size("newton_schulz_workspace_size", batch, m, n);
    if (rc) return rc;
    NsBuffers w;
    *bytes = ns_layout(ns_shape(batch, m, n), nullptr, &w);
    return SPOPT_OK;
}

extern "C" int newton_schulz(const void* g, int32_t dtype, int64_t batch, int64_t m, int64_t n,
                             const spopt_ns_config* config, void* out, void* workspace,
                             size_t workspace_bytes, void* stream, uint32_t flags) {
    hipStream_t s = (hipStream_t)stream;
    if (config == nullptr) return fail(SPOPT_EINVAL, "newton_schulz: NULL configuration");
    int rc = ns_check_size("newton_schulz", batch, m, n);
    if (rc) return rc;
    const NsShape sh = ns_shape(batch, m, n);
    rc = ns_enter("newton_schulz", g, dtype, out, sh, *config, workspace, workspace_bytes, s,
                  flags);
    if (rc || batch == 0) return rc;
    NsStep st{};
    st.out = out;
    if (dtype == SPOPT_DTYPE_F32)
        return ns_run(sh, Source<float>{(const float*)g, nullptr, 0.f, 0}, nullptr, *config,
                      workspace, kOut, st, s);
    return ns_run(sh, Source<__bf16>{(const __bf16*)g, nullptr, 0.f, 0}, nullptr, *config,
                  workspace, kOut, st, s);
}

extern "C" int muon_step(void* params, int32_t pdtype, float* buf, const void* g, int32_t gdtype,
                         int64_t batch, int64_t m, int64_t n, const spopt_muon_config* config,
                         void* workspace, size_t workspace_bytes, void* stream, uint32_t flags) {
    hipStream_t s = (hipStream_t)stream;
    if (config == nullptr) return fail(SPOPT_EINVAL, "muon_step: NULL configuration");
    const spopt_muon_config& c = *config;
    if (!(c.lr >= 0.0) || !isfinite(c.lr))
        return fail(SPOPT_EINVAL, "muon_step: lr must be finite and >= 0");
    if (!(c.momentum >= 0.0 && c.momentum < 1.0))
        return fail(SPOPT_EINVAL, "muon_step: momentum must lie in [0, 1)");
    if (!(c.weight_decay >= 0.0) || !isfinite(c.weight_decay))
        return fail(SPOPT_EINVAL, "muon_step: weight_decay must be finite and >= 0");
    if (!isfinite(c.scale)) return fail(SPOPT_EINVAL, "muon_step: scale must be finite");
    if (c.nesterov != 0 && c.nesterov != 1)
        return fail(SPOPT_EINVAL, "muon_step: nesterov must be 0 or 1");
    if (!is_matrix_type(pdtype))
        return fail(SPOPT_EINVAL, "muon_step: weight type %d is neither float32 nor bfloat16",
                    pdtype);
    int rc = ns_check_size("muon_step", batch, m, n);
    if (rc) return rc;
    if (batch > 0 && c.momentum != 0.0 && buf == nullptr)
        return fail(SPOPT_EINVAL, "muon_step: a momentum needs its buffer");
    const NsShape sh = ns_shape(batch, m, n);
    rc = ns_enter("muon_step", g, gdtype, params, sh, c.ns, workspace, workspace_bytes, s,
                  flags);
    if (rc || batch == 0) return rc;
    NsStep st{};
    st.out = params;
    st.keep = (float)(1.0 - c.lr * c.weight_decay);
    st.move = (float)(c.lr * c.scale);
    const int last = pdtype == SPOPT_DTYPE_F32 ? kParam32 : kParam16;
    const int kind = c.momentum == 0.0 ? 0 : c.nesterov ? 2 : 1;
    float* b = kind ? buf : nullptr;
    if (gdtype == SPOPT_DTYPE_F32)
        return ns_run(sh, Source<float>{(const float*)g, b, (float)c.momentum, kind}, b, c.ns,
                      workspace, last, st, s);
    return ns_run(sh, Source<__bf16>{(const __bf16*)g, b, (float)c.momentum, kind}, b, c.ns,
                  workspace, last, st, s);
}
