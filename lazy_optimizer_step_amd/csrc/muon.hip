// muon.hip - Newton-Schulz orthogonalisation of matrices and the Muon step.
//
// With X the r x c iterate (r <= c, the input transposed where it is taller
// than wide), one step is three products:
//   A = X X^T,   B = b A + c A A,   X <- a X + B X.
// Every product is written as P Q^T with both operands' inner axis adjacent,
// which is what the matrix cores' operands take: A from the rows of X, A A
// from the rows of A (A is symmetric), B X from the rows of X^T, which the
// kernel that writes X writes as well.
//
// Types.  The operands are float16 and the sums float32.  float16 carries 11
// bits against bfloat16's 8 at the same rate; its range is met by powers of
// two in front: X * 2^8, A and B * 2^12 (entries are bounded by the largest
// singular value, which the host checks).  X is also kept in float32 for the
// a X term: in the directions of small singular values B is near zero, so
// rounding errors of X there would come in through a X alone, and grow by
// a factor of a in every step.  Errors against 64 bits, relative to the
// result's norm, for 256 to 1024 rows and Gaussian, low-rank and decaying
// spectra: at most 1.7e-3 so; 7e-3 with X in float16 alone, 6e-2 with all of
// it in bfloat16.
#include <math.h>

#include "dense.hpp"

namespace spopt {

typedef _Float16 half8 __attribute__((ext_vector_type(8)));
typedef float float4v __attribute__((ext_vector_type(4)));

constexpr int kTile = 64;                    // rows, columns and inner axis are padded to it
constexpr float kXScale = 256.f;             // 2^8
constexpr float kAScale = 4096.f;            // 2^12
constexpr int kNormParts = 256;              // partial sums of a matrix's norm, at most

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
// of sum(U^2), in double.  Block (x, z): slice x of matrix z.
template <class G>
__global__ __launch_bounds__(256) void k_ns_norm(Source<G> u, float* buf, int64_t numel,
                                                 double* part) {
    __shared__ double lds[4];
    const int64_t base = (int64_t)blockIdx.y * numel;
    double s = 0.;
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < numel;
         i += (int64_t)gridDim.x * 256) {
        if (u.kind != 0) buf[base + i] = u.mu * buf[base + i] + (float)u.g[base + i];
        const double v = (double)u.at(base + i);
        s += v * v;
    }
    s = block_sum_d(s, lds);
    if (threadIdx.x == 0) part[(int64_t)blockIdx.y * kNormParts + blockIdx.x] = s;
}

struct NsBuffers {
    float* x32;      // [batch][rp * cp]
    _Float16* x16;   // [batch][rp * cp]   X * 2^8
    _Float16* xt[2]; // [batch][cp * rp]   X^T * 2^8
    _Float16* a16;   // [batch][rp * rp]   A * 2^12
    _Float16* b16;   // [batch][rp * rp]   B * 2^12
    double* part;    // [batch][kNormParts]
};

struct NsShape {
    int64_t batch, m, n;
    int r, c, rp, cp;
    bool flip;       // X is the input's transpose
};

// X0 = U / (|U| + eps) into the padded buffers, rows and columns beyond the
// matrix as zeros.  One 64 x 64 tile of X per block.
template <class G>
__global__ __launch_bounds__(256) void k_ns_init(Source<G> u, NsBuffers w, NsShape sh, int parts,
                                                 double eps) {
    __shared__ double lds[4];
    __shared__ float tile[kTile][kTile + 1];
    const int64_t z = blockIdx.z;
    const double sq = block_sum_d(
        (int)threadIdx.x < parts ? w.part[z * kNormParts + threadIdx.x] : 0., lds);
    const double scale = 1.0 / (sqrt(sq) + eps);
    const int i0 = blockIdx.y * kTile, j0 = blockIdx.x * kTile;
    const int q = threadIdx.x & 63, k = threadIdx.x >> 6;
    const int64_t base = z * sh.m * sh.n;
    for (int t = k; t < kTile; t += 4) {
        // Read along the input's rows: those of X, or X's columns.
        const int i = sh.flip ? i0 + q : i0 + t, j = sh.flip ? j0 + t : j0 + q;
        float v = 0.f;
        if (i < sh.r && j < sh.c)
            v = (float)((double)u.at(base + (sh.flip ? (int64_t)j * sh.r + i
                                                     : (int64_t)i * sh.c + j)) * scale);
        if (sh.flip)
            tile[q][t] = v;
        else
            tile[t][q] = v;
    }
    __syncthreads();
    const int64_t xb = z * sh.rp * sh.cp;
    for (int t = k; t < kTile; t += 4) {
        const int64_t o = xb + (int64_t)(i0 + t) * sh.cp + j0 + q;
        w.x32[o] = tile[t][q];
        w.x16[o] = (_Float16)(tile[t][q] * kXScale);
        w.xt[0][xb + (int64_t)(j0 + t) * sh.rp + i0 + q] = (_Float16)(tile[q][t] * kXScale);
    }
}

enum : int { kGram = 0, kPoly = 1, kNext = 2, kOut = 3, kParam32 = 4, kParam16 = 5 };

struct NsStep {
    float a, b, c;
    void* out;       // kOut: bfloat16; kParam*: the weight
    float keep, move;  // kParam*: p <- keep * p - move * X
};

// One product P Q^T over 64 x 64 tiles, the inner axis 64 at a time through
// LDS, and what its result is for:
//   kGram  A = X X^T           kPoly  B = b A + c A A     (lower tiles, mirrored)
//   kNext  X <- a X + B X      kOut / kParam*  the last step's X, written out
template <int MODE>
__global__ __launch_bounds__(256) void k_ns_gemm(NsBuffers w, NsShape sh, NsStep st, int from) {
    constexpr int LD = kTile + 8;  // 144-byte rows: 16-byte reads of 16 rows meet each bank twice
    __shared__ __align__(16) _Float16 lp[kTile * LD], lq[kTile * LD];
    const int64_t z = blockIdx.z;
    const int64_t nx = (int64_t)sh.rp * sh.cp, na = (int64_t)sh.rp * sh.rp;
    const _Float16 *p, *q;
    int64_t k_len;
    if (MODE == kGram) {
        p = q = w.x16 + z * nx;
        k_len = sh.cp;
    } else if (MODE == kPoly) {
        p = q = w.a16 + z * na;
        k_len = sh.rp;
    } else {
        p = w.b16 + z * na;
        q = w.xt[from] + z * nx;
        k_len = sh.rp;
    }
    int ti = blockIdx.y, tj = blockIdx.x;
    if (MODE <= kPoly && tj > ti) return;
    const int i0 = ti * kTile, j0 = tj * kTile;
    const int lane = lane_id(), wv = threadIdx.x >> 6;
    const int wi = (wv >> 1) * 32, wj = (wv & 1) * 32;
    float4v acc[2][2] = {};
    for (int64_t k0 = 0; k0 < k_len; k0 += kTile) {
        __syncthreads();
        for (int t = threadIdx.x; t < kTile * 8; t += 256) {
            const int row = t >> 3, ch = (t & 7) * 8;
            *(half8*)(lp + row * LD + ch) = *(const half8*)(p + (i0 + row) * k_len + k0 + ch);
            *(half8*)(lq + row * LD + ch) = *(const half8*)(q + (j0 + row) * k_len + k0 + ch);
        }
        __syncthreads();
#pragma unroll
        for (int kk = 0; kk < kTile; kk += 32) {
            half8 fa[2], fb[2];
            const int ko = kk + (lane >> 4) * 8;
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                fa[t] = *(const half8*)(lp + (wi + t * 16 + (lane & 15)) * LD + ko);
                fb[t] = *(const half8*)(lq + (wj + t * 16 + (lane & 15)) * LD + ko);
            }
#pragma unroll
            for (int x = 0; x < 2; ++x)
#pragma unroll
                for (int y = 0; y < 2; ++y)
                    acc[x][y] = __builtin_amdgcn_mfma_f32_16x16x32_f16(fa[x], fb[y], acc[x][y], 0,
                                                                       0, 0);
        }
    }
#pragma unroll
    for (int x = 0; x < 2; ++x)
#pragma unroll
        for (int y = 0; y < 2; ++y)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int i = i0 + wi + x * 16 + (lane >> 4) * 4 + e;
                const int j = j0 + wj + y * 16 + (lane & 15);
                const float v = acc[x][y][e];
                if (MODE == kGram || MODE == kPoly) {
                    const int64_t o = z * na + (int64_t)i * sh.rp + j;
                    const _Float16 h =
                        MODE == kGram
                            ? (_Float16)(v * (kAScale / (kXScale * kXScale)))
                            : (_Float16)(st.b * (float)w.a16[o] + st.c * (v / kAScale));
                    _Float16* d = MODE == kGram ? w.a16 : w.b16;
                    d[o] = h;
                    d[z * na + (int64_t)j * sh.rp + i] = h;
                } else {
                    const int64_t o = z * nx + (int64_t)i * sh.cp + j;
                    const float xn = st.a * w.x32[o] + v / (kAScale * kXScale);
                    if (MODE == kNext) {
                        const _Float16 h = (_Float16)(xn * kXScale);
                        w.x32[o] = xn;
                        w.x16[o] = h;
                        w.xt[from ^ 1][z * nx + (int64_t)j * sh.rp + i] = h;
                    } else if (i < sh.r && j < sh.c) {
                        const int64_t d = z * sh.m * sh.n + (sh.flip ? (int64_t)j * sh.r + i
                                                                     : (int64_t)i * sh.c + j);
                        if (MODE == kOut)
                            ((__bf16*)st.out)[d] = (__bf16)xn;
                        else if (MODE == kParam32)
                            ((float*)st.out)[d] = st.keep * ((float*)st.out)[d] - st.move * xn;
                        else
                            ((__bf16*)st.out)[d] =
                                (__bf16)(st.keep * (float)((__bf16*)st.out)[d] - st.move * xn);
                    }
                }
            }
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

// Lays the buffers out from `base` (NULL to count only); returns the bytes.
static size_t ns_layout(const NsShape& s, char* base, NsBuffers* w) {
    size_t at = 0;
    auto take = [&](size_t bytes) {
        char* p = base ? base + at : nullptr;
        at += align_up(bytes, 256);
        return p;
    };
    const size_t nx = (size_t)s.batch * s.rp * s.cp, na = (size_t)s.batch * s.rp * s.rp;
    w->part = (double*)take((size_t)s.batch * kNormParts * sizeof(double));
    w->x32 = (float*)take(nx * 4);
    w->x16 = (_Float16*)take(nx * 2);
    w->xt[0] = (_Float16*)take(nx * 2);
    w->xt[1] = (_Float16*)take(nx * 2);
    w->a16 = (_Float16*)take(na * 2);
    w->b16 = (_Float16*)take(na * 2);
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

template <class G>
static int ns_run(const NsShape& sh, Source<G> u, float* buf, const spopt_ns_config& c,
                  NsBuffers w, int last, NsStep st, hipStream_t s) {
    const int64_t numel = sh.m * sh.n;
    int64_t parts = ceil_div(numel, 256 * 16);
    if (parts > kNormParts) parts = kNormParts;
    st.a = (float)c.coef[0];
    st.b = (float)c.coef[1];
    st.c = (float)c.coef[2];
    const int tr = sh.rp / kTile, tc = sh.cp / kTile;
    // The batch is the grid's last axis, at most 65535 matrices at a time.
    for (int64_t z0 = 0; z0 < sh.batch; z0 += 65535) {
        const unsigned nb = (unsigned)(sh.batch - z0 < 65535 ? sh.batch - z0 : 65535);
        const int64_t nx = (int64_t)sh.rp * sh.cp, na = (int64_t)sh.rp * sh.rp;
        NsBuffers v = w;
        v.part += z0 * kNormParts;
        v.x32 += z0 * nx;
        v.x16 += z0 * nx;
        v.xt[0] += z0 * nx;
        v.xt[1] += z0 * nx;
        v.a16 += z0 * na;
        v.b16 += z0 * na;
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
            k_ns_gemm<kGram><<<dim3(tr, tr, nb), 256, 0, s>>>(v, sh, sz, from);
            k_ns_gemm<kPoly><<<dim3(tr, tr, nb), 256, 0, s>>>(v, sh, sz, from);
            const dim3 gx(tc, tr, nb);
            if (k + 1 < c.steps)
                k_ns_gemm<kNext><<<gx, 256, 0, s>>>(v, sh, sz, from);
            else if (last == kOut)
                k_ns_gemm<kOut><<<gx, 256, 0, s>>>(v, sh, sz, from);
            else if (last == kParam32)
                k_ns_gemm<kParam32><<<gx, 256, 0, s>>>(v, sh, sz, from);
            else
                k_ns_gemm<kParam16><<<gx, 256, 0, s>>>(v, sh, sz, from);
            SPOPT_LAUNCHED();
        }
    }
    return SPOPT_OK;
}

static bool is_matrix_type(int32_t t) { return t == SPOPT_DTYPE_F32 || t == SPOPT_DTYPE_BF16; }

// What newton_schulz and muon_step check alike; fills the workspace's layout.
static int ns_enter(const char* what, const void* g, int32_t gdtype, const void* out,
                    const NsShape& sh, const spopt_ns_config& c, void* workspace,
                    size_t workspace_bytes, NsBuffers* w, hipStream_t s, uint32_t flags) {
    if (!is_matrix_type(gdtype))
        return fail(SPOPT_EINVAL, "%s: gradient type %d is neither float32 nor bfloat16", what,
                    gdtype);
    int rc = ns_check_config(what, c);
    if (rc) return rc;
    if (sh.batch > 0 && (g == nullptr || out == nullptr))
        return fail(SPOPT_EINVAL, "%s: NULL matrix", what);
    const size_t need = ns_layout(sh, nullptr, w);
    if (sh.batch > 0 && (workspace == nullptr || !aligned16(workspace) || workspace_bytes < need))
        return fail(SPOPT_EWORKSPACE, "%s: workspace of %zu bytes, needs %zu", what,
                    workspace_bytes, need);
    ns_layout(sh, (char*)workspace, w);
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
    NsBuffers w;
    rc = ns_enter("newton_schulz", g, dtype, out, sh, *config, workspace, workspace_bytes, &w, s,
                  flags);
    if (rc || batch == 0) return rc;
    NsStep st{};
    st.out = out;
    if (dtype == SPOPT_DTYPE_F32)
        return ns_run(sh, Source<float>{(const float*)g, nullptr, 0.f, 0}, nullptr, *config, w,
                      kOut, st, s);
    return ns_run(sh, Source<__bf16>{(const __bf16*)g, nullptr, 0.f, 0}, nullptr, *config, w, kOut,
                  st, s);
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
    NsBuffers w;
    rc = ns_enter("muon_step", g, gdtype, params, sh, c.ns, workspace, workspace_bytes, &w, s,
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
        return ns_run(sh, Source<float>{(const float*)g, b, (float)c.momentum, kind}, b, c.ns, w,
                      last, st, s);
    return ns_run(sh, Source<__bf16>{(const __bf16*)g, b, (float)c.momentum, kind}, b, c.ns, w,
                  last, st, s);
}
