// dropout.hip - dropout with its mask from a counter-based generator.
//
// Eight values take one Philox4x32-10 block of 128 bits, 16 bits each: 20
// products of 32 by 32 bits for eight values, where 32 bits a value would take
// twice as many and, of 16-bit types, about as long as HBM takes for the values.
// So p counts in steps of 2^-16, and the factor in front of what is kept is
// 2^16 / (2^16 - q) of the q taken, which leaves the mean unbiased.
#include "dense.hpp"

namespace spopt {

struct DropArgs {
    uint64_t seed, offset;
    const int64_t* d_seed;
    uint32_t q;       // round(p 2^16)
    float factor;
};

// The generator's ten rounds (Salmon et al., 2011) for one counter.
__device__ __forceinline__ void philox(uint64_t index, uint64_t offset, uint64_t seed,
                                       uint32_t (&out)[4]) {
    uint32_t c0 = (uint32_t)index, c1 = (uint32_t)(index >> 32);
    uint32_t c2 = (uint32_t)offset, c3 = (uint32_t)(offset >> 32);
    uint32_t k0 = (uint32_t)seed, k1 = (uint32_t)(seed >> 32);
#pragma unroll
    for (int r = 0; r < 10; ++r) {
        const uint64_t a = (uint64_t)c0 * 0xD2511F53u, b = (uint64_t)c2 * 0xCD9E8D57u;
        c0 = (uint32_t)(b >> 32) ^ c1 ^ k0;
        c2 = (uint32_t)(a >> 32) ^ c3 ^ k1;
        c1 = (uint32_t)b;
        c3 = (uint32_t)a;
        k0 += 0x9E3779B9u;
        k1 += 0xBB67AE85u;
    }
    out[0] = c0;
    out[1] = c1;
    out[2] = c2;
    out[3] = c3;
}

// What becomes of eight values: dropped ones give 0 whatever they hold.
template <bool RES>
__device__ __forceinline__ void drop8(const DropArgs& a, uint64_t seed, uint64_t chunk,
                                      float (&v)[8], const float (&res)[8]) {
    uint32_t bits[4];
    philox(chunk, a.offset, seed, bits);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const uint32_t b = e & 1 ? bits[e / 2] >> 16 : bits[e / 2] & 0xFFFFu;
        v[e] = b >= a.q ? v[e] * a.factor : 0.f;
        if (RES) v[e] += res[e];
    }
}

// Rows that follow one another without a gap are one run of values, of which a
// thread takes eight at a time (16 bytes a load, 32 of float32).  HBM bounds it:
// 16384 x 4096 bfloat16 with a residual 76.8 us, 5.2 TB/s, what a copy reaches; 65536 x
// 128 float32 11.8 us (part of it in the last-level cache).
template <class T, bool RES>
__global__ __launch_bounds__(256) void k_dropout(const T* x, const T* res, T* y, int64_t numel,
                                                 DropArgs a) {
    const uint64_t seed = a.d_seed ? (uint64_t)*a.d_seed : a.seed;
    const int64_t whole = numel / 8;
    const int64_t step = (int64_t)gridDim.x * 256;
    for (int64_t c = (int64_t)blockIdx.x * 256 + threadIdx.x; c < whole; c += step) {
        float v[8], r[8] = {};
        load_v<T, 8>(x + c * 8, v);
        if (RES) load_v<T, 8>(res + c * 8, r);
        drop8<RES>(a, seed, (uint64_t)c, v, r);
        store_v<T, 8>(y + c * 8, v);
    }
    const int left = (int)(numel - whole * 8);
    if (left != 0 && blockIdx.x == 0 && threadIdx.x == 0) {
        float v[8] = {}, r[8] = {};
        for (int e = 0; e < left; ++e) {
            v[e] = (float)x[whole * 8 + e];
            if (RES) r[e] = (float)res[whole * 8 + e];
        }
        drop8<RES>(a, seed, (uint64_t)whole, v, r);
        for (int e = 0; e < left; ++e) y[whole * 8 + e] = (T)v[e];
    }
}

// Rows with gaps between them.  Eight values may run over the end of a row, and are
// then taken one by one: 16384 x 4096 bfloat16 in rows of 4160 46 us (torch's copy of them
// 45), 4091 columns in rows of 4160 78 (46), 65536 x 125 in rows of 128 23 (9).
template <class T, bool RES>
__global__ __launch_bounds__(256) void k_dropout_rows(const T* x, int64_t xs, const T* res,
                                                      int64_t rs, T* y, int64_t ys, int64_t rows,
                                                      int64_t cols, FastDiv by, DropArgs a) {
    const uint64_t seed = a.d_seed ? (uint64_t)*a.d_seed : a.seed;
    const int64_t numel = rows * cols, chunks = (numel + 7) / 8;
    const int64_t step = (int64_t)gridDim.x * 256;
    for (int64_t c = (int64_t)blockIdx.x * 256 + threadIdx.x; c < chunks; c += step) {
        uint64_t rem;
        int64_t i = (int64_t)by.div((uint64_t)(c * 8), &rem), j = (int64_t)rem;
        float v[8] = {}, r[8] = {};
        if (j + 8 <= cols) {
            load_v<T, 8>(x + i * xs + j, v);
            if (RES) load_v<T, 8>(res + i * rs + j, r);
            drop8<RES>(a, seed, (uint64_t)c, v, r);
            store_v<T, 8>(y + i * ys + j, v);
            continue;
        }
        const int n = numel - c * 8 < 8 ? (int)(numel - c * 8) : 8;
        int64_t i2 = i, j2 = j;
        for (int e = 0; e < n; ++e) {
            v[e] = (float)x[i2 * xs + j2];
            if (RES) r[e] = (float)res[i2 * rs + j2];
            if (++j2 == cols) {
                j2 = 0;
                ++i2;
            }
        }
        drop8<RES>(a, seed, (uint64_t)c, v, r);
        for (int e = 0; e < n; ++e) {
            y[i * ys + j] = (T)v[e];
            if (++j == cols) {
                j = 0;
                ++i;
            }
        }
    }
}

template <class T>
static void dropout_launch(const void* x, int64_t xs, const void* res, int64_t rs, void* y,
                           int64_t ys, int64_t rows, int64_t cols, const DropArgs& a,
                           hipStream_t s) {
    const int64_t blocks = ceil_div(rows * cols, 8 * 256);
    const unsigned grid = (unsigned)(blocks < 4096 ? blocks : 4096);
    const T *tx = (const T*)x, *tr = (const T*)res;
    T* const ty = (T*)y;
    if (rows == 1 || (xs == cols && ys == cols && (res == nullptr || rs == cols))) {
        if (res)
            k_dropout<T, true><<<grid, 256, 0, s>>>(tx, tr, ty, rows * cols, a);
        else
            k_dropout<T, false><<<grid, 256, 0, s>>>(tx, tr, ty, rows * cols, a);
        return;
    }
    const FastDiv by = FastDiv::make((uint64_t)cols);
    if (res)
        k_dropout_rows<T, true><<<grid, 256, 0, s>>>(tx, xs, tr, rs, ty, ys, rows, cols, by, a);
    else
        k_dropout_rows<T, false><<<grid, 256, 0, s>>>(tx, xs, tr, rs, ty, ys, rows, cols, by, a);
}

static int dropout_run(const char* what, const void* x, int64_t xs, const void* res, int64_t rs,
                       int64_t rows, int64_t cols, int32_t dtype, double p, uint64_t seed,
                       const int64_t* d_seed, uint64_t offset, void* y, int64_t ys, hipStream_t s,
                       uint32_t flags) {
    if (rows < 0 || cols < 1 || rows > INT64_MAX / 16 / cols)
        return fail(SPOPT_EINVAL, "%s: bad size %lld x %lld", what, (long long)rows,
                    (long long)cols);
    if (dtype != SPOPT_DTYPE_F32 && dtype != SPOPT_DTYPE_BF16 && dtype != SPOPT_DTYPE_F16)
        return fail(SPOPT_EINVAL, "%s: unknown element type %d", what, dtype);
    if (!(p >= 0.0 && p <= 1.0)) return fail(SPOPT_EINVAL, "%s: p must lie in [0, 1]", what);
    if (rows > 0 && (x == nullptr || y == nullptr))
        return fail(SPOPT_EINVAL, "%s: NULL input or output", what);
    if (rows > 1 && (xs < cols || ys < cols || (res != nullptr && rs < cols)))
        return fail(SPOPT_EINVAL, "%s: a row stride below cols", what);
    if (rows == 0) return SPOPT_OK;
    if (flags & SPOPT_VALIDATE) {
        const int rc = validate_on_device(s, false, what, [&](uint32_t* status) {
            const int e = launch_check_finite(x, dtype, rows, cols, xs, status, s);
            return e || res == nullptr ? e
                                       : launch_check_finite(res, dtype, rows, cols, rs, status, s);
        });
        if (rc) return rc;
    }
    DropArgs a{seed, offset, d_seed, (uint32_t)(p * 65536.0 + 0.5), 0.f};
    if (a.q < 65536) a.factor = (float)(65536.0 / (65536.0 - (double)a.q));
    if (dtype == SPOPT_DTYPE_F32)
        dropout_launch<float>(x, xs, res, rs, y, ys, rows, cols, a, s);
    else if (dtype == SPOPT_DTYPE_BF16)
        dropout_launch<__bf16>(x, xs, res, rs, y, ys, rows, cols, a, s);
    else
        dropout_launch<_Float16>(x, xs, res, rs, y, ys, rows, cols, a, s);
    SPOPT_LAUNCHED();
    return SPOPT_OK;
}

}  // namespace spopt

using namespace spopt;

extern "C" int dropout_forward(const void* x, int64_t x_stride, const void* residual,
                               int64_t residual_stride, int64_t rows, int64_t cols, int32_t dtype,
                               double p, uint64_t seed, const int64_t* d_seed, uint64_t offset,
                               void* y, int64_t y_stride, void* stream, uint32_t flags) {
    return dropout_run("dropout_forward", x, x_stride, residual, residual_stride, rows, cols, dtype,
                       p, seed, d_seed, offset, y, y_stride, (hipStream_t)stream, flags);
}

extern "C" int dropout_backward(const void* dy, int64_t dy_stride, int64_t rows, int64_t cols,
                                int32_t dtype, double p, uint64_t seed, const int64_t* d_seed,
                                uint64_t offset, void* dx, int64_t dx_stride, void* stream,
                                uint32_t flags) {
    return dropout_run("dropout_backward", dy, dy_stride, nullptr, 0, rows, cols, dtype, p, seed,
                       d_seed, offset, dx, dx_stride, (hipStream_t)stream, flags);
}
