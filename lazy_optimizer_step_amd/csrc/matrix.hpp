// matrix.hpp - what the tiled matrix products share: loads straight into LDS,
// waits for them, transposing reads, and the order of tiles.
#pragma once

#include "common.hpp"

namespace spopt {

typedef _Float16 half4 __attribute__((ext_vector_type(4)));
typedef _Float16 half8 __attribute__((ext_vector_type(8)));
typedef float float4v __attribute__((ext_vector_type(4)));

constexpr int kTile = 64;                    // rows, columns and inner axis are padded to it

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
// is listed as clobbered), and no instruction that it makes of the sources that
// include this reads it.
__device__ __forceinline__ void load_lds16(const void* from, void* to) {
    const uint32_t m0 = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) void*)to;
    asm volatile("s_mov_b32 m0, %1\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, off" ::"v"(from),
                 "s"(m0)
                 : "memory");
}

// The same from `off` bytes behind an address that all lanes share.
__device__ __forceinline__ void load_lds16_from(const void* from, uint32_t off, void* to) {
    const uint32_t m0 = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) void*)to;
    const uint64_t at = (uint64_t)from;
    const uint64_t base = (uint64_t)(uint32_t)__builtin_amdgcn_readfirstlane((int)(at >> 32)) << 32 |
                          (uint32_t)__builtin_amdgcn_readfirstlane((int)at);
    asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, %1" ::"v"(off),
                 "s"(base), "s"(m0)
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

}  // namespace spopt
