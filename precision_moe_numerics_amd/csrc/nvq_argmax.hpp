// nvq_argmax.hpp -- the routers' choice: order-preserving integer keys of fp64
// values and an argmax over groups of lanes (the largest key, then the lower
// index).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace nvq {

// Unsigned integers in the order of fp64 values; -0 becomes +0 first, so equal
// values have equal keys.
__device__ __forceinline__ uint64_t order_key(double v) {
    const uint64_t b = (uint64_t)__double_as_longlong(v + 0.0);
    return (b >> 63) ? ~b : (b | 0x8000000000000000ull);
}

template <int CTRL>
__device__ __forceinline__ uint32_t dpp_u32(uint32_t v) {
    return (uint32_t)__builtin_amdgcn_mov_dpp((int)v, CTRL, 0xF, 0xF, true);
}

__device__ __forceinline__ void argmax_take(uint64_t& k, int& e, uint64_t ok, int oe) {
    const bool take = ok > k || (ok == k && oe < e);
    k = take ? ok : k;
    e = take ? oe : e;
}

template <int CTRL>
__device__ __forceinline__ void argmax_dpp(uint64_t& k, int& e) {
    const uint64_t ok = ((uint64_t)dpp_u32<CTRL>((uint32_t)(k >> 32)) << 32) | dpp_u32<CTRL>((uint32_t)k);
    argmax_take(k, e, ok, (int)dpp_u32<CTRL>((uint32_t)e));
}

__device__ __forceinline__ void argmax_xor(uint64_t& k, int& e, int off) {
    const uint64_t ok = ((uint64_t)(uint32_t)__shfl_xor((int)(k >> 32), off, 64) << 32) |
                        (uint32_t)__shfl_xor((int)(uint32_t)k, off, 64);
    argmax_take(k, e, ok, __shfl_xor(e, off, 64));
}

// All-reduce over aligned groups of G lanes: every lane ends with the
// group's (largest key, lowest expert among those).
template <int G>
__device__ __forceinline__ void group_argmax(uint64_t& k, int& e) {
    argmax_dpp<0xB1>(k, e);   // lane ^ 1
    argmax_dpp<0x4E>(k, e);   // lane ^ 2
    argmax_dpp<0x141>(k, e);  // mirror within 8 lanes
    argmax_dpp<0x140>(k, e);  // mirror within 16 lanes
    if (G == 64) {
        argmax_xor(k, e, 16);
        argmax_xor(k, e, 32);
    }
}

}  // namespace nvq
