// Shared pieces of the low-precision training operators (include/qsgd_ops.h):
// element types, loads and stores of eight elements at any element alignment,
// wave reductions.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "qsgd_ops.h"

namespace qsgd {
namespace ops {

using bf16 = __bf16;
using f16 = _Float16;
typedef int v4i __attribute__((ext_vector_type(4)));

// Eight consecutive elements as fp32. The copy carries the element's own
// alignment, for which gfx950 still issues 16-byte loads (global memory is read
// at any byte address).
template <class T>
__device__ __forceinline__ void load8(const T *p, float (&f)[8]) {
    T v[8];
    __builtin_memcpy(v, p, sizeof(v));
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = (float)v[i];
}

// Eight elements that were loaded as words.
__device__ __forceinline__ void unpack(const uint32_t (&w)[8], float (&f)[8], float) {
#pragma unroll
    for (int j = 0; j < 8; ++j) f[j] = __uint_as_float(w[j]);
}
__device__ __forceinline__ void unpack(const uint32_t (&w)[4], float (&f)[8], bf16) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        f[2 * j] = __uint_as_float(w[j] << 16);
        f[2 * j + 1] = __uint_as_float(w[j] & 0xffff0000u);
    }
}
__device__ __forceinline__ void unpack(const uint32_t (&w)[4], float (&f)[8], f16) {
    typedef f16 pair __attribute__((ext_vector_type(2)));
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const pair v = __builtin_bit_cast(pair, w[j]);
        f[2 * j] = (float)v[0];
        f[2 * j + 1] = (float)v[1];
    }
}

// Elements [c, c + 8) of a row of n, as words; those past its end are 0. In two
// parts, so that a thread's loads can all be issued before the first is looked at:
// fetch() loads eight elements that exist without a branch (the row's last ones
// where c + 8 passes its end), settle() moves them to their places in the few
// threads at the row's end.
template <class T>
struct Eight {
    uint32_t w[2 * sizeof(T)];
};
template <class T>
__device__ __forceinline__ void fetch(const T *row, uint32_t c, uint32_t n, Eight<T> &v) {
    if (n >= 8) {
        __builtin_memcpy(v.w, row + min(c, n - 8), sizeof(v.w));
    } else {  // a row of a few elements
        T e[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) e[i] = (uint32_t)i < n ? row[i] : (T)0.0f;
        __builtin_memcpy(v.w, e, sizeof(v.w));
    }
}
template <class T>
__device__ __forceinline__ void settle(uint32_t c, uint32_t n, Eight<T> &v, float (&f)[8]) {
    unpack(v.w, f, T{});
    const uint32_t from = n >= 8 ? min(c, n - 8) : 0u;
    if (c == from) return;
    const uint32_t by = c - from;  // the elements before c
#pragma unroll
    for (int s = 1; s < 8; s *= 2) {
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] = by & s ? (i + s < 8 ? f[i + s] : 0.0f) : f[i];
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = by >= 8 ? 0.0f : f[i];
}

// load8, of which only `count` elements (below 8, possibly none) exist; the
// others read as `fill`.
template <class T>
__device__ __forceinline__ void load_part(const T *p, int count, float fill, float (&f)[8]) {
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = i < count ? (float)p[i] : fill;
}

template <class T>
__device__ __forceinline__ void load_upto8(const T *p, int64_t left, float fill, float (&f)[8]) {
    if (left >= 8) load8(p, f);
    else load_part(p, (int)left, fill, f);
}

// Makes the compiler take a value as new, so that what it derived from it before
// (here: the row in fp32) is not kept in registers for its next use.
__device__ __forceinline__ void keep(uint32_t &v) { asm volatile("" : "+v"(v)); }

// Two at a time: gfx950 rounds a pair to bfloat16 in one instruction.
template <class T>
__device__ __forceinline__ void store8(T *p, const float (&f)[8]) {
    typedef float pair32 __attribute__((ext_vector_type(2)));
    typedef T pair __attribute__((ext_vector_type(2)));
    pair v[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = __builtin_convertvector((pair32){f[2 * i], f[2 * i + 1]}, pair);
    __builtin_memcpy(p, v, sizeof(v));
}

// Reductions over a wave in registers: rows of 16 lanes by shifts, then the rows'
// last lanes broadcast on. Lane 63 has the result, which all lanes get.
template <int CTRL, int ROWS>
__device__ __forceinline__ uint32_t dpp(uint32_t none, uint32_t v) {
    return (uint32_t)__builtin_amdgcn_update_dpp((int)none, (int)v, CTRL, ROWS, 0xf, false);
}
template <class F>
__device__ __forceinline__ uint32_t wave_reduce(uint32_t v, uint32_t none, F f) {
    v = f(v, dpp<0x111, 0xf>(none, v));  // row_shr 1, 2, 4, 8
    v = f(v, dpp<0x112, 0xf>(none, v));
    v = f(v, dpp<0x114, 0xf>(none, v));
    v = f(v, dpp<0x118, 0xf>(none, v));
    v = f(v, dpp<0x142, 0xa>(none, v));  // row_bcast 15, 31
    v = f(v, dpp<0x143, 0xc>(none, v));
    return (uint32_t)__builtin_amdgcn_readlane((int)v, 63);
}
__device__ __forceinline__ uint32_t wave_max(uint32_t v) {
    return wave_reduce(v, 0u, [](uint32_t a, uint32_t b) { return max(a, b); });
}
__device__ __forceinline__ float wave_max(float v) {
    return __uint_as_float(wave_reduce(__float_as_uint(v), 0xff800000u, [](uint32_t a, uint32_t b) {
        return __float_as_uint(fmaxf(__uint_as_float(a), __uint_as_float(b)));
    }));
}
__device__ __forceinline__ float wave_sum(float v) {
    return __uint_as_float(wave_reduce(__float_as_uint(v), 0u, [](uint32_t a, uint32_t b) {
        return __float_as_uint(__uint_as_float(a) + __uint_as_float(b));
    }));
}

// A launch of `blocks` workgroups as a grid of two dimensions (one dimension of a
// grid holds fewer than 2^32 threads), and the workgroup's number in it, which
// may be past the last one.
inline dim3 grid_of(uint64_t blocks) {
    const uint64_t x = blocks < (1u << 20) ? blocks : (1u << 20);
    return dim3((uint32_t)x, (uint32_t)((blocks + x - 1) / x));
}
__device__ __forceinline__ uint64_t block_index() { return (uint64_t)blockIdx.y * gridDim.x + blockIdx.x; }

inline bool is_float(qsgd_dtype t) { return t == QSGD_F32 || t == QSGD_F16 || t == QSGD_BF16; }
inline uint64_t bytes_of(qsgd_dtype t) { return t == QSGD_F32 || t == QSGD_I32 ? 4 : t == QSGD_I64 ? 8 : 2; }
inline bool aligned_to(const void *p, uint64_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }
inline uint64_t round_up(uint64_t v, uint64_t to) { return (v + to - 1) / to * to; }
inline uint64_t div_up(uint64_t v, uint64_t by) { return (v + by - 1) / by; }
inline qsgd_status launched() { return hipGetLastError() == hipSuccess ? QSGD_OK : QSGD_ERR_LAUNCH; }

constexpr uint64_t kMaxDim = (1ull << 31) - 1;

// Calls f with a value of the element type.
template <class F>
qsgd_status with_type(qsgd_dtype t, F f) {
    switch (t) {
        case QSGD_F32: return f(float{});
        case QSGD_F16: return f(f16{});
        case QSGD_BF16: return f(bf16{});
        default: return QSGD_ERR_INVALID_ARG;
    }
}

}  // namespace ops
}  // namespace qsgd
