// mxfp4.hpp -- quantisation to microscaled 4-bit floating point, as device
// functions: a kernel of its own and the gated product's epilogue (mxfp4.hip),
// and a part of the selection's launch (moe.hip).
//
// b = floor(log2 max|x|) + 125 of a block of 32, code = nearest(x / 2^(b - 127)).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "internal.hpp"

namespace drgg {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

// v of lane l ^ 1, l ^ 2
__device__ __forceinline__ uint32_t quad_max(uint32_t v) {
    v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0xB1, 0xF, 0xF, false));
    return max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x4E, 0xF, 0xF, false));
}
// or over the row of 16 of values that agree within each quad
__device__ __forceinline__ uint32_t or_quads(uint32_t v) {
    v |= (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x124, 0xF, 0xF, false);
    return v | (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x128, 0xF, 0xF, false);
}

// The scale byte for a largest magnitude given as bits: its exponent field
// less 2 (the largest code is 1.5 * 2^2), 255 for infinity and NaN.
__device__ __forceinline__ uint32_t scale_byte(uint32_t most) {
    const int e = (int)(most >> 23);
    return e == 255 ? 255u : e > 2 ? (uint32_t)(e - 2) : 0u;
}
// 2^(127 - b), by which the values are multiplied, for a finite block (b is at
// most 252).  Exact; a result below FP32's normal range is far below half the
// smallest code.
__device__ __forceinline__ float scale_inverse(uint32_t b) { return __uint_as_float((254u - b) << 23); }
// eight codes, the first in the lowest bits.  The conversion rounds to the
// nearest code, ties to even, and limits to 6.
__device__ __forceinline__ uint32_t codes8(const float (&y)[8]) {
    uint32_t q = 0;
    q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, y[0], y[1], 1.f, 0);
    q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, y[2], y[3], 1.f, 1);
    q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, y[4], y[5], 1.f, 2);
    return __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, y[6], y[7], 1.f, 3);
}

template <bool BF16>
__device__ __forceinline__ void load8(float (&f)[8], const void* X, int64_t i) {
    if constexpr (BF16) {
        const u32x4 v = reinterpret_cast<const u32x4*>(X)[i];
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            f[2 * r] = __uint_as_float(v[r] << 16);
            f[2 * r + 1] = __uint_as_float(v[r] & 0xFFFF0000u);
        }
    } else {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const f32x4 v = reinterpret_cast<const f32x4*>(X)[2 * i + h];
#pragma unroll
            for (int r = 0; r < 4; ++r) f[4 * h + r] = v[r];
        }
    }
}

// Columns 256 kb .. +255 of row t by half a wave: lane l has columns 8l .. 8l+7,
// four lanes a block of 32.  The maxima are two exchanges within quads; the codes
// leave as one dword per lane, the scales of 128 columns as one dword of the
// row of 16 lanes that holds them.  Called by whole waves; a row past the last
// writes nothing.
//
// Bound by memory: 49152 FP32 rows of 2048 (456 MB) in 88 us where other kernels'
// data lie between two calls (75 with the same rows again, part of them in the
// last-level cache), 131072 BF16 rows (680 MB) in 118 to 131 us: 5.2 and 5.2 to 5.8
// TB/s, a large copy reaches 5.0.
template <bool BF16>
__device__ __forceinline__ void quantize_mx_piece(const MxQuantArgs& a, int64_t t, int64_t kb) {
    const int l = threadIdx.x & 31;
    const int64_t c = 256 * kb + 8 * l;
    const bool live = t < a.T && c < a.K;
    float f[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    if (live) load8<BF16>(f, a.X, (t * a.K + c) / 8);
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(f[i]) & 0x7FFFFFFFu);
    const uint32_t b = scale_byte(quad_max(m));
    const float by = scale_inverse(b);
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = b == 255 ? 0.f : f[i] * by;
    if (live) reinterpret_cast<uint32_t*>(a.codes)[(t * a.K + c) / 8] = codes8(f);
    const uint32_t four = or_quads(live ? b << (8 * ((l >> 2) & 3)) : 0u);
    if ((l & 15) == 0 && t < a.T) reinterpret_cast<uint32_t*>(a.scales)[(kb * a.T + t) * 2 + (l >> 4)] = four;
}

}  // namespace drgg
