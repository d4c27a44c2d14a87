// quantize.hpp -- row quantisation to 8-bit codes, as a device function: a kernel
// of its own (int8.hip), and a part of the selection's launch (moe.hip).
//
//   s = max|x| / 127,  q = round(127 x / max|x|)
//
// 16 values of a row per thread and step (16-byte code stores).  127 x is
// exact for BF16 x, so that x = max|x| / 2 is a true tie (63.5, to 64); the
// division is the correctly rounded one.  Rows whose largest value is beyond
// 2^120 are scaled by 2^-8 first (exact), so that 127 x stays finite.  A row
// that holds an infinity or NaN gets scale NaN and codes 0: every product
// with it is NaN, and no other row's is.

#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "internal.hpp"

namespace drgg {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

template <bool BF16>
__device__ __forceinline__ void load16(float (&f)[16], const void* X, int64_t i) {
    if constexpr (BF16) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const u32x4 v = reinterpret_cast<const u32x4*>(X)[2 * i + h];
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                f[8 * h + 2 * r] = __uint_as_float(v[r] << 16);
                f[8 * h + 2 * r + 1] = __uint_as_float(v[r] & 0xFFFF0000u);
            }
        }
    } else {
#pragma unroll
        for (int h = 0; h < 4; ++h) {
            const f32x4 v = reinterpret_cast<const f32x4*>(X)[4 * i + h];
#pragma unroll
            for (int r = 0; r < 4; ++r) f[4 * h + r] = v[r];
        }
    }
}

// HELD: a thread's values of the row (at most 16) stay in registers between
// the maximum and the codes; longer rows are read again, from L2.  Bound by
// memory: 504 MB for 131072 FP32 rows of 768 in 87 us (5.8 TB/s), 101 MB for
// 16384 BF16 rows of 2048 in 26 us, 94 and 30 us when the row is read twice.
//
// Thread (x, y) of a workgroup of nx * ny, which is number `block` of `blocks`:
// nx (a power of two, at most 256) threads along a row, ny rows at a time.
// part: a word of LDS per wave.  Called by all threads.
template <bool BF16, bool HELD>
__device__ __forceinline__ void quantize_rows(const QuantArgs& a, uint32_t* part, int x, int y, int nx, int ny,
                                              int64_t block, int64_t blocks) {
    const int64_t R = a.T * a.k;
    // whole blocks of rows: every thread takes part in the maxima
    for (int64_t t0 = block * ny; t0 < a.T; t0 += blocks * ny) {
        const int64_t t = t0 + y;
        const bool live = t < a.T;
        // the largest magnitude as bits: their unsigned order is the order of
        // the magnitudes, with infinity and NaN above every finite value
        uint32_t m = 0;
        float f[16];
        if (live)
            for (int64_t c = x; c < a.C; c += nx) {
                load16<BF16>(f, a.X, t * a.C + c);
#pragma unroll
                for (int i = 0; i < 16; ++i) m = max(m, __float_as_uint(f[i]) & 0x7FFFFFFFu);
                if constexpr (HELD) break;
            }
        const int width = nx < 64 ? nx : 64;
        for (int d = 1; d < width; d <<= 1) m = max(m, (uint32_t)__shfl_xor((int)m, d, 64));
        if (nx > 64) {
            const int tid = y * nx + x;
            __syncthreads();   // the last rows' maxima have been read
            if ((tid & 63) == 0) part[tid >> 6] = m;
            __syncthreads();
            const int w0 = y * (nx / 64);
            for (int w = 0; w < nx / 64; ++w) m = max(m, part[w0 + w]);
        }
        const bool bad = m >= 0x7F800000u;
        const float most = __uint_as_float(m);
        const float scale = bad ? __uint_as_float(0x7FC00000u) : most / 127.f;
        const float down = most > 0x1p120f ? 0x1p-8f : 1.f;
        const float by = bad || m == 0 ? 1.f : most * down;
        for (int64_t c = x; live && c < a.C; c += nx) {
            if constexpr (!HELD) load16<BF16>(f, a.X, t * a.C + c);
            u32x4 out;
#pragma unroll
            for (int h = 0; h < 4; ++h) {
                uint32_t v = 0;
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const int q = bad ? 0 : (int)rintf(f[4 * h + r] * down * 127.f / by);
                    v |= (uint32_t)(q & 0xFF) << (8 * r);
                }
                out[h] = v;
            }
            for (int j = 0; j < a.k; ++j) {
                const int64_t p = a.positions ? a.positions[t * a.k + j] : t;
                if (p < 0 || p >= R) continue;
                reinterpret_cast<u32x4*>(a.q)[p * a.C + c] = out;
                if (c == 0) a.scale[p] = scale;
            }
            if constexpr (HELD) break;
        }
    }
}

// threads along a row of C groups
inline unsigned quantize_threads(int64_t C) {
    unsigned x = 1;
    while (x < 256 && x < C) x *= 2;
    return x;
}

}  // namespace drgg
