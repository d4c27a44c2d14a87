// products.hpp -- what the kernels of the 8-bit and 4-bit products (int8.hip,
// mxfp4.hip) share: the gate, the few-row programs' work items, and a tile
// epilogue whose values are made on the way.  Included by kernel files only.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "engine.hpp"

namespace drgg {

typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
    typedef float f32x2 __attribute__((ext_vector_type(2)));
    return __builtin_bit_cast(uint32_t, __builtin_convertvector((f32x2{lo, hi}), bf16x2));
}

// silu(g) u = g u / (1 + exp(-g)).  The exponential and the reciprocal are the
// hardware's, within 1 ulp each; the exponential's argument is rounded before,
// which moves the result by |g| 2^-24 of it, a third of what the three roundings
// of g itself (the sum, two scales) do.  Below g = -87 the sigmoid leaves FP32's
// normal range and the result is 0, off by less than 2^-100 |g u|.  With the
// library's expf and a correctly rounded division the gate was the larger part
// of the gated product's epilogue.
__device__ __forceinline__ float gate(float g, float u) {
    return g * __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(g * -1.44269504f)) * u;
}

// The block of this workgroup among those of all groups (ntn column blocks
// times ceil(T_e / TOK) token blocks each, token blocks innermost: their
// weights are then read by one XCD), or false.  Every wave finds it by
// itself: lane i holds group i of 64.
struct RowsItem {
    int e, nt;
    int64_t m0, hi;
};
template <int TOK>
__device__ __forceinline__ bool find_rows_item(const int32_t* offs, int32_t E, int64_t M, int32_t ntn, RowsItem* it) {
    const int lane = threadIdx.x & 63;
    auto bounds = [&](int e, int64_t* lo, int64_t* hi) {
        if (!offs) {
            *lo = 0;
            *hi = M;
        } else {
            *lo = min<int64_t>(max<int64_t>(offs[e], 0), M);
            *hi = min<int64_t>(max<int64_t>(offs[e + 1], *lo), M);
        }
    };
    auto items = [&](int e) {
        int64_t lo, hi;
        bounds(e, &lo, &hi);
        return (int32_t)((hi - lo + TOK - 1) / TOK) * ntn;
    };
    int32_t total = 0;
    for (int e0 = 0; e0 < E; e0 += 64)
        total += __shfl(wave_incl_sum(e0 + lane < E ? items(e0 + lane) : 0), 63, 64);
    total = uni(total);
    if ((int64_t)blockIdx.x >= total) return false;
    int32_t w = (int32_t)xcd_remap(blockIdx.x, total);
    for (int e0 = 0;; e0 += 64) {   // ends: w < total
        const int32_t n = e0 + lane < E ? items(e0 + lane) : 0;
        const int32_t incl = wave_incl_sum(n);
        const unsigned long long past = __ballot(incl > w);
        if (past) {
            const int l = __ffsll((long long)past) - 1;
            it->e = e0 + l;
            w -= uni(__shfl(incl - n, l, 64));
            break;
        }
        w -= uni(__shfl(incl, 63, 64));
    }
    int64_t lo;
    bounds(it->e, &lo, &it->hi);
    const int32_t rt = (int32_t)((it->hi - lo + TOK - 1) / TOK);
    it->nt = w / rt;
    it->m0 = lo + (int64_t)(w % rt) * TOK;
    return true;
}

// Write a finished tile as store_tile_lines (engine.hpp) does, from values that
// are made on the way: value(i, j, q) gives the four of row block i at columns
// 32j + 8q + 4*(lane/32) .. +3 of the wave's part, which starts at column rb
// and has NJ blocks of 32.  A segment's values are made by all lanes before its
// rounds, in which only the lanes that own a round's rows write (made inside
// the rounds they would cost 32/R times the instructions: 131072x1536x2048 428
// instead of 407 us).
template <bool OUT_BF16, int R, class Mma, int NJ, class Value>
__device__ __forceinline__ void store_tile_values(Value value, int rb, lds_t* scr, void* out, int64_t ld, int rows,
                                                  int cols) {
    typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
    typedef float f32x2 __attribute__((ext_vector_type(2)));
    typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
    constexpr int ES = OUT_BF16 ? 2 : 4;
    constexpr int SEG = 128 / ES;   // columns per 128-byte segment
    constexpr int BPS = SEG / 32;   // 32-column blocks per segment
    static_assert(R == 8 || R == 16, "rounds of 8 or 16 rows");
    static_assert(NJ % BPS == 0, "whole segments per wave");
    int lane = threadIdx.x & 63;
    asm volatile("" : "+v"(lane));
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int ra = Mma::wave_row(wave);
    lds_t* sw = scr + wave * (R * 128);
    const int r = lane & 31, h = lane >> 5;
    const int rr = r % R;   // this lane's scratch row in the round that owns it
    const int sx = rr & 7;
#pragma unroll
    for (int i = 0; i < Mma::kBI; ++i) {
        const int r0 = ra + 32 * i;
        const __amdgpu_buffer_rsrc_t rs = make_rsrc(reinterpret_cast<char*>(out) + (int64_t)r0 * ld * ES);
#pragma unroll
        for (int g = 0; g < NJ / BPS; ++g) {
            const int c0 = rb + g * SEG;
            u32x2 half[OUT_BF16 ? BPS : 1][4];
            u32x4 full[OUT_BF16 ? 1 : BPS][4];
#pragma unroll
            for (int b = 0; b < BPS; ++b)
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const f32x4 a = value(i, g * BPS + b, q);
                    if constexpr (OUT_BF16)
                        half[b][q] = u32x2{
                            __builtin_bit_cast(uint32_t, __builtin_convertvector((f32x2{a[0], a[1]}), bf16x2)),
                            __builtin_bit_cast(uint32_t, __builtin_convertvector((f32x2{a[2], a[3]}), bf16x2))};
                    else
                        full[b][q] = __builtin_bit_cast(u32x4, a);
                }
#pragma unroll
            for (int s = 0; s < 32 / R; ++s) {
                if (r / R == s) {
#pragma unroll
                    for (int b = 0; b < BPS; ++b)
#pragma unroll
                        for (int q = 0; q < 4; ++q) {
                            if constexpr (OUT_BF16)   // columns 32b + 8q + 4h .. +3: chunk 4b + q, its half h
                                *reinterpret_cast<__attribute__((address_space(3))) u32x2*>(
                                    sw + rr * 128 + (((4 * b + q) ^ sx) << 4) + 8 * h) = half[b][q];
                            else   // columns 8q + 4h .. +3: chunk 2q + h
                                *reinterpret_cast<__attribute__((address_space(3))) u32x4*>(
                                    sw + rr * 128 + (((2 * q + h) ^ sx) << 4)) = full[b][q];
                        }
                }
                wave_lds_sync();   // the round's rows are in the scratch
#pragma unroll
                for (int k = 0; k < R / 8; ++k) {
                    const int idx = lane + 64 * k, row = idx >> 3, c = idx & 7;
                    const u32x4 v = *reinterpret_cast<const __attribute__((address_space(3))) u32x4*>(
                        sw + row * 128 + ((c ^ (row & 7)) << 4));
                    const int rowb = s * R + row;            // row within the 32-row block
                    const int col = c0 + c * (16 / ES);
                    const uint32_t o = r0 + rowb < rows && col < cols ? (uint32_t)((rowb * ld + col) * ES) : kOOB;
                    __builtin_amdgcn_raw_buffer_store_b128(v, rs, o, 0, kCpolNT);
                }
                wave_lds_sync();   // read back before the next round overwrites it
            }
        }
    }
}

}  // namespace drgg
