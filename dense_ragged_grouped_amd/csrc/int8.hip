// int8.hip -- gfx950 (CDNA4) kernels of the 8-bit integer products:
//
//   quantisation   s = max|x| / 127,  q = round(127 x / max|x|)   per row
//   product        Y[t,n] = xs[t] ws[e,n] sum_k Xq[t,k] Wq[e,n,k]
//   gated product  Y[t,i] = silu(g) u,  g, u = columns i and N/2 + i of the product
//
// The sum is an exact 32-bit integer (K <= kInt8MaxK), so no order or split
// of it changes a result; it is scaled in FP32 and rounded once.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "engine.hpp"
#include "internal.hpp"
#include "plan.hpp"
#include "quantize.hpp"

namespace drgg {

namespace {

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

// quantisation (quantize.hpp): blockDim.x threads along a row
template <bool BF16, bool HELD>
__global__ __launch_bounds__(256) void quantize_int8_kernel(QuantArgs a) {
    __shared__ uint32_t part[4];
    quantize_rows<BF16, HELD>(a, part, threadIdx.x, threadIdx.y, blockDim.x, blockDim.y, blockIdx.x, gridDim.x);
}

// ---------------------------------------------------------------------------
// product, few rows per group
//
// A workgroup computes a block of 16*NB weight rows (gated: 8*NB gate rows and
// their up rows) and up to TOK = 32 or 64 tokens of one group; its W waves
// split K in steps of 64 values, each computing the whole block, and add their
// integer sums through LDS.  Fragments go from memory to registers directly:
// lane l of a v_mfma_i32_16x16x64_i8 holds values 16*(l/16) .. +15 of row
// l%16, one 16-byte load, for the weights (first operand) as for the tokens;
// the result has token l%16 and weight rows 4*(l/16) .. +3 in lane l.  There
// is no barrier before the sums and a long reduction is W times shorter for
// each wave, which is what counts while few blocks or few rows leave the CUs
// idle; with more rows the tiles below move fewer bytes per product.
//
// Blocks of tokens are 16, 32 or 64 long by what is left of the group; U steps
// are loaded before the first is used.  Rows and reduction positions outside
// the operands carry an out-of-range offset and read as zero.  int8_program
// (plan.hpp) says which NB, W and TOK run when.
//
// Bound by the weights' bytes on many experts (64 rows on 32 of 1536x2048, 88
// MB: 17 us, 5.0 TB/s), by latency on one (one row through 4096x4096: 6 us).

// The block of this workgroup among those of all groups (ntn column blocks
// times ceil(T_e / TOK) token blocks each, token blocks innermost: their
// weights are then read by one XCD), or false.  Every wave finds it by
// itself: lane i holds group i of 64.
struct RowsItem {
    int e, nt;
    int64_t m0, hi;
};
template <int TOK>
__device__ __forceinline__ bool find_rows_item(const Int8Args& a, int32_t ntn, RowsItem* it) {
    const int lane = threadIdx.x & 63;
    auto bounds = [&](int e, int64_t* lo, int64_t* hi) {
        if (!a.offs) {
            *lo = 0;
            *hi = a.M;
        } else {
            *lo = min<int64_t>(max<int64_t>(a.offs[e], 0), a.M);
            *hi = min<int64_t>(max<int64_t>(a.offs[e + 1], *lo), a.M);
        }
    };
    auto items = [&](int e) {
        int64_t lo, hi;
        bounds(e, &lo, &hi);
        return (int32_t)((hi - lo + TOK - 1) / TOK) * ntn;
    };
    int32_t total = 0;
    for (int e0 = 0; e0 < a.E; e0 += 64)
        total += __shfl(wave_incl_sum(e0 + lane < a.E ? items(e0 + lane) : 0), 63, 64);
    total = uni(total);
    if ((int64_t)blockIdx.x >= total) return false;
    int32_t w = (int32_t)xcd_remap(blockIdx.x, total);
    for (int e0 = 0;; e0 += 64) {   // ends: w < total
        const int32_t n = e0 + lane < a.E ? items(e0 + lane) : 0;
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

// the scale of product row t (0 for a gathered row that is none)
template <bool GATHERED>
__device__ __forceinline__ float x_scale(const Int8Args& a, int64_t t) {
    if constexpr (!GATHERED) return a.xs[t];
    const int32_t from = a.rows[t];
    return (uint32_t)from < (uint32_t)a.T ? a.xs[from] : 0.f;
}

template <bool OUT_BF16, bool GATED, bool GATHERED, int NB, int MB, int W, int U>
__device__ __forceinline__ void int8_rows_block(const Int8Args& a, const RowsItem& it, i32x4 (&sums)[W][NB][64]) {
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int r = lane & 15, g = lane >> 4;
    const int64_t NO = GATED ? a.N / 2 : a.N;
    constexpr int NC = GATED ? NB / 2 : NB;          // blocks of 16 output columns
    const int64_t n0 = (int64_t)it.nt * 16 * NC;
    const int K = (int)a.K;
    const auto rx = make_rsrc(GATHERED ? a.X : a.X + it.m0 * a.K);
    const int8_t* w0 = a.W + ((int64_t)it.e * a.N + n0) * a.K;
    const auto rw = make_rsrc(w0);
    const auto rw2 = make_rsrc(GATED ? w0 + NO * a.K : w0);
    // a row's byte offset; reduction values it has from this lane's 16 on
    int off[4], xoff[MB], xk[MB], wk[NC];
#pragma unroll
    for (int b = 0; b < 4; ++b) off[b] = (16 * b + r) * K + 16 * g;
#pragma unroll
    for (int b = 0; b < MB; ++b) {
        const bool ok = it.m0 + 16 * b + r < it.hi;
        xoff[b] = off[b];
        xk[b] = ok ? K - 16 * g : 0;
        if constexpr (GATHERED) {   // T * K < 2^31
            const int32_t from = ok ? a.rows[it.m0 + 16 * b + r] : -1;
            if ((uint32_t)from < (uint32_t)a.T) xoff[b] = from * K + 16 * g;
            else xk[b] = 0;
        }
    }
#pragma unroll
    for (int b = 0; b < NC; ++b) wk[b] = n0 + 16 * b + r < NO ? K - 16 * g : 0;
    i32x4 acc[NB][MB] = {};
    for (int k0 = wave * 64; k0 < K; k0 += 64 * W * U) {
        u32x4 fx[U][MB], fw[U][NB];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int k = k0 + 64 * W * u;
#pragma unroll
            for (int b = 0; b < NB; ++b)
                fw[u][b] = __builtin_amdgcn_raw_buffer_load_b128(b < NC ? rw : rw2,
                                                                 k < wk[b % NC] ? (uint32_t)(off[b % NC] + k) : kOOB, 0, 0);
#pragma unroll
            for (int b = 0; b < MB; ++b)
                fx[u][b] = __builtin_amdgcn_raw_buffer_load_b128(rx, k < xk[b] ? (uint32_t)(xoff[b] + k) : kOOB, 0, 0);
        }
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int b = 0; b < NB; ++b)
#pragma unroll
                for (int m = 0; m < MB; ++m)
                    acc[b][m] = __builtin_amdgcn_mfma_i32_16x16x64_i8(__builtin_bit_cast(i32x4, fw[u][b]),
                                                                      __builtin_bit_cast(i32x4, fx[u][m]), acc[b][m], 0, 0, 0);
    }
    // the waves' sums, one block of 16 tokens at a time
#pragma unroll
    for (int m = 0; m < MB; ++m) {
        if (m > 0) __syncthreads();
#pragma unroll
        for (int b = 0; b < NB; ++b) sums[wave][b][lane] = acc[b][m];
        __syncthreads();
        if (wave >= NC) continue;
        i32x4 c0 = sums[0][wave][lane], c1 = c0;
        if constexpr (GATED) c1 = sums[0][NC + wave][lane];
#pragma unroll
        for (int v = 1; v < W; ++v) {
            c0 += sums[v][wave][lane];
            if constexpr (GATED) c1 += sums[v][NC + wave][lane];
        }
        const int64_t t = it.m0 + 16 * m + r, n = n0 + 16 * wave + 4 * g;
        if (t < it.hi && n < NO) {   // NO is a multiple of 4
            const float xs = x_scale<GATHERED>(a, t);
            const float* ws = a.ws + (int64_t)it.e * a.N + n;
            const f32x4 s0 = *reinterpret_cast<const f32x4*>(ws);
            f32x4 y, s1 = s0;
            if constexpr (GATED) s1 = *reinterpret_cast<const f32x4*>(ws + NO);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                y[i] = (float)c0[i] * s0[i] * xs;
                if constexpr (GATED) y[i] = gate(y[i], (float)c1[i] * s1[i] * xs);
            }
            if constexpr (OUT_BF16)
                *reinterpret_cast<u32x2*>(static_cast<uint16_t*>(a.out) + t * NO + n) =
                    u32x2{pack_bf16(y[0], y[1]), pack_bf16(y[2], y[3])};
            else
                *reinterpret_cast<f32x4*>(static_cast<float*>(a.out) + t * NO + n) = y;
        }
    }
}

// With TOK = 32 at most 80 registers (six waves per SIMD), so that the blocks
// of many experts are resident at once.
template <bool OUT_BF16, bool GATED, bool GATHERED, int NB, int W, int TOK>
__global__ __launch_bounds__(64 * W, TOK == 32 ? 6 : 2) void int8_rows_kernel(Int8Args a) {
    __shared__ i32x4 sums[W][NB][64];
    RowsItem it;
    const int64_t NO = GATED ? a.N / 2 : a.N;
    constexpr int kCols = 16 * (GATED ? NB / 2 : NB);
    if (!find_rows_item<TOK>(a, (int32_t)((NO + kCols - 1) / kCols), &it)) return;
    const int64_t left = it.hi - it.m0;
    if constexpr (TOK == 32) {
        if (left <= 16) int8_rows_block<OUT_BF16, GATED, GATHERED, NB, 1, W, 2>(a, it, sums);
        else int8_rows_block<OUT_BF16, GATED, GATHERED, NB, 2, W, 1>(a, it, sums);
    } else {
        if (left <= 16) int8_rows_block<OUT_BF16, GATED, GATHERED, NB, 1, W, 4>(a, it, sums);
        else if (left <= 32) int8_rows_block<OUT_BF16, GATED, GATHERED, NB, 2, W, 4>(a, it, sums);
        else int8_rows_block<OUT_BF16, GATED, GATHERED, NB, 4, W, 2>(a, it, sums);
    }
}

template <bool GATED, int NB, int W, int TOK>
hipError_t launch_int8_rows(const Int8Args& a, bool bf16, hipStream_t s) {
    const int64_t ntn = ceil_div(GATED ? a.N / 2 : a.N, 16 * (GATED ? NB / 2 : NB));
    // ceil(T_e / TOK) over the groups is at most M / TOK and one for each group with rows
    const int64_t most = (a.M / TOK + (a.M < a.E ? a.M : a.E)) * ntn;
    const dim3 grid((unsigned)most), block(64 * W);
    timing_mark("int8_rows_kernel", s);
    if (a.rows) {
        if (bf16) hipLaunchKernelGGL((int8_rows_kernel<true, GATED, true, NB, W, TOK>), grid, block, 0, s, a);
        else hipLaunchKernelGGL((int8_rows_kernel<false, GATED, true, NB, W, TOK>), grid, block, 0, s, a);
    } else {
        if (bf16) hipLaunchKernelGGL((int8_rows_kernel<true, GATED, false, NB, W, TOK>), grid, block, 0, s, a);
        else hipLaunchKernelGGL((int8_rows_kernel<false, GATED, false, NB, W, TOK>), grid, block, 0, s, a);
    }
    timing_end(s);
    return hipGetLastError();
}

// ---------------------------------------------------------------------------
// product, many rows per group

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

// The BF16 forward's persistent tile walk and main loop (engine.hpp) on 8-bit
// elements: the same bytes per step, twice the products.  A gated tile's
// columns are BN/2 gate rows of W and their BN/2 up rows in alternating
// blocks of 32 (a paired operand), so that a lane holds a gate and its up in
// the accumulators of neighbouring blocks.  The epilogue scales (and gates)
// the sums as they pass to the staged whole-line stores.
//
// 131072x1536x2048 in 8 groups, BF16 out: 407 to 462 us from run to run (2.0 to
// 1.8 POP/s; a large library product reaches 2.1 to 2.3 on this card).  Of a 256x256 tile's time
// 0.83 us per 64 reduction values are the main loop (2.4 POP/s; 20 % faster on
// zeros, so a part of it is the clock under load, the rest the loads' path as
// in BF16) and about 6.7 us its epilogue and switch: without the global stores
// the call takes 384 us, without the epilogue 355.
//
// 128x128 tiles share a CU in pairs, so their four waves get at most 256 of a
// SIMD's 512 registers per lane (unbounded, the gathered FP32 variants took 260
// and had a CU each: E = 57, gated, 20976x544x816 gathered 43.8 instead of 31.2 us).
template <int BM, int BN, bool OUT_BF16, bool GATED, bool GATHERED, int WAVES>
__global__ __launch_bounds__(64 * WAVES, BM == 128 && BN == 128 ? 2 : 1) void int8_tile_kernel(Int8Args a) {
    DRGG_STAGES(BM, BN, true, true, stg);
    __shared__ SchedOf<16> sch;
    __shared__ __attribute__((aligned(16))) char ep[WAVES * ep_rows(BM, BN) * 128];
    using Mma = TileMma<BM, BN, true, true, WAVES, Int8>;
    constexpr int BC = GATED ? BN / 2 : BN;             // output columns per tile
    constexpr int NJ = GATED ? Mma::kBJ / 2 : Mma::kBJ; // blocks of 32 of them per wave
    const int64_t NO = GATED ? a.N / 2 : a.N, K2 = a.K / 2;
    const int32_t ntn = (int32_t)((NO + BC - 1) / BC);
    build_schedule(sch, a.offs, a.E, a.M, a.M, [=](int, int32_t T) { return ceil_div32(T, BM) * ntn; });
    const int64_t total = uni(sch.prefix[a.E]);
    const int64_t G = gridDim.x;
    int64_t w = xcd_remap(blockIdx.x, G);
    auto more = [&]() { return w < total; };
    auto next = [&](TileInfo& t) {
        const int e = uni(find_expert(sch, a.E, (int32_t)w));
        const int32_t oe = uni(sch.offs[e]), oe1 = uni(sch.offs[e + 1]);
        const int32_t local = (int32_t)w - uni(sch.prefix[e]);
        const int32_t mt = local / ntn, nt = local % ntn;
        t.o0 = oe + (int64_t)mt * BM;
        t.o1 = (int64_t)nt * BC;
        t.rows = (int32_t)min<int64_t>(BM, oe1 - t.o0);
        t.cols = (int32_t)min<int64_t>(BC, NO - t.o1);
        t.e = e;
        t.A = GATHERED ? Operand{reinterpret_cast<const uint16_t*>(a.X), K2, t.rows, (int32_t)K2, 0, a.rows + t.o0, a.T}
                       : Operand{reinterpret_cast<const uint16_t*>(a.X + t.o0 * a.K), K2, t.rows, (int32_t)K2};
        t.B = Operand{reinterpret_cast<const uint16_t*>(a.W + ((int64_t)e * a.N + t.o1) * a.K), K2, t.cols,
                      (int32_t)K2, NO * a.K};
        w += G;
    };
    // A tile's scales: BM of its tokens, then BN of its weight rows (gated:
    // BN/2 gate, then BN/2 up), 64 per wave load.  Two buffers: the next
    // tile's land while the current one is computed.  Positions past the
    // tile's rows and columns hold zeros.
    __shared__ __attribute__((aligned(256))) float scales[2][BM + BN];
    int put = 0, got = 0;
    auto loads = [&](const TileInfo& t) {
        const int lane = threadIdx.x & 63;
        const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
        const float* ws = a.ws + (int64_t)t.e * a.N + t.o1;
#pragma unroll
        for (int c0 = 0; c0 < BM + BN; c0 += 64 * WAVES) {
            const int c = c0 + wave * 64;   // of the tile's BM + BN scales
            if (c >= BM + BN) break;
            const bool up = GATED && c >= BM + BC;
            const float* from = c < BM ? a.xs + t.o0 + c : ws + (up ? NO - BC : 0) + (c - BM);
            const int left = c < BM ? t.rows - c : t.cols - (c - BM - (up ? BC : 0));
            uint32_t at = lane < left ? lane * 4 : kOOB;
            if (GATHERED && c < BM) {
                const int32_t row = lane < left ? a.rows[t.o0 + c + lane] : -1;
                at = (uint32_t)row < (uint32_t)a.T ? (uint32_t)row * 4 : kOOB;
                from = a.xs;
            }
            __builtin_amdgcn_raw_ptr_buffer_load_lds(make_rsrc(from), (lds_void_t*)((lds_t*)scales[put] + c * 4), 4, at, 0,
                                                     0, 0);
        }
        put ^= 1;
    };
    auto finish = [&](const TileInfo& t, const Mma& mma) {
        int lane = threadIdx.x & 63;
        asm volatile("" : "+v"(lane));
        const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
        const int rb = GATED ? Mma::wave_col(wave) / 2 : Mma::wave_col(wave);
        typedef const __attribute__((address_space(3))) float lds_f32;
        typedef const __attribute__((address_space(3))) f32x4 lds_f32x4;
        const lds_t* sc = (const lds_t*)scales[got];
        got ^= 1;
        float sx[Mma::kBI];
#pragma unroll
        for (int i = 0; i < Mma::kBI; ++i)
            sx[i] = *reinterpret_cast<lds_f32*>(sc + 4 * (Mma::wave_row(wave) + 32 * i + (lane & 31)));
        const lds_t* sw = sc + 4 * (BM + rb + 4 * (lane >> 5));
        auto value = [&](int i, int j, int q) {
            const f32x4 w = *reinterpret_cast<lds_f32x4*>(sw + 4 * (32 * j + 8 * q));
            f32x4 y;
            if constexpr (GATED) {
                const f32x4 v = *reinterpret_cast<lds_f32x4*>(sw + 4 * (BC + 32 * j + 8 * q));
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    y[r] = gate((float)mma.acc[i][2 * j][4 * q + r] * w[r] * sx[i],
                                (float)mma.acc[i][2 * j + 1][4 * q + r] * v[r] * sx[i]);
            } else {
#pragma unroll
                for (int r = 0; r < 4; ++r) y[r] = (float)mma.acc[i][j][4 * q + r] * w[r] * sx[i];
            }
            return y;
        };
        const int64_t o = t.o0 * NO + t.o1;
        void* base = OUT_BF16 ? (void*)(static_cast<uint16_t*>(a.out) + o) : (void*)(static_cast<float*>(a.out) + o);
        store_tile_values<OUT_BF16, ep_rows(BM, BN), Mma, NJ>(value, rb, (lds_t*)ep, base, NO, t.rows, t.cols);
    };
    TileRunner<BM, BN, true, true, WAVES, Int8, GATED, GATHERED> runner;
    runner.st = stg;
    runner.run(more, next, finish, loads);
}

template <int BM, int BN, int WAVES, bool GATED, bool GATHERED>
void launch_int8_tile_t(const Int8Args& a, bool bf16, dim3 grid, hipStream_t s) {
    const dim3 block(64 * WAVES);
    constexpr bool kBf16 = !GATED || BN >= 256;   // a gated 128x128 tile has 32 columns per wave, half a BF16 line
    if constexpr (kBf16)
        if (bf16) {
            hipLaunchKernelGGL((int8_tile_kernel<BM, BN, true, GATED, GATHERED, WAVES>), grid, block, 0, s, a);
            return;
        }
    hipLaunchKernelGGL((int8_tile_kernel<BM, BN, false, GATED, GATHERED, WAVES>), grid, block, 0, s, a);
}

template <int BM, int BN, int WAVES>
hipError_t launch_int8_tile(const Int8Args& a, bool gated, bool bf16, int64_t grid_n, hipStream_t s) {
    const dim3 grid((unsigned)grid_n);
    timing_mark("int8_tile_kernel", s);
    if (gated && a.rows) launch_int8_tile_t<BM, BN, WAVES, true, true>(a, bf16, grid, s);
    else if (gated) launch_int8_tile_t<BM, BN, WAVES, true, false>(a, bf16, grid, s);
    else if (a.rows) launch_int8_tile_t<BM, BN, WAVES, false, true>(a, bf16, grid, s);
    else launch_int8_tile_t<BM, BN, WAVES, false, false>(a, bf16, grid, s);
    timing_end(s);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_quantize_int8(const void* X, bool bf16, int64_t T, int64_t K, const int32_t* positions, int32_t k,
                                int8_t* q, float* scale, hipStream_t s) {
    QuantArgs a{X, positions, q, scale, T, K / 16, k};
    const unsigned x = quantize_threads(a.C);
    // a launch has fewer than 2^32 threads: blocks walk the rows beyond
    const dim3 block(x, 256 / x);
    const int64_t n = ceil_div(T, block.y), most = 65536;
    const dim3 grid((unsigned)(n < most ? n : most));
    timing_mark("quantize_int8_kernel", s);
    if (a.C <= x) {
        if (bf16) hipLaunchKernelGGL((quantize_int8_kernel<true, true>), grid, block, 0, s, a);
        else hipLaunchKernelGGL((quantize_int8_kernel<false, true>), grid, block, 0, s, a);
    } else {
        if (bf16) hipLaunchKernelGGL((quantize_int8_kernel<true, false>), grid, block, 0, s, a);
        else hipLaunchKernelGGL((quantize_int8_kernel<false, false>), grid, block, 0, s, a);
    }
    timing_end(s);
    return hipGetLastError();
}

template <bool GATED>
hipError_t launch_int8_program(const Int8Args& a, const Int8Program& p, bool bf16, hipStream_t s) {
    if (p.tok == 32) return launch_int8_rows<GATED, 4, 4, 32>(a, bf16, s);
    if (p.waves == 4) return launch_int8_rows<GATED, 4, 4, 64>(a, bf16, s);
    if (p.nb == 4) return launch_int8_rows<GATED, 4, 8, 64>(a, bf16, s);
    if constexpr (!GATED)
        if (p.nb == 1) return launch_int8_rows<false, 1, 8, 64>(a, bf16, s);
    return launch_int8_rows<GATED, 2, 8, 64>(a, bf16, s);
}

hipError_t launch_int8(const Int8Args& a, bool gated, bool bf16, int cus, int forced_tile, hipStream_t s) {
    const Int8Program p = int8_program(a.E, a.M, a.N, a.K, gated, bf16, forced_tile);
    if (p.tile == kTileAuto)
        return gated ? launch_int8_program<true>(a, p, bf16, s) : launch_int8_program<false>(a, p, bf16, s);
    const int64_t cols_out = gated ? a.N / 2 : a.N, bc = gated ? 128 : 256;
    auto grid = [&](int64_t bm, int64_t bcols, int64_t per_cu) {
        const int64_t most = (a.M / bm + (a.M < a.E ? a.M : a.E)) * ceil_div(cols_out, bcols);
        return most < per_cu * cus ? most : per_cu * cus;
    };
    if (p.tile == kTile256x256) return launch_int8_tile<256, 256, 8>(a, gated, bf16, grid(256, bc, 1), s);
    if (p.tile == kTile128x256) return launch_int8_tile<128, 256, 4>(a, gated, bf16, grid(128, bc, 1), s);
    return launch_int8_tile<128, 128, 4>(a, gated, bf16, grid(128, bc / 2, 2), s);
}

}  // namespace drgg
