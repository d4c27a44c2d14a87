// mxfp4.hip -- gfx950 (CDNA4) kernels of microscaled 4-bit floating point:
// blocks of 32 values along a row with a scale 2^(b - 127), elements of two
// exponent bits and one mantissa bit.
//
//   quantisation   b = floor(log2 max|x|) + 125,  code = nearest(x / 2^(b - 127))
//   product        Y[t,n] = sum over blocks of 2^(bx + bw - 254) <x, w>
//   gated product  Y[t,i] = silu(g) u,  g, u = columns i and N/2 + i of the product
//
// Codes are rows of K/2 bytes; the scale bytes of 256 columns (one line of 128
// code bytes) stand side by side, [ceil(K/256)][rows][8], so that the scales a
// tile needs are runs of memory and no row's scales are unaligned.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "engine.hpp"
#include "internal.hpp"
#include "mxfp4.hpp"
#include "plan.hpp"
#include "products.hpp"

namespace drgg {

namespace {

typedef int32_t i32x8 __attribute__((ext_vector_type(8)));

struct MxRowArgs {   // dequantisation
    const uint8_t* codes;
    const uint8_t* scales;
    void* X;
    int64_t T, K;
};

template <bool BF16>
__global__ __launch_bounds__(256) void quantize_mxfp4_kernel(MxQuantArgs a) {
    for (int64_t t0 = (int64_t)blockIdx.y * 8; t0 < a.T; t0 += (int64_t)gridDim.y * 8)
        quantize_mx_piece<BF16>(a, t0 + (threadIdx.x >> 5), blockIdx.x);
}

// The values of eight codes: converted with scale 1 and moved by the block's
// exponent, so that 2^-127, which is below FP32's normal range, needs no care.
template <bool BF16>
__global__ __launch_bounds__(256) void dequantize_mxfp4_kernel(MxRowArgs a) {
    typedef float f32x2 __attribute__((ext_vector_type(2)));
    const int l = threadIdx.x & 31;
    const int64_t kb = blockIdx.x, c = 256 * kb + 8 * l;
    if (c >= a.K) return;
    for (int64_t t = (int64_t)blockIdx.y * 8 + (threadIdx.x >> 5); t < a.T; t += (int64_t)gridDim.y * 8) {
        const uint32_t q = reinterpret_cast<const uint32_t*>(a.codes)[(t * a.K + c) / 8];
        const int b = a.scales[(kb * a.T + t) * 8 + (l >> 2)];
        const f32x2 p0 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q, 1.f, 0);
        const f32x2 p1 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q, 1.f, 1);
        const f32x2 p2 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q, 1.f, 2);
        const f32x2 p3 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q, 1.f, 3);
        float f[8] = {p0[0], p0[1], p1[0], p1[1], p2[0], p2[1], p3[0], p3[1]};
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] = b == 255 ? __uint_as_float(0x7FC00000u) : ldexpf(f[i], b - 127);
        if constexpr (BF16) {
            static_cast<u32x4*>(a.X)[(t * a.K + c) / 8] =
                u32x4{pack_bf16(f[0], f[1]), pack_bf16(f[2], f[3]), pack_bf16(f[4], f[5]), pack_bf16(f[6], f[7])};
        } else {
            f32x4* out = static_cast<f32x4*>(a.X) + (t * a.K + c) / 4;
            out[0] = f32x4{f[0], f[1], f[2], f[3]};
            out[1] = f32x4{f[4], f[5], f[6], f[7]};
        }
    }
}

// Workgroups of neighbouring columns follow one another, so that those running at
// once read whole rows (rows first, 131072 BF16 rows of 2048 took 164 instead of
// 126 us and their values 175 instead of 127).
dim3 mx_row_grid(int64_t T, int64_t K) {
    // a launch has fewer than 2^32 threads and 65536 rows of workgroups: they walk the rows beyond
    const int64_t kb = ceil_div(K, 256), n = ceil_div(T, 8), most = (int64_t(1) << 23) / kb;
    const int64_t y = n < most ? n : most;
    return dim3((unsigned)kb, (unsigned)(y < 65535 ? y : 65535));
}

// ---------------------------------------------------------------------------
// product, few rows per group
//
// The work items of the 8-bit few-row program (products.hpp): a workgroup
// computes a block of 16*NB weight rows (gated: 8*NB gate rows and their up
// rows) and up to TOK tokens of one group; its W waves split K in pieces of 256
// columns (one line of a row's codes, eight scale bytes), each computing the
// whole block, and add their sums through LDS in the waves' order.  Fragments
// go from memory to registers directly: lane l of a
// v_mfma_scale_f32_16x16x128_f8f6f4 holds the block of 32 columns 32*(l/16) ..
// +31 of row l%16, one 16-byte load, and that block's scale byte; the result
// has token l%16 and weight rows 4*(l/16) .. +3 in lane l.  A row's eight scale
// bytes of a piece are one load; the lane's two of them are permuted into bytes
// 0 and 1, which the two steps' MFMAs select.  Rows and columns outside the
// operands carry an out-of-range offset and read as zero.
//
// One row through 4096x4096 takes 5.0 us (8.9 MB, 1.8 us at the rate of a copy):
// latency.  32 rows on 32 experts of 1536x2048 10.5 us (about 33 MB, 6.6 us).

// What a product leaves: FP32 or BF16 values, or (gated) codes and scales, those
// of quantize_mxfp4 on the FP32 values, so that the next product's operand is made
// here: 131072 rows of 768 save 403 MB of writes and as much reading.
enum MxOut { kOutFp32, kOutBf16, kOutMx };

__device__ __forceinline__ i32x8 fragment(u32x4 v) {   // 4-bit elements fill half of the operand's registers
    const i32x4 a = __builtin_bit_cast(i32x4, v);
    return __builtin_shufflevector(a, a, 0, 1, 2, 3, -1, -1, -1, -1);
}

template <MxOut OUT, bool GATED, bool GATHERED, int NB, int MB, int W, int U>
__device__ __forceinline__ void mx_rows_block(const MxArgs& a, const RowsItem& it, f32x4 (&sums)[W][NB][64]) {
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int r = lane & 15, g = lane >> 4;
    const int64_t NO = GATED ? a.N / 2 : a.N;
    constexpr int NC = GATED ? NB / 2 : NB;          // blocks of 16 output columns
    const int64_t n0 = (int64_t)it.nt * 16 * NC;
    const int B = (int)(a.K / 2);                    // bytes per row
    const auto rx = make_rsrc(GATHERED ? a.X : a.X + it.m0 * B);
    const uint8_t* w0 = a.W + ((int64_t)it.e * a.N + n0) * B;
    const auto rw = make_rsrc(w0);
    const auto rw2 = make_rsrc(GATED ? w0 + NO * B : w0);
    // a row's byte offset, and bytes it has from this lane's 16 on
    int off[4], xk[MB], wk[NC];
    int32_t from[MB];   // rows of X; T * B < 2^31
#pragma unroll
    for (int b = 0; b < MB; ++b) {
        const bool ok = it.m0 + 16 * b + r < it.hi;
        xk[b] = ok ? B - 16 * g : 0;
        from[b] = GATHERED ? ok ? a.rows[it.m0 + 16 * b + r] : -1 : 16 * b + r;
    }
#pragma unroll
    for (int b = 0; b < 4; ++b) off[b] = (16 * b + r) * B + 16 * g;
#pragma unroll
    for (int b = 0; b < NC; ++b) wk[b] = n0 + 16 * b + r < NO ? B - 16 * g : 0;
    const int64_t xrows = GATHERED ? a.T : a.M, wrows = (int64_t)a.E * a.N;
    const uint8_t* xs0 = a.xs + (GATHERED ? 0 : it.m0 * 8);
    const uint8_t* ws0 = a.ws + ((int64_t)it.e * a.N + n0) * 8;
    const uint32_t pick = 0x0c0c0400u + 0x0101u * g;   // byte g of either dword
    f32x4 acc[NB][MB] = {};
    for (int k0 = wave * 128; k0 < B; k0 += 128 * W * U) {
        u32x4 fx[U][2][MB], fw[U][2][NB];
        u32x2 sx[U][MB], sw[U][NB];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int k = k0 + 128 * W * u;
            const auto rxs = make_rsrc(xs0 + (int64_t)(k >> 7) * xrows * 8);
            const uint8_t* wsk = ws0 + (int64_t)(k >> 7) * wrows * 8;
            const auto rws = make_rsrc(wsk), rws2 = make_rsrc(GATED ? wsk + NO * 8 : wsk);
#pragma unroll
            for (int b = 0; b < NB; ++b) {
#pragma unroll
                for (int s = 0; s < 2; ++s)
                    fw[u][s][b] = __builtin_amdgcn_raw_buffer_load_b128(
                        b < NC ? rw : rw2, k + 64 * s < wk[b % NC] ? (uint32_t)(off[b % NC] + k + 64 * s) : kOOB, 0, 0);
                sw[u][b] = __builtin_amdgcn_raw_buffer_load_b64(
                    b < NC ? rws : rws2, k < wk[b % NC] ? (uint32_t)(16 * (b % NC) + r) * 8 : kOOB, 0, 0);
            }
            // the tokens' rows after the weights: where they are gathered, their
            // indices arrive behind the first weights' loads
#pragma unroll
            for (int b = 0; b < MB; ++b) {
                const int left = !GATHERED || (uint32_t)from[b] < (uint32_t)a.T ? xk[b] - k : 0;
                const uint32_t at = (uint32_t)(from[b] * B + 16 * g + k);
#pragma unroll
                for (int s = 0; s < 2; ++s)
                    fx[u][s][b] = __builtin_amdgcn_raw_buffer_load_b128(rx, 64 * s < left ? at + 64 * s : kOOB, 0, 0);
                sx[u][b] = __builtin_amdgcn_raw_buffer_load_b64(rxs, 0 < left ? (uint32_t)from[b] * 8 : kOOB, 0, 0);
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            uint32_t px[MB], pw[NB];   // the lane's blocks of the two steps in bytes 0 and 1
#pragma unroll
            for (int b = 0; b < NB; ++b) pw[b] = __builtin_amdgcn_perm(sw[u][b][1], sw[u][b][0], pick);
#pragma unroll
            for (int m = 0; m < MB; ++m) px[m] = __builtin_amdgcn_perm(sx[u][m][1], sx[u][m][0], pick);
#pragma unroll
            for (int b = 0; b < NB; ++b)
#pragma unroll
                for (int m = 0; m < MB; ++m) {
                    acc[b][m] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
                        fragment(fw[u][0][b]), fragment(fx[u][0][m]), acc[b][m], 4, 4, 0, pw[b], 0, px[m]);
                    acc[b][m] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
                        fragment(fw[u][1][b]), fragment(fx[u][1][m]), acc[b][m], 4, 4, 1, pw[b], 1, px[m]);
                }
        }
    }
    // the waves' sums, one block of 16 tokens at a time
#pragma unroll
    for (int m = 0; m < MB; ++m) {
        if (m > 0) __syncthreads();
#pragma unroll
        for (int b = 0; b < NB; ++b) sums[wave][b][lane] = acc[b][m];
        __syncthreads();
        if constexpr (OUT == kOutMx) {
            // wave 0 finishes the block's 32 columns: lane l has columns 4*(l/16) .. +3 of
            // either half for token l%16
            static_assert(GATED && NC == 2, "a block of 32 columns per workgroup");
            if (wave > 0) continue;
            f32x4 y[2];
            uint32_t most = 0;
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                f32x4 v0 = sums[0][c][lane], v1 = sums[0][2 + c][lane];
#pragma unroll
                for (int v = 1; v < W; ++v) {
                    v0 += sums[v][c][lane];
                    v1 += sums[v][2 + c][lane];
                }
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    y[c][i] = gate(v0[i], v1[i]);
                    most = max(most, __float_as_uint(y[c][i]) & 0x7FFFFFFFu);
                }
            }
            most = max(most, (uint32_t)__shfl_xor((int)most, 16, 64));
            most = max(most, (uint32_t)__shfl_xor((int)most, 32, 64));
            const uint32_t byte = scale_byte(most);
            const float by = scale_inverse(byte);
            float f[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) f[i] = byte == 255 ? 0.f : y[i >> 2][i & 3] * by;
            const uint32_t q = codes8(f);
            const int64_t t = it.m0 + 16 * m + r;
            if (t < it.hi) {
                uint16_t* codes = reinterpret_cast<uint16_t*>(static_cast<uint8_t*>(a.out) + t * (NO / 2) + n0 / 2);
                codes[g] = (uint16_t)q;
                codes[4 + g] = (uint16_t)(q >> 16);
                if (g == 0) {
                    uint8_t* scales = a.out_scales + ((n0 >> 8) * a.M + t) * 8;
                    const int at = (int)(n0 >> 5) & 7;
                    scales[at] = (uint8_t)byte;
                    if (n0 + 32 >= NO)
                        for (int i = at + 1; i < 8; ++i) scales[i] = 0;
                }
            }
            continue;
        }
        if (wave >= NC) continue;
        f32x4 c0 = sums[0][wave][lane], c1 = c0;
        if constexpr (GATED) c1 = sums[0][NC + wave][lane];
#pragma unroll
        for (int v = 1; v < W; ++v) {
            c0 += sums[v][wave][lane];
            if constexpr (GATED) c1 += sums[v][NC + wave][lane];
        }
        const int64_t t = it.m0 + 16 * m + r, n = n0 + 16 * wave + 4 * g;
        if (t < it.hi && n < NO) {   // NO is a multiple of 4
            f32x4 y = c0;
            if constexpr (GATED) {
#pragma unroll
                for (int i = 0; i < 4; ++i) y[i] = gate(c0[i], c1[i]);
            }
            if constexpr (OUT == kOutBf16)
                *reinterpret_cast<u32x2*>(static_cast<uint16_t*>(a.out) + t * NO + n) =
                    u32x2{pack_bf16(y[0], y[1]), pack_bf16(y[2], y[3])};
            else
                *reinterpret_cast<f32x4*>(static_cast<float*>(a.out) + t * NO + n) = y;
        }
    }
}

template <MxOut OUT, bool GATED, bool GATHERED, int NB, int W, int TOK>
__global__ __launch_bounds__(64 * W, 2) void mx_rows_kernel(MxArgs a) {
    __shared__ f32x4 sums[W][NB][64];
    RowsItem it;
    const int64_t NO = GATED ? a.N / 2 : a.N;
    constexpr int kCols = 16 * (GATED ? NB / 2 : NB);
    if (!find_rows_item<TOK>(a.offs, a.E, a.M, (int32_t)((NO + kCols - 1) / kCols), &it)) return;
    const int64_t left = it.hi - it.m0;   // of the group; this block's are at most TOK
    if (left <= 16) mx_rows_block<OUT, GATED, GATHERED, NB, 1, W, 2>(a, it, sums);
    else if (TOK == 32 || left <= 32) mx_rows_block<OUT, GATED, GATHERED, NB, 2, W, 1>(a, it, sums);
    else if constexpr (TOK > 32) mx_rows_block<OUT, GATED, GATHERED, NB, 4, W, 1>(a, it, sums);
}

template <bool GATED, int NB, int W, int TOK>
hipError_t launch_mx_rows(const MxArgs& a, bool bf16, hipStream_t s) {
    const int64_t ntn = ceil_div(GATED ? a.N / 2 : a.N, 16 * (GATED ? NB / 2 : NB));
    // ceil(T_e / TOK) over the groups is at most M / TOK and one for each group with rows
    const int64_t most = (a.M / TOK + (a.M < a.E ? a.M : a.E)) * ntn;
    const dim3 grid((unsigned)most), block(64 * W);
    timing_mark("mx_rows_kernel", s);
    auto launch = [&](auto gathered) {
        constexpr bool G = decltype(gathered)::value;
        if constexpr (GATED && G && NB == 4)
            if (a.out_scales) {
                hipLaunchKernelGGL((mx_rows_kernel<kOutMx, GATED, G, NB, W, TOK>), grid, block, 0, s, a);
                return;
            }
        if (bf16) hipLaunchKernelGGL((mx_rows_kernel<kOutBf16, GATED, G, NB, W, TOK>), grid, block, 0, s, a);
        else hipLaunchKernelGGL((mx_rows_kernel<kOutFp32, GATED, G, NB, W, TOK>), grid, block, 0, s, a);
    };
    if (a.rows) launch(std::true_type{});
    else launch(std::false_type{});
    timing_end(s);
    return hipGetLastError();
}

// ---------------------------------------------------------------------------
// product, many rows per group
//
// The tile engine (engine.hpp) on 4-bit elements: a pair of stages is 256 values
// (128 bytes, eight blocks) of a row and has four sub-steps, in each of which the
// MFMA takes one block from either half of the lanes.  Which one is free, as long
// as both operands agree: sub-step q takes block q and, in the upper half, block
// 4 + q.  The blocks a lane sees in a pair are then neighbours, and their four
// scale bytes one aligned dword, which the four sub-steps' MFMAs select from by an
// immediate: no instruction handles a scale but the LDS read.  (In the order of
// the 8-bit product the scales of a stage had to be permuted into place: on one
// card 299 to 309 us for 8192x8192x8192, 295 to 298 in this one.)  The scales
// of a pair (eight bytes a row) are loaded beside its codes and land behind them
// in its buffer.  A pair of stages lands as one, so that the upper half may read
// ahead of the stage.

struct Mxfp4 {};

constexpr int mx_buffer_bytes(int rows) { return rows * (4 * kStageK + 8); }   // codes of a pair of stages, then scales

#define DRGG_MX_BUFFERS(ROWS, name)                                                       \
    __shared__ __attribute__((aligned(256))) char name##0[mx_buffer_bytes(ROWS)];         \
    __shared__ __attribute__((aligned(256))) char name##1[mx_buffer_bytes(ROWS)]
#define DRGG_MX_STAGES(BM, BN, name)                                                      \
    DRGG_MX_BUFFERS(BM, name##_a);                                                        \
    DRGG_MX_BUFFERS(BN, name##_b);                                                        \
    const Stages name{{(lds_t*)name##_a0, (lds_t*)name##_a0, (lds_t*)name##_a1, (lds_t*)name##_a1}, \
                      {(lds_t*)name##_b0, (lds_t*)name##_b0, (lds_t*)name##_b1, (lds_t*)name##_b1}}

// The codes as StageLoader brings them, then ROWS/32 wave instructions of 4 bytes
// a lane: lane l of instruction g has dword l%2 of row 32 g + l/2.
// An operand that is not gathered says in `of` which row of its scales is its
// first.
template <int ROWS, int WAVES, bool PAIRED, bool GATHERED>
struct MxLoader : StageLoader<ROWS, true, WAVES, PAIRED, GATHERED> {
    using Codes = StageLoader<ROWS, true, WAVES, PAIRED, GATHERED>;
    static constexpr int kCodes = Codes::kPerWave, kScales = ROWS / 32 / WAVES;
    static constexpr int kPerWave = kCodes + kScales;
    static_assert(kScales >= 1, "every wave loads scales");
    uint32_t soff[kScales];
    const uint8_t* scales;      // of the operand's first row
    // set once by the kernel: the scales of row 0, the bytes from the scales of
    // 256 columns to the next, and (paired) the rows to the second run
    const uint8_t* all_scales;
    int64_t scale_step;
    int32_t pair_rows;

    __device__ __forceinline__ void init(const Operand& op) {
        Codes::init(op);
        int lane = threadIdx.x & 63;
        asm volatile("" : "+v"(lane));
        const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
        scales = all_scales + (GATHERED ? 0 : op.of * 8);
#pragma unroll
        for (int i = 0; i < kScales; ++i) {
            const int row = (wave * kScales + i) * 32 + (lane >> 1);
            int from = PAIRED ? (row & 31) + 32 * (row >> 6) : row;
            bool ok = from < op.nvalid;
            if constexpr (GATHERED) {
                from = ok ? op.index[from] : 0;
                ok = ok && (uint32_t)from < (uint32_t)op.of;
            }
            if (PAIRED && (row & 32)) from += pair_rows;
            soff[i] = ok ? (uint32_t)(from * 8 + 4 * (lane & 1)) : kOOB;
        }
    }
    __device__ __forceinline__ void issue(lds_t* buf, int L, bool valid) const { issue_part<0, kPerWave>(buf, L, valid); }
    template <int J0, int J1>
    __device__ __forceinline__ void issue_part(lds_t* buf, int L, bool valid) const {
        constexpr int c1 = J1 < kCodes ? J1 : kCodes, s0 = J0 > kCodes ? J0 - kCodes : 0, s1 = J1 - kCodes;
        if constexpr (J0 < c1) Codes::template issue_part<J0, c1>(buf, L, valid);
        if constexpr (s0 < s1) {
            const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
            const __amdgpu_buffer_rsrc_t r = make_rsrc(scales + (L >> 1) * scale_step);
            const int lane = threadIdx.x & 63;
            const bool in = valid && (L + (lane & 1)) * kStageK < this->klen;
#pragma unroll
            for (int i = s0; i < s1; ++i)
                __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_void_t*)(buf + ROWS * 4 * kStageK + (wave * kScales + i) * 256),
                                                         4, in ? soff[i] : kOOB, 0, 0, 0);
        }
    }
};

// the fragment of block 2 (ST % 2) + s, in the upper half of the lanes 4 + that
template <int ST>
__device__ __forceinline__ i32x4 mx_read_frag(const lds_t* buf, int rb, int s, int l) {
    const int row = rb + (l & 31), c = 4 * (l >> 5) + 2 * (ST & 1) + s;
    return *reinterpret_cast<const __attribute__((address_space(3))) i32x4*>(buf + row * (4 * kStageK) + ((c ^ swzK(row)) << 4));
}

// The products of a tile (TileMma's wave grid and accumulator layout).
template <int BM, int BN, int WAVES>
struct MxMma {
    using Grid = TileMma<BM, BN, true, true, WAVES, Bf16>;
    __device__ static __forceinline__ int wave_row(int wave) { return Grid::wave_row(wave); }
    __device__ static __forceinline__ int wave_col(int wave) { return Grid::wave_col(wave); }
    static constexpr int kBI = Grid::kBI, kBJ = Grid::kBJ, kBN = BN;
    static constexpr int kReads = kBI + kBJ, kMfmas = kBI * kBJ;
    f32x16 acc[kBI][kBJ];
    i32x4 fa[2][kBI], fb[2][kBJ];
    uint32_t sa[2][kBI], sb[2][kBJ];   // of the pair of stages in buffer 0 and 1

    __device__ __forceinline__ void zero() {
#pragma unroll
        for (int i = 0; i < kBI; ++i)
#pragma unroll
            for (int j = 0; j < kBJ; ++j)
#pragma unroll
                for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.f;
    }

    template <int F, int ST>
    __device__ __forceinline__ void read(const Stages& st, int s) {
        const int l = threadIdx.x & 63;
        const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
        const int ra = wave_row(wave), rb = wave_col(wave);
        if constexpr (F == 0 && !(ST & 1)) {
            typedef const __attribute__((address_space(3))) uint32_t lds_u32;
            const int o = (l & 31) * 8 + 4 * (l >> 5);   // consecutive dwords over the lanes: no bank conflict
#pragma unroll
            for (int i = 0; i < kBI; ++i)
                sa[ST >> 1][i] = *reinterpret_cast<lds_u32*>(st.a[ST] + BM * 4 * kStageK + (ra + 32 * i) * 8 + o);
#pragma unroll
            for (int j = 0; j < kBJ; ++j)
                sb[ST >> 1][j] = *reinterpret_cast<lds_u32*>(st.b[ST] + BN * 4 * kStageK + (rb + 32 * j) * 8 + o);
        }
        fa[F][0] = mx_read_frag<ST>(st.a[ST], ra, s, l);
#pragma unroll
        for (int j = 0; j < kBJ; ++j) fb[F][j] = mx_read_frag<ST>(st.b[ST], rb + 32 * j, s, l);
#pragma unroll
        for (int i = 1; i < kBI; ++i) fa[F][i] = mx_read_frag<ST>(st.a[ST], ra + 32 * i, s, l);
    }

    template <int F, int ST, bool FIRST = false>
    __device__ __forceinline__ void mfma() {
        constexpr int kByte = 2 * (ST & 1) + F;
#pragma unroll
        for (int i = 0; i < kBI; ++i)
#pragma unroll
            for (int j = 0; j < kBJ; ++j)
                acc[i][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(
                    fragment(__builtin_bit_cast(u32x4, fb[F][j])), fragment(__builtin_bit_cast(u32x4, fa[F][i])),
                    FIRST ? f32x16{} : acc[i][j], 4, 4, kByte, sb[ST >> 1][j], kByte, sa[ST >> 1][i]);
    }
};

}  // namespace

template <>
struct EngineParts<Mxfp4> {
    template <int BM, int BN, bool AK, bool BK, int WAVES>
    using Mma = MxMma<BM, BN, WAVES>;
    template <int ROWS, bool KMAJ, int WAVES, bool PAIRED, bool GATHERED>
    using Loader = MxLoader<ROWS, WAVES, PAIRED, GATHERED>;
};

namespace {

constexpr int mx_ep_rows(int bm, int bn) { return bm == 128 && bn == 256 ? 16 : 8; }   // what the scales leave room for

// Write a gated tile as codes and scales: value(i, j, q) as store_tile_values
// takes it.  A row's 32 columns are held by two lanes, 16 values each, in runs of
// four that alternate; after their halves are exchanged each lane has eight
// neighbouring bytes of codes.  Columns past the tile's are zeros (their operands
// are), so their scales are 0; behind the last tile's the rest of the scales'
// eight bytes is cleared too.
template <class Mma, int NJ, class Value>
__device__ __forceinline__ void store_tile_mx(Value value, int rb, const MxArgs& a, int64_t o0, int64_t o1, int rows, int cols) {
    static_assert(NJ == 2 || NJ == 1, "one or two blocks per wave and row");
    int lane = threadIdx.x & 63;
    asm volatile("" : "+v"(lane));
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int ra = Mma::wave_row(wave), r = lane & 31, h = lane >> 5;
    const int64_t I = a.N / 2;
#pragma unroll
    for (int i = 0; i < Mma::kBI; ++i) {
        const int row = ra + 32 * i + r;
        const bool live = row < rows;
        uint8_t* codes = static_cast<uint8_t*>(a.out) + (o0 + row) * (I / 2) + (o1 + rb) / 2 + 8 * h;
        uint32_t bytes = 0;
#pragma unroll
        for (int j = 0; j < NJ; ++j) {
            float f[16];
            uint32_t most = 0;
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const f32x4 y = value(i, j, q);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    f[4 * q + e] = y[e];
                    most = max(most, __float_as_uint(y[e]) & 0x7FFFFFFFu);
                }
            }
            most = max(most, (uint32_t)__shfl_xor((int)most, 32, 64));
            const uint32_t b = scale_byte(most);
            const float by = scale_inverse(b);
            bytes |= b << (8 * j);
#pragma unroll
            for (int e = 0; e < 16; ++e) f[e] = b == 255 ? 0.f : f[e] * by;
            // runs of four values, two bytes each: 0 and 1, then 2 and 3
            const uint32_t lo = codes8({f[0], f[1], f[2], f[3], f[4], f[5], f[6], f[7]});
            const uint32_t hi = codes8({f[8], f[9], f[10], f[11], f[12], f[13], f[14], f[15]});
            // lower lanes: their own runs 0, 1 and the upper lane's; upper lanes: the lower lane's runs 2, 3 and their own
            const auto x = __builtin_amdgcn_permlane32_swap(lo, hi, false, false);
            const u32x2 d = {__builtin_amdgcn_perm(x[1], x[0], 0x05040100u), __builtin_amdgcn_perm(x[1], x[0], 0x07060302u)};
            if (live && rb + 32 * j < cols) *reinterpret_cast<u32x2*>(codes + 16 * j) = d;
        }
        if (live && h == 0) {
            const int64_t c = o1 + rb;
            uint8_t* scales = a.out_scales + ((c >> 8) * a.M + o0 + row) * 8;
            const int at = (int)(c >> 5) & 7;
            if constexpr (NJ == 2) *reinterpret_cast<uint16_t*>(scales + at) = (uint16_t)bytes;
            else scales[at] = (uint8_t)bytes;
            if (o1 + cols == I && rb + 32 * NJ >= Mma::kBN / 2)   // the last columns' wave of the last tile
                for (int e = at + NJ; e < 8; e += 2) *reinterpret_cast<uint16_t*>(scales + e) = 0;
        }
    }
}

// The 8-bit product's walk and epilogue without scales of whole rows.
//
// 131072x1536x2048 in 8 groups, BF16 out: 248 to 277 us (3.3 to 3.0 PFLOP/s);
// 8192x8192x8192 264 us (4.2; a large library product of the same operands 3.1),
// 16384 cubed 2070 us (4.25; 3.4).  A 256x256 tile takes 0.77 to 0.92 us per step
// of 64 bytes, more on slower cards and on codes that toggle more bits: the clock
// is the power limit's (1.79 GHz; on zeros 8192 cubed takes 204 us), the matrix
// pipe busy 54 % of the time.  About 6 us are a tile's epilogue and switch, 30 % at
// K = 2048.  Measured and not taken: 4 waves of 128x128 each (295 us against 282 at
// 8192 cubed), stores without the non-temporal hint (302 against 277 to 285), and
// waiting for a tile's stores only inside the next tile's main loop (no change).
template <int BM, int BN, MxOut OUT, bool GATED, bool GATHERED, int WAVES>
__global__ __launch_bounds__(64 * WAVES, BM == 128 && BN == 128 ? 2 : 1) void mx_tile_kernel(MxArgs a) {
    DRGG_MX_STAGES(BM, BN, stg);
    __shared__ SchedOf<16, BM == 128 && BN == 128 ? kMx128MaxExperts : kMaxExperts> sch;
    __shared__ __attribute__((aligned(16))) char ep[OUT == kOutMx ? 16 : WAVES * mx_ep_rows(BM, BN) * 128];
    using Runner = TileRunner<BM, BN, true, true, WAVES, Mxfp4, GATED, GATHERED>;
    using Mma = typename Runner::Mma;
    constexpr int BC = GATED ? BN / 2 : BN;             // output columns per tile
    constexpr int NJ = GATED ? Mma::kBJ / 2 : Mma::kBJ; // blocks of 32 of them per wave
    const int64_t NO = GATED ? a.N / 2 : a.N, K2 = a.K / 4;   // K2: a row in the engine's units of 2 bytes
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
        const int64_t row = (int64_t)e * a.N + t.o1;
        t.A = GATHERED ? Operand{reinterpret_cast<const uint16_t*>(a.X), K2, t.rows, (int32_t)K2, 0, a.rows + t.o0, a.T}
                       : Operand{reinterpret_cast<const uint16_t*>(a.X) + t.o0 * K2, K2, t.rows, (int32_t)K2, 0, nullptr, t.o0};
        t.B = Operand{reinterpret_cast<const uint16_t*>(a.W) + row * K2, K2, t.cols, (int32_t)K2, NO * K2 * 2, nullptr, row};
        w += G;
    };
    auto finish = [&](const TileInfo& t, const Mma& mma) {
        const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
        const int rb = GATED ? Mma::wave_col(wave) / 2 : Mma::wave_col(wave);
        auto value = [&](int i, int j, int q) {
            f32x4 y;
#pragma unroll
            for (int r = 0; r < 4; ++r)
                y[r] = GATED ? gate(mma.acc[i][2 * j % Mma::kBJ][4 * q + r], mma.acc[i][(2 * j + 1) % Mma::kBJ][4 * q + r])
                             : mma.acc[i][j][4 * q + r];
            return y;
        };
        if constexpr (OUT == kOutMx) {
            store_tile_mx<Mma, NJ>(value, rb, a, t.o0, t.o1, t.rows, t.cols);
        } else {
            constexpr bool kBf16 = OUT == kOutBf16;
            const int64_t o = t.o0 * NO + t.o1;
            void* base = kBf16 ? (void*)(static_cast<uint16_t*>(a.out) + o) : (void*)(static_cast<float*>(a.out) + o);
            store_tile_values<kBf16, mx_ep_rows(BM, BN), Mma, NJ>(value, rb, (lds_t*)ep, base, NO, t.rows, t.cols);
        }
    };
    Runner runner;
    runner.st = stg;
    runner.la.all_scales = a.xs;
    runner.la.scale_step = 8 * (GATHERED ? a.T : a.M);
    runner.lb.all_scales = a.ws;
    runner.lb.scale_step = 8 * (int64_t)a.E * a.N;
    runner.lb.pair_rows = (int32_t)NO;
    runner.run(more, next, finish);
}

template <int BM, int BN, int WAVES, bool GATED, bool GATHERED>
void launch_mx_tile_t(const MxArgs& a, bool bf16, dim3 grid, hipStream_t s) {
    const dim3 block(64 * WAVES);
    constexpr bool kBf16 = !GATED || BN >= 256;   // a gated 128x128 tile has 32 columns per wave, half a BF16 line
    if constexpr (GATED && GATHERED)
        if (a.out_scales) {
            hipLaunchKernelGGL((mx_tile_kernel<BM, BN, kOutMx, GATED, GATHERED, WAVES>), grid, block, 0, s, a);
            return;
        }
    if constexpr (kBf16)
        if (bf16) {
            hipLaunchKernelGGL((mx_tile_kernel<BM, BN, kOutBf16, GATED, GATHERED, WAVES>), grid, block, 0, s, a);
            return;
        }
    hipLaunchKernelGGL((mx_tile_kernel<BM, BN, kOutFp32, GATED, GATHERED, WAVES>), grid, block, 0, s, a);
}

template <int BM, int BN, int WAVES>
hipError_t launch_mx_tile(const MxArgs& a, bool gated, bool bf16, int64_t grid_n, hipStream_t s) {
    const dim3 grid((unsigned)grid_n);
    timing_mark("mx_tile_kernel", s);
    if (gated && a.rows) launch_mx_tile_t<BM, BN, WAVES, true, true>(a, bf16, grid, s);
    else if (gated) launch_mx_tile_t<BM, BN, WAVES, true, false>(a, bf16, grid, s);
    else if (a.rows) launch_mx_tile_t<BM, BN, WAVES, false, true>(a, bf16, grid, s);
    else launch_mx_tile_t<BM, BN, WAVES, false, false>(a, bf16, grid, s);
    timing_end(s);
    return hipGetLastError();
}

template <bool GATED>
hipError_t launch_mx_program(const MxArgs& a, const Int8Program& p, bool bf16, hipStream_t s) {
    if (p.tok == 32) return launch_mx_rows<GATED, 4, 4, 32>(a, bf16, s);
    if (p.waves == 4) return launch_mx_rows<GATED, 4, 4, 64>(a, bf16, s);
    if (p.nb == 4) return launch_mx_rows<GATED, 4, 8, 64>(a, bf16, s);
    if constexpr (!GATED)
        if (p.nb == 1) return launch_mx_rows<false, 1, 8, 64>(a, bf16, s);
    return launch_mx_rows<GATED, 2, 8, 64>(a, bf16, s);
}

}  // namespace

hipError_t launch_quantize_mxfp4(const void* X, bool bf16, int64_t T, int64_t K, uint8_t* codes, uint8_t* scales,
                                 hipStream_t s) {
    const MxQuantArgs a{X, codes, scales, T, K};
    timing_mark("quantize_mxfp4_kernel", s);
    if (bf16) hipLaunchKernelGGL(quantize_mxfp4_kernel<true>, mx_row_grid(T, K), dim3(256), 0, s, a);
    else hipLaunchKernelGGL(quantize_mxfp4_kernel<false>, mx_row_grid(T, K), dim3(256), 0, s, a);
    timing_end(s);
    return hipGetLastError();
}

hipError_t launch_dequantize_mxfp4(const uint8_t* codes, const uint8_t* scales, int64_t T, int64_t K, bool bf16,
                                   void* X, hipStream_t s) {
    const MxRowArgs a{codes, scales, X, T, K};
    timing_mark("dequantize_mxfp4_kernel", s);
    if (bf16) hipLaunchKernelGGL(dequantize_mxfp4_kernel<true>, mx_row_grid(T, K), dim3(256), 0, s, a);
    else hipLaunchKernelGGL(dequantize_mxfp4_kernel<false>, mx_row_grid(T, K), dim3(256), 0, s, a);
    timing_end(s);
    return hipGetLastError();
}

hipError_t launch_mxfp4(const MxArgs& a, bool gated, bool bf16, int cus, int forced_tile, hipStream_t s) {
    if (a.out_scales && !(gated && a.rows)) return hipErrorInvalidValue;   // codes leave the block's first product alone
    const Int8Program p = mxfp4_program(a.E, a.M, a.N, a.K, gated, bf16, a.out_scales != nullptr, forced_tile);
    if (p.tile == kTileAuto)
        return gated ? launch_mx_program<true>(a, p, bf16, s) : launch_mx_program<false>(a, p, bf16, s);
    const int64_t cols_out = gated ? a.N / 2 : a.N, bc = gated ? 128 : 256;
    auto grid = [&](int64_t bm, int64_t bcols, int64_t per_cu) {
        const int64_t most = (a.M / bm + (a.M < a.E ? a.M : a.E)) * ceil_div(cols_out, bcols);
        return most < per_cu * cus ? most : per_cu * cus;
    };
    if (p.tile == kTile256x256) return launch_mx_tile<256, 256, 8>(a, gated, bf16, grid(256, bc, 1), s);
    if (p.tile == kTile128x256) return launch_mx_tile<128, 256, 4>(a, gated, bf16, grid(128, bc, 1), s);
    return launch_mx_tile<128, 128, 4>(a, gated, bf16, grid(128, bc / 2, 2), s);
}

}  // namespace drgg
