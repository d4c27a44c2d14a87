// gate.hip -- gfx950 (CDNA4) kernels of the gated activation that keeps its
// inputs in 8 bits, and of its backward pass from what was kept.
//
//   h[p] = w silu(g) u                      p the row of pair (t, j), w its weight
//   codes = round(127 x / m), scale = m / 127, m = max|x| over 128 columns of g or u
//   dGU[p] = w dh (u s (1 + g (1 - s)), g s),  s = 1 / (1 + exp(-g))
//   dw = sum of dh g s u
//
// Both are bound by memory.  Sixteen lanes, one DPP row, hold the 128 columns
// that share a scale, eight of gate and the same eight of up per lane, so that
// a maximum is four rotations in the vector unit and every access 8 or 16
// bytes.  Rows of weight 0 (masked pairs) get zeros in h and dGU whatever they
// hold.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "internal.hpp"
#include "plan.hpp"

namespace drgg {

namespace {

typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

struct GateArgs {
    const void* src;        // forward: GU; backward: dh
    const int8_t* kept;     // backward: codes
    const float* kept_scale;
    const int32_t* positions;
    const float* weights;
    void* h;
    int8_t* codes;          // forward
    float* scale;
    void* dGU;              // backward
    float* dweights;
    int64_t R, C;           // pairs; pieces of 8 columns in a half
};

template <int N>
__device__ __forceinline__ uint32_t rotate16(uint32_t v) {
    return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x120 + N, 0xF, 0xF, false);
}
__device__ __forceinline__ uint32_t max16(uint32_t v) {
    v = max(v, rotate16<8>(v));
    v = max(v, rotate16<4>(v));
    v = max(v, rotate16<2>(v));
    return max(v, rotate16<1>(v));
}
__device__ __forceinline__ float sum16(float v) {
    v += __uint_as_float(rotate16<8>(__float_as_uint(v)));
    v += __uint_as_float(rotate16<4>(__float_as_uint(v)));
    v += __uint_as_float(rotate16<2>(__float_as_uint(v)));
    return v + __uint_as_float(rotate16<1>(__float_as_uint(v)));
}

__device__ __forceinline__ float bf16_at(u32x4 v, int i) {
    return __uint_as_float(i & 1 ? v[i >> 1] & 0xFFFF0000u : v[i >> 1] << 16);
}
__device__ __forceinline__ u32x4 to_bf16(const float (&f)[8]) {
    u32x4 v;
#pragma unroll
    for (int i = 0; i < 4; ++i)
        v[i] = __builtin_bit_cast(uint32_t, __builtin_convertvector((f32x2{f[2 * i], f[2 * i + 1]}), bf16x2));
    return v;
}

// 1 / (1 + exp(-g)): the hardware's exponential and reciprocal, within 1 ulp
// each; the exponential's argument is rounded before, |g| 2^-24 of the result.
__device__ __forceinline__ float sigmoid(float g) {
    return __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(g * -1.44269504f));
}

// Codes of eight values and, for the block's 16 lanes, its scale.  a = 127 x is
// exact for BF16 x (times a power of two for blocks near FP32's limits).  The
// quotient a / m is the product with m's approximate reciprocal and one
// correction by the exact remainder: where it is a half exactly (x = m / 2: 63.5,
// to 64) the correction makes it so, and elsewhere it is at least 2^-17 of itself
// from one (a quotient of 15 and 8 bits), so that the code is that of the exact
// quotient.  Adding 1.5 * 2^23 rounds it to an integer, ties to even, in the low
// byte.  With correctly rounded divisions instead, 131072 rows of 2 x 768 took 201
// us.
__device__ __forceinline__ u32x2 keep8(u32x4 v, float* scale) {
    uint32_t bits = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) bits = max(bits, __float_as_uint(bf16_at(v, i)) & 0x7FFFFFFFu);
    bits = max16(bits);
    const bool bad = bits >= 0x7F800000u;
    const float most = __uint_as_float(bits);
    *scale = bad ? __uint_as_float(0x7FC00000u) : most / 127.f;
    const float by = most > 0x1p100f ? 0x1p-64f : most < 0x1p-60f ? 0x1p64f : 1.f;
    const float m = bad || bits == 0 ? 1.f : most * by, inverse = __builtin_amdgcn_rcpf(m), by127 = 127.f * by;
    uint32_t c[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float a = bf16_at(v, i) * by127, q = a * inverse;
        c[i] = __float_as_uint(__builtin_fmaf(__builtin_fmaf(-q, m, a), inverse, q) + 12582912.f);
    }
    u32x2 codes;
#pragma unroll
    for (int h = 0; h < 2; ++h)
        codes[h] = bad ? 0u
                       : __builtin_amdgcn_perm(__builtin_amdgcn_perm(c[4 * h + 3], c[4 * h + 2], 0x0c0c0400u),
                                               __builtin_amdgcn_perm(c[4 * h + 1], c[4 * h], 0x0c0c0400u), 0x05040100u);
    return codes;
}

// 131072 rows of 2 x 768 in 150 to 167 us, of 812 MB: 5.4 to 4.9 TB/s; a large copy
// reaches 5.1.
__global__ __launch_bounds__(256) void moe_gate_int8_kernel(GateArgs a) {
    const int64_t B = (a.C + 15) / 16;   // scales of a half
    for (int64_t r0 = (int64_t)blockIdx.x * blockDim.y; r0 < a.R; r0 += (int64_t)gridDim.x * blockDim.y) {
        const int64_t r = r0 + threadIdx.y;
        const int64_t p = r < a.R ? a.positions[r] : -1;
        if (p < 0 || p >= a.R) continue;   // all of the row's lanes
        const float w = a.weights[r];
        for (int64_t c = threadIdx.x; c < 16 * B; c += blockDim.x) {
            const bool in = c < a.C;
            u32x4 g = {0, 0, 0, 0}, u = g;
            if (in) {
                // not read again (32768 rows of 2 x 2048: 106 us with plain loads, 90 with
                // the hint; 131072 rows of 2 x 768: 167 either way)
                g = __builtin_nontemporal_load(static_cast<const u32x4*>(a.src) + p * 2 * a.C + c);
                u = __builtin_nontemporal_load(static_cast<const u32x4*>(a.src) + p * 2 * a.C + a.C + c);
            }
            float f[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float x = bf16_at(g, i);
                f[i] = w != 0.f ? w * (x * sigmoid(x) * bf16_at(u, i)) : 0.f;
            }
            float sg, su;
            const u32x2 qg = keep8(g, &sg), qu = keep8(u, &su);
            if (in) {
                static_cast<u32x4*>(a.h)[p * a.C + c] = to_bf16(f);
                reinterpret_cast<u32x2*>(a.codes)[p * 2 * a.C + c] = qg;
                reinterpret_cast<u32x2*>(a.codes)[p * 2 * a.C + a.C + c] = qu;
            }
            if ((threadIdx.x & 15) == 0) {
                a.scale[p * 2 * B + (c >> 4)] = sg;
                a.scale[p * 2 * B + B + (c >> 4)] = su;
            }
        }
    }
}

// 131072 rows of 2 x 768 in 203 to 217 us, of 1.0 GB: 5.0 to 4.7 TB/s.
__global__ __launch_bounds__(256) void moe_gate_int8_grad_kernel(GateArgs a) {
    __shared__ float part[16];   // a sum per 16 lanes
    const int64_t B = (a.C + 15) / 16;
    // whole blocks of pairs: every thread takes part in the sums
    for (int64_t r0 = (int64_t)blockIdx.x * blockDim.y; r0 < a.R; r0 += (int64_t)gridDim.x * blockDim.y) {
        const int64_t r = r0 + threadIdx.y;
        const int64_t p = r < a.R ? a.positions[r] : -1;
        const bool live = p >= 0 && p < a.R;
        const float w = live ? a.weights[r] : 0.f;
        float dot = 0.f;
        if (live)
            for (int64_t c = threadIdx.x; c < a.C; c += blockDim.x) {
                const u32x4 dh = static_cast<const u32x4*>(a.src)[p * a.C + c];
                const u32x2 qg = reinterpret_cast<const u32x2*>(a.kept)[p * 2 * a.C + c];
                const u32x2 qu = reinterpret_cast<const u32x2*>(a.kept)[p * 2 * a.C + a.C + c];
                const float sg = a.kept_scale[p * 2 * B + (c >> 4)], su = a.kept_scale[p * 2 * B + B + (c >> 4)];
                float dg[8], du[8], h[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float g = sg * (float)(int8_t)(qg[i >> 2] >> (8 * (i & 3)));
                    const float u = su * (float)(int8_t)(qu[i >> 2] >> (8 * (i & 3)));
                    const float s = sigmoid(g), d = bf16_at(dh, i), gs = g * s, act = gs * u;
                    dot += d * act;
                    h[i] = w != 0.f ? w * act : 0.f;
                    du[i] = w != 0.f ? w * d * gs : 0.f;
                    dg[i] = w != 0.f ? w * d * (u * (s + gs * (1.f - s))) : 0.f;
                }
                static_cast<u32x4*>(a.h)[p * a.C + c] = to_bf16(h);
                static_cast<u32x4*>(a.dGU)[p * 2 * a.C + c] = to_bf16(dg);
                static_cast<u32x4*>(a.dGU)[p * 2 * a.C + a.C + c] = to_bf16(du);
            }
        dot = sum16(dot);
        const int n = blockDim.x >> 4, at = threadIdx.y * n + (threadIdx.x >> 4);
        __syncthreads();   // the last pairs' sums have been read
        if ((threadIdx.x & 15) == 0) part[at] = dot;
        __syncthreads();
        if (threadIdx.x == 0 && r < a.R) {
            for (int i = 1; i < n; ++i) dot += part[at + i];
            a.dweights[r] = dot;
        }
    }
}

// threads along a row: whole rows of 16 lanes, at most 256
dim3 gate_block(int64_t C) {
    const int64_t x = round_up(C, 16) < 256 ? round_up(C, 16) : 256;
    return dim3((unsigned)x, (unsigned)(256 / x));
}
// a launch has fewer than 2^32 threads: blocks walk the pairs beyond
dim3 gate_grid(int64_t R, dim3 block) {
    const int64_t n = ceil_div(R, block.y), most = 65536;
    return dim3((unsigned)(n < most ? n : most));
}

}  // namespace

hipError_t launch_moe_gate_int8(const void* GU, const int32_t* positions, const float* weights, int64_t T, int32_t k,
                                int64_t I, void* h, int8_t* codes, float* scale, hipStream_t s) {
    GateArgs a{};
    a.src = GU;
    a.positions = positions;
    a.weights = weights;
    a.h = h;
    a.codes = codes;
    a.scale = scale;
    a.R = T * k;
    a.C = I / 8;
    const dim3 block = gate_block(a.C);
    timing_mark("moe_gate_int8_kernel", s);
    hipLaunchKernelGGL(moe_gate_int8_kernel, gate_grid(a.R, block), block, 0, s, a);
    timing_end(s);
    return hipGetLastError();
}

hipError_t launch_moe_gate_int8_grad(const void* dh, const int8_t* codes, const float* scale, const int32_t* positions,
                                     const float* weights, int64_t T, int32_t k, int64_t I, void* dGU, void* h,
                                     float* dweights, hipStream_t s) {
    GateArgs a{};
    a.src = dh;
    a.kept = codes;
    a.kept_scale = scale;
    a.positions = positions;
    a.weights = weights;
    a.h = h;
    a.dGU = dGU;
    a.dweights = dweights;
    a.R = T * k;
    a.C = I / 8;
    const dim3 block = gate_block(a.C);
    timing_mark("moe_gate_int8_grad_kernel", s);
    hipLaunchKernelGGL(moe_gate_int8_grad_kernel, gate_grid(a.R, block), block, 0, s, a);
    timing_end(s);
    return hipGetLastError();
}

}  // namespace drgg
