// moe.hip -- gfx950 (CDNA4) kernels around the grouped products of an expert
// layer: the router's selection and its gradient, and the movement of rows
// between the token order and the grouped order, with its gradients.
//
// All of them are bound by memory or, for a few tokens, by launch latency.
// Nothing here uses an atomic whose order could change a result.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "internal.hpp"
#include "plan.hpp"

namespace drgg {

namespace {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

// ---------------------------------------------------------------------------
// selection
//
// One wave per token.  Lane l holds the logits of experts 4l .. 4l+3 of every
// 256 (V groups of 256 cover E).  A logit is compared through a 32-bit key
// whose unsigned order is the order of the values (NaN above +inf, -0 equal
// to +0); key 0 marks an expert already taken or past E.  Each of the k
// rounds takes the largest key of the wave, at the lowest expert index among
// equals; lane j keeps round j's choice.

__device__ __forceinline__ uint32_t order_key(float v) {
    if (v != v) return 0xFFFFFFFFu;
    const uint32_t u = __float_as_uint(v + 0.f);   // -0 + 0 = +0
    return u & 0x80000000u ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ float key_value(uint32_t k) {
    return __uint_as_float(k & 0x80000000u ? k & 0x7FFFFFFFu : ~k);   // NaN: 0x7FFFFFFF, a NaN
}

__device__ __forceinline__ uint32_t wave_max_u32(uint32_t v) {
#pragma unroll
    for (int m = 1; m < 64; m <<= 1) {
        const uint32_t o = __shfl_xor(v, m, 64);
        v = o > v ? o : v;
    }
    return v;
}
__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
    for (int m = 1; m < 64; m <<= 1) v += __shfl_xor(v, m, 64);
    return v;
}

// The logits of one token as keys (expert 256*c + 4*lane + i in key[c][i]).
template <int V>
__device__ __forceinline__ void load_keys(uint32_t (&key)[V][4], const float* row, int E, int lane) {
    const bool vec = (E & 3) == 0;
#pragma unroll
    for (int c = 0; c < V; ++c) {
        const int e = 256 * c + 4 * lane;
        if (vec) {
            if (e < E) {
                const f32x4 v = *reinterpret_cast<const f32x4*>(row + e);
#pragma unroll
                for (int i = 0; i < 4; ++i) key[c][i] = order_key(v[i]);
            } else {
#pragma unroll
                for (int i = 0; i < 4; ++i) key[c][i] = 0;
            }
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) key[c][i] = e + i < E ? order_key(row[e + i]) : 0;
        }
    }
}

struct RouteArgs {
    const float* logits;
    int32_t* experts;
    float* weights;
    int32_t* offsets;
    int32_t* positions;
    int32_t* table;   // [blocks][E] counts, then their exclusive prefix over the blocks; then [E] totals
    int64_t T, blocks;
    int32_t E, k, renormalize;
};

constexpr int kRouteThreads = 1024, kRouteWaves = kRouteThreads / 64;
constexpr int kRouteTokens = 64;   // tokens per block: one 64-bit mask per expert

// Exclusive scan of one value per thread (thread order), of at most 1024
// threads; `tmp` holds a word per wave.  Called by all threads.
__device__ __forceinline__ int32_t block_prefix(int32_t v, int32_t* tmp) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    int32_t x = v;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const int32_t y = __shfl_up(x, d, 64);
        if (lane >= d) x += y;
    }
    if (lane == 63) tmp[wave] = x;
    __syncthreads();
    int32_t before = 0;
    for (int w = 0; w < wave; ++w) before += tmp[w];
    return before + x - v;
}

// Experts, weights, and each pair's rank among the block's earlier tokens of
// the same expert.  The rank comes from one bit per token and expert: the
// tokens of a block are ordered by their bit, so ranks and counts are
// popcounts, whatever order the bits were set in.  With a single block the
// offsets and final positions are written here; otherwise the counts go to
// the table and positions hold the ranks for moe_place_kernel.
template <int V>
__global__ __launch_bounds__(kRouteThreads) void moe_select_kernel(RouteArgs a) {
    __shared__ unsigned long long mask[256 * V];
    __shared__ int32_t start[256 * V], tmp[kRouteWaves];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int E = a.E, k = a.k;
    for (int e = threadIdx.x; e < E; e += kRouteThreads) mask[e] = 0;
    __syncthreads();
    const int64_t t0 = (int64_t)blockIdx.x * kRouteTokens;
    constexpr int kPer = kRouteTokens / kRouteWaves;
    int32_t mine[kPer];
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        const int tl = i * kRouteWaves + wave;
        const int64_t t = t0 + tl;
        mine[i] = 0;
        if (t >= a.T) continue;
        uint32_t key[V][4];
        load_keys<V>(key, a.logits + t * E, E, lane);
        uint32_t top = 0, kept = 0;
        for (int j = 0; j < k; ++j) {
            uint32_t m = 0;
#pragma unroll
            for (int c = 0; c < V; ++c)
#pragma unroll
                for (int q = 0; q < 4; ++q) m = key[c][q] > m ? key[c][q] : m;
            const uint32_t best = wave_max_u32(m);
            // the lowest expert with that key: groups in order, then lanes, then the lane's four
            int32_t e = 0;
            bool done = false;
#pragma unroll
            for (int c = 0; c < V; ++c) {
                int q = 4;
#pragma unroll
                for (int r = 3; r >= 0; --r) q = key[c][r] == best ? r : q;
                const unsigned long long has = __ballot(q < 4);
                if (!done && has) {
                    const int l = __ffsll((long long)has) - 1;
                    e = 256 * c + 4 * l + __shfl(q, l, 64);
                    if (lane == l) {
#pragma unroll
                        for (int r = 0; r < 4; ++r) key[c][r] = r == q ? 0 : key[c][r];
                    }
                    done = true;
                }
            }
            if (j == 0) top = best;
            if (lane == j) {
                kept = best;
                mine[i] = e;
            }
        }
        // softmax over the chosen (lanes 0 .. k-1), or over all experts
        const float most = key_value(top), v = key_value(kept);
        const bool none = most == -INFINITY;   // every expert is masked: all weights 0
        float p = lane < k && !none ? expf(v - most) : 0.f, total;
        if (a.renormalize) {
            total = wave_sum(p);
        } else {
            // the keys of the chosen are gone: their terms are the p of lanes 0 .. k-1
            float s = p;
            if (!none) {
#pragma unroll
                for (int c = 0; c < V; ++c)
#pragma unroll
                    for (int q = 0; q < 4; ++q) s += key[c][q] ? expf(key_value(key[c][q]) - most) : 0.f;
            }
            total = wave_sum(s);
        }
        if (lane < k) {
            a.experts[t * k + lane] = mine[i];
            a.weights[t * k + lane] = none ? 0.f : p / total;
            atomicOr(&mask[mine[i]], 1ull << tl);
        }
    }
    __syncthreads();
    const bool single = a.blocks == 1;
    if (single) {
        const int32_t n = (int)threadIdx.x < E ? __popcll(mask[threadIdx.x]) : 0;
        const int32_t s = block_prefix(n, tmp);
        if ((int)threadIdx.x < E) {
            start[threadIdx.x] = s;
            a.offsets[threadIdx.x] = s;
            if ((int)threadIdx.x == E - 1) a.offsets[E] = s + n;
        }
        __syncthreads();
    } else {
        for (int e = threadIdx.x; e < E; e += kRouteThreads)
            a.table[(int64_t)blockIdx.x * E + e] = __popcll(mask[e]);
    }
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        const int tl = i * kRouteWaves + wave;
        const int64_t t = t0 + tl;
        if (t >= a.T || lane >= k) continue;
        const int e = mine[i];
        const int32_t r = __popcll(mask[e] & ((1ull << tl) - 1));
        a.positions[t * k + lane] = single ? start[e] + r : r;
    }
}

// The table's columns to exclusive prefixes over the blocks, and each
// expert's total.  One lane per expert; the 16 waves of a workgroup each take
// a run of blocks, sum it, and write its prefixes.
__global__ __launch_bounds__(kRouteThreads) void moe_scan_kernel(RouteArgs a) {
    __shared__ int32_t sums[kRouteWaves][64];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int e = blockIdx.x * 64 + lane;
    const bool ok = e < a.E;
    const int64_t per = (a.blocks + kRouteWaves - 1) / kRouteWaves;
    const int64_t lo = min(wave * per, a.blocks), hi = min(lo + per, a.blocks);
    int32_t s = 0;
    if (ok)
        for (int64_t b = lo; b < hi; ++b) s += a.table[b * a.E + e];
    sums[wave][lane] = s;
    __syncthreads();
    int32_t acc = 0;
    for (int w = 0; w < wave; ++w) acc += sums[w][lane];
    if (ok) {
        for (int64_t b = lo; b < hi; ++b) {
            const int32_t n = a.table[b * a.E + e];
            a.table[b * a.E + e] = acc;
            acc += n;
        }
        if (wave == kRouteWaves - 1) a.table[a.blocks * a.E + e] = acc;
    }
}

// positions += the expert's offset + its pairs in earlier blocks.
__global__ __launch_bounds__(kRouteThreads) void moe_place_kernel(RouteArgs a) {
    __shared__ int32_t base[kMaxExperts], tmp[kRouteWaves];
    const int E = a.E;
    const int tid = threadIdx.x;
    const int32_t n = tid < E ? a.table[a.blocks * E + tid] : 0;
    const int32_t s = block_prefix(n, tmp);
    if (tid < E) {
        base[tid] = s + a.table[(int64_t)blockIdx.x * E + tid];
        if (blockIdx.x == 0) {
            a.offsets[tid] = s;
            if (tid == E - 1) a.offsets[E] = s + n;
        }
    }
    __syncthreads();
    const int64_t p0 = (int64_t)blockIdx.x * kRouteTokens * a.k;
    const int64_t p1 = min(p0 + (int64_t)kRouteTokens * a.k, a.T * a.k);
    for (int64_t p = p0 + tid; p < p1; p += kRouteThreads) a.positions[p] += base[a.experts[p]];
}

struct RouteGradArgs {
    const float* dweights;
    const float* logits;
    const int32_t* experts;
    const float* weights;
    float* dlogits;
    int64_t T;
    int32_t E, k, renormalize;
};

// dlogits of one token per wave.  With s = sum_j w_j dw_j:
//   softmax over the chosen: w_j (dw_j - s) at the chosen, 0 elsewhere;
//   softmax over all: p_e ((dw at the chosen, else 0) - s), where the p of
//   every expert is recomputed from the logits.
// Lane j holds pair j; every lane writes its experts 4l .. 4l+3 of each 256.
template <int V>
__global__ __launch_bounds__(256) void moe_route_grad_kernel(RouteGradArgs a) {
    const int lane = threadIdx.x & 63;
    const int64_t t = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
    if (t >= a.T) return;
    const int E = a.E, k = a.k;
    int32_t e = -1;
    float w = 0.f, d = 0.f;
    if (lane < k) {
        e = a.experts[t * k + lane];
        w = a.weights[t * k + lane];
        d = a.dweights[t * k + lane];
    }
    const float s = wave_sum(w * d);
    float g[V][4];
    if (a.renormalize) {
        const float v = w * (d - s);
#pragma unroll
        for (int c = 0; c < V; ++c)
#pragma unroll
            for (int i = 0; i < 4; ++i) g[c][i] = 0.f;
        for (int j = 0; j < k; ++j) {
            const int32_t ej = __shfl(e, j, 64);
            const float vj = __shfl(v, j, 64);
#pragma unroll
            for (int c = 0; c < V; ++c)
#pragma unroll
                for (int i = 0; i < 4; ++i) g[c][i] = ej == 256 * c + 4 * lane + i ? vj : g[c][i];
        }
    } else {
        uint32_t key[V][4], m = 0;
        load_keys<V>(key, a.logits + t * E, E, lane);
#pragma unroll
        for (int c = 0; c < V; ++c)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                m = key[c][i] > m ? key[c][i] : m;
                g[c][i] = -s;
            }
        for (int j = 0; j < k; ++j) {
            const int32_t ej = __shfl(e, j, 64);
            const float dj = __shfl(d, j, 64);
#pragma unroll
            for (int c = 0; c < V; ++c)
#pragma unroll
                for (int i = 0; i < 4; ++i) g[c][i] = ej == 256 * c + 4 * lane + i ? dj - s : g[c][i];
        }
        const float most = key_value(wave_max_u32(m));
        const bool none = most == -INFINITY;
        float total = 0.f, p[V][4];
#pragma unroll
        for (int c = 0; c < V; ++c)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                p[c][i] = key[c][i] && !none ? expf(key_value(key[c][i]) - most) : 0.f;
                total += p[c][i];
            }
        total = wave_sum(total);
#pragma unroll
        for (int c = 0; c < V; ++c)
#pragma unroll
            for (int i = 0; i < 4; ++i) g[c][i] = none ? 0.f : p[c][i] / total * g[c][i];
    }
    float* out = a.dlogits + t * E;
#pragma unroll
    for (int c = 0; c < V; ++c) {
        const int e0 = 256 * c + 4 * lane;
        if ((E & 3) == 0) {
            if (e0 < E) *reinterpret_cast<f32x4*>(out + e0) = f32x4{g[c][0], g[c][1], g[c][2], g[c][3]};
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (e0 + i < E) out[e0 + i] = g[c][i];
        }
    }
}

// ---------------------------------------------------------------------------
// rows
//
// A row is H values, H a multiple of 8; one thread moves 8 of them (16 bytes
// of BF16, 32 of FP32) at a time.  Threads (x, y) of a block: x along the
// row, y over tokens (rows shorter than 256 pieces share a block).  Each
// token's row is read once and its k grouped rows are read or written once,
// so no order of the grouped rows is needed but the positions.  A position
// outside [0, T*k) is skipped: no access leaves the buffers.

template <bool BF16>
struct Piece;   // 8 values of a row
template <>
struct Piece<true> {
    u32x4 v;
    __device__ __forceinline__ void load(const void* p, int64_t i) { v = reinterpret_cast<const u32x4*>(p)[i]; }
    __device__ __forceinline__ void store(void* p, int64_t i) const { reinterpret_cast<u32x4*>(p)[i] = v; }
    __device__ __forceinline__ float get(int i) const {
        return __uint_as_float(i & 1 ? v[i >> 1] & 0xFFFF0000u : v[i >> 1] << 16);
    }
    __device__ __forceinline__ void set(const float (&f)[8]) {
        typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
        typedef float f32x2 __attribute__((ext_vector_type(2)));
#pragma unroll
        for (int i = 0; i < 4; ++i)
            v[i] = __builtin_bit_cast(uint32_t, __builtin_convertvector((f32x2{f[2 * i], f[2 * i + 1]}), bf16x2));
    }
};
template <>
struct Piece<false> {
    f32x4 v[2];
    __device__ __forceinline__ void load(const void* p, int64_t i) {
        v[0] = reinterpret_cast<const f32x4*>(p)[2 * i];
        v[1] = reinterpret_cast<const f32x4*>(p)[2 * i + 1];
    }
    __device__ __forceinline__ void store(void* p, int64_t i) const {
        reinterpret_cast<f32x4*>(p)[2 * i] = v[0];
        reinterpret_cast<f32x4*>(p)[2 * i + 1] = v[1];
    }
    __device__ __forceinline__ float get(int i) const { return v[i >> 2][i & 3]; }
    __device__ __forceinline__ void set(const float (&f)[8]) {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i >> 2][i & 3] = f[i];
    }
};

struct RowArgs {
    const void* src;         // dispatch: token rows; combine: grouped rows; combine_grad: dout, token rows
    const void* rows;        // combine_grad: the grouped rows
    const int32_t* positions;
    const float* weights;    // combine: may be null (all 1)
    void* dst;
    float* dweights;
    int64_t T, C;            // C: pieces per row
    int32_t k;
};

template <bool BF16>
__global__ __launch_bounds__(256) void moe_dispatch_kernel(RowArgs a) {
    const int64_t t = (int64_t)blockIdx.x * blockDim.y + threadIdx.y;
    if (t >= a.T) return;
    const int64_t R = a.T * a.k;
    for (int64_t c = threadIdx.x; c < a.C; c += blockDim.x) {
        Piece<BF16> x;
        x.load(a.src, t * a.C + c);
        for (int j = 0; j < a.k; ++j) {
            const int64_t p = a.positions[t * a.k + j];
            if (p >= 0 && p < R) x.store(a.dst, p * a.C + c);
        }
    }
}

// FP32 sum over j in order, one rounding.
template <bool BF16>
__global__ __launch_bounds__(256) void moe_combine_kernel(RowArgs a) {
    const int64_t t = (int64_t)blockIdx.x * blockDim.y + threadIdx.y;
    if (t >= a.T) return;
    const int64_t R = a.T * a.k;
    for (int64_t c = threadIdx.x; c < a.C; c += blockDim.x) {
        float s[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
        for (int j = 0; j < a.k; ++j) {
            const int64_t p = a.positions[t * a.k + j];
            if (p < 0 || p >= R) continue;
            const float w = a.weights ? a.weights[t * a.k + j] : 1.f;
            Piece<BF16> x;
            x.load(a.src, p * a.C + c);
#pragma unroll
            for (int i = 0; i < 8; ++i) s[i] += w * x.get(i);
        }
        Piece<BF16> y;
        y.set(s);
        y.store(a.dst, t * a.C + c);
    }
}

// drows[position] = w * dout (one rounding) and dweights = <dout, row>, an
// FP32 sum: per thread over its pieces, then over the token's threads in a
// fixed tree.
template <bool BF16>
__global__ __launch_bounds__(256) void moe_combine_grad_kernel(RowArgs a) {
    __shared__ float part[4];
    const int64_t t = (int64_t)blockIdx.x * blockDim.y + threadIdx.y;
    const int64_t R = a.T * a.k;
    const bool live = t < a.T;
    for (int j = 0; j < a.k; ++j) {
        float dot = 0.f;
        int64_t p = live ? a.positions[t * a.k + j] : -1;
        if (p >= R) p = -1;
        if (p >= 0) {
            const float w = a.weights[t * a.k + j];
            for (int64_t c = threadIdx.x; c < a.C; c += blockDim.x) {
                Piece<BF16> g, x, y;
                g.load(a.src, t * a.C + c);
                x.load(a.rows, p * a.C + c);
                float f[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    dot += g.get(i) * x.get(i);
                    f[i] = w * g.get(i);
                }
                y.set(f);
                y.store(a.dst, p * a.C + c);
            }
        }
        // the token's threads: up to 64 lanes of one wave, then whole waves
        const int width = blockDim.x < 64 ? blockDim.x : 64;
        for (int m = 1; m < width; m <<= 1) dot += __shfl_xor(dot, m, 64);
        if (blockDim.x > 64) {
            const int wave = (threadIdx.y * blockDim.x + threadIdx.x) >> 6;
            __syncthreads();
            if ((threadIdx.x & 63) == 0) part[wave] = dot;
            __syncthreads();
            if (threadIdx.x == 0) {
                dot = 0.f;
                for (unsigned q = 0; q < blockDim.x / 64; ++q) dot += part[wave + q];
            }
        }
        if (threadIdx.x == 0 && live) a.dweights[t * a.k + j] = dot;
    }
}

// threads along a row: a power of two, at most 256
dim3 row_block(int64_t C) {
    unsigned x = 1;
    while (x < 256 && x < C) x *= 2;
    return dim3(x, 256 / x);
}

}  // namespace

// one block also without tokens: it writes the offsets
int64_t route_blocks(int64_t T) { return T > 0 ? ceil_div(T, kRouteTokens) : 1; }

hipError_t launch_moe_route(const float* logits, int64_t T, int32_t E, int32_t k, int renormalize, int32_t* experts,
                            float* weights, int32_t* offsets, int32_t* positions, int32_t* table, hipStream_t s) {
    RouteArgs a{logits, experts, weights, offsets, positions, table, T, route_blocks(T), E, k, renormalize};
    const dim3 grid((unsigned)a.blocks), block(kRouteThreads);
    timing_mark("moe_select_kernel", s);
    if (E <= 256) hipLaunchKernelGGL(moe_select_kernel<1>, grid, block, 0, s, a);
    else if (E <= 512) hipLaunchKernelGGL(moe_select_kernel<2>, grid, block, 0, s, a);
    else hipLaunchKernelGGL(moe_select_kernel<4>, grid, block, 0, s, a);
    hipError_t err = hipGetLastError();
    if (err == hipSuccess && a.blocks > 1) {
        timing_mark("moe_scan_kernel", s);
        hipLaunchKernelGGL(moe_scan_kernel, dim3((unsigned)ceil_div(E, 64)), block, 0, s, a);
        err = hipGetLastError();
        if (err == hipSuccess) {
            timing_mark("moe_place_kernel", s);
            hipLaunchKernelGGL(moe_place_kernel, grid, block, 0, s, a);
            err = hipGetLastError();
        }
    }
    timing_end(s);
    return err;
}

hipError_t launch_moe_route_grad(const float* dweights, const float* logits, const int32_t* experts,
                                 const float* weights, int64_t T, int32_t E, int32_t k, int renormalize,
                                 float* dlogits, hipStream_t s) {
    RouteGradArgs a{dweights, logits, experts, weights, dlogits, T, E, k, renormalize};
    const dim3 grid((unsigned)ceil_div(T, 4)), block(256);
    timing_mark("moe_route_grad_kernel", s);
    if (E <= 256) hipLaunchKernelGGL(moe_route_grad_kernel<1>, grid, block, 0, s, a);
    else if (E <= 512) hipLaunchKernelGGL(moe_route_grad_kernel<2>, grid, block, 0, s, a);
    else hipLaunchKernelGGL(moe_route_grad_kernel<4>, grid, block, 0, s, a);
    timing_end(s);
    return hipGetLastError();
}

hipError_t launch_moe_dispatch(const void* X, const int32_t* positions, int64_t T, int32_t k, int64_t H, bool bf16,
                               void* rows, hipStream_t s) {
    RowArgs a{X, nullptr, positions, nullptr, rows, nullptr, T, H / 8, k};
    const dim3 block = row_block(a.C), grid((unsigned)ceil_div(T, block.y));
    timing_mark("moe_dispatch_kernel", s);
    if (bf16) hipLaunchKernelGGL(moe_dispatch_kernel<true>, grid, block, 0, s, a);
    else hipLaunchKernelGGL(moe_dispatch_kernel<false>, grid, block, 0, s, a);
    timing_end(s);
    return hipGetLastError();
}

hipError_t launch_moe_combine(const void* rows, const int32_t* positions, const float* weights, int64_t T, int32_t k,
                              int64_t H, bool bf16, void* out, hipStream_t s) {
    RowArgs a{rows, nullptr, positions, weights, out, nullptr, T, H / 8, k};
    const dim3 block = row_block(a.C), grid((unsigned)ceil_div(T, block.y));
    timing_mark("moe_combine_kernel", s);
    if (bf16) hipLaunchKernelGGL(moe_combine_kernel<true>, grid, block, 0, s, a);
    else hipLaunchKernelGGL(moe_combine_kernel<false>, grid, block, 0, s, a);
    timing_end(s);
    return hipGetLastError();
}

hipError_t launch_moe_combine_grad(const void* dout, const void* rows, const int32_t* positions, const float* weights,
                                   int64_t T, int32_t k, int64_t H, bool bf16, void* drows, float* dweights,
                                   hipStream_t s) {
    RowArgs a{dout, rows, positions, weights, drows, dweights, T, H / 8, k};
    const dim3 block = row_block(a.C), grid((unsigned)ceil_div(T, block.y));
    timing_mark("moe_combine_grad_kernel", s);
    if (bf16) hipLaunchKernelGGL(moe_combine_grad_kernel<true>, grid, block, 0, s, a);
    else hipLaunchKernelGGL(moe_combine_grad_kernel<false>, grid, block, 0, s, a);
    timing_end(s);
    return hipGetLastError();
}

}  // namespace drgg
