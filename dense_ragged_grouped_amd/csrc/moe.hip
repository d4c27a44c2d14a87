// moe.hip -- gfx950 (CDNA4) kernels around the grouped products of an expert
// layer: the router's selection and its gradient, and the movement of rows
// between the token order and the grouped order, with its gradients.
//
// All of them are bound by memory or, for a few tokens, by launch latency.
// Nothing here uses an atomic whose order could change a result.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "internal.hpp"
#include "plan.hpp"
#include "quantize.hpp"

namespace drgg {

namespace {

// ---------------------------------------------------------------------------
// selection
//
// Sixteen lanes per token, one DPP row, so that a wave works on four tokens
// and a maximum over a token's lanes is four rotations in the vector unit.
// Lane l of the row holds the logits of experts 64c + 4l + i in key[4c + i].
// A logit is compared through a 32-bit key whose unsigned order is the order
// of the values (NaN above +inf, -0 equal to +0); key 0 marks an expert
// already taken or past E.  Each of the k rounds takes the largest key of the
// row, at the lowest expert index among equals; lane j % 16 keeps round j's
// choice in its slot j / 16.

__device__ __forceinline__ uint32_t order_key(float v) {
    if (v != v) return 0xFFFFFFFFu;
    const uint32_t u = __float_as_uint(v + 0.f);   // -0 + 0 = +0
    return u & 0x80000000u ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ float key_value(uint32_t k) {
    return __uint_as_float(k & 0x80000000u ? k & 0x7FFFFFFFu : ~k);   // NaN: 0x7FFFFFFF, a NaN
}

// v of the lane N places on in the row of 16 (cyclic)
template <int N>
__device__ __forceinline__ uint32_t row_rotate(uint32_t v) {
    return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x120 + N, 0xF, 0xF, false);
}
__device__ __forceinline__ uint32_t row_max(uint32_t v) {
    v = max(v, row_rotate<8>(v));
    v = max(v, row_rotate<4>(v));
    v = max(v, row_rotate<2>(v));
    return max(v, row_rotate<1>(v));
}
__device__ __forceinline__ uint32_t row_min(uint32_t v) {
    v = min(v, row_rotate<8>(v));
    v = min(v, row_rotate<4>(v));
    v = min(v, row_rotate<2>(v));
    return min(v, row_rotate<1>(v));
}
// the same bits in all lanes: every lane adds the same pairs of pairs
__device__ __forceinline__ float row_sum(float v) {
    v += __uint_as_float(row_rotate<8>(__float_as_uint(v)));
    v += __uint_as_float(row_rotate<4>(__float_as_uint(v)));
    v += __uint_as_float(row_rotate<2>(__float_as_uint(v)));
    return v + __uint_as_float(row_rotate<1>(__float_as_uint(v)));
}

// The logits of one token as keys; none when !live.
template <int V>
__device__ __forceinline__ void load_keys(uint32_t (&key)[V], const float* row, int E, int l, bool live) {
    const bool vec = (E & 3) == 0;
#pragma unroll
    for (int c = 0; c < V / 4; ++c) {
        const int e = 64 * c + 4 * l;
        f32x4 v = {0.f, 0.f, 0.f, 0.f};
        if (vec) {
            if (live && e < E) v = *reinterpret_cast<const f32x4*>(row + e);
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (live && e + i < E) v[i] = row[e + i];
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) key[4 * c + i] = live && e + i < E ? order_key(v[i]) : 0;
    }
}

struct RouteArgs {
    const float* logits;
    int32_t* experts;
    float* weights;
    int32_t* offsets;
    int32_t* positions;
    int32_t* tokens;   // may be null
    void* table;   // counts per block and expert, see moe_select_kernel
    int64_t T, blocks;
    int32_t E, k, renormalize;
};

constexpr int kRouteThreads = 1024, kRouteWaves = kRouteThreads / 64;
constexpr int kRouteTokens = 64;   // tokens per block: four per wave, one 64-bit mask per expert
// up to this many blocks moe_place_kernel sums the earlier blocks' counts
// itself (each block reads every count, E bytes per block: 64 KB of L2 reads
// each for 16384 tokens on 256 experts); beyond, a scan kernel does it once
constexpr int64_t kRouteBytes = 512;

__device__ __forceinline__ int table_stride(int E) { return (E + 3) & ~3; }

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
// offsets and final positions are written here; otherwise positions hold the
// ranks for moe_place_kernel and the counts go to the table: bytes (at most
// 64 each) [blocks][E rounded up to 4], or with more than kRouteBytes blocks
// words [blocks][E] for moe_scan_kernel.
// Bound by the k dependent rounds: 12 us for 16384 tokens, k = 8 of 256 experts
// (16.8 MB of logits, 3.4 us at the rate of a large copy), of which the rounds'
// 88 vector instructions take about 4.7 us to issue and the rest is waiting, part
// of it between a compare and the select that reads its mask; 4 us for 2039 tokens, k = 2 of 32; with a wave per token and shuffles through LDS
// 21 and 12 us.
template <int V, int S>
__device__ __forceinline__ void select_tokens(const RouteArgs& a) {
    __shared__ unsigned long long mask[16 * V];
    __shared__ int32_t start[16 * V], tmp[kRouteWaves];
    const int lane = threadIdx.x & 63, l = lane & 15;
    const int E = a.E, k = a.k;
    for (int e = threadIdx.x; e < E; e += kRouteThreads) mask[e] = 0;
    __syncthreads();
    const int tl = threadIdx.x >> 4;   // token of the block
    const int64_t t = (int64_t)blockIdx.x * kRouteTokens + tl;
    const bool live = t < a.T;
    uint32_t key[V], kept[S], top = 0;
    int32_t mine[S];
    load_keys<V>(key, a.logits + t * E, E, l, live);
    // a wave without tokens does not compete with the others
    const int rounds = (int64_t)blockIdx.x * kRouteTokens + (__builtin_amdgcn_readfirstlane(threadIdx.x) >> 4) < a.T ? k : 0;
    for (int j = 0; j < rounds; ++j) {
        uint32_t m[V];
#pragma unroll
        for (int i = 0; i < V; ++i) m[i] = key[i];
#pragma unroll
        for (int d = 1; d < V; d *= 2)
#pragma unroll
            for (int i = 0; i < V; i += 2 * d) m[i] = max(m[i], m[i + d]);
        const uint32_t best = row_max(m[0]);
        // the lane's lowest expert with that key (no chain through the keys:
        // a wave alone on its SIMD waits for every dependent result)
        uint32_t is[V];
#pragma unroll
        for (int i = 0; i < V; ++i) is[i] = key[i] == best ? (uint32_t)(64 * (i >> 2) + (i & 3)) : 0xFFFFu;
#pragma unroll
        for (int d = 1; d < V; d *= 2)
#pragma unroll
            for (int i = 0; i < V; i += 2 * d) is[i] = min(is[i], is[i + d]);
        const uint32_t e = row_min(is[0] + 4 * l);   // above every index where there is none
        const uint32_t mine_at = e - 4 * l;          // the taken key's place, if it is this lane's
#pragma unroll
        for (int i = 0; i < V; ++i) key[i] = mine_at == (uint32_t)(64 * (i >> 2) + (i & 3)) ? 0u : key[i];
        if (j == 0) top = best;
#pragma unroll
        for (int s = 0; s < S; ++s)
            if (j == 16 * s + l) {
                kept[s] = best;
                mine[s] = (int32_t)e;
            }
    }
    // softmax over the chosen, or over all experts (the keys of the chosen
    // are gone, their terms are the p)
    const float most = key_value(top);
    const bool none = most == -INFINITY;   // every expert is masked: all weights 0
    float p[S], total = 0.f;
#pragma unroll
    for (int s = 0; s < S; ++s) {
        p[s] = 16 * s + l < k && !none ? expf(key_value(kept[s]) - most) : 0.f;
        total += p[s];
    }
    if (!a.renormalize && !none) {
#pragma unroll
        for (int i = 0; i < V; ++i) total += key[i] ? expf(key_value(key[i]) - most) : 0.f;
    }
    total = row_sum(total);
    if (live) {
#pragma unroll
        for (int s = 0; s < S; ++s) {
            const int j = 16 * s + l;
            if (j < k) {
                a.experts[t * k + j] = mine[s];
                a.weights[t * k + j] = none ? 0.f : p[s] / total;
                atomicOr(&mask[mine[s]], 1ull << tl);
            }
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
    } else if (a.blocks <= kRouteBytes) {
        const int stride = table_stride(E);
        for (int e = threadIdx.x; e < stride; e += kRouteThreads)
            static_cast<uint8_t*>(a.table)[(int64_t)blockIdx.x * stride + e] = e < E ? (uint8_t)__popcll(mask[e]) : 0;
    } else {
        for (int e = threadIdx.x; e < E; e += kRouteThreads)
            static_cast<int32_t*>(a.table)[(int64_t)blockIdx.x * E + e] = __popcll(mask[e]);
    }
    if (!live) return;
#pragma unroll
    for (int s = 0; s < S; ++s) {
        const int j = 16 * s + l;
        if (j < k) {
            int32_t r = __popcll(mask[mine[s]] & ((1ull << tl) - 1));
            if (single) {
                r += start[mine[s]];
                if (a.tokens) a.tokens[r] = (int32_t)t;
            }
            a.positions[t * k + j] = r;
        }
    }
}

template <int V, int S>
__global__ __launch_bounds__(kRouteThreads) void moe_select_kernel(RouteArgs a) {
    select_tokens<V, S>(a);
}

// The selection and, on workgroups after its own, the quantisation of the same
// tokens' rows (BF16, at most 4096 values: HELD).  They need nothing of each
// other; in one launch the one fills the other's waits, and a launch less
// counts for a few tokens (8 tokens: 3.5 us of the serving block's 38).
template <int V, int S>
__global__ __launch_bounds__(kRouteThreads) void moe_select_quantize_kernel(RouteArgs a, QuantArgs q, int nx) {
    __shared__ uint32_t part[kRouteWaves];
    if (blockIdx.x < a.blocks)
        select_tokens<V, S>(a);
    else
        quantize_rows<true, true>(q, part, threadIdx.x & (nx - 1), threadIdx.x / nx, nx, kRouteThreads / nx,
                                  blockIdx.x - a.blocks, gridDim.x - a.blocks);
}

// More than kRouteBytes blocks: the table's columns to exclusive prefixes over
// the blocks, and each expert's total after them.  One lane per expert; the
// 16 waves of a workgroup each take a run of blocks, sum it, and write its
// prefixes.
__global__ __launch_bounds__(kRouteThreads) void moe_scan_kernel(RouteArgs a) {
    __shared__ int32_t sums[kRouteWaves][64];
    int32_t* table = static_cast<int32_t*>(a.table);
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int e = blockIdx.x * 64 + lane;
    const bool ok = e < a.E;
    const int64_t per = (a.blocks + kRouteWaves - 1) / kRouteWaves;
    const int64_t lo = min(wave * per, a.blocks), hi = min(lo + per, a.blocks);
    int32_t s = 0;
    if (ok)
        for (int64_t b = lo; b < hi; ++b) s += table[b * a.E + e];
    sums[wave][lane] = s;
    __syncthreads();
    int32_t acc = 0;
    for (int w = 0; w < wave; ++w) acc += sums[w][lane];
    if (ok) {
        for (int64_t b = lo; b < hi; ++b) {
            const int32_t n = table[b * a.E + e];
            table[b * a.E + e] = acc;
            acc += n;
        }
        if (wave == kRouteWaves - 1) table[a.blocks * a.E + e] = acc;
    }
}

// positions += the expert's offset + its pairs in earlier blocks.  BYTES: the
// block sums the count bytes of all blocks itself, four experts per thread
// and the blocks cut into at most 16 slices over the other threads; two
// 16-bit sums per word hold them (kRouteBytes * 64 < 2^16).
template <bool BYTES>
__global__ __launch_bounds__(kRouteThreads) void moe_place_kernel(RouteArgs a) {
    __shared__ int32_t base[kMaxExperts], tmp[kRouteWaves];
    __shared__ u32x4 part[BYTES ? kRouteThreads : 1];
    const int E = a.E, tid = threadIdx.x;
    int32_t before = 0, n = 0;   // of expert tid: pairs in earlier blocks, and in all
    if constexpr (BYTES) {
        static_assert(kRouteBytes * kRouteTokens < 65536, "16-bit sums");
        const int quads = table_stride(E) / 4, slices = min(kRouteThreads / quads, 16);
        const int q = tid % quads, sl = tid / quads, blocks = (int)a.blocks, me = (int)blockIdx.x;
        u32x4 s = {0, 0, 0, 0};   // earlier: experts 0 and 2, 1 and 3 of the quad; all: the same
        if (sl < slices) {
            const uint32_t* col = static_cast<const uint32_t*>(a.table) + q;
#pragma unroll 8
            for (int b = sl; b < blocks; b += slices) {
                const uint32_t v = col[(int64_t)b * quads];
                const uint32_t even = v & 0x00FF00FFu, odd = (v >> 8) & 0x00FF00FFu;
                s[0] += b < me ? even : 0;
                s[1] += b < me ? odd : 0;
                s[2] += even;
                s[3] += odd;
            }
        }
        part[tid] = s;
        __syncthreads();
        if (tid < E) {
            const int i = tid & 3;
            for (int w = 0; w < slices; ++w) {
                const u32x4 v = part[w * quads + tid / 4];
                before += (v[i & 1] >> (8 * (i & 2))) & 0xFFFFu;
                n += (v[2 + (i & 1)] >> (8 * (i & 2))) & 0xFFFFu;
            }
        }
    } else if (tid < E) {
        before = static_cast<const int32_t*>(a.table)[(int64_t)blockIdx.x * E + tid];
        n = static_cast<const int32_t*>(a.table)[a.blocks * E + tid];
    }
    const int32_t s = block_prefix(n, tmp);
    if (tid < E) {
        base[tid] = s + before;
        if (blockIdx.x == 0) {
            a.offsets[tid] = s;
            if (tid == E - 1) a.offsets[E] = s + n;
        }
    }
    __syncthreads();
    const int64_t p0 = (int64_t)blockIdx.x * kRouteTokens * a.k;
    const int64_t p1 = min(p0 + (int64_t)kRouteTokens * a.k, a.T * a.k);
    // pair / k by a multiplication, exact for the block's pairs (below 64 * 64)
    const uint32_t by_k = ((1u << 20) + a.k - 1) / a.k;
    for (int64_t p = p0 + tid; p < p1; p += kRouteThreads) {
        const int32_t at = a.positions[p] + base[a.experts[p]];
        a.positions[p] = at;
        if (a.tokens) a.tokens[at] = (int32_t)(blockIdx.x * kRouteTokens + (((uint32_t)(p - p0) * by_k) >> 20));
    }
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

// dlogits, sixteen lanes per token as above.  With s = sum_j w_j dw_j:
//   softmax over the chosen: w_j (dw_j - s) at the chosen, 0 elsewhere;
//   softmax over all: p_e (dw_e - s), dw_e = 0 but at the chosen, where p_e
//   is w_j; the p are recomputed from the logits.
// An expert of probability 0 gets 0 and its dw_j is not used: a masked
// expert's row, and so its dw_j, may hold anything.
// The row is first written as if no expert were chosen, then lane j writes
// the chosen ones; the fence between makes the second store the last.
template <int V>
__global__ __launch_bounds__(256) void moe_route_grad_kernel(RouteGradArgs a) {
    const int l = threadIdx.x & 15;
    const int64_t t = (int64_t)blockIdx.x * 16 + (threadIdx.x >> 4);
    const int E = a.E, k = a.k;
    const bool live = t < a.T;
    float s = 0.f;
    if (live)
        for (int j = l; j < k; j += 16) {
            const float w = a.weights[t * k + j];
            s += w != 0.f ? w * a.dweights[t * k + j] : 0.f;
        }
    s = row_sum(s);
    float g[V];
    if (a.renormalize) {
#pragma unroll
        for (int i = 0; i < V; ++i) g[i] = 0.f;
    } else {
        uint32_t key[V], m = 0;
        load_keys<V>(key, a.logits + t * E, E, l, live);
#pragma unroll
        for (int i = 0; i < V; ++i) m = max(m, key[i]);
        const float most = key_value(row_max(m));
        const bool none = most == -INFINITY;
        float total = 0.f;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            g[i] = key[i] && !none ? expf(key_value(key[i]) - most) : 0.f;
            total += g[i];
        }
        total = row_sum(total);
#pragma unroll
        for (int i = 0; i < V; ++i) g[i] = g[i] == 0.f ? 0.f : -s * (g[i] / total);
    }
    float* out = a.dlogits + t * E;
    if (live) {
#pragma unroll
        for (int c = 0; c < V / 4; ++c) {
            const int e = 64 * c + 4 * l;
            if ((E & 3) == 0) {
                if (e < E) *reinterpret_cast<f32x4*>(out + e) = f32x4{g[4 * c], g[4 * c + 1], g[4 * c + 2], g[4 * c + 3]};
            } else {
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (e + i < E) out[e + i] = g[4 * c + i];
            }
        }
    }
    __syncthreads();   // the row's stores are performed before the ones below
    if (live)
        for (int j = l; j < k; j += 16) {
            const int32_t e = a.experts[t * k + j];
            const float w = a.weights[t * k + j];
            if (e >= 0 && e < E) out[e] = w != 0.f ? w * (a.dweights[t * k + j] - s) : 0.f;
        }
}

// fn(V), the keys per lane for E experts, as an integral constant
template <class Fn>
void for_experts(int32_t E, Fn&& fn) {
    if (E <= 64) fn(std::integral_constant<int, 4>{});
    else if (E <= 128) fn(std::integral_constant<int, 8>{});
    else if (E <= 256) fn(std::integral_constant<int, 16>{});
    else if (E <= 512) fn(std::integral_constant<int, 32>{});
    else fn(std::integral_constant<int, 64>{});
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
    const int64_t R = a.T * a.k, step = (int64_t)gridDim.x * blockDim.y;
    for (int64_t t = (int64_t)blockIdx.x * blockDim.y + threadIdx.y; t < a.T; t += step)
        for (int64_t c = threadIdx.x; c < a.C; c += blockDim.x) {
            Piece<BF16> x;
            x.load(a.src, t * a.C + c);
            for (int j = 0; j < a.k; ++j) {
                const int64_t p = a.positions[t * a.k + j];
                if (p >= 0 && p < R) x.store(a.dst, p * a.C + c);
            }
        }
}

// The grouped rows of pairs j0 .. j0+3 of token t and their weights; row -1
// for a pair past k, a position outside the rows, or a token past the end.
constexpr int kPairs = 4;
__device__ __forceinline__ void load_pairs(const RowArgs& a, int64_t t, int j0, int64_t (&row)[kPairs],
                                           float (&w)[kPairs]) {
    const int64_t R = a.T * a.k;
#pragma unroll
    for (int u = 0; u < kPairs; ++u) {
        const bool in = t < a.T && j0 + u < a.k;
        const int64_t p = in ? a.positions[t * a.k + j0 + u] : -1;
        row[u] = p < R ? p : -1;
        w[u] = in && a.weights ? a.weights[t * a.k + j0 + u] : 1.f;
    }
}

// FP32 sum over j in order, one rounding.  Four rows are loaded before the
// first is added.  Bound by memory: 604 MB for 16384 tokens, k = 8, H = 2048 in
// BF16 in 117 to 135 us (5.2 to 4.5 TB/s; a large copy reaches 5.0), 140 us with
// one row at a time.  Non-temporal loads and stores gained 7 % there and cost
// 15 to 25 % where the rows or the result still fit the last-level cache.
template <bool BF16>
__global__ __launch_bounds__(256) void moe_combine_kernel(RowArgs a) {
    const int64_t step = (int64_t)gridDim.x * blockDim.y;
    for (int64_t t = (int64_t)blockIdx.x * blockDim.y + threadIdx.y; t < a.T; t += step)
        for (int64_t c = threadIdx.x; c < a.C; c += blockDim.x) {
            float s[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
            for (int j0 = 0; j0 < a.k; j0 += kPairs) {
                int64_t row[kPairs];
                float w[kPairs];
                load_pairs(a, t, j0, row, w);
                Piece<BF16> x[kPairs];
#pragma unroll
                for (int u = 0; u < kPairs; ++u)
                    if (row[u] >= 0) x[u].load(a.src, row[u] * a.C + c);
#pragma unroll
                for (int u = 0; u < kPairs; ++u)
                    if (row[u] >= 0) {
#pragma unroll
                        for (int i = 0; i < 8; ++i) s[i] += w[u] * x[u].get(i);
                    }
            }
            Piece<BF16> y;
            y.set(s);
            y.store(a.dst, t * a.C + c);
        }
}

// drows[position] = w * dout (one rounding) and dweights = <dout, row>, an
// FP32 sum: per thread over its pieces, then over the token's threads in a
// fixed tree.  Four pairs at a time.  Bound by memory: 1.14 GB at those sizes
// in 210 to 226 us.
template <bool BF16>
__global__ __launch_bounds__(256) void moe_combine_grad_kernel(RowArgs a) {
    __shared__ float part[4][kPairs];
    // whole blocks of tokens: every thread takes part in the sums
    for (int64_t t0 = (int64_t)blockIdx.x * blockDim.y; t0 < a.T; t0 += (int64_t)gridDim.x * blockDim.y) {
        const int64_t t = t0 + threadIdx.y;
        for (int j0 = 0; j0 < a.k; j0 += kPairs) {
            int64_t row[kPairs];
            float w[kPairs], dot[kPairs] = {0.f, 0.f, 0.f, 0.f};
            load_pairs(a, t, j0, row, w);
            if (t < a.T)
                for (int64_t c = threadIdx.x; c < a.C; c += blockDim.x) {
                    Piece<BF16> g, x[kPairs];
                    g.load(a.src, t * a.C + c);
#pragma unroll
                    for (int u = 0; u < kPairs; ++u)
                        if (row[u] >= 0) x[u].load(a.rows, row[u] * a.C + c);
#pragma unroll
                    for (int u = 0; u < kPairs; ++u)
                        if (row[u] >= 0) {
                            float f[8];
#pragma unroll
                            for (int i = 0; i < 8; ++i) {
                                dot[u] += g.get(i) * x[u].get(i);
                                f[i] = w[u] * g.get(i);
                            }
                            Piece<BF16> y;
                            y.set(f);
                            y.store(a.dst, row[u] * a.C + c);
                        }
                }
            // the token's threads: up to 64 lanes of one wave, then whole waves
            const int width = blockDim.x < 64 ? blockDim.x : 64;
            for (int m = 1; m < width; m <<= 1)
#pragma unroll
                for (int u = 0; u < kPairs; ++u) dot[u] += __shfl_xor(dot[u], m, 64);
            if (blockDim.x > 64) {
                const int wave = (threadIdx.y * blockDim.x + threadIdx.x) >> 6;
                __syncthreads();
                if ((threadIdx.x & 63) == 0)
#pragma unroll
                    for (int u = 0; u < kPairs; ++u) part[wave][u] = dot[u];
                __syncthreads();
                if (threadIdx.x == 0) {
#pragma unroll
                    for (int u = 0; u < kPairs; ++u) dot[u] = 0.f;
                    for (unsigned q = 0; q < blockDim.x / 64; ++q)
#pragma unroll
                        for (int u = 0; u < kPairs; ++u) dot[u] += part[wave + q][u];
                }
            }
            if (threadIdx.x == 0 && t < a.T)
#pragma unroll
                for (int u = 0; u < kPairs; ++u)
                    if (j0 + u < a.k) a.dweights[t * a.k + j0 + u] = dot[u];
        }
    }
}

// threads along a row: a power of two, at most 256
dim3 row_block(int64_t C) {
    unsigned x = 1;
    while (x < 256 && x < C) x *= 2;
    return dim3(x, 256 / x);
}
// a launch has fewer than 2^32 threads: blocks walk the tokens beyond
dim3 row_grid(int64_t T, dim3 block) {
    const int64_t n = ceil_div(T, block.y), most = 65536;
    return dim3((unsigned)(n < most ? n : most));
}

}  // namespace

// one block also without tokens: it writes the offsets
static int64_t route_blocks(int64_t T) { return T > 0 ? ceil_div(T, kRouteTokens) : 1; }

size_t route_table_bytes(int64_t T, int32_t E) {
    const int64_t n = route_blocks(T);   // at most 2^25, so the table stays below 2^38 bytes
    if (n == 1) return 0;
    return (size_t)(n <= kRouteBytes ? n * round_up(E, 4) : (n + 1) * E * 4);
}

hipError_t launch_moe_route(const float* logits, int64_t T, int32_t E, int32_t k, int renormalize, int32_t* experts,
                            float* weights, int32_t* offsets, int32_t* positions, int32_t* tokens, void* table,
                            hipStream_t s, const QuantArgs* quantize) {
    RouteArgs a{logits, experts, weights, offsets, positions, tokens, table, T, route_blocks(T), E, k, renormalize};
    const dim3 grid((unsigned)a.blocks), block(kRouteThreads);
    if (quantize) {
        const int nx = (int)quantize_threads(quantize->C);
        const int64_t n = ceil_div(T, kRouteThreads / nx);
        const dim3 both((unsigned)(a.blocks + (n < 65536 ? n : 65536)));
        timing_mark("moe_select_quantize_kernel", s);
        for_experts(E, [&](auto v) {
            constexpr int V = decltype(v)::value;
            if (k <= 16) hipLaunchKernelGGL((moe_select_quantize_kernel<V, 1>), both, block, 0, s, a, *quantize, nx);
            else hipLaunchKernelGGL((moe_select_quantize_kernel<V, 4>), both, block, 0, s, a, *quantize, nx);
        });
    } else {
        timing_mark("moe_select_kernel", s);
        for_experts(E, [&](auto v) {
            constexpr int V = decltype(v)::value;
            if (k <= 16) hipLaunchKernelGGL((moe_select_kernel<V, 1>), grid, block, 0, s, a);
            else hipLaunchKernelGGL((moe_select_kernel<V, 4>), grid, block, 0, s, a);
        });
    }
    if (a.blocks > kRouteBytes) {
        timing_mark("moe_scan_kernel", s);
        hipLaunchKernelGGL(moe_scan_kernel, dim3((unsigned)ceil_div(E, 64)), block, 0, s, a);
    }
    if (a.blocks > 1) {
        timing_mark("moe_place_kernel", s);
        if (a.blocks > kRouteBytes) hipLaunchKernelGGL(moe_place_kernel<false>, grid, block, 0, s, a);
        else hipLaunchKernelGGL(moe_place_kernel<true>, grid, block, 0, s, a);
    }
    timing_end(s);
    return hipGetLastError();
}

hipError_t launch_moe_route_grad(const float* dweights, const float* logits, const int32_t* experts,
                                 const float* weights, int64_t T, int32_t E, int32_t k, int renormalize,
                                 float* dlogits, hipStream_t s) {
    RouteGradArgs a{dweights, logits, experts, weights, dlogits, T, E, k, renormalize};
    const dim3 grid((unsigned)ceil_div(T, 16)), block(256);
    timing_mark("moe_route_grad_kernel", s);
    for_experts(E, [&](auto v) {
        hipLaunchKernelGGL(moe_route_grad_kernel<decltype(v)::value>, grid, block, 0, s, a);
    });
    timing_end(s);
    return hipGetLastError();
}

hipError_t launch_moe_dispatch(const void* X, const int32_t* positions, int64_t T, int32_t k, int64_t H, bool bf16,
                               void* rows, hipStream_t s) {
    RowArgs a{X, nullptr, positions, nullptr, rows, nullptr, T, H / 8, k};
    const dim3 block = row_block(a.C), grid = row_grid(T, block);
    timing_mark("moe_dispatch_kernel", s);
    if (bf16) hipLaunchKernelGGL(moe_dispatch_kernel<true>, grid, block, 0, s, a);
    else hipLaunchKernelGGL(moe_dispatch_kernel<false>, grid, block, 0, s, a);
    timing_end(s);
    return hipGetLastError();
}

hipError_t launch_moe_combine(const void* rows, const int32_t* positions, const float* weights, int64_t T, int32_t k,
                              int64_t H, bool bf16, void* out, hipStream_t s) {
    RowArgs a{rows, nullptr, positions, weights, out, nullptr, T, H / 8, k};
    const dim3 block = row_block(a.C), grid = row_grid(T, block);
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
    const dim3 block = row_block(a.C), grid = row_grid(T, block);
    timing_mark("moe_combine_grad_kernel", s);
    if (bf16) hipLaunchKernelGGL(moe_combine_grad_kernel<true>, grid, block, 0, s, a);
    else hipLaunchKernelGGL(moe_combine_grad_kernel<false>, grid, block, 0, s, a);
    timing_end(s);
    return hipGetLastError();
}

}  // namespace drgg
