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
#include "mxfp4.hpp"
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

// ---------------------------------------------------------------------------
// selection by scores
//
// The same rounds on keys of v = s + bias, s the sigmoid or softmax score.  A
// choice is that of 64-bit values: FP32 values are off by at most `off` (see
// below), so where two that decide something -- neighbours among the chosen,
// the last chosen and the best left, the last kept group and the best left --
// are no further apart than both errors, the token is chosen again from values
// in 64 bits, by its whole wave.

struct ScoreArgs {
    const float* bias;
    int32_t groups, top_groups, best;
    int32_t by_logits;   // no bias, one group: the order is that of the logits
    float scale;
};

// The largest key of the row of lanes.  Four running values (a wave alone on
// its SIMD waits for every dependent result; a tree would hold V/2 more).
template <int V>
__device__ __forceinline__ uint32_t best_key(const uint32_t (&key)[V]) {
    uint32_t m[4] = {key[0], key[1], key[2], key[3]};
#pragma unroll
    for (int i = 4; i < V; ++i) m[i & 3] = max(m[i & 3], key[i]);
    return row_max(max(max(m[0], m[1]), max(m[2], m[3])));
}
// the lowest expert with it, whose key becomes 0
template <int V>
__device__ __forceinline__ uint32_t take_best(uint32_t (&key)[V], int l, uint32_t* best) {
    *best = best_key<V>(key);
    uint32_t is[4] = {0xFFFFu, 0xFFFFu, 0xFFFFu, 0xFFFFu};
#pragma unroll
    for (int i = V - 1; i >= 0; --i) is[i & 3] = key[i] == *best ? (uint32_t)(64 * (i >> 2) + (i & 3)) : is[i & 3];
    const uint32_t e = row_min(min(min(is[0], is[1]), min(is[2], is[3])) + 4 * l);   // above every index where there is none
    const uint32_t mine_at = e - 4 * l;          // the taken key's place, if it is this lane's
#pragma unroll
    for (int i = 0; i < V; ++i) key[i] = mine_at == (uint32_t)(64 * (i >> 2) + (i & 3)) ? 0u : key[i];
    return e;
}

constexpr float kUnit = 0x1p-24f;   // half a step of FP32, relative

// the score of a logit; most and total: the softmax's (most finite)
template <bool SIGMOID, class F>
__device__ __forceinline__ F score(float x, F most, F total) {
    if constexpr (SIGMOID) {
        const F e = exp(-fabs((F)x)), q = 1 / (1 + e);
        return x < 0 ? e * q : q;   // NaN: q
    } else {
        return exp((F)x - most) / total;
    }
}
// v; every part is computed and then chosen from (a branch per expert costs
// more than the exponential)
template <bool SIGMOID, class F>
__device__ __forceinline__ F score_value(float x, float bias, F most, F total) {
    const F v = score<SIGMOID, F>(x, most, total) + (F)bias;
    return ((x == -INFINITY) | (bias == -INFINITY)) ? (F)-INFINITY : v;
}

// The same in FP32 with the hardware's exponential and reciprocal, within
// `off` (select_by_scores) of it; inverse = 1 / total.
template <bool SIGMOID>
__device__ __forceinline__ float score_value32(float x, float bias, float most, float inverse) {
    float v;
    if constexpr (SIGMOID) {
        const float e = __builtin_amdgcn_exp2f(fabsf(x) * -1.44269504f), q = __builtin_amdgcn_rcpf(1.f + e);
        v = (x < 0 ? e * q : q) + bias;
    } else {
        v = __builtin_amdgcn_exp2f((x - most) * 1.44269504f) * inverse + bias;
    }
    return ((x == -INFINITY) | (bias == -INFINITY)) ? -INFINITY : v;
}

// the two largest of two pairs' four keys
__device__ __forceinline__ void merge_two(uint32_t& one, uint32_t& two, uint32_t o1, uint32_t o2) {
    two = max(min(one, o1), max(two, o2));
    one = max(one, o1);
}
template <int CTRL>
__device__ __forceinline__ void merge_lanes(uint32_t& one, uint32_t& two) {
    merge_two(one, two, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)one, CTRL, 0xF, 0xF, false),
              (uint32_t)__builtin_amdgcn_update_dpp(0, (int)two, CTRL, 0xF, 0xF, false));
}
// a group's value from its two largest keys (0: none)
__device__ __forceinline__ uint32_t group_key(uint32_t one, uint32_t two, int best) {
    const uint32_t sum = order_key(key_value(one) + key_value(two));
    return best == 2 && two != 0 && key_value(two) != -INFINITY ? sum : one;
}

__device__ __forceinline__ uint64_t order_key64(double v) {
    const uint64_t u = __builtin_bit_cast(uint64_t, v + 0.0), key = u >> 63 ? ~u : u | 1ull << 63;
    return v != v ? ~0ull : key;
}
__device__ __forceinline__ double key_value64(uint64_t k) {
    return __builtin_bit_cast(double, k >> 63 ? k & ~(1ull << 63) : ~k);   // NaN: all ones, a NaN
}
// fn(v, v of other lanes) over the wave, in all lanes: rotations in the rows of
// 16, then exchanges of rows and halves, all in the vector unit (shuffles through
// LDS would wait some hundred cycles each, twelve times)
template <class Fn>
__device__ __forceinline__ uint64_t wave_reduce64(uint64_t v, Fn fn) {
    auto both = [](uint32_t lo, uint32_t hi) { return (uint64_t)hi << 32 | lo; };
    v = fn(v, both(row_rotate<8>((uint32_t)v), row_rotate<8>((uint32_t)(v >> 32))));
    v = fn(v, both(row_rotate<4>((uint32_t)v), row_rotate<4>((uint32_t)(v >> 32))));
    v = fn(v, both(row_rotate<2>((uint32_t)v), row_rotate<2>((uint32_t)(v >> 32))));
    v = fn(v, both(row_rotate<1>((uint32_t)v), row_rotate<1>((uint32_t)(v >> 32))));
    // even rows on one side, odd rows on the other; then the halves
    auto lo = __builtin_amdgcn_permlane16_swap((uint32_t)v, (uint32_t)v, false, false);
    auto hi = __builtin_amdgcn_permlane16_swap((uint32_t)(v >> 32), (uint32_t)(v >> 32), false, false);
    v = fn(both(lo[0], hi[0]), both(lo[1], hi[1]));
    lo = __builtin_amdgcn_permlane32_swap((uint32_t)v, (uint32_t)v, false, false);
    hi = __builtin_amdgcn_permlane32_swap((uint32_t)(v >> 32), (uint32_t)(v >> 32), false, false);
    return fn(both(lo[0], hi[0]), both(lo[1], hi[1]));
}
__device__ __forceinline__ uint64_t wave_max64(uint64_t v) {
    return wave_reduce64(v, [](uint64_t a, uint64_t b) { return a > b ? a : b; });
}
// the same bits in all lanes: every lane adds the same pairs of pairs
__device__ __forceinline__ double wave_sum64(double v) {
    return __builtin_bit_cast(double, wave_reduce64(__builtin_bit_cast(uint64_t, v), [](uint64_t a, uint64_t b) {
        return __builtin_bit_cast(uint64_t, __builtin_bit_cast(double, a) + __builtin_bit_cast(double, b));
    }));
}

// The largest of a wave's N*64 keys (lane l's i-th is expert 64 i + l), which
// becomes 0, and its lowest expert.
template <int N>
__device__ __forceinline__ uint64_t take_best64(uint64_t (&key)[N], int* expert) {
    uint64_t m = key[0];
#pragma unroll
    for (int i = 1; i < N; ++i) m = key[i] > m ? key[i] : m;
    m = wave_max64(m);
    int at = -1;
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const unsigned long long has = __ballot(key[i] == m);
        if (at < 0 && has) at = 64 * i + __ffsll((long long)has) - 1;
    }
    const int lane = threadIdx.x & 63;
#pragma unroll
    for (int i = 0; i < N; ++i)
        if (at == 64 * i + lane) key[i] = 0;
    *expert = at;
    return m;
}

// Token t's choice from values in 64 bits, by one wave; chosen(j, e) for each
// round.  The groups that take part are those of `open` unless regroup.
template <int N, bool SIGMOID, class Chosen>
__device__ __forceinline__ void choose64(const RouteArgs& a, const ScoreArgs& c, const float* bias, int64_t t,
                                         unsigned long long open, bool regroup, Chosen chosen) {
    int lane = threadIdx.x & 63;
    asm volatile("" : "+v"(lane));
    float x[N], top = -INFINITY;
#pragma unroll
    for (int i = 0; i < N; ++i) {
        x[i] = 64 * i + lane < a.E ? a.logits[t * a.E + 64 * i + lane] : -INFINITY;
        top = fmaxf(top, x[i]);
    }
    double most = 0, total = 1;
    if constexpr (!SIGMOID) {
        top = (float)key_value64(wave_max64(order_key64(top)));
        most = top == -INFINITY ? 0.0 : (double)top;
        total = 0;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            total += exp((double)x[i] - most);
            __builtin_amdgcn_sched_barrier(0);
        }
        total = wave_sum64(total);
    }
    uint64_t key[N];
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const int e = 64 * i + lane;
        const float b = bias[e < a.E ? e : 0];
        key[i] = e >= a.E ? 0 : order_key64(score_value<SIGMOID, double>(x[i], b, most, total));
        __builtin_amdgcn_sched_barrier(0);   // one at a time: sixteen exponentials side by side do not fit the registers
    }
    const int size = a.E / c.groups;
    if (regroup) {
        uint64_t rank = 0;   // lane g: the value of group g
        for (int g = 0; g < c.groups; ++g) {
            uint64_t in[N];
            int at;
#pragma unroll
            for (int i = 0; i < N; ++i) in[i] = (unsigned)(64 * i + lane - g * size) < (unsigned)size ? key[i] : 0;
            uint64_t v = take_best64<N>(in, &at);
            if (c.best == 2 && size > 1) {
                const double one = key_value64(v), two = key_value64(take_best64<N>(in, &at));
                if (two != -INFINITY) v = order_key64(one + two);
            }
            if (lane == g) rank = v;
        }
        int ahead = 0;   // groups before this lane's
        for (int g = 0; g < c.groups; ++g) {
            const uint64_t v = __shfl((unsigned long long)rank, g, 64);
            ahead += v > rank || (v == rank && g < lane);
        }
        open = __ballot(lane < c.groups && ahead < c.top_groups);
    }
    if (c.groups > 1) {
        // e / size for e < 1024 by a multiplication
        const uint32_t by_size = ((1u << 20) + size - 1) / size;
#pragma unroll
        for (int i = 0; i < N; ++i) key[i] = open >> (((64 * i + lane) * by_size) >> 20 & 63) & 1 ? key[i] : 0;
    }
    for (int j = 0; j < a.k; ++j) {
        int e;
        take_best64<N>(key, &e);
        chosen(j, e);
    }
}

// One token of the block (number tl of its 64) per row of lanes.  `far`: the
// largest finite |bias|.
template <int V, int S, bool SIGMOID>
__device__ __forceinline__ void select_by_scores(const RouteArgs& a, const ScoreArgs& c, const float* bias, float far,
                                                 unsigned long long* mask, int tl, int32_t (&mine)[S]) {
    // opaque: what depends on the lane alone would otherwise be hoisted out of
    // the loop over the block's tokens and held in registers
    int lane = threadIdx.x & 63;
    asm volatile("" : "+v"(lane));
    const int l = lane & 15;
    const int E = a.E, k = a.k;
    const int64_t t = (int64_t)blockIdx.x * kRouteTokens + tl;
    const bool live = t < a.T;
    const float* row = a.logits + t * E;
    uint32_t key[V];
    load_keys<V>(key, row, E, l, live);
    // the softmax's maximum and sum
    float most = 0.f, total = 1.f;
    if constexpr (!SIGMOID) {
        uint32_t m = 0;
#pragma unroll
        for (int i = 0; i < V; ++i) m = max(m, key[i]);
        most = key_value(row_max(m));   // NaN if there is one
        if (most == -INFINITY) most = 0.f;
        total = 0.f;
#pragma unroll
        for (int i = 0; i < V; ++i) total += key[i] ? __builtin_amdgcn_exp2f((key_value(key[i]) - most) * 1.44269504f) : 0.f;
        total = row_sum(total);
    }
    const float inverse = SIGMOID ? 1.f : 1.f / total;
    // An FP32 value's error, with half steps u = 2^-24 (the hardware's
    // exponential and reciprocal are within 2 u of themselves).  Sigmoid with
    // e = exp(-|x|): the exponent is rounded, u |x| e <= 0.37 u, e itself 2 u e
    // (both times at most e' = 1 / (1 + e)^2 <= 1 where e is small and 1/4 where
    // it is 1: 0.9 u together), 1 + e u, the reciprocal 2 u, e q u / 2: 4.5 u in
    // all.  Softmax: two roundings of the exponent, 2 u |x - most| p <= 0.74 u,
    // and at most (V + 16) u p from the exponential, the sum and its inverse.
    // The bias adds a rounding, u |v|.
    const float off = SIGMOID ? 4.5f * kUnit : (1.f + (V + 16) * inverse) * kUnit;
    bool close = false;
    auto near = [&](uint32_t hi, uint32_t lo, float within) {
        const float h = key_value(hi), d = h - key_value(lo);   // infinity or NaN unless both are finite
        return fabsf(h) < INFINITY && d <= within;
    };
    if (!c.by_logits) {   // values in the logits' place, four experts at a time
#pragma unroll
        for (int q = 0; q < V / 4; ++q) {
            const f32x4 b = *reinterpret_cast<const f32x4*>(&bias[64 * q + 4 * l]);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const uint32_t v = order_key(score_value32<SIGMOID>(key_value(key[4 * q + i]), b[i], most, inverse));
                key[4 * q + i] = key[4 * q + i] != 0 ? v : 0u;
            }
            if constexpr (V > 16) __builtin_amdgcn_sched_barrier(0);   // side by side they do not fit the registers
        }
    }
    unsigned long long open = 0;   // the groups that take part
    bool regroup = false;
    if (c.groups > 1) {
        const int size = E / c.groups;
        // A margin that holds for every group: values are sums of at most two v, each
        // below 1 + far.  Biases far from the scores (a finite mask, of experts that
        // nobody chooses) make it too wide; what lies within it is then compared by
        // each group's own error.  (16384 tokens, 4 of 8 groups of 32, one bias of
        // -1e9: 28 us; by the wide margin alone all tokens were chosen again, 86.)
        const float within = (4.f * off + 8.f * kUnit * (1.f + far)) * 1.01f;
        float kept = INFINITY, others = -INFINITY;   // the least of the kept, the most of the others, by their errors
        auto take_error = [&](uint32_t one, uint32_t two, bool in) {
            const float v = key_value(group_key(one, two, c.best));
            const float a = fabsf(key_value(one)), b = c.best == 2 && two != 0 ? fabsf(key_value(two)) : 0.f;
            // two values, each within off and a rounding, the rounding of their sum and of these
            const float m = fmaxf(a < INFINITY ? a : 0.f, b < INFINITY ? b : 0.f);
            const float error = (2.f * off + 6.f * kUnit * m) * 1.01f;
            if (one != 0 && in) kept = fminf(kept, v - error);
            if (one != 0 && !in) others = fmaxf(others, v + error);
        };
        uint32_t last = 0, left;
        if (size >= 4 && (size & (size - 1)) == 0) {
            // Groups of 4, 8, .. neighbours: a lane's four keys are of one group,
            // and so are those of size / 4 lanes, or of size / 64 runs.  A lane
            // keeps its runs' groups' values.  (16384 tokens, 4 of 8 groups of 32:
            // 4 us more than a bias alone; the way below took 20 more.)
            const int shift = __builtin_ctz(size);
            auto largest = [&](uint32_t (&one)[V / 4], uint32_t (&two)[V / 4]) {
#pragma unroll
                for (int q = 0; q < V / 4; ++q) {
                    one[q] = max(key[4 * q], key[4 * q + 1]);
                    two[q] = min(key[4 * q], key[4 * q + 1]);
                    merge_two(one[q], two[q], max(key[4 * q + 2], key[4 * q + 3]), min(key[4 * q + 2], key[4 * q + 3]));
                    if (size >= 8) merge_lanes<0xB1>(one[q], two[q]);     // lane l ^ 1
                    if (size >= 16) merge_lanes<0x4E>(one[q], two[q]);    // l ^ 2
                    if (size >= 32) merge_lanes<0x141>(one[q], two[q]);   // 7 - l of 8: the other quad
                    if (size >= 64) merge_lanes<0x140>(one[q], two[q]);   // 15 - l: the other eight
                }
#pragma unroll
                for (int d = 1; d < V / 4; d *= 2)
                    if (64 * d < size) {
#pragma unroll
                        for (int q = 0; q < V / 4; ++q)
                            if (!(q & d)) {
                                merge_two(one[q], two[q], one[q + d], two[q + d]);
                                one[q + d] = one[q];
                                two[q + d] = two[q];
                            }
                    }
            };
            uint32_t one[V / 4], two[V / 4];
            largest(one, two);
#pragma unroll
            for (int q = 0; q < V / 4; ++q) one[q] = group_key(one[q], two[q], c.best);
            auto best_left = [&]() {
                uint32_t m = one[0];
#pragma unroll
                for (int q = 1; q < V / 4; ++q) m = max(m, one[q]);
                return row_max(m);
            };
            for (int j = 0; j < c.top_groups; ++j) {
                last = best_left();
                uint32_t at = 64;
#pragma unroll
                for (int q = V / 4 - 1; q >= 0; --q) at = one[q] == last ? (uint32_t)((64 * q + 4 * l) >> shift) : at;
                at = row_min(at);
#pragma unroll
                for (int q = 0; q < V / 4; ++q) one[q] = at == (uint32_t)((64 * q + 4 * l) >> shift) ? 0u : one[q];
                open |= 1ull << (at & 63);
            }
            left = best_left();
            regroup = left != 0 && near(last, left, within);
            if (regroup && far > 1.f) {
                largest(one, two);
#pragma unroll
                for (int q = 0; q < V / 4; ++q) take_error(one[q], two[q], open >> (((64 * q + 4 * l) >> shift) & 63) & 1);
                regroup = row_max(order_key(others)) >= row_min(order_key(kept));
            }
#pragma unroll
            for (int q = 0; q < V / 4; ++q) {
                const bool in = open >> (((64 * q + 4 * l) >> shift) & 63) & 1;
#pragma unroll
                for (int i = 0; i < 4; ++i) key[4 * q + i] = in ? key[4 * q + i] : 0u;
            }
        } else {
            // the sixteen lanes take the groups in turn, their values made again
            uint32_t one[4], two[4], rank[4];
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const int g = 16 * q + l;
                one[q] = two[q] = 0;
                if (live && g < c.groups)
                    for (int e = g * size; e < (g + 1) * size; ++e) {
                        const uint32_t v = order_key(score_value32<SIGMOID>(row[e], bias[e], most, inverse));
                        merge_two(one[q], two[q], v, 0);
                    }
                rank[q] = group_key(one[q], two[q], c.best);
            }
            for (int j = 0; j < c.top_groups; ++j) {
                last = row_max(max(max(rank[0], rank[1]), max(rank[2], rank[3])));
                uint32_t at = 64;
#pragma unroll
                for (int q = 3; q >= 0; --q) at = rank[q] == last ? (uint32_t)(16 * q + l) : at;
                at = row_min(at);
#pragma unroll
                for (int q = 0; q < 4; ++q) rank[q] = at == (uint32_t)(16 * q + l) ? 0u : rank[q];
                open |= 1ull << (at & 63);
            }
            left = row_max(max(max(rank[0], rank[1]), max(rank[2], rank[3])));
            regroup = left != 0 && near(last, left, within);
            if (regroup && far > 1.f) {
#pragma unroll
                for (int q = 0; q < 4; ++q) take_error(one[q], two[q], open >> (16 * q + l) & 1);
                regroup = row_max(order_key(others)) >= row_min(order_key(kept));
            }
            // e / size for e < 1024 by a multiplication
            const uint32_t by_size = ((1u << 20) + size - 1) / size;
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const uint32_t e = 64 * (i >> 2) + 4 * l + (i & 3);
                key[i] = open >> ((e * by_size) >> 20 & 63) & 1 ? key[i] : 0u;
            }
        }
        // sums beyond 2^126 may have left FP32's range
        regroup |= left != 0 && far > 0x1p126f && !(fabsf(key_value(last)) <= 0x1p126f);
    }
    // a wave without tokens does not compete with the others
    const int64_t t0 = (int64_t)blockIdx.x * kRouteTokens + __builtin_amdgcn_readfirstlane(tl);   // the wave's first
    const int rounds = t0 < a.T ? k : 0;
    uint32_t kept[S];   // lane j % 16 keeps round j's value in its slot j / 16
#pragma unroll
    for (int s = 0; s < S; ++s) kept[s] = 0;
    for (int j = 0; j < rounds; ++j) {
        uint32_t best;
        const uint32_t e = take_best<V>(key, l, &best);
#pragma unroll
        for (int s = 0; s < S; ++s)
            if (j == 16 * s + l) {
                kept[s] = best;
                mine[s] = (int32_t)e;
            }
    }
    if (!c.by_logits) {
        // each of the chosen and the best of the rest against the one before
        const uint32_t rest = best_key<V>(key);
#pragma unroll
        for (int s = 0; s < S; ++s) {
            const int j = 16 * s + l;
            uint32_t before = row_rotate<1>(kept[s]);   // lane l - 1's
            if (l == 0) before = 0;
            if (s > 0) {
                const uint32_t wrap = row_rotate<1>(kept[s > 0 ? s - 1 : 0]);   // in lane 0 the last slot's lane 15
                if (l == 0) before = wrap;
            }
            const uint32_t it = j < k ? kept[s] : j == k ? rest : 0u;
            if (before != 0 && it != 0) close |= near(before, it, (2.f * off + 2.f * kUnit * fabsf(key_value(before))) * 1.01f);
            if (s == S - 1 && k == 16 * S && l == 15 && rest != 0)   // no lane is left for the rest
                close |= near(kept[s], rest, (2.f * off + 2.f * kUnit * fabsf(key_value(kept[s]))) * 1.01f);
        }
    }
    // the tokens of this wave that FP32 does not decide
    unsigned long long undecided = __ballot((close || regroup) && live);   // any lane of a row
    const unsigned long long groups_too = __ballot(regroup);
    while (undecided) {
        const int at = __ffsll((long long)undecided) - 1;   // a lane of the token's row
        undecided &= ~(0xFFFFull << (at & ~15));
        const unsigned long long its_open = (unsigned long long)(uint32_t)__builtin_amdgcn_readlane((int)(open >> 32), at) << 32 |
                                            (uint32_t)__builtin_amdgcn_readlane((int)open, at);
        choose64<V / 4, SIGMOID>(a, c, bias, t0 + (at >> 4), its_open, groups_too >> at & 1, [&](int j, int e) {
#pragma unroll
            for (int s = 0; s < S; ++s)
                if (lane >> 4 == at >> 4 && j == 16 * s + l) mine[s] = e;
        });
    }
    // Weights.  Renormalised sigmoids are taken relative to the largest
    // exp(min(x, 0)) among the chosen: the same ratio, also where every score is
    // below FP32's range.
    float x[S], p[S], m = -INFINITY, sum = 0.f;
    bool in[S];
#pragma unroll
    for (int s = 0; s < S; ++s) {
        const bool has = live && 16 * s + l < k;
        x[s] = has ? row[mine[s]] : -INFINITY;
        in[s] = has && x[s] != -INFINITY && bias[has ? mine[s] : 0] != -INFINITY;
        if (in[s]) m = fmaxf(m, SIGMOID ? fminf(x[s], 0.f) : x[s]);   // a NaN is passed over here and comes back below
    }
    if (a.renormalize) {
        m = key_value(row_max(order_key(m)));
        if (m == -INFINITY) m = 0.f;   // none but masked experts (or NaN)
    } else {
        m = SIGMOID ? 0.f : most;
    }
#pragma unroll
    for (int s = 0; s < S; ++s) {
        const float shared = expf(fminf(x[s], 0.f) - m) / (1.f + expf(-fabsf(x[s])));
        const float e = !SIGMOID ? expf(x[s] - m) : x[s] != x[s] ? x[s] : shared;
        p[s] = in[s] ? e : 0.f;
        sum += p[s];
    }
    sum = a.renormalize ? row_sum(sum) : SIGMOID ? 1.f : total;
    if (!SIGMOID && total != total) sum = total;
    if (live) {
#pragma unroll
        for (int s = 0; s < S; ++s) {
            const int j = 16 * s + l;
            if (j < k) {
                a.experts[t * k + j] = mine[s];
                a.weights[t * k + j] = in[s] ? c.scale * (p[s] / sum) : 0.f;
                atomicOr(&mask[mine[s]], 1ull << tl);
            }
        }
    }
}

// The block of 64 tokens, THREADS / 16 at a time, then their pairs' ranks and the
// counts as moe_select_kernel leaves them.  More than 512 experts take 256
// threads: with 1024 a lane has 128 registers, with 512 256, and 64 keys do not
// fit them beside the rest.
//
// 16384 tokens, k = 8 of 256 experts, normal logits: 13 us without groups and bias
// (moe_select_kernel 12), 17 with a bias, 20 with 4 of 8 groups; of the last two 3
// to 5 us are the 13 tokens or so of these that are chosen again in 64 bits, at
// the end of blocks that the others wait for.  The time depends on the values: equal
// ones count as undecided, and so do sigmoids that FP32 does not tell apart.  Logits
// rounded to BF16 take 24 us with a bias, 37 with a bias of zeros or none (a third of
// the tokens chosen again), logits of standard deviation 8 26 with a bias, and 82
// without; all logits equal 82.
template <int V, int S, int THREADS, bool SIGMOID>
__global__ __launch_bounds__(THREADS) void moe_select_scores_kernel(RouteArgs a, ScoreArgs c, MxQuantArgs quant) {
    if (blockIdx.x >= a.blocks) {   // the rows' quantisation, half a wave per row and 256 columns
        const int64_t n = quant.T * ceil_div(quant.K, 256);
        for (int64_t p = (int64_t)(blockIdx.x - a.blocks) * (THREADS / 32); p < n; p += (int64_t)(gridDim.x - a.blocks) * (THREADS / 32)) {
            const int64_t u = p + (threadIdx.x >> 5);
            quantize_mx_piece<true>(quant, u < n ? u % quant.T : quant.T, u < n ? u / quant.T : 0);
        }
        return;
    }
    __shared__ unsigned long long mask[16 * V];
    __shared__ int32_t start[16 * V], tmp[THREADS / 64];
    __shared__ __attribute__((aligned(16))) float bias[16 * V];
    __shared__ float widest[THREADS / 64];
    const int E = a.E, k = a.k, tid = threadIdx.x, l = tid & 15;
    float far = 0.f;
    for (int e = tid; e < 16 * V; e += THREADS) {
        const float b = c.bias && e < E ? c.bias[e] : 0.f;
        bias[e] = b;
        if (fabsf(b) < INFINITY) far = fmaxf(far, fabsf(b));
        mask[e] = 0;
    }
    for (int m = 1; m < 64; m <<= 1) far = fmaxf(far, __shfl_xor(far, m, 64));
    if ((tid & 63) == 0) widest[tid >> 6] = far;
    __syncthreads();
    for (int w = 0; w < THREADS / 64; ++w) far = fmaxf(far, widest[w]);
    constexpr bool kOnce = THREADS / 16 == kRouteTokens;
    int32_t mine[S];
    for (int tl = tid >> 4; tl < kRouteTokens; tl += THREADS / 16)
        select_by_scores<V, S, SIGMOID>(a, c, bias, far, mask, tl, mine);
    __syncthreads();
    const bool single = a.blocks == 1;
    if (single) {
        // threads hold neighbouring experts, so that their sums are in order
        constexpr int kPer = 16 * V > THREADS ? 16 * V / THREADS : 1;
        int32_t n[kPer], sum = 0;
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            n[i] = kPer * tid + i < E ? __popcll(mask[kPer * tid + i]) : 0;
            sum += n[i];
        }
        int32_t at = block_prefix(sum, tmp);
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            const int e = kPer * tid + i;
            if (e < E) start[e] = a.offsets[e] = at;
            at += n[i];
            if (e == E - 1) a.offsets[E] = at;
        }
        __syncthreads();
    } else if (a.blocks <= kRouteBytes) {
        const int stride = table_stride(E);
        for (int e = tid; e < stride; e += THREADS)
            static_cast<uint8_t*>(a.table)[(int64_t)blockIdx.x * stride + e] = e < E ? (uint8_t)__popcll(mask[e]) : 0;
    } else {
        for (int e = tid; e < E; e += THREADS)
            static_cast<int32_t*>(a.table)[(int64_t)blockIdx.x * E + e] = __popcll(mask[e]);
    }
    for (int tl = tid >> 4; tl < kRouteTokens; tl += THREADS / 16) {
        const int64_t t = (int64_t)blockIdx.x * kRouteTokens + tl;
        if (t >= a.T) break;
#pragma unroll
        for (int s = 0; s < S; ++s) {
            const int j = 16 * s + l;
            if (j >= k) break;
            const int32_t e = kOnce ? mine[s] : a.experts[t * k + j];   // this thread's own store
            int32_t r = __popcll(mask[e] & ((1ull << tl) - 1));
            if (single) {
                r += start[e];
                if (a.tokens) a.tokens[r] = (int32_t)t;
            }
            a.positions[t * k + j] = r;
        }
    }
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

// The same for weights from scores: with r = sum_j w_j dw_j / scale,
//   sigmoid:  w_j (1 - s_j) (dw_j - r), without the r where the weights are not
//             renormalised;  1 - s = sigmoid(-x)
//   softmax:  as above, with r for s
// Renormalised weights add up to the scale, so that dw_j - r stays what it is when
// the same is taken from every dw.  With the heaviest expert's taken, r is the sum
// over the others alone: exactly 0 where only one is chosen (dw - (scale dw) / scale
// is not: at scale 2.5 it is off by up to 2^-23 of dw for an eighth of the tokens),
// and where one has nearly all the weight the small difference keeps its digits.
// Weights that a caller has changed may have another sum: for those the formula as
// it stands.  The selection's sum is within 18 half steps of the scale (its sum of
// scores and this one 8 each, quotient and factor one each); 64 are let pass.
template <int V>
__global__ __launch_bounds__(256) void moe_route_scores_grad_kernel(RouteGradArgs a, int sigmoid, float scale) {
    const int l = threadIdx.x & 15;
    const int64_t t = (int64_t)blockIdx.x * 16 + (threadIdx.x >> 4);
    const int E = a.E, k = a.k;
    const bool live = t < a.T;
    // lane l has the chosen l, l + 16, ..
    float w[4], dw[4];
    int32_t expert[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const bool has = live && 16 * i + l < k;
        const int64_t at = t * k + 16 * i + l;
        w[i] = has ? a.weights[at] : 0.f;
        dw[i] = has ? a.dweights[at] : 0.f;
        expert[i] = has ? a.experts[at] : -1;
    }
    if (a.renormalize) {
        uint32_t heaviest = 0;   // weights are not negative: their bits are ordered as they are
        float its = 0.f, sum = 0.f;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            sum += w[i];
            its = __float_as_uint(w[i]) > heaviest ? dw[i] : its;
            heaviest = max(heaviest, __float_as_uint(w[i]));
        }
        const bool mine = row_min(heaviest == row_max(heaviest) ? l : 16u) == (uint32_t)l;   // the first lane that has it
        const float base = __uint_as_float(row_max(mine ? __float_as_uint(its) : 0u));
        if (fabsf(row_sum(sum) - scale) <= 64 * kUnit * scale) {
#pragma unroll
            for (int i = 0; i < 4; ++i) dw[i] -= base;
        }
    }
    float r = 0.f;
    if (!(sigmoid && !a.renormalize)) {
#pragma unroll
        for (int i = 0; i < 4; ++i) r += w[i] != 0.f ? w[i] * dw[i] : 0.f;
    }
    r = row_sum(r);
    float g[V];
    if (a.renormalize || sigmoid) {
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
        for (int i = 0; i < V; ++i) g[i] = g[i] == 0.f ? 0.f : -r * (g[i] / total);
    }
    r /= scale;
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
#pragma unroll
    for (int i = 0; i < 4; ++i)
        if (expert[i] >= 0 && expert[i] < E && w[i] != 0.f) {   // of weight 0: as if not chosen
            const float by = sigmoid ? score<true, float>(-a.logits[t * E + expert[i]], 0.f, 1.f) : 1.f;
            out[expert[i]] = w[i] * by * (dw[i] - r);
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

// the places of the pairs, where the selection took more than one block
static hipError_t finish_route(const RouteArgs& a, hipStream_t s) {
    const dim3 grid((unsigned)a.blocks), block(kRouteThreads);
    if (a.blocks > kRouteBytes) {
        timing_mark("moe_scan_kernel", s);
        hipLaunchKernelGGL(moe_scan_kernel, dim3((unsigned)ceil_div(a.E, 64)), block, 0, s, a);
    }
    if (a.blocks > 1) {
        timing_mark("moe_place_kernel", s);
        if (a.blocks > kRouteBytes) hipLaunchKernelGGL(moe_place_kernel<false>, grid, block, 0, s, a);
        else hipLaunchKernelGGL(moe_place_kernel<true>, grid, block, 0, s, a);
    }
    timing_end(s);
    return hipGetLastError();
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
    return finish_route(a, s);
}

hipError_t launch_moe_route_scores(const float* logits, int64_t T, int32_t E, int32_t k, const drgg_scoring& c,
                                   int32_t* experts, float* weights, int32_t* offsets, int32_t* positions,
                                   int32_t* tokens, void* table, hipStream_t s, const MxQuantArgs* quantize) {
    RouteArgs a{logits, experts, weights, offsets, positions, tokens, table, T, route_blocks(T), E, k, c.renormalize != 0};
    const ScoreArgs sc{c.bias, c.groups, c.top_groups, c.best, !c.bias && c.groups == 1, c.scale};
    const MxQuantArgs quant = quantize ? *quantize : MxQuantArgs{};
    timing_mark("moe_select_scores_kernel", s);
    for_experts(E, [&](auto v) {
        constexpr int V = decltype(v)::value;
        constexpr int kThreads = V <= 32 ? 1024 : 256;
        const dim3 grid((unsigned)(a.blocks + (quantize ? ceil_div(quantize->T * ceil_div(quantize->K, 256), kThreads / 32) : 0)));
        const dim3 block(kThreads);
        if (c.score == DRGG_SCORE_SIGMOID) {
            if (k <= 16) hipLaunchKernelGGL((moe_select_scores_kernel<V, 1, kThreads, true>), grid, block, 0, s, a, sc, quant);
            else hipLaunchKernelGGL((moe_select_scores_kernel<V, 4, kThreads, true>), grid, block, 0, s, a, sc, quant);
        } else {
            if (k <= 16) hipLaunchKernelGGL((moe_select_scores_kernel<V, 1, kThreads, false>), grid, block, 0, s, a, sc, quant);
            else hipLaunchKernelGGL((moe_select_scores_kernel<V, 4, kThreads, false>), grid, block, 0, s, a, sc, quant);
        }
    });
    return finish_route(a, s);
}

hipError_t launch_moe_route_scores_grad(const float* dweights, const float* logits, const int32_t* experts,
                                        const float* weights, int64_t T, int32_t E, int32_t k, const drgg_scoring& c,
                                        float* dlogits, hipStream_t s) {
    RouteGradArgs a{dweights, logits, experts, weights, dlogits, T, E, k, c.renormalize != 0};
    const dim3 grid((unsigned)ceil_div(T, 16)), block(256);
    timing_mark("moe_route_scores_grad_kernel", s);
    for_experts(E, [&](auto v) {
        hipLaunchKernelGGL(moe_route_scores_grad_kernel<decltype(v)::value>, grid, block, 0, s, a,
                           (int)(c.score == DRGG_SCORE_SIGMOID), c.scale);
    });
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
