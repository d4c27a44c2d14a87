// engine.hpp -- the tile engine of the gfx950 matrix-product kernels
// (kernels.hip: BF16; int8.hip: 8-bit integers; mxfp4.hip: microscaled 4-bit
// floating point): ragged schedules, operand staging, the MFMA main loop and the
// staged epilogue.  Included by kernel files only.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>
#include <utility>

#include "internal.hpp"
#include "plan.hpp"

namespace drgg {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef int32_t i32x4 __attribute__((ext_vector_type(4)));
typedef int32_t i32x16 __attribute__((ext_vector_type(16)));

// The element type of a product: fragment, accumulator and MFMA.  The engine
// moves 16-byte pieces and counts the reduction in 2-byte units: one BF16
// value, or a pair of 8-bit ones.  A fragment is 16 bytes of a tile row per
// lane either way (8 BF16 values, 16 8-bit ones), and the MFMA shapes agree:
// 32x32 outputs, the lower half of the lanes on the first 16 bytes of a
// sub-step's 32 and the upper half on the last.
struct Bf16 {
    typedef bf16x8 Frag;
    typedef f32x16 Acc;
    static __device__ __forceinline__ Acc mfma(Frag b, Frag a, Acc c) {
        return __builtin_amdgcn_mfma_f32_32x32x16_bf16(b, a, c, 0, 0, 0);
    }
};
struct Int8 {
    typedef i32x4 Frag;
    typedef i32x16 Acc;
    static __device__ __forceinline__ Acc mfma(Frag b, Frag a, Acc c) {
        return __builtin_amdgcn_mfma_i32_32x32x32_i8(b, a, c, 0, 0, 0);
    }
};

constexpr int kThreads = 256;       // fold / zero / router kernels
// Grouped-GEMM kernels run 4 waves (one per SIMD) or, for the 256x256
// forward and data-gradient tiles, 8 (two per SIMD, each on half the
// accumulators): a second wave per SIMD covers the stalls of the first.
constexpr int kGemmWaves = 4;
constexpr int kGemmThreads = 64 * kGemmWaves;
constexpr int kMaxGemmThreads = 512;

// ---------------------------------------------------------------------------
// small helpers

__device__ __forceinline__ uint16_t f32_to_bf16(float f) {
    // round to nearest, ties to even; NaN stays a (quiet) NaN
    uint32_t u = __float_as_uint(f);
    if ((u & 0x7fffffffu) > 0x7f800000u) return (uint16_t)((u >> 16) | 0x40u);
    u += 0x7fffu + ((u >> 16) & 1u);
    return (uint16_t)(u >> 16);
}

__device__ __forceinline__ float bf16_to_f32(uint16_t h) {
    return __uint_as_float((uint32_t)h << 16);
}

// ---------------------------------------------------------------------------
// ragged work decode

// LDS pointers keep their address space in the type, so that every access
// compiles to ds_* instructions (a generic pointer would become a flat access
// that also waits for outstanding global loads).
typedef __attribute__((address_space(3))) void lds_void_t;
typedef __attribute__((address_space(3))) char lds_t;

// SCAN: words of scratch; the schedule alone needs one per wave and one more.
// MOST: the experts it has room for.
template <int SCAN, int MOST = kMaxExperts>
struct SchedOf {
    int32_t offs[MOST + 1];    // clamped, non-decreasing offsets
    int32_t prefix[MOST + 1];  // exclusive prefix of work per expert
    int32_t scan[SCAN];
};
using Sched = SchedOf<kMaxGemmThreads>;

// Exclusive scan of v over the workgroup's threads (in thread order), with
// the sum (MAX = false) or the maximum (MAX = true, identity 0: the values
// are non-negative); *total gets the reduction over all threads.  Inclusive
// scans within each wave by lane shuffles, then one pass over the (at most
// 8) wave results in `tmp` (LDS, one word per wave plus one).  A serial pass
// over every thread's value, or a barrier per doubling step, costs
// microseconds at kernel start; this costs a few hundred cycles.  Must be
// called by all threads; ends with a barrier.
template <bool MAX = false, class Ptr>
__device__ int32_t block_exclusive_scan(int32_t v, Ptr tmp, int32_t* total) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, nw = blockDim.x >> 6;
    int32_t x = v;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const int32_t y = __shfl_up(x, d, 64);
        if (lane >= d) x = MAX ? max(x, y) : x + y;
    }
    const int32_t excl_in_wave = MAX ? __shfl_up(x, 1, 64) : x - v;
    if (lane == 63) tmp[wave] = x;
    __syncthreads();
    if (threadIdx.x == 0) {
        int32_t acc = 0;
        for (int w = 0; w < nw; ++w) {
            const int32_t t = tmp[w];
            tmp[w] = acc;
            acc = MAX ? max(acc, t) : acc + t;
        }
        tmp[nw] = acc;
    }
    __syncthreads();
    const int32_t before = tmp[wave];
    const int32_t r = MAX ? max(before, lane > 0 ? excl_in_wave : 0) : before + excl_in_wave;
    *total = tmp[nw];
    __syncthreads();
    return r;
}

// Lanes of one wave exchanging data through LDS: the fences order each
// lane's accesses before and after this point for the compiler (no
// instruction is emitted; the wave's DS instructions execute in order).
__device__ __forceinline__ void wave_lds_sync() {
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

// Inclusive scans (maximum, sum) over the 64 lanes of a wave.  With fewer
// than kWaveExperts experts the prologue steps below run on wave 0 alone:
// shuffles instead of the workgroup scans, one barrier instead of three or
// more per step (each costs a few hundred cycles at kernel start).
constexpr int kWaveExperts = 64;
__device__ __forceinline__ int32_t wave_incl_max(int32_t x) {
    const int lane = threadIdx.x & 63;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const int32_t y = __shfl_up(x, d, 64);
        if (lane >= d) x = max(x, y);
    }
    return x;
}
__device__ __forceinline__ int32_t wave_incl_sum(int32_t x) {
    const int lane = threadIdx.x & 63;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const int32_t y = __shfl_up(x, d, 64);
        if (lane >= d) x += y;
    }
    return x;
}

// Fills s.offs[0..E] with the offsets clamped into [0, M] (and made
// non-decreasing), and s.prefix[0..E] with the exclusive prefix of
// work(e, T_e).  With no offsets array (a batched call) the groups are
// uniform: offs[e] = e * T.  With fewer than kWaveExperts experts wave 0
// does it all (offsets on lanes 0..E, shuffle scans).  Must be called by all
// threads; ends with a barrier.
template <int SCAN, int MOST, class WorkFn>
__device__ void build_schedule(SchedOf<SCAN, MOST>& s, const int32_t* __restrict__ offs, int E, int64_t M, int64_t T,
                               WorkFn work) {
    const int tid = threadIdx.x, nthr = blockDim.x;
    if (E < kWaveExperts) {
        // lane e of wave 0 holds offset e (e <= E)
        if (tid < 64) {
            int64_t v = 0;
            if (tid <= E) v = offs ? (int64_t)offs[tid] : tid * T;
            v = v < 0 ? 0 : (v > M ? M : v);
            const int32_t o = wave_incl_max(tid <= E ? (int32_t)v : 0);
            const int32_t o1 = __shfl_down(o, 1, 64);
            const int32_t wk = tid < E ? work(tid, o1 - o) : 0;
            const int32_t incl = wave_incl_sum(wk);
            if (tid <= E) {
                s.offs[tid] = o;
                s.prefix[tid] = incl - wk;
            }
        }
        __syncthreads();
        return;
    }
    int32_t* tmp = s.scan;   // free until the prefix is written
    for (int e = tid; e <= E; e += nthr) {
        int64_t v = offs ? (int64_t)offs[e] : e * T;
        v = v < 0 ? 0 : (v > M ? M : v);
        s.offs[e] = (int32_t)v;
    }
    __syncthreads();
    // make non-decreasing (a running max); E <= 1024, one run per thread
    const int per = (E + nthr) / nthr;   // covers indices 0..E
    const int lo = min(tid * per, E + 1);
    const int hi = min(lo + per, E + 1);
    int32_t run = 0;
    for (int i = lo; i < hi; ++i) run = max(run, s.offs[i]);
    int32_t total;
    int32_t carry = block_exclusive_scan<true>(run, tmp, &total);
    for (int i = lo; i < hi; ++i) {
        carry = max(carry, s.offs[i]);
        s.offs[i] = carry;
    }
    __syncthreads();
    // work counts and their exclusive prefix
    int32_t local = 0;
    for (int e = lo; e < hi && e < E; ++e) local += work(e, s.offs[e + 1] - s.offs[e]);
    int32_t acc = block_exclusive_scan(local, tmp, &total);
    for (int e = lo; e < hi; ++e) {
        s.prefix[e] = acc;
        if (e < E) acc += work(e, s.offs[e + 1] - s.offs[e]);
    }
    __syncthreads();
}

// Weight-gradient work order: longest token chunks first.  Items of one
// expert all cost about the same (a tile over one chunk of its tokens), so
// the experts are put in decreasing order of chunk length (ties: expert
// index) and, for the persistent walk below, the rounds alternate direction
// ("snake"): the longest items of round r and the shortest of round r+1 land
// on the same workgroup.  On the Zipf-routed E=32 workload that balances the
// workgroups to 96 % of the mean load, against 81 % in expert order.
//
// rank_experts writes that order as 16-bit expert ids over s.scan (which
// build_schedule no longer needs): expert_at(s, p) is the expert at position
// p.  position_prefix then rebuilds s.prefix[0..npos] as the exclusive
// prefix of work(p) over positions p < npos (a plan may give an expert more
// than one position: the tail-only plan of the deterministic weight
// gradient has its whole tiles at p and its chunks at E + p).  `scr` is
// 4 KB of LDS that is free until the first stage load; `clen(e)` is expert
// e's chunk length.  Both must be called by all threads and end with a
// barrier; rank_experts after build_schedule.
static_assert(kMaxExperts <= 2 * kMaxGemmThreads && kMaxExperts <= 32767, "16-bit expert order in Sched::scan");
__device__ __forceinline__ int expert_at(const Sched& s, int p) {
    return reinterpret_cast<const int16_t*>(s.scan)[p];
}
template <class LenFn>
__device__ void rank_experts(Sched& s, lds_t* scr, int E, LenFn clen) {
    static_assert(kMaxExperts <= 4 * kGemmThreads, "at most four experts per thread");
    const int tid = threadIdx.x, nthr = blockDim.x;
    auto* key = reinterpret_cast<__attribute__((address_space(3))) int32_t*>(scr);
    if (E < kWaveExperts) {   // wave 0: lane e ranks expert e (keys exchanged through LDS)
        if (tid < 64) {
            const int32_t k0 = tid < E ? clen(tid) : 0;
            if (tid < E) key[tid] = k0;
            wave_lds_sync();
            int32_t r = 0;
            for (int f = 0; f < E; ++f) {
                const int32_t kf = key[f];
                r += kf > k0 || (kf == k0 && f < tid);
            }
            if (tid < E) reinterpret_cast<int16_t*>(s.scan)[r] = (int16_t)tid;
        }
        __syncthreads();
        return;
    }
    for (int e = tid; e < E; e += nthr) key[e] = clen(e);
    __syncthreads();
    // rank of expert e: experts with a longer chunk, or as long and a lower
    // index, go first; each thread ranks its (up to four) experts in one
    // pass over the keys
    int32_t k4[4], r4[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
        const int e = tid + u * nthr;
        k4[u] = e < E ? key[e] : 0;
        r4[u] = 0;
    }
    if (E <= nthr) {
        // one expert per thread; waves without an expert skip the pass
        if ((tid & ~63) < E)
            for (int f = 0; f < E; ++f) {
                const int32_t kf = key[f];
                r4[0] += kf > k4[0] || (kf == k4[0] && f < tid);
            }
    } else {
        for (int f = 0; f < E; ++f) {
            const int32_t kf = key[f];
#pragma unroll
            for (int u = 0; u < 4; ++u) r4[u] += kf > k4[u] || (kf == k4[u] && f < tid + u * nthr);
        }
    }
    __syncthreads();   // the keys are read; s.scan may be overwritten
    int16_t* perm = reinterpret_cast<int16_t*>(s.scan);
#pragma unroll
    for (int u = 0; u < 4; ++u)
        if (tid + u * nthr < E) perm[r4[u]] = (int16_t)(tid + u * nthr);
    __syncthreads();
}
template <class WorkFn>
__device__ void position_prefix(Sched& s, lds_t* scr, int npos, WorkFn work) {
    const int tid = threadIdx.x, nthr = blockDim.x;
    if (npos <= 2 * kWaveExperts) {   // wave 0: lane l holds positions 2l and 2l+1
        if (tid < 64) {
            const int q0 = 2 * tid, q1 = q0 + 1;
            const int32_t w0 = q0 < npos ? work(q0) : 0, w1 = q1 < npos ? work(q1) : 0;
            const int32_t incl = wave_incl_sum(w0 + w1);
            if (q0 < npos) s.prefix[q0] = incl - w0 - w1;
            if (q1 < npos) s.prefix[q1] = incl - w1;
            if (tid == 63) s.prefix[npos] = incl;
        }
        __syncthreads();
        return;
    }
    // per-thread runs of positions, then a scan of the run sums
    const int per = (npos + nthr - 1) / nthr;
    const int lo = min(tid * per, npos), hi = min(lo + per, npos);
    int32_t run = 0;
    for (int q = lo; q < hi; ++q) run += work(q);
    int32_t total;
    int32_t acc = block_exclusive_scan(run, reinterpret_cast<__attribute__((address_space(3))) int32_t*>(scr), &total);
    for (int q = lo; q < hi; ++q) {
        s.prefix[q] = acc;
        acc += work(q);
    }
    if (tid == 0) s.prefix[npos] = total;
    __syncthreads();
}

// Work item of round r for the workgroup at (XCD-remapped) index wb of G:
// rounds alternate direction.
__device__ __forceinline__ int64_t snake_item(int64_t r, int64_t wb, int64_t G) {
    return r * G + ((r & 1) ? G - 1 - wb : wb);
}

// Values read from LDS arrive in vector registers even when every lane reads
// the same address; the tile decode is wave-uniform, so it is moved to scalar
// registers (keeps the per-tile state out of the VGPR budget).
__device__ __forceinline__ int32_t uni(int32_t v) { return __builtin_amdgcn_readfirstlane(v); }

// Largest e < n with prefix[e] <= w (so that prefix[e] <= w < prefix[e+1]
// when w < prefix[n]); n is the number of experts, or of positions of a
// plan's walk.
template <int SCAN, int MOST>
__device__ __forceinline__ int find_expert(const SchedOf<SCAN, MOST>& s, int n, int32_t w) {
    int lo = 0, hi = n;   // answer in [0, n)
    while (lo < hi) {
        int mid = (lo + hi + 1) >> 1;
        if (s.prefix[mid] <= w) lo = mid; else hi = mid - 1;
    }
    return lo;
}

// The deterministic weight gradient's chunk rule (device side of
// wgrad_chunking in plan.hpp), in 32-bit unsigned arithmetic: T < 2^31, and a
// chunk_max of T or more gives one chunk, so it is clamped to T first.  (A
// 64-bit division is a long integer sequence on this GPU; the prologues
// evaluate these per expert and the walk per tile.)
__device__ __forceinline__ int32_t chunk_len_dev(int32_t T, int64_t chunk_max) {
    if (T <= 0) return 0;
    const uint32_t t = (uint32_t)T;
    const uint32_t cm = chunk_max < (int64_t)t ? (uint32_t)chunk_max : t;
    const uint32_t s = (t + cm - 1) / cm;
    const uint32_t l = (t + s - 1) / s;
    return (int32_t)(((l + kTileK - 1) / kTileK) * kTileK);
}
__device__ __forceinline__ int32_t chunks_dev(int32_t T, int64_t chunk_max) {
    const int32_t l = chunk_len_dev(T, chunk_max);
    return l ? (int32_t)(((uint32_t)T + (uint32_t)l - 1) / (uint32_t)l) : 0;
}

// Maximum / minimum of a 64-bit value over the lanes of a wave (butterfly
// shuffles).  An LDS atomic issued by every lane is expanded by the compiler
// into a loop over the active lanes, 64 dependent steps per wave; reducing
// first leaves one atomic per wave.
__device__ __forceinline__ uint64_t wave_max_u64(uint64_t v) {
#pragma unroll
    for (int m = 1; m < 64; m <<= 1) {
        const uint64_t o = __shfl_xor((unsigned long long)v, m, 64);
        v = o > v ? o : v;
    }
    return v;
}
__device__ __forceinline__ uint64_t wave_min_u64(uint64_t v) {
#pragma unroll
    for (int m = 1; m < 64; m <<= 1) {
        const uint64_t o = __shfl_xor((unsigned long long)v, m, 64);
        v = o < v ? o : v;
    }
    return v;
}

// Estimated time of a planned walk on `workers` workgroups: the items
// 0 .. prefix[npos]-1 handed out in snake rounds, as the persistent kernels
// hand them out, each costing len(its position) plus kItemOverheadTokens
// tokens; returns the largest per-workgroup load.  The deterministic weight
// gradient chooses between its two plans with it on kRuleCUs reference
// workgroups (a function of the plan only, never of the device); the split
// program on its live grid.  `red` is an LDS word; `tab` is LDS scratch for
// npos words (the lengths, read once per position).  A workgroup's items
// have increasing indices, so their positions are found by advancing one
// pointer.  Must be called by all threads; ends with a barrier.
template <class LenFn>
__device__ uint64_t walk_makespan(const Sched& s, int npos, LenFn len, unsigned long long* red,
                                  __attribute__((address_space(3))) uint32_t* tab, int64_t workers = kRuleCUs) {
    if (threadIdx.x == 0) *red = 0;
    for (int q = threadIdx.x; q < npos; q += blockDim.x) tab[q] = (uint32_t)len(q);
    __syncthreads();
    const int64_t total = s.prefix[npos];
    uint64_t worst = 0;
    for (int64_t b = threadIdx.x; b < workers; b += blockDim.x) {
        uint64_t load = 0;
        int q = 0;
        for (int64_t r = 0;; ++r) {
            const int64_t i = snake_item(r, b, workers);
            if (i >= total) break;   // later rounds hold only larger indices
            while (s.prefix[q + 1] <= i) ++q;   // stops below npos: i < prefix[npos]
            load += (uint64_t)tab[q] + (uint64_t)kItemOverheadTokens;
        }
        worst = load > worst ? load : worst;
    }
    worst = wave_max_u64(worst);
    if ((threadIdx.x & 63) == 0) atomicMax(red, (unsigned long long)worst);
    __syncthreads();
    const uint64_t m = *red;
    __syncthreads();
    return m;
}

// Workgroup b of G -> logical work index.  Workgroups are dispatched to the
// 8 XCDs round-robin (b % 8); this gives each XCD a contiguous run of work
// items so that tiles sharing operand panels share that XCD's L2.
__device__ __forceinline__ int64_t xcd_remap(int64_t b, int64_t G) {
    const int64_t x = b & 7, i = b >> 3;
    const int64_t q = G >> 3, r = G & 7;
    return x * q + (x < r ? x : r) + i;
}

// ---------------------------------------------------------------------------
// operand tiles

// A view of one operand of a tile: element (i, kk) with i in [0, nvalid) the
// output index inside the tile and kk the reduction index from the start of
// the reduction range [0, klen).
//   K-major:  base[i * ld + kk]   (reduction index contiguous)
//   MN-major: base[kk * ld + i]   (output index contiguous; nvalid % 8 == 0)
// Everything outside reads as zero.
// A paired operand (K-major; gate and up rows of one weight matrix) is two
// runs of nvalid rows, the second `pair` bytes after the first, and its tile
// rows alternate between them in blocks of 32: tile rows 64p .. 64p+31 are
// rows 32p .. 32p+31 of the first run, 64p+32 .. 64p+63 those of the second.
struct Operand {
    const uint16_t* base;
    int64_t ld;
    int32_t nvalid;
    int32_t klen;
    int64_t pair = 0;
    // A gathered operand (K-major): tile row i is row index[i] of the `of` rows
    // at base; a row whose index is outside reads as zero.
    const int32_t* index = nullptr;
    int64_t of = 0;
};

typedef short v4i16 __attribute__((ext_vector_type(4)));
typedef short v8i16 __attribute__((ext_vector_type(8)));

// Buffer descriptor over [base, base + 2 GB): raw (stride 0) addressing with
// range checking.  A lane whose offset is kOOB lies past the range, and its
// load writes zeros to LDS; this is how every mask below is applied.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t make_rsrc(const void* base) {
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(base), (short)0, 0x7FFFFFF0, 0x00020000);
}
constexpr uint32_t kOOB = 0xFFFFFFF0u;
// Cache-policy operand of a buffer store: the non-temporal (nt) hint, for
// output that this kernel never reads back, so that it is evicted before the
// operand panels that the workgroups of an XCD share through L2.
constexpr int kCpolNT = 2;

// ---------------------------------------------------------------------------
// main-loop pipeline
//
// The reduction runs in stages of kStageK = 32 values.  Each operand has
// kStages = 4 LDS buffers; stage s lives in buffer s % 4.  A step computes
// one stage in two MFMA sub-steps of 16 and is cut in half by the one
// workgroup barrier of the step:
//
//   sub-step 0   MFMAs of sub-step 0 (fragments already in registers),
//                LDS reads of the sub-step 1 fragments
//   barrier      after this wave's loads of stage s+1 have landed and its
//                LDS reads of stage s have returned
//   sub-step 1   MFMAs of sub-step 1, LDS reads of the next stage's sub-step
//                0 fragments, and the global loads of stage s+4 into the
//                buffer stage s has just freed
//
// so a load has three steps between its issue and its first use, and the
// MFMA pipe is fed from registers while the barrier and the next stage's
// first reads resolve.  Global loads go straight from HBM to LDS (16-byte
// buffer loads with an LDS destination), and the MFMAs, LDS reads and
// global loads of a sub-step are interleaved one by one.
//
// The stage stream runs through consecutive tiles of a workgroup without a
// break: the loads of the last three steps of a tile fetch the first stages
// of the next tile.  Every tile runs a multiple of four steps (padding steps
// compute nothing) so that each tile starts in buffer 0 and every buffer
// index is a compile-time constant; the eight buffers are distinct
// __shared__ arrays, so the compiler sees that a read of one buffer does not
// alias the loads in flight into another and never waits for those.

constexpr int kSubSteps = kStageK / kMfmaK;   // 2
static_assert(kSubSteps == 2, "the step schedule assumes two MFMA sub-steps per stage");

// s_waitcnt with vmcnt(N) and lgkmcnt(0) (expcnt left free).  GFX9 encoding:
// vmcnt in bits [3:0] and [15:14], expcnt [6:4], lgkmcnt [11:8].
template <int N>
__device__ __forceinline__ void wait_vm_lgkm() {
    static_assert(N >= 0 && N < 64, "vmcnt has 6 bits");
    __builtin_amdgcn_s_waitcnt((N & 15) | ((N >> 4) << 14) | (7 << 4));
}

// Workgroup barrier without a memory fence: the waits above are the only
// synchronisation the pipeline needs, and a fence would drain every load in
// flight.  The "memory" clobber keeps the compiler from moving memory
// accesses across it.
__device__ __forceinline__ void barrier_nofence() {
    __builtin_amdgcn_sched_barrier(0);
    asm volatile("s_barrier" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
}

// Scheduling groups (masks of __builtin_amdgcn_sched_group_barrier).
constexpr int kSchedMfma = 0x008, kSchedVmemRead = 0x020, kSchedDsRead = 0x100;

// Interleave NM MFMAs with NR LDS reads and NL global loads of the same
// region: the reads spread over the first half of the MFMAs (they feed the
// next sub-step), the loads over all of them.  Used when both operands are
// K-major; with transposed (MN-major) reads the compiler's own order is
// faster, as measured.
template <int NM, int NR, int NL, int T>
__device__ __forceinline__ void sched_slot() {
    __builtin_amdgcn_sched_group_barrier(kSchedMfma, 1, 0);
    constexpr int H = NM / 2;   // the reads go out during the first half
    constexpr int r = T < H ? NR * (T + 1) / H - NR * T / H : 0;
    constexpr int l = NL * (T + 1) / NM - NL * T / NM;
    if constexpr (r > 0) __builtin_amdgcn_sched_group_barrier(kSchedDsRead, r, 0);
    if constexpr (l > 0) __builtin_amdgcn_sched_group_barrier(kSchedVmemRead, l, 0);
}
template <int NM, int NR, int NL, int... T>
__device__ __forceinline__ void sched_interleave_impl(std::integer_sequence<int, T...>) {
    (sched_slot<NM, NR, NL, T>(), ...);
}
template <int NM, int NR, int NL>
__device__ __forceinline__ void sched_interleave() {
    sched_interleave_impl<NM, NR, NL>(std::make_integer_sequence<int, NM>{});
}

// LDS layouts:
//   K-major operands (reduction index contiguous in memory) are staged in
//   pairs of stages: a pair buffer holds ROWS rows of 64 reduction values
//   (128 B = 8 chunks of 16 B), stage 2p in the first four chunks of each
//   row and stage 2p+1 in the last four.  Loading a pair moves whole 128-byte
//   lines (a 32-value stage alone would be half a line per row, twice the
//   memory requests and address translations per byte).  Chunk c of row r
//   sits at c ^ swzK(r), which puts the 16 rows an MFMA operand read covers
//   per pass (one chunk each) on 16 distinct 16-byte bank groups, and any 8
//   consecutive rows on 8.
//   MN-major operands: one buffer per stage, 32 rows (reduction index) of
//   ROWS output indices (ROWS*2 B = CPR chunks), already whole lines in
//   memory; chunk c of row r sits at c ^ swzMN(r).  A transposed read has
//   each group of 32 lanes read 4 rows at the same 4 chunks (c0 .. c0+3, c0
//   a multiple of 4), each group of 16 lanes 2 of those chunks.  The XOR
//   values 0, 10, 12, 6 for r % 4 = 0..3 send the 4 rows to 4 different
//   64-byte bank groups of a 256-byte window (bits 2-3 of the chunk index
//   all differ) and, for the 16-lane halves, to 4 different 32-byte groups of
//   a 128-byte window (bits 1-2 all differ): no bank conflicts with either
//   32 or 64 banks.
__device__ __forceinline__ int swzK(int row) { return (row & 7) ^ ((row >> 3) & 1); }
template <int CPR>
__device__ __forceinline__ int swzMN(int row) {
    return ((0x6CA0 >> (4 * (row & 3))) & 15) & (CPR - 1);
}

// Loads stages of an operand from HBM into LDS with 16-byte buffer loads (no
// registers in between): a K-major operand two stages (one pair buffer) at a
// time, an MN-major operand one stage at a time.  Either way one load is
// ROWS*64*SPAN bytes = ROWS*SPAN/16 wave instructions of 1 KB, of which each
// of the 4 waves issues a quarter.  Lane l of instruction g writes LDS bytes
// [g*1024 + 16*l, +16); the swizzle is applied by choosing which global
// chunk the lane fetches.
template <int ROWS, bool KMAJ, int WAVES, bool PAIRED = false, bool GATHERED = false>
struct StageLoader {
    static constexpr int kSpan = KMAJ ? 2 : 1;   // stages per load
    static constexpr int kPerWave = ROWS * kStageK * 2 * kSpan / 1024 / WAVES;
    static_assert(kPerWave >= 1, "every wave issues at least one load per stage");
    static constexpr int kRowBytes = KMAJ ? 2 * kStageK * 2 : ROWS * 2;
    static constexpr int kCPR = kRowBytes / 16;
    static_assert(ROWS % 64 == 0, "tile rows must be a multiple of 64");
    uint32_t off[kPerWave];   // byte offset of this lane's 16 bytes from the load base (kOOB if masked)
    int32_t kp[kPerWave];     // reduction position of those 16 bytes from the first stage loaded
    int64_t step_bytes;       // byte distance between consecutive stages
    const char* base;
    int64_t pair;             // paired operands: bytes to the second run
    int32_t klen;

    __device__ __forceinline__ void init(const Operand& op) {
        // opaque lane index: keeps the lane-dependent offset arithmetic here
        // instead of hoisted (and held in registers) across the tile loop
        int lane = threadIdx.x & 63;
        asm volatile("" : "+v"(lane));
        const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
        base = reinterpret_cast<const char*>(op.base);
        if constexpr (PAIRED) pair = op.pair;
        klen = op.klen;
        step_bytes = KMAJ ? kStageK * 2 : (int64_t)kStageK * op.ld * 2;
#pragma unroll
        for (int i = 0; i < kPerWave; ++i) {
            const int b = (wave * kPerWave + i) * 1024 + lane * 16;
            const int row = b / kRowBytes, phys = (b % kRowBytes) / 16;
            if constexpr (KMAJ) {
                const int logical = phys ^ swzK(row);
                int from = PAIRED ? (row & 31) + 32 * (row >> 6) : row;
                bool ok = from < op.nvalid;
                if constexpr (GATHERED) {
                    static_assert(KMAJ, "rows are gathered whole");
                    from = ok ? op.index[from] : 0;
                    ok = ok && (uint32_t)from < (uint32_t)op.of;   // of * ld * 2 < 2^31, checked by the caller
                }
                off[i] = ok ? (uint32_t)(from * op.ld * 2 + logical * 16) : kOOB;
                kp[i] = logical * 8;
            } else {
                const int col = (phys ^ swzMN<kCPR>(row)) * 8;
                off[i] = col < op.nvalid ? (uint32_t)(row * op.ld * 2 + col * 2) : kOOB;
                kp[i] = row;
            }
        }
    }

    // Issue the load of stage L (stages L, L+1 for a K-major operand) into
    // `buf`; reduction positions at or past klen read as zero, and so does
    // everything when !valid (or when L lies past the last stage): such a
    // load accesses no memory.
    __device__ __forceinline__ void issue(lds_t* buf, int L, bool valid) const {
        issue_part<0, kPerWave>(buf, L, valid);
    }
    // instructions J0 .. J1-1 of that load (a load may be spread over steps)
    template <int J0, int J1>
    __device__ __forceinline__ void issue_part(lds_t* buf, int L, bool valid) const {
        const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
        const __amdgpu_buffer_rsrc_t r = make_rsrc(base + L * step_bytes);
        const int rem = valid ? klen - L * kStageK : 0;
#pragma unroll
        for (int i = J0; i < J1; ++i) {
            const uint32_t o = kp[i] < rem ? off[i] : kOOB;
            // a wave instruction covers 8 rows of 128 bytes, so rows of one
            // block of 32 and of one run of a paired operand
            static_assert(!PAIRED || (KMAJ && kRowBytes == 128), "8 rows per wave instruction");
            const bool second = PAIRED && (((wave * kPerWave + i) >> 2) & 1);
            __builtin_amdgcn_raw_ptr_buffer_load_lds(
                second ? make_rsrc(base + L * step_bytes + pair) : r, (lds_void_t*)(buf + (wave * kPerWave + i) * 1024), 16, o, 0, 0, 0);
        }
    }
};

// MFMA operand fragment: lane l gets the 8 reduction values 16*s + 8*(l/32)
// .. +7 of tile row rb + (l & 31) from the stage in `buf` (for a K-major pair
// buffer, the stage in half h).
template <int ROWS, bool KMAJ>
__device__ __forceinline__ bf16x8 read_frag(const lds_t* buf, int h, int rb, int s, int l) {
    if constexpr (KMAJ) {
        const int row = rb + (l & 31), c = 4 * h + 2 * s + (l >> 5);
        return *reinterpret_cast<const __attribute__((address_space(3))) bf16x8*>(
            buf + row * (4 * kStageK) + ((c ^ swzK(row)) << 4));
    } else {
        // ds_read_b64_tr_b16: in a group of 16 lanes, lane 4j+q addresses
        // 4 values of row kbase+j at column col0+4q; lane i receives column
        // col0+i of rows kbase..kbase+3.
        constexpr int CPR = ROWS * 2 / 16;
        const int g = l >> 4, j = (l >> 2) & 3, q = l & 3;
        const int col = rb + 16 * (g & 1) + 4 * q;
        const int chunk = col >> 3, within = (col & 7) * 2;
        const int r0 = 16 * s + 8 * (g >> 1) + j, r1 = r0 + 4;
        typedef __attribute__((address_space(3))) v4i16 lds_v4i16;
        v4i16 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
            (lds_v4i16*)(buf + r0 * ROWS * 2 + ((chunk ^ swzMN<CPR>(r0)) << 4) + within));
        v4i16 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
            (lds_v4i16*)(buf + r1 * ROWS * 2 + ((chunk ^ swzMN<CPR>(r1)) << 4) + within));
        v8i16 v = __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
        return __builtin_bit_cast(bf16x8, v);
    }
}

// One tile of work for the persistent driver: the two operand views and the
// kernel's own output coordinates.
struct TileInfo {
    Operand A, B;
    int64_t o0, o1;      // output row / column base (kernel specific)
    int32_t rows, cols;  // valid output rows / columns of the tile
    int32_t e, aux, aux2;  // expert and kernel-specific tags
};

// The LDS buffers of a kernel, indexed by stage % 4: for a K-major operand
// entries 2p and 2p+1 name the same pair buffer p, for an MN-major operand
// each entry is its own buffer.  Every buffer is a distinct __shared__ array
// (see above).
struct Stages {
    lds_t* a[kStages];
    lds_t* b[kStages];
};

#define DRGG_STAGE_BUFS(ROWS, KMAJ, name)                                                        \
    __shared__ __attribute__((aligned(256))) char name##0[(KMAJ ? 2 : 1) * (ROWS) * kStageK * 2]; \
    __shared__ __attribute__((aligned(256))) char name##1[(KMAJ ? 2 : 1) * (ROWS) * kStageK * 2]; \
    __shared__ __attribute__((aligned(256))) char name##2[(KMAJ ? 0 : 1) * (ROWS) * kStageK * 2 + 16]; \
    __shared__ __attribute__((aligned(256))) char name##3[(KMAJ ? 0 : 1) * (ROWS) * kStageK * 2 + 16]

#define DRGG_STAGE_PTRS(KMAJ, name)                                                              \
    KMAJ ? (lds_t*)name##0 : (lds_t*)name##0, KMAJ ? (lds_t*)name##0 : (lds_t*)name##1,          \
    KMAJ ? (lds_t*)name##1 : (lds_t*)name##2, KMAJ ? (lds_t*)name##1 : (lds_t*)name##3

#define DRGG_STAGES(BM, BN, AK, BK, name)                                                        \
    DRGG_STAGE_BUFS(BM, AK, name##_a);                                                           \
    DRGG_STAGE_BUFS(BN, BK, name##_b);                                                           \
    const Stages name{{DRGG_STAGE_PTRS(AK, name##_a)}, {DRGG_STAGE_PTRS(BK, name##_b)}}

// The accumulators and operand fragments of one BMxBN tile on 4 waves (one
// per SIMD, a 2x2 wave grid) or 8 waves (two per SIMD, a 4x2 grid for
// 256-row tiles): each wave owns a block of 32x32 MFMA tiles whose FP32
// accumulators stay in registers.  The MFMA takes the B-side fragment as its first operand,
// so that the accumulator of lane l holds tile row l%32 and, in registers
// 4q..4q+3, four consecutive tile columns 8q + 4*(l/32) .. +3: a lane's
// outputs leave as 8- or 16-byte stores.
template <int BM, int BN, bool AK, bool BK, int WAVES = kGemmWaves, class El = Bf16>
struct TileMma {
    // wave grid: kWGM waves along the tile rows, kWGN along its columns
    static constexpr int kWGM = (WAVES == 8 && BM >= 256) ? 4 : 2;
    static constexpr int kWGN = WAVES / kWGM;
    static constexpr int WM = BM / kWGM, WN = BN / kWGN;
    __device__ static __forceinline__ int wave_row(int wave) { return (wave / kWGN) * WM; }
    __device__ static __forceinline__ int wave_col(int wave) { return (wave % kWGN) * WN; }
    static constexpr int kBI = WM / 32, kBJ = WN / 32;
    static_assert(kBI >= 1 && kBJ >= 1, "tile too small for the 2x2 wave grid");
    // LDS reads per sub-step: one per 32-row block (K-major), two (MN-major)
    static constexpr int kReads = kBI * (AK ? 1 : 2) + kBJ * (BK ? 1 : 2);
    static constexpr int kMfmas = kBI * kBJ;
    typename El::Acc acc[kBI][kBJ];
    typename El::Frag fa[2][kBI], fb[2][kBJ];   // fragments of sub-step 0 and 1

    __device__ __forceinline__ void zero() {
#pragma unroll
        for (int i = 0; i < kBI; ++i)
#pragma unroll
            for (int j = 0; j < kBJ; ++j)
#pragma unroll
                for (int r = 0; r < 16; ++r) acc[i][j][r] = 0;
    }

    // fragments of sub-step s of stage ST (its buffers in st) into set F
    template <int F, int ST>
    __device__ __forceinline__ void read(const Stages& st, int s) {
        const int l = threadIdx.x & 63;
        const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
        const int ra = wave_row(wave), rb = wave_col(wave);
        // in the order the MFMAs consume them
        typedef typename El::Frag Frag;
        fa[F][0] = __builtin_bit_cast(Frag, read_frag<BM, AK>(st.a[ST], ST & 1, ra, s, l));
#pragma unroll
        for (int j = 0; j < kBJ; ++j)
            fb[F][j] = __builtin_bit_cast(Frag, read_frag<BN, BK>(st.b[ST], ST & 1, rb + 32 * j, s, l));
#pragma unroll
        for (int i = 1; i < kBI; ++i)
            fa[F][i] = __builtin_bit_cast(Frag, read_frag<BM, AK>(st.a[ST], ST & 1, ra + 32 * i, s, l));
    }

    // products of sub-step F of stage ST (% 4).  FIRST: the tile's first products, accumulated onto zero (this is what
    // clears the accumulators between tiles)
    template <int F, int ST, bool FIRST = false>
    __device__ __forceinline__ void mfma() {
#pragma unroll
        for (int i = 0; i < kBI; ++i)
#pragma unroll
            for (int j = 0; j < kBJ; ++j)
                acc[i][j] = El::mfma(fb[F][j], fa[F][i], FIRST ? typename El::Acc{} : acc[i][j]);
    }
};

// Write a finished tile: out[row * ld + col] = tile[row][col] rounded once to
// the output type, for row < rows and col < cols (cols a multiple of 4).
// Each lane stores its four consecutive columns as one 8- or 16-byte buffer
// store; lanes outside the valid region get an out-of-range offset, and
// their stores are dropped by the hardware range check, so the epilogue has
// no branches.  Each 32-row block gets its own descriptor, which keeps the
// per-lane offsets below 2^31 for ld <= 2^22.
template <bool OUT_BF16, class Mma>
__device__ __forceinline__ void store_tile(const Mma& mma, void* out, int64_t ld, int rows, int cols) {
    typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
    typedef float f32x2 __attribute__((ext_vector_type(2)));
    typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
    constexpr int ES = OUT_BF16 ? 2 : 4;
    // opaque lane index: the offsets do not depend on the tile and would
    // otherwise be hoisted out of the tile loop and held in registers
    int lane = threadIdx.x & 63;
    asm volatile("" : "+v"(lane));
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int ra = Mma::wave_row(wave), rb = Mma::wave_col(wave);
    const int r = lane & 31;
#pragma unroll
    for (int i = 0; i < Mma::kBI; ++i) {
        const int r0 = ra + 32 * i;
        const __amdgpu_buffer_rsrc_t rs = make_rsrc(reinterpret_cast<char*>(out) + (int64_t)r0 * ld * ES);
        const bool rok = r0 + r < rows;
#pragma unroll
        for (int j = 0; j < Mma::kBJ; ++j) {
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const int c = rb + 32 * j + 8 * q + 4 * (lane >> 5);
                const uint32_t o = rok && c < cols ? (uint32_t)((r * ld + c) * ES) : kOOB;
                const f32x16& a = mma.acc[i][j];
                if constexpr (OUT_BF16) {
                    const bf16x2 lo = __builtin_convertvector((f32x2{a[4 * q], a[4 * q + 1]}), bf16x2);
                    const bf16x2 hi = __builtin_convertvector((f32x2{a[4 * q + 2], a[4 * q + 3]}), bf16x2);
                    const u32x2 d = {__builtin_bit_cast(uint32_t, lo), __builtin_bit_cast(uint32_t, hi)};
                    __builtin_amdgcn_raw_buffer_store_b64(d, rs, o, 0, 0);
                } else {
                    const u32x4 d = {__float_as_uint(a[4 * q]), __float_as_uint(a[4 * q + 1]),
                                     __float_as_uint(a[4 * q + 2]), __float_as_uint(a[4 * q + 3])};
                    __builtin_amdgcn_raw_buffer_store_b128(d, rs, o, 0, 0);
                }
            }
            __builtin_amdgcn_sched_barrier(0);
        }
    }
}

// Write a finished tile like store_tile, but so that every global store
// instruction writes whole 128-byte lines (R = ep_rows of the tile, from
// plan.hpp, which sizes the LDS for it), with the non-temporal hint.  In the
// accumulator layout a lane owns one row of each 32x32 block, so a direct
// store touches 32 rows (32 lines, 16 or 32 bytes each) per instruction;
// written back-to-back by every workgroup at a tile boundary, those partial
// lines cost more than the rest of the epilogue.  Here each wave moves its
// blocks through its own R x 128-byte LDS scratch `scr`: a 128-byte row
// segment (64 BF16 or 32 FP32 columns, i.e. two or one 32-column blocks) of R
// rows at a time, written by the lanes that own those rows and read back as
// 16-byte chunks, eight lanes per row, then stored with 16-byte buffer stores
// (R/8 rows of whole lines per instruction).  Chunk c of scratch row rr sits
// at 16 * (c ^ (rr & 7)), so the read-back is free of bank conflicts.  Masking
// as in store_tile; cols must be a multiple of 8 (BF16) or 4 (FP32).  The
// scratch is private to the wave, so a wave-level sync between the phases is
// all it needs.  CPOL is the stores' cache policy: non-temporal for outputs;
// 0 for data read back soon (the weight gradient's chunk partials, which the
// fold then finds in the last-level cache).
template <bool OUT_BF16, int R, int CPOL = kCpolNT, class Mma>
__device__ __forceinline__ void store_tile_lines(const Mma& mma, lds_t* scr, void* out, int64_t ld, int rows,
                                                 int cols) {
    typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
    typedef float f32x2 __attribute__((ext_vector_type(2)));
    typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
    constexpr int ES = OUT_BF16 ? 2 : 4;
    constexpr int SEG = 128 / ES;   // columns per 128-byte segment
    constexpr int BPS = SEG / 32;   // 32-column blocks per segment
    constexpr int CPL = R / 8;      // read-back chunks per lane and round
    static_assert(R == 8 || R == 16, "rounds of 8 or 16 rows");
    static_assert(Mma::kBJ % BPS == 0, "whole segments per wave");
    int lane = threadIdx.x & 63;
    asm volatile("" : "+v"(lane));
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int ra = Mma::wave_row(wave), rb = Mma::wave_col(wave);
    lds_t* sw = scr + wave * (R * 128);
    const int r = lane & 31, h = lane >> 5;
    const int rr = r % R;   // this lane's scratch row in the round that owns it
    const int sx = rr & 7;
#pragma unroll
    for (int i = 0; i < Mma::kBI; ++i) {
        const int r0 = ra + 32 * i;
        const __amdgpu_buffer_rsrc_t rs = make_rsrc(reinterpret_cast<char*>(out) + (int64_t)r0 * ld * ES);
#pragma unroll
        for (int g = 0; g < Mma::kBJ / BPS; ++g) {
            const int c0 = rb + g * SEG;
#pragma unroll
            for (int s = 0; s < 32 / R; ++s) {
                if (r / R == s) {
#pragma unroll
                    for (int b = 0; b < BPS; ++b) {
                        const f32x16& a = mma.acc[i][g * BPS + b];
#pragma unroll
                        for (int q = 0; q < 4; ++q) {
                            if constexpr (OUT_BF16) {
                                // columns 32b + 8q + 4h .. +3: chunk 4b + q, its half h
                                const bf16x2 lo = __builtin_convertvector((f32x2{a[4 * q], a[4 * q + 1]}), bf16x2);
                                const bf16x2 hi = __builtin_convertvector((f32x2{a[4 * q + 2], a[4 * q + 3]}), bf16x2);
                                *reinterpret_cast<__attribute__((address_space(3))) u32x2*>(
                                    sw + rr * 128 + (((4 * b + q) ^ sx) << 4) + 8 * h) =
                                    u32x2{__builtin_bit_cast(uint32_t, lo), __builtin_bit_cast(uint32_t, hi)};
                            } else {
                                // columns 8q + 4h .. +3: chunk 2q + h
                                *reinterpret_cast<__attribute__((address_space(3))) u32x4*>(
                                    sw + rr * 128 + (((2 * q + h) ^ sx) << 4)) =
                                    u32x4{__float_as_uint(a[4 * q]), __float_as_uint(a[4 * q + 1]),
                                          __float_as_uint(a[4 * q + 2]), __float_as_uint(a[4 * q + 3])};
                            }
                        }
                    }
                }
                wave_lds_sync();   // the round's rows are in the scratch
#pragma unroll
                for (int k = 0; k < CPL; ++k) {
                    const int idx = lane + 64 * k, row = idx >> 3, c = idx & 7;
                    const u32x4 v = *reinterpret_cast<const __attribute__((address_space(3))) u32x4*>(
                        sw + row * 128 + ((c ^ (row & 7)) << 4));
                    const int rowb = s * R + row;            // row within the 32-row block
                    const int col = c0 + c * (16 / ES);
                    const uint32_t o = r0 + rowb < rows && col < cols ? (uint32_t)((rowb * ld + col) * ES) : kOOB;
                    __builtin_amdgcn_raw_buffer_store_b128(v, rs, o, 0, CPOL);
                }
                wave_lds_sync();   // read back before the next round overwrites it
            }
        }
    }
}

// What a runner is made of, by element type: loads and products of whole
// values here; block-scaled elements have their own (mxfp4.hip).
template <class El>
struct EngineParts {
    template <int BM, int BN, bool AK, bool BK, int WAVES>
    using Mma = TileMma<BM, BN, AK, BK, WAVES, El>;
    template <int ROWS, bool KMAJ, int WAVES, bool PAIRED, bool GATHERED>
    using Loader = StageLoader<ROWS, KMAJ, WAVES, PAIRED, GATHERED>;
};

// Issue schedule of the stage loads of a 4-wave runner (steps t of the
// global step sequence; the prologue acts as steps -4 .. -1).  A K-major operand loads stages t+3
// and t+4 at odd steps (into the pair buffer whose two stages t-1 and t were
// read by then), an MN-major operand stage t+4 at every step; within a step
// A goes before B.  The pipeline waits, at the barrier of step s, until
// stage s+1 of both operands has landed: with buffer loads returning in
// issue order, that is "at most N pending", N the number of loads issued
// after the last one of stage s+1.
template <bool AK, bool BK, int CA, int CB>
struct IssuePlan {
    static constexpr int loads_at(int t, int op) {
        const bool k = op == 0 ? AK : BK;
        const int c = op == 0 ? CA : CB;
        return k ? ((t & 1) ? c : 0) : c;
    }
    static constexpr int issue_step(bool k, int X) { return k ? ((X & 1) ? X - 4 : X - 3) : X - 4; }
    // loads issued after those of stage X, up to and including step `upto`
    static constexpr int after(int X, int upto) {
        const int ta = issue_step(AK, X), tb = issue_step(BK, X);
        const int last = 2 * ta > 2 * tb + 1 ? 2 * ta : 2 * tb + 1;
        int n = 0;
        for (int t = (ta < tb ? ta : tb); t <= upto; ++t)
            for (int op = 0; op < 2; ++op)
                if (2 * t + op > last) n += loads_at(t, op);
        return n;
    }
    static constexpr int at_barrier(int s) { return after(s + 1, s - 1); }   // wait at step s
    static constexpr int prologue = after(0, -1);                              // wait for stage 0
};

// A kernel's own loads for a tile (to LDS, in flight beside the stages'): none.
struct NoLoads {
    __device__ __forceinline__ void operator()(const TileInfo&) const {}
};

// Persistent tile loop over the stage pipeline.  `more()` tells whether this
// workgroup has another tile and `next(t)` decodes it; `finish(t, mma)`
// writes a finished tile from the accumulators.  Every step has the same
// shape (up to the parity that decides whether a K-major pair is loaded):
// it runs both MFMA sub-steps and issues its loads.  Stages past the end of a
// tile (the padding up to a multiple of four, or past the last tile) are
// "loaded" with every lane masked, which writes zeros to LDS without
// touching memory, so the MFMAs of a padding step add zeros and no branch is
// taken around the accumulators.  The next tile is decoded at the start of
// step nk4-4, whose loads fetch its first stage.  `loads(t)` may issue LDS
// loads that belong to a tile: it is called once per tile, before the first
// tile's stages or else right after the barrier of the step that decodes the
// tile (so after every wave has left the epilogue before the current tile),
// and what it loads has landed for every wave by the tile's epilogue.  Must be
// called by all threads.
template <int BM, int BN, bool AK, bool BK, int WAVES = kGemmWaves, class El = Bf16, bool PAIRED_B = false,
          bool GATHERED_A = false>
struct TileRunner {
    using Mma = typename EngineParts<El>::template Mma<BM, BN, AK, BK, WAVES>;
    using LA = typename EngineParts<El>::template Loader<BM, AK, WAVES, false, GATHERED_A>;
    using LB = typename EngineParts<El>::template Loader<BN, BK, WAVES, PAIRED_B, false>;
    using Plan = IssuePlan<AK, BK, LA::kPerWave, LB::kPerWave>;
    Mma mma;
    LA la;
    LB lb;
    Stages st;
    TileInfo cur, nxt;
    int nk, nk4, nk_nxt;
    bool has_next;

    // The first step group of a tile accumulates onto zero instead of
    // clearing the accumulators first.  Only with 8 waves, whose accumulators
    // live in VGPRs: with 4 waves they sit in AGPRs, and the extra copy of
    // the group makes the compiler move them out and spill.
    static constexpr bool kPeel = WAVES == 8;

    static __device__ __forceinline__ int stages_of(const TileInfo& t) {
        return (t.A.klen + kStageK - 1) / kStageK;
    }
    // steps run for a tile of n stages: whole groups of kStages (the stages
    // past n load zeros), at least the peeled group.  The next tile is
    // decoded inside a group's steps, so every tile must have at least one
    // reduction value: a tile of none would never hand over to the next one
    // (the callers' walks hold no item of zero length).  Forcing a group
    // here instead makes the compiler spill the 4-wave kernels' accumulators.
    static __device__ __forceinline__ int round4(int n) {
        const int r = (n + kStages - 1) & ~(kStages - 1);
        return kPeel && r < kStages ? kStages : r;
    }

    // With 8 waves the workgroup barrier is passed at odd steps only: the
    // two waves of a SIMD stop issuing MFMAs at a barrier, and with two of
    // them per SIMD that stall is the larger cost.  The loads then belong to
    // the odd steps: step t loads stages t+3 and t+4 into the buffers of
    // stages t-1 and t, which every wave has finished reading at its
    // barrier, and that barrier waits for all loads in flight: those of
    // stages t+1 and t+2, which steps t and t+1 read.
    static constexpr bool kBar2 = WAVES == 8;

    // With kBar2 the loads of an odd step t (stages t+3 and t+4: kNLT wave
    // instructions per wave, A's before B's) may be spread over three
    // sub-steps: instructions [0, kS1) go out in sub-step 1 of step t,
    // [kS1, kS2) in sub-step 0 of step t+1 and [kS2, kNLT) in its sub-step 1,
    // interleaved with their MFMAs.  All of them still land before the
    // barrier of step t+2, which waits for every load in flight.  The last
    // odd step of a tile fetches the next tile's stages 2 and 3, and that
    // tile's first step issues the rest; the prologue issues the first
    // tile's stages 0 and 1 and part of 2 and 3 in the same way.  As
    // measured, spreading pays with a transposed (MN-major) B operand, read
    // back with two LDS instructions per fragment: 3/3/2 of the 8 gained 4 %
    // on the data gradient without W^T and 1 % on the weight gradient (8 of
    // 8 at the odd step and the other splits tried were slower); with both
    // operands K-major it gained nothing or lost, so they issue everything
    // at the odd step.
    static constexpr int kNLT = (AK ? 1 : 2) * LA::kPerWave + (BK ? 1 : 2) * LB::kPerWave;
    static constexpr int kS1 = kBar2 && !BK && kNLT == 8 ? 3 : kNLT;
    static constexpr int kS2 = kBar2 && !BK && kNLT == 8 ? 6 : kNLT;
    // the step that switches the loaders to the next tile: the first one
    // whose loads fetch from it
    static constexpr int kReinitST = kBar2 ? 1 : 0;

    // Instructions [I0, I1) of the loads of odd step kt_odd (STO = kt_odd % 4).
    template <int STO, int I0, int I1, int Q>
    __device__ __forceinline__ void issue_odd_entry(int kt_odd) {
        // entry Q: a load of A for Q < nA, else of B; a K-major operand has
        // one (the pair t+3, t+4), an MN-major one two (t+3, then t+4)
        constexpr int nA = AK ? 1 : 2;
        constexpr bool isA = Q < nA;
        constexpr int P = isA ? LA::kPerWave : LB::kPerWave;
        constexpr int start = isA ? Q * LA::kPerWave : nA * LA::kPerWave + (Q - nA) * LB::kPerWave;
        constexpr int j0 = I0 - start < 0 ? 0 : I0 - start > P ? P : I0 - start;
        constexpr int j1 = I1 - start < 0 ? 0 : I1 - start > P ? P : I1 - start;
        if constexpr (j0 < j1) {
            constexpr int d = 3 + (isA ? Q : Q - nA);
            const int L = kt_odd + d;
            const int Ls = L < nk4 ? L : L - nk4;
            if constexpr (isA) la.template issue_part<j0, j1>(st.a[(STO + d) % kStages], Ls, L < nk4 || has_next);
            else lb.template issue_part<j0, j1>(st.b[(STO + d) % kStages], Ls, L < nk4 || has_next);
        }
    }
    template <int STO, int I0, int I1, int... Q>
    __device__ __forceinline__ void issue_odd_entries(int kt_odd, std::integer_sequence<int, Q...>) {
        (issue_odd_entry<STO, I0, I1, Q>(kt_odd), ...);
    }
    template <int STO, int I0, int I1>
    __device__ __forceinline__ void issue_odd(int kt_odd) {
        if constexpr (I0 < I1)
            issue_odd_entries<STO, I0, I1>(kt_odd, std::make_integer_sequence<int, (AK ? 1 : 2) + (BK ? 1 : 2)>{});
    }

    // Without kBar2, the loads of step t (t % 4 == ST) for operand loader
    // `ld`: stage t+4, or for a K-major operand at odd t the pair t+3, t+4,
    // of this tile or, past nk4, of the next one (the loaders then point at
    // the next tile).
    template <int ST, bool K, class Ld>
    __device__ __forceinline__ void issue(Ld& ld, lds_t* const* bufs, int kt) {
        static_assert(!kBar2, "with kBar2 the loads go through issue_odd");
        if constexpr (!K || (ST & 1)) {
            const int L = kt + (K ? 3 : 4);
            const int Ls = L < nk4 ? L : L - nk4;
            ld.issue(bufs[(ST + (K ? 3 : 4)) % kStages], Ls, L < nk4 || has_next);
        }
    }

    // Sub-step 1 of odd step kt with kBar2: its MFMAs, the loads [0, N) of
    // the step, the sub-step 0 fragments of stage kt+1.
    template <int ST, int N>
    __device__ __forceinline__ void odd_substep1(int kt) {
        issue_odd<ST, 0, N>(kt);
        mma.template read<0, (ST + 1) % kStages>(st, 0);
        mma.template mfma<1, ST>();
        if constexpr (AK && BK) sched_interleave<Mma::kMfmas, Mma::kReads, N>();
    }

    // Step kt of the current tile; ST = kt % 4; FIRST for step 0.
    template <int ST, bool FIRST = false, class Next, class Loads>
    __device__ __forceinline__ void step(int kt, Next& next, Loads& loads) {
        constexpr int NX = (ST + 1) % kStages;
        constexpr int STO = (ST + kStages - 1) % kStages;
        // with kBar2 an even step issues the deferred loads of step kt-1 (for
        // a tile's first step, those of the previous tile's last step or of
        // the prologue: its stages 2 and 3)
        constexpr bool DEF = kBar2 && !(ST & 1);
        // loads issued in this step without kBar2 (the schedule hints place them)
        constexpr int NL = (AK && !(ST & 1) ? 0 : LA::kPerWave) + (BK && !(ST & 1) ? 0 : LB::kPerWave);
        if constexpr (ST == kReinitST) {
            if (kt - ST + kStages == nk4 && has_next) {
                next(nxt);
                nk_nxt = stages_of(nxt);
                la.init(nxt.A);
                lb.init(nxt.B);
            }
        }
        __builtin_amdgcn_sched_barrier(0);
        // sub-step 0: its MFMAs; the sub-step 1 fragments
        mma.template read<1, ST>(st, 1);
        if constexpr (DEF) issue_odd<STO, kS1, kS2>(kt - 1);
        mma.template mfma<0, ST, FIRST>();
        if constexpr (AK && BK) sched_interleave<Mma::kMfmas, Mma::kReads, DEF ? kS2 - kS1 : 0>();
        __builtin_amdgcn_sched_barrier(0);
        // stage kt+1 has landed for every wave, and every wave is done
        // reading stage kt
        if constexpr (!kBar2 || (ST & 1)) {
            wait_vm_lgkm<kBar2 ? 0 : Plan::at_barrier(4 + ST)>();
            barrier_nofence();
        }
        if constexpr (ST == kReinitST && !std::is_same<Loads, NoLoads>::value) {
            static_assert(!kBar2 || (ST & 1), "the decoding step passes a barrier");
            if (kt - ST + kStages == nk4 && has_next) loads(nxt);
        }
        // sub-step 1: its MFMAs; the loads into the buffers just freed; the
        // sub-step 0 fragments of stage kt+1
        if constexpr (kBar2 && (ST & 1)) {
            odd_substep1<ST, kS1>(kt);
        } else if constexpr (kBar2) {
            if constexpr (DEF) issue_odd<STO, kS2, kNLT>(kt - 1);
            mma.template read<0, NX>(st, 0);
            mma.template mfma<1, ST>();
            if constexpr (AK && BK) sched_interleave<Mma::kMfmas, Mma::kReads, DEF ? kNLT - kS2 : 0>();
        } else {
            issue<ST, AK>(la, st.a, kt);
            issue<ST, BK>(lb, st.b, kt);
            mma.template read<0, NX>(st, 0);
            mma.template mfma<1, ST>();
            if constexpr (AK && BK) sched_interleave<Mma::kMfmas, Mma::kReads, NL>();
        }
        __builtin_amdgcn_sched_barrier(0);
    }

    template <class More, class Next, class Finish, class Loads = NoLoads>
    __device__ __forceinline__ void run(More more, Next next, Finish finish, Loads loads = Loads{}) {
        if (!more()) return;
        next(cur);
        nk = stages_of(cur);
        nk4 = round4(nk);
        has_next = false;
        loads(cur);
        la.init(cur.A);
        lb.init(cur.B);
        if constexpr (kBar2) {
            // prologue: stages 0, 1 and the first part of 2, 3, as odd
            // steps -3 and -1 would issue them; then wait for stages 0 and 1
            // (step 0 reads both)
            issue_odd<1, 0, kNLT>(-3);
            issue_odd<3, 0, kS1>(-1);
            wait_vm_lgkm<kS1>();
        } else {
            // prologue: stages 0..3 (zeros past nk) in the order of steps -4..-1
#pragma unroll
            for (int t = -4; t < 0; ++t) {
#pragma unroll
                for (int op = 0; op < 2; ++op) {
                    const bool k = op == 0 ? AK : BK;
                    if (k && !(t & 1)) continue;
                    const int L = t + (k ? 3 : 4);
                    if (op == 0) la.issue(st.a[L], L, true);
                    else lb.issue(st.b[L], L, true);
                }
            }
            // stage 0 landed
            wait_vm_lgkm<Plan::prologue>();
        }
        barrier_nofence();
        mma.template read<0, 0>(st, 0);
        for (;;) {
            has_next = more();
            nk_nxt = 0;
            int kt0 = 0;
            if constexpr (kPeel) {
                step<0, true>(0, next, loads);
                step<1>(1, next, loads);
                step<2>(2, next, loads);
                step<3>(3, next, loads);
                kt0 = kStages;
            } else {
                mma.zero();
            }
            for (int kt = kt0; kt < nk4; kt += kStages) {
                step<0>(kt, next, loads);
                step<1>(kt + 1, next, loads);
                step<2>(kt + 2, next, loads);
                step<3>(kt + 3, next, loads);
            }
            finish(cur, mma);
            if (!has_next) break;
            cur = nxt;
            nk = nk_nxt;
            nk4 = round4(nk);
        }
        // the masked loads past the last tile are still in flight
        __builtin_amdgcn_s_waitcnt(0);
    }
};

}  // namespace drgg
