// internal.hpp -- declarations shared by the C ABI (api.cpp, api_moe.cpp,
// api_experts.cpp) and the kernel launchers (the .hip files).  Not part of the
// public interface.
#pragma once

#include <hip/hip_runtime.h>

#include <cstddef>
#include <cstdint>

#include "../../include/drgg.h"

namespace drgg {

// ---- argument checks shared by the C ABI's files ---------------------------

constexpr int64_t kMaxBytes = (int64_t)1 << 62;

// checked a * b for non-negative operands
inline bool mul_ok(int64_t a, int64_t b, int64_t* out) {
    if (a < 0 || b < 0) return false;
    if (a != 0 && b > kMaxBytes / a) return false;
    *out = a * b;
    return true;
}

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// DRGG_EDEVICE, with the HIP error kept for drgg_status_string (api.cpp)
drgg_status device_error(hipError_t e);
inline drgg_status launch_status(hipError_t e) { return e == hipSuccess ? DRGG_OK : device_error(e); }

// DRGG_KNOB_TILE (api.cpp)
int knob_tile();

// CU count of the current device (api.cpp)
drgg_status current_cu_count(int* cus);

// Debug check of the group offsets (api.cpp): whether it is on, and the check.
bool checks_offsets();
drgg_status check_offsets_sync(const int32_t* offs, int32_t E, int64_t M, hipStream_t s);

// Arguments of the grouped-GEMM kernels, passed by value.
struct GemmArgs {
    const uint16_t* A;     // fwd: X   dgrad: G   wgrad: G  (BF16 bits)
    const uint16_t* B;     // fwd: W   dgrad: W   wgrad: X
    const int32_t* offs;   // group offsets [E+1], device (null: uniform groups of T rows)
    void* out;             // Y / dX / dW
    float* partial;        // det wgrad: chunk partial slots [slot][N][K]
    int32_t* fold_info;    // det wgrad: [E][4] = T_e, chunks_e, first slot, 0 (chunk kernel -> fold)
    float* tilesum;        // non-det wgrad: FP32 tile sums [E*P][BM*BN]
    uint32_t* tickets;     // non-det wgrad: [E*P]
    int64_t M, N, K;
    // Token-major operands and the fwd/dgrad output: row r (its index in the
    // offsets' row space) of group e starts at element base + r * rs + e * gs.
    // Grouped calls: rs = the row length, gs = 0.  Batched calls (offs null,
    // groups of T rows): rs = the row stride, gs = batch stride - T * rs.
    int64_t a_rs, a_gs;    // A: fwd X, dgrad G, wgrad G
    int64_t b_rs, b_gs;    // wgrad B: X
    int64_t o_rs, o_gs;    // fwd Y, dgrad dX
    int64_t T;             // offs null: group e is rows e*T .. e*T+T-1
    int64_t chunk_max;     // det wgrad: longest chunk
    int64_t items_max;     // workgroups launched (fwd/dgrad/det wgrad)
    int32_t E;
    int32_t reverse;       // walk work items in reverse (test knob)
    int32_t delay_seed;    // split program: seeded delays before tail arrivals (test knob; 0 = off)
    int32_t* report;       // split program: if set, workgroup 0 writes its tail decision here (test aid)
    int32_t zero_empty;    // det wgrad: no expert can have two chunks, so no fold runs and the chunk
                           // kernel writes the zero output of experts without tokens itself
};

// op 0: forward; 1: data gradient; 2: data gradient with a.B = W^T [E][K][N]
hipError_t launch_fwd_dgrad(int op, int tile, const GemmArgs& a, bool bf16, hipStream_t s);
hipError_t launch_transpose_w(const uint16_t* W, uint16_t* WT, int32_t E, int64_t N, int64_t K, hipStream_t s);
hipError_t launch_wgrad_det(int tile, const GemmArgs& a, bool bf16, hipStream_t s);
hipError_t launch_wgrad_atomic(int tile, const GemmArgs& a, int64_t grid_n, bool bf16, hipStream_t s);
hipError_t launch_router(const float* X, const float* Wr, float* out, int64_t M, int64_t N, int64_t K,
                         hipStream_t s);
hipError_t launch_router_ks(const float* X, const float* Wr, float* out, float* part, int64_t M, int64_t N,
                            int64_t K, int64_t ks, int64_t kq, hipStream_t s);
hipError_t launch_zero(void* p, size_t bytes, hipStream_t s);

// The fixed device workspace of grouped_gemm_wgrad_noalloc: its size, and the
// device address of the current device's copy (looked up once per device).
constexpr size_t kScratchBytes = size_t(64) << 20;
hipError_t scratch_buffer(void** ptr);
hipError_t launch_hold_cus(int n, uint64_t ticks, hipStream_t s);

// ---- the expert layer's operators (moe.hip, int8.hip) -----------------------

// Arguments of the row quantisation (quantize.hpp): X [T, 16 C] to codes and scales.
struct QuantArgs {
    const void* X;
    const int32_t* positions;   // null: row t stays row t
    int8_t* q;
    float* scale;
    int64_t T, C;               // C: groups of 16 values per row
    int32_t k;
};
// the longest BF16 rows, and the most values, that the selection's launch quantises too
constexpr int64_t kSelectQuantizeK = 4096, kSelectQuantizeMost = int64_t(1) << 23;

size_t route_table_bytes(int64_t T, int32_t E);   // the selection's workspace; 0 for one workgroup
hipError_t launch_moe_route(const float* logits, int64_t T, int32_t E, int32_t k, int renormalize, int32_t* experts,
                            float* weights, int32_t* offsets, int32_t* positions, int32_t* tokens, void* table,
                            hipStream_t s, const QuantArgs* quantize = nullptr);
hipError_t launch_moe_route_grad(const float* dweights, const float* logits, const int32_t* experts,
                                 const float* weights, int64_t T, int32_t E, int32_t k, int renormalize,
                                 float* dlogits, hipStream_t s);
hipError_t launch_moe_dispatch(const void* X, const int32_t* positions, int64_t T, int32_t k, int64_t H, bool bf16,
                               void* rows, hipStream_t s);
hipError_t launch_moe_combine(const void* rows, const int32_t* positions, const float* weights, int64_t T, int32_t k,
                              int64_t H, bool bf16, void* out, hipStream_t s);
hipError_t launch_moe_combine_grad(const void* dout, const void* rows, const int32_t* positions, const float* weights,
                                   int64_t T, int32_t k, int64_t H, bool bf16, void* drows, float* dweights,
                                   hipStream_t s);
hipError_t launch_quantize_int8(const void* X, bool bf16, int64_t T, int64_t K, const int32_t* positions, int32_t k,
                                int8_t* q, float* scale, hipStream_t s);

// Arguments of the 8-bit products: X [M,K], W [E,N,K] codes, xs [M], ws [E,N]
// scales, offs [E+1] on the device (null: one group of all M rows).
struct Int8Args {
    const int8_t* X;
    const int8_t* W;
    const float* xs;
    const float* ws;
    const int32_t* offs;
    void* out;
    int64_t M, N, K;
    int32_t E;
    const int32_t* rows = nullptr;   // row r of the product is row rows[r] of X [T,K] and xs [T] (null: row r)
    int64_t T = 0;
};
// the longest reduction whose sum fits 32 bits for any codes: 131056 * 128^2 < 2^31
constexpr int64_t kInt8MaxK = 131056;
hipError_t launch_int8(const Int8Args& a, bool gated, bool bf16, int cus, int forced_tile, hipStream_t s);

// ---- selection by scores (moe.hip), 4-bit products (mxfp4.hip), kept activations (gate.hip)

// Arguments of the 4-bit quantisation (mxfp4.hpp): X [T,K] to codes and scales.
struct MxQuantArgs {
    const void* X;
    uint8_t* codes;
    uint8_t* scales;
    int64_t T, K;
};
// The most values that the scored selection's launch quantises too: the serving
// block (E = 32, k = 8, H 2048, I 768) takes 32.1 instead of 34.2 us for 8 tokens,
// 45.4 for 47.6 at 256 and 74 for 77 at 1024; at 2048 tokens both take 103.
constexpr int64_t kSelectMxMost = int64_t(1) << 21;

// The scored selection; its workspace is moe_route's.  quantize: also the
// quantisation of these BF16 rows, which needs nothing of the selection.
hipError_t launch_moe_route_scores(const float* logits, int64_t T, int32_t E, int32_t k, const drgg_scoring& scoring,
                                   int32_t* experts, float* weights, int32_t* offsets, int32_t* positions,
                                   int32_t* tokens, void* table, hipStream_t s, const MxQuantArgs* quantize = nullptr);
hipError_t launch_moe_route_scores_grad(const float* dweights, const float* logits, const int32_t* experts,
                                        const float* weights, int64_t T, int32_t E, int32_t k,
                                        const drgg_scoring& scoring, float* dlogits, hipStream_t s);

hipError_t launch_quantize_mxfp4(const void* X, bool bf16, int64_t T, int64_t K, uint8_t* codes, uint8_t* scales,
                                 hipStream_t s);
hipError_t launch_dequantize_mxfp4(const uint8_t* codes, const uint8_t* scales, int64_t T, int64_t K, bool bf16,
                                   void* X, hipStream_t s);

// Arguments of the 4-bit products: X [M,K/2], W [E,N,K/2] codes, xs, ws scale
// bytes [ceil(K/256)][M], [E*N] rows of 8; the rest as in Int8Args.
struct MxArgs {
    const uint8_t* X;
    const uint8_t* W;
    const uint8_t* xs;
    const uint8_t* ws;
    const int32_t* offs;
    void* out;
    int64_t M, N, K;
    int32_t E;
    const int32_t* rows = nullptr;   // row r of the product is row rows[r] of X and xs, T rows (null: row r)
    int64_t T = 0;
    uint8_t* out_scales = nullptr;   // gated with rows: out are codes [M,N/4], with these scales (null: values)
};
hipError_t launch_mxfp4(const MxArgs& a, bool gated, bool bf16, int cus, int forced_tile, hipStream_t s);

hipError_t launch_moe_gate_int8(const void* GU, const int32_t* positions, const float* weights, int64_t T, int32_t k,
                                int64_t I, void* h, int8_t* codes, float* scale, hipStream_t s);
hipError_t launch_moe_gate_int8_grad(const void* dh, const int8_t* codes, const float* scale, const int32_t* positions,
                                     const float* weights, int64_t T, int32_t k, int64_t I, void* dGU, void* h,
                                     float* dweights, hipStream_t s);

// Per-launch timing marks (a measurement knob, off by default): when on, an
// event is recorded on the stream before every kernel launch of a call and
// once after the last one, so each kernel's duration can be read back.
void timing_mark(const char* kernel, hipStream_t s);   // before a launch
void timing_end(hipStream_t s);                         // after the last launch

}  // namespace drgg
