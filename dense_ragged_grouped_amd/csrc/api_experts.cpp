// api_experts.cpp -- the C ABI of the selection by scores, the products in
// microscaled 4-bit floating point and the activation kept in 8 bits (declared
// in include/drgg.h).  Argument checks in checked 64-bit arithmetic, then
// launches (moe.hip, mxfp4.hip, gate.hip) on the caller's stream.
#include <hip/hip_runtime.h>

#include <cmath>
#include <cstdint>

#include "../../include/drgg.h"
#include "internal.hpp"
#include "plan.hpp"

namespace drgg {
namespace {

bool aligned(const void* p, unsigned n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
// rows of E logits are read and written four at a time where all of them start aligned
bool aligned_logits(const void* p, int32_t E) { return aligned(p, E % 4 ? 4 : 16); }

drgg_status check_pairs(int64_t T, int32_t k) {
    int64_t r;
    if (k < 1 || k > 64) return DRGG_EINVAL;
    if (T < 0 || !mul_ok(T, k, &r) || r > INT32_MAX) return DRGG_ESHAPE;
    return DRGG_OK;
}

bool score_ok(const drgg_scoring* c) {
    return c && (c->score == DRGG_SCORE_SOFTMAX || c->score == DRGG_SCORE_SIGMOID) && c->scale > 0 && std::isfinite(c->scale);
}

// sizes of a selection, and the scoring (null: the plain one)
drgg_status check_scores(int64_t T, int32_t E, int32_t k, const drgg_scoring* c) {
    if (E < 1 || E > kMaxExperts || k > E) return DRGG_EINVAL;
    if (c) {
        if (!score_ok(c) || c->groups < 1 || c->groups > 64 || E % c->groups || c->top_groups < 1 ||
            c->top_groups > c->groups || (c->best != 1 && c->best != 2) || k > c->top_groups * (E / c->groups))
            return DRGG_EINVAL;
        if (!aligned(c->bias, 4)) return DRGG_EALIGN;
    }
    if (T > (int64_t(1) << 27)) return DRGG_ESHAPE;   // 16 threads per token in one launch
    return check_pairs(T, k);
}

drgg_status check_mx_rows(int64_t T, int64_t K, drgg_dtype dt) {
    if (dt != DRGG_BF16 && dt != DRGG_FP32) return DRGG_EINVAL;
    if (T < 0 || T > INT32_MAX || K < 32 || K > (1 << 22)) return DRGG_ESHAPE;
    return K % 32 ? DRGG_EALIGN : DRGG_OK;
}

// whether T rows of B bytes can be gathered: their offsets are 32 bits wide
bool can_gather(int64_t T, int64_t B) { return T * B <= INT32_MAX - 4096; }

int64_t mx_scale_bytes(int64_t rows, int64_t K) { return ceil_div(K, 256) * rows * 8; }

drgg_status run_mxfp4(const uint8_t* Xq, const uint8_t* xs, const uint8_t* Wq, const uint8_t* ws, const int32_t* offs,
                      const int32_t* rows, int64_t T, int32_t E, int64_t M, int64_t N, int64_t K, int gated,
                      drgg_dtype dt, void* Y, hipStream_t s) {
    if (E < 1 || E > kMaxExperts) return DRGG_EINVAL;
    if (dt != DRGG_BF16 && dt != DRGG_FP32) return DRGG_EINVAL;
    const int64_t na = gated ? 16 : 8;
    if (M < 0 || M > INT32_MAX || N < na || N > (1 << 22) || K < 32 || K > (1 << 22)) return DRGG_ESHAPE;
    if (N % na || K % 32) return DRGG_EALIGN;
    if (rows && (T < 1 || T > INT32_MAX || !can_gather(T, K / 2))) return DRGG_ESHAPE;
    if (!Wq || !ws || (M > 0 && (!Xq || !xs || !Y))) return DRGG_EINVAL;
    if (!aligned16(Xq) || !aligned16(Wq) || !aligned16(Y) || !aligned(xs, 8) || !aligned(ws, 8) || !aligned(offs, 4) ||
        !aligned(rows, 4))
        return DRGG_EALIGN;
    if (offs && checks_offsets()) {
        drgg_status st = check_offsets_sync(offs, E, M, s);
        if (st != DRGG_OK) return st;
    }
    if (M == 0) return DRGG_OK;
    int cus = 0;
    drgg_status st = current_cu_count(&cus);
    if (st != DRGG_OK) return st;
    return launch_status(launch_mxfp4(MxArgs{Xq, Wq, xs, ws, offs, Y, M, N, K, E, rows, T}, gated != 0, dt == DRGG_BF16, cus,
                                      knob_tile(), s));
}

// The parts of moe_ffn_mxfp4's workspace (byte offsets, multiples of 256).  The
// experts' outputs y take the place of the codes of X, which are no longer
// needed by then.  They are BF16, as in the 8-bit block: bytes bound their way to
// memory and back (16384 tokens, k = 8, H 2048: 537 MB each way, about 210 of 570
// us; FP32 would be twice that).  Their rounding and that of the sum make 0.24 % of
// the result, that of the sum alone 0.17 %.
struct MxFfnLayout {
    int64_t experts, weights, offsets, positions, tokens, table, hq, hs, x, xs, y, bytes;
};
drgg_status mx_ffn_layout(int64_t T, int32_t E, int32_t k, int64_t H, int64_t I, const drgg_scoring* c, MxFfnLayout* L) {
    drgg_status st = check_scores(T, E, k, c);
    if (st != DRGG_OK) return st;
    if (H < 32 || H > (1 << 22) || I < 32 || I > (1 << 21)) return DRGG_ESHAPE;
    if (H % 32 || I % 32) return DRGG_EALIGN;
    if (!can_gather(T, H / 2)) return DRGG_ESHAPE;
    const int64_t R = T * k;   // below 2^31; a row of any part is below 2^24 bytes
    int64_t at = 0;
    auto part = [&](int64_t n) {
        const int64_t o = at;
        at += round_up(n, 256);
        return o;
    };
    L->experts = part(R * 4);
    L->weights = part(R * 4);
    L->offsets = part(((int64_t)E + 1) * 4);
    L->positions = part(R * 4);
    L->tokens = part(R * 4);
    L->table = part((int64_t)route_table_bytes(T, E));
    L->hq = part(R * (I / 2));
    L->hs = part(mx_scale_bytes(R, I));
    L->y = at;
    L->x = part(T * (H / 2));
    L->xs = part(mx_scale_bytes(T, H));
    const int64_t y = L->y + round_up(R * H * 2, 256);
    L->bytes = at > y ? at : y;
    return DRGG_OK;
}

drgg_status check_gate(int64_t T, int32_t k, int64_t I) {
    drgg_status st = check_pairs(T, k);
    if (st != DRGG_OK) return st;
    if (I < 8 || I > (1 << 21)) return DRGG_ESHAPE;
    return I % 8 ? DRGG_EALIGN : DRGG_OK;
}

}  // namespace
}  // namespace drgg

using namespace drgg;

extern "C" {

drgg_status moe_route_scores(const float* logits, int64_t T, int32_t E, int32_t k, const drgg_scoring* scoring,
                             int32_t* experts, float* weights, int32_t* group_offsets, int32_t* positions,
                             int32_t* tokens, void* workspace, size_t workspace_bytes, hipStream_t stream) {
    if (!scoring) return DRGG_EINVAL;
    drgg_status st = check_scores(T, E, k, scoring);
    if (st != DRGG_OK) return st;
    if (!group_offsets || (T > 0 && (!logits || !experts || !weights || !positions))) return DRGG_EINVAL;
    if (!aligned_logits(logits, E) || !aligned(experts, 4) || !aligned(weights, 4) || !aligned(group_offsets, 4) ||
        !aligned(positions, 4) || !aligned(tokens, 4))
        return DRGG_EALIGN;
    const size_t need = route_table_bytes(T, E);
    if (need > 0) {
        if (!workspace || workspace_bytes < need) return DRGG_EWORKSPACE;
        if (!aligned16(workspace)) return DRGG_EALIGN;
    }
    return launch_status(launch_moe_route_scores(logits, T, E, k, *scoring, experts, weights, group_offsets, positions,
                                                 tokens, workspace, stream));
}

drgg_status moe_route_scores_grad(const float* dweights, const float* logits, const int32_t* experts,
                                  const float* weights, int64_t T, int32_t E, int32_t k, const drgg_scoring* scoring,
                                  float* dlogits, hipStream_t stream) {
    if (!score_ok(scoring)) return DRGG_EINVAL;
    drgg_status st = check_scores(T, E, k, nullptr);
    if (st != DRGG_OK) return st;
    if (T > 0 && (!dweights || !logits || !experts || !weights || !dlogits)) return DRGG_EINVAL;
    if (!aligned_logits(logits, E) || !aligned_logits(dlogits, E) || !aligned(dweights, 4) || !aligned(experts, 4) ||
        !aligned(weights, 4))
        return DRGG_EALIGN;
    if (T == 0) return DRGG_OK;
    return launch_status(launch_moe_route_scores_grad(dweights, logits, experts, weights, T, E, k, *scoring, dlogits, stream));
}

drgg_status quantize_mxfp4(const void* X, drgg_dtype dtype, int64_t T, int64_t K, uint8_t* codes, uint8_t* scales,
                           hipStream_t stream) {
    drgg_status st = check_mx_rows(T, K, dtype);
    if (st != DRGG_OK) return st;
    if (T > 0 && (!X || !codes || !scales)) return DRGG_EINVAL;
    if (!aligned16(X) || !aligned16(codes) || !aligned(scales, 8)) return DRGG_EALIGN;
    if (T == 0) return DRGG_OK;
    return launch_status(launch_quantize_mxfp4(X, dtype == DRGG_BF16, T, K, codes, scales, stream));
}

drgg_status dequantize_mxfp4(const uint8_t* codes, const uint8_t* scales, int64_t T, int64_t K, drgg_dtype dtype,
                             void* X, hipStream_t stream) {
    drgg_status st = check_mx_rows(T, K, dtype);
    if (st != DRGG_OK) return st;
    if (T > 0 && (!X || !codes || !scales)) return DRGG_EINVAL;
    if (!aligned16(X) || !aligned16(codes) || !aligned(scales, 8)) return DRGG_EALIGN;
    if (T == 0) return DRGG_OK;
    return launch_status(launch_dequantize_mxfp4(codes, scales, T, K, dtype == DRGG_BF16, X, stream));
}

drgg_status grouped_gemm_mxfp4(const uint8_t* Xq, const uint8_t* x_scale, const uint8_t* Wq, const uint8_t* w_scale,
                               const int32_t* group_offsets, const int32_t* rows, int64_t T, int32_t E, int64_t M,
                               int64_t N, int64_t K, int gated, drgg_dtype out_dtype, void* Y, hipStream_t stream) {
    if (!group_offsets) return DRGG_EINVAL;
    return run_mxfp4(Xq, x_scale, Wq, w_scale, group_offsets, rows, T, E, M, N, K, gated, out_dtype, Y, stream);
}

drgg_status gemm_mxfp4(const uint8_t* Xq, const uint8_t* x_scale, const uint8_t* Wq, const uint8_t* w_scale, int64_t M,
                       int64_t N, int64_t K, int gated, drgg_dtype out_dtype, void* Y, hipStream_t stream) {
    return run_mxfp4(Xq, x_scale, Wq, w_scale, nullptr, nullptr, 0, 1, M, N, K, gated, out_dtype, Y, stream);
}

drgg_status moe_ffn_mxfp4_workspace_size(int64_t T, int32_t E, int32_t k, int64_t H, int64_t I, size_t* bytes) {
    if (!bytes) return DRGG_EINVAL;
    MxFfnLayout L;
    drgg_status st = mx_ffn_layout(T, E, k, H, I, nullptr, &L);
    if (st != DRGG_OK) return st;
    *bytes = (size_t)L.bytes;
    return DRGG_OK;
}

drgg_status moe_ffn_mxfp4(const void* X, const float* logits, const uint8_t* W1q, const uint8_t* w1_scale,
                          const uint8_t* W2q, const uint8_t* w2_scale, int64_t T, int32_t E, int32_t k, int64_t H,
                          int64_t I, const drgg_scoring* scoring, void* out, void* workspace, size_t workspace_bytes,
                          hipStream_t stream) {
    MxFfnLayout L;
    drgg_status st = mx_ffn_layout(T, E, k, H, I, scoring, &L);
    if (st != DRGG_OK) return st;
    if (!W1q || !w1_scale || !W2q || !w2_scale || (T > 0 && (!X || !logits || !out))) return DRGG_EINVAL;
    if (!aligned16(X) || !aligned_logits(logits, E) || !aligned16(W1q) || !aligned(w1_scale, 8) || !aligned16(W2q) ||
        !aligned(w2_scale, 8) || !aligned16(out))
        return DRGG_EALIGN;
    if (T == 0) return DRGG_OK;
    if (!workspace || workspace_bytes < (size_t)L.bytes) return DRGG_EWORKSPACE;
    if (!aligned16(workspace)) return DRGG_EALIGN;
    char* ws = static_cast<char*>(workspace);
    auto* experts = reinterpret_cast<int32_t*>(ws + L.experts);
    auto* weights = reinterpret_cast<float*>(ws + L.weights);
    auto* offsets = reinterpret_cast<int32_t*>(ws + L.offsets);
    auto* positions = reinterpret_cast<int32_t*>(ws + L.positions);
    auto* tokens = reinterpret_cast<int32_t*>(ws + L.tokens);
    auto* x = reinterpret_cast<uint8_t*>(ws + L.x);
    auto* xs = reinterpret_cast<uint8_t*>(ws + L.xs);
    auto* hq = reinterpret_cast<uint8_t*>(ws + L.hq);
    auto* hs = reinterpret_cast<uint8_t*>(ws + L.hs);
    int cus = 0;
    st = current_cu_count(&cus);
    if (st != DRGG_OK) return st;
    const int64_t R = T * k;
    // the scored selection's launch quantises few tokens' rows too
    const MxQuantArgs rows{X, x, xs, T, H};
    const bool together = scoring && T * H <= kSelectMxMost;
    hipError_t e = scoring ? launch_moe_route_scores(logits, T, E, k, *scoring, experts, weights, offsets, positions, tokens,
                                                     ws + L.table, stream, together ? &rows : nullptr)
                           : launch_moe_route(logits, T, E, k, 1, experts, weights, offsets, positions, tokens,
                                              ws + L.table, stream);
    if (e == hipSuccess && !together) e = launch_quantize_mxfp4(X, true, T, H, x, xs, stream);
    if (e == hipSuccess)
        e = launch_mxfp4(MxArgs{x, W1q, xs, w1_scale, offsets, hq, R, 2 * I, H, E, tokens, T, hs}, true, false, cus,
                         knob_tile(), stream);
    if (e == hipSuccess)
        e = launch_mxfp4(MxArgs{hq, W2q, hs, w2_scale, offsets, ws + L.y, R, H, I, E}, false, true, cus, knob_tile(), stream);
    if (e == hipSuccess) e = launch_moe_combine(ws + L.y, positions, weights, T, k, H, true, out, stream);
    return launch_status(e);
}

drgg_status moe_gate_int8(const void* GU, const int32_t* positions, const float* weights, int64_t T, int32_t k,
                          int64_t I, void* h, int8_t* codes, float* scale, hipStream_t stream) {
    drgg_status st = check_gate(T, k, I);
    if (st != DRGG_OK) return st;
    if (T > 0 && (!GU || !positions || !weights || !h || !codes || !scale)) return DRGG_EINVAL;
    if (!aligned16(GU) || !aligned16(h) || !aligned(codes, 8) || !aligned(positions, 4) || !aligned(weights, 4) ||
        !aligned(scale, 4))
        return DRGG_EALIGN;
    if (T == 0) return DRGG_OK;
    return launch_status(launch_moe_gate_int8(GU, positions, weights, T, k, I, h, codes, scale, stream));
}

drgg_status moe_gate_int8_grad(const void* dh, const int8_t* codes, const float* scale, const int32_t* positions,
                               const float* weights, int64_t T, int32_t k, int64_t I, void* dGU, void* h,
                               float* dweights, hipStream_t stream) {
    drgg_status st = check_gate(T, k, I);
    if (st != DRGG_OK) return st;
    if (T > 0 && (!dh || !codes || !scale || !positions || !weights || !dGU || !h || !dweights)) return DRGG_EINVAL;
    if (!aligned16(dh) || !aligned(codes, 8) || !aligned16(dGU) || !aligned16(h) || !aligned(scale, 4) ||
        !aligned(positions, 4) || !aligned(weights, 4) || !aligned(dweights, 4))
        return DRGG_EALIGN;
    if (T == 0) return DRGG_OK;
    return launch_status(launch_moe_gate_int8_grad(dh, codes, scale, positions, weights, T, k, I, dGU, h, dweights, stream));
}

}  // extern "C"
