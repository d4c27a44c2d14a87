// api_moe.cpp -- the C ABI of the operators around the grouped products
// (declared in include/drgg.h): the router's selection, the movement of rows,
// and the 8-bit integer products.  Argument checks in checked 64-bit
// arithmetic, then launches (moe.hip, int8.hip) on the caller's stream.
#include <hip/hip_runtime.h>

#include <cstdint>

#include "../../include/drgg.h"
#include "internal.hpp"
#include "plan.hpp"

namespace drgg {
namespace {

bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }
// rows of E logits are read and written four at a time where all of them start aligned
bool aligned_logits(const void* p, int32_t E) { return E % 4 ? aligned4(p) : aligned16(p); }

drgg_status check_pairs(int64_t T, int32_t k) {
    int64_t r;
    if (k < 1 || k > 64) return DRGG_EINVAL;
    if (T < 0 || !mul_ok(T, k, &r) || r > INT32_MAX) return DRGG_ESHAPE;
    return DRGG_OK;
}

drgg_status check_route(int64_t T, int32_t E, int32_t k) {
    if (E < 1 || E > kMaxExperts || k > E) return DRGG_EINVAL;
    if (T > (int64_t(1) << 27)) return DRGG_ESHAPE;   // 16 threads per token in one launch
    return check_pairs(T, k);
}

drgg_status check_rows(int64_t T, int32_t k, int64_t H, drgg_dtype dt) {
    if (dt != DRGG_BF16 && dt != DRGG_FP32) return DRGG_EINVAL;
    drgg_status st = check_pairs(T, k);
    if (st != DRGG_OK) return st;
    if (H < 8 || H > (1 << 22)) return DRGG_ESHAPE;
    return H % 8 ? DRGG_EALIGN : DRGG_OK;
}

// whether T rows of K codes can be gathered: their offsets are 32 bits wide
bool can_gather(int64_t T, int64_t K) { return T * K <= INT32_MAX - 4096; }

drgg_status run_int8(const int8_t* Xq, const float* x_scale, const int8_t* Wq, const float* w_scale,
                     const int32_t* offs, const int32_t* rows, int64_t T, int32_t E, int64_t M, int64_t N, int64_t K,
                     int gated, drgg_dtype dt, void* Y, hipStream_t s) {
    if (E < 1 || E > kMaxExperts) return DRGG_EINVAL;
    if (dt != DRGG_BF16 && dt != DRGG_FP32) return DRGG_EINVAL;
    const int64_t na = gated ? 16 : 8;
    if (M < 0 || M > INT32_MAX || N < na || N > (1 << 22) || K < 16 || K > kInt8MaxK) return DRGG_ESHAPE;
    if (N % na || K % 16) return DRGG_EALIGN;
    if (rows && (T < 1 || T > INT32_MAX || !can_gather(T, K))) return DRGG_ESHAPE;
    if (!Wq || !w_scale || (M > 0 && (!Xq || !x_scale || !Y))) return DRGG_EINVAL;
    if (!aligned16(Xq) || !aligned16(Wq) || !aligned16(Y) || !aligned16(w_scale) || !aligned4(x_scale) ||
        !aligned4(offs) || !aligned4(rows))
        return DRGG_EALIGN;
    if (offs && checks_offsets()) {
        drgg_status st = check_offsets_sync(offs, E, M, s);
        if (st != DRGG_OK) return st;
    }
    if (M == 0) return DRGG_OK;
    int cus = 0;
    drgg_status st = current_cu_count(&cus);
    if (st != DRGG_OK) return st;
    Int8Args a{Xq, Wq, x_scale, w_scale, offs, Y, M, N, K, E, rows, T};
    return launch_status(launch_int8(a, gated != 0, dt == DRGG_BF16, cus, knob_tile(), s));
}

// The parts of moe_ffn_int8's workspace (byte offsets, multiples of 256).  The
// experts' outputs y take the place of the codes of X and the activation,
// which are no longer needed by then.  X is quantised once per token and its
// rows gathered by the first product, or, where they are too many for that,
// written k times into the grouped order.
struct FfnLayout {
    int64_t experts, weights, offsets, positions, tokens, table, xs, hs, hq, x, h, y, bytes;
    bool gather;
};
drgg_status ffn_layout(int64_t T, int32_t E, int32_t k, int64_t H, int64_t I, FfnLayout* L) {
    drgg_status st = check_route(T, E, k);
    if (st != DRGG_OK) return st;
    if (H < 16 || H > kInt8MaxK || I < 16 || I > kInt8MaxK) return DRGG_ESHAPE;
    if (H % 16 || I % 16) return DRGG_EALIGN;
    const int64_t R = T * k;   // below 2^31; a row of any part is below 2^20 bytes
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
    L->xs = part(R * 4);
    L->hs = part(R * 4);
    L->hq = part(R * I);
    L->gather = can_gather(T, H);
    const int64_t x = round_up((L->gather ? T : R) * H, 256);
    L->x = L->y = at;
    L->h = at + x;
    const int64_t both = x + round_up(R * I * 4, 256), y = round_up(R * H * 2, 256);
    L->bytes = at + (both > y ? both : y);
    return DRGG_OK;
}

}  // namespace
}  // namespace drgg

using namespace drgg;

extern "C" {

drgg_status moe_route_workspace_size(int64_t T, int32_t E, int32_t k, size_t* bytes) {
    if (!bytes) return DRGG_EINVAL;
    drgg_status st = check_route(T, E, k);
    if (st != DRGG_OK) return st;
    *bytes = route_table_bytes(T, E);
    return DRGG_OK;
}

drgg_status moe_route(const float* logits, int64_t T, int32_t E, int32_t k, int renormalize, int32_t* experts,
                      float* weights, int32_t* group_offsets, int32_t* positions, int32_t* tokens, void* workspace,
                      size_t workspace_bytes, hipStream_t stream) {
    drgg_status st = check_route(T, E, k);
    if (st != DRGG_OK) return st;
    if (!group_offsets || (T > 0 && (!logits || !experts || !weights || !positions))) return DRGG_EINVAL;
    if (!aligned_logits(logits, E) || !aligned4(experts) || !aligned4(weights) || !aligned4(group_offsets) ||
        !aligned4(positions) || !aligned4(tokens))
        return DRGG_EALIGN;
    const size_t need = route_table_bytes(T, E);
    if (need > 0) {
        if (!workspace || workspace_bytes < need) return DRGG_EWORKSPACE;
        if (!aligned16(workspace)) return DRGG_EALIGN;
    }
    return launch_status(launch_moe_route(logits, T, E, k, renormalize != 0, experts, weights, group_offsets, positions,
                                          tokens, workspace, stream));
}

drgg_status moe_route_grad(const float* dweights, const float* logits, const int32_t* experts, const float* weights,
                           int64_t T, int32_t E, int32_t k, int renormalize, float* dlogits, hipStream_t stream) {
    drgg_status st = check_route(T, E, k);
    if (st != DRGG_OK) return st;
    if (T > 0 && (!dweights || !logits || !experts || !weights || !dlogits)) return DRGG_EINVAL;
    if (!aligned_logits(logits, E) || !aligned_logits(dlogits, E) || !aligned4(dweights) || !aligned4(experts) || !aligned4(weights))
        return DRGG_EALIGN;
    if (T == 0) return DRGG_OK;
    return launch_status(
        launch_moe_route_grad(dweights, logits, experts, weights, T, E, k, renormalize != 0, dlogits, stream));
}

drgg_status moe_dispatch(const void* X, const int32_t* positions, int64_t T, int32_t k, int64_t H, drgg_dtype dtype,
                         void* rows, hipStream_t stream) {
    drgg_status st = check_rows(T, k, H, dtype);
    if (st != DRGG_OK) return st;
    if (T > 0 && (!X || !positions || !rows)) return DRGG_EINVAL;
    if (!aligned16(X) || !aligned16(rows) || !aligned4(positions)) return DRGG_EALIGN;
    if (T == 0) return DRGG_OK;
    return launch_status(launch_moe_dispatch(X, positions, T, k, H, dtype == DRGG_BF16, rows, stream));
}

drgg_status moe_combine(const void* rows, const int32_t* positions, const float* weights, int64_t T, int32_t k,
                        int64_t H, drgg_dtype dtype, void* out, hipStream_t stream) {
    drgg_status st = check_rows(T, k, H, dtype);
    if (st != DRGG_OK) return st;
    if (T > 0 && (!rows || !positions || !out)) return DRGG_EINVAL;
    if (!aligned16(rows) || !aligned16(out) || !aligned4(positions) || !aligned4(weights)) return DRGG_EALIGN;
    if (T == 0) return DRGG_OK;
    return launch_status(launch_moe_combine(rows, positions, weights, T, k, H, dtype == DRGG_BF16, out, stream));
}

drgg_status moe_combine_grad(const void* dout, const void* rows, const int32_t* positions, const float* weights,
                             int64_t T, int32_t k, int64_t H, drgg_dtype dtype, void* drows, float* dweights,
                             hipStream_t stream) {
    drgg_status st = check_rows(T, k, H, dtype);
    if (st != DRGG_OK) return st;
    if (T > 0 && (!dout || !rows || !positions || !weights || !drows || !dweights)) return DRGG_EINVAL;
    if (!aligned16(dout) || !aligned16(rows) || !aligned16(drows) || !aligned4(positions) || !aligned4(weights) ||
        !aligned4(dweights))
        return DRGG_EALIGN;
    if (T == 0) return DRGG_OK;
    return launch_status(launch_moe_combine_grad(dout, rows, positions, weights, T, k, H, dtype == DRGG_BF16, drows,
                                                 dweights, stream));
}

drgg_status quantize_int8(const void* X, drgg_dtype dtype, int64_t T, int64_t K, const int32_t* positions, int32_t k,
                          int8_t* q, float* scale, hipStream_t stream) {
    if (dtype != DRGG_BF16 && dtype != DRGG_FP32) return DRGG_EINVAL;
    if (T > 0 && !positions && k != 1) return DRGG_EINVAL;
    drgg_status st = check_pairs(T, k);
    if (st != DRGG_OK) return st;
    if (K < 16 || K > (1 << 22)) return DRGG_ESHAPE;
    if (K % 16) return DRGG_EALIGN;
    if (T > 0 && (!X || !q || !scale)) return DRGG_EINVAL;
    if (!aligned16(X) || !aligned16(q) || !aligned4(scale) || !aligned4(positions)) return DRGG_EALIGN;
    if (T == 0) return DRGG_OK;
    return launch_status(launch_quantize_int8(X, dtype == DRGG_BF16, T, K, positions, k, q, scale, stream));
}

drgg_status grouped_gemm_int8(const int8_t* Xq, const float* x_scale, const int8_t* Wq, const float* w_scale,
                              const int32_t* group_offsets, const int32_t* rows, int64_t T, int32_t E, int64_t M,
                              int64_t N, int64_t K, int gated, drgg_dtype out_dtype, void* Y, hipStream_t stream) {
    if (!group_offsets) return DRGG_EINVAL;
    return run_int8(Xq, x_scale, Wq, w_scale, group_offsets, rows, T, E, M, N, K, gated, out_dtype, Y, stream);
}

drgg_status gemm_int8(const int8_t* Xq, const float* x_scale, const int8_t* Wq, const float* w_scale, int64_t M,
                      int64_t N, int64_t K, int gated, drgg_dtype out_dtype, void* Y, hipStream_t stream) {
    return run_int8(Xq, x_scale, Wq, w_scale, nullptr, nullptr, 0, 1, M, N, K, gated, out_dtype, Y, stream);
}

drgg_status moe_ffn_int8_workspace_size(int64_t T, int32_t E, int32_t k, int64_t H, int64_t I, size_t* bytes) {
    if (!bytes) return DRGG_EINVAL;
    FfnLayout L;
    drgg_status st = ffn_layout(T, E, k, H, I, &L);
    if (st != DRGG_OK) return st;
    *bytes = (size_t)L.bytes;
    return DRGG_OK;
}

drgg_status moe_ffn_int8(const void* X, const float* logits, const int8_t* W1q, const float* w1_scale,
                         const int8_t* W2q, const float* w2_scale, int64_t T, int32_t E, int32_t k, int64_t H,
                         int64_t I, int renormalize, void* out, void* workspace, size_t workspace_bytes,
                         hipStream_t stream) {
    FfnLayout L;
    drgg_status st = ffn_layout(T, E, k, H, I, &L);
    if (st != DRGG_OK) return st;
    if (!W1q || !w1_scale || !W2q || !w2_scale || (T > 0 && (!X || !logits || !out))) return DRGG_EINVAL;
    if (!aligned16(X) || !aligned_logits(logits, E) || !aligned16(W1q) || !aligned16(w1_scale) || !aligned16(W2q) ||
        !aligned16(w2_scale) || !aligned16(out))
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
    auto* xs = reinterpret_cast<float*>(ws + L.xs);
    auto* hs = reinterpret_cast<float*>(ws + L.hs);
    auto* hq = reinterpret_cast<int8_t*>(ws + L.hq);
    auto* x = reinterpret_cast<int8_t*>(ws + L.x);
    int cus = 0;
    st = current_cu_count(&cus);
    if (st != DRGG_OK) return st;
    const int64_t R = T * k;
    // the selection's launch quantises the rows too, where they are gathered,
    // fit it and are few: its workgroups of 1024 threads move rows more slowly
    // (16384 tokens of 2048: 36 us against 6 + 26), which a launch less
    // outweighs up to some thousand tokens (8 tokens: 5.3 us against 3.7 + 3.6)
    const QuantArgs rows{X, nullptr, x, xs, T, H / 16, 1};
    const bool together = L.gather && H <= kSelectQuantizeK && T * H <= kSelectQuantizeMost;
    hipError_t e = launch_moe_route(logits, T, E, k, renormalize != 0, experts, weights, offsets, positions,
                                    L.gather ? tokens : nullptr, ws + L.table, stream, together ? &rows : nullptr);
    if (e == hipSuccess && !together)
        e = launch_quantize_int8(X, true, T, H, L.gather ? nullptr : positions, L.gather ? 1 : k, x, xs, stream);
    if (e == hipSuccess)
        e = launch_int8(Int8Args{x, W1q, xs, w1_scale, offsets, ws + L.h, R, 2 * I, H, E, L.gather ? tokens : nullptr, T},
                        true, false, cus, knob_tile(), stream);
    if (e == hipSuccess) e = launch_quantize_int8(ws + L.h, false, R, I, nullptr, 1, hq, hs, stream);
    if (e == hipSuccess)
        e = launch_int8(Int8Args{hq, W2q, hs, w2_scale, offsets, ws + L.y, R, H, I, E}, false, true, cus, knob_tile(), stream);
    if (e == hipSuccess) e = launch_moe_combine(ws + L.y, positions, weights, T, k, H, true, out, stream);
    return launch_status(e);
}

}  // extern "C"
