// Sanitizer driver for the host code of the scored selection, the 4-bit products
// and the kept activation (api_experts.cpp, built with g++
// -fsanitize=address,undefined by tests/test_host_experts.py; test
// infrastructure only).  The kernel launchers are stubs that record the buffers
// the serving block gives them; the driver checks that no two buffers that are
// alive at once overlap and that all lie inside the workspace.  Prints "ok" and
// returns 0 when all holds.
#include <cstdio>
#include <vector>

#include "drgg.h"
#include "internal.hpp"
#include "plan.hpp"

static int fails = 0;
#define EXPECT(cond)                                                   \
    do {                                                               \
        if (!(cond)) {                                                 \
            std::fprintf(stderr, "line %d: %s\n", __LINE__, #cond);    \
            ++fails;                                                   \
        }                                                              \
    } while (0)

struct Span {
    const char* lo;
    const char* hi;
    Span() : lo(nullptr), hi(nullptr) {}
    Span(const void* p, int64_t n) : lo(static_cast<const char*>(p)), hi(lo + n) {}
    bool apart(const Span& o) const { return hi <= o.lo || o.hi <= lo; }
};
static const char* ws_lo;
static const char* ws_hi;
static std::vector<Span> routed;   // written by the selection, read to the end
static std::vector<Span> alive;    // the block's rows that a later step still reads
static Span x, xs, hq, hs, y;
static int step;
static bool scored;
static void fresh(const Span& s) {
    EXPECT(s.lo >= ws_lo && s.hi <= ws_hi);
    for (const Span& r : routed) EXPECT(s.apart(r));
    for (const Span& r : alive) EXPECT(s.apart(r));
}
static int64_t scale_bytes(int64_t rows, int64_t K) { return (K + 255) / 256 * rows * 8; }

namespace drgg {
drgg_status device_error(hipError_t) { return DRGG_EDEVICE; }
drgg_status current_cu_count(int* cus) {
    *cus = 256;
    return DRGG_OK;
}
int knob_tile() { return 0; }
bool checks_offsets() { return false; }
drgg_status check_offsets_sync(const int32_t*, int32_t, int64_t, hipStream_t) { return DRGG_OK; }
size_t route_table_bytes(int64_t T, int32_t E) { return T > 64 ? (size_t)(T / 64 + 2) * (size_t)E * 4 : 0; }

static hipError_t route(int64_t T, int32_t E, int32_t k, int32_t* experts, float* weights, int32_t* offsets,
                        int32_t* positions, int32_t* tokens, void* table, bool by_scores) {
    EXPECT(step++ == 0 && by_scores == scored);
    const int64_t R = T * k;
    routed.clear();
    alive.clear();
    for (const Span& s : {Span(experts, R * 4), Span(weights, R * 4), Span(offsets, ((int64_t)E + 1) * 4), Span(positions, R * 4),
                          Span(tokens, R * 4), Span(table, (int64_t)route_table_bytes(T, E))}) {
        fresh(s);
        routed.push_back(s);
    }
    return hipSuccess;
}
hipError_t launch_moe_route(const float*, int64_t T, int32_t E, int32_t k, int renormalize, int32_t* experts, float* weights,
                            int32_t* offsets, int32_t* positions, int32_t* tokens, void* table, hipStream_t,
                            const QuantArgs* quantize) {
    EXPECT(renormalize == 1 && !quantize);
    return route(T, E, k, experts, weights, offsets, positions, tokens, table, false);
}
hipError_t launch_moe_route_scores(const float*, int64_t T, int32_t E, int32_t k, const drgg_scoring&, int32_t* experts,
                                   float* weights, int32_t* offsets, int32_t* positions, int32_t* tokens, void* table,
                                   hipStream_t, const MxQuantArgs* quantize) {
    route(T, E, k, experts, weights, offsets, positions, tokens, table, true);
    if (quantize) launch_quantize_mxfp4(quantize->X, true, quantize->T, quantize->K, quantize->codes, quantize->scales, nullptr);
    return hipSuccess;
}
hipError_t launch_moe_route_scores_grad(const float*, const float*, const int32_t*, const float*, int64_t, int32_t, int32_t,
                                        const drgg_scoring&, float*, hipStream_t) { return hipSuccess; }
hipError_t launch_quantize_mxfp4(const void* X, bool bf16, int64_t T, int64_t K, uint8_t* codes, uint8_t* scales,
                                 hipStream_t) {
    const Span c(codes, T * K / 2), s(scales, scale_bytes(T, K));
    fresh(c);
    EXPECT(c.apart(s));
    fresh(s);
    EXPECT(step++ == 1 && bf16);
    x = c;
    xs = s;
    alive = {x, xs};
    return hipSuccess;
}
hipError_t launch_dequantize_mxfp4(const uint8_t*, const uint8_t*, int64_t, int64_t, bool, void*, hipStream_t) {
    return hipSuccess;
}
hipError_t launch_mxfp4(const MxArgs& a, bool gated, bool bf16, int, int, hipStream_t) {
    if (gated) {
        EXPECT(step++ == 2 && !bf16 && a.rows && a.out_scales);
        EXPECT((const char*)a.X == x.lo && (const char*)a.xs == xs.lo);
        hq = Span(a.out, a.M * (a.N / 4));
        fresh(hq);
        hs = Span(a.out_scales, scale_bytes(a.M, a.N / 2));
        fresh(hs);
        EXPECT(hq.apart(hs));
        alive = {hq, hs};
    } else {
        EXPECT(step++ == 3 && bf16 && !a.rows && !a.out_scales);
        EXPECT((const char*)a.X == hq.lo && (const char*)a.xs == hs.lo);
        y = Span(a.out, a.M * a.N * 2);
        fresh(y);
        alive = {y};
    }
    return hipSuccess;
}
hipError_t launch_moe_combine(const void* rows, const int32_t*, const float*, int64_t, int32_t, int64_t, bool bf16, void*,
                              hipStream_t) {
    EXPECT(step++ == 4 && bf16 && rows == y.lo);
    return hipSuccess;
}
hipError_t launch_moe_gate_int8(const void*, const int32_t*, const float*, int64_t, int32_t, int64_t, void*, int8_t*, float*,
                                hipStream_t) { return hipSuccess; }
hipError_t launch_moe_gate_int8_grad(const void*, const int8_t*, const float*, const int32_t*, const float*, int64_t, int32_t,
                                     int64_t, void*, void*, float*, hipStream_t) { return hipSuccess; }
}  // namespace drgg

int main() {
    char* const A = reinterpret_cast<char*>(0x100000);   // fake, aligned, never dereferenced
    auto* f = reinterpret_cast<float*>(A);
    auto* b = reinterpret_cast<uint8_t*>(A);
    drgg_scoring c{DRGG_SCORE_SIGMOID, 1, 1, 2, 1, 1.f, f};
    const int64_t cases[][5] = {{1, 8, 2, 32, 32}, {63, 57, 7, 1792, 544}, {65, 1024, 64, 64, 32}, {16384, 32, 8, 2048, 768},
                                {1000, 2, 1, 4194304, 32}, {33, 4, 4, 32, 2097152}, {100000, 3, 3, 32768, 32},
                                {1000000, 64, 8, 4064, 96}};
    for (const auto& v : cases)
        for (const bool by : {false, true}) {
            size_t need = 0;
            EXPECT(moe_ffn_mxfp4_workspace_size(v[0], (int32_t)v[1], (int32_t)v[2], v[3], v[4], &need) == DRGG_OK);
            ws_lo = reinterpret_cast<char*>(int64_t(1) << 44);
            ws_hi = ws_lo + need;
            step = 0;
            scored = by;
            EXPECT(moe_ffn_mxfp4(A, f, b, b, b, b, v[0], (int32_t)v[1], (int32_t)v[2], v[3], v[4], by ? &c : nullptr, A,
                                 const_cast<char*>(ws_lo), need, nullptr) == DRGG_OK);
            EXPECT(step == 5);
            EXPECT(moe_ffn_mxfp4(A, f, b, b, b, b, v[0], (int32_t)v[1], (int32_t)v[2], v[3], v[4], by ? &c : nullptr, A,
                                 const_cast<char*>(ws_lo), need - 1, nullptr) == DRGG_EWORKSPACE);
        }
    size_t need = 0;
    EXPECT(moe_ffn_mxfp4_workspace_size(int64_t(1) << 27, 1024, 1, 4194304, 2097152, &need) == DRGG_ESHAPE);
    EXPECT(moe_ffn_mxfp4_workspace_size((int64_t(1) << 63) - 1, 1024, 1, 4194304, 2097152, &need) == DRGG_ESHAPE);
    if (fails == 0) std::puts("ok");
    return fails ? 1 : 0;
}
