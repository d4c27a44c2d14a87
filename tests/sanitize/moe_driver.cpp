// Sanitizer driver for the host code of the expert-layer entry points
// (api_moe.cpp, built with g++ -fsanitize=address,undefined by
// tests/test_sanitize_moe.py; test infrastructure only).  The kernel launchers
// and the device queries are stubs: the launchers of the serving block record
// the buffers they are given, and the driver checks that no two buffers that
// are alive at once overlap and that all lie inside the workspace.  Also the
// tile rule of the 8-bit product.  Prints "ok" and returns 0 when all holds.
#include <cstdio>
#include <cstdlib>
#include <vector>

#include "drgg.h"
#include "internal.hpp"
#include "plan.hpp"

static int fails = 0;
static void fail(const char* what, int line) {
    std::fprintf(stderr, "line %d: %s\n", line, what);
    ++fails;
}
#define EXPECT(cond)                       \
    do {                                   \
        if (!(cond)) fail(#cond, __LINE__); \
    } while (0)

struct Span {
    const char* lo;
    const char* hi;
    Span(const void* p, int64_t n) : lo(static_cast<const char*>(p)), hi(lo + n) {}
    bool apart(const Span& o) const { return hi <= o.lo || o.hi <= lo; }
};
static std::vector<Span> routed;          // written by the selection, read to the end
static std::vector<const char*> steps;
static const char* ws_lo;
static const char* ws_hi;
static bool inside(const Span& s) { return s.lo >= ws_lo && s.hi <= ws_hi; }
static void apart_from_routed(const Span& s) {
    EXPECT(inside(s));
    for (const Span& r : routed) EXPECT(s.apart(r));
}
static Span codes(nullptr, 0), scales(nullptr, 0), hidden(nullptr, 0), hcodes(nullptr, 0), hscales(nullptr, 0),
    result(nullptr, 0);
static bool gathers;

namespace drgg {
drgg_status device_error(hipError_t) { return DRGG_EDEVICE; }
int knob_tile() { return 0; }
drgg_status current_cu_count(int* cus) {
    *cus = 256;
    return DRGG_OK;
}
bool checks_offsets() { return false; }
drgg_status check_offsets_sync(const int32_t*, int32_t, int64_t, hipStream_t) { return DRGG_OK; }
size_t route_table_bytes(int64_t T, int32_t E) { return T > 64 ? (size_t)(T / 64 + 2) * (size_t)E * 4 : 0; }
hipError_t launch_moe_route(const float*, int64_t T, int32_t E, int32_t k, int, int32_t* experts, float* weights,
                            int32_t* offsets, int32_t* positions, int32_t* tokens, void* table, hipStream_t,
                            const QuantArgs* quantize) {
    steps.push_back("route");
    const int64_t R = T * k;
    routed = {{experts, R * 4}, {weights, R * 4}, {offsets, (E + 1) * 4}, {positions, R * 4}};
    gathers = tokens != nullptr;
    if (tokens) routed.push_back({tokens, R * 4});
    if (route_table_bytes(T, E)) routed.push_back({table, (int64_t)route_table_bytes(T, E)});
    for (size_t i = 0; i < routed.size(); ++i) {
        EXPECT(inside(routed[i]));
        for (size_t j = 0; j < i; ++j) EXPECT(routed[i].apart(routed[j]));
    }
    if (quantize) {
        EXPECT(gathers && quantize->k == 1 && !quantize->positions && quantize->T == T);
        codes = Span(quantize->q, T * quantize->C * 16);
        scales = Span(quantize->scale, T * 4);
        apart_from_routed(codes);
        apart_from_routed(scales);
        EXPECT(codes.apart(scales));
    }
    return hipSuccess;
}
hipError_t launch_moe_route_grad(const float*, const float*, const int32_t*, const float*, int64_t, int32_t, int32_t,
                                 int, float*, hipStream_t) { return hipSuccess; }
hipError_t launch_moe_dispatch(const void*, const int32_t*, int64_t, int32_t, int64_t, bool, void*, hipStream_t) {
    return hipSuccess;
}
hipError_t launch_moe_combine(const void* rows, const int32_t*, const float*, int64_t, int32_t, int64_t, bool, void*,
                              hipStream_t) {
    steps.push_back("combine");
    EXPECT(rows == result.lo || result.lo == nullptr);
    return hipSuccess;
}
hipError_t launch_moe_combine_grad(const void*, const void*, const int32_t*, const float*, int64_t, int32_t, int64_t,
                                   bool, void*, float*, hipStream_t) { return hipSuccess; }
hipError_t launch_quantize_int8(const void* X, bool bf16, int64_t T, int64_t K, const int32_t* positions, int32_t k,
                                int8_t* q, float* scale, hipStream_t) {
    steps.push_back("quantize");
    const Span c(q, T * k * K), s(scale, T * k * 4);
    if (!ws_lo) return hipSuccess;
    apart_from_routed(c);
    apart_from_routed(s);
    EXPECT(c.apart(s));
    if (bf16) {
        EXPECT((positions == nullptr) == gathers);
        codes = c;
        scales = s;
    } else {   // the activation, still needed while its codes are written
        EXPECT(X == hidden.lo && c.apart(hidden) && s.apart(hidden));
        hcodes = c;
        hscales = s;
    }
    return hipSuccess;
}
hipError_t launch_int8(const Int8Args& a, bool gated, bool bf16, int, int, hipStream_t) {
    steps.push_back(gated ? "gated" : "product");
    if (!ws_lo) return hipSuccess;
    if (gated) {
        EXPECT(!bf16 && (const char*)a.X == codes.lo && (const char*)a.xs == scales.lo);
        EXPECT((a.rows != nullptr) == gathers);
        hidden = Span(a.out, a.M * (a.N / 2) * 4);
        apart_from_routed(hidden);
        EXPECT(hidden.apart(codes) && hidden.apart(scales));
    } else {
        EXPECT(bf16 && (const char*)a.X == hcodes.lo && (const char*)a.xs == hscales.lo && !a.rows);
        result = Span(a.out, a.M * a.N * 2);
        apart_from_routed(result);
        EXPECT(result.apart(hcodes) && result.apart(hscales));
    }
    return hipSuccess;
}
}  // namespace drgg

int main() {
    using namespace drgg;
    char* const A = reinterpret_cast<char*>(0x100000);   // fake, aligned, never dereferenced
    auto* f = reinterpret_cast<float*>(A);
    auto* b = reinterpret_cast<int8_t*>(A);
    const int64_t cases[][5] = {{1, 8, 2, 16, 16}, {63, 57, 7, 1776, 528}, {65, 1024, 64, 48, 16},
                                {16384, 32, 8, 2048, 768}, {16500, 2, 1, 131056, 16}, {33, 4, 4, 16, 4096},
                                {100000, 3, 3, 32768, 32}, {70, 8, 2, 4112, 48}, {70, 8, 2, 4096, 48}};
    for (const auto& c : cases) {
        size_t need = 0;
        EXPECT(moe_ffn_int8_workspace_size(c[0], (int32_t)c[1], (int32_t)c[2], c[3], c[4], &need) == DRGG_OK);
        ws_lo = reinterpret_cast<char*>(int64_t(1) << 40);
        ws_hi = ws_lo + need;
        steps.clear();
        result = Span(nullptr, 0);
        EXPECT(moe_ffn_int8(A, f, b, f, b, f, c[0], (int32_t)c[1], (int32_t)c[2], c[3], c[4], 1, A,
                            const_cast<char*>(ws_lo), need, nullptr) == DRGG_OK);
        const bool together = c[3] <= kSelectQuantizeK && c[0] * c[3] <= kSelectQuantizeMost;
        EXPECT(steps.size() == (together ? 5 : 6));
        EXPECT(gathers == (c[0] * c[3] <= INT32_MAX - 4096));
        EXPECT(moe_ffn_int8(A, f, b, f, b, f, c[0], (int32_t)c[1], (int32_t)c[2], c[3], c[4], 1, A,
                            const_cast<char*>(ws_lo), need - 1, nullptr) == DRGG_EWORKSPACE);
    }
    size_t n;
    EXPECT(moe_ffn_int8_workspace_size(int64_t(1) << 26, 64, 32, 64, 64, &n) == DRGG_ESHAPE);
    EXPECT(moe_ffn_int8_workspace_size(4, 8, 2, 64, 64, nullptr) == DRGG_EINVAL);
    EXPECT(moe_route_workspace_size(4, 8, 2, nullptr) == DRGG_EINVAL);
    // the single calls reach their launchers with valid arguments
    ws_lo = nullptr;
    auto* o = reinterpret_cast<int32_t*>(A);
    EXPECT(grouped_gemm_int8(b, f, b, f, o, nullptr, 0, 2, 100, 64, 64, 0, DRGG_BF16, A, nullptr) == DRGG_OK);
    EXPECT(gemm_int8(b, f, b, f, 100, 64, 131056, 1, DRGG_FP32, A, nullptr) == DRGG_OK);
    EXPECT(quantize_int8(A, DRGG_FP32, 3, 64, nullptr, 1, b, f, nullptr) == DRGG_OK);
    // the tile rule: one group, exact counts
    EXPECT(int8_tile(1, 16384, 4096, 16, 32, true) == kTile256x256);
    EXPECT(int8_tile(1, 2048, 4096, 16, 32, true) == kTile128x256);
    EXPECT(int8_tile(1, 6559, 976, 10, 20, true) == kTile128x128);
    EXPECT(int8_tile(1, 6559, 976, 10, 20, false) != kTile128x128);
    EXPECT(int8_tile(8, 131072, 2048, 6, 12, true) == kTile256x256);
    for (int64_t e = 1; e <= 1024; e *= 4)
        for (int64_t m = 1; m < (int64_t(1) << 31); m *= 7)
            for (int64_t k = 16; k <= kInt8MaxK; k *= 3) {
                const int t = int8_tile(e, m, k, 16384, 32768, false);
                EXPECT(t == kTile256x256 || t == kTile128x256);
            }
    if (fails) return 1;
    std::printf("ok\n");
    return 0;
}
