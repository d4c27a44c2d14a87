// Driver for the 32-bit counts that the kernels share with the host
// (plan.hpp), built with g++ -fsanitize=address,undefined by
// tests/test_counts.py: the numbers of tiles and chunks of the longest groups.
// Prints "ok" and returns 0 when all holds.
#include <cstdio>

#include "plan.hpp"

int main() {
    int fails = 0;
    const int32_t most = INT32_MAX;
    const int32_t counts[] = {0, 1, 2, 63, 64, 127, 128, 129, 255, 256, 257, 1 << 30, (1 << 30) + 1, most - 256,
                              most - 255, most - 254, most - 127, most - 1, most};
    const int32_t lengths[] = {1, 2, 3, 64, 128, 192, 256, 512, 1 << 23, (1 << 30) + 64, most - 63, most};
    for (int32_t t : counts)
        for (int32_t n : lengths) {
            const int64_t want = drgg::ceil_div(t, n);
            if (drgg::ceil_div32(t, n) != want) {
                std::fprintf(stderr, "ceil(%d / %d): %d, expected %lld\n", t, n, drgg::ceil_div32(t, n), (long long)want);
                ++fails;
            }
        }
    if (fails) return 1;
    std::puts("ok");
    return 0;
}
