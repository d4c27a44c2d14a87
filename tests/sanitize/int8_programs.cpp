// Which program an 8-bit product runs in (plan.hpp), built with g++ by
// tests/test_int8_programs.py: reads "E M N K gated bf16" lines and prints
// "tile nb waves tok" for each.
#include <cstdio>

#include "plan.hpp"

int main() {
    long long E, M, N, K;
    int gated, bf16;
    while (std::scanf("%lld %lld %lld %lld %d %d", &E, &M, &N, &K, &gated, &bf16) == 6) {
        const drgg::Int8Program p = drgg::int8_program(E, M, N, K, gated != 0, bf16 != 0, 0);
        std::printf("%d %d %d %d\n", p.tile, p.nb, p.waves, p.tok);
    }
    return 0;
}
