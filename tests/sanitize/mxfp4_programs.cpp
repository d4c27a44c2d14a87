// Which program a 4-bit product runs in (plan.hpp), built with g++ by
// tests/test_mxfp4_programs.py: reads "E M N K gated bf16 codes tile" lines and
// prints "tile nb waves tok" for each.
#include <cstdio>

#include "plan.hpp"

int main() {
    long long E, M, N, K;
    int gated, bf16, codes, tile;
    while (std::scanf("%lld %lld %lld %lld %d %d %d %d", &E, &M, &N, &K, &gated, &bf16, &codes, &tile) == 8) {
        const drgg::Int8Program p = drgg::mxfp4_program(E, M, N, K, gated != 0, bf16 != 0, codes != 0, tile);
        std::printf("%d %d %d %d\n", p.tile, p.nb, p.waves, p.tok);
    }
    return 0;
}
