// Reads lines "mode P E N K" (mode 0, 1, 2: y, dx, dw) and prints for each the kernel that
// matmul_rule.h picks.
#include <stdio.h>

#include "matmul_rule.h"

int main() {
    static const char* const names[] = {"stream",      "split32", "tile64_parts", "tile64",
                                        "tile128_deep", "tile128", "tile256"};
    moe::MatmulSizes a;
    long long P, E, N, K;
    while (scanf("%d %lld %lld %lld %lld", &a.mode, &P, &E, &N, &K) == 5) {
        a.P = P;
        a.E = E;
        a.N = N;
        a.K = K;
        printf("%s\n", names[static_cast<int>(moe::choose_matmul(a))]);
    }
    return 0;
}
