// Reads lines "P E N K group" and prints for each the shape that int4_rule.h picks; with an argument, all shapes' names.
#include <stdio.h>

#include "int4_rule.h"

int main(int argc, char**) {
    char names[static_cast<int>(moe::Int4Shape::kCount)][32];
    for (int i = 0; i < static_cast<int>(moe::Int4Shape::kCount); ++i) {
        const moe::Int4Cost& c = moe::kInt4Costs[i];
        int n = snprintf(names[i], sizeof(names[i]), "%dx%d", c.rows, c.cols);
        if (c.parts > 1) snprintf(names[i] + n, sizeof(names[i]) - n, "p%d", c.parts);
    }
    if (argc > 1) {
        for (const auto& n : names) printf("%s\n", n);
        return 0;
    }
    long long P, E, N, K;
    int group;
    while (scanf("%lld %lld %lld %lld %d", &P, &E, &N, &K, &group) == 5)
        printf("%s\n", names[static_cast<int>(moe::choose_int4(P, E, N, K, group))]);
    return 0;
}
