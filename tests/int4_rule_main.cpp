// Reads lines "P E N" and prints for each the shape that int4_rule.h picks; with an argument, all shapes' names.
#include <stdio.h>

#include "int4_rule.h"

int main(int argc, char**) {
    static const char* const names[] = {"few_wide", "few", "rows16", "rows32", "rows64", "tile64", "tile128"};
    if (argc > 1) {
        for (const char* n : names) printf("%s\n", n);
        return 0;
    }
    long long P, E, N;
    while (scanf("%lld %lld %lld", &P, &E, &N) == 3) printf("%s\n", names[static_cast<int>(moe::choose_int4(P, E, N))]);
    return 0;
}
