// The search for a row's sequence among the packed sequences' bounds, up to the most
// sequences that a call takes.
#include <stdio.h>
#include <stdlib.h>

#include "../../gated_delta_rule_24_amd/csrc/gdr_attn.h"

static int fail(const char* what, int got, int want) {
    printf("%s: got %d, want %d\n", what, got, want);
    return 1;
}

int main() {
    const int small[] = {0, 3, 3, 7, 12}, want[] = {0, 0, 0, 2, 2, 2, 2, 3, 3, 3, 3, 3, 4, 4};
    for (int t = 0; t < 14; ++t) {
        const int got = gdr::last_at_most(small, 4, t);
        if (got != want[t]) return fail("small", got, want[t]);
    }
    for (int n = 1; n <= 200; ++n) {                  // every length: bounds i / 2
        int cu[201];
        for (int i = 0; i <= n; ++i) cu[i] = i / 2;
        for (int t = 0; t <= n / 2; ++t) {
            const int last = 2 * t + 1 <= n ? 2 * t + 1 : n, got = gdr::last_at_most(cu, n, t);
            if (got != last) return fail("lengths", got, last);
        }
    }
    const int most = 1 << 30;                         // all empty but the last; never written, so mostly not there
    int* cu = static_cast<int*>(calloc((size_t)most + 1, sizeof(int)));
    if (!cu) { printf("skipped: no memory\n"); return 0; }
    cu[most] = 100;
    const int got = gdr::last_at_most(cu, most, 50), end = gdr::last_at_most(cu, most, 100);
    free(cu);
    if (got != most - 1) return fail("most sequences", got, most - 1);
    if (end != most) return fail("behind the last", end, most);
    printf("ok\n");
    return 0;
}
