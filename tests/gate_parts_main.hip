// The parts of a gate's gradient that residual_gates_kernel reads, on the host: over
// boundaries in order they are those that the rows' runs leave, over any other ones
// they lie among the runs + sequences parts that there are.
#include <stdio.h>
#include <stdlib.h>

#include "fpstok_residual.h"

using namespace fpstok;

int main() {
    int failures = 0;
    srand(7);
    for (int n = 0; n < 200000; ++n) {
        const int B = 1 + rand() % 6, rows = 1 + rand() % 60, most = 1 + rand() % 20;
        const bool in_order = n % 2 == 0;
        int cu[8];
        cu[0] = rand() % (rows + 1);
        for (int b = 1; b <= B; ++b)
            cu[b] = in_order ? cu[b - 1] + rand() % (rows - cu[b - 1] + 1) : rand() % (rows + 1);
        const int runs = most < rows ? most : rows;
        const int64_t first = cu[0], last = cu[B];
        const int live = last > first ? (int)(last - first) : 0;
        const int per = live > 0 ? (live + runs - 1) / runs : 1;
        for (int b = 0; b < B; ++b) {
            const int len = cu[b + 1] > cu[b] ? cu[b + 1] - cu[b] : 0;
            const GateParts p = gate_parts(cu[b], len, first, last, per, b);
            if (p.n < 0 || (p.n > 0 && (p.first < 0 || p.first + p.n > runs + B))) {
                printf("sequence %d of %d: parts %lld + %d of %d\n", b, B, (long long)p.first, p.n,
                       runs + B);
                ++failures;
            }
            if (!in_order) continue;
            if ((len > 0) != (p.n > 0)) ++failures;
            if (len > 0 && (p.first != (cu[b] - first) / per + b ||
                            p.first + p.n - 1 != (cu[b + 1] - 1 - first) / per + b))
                ++failures;
        }
    }
    printf("%d failures\nparts ok\n", failures);
    return failures != 0;
}
