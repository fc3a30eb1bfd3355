// Drives the walk over the plane of entries (EntryWalk) on the host, block after
// block as the attention kernels ask for them, over the last row of a plane whose end
// is the end of mapped memory: a load past it ends the program.  Every block with
// keys in the sequence has to get its own entries.
#include <stdio.h>
#include <string.h>
#include <sys/mman.h>
#include <unistd.h>

#include "fpstok_attention_kernels.h"

using namespace fpstok;

static int failures = 0;

static void walk(const uint32_t* row, int tk, int first, int BN, int NB, int half) {
    EntryWalk w;
    w.row = row + half * 4;
    w.last = (tk - 1) & ~31;
    w.begin(true, first);
    for (int j0 = first; j0 < tk; j0 += BN)
        for (int b = 0; b < BN; b += 32 * NB) {
            if (j0 + b >= tk) continue;  // no row sees a key of it
            for (int k = 0; k < NB; ++k) {
                const int j = j0 + b + 32 * k;
                const u32x16 x = w.planed_block(j, j + 32);
                if (j >= tk) continue;
                for (int e = 0; e < 16; ++e)
                    if (x[e] != (uint32_t)(j + half * 4 + (e >> 2) * 8 + (e & 3))) ++failures;
            }
        }
}

int main() {
    const size_t page = (size_t)sysconf(_SC_PAGESIZE);
    char* at = (char*)mmap(nullptr, 2 * page, PROT_READ | PROT_WRITE, MAP_PRIVATE | MAP_ANONYMOUS,
                           -1, 0);
    if (at == (char*)MAP_FAILED || mprotect(at + page, page, PROT_NONE) != 0) return 2;
    for (int tk = 1; tk <= 320; ++tk) {
        const int pitch = (tk + 31) & ~31;
        uint32_t* row = (uint32_t*)(at + page) - pitch;
        for (int j = 0; j < pitch; ++j) row[j] = (uint32_t)j;
        for (int half = 0; half < 2; ++half)
            for (int first = 0; first < tk; first += 64) {
                printf("tk %d, from %d\n", tk, first);
                fflush(stdout);
                walk(row, tk, first, 32, 1, half);
                walk(row, tk, first, 64, 1, half);
                walk(row, tk, first, 64, 2, half);
            }
    }
    printf("%d failures\nwalks ok\n", failures);
    return failures != 0;
}
