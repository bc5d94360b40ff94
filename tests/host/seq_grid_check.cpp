// The grids of the sequence operators' launches (csrc/lores_seq.h): every number
// of work-groups that the entry points allow becomes a grid that a launch takes,
// and every work-group has one place in it.
#include <cstdio>

#include "../../quantized_linear_recurrence_amd/csrc/lores_seq.h"

int main() {
    int bad = 0;
    const int64_t most = (int64_t)0x7fffffff;
    for (int s = 0; s <= 31; ++s)
        for (int64_t o = -3; o <= 3; ++o) {
            const int64_t n = ((int64_t)1 << s) + o;
            if (n < 1 || n > most) continue;
            const dim3 g = lores::grid_of(n);
            const int64_t all = (int64_t)g.x * g.y;
            // 1024 threads at most; y counts work-groups of one row each
            const bool fits = (int64_t)g.x * 1024 < ((int64_t)1 << 32) && g.y <= 65535 && g.z == 1;
            const bool covers = all >= n && all - n < g.x;
            // rows follow each other without a gap
            bool order = lores::block_at(0, 0) == 0 && lores::block_at(g.x - 1, g.y - 1) == all - 1;
            if (g.y > 1) order = order && lores::block_at(0, 1) == (int64_t)g.x && g.x % 8 == 0;
            if (!(fits && covers && order)) {
                std::printf("%lld work-groups: grid %u x %u\n", (long long)n, g.x, g.y);
                ++bad;
            }
        }
    if (!bad) std::printf("grids ok\n");
    return bad ? 1 : 0;
}
