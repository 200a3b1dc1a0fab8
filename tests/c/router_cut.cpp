// Cuts rows of many shapes and says what is wrong with the first bad cut (tests/test_router_cut.py).
#include <initializer_list>

#include <stdio.h>

#include "fc_router_cut.h"

using namespace fc;

static int look(int64_t sequences, int64_t tokens, int64_t groups, int experts, int step, int row_bytes)
{
    const RouterShape n = {sequences, tokens, experts, 1, groups, false};
    const RouterCut c = router_cut(n, step, 4, step, 100, 300, [&](int warps, int rows) {
        return (size_t)warps * rows * row_bytes + 4 * experts;
    });
    const int64_t most = router_parts(sequences, tokens, groups);
    const char *wrong = nullptr;
    if (most < 1) wrong = "no parts";
    if (c.parts < 1 || c.parts > most) wrong = "parts";
    if (c.rows < step || c.rows > 32 || c.rows % step) wrong = "rows";
    if (c.warps < 1 || c.warps > FC_ROUTER_WARPS || FC_ROUTER_WARPS % c.warps) wrong = "warps";
    if (c.joins != (groups * c.parts <= FC_ROUTER_JOIN)) wrong = "joins";
    if (groups * c.parts > INT32_MAX) wrong = "grid";
    if (wrong)
        printf("%s: %lld x %lld in %lld groups, %d experts: %d parts of %lld, %d rows, %d warps\n",
               wrong, (long long)sequences, (long long)tokens, (long long)groups, experts, c.parts,
               (long long)most, c.rows, c.warps);
    return wrong != nullptr;
}

int main()
{
    const int64_t sizes[] = {0, 1, 2, 3, 7, 16, 31, 33, 64, 1000, 1216, 1217, 4096, 40001, 131072,
                             1 << 24, INT32_MAX};
    for (const int64_t sequences : sizes)
        for (const int64_t tokens : sizes)
            for (const int step : {1, 2, 8, 16, 32})
                for (const int row_bytes : {12, 100, 1300})
                    for (const int apart : {0, 1}) {
                        const int64_t groups = apart ? sequences : 1;
                        if (sequences * tokens > INT32_MAX || groups == 0) continue;
                        if (look(sequences, tokens, groups, row_bytes / 2, step, row_bytes)) return 1;
                    }
    return 0;
}
