// Prints which kernel csrc/ops_internal.h chooses (host code the launchers
// run) for shapes given on the command line, each behind the shape:
//   product E N H maxEntries numRows ...              -> its ProductForm
//   route E K G keep T softmax biased aligned ...     -> lanes perLane inRow
//   grad E K aligned ...                              -> lanes perLane inRow
#include <cstdio>
#include <cstdlib>
#include <cstring>

#include "../../combine_count_amd/csrc/ops_internal.h"

int main(int argc, char **argv) {
    if (argc < 2) return 2;
    const bool product = !std::strcmp(argv[1], "product"), route = !std::strcmp(argv[1], "route");
    const int step = product ? 5 : route ? 8 : 3;
    for (int i = 2; i + step - 1 < argc; i += step) {
        int v[8];
        for (int j = 0; j < step; ++j) std::printf("%d ", v[j] = std::atoi(argv[i + j]));
        if (product) {
            std::printf("%d\n", (int)epdc::plan_product(v[0], v[1], v[2], v[3], v[4]));
        } else {
            const epdc::RoutePlan p = route ? epdc::plan_route(v[0], v[1], v[2], v[3], v[4], v[5], v[6], v[7])
                                            : epdc::plan_route_grad(v[0], v[1], v[2]);
            std::printf("%d %d %d\n", p.lanes, p.perLane, (int)p.inRow);
        }
    }
    return 0;
}
