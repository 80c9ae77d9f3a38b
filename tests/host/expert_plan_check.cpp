// Prints which kernel csrc/ops_internal.h chooses (host code the launchers
// run) for products given on the command line, each behind its shape:
//   kind E N H maxEntries ...  -> its DenseForm
#include <cstdio>
#include <cstdlib>

#include "../../combine_count_amd/csrc/ops_internal.h"

int main(int argc, char **argv) {
    for (int i = 1; i + 4 < argc; i += 5) {
        int v[5];
        for (int j = 0; j < 5; ++j) std::printf("%d ", v[j] = std::atoi(argv[i + j]));
        std::printf("%d\n", (int)epdc::plan_dense((epdc::DenseKind)v[0], v[1], v[2], v[3], v[4]));
    }
    return 0;
}
