// Prints which kernel csrc/ops_internal.h chooses (host code the launchers
// run) for shapes given on the command line:
//   product E N H maxEntries numRows ...  -> the shape and its ProductForm
#include <cstdio>
#include <cstdlib>
#include <cstring>

#include "../../combine_count_amd/csrc/ops_internal.h"

int main(int argc, char **argv) {
    if (argc < 2 || std::strcmp(argv[1], "product")) return 2;
    for (int i = 2; i + 4 < argc; i += 5) {
        int v[5];
        for (int j = 0; j < 5; ++j) v[j] = std::atoi(argv[i + j]);
        std::printf("%d %d %d %d %d %d\n", v[0], v[1], v[2], v[3], v[4],
                    (int)epdc::plan_product(v[0], v[1], v[2], v[3], v[4]));
    }
    return 0;
}
