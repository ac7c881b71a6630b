// Answers what the MXFP4 products' rules choose, read from csrc/host_pack.cpp
// itself: one line in, one line out.
//   d A4 M K N  ->  tile, slices of K        (dense)
//   g A4 S E N  ->  tile, or -1 for the kernel for few rows (grouped)
#include <cstdio>

#include "qgemm_internal.h"

int main() {
    char kind;
    int a4, x, y, z;
    while (std::scanf(" %c %d %d %d %d", &kind, &a4, &x, &y, &z) == 5) {
        if (kind == 'd') {
            const qg::MxPlan p = qg::mx_dense_plan(a4 != 0, x, y, z);
            std::printf("%d %d\n", (int)p.shape, p.nsplit);
        } else {
            std::printf("%d 1\n", qg::mx_grouped_decode(x, y, z) ? -1 : (int)qg::mx_grouped_shape(a4 != 0, x, y, z));
        }
    }
}
