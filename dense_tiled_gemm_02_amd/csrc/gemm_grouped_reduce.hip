// Variants of the grouped weight gradient, the product that contracts over a
// group's rows (grouped_kernel.h): A^T is A stored K x M, B is row-major.
#include "grouped_kernel.h"

namespace dtg {
namespace {

const GroupedEntry kTable[] = {
    GROUPED_REDUCE(256, 256, 64, 2, 4, 16, 2),
    GROUPED_REDUCE(128, 256, 64, 2, 4, 16, 3),
    GROUPED_REDUCE(128, 128, 64, 2, 4, 16, 2),
    GROUPED_REDUCE(128, 128, 32, 2, 2, 16, 2),
    GROUPED_REDUCE(64, 64, 64, 2, 2, 16, 4),
};

}  // namespace

const GroupedEntry* grouped_reduce_table(int* count) {
    *count = static_cast<int>(sizeof(kTable) / sizeof(kTable[0]));
    return kTable;
}

}  // namespace dtg
