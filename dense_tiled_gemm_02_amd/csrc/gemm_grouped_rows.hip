// Variants of the grouped product over ragged rows (grouped_kernel.h).
#include "grouped_kernel.h"

namespace dtg {
namespace {

const GroupedEntry kTable[] = {
    GROUPED_ROWS(256, 256, 64, 2, 4, 16, 2),
    GROUPED_ROWS(128, 256, 64, 2, 4, 16, 3),
    GROUPED_ROWS(128, 128, 64, 2, 4, 16, 4),
    GROUPED_ROWS(128, 128, 64, 2, 4, 16, 2),
    GROUPED_ROWS(64, 64, 64, 2, 2, 16, 4),
};

}  // namespace

const GroupedEntry* grouped_rows_table(int* count) {
    *count = static_cast<int>(sizeof(kTable) / sizeof(kTable[0]));
    return kTable;
}

}  // namespace dtg
