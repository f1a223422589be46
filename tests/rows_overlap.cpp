// C entry for tests/test_row_outputs.py: whether rows of two arrays share a byte.
#include "../shared_prefix_fan_gb300/csrc/rows.h"

extern "C" int rows_share(uint64_t a, int64_t a_stride, uint64_t b, int64_t b_stride, int64_t n, int64_t row) {
    return fanout::rows_overlap(reinterpret_cast<const void*>(a), a_stride,
                                reinterpret_cast<const void*>(b), b_stride, n, row)
               ? 1
               : 0;
}
