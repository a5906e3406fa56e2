// Words of a row of int8 codes as the row kernels fetch them: what lies behind
// the last column (another array, or nothing at all) does not enter.
#include <cstdio>
#include <cstring>

#include "../../block_wise_mixed_b200/csrc/k_i8_rows.cuh"

int main() {
    alignas(16) int8_t row[48];
    for (int cols = 1; cols <= 32; ++cols)
        for (int behind = -1; behind <= 1; behind += 2) {
            std::memset(row, behind, sizeof row);
            for (int c = 0; c < cols; ++c) row[c] = (int8_t)(c * 7 - 100);
            for (int w = 0; w < 12; ++w) {
                uint32_t want = 0;
                for (int j = 0; j < 4; ++j)
                    if (4 * w + j < cols) want |= (uint32_t)(uint8_t)row[4 * w + j] << (8 * j);
                const uint32_t got = mpq::i8_codes_word(row, w, cols);
                if (got != want) {
                    std::printf("cols %d word %d: %08x, not %08x\n", cols, w, got, want);
                    return 1;
                }
            }
        }
    std::printf("ok\n");
    return 0;
}
