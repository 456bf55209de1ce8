// Walks the rows of the norms' forward pass as its lanes do, on the host: every
// row is taken once, and no lane asks for a row, or for a shared gate's row, that
// does not exist.  Prints the number of walks; the first wrong one ends it.
#include <cstdio>
#include <vector>

#include "row_walk.hpp"

int main()
{
    long walks = 0;
    for (int lanes : {8, 16, 32, 64, 0})  // of a row; 0: a workgroup
        for (int64_t rows = 1; rows <= 70; ++rows)
            for (int64_t gate_rows = 1; gate_rows <= rows; ++gate_rows) {
                if (rows % gate_rows != 0) continue;
                for (int64_t per = 1; per <= 3; ++per) {
                    const int step = lanes ? 64 / lanes : 1, waves = lanes ? 4 : 1;
                    const int64_t at_once = static_cast<int64_t>(step) * waves;
                    const int64_t grid = (rows + at_once * per - 1) / (at_once * per);
                    std::vector<int> taken(rows, 0);
                    for (int64_t wave = 0; wave < grid * waves; ++wave) {
                        const convmi::RowWalk walk(wave, step, per, rows);
                        for (int sub = 0; sub < step; ++sub)
                            for (int64_t r = walk.first; walk.has(r, sub); r += step) {
                                const int64_t row = r + sub;
                                if (row >= rows || row / gate_rows >= rows / gate_rows || taken[row]++) {
                                    std::printf("lanes %d rows %ld gate_rows %ld per %ld: wave %ld takes row %ld\n", lanes,
                                                static_cast<long>(rows), static_cast<long>(gate_rows), static_cast<long>(per),
                                                static_cast<long>(wave), static_cast<long>(row));
                                    return 1;
                                }
                            }
                    }
                    for (int64_t r = 0; r < rows; ++r)
                        if (taken[r] != 1) return std::printf("lanes %d rows %ld: row %ld is left out\n", lanes, static_cast<long>(rows), static_cast<long>(r)), 1;
                    ++walks;
                }
            }
    std::printf("%ld walks\n", walks);
    return 0;
}
