// How the norms' forward pass hands out its rows.  Apart from the kernel, and
// constexpr, so that the host can walk every lane's rows as well.
#pragma once

#include <cstdint>

namespace convmi {

// The piece of the rows that wave `wave` takes (a workgroup's, where a row takes
// one): `step` rows at a time, one for each of its groups of lanes, `per` times.
struct RowWalk {
    int64_t first, end;
    constexpr RowWalk(int64_t wave, int step, int64_t per, int64_t rows)
        : first(wave * step * per), end(rows < first + step * per ? rows : first + step * per)
    {
    }
    // Whether group `sub` has a row when the wave is at row r.  A group without
    // one leaves the walk before it reads anything: the gate row that its row
    // would share may lie past the gate's end.
    constexpr bool has(int64_t r, int sub) const { return sub < end - r; }
};

}  // namespace convmi
