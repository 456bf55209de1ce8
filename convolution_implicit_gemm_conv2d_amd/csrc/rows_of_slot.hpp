// Rows of a batch of tokens by the slot of the pool that holds their state.
#pragma once

#include "common.hpp"

namespace convmi {

// Calls f(row, slot) for the rows that the workgroup of `row` has to do: `row`
// itself, and the later ones of the same slot after it, in order; none if an
// earlier row has that slot, since that row's workgroup does them all.  A slot
// outside the pool is a row without a state: f(row, -1).  Without slots a row's
// slot is its number.  All threads of the workgroup call it.
template <typename F>
__device__ __forceinline__ void each_row_of_slot(const int* slots, int rows, int count, int row, F f)
{
    if (!slots) {
        f(row, row);
        return;
    }
    const int slot = slots[row];
    if (slot < 0 || slot >= count) {
        f(row, -1);
        return;
    }
    bool other = false;
    for (int i = threadIdx.x; i < rows; i += blockDim.x) other |= i != row && slots[i] == slot;
    if (!__syncthreads_or(other)) {
        f(row, slot);
        return;
    }
    for (int i = 0; i < row; ++i)
        if (slots[i] == slot) return;
    for (int i = row; i < rows; ++i)
        if (slots[i] == slot) f(i, slot);  // each thread reads back only what it wrote itself
}

}  // namespace convmi
