// Rows of a batch of tokens by the slot of the pool that holds their state.
#pragma once

#include "common.hpp"

namespace convmi {

// Does the rows that the workgroup of `row` has to do: `row` itself, and the
// later ones of the same slot after it, in order; none if an earlier row has that
// slot, since that row's workgroup does them all.  read(row, slot) loads what a row
// needs, finish(row, slot) computes and stores it; absent(row) is called for a row
// whose slot lies outside the pool.  Without slots a row's slot is its number.  All threads
// of the workgroup call it.  The rows' own loads are out while the slots are
// compared, four at a time: every workgroup reads all slots, which costs from about a thousand
// rows on (4096 rows of 1024 channels: convolution 49 us one by one, 35 so, 19 without
// slots; scan 247, 193 and 147).
template <typename R, typename F, typename A>
__device__ __forceinline__ void each_row_of_slot(const int* slots, int rows, int count, int row, R read, F finish, A absent)
{
    const int slot = slots ? slots[row] : row;
    if (slot < 0 || slot >= count) {
        absent(row);
        return;
    }
    read(row, slot);
    if (slots) {
        typedef int four __attribute__((ext_vector_type(4), aligned(4)));
        int same = 0;  // rows of this slot
        const int whole = rows & ~3;
        for (int i = threadIdx.x * 4; i < whole; i += blockDim.x * 4) {
            const four t = *reinterpret_cast<const four*>(slots + i);
            same += (t.x == slot) + (t.y == slot) + (t.z == slot) + (t.w == slot);
        }
        if (threadIdx.x < rows - whole) same += slots[whole + threadIdx.x] == slot;
        // its own row is one of them, found by one thread
        const bool other = same > (row < whole ? row / 4 % blockDim.x == threadIdx.x : row - whole == threadIdx.x);
        if (__syncthreads_or(other)) {
            for (int i = 0; i < row; ++i)
                if (slots[i] == slot) return;
            for (int i = row; i < rows; ++i)
                if (slots[i] == slot) {  // each thread reads back only what it wrote itself
                    read(i, slot);
                    finish(i, slot);
                }
            return;
        }
    }
    finish(row, slot);
}

}  // namespace convmi
