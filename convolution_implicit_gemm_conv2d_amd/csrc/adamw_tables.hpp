// How AdamW's launches cut a list of tensors into tables (host only).
//
// A launch takes a table of tensors as its argument and has a workgroup for each
// chunk of them.  A grid holds fewer than 2^32 lanes, so a table ends at kMostChunks;
// a tensor that does not fit goes on in the next table, at a multiple of a chunk
// and so of the blocks that share a scale.
#pragma once

#include <cstddef>
#include <cstdint>

namespace convmi {

// Elements in a chunk: four a lane of a workgroup, so that fp32 arrays are read
// and written in whole lines.  Every chunk has a workgroup of its own, which the device
// gives out as others end (250 M elements, 32-bit states, in one comparison: 2048
// workgroups that walk over chunks of 32768 took 1427 us, a workgroup for each 4096,
// 2048 and 1024 elements 1204, 1128 and 1032; cards and runs differ by 5 %).
constexpr int kAdamThreads = 256, kAdamElements = 4;  // of a lane
constexpr uint32_t kAdamChunk = kAdamThreads * kAdamElements;
constexpr uint32_t kMostChunks = (uint32_t(1) << 24) - 1;
static_assert(uint64_t(kMostChunks) * kAdamThreads < (uint64_t(1) << 32), "a grid's lanes");

// Where the next table begins.
struct ListPlace {
    int tensor = 0;
    uint64_t chunk = 0;  // of it
};

// Goes on to a chunk that exists; false behind the last one.
inline bool more_chunks(const size_t* counts, int n, ListPlace& at)
{
    while (at.tensor < n && at.chunk * kAdamChunk >= counts[at.tensor]) at = ListPlace{at.tensor + 1, 0};
    return at.tensor < n;
}

// Fills a table of `entries` tensors from `at` on, which moves behind it:
// take(entry, tensor, first element, elements, first chunk).  Returns its chunks.
template <typename Take>
uint32_t fill_table(const size_t* counts, int n, int entries, uint32_t most, ListPlace& at, Take take)
{
    uint32_t chunks = 0;
    for (int k = 0; k < entries && chunks < most && more_chunks(counts, n, at); ++k) {
        const uint64_t first = at.chunk * kAdamChunk, left = counts[at.tensor] - first, room = static_cast<uint64_t>(most - chunks) * kAdamChunk;
        const uint64_t count = left < room ? left : room;
        take(k, at.tensor, first, count, chunks);
        const uint32_t now = static_cast<uint32_t>((count + kAdamChunk - 1) / kAdamChunk);
        chunks += now;
        at.chunk += now;
    }
    return chunks;
}

}  // namespace convmi
