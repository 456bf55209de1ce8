// Walks lists through AdamW's tables: every element exactly once, in order, no
// table past its entries or past the lanes of a grid, cuts at whole chunks.
#include "adamw_tables.hpp"

#include <cstdio>
#include <vector>

using namespace convmi;

static int wrong(const char* what, int list)
{
    std::printf("list %d: %s\n", list, what);
    return 1;
}

int main()
{
    const size_t huge = (size_t(1) << 38) - 1, grid = size_t(kMostChunks) * kAdamChunk;
    const std::vector<std::vector<size_t>> lists = {
        {}, {0}, {0, 0, 5, 0}, {1}, {1024, 1025, 1023}, {grid}, {grid + 1}, {grid - 1, 1, 1}, {7, grid, 9}, {huge}, {3, huge, huge, 0, 2}, std::vector<size_t>(1000, 10),
        {grid - 1024, 1024, 1}, {grid - 1023, 1024}};
    int tables = 0, n = 0;
    for (const auto& counts : lists) {
        for (int entries : {1, 12, 48})
            for (uint32_t most : {kMostChunks, 5u}) {
                if (most == 5u && counts.size() && counts[0] + (counts.size() > 1 ? counts[1] : 0) > (size_t(1) << 24)) continue;  // millions of tables
                ListPlace at;
                int tensor = 0;
                uint64_t done = 0;  // elements of it
                while (more_chunks(counts.data(), static_cast<int>(counts.size()), at)) {
                    uint32_t next = 0;
                    int used = 0, bad = 0;
                    const uint32_t chunks = fill_table(counts.data(), static_cast<int>(counts.size()), entries, most, at,
                                                       [&](int k, int i, uint64_t first, uint64_t count, uint32_t begin) {
                                                           while (tensor < i) {
                                                               if (done != counts[tensor]) bad = 1;
                                                               ++tensor, done = 0;
                                                           }
                                                           if (k != used++ || i != tensor || first != done || first % kAdamChunk || !count || begin != next) bad = 1;
                                                           next += static_cast<uint32_t>((count + kAdamChunk - 1) / kAdamChunk);
                                                           done += count;
                                                       });
                    if (bad) return wrong("an entry is not the next part of the list", n);
                    if (!used || used > entries || !chunks || chunks > most || chunks != next) return wrong("a table does not fit", n);
                    ++tables;
                }
                for (; tensor < static_cast<int>(counts.size()); ++tensor, done = 0)
                    if (done != counts[tensor]) return wrong("elements are left", n);
            }
        ++n;
    }
    std::printf("%d tables\n", tables);
    return 0;
}
