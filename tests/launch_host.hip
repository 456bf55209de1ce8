// Launches that no grid can hold are refused before the runtime sees them.
#include "common.hpp"

#include <cstdio>

namespace convmi {
ArmedEvents& armed_events()
{
    static ArmedEvents e{nullptr, nullptr};
    return e;
}
}  // namespace convmi

__global__ void nothing(int) {}

int main()
{
    const dim3 grids[] = {dim3(1u << 24), dim3((1u << 24) + 5), dim3(1u << 31), dim3(1, 1u << 31)}, blocks[] = {dim3(256), dim3(256), dim3(256), dim3(1, 2)};
    for (int i = 0; i < 4; ++i)
        if (convmi::launch(nothing, grids[i], blocks[i], 0, nullptr, 1) != hipErrorInvalidConfiguration) {
            std::printf("grid %d was not refused\n", i);
            return 1;
        }
    std::printf("4 refused\n");
    return 0;
}
