// The scan's launches for one type.
#pragma once

#include "scan_bwd.hpp"
#include "scan_fwd.hpp"
#include "scan_launch.hpp"

namespace convmi {
namespace scan {

template <typename T, int GR, int NS>
hipError_t run_one(int run, const ScanArgs& a, int items, hipStream_t s)
{
    constexpr bool kGradient = NS != 3 && (GR > 4 || NS == 1);  // what the plan takes for it
    const int64_t blocks = static_cast<int64_t>(a.groups) * a.blocks * items;
    if (run == kRunSums) {
        const int64_t n = (a.sum_rows * 2 * a.n + 255) / 256;
        if (a.groups > 65535) return hipErrorInvalidConfiguration;
        return launch(sum_bc_kernel<T>, dim3(static_cast<unsigned>(n), a.groups), dim3(256), 0, s, a);
    }
    if (blocks > kMostBlocks) return hipErrorInvalidConfiguration;
    const dim3 grid(static_cast<unsigned>(blocks)), threads(kThreads);
    switch (run) {
    case kRunOutputs: return launch(fwd_kernel<T, GR, NS, kOutputs>, grid, threads, 0, s, a);
    case kRunStates: return launch(fwd_kernel<T, GR, NS, kStates>, grid, threads, 0, s, a);
    case kRunEnds: return launch(fwd_kernel<T, GR, NS, kEnds>, grid, threads, 0, s, a);
    case kRunBack:
        if constexpr (kGradient) return launch(back_kernel<T, GR, NS>, grid, threads, 0, s, a);
        else return hipErrorInvalidConfiguration;
    default:
        if constexpr (kGradient) return launch(bwd_kernel<T, GR, NS>, grid, threads, 0, s, a);
        else return hipErrorInvalidConfiguration;
    }
}

template <typename T>
hipError_t run_of(int run, int gr, int ns, const ScanArgs& a, int items, hipStream_t s)
{
#define CONVMI_SCAN(GR, NS) \
    if (gr == GR && ns == NS) return run_one<T, GR, NS>(run, a, items, s);
    CONVMI_SCAN(4, 1) CONVMI_SCAN(4, 2) CONVMI_SCAN(4, 3) CONVMI_SCAN(4, 4)
    CONVMI_SCAN(8, 1) CONVMI_SCAN(8, 2) CONVMI_SCAN(8, 3) CONVMI_SCAN(8, 4) CONVMI_SCAN(16, 3) CONVMI_SCAN(16, 4)
#undef CONVMI_SCAN
    return hipErrorInvalidConfiguration;
}

}  // namespace scan
}  // namespace convmi
