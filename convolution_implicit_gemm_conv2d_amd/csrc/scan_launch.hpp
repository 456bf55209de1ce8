// The scan's kernels by type, as scan.hip calls them.
#pragma once

#include "scan.hpp"

namespace convmi {
namespace scan {

constexpr int64_t kMostBlocks = (int64_t(1) << 24) - 1;  // of 256 lanes: a grid holds fewer than 2^32

enum Run { kRunOutputs, kRunStates, kRunEnds, kRunBack, kRunGradient, kRunSums };

// One launch over `items` shares of the rows with `gr` groups of `ns` states.
hipError_t scan_kernels_bf16(int run, int gr, int ns, const ScanArgs& a, int items, hipStream_t s);
hipError_t scan_kernels_f32(int run, int gr, int ns, const ScanArgs& a, int items, hipStream_t s);

}  // namespace scan
}  // namespace convmi
