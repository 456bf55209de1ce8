// The scan's kernels for fp32.
#include "scan_kernels.hpp"

namespace convmi {
namespace scan {

hipError_t scan_kernels_f32(int run, int gr, int ns, const ScanArgs& a, int items, hipStream_t s)
{
    return run_of<float>(run, gr, ns, a, items, s);
}

}  // namespace scan
}  // namespace convmi
