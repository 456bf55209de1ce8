// The scan's kernels for bf16.
#include "scan_kernels.hpp"

namespace convmi {
namespace scan {

hipError_t scan_kernels_bf16(int run, int gr, int ns, const ScanArgs& a, int items, hipStream_t s)
{
    return run_of<bf16_t>(run, gr, ns, a, items, s);
}

}  // namespace scan
}  // namespace convmi
