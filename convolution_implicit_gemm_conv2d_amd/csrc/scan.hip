// Selective scan: its plan (the lanes' layout, pieces of the rows), workspaces
// and launches.  The kernels of the two types are built by scan_bf16.hip and
// scan_f32.hip.
#include "scan_launch.hpp"

#include <algorithm>

namespace convmi {
namespace scan {

namespace {

size_t up(size_t n) { return (n + 15) & ~size_t(15); }

// Workgroups that one range of rows gives with GR groups of lanes.
int64_t blocks_of(const ScanArgs& a, int gr) { return (a.per_group + kWaves * (64 / gr) - 1) / (kWaves * (64 / gr)); }

// Groups of lanes and states of a lane: four groups hold up to 16 states, the
// fewest instructions a row (its LDS reads and merges are shared by four
// states).  Pieces of the rows where the sequences alone leave the device
// empty, or where their lengths are the device's own knowledge.
struct Plan {
    int gr, ns;
};
Plan plan(ScanArgs& a, bool packed)
{
    Plan p;
    p.gr = a.n <= 16 ? 4 : a.n <= 32 ? 8 : 16;
    p.ns = (a.n + p.gr - 1) / p.gr;
    a.blocks = static_cast<int>(blocks_of(a, p.gr));
    const int64_t one = static_cast<int64_t>(a.groups) * a.blocks * kWaves;  // waves of a range of rows
    constexpr int64_t kFill = 2048;                                        // two waves for each SIMD
    const int64_t want = std::min<int64_t>((kFill + one - 1) / one, (a.rows + 63) / 64);
    a.pieces = 0;
    a.piece_rows = 0;
    if (a.rows > 0 && (packed || (a.seqs < want && one * a.seqs < kFill / 2))) {
        const int64_t rows = (a.rows + want - 1) / want;
        a.piece_rows = (rows + kTile - 1) / kTile * kTile;
        a.pieces = static_cast<int>((a.rows + a.piece_rows - 1) / a.piece_rows);
    }
    return p;
}

size_t ends_bytes(const ScanArgs& a) { return a.pieces > 1 ? up(a.pieces * static_cast<size_t>(a.channels) * a.n * 4) + up(a.pieces * static_cast<size_t>(a.channels) * 4) : 0; }
char* take_ends(ScanArgs& a, char* at)
{
    a.ends = reinterpret_cast<float*>(at);
    at += up(a.pieces * static_cast<size_t>(a.channels) * a.n * 4);
    a.sums = reinterpret_cast<float*>(at);
    return at + up(a.pieces * static_cast<size_t>(a.channels) * 4);
}
int items(const ScanArgs& a) { return a.pieces > 0 ? a.pieces : a.seqs; }

}  // namespace
}  // namespace scan

using namespace scan;

size_t scan_saved(int64_t rows, int channels, int n)
{
    return static_cast<size_t>((rows + kScanTile - 1) / kScanTile) * channels * n * 4;
}

size_t scan_fwd_workspace(const ScanArgs& args, bool packed)
{
    ScanArgs a = args;
    plan(a, packed);
    return ends_bytes(a);
}

size_t scan_bwd_workspace(const ScanArgs& args, bool packed, bool saved)
{
    ScanArgs a = args;
    plan(a, packed);
    const size_t cb = static_cast<size_t>(a.groups) * a.blocks, n = items(a);
    return (saved ? 0 : up(scan_saved(a.rows, a.channels, a.n))) + ends_bytes(a) + up(cb * a.rows * 2 * a.n * 4) +
           up(n * a.channels * a.n * 4) + 2 * up(n * a.channels * 4);
}

hipError_t launch_scan_fwd(ScanArgs a, int dtype, void* workspace, hipStream_t s)
{
    if (a.seqs == 0) return hipSuccess;
    const Plan p = plan(a, a.starts != nullptr);
    const bool passes = a.pieces > 1;
    if (passes) take_ends(a, static_cast<char*>(workspace));
    auto go = dtype ? scan_kernels_bf16 : scan_kernels_f32;
    CallEvents events;
    if (passes) {
        events.next(false);
        if (hipError_t e = go(kRunEnds, p.gr, p.ns, a, items(a), s)) return e;
    }
    events.next(true);
    return go(kRunOutputs, p.gr, p.ns, a, items(a), s);
}

hipError_t launch_scan_bwd(ScanArgs a, const ScanGrads& g, int dtype, void* workspace, hipStream_t s)
{
    const Plan p = plan(a, a.starts != nullptr);
    const bool passes = a.pieces > 1, again = !a.saved;
    char* at = static_cast<char*>(workspace);
    if (again) {
        a.saved = reinterpret_cast<float*>(at);
        at += up(scan_saved(a.rows, a.channels, a.n));
    }
    if (passes) at = take_ends(a, at);
    const size_t cb = static_cast<size_t>(a.groups) * a.blocks;
    const int n = items(a);
    a.part_bc = reinterpret_cast<float*>(at);
    at += up(cb * a.rows * 2 * a.n * 4);
    a.part_a = reinterpret_cast<float*>(at);
    at += up(static_cast<size_t>(n) * a.channels * a.n * 4);
    a.part_d = reinterpret_cast<float*>(at);
    at += up(static_cast<size_t>(n) * a.channels * 4);
    a.part_bias = reinterpret_cast<float*>(at);
    SumArgs sums{};
    const int64_t all = static_cast<int64_t>(a.channels) * a.n;
    if (g.dA) add_sum(sums, a.part_a, all, all, n, g.dA);
    if (g.dD) add_sum(sums, a.part_d, a.channels, a.channels, n, g.dD);
    if (g.dbias) add_sum(sums, a.part_bias, a.channels, a.channels, n, g.dbias);
    const bool bc = (a.dB || a.dC) && a.rows > 0;
    auto go = dtype ? scan_kernels_bf16 : scan_kernels_f32;
    CallEvents events;
    hipError_t e = hipSuccess;
    if (again && a.rows > 0) {
        if (passes) {
            events.next(false);
            if ((e = go(kRunEnds, p.gr, p.ns, a, n, s))) return e;
        }
        events.next(false);
        if ((e = go(kRunStates, p.gr, p.ns, a, n, s))) return e;
    }
    if (passes) {
        events.next(false);
        if ((e = go(kRunBack, p.gr, p.ns, a, n, s))) return e;
    }
    if (n > 0) {
        events.next(!bc && !sums.jobs);
        if ((e = go(kRunGradient, p.gr, p.ns, a, n, s))) return e;
    }
    if (bc) {
        events.next(!sums.jobs);
        if ((e = go(kRunSums, p.gr, p.ns, a, n, s))) return e;
    }
    if (!sums.jobs) return e;
    events.next(true);
    return launch_sums(sums, 0, s);
}

}  // namespace convmi
