// Selective scan: its plan (the lanes' layout, pieces of the rows), workspaces
// and launches.  The kernels of the two types are built by scan_bf16.hip and
// scan_f32.hip.
#include "scan_launch.hpp"

#include <algorithm>
#include <cmath>

namespace convmi {
namespace scan {

namespace {

size_t up(size_t n) { return (n + 15) & ~size_t(15); }

// Workgroups that one range of rows gives with GR groups of lanes.
int64_t blocks_of(const ScanArgs& a, int gr) { return (a.per_group + kWaves * (64 / gr) - 1) / (kWaves * (64 / gr)); }

// Groups of lanes, states of a lane, and pieces of the rows.
//
// Few groups cost the fewest instructions: a row's LDS reads and merges are
// shared by more states of a lane.  But one wave on a SIMD cannot fill it (an exp2
// with four multiply-adds takes 31 cycles there, 23 with two waves, 20 with eight), so with
// less than two waves for each SIMD twice the groups are better (4 x 4096 rows of 4096
// channels, 16 states: 395 us with 4 groups, 376 with 8), and the gradient, whose
// 244 registers leave room for two waves in any case, always takes them (8 x 2048 rows of
// 2048 channels, forward and gradient: 832 us and 788).  With less than one wave for each SIMD
// the rows are cut into pieces, which cost a pass more over them (16384 rows of 1024
// channels: 141 us in pieces, 280 in whole).  So are packed rows always: their
// lengths are the device's own knowledge, and one long sequence among short ones
// would otherwise keep a few waves busy alone.
struct Plan {
    int gr, ns;
};
constexpr int64_t kSimds = 1024;
int64_t waves_of(const ScanArgs& a, int gr) { return static_cast<int64_t>(a.groups) * blocks_of(a, gr) * kWaves; }  // of a range of rows

Plan plan(ScanArgs& a, bool packed, bool gradient)
{
    const int few = a.n <= 16 ? 4 : a.n <= 32 ? 8 : 16, many = a.n <= 4 ? 4 : a.n <= 32 ? 8 : 16;
    const bool whole = a.rows == 0 || (!packed && a.seqs * waves_of(a, many) >= kSimds);
    Plan p;
    p.gr = gradient || (whole && a.seqs * waves_of(a, few) < 2 * kSimds) ? many : few;
    p.ns = (a.n + p.gr - 1) / p.gr;
    // three states of a lane cost the gradient more registers than four
    if (gradient && p.ns == 3) p.ns = 4;
    a.blocks = static_cast<int>(blocks_of(a, p.gr));
    a.pieces = 0;
    a.piece_rows = 0;
    if (whole) return p;
    // Two waves for each SIMD, 32 rows in a piece at least, and no pieces below 128 rows.
    // 2048 channels, a prompt's call (and forward with gradient): 256 rows take 15.5 us (46.7) in
    // pieces of 32, 19.6 (55.9) in pieces of 64, 28.5 (93.6) in whole; 128 rows 14.3 (42.0)
    // and 16.5 (56.8) in whole; 64 rows 13.8 (40.1) and 10.5 (38.2) in whole.
    // A piece reads the ends of all before it, so at most as many pieces as a piece has rows
    // (16384 rows of 64 channels: 128 pieces 57 us, 256 74 us, 512 163 us; 64 were 66 us).
    const int64_t most = a.rows < 128 ? 1 : std::min(a.rows / 32, static_cast<int64_t>(std::sqrt(static_cast<double>(a.rows))));
    const int64_t want = std::min((2 * kSimds + waves_of(a, p.gr) - 1) / waves_of(a, p.gr), most);
    if (!packed && want <= a.seqs) return p;
    const int64_t rows = (a.rows + want - 1) / want;
    a.piece_rows = (rows + kTile - 1) / kTile * kTile;
    a.pieces = static_cast<int>((a.rows + a.piece_rows - 1) / a.piece_rows);
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
    plan(a, packed, false);
    return ends_bytes(a);
}

size_t scan_bwd_workspace(const ScanArgs& args, bool packed, bool saved)
{
    ScanArgs a = args;
    plan(a, packed, true);
    const size_t cb = static_cast<size_t>(a.groups) * a.blocks, n = items(a);
    return (saved ? 0 : up(scan_saved(a.rows, a.channels, a.n))) + ends_bytes(a) + up(cb * a.rows * 2 * a.n * 4) +
           up(n * a.channels * a.n * 4) + 2 * up(n * a.channels * 4);
}

hipError_t launch_scan_fwd(ScanArgs a, int dtype, void* workspace, hipStream_t s)
{
    if (a.seqs == 0) return hipSuccess;
    const Plan p = plan(a, a.starts != nullptr, false);
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
    const Plan p = plan(a, a.starts != nullptr, true);
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
