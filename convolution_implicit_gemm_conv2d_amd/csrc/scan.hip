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

// Whole sequences.  A workgroup takes as many, one after another, as leave no more than
// kMostShares workgroups: they fill the device sixteen times at least, and dA, dD and the
// bias's gradient have a partial sum for each of a launch's workgroups, not for each sequence
// (a million sequences of a row have a partial as large as their states otherwise).
// The gradient's partials of dB and dC, 2 N values for each row and workgroup's
// channels, take no more than kPartBytes where launches of kFill workgroups are
// less; sequences past those go to a next launch, which adds to its workgroups' partial sums.
constexpr int64_t kMostShares = 1 << 14, kFill = 1 << 13, kPartBytes = int64_t(1) << 30;
void walk(ScanArgs& a, bool gradient)
{
    const int64_t per = static_cast<int64_t>(a.groups) * a.blocks, bytes = per * a.len * 2 * a.n * 4;
    int64_t seqs = a.seqs;
    if (gradient) {
        const int64_t most = std::max(kPartBytes / std::max<int64_t>(bytes, 1), (kFill + per - 1) / per);
        seqs = (seqs + most - 1) / most;  // launches
        seqs = seqs > 1 ? (a.seqs + seqs - 1) / seqs : a.seqs;
    }
    a.walk = static_cast<int>(std::max<int64_t>(1, (seqs * per + kMostShares - 1) / kMostShares));
    seqs = (seqs + a.walk - 1) / a.walk * a.walk;
    a.launch_seqs = static_cast<int>(std::min<int64_t>(seqs, a.seqs));
}

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
    walk(a, gradient);
    a.part_rows = a.launch_seqs * a.len;
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
    a.part_rows = a.rows;
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
// Shares of a launch: of all rows, or with `seqs` sequences.
int items(const ScanArgs& a, int seqs) { return a.pieces > 0 ? a.pieces : static_cast<int>((static_cast<int64_t>(seqs) + a.walk - 1) / a.walk); }

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
    const size_t cb = static_cast<size_t>(a.groups) * a.blocks, n = items(a, a.launch_seqs);
    return (saved ? 0 : up(scan_saved(a.rows, a.channels, a.n))) + ends_bytes(a) + up(cb * a.part_rows * 2 * a.n * 4) +
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
        if (hipError_t e = go(kRunEnds, p.gr, p.ns, a, items(a, a.seqs), s)) return e;
    }
    events.next(true);
    return go(kRunOutputs, p.gr, p.ns, a, items(a, a.seqs), s);
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
    const int n = items(a, a.launch_seqs);
    float* part_bc = reinterpret_cast<float*>(at);
    at += up(cb * a.part_rows * 2 * a.n * 4);
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
        ScanArgs all_seqs = a;
        walk(all_seqs, false);
        if ((e = go(kRunStates, p.gr, p.ns, all_seqs, items(all_seqs, a.seqs), s))) return e;
    }
    if (passes) {
        events.next(false);
        if ((e = go(kRunBack, p.gr, p.ns, a, n, s))) return e;
    }
    for (int64_t seq = 0; n > 0 && seq < a.seqs; seq += a.launch_seqs) {
        const bool end = a.pieces > 0 || seq + a.launch_seqs >= a.seqs;
        a.seq0 = static_cast<int>(seq);
        const int64_t row0 = a.pieces > 0 ? 0 : seq * a.len, rows = std::min(a.part_rows, a.rows - row0);
        a.part_bc = part_bc - row0 * 2 * a.n;  // the kernel counts rows from the first of all
        events.next(end && !bc && !sums.jobs);
        if ((e = go(kRunGradient, p.gr, p.ns, a, end && a.pieces == 0 ? items(a, a.seqs - a.seq0) : n, s))) return e;
        // one launch, but for rows of more values than a grid has lanes
        const int64_t most = kMostBlocks * 256 / (2 * a.n);
        for (int64_t r = 0; bc && r < rows; r += most) {
            ScanArgs b = a;
            b.part_bc = part_bc + r * 2 * a.n;
            b.row0 = row0 + r;
            b.sum_rows = std::min(most, rows - r);
            events.next(end && !sums.jobs && r + most >= rows);
            if ((e = go(kRunSums, p.gr, p.ns, b, 0, s))) return e;
        }
        if (end) break;
    }
    if (!sums.jobs) return e;
    events.next(true);
    return launch_sums(sums, 0, s);
}

}  // namespace convmi
