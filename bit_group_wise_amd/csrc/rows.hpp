// rows.hpp -- which rows of a grouped product a workgroup works on.
//
// A grouped product's rows lie in groups (the rows of one expert), given by
// their offsets on the device, so the host knows their number and no more
// when it launches.  The grid therefore counts pieces of up to CH rows of one
// group at their largest possible number, and every wave finds its piece
// itself: 64 groups at a time, one per lane, with prefix sums over the lanes.
// Offsets are taken as they can be: inside 0 .. rows, and one that falls
// below an earlier one as that one (its group is empty), so that no piece
// leaves the arrays, no row is in two of them, and their number stays within
// the grid whatever the offsets hold.
#pragma once

#include "q4_common.hpp"

namespace q4 {

// The lanes' values of lower or equal number combined: rows of 16 lanes
// first, then the rows' last lanes handed on (0 is neutral in both uses).
template <class Op>
__device__ __forceinline__ int wave_scan(int v, Op op)
{
    v = op(v, __builtin_amdgcn_update_dpp(0, v, 0x111, 0xf, 0xf, false));  // one lane up in its row
    v = op(v, __builtin_amdgcn_update_dpp(0, v, 0x112, 0xf, 0xf, false));  // two
    v = op(v, __builtin_amdgcn_update_dpp(0, v, 0x114, 0xf, 0xf, false));  // four
    v = op(v, __builtin_amdgcn_update_dpp(0, v, 0x118, 0xf, 0xf, false));  // eight
    v = op(v, __builtin_amdgcn_update_dpp(0, v, 0x142, 0xa, 0xf, false));  // lane 15 of rows 0 and 2 to rows 1 and 3
    v = op(v, __builtin_amdgcn_update_dpp(0, v, 0x143, 0xc, 0xf, false));  // lane 31 to rows 2 and 3
    return v;
}

// Rows lo .. hi - 1 of group `group` (-1: no such piece).
struct Piece {
    int group, lo, hi;
};

// Groups base + lane of a launch: their first rows and numbers of rows.
struct GroupLane {
    int start, n;
};
__device__ __forceinline__ GroupLane group_lane(const int32_t *__restrict__ offsets, int groups, int rows, int base,
                                                int lane, int &highest)
{
    const int e = base + lane;
    const bool in = e < groups;
    const int a = in ? min(max(offsets[e], 0), rows) : 0;
    const int b = in ? min(max(offsets[e + 1], 0), rows) : 0;
    const int start = max(wave_scan(a, [](int p, int q) { return max(p, q); }), highest);
    highest = __builtin_amdgcn_readlane(start, 63);
    return GroupLane{start, in ? max(b - start, 0) : 0};
}

// The number of pieces of the launch; of up to 64 groups also what the lanes
// hold of them, for piece_in.
template <int CH>
__device__ __forceinline__ int count_pieces(const int32_t *__restrict__ offsets, int groups, int rows, GroupLane &g,
                                            int &upto)
{
    const int lane = threadIdx.x & 63;
    int highest = 0, total = 0;
    for (int base = 0; base < groups; base += 64) {
        g = group_lane(offsets, groups, rows, base, lane, highest);
        upto = wave_scan((g.n + CH - 1) / CH, [](int p, int q) { return p + q; });
        total += __builtin_amdgcn_readlane(upto, 63);
    }
    return total;
}
// Piece `want` of those of the 64 groups from `base` (upto: the lanes' pieces
// up to theirs).
template <int CH>
__device__ __forceinline__ Piece piece_in(const GroupLane &g, int upto, int base, int want)
{
    const int l = (int)__builtin_ctzll(__ballot(upto > want) | 1ull << 63);
    const int before = l ? __builtin_amdgcn_readlane(upto, l > 0 ? l - 1 : 0) : 0;
    const int start = __builtin_amdgcn_readlane(g.start, l), n = __builtin_amdgcn_readlane(g.n, l);
    const int lo = start + (want - before) * CH;
    return Piece{base + l, lo, min(lo + CH, start + n)};
}
// Piece `want`, below their number, of the launch.
template <int CH>
__device__ __forceinline__ Piece piece_at(const int32_t *__restrict__ offsets, int groups, int rows, int want)
{
    const int lane = threadIdx.x & 63;
    int highest = 0;
    for (int base = 0;; base += 64) {
        const GroupLane g = group_lane(offsets, groups, rows, base, lane, highest);
        const int upto = wave_scan((g.n + CH - 1) / CH, [](int p, int q) { return p + q; });
        const int here = __builtin_amdgcn_readlane(upto, 63);
        if (want < here || base + 64 >= groups)
            return piece_in<CH>(g, upto, base, want);
        want -= here;
    }
}

// Piece `block % pieces` of the launch and `block / pieces` in other, or
// group -1 for a block past all pieces: block counts pieces fastest, so the
// blocks that have work are the grid's first ones.
template <int CH>
__device__ __forceinline__ Piece find_piece(const int32_t *__restrict__ offsets, int groups, int rows, unsigned block,
                                            int others, int &other)
{
    GroupLane g{};
    int upto = 0;
    const int total = count_pieces<CH>(offsets, groups, rows, g, upto);
    if (total == 0 || block / (unsigned)total >= (unsigned)others)
        return Piece{-1, 0, 0};
    other = (int)(block / (unsigned)total);
    const int want = (int)(block % (unsigned)total);
    return groups > 64 ? piece_at<CH>(offsets, groups, rows, want) : piece_in<CH>(g, upto, 0, want);
}

// The same with the pieces in order of their size in quarters of CH rows,
// whole ones first: where a workgroup's time goes by that, the short ones fill
// up what the last whole round of workgroups leaves.
template <int CH>
__device__ __forceinline__ Piece find_piece_long_first(const int32_t *__restrict__ offsets, int groups, int rows,
                                                       unsigned block, int others, int &other)
{
    const int lane = threadIdx.x & 63;
    const auto add = [](int p, int q) { return p + q; };
    // pieces of q quarters in a group of n rows: all whole ones and the last
    const auto pieces = [](int n, int q) { return (q == 4 ? n / CH : 0) + ((n % CH * 4 + CH - 1) / CH == q ? 1 : 0); };
    int highest = 0, count[5] = {};
    for (int base = 0; base < groups; base += 64) {
        const GroupLane g = group_lane(offsets, groups, rows, base, lane, highest);
        count[4] += __builtin_amdgcn_readlane(wave_scan(pieces(g.n, 4), add), 63);
#pragma unroll
        for (int q = 1; q < 4; ++q)
            count[q] += (int)__popcll(__ballot(pieces(g.n, q) != 0));
    }
    int q = 4, of = count[4];
#pragma unroll
    for (int c = 4; c > 1; --c) {
        if (q == c && block >= (unsigned)count[c] * (unsigned)others) {
            block -= (unsigned)count[c] * (unsigned)others;
            q = c - 1;
            of = count[c - 1];
        }
    }
    if (of == 0 || block / (unsigned)of >= (unsigned)others)
        return Piece{-1, 0, 0};
    other = (int)(block / (unsigned)of);
    int want = (int)(block % (unsigned)of);
    highest = 0;
    for (int base = 0;; base += 64) {
        const GroupLane g = group_lane(offsets, groups, rows, base, lane, highest);
        const int upto = wave_scan(pieces(g.n, q), add);
        const int here = __builtin_amdgcn_readlane(upto, 63);
        if (want >= here && base + 64 < groups) {
            want -= here;
            continue;
        }
        const int l = (int)__builtin_ctzll(__ballot(upto > want) | 1ull << 63);
        const int before = l ? __builtin_amdgcn_readlane(upto, l > 0 ? l - 1 : 0) : 0;
        const int start = __builtin_amdgcn_readlane(g.start, l), n = __builtin_amdgcn_readlane(g.n, l);
        // (a group's last piece comes behind its whole ones)
        const int lo = start + (q == 4 ? want - before : n / CH) * CH;
        return Piece{base + l, lo, min(lo + CH, start + n)};
    }
}

// The most pieces that `rows` rows in `groups` groups make: every group but
// for whole pieces adds at most one.
inline int64_t most_pieces(int64_t rows, int64_t groups, int ch)
{
    return rows / ch + (groups < rows ? groups : rows);
}

}  // namespace q4
