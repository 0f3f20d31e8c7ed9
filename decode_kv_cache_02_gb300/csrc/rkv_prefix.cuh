// rkv_prefix.cuh -- what the kernels of attention over shared prefixes have in
// common: the line of work, and how sums over parts of the rows are joined.
//
// Queries that share a prefix and a KV head are rows of one problem, cut into
// tiles; a tile goes over the prefix in units of rows.  All tiles of all prefixes and
// heads lie one after another on a line of units that is cut into equal runs, one a
// block, so ragged prefixes and groups are balanced whatever their sizes; a tile cut
// by a run's end is joined by a second launch.  With more queries a prefix than a tile
// holds, blocks go in teams that take neighbouring tiles over the same rows at the same
// time, so that those come from HBM once: the line's tiles are then a team's.
#pragma once

#include <float.h>

#include "rkv_common.cuh"
#include "rkv_internal.h"

namespace rkv {
namespace prefix {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kNone = -FLT_MAX;  // no maximum yet

struct Params {
    const void* k;
    const void* v;
    const int32_t* table;  // of the prefixes
    const int32_t* lens;
    const int32_t* cu;     // first sequence of each prefix (nullptr: every one has `per`)
    int P, per, max_blocks, log2bs, num_blocks, max_rows;
    int S, H, G, T, R;     // R = T * G rows a sequence and KV head
    const void* q;
    void* out;
    int64_t q_seq, q_tok, q_head, o_seq, o_tok, o_head;
    float* lse;
    // the sums over the sequences' own rows: [S, T, heads][D] and (maximum, sum)
    const float* own;
    const float2* own_ml;
    float4* partial;       // [slot][D / 4][tile]
    float2* partial_ml;    // [slot][tile]
    int4* joins;           // [block]: first sequence, head and first row of a tile, join_of()
    int tile, runs, lead, team;
    float scale, slack;    // of base-2 logits, positive; how far they may pass the maximum
    uint32_t flip;         // scale < 0: the queries change their signs
    DeviceStatus* status;
};

RKV_DEV float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// What a part with sums relative to 2^m counts beside a common reference mx: an
// empty part nothing, one whose logits are all NaN its NaN.
RKV_DEV float weight(float m, float l, float mx) {
    if (m == -INFINITY) return l != l ? 1.f : 0.f;
    return ex2(m - mx);
}
// The base-2 logit m * scale in fp32 (-inf: none), and 2^ what that rounding left.
RKV_DEV float base_of(float m, float scale, float& fix) {
    fix = 1.f;
    if (m == kNone) return -INFINITY;
    const float z = __fmul_rn(m, scale), rest = fmaf(m, scale, -z);
    if (fabsf(z) <= FLT_MAX && fabsf(rest) <= 32.f) fix = ex2(rest);
    return z;
}

// ------------------------------------------------------------------ line --

// Groups are the P prefixes and, behind them, the sequences without one (a prefix of
// no rows).  A group ends where the next begins, never before it begins and never past
// the last sequence, whatever cu holds, so every sequence is in one group.
RKV_DEV int end_of(const Params& p, int i) {
    if (i >= p.P) return p.S;
    const int64_t e = p.cu ? (int64_t)p.cu[i + 1] : (int64_t)(i + 1) * p.per;
    return e < 0 ? 0 : (e > p.S ? p.S : (int)e);
}
RKV_DEV int len_of(const Params& p, int i) {
    if (i >= p.P) return 0;
    const int n = p.lens[i];
    return n < 0 ? 0 : (n > p.max_rows ? p.max_rows : n);
}
// Units of a (team's) tile; an empty prefix has one too (its queries' outputs are written by
// it).  On the line a tile is p.lead places longer: what its beginning and end cost.
template <int UNIT>
RKV_DEV uint32_t units_of(int rows) {
    return rows <= UNIT ? 1u : (uint32_t)(rows - 1) / UNIT + 1u;
}
RKV_DEV uint32_t tiles_of(const Params& p, int seqs) {
    const uint32_t rows = (uint32_t)(p.tile * p.team);
    return ((uint32_t)seqs * (uint32_t)p.R + rows - 1u) / rows;
}

struct Place {
    uint32_t n, runs;  // units and runs in use
    uint32_t u0, u1;   // the run (empty: none for this block)
    uint32_t start;    // first unit of the current tile
    int i, seq0, seqs, len, h, tile;  // group, its sequences and rows; head, tile
};
RKV_DEV uint32_t first_of(const Place& pl, uint32_t i) {
    const uint32_t per = pl.n / pl.runs, more = pl.n - per * pl.runs;
    return i * per + (i < more ? i : more);
}
RKV_DEV uint32_t run_of(const Place& pl, uint32_t u) {
    const uint32_t per = pl.n / pl.runs, more = pl.n - per * pl.runs;
    const uint32_t big = more * (per + 1);
    return u < big ? u / (per + 1) : more + (u - big) / per;
}
// By a whole warp, every lane with its stretch of groups (the first of which it looks up
// once: most calls have no more than 32).
template <int UNIT>
RKV_DEV Place find_place(const Params& p, uint32_t run) {
    const int lane = threadIdx.x & 31;
    const int groups = p.P + 1, each = (groups + 31) / 32;
    const int a = min(lane * each, groups), b = min(a + each, groups);
    const int end0 = a < b ? end_of(p, a) : 0, len0 = a < b ? len_of(p, a) : 0;
    int top = end0;  // the largest end so far
    for (int i = a + 1; i < b; ++i) top = max(top, end_of(p, i));
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, top, o);
        if (lane >= o) top = max(top, y);
    }
    const int before = __shfl_up_sync(0xffffffffu, top, 1);
    const int from = lane == 0 ? 0 : before;
    uint32_t sum = 0;
    bool wrong = false;
    for (int i = a, at = from; i < b; ++i) {
        const int e = max(at, i == a ? end0 : end_of(p, i));
        sum += tiles_of(p, e - at) * (uint32_t)p.H *
               (units_of<UNIT>(i == a ? len0 : len_of(p, i)) + p.lead);
        if (run == 0 && p.cu && i < p.P) wrong |= p.cu[i + 1] != e || (i == 0 && p.cu[0] != 0);
        at = e;
    }
    if (wrong) set_error(p.status, kDevErrIndex, (unsigned)a);
    uint32_t upto = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint32_t y = __shfl_up_sync(0xffffffffu, upto, o);
        if (lane >= o) upto += y;
    }
    Place pl;
    pl.n = __shfl_sync(0xffffffffu, upto, 31);
    pl.runs = min((uint32_t)p.runs, pl.n);
    pl.u0 = pl.u1 = 0;
    if (run < pl.runs) {
        pl.u0 = first_of(pl, run);
        pl.u1 = first_of(pl, run + 1);
    }
    uint32_t first = upto - sum;
    pl.i = a;
    pl.seq0 = from;
    pl.seqs = 0;
    pl.len = 0;
    const bool mine = first <= pl.u0 && pl.u0 < upto;
    if (mine) {
        for (;; ++pl.i) {
            const int e = max(pl.seq0, pl.i == a ? end0 : end_of(p, pl.i));
            pl.len = pl.i == a ? len0 : len_of(p, pl.i);
            pl.seqs = e - pl.seq0;
            const uint32_t w = tiles_of(p, pl.seqs) * (uint32_t)p.H * (units_of<UNIT>(pl.len) + p.lead);
            if (pl.u0 < first + w) break;
            first += w;
            pl.seq0 = e;
        }
    }
    const int owner = __ffs(__ballot_sync(0xffffffffu, mine)) - 1;
    pl.i = __shfl_sync(0xffffffffu, pl.i, owner);
    pl.seq0 = __shfl_sync(0xffffffffu, pl.seq0, owner);
    pl.seqs = __shfl_sync(0xffffffffu, pl.seqs, owner);
    pl.len = __shfl_sync(0xffffffffu, pl.len, owner);
    first = __shfl_sync(0xffffffffu, first, owner);
    const uint32_t n_s = units_of<UNIT>(pl.len) + p.lead, tiles = tiles_of(p, pl.seqs);
    const uint32_t at = (pl.u0 - first) / n_s;
    pl.h = (int)(at / tiles);
    pl.tile = (int)(at - pl.h * tiles);
    pl.start = first + at * n_s;
    return pl;
}

// A piece of a tile that a block works on.
struct Piece {
    // rows of the tile in use (none or less: past the queries), from row0 of the group on
    int i, seq0, rows, h, row0, len, c0, c1;
    uint32_t slot, parts;  // parts: runs that share the tile, where it begins here
    bool whole, begins;
};
// The next piece of the run (false: none left), which then starts behind it.
template <int UNIT>
RKV_DEV bool next_piece(const Params& p, uint32_t run, int member, Place& pl, Piece& c) {
    while (pl.u0 < pl.u1) {
        c.i = pl.i;
        c.seq0 = pl.seq0;
        c.h = pl.h;
        c.row0 = (pl.tile * p.team + member) * p.tile;
        c.rows = min(p.tile, pl.seqs * p.R - c.row0);
        c.len = pl.len;
        const uint32_t n_s = units_of<UNIT>(c.len), lead = p.lead, n_l = n_s + lead;
        const uint32_t from = pl.u0 - pl.start, to = min(n_l, pl.u1 - pl.start);
        const uint32_t j = from > lead ? from - lead : 0, e = to > lead ? to - lead : 0;
        c.c0 = j * UNIT;
        c.c1 = e == n_s ? c.len : e * UNIT;
        c.whole = j == 0 && e == n_s;
        c.begins = j == 0;
        c.slot = 2 * (run * p.team + member) + (j > 0 ? 0 : 1);
        c.parts = j > 0 || c.whole || e == 0 ? 0 : run_of(pl, pl.start + n_l - 1) - run + 1;
        pl.u0 = pl.start + to;
        if (to == n_l) {
            pl.start += n_l;
            if (++pl.tile == (int)tiles_of(p, pl.seqs)) {
                pl.tile = 0;
                if (++pl.h == p.H) {
                    pl.h = 0;
                    do {
                        pl.seq0 += pl.seqs;
                        ++pl.i;
                        pl.seqs = pl.i <= p.P ? max(pl.seq0, end_of(p, pl.i)) - pl.seq0 : 1;
                    } while (pl.seqs == 0);
                    if (pl.u0 < pl.u1) pl.len = len_of(p, pl.i);
                }
            }
        }
        if (e > j) return true;
    }
    return false;
}
// Sequence, token and query head of row `row` of a group.
RKV_DEV void place_of_row(const Params& p, int seq0, int h, int row, int& s, int& tk, int& hd) {
    const int i = row / p.R, x = row - i * p.R;
    s = seq0 + i;
    tk = x / p.G;
    hd = h * p.G + x - tk * p.G;
}
// The rows (up to 256) and parts of a tile that has to be joined; 0: nothing to join.
RKV_DEV int join_of(int rows, uint32_t parts) { return parts == 0 ? 0 : rows | (int)(parts << 9); }
RKV_DEV int rows_of(int join) { return join & 511; }
RKV_DEV int parts_of(int join) { return join >> 9; }
RKV_DEV bool bad_length(const Params& p, const Piece& c) {
    return c.begins && c.h == 0 && c.row0 == 0 && c.i < p.P && p.lens[c.i] != c.len;
}

RKV_DEV void store4(float* p, float4 v) { *reinterpret_cast<float4*>(p) = v; }
RKV_DEV void store4(__nv_bfloat16* p, float4 v) {
    const __nv_bfloat162 a = __floats2bfloat162_rn(v.x, v.y), b = __floats2bfloat162_rn(v.z, v.w);
    *reinterpret_cast<uint2*>(p) = make_uint2(*reinterpret_cast<const uint32_t*>(&a),
                                              *reinterpret_cast<const uint32_t*>(&b));
}

// The join of a query's sums over its prefix (relative to 2^m: l, and v of values)
// with those over its sequence's own rows.
struct Joined {
    float fp, fo, inv, lse;
};
RKV_DEV Joined join_own(float m, float l, float2 own) {
    Joined j;
    const float mx = fmaxf(m, own.x);
    j.fp = weight(m, l, mx);
    j.fo = weight(own.x, own.y, mx);
    const float sum = l * j.fp + own.y * j.fo;
    j.inv = sum == 0.f ? 0.f : 1.f / sum;
    j.lse = sum == 0.f ? -INFINITY : (mx + log2f(sum)) * kLn2;
    return j;
}
RKV_DEV float4 join4(const Joined& j, float4 v, float4 o) {
    return make_float4((v.x * j.fp + o.x * j.fo) * j.inv, (v.y * j.fp + o.y * j.fo) * j.inv,
                       (v.z * j.fp + o.z * j.fo) * j.inv, (v.w * j.fp + o.w * j.fo) * j.inv);
}

// The pass over the prefixes on the tensor cores (k_prefix_tc.cu), and whether it takes
// a call's pools.
bool tc_takes(const PrefixArgs& a);
cudaError_t launch_tc(const Params& p, int d, cudaStream_t s);

}  // namespace prefix
}  // namespace rkv
