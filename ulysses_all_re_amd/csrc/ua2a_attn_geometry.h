// Index math of the attention operators (ua2a_attn.h): which positions a query
// sees, which tiles of keys a workgroup walks, and rotary angles.  Shared by
// the kernels (ua2a_attn_*.hip), the host code that fills it
// (ua2a_attn_host.cpp) and a CPU check that carries the calls out with it.
#pragma once

#include "ua2a_act_geometry.h"

namespace ua2a {

// -------------------------------------------------------------------- windows
// With c(x) = x / chunk a query at position p sees the positions j < end with
//   c(p) - left <= c(j) <= c(p) + right,  and j < sinks;
// with right = 0 nothing past its own chunk, sinks or not.  left, right < 0:
// no bound on that side.
struct WindowGeom {
    int32_t left, right, sinks;
    uint32_t chunk;
    Div32 d_chunk;
};

// What one query sees: [lo, hi) and [0, sk).
struct Seen {
    int32_t lo, hi, sk;
};

// Positions of a tile are unsigned: the last tile of the largest cache reaches 2^31.
UA2A_HD bool sees(const Seen& s, uint32_t j)
{
    return (j >= static_cast<uint32_t>(s.lo) && j < static_cast<uint32_t>(s.hi)) || j < static_cast<uint32_t>(s.sk);
}

// p in [0, end).  All three grow with p.
UA2A_HD Seen seen_by(const WindowGeom& g, int32_t p, int32_t end)
{
    const int64_t c = fdiv(static_cast<uint32_t>(p), g.d_chunk);
    Seen s;
    s.hi = end;
    if (g.right >= 0) {
        const int64_t hi = (c + g.right + 1) * g.chunk;
        if (hi < end) s.hi = static_cast<int32_t>(hi);
    }
    s.lo = 0;
    if (g.left >= 0 && c > g.left) s.lo = static_cast<int32_t>((c - g.left) * g.chunk);
    const int32_t most = g.right == 0 ? s.hi : end;
    s.sk = g.sinks < most ? g.sinks : most;
    return s;
}

// The queries that see a position of [k0, k1), all of them in [0, end): a range
// of positions that holds them (every one of it sees some, or lies between).
struct Span32 {
    int32_t first, last;
};

UA2A_HD Span32 seers_of(const WindowGeom& g, int32_t k0, int32_t k1, int32_t end)
{
    Span32 s;
    const int64_t c0 = fdiv(static_cast<uint32_t>(k0), g.d_chunk), c1 = fdiv(static_cast<uint32_t>(k1 - 1), g.d_chunk);
    s.first = 0;
    if (g.right >= 0 && c0 > g.right) {
        const int64_t lo = (c0 - g.right) * g.chunk;
        s.first = lo < end ? static_cast<int32_t>(lo) : end;
    }
    s.last = end;
    if (g.left >= 0) {
        const int64_t hi = (c1 + g.left + 1) * g.chunk;
        if (hi < end) s.last = static_cast<int32_t>(hi);
    }
    if (k0 < g.sinks) {
        s.last = end;
        if (g.right != 0) s.first = 0;
    }
    return s;
}

// -------------------------------------------------------------------- queries
// The queries of one key head: n tokens of a sequence times the `group` query
// heads that share it, row = token * group + member.  A unit is one key head
// of one sequence on one rank.
struct AttnGeom {
    WindowGeom win;
    uint32_t units;              // ranks * sequences * key heads of a rank
    uint32_t seqs;               // sequences of a rank
    uint32_t kvl, hl, group;     // key heads and query heads of a rank, hl = kvl * group
    uint32_t D, nb;
    uint32_t n;                  // query tokens of a sequence
    uint32_t rows;               // n * group, < 2^31
    uint32_t tiles;              // tiles of rows, or (backward, keys) of keys
    uint32_t keys;               // positions of a sequence
    uint32_t splits;             // parts of a walk
    uint32_t items;              // units * tiles * splits
    uint32_t order;              // 1: a unit's tiles from the last to the first
    Div32 d_splits, d_tiles, d_kvl, d_seqs, d_group, d_rows;
};

constexpr uint32_t kAttnXcds = 8;

// Workgroups go to the XCDs in turn; each XCD takes a stretch of consecutive
// items, so the workgroups that walk the same keys share an L2.
UA2A_HD uint32_t attn_item(const AttnGeom& g, uint32_t id)
{
    const uint32_t per = (g.items + kAttnXcds - 1) / kAttnXcds;
    const uint32_t i = id / kAttnXcds, item = (id % kAttnXcds) * per + i;
    return i < per && item < g.items ? item : g.items;
}

// Which of `tiles` comes i-th: where walks grow from tile to tile, the last first, so
// that what ends last is short.
UA2A_HD uint32_t tile_in_order(uint32_t order, uint32_t tiles, uint32_t i) { return order != 0 ? tiles - 1 - i : i; }

struct AttnPlace {
    uint32_t unit, tile, split;
    uint32_t seq;                // of all ranks: rank * seqs + sequence
    uint32_t kvh;                // key head of the rank
    uint32_t i;                  // sequence of the rank
};

UA2A_HD AttnPlace attn_place(const AttnGeom& g, uint32_t item)
{
    AttnPlace p;
    const uint32_t ut = fdiv(item, g.d_splits);
    p.split = item - ut * g.splits;
    p.unit = fdiv(ut, g.d_tiles);
    p.tile = tile_in_order(g.order, g.tiles, ut - p.unit * g.tiles);
    p.seq = fdiv(p.unit, g.d_kvl);
    p.kvh = p.unit - p.seq * g.kvl;
    p.i = p.seq - fdiv(p.seq, g.d_seqs) * g.seqs;
    return p;
}

// A sequence's query tokens that exist, [first, last), the position of token
// 0, and how many positions hold keys.
struct AttnSeq {
    int64_t start;
    int32_t first, last;
    int32_t end;
};

UA2A_HD AttnSeq attn_seq(const AttnGeom& g, int64_t start, int64_t count)
{
    AttnSeq s;
    s.start = start;
    const int64_t first = start < 0 ? -start : 0;
    int64_t last = count < static_cast<int64_t>(g.n) ? count : g.n;
    if (last > static_cast<int64_t>(g.keys) - start) last = static_cast<int64_t>(g.keys) - start;
    if (first >= last) {
        s.first = s.last = s.end = 0;
        return s;
    }
    s.first = static_cast<int32_t>(first);
    s.last = static_cast<int32_t>(last);
    s.end = static_cast<int32_t>(start + last);
    return s;
}

// The token of a row, moved to the nearest that exists; the sequence has one.
UA2A_HD int32_t near_token(const AttnGeom& g, const AttnSeq& s, uint32_t row)
{
    int32_t t = static_cast<int32_t>(fdiv(row, g.d_group));
    if (t < s.first) t = s.first;
    return t < s.last ? t : s.last - 1;
}

UA2A_HD Seen seen_by_row(const AttnGeom& g, const AttnSeq& s, uint32_t row)
{
    return seen_by(g.win, static_cast<int32_t>(s.start + near_token(g, s, row)), s.end);
}

// The tiles of `size` keys that rows see of whose first row sees `a`, and
// whose last `b`: [0, sinks) and [from, to).
struct KeyWalk {
    uint32_t sinks, from, total;
};

UA2A_HD KeyWalk key_walk(const Seen& a, const Seen& b, uint32_t size)
{
    KeyWalk w;
    w.sinks = (static_cast<uint32_t>(b.sk) + size - 1) / size;
    w.from = static_cast<uint32_t>(a.lo) / size;
    if (w.from < w.sinks) w.from = w.sinks;
    const uint32_t to = (static_cast<uint32_t>(b.hi) + size - 1) / size;
    w.total = w.sinks + (to > w.from ? to - w.from : 0);
    return w;
}

UA2A_HD uint32_t walk_tile(const KeyWalk& w, uint32_t i) { return i < w.sinks ? i : w.from + (i - w.sinks); }

// Part `split` of `splits` of a walk: [first, last).
UA2A_HD uint32_t split_at(uint32_t total, uint32_t splits, uint32_t split)
{
    return static_cast<uint32_t>(static_cast<uint64_t>(total) * split / splits);
}

// Whether each (all) or any of the rows between those that see `a` and `b` sees
// a position of [k0, k1).
UA2A_HD bool all_seen(const Seen& a, const Seen& b, uint32_t k0, uint32_t k1)
{
    return (static_cast<uint32_t>(b.lo) <= k0 && k1 <= static_cast<uint32_t>(a.hi)) || k1 <= static_cast<uint32_t>(a.sk);
}
UA2A_HD bool none_seen(const Seen& a, const Seen& b, uint32_t k0, uint32_t k1)
{
    return (k0 >= static_cast<uint32_t>(b.hi) || k1 <= static_cast<uint32_t>(a.lo)) && k0 >= static_cast<uint32_t>(b.sk);
}

// How a workgroup of 256 lanes joins rows' parts: `wide` lanes (four values each)
// take kJoinEach parts at a time, `at_once` such groups a row, `rows` rows.
constexpr uint32_t kJoinEach = 8;
struct JoinShape {
    uint32_t wide, at_once, rows;
};

UA2A_HD JoinShape join_shape(const AttnGeom& g)
{
    JoinShape s;
    s.wide = g.D > 64 ? 32 : g.D > 32 ? 16 : 8;
    const uint32_t groups = 256 / s.wide;
    s.at_once = 1;
    while (s.at_once * kJoinEach < g.splits && s.at_once < groups) s.at_once *= 2;
    s.rows = groups / s.at_once;
    return s;
}

// ------------------------------------------------------------- keys' gradients
// A unit's tiles of keys: the first `lead` (span keys) are walked in lead_parts
// parts each, the others in rest_parts.  Parts' sums lie in the workspace, the
// lead tiles' first, [parts][units][keys] each.
struct KeyTiles {
    uint32_t lead, span;
    uint32_t lead_parts, rest_parts;
    uint32_t per_unit;           // lead * lead_parts + (tiles - lead) * rest_parts
    Div32 d_per_unit, d_lead_parts, d_rest_parts;
    int64_t rest_line;           // where the other tiles' sums start, in keys
    uint32_t per_group;          // join: keys of a workgroup, D / 2 lanes each
    Div32 d_lanes, d_keys;       // ... by D / 2, and by the keys of a unit that may have parts
};

struct KeyPlace {
    AttnPlace at;
    uint32_t parts;              // of the tile's walk
};

UA2A_HD KeyPlace key_place(const AttnGeom& g, const KeyTiles& t, uint32_t item)
{
    KeyPlace p;
    p.at.unit = fdiv(item, t.d_per_unit);
    uint32_t i = item - p.at.unit * t.per_unit;
    const uint32_t leading = t.lead * t.lead_parts;
    if (i < leading) {
        p.at.tile = fdiv(i, t.d_lead_parts);
        p.at.split = i - p.at.tile * t.lead_parts;
        p.parts = t.lead_parts;
    } else {
        i -= leading;
        const uint32_t tile = fdiv(i, t.d_rest_parts);
        p.at.split = i - tile * t.rest_parts;
        p.at.tile = t.lead + tile_in_order(g.order, g.tiles - t.lead, tile);
        p.parts = t.rest_parts;
    }
    p.at.seq = fdiv(p.at.unit, g.d_kvl);
    p.at.kvh = p.at.unit - p.at.seq * g.kvl;
    p.at.i = p.at.seq - fdiv(p.at.seq, g.d_seqs) * g.seqs;
    return p;
}

// Where part `split` of key j keeps its sums, in keys of dk's and dv's values.
UA2A_HD int64_t part_line(const AttnGeom& g, const KeyTiles& t, uint32_t unit, uint32_t split, uint32_t j)
{
    const int64_t of = static_cast<int64_t>(split) * g.units + unit;
    return j < t.span ? of * t.span + j : t.rest_line + of * (g.keys - t.span) + (j - t.span);
}

// The tiles of `size` rows that hold the rows of tokens [first, last).
struct RowWalk {
    uint32_t from, total;
};

UA2A_HD RowWalk row_walk(const AttnGeom& g, const Span32& s, uint32_t size)
{
    RowWalk w;
    w.from = static_cast<uint32_t>(s.first) * g.group / size;
    const uint32_t to = (static_cast<uint32_t>(s.last) * g.group + size - 1) / size;
    w.total = to > w.from ? to - w.from : 0;
    return w;
}

// --------------------------------------------------------------------- rotary
// Pair i of a head turns by position * turns[i] / 2^64 turns: a position's
// angle modulo a turn is then the product modulo 2^64, exactly.
struct RopeGeom {
    ActShape sh;
    uint32_t pairs;              // pairs that turn, of values 2i and 2i + 1, or (halves) i and i + pairs
    uint32_t halves;
    uint32_t inverse;
    uint32_t from_a, to_a;       // layouts: 1 for A
    uint32_t per_plane;          // positions [naxes][B][SG], else [naxes][SG]
    uint32_t naxes;
    int64_t axis_stride;         // positions of an axis
    uint32_t tokens;             // w * B * S
    uint32_t slots;              // lane slots of a head
    uint32_t turning;            // ... that hold pairs; the others are copied
    uint32_t heads_at_once;      // heads that a token's lanes take at once
    uint32_t lanes;              // of a token
    uint32_t per_group;          // tokens of a workgroup
    Div32 d_lanes, d_slots, d_SG, d_pairs;
};

}  // namespace ua2a
