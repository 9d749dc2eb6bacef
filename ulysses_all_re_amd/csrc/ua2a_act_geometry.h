// Index math of the activation operators: norms joined with the exchange and
// the 8-bit cache.  Shared by the kernels (ua2a_act_*.hip), the host
// code that fills it (ua2a_act_host.cpp) and a CPU check that walks every lane.
//
// Two layouts of one tensor (see ua2a.h): P [w][B][S][H][D] and
// A [w][B][S*w][H/w][D].  Head h of token (j, b, s) starts at element
//   P: ((j*B + b)*S + s)*H*D + h*D
//   A: (h / hl)*a_rank + ((b*S*w + j*S + s)*hl + h % hl)*D,  hl = H/w, a_rank = B*S*w*hl*D
// 8-bit tensors hold one code per value in the same places, and one scale per
// block of 32 values along D (a head's last block may be shorter): the same
// places again with D replaced by nb = ceil(D / 32).
#pragma once

#include "ua2a_geometry.h"

namespace ua2a {

constexpr uint32_t kBlockValues = 32;    // values that share a scale

// What the two layouts' offsets are made of.
struct ActShape {
    uint32_t H, D, nb, hl;
    uint32_t S, B, SG;           // SG = S * w
    Div32 d_hl, d_S, d_B, d_run;
    uint32_t run;                // hl * D: values of a token on one A rank
    int64_t a_rank;              // A: values from one rank to the next
    int64_t a_rank_scales;       // ... and scales
};

// Where one token's heads lie: element (or scale) offset of head h is
//   P: p * H * D + h * D;   A: (h / hl) * a_rank + (a * hl + h % hl) * D.
struct TokenPlace {
    uint32_t p;                  // token of the P side, (j*B + b)*S + s
    uint32_t a;                  // row of every A rank, b*SG + j*S + s
};

UA2A_HD TokenPlace token_place(const ActShape& g, uint32_t token)
{
    const uint32_t jb = fdiv(token, g.d_S);
    const uint32_t s = token - jb * g.S;
    const uint32_t j = fdiv(jb, g.d_B);
    const uint32_t b = jb - j * g.B;
    return TokenPlace{token, b * g.SG + j * g.S + s};
}

// Element offset of value d of head h on the A side; with per = nb and
// rank = a_rank_scales, the offset of scale d.
UA2A_HD int64_t a_offset(const ActShape& g, uint32_t arow, uint32_t h, uint32_t per, int64_t rank, uint32_t d)
{
    const uint32_t r = fdiv(h, g.d_hl);
    const uint32_t k = h - r * g.hl;
    return static_cast<int64_t>(r) * rank + (static_cast<int64_t>(arow) * g.hl + k) * per + d;
}

// The A offset of value e of a token's H * D.
UA2A_HD int64_t a_offset_of_value(const ActShape& g, uint32_t e)
{
    const uint32_t r = fdiv(e, g.d_run);
    return static_cast<int64_t>(r) * g.a_rank + (e - r * g.run);
}

// --------------------------------------------------------------------- norms
// A segment is what `lanes` lanes work on together: a token's H heads where
// one norm covers them all, or a head that is a norm by itself; or a bundle of
// heads with a norm each, 2^head_log lanes apiece.  Its lanes are a power of
// two, or a workgroup of whole waves.  The unit of a
// lane is a slot of V consecutive values of one head.  A block of 32 values is
// 32/V slots, and heads are padded to whole blocks (in bundles to 2^head_log
// slots), so a block's slots are consecutive lanes, aligned to 32/V: its
// largest value is found by exchanging lanes in a group.
struct NormGeom {
    ActShape sh;
    uint32_t cols;               // values of the weight: H*D, with a norm per head D
    uint32_t heads;              // heads of a segment
    uint32_t per_token;          // segments of a token
    uint32_t slots;              // slots of a segment, padding included
    uint32_t q_log;              // slots of a block = 2^q_log
    uint32_t head_log;           // bundles: slots of a head = 2^head_log; else 0
    uint32_t padded;             // 1: some lanes' slots are padding
    uint32_t dense;              // 1: heads are whole blocks, so slot k holds values k*V .. of the segment
    uint32_t lanes;
    uint32_t per_log;            // segments of a workgroup = 2^per_log
    uint32_t segs;               // segments in all
    uint32_t groups;             // workgroups' worth of segments
    Div32 d_nb, d_per;
};

struct Slot {
    uint32_t hh;                 // head within the segment
    uint32_t blk;                // block within the head
    uint32_t d;                  // first value within the head
    uint32_t ok;                 // 0: padding
};

UA2A_HD Slot slot_at(const NormGeom& g, uint32_t slot, uint32_t hh, uint32_t blk, uint32_t V)
{
    Slot s;
    s.hh = hh;
    s.blk = blk;
    s.d = blk * kBlockValues + (slot & ((1u << g.q_log) - 1)) * V;
    s.ok = (slot < g.slots && s.d < g.sh.D) ? 1u : 0u;
    return s;
}

UA2A_HD Slot bundle_slot(const NormGeom& g, uint32_t slot, uint32_t V)
{
    return slot_at(g, slot, slot >> g.head_log, (slot & ((1u << g.head_log) - 1)) >> g.q_log, V);
}

UA2A_HD Slot norm_slot(const NormGeom& g, uint32_t slot, uint32_t V)
{
    const uint32_t b = slot >> g.q_log;
    const uint32_t hh = fdiv(b, g.d_nb);
    return slot_at(g, slot, hh, b - hh * g.sh.nb, V);
}

// What a lane needs of one segment: the token's places, its first head, and
// whether there is one (lanes past the last segment look at the first).
struct Segment {
    TokenPlace at;
    uint32_t h0;
    uint32_t seg;
    uint32_t live;
};

UA2A_HD Segment segment_of(const NormGeom& g, uint32_t group, uint32_t within)
{
    const uint32_t seg = (group << g.per_log) + within;         // within: segment of the workgroup
    Segment s;
    s.live = seg < g.segs ? 1u : 0u;
    s.seg = s.live ? seg : 0u;
    const uint32_t token = fdiv(s.seg, g.d_per);
    s.h0 = (s.seg - token * g.per_token) * g.heads;
    s.at = token_place(g.sh, token);
    return s;
}

// Offset of a slot's first value, and of its block's scale, on the P or the A side.
UA2A_HD int64_t value_at(const NormGeom& g, const Segment& s, const Slot& sl, bool a_side)
{
    const uint32_t h = s.h0 + sl.hh;
    if (a_side) return a_offset(g.sh, s.at.a, h, g.sh.D, g.sh.a_rank, sl.d);
    return (static_cast<int64_t>(s.at.p) * g.sh.H + h) * g.sh.D + sl.d;
}

UA2A_HD int64_t scale_at(const NormGeom& g, const Segment& s, const Slot& sl, bool a_side)
{
    const uint32_t h = s.h0 + sl.hh;
    if (a_side) return a_offset(g.sh, s.at.a, h, g.sh.nb, g.sh.a_rank_scales, sl.blk);
    return (static_cast<int64_t>(s.at.p) * g.sh.H + h) * g.sh.nb + sl.blk;
}

// How a norm's segments lie on lanes: one norm on part of a wave (a power of
// two of lanes, so several share it), on a workgroup, or on one, two or four
// waves of a workgroup of four; bundles of heads on a wave, or several bundles
// sharing one.
constexpr int32_t kSpanPart = 0, kSpanWide = 1, kSpanWaves = 2, kSpanBundle = 3, kSpanBundles = 4;
enum Span { kPart = kSpanPart, kWide = kSpanWide, kWaves = kSpanWaves, kBundle = kSpanBundle, kBundles = kSpanBundles };
UA2A_HD constexpr bool one_norm(Span s) { return s == kPart || s == kWide || s == kWaves; }

// The lane of the segment, and the segment of the workgroup, of a workgroup's lane.
template <Span SPAN>
UA2A_HD uint32_t segment_lane(const NormGeom& g, uint32_t tid)
{
    return SPAN == kWide ? tid : tid & (g.lanes - 1);
}
template <Span SPAN>
UA2A_HD uint32_t segment_within(const NormGeom& g, uint32_t tid)
{
    if constexpr (SPAN == kWide) return 0;
    return tid >> (31 - __builtin_clz(g.lanes));
}

// What a lane needs to know of its slots, whatever the segment: offsets from
// the segment's first value on either side, and which slots are no padding
// (those look at the segment's first value and are not counted).  The A
// offset counts the heads' ranks, so it has 64 bits; a bundle may start at any
// head, so its A offsets are worked out for each.
template <int ITEMS>
struct LaneSlots {
    int64_t a[ITEMS];
    uint32_t p[ITEMS];
    uint32_t ok;                 // bit per slot
};

template <Span SPAN, int V>
UA2A_HD Slot slot_of(const NormGeom& g, uint32_t lane, int it)
{
    const uint32_t slot = lane + static_cast<uint32_t>(it) * g.lanes;
    return one_norm(SPAN) ? norm_slot(g, slot, V) : bundle_slot(g, slot, V);
}

template <Span SPAN, int V, int ITEMS>
UA2A_HD LaneSlots<ITEMS> lane_slots(const NormGeom& g, uint32_t lane)
{
    LaneSlots<ITEMS> l;
    l.ok = 0;
    if (one_norm(SPAN) && g.dense) {
#pragma unroll
        for (int it = 0; it < ITEMS; ++it) {
            const uint32_t slot = lane + static_cast<uint32_t>(it) * g.lanes;
            const bool ok = slot < g.slots;
            l.p[it] = ok ? slot * V : 0;
            l.a[it] = a_offset_of_value(g.sh, l.p[it]);
            l.ok |= (ok ? 1u : 0u) << it;
        }
        return l;
    }
#pragma unroll
    for (int it = 0; it < ITEMS; ++it) {
        const Slot s = slot_of<SPAN, V>(g, lane, it);
        l.p[it] = s.ok ? s.hh * g.sh.D + s.d : 0;
        l.a[it] = s.ok && one_norm(SPAN) ? a_offset(g.sh, 0, s.hh, g.sh.D, g.sh.a_rank, s.d) : 0;
        l.ok |= s.ok << it;
    }
    return l;
}

// Offset of a slot's weights: of the segment's values, in bundles of a head's.
template <Span SPAN, int V, int ITEMS>
UA2A_HD uint32_t weight_offset(const NormGeom& g, const LaneSlots<ITEMS>& l, uint32_t lane, int it)
{
    if constexpr (one_norm(SPAN)) return l.p[it];
    return l.ok & 1 ? slot_of<SPAN, V>(g, lane, 0).d : 0;
}

// A segment's first value (and scale) on either side; for bundles the A side
// is the row's first head of a rank, and h0 the segment's first head.
struct SegmentBase {
    int64_t p, a, ps, as;
    uint32_t seg;
    uint32_t token;
    uint32_t h0;
    bool live;
};

template <Span SPAN>
UA2A_HD SegmentBase segment_base(const NormGeom& g, uint32_t group, uint32_t within)
{
    const Segment s = segment_of(g, group, within);
    const Slot first = {0, 0, 0, 1};
    SegmentBase b;
    b.p = value_at(g, s, first, false);
    b.ps = scale_at(g, s, first, false);
    if constexpr (one_norm(SPAN)) {
        b.a = value_at(g, s, first, true);
        b.as = scale_at(g, s, first, true);
    } else {
        b.a = static_cast<int64_t>(s.at.a) * g.sh.hl * g.sh.D;
        b.as = static_cast<int64_t>(s.at.a) * g.sh.hl * g.sh.nb;
    }
    b.seg = s.seg;
    b.token = s.at.p;
    b.h0 = s.h0;
    b.live = s.live;
    return b;
}

// Where the segment's offsets are used: on the A side a bundle's depend on its
// first head; scales' are worked out on the spot, for only calls with 8 bits
// ask for them.
template <Span SPAN, int V, int ITEMS>
struct SlotPlaces {
    const NormGeom& g;
    const SegmentBase& s;
    const LaneSlots<ITEMS>& l;
    uint32_t lane;

    UA2A_HD Slot slot(int it) const { return slot_of<SPAN, V>(g, lane, it); }
    UA2A_HD bool ok(int it) const { return l.ok >> it & 1; }
    UA2A_HD uint32_t p(int it) const { return l.p[it]; }
    UA2A_HD int64_t a(int it) const
    {
        if constexpr (one_norm(SPAN)) return l.a[it];
        const Slot sl = slot(it);
        return sl.ok ? a_offset(g.sh, 0, s.h0 + sl.hh, g.sh.D, g.sh.a_rank, sl.d) : 0;
    }
    UA2A_HD uint32_t scale_p(int it) const
    {
        if (!ok(it)) return 0;
        // one norm: blocks in the order of the slots
        if constexpr (one_norm(SPAN)) return (lane + static_cast<uint32_t>(it) * g.lanes) / (kBlockValues / V);
        const Slot sl = slot(it);
        return sl.hh * g.sh.nb + sl.blk;
    }
    UA2A_HD int64_t scale_a(int it) const
    {
        const Slot sl = slot(it);
        return a_offset(g.sh, 0, (one_norm(SPAN) ? 0 : s.h0) + sl.hh, g.sh.nb, g.sh.a_rank_scales, sl.blk);
    }
    // index of the slot's rstd
    UA2A_HD uint32_t stat(int it) const
    {
        if constexpr (one_norm(SPAN)) return s.seg;
        return s.token * g.sh.H + s.h0 + (ok(it) ? slot(it).hh : 0);
    }
};

// --------------------------------------------------------------------- cache
// Codes [2][w][seqs][cap][hl][D], scales [2][w][seqs][cap][hl][nb].  A call's
// token t of sequence i has position starts[i] + t; it exists when
// t < counts[i] and the position lies in [0, cap).
struct CacheGeom {
    ActShape sh;
    uint32_t seqs, each;         // sequences, tokens of each in this call
    uint32_t dense;              // 1: heads are whole blocks
    uint32_t q_log;
    int64_t cap;
    int64_t part;                // values from the keys' codes to the values' codes
    int64_t part_scales;
    Div32 d_nb, d_each, d_D;
    // write: a token's slots (as a norm's, heads padded to whole blocks) lie on
    // `lanes` lanes, a power of two, or on `chunks` workgroups
    uint32_t rows, slots, lanes, chunks, per_log, groups;
    uint32_t run_log;            // 2^run_log consecutive workgroups per XCD in turn
    Div32 d_chunks;
    // read: a sequence's tokens on one rank are one span of values on both
    // sides, cut into tiles of one vector per lane
    uint32_t spans, tiles;
    Div32 d_tiles, d_seqs;
};

constexpr uint32_t kCacheXcds = 8;

// A cache launch's workgroups: up to 2^kCacheGridLog along x (2^31 lanes of
// workgroups of 256), the rest along y.
constexpr uint32_t kCacheGridLog = 23;
UA2A_HD uint32_t cache_workgroup(uint32_t x, uint32_t y) { return (y << kCacheGridLog) + x; }

// The group of tokens of a write's workgroup: workgroups go to the XCDs in
// turn, and 2^run_log consecutive groups to one of them.
UA2A_HD uint32_t cache_group(const CacheGeom& g, uint32_t id)
{
    const uint32_t xcd = id % kCacheXcds, q = id / kCacheXcds;
    return ((((q >> g.run_log) * kCacheXcds) + xcd) << g.run_log) + (q & ((1u << g.run_log) - 1));
}

struct WriteLane {
    uint32_t token;              // of P
    uint32_t slot;               // of the token
    uint32_t in;                 // 0: none
};

// within: the lanes' part of the workgroup, tid / lanes.
UA2A_HD WriteLane write_lane(const CacheGeom& g, uint32_t group, uint32_t within, uint32_t tid)
{
    const uint32_t seg = (group << g.per_log) + within;
    WriteLane l;
    l.token = fdiv(seg, g.d_chunks);
    l.slot = (seg - l.token * g.chunks) * g.lanes + (tid & (g.lanes - 1));
    l.in = (l.token < g.rows && l.slot < g.slots) ? 1u : 0u;
    return l;
}

// A sequence's tokens in this call that exist: [first, last), positions from `start`.
struct CacheSpan {
    int64_t start;
    int64_t first, last;
};

UA2A_HD CacheSpan cache_span(const CacheGeom& g, int64_t start, int64_t count)
{
    CacheSpan s;
    s.start = start;
    s.first = s.start < 0 ? -s.start : 0;
    s.last = count;
    if (s.last > static_cast<int64_t>(g.each)) s.last = g.each;
    if (s.last > g.cap - s.start) s.last = g.cap - s.start;
    return s;
}

// The scale of value e0 + f of a span of whole heads, e0 uniform, f < 2^16: the
// head by 32-bit arithmetic but for spans past 2^32 values.
UA2A_HD int64_t scale_of_value(const CacheGeom& g, int64_t e0, uint32_t f)
{
    const int64_t h0 = (e0 >> 32) == 0 ? static_cast<int64_t>(fdiv(static_cast<uint32_t>(e0), g.d_D)) : e0 / g.sh.D;
    const uint32_t x = static_cast<uint32_t>(e0 - h0 * g.sh.D) + f;             // < D + 2^16
    const uint32_t h = fdiv(x, g.d_D);
    return (h0 + h) * g.sh.nb + (x - h * g.sh.D) / kBlockValues;
}

}  // namespace ua2a
