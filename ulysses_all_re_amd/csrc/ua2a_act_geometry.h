// Index math of the activation operators: norms joined with the exchange and
// the 8-bit cache.  Shared by the kernels (ua2a_act_kernels.hip), the host
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

// --------------------------------------------------------------------- cache
// Codes [2][w][seqs][cap][hl][D], scales [2][w][seqs][cap][hl][nb].  A call's
// token t of sequence i has position starts[i] + t; it exists when
// t < counts[i] and the position lies in [0, cap).
struct CacheGeom {
    ActShape sh;
    uint32_t w;
    uint32_t seqs, each;         // sequences, tokens of each in this call
    int64_t cap;
    uint32_t q_log;
    uint32_t slots;              // slots of a row: write, one token's H heads; read, one rank's hl heads
    uint32_t rows;               // write: tokens; read: w * seqs * each
    int64_t part;                // values from the keys' codes to the values' codes
    int64_t part_scales;
    Div32 d_nb, d_slots, d_each, d_seqs;
};

// One lane's slot of a cache call, for slot idx < rows * slots.
struct CacheSlot {
    uint32_t row;                // write: token of P; read: row of the output
    uint32_t h;                  // head of the row: of all H (write), of the rank's (read)
    uint32_t blk, d;             // block, first value (d >= D: padding)
    uint32_t r, i, t;            // rank, sequence, token of the sequence
};

UA2A_HD CacheSlot cache_slot(const CacheGeom& g, uint32_t idx, uint32_t V, bool write)
{
    CacheSlot c;
    c.row = fdiv(idx, g.d_slots);
    const uint32_t slot = idx - c.row * g.slots;
    const uint32_t b = slot >> g.q_log;
    c.h = fdiv(b, g.d_nb);
    c.blk = b - c.h * g.sh.nb;
    c.d = c.blk * kBlockValues + (slot & ((1u << g.q_log) - 1)) * V;
    if (write) {
        const uint32_t a = token_place(g.sh, c.row).a;
        c.i = fdiv(a, g.d_each);
        c.t = a - c.i * g.each;
        c.r = fdiv(c.h, g.sh.d_hl);
    } else {
        const uint32_t ri = fdiv(c.row, g.d_each);
        c.t = c.row - ri * g.each;
        c.r = fdiv(ri, g.d_seqs);
        c.i = ri - c.r * g.seqs;
    }
    return c;
}

// Row of the cache, counted over its [w][seqs][cap] rows, for a slot's token;
// -1 where there is none.  starts null: 0; counts null: all of the call's.
UA2A_HD int64_t cache_row(const CacheGeom& g, const CacheSlot& s, const int32_t* starts, const int32_t* counts)
{
    const int64_t pos = (starts ? static_cast<int64_t>(starts[s.i]) : 0) + s.t;
    const int64_t count = counts ? static_cast<int64_t>(counts[s.i]) : static_cast<int64_t>(g.each);
    if (static_cast<int64_t>(s.t) >= count || pos < 0 || pos >= g.cap) return -1;
    return (static_cast<int64_t>(s.r) * g.seqs + s.i) * g.cap + pos;
}

}  // namespace ua2a
