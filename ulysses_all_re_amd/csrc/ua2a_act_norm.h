// What the norm kernels, forward and backward, share: the lanes' places in a
// segment and the weights.
#pragma once

#include "ua2a_act_device.h"

namespace ua2a {
namespace {

enum Span { kPart = kSpanPart, kWide = kSpanWide, kWaves = kSpanWaves, kBundle = kSpanBundle, kBundles = kSpanBundles };
constexpr bool one_norm(Span s) { return s == kPart || s == kWide || s == kWaves; }

// The lane of the segment, and the segment of the workgroup.  A segment of
// whole waves is the same in every lane, so what follows from it is scalar.
template <Span SPAN>
__device__ __forceinline__ uint32_t segment_lane(const NormGeom& g)
{
    return SPAN == kWide ? threadIdx.x : threadIdx.x & (g.lanes - 1);
}
template <Span SPAN>
__device__ __forceinline__ uint32_t segment_within(const NormGeom& g)
{
    if constexpr (SPAN == kWide) return 0;
    uint32_t tid = threadIdx.x;
    if constexpr (SPAN == kWaves || SPAN == kBundle) tid = __builtin_amdgcn_readfirstlane(tid);
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
__device__ __forceinline__ Slot slot_of(const NormGeom& g, uint32_t lane, int it)
{
    const uint32_t slot = lane + static_cast<uint32_t>(it) * g.lanes;
    return one_norm(SPAN) ? norm_slot(g, slot, V) : bundle_slot(g, slot, V);
}

template <Span SPAN, int V, int ITEMS>
__device__ __forceinline__ LaneSlots<ITEMS> lane_slots(const NormGeom& g, uint32_t lane)
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
__device__ __forceinline__ uint32_t weight_offset(const NormGeom& g, const LaneSlots<ITEMS>& l, uint32_t lane, int it)
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
__device__ __forceinline__ SegmentBase segment_base(const NormGeom& g, uint32_t group)
{
    const Segment s = segment_of(g, group, segment_within<SPAN>(g));
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
struct Places {
    const NormGeom& g;
    const SegmentBase& s;
    LaneSlots<ITEMS>& l;
    uint32_t lane;

    __device__ __forceinline__ Places(const NormGeom& g_, const SegmentBase& s_, LaneSlots<ITEMS>& l_, uint32_t lane_)
        : g(g_), s(s_), l(l_), lane(lane_)
    {
        // nothing derived from these is kept from one segment to the next
        forget(lane);
#pragma unroll
        for (int it = 0; it < ITEMS; ++it) {
            forget(l.a[it]);
            forget(l.p[it]);
        }
    }
    __device__ __forceinline__ Slot slot(int it) const
    {
        return slot_of<SPAN, V>(g, lane, it);
    }
    __device__ __forceinline__ bool ok(int it) const { return l.ok >> it & 1; }
    __device__ __forceinline__ uint32_t p(int it) const { return l.p[it]; }
    __device__ __forceinline__ int64_t a(int it) const
    {
        if constexpr (one_norm(SPAN)) return l.a[it];
        const Slot sl = slot(it);
        return sl.ok ? a_offset(g.sh, 0, s.h0 + sl.hh, g.sh.D, g.sh.a_rank, sl.d) : 0;
    }
    __device__ __forceinline__ uint32_t scale_p(int it) const
    {
        if (!ok(it)) return 0;
        // one norm: blocks in the order of the slots
        if constexpr (one_norm(SPAN)) return (lane + static_cast<uint32_t>(it) * g.lanes) / (kBlockValues / V);
        const Slot sl = slot(it);
        return sl.hh * g.sh.nb + sl.blk;
    }
    __device__ __forceinline__ int64_t scale_a(int it) const
    {
        const Slot sl = slot(it);
        return a_offset(g.sh, 0, (one_norm(SPAN) ? 0 : s.h0) + sl.hh, g.sh.nb, g.sh.a_rank_scales, sl.blk);
    }
    // index of the slot's rstd
    __device__ __forceinline__ uint32_t stat(int it) const
    {
        if constexpr (one_norm(SPAN)) return s.seg;
        return s.token * g.sh.H + s.h0 + (ok(it) ? slot(it).hh : 0);
    }
};

// The weights of a lane's slots as they are stored (W is the type or float);
// the ones of a norm without weights are not looked at.  They may start at any
// value (a view into a flat buffer of parameters): the loads are the same whole
// vectors, which global memory takes at any address.
template <class W, int V>
struct Weights {
    static constexpr int kRaws = sizeof(W) * V / 16 > 0 ? sizeof(W) * V / 16 : 1;
    typename Raw<W, V == 1 ? 1 : 16 / sizeof(W)>::type raw[kRaws];
    __device__ __forceinline__ void load(const void* weight, uint32_t at)
    {
        typedef typename Raw<W, V == 1 ? 1 : 16 / sizeof(W)>::type R;
        typedef R Anywhere __attribute__((aligned(sizeof(W))));
        const Anywhere* p = reinterpret_cast<const Anywhere*>(static_cast<const W*>(weight) + at);
#pragma unroll
        for (int k = 0; k < kRaws; ++k) raw[k] = p[k];
    }
    __device__ __forceinline__ void get(float (&f)[V])
    {
        constexpr int N = V == 1 ? 1 : 16 / sizeof(W);
#pragma unroll
        for (int k = 0; k < kRaws; ++k) {
            forget(raw[k]);
            float part[N];
            unpack<W, N>(raw[k], part);
#pragma unroll
            for (int i = 0; i < N; ++i) f[k * N + i] = part[i];
        }
    }
};

// Sum over the lanes of a segment, in every lane of it; segments wider than a
// wave join their waves' sums through LDS, in the waves' order.  `red` holds
// one sum per wave, for two rounds in turn: a wave writes round n + 2 only
// after the barrier of round n + 1, which every wave reaches with round n
// read.
template <Span SPAN>
__device__ __forceinline__ float segment_sum(float x, uint32_t lanes, float (*red)[16], uint32_t round)
{
    if constexpr (SPAN == kPart) return group_sum(x, lanes);
    x = group_sum(x, 64);
    if (lanes <= 64) return x;
    const uint32_t wave = threadIdx.x >> 6;
    const uint32_t waves = lanes >> 6;
    float* r = red[round & 1];
    if ((threadIdx.x & 63) == 0) r[wave] = x;
    __syncthreads();
    const uint32_t first = SPAN == kWide ? 0 : wave & ~(waves - 1);
    x = 0.f;
    for (uint32_t k = 0; k < waves; ++k) x += r[first + k];
    return x;
}

// Sums over a slot's norm: bundles sum each slot over its head's lanes,
// others all slots over the segment's.
template <Span SPAN, int ITEMS>
__device__ __forceinline__ void norm_sums(const NormGeom& g, float (&x)[ITEMS], float (*red)[16], uint32_t round)
{
    if constexpr (one_norm(SPAN)) {
        float t = x[0];
#pragma unroll
        for (int it = 1; it < ITEMS; ++it) t += x[it];
        t = segment_sum<SPAN>(t, g.lanes, red, round);
#pragma unroll
        for (int it = 0; it < ITEMS; ++it) x[it] = t;
    } else {
#pragma unroll
        for (int it = 0; it < ITEMS; ++it) x[it] = group_sum(x[it], 1u << g.head_log);
    }
}

}  // namespace

// K<T, W, V, span, slots per lane, most lanes of a workgroup>::fn() for a
// launch.  The forward kernels have one slot per lane wherever a workgroup
// holds the norm; the backward ones keep sums per slot, so several.
template <class T, class W, int V, template <class, class, int, Span, int, int> class K>
const void* norm_pick(const ActLaunch& L)
{
    if (L.span == kPart) return K<T, W, V, kPart, 1, kActBlock>::fn();
    if (L.span == kWide) {
        switch (L.items) {
        case 1: return K<T, W, V, kWide, 1, kActBigBlock>::fn();
        case 2: return K<T, W, V, kWide, 2, kActBigBlock>::fn();
        case 4: return K<T, W, V, kWide, 4, kActBigBlock>::fn();
        case 8: return K<T, W, V, kWide, 8, kActBigBlock>::fn();
        }
    }
    if constexpr (V > 1) {
        if (L.span == kBundle && L.items == 1) return K<T, W, V, kBundle, 1, kActBlock>::fn();
        if (L.span == kBundles && L.items == 1) return K<T, W, V, kBundles, 1, kActBlock>::fn();
        if constexpr (K<T, W, V, kPart, 1, kActBlock>::kManyItems) {
            if (L.span == kBundle && L.items == 2) return K<T, W, V, kBundle, 2, kActBlock>::fn();
            if (L.span == kWaves) switch (L.items) {
                case 2: return K<T, W, V, kWaves, 2, kActBlock>::fn();
                case 3: return K<T, W, V, kWaves, 3, kActBlock>::fn();
                case 4: return K<T, W, V, kWaves, 4, kActBlock>::fn();
                case 5: return K<T, W, V, kWaves, 5, kActBlock>::fn();
                }
        }
    }
    return nullptr;
}

// The kernel of a launch's type, weight type and lanes.
template <template <class, class, int, Span, int, int> class K>
const void* norm_pick_type(const ActLaunch& L, bool weight_f32)
{
    if (L.type == UA2A_TYPE_BF16) {
        if (weight_f32) return L.V == 8 ? norm_pick<__bf16, float, 8, K>(L) : norm_pick<__bf16, float, 1, K>(L);
        return L.V == 8 ? norm_pick<__bf16, __bf16, 8, K>(L) : norm_pick<__bf16, __bf16, 1, K>(L);
    }
    if (L.type == UA2A_TYPE_FP16) {
        if (weight_f32) return L.V == 8 ? norm_pick<_Float16, float, 8, K>(L) : norm_pick<_Float16, float, 1, K>(L);
        return L.V == 8 ? norm_pick<_Float16, _Float16, 8, K>(L) : norm_pick<_Float16, _Float16, 1, K>(L);
    }
    return L.V == 4 ? norm_pick<float, float, 4, K>(L) : norm_pick<float, float, 1, K>(L);
}

}  // namespace ua2a
