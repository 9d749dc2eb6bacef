// What the norm kernels, forward and backward, share: the lanes' segments, the
// weights and the sums.
#pragma once

#include "ua2a_act_device.h"

namespace ua2a {
namespace {

// The segment of this lane's workgroup.  A segment of whole waves is the same in
// every lane, so what follows from it is scalar.
template <Span SPAN>
__device__ __forceinline__ uint32_t my_segment(const NormGeom& g)
{
    uint32_t tid = threadIdx.x;
    if constexpr (SPAN == kWaves || SPAN == kBundle) tid = __builtin_amdgcn_readfirstlane(tid);
    return segment_within<SPAN>(g, tid);
}

// SlotPlaces of which nothing derived is kept from one segment to the next.
template <Span SPAN, int V, int ITEMS>
struct Places : SlotPlaces<SPAN, V, ITEMS> {
    __device__ __forceinline__ Places(const NormGeom& g, const SegmentBase& s, LaneSlots<ITEMS>& l, uint32_t lane_)
        : SlotPlaces<SPAN, V, ITEMS>{g, s, l, lane_}
    {
        forget(this->lane);
#pragma unroll
        for (int it = 0; it < ITEMS; ++it) {
            forget(l.a[it]);
            forget(l.p[it]);
        }
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
