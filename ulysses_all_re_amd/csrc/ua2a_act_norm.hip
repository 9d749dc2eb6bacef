// gfx950 kernels of the RMS norm joined with the exchange (ua2a_act.h).
#include "ua2a_act_norm.h"

namespace ua2a {
namespace {

// RMS norm joined with the exchange.  A segment's lanes hold it in registers
// between the pass that sums its squares and the one that writes, so every
// value is read once.
template <class T, class W, int V, Span SPAN, int ITEMS, int BLOCK>
__global__ __launch_bounds__(BLOCK) void ua2a_norm_kernel(NormArgs a, int32_t mode1)
{
    __shared__ float red[2][16];
    const NormGeom& g = a.g;
    const uint32_t lane = threadIdx.x & ((1u << g.lanes_log) - 1);
    LaneSlots<ITEMS> l = lane_slots<SPAN, V, ITEMS>(g, lane);
    // a bundle's slots of one lane are the same values of different heads
    constexpr int kWeights = SPAN == kOne ? ITEMS : 1;
    Weights<W, V> wt[kWeights];
    if (a.weight != nullptr) {
#pragma unroll
        for (int it = 0; it < kWeights; ++it) wt[it].load(a.weight, weight_offset<SPAN, V>(g, l, lane, it));
    }
    uint32_t round = 0;
    for (uint32_t group = blockIdx.x; group < g.groups; group += gridDim.x, ++round) {
        const SegmentBase s = segment_base<SPAN, BLOCK, ITEMS>(g, group);
        const Places<SPAN, V, ITEMS> at(g, s, l, lane);
        typename Raw<T, V>::type h[ITEMS];
        if (mode1) {
#pragma unroll
            for (int it = 0; it < ITEMS; ++it) h[it] = load_values<T, V>(static_cast<const T*>(a.x) + s.a, at.a(it));
        } else {
#pragma unroll
            for (int it = 0; it < ITEMS; ++it) h[it] = load_values<T, V>(static_cast<const T*>(a.x) + s.p, at.p(it));
        }
        if (a.residual != nullptr) {
            typename Raw<T, V>::type r[ITEMS];
#pragma unroll
            for (int it = 0; it < ITEMS; ++it)
                r[it] = load_values<T, V>(static_cast<const T*>(a.residual) + s.p, at.p(it));
#pragma unroll
            for (int it = 0; it < ITEMS; ++it) {
                float f[V], e[V];
                unpack<T, V>(h[it], f);
                unpack<T, V>(r[it], e);
#pragma unroll
                for (int i = 0; i < V; ++i) f[i] += e[i];
                h[it] = pack<T, V>(f);
                if (s.live && at.ok(it)) store_values<T, V>(static_cast<T*>(a.sum) + s.p, at.p(it), h[it]);
            }
        }
        float rstd[ITEMS];
#pragma unroll
        for (int it = 0; it < ITEMS; ++it) {
            // padding counts nothing, here and in its block's magnitude
            if (g.padded && !at.ok(it)) h[it] = typename Raw<T, V>::type{};
            rstd[it] = squares<T, V>(h[it], 0.f);
        }
        norm_sums<SPAN, ITEMS>(g, rstd, red, round);
#pragma unroll
        for (int it = 0; it < ITEMS; ++it) {
            if (it == 0 || SPAN != kOne) {
                rstd[it] = 1.f / __fsqrt_rn(rstd[it] * a.inv_len + a.eps);
                const uint32_t norm_lane = SPAN == kOne ? lane : lane & ((1u << g.head_log) - 1);
                if (a.rstd != nullptr && norm_lane == 0 && s.live && at.ok(it)) a.rstd[at.stat(it)] = rstd[it];
            } else {
                rstd[it] = rstd[0];
            }
        }
        const bool first = (lane & ((1u << q_log_of<V>()) - 1)) == 0;      // of its block's lanes
        if (a.saved_format) {
#pragma unroll
            for (int it = 0; it < ITEMS; ++it) {
                uint32_t byte;
                const auto c = encode_raw<T, V>(h[it], a.saved_format, &byte);
                if (s.live && at.ok(it)) {
                    store_once(a.saved + s.p + at.p(it), c);
                    if (first) (a.saved_scales + s.ps)[at.scale_p(it)] = static_cast<uint8_t>(byte);
                }
            }
        }
#pragma unroll
        for (int it = 0; it < ITEMS; ++it) {
            const bool write = s.live && at.ok(it);
            float f[V];
            forget(h[it]);
            unpack<T, V>(h[it], f);
#pragma unroll
            for (int i = 0; i < V; ++i) f[i] *= rstd[it];
            if (a.weight != nullptr) {
                float wf[V];
                wt[SPAN == kOne ? it : 0].get(wf);
#pragma unroll
                for (int i = 0; i < V; ++i) f[i] *= wf[i];
            }
            if (a.out_format) {
                uint32_t byte;
                const auto c = encode<V>(f, a.out_format, &byte);
                if (write) {
                    if (mode1) {
                        store_once(static_cast<uint8_t*>(a.out) + s.p + at.p(it), c);
                        if (first) (a.out_scales + s.ps)[at.scale_p(it)] = static_cast<uint8_t>(byte);
                    } else {
                        store_once(static_cast<uint8_t*>(a.out) + s.a + at.a(it), c);
                        if (first) (a.out_scales + s.as)[at.scale_a(it)] = static_cast<uint8_t>(byte);
                    }
                }
            } else if (write) {
                const auto r = pack<T, V>(f);
                if (mode1)
                    store_values<T, V>(static_cast<T*>(a.out) + s.p, at.p(it), r);
                else
                    store_values<T, V>(static_cast<T*>(a.out) + s.a, at.a(it), r);
            }
        }
    }
}

template <class T, class W, int V, Span SPAN, int ITEMS, int BLOCK>
struct NormKernel {
    static const void* fn() { return reinterpret_cast<const void*>(&ua2a_norm_kernel<T, W, V, SPAN, ITEMS, BLOCK>); }
};

}  // namespace

const void* norm_kernel(const ActLaunch& L) { return norm_pick_type<NormKernel>(L, L.norm.weight_f32); }

}  // namespace ua2a
