// gfx950 kernels of the RMS norm joined with the exchange (ua2a_act.h).
#include "ua2a_act_norm.h"

namespace ua2a {
namespace {

// RMS norm joined with the exchange: y = h * rstd * weight, rstd = 1 /
// sqrt(mean(h^2) + eps).  A segment's lanes hold it in registers between the
// pass that sums its squares and the one that writes, so every value is read
// once and HBM bandwidth bounds it.  One workgroup per group of segments:
// workgroups that walk over several are slower (video-DiT with a checkpoint:
// 334 us against 370 with 8192 workgroups and 395 with 1024), as those drift
// apart and the rows in flight with them.  Measured: video-DiT, whole tokens,
// e4m3 checkpoint 341 us (5.7 TB/s), per head 313 us (6.2 TB/s); 4096 tokens of
// 4096 with residual and 8-bit result 23.4 us (5.0 TB/s).
template <class T, class W, int V, Span SPAN, int ITEMS, int BLOCK>
__global__ __launch_bounds__(BLOCK) void ua2a_norm_kernel(NormArgs a)
{
    __shared__ float red[2][16];
    const NormGeom& g = a.g;
    const uint32_t flags = a.flags;
    const bool mode1 = flags & kNormMode1;
    const uint32_t group = blockIdx.y * gridDim.x + blockIdx.x;
    if (group >= g.groups) return;
    const uint32_t lane = segment_lane<SPAN>(g, threadIdx.x);
    LaneSlots<ITEMS> l = lane_slots<SPAN, V, ITEMS>(g, lane);
    const SegmentBase s = segment_base<SPAN>(g, group, my_segment<SPAN>(g));
    const Places<SPAN, V, ITEMS> at(g, s, l, lane);
    typename Raw<T, V>::type h[ITEMS];
    if (mode1) {
#pragma unroll
        for (int it = 0; it < ITEMS; ++it) h[it] = load_values<T, V>(static_cast<const T*>(a.x) + s.a, at.a(it));
    } else {
#pragma unroll
        for (int it = 0; it < ITEMS; ++it) h[it] = load_values<T, V>(static_cast<const T*>(a.x) + s.p, at.p(it));
    }
    // a bundle's slots of one lane are the same values of different heads
    constexpr int kWeights = one_norm(SPAN) ? ITEMS : 1;
    Weights<W, V> wt[kWeights];
    if (flags & kNormWeight) {
#pragma unroll
        for (int it = 0; it < kWeights; ++it) wt[it].load(a.weight, weight_offset<SPAN, V>(g, l, lane, it));
    }
    if (flags & kNormResidual) {
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
    norm_sums<SPAN, ITEMS>(g, rstd, red, 0);
#pragma unroll
    for (int it = 0; it < ITEMS; ++it) {
        if (it == 0 || !one_norm(SPAN))
            rstd[it] = 1.f / __fsqrt_rn(rstd[it] * a.inv_len + a.eps);
        else
            rstd[it] = rstd[0];
    }
    if (flags & kNormRstd) {
        const bool writes = (one_norm(SPAN) ? lane : lane & ((1u << g.head_log) - 1)) == 0 && s.live;
#pragma unroll
        for (int it = 0; it < (one_norm(SPAN) ? 1 : ITEMS); ++it)
            if (writes && at.ok(it)) a.rstd[at.stat(it)] = rstd[it];
    }
    // of padding, or past the last segment, nothing is stored
    const bool masked = g.padded || group + 1 == g.groups;
    const auto stored = [&](int it) { return !masked || (s.live && at.ok(it)); };
    const bool first = (lane & ((1u << q_log_of<V>()) - 1)) == 0;          // of its block's lanes
    if (flags & kNormSaved8) {
        const int32_t format = flags & kNormSavedE5M2 ? UA2A_FORMAT_E5M2 : UA2A_FORMAT_E4M3;
#pragma unroll
        for (int it = 0; it < ITEMS; ++it) {
            uint32_t byte;
            const auto c = encode_raw<T, V>(h[it], format, &byte);
            if (stored(it)) {
                store_once(a.saved + s.p + at.p(it), c);
                if (first) (a.saved_scales + s.ps)[at.scale_p(it)] = static_cast<uint8_t>(byte);
            }
        }
    }
    const auto normed = [&](int it, float(&f)[V]) {
        forget(h[it]);
        unpack<T, V>(h[it], f);
#pragma unroll
        for (int i = 0; i < V; ++i) f[i] *= rstd[it];
        if (flags & kNormWeight) {
            float wf[V];
            wt[one_norm(SPAN) ? it : 0].get(wf);
#pragma unroll
            for (int i = 0; i < V; ++i) f[i] *= wf[i];
        }
    };
    if (flags & kNormOut8) {
        const int32_t format = flags & kNormOutE5M2 ? UA2A_FORMAT_E5M2 : UA2A_FORMAT_E4M3;
#pragma unroll
        for (int it = 0; it < ITEMS; ++it) {
            float f[V];
            normed(it, f);
            uint32_t byte;
            const auto c = encode<V>(f, format, &byte);
            if (stored(it)) {
                if (mode1) {
                    store_once(static_cast<uint8_t*>(a.out) + s.p + at.p(it), c);
                    if (first) (a.out_scales + s.ps)[at.scale_p(it)] = static_cast<uint8_t>(byte);
                } else {
                    store_once(static_cast<uint8_t*>(a.out) + s.a + at.a(it), c);
                    if (first) (a.out_scales + s.as)[at.scale_a(it)] = static_cast<uint8_t>(byte);
                }
            }
        }
        return;
    }
#pragma unroll
    for (int it = 0; it < ITEMS; ++it) {
        float f[V];
        normed(it, f);
        const auto r = pack<T, V>(f);
        if (stored(it)) {
            if (mode1)
                store_values<T, V>(static_cast<T*>(a.out) + s.p, at.p(it), r);
            else
                store_values<T, V>(static_cast<T*>(a.out) + s.a, at.a(it), r);
        }
    }
}

template <class T, class W, int V, Span SPAN, int ITEMS, int BLOCK>
struct NormKernel {
    static constexpr bool kManyItems = false;
    static const void* fn() { return reinterpret_cast<const void*>(&ua2a_norm_kernel<T, W, V, SPAN, ITEMS, BLOCK>); }
};

}  // namespace

const void* norm_kernel(const ActLaunch& L) { return norm_pick_type<NormKernel>(L, L.norm.weight_f32); }

}  // namespace ua2a
