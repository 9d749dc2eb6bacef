// gfx950 kernels of the backward pass of the RMS norm joined with the exchange
// (ua2a_act.h).
#include "ua2a_act_norm.h"

namespace ua2a {
namespace {

// Backward pass of the norm and its exchange.  Workgroups walk over segments
// and keep the sums of dweight for their lanes' slots in registers; at the
// end each workgroup writes one row of partial sums.
template <class T, class W, bool SAVED8, int V, Span SPAN, int ITEMS, int BLOCK>
__global__ __launch_bounds__(BLOCK) void ua2a_norm_grad_kernel(NormGradArgs a, int32_t mode1)
{
    __shared__ float red[2][16];
    __shared__ float join[BLOCK * V];
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
    constexpr int kNorms = SPAN == kOne ? 1 : ITEMS;     // norms of a lane
    float dw[kWeights][V];
#pragma unroll
    for (int it = 0; it < kWeights; ++it)
#pragma unroll
        for (int i = 0; i < V; ++i) dw[it][i] = 0.f;
    typedef typename std::conditional<SAVED8, typename Codes<V>::type, typename Raw<T, V>::type>::type Held;
    struct Loaded {              // what the lane holds of a segment
        SegmentBase s;
        typename Raw<T, V>::type dy[ITEMS];
        Held h[ITEMS];
        uint32_t hs[ITEMS];
        float rstd[kNorms];
    };
    const auto load = [&](uint32_t group, Loaded& x) {
        x.s = segment_base<SPAN, BLOCK, ITEMS>(g, group);
        const SegmentBase& s = x.s;
        const Places<SPAN, V, ITEMS> at(g, s, l, lane);
        if (mode1) {
#pragma unroll
            for (int it = 0; it < ITEMS; ++it) x.dy[it] = load_values<T, V>(static_cast<const T*>(a.dy) + s.p, at.p(it));
        } else {
#pragma unroll
            for (int it = 0; it < ITEMS; ++it) x.dy[it] = load_values<T, V>(static_cast<const T*>(a.dy) + s.a, at.a(it));
        }
        if constexpr (SAVED8) {
#pragma unroll
            for (int it = 0; it < ITEMS; ++it) {
                x.h[it] = load_once<Held>(static_cast<const uint8_t*>(a.saved) + s.p + at.p(it));
                x.hs[it] = at.ok(it) ? (a.saved_scales + s.ps)[at.scale_p(it)] : 0u;
            }
        } else if (a.saved_gathered) {
#pragma unroll
            for (int it = 0; it < ITEMS; ++it) x.h[it] = load_values<T, V>(static_cast<const T*>(a.saved) + s.a, at.a(it));
        } else {
#pragma unroll
            for (int it = 0; it < ITEMS; ++it) x.h[it] = load_values<T, V>(static_cast<const T*>(a.saved) + s.p, at.p(it));
        }
#pragma unroll
        for (int it = 0; it < kNorms; ++it) x.rstd[it] = a.rstd[at.stat(it)];
    };
    uint32_t round = 0;
    Loaded next;
    load(blockIdx.x, next);                                     // the grid has no more workgroups than groups
    for (uint32_t group = blockIdx.x; group < g.groups; group += gridDim.x, ++round) {
        Loaded x = next;
        const SegmentBase& s = x.s;
        const Places<SPAN, V, ITEMS> at(g, s, l, lane);
        typename Raw<T, V>::type ds[ITEMS];
        if (a.dsum != nullptr) {
#pragma unroll
            for (int it = 0; it < ITEMS; ++it) ds[it] = load_values<T, V>(static_cast<const T*>(a.dsum) + s.p, at.p(it));
        }
        // the next segment is on its way while this one is worked on
        if (group + gridDim.x < g.groups) load(group + gridDim.x, next);
        auto& dy = x.dy;
        auto& h = x.h;
        auto& hs = x.hs;
        // lanes of padding, or past the last segment, count nothing
        const bool masked = g.padded || group + 1 == g.groups;
        // what was normed, up to the factor that stands beside it: its scale
        const auto normed = [&](int it, float(&n)[V]) {
            if constexpr (SAVED8)
                code_values<V>(h[it], a.saved_format, n);
            else
                unpack<T, V>(h[it], n);
        };
        float mean[ITEMS];
#pragma unroll
        for (int it = 0; it < ITEMS; ++it) {
            if (masked && !(s.live && at.ok(it))) {
                dy[it] = typename Raw<T, V>::type{};
                h[it] = {};
            }
            float d[V], n[V], p = 0.f;
            unpack<T, V>(dy[it], d);
            normed(it, n);
            const float rstd = x.rstd[SPAN == kOne ? 0 : it];
            const float r = SAVED8 ? rstd * scale_of(hs[it]) : rstd;
#pragma unroll
            for (int i = 0; i < V; ++i) {
                n[i] = d[i] * (n[i] * r);
                dw[SPAN == kOne ? it : 0][i] += n[i];
            }
            if (a.weight != nullptr) {
                float wf[V];
                wt[SPAN == kOne ? it : 0].get(wf);
#pragma unroll
                for (int i = 0; i < V; ++i) p += n[i] * wf[i];
            } else {
#pragma unroll
                for (int i = 0; i < V; ++i) p += n[i];
            }
            mean[it] = p;
        }
        norm_sums<SPAN, ITEMS>(g, mean, red, round);
#pragma unroll
        for (int it = 0; it < ITEMS; ++it) {
            float d[V], n[V];
            forget(dy[it]);
            forget(h[it]);
            unpack<T, V>(dy[it], d);
            normed(it, n);
            if (a.weight != nullptr) {
                float wf[V];
                wt[SPAN == kOne ? it : 0].get(wf);
#pragma unroll
                for (int i = 0; i < V; ++i) d[i] *= wf[i];
            }
            // the powers of two leave the factor's rounding alone
            const float rstd = x.rstd[SPAN == kOne ? 0 : it];
            const float m = rstd * (mean[it] * a.inv_len);
            const float r = SAVED8 ? m * scale_of(hs[it]) : m;
#pragma unroll
            for (int i = 0; i < V; ++i) d[i] = rstd * (d[i] - n[i] * r);
            if (a.dsum != nullptr) {
                float e[V];
                unpack<T, V>(ds[it], e);
#pragma unroll
                for (int i = 0; i < V; ++i) d[i] += e[i];
            }
            if (s.live && at.ok(it)) {
                const auto r16 = pack<T, V>(d);
                if (mode1)
                    store_values<T, V>(static_cast<T*>(a.dx) + s.a, at.a(it), r16);
                else
                    store_values<T, V>(static_cast<T*>(a.dx) + s.p, at.p(it), r16);
                if (a.dresidual != nullptr) store_values<T, V>(static_cast<T*>(a.dresidual) + s.p, at.p(it), r16);
            }
        }
    }
    if (a.partial == nullptr) return;
    // one row of sums per workgroup; lanes with the same weights are joined in
    // order: the workgroup's segments, and in bundles their heads
    const uint32_t lanes = 1u << (SPAN == kOne ? g.lanes_log : g.head_log);
    const uint32_t per = BLOCK / lanes;
    float* row = a.partial + static_cast<int64_t>(blockIdx.x) * g.cols;
#pragma unroll
    for (int it = 0; it < kWeights; ++it) {
        if (per > 1) {
            __syncthreads();
#pragma unroll
            for (int i = 0; i < V; ++i) join[i * BLOCK + threadIdx.x] = dw[it][i];
            __syncthreads();
        }
        if (threadIdx.x < lanes && (l.ok >> it & 1)) {
            const uint32_t to = weight_offset<SPAN, V>(g, l, lane, it);
#pragma unroll
            for (int i = 0; i < V; ++i) {
                float t = dw[it][i];
#pragma unroll 1
                for (uint32_t k = 1; k < per; ++k) t += join[i * BLOCK + k * lanes + threadIdx.x];
                row[to + i] = t;
            }
        }
    }
}

// Column sums of the workgroups' rows: 32 columns per workgroup, 32 lanes
// down each, joined in order.
__global__ __launch_bounds__(1024) void ua2a_columns_kernel(ColumnArgs a)
{
    __shared__ float part[32][33];
    const uint32_t c = blockIdx.x * 32 + (threadIdx.x & 31);
    const uint32_t r0 = threadIdx.x >> 5;
    float t = 0.f;
    if (c < a.cols)
        for (uint32_t r = r0; r < a.rows; r += 32) t += a.partial[static_cast<int64_t>(r) * a.cols + c];
    part[r0][threadIdx.x & 31] = t;
    __syncthreads();
    if (r0 == 0 && c < a.cols) {
        t = 0.f;
        for (uint32_t k = 0; k < 32; ++k) t += part[k][threadIdx.x];
        a.out[c] = t;
    }
}

template <class T, class W, int V, Span SPAN, int ITEMS, int BLOCK>
struct GradKernel {
    static const void* fn() { return reinterpret_cast<const void*>(&ua2a_norm_grad_kernel<T, W, false, V, SPAN, ITEMS, BLOCK>); }
};
template <class T, class W, int V, Span SPAN, int ITEMS, int BLOCK>
struct GradKernel8 {
    static const void* fn() { return reinterpret_cast<const void*>(&ua2a_norm_grad_kernel<T, W, true, V, SPAN, ITEMS, BLOCK>); }
};

}  // namespace

const void* norm_grad_kernel(const ActLaunch& L)
{
    return L.grad.saved_format ? norm_pick_type<GradKernel8>(L, L.grad.weight_f32)
                               : norm_pick_type<GradKernel>(L, L.grad.weight_f32);
}

const void* columns_kernel() { return reinterpret_cast<const void*>(&ua2a_columns_kernel); }

}  // namespace ua2a
