// gfx950 kernels of the backward pass of the RMS norm joined with the exchange
// (ua2a_act.h).
#include "ua2a_act_norm.h"

namespace ua2a {
namespace {

// Backward pass of the norm and its exchange: with g = dy * weight and n = h *
// rstd, dh = rstd * (g - n * mean(g * n)) + dsum and dweight = sum(dy * n).
// One pass over dy and h; a segment stays in registers between its sum and its
// result.  Workgroups walk over segments, a fixed set each, and keep the sums of
// dweight for their lanes' slots in registers, so the order of the sums is
// fixed; at the end each workgroup writes one row of partial sums.  Those
// registers leave two waves per SIMD, so the next segment's loads are issued
// before one is worked on.  Measured: video-DiT from an e4m3 checkpoint 367 us
// (5.3 TB/s; without the early loads 374 on a card where this form took 347),
// from the values 394 us (5.9 TB/s).
template <class T, class W, bool SAVED8, int V, Span SPAN, int ITEMS, int BLOCK>
__global__ __launch_bounds__(BLOCK) void ua2a_norm_grad_kernel(NormGradArgs a)
{
    __shared__ float red[2][16];
    __shared__ float join[SPAN == kWide ? 1 : BLOCK * V];
    const NormGeom& g = a.g;
    const uint32_t flags = a.flags;
    const bool mode1 = flags & kNormMode1;
    const uint32_t lane = segment_lane<SPAN>(g, threadIdx.x);
    LaneSlots<ITEMS> l = lane_slots<SPAN, V, ITEMS>(g, lane);
    // a bundle's slots of one lane are the same values of different heads
    constexpr int kWeights = one_norm(SPAN) ? ITEMS : 1;
    Weights<W, V> wt[kWeights];
    if (flags & kNormWeight) {
#pragma unroll
        for (int it = 0; it < kWeights; ++it) wt[it].load(a.weight, weight_offset<SPAN, V>(g, l, lane, it));
    }
    constexpr int kNorms = one_norm(SPAN) ? 1 : ITEMS;     // norms of a lane
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
        x.s = segment_base<SPAN>(g, group, my_segment<SPAN>(g));
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
                x.hs[it] = (a.saved_scales + s.ps)[at.scale_p(it)];
            }
        } else if ((flags & kNormGathered)) {
#pragma unroll
            for (int it = 0; it < ITEMS; ++it) x.h[it] = load_values<T, V>(static_cast<const T*>(a.saved) + s.a, at.a(it));
        } else {
#pragma unroll
            for (int it = 0; it < ITEMS; ++it) x.h[it] = load_values<T, V>(static_cast<const T*>(a.saved) + s.p, at.p(it));
        }
#pragma unroll
        for (int it = 0; it < kNorms; ++it) x.rstd[it] = a.rstd[at.stat(it)];
    };
    const auto work = [&](uint32_t group, Loaded& x, uint32_t after, Loaded& next, uint32_t round) {
        const SegmentBase& s = x.s;
        const Places<SPAN, V, ITEMS> at(g, s, l, lane);
        typename Raw<T, V>::type ds[ITEMS];
        if (flags & kNormResidual) {
#pragma unroll
            for (int it = 0; it < ITEMS; ++it) ds[it] = load_values<T, V>(static_cast<const T*>(a.dsum) + s.p, at.p(it));
        }
        // the next segment is on its way while this one is worked on
        if (after < g.groups) load(after, next);
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
            const float rstd = x.rstd[one_norm(SPAN) ? 0 : it];
            const float r = SAVED8 ? rstd * read_scale_of(hs[it]) : rstd;
            float* const sums = dw[one_norm(SPAN) ? it : 0];
            // n * dy with n near 1: h * dy may leave 32 bits where no result does
            // (one operation more per value, 0.5 % of the time)
#pragma unroll
            for (int i = 0; i < V; ++i) {
                n[i] *= r;
                sums[i] += n[i] * d[i];
                n[i] *= d[i];
            }
            if (flags & kNormWeight) {
                float wf[V];
                wt[one_norm(SPAN) ? it : 0].get(wf);
#pragma unroll
                for (int i = 0; i < V; ++i) p += n[i] * wf[i];
            } else {
#pragma unroll
                for (int i = 0; i < V; ++i) p += n[i];
            }
            mean[it] = p;
        }
        // A lane of padding looks at another slot's rstd, scale and weight: a NaN or
        // an infinity among them passes the product with its zeros, so its part of
        // the norm's sum is zero by itself.  (Its sums of dweight are not used; a
        // lane past the last segment looks at the same slot of the first, whose own
        // lane adds such a NaN to dweight anyway.)
        if (masked) {
#pragma unroll
            for (int it = 0; it < ITEMS; ++it)
                if (!at.ok(it)) mean[it] = 0.f;
        }
        norm_sums<SPAN, ITEMS>(g, mean, red, round);
#pragma unroll
        for (int it = 0; it < ITEMS; ++it) {
            float d[V], n[V];
            forget(dy[it]);
            forget(h[it]);
            unpack<T, V>(dy[it], d);
            normed(it, n);
            if (flags & kNormWeight) {
                float wf[V];
                wt[one_norm(SPAN) ? it : 0].get(wf);
#pragma unroll
                for (int i = 0; i < V; ++i) d[i] *= wf[i];
            }
            // the powers of two leave the factor's rounding alone
            const float rstd = x.rstd[one_norm(SPAN) ? 0 : it];
            const float m = rstd * (mean[it] * a.inv_len);
            const float r = SAVED8 ? m * read_scale_of(hs[it]) : m;
#pragma unroll
            for (int i = 0; i < V; ++i) d[i] = rstd * (d[i] - n[i] * r);
            if (flags & kNormResidual) {
                float e[V];
                unpack<T, V>(ds[it], e);
#pragma unroll
                for (int i = 0; i < V; ++i) d[i] += e[i];
            }
            const auto r16 = pack<T, V>(d);
            if (!masked || (s.live && at.ok(it))) {
                if (mode1)
                    store_values<T, V>(static_cast<T*>(a.dx) + s.a, at.a(it), r16);
                else
                    store_values<T, V>(static_cast<T*>(a.dx) + s.p, at.p(it), r16);
                if (flags & kNormApart) store_values<T, V>(static_cast<T*>(a.dresidual) + s.p, at.p(it), r16);
            }
        }
    };
    // Two segments' worth of registers in turn: handing one over to the other
    // would wait for its loads.
    Loaded one, two;
    uint32_t group = blockIdx.x;                                // the grid has no more workgroups than groups
    load(group, one);
    for (;;) {
        uint32_t after = group + gridDim.x;
        work(group, one, after, two, 0);
        if (after >= g.groups) break;
        group = after + gridDim.x;
        work(after, two, group, one, 1);
        if (group >= g.groups) break;
    }
    if (!(flags & kNormPartial)) return;
    // One row of sums per workgroup.  Lanes with the same weights (the
    // workgroup's segments; in bundles their heads too) are joined within a
    // wave by exchanging lanes, then over its waves through LDS, in a fixed
    // order.
    float* row = a.partial + static_cast<int64_t>(blockIdx.x) * g.cols;
    const uint32_t lanes = one_norm(SPAN) ? g.lanes : 1u << g.head_log;                           // lanes with different weights
    const uint32_t apart = lanes < 64 ? lanes : 64;             // ... of a wave
    const uint32_t per = SPAN == kWide ? 1 : BLOCK / (lanes < 64 ? 64 : lanes);    // waves (segments) to join
#pragma unroll
    for (int it = 0; it < kWeights; ++it) {
        for (uint32_t step = apart; step < 64; step *= 2) {
#pragma unroll
            for (int i = 0; i < V; ++i) dw[it][i] += __shfl_xor(dw[it][i], static_cast<int>(step));
        }
        if (SPAN != kWide && per > 1) {
            __syncthreads();
#pragma unroll
            for (int i = 0; i < V; ++i) join[i * BLOCK + threadIdx.x] = dw[it][i];
            __syncthreads();
        }
        if (threadIdx.x < lanes && (l.ok >> it & 1)) {
            const uint32_t to = weight_offset<SPAN, V>(g, l, lane, it);
            const uint32_t next_one = lanes < 64 ? 64 : lanes;
            for (uint32_t k = 1; SPAN != kWide && k < per; ++k) {
#pragma unroll
                for (int i = 0; i < V; ++i) dw[it][i] += join[i * BLOCK + k * next_one + threadIdx.x];
            }
#pragma unroll
            for (int i = 0; i < V; ++i) row[to + i] = dw[it][i];
        }
    }
}

// Column sums of the workgroups' rows, joined in a fixed order: 2^across_log
// columns per workgroup, its other lanes down the rows with eight loads in
// flight each.  Few columns take narrow workgroups, so that a lane has few rows
// to wait for (64 columns of 1024 rows: 32 wide 3.9 us).
constexpr int kColumnsBlock = 1024;
__global__ __launch_bounds__(kColumnsBlock) void ua2a_columns_kernel(ColumnArgs a)
{
    __shared__ float part[kColumnsBlock / 64][64];
    const uint32_t across = 1u << a.across_log;
    const uint32_t down = kColumnsBlock >> a.across_log;
    const uint32_t c = blockIdx.x * across + (threadIdx.x & (across - 1));
    float t = 0.f;
    if (c < a.cols) {
        const float* p = a.partial + c;
        uint32_t r = threadIdx.x >> a.across_log;
        for (; r + 7 * down < a.rows; r += 8 * down) {
            float v[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) v[k] = p[static_cast<int64_t>(r + k * down) * a.cols];
#pragma unroll
            for (int k = 0; k < 8; ++k) t += v[k];
        }
        for (; r < a.rows; r += down) t += p[static_cast<int64_t>(r) * a.cols];
    }
    for (uint32_t step = across; step < 64; step *= 2) t += __shfl_xor(t, static_cast<int>(step));
    const uint32_t lane = threadIdx.x & 63;
    if (lane < across) part[threadIdx.x >> 6][lane] = t;
    __syncthreads();
    if (threadIdx.x < across && c < a.cols) {
        t = 0.f;
#pragma unroll
        for (int k = 0; k < kColumnsBlock / 64; ++k) t += part[k][threadIdx.x];
        a.out[c] = t;
    }
}

template <class T, class W, int V, Span SPAN, int ITEMS, int BLOCK>
struct GradKernel {
    static constexpr bool kManyItems = true;
    static const void* fn() { return reinterpret_cast<const void*>(&ua2a_norm_grad_kernel<T, W, false, V, SPAN, ITEMS, BLOCK>); }
};
template <class T, class W, int V, Span SPAN, int ITEMS, int BLOCK>
struct GradKernel8 {
    static constexpr bool kManyItems = true;
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
