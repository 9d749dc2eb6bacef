// gfx950 kernel of rotary positions, joined with the exchange or within a
// layout (ua2a_attn.h).  Each value is read once and written once, so HBM
// bandwidth bounds it, as long as what the angles cost is kept off that path: a
// workgroup works out its tokens' cosines and sines once, a pair a lane, and
// hands them round in LDS.  75,600 tokens of 40 heads of 128 in bf16 (1.55 GB): 266 us,
// 5.8 TB/s, the plain exchange 235; 256 lanes a token 273, 32 and 16 lanes 277 and
// 285, the next heads' loads ahead of this batch's stores 287.
#include "ua2a_act_device.h"
#include "ua2a_attn_internal.h"

namespace ua2a {
namespace {

// position * turns modulo 2^64, its upper word: a fraction of a turn in 32 bits.
__device__ __forceinline__ uint32_t turn_of(int32_t position, uint64_t turns)
{
    const uint32_t p = static_cast<uint32_t>(position), lo = static_cast<uint32_t>(turns),
                   hi = static_cast<uint32_t>(turns >> 32);
    return __umulhi(p, lo) + p * hi - (position < 0 ? lo : 0u);
}

// Cosine and sine of a fraction of a turn: the nearest quarter turn, and their
// series (Taylor's, to the terms below 2^-26) over the rest, within pi / 4.
__device__ __forceinline__ void cos_sin(uint32_t turn, float* c, float* s)
{
    const uint32_t quarter = (turn + 0x20000000u) >> 30;
    const float x = static_cast<float>(static_cast<int32_t>(turn - (quarter << 30))) * 1.4629180792671596e-9f;   // 2 pi / 2^32
    const float z = x * x;
    float sx = __builtin_fmaf(z, 2.7557319e-6f, -1.9841270e-4f);                 // 1 / 9!, 1 / 7!
    sx = __builtin_fmaf(z, sx, 8.3333333e-3f);                                   // 1 / 5!
    sx = __builtin_fmaf(z, sx, -1.6666667e-1f);
    sx = __builtin_fmaf(z * x, sx, x);
    float cx = __builtin_fmaf(z, -2.7557319e-7f, 2.4801587e-5f);                 // 1 / 10!, 1 / 8!
    cx = __builtin_fmaf(z, cx, -1.3888889e-3f);                                  // 1 / 6!
    cx = __builtin_fmaf(z, cx, 4.1666667e-2f);
    cx = __builtin_fmaf(z, cx, -0.5f);
    cx = __builtin_fmaf(z, cx, 1.f);
    const bool swap = quarter & 1;
    const float a = swap ? sx : cx, b = swap ? cx : sx;
    // quarter 0: (c, s); 1: (-s, c); 2: (-c, -s); 3: (s, -c)
    *c = ((quarter + 1) & 2) != 0 ? -a : a;
    *s = (quarter & 2) != 0 ? -b : b;
}

// The angle of a pair for the token in place `where` of the positions.
__device__ __forceinline__ void angle_of(const RopeArgs& a, uint32_t pair, uint32_t where, float* c, float* s)
{
    const RopeGeom& g = a.g;
    int32_t axis = a.axes[pair];
    axis = axis < 0 ? 0 : axis;
    axis = axis < static_cast<int32_t>(g.naxes) ? axis : static_cast<int32_t>(g.naxes) - 1;
    const int32_t pos = a.positions[static_cast<int64_t>(axis) * g.axis_stride + where];
    cos_sin(turn_of(pos, a.turns[pair]), c, s);
    if (g.inverse) *s = -*s;
}

__device__ __forceinline__ uint32_t position_of(const RopeGeom& g, const TokenPlace& at)
{
    return g.per_plane ? at.a : at.a - fdiv(at.a, g.d_SG) * g.sh.SG;
}

// A lane turns slot `slot` of a head for every `heads_at_once`-th head of a
// token.  A slot is V values at d (pairs side by side, V / 2 of them; or, past
// the pairs, values to copy), with HALVES V values at d and V at d + pairs
// (those slots come first, then the values to copy), and with V = 1 one pair
// either way, or one value.  TABLE: the angles come from LDS (video-DiT: 270 us
// with each lane's own); otherwise a lane works its own out (V = 1, and heads of
// more than 256 slots).
template <class T, int V, bool HALVES, bool TABLE>
__global__ __launch_bounds__(kRopeBlock) void ua2a_rope_kernel(RopeArgs a)
{
    constexpr bool kTwo = HALVES || V == 1;                      // a slot's pairs lie in two vectors
    constexpr int NP = kTwo ? V : V / 2;
    constexpr int kBatch = 4;                                    // heads whose loads are on their way together
    typedef typename Raw<T, V>::type R;
    const RopeGeom& g = a.g;
    // [token][pair]: at most 256 / slots tokens of slots * V pairs
    __shared__ f32x2v table[TABLE ? kRopeBlock * (HALVES ? V : V / 2) : 1];
    const uint32_t wg = (blockIdx.y << kAttnGridLog) + blockIdx.x;
    const uint32_t within = fdiv(threadIdx.x, g.d_lanes), lane = threadIdx.x - within * g.lanes;
    const int64_t first = static_cast<int64_t>(wg) * g.per_group;
    const bool in = within < g.per_group && first + within < static_cast<int64_t>(g.tokens);
    if constexpr (!TABLE) {
        if (!in) return;
    }
    const TokenPlace at = token_place(g.sh, in ? static_cast<uint32_t>(first + within) : 0);
    const uint32_t where = position_of(g, at);
    const uint32_t h0 = fdiv(lane, g.d_slots);
    const uint32_t D = g.sh.D, H = g.sh.H, turning = g.turning;
    for (uint32_t slot = lane - h0 * g.slots; TABLE || slot < g.slots; slot += g.lanes) {
        // first value, the second vector's distance, and which of the pairs turn
        const bool pairs_here = slot < turning;
        uint32_t d, far = 0;
        if constexpr (HALVES) {
            d = pairs_here ? slot * V : 2 * g.pairs + (slot - turning) * V;
            far = g.pairs;
        } else if constexpr (V == 1) {
            d = !pairs_here ? 2 * g.pairs + (slot - turning) : g.halves ? slot : 2 * slot;
            far = g.halves ? g.pairs : 1;
        } else {
            d = slot * V;
        }
        const auto offset = [&](uint32_t h, bool a_side) {
            return a_side ? a_offset(g.sh, at.a, h, D, g.sh.a_rank, d) : (static_cast<int64_t>(at.p) * H + h) * D + d;
        };
        const bool two = kTwo && pairs_here;
        R lo[kBatch], hi[kTwo ? kBatch : 1];
        const auto load = [&](uint32_t h) {
#pragma unroll
            for (int k = 0; k < kBatch; ++k) {
                const uint32_t hh = h + k * g.heads_at_once;
                if (hh >= H || !in) continue;
                const int64_t from = offset(hh, g.from_a);
                lo[k] = load_values<T, V>(a.x, from);
                if constexpr (kTwo)
                    if (two) hi[k] = load_values<T, V>(a.x, from + far);
            }
        };
        load(h0);                                                // on their way while the angles are worked out
        float c[NP], s[NP];
        if constexpr (TABLE) {
            for (uint32_t e = threadIdx.x; e < g.per_group * g.pairs; e += blockDim.x) {
                const uint32_t t = fdiv(e, g.d_pairs), pair = e - t * g.pairs;
                if (first + t >= static_cast<int64_t>(g.tokens)) break;
                const TokenPlace place = token_place(g.sh, static_cast<uint32_t>(first + t));
                f32x2v cs;
                float x, y;
                angle_of(a, pair, position_of(g, place), &x, &y);
                cs[0] = x;
                cs[1] = y;
                table[e] = cs;
            }
            __syncthreads();
            if (!in) return;
        }
#pragma unroll
        for (int i = 0; i < NP; ++i) {
            const uint32_t pair = kTwo ? (HALVES ? d : slot) + i : d / 2 + i;
            c[i] = 1.f;
            s[i] = 0.f;
            if (!pairs_here || pair >= g.pairs) continue;
            if constexpr (TABLE) {
                const f32x2v cs = table[within * g.pairs + pair];
                c[i] = cs[0];
                s[i] = cs[1];
            } else {
                angle_of(a, pair, where, &c[i], &s[i]);
            }
        }
        const auto turn = [&](uint32_t h) {
#pragma unroll
            for (int k = 0; k < kBatch; ++k) {
                const uint32_t hh = h + k * g.heads_at_once;
                if (hh >= H) continue;
                const int64_t to = offset(hh, g.to_a);
                float x[V];
                unpack<T, V>(lo[k], x);
                if constexpr (kTwo) {
                    if (two) {
                        float y[V], u[V], z[V];
                        unpack<T, V>(hi[k], y);
#pragma unroll
                        for (int i = 0; i < V; ++i) {
                            u[i] = __builtin_fmaf(x[i], c[i], -(y[i] * s[i]));
                            z[i] = __builtin_fmaf(y[i], c[i], x[i] * s[i]);
                        }
                        store_values<T, V>(a.out, to, pack<T, V>(u));
                        store_values<T, V>(a.out, to + far, pack<T, V>(z));
                        continue;
                    }
                    store_values<T, V>(a.out, to, lo[k]);
                } else {
                    float u[V];
#pragma unroll
                    for (int i = 0; i < NP; ++i) {
                        // past the pairs values stay as they are, infinities too
                        const bool turns = d / 2 + i < g.pairs;
                        u[2 * i] = turns ? __builtin_fmaf(x[2 * i], c[i], -(x[2 * i + 1] * s[i])) : x[2 * i];
                        u[2 * i + 1] = turns ? __builtin_fmaf(x[2 * i + 1], c[i], x[2 * i] * s[i]) : x[2 * i + 1];
                    }
                    store_values<T, V>(a.out, to, pack<T, V>(u));
                }
            }
        };
        const uint32_t batch = g.heads_at_once * kBatch;
        for (uint32_t h = h0; h < H; h += batch) {
            turn(h);
            load(h + batch);
        }
        if constexpr (TABLE) return;                             // one slot a lane
    }
}

template <class T, int V>
const void* typed_fn(const AttnLaunch& L)
{
    if constexpr (V == 1) {
        return reinterpret_cast<const void*>(&ua2a_rope_kernel<T, 1, false, false>);
    } else {
        if (L.rope.g.slots > kRopeBlock)
            return L.rope.g.halves ? reinterpret_cast<const void*>(&ua2a_rope_kernel<T, V, true, false>)
                                   : reinterpret_cast<const void*>(&ua2a_rope_kernel<T, V, false, false>);
        return L.rope.g.halves ? reinterpret_cast<const void*>(&ua2a_rope_kernel<T, V, true, true>)
                               : reinterpret_cast<const void*>(&ua2a_rope_kernel<T, V, false, true>);
    }
}

}  // namespace

const void* rope_kernel(const AttnLaunch& L)
{
    if (L.type == UA2A_TYPE_BF16) return L.V == 8 ? typed_fn<__bf16, 8>(L) : typed_fn<__bf16, 1>(L);
    if (L.type == UA2A_TYPE_FP16) return L.V == 8 ? typed_fn<_Float16, 8>(L) : typed_fn<_Float16, 1>(L);
    return L.V == 4 ? typed_fn<float, 4>(L) : typed_fn<float, 1>(L);
}

}  // namespace ua2a
