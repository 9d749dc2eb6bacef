// gfx950 kernels of the 8-bit key/value cache (ua2a_act.h): the exchange of
// new keys and values into it, quantised, and reading it back.  Each value is
// read once and written once, so HBM bandwidth bounds them.
#include "ua2a_act_device.h"

namespace ua2a {
namespace {

// New keys and values in P, quantised into their places.  A workgroup moves one
// vector of each per lane, of one token or of several short ones (keys and
// values together: finding the place takes longer than moving one vector);
// UNIFORM: a wave's lanes share the token, so its sequence, position and
// whether it exists are scalar work.  A rank's share of a token is short (hl*D
// codes, hl*nb scales), so groups of consecutive tokens go to one XCD, whose
// L2 then puts whole lines together (a prompt of 16,384 tokens, 16 heads: 40.5
// us in runs of 16, 42.6 one by one; with keys and values apart).  Measured: that
// prompt 35 us (5.8 TB/s), 40 heads 82 us (6.2 TB/s).
template <class T, int V, bool UNIFORM>
__global__ __launch_bounds__(kActBlock) void ua2a_cache_write_kernel(CacheArgs a)
{
    const CacheGeom& g = a.g;
    const uint32_t group = cache_group(g, cache_workgroup(blockIdx.x, blockIdx.y));
    if (group >= g.groups) return;
    uint32_t tid = threadIdx.x;
    if constexpr (UNIFORM) tid = __builtin_amdgcn_readfirstlane(tid);
    const WriteLane l = write_lane(g, group, tid >> (31 - __builtin_clz(g.lanes)), 0);
    const uint32_t slot = l.slot + (threadIdx.x & (g.lanes - 1));
    const bool in = l.token < g.rows && slot < g.slots;
    const uint32_t token = l.token < g.rows ? l.token : 0;
    const TokenPlace at = token_place(g.sh, token);
    const uint32_t i = fdiv(at.a, g.d_each);
    const uint32_t t = at.a - i * g.each;
    // both from memory at once; without counts the second is not looked at
    const int32_t start = a.starts[i];
    const int32_t count = (a.counts != nullptr ? a.counts : a.starts)[i];
    const CacheSpan s = cache_span(g, start, a.counts != nullptr ? static_cast<int64_t>(count) : g.each);
    const bool live = t >= s.first && t < s.last;
    if constexpr (UNIFORM) {
        if (!live) return;
    }
    // value e of the token's H * D: of rank r, rest of its hl * D
    uint32_t e = slot * V, blk = 0;
    bool ok = in && live;
    if (!g.dense) {
        const uint32_t b = slot >> g.q_log;
        const uint32_t h = fdiv(b, g.d_nb);
        blk = b - h * g.sh.nb;
        const uint32_t d = blk * kBlockValues + (slot & ((1u << g.q_log) - 1)) * V;
        ok = ok && d < g.sh.D;
        e = h * g.sh.D + d;
    }
    const int64_t from = static_cast<int64_t>(token) * (g.sh.H * g.sh.D);
    typename Raw<T, V>::type raw[2] = {};
    if (ok && a.k != nullptr) raw[0] = load_values<T, V>(static_cast<const T*>(a.k) + from, e);
    if (ok && a.v != nullptr) raw[1] = load_values<T, V>(static_cast<const T*>(a.v) + from, e);
    const uint32_t r = fdiv(e, g.sh.d_run);
    const uint32_t rest = e - r * g.sh.run;
    const int64_t rank = static_cast<int64_t>(g.seqs) * g.cap;                  // positions of a rank
    const int64_t row = static_cast<int64_t>(i) * g.cap + (s.start + t);
    const uint32_t nscales = g.sh.hl * g.sh.nb;                                 // of a position on one rank
    uint8_t* codes = a.codes + row * g.sh.run + (r * (rank * g.sh.run) + rest);
    uint8_t* scales = a.scales + row * nscales +
                      (r * (rank * nscales) + (g.dense ? rest / kBlockValues : fdiv(rest, g.d_D) * g.sh.nb + blk));
#pragma unroll
    for (int part = 0; part < 2; ++part) {
        if ((part ? a.v : a.k) == nullptr) continue;
        uint32_t byte;
        const auto c = encode_raw<T, V>(raw[part], a.format, &byte);
        if (!ok) continue;
        store_once(codes + (part ? g.part : 0), c);
        if ((slot & ((1u << g.q_log) - 1)) == 0) scales[part ? g.part_scales : 0] = static_cast<uint8_t>(byte);
    }
}

// Positions of the cache back in the type.  What a rank holds of a sequence is
// one stretch of the cache and of the output, so a workgroup's part of it is
// scalar work and a lane moves one vector of keys and one of values.  Measured:
// 75,600 positions of 40 heads 378 us (6.2 TB/s; keys and values in halves of the
// grid 409).
template <class T, int V>
__global__ __launch_bounds__(kActBlock) void ua2a_cache_read_kernel(CacheArgs a)
{
    const CacheGeom& g = a.g;
    const uint32_t wg = cache_workgroup(blockIdx.x, blockIdx.y);
    const uint32_t ri = fdiv(wg, g.d_tiles);                    // (rank, sequence)
    const uint32_t tile = wg - ri * g.tiles;
    const uint32_t r = fdiv(ri, g.d_seqs);
    const uint32_t i = ri - r * g.seqs;
    const CacheSpan s = cache_span(g, a.starts ? static_cast<int64_t>(a.starts[i]) : 0,
                                   a.counts ? static_cast<int64_t>(a.counts[i]) : static_cast<int64_t>(g.each));
    const int64_t e = (static_cast<int64_t>(tile) * blockDim.x + threadIdx.x) * V;
    // past the last span too, here rather than ahead of the loads (read_ragged 12.1 us)
    if (e < s.first * g.sh.run || e >= s.last * g.sh.run || ri >= g.spans) return;
    const int64_t row = static_cast<int64_t>(ri) * g.cap + s.start;             // of the span's first token
    const uint32_t nscales = g.sh.hl * g.sh.nb;
    const int64_t at_scale = g.dense ? e / kBlockValues
                                     : scale_of_value(g, static_cast<int64_t>(tile) * (blockDim.x * V), threadIdx.x * V);
    const uint8_t* codes = a.codes + row * g.sh.run + e;
    const uint8_t* scales = a.scales + row * nscales + at_scale;
    const int64_t to = static_cast<int64_t>(ri) * g.each * g.sh.run;
    typename Codes<V>::type c[2] = {};
    uint32_t byte[2] = {};
#pragma unroll
    for (int part = 0; part < 2; ++part) {
        if ((part ? a.v_out : a.k_out) == nullptr) continue;
        c[part] = load_once<typename Codes<V>::type>(codes + (part ? g.part : 0));
        byte[part] = scales[part ? g.part_scales : 0];
    }
#pragma unroll
    for (int part = 0; part < 2; ++part) {
        void* out = part ? a.v_out : a.k_out;
        if (out == nullptr) continue;
        store_values<T, V>(static_cast<T*>(out) + to, e, decode_raw<T, V>(c[part], byte[part], a.format));
    }
}

template <class T, int V>
const void* typed_fn(const ActLaunch& L)
{
    if (L.kernel == ActKernel::CacheRead) return reinterpret_cast<const void*>(&ua2a_cache_read_kernel<T, V>);
    return L.cache.g.lanes >= 64 ? reinterpret_cast<const void*>(&ua2a_cache_write_kernel<T, V, true>)
                                 : reinterpret_cast<const void*>(&ua2a_cache_write_kernel<T, V, false>);
}

}  // namespace

const void* cache_kernel(const ActLaunch& L)
{
    if (L.type == UA2A_TYPE_BF16) return L.V == 8 ? typed_fn<__bf16, 8>(L) : typed_fn<__bf16, 1>(L);
    if (L.type == UA2A_TYPE_FP16) return L.V == 8 ? typed_fn<_Float16, 8>(L) : typed_fn<_Float16, 1>(L);
    return L.V == 4 ? typed_fn<float, 4>(L) : typed_fn<float, 1>(L);
}

}  // namespace ua2a
