// gfx950 kernels of the 8-bit key/value cache (ua2a_act.h): the exchange of
// new keys and values into it, quantised, and reading it back.  Each value is
// read once and written once, so HBM bandwidth bounds them.
#include "ua2a_act_device.h"

namespace ua2a {
namespace {

// New keys (grid y = 0) and values (1) in P, quantised into their places.
template <class T, int V>
__global__ __launch_bounds__(kActBlock) void ua2a_cache_write_kernel(CacheArgs a)
{
    const CacheGeom& g = a.g;
    const void* x = blockIdx.y ? a.v : a.k;
    if (x == nullptr) return;
    const uint32_t idx = blockIdx.x * kActBlock + threadIdx.x;
    const bool in = idx < g.rows * g.slots;
    const CacheSlot s = cache_slot(g, in ? idx : 0, V, true);
    const int64_t row = cache_row(g, s, a.starts, a.counts);
    const bool ok = in && row >= 0 && s.d < g.sh.D;
    typename Raw<T, V>::type raw{};
    if (ok) raw = load_values<T, V>(x, (static_cast<int64_t>(s.row) * g.sh.H + s.h) * g.sh.D + s.d);
    uint32_t byte;
    const auto c = encode_raw<T, V>(raw, a.format, &byte);
    if (!ok) return;
    const int64_t head = row * g.sh.hl + (s.h - s.r * g.sh.hl);
    store_once(a.codes + (blockIdx.y ? g.part : 0) + head * g.sh.D + s.d, c);
    if (s.d == s.blk * kBlockValues)
        a.scales[(blockIdx.y ? g.part_scales : 0) + head * g.sh.nb + s.blk] = static_cast<uint8_t>(byte);
}

// Positions of the cache back in the type.
template <class T, int V>
__global__ __launch_bounds__(kActBlock) void ua2a_cache_read_kernel(CacheArgs a)
{
    const CacheGeom& g = a.g;
    void* out = blockIdx.y ? a.v_out : a.k_out;
    if (out == nullptr) return;
    const uint32_t idx = blockIdx.x * kActBlock + threadIdx.x;
    if (idx >= g.rows * g.slots) return;
    const CacheSlot s = cache_slot(g, idx, V, false);
    const int64_t row = cache_row(g, s, a.starts, a.counts);
    if (row < 0 || s.d >= g.sh.D) return;
    const int64_t head = row * g.sh.hl + s.h;
    const auto c = load_once<typename Codes<V>::type>(a.codes + (blockIdx.y ? g.part : 0) + head * g.sh.D + s.d);
    const uint32_t byte = a.scales[(blockIdx.y ? g.part_scales : 0) + head * g.sh.nb + s.blk];
    store_values<T, V>(out, (static_cast<int64_t>(s.row) * g.sh.hl + s.h) * g.sh.D + s.d,
                       decode_raw<T, V>(c, byte, a.format));
}

template <class T, int V>
const void* typed_fn(const ActLaunch& L)
{
    return L.kernel == ActKernel::CacheWrite ? reinterpret_cast<const void*>(&ua2a_cache_write_kernel<T, V>)
                                             : reinterpret_cast<const void*>(&ua2a_cache_read_kernel<T, V>);
}

}  // namespace

const void* cache_kernel(const ActLaunch& L)
{
    if (L.type == UA2A_TYPE_BF16) return L.V == 8 ? typed_fn<__bf16, 8>(L) : typed_fn<__bf16, 1>(L);
    if (L.type == UA2A_TYPE_FP16) return L.V == 8 ? typed_fn<_Float16, 8>(L) : typed_fn<_Float16, 1>(L);
    return L.V == 4 ? typed_fn<float, 4>(L) : typed_fn<float, 1>(L);
}

}  // namespace ua2a
