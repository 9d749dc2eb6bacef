// gfx950 (MI355X, CDNA4) kernels of the activation operators (ua2a_act.h):
// RMS norms joined with the Ulysses exchange and their backward pass, and the
// 8-bit key/value cache.
//
// All of them read each input once and write each output once; a norm's few
// operations per value hide behind that, so they are bound by HBM bandwidth
// like the exchange itself, and need no MFMA.
#include <hip/hip_runtime.h>

#include "ua2a_act_internal.h"

namespace ua2a {
namespace {

typedef uint32_t u32x2v __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4v __attribute__((ext_vector_type(4)));
typedef float f32x2v __attribute__((ext_vector_type(2)));

// ------------------------------------------------------------------ values

// V values of type T as they are loaded and stored: 16 bytes, or one value.
template <class T, int V>
struct Raw {
    typedef u32x4v type;
};
template <>
struct Raw<__bf16, 1> {
    typedef uint16_t type;
};
template <>
struct Raw<_Float16, 1> {
    typedef uint16_t type;
};
template <>
struct Raw<float, 1> {
    typedef uint32_t type;
};

// V codes: one byte each.
template <int V>
struct Codes;
template <>
struct Codes<8> {
    typedef u32x2v type;
};
template <>
struct Codes<4> {
    typedef uint32_t type;
};
template <>
struct Codes<1> {
    typedef uint8_t type;
};

template <class T, int V>
__device__ __forceinline__ void unpack(typename Raw<T, V>::type r, float (&f)[V])
{
    if constexpr (V == 1) {
        f[0] = static_cast<float>(__builtin_bit_cast(T, r));
    } else {
        typedef T vec __attribute__((ext_vector_type(V)));
        const vec v = __builtin_bit_cast(vec, r);
#pragma unroll
        for (int i = 0; i < V; ++i) f[i] = static_cast<float>(v[i]);
    }
}

template <class T, int V>
__device__ __forceinline__ typename Raw<T, V>::type pack(const float (&f)[V])
{
    if constexpr (V == 1) {
        return __builtin_bit_cast(typename Raw<T, 1>::type, static_cast<T>(f[0]));
    } else {
        typedef T vec __attribute__((ext_vector_type(V)));
        vec v;
#pragma unroll
        for (int i = 0; i < V; ++i) v[i] = static_cast<T>(f[i]);
        return __builtin_bit_cast(u32x4v, v);
    }
}

template <class R>
__device__ __forceinline__ R load_once(const void* p)
{
    return __builtin_nontemporal_load(static_cast<const R*>(p));
}
template <class R>
__device__ __forceinline__ void store_once(void* p, R r)
{
    __builtin_nontemporal_store(r, static_cast<R*>(p));
}

template <class T, int V>
__device__ __forceinline__ typename Raw<T, V>::type load_values(const void* base, int64_t at)
{
    return load_once<typename Raw<T, V>::type>(static_cast<const T*>(base) + at);
}
template <class T, int V>
__device__ __forceinline__ void store_values(void* base, int64_t at, typename Raw<T, V>::type r)
{
    store_once(static_cast<T*>(base) + at, r);
}

// ------------------------------------------------------------- lane exchange

template <int CTRL>
__device__ __forceinline__ uint32_t dpp(uint32_t x)
{
    return static_cast<uint32_t>(__builtin_amdgcn_update_dpp(0, static_cast<int>(x), CTRL, 0xf, 0xf, true));
}
constexpr int kDppXor1 = 0xB1;         // quad_perm [1,0,3,2]
constexpr int kDppXor2 = 0x4E;         // quad_perm [2,3,0,1]
constexpr int kDppHalfMirror = 0x141;  // lane i <-> 7 - i of 8
constexpr int kDppMirror = 0x140;      // lane i <-> 15 - i of 16

// Largest value over aligned groups of 2^LOG lanes.  After the first two
// steps quads are uniform, so a mirror is as good as an exclusive-or.
template <int LOG>
__device__ __forceinline__ uint32_t group_max(uint32_t x)
{
    if constexpr (LOG >= 1) x = max(x, dpp<kDppXor1>(x));
    if constexpr (LOG >= 2) x = max(x, dpp<kDppXor2>(x));
    if constexpr (LOG >= 3) x = max(x, dpp<kDppHalfMirror>(x));
    if constexpr (LOG >= 4) x = max(x, dpp<kDppMirror>(x));
    if constexpr (LOG >= 5) x = max(x, static_cast<uint32_t>(__shfl_xor(static_cast<int>(x), 16)));
    return x;
}

template <int CTRL>
__device__ __forceinline__ float dpp_add(float x)
{
    return x + __uint_as_float(dpp<CTRL>(__float_as_uint(x)));
}

// Sum over aligned groups of 2^log lanes of a wave (log is uniform).
__device__ __forceinline__ float group_sum(float x, uint32_t log)
{
    if (log >= 1) x = dpp_add<kDppXor1>(x);
    if (log >= 2) x = dpp_add<kDppXor2>(x);
    if (log >= 3) x = dpp_add<kDppHalfMirror>(x);
    if (log >= 4) x = dpp_add<kDppMirror>(x);
    if (log >= 5) x += __shfl_xor(x, 16);
    if (log >= 6) x += __shfl_xor(x, 32);
    return x;
}

// Sum over the 2^log lanes of a segment, in every lane of it; segments wider
// than a wave join their waves' sums through LDS, in the waves' order.  `red`
// holds one sum per wave, for two rounds in turn: a wave writes round n + 2
// only after the barrier of round n + 1, which every wave reaches with round
// n read.
__device__ __forceinline__ float segment_sum(float x, uint32_t log, float (*red)[16], uint32_t round)
{
    x = group_sum(x, log);
    if (log <= 6) return x;
    const uint32_t wave = threadIdx.x >> 6;
    const uint32_t waves = 1u << (log - 6);
    float* r = red[round & 1];
    if ((threadIdx.x & 63) == 0) r[wave] = x;
    __syncthreads();
    const uint32_t first = wave & ~(waves - 1);
    x = 0.f;
    for (uint32_t k = 0; k < waves; ++k) x += r[first + k];
    return x;
}

// ----------------------------------------------------------- 8 bits with scales

template <int V>
constexpr int q_log_of()
{
    return V == 8 ? 2 : V == 4 ? 3 : 5;
}

// The scale byte of a block from the bits of its largest finite magnitude.
// With m = 1.f * 2^e the least k with m <= 1.75 * 2^(top + k) is e - top, one
// more where 1.f > 1.75; adding 0x1fffff carries into the exponent in just
// that case.  The byte is k + 127.
__device__ __forceinline__ uint32_t scale_byte(uint32_t bits, int32_t format)
{
    const int32_t top = format == UA2A_FORMAT_E4M3 ? 8 : 15;
    const int32_t k = static_cast<int32_t>((bits + 0x1fffffu) >> 23) - top;
    return k < 0 ? 0u : static_cast<uint32_t>(k);
}
// 2^(byte - 127) and its inverse; byte is at most 254 and 247 respectively.
__device__ __forceinline__ float scale_of(uint32_t byte)
{
    return __uint_as_float(byte ? byte << 23 : 0x400000u);
}
__device__ __forceinline__ float inverse_scale(uint32_t byte) { return __uint_as_float((254u - byte) << 23); }

// Codes of V values of a block shared by 2^q_log lanes, and its scale byte.
// Multiplying by a power of two is exact where the code is not zero, so the
// conversion's rounding is the only one.  Infinities and NaN stay out of the
// block's magnitude (looked for only when one shows up: their bits are the
// largest), and convert to what the formats have for them.
template <int V>
__device__ __forceinline__ typename Codes<V>::type encode(const float (&f)[V], int32_t format, uint32_t* byte)
{
    constexpr uint32_t kInf = 0x7f800000u;
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < V; ++i) m = max(m, __float_as_uint(f[i]) & 0x7fffffffu);
    uint32_t top = group_max<q_log_of<V>()>(m);
    if (__builtin_amdgcn_ballot_w64(top >= kInf) != 0) {
        m = 0;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const uint32_t a = __float_as_uint(f[i]) & 0x7fffffffu;
            m = max(m, a < kInf ? a : 0u);
        }
        top = group_max<q_log_of<V>()>(m);
    }
    const uint32_t s = scale_byte(top, format);
    const float inv = inverse_scale(s);
    *byte = s;
    if constexpr (V == 1) {
        const float a = f[0] * inv;
        const int c = format == UA2A_FORMAT_E4M3 ? __builtin_amdgcn_cvt_pk_fp8_f32(a, a, 0, false)
                                                 : __builtin_amdgcn_cvt_pk_bf8_f32(a, a, 0, false);
        return static_cast<uint8_t>(c & 0xff);
    } else {
        int c[V / 4];
        if (format == UA2A_FORMAT_E4M3) {
#pragma unroll
            for (int i = 0; i < V / 4; ++i) {
                c[i] = __builtin_amdgcn_cvt_pk_fp8_f32(f[4 * i] * inv, f[4 * i + 1] * inv, 0, false);
                c[i] = __builtin_amdgcn_cvt_pk_fp8_f32(f[4 * i + 2] * inv, f[4 * i + 3] * inv, c[i], true);
            }
        } else {
#pragma unroll
            for (int i = 0; i < V / 4; ++i) {
                c[i] = __builtin_amdgcn_cvt_pk_bf8_f32(f[4 * i] * inv, f[4 * i + 1] * inv, 0, false);
                c[i] = __builtin_amdgcn_cvt_pk_bf8_f32(f[4 * i + 2] * inv, f[4 * i + 3] * inv, c[i], true);
            }
        }
        if constexpr (V == 8)
            return u32x2v{static_cast<uint32_t>(c[0]), static_cast<uint32_t>(c[1])};
        else
            return static_cast<uint32_t>(c[0]);
    }
}

// code * scale for values that become a T.  The product is exact in 32 bits
// (codes are multiples of 2^-16, scales at least 2^-127) unless the block's
// largest value, rounded up, passes what T holds: that takes a scale of
// 2^(T's largest exponent - the format's + 1) at least, looked for per block,
// and such finite codes give T's largest value.
template <class T, int V>
__device__ __forceinline__ void decode(typename Codes<V>::type c, uint32_t byte, int32_t format, float (&f)[V])
{
    const float s = scale_of(byte);
    uint32_t w[V == 8 ? 2 : 1];
    if constexpr (V == 8) {
        w[0] = c[0];
        w[1] = c[1];
    } else {
        w[0] = c;
    }
#pragma unroll
    for (int i = 0; i < (V + 3) / 4; ++i) {
        f32x2v lo, hi;
        if (format == UA2A_FORMAT_E4M3) {
            lo = __builtin_amdgcn_cvt_pk_f32_fp8(static_cast<int>(w[i]), false);
            hi = __builtin_amdgcn_cvt_pk_f32_fp8(static_cast<int>(w[i]), true);
        } else {
            lo = __builtin_amdgcn_cvt_pk_f32_bf8(static_cast<int>(w[i]), false);
            hi = __builtin_amdgcn_cvt_pk_f32_bf8(static_cast<int>(w[i]), true);
        }
        f[4 * i] = lo[0];
        if constexpr (V > 1) {
            f[4 * i + 1] = lo[1];
            f[4 * i + 2] = hi[0];
            f[4 * i + 3] = hi[1];
        }
    }
    constexpr bool kHalf = __is_same(T, _Float16);
    const uint32_t high = 127u + (kHalf ? 15u : 127u) - (format == UA2A_FORMAT_E4M3 ? 8u : 15u) + 1u;
    if (__builtin_amdgcn_ballot_w64(byte >= high) == 0) {
#pragma unroll
        for (int i = 0; i < V; ++i) f[i] *= s;
    } else {
        const float most = kHalf ? 65504.f : __uint_as_float(__is_same(T, float) ? 0x7f7fffffu : 0x7f7f0000u);
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const float r = f[i] * s;
            const bool past = fabsf(f[i]) < __uint_as_float(0x7f800000u) && fabsf(r) > most;
            f[i] = past ? copysignf(most, r) : r;
        }
    }
}

// ------------------------------------------------------------------- norms

// The weights of a lane's slots, in 32 bits (ones without a weight tensor,
// zero in padding).
template <class T, int V, int ITEMS>
__device__ __forceinline__ void load_weights(const NormGeom& g, const void* weight, int32_t f32, uint32_t lane,
                                             float (&wt)[ITEMS][V])
{
#pragma unroll
    for (int it = 0; it < ITEMS; ++it) {
        const Slot s = slot_of(g, lane + (static_cast<uint32_t>(it) << g.lanes_log), V);
        const uint32_t at = s.ok ? s.hh * g.sh.D + s.d : 0;
        if (weight == nullptr) {
#pragma unroll
            for (int i = 0; i < V; ++i) wt[it][i] = 1.f;
        } else if (f32) {
#pragma unroll
            for (int i = 0; i < V; ++i) wt[it][i] = static_cast<const float*>(weight)[at + i];
        } else {
            unpack<T, V>(*reinterpret_cast<const typename Raw<T, V>::type*>(static_cast<const T*>(weight) + at),
                         wt[it]);
        }
    }
}

// RMS norm joined with the exchange.  A segment's lanes hold it in registers
// between the pass that sums its squares and the one that writes, so every
// value is read once.
template <class T, int V, int ITEMS, int BLOCK>
__global__ __launch_bounds__(BLOCK) void ua2a_norm_kernel(NormArgs a, int32_t mode1)
{
    __shared__ float red[2][16];
    const NormGeom& g = a.g;
    const uint32_t lane = threadIdx.x & ((1u << g.lanes_log) - 1);
    float wt[ITEMS][V];
    load_weights<T, V, ITEMS>(g, a.weight, a.weight_f32, lane, wt);
    uint32_t round = 0;
    for (uint32_t group = blockIdx.x; group < g.groups; group += gridDim.x, ++round) {
        const Segment s = segment_of(g, group, threadIdx.x, BLOCK);
        typename Raw<T, V>::type h[ITEMS];
#pragma unroll
        for (int it = 0; it < ITEMS; ++it) {
            Slot sl = slot_of(g, lane + (static_cast<uint32_t>(it) << g.lanes_log), V);
            if (!sl.ok) sl.hh = sl.d = 0;
            h[it] = load_values<T, V>(a.x, value_at(g, s, sl, mode1));
        }
        if (a.residual != nullptr) {
            typename Raw<T, V>::type r[ITEMS];
#pragma unroll
            for (int it = 0; it < ITEMS; ++it) {
                Slot sl = slot_of(g, lane + (static_cast<uint32_t>(it) << g.lanes_log), V);
                if (!sl.ok) sl.hh = sl.d = 0;
                r[it] = load_values<T, V>(a.residual, value_at(g, s, sl, false));
            }
#pragma unroll
            for (int it = 0; it < ITEMS; ++it) {
                const Slot sl = slot_of(g, lane + (static_cast<uint32_t>(it) << g.lanes_log), V);
                float f[V], e[V];
                unpack<T, V>(h[it], f);
                unpack<T, V>(r[it], e);
#pragma unroll
                for (int i = 0; i < V; ++i) f[i] += e[i];
                h[it] = pack<T, V>(f);
                if (sl.ok && s.live) store_values<T, V>(a.sum, value_at(g, s, sl, false), h[it]);
            }
        }
        float ss = 0.f;
#pragma unroll
        for (int it = 0; it < ITEMS; ++it) {
            const Slot sl = slot_of(g, lane + (static_cast<uint32_t>(it) << g.lanes_log), V);
            float f[V], sq = 0.f;
            unpack<T, V>(h[it], f);
#pragma unroll
            for (int i = 0; i < V; ++i) sq += f[i] * f[i];
            ss += sl.ok ? sq : 0.f;
        }
        const float mean = segment_sum(ss, g.lanes_log, red, round) * a.inv_len;
        const float rstd = 1.f / __fsqrt_rn(mean + a.eps);
        if (a.rstd != nullptr && lane == 0 && s.live) a.rstd[s.seg] = rstd;
#pragma unroll
        for (int it = 0; it < ITEMS; ++it) {
            const Slot sl = slot_of(g, lane + (static_cast<uint32_t>(it) << g.lanes_log), V);
            const bool write = sl.ok && s.live;
            float f[V];
            unpack<T, V>(h[it], f);
            if (!sl.ok) {
#pragma unroll
                for (int i = 0; i < V; ++i) f[i] = 0.f;
            }
            if (a.saved_format) {
                uint32_t byte;
                const auto c = encode<V>(f, a.saved_format, &byte);
                if (write) {
                    store_once(a.saved + value_at(g, s, sl, false), c);
                    if ((lane & ((1u << q_log_of<V>()) - 1)) == 0)
                        a.saved_scales[scale_at(g, s, sl, false)] = static_cast<uint8_t>(byte);
                }
            }
#pragma unroll
            for (int i = 0; i < V; ++i) f[i] = f[i] * rstd * wt[it][i];
            if (a.out_format) {
                uint32_t byte;
                const auto c = encode<V>(f, a.out_format, &byte);
                if (write) {
                    store_once(static_cast<uint8_t*>(a.out) + value_at(g, s, sl, !mode1), c);
                    if ((lane & ((1u << q_log_of<V>()) - 1)) == 0)
                        a.out_scales[scale_at(g, s, sl, !mode1)] = static_cast<uint8_t>(byte);
                }
            } else if (write) {
                store_values<T, V>(a.out, value_at(g, s, sl, !mode1), pack<T, V>(f));
            }
        }
    }
}

// Backward pass of the norm and its exchange.  Workgroups walk over segments
// and keep the sums of dweight for their lanes' slots in registers; at the
// end each workgroup writes one row of partial sums.
template <class T, int V, int ITEMS, int BLOCK>
__global__ __launch_bounds__(BLOCK) void ua2a_norm_grad_kernel(NormGradArgs a, int32_t mode1)
{
    __shared__ float red[2][16];
    __shared__ float join[BLOCK * V];
    const NormGeom& g = a.g;
    const uint32_t lane = threadIdx.x & ((1u << g.lanes_log) - 1);
    float wt[ITEMS][V], dw[ITEMS][V];
    load_weights<T, V, ITEMS>(g, a.weight, a.weight_f32, lane, wt);
#pragma unroll
    for (int it = 0; it < ITEMS; ++it)
#pragma unroll
        for (int i = 0; i < V; ++i) dw[it][i] = 0.f;
    uint32_t round = 0;
    for (uint32_t group = blockIdx.x; group < g.groups; group += gridDim.x, ++round) {
        const Segment s = segment_of(g, group, threadIdx.x, BLOCK);
        typename Raw<T, V>::type dy[ITEMS], hv[ITEMS];
        typename Codes<V>::type hc[ITEMS];
        uint32_t hs[ITEMS];
        const float rstd = s.live ? a.rstd[s.seg] : 0.f;
#pragma unroll
        for (int it = 0; it < ITEMS; ++it) {
            Slot sl = slot_of(g, lane + (static_cast<uint32_t>(it) << g.lanes_log), V);
            if (!sl.ok) sl.hh = sl.d = sl.blk = 0;
            dy[it] = load_values<T, V>(a.dy, value_at(g, s, sl, !mode1));
            if (a.saved_format) {
                hc[it] = load_once<typename Codes<V>::type>(static_cast<const uint8_t*>(a.saved) +
                                                            value_at(g, s, sl, false));
                hs[it] = a.saved_scales[scale_at(g, s, sl, false)];
            } else {
                hv[it] = load_values<T, V>(a.saved, value_at(g, s, sl, a.saved_gathered));
            }
        }
        const auto normed = [&](int it, float(&n)[V]) {
            if (a.saved_format)
                decode<float, V>(hc[it], hs[it], a.saved_format, n);
            else
                unpack<T, V>(hv[it], n);
#pragma unroll
            for (int i = 0; i < V; ++i) n[i] *= rstd;
        };
        float dot = 0.f;
#pragma unroll
        for (int it = 0; it < ITEMS; ++it) {
            const Slot sl = slot_of(g, lane + (static_cast<uint32_t>(it) << g.lanes_log), V);
            float d[V], n[V], p = 0.f;
            unpack<T, V>(dy[it], d);
            normed(it, n);
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const float t = d[i] * n[i];
                p += t * wt[it][i];
                dw[it][i] += (sl.ok && s.live) ? t : 0.f;
            }
            dot += sl.ok ? p : 0.f;
        }
        const float mean = segment_sum(dot, g.lanes_log, red, round) * a.inv_len;
#pragma unroll
        for (int it = 0; it < ITEMS; ++it) {
            const Slot sl = slot_of(g, lane + (static_cast<uint32_t>(it) << g.lanes_log), V);
            float d[V], n[V];
            unpack<T, V>(dy[it], d);
            normed(it, n);
#pragma unroll
            for (int i = 0; i < V; ++i) d[i] = rstd * (d[i] * wt[it][i] - n[i] * mean);
            if (sl.ok && s.live) {
                const int64_t p = value_at(g, s, sl, false);
                if (a.dsum != nullptr) {
                    float e[V];
                    unpack<T, V>(load_values<T, V>(a.dsum, p), e);
#pragma unroll
                    for (int i = 0; i < V; ++i) d[i] += e[i];
                }
                const auto r = pack<T, V>(d);
                store_values<T, V>(a.dx, mode1 ? value_at(g, s, sl, true) : p, r);
                if (a.dresidual != nullptr) store_values<T, V>(a.dresidual, p, r);
            }
        }
    }
    if (a.partial == nullptr) return;
    // one row of sums per workgroup, the workgroup's segments joined in order
    const uint32_t lanes = 1u << g.lanes_log;
    const uint32_t per = BLOCK >> g.lanes_log;
    float* row = a.partial + static_cast<int64_t>(blockIdx.x) * g.len;
#pragma unroll
    for (int it = 0; it < ITEMS; ++it) {
        const Slot sl = slot_of(g, lane + (static_cast<uint32_t>(it) << g.lanes_log), V);
        if (per > 1) {
            __syncthreads();
#pragma unroll
            for (int i = 0; i < V; ++i) join[i * BLOCK + threadIdx.x] = dw[it][i];
            __syncthreads();
        }
        if (threadIdx.x < lanes && sl.ok) {
#pragma unroll
            for (int i = 0; i < V; ++i) {
                float t = dw[it][i];
                for (uint32_t k = 1; k < per; ++k) t += join[i * BLOCK + k * lanes + threadIdx.x];
                row[sl.hh * g.sh.D + sl.d + i] = t;
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

// ------------------------------------------------------------------- cache

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
    float f[V];
#pragma unroll
    for (int k = 0; k < V; ++k) f[k] = 0.f;
    if (ok) unpack<T, V>(load_values<T, V>(x, (static_cast<int64_t>(s.row) * g.sh.H + s.h) * g.sh.D + s.d), f);
    uint32_t byte;
    const auto c = encode<V>(f, a.format, &byte);
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
    float f[V];
    decode<T, V>(c, byte, a.format, f);
    store_values<T, V>(out, (static_cast<int64_t>(s.row) * g.sh.hl + s.h) * g.sh.D + s.d, pack<T, V>(f));
}

// ------------------------------------------------------------------- launch

template <class T, int V>
const void* norm_fn(const ActLaunch& L)
{
    if constexpr (V == 1) {
        if (L.block == kActBlock && L.items == 1)
            return reinterpret_cast<const void*>(&ua2a_norm_kernel<T, 1, 1, kActBlock>);
        if (L.block == kActBlock && L.items == 5)
            return reinterpret_cast<const void*>(&ua2a_norm_kernel<T, 1, 5, kActBlock>);
        if (L.block == kActBigBlock && L.items == 8)
            return reinterpret_cast<const void*>(&ua2a_norm_kernel<T, 1, 8, kActBigBlock>);
    } else {
        if (L.block == kActBlock) switch (L.items) {
            case 1: return reinterpret_cast<const void*>(&ua2a_norm_kernel<T, V, 1, kActBlock>);
            case 2: return reinterpret_cast<const void*>(&ua2a_norm_kernel<T, V, 2, kActBlock>);
            case 3: return reinterpret_cast<const void*>(&ua2a_norm_kernel<T, V, 3, kActBlock>);
            case 4: return reinterpret_cast<const void*>(&ua2a_norm_kernel<T, V, 4, kActBlock>);
            case 5: return reinterpret_cast<const void*>(&ua2a_norm_kernel<T, V, 5, kActBlock>);
            }
        if (L.block == kActBigBlock) switch (L.items) {
            case 2: return reinterpret_cast<const void*>(&ua2a_norm_kernel<T, V, 2, kActBigBlock>);
            case 4: return reinterpret_cast<const void*>(&ua2a_norm_kernel<T, V, 4, kActBigBlock>);
            case 8: return reinterpret_cast<const void*>(&ua2a_norm_kernel<T, V, 8, kActBigBlock>);
            }
    }
    return nullptr;
}

template <class T, int V>
const void* norm_grad_fn(const ActLaunch& L)
{
    if constexpr (V == 1) {
        if (L.block == kActBlock && L.items == 1)
            return reinterpret_cast<const void*>(&ua2a_norm_grad_kernel<T, 1, 1, kActBlock>);
        if (L.block == kActBlock && L.items == 5)
            return reinterpret_cast<const void*>(&ua2a_norm_grad_kernel<T, 1, 5, kActBlock>);
        if (L.block == kActBigBlock && L.items == 8)
            return reinterpret_cast<const void*>(&ua2a_norm_grad_kernel<T, 1, 8, kActBigBlock>);
    } else {
        if (L.block == kActBlock) switch (L.items) {
            case 1: return reinterpret_cast<const void*>(&ua2a_norm_grad_kernel<T, V, 1, kActBlock>);
            case 2: return reinterpret_cast<const void*>(&ua2a_norm_grad_kernel<T, V, 2, kActBlock>);
            case 3: return reinterpret_cast<const void*>(&ua2a_norm_grad_kernel<T, V, 3, kActBlock>);
            case 4: return reinterpret_cast<const void*>(&ua2a_norm_grad_kernel<T, V, 4, kActBlock>);
            case 5: return reinterpret_cast<const void*>(&ua2a_norm_grad_kernel<T, V, 5, kActBlock>);
            }
        if (L.block == kActBigBlock) switch (L.items) {
            case 2: return reinterpret_cast<const void*>(&ua2a_norm_grad_kernel<T, V, 2, kActBigBlock>);
            case 4: return reinterpret_cast<const void*>(&ua2a_norm_grad_kernel<T, V, 4, kActBigBlock>);
            case 8: return reinterpret_cast<const void*>(&ua2a_norm_grad_kernel<T, V, 8, kActBigBlock>);
            }
    }
    return nullptr;
}

template <class T, int V>
const void* typed_fn(const ActLaunch& L)
{
    switch (L.kernel) {
    case ActKernel::Norm: return norm_fn<T, V>(L);
    case ActKernel::NormGrad: return norm_grad_fn<T, V>(L);
    case ActKernel::CacheWrite: return reinterpret_cast<const void*>(&ua2a_cache_write_kernel<T, V>);
    case ActKernel::CacheRead: return reinterpret_cast<const void*>(&ua2a_cache_read_kernel<T, V>);
    default: return nullptr;
    }
}

}  // namespace

int act_launch(const ActLaunch& L, void* stream)
{
    const void* fn = nullptr;
    if (L.kernel == ActKernel::Columns)
        fn = reinterpret_cast<const void*>(&ua2a_columns_kernel);
    else if (L.type == UA2A_TYPE_BF16)
        fn = L.V == 8 ? typed_fn<__bf16, 8>(L) : typed_fn<__bf16, 1>(L);
    else if (L.type == UA2A_TYPE_FP16)
        fn = L.V == 8 ? typed_fn<_Float16, 8>(L) : typed_fn<_Float16, 1>(L);
    else
        fn = L.V == 4 ? typed_fn<float, 4>(L) : typed_fn<float, 1>(L);
    if (fn == nullptr) return static_cast<int>(hipErrorInvalidValue);
    int32_t mode = L.mode;
    void* args[2] = {nullptr, &mode};
    switch (L.kernel) {
    case ActKernel::Norm: args[0] = const_cast<NormArgs*>(&L.norm); break;
    case ActKernel::NormGrad: args[0] = const_cast<NormGradArgs*>(&L.grad); break;
    case ActKernel::Columns: args[0] = const_cast<ColumnArgs*>(&L.columns); break;
    default: args[0] = const_cast<CacheArgs*>(&L.cache); break;
    }
    const hipError_t e = hipLaunchKernel(fn, dim3(L.grid_x, L.grid_y, 1), dim3(L.block), args, 0,
                                         static_cast<hipStream_t>(stream));
    return e == hipSuccess ? 0 : static_cast<int>(e);
}

}  // namespace ua2a
