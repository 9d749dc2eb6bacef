// Device functions that the activation operators' kernels share: values as
// they are stored, sums over lanes, and 8 bits with scales.
#pragma once

#include <hip/hip_runtime.h>

#include <type_traits>

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

// Sum over aligned groups of `lanes` lanes of a wave, a power of two (uniform).
__device__ __forceinline__ float group_sum(float x, uint32_t lanes)
{
    if (lanes > 1) x = dpp_add<kDppXor1>(x);
    if (lanes > 2) x = dpp_add<kDppXor2>(x);
    if (lanes > 4) x = dpp_add<kDppHalfMirror>(x);
    if (lanes > 8) x = dpp_add<kDppMirror>(x);
    if (lanes > 16) x += __shfl_xor(x, 16);
    if (lanes > 32) x += __shfl_xor(x, 32);
    return x;
}

// Two values of a 2-byte type from their word.  (By value: a cast of a vector's
// element in place would take the vector's first.)
typedef __bf16 bf16x2v __attribute__((ext_vector_type(2)));
typedef _Float16 f16x2v __attribute__((ext_vector_type(2)));

template <class T>
__device__ __forceinline__ auto pair_of(uint32_t word)
{
    if constexpr (__is_same(T, __bf16))
        return __builtin_bit_cast(bf16x2v, word);
    else
        return __builtin_bit_cast(f16x2v, word);
}

// Sum of the squares of V values in 32 bits; pairs of the 2-byte types by the
// dot instructions, which widen them exactly.
template <class T, int V>
__device__ __forceinline__ float squares(typename Raw<T, V>::type r, float sum)
{
    if constexpr (V == 8) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const auto p = pair_of<T>(r[i]);
            if constexpr (__is_same(T, __bf16))
                sum = __builtin_amdgcn_fdot2_f32_bf16(p, p, sum, false);
            else
                sum = __builtin_amdgcn_fdot2(p, p, sum, false);
        }
    } else {
        float f[V];
        unpack<T, V>(r, f);
#pragma unroll
        for (int i = 0; i < V; ++i) sum += f[i] * f[i];
    }
    return sum;
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
// 2^(byte - 127), byte at most 254.
__device__ __forceinline__ float scale_of(uint32_t byte)
{
    return __uint_as_float(byte ? byte << 23 : 0x400000u);
}
// The same of a byte that was read: 255 is NaN.  One bit below the exponent
// makes both of its ends what they stand for.
__device__ __forceinline__ float read_scale_of(uint32_t byte)
{
    return __uint_as_float(byte << 23 | (((byte + 1) & 0xfe) == 0 ? 0x400000u : 0u));
}

// The codes of V values at a scale, by gfx950's scaled conversions: each
// divides by the power of two exactly and rounds once to nearest even
// (checked over every 16-bit pattern at every scale), infinities and NaN
// become what the format has for them.
typedef short s16x2v __attribute__((ext_vector_type(2)));

template <class P>
__device__ __forceinline__ uint32_t convert4(P lo, P hi, float scale, int32_t format)
{
    s16x2v c = {0, 0};
    if constexpr (__is_same(P, bf16x2v)) {
        if (format == UA2A_FORMAT_E4M3) {
            c = __builtin_amdgcn_cvt_scalef32_pk_fp8_bf16(c, lo, scale, false);
            c = __builtin_amdgcn_cvt_scalef32_pk_fp8_bf16(c, hi, scale, true);
        } else {
            c = __builtin_amdgcn_cvt_scalef32_pk_bf8_bf16(c, lo, scale, false);
            c = __builtin_amdgcn_cvt_scalef32_pk_bf8_bf16(c, hi, scale, true);
        }
    } else if constexpr (__is_same(P, f16x2v)) {
        if (format == UA2A_FORMAT_E4M3) {
            c = __builtin_amdgcn_cvt_scalef32_pk_fp8_f16(c, lo, scale, false);
            c = __builtin_amdgcn_cvt_scalef32_pk_fp8_f16(c, hi, scale, true);
        } else {
            c = __builtin_amdgcn_cvt_scalef32_pk_bf8_f16(c, lo, scale, false);
            c = __builtin_amdgcn_cvt_scalef32_pk_bf8_f16(c, hi, scale, true);
        }
    } else {
        if (format == UA2A_FORMAT_E4M3) {
            c = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(c, lo[0], lo[1], scale, false);
            c = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(c, hi[0], hi[1], scale, true);
        } else {
            c = __builtin_amdgcn_cvt_scalef32_pk_bf8_f32(c, lo[0], lo[1], scale, false);
            c = __builtin_amdgcn_cvt_scalef32_pk_bf8_f32(c, hi[0], hi[1], scale, true);
        }
    }
    return __builtin_bit_cast(uint32_t, c);
}

constexpr uint32_t kInfBits = 0x7f800000u;

// Codes of V values in 32 bits of a block shared by 2^q_log lanes, and its
// scale byte.  Infinities and NaN stay out of the block's magnitude (looked
// for only when one shows up: their bits are the largest).
template <int V>
__device__ __forceinline__ typename Codes<V>::type encode(const float (&f)[V], int32_t format, uint32_t* byte)
{
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < V; ++i) m = max(m, __float_as_uint(f[i]) & 0x7fffffffu);
    uint32_t top = group_max<q_log_of<V>()>(m);
    if (__builtin_amdgcn_ballot_w64(top >= kInfBits) != 0) {
        m = 0;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const uint32_t a = __float_as_uint(f[i]) & 0x7fffffffu;
            m = max(m, a < kInfBits ? a : 0u);
        }
        top = group_max<q_log_of<V>()>(m);
    }
    *byte = scale_byte(top, format);
    const float scale = scale_of(*byte);
    if constexpr (V == 1) {
        return static_cast<uint8_t>(convert4(f32x2v{f[0], f[0]}, f32x2v{f[0], f[0]}, scale, format));
    } else {
        const uint32_t c0 = convert4(f32x2v{f[0], f[1]}, f32x2v{f[2], f[3]}, scale, format);
        if constexpr (V == 8)
            return u32x2v{c0, convert4(f32x2v{f[4], f[5]}, f32x2v{f[6], f[7]}, scale, format)};
        else
            return c0;
    }
}

// The same of values as they are stored; for the 16-byte vectors of the
// 2-byte types without widening them: the largest magnitude is a packed
// integer maximum, and the conversions take pairs.
template <class T, int V>
__device__ __forceinline__ typename Codes<V>::type encode_raw(typename Raw<T, V>::type r, int32_t format, uint32_t* byte)
{
    if constexpr (V != 8) {
        float f[V];
        unpack<T, V>(r, f);
        return encode<V>(f, format, byte);
    } else {
        typedef uint16_t u16x2v __attribute__((ext_vector_type(2)));
        constexpr uint32_t kInf = __is_same(T, __bf16) ? 0x7f80u : 0x7c00u;
        u16x2v t[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) t[i] = __builtin_bit_cast(u16x2v, r[i] & 0x7fff7fffu);
        const auto join = [&]() {
            const u16x2v m = __builtin_elementwise_max(__builtin_elementwise_max(t[0], t[1]),
                                                       __builtin_elementwise_max(t[2], t[3]));
            return group_max<2>(max(static_cast<uint32_t>(m[0]), static_cast<uint32_t>(m[1])));
        };
        uint32_t top = join();
        if (__builtin_amdgcn_ballot_w64(top >= kInf) != 0) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                t[i] = u16x2v{t[i][0] < kInf ? t[i][0] : uint16_t(0), t[i][1] < kInf ? t[i][1] : uint16_t(0)};
            top = join();
        }
        if constexpr (__is_same(T, __bf16)) {
            *byte = scale_byte(top << 16, format);
            const float scale = scale_of(*byte);
            return u32x2v{convert4(pair_of<T>(r[0]), pair_of<T>(r[1]), scale, format),
                          convert4(pair_of<T>(r[2]), pair_of<T>(r[3]), scale, format)};
        } else {
            const float wide = static_cast<float>(__builtin_bit_cast(_Float16, static_cast<uint16_t>(top)));
            *byte = scale_byte(__float_as_uint(wide), format);
            const float scale = scale_of(*byte);
            return u32x2v{convert4(pair_of<T>(r[0]), pair_of<T>(r[1]), scale, format),
                          convert4(pair_of<T>(r[2]), pair_of<T>(r[3]), scale, format)};
        }
    }
}

// The values of codes, without their scale (exact).
template <int V>
__device__ __forceinline__ void code_values(typename Codes<V>::type c, int32_t format, float (&f)[V])
{
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
}

// Codes back in the type, as they are stored: code * scale, exact in 32 bits
// (codes are multiples of 2^-16, scales at least 2^-127), rounded once.  Only
// a block's largest value, rounded up, can pass what T holds; that takes a
// scale of 2^(T's largest exponent - the format's + 1) at least, looked for
// per block, and such finite codes give T's largest value.
template <class T, int V>
__device__ __forceinline__ typename Raw<T, V>::type decode_raw(typename Codes<V>::type c, uint32_t byte, int32_t format)
{
    constexpr bool kHalf = __is_same(T, _Float16);
    const float s = read_scale_of(byte);
    const uint32_t high = 127u + (kHalf ? 15u : 127u) - (format == UA2A_FORMAT_E4M3 ? 8u : 15u) + 1u;
    float f[V];
    if (__builtin_amdgcn_ballot_w64(byte >= high) == 0) {
        if constexpr (V == 8) {
            u32x4v r;
            if constexpr (kHalf) {
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    if (format == UA2A_FORMAT_E4M3) {
                        r[2 * i] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(c[i], s, false));
                        r[2 * i + 1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(c[i], s, true));
                    } else {
                        r[2 * i] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_bf8(c[i], s, false));
                        r[2 * i + 1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_bf8(c[i], s, true));
                    }
                }
            } else {
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    if (format == UA2A_FORMAT_E4M3) {
                        r[2 * i] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(c[i], s, false));
                        r[2 * i + 1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(c[i], s, true));
                    } else {
                        r[2 * i] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_bf8(c[i], s, false));
                        r[2 * i + 1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_bf8(c[i], s, true));
                    }
                }
            }
            return r;
        } else {
            code_values<V>(c, format, f);
#pragma unroll
            for (int i = 0; i < V; ++i) f[i] *= s;
        }
    } else {
        const float most = kHalf ? 65504.f : __uint_as_float(__is_same(T, float) ? 0x7f7fffffu : 0x7f7f0000u);
        code_values<V>(c, format, f);
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const float v = f[i] * s;
            const bool past = fabsf(f[i]) < __uint_as_float(kInfBits) && fabsf(v) > most;
            f[i] = past ? copysignf(most, v) : v;
        }
    }
    return pack<T, V>(f);
}

// Keeps the compiler from carrying what it computes from x across this point:
// values are unpacked again from the registers they were loaded into (one
// operation each), which holds a lane's registers to a third of what keeping
// them in 32 bits between the two passes takes.
template <class R>
__device__ __forceinline__ void forget(R& x)
{
    if constexpr (sizeof(R) >= 4) asm volatile("" : "+v"(x));
}

}  // namespace
}  // namespace ua2a
