// Device functions that the attention kernels share: matrix tiles, their
// operands in LDS, and rows of keys on their way there.
//
// Matrix tiles are 32 x 32, 16 deep (v_mfma_f32_32x32x16).  Lane l of a wave
// has column l % 32 of B and of the result, row l % 32 of A; of the depth the
// half h = l / 32 has eight places, and of the result's rows 8g + 4h .. + 3 in
// its registers 4g .. 4g + 3.  A result goes into the next product as B
// without leaving its lane: its registers 8s .. 8s + 7 are the depth places of
// step s if A's depth runs in the order 16s + 4h + (0..3), 16s + 8 + 4h + (0..3),
// and that is what `transposed` reads.
#pragma once

#include "ua2a_act_device.h"
#include "ua2a_attn_internal.h"

namespace ua2a {
namespace {

typedef float f32x16v __attribute__((ext_vector_type(16)));
typedef float f32x4v __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8v __attribute__((ext_vector_type(8)));
typedef _Float16 f16x8v __attribute__((ext_vector_type(8)));
typedef short s16x4v __attribute__((ext_vector_type(4)));

template <class T>
__device__ __forceinline__ f32x16v mfma(u32x4v a, u32x4v b, f32x16v c)
{
    if constexpr (__is_same(T, __bf16))
        return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8v, a), __builtin_bit_cast(bf16x8v, b), c,
                                                       0, 0, 0);
    else
        return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8v, a), __builtin_bit_cast(f16x8v, b), c, 0,
                                                      0, 0);
}

// Two values in 32 bits rounded to the type, the first in the low half.
template <class T>
__device__ __forceinline__ uint32_t pack2(float a, float b)
{
    typedef T vec __attribute__((ext_vector_type(2)));
    const vec v = {static_cast<T>(a), static_cast<T>(b)};
    return __builtin_bit_cast(uint32_t, v);
}

// A result that is finite within the type.  The weights of a row's sums are rounded and the
// sum of the weights is not, so a mean of the type's largest values may come out a little
// past it: that is the largest, no infinity.
template <class T>
constexpr float kMost = __is_same(T, __bf16) ? 3.3895314e38f : 65504.f;
template <class T>
__device__ __forceinline__ float within(float x)
{
    return fabsf(x) < __builtin_inff() ? fminf(fmaxf(x, -kMost<T>), kMost<T>) : x;
}

// Registers 8s .. 8s + 7 of a result, rounded to the type: B's operand of depth step s.
template <class T>
__device__ __forceinline__ u32x4v operand_of(const f32x16v& c, int s)
{
    u32x4v r;
#pragma unroll
    for (int i = 0; i < 4; ++i) r[i] = pack2<T>(c[8 * s + 2 * i], c[8 * s + 2 * i + 1]);
    return r;
}

// A row's weights are held as exp2(score - base).  The base follows the row's largest
// score: set kLift under it, and set again when a score is more than kAhead over it, so
// that sums are rescaled a few times in all.  32 bits and bf16 have exponents to spare.
// fp16 has 11 digits from 2^-14 to 2^15 and loses them below, so there the largest is
// held between 2^13 and 2^15: weights keep their digits to 2^-27 of the largest, and half
// a step is 2^-38 of it (2^-14 and 2^-25 without: beside a token 17.4 nats above them the
// others of its walk were nothing).
template <class T>
constexpr float kLift = __is_same(T, __bf16) ? 0.f : 13.f;
template <class T>
constexpr float kAhead = __is_same(T, __bf16) ? 8.f : 15.f;

// A weight's exponent is fma(score, scale2, -base), and the base is a rounded product: the
// largest score's own exponent is off by up to half a step of its size, which the sums and
// their divisor share.  Past kFar, a step of 2^-7, both are taken from rounded products and
// nothing is lifted, or from 2^26 on weights would pass fp16, and from 2^33 on 32 bits.
constexpr float kFar = 65536.f;
__device__ __forceinline__ bool far_base(float m) { return fabsf(m) > kFar && fabsf(m) < __builtin_inff(); }

template <class T>
__device__ __forceinline__ float base_of(float top)
{
    return far_base(top) ? top : top - kLift<T>;
}

// Whether a row whose largest score is `top` needs another base.  The difference is exact
// where it is small; infinite where there was no score.
template <class T>
__device__ __forceinline__ bool ahead_of(float top, float m)
{
    return top - m > kAhead<T>;
}

__device__ __forceinline__ float far_exponent(float score, float scale2, float m)
{
    float x = score * scale2;
    asm("" : "+v"(x));                                           // no fma of the two
    return x - m;
}

// Log of a row's sum from its base m and the sum l of its weights; the lift is taken out
// first (exactly), so that one near zero keeps its digits.
template <class T>
__device__ __forceinline__ float lse_of(float m, float l)
{
    return l != 0.f ? (m + kLift<T>) * kLn2 + logf(l * (1.f / static_cast<float>(1 << static_cast<int>(kLift<T>)))) : -__builtin_inff();
}

// What rounding to a pair of the type left of two values, rounded itself.
template <class T>
__device__ __forceinline__ uint32_t rest2(float a, float b, uint32_t rounded)
{
    const auto x = pair_of<T>(rounded);
    return pack2<T>(a - static_cast<float>(x[0]), b - static_cast<float>(x[1]));
}

// What operand_of's rounding left.
template <class T>
__device__ __forceinline__ u32x4v rest_of(const f32x16v& c, u32x4v rounded, int s)
{
    u32x4v r;
#pragma unroll
    for (int i = 0; i < 4; ++i) r[i] = rest2<T>(c[8 * s + 2 * i], c[8 * s + 2 * i + 1], rounded[i]);
    return r;
}

// The largest, and the sum, of a value and the other half's (lane 32 places on or back).
__device__ __forceinline__ float max_halves(float x)
{
    const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    return fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
}
__device__ __forceinline__ float add_halves(float x)
{
    const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}

// A tile of rows in LDS, DP values each, in chunks of 16 bytes.  Row r keeps its
// chunk c in place c ^ f(r), so that what lanes read together lies in different
// banks: eight rows' chunks of one place (`along`), and four rows' pairs of
// neighbouring chunks (`transposed`).  Offsets in bytes; f does not change with
// multiples of 16 rows, and xor takes the depth step apart from the lane's part.
template <int DP>
constexpr uint32_t kRow = DP * 2;
template <int DP>
__device__ __forceinline__ uint32_t swizzle(uint32_t row)
{
    if constexpr (DP % 64 == 0)
        return ((row & 3) << 1 | (row >> 2 & 1) | (DP == 128 ? row & 8 : 0)) << 4;
    else
        return (row >> 1 & 3) << 4;
}
// Where chunk c (a multiple of 16 bytes along the row) of a row is kept.
template <int DP>
__device__ __forceinline__ uint32_t place_of(uint32_t row, uint32_t bytes)
{
    return row * kRow<DP> + (bytes ^ swizzle<DP>(row));
}

// A's operand with a row of the tile per lane: rows row0 .. + 31 (row0 a multiple
// of 32), depth step ks along the row.
template <int DP>
__device__ __forceinline__ u32x4v along(const char* tile, uint32_t row0, int ks)
{
    constexpr uint32_t kMask = DP % 64 == 0 ? ~0u : 63u;
    const uint32_t lane = threadIdx.x & 63;
    const uint32_t mine = place_of<DP>(lane & 31, (lane >> 5) * 16);
    return *reinterpret_cast<const u32x4v*>(tile + row0 * kRow<DP> + (ks * 32 & ~kMask) + (mine ^ (ks * 32 & kMask)));
}

// A's operand with a column of the tile per lane, the depth along the rows in
// the order above: rows row0 + 16s .. + 15 (row0 a multiple of 16), columns 32 * db ...
// ds_read_b64_tr_b16 hands lane i of 16 lanes value i of the four rows whose
// 32 bytes their addresses name, four lanes a row.
template <int DP>
__device__ __forceinline__ u32x4v transposed(const char* tile, uint32_t row0, int s, int db)
{
    const uint32_t lane = threadIdx.x & 63;
    const uint32_t row = (lane >> 5) * 4 + ((lane & 15) >> 2);
    const uint32_t mine = place_of<DP>(row, (lane >> 4 & 1) * 32 + (lane >> 1 & 1) * 16) + (lane & 1) * 8;
    uint32_t at = mine + db * 64;
    if constexpr (DP % 64 == 0) at = mine ^ (db * 64);
    typedef __attribute__((address_space(3))) s16x4v lds4;
    char* const p = const_cast<char*>(tile) + (row0 + 16 * s) * kRow<DP>;
    const s16x4v a = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4*)(p + at));
    const s16x4v b = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4*)(p + 8 * kRow<DP> + (DP == 128 ? at ^ 128u : at)));
    const u32x2v x = __builtin_bit_cast(u32x2v, a), y = __builtin_bit_cast(u32x2v, b);
    return u32x4v{x[0], x[1], y[0], y[1]};
}

// A tile of ROWS rows from memory straight into LDS: a wave's load moves 64
// chunks, 16 bytes a lane, to consecutive places; lanes fetch the chunks that
// belong there.  Reads past the descriptor's bytes give zeros: rows that do not
// exist, and chunks past D (kNowhere).  The loads are outstanding until
// `arrived`, which the compiler does not know: nothing may read the tile before.  Nor does
// it know of the wait there: registers that it loads before a loop it waits for once more
// at their first use within, and for the loads to LDS issued since.
constexpr uint32_t kNowhere = 0x80000000u;

template <int DP, int ROWS>
struct TileLoads {
    static constexpr int kAcross = DP / 8;
    static constexpr int kTotal = ROWS * kAcross / 64;           // loads of all waves
    static constexpr int N = (kTotal + 3) / 4;
    static constexpr uint32_t kBytes = ROWS * DP * 2;

    // the tile's row of this lane's load n, and which bytes of it
    __device__ __forceinline__ static uint32_t row(int n, uint32_t wave)
    {
        return ((n * 4 + wave) * 64 + (threadIdx.x & 63)) / kAcross;
    }
    __device__ __forceinline__ static uint32_t bytes(int n, uint32_t wave, uint32_t D)
    {
        const uint32_t r = row(n, wave), place = ((n * 4 + wave) * 64 + (threadIdx.x & 63)) % kAcross;
        const uint32_t at = (place * 16) ^ swizzle<DP>(r);
        return at < D * 2 ? at : kNowhere;
    }
    // uniform: whether the wave has a load n
    __device__ __forceinline__ static bool has(int n, uint32_t wave) { return n * 4 + 3 < kTotal || n * 4 + wave < kTotal; }
};

// What a descriptor's reads start from and how many bytes there are (uniform).
__device__ __forceinline__ u32x4v descriptor(const void* base, uint32_t bytes)
{
    const uint64_t b = reinterpret_cast<uint64_t>(base);
    return u32x4v{static_cast<uint32_t>(__builtin_amdgcn_readfirstlane(static_cast<uint32_t>(b))),
                  static_cast<uint32_t>(__builtin_amdgcn_readfirstlane(static_cast<uint32_t>(b >> 32) & 0xffffu)),
                  static_cast<uint32_t>(__builtin_amdgcn_readfirstlane(bytes)), 0x00020000u};
}

// The same for the compiler's own buffer loads.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t resource(const void* base, uint32_t bytes)
{
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(base), 0, static_cast<int>(bytes), 0x00020000);
}

// One load of a wave: 16 bytes from `offset` of each lane to consecutive places
// from `to` on.  The destination comes in m0, which is put back.
__device__ __forceinline__ void load_to_lds(u32x4v from, uint32_t offset, const char* to)
{
    typedef __attribute__((address_space(3))) const char lds;
    const uint32_t at = __builtin_amdgcn_readfirstlane(static_cast<uint32_t>(reinterpret_cast<uintptr_t>((lds*)to)));
    uint32_t m0;
    asm volatile("s_mov_b32 %0, m0\n\ts_mov_b32 m0, %1\n\ts_nop 0\n\tbuffer_load_dwordx4 %2, %3, 0 offen lds\n\ts_mov_b32 m0, %0"
                 : "=&s"(m0)
                 : "s"(at), "v"(offset), "s"(from)
                 : "memory");
}

// This wave's loads have arrived; after the barrier everyone's have, and what
// was read before it may be overwritten.
__device__ __forceinline__ void arrived()
{
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    __syncthreads();
}

// B's operands of a row per lane, straight from memory: chunk ks * 2 + half.
// Values past D are zeros.
template <int DP>
__device__ __forceinline__ void row_operands(const void* row, uint32_t D, uint32_t half, bool live, u32x4v (&r)[DP / 16])
{
#pragma unroll
    for (int ks = 0; ks < DP / 16; ++ks) {
        const uint32_t d = ks * 16 + half * 8;
        r[ks] = u32x4v{0, 0, 0, 0};
        if (live && d < D) r[ks] = *reinterpret_cast<const u32x4v*>(static_cast<const uint16_t*>(row) + d);
    }
}

// Where a row's values start: of q and out, and its place among the statistics.
struct RowPlace {
    int64_t at;                  // elements
    int64_t stat;                // lse
    uint32_t row;
    int32_t t;
};

__device__ __forceinline__ RowPlace row_place(const AttnGeom& g, const AttnPlace& p, uint32_t row)
{
    RowPlace r;
    const uint32_t t = fdiv(row, g.d_group);
    const uint32_t head = p.kvh * g.group + (row - t * g.group);
    r.row = row;
    r.t = static_cast<int32_t>(t);
    r.at = ((static_cast<int64_t>(p.seq) * g.n + t) * g.hl + head) * g.D;
    r.stat = (static_cast<int64_t>(p.seq) * g.hl + head) * g.n + t;
    return r;
}

// Infinities and NaN among eight values: whether there are any, the values with
// zeros in their places, and a bit for each that is NaN or the infinity of a
// sign (0 or 0x8000).
template <class T>
__device__ __forceinline__ constexpr uint32_t exponent_bits()
{
    return __is_same(T, __bf16) ? 0x7f80u : 0x7c00u;
}
template <class T>
__device__ __forceinline__ bool unbounded(u32x4v r)
{
    constexpr uint32_t kExp = exponent_bits<T>() * 0x10001u;
    constexpr uint32_t kOne = __is_same(T, __bf16) ? 0x00800080u : 0x04000400u;
    uint32_t any = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) any |= (r[i] & kExp) + kOne;
    return (any & 0x80008000u) != 0;
}
template <class T>
__device__ __forceinline__ u32x4v finite_part(u32x4v v)
{
    constexpr uint32_t kExp = exponent_bits<T>();
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if ((v[i] & kExp) == kExp) v[i] &= 0xffff0000u;
        if ((v[i] >> 16 & kExp) == kExp) v[i] &= 0xffffu;
    }
    return v;
}
template <class T>
__device__ __forceinline__ uint32_t unbounded_bits(u32x4v v, uint32_t sign)
{
    constexpr uint32_t kExp = exponent_bits<T>();
    uint32_t bits = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const uint32_t w = v[i / 2] >> (i % 2 * 16) & 0xffffu;
        if (w == (kExp | sign) || (w & 0x7fffu) > kExp) bits |= 1u << i;
    }
    return bits;
}

// Infinities and NaN of a tile's values become zeros, and a bit each in `wild`
// ([row][2][DP / 8] bytes: +inf or NaN, -inf or NaN).  Returns whether this chunk
// had any.
template <class T, int DP>
__device__ __forceinline__ bool tame(u32x4v& v, uint8_t* wild, uint32_t row, uint32_t chunk)
{
    const bool mine = unbounded<T>(v);
    uint32_t up = 0, down = 0;
    if (mine) {
        up = unbounded_bits<T>(v, 0);
        down = unbounded_bits<T>(v, 0x8000u);
        v = finite_part<T>(v);
    }
    uint8_t* bits = wild + row * (DP / 4) + chunk;
    bits[0] = static_cast<uint8_t>(up);
    bits[DP / 8] = static_cast<uint8_t>(down);
    return mine;
}

// Eight codes in the type, code * scale rounded once, by the scaled conversions;
// for scales at which no code passes what the type holds (decode_raw is for all).
template <class T, bool E4M3>
__device__ __forceinline__ u32x4v decode8(u32x2v c, uint32_t byte)
{
    const float s = read_scale_of(byte);
    u32x4v r;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        if constexpr (__is_same(T, __bf16)) {
            if constexpr (E4M3) {
                r[2 * i] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(c[i], s, false));
                r[2 * i + 1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(c[i], s, true));
            } else {
                r[2 * i] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_bf8(c[i], s, false));
                r[2 * i + 1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_bf8(c[i], s, true));
            }
        } else {
            if constexpr (E4M3) {
                r[2 * i] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(c[i], s, false));
                r[2 * i + 1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(c[i], s, true));
            } else {
                r[2 * i] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_bf8(c[i], s, false));
                r[2 * i + 1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_bf8(c[i], s, true));
            }
        }
    }
    return r;
}

// The same over a tile of `rows` rows in LDS, by `lanes` lanes: returns whether this
// lane met any.
template <class T, int DP>
__device__ __forceinline__ bool tame_tile(char* tile, uint8_t* wild, uint32_t rows, uint32_t lane, uint32_t lanes)
{
    bool odd = false;
#pragma unroll 1
    for (uint32_t i = lane; i < rows * (DP / 8); i += lanes) {
        const uint32_t row = i / (DP / 8), chunk = i % (DP / 8);
        char* const p = tile + place_of<DP>(row, chunk * 16);
        u32x4v v = *reinterpret_cast<const u32x4v*>(p);
        if (tame<T, DP>(v, wild, row, chunk)) {
            *reinterpret_cast<u32x4v*>(p) = v;
            odd = true;
        }
    }
    return odd;
}

// A tile of a cache decoded once more, as decode_raw does, which keeps codes past
// the type's largest value there: for scales at which there are such.  The codes
// and scales of `rows` positions are read again.
template <class T, int DP>
__device__ __forceinline__ void decode_again(char* tile, const AttnGeom& g, const uint8_t* codes, const uint8_t* scales,
                                             int32_t rows, int32_t format, uint32_t lane, uint32_t lanes)
{
#pragma unroll 1
    for (uint32_t i = lane; i < static_cast<uint32_t>(rows) * (DP / 8); i += lanes) {
        const uint32_t row = i / (DP / 8), chunk = i % (DP / 8), d = chunk * 8;
        if (d >= g.D) continue;
        const u32x2v c = *reinterpret_cast<const u32x2v*>(codes + static_cast<int64_t>(row) * g.kvl * g.D + d);
        const uint32_t byte = scales[static_cast<int64_t>(row) * g.kvl * g.nb + d / kBlockValues];
        *reinterpret_cast<u32x4v*>(tile + place_of<DP>(row, chunk * 16)) = decode_raw<T, 8>(c, byte, format);
    }
}

// The least scale byte at which a code may pass the type's largest value.
template <class T>
__device__ __forceinline__ uint32_t high_scale(int32_t format)
{
    return 127u + (__is_same(T, _Float16) ? 15u : 127u) - (format == UA2A_FORMAT_E4M3 ? 8u : 15u) + 1u;
}

// Four values d .. of a row's sums, with its maximum and sum: the result, or a
// part's place in the workspace.  The lane of d = 0 writes the statistics.
template <class T>
__device__ __forceinline__ void finish_row(const AttnArgs& a, const AttnPlace& at, const AttnSeq& seq, uint32_t row,
                                           uint32_t d, f32x4v x, float m, float l)
{
    const AttnGeom& g = a.g;
    const RowPlace pl = row_place(g, at, row);
    const bool live = pl.t >= seq.first && pl.t < seq.last;
    if (g.splits > 1) {
        const int64_t line = (static_cast<int64_t>(at.split) * g.units + at.unit) * g.rows + row;
        *reinterpret_cast<f32x4v*>(a.partial + line * g.D + d) = x;
        if (d == 0) {
            a.stats[line * 2] = live ? m : -__builtin_inff();
            a.stats[line * 2 + 1] = live ? l : 0.f;
        }
        return;
    }
    if (!live && a.keep) return;
    const float inv = live && l != 0.f ? 1.f / l : 0.f;
    u32x2v y = {0, 0};
    if (live)
        y = u32x2v{pack2<T>(within<T>(x[0] * inv), within<T>(x[1] * inv)), pack2<T>(within<T>(x[2] * inv), within<T>(x[3] * inv))};
    *reinterpret_cast<u32x2v*>(static_cast<uint16_t*>(a.out) + pl.at + d) = y;
    if (d == 0 && a.lse != nullptr) a.lse[pl.stat] = live ? lse_of<T>(m, l) : -__builtin_inff();
}

}  // namespace
}  // namespace ua2a
