// gfx950 kernel of single tokens over the 8-bit cache (ua2a_attn.h): at most 16
// rows (query tokens times the heads that share a key head) over many keys, so
// the codes' bytes bound it.
//
// The waves of a workgroup take tiles of 32 keys in turn and share nothing until
// the end: no barrier stands between a wave and its loads, which run two tiles
// ahead in registers.  A tile is decoded into the wave's own stretch of LDS,
// whose rows then feed matrix tiles of 16 x 16, 32 deep
// (v_mfma_f32_16x16x32): lane l has column l % 16 of B and of the result, row
// l % 16 of A; quarter c = l / 16 has eight of the depth, and the result's rows
// 4c .. 4c + 3.  Two results of 16 keys are B of the product with the values, if
// its depth runs 4c + (0..3), 16 + 4c + (0..3).
//
// 32 sequences' single tokens, 4 heads each of 8 key heads of 128, a window of 4096
// positions (277 MB of codes): 54-61 us, 62 with codes kept in the caches, 80 in tiles
// shared by the workgroup behind barriers.  Twice the bytes take 98 us: 5.6 TB/s, and
// about 15 us of ramp and join in every call.  Two workgroups are resident on a CU;
// three spill, and more workgroups than fit gain nothing.
#include "ua2a_attn_device.h"

namespace ua2a {
namespace {

constexpr uint32_t kTileKeys = 32;
constexpr int kNonTemporal = 2;              // a buffer load's cache policy: nt

__device__ __forceinline__ int32_t least_of(int32_t a, uint32_t b)
{
    return a < static_cast<int32_t>(b) ? a : static_cast<int32_t>(b);
}

template <class T>
__device__ __forceinline__ f32x4v mfma16(u32x4v a, u32x4v b, f32x4v c)
{
    if constexpr (__is_same(T, __bf16))
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8v, a), __builtin_bit_cast(bf16x8v, b), c,
                                                       0, 0, 0);
    else
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8v, a), __builtin_bit_cast(f16x8v, b), c, 0,
                                                      0, 0);
}

// A wave's tile of keys and values on its way from memory: CH pieces of 16 codes
// per lane of each, and their scales.
template <class T, int DP>
struct WaveCodes {
    static constexpr int kAcross = DP / 16;                      // pieces of a row
    static constexpr int CH = kTileKeys * kAcross / 64;
    u32x4v k[CH], v[CH];
    uint32_t ks[CH], vs[CH];

    // Which piece of which row.  Rows of 128: eight lanes take four pieces of two
    // rows four apart, whose places in LDS lie in different banks.
    __device__ __forceinline__ static uint32_t row(int c)
    {
        const uint32_t lane = threadIdx.x & 63;
        if constexpr (DP == 128) return c * 8 + ((lane >> 3 & 3) | (lane & 4));
        return (lane + c * 64) / kAcross;
    }
    __device__ __forceinline__ static uint32_t piece(int c)
    {
        const uint32_t lane = threadIdx.x & 63;
        if constexpr (DP == 128) return (lane & 3) | (lane >> 3 & 4);
        return (lane + c * 64) % kAcross;
    }

    // j0: the tile's first position of this key head, in heads of D codes.  What
    // lies at or past `rows` positions is zeros (none: no row), past D too but
    // for the eight codes of a piece that holds D, which `put` clears.
    __device__ __forceinline__ void load(const AttnArgs& a, int64_t j0, int32_t rows)
    {
        const AttnGeom& g = a.g;
        const uint32_t step = g.kvl * g.D, sstep = g.kvl * g.nb;
        // up to the last row's D codes: its last piece may reach past them, where the tensor may end
        const uint32_t last = static_cast<uint32_t>(rows) - 1;
        const uint32_t bytes = rows > 0 ? last * step + g.D : 0, sbytes = rows > 0 ? last * sstep + g.nb : 0;
        const auto kd = resource(a.codes + j0 * g.D, bytes), vd = resource(a.codes + a.part + j0 * g.D, bytes);
        const auto ksd = resource(a.scales + j0 * g.nb, sbytes), vsd = resource(a.scales + a.part_scales + j0 * g.nb, sbytes);
#pragma unroll
        for (int c = 0; c < CH; ++c) {
            const uint32_t d = piece(c) * 16;
            const bool ok = d < g.D;
            const uint32_t at = ok ? row(c) * step + d : kNowhere, sat = ok ? row(c) * sstep + d / kBlockValues : kNowhere;
            // not kept in the caches, for nobody reads them again (62 us against 56)
            k[c] = __builtin_bit_cast(u32x4v, __builtin_amdgcn_raw_buffer_load_b128(kd, at, 0, kNonTemporal));
            v[c] = __builtin_bit_cast(u32x4v, __builtin_amdgcn_raw_buffer_load_b128(vd, at, 0, kNonTemporal));
            ks[c] = __builtin_amdgcn_raw_buffer_load_b8(ksd, sat, 0, 0);
            vs[c] = __builtin_amdgcn_raw_buffer_load_b8(vsd, sat, 0, 0);
        }
    }

    // One of them into the wave's tile.  Returns the largest scale byte.
    template <bool E4M3>
    __device__ __forceinline__ static uint32_t put(const u32x4v (&x)[CH], const uint32_t (&xs)[CH], char* tile, uint32_t D)
    {
        uint32_t top = 0;
#pragma unroll
        for (int c = 0; c < CH; ++c) {
            const bool whole = piece(c) * 16 + 16 <= D;
            const u32x2v lo = {x[c][0], x[c][1]}, hi = {whole ? x[c][2] : 0u, whole ? x[c][3] : 0u};
            *reinterpret_cast<u32x4v*>(tile + place_of<DP>(row(c), piece(c) * 32)) = decode8<T, E4M3>(lo, xs[c]);
            *reinterpret_cast<u32x4v*>(tile + place_of<DP>(row(c), piece(c) * 32 + 16)) = decode8<T, E4M3>(hi, xs[c]);
            top = max(top, xs[c]);
        }
        return top;
    }

    // Whether there are infinities or NaN among this lane's codes of e5m2 (what lies
    // past D may count too).  e4m3 has none but NaN, and scales past the type give none.
    __device__ __forceinline__ static bool unbounded(const u32x4v (&x)[CH])
    {
        uint32_t any = 0;
#pragma unroll
        for (int c = 0; c < CH; ++c)
#pragma unroll
            for (int i = 0; i < 4; ++i) any |= (x[c][i] & 0x7c7c7c7cu) + 0x04040404u;
        return (any & 0x80808080u) != 0;
    }
};

// Lanes of a wave read what others of it wrote: a wave's LDS operations run in
// order, so it is the compiler that must keep them so.
__device__ __forceinline__ void wave_order()
{
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
}

// The largest of a value and the neighbouring quarter's (lane 16 places on or back).
__device__ __forceinline__ float max_quarters(float x)
{
    const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    return fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
}

// A's operand with a row of the tile per lane, rows row0 .. + 15, depth step ks.
template <int DP>
__device__ __forceinline__ u32x4v along16(const char* tile, uint32_t row0, int ks)
{
    const uint32_t lane = threadIdx.x & 63;
    const uint32_t mine = place_of<DP>(lane & 15, (lane >> 4) * 16);
    uint32_t at = mine + ks * 64;
    if constexpr (DP % 64 == 0) at = mine ^ (ks * 64);
    return *reinterpret_cast<const u32x4v*>(tile + row0 * kRow<DP> + at);
}

// A's operand with a column per lane, columns 16 * db .., the 32 rows as depth in
// the order above.
template <int DP>
__device__ __forceinline__ u32x4v transposed16(const char* tile, int db)
{
    const uint32_t lane = threadIdx.x & 63;
    const uint32_t row = (lane >> 4) * 4 + ((lane & 15) >> 2);
    const uint32_t mine = place_of<DP>(row, (lane >> 1 & 1) * 16) + (lane & 1) * 8;
    uint32_t at;
    if constexpr (DP % 64 == 0)
        at = mine ^ (db * 32);
    else
        at = (mine ^ (db % 2 * 32)) + db / 2 * 64;
    typedef __attribute__((address_space(3))) s16x4v lds4;
    char* const p = const_cast<char*>(tile) + at;
    const s16x4v a = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4*)p);
    const s16x4v b = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4*)(p + 16 * kRow<DP>));
    const u32x2v x = __builtin_bit_cast(u32x2v, a), y = __builtin_bit_cast(u32x2v, b);
    return u32x4v{x[0], x[1], y[0], y[1]};
}

template <class T, int DP, bool E4M3>
__global__ __launch_bounds__(kAttnBlock, 2) void ua2a_attention_decode_kernel(AttnArgs a)
{
    constexpr uint32_t kTile = kTileKeys * kRow<DP>;
    __shared__ __attribute__((aligned(16))) char lds[4 * kTile];             // each wave's keys, then its values
    __shared__ __attribute__((aligned(16))) uint8_t wilds[4 * kTileKeys * (DP / 4)];
    __shared__ float stat[5 * kDecodeRows * 2];                              // the waves', then joined
    const AttnGeom& g = a.g;
    const uint32_t item = attn_item(g, (blockIdx.y << kAttnGridLog) + blockIdx.x);
    if (item >= g.items) return;
    const AttnPlace at = attn_place(g, item);
    const uint32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
    const uint32_t quarter = lane >> 4, col = lane & 15;
    char* const tile = lds + wave * kTile;
    uint8_t* const wild = wilds + wave * kTileKeys * (DP / 4);
    const AttnSeq seq = attn_seq(g, static_cast<int64_t>(a.starts[at.i]),
                                 a.counts != nullptr ? static_cast<int64_t>(a.counts[at.i]) : static_cast<int64_t>(g.n));
    const uint32_t past = g.rows;
    const bool in = col < past;
    const RowPlace place = row_place(g, at, in ? col : past - 1);
    const bool live = in && place.t >= seq.first && place.t < seq.last;

    f32x4v o[DP / 16];
#pragma unroll
    for (int db = 0; db < DP / 16; ++db) o[db] = f32x4v{0.f, 0.f, 0.f, 0.f};
    float m = -__builtin_inff(), l = 0.f;
    bool far = false;                                                        // uniform: some row's base is (far_base)
    if (seq.last > seq.first) {
        const Seen top = seen_by_row(g, seq, 0), bottom = seen_by_row(g, seq, past - 1);
        const Seen seen = seen_by_row(g, seq, place.row);
        const KeyWalk walk = key_walk(top, bottom, kTileKeys);
        const uint32_t from = split_at(walk.total, g.splits, at.split), to = split_at(walk.total, g.splits, at.split + 1);
        u32x4v q[DP / 32];
#pragma unroll
        for (int ks = 0; ks < DP / 32; ++ks) {
            const uint32_t d = ks * 32 + quarter * 8;
            q[ks] = u32x4v{0, 0, 0, 0};
            if (live && d < g.D) q[ks] = *reinterpret_cast<const u32x4v*>(static_cast<const uint16_t*>(a.q) + place.at + d);
        }
        const int64_t base = static_cast<int64_t>(at.seq) * g.keys * g.kvl + at.kvh;
        const auto position = [&](uint32_t i) { return walk_tile(walk, i) * kTileKeys; };
        WaveCodes<T, DP> next[2];
        const auto load = [&](uint32_t i, WaveCodes<T, DP>& w) {
            const uint32_t k0 = i < to ? position(i) : 0;
            w.load(a, base + static_cast<int64_t>(k0) * g.kvl, i < to ? least_of(seq.end - static_cast<int32_t>(k0), kTileKeys) : 0);
        };
        const auto step = [&](uint32_t i, WaveCodes<T, DP>& w) {
            const uint32_t k0 = i < to ? position(i) : 0, k1 = k0 + kTileKeys;
            const bool masked = i >= to || !all_seen(top, bottom, k0, k1);
            const int64_t j0 = base + static_cast<int64_t>(k0) * g.kvl;
            const int32_t rows = i < to ? least_of(seq.end - static_cast<int32_t>(k0), kTileKeys) : 0;
            constexpr int32_t kFormat = E4M3 ? UA2A_FORMAT_E4M3 : UA2A_FORMAT_E5M2;
            const uint32_t ktop = WaveCodes<T, DP>::template put<E4M3>(w.k, w.ks, tile, g.D);
            if (__builtin_amdgcn_ballot_w64(ktop >= high_scale<T>(kFormat)) != 0) {
                wave_order();                                    // over what other lanes put there
                decode_again<T, DP>(tile, g, a.codes + j0 * g.D, a.scales + j0 * g.nb, rows, kFormat, lane, 64);
            }
            wave_order();
            f32x4v s[2];
#pragma unroll
            for (int b = 0; b < 2; ++b) {
                s[b] = f32x4v{0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int ks = 0; ks < DP / 32; ++ks) s[b] = mfma16<T>(along16<DP>(tile, b * 16, ks), q[ks], s[b]);
            }
            wave_order();
            const uint32_t vtop = WaveCodes<T, DP>::template put<E4M3>(w.v, w.vs, tile, g.D);
            // zero times an infinity is NaN, and the weights' second parts may be zero or less
            const bool apart = masked || (!E4M3 && __builtin_amdgcn_ballot_w64(WaveCodes<T, DP>::unbounded(w.v)) != 0);
            load(i + 8, w);
            if (__builtin_amdgcn_ballot_w64(vtop >= high_scale<T>(kFormat)) != 0) {
                wave_order();
                decode_again<T, DP>(tile, g, a.codes + a.part + j0 * g.D, a.scales + a.part_scales + j0 * g.nb, rows, kFormat,
                                    lane, 64);
            }
            wave_order();
            bool odd = false;
            if (apart) {
                odd = __builtin_amdgcn_ballot_w64(tame_tile<T, DP>(tile, wild, kTileKeys, lane, 64)) != 0;
                wave_order();
            }
            if (i >= to) return;
            if (masked) {
#pragma unroll
                for (int x = 0; x < 8; ++x)
                    if (!sees(seen, k0 + (x / 4 * 16 + quarter * 4 + x % 4))) s[x / 4][x % 4] = -__builtin_inff();
            }
            float high = -__builtin_inff();
#pragma unroll
            for (int x = 0; x < 8; ++x) high = fmaxf(high, s[x / 4][x % 4]);
            high = max_halves(max_quarters(high)) * a.scale2;
            const bool grow = ahead_of<T>(high, m);
            if (__builtin_amdgcn_ballot_w64(grow) != 0) {
                const float now = fmaxf(m, base_of<T>(high)), f = now == m ? 1.f : __builtin_amdgcn_exp2f(m - now);
                m = now;
                far = __builtin_amdgcn_ballot_w64(far_base(now)) != 0;
                l *= f;
#pragma unroll
                for (int db = 0; db < DP / 16; ++db) o[db] *= f;
            }
            const float mm = m == -__builtin_inff() ? 0.f : m;
            float times = a.scale2, plus = -mm;
            if (far) {
#pragma unroll
                for (int x = 0; x < 8; ++x) s[x / 4][x % 4] = far_exponent(s[x / 4][x % 4], a.scale2, mm);
                times = 1.f;
                plus = 0.f;
            }
#pragma unroll
            for (int x = 0; x < 8; ++x) {
                s[x / 4][x % 4] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[x / 4][x % 4], times, plus));
                l += s[x / 4][x % 4];
            }
            const u32x4v p = {pack2<T>(s[0][0], s[0][1]), pack2<T>(s[0][2], s[0][3]), pack2<T>(s[1][0], s[1][1]),
                              pack2<T>(s[1][2], s[1][3])};
            // as two values of the type, for the products are not what bounds this kernel
            // (60.5 us, with one 59.7; an error of 1.0 times the result's own rounding's, with one 1.4)
            const u32x4v rest = {rest2<T>(s[0][0], s[0][1], p[0]), rest2<T>(s[0][2], s[0][3], p[1]),
                                 rest2<T>(s[1][0], s[1][1], p[2]), rest2<T>(s[1][2], s[1][3], p[3])};
#pragma unroll
            for (int db = 0; db < DP / 16; ++db) {
                const u32x4v v = transposed16<DP>(tile, db);
                o[db] = mfma16<T>(v, p, o[db]);
                o[db] = mfma16<T>(v, rest, o[db]);
            }
            if (!odd) return;
            uint32_t up[DP / 32], down[DP / 32];
#pragma unroll
            for (int w = 0; w < DP / 32; ++w) up[w] = down[w] = 0;
#pragma unroll 1
            for (uint32_t j = 0; j < kTileKeys; ++j) {
                const bool see = sees(seen, k0 + j);
                const uint32_t* bits = reinterpret_cast<const uint32_t*>(wild + j * (DP / 4));
#pragma unroll
                for (int w = 0; w < DP / 32; ++w) {
                    up[w] |= see ? bits[w] : 0u;
                    down[w] |= see ? bits[DP / 32 + w] : 0u;
                }
            }
#pragma unroll
            for (int db = 0; db < DP / 16; ++db)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const uint32_t bit = db % 2 * 16 + quarter * 4 + i;
                    if (up[db / 2] >> bit & 1) o[db][i] += __builtin_inff();
                    if (down[db / 2] >> bit & 1) o[db][i] -= __builtin_inff();
                }
        };
        // tiles from + wave, + 4, ...: two of them on their way
        // (in this order: a wait counts the loads behind the one it is for)
        load(from + wave, next[0]);
        asm volatile("" ::: "memory");
        load(from + wave + 4, next[1]);
        for (uint32_t i = from + wave; i < to; i += 8) {
            step(i, next[0]);
            wave_order();
            step(i + 4, next[1]);                                // past the last: a tile of zeros that is not used
            wave_order();
        }
    }
    l = add_halves(l + __shfl_xor(l, 16));
    if (quarter == 0) {
        stat[(wave * kDecodeRows + col) * 2] = m;
        stat[(wave * kDecodeRows + col) * 2 + 1] = l;
    }
    __syncthreads();
    float most = -__builtin_inff(), sum = 0.f;
#pragma unroll
    for (int w = 0; w < 4; ++w) most = fmaxf(most, stat[(w * kDecodeRows + col) * 2]);
    const float mm = most == -__builtin_inff() ? 0.f : most;
#pragma unroll
    for (int w = 0; w < 4; ++w)
        sum += stat[(w * kDecodeRows + col) * 2 + 1] * __builtin_amdgcn_exp2f(stat[(w * kDecodeRows + col) * 2] - mm);
    const float f = __builtin_amdgcn_exp2f(m - mm);
    float* const sums = reinterpret_cast<float*>(lds);           // [wave][row][DP]
#pragma unroll
    for (int db = 0; db < DP / 16; ++db)
        *reinterpret_cast<f32x4v*>(sums + (wave * kDecodeRows + col) * DP + db * 16 + quarter * 4) = o[db] * f;
    if (quarter == 0 && wave == 0) {
        stat[(4 * kDecodeRows + col) * 2] = most;
        stat[(4 * kDecodeRows + col) * 2 + 1] = sum;
    }
    __syncthreads();
    for (uint32_t i = threadIdx.x; i < kDecodeRows * (DP / 4); i += kAttnBlock) {
        const uint32_t c = i / (DP / 4), d = i % (DP / 4) * 4;
        if (c >= past || d >= g.D) continue;
        f32x4v x = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int w = 0; w < 4; ++w) x += *reinterpret_cast<const f32x4v*>(sums + (w * kDecodeRows + c) * DP + d);
        finish_row<T>(a, at, seq, c, d, x, stat[(4 * kDecodeRows + c) * 2], stat[(4 * kDecodeRows + c) * 2 + 1]);
    }
}

template <class T, int DP>
const void* sized_fn(const AttnLaunch& L)
{
    return L.attn.format == UA2A_FORMAT_E4M3 ? reinterpret_cast<const void*>(&ua2a_attention_decode_kernel<T, DP, true>)
                                             : reinterpret_cast<const void*>(&ua2a_attention_decode_kernel<T, DP, false>);
}

template <class T>
const void* typed_fn(const AttnLaunch& L)
{
    switch (L.DP) {
    case 32: return sized_fn<T, 32>(L);
    case 64: return sized_fn<T, 64>(L);
    case 96: return sized_fn<T, 96>(L);
    case 128: return sized_fn<T, 128>(L);
    }
    return nullptr;
}

}  // namespace

const void* decode_kernel(const AttnLaunch& L)
{
    return L.type == UA2A_TYPE_BF16 ? typed_fn<__bf16>(L) : typed_fn<_Float16>(L);
}

}  // namespace ua2a
