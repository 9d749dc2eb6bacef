// gfx950 kernels of windowed attention (ua2a_attn.h): of gathered heads, and of
// new tokens over the 8-bit cache.
//
// One pass over the keys with the running maximum m and sum l of each row's
// softmax, in 32 bits: o = sum exp(s - m) v, rescaled when m grows.  A row is
// a query token and head; heads that share a key head lie in one tile, so its
// keys are read once for all of them.  A wave has 32 rows as the columns of its
// matrix tiles: scores come as keys x rows, so a row's maximum and sum are a
// lane's own work but for the other half's, and the weights go on to the
// product with the values from the registers they are in.
//
// The matrix products and the exponentials take its time, about as much of either with
// heads of 128: 40 heads over 75,600 tokens, a window of three frames of 3600 and
// the first, take 21.4 ms (22.4 on a slower card), 966 TFLOP/s, where a product of two
// 8192 x 8192 matrices by the library reaches 1162 (matrix units busy 44 % of the time,
// the others 42, waves waiting a third).  Part of that waiting is the next tile's loads:
// the compiler knows nothing of the wait in `arrived`, takes the rows' operands for
// outstanding still, and waits for all loads before the first product of each tile.
// The other workgroup on the CU fills most of it; the variants below were timed with it.
// Everything visible, 32 heads of 128 over 8192 tokens: 938 TFLOP/s; heads of 64, with
// as many exponentials for half the products, 886; a window of 1024 of such, whose walks
// are 18 tiles with a quarter of them masked, 500 to 670.  A cache's keys are decoded on
// their way (1560 tokens of 12 heads over 7,800 positions: 610 TFLOP/s).  Tiles go
// straight from memory to LDS, in two buffers with a barrier a tile (24.6 ms through
// registers, 22.5 so); a row's halves are joined in registers and
// the wave at its products has priority (21.5).  Blocks of 32 keys worked on in turn,
// one's products beside the other's exponentials, spill (43 ms; heads of 64 207 us
// against 150); bounds of a mask as constants gain nothing (22.8).
#include "ua2a_attn_device.h"

namespace ua2a {
namespace {

// The keys and values of a tile of a cache on their way to LDS: CH chunks of
// eight codes per lane of each, decoded when they are stored.
template <class T, int DP, int KEYS>
struct CodeLoads {
    static constexpr int kAcross = DP / 8;                       // chunks of a row
    static constexpr int CH = KEYS * kAcross / static_cast<int>(kAttnBlock);
    u32x2v k[CH], v[CH];
    uint32_t ks[CH], vs[CH];

    __device__ __forceinline__ static uint32_t row(int c) { return (threadIdx.x + c * kAttnBlock) / kAcross; }
    __device__ __forceinline__ static uint32_t chunk(int c) { return (threadIdx.x + c * kAttnBlock) % kAcross; }

    // j0: the tile's first position of this key head, in heads of D codes.  What
    // lies at or past `rows` positions, or past D, is zeros.
    __device__ __forceinline__ void load(const AttnArgs& a, int64_t j0, int32_t rows)
    {
        const AttnGeom& g = a.g;
        const uint32_t step = g.kvl * g.D, sstep = g.kvl * g.nb;
        const uint32_t bytes = static_cast<uint32_t>(rows) * step, sbytes = static_cast<uint32_t>(rows) * sstep;
        const auto kd = resource(a.codes + j0 * g.D, bytes), vd = resource(a.codes + a.part + j0 * g.D, bytes);
        const auto ksd = resource(a.scales + j0 * g.nb, sbytes), vsd = resource(a.scales + a.part_scales + j0 * g.nb, sbytes);
#pragma unroll
        for (int c = 0; c < CH; ++c) {
            const uint32_t d = chunk(c) * 8;
            const bool ok = d < g.D;
            const uint32_t at = ok ? row(c) * step + d : kNowhere, sat = ok ? row(c) * sstep + d / kBlockValues : kNowhere;
            k[c] = __builtin_bit_cast(u32x2v, __builtin_amdgcn_raw_buffer_load_b64(kd, at, 0, 0));
            v[c] = __builtin_bit_cast(u32x2v, __builtin_amdgcn_raw_buffer_load_b64(vd, at, 0, 0));
            ks[c] = __builtin_amdgcn_raw_buffer_load_b8(ksd, sat, 0, 0);
            vs[c] = __builtin_amdgcn_raw_buffer_load_b8(vsd, sat, 0, 0);
        }
    }
    template <bool E4M3>
    __device__ __forceinline__ void put(char* ktile, char* vtile) const
    {
#pragma unroll
        for (int c = 0; c < CH; ++c) {
            const uint32_t at = place_of<DP>(row(c), chunk(c) * 16);
            *reinterpret_cast<u32x4v*>(ktile + at) = decode8<T, E4M3>(k[c], ks[c]);
            *reinterpret_cast<u32x4v*>(vtile + at) = decode8<T, E4M3>(v[c], vs[c]);
        }
    }
    // Returns the largest scale byte.
    __device__ __forceinline__ uint32_t store(char* ktile, char* vtile, int32_t format) const
    {
        if (format == UA2A_FORMAT_E4M3)
            put<true>(ktile, vtile);
        else
            put<false>(ktile, vtile);
        uint32_t top = 0;
#pragma unroll
        for (int c = 0; c < CH; ++c) top = max(top, max(ks[c], vs[c]));
        return top;
    }
};

// The running softmax of a wave's 32 rows and their sums over the values.
template <class T, int DP>
struct Rows {
    f32x16v o[DP / 32];
    float m;                     // the weights' base, times log2(e); -inf until the row has seen a key
    float l;                     // of this half's keys
    bool far;                    // uniform: some row's base is (far_base)

    __device__ __forceinline__ void clear()
    {
#pragma unroll
        for (int db = 0; db < DP / 32; ++db)
#pragma unroll
            for (int i = 0; i < 16; ++i) o[db][i] = 0.f;
        m = -__builtin_inff();
        l = 0.f;
        far = false;
    }
};

// One tile of 32 * NK keys for a wave: scores, softmax, sums.  k0: position of
// the tile's row `row0`.  masked: some row does not see some key.  odd: the
// tile's values had infinities or NaN, which a row must take only of keys it
// sees (zero times them is NaN): zeros are in their places, and `wild` says
// where they were.
//
// The base lags (kLift, kAhead), which costs no precision.  The weights are rounded to
// the type for the product (relative half a step of it, as its operands are), their sum
// is not.
template <class T, int DP, int NK>
__device__ __forceinline__ void attend(Rows<T, DP>& r, const u32x4v (&q)[DP / 16], const char* ktile, const char* vtile,
                                       const uint8_t* wild, uint32_t row0, uint32_t k0, const Seen& seen, float scale2,
                                       bool masked, bool odd)
{
    const uint32_t half = (threadIdx.x & 63) >> 5;
    f32x16v s[NK];
    __builtin_amdgcn_s_setprio(1);
#pragma unroll
    for (int b = 0; b < NK; ++b) {
#pragma unroll
        for (int i = 0; i < 16; ++i) s[b][i] = 0.f;
#pragma unroll
        for (int ks = 0; ks < DP / 16; ++ks)
            s[b] = mfma<T>(along<DP>(ktile, row0 + b * 32, ks), q[ks], s[b]);
    }
    __builtin_amdgcn_s_setprio(0);
    const auto key = [&](int b, int i) {
        return k0 + (b * 32 + (i / 4) * 8 + half * 4 + i % 4);
    };
    if (masked) {
#pragma unroll
        for (int b = 0; b < NK; ++b)
#pragma unroll
            for (int i = 0; i < 16; ++i)
                if (!sees(seen, key(b, i))) s[b][i] = -__builtin_inff();
    }
    float top = -__builtin_inff();
#pragma unroll
    for (int b = 0; b < NK; ++b)
#pragma unroll
        for (int i = 0; i < 16; ++i) top = fmaxf(top, s[b][i]);
    top = max_halves(top) * scale2;
    const bool grow = ahead_of<T>(top, r.m);
    if (__builtin_amdgcn_ballot_w64(grow) != 0) {
        const float next = fmaxf(r.m, base_of<T>(top));
        const float f = next == r.m ? 1.f : __builtin_amdgcn_exp2f(r.m - next);
        r.m = next;
        r.far = __builtin_amdgcn_ballot_w64(far_base(next)) != 0;
        r.l *= f;
#pragma unroll
        for (int db = 0; db < DP / 32; ++db)
#pragma unroll
            for (int i = 0; i < 16; ++i) r.o[db][i] *= f;
    }
    const float m = r.m == -__builtin_inff() ? 0.f : r.m;
    float times = scale2, plus = -m;
    if (r.far) {
#pragma unroll
        for (int b = 0; b < NK; ++b)
#pragma unroll
            for (int i = 0; i < 16; ++i) s[b][i] = far_exponent(s[b][i], scale2, m);
        times = 1.f;
        plus = 0.f;
    }
    float sum = 0.f;
#pragma unroll
    for (int b = 0; b < NK; ++b)
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            s[b][i] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[b][i], times, plus));
            sum += s[b][i];
        }
    r.l += sum;
    u32x4v p[2 * NK];
#pragma unroll
    for (int b = 0; b < NK; ++b)
#pragma unroll
        for (int t = 0; t < 2; ++t) p[2 * b + t] = operand_of<T>(s[b], t);
    __builtin_amdgcn_s_setprio(1);
#pragma unroll
    for (int db = 0; db < DP / 32; ++db)
#pragma unroll
        for (int t = 0; t < 2 * NK; ++t) r.o[db] = mfma<T>(transposed<DP>(vtile, row0, t, db), p[t], r.o[db]);
    __builtin_amdgcn_s_setprio(0);
    if (!odd) return;
    // the tile's infinities and NaN: of the keys that the row sees, one bit per value
    uint32_t up[DP / 32], down[DP / 32];
#pragma unroll
    for (int db = 0; db < DP / 32; ++db) up[db] = down[db] = 0;
#pragma unroll 1
    for (uint32_t j = 0; j < 32 * NK; ++j) {
        const bool see = sees(seen, k0 + j);
#pragma unroll
        for (int db = 0; db < DP / 32; ++db) {
            const uint32_t* bits = reinterpret_cast<const uint32_t*>(wild + (row0 + j) * (DP / 4)) + db;
            up[db] |= see ? bits[0] : 0u;
            down[db] |= see ? bits[DP / 32] : 0u;
        }
    }
#pragma unroll
    for (int db = 0; db < DP / 32; ++db)
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            const uint32_t bit = (i / 4) * 8 + half * 4 + i % 4;
            if (up[db] >> bit & 1) r.o[db][i] += __builtin_inff();
            if (down[db] >> bit & 1) r.o[db][i] -= __builtin_inff();
        }
}

// SHARED false: each wave has 32 rows of the workgroup's 128, and all walk tiles
// of 64 keys.  SHARED true (at most 32 rows, of a cache 17 at least): the waves have the
// same rows and a quarter of each tile of 128 keys, and their sums are joined in
// LDS.
template <class T, int DP, bool CODES, bool SHARED>
__global__ __launch_bounds__(kAttnBlock, 2) void ua2a_attention_kernel(AttnArgs a)
{
    constexpr int KEYS = SHARED ? kAttnSplitKeys : kAttnKeys;
    constexpr int NK = SHARED ? 1 : KEYS / 32;
    constexpr uint32_t kTile = KEYS * kRow<DP>;
    // two buffers of keys and values where loads go straight to LDS; a wave's
    // sums (SHARED) take the place of one
    constexpr uint32_t kBuffers = CODES || SHARED ? 1 : 2;
    __shared__ __attribute__((aligned(1024))) char lds[kBuffers * 2 * kTile];
    __shared__ __attribute__((aligned(16))) uint8_t wild[KEYS * (DP / 4)];
    __shared__ uint32_t odd_tile, high_tile;
    __shared__ float stat[SHARED ? 5 * 32 * 2 : 1];            // the waves', then joined
    const AttnGeom& g = a.g;
    const uint32_t item = attn_item(g, (blockIdx.y << kAttnGridLog) + blockIdx.x);
    if (item >= g.items) return;
    const AttnPlace at = attn_place(g, item);
    const uint32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
    const uint32_t half = lane >> 5, col = lane & 31;
    const AttnSeq seq = attn_seq(g, a.starts != nullptr ? static_cast<int64_t>(a.starts[at.i]) : 0,
                                 a.counts != nullptr ? static_cast<int64_t>(a.counts[at.i]) : static_cast<int64_t>(g.n));
    const uint32_t first = at.tile * (SHARED ? kAttnWaveRows : kAttnRows);
    const uint32_t past = umin32(first + (SHARED ? kAttnWaveRows : kAttnRows), g.rows);
    const uint32_t wfirst = SHARED ? first : first + wave * kAttnWaveRows;
    const uint32_t row = wfirst + col;
    const bool in = row < past;
    const RowPlace place = row_place(g, at, in ? row : past - 1);
    const bool live = in && place.t >= seq.first && place.t < seq.last;

    Rows<T, DP> r;
    r.clear();
    // no query of the tile exists: nothing to walk
    const bool some = static_cast<int32_t>(fdiv(first, g.d_group)) < seq.last &&
                      static_cast<int32_t>(fdiv(past - 1, g.d_group)) >= seq.first;
    if (some) {
        const Seen top = seen_by_row(g, seq, first), bottom = seen_by_row(g, seq, past - 1);
        const KeyWalk walk = key_walk(top, bottom, KEYS);
        const uint32_t from = split_at(walk.total, g.splits, at.split), to = split_at(walk.total, g.splits, at.split + 1);
        const uint32_t wlast = umin32(wfirst + kAttnWaveRows, past) - 1;
        const bool rows = wfirst < past;                         // of the wave
        const Seen wtop = rows ? seen_by_row(g, seq, wfirst) : bottom, wbottom = rows ? seen_by_row(g, seq, wlast) : bottom;
        const Seen seen = seen_by_row(g, seq, place.row);
        u32x4v q[DP / 16];
        row_operands<DP>(static_cast<const uint16_t*>(a.q) + place.at, g.D, half, live, q);

        const int64_t base = static_cast<int64_t>(at.seq) * g.keys * g.kvl + at.kvh;
        if (threadIdx.x == 0) odd_tile = high_tile = ~0u;
        const auto position = [&](uint32_t i) { return walk_tile(walk, i) * KEYS; };
        // the keys of the tile from k0 on that exist
        const auto keys_of = [&](uint32_t k0) {
            const int32_t n = seq.end - static_cast<int32_t>(k0);
            return n < KEYS ? n : KEYS;
        };
        // whether some row of the workgroup does not see some key of tile i
        const auto part_seen = [&](uint32_t k0) { return !all_seen(top, bottom, k0, k0 + KEYS); };
        const auto work = [&](uint32_t i, uint32_t k0, const char* ktile, const char* vtile, bool look) {
            const uint32_t row0 = SHARED ? wave * 32 : 0;
            const uint32_t wk0 = k0 + row0;
            if (!rows || none_seen(wtop, wbottom, wk0, wk0 + 32 * NK)) return;
            attend<T, DP, NK>(r, q, ktile, vtile, wild, row0, wk0, seen, a.scale2,
                              !all_seen(wtop, wbottom, wk0, wk0 + 32 * NK), look && odd_tile == i);
        };
        if constexpr (CODES) {
            CodeLoads<T, DP, KEYS> loads;
            const auto load = [&](uint32_t i) {
                const uint32_t k0 = position(i);
                loads.load(a, base + static_cast<int64_t>(k0) * g.kvl, keys_of(k0));
            };
            if (from < to) load(from);
            for (uint32_t i = from; i < to; ++i) {
                const uint32_t k0 = position(i);
                const bool look = part_seen(k0);
                __syncthreads();                                 // the last tile has been read
                if (loads.store(lds, lds + kTile, a.format) >= high_scale<T>(a.format)) high_tile = i;
                if (i + 1 < to) load(i + 1);
                __syncthreads();
                if (high_tile == i) {
                    const int64_t j0 = base + static_cast<int64_t>(k0) * g.kvl;
                    const int32_t n = keys_of(k0);
                    const uint8_t *codes = a.codes + j0 * g.D, *scales = a.scales + j0 * g.nb;
                    decode_again<T, DP>(lds, g, codes, scales, n, a.format, threadIdx.x, kAttnBlock);
                    decode_again<T, DP>(lds + kTile, g, codes + a.part, scales + a.part_scales, n, a.format, threadIdx.x,
                                        kAttnBlock);
                    __syncthreads();
                }
                if (look) {
                    if (tame_tile<T, DP>(lds + kTile, wild, KEYS, threadIdx.x, kAttnBlock)) odd_tile = i;
                    __syncthreads();
                }
                work(i, k0, lds, lds + kTile, look);
            }
        } else {
            typedef TileLoads<DP, KEYS> Loads;
            uint32_t offset[Loads::N];
            const uint32_t row_bytes = g.kvl * g.D * 2;
#pragma unroll
            for (int n = 0; n < Loads::N; ++n) {
                const uint32_t bytes = Loads::bytes(n, wave, g.D);
                offset[n] = bytes == kNowhere ? kNowhere : Loads::row(n, wave) * row_bytes + bytes;
            }
            const auto load = [&](uint32_t i, char* tile) {
                const uint32_t k0 = position(i);
                const int64_t start = (base + static_cast<int64_t>(k0) * g.kvl) * g.D * 2;
                const uint32_t bytes = static_cast<uint32_t>(keys_of(k0)) * row_bytes;
                const u32x4v k = descriptor(static_cast<const char*>(a.k) + start, bytes),
                             v = descriptor(static_cast<const char*>(a.v) + start, bytes);
#pragma unroll
                for (int n = 0; n < Loads::N; ++n) {
                    if (!Loads::has(n, wave)) continue;
                    char* const to_lds = tile + (n * 4 + wave) * 1024;
                    load_to_lds(k, offset[n], to_lds);
                    load_to_lds(v, offset[n], to_lds + kTile);
                }
            };
            char* tile = lds;
            char* other = lds + (kBuffers - 1) * 2 * kTile;
            if (from < to && kBuffers == 2) load(from, tile);
            for (uint32_t i = from; i < to; ++i) {
                const uint32_t k0 = position(i);
                const bool look = part_seen(k0);
                if constexpr (kBuffers == 1) {
                    __syncthreads();                             // the last tile has been read
                    load(i, tile);
                }
                arrived();
                if (kBuffers == 2 && i + 1 < to) load(i + 1, other);
                if (look) {
                    if (tame_tile<T, DP>(tile + kTile, wild, KEYS, threadIdx.x, kAttnBlock)) odd_tile = i;
                    __syncthreads();
                }
                work(i, k0, tile, tile + kTile, look);
                if constexpr (kBuffers == 2) {
                    char* const t = tile;
                    tile = other;
                    other = t;
                }
            }
        }
    }
    __syncthreads();
    r.l = add_halves(r.l);
    if constexpr (SHARED) {
        // the four waves' maxima and sums, then their values' sums, 32 rows of DP each
        if (half == 0) {
            stat[(wave * 32 + col) * 2] = r.m;
            stat[(wave * 32 + col) * 2 + 1] = r.l;
        }
        __syncthreads();
        float m = -__builtin_inff(), l = 0.f;
#pragma unroll
        for (int w = 0; w < 4; ++w) m = fmaxf(m, stat[(w * 32 + col) * 2]);
        const float mm = m == -__builtin_inff() ? 0.f : m;
#pragma unroll
        for (int w = 0; w < 4; ++w)
            l += stat[(w * 32 + col) * 2 + 1] * __builtin_amdgcn_exp2f(stat[(w * 32 + col) * 2] - mm);
        const float f = __builtin_amdgcn_exp2f(r.m - mm);
        float* sums = reinterpret_cast<float*>(lds);             // [wave][row][DP]: no more than the tiles take
#pragma unroll
        for (int db = 0; db < DP / 32; ++db)
#pragma unroll
            for (int b = 0; b < 4; ++b) {
                f32x4v x;
#pragma unroll
                for (int i = 0; i < 4; ++i) x[i] = r.o[db][4 * b + i] * f;
                *reinterpret_cast<f32x4v*>(sums + (wave * 32 + col) * DP + db * 32 + b * 8 + half * 4) = x;
            }
        if (half == 0 && wave == 0) {
            stat[(128 + col) * 2] = m;
            stat[(128 + col) * 2 + 1] = l;
        }
        __syncthreads();
        for (uint32_t i = threadIdx.x; i < 32 * (DP / 4); i += kAttnBlock) {
            const uint32_t c = i / (DP / 4), d = i % (DP / 4) * 4;
            if (first + c >= past || d >= g.D) continue;
            f32x4v x = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int w = 0; w < 4; ++w) x += *reinterpret_cast<const f32x4v*>(sums + (w * 32 + c) * DP + d);
            finish_row<T>(a, at, seq, first + c, d, x, stat[(128 + c) * 2], stat[(128 + c) * 2 + 1]);
        }
        return;
    }
    if (!in) return;
    if (g.splits > 1) {
        const int64_t line = static_cast<int64_t>(at.split) * g.units * g.rows + static_cast<int64_t>(at.unit) * g.rows + row;
#pragma unroll
        for (int db = 0; db < DP / 32; ++db)
#pragma unroll
            for (int b = 0; b < 4; ++b) {
                const uint32_t d = db * 32 + b * 8 + half * 4;
                if (d < g.D)
                    *reinterpret_cast<f32x4v*>(a.partial + line * g.D + d) =
                        f32x4v{r.o[db][4 * b], r.o[db][4 * b + 1], r.o[db][4 * b + 2], r.o[db][4 * b + 3]};
            }
        if (half == 0) {
            a.stats[line * 2] = live ? r.m : -__builtin_inff();
            a.stats[line * 2 + 1] = live ? r.l : 0.f;
        }
        return;
    }
    if (!live && a.keep) return;
    float inv = live && r.l != 0.f ? 1.f / r.l : 0.f, top = 0.f;
#pragma unroll
    for (int db = 0; db < DP / 32; ++db)
#pragma unroll
        for (int i = 0; i < 16; ++i) top = fmaxf(top, fabsf(r.o[db][i]));
    // rare, so one look at the largest (`within` on each: 66 tokens of 4 heads of 80 8.6 us, 8.2)
    if (top * inv > kMost<T>) {
#pragma unroll
        for (int db = 0; db < DP / 32; ++db)
#pragma unroll
            for (int i = 0; i < 16; ++i) r.o[db][i] = within<T>(r.o[db][i] * inv);
        inv = 1.f;
    }
#pragma unroll
    for (int db = 0; db < DP / 32; ++db)
#pragma unroll
        for (int b = 0; b < 4; ++b) {
            const uint32_t d = db * 32 + b * 8 + half * 4;
            u32x2v y = {0, 0};
            if (live)
                y = u32x2v{pack2<T>(r.o[db][4 * b] * inv, r.o[db][4 * b + 1] * inv),
                           pack2<T>(r.o[db][4 * b + 2] * inv, r.o[db][4 * b + 3] * inv)};
            if (d < g.D) *reinterpret_cast<u32x2v*>(static_cast<uint16_t*>(a.out) + place.at + d) = y;
        }
    if (half == 0 && a.lse != nullptr)
        a.lse[place.stat] = live ? lse_of<T>(r.m, r.l) : -__builtin_inff();
}

// The parts of rows whose keys were walked by several workgroups, joined.  A group
// of D / 4 lanes has four values each of eight parts, whose loads are on their way
// together; more parts take more groups, up to a workgroup (64 parts of 16 rows:
// 23 us with two parts at once, 6.5 with 64; 3 parts of 18,720 rows: 20 us with a
// group for each part).
template <class T>
__global__ __launch_bounds__(kAttnBlock) void ua2a_attention_join_kernel(AttnArgs a)
{
    __shared__ f32x4v sums[kAttnBlock];
    __shared__ float tops[kAttnBlock], totals[kAttnBlock];
    const AttnGeom& g = a.g;
    const uint32_t count = g.units * g.rows;                     // < 2^31
    const int64_t lines = count;
    const JoinShape js = join_shape(g);
    const uint32_t d = (threadIdx.x & (js.wide - 1)) * 4, group = threadIdx.x / js.wide, mine = group & (js.at_once - 1);
    const uint32_t line = ((blockIdx.y << kAttnGridLog) + blockIdx.x) * js.rows + group / js.at_once;
    const bool in = line < count;
    AttnPlace at;
    at.unit = in ? fdiv(line, g.d_rows) : 0;
    at.seq = fdiv(at.unit, g.d_kvl);
    at.kvh = at.unit - at.seq * g.kvl;
    at.i = at.seq - fdiv(at.seq, g.d_seqs) * g.seqs;
    const RowPlace pl = row_place(g, at, in ? line - at.unit * g.rows : 0);
    const AttnSeq seq = attn_seq(g, a.starts != nullptr ? static_cast<int64_t>(a.starts[at.i]) : 0,
                                 a.counts != nullptr ? static_cast<int64_t>(a.counts[at.i]) : static_cast<int64_t>(g.n));
    const bool live = in && pl.t >= seq.first && pl.t < seq.last;
    float m = -__builtin_inff(), l = 0.f;
    f32x4v x = {0.f, 0.f, 0.f, 0.f};
    constexpr int kEach = kJoinEach;
    for (uint32_t s0 = mine; live && s0 < g.splits; s0 += js.at_once * kEach) {
        float sm[kEach], sl[kEach];
        f32x4v sx[kEach];
#pragma unroll
        for (int b = 0; b < kEach; ++b) {
            const uint32_t s = s0 + b * js.at_once;
            sm[b] = -__builtin_inff();
            sl[b] = 0.f;
            sx[b] = f32x4v{0.f, 0.f, 0.f, 0.f};
            if (s >= g.splits) continue;
            sm[b] = a.stats[(s * lines + line) * 2];
            sl[b] = a.stats[(s * lines + line) * 2 + 1];
            if (d < g.D) sx[b] = *reinterpret_cast<const f32x4v*>(a.partial + (s * lines + line) * g.D + d);
        }
        float now = m;
#pragma unroll
        for (int b = 0; b < kEach; ++b) now = fmaxf(now, sm[b]);
        const float mm = now == -__builtin_inff() ? 0.f : now;
        const float f = __builtin_amdgcn_exp2f(m - mm);
        l *= f;
        x *= f;
#pragma unroll
        for (int b = 0; b < kEach; ++b) {
            const float w = __builtin_amdgcn_exp2f(sm[b] - mm);
            l += sl[b] * w;
            x += sx[b] * w;
        }
        m = now;
    }
    sums[threadIdx.x] = x;
    tops[threadIdx.x] = m;
    totals[threadIdx.x] = l;
    __syncthreads();
    if (mine != 0 || d >= g.D || !in || (!live && a.keep)) return;
    for (uint32_t b = 0; b < js.at_once; ++b) m = fmaxf(m, tops[threadIdx.x + b * js.wide]);
    const float mm = m == -__builtin_inff() ? 0.f : m;
    x = f32x4v{0.f, 0.f, 0.f, 0.f};
    l = 0.f;
    for (uint32_t b = 0; b < js.at_once; ++b) {
        const float w = __builtin_amdgcn_exp2f(tops[threadIdx.x + b * js.wide] - mm);
        l += totals[threadIdx.x + b * js.wide] * w;
        x += sums[threadIdx.x + b * js.wide] * w;
    }
    const float inv = l != 0.f ? 1.f / l : 0.f;
    u32x2v y = {0, 0};
    if (live)
        y = u32x2v{pack2<T>(within<T>(x[0] * inv), within<T>(x[1] * inv)), pack2<T>(within<T>(x[2] * inv), within<T>(x[3] * inv))};
    *reinterpret_cast<u32x2v*>(static_cast<uint16_t*>(a.out) + pl.at + d) = y;
    if (d == 0 && a.lse != nullptr) a.lse[pl.stat] = live ? lse_of<T>(m, l) : -__builtin_inff();
}

template <class T, int DP>
const void* sized_fn(const AttnLaunch& L)
{
    const bool codes = L.attn.codes != nullptr;
    if (codes)
        return L.shared ? reinterpret_cast<const void*>(&ua2a_attention_kernel<T, DP, true, true>)
                        : reinterpret_cast<const void*>(&ua2a_attention_kernel<T, DP, true, false>);
    return L.shared ? reinterpret_cast<const void*>(&ua2a_attention_kernel<T, DP, false, true>)
                    : reinterpret_cast<const void*>(&ua2a_attention_kernel<T, DP, false, false>);
}

template <class T>
const void* typed_fn(const AttnLaunch& L)
{
    if (L.kernel == AttnKernel::Join) return reinterpret_cast<const void*>(&ua2a_attention_join_kernel<T>);
    switch (L.DP) {
    case 32: return sized_fn<T, 32>(L);
    case 64: return sized_fn<T, 64>(L);
    case 96: return sized_fn<T, 96>(L);
    case 128: return sized_fn<T, 128>(L);
    }
    return nullptr;
}

}  // namespace

const void* attention_kernel(const AttnLaunch& L)
{
    return L.type == UA2A_TYPE_BF16 ? typed_fn<__bf16>(L) : typed_fn<_Float16>(L);
}

}  // namespace ua2a
