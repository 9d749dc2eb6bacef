// gfx950 kernels of windowed attention's backward pass (ua2a_attn.h).
//
// With P = exp(scale s - lse), delta = sum(dout * out) of a row and
// dS = P * (dout v^T - delta):
//   dq = scale dS k,  dk = scale dS^T q,  dv = P^T dout.
// The first two products (s and dout v^T) are made twice, once where rows keep
// their sums (dq) and once where keys keep theirs (dk, dv): seven products
// instead of five (and an eighth, for dS's second part), and in return no atomics,
// so equal inputs give equal bits.
//
// The matrix products and what stands between them bound the first kernel, waiting the
// second: 12 heads of 128 over 32,760 tokens, a window of three frames of 1560 and the
// first, take 2.1 ms and 3.1 (matrix units busy 60 % and 39 % of the time, waves waiting
// 33 % and 59 %); the eight products alone would be 4.0 ms at a large matrix product's
// rate.  Some of the waiting is for operands in LDS, some for memory in every tile: the
// next tile's lse and delta pass through registers, whose wait takes the tile's loads with
// it, and both kernels wait for the next tile where they first use operands that were
// loaded before the loop (see TileLoads).
#include "ua2a_attn_device.h"

namespace ua2a {
namespace {

__device__ __forceinline__ float dot2_sum(u32x4v a, u32x4v b, float sum, __bf16)
{
#pragma unroll
    for (int i = 0; i < 4; ++i)
        sum = __builtin_amdgcn_fdot2_f32_bf16(pair_of<__bf16>(a[i]), pair_of<__bf16>(b[i]), sum, false);
    return sum;
}
__device__ __forceinline__ float dot2_sum(u32x4v a, u32x4v b, float sum, _Float16)
{
#pragma unroll
    for (int i = 0; i < 4; ++i) sum = __builtin_amdgcn_fdot2(pair_of<_Float16>(a[i]), pair_of<_Float16>(b[i]), sum, false);
    return sum;
}

// lse times log2(e), such that a row without weight (-inf) gets none.
__device__ __forceinline__ float lse2_of(float lse)
{
    return lse == -__builtin_inff() ? __builtin_inff() : lse * kLog2e;
}

template <int N>
__device__ __forceinline__ void zero(f32x16v (&x)[N])
{
#pragma unroll
    for (int b = 0; b < N; ++b)
#pragma unroll
        for (int i = 0; i < 16; ++i) x[b][i] = 0.f;
}

// A lane's column of a transposed sum, times `factor`, as a row of values.
template <class T, int DP>
__device__ __forceinline__ void store_row(void* out, int64_t at, uint32_t D, const f32x16v (&x)[DP / 32], float factor,
                                          bool live)
{
    const uint32_t half = (threadIdx.x & 63) >> 5;
#pragma unroll
    for (int db = 0; db < DP / 32; ++db)
#pragma unroll
        for (int b = 0; b < 4; ++b) {
            const uint32_t d = db * 32 + b * 8 + half * 4;
            u32x2v y = {0, 0};
            if (live)
                y = u32x2v{pack2<T>(x[db][4 * b] * factor, x[db][4 * b + 1] * factor),
                           pack2<T>(x[db][4 * b + 2] * factor, x[db][4 * b + 3] * factor)};
            if (d < D) *reinterpret_cast<u32x2v*>(static_cast<uint16_t*>(out) + at + d) = y;
        }
}

// The largest of a value over a wave's lanes.
__device__ __forceinline__ float max_wave(float x)
{
#pragma unroll
    for (int by = 1; by < 64; by *= 2) x = fmaxf(x, __shfl_xor(x, by));
    return x;
}

// The exponent of a value that is not below zero: 2^e <= x < 2^(e + 1); 128 of infinity.
__device__ __forceinline__ int32_t exponent_of(float x) { return static_cast<int32_t>(__float_as_uint(x) >> 23) - 127; }

__device__ __forceinline__ int32_t clamped(int32_t x, int32_t lo, int32_t hi) { return x < lo ? lo : x < hi ? x : hi; }

__device__ __forceinline__ float power_of_two(int32_t e) { return __uint_as_float(static_cast<uint32_t>(e + 127) << 23); }

// dq, and delta for the other kernel.  As forward, a wave has 32 rows as columns
// of its matrix tiles and walks tiles of 64 keys: scores and dout v^T come as
// keys x rows, dS goes on to its product with k from the registers it is in.  A
// row's dS add up to zero, so what rounding leaves of them weighs more than in the
// other sums; dS goes in as two values of the type (an error of dq of 1.45 times
// its own rounding's falls to 1.0 times; three products become four, 1.69 ms 2.13).
//
// In fp16 a row's dS go in times 2^lift, which comes out of its sums in 32 bits: with many
// keys P alone is among fp16's subnormals, where the second part has nothing left to say
// (24,576 keys, dout of 1e-3: 20 times its own rounding's).  The lift puts |dout| at 2^8, and
// a dS then is about 2^8 P |v|'s share of it.  Where one passes the type all the same (values
// in the hundreds), the workgroup walks its keys once more with that row's lift 14 lower,
// at which none can: |dS| <= P |dout| (|v| + |out|) < 2^9 * 2^20.5 with heads of 128.
template <class T, int DP>
__global__ __launch_bounds__(kAttnBlock, 2) void ua2a_attention_rows_kernel(AttnGradArgs a)
{
    constexpr int KEYS = kAttnKeys, NK = KEYS / 32;
    constexpr uint32_t kTile = KEYS * kRow<DP>;
    constexpr bool kLifted = !__is_same(T, __bf16);
    __shared__ __attribute__((aligned(1024))) char lds[4 * kTile];           // two buffers of keys and values
    __shared__ float sizes[kLifted ? 4 : 1][2];                              // the waves' largest |dout| and |delta|
    __shared__ uint32_t passed;                                              // a dS passed the type
    const AttnGeom& g = a.g;
    const uint32_t item = attn_item(g, (blockIdx.y << kAttnGridLog) + blockIdx.x);
    if (item >= g.items) return;
    const AttnPlace at = attn_place(g, item);
    const uint32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
    const uint32_t half = lane >> 5, col = lane & 31;
    const AttnSeq seq = attn_seq(g, 0, a.counts != nullptr ? static_cast<int64_t>(a.counts[at.i]) : static_cast<int64_t>(g.n));
    const uint32_t first = at.tile * kAttnRows, past = umin32(first + kAttnRows, g.rows);
    const uint32_t wfirst = first + wave * kAttnWaveRows, row = wfirst + col;
    const bool in = row < past, rows = wfirst < past;
    const RowPlace place = row_place(g, at, in ? row : past - 1);
    const bool live = in && place.t < seq.last;
    f32x16v dq[DP / 32];
    zero(dq);
    if (static_cast<int32_t>(fdiv(first, g.d_group)) < seq.last) {
        const Seen top = seen_by_row(g, seq, first), bottom = seen_by_row(g, seq, past - 1);
        const KeyWalk walk = key_walk(top, bottom, KEYS);
        const uint32_t wlast = umin32(wfirst + kAttnWaveRows, past) - 1;
        const Seen wtop = rows ? seen_by_row(g, seq, wfirst) : bottom, wbottom = rows ? seen_by_row(g, seq, wlast) : bottom;
        const Seen seen = seen_by_row(g, seq, place.row);
        u32x4v q[DP / 16], go[DP / 16];
        float delta = 0.f;
        {
            u32x4v o[DP / 16];
            row_operands<DP>(static_cast<const uint16_t*>(a.dout) + place.at, g.D, half, live, go);
            row_operands<DP>(static_cast<const uint16_t*>(a.out) + place.at, g.D, half, live, o);
#pragma unroll
            for (int ks = 0; ks < DP / 16; ++ks) delta = dot2_sum(go[ks], o[ks], delta, T{});
            delta = add_halves(delta);
        }
        if (live && half == 0) a.delta[static_cast<int64_t>(at.unit) * g.rows + row] = delta;
        row_operands<DP>(static_cast<const uint16_t*>(a.q) + place.at, g.D, half, live, q);
        float lse2 = live ? lse2_of(a.lse[place.stat]) : __builtin_inff();
        int32_t lift = 0;
        if constexpr (kLifted) {
            float norm = 0.f;                                    // |dout|^2
#pragma unroll
            for (int ks = 0; ks < DP / 16; ++ks) norm = dot2_sum(go[ks], go[ks], norm, T{});
            norm = add_halves(norm);
            lift = clamped(8 - (exponent_of(norm) >> 1), -16, 32);
            lse2 -= static_cast<float>(lift);
            const float most = max_wave(norm), far = max_wave(fabsf(delta));
            if (lane == 0) {
                sizes[wave][0] = most;
                sizes[wave][1] = far;
            }
            if (threadIdx.x == 0) passed = 0;
        }
        const int64_t base = static_cast<int64_t>(at.seq) * g.keys * g.kvl + at.kvh;
        typedef TileLoads<DP, KEYS> Loads;
        uint32_t offset[Loads::N];
        const uint32_t row_bytes = g.kvl * g.D * 2;
#pragma unroll
        for (int n = 0; n < Loads::N; ++n) {
            const uint32_t bytes = Loads::bytes(n, wave, g.D);
            offset[n] = bytes == kNowhere ? kNowhere : Loads::row(n, wave) * row_bytes + bytes;
        }
        const auto position = [&](uint32_t i) { return walk_tile(walk, i) * KEYS; };
        const auto load = [&](uint32_t i, char* tile) {
            const uint32_t k0 = position(i);
            const int64_t start = (base + static_cast<int64_t>(k0) * g.kvl) * g.D * 2;
            const int32_t left = seq.end - static_cast<int32_t>(k0);
            const uint32_t bytes = static_cast<uint32_t>(left < KEYS ? left : KEYS) * row_bytes;
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
        char *ktile = lds, *other = lds + 2 * kTile;
        const auto walk_keys = [&]() {
            load(0, ktile);
            for (uint32_t i = 0; i < walk.total; ++i) {
                const uint32_t k0 = position(i);
                char* const vtile = ktile + kTile;
                arrived();
                if (i + 1 < walk.total) load(i + 1, other);
#pragma unroll
                for (int b = 0; b < NK; ++b) {
                    const uint32_t bk0 = k0 + b * 32;
                    if (!rows || none_seen(wtop, wbottom, bk0, bk0 + 32)) continue;
                    const bool masked = !all_seen(wtop, wbottom, bk0, bk0 + 32);
                    f32x16v s, dp;
#pragma unroll
                    for (int x = 0; x < 16; ++x) {
                        s[x] = 0.f;
                        dp[x] = -delta;
                    }
#pragma unroll
                    for (int ks = 0; ks < DP / 16; ++ks) s = mfma<T>(along<DP>(ktile, b * 32, ks), q[ks], s);
#pragma unroll
                    for (int ks = 0; ks < DP / 16; ++ks) dp = mfma<T>(along<DP>(vtile, b * 32, ks), go[ks], dp);
#pragma unroll
                    for (int x = 0; x < 16; ++x) dp[x] *= __builtin_amdgcn_exp2f(__builtin_fmaf(s[x], a.scale2, -lse2));
                    if (masked) {
#pragma unroll
                        for (int x = 0; x < 16; ++x)
                            if (!sees(seen, bk0 + ((x / 4) * 8 + half * 4 + x % 4))) dp[x] = 0.f;
                    }
                    const u32x4v ds[2] = {operand_of<T>(dp, 0), operand_of<T>(dp, 1)};
                    const u32x4v rest[2] = {rest_of<T>(dp, ds[0], 0), rest_of<T>(dp, ds[1], 1)};
#pragma unroll
                    for (int db = 0; db < DP / 32; ++db)
#pragma unroll
                        for (int t = 0; t < 2; ++t) {
                            const u32x4v k = transposed<DP>(ktile, b * 32, t, db);
                            dq[db] = mfma<T>(k, ds[t], dq[db]);
                            dq[db] = mfma<T>(k, rest[t], dq[db]);
                        }
                }
                char* const t = ktile;
                ktile = other;
                other = t;
            }
        };
        walk_keys();
        if constexpr (kLifted) {
            // an infinite dS leaves no finite value in its row: infinity times zero is NaN
            const bool past_range = live && !(fabsf(dq[0][0]) < __builtin_inff());
            if (past_range) passed = 1;
            if (threadIdx.x == 0) {
                float most = 0.f, far = 0.f;
#pragma unroll
                for (int w = 0; w < 4; ++w) {
                    most = fmaxf(most, sizes[w][0]);
                    far = fmaxf(far, sizes[w][1]);
                }
                float* const to = a.sizes + (static_cast<int64_t>(at.unit) * g.tiles + at.tile) * 2;
                to[0] = sqrtf(most);
                to[1] = far;
            }
            __syncthreads();
            if (passed != 0) {
                if (past_range) {
                    lift -= 14;
                    lse2 += 14.f;
                }
                zero(dq);
                walk_keys();
            }
            const float down = power_of_two(-lift);
#pragma unroll
            for (int db = 0; db < DP / 32; ++db)
#pragma unroll
                for (int x = 0; x < 16; ++x) dq[db][x] *= down;
        }
    }
    if (in) store_row<T, DP>(a.dq, place.at, g.D, dq, a.scale, live);
}

// dk and dv.  A wave has 32 keys as columns of its matrix tiles and walks the
// rows that see one of the workgroup's 128 keys, tile by tile: scores and
// dout v^T come as rows x keys, and P and dS go on from their registers to the
// products with dout and q.  Where a tile's walk is long for the call, workgroups of
// their own walk parts of it, whose sums a third kernel joins in order.
//
// In fp16 P and dS go in times 2^lift, between 1 and 2^15, which comes out of the sums in 32
// bits: with many keys both are among fp16's subnormals otherwise (24,576 keys, dout of
// 1e-3: dk off by 20 times its own rounding).  The workgroup takes the largest lift at
// which no dS can pass 2^15, from its own |v| and the largest |dout| and |delta| that the
// rows' kernel left for each of its tiles: |dS| <= P (|dout| |v| + |delta|).
template <class T, int DP>
__global__ __launch_bounds__(kAttnBlock, 2) void ua2a_attention_keys_kernel(AttnGradArgs a)
{
    // Of the four operands that a wave keeps for the whole walk the keys' do not fit
    // the registers beside sums of 128 values (they spill: 3.46 ms against 3.02), so
    // they lie in LDS, and tiles of rows are half as long (which alone costs a fifth:
    // heads of 64, 102 us against 128).
    constexpr bool kKeysInLds = DP == 128;
    constexpr int ROWS = kKeysInLds ? 32 : 64;
    constexpr uint32_t kTile = ROWS * kRow<DP>;
    constexpr uint32_t kKeyTile = kKeysInLds ? kAttnGradKeys * kRow<DP> : 0;
    // two buffers of q and dout, and the workgroup's keys
    __shared__ __attribute__((aligned(1024))) char lds[4 * kTile + kKeyTile];
    char* const ktile = lds + 4 * kTile;
    __shared__ __attribute__((aligned(16))) float stats[2 * 2 * ROWS];       // ... of lse and -delta
    constexpr bool kLifted = !__is_same(T, __bf16);
    __shared__ float sizes[kLifted ? 4 : 1][3];                              // the waves' largest |v|^2, |dout| and |delta|
    const AttnGeom& g = a.g;
    const uint32_t item = attn_item(g, (blockIdx.y << kAttnGridLog) + blockIdx.x);
    if (item >= g.items) return;
    const KeyPlace at = key_place(g, a.keys, item);
    const uint32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
    const uint32_t half = lane >> 5, col = lane & 31;
    const AttnSeq seq = attn_seq(g, 0, a.counts != nullptr ? static_cast<int64_t>(a.counts[at.at.i]) : static_cast<int64_t>(g.n));
    const uint32_t first = at.at.tile * kAttnGradKeys, past = umin32(first + kAttnGradKeys, g.keys);
    const uint32_t j = first + wave * 32 + col;
    const bool in = j < past, live = in && static_cast<int32_t>(j) < seq.end;
    const int64_t to = ((static_cast<int64_t>(at.at.seq) * g.keys + (in ? j : first)) * g.kvl + at.at.kvh) * g.D;
    f32x16v dk[DP / 32], dv[DP / 32];
    zero(dk);
    zero(dv);
    float down = 1.f;                                            // undoes the lift of P and dS
    if (static_cast<int32_t>(first) < seq.end) {
        u32x4v v[DP / 16], k[kKeysInLds ? 1 : DP / 16];
        row_operands<DP>(static_cast<const uint16_t*>(a.v) + to, g.D, half, live, v);
        if constexpr (!kKeysInLds) {
            row_operands<DP>(static_cast<const uint16_t*>(a.k) + to, g.D, half, live, k);
        } else {
            typedef TileLoads<DP, kAttnGradKeys> Loads;
            const uint32_t row_bytes = g.kvl * g.D * 2;
            const int64_t start = ((static_cast<int64_t>(at.at.seq) * g.keys + first) * g.kvl + at.at.kvh) * g.D * 2;
            const int32_t n = static_cast<int32_t>(past) < seq.end ? static_cast<int32_t>(past - first) : seq.end - static_cast<int32_t>(first);
            const u32x4v from_k = descriptor(static_cast<const char*>(a.k) + start, static_cast<uint32_t>(n) * row_bytes);
#pragma unroll
            for (int i = 0; i < Loads::N; ++i) {
                if (!Loads::has(i, wave)) continue;
                const uint32_t bytes = Loads::bytes(i, wave, g.D);
                load_to_lds(from_k, bytes == kNowhere ? kNowhere : Loads::row(i, wave) * row_bytes + bytes,
                            ktile + (i * 4 + wave) * 1024);
            }
        }
        // the rows that see this lane's key, and those that see one of the workgroup's
        const Span32 mine = live ? seers_of(g.win, static_cast<int32_t>(j), static_cast<int32_t>(j) + 1, seq.end) : Span32{0, 0};
        const uint32_t ra = static_cast<uint32_t>(mine.first) * g.group, rb = static_cast<uint32_t>(mine.last) * g.group;
        const int32_t end = static_cast<int32_t>(past) < seq.end ? static_cast<int32_t>(past) : seq.end;
        const RowWalk walk = row_walk(g, seers_of(g.win, static_cast<int32_t>(first), end, seq.end), ROWS);
        const uint32_t from = split_at(walk.total, at.parts, at.at.split), upto = split_at(walk.total, at.parts, at.at.split + 1);
        const uint32_t live_rows = static_cast<uint32_t>(seq.last) * g.group;
        int32_t lift = 0;
        if constexpr (kLifted) {
            float norm = 0.f, most = 0.f, far = 0.f;             // |v|^2; of the rows to walk, |dout| and |delta|
#pragma unroll
            for (int ks = 0; ks < DP / 16; ++ks) norm = dot2_sum(v[ks], v[ks], norm, T{});
            norm = add_halves(norm);
            const uint32_t tiles = (g.rows + kAttnRows - 1) / kAttnRows;
            if (from < upto) {
                const uint32_t last = umin32((walk.from + upto) * ROWS, live_rows);
                for (uint32_t t = (walk.from + from) * ROWS / kAttnRows + threadIdx.x; t * kAttnRows < last; t += kAttnBlock) {
                    const float* const of = a.sizes + (static_cast<int64_t>(at.at.unit) * tiles + t) * 2;
                    most = fmaxf(most, of[0]);
                    far = fmaxf(far, of[1]);
                }
            }
            norm = max_wave(norm);
            most = max_wave(most);
            far = max_wave(far);
            if (lane == 0) {
                sizes[wave][0] = norm;
                sizes[wave][1] = most;
                sizes[wave][2] = far;
            }
            __syncthreads();
#pragma unroll
            for (int w = 0; w < 4; ++w) {
                norm = fmaxf(norm, sizes[w][0]);
                most = fmaxf(most, sizes[w][1]);
                far = fmaxf(far, sizes[w][2]);
            }
            // P to 1, and any dS, within 2^15, where that takes no less than 1
            lift = __builtin_amdgcn_readfirstlane(clamped(14 - exponent_of(sqrtf(norm) * most + far), 0, 15));
            down = power_of_two(-lift);
        }
        typedef TileLoads<DP, ROWS> Loads;
        uint32_t bytes[Loads::N];
#pragma unroll
        for (int n = 0; n < Loads::N; ++n) bytes[n] = Loads::bytes(n, wave, g.D);
        const uint32_t token_bytes = g.hl * g.D * 2, head_bytes = g.D * 2;
        const auto load = [&](uint32_t i, char* tile, float* stat) {
            const uint32_t r0 = (walk.from + i) * ROWS, t0 = fdiv(r0, g.d_group);
            const int64_t start = row_place(g, at.at, t0 * g.group).at * 2;
            const u32x4v q = descriptor(static_cast<const char*>(a.q) + start, kNowhere),
                         go = descriptor(static_cast<const char*>(a.dout) + start, kNowhere);
#pragma unroll
            for (int n = 0; n < Loads::N; ++n) {
                if (!Loads::has(n, wave)) continue;
                const uint32_t r = r0 + Loads::row(n, wave), t = fdiv(r, g.d_group);
                const uint32_t off = (t - t0) * token_bytes + (r - t * g.group) * head_bytes + bytes[n];
                const uint32_t from_row = bytes[n] == kNowhere || r >= live_rows ? kNowhere : off;
                char* const to_lds = tile + (n * 4 + wave) * 1024;
                load_to_lds(q, from_row, to_lds);
                load_to_lds(go, from_row, to_lds + kTile);
            }
            if (threadIdx.x < 2 * ROWS) {
                const uint32_t r = r0 + (threadIdx.x & (ROWS - 1));
                const bool is_lse = threadIdx.x < ROWS;
                float x = is_lse ? __builtin_inff() : 0.f;
                if (r < live_rows)
                    x = is_lse ? lse2_of(a.lse[row_place(g, at.at, r).stat]) - static_cast<float>(lift)
                               : -a.delta[static_cast<int64_t>(at.at.unit) * g.rows + r];
                stat[threadIdx.x] = x;
            }
        };
        char *tile = lds, *other = lds + 2 * kTile;
        float *stat = stats, *other_stat = stats + 2 * ROWS;
        if (from < upto) load(from, tile, stat);
        for (uint32_t i = from; i < upto; ++i) {
            const char *qtile = tile, *gtile = tile + kTile;
            arrived();
            if (i + 1 < upto) load(i + 1, other, other_stat);
#pragma unroll 1
            for (uint32_t half_tile = 0; half_tile < ROWS / 32; ++half_tile) {
                const uint32_t row0 = half_tile * 32, r0 = (walk.from + i) * ROWS + row0;
                const bool none = r0 + 32 <= ra || r0 >= rb, all = ra <= r0 && r0 + 32 <= rb;
                if (__builtin_amdgcn_ballot_w64(live && !none) == 0) continue;
                const bool masked = __builtin_amdgcn_ballot_w64(live && !all) != 0;
                f32x16v s, dp;
#pragma unroll
                for (int b = 0; b < 4; ++b) {
                    const f32x4v d = *reinterpret_cast<const f32x4v*>(stat + ROWS + row0 + b * 8 + half * 4);
#pragma unroll
                    for (int x = 0; x < 4; ++x) {
                        s[4 * b + x] = 0.f;
                        dp[4 * b + x] = d[x];
                    }
                }
#pragma unroll
                for (int ks = 0; ks < DP / 16; ++ks) {
                    if constexpr (kKeysInLds)
                        s = mfma<T>(along<DP>(qtile, row0, ks), along<DP>(ktile, wave * 32, ks), s);
                    else
                        s = mfma<T>(along<DP>(qtile, row0, ks), k[ks], s);
                }
#pragma unroll
                for (int ks = 0; ks < DP / 16; ++ks) dp = mfma<T>(along<DP>(gtile, row0, ks), v[ks], dp);
#pragma unroll
                for (int b = 0; b < 4; ++b) {
                    const f32x4v l = *reinterpret_cast<const f32x4v*>(stat + row0 + b * 8 + half * 4);
#pragma unroll
                    for (int x = 0; x < 4; ++x)
                        s[4 * b + x] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[4 * b + x], a.scale2, -l[x]));
                }
                if (masked) {
#pragma unroll
                    for (int x = 0; x < 16; ++x) {
                        const uint32_t r = r0 + (x / 4) * 8 + half * 4 + x % 4;
                        if (!(r >= ra && r < rb)) s[x] = dp[x] = 0.f;
                    }
                }
#pragma unroll
                for (int x = 0; x < 16; ++x) dp[x] *= s[x];
                const u32x4v p[2] = {operand_of<T>(s, 0), operand_of<T>(s, 1)};
                const u32x4v ds[2] = {operand_of<T>(dp, 0), operand_of<T>(dp, 1)};
#pragma unroll
                for (int db = 0; db < DP / 32; ++db)
#pragma unroll
                    for (int t = 0; t < 2; ++t) dv[db] = mfma<T>(transposed<DP>(gtile, row0, t, db), p[t], dv[db]);
#pragma unroll
                for (int db = 0; db < DP / 32; ++db)
#pragma unroll
                    for (int t = 0; t < 2; ++t) dk[db] = mfma<T>(transposed<DP>(qtile, row0, t, db), ds[t], dk[db]);
            }
            char* const t = tile;
            tile = other;
            other = t;
            float* const u = stat;
            stat = other_stat;
            other_stat = u;
        }
    }
    if (!in) return;
    if constexpr (kLifted) {
#pragma unroll
        for (int db = 0; db < DP / 32; ++db)
#pragma unroll
            for (int x = 0; x < 16; ++x) {
                dk[db][x] *= down;
                dv[db][x] *= down;
            }
    }
    if (at.parts > 1) {
        float* line = a.partial + part_line(g, a.keys, at.at.unit, at.at.split, j) * 2 * g.D;
#pragma unroll
        for (int db = 0; db < DP / 32; ++db)
#pragma unroll
            for (int b = 0; b < 4; ++b) {
                const uint32_t d = db * 32 + b * 8 + half * 4;
                if (d >= g.D) continue;
                f32x4v x, y;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    x[e] = live ? dk[db][4 * b + e] : 0.f;
                    y[e] = live ? dv[db][4 * b + e] : 0.f;
                }
                *reinterpret_cast<f32x4v*>(line + d) = x;
                *reinterpret_cast<f32x4v*>(line + g.D + d) = y;
            }
        return;
    }
    store_row<T, DP>(a.dk, to, g.D, dk, a.scale, live);
    store_row<T, DP>(a.dv, to, g.D, dv, 1.f, live);
}

// The parts of keys whose rows were walked by several workgroups, joined in
// order: 2 * D / 4 lanes a key.
template <class T>
__global__ __launch_bounds__(kAttnBlock) void ua2a_attention_keys_join_kernel(AttnGradArgs a)
{
    const AttnGeom& g = a.g;
    const uint32_t per = g.D / 2, here = fdiv(threadIdx.x, a.keys.d_lanes);
    const uint32_t keys = a.keys.rest_parts > 1 ? g.keys : a.keys.span;      // of a unit that may have parts
    const uint32_t line = ((blockIdx.y << kAttnGridLog) + blockIdx.x) * a.keys.per_group + here;   // unit * keys + key
    if (here >= a.keys.per_group || line >= g.units * keys) return;
    const uint32_t c = (threadIdx.x - here * per) * 4;                       // of dk's and dv's D
    const uint32_t unit = fdiv(line, a.keys.d_keys), j = line - unit * keys;
    const uint32_t parts = j < a.keys.span ? a.keys.lead_parts : a.keys.rest_parts;
    if (parts <= 1) return;
    const uint32_t seq = fdiv(unit, g.d_kvl), kvh = unit - seq * g.kvl;
    f32x4v x = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
    for (uint32_t s = 0; s < parts; ++s)
        x += *reinterpret_cast<const f32x4v*>(a.partial + part_line(g, a.keys, unit, s, j) * 2 * g.D + c);
    const bool is_v = c >= g.D;
    const float f = is_v ? 1.f : a.scale;
    const int64_t to = ((static_cast<int64_t>(seq) * g.keys + j) * g.kvl + kvh) * g.D + (is_v ? c - g.D : c);
    *reinterpret_cast<u32x2v*>(static_cast<uint16_t*>(is_v ? a.dv : a.dk) + to) =
        u32x2v{pack2<T>(x[0] * f, x[1] * f), pack2<T>(x[2] * f, x[3] * f)};
}

template <class T, int DP>
const void* sized_fn(const AttnLaunch& L)
{
    return L.kernel == AttnKernel::GradRows ? reinterpret_cast<const void*>(&ua2a_attention_rows_kernel<T, DP>)
                                            : reinterpret_cast<const void*>(&ua2a_attention_keys_kernel<T, DP>);
}

template <class T>
const void* typed_fn(const AttnLaunch& L)
{
    if (L.kernel == AttnKernel::GradJoin) return reinterpret_cast<const void*>(&ua2a_attention_keys_join_kernel<T>);
    switch (L.DP) {
    case 32: return sized_fn<T, 32>(L);
    case 64: return sized_fn<T, 64>(L);
    case 96: return sized_fn<T, 96>(L);
    case 128: return sized_fn<T, 128>(L);
    }
    return nullptr;
}

}  // namespace

const void* attention_grad_kernel(const AttnLaunch& L)
{
    return L.type == UA2A_TYPE_BF16 ? typed_fn<__bf16>(L) : typed_fn<_Float16>(L);
}

}  // namespace ua2a
