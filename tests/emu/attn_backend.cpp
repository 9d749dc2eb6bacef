// A backend of the attention operators (tests only): carries the launches out on
// host memory in double, along the same walks, tiles, parts and places that the
// kernels take (ua2a_attn_geometry.h), and checks every place it writes: inside
// its buffer, and once.
#include <math.h>
#include <string.h>

#include <map>
#include <vector>

#include "ua2a_act_internal.h"
#include "ua2a_attn_internal.h"

namespace {

int64_t g_errors = 0;
int64_t g_last[8];
int32_t g_dry = 0;

void bad() { ++g_errors; }

// which places of the call's outputs have been written
std::map<const void*, std::vector<uint8_t>> g_written;
void wrote(const void* base, int64_t at, int64_t size)
{
    auto& w = g_written[base];
    if (w.empty()) w.assign(static_cast<size_t>(size), 0);
    if (at < 0 || at >= size || w[static_cast<size_t>(at)]++) bad();
}

double half_value(uint16_t u)
{
    const int e = u >> 10 & 31, m = u & 1023;
    const double v = e == 31 ? (m ? NAN : INFINITY) : e ? ldexp(1024 + m, e - 25) : ldexp(m, -24);
    return u & 0x8000 ? -v : v;
}
double get(const void* p, int64_t at, int32_t type)
{
    if (type == UA2A_TYPE_FP32) return static_cast<const float*>(p)[at];
    const uint16_t u = static_cast<const uint16_t*>(p)[at];
    if (type == UA2A_TYPE_FP16) return half_value(u);
    const uint32_t w = uint32_t(u) << 16;
    float f;
    memcpy(&f, &w, 4);
    return f;
}
// (fp16 results are not needed: the tests take bf16 and fp32 here)
void put(void* p, int64_t at, double v, int32_t type, int64_t size)
{
    wrote(p, at, size);
    if (type == UA2A_TYPE_FP32) {
        static_cast<float*>(p)[at] = static_cast<float>(v);
        return;
    }
    const float f = static_cast<float>(v);
    uint32_t u;
    memcpy(&u, &f, 4);
    if (f == f) u += 0x7fffu + ((u >> 16) & 1);
    static_cast<uint16_t*>(p)[at] = static_cast<uint16_t>(u >> 16);
}

double code_value(uint8_t c, int32_t format)
{
    const int mb = format == UA2A_FORMAT_E4M3 ? 3 : 2, bias = format == UA2A_FORMAT_E4M3 ? 7 : 15;
    const int e = (c & 0x7f) >> mb, m = c & ((1 << mb) - 1);
    if (format == UA2A_FORMAT_E4M3 ? (c & 0x7f) == 0x7f : e == 31) return m || mb == 3 ? NAN : c & 0x80 ? -INFINITY : INFINITY;
    const double v = e ? ldexp((1 << mb) + m, e - bias - mb) : ldexp(m, 1 - bias - mb);
    return c & 0x80 ? -v : v;
}

}  // namespace

namespace ua2a {
namespace {

AttnSeq seq_of(const AttnArgs& a, const AttnPlace& p)
{
    return attn_seq(a.g, a.starts ? a.starts[p.i] : 0, a.counts ? static_cast<int64_t>(a.counts[p.i]) : a.g.n);
}
int64_t row_at(const AttnGeom& g, const AttnPlace& p, uint32_t row)
{
    const uint32_t t = row / g.group;
    return ((int64_t(p.seq) * g.n + t) * g.hl + p.kvh * g.group + row % g.group) * g.D;
}
int64_t stat_at(const AttnGeom& g, const AttnPlace& p, uint32_t row)
{
    return (int64_t(p.seq) * g.hl + p.kvh * g.group + row % g.group) * g.n + row / g.group;
}

struct Kv {
    const AttnArgs& a;
    const AttnPlace& p;
    int32_t type;
    double at(bool value, int64_t j, uint32_t d) const
    {
        const AttnGeom& g = a.g;
        const int64_t head = (int64_t(p.seq) * g.keys + j) * g.kvl + p.kvh;
        if (j < 0 || j >= g.keys) {
            bad();
            return 0;
        }
        if (a.codes == nullptr) return get(value ? a.v : a.k, head * g.D + d, type);
        const double c = code_value(a.codes[(value ? a.part : 0) + head * g.D + d], a.format);
        return ldexp(c, int(a.scales[(value ? a.part_scales : 0) + head * g.nb + d / kBlockValues]) - 127);
    }
};

void finish(const AttnArgs& a, const AttnPlace& p, const AttnSeq& s, uint32_t row, int32_t type, const std::vector<double>& x,
            double m, double l)
{
    const AttnGeom& g = a.g;
    const int32_t t = static_cast<int32_t>(row / g.group);
    const bool live = t >= s.first && t < s.last;
    if (!live && a.keep) return;
    const int64_t size = int64_t(g.units) * g.rows * g.D;
    for (uint32_t d = 0; d < g.D; ++d)
        put(a.out, row_at(g, p, row) + d, live && l != 0 ? x[d] / l : 0, type, size);
    if (a.lse != nullptr) {
        wrote(a.lse, stat_at(g, p, row), int64_t(g.units) * g.rows);
        a.lse[stat_at(g, p, row)] = static_cast<float>(live && l != 0 ? m + log(l) : -INFINITY);
    }
}

void forward(const AttnLaunch& L, uint32_t id)
{
    const AttnArgs& a = L.attn;
    const AttnGeom& g = a.g;
    const uint32_t item = attn_item(g, id);
    if (item >= g.items) return;
    const AttnPlace p = attn_place(g, item);
    const AttnSeq s = seq_of(a, p);
    const bool decode = L.kernel == AttnKernel::Decode;
    const uint32_t per = decode ? kDecodeRows : L.shared ? kAttnWaveRows : kAttnRows;
    const uint32_t size = decode ? 32 : L.shared ? kAttnSplitKeys : kAttnKeys;
    const uint32_t first = p.tile * per, past = umin32(first + per, g.rows);
    const bool some = int32_t(first / g.group) < s.last && int32_t((past - 1) / g.group) >= s.first;
    KeyWalk walk = {0, 0, 0};
    Seen top = {0, 0, 0}, bottom = {0, 0, 0};
    if (some) {
        top = seen_by_row(g, s, first);
        bottom = seen_by_row(g, s, past - 1);
        walk = key_walk(top, bottom, size);
    }
    const uint32_t from = split_at(walk.total, g.splits, p.split), to = split_at(walk.total, g.splits, p.split + 1);
    const Kv kv = {a, p, L.type};
    for (uint32_t row = first; row < past; ++row) {
        const int32_t t = static_cast<int32_t>(row / g.group);
        const bool live = t >= s.first && t < s.last;
        std::vector<double> x(g.D, 0);
        double m = -INFINITY, l = 0;
        std::vector<std::pair<int64_t, double>> sc;
        if (live) {
            const Seen seen = seen_by_row(g, s, row);
            for (uint32_t i = from; i < to; ++i) {
                const int32_t k0 = static_cast<int32_t>(walk_tile(walk, i) * size);
                for (int32_t j = k0; j < k0 + int32_t(size) && j < s.end; ++j) {
                    const bool see = sees(seen, j);
                    if (all_seen(top, bottom, k0, k0 + int32_t(size)) && !see) bad();
                    if (none_seen(top, bottom, k0, k0 + int32_t(size)) && see) bad();
                    if (!see) continue;
                    double dot = 0;
                    for (uint32_t d = 0; d < g.D; ++d) dot += get(a.q, row_at(g, p, row) + d, L.type) * kv.at(false, j, d);
                    sc.push_back({j, dot * a.scale2 / kLog2e});
                    if (sc.back().second > m) m = sc.back().second;
                }
            }
            for (const auto& e : sc) {
                const double w = exp(e.second - m);
                l += w;
                for (uint32_t d = 0; d < g.D; ++d) x[d] += w * kv.at(true, e.first, d);
            }
        }
        if (g.splits == 1) {
            finish(a, p, s, row, L.type, x, m, l);
            continue;
        }
        const int64_t lines = int64_t(g.units) * g.rows, line = int64_t(p.split) * lines + int64_t(p.unit) * g.rows + row;
        for (uint32_t d = 0; d < g.D; ++d) {
            wrote(a.partial, line * g.D + d, g.splits * lines * g.D);
            a.partial[line * g.D + d] = static_cast<float>(x[d]);
        }
        wrote(a.stats, line, g.splits * lines);
        a.stats[line * 2] = static_cast<float>(m * kLog2e);
        a.stats[line * 2 + 1] = static_cast<float>(l);
    }
}

void join(const AttnLaunch& L, uint32_t id)
{
    const AttnArgs& a = L.attn;
    const AttnGeom& g = a.g;
    const JoinShape js = join_shape(g);
    if (js.wide * 4 < g.D || js.rows * js.at_once * js.wide != 256) bad();
    for (uint32_t k = 0; k < js.rows; ++k) {
        const uint32_t line = id * js.rows + k;
        if (line >= g.units * g.rows) return;
        AttnPlace p;
        p.unit = fdiv(line, g.d_rows);
        p.seq = p.unit / g.kvl;
        p.kvh = p.unit % g.kvl;
        p.i = p.seq % g.seqs;
        const AttnSeq s = seq_of(a, p);
        const int64_t lines = int64_t(g.units) * g.rows;
        double m = -INFINITY, l = 0;
        for (uint32_t i = 0; i < g.splits; ++i) m = fmax(m, a.stats[(i * lines + line) * 2]);
        std::vector<double> x(g.D, 0);
        for (uint32_t i = 0; i < g.splits; ++i) {
            const double w = m == -INFINITY ? 0 : exp2(a.stats[(i * lines + line) * 2] - m);
            l += w * a.stats[(i * lines + line) * 2 + 1];
            for (uint32_t d = 0; d < g.D; ++d) x[d] += w * a.partial[(i * lines + line) * g.D + d];
        }
        finish(a, p, s, line - p.unit * g.rows, L.type, x, m / kLog2e, l);
    }
}

struct GradRow {
    double p, ds;
};
GradRow grad_of(const AttnGradArgs& a, const AttnPlace& at, uint32_t row, int64_t j, int32_t type)
{
    const AttnGeom& g = a.g;
    const int64_t q = row_at(g, at, row), k = ((int64_t(at.seq) * g.keys + j) * g.kvl + at.kvh) * g.D;
    double s = 0, dp = 0, delta = 0;
    for (uint32_t d = 0; d < g.D; ++d) {
        const double go = get(a.dout, q + d, type);
        s += get(a.q, q + d, type) * get(a.k, k + d, type);
        dp += go * get(a.v, k + d, type);
        delta += go * get(a.out, q + d, type);
    }
    GradRow r;
    r.p = exp(s * a.scale - a.lse[stat_at(g, at, row)]);
    r.ds = r.p * (dp - delta);
    return r;
}

void grad_rows(const AttnLaunch& L, uint32_t id)
{
    const AttnGradArgs& a = L.grad;
    const AttnGeom& g = a.g;
    const uint32_t item = attn_item(g, id);
    if (item >= g.items) return;
    const AttnPlace p = attn_place(g, item);
    const AttnSeq s = attn_seq(g, 0, a.counts ? static_cast<int64_t>(a.counts[p.i]) : g.n);
    const uint32_t first = p.tile * kAttnRows, past = umin32(first + kAttnRows, g.rows);
    for (uint32_t row = first; row < past; ++row) {
        const bool live = int32_t(row / g.group) < s.last;
        std::vector<double> x(g.D, 0);
        if (live) {
            const KeyWalk walk = key_walk(seen_by_row(g, s, first), seen_by_row(g, s, past - 1), kAttnKeys);
            const Seen seen = seen_by_row(g, s, row);
            for (uint32_t i = 0; i < walk.total; ++i)
                for (uint32_t e = 0; e < kAttnKeys; ++e) {
                    const int32_t j = static_cast<int32_t>(walk_tile(walk, i) * kAttnKeys + e);
                    if (j >= s.end || !sees(seen, j)) continue;
                    const GradRow r = grad_of(a, p, row, j, L.type);
                    for (uint32_t d = 0; d < g.D; ++d)
                        x[d] += r.ds * get(a.k, ((int64_t(p.seq) * g.keys + j) * g.kvl + p.kvh) * g.D + d, L.type);
                }
        }
        wrote(a.delta, int64_t(p.unit) * g.rows + row, int64_t(g.units) * g.rows);
        for (uint32_t d = 0; d < g.D; ++d)
            put(a.dq, row_at(g, p, row) + d, x[d] * a.scale, L.type, int64_t(g.units) * g.rows * g.D);
    }
}

int64_t lines_of(const AttnGradArgs& a)
{
    const KeyTiles& t = a.keys;
    return t.rest_line + (t.rest_parts > 1 ? int64_t(t.rest_parts) * a.g.units * (a.g.keys - t.span) : 0);
}

void grad_keys(const AttnLaunch& L, uint32_t id)
{
    const AttnGradArgs& a = L.grad;
    const AttnGeom& g = a.g;
    const uint32_t item = attn_item(g, id), size = L.DP == 128 ? 32 : 64;
    if (item >= g.items) return;
    const KeyPlace kp = key_place(g, a.keys, item);
    const AttnPlace& p = kp.at;
    if (p.unit >= g.units || p.tile >= g.tiles || p.split >= kp.parts) bad();
    const AttnSeq s = attn_seq(g, 0, a.counts ? static_cast<int64_t>(a.counts[p.i]) : g.n);
    const int32_t first = static_cast<int32_t>(p.tile * kAttnGradKeys);
    const int32_t past = static_cast<int32_t>(umin32(first + kAttnGradKeys, g.keys));
    const int64_t kv = int64_t(g.units) * g.keys * g.D;
    RowWalk walk = {0, 0};
    if (first < s.end) walk = row_walk(g, seers_of(g.win, first, past < s.end ? past : s.end, s.end), size);
    const uint32_t from = split_at(walk.total, kp.parts, p.split), to = split_at(walk.total, kp.parts, p.split + 1);
    for (int32_t j = first; j < past; ++j) {
        std::vector<double> dk(g.D, 0), dv(g.D, 0);
        if (j < s.end) {
            const Span32 mine = seers_of(g.win, j, j + 1, s.end);
            const uint32_t ra = uint32_t(mine.first) * g.group, rb = uint32_t(mine.last) * g.group;
            for (uint32_t i = from; i < to; ++i)
                for (uint32_t e = 0; e < size; ++e) {
                    const uint32_t row = (walk.from + i) * size + e;
                    if (row < ra || row >= rb) continue;
                    if (int32_t(row / g.group) >= s.last || !sees(seen_by_row(g, s, row), j)) bad();
                    const GradRow r = grad_of(a, p, row, j, L.type);
                    for (uint32_t d = 0; d < g.D; ++d) {
                        dk[d] += r.ds * get(a.q, row_at(g, p, row) + d, L.type);
                        dv[d] += r.p * get(a.dout, row_at(g, p, row) + d, L.type);
                    }
                }
        }
        for (uint32_t d = 0; d < g.D; ++d) {
            const int64_t to_kv = ((int64_t(p.seq) * g.keys + j) * g.kvl + p.kvh) * g.D + d;
            if (kp.parts == 1) {
                put(a.dk, to_kv, dk[d] * a.scale, L.type, kv);
                put(a.dv, to_kv, dv[d], L.type, kv);
                continue;
            }
            const int64_t line = part_line(g, a.keys, p.unit, p.split, static_cast<uint32_t>(j)) * 2 * g.D;
            for (int h = 0; h < 2; ++h) {
                wrote(a.partial, line + h * g.D + d, lines_of(a) * 2 * g.D);
                a.partial[line + h * g.D + d] = static_cast<float>(h ? dv[d] : dk[d]);
            }
        }
    }
}

void grad_join(const AttnLaunch& L, uint32_t id)
{
    const AttnGradArgs& a = L.grad;
    const AttnGeom& g = a.g;
    const uint32_t keys = a.keys.rest_parts > 1 ? g.keys : a.keys.span;
    if (a.keys.per_group * (g.D / 2) > kAttnBlock || a.keys.d_keys.d != keys) bad();
    for (uint32_t k = 0; k < a.keys.per_group; ++k) {
        const uint32_t line = id * a.keys.per_group + k;
        if (line >= g.units * keys) return;
        const uint32_t unit = fdiv(line, a.keys.d_keys), j = line - unit * keys;
        const uint32_t parts = j < a.keys.span ? a.keys.lead_parts : a.keys.rest_parts;
        if (parts <= 1) continue;
        const uint32_t seq = unit / g.kvl, kvh = unit % g.kvl;
        for (uint32_t d = 0; d < 2 * g.D; ++d) {
            double x = 0;
            for (uint32_t s = 0; s < parts; ++s) x += a.partial[part_line(g, a.keys, unit, s, j) * 2 * g.D + d];
            const bool v = d >= g.D;
            put(v ? a.dv : a.dk, ((int64_t(seq) * g.keys + j) * g.kvl + kvh) * g.D + d % g.D, v ? x : x * a.scale, L.type,
                int64_t(g.units) * g.keys * g.D);
        }
    }
}

void rope(const AttnLaunch& L, uint32_t id)
{
    const RopeArgs& a = L.rope;
    const RopeGeom& g = a.g;
    const uint32_t V = static_cast<uint32_t>(L.V), D = g.sh.D;
    const int64_t size = int64_t(g.tokens) * g.sh.H * D;
    for (uint32_t tid = 0; tid < kRopeBlock; ++tid) {
        const uint32_t within = tid / g.lanes, lane = tid % g.lanes;
        const int64_t token = int64_t(id) * g.per_group + within;
        if (within >= g.per_group || token >= g.tokens) continue;
        const TokenPlace at = token_place(g.sh, static_cast<uint32_t>(token));
        const uint32_t where = g.per_plane ? at.a : at.a % g.sh.SG, h0 = lane / g.slots;
        for (uint32_t slot = lane % g.slots; slot < g.slots; slot += g.lanes) {
            const bool pairs = slot < g.turning;
            const bool apart = g.halves && V > 1;
            uint32_t d = slot * V, far = 0;
            if (apart) {
                d = pairs ? slot * V : 2 * g.pairs + (slot - g.turning) * V;
                far = g.pairs;
            } else if (V == 1) {
                d = !pairs ? 2 * g.pairs + (slot - g.turning) : g.halves ? slot : 2 * slot;
                far = g.halves ? g.pairs : 1;
            }
            for (uint32_t h = h0; h < g.sh.H; h += g.heads_at_once) {
                const auto offset = [&](bool A) {
                    return A ? a_offset(g.sh, at.a, h, D, g.sh.a_rank, d) : (int64_t(at.p) * g.sh.H + h) * D + d;
                };
                const int64_t from = offset(g.from_a), to = offset(g.to_a);
                const auto turn = [&](uint32_t pair, int64_t u, int64_t z) {
                    const int64_t pos = a.positions[a.axes[pair] * g.axis_stride + where];
                    const uint64_t f = static_cast<uint64_t>(pos) * a.turns[pair];
                    const double angle = ldexp(static_cast<double>(f), -64) * 2 * M_PI;
                    const double c = cos(angle), s = g.inverse ? -sin(angle) : sin(angle);
                    const double x = get(a.x, from + u, L.type), y = get(a.x, from + z, L.type);
                    put(a.out, to + u, x * c - y * s, L.type, size);
                    put(a.out, to + z, y * c + x * s, L.type, size);
                };
                const auto copy = [&](int64_t u) { put(a.out, to + u, get(a.x, from + u, L.type), L.type, size); };
                if (V == 1 || apart) {
                    for (uint32_t i = 0; i < V; ++i) {
                        if (!pairs) copy(i);
                        else turn((apart ? d : slot) + i, i, i + far);
                    }
                } else {
                    for (uint32_t i = 0; i < V; i += 2) {
                        if (d / 2 + i / 2 < g.pairs) {
                            turn(d / 2 + i / 2, i, i + 1);
                        } else {
                            copy(i);
                            copy(i + 1);
                        }
                    }
                }
            }
        }
    }
}

}  // namespace

int attn_launch(const AttnLaunch& L, void*)
{
    const int64_t last[] = {int64_t(L.kernel), L.grid_x, L.grid_y, L.attn.g.splits, L.V, L.DP, L.shared,
                            int64_t(L.grad.keys.lead_parts) << 32 | L.grad.keys.rest_parts};
    memcpy(g_last, last, sizeof last);
    if (L.grid_x < 1 || L.grid_y < 1 || L.grid_y > 65535 || L.grid_x > (1u << kAttnGridLog)) bad();
    if (g_dry) return 0;
    g_written.clear();
    for (uint32_t y = 0; y < L.grid_y; ++y)
        for (uint32_t x = 0; x < L.grid_x; ++x) {
            const uint32_t id = (y << kAttnGridLog) + x;
            switch (L.kernel) {
            case AttnKernel::Rope: rope(L, id); break;
            case AttnKernel::Forward:
            case AttnKernel::Decode: forward(L, id); break;
            case AttnKernel::Join: join(L, id); break;
            case AttnKernel::GradRows: grad_rows(L, id); break;
            case AttnKernel::GradKeys: grad_keys(L, id); break;
            case AttnKernel::GradJoin: grad_join(L, id); break;
            }
        }
    return 0;
}

int act_launch(const ActLaunch&, void*) { return 1; }
int backend_current_device(int32_t* device)
{
    *device = 0;
    return 0;
}
int backend_launch(const Launch&, void*) { return 1; }
const char* backend_error_name(int) { return "none"; }
int backend_scratch_window(int32_t, uint8_t** window)
{
    *window = nullptr;
    return 1;
}

}  // namespace ua2a

extern "C" {
int64_t ua2a_attn_emu_errors(void) { return g_errors; }
int64_t ua2a_attn_emu_last(int32_t k) { return g_last[k]; }
void ua2a_attn_emu_dry(int32_t on) { g_dry = on; }

// What the kernels take of a tile of `size` keys from k0 on, for rows at positions p0 .. p1 of a
// sequence of `end` keys: 1 all seen, 2 none seen; and in sees[] what the row at p0 sees of each.
int32_t ua2a_attn_emu_tile(const ua2a_window_t* w, int32_t p0, int32_t p1, int32_t end, uint32_t k0, uint32_t size,
                           uint8_t* seen)
{
    using namespace ua2a;
    WindowGeom g;
    g.left = static_cast<int32_t>(w->left);
    g.right = static_cast<int32_t>(w->right);
    g.sinks = static_cast<int32_t>(w->sinks);
    g.chunk = static_cast<uint32_t>(w->chunk);
    g.d_chunk = make_div32(g.chunk);
    const Seen a = seen_by(g, p0, end), b = seen_by(g, p1, end);
    for (uint32_t i = 0; i < size; ++i) seen[i] = sees(a, k0 + i);
    return (all_seen(a, b, k0, k0 + size) ? 1 : 0) | (none_seen(a, b, k0, k0 + size) ? 2 : 0);
}
}
