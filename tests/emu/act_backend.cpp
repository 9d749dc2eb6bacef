// Host stand-in for the device side of the activation operators (tests only):
// every launch is carried out lane by lane on host memory with the index
// functions of ua2a_act_geometry.h, the arithmetic written plainly.
// Each access is checked against the size of the buffer it belongs to, and
// each output byte may be written once; a violation sets an error that the
// test reads.  The norm kernels address their lanes' slots by offsets from a
// segment's base: those functions are walked too, for the kernel that the
// launch takes, and compared with the slots' own places (check_places).  The exchange's own launches are not part of this library.
#include <math.h>
#include <stdint.h>
#include <string.h>

#include <vector>

#include "ua2a_act_internal.h"

using namespace ua2a;

namespace {

int g_error = 0;              // first violation: 1 read, 2 write, 3 written twice, 4 place, 5 no such kernel
int g_launches = 0;
int g_dry = 0;                // launches are recorded only
ActLaunch g_last;

void flag(int e)
{
    if (!g_error) g_error = e;
}

struct Buf {
    uint8_t* p;
    int64_t bytes;
    std::vector<uint8_t> hits;
    Buf(const void* q, int64_t n) : p(static_cast<uint8_t*>(const_cast<void*>(q))), bytes(q ? n : 0) {}
    bool in(int64_t at, int64_t n) const { return at >= 0 && at + n <= bytes; }
    bool write(int64_t at, int64_t n)
    {
        if (!in(at, n)) {
            flag(2);
            return false;
        }
        if (hits.empty()) hits.assign(static_cast<size_t>(bytes), 0);
        for (int64_t k = at; k < at + n; ++k)
            if (hits[static_cast<size_t>(k)]++) flag(3);
        return true;
    }
};

float bits_f(uint32_t u)
{
    float f;
    memcpy(&f, &u, 4);
    return f;
}
uint32_t f_bits(float f)
{
    uint32_t u;
    memcpy(&u, &f, 4);
    return u;
}

float half_value(uint16_t u)
{
    const int e = u >> 10 & 31, m = u & 1023;
    const double v = e == 31 ? (m ? NAN : INFINITY) : e ? ldexp(1024 + m, e - 25) : ldexp(m, -24);
    return static_cast<float>(u & 0x8000 ? -v : v);
}

uint16_t half_of(float f)
{
    const uint16_t sign = signbit(f) ? 0x8000 : 0;
    const double a = fabs(static_cast<double>(f));
    if (f != f) return sign | 0x7e00;
    if (a >= 65520.0) return sign | 0x7c00;
    int e = -14;
    if (a != 0) {
        frexp(a, &e);
        e = e - 1 < -14 ? -14 : e - 1;
    }
    const int n = static_cast<int>(nearbyint(ldexp(a, 10 - e)));   // steps of the value's size
    return sign | static_cast<uint16_t>(((e + 14) << 10) + n);     // a carry moves on to the exponent
}

// one value of the type at element `at`
float get(const Buf& b, int64_t at, int32_t type)
{
    const int64_t e = type == UA2A_TYPE_FP32 ? 4 : 2;
    if (!b.in(at * e, e)) {
        flag(1);
        return 0.f;
    }
    if (type == UA2A_TYPE_FP32) {
        float f;
        memcpy(&f, b.p + at * 4, 4);
        return f;
    }
    uint16_t u;
    memcpy(&u, b.p + at * 2, 2);
    if (type == UA2A_TYPE_BF16) return bits_f(uint32_t(u) << 16);
    return half_value(u);
}

float round_to(float f, int32_t type)
{
    if (type == UA2A_TYPE_FP32) return f;
    if (type == UA2A_TYPE_FP16) return half_value(half_of(f));
    if (f != f) return f;
    uint32_t u = f_bits(f);
    u += 0x7fffu + ((u >> 16) & 1);
    return bits_f(u & 0xffff0000u);
}

void put(Buf& b, int64_t at, float f, int32_t type)
{
    const int64_t e = type == UA2A_TYPE_FP32 ? 4 : 2;
    if (!b.write(at * e, e)) return;
    if (type == UA2A_TYPE_FP32) {
        memcpy(b.p + at * 4, &f, 4);
        return;
    }
    uint16_t u;
    if (type == UA2A_TYPE_BF16) {
        u = static_cast<uint16_t>(f_bits(round_to(f, type)) >> 16);
    } else {
        u = half_of(f);
    }
    memcpy(b.p + at * 2, &u, 2);
}

void put8(Buf& b, int64_t at, uint8_t v)
{
    if (b.write(at, 1)) b.p[at] = v;
}
uint8_t get8(const Buf& b, int64_t at)
{
    if (b.in(at, 1)) return b.p[at];
    flag(1);
    return 0;
}

struct Format {
    int mantissa, bias;
    uint8_t nan, inf;
    double most;
};
Format format_of(int32_t f)
{
    if (f == UA2A_FORMAT_E4M3) return {3, 7, 0x7f, 0x7f, 448.0};
    return {2, 15, 0x7f, 0x7c, 57344.0};
}

double code_value(uint8_t c, int32_t f)
{
    const Format q = format_of(f);
    const int mag = c & 0x7f, e = mag >> q.mantissa, m = mag & ((1 << q.mantissa) - 1);
    double v;
    if (f == UA2A_FORMAT_E4M3 ? mag == 0x7f : mag > 0x7c)
        v = NAN;
    else if (f == UA2A_FORMAT_E5M2 && mag == 0x7c)
        v = INFINITY;
    else if (e == 0)
        v = ldexp(m, 1 - q.bias - q.mantissa);
    else
        v = ldexp((1 << q.mantissa) + m, e - q.bias - q.mantissa);
    return (c & 0x80) ? -v : v;
}

uint8_t code_of(double x, int32_t f)
{
    const Format q = format_of(f);
    const uint8_t sign = signbit(x) ? 0x80 : 0;
    if (x != x) return sign | q.nan;
    if (isinf(x)) return sign | q.inf;
    const double a = fabs(x);
    if (a == 0) return sign;
    int e;
    frexp(a, &e);
    e -= 1;
    if (e < 1 - q.bias) e = 1 - q.bias;
    double n = nearbyint(ldexp(a, q.mantissa - e));            // steps of the value's size
    if (n >= (2 << q.mantissa)) {
        n /= 2;
        e += 1;
    }
    if (n < (1 << q.mantissa)) return sign | static_cast<uint8_t>(n);   // subnormal
    return sign | static_cast<uint8_t>(((e + q.bias) << q.mantissa) + (static_cast<int>(n) - (1 << q.mantissa)));
}

// what a scale byte stands for
double scale_value(uint8_t s) { return s == 255 ? NAN : ldexp(1.0, s - 127); }

// scale exponent of a block's values, by search
int scale_exponent(const std::vector<float>& v, int32_t f)
{
    double m = 0;
    for (float x : v)
        if (isfinite(x) && fabs(x) > m) m = fabs(x);
    int k = -127;
    while (k < 127 && m > ldexp(format_of(f).most, k)) ++k;
    return k;
}

// quantises a head (D values) and stores codes and scales
void put_head(Buf& codes, Buf& scales, int64_t at, int64_t scale0, const std::vector<float>& v, int32_t f)
{
    for (size_t lo = 0; lo < v.size(); lo += kBlockValues) {
        const size_t hi = lo + kBlockValues < v.size() ? lo + kBlockValues : v.size();
        const int k = scale_exponent(std::vector<float>(v.begin() + lo, v.begin() + hi), f);
        for (size_t i = lo; i < hi; ++i) put8(codes, at + i, code_of(ldexp(static_cast<double>(v[i]), -k), f));
        put8(scales, scale0 + lo / kBlockValues, static_cast<uint8_t>(k + 127));
    }
}

// Every lane slot of a norm launch: fn(segment, slot), in the kernel's order.
template <class F>
void norm_lanes(const ActLaunch& L, const NormGeom& g, F fn)
{
    const uint32_t wgs = L.grid_x * L.grid_y;
    for (uint32_t wg = 0; wg < wgs; ++wg)
        for (uint32_t group = wg; group < g.groups; group += wgs)
            for (uint32_t tid = 0; tid < L.block; ++tid) {
                const Segment s = segment_of(g, group, tid / g.lanes);
                if (!s.live) continue;
                const uint32_t lane = tid % g.lanes;
                for (int32_t it = 0; it < L.items; ++it) {
                    const uint32_t slot = lane + static_cast<uint32_t>(it) * g.lanes;
                    const Slot sl = g.head_log ? bundle_slot(g, slot, static_cast<uint32_t>(L.V))
                                           : norm_slot(g, slot, static_cast<uint32_t>(L.V));
                    if (sl.ok) fn(s, sl);
                }
            }
}

int64_t scales_of(const NormGeom& g) { return int64_t(g.segs) * g.heads * g.sh.nb; }
int64_t values_of(const NormGeom& g) { return int64_t(g.segs) * g.heads * g.sh.D; }
// the norm that a slot belongs to, counted over all, and its number
bool per_head(const NormGeom& g) { return g.cols == g.sh.D; }
int64_t stats_of(const NormGeom& g) { return int64_t(g.segs) * (per_head(g) ? g.heads : 1); }
size_t stat(const NormGeom& g, const Segment& s, const Slot& sl)
{
    return per_head(g) ? static_cast<size_t>(s.at.p) * g.sh.H + s.h0 + sl.hh : s.at.p;
}
int64_t weight_at(const NormGeom& g, const Slot& sl) { return (per_head(g) ? 0 : int64_t(sl.hh) * g.sh.D) + sl.d; }

// What every lane of a norm kernel would address, padding and lanes past the
// last segment included: where a slot has values the place of those, else some
// place within the buffers.
template <Span SPAN, int V, int ITEMS>
void check_lanes(const ActLaunch& L, const NormGeom& g)
{
    const int64_t n = values_of(g), ns = scales_of(g);
    for (uint32_t group = 0; group < g.groups; ++group)
        for (uint32_t tid = 0; tid < L.block; ++tid) {
            const uint32_t lane = segment_lane<SPAN>(g, tid), within = segment_within<SPAN>(g, tid);
            if (lane != tid % g.lanes || within != tid / g.lanes) flag(4);
            const LaneSlots<ITEMS> l = lane_slots<SPAN, V, ITEMS>(g, lane);
            const SegmentBase b = segment_base<SPAN>(g, group, within);
            const SlotPlaces<SPAN, V, ITEMS> at{g, b, l, lane};
            const Segment s = segment_of(g, group, within);
            if (b.live != (s.live != 0)) flag(4);
            for (int it = 0; it < ITEMS; ++it) {
                const uint32_t slot = lane + static_cast<uint32_t>(it) * g.lanes;
                const Slot sl = g.head_log ? bundle_slot(g, slot, V) : norm_slot(g, slot, V);
                const int64_t p = b.p + at.p(it), a = b.a + at.a(it), sp = b.ps + at.scale_p(it), st = at.stat(it);
                const int64_t wt = weight_offset<SPAN, V>(g, l, lane, it);
                if (p < 0 || p + V > n || a < 0 || a + V > n || p % V || a % V || wt < 0 || wt + V > g.cols || wt % V ||
                    sp < 0 || sp >= ns || st < 0 || st >= stats_of(g))
                    flag(4);
                if (at.ok(it) != (sl.ok != 0) || (!sl.ok && !g.padded)) flag(4);
                if (!sl.ok) continue;
                if (p != value_at(g, s, sl, false) || a != value_at(g, s, sl, true) || sp != scale_at(g, s, sl, false) ||
                    b.as + at.scale_a(it) != scale_at(g, s, sl, true) || wt != weight_at(g, sl) ||
                    st != static_cast<int64_t>(stat(g, s, sl)))
                    flag(4);
            }
        }
}

// The kernels that are built: the slots per lane of each span.
template <int V>
void check_places_of(const ActLaunch& L, const NormGeom& g)
{
    const bool grad = L.kernel == ActKernel::NormGrad;
    if (L.span == kSpanPart && L.items == 1) return check_lanes<kPart, V, 1>(L, g);
    if (L.span == kSpanWide && L.items == 1) return check_lanes<kWide, V, 1>(L, g);
    if (L.span == kSpanWide && L.items == 2) return check_lanes<kWide, V, 2>(L, g);
    if (L.span == kSpanWide && L.items == 4) return check_lanes<kWide, V, 4>(L, g);
    if (L.span == kSpanWide && L.items == 8) return check_lanes<kWide, V, 8>(L, g);
    if (V == 1) return flag(5);
    if (L.span == kSpanBundle && L.items == 1) return check_lanes<kBundle, V, 1>(L, g);
    if (L.span == kSpanBundles && L.items == 1) return check_lanes<kBundles, V, 1>(L, g);
    if (grad && L.span == kSpanBundle && L.items == 2) return check_lanes<kBundle, V, 2>(L, g);
    if (grad && L.span == kSpanWaves && L.items == 2) return check_lanes<kWaves, V, 2>(L, g);
    if (grad && L.span == kSpanWaves && L.items == 3) return check_lanes<kWaves, V, 3>(L, g);
    if (grad && L.span == kSpanWaves && L.items == 4) return check_lanes<kWaves, V, 4>(L, g);
    if (grad && L.span == kSpanWaves && L.items == 5) return check_lanes<kWaves, V, 5>(L, g);
    flag(5);
}
void check_places(const ActLaunch& L, const NormGeom& g)
{
    if (L.V == 1)
        check_places_of<1>(L, g);
    else if (L.V == (L.type == UA2A_TYPE_FP32 ? 4 : 8))
        L.V == 4 ? check_places_of<4>(L, g) : check_places_of<8>(L, g);
    else
        flag(5);
}

void norm(const ActLaunch& L)
{
    check_places(L, L.norm.g);
    const NormArgs& a = L.norm;
    const bool mode1 = a.flags & kNormMode1;
    const int32_t out_format = !(a.flags & kNormOut8) ? 0 : a.flags & kNormOutE5M2 ? UA2A_FORMAT_E5M2 : UA2A_FORMAT_E4M3;
    const int32_t saved_format =
        !(a.flags & kNormSaved8) ? 0 : a.flags & kNormSavedE5M2 ? UA2A_FORMAT_E5M2 : UA2A_FORMAT_E4M3;
    const NormGeom& g = a.g;
    const int64_t n = values_of(g), e = L.type == UA2A_TYPE_FP32 ? 4 : 2;
    Buf x(a.x, n * e), res(a.residual, n * e), w(a.flags & kNormWeight ? a.weight : nullptr, int64_t(g.cols) * (a.weight_f32 ? 4 : e));
    Buf out(a.out, out_format ? n : n * e), osc(a.out_scales, scales_of(g)), sum(a.sum, n * e), saved(a.saved, n),
        ssc(a.saved_scales, scales_of(g)), rstd(a.flags & kNormRstd ? a.rstd : nullptr, stats_of(g) * 4);
    std::vector<double> ss(static_cast<size_t>(stats_of(g)), 0.0);
    std::vector<float> h(static_cast<size_t>(n)), y(static_cast<size_t>(n));   // P order
    norm_lanes(L, g, [&](const Segment& s, const Slot& sl) {
        for (int32_t i = 0; i < L.V; ++i) {
            const int64_t p = value_at(g, s, sl, false) + i;
            float v = get(x, value_at(g, s, sl, mode1) + i, L.type);
            if (a.flags & kNormResidual) {
                v = round_to(v + get(res, p, L.type), L.type);
                put(sum, p, v, L.type);
            }
            h[static_cast<size_t>(p)] = v;
            ss[stat(g, s, sl)] += double(v) * v;
        }
    });
    norm_lanes(L, g, [&](const Segment& s, const Slot& sl) {
        const double r = 1.0 / sqrt(ss[stat(g, s, sl)] * a.inv_len + a.eps);
        for (int32_t i = 0; i < L.V; ++i) {
            const int64_t p = value_at(g, s, sl, false) + i;
            const float wt = w.p ? get(w, weight_at(g, sl) + i, a.weight_f32 ? UA2A_TYPE_FP32 : L.type) : 1.f;
            y[static_cast<size_t>(p)] = static_cast<float>(h[static_cast<size_t>(p)] * r * wt);
            if (!out_format) put(out, value_at(g, s, sl, !mode1) + i, y[static_cast<size_t>(p)], L.type);
        }
        if (rstd.p && (per_head(g) || sl.hh == 0) && sl.d == 0) put(rstd, static_cast<int64_t>(stat(g, s, sl)), static_cast<float>(r), UA2A_TYPE_FP32);
        if (sl.d == 0) {                                        // a head's first slot: the whole head's 8 bits
            const int64_t p = value_at(g, s, sl, false);
            const auto head = [&](const std::vector<float>& v) {
                return std::vector<float>(v.begin() + p, v.begin() + p + g.sh.D);
            };
            if (saved_format)
                put_head(saved, ssc, p, scale_at(g, s, sl, false), head(h), saved_format);
        }
    });
    if (out_format)
        norm_lanes(L, g, [&](const Segment& s, const Slot& sl) {
            if (sl.d != 0) return;
            const int64_t p = value_at(g, s, sl, false);
            put_head(out, osc, value_at(g, s, sl, !mode1), scale_at(g, s, sl, !mode1),
                     std::vector<float>(y.begin() + p, y.begin() + p + g.sh.D), out_format);
        });
}

void norm_grad(const ActLaunch& L)
{
    check_places(L, L.grad.g);
    const NormGradArgs& a = L.grad;
    const bool mode1 = a.flags & kNormMode1;
    const NormGeom& g = a.g;
    const int64_t n = values_of(g), e = L.type == UA2A_TYPE_FP32 ? 4 : 2;
    Buf dy(a.dy, n * e), dsum(a.flags & kNormResidual ? a.dsum : nullptr, n * e), saved(a.saved, a.saved_format ? n : n * e), ssc(a.saved_scales, scales_of(g)),
        w(a.flags & kNormWeight ? a.weight : nullptr, int64_t(g.cols) * (a.weight_f32 ? 4 : e)), rstd(a.rstd, stats_of(g) * 4);
    Buf dx(a.dx, n * e), dres(a.flags & kNormApart ? a.dresidual : nullptr, n * e), partial(a.flags & kNormPartial ? a.partial : nullptr, int64_t(L.grid_x) * g.cols * 4);
    std::vector<double> dot(static_cast<size_t>(stats_of(g)), 0.0), dw(g.cols, 0.0);
    const auto each = [&](const Segment& s, const Slot& sl, int32_t i, double* gy, double* nh, double* d) {
        *d = get(dy, value_at(g, s, sl, !mode1) + i, L.type);
        double h;
        if (a.saved_format)
            h = code_value(get8(saved, value_at(g, s, sl, false) + i), a.saved_format) *
                scale_value(get8(ssc, scale_at(g, s, sl, false)));
        else
            h = get(saved, value_at(g, s, sl, (a.flags & kNormGathered) != 0) + i, L.type);
        const float wt = w.p ? get(w, weight_at(g, sl) + i, a.weight_f32 ? UA2A_TYPE_FP32 : L.type) : 1.f;
        *nh = h * get(rstd, static_cast<int64_t>(stat(g, s, sl)), UA2A_TYPE_FP32);
        *gy = *d * wt;
    };
    norm_lanes(L, g, [&](const Segment& s, const Slot& sl) {
        for (int32_t i = 0; i < L.V; ++i) {
            double gy, nh, d;
            each(s, sl, i, &gy, &nh, &d);
            dot[stat(g, s, sl)] += gy * nh;
            dw[static_cast<size_t>(weight_at(g, sl) + i)] += d * nh;
        }
    });
    norm_lanes(L, g, [&](const Segment& s, const Slot& sl) {
        for (int32_t i = 0; i < L.V; ++i) {
            double gy, nh, d;
            each(s, sl, i, &gy, &nh, &d);
            const int64_t p = value_at(g, s, sl, false) + i;
            double r = get(rstd, static_cast<int64_t>(stat(g, s, sl)), UA2A_TYPE_FP32) * (gy - nh * dot[stat(g, s, sl)] * a.inv_len);
            if (dsum.p) r += get(dsum, p, L.type);
            put(dx, mode1 ? value_at(g, s, sl, true) + i : p, static_cast<float>(r), L.type);
            if (dres.p) put(dres, p, static_cast<float>(r), L.type);
        }
    });
    if (partial.p)                                              // everything in the first workgroup's row
        for (int64_t k = 0; k < int64_t(L.grid_x) * g.cols; ++k)
            put(partial, k, k < g.cols ? static_cast<float>(dw[static_cast<size_t>(k)]) : 0.f, UA2A_TYPE_FP32);
}

void columns(const ActLaunch& L)
{
    const ColumnArgs& a = L.columns;
    Buf in(a.partial, int64_t(a.rows) * a.cols * 4), out(a.out, int64_t(a.cols) * 4);
    for (uint32_t c = 0; c < L.grid_x << a.across_log; ++c) {
        if (c >= a.cols) continue;
        float t = 0.f;
        for (uint32_t r = 0; r < a.rows; ++r) t += get(in, int64_t(r) * a.cols + c, UA2A_TYPE_FP32);
        put(out, c, t, UA2A_TYPE_FP32);
    }
}

void cache_write(const ActLaunch& L)
{
    const CacheArgs& a = L.cache;
    const CacheGeom& g = a.g;
    const int64_t e = L.type == UA2A_TYPE_FP32 ? 4 : 2, nval = int64_t(g.rows) * g.sh.H * g.sh.D;
    Buf codes(a.codes, 2 * g.part), scales(a.scales, 2 * g.part_scales);
    for (uint32_t y = 0; y < 2; ++y) {
        Buf val(y ? a.v : a.k, nval * e);
        if (!val.p) continue;
        std::vector<uint8_t> seen(static_cast<size_t>(g.rows) * g.slots, 0);
        for (uint32_t wg = 0; wg < L.grid_x * L.grid_y; ++wg) {
            const uint32_t group = cache_group(g, cache_workgroup(wg % L.grid_x, wg / L.grid_x));
            if (group >= g.groups) continue;
            for (uint32_t tid = 0; tid < L.block; ++tid) {
                const WriteLane l = write_lane(g, group, tid / g.lanes, tid);
                if (!l.in) continue;
                if (seen[static_cast<size_t>(l.token) * g.slots + l.slot]++) flag(3);
                const TokenPlace at = token_place(g.sh, l.token);
                const uint32_t i = fdiv(at.a, g.d_each), t = at.a - i * g.each;
                if (i >= g.seqs) {
                    flag(1);
                    continue;
                }
                const CacheSpan s = cache_span(g, a.starts ? a.starts[i] : 0, a.counts ? a.counts[i] : int64_t(g.each));
                if (t < s.first || t >= s.last) continue;
                const uint32_t b = l.slot >> g.q_log, h = fdiv(b, g.d_nb);
                const uint32_t d = (b - h * g.sh.nb) * kBlockValues +
                                   (l.slot & ((1u << g.q_log) - 1)) * static_cast<uint32_t>(L.V);
                if (g.dense && h * g.sh.D + d != l.slot * static_cast<uint32_t>(L.V)) flag(1);
                if (d != 0) continue;                           // a head's first slot does the head
                const uint32_t r = fdiv(h * g.sh.D, g.sh.d_run), rest = h * g.sh.D - r * g.sh.run;
                const int64_t row = (int64_t(r) * g.seqs + i) * g.cap + s.start + t;
                std::vector<float> v;
                for (uint32_t k = 0; k < g.sh.D; ++k)
                    v.push_back(get(val, (int64_t(l.token) * g.sh.H + h) * g.sh.D + k, L.type));
                put_head(codes, scales, (y ? g.part : 0) + row * g.sh.run + rest,
                         (y ? g.part_scales : 0) + row * g.sh.hl * g.sh.nb + int64_t(fdiv(rest, g.d_D)) * g.sh.nb, v,
                         a.format);
            }
        }
        for (uint8_t n : seen)
            if (n != 1) flag(2);
    }
}

void cache_read(const ActLaunch& L)
{
    const CacheArgs& a = L.cache;
    const CacheGeom& g = a.g;
    const int64_t e = L.type == UA2A_TYPE_FP32 ? 4 : 2, span = int64_t(g.each) * g.sh.run;
    Buf codes(a.codes, 2 * g.part), scales(a.scales, 2 * g.part_scales);
    for (uint32_t y = 0; y < 2; ++y) {
        Buf val(y ? a.v_out : a.k_out, g.spans * span * e);
        if (!val.p) continue;
        for (uint32_t id = 0; id < L.grid_x * L.grid_y; ++id) {
            const uint32_t wg = cache_workgroup(id % L.grid_x, id / L.grid_x);
            const uint32_t ri = fdiv(wg, g.d_tiles), tile = wg - ri * g.tiles, r = fdiv(ri, g.d_seqs), i = ri - r * g.seqs;
            if (ri >= g.spans) continue;
            if (i >= g.seqs) {
                flag(1);
                continue;
            }
            const CacheSpan s = cache_span(g, a.starts ? a.starts[i] : 0, a.counts ? a.counts[i] : int64_t(g.each));
            for (uint32_t tid = 0; tid < L.block; ++tid) {
                const int64_t at = (int64_t(tile) * L.block + tid) * L.V;
                if (at < s.first * g.sh.run || at >= s.last * g.sh.run) continue;
                const int64_t row = int64_t(ri) * g.cap + s.start;
                for (int32_t k = 0; k < L.V; ++k) {
                    const int64_t h = (at + k) / g.sh.D, d = (at + k) % g.sh.D;
                    if (k == 0 && !g.dense && scale_of_value(g, int64_t(tile) * L.block * L.V, tid * L.V) !=
                                                  h * g.sh.nb + d / kBlockValues)
                        flag(1);
                    double f = code_value(get8(codes, (y ? g.part : 0) + row * g.sh.run + at + k), a.format) *
                               scale_value(get8(scales, (y ? g.part_scales : 0) + row * g.sh.hl * g.sh.nb + h * g.sh.nb +
                                                            d / kBlockValues));
                    const double most = L.type == UA2A_TYPE_FP16 ? 65504.0
                                        : bits_f(L.type == UA2A_TYPE_FP32 ? 0x7f7fffffu : 0x7f7f0000u);
                    if (isfinite(f) && fabs(f) > most) f = f < 0 ? -most : most;
                    put(val, ri * span + at + k, static_cast<float>(f), L.type);
                }
            }
        }
    }
}

}  // namespace

namespace ua2a {

int act_launch(const ActLaunch& L, void*)
{
    ++g_launches;
    g_last = L;
    if (g_dry) return 0;
    switch (L.kernel) {
    case ActKernel::Norm: norm(L); break;
    case ActKernel::NormGrad: norm_grad(L); break;
    case ActKernel::Columns: columns(L); break;
    case ActKernel::CacheWrite: cache_write(L); break;
    case ActKernel::CacheRead: cache_read(L); break;
    }
    return 0;
}

int backend_current_device(int32_t* device)
{
    *device = 0;
    return 0;
}
int backend_launch(const Launch&, void*) { return -1; }
const char* backend_error_name(int) { return "emulated"; }
int backend_scratch_window(int32_t, uint8_t**) { return -1; }

}  // namespace ua2a

extern "C" {
int ua2a_act_emu_error() { return g_error; }
int ua2a_act_emu_launches() { return g_launches; }
void ua2a_act_emu_reset()
{
    g_error = 0;
    g_launches = 0;
}
void ua2a_act_emu_dry(int on) { g_dry = on; }
int ua2a_act_emu_last(int what)   // 0 V, 1 items, 2 block, 3 grid, 4 lanes, 5 grid along y,
                                  // 6 groups of segments, 7 span
{
    const NormGeom& g = g_last.kernel == ActKernel::NormGrad ? g_last.grad.g : g_last.norm.g;
    switch (what) {
    case 0: return g_last.V;
    case 1: return g_last.items;
    case 2: return static_cast<int>(g_last.block);
    case 3: return static_cast<int>(g_last.grid_x);
    case 5: return static_cast<int>(g_last.grid_y);
    case 6: return static_cast<int>(g.groups);
    case 7: return g_last.span;
    default: return static_cast<int>(g.lanes);
    }
}
}
