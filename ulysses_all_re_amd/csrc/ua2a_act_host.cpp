// Host side of the activation operators' C ABI (ua2a_act.h): argument checks,
// launch shapes and launches.  Like the exchange's calls, each validates every
// pointer and range before it launches, judges overlap by byte ranges, and
// disables the plan for good when a launch fails.
#include <math.h>
#include <stdio.h>
#include <string.h>

#include "ua2a_act_internal.h"

using namespace ua2a;

namespace {

constexpr int64_t kMaxSegments = int64_t(1) << 31;
constexpr int64_t kMaxPieces = (int64_t(1) << 31) - 1;                   // vectors of a cache call's tensor
constexpr int64_t kMaxCacheValues = int64_t(1) << 38;

struct Range {
    const void* p;
    int64_t bytes;
};

bool overlap(const Range& a, const Range& b)
{
    const uintptr_t pa = reinterpret_cast<uintptr_t>(a.p), pb = reinterpret_cast<uintptr_t>(b.p);
    return a.p != nullptr && b.p != nullptr && a.bytes > 0 && b.bytes > 0 &&
           pa < pb + static_cast<uintptr_t>(b.bytes) && pb < pa + static_cast<uintptr_t>(a.bytes);
}

// Whether an output overlaps another output or an input.
bool aliased(const Range* outs, int nouts, const Range* ins, int nins)
{
    for (int i = 0; i < nouts; ++i) {
        for (int k = i + 1; k < nouts; ++k)
            if (overlap(outs[i], outs[k])) return true;
        for (int k = 0; k < nins; ++k)
            if (overlap(outs[i], ins[k])) return true;
    }
    return false;
}

bool misaligned(const void* p, uintptr_t to) { return reinterpret_cast<uintptr_t>(p) % to != 0; }

int32_t type_bytes(int32_t type)
{
    return type == UA2A_TYPE_FP32 ? 4 : type == UA2A_TYPE_BF16 || type == UA2A_TYPE_FP16 ? 2 : 0;
}

bool good_format(int32_t f) { return f == UA2A_FORMAT_E4M3 || f == UA2A_FORMAT_E5M2; }

int fail(ua2a_plan_t plan, const char* what, int err)
{
    plan->disabled = 1;
    snprintf(plan->reason, sizeof plan->reason, "%s failed: %s", what, backend_error_name(err));
    return UA2A_ERR_HIP;
}

int check_device(ua2a_plan_t plan)
{
    int32_t dev = -1;
    const int err = backend_current_device(&dev);
    if (err != 0) return fail(plan, "querying the current device", err);
    return dev == plan->device ? UA2A_OK : UA2A_ERR_DEVICE;
}

int64_t tokens_of(const ua2a_plan_s* p) { return p->layout.tensor_elems / (p->H * p->D); }

ActShape shape_of(const ua2a_plan_s* p)
{
    ActShape g;
    g.H = static_cast<uint32_t>(p->H);
    g.D = static_cast<uint32_t>(p->D);
    g.nb = static_cast<uint32_t>((p->D + kBlockValues - 1) / kBlockValues);
    g.hl = static_cast<uint32_t>(p->H / p->w);
    g.S = static_cast<uint32_t>(p->S_local);
    g.B = static_cast<uint32_t>(p->B);
    g.SG = static_cast<uint32_t>(p->S_local * p->w);           // < 2^32 by the plan's limits
    g.d_hl = make_div32(g.hl);
    g.d_S = make_div32(g.S);
    g.d_B = make_div32(g.B);
    g.run = static_cast<uint32_t>(p->H / p->w * p->D);         // < 2^31 by the plan's limits
    g.d_run = make_div32(g.run);
    const int64_t rows = p->B * p->S_local * p->w;             // of one A rank
    g.a_rank = rows * g.hl * g.D;
    g.a_rank_scales = rows * g.hl * g.nb;
    return g;
}

uint32_t log2_of(uint32_t pow2)
{
    uint32_t l = 0;
    while ((1u << l) < pow2) ++l;
    return l;
}

// Segments, lanes and slots of a norm with V values per slot.
//
// One norm per segment: up to 64 slots get a lane each (the next power of
// two).  More: forward a workgroup to itself, of no more whole waves than it
// needs with one, two or four slots per lane, up to kActBlock lanes (measured:
// single precision, 288 slots, 82 us against 88 with 512 lanes; 640 slots 341
// against 339, and 489 with 640 lanes); backward the fewest of one, two or four
// waves with at most kActItems slots each.  Beyond them up to kActBigBlock lanes,
// backward with as few slots per lane as those allow (12,288 values from 8 bits:
// two slots on 768 lanes 205 us, four on 384 773).  The lanes of so wide a
// workgroup have 128 registers: eight slots, backward four too, spill (24,576
// values backward 768 us; 49,152 forward 273, four slots at 32,768 190).
//
// A norm per head of up to 64 slots (the next power of two): heads in
// bundles, which leaves all sums within a wave.  A bundle's lanes are the most
// of 64 whose heads divide H; its slots per lane one forward (video-DiT heads
// with a checkpoint: 313 us, with five 341), backward two where they divide the
// rest (360 us; one 365, five 390).
int norm_geometry(const ua2a_plan_s* p, int32_t per_head, int32_t V, bool backward, NormGeom* g, ActLaunch* L)
{
    g->sh = shape_of(p);
    const uint32_t q = kBlockValues / static_cast<uint32_t>(V);
    const int64_t head_slots = int64_t(g->sh.nb) * q;
    uint32_t lanes = 1, n = 1;
    int64_t slots = (per_head ? 1 : p->H) * head_slots;
    L->block = kActBlock;
    g->heads = per_head ? 1u : g->sh.H;
    g->head_log = 0;
    if (per_head && head_slots <= 64 && V > 1) {
        uint32_t hq = 1;
        while (hq < head_slots) hq *= 2;
        lanes = 64;
        while (g->sh.H % (lanes / hq) != 0) lanes /= 2;        // lanes == hq divides at the latest
        n = backward && (g->sh.H / (lanes / hq)) % 2 == 0 ? 2 : 1;     // lanes < 64 leave an odd number
        L->span = lanes == 64 ? kSpanBundle : kSpanBundles;
        g->heads = lanes / hq * n;
        g->head_log = log2_of(hq);
        slots = int64_t(g->heads) * hq;
        g->padded = (p->D % kBlockValues != 0 || hq != head_slots) ? 1u : 0u;
    } else {
        if (slots > int64_t(kActBigBlock) * kActBigItems) return UA2A_ERR_SHAPE;
        if (slots <= 64) {
            while (lanes < slots) lanes *= 2;
            L->span = kSpanPart;
        } else if (backward && V > 1 && slots <= int64_t(kActBlock) * kActItems) {
            lanes = 64;
            while (lanes * kActItems < slots) lanes *= 2;
            n = static_cast<uint32_t>((slots + lanes - 1) / lanes);
            L->span = kSpanWaves;
        } else {
            while (!backward && kActBlock * n < slots && n < 4) n *= 2;
            while (kActBigBlock * n < slots) n *= 2;            // 1, 2, 4 or 8
            lanes = static_cast<uint32_t>((slots + n - 1) / n + 63) / 64 * 64;
            L->block = lanes;
            L->span = kSpanWide;
        }
        g->padded = (p->D % kBlockValues != 0 || int64_t(lanes) * n != slots) ? 1u : 0u;
    }
    g->dense = (p->D % kBlockValues == 0 && g->head_log == 0) ? 1u : 0u;
    g->per_token = g->sh.H / g->heads;
    const int64_t segs = tokens_of(p) * g->per_token;
    if (tokens_of(p) * (per_head ? p->H : 1) >= kMaxSegments) return UA2A_ERR_SHAPE;
    L->items = static_cast<int32_t>(n);
    g->cols = static_cast<uint32_t>((per_head ? 1 : p->H) * p->D);
    g->slots = static_cast<uint32_t>(slots);
    g->q_log = log2_of(q);
    g->lanes = lanes;
    g->per_log = log2_of(L->block / lanes);
    g->segs = static_cast<uint32_t>(segs);
    g->groups = static_cast<uint32_t>((segs + (int64_t(1) << g->per_log) - 1) >> g->per_log);
    g->d_nb = make_div32(g->sh.nb);
    g->d_per = make_div32(g->per_token);
    return UA2A_OK;
}

// Most workgroups of a backward launch, each walking over segments: about as many
// as the device holds at once of the kernels with 2-byte values and weights (they
// keep sums in registers, so fewer fit as the slots per lane grow).  A grid that
// is no multiple of what is resident leaves part of the device idle at the end:
// video-DiT with five slots per lane 354 us with 512 workgroups, 451 with 768,
// 377 with 1024.  The rule sees slots only.  Of the kernels with a weight in
// single precision 256 workgroups of five slots are resident, 512 of three: two
// rounds, and one and a half (video-DiT 514 us, 359 with the weight in bf16).  Of
// those with single-precision values more would fit (four slots 768, two 1280),
// and of kSpanWide workgroups past 512 lanes one per CU.
uint32_t grad_grid(int32_t span, int32_t items)
{
    if (span == kSpanWide) return 512;
    return items >= 4 ? 512 : items == 3 ? 768 : 1024;
}

uint32_t least(uint32_t a, uint32_t b) { return a < b ? a : b; }

// What every call checks first.
int check_plan(ua2a_plan_t plan, int32_t type)
{
    if (plan == nullptr) return UA2A_ERR_INVALID_ARG;
    if (plan->disabled) return UA2A_ERR_DISABLED;
    if (type_bytes(type) == 0 || type_bytes(type) != plan->elem_bytes) return UA2A_ERR_INVALID_ARG;
    return UA2A_OK;
}

int check_cache(ua2a_plan_t plan, const ua2a_cache_t* c, int64_t* values, int64_t* scales)
{
    if (c == nullptr || c->codes == nullptr || c->scales == nullptr || !good_format(c->format))
        return UA2A_ERR_INVALID_ARG;
    if (c->sequences < 1 || c->capacity < 1 || c->capacity > INT32_MAX || c->sequences > INT32_MAX)
        return UA2A_ERR_SHAPE;
    const int64_t row = plan->H * plan->D;                     // one position on all ranks
    if (c->sequences > kMaxCacheValues / c->capacity || c->sequences * c->capacity > kMaxCacheValues / (2 * row))
        return UA2A_ERR_SHAPE;
    const int64_t nb = (plan->D + kBlockValues - 1) / kBlockValues;
    *values = 2 * c->sequences * c->capacity * row;
    *scales = 2 * c->sequences * c->capacity * plan->H * nb;
    return UA2A_OK;
}

void cache_geometry(ua2a_plan_t plan, const ua2a_cache_t* c, int32_t V, int64_t each, CacheGeom* g)
{
    g->sh = shape_of(plan);
    g->seqs = static_cast<uint32_t>(c->sequences);
    g->each = static_cast<uint32_t>(each);
    g->dense = plan->D % kBlockValues == 0 ? 1u : 0u;
    g->q_log = log2_of(kBlockValues / static_cast<uint32_t>(V));
    g->cap = c->capacity;
    g->part = c->sequences * c->capacity * plan->H * plan->D;
    g->part_scales = c->sequences * c->capacity * plan->H * g->sh.nb;
    g->d_nb = make_div32(g->sh.nb);
    g->d_each = make_div32(g->each);
    g->d_D = make_div32(g->sh.D);
    g->d_seqs = make_div32(g->seqs);
}

// `wgs` workgroups, within what a dispatch counts along x (cache_workgroup takes
// the two parts together again).
void cache_grid(int64_t wgs, ActLaunch* L)
{
    const int64_t along = int64_t(1) << kCacheGridLog;
    L->grid_x = static_cast<uint32_t>(wgs < along ? wgs : along);
    L->grid_y = static_cast<uint32_t>((wgs + along - 1) >> kCacheGridLog);
}

}  // namespace

extern "C" {

int ua2a_norm_exchange(ua2a_plan_t plan, int32_t mode, const ua2a_norm_t* n, void* stream)
{
    if (n == nullptr) return UA2A_ERR_INVALID_ARG;
    int rc = check_plan(plan, n->type);
    if (rc != UA2A_OK) return rc;
    if ((mode != 0 && mode != 1) || (n->per_head != 0 && n->per_head != 1)) return UA2A_ERR_INVALID_ARG;
    if (n->x == nullptr || n->out == nullptr || (n->residual == nullptr) != (n->sum == nullptr))
        return UA2A_ERR_INVALID_ARG;
    if (!(n->eps > 0.f) || isinf(n->eps)) return UA2A_ERR_INVALID_ARG;
    if (n->weight != nullptr && n->weight_type != n->type && n->weight_type != UA2A_TYPE_FP32)
        return UA2A_ERR_INVALID_ARG;
    if (n->out_format != UA2A_FORMAT_NONE && !good_format(n->out_format)) return UA2A_ERR_INVALID_ARG;
    if (n->saved_format != UA2A_FORMAT_NONE && !good_format(n->saved_format)) return UA2A_ERR_INVALID_ARG;
    if ((n->out_format != UA2A_FORMAT_NONE) != (n->out_scales != nullptr)) return UA2A_ERR_INVALID_ARG;
    if ((n->saved_format != UA2A_FORMAT_NONE) != (n->saved != nullptr) || (n->saved == nullptr) != (n->saved_scales == nullptr))
        return UA2A_ERR_INVALID_ARG;

    const uintptr_t e = static_cast<uintptr_t>(plan->elem_bytes);
    const int32_t wbytes = type_bytes(n->weight_type);
    if (misaligned(n->x, e) || misaligned(n->residual, e) || misaligned(n->sum, e) ||
        (!n->out_format && misaligned(n->out, e)) ||
        (n->weight != nullptr && misaligned(n->weight, static_cast<uintptr_t>(wbytes))) || misaligned(n->rstd, 4))
        return UA2A_ERR_ALIGN;
    const bool wide = (plan->D * plan->elem_bytes) % 16 == 0 && !misaligned(n->x, 16) && !misaligned(n->residual, 16) &&
                      !misaligned(n->sum, 16) && !misaligned(n->saved, 8) &&
                      !misaligned(n->out, n->out_format ? 8 : 16);
    ActLaunch L;
    memset(&L, 0, sizeof L);
    L.kernel = ActKernel::Norm;
    L.type = n->type;
    L.V = wide ? 16 / plan->elem_bytes : 1;
    NormArgs& a = L.norm;
    rc = norm_geometry(plan, n->per_head, L.V, false, &a.g, &L);
    if (rc != UA2A_OK) return rc;

    const int64_t values = plan->layout.tensor_elems, bytes = plan->layout.tensor_bytes;
    const int64_t nscales = tokens_of(plan) * plan->H * a.g.sh.nb;
    const int64_t nstats = tokens_of(plan) * (n->per_head ? plan->H : 1);
    const Range ins[] = {{n->x, bytes}, {n->residual, bytes},
                         {n->weight, n->weight != nullptr ? int64_t(a.g.cols) * wbytes : 0}};
    const Range outs[] = {{n->out, n->out_format ? values : bytes}, {n->out_scales, nscales}, {n->sum, bytes},
                          {n->saved, values}, {n->saved_scales, nscales}, {n->rstd, nstats * 4}};
    if (aliased(outs, 6, ins, 3)) return UA2A_ERR_ALIAS;
    rc = check_device(plan);
    if (rc != UA2A_OK) return rc;

    a.x = n->x;
    a.residual = n->residual;
    a.weight = n->weight;
    a.out = n->out;
    a.out_scales = static_cast<uint8_t*>(n->out_scales);
    a.sum = n->sum;
    a.saved = static_cast<uint8_t*>(n->saved);
    a.saved_scales = static_cast<uint8_t*>(n->saved_scales);
    a.rstd = n->rstd;
    a.eps = n->eps;
    a.inv_len = 1.f / static_cast<float>(a.g.cols);
    a.weight_f32 = n->weight_type == UA2A_TYPE_FP32 ? 1 : 0;
    a.flags = (mode == 1 ? kNormMode1 : 0) | (n->weight != nullptr ? kNormWeight : 0) |
              (n->residual != nullptr ? kNormResidual : 0) | (n->rstd != nullptr ? kNormRstd : 0) |
              (n->out_format ? kNormOut8 : 0) | (n->out_format == UA2A_FORMAT_E5M2 ? kNormOutE5M2 : 0) |
              (n->saved_format ? kNormSaved8 : 0) | (n->saved_format == UA2A_FORMAT_E5M2 ? kNormSavedE5M2 : 0);
    // one workgroup per group of segments, within what a dispatch counts along x
    L.grid_x = least(a.g.groups, static_cast<uint32_t>(kMaxGridWorkItems / L.block));
    L.grid_y = (a.g.groups + L.grid_x - 1) / L.grid_x;
    const int err = act_launch(L, stream);
    return err == 0 ? UA2A_OK : fail(plan, "launching the norm kernel", err);
}

int ua2a_norm_workspace(ua2a_plan_t plan, int32_t per_head, int64_t* bytes)
{
    if (plan == nullptr || bytes == nullptr || (per_head != 0 && per_head != 1)) return UA2A_ERR_INVALID_ARG;
    // the wide vectors and single values lie differently on the lanes: room for either
    *bytes = 0;
    int found = UA2A_ERR_SHAPE;
    for (const int32_t V : {16 / plan->elem_bytes, 1}) {
        NormGeom g;
        ActLaunch L;
        if (V > 16 / 2 || norm_geometry(plan, per_head, V, true, &g, &L) != UA2A_OK) continue;
        const int64_t need = int64_t(least(g.groups, grad_grid(L.span, L.items))) * g.cols * 4;
        if (need > *bytes) *bytes = need;
        found = UA2A_OK;
    }
    return found;
}

int ua2a_norm_exchange_backward(ua2a_plan_t plan, int32_t mode, const ua2a_norm_grad_t* n, void* stream)
{
    if (n == nullptr) return UA2A_ERR_INVALID_ARG;
    int rc = check_plan(plan, n->type);
    if (rc != UA2A_OK) return rc;
    if ((mode != 0 && mode != 1) || (n->per_head != 0 && n->per_head != 1)) return UA2A_ERR_INVALID_ARG;
    if (n->dy == nullptr || n->saved == nullptr || n->rstd == nullptr || n->dx == nullptr) return UA2A_ERR_INVALID_ARG;
    if (n->weight != nullptr && n->weight_type != n->type && n->weight_type != UA2A_TYPE_FP32)
        return UA2A_ERR_INVALID_ARG;
    if (n->saved_format != UA2A_FORMAT_NONE && !good_format(n->saved_format)) return UA2A_ERR_INVALID_ARG;
    if ((n->saved_format != UA2A_FORMAT_NONE) != (n->saved_scales != nullptr)) return UA2A_ERR_INVALID_ARG;
    if (n->saved_gathered != 0 && (n->saved_gathered != 1 || mode != 1 || n->saved_format != UA2A_FORMAT_NONE))
        return UA2A_ERR_INVALID_ARG;
    if ((n->dresidual != nullptr && mode != 1) || (n->dweight != nullptr && n->workspace == nullptr) ||
        n->workspace_bytes < 0)
        return UA2A_ERR_INVALID_ARG;

    const uintptr_t e = static_cast<uintptr_t>(plan->elem_bytes);
    const int32_t wbytes = type_bytes(n->weight_type);
    if (misaligned(n->dy, e) || misaligned(n->dsum, e) || misaligned(n->dx, e) || misaligned(n->dresidual, e) ||
        (!n->saved_format && misaligned(n->saved, e)) ||
        (n->weight != nullptr && misaligned(n->weight, static_cast<uintptr_t>(wbytes))) || misaligned(n->rstd, 4) ||
        misaligned(n->dweight, 4) || misaligned(n->workspace, 16))
        return UA2A_ERR_ALIGN;
    const bool wide = (plan->D * plan->elem_bytes) % 16 == 0 && !misaligned(n->dy, 16) && !misaligned(n->dsum, 16) &&
                      !misaligned(n->dx, 16) && !misaligned(n->dresidual, 16) &&
                      !misaligned(n->saved, n->saved_format ? 8 : 16);
    ActLaunch L;
    memset(&L, 0, sizeof L);
    L.kernel = ActKernel::NormGrad;
    L.type = n->type;
    L.V = wide ? 16 / plan->elem_bytes : 1;
    NormGradArgs& a = L.grad;
    rc = norm_geometry(plan, n->per_head, L.V, true, &a.g, &L);
    if (rc != UA2A_OK) return rc;
    L.grid_x = least(a.g.groups, grad_grid(L.span, L.items));
    L.grid_y = 1;

    const int64_t values = plan->layout.tensor_elems, bytes = plan->layout.tensor_bytes;
    const int64_t nscales = tokens_of(plan) * plan->H * a.g.sh.nb;
    const int64_t nstats = tokens_of(plan) * (n->per_head ? plan->H : 1);
    const int64_t wspace = n->dweight != nullptr ? int64_t(L.grid_x) * a.g.cols * 4 : 0;
    if (n->workspace_bytes < wspace) return UA2A_ERR_CAPACITY;
    const Range ins[] = {{n->dy, bytes}, {n->dsum, bytes}, {n->saved, n->saved_format ? values : bytes},
                         {n->saved_scales, nscales}, {n->rstd, nstats * 4},
                         {n->weight, n->weight != nullptr ? int64_t(a.g.cols) * wbytes : 0}};
    const Range outs[] = {{n->dx, bytes}, {n->dresidual, bytes}, {n->dweight, int64_t(a.g.cols) * 4},
                          {n->workspace, wspace}};
    if (aliased(outs, 4, ins, 6)) return UA2A_ERR_ALIAS;
    rc = check_device(plan);
    if (rc != UA2A_OK) return rc;

    a.dy = n->dy;
    a.dsum = n->dsum;
    a.saved = n->saved;
    a.saved_scales = static_cast<const uint8_t*>(n->saved_scales);
    a.weight = n->weight;
    a.rstd = n->rstd;
    a.dx = n->dx;
    a.dresidual = n->dresidual;
    a.partial = n->dweight != nullptr ? static_cast<float*>(n->workspace) : nullptr;
    a.inv_len = 1.f / static_cast<float>(a.g.cols);
    a.weight_f32 = n->weight_type == UA2A_TYPE_FP32 ? 1 : 0;
    a.saved_format = n->saved_format;
    a.flags = (mode == 1 ? kNormMode1 : 0) | (n->weight != nullptr ? kNormWeight : 0) |
              (n->dsum != nullptr ? kNormResidual : 0) | (n->dweight != nullptr ? kNormPartial : 0) |
              (n->dresidual != nullptr ? kNormApart : 0) | (n->saved_gathered ? kNormGathered : 0);
    int err = act_launch(L, stream);
    if (err != 0) return fail(plan, "launching the norm's backward kernel", err);
    if (n->dweight == nullptr) return UA2A_OK;
    const uint32_t rows = L.grid_x, cols = a.g.cols;
    L.kernel = ActKernel::Columns;
    L.columns.partial = static_cast<const float*>(n->workspace);
    L.columns.out = n->dweight;
    L.columns.rows = rows;
    L.columns.cols = cols;
    L.columns.across_log = cols >= 1024 ? 5 : 3;                // lines of 128 bytes, or of 32
    L.block = 1024;
    L.grid_x = (cols + (1u << L.columns.across_log) - 1) >> L.columns.across_log;
    err = act_launch(L, stream);
    return err == 0 ? UA2A_OK : fail(plan, "launching the weight gradient's sum", err);
}

int ua2a_cache_write(ua2a_plan_t plan, const ua2a_cache_t* c, int32_t type, const void* k, const void* v,
                     const int32_t* starts, const int32_t* counts, void* stream)
{
    int rc = check_plan(plan, type);
    if (rc != UA2A_OK) return rc;
    int64_t values, nscales;
    rc = check_cache(plan, c, &values, &nscales);
    if (rc != UA2A_OK) return rc;
    if ((k == nullptr && v == nullptr) || starts == nullptr) return UA2A_ERR_INVALID_ARG;
    const int64_t gathered = plan->B * plan->S_local * plan->w;
    if (gathered % c->sequences != 0) return UA2A_ERR_SHAPE;
    const uintptr_t e = static_cast<uintptr_t>(plan->elem_bytes);
    if (misaligned(k, e) || misaligned(v, e) || misaligned(starts, 4) || misaligned(counts, 4)) return UA2A_ERR_ALIGN;
    const bool wide = (plan->D * plan->elem_bytes) % 16 == 0 && !misaligned(k, 16) && !misaligned(v, 16) &&
                      !misaligned(c->codes, 8);
    ActLaunch L;
    memset(&L, 0, sizeof L);
    L.kernel = ActKernel::CacheWrite;
    L.type = type;
    L.V = wide ? 16 / plan->elem_bytes : 1;
    CacheArgs& a = L.cache;
    cache_geometry(plan, c, L.V, gathered / c->sequences, &a.g);
    CacheGeom& g = a.g;
    const int64_t row = plan->H * g.sh.nb * (kBlockValues / L.V);
    if (row > kMaxPieces / gathered) return UA2A_ERR_SHAPE;
    g.rows = static_cast<uint32_t>(gathered);
    g.slots = static_cast<uint32_t>(row);
    g.lanes = 1;
    while (g.lanes < kActBlock && g.lanes < g.slots) g.lanes *= 2;
    g.chunks = (g.slots + g.lanes - 1) / g.lanes;
    g.d_chunks = make_div32(g.chunks);
    g.per_log = log2_of(kActBlock / g.lanes);
    const int64_t groups = ((gathered * g.chunks) + (int64_t(1) << g.per_log) - 1) >> g.per_log;
    // as many groups in a row to an XCD as fill lines of a rank's scales
    g.run_log = 0;
    while (g.run_log < 6 && (int64_t(g.sh.hl) * g.sh.nb << (g.run_log + g.per_log)) < kLineBytes * g.chunks) ++g.run_log;
    const int64_t turn = int64_t(kCacheXcds) << g.run_log;
    const int64_t wgs = (groups + turn - 1) / turn * turn;     // below 2^25: the lanes are less than twice the pieces
    g.groups = static_cast<uint32_t>(groups);
    const int64_t bytes = plan->layout.tensor_bytes;
    const Range ins[] = {{k, bytes}, {v, bytes}, {starts, c->sequences * 4}, {counts, c->sequences * 4}};
    const Range outs[] = {{c->codes, values}, {c->scales, nscales}};
    if (aliased(outs, 2, ins, 4)) return UA2A_ERR_ALIAS;
    rc = check_device(plan);
    if (rc != UA2A_OK) return rc;
    a.k = k;
    a.v = v;
    a.codes = static_cast<uint8_t*>(c->codes);
    a.scales = static_cast<uint8_t*>(c->scales);
    a.starts = starts;
    a.counts = counts;
    a.format = c->format;
    L.block = kActBlock;
    cache_grid(wgs, &L);
    const int err = act_launch(L, stream);
    return err == 0 ? UA2A_OK : fail(plan, "launching the cache write", err);
}

int ua2a_cache_read(ua2a_plan_t plan, const ua2a_cache_t* c, int32_t type, int64_t n, const int32_t* starts,
                    const int32_t* counts, void* k_out, void* v_out, void* stream)
{
    int rc = check_plan(plan, type);
    if (rc != UA2A_OK) return rc;
    int64_t values, nscales;
    rc = check_cache(plan, c, &values, &nscales);
    if (rc != UA2A_OK) return rc;
    if (k_out == nullptr && v_out == nullptr) return UA2A_ERR_INVALID_ARG;
    if (n < 1 || n > INT32_MAX) return UA2A_ERR_SHAPE;
    const uintptr_t e = static_cast<uintptr_t>(plan->elem_bytes);
    if (misaligned(k_out, e) || misaligned(v_out, e) || misaligned(starts, 4) || misaligned(counts, 4))
        return UA2A_ERR_ALIGN;
    const bool wide = (plan->D * plan->elem_bytes) % 16 == 0 && !misaligned(k_out, 16) && !misaligned(v_out, 16) &&
                      !misaligned(c->codes, 8);
    ActLaunch L;
    memset(&L, 0, sizeof L);
    L.kernel = ActKernel::CacheRead;
    L.type = type;
    L.V = wide ? 16 / plan->elem_bytes : 1;
    CacheArgs& a = L.cache;
    cache_geometry(plan, c, L.V, n, &a.g);
    CacheGeom& g = a.g;
    const int64_t spans = c->sequences * plan->w, each = g.sh.run / static_cast<uint32_t>(L.V);
    if (n > kMaxPieces / each || spans > kMaxPieces / (n * each)) return UA2A_ERR_SHAPE;
    // a span's vectors, on whole waves of up to kActBlock lanes
    const int64_t rows = spans * n, vectors = n * each;
    L.block = vectors >= kActBlock ? kActBlock : static_cast<uint32_t>((vectors + 63) / 64 * 64);
    const int64_t tiles = (vectors + L.block - 1) / L.block;
    g.spans = static_cast<uint32_t>(spans);
    g.tiles = static_cast<uint32_t>(tiles);
    g.d_tiles = make_div32(g.tiles);
    const int64_t bytes = rows * a.g.sh.hl * plan->D * plan->elem_bytes;
    const Range ins[] = {{c->codes, values}, {c->scales, nscales}, {starts, c->sequences * 4},
                         {counts, c->sequences * 4}};
    const Range outs[] = {{k_out, bytes}, {v_out, bytes}};
    if (aliased(outs, 2, ins, 4)) return UA2A_ERR_ALIAS;
    rc = check_device(plan);
    if (rc != UA2A_OK) return rc;
    a.k_out = k_out;
    a.v_out = v_out;
    a.codes = static_cast<uint8_t*>(c->codes);
    a.scales = static_cast<uint8_t*>(c->scales);
    a.starts = starts;
    a.counts = counts;
    a.format = c->format;
    cache_grid(spans * tiles, &L);                             // no more workgroups than pieces
    const int err = act_launch(L, stream);
    return err == 0 ? UA2A_OK : fail(plan, "launching the cache read", err);
}

}  // extern "C"
