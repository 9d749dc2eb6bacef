// Host side of the attention operators' C ABI (ua2a_attn.h): argument checks,
// launch shapes and launches, as for the activation operators: every pointer
// and range is validated before anything is launched, overlap is judged by byte
// ranges, and a launch that fails disables the plan for good.
#include <math.h>
#include <string.h>

#include "ua2a_act_checks.h"
#include "ua2a_attn_internal.h"

using namespace ua2a;

namespace {

constexpr int64_t kMost32 = (int64_t(1) << 31) - 1;
constexpr int64_t kMostRow = int64_t(1) << 22;               // values of a position on one rank
constexpr int64_t kMostValues = int64_t(1) << 38;            // of a tensor or a cache

// `wgs` workgroups, within what a dispatch counts along x.
void attn_grid(int64_t wgs, AttnLaunch* L)
{
    const int64_t along = int64_t(1) << kAttnGridLog;
    L->grid_x = static_cast<uint32_t>(wgs < along ? wgs : along);
    L->grid_y = static_cast<uint32_t>((wgs + along - 1) >> kAttnGridLog);
}

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

int check_attention(ua2a_plan_t plan, int32_t type, const ua2a_window_t& w)
{
    const int rc = check_plan(plan, type);
    if (rc != UA2A_OK) return rc;
    if (type == UA2A_TYPE_FP32) return UA2A_ERR_INVALID_ARG;
    if (w.left < -1 || w.right < -1 || w.sinks < 0 || w.chunk < 1 || w.left > kMost32 || w.right > kMost32 ||
        w.sinks > kMost32 || w.chunk > kMost32)
        return UA2A_ERR_INVALID_ARG;
    return UA2A_OK;
}

// Also in powers of two, as the kernels have it.
bool good_scale(float s) { return s > 0.f && !isinf(s * kLog2e); }

// The shapes of a call of n queries for each of `seqs` sequences a rank over
// `keys` positions; tiles, splits and items are left to the caller.
int attn_geometry(const ua2a_plan_s* p, const ua2a_window_t& w, int64_t kv_heads, int64_t seqs, int64_t n, int64_t keys,
                  AttnGeom* g)
{
    if (p->D % 8 != 0 || p->D > 128 || kv_heads < 1 || kv_heads % p->w != 0 || p->H % kv_heads != 0 ||
        p->H / p->w * p->D > kMostRow || n < 1 || keys > kMost32)
        return UA2A_ERR_SHAPE;
    const int64_t hl = p->H / p->w, ranks = p->w * seqs;
    if (n > kMost32 / hl || ranks > kMost32 / (n * hl) || keys > kMostValues / (hl * p->D) ||
        ranks > kMostValues / (keys * hl * p->D))
        return UA2A_ERR_SHAPE;
    memset(g, 0, sizeof *g);
    g->win.left = static_cast<int32_t>(w.left);
    g->win.right = static_cast<int32_t>(w.right);
    g->win.sinks = static_cast<int32_t>(w.sinks);
    g->win.chunk = static_cast<uint32_t>(w.chunk);
    g->win.d_chunk = make_div32(g->win.chunk);
    g->hl = static_cast<uint32_t>(hl);
    g->kvl = static_cast<uint32_t>(kv_heads / p->w);
    g->group = g->hl / g->kvl;
    g->units = static_cast<uint32_t>(ranks * g->kvl);
    g->seqs = static_cast<uint32_t>(seqs);
    g->D = static_cast<uint32_t>(p->D);
    g->nb = static_cast<uint32_t>(ceil_div(p->D, kBlockValues));
    g->n = static_cast<uint32_t>(n);
    g->rows = static_cast<uint32_t>(n * g->group);
    g->keys = static_cast<uint32_t>(keys);
    g->d_kvl = make_div32(g->kvl);
    g->d_seqs = make_div32(g->seqs);
    g->d_group = make_div32(g->group);
    g->d_rows = make_div32(g->rows);
    return UA2A_OK;
}

// Most positions that `rows` consecutive rows see between them.
int64_t most_seen(const AttnGeom& g, int64_t rows)
{
    if (g.win.left < 0 || g.win.right < 0) return g.keys;
    const int64_t tokens = ceil_div(rows, g.group) + 1;
    const int64_t chunk = g.win.chunk, chunks = int64_t(g.win.left) + g.win.right + 1;
    if (chunks > g.keys / chunk) return g.keys;
    const int64_t seen = chunks * chunk + (chunk > 1 ? chunk : 0) + tokens + g.win.sinks;
    return seen < g.keys ? seen : g.keys;
}

// Whether walks grow from tile to tile: of rows where the left reaches further than
// the right, of keys the other way round.  They then run from the last tile to the
// first, so that what ends last is short: 32 heads of 128 over 8192 tokens, causal,
// 612 us, 684 from the first (heads of 64 369, 420), 8 over 32,768 2150, 2550, backward
// 8110, 8800; a window of 1024 of 6124 tokens 148, 154; long and short walks in turn 8 %
// slower than from the first.
uint32_t order_of(const AttnGeom& g, bool keys)
{
    const int64_t left = g.win.left < 0 ? kMost32 + 1 : g.win.left, right = g.win.right < 0 ? kMost32 + 1 : g.win.right;
    return keys ? right > left : right < left;
}

void set_items(AttnGeom* g, int64_t tiles, int64_t splits)
{
    g->tiles = static_cast<uint32_t>(tiles);
    g->splits = static_cast<uint32_t>(splits);
    g->items = static_cast<uint32_t>(int64_t(g->units) * tiles * splits);
    g->d_tiles = make_div32(g->tiles);
    g->d_splits = make_div32(g->splits);
}

int64_t workgroups(const AttnGeom& g) { return ceil_div(g.items, kAttnXcds) * kAttnXcds; }

int32_t padded_head(int64_t D) { return static_cast<int32_t>(ceil_div(D, 32) * 32); }

// How a forward call's rows and keys go to workgroups.  Up to 32 rows of a key
// head lie in one tile, whose keys the waves share out.  With fewer workgroups
// than the device holds at once (two a CU), a tile's keys are split among
// several, each with four tiles of keys at least.
void forward_shape(AttnGeom* g, AttnLaunch* L)
{
    L->shared = g->rows <= kAttnWaveRows ? 1 : 0;
    const int64_t per = L->shared ? kAttnWaveRows : kAttnRows, size = L->shared ? kAttnSplitKeys : kAttnKeys;
    const int64_t tiles = ceil_div(g->rows, per), all = int64_t(g->units) * tiles;
    int64_t splits = 1;
    if (all < 512) {
        splits = 512 / all;
        const int64_t most = most_seen(*g, per) / (4 * size);
        if (splits > most) splits = most;
        if (splits < 1) splits = 1;
    }
    set_items(g, tiles, splits);
    g->order = order_of(*g, false);
    L->DP = padded_head(g->D);
    L->block = kAttnBlock;
}

int64_t forward_workspace(const AttnGeom& g)
{
    if (g.splits == 1) return 0;
    const int64_t lines = int64_t(g.splits) * g.units * g.rows;
    return ceil_div(lines * (g.D + 2) * 4, 16) * 16;
}

int launch_forward(ua2a_plan_t plan, AttnLaunch* L, void* workspace, void* stream)
{
    const AttnGeom& g = L->attn.g;
    if (g.splits > 1) {
        L->attn.partial = static_cast<float*>(workspace);
        L->attn.stats = L->attn.partial + int64_t(g.splits) * g.units * g.rows * g.D;
    }
    // up to 16 rows of a cache have a kernel of their own
    L->kernel = L->attn.codes != nullptr && g.rows <= kDecodeRows ? AttnKernel::Decode : AttnKernel::Forward;
    attn_grid(workgroups(g), L);
    int err = attn_launch(*L, stream);
    if (err != 0) return fail(plan, "launching the attention kernel", err);
    if (g.splits == 1) return UA2A_OK;
    L->kernel = AttnKernel::Join;
    attn_grid(ceil_div(int64_t(g.units) * g.rows, join_shape(g).rows), L);
    err = attn_launch(*L, stream);
    return err == 0 ? UA2A_OK : fail(plan, "launching the join of attention's parts", err);
}

int plan_attention(ua2a_plan_t plan, const ua2a_attention_t* n, AttnLaunch* L)
{
    if (n == nullptr) return UA2A_ERR_INVALID_ARG;
    int rc = check_attention(plan, n->type, n->window);
    if (rc != UA2A_OK) return rc;
    const int64_t SG = plan->S_local * plan->w;
    memset(L, 0, sizeof *L);
    L->type = n->type;
    rc = attn_geometry(plan, n->window, n->kv_heads, plan->B, SG, SG, &L->attn.g);
    if (rc == UA2A_OK) forward_shape(&L->attn.g, L);
    return rc;
}

int plan_cache(ua2a_plan_t plan, const ua2a_cache_t* c, const ua2a_cache_attention_t* n, AttnLaunch* L)
{
    if (c == nullptr || n == nullptr || !good_format(c->format)) return UA2A_ERR_INVALID_ARG;
    int rc = check_attention(plan, n->type, n->window);
    if (rc != UA2A_OK) return rc;
    if (c->sequences < 1 || c->capacity < 1 || c->sequences > kMost32 || n->n > kMost32) return UA2A_ERR_SHAPE;
    memset(L, 0, sizeof *L);
    L->type = n->type;
    rc = attn_geometry(plan, n->window, n->kv_heads, c->sequences, n->n, c->capacity, &L->attn.g);
    if (rc == UA2A_OK) forward_shape(&L->attn.g, L);
    return rc;
}

// Most rows that see one of a tile's keys, sinks apart.
int64_t most_seers(const AttnGeom& g)
{
    if (g.win.left < 0 || g.win.right < 0) return g.rows;
    const int64_t chunk = g.win.chunk, chunks = int64_t(g.win.left) + g.win.right + 1;
    if (chunks > g.keys / chunk) return g.rows;
    const int64_t tokens = chunks * chunk + (chunk > 1 ? chunk : 0) + kAttnGradKeys;
    return tokens < g.n ? tokens * g.group : g.rows;
}

// The sizes of tiles of rows, whole lines of 16 bytes
int64_t size_floats(const AttnGeom& g) { return ceil_div(int64_t(g.units) * ceil_div(g.rows, kAttnRows) * 2, 4) * 4; }

// How the keys' gradients go to workgroups.  Sinks are seen by all rows, other
// keys by a window of them, so a tile of sinks would be walked long after the
// rest: tiles are walked in parts of about a window, and of less where the call
// is small: as much as leaves two parts for each workgroup that the device holds
// at once (512), but 512 rows at least, for a part's sums go through the
// workspace (no more than 64 parts of a tile, and 256 MiB).  A
// call of eight units of 6,124 keys at most, four rows a key, heads of 64, took
// 231-258 us, with one part for each workgroup 245-266 (the same lengths).
void backward_shape(AttnGradArgs* a)
{
    AttnGeom& g = a->g;
    KeyTiles& t = a->keys;
    const int64_t tiles = ceil_div(g.keys, kAttnGradKeys), most = most_seers(g);
    const int64_t sinks = g.win.sinks < static_cast<int64_t>(g.keys) ? g.win.sinks : g.keys;
    const int64_t lead = most < g.rows ? ceil_div(sinks, kAttnGradKeys) : 0;
    const int64_t span = lead * kAttnGradKeys < g.keys ? lead * kAttnGradKeys : g.keys;
    const int64_t all = g.units * (lead * g.rows + (tiles - lead) * most);
    int64_t part = all / 1024 < most ? all / 1024 : most;
    if (part < 512) part = 512;
    int64_t first, rest;
    for (;; part *= 2) {
        first = (g.rows + part / 2) / part;                      // the nearest
        rest = (most + part / 2) / part;
        first = lead == 0 || first < 1 ? 1 : first > 64 ? 64 : first;
        rest = rest < 1 ? 1 : rest > 64 ? 64 : rest;
        const int64_t lines = (first > 1 ? first * span : 0) + (rest > 1 ? rest * (g.keys - span) : 0);
        if (lines == 0 || lines * g.units * g.D * 8 + size_floats(g) * 4 <= (int64_t(256) << 20)) break;
    }
    set_items(&g, tiles, 1);
    g.order = order_of(g, true);
    t.lead = static_cast<uint32_t>(lead);
    t.span = static_cast<uint32_t>(span);
    t.lead_parts = static_cast<uint32_t>(first);
    t.rest_parts = static_cast<uint32_t>(rest);
    t.per_unit = static_cast<uint32_t>(lead * first + (tiles - lead) * rest);
    t.d_per_unit = make_div32(t.per_unit);
    t.d_lead_parts = make_div32(t.lead_parts);
    t.d_rest_parts = make_div32(t.rest_parts);
    t.per_group = kAttnBlock / (g.D / 2);
    t.d_lanes = make_div32(g.D / 2);
    t.d_keys = make_div32(t.rest_parts > 1 || t.span == 0 ? g.keys : t.span);
    t.rest_line = first > 1 ? first * g.units * span : 0;
    g.items = g.units * t.per_unit;
}

int64_t part_lines(const AttnGradArgs& a)
{
    const KeyTiles& t = a.keys;
    return t.rest_line + (t.rest_parts > 1 ? int64_t(t.rest_parts) * a.g.units * (a.g.keys - t.span) : 0);
}

// delta's place, whole lines of 16 bytes
int64_t delta_floats(const AttnGeom& g) { return ceil_div(int64_t(g.units) * g.rows, 4) * 4; }

int64_t backward_workspace(const AttnGradArgs& a)
{
    return (delta_floats(a.g) + size_floats(a.g) + part_lines(a) * 2 * a.g.D) * 4;
}

int plan_backward(ua2a_plan_t plan, const ua2a_attention_grad_t* n, AttnLaunch* L)
{
    if (n == nullptr) return UA2A_ERR_INVALID_ARG;
    int rc = check_attention(plan, n->type, n->window);
    if (rc != UA2A_OK) return rc;
    const int64_t SG = plan->S_local * plan->w;
    memset(L, 0, sizeof *L);
    L->type = n->type;
    rc = attn_geometry(plan, n->window, n->kv_heads, plan->B, SG, SG, &L->grad.g);
    if (rc != UA2A_OK) return rc;
    backward_shape(&L->grad);
    L->DP = padded_head(L->grad.g.D);
    L->block = kAttnBlock;
    return UA2A_OK;
}

}  // namespace

extern "C" {

int ua2a_rope(ua2a_plan_t plan, const ua2a_rope_t* n, void* stream)
{
    if (n == nullptr) return UA2A_ERR_INVALID_ARG;
    int rc = check_plan(plan, n->type);
    if (rc != UA2A_OK) return rc;
    for (const int32_t flag : {n->halves, n->inverse, n->per_plane, n->from, n->to})
        if (flag != 0 && flag != 1) return UA2A_ERR_INVALID_ARG;
    if (n->x == nullptr || n->out == nullptr || n->positions == nullptr || n->turns == nullptr || n->axes == nullptr)
        return UA2A_ERR_INVALID_ARG;
    const int64_t SG = plan->S_local * plan->w, each = n->per_plane ? plan->B * SG : SG;
    if (n->pairs < 1 || n->pairs > plan->D / 2 || n->naxes < 1 || tokens_of(plan) > kMost32 || each > kMost32 / n->naxes)
        return UA2A_ERR_SHAPE;
    const uintptr_t e = static_cast<uintptr_t>(plan->elem_bytes);
    if (misaligned(n->x, e) || misaligned(n->out, e) || misaligned(n->positions, 4) || misaligned(n->axes, 4) ||
        misaligned(n->turns, 8))
        return UA2A_ERR_ALIGN;
    AttnLaunch L;
    memset(&L, 0, sizeof L);
    L.kernel = AttnKernel::Rope;
    L.type = n->type;
    // vectors of 16 bytes, where heads and (in halves) their halves are whole ones
    const int32_t V = 16 / plan->elem_bytes;
    const bool wide = plan->D % V == 0 && !misaligned(n->x, 16) && !misaligned(n->out, 16) &&
                      (!n->halves || n->pairs % V == 0);
    L.V = wide ? V : 1;
    RopeGeom& g = L.rope.g;
    g.sh = shape_of(plan);
    g.pairs = static_cast<uint32_t>(n->pairs);
    g.halves = static_cast<uint32_t>(n->halves);
    g.inverse = static_cast<uint32_t>(n->inverse);
    g.from_a = static_cast<uint32_t>(n->from);
    g.to_a = static_cast<uint32_t>(n->to);
    g.per_plane = static_cast<uint32_t>(n->per_plane);
    g.naxes = static_cast<uint32_t>(n->naxes);
    g.axis_stride = each;
    g.tokens = static_cast<uint32_t>(tokens_of(plan));
    const uint32_t D = g.sh.D, rest = D - 2 * g.pairs, v = static_cast<uint32_t>(L.V);
    if (wide && !n->halves) {
        g.slots = g.turning = D / v;
    } else {
        g.turning = g.pairs / v;
        g.slots = g.turning + rest / v;
    }
    // a token's lanes: as many heads as divide H and fit a wave, but in a call that
    // fills the device a lane turns four heads at least, which its angles serve
    // (16 heads of 64 in halves, 50 MB: 17 us, 26 with one head a lane; 32 tokens:
    // 5.9 us with four, 5.2 with one)
    const uint32_t least_heads = tokens_of(plan) * g.sh.H * g.slots >= (1 << 18) ? 4 : 1;
    g.heads_at_once = 1;
    for (uint32_t k = 1; k * least_heads <= g.sh.H && k * g.slots <= 64; ++k)
        if (g.sh.H % k == 0) g.heads_at_once = k;
    g.lanes = least(g.slots * g.heads_at_once, kRopeBlock);
    g.per_group = kRopeBlock / g.lanes;
    g.d_lanes = make_div32(g.lanes);
    g.d_slots = make_div32(g.slots);
    g.d_SG = make_div32(g.sh.SG);
    g.d_pairs = make_div32(g.pairs);
    const int64_t bytes = plan->layout.tensor_bytes;
    const Range ins[] = {{n->positions, each * n->naxes * 4}, {n->turns, int64_t(n->pairs) * 8},
                         {n->axes, int64_t(n->pairs) * 4},
                         {n->from == n->to && n->x == n->out ? nullptr : n->x, bytes}};
    const Range outs[] = {{n->out, bytes}};
    if (aliased(outs, 1, ins, 4)) return UA2A_ERR_ALIAS;
    rc = check_device(plan);
    if (rc != UA2A_OK) return rc;
    L.rope.x = n->x;
    L.rope.out = n->out;
    L.rope.positions = n->positions;
    L.rope.turns = n->turns;
    L.rope.axes = n->axes;
    L.block = kRopeBlock;
    attn_grid(ceil_div(g.tokens, g.per_group), &L);
    const int err = attn_launch(L, stream);
    return err == 0 ? UA2A_OK : fail(plan, "launching the rotary kernel", err);
}

int ua2a_attention_workspace(ua2a_plan_t plan, const ua2a_attention_t* n, int64_t* bytes)
{
    if (bytes == nullptr) return UA2A_ERR_INVALID_ARG;
    AttnLaunch L;
    const int rc = plan_attention(plan, n, &L);
    if (rc == UA2A_OK) *bytes = forward_workspace(L.attn.g);
    return rc;
}

int ua2a_attention(ua2a_plan_t plan, const ua2a_attention_t* n, void* stream)
{
    AttnLaunch L;
    int rc = plan_attention(plan, n, &L);
    if (rc != UA2A_OK) return rc;
    if (n->q == nullptr || n->k == nullptr || n->v == nullptr || n->out == nullptr || !good_scale(n->scale))
        return UA2A_ERR_INVALID_ARG;
    if (misaligned(n->q, 16) || misaligned(n->k, 16) || misaligned(n->v, 16) || misaligned(n->out, 16) ||
        misaligned(n->lse, 4) || misaligned(n->counts, 4) || misaligned(n->workspace, 16))
        return UA2A_ERR_ALIGN;
    const AttnGeom& g = L.attn.g;
    const int64_t need = forward_workspace(g);
    if (need > 0 && n->workspace == nullptr) return UA2A_ERR_INVALID_ARG;
    if (n->workspace_bytes < need) return UA2A_ERR_CAPACITY;
    const int64_t bytes = plan->layout.tensor_bytes, kv = bytes / plan->H * n->kv_heads;
    const Range ins[] = {{n->q, bytes}, {n->k, kv}, {n->v, kv}, {n->counts, plan->B * 4}};
    const Range outs[] = {{n->out, bytes}, {n->lse, int64_t(g.units) * g.rows * 4}, {n->workspace, need}};
    if (aliased(outs, 3, ins, 4)) return UA2A_ERR_ALIAS;
    rc = check_device(plan);
    if (rc != UA2A_OK) return rc;
    L.attn.q = n->q;
    L.attn.k = n->k;
    L.attn.v = n->v;
    L.attn.out = n->out;
    L.attn.lse = n->lse;
    L.attn.counts = n->counts;
    L.attn.scale2 = n->scale * kLog2e;
    return launch_forward(plan, &L, n->workspace, stream);
}

int ua2a_cache_attention_workspace(ua2a_plan_t plan, const ua2a_cache_t* c, const ua2a_cache_attention_t* n, int64_t* bytes)
{
    if (bytes == nullptr) return UA2A_ERR_INVALID_ARG;
    AttnLaunch L;
    const int rc = plan_cache(plan, c, n, &L);
    if (rc == UA2A_OK) *bytes = forward_workspace(L.attn.g);
    return rc;
}

int ua2a_cache_attention(ua2a_plan_t plan, const ua2a_cache_t* c, const ua2a_cache_attention_t* n, void* stream)
{
    AttnLaunch L;
    int rc = plan_cache(plan, c, n, &L);
    if (rc != UA2A_OK) return rc;
    if (c->codes == nullptr || c->scales == nullptr || n->q == nullptr || n->out == nullptr || n->starts == nullptr ||
        !good_scale(n->scale))
        return UA2A_ERR_INVALID_ARG;
    if (misaligned(n->q, 16) || misaligned(n->out, 16) || misaligned(c->codes, 8) || misaligned(n->starts, 4) ||
        misaligned(n->counts, 4) || misaligned(n->workspace, 16))
        return UA2A_ERR_ALIGN;
    AttnArgs& a = L.attn;
    const AttnGeom& g = a.g;
    const int64_t need = forward_workspace(g);
    if (need > 0 && n->workspace == nullptr) return UA2A_ERR_INVALID_ARG;
    if (n->workspace_bytes < need) return UA2A_ERR_CAPACITY;
    const int64_t bytes = int64_t(g.units) * g.rows * g.D * 2, positions = int64_t(g.units) * g.keys;
    const Range ins[] = {{n->q, bytes}, {c->codes, 2 * positions * g.D}, {c->scales, 2 * positions * g.nb},
                         {n->starts, c->sequences * 4}, {n->counts, c->sequences * 4}};
    const Range outs[] = {{n->out, bytes}, {n->workspace, need}};
    if (aliased(outs, 2, ins, 5)) return UA2A_ERR_ALIAS;
    rc = check_device(plan);
    if (rc != UA2A_OK) return rc;
    a.q = n->q;
    a.out = n->out;
    a.starts = n->starts;
    a.counts = n->counts;
    a.codes = static_cast<const uint8_t*>(c->codes);
    a.scales = static_cast<const uint8_t*>(c->scales);
    a.part = positions * g.D;
    a.part_scales = positions * g.nb;
    a.format = c->format;
    a.keep = 1;
    a.scale2 = n->scale * kLog2e;
    return launch_forward(plan, &L, n->workspace, stream);
}

int ua2a_attention_backward_workspace(ua2a_plan_t plan, const ua2a_attention_grad_t* n, int64_t* bytes)
{
    if (bytes == nullptr) return UA2A_ERR_INVALID_ARG;
    AttnLaunch L;
    const int rc = plan_backward(plan, n, &L);
    if (rc == UA2A_OK) *bytes = backward_workspace(L.grad);
    return rc;
}

int ua2a_attention_backward(ua2a_plan_t plan, const ua2a_attention_grad_t* n, void* stream)
{
    AttnLaunch L;
    int rc = plan_backward(plan, n, &L);
    if (rc != UA2A_OK) return rc;
    for (const void* p : {n->dout, n->q, n->k, n->v, n->out, static_cast<const void*>(n->lse),
                          static_cast<const void*>(n->dq), static_cast<const void*>(n->dk), static_cast<const void*>(n->dv),
                          static_cast<const void*>(n->workspace)})
        if (p == nullptr) return UA2A_ERR_INVALID_ARG;
    if (!good_scale(n->scale)) return UA2A_ERR_INVALID_ARG;
    for (const void* p : {n->dout, n->q, n->k, n->v, n->out, static_cast<const void*>(n->dq),
                          static_cast<const void*>(n->dk), static_cast<const void*>(n->dv),
                          static_cast<const void*>(n->workspace)})
        if (misaligned(p, 16)) return UA2A_ERR_ALIGN;
    if (misaligned(n->lse, 4) || misaligned(n->counts, 4)) return UA2A_ERR_ALIGN;
    AttnGradArgs& a = L.grad;
    AttnGeom& g = a.g;
    const int64_t need = backward_workspace(a);
    if (n->workspace_bytes < need) return UA2A_ERR_CAPACITY;
    const int64_t bytes = plan->layout.tensor_bytes, kv = bytes / plan->H * n->kv_heads, lines = int64_t(g.units) * g.rows;
    const Range ins[] = {{n->dout, bytes}, {n->q, bytes}, {n->k, kv}, {n->v, kv}, {n->out, bytes}, {n->lse, lines * 4},
                         {n->counts, plan->B * 4}};
    const Range outs[] = {{n->dq, bytes}, {n->dk, kv}, {n->dv, kv}, {n->workspace, need}};
    if (aliased(outs, 4, ins, 7)) return UA2A_ERR_ALIAS;
    rc = check_device(plan);
    if (rc != UA2A_OK) return rc;
    a.q = n->q;
    a.k = n->k;
    a.v = n->v;
    a.out = n->out;
    a.dout = n->dout;
    a.lse = n->lse;
    a.counts = n->counts;
    a.dq = n->dq;
    a.dk = n->dk;
    a.dv = n->dv;
    a.scale = n->scale;
    a.scale2 = n->scale * kLog2e;
    a.delta = static_cast<float*>(n->workspace);
    a.sizes = a.delta + delta_floats(g);
    a.partial = a.sizes + size_floats(g);
    const AttnGeom by_keys = g;
    L.kernel = AttnKernel::GradRows;
    set_items(&g, ceil_div(g.rows, kAttnRows), 1);
    g.order = order_of(g, false);
    attn_grid(workgroups(g), &L);
    int err = attn_launch(L, stream);
    if (err != 0) return fail(plan, "launching attention's backward kernel of rows", err);
    g = by_keys;
    L.kernel = AttnKernel::GradKeys;
    attn_grid(workgroups(g), &L);
    err = attn_launch(L, stream);
    if (err != 0) return fail(plan, "launching attention's backward kernel of keys", err);
    if (part_lines(a) == 0) return UA2A_OK;
    L.kernel = AttnKernel::GradJoin;
    attn_grid(ceil_div(int64_t(g.units) * a.keys.d_keys.d, a.keys.per_group), &L);
    err = attn_launch(L, stream);
    return err == 0 ? UA2A_OK : fail(plan, "launching the join of the keys' gradients", err);
}

}  // extern "C"
