// What the host sides of the activation and attention operators share: argument
// checks, overlap by byte ranges, and a plan's shape for the kernels.  Each
// source that includes this has its own copy.
#pragma once

#include <stdio.h>

#include "ua2a_act.h"
#include "ua2a_act_geometry.h"
#include "ua2a_internal.h"

namespace ua2a {
namespace {

struct Range {
    const void* p;
    int64_t bytes;
};

[[maybe_unused]] inline bool overlap(const Range& a, const Range& b)
{
    const uintptr_t pa = reinterpret_cast<uintptr_t>(a.p), pb = reinterpret_cast<uintptr_t>(b.p);
    return a.p != nullptr && b.p != nullptr && a.bytes > 0 && b.bytes > 0 &&
           pa < pb + static_cast<uintptr_t>(b.bytes) && pb < pa + static_cast<uintptr_t>(a.bytes);
}

// Whether an output overlaps another output or an input.
[[maybe_unused]] inline bool aliased(const Range* outs, int nouts, const Range* ins, int nins)
{
    for (int i = 0; i < nouts; ++i) {
        for (int k = i + 1; k < nouts; ++k)
            if (overlap(outs[i], outs[k])) return true;
        for (int k = 0; k < nins; ++k)
            if (overlap(outs[i], ins[k])) return true;
    }
    return false;
}

[[maybe_unused]] inline bool misaligned(const void* p, uintptr_t to) { return reinterpret_cast<uintptr_t>(p) % to != 0; }

[[maybe_unused]] inline int32_t type_bytes(int32_t type)
{
    return type == UA2A_TYPE_FP32 ? 4 : type == UA2A_TYPE_BF16 || type == UA2A_TYPE_FP16 ? 2 : 0;
}

[[maybe_unused]] inline bool good_format(int32_t f) { return f == UA2A_FORMAT_E4M3 || f == UA2A_FORMAT_E5M2; }

[[maybe_unused]] inline int fail(ua2a_plan_t plan, const char* what, int err)
{
    plan->disabled = 1;
    snprintf(plan->reason, sizeof plan->reason, "%s failed: %s", what, backend_error_name(err));
    return UA2A_ERR_HIP;
}

[[maybe_unused]] inline int check_device(ua2a_plan_t plan)
{
    int32_t dev = -1;
    const int err = backend_current_device(&dev);
    if (err != 0) return fail(plan, "querying the current device", err);
    return dev == plan->device ? UA2A_OK : UA2A_ERR_DEVICE;
}

[[maybe_unused]] inline int64_t tokens_of(const ua2a_plan_s* p) { return p->layout.tensor_elems / (p->H * p->D); }

[[maybe_unused]] inline ActShape shape_of(const ua2a_plan_s* p)
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

[[maybe_unused]] inline uint32_t log2_of(uint32_t pow2)
{
    uint32_t l = 0;
    while ((1u << l) < pow2) ++l;
    return l;
}

[[maybe_unused]] inline uint32_t least(uint32_t a, uint32_t b) { return a < b ? a : b; }

// What every call checks first.
[[maybe_unused]] inline int check_plan(ua2a_plan_t plan, int32_t type)
{
    if (plan == nullptr) return UA2A_ERR_INVALID_ARG;
    if (plan->disabled) return UA2A_ERR_DISABLED;
    if (type_bytes(type) == 0 || type_bytes(type) != plan->elem_bytes) return UA2A_ERR_INVALID_ARG;
    return UA2A_OK;
}

}  // namespace
}  // namespace ua2a
