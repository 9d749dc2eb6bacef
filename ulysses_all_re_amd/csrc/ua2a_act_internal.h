// Internal declarations shared by the activation operators' host code
// (ua2a_act_host.cpp) and kernels (ua2a_act_*.hip).
#pragma once

#include "ua2a_act.h"
#include "ua2a_act_geometry.h"
#include "ua2a_internal.h"

namespace ua2a {

constexpr uint32_t kActBlock = 256;          // lanes per workgroup
constexpr uint32_t kActBigBlock = 1024;      // most lanes of a workgroup that one norm has to itself
constexpr uint32_t kActItems = 5;            // most slots per lane of a kActBlock workgroup
constexpr uint32_t kActBigItems = 8;         // ... of a workgroup that one norm has to itself

// What a norm call is about, one bit each.
constexpr uint32_t kNormMode1 = 1;           // x, or dx, in A; out, or dy, in P
constexpr uint32_t kNormWeight = 2;
constexpr uint32_t kNormResidual = 4;        // forward: added; backward: dsum is there
constexpr uint32_t kNormRstd = 8;            // forward: rstd is written
constexpr uint32_t kNormPartial = 16;        // backward: dweight's sums are wanted
constexpr uint32_t kNormApart = 32;          // backward: dresidual is written
constexpr uint32_t kNormGathered = 64;       // backward: what was normed is in A
constexpr uint32_t kNormOut8 = 128;          // forward: out in 8 bits
constexpr uint32_t kNormSaved8 = 256;        // forward: the checkpoint is written
constexpr uint32_t kNormOutE5M2 = 512;       // formats: e4m3, or this
constexpr uint32_t kNormSavedE5M2 = 1024;

struct NormArgs {
    NormGeom g;
    uint32_t flags;
    float eps;
    float inv_len;               // 1 / values of a norm
    int32_t weight_f32;
    const void* x;
    const void* weight;
    void* out;
    const void* residual;
    void* sum;
    float* rstd;
    uint8_t* saved;
    uint8_t* saved_scales;
    uint8_t* out_scales;
};

struct NormGradArgs {
    NormGeom g;
    uint32_t flags;
    float inv_len;
    int32_t weight_f32;
    int32_t saved_format;
    const void* dy;
    const void* saved;
    const uint8_t* saved_scales;
    const float* rstd;
    const void* weight;
    const void* dsum;
    void* dx;
    void* dresidual;
    float* partial;              // [grid][cols]
};

struct ColumnArgs {              // dweight[c] = sum over rows of partial[row][c]
    const float* partial;
    float* out;
    uint32_t rows, cols;
    uint32_t across_log;         // columns of a workgroup = 2^across_log
};

struct CacheArgs {
    CacheGeom g;
    const void* k;               // write: inputs; read: null
    const void* v;
    void* k_out;                 // read: outputs
    void* v_out;
    uint8_t* codes;
    uint8_t* scales;
    const int32_t* starts;
    const int32_t* counts;
    int32_t format;
};

enum class ActKernel : int32_t { Norm, NormGrad, Columns, CacheWrite, CacheRead };

struct ActLaunch {
    ActKernel kernel;
    int32_t type;                // UA2A_TYPE_*
    int32_t V;                   // values per lane slot: 16 / elem_bytes, or 1
    int32_t items;               // norms: slots per lane (a compiled count)
    int32_t span;                // norms: how segments lie on lanes (kSpan...)
    uint32_t block, grid_x, grid_y;
    NormArgs norm;
    NormGradArgs grad;
    ColumnArgs columns;
    CacheArgs cache;
};

int act_launch(const ActLaunch& launch, void* stream);   // 0 or a backend error code

}  // namespace ua2a
