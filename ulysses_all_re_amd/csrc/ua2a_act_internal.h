// Internal declarations shared by the activation operators' host code
// (ua2a_act_host.cpp) and kernels (ua2a_act_kernels.hip).
#pragma once

#include "ua2a_act.h"
#include "ua2a_act_geometry.h"
#include "ua2a_internal.h"

namespace ua2a {

constexpr uint32_t kActBlock = 256;          // lanes per workgroup
constexpr uint32_t kActBigBlock = 1024;      // ... for norms longer than kActItems * kActBlock slots
constexpr uint32_t kActItems = 5;            // most slots per lane of a kActBlock workgroup
constexpr uint32_t kActBigItems = 8;         // ... of a kActBigBlock workgroup

struct NormArgs {
    NormGeom g;
    const void* x;
    const void* residual;
    const void* weight;
    void* out;
    uint8_t* out_scales;
    void* sum;
    uint8_t* saved;
    uint8_t* saved_scales;
    float* rstd;
    float eps;
    float inv_len;               // 1 / values of a norm
    int32_t weight_f32;
    int32_t out_format;
    int32_t saved_format;
};

struct NormGradArgs {
    NormGeom g;
    const void* dy;
    const void* dsum;
    const void* saved;
    const uint8_t* saved_scales;
    const void* weight;
    const float* rstd;
    void* dx;
    void* dresidual;
    float* partial;              // [grid][cols], or null without dweight
    float inv_len;
    int32_t weight_f32;
    int32_t saved_format;
    int32_t saved_gathered;
};

struct ColumnArgs {              // dweight[c] = sum over rows of partial[row][c]
    const float* partial;
    float* out;
    uint32_t rows, cols;
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
    int32_t span;                // norms: how segments lie on lanes (Span of ua2a_act_norm.h)
    int32_t mode;
    uint32_t block, grid_x, grid_y;
    NormArgs norm;
    NormGradArgs grad;
    ColumnArgs columns;
    CacheArgs cache;
};

int act_launch(const ActLaunch& launch, void* stream);   // 0 or a backend error code

}  // namespace ua2a
