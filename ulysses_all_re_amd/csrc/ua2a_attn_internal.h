// Internal declarations shared by the attention operators' host code
// (ua2a_attn_host.cpp) and kernels (ua2a_attn_*.hip, ua2a_rope.hip).
#pragma once

#include "ua2a_attn.h"
#include "ua2a_attn_geometry.h"
#include "ua2a_internal.h"

namespace ua2a {

constexpr uint32_t kRopeBlock = 256;         // lanes per workgroup of the rotary kernel
constexpr uint32_t kAttnBlock = 256;         // lanes per workgroup, four waves
constexpr uint32_t kAttnWaveRows = 32;       // rows of a wave, the columns of its matrix tiles
constexpr uint32_t kDecodeRows = 16;         // most rows of the kernel of single tokens
constexpr uint32_t kAttnRows = 128;          // rows of a workgroup whose waves take rows of their own
constexpr uint32_t kAttnKeys = 64;           // keys of a tile that four waves share
constexpr uint32_t kAttnSplitKeys = 128;     // keys of a tile whose quarters go to the waves
constexpr uint32_t kAttnGradKeys = 128;      // keys of a workgroup of their gradients
constexpr uint32_t kAttnGridLog = 23;        // workgroups along x: 2^31 lanes
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

struct AttnArgs {
    AttnGeom g;
    const void* q;
    const void* k;               // null: the cache
    const void* v;
    void* out;
    float* lse;                  // [ranks][seqs][hl][n] or null
    const int32_t* starts;       // null: 0
    const int32_t* counts;       // null: n
    const uint8_t* codes;        // keys'; the values' lie `part` further
    const uint8_t* scales;
    int64_t part, part_scales;
    int32_t format;
    int32_t keep;                // 1: rows without a query stay as they are; 0: zeros
    float scale2;                // the scores' factor times log2(e)
    float* partial;              // splits > 1: [splits][units * rows][D] sums and [..][2] statistics
    float* stats;
};

struct AttnGradArgs {
    AttnGeom g;                  // tiles: of rows, then of keys
    KeyTiles keys;
    const void* q;
    const void* k;
    const void* v;
    const void* out;
    const void* dout;
    const float* lse;
    const int32_t* counts;
    void* dq;
    void* dk;
    void* dv;
    float* delta;                // [units][rows]
    float* sizes;                // [units][tiles of rows][2]: largest |dout| and |delta| of the tile's rows
    float scale, scale2;
    float* partial;              // parts' sums: [KeyTiles' lines][2][D]
};

struct RopeArgs {
    RopeGeom g;
    const void* x;
    void* out;
    const int32_t* positions;
    const uint64_t* turns;       // [pairs]
    const int32_t* axes;         // [pairs]
};

enum class AttnKernel : int32_t { Rope, Forward, Decode, Join, GradRows, GradKeys, GradJoin };

struct AttnLaunch {
    AttnKernel kernel;
    int32_t type;                // UA2A_TYPE_*
    int32_t V;                   // rope: values per lane slot
    int32_t DP;                  // head values padded to 32, 64, 96 or 128
    int32_t shared;              // forward: 1, all waves the same rows and keys of their own
    uint32_t block, grid_x, grid_y;
    AttnArgs attn;
    AttnGradArgs grad;
    RopeArgs rope;
};

int attn_launch(const AttnLaunch& launch, void* stream);   // 0 or a backend error code

}  // namespace ua2a
