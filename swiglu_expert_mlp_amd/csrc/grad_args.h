// Launch arguments of the experts' backward products (shared by host and device code).
#pragma once

#include "common.h"

namespace moe {

struct GradArgs {
    const int2* tiles;         // (expert, first row) per 64-row M tile
    const int2* tiles_big;     // (expert, first row) per 256-row M tile
    const int32_t* offsets;    // [E + 1]
    const WsHeader* hdr;
    const int32_t* perm_src;   // grouped row -> route t * topk + j (canonical order)
    const float* prob;         // by route, canonical order
    int E, H, F, topk;
    const uint16_t* x;         // bf16 [T_cap][H]
    const uint16_t* d_out;     // bf16 [T_cap][H]
    const uint16_t* w1;        // packed sections of the kernel weights
    const uint16_t* w2;
    const int8_t* codes;       // [rows][2F], interleaved blocks of 32
    const uint8_t* scales;     // [rows][F / 16]
    uint16_t* dgu;             // bf16 [rows][2F]
    uint16_t* hp;              // bf16 [rows][F]
    uint16_t* dx;              // [rows][H], 16-bit codes (grad_dx.h)
    uint8_t* dx_scale;         // [rows][H / 16], their scale bytes
    float* part;               // fp32 [rows][F / 32]
    int32_t* row_tok;          // int32 [rows]: token of each grouped row
    void* d_w1;                // [E][2F][H], gate rows first
    void* d_w2;                // [E][H][F]
};

}  // namespace moe
