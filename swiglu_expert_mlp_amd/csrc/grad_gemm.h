// The experts' backward pass: grouped products on CDNA4 MFMA, bf16 operands, fp32
// accumulate, 256 x 256 output tiles.
//
// With r a grouped row (expert e, token t, probability p) and the interleaved gate/up
// order of the kernel weights for the columns of dgu and the rows of W1:
//   rows, SWIGLU   raw[r][f] = sum_h d_out[t][h] W2_e[h][f], then per element, from the
//                  8-bit gate g and up u:  s = 1 / (1 + exp(-g)),  h = g s u,
//                    dgu[r] = p raw (u s (1 + g (1 - s)),  g s),   hp[r] = p h,
//                    part[r][f / 32] = sum over 32 columns of raw h
//   rows, plain    dx[r][h] = sum_n dgu[r][n] W1_e[n][h]
//   weights        dW1_e[n][h] = sum_r dgu[r][n] x[t][h]
//                  dW2_e[h][f] = sum_r d_out[t][h] hp[r][f]
// dgu and hp are rounded to bf16, the operand type of the next product; dx is kept in
// 16-bit integers with a scale per 16 columns (grad_dx.h: half the bytes of fp32 rows, 1/128
// of bf16's error at the block's largest); every sum is fp32.
//
// Every product but the rows' first operand runs over an index that is not contiguous in
// memory: the rows products over the rows of the kernel weights, which hold 8
// neighbouring columns together, the weight products over the grouped rows themselves.
// ds_read_b64_tr_b16 turns 4 x 16 blocks of 16-bit elements on the way from LDS to
// registers, so no operand is ever transposed in memory and the backward pass reads the
// same packed weights as the forward.  Of each 16 lanes, lane j names 4 contiguous
// elements of row j / 4 (columns 4 (j % 4) ..) and lane i receives column i of the 4 rows.
//
// The tile loop is the 256-row forward's (gemm_bf16_big.h): 8 waves of 128 x 64, two
// LDS stages of 64 along the sum by direct global->LDS loads, one barrier a stage, the
// next tile's first two stages issued before the epilogue, which has LDS of its own.
//
// Measured (16,384 tokens, top-8 of 128 experts, hidden 2048, FFN 1024; the library's dense
// bf16 product of 8192^3 runs at 1.21 PF/s): the product before the SwiGLU 769 us (0.72
// PF/s; its epilogue, 23 vector instructions an element, is a fifth of it), the one after it
// 1064 (1.03), the weights' 1571 (1.05; a fp32 result, twice the bytes stored, takes the call from
// 3515 to 3784, 4,096 skewed tokens from 1351 to 1602, 1,000 tokens on 64 experts 435 to 519).  What bounds them: the matrix units are busy 60 % of
// the cycles at 1.8 to 1.9 GHz, the clock that the power limit leaves; with the loads taken
// out of a copy the two large ones take 870 and 1360 us, with the MFMAs out 890 and 1270.
// Not bound by LDS: with the bank conflicts of the row operand's reads removed (40 % of the
// LDS cycles) the times stayed.
#pragma once

#include "gemm_bf16_big.h"
#include "grad_args.h"
#include "grad_dx.h"

namespace moe {

typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef short s16x8 __attribute__((ext_vector_type(8)));
typedef __attribute__((address_space(3))) s16x4 lds_s16x4;

// Zeros, the source of loads that lie past the end of a sum (1 KB: a block of weights)
__device__ const uint32_t grad_zeros[256] __attribute__((aligned(16))) = {};

// 8 elements along the sum for one column of an MFMA operand: two transposing reads,
// the second `step` bytes after the first
__device__ __forceinline__ bf16x8 grad_tr(const char* p, int step)
{
    const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)p);
    const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(p + step));
    const s16x8 v = {lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
    return __builtin_bit_cast(bf16x8, v);
}

// The tile range of this workgroup's XCD: 8 contiguous ranges, walked in steps of the
// XCD's workgroups (gridDim.x / 8)
struct GradRange { int first, end, step; };
__device__ __forceinline__ GradRange grad_range(int total)
{
    const int xcd = blockIdx.x & 7, chunk = (total + 7) / 8;
    return {xcd * chunk + (int)(blockIdx.x >> 3), min(total, (xcd + 1) * chunk), (int)(gridDim.x >> 3)};
}

template <int STORES>
__device__ __forceinline__ void grad_dummy_stores(void* p, int lane)
{
    // the K loop counts the previous tile's stores; before the first tile the same number
    // go to an empty descriptor, whose range check drops them (distinct offsets, so that
    // none is merged away)
    const __amdgpu_buffer_rsrc_t none = __builtin_amdgcn_make_buffer_rsrc(p, (short)0, 0, kBigRsrcWord3);
#pragma unroll
    for (int k = 0; k < STORES; ++k)
        __builtin_amdgcn_raw_buffer_store_b128(u32x4_t{0u, 0u, 0u, 0u}, none, 16 * lane + 1024 * k, 0, 0);
}

struct GradFrag {
    bf16x8 a[4], b[2];
};

// The operands go in swapped, so that a block's results come transposed: lane l holds row
// l % 32 and columns 8 (v / 4) + 4 (l / 32) + v % 4, four neighbouring ones at a time, and
// leaves them in LDS by 16-byte writes (one value a write otherwise)
__device__ __forceinline__ f32x16 grad_mfma(bf16x8 a, bf16x8 b, f32x16 acc)
{
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(b, a, acc, 0, 0, 0);
}

__device__ __forceinline__ void grad_mma(f32x16 (&acc)[4][2], const GradFrag& f)
{
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j) acc[i][j] = grad_mfma(f.a[i], f.b[j], acc[i][j]);
}

// One sub-step of 16 along the sum: the MFMAs of `cur` with the READS fragment reads of
// the next sub-step spread between them, and DMA direct loads (4 or 8) issued just before,
// with ALU scalar and vector instructions of their addresses a MFMA, so that no wave stands at
// its loads with its matrix unit idle (16K tokens: rows after the SwiGLU 1077 -> 1063 us, before
// it 784 -> 777, weights 1705 -> 1669); nothing else crosses its ends
template <int READS, int DMA = 0, int ALU = 0, typename Read>
__device__ __forceinline__ void grad_phase(f32x16 (&acc)[4][2], const GradFrag& cur, Read read, GradFrag& nxt)
{
    read(nxt);
    grad_mma(acc, cur);
    constexpr int two = READS > 8 ? READS - 8 : 0;       // MFMAs followed by two reads
    auto extra = [&](int k) {
        if constexpr (DMA > 0) {
            if constexpr (ALU > 0) {
                __builtin_amdgcn_sched_group_barrier(0x004, ALU, 0);
                __builtin_amdgcn_sched_group_barrier(0x002, ALU, 0);
            }
            if (k % (8 / DMA) == 8 / DMA - 1) __builtin_amdgcn_sched_group_barrier(0x010, 1, 0);
        }
    };
#pragma unroll
    for (int k = 0; k < two; ++k) {
        __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
        __builtin_amdgcn_sched_group_barrier(0x100, 2, 0);
        extra(k);
    }
#pragma unroll
    for (int k = two; k < 8; ++k) {
        __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
        __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
        extra(k);
    }
    __builtin_amdgcn_sched_barrier(0);
}

// The sum over nst stages (nst >= 1) of a tile.  On entry this wave's loads of stages 0
// and 1 are in flight into s0 and s1, followed by AFTER stores.  read(Q, stage, frag)
// reads the fragments of sub-step Q; issue(stage, s) loads stage s (unconditional, so that
// no path differs in its loads in flight: past the last stage it loads that one again,
// into the buffer that no later read of the tile uses).  One last grad_mma for every path:
// with a copy of it on each, the compiler kept the accumulators twice and spilled.
template <int READS, int AFTER, typename Read, typename Issue>
__device__ __forceinline__ void grad_kloop(int nst, char* s0, char* s1, f32x16 (&acc)[4][2],
                                           Read read, Issue issue)
{
    static_assert(AFTER + 9 <= 63, "vmcnt bound");
    GradFrag x, y;
    using Q0 = std::integral_constant<int, 0>;
    using Q1 = std::integral_constant<int, 1>;
    using Q2 = std::integral_constant<int, 2>;
    using Q3 = std::integral_constant<int, 3>;
    BIG_WAIT_VMCNT(AFTER);
    __builtin_amdgcn_s_barrier();
    read(Q0{}, s0, x);
    auto body = [&](const char* cur) {
        grad_phase<READS>(acc, x, [&](GradFrag& n) { read(Q1{}, cur, n); }, y);
        grad_phase<READS>(acc, y, [&](GradFrag& n) { read(Q2{}, cur, n); }, x);
        grad_phase<READS>(acc, x, [&](GradFrag& n) { read(Q3{}, cur, n); }, y);
    };
    // this wave's loads of the next stage landed (N younger operations may be in flight)
    // and its reads of the current one are done; after the barrier both hold for every
    // wave, and the current buffer may be refilled
    auto boundary = [&](auto NC) {
        constexpr int N = decltype(NC)::value;
        __builtin_amdgcn_sched_barrier(0);
        BIG_WAIT_VMCNT(N);
        __builtin_amdgcn_s_waitcnt(0xC07F);          // lgkmcnt(0)
        __builtin_amdgcn_s_barrier();
        __builtin_amdgcn_sched_barrier(0);
    };
    auto into = [&](const char* nxt) {
        grad_phase<READS, 8>(acc, y, [&](GradFrag& n) { read(Q0{}, nxt, n); }, x);
    };
    using Now = std::integral_constant<int, 0>;
    body(s0);
    if (nst > 1) {
        boundary(std::integral_constant<int, AFTER>{});
        issue(s0, min(2, nst - 1));
        into(s1);
        int s = 1;
        for (; s + 2 < nst; s += 2) {
            body(s1);
            boundary(Now{});
            issue(s1, s + 2);
            into(s0);
            body(s0);
            boundary(Now{});
            issue(s0, min(s + 3, nst - 1));
            into(s1);
        }
        body(s1);
        if (s + 1 < nst) {
            boundary(Now{});
            into(s0);
            body(s0);
        }
    }
    grad_mma(acc, y);
}

// grad_kloop with the two stages in halves of 32 along the sum (h0, h1 the first stage's, h2,
// h3 the second's) that are refilled one by one, so three halves instead of one stage are in
// flight, for two barriers a stage.  LOADS: direct loads of a half per wave.  On entry four
// halves are in flight, the last of them h3 or h1, followed by AFTER stores.  read(Q, half,
// frag): sub-step Q = 0, 1 of a half; issue(slot, half): refills that half, with the tile's
// next one or, past its last, with the next tile's half of that slot.
template <int READS, int AFTER, int LOADS, typename Read, typename Issue>
__device__ __forceinline__ void grad_kloop_halves(int nst, char* h0, char* h1, char* h2, char* h3,
                                                  f32x16 (&acc)[4][2], Read read, Issue issue)
{
    static_assert(AFTER + 2 * LOADS <= 63, "vmcnt bound");
    GradFrag x, y;
    using Q0 = std::integral_constant<int, 0>;
    using Q1 = std::integral_constant<int, 1>;
    BIG_WAIT_VMCNT(AFTER + LOADS);
    __builtin_amdgcn_s_barrier();
    read(Q0{}, h0, x);
    // N: the operations younger than the next half that may be in flight.  It has landed then,
    // and every wave's reads of `cur` are done: `cur` is refilled
    auto boundary = [&](auto NC, auto SC, char* cur) {
        __builtin_amdgcn_sched_barrier(0);
        BIG_WAIT_VMCNT(decltype(NC)::value);
        __builtin_amdgcn_s_waitcnt(0xC07F);          // lgkmcnt(0)
        __builtin_amdgcn_s_barrier();
        __builtin_amdgcn_sched_barrier(0);
        issue(SC, cur);
    };
    auto body = [&](auto NC, auto SC, char* a, char* b) {
        grad_phase<READS>(acc, x, [&](GradFrag& n) { read(Q1{}, a, n); }, y);
        boundary(NC, SC, a);
        grad_phase<READS, 4, 6>(acc, y, [&](GradFrag& n) { read(Q0{}, b, n); }, x);
        grad_phase<READS>(acc, x, [&](GradFrag& n) { read(Q1{}, b, n); }, y);
    };
    auto into = [&](auto NC, auto SC, char* b, char* c) {
        boundary(NC, SC, b);
        grad_phase<READS, 4, 6>(acc, y, [&](GradFrag& n) { read(Q0{}, c, n); }, x);
    };
    using S0 = std::integral_constant<int, 0>;
    using S1 = std::integral_constant<int, 1>;
    using S2 = std::integral_constant<int, 2>;
    using S3 = std::integral_constant<int, 3>;
    using Two = std::integral_constant<int, 2 * LOADS>;
    body(std::integral_constant<int, AFTER>{}, S0{}, h0, h1);       // the first four have landed
    if (nst > 1) {
        into(std::integral_constant<int, AFTER + LOADS>{}, S1{}, h1, h2);
        body(std::integral_constant<int, AFTER + 2 * LOADS>{}, S2{}, h2, h3);
        int s = 2;
        for (; s + 2 <= nst; s += 2) {
            into(Two{}, S3{}, h3, h0);
            body(Two{}, S0{}, h0, h1);
            into(Two{}, S1{}, h1, h2);
            body(Two{}, S2{}, h2, h3);
        }
        if (s < nst) {
            into(Two{}, S3{}, h3, h0);
            body(Two{}, S0{}, h0, h1);
        }
    }
    grad_mma(acc, y);
}

// A wave's results leave through its LDS region, a block at a time.  fp32: 32 rows of 128
// bytes, 16-byte chunk c of row r at c ^ ((r / 2) % 8); bf16: 32 rows of 64 columns, also 128
// bytes, placed the same way.  (Two rows span the banks, so 16 rows' writes of one chunk, and
// the reads of 8 rows' halves, fall on distinct ones.)  The offsets are opaque: with a
// constant part folded into the instruction the compiler waited for the next tile's direct
// loads before the write.
__device__ __forceinline__ int grad_at(int row, int chunk) { return row * 128 + 16 * (chunk ^ ((row >> 1) & 7)); }

__device__ __forceinline__ void grad_block_to_lds(const f32x16& acc, char* ep, int lane)
{
    const int r = lane & 31, hi = lane >> 5;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        int ea = grad_at(r, 2 * q + hi);
        asm volatile("" : "+v"(ea));
        *(f32x4*)(ep + ea) = f32x4{acc[4 * q], acc[4 * q + 1], acc[4 * q + 2], acc[4 * q + 3]};
    }
}

// 16 neighbouring columns (half h) of a row of the block
__device__ __forceinline__ void grad_read16(const char* ep, int row, int h, float (&v)[16])
{
#pragma unroll
    for (int c = 0; c < 4; ++c) {
        const f32x4 u = *(const f32x4*)(ep + grad_at(row, 4 * h + c));
#pragma unroll
        for (int m = 0; m < 4; ++m) v[4 * c + m] = u[m];
    }
}

// Two values rounded to bf16 (nearest even) by one instruction (rounded one by one and put
// together they were four, a sixth of the SwiGLU's backward)
__device__ __forceinline__ uint32_t grad_pair(float a, float b)
{
    typedef float f32x2 __attribute__((ext_vector_type(2)));
    typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
    return __builtin_bit_cast(uint32_t, __builtin_convertvector((f32x2{a, b}), bf16x2));
}

__device__ __forceinline__ void grad_blocks_to_lds_bf16(const f32x16 (&acc)[2], char* ep, int lane)
{
    const int r = lane & 31, hi = lane >> 5;
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            int ea = grad_at(r, 4 * j + q) + 8 * hi;
            asm volatile("" : "+v"(ea));
            *(uint2*)(ep + ea) = make_uint2(grad_pair(acc[j][4 * q], acc[j][4 * q + 1]),
                                            grad_pair(acc[j][4 * q + 2], acc[j][4 * q + 3]));
        }
}

// ---------------------------------------------------------------- rows products

// What 16 neighbouring columns of a row need from memory: kept gate and up codes and the
// two scale bytes of their block
struct GradKept {
    u32x4_t cg, cu;
    uint16_t sc;
};
__device__ __forceinline__ GradKept grad_kept(const GradArgs& g, int64_t row, int block, int half)
{
    const int8_t* c = g.codes + row * 2 * g.F + 64 * block + 16 * half;
    return {*(const u32x4_t*)c, *(const u32x4_t*)(c + 32), *(const uint16_t*)(g.scales + row * (g.F / 16) + 2 * block)};
}

// The SwiGLU's backward of 16 columns: bf16 pairs of the gate's and up's gradients and of
// p h; returns the sum of raw h
__device__ __forceinline__ float grad_swiglu16(const float (&raw)[16], const GradKept& k, float p, uint32_t (&og)[8],
                                               uint32_t (&ou)[8], uint32_t (&oh)[8])
{
    const float sg = ckpt_scale(k.sc & 0xff), su = ckpt_scale(k.sc >> 8);
    float dot = 0.0f;
#pragma unroll
    for (int m = 0; m < 16; m += 2) {
        float vg[2], vu[2], vh[2];
#pragma unroll
        for (int n = 0; n < 2; ++n) {
            const int sh = 24 - 8 * ((m + n) & 3);
            const float gate = (float)((int)(k.cg[(m + n) >> 2] << sh) >> 24) * sg;
            const float up = (float)((int)(k.cu[(m + n) >> 2] << sh) >> 24) * su;
            const float s = __builtin_amdgcn_rcpf(1.0f + __expf(-gate));
            const float silu = gate * s;
            const float h = silu * up;
            dot = __builtin_fmaf(raw[m + n], h, dot);
            const float dh = raw[m + n] * p;
            vu[n] = dh * silu;
            vg[n] = dh * up * __builtin_fmaf(silu, 1.0f - s, s);
            vh[n] = h * p;
        }
        og[m / 2] = grad_pair(vg[0], vg[1]);
        ou[m / 2] = grad_pair(vu[0], vu[1]);
        oh[m / 2] = grad_pair(vh[0], vh[1]);
    }
    return dot;
}

// Stores of grad_swiglu16's results: row `row` of the tile, columns 16 half .. of `block`
// (past the last block: outside the descriptors, which drop them)
__device__ __forceinline__ void grad_swiglu_store(__amdgpu_buffer_rsrc_t gu, __amdgpu_buffer_rsrc_t hr, int F, int row,
                                                  int block, int half, const uint32_t (&og)[8], const uint32_t (&ou)[8],
                                                  const uint32_t (&oh)[8])
{
    const bool cols = block * 32 < F;
    const int og0 = cols ? (row * 2 * F + 64 * block + 16 * half) * 2 : 0x7ffffe00;
    const int oh0 = cols ? (row * F + 32 * block + 16 * half) * 2 : 0x7ffffe00;
#pragma unroll
    for (int hf = 0; hf < 2; ++hf) {
        const u32x4_t a = {og[4 * hf], og[4 * hf + 1], og[4 * hf + 2], og[4 * hf + 3]};
        const u32x4_t b = {ou[4 * hf], ou[4 * hf + 1], ou[4 * hf + 2], ou[4 * hf + 3]};
        const u32x4_t c = {oh[4 * hf], oh[4 * hf + 1], oh[4 * hf + 2], oh[4 * hf + 3]};
        __builtin_amdgcn_raw_buffer_store_b128(a, gu, og0 + 16 * hf, 0, 0);
        __builtin_amdgcn_raw_buffer_store_b128(b, gu, og0 + 64 + 16 * hf, 0, 0);
        __builtin_amdgcn_raw_buffer_store_b128(c, hr, oh0 + 16 * hf, 0, 0);
    }
}

// The first column tile of the SWIGLU product leaves the token of every row for the weight
// products: 8 lanes hold a row's, the first stores it (a store for all, which the descriptor
// drops for the others and for rows past `rows`: no branch among the loads in flight)
__device__ __forceinline__ void grad_leave_token(const GradArgs& g, int row0, int rows, int r, int tok, int lane)
{
    const __amdgpu_buffer_rsrc_t d =
        __builtin_amdgcn_make_buffer_rsrc((void*)(g.row_tok + row0), (short)0, 4 * rows, kBigRsrcWord3);
    __builtin_amdgcn_raw_buffer_store_b32((uint32_t)tok, d, (lane & 7) == 0 ? 4 * r : 0x7ffffff0, 0, 0);
}

// The epilogue of one 32 x 32 block of either rows product, shared by the tile designs: lane
// = row lane / 2 and 16 columns (half lane % 2).
struct GradOut {
    __amdgpu_buffer_rsrc_t o0, o1;     // SWIGLU: rows of dgu, of hp; else of dx, of its scales
};
template <bool SWIGLU>
__device__ __forceinline__ GradOut grad_out(const GradArgs& g, int row0, int rows)
{
    if constexpr (SWIGLU)
        return {__builtin_amdgcn_make_buffer_rsrc((void*)(g.dgu + (int64_t)row0 * 2 * g.F), (short)0, rows * 4 * g.F,
                                                  kBigRsrcWord3),
                __builtin_amdgcn_make_buffer_rsrc((void*)(g.hp + (int64_t)row0 * g.F), (short)0, rows * 2 * g.F,
                                                  kBigRsrcWord3)};
    else
        return {__builtin_amdgcn_make_buffer_rsrc((void*)(g.dx + (int64_t)row0 * g.H), (short)0, rows * 2 * g.H,
                                                  kBigRsrcWord3),
                __builtin_amdgcn_make_buffer_rsrc((void*)(g.dx_scale + (int64_t)row0 * (g.H / 16)), (short)0,
                                                  rows * (g.H / 16), kBigRsrcWord3)};
}

// SWIGLU: block `block` of the FFN, rows tr .. tr + 31 of the tile's `rows` from row0 on
__device__ __forceinline__ void grad_swiglu_block(const GradArgs& g, const GradOut& o, const f32x16& acc, char* ep,
                                                  int lane, const GradKept& kept, float p, int row0, int rows, int tr,
                                                  int block)
{
    grad_block_to_lds(acc, ep, lane);
    float raw[16];
    const int row = tr + (lane >> 1), half = lane & 1;
    grad_read16(ep, lane >> 1, half, raw);
    uint32_t og[8], ou[8], oh[8];
    float dot = grad_swiglu16(raw, kept, p, og, ou, oh);
    grad_swiglu_store(o.o0, o.o1, g.F, row, block, half, og, ou, oh);
    dot += __shfl_xor(dot, 1);
    if (half == 0 && row < rows && 32 * block < g.F) g.part[(int64_t)(row0 + row) * (g.F / 32) + block] = dot;
}

// dx: columns 32 block .. of 32 rows, 16 bits a value (grad_dx.h)
__device__ __forceinline__ void grad_dx_block(const GradArgs& g, const GradOut& o, const f32x16& acc, char* ep, int lane,
                                              int tr, int block)
{
    grad_block_to_lds(acc, ep, lane);
    float v[16];
    const int row = tr + (lane >> 1), half = lane & 1;
    grad_read16(ep, lane >> 1, half, v);
    uint32_t w[8];
    const uint32_t byte = dx_pack16(v, w);
    const bool cols = 32 * block < g.H;
    const int at = cols ? (row * g.H + 32 * block + 16 * half) * 2 : 0x7ffffe00;
    __builtin_amdgcn_raw_buffer_store_b128(u32x4_t{w[0], w[1], w[2], w[3]}, o.o0, at, 0, 0);
    __builtin_amdgcn_raw_buffer_store_b128(u32x4_t{w[4], w[5], w[6], w[7]}, o.o0, at + 16, 0, 0);
    __builtin_amdgcn_raw_buffer_store_b8((uint8_t)byte, o.o1, cols ? row * (g.H / 16) + 2 * block + half : 0x7ffffe00, 0, 0);
}

// Stores of a 32 x 32 block that every lane issues (SWIGLU: and one of partial sums)
constexpr int grad_block_stores(bool swiglu) { return swiglu ? 6 : 3; }

// WIDE: 64-bit addresses, and a sum that may be an odd multiple of 32.  Otherwise the direct
// loads go through descriptors, the lane's offset fixed for the tile and the place in the
// sum a scalar offset, so that a stage's loads cost no vector instruction (16K tokens, the
// plain product 1250 us with 64-bit addresses, 1090 so).  A hidden size that is an odd multiple
// of 32 takes the product before the SwiGLU here with 64-bit addresses (its kept values wait
// behind the next tile's loads): 8,192 tokens, top-6 of 64 experts, FFN 1024, 367 us at hidden
// 2080 against 332 at 2112.
template <bool SWIGLU, bool WIDE>
__device__ __forceinline__ void grad_rows_tiles(const GradArgs& g)
{
    __shared__ __attribute__((aligned(1024))) char lds0[kBigStage];
    __shared__ __attribute__((aligned(1024))) char lds1[kBigStage];
    __shared__ __attribute__((aligned(1024))) char lds_x[8 * kBigEpi];

    const int lane = threadIdx.x & 63;
    const int wid = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wm = wid >> 2, wn = wid & 3;
    const int N = SWIGLU ? g.F : g.H;                    // output columns
    const int Kc = SWIGLU ? g.H : 2 * g.F;               // the sum
    const uint16_t* const A = SWIGLU ? g.d_out : g.dgu;
    const uint16_t* const W = SWIGLU ? g.w2 : g.w1;
    const int nt16 = Kc / 16, ks = N / 32;               // the packed section: rows / 16, columns / 32
    const int NT = (N + kBigTN - 1) / kBigTN;
    const int total = ld_const(&g.hdr->n_tiles_big) * NT;
    const int nst = (Kc + kBigKS - 1) / kBigKS;

    struct TilePos { int e, row0, rows, n0; };
    auto locate = [&](int tile) {
        const int mt = tile / NT;
        // the tiles of one expert keep their index range, walked column tile by column tile
        const int e = ld_const(&g.tiles_big[mt].x), first = ld_const(&g.tiles_big[mt].y);
        const int base = ld_const(g.offsets + e), cnt = ld_const(g.offsets + e + 1) - base;
        const int m_e = (cnt + kBigTM - 1) / kBigTM;
        const int b_e = mt - (first - base) / kBigTM;
        const int u = tile - b_e * NT;
        const int nt = u / m_e, mi = u - nt * m_e;
        return TilePos{e, base + mi * kBigTM, min(kBigTM, cnt - mi * kBigTM), nt * kBigTN};
    };

    // activations: lane -> row 32 wid + 8 i + lane / 8 (past the tile's rows the last one, or zeros),
    // 16-byte chunk (lane % 8) ^ (row % 8) at slot lane % 8.  Weights: this wave's 32-column
    // block of the tile, whose 4 row blocks of a stage are 4 KB contiguous; inside a 1 KB
    // block [chunk q of 8 columns][row n of 16] the 16-byte slot q 16 + n' holds row n' ^ 4 q,
    // so that the 4 rows x 4 chunks that 32 lanes read together lie on distinct banks.
    const char* arow[kBigALoads];
    const char* wbase;
    __amdgpu_buffer_rsrc_t ar, wr;
    int aoff[kBigALoads];
    int s32;
    const int wlane = 16 * ((lane & 48) | ((lane & 15) ^ (4 * (lane >> 4))));
    // the routes of a tile's rows: loaded before the K loop of the tile before it
    int look[kBigALoads] = {};
    auto lookup = [&](const TilePos& p) {
        if constexpr (SWIGLU)
#pragma unroll
            for (int i = 0; i < kBigALoads; ++i)
                look[i] = g.perm_src[p.row0 + min(32 * wid + 8 * i + (lane >> 3), p.rows - 1)];
    };
    auto sources = [&](const TilePos& p) {
#pragma unroll
        for (int i = 0; i < kBigALoads; ++i) {
            const int rr = 32 * wid + 8 * i + (lane >> 3);
            int64_t src = p.row0 + min(rr, p.rows - 1);
            if constexpr (SWIGLU) {
                const int tok = look[i] / g.topk;
                grad_leave_token(g, p.row0, p.n0 == 0 ? p.rows : 0, rr, tok, lane);
                src = tok;
            }
            if constexpr (WIDE) arow[i] = (const char*)(A + src * Kc);
            else if (SWIGLU)
                aoff[i] = (int)src * 2 * Kc + 16 * ((lane & 7) ^ (rr & 7));
            else    // (rows past the tile's: zeros, 1085 -> 1067 us against the last row again; the
                    // gathering product got slower with them, 778 -> 817)
                aoff[i] = rr < p.rows ? rr * 2 * Kc + 16 * ((lane & 7) ^ (rr & 7)) : (int)0x80000000;
        }
        const uint16_t* w = W + (int64_t)p.e * Kc * N;
        if constexpr (WIDE) wbase = (const char*)w;
        else {
            ar = __builtin_amdgcn_make_buffer_rsrc((void*)(SWIGLU ? A : A + (int64_t)p.row0 * Kc), (short)0, 0x7fffffff,
                                                   kBigRsrcWord3);
            wr = __builtin_amdgcn_make_buffer_rsrc((void*)w, (short)0, 2 * Kc * N, kBigRsrcWord3);
        }
        s32 = min(p.n0 / 32 + wid, ks - 1);
    };
    auto issue = [&](char* st, int s) {
        const int grp = s >> 3;
        const int w = min(32, nt16 - 32 * grp);
        if constexpr (!WIDE) {
#pragma unroll
            for (int i = 0; i < kBigALoads; ++i)
                __builtin_amdgcn_raw_ptr_buffer_load_lds(ar, (lds_void_t*)(st + (4 * wid + i) * 1024), 16, aoff[i], 128 * s,
                                                         0, 0);
            const int wo = (grp * 32 * ks + s32 * w + ((4 * s) & 31)) * 1024;
#pragma unroll
            for (int i = 0; i < 4; ++i)
                __builtin_amdgcn_raw_ptr_buffer_load_lds(wr, (lds_void_t*)(st + kBigWOff + (4 * wid + i) * 1024), 16, wlane,
                                                         wo + 1024 * i, 0, 0);
            return;
        }
#pragma unroll
        for (int i = 0; i < kBigALoads; ++i) {
            const int rr = 32 * wid + 8 * i + (lane >> 3);
            const int c = 8 * s + ((lane & 7) ^ (rr & 7));
            big_load_block(c < Kc / 8 ? arow[i] + 16 * c : (const char*)grad_zeros, st + (4 * wid + i) * 1024);
        }
        // (the last stage of a sum that is an odd multiple of 32 holds zeros on both sides: zeros
        // against weights would make an infinite weight's sums NaN)
        const char* wp = wbase + ((int64_t)grp * 32 * ks + (int64_t)s32 * w + ((4 * s) & 31)) * 1024;
#pragma unroll
        for (int i = 0; i < 4; ++i)
            big_load_block((4 * s + i < nt16 ? wp + i * 1024 : (const char*)grad_zeros) + wlane,
                           st + kBigWOff + (4 * wid + i) * 1024);
    };
    // fragments of sub-step Q: A row l % 32, chunk 2 Q + l / 32 at its slot; B one 1 KB
    // block (16 of the sum x 32 columns), rows 8 (l / 32) + {0, 4} + (l % 16) / 4
    int a_off[4], b_off[2];
    {
        const int r = lane & 31, hi = lane >> 5;
#pragma unroll
        for (int q = 0; q < 4; ++q) a_off[q] = (128 * wm + r) * 128 + 16 * ((2 * q + hi) ^ (r & 7));
        const int j = lane & 15, q = 2 * ((lane >> 4) & 1) + ((j & 3) >> 1);
#pragma unroll
        for (int t = 0; t < 2; ++t)
            b_off[t] = kBigWOff + 8 * wn * 1024 + q * 256 + 16 * ((8 * hi + 4 * t + (j >> 2)) ^ (4 * q)) + 8 * (j & 1);
    }
    auto read = [&](auto QC, const char* st, GradFrag& f) {
        constexpr int Q = decltype(QC)::value;
#pragma unroll
        for (int j = 0; j < 2; ++j)
            f.b[j] = grad_tr(st + b_off[0] + (4 * j + Q) * 1024, b_off[1] - b_off[0]);
#pragma unroll
        for (int i = 0; i < 4; ++i) f.a[i] = big_frag<OpBf16>(st + a_off[Q] + 32 * 128 * i);
    };

    const GradRange range = grad_range(total);
    int tile = range.first;
    if (tile >= range.end) return;
    TilePos pos = locate(tile), npos = pos;
    lookup(pos);
    sources(pos);
    issue(lds0, 0);
    issue(lds1, min(1, nst - 1));
    constexpr int kStores = 8 * grad_block_stores(SWIGLU);
    constexpr int kLook = SWIGLU ? kBigALoads : 0;
    grad_dummy_stores<kStores>(g.dgu, lane);
    char* const ep = lds_x + wid * kBigEpi;
    while (true) {
        const int row0 = pos.row0, rows = pos.rows, n0 = pos.n0;
        f32x16 acc[4][2];
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 2; ++j)
#pragma unroll
                for (int v = 0; v < 16; ++v) acc[i][j][v] = 0.0f;
        const int next = tile + range.step;
        const bool more = next < range.end;
        if (more) npos = locate(next);
        lookup(npos);
        grad_kloop<8, kStores + kLook>(nst, lds0, lds1, acc, read, issue);
        __builtin_amdgcn_s_waitcnt(0xC07F);         // lgkmcnt(0)
        __builtin_amdgcn_s_barrier();
        int elane = lane;
        asm volatile("" : "+v"(elane));

        // SWIGLU: everything the epilogue reads from memory, before the next tile's loads, by 8
        // blocks of 32 x 32 (row block q / 2, column block q % 2); the second half of them after
        // the first two (all at once spilled)
        GradKept kept[8];
        float pr0 = 0.0f, pr1 = 0.0f;
        const int prow = elane >> 1, ib = n0 / 32 + 2 * wn;
        auto load_kept = [&](int q) {
            kept[q] = grad_kept(g, row0 + min(128 * wm + 32 * (q >> 1) + prow, rows - 1),
                                min(ib + (q & 1), g.F / 32 - 1), elane & 1);
        };
        if constexpr (SWIGLU) {
            const int r0 = min(128 * wm + elane, rows - 1), r1 = min(128 * wm + elane + 64, rows - 1);
            pr0 = g.prob[g.perm_src[row0 + r0]];
            pr1 = g.prob[g.perm_src[row0 + r1]];
#pragma unroll
            for (int q = 0; q < 4; ++q) load_kept(q);
        }
        sources(npos);
        issue(lds0, 0);
        issue(lds1, min(1, nst - 1));

        const GradOut out = grad_out<SWIGLU>(g, row0, rows);
#pragma unroll
        for (int q = 0; q < 8; ++q) {
            const int i = q >> 1, tr = 128 * wm + 32 * i;
            if constexpr (SWIGLU) {
                if (q == 2) {
                    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
                    for (int n = 4; n < 8; ++n) load_kept(n);
                }
                __builtin_amdgcn_sched_barrier(0);
                const float p = lane_value(4 * (32 * (i & 1) + prow), i < 2 ? pr0 : pr1);
                grad_swiglu_block(g, out, acc[i][q & 1], ep, elane, kept[q], p, row0, rows, tr, ib + (q & 1));
            } else {
                grad_dx_block(g, out, acc[i][q & 1], ep, elane, tr, ib + (q & 1));
            }
        }
        if (!more) {
            BIG_WAIT_VMCNT(0);          // the repeated loads land before the LDS is released
            break;
        }
        tile = next;
        pos = npos;
    }
}

// The 64-row tiles (experts with at most 128 rows): 64 x 256, 8 waves of 64 x 32, the
// arithmetic of the 256-row tiles (the same MFMAs in the same order, so a row's results do
// not depend on the tile that computes them).  The weights stream from memory, each byte for
// at most 64 rows: three LDS stages of 64 along the sum (8 KB of rows, 32 KB of weights), two
// of them in flight, a barrier a stage.  Measured at 1,000 tokens, top-6 of 64 experts, hidden
// 2048, FFN 1024: 88 us before the SwiGLU, 138 after it, bound by the 1.43 GB that the latter
// brings through the L2s at 10.3 TB/s, 2 of 34 stages a tile its last one again (125 with the
// MFMAs taken out of a copy, 118 with all weights in the L2s; no change with four stages or with
// fragments read a stage ahead).  With the
// 256-row tiles in their place (three quarters and more of every tile empty) both products
// took 467 us instead of 266 at 1,000 tokens on 64 experts, and 42 instead of 20 at 64 tokens.
// take_big: this launch also takes the 256-row tiles, as four of 64 rows each.
constexpr int kGradSmallStage = 40 * 1024;
constexpr int kGradSmallW = 8 * 1024;           // weight part of a stage
constexpr int kGradSmallLoads = 5;              // direct loads per wave per stage

template <bool SWIGLU>
__device__ __forceinline__ void grad_small_tiles(const GradArgs& g, bool take_big)
{
    __shared__ __attribute__((aligned(1024))) char lds0[kGradSmallStage];
    __shared__ __attribute__((aligned(1024))) char lds1[kGradSmallStage];
    __shared__ __attribute__((aligned(1024))) char lds2[kGradSmallStage];
    __shared__ __attribute__((aligned(1024))) char lds_x[8 * kBigEpi];

    const int lane = threadIdx.x & 63;
    const int wid = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int N = SWIGLU ? g.F : g.H;                    // output columns
    const int Kc = SWIGLU ? g.H : 2 * g.F;               // the sum
    const uint16_t* const A = SWIGLU ? g.d_out : g.dgu;
    const uint16_t* const W = SWIGLU ? g.w2 : g.w1;
    const int nt16 = Kc / 16, ks = N / 32;
    const int NT = (N + kBigTN - 1) / kBigTN;
    const int n_small = ld_const(&g.hdr->n_tiles), n_big = take_big ? ld_const(&g.hdr->n_tiles_big) : 0;
    const int total = (n_small + 4 * n_big) * NT;
    const int nst = (Kc + kBigKS - 1) / kBigKS;

    struct TilePos { int e, row0, rows, n0; };
    auto locate = [&](int tile) {
        const int mt = tile / NT;
        const bool big = mt >= n_small;
        const int2* te = big ? g.tiles_big + ((mt - n_small) >> 2) : g.tiles + mt;
        const int e = ld_const(&te->x), row0 = ld_const(&te->y) + (big ? kBM * ((mt - n_small) & 3) : 0);
        return TilePos{e, row0, min(kBM, ld_const(g.offsets + e + 1) - row0), (tile - mt * NT) * kBigTN};
    };
    // the next tile with rows (the last quarters of a 256-row tile may have none)
    auto advance = [&](int tile, TilePos& p) {
        for (; tile < total; tile += (int)gridDim.x) {
            p = locate(tile);
            if (p.rows > 0) break;
        }
        return tile;
    };

    // as in the 256-row tiles: rows 8 wid + lane / 8, the wave's 32-column weight block
    const char* arow;
    const char* wbase;
    int s32, look = 0, route[2] = {};
    const int myrow = 8 * wid + (lane >> 3), achunk = (lane & 7) ^ (lane >> 3);
    const int wlane = 16 * ((lane & 48) | ((lane & 15) ^ (4 * (lane >> 4))));
    auto lookup = [&](const TilePos& p) {
        if constexpr (SWIGLU) {
            look = g.perm_src[p.row0 + min(myrow, p.rows - 1)];
#pragma unroll
            for (int i = 0; i < 2; ++i) route[i] = g.perm_src[p.row0 + min(32 * i + (lane >> 1), p.rows - 1)];
        }
    };
    auto sources = [&](const TilePos& p) {
        int64_t src = p.row0 + min(myrow, p.rows - 1);
        if constexpr (SWIGLU) {
            const int tok = look / g.topk;
            // (the routes have landed with it: awaited here, not among the next loads in flight)
            asm volatile("" : "+v"(route[0]), "+v"(route[1]));
            grad_leave_token(g, p.row0, p.n0 == 0 ? p.rows : 0, myrow, tok, lane);
            src = tok;
        }
        arow = (const char*)(A + src * Kc);
        wbase = (const char*)(W + (int64_t)p.e * Kc * N);
        s32 = min(p.n0 / 32 + wid, ks - 1);
    };
    auto issue = [&](char* st, int s) {
        const int c = 8 * s + achunk;
        big_load_block(c < Kc / 8 ? arow + 16 * c : (const char*)grad_zeros, st + wid * 1024);
        const int grp = s >> 3;
        const int w = min(32, nt16 - 32 * grp);
        const char* wp = wbase + ((int64_t)grp * 32 * ks + (int64_t)s32 * w + ((4 * s) & 31)) * 1024;
#pragma unroll
        for (int i = 0; i < 4; ++i)             // (past the sum's end zeros, as in the 256-row tiles)
            big_load_block((4 * s + i < nt16 ? wp + i * 1024 : (const char*)grad_zeros) + wlane,
                           st + kGradSmallW + (4 * wid + i) * 1024);
    };
    int a_off[4], b_off[2];
    {
        const int r = lane & 31, hi = lane >> 5;
#pragma unroll
        for (int q = 0; q < 4; ++q) a_off[q] = r * 128 + 16 * ((2 * q + hi) ^ (r & 7));
        const int j = lane & 15, q = 2 * ((lane >> 4) & 1) + ((j & 3) >> 1);
#pragma unroll
        for (int t = 0; t < 2; ++t)
            b_off[t] = kGradSmallW + 4 * wid * 1024 + q * 256 + 16 * ((8 * hi + 4 * t + (j >> 2)) ^ (4 * q)) + 8 * (j & 1);
    }

    TilePos pos{}, npos{};
    int tile = advance(xcd_first_tile(), pos);
    if (tile >= total) return;
    constexpr int kStores = 2 * grad_block_stores(SWIGLU);
    // the epilogue's own loads (kept values and probabilities) and the next tile's lookup, all
    // before the K loop: after it they were two round trips of every tile
    constexpr int kLook = SWIGLU ? 11 : 0;
    lookup(pos);
    sources(pos);
    issue(lds0, 0);
    issue(lds1, min(1, nst - 1));
    grad_dummy_stores<kStores>(g.dgu, lane);
    char* const ep = lds_x + wid * kBigEpi;
    while (true) {
        const int row0 = pos.row0, rows = pos.rows, n0 = pos.n0;
        npos = pos;
        const int next = advance(tile + (int)gridDim.x, npos);
        const bool more = next < total;
        if (!more) npos = pos;
        const int half = lane & 1, prow = lane >> 1;
        const int ib = n0 / 32 + wid;
        GradKept kept[2];
        float p[2];
        if constexpr (SWIGLU) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                p[i] = g.prob[route[i]];
                kept[i] = grad_kept(g, row0 + min(32 * i + prow, rows - 1), min(ib, g.F / 32 - 1), half);
            }
        }
        lookup(npos);
        f32x16 acc[2];
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int v = 0; v < 16; ++v) acc[i][v] = 0.0f;
        // stage s is in cur, stage s + 1 in flight; stage s + 2 goes where stage s - 1 was
        // (past the last stage that one again, which no later read of the tile uses).  AFTER:
        // what is younger than stage s + 1 and may still be in flight, at stage 0 the stores of
        // the tile before and this tile's lookup.
        auto step = [&](auto AC, int s, const char* cur, char* refill) {
            BIG_WAIT_VMCNT(kGradSmallLoads + decltype(AC)::value);
            __builtin_amdgcn_s_waitcnt(0xC07F);     // lgkmcnt(0): this wave's reads of stage s - 1 are done
            __builtin_amdgcn_s_barrier();
            issue(refill, min(s + 2, nst - 1));
            bf16x8 a[4][2], b[4];
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                b[q] = grad_tr(cur + b_off[0] + q * 1024, b_off[1] - b_off[0]);
#pragma unroll
                for (int i = 0; i < 2; ++i) a[q][i] = big_frag<OpBf16>(cur + a_off[q] + 4096 * i);
            }
#pragma unroll
            for (int q = 0; q < 4; ++q)
#pragma unroll
                for (int i = 0; i < 2; ++i)
                    acc[i] = grad_mfma(a[q][i], b[q], acc[i]);
        };
        using Now = std::integral_constant<int, 0>;
        step(std::integral_constant<int, kStores + kLook>{}, 0, lds0, lds2);
        int s = 1;
        for (; s + 3 <= nst; s += 3) {
            step(Now{}, s, lds1, lds0);
            step(Now{}, s + 1, lds2, lds1);
            step(Now{}, s + 2, lds0, lds2);
        }
        if (s < nst) {
            step(Now{}, s, lds1, lds0);
            if (s + 1 < nst) step(Now{}, s + 1, lds2, lds1);
        }
        int elane = lane;
        asm volatile("" : "+v"(elane));
        __builtin_amdgcn_s_waitcnt(0xC07F);         // lgkmcnt(0)
        __builtin_amdgcn_s_barrier();               // every wave has read its last stage
        sources(npos);
        issue(lds0, 0);
        issue(lds1, min(1, nst - 1));
        const GradOut out = grad_out<SWIGLU>(g, row0, rows);
#pragma unroll
        for (int i = 0; i < 2; ++i)
            if constexpr (SWIGLU)
                grad_swiglu_block(g, out, acc[i], ep, elane, kept[i], p[i], row0, rows, 32 * i, ib);
            else
                grad_dx_block(g, out, acc[i], ep, elane, 32 * i, ib);
        if (!more) {
            BIG_WAIT_VMCNT(0);          // the repeated loads land before the LDS is released
            break;
        }
        tile = next;
        pos = npos;
    }
}

// ---------------------------------------------------------------- weight products

// The number of experts e < E whose work before them, offsets[e] + kGradTileRows e, is at
// most `target` (it grows with e), counted by all lanes of a wave at once
constexpr int kGradTileRows = 256;      // rows that a tile's fixed cost weighs as much as
__device__ __forceinline__ int grad_experts_below(const int32_t* offsets, int E, int64_t target, int lane)
{
    int n = 0;
    for (int e0 = 0; e0 < E; e0 += 64) {
        const int e = e0 + lane;
        const bool le = e < E && (int64_t)offsets[min(e, E - 1)] + (int64_t)kGradTileRows * e <= target;
        n += __popcll(__ballot(le));
    }
    return n;
}

// The first of `per_e` E tiles of part x of 8: the parts are contiguous and hold about the
// same work, a tile of expert e weighing its rows + kGradTileRows (with parts of equally
// many tiles the XCD of the fullest experts ran on alone)
__device__ __forceinline__ int grad_part(const int32_t* offsets, int E, int per_e, int x, int lane)
{
    if (x <= 0) return 0;
    if (x >= 8) return E * per_e;
    const int64_t target = ((int64_t)ld_const(offsets + E) + (int64_t)kGradTileRows * E) * x / 8;
    const int e = __builtin_amdgcn_readfirstlane(grad_experts_below(offsets, E, target, lane) - 1);      // >= 0: expert 0 has none before it
    const int64_t row0 = ld_const(offsets + e);
    const int64_t before = row0 + (int64_t)kGradTileRows * e;
    const int64_t own = ld_const(offsets + e + 1) - row0 + kGradTileRows;
    return e * per_e + (int)((target - before) * per_e / own);
}

// FP32: gradients of the weights in fp32, else bf16.  WIDE: 64-bit addresses; otherwise
// descriptors of the expert's own rows and of the gathered matrix, and an offset past them
// for rows past the expert's last (a load out of a descriptor's range brings zeros).
template <bool FP32, bool WIDE>
__device__ __forceinline__ void grad_weight_tiles(const GradArgs& g)
{
    constexpr int kHalf = kBigStage / 2;            // 32 rows of P, then of Q, 512 bytes each
    constexpr int kHalfQ = kHalf / 2;
    __shared__ __attribute__((aligned(1024))) char lds0[kHalf];
    __shared__ __attribute__((aligned(1024))) char lds1[kHalf];
    __shared__ __attribute__((aligned(1024))) char lds2[kHalf];
    __shared__ __attribute__((aligned(1024))) char lds3[kHalf];
    __shared__ __attribute__((aligned(1024))) char lds_x[8 * kBigEpi];

    const int lane = threadIdx.x & 63;
    const int wid = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wm = wid >> 2, wn = wid & 3;
    const int H = g.H, F = g.F;
    const int mt1 = (2 * F + kBigTM - 1) / kBigTM, nt1 = (H + kBigTN - 1) / kBigTN;
    const int mt2 = (H + kBigTM - 1) / kBigTM, nt2 = (F + kBigTN - 1) / kBigTN;
    const int t1 = mt1 * nt1, per_e = t1 + mt2 * nt2;

    // a tile: M columns of the row matrix P against N columns of Q, over the expert's rows.
    // W1: P = dgu (its own rows), Q = x (gathered); W2: P = d_out (gathered), Q = hp.
    struct TilePos { int e, row0, cnt, m0, n0, w2; };
    auto locate = [&](int tile) {
        const int e = tile / per_e;
        int u = tile - e * per_e;
        const int w2 = u >= t1;
        if (w2) u -= t1;
        const int nt = w2 ? nt2 : nt1;
        const int mi = u / nt;
        const int base = ld_const(g.offsets + e);
        return TilePos{e, base, ld_const(g.offsets + e + 1) - base, mi * kBigTM, (u - mi * nt) * kBigTN, w2};
    };

    // 16-byte chunk c of row r lies at chunk c ^ 4 (r % 4), so that the 4 rows x 4 chunks that
    // 32 lanes read together lie on distinct banks.  Wave w loads rows 4 w .. 4 w + 3 of both
    // matrices, two rows an instruction.  Rows past the expert's last read zeros on both sides.
    // The own rows' pointers advance by 32 rows a half; a gathered row is one multiply-add of
    // its token, which comes by a scalar load a half ahead from the table that the first
    // product left (with the row and its token worked out anew each stage these were 4.6
    // vector instructions per MFMA).
    // The loads run ahead across tiles: a half that the tile has no more use for is refilled
    // with the next tile's, whose sources are worked out before the tile's K loop.
    const int odd = lane >> 5;
    struct Tok { int t[4]; };
    struct Src {
        const char *own[2], *gcol[2];          // WIDE: own rows, gathered matrix, at the lane's column
        const uint16_t *obase, *gbase;         // else what their descriptors hold, and offsets
        int orecs;
        int ooff[2], goff[2];
        uint32_t ostep;                        // bytes of 32 own rows
        int left;                              // rows from the wave's first of the half on
        int oslot, gslot;                      // where own and gathered rows lie in a half
    };
    auto tokens = [&](const int32_t* p) { return Tok{{ld_const(p), ld_const(p + 1), ld_const(p + 2), ld_const(p + 3)}}; };
    auto sources = [&](const TilePos& p) {
        Src c;
        const int ow = p.w2 ? F : 2 * F;                         // columns of the own matrix
        const int o0 = p.w2 ? p.n0 : p.m0, g0 = p.w2 ? p.m0 : p.n0;
        const uint16_t* ob = p.w2 ? g.hp : g.dgu;
        const uint16_t* gb = p.w2 ? g.d_out : g.x;
        c.oslot = p.w2 ? kHalfQ : 0;
        c.gslot = p.w2 ? 0 : kHalfQ;
        c.ostep = 64u * (uint32_t)ow;
        c.left = p.cnt - 4 * wid;
        const int row = 4 * wid + odd;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            // the slot's chunk; a column past the matrix reads its last chunk (never stored)
            const int k = 8 * ((lane & 31) ^ (4 * (2 * i + odd)));
            if constexpr (WIDE) {
                c.gcol[i] = (const char*)(gb + min(g0 + k, H - 8));
                c.own[i] = (const char*)(ob + min(o0 + k, ow - 8) + ((int64_t)p.row0 + row + 2 * i) * ow);
            } else {
                c.goff[i] = 2 * min(g0 + k, H - 8);
                c.ooff[i] = 2 * (min(o0 + k, ow - 8) + (row + 2 * i) * ow);
            }
        }
        c.obase = ob + (int64_t)p.row0 * ow;
        c.gbase = gb;
        c.orecs = WIDE ? 0 : p.cnt * ow * 2;
        return c;
    };
    // half `h` of c's rows into st, h counted from where c's offsets stand
    auto issue_rows = [&](char* st, const Src& c, int h, const Tok& t) {
        const int left = c.left - 32 * h;
        const uint32_t pitch = 2u * (uint32_t)H;
        __amdgpu_buffer_rsrc_t orsrc, grsrc;
        if constexpr (!WIDE) {
            orsrc = __builtin_amdgcn_make_buffer_rsrc((void*)c.obase, (short)0, c.orecs, kBigRsrcWord3);
            grsrc = __builtin_amdgcn_make_buffer_rsrc((void*)c.gbase, (short)0, 0x7fffffff, kBigRsrcWord3);
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            void* const od = st + c.oslot + (2 * wid + i) * 1024;
            void* const gd = st + c.gslot + (2 * wid + i) * 1024;
            if constexpr (WIDE) {
                const bool in = left > 2 * i + odd;
                const uint32_t tk = (uint32_t)(odd ? t.t[2 * i + 1] : t.t[2 * i]);
                big_load_block(in ? c.own[i] + (uint64_t)c.ostep * h : (const char*)grad_zeros, od);
                big_load_block(in ? c.gcol[i] + (uint64_t)tk * pitch : (const char*)grad_zeros, gd);
            } else {
                // (scalar: the offsets of the instruction's two rows)
                const uint32_t s0 = left > 2 * i ? (uint32_t)t.t[2 * i] * pitch : 0x80000000u;
                const uint32_t s1 = left > 2 * i + 1 ? (uint32_t)t.t[2 * i + 1] * pitch : 0x80000000u;
                __builtin_amdgcn_raw_ptr_buffer_load_lds(orsrc, (lds_void_t*)od, 16, c.ooff[i] + (int)c.ostep * h, 0, 0, 0);
                __builtin_amdgcn_raw_ptr_buffer_load_lds(grsrc, (lds_void_t*)gd, 16, (int)(odd ? s1 : s0) + c.goff[i], 0, 0, 0);
            }
        }
    };
    // cur stands at the tile's next half to issue (the fifth when its K loop begins), with that
    // half's tokens; nxt at the next tile's first, with the tokens of its first four
    Src cur, nxt;
    const int32_t* toks = nullptr;
    Tok tok, ahead[4];
    int to_issue = 0;                      // halves of the tile that are not issued yet
    auto look_ahead = [&](const TilePos& p) {
        nxt = sources(p);
#pragma unroll
        for (int h = 0; h < 4; ++h) ahead[h] = tokens(g.row_tok + p.row0 + 32 * h + 4 * wid);
    };
    auto issue = [&](auto SC, char* st) {
        // (one set of loads whose sources are chosen: with a set on either side of a branch the
        // compiler waited for all in flight before later fragment reads)
        constexpr int j = decltype(SC)::value;
        const bool own_half = to_issue > 0;
        auto pick = [&](auto a, auto b) { return own_half ? a : b; };       // (by value)
        Src c = nxt;
        Tok t = ahead[j];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            if constexpr (WIDE) {
                c.own[i] = pick(cur.own[i], nxt.own[i] + (uint64_t)nxt.ostep * j);
                c.gcol[i] = pick(cur.gcol[i], nxt.gcol[i]);
                cur.own[i] += cur.ostep;
            } else {
                c.ooff[i] = pick(cur.ooff[i], nxt.ooff[i] + (int)nxt.ostep * j);
                c.goff[i] = pick(cur.goff[i], nxt.goff[i]);
                cur.ooff[i] += (int)cur.ostep;
            }
        }
        c.obase = pick(cur.obase, nxt.obase);
        c.gbase = pick(cur.gbase, nxt.gbase);
        c.orecs = pick(cur.orecs, nxt.orecs);
        c.left = pick(cur.left, nxt.left - 32 * j);
        c.oslot = pick(cur.oslot, nxt.oslot);
        c.gslot = pick(cur.gslot, nxt.gslot);
#pragma unroll
        for (int i = 0; i < 4; ++i) t.t[i] = pick(tok.t[i], ahead[j].t[i]);
        issue_rows(st, c, 0, t);
        cur.left -= 32;
        toks += 32;
        tok = tokens(pick(toks, g.row_tok));      // (the table is 512 entries longer than the rows)
        --to_issue;
    };
    auto stages_of = [&](const TilePos& p) { return (p.cnt + 63) / 64; };
    // the halves of the next tile that the K loop of `p` has not issued (bit j: slot j), then
    // the next tile becomes the current one
    auto turn = [&](int missing, const TilePos& p) {
        if (missing & 1) issue_rows(lds0, nxt, 0, ahead[0]);
        if (missing & 2) issue_rows(lds1, nxt, 1, ahead[1]);
        if (missing & 4) issue_rows(lds2, nxt, 2, ahead[2]);
        if (missing & 8) issue_rows(lds3, nxt, 3, ahead[3]);
        cur = nxt;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            if constexpr (WIDE) cur.own[i] += 4 * (uint64_t)cur.ostep;
            else cur.ooff[i] += 4 * (int)cur.ostep;
        }
        cur.left -= 128;
        to_issue = 2 * stages_of(p) - 4;
        toks = g.row_tok + p.row0 + 128 + 4 * wid;
        tok = tokens(toks);
    };
    // fragments of sub-step Q of a half: rows 16 Q + 8 (l / 32) + {0, 4} + (l % 16) / 4, the
    // lane's 4 columns of each 32-column block
    int a_off[4], b_off[2];
    {
        const int j = lane & 15, jj = j >> 2;
        const int base = (8 * (lane >> 5) + jj) * 512 + 16 * (2 * ((lane >> 4) & 1) + ((j & 3) >> 1)) + 8 * (j & 1);
#pragma unroll
        for (int i = 0; i < 4; ++i) a_off[i] = base + 64 * ((4 * wm + i) ^ jj);
#pragma unroll
        for (int i = 0; i < 2; ++i) b_off[i] = kHalfQ + base + 64 * ((2 * wn + i) ^ jj);
    }
    auto read = [&](auto QC, const char* st, GradFrag& f) {
        constexpr int Q = decltype(QC)::value;
#pragma unroll
        for (int j = 0; j < 2; ++j) f.b[j] = grad_tr(st + b_off[j] + 8192 * Q, 2048);
#pragma unroll
        for (int i = 0; i < 4; ++i) f.a[i] = grad_tr(st + a_off[i] + 8192 * Q, 2048);
    };

    const int xcd = blockIdx.x & 7;
    const int end = grad_part(g.offsets, g.E, per_e, xcd + 1, lane);
    int tile = grad_part(g.offsets, g.E, per_e, xcd, lane) + (int)(blockIdx.x >> 3);
    if (tile >= end) return;
    TilePos pos = locate(tile), npos = pos;
    look_ahead(pos);
    turn(15, pos);
    constexpr int kStores = FP32 ? 32 : 16;
    grad_dummy_stores<kStores>(g.dgu, lane);
    char* const ep = lds_x + wid * kBigEpi;
    while (true) {
        f32x16 acc[4][2];
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 2; ++j)
#pragma unroll
                for (int v = 0; v < 16; ++v) acc[i][j][v] = 0.0f;
        const int next = tile + (int)(gridDim.x >> 3);
        const bool more = next < end;
        if (more) npos = locate(next);
        look_ahead(npos);
        const int nst = stages_of(pos);
        if (nst > 0)
            grad_kloop_halves<12, kStores, 4>(nst, lds0, lds1, lds2, lds3, acc, read, issue);
        else
            BIG_WAIT_VMCNT(kStores);                // its loads land before the next tile's go out
        __builtin_amdgcn_s_waitcnt(0xC07F);         // lgkmcnt(0)
        __builtin_amdgcn_s_barrier();
        // a K loop of n stages refills 2 n - 1 halves: all but its last, or with one stage the first
        turn(nst == 0 ? 15 : nst == 1 ? 14 : nst & 1 ? 2 : 8, npos);

        int elane = lane;
        asm volatile("" : "+v"(elane));
        const int M = pos.w2 ? H : 2 * F, N = pos.w2 ? F : H;
        void* const out = pos.w2 ? g.d_w2 : g.d_w1;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            // a 32-row block: of the interleaved order of W1, gate and up by turns
            const int blk = pos.m0 / 32 + 4 * wm + i;
            const int row = pos.w2 ? 32 * blk : (blk & 1 ? F : 0) + 32 * (blk >> 1);
            const int64_t at = ((int64_t)pos.e * M + row) * N;
            const int recs = 32 * blk < M ? 32 * N * (FP32 ? 4 : 2) : 0;
            const __amdgpu_buffer_rsrc_t orr = __builtin_amdgcn_make_buffer_rsrc(
                FP32 ? (void*)((float*)out + at) : (void*)((uint16_t*)out + at), (short)0, recs, kBigRsrcWord3);
            // a lane's 16 bytes: row elane / 8 of 8, chunk elane % 8 of a row's 128 bytes.  The
            // gradients are not read here again: non-temporal (16K tokens 1781 -> 1737 us,
            // 4,096 776 -> 751, 1,000 the same)
            const int c = elane & 7;
            if constexpr (FP32) {
#pragma unroll
                for (int jb = 0; jb < 2; ++jb) {
                    grad_block_to_lds(acc[i][jb], ep, elane);
                    const int col = pos.n0 + 64 * wn + 32 * jb + 4 * c;
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const int rr = (elane >> 3) + 8 * k;
                        const u32x4_t val = *(const u32x4_t*)(ep + grad_at(rr, c));
                        __builtin_amdgcn_raw_buffer_store_b128(val, orr, col < N ? (rr * N + col) * 4 : 0x7ffffff0, 0,
                                                               kNonTemporal);
                    }
                }
            } else {
                grad_blocks_to_lds_bf16(acc[i], ep, elane);
                const int col = pos.n0 + 64 * wn + 8 * c;
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const int rr = (elane >> 3) + 8 * k;
                    const u32x4_t val = *(const u32x4_t*)(ep + grad_at(rr, c));
                    __builtin_amdgcn_raw_buffer_store_b128(val, orr, col < N ? (rr * N + col) * 2 : 0x7ffffff0, 0, kNonTemporal);
                }
            }
        }
        if (!more) {
            BIG_WAIT_VMCNT(0);          // the repeated loads land before the LDS is released
            break;
        }
        tile = next;
        pos = npos;
    }
}

}  // namespace moe
