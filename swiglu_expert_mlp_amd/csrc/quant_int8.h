// int8 rows: quantization of the activations (one scale per row) and the
// kernel-weight buffer of the int8 experts (one scale per weight row).
//
//   s = amax / 127,  q = sign(v) floor(127 |v| / amax + 1/2)
//
// (round half away from zero), amax the row's largest magnitude.  A row of
// zeros has scale 0 and codes 0; a row that holds an infinity or a NaN has
// scale NaN, so that every output it reaches is NaN.
//
// The kernels evaluate q as round-to-nearest of v r with r = 127 / amax
// (1 + 2^-20).  For bf16 v and amax this is the formula's value exactly: with
// |v| = a 2^i and amax = b 2^j (a, b <= 255), 127 |v| / amax is a tie only if
// 254 a = (2 n + 1) b 2^m, and otherwise lies at least 1 / (2 b 2^m) from one,
// a relative distance of at least 1 / (2 * 127 * 255) = 1.5e-5; r is off by a
// relative 2^-20 plus three roundings of 2^-24, that is by 0.7e-6 to 1.2e-6, so
// ties are pushed outwards and nothing else crosses one.  The product and the
// rounding are one fused multiply-add onto 1.5 * 2^23, whose low byte is q.
#pragma once

#include "common.h"

namespace moe {

typedef unsigned short u16x2 __attribute__((ext_vector_type(2)));

// magnitudes of a pair of bf16, and the larger ones of two pairs
__device__ __forceinline__ uint32_t pair_max(uint32_t m, uint32_t w)
{
    const u16x2 a = __builtin_bit_cast(u16x2, m), b = __builtin_bit_cast(u16x2, w & 0x7fff7fffu);
    return __builtin_bit_cast(uint32_t, __builtin_elementwise_max(a, b));
}

// largest value of the 16 lanes of a DPP row, in all of them
__device__ __forceinline__ int row16_max_int(int v)
{
    v = max(v, __builtin_amdgcn_update_dpp(v, v, 0x121, 0xf, 0xf, false));   // row_ror 1, 2, 4, 8
    v = max(v, __builtin_amdgcn_update_dpp(v, v, 0x122, 0xf, 0xf, false));
    v = max(v, __builtin_amdgcn_update_dpp(v, v, 0x124, 0xf, 0xf, false));
    v = max(v, __builtin_amdgcn_update_dpp(v, v, 0x128, 0xf, 0xf, false));
    return v;
}

// A row's quantizer from the bf16 bits of its largest magnitude.
struct RowQuant {
    float pre;      // 2^64 for rows below 2^-60, whose 127 / amax could overflow
    float mul;      // 127 / (amax pre) (1 + 2^-20); 0 for a row of zeros
    bool bad;       // the row holds an infinity or a NaN
    float scale;
};

__device__ __forceinline__ RowQuant row_quant(uint32_t amax_bits)
{
    RowQuant q;
    const float amax = bf16_bits_to_f32(amax_bits);
    q.bad = amax_bits >= 0x7f80u;
    q.pre = amax < 0x1p-60f ? 0x1p64f : 1.0f;
    q.mul = amax_bits == 0 || q.bad ? 0.0f : 127.0f / (amax * q.pre) * (1.0f + 0x1p-20f);
    q.scale = q.bad ? __uint_as_float(0x7fc00000u) : amax / 127.0f;
    return q;
}

// four codes (one per byte) of two pairs of bf16
__device__ __forceinline__ uint32_t quant4(uint32_t w0, uint32_t w1, const RowQuant& q)
{
    constexpr float kMagic = 12582912.0f;        // 1.5 * 2^23
    const float v[4] = {bf16_bits_to_f32(w0 & 0xffffu), __uint_as_float(w0 & 0xffff0000u),
                        bf16_bits_to_f32(w1 & 0xffffu), __uint_as_float(w1 & 0xffff0000u)};
    uint32_t b[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) b[i] = __float_as_uint(__builtin_fmaf(v[i] * q.pre, q.mul, kMagic));
    const uint32_t lo = __builtin_amdgcn_perm(b[1], b[0], 0x0c0c0400u);
    const uint32_t hi = __builtin_amdgcn_perm(b[3], b[2], 0x0c0c0400u);
    return q.bad ? 0u : __builtin_amdgcn_perm(hi, lo, 0x05040100u);
}

// Activation rows to quantize: src bf16 [rows][K] -> codes [rows][Kp] (zero past K)
// and one scale per row, for the first clamp(*n_rows, 0, cap) rows.
struct QuantRows {
    const uint16_t* src;
    const int32_t* n_rows;
    int64_t cap;
    int K, Kp;
    uint8_t* codes;
    float* scales;
};

// Rows first, first + step, ... below end, RPW = 64 / LPR at a time (a wave's share).
// LPR lanes take a row, each lane 8 elements (16 bytes) at a time; NI chunks a lane
// hold the row in registers, so it is read once (NI = 0: read twice).  Memory bound:
// 2 K bytes in, Kp out per row.
template <int LPR, int NI>
__device__ __forceinline__ void quant_row_range(const QuantRows& a, int64_t first, int64_t end, int64_t step)
{
    const int lane = threadIdx.x & 63, l = lane % LPR;
    const int kc = a.K / 8, kpc = a.Kp / 8;
    for (int64_t r0 = first; r0 < end; r0 += step) {
        const int64_t r = r0 + lane / LPR;
        const bool in = r < end;                 // (the other lanes stay for the row maximum)
        const uint4* row = (const uint4*)(a.src + (in ? r : r0) * a.K);
        uint2* out = (uint2*)(a.codes + (in ? r : r0) * a.Kp);
        constexpr int NV = NI > 0 ? NI : 1;
        uint4 v[NV];
        uint32_t m = 0;
        if constexpr (NI > 0) {
#pragma unroll
            for (int i = 0; i < NI; ++i) {
                const int c = i * LPR + l;
                v[i] = c < kc ? row[c] : make_uint4(0, 0, 0, 0);
            }
#pragma unroll
            for (int i = 0; i < NI; ++i)
                m = pair_max(pair_max(pair_max(pair_max(m, v[i].x), v[i].y), v[i].z), v[i].w);
        } else {
            for (int c = l; c < kc; c += LPR) {
                const uint4 w = row[c];
                m = pair_max(pair_max(pair_max(pair_max(m, w.x), w.y), w.z), w.w);
            }
        }
        int amax = row16_max_int(max((int)(m & 0xffffu), (int)(m >> 16)));
        if constexpr (LPR == 64)
            amax = max(max(__builtin_amdgcn_readlane(amax, 0), __builtin_amdgcn_readlane(amax, 16)),
                       max(__builtin_amdgcn_readlane(amax, 32), __builtin_amdgcn_readlane(amax, 48)));
        const RowQuant q = row_quant((uint32_t)amax);
        auto put = [&](int c, const uint4& w) {
            if (in && c < kpc) out[c] = make_uint2(quant4(w.x, w.y, q), quant4(w.z, w.w, q));
        };
        if constexpr (NI > 0) {
#pragma unroll
            for (int i = 0; i < NI; ++i) put(i * LPR + l, v[i]);
        } else {
            for (int c = l; c < kpc; c += LPR) put(c, c < kc ? row[c] : make_uint4(0, 0, 0, 0));
        }
        if (in && l == 0) a.scales[r] = q.scale;
    }
}

// The rows of one workgroup of 256 threads, number `block` of `blocks`.
template <int LPR, int NI>
__device__ __forceinline__ void quant_rows(const QuantRows& a, int block, int blocks)
{
    constexpr int RPW = kWave / LPR;             // rows per wave
    const int32_t n = *a.n_rows;
    const int64_t rows = n < 0 ? 0 : (n > a.cap ? a.cap : n);
    quant_row_range<LPR, NI>(a, ((int64_t)block * 4 + (threadIdx.x >> 6)) * RPW, rows, (int64_t)blocks * 4 * RPW);
}

// The rows of M tiles (of bm rows at most, a multiple of 16), 16 at a time.
struct QuantTiles {
    const int2* tiles;         // (expert, first row)
    const int32_t* n_tiles;
    const int32_t* offsets;    // [E + 1]
    int bm;
};

template <int LPR, int NI>
__device__ __forceinline__ void quant_tile_rows(const QuantRows& a, const QuantTiles& t, int block, int blocks)
{
    constexpr int RPW = kWave / LPR;
    const int per = t.bm / 16, n = *t.n_tiles * per;
    for (int u = block; u < n; u += blocks) {
        const int2 te = t.tiles[u / per];
        const int r0 = te.y + 16 * (u % per);
        const int end = min(min(r0 + 16, te.y + t.bm), t.offsets[te.x + 1]);
        quant_row_range<LPR, NI>(a, r0 + (threadIdx.x >> 6) * RPW, end, 4 * RPW);
    }
}

}  // namespace moe
