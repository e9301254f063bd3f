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

// Activation rows: src bf16 [rows][K] -> codes [rows][Kp] (zero past K) and one
// scale per row, for the first clamp(*n_rows, 0, cap) rows.  LPR lanes take a
// row, each lane 8 elements (16 bytes) at a time; NI chunks a lane hold the row
// in registers, so it is read once (NI = 0, rows above 8192: read twice).
// Memory bound: 2 K bytes in, Kp out per row.
template <int LPR, int NI>
__global__ void __launch_bounds__(256) quant_rows_int8_kernel(const uint16_t* __restrict__ src,
                                                              const int32_t* __restrict__ n_rows, int64_t cap,
                                                              int K, int Kp, uint8_t* __restrict__ codes,
                                                              float* __restrict__ scales)
{
    const int32_t n = *n_rows;
    const int64_t rows = n < 0 ? 0 : (n > cap ? cap : n);
    constexpr int RPW = kWave / LPR;             // rows per wave
    const int lane = threadIdx.x & 63, l = lane % LPR;
    const int kc = K / 8, kpc = Kp / 8;
    const int64_t wave = (int64_t)blockIdx.x * (blockDim.x / kWave) + (threadIdx.x >> 6);
    const int64_t step = (int64_t)gridDim.x * (blockDim.x / kWave) * RPW;
    for (int64_t r0 = wave * RPW; r0 < rows; r0 += step) {
        const int64_t r = r0 + lane / LPR;
        const bool in = r < rows;                // (the other lanes stay for the row maximum)
        const uint4* row = (const uint4*)(src + (in ? r : r0) * K);
        uint2* out = (uint2*)(codes + (in ? r : r0) * Kp);
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
        if (in && l == 0) scales[r] = q.scale;
    }
}

hipError_t launch_quant_rows_int8(const uint16_t* src, const int32_t* n_rows, int64_t cap, int K, int Kp,
                                  uint8_t* codes, float* scales, int num_cu, hipStream_t s)
{
    const dim3 block(256);
    auto go = [&](auto kernel, int rows_per_wg) {
        // as many workgroups as the capacity has rows for, at most 8 per CU
        int64_t blocks = (cap + rows_per_wg - 1) / rows_per_wg;
        if (blocks > (int64_t)num_cu * 8) blocks = (int64_t)num_cu * 8;
        if (blocks < 1) blocks = 1;
        hipLaunchKernelGGL(kernel, dim3((unsigned)blocks), block, 0, s, src, n_rows, cap, K, Kp, codes, scales);
    };
    // 16 lanes a row up to 512 codes (a whole wave would leave lanes idle), else 64
    if (Kp <= 128) go(quant_rows_int8_kernel<16, 1>, 16);
    else if (Kp <= 256) go(quant_rows_int8_kernel<16, 2>, 16);
    else if (Kp <= 512) go(quant_rows_int8_kernel<16, 4>, 16);
    else if (Kp <= 1024) go(quant_rows_int8_kernel<64, 2>, 4);
    else if (Kp <= 2048) go(quant_rows_int8_kernel<64, 4>, 4);
    else if (Kp <= 4096) go(quant_rows_int8_kernel<64, 8>, 4);
    else if (Kp <= 8192) go(quant_rows_int8_kernel<64, 16>, 4);
    else go(quant_rows_int8_kernel<64, 0>, 4);
    return hipGetLastError();
}

__device__ __forceinline__ int64_t int8_fc1_src_row(int64_t packed, int64_t F)
{
    const int64_t b = packed >> 6, i = packed & 63;
    return i < 32 ? 32 * b + i : F + 32 * b + (i - 32);
}

// Kernel weights.  A workgroup takes one 16-row column block of an expert at a
// time: 16 threads per row find its scale (CODES: it is given), then the
// block's 16-byte pieces (16 codes of one row) are written in buffer order, 1 KB
// a wave.  Blocks of 16 rows x 64 K in the bf16 blocks' order (wblock_index).
template <bool CODES>
__global__ void __launch_bounds__(256) pack_int8_kernel(const void* __restrict__ src,
                                                        const float* __restrict__ src_scale,
                                                        uint8_t* __restrict__ codes, float* __restrict__ scales,
                                                        int E, int N, int K, int Kp, int F, int fc1)
{
    __shared__ RowQuant rq[16];
    const int64_t nt = N / 16, ks = Kp / 64;
    for (int64_t b = blockIdx.x; b < (int64_t)E * nt; b += gridDim.x) {
        const int64_t e = b / nt, n16 = b - e * nt;
        {
            const int r = threadIdx.x >> 4, l = threadIdx.x & 15;
            const int64_t n = n16 * 16 + r;
            const int64_t srow = e * N + (fc1 ? int8_fc1_src_row(n, F) : n);
            if constexpr (CODES) {
                if (l == 0) scales[e * N + n] = src_scale[srow];
            } else {
                const uint4* row = (const uint4*)((const uint16_t*)src + srow * K);
                uint32_t m = 0;
                for (int c = l; c < K / 8; c += 16) {
                    const uint4 w = row[c];
                    m = pair_max(pair_max(pair_max(pair_max(m, w.x), w.y), w.z), w.w);
                }
                const int amax = row16_max_int(max((int)(m & 0xffffu), (int)(m >> 16)));
                const RowQuant q = row_quant((uint32_t)amax);
                if (l == 0) {
                    rq[r] = q;
                    scales[e * N + n] = q.scale;
                }
            }
        }
        __syncthreads();
        for (int64_t p = threadIdx.x; p < ks * 64; p += blockDim.x) {
            const int64_t s = p >> 6;
            const int lane = (int)(p & 63);
            const int64_t n = n16 * 16 + (lane & 15), k = s * 64 + (lane >> 4) * 16;
            const int64_t srow = e * N + (fc1 ? int8_fc1_src_row(n, F) : n);
            uint4 o = make_uint4(0, 0, 0, 0);
            if (k < K) {                         // K is a multiple of 32: pieces are whole
                if constexpr (CODES) {
                    o = *(const uint4*)((const uint8_t*)src + srow * K + k);
                } else {
                    const RowQuant q = rq[lane & 15];
                    const uint4* v = (const uint4*)((const uint16_t*)src + srow * K + k);
                    const uint4 a = v[0], c = v[1];
                    o = make_uint4(quant4(a.x, a.y, q), quant4(a.z, a.w, q), quant4(c.x, c.y, q), quant4(c.z, c.w, q));
                }
            }
            ((uint4*)codes)[(e * nt * ks + wblock_index(n16, s, nt, ks)) * 64 + lane] = o;
        }
        __syncthreads();                         // rq is read until here
    }
}

// Section sizes of the int8 buffer: codes of FC1 and FC2, scales of FC1 and FC2.
void int8_section_bytes(int E, int H, int F, size_t* c1, size_t* c2, size_t* s1, size_t* s2)
{
    auto up256 = [](size_t v) { return (v + 255) / 256 * 256; };
    *c1 = up256((size_t)E * 2 * F * int8_pitch(H));
    *c2 = up256((size_t)E * H * int8_pitch(F));
    *s1 = up256((size_t)E * 2 * F * 4);
    *s2 = up256((size_t)E * H * 4);
}

// codes != 0: w1, w2 are int8 codes with the scales ws1 [E][2F], ws2 [E][H];
// else bf16 weights.
hipError_t launch_pack_int8(const void* w1, const float* ws1, const void* w2, const float* ws2, int codes,
                            uint8_t* kbuf, int E, int H, int F, int num_cu, hipStream_t s)
{
    size_t c1, c2, s1, s2;
    int8_section_bytes(E, H, F, &c1, &c2, &s1, &s2);
    float* q1 = (float*)(kbuf + c1 + c2);
    float* q2 = (float*)(kbuf + c1 + c2 + s1);
    const dim3 grid(num_cu * 8), block(256);
    if (codes) {
        hipLaunchKernelGGL(pack_int8_kernel<true>, grid, block, 0, s, w1, ws1, kbuf, q1, E, 2 * F, H, int8_pitch(H), F, 1);
        hipLaunchKernelGGL(pack_int8_kernel<true>, grid, block, 0, s, w2, ws2, kbuf + c1, q2, E, H, F, int8_pitch(F), F, 0);
    } else {
        hipLaunchKernelGGL(pack_int8_kernel<false>, grid, block, 0, s, w1, ws1, kbuf, q1, E, 2 * F, H, int8_pitch(H), F, 1);
        hipLaunchKernelGGL(pack_int8_kernel<false>, grid, block, 0, s, w2, ws2, kbuf + c1, q2, E, H, F, int8_pitch(F), F, 0);
    }
    return hipGetLastError();
}

}  // namespace moe
