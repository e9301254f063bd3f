// Launches of the int8 quantization (quant_int8.h) and the kernel-weight buffer of
// the int8 experts.
#include "quant_int8.h"

namespace moe {

// TILES: the rows of the M tiles of one table (of an expert size); else all of them.
// 131,072 SwiGLU rows of 1024: 69 us, 5.8 TB/s of its 2 + 1 bytes an element (a large
// device copy moves 5.1 TB/s); 1,536 rows: 4.8 us, four dependent round trips.
template <int LPR, int NI, bool TILES>
__global__ void __launch_bounds__(256) quant_rows_int8_kernel(QuantRows a, QuantTiles t)
{
    if constexpr (TILES) quant_tile_rows<LPR, NI>(a, t, blockIdx.x, gridDim.x);
    else quant_rows<LPR, NI>(a, blockIdx.x, gridDim.x);
}

template <bool TILES>
static void launch_quant(const QuantRows& a, const QuantTiles& t, int num_cu, hipStream_t s)
{
    const int64_t cap = a.cap;
    const int Kp = a.Kp;
    auto go = [&](auto kernel, int rows_per_wg) {
        // as many workgroups as the capacity has rows for, at most 8 per CU
        int64_t blocks = (cap + rows_per_wg - 1) / rows_per_wg;
        if (blocks > (int64_t)num_cu * 8) blocks = (int64_t)num_cu * 8;
        if (blocks < 1) blocks = 1;
        hipLaunchKernelGGL(kernel, dim3((unsigned)blocks), dim3(256), 0, s, a, t);
    };
    // 16 lanes a row up to 512 codes (a whole wave would leave lanes idle), else 64.
    // (By tiles only where FC2 has 256-row tiles, from 256 codes on.)
    if constexpr (!TILES) {
        if (Kp <= 128) return go(quant_rows_int8_kernel<16, 1, false>, 16);
    }
    if (Kp <= 256) go(quant_rows_int8_kernel<16, 2, TILES>, 16);
    else if (Kp <= 512) go(quant_rows_int8_kernel<16, 4, TILES>, 16);
    else if (Kp <= 1024) go(quant_rows_int8_kernel<64, 2, TILES>, 4);
    else if (Kp <= 2048) go(quant_rows_int8_kernel<64, 4, TILES>, 4);
    else if (Kp <= 4096) go(quant_rows_int8_kernel<64, 8, TILES>, 4);
    else if (Kp <= 8192) go(quant_rows_int8_kernel<64, 16, TILES>, 4);
    else go(quant_rows_int8_kernel<64, 0, TILES>, 4);   // read twice
}

// tiles (optional): only the rows of this table's M tiles
hipError_t launch_quant_rows_int8(const QuantRows& a, const QuantTiles* tiles, int num_cu, hipStream_t s)
{
    if (tiles) launch_quant<true>(a, *tiles, num_cu, s);
    else launch_quant<false>(a, QuantTiles{}, num_cu, s);
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
