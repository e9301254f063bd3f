// K3 / K4, int8: grouped expert GEMMs on the CDNA4 int8 MFMA (32x32x32), int32
// accumulate, one fp32 scale per activation row and per weight row:
//   FC1  g, u = (float)(sum_k xq[t,k] wq[n,k]) * sw[n] * sx[t], h = silu(g) u
//        rounded to bf16 (the FC2 input of the bf16 path, quantized per row by
//        the launch between the two GEMMs: its scale needs the whole row);
//   FC2  O = (float)(sum_f hq[r,f] wq[m,f]) * sw[m] * sh[r], fp32 rows.
// The sums are exact (|code| <= 128 and K < 131072 keep them inside int32), so
// every tile design gives the same bits whatever its K order; the two fp32
// multiplies run in one order everywhere (scale_col, scale_row).
//
// The tiles are the bf16 ones (gemm_bf16_big.h, gemm_bf16_small.h) with a pair
// of codes in place of a bf16 element: the same 16 bytes a lane and cycles per
// MFMA, half the bytes and MFMAs per row.  Rows are padded with zero codes to a
// multiple of 128 (64 below 256; common.h), so that every K from 224 on takes
// the 256-row design's 128-byte stages.
//
// What bounds it (one MI355X).  16,384 tokens, 128 experts, top-8, hidden 2048, FFN
// 1024: FC1 605 us, FC2 430 us.  With the rows that pad each expert to whole tiles
// (12 %) FC1 runs at 2.03 PetaOPS, a library's dense int8 product of 16384 x 8192 x
// 8192 at 2.19; its MFMAs and epilogues alone take 430 us and its loads alone 450, but
// the shader clock falls to 1.86 GHz (2.4 nominal): it is at the power limit, where
// neither a deeper weight ring (1.3 % of the forward), nor operands resident in the
// L2 (6 %), nor fewer tiles of mostly empty rows (none) gains much.  FC2 runs at 1.43
// PetaOPS, its MFMAs busy for 36 % of the CUs' cycles (FC1 55 %), the clock at 2.05
// GHz: what bounds it is its 1.07 GB of fp32 rows.  Without their stores it takes 307
// us, without MFMAs still 395, with operands resident in the L2 no less.  256 tokens, 64 experts: FC1 45 us, 5.9 TB/s of weights, FC2 27 us (4.9, a third of it the
// first loads' and last stores' latency): the HBM rate of contiguous 32 KB reads (6.1).
#include <hip/hip_ext.h>

#include "gemm_bf16_big.h"
#include "gemm_bf16_small.h"

namespace moe {

template <bool FC1, bool PROB>
__global__ void __launch_bounds__(512, 1) gemm_int8_small_kernel(GemmArgs g)
{
    __shared__ __attribute__((aligned(1024))) char smem[kSmallLds];
    // as the bf16 kernel: the counts and the first tile's entry in one round trip
    const int n_big = g.small_takes_big ? ld_const(&g.hdr->n_tiles_big) : 0;
    const int n_small = ld_const(&g.hdr->n_tiles);
    const int multi = ld_const(&g.hdr->multi_tile);
    const int* te0 = (const int*)(g.tiles + min(xcd_first_tile() / small_col_tiles(g), g.max_tiles - 1));
    const int e0 = ld_const(te0), row00 = ld_const(te0 + 1);
    asm volatile("" : : "s"(n_big), "s"(n_small), "s"(multi), "s"(e0), "s"(row00));
    if (multi) small_tiles<OpInt8, FC1, PROB, 0, 0>(g, smem, n_small, n_big, e0, row00);
    else small_tiles<OpInt8, FC1, PROB, 0, kNonTemporal>(g, smem, n_small, n_big, e0, row00);
}

// FC2's policies follow the bytes of its fp32 rows (hidden 2048, FFN 1024, a forward):
// rows that fit the 256 MB Infinity Cache are stored as usual, for the combine to find
// there (2,048 tokens x top-6: 188 us, 192 non-temporally; 3,000 x 8: 340 / 347), larger
// ones non-temporally, so that they do not displace the operands (4,096 x 8: 455, 463 as
// usual; 16,384 x 8: 1289 / 1308).  Weights are read non-temporally too where the rows are
// past twice that cache (12,000 x 8: 981, 994 as usual; 16,384 x 8: 1336 / 1360); below,
// some are found in it (6,000 x 8: 595, 607 non-temporally; 8,192 x 6: 558 / 562).
template <bool FC1, bool PROB, int WPOL, int RPOL>
__global__ void __launch_bounds__(512, 1) gemm_int8_big_kernel(GemmArgs g)
{
    big_tiles<OpInt8, FC1, PROB, WPOL, RPOL>(g, ld_const(&g.hdr->n_tiles_big));
}

// One GEMM stage: the 256-row launch on s (unless the 64-row kernel takes its
// tiles), the 64-row launch on s_small (s if null).  t0 / t1 as launch_gemm_bf16.
// max_rows: the most grouped rows that the capacity can have.
hipError_t launch_gemm_int8(bool fc1, const GemmArgs& g, int64_t max_rows, int num_cu, hipStream_t s, hipEvent_t t0,
                            hipEvent_t t1, hipStream_t s_small)
{
    if (!g.a_scale || !g.w_scale || g.K < 32 || g.K % 32 != 0 || g.N < 32 || g.N % 32 != 0)
        return hipErrorInvalidValue;
    const dim3 grid((unsigned)(num_cu >= 8 ? num_cu / 8 * 8 : 8)), block(512);
    auto go = [&](auto kernel, hipEvent_t e0, hipEvent_t e1, hipStream_t st) {
        if (e0 || e1)
            hipExtLaunchKernelGGL(kernel, grid, block, 0, st, e0, e1, 0, g);
        else
            hipLaunchKernelGGL(kernel, grid, block, 0, st, g);
    };
    const bool prob = fc1 && g.row_prob != nullptr;
    hipEvent_t small_start = t0;
    hipStream_t ss = s;
    if (!g.small_takes_big) {
        const int64_t row_bytes = max_rows * g.N * 4, cache = (int64_t)256 << 20;
        if (prob) go(gemm_int8_big_kernel<true, true, 0, 0>, t0, nullptr, s);
        else if (fc1) go(gemm_int8_big_kernel<true, false, 0, 0>, t0, nullptr, s);
        else if (row_bytes < cache) go(gemm_int8_big_kernel<false, false, 0, 0>, t0, nullptr, s);
        else if (row_bytes < 2 * cache) go(gemm_int8_big_kernel<false, false, 0, kNonTemporal>, t0, nullptr, s);
        else go(gemm_int8_big_kernel<false, false, kNonTemporal, kNonTemporal>, t0, nullptr, s);
        small_start = nullptr;
        if (s_small) ss = s_small;
    }
    if (prob) go(gemm_int8_small_kernel<true, true>, small_start, t1, ss);
    else if (fc1) go(gemm_int8_small_kernel<true, false>, small_start, t1, ss);
    else go(gemm_int8_small_kernel<false, false>, small_start, t1, ss);
    return hipGetLastError();
}

}  // namespace moe
