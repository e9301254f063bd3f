// Launches of the experts' backward products (grad_gemm.h): the rows' gradients before and
// after the SwiGLU, then both weights' gradients in one launch.
#include "grad_gemm.h"

namespace moe {

template <bool SWIGLU, bool WIDE>
__global__ void __launch_bounds__(512, 1) grad_rows_kernel(GradArgs g)
{
    grad_rows_tiles<SWIGLU, WIDE>(g);
}

template <bool SWIGLU>
__global__ void __launch_bounds__(512, 1) grad_small_kernel(GradArgs g, int take_big)
{
    grad_small_tiles<SWIGLU>(g, take_big != 0);
}

template <bool FP32, bool WIDE>
__global__ void __launch_bounds__(512, 1) grad_weight_kernel(GradArgs g)
{
    grad_weight_tiles<FP32, WIDE>(g);
}

// Capacities up to 1024 run the 64-row tiles alone, for one launch less a product.  1,000
// tokens, 64-row tiles alone against both (hidden 2048, FFN 1024): top-2 of 2 experts 113 us
// / 155, of 8 150 / 176, top-4 of 32 285 / 347, top-6 of 64 473 / 474; 500 tokens, top-2 of 8,
// 109 / 206; only many rows of large experts cross below it (top-4 of 8, hidden 4096, FFN
// 2048: 671 / 572).
bool grad_takes_big(int64_t T_cap) { return T_cap <= 1024; }

// 32-bit byte offsets do not reach: in the gathered rows, in an expert's rows (at most one a
// token) or in its weights
static bool grad_wide(const GradArgs& g, int64_t T_cap)
{
    const int64_t lim = (int64_t)1 << 31;
    return T_cap * 2 * g.H >= lim || T_cap * 4 * g.F >= lim || (int64_t)4 * g.F * g.H >= lim;
}

static dim3 grad_grid(int num_cu)       // a multiple of 8: the tiles are split over the 8 XCDs
{
    return dim3((unsigned)(num_cu >= 8 ? num_cu / 8 * 8 : 8));
}

// The rows' products: those of the experts with at most 128 rows on `small`, the others' on
// `s` (the two are disjoint, and each design's second product reads its own first one's rows)
hipError_t launch_grad_rows(const GradArgs& g, int64_t T_cap, int num_cu, hipStream_t s, hipStream_t small)
{
    const dim3 grid = grad_grid(num_cu), block(512);
    const int take_big = grad_takes_big(T_cap);
    const bool wide = grad_wide(g, T_cap);
    if (!take_big) {
        if (wide || g.H % 64) hipLaunchKernelGGL((grad_rows_kernel<true, true>), grid, block, 0, s, g);
        else hipLaunchKernelGGL((grad_rows_kernel<true, false>), grid, block, 0, s, g);
    }
    hipLaunchKernelGGL(grad_small_kernel<true>, grid, block, 0, small, g, take_big);
    if (!take_big) {
        if (wide) hipLaunchKernelGGL((grad_rows_kernel<false, true>), grid, block, 0, s, g);
        else hipLaunchKernelGGL((grad_rows_kernel<false, false>), grid, block, 0, s, g);
    }
    hipLaunchKernelGGL(grad_small_kernel<false>, grid, block, 0, small, g, take_big);
    return hipGetLastError();
}

hipError_t launch_grad_weights(const GradArgs& g, int64_t T_cap, bool fp32, int num_cu, hipStream_t s)
{
    const dim3 grid = grad_grid(num_cu), block(512);
    const bool wide = grad_wide(g, T_cap);
    if (fp32 && wide) hipLaunchKernelGGL((grad_weight_kernel<true, true>), grid, block, 0, s, g);
    else if (fp32) hipLaunchKernelGGL((grad_weight_kernel<true, false>), grid, block, 0, s, g);
    else if (wide) hipLaunchKernelGGL((grad_weight_kernel<false, true>), grid, block, 0, s, g);
    else hipLaunchKernelGGL((grad_weight_kernel<false, false>), grid, block, 0, s, g);
    return hipGetLastError();
}

}  // namespace moe
