// Tokens sorted by expert and back, and their gradients.
//
//   dispatch           rows[row_of[t][j]] = x[t]
//   combine            out[t] = sum over j of p[t][j] rows[row_of[t][j]], an fp32 fused
//                      multiply-add chain from +0 in ascending row (so expert) order, rounded
//                      once; without probabilities every p is 1, which is the gradient of
//                      dispatch
//   combine backward   d_rows[row_of[t][j]] = p[t][j] d_out[t],
//                      d_probs[t][j] = sum over columns of d_out[t] rows[row_of[t][j]]
// row_of outside [0, T_cap k): a route without a row adds nothing and has a gradient of 0.
//
// Bound by memory: every row is touched once.  A thread takes 8 neighbouring columns of a
// token (16 bytes of bf16) with all k rows' accesses in flight at once.
#include "common.h"

namespace moe {

typedef float f4v __attribute__((ext_vector_type(4)));
typedef unsigned u4v __attribute__((ext_vector_type(4)));

__device__ __forceinline__ int64_t rows_live(const int32_t* live_ptr, int64_t T_cap)
{
    const int32_t live = *live_ptr;
    return live < 0 ? 0 : (live > T_cap ? T_cap : live);
}

// 8 neighbouring columns of a row, fp32 or bf16 in memory
template <bool BF16>
struct Row8;
template <>
struct Row8<true> {
    u4v v;
    __device__ __forceinline__ void load(const void* base, int64_t at) { v = __builtin_nontemporal_load((const u4v*)((const uint16_t*)base + at)); }
    __device__ __forceinline__ void get(float (&f)[8]) const
    {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            f[2 * i] = __uint_as_float(v[i] << 16);
            f[2 * i + 1] = __uint_as_float(v[i] & 0xffff0000u);
        }
    }
    __device__ __forceinline__ void zero() { v = u4v{0u, 0u, 0u, 0u}; }
    __device__ __forceinline__ void set(const float (&f)[8])
    {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            v[i] = (uint32_t)f32_to_bf16_bits(f[2 * i]) | ((uint32_t)f32_to_bf16_bits(f[2 * i + 1]) << 16);
    }
    __device__ __forceinline__ void store(void* base, int64_t at) const { __builtin_nontemporal_store(v, (u4v*)((uint16_t*)base + at)); }
};
template <>
struct Row8<false> {
    f4v a, b;
    __device__ __forceinline__ void load(const void* base, int64_t at)
    {
        a = __builtin_nontemporal_load((const f4v*)((const float*)base + at));
        b = __builtin_nontemporal_load((const f4v*)((const float*)base + at) + 1);
    }
    __device__ __forceinline__ void get(float (&f)[8]) const
    {
#pragma unroll
        for (int i = 0; i < 4; ++i) { f[i] = a[i]; f[4 + i] = b[i]; }
    }
    __device__ __forceinline__ void zero() { a = b = f4v{0.f, 0.f, 0.f, 0.f}; }
    __device__ __forceinline__ void set(const float (&f)[8])
    {
#pragma unroll
        for (int i = 0; i < 4; ++i) { a[i] = f[i]; b[i] = f[4 + i]; }
    }
    __device__ __forceinline__ void store(void* base, int64_t at) const
    {
        __builtin_nontemporal_store(a, (f4v*)((float*)base + at));
        __builtin_nontemporal_store(b, (f4v*)((float*)base + at) + 1);
    }
};

// ---------------------------------------------------------------- dispatch

struct DispatchArgs {
    const void* x;             // [T_cap][H]
    const int32_t* ids;        // [T_cap][k], the caller's order
    const int32_t* dst;        // rows by route, canonical order (-1: none)
    const int32_t* offsets;    // [E + 1]
    const int32_t* live;
    int64_t T_cap;
    int E, H;
    void* rows;
    int32_t* row_of;           // [T_cap][k], the caller's order
    int32_t* offsets_out;      // [E + 1]
};

template <int K, bool BF16>
__global__ void __launch_bounds__(256) dispatch_kernel(DispatchArgs a)
{
    const int64_t T = rows_live(a.live, a.T_cap);
    const int nc = a.H / 8;
    const int64_t i0 = (int64_t)blockIdx.x * blockDim.x + threadIdx.x, step = (int64_t)gridDim.x * blockDim.x;
    for (int64_t e = i0; e <= a.E; e += step) a.offsets_out[e] = a.offsets[e];
    for (int64_t i = i0; i < T * nc; i += step) {
        const int64_t t = i / nc;
        const int c = (int)(i - t * nc);
        Row8<BF16> v;
        v.load(a.x, t * a.H + 8 * c);
        int d[K];
#pragma unroll
        for (int j = 0; j < K; ++j) d[j] = a.dst[t * K + j];
#pragma unroll
        for (int j = 0; j < K; ++j)
            if (d[j] >= 0) v.store(a.rows, (int64_t)d[j] * a.H + 8 * c);
        if (c == 0) {
            // the canonical order is a stable sort by id: a route's place is its id's rank
            int id[K];
#pragma unroll
            for (int j = 0; j < K; ++j) id[j] = a.ids[t * K + j];
#pragma unroll
            for (int j = 0; j < K; ++j) {
                int rank = 0, r = -1;
#pragma unroll
                for (int i2 = 0; i2 < K; ++i2) rank += (id[i2] < id[j] || (id[i2] == id[j] && i2 < j)) ? 1 : 0;
#pragma unroll
                for (int i2 = 0; i2 < K; ++i2) r = i2 == rank ? d[i2] : r;
                a.row_of[t * K + j] = r;
            }
        }
    }
}

// ---------------------------------------------------------------- combine

struct CombineArgs {
    const void* rows;          // [.][H]
    const int32_t* row_of;     // [T_cap][k]
    const float* probs;        // [T_cap][k] or null (every p is 1)
    const int32_t* live;
    int64_t T_cap;
    int H;
    void* out;                 // [T_cap][H]
};

// ascending by row, the routes without a row (as the largest unsigned) last
template <int K>
__device__ __forceinline__ void rows_sort(uint32_t (&d)[K], float (&p)[K])
{
#pragma unroll
    for (int x = 1; x < K; ++x)
#pragma unroll
        for (int y = x; y > 0; --y) {
            const bool sw = d[y - 1] > d[y];
            const uint32_t lo = sw ? d[y] : d[y - 1], hi = sw ? d[y - 1] : d[y];
            const float pl = sw ? p[y] : p[y - 1], ph = sw ? p[y - 1] : p[y];
            d[y - 1] = lo; d[y] = hi;
            p[y - 1] = pl; p[y] = ph;
        }
}

template <int K, bool IN_BF16, bool OUT_BF16>
__global__ void __launch_bounds__(256) combine_kernel(CombineArgs a)
{
    const int64_t T = rows_live(a.live, a.T_cap);
    const int nc = a.H / 8;
    const int64_t i0 = (int64_t)blockIdx.x * blockDim.x + threadIdx.x, step = (int64_t)gridDim.x * blockDim.x;
    for (int64_t i = i0; i < T * nc; i += step) {
        const int64_t t = i / nc;
        const int c = (int)(i - t * nc);
        uint32_t d[K];
        float p[K];
#pragma unroll
        for (int j = 0; j < K; ++j) {
            const uint32_t r = (uint32_t)a.row_of[t * K + j];
            d[j] = r < (uint64_t)a.T_cap * K ? r : 0xffffffffu;
            p[j] = a.probs ? a.probs[t * K + j] : 1.0f;
        }
        rows_sort<K>(d, p);
        Row8<IN_BF16> v[K];
#pragma unroll
        for (int j = 0; j < K; ++j)
            if (d[j] != 0xffffffffu) v[j].load(a.rows, (int64_t)d[j] * a.H + 8 * c);
            else v[j].zero();
        float acc[8] = {};
#pragma unroll
        for (int j = 0; j < K; ++j) {
            if (d[j] == 0xffffffffu) continue;
            float f[8];
            v[j].get(f);
#pragma unroll
            for (int n = 0; n < 8; ++n) acc[n] = __builtin_fmaf(p[j], f[n], acc[n]);
        }
        Row8<OUT_BF16> o;
        o.set(acc);
        o.store(a.out, t * a.H + 8 * c);
    }
}

// ---------------------------------------------------------------- combine backward

struct CombineBwdArgs {
    const void* d_out;         // [T_cap][H]
    const void* rows;          // [.][H], or null with d_probs
    const int32_t* row_of;
    const float* probs;
    const int32_t* live;
    int64_t T_cap;
    int H;
    void* d_rows;              // [.][H], of the rows' type
    float* d_probs;            // [T_cap][k] or null
};

// A wave per token
template <int K, bool ROWS_BF16, bool OUT_BF16, bool PROBS>
__global__ void __launch_bounds__(256) combine_bwd_kernel(CombineBwdArgs a)
{
    const int64_t T = rows_live(a.live, a.T_cap);
    const int nc = a.H / 8, lane = threadIdx.x & 63;
    const int64_t waves = (int64_t)gridDim.x * (blockDim.x >> 6);
    for (int64_t t = (int64_t)blockIdx.x * (blockDim.x >> 6) + (threadIdx.x >> 6); t < T; t += waves) {
        int32_t d[K];
        float p[K], dot[K];
#pragma unroll
        for (int j = 0; j < K; ++j) {
            d[j] = a.row_of[t * K + j];
            if ((uint32_t)d[j] >= (uint64_t)a.T_cap * K) d[j] = -1;
            p[j] = a.probs[t * K + j];
            dot[j] = 0.0f;
        }
        for (int c = lane; c < nc; c += 64) {
            Row8<OUT_BF16> g;
            g.load(a.d_out, t * a.H + 8 * c);
            Row8<ROWS_BF16> v[K];
            if constexpr (PROBS) {
#pragma unroll
                for (int j = 0; j < K; ++j)
                    if (d[j] >= 0) v[j].load(a.rows, (int64_t)d[j] * a.H + 8 * c);
                    else v[j].zero();
            }
            float gf[8];
            g.get(gf);
#pragma unroll
            for (int j = 0; j < K; ++j) {
                if (d[j] < 0) continue;
                float f[8];
                if constexpr (PROBS) {
                    v[j].get(f);
#pragma unroll
                    for (int n = 0; n < 8; ++n) dot[j] = __builtin_fmaf(gf[n], f[n], dot[j]);
                }
#pragma unroll
                for (int n = 0; n < 8; ++n) f[n] = p[j] * gf[n];
                Row8<ROWS_BF16> o;
                o.set(f);
                o.store(a.d_rows, (int64_t)d[j] * a.H + 8 * c);
            }
        }
        if constexpr (PROBS) {
#pragma unroll
            for (int j = 0; j < K; ++j) {
#pragma unroll
                for (int off = 32; off > 0; off >>= 1) dot[j] += __shfl_xor(dot[j], off);
                if (lane == 0) a.d_probs[t * K + j] = dot[j];
            }
        }
    }
}

// ---------------------------------------------------------------- experts' backward: ends

// d_probs[t][j] of the caller's route j from the partial sums of its row
__global__ void __launch_bounds__(256) grad_probs_kernel(const float* part, int n_part, const int32_t* ids,
                                                         const int32_t* dst, const int32_t* live, int64_t T_cap, int k,
                                                         float* d_probs)
{
    const int64_t T = rows_live(live, T_cap);
    for (int64_t r = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; r < T * k; r += (int64_t)gridDim.x * blockDim.x) {
        const int64_t t = r / k;
        const int j = (int)(r - t * k);
        const int id = ids[r];
        int rank = 0;
        for (int i = 0; i < k; ++i) {
            const int o = ids[t * k + i];
            rank += (o < id || (o == id && i < j)) ? 1 : 0;
        }
        const int d = dst[t * k + rank];
        float s = 0.0f;
        if (d >= 0)
            for (int i = 0; i < n_part; ++i) s += part[(int64_t)d * n_part + i];
        d_probs[r] = s;
    }
}

// fp32 rows rounded to bf16, the operand type of the products
__global__ void __launch_bounds__(256) cast_rows_kernel(const float* in, const int32_t* live, int64_t T_cap, int H,
                                                        uint16_t* out)
{
    const int64_t n = rows_live(live, T_cap) * (H / 8);
    for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < n; i += (int64_t)gridDim.x * blockDim.x) {
        Row8<false> v;
        v.load(in, 8 * i);
        float f[8];
        v.get(f);
        Row8<true> o;
        o.set(f);
        *(u4v*)(out + 8 * i) = o.v;
    }
}

// ---------------------------------------------------------------- launches

static dim3 rows_grid(int64_t threads, int num_cu)
{
    int64_t b = (threads + 255) / 256;
    const int64_t most = (int64_t)num_cu * 16;
    if (b > most) b = most;
    return dim3((unsigned)(b < 1 ? 1 : b));
}

#define ROWS_K(M)                                                                          \
    switch (k) {                                                                           \
        M(1) M(2) M(3) M(4) M(5) M(6) M(7) M(8) M(9) M(10) M(11) M(12) M(13) M(14) M(15) M(16) \
        default: return hipErrorInvalidValue;                                              \
    }

hipError_t launch_dispatch(const void* x, int bf16, const int32_t* ids, const int32_t* dst, const int32_t* offsets,
                           const int32_t* live, int64_t T_cap, int E, int k, int H, void* rows,
                           int32_t* row_of, int32_t* offsets_out, int num_cu, hipStream_t s)
{
    const DispatchArgs a{x, ids, dst, offsets, live, T_cap, E, H, rows, row_of, offsets_out};
    const dim3 g = rows_grid(T_cap * (H / 8), num_cu), b(256);
#define M(K)                                                                                   \
    case K:                                                                                    \
        if (bf16) hipLaunchKernelGGL((dispatch_kernel<K, true>), g, b, 0, s, a);               \
        else hipLaunchKernelGGL((dispatch_kernel<K, false>), g, b, 0, s, a);                   \
        break;
    ROWS_K(M)
#undef M
    return hipGetLastError();
}

hipError_t launch_combine(const void* rows, int in_bf16, const int32_t* row_of, const float* probs,
                          const int32_t* live, int64_t T_cap, int k, int H, void* out, int out_bf16, int num_cu,
                          hipStream_t s)
{
    const CombineArgs a{rows, row_of, probs, live, T_cap, H, out};
    const dim3 g = rows_grid(T_cap * (H / 8), num_cu), b(256);
#define M(K)                                                                                   \
    case K:                                                                                    \
        if (in_bf16 && out_bf16) hipLaunchKernelGGL((combine_kernel<K, true, true>), g, b, 0, s, a);   \
        else if (in_bf16) hipLaunchKernelGGL((combine_kernel<K, true, false>), g, b, 0, s, a);         \
        else if (out_bf16) hipLaunchKernelGGL((combine_kernel<K, false, true>), g, b, 0, s, a);        \
        else hipLaunchKernelGGL((combine_kernel<K, false, false>), g, b, 0, s, a);                     \
        break;
    ROWS_K(M)
#undef M
    return hipGetLastError();
}

hipError_t launch_combine_backward(const void* d_out, int out_bf16, const void* rows, int rows_bf16,
                                   const int32_t* row_of, const float* probs, const int32_t* live, int64_t T_cap,
                                   int k, int H, void* d_rows, float* d_probs, int num_cu, hipStream_t s)
{
    const CombineBwdArgs a{d_out, rows, row_of, probs, live, T_cap, H, d_rows, d_probs};
    const dim3 g = rows_grid(T_cap * 64, num_cu), b(256);
#define GO(K, R, O)                                                                                    \
    if (d_probs) hipLaunchKernelGGL((combine_bwd_kernel<K, R, O, true>), g, b, 0, s, a);               \
    else hipLaunchKernelGGL((combine_bwd_kernel<K, R, O, false>), g, b, 0, s, a)
#define M(K)                                                                                   \
    case K:                                                                                    \
        if (rows_bf16 && out_bf16) { GO(K, true, true); }                                      \
        else if (rows_bf16) { GO(K, true, false); }                                            \
        else if (out_bf16) { GO(K, false, true); }                                             \
        else { GO(K, false, false); }                                                          \
        break;
    ROWS_K(M)
#undef M
#undef GO
    return hipGetLastError();
}

hipError_t launch_grad_probs(const float* part, int n_part, const int32_t* ids, const int32_t* dst,
                             const int32_t* live, int64_t T_cap, int k, float* d_probs, int num_cu, hipStream_t s)
{
    hipLaunchKernelGGL(grad_probs_kernel, rows_grid(T_cap * k, num_cu), dim3(256), 0, s, part, n_part, ids, dst, live,
                       T_cap, k, d_probs);
    return hipGetLastError();
}

hipError_t launch_cast_rows(const float* in, const int32_t* live, int64_t T_cap, int H, uint16_t* out, int num_cu,
                            hipStream_t s)
{
    hipLaunchKernelGGL(cast_rows_kernel, rows_grid(T_cap * (H / 8), num_cu), dim3(256), 0, s, in, live, T_cap, H, out);
    return hipGetLastError();
}

}  // namespace moe
