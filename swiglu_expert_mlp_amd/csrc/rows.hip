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
// Bound by memory: every row is touched once.  A thread takes 16 bytes of neighbouring
// columns of a token's rows, with all k rows' accesses in flight at once.  Measured at 16,384
// tokens, top-8, hidden 2048 (a large device copy runs at 5.1 TB/s, read and written): the
// copy of dispatch 118 us (5.1 TB/s), sums of fp32 rows 202 to 228 a launch and 207 to 212 a
// call (5.8), both gradients of bf16 rows 230 (5.0), x's and the probabilities' gradients of the
// experts 115 (5.7).
// The sums take columns of tokens as they come, so every hidden size runs at that rate (131,072
// tokens of hidden 64, bf16: 31 us).  dispatch above 256 tokens and the gradients of combine give
// a wave up to 64 columns of one token, so below 1 KB a row the launch is bound by its waves, not
// by bytes: hidden 64 in bf16, 131,072 tokens, 139 us (1.2 TB/s) and 154 (1.9), hidden 128 160 and
// 169, hidden 256 198 (3.1) and 219 (5.3); hidden 544, 49,152 tokens, 144 (3.4) and 195 (4.7).
#include "common.h"
#include "grad_dx.h"

namespace moe {

typedef unsigned u4v __attribute__((ext_vector_type(4)));

__device__ __forceinline__ int64_t rows_live(const int32_t* live_ptr, int64_t T_cap)
{
    const int32_t live = *live_ptr;
    return live < 0 ? 0 : (live > T_cap ? T_cap : live);
}

// N neighbouring columns of a row, fp32 or bf16 in memory.  Each is touched once:
// non-temporal accesses (as in the forward's combine).
typedef unsigned u2v __attribute__((ext_vector_type(2)));
template <bool BF16, int N>
struct RowN {
    static constexpr int kWords = BF16 ? N / 2 : N;              // 32-bit words
    uint32_t w[kWords];
    __device__ __forceinline__ void load(const void* base, int64_t at)
    {
        const char* p = (const char*)base + at * (BF16 ? 2 : 4);
        if constexpr (kWords >= 4) {
#pragma unroll
            for (int i = 0; i < kWords / 4; ++i) {
                const u4v v = __builtin_nontemporal_load((const u4v*)p + i);
#pragma unroll
                for (int n = 0; n < 4; ++n) w[4 * i + n] = v[n];
            }
        } else {
            const u2v v = __builtin_nontemporal_load((const u2v*)p);
            w[0] = v[0];
            w[1] = v[1];
        }
    }
    __device__ __forceinline__ void store(void* base, int64_t at) const
    {
        char* p = (char*)base + at * (BF16 ? 2 : 4);
        if constexpr (kWords >= 4) {
#pragma unroll
            for (int i = 0; i < kWords / 4; ++i)
                __builtin_nontemporal_store(u4v{w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]}, (u4v*)p + i);
        } else {
            __builtin_nontemporal_store(u2v{w[0], w[1]}, (u2v*)p);
        }
    }
    __device__ __forceinline__ void get(float (&f)[N]) const
    {
#pragma unroll
        for (int i = 0; i < kWords; ++i)
            if constexpr (BF16) {
                f[2 * i] = __uint_as_float(w[i] << 16);
                f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
            } else {
                f[i] = __uint_as_float(w[i]);
            }
    }
    __device__ __forceinline__ void set(const float (&f)[N])
    {
#pragma unroll
        for (int i = 0; i < kWords; ++i)
            if constexpr (BF16)
                w[i] = (uint32_t)f32_to_bf16_bits(f[2 * i]) | ((uint32_t)f32_to_bf16_bits(f[2 * i + 1]) << 16);
            else
                w[i] = __float_as_uint(f[i]);
    }
    __device__ __forceinline__ void zero()
    {
#pragma unroll
        for (int i = 0; i < kWords; ++i) w[i] = 0;
    }
};

// Columns of a thread: 16 bytes of the rows (with 32 bytes of fp32 a wave's instruction
// took every other 16 bytes: the 16K-token sum of fp32 rows 241 us instead of 225)
template <bool BF16>
constexpr int row_cols() { return BF16 ? 8 : 4; }

// ---------------------------------------------------------------- dispatch

struct DispatchArgs {
    const void* x;             // [T_cap][H]
    const int32_t* ids;        // [T_cap][k], the caller's order
    // what the permutation's first two launches left (more than one chunk of tokens)
    const int32_t* sorted_ids; // [T_cap][k], canonical order
    const int32_t* local_rank; // [T_cap][k]: rank in the chunk, -1 for a route without a row
    const int32_t* chunk_base; // [chunks][E]
    const int32_t* offsets;    // [E + 1]
    const int32_t* live;
    WsHeader* hdr;
    int64_t T_cap;
    int E, H;
    void* rows;
    int32_t* row_of;           // [T_cap][k], the caller's order
    int32_t* offsets_out;      // [E + 1]
};

// A wave takes up to 1 KB of a token at a time, lane j holding route j's row, worked out from
// the permutation's ranks (worked out by every thread, 16K tokens took 146 us instead of 127)
template <int K, bool BF16>
__global__ void __launch_bounds__(256) dispatch_kernel(DispatchArgs a)
{
    const int64_t T = rows_live(a.live, a.T_cap);
    constexpr int N = row_cols<BF16>();
    const int nc = a.H / N, parts = (nc + 63) / 64;
    const int lane = threadIdx.x & 63;
    for (int64_t e = (int64_t)blockIdx.x * 256 + threadIdx.x; e <= a.E; e += (int64_t)gridDim.x * 256)
        a.offsets_out[e] = a.offsets[e];
    const int64_t waves = (int64_t)gridDim.x * 4;
    const int64_t first = (int64_t)blockIdx.x * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    for (int64_t job = first; job < T * parts; job += waves) {
        const int64_t t = job / parts;
        const int part = (int)(job - t * parts), c = 64 * part + lane;
        RowN<BF16, N> v;
        if (c < nc) v.load(a.x, t * a.H + N * c);
        int d = -1;
        if (lane < K) {
            const int e = a.sorted_ids[t * K + lane];
            d = a.local_rank[t * K + lane];
            if (d >= 0) d += a.offsets[e] + a.chunk_base[t / kChunkTok * a.E + e];
        }
#pragma unroll
        for (int j = 0; j < K; ++j) {
            const int r = __builtin_amdgcn_readlane(d, j);
            if (r >= 0 && c < nc) v.store(a.rows, (int64_t)r * a.H + N * c);
        }
        if (part == 0) {
            // the canonical order is a stable sort by id: a route's place is its id's rank
            const int id = a.ids[t * K + min(lane, K - 1)];
            int rank = 0;
#pragma unroll
            for (int i = 0; i < K; ++i) {
                const int o = __builtin_amdgcn_readlane(id, i);
                rank += (o < id || (o == id && i < lane)) ? 1 : 0;
            }
            const int r = __builtin_amdgcn_ds_bpermute(4 * rank, d);
            if (lane < K) a.row_of[t * K + lane] = r;
        }
    }
}

// Up to 256 tokens: one launch, every workgroup working out the whole permutation in LDS (a
// map of each expert's tokens, as the forward's permutation has it) and copying its own
// tokens; the first also writes the indices.  256 tokens, 64 experts, top-6: 11.2 us with
// the permutation in a launch of its own, 5.8 so.
template <int K, bool BF16>
__global__ void __launch_bounds__(256) dispatch_small_kernel(DispatchArgs a)
{
    __shared__ __attribute__((aligned(16))) uint32_t bm[kMaxExperts * (kChunkTok / 32)];
    __shared__ int off[kMaxExperts];
    __shared__ int dst[kChunkTok * K];
    __shared__ int wave_sum[4];
    __shared__ uint32_t wave_err[4];
    constexpr int N = row_cols<BF16>();
    const int nc = a.H / N, tid = threadIdx.x, lane = tid & 63, wid = tid >> 6;
    const int E = a.E;
    int id[K];
#pragma unroll
    for (int j = 0; j < K; ++j) id[j] = tid < a.T_cap ? a.ids[tid * K + j] : -1;
    const int32_t live = *a.live;
    const int T = (int)rows_live(a.live, a.T_cap);
    for (int i = tid; i < E * (kChunkTok / 32); i += 256) bm[i] = 0;
    __syncthreads();
    uint32_t err = 0;
    bool keep[K];
#pragma unroll
    for (int j = 0; j < K; ++j) {
        const bool in = id[j] >= 0 && id[j] < E;
        bool dup = false;
#pragma unroll
        for (int i = 0; i < j; ++i) dup |= id[i] == id[j];
        keep[j] = tid < T && in && !dup;
        if (tid < T) err |= (in ? 0u : kErrBadId) | (dup ? kErrDupId : 0u);
        if (keep[j]) atomicOr(&bm[id[j] * 8 + (tid >> 5)], 1u << (tid & 31));
    }
    __syncthreads();
    // experts 4 tid .. 4 tid + 3: their counts, then the exclusive sum over all before
    int cnt[4], mine = 0;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        cnt[q] = 0;
        if (4 * tid + q < E)
#pragma unroll
            for (int w = 0; w < 8; ++w) cnt[q] += __popc(bm[(4 * tid + q) * 8 + w]);
        mine += cnt[q];
    }
    int sum = mine;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
        const int up = __shfl_up(sum, o, kWave);
        if (lane >= o) sum += up;
    }
    const uint64_t bad = __ballot(err & kErrBadId), dupl = __ballot(err & kErrDupId);
    if (lane == 63) wave_sum[wid] = sum;
    if (lane == 0) wave_err[wid] = (bad ? kErrBadId : 0u) | (dupl ? kErrDupId : 0u);
    __syncthreads();
    int before = sum - mine, total = 0;
#pragma unroll
    for (int w = 0; w < 4; ++w) {
        if (w < wid) before += wave_sum[w];
        total += wave_sum[w];
    }
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        if (4 * tid + q < E) {
            off[4 * tid + q] = before;
            if (blockIdx.x == 0) a.offsets_out[4 * tid + q] = before;
        }
        before += cnt[q];
    }
    __syncthreads();
    // a route's row: its expert's first, and the expert's tokens below this one
#pragma unroll
    for (int j = 0; j < K; ++j) {
        int r = -1;
        if (keep[j]) {
            r = off[id[j]];
            const uint32_t* m = bm + id[j] * 8;
#pragma unroll
            for (int w = 0; w < 8; ++w)
                r += __popc(m[w] & (w < (tid >> 5) ? ~0u : w == (tid >> 5) ? (1u << (tid & 31)) - 1u : 0u));
        }
        dst[tid * K + j] = r;
        if (blockIdx.x == 0 && tid < T) a.row_of[tid * K + j] = r;
    }
    if (blockIdx.x == 0 && tid == 0) {
        a.offsets_out[E] = total;
        uint32_t all = (live < 0 ? kErrLiveNeg : 0u) | (live > a.T_cap ? kErrLiveHigh : 0u);
#pragma unroll
        for (int w = 0; w < 4; ++w) all |= wave_err[w];
        a.hdr->err = all;
        a.hdr->mark = kErrMark;
        a.hdr->T = T;
        a.hdr->n_rows = total;
        a.hdr->tag = kOtherTag;                          // holds no forward's rows
    }
    __syncthreads();
    // tokens blockIdx.x, blockIdx.x + gridDim.x, ..
    const int mine_n = T > (int)blockIdx.x ? (T - 1 - (int)blockIdx.x) / (int)gridDim.x + 1 : 0;
    for (int i = tid; i < mine_n * nc; i += 256) {
        const int n = i / nc, c = i - n * nc;
        const int t = blockIdx.x + n * gridDim.x;
        RowN<BF16, N> v;
        v.load(a.x, (int64_t)t * a.H + N * c);
#pragma unroll
        for (int j = 0; j < K; ++j) {
            const int r = dst[t * K + j];
            if (r >= 0) v.store(a.rows, (int64_t)r * a.H + N * c);
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

// The tokens' columns of workgroup `block` of `blocks`
template <int K, bool IN_BF16, bool OUT_BF16>
__device__ __forceinline__ void combine_tokens(const CombineArgs& a, int block, int blocks)
{
    const int64_t T = rows_live(a.live, a.T_cap);
    constexpr int N = row_cols<IN_BF16>();
    const int nc = a.H / N;
    const int64_t i0 = (int64_t)block * blockDim.x + threadIdx.x, step = (int64_t)blocks * blockDim.x;
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
        RowN<IN_BF16, N> v[K];
#pragma unroll
        for (int j = 0; j < K; ++j)
            if (d[j] != 0xffffffffu) v[j].load(a.rows, (int64_t)d[j] * a.H + N * c);
            else v[j].zero();
        float acc[N] = {};
#pragma unroll
        for (int j = 0; j < K; ++j) {
            if (d[j] == 0xffffffffu) continue;
            float f[N];
            v[j].get(f);
#pragma unroll
            for (int n = 0; n < N; ++n) acc[n] = __builtin_fmaf(p[j], f[n], acc[n]);
        }
        RowN<OUT_BF16, N> o;
        o.set(acc);
        o.store(a.out, t * a.H + N * c);
    }
}

template <int K, bool IN_BF16, bool OUT_BF16>
__global__ void __launch_bounds__(256) combine_kernel(CombineArgs a)
{
    combine_tokens<K, IN_BF16, OUT_BF16>(a, blockIdx.x, gridDim.x);
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
    constexpr int N = row_cols<ROWS_BF16>();
    const int nc = a.H / N, lane = threadIdx.x & 63;
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
            RowN<OUT_BF16, N> g;
            g.load(a.d_out, t * a.H + N * c);
            RowN<ROWS_BF16, N> v[K];
            if constexpr (PROBS) {
#pragma unroll
                for (int j = 0; j < K; ++j)
                    if (d[j] >= 0) v[j].load(a.rows, (int64_t)d[j] * a.H + N * c);
                    else v[j].zero();
            }
            float gf[N];
            g.get(gf);
#pragma unroll
            for (int j = 0; j < K; ++j) {
                if (d[j] < 0) continue;
                float f[N];
                if constexpr (PROBS) {
                    v[j].get(f);
#pragma unroll
                    for (int n = 0; n < N; ++n) dot[j] = __builtin_fmaf(gf[n], f[n], dot[j]);
                }
#pragma unroll
                for (int n = 0; n < N; ++n) f[n] = p[j] * gf[n];
                RowN<ROWS_BF16, N> o;
                o.set(f);
                o.store(a.d_rows, (int64_t)d[j] * a.H + N * c);
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

// d_x from the rows of its gradient (an fp32 sum in ascending row order), by the first `blocks_x` workgroups, and
// d_probs[t][j] of the caller's route j from the n_part partial sums of its row, 8 lanes a
// route (in the same launch: a launch of its own cost 3 us at 64 tokens, and a thread a route
// 27 us at 16K tokens)
struct GradEndsArgs {
    const uint16_t* dx;        // [rows][H] codes and [rows][H / 16] scales of x's gradient
    const uint8_t* dx_scale;
    const int32_t* dst;        // rows by route, canonical order
    const int32_t* live;
    int64_t T_cap;
    int H;
    uint16_t* d_x;             // bf16 [T_cap][H]
    const float* part;
    int n_part;
    const int32_t* ids;
    float* d_probs;
    int blocks_x;
};

template <int K>
__global__ void __launch_bounds__(256) grad_ends_kernel(GradEndsArgs a)
{
    const int64_t T = rows_live(a.live, a.T_cap);
    if ((int)blockIdx.x < a.blocks_x) {
        const int nc = a.H / 8;
        for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < T * nc; i += (int64_t)a.blocks_x * 256) {
            const int64_t t = i / nc;
            const int c = (int)(i - t * nc);
            int d[K];
            uint32_t b[K];
            RowN<true, 8> v[K];
#pragma unroll
            for (int j = 0; j < K; ++j) d[j] = a.dst[t * K + j];
#pragma unroll
            for (int j = 0; j < K; ++j) {
                b[j] = 0;
                v[j].zero();
                if (d[j] >= 0) {
                    v[j].load(a.dx, (int64_t)d[j] * a.H + 8 * c);
                    b[j] = a.dx_scale[(int64_t)d[j] * (a.H / 16) + (c >> 1)];
                }
            }
            float acc[8] = {};
#pragma unroll
            for (int j = 0; j < K; ++j) {
                if (d[j] < 0) continue;
#pragma unroll
                for (int n = 0; n < 4; ++n) {
                    float lo, hi;
                    dx_unpack(v[j].w[n], b[j], lo, hi);
                    acc[2 * n] += lo;
                    acc[2 * n + 1] += hi;
                }
            }
            RowN<true, 8> o;
            o.set(acc);
            o.store(a.d_x, t * a.H + 8 * c);
        }
        return;
    }
    const int sub = threadIdx.x & 7;
    const int64_t first = (int64_t)(blockIdx.x - a.blocks_x) * 32 + (threadIdx.x >> 3);
    for (int64_t r = first; r < T * K; r += (int64_t)(gridDim.x - a.blocks_x) * 32) {
        const int64_t t = r / K;
        const int j = (int)(r - t * K);
        const int id = a.ids[r];
        int rank = 0;                                   // the route's place in the canonical order
#pragma unroll
        for (int i = 0; i < K; ++i) {
            const int o = a.ids[t * K + i];
            rank += (o < id || (o == id && i < j)) ? 1 : 0;
        }
        const int d = a.dst[t * K + rank];
        float s = 0.0f;
        if (d >= 0)
            for (int i = sub; i < a.n_part; i += 8) s += a.part[(int64_t)d * a.n_part + i];
        s += __shfl_xor(s, 1);
        s += __shfl_xor(s, 2);
        s += __shfl_xor(s, 4);
        if (sub == 0) a.d_probs[r] = s;
    }
}

// fp32 rows rounded to bf16, the operand type of the products
__global__ void __launch_bounds__(256) cast_rows_kernel(const float* in, const int32_t* live, int64_t T_cap, int H,
                                                        uint16_t* out)
{
    const int64_t n = rows_live(live, T_cap) * (H / 8);
    for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < n; i += (int64_t)gridDim.x * blockDim.x) {
        RowN<false, 8> v;
        v.load(in, 8 * i);
        float f[8];
        v.get(f);
        RowN<true, 8> o;
        o.set(f);
        *(u4v*)(out + 8 * i) = u4v{o.w[0], o.w[1], o.w[2], o.w[3]};
    }
}

// ---------------------------------------------------------------- launches

// Up to 64 workgroups a CU, looping above that: at 16K tokens (hidden 2048, top-8) sums of
// fp32 rows 206 us against 222 with 16 a CU, dispatch 117 against 126; workgroups past the
// live tokens of a large capacity start and exit (6 us for 16,384 of them)
static dim3 rows_grid(int64_t threads, int num_cu)
{
    int64_t b = (threads + 255) / 256;
    const int64_t most = (int64_t)num_cu * 64;
    if (b > most) b = most;
    return dim3((unsigned)(b < 1 ? 1 : b));
}

#define ROWS_K(M)                                                                          \
    switch (k) {                                                                           \
        M(1) M(2) M(3) M(4) M(5) M(6) M(7) M(8) M(9) M(10) M(11) M(12) M(13) M(14) M(15) M(16) \
        default: return hipErrorInvalidValue;                                              \
    }

bool dispatch_in_one(int64_t T_cap) { return T_cap <= kChunkTok; }

hipError_t launch_dispatch(const void* x, int bf16, const int32_t* ids, char* ws, const WsLayout& L,
                           const int32_t* live, int64_t T_cap, int E, int k, int H, void* rows, int32_t* row_of,
                           int32_t* offsets_out, int num_cu, hipStream_t s)
{
    const DispatchArgs a{x, ids, (const int32_t*)(ws + L.sorted_ids), (const int32_t*)(ws + L.local_rank),
                         (const int32_t*)(ws + L.chunk_base), (const int32_t*)(ws + L.offsets), live,
                         (WsHeader*)(ws + L.hdr), T_cap, E, H, rows, row_of, offsets_out};
    const bool one = dispatch_in_one(T_cap);
    const dim3 b(256);
    const int nc = H / (bf16 ? 8 : 4);
    dim3 g = rows_grid(one ? T_cap * nc : T_cap * ((nc + 63) / 64 * 64), num_cu);
    if (one) g = dim3((unsigned)(g.x < (unsigned)num_cu ? g.x : (unsigned)num_cu));
#define M(K)                                                                                   \
    case K:                                                                                    \
        if (one && bf16) hipLaunchKernelGGL((dispatch_small_kernel<K, true>), g, b, 0, s, a);  \
        else if (one) hipLaunchKernelGGL((dispatch_small_kernel<K, false>), g, b, 0, s, a);    \
        else if (bf16) hipLaunchKernelGGL((dispatch_kernel<K, true>), g, b, 0, s, a);          \
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
    const dim3 g = rows_grid(T_cap * (H / (in_bf16 ? 8 : 4)), num_cu), b(256);
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

hipError_t launch_grad_ends(const uint16_t* rows, const uint8_t* scales, const int32_t* dst, const float* part, int n_part, const int32_t* ids,
                            const int32_t* live, int64_t T_cap, int k, int H, void* d_x, float* d_probs, int num_cu,
                            hipStream_t s)
{
    const dim3 gx = rows_grid(T_cap * (H / 8), num_cu), gp = rows_grid(T_cap * k * 8, num_cu), b(256);
    const GradEndsArgs a{rows, scales, dst, live, T_cap, H, (uint16_t*)d_x, part, n_part, ids, d_probs, (int)gx.x};
#define M(K)                                                                                   \
    case K:                                                                                    \
        hipLaunchKernelGGL(grad_ends_kernel<K>, dim3(gx.x + gp.x), b, 0, s, a);                \
        break;
    ROWS_K(M)
#undef M
    return hipGetLastError();
}

hipError_t launch_cast_rows(const float* in, const int32_t* live, int64_t T_cap, int H, uint16_t* out, int num_cu,
                            hipStream_t s)
{
    hipLaunchKernelGGL(cast_rows_kernel, rows_grid(T_cap * (H / 8), num_cu), dim3(256), 0, s, in, live, T_cap, H, out);
    return hipGetLastError();
}

}  // namespace moe
