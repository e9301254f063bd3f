// Training operators of the router: the balance and z losses with per-expert
// counts, the gradient of the logits, and the gradient of the combine's
// probabilities.
//
// With p_t = softmax(z_t) over the E logits of token t, N counted tokens (live,
// and not masked), c_e the number of their routes to expert e:
//   balance = E / (k N^2) sum_e c_e sum_t p_te      (1 for a balanced router)
//   z       = 1 / N sum_t lse(z_t)^2
// and, for gradients gb, gz of the two losses and d_tj of the selected
// probabilities q_tj = exp(z_tj) / sum_i exp(z_ti) (i, j over the token's routes),
//   dz_te = gb E / (k N^2) p_te (c_e - sum_i p_ti c_i) + gz 2 lse_t / N p_te
//         + [e = id_tj] q_tj (d_tj - sum_i q_ti d_ti).
//
// Both logit kernels are one pass over the logits.  A token is 16 lanes (E up to
// 256: four tokens a wave, so that a 64-expert row is one 16-byte load a lane) or a
// whole wave (more experts), its logits in registers, the next token's loads in
// flight while one is computed.  Sums are fp32 in a fixed order: a lane's tokens,
// a workgroup's waves through LDS, the workgroups' partials in the second launch;
// nothing is added by floating-point atomics.
#include "common.h"

namespace moe {

constexpr int kBalThreads = 1024, kBalWaves = kBalThreads / kWave;
constexpr int kBalMaxBlocks = 512;             // partials of the balance workspace
constexpr int kGradThreads = 512, kGradWaves = kGradThreads / kWave;

typedef float f32x4_t __attribute__((ext_vector_type(4)));

template <int CTRL>
__device__ __forceinline__ float dpp(float v)
{
    return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), CTRL, 0xf, 0xf, true));
}
__device__ __forceinline__ float lane_of(float v, int lane)
{
    return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), lane));
}

// Sum (maximum) over the LPT lanes of a token, the same bits in each of them:
// lane i with i ^ 1, i ^ 2, then the mirrored lane of 8 and of 16 (equal quads and
// halves by then), then the four rows of a wave in order.
template <int LPT>
__device__ __forceinline__ float token_sum(float v)
{
    v += dpp<0xB1>(v);
    v += dpp<0x4E>(v);
    v += dpp<0x141>(v);
    v += dpp<0x140>(v);
    if constexpr (LPT == 64) v = ((lane_of(v, 0) + lane_of(v, 16)) + lane_of(v, 32)) + lane_of(v, 48);
    return v;
}
template <int LPT>
__device__ __forceinline__ float token_max(float v)
{
    v = fmaxf(v, dpp<0xB1>(v));
    v = fmaxf(v, dpp<0x4E>(v));
    v = fmaxf(v, dpp<0x141>(v));
    v = fmaxf(v, dpp<0x140>(v));
    if constexpr (LPT == 64)
        v = fmaxf(fmaxf(lane_of(v, 0), lane_of(v, 16)), fmaxf(lane_of(v, 32), lane_of(v, 48)));
    return v;
}

// LDS accesses of one wave complete in program order: only the compiler has to
// keep them so
__device__ __forceinline__ void lds_order() { asm volatile("" : : : "memory"); }

// Sum over the waves of a workgroup of each wave's lane-0 value, in wave order.
template <int WAVES, typename T>
__device__ __forceinline__ T block_sum(T v, T* lds)
{
    const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6;
    __syncthreads();
    if (lane == 0) lds[wv] = v;
    __syncthreads();
    T s = 0;
#pragma unroll
    for (int w = 0; w < WAVES; ++w) s += lds[w];
    return s;
}

// sum over a wave, in every lane
__device__ __forceinline__ float wave_sum(float v) { return token_sum<64>(v); }
__device__ __forceinline__ int wave_sum(int v)
{
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o, kWave);
    return v;
}

// One token's logits: 4 N per lane.  VEC (E a multiple of 4, so rows are 16-byte
// aligned): lane l holds elements 4 (i LPT + l) + q; else i LPT 4 + q LPT + l.
// STREAM: non-temporal loads (a compile-time choice: of two loads of one address the
// compiler makes one).
template <int LPT, int N, bool VEC, bool STREAM>
struct Row {
    float z[4 * N];
    static __device__ __forceinline__ int at(int l, int i, int q)
    {
        return VEC ? 4 * (i * LPT + l) + q : (4 * i + q) * LPT + l;
    }
    __device__ __forceinline__ void load(const float* row, int l, int E)
    {
#pragma unroll
        for (int i = 0; i < N; ++i) {
            if constexpr (VEC) {
                f32x4_t v = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
                if (at(l, i, 0) < E) {
                    if constexpr (STREAM) v = __builtin_nontemporal_load((const f32x4_t*)(row + at(l, i, 0)));
                    else v = *(const f32x4_t*)(row + at(l, i, 0));
                }
#pragma unroll
                for (int q = 0; q < 4; ++q) z[4 * i + q] = v[q];
            } else {
#pragma unroll
                for (int q = 0; q < 4; ++q) z[4 * i + q] = at(l, i, q) < E ? row[at(l, i, q)] : -INFINITY;
            }
        }
    }
    // z becomes the softmax (all 0 for a row of -inf, which leaves nothing, and
    // then lse is 0 too); returns lse.  fmaxf drops NaN, so the maximum does not
    // tell a row of -inf from one that has NaN besides: the sum does, being 0 only
    // for the first (a finite maximum adds exp(0)) and NaN for the second.  The
    // exponential and the logarithm are the hardware's base-2 ones times a rounded
    // constant, off by (2 |z - m| + 2) 2^-24 of an exponential.  256 tokens' losses come
    // out to 1e-7 (a plain fp32 form: 3e-8); expf and logf in their place take 6.5 us
    // there, 5.5 so, and 54.8 / 50.6 at 65,536 x 1024.
    __device__ __forceinline__ float softmax()
    {
        float m = z[0];
#pragma unroll
        for (int i = 1; i < 4 * N; ++i) m = fmaxf(m, z[i]);
        m = token_max<LPT>(m);
        if (m == -INFINITY) m = 0.0f;
        float s = 0.0f;
#pragma unroll
        for (int i = 0; i < 4 * N; ++i) {
            z[i] = __expf(z[i] - m);
            s += z[i];
        }
        s = token_sum<LPT>(s);
        const bool none = s == 0.0f;
        const float r = none ? 0.0f : 1.0f / s;
#pragma unroll
        for (int i = 0; i < 4 * N; ++i) z[i] *= r;
        return none ? 0.0f : m + __logf(s);
    }
};

struct BalanceArgs {
    const float* logits;
    const int32_t* ids;
    const int32_t* live;
    const uint8_t* mask;       // or null: every live token counts
    int64_t T_cap;
    int E, k;
    float* losses;             // [2]: balance, z
    int32_t* counts;           // [E + 1]: per expert, then the counted tokens
    float* prob_sums;          // [E]
    // workspace: partials of each workgroup of the first launch
    WsHeader* hdr;             // a forward's, if the buffer held one: its tag is cleared
    uint32_t* ticket;          // second launch's workgroups that are done
    float* part_dot;           // their sums of c_e sum_t p_te
    float* part_z;
    int32_t* part_n;
    float* part_p;             // [blocks][E]
    int32_t* part_c;           // [blocks][E]
};

__device__ __forceinline__ void write_losses(const BalanceArgs& a, float dot, float z, int n)
{
    const float inv = n > 0 ? 1.0f / (float)n : 0.0f;
    a.losses[0] = (float)a.E / (float)a.k * inv * (dot * inv);
    a.losses[1] = z * inv;
    a.counts[a.E] = n;
}

template <int LPT, int N, bool VEC, bool STREAM>
__global__ void __launch_bounds__(kBalThreads) balance_kernel(BalanceArgs a)
{
    constexpr int GPW = kWave / LPT;            // tokens per wave
    __shared__ float slot[kBalWaves * LPT * 4 * N];
    __shared__ int cnt[LPT * 4 * N];
    __shared__ float lds_f[kBalWaves];
    __shared__ int lds_i[kBalWaves];
    const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6, l = lane % LPT;
    const int E = a.E, k = a.k;
    const int32_t live = *a.live;
    const int64_t T = live < 0 ? 0 : (live > a.T_cap ? a.T_cap : live);
    for (int e = threadIdx.x; e < E; e += kBalThreads) cnt[e] = 0;
    __syncthreads();

    float acc[4 * N];
#pragma unroll
    for (int i = 0; i < 4 * N; ++i) acc[i] = 0.0f;
    float zs = 0.0f;
    int n = 0;
    struct Tok {
        Row<LPT, N, VEC, STREAM> r;
        int keep, id;
    };
    auto fetch = [&](int64_t t0, Tok& x) {
        const int64_t t = t0 + lane / LPT, tc = t < T ? t : T - 1;
        x.r.load(a.logits + tc * E, l, E);
        x.keep = t < T && (!a.mask || a.mask[tc] != 0);
        x.id = l < k ? a.ids[tc * k + l] : -1;
    };
    const int64_t stride = (int64_t)gridDim.x * kBalWaves * GPW;
    int64_t t0 = ((int64_t)blockIdx.x * kBalWaves + wv) * GPW;
    Tok cur, nxt;
    if (t0 < T) fetch(t0, cur);
    for (; t0 < T; t0 += stride) {
        if (t0 + stride < T) fetch(t0 + stride, nxt);
        const float lse = cur.r.softmax();
        if (cur.keep) {
#pragma unroll
            for (int i = 0; i < 4 * N; ++i) acc[i] += cur.r.z[i];
            zs += lse * lse;
            n += 1;
            if (cur.id >= 0 && cur.id < E) atomicAdd(&cnt[cur.id], 1);
        }
        cur = nxt;
    }
    // the tokens of a wave, then the waves
#pragma unroll
    for (int o = LPT; o < kWave; o <<= 1) {
#pragma unroll
        for (int i = 0; i < 4 * N; ++i) acc[i] += __shfl_xor(acc[i], o, kWave);
        zs += __shfl_xor(zs, o, kWave);
        n += __shfl_xor(n, o, kWave);
    }
    if (lane < LPT)
#pragma unroll
        for (int i = 0; i < N; ++i)
#pragma unroll
            for (int q = 0; q < 4; ++q) slot[wv * (LPT * 4 * N) + Row<LPT, N, VEC, STREAM>::at(l, i, q)] = acc[4 * i + q];
    if (lane == 0) {
        lds_f[wv] = zs;
        lds_i[wv] = n;
    }
    __syncthreads();
    const bool whole = gridDim.x == 1;
    float dot = 0.0f;
    for (int e = threadIdx.x; e < E; e += kBalThreads) {
        float s = 0.0f;
#pragma unroll
        for (int w = 0; w < kBalWaves; ++w) s += slot[w * (LPT * 4 * N) + e];
        if (whole) {
            a.prob_sums[e] = s;
            a.counts[e] = cnt[e];
            dot += (float)cnt[e] * s;
        } else {
            a.part_p[(int64_t)blockIdx.x * E + e] = s;
            a.part_c[(int64_t)blockIdx.x * E + e] = cnt[e];
        }
    }
    float z_all = 0.0f;
    int n_all = 0;
    if (threadIdx.x == 0)
#pragma unroll
        for (int w = 0; w < kBalWaves; ++w) {
            z_all += lds_f[w];
            n_all += lds_i[w];
        }
    if (whole) {
        dot = block_sum<kBalWaves>(wave_sum(dot), lds_f);
        if (threadIdx.x == 0) write_losses(a, dot, z_all, n_all);
    } else if (threadIdx.x == 0) {
        a.part_z[blockIdx.x] = z_all;
        a.part_n[blockIdx.x] = n_all;
        if (blockIdx.x == 0) {
            *a.ticket = 0;
            a.hdr->err = 0;
            a.hdr->mark = kErrMark;
            a.hdr->tag = 0;
        }
    }
}

// Second launch: a workgroup sums the partials of EP experts, 1024 / EP threads an
// expert.  With more than one workgroup (E above EP) the last one to finish adds
// their parts of the loss in order; the ticket that tells starts at zero in every
// call: the first launch clears it.  A release at device scope writes the L2 back,
// so up to 128 experts one workgroup takes them all.
template <int EP>
__global__ void __launch_bounds__(kBalThreads) balance_finish_kernel(BalanceArgs a, int blocks)
{
    constexpr int PER = kBalThreads / EP;       // threads per expert
    __shared__ float ps[PER][EP];
    __shared__ int cs[PER][EP];
    __shared__ float lds_f[kBalWaves];
    __shared__ int lds_i[kBalWaves];
    __shared__ float lds_d[EP / kWave];
    const int E = a.E, x = threadIdx.x % EP, y = threadIdx.x / EP;
    const int e = blockIdx.x * EP + x, ec = e < E ? e : E - 1;
    float zb = 0.0f;
    int nb = 0;
    if (threadIdx.x < (unsigned)blocks) {        // blocks <= kBalMaxBlocks < the workgroup
        zb = a.part_z[threadIdx.x];
        nb = a.part_n[threadIdx.x];
    }
    float s = 0.0f;
    int c = 0;
#pragma unroll 16
    for (int b = y; b < blocks; b += PER) {
        s += a.part_p[(int64_t)b * E + ec];
        c += a.part_c[(int64_t)b * E + ec];
    }
    ps[y][x] = s;
    cs[y][x] = c;
    zb = wave_sum(zb);
    nb = wave_sum(nb);
    if ((threadIdx.x & 63) == 0) {
        lds_f[threadIdx.x >> 6] = zb;
        lds_i[threadIdx.x >> 6] = nb;
    }
    __syncthreads();
    float dot = 0.0f;
    if (threadIdx.x < EP) {
        s = 0.0f;
        c = 0;
#pragma unroll
        for (int w = 0; w < PER; ++w) {
            s += ps[w][x];
            c += cs[w][x];
        }
        if (e < E) {
            a.prob_sums[e] = s;
            a.counts[e] = c;
            dot = (float)c * s;
        }
    }
    // (only the first EP / 64 waves have a part of it)
    dot = wave_sum(dot);
    if (threadIdx.x < EP && (threadIdx.x & 63) == 0) lds_d[threadIdx.x >> 6] = dot;
    if constexpr (EP > kWave) __syncthreads();
    if (threadIdx.x != 0) return;
    dot = 0.0f;
    float z = 0.0f;
    int n = 0;
#pragma unroll
    for (int w = 0; w < EP / kWave; ++w) dot += lds_d[w];
#pragma unroll
    for (int w = 0; w < kBalWaves; ++w) {
        z += lds_f[w];
        n += lds_i[w];
    }
    if (gridDim.x == 1) {
        write_losses(a, dot, z, n);
        return;
    }
    __hip_atomic_store(&a.part_dot[blockIdx.x], dot, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    const uint32_t before = __hip_atomic_fetch_add(a.ticket, 1u, __ATOMIC_ACQ_REL, __HIP_MEMORY_SCOPE_AGENT);
    if (before == gridDim.x - 1) {
        float d = 0.0f;
        for (unsigned g = 0; g < gridDim.x; ++g)
            d += __hip_atomic_load(&a.part_dot[g], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        write_losses(a, d, z, n);
    }
}

static size_t up256(size_t v) { return (v + 255) / 256 * 256; }

// tokens that a workgroup of the first launch takes at a time
static int64_t balance_tokens(int E) { return E <= 256 ? kBalWaves * 4 : kBalWaves; }

static int64_t balance_blocks(int E, int64_t T_cap, int64_t most)
{
    // One workgroup (then the whole operator is one launch) up to four turns of
    // it, else one turn a workgroup: the crossover for every width.  One launch
    // against two, us: 64 experts, 256 tokens 5.5 / 5.8-7.4, 384 7.0 / 5.9-7.4, 512
    // 8.4 / 5.9-7.4; 128 experts, 256 tokens 6.6 / 6.4-7.4, 512 10.3 / 6.6-7.4; 256
    // experts, 128 tokens 6.3 / 8.3, 256 9.0 / 8.4; 512 experts, 64 tokens 6.4 / 7.8,
    // 128 10.5 / 7.9; 1024 experts, 64 tokens 8.8 / 9.3, 128 14.3 / 9.4 (ranges: the
    // second launch's cost differs between processes)
    const int64_t per = balance_tokens(E);
    if (T_cap <= 4 * per) return 1;
    const int64_t b = (T_cap + per - 1) / per;
    return b < most ? b : most;
}

// Logits past the 256 MB Infinity Cache are read (and their gradient written)
// non-temporally (65,536 x 1024: balance 58.7 -> 52.4 us, route_backward 106.4 -> 97.9); smaller
// ones, which the router has just written, are not (16,384 x 128: 9.4 us, 9.9
// non-temporally).
static bool stream_logits(int E, int64_t T_cap) { return T_cap * E * 4 >= ((int64_t)256 << 20); }

size_t balance_ws_bytes(int E, int64_t T_cap)
{
    const size_t b = (size_t)balance_blocks(E, T_cap, kBalMaxBlocks);
    return sizeof(WsHeader) + up256(4) + up256(4 * kMaxExperts / kWave) + 2 * up256(4 * b) + 2 * up256(4 * b * E);
}

#define ROW_BY_E(E, CALL, VEC, STREAM)                                                            \
    do {                                                                                          \
        if ((E) <= 64) CALL(16, 1, VEC, STREAM);                                                  \
        else if ((E) <= 128) CALL(16, 2, VEC, STREAM);                                            \
        else if ((E) <= 256) CALL(16, 4, VEC, STREAM);                                            \
        else if ((E) <= 512) CALL(64, 2, VEC, STREAM);                                            \
        else CALL(64, 4, VEC, STREAM);                                                            \
    } while (0)
// the rows of E not a multiple of 4 are not aligned: four-byte accesses, never streamed
#define ROW_DISPATCH(E, T_cap, CALL)                                                              \
    do {                                                                                          \
        if ((E) % 4 != 0) ROW_BY_E(E, CALL, false, false);                                        \
        else if (stream_logits(E, T_cap)) ROW_BY_E(E, CALL, true, true);                          \
        else ROW_BY_E(E, CALL, true, false);                                                      \
    } while (0)

hipError_t launch_balance(const float* logits, const int32_t* ids, int64_t T_cap, const int32_t* live,
                          const uint8_t* mask, int E, int k, float* losses, int32_t* counts, float* prob_sums,
                          char* ws, int num_cu, hipStream_t s)
{
    const int64_t blocks = balance_blocks(E, T_cap, num_cu < kBalMaxBlocks ? num_cu : kBalMaxBlocks);
    BalanceArgs a{logits, ids, live, mask, T_cap, E, k, losses, counts, prob_sums};
    size_t o = 0;
    auto take = [&](size_t bytes) { char* p = ws + o; o += up256(bytes); return p; };
    a.hdr = (WsHeader*)take(sizeof(WsHeader));
    a.ticket = (uint32_t*)take(4);
    a.part_dot = (float*)take(4 * kMaxExperts / kWave);
    a.part_z = (float*)take(4 * blocks);
    a.part_n = (int32_t*)take(4 * blocks);
    a.part_p = (float*)take(4 * blocks * E);
    a.part_c = (int32_t*)take(4 * blocks * E);
#define BALANCE(LPT, N, VEC, STREAM) \
    hipLaunchKernelGGL((balance_kernel<LPT, N, VEC, STREAM>), dim3((unsigned)blocks), dim3(kBalThreads), 0, s, a)
    ROW_DISPATCH(E, T_cap, BALANCE);
#undef BALANCE
    if (blocks > 1) {
        if (E > 64 && E <= 128)
            hipLaunchKernelGGL(balance_finish_kernel<128>, dim3(1), dim3(kBalThreads), 0, s, a, (int)blocks);
        else
            hipLaunchKernelGGL(balance_finish_kernel<64>, dim3((unsigned)((E + 63) / 64)), dim3(kBalThreads), 0, s, a,
                               (int)blocks);
    }
    return hipGetLastError();
}

struct RouteGradArgs {
    const float* logits;
    const int32_t* ids;
    const float* probs;        // with d_probs, or null: no gradient of the probabilities
    const float* d_probs;
    const int32_t* live;
    const uint8_t* mask;
    const int32_t* counts;     // [E + 1], with d_losses, or null: no gradient of the losses
    const float* d_losses;     // [2]
    float* d_logits;
    int64_t T_cap;
    int E, k;
};

// The sparse terms reach the lanes that hold their experts through one LDS row per
// token (zero between tokens).  The balance term is taken with c_e - k N / E in
// place of c_e (the gradient is the same, sum_e p_te being 1), an exact integer
// difference, so nothing is lost where the loads are nearly even.
template <int LPT, int N, bool VEC, bool STREAM>
__global__ void __launch_bounds__(kGradThreads) route_backward_kernel(RouteGradArgs a)
{
    constexpr int GPW = kWave / LPT;
    constexpr int W = LPT * 4 * N;              // floats of a token's LDS row
    __shared__ __attribute__((aligned(16))) float rows[kGradWaves * GPW * W];
    const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6, l = lane % LPT;
    const int E = a.E, k = a.k;
    const int32_t live = *a.live;
    const int64_t T = live < 0 ? 0 : (live > a.T_cap ? a.T_cap : live);
    const int64_t stride = (int64_t)gridDim.x * kGradWaves * GPW;
    int64_t t0 = ((int64_t)blockIdx.x * kGradWaves + wv) * GPW;
    if (t0 >= T) return;                        // (no barrier below)
    float* const row = rows + (wv * GPW + lane / LPT) * W;
    float ce[4 * N];                            // gb / (k N^2) (E c_e - k N) of this lane's experts
    float gz = 0.0f;
#pragma unroll
    for (int i = 0; i < 4 * N; ++i) ce[i] = 0.0f;
    if (a.counts) {
        const int n = a.counts[E];
        const float inv = n > 0 ? 1.0f / (float)n : 0.0f;
        const float gb = a.d_losses[0] / (float)k * inv * inv;
        gz = 2.0f * a.d_losses[1] * inv;
#pragma unroll
        for (int i = 0; i < N; ++i)
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const int e = Row<LPT, N, VEC, STREAM>::at(l, i, q);
                if (e < E) ce[4 * i + q] = gb * (float)((int64_t)a.counts[e] * E - (int64_t)k * n);
            }
    }
    if (a.d_probs)
        for (int i = l; i < W; i += LPT) row[i] = 0.0f;
    struct Tok {
        Row<LPT, N, VEC, STREAM> r;
        int keep, id;
        float q, d;
    };
    auto fetch = [&](int64_t t0, Tok& x) {
        const int64_t t = t0 + lane / LPT, tc = t < T ? t : T - 1;
        x.id = -1;
        x.q = x.d = 0.0f;
        if (a.d_probs && l < k) {
            x.id = a.ids[tc * k + l];
            x.q = a.probs[tc * k + l];
            x.d = a.d_probs[tc * k + l];
        }
        x.keep = a.counts && (!a.mask || a.mask[tc] != 0);
        if (a.counts) x.r.load(a.logits + tc * E, l, E);
    };
    Tok cur, nxt;
    fetch(t0, cur);
    for (; t0 < T; t0 += stride) {
        if (t0 + stride < T) fetch(t0 + stride, nxt);
        const int64_t t = t0 + lane / LPT;
        float g[4 * N];
#pragma unroll
        for (int i = 0; i < 4 * N; ++i) g[i] = 0.0f;
        if (a.counts) {
            const float lse = cur.r.softmax();
            float mean = 0.0f;
#pragma unroll
            for (int i = 0; i < 4 * N; ++i) mean += cur.r.z[i] * ce[i];
            const float shift = gz * lse - token_sum<LPT>(mean);
#pragma unroll
            for (int i = 0; i < 4 * N; ++i) g[i] = cur.keep ? cur.r.z[i] * (ce[i] + shift) : 0.0f;
        }
        if (a.d_probs) {
            bool ok = cur.id >= 0 && cur.id < E;
            // a repeated id: every lane writes its place, one of them stays
            if (ok) row[cur.id] = (float)l;
            lds_order();
            const bool lost = ok && row[cur.id] != (float)l;
            if (__ballot(lost)) {
                // only the first of equal ids is kept, as in the forward
                for (int i = 0; i < k; ++i) {
                    const int other = __shfl(cur.id, i, LPT);
                    if (i < l && other == cur.id) ok = false;
                }
            }
            const float q = ok ? cur.q : 0.0f, d = ok ? cur.d : 0.0f;
            const float v = q * (d - token_sum<LPT>(q * d));
            lds_order();
            if (ok) row[cur.id] = v;
            lds_order();
#pragma unroll
            for (int i = 0; i < N; ++i)
#pragma unroll
                for (int q4 = 0; q4 < 4; ++q4) g[4 * i + q4] += row[Row<LPT, N, VEC, STREAM>::at(l, i, q4)];
            lds_order();
            if (ok) row[cur.id] = 0.0f;
        }
        if (t < T) {
            float* out = a.d_logits + t * E;
#pragma unroll
            for (int i = 0; i < N; ++i) {
                if constexpr (VEC) {
                    const int e = Row<LPT, N, VEC, STREAM>::at(l, i, 0);
                    const f32x4_t v = {g[4 * i], g[4 * i + 1], g[4 * i + 2], g[4 * i + 3]};
                    if (e < E) {
                        if constexpr (STREAM) __builtin_nontemporal_store(v, (f32x4_t*)(out + e));
                        else *(f32x4_t*)(out + e) = v;
                    }
                } else {
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        const int e = Row<LPT, N, VEC, STREAM>::at(l, i, q);
                        if (e < E) out[e] = g[4 * i + q];
                    }
                }
            }
        }
        cur = nxt;
    }
}

hipError_t launch_route_backward(const float* logits, const int32_t* ids, const float* probs, const float* d_probs,
                                 int64_t T_cap, const int32_t* live, const uint8_t* mask, const int32_t* counts,
                                 const float* d_losses, float* d_logits, int E, int k, int num_cu, hipStream_t s)
{
    const RouteGradArgs a{logits, ids, probs, d_probs, live, mask, counts, d_losses, d_logits, T_cap, E, k};
    const int64_t per = kGradWaves * (E <= 256 ? 4 : 1);
    int64_t blocks = (T_cap + per - 1) / per;
    if (blocks > (int64_t)num_cu * 4) blocks = (int64_t)num_cu * 4;
    if (blocks < 1) blocks = 1;
#define ROUTE_GRAD(LPT, N, VEC, STREAM) \
    hipLaunchKernelGGL((route_backward_kernel<LPT, N, VEC, STREAM>), dim3((unsigned)blocks), dim3(kGradThreads), 0, s, a)
    ROW_DISPATCH(E, T_cap, ROUTE_GRAD);
#undef ROUTE_GRAD
    return hipGetLastError();
}

// Gradient of the combine's probabilities: with O the fp32 FC2 rows that the last
// forward left in its workspace,
//   d_probs[t][j] = sum_m d_out[t][m] O[row of route (t, j)][m],
// 0 for a dropped route, in the order in which the caller listed the ids.
// Memory bound: k rows of 4 H bytes and one of d_out per token.  K is a template
// parameter so that a token's row loads are all in flight.  TPT threads take a
// token: a wave when there are many, a workgroup of 512 when there are few (16,384
// tokens, top-8, hidden 2048: 183 us, 6.6 TB/s, against 187 with a workgroup each; 256
// tokens, top-6: 4.7 us against 14.3 with a wave each).
struct ProbsGradArgs {
    WsHeader* hdr;
    uint64_t tag;              // of the forward whose rows are read (WsHeader::tag)
    const float* O;
    const int32_t* dst;
    const int32_t* ids;
    const void* d_out;
    float* d_probs;
    int64_t T_cap;
    int H;
};

template <int K, bool BF16, int TPT>
__global__ void __launch_bounds__(512) probs_backward_kernel(ProbsGradArgs a)
{
    static_assert(TPT == 64 || TPT == 512, "a wave or a workgroup per token");
    __shared__ float part[8][K];
    const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6;
    constexpr int TOK = 512 / TPT;              // tokens per workgroup
    // the first token's row indices go out beside the header (workspace bytes that
    // exist up to T_cap, unused unless the header says that they are a forward's)
    int64_t t = (int64_t)blockIdx.x * TOK + (TPT == 64 ? wv : 0);
    int32_t d[K];
    auto indices = [&]() {
#pragma unroll
        for (int j = 0; j < K; ++j) d[j] = t < a.T_cap ? a.dst[t * K + j] : -1;
    };
    indices();
    const bool stale = a.hdr->tag != a.tag;
    if (stale || a.hdr->weighted) {
        // the bit joins those of an earlier call; in a workspace of none it is the word
        if (blockIdx.x == 0 && threadIdx.x == 0) {
            a.hdr->err = (a.hdr->mark == kErrMark ? a.hdr->err : 0u) | (stale ? kErrNoRows : kErrWeightedRows);
            a.hdr->mark = kErrMark;
        }
        return;
    }
    const uint32_t n_rows = (uint32_t)a.hdr->n_rows;
    const int64_t T = a.hdr->T < a.T_cap ? a.hdr->T : a.T_cap;
    const int H4 = a.H >> 2;                    // H is a multiple of 32
    for (; t < T; t += (int64_t)gridDim.x * TOK, indices()) {
        float acc[K];
#pragma unroll
        for (int j = 0; j < K; ++j) {
            if ((uint32_t)d[j] >= n_rows) d[j] = -1;
            acc[j] = 0.0f;
        }
        const int32_t id = lane < K ? a.ids[t * K + lane] : 0;
        for (int c = threadIdx.x % TPT; c < H4; c += TPT) {
            f32x4_t o[K], g;
#pragma unroll
            for (int j = 0; j < K; ++j) {
                o[j] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
                if (d[j] >= 0) o[j] = __builtin_nontemporal_load((const f32x4_t*)(a.O + (int64_t)d[j] * a.H) + c);
            }
            if constexpr (BF16) {
                const uint2 w = ((const uint2*)((const uint16_t*)a.d_out + t * a.H))[c];
                g = f32x4_t{bf16_bits_to_f32(w.x & 0xffffu), __uint_as_float(w.x & 0xffff0000u),
                            bf16_bits_to_f32(w.y & 0xffffu), __uint_as_float(w.y & 0xffff0000u)};
            } else {
                g = __builtin_nontemporal_load((const f32x4_t*)((const float*)a.d_out + t * a.H) + c);
            }
#pragma unroll
            for (int j = 0; j < K; ++j)
                if (d[j] >= 0)
#pragma unroll
                    for (int q = 0; q < 4; ++q) acc[j] = __builtin_fmaf(g[q], o[j][q], acc[j]);
        }
        // the place of listed route `lane` in canonical order (ascending id, equal
        // ids as listed)
        int rank = 0;
#pragma unroll
        for (int i = 0; i < K; ++i) {
            const int32_t other = __builtin_amdgcn_readlane(id, i);
            rank += other < id || (other == id && i < lane) ? 1 : 0;
        }
        float out = 0.0f;
#pragma unroll
        for (int j = 0; j < K; ++j) {
            const float s = wave_sum(acc[j]);
            if constexpr (TPT == 64) {
                if (rank == j) out = s;
            } else if (lane == 0) {
                part[wv][j] = s;
            }
        }
        if constexpr (TPT == 512) {
            __syncthreads();
            if (threadIdx.x < K)
#pragma unroll
                for (int w = 0; w < 8; ++w) out += part[w][rank];
            if (threadIdx.x < K) a.d_probs[t * K + threadIdx.x] = out;
            __syncthreads();                    // part is read until here
        } else if (lane < K) {
            a.d_probs[t * K + lane] = out;
        }
    }
}

hipError_t launch_probs_backward(WsHeader* hdr, uint64_t tag, const float* O, const int32_t* dst,
                                 const int32_t* ids, const void* d_out, int bf16, float* d_probs, int64_t T_cap, int k,
                                 int H, int num_cu, hipStream_t s)
{
    const ProbsGradArgs a{hdr, tag, O, dst, ids, d_out, d_probs, T_cap, H};
    const bool few = T_cap <= (int64_t)num_cu * 8;
    int64_t blocks = few ? T_cap : (T_cap + 7) / 8;
    if (blocks > (int64_t)num_cu * 8) blocks = (int64_t)num_cu * 8;
    const dim3 g((unsigned)(blocks < 1 ? 1 : blocks)), b(512);
#define PROBS_CASE(KK)                                                                                  \
    case KK:                                                                                            \
        if (bf16 && few) hipLaunchKernelGGL((probs_backward_kernel<KK, true, 512>), g, b, 0, s, a);     \
        else if (bf16) hipLaunchKernelGGL((probs_backward_kernel<KK, true, 64>), g, b, 0, s, a);        \
        else if (few) hipLaunchKernelGGL((probs_backward_kernel<KK, false, 512>), g, b, 0, s, a);       \
        else hipLaunchKernelGGL((probs_backward_kernel<KK, false, 64>), g, b, 0, s, a);                 \
        break;
    switch (k) {
        PROBS_CASE(1) PROBS_CASE(2) PROBS_CASE(3) PROBS_CASE(4) PROBS_CASE(5) PROBS_CASE(6) PROBS_CASE(7)
        PROBS_CASE(8) PROBS_CASE(9) PROBS_CASE(10) PROBS_CASE(11) PROBS_CASE(12) PROBS_CASE(13) PROBS_CASE(14)
        PROBS_CASE(15) PROBS_CASE(16)
        default: return hipErrorInvalidValue;
    }
#undef PROBS_CASE
    return hipGetLastError();
}

}  // namespace moe
