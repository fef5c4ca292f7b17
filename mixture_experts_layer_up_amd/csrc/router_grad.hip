// router_grad.hip -- the router in training: its balance loss with per-expert
// counts, and the gradient of its logits.
//
// With p_t = softmax(logits_t) over all E experts and the chosen ids of the k
// slots, over the N_s tokens of sequence s that take part:
//   n[s, e] = #{(t, j): id[t, j] = e},   P[s, e] = sum_t p[t, e] / N_s
//   L_s = E / (k N_s) sum_e n[s, e] P[s, e],   L = mean of L_s over N_s > 0
// The counts are constants of the gradient; dL reaches the logits through p:
//   g[s, e] = dL E n[s, e] / (k N_s^2 S'),   S' = sequences with N_s > 0
//   dlogits[t, e] = p[t, e] (g[s, e] - sum_f p[t, f] g[s, f])
// and the routing weights' gradient dw (w = the k softmax weights):
//   method 0 (softmax over the selected): dlogits[id_j] += w_j (dw_j - sum_i w_i dw_i)
//   method 1 (over all, at the selected): dlogits[id_j] += w_j dw_j,
//                                         dlogits[e] -= p_e sum_i w_i dw_i
// Rows of tokens that take no part are 0.
//
// All are one pass over [T, E] fp32, so memory bound for large batches: one
// wave per token, lane l holding experts l, l + 64, ... in registers, the row
// read once.  Sums over tokens run in a fixed order (registers, then waves,
// then chunks), in fp32; nothing is added atomically but integers.
//
// Measured: 32768 tokens, 256 experts, 9 sequences, a tenth of the tokens
// padding: balance loss 15.4 us (34 MB, 2.2 TB/s; by count about 6 us of it
// is the issue of the exponentials and row sums, the rest a block's chain: rows, sums over waves, counts)
// and 6.5 us for the reduction over chunks; gradient 21.8 us (70 MB, 3.2 TB/s).
// 64 tokens, 128 experts: 4.7 and 4.2 us, launch latency.
#include <algorithm>
#include <type_traits>

#include "device_common.h"
#include "kernels_router.h"

namespace moe_lora {
namespace {

constexpr int kBalanceWaves = 8;
constexpr int kBalanceThreads = kBalanceWaves * kWave;

__device__ __forceinline__ int seq_offset(const TokenSet &s, int i)
{
    if (!s.offsets)
        return i == 0 ? 0 : s.T;
    return min(max(s.offsets[i], 0), s.T);
}

// First sequence that ends behind token t (S when there is none), by a whole
// wave: 64 offsets at a time instead of one per dependent load.
__device__ __forceinline__ int seq_behind(const TokenSet &s, int t, int lane)
{
    int lo = 0, hi = s.S;  // the answer lies in [lo, hi]
    while (hi - lo > kWave) {
        const int mid = (lo + hi) >> 1;
        if (__builtin_amdgcn_readfirstlane(seq_offset(s, mid + 1)) > t)
            hi = mid;
        else
            lo = mid + 1;
    }
    const bool behind = lo + lane < hi && seq_offset(s, lo + lane + 1) > t;
    const unsigned long long m = __ballot(behind);
    return m ? lo + __builtin_ctzll(m) : hi;
}

// Sum and maximum over a wave, the same value on every lane: row shifts and
// broadcasts within the vector unit (a shuffle through LDS takes about ten
// times as long, and these reductions are the kernels' dependent chain).
template <int kCtrl, int kRows>
__device__ __forceinline__ float dpp_move(float identity, float v)
{
    return __int_as_float(__builtin_amdgcn_update_dpp(__float_as_int(identity), __float_as_int(v), kCtrl, kRows,
                                                     0xf, false));
}

__device__ __forceinline__ float last_lane(float v)
{
    return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), 63));
}

__device__ __forceinline__ float wave_sum(float v)
{
    v += dpp_move<0x111, 0xf>(0.0f, v);  // from 1, 2, 4, 8 lanes below in the row of 16
    v += dpp_move<0x112, 0xf>(0.0f, v);
    v += dpp_move<0x114, 0xf>(0.0f, v);
    v += dpp_move<0x118, 0xf>(0.0f, v);
    v += dpp_move<0x142, 0xa>(0.0f, v);  // row ends into the next row
    v += dpp_move<0x143, 0xc>(0.0f, v);  // lane 31 into the upper half
    return last_lane(v);
}

__device__ __forceinline__ float wave_max(float v)
{
    const float low = -INFINITY;
    v = fmaxf(v, dpp_move<0x111, 0xf>(low, v));
    v = fmaxf(v, dpp_move<0x112, 0xf>(low, v));
    v = fmaxf(v, dpp_move<0x114, 0xf>(low, v));
    v = fmaxf(v, dpp_move<0x118, 0xf>(low, v));
    v = fmaxf(v, dpp_move<0x142, 0xa>(low, v));
    v = fmaxf(v, dpp_move<0x143, 0xc>(low, v));
    return last_lane(v);
}

__device__ __forceinline__ int wave_sum(int v)
{
#pragma unroll
    for (int off = 32; off >= 1; off >>= 1)
        v += __shfl_xor(v, off);
    return v;
}

// exp(x) for x <= 0 to about an fp32 ulp: 2^t with t = x log2 e rounded, times
// the factor of what the rounding left (the hardware 2^t itself is within an
// ulp).  Below -150, where the result is 0, x is cut off so that -inf stays
// out of the remainder; NaN stays NaN.
__device__ __forceinline__ float exp_neg(float x)
{
    x = x < -150.0f ? -150.0f : x;
    constexpr float kHi = 1.44269502162933349609375f, kLo = 1.925963033500011e-8f;  // log2 e
    const float t = x * kHi;
    const float rest = fmaf(x, kLo, fmaf(x, kHi, -t));
    const float e = __builtin_amdgcn_exp2f(t);
    return fmaf(e, rest * 0.693147180559945f, e);
}

// Row of E logits -> exp(x - max) in x and the reciprocal of their sum.  A row
// of -inf only has no distribution: all its probabilities are 0.
template <int NV>
__device__ __forceinline__ float softmax_row(float (&x)[NV])
{
    float m = x[0];
#pragma unroll
    for (int i = 1; i < NV; ++i)
        m = fmaxf(m, x[i]);
    m = wave_max(m);
    m = m == -INFINITY ? 0.0f : m;
    float sum = 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        x[i] = exp_neg(x[i] - m);
        sum += x[i];
    }
    sum = wave_sum(sum);
    return sum == 0.0f ? 0.0f : 1.0f / sum;
}

template <int NV>
__device__ __forceinline__ void load_row(float (&x)[NV], const float *row, int E, int lane)
{
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int e = lane + kWave * i;
        x[i] = e < E ? row[e] : -INFINITY;
    }
}

// One block's share of one sequence, tokens [a, b): probability sums in
// red[0], counts in hist, tokens that take part returned to every thread.
template <int NV>
__device__ __forceinline__ int balance_segment(const BalanceArgs &g, int a, int b,
                                               float (*red)[NV * kWave], int *hist, int *taken)
{
    constexpr int kTokens = NV >= 16 ? 1 : NV == 8 ? 2 : 4;  // rows of a wave in flight
    const int tid = threadIdx.x, lane = tid & (kWave - 1), wave = wave_id();
    // the ids travel while the rows are worked on (T k <= 2^24)
    const int i0 = a * g.k + tid, i1 = b * g.k;
    const int id0 = i0 < i1 ? g.ids[i0] : -1;
    for (int e = tid; e < g.E; e += kBalanceThreads)
        hist[e] = 0;

    float sum[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i)
        sum[i] = 0.0f;
    int n = 0;
    for (int t0 = a + wave; t0 < b; t0 += kBalanceWaves * kTokens) {
        float x[kTokens][NV];
        bool in[kTokens];
#pragma unroll
        for (int q = 0; q < kTokens; ++q) {
            const int t = min(t0 + q * kBalanceWaves, b - 1);
            load_row(x[q], g.logits + (size_t)t * g.E, g.E, lane);
            in[q] = t0 + q * kBalanceWaves < b && (!g.tok.mask || g.tok.mask[t]);
        }
#pragma unroll
        for (int q = 0; q < kTokens; ++q) {
            const float r = softmax_row(x[q]);
#pragma unroll
            for (int i = 0; i < NV; ++i)
                sum[i] += in[q] ? x[q][i] * r : 0.0f;  // a select: a masked row may hold NaN
            n += in[q];
        }
    }
#pragma unroll
    for (int i = 0; i < NV; ++i)
        red[wave][lane + kWave * i] = sum[i];
    if (lane == 0)
        taken[wave] = n;
    __syncthreads();
    for (int i = i0; i < i1; i += kBalanceThreads) {
        const int e = i == i0 ? id0 : g.ids[i];
        if (e >= 0 && e < g.E && (!g.tok.mask || g.tok.mask[i / g.k]))
            atomicAdd(&hist[e], 1);
    }
    for (int e = tid; e < g.E; e += kBalanceThreads) {
        float v = red[0][e];
#pragma unroll
        for (int w = 1; w < kBalanceWaves; ++w)
            v += red[w][e];
        red[0][e] = v;
    }
    int total = 0;
#pragma unroll
    for (int w = 0; w < kBalanceWaves; ++w)
        total += taken[w];
    __syncthreads();
    return total;
}

// Chunks of tokens, one block each; a chunk that several sequences share is
// done sequence by sequence.  Walking a batch, each step goes on to the next
// chunk or the next sequence, so row c + s is written by one block only.
template <int NV>
__global__ __launch_bounds__(kBalanceThreads) void balance_chunk_kernel(BalanceArgs g)
{
    __shared__ float red[kBalanceWaves][NV * kWave];
    __shared__ int hist[NV * kWave];
    __shared__ int taken[kBalanceWaves];
    const int c = blockIdx.x, tid = threadIdx.x;
    if (c == 0 && tid == 0)
        *g.ticket = 0;
    const int end = min((c + 1) * g.chunk, g.tok.T);
    int pos = max(c * g.chunk, seq_offset(g.tok, 0));
    while (pos < end) {
        const int s = seq_behind(g.tok, pos, tid & (kWave - 1));
        if (s >= g.tok.S)
            break;
        const int a = max(pos, seq_offset(g.tok, s)), b = min(end, seq_offset(g.tok, s + 1));
        if (a >= b)
            break;
        const int n = balance_segment<NV>(g, a, b, red, hist, taken);
        const size_t row = (size_t)c + s;
        for (int e = tid; e < g.E; e += kBalanceThreads) {
            g.part_p[row * g.E + e] = red[0][e];
            g.part_n[row * g.E + e] = hist[e];
        }
        if (tid == 0)
            g.part_t[row] = n;
        __syncthreads();
        pos = b;
    }
}

// Sums the chunks of one sequence for 64 experts; the block that finishes
// last adds up the loss.
constexpr int kReduceRows = 8;

__global__ __launch_bounds__(kReduceRows * 64) void balance_reduce_kernel(BalanceArgs g)
{
    __shared__ float red_p[kReduceRows][64];
    __shared__ int red_n[kReduceRows][64];
    __shared__ int red_t[kReduceRows * 64];
    __shared__ bool last;
    const int tid = threadIdx.x, lane = tid & 63, r = tid >> 6;
    const int s = blockIdx.y, e = blockIdx.x * 64 + lane;
    const int a = seq_offset(g.tok, s), b = seq_offset(g.tok, s + 1);
    const int c0 = a / g.chunk, c1 = b > a ? (b - 1) / g.chunk + 1 : c0;
    float p = 0.0f;
    int n = 0, t = 0;
    if (e < g.E) {
#pragma unroll 4
        for (int c = c0 + r; c < c1; c += kReduceRows) {
            p += g.part_p[((size_t)c + s) * g.E + e];
            n += g.part_n[((size_t)c + s) * g.E + e];
        }
    }
    for (int c = c0 + tid; c < c1; c += kReduceRows * 64)
        t += g.part_t[(size_t)c + s];
    red_p[r][lane] = p;
    red_n[r][lane] = n;
    red_t[tid] = t;
    __syncthreads();
    if (r == 0) {
        int N = 0;
#pragma unroll
        for (int i = 0; i < kReduceRows; ++i) {
            N += red_t[i * 64 + lane];
            if (i) {
                p += red_p[i][lane];
                n += red_n[i][lane];
            }
        }
        N = wave_sum(N);
        const float inv = N > 0 ? 1.0f / (float)N : 0.0f;
        const float mean = p * inv;
        if (e < g.E) {
            g.counts[(size_t)s * g.E + e] = n;
            g.probs[(size_t)s * g.E + e] = mean;
        }
        const float l = wave_sum(e < g.E ? (float)n * inv * mean : 0.0f);
        if (lane == 0) {
            // other blocks, maybe on other XCDs, read these two in this launch
            __hip_atomic_store(g.part_loss + (size_t)s * gridDim.x + blockIdx.x, l, __ATOMIC_RELAXED,
                               __HIP_MEMORY_SCOPE_AGENT);
            if (blockIdx.x == 0)
                __hip_atomic_store(g.tokens + s, N, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
            last = __hip_atomic_fetch_add(g.ticket, 1u, __ATOMIC_ACQ_REL, __HIP_MEMORY_SCOPE_AGENT) ==
                   gridDim.x * gridDim.y - 1;
        }
    }
    __syncthreads();
    if (!last)
        return;
    // every thread's share in ascending order, then a fixed tree
    float sum = 0.0f;
    int live = 0;
    const size_t parts = (size_t)gridDim.x * gridDim.y;
    for (size_t i = tid; i < parts; i += kReduceRows * 64)
        sum += __hip_atomic_load(g.part_loss + i, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    for (int i = tid; i < g.tok.S; i += kReduceRows * 64)
        live += __hip_atomic_load(g.tokens + i, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) > 0;
    sum = wave_sum(sum);
    live = wave_sum(live);
    __syncthreads();
    if (lane == 0) {
        red_p[r][0] = sum;
        red_n[r][0] = live;
    }
    __syncthreads();
    if (tid == 0) {
        float v = 0.0f;
        int m = 0;
        for (int i = 0; i < kReduceRows; ++i) {
            v += red_p[i][0];
            m += red_n[i][0];
        }
        *g.loss = m > 0 ? v * (float)g.E / (float)g.k / (float)m : 0.0f;
    }
}

// The whole batch in one block: small batches, where a second launch would
// cost more than the work.
template <int NV>
__global__ __launch_bounds__(kBalanceThreads) void balance_small_kernel(BalanceArgs g)
{
    __shared__ float red[kBalanceWaves][NV * kWave];
    __shared__ int hist[NV * kWave];
    __shared__ int taken[kBalanceWaves];
    __shared__ float part[kBalanceWaves];
    const int tid = threadIdx.x, lane = tid & (kWave - 1), wave = wave_id();
    float loss = 0.0f;
    int live = 0;
    for (int s = 0; s < g.tok.S; ++s) {
        const int a = seq_offset(g.tok, s), b = max(a, seq_offset(g.tok, s + 1));
        const int N = balance_segment<NV>(g, a, b, red, hist, taken);
        const float inv = N > 0 ? 1.0f / (float)N : 0.0f;
        float l = 0.0f;
        for (int e = tid; e < g.E; e += kBalanceThreads) {
            const int n = hist[e];
            const float mean = red[0][e] * inv;
            g.counts[(size_t)s * g.E + e] = n;
            g.probs[(size_t)s * g.E + e] = mean;
            l += (float)n * inv * mean;
        }
        l = wave_sum(l);
        if (lane == 0)
            part[wave] = l;
        __syncthreads();
        if (tid == 0) {
            g.tokens[s] = N;
            for (int w = 0; w < kBalanceWaves; ++w)
                loss += part[w];
        }
        live += N > 0;
        __syncthreads();
    }
    if (tid == 0)
        *g.loss = live > 0 ? loss * (float)g.E / (float)g.k / (float)live : 0.0f;
}

// ------------------------------------------------------------ the gradient

constexpr int kBackWaves = 4;
constexpr int kRowFloats = 1024;  // LDS floats per wave for the scattered routing part

// Tokens of a batch: their slots fit the wave's lanes (kp = k rounded up to a
// power of two), their rows its LDS and registers.
constexpr int max_batch(int NV) { return NV >= 16 ? 1 : NV == 8 ? 2 : 4; }

// A wave takes a run of consecutive tokens in batches of `batch`: the logits of
// the whole batch are loaded first; then lanes side by side (kp a token)
// compute the routing part and scatter it into rows in LDS; then each row is
// finished and written.
template <int NV, bool kSoftmax>
__global__ __launch_bounds__(kBackWaves * kWave) void route_backward_kernel(RouteBackwardArgs g, int kp,
                                                                            int batch, int run)
{
    constexpr int kBatch = max_batch(NV);
    __shared__ float rows[kBackWaves][kRowFloats];
    __shared__ int live_part[kBackWaves];
    const int tid = threadIdx.x, lane = tid & (kWave - 1), wave = wave_id();
    float *row = rows[wave];
    const bool balance = g.counts != nullptr;

    const long long first = ((long long)blockIdx.x * kBackWaves + wave) * run;
    const int t_begin = (int)min((long long)g.tok.T, first), t_end = (int)min((long long)g.tok.T, first + run);
    float x[kBatch][NV];
    auto load_batch = [&](int t0) {
        if (kSoftmax) {
#pragma unroll
            for (int q = 0; q < kBatch; ++q)
                if (q < batch)
                    load_row(x[q], g.logits + (size_t)min(t0 + q, g.tok.T - 1) * g.E, g.E, lane);
        }
    };
    load_batch(min(t_begin, g.tok.T - 1));

    float coef = 0.0f;
    if (balance) {  // dL E / (k S'), S' = sequences with tokens
        int live = 0;
        for (int i = tid; i < g.tok.S; i += kBackWaves * kWave)
            live += g.tokens[i] > 0;
        live = wave_sum(live);
        if (lane == 0)
            live_part[wave] = live;
        __syncthreads();
        live = 0;
        for (int w = 0; w < kBackWaves; ++w)
            live += live_part[w];
        coef = live > 0 ? *g.d_loss * (float)g.E / ((float)g.k * (float)live) : 0.0f;
    }
    if (t_begin >= t_end)
        return;
    if (g.d_weights) {
        for (int i = lane; i < batch * g.E; i += kWave)
            row[i] = 0.0f;
    }

    int seq = -1, seq_begin = 0, seq_end = 0;  // the sequence whose g is in registers
    float gr[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i)
        gr[i] = 0.0f;

    const int q_of = lane / kp, j_of = lane % kp;
    for (int t0 = t_begin; t0 < t_end; t0 += batch) {
        const int nb = min(batch, t_end - t0);
        if (t0 > t_begin)
            load_batch(t0);
        float inside = 0.0f;  // sum_i w_i dw_i of the lane's token
        int at = -1;
        if (g.d_weights) {
            const bool slot = q_of < nb && j_of < g.k;
            const size_t i = (size_t)(t0 + (slot ? q_of : 0)) * g.k + (slot ? j_of : 0);
            const int id = g.ids[i];
            const float w = g.weights[i], dw = g.d_weights[i];
            const bool ok = slot && id >= 0 && id < g.E;
            inside = ok ? w * dw : 0.0f;
            for (int off = kp >> 1; off >= 1; off >>= 1)
                inside += __shfl_xor(inside, off);
            float v = ok ? (g.method == 0 ? w * (dw - inside) : w * dw) : 0.0f;
            at = ok ? q_of * g.E + id : -1;
            // an id given twice for one token: its first slot carries the sum
            if (at >= 0)
                row[at] = __int_as_float(lane);
            __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
            const bool alone = at < 0 || __float_as_int(row[at]) == lane;
            if (__ballot(!alone)) {
                float total = 0.0f;
                bool is_first = true;
                for (int o = 0; o < kp; ++o) {
                    const int other = __shfl(at, q_of * kp + o);
                    const float vo = __shfl(v, q_of * kp + o);
                    if (other == at) {
                        total += vo;
                        is_first = is_first && o >= j_of;
                    }
                }
                v = total;
                if (at >= 0 && is_first)
                    row[at] = v;
            } else if (at >= 0) {
                row[at] = v;
            }
            __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        }
#pragma unroll
        for (int q = 0; q < kBatch; ++q) {
            if (q >= nb)
                break;
            const int t = t0 + q;
            if (t >= seq_end || t < seq_begin) {
                seq = seq_behind(g.tok, t, lane);
                const bool real = seq < g.tok.S;
                seq_begin = real ? seq_offset(g.tok, seq) : t;
                seq_end = real ? seq_offset(g.tok, seq + 1) : g.tok.T;
                if (seq_begin > t) {  // between sequences
                    seq_end = seq_begin;
                    seq_begin = t;
                    seq = g.tok.S;
                }
                if (balance) {
                    const bool has = seq < g.tok.S;
                    const float N = has ? (float)g.tokens[seq] : 0.0f;
                    const float f = N > 0.0f ? coef / (N * N) : 0.0f;
#pragma unroll
                    for (int i = 0; i < NV; ++i) {
                        const int e = lane + kWave * i;
                        gr[i] = has && e < g.E ? f * (float)g.counts[(size_t)seq * g.E + e] : 0.0f;
                    }
                }
            }
            const bool in = seq < g.tok.S && (!g.tok.mask || g.tok.mask[t]);
            float d[NV];
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int e = lane + kWave * i;
                d[i] = g.d_weights && e < g.E ? row[q * g.E + e] : 0.0f;
            }
            if (kSoftmax) {
                const float r = softmax_row(x[q]);
                float dot = 0.0f;
#pragma unroll
                for (int i = 0; i < NV; ++i)
                    dot += x[q][i] * gr[i];
                dot = wave_sum(dot) * r;
                const float all = dot + (g.method == 1 ? __shfl(inside, q * kp) : 0.0f);
#pragma unroll
                for (int i = 0; i < NV; ++i)
                    d[i] += x[q][i] * r * (gr[i] - all);
            }
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int e = lane + kWave * i;
                if (e < g.E)
                    g.d_logits[(size_t)t * g.E + e] = in ? d[i] : 0.0f;
            }
        }
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        if (at >= 0)
            row[at] = 0.0f;
    }
}

template <typename F>
void with_nv(int E, F f)
{
    if (E <= 64)
        f(std::integral_constant<int, 1>{});
    else if (E <= 128)
        f(std::integral_constant<int, 2>{});
    else if (E <= 256)
        f(std::integral_constant<int, 4>{});
    else if (E <= 512)
        f(std::integral_constant<int, 8>{});
    else
        f(std::integral_constant<int, 16>{});
}

// Batches that one block does: where its walk through the sequences, one after
// another, is shorter than a second launch.  One block / two launches in us, by
// sequences:       1           2           4           8          16
//   32 tokens, 128 experts
//              3.9 / 8.5   6.0 / 10.7  10.5 / 15.4  16.9 / 21.8  32.3 / 37.0
//   64 tokens, 128 experts
//              5.1 / 8.5   6.2 / 8.2   10.6 / 10.8  19.8 / 15.5  32.3 / 21.9
//   64 tokens, 256 experts
//              6.1 / 9.1   7.3 / 9.2   12.8 / 12.1  24.3 / 17.9  38.1 / 24.8
//   128 tokens, 128 experts
//              8.0 / 8.3   8.7 / 8.6   10.8 / 8.6   19.9 / 11.1  38.0 / 15.7
//   128 tokens, 256 experts
//             10.1 / 8.9  10.6 / 9.2   13.1 / 9.3   24.3 / 12.1  47.1 / 18.2
// 32 tokens are one chunk of the two launches, which walk them as well.
bool balance_is_small(int T, int E, int S)
{
    return T <= 32 ? S <= 16 : T <= 128 && T * E <= 16384 && T * S <= 256;
}

} // namespace

int balance_chunk(int T)
{
    // 512 chunks (two blocks per CU) when there are enough tokens, at least
    // four tokens per wave
    const int c = (T + 511) / 512;
    return std::max(32, (c + 31) / 32 * 32);
}

namespace {

struct BalanceLayout {
    size_t p, n, t, loss, ticket, total;
};

BalanceLayout balance_regions(int T, int E, int S)
{
    const size_t rows = (size_t)(T + balance_chunk(T) - 1) / balance_chunk(T) + S;
    auto up = [](size_t v) { return (v + 255) / 256 * 256; };
    BalanceLayout l;
    l.p = 0;
    l.n = up(rows * E * 4);
    l.t = l.n + up(rows * E * 4);
    l.loss = l.t + up(rows * 4);
    l.ticket = l.loss + up((size_t)S * ((E + 63) / 64) * 4);
    l.total = l.ticket + 256;
    return l;
}

} // namespace

size_t balance_workspace(int T, int E, int S)
{
    return balance_is_small(T, E, S) ? 0 : balance_regions(T, E, S).total;
}

void balance_layout(BalanceArgs *a, void *workspace)
{
    a->chunk = balance_chunk(a->tok.T);
    a->n_chunks = (a->tok.T + a->chunk - 1) / a->chunk;
    const BalanceLayout l = balance_regions(a->tok.T, a->E, a->tok.S);
    char *ws = static_cast<char *>(workspace);
    a->part_p = reinterpret_cast<float *>(ws + l.p);
    a->part_n = reinterpret_cast<int32_t *>(ws + l.n);
    a->part_t = reinterpret_cast<int32_t *>(ws + l.t);
    a->part_loss = reinterpret_cast<float *>(ws + l.loss);
    a->ticket = reinterpret_cast<uint32_t *>(ws + l.ticket);
}

hipError_t launch_balance(const BalanceArgs &a, hipStream_t s)
{
    if (balance_is_small(a.tok.T, a.E, a.tok.S)) {
        with_nv(a.E, [&](auto nv) {
            hipLaunchKernelGGL((balance_small_kernel<decltype(nv)::value>), dim3(1),
                               dim3(kBalanceThreads), 0, s, a);
        });
        return hipGetLastError();
    }
    with_nv(a.E, [&](auto nv) {
        hipLaunchKernelGGL((balance_chunk_kernel<decltype(nv)::value>), dim3(std::max(1, a.n_chunks)),
                           dim3(kBalanceThreads), 0, s, a);
    });
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess)
        return e;
    hipLaunchKernelGGL(balance_reduce_kernel, dim3((a.E + 63) / 64, a.tok.S), dim3(kReduceRows * 64),
                       0, s, a);
    return hipGetLastError();
}

hipError_t launch_route_backward(const RouteBackwardArgs &a, hipStream_t s)
{
    if (a.tok.T <= 0)
        return hipSuccess;
    int kp = 1;
    while (kp < a.k)
        kp *= 2;
    const int nv = a.E <= 64 ? 1 : a.E <= 128 ? 2 : a.E <= 256 ? 4 : a.E <= 512 ? 8 : 16;
    // about 8 waves per SIMD when there are tokens for it
    const int per = (a.tok.T + 8191) / 8192;
    const int batch = std::max(1, std::min(std::min(kWave / kp, kRowFloats / a.E), std::min(max_batch(nv), per)));
    const int run = (per + batch - 1) / batch * batch;
    const int waves = (a.tok.T + run - 1) / run;
    const dim3 grid((waves + kBackWaves - 1) / kBackWaves), block(kBackWaves * kWave);
    const bool softmax = a.counts != nullptr || (a.method == 1 && a.d_weights);
    with_nv(a.E, [&](auto nv) {
        if (softmax)
            hipLaunchKernelGGL((route_backward_kernel<decltype(nv)::value, true>), grid, block, 0, s, a,
                               kp, batch, run);
        else
            hipLaunchKernelGGL((route_backward_kernel<decltype(nv)::value, false>), grid, block, 0, s, a,
                               kp, batch, run);
    });
    return hipGetLastError();
}

} // namespace moe_lora
