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

// First sequence that ends behind token t (S when there is none).
__device__ __forceinline__ int seq_behind(const TokenSet &s, int t)
{
    int lo = 0, hi = s.S;
    while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (seq_offset(s, mid + 1) > t)
            hi = mid;
        else
            lo = mid + 1;
    }
    return lo;
}

__device__ __forceinline__ float wave_max(float v)
{
#pragma unroll
    for (int off = 32; off >= 1; off >>= 1)
        v = fmaxf(v, __shfl_xor(v, off));
    return v;
}

__device__ __forceinline__ float wave_sum(float v)
{
#pragma unroll
    for (int off = 32; off >= 1; off >>= 1)
        v += __shfl_xor(v, off);
    return v;
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
        x[i] = expf(x[i] - m);
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
    constexpr int kTokens = NV >= 8 ? 1 : 2;  // rows of a wave in flight
    const int tid = threadIdx.x, lane = tid & (kWave - 1), wave = wave_id();
    for (int e = tid; e < g.E; e += kBalanceThreads)
        hist[e] = 0;
    __syncthreads();

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
    for (size_t i = (size_t)a * g.k + tid; i < (size_t)b * g.k; i += kBalanceThreads) {
        const int e = g.ids[i];
        if (e >= 0 && e < g.E && (!g.tok.mask || g.tok.mask[i / g.k]))
            atomicAdd(&hist[e], 1);
    }
#pragma unroll
    for (int i = 0; i < NV; ++i)
        red[wave][lane + kWave * i] = sum[i];
    if (lane == 0)
        taken[wave] = n;
    __syncthreads();
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
        const int s = seq_behind(g.tok, pos);
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
constexpr int kReduceRows = 16;

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
#pragma unroll
        for (int off = 32; off >= 1; off >>= 1)
            N += __shfl_xor(N, off);
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
            __threadfence();
            last = atomicAdd(g.ticket, 1u) == gridDim.x * gridDim.y - 1;
        }
    }
    __syncthreads();
    if (!last)
        return;
    __threadfence();
    // every thread's share in ascending order, then a fixed tree
    float sum = 0.0f;
    int live = 0;
    const size_t parts = (size_t)gridDim.x * gridDim.y;
    for (size_t i = tid; i < parts; i += kReduceRows * 64)
        sum += __hip_atomic_load(g.part_loss + i, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    for (int i = tid; i < g.tok.S; i += kReduceRows * 64)
        live += __hip_atomic_load(g.tokens + i, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) > 0;
    sum = wave_sum(sum);
#pragma unroll
    for (int off = 32; off >= 1; off >>= 1)
        live += __shfl_xor(live, off);
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
constexpr int kRowFloats = 2048;  // LDS floats per wave for the scattered routing part

// A wave takes a run of consecutive tokens, in batches of `batch` tokens whose
// k slots its lanes hold side by side (kp lanes a token): one pass computes
// their routing part and scatters it into rows in LDS; then each row is
// finished and written.
template <int NV, bool kSoftmax>
__global__ __launch_bounds__(kBackWaves * kWave) void route_backward_kernel(RouteBackwardArgs g, int kp,
                                                                            int batch, int run)
{
    __shared__ float rows[kBackWaves][kRowFloats];
    __shared__ int live_part[kBackWaves];
    const int tid = threadIdx.x, lane = tid & (kWave - 1), wave = wave_id();
    float *row = rows[wave];
    const bool balance = g.counts != nullptr;

    float coef = 0.0f;
    if (balance) {  // dL E / (k S'), S' = sequences with tokens
        int live = 0;
        for (int i = tid; i < g.tok.S; i += kBackWaves * kWave)
            live += g.tokens[i] > 0;
#pragma unroll
        for (int off = 32; off >= 1; off >>= 1)
            live += __shfl_xor(live, off);
        if (lane == 0)
            live_part[wave] = live;
        __syncthreads();
        live = 0;
        for (int w = 0; w < kBackWaves; ++w)
            live += live_part[w];
        coef = live > 0 ? *g.d_loss * (float)g.E / ((float)g.k * (float)live) : 0.0f;
    }

    const long long first = ((long long)blockIdx.x * kBackWaves + wave) * run;
    if (first >= g.tok.T)
        return;
    const int t_begin = (int)first, t_end = (int)min((long long)g.tok.T, first + run);
    for (int i = lane; i < batch * g.E; i += kWave)
        row[i] = 0.0f;

    int seq = -1, seq_begin = 0, seq_end = 0;  // the sequence whose g is in registers
    float gr[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i)
        gr[i] = 0.0f;

    const int q_of = lane / kp, j_of = lane % kp;
    for (int t0 = t_begin; t0 < t_end; t0 += batch) {
        const int nb = min(batch, t_end - t0);
        float inside = 0.0f;  // sum_i w_i dw_i of the lane's token
        int at = -1;
        if (g.d_weights) {
            const bool slot = q_of < nb && j_of < g.k;
            const size_t x = (size_t)(t0 + (slot ? q_of : 0)) * g.k + (slot ? j_of : 0);
            const int id = g.ids[x];
            const float w = g.weights[x], dw = g.d_weights[x];
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
                for (int i = 0; i < kp; ++i) {
                    const int other = __shfl(at, q_of * kp + i);
                    const float vi = __shfl(v, q_of * kp + i);
                    if (other == at) {
                        total += vi;
                        is_first = is_first && i >= j_of;
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
        for (int q = 0; q < nb; ++q) {
            const int t = t0 + q;
            if (t >= seq_end || t < seq_begin) {
                seq = seq_behind(g.tok, t);
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
                float x[NV];
                load_row(x, g.logits + (size_t)t * g.E, g.E, lane);
                const float r = softmax_row(x);
                float dot = 0.0f;
#pragma unroll
                for (int i = 0; i < NV; ++i)
                    dot += x[i] * gr[i];
                dot = wave_sum(dot) * r;
                const float all = dot + (g.method == 1 ? __shfl(inside, q * kp) : 0.0f);
#pragma unroll
                for (int i = 0; i < NV; ++i)
                    d[i] += x[i] * r * (gr[i] - all);
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

// Batches that one block does: up to 128 tokens and 16 sequences.
bool balance_is_small(int T, int S) { return T <= 128 && S <= 16; }

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
    return balance_is_small(T, S) ? 0 : balance_regions(T, E, S).total;
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
    if (balance_is_small(a.tok.T, a.tok.S)) {
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
    // tokens whose slots fit the wave's lanes and whose rows fit its LDS
    int batch = std::max(1, std::min(kWave / kp, kRowFloats / a.E));
    // about 8 waves per SIMD when there are tokens for it
    const int per = (a.tok.T + 8191) / 8192;
    batch = std::min(batch, per);
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
