// The router's balance loss and z-loss with their gradient with respect to the logits.
//
// p_t = softmax(l_t) over the E experts. For each sequence s (a run of tokens; a token mask leaves padding
// out), n_s = its valid tokens, counts[s, e] = its slots routed to e, P[s, e] = mean of p_t[e]:
//   loss0 = alpha / S' * sum_s sum_e f[s, e] P[s, e],  f = E counts / (k n_s),  S' = sequences with n_s > 0
//   loss1 = beta / N * sum_t lse_t^2,                  lse_t = log sum_e exp(l_t[e]),  N = sum_s n_s
// (the auxiliary loss over expert load fractions of the DeepSeek-V4 lecture page, 2.3, and the DeepSeek MoE
// page, ch. 1, in its product form: counts are constants, the gradient flows through P). With upstream
// gradients g0, g1 and c[s, e] = g0 alpha f / (S' n_s):
//   dl_t[e] = p_t[e] (c[s, e] - sum_j p_t[j] c[s, j]) + 2 g1 beta / N lse_t p_t[e].
//
// Both passes read each logit once, and that read bounds them when T E is large; at a step's usual size the
// 8 MB of logits sit in L2 and launches are the time, so the forward is two launches (one for few tokens) and the
// backward one, each set up while the one before it runs. A group of 4 to 32 lanes takes a token, 16 experts a lane: the row stays
// in registers between its maximum, its sum and its use, and the shuffles of a row are shared by the tokens of a
// warp (131072 x 256: 40.6 us with 32 lanes a token, 33.6 with 16). 32 warps an SM keep enough reads in flight; a
// value costs about five instructions (maximum, exp2 of one fused multiply-add, sum, accumulation), below the
// memory's pace. The forward cuts the tokens into at most 296 chunks (two blocks an SM); chunk c of sequence s
// leaves one row of partial sums at index c + s, which is unique because the cuts between chunks and sequences,
// taken in order, each move c or s up by one. No float is added atomically, so results repeat bit for bit.
// Measured on a B200, replayed: 128 x 256 forward and backward 9.9 us, 8192 x 256 14.6 us (launches); 65536 x 512
// 84 us, of it 33 the forward's read (134 MB: 4.1 TB/s), 12 its join, 42 the gradient (134 MB read and as many written).
// The gradient reads the logits again because it is a call of its own: its factors come from topk_idx, the mask, the
// offsets and dloss, not from the loss. The one-launch form spills 56 bytes a thread where E is no multiple of 4.
#include <math.h>

#include <algorithm>

#include "../../include/moe_fp8.h"
#include "common.cuh"

namespace moe {

moe_status_t current_device(int* num_sms, int** status);

namespace {

constexpr int kFwdThreads = 512, kBwdThreads = 256;
constexpr int kMostTokens = 1 << 30;     // a chunk past the last token still fits an int
constexpr int kMaxChunks = 296;          // two forward blocks on each of 148 SMs
constexpr int kBwdTokens = 16;           // tokens a backward block takes at least
constexpr float kLog2e = 1.4426950408889634f;

// Tokens of a forward chunk: a multiple of 16, at most kMaxChunks chunks.
int chunk_tokens(int T) { return std::max(16, ((T + kMaxChunks - 1) / kMaxChunks + 15) / 16 * 16); }
int chunks_of(int T) { return (T + chunk_tokens(T) - 1) / chunk_tokens(T); }

// The reduction's blocks: with few sequences, each of up to 296 cuts, 8 columns x 32 rows; with many, whose cuts
// are few, 32 columns.
constexpr int kRedThreads = 256, kRedDepth = 10;
int red_cols(int S) { return S <= 16 ? 8 : 32; }

// The forward's scratch: one row per (chunk, sequence) cut, and each reducing block's share of the loss.
struct BalWs {
    float* psum;        // [cuts, E] sums of p
    int32_t* hist;      // [cuts, E] slots
    double* zsum;       // [cuts] sums of lse^2: a row far from zero has one outside fp32
    int32_t* nval;      // [cuts] valid tokens
    double* part;       // [S, column blocks] sum_e counts * psum over the block's columns
    double* zpart;      // [S]
    unsigned* ticket;   // blocks of the reduction that are done
    size_t total;
};

// Sized so that a larger T, E or S never takes less: chunks as if none were longer than 16 tokens until there are
// kMaxChunks, column blocks of 8.
BalWs carve_balance(int T, int E, int S, void* base) {
    BalWs w;
    const size_t cuts = static_cast<size_t>(std::min(kMaxChunks, (T + 15) / 16)) + S, nx = (E + 7) / 8;
    uint8_t* p = static_cast<uint8_t*>(base);
    size_t off = 0;
    auto take = [&](size_t bytes) {
        uint8_t* q = p ? p + off : nullptr;
        off += (bytes + 255) / 256 * 256;
        return q;
    };
    w.psum = reinterpret_cast<float*>(take(4 * cuts * E));
    w.hist = reinterpret_cast<int32_t*>(take(4 * cuts * E));
    w.zsum = reinterpret_cast<double*>(take(8 * cuts));
    w.nval = reinterpret_cast<int32_t*>(take(4 * cuts));
    w.part = reinterpret_cast<double*>(take(8 * static_cast<size_t>(S) * nx));
    w.zpart = reinterpret_cast<double*>(take(8 * static_cast<size_t>(S)));
    w.ticket = reinterpret_cast<unsigned*>(take(4));
    w.total = off;
    return w;
}

// First token of sequence s (offsets[S]: one past the last), forced into [0, T]; no offsets: one sequence of all.
__device__ __forceinline__ int seq_start(const int32_t* offsets, int s, int T) {
    return offsets ? min(max(offsets[s], 0), T) : (s ? T : 0);
}

// The first sequence that ends behind token t (S if none does), the whole block together: the sequences that end
// before it are counted side by side (one round trip to memory, where a search would take one a step), or, of
// very many, searched for.
__device__ __forceinline__ int seq_behind(const int32_t* offsets, int S, int T, int t) {
    if (!offsets) return 0;
    if (S <= 4 * static_cast<int>(blockDim.x)) {
        int n = 0;
        for (int s0 = 0; s0 < S; s0 += blockDim.x) {
            const int s = s0 + threadIdx.x;
            n += __syncthreads_count(s < S && seq_start(offsets, s + 1, T) <= t);
        }
        return n;
    }
    int lo = 0, hi = S;
    while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (seq_start(offsets, mid + 1, T) > t) hi = mid; else lo = mid + 1;
    }
    return lo;
}

// Experts of a lane: value i of lane j of a G-lane group is expert 4 (j + G (i / 4)) + i % 4 where rows can
// be read 16 bytes at a time (E a multiple of 4), else j + G i.
template <int G, bool VEC>
__device__ __forceinline__ int expert_of(int i, int j) {
    return VEC ? 4 * (j + G * (i >> 2)) + (i & 3) : j + G * i;
}

template <int G, int V, bool VEC>
__device__ __forceinline__ void load_row(const float* __restrict__ row, int E, int j, float fill, float (&v)[V]) {
    if constexpr (VEC) {
#pragma unroll
        for (int q = 0; q < V / 4; ++q) {
            const int e = 4 * (j + G * q);
            float4 f = make_float4(fill, fill, fill, fill);
            if (e < E) f = __ldg(reinterpret_cast<const float4*>(row + e));
            v[4 * q] = f.x; v[4 * q + 1] = f.y; v[4 * q + 2] = f.z; v[4 * q + 3] = f.w;
        }
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i) v[i] = j + G * i < E ? __ldg(row + j + G * i) : fill;
    }
}

// Sum and maximum over a G-lane group (every lane gets the result).
template <int G>
__device__ __forceinline__ float group_max(float v) {
#pragma unroll
    for (int o = G / 2; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
    return v;
}
template <int G>
__device__ __forceinline__ float group_sum(float v) {
#pragma unroll
    for (int o = G / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// exp(v - m) as 2^(v log2 e - m log2 e); c = m log2 e. Rounding c scales a whole row alike, which its sum undoes.
__device__ __forceinline__ float exp_from(float v, float c) { return exp2f(fmaf(v, kLog2e, -c)); }

// Rows whose maximum or lse is farther than this from zero (all of a row at the type's lowest value, say) are shifted to
// it first: the rounding of c shows in the forward's lse, as much as lse's own, and from about 2^30 on would leave exp2's
// range.
constexpr float kFar = 64.0f;

__device__ __forceinline__ double warp_sum(double v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// ---------------------------------------------------------------- forward, pass 1: partial sums of every cut
template <int G, int V, bool VEC>
__device__ __forceinline__ void
partial_sums(const float* __restrict__ logits, const int32_t* __restrict__ idx, const uint8_t* __restrict__ mask,
             const int32_t* __restrict__ offsets, int T, int E, int k, int S, int C, const BalWs& w,
             float* __restrict__ lse) {
    constexpr int kW = kFwdThreads / 32, kRows = kW * (32 / G);     // warps; tokens the block takes at a time
    extern __shared__ float sm_red[];                               // [kW][E]
    __shared__ int sm_hist[kMaxE];
    __shared__ double sm_z[kW];
    __shared__ int sm_n[kW];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, j = lane % G;
    const int c0 = blockIdx.x * C, c1 = min(c0 + C, T);
    for (int s = seq_behind(offsets, S, T, c0); s < S; ++s) {
        const int a = max(seq_start(offsets, s, T), c0), b = min(seq_start(offsets, s + 1, T), c1);
        if (a >= c1) break;                          // this sequence, and with it every later one, starts behind
        if (a >= b) continue;
        for (int e = threadIdx.x; e < E; e += kFwdThreads) sm_hist[e] = 0;
        __syncthreads();
        float acc[V];
#pragma unroll
        for (int i = 0; i < V; ++i) acc[i] = 0.0f;
        double z = 0.0;
        int n = 0;
        for (int t0 = a; t0 < b; t0 += kRows) {
            // the row, the token's mask and its first slots in one trip to memory
            const int t = t0 + warp * (32 / G) + lane / G, tt = t < b ? t : a;
            float v[V];
            load_row<G, V, VEC>(logits + static_cast<int64_t>(tt) * E, E, j, -INFINITY, v);
            const int slot = j < k ? idx[static_cast<int64_t>(tt) * k + j] : -1;
            const bool on = (!mask || mask[tt]) && t < b;
            if (on) {
                if (slot >= 0 && slot < E) atomicAdd(&sm_hist[slot], 1);
                for (int i = j + G; i < k; i += G) {
                    const int e = idx[static_cast<int64_t>(t) * k + i];
                    if (e >= 0 && e < E) atomicAdd(&sm_hist[e], 1);
                }
            }
            float m = v[0];
#pragma unroll
            for (int i = 1; i < V; ++i) m = fmaxf(m, v[i]);   // a NaN comes back through the sum
            m = group_max<G>(m);
            float mc = m * kLog2e;
            if (fabsf(m) > kFar) {
                mc = 0.0f;
#pragma unroll
                for (int i = 0; i < V; ++i) v[i] -= m;
            }
            float sum = 0.0f;
#pragma unroll
            for (int i = 0; i < V; ++i) {
                // a lane's places behind the last expert hold -inf: 0, or NaN in a row that is NaN anyway
                v[i] = exp_from(v[i], mc);
                sum += v[i];
            }
            sum = group_sum<G>(sum);
            if (on) {
                const float r = 1.0f / sum, l = m + logf(sum);
#pragma unroll
                for (int i = 0; i < V; ++i) acc[i] = fmaf(v[i], r, acc[i]);
                z = fma(static_cast<double>(l), static_cast<double>(l), z);
                ++n;
                if (j == 0) lse[t] = l;
            } else if (t < b && j == 0) {
                lse[t] = 0.0f;
            }
        }
        // the warp's token groups, then the warps
#pragma unroll
        for (int o = G; o < 32; o <<= 1) {
#pragma unroll
            for (int i = 0; i < V; ++i) acc[i] += __shfl_xor_sync(0xffffffffu, acc[i], o);
            z += __shfl_xor_sync(0xffffffffu, z, o);
            n += __shfl_xor_sync(0xffffffffu, n, o);
        }
        if (lane < G) {
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const int e = expert_of<G, VEC>(i, j);
                if (e < E) sm_red[warp * E + e] = acc[i];
            }
        }
        if (lane == 0) { sm_z[warp] = z; sm_n[warp] = n; }
        __syncthreads();
        const int64_t cut = static_cast<int64_t>(blockIdx.x) + s;
        for (int e = threadIdx.x; e < E; e += kFwdThreads) {
            float x = 0.0f;
#pragma unroll
            for (int r = 0; r < kW; ++r) x += sm_red[r * E + e];
            w.psum[cut * E + e] = x;
            w.hist[cut * E + e] = sm_hist[e];
        }
        if (warp == 0) {
            const double x = warp_sum(lane < kW ? sm_z[lane] : 0.0);
            const int m = __reduce_add_sync(0xffffffffu, lane < kW ? sm_n[lane] : 0);
            if (lane == 0) {
                w.zsum[cut] = x;
                w.nval[cut] = m;
            }
        }
        __syncthreads();
    }
}

template <int G, int V, bool VEC>
__global__ void __launch_bounds__(kFwdThreads, 2)
balance_partial_kernel(const float* __restrict__ logits, const int32_t* __restrict__ idx,
                       const uint8_t* __restrict__ mask, const int32_t* __restrict__ offsets, int T, int E, int k,
                       int S, int C, BalWs w, float* __restrict__ lse) {
    dependents_may_launch();
    wait_for_producers();
    if (blockIdx.x == 0 && threadIdx.x == 0) *w.ticket = 0;
    partial_sums<G, V, VEC>(logits, idx, mask, offsets, T, E, k, S, C, w, lse);
}

// The blocks' shares of the losses, added in a fixed order by one block of W warps.
template <int W>
__device__ __forceinline__ void finish_losses(const BalWs& w, int S, int nx, int E, int k, float alpha, float beta,
                                              float* __restrict__ loss, int32_t* valid) {
    __shared__ double sm_0[W], sm_1[W];
    __shared__ int sm_f[W], sm_t[W];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    double l0 = 0.0, l1 = 0.0;
    int full = 0, total = 0;
    for (int64_t i = threadIdx.x; i < static_cast<int64_t>(S) * nx; i += 32 * W) l0 += __ldcg(w.part + i);
    for (int i = threadIdx.x; i < S; i += 32 * W) {
        const int v = __ldcg(valid + i);
        l1 += __ldcg(w.zpart + i);
        full += v > 0;
        total += v;
    }
    l0 = warp_sum(l0);
    l1 = warp_sum(l1);
    full = __reduce_add_sync(0xffffffffu, full);
    total = __reduce_add_sync(0xffffffffu, total);
    if (lane == 0) { sm_0[warp] = l0; sm_1[warp] = l1; sm_f[warp] = full; sm_t[warp] = total; }
    __syncthreads();
    if (threadIdx.x == 0) {
        l0 = l1 = 0.0;
        full = total = 0;
#pragma unroll
        for (int i = 0; i < W; ++i) { l0 += sm_0[i]; l1 += sm_1[i]; full += sm_f[i]; total += sm_t[i]; }
        loss[0] = static_cast<float>(alpha * l0 * E / (static_cast<double>(k) * max(full, 1)));
        loss[1] = static_cast<float>(beta * l1 / max(total, 1));
        valid[S] = full;
        valid[S + 1] = total;
    }
}

// Offsets that are not non-decreasing within [0, T] are reported.
__device__ __forceinline__ void check_offsets(const int32_t* offsets, int s, int a, int b, int* status) {
    if (offsets && (offsets[s] != a || offsets[s + 1] != b || a > b)) set_status(status, kStatusCapacity);
}

// Few tokens: the whole forward as one cluster of up to 8 blocks, a chunk each; then a warp takes 32 columns of a
// sequence over its few cuts, and the first block the losses. One launch less on the host (2 us), and 7.2 us instead of
// 7.9 on the GPU at 128 x 256; at 512 x 512 eight SMs are too few (10.4 us against 8.6).
constexpr int kSmallTokens = 256, kSmallBlocks = 8;
template <int G, int V, bool VEC>
__global__ void __launch_bounds__(kFwdThreads)
balance_small_kernel(const float* __restrict__ logits, const int32_t* __restrict__ idx,
                     const uint8_t* __restrict__ mask, const int32_t* __restrict__ offsets, int T, int E, int k, int S,
                     int C, BalWs w, float* __restrict__ lse, float alpha, float beta, float* __restrict__ loss,
                     int32_t* __restrict__ counts, float* __restrict__ mean_prob, int32_t* valid, int* status) {
    constexpr int kW = kFwdThreads / 32;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, nx = (E + 31) / 32;
    dependents_may_launch();
    wait_for_producers();
    partial_sums<G, V, VEC>(logits, idx, mask, offsets, T, E, k, S, C, w, lse);
    __syncwarp();
    cluster_sync();                                     // every block's cuts are in memory
    for (int item = blockIdx.x * kW + warp; item < S * nx; item += gridDim.x * kW) {
        const int s = item / nx, x = item - s * nx, e = x * 32 + lane;
        const int a = seq_start(offsets, s, T), b = seq_start(offsets, s + 1, T);
        if (x == 0 && lane == 0) check_offsets(offsets, s, a, b, status);
        const int lo = a / C, hi = b > a ? (b - 1) / C + 1 : lo;
        double p = 0.0;
        int h = 0;
#pragma unroll
        for (int i = 0; i < kSmallBlocks; ++i) {
            const bool in = lo + i < hi && e < E;
            const int64_t at = (static_cast<int64_t>(lo) + i + s) * E + e;
            p += in ? __ldcg(w.psum + at) : 0.0f;
            h += in ? __ldcg(w.hist + at) : 0;
        }
        const bool mine = lo + lane < hi;
        const int n = __reduce_add_sync(0xffffffffu, mine ? __ldcg(w.nval + lo + lane + s) : 0);
        const double z = warp_sum(mine ? __ldcg(w.zsum + lo + lane + s) : 0.0);
        const double inv = n > 0 ? 1.0 / n : 0.0;
        if (e < E) {
            mean_prob[static_cast<int64_t>(s) * E + e] = static_cast<float>(p * inv);
            counts[static_cast<int64_t>(s) * E + e] = h;
        }
        const double share = warp_sum(e < E ? p * h * inv * inv : 0.0);
        if (lane == 0) {
            w.part[item] = share;
            if (x == 0) { w.zpart[s] = z; valid[s] = n; }
        }
    }
    __syncwarp();
    cluster_sync();
    if (blockIdx.x == 0) finish_losses<kW>(w, S, nx, E, k, alpha, beta, loss, valid);
}

// ---------------------------------------------------------------- forward, pass 2: the cuts of each sequence
// Grid (column blocks, sequences); COLS columns a block, 256 / COLS partial rows side by side and kRedDepth of
// those in flight. The last block to finish adds the blocks' shares of the losses in a fixed order.
template <int COLS>
__global__ void __launch_bounds__(kRedThreads)
balance_reduce_kernel(const int32_t* __restrict__ offsets, int T, int E, int k, int S, int C, float alpha, float beta,
                      BalWs w, float* __restrict__ loss, int32_t* __restrict__ counts, float* __restrict__ mean_prob,
                      int32_t* valid, int* status) {
    constexpr int kRows = kRedThreads / COLS, kW = kRedThreads / 32;
    __shared__ double sm_p[kW][COLS];
    __shared__ int sm_h[kW][COLS];
    __shared__ double sm_z[kW];
    __shared__ int sm_n[kW];
    __shared__ bool sm_last;
    const int col = threadIdx.x % COLS, r0 = threadIdx.x / COLS, s = blockIdx.y;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int e = blockIdx.x * COLS + col;
    dependents_may_launch();
    wait_for_producers();
    const int a = seq_start(offsets, s, T), b = seq_start(offsets, s + 1, T);
    if (threadIdx.x == 0 && blockIdx.x == 0) check_offsets(offsets, s, a, b, status);
    const int lo = a / C, hi = b > a ? (b - 1) / C + 1 : lo;       // chunks that hold some of the sequence
    double p = 0.0, z = 0.0;       // a run's sums are fp32, their total has more bits
    int h = 0, n = 0;
    for (int c = lo + threadIdx.x; c < hi; c += kRedThreads) {
        n += w.nval[c + s];
        if (blockIdx.x == 0) z += w.zsum[c + s];
    }
    if (e < E) {
        for (int c0 = lo + r0; c0 < hi; c0 += kRows * kRedDepth) {
            float pv[kRedDepth];
            int hv[kRedDepth];
#pragma unroll
            for (int i = 0; i < kRedDepth; ++i) {
                const int64_t at = (static_cast<int64_t>(c0) + i * kRows + s) * E + e;
                const bool in = c0 + i * kRows < hi;
                pv[i] = in ? w.psum[at] : 0.0f;
                hv[i] = in ? w.hist[at] : 0;
            }
#pragma unroll
            for (int i = 0; i < kRedDepth; ++i) { p += pv[i]; h += hv[i]; }
        }
    }
#pragma unroll
    for (int o = COLS; o < 32; o <<= 1) {
        p += __shfl_xor_sync(0xffffffffu, p, o);
        h += __shfl_xor_sync(0xffffffffu, h, o);
    }
    n = __reduce_add_sync(0xffffffffu, n);
    if (blockIdx.x == 0) z = warp_sum(z);
    if (lane < COLS) { sm_p[warp][lane] = p; sm_h[warp][lane] = h; }
    if (lane == 0) { sm_n[warp] = n; sm_z[warp] = z; }
    __syncthreads();
    if (warp == 0) {
        n = 0;
        z = 0.0;
#pragma unroll
        for (int i = 0; i < kW; ++i) { n += sm_n[i]; z += sm_z[i]; }
        double share = 0.0;
        if (lane < COLS && e < E) {
            double ps = 0.0;
            int hs = 0;
#pragma unroll
            for (int i = 0; i < kW; ++i) { ps += sm_p[i][lane]; hs += sm_h[i][lane]; }
            const double inv = n > 0 ? 1.0 / n : 0.0;
            mean_prob[static_cast<int64_t>(s) * E + e] = static_cast<float>(ps * inv);
            counts[static_cast<int64_t>(s) * E + e] = hs;
            share = ps * hs * inv * inv;                     // times E / k at the end
        }
        share = warp_sum(share);
        if (lane == 0) {
            w.part[static_cast<int64_t>(s) * gridDim.x + blockIdx.x] = share;
            if (blockIdx.x == 0) { w.zpart[s] = z; valid[s] = n; }
            __threadfence();
            sm_last = atomicAdd(w.ticket, 1u) == gridDim.x * gridDim.y - 1;
        }
    }
    __syncthreads();
    if (!sm_last) return;
    __threadfence();
    finish_losses<kW>(w, S, gridDim.x, E, k, alpha, beta, loss, valid);
}

// ---------------------------------------------------------------- backward
template <int G, int V, bool VEC>
__global__ void __launch_bounds__(kBwdThreads, 4)
balance_backward_kernel(const float* __restrict__ logits, const float* __restrict__ lse,
                        const int32_t* __restrict__ counts, const int32_t* __restrict__ valid,
                        const uint8_t* __restrict__ mask, const int32_t* __restrict__ offsets, int T, int E, int k,
                        int S, int C, float alpha, float beta, const float* __restrict__ dloss,
                        float* __restrict__ dlogits) {
    constexpr int kRows = kBwdThreads / 32 * (32 / G);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, j = lane % G;
    const int c0 = blockIdx.x * C, c1 = min(c0 + C, T);
    dependents_may_launch();
    wait_for_producers();
    const float g0 = dloss ? dloss[0] : 1.0f, g1 = dloss ? dloss[1] : 1.0f;
    const float zc = 2.0f * g1 * beta / static_cast<float>(max(valid[S + 1], 1));
    for (int s = seq_behind(offsets, S, T, c0); s < S; ++s) {
        const int a = max(seq_start(offsets, s, T), c0), b = min(seq_start(offsets, s + 1, T), c1);
        if (a >= c1) break;
        if (a >= b) continue;
        const double n = max(valid[s], 1);
        const float scale = static_cast<float>(static_cast<double>(g0) * alpha * E / (static_cast<double>(k) * n * n * max(valid[S], 1)));
        float c[V];
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int e = expert_of<G, VEC>(i, j);
            c[i] = e < E ? scale * static_cast<float>(counts[static_cast<int64_t>(s) * E + e]) : 0.0f;
        }
        for (int t0 = a; t0 < b; t0 += kRows) {
            const int t = t0 + warp * (32 / G) + lane / G;
            const int64_t tt = t < b ? t : a;
            const bool on = (!mask || mask[tt]) && t < b;
            const float l = lse[tt];
            float lc = l * kLog2e;
            float v[V];
            load_row<G, V, VEC>(logits + tt * E, E, j, -INFINITY, v);
            const bool far = fabsf(l) > kFar;
            if (__any_sync(0xffffffffu, far)) {
                float m = v[0];
#pragma unroll
                for (int i = 1; i < V; ++i) m = fmaxf(m, v[i]);
                m = group_max<G>(m);
                if (far) {
                    lc = 0.0f;
#pragma unroll
                    for (int i = 0; i < V; ++i) v[i] -= m;
                }
            }
            // exp(l - lse) up to a factor near 1 that the rounding of lse and of lse log2 e leaves: the row's sum undoes it
            float dot = 0.0f, sum = 0.0f;
#pragma unroll
            for (int i = 0; i < V; ++i) {
                v[i] = exp_from(v[i], lc);
                sum += v[i];
                dot = fmaf(v[i], c[i], dot);
            }
            sum = group_sum<G>(sum);
            dot = group_sum<G>(dot);
            if (t < b) {
                const float r = 1.0f / sum, shift = fmaf(zc, l, -dot * r);
                float* out = dlogits + static_cast<int64_t>(t) * E;
#pragma unroll
                for (int i = 0; i < V; ++i) v[i] = on ? v[i] * r * (c[i] + shift) : 0.0f;
                if constexpr (VEC) {
#pragma unroll
                    for (int q = 0; q < V / 4; ++q)
                        if (4 * (j + G * q) < E)
                            *reinterpret_cast<float4*>(out + 4 * (j + G * q)) = make_float4(v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]);
                } else {
#pragma unroll
                    for (int i = 0; i < V; ++i)
                        if (j + G * i < E) out[j + G * i] = v[i];
                }
            }
        }
    }
}

// ---------------------------------------------------------------- launches
// Calls f(tag) with the group size, values a lane and vector width for E experts.
template <int G_, bool VEC_>
struct RowForm { static constexpr int G = G_, V = 16; static constexpr bool VEC = VEC_; };

template <typename F>
cudaError_t with_row_form(int E, F f) {
    const bool vec = E % 4 == 0;
    if (E <= 64) return vec ? f(RowForm<4, true>()) : f(RowForm<4, false>());
    if (E <= 128) return vec ? f(RowForm<8, true>()) : f(RowForm<8, false>());
    if (E <= 256) return vec ? f(RowForm<16, true>()) : f(RowForm<16, false>());
    return vec ? f(RowForm<32, true>()) : f(RowForm<32, false>());
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }
bool ptr_ok(const void* p) { return p != nullptr && aligned16(p); }

moe_status_t check_balance(int T, int E, int k, int S, const void* offsets, float alpha, float beta) {
    if (T < 0 || E <= 0 || k <= 0 || S <= 0 || !isfinite(alpha) || !isfinite(beta)) return MOE_ERR_INVALID_ARG;
    if (E > MOE_MAX_EXPERTS || k > MOE_MAX_TOPK || S > MOE_MAX_SEQUENCES) return MOE_ERR_UNSUPPORTED_SHAPE;
    if (k > E || (!offsets && S != 1)) return MOE_ERR_INVALID_ARG;
    if (T > kMostTokens || static_cast<int64_t>(T) * k >= (1ll << 31)) return MOE_ERR_UNSUPPORTED_SHAPE;
    return MOE_OK;
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" {

size_t moe_balance_workspace_size(int T, int E, int S) {
    if (T < 0 || T > kMostTokens || E <= 0 || E > MOE_MAX_EXPERTS || S <= 0 || S > MOE_MAX_SEQUENCES) return 0;
    return carve_balance(T, E, S, nullptr).total;
}

moe_status_t moe_balance_loss(int T, int E, int k, const float* logits, const int32_t* topk_idx,
                              const uint8_t* token_mask, const int32_t* seq_offsets, int S, float alpha, float beta,
                              float* loss, int32_t* counts, float* mean_prob, float* lse, int32_t* seq_valid, void* ws,
                              size_t ws_bytes, void* stream) {
    moe_status_t st = check_balance(T, E, k, S, seq_offsets, alpha, beta);
    if (st != MOE_OK) return st;
    if (!ptr_ok(loss) || !ptr_ok(counts) || !ptr_ok(mean_prob) || !ptr_ok(seq_valid) || !ptr_ok(ws) ||
        !aligned16(token_mask) || !aligned16(seq_offsets))
        return MOE_ERR_INVALID_ARG;
    if (T > 0 && (!ptr_ok(logits) || !ptr_ok(topk_idx) || !ptr_ok(lse))) return MOE_ERR_INVALID_ARG;
    const BalWs w = carve_balance(T, E, S, ws);
    if (ws_bytes < w.total) return MOE_ERR_WORKSPACE_TOO_SMALL;
    int num_sms, *status;
    if ((st = current_device(&num_sms, &status)) != MOE_OK) return st;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const int C = chunk_tokens(T);
    cudaError_t err;
    if (T > 0 && T <= kSmallTokens) {
        const int Cs = std::max(16, (T + 16 * kSmallBlocks - 1) / (16 * kSmallBlocks) * 16), blocks = (T + Cs - 1) / Cs;
        err = with_row_form(E, [&](auto f) {
            using F = decltype(f);
            cudaLaunchConfig_t cfg = {};
            cudaLaunchAttribute attr[2];
            attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
            attr[0].val.programmaticStreamSerializationAllowed = 1;
            attr[1].id = cudaLaunchAttributeClusterDimension;
            attr[1].val.clusterDim.x = blocks;
            attr[1].val.clusterDim.y = 1;
            attr[1].val.clusterDim.z = 1;
            cfg.gridDim = dim3(blocks);
            cfg.blockDim = dim3(kFwdThreads);
            cfg.dynamicSmemBytes = sizeof(float) * (kFwdThreads / 32) * E;
            cfg.stream = s;
            cfg.attrs = attr;
            cfg.numAttrs = 2;
            return cudaLaunchKernelEx(&cfg, balance_small_kernel<F::G, F::V, F::VEC>, logits, topk_idx, token_mask, seq_offsets, T,
                                      E, k, S, Cs, w, lse, alpha, beta, loss, counts, mean_prob, seq_valid, status);
        });
        return err == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
    }
    if (T > 0) {
        err = with_row_form(E, [&](auto f) {
            using F = decltype(f);
            return launch_dependent(balance_partial_kernel<F::G, F::V, F::VEC>, dim3(chunks_of(T)), dim3(kFwdThreads),
                                    sizeof(float) * (kFwdThreads / 32) * E, s, logits, topk_idx, token_mask,
                                    seq_offsets, T, E, k, S, C, w, lse);
        });
    } else {
        err = cudaMemsetAsync(w.ticket, 0, sizeof(unsigned), s);   // no tokens: the reduction alone, over nothing
    }
    if (err == cudaSuccess) {
        const int cols = red_cols(S);
        err = launch_dependent(cols == 8 ? balance_reduce_kernel<8> : balance_reduce_kernel<32>, dim3((E + cols - 1) / cols, S),
                               dim3(kRedThreads), 0, s, seq_offsets, T, E, k, S, C, alpha, beta, w, loss, counts, mean_prob,
                               seq_valid, status);
    }
    return err == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

moe_status_t moe_balance_loss_backward(int T, int E, int k, const float* logits, const float* lse,
                                       const int32_t* counts, const int32_t* seq_valid, const uint8_t* token_mask,
                                       const int32_t* seq_offsets, int S, float alpha, float beta, const float* dloss,
                                       float* dlogits, void* stream) {
    moe_status_t st = check_balance(T, E, k, S, seq_offsets, alpha, beta);
    if (st != MOE_OK) return st;
    if (!aligned16(token_mask) || !aligned16(seq_offsets) || !aligned16(dloss)) return MOE_ERR_INVALID_ARG;
    if (T > 0 && (!ptr_ok(logits) || !ptr_ok(lse) || !ptr_ok(counts) || !ptr_ok(seq_valid) || !ptr_ok(dlogits)))
        return MOE_ERR_INVALID_ARG;
    int num_sms, *status;
    if ((st = current_device(&num_sms, &status)) != MOE_OK) return st;
    if (T == 0) return MOE_OK;
    const cudaError_t err = with_row_form(E, [&](auto f) {
        using F = decltype(f);
        // a block's tokens: whole turns of its rows, several only where enough blocks are left to fill the GPU
        const int turn = kBwdThreads / 32 * (32 / F::G);
        const int C = std::max(std::max(kBwdTokens, turn), (T / (4 * num_sms) + turn - 1) / turn * turn);
        return launch_dependent(balance_backward_kernel<F::G, F::V, F::VEC>, dim3((T + C - 1) / C), dim3(kBwdThreads), 0,
                                static_cast<cudaStream_t>(stream), logits, lse, counts, seq_valid, token_mask, seq_offsets, T,
                                E, k, S, C, alpha, beta, dloss, dlogits);
    });
    return err == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

}  // extern "C"
