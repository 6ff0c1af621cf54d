// A dense gradient of the router's logits through its linear layer (logits = x W_g^T + b):
//   dx = dx0 + dl W_g [T, H] bf16,  dWg = dWg0 + dl^T x [E, H] fp32,  db = db0 + sum_t dl.
//
// 4 T H E flops against x read once, dx0 read and dx written: at 256 experts the products and the traffic cost
// about the same, so both products run on the tensor cores and dx is bound by its own traffic.
//
//  1. Preparation. dl goes into three bf16 parts (8 + 8 + 8 bits, all of fp32) for dWg, with partial column sums for
//     db. W_g goes into two, and dx = d1 w1 + d1 w2 + d2 w1: a term is off by 2^-18 of it on average, 3 2^-16 at most
//     (half a step of bf16, 2^-8, twice over; three times: W_g's rest, dl's, d2 w2). Fewer bits would show: rows of a
//     softmax's gradient sum to zero, so what W_g's rows share cancels while its rounding errors do not (256 experts, a
//     shared row of 100 times their spread: fp16 operands leave dx 2.6e-2 off, these 4e-4, its own rounding is 1.7e-3).
//     bf16 needs no scales: nothing has to be known before the parts are made, so this is one launch.
//  2. router_products_kernel, dx: a CTA keeps its W_g panel (all experts x 256 or 128 columns) in shared memory and
//     streams token tiles through it (without that the panels alone would cost more L2 traffic than dx does HBM
//     traffic), the next box of dx0 loading meanwhile. dWg: the transposed product, x^T (rows h) by the parts of
//     dl, both operands read as they lie in memory (MN-major), so E is the MMA's N and a few experts cost little:
//     up to 64 experts the three parts lie side by side in one N of 48, 96 or 192 (an MMA of N <= 112 takes as
//     long as one of 112). The tensor cores drop bits when they add to a long sum, so every 128 tokens the sum
//     moves from tensor memory into fp32 registers. The work of either product is dealt out evenly as one run of
//     units a CTA (or pair); for dWg it leaves one partial tile per tile it touched, at index tile + its own index
//     (unique: both only rise), and
//  3. router_finish_kernel adds the partial tiles in order, and db. No float atomics: results repeat.
//
// Measured on a B200, replayed: 8192 x 7168 x 256 159 us (383 MB; 180 GFLOP of MMAs, 148 us of it the products at 1.2
// PFLOP/s, where the power cap takes the clock to 1.6 GHz in one launch and below in many: 189 us a call among others;
// with one fp16 product for dx, which lost the bits named above, 125 and 150), 4096 x 4096 x 64 34.6 us (products 28: dx's
// traffic, and filling two pipelines), 5003 x 1408 x 100 28.5 us (latency of three launches), 256 x 512 x 8 4.9 us (one
// launch). The products' 232 registers a thread leave 20 to 28 bytes of spills.
#include <algorithm>

#include "../../include/moe_fp8.h"
#include "common.cuh"

namespace moe {

moe_status_t current_device(int* num_sms, int** status);

namespace {

constexpr uint64_t kRbWaitNs = 4000000000ull;
constexpr int kRbBox = 64 * 64 * 2;            // a 64 x 64 operand box: 8 KB
constexpr int kRbThreads = 384;                // TMA, MMA, two idle warps, eight epilogue warps
constexpr int kPrepTokens = 32;                // tokens of a dl preparation block, four a warp
constexpr int kRbChunk = 128;                  // tokens summed in tensor memory before promotion

__device__ __forceinline__ uint16_t bf16_bits(float f) { return __bfloat16_as_ushort(__float2bfloat16_rn(f)); }

// ---------------------------------------------------------------- 1. preparation
// The first dl_blocks blocks: dl rows -> three bf16 parts and the block's column sums; a warp takes a token at a time, Q
// groups of four experts a lane (16-byte reads where E is a multiple of 4). Value e of part p of token t goes to
// t * row + p * part + e, with zeros behind the last expert up to `width`. The others: W_g -> two bf16 parts [2][E][H],
// 4096 values a block.
constexpr int kPrepW = 4096;

// The first part holds an infinite or NaN value alone; what is left of a finite one is exact.
__device__ __forceinline__ float rest_of(float r, uint16_t b) { return fabsf(r) <= 3.0e38f ? r - bf16_bits_to_f32(b) : 0.0f; }
__device__ __forceinline__ void put4(uint16_t* dst, const uint16_t (&u)[4]) {
    *reinterpret_cast<uint2*>(dst) = make_uint2(u[0] | static_cast<uint32_t>(u[1]) << 16, u[2] | static_cast<uint32_t>(u[3]) << 16);
}

template <int Q, bool VEC>
__global__ void __launch_bounds__(256)
router_prep_parts_kernel(const float* __restrict__ dl, const float* __restrict__ Wg, int T, int H, int E, int width,
                         int64_t row, int64_t part, int dl_blocks, uint16_t* __restrict__ parts,
                         float* __restrict__ dbpart, uint16_t* __restrict__ w2) {
    __shared__ float sm[8][Q * 128];
    dependents_may_launch();
    wait_for_producers();
    if (static_cast<int>(blockIdx.x) >= dl_blocks) {
        const int64_t n = static_cast<int64_t>(E) * H, i0 = static_cast<int64_t>(blockIdx.x - dl_blocks) * kPrepW + threadIdx.x * 4;
        float4 f[kPrepW / 1024];
#pragma unroll
        for (int i = 0; i < kPrepW / 1024; ++i)
            if (i0 + i * 1024 < n) f[i] = *reinterpret_cast<const float4*>(Wg + i0 + i * 1024);
#pragma unroll
        for (int i = 0; i < kPrepW / 1024; ++i)
            if (i0 + i * 1024 < n) {
                const float v[4] = {f[i].x, f[i].y, f[i].z, f[i].w};
                uint16_t b[2][4];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    b[0][j] = bf16_bits(v[j]);
                    b[1][j] = bf16_bits(rest_of(v[j], b[0][j]));
                }
                put4(w2 + i0 + i * 1024, b[0]);
                put4(w2 + n + i0 + i * 1024, b[1]);
            }
        return;
    }
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int t0 = blockIdx.x * kPrepTokens + warp;
    float v[kPrepTokens / 8][4 * Q], sum[4 * Q] = {};
#pragma unroll
    for (int k = 0; k < kPrepTokens / 8; ++k) {
        const int t = t0 + 8 * k;
#pragma unroll
        for (int q = 0; q < Q; ++q) {
            const int e = 4 * (lane + 32 * q);
            const float* p = dl + static_cast<int64_t>(t) * E + e;
            if constexpr (VEC) {
                float4 f = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                if (t < T && e < E) f = *reinterpret_cast<const float4*>(p);
                v[k][4 * q] = f.x; v[k][4 * q + 1] = f.y; v[k][4 * q + 2] = f.z; v[k][4 * q + 3] = f.w;
            } else {
#pragma unroll
                for (int i = 0; i < 4; ++i) v[k][4 * q + i] = t < T && e + i < E ? p[i] : 0.0f;
            }
        }
    }
#pragma unroll
    for (int k = 0; k < kPrepTokens / 8; ++k) {
        const int t = t0 + 8 * k;
#pragma unroll
        for (int q = 0; q < Q; ++q) {
            const int e = 4 * (lane + 32 * q);
            uint16_t b[3][4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                float r = v[k][4 * q + i];
                sum[4 * q + i] += r;
#pragma unroll
                for (int p = 0; p < 3; ++p) {
                    b[p][i] = bf16_bits(r);
                    r = rest_of(r, b[p][i]);
                }
            }
            if (t < T && e < width) {
#pragma unroll
                for (int p = 0; p < 3; ++p) put4(parts + t * row + p * part + e, b[p]);
            }
        }
    }
#pragma unroll
    for (int i = 0; i < 4 * Q; ++i) sm[warp][4 * (lane + 32 * (i / 4)) + i % 4] = sum[i];
    __syncthreads();
    for (int e = threadIdx.x; e < E; e += 256) {
        float s = 0.0f;
#pragma unroll
        for (int i = 0; i < 8; ++i) s += sm[i][e];
        dbpart[static_cast<int64_t>(blockIdx.x) * E + e] = s;
    }
}

// ---------------------------------------------------------------- 2. the products
// PAIR (above 128 experts): CTA pairs, 256 tokens x `kPanel` columns of dx, 256 columns x 256 experts of dWg. The
// operand that both halves of a tile need is then held once a pair: 64 KB a stage cross from L2 where single CTAs
// would load 112 KB for the same MMAs. Otherwise single CTAs, 128 x 256 and 128 x `pitch` (16, 32, 64 or 128). KB:
// 64-expert blocks of the W_g panel, of both its parts in turn; WB: 64-column boxes of one that a CTA holds; AS: blocks of
// the tokens' ring, NB: dx0 / dx boxes an epilogue warp holds (what the panel leaves room for). The panel is 256 columns
// wide, above 256 experts 128.
// Units are dealt out as runs: group g of G takes [g U / G, (g + 1) U / G).
constexpr int kDwStages = 4;                                               // barriers; the ring's depth goes by E
constexpr int kDwRing = 24 * kRbBox;                                       // its bytes: 192 KB
constexpr int kDwRegsLow = 40, kDwRegsHigh = 232;                          // as in the grouped GEMM:
constexpr int kDwRegsSplit = 128 * kDwRegsLow + 256 * kDwRegsHigh;        // what the launch must have allocated

template <int KB, int WB, int AS, int NB>
struct SmemDx {
    uint8_t w[KB][WB * kRbBox];                        // the CTA's panel columns (of a pair's half of them)
    uint8_t a[AS][2 * kRbBox];                         // 64 experts of 128 tokens
    uint8_t stage[8][NB][4096];                        // per epilogue warp: 32 rows x 64 columns, bf16
};
// dWg's ring: a stage is 2 boxes of x (128 columns), then boxes of 64 columns of dl's parts. PAIR: 64 tokens, 2 boxes
// a part (64 KB); pitch 128 likewise; up to pitch 64 a whole chunk of 128 tokens and 1, 2 or 3 boxes of the parts side by
// side (48, 64 or 80 KB).
struct SmemDw {
    uint8_t ring[kDwRing];
};
template <int KB, int WB, int AS, int NB>
struct SmemP {
    union {
        SmemDx<KB, WB, AS, NB> dx;
        SmemDw dw;
    };
    uint64_t wfull, wempty;
    uint64_t afull[AS], aempty[AS];
    uint64_t eload[8][NB];
    uint64_t full[kDwStages], empty[kDwStages];
    uint64_t tfull[2][2], tempty[2][2];        // [product][accumulator]
    uint32_t tmem_base;
    volatile int abort_flag;
};

__host__ __device__ __forceinline__ int unit_start(int U, int G, int g) { return static_cast<int>(static_cast<int64_t>(U) * g / G); }
// The group that holds unit u: the largest g with unit_start(g) <= u.
inline int group_of(int U, int G, int u) { return static_cast<int>((static_cast<int64_t>(u + 1) * G + U - 1) / U - 1); }

struct RouterArgs {
    int T, H, E;
    int has_base;
    int Gx, Gw;               // groups that share dx's units, dWg's units
    int etiles;               // expert tiles of dWg
    int pitch;                // single CTAs: columns of a part of dl, its experts rounded up
    int Ux, Uw;
    float* part;
    int* status;
};

template <bool PAIR, int KB, int WB, int AS, int NB>
__global__ void __launch_bounds__(kRbThreads, 1)
router_products_kernel(const __grid_constant__ CUtensorMap tm_dl, const __grid_constant__ CUtensorMap tm_w,
                       const __grid_constant__ CUtensorMap tm_in, const __grid_constant__ CUtensorMap tm_out,
                       const __grid_constant__ CUtensorMap tm_x, const __grid_constant__ CUtensorMap tm_d,
                       const RouterArgs g) {
    constexpr int kTok = PAIR ? 256 : 128;                      // tokens of a dx tile
    constexpr int kRows = PAIR ? 256 : 128, kCols = PAIR ? 256 : 128;   // dWg tile: columns of x, experts
    constexpr int kPanel = (PAIR ? 2 : 1) * 64 * WB, kBoxes = kPanel / 128;     // its boxes of a unit, an epilogue warp
    extern __shared__ uint8_t smem_raw[];
    using SP = SmemP<KB, WB, AS, NB>;
    SP& sm = *reinterpret_cast<SP*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = PAIR ? cluster_ctarank() : 0;
    const int grp = PAIR ? static_cast<int>(cluster_id_x()) : static_cast<int>(blockIdx.x);
    if (threadIdx.x == 0) {
        mbar_init(&sm.wfull, 1);
        mbar_init(&sm.wempty, 1);
        for (int s = 0; s < AS; ++s) { mbar_init(&sm.afull[s], 1); mbar_init(&sm.aempty[s], 1); }
        for (int s = 0; s < kDwStages; ++s) { mbar_init(&sm.full[s], 1); mbar_init(&sm.empty[s], 1); }
        for (int p = 0; p < 2; ++p)
            for (int i = 0; i < 2; ++i) { mbar_init(&sm.tfull[p][i], 1); mbar_init(&sm.tempty[p][i], PAIR ? 16 : 8); }
        for (int i = 0; i < 8; ++i)
            for (int n = 0; n < NB; ++n) mbar_init(&sm.eload[i][n], 1);
        sm.abort_flag = 0;
        fence_mbar_init();
    }
    if (warp == 1) {
        if constexpr (PAIR) { tmem_alloc_pair(&sm.tmem_base, 512); tmem_relinquish_pair(); }
        else { tmem_alloc(&sm.tmem_base, 512); tmem_relinquish(); }
    }
    if (threadIdx.x == 0) {
        prefetch_tensormap(&tm_dl); prefetch_tensormap(&tm_w); prefetch_tensormap(&tm_in);
        prefetch_tensormap(&tm_out); prefetch_tensormap(&tm_x); prefetch_tensormap(&tm_d);
    }
    tc_fence_before();
    if constexpr (PAIR) cluster_sync(); else __syncthreads();
    tc_fence_after();
    const uint32_t tmem = sm.tmem_base;
    dependents_may_launch();
    wait_for_producers();
    auto fail = [&]() {
        set_status(g.status, kStatusTimeout);
        sm.abort_flag = 1;
        if constexpr (PAIR) st_shared_cluster_u32(mapa_shared(smem_u32((const void*)&sm.abort_flag), rank ^ 1u), 1u);
    };
    auto leader_bar = [&](uint64_t* bar) -> uint32_t { return PAIR ? mapa_shared(smem_u32(bar), 0) : 0u; };
    auto release = [&](uint64_t* bar) {       // an accumulator buffer, by one lane of an epilogue warp
        if (PAIR && rank) mbar_arrive_cluster(leader_bar(bar));
        else mbar_arrive(bar);
    };

    // ======== dx: unit u = token tile u % ttiles of panel u / ttiles
    const int ttiles = (g.T + kTok - 1) / kTok, kblocks = (g.E + 63) / 64;
    const int x0 = grp < g.Gx ? unit_start(g.Ux, g.Gx, grp) : 0, x1 = grp < g.Gx ? unit_start(g.Ux, g.Gx, grp + 1) : 0;
    // ======== dWg: unit u = 128-token chunk u % chunks of tile u / chunks
    const int chunks = (g.T + kRbChunk - 1) / kRbChunk;
    const int u0 = grp < g.Gw ? unit_start(g.Uw, g.Gw, grp) : 0, u1 = grp < g.Gw ? unit_start(g.Uw, g.Gw, grp + 1) : 0;
    const bool wide = !PAIR && g.pitch <= 64;                           // the parts side by side in one MMA
    const int ts = wide ? 128 : 64;                                     // tokens of a stage
    const int dboxes = wide ? (3 * g.pitch + 63) / 64 : 6;
    const uint32_t box = ts * 128, stage_bytes = (2 + dboxes) * box;
    const uint32_t depth = kDwRing / stage_bytes;
    auto stage_x = [&](uint32_t s) { return sm.dw.ring + s * stage_bytes; };
    auto stage_d = [&](uint32_t s, int i) { return sm.dw.ring + s * stage_bytes + (2 + i) * box; };

    // The products are independent: half of the groups begin with dWg, so that dx's traffic and dWg's products run
    // beside each other on the GPU. Between the two a group's MMAs are complete (their accumulators were waited
    // for), and its stores have left shared memory.
    const int dx_turn = grp & 1;
    auto turn_over = [&]() {
        __syncwarp();
        if constexpr (PAIR) cluster_sync(); else __syncthreads();
    };
    if (warp < 4) {
        setmaxnreg_dec<kDwRegsLow>();
        for (int turn = 0; turn < 2; ++turn) {
            if (turn == dx_turn) {
                if (warp == 0 && lane == 0) {
                    uint32_t it = 0, panels = 0;
                    int have = -1;
                    bool ok = !sm.abort_flag;
                    for (int u = x0; ok && u < x1; ++u) {
                        const int panel = u / ttiles, tile = u - panel * ttiles;
                        if (panel != have) {
                            // the panel before it is no longer read: its last MMAs have committed
                            if (panels > 0 && !mbar_wait(&sm.wempty, (panels - 1) & 1, kRbWaitNs)) { fail(); break; }
                            have = panel;
                            ++panels;
                            const int c0 = panel * kPanel + static_cast<int>(rank) * 64 * WB;
                            // both parts of the panel (PAIR: of this CTA's half of it)
                            if (rank == 0) mbar_arrive_expect_tx(&sm.wfull, (PAIR ? 2u : 1u) * 2 * kblocks * WB * kRbBox);
                            for (int kb = 0; kb < 2 * kblocks; ++kb)
                                for (int i = 0; i < WB; ++i) {
                                    if constexpr (PAIR)
                                        tma_load_3d_pair(sm.dx.w[kb] + i * kRbBox, &tm_w, leader_bar(&sm.wfull), c0 + 64 * i, (kb >> 1) * 64, kb & 1);
                                    else
                                        tma_load_3d(sm.dx.w[kb] + i * kRbBox, &tm_w, &sm.wfull, c0 + 64 * i, (kb >> 1) * 64, kb & 1);
                                }
                        }
                        // the tile's dl, its first part and its second, block by block
                        for (int kb = 0; kb < 2 * kblocks; ++kb, ++it) {
                            const int s = it % AS;
                            if (!mbar_wait(&sm.aempty[s], ((it / AS) & 1) ^ 1, kRbWaitNs)) { fail(); ok = false; break; }
                            if (rank == 0) mbar_arrive_expect_tx(&sm.afull[s], (PAIR ? 2u : 1u) * 2 * kRbBox);
                            if constexpr (PAIR)
                                tma_load_3d_pair(sm.dx.a[s], &tm_dl, leader_bar(&sm.afull[s]), (kb >> 1) * 64, tile * kTok + static_cast<int>(rank) * 128, kb & 1);
                            else
                                tma_load_2d(sm.dx.a[s], &tm_dl, &sm.afull[s], (kb & 1) * g.pitch + (kb >> 1) * 64, tile * kTok);
                        }
                    }
                } else if (warp == 1 && lane == 0 && rank == 0) {
                    uint32_t it = 0, ti = 0, panels = 0;
                    int have = -1;
                    const uint32_t idesc = f16_idesc(kTok, kPanel, true, false, true);
                    bool ok = !sm.abort_flag;
                    for (int u = x0; ok && u < x1 && !sm.abort_flag; ++u, ++ti) {
                        const int panel = u / ttiles;
                        if (panel != have) {
                            have = panel;
                            if (!mbar_wait(&sm.wfull, panels & 1, kRbWaitNs)) { fail(); break; }
                            ++panels;
                        }
                        const uint32_t buf = ti & 1, d = tmem + buf * 256;
                        if (!mbar_wait(&sm.tempty[0][buf], ((ti >> 1) & 1) ^ 1, kRbWaitNs)) { fail(); break; }
                        tc_fence_after();
                        for (int kb = 0; kb < 2 * kblocks; ++kb, ++it) {
                            const int s = it % AS;
                            if (!mbar_wait(&sm.afull[s], (it / AS) & 1, kRbWaitNs)) { fail(); ok = false; break; }
                            tc_fence_after();
                            // 16 experts on (the descriptors hold address / 16): 32 bytes in a row, 2048 in the panel
                            const uint64_t da = sw128_kmajor_desc(smem_u32(sm.dx.a[s]));
                            const uint64_t db = sw128_mnmajor_desc(smem_u32(sm.dx.w[kb & ~1]), kRbBox);
#pragma unroll
                            for (int kk = 0; kk < 4; ++kk) {
                                if constexpr (PAIR) umma_f16_pair(d, da + kk * 2, db + kk * 128, idesc, kb + kk > 0);
                                else umma_f16(d, da + kk * 2, db + kk * 128, idesc, kb + kk > 0);
                            }
                            if (!(kb & 1)) {                       // the first part of dl also meets the second of W_g
                                const uint64_t d2 = sw128_mnmajor_desc(smem_u32(sm.dx.w[kb | 1]), kRbBox);
#pragma unroll
                                for (int kk = 0; kk < 4; ++kk) {
                                    if constexpr (PAIR) umma_f16_pair(d, da + kk * 2, d2 + kk * 128, idesc, 1);
                                    else umma_f16(d, da + kk * 2, d2 + kk * 128, idesc, 1);
                                }
                            }
                            if constexpr (PAIR) umma_commit_pair(&sm.aempty[s], 0x3); else umma_commit(&sm.aempty[s]);
                        }
                        if (ok) {
                            if constexpr (PAIR) umma_commit_pair(&sm.tfull[0][buf], 0x3); else umma_commit(&sm.tfull[0][buf]);
                            if (u + 1 < x1 && (u + 1) / ttiles != panel) {
                                if constexpr (PAIR) umma_commit_pair(&sm.wempty, 0x3); else umma_commit(&sm.wempty);
                            }
                        }
                    }
                }
            } else {
                if (warp == 0 && lane == 0) {
                    uint32_t it = 0;
                    bool ok = !sm.abort_flag;
                    const uint32_t bytes = (PAIR ? 2u : 1u) * stage_bytes;
                    for (int u = u0; ok && u < u1; ++u) {
                        const int tile = u / chunks, t0 = (u - tile * chunks) * kRbChunk;
                        const int h0 = tile / g.etiles * kRows + static_cast<int>(rank) * 128;
                        const int e0 = tile % g.etiles * kCols + static_cast<int>(rank) * 128;
                        for (int t = t0; t < min(t0 + kRbChunk, g.T); t += ts, ++it) {
                            const uint32_t s = it % depth;
                            if (!mbar_wait(&sm.empty[s], ((it / depth) & 1) ^ 1, kRbWaitNs)) { fail(); ok = false; break; }
                            if (rank == 0) mbar_arrive_expect_tx(&sm.full[s], bytes);
                            if constexpr (PAIR) {
                                const uint32_t fb = leader_bar(&sm.full[s]);
                                for (int i = 0; i < 2; ++i) tma_load_3d_pair(stage_x(s) + i * box, &tm_x, fb, h0 + 64 * i, t, 0);
                                for (int i = 0; i < 6; ++i) tma_load_3d_pair(stage_d(s, i), &tm_d, fb, e0 + 64 * (i & 1), t, i >> 1);
                            } else {
                                for (int i = 0; i < 2; ++i) tma_load_3d(stage_x(s) + i * box, &tm_x, &sm.full[s], h0 + 64 * i, t, 0);
                                for (int i = 0; i < dboxes; ++i) tma_load_3d(stage_d(s, i), &tm_d, &sm.full[s], 64 * i, t, 0);
                            }
                        }
                    }
                } else if (warp == 1 && lane == 0 && rank == 0) {
                    uint32_t it = 0, ci = 0;
                    bool ok = !sm.abort_flag;
                    const uint32_t idesc = f16_idesc(kRows, PAIR ? 256 : wide ? 3 * g.pitch : 128, true, true, true);
                    for (int u = u0; ok && u < u1 && !sm.abort_flag; ++u, ++ci) {
                        const int t0 = u % chunks * kRbChunk;
                        const uint32_t buf = ci & 1, d = tmem + buf * 256;
                        if (!mbar_wait(&sm.tempty[1][buf], ((ci >> 1) & 1) ^ 1, kRbWaitNs)) { fail(); break; }
                        tc_fence_after();
                        for (int t = t0; t < min(t0 + kRbChunk, g.T); t += ts, ++it) {
                            const uint32_t s = it % depth;
                            if (!mbar_wait(&sm.full[s], (it / depth) & 1, kRbWaitNs)) { fail(); ok = false; break; }
                            tc_fence_after();
                            // the descriptors hold address / 16: a slice of 16 tokens is 2048 bytes on
                            const uint64_t da = sw128_mnmajor_desc(smem_u32(stage_x(s)), box);
                            const uint64_t db = sw128_mnmajor_desc(smem_u32(stage_d(s, 0)), box);
                            if (wide) {
#pragma unroll
                                for (int kk = 0; kk < 8; ++kk) umma_f16(d, da + kk * 128, db + kk * 128, idesc, kk > 0);
                            } else {
                                // the three parts of a slice share x, which the tensor core then reads once
#pragma unroll
                                for (int kk = 0; kk < 4; ++kk) {
                                    const uint64_t a = da + kk * 128, b = db + kk * 128;
                                    umma_f16_keep<PAIR, KeepA::kFill>(d, a, b, idesc, kk > 0 || t > t0);
                                    umma_f16_keep<PAIR, KeepA::kUse>(d, a, b + 2 * kRbBox / 16, idesc, 1);
                                    umma_f16_keep<PAIR, KeepA::kLast>(d, a, b + 4 * kRbBox / 16, idesc, 1);
                                }
                            }
                            if constexpr (PAIR) umma_commit_pair(&sm.empty[s], 0x3); else umma_commit(&sm.empty[s]);
                        }
                        if (ok) { if constexpr (PAIR) umma_commit_pair(&sm.tfull[1][buf], 0x3); else umma_commit(&sm.tfull[1][buf]); }
                    }
                }
            }
            turn_over();
        }
    } else {
        setmaxnreg_inc<kDwRegsHigh>();
        for (int turn = 0; turn < 2; ++turn) {
            if (turn == dx_turn) {
                const int ew = warp - 4, q = warp & 3, half = ew >> 2;
                // the warp's 32 rows x half a panel of a unit as kBoxes boxes of 64 columns; box j goes through buffer
                // j % NB: dx0 comes in one box ahead, dx leaves from the same place
                const uint32_t boxes = static_cast<uint32_t>(kBoxes * (x1 - x0));
                auto place = [&](uint32_t j, int& row0, int& col0) {
                    const int u = x0 + static_cast<int>(j / kBoxes);
                    const int panel = u / ttiles, tile = u - panel * ttiles;
                    row0 = tile * kTok + static_cast<int>(rank) * 128 + q * 32;
                    col0 = panel * kPanel + half * (kPanel / 2) + 64 * static_cast<int>(j % kBoxes);
                };
                auto fetch = [&](uint32_t j) {         // lane 0
                    int row0, col0;
                    place(j, row0, col0);
                    uint64_t* bar = &sm.eload[ew][j % NB];
                    mbar_arrive_expect_tx(bar, 4096);
                    tma_load_2d(sm.dx.stage[ew][j % NB], &tm_in, bar, col0, row0);
                };
                if (g.has_base && lane == 0 && boxes > 0 && !sm.abort_flag) fetch(0);
                for (uint32_t j = 0; j < boxes; ++j) {
                    if (sm.abort_flag) break;
                    const uint32_t ti = j / kBoxes, buf = ti & 1, n = j % NB;
                    int row0, col0;
                    place(j, row0, col0);
                    if (lane == 0) {
                        bulk_wait_read<NB - 2>();      // box j + 1 - NB has left the buffer that box j + 1 goes to
                        if (g.has_base && j + 1 < boxes) fetch(j + 1);
                    }
                    __syncwarp();
                    if (j % kBoxes == 0) {
                        if (!mbar_wait(&sm.tfull[0][buf], (ti >> 1) & 1, kRbWaitNs)) { fail(); break; }
                        tc_fence_after();
                    }
                    if (g.has_base && !mbar_wait(&sm.eload[ew][n], (j / NB) & 1, kRbWaitNs)) { fail(); break; }
                    const uint32_t taddr = tmem + (static_cast<uint32_t>(q * 32) << 16) + buf * 256 + half * (kPanel / 2) + 64 * (j % kBoxes);
#pragma unroll
                    for (int i = 0; i < 2; ++i) {      // 32 columns at a time
                        float v[32];
                        tmem_ld32(taddr + 32 * i, v);
                        // 16-byte piece p of row `lane` sits at p ^ (lane & 7)
                        const uint32_t st = smem_u32(sm.dx.stage[ew][n]) + lane * 128;
                        auto at = [&](int p) { return st + (((i * 4 + p) ^ (lane & 7)) << 4); };
                        uint32_t b[4][4] = {};
                        if (g.has_base) {
#pragma unroll
                            for (int p = 0; p < 4; ++p)
                                asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(b[p][0]), "=r"(b[p][1]), "=r"(b[p][2]), "=r"(b[p][3]) : "r"(at(p)) : "memory");
                        }
                        tmem_ld_wait();
                        if (i == 1 && j % kBoxes == kBoxes - 1) {
                            tc_fence_before();
                            __syncwarp();
                            if (lane == 0) release(&sm.tempty[0][buf]);
                        }
#pragma unroll
                        for (int p = 0; p < 4; ++p) {
                            uint32_t o[4];
#pragma unroll
                            for (int k = 0; k < 4; ++k) {
                                const float2 y = __fadd2_rn(make_float2(v[p * 8 + 2 * k], v[p * 8 + 2 * k + 1]),
                                                            make_float2(__uint_as_float(b[p][k] << 16), __uint_as_float(b[p][k] & 0xffff0000u)));
                                const __nv_bfloat162 r = __floats2bfloat162_rn(y.x, y.y);
                                o[k] = *reinterpret_cast<const uint32_t*>(&r);
                            }
                            st_shared_v4(at(p), o[0], o[1], o[2], o[3]);
                        }
                    }
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) {
                        if (row0 < g.T && col0 < g.H) tma_store_2d(&tm_out, sm.dx.stage[ew][n], col0, row0);
                        bulk_commit();
                    }
                }
                if (lane == 0) bulk_wait_read_all();
            } else {
                // promotion: warp = lane quadrant q x half of the experts
                constexpr int kMine = PAIR ? 128 : 64;
                const int q = warp & 3, half = (warp - 4) >> 2;
                const int mine = PAIR ? kMine : g.pitch / 2, cols = PAIR ? kCols : g.pitch;
                float acc[kMine];
                uint32_t ci = 0;
                for (int u = u0; u < u1; ++u, ++ci) {
                    if (sm.abort_flag) break;
                    const int tile = u / chunks;
                    const bool begin = u == u0 || u % chunks == 0, end = u + 1 == u1 || (u + 1) % chunks == 0;
                    if (begin) {
#pragma unroll
                        for (int i = 0; i < kMine; ++i) acc[i] = 0.0f;
                    }
                    const uint32_t buf = ci & 1;
                    if (!mbar_wait(&sm.tfull[1][buf], (ci >> 1) & 1, kRbWaitNs)) { fail(); break; }
                    tc_fence_after();
                    const uint32_t taddr = tmem + (static_cast<uint32_t>(q * 32) << 16) + buf * 256 + half * mine;
                    if (!wide) {
#pragma unroll
                        for (int c = 0; c < kMine / 32; ++c) {
                            float v[32];
                            tmem_ld32(taddr + 32 * c, v);
                            tmem_ld_wait();
#pragma unroll
                            for (int i = 0; i < 32; ++i) acc[32 * c + i] += v[i];
                        }
                    } else if (g.pitch == 64) {
#pragma unroll
                        for (int p = 0; p < 3; ++p) {
                            float v[32];
                            tmem_ld32(taddr + 64 * p, v);
                            tmem_ld_wait();
#pragma unroll
                            for (int i = 0; i < 32; ++i) acc[i] += v[i];
                        }
                    } else {
                        // 16 columns of each part (at pitch 16 the upper 8 are another warp's or nobody's, and not kept)
#pragma unroll
                        for (int p = 0; p < 3; ++p) {
                            float v[16];
                            tmem_ld16(taddr + g.pitch * p, v);
                            tmem_ld_wait();
#pragma unroll
                            for (int i = 0; i < 16; ++i) acc[i] += v[i];
                        }
                    }
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) release(&sm.tempty[1][buf]);
                    if (end) {
                        // partial tile [cols][kRows]: a warp's store is 32 consecutive rows of one expert
                        float* dst = g.part + (static_cast<int64_t>(tile) + grp) * cols * kRows + rank * 128 + q * 32 + lane;
                        const int ecount = min(g.E - tile % g.etiles * cols, (half + 1) * mine);
#pragma unroll
                        for (int i = 0; i < kMine; ++i)
                            if (half * mine + i < ecount) dst[(half * mine + i) * kRows] = acc[i];
                    }
                }
            }
            turn_over();
        }
        if (lane == 0) bulk_wait_all();               // dx's stores have completed
    }
    __syncwarp();
    tc_fence_before();
    if constexpr (PAIR) cluster_sync(); else __syncthreads();
    if (sm.abort_flag) {
        const uint64_t t0 = globaltimer_ns();
        while (globaltimer_ns() - t0 < 200000) __nanosleep(1000);   // copies and MMAs in flight land
    }
    if constexpr (PAIR) cluster_sync(); else __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        if constexpr (PAIR) tmem_dealloc_pair(tmem, 512); else tmem_dealloc(tmem, 512);
    }
}

// ---------------------------------------------------------------- 3. sums of the partial tiles, db
// The groups that touched each tile: first[t] .. last[t] (at most 128 tiles, 160 groups).
struct TileGroups {
    uint8_t first[128], last[128];
};

// Block (x, e): 1024 columns of expert e, four a thread; the first 32 threads of column block 0 also db[e].
__global__ void __launch_bounds__(256)
router_finish_kernel(const float* __restrict__ part, const float* __restrict__ dbpart, const __grid_constant__ TileGroups tg,
                     int H, int E, int rows, int cols, int etiles, int summed, int db_blocks, const float* dWg0,
                     const float* db0, float* dWg, float* db) {
    const int e = blockIdx.y, h = (blockIdx.x * 256 + threadIdx.x) * 4;
    dependents_may_launch();
    wait_for_producers();
    if (h < H) {
        const int64_t at = static_cast<int64_t>(e) * H + h;
        float4 s = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        if (dWg0) s = *reinterpret_cast<const float4*>(dWg0 + at);
        if (summed) {
            const int tile = h / rows * etiles + e / cols, g0 = tg.first[tile], n = tg.last[tile] - g0 + 1;
            const int64_t step = static_cast<int64_t>(cols) * rows;
            const float* p = part + (tile + g0) * step + static_cast<int64_t>(e % cols) * rows + h % rows;
            float4 a = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            for (int g = 0; g < n; g += 4) {
                float4 v[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) v[i] = g + i < n ? *reinterpret_cast<const float4*>(p + (g + i) * step) : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
                for (int i = 0; i < 4; ++i) { a.x += v[i].x; a.y += v[i].y; a.z += v[i].z; a.w += v[i].w; }
            }
            s.x += a.x; s.y += a.y; s.z += a.z; s.w += a.w;
        }
        *reinterpret_cast<float4*>(dWg + at) = s;
    }
    if (blockIdx.x == 0 && threadIdx.x < 32) {
        double s = 0.0;
#pragma unroll 4
        for (int b = threadIdx.x; b < db_blocks; b += 32) s += dbpart[static_cast<int64_t>(b) * E + e];
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
        if (threadIdx.x == 0) db[e] = static_cast<float>(s + (db0 ? db0[e] : 0.0));
    }
}

// ---------------------------------------------------------------- few tokens: both products on the CUDA cores
// One launch instead of four, fp32 throughout. The first dx_blocks blocks: 16 tokens x 256 columns of dx, a thread 4
// tokens x 4 columns, dl transposed in shared memory. The others: 64 columns x 16 experts of dWg over all tokens, a
// thread 4 columns x 16 experts of every 16th token, the 16 slices added in order; those of column tile 0 also db.
constexpr int kDirTok = 16, kDirCols = 256;              // dx tile
constexpr int kDirH = 64, kDirE = 16, kDirChunk = 128;   // dWg tile, tokens of dl staged at a time

template <bool BASE>
__global__ void __launch_bounds__(256)
router_direct_kernel(const uint16_t* __restrict__ x, const float* __restrict__ Wg, const float* __restrict__ dl, int T, int H,
                     int E, int dx_blocks, const uint16_t* dx0, const float* dWg0, const float* db0, uint16_t* dx,
                     float* dWg, float* db) {
    extern __shared__ float sm_f[];
    const int tid = threadIdx.x;
    dependents_may_launch();
    wait_for_producers();
    if (static_cast<int>(blockIdx.x) < dx_blocks) {
        const int ct = (H + kDirCols - 1) / kDirCols;
        const int t0 = blockIdx.x / ct * kDirTok, h = blockIdx.x % ct * kDirCols + (tid & 63) * 4, tg = tid >> 6;
        float* sd = sm_f;                                 // [E][16]
        for (int i = tid; i < E * kDirTok; i += 256) {
            const int t = i / E, e = i - t * E;
            sd[e * kDirTok + t] = t0 + t < T ? dl[static_cast<int64_t>(t0 + t) * E + e] : 0.0f;
        }
        __syncthreads();
        if (h >= H) return;
        float acc[4][4] = {};
#pragma unroll 8
        for (int e = 0; e < E; ++e) {
            const float4 w = __ldg(reinterpret_cast<const float4*>(Wg + static_cast<int64_t>(e) * H + h));
            const float4 d = *reinterpret_cast<const float4*>(sd + e * kDirTok + tg * 4);
            const float dd[4] = {d.x, d.y, d.z, d.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                acc[i][0] = fmaf(dd[i], w.x, acc[i][0]);
                acc[i][1] = fmaf(dd[i], w.y, acc[i][1]);
                acc[i][2] = fmaf(dd[i], w.z, acc[i][2]);
                acc[i][3] = fmaf(dd[i], w.w, acc[i][3]);
            }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int t = t0 + tg * 4 + i;
            if (t >= T) break;
            const int64_t at = static_cast<int64_t>(t) * H + h;
            if (BASE) {
                const uint2 b = *reinterpret_cast<const uint2*>(dx0 + at);
                acc[i][0] += __uint_as_float(b.x << 16);
                acc[i][1] += __uint_as_float(b.x & 0xffff0000u);
                acc[i][2] += __uint_as_float(b.y << 16);
                acc[i][3] += __uint_as_float(b.y & 0xffff0000u);
            }
            const __nv_bfloat162 lo = __floats2bfloat162_rn(acc[i][0], acc[i][1]), hi = __floats2bfloat162_rn(acc[i][2], acc[i][3]);
            *reinterpret_cast<uint2*>(dx + at) = make_uint2(*reinterpret_cast<const uint32_t*>(&lo), *reinterpret_cast<const uint32_t*>(&hi));
        }
        return;
    }
    const int b = blockIdx.x - dx_blocks, ht = H / kDirH;
    const int h = b % ht * kDirH + (tid & 15) * 4, e0 = b / ht * kDirE, slice = tid >> 4;
    float* sd = sm_f;                                     // [128][16], then the slices' sums [16][16][64]
    float acc[kDirE][4] = {};
    float dsum = 0.0f;
    for (int c0 = 0; c0 < T; c0 += kDirChunk) {
        uint2 xv[kDirChunk / 16];
#pragma unroll
        for (int i = 0; i < kDirChunk / 16; ++i) {
            const int t = c0 + slice + 16 * i;
            xv[i] = t < T ? *reinterpret_cast<const uint2*>(x + static_cast<int64_t>(t) * H + h) : make_uint2(0u, 0u);
        }
#pragma unroll
        for (int i = 0; i < kDirChunk * kDirE / 256; ++i) {
            const int j = tid + 256 * i, t = c0 + j / kDirE, e = e0 + j % kDirE;
            sd[j] = t < T && e < E ? dl[static_cast<int64_t>(t) * E + e] : 0.0f;
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < kDirChunk / 16; ++i) {
            const float xx[4] = {__uint_as_float(xv[i].x << 16), __uint_as_float(xv[i].x & 0xffff0000u),
                                 __uint_as_float(xv[i].y << 16), __uint_as_float(xv[i].y & 0xffff0000u)};
            const float* d = sd + (slice + 16 * i) * kDirE;
#pragma unroll
            for (int e = 0; e < kDirE; e += 4) {
                const float4 f = *reinterpret_cast<const float4*>(d + e);
                const float ff[4] = {f.x, f.y, f.z, f.w};
#pragma unroll
                for (int j = 0; j < 4; ++j)
#pragma unroll
                    for (int c = 0; c < 4; ++c) acc[e + j][c] = fmaf(ff[j], xx[c], acc[e + j][c]);
            }
            dsum += d[tid & 15];
        }
        __syncthreads();
    }
#pragma unroll
    for (int e = 0; e < kDirE; ++e)
        *reinterpret_cast<float4*>(sm_f + (slice * kDirE + e) * kDirH + (tid & 15) * 4) = make_float4(acc[e][0], acc[e][1], acc[e][2], acc[e][3]);
    __syncthreads();
    {
        // the slices of (expert tid / 16, four columns)
        const int e = tid >> 4, col = (tid & 15) * 4;
        float4 s = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            const float4 v = *reinterpret_cast<const float4*>(sm_f + (i * kDirE + e) * kDirH + col);
            s.x += v.x; s.y += v.y; s.z += v.z; s.w += v.w;
        }
        if (e0 + e < E) {
            const int64_t at = static_cast<int64_t>(e0 + e) * H + h;
            if (dWg0) {
                const float4 v = *reinterpret_cast<const float4*>(dWg0 + at);
                s.x += v.x; s.y += v.y; s.z += v.z; s.w += v.w;
            }
            *reinterpret_cast<float4*>(dWg + at) = s;
        }
    }
    if (b % ht == 0) {
        __syncthreads();
        sm_f[tid] = dsum;                                 // [slice][expert]
        __syncthreads();
        if (tid < kDirE && e0 + tid < E) {
            float s = 0.0f;
#pragma unroll
            for (int i = 0; i < 16; ++i) s += sm_f[i * kDirE + tid];
            db[e0 + tid] = s + (db0 ? db0[e0 + tid] : 0.0f);
        }
    }
}

// ---------------------------------------------------------------- workspace and launches
struct RbPlan {
    bool pair;
    int rows, cols, htiles, etiles, chunks;
    int U;
    int most_groups;      // partial tiles: htiles * etiles + groups
};

RbPlan plan_of(int T, int H, int E) {
    RbPlan p;
    p.pair = E > 128;
    p.rows = p.pair ? 256 : 128;
    p.cols = p.pair ? 256 : E <= 16 ? 16 : E <= 32 ? 32 : E <= 64 ? 64 : 128;
    p.htiles = (H + p.rows - 1) / p.rows;
    p.etiles = (E + p.cols - 1) / p.cols;
    p.chunks = (T + kRbChunk - 1) / kRbChunk;
    p.U = p.htiles * p.etiles * p.chunks;      // below 2^31: T is below 2^24
    p.most_groups = p.pair ? 80 : 160;
    return p;
}

struct RbWs {
    uint16_t* w2;        // W_g in two bf16 parts [2][E][H]
    uint16_t* parts;     // dl in bf16 parts: [3][T][ld] (pairs), else [T][3][pitch]
    float* dbpart;
    float* part;
    size_t total;
};

RbWs carve_router(int T, int H, int E, void* base) {
    RbWs w;
    const size_t ld = (E + 7) / 8 * 8;
    const RbPlan pl = plan_of(T, H, E);
    uint8_t* p = static_cast<uint8_t*>(base);
    size_t off = 0;
    auto take = [&](size_t bytes) {
        uint8_t* r = p ? p + off : nullptr;
        off += (bytes + 255) / 256 * 256;
        return r;
    };
    w.w2 = reinterpret_cast<uint16_t*>(take(4ull * E * H));
    w.parts = reinterpret_cast<uint16_t*>(take(6ull * T * (pl.pair ? ld : pl.cols)));
    w.dbpart = reinterpret_cast<float*>(take(4ull * ((T + kPrepTokens - 1) / kPrepTokens) * E));
    w.part = reinterpret_cast<float*>(take(4ull * (static_cast<size_t>(pl.htiles) * pl.etiles + pl.most_groups) * pl.rows * pl.cols));
    w.total = off;
    return w;
}

// [depth][rows][cols] of bf16 values, rows ld apart, boxes of 64 columns x by rows, 128-byte swizzle.
bool make_map16(CUtensorMap* m, const void* base, int64_t cols, int64_t rows, int depth, int64_t ld, int by,
                int dims_n) {
    EncodeTiledFn fn = tensor_map_encoder();
    if (!fn) return false;
    const cuuint64_t dims[3] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(rows), static_cast<cuuint64_t>(depth)};
    const cuuint64_t strides[2] = {static_cast<cuuint64_t>(2 * ld), static_cast<cuuint64_t>(2 * ld * rows)};
    const cuuint32_t box[3] = {64, static_cast<cuuint32_t>(by), 1};
    const cuuint32_t es[3] = {1, 1, 1};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, dims_n, const_cast<void*>(base),
              dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
              CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Up to 512 tokens and 2^25 products of either kind the one launch wins. Measured on a B200 (us, replayed; direct /
// tensor cores): 256 x 512 x 8 4.8 / 14.7, 256 x 2048 x 64 (2^25) 7.6 / 15.9, 512 x 4096 x 64 (2^27) 24.6 / 17.5,
// 4096 x 512 x 16 (2^25) 49 / 22.
bool use_direct(int T, int H, int E) { return T <= 512 && static_cast<int64_t>(T) * H * E <= (1ll << 25); }

cudaError_t launch_direct(const uint16_t* x, const float* Wg, const float* dl, int T, int H, int E, const uint16_t* dx0,
                          const float* dWg0, const float* db0, uint16_t* dx, float* dWg, float* db, cudaStream_t s) {
    auto kern = dx0 ? router_direct_kernel<true> : router_direct_kernel<false>;
    const int smem = sizeof(float) * std::max(E * kDirTok, 16 * kDirE * kDirH);
    const cudaError_t err = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (err != cudaSuccess) return err;
    const int dx_blocks = (T + kDirTok - 1) / kDirTok * ((H + kDirCols - 1) / kDirCols);
    const int dw_blocks = H / kDirH * ((E + kDirE - 1) / kDirE);
    return launch_dependent(kern, dim3(dx_blocks + dw_blocks), dim3(256), smem, s, x, Wg, dl, T, H, E, dx_blocks, dx0, dWg0, db0,
                            dx, dWg, db);
}

template <bool PAIR, int KB, int WB, int AS, int NB>
cudaError_t launch_products(const CUtensorMap (&m)[6], const RouterArgs& g, int groups, cudaStream_t s) {
    auto kern = router_products_kernel<PAIR, KB, WB, AS, NB>;
    const size_t smem = sizeof(SmemP<KB, WB, AS, NB>) + 1024;
    cudaError_t err = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
    if (err != cudaSuccess) return err;
    // a setmaxnreg.inc can only draw on what the block was launched with: refuse a build with less
    cudaFuncAttributes fa;
    if ((err = cudaFuncGetAttributes(&fa, kern)) != cudaSuccess) return err;
    if (fa.numRegs * kRbThreads < kDwRegsSplit) return cudaErrorInvalidConfiguration;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = 2;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.gridDim = dim3(PAIR ? 2 * groups : groups);
    cfg.blockDim = dim3(kRbThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = PAIR ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kern, m[0], m[1], m[2], m[3], m[4], m[5], g);
}

moe_status_t check_router(int T, int H, int E) {
    if (T < 0 || H <= 0 || E <= 0) return MOE_ERR_INVALID_ARG;
    if (H % kGroup || H > 16384 || E > MOE_MAX_EXPERTS || T >= (1 << 24)) return MOE_ERR_UNSUPPORTED_SHAPE;
    return MOE_OK;
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }
bool ptr_ok(const void* p) { return p != nullptr && aligned16(p); }

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" {

size_t moe_router_backward_workspace_size(int T, int H, int E) {
    if (check_router(T, H, E) != MOE_OK) return 0;
    return carve_router(T, H, E, nullptr).total;
}

moe_status_t moe_router_backward(int T, int H, int E, const void* x, const float* Wg, const float* dlogits,
                                 const void* dx0, const float* dWg0, const float* db0, void* dx, float* dWg, float* db,
                                 void* ws, size_t ws_bytes, void* stream) {
    moe_status_t st = check_router(T, H, E);
    if (st != MOE_OK) return st;
    if (T > 0 && (!ptr_ok(x) || !ptr_ok(Wg) || !ptr_ok(dlogits) || !ptr_ok(dx))) return MOE_ERR_INVALID_ARG;
    if (!aligned16(dx0) || !aligned16(dWg0) || !aligned16(db0) || !ptr_ok(dWg) || !ptr_ok(db) || !ptr_ok(ws) ||
        (reinterpret_cast<uintptr_t>(ws) & 255))
        return MOE_ERR_INVALID_ARG;
    const RbWs w = carve_router(T, H, E, ws);
    if (ws_bytes < w.total) return MOE_ERR_WORKSPACE_TOO_SMALL;
    int num_sms, *status;
    if ((st = current_device(&num_sms, &status)) != MOE_OK) return st;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const RbPlan p = plan_of(T, H, E);
    const int ld = (E + 7) / 8 * 8, db_blocks = (T + kPrepTokens - 1) / kPrepTokens;
    auto ok = [](cudaError_t e) { return e == cudaSuccess; };
    if (T > 0 && use_direct(T, H, E))
        return ok(launch_direct(static_cast<const uint16_t*>(x), Wg, dlogits, T, H, E, static_cast<const uint16_t*>(dx0), dWg0, db0,
                                static_cast<uint16_t*>(dx), dWg, db, s))
                   ? MOE_OK
                   : MOE_ERR_CUDA;
    TileGroups tg = {};
    if (T > 0) {
        CUtensorMap m[6];
        // dl's parts: three planes of T rows (pairs), or side by side in each row
        const int width = p.pair ? ld : p.cols, ts = p.cols <= 64 ? 128 : 64;
        const int64_t row = p.pair ? ld : 3 * p.cols, part = p.pair ? static_cast<int64_t>(T) * ld : p.cols;
        const int w_blocks = static_cast<int>((static_cast<int64_t>(E) * H + kPrepW - 1) / kPrepW);
        const bool vec = E % 4 == 0;
        auto prep = E <= 128   ? (vec ? router_prep_parts_kernel<1, true> : router_prep_parts_kernel<1, false>)
                    : E <= 256 ? (vec ? router_prep_parts_kernel<2, true> : router_prep_parts_kernel<2, false>)
                               : (vec ? router_prep_parts_kernel<4, true> : router_prep_parts_kernel<4, false>);
        if (!ok(launch_dependent(prep, dim3(db_blocks + w_blocks), dim3(256), 0, s, dlogits, Wg, T, H, E, width, row, part, db_blocks,
                                 w.parts, w.dbpart, w.w2)))
            return MOE_ERR_CUDA;
        bool mapped = make_map16(&m[1], w.w2, H, E, 2, H, 64, 3) && make_map16(&m[2], dx0 ? dx0 : dx, H, T, 1, H, 32, 2) &&
                      make_map16(&m[3], dx, H, T, 1, H, 32, 2) && make_map16(&m[4], x, H, T, 1, H, ts, 3);
        if (p.pair)
            mapped = mapped && make_map16(&m[0], w.parts, E, T, 3, ld, 128, 3) && make_map16(&m[5], w.parts, E, T, 3, ld, 64, 3);
        else
            mapped = mapped && make_map16(&m[0], w.parts, row, T, 1, row, 128, 2) && make_map16(&m[5], w.parts, row, T, 1, row, ts, 3);
        if (!mapped) return MOE_ERR_CUDA;
        RouterArgs g;
        g.T = T;
        g.H = H;
        g.E = E;
        g.has_base = dx0 != nullptr;
        const int tok = p.pair ? 256 : 128, panel = E > 256 ? 128 : 256, groups = std::min(p.pair ? num_sms / 2 : num_sms, p.most_groups);
        g.Ux = (H + panel - 1) / panel * ((T + tok - 1) / tok);
        g.Uw = p.U;
        g.Gx = std::min(groups, g.Ux);
        g.Gw = std::min(groups, g.Uw);
        for (int t = 0; t < p.htiles * p.etiles; ++t) {
            tg.first[t] = static_cast<uint8_t>(group_of(g.Uw, g.Gw, t * p.chunks));
            tg.last[t] = static_cast<uint8_t>(group_of(g.Uw, g.Gw, (t + 1) * p.chunks - 1));
        }
        g.etiles = p.etiles;
        g.pitch = p.cols;
        g.part = w.part;
        g.status = status;
        const int used = std::max(g.Gx, g.Gw);
        const cudaError_t err = E <= 64    ? launch_products<false, 2, 4, 4, 3>(m, g, used, s)
                                : E <= 128 ? launch_products<false, 4, 4, 2, 2>(m, g, used, s)
                                : E <= 256 ? launch_products<true, 8, 2, 2, 2>(m, g, used, s)
                                           : launch_products<true, 16, 1, 2, 2>(m, g, used, s);
        if (!ok(err)) return MOE_ERR_CUDA;
    }
    return ok(launch_dependent(router_finish_kernel, dim3((H + 1023) / 1024, E), dim3(256), 0, s, w.part, w.dbpart, tg, H, E, p.rows,
                               p.cols, p.etiles, T > 0 ? 1 : 0, db_blocks, dWg0, db0, dWg, db))
               ? MOE_OK
               : MOE_ERR_CUDA;
}

}  // extern "C"
