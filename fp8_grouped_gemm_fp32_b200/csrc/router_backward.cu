// A dense gradient of the router's logits through its linear layer (logits = x W_g^T + b):
//   dx = dx0 + dl W_g [T, H] bf16,  dWg = dWg0 + dl^T x [E, H] fp32,  db = db0 + sum_t dl.
//
// 4 T H E multiply-adds x 2 against x read once, dx0 read and dx written: at 256 experts the products and the
// traffic cost about the same, so both products run on the tensor cores and dx is bound by its own traffic.
//
//  1. router_prep_w_kernel, router_prep_dl_kernel: fp16 copies for dx, each expert's W_g row scaled by a power
//     of two so that its largest entry lies in [512, 1024), that power moved into dl, then each token's dl row
//     scaled likewise (undone in dx's epilogue); dl in three bf16 parts (8 + 8 + 8 bits, all of fp32) for dWg;
//     partial column sums of dl for db.
//  2. router_dx_kernel: one fp16 product. fp16 keeps 11 bits, so dx is off by about an eighth of the step it
//     is rounded with; bf16 parts would need three products for that. A CTA keeps its W_g panel (all experts x
//     256 columns, or 128 above 256 experts) in shared memory and streams token tiles through it: without that
//     the panels alone would cost more L2 traffic than dx does HBM traffic.
//  3. router_dw_kernel: the transposed product, x^T (rows h) by the parts of dl, both operands read as they
//     lie in memory (MN-major), so E is the MMA's N and a few experts cost little. The tensor cores drop bits
//     when they add to a long sum, so every 128 tokens the sum moves from tensor memory into fp32 registers.
//     The (tile, 128 tokens) units are dealt out evenly; a CTA (pair) leaves one partial tile per tile it
//     touched, at index tile + its own index (unique: both only rise), and
//  4. router_finish_kernel adds the partial tiles in order, and db. No float atomics: results repeat.
#include <cmath>

#include <algorithm>

#include <cuda_fp16.h>

#include "../../include/moe_fp8.h"
#include "common.cuh"

namespace moe {

moe_status_t current_device(int* num_sms, int** status);

namespace {

constexpr uint64_t kRbWaitNs = 4000000000ull;
constexpr int kRbBox = 64 * 64 * 2;            // a 64 x 64 operand box: 8 KB
constexpr int kRbThreads = 384;                // TMA, MMA, two idle warps, eight epilogue warps
constexpr int kPrepTokens = 32;                // tokens of a dl preparation block
constexpr int kRbChunk = 128;                  // tokens summed in tensor memory before promotion

__device__ __forceinline__ uint16_t bf16_bits(float f) { return __bfloat16_as_ushort(__float2bfloat16_rn(f)); }

// 2^(9 - exponent of m), so that m times it lies in [512, 1024), and its inverse; 1 for m = 0, infinite or NaN.
__device__ __forceinline__ float2 pow2_scale(float m) {
    if (!(m > 0.0f) || m > 3.0e38f) return make_float2(1.0f, 1.0f);
    const int e = min(max(9 - ilogbf(m), -100), 100);
    return make_float2(exp2f(static_cast<float>(e)), exp2f(static_cast<float>(-e)));
}

// ---------------------------------------------------------------- 1. preparation
// W_g row e -> fp16, scaled; wscale[e] = the inverse of the scale.
__global__ void __launch_bounds__(256)
router_prep_w_kernel(const float* __restrict__ Wg, int H, uint16_t* __restrict__ wh, float* __restrict__ wscale) {
    __shared__ float sm[8];
    const int64_t base = static_cast<int64_t>(blockIdx.x) * H;
    float m = 0.0f;
    for (int h = threadIdx.x * 4; h < H; h += 1024) {
        const float4 f = *reinterpret_cast<const float4*>(Wg + base + h);
        m = fmaxf(m, fmaxf(fmaxf(fabsf(f.x), fabsf(f.y)), fmaxf(fabsf(f.z), fabsf(f.w))));
    }
    m = warp_max(m);
    if ((threadIdx.x & 31) == 0) sm[threadIdx.x >> 5] = m;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 8; ++i) m = fmaxf(m, sm[i]);
    const float2 sc = pow2_scale(m);
    if (threadIdx.x == 0) wscale[blockIdx.x] = sc.y;
    for (int h = threadIdx.x * 4; h < H; h += 1024) {
        const float4 f = *reinterpret_cast<const float4*>(Wg + base + h);
        const __half2 a = __floats2half2_rn(f.x * sc.x, f.y * sc.x), b = __floats2half2_rn(f.z * sc.x, f.w * sc.x);
        *reinterpret_cast<uint2*>(wh + base + h) =
            make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
    }
}

// dl rows -> fp16 (times the experts' inverse scales, then scaled per token; tscale[t] undoes it), three bf16
// parts [3][T][ld], and the block's column sums. A warp takes a token at a time, lane j experts j, j + 32, ...
__global__ void __launch_bounds__(256)
router_prep_dl_kernel(const float* __restrict__ dl, const float* __restrict__ wscale, int T, int E, int ld,
                      uint16_t* __restrict__ dlh, float* __restrict__ tscale, uint16_t* __restrict__ parts,
                      float* __restrict__ dbpart) {
    constexpr int V = kMaxE / 32;
    __shared__ float sm[8][kMaxE];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int t0 = blockIdx.x * kPrepTokens, t1 = min(t0 + kPrepTokens, T);
    const int64_t plane = static_cast<int64_t>(T) * ld;
    const int nv = (E + 31) / 32;
    float sum[V], w[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
        sum[i] = 0.0f;
        w[i] = i < nv && lane + 32 * i < E ? wscale[lane + 32 * i] : 0.0f;
    }
    for (int t = t0 + warp; t < t1; t += 8) {
        float v[V];
        float m = 0.0f;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int e = lane + 32 * i;
            v[i] = i < nv && e < E ? dl[static_cast<int64_t>(t) * E + e] : 0.0f;
            sum[i] += v[i];
            m = fmaxf(m, fabsf(v[i] * w[i]));
        }
        const float2 sc = pow2_scale(warp_max(m));
        if (lane == 0) tscale[t] = sc.y;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int e = lane + 32 * i;
            if (i < nv && e < E) {
                const int64_t at = static_cast<int64_t>(t) * ld + e;
                dlh[at] = __half_as_ushort(__float2half_rn(v[i] * w[i] * sc.x));
                float r = v[i];
#pragma unroll
                for (int p = 0; p < 3; ++p) {
                    const uint16_t b = bf16_bits(r);
                    parts[p * plane + at] = b;
                    // what is left is exact; an infinite or NaN value is carried by its first part alone
                    r = fabsf(r) <= 3.0e38f ? r - bf16_bits_to_f32(b) : 0.0f;
                }
            }
        }
    }
#pragma unroll
    for (int i = 0; i < V; ++i)
        if (lane + 32 * i < E) sm[warp][lane + 32 * i] = sum[i];
    __syncthreads();
    for (int e = threadIdx.x; e < E; e += 256) {
        float s = 0.0f;
#pragma unroll
        for (int i = 0; i < 8; ++i) s += sm[i][e];
        dbpart[static_cast<int64_t>(blockIdx.x) * E + e] = s;
    }
}

// ---------------------------------------------------------------- 2. dx
// PN columns of H a CTA, KB = 64-expert blocks of the panel (PN x KB x 128 bytes <= 128 KB).
template <int PN>
struct SmemX {
    static constexpr int kStages = 2;
    static constexpr int kPanelBlocks = 4 * 256 / PN;
    uint8_t w[kPanelBlocks][PN * 128];
    uint8_t a[kStages][2 * kRbBox];
    uint8_t stage[8][PN / 128][4096];          // per epilogue warp: 32 rows x 64 columns, bf16
    uint64_t wfull;
    uint64_t full[kStages];
    uint64_t empty[kStages];
    uint64_t tfull[2];
    uint64_t tempty[2];
    uint64_t eload[8];
    uint32_t tmem_base;
    volatile int abort_flag;
};

template <int PN, bool BASE>
__global__ void __launch_bounds__(kRbThreads, 1)
router_dx_kernel(const __grid_constant__ CUtensorMap tm_dl, const __grid_constant__ CUtensorMap tm_w,
                 const __grid_constant__ CUtensorMap tm_in, const __grid_constant__ CUtensorMap tm_out,
                 const float* __restrict__ tscale, int T, int H, int E, int panels, int* status) {
    extern __shared__ uint8_t smem_raw[];
    using SX = SmemX<PN>;
    SX& sm = *reinterpret_cast<SX*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int KB = (E + 63) / 64;
    const int panel = blockIdx.x % panels, n0 = panel * PN;
    // the CTAs of a panel take its token tiles in turn
    const int first = blockIdx.x / panels, step = (gridDim.x - panel + panels - 1) / panels;
    const int tiles = (T + 127) / 128;
    if (threadIdx.x == 0) {
        mbar_init(&sm.wfull, 1);
        for (int s = 0; s < SX::kStages; ++s) { mbar_init(&sm.full[s], 1); mbar_init(&sm.empty[s], 1); }
        for (int i = 0; i < 2; ++i) { mbar_init(&sm.tfull[i], 1); mbar_init(&sm.tempty[i], 8); }
        for (int i = 0; i < 8; ++i) mbar_init(&sm.eload[i], 1);
        sm.abort_flag = 0;
        fence_mbar_init();
    }
    if (warp == 1) { tmem_alloc(&sm.tmem_base, 512); tmem_relinquish(); }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = sm.tmem_base;
    auto fail = [&]() { set_status(status, kStatusTimeout); sm.abort_flag = 1; };

    if (warp == 0) {
        if (lane == 0) {
            if (first < tiles) {
                mbar_arrive_expect_tx(&sm.wfull, KB * PN * 128);
                for (int kb = 0; kb < KB; ++kb)
                    for (int i = 0; i < PN / 64; ++i)
                        tma_load_2d(sm.w[kb] + i * kRbBox, &tm_w, &sm.wfull, n0 + 64 * i, kb * 64);
            }
            uint32_t it = 0;
            bool ok = true;
            for (int tile = first; ok && tile < tiles; tile += step)
                for (int kb = 0; kb < KB; ++kb, ++it) {
                    const int s = it % SX::kStages;
                    if (!mbar_wait(&sm.empty[s], ((it / SX::kStages) & 1) ^ 1, kRbWaitNs)) { fail(); ok = false; break; }
                    mbar_arrive_expect_tx(&sm.full[s], 2 * kRbBox);
                    tma_load_2d(sm.a[s], &tm_dl, &sm.full[s], kb * 64, tile * 128);
                }
        }
    } else if (warp == 1) {
        if (lane == 0 && first < tiles) {
            uint32_t it = 0, ti = 0;
            const uint32_t idesc = f16_idesc(128, PN, false, false, true);
            bool ok = mbar_wait(&sm.wfull, 0, kRbWaitNs);
            if (!ok) fail();
            for (int tile = first; ok && tile < tiles && !sm.abort_flag; tile += step, ++ti) {
                const uint32_t buf = ti & 1, d = tmem + buf * 256;
                if (!mbar_wait(&sm.tempty[buf], ((ti >> 1) & 1) ^ 1, kRbWaitNs)) { fail(); break; }
                for (int kb = 0; kb < KB; ++kb, ++it) {
                    const int s = it % SX::kStages;
                    if (!mbar_wait(&sm.full[s], (it / SX::kStages) & 1, kRbWaitNs)) { fail(); ok = false; break; }
                    tc_fence_after();
                    const uint32_t a0 = smem_u32(sm.a[s]), b0 = smem_u32(sm.w[kb]);
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk)
                        umma_f16(d, sw128_kmajor_desc(a0 + kk * 32), sw128_mnmajor_desc(b0 + kk * 2048, kRbBox), idesc,
                                 kb + kk > 0);
                    umma_commit(&sm.empty[s]);
                }
                if (ok) umma_commit(&sm.tfull[buf]);
            }
        }
    } else if (warp >= 4) {
        constexpr int kSubs = PN / 128;         // 64-column boxes of a warp: its half of the panel
        const int ew = warp - 4, q = warp & 3, half = ew >> 2;
        uint32_t ti = 0;
        for (int tile = first; tile < tiles; tile += step, ++ti) {
            if (sm.abort_flag) break;
            const uint32_t buf = ti & 1;
            const int row0 = tile * 128 + q * 32, col0 = n0 + half * (PN / 2);
            const float sc = row0 + lane < T ? tscale[row0 + lane] : 0.0f;
            if (lane == 0) {
                bulk_wait_read_all();
                if (BASE) {
                    mbar_arrive_expect_tx(&sm.eload[ew], kSubs * 4096);
                    for (int i = 0; i < kSubs; ++i)
                        tma_load_2d(sm.stage[ew][i], &tm_in, &sm.eload[ew], col0 + 64 * i, row0);
                }
            }
            __syncwarp();
            if (!mbar_wait(&sm.tfull[buf], (ti >> 1) & 1, kRbWaitNs)) { fail(); break; }
            tc_fence_after();
            if (BASE && !mbar_wait(&sm.eload[ew], ti & 1, kRbWaitNs)) { fail(); break; }
            const uint32_t taddr = tmem + (static_cast<uint32_t>(q * 32) << 16) + buf * 256 + half * (PN / 2);
#pragma unroll
            for (int i = 0; i < kSubs; ++i) {
                float v[2][32];
                tmem_ld32(taddr + 64 * i, v[0]);
                tmem_ld32(taddr + 64 * i + 32, v[1]);
                tmem_ld_wait();
                if (i == kSubs - 1) {
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&sm.tempty[buf]);
                }
                const uint32_t st = smem_u32(sm.stage[ew][i]) + lane * 128;
#pragma unroll
                for (int p = 0; p < 8; ++p) {
                    const uint32_t at = st + ((p ^ (lane & 7)) << 4);
                    uint32_t b[4] = {0, 0, 0, 0}, o[4];
                    if (BASE)
                        asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(b[0]), "=r"(b[1]), "=r"(b[2]), "=r"(b[3]) : "r"(at) : "memory");
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const int c = (p & 3) * 8 + 2 * j;
                        const float x = fmaf(v[p >> 2][c], sc, __uint_as_float(b[j] << 16));
                        const float y = fmaf(v[p >> 2][c + 1], sc, __uint_as_float(b[j] & 0xffff0000u));
                        const __nv_bfloat162 r = __floats2bfloat162_rn(x, y);
                        o[j] = *reinterpret_cast<const uint32_t*>(&r);
                    }
                    st_shared_v4(at, o[0], o[1], o[2], o[3]);
                }
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
                if (row0 < T)
                    for (int i = 0; i < kSubs; ++i)
                        if (col0 + 64 * i < H) tma_store_2d(&tm_out, sm.stage[ew][i], col0 + 64 * i, row0);
                bulk_commit();
            }
        }
    }
    if (warp >= 4 && lane == 0) bulk_wait_all();
    tc_fence_before();
    __syncthreads();
    if (sm.abort_flag) {
        const uint64_t t0 = globaltimer_ns();
        while (globaltimer_ns() - t0 < 200000) __nanosleep(1000);   // copies and MMAs in flight land
    }
    __syncthreads();
    if (warp == 1) { tc_fence_after(); tmem_dealloc(tmem, 512); }
}

// ---------------------------------------------------------------- 3. partial tiles of dWg^T
// PAIR: 256 rows of H x 256 experts by a CTA pair (128 of each in either CTA); otherwise 128 rows x up to 128
// experts by one CTA. Unit u of U = tiles * chunks is chunk u % chunks of tile u / chunks; group g of G takes
// units [g U / G, (g + 1) U / G).
constexpr int kDwStages = 3;
constexpr int kDwRegsLow = 40, kDwRegsHigh = 232;                          // as in the grouped GEMM:
constexpr int kDwRegsSplit = 128 * kDwRegsLow + 256 * kDwRegsHigh;        // what the launch must have allocated

struct SmemW {
    uint8_t x[kDwStages][2 * kRbBox];          // 64 tokens x 128 columns of x
    uint8_t d[kDwStages][3][2 * kRbBox];       // 64 tokens x 128 experts of each part
    uint64_t full[kDwStages];
    uint64_t empty[kDwStages];
    uint64_t tfull[2];
    uint64_t tempty[2];
    uint32_t tmem_base;
    volatile int abort_flag;
};

__host__ __device__ __forceinline__ int64_t unit_start(int64_t U, int G, int g) { return U * g / G; }
// The group that holds unit u: the largest g with unit_start(g) <= u.
__device__ __forceinline__ int group_of(int64_t U, int G, int64_t u) { return static_cast<int>(((u + 1) * G + U - 1) / U - 1); }

template <bool PAIR>
__global__ void __launch_bounds__(kRbThreads, 1)
router_dw_kernel(const __grid_constant__ CUtensorMap tm_x, const __grid_constant__ CUtensorMap tm_d, int T, int H,
                 int E, int etiles, int64_t U, int G, float* __restrict__ part, int* status) {
    constexpr int kRows = PAIR ? 256 : 128, kCols = PAIR ? 256 : 128;
    extern __shared__ uint8_t smem_raw[];
    SmemW& sm = *reinterpret_cast<SmemW*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = PAIR ? cluster_ctarank() : 0;
    const int grp = PAIR ? static_cast<int>(cluster_id_x()) : static_cast<int>(blockIdx.x);
    const int chunks = (T + kRbChunk - 1) / kRbChunk;
    const int64_t u0 = unit_start(U, G, grp), u1 = unit_start(U, G, grp + 1);
    if (threadIdx.x == 0) {
        for (int s = 0; s < kDwStages; ++s) { mbar_init(&sm.full[s], 1); mbar_init(&sm.empty[s], 1); }
        for (int i = 0; i < 2; ++i) { mbar_init(&sm.tfull[i], 1); mbar_init(&sm.tempty[i], PAIR ? 16 : 8); }
        sm.abort_flag = 0;
        fence_mbar_init();
    }
    if (warp == 1) {
        if constexpr (PAIR) { tmem_alloc_pair(&sm.tmem_base, 512); tmem_relinquish_pair(); }
        else { tmem_alloc(&sm.tmem_base, 512); tmem_relinquish(); }
    }
    tc_fence_before();
    if constexpr (PAIR) cluster_sync(); else __syncthreads();
    tc_fence_after();
    const uint32_t tmem = sm.tmem_base;
    auto fail = [&]() {
        set_status(status, kStatusTimeout);
        sm.abort_flag = 1;
        if constexpr (PAIR) st_shared_cluster_u32(mapa_shared(smem_u32((const void*)&sm.abort_flag), rank ^ 1u), 1u);
    };
    const int ebox = PAIR ? 2 : (E + 63) / 64;       // 64-expert boxes of each part a CTA loads

    if (warp < 4) {
        setmaxnreg_dec<kDwRegsLow>();
        if (warp == 0 && lane == 0) {
            uint32_t it = 0;
            bool ok = true;
            const uint32_t bytes = (PAIR ? 2u : 1u) * (2 + 3 * ebox) * kRbBox;
            for (int64_t u = u0; ok && u < u1; ++u) {
                const int tile = static_cast<int>(u / chunks), t0 = static_cast<int>(u - static_cast<int64_t>(tile) * chunks) * kRbChunk;
                const int h0 = tile / etiles * kRows + static_cast<int>(rank) * 128;
                const int e0 = tile % etiles * kCols + static_cast<int>(rank) * 128;
                for (int t = t0; t < min(t0 + kRbChunk, T); t += 64, ++it) {
                    const int s = it % kDwStages;
                    if (!mbar_wait(&sm.empty[s], ((it / kDwStages) & 1) ^ 1, kRbWaitNs)) { fail(); ok = false; break; }
                    if constexpr (PAIR) {
                        const uint32_t fb = mapa_shared(smem_u32(&sm.full[s]), 0);
                        if (rank == 0) mbar_arrive_expect_tx(&sm.full[s], bytes);
                        for (int i = 0; i < 2; ++i) tma_load_3d_pair(sm.x[s] + i * kRbBox, &tm_x, fb, h0 + 64 * i, t, 0);
                        for (int p = 0; p < 3; ++p)
                            for (int i = 0; i < 2; ++i) tma_load_3d_pair(sm.d[s][p] + i * kRbBox, &tm_d, fb, e0 + 64 * i, t, p);
                    } else {
                        mbar_arrive_expect_tx(&sm.full[s], bytes);
                        for (int i = 0; i < 2; ++i) tma_load_3d(sm.x[s] + i * kRbBox, &tm_x, &sm.full[s], h0 + 64 * i, t, 0);
                        for (int p = 0; p < 3; ++p)
                            for (int i = 0; i < ebox; ++i) tma_load_3d(sm.d[s][p] + i * kRbBox, &tm_d, &sm.full[s], e0 + 64 * i, t, p);
                    }
                }
            }
        } else if (warp == 1 && lane == 0 && rank == 0) {
            uint32_t it = 0, ci = 0;
            bool ok = true;
            const uint32_t idesc = f16_idesc(kRows, PAIR ? 256 : (E + 15) / 16 * 16, true, true, true);
            for (int64_t u = u0; ok && u < u1 && !sm.abort_flag; ++u, ++ci) {
                const int t0 = static_cast<int>(u % chunks) * kRbChunk;
                const uint32_t buf = ci & 1, d = tmem + buf * 256;
                if (!mbar_wait(&sm.tempty[buf], ((ci >> 1) & 1) ^ 1, kRbWaitNs)) { fail(); break; }
                for (int t = t0; t < min(t0 + kRbChunk, T); t += 64, ++it) {
                    const int s = it % kDwStages;
                    if (!mbar_wait(&sm.full[s], (it / kDwStages) & 1, kRbWaitNs)) { fail(); ok = false; break; }
                    tc_fence_after();
                    const uint32_t a0 = smem_u32(sm.x[s]);
#pragma unroll
                    for (int p = 0; p < 3; ++p) {
                        const uint32_t b0 = smem_u32(sm.d[s][p]);
#pragma unroll
                        for (int kk = 0; kk < 4; ++kk) {
                            const uint64_t da = sw128_mnmajor_desc(a0 + kk * 2048, kRbBox);
                            const uint64_t db = sw128_mnmajor_desc(b0 + kk * 2048, kRbBox);
                            const uint32_t acc = t > t0 || p + kk > 0;
                            if constexpr (PAIR) umma_f16_pair(d, da, db, idesc, acc);
                            else umma_f16(d, da, db, idesc, acc);
                        }
                    }
                    if constexpr (PAIR) umma_commit_pair(&sm.empty[s], 0x3); else umma_commit(&sm.empty[s]);
                }
                if (ok) { if constexpr (PAIR) umma_commit_pair(&sm.tfull[buf], 0x3); else umma_commit(&sm.tfull[buf]); }
            }
        }
    } else {
        setmaxnreg_inc<kDwRegsHigh>();
        // promotion: warp = lane quadrant q x half of the experts' columns
        constexpr int kMine = kCols / 2;
        const int q = warp & 3, half = (warp - 4) >> 2;
        const uint32_t tempty0 = PAIR ? mapa_shared(smem_u32(&sm.tempty[0]), 0) : 0u;
        float acc[kMine];
        uint32_t ci = 0;
        for (int64_t u = u0; u < u1; ++u, ++ci) {
            if (sm.abort_flag) break;
            const int tile = static_cast<int>(u / chunks);
            const bool begin = u == u0 || u % chunks == 0, end = u + 1 == u1 || (u + 1) % chunks == 0;
            if (begin) {
#pragma unroll
                for (int i = 0; i < kMine; ++i) acc[i] = 0.0f;
            }
            const uint32_t buf = ci & 1;
            if (!mbar_wait(&sm.tfull[buf], (ci >> 1) & 1, kRbWaitNs)) { fail(); break; }
            tc_fence_after();
            const uint32_t taddr = tmem + (static_cast<uint32_t>(q * 32) << 16) + buf * 256 + half * kMine;
#pragma unroll
            for (int c = 0; c < kMine / 32; ++c) {
                float v[32];
                tmem_ld32(taddr + 32 * c, v);
                tmem_ld_wait();
#pragma unroll
                for (int i = 0; i < 32; ++i) acc[32 * c + i] += v[i];
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
                if (PAIR && rank) mbar_arrive_cluster(tempty0 + buf * static_cast<uint32_t>(sizeof(uint64_t)));
                else mbar_arrive(&sm.tempty[buf]);
            }
            if (end) {
                // partial tile [kCols][kRows]: a warp's store is 32 consecutive rows of one expert
                float* dst = part + (static_cast<int64_t>(tile) + grp) * kCols * kRows + rank * 128 + q * 32 + lane;
                const int ecount = E - tile % etiles * kCols;
#pragma unroll
                for (int i = 0; i < kMine; ++i)
                    if (half * kMine + i < ecount) dst[(half * kMine + i) * kRows] = acc[i];
            }
        }
    }
    tc_fence_before();
    if constexpr (PAIR) cluster_sync(); else __syncthreads();
    if (sm.abort_flag) {
        const uint64_t t0 = globaltimer_ns();
        while (globaltimer_ns() - t0 < 200000) __nanosleep(1000);
    }
    if constexpr (PAIR) cluster_sync(); else __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        if constexpr (PAIR) tmem_dealloc_pair(tmem, 512); else tmem_dealloc(tmem, 512);
    }
}

// ---------------------------------------------------------------- 4. sums of the partial tiles, db
__global__ void __launch_bounds__(256)
router_finish_kernel(const float* __restrict__ part, const float* __restrict__ dbpart, int T, int H, int E, int rows,
                     int cols, int etiles, int chunks, int64_t U, int G, int db_blocks, const float* dWg0,
                     const float* db0, float* dWg, float* db) {
    const int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
    const int64_t n = static_cast<int64_t>(E) * (H / 4);
    if (i < n) {
        const int e = static_cast<int>(i / (H / 4)), h = static_cast<int>(i % (H / 4)) * 4;
        float4 s = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        if (dWg0) s = *reinterpret_cast<const float4*>(dWg0 + static_cast<int64_t>(e) * H + h);
        if (U > 0) {
            const int tile = h / rows * etiles + e / cols;
            const int g0 = group_of(U, G, static_cast<int64_t>(tile) * chunks);
            const int g1 = group_of(U, G, static_cast<int64_t>(tile + 1) * chunks - 1);
            float4 a = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            for (int g = g0; g <= g1; ++g) {
                const float4 p = *reinterpret_cast<const float4*>(
                    part + ((static_cast<int64_t>(tile) + g) * cols + e % cols) * rows + h % rows);
                a.x += p.x; a.y += p.y; a.z += p.z; a.w += p.w;
            }
            s.x += a.x; s.y += a.y; s.z += a.z; s.w += a.w;
        }
        *reinterpret_cast<float4*>(dWg + static_cast<int64_t>(e) * H + h) = s;
    }
    // db: a warp an expert, the first warps of the grid
    const int64_t e = i >> 5;
    if (e < E) {
        const int lane = threadIdx.x & 31;
        double s = 0.0;
        for (int b = lane; b < db_blocks; b += 32) s += dbpart[static_cast<int64_t>(b) * E + e];
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
        if (lane == 0) db[e] = static_cast<float>(s + (db0 ? db0[e] : 0.0));
    }
}

// ---------------------------------------------------------------- workspace and launches
struct RbPlan {
    bool pair;
    int rows, cols, htiles, etiles, chunks;
    int64_t U;
    int most_groups;      // partial tiles: htiles * etiles + groups
};

// Experts above 128 run as CTA pairs: their operand of dl is then read once for 256 columns of x, and 64 KB a
// stage instead of 112 KB cross from L2 for the same MMAs.
RbPlan plan_of(int T, int H, int E) {
    RbPlan p;
    p.pair = E > 128;
    p.rows = p.pair ? 256 : 128;
    p.cols = p.pair ? 256 : 128;
    p.htiles = (H + p.rows - 1) / p.rows;
    p.etiles = (E + p.cols - 1) / p.cols;
    p.chunks = (T + kRbChunk - 1) / kRbChunk;
    p.U = static_cast<int64_t>(p.htiles) * p.etiles * p.chunks;
    p.most_groups = p.pair ? 80 : 160;
    return p;
}

struct RbWs {
    uint16_t* wh;
    float* wscale;
    uint16_t* dlh;
    float* tscale;
    uint16_t* parts;
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
    w.wh = reinterpret_cast<uint16_t*>(take(2ull * E * H));
    w.wscale = reinterpret_cast<float*>(take(4ull * E));
    w.dlh = reinterpret_cast<uint16_t*>(take(2ull * T * ld));
    w.tscale = reinterpret_cast<float*>(take(4ull * T));
    w.parts = reinterpret_cast<uint16_t*>(take(6ull * T * ld));
    w.dbpart = reinterpret_cast<float*>(take(4ull * ((T + kPrepTokens - 1) / kPrepTokens) * E));
    w.part = reinterpret_cast<float*>(take(4ull * (static_cast<size_t>(pl.htiles) * pl.etiles + pl.most_groups) * pl.rows * pl.cols));
    w.total = off;
    return w;
}

// [depth][rows][cols] of 16-bit values, rows ld apart, boxes of 64 columns x by rows, 128-byte swizzle.
bool make_map16(CUtensorMap* m, const void* base, bool bf16, int64_t cols, int64_t rows, int depth, int64_t ld, int by,
                int dims_n) {
    EncodeTiledFn fn = tensor_map_encoder();
    if (!fn) return false;
    const cuuint64_t dims[3] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(rows), static_cast<cuuint64_t>(depth)};
    const cuuint64_t strides[2] = {static_cast<cuuint64_t>(2 * ld), static_cast<cuuint64_t>(2 * ld * rows)};
    const cuuint32_t box[3] = {64, static_cast<cuuint32_t>(by), 1};
    const cuuint32_t es[3] = {1, 1, 1};
    return fn(m, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, dims_n, const_cast<void*>(base),
              dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
              CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int PN, bool BASE>
cudaError_t launch_dx(const CUtensorMap& dl, const CUtensorMap& w, const CUtensorMap& in, const CUtensorMap& out,
                      const float* tscale, int T, int H, int E, int* status, int num_sms, cudaStream_t s) {
    const size_t smem = sizeof(SmemX<PN>) + 1024;
    cudaError_t err = cudaFuncSetAttribute(router_dx_kernel<PN, BASE>, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
    if (err != cudaSuccess) return err;
    const int panels = (H + PN - 1) / PN, tiles = (T + 127) / 128;
    const int64_t grid = std::min<int64_t>(std::max(num_sms, panels), static_cast<int64_t>(panels) * tiles);
    router_dx_kernel<PN, BASE><<<static_cast<int>(grid), kRbThreads, smem, s>>>(dl, w, in, out, tscale, T, H, E, panels, status);
    return cudaGetLastError();
}

template <bool PAIR>
cudaError_t launch_dw(const CUtensorMap& x, const CUtensorMap& d, int T, int H, int E, const RbPlan& p, float* part,
                      int* status, int num_sms, cudaStream_t s, int* groups) {
    auto kern = router_dw_kernel<PAIR>;
    const size_t smem = sizeof(SmemW) + 1024;
    cudaError_t err = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
    if (err != cudaSuccess) return err;
    cudaFuncAttributes fa;
    if ((err = cudaFuncGetAttributes(&fa, kern)) != cudaSuccess) return err;
    if (fa.numRegs * kRbThreads < kDwRegsSplit) return cudaErrorInvalidConfiguration;
    int G = std::min(PAIR ? num_sms / 2 : num_sms, p.most_groups);
    G = static_cast<int>(std::min<int64_t>(G, p.U));
    *groups = G;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    cfg.gridDim = dim3(PAIR ? 2 * G : G);
    cfg.blockDim = dim3(kRbThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 2;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = PAIR ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, kern, x, d, T, H, E, p.etiles, p.U, G, part, status);
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
    int G = 1;
    if (T > 0) {
        router_prep_w_kernel<<<E, 256, 0, s>>>(Wg, H, w.wh, w.wscale);
        router_prep_dl_kernel<<<db_blocks, 256, 0, s>>>(dlogits, w.wscale, T, E, ld, w.dlh, w.tscale, w.parts, w.dbpart);
        if (!ok(cudaGetLastError())) return MOE_ERR_CUDA;
        CUtensorMap m_dl, m_w, m_in, m_out, m_x, m_d;
        if (!make_map16(&m_dl, w.dlh, false, E, T, 1, ld, 128, 2) || !make_map16(&m_w, w.wh, false, H, E, 1, H, 64, 2) ||
            !make_map16(&m_in, dx0 ? dx0 : dx, true, H, T, 1, H, 32, 2) || !make_map16(&m_out, dx, true, H, T, 1, H, 32, 2) ||
            !make_map16(&m_x, x, true, H, T, 1, H, 64, 3) || !make_map16(&m_d, w.parts, true, E, T, 3, ld, 64, 3))
            return MOE_ERR_CUDA;
        cudaError_t err;
        if (E <= 256)
            err = dx0 ? launch_dx<256, true>(m_dl, m_w, m_in, m_out, w.tscale, T, H, E, status, num_sms, s)
                      : launch_dx<256, false>(m_dl, m_w, m_in, m_out, w.tscale, T, H, E, status, num_sms, s);
        else
            err = dx0 ? launch_dx<128, true>(m_dl, m_w, m_in, m_out, w.tscale, T, H, E, status, num_sms, s)
                      : launch_dx<128, false>(m_dl, m_w, m_in, m_out, w.tscale, T, H, E, status, num_sms, s);
        if (!ok(err)) return MOE_ERR_CUDA;
        err = p.pair ? launch_dw<true>(m_x, m_d, T, H, E, p, w.part, status, num_sms, s, &G)
                     : launch_dw<false>(m_x, m_d, T, H, E, p, w.part, status, num_sms, s, &G);
        if (!ok(err)) return MOE_ERR_CUDA;
    }
    const int64_t work = std::max<int64_t>(static_cast<int64_t>(E) * (H / 4), 32ll * E);
    router_finish_kernel<<<static_cast<int>((work + 255) / 256), 256, 0, s>>>(
        w.part, w.dbpart, T, H, E, p.rows, p.cols, p.etiles, p.chunks, p.U, G, db_blocks, dWg0, db0, dWg, db);
    return ok(cudaGetLastError()) ? MOE_OK : MOE_ERR_CUDA;
}

}  // extern "C"
