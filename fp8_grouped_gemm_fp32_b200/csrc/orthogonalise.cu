// Orthogonalised weight updates: X = G / (|G|_F + eps), then `steps` times
//     A = X X^T,  B = b A + c A^2,  X <- a X + B X          (on the shorter side: X^T X where G is tall)
// which drives X's singular values towards one value without a decomposition (Newton-Schulz iteration of the
// matrix sign, in the quintic form), and O = scale X.
//
// All of it is matrix products, and the tensor cores bound it: with s <= l the sides, a step is s^2 l (A: half
// of a symmetric product) + s^3 (A^2, half) + 2 s^2 l flops. One persistent kernel runs every product of every
// step: 256 x 256 tiles of CTA pairs (tcgen05 cta_group::2), or 128 x 128 tiles of single CTAs where there are
// few; K blocks of 64 by TMA in a ring, two accumulators in tensor memory. A tile waits on its own matrix's counter
// only, so the matrices of a batch fill each other's dependencies and the tail of one product overlaps the head of the
// next; symmetric products compute the tiles on and below the diagonal and store each twice, the second time transposed
// (few tiles: all of them).
//
// Precision. Operands are fp16 (11 bits), sums fp32. The iteration multiplies X's small singular directions
// by a, about 3.4, every step, and with them any rounding noise there: fp16 X alone ends up to 10 % off on
// gradients of low rank. The noise grows only through the a X term, since B is near zero on those directions,
// so X is carried as the sum of two fp16 values (22 bits): the first feeds the products, both enter a X in
// the epilogue. That costs no tensor work. X is stored times a power of two near 32 sqrt(l), so that the second value
// keeps its bits at the start, where entries of X are near 1 / sqrt(s l); A and B times 64. With five steps the result is
// closer than the rounding of O to bf16. Directions that G lacks altogether hold nothing but noise, which a^steps
// multiplies: X's own 2^-23 or so of its size, and what the tensor cores drop of the sums over s. For G of rank 1 (random
// factors) the two together stay below the noise of the same iteration in fp32 (10 steps, s = 200, 512, 1024: 0.020, 0.029, 0.055
// against 0.035, 0.056, 0.079; X stored times sqrt(l) alone: 0.060, 0.090, 0.154); at rank 8 the sums leave 0.014, 0.039
// and 0.085 where fp32 leaves 0.016, 0.027 and 0.039.
//
// Large matrices with l >= 1.5 s take their first two steps at once: X_2 = (a I + B_2)(a I + B_1) X_0 with A_2 =
// (a I + B_1)^2 A_1, all in s x s products, 3 s^2 l + 5 s^3 flops instead of 6 s^2 l + 2 s^3 (a fifth to a third
// less for these two). A later pair must not: A_2 then carries A_1's rounding noise, grown by a^2, into directions
// that the products with X would have resolved (2 to 3 times the error); in the first pair it does not show.
//
// Measured on a B200, 5 steps: four of 4096 x 2048 1009 us (1.19 PFLOP/s, symmetric products counted half), 1220 us when
// run on and on under the power cap (1.2 - 1.4 GHz): a K block takes 633 to 709 cycles, its MMAs 512. Sixteen of 256 x 512
// 97 us: 15 products one after another at 6.6 us (12,700 cycles), of which the MMAs of K = 512 at 32 KB a K block take
// 4600, the epilogue 750 (A) to 2200 (update), its stores and their release 2500, the next tile's poll and first loads
// the rest. Plain stores in place of the bulk stores are no faster (the release waits for them as long).
#include <cmath>

#include <algorithm>

#include <cuda_fp16.h>

#include "../../include/moe_fp8.h"
#include "common.cuh"

namespace moe {

moe_status_t current_device(int* num_sms, int** status);

namespace {

constexpr uint64_t kOrthoWaitNs = 4000000000ull;
constexpr int kOK = 64;                      // K values a stage holds: 128 bytes
constexpr int kOStages = 5;
constexpr int kOBox = 64 * kOK * 2;          // one 64 x 64 box of an operand: 8 KB
constexpr int kOOper = 2 * kOBox;            // a CTA's 128 rows of an operand
// "What a tile needs is there", from the producer to the epilogue warps, a barrier a tile in turn. While an epilogue
// warp is at a tile the producer is at most 2 (accumulators) + kOStages (tiles of one K block in the ring) ahead, so a
// barrier is not reused before it was waited for.
constexpr int kOReady = 16;
static_assert(kOReady > kOStages + 3, "a tile's barrier must outlast the tiles in flight");
// "Every epilogue warp has stored its part of a tile", a barrier a counted tile in turn. Only the counting warp waits for
// it, so another may be ahead: of a slow warp at tile n (accumulator released, box not stored) by two tiles at most, since
// tile n + 3's accumulator is computed once every warp has released that of n + 1. One barrier would take a quick
// warp's arrivals of n + 1 and n + 2 for the slow one's and count n while its box is not in memory.
constexpr int kOStored = 4;
static_assert(kOStored >= 3, "a warp may be two tiles ahead of another");
constexpr int kOThreads = 384;               // TMA, MMA, two idle warps, eight epilogue warps
constexpr int kOEpi = 8;
constexpr float kPScale = 64.0f;             // A and B are stored times this
constexpr int kMaxSteps = 32;
// X is stored times 2^kSpareBits and a power of two near sqrt(l), at most 2^7: values stay at 8 2^12 at most, half of what
// fp16 holds, and start near 2^5 / sqrt(s), where the second part keeps its 11 bits.
constexpr int kSpareBits = 5;
constexpr int kDoneStride = 32;              // matrices' counters lie 128 bytes apart: each is polled by many CTAs

struct SmemO {
    uint8_t a[kOStages][kOOper];
    uint8_t b[kOStages][kOOper];
    uint8_t stage[kOEpi][2][4096];           // per epilogue warp: 32 rows x 64 columns of 16-bit values, twice
    uint64_t full[kOStages];
    uint64_t empty[kOStages];
    uint64_t tfull[2];
    uint64_t tempty[2];
    uint64_t eload[kOEpi];
    uint64_t stored[kOStored];
    uint64_t ready[kOReady];
    uint32_t tmem_base;
    volatile int abort_flag;
};

// Tensor maps over a wave's buffers, [matrices][rows][columns] of fp16: operand boxes of 64 x 64 values,
// epilogue boxes of 64 columns x 32 rows and, for transposed stores, 32 columns x 64 rows. hi: both buffers of X's first
// parts, matrix b of buffer i at i * mats + b; sq: the s x s matrices, slot i at i * mats + b.
struct OrthoMaps {
    CUtensorMap hi_op, hi_ep, lo_ep;
    CUtensorMap sq_op, sq_ep, sq_tr;
};

// out = cxy X Y + cu U + cv V on slots of symmetric matrices (u, v: -1 for none; all are stored times 64).
struct OrthoSym {
    int x, y, u, v, out;
    float cxy, cu, cv;
};

// The iteration as groups of products: A (slot 0) from X, then nsym symmetric products, then the update X <- ca X + Q X
// with Q in slot 1. The first group may be two steps in one.
constexpr int kSlots = 6, kMostSym = 5;
struct OrthoArgs {
    int M, N;                // rows and columns of a matrix
    int mats;                // matrices of the wave
    int groups;
    int interleaved;
    int square;              // single CTAs: symmetric products compute every tile (else those on and below the diagonal,
                             // stored twice)
    int nsym0;               // symmetric products of the first group (1 or 5); the others have one
    OrthoSym sym0[kMostSym], sym;
    float ca0, ca;
    float out_scale;         // scale / the power of two X is stored with
    float gram_scale;        // 64 / that power squared
    uint16_t* O;             // the wave's first matrix
    unsigned* done;          // [mats][kDoneStride] finished tiles, counted by every CTA
    int* status;
};

// One tile of one product: matrix b, product 0 = A, 1 .. nsym symmetric, nsym + 1 = the update.
enum OrthoKind { kGram, kSym, kUpdate };
struct OrthoTile {
    int group, b, ti, tj;
    OrthoKind kind;
    const OrthoSym* sym;
};

template <bool PAIR>
struct OrthoShape {
    static constexpr int kEdge = PAIR ? 256 : 128;
    int s, l, nb, rb, cb, ns, nu;     // sides, tiles: symmetric per side, update rows / columns, per product
    bool tall;
    __device__ OrthoShape(const OrthoArgs& g) {
        tall = g.M > g.N;
        s = min(g.M, g.N);
        l = max(g.M, g.N);
        nb = (s + kEdge - 1) / kEdge;
        ns = !PAIR && g.square ? nb * nb : nb * (nb + 1) / 2;
        rb = (g.M + kEdge - 1) / kEdge;
        cb = (g.N + kEdge - 1) / kEdge;
        nu = rb * cb;
    }
};

// Walks this cluster's tiles: products in order, each over all matrices, every `stride`-th tile.
template <bool PAIR>
struct OrthoWalk {
    const OrthoArgs& g;
    const OrthoShape<PAIR>& sh;
    int pos, group, prod, stride;
    int before;                            // tiles of a matrix in the products before this one
    __device__ OrthoWalk(const OrthoArgs& g_, const OrthoShape<PAIR>& sh_, int first, int stride_)
        : g(g_), sh(sh_), pos(first), group(0), prod(0), stride(stride_), before(0) {
        settle();
    }
    __device__ int nsym() const { return group == 0 ? g.nsym0 : 1; }
    __device__ int per_matrix() const { return prod > nsym() ? sh.nu : sh.ns; }
    __device__ void settle() {
        while (group < g.groups && pos >= g.mats * per_matrix()) {
            pos -= g.mats * per_matrix();
            before += per_matrix();
            if (prod > nsym()) { prod = 0; ++group; } else { ++prod; }
        }
    }
    __device__ bool more() const { return group < g.groups; }
    __device__ void next() { pos += stride; settle(); }
    __device__ OrthoTile tile() const {
        OrthoTile t;
        t.group = group;
        t.kind = prod == 0 ? kGram : prod > nsym() ? kUpdate : kSym;
        t.sym = group == 0 ? &g.sym0[t.kind == kSym ? prod - 1 : 0] : &g.sym;
        t.b = pos / per_matrix();
        const int i = pos - t.b * per_matrix();
        if (t.kind == kUpdate) {
            // the shorter side runs fastest: neighbours share the longer operand's panel
            if (sh.tall) { t.ti = i / sh.cb; t.tj = i - t.ti * sh.cb; }
            else { t.tj = i / sh.rb; t.ti = i - t.tj * sh.rb; }
        } else if (!PAIR && g.square) {
            t.ti = i / sh.nb;
            t.tj = i - t.ti * sh.nb;
        } else {
            int r = static_cast<int>((sqrtf(8.0f * i + 1.0f) - 1.0f) * 0.5f);
            while ((r + 1) * (r + 2) / 2 <= i) ++r;
            while (r * (r + 1) / 2 > i) --r;
            t.ti = r;
            t.tj = i - r * (r + 1) / 2;
        }
        return t;
    }
    // Finished tiles (each CTA of a pair counts its half) its matrix needs before this tile may start: all
    // earlier products'.
    __device__ unsigned needs() const { return static_cast<unsigned>(before) * (PAIR ? 2 : 1); }
};

// Whether both operands of a tile are the same rows (a diagonal tile of A or of a square).
__device__ __forceinline__ bool same_rows(const OrthoTile& t) {
    return t.ti == t.tj && (t.kind == kGram || (t.kind == kSym && t.sym->x == t.sym->y));
}

__device__ __forceinline__ uint32_t pack_half2(float x, float y) {
    const __half2 h = __floats2half2_rn(x, y);
    return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ float2 unpack_half2(uint32_t u) {
    return __half22float2(*reinterpret_cast<const __half2*>(&u));
}
__device__ __forceinline__ uint4 ld_shared_v4(uint32_t addr) {
    uint4 v;
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr) : "memory");
    return v;
}

// Row r of matrix m in the caller's array (interleaved: blocks of 128 rows of two matrices in turn).
__device__ __forceinline__ int64_t user_row(int m, int r, int M, int interleaved) {
    if (!interleaved) return static_cast<int64_t>(m) * M + r;
    return static_cast<int64_t>(m >> 1) * 2 * M + (r / kGroup * 2 + (m & 1)) * kGroup + r % kGroup;
}

template <bool PAIR>
__global__ void __launch_bounds__(kOThreads, 1)
ortho_steps_kernel(const __grid_constant__ OrthoMaps maps, const __grid_constant__ OrthoArgs g) {
    extern __shared__ uint8_t smem_raw[];
    SmemO& sm = *reinterpret_cast<SmemO*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    constexpr int kEdge = PAIR ? 256 : 128;
    const uint32_t rank = PAIR ? cluster_ctarank() : 0;
    const OrthoShape<PAIR> sh(g);
    OrthoWalk<PAIR> w(g, sh, static_cast<int>(PAIR ? cluster_id_x() : blockIdx.x),
                      static_cast<int>(PAIR ? cluster_count_x() : gridDim.x));

    if (threadIdx.x == 0) {
        for (int s = 0; s < kOStages; ++s) {
            mbar_init(&sm.full[s], 1);       // the leader arms it with both CTAs' bytes
            mbar_init(&sm.empty[s], 1);      // the commit of the stage's MMAs reaches both CTAs
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&sm.tfull[i], 1);
            mbar_init(&sm.tempty[i], (PAIR ? 2 : 1) * kOEpi);
        }
        for (int i = 0; i < kOEpi; ++i) mbar_init(&sm.eload[i], 1);
        for (int i = 0; i < kOStored; ++i) mbar_init(&sm.stored[i], kOEpi);
        for (int i = 0; i < kOReady; ++i) mbar_init(&sm.ready[i], 1);
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
        set_status(g.status, kStatusTimeout);
        sm.abort_flag = 1;
        if constexpr (PAIR) st_shared_cluster_u32(mapa_shared(smem_u32((const void*)&sm.abort_flag), rank ^ 1u), 1u);
    };
    // Waits until matrix b's counter reaches `need`, then lets later TMA accesses see what was stored before it.
    auto wait_for = [&](int b, unsigned need) -> bool {
        const unsigned* done = g.done + b * kDoneStride;
        if (load_acquire_gpu(done) < need) {
            const uint64_t t0 = globaltimer_ns();
            while (load_acquire_gpu(done) < need) {
                if (sm.abort_flag || globaltimer_ns() - t0 > kOrthoWaitNs) return false;
                __nanosleep(20);
            }
        }
        fence_proxy_async();
        return true;
    };

    if (warp == 0) {
        // ---------------- producer: this CTA's 128 rows of the A operand and its half of the B operand
        if (lane == 0) {
            uint32_t it = 0, ti = 0;
            bool ok = true;
            for (; ok && w.more(); w.next(), ++ti) {
                const OrthoTile t = w.tile();
                if (!wait_for(t.b, w.needs())) { fail(); break; }
                mbar_arrive(&sm.ready[ti % kOReady]);                  // for the epilogue warps' loads of this tile
                // A: X X^T (X^T X); symmetric: X Y of their slots; update: Q X (X Q)
                const int hz = (t.group & 1) * g.mats + t.b;
                const bool a_hi = t.kind == kGram || (t.kind == kUpdate && sh.tall);
                const bool b_hi = t.kind == kGram || (t.kind == kUpdate && !sh.tall);
                const CUtensorMap* ma = a_hi ? &maps.hi_op : &maps.sq_op;
                const CUtensorMap* mb = b_hi ? &maps.hi_op : &maps.sq_op;
                const int za = a_hi ? hz : (t.kind == kUpdate ? 1 : t.sym->x) * g.mats + t.b;
                const int zb = b_hi ? hz : (t.kind == kUpdate ? 1 : t.sym->y) * g.mats + t.b;
                const bool a_mn = t.kind == kGram && sh.tall;
                const bool b_mn = (t.kind == kGram && sh.tall) || (t.kind == kUpdate && !sh.tall);
                const int K = t.kind == kGram ? sh.l : sh.s;
                const bool same = same_rows(t);
                const int ra = t.ti * kEdge + static_cast<int>(rank) * 128, rb = t.tj * kEdge + static_cast<int>(rank) * 128;
                for (int k0 = 0; k0 < K; k0 += kOK, ++it) {
                    const int s = it % kOStages;
                    if (!mbar_wait(&sm.empty[s], ((it / kOStages) & 1) ^ 1, kOrthoWaitNs)) { fail(); ok = false; break; }
                    const uint32_t fb = PAIR ? mapa_shared(smem_u32(&sm.full[s]), 0) : 0u;
                    if (rank == 0) mbar_arrive_expect_tx(&sm.full[s], (PAIR ? 2 : 1) * (same ? 1 : 2) * kOOper);
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const int ya = ra + 64 * i, yb = rb + 64 * i;
                        if constexpr (PAIR) {
                            tma_load_3d_pair(sm.a[s] + i * kOBox, ma, fb, a_mn ? ya : k0, a_mn ? k0 : ya, za);
                            if (!same) tma_load_3d_pair(sm.b[s] + i * kOBox, mb, fb, b_mn ? yb : k0, b_mn ? k0 : yb, zb);
                        } else {
                            tma_load_3d(sm.a[s] + i * kOBox, ma, &sm.full[s], a_mn ? ya : k0, a_mn ? k0 : ya, za);
                            if (!same) tma_load_3d(sm.b[s] + i * kOBox, mb, &sm.full[s], b_mn ? yb : k0, b_mn ? k0 : yb, zb);
                        }
                    }
                }
            }
        }
    } else if (warp == 1) {
        // ---------------- MMA issuer: the leader, for both CTAs
        if (lane == 0 && rank == 0) {
            uint32_t it = 0, ti = 0;
            bool ok = true;
            for (; ok && w.more() && !sm.abort_flag; w.next(), ++ti) {
                const OrthoTile t = w.tile();
                const bool a_mn = t.kind == kGram && sh.tall;
                const bool b_mn = (t.kind == kGram && sh.tall) || (t.kind == kUpdate && !sh.tall);
                const int K = t.kind == kGram ? sh.l : sh.s;
                const bool same = same_rows(t);
                const uint32_t idesc = f16_idesc(kEdge, kEdge, false, a_mn, b_mn);
                const uint32_t a_step = a_mn ? 128 : 2, b_step = b_mn ? 128 : 2;
                const uint32_t buf = ti & 1, d = tmem + buf * kEdge;
                if (!mbar_wait(&sm.tempty[buf], ((ti >> 1) & 1) ^ 1, kOrthoWaitNs)) { fail(); break; }
                tc_fence_after();
                for (int k0 = 0; k0 < K; k0 += kOK, ++it) {
                    const int s = it % kOStages;
                    if (!mbar_wait(&sm.full[s], (it / kOStages) & 1, kOrthoWaitNs)) { fail(); ok = false; break; }
                    tc_fence_after();
                    // 16 K values on (the descriptors hold address / 16): 32 bytes in a K-major row, 16 rows of 128 bytes
                    // of an MN-major box
                    uint64_t da = a_mn ? sw128_mnmajor_desc(smem_u32(sm.a[s]), kOBox) : sw128_kmajor_desc(smem_u32(sm.a[s]));
                    const uint32_t b0 = smem_u32(same ? sm.a[s] : sm.b[s]);
                    uint64_t db = b_mn ? sw128_mnmajor_desc(b0, kOBox) : sw128_kmajor_desc(b0);
#pragma unroll
                    for (int kk = 0; kk < kOK / 16; ++kk, da += a_step, db += b_step) {
                        if constexpr (PAIR) umma_f16_pair(d, da, db, idesc, k0 + kk > 0);
                        else umma_f16(d, da, db, idesc, k0 + kk > 0);
                    }
                    if constexpr (PAIR) umma_commit_pair(&sm.empty[s], 0x3); else umma_commit(&sm.empty[s]);
                }
                if (ok) { if constexpr (PAIR) umma_commit_pair(&sm.tfull[buf], 0x3); else umma_commit(&sm.tfull[buf]); }
            }
        }
    } else if (warp >= 4) {
        // ---------------- epilogue: warp = lane quadrant q x column half; 64 columns at a time through its stage
        const int ew = warp - 4, q = warp & 3, half = ew >> 2;
        const uint32_t st0 = smem_u32(sm.stage[ew][0]), st1 = smem_u32(sm.stage[ew][1]);
        const uint32_t tempty0 = PAIR ? mapa_shared(smem_u32(&sm.tempty[0]), 0) : 0u;
        constexpr int kSubs = kEdge / 128;
        uint32_t ti = 0, loads = 0, tiles = 0;
        bool ok = true;
        for (; ok && w.more(); w.next(), ++ti) {
            if (sm.abort_flag) break;
            const OrthoTile t = w.tile();
            const uint32_t buf = ti & 1;
            const int row0 = t.ti * kEdge + static_cast<int>(rank) * 128 + q * 32;
            const bool update = t.kind == kUpdate;
            const int rows = update ? g.M : sh.s, cols = update ? g.N : sh.s;
            const int cur = t.group & 1;
            const bool last = update && t.group == g.groups - 1;
            const bool mirror = !update && t.ti != t.tj && (PAIR || !g.square);
            // what comes in: X's two parts, or a symmetric product's addends
            const bool in0 = update || (t.kind == kSym && t.sym->u >= 0), in1 = update || (t.kind == kSym && t.sym->v >= 0);
            const float ca = t.group == 0 ? g.ca0 : g.ca, inv = 1.0f / kPScale;
            const float cxy = t.kind == kGram ? g.gram_scale : t.sym->cxy, cu = t.sym->cu, cv = t.sym->cv;
#pragma unroll 1
            for (int sub = 0; sub < kSubs; ++sub) {
                const int col0 = t.tj * kEdge + half * (kEdge / 2) + sub * 64;
                // the stage is free once the last stores have read it; then the tile's own values come in
                int good = 1;
                if (lane == 0) {
                    bulk_wait_read_all();
                    if (in0 || in1) {
                        if (sub == 0) {
                            good = mbar_wait(&sm.ready[ti % kOReady], (ti / kOReady) & 1, kOrthoWaitNs);
                            fence_proxy_async();
                        }
                        if (good) {
                            mbar_arrive_expect_tx(&sm.eload[ew], in0 && in1 ? 8192 : 4096);
                            if (in0)
                                tma_load_3d(sm.stage[ew][0], update ? &maps.hi_ep : &maps.sq_ep, &sm.eload[ew], col0, row0,
                                            (update ? cur : t.sym->u) * g.mats + t.b);
                            if (in1)
                                tma_load_3d(sm.stage[ew][1], update ? &maps.lo_ep : &maps.sq_ep, &sm.eload[ew], col0, row0,
                                            (update ? 0 : t.sym->v) * g.mats + t.b);
                        }
                    }
                }
                if (!__shfl_sync(0xffffffffu, good, 0)) { fail(); ok = false; break; }
                if (sub == 0) {
                    if (!mbar_wait(&sm.tfull[buf], (ti >> 1) & 1, kOrthoWaitNs)) { fail(); ok = false; break; }
                    tc_fence_after();
                }
                if (in0 || in1) {
                    if (!mbar_wait(&sm.eload[ew], loads & 1, kOrthoWaitNs)) { fail(); ok = false; break; }
                    ++loads;
                }
                const uint32_t taddr = tmem + (static_cast<uint32_t>(q * 32) << 16) + buf * kEdge + half * (kEdge / 2) + sub * 64;
                float v[2][32];
                tmem_ld32(taddr, v[0]);
                tmem_ld32(taddr + 32, v[1]);
                tmem_ld_wait();
                if (sub == kSubs - 1) {
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) {
                        if (PAIR && rank) mbar_arrive_cluster(tempty0 + buf * static_cast<uint32_t>(sizeof(uint64_t)));
                        else mbar_arrive(&sm.tempty[buf]);
                    }
                }
                // 16-byte piece p (8 columns) of row `lane` sits at p ^ (lane & 7) (128-byte swizzle); four at a time,
                // all of a turn's reads before its writes, which are in place
                auto at = [&](int p) { return static_cast<uint32_t>(lane * 128 + ((p ^ (lane & 7)) << 4)); };
                if (!update) {
#pragma unroll
                    for (int i = 0; i < 64; ++i) v[i >> 5][i & 31] *= cxy;
                    if (in1) {
                        // the second addend first and whole: the transposed box goes over it
#pragma unroll
                        for (int p = 0; p < 8; ++p) {
                            const uint4 r = ld_shared_v4(st1 + at(p));
                            const uint32_t rr[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                const float2 f = unpack_half2(rr[i]);
                                float (&x)[32] = v[p >> 2];
                                x[(p & 3) * 8 + 2 * i] = fmaf(cv, f.x, x[(p & 3) * 8 + 2 * i]);
                                x[(p & 3) * 8 + 2 * i + 1] = fmaf(cv, f.y, x[(p & 3) * 8 + 2 * i + 1]);
                            }
                        }
                        __syncwarp();
                    }
                }
#pragma unroll
                for (int hp = 0; hp < 2; ++hp) {
                    float (&x)[32] = v[hp];
                    uint32_t o[4][4];
                    if (update) {
                        uint4 u[4], r[4];
#pragma unroll
                        for (int p = 0; p < 4; ++p) { u[p] = ld_shared_v4(st0 + at(hp * 4 + p)); r[p] = ld_shared_v4(st1 + at(hp * 4 + p)); }
#pragma unroll
                        for (int p = 0; p < 4; ++p) {
                            const uint32_t uu[4] = {u[p].x, u[p].y, u[p].z, u[p].w}, rr[4] = {r[p].x, r[p].y, r[p].z, r[p].w};
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                const float2 h = unpack_half2(uu[i]), lo = unpack_half2(rr[i]);
                                float& x0 = x[p * 8 + 2 * i];
                                float& x1 = x[p * 8 + 2 * i + 1];
                                const float2 y = __ffma2_rn(make_float2(ca, ca), __fadd2_rn(h, lo),
                                                            __fmul2_rn(make_float2(inv, inv), make_float2(x0, x1)));
                                x0 = y.x;
                                x1 = y.y;
                                if (last) {
                                    const __nv_bfloat162 b2 = __floats2bfloat162_rn(g.out_scale * x0, g.out_scale * x1);
                                    o[p][i] = *reinterpret_cast<const uint32_t*>(&b2);
                                } else {
                                    o[p][i] = pack_half2(x0, x1);
                                }
                            }
                        }
                        if (!last) {
#pragma unroll
                            for (int p = 0; p < 4; ++p) {
                                uint32_t l[4];
#pragma unroll
                                for (int i = 0; i < 4; ++i) {
                                    const float2 h = unpack_half2(o[p][i]);
                                    l[i] = pack_half2(x[p * 8 + 2 * i] - h.x, x[p * 8 + 2 * i + 1] - h.y);
                                }
                                st_shared_v4(st1 + at(hp * 4 + p), l[0], l[1], l[2], l[3]);
                            }
                        }
                    } else {
                        if (in0) {
                            uint4 u[4];
#pragma unroll
                            for (int p = 0; p < 4; ++p) u[p] = ld_shared_v4(st0 + at(hp * 4 + p));
#pragma unroll
                            for (int p = 0; p < 4; ++p) {
                                const uint32_t uu[4] = {u[p].x, u[p].y, u[p].z, u[p].w};
#pragma unroll
                                for (int i = 0; i < 4; ++i) {
                                    const float2 f = unpack_half2(uu[i]);
                                    o[p][i] = pack_half2(fmaf(cu, f.x, x[p * 8 + 2 * i]), fmaf(cu, f.y, x[p * 8 + 2 * i + 1]));
                                }
                            }
                        } else {
#pragma unroll
                            for (int p = 0; p < 4; ++p)
#pragma unroll
                                for (int i = 0; i < 4; ++i) o[p][i] = pack_half2(x[p * 8 + 2 * i], x[p * 8 + 2 * i + 1]);
                        }
                        if (mirror) {
                            // the transposed box: row j (a column here) of 32 values, 64-byte swizzle
#pragma unroll
                            for (int i = 0; i < 32; ++i) {
                                const int j = hp * 32 + i;
                                const uint32_t to = st1 + j * 64 + ((((lane >> 3) ^ (j >> 1)) & 3) << 4) + (lane & 7) * 2;
                                const uint16_t h = static_cast<uint16_t>(o[i >> 3][(i >> 1) & 3] >> (16 * (i & 1)));
                                asm volatile("st.shared.u16 [%0], %1;" ::"r"(to), "h"(h) : "memory");
                            }
                        }
                    }
#pragma unroll
                    for (int p = 0; p < 4; ++p) st_shared_v4(st0 + at(hp * 4 + p), o[p][0], o[p][1], o[p][2], o[p][3]);
                }
                if (last) {
                    // rows leave 16 bytes a lane, eight lanes a row; sizes that are no multiple of 8 by the value, 32 in a row
                    __syncwarp();
                    if (g.N % 8 == 0) {
#pragma unroll 1
                        for (int i = 0; i < 8; ++i) {
                            const int r = i * 4 + (lane >> 3), p = lane & 7;
                            const int grow = row0 + r, gcol = col0 + p * 8;
                            if (grow < rows && gcol < cols)
                                *reinterpret_cast<uint4*>(g.O + user_row(t.b, grow, g.M, g.interleaved) * g.N + gcol) =
                                    ld_shared_v4(st0 + r * 128 + ((p ^ (r & 7)) << 4));
                        }
                    } else {
                        // the 32 rows lie one after another (a block of 128 is one matrix's)
                        uint16_t* dst = g.O + user_row(t.b, row0, g.M, g.interleaved) * g.N + col0;
                        const uint16_t* src = reinterpret_cast<const uint16_t*>(sm.stage[ew][0]);
#pragma unroll 4
                        for (int r = 0; r < 32; ++r) {
#pragma unroll
                            for (int c = lane; c < 64; c += 32)
                                if (row0 + r < rows && col0 + c < cols)
                                    dst[static_cast<int64_t>(r) * g.N + c] = src[r * 64 + (((c >> 3) ^ (r & 7)) << 3) + (c & 7)];
                        }
                    }
                    fence_proxy_async_smem();
                    __syncwarp();
                } else {
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) {
                        if (row0 < rows && col0 < cols) {
                            const int z = (update ? cur ^ 1 : t.kind == kGram ? 0 : t.sym->out) * g.mats + t.b;
                            tma_store_3d(update ? &maps.hi_ep : &maps.sq_ep, sm.stage[ew][0], col0, row0, z);
                            if (update) tma_store_3d(&maps.lo_ep, sm.stage[ew][1], col0, row0, t.b);
                            if (mirror) tma_store_3d(&maps.sq_tr, sm.stage[ew][1], row0, col0, z);
                        }
                        bulk_commit();
                    }
                }
            }
            if (ok && !last) {
                // the tile is in memory once every warp's stores are (a completed bulk store is visible to its
                // thread): one thread counts it for all
                int good = 1;
                if (lane == 0) {
                    bulk_wait_all();
                    mbar_arrive(&sm.stored[tiles % kOStored]);
                    if (ew == 0) {
                        good = mbar_wait(&sm.stored[tiles % kOStored], (tiles / kOStored) & 1, kOrthoWaitNs);
                        if (good) add_release_gpu(g.done + t.b * kDoneStride, 1);
                    }
                }
                ++tiles;
                if (!__shfl_sync(0xffffffffu, good, 0)) { fail(); break; }
            }
        }
    }

    if (warp >= 4 && lane == 0) bulk_wait_all();
    __syncwarp();
    tc_fence_before();
    // neither CTA of a pair leaves while the leader's MMAs may read the other's shared memory
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

// ---------------------------------------------------------------- the norm, and X in two fp16 parts
constexpr int kNormThreads = 256, kNormVals = 8;     // values a thread takes at a time
constexpr int kNormBlocks = 296;

int norm_blocks(int64_t n) {
    return static_cast<int>(std::min<int64_t>(kNormBlocks, (n + kNormThreads * kNormVals - 1) / (kNormThreads * kNormVals)));
}

// Place in the caller's array of value e (below 2^28) of the wave's matrix m (offset from the wave's first matrix).
__device__ __forceinline__ int64_t user_at(uint32_t e, int m, int M, int N, int interleaved) {
    if (!interleaved) return static_cast<int64_t>(m) * M * N + e;
    const uint32_t slab = kGroup * static_cast<uint32_t>(N), q = e / slab;
    return static_cast<int64_t>(m >> 1) * 2 * M * N + (2 * static_cast<int64_t>(q) + (m & 1)) * slab + (e - q * slab);
}

// A thread's eight values of matrix m (n in all) from a block's run of 2048: VEC (rows of whole 16-byte pieces): eight in
// a row from e on, else every 256th.
template <bool VEC>
__device__ __forceinline__ uint32_t first_val(uint32_t run) {
    return run * (kNormThreads * kNormVals) + threadIdx.x * (VEC ? kNormVals : 1);
}
template <bool F32, bool VEC>
__device__ __forceinline__ void load_vals(const void* G, uint32_t e, uint32_t n, int m, int M, int N, int interleaved,
                                          float (&v)[kNormVals]) {
    if constexpr (VEC) {
        const int64_t at = user_at(e, m, M, N, interleaved);
        if constexpr (F32) {
            const float4* p = reinterpret_cast<const float4*>(static_cast<const float*>(G) + at);
            const float4 x = p[0], y = p[1];
            v[0] = x.x; v[1] = x.y; v[2] = x.z; v[3] = x.w; v[4] = y.x; v[5] = y.y; v[6] = y.z; v[7] = y.w;
        } else {
            const uint4 u = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(G) + at);
            const uint32_t uu[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                v[2 * i] = __uint_as_float(uu[i] << 16);
                v[2 * i + 1] = __uint_as_float(uu[i] & 0xffff0000u);
            }
        }
    } else {
#pragma unroll
        for (int i = 0; i < kNormVals; ++i) {
            v[i] = 0.0f;
            if (e + i * kNormThreads < n) {
                const int64_t at = user_at(e + i * kNormThreads, m, M, N, interleaved);
                v[i] = F32 ? static_cast<const float*>(G)[at] : bf16_bits_to_f32(static_cast<const uint16_t*>(G)[at]);
            }
        }
    }
}

__device__ __forceinline__ double block_sum_f64(double v, double* scratch) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    if ((threadIdx.x & 31) == 0) scratch[threadIdx.x >> 5] = v;
    __syncthreads();
    double s = 0.0;
#pragma unroll
    for (int i = 0; i < kNormThreads / 32; ++i) s += scratch[i];
    return s;
}

// Sums of squares in fp64 (fp32 would overflow from 2^64 on and lose small gradients below 2^-63).
template <bool F32, bool VEC>
__global__ void __launch_bounds__(kNormThreads)
ortho_norm_kernel(const void* __restrict__ G, int M, int N, int interleaved, double* __restrict__ part,
                  unsigned* __restrict__ done) {
    __shared__ double scratch[kNormThreads / 32];
    const int m = blockIdx.y;
    const uint32_t n = static_cast<uint32_t>(M) * N;
    dependents_may_launch();
    wait_for_producers();
    if (blockIdx.x == 0 && threadIdx.x == 0) done[m * kDoneStride] = 0;
    double s = 0.0;
    for (uint32_t run = blockIdx.x, e; (e = first_val<VEC>(run)) < n; run += gridDim.x) {
        float v[kNormVals];
        load_vals<F32, VEC>(G, e, n, m, M, N, interleaved, v);
#pragma unroll
        for (int i = 0; i < kNormVals; ++i) s = fma(static_cast<double>(v[i]), static_cast<double>(v[i]), s);
    }
    s = block_sum_f64(s, scratch);
    if (threadIdx.x == 0) part[static_cast<int64_t>(m) * gridDim.x + blockIdx.x] = s;
}

template <bool F32, bool VEC>
__global__ void __launch_bounds__(kNormThreads)
ortho_convert_kernel(const void* __restrict__ G, int M, int N, int ldx, int interleaved, const double* __restrict__ part,
                     double eps, double xscale, uint16_t* __restrict__ hi, uint16_t* __restrict__ lo) {
    __shared__ double scratch[kNormThreads / 32];
    const int m = blockIdx.y;
    const uint32_t n = static_cast<uint32_t>(M) * N;
    wait_for_producers();
    double s = 0.0;
    for (int i = threadIdx.x; i < static_cast<int>(gridDim.x); i += kNormThreads) s += part[static_cast<int64_t>(m) * gridDim.x + i];
    s = block_sum_f64(s, scratch);
    const double inv = xscale / (sqrt(s) + eps);
    const int64_t base = static_cast<int64_t>(m) * M * ldx;
    for (uint32_t run = blockIdx.x, e; (e = first_val<VEC>(run)) < n; run += gridDim.x) {
        float v[kNormVals];
        load_vals<F32, VEC>(G, e, n, m, M, N, interleaved, v);
        alignas(16) uint16_t h[kNormVals], r[kNormVals];
#pragma unroll
        for (int i = 0; i < kNormVals; ++i) {
            // in fp64: 1 / norm of a tiny gradient is outside fp32
            const float x = static_cast<float>(v[i] * inv);
            const __half a = __float2half_rn(x);
            h[i] = __half_as_ushort(a);
            r[i] = __half_as_ushort(__float2half_rn(x - __half2float(a)));
        }
        if constexpr (VEC) {
            *reinterpret_cast<uint4*>(hi + base + e) = *reinterpret_cast<const uint4*>(h);
            *reinterpret_cast<uint4*>(lo + base + e) = *reinterpret_cast<const uint4*>(r);
        } else {
#pragma unroll
            for (int i = 0; i < kNormVals; ++i)
                if (e + i * kNormThreads < n) {
                    const uint32_t row = (e + i * kNormThreads) / N, col = e + i * kNormThreads - row * N;
                    const int64_t at = base + static_cast<int64_t>(row) * ldx + col;
                    hi[at] = h[i];
                    lo[at] = r[i];
                }
        }
    }
}

// ---------------------------------------------------------------- a shorter side of at most 128
// Here a step's products are small and the way between them is the time, so one launch does everything and only X
// crosses between CTAs, once a step. Each CTA owns 128 columns of Y (X, or X^T where G is tall: s rows, l columns), in
// fp32 registers, with their fp16 values as an MMA operand in shared memory; it computes A over all of Y itself (all
// CTAs of a matrix the same bits: one order of K blocks), then B, in shared memory too, and its columns of the update.
// The first exchange is the partial sums of |G|^2. Measured on a B200 (us in turn, graphs of ten calls, against the kernel
// above with its two preparing launches): 64 x 64 28 / 56, 148 of them 31 / 129, 8 of 128 x 256 52 / 79, 2 of 100 x 1000
// 70 / 101, 128 x 4096 158 / 165, 64 of 128 x 512 119 / 135. A step is 5500 cycles and an exchange 5000 to 7000 more. A
// thread's 64 values of X, 32 words of an operand and the norm's fp64 sums exceed its 168 registers: 310 (fp32) to 406
// (bf16) bytes of spills.
constexpr int kNStages = 5;

struct SmemN {
    uint8_t ring[kNStages][kOOper];      // K blocks of Y: 128 rows x 64 columns
    uint8_t y[2][kOOper];                // this CTA's columns, two blocks of 64
    uint8_t p[2][kOOper];                // 64 A
    uint8_t q[2][kOOper];                // 64 B
    uint64_t full[kNStages], empty[kNStages];
    uint64_t acc[3];                     // A, A^2 and B Y are in tensor memory
    uint64_t norm, p_ready, q_ready, y_ready, y_stored;
    double red[kOEpi];
    double inv;
    uint32_t tmem_base;
    volatile int abort_flag;
};

struct NarrowArgs {
    const void* G;
    int M, N, tiles;                     // tiles: CTAs of a matrix
    int interleaved, steps;
    float a, b, c;
    double eps, xscale;
    float out_scale, gram_scale;
    uint16_t* O;
    double* part;                        // [mats][tiles]
    unsigned* done;                      // [mats][kDoneStride], zero at the start
    int* status;
};

template <bool F32>
__global__ void __launch_bounds__(kOThreads, 1)
ortho_narrow_kernel(const __grid_constant__ CUtensorMap tm_y, const __grid_constant__ NarrowArgs g) {
    extern __shared__ uint8_t smem_raw[];
    SmemN& sm = *reinterpret_cast<SmemN*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int m = blockIdx.x / g.tiles, own = blockIdx.x % g.tiles, mats = gridDim.x / g.tiles;
    const bool tall = g.M > g.N;
    const int s = min(g.M, g.N), l = max(g.M, g.N);
    if (threadIdx.x == 0) {
        for (int i = 0; i < kNStages; ++i) { mbar_init(&sm.full[i], 1); mbar_init(&sm.empty[i], 1); }
        for (int i = 0; i < 3; ++i) mbar_init(&sm.acc[i], 1);
        mbar_init(&sm.norm, 1);
        mbar_init(&sm.p_ready, kOEpi);
        mbar_init(&sm.q_ready, kOEpi);
        mbar_init(&sm.y_ready, kOEpi);
        mbar_init(&sm.y_stored, kOEpi);
        sm.abort_flag = 0;
        fence_mbar_init();
    }
    if (warp == 1) { tmem_alloc(&sm.tmem_base, 512); tmem_relinquish(); }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = sm.tmem_base;
    unsigned* const done = g.done + m * kDoneStride;
    auto fail = [&]() { set_status(g.status, kStatusTimeout); sm.abort_flag = 1; };
    auto wait_for = [&](unsigned need) -> bool {
        const uint64_t t0 = globaltimer_ns();
        while (load_acquire_gpu(done) < need)
            if (sm.abort_flag || globaltimer_ns() - t0 > kOrthoWaitNs) return false;
        return true;
    };

    if (warp == 0) {
        // ---------------- producer: the other CTAs' columns of Y
        if (lane == 0 && g.tiles > 1) {
            uint32_t it = 0;
            bool ok = true;
            for (int step = 0; ok && step < g.steps; ++step) {
                // counted once for the norm and once for every Y before this step's
                if (!wait_for(static_cast<unsigned>(step + 2) * g.tiles)) { fail(); break; }
                fence_proxy_async();
                for (int kb = 0; kb < 2 * g.tiles; ++kb) {
                    if (kb >> 1 == own) continue;
                    const int st = it % kNStages;
                    if (!mbar_wait(&sm.empty[st], ((it / kNStages) & 1) ^ 1, kOrthoWaitNs)) { fail(); ok = false; break; }
                    mbar_arrive_expect_tx(&sm.full[st], kOOper);
                    tma_load_3d(sm.ring[st], &tm_y, &sm.full[st], kb * 64, 0, (step & 1) * mats + m);
                    ++it;
                }
            }
        }
    } else if (warp == 1) {
        // ---------------- MMA issuer
        if (lane == 0) {
            uint32_t it = 0;
            const uint32_t kk_desc = f16_idesc(128, 128, false, false, false), km_desc = f16_idesc(128, 128, false, false, true);
            bool ok = true;
            for (int step = 0; ok && step < g.steps && !sm.abort_flag; ++step) {
                if (!mbar_wait(&sm.y_ready, step & 1, kOrthoWaitNs)) { fail(); break; }
                tc_fence_after();
                for (int kb = 0; kb < 2 * g.tiles; ++kb) {
                    const bool mine = kb >> 1 == own;
                    const int st = it % kNStages;
                    if (!mine && !mbar_wait(&sm.full[st], (it / kNStages) & 1, kOrthoWaitNs)) { fail(); ok = false; break; }
                    tc_fence_after();
                    const uint64_t d = sw128_kmajor_desc(smem_u32(mine ? sm.y[kb & 1] : sm.ring[st]));
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk) umma_f16(tmem, d + kk * 2, d + kk * 2, kk_desc, kb + kk > 0);
                    if (!mine) {
                        umma_commit(&sm.empty[st]);
                        ++it;
                    }
                }
                if (!ok) break;
                umma_commit(&sm.acc[0]);
                if (!mbar_wait(&sm.p_ready, step & 1, kOrthoWaitNs)) { fail(); break; }
                tc_fence_after();
#pragma unroll
                for (int kb = 0; kb < 2; ++kb) {
                    const uint64_t d = sw128_kmajor_desc(smem_u32(sm.p[kb]));
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk) umma_f16(tmem + 128, d + kk * 2, d + kk * 2, kk_desc, kb + kk > 0);
                }
                umma_commit(&sm.acc[1]);
                if (!mbar_wait(&sm.q_ready, step & 1, kOrthoWaitNs)) { fail(); break; }
                tc_fence_after();
                // B (K-major) times this CTA's Y (MN-major: 64-column blocks of 128 rows)
                const uint64_t dy = sw128_mnmajor_desc(smem_u32(sm.y[0]), kOOper);
#pragma unroll
                for (int kb = 0; kb < 2; ++kb) {
                    const uint64_t d = sw128_kmajor_desc(smem_u32(sm.q[kb]));
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk) umma_f16(tmem + 256, d + kk * 2, dy + (kb * 4 + kk) * 128, km_desc, kb + kk > 0);
                }
                umma_commit(&sm.acc[2]);
            }
        }
    } else if (warp >= 4) {
        // ---------------- the rest: a thread holds row `row`, 64 columns (of Y: col0 ..)
        const int ew = warp - 4, q = warp & 3, half = ew >> 2;
        const int row = q * 32 + lane, col0 = own * 128 + half * 64;
        const uint32_t lanes = static_cast<uint32_t>(q * 32) << 16;
        auto at = [&](int p) { return static_cast<uint32_t>(row * 128 + ((p ^ (row & 7)) << 4)); };
        auto put = [&](uint8_t (*blocks)[kOOper], const uint32_t (&o)[32]) {
            const uint32_t base = smem_u32(blocks[half]);
#pragma unroll
            for (int p = 0; p < 8; ++p) st_shared_v4(base + at(p), o[4 * p], o[4 * p + 1], o[4 * p + 2], o[4 * p + 3]);
        };
        auto arrive = [&](uint64_t* bar) {
            fence_proxy_async_smem();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar);
        };
        // Memory is read and written along the caller's rows, 64 accesses of a lane in flight: those are the lanes where
        // G is tall, else this warp's 32 x 64 values go through shared memory, column c of row r at r * 64 + (c ^ r).
        // The 32 rows of a warp (the 64 of its columns, where tall) lie one after another in the caller's array.
        float* const turn = reinterpret_cast<float*>(sm.p[0]) + ew * 2048;
        const int64_t base = tall ? user_row(m, col0, g.M, g.interleaved) * g.N + row
                                  : user_row(m, q * 32, g.M, g.interleaved) * g.N + col0 + lane;
        auto load = [&](int64_t e) {
            return F32 ? static_cast<const float*>(g.G)[e] : bf16_bits_to_f32(static_cast<const uint16_t*>(g.G)[e]);
        };
        float x[64];
        bool ok = true;
        // Y's tile and the norm
        if (tall) {
#pragma unroll
            for (int i = 0; i < 64; ++i) x[i] = row < s && col0 + i < l ? load(base + static_cast<int64_t>(i) * g.N) : 0.0f;
        } else {
#pragma unroll
            for (int i = 0; i < 64; ++i) {
                const int r = i >> 1, c = 32 * (i & 1);
                x[i] = q * 32 + r < s && col0 + c + lane < l ? load(base + static_cast<int64_t>(r) * g.N + c) : 0.0f;
            }
#pragma unroll
            for (int i = 0; i < 64; ++i) turn[(i >> 1) * 64 + ((32 * (i & 1) + lane) ^ (i >> 1))] = x[i];
            __syncwarp();
#pragma unroll
            for (int i = 0; i < 64; ++i) x[i] = turn[lane * 64 + (i ^ lane)];
        }
        double sq[4] = {};
#pragma unroll
        for (int i = 0; i < 64; ++i) sq[i & 3] = fma(static_cast<double>(x[i]), static_cast<double>(x[i]), sq[i & 3]);
        double ss = (sq[0] + sq[1]) + (sq[2] + sq[3]);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
        int good = 1;
        if (lane == 0) {
            sm.red[ew] = ss;
            mbar_arrive(&sm.y_stored);
            if (ew == 0) {
                good = mbar_wait(&sm.y_stored, 0, kOrthoWaitNs);
                double t = 0.0;
                for (int i = 0; i < kOEpi; ++i) t += sm.red[i];
                if (good && g.tiles > 1) {
                    g.part[static_cast<int64_t>(m) * g.tiles + own] = t;
                    add_release_gpu(done, 1);
                    good = wait_for(g.tiles);
                    t = 0.0;
                    for (int i = 0; good && i < g.tiles; ++i) t += __ldcg(g.part + static_cast<int64_t>(m) * g.tiles + i);
                }
                sm.inv = g.xscale / (sqrt(t) + g.eps);
                if (good) mbar_arrive(&sm.norm);
            }
        }
        good = __shfl_sync(0xffffffffu, good, 0);
        if (!good || !mbar_wait(&sm.norm, 0, kOrthoWaitNs)) { fail(); ok = false; }
        const double inv = sm.inv;
        if (inv > 1e-30 && inv < 1e30) {
            const float f = static_cast<float>(inv);
#pragma unroll
            for (int i = 0; i < 64; ++i) x[i] *= f;
        } else {                                         // the inverse of such a norm leaves fp32, or is not a number
#pragma unroll
            for (int i = 0; i < 64; ++i) x[i] = static_cast<float>(x[i] * inv);
        }
        // this CTA's Y: operand, and (other CTAs' operand) to memory
        auto publish = [&](int buf, uint32_t phase) -> bool {
            uint32_t o[32];
#pragma unroll
            for (int i = 0; i < 32; ++i) o[i] = pack_half2(x[2 * i], x[2 * i + 1]);
            put(sm.y, o);
            arrive(&sm.y_ready);
            if (g.tiles == 1) return true;
            int fine = 1;
            if (lane == 0) {
                mbar_arrive(&sm.y_stored);               // (behind the fence: the blocks are whole when it completes)
                if (ew == 0) {
                    fine = mbar_wait(&sm.y_stored, phase, kOrthoWaitNs);
                    if (fine) {
                        for (int i = 0; i < 2; ++i)
                            if (own * 128 + 64 * i < l) tma_store_3d(&tm_y, sm.y[i], own * 128 + 64 * i, 0, buf * mats + m);
                        bulk_commit();
                        bulk_wait_all();
                        add_release_gpu(done, 1);
                    }
                }
            }
            return __shfl_sync(0xffffffffu, fine, 0) != 0;
        };
        if (ok && !publish(0, 1)) { fail(); ok = false; }
        const float quad = g.c * (1.0f / kPScale), unit = 1.0f / kPScale;
        for (int step = 0; ok && step < g.steps; ++step) {
            if (sm.abort_flag) break;
            uint32_t o[32];
            if (!mbar_wait(&sm.acc[0], step & 1, kOrthoWaitNs)) { fail(); break; }
            tc_fence_after();
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                float v[32];
                tmem_ld32(tmem + lanes + half * 64 + 32 * h, v);
                tmem_ld_wait();
#pragma unroll
                for (int i = 0; i < 16; ++i) o[16 * h + i] = pack_half2(v[2 * i] * g.gram_scale, v[2 * i + 1] * g.gram_scale);
            }
            put(sm.p, o);
            arrive(&sm.p_ready);
            if (!mbar_wait(&sm.acc[1], step & 1, kOrthoWaitNs)) { fail(); break; }
            tc_fence_after();
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                float v[32];
                tmem_ld32(tmem + lanes + 128 + half * 64 + 32 * h, v);
                tmem_ld_wait();
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    const float2 f = unpack_half2(o[16 * h + i]);
                    o[16 * h + i] = pack_half2(fmaf(g.b, f.x, quad * v[2 * i]), fmaf(g.b, f.y, quad * v[2 * i + 1]));
                }
            }
            put(sm.q, o);
            arrive(&sm.q_ready);
            if (!mbar_wait(&sm.acc[2], step & 1, kOrthoWaitNs)) { fail(); break; }
            tc_fence_after();
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                float v[32];
                tmem_ld32(tmem + lanes + 256 + half * 64 + 32 * h, v);
                tmem_ld_wait();
#pragma unroll
                for (int i = 0; i < 32; ++i) x[32 * h + i] = fmaf(g.a, x[32 * h + i], unit * v[i]);
            }
            if (step + 1 < g.steps && !publish((step + 1) & 1, step & 1)) { fail(); break; }
        }
        if (ok && !sm.abort_flag) {
            auto bits = [&](float f) { return __bfloat16_as_ushort(__float2bfloat16_rn(g.out_scale * f)); };
            if (tall) {
#pragma unroll
                for (int i = 0; i < 64; ++i)
                    if (row < s && col0 + i < l) g.O[base + static_cast<int64_t>(i) * g.N] = bits(x[i]);
            } else {
#pragma unroll
                for (int i = 0; i < 64; ++i) turn[lane * 64 + (i ^ lane)] = x[i];
                __syncwarp();
#pragma unroll
                for (int i = 0; i < 64; ++i) {
                    const int r = i >> 1, c = 32 * (i & 1);
                    if (q * 32 + r < s && col0 + c + lane < l)
                        g.O[base + static_cast<int64_t>(r) * g.N + c] = bits(turn[r * 64 + ((c + lane) ^ r)]);
                }
            }
        }
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    if (sm.abort_flag) {
        const uint64_t t0 = globaltimer_ns();
        while (globaltimer_ns() - t0 < 200000) __nanosleep(1000);   // copies and MMAs in flight land
    }
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

// ---------------------------------------------------------------- workspace and launches
// A wave holds enough matrices to give every CTA pair a tile of the symmetric products, twice over, and never
// fewer than two (one fills the other's waits); a batch is cut into equal waves that use the workspace in turn.
int most_of(int M, int N) {
    const int nb = (std::min(M, N) + 255) / 256, ns = nb * (nb + 1) / 2;
    return std::max(2, (148 + ns - 1) / ns);
}
int wave_of(int mats, int M, int N, int interleaved) {
    const int most = most_of(M, N);
    const int waves = (mats + most - 1) / most;
    int w = (mats + waves - 1) / waves;
    if (interleaved) w = (w + 1) / 2 * 2;            // a wave starts at a first matrix
    return w;
}

// The first two steps at once. Measured on a B200 (us in turn, step by step / merged; graphs of ten calls, and for a second
// on and on under the power cap): two of 2048 x 7168 932 / 824 and 1118 / 991, four of 4096 x 2048 1090 / 1009 and
// 1322 / 1220, one of 2048 x 4096 411 / 403 and 419 / 407, four of 1024 x 2048 253 / 259 and 259 / 259: below 1024 the one
// product more in a row costs what the flops save.
bool merges(int M, int N) { return std::min(M, N) >= 1024 && 2 * std::max(M, N) >= 3 * std::min(M, N); }

struct OrthoWs {
    uint16_t* hi;        // two buffers of X's first parts
    uint16_t* lo;
    uint16_t* sq;        // the slots of s x s matrices
    double* part;
    unsigned* done;
    size_t total;
};

OrthoWs carve_ortho(int wave, int M, int N, void* base) {
    OrthoWs w;
    const size_t ldx = (N + 7) / 8 * 8, s = std::min(M, N), lds = (s + 7) / 8 * 8;
    uint8_t* p = static_cast<uint8_t*>(base);
    size_t off = 0;
    auto take = [&](size_t bytes) {
        uint8_t* r = p ? p + off : nullptr;
        off += (bytes + 255) / 256 * 256;
        return r;
    };
    w.hi = reinterpret_cast<uint16_t*>(take(2 * 2 * wave * M * ldx));
    w.lo = reinterpret_cast<uint16_t*>(take(2 * wave * M * ldx));
    w.sq = reinterpret_cast<uint16_t*>(take(2 * (merges(M, N) ? kSlots : 2) * wave * s * lds));
    w.part = reinterpret_cast<double*>(take(8ull * wave * kNormBlocks));
    w.done = reinterpret_cast<unsigned*>(take(4ull * wave * kDoneStride));
    w.total = off;
    return w;
}

// [mats][rows][cols] of fp16, rows ld values apart, in boxes of bx columns x by rows.
bool make_half_map(CUtensorMap* m, const void* base, int mats, int rows, int cols, int bx, int by) {
    EncodeTiledFn fn = tensor_map_encoder();
    if (!fn) return false;
    const cuuint64_t ld = (cols + 7) / 8 * 8;
    const cuuint64_t dims[3] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(rows), static_cast<cuuint64_t>(mats)};
    const cuuint64_t strides[2] = {2 * ld, 2 * ld * static_cast<cuuint64_t>(rows)};
    const cuuint32_t box[3] = {static_cast<cuuint32_t>(bx), static_cast<cuuint32_t>(by), 1};
    const cuuint32_t es[3] = {1, 1, 1};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3, const_cast<void*>(base), dims, strides, box, es,
              CU_TENSOR_MAP_INTERLEAVE_NONE, bx == 64 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
              CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

moe_status_t check_ortho(int batch, int M, int N, int interleaved) {
    if (batch < 0 || M <= 0 || N <= 0 || (interleaved != 0 && interleaved != 1)) return MOE_ERR_INVALID_ARG;
    if (M > 16384 || N > 16384 || batch > 16384) return MOE_ERR_UNSUPPORTED_SHAPE;
    if (interleaved && M % kGroup) return MOE_ERR_UNSUPPORTED_SHAPE;
    return MOE_OK;
}

// Whether every X and B of the iteration stays inside what fp16 holds: bounds the largest singular value after
// each step from that before it (|a x + b x^3 + c x^5| over [0, r] has its maximum at r or where the derivative
// is zero), and |b x^2 + c x^4| likewise.
// Two steps at once stay inside with them: with r the bound after the first, the odd quintic p is at most r on
// [0, 1] and 8 on [0, r], so by Bernstein's inequality |p(x) / x| is at most 5 pi / 2 r and 5 pi / 2 8 / r there and
// a^2 <= 5 r 40 / r; Q = (a I + B_2)(a I + B_1) - a^2 I is then below 700, times 64 below 2^16 - 2^14.
bool coefficients_ok(int steps, float a, float b, float c) {
    if (!std::isfinite(a) || !std::isfinite(b) || !std::isfinite(c)) return false;
    const double A = a, B = b, C = c;
    double r2 = 1.0;                                   // the largest singular value, squared
    for (int i = 0; i < steps; ++i) {
        auto poly = [&](double u) { return std::abs(A + B * u + C * u * u) * std::sqrt(u); };
        auto gram = [&](double u) { return std::abs(B * u + C * u * u); };
        double top = poly(r2), bmax = gram(r2);
        const double disc = 9.0 * B * B - 20.0 * A * C;
        if (C != 0.0 && disc >= 0.0)
            for (double sgn : {-1.0, 1.0}) {
                const double u = (-3.0 * B + sgn * std::sqrt(disc)) / (10.0 * C);
                if (u > 0.0 && u < r2) top = std::max(top, poly(u));
            }
        if (C == 0.0 && B != 0.0 && -A / (3.0 * B) > 0.0 && -A / (3.0 * B) < r2) top = std::max(top, poly(-A / (3.0 * B)));
        if (C != 0.0 && -B / (2.0 * C) > 0.0 && -B / (2.0 * C) < r2) bmax = std::max(bmax, gram(-B / (2.0 * C)));
        if (!(top <= 8.0) || !(bmax <= 256.0)) return false;
        r2 = std::max(top * top, 1e-30);
    }
    return true;
}

// Tiles of the widest product (the update) of one matrix.
template <bool PAIR>
int tiles_of(int M, int N) {
    constexpr int kEdge = PAIR ? 256 : 128;
    return ((M + kEdge - 1) / kEdge) * ((N + kEdge - 1) / kEdge);
}

// Pair tiles (256 x 256) need half the L2 traffic a product; 128 x 128 tiles of single CTAs quarter a tile's latency
// and spread few tiles over all SMs. Measured on a B200 (us, single / pair), by the update's pair tiles of a wave:
// 2 (256 x 512) 95 / 120, 16 (1024 x 1024) 147 / 185, 32 (16 of 256 x 512) 105 / 126, 32 (1024 x 2048) 179 / 212,
// 64 (2048 x 2048) 290 / 273, 128 (4 of 1024 x 2048) 258 / 246, 128 (2048 x 4096) 459 / 396, 512 (4 of 4096 x 2048)
// 1570 / 1061.
bool use_pairs(int mats, int M, int N) { return static_cast<int64_t>(mats) * tiles_of<true>(M, N) >= 56; }

// Where all tiles of a symmetric product run at once, storing a tile the second time, transposed, costs more than a CTA
// that has nothing else to do computing it. Measured on a B200 (us, twice / all tiles): 256 x 512 92 / 85, 16 of them 104 /
// 99, three of 1001 x 333 134 / 127, 1024 x 1024 152 / 145, 1024 x 2048 185 / 177.
bool use_square(int mats, int side, int num_sms) {
    const int nb = (side + 127) / 128;
    return static_cast<int64_t>(mats) * nb * nb <= num_sms;
}

// The narrow kernel's CTAs all compute A, so a matrix of many of them only where all matrices run at once.
int narrow_tiles(int M, int N) { return (std::max(M, N) + 127) / 128; }
bool use_narrow(int mats, int M, int N) {
    const int t = narrow_tiles(M, N);
    return std::min(M, N) <= 128 && (t <= 4 || static_cast<int64_t>(mats) * t <= 148);
}

struct NarrowWs {
    uint16_t* y;         // two buffers of the wave's Y
    double* part;
    unsigned* done;
    size_t total;
};
constexpr int kNarrowSms = 148;
NarrowWs carve_narrow(int mats, int M, int N, void* base) {
    NarrowWs w;
    const int t = narrow_tiles(M, N);
    const size_t wave = std::min(mats, kNarrowSms / t), s = std::min(M, N), ld = (std::max(M, N) + 7) / 8 * 8;
    uint8_t* p = static_cast<uint8_t*>(base);
    size_t off = 0;
    auto take = [&](size_t bytes) {
        uint8_t* r = p ? p + off : nullptr;
        off += (bytes + 255) / 256 * 256;
        return r;
    };
    w.y = reinterpret_cast<uint16_t*>(take(2 * 2 * wave * s * ld));
    w.part = reinterpret_cast<double*>(take(8 * wave * t));
    w.done = reinterpret_cast<unsigned*>(take(4 * wave * kDoneStride));
    w.total = off;
    return w;
}

// What `mats` matrices need, and what they or any fewer do: equal waves of a large batch may be smaller than a smaller
// batch's one wave, and a short side's kernel goes by the batch.
size_t need_of(int mats, int M, int N, int interleaved) {
    if (use_narrow(mats, M, N)) return carve_narrow(mats, M, N, nullptr).total;
    return carve_ortho(wave_of(mats, M, N, interleaved), M, N, nullptr).total;
}
size_t most_needed(int mats, int M, int N, int interleaved) {
    size_t most = 0;
    if (use_narrow(1, M, N)) {
        const int t = narrow_tiles(M, N);
        most = carve_narrow(t <= 4 ? mats : std::min(mats, kNarrowSms / t), M, N, nullptr).total;
    }
    if (!use_narrow(mats, M, N)) {
        int wave = std::min(mats, most_of(M, N));
        if (interleaved) wave = (wave + 1) / 2 * 2;
        most = std::max(most, carve_ortho(wave, M, N, nullptr).total);
    }
    return most;
}

template <bool F32>
cudaError_t launch_prepare(const void* G, int mats, const OrthoArgs& g, const OrthoWs& w, double eps, double xscale,
                           cudaStream_t s) {
    const dim3 grid(norm_blocks(static_cast<int64_t>(g.M) * g.N), mats), block(kNormThreads);
    const int ldx = (g.N + 7) / 8 * 8;
    const bool vec = g.N % 8 == 0;
    const cudaError_t err = launch_dependent(vec ? ortho_norm_kernel<F32, true> : ortho_norm_kernel<F32, false>, grid, block, 0, s,
                                             G, g.M, g.N, g.interleaved, w.part, w.done);
    if (err != cudaSuccess) return err;
    return launch_dependent(vec ? ortho_convert_kernel<F32, true> : ortho_convert_kernel<F32, false>, grid, block, 0, s, G, g.M,
                            g.N, ldx, g.interleaved, w.part, eps, xscale, w.hi, w.lo);
}

template <bool PAIR>
cudaError_t launch_steps(const OrthoMaps& maps, const OrthoArgs& g, int num_sms, cudaStream_t s) {
    auto kern = ortho_steps_kernel<PAIR>;
    const size_t smem = sizeof(SmemO) + 1024;
    cudaError_t err = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
    if (err != cudaSuccess) return err;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeCooperative;      // blocks wait on one another: all of them or none
    attr[0].val.cooperative = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = 2;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.blockDim = dim3(kOThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    int units = num_sms;                              // blocks, or pairs, that fit on the device at once
    if constexpr (PAIR) {
        static int clusters[64] = {0};
        int dev = 0;
        if ((err = cudaGetDevice(&dev)) != cudaSuccess) return err;
        if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
        units = __atomic_load_n(&clusters[dev], __ATOMIC_RELAXED);
        if (units == 0) {
            cfg.gridDim = dim3(2 * (num_sms / 2));
            cfg.attrs = attr + 1;
            cfg.numAttrs = 1;
            if ((err = cudaOccupancyMaxActiveClusters(&units, kern, &cfg)) != cudaSuccess) return err;
            if (units <= 0) return cudaErrorInvalidConfiguration;
            __atomic_store_n(&clusters[dev], units, __ATOMIC_RELAXED);
        }
    }
    units = static_cast<int>(std::min<int64_t>(units, static_cast<int64_t>(g.mats) * tiles_of<PAIR>(g.M, g.N)));
    cfg.gridDim = dim3(PAIR ? 2 * units : units);
    cfg.attrs = attr;
    cfg.numAttrs = PAIR ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kern, maps, g);
}

template <bool F32>
cudaError_t launch_narrow(NarrowArgs g, const NarrowWs& w, int mats, int num_sms, cudaStream_t s) {
    const size_t smem = sizeof(SmemN) + 1024;
    cudaError_t err = cudaFuncSetAttribute(ortho_narrow_kernel<F32>, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
    if (err != cudaSuccess) return err;
    // every wave at once on the GPU; of interleaved pairs both
    int wave = std::min(mats, std::min(num_sms, kNarrowSms) / g.tiles);
    if (g.interleaved) wave &= ~1;
    if (wave <= 0) return cudaErrorInvalidConfiguration;
    const uint8_t* G = static_cast<const uint8_t*>(g.G);
    uint16_t* const O = g.O;
    for (int m0 = 0; m0 < mats; m0 += wave) {
        const int n = std::min(wave, mats - m0);
        const size_t first = static_cast<size_t>(m0) * g.M * g.N;
        CUtensorMap map;
        if (!make_half_map(&map, w.y, 2 * n, std::min(g.M, g.N), std::max(g.M, g.N), 64, 128)) return cudaErrorInvalidValue;
        g.G = G + first * (F32 ? 4 : 2);
        g.O = O + first;
        if (g.tiles > 1 && (err = cudaMemsetAsync(w.done, 0, 4ull * n * kDoneStride, s)) != cudaSuccess) return err;
        cudaLaunchConfig_t cfg = {};
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeCooperative;      // the CTAs of a matrix wait on one another
        attr[0].val.cooperative = 1;
        cfg.gridDim = dim3(n * g.tiles);
        cfg.blockDim = dim3(kOThreads);
        cfg.dynamicSmemBytes = smem;
        cfg.stream = s;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        if ((err = cudaLaunchKernelEx(&cfg, ortho_narrow_kernel<F32>, map, g)) != cudaSuccess) return err;
    }
    return cudaSuccess;
}

bool ptr_ok(const void* p) { return p != nullptr && (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" {

size_t moe_orthogonalise_workspace_size(int batch, int M, int N, int interleaved) {
    if (check_ortho(batch, M, N, interleaved) != MOE_OK || batch == 0) return 0;
    return most_needed(batch * (interleaved ? 2 : 1), M, N, interleaved);
}

moe_status_t moe_orthogonalise(int batch, int M, int N, int interleaved, const void* G, int g_type, int steps, float a,
                               float b, float c, float eps, float scale, void* O, void* ws, size_t ws_bytes,
                               void* stream) {
    moe_status_t st = check_ortho(batch, M, N, interleaved);
    if (st != MOE_OK) return st;
    if (g_type != MOE_TYPE_BF16 && g_type != MOE_TYPE_FP32) return MOE_ERR_INVALID_ARG;
    if (steps <= 0 || steps > kMaxSteps || !coefficients_ok(steps, a, b, c)) return MOE_ERR_INVALID_ARG;
    if (!std::isfinite(eps) || eps < 0.0f || !std::isfinite(scale)) return MOE_ERR_INVALID_ARG;
    if (batch == 0) return MOE_OK;
    if (!ptr_ok(G) || !ptr_ok(O) || !ptr_ok(ws) || (reinterpret_cast<uintptr_t>(ws) & 255)) return MOE_ERR_INVALID_ARG;
    const int mats = batch * (interleaved ? 2 : 1), wave = wave_of(mats, M, N, interleaved);
    const bool narrow = use_narrow(mats, M, N);
    const OrthoWs w = carve_ortho(wave, M, N, ws);
    const NarrowWs nw = carve_narrow(mats, M, N, ws);
    if (ws_bytes < need_of(mats, M, N, interleaved)) return MOE_ERR_WORKSPACE_TOO_SMALL;
    int num_sms, *status;
    if ((st = current_device(&num_sms, &status)) != MOE_OK) return st;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const double xscale = std::exp2(std::floor(0.5 * std::log2(static_cast<double>(std::max(M, N))) + 0.5) + kSpareBits);
    const size_t size = g_type == MOE_TYPE_FP32 ? 4 : 2;
    const int side = std::min(M, N);
    if (narrow) {
        NarrowArgs g;
        g.G = G;
        g.M = M;
        g.N = N;
        g.tiles = narrow_tiles(M, N);
        g.interleaved = interleaved;
        g.steps = steps;
        g.a = a;
        g.b = b;
        g.c = c;
        g.eps = eps;
        g.xscale = xscale;
        g.out_scale = static_cast<float>(scale / xscale);
        g.gram_scale = static_cast<float>(kPScale / (xscale * xscale));
        g.O = static_cast<uint16_t*>(O);
        g.part = nw.part;
        g.done = nw.done;
        g.status = status;
        const cudaError_t err = g_type == MOE_TYPE_FP32 ? launch_narrow<true>(g, nw, mats, num_sms, s)
                                                        : launch_narrow<false>(g, nw, mats, num_sms, s);
        return err == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
    }
    for (int m0 = 0; m0 < mats; m0 += wave) {
        OrthoArgs g;
        g.M = M;
        g.N = N;
        g.mats = std::min(wave, mats - m0);
        g.interleaved = interleaved;
        const bool pairs = use_pairs(g.mats, M, N);
        g.square = !pairs && use_square(g.mats, side, num_sms);
        // slots: 0 A, 1 Q; of two steps in one also 2 B_1, 3 B_1 A, 4 A_2, 5 B_2
        const float f = 1.0f / kPScale;
        const bool two = steps >= 2 && merges(M, N);
        g.sym = {0, 0, 0, -1, 1, c * f, b, 0.0f};
        g.sym0[0] = two ? OrthoSym{0, 0, 0, -1, 2, c * f, b, 0.0f} : g.sym;
        g.sym0[1] = {2, 0, -1, -1, 3, f, 0.0f, 0.0f};
        g.sym0[2] = {2, 3, 0, 3, 4, f, a * a, 2.0f * a};
        g.sym0[3] = {4, 4, 4, -1, 5, c * f, b, 0.0f};
        g.sym0[4] = {5, 2, 2, 5, 1, f, a, a};
        g.nsym0 = two ? kMostSym : 1;
        g.groups = two ? steps - 1 : steps;
        g.ca0 = two ? a * a : a;
        g.ca = a;
        g.out_scale = static_cast<float>(scale / xscale);
        g.gram_scale = static_cast<float>(kPScale / (xscale * xscale));
        const size_t first = static_cast<size_t>(m0) * M * N;
        g.O = static_cast<uint16_t*>(O) + first;
        g.done = w.done;
        g.status = status;
        const void* gw = static_cast<const uint8_t*>(G) + first * size;
        OrthoMaps maps;
        const int slots = merges(M, N) ? kSlots : 2;
        if (!make_half_map(&maps.hi_op, w.hi, 2 * g.mats, M, N, 64, 64) || !make_half_map(&maps.hi_ep, w.hi, 2 * g.mats, M, N, 64, 32) ||
            !make_half_map(&maps.lo_ep, w.lo, g.mats, M, N, 64, 32) ||
            !make_half_map(&maps.sq_op, w.sq, slots * g.mats, side, side, 64, 64) ||
            !make_half_map(&maps.sq_ep, w.sq, slots * g.mats, side, side, 64, 32) ||
            !make_half_map(&maps.sq_tr, w.sq, slots * g.mats, side, side, 32, 64))
            return MOE_ERR_CUDA;
        cudaError_t err = g_type == MOE_TYPE_FP32 ? launch_prepare<true>(gw, g.mats, g, w, eps, xscale, s)
                                                  : launch_prepare<false>(gw, g.mats, g, w, eps, xscale, s);
        if (err == cudaSuccess)
            err = pairs ? launch_steps<true>(maps, g, num_sms, s) : launch_steps<false>(maps, g, num_sms, s);
        if (err != cudaSuccess) return MOE_ERR_CUDA;
    }
    return MOE_OK;
}

}  // extern "C"
