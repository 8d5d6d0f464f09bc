// k_ffn.cu -- the products of the gated feed-forward block and its backward pass on the
// fifth-generation tensor cores:
//     forward    [a | b] = x . W_up^T,  act = silu(a) * b      (one kernel: FFN_UP)
//                y = act . W_down^T
//     backward   d_act = dy . W_down  -> du, act from u         (one kernel: FFN_DACT)
//                dx = du . W_up,  dW_up = du^T . x,  dW_down = dy^T . act
//
// One kernel for all: C[M, N] = A . B^T over K, each operand stored with K contiguous or
// with M (N) contiguous.  A stage of the shared-memory ring holds 128 x 64 of A and
// 128 x 64 of B as four 64 x 64 boxes of 8 KiB that the tensor copy writes in the 128-byte
// swizzle; a box has the contiguous dimension of its operand along its rows, so both
// layouts cost the same copies and differ only in the matrix descriptor (smem_desc_mn) and
// the instruction descriptor's major bits.  No operand is transposed in memory.
// Two shapes: a cluster of two CTAs on a 256 x 256 tile (cta_group::2, each CTA loading
// half of A and half of B), and one CTA on a 128 x 128 tile where M is at most 128.
// Everything outside a tensor is read as zero by the tensor copies (ragged M, N and K) and
// never stored.
//
// Few tiles, long K: the K range is cut into `splits` and every (tile, split) is a work
// item; partial sums go to an f32 workspace and k_join adds them in a fixed order and
// applies the epilogue (see plan()).
//
// Warp roles: 0 copies, 1 issues MMAs into one of two TMEM accumulators, the others are the
// epilogue.  Every wait is bounded; one that gives up raises an error flag and the CTA
// drains its copies and MMAs, frees its TMEM and returns.
#include <algorithm>
#include <mutex>

#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_bf16.h>

#include "common.cuh"
#include "launch.h"
#include "tcgen05.cuh"
#include "train.h"

namespace sol {
namespace ffn {

constexpr int BM = 128;                    // accumulator rows per CTA
constexpr int BK = 64;                     // K per stage
constexpr int UK = 16;                     // K of one tcgen05.mma
constexpr int BOX = 64;                    // a box is BOX x BOX
constexpr int BOX_BYTES = BOX * BOX * 2;   // 8 KiB
constexpr int OP_BYTES = 2 * BOX_BYTES;    // one operand of a stage
constexpr int STAGE_BYTES = 2 * OP_BYTES;  // 32 KiB
constexpr int STAGES = 7;
constexpr int GROUP_M = 16;                // m-blocks per raster group (L2 reuse)
constexpr int EPI_WARP0 = 2;
constexpr uint32_t kWaitLimit = 4096;      // polls of <= ~1 ms each
constexpr uint32_t kPollLimit = 1u << 26;  // polls without a suspend hint
constexpr int B200_SMS = 148;              // plan() is a function of the sizes alone

enum Mode : int { STORE = FFN_STORE, UP = FFN_UP, DACT = FFN_DACT, PART = 3 };

template <bool PAIR> __host__ __device__ constexpr int tile_m() { return PAIR ? 2 * BM : BM; }
template <bool PAIR> __host__ __device__ constexpr int tile_n() { return PAIR ? 256 : 128; }

// Epilogue warps: four (one per TMEM lane quarter) where the epilogue only stores, eight
// where it also computes (two per quarter, half of the columns each).
__host__ __device__ constexpr int epi_warps(int mode) { return mode == UP || mode == DACT ? 8 : 4; }
__host__ __device__ constexpr int block_threads(int mode) { return 64 + 32 * epi_warps(mode); }

struct Bars {
    uint64_t full[STAGES], empty[STAGES], acc_full[2], acc_empty[2], drain;
    int32_t peer_last[STAGES];  // leader: phase of the peer's last copy per stage (-1: none)
    uint32_t tmem_base;
    volatile int32_t abort;
};
constexpr size_t kSmemBytes = 1024 + (size_t)STAGES * STAGE_BYTES + sizeof(Bars);

__device__ uint32_t g_error;

struct Params {
    int32_t M, N, kblocks;       // N: columns of the output (UP: inner)
    int32_t tiles_m, tiles_n;
    int32_t splits, kb_split;    // K cut into `splits` ranges of kb_split blocks (the last may be shorter)
    int64_t items;               // tiles_m * tiles_n * splits
    void* out;
    int64_t ld_out;
    int32_t out_f32, accumulate;
    bf16* u;
    int64_t ld_u;
    bf16* du;
    int64_t ld_du;
    float* partial;              // [splits, M, N]
};

// Shared-memory descriptor of an operand tile with M (N) contiguous, in boxes of 64
// (M) x 64 (K): a box is 64 rows (one K each) of 128 bytes, eight rows to a 1024-byte
// swizzle atom.  Leading byte offset: from one 64-wide box to the next along M (8 KiB);
// stride byte offset: from eight K to the next eight (1024 B).
__device__ __forceinline__ uint64_t smem_desc_mn(uint32_t addr)
{
    return (uint64_t)((addr >> 4) & 0x3FFFu) | ((uint64_t)(BOX_BYTES >> 4) << 16) | ((uint64_t)(1024u >> 4) << 32) |
           ((uint64_t)1u << 46) | ((uint64_t)2u << 61);
}

struct Item {
    int32_t m_blk, n_blk, split, kb0, kb1;
};

__device__ __forceinline__ Item item_at(int64_t i, const Params& p)
{
    Item it;
    const int64_t tiles = (int64_t)p.tiles_m * p.tiles_n;
    it.split = (int32_t)(i / tiles);
    const int64_t t = i - it.split * tiles;
    const int32_t per_group = GROUP_M * p.tiles_n;
    const int32_t g = (int32_t)(t / per_group);
    const int32_t gm = min(GROUP_M, p.tiles_m - g * GROUP_M);
    const int32_t local = (int32_t)(t - (int64_t)g * per_group);
    it.m_blk = g * GROUP_M + local % gm;
    it.n_blk = local / gm;
    it.kb0 = it.split * p.kb_split;
    it.kb1 = min(it.kb0 + p.kb_split, p.kblocks);
    return it;
}

struct Where {
    uint32_t rank;
    int64_t worker, n_workers;
};

template <bool PAIR> __device__ __forceinline__ bool wait_or_abort(uint32_t bar, uint32_t parity, Bars* b)
{
    const uint32_t limit = PAIR ? kPollLimit : kWaitLimit;
    for (uint32_t i = 0; i < limit; ++i) {
        if (PAIR ? tc::mbar_poll_cluster(bar, parity) : mbar_try_wait(bar, parity)) return true;
        if ((i & 15u) == 15u && b->abort) return false;
    }
    return false;
}

__device__ __forceinline__ void raise_abort(Bars* b, uint32_t code)
{
    b->abort = 1;
    atomicOr(&g_error, code);
}

// Producer (one thread per CTA): this CTA's 128 rows of A and its 128 rows of B (64 of the
// gated half and 64 of the other for UP in the single shape; in a pair the leader loads the
// gated half, the peer the other).  The peer's copies complete on the leader's barrier,
// which the leader armed for both CTAs' bytes.
template <int MODE, bool A_MN, bool B_MN, bool PAIR>
__device__ void run_producer(const CUtensorMap* tmA, const CUtensorMap* tmB, const Params& p, uint8_t* ring, Bars* b,
                             const Where& w)
{
    const bool remote = PAIR && w.rank == 1;
    int s = 0;
    uint32_t phase = 0;
    int32_t last[STAGES];
#pragma unroll
    for (int i = 0; i < STAGES; ++i) last[i] = -1;
    for (int64_t i = w.worker; i < p.items && !b->abort; i += w.n_workers) {
        const Item it = item_at(i, p);
        const int32_t ma = it.m_blk * tile_m<PAIR>() + (int32_t)w.rank * BM;
        int32_t n0, n1;
        if (MODE == UP) {
            if (PAIR) {
                n0 = it.n_blk * 128 + (w.rank ? p.N : 0);
                n1 = n0 + BOX;
            } else {
                n0 = it.n_blk * 64;
                n1 = p.N + n0;
            }
        } else {
            n0 = it.n_blk * tile_n<PAIR>() + (int32_t)w.rank * 128;
            n1 = n0 + BOX;
        }
        for (int kb = it.kb0; kb < it.kb1; ++kb) {
            if (!wait_or_abort<PAIR>(smem_u32(&b->empty[s]), phase ^ 1u, b)) {
                raise_abort(b, 1u);
                break;
            }
            const uint32_t dst = smem_u32(ring + (size_t)s * STAGE_BYTES);
            const int32_t k = kb * BK;
            uint32_t bar = smem_u32(&b->full[s]);
            if (remote)
                bar = tc::mapa(bar, 0);
            else
                mbar_arrive_expect_tx(bar, PAIR ? 2 * STAGE_BYTES : STAGE_BYTES);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int32_t m = ma + h * BOX, n = h ? n1 : n0;
                const uint32_t da = dst + h * BOX_BYTES, db = dst + OP_BYTES + h * BOX_BYTES;
                if (remote) {
                    tc::tma_load_2d_pair(da, tmA, A_MN ? m : k, A_MN ? k : m, bar);
                    tc::tma_load_2d_pair(db, tmB, B_MN ? n : k, B_MN ? k : n, bar);
                } else {
                    tc::tma_load_2d(da, tmA, A_MN ? m : k, A_MN ? k : m, bar);
                    tc::tma_load_2d(db, tmB, B_MN ? n : k, B_MN ? k : n, bar);
                }
            }
            last[s] = (int32_t)phase;
            if (++s == STAGES) {
                s = 0;
                phase ^= 1u;
            }
        }
    }
    // every copy issued must have landed before its CTA may exit
    if (remote) {
#pragma unroll
        for (int i = 0; i < STAGES; ++i)
            tc::st_cluster_u32(tc::mapa(smem_u32(&b->peer_last[i]), 0), (uint32_t)last[i]);
        return;
    }
#pragma unroll
    for (int i = 0; i < STAGES; ++i)
        if (last[i] >= 0 && !mbar_wait_bounded(smem_u32(&b->full[i]), (uint32_t)last[i], kWaitLimit))
            atomicOr(&g_error, 2u);
}

// MMA issuer (one thread; the leader's in a pair).
template <bool A_MN, bool B_MN, bool PAIR>
__device__ void run_mma(const Params& p, uint8_t* ring, Bars* b, const Where& w)
{
    const uint32_t idesc = tc::idesc_bf16_f32(tile_m<PAIR>(), tile_n<PAIR>()) | (A_MN ? 1u << 15 : 0u) |
                           (B_MN ? 1u << 16 : 0u);
    // UK elements of K further: 32 bytes inside a swizzled row, or two 8-row atoms
    constexpr uint64_t A_STEP = A_MN ? 2048 >> 4 : 32 >> 4, B_STEP = B_MN ? 2048 >> 4 : 32 >> 4;
    int s = 0;
    uint32_t phase = 0;
    int64_t n = 0;
    for (int64_t i = w.worker; i < p.items && !b->abort; i += w.n_workers, ++n) {
        const Item it = item_at(i, p);
        const int ab = (int)(n & 1);
        if (!wait_or_abort<PAIR>(smem_u32(&b->acc_empty[ab]), (uint32_t)((n >> 1) & 1) ^ 1u, b)) {
            raise_abort(b, 4u);
            break;
        }
        tc::fence_after_sync();
        const uint32_t d = b->tmem_base + (uint32_t)(ab * tile_n<PAIR>());
        bool ok = true;
        for (int kb = it.kb0; kb < it.kb1; ++kb) {
            if (!wait_or_abort<PAIR>(smem_u32(&b->full[s]), phase, b)) {
                raise_abort(b, 8u);
                ok = false;
                break;
            }
            tc::fence_after_sync();
            const uint32_t a_addr = smem_u32(ring + (size_t)s * STAGE_BYTES), b_addr = a_addr + OP_BYTES;
            const uint64_t a_desc = A_MN ? smem_desc_mn(a_addr) : tc::smem_desc_sw128(a_addr);
            const uint64_t b_desc = B_MN ? smem_desc_mn(b_addr) : tc::smem_desc_sw128(b_addr);
#pragma unroll
            for (int kk = 0; kk < BK / UK; ++kk) {
                const uint32_t acc = (kb > it.kb0 || kk) ? 1u : 0u;
                if (PAIR)
                    tc::mma_bf16_pair(d, a_desc + kk * A_STEP, b_desc + kk * B_STEP, idesc, acc);
                else
                    tc::mma_bf16(d, a_desc + kk * A_STEP, b_desc + kk * B_STEP, idesc, acc);
            }
            const uint32_t e = smem_u32(&b->empty[s]);
            if (PAIR) {
                tc::commit_pair(e);
                tc::commit_pair(tc::mapa(e, 1));
            } else {
                tc::commit(e);
            }
            if (++s == STAGES) {
                s = 0;
                phase ^= 1u;
            }
        }
        if (!ok) break;
        const uint32_t f = smem_u32(&b->acc_full[ab]);
        if (PAIR) {
            tc::commit_pair(f);
            tc::commit_pair(tc::mapa(f, 1));
        } else {
            tc::commit(f);
        }
    }
    if (PAIR)
        tc::commit_pair(smem_u32(&b->drain));
    else
        tc::commit(smem_u32(&b->drain));
    if (!mbar_wait_bounded(smem_u32(&b->drain), 0u, kWaitLimit)) atomicOr(&g_error, 16u);
}

// ---------------------------------------------------------------------------------
// The activation and its gradient, in fp32 with one ex2 and one reciprocal on the MUFU
// pipe (relative error a few 1e-7, far below half a bf16 step).

__device__ __forceinline__ float sigmoid_fast(float a)
{
    float e, r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(-1.4426950408889634f * a));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.f + e));
    return r;
}

// d = d_act; on return a = da, b = db, d = act
__device__ __forceinline__ void dact_one(float& d, float& a, float& b)
{
    const float s = sigmoid_fast(a), as = a * s;
    const float da = d * b * s * fmaf(a, 1.f - s, 1.f), db = d * as;
    d = as * b;
    a = da;
    b = db;
}

// Eight output values of one row from column `col` on: to bf16 or f32, optionally added to
// what is there.
__device__ __forceinline__ void store8(const Params& p, int64_t row, int32_t col, float* v)
{
    if (p.out_f32) {
        float* dst = static_cast<float*>(p.out) + row * p.ld_out + col;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            float4* q = reinterpret_cast<float4*>(dst + 4 * h);
            float4 x = make_float4(v[4 * h], v[4 * h + 1], v[4 * h + 2], v[4 * h + 3]);
            if (p.accumulate) {
                const float4 o = *q;
                x = make_float4(x.x + o.x, x.y + o.y, x.z + o.z, x.w + o.w);
            }
            *q = x;
        }
    } else {
        bf16* dst = static_cast<bf16*>(p.out) + row * p.ld_out + col;
        if (p.accumulate) {
            float o[8];
            unpack<bf16>(ld_plain(dst), o);
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] += o[e];
        }
        *reinterpret_cast<uint4*>(dst) = pack<bf16>(v);
    }
}

// act (and u) of eight columns
__device__ __forceinline__ void up8(const Params& p, int64_t row, int32_t col, float* a, const float* b)
{
    if (p.u) {
        *reinterpret_cast<uint4*>(p.u + row * p.ld_u + col) = pack<bf16>(a);
        *reinterpret_cast<uint4*>(p.u + row * p.ld_u + p.N + col) = pack<bf16>(b);
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) a[e] = a[e] * sigmoid_fast(a[e]) * b[e];
    *reinterpret_cast<uint4*>(static_cast<bf16*>(p.out) + row * p.ld_out + col) = pack<bf16>(a);
}

// du and act of eight columns from d_act and the loaded a and b
__device__ __forceinline__ void dact8(const Params& p, int64_t row, int32_t col, float* d, const uint4& ua,
                                      const uint4& ub)
{
    float a[8], b[8];
    unpack<bf16>(ua, a);
    unpack<bf16>(ub, b);
#pragma unroll
    for (int e = 0; e < 8; ++e) dact_one(d[e], a[e], b[e]);
    *reinterpret_cast<uint4*>(p.du + row * p.ld_du + col) = pack<bf16>(a);
    *reinterpret_cast<uint4*>(p.du + row * p.ld_du + p.N + col) = pack<bf16>(b);
    if (p.out) *reinterpret_cast<uint4*>(static_cast<bf16*>(p.out) + row * p.ld_out + col) = pack<bf16>(d);
}

// Epilogue: thread (warp w, lane l) owns accumulator row 32 * (w % 4) + l of this CTA and,
// with eight warps, half of its columns.
template <int MODE, bool PAIR> __device__ void run_epilogue(const Params& p, Bars* b, const Where& w)
{
    constexpr int EW = epi_warps(MODE), H = EW / 4, TN = tile_n<PAIR>();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int quarter = warp & 3, part = (warp - EPI_WARP0) / 4;
    int64_t n = 0;
    for (int64_t i = w.worker; i < p.items; i += w.n_workers, ++n) {
        const Item it = item_at(i, p);
        const int ab = (int)(n & 1);
        const bool got = wait_or_abort<PAIR>(smem_u32(&b->acc_full[ab]), (uint32_t)((n >> 1) & 1), b);
        if (!__all_sync(0xffffffffu, got)) {
            raise_abort(b, 32u);
            break;
        }
        tc::fence_after_sync();
        const int64_t row = (int64_t)it.m_blk * tile_m<PAIR>() + (int64_t)w.rank * BM + quarter * 32 + lane;
        const bool live = row < p.M;
        const uint32_t t = b->tmem_base + ((uint32_t)(quarter * 32) << 16) + (uint32_t)(ab * TN);
        float v[32];
        if constexpr (MODE == UP) {
            constexpr int HALF = TN / 2, CH = HALF / 32;  // a in columns [0, HALF), b behind them
            float g[32];
#pragma unroll 1
            for (int c = part * (CH / H); c < (part + 1) * (CH / H); ++c) {
                const int32_t col = it.n_blk * HALF + 32 * c;
                tc::ld32(t + 32 * c, v);
                tc::ld32(t + HALF + 32 * c, g);
                if (!live) continue;
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if (col + 8 * j < p.N) up8(p, row, col + 8 * j, v + 8 * j, g + 8 * j);
            }
        } else {
            constexpr int CH = TN / 32;
#pragma unroll 1
            for (int c = part * (CH / H); c < (part + 1) * (CH / H); ++c) {
                const int32_t col = it.n_blk * TN + 32 * c;
                uint4 ua[4], ub[4];
                if constexpr (MODE == DACT) {
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        if (live && col + 8 * j < p.N) {
                            ua[j] = ld_stream_ro(p.u + row * p.ld_u + col + 8 * j);
                            ub[j] = ld_stream_ro(p.u + row * p.ld_u + p.N + col + 8 * j);
                        }
                }
                tc::ld32(t + 32 * c, v);
                if (!live) continue;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    if (col + 8 * j >= p.N) continue;
                    if constexpr (MODE == DACT) {
                        dact8(p, row, col + 8 * j, v + 8 * j, ua[j], ub[j]);
                    } else if constexpr (MODE == STORE) {
                        store8(p, row, col + 8 * j, v + 8 * j);
                    } else {
                        float4* q = reinterpret_cast<float4*>(p.partial + ((int64_t)it.split * p.M + row) * p.N + col +
                                                              8 * j);
                        q[0] = make_float4(v[8 * j], v[8 * j + 1], v[8 * j + 2], v[8 * j + 3]);
                        q[1] = make_float4(v[8 * j + 4], v[8 * j + 5], v[8 * j + 6], v[8 * j + 7]);
                    }
                }
            }
        }
        tc::fence_before_sync();
        __syncwarp();
        if (lane == 0) {
            const uint32_t e = smem_u32(&b->acc_empty[ab]);
            if (PAIR)
                tc::mbar_arrive_cluster(tc::mapa(e, 0));
            else
                tc::mbar_arrive(e);
        }
    }
}

template <int MODE, bool A_MN, bool B_MN, bool PAIR>
__global__ void __launch_bounds__(block_threads(MODE), 1)
    k_product(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
              const __grid_constant__ Params p)
{
    extern __shared__ uint8_t smem_raw[];
    uint8_t* ring = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    Bars* b = reinterpret_cast<Bars*>(ring + (size_t)STAGES * STAGE_BYTES);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    constexpr uint32_t TMEM_COLS = 2 * tile_n<PAIR>();
    Where w;
    w.rank = PAIR ? tc::cluster_rank() : 0u;
    w.worker = PAIR ? blockIdx.x / 2 : blockIdx.x;
    w.n_workers = PAIR ? gridDim.x / 2 : gridDim.x;

    if (threadIdx.x == 0) {
#pragma unroll
        for (int i = 0; i < STAGES; ++i) {
            mbar_init(smem_u32(&b->full[i]), 1);
            mbar_init(smem_u32(&b->empty[i]), 1);
            b->peer_last[i] = -1;
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            mbar_init(smem_u32(&b->acc_full[i]), 1);
            mbar_init(smem_u32(&b->acc_empty[i]), (PAIR ? 2 : 1) * epi_warps(MODE));
        }
        mbar_init(smem_u32(&b->drain), 1);
        b->abort = 0;
        mbar_fence_init();
        tc::prefetch_tmap(&tmA);
        tc::prefetch_tmap(&tmB);
    }
    if (warp == 1) {
        if constexpr (PAIR) {
            tc::tmem_alloc_pair(smem_u32(&b->tmem_base), TMEM_COLS);
            tc::tmem_relinquish_pair();
        } else {
            tc::tmem_alloc(smem_u32(&b->tmem_base), TMEM_COLS);
            tc::tmem_relinquish();
        }
    }
    tc::fence_before_sync();
    __syncthreads();
    if constexpr (PAIR) tc::cluster_sync();  // both CTAs' barriers exist before any remote arrival
    tc::fence_after_sync();

    if (warp == 0) {
        if (lane == 0) run_producer<MODE, A_MN, B_MN, PAIR>(&tmA, &tmB, p, ring, b, w);
    } else if (warp == 1) {
        if (lane == 0 && w.rank == 0) run_mma<A_MN, B_MN, PAIR>(p, ring, b, w);
    } else {
        run_epilogue<MODE, PAIR>(p, b, w);
    }

    tc::fence_before_sync();
    __syncthreads();
    if constexpr (PAIR) {
        tc::cluster_sync();  // the leader's MMAs have drained; the peer's last phases are in peer_last
        if (w.rank == 0 && threadIdx.x == 0) {
#pragma unroll
            for (int i = 0; i < STAGES; ++i) {
                const int32_t ph = b->peer_last[i];
                if (ph >= 0 && !mbar_wait_bounded(smem_u32(&b->full[i]), (uint32_t)ph, kWaitLimit))
                    atomicOr(&g_error, 2u);
            }
        }
        tc::cluster_sync();  // every copy into either CTA has landed
    }
    if (warp == 1) {
        tc::fence_after_sync();
        if constexpr (PAIR)
            tc::tmem_dealloc_pair(b->tmem_base, TMEM_COLS);
        else
            tc::tmem_dealloc(b->tmem_base, TMEM_COLS);
    }
}

// Adds the partial sums of a split product in the order of the splits and applies its
// epilogue; eight columns a thread.  UP: the partials hold [a | b] (2 * N columns).
template <int MODE> __global__ void __launch_bounds__(256) k_join(const __grid_constant__ Params p)
{
    const int64_t per_row = p.N / 8, total = (int64_t)p.M * per_row;
    const int64_t width = MODE == UP ? 2 * (int64_t)p.N : p.N, plane = (int64_t)p.M * width;
    for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < total; i += (int64_t)gridDim.x * blockDim.x) {
        const int64_t row = i / per_row;
        const int32_t col = (int32_t)(i - row * per_row) * 8;
        float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f}, g[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
        const float* q = p.partial + row * width + col;
        for (int s = 0; s < p.splits; ++s, q += plane) {
            float f[8];
            unpack<float>(ld_stream(q), f);
            unpack<float>(ld_stream(q + 4), f + 4);
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] += f[e];
            if constexpr (MODE == UP) {
                unpack<float>(ld_stream(q + p.N), f);
                unpack<float>(ld_stream(q + p.N + 4), f + 4);
#pragma unroll
                for (int e = 0; e < 8; ++e) g[e] += f[e];
            }
        }
        if constexpr (MODE == UP)
            up8(p, row, col, v, g);
        else if constexpr (MODE == DACT)
            dact8(p, row, col, v, ld_stream_ro(p.u + row * p.ld_u + col), ld_stream_ro(p.u + row * p.ld_u + p.N + col));
        else
            store8(p, row, col, v);
    }
}

}  // namespace ffn

// ---------------------------------------------------------------------------------
// Host side.

namespace {

PFN_cuTensorMapEncodeTiled_v12000 encode_fn()
{
    static PFN_cuTensorMapEncodeTiled_v12000 fn = [] {
        void* f = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q) !=
                cudaSuccess ||
            q != cudaDriverEntryPointSuccess)
            f = nullptr;
        return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(f);
    }();
    return fn;
}

// Boxes of 64 x 64 in the 128-byte swizzle; what lies outside the tensor reads as zero.
bool make_map(CUtensorMap* m, const Mat& t)
{
    auto fn = encode_fn();
    if (!fn) return false;
    const cuuint64_t dims[2] = {(cuuint64_t)t.cols, (cuuint64_t)t.rows};
    const cuuint64_t strides[1] = {(cuuint64_t)t.ld * 2};
    const cuuint32_t box[2] = {ffn::BOX, ffn::BOX};
    const cuuint32_t estr[2] = {1, 1};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(t.p), dims, strides, box, estr,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Tile shape and K split of a product, from its sizes alone.
struct Plan {
    bool pair;
    int32_t tiles_m, tiles_n, kblocks, splits, kb_split;
};

Plan plan(FfnEpi epi, int64_t M, int64_t N, int64_t K)
{
    Plan r;
    r.pair = M > ffn::BM;
    const int64_t tm = r.pair ? 256 : 128, tn = r.pair ? 256 : 128, workers = r.pair ? ffn::B200_SMS / 2 : ffn::B200_SMS;
    r.kblocks = (int32_t)((K + ffn::BK - 1) / ffn::BK);
    // microseconds: a k-block of a tile with every worker busy, a tile's fill and drain, the
    // f32 partials written and read at 5 TB/s, the second launch
    const double t_kb = r.pair ? 0.44 : 0.37, t_tile = 1.0, t_join = 4.0, mb = (double)M * (double)N * 8e-6 / 5.0 *
                                                                            (epi == FFN_UP ? 2 : 1);
    double best = 0;
    r.splits = 0;
    for (int32_t want = 1; want <= 32; ++want) {
        const int32_t kb = std::max(1, (r.kblocks + want - 1) / want), s = std::max(1, (r.kblocks + kb - 1) / kb);
        if (s != want) continue;
        const int64_t nt = epi == FFN_UP && s == 1 ? tn / 2 : tn, n = epi == FFN_UP && s > 1 ? 2 * N : N;
        const int64_t tiles = ((M + tm - 1) / tm) * ((n + nt - 1) / nt);
        const double waves = (double)((tiles * s + workers - 1) / workers);
        const double t = waves * (kb * t_kb + t_tile) + (s > 1 ? s * mb + t_join : 0.0);
        if (!r.splits || t < best) {
            best = t;
            r.splits = s;
            r.kb_split = kb;
            r.tiles_m = (int32_t)((M + tm - 1) / tm);
            r.tiles_n = (int32_t)((n + nt - 1) / nt);
        }
    }
    return r;
}

template <int MODE, bool A_MN, bool B_MN, bool PAIR>
cudaError_t launch_kernel(const CUtensorMap& ma, const CUtensorMap& mb, const ffn::Params& p, cudaStream_t s)
{
    auto kern = ffn::k_product<MODE, A_MN, B_MN, PAIR>;
    constexpr int kMaxDevices = 64;
    static int workers_dev[kMaxDevices] = {};  // resident CTAs or pairs, once the attribute is set
    static std::mutex mu;
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= kMaxDevices) return cudaErrorInvalidDevice;
    cudaLaunchAttribute la[1];
    la[0].id = cudaLaunchAttributeClusterDimension;
    la[0].val.clusterDim.x = 2;
    la[0].val.clusterDim.y = 1;
    la[0].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.blockDim = dim3(ffn::block_threads(MODE));
    cfg.dynamicSmemBytes = ffn::kSmemBytes;
    cfg.stream = s;
    if (PAIR) {
        cfg.attrs = la;
        cfg.numAttrs = 1;
    }
    int64_t workers;
    {
        std::lock_guard<std::mutex> lk(mu);
        if (!workers_dev[dev]) {
            e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)ffn::kSmemBytes);
            if (e != cudaSuccess) return e;
            int n = sm_count();
            if (PAIR) {
                cudaLaunchConfig_t q = cfg;
                q.gridDim = dim3(2 * (sm_count() / 2));
                if (cudaOccupancyMaxActiveClusters(&n, kern, &q) != cudaSuccess || n < 1) n = sm_count() / 2;
            }
            workers_dev[dev] = n;
        }
        workers = workers_dev[dev];
    }
    workers = std::min<int64_t>(p.items, workers);
    cfg.gridDim = dim3((unsigned)(PAIR ? 2 * workers : workers));
    return cudaLaunchKernelEx(&cfg, kern, ma, mb, p);
}

template <int MODE, bool A_MN, bool B_MN>
cudaError_t launch_shape(bool pair, const CUtensorMap& ma, const CUtensorMap& mb, const ffn::Params& p, cudaStream_t s)
{
    return pair ? launch_kernel<MODE, A_MN, B_MN, true>(ma, mb, p, s)
                : launch_kernel<MODE, A_MN, B_MN, false>(ma, mb, p, s);
}

// The operand layouts that the block uses: K | K (forward), K | N (d_act, dx), M | N (dW).
template <int MODE>
cudaError_t launch_layout(bool pair, bool a_mn, bool b_mn, const CUtensorMap& ma, const CUtensorMap& mb,
                          const ffn::Params& p, cudaStream_t s)
{
    if (a_mn && b_mn) return launch_shape<MODE, true, true>(pair, ma, mb, p, s);
    if (!a_mn && b_mn) return launch_shape<MODE, false, true>(pair, ma, mb, p, s);
    if (!a_mn && !b_mn) return launch_shape<MODE, false, false>(pair, ma, mb, p, s);
    return cudaErrorInvalidValue;
}

template <int MODE> cudaError_t launch_join(const ffn::Params& p, cudaStream_t s)
{
    const int64_t n = (int64_t)p.M * (p.N / 8);
    const int64_t grid = std::min<int64_t>((n + 255) / 256, (int64_t)sm_count() * 16);
    ffn::k_join<MODE><<<(unsigned)grid, 256, 0, s>>>(p);
    return cudaGetLastError();
}

}  // namespace

size_t ffn_partial_bytes(FfnEpi epi, int64_t M, int64_t N, int64_t K)
{
    const Plan r = plan(epi, M, N, K);
    return r.splits > 1 ? (size_t)r.splits * (size_t)M * (size_t)N * (epi == FFN_UP ? 8 : 4) : 0;
}

cudaError_t launch_ffn_product(const FfnProduct& g, cudaStream_t s)
{
    if (g.M == 0 || g.N == 0) return cudaSuccess;
    CUtensorMap ma, mb;
    if (!make_map(&ma, g.a) || !make_map(&mb, g.b)) {
        record_error("tensor map encoding failed (cuTensorMapEncodeTiled unavailable or refused the layout)");
        return cudaErrorInvalidValue;
    }
    const Plan r = plan(g.epi, g.M, g.N, g.K);
    ffn::Params p{};
    p.M = (int32_t)g.M;
    p.N = (int32_t)g.N;
    p.kblocks = r.kblocks;
    p.tiles_m = r.tiles_m;
    p.tiles_n = r.tiles_n;
    p.splits = r.splits;
    p.kb_split = r.kb_split;
    p.items = (int64_t)r.tiles_m * r.tiles_n * r.splits;
    p.out = g.out;
    p.ld_out = g.ld_out;
    p.out_f32 = g.out_f32;
    p.accumulate = g.accumulate;
    p.u = static_cast<bf16*>(g.u);
    p.ld_u = g.ld_u;
    p.du = static_cast<bf16*>(g.du);
    p.ld_du = g.ld_du;
    p.partial = g.partial;
    if (r.splits == 1) {
        if (g.epi == FFN_UP) return launch_shape<ffn::UP, false, false>(r.pair, ma, mb, p, s);
        if (g.epi == FFN_DACT) return launch_shape<ffn::DACT, false, true>(r.pair, ma, mb, p, s);
        return launch_layout<ffn::STORE>(r.pair, g.a_mn, g.b_mn, ma, mb, p, s);
    }
    ffn::Params q = p;
    if (g.epi == FFN_UP) q.N = 2 * p.N;
    cudaError_t e = launch_layout<ffn::PART>(r.pair, g.a_mn, g.b_mn, ma, mb, q, s);
    if (e != cudaSuccess) return e;
    if (g.epi == FFN_UP) return launch_join<ffn::UP>(p, s);
    if (g.epi == FFN_DACT) return launch_join<ffn::DACT>(p, s);
    return launch_join<ffn::STORE>(p, s);
}

uint32_t ffn_device_error(bool clear)
{
    uint32_t v = 0;
    if (cudaMemcpyFromSymbol(&v, ffn::g_error, sizeof v) != cudaSuccess) return 0xffffffffu;
    if (clear && v) {
        const uint32_t z = 0;
        cudaMemcpyToSymbol(ffn::g_error, &z, sizeof z);
    }
    return v;
}

}  // namespace sol
