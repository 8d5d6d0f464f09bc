// k_ffn.cu -- the products of the gated feed-forward block and its backward pass on the
// fifth-generation tensor cores:
//     forward    [a | b] = x . W_up^T,  act = silu(a) * b      (one kernel: FFN_UP)
//                y = act . W_down^T
//     backward   d_act = dy . W_down  -> du, act from u         (one kernel: FFN_DACT)
//                dx = du . W_up,  dW_up = du^T . x,  dW_down = dy^T . act
//
// One kernel for all: C[M, N] = A . B^T over K, each operand stored with K contiguous or
// with M (N) contiguous; the last three run in one launch, which fills the GPU where each alone would
// leave a part of it idle.  A stage of the shared-memory ring holds 128 x 64 of A and
// 128 x 64 of B as four 64 x 64 boxes of 8 KiB that the tensor copy writes in the 128-byte
// swizzle; a box has the contiguous dimension of its operand along its rows, so both
// layouts cost the same copies and differ only in the matrix descriptor (smem_desc_mn) and
// the instruction descriptor's major bits.  No operand is transposed in memory.
// Three tile shapes (Tile): one CTA on 128 x 128, and a cluster of two CTAs (cta_group::2, each
// loading half of A and half of B) on 256 x 256 or 512 x 256; plan() takes the one whose estimated
// time is least.
//
// At d 5120, width 13,824 and 31,248 tokens: forward with u kept 10.0 to 10.5 ms (1.32 to 1.26 PFLOP/s), backward
// 21.4 to 23.0 ms (1.24 to 1.15), both at the power cap, where cuBLAS alone reaches 1.38; at 1,252 tokens 0.48
// and 0.98 ms; few tokens of small blocks go to k_ffn_small.cu.  Weight gradients in f32, or added to what
// is there, leave by the slower way that finish16 describes.
// Everything outside a tensor is read as zero by the tensor copies (ragged M, N and K) and
// never stored.
//
// The tiles that do not fill a last round of the persistent workers would leave most of them
// idle for a whole tile: their K ranges are instead laid end to end and cut into equal pieces,
// one a worker (see plan()).  A piece that is not a whole tile goes to an f32 slot of the
// workspace; k_join adds the pieces of a tile in the order of K and applies the epilogue.
//
// The kernels of one call are launched so that the next one's set-up overlaps the last one's
// end (programmatic dependent launch); every thread waits for the end of the kernel before
// (griddep_wait) ahead of its first access to global memory.
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
// m-blocks per raster group: 74 pairs then work on 8 x 9 tiles at a time, which read the fewest
// distinct rows of A and B.  DRAM reads of dx and dW_up at 31,248 tokens 13.4 GB each, 14.4 (and up
// to 25) with 16, 19 with 4; the whole backward pass 21.6 against 22.5 ms at the power cap.
constexpr int GROUP_M = 8;
constexpr int EPI_WARP0 = 2;
constexpr uint32_t kWaitLimit = 4096;      // polls of <= ~1 ms each
constexpr uint32_t kPollLimit = 1u << 26;  // polls without a suspend hint
constexpr int B200_SMS = 148;              // plan() is a function of the sizes alone

enum Mode : int { STORE = FFN_STORE, UP = FFN_UP, DACT = FFN_DACT };

// Tile shapes:
//   SINGLE  one CTA, 128 x 128, two accumulators in TMEM;
//   PAIR    two CTAs on two SMs, 256 x 256 (256-row MMAs, each CTA loading half of A and half of
//           B), two accumulators, so that the epilogue of a tile runs under the next tile;
//   WIDE    the same pair on 512 x 256: two MMAs a step share B, a quarter less comes from L2
//           than by two PAIR tiles (which bound PAIR: 64 KiB a k-block and pair, 11 TB/s in
//           all); the accumulators fill TMEM, so that the epilogue stands between two tiles.
enum Shape : int { SINGLE = 0, PAIR = 1, WIDE = 2 };
template <int S> struct Tile {
    static constexpr bool PAIRED = S != SINGLE;
    static constexpr int HALVES = S == WIDE ? 2 : 1;  // 128-row halves of A a CTA holds
    static constexpr int ROWS = BM * HALVES;          // rows of a CTA
    static constexpr int M = PAIRED ? 2 * ROWS : ROWS, N = PAIRED ? 256 : 128;
    static constexpr int A_BYTES = ROWS * BK * 2, STAGE_BYTES = A_BYTES + 128 * BK * 2;
    static constexpr int ACCS = S == WIDE ? 1 : 2;    // accumulators in TMEM
    static constexpr int TMEM_COLS = S == SINGLE ? 256 : 512;
};
constexpr int MAX_STAGES = 5;

// Epilogue warps: four (one per TMEM lane quarter) where the epilogue only stores, eight
// where it also computes (two per quarter, half of the columns each) or holds up the MMAs (two
// per quarter, half of the rows each).
__host__ __device__ constexpr int epi_warps(int mode, int shape) { return mode != STORE || shape == WIDE ? 8 : 4; }
__host__ __device__ constexpr int block_threads(int mode, int shape) { return 64 + 32 * epi_warps(mode, shape); }
// Staging of the epilogue warps, and stages of the ring in what is left (PAIR: five are as fast as
// seven; d_act with four took 162 us of 152 for 1,252 tokens at full width).  A SINGLE tile of d_act
// brings all of its u at once.
__host__ __device__ constexpr int epi_bytes(int mode, int shape)
{
    return shape == WIDE ? 32768 : mode == DACT && shape == SINGLE ? 98304 : 49152;
}
__host__ __device__ constexpr int stages(int mode, int shape) { return shape == WIDE || (mode == DACT && shape == SINGLE) ? 4 : 5; }

struct Bars {
    uint64_t full[MAX_STAGES], empty[MAX_STAGES], acc_full[2], acc_empty[2], drain;
    uint64_t u_full[8];         // DACT: a warp's pieces of u have landed
    int32_t peer_last[MAX_STAGES];  // leader: phase of the peer's last copy per stage (-1: none)
    uint32_t tmem_base;
    volatile int32_t abort;
};
template <int MODE, int S> constexpr size_t smem_bytes()
{
    return 1024 + (size_t)stages(MODE, S) * Tile<S>::STAGE_BYTES + epi_bytes(MODE, S) + sizeof(Bars);
}
static_assert(smem_bytes<STORE, WIDE>() <= 232448 && smem_bytes<UP, PAIR>() <= 232448 && smem_bytes<DACT, SINGLE>() <= 232448,
              "shared memory of a CTA");

__device__ uint32_t g_error;

constexpr int MAX_PRODUCTS = 3;

// One product of a launch.  Its tiles [0, whole) are worked on whole, one after another by each
// worker; tiles [whole, tiles) are the rest, which all products of the launch share out together.
struct Product {
    int32_t M, N, kblocks;       // N: columns of the output (UP: inner)
    int32_t tiles_m, tiles_n;
    int64_t whole, tiles;
    int32_t a_mn;                // STORE: A is stored with M contiguous
    int32_t stage_bytes;         // bytes that the copies of one CTA and stage bring
    int32_t a_blocks, b_blocks;  // 1: one copy brings a CTA's rows of the operand (see make_map)
    int32_t out_f32, accumulate;
    int32_t wide;                // rows of out, u and du (and their second halves) begin on 32-byte boundaries
    void* out;
    int64_t ld_out;
};
struct Params {
    Product g[MAX_PRODUCTS];
    int32_t n;                   // products
    int32_t pieces, piece_kb;    // the rest's K end to end in `pieces` of piece_kb blocks; 0: whole tiles
    int64_t rest_tiles, rest_kb;
    bf16* u;
    int64_t ld_u;
    bf16* du;
    int64_t ld_du;
    float* slots;                // f32 [2 * pieces, TN / 8, TM, 8]: pieces that are not whole tiles
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

// Tensor maps of one launch: the operands, and what the epilogue copies through shared memory
// (STORE: out; UP and DACT: act, the halves of u, the halves of du; boxes as in out_map).
struct Maps {
    CUtensorMap a[MAX_PRODUCTS], b[MAX_PRODUCTS], out[MAX_PRODUCTS], u_a, u_b, du_a, du_b;
};

// A piece of work: K blocks [kb0, kb1) of a tile of product g; slot >= 0 where they are not all
// of its K.
struct Piece {
    int32_t g, m_blk, n_blk, kb0, kb1;
    int64_t slot;
};

// Tile t -> its blocks of rows and columns, in groups of GROUP_M m-blocks so that the tiles
// worked on at one time share rows of A and of B in L2.
__device__ __forceinline__ void tile_at(int64_t t, const Product& p, int32_t& m_blk, int32_t& n_blk)
{
    const uint32_t per_group = GROUP_M * (uint32_t)p.tiles_n, g = (uint32_t)t / per_group;  // tiles: below 2^31
    const uint32_t gm = min((uint32_t)GROUP_M, (uint32_t)p.tiles_m - g * GROUP_M);
    const uint32_t local = (uint32_t)t - g * per_group;
    m_blk = (int32_t)(g * GROUP_M + local % gm);
    n_blk = (int32_t)(local / gm);
}

// The pieces of one worker, the same sequence for every role: its whole tiles of each product, then
// its part of the rest: whole tiles, or a share of their K end to end.  A share begins inside a
// tile (slot 0 of the share) at most once and ends inside another (slot 1) at most once.
struct Walk {
    int32_t g;
    int64_t t, q, end, share, worker;
};

__device__ __forceinline__ Walk walk_begin(int64_t worker) { return Walk{0, worker, 0, 0, worker, worker}; }

__device__ __forceinline__ bool walk_next(Walk& w, const Params& p, int64_t n_workers, Piece& x)
{
    for (; w.g < p.n; ++w.g, w.t = w.worker) {
        const Product& c = p.g[w.g];
        if (w.t < c.whole) {
            x.g = w.g;
            x.kb0 = 0;
            x.kb1 = c.kblocks;
            x.slot = -1;
            tile_at(w.t, c, x.m_blk, x.n_blk);
            w.t += n_workers;
            return true;
        }
    }
    if (!p.pieces) {
        int64_t r = w.share;
        if (r >= p.rest_tiles) return false;
        w.share += n_workers;
        int32_t g = 0;
        for (; r >= p.g[g].tiles - p.g[g].whole; ++g) r -= p.g[g].tiles - p.g[g].whole;
        x.g = g;
        x.kb0 = 0;
        x.kb1 = p.g[g].kblocks;
        x.slot = -1;
        tile_at(p.g[g].whole + r, p.g[g], x.m_blk, x.n_blk);
        return true;
    }
    if (w.q >= w.end) {
        if (w.share >= p.pieces) return false;
        w.q = w.share * p.piece_kb;
        w.end = min(w.q + p.piece_kb, p.rest_kb);
        w.t = w.share;  // from here on: the share at work
        w.share += n_workers;
    }
    int64_t q = w.q;
    int32_t g = 0;
    for (;; ++g) {
        const int64_t kb = (p.g[g].tiles - p.g[g].whole) * p.g[g].kblocks;
        if (q < kb) break;
        q -= kb;
    }
    const Product& c = p.g[g];
    const int64_t tile = q / c.kblocks;
    x.g = g;
    x.kb0 = (int32_t)(q - tile * c.kblocks);
    x.kb1 = (int32_t)min((int64_t)c.kblocks, x.kb0 + (w.end - w.q));
    tile_at(c.whole + tile, c, x.m_blk, x.n_blk);
    x.slot = x.kb0 == 0 && x.kb1 == c.kblocks ? -1 : 2 * w.t + (x.kb0 == 0 ? 1 : 0);
    w.q += x.kb1 - x.kb0;
    return true;
}

__device__ __forceinline__ void griddep_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void griddep_launch() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

struct Where {
    uint32_t rank;
    int64_t worker, n_workers;
};

template <bool PAIRED> __device__ __forceinline__ bool wait_or_abort(uint32_t bar, uint32_t parity, Bars* b)
{
    const uint32_t limit = PAIRED ? kPollLimit : kWaitLimit;
    for (uint32_t i = 0; i < limit; ++i) {
        if (PAIRED ? tc::mbar_poll_cluster(bar, parity) : mbar_try_wait(bar, parity)) return true;
        if ((i & 15u) == 15u && b->abort) return false;
    }
    return false;
}

__device__ __forceinline__ void raise_abort(Bars* b, uint32_t code)
{
    b->abort = 1;
    atomicOr(&g_error, code);
}

// A CTA's rows of one operand, BOXES times 64 of them ([x0, x0 + 64), [x1, x1 + 64), then on from x0 + 128),
// for the 64 K from k on: one copy where the map's box holds them all, else one for each 64.
template <int BOXES>
__device__ __forceinline__ void load_operand(bool mn, uint32_t dst, const CUtensorMap* map, int32_t form, int32_t x0,
                                             int32_t x1, int32_t k, uint32_t bar, bool remote)
{
    if (mn && form) {
        remote ? tc::tma_load_3d_pair(dst, map, 0, k, x0 / BOX, bar) : tc::tma_load_3d(dst, map, 0, k, x0 / BOX, bar);
        return;
    }
#pragma unroll
    for (int i = 0; i < BOXES; ++i) {
        const int32_t x = i == 1 ? x1 : x0 + i * BOX, c = mn ? x : k, r = mn ? k : x;
        remote ? tc::tma_load_2d_pair(dst + i * BOX_BYTES, map, c, r, bar) : tc::tma_load_2d(dst + i * BOX_BYTES, map, c, r, bar);
        if (form) return;
    }
}

// Producer (one thread per CTA): this CTA's 128 rows of A and its 128 rows of B (64 of the
// gated half and 64 of the other for UP in the single shape; in a pair the leader loads the
// gated half, the peer the other).  The peer's copies complete on the leader's barrier,
// which the leader armed for both CTAs' bytes.
template <int MODE, bool B_MN, int S>
__device__ void run_producer(const Maps& maps, const Params& p, uint8_t* ring, Bars* b, const Where& w)
{
    using T = Tile<S>;
    constexpr int STAGES = stages(MODE, S);
    const bool remote = T::PAIRED && w.rank == 1;
    int s = 0;
    uint32_t phase = 0;
    int32_t last[STAGES];
#pragma unroll
    for (int i = 0; i < STAGES; ++i) last[i] = -1;
    Walk walk = walk_begin(w.worker);
    Piece it;
    while (!b->abort && walk_next(walk, p, w.n_workers, it)) {
        const Product& c = p.g[it.g];
        const CUtensorMap *tmA = &maps.a[it.g], *tmB = &maps.b[it.g];
        const bool a_mn = MODE == STORE && B_MN && c.a_mn;
        const int32_t ma = it.m_blk * T::M + (int32_t)w.rank * T::ROWS;
        int32_t n0, n1;
        if (MODE == UP) {
            if (T::PAIRED) {
                n0 = it.n_blk * 128 + (w.rank ? c.N : 0);
                n1 = n0 + BOX;
            } else {
                n0 = it.n_blk * 64;
                n1 = c.N + n0;
            }
        } else {
            n0 = it.n_blk * T::N + (int32_t)w.rank * 128;
            n1 = n0 + BOX;
        }
        for (int kb = it.kb0; kb < it.kb1; ++kb) {
            if (!wait_or_abort<T::PAIRED>(smem_u32(&b->empty[s]), phase ^ 1u, b)) {
                raise_abort(b, 1u);
                break;
            }
            const uint32_t dst = smem_u32(ring + (size_t)s * T::STAGE_BYTES);
            uint32_t bar = smem_u32(&b->full[s]);
            if (remote)
                bar = tc::mapa(bar, 0);
            else
                mbar_arrive_expect_tx(bar, T::PAIRED ? 2 * c.stage_bytes : c.stage_bytes);
            load_operand<T::ROWS / BOX>(a_mn, dst, tmA, c.a_blocks, ma, ma + BOX, kb * BK, bar, remote);
            load_operand<2>(B_MN, dst + T::A_BYTES, tmB, c.b_blocks, n0, n1, kb * BK, bar, remote);
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
template <int MODE, bool B_MN, int S>
__device__ void run_mma(const Params& p, uint8_t* ring, Bars* b, const Where& w)
{
    using T = Tile<S>;
    const uint32_t idesc0 = tc::idesc_bf16_f32(T::PAIRED ? 2 * BM : BM, T::N) | (B_MN ? 1u << 16 : 0u);
    // UK elements of K further: 32 bytes inside a swizzled row, or two 8-row atoms
    constexpr uint64_t B_STEP = B_MN ? 2048 >> 4 : 32 >> 4;
    constexpr uint64_t A_HALF = BM * BK * 2 >> 4;
    int s = 0;
    uint32_t phase = 0;
    int64_t n = 0;
    Walk walk = walk_begin(w.worker);
    Piece next;
    bool more = walk_next(walk, p, w.n_workers, next);
    for (; more && !b->abort; ++n) {
        const Piece it = next;
        const bool a_mn = MODE == STORE && B_MN && p.g[it.g].a_mn;
        const uint32_t idesc = idesc0 | (a_mn ? 1u << 15 : 0u);
        const uint64_t a_step = a_mn ? 2048 >> 4 : 32 >> 4;
        const int ab = T::ACCS == 2 ? (int)(n & 1) : 0;
        const uint32_t acc_phase = (uint32_t)(T::ACCS == 2 ? n >> 1 : n) & 1u;
        if (!wait_or_abort<T::PAIRED>(smem_u32(&b->acc_empty[ab]), acc_phase ^ 1u, b)) {
            raise_abort(b, 4u);
            break;
        }
        tc::fence_after_sync();
        const uint32_t d = b->tmem_base + (uint32_t)(ab * T::N);
        bool ok = true;
        for (int kb = it.kb0; kb < it.kb1; ++kb) {
            if (!wait_or_abort<T::PAIRED>(smem_u32(&b->full[s]), phase, b)) {
                raise_abort(b, 8u);
                ok = false;
                break;
            }
            tc::fence_after_sync();
            const uint32_t a_addr = smem_u32(ring + (size_t)s * T::STAGE_BYTES), b_addr = a_addr + T::A_BYTES;
            const uint64_t a_desc = a_mn ? smem_desc_mn(a_addr) : tc::smem_desc_sw128(a_addr);
            const uint64_t b_desc = B_MN ? smem_desc_mn(b_addr) : tc::smem_desc_sw128(b_addr);
#pragma unroll
            for (int kk = 0; kk < BK / UK; ++kk) {
                const uint32_t acc = (kb > it.kb0 || kk) ? 1u : 0u;
#pragma unroll
                for (int h = 0; h < T::HALVES; ++h) {
                    if (T::PAIRED)
                        tc::mma_bf16_pair(d + h * T::N, a_desc + h * A_HALF + kk * a_step, b_desc + kk * B_STEP, idesc, acc);
                    else
                        tc::mma_bf16(d, a_desc + kk * a_step, b_desc + kk * B_STEP, idesc, acc);
                }
            }
            const uint32_t e = smem_u32(&b->empty[s]);
            if (T::PAIRED) {
                tc::commit_pair(e);
                tc::commit_pair(tc::mapa(e, 1));
            } else {
                tc::commit(e);
            }
            if (++s == stages(MODE, S)) {
                s = 0;
                phase ^= 1u;
            }
            if (kb == it.kb0) more = walk_next(walk, p, w.n_workers, next);  // while the MMAs run
        }
        if (!ok) break;
        const uint32_t f = smem_u32(&b->acc_full[ab]);
        if (T::PAIRED) {
            tc::commit_pair(f);
            tc::commit_pair(tc::mapa(f, 1));
        } else {
            tc::commit(f);
        }
    }
    if (T::PAIRED)
        tc::commit_pair(smem_u32(&b->drain));
    else
        tc::commit(smem_u32(&b->drain));
    if (!mbar_wait_bounded(smem_u32(&b->drain), 0u, kWaitLimit)) atomicOr(&g_error, 16u);
}

// ---------------------------------------------------------------------------------
// The activation and its gradient, in fp32 with one ex2 and one reciprocal on the MUFU
// pipe.  Relative error a few 1e-7, and |a| * 6e-8 from rounding the argument of ex2: at most some
// 1e-5 before the sigmoid of a negative a vanishes, far below half a bf16 step (2e-3).

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

// 32 bytes in one instruction (both on a 32-byte boundary): a row-per-thread epilogue touches
// whole 32-byte sectors with it.
__device__ __forceinline__ void st256(void* p, const uint4& a, const uint4& b)
{
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(a.x), "r"(a.y), "r"(a.z),
                 "r"(a.w), "r"(b.x), "r"(b.y), "r"(b.z), "r"(b.w)
                 : "memory");
}
__device__ __forceinline__ void ld256(const void* p, uint4& a, uint4& b)
{
    asm volatile("ld.global.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(a.x), "=r"(a.y), "=r"(a.z), "=r"(a.w), "=r"(b.x), "=r"(b.y), "=r"(b.z), "=r"(b.w)
                 : "l"(p)
                 : "memory");
}

// Stores the first `n` (8 or 16) of 16 bf16 values.
__device__ __forceinline__ void put16(bf16* dst, const float* v, int n, int wide)
{
    const uint4 lo = pack<bf16>(v), hi = pack<bf16>(v + 8);
    if (wide && n == 16) {
        st256(dst, lo, hi);
    } else {
        *reinterpret_cast<uint4*>(dst) = lo;
        if (n == 16) *reinterpret_cast<uint4*>(dst + 8) = hi;
    }
}
__device__ __forceinline__ void get16(const bf16* src, uint4& lo, uint4& hi, int n, int wide)
{
    if (wide && n == 16) {
        ld256(src, lo, hi);
    } else {
        lo = ld_plain(src);
        hi = n == 16 ? ld_plain(src + 8) : make_uint4(0, 0, 0, 0);
    }
}

// The epilogue of 16 columns of one row, the first n of them inside the output.  STORE: v is
// the product.  UP: v and g are a and b.  DACT: v is d_act, ua and ub hold a and b.
//
// It ends k_join's tiles, and the whole tiles of gradients in f32 or added to what is there, straight from
// registers: 16 or 32 bytes a lane into 32 rows, on a 512 x 256 tile with nothing to hide it.  Backward pass at d 5120,
// width 13,824, us: 1,252 tokens bf16 set (through shared memory) 860, bf16 added 1,100, f32 set 1,140, f32 added 2,400;
// 31,248 tokens 21,800, 22,100, 22,000, 24,800.
template <int MODE>
__device__ __forceinline__ void finish16(const Params& q, const Product& p, int64_t row, int32_t col, int n, float* v, const float* g,
                                         const uint4* ua, const uint4* ub)
{
    if constexpr (MODE == UP) {
        if (q.u) {
            put16(q.u + row * q.ld_u + col, v, n, p.wide);
            put16(q.u + row * q.ld_u + p.N + col, g, n, p.wide);
        }
#pragma unroll
        for (int e = 0; e < 16; ++e) v[e] = v[e] * sigmoid_fast(v[e]) * g[e];
        put16(static_cast<bf16*>(p.out) + row * p.ld_out + col, v, n, p.wide);
    } else if constexpr (MODE == DACT) {
        float a[16], b[16];
        unpack<bf16>(ua[0], a);
        unpack<bf16>(ua[1], a + 8);
        unpack<bf16>(ub[0], b);
        unpack<bf16>(ub[1], b + 8);
#pragma unroll
        for (int e = 0; e < 16; ++e) dact_one(v[e], a[e], b[e]);
        put16(q.du + row * q.ld_du + col, a, n, p.wide);
        put16(q.du + row * q.ld_du + p.N + col, b, n, p.wide);
        if (p.out) put16(static_cast<bf16*>(p.out) + row * p.ld_out + col, v, n, p.wide);
    } else if (p.out_f32) {
        float* dst = static_cast<float*>(p.out) + row * p.ld_out + col;
#pragma unroll
        for (int h = 0; h < 4; ++h) {
            if (4 * h >= n) break;
            float4* at = reinterpret_cast<float4*>(dst + 4 * h);
            float4 x = make_float4(v[4 * h], v[4 * h + 1], v[4 * h + 2], v[4 * h + 3]);
            if (p.accumulate) {
                const float4 o = *at;
                x = make_float4(x.x + o.x, x.y + o.y, x.z + o.z, x.w + o.w);
            }
            *at = x;
        }
    } else {
        bf16* dst = static_cast<bf16*>(p.out) + row * p.ld_out + col;
        if (p.accumulate) {  // added in fp32, rounded once
            uint4 lo, hi;
            get16(dst, lo, hi, n, p.wide);
            float o[16];
            unpack<bf16>(lo, o);
            unpack<bf16>(hi, o + 8);
#pragma unroll
            for (int e = 0; e < 16; ++e) v[e] += o[e];
        }
        put16(dst, v, n, p.wide);
    }
}

// Columns of [col, col + 16) inside a width of N (a multiple of 8).
__device__ __forceinline__ int inside(int32_t col, int32_t N) { return min(max(N - col, 0), 16); }

__device__ __forceinline__ void sts16(uint32_t a, const uint4& v)
{
    asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(a), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}
__device__ __forceinline__ uint4 lds16(uint32_t a)
{
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a));
    return v;
}

// Staging of an epilogue warp: boxes of 32 rows, a row a lane, of 32 columns (64 bytes, 64-byte
// swizzle) or 64 columns (128 bytes, 128-byte swizzle).  Address of 16-byte vector c of a row:
// the eight lanes of a quarter-warp hit eight different bank groups.
__device__ __forceinline__ uint32_t cell64(uint32_t box, int row, int c) { return box + row * 64 + ((c ^ (row >> 1)) & 3) * 16; }
__device__ __forceinline__ uint32_t cell128(uint32_t box, int row, int c) { return box + row * 128 + ((c ^ row) & 7) * 16; }
constexpr int BOX32 = 32 * 64, BOX64 = 32 * 128;

// Epilogue: thread (warp w, lane l) owns accumulator row 32 * (w % 4) + l of this CTA and,
// with eight warps, half of its columns.  bf16 outputs go through shared memory and leave as
// tensor copies: whole rows of 64 or 128 bytes, clipped to the tensor, and no thread waits for
// them.  (Straight from registers a warp's store touched 32 rows; at d 1000, width 2504, 4,099
// tokens, d_act took 83 us.)  DACT brings u the same way, the first piece of a tile while its
// product still runs.
template <int MODE, int S>
__device__ void run_epilogue(const Maps& maps, const Params& p, uint32_t staging, Bars* b, const Where& w)
{
    using T = Tile<S>;
    constexpr int EW = epi_warps(MODE, S), TN = T::N, TM = T::M;
    constexpr int H = EW / 4 / T::HALVES;            // warps that share a row's columns
    constexpr int WIDTH = MODE == UP ? TN / 2 : TN;  // UP: a in columns [0, WIDTH), b behind them
    constexpr int CH = WIDTH / 32 / H;               // steps of 32 columns of a warp
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int quarter = warp & 3, group = (warp - EPI_WARP0) / 4;
    const int half = T::HALVES == 2 ? group : 0, part = T::HALVES == 2 ? 0 : group;
    constexpr int SPACE = epi_bytes(MODE, S) / EW;  // staging of a warp
    const uint32_t box = staging + (warp - EPI_WARP0) * SPACE;
    const uint32_t u_bar = smem_u32(&b->u_full[(warp - EPI_WARP0) & 7]);
    uint32_t u_phase = 0;
    bool u_pending = false, ok = true;
    int turn = 0;  // the box that is written next
    int64_t n = 0;
    Walk walk = walk_begin(w.worker);
    Piece it;
    for (; ok && walk_next(walk, p, w.n_workers, it); ++n) {
        const Product& c0 = p.g[it.g];
        const int32_t M = c0.M, N = c0.N;
        const int ab = T::ACCS == 2 ? (int)(n & 1) : 0;
        const uint32_t acc_phase = (uint32_t)(T::ACCS == 2 ? n >> 1 : n) & 1u;
        const int32_t row0 = it.m_blk * TM + (int32_t)w.rank * T::ROWS + half * BM + quarter * 32;  // of this warp
        const int32_t col0 = it.n_blk * WIDTH + part * CH * 32;
        const bool whole = it.slot < 0;
        // DACT: a set of boxes (a, b, act) for each 32 columns whose u is fetched at a time
        constexpr int SETS = MODE == DACT && S == SINGLE ? CH : 1;
        auto fetch_u = [&](int32_t col) {  // lane 0, once the boxes are free
            if (lane == 0) {
                const int n = min(SETS, (N - col + 31) / 32);
                tc::bulk_wait_read<0>();
                mbar_arrive_expect_tx(u_bar, 2 * n * BOX32);
                for (int i = 0; i < n; ++i) {
                    tc::tma_load_2d(box + 3 * i * BOX32, &maps.u_a, col + 32 * i, row0, u_bar);
                    tc::tma_load_2d(box + (3 * i + 1) * BOX32, &maps.u_b, col + 32 * i, row0, u_bar);
                }
            }
            u_pending = true;
        };
        if (MODE == DACT && whole && row0 < M && col0 < N) fetch_u(col0);
        const bool got = wait_or_abort<T::PAIRED>(smem_u32(&b->acc_full[ab]), acc_phase, b);
        if (!__all_sync(0xffffffffu, got)) {
            raise_abort(b, 32u);
            break;
        }
        tc::fence_after_sync();
        const uint32_t t = b->tmem_base + ((uint32_t)(quarter * 32) << 16) + (uint32_t)(ab * TN + half * TN + part * CH * 32);
        float v[32], g[MODE == UP ? 32 : 1];
#pragma unroll 1
        for (int c = 0; c < CH && ok; ++c) {
            const int32_t col = col0 + 32 * c;
            tc::ld32(t + 32 * c, v);
            if constexpr (MODE == UP) tc::ld32(t + WIDTH + 32 * c, g);
            if (row0 >= M || col >= N) continue;
            if (!whole) {
                // [column group of 8][row][8]: a warp's 32 rows are 1 KiB in a row
                if (row0 + lane >= M) continue;
                float* q = p.slots + ((it.slot * (TN / 8) + 4 * (part * CH + c)) * TM + (row0 - it.m_blk * TM) + lane) * 8;
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    st256(q + j * TM * 8, *reinterpret_cast<uint4*>(v + 8 * j), *reinterpret_cast<uint4*>(v + 8 * j + 4));
                if constexpr (MODE == UP) {
                    q += (WIDTH / 8) * TM * 8;
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        st256(q + j * TM * 8, *reinterpret_cast<uint4*>(g + 8 * j), *reinterpret_cast<uint4*>(g + 8 * j + 4));
                }
                continue;
            }
            if constexpr (MODE == STORE) {
                if (c0.out_f32 || c0.accumulate) {
                    const int n0 = inside(col, N), n1 = inside(col + 16, N);
                    if (row0 + lane < M) {
                        if (n0) finish16<MODE>(p, c0, row0 + lane, col, n0, v, g, nullptr, nullptr);
                        if (n1) finish16<MODE>(p, c0, row0 + lane, col + 16, n1, v + 16, g, nullptr, nullptr);
                    }
                    continue;
                }
                // boxes of 64 columns in turn, from tile to tile
                constexpr int BOXES = SPACE / BOX64;
                const uint32_t dst = box + turn * BOX64;
                if (!(c & 1)) {
                    if (lane == 0) tc::bulk_wait_read<BOXES - 1>();
                    __syncwarp();
                }
#pragma unroll
                for (int j = 0; j < 4; ++j) sts16(cell128(dst, lane, 4 * (c & 1) + j), pack<bf16>(v + 8 * j));
                if ((c & 1) || col + 32 >= N) {
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) {
                        tc::tma_store_2d(&maps.out[it.g], dst, col - 32 * (c & 1), row0);
                        tc::bulk_commit();
                    }
                    turn = turn + 1 == BOXES ? 0 : turn + 1;
                }
            } else if constexpr (MODE == UP && SPACE < 3 * BOX32) {
                // two boxes: a and b, then act in the first of them; act alone takes them in turn
                if (p.u) {
                    if (lane == 0) tc::bulk_wait_read<0>();
                    __syncwarp();
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        sts16(cell64(box, lane, j), pack<bf16>(v + 8 * j));
                        sts16(cell64(box + BOX32, lane, j), pack<bf16>(g + 8 * j));
                    }
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) {
                        tc::tma_store_2d(&maps.u_a, box, col, row0);
                        tc::tma_store_2d(&maps.u_b, box + BOX32, col, row0);
                        tc::bulk_commit();
                    }
                }
#pragma unroll
                for (int e = 0; e < 32; ++e) v[e] = v[e] * sigmoid_fast(v[e]) * g[e];
                const uint32_t dst = p.u ? box : box + turn * BOX32;
                if (lane == 0) {
                    if (p.u)
                        tc::bulk_wait_read<0>();
                    else
                        tc::bulk_wait_read<1>();
                }
                __syncwarp();
#pragma unroll
                for (int j = 0; j < 4; ++j) sts16(cell64(dst, lane, j), pack<bf16>(v + 8 * j));
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) {
                    tc::tma_store_2d(&maps.out[it.g], dst, col, row0);
                    tc::bulk_commit();
                }
                turn ^= 1;
            } else if constexpr (MODE == UP) {
                if (lane == 0) tc::bulk_wait_read<0>();
                __syncwarp();
                if (p.u) {
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        sts16(cell64(box, lane, j), pack<bf16>(v + 8 * j));
                        sts16(cell64(box + BOX32, lane, j), pack<bf16>(g + 8 * j));
                    }
                }
#pragma unroll
                for (int e = 0; e < 32; ++e) v[e] = v[e] * sigmoid_fast(v[e]) * g[e];
#pragma unroll
                for (int j = 0; j < 4; ++j) sts16(cell64(box + 2 * BOX32, lane, j), pack<bf16>(v + 8 * j));
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) {
                    if (p.u) {
                        tc::tma_store_2d(&maps.u_a, box, col, row0);
                        tc::tma_store_2d(&maps.u_b, box + BOX32, col, row0);
                    }
                    tc::tma_store_2d(&maps.out[it.g], box + 2 * BOX32, col, row0);
                    tc::bulk_commit();
                }
            } else {
                if (c % SETS == 0) {
                    ok = __all_sync(0xffffffffu, mbar_wait_bounded(u_bar, u_phase, kWaitLimit));
                    if (!ok) {
                        raise_abort(b, 64u);
                        break;
                    }
                    u_phase ^= 1u;
                    u_pending = false;
                }
                const uint32_t set = box + (c % SETS) * 3 * BOX32;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const uint32_t ca = cell64(set, lane, j), cb = cell64(set + BOX32, lane, j);
                    float fa[8], fb[8];
                    unpack<bf16>(lds16(ca), fa);
                    unpack<bf16>(lds16(cb), fb);
#pragma unroll
                    for (int e = 0; e < 8; ++e) dact_one(v[8 * j + e], fa[e], fb[e]);
                    sts16(ca, pack<bf16>(fa));
                    sts16(cb, pack<bf16>(fb));
                    sts16(cell64(set + 2 * BOX32, lane, j), pack<bf16>(v + 8 * j));
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) {
                    tc::tma_store_2d(&maps.du_a, set, col, row0);
                    tc::tma_store_2d(&maps.du_b, set + BOX32, col, row0);
                    if (c0.out) tc::tma_store_2d(&maps.out[it.g], set + 2 * BOX32, col, row0);
                    tc::bulk_commit();
                }
                if ((c + 1) % SETS == 0 && c + 1 < CH && col + 32 < N) fetch_u(col + 32);
            }
        }
        tc::fence_before_sync();
        __syncwarp();
        if (lane == 0) {
            const uint32_t e = smem_u32(&b->acc_empty[ab]);
            if (T::PAIRED)
                tc::mbar_arrive_cluster(tc::mapa(e, 0));
            else
                tc::mbar_arrive(e);
        }
    }
    // copies into this warp's boxes, and the reads of those out of them, end before its CTA does
    if (MODE == DACT && u_pending && !mbar_wait_bounded(u_bar, u_phase, kWaitLimit)) atomicOr(&g_error, 64u);
    if (lane == 0) tc::bulk_wait_read<0>();
    __syncwarp();
}

template <int MODE, bool B_MN, int S>
__global__ void __launch_bounds__(block_threads(MODE, S), 1)
    k_product(const __grid_constant__ Maps maps, const __grid_constant__ Params p)
{
    using T = Tile<S>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* ring = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    uint8_t* staging = ring + (size_t)stages(MODE, S) * T::STAGE_BYTES;
    Bars* b = reinterpret_cast<Bars*>(staging + epi_bytes(MODE, S));
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    Where w;
    w.rank = T::PAIRED ? tc::cluster_rank() : 0u;
    w.worker = T::PAIRED ? blockIdx.x / 2 : blockIdx.x;
    w.n_workers = T::PAIRED ? gridDim.x / 2 : gridDim.x;

    if (threadIdx.x == 0) {
#pragma unroll
        for (int i = 0; i < stages(MODE, S); ++i) {
            mbar_init(smem_u32(&b->full[i]), 1);
            mbar_init(smem_u32(&b->empty[i]), 1);
            b->peer_last[i] = -1;
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            mbar_init(smem_u32(&b->acc_full[i]), 1);
            mbar_init(smem_u32(&b->acc_empty[i]), (T::PAIRED ? 2 : 1) * epi_warps(MODE, S));
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) mbar_init(smem_u32(&b->u_full[i]), 1);
        mbar_init(smem_u32(&b->drain), 1);
        b->abort = 0;
        mbar_fence_init();
        for (int i = 0; i < p.n; ++i) {
            tc::prefetch_tmap(&maps.a[i]);
            tc::prefetch_tmap(&maps.b[i]);
        }
    }
    if (warp == 1) {
        if constexpr (T::PAIRED) {
            tc::tmem_alloc_pair(smem_u32(&b->tmem_base), T::TMEM_COLS);
            tc::tmem_relinquish_pair();
        } else {
            tc::tmem_alloc(smem_u32(&b->tmem_base), T::TMEM_COLS);
            tc::tmem_relinquish();
        }
    }
    tc::fence_before_sync();
    __syncthreads();
    if constexpr (T::PAIRED) tc::cluster_sync();  // both CTAs' barriers exist before any remote arrival
    tc::fence_after_sync();

    griddep_launch();
    griddep_wait();
    if (warp == 0) {
        if (lane == 0) run_producer<MODE, B_MN, S>(maps, p, ring, b, w);
    } else if (warp == 1) {
        if (lane == 0 && w.rank == 0) run_mma<MODE, B_MN, S>(p, ring, b, w);
    } else {
        run_epilogue<MODE, S>(maps, p, smem_u32(staging), b, w);
    }

    tc::fence_before_sync();
    __syncthreads();
    if constexpr (T::PAIRED) {
        tc::cluster_sync();  // the leader's MMAs have drained; the peer's last phases are in peer_last
        if (w.rank == 0 && threadIdx.x == 0) {
#pragma unroll
            for (int i = 0; i < stages(MODE, S); ++i) {
                const int32_t ph = b->peer_last[i];
                if (ph >= 0 && !mbar_wait_bounded(smem_u32(&b->full[i]), (uint32_t)ph, kWaitLimit))
                    atomicOr(&g_error, 2u);
            }
        }
        tc::cluster_sync();  // every copy into either CTA has landed
    }
    if (warp == 1) {
        tc::fence_after_sync();
        if constexpr (T::PAIRED)
            tc::tmem_dealloc_pair(b->tmem_base, T::TMEM_COLS);
        else
            tc::tmem_dealloc(b->tmem_base, T::TMEM_COLS);
    }
}

// Adds the pieces of the streamed tiles in the order of K and applies the epilogue.  One tile
// a blockIdx.y; a warp takes 4 rows x 8 groups of 16 columns, so that slots are read in runs
// of 128 bytes and rows are written in runs of 256.
template <int MODE, int S> __global__ void __launch_bounds__(256) k_join(const __grid_constant__ Params p)
{
    constexpr int TM = Tile<S>::M, TN = Tile<S>::N, WIDTH = MODE == UP ? TN / 2 : TN, GROUPS = WIDTH / 16;
    griddep_launch();
    griddep_wait();
    int64_t tile = blockIdx.y, first = 0;  // this tile's K among the rest's
    int g = 0;
    for (; tile >= p.g[g].tiles - p.g[g].whole; ++g) {
        const int64_t n = p.g[g].tiles - p.g[g].whole;
        tile -= n;
        first += n * p.g[g].kblocks;
    }
    const Product& c0 = p.g[g];
    first += tile * c0.kblocks;
    const int64_t w0 = first / p.piece_kb, w1 = (first + c0.kblocks - 1) / p.piece_kb;
    if (w0 == w1) return;  // the whole tile was one worker's
    int32_t m_blk, n_blk;
    tile_at(c0.whole + tile, c0, m_blk, n_blk);
    const int rows = (int)min((int64_t)TM, (int64_t)c0.M - (int64_t)m_blk * TM);
    const int lane = threadIdx.x & 31;
    constexpr int ACROSS = GROUPS < 8 ? GROUPS : 8, STEPS = GROUPS / ACROSS;
    for (int i = (blockIdx.x * blockDim.x + threadIdx.x) >> 5; i < (rows + 3) / 4 * STEPS;
         i += gridDim.x * blockDim.x >> 5) {
        if (lane >= 4 * ACROSS) break;
        const int r = (i / STEPS) * 4 + (lane & 3), c = (i % STEPS) * ACROSS + (lane >> 2);
        const int64_t row = (int64_t)m_blk * TM + r;
        const int32_t col = n_blk * WIDTH + 16 * c;
        const int n = inside(col, c0.N);
        if (r >= rows || n == 0) continue;
        float v[16] = {}, g[16] = {};
#pragma unroll 2
        for (int64_t w = w0; w <= w1; ++w) {
            const int64_t slot = 2 * w + (w * p.piece_kb <= first ? 1 : 0);
            const float* q = p.slots + ((slot * (TN / 8) + 2 * c) * TM + r) * 8;
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                float f[8];
                unpack<float>(ld_plain(q + j * TM * 8), f);
                unpack<float>(ld_plain(q + j * TM * 8 + 4), f + 4);
#pragma unroll
                for (int e = 0; e < 8; ++e) v[8 * j + e] += f[e];
                if constexpr (MODE == UP) {
                    const float* qb = q + (WIDTH / 8 + j) * TM * 8;
                    unpack<float>(ld_plain(qb), f);
                    unpack<float>(ld_plain(qb + 4), f + 4);
#pragma unroll
                    for (int e = 0; e < 8; ++e) g[8 * j + e] += f[e];
                }
            }
        }
        uint4 ua[2], ub[2];
        if constexpr (MODE == DACT) {
            get16(p.u + row * p.ld_u + col, ua[0], ua[1], n, c0.wide);
            get16(p.u + row * p.ld_u + c0.N + col, ub[0], ub[1], n, c0.wide);
        }
        finish16<MODE>(p, c0, row, col, n, v, g, ua, ub);
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

// Tensor map of an operand in the 128-byte swizzle; what lies outside the tensor reads as zero.  Sets
// *both where one copy brings all rows of a CTA:
//   K contiguous: boxes of 64 K x `rows` rows, those of a CTA or, where the only tile has fewer, as many as it has (rows
//   of the shared-memory tile that nothing is copied to give accumulator rows that nothing reads);
//   64 where the halves are apart;
//   M (N) contiguous: the 64-wide column blocks as a third dimension, boxes of 64 x 64 x rows / 64, where the width
//   is a multiple of 64, so that no block reaches into the next row.
bool make_map(CUtensorMap* m, const Mat& t, bool mn, int32_t rows, int32_t* both)
{
    auto fn = encode_fn();
    if (!fn) return false;
    const bool blocks = mn && t.cols % ffn::BOX == 0;
    *both = mn ? blocks : rows != ffn::BOX;
    const cuuint64_t dims[3] = {(cuuint64_t)(blocks ? ffn::BOX : t.cols), (cuuint64_t)t.rows,
                                (cuuint64_t)(t.cols / ffn::BOX)};
    const cuuint64_t strides[2] = {(cuuint64_t)t.ld * 2, ffn::BOX * 2};
    const cuuint32_t box[3] = {ffn::BOX, (cuuint32_t)(mn ? ffn::BOX : rows), (cuuint32_t)(rows / ffn::BOX)};
    const cuuint32_t estr[3] = {1, 1, 1};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, blocks ? 3 : 2, const_cast<void*>(t.p), dims, strides, box, estr,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Tensor map of what an epilogue copies: boxes of 32 rows of `cols` columns (32 or 64).
bool out_map(CUtensorMap* m, const void* p, int64_t rows, int64_t width, int64_t ld, int32_t cols)
{
    auto fn = encode_fn();
    if (!fn) return false;
    const cuuint64_t dims[2] = {(cuuint64_t)width, (cuuint64_t)rows};
    const cuuint64_t strides[1] = {(cuuint64_t)ld * 2};
    const cuuint32_t box[2] = {(cuuint32_t)cols, 32};
    const cuuint32_t estr[2] = {1, 1};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(p), dims, strides, box, estr,
              CU_TENSOR_MAP_INTERLEAVE_NONE, cols == 64 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
              CU_TENSOR_MAP_L2_PROMOTION_NONE, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// The maps of a product's epilogue.
bool out_maps(ffn::Maps& m, int i, const FfnProduct& g)
{
    auto one = [&](CUtensorMap* t, const void* p, int64_t ld, int32_t cols) {
        return !p || out_map(t, p, g.M, g.N, ld, cols);
    };
    const bf16 *u = static_cast<const bf16*>(g.u), *du = static_cast<const bf16*>(g.du);
    if (g.epi == FFN_STORE) return g.out_f32 || g.accumulate || one(&m.out[i], g.out, g.ld_out, 64);
    return one(&m.out[i], g.out, g.ld_out, 32) && one(&m.u_a, u, g.ld_u, 32) && one(&m.u_b, u ? u + g.N : u, g.ld_u, 32) &&
           one(&m.du_a, du, g.ld_du, 32) && one(&m.du_b, du ? du + g.N : du, g.ld_du, 32);
}

// Tile shape of a launch and how its last tiles are shared out, from its products' sizes alone.
struct Plan {
    int shape, n;
    int32_t pieces, piece_kb;
    struct One {
        int32_t tiles_m, tiles_n, kblocks;
        int64_t tiles, whole;
    } g[ffn::MAX_PRODUCTS];
    int64_t rest, rest_kb;
};

// What a shape costs, in microseconds, from runs of all shapes at some twenty sizes (d 64 to
// 5120, width 64 to 13,824, 64 to 30,000 tokens): the launch with its first fill and last drain, a k-block with
// few workers and with all of them busy (the copies from L2 then bound SINGLE and PAIR), the least
// time of a tile (its epilogue), and what a tile adds to that where the epilogue stands alone.
struct ShapeCost {
    double launch, kb_few, kb_busy, tile, alone;
};
constexpr ShapeCost kCost[3] = {{4.0, 0.25, 0.43, 1.0, 0.0}, {6.0, 0.31, 0.43, 2.5, 0.0}, {9.0, 0.60, 0.70, 2.5, 4.0}};

// The cheaper way to share out the last tiles of a shape; returns the launch's cost.
double share_out(Plan& r, const ShapeCost& c, int64_t workers, double slot_mb)
{
    const auto kb_time = [&](int64_t active) {
        return std::max(c.kb_few, c.kb_busy * (double)std::min(active, workers) / (double)workers);
    };
    double cost = c.launch;
    r.rest = r.rest_kb = 0;
    r.pieces = r.piece_kb = 0;
    for (int i = 0; i < r.n; ++i) {
        Plan::One& g = r.g[i];
        const int64_t rest = g.tiles % workers;
        g.whole = g.tiles - rest;
        cost += (double)(g.tiles / workers) * (std::max(g.kblocks * c.kb_busy, c.tile) + c.alone);
        r.rest += rest;
        r.rest_kb += rest * g.kblocks;
    }
    if (!r.rest) return cost;
    // whole tiles, the longest first: a round takes as long as its first tile
    double best = 0;
    int64_t seen = 0, round = 0;
    for (int i = 0; i < r.n; ++i) {
        seen += r.g[i].tiles - r.g[i].whole;
        for (; round < seen; round += workers)
            best += std::max(r.g[i].kblocks * kb_time(r.rest - round), c.tile) + c.alone;
    }
    best += c.tile;
    const int64_t least = (r.rest_kb + workers - 1) / workers;
    for (int s : {2, 3, 4, 6, 8, 12, 16, 24, 32}) {
        if (s > r.g[0].kblocks) break;
        const int64_t kb = std::max<int64_t>(least, (r.g[0].kblocks + s - 1) / s), pieces = (r.rest_kb + kb - 1) / kb;
        // the join: its launch, a tile's pieces one after another, the slots written and read
        const double join = 3.0 + 0.15 * (double)((pieces + r.rest - 1) / r.rest) + 2.0 * slot_mb * (double)pieces / 5.0;
        const double t = (double)kb * kb_time(pieces) + c.tile + c.alone + join;
        if (t < best) {
            best = t;
            r.pieces = (int32_t)pieces;
            r.piece_kb = (int32_t)kb;
        }
    }
    return cost + best;
}

// The products of a launch must be in the order of K, longest first.
Plan plan(const FfnProduct* p, int n)
{
    Plan best{};
    double cost = 0;
    int64_t most = 0;
    for (int i = 0; i < n; ++i) most = std::max(most, p[i].M);
    for (int shape = ffn::SINGLE; shape <= ffn::WIDE; ++shape) {
        if ((shape == ffn::PAIR && most <= 128) || (shape == ffn::WIDE && (most <= 256 || p[0].epi == FFN_DACT))) continue;
        Plan r{};
        r.shape = shape;
        r.n = n;
        const int64_t tm = shape == ffn::SINGLE ? 128 : shape == ffn::PAIR ? 256 : 512;
        const int64_t tw = shape == ffn::SINGLE ? 128 : 256, tn = p[0].epi == FFN_UP ? tw / 2 : tw;
        for (int i = 0; i < n; ++i) {
            Plan::One& g = r.g[i];
            g.kblocks = (int32_t)((p[i].K + ffn::BK - 1) / ffn::BK);
            g.tiles_m = (int32_t)((p[i].M + tm - 1) / tm);
            g.tiles_n = (int32_t)((p[i].N + tn - 1) / tn);
            g.tiles = (int64_t)g.tiles_m * g.tiles_n;
        }
        const double slot_mb = (double)std::min(most, tm) * (double)tw * 4e-6;
        const double c = share_out(r, kCost[shape], shape == ffn::SINGLE ? ffn::B200_SMS : ffn::B200_SMS / 2, slot_mb);
        if (!cost || c < cost) {
            best = r;
            cost = c;
        }
    }
    return best;
}

template <int MODE, bool B_MN, int S>
cudaError_t launch_kernel(const ffn::Maps& maps, const ffn::Params& p, bool after, cudaStream_t s)
{
    auto kern = ffn::k_product<MODE, B_MN, S>;
    constexpr bool PAIRED = ffn::Tile<S>::PAIRED;
    constexpr int kMaxDevices = 64;
    static int workers_dev[kMaxDevices] = {};  // resident CTAs or pairs, once the attribute is set
    static std::mutex mu;
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= kMaxDevices) return cudaErrorInvalidDevice;
    cudaLaunchAttribute la[2];
    la[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    la[0].val.programmaticStreamSerializationAllowed = 1;
    la[1].id = cudaLaunchAttributeClusterDimension;
    la[1].val.clusterDim.x = 2;
    la[1].val.clusterDim.y = 1;
    la[1].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.blockDim = dim3(ffn::block_threads(MODE, S));
    cfg.dynamicSmemBytes = ffn::smem_bytes<MODE, S>();
    cfg.stream = s;
    cfg.attrs = after ? la : la + 1;
    cfg.numAttrs = (after ? 1 : 0) + (PAIRED ? 1 : 0);
    int64_t workers;
    {
        std::lock_guard<std::mutex> lk(mu);
        if (!workers_dev[dev]) {
            e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)ffn::smem_bytes<MODE, S>());
            if (e != cudaSuccess) return e;
            int n = sm_count();
            if (PAIRED) {
                cudaLaunchConfig_t q = cfg;
                q.attrs = la + 1;
                q.numAttrs = 1;
                q.gridDim = dim3(2 * (sm_count() / 2));
                if (cudaOccupancyMaxActiveClusters(&n, kern, &q) != cudaSuccess || n < 1) n = sm_count() / 2;
            }
            workers_dev[dev] = n;
        }
        workers = workers_dev[dev];
    }
    int64_t items = p.pieces ? p.pieces : p.rest_tiles;
    for (int i = 0; i < p.n; ++i) items = std::max(items, p.g[i].whole);
    workers = std::min(items, workers);
    cfg.gridDim = dim3((unsigned)(PAIRED ? 2 * workers : workers));
    return cudaLaunchKernelEx(&cfg, kern, maps, p);
}

template <int MODE, int S> cudaError_t launch_join(const ffn::Params& p, cudaStream_t s)
{
    // a warp takes 4 rows x up to 128 columns of one tile
    int64_t most = 0;
    for (int i = 0; i < p.n; ++i) most = std::max<int64_t>(most, p.g[i].M);
    const int64_t warps = (std::min<int64_t>(most, ffn::Tile<S>::M) + 3) / 4 *
                          std::max(1, ffn::Tile<S>::N / (MODE == ffn::UP ? 256 : 128));
    cudaLaunchAttribute la[1];
    la[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    la[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.blockDim = dim3(256);
    cfg.gridDim = dim3((unsigned)((warps + 7) / 8), (unsigned)p.rest_tiles);
    cfg.stream = s;
    cfg.attrs = la;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, ffn::k_join<MODE, S>, p);
}

template <int MODE, bool B_MN, int S>
cudaError_t launch_both(const ffn::Maps& maps, const ffn::Params& p, bool after, cudaStream_t s)
{
    const cudaError_t e = launch_kernel<MODE, B_MN, S>(maps, p, after, s);
    return e != cudaSuccess || !p.pieces ? e : launch_join<MODE, S>(p, s);
}

template <int MODE, bool B_MN>
cudaError_t launch_shape(int shape, const ffn::Maps& maps, const ffn::Params& p, bool after, cudaStream_t s)
{
    if (shape == ffn::SINGLE) return launch_both<MODE, B_MN, ffn::SINGLE>(maps, p, after, s);
    if (shape == ffn::PAIR) return launch_both<MODE, B_MN, ffn::PAIR>(maps, p, after, s);
    if constexpr (MODE != ffn::DACT) return launch_both<MODE, B_MN, ffn::WIDE>(maps, p, after, s);
    return cudaErrorInvalidValue;
}

bool on32(const void* p, int64_t ld, int64_t esz) { return (reinterpret_cast<uintptr_t>(p) & 31u) == 0 && ld * esz % 32 == 0; }

}  // namespace

size_t ffn_slot_bytes(int64_t rows)
{
    // two slots a worker: 148 CTAs with 128 x 128, 74 pairs with 256 x 256 or 512 x 256
    const size_t one = rows <= 128 ? 2 * 128 * 128 : rows <= 256 ? 256 * 256 : 512 * 256;
    return 2 * (ffn::B200_SMS / 2) * one * 4;
}

cudaError_t launch_ffn_products(FfnProduct* g, int n, bool after, cudaStream_t s)
{
    std::sort(g, g + n, [](const FfnProduct& a, const FfnProduct& b) { return a.K > b.K; });
    const Plan r = plan(g, n);
    ffn::Maps maps;
    ffn::Params p{};
    p.n = n;
    p.pieces = r.pieces;
    p.piece_kb = r.piece_kb;
    p.rest_tiles = r.rest;
    p.rest_kb = r.rest_kb;
    p.u = static_cast<bf16*>(g[0].u);
    p.ld_u = g[0].ld_u;
    p.du = static_cast<bf16*>(g[0].du);
    p.ld_du = g[0].ld_du;
    p.slots = g[0].slots;
    for (int i = 0; i < n; ++i) {
        ffn::Product& c = p.g[i];
        if (r.g[i].tiles >= (int64_t)1 << 31) {
            record_error("the product has more than 2^31 tiles");
            return cudaErrorInvalidValue;
        }
        int32_t a_rows = r.shape == ffn::WIDE ? 2 * ffn::BM : ffn::BM;
        if (r.shape == ffn::SINGLE && !g[i].a_mn && r.g[i].tiles_m == 1) a_rows = (int32_t)((g[i].M + 7) / 8 * 8);
        if (a_rows == ffn::BOX) a_rows += 8;  // 64 means two boxes
        c.stage_bytes = a_rows * ffn::BK * 2 + ffn::BM * ffn::BK * 2;
        const int32_t b_rows = g[i].epi == FFN_UP && r.shape == ffn::SINGLE ? ffn::BOX : ffn::BM;
        if (!make_map(&maps.a[i], g[i].a, g[i].a_mn, a_rows, &c.a_blocks) ||
            !make_map(&maps.b[i], g[i].b, g[i].b_mn, b_rows, &c.b_blocks) || !out_maps(maps, i, g[i])) {
            record_error("tensor map encoding failed (cuTensorMapEncodeTiled unavailable or refused the layout)");
            return cudaErrorInvalidValue;
        }
        c.M = (int32_t)g[i].M;
        c.N = (int32_t)g[i].N;
        c.kblocks = r.g[i].kblocks;
        c.tiles_m = r.g[i].tiles_m;
        c.tiles_n = r.g[i].tiles_n;
        c.tiles = r.g[i].tiles;
        c.whole = r.g[i].whole;
        c.a_mn = g[i].a_mn;
        c.out = g[i].out;
        c.ld_out = g[i].ld_out;
        c.out_f32 = g[i].out_f32;
        c.accumulate = g[i].accumulate;
        c.wide = on32(c.out, c.ld_out, c.out_f32 ? 4 : 2) && on32(p.u, p.ld_u, 2) && on32(p.du, p.ld_du, 2) &&
                 (g[i].epi == FFN_STORE || c.N % 16 == 0);
    }
    if (g[0].epi == FFN_UP) return launch_shape<ffn::UP, false>(r.shape, maps, p, after, s);
    if (g[0].epi == FFN_DACT) return launch_shape<ffn::DACT, true>(r.shape, maps, p, after, s);
    if (g[0].b_mn) return launch_shape<ffn::STORE, true>(r.shape, maps, p, after, s);
    return launch_shape<ffn::STORE, false>(r.shape, maps, p, after, s);
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
