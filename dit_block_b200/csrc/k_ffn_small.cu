// k_ffn_small.cu -- the gated feed-forward block for a few tokens (a denoising server's
// smallest batches, single tokens): y = (silu(x Wg^T) * (x Wu^T)) Wd^T, and its backward pass.
//
// Bound by the weights' bytes: 6 * d * inner of them against some tens of kilobytes of
// everything else.  The weights are streamed once, straight from HBM to registers in rows of
// consecutive 16-byte vectors (the tiles of k_ffn.cu would read each row 128 bytes at a time
// and multiply 128 rows of mostly nothing), and multiplied by m16n8k16 tensor instructions:
// 16 rows of weights by 8 tokens.  Which k of a 32-wide chunk a register stands for does not
// matter as long as both operands agree, so that a lane's 16-byte vector of a weight row and
// of a token's row are used as they come.
//
// A CTA takes up to 32 tokens and 16 rows of weights (up projection: 8 of the gated half and the 8 of the other
// half that they meet, so that a thread ends up with a and b of the same value), its warps a
// share of K each; the shares are added through shared memory in the order of the warps.
// Where that leaves most SMs without work (few outputs, long sums), a cluster of up to eight CTAs
// shares the sums, which are added through distributed shared memory in the order of k (200 x 13000, one
// token: 14.4 -> 8.7 us; its backward pass 45 -> 16).  The second kernel is launched to overlap the first one's
// end (programmatic dependent launch) and starts by loading weights, which do not depend on it.
//
// The backward pass for a few tokens in the same way: one kernel for d_act, du and act, one for dx and
// the weight gradients, whose products over the tokens need no shared memory.  Bound by the launches and a
// few loads that wait for each other (d 256, width 512, 32 tokens: 8.1 us, 15.8 as tiles of
// k_ffn.cu), and by HBM at the block's full size (one token: 181 us for 850 MB, 4.7 TB/s).
#include <cuda_bf16.h>

#include "common.cuh"
#include "launch.h"
#include "tcgen05.cuh"
#include "train.h"

namespace sol {
namespace ffn_small {

constexpr int CHUNK = 32;  // k of one step: a lane's 16-byte vector from each of 4 lanes a row
// Chunks whose loads a warp has in flight together, and warps an SM: 2 x 32 measured fastest at d
// 5120, width 13,824, one token (70.3 us = 6.04 TB/s; 4 x 32 81.8, 4 x 16 84.6, 8 x 24 97.9: they spill).
constexpr int U = 2, SM_WARPS = 32;

struct Params {
    const bf16* x;  // tokens: x (up) or act (down)
    int64_t ld_x;
    const bf16* w;
    int64_t ld_w;
    bf16* out;  // act or y
    int64_t ld_out;
    bf16* u;  // up: kept u or NULL
    int64_t ld_u;
    int32_t T, rows, K;  // tokens; outputs a token (inner or d); inner dimension
    int32_t split_log;   // 2^split_log CTAs (a cluster) share the K of the same outputs
};

// How many CTAs share the k of an output, as a power of two: more than one while they are at most `few`, and
// while each still has `least` of it.
int32_t split_of(int64_t ctas, int64_t few, int64_t k, int64_t least)
{
    int32_t log = 0;
    while (log < 3 && ctas << log <= few && k >= (2 * least) << log) ++log;
    return log;
}

// The same shared-memory word of CTA `rank` of the cluster.
__device__ __forceinline__ float peer(const float& x, int rank)
{
    float v;
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(tc::mapa(smem_u32(&x), rank)) : "memory");
    return v;
}

__device__ __forceinline__ void mma(float* c, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1)
{
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
                 "{%0, %1, %2, %3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint4 ld_weights(const bf16* p)
{
    uint4 v;
    asm volatile("ld.global.nc.L1::no_allocate.L2::256B.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p));
    return v;
}

template <bool UP, int NT, int WARPS, bool SPLIT>
__global__ void __launch_bounds__(32 * WARPS, (NT > 2 ? SM_WARPS / 2 : SM_WARPS) / WARPS) k_small(const __grid_constant__ Params p)
{
    constexpr int OUT = UP ? 8 : 16;  // outputs a token of this CTA
    __shared__ float red[WARPS][16][8 * NT + 1];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const int32_t split = SPLIT ? 1 << p.split_log : 1, rank = (int)blockIdx.x & (split - 1);
    const int32_t j0 = (SPLIT ? (int)blockIdx.x >> p.split_log : (int)blockIdx.x) * OUT;
    const int32_t t0 = blockIdx.y * 8 * NT, T = min(p.T - t0, 8 * NT);  // this CTA's tokens
    const bf16* px = p.x + t0 * p.ld_x;
    // rows g and g + 8 of the tensor instruction
    const int32_t ra = j0 + g, rb = UP ? p.rows + j0 + g : j0 + 8 + g;
    const bool la = ra < p.rows, lb = UP ? la : rb < p.rows;
    const int32_t chunks = (p.K + CHUNK - 1) / CHUNK, share = (chunks + split * WARPS - 1) / (split * WARPS);
    const int32_t c0 = min((rank * WARPS + warp) * share, chunks), c1 = min(c0 + share, chunks);
    const bf16* wa = p.w + ra * p.ld_w + 8 * t;
    const bf16* wb = p.w + rb * p.ld_w + 8 * t;
    const uint4 zero = make_uint4(0, 0, 0, 0);
    float acc[NT][4] = {};
    uint4 a[U], b[U];

    auto weights = [&](int32_t c) {
#pragma unroll
        for (int i = 0; i < U; ++i) {
            const int32_t k = (c + i) * CHUNK;
            const bool in = c + i < c1 && k + 8 * t < p.K;
            a[i] = in && la ? ld_weights(wa + k) : zero;
            b[i] = in && lb ? ld_weights(wb + k) : zero;
        }
    };
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    weights(c0);
    asm volatile("griddepcontrol.wait;" ::: "memory");  // the tokens are the previous kernel's
    for (int32_t c = c0; c < c1; c += U) {
        if (c > c0) weights(c);
#pragma unroll
        for (int i = 0; i < U; ++i) {
            const int32_t k = (c + i) * CHUNK + 8 * t;
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                const uint4 x = c + i < c1 && k < p.K && 8 * n + g < T
                                    ? *reinterpret_cast<const uint4*>(px + (8 * n + g) * p.ld_x + k)
                                    : zero;
                mma(acc[n], a[i].x, b[i].x, a[i].y, b[i].y, x.x, x.y);
                mma(acc[n], a[i].z, b[i].z, a[i].w, b[i].w, x.z, x.w);
            }
        }
    }
    // accumulator: rows g, g + 8, tokens 2t, 2t + 1 of each group of eight
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        red[warp][g][8 * n + 2 * t] = acc[n][0];
        red[warp][g][8 * n + 2 * t + 1] = acc[n][1];
        red[warp][g + 8][8 * n + 2 * t] = acc[n][2];
        red[warp][g + 8][8 * n + 2 * t + 1] = acc[n][3];
    }
    __syncthreads();
    if constexpr (SPLIT) {  // this CTA's sum, over its first warp's, for the cluster to read
        for (int i = threadIdx.x; i < 16 * T; i += 32 * WARPS) {
            float v = 0.f;
#pragma unroll
            for (int s = 0; s < WARPS; ++s) v += red[s][i % 16][i / 16];
            red[0][i % 16][i / 16] = v;
        }
        tc::cluster_sync();
    }
    for (int i = threadIdx.x; i < OUT * T; i += 32 * WARPS) {
        const int j = i % OUT, n = i / OUT;
        const int64_t row = t0 + n;
        if (j0 + j >= p.rows || (j & (split - 1)) != rank) continue;
        float v = 0.f, v2 = 0.f;
        if constexpr (SPLIT) {  // in the order of k
            for (int r = 0; r < split; ++r) {
                v += peer(red[0][j][n], r);
                if (UP) v2 += peer(red[0][j + 8][n], r);
            }
        } else {
#pragma unroll
            for (int s = 0; s < WARPS; ++s) {
                v += red[s][j][n];
                if (UP) v2 += red[s][j + 8][n];
            }
        }
        if (UP) {
            if (p.u) {
                p.u[row * p.ld_u + j0 + j] = __float2bfloat16_rn(v);
                p.u[row * p.ld_u + p.rows + j0 + j] = __float2bfloat16_rn(v2);
            }
            v = v / (1.f + __expf(-v)) * v2;
        }
        p.out[row * p.ld_out + j0 + j] = __float2bfloat16_rn(v);
    }
    if constexpr (SPLIT) tc::cluster_sync();  // the others may still be reading this CTA's sum
}

template <bool UP, int NT, int WARPS> cudaError_t launch(Params p, bool after, cudaStream_t s)
{
    const int32_t across = (p.rows + (UP ? 7 : 15)) / (UP ? 8 : 16), groups = (p.T + 8 * NT - 1) / (8 * NT);
    p.split_log = split_of((int64_t)across * groups, 74, p.K, CHUNK * 2 * WARPS);
    cudaLaunchAttribute la[3];
    la[0].id = la[2].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    la[0].val.programmaticStreamSerializationAllowed = la[2].val.programmaticStreamSerializationAllowed = after;
    la[1].id = cudaLaunchAttributeClusterDimension;
    la[1].val.clusterDim.x = 1u << p.split_log;
    la[1].val.clusterDim.y = la[1].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.blockDim = dim3(32 * WARPS);
    cfg.gridDim = dim3((unsigned)across << p.split_log, (unsigned)groups);
    cfg.stream = s;
    cfg.attrs = p.split_log ? la + 1 : la;
    cfg.numAttrs = (after ? 1 : 0) + (p.split_log ? 1 : 0);
    return cudaLaunchKernelEx(&cfg, p.split_log ? k_small<UP, NT, WARPS, true> : k_small<UP, NT, WARPS, false>, p);
}

// Sixteen warps a CTA where there is at most one CTA an SM, else eight.
template <bool UP> cudaError_t launch(const Params& p, bool after, cudaStream_t s)
{
    const bool few = (p.rows + (UP ? 7 : 15)) / (UP ? 8 : 16) <= 148;
    if (p.T <= 8) return few ? launch<UP, 1, 16>(p, after, s) : launch<UP, 1, 8>(p, after, s);
    if (p.T <= 16) return few ? launch<UP, 2, 16>(p, after, s) : launch<UP, 2, 8>(p, after, s);
    return few ? launch<UP, 4, 16>(p, after, s) : launch<UP, 4, 8>(p, after, s);
}

// ---------------------------------------------------------------------------------
// Backward.  Here the weights lie with the outputs' dimension contiguous and k from row to row: a
// lane loads the same few columns of four rows, and byte permutations pair up two rows as the
// tensor instruction wants them (a register holds two consecutive k).

constexpr int BACK_WARPS = 8, BACK_N = 32;  // warps of a CTA; outputs a token of one (of d_act or dx)
constexpr int BACK_FEW = 80;                // CTAs of a product up to which two share the k of an output
constexpr int GRAD_M = 64, GRAD_N = 32;     // a warp's tile of a weight gradient

struct Back {
    const bf16 *dy, *x, *u, *w_up, *w_down;
    int64_t ld_dy, ld_x, ld_u, ld_wu, ld_wd;
    bf16 *act, *du, *dx;
    void *dw_up, *dw_down;
    int64_t ld_dx, ld_dwu, ld_dwd;
    int32_t T, d, inner;
    int32_t out_f32, accumulate;
    int32_t dx_ctas, up_tiles, down_tiles;  // work of k_back_grads
    int32_t split_log;                      // 2^split_log CTAs (a cluster) share the k of the same outputs
};
template <int MT> using Red = float[BACK_WARPS][16 * MT][BACK_N + 1];

// Halfword `odd` of two words, the first in the lower half.
__device__ __forceinline__ uint32_t pair_up(uint32_t lower, uint32_t upper, int odd)
{
    return __byte_perm(lower, upper, odd ? 0x7632 : 0x5410);
}
__device__ __forceinline__ uint32_t word(const uint2& v, int i) { return i ? v.y : v.x; }
__device__ __forceinline__ uint32_t word(const uint4& v, int i) { return i < 2 ? (i ? v.y : v.x) : (i == 2 ? v.z : v.w); }

// x[T, K] . w[K, N] for columns [n0, n0 + BACK_N), a warp's share of K at a time: each warp's sum in red.  `rank`
// of the `split` CTAs of a cluster.  Register e of a lane's column group stands for column 4 * group + e.  `dependent`: x is written by
// the kernel before.
template <int MT, bool SPLIT>
__device__ __forceinline__ void rows_by_weights(Red<MT>& red, const bf16* w, int64_t ld_w, int32_t N, int32_t n0,
                                                const bf16* x, int64_t ld_x, int32_t T, int32_t K, int32_t rank, int32_t split,
                                                bool dependent)
{
    constexpr int U = 4;  // chunks in flight
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const int32_t chunks = (K + 15) / 16, share = (chunks + split * BACK_WARPS - 1) / (split * BACK_WARPS);
    const int32_t c0 = min((rank * BACK_WARPS + warp) * share, chunks), c1 = min(c0 + share, chunks);
    const int32_t n = n0 + 4 * g;
    const uint2 zero = make_uint2(0, 0);
    float acc[MT][4][4] = {};
    uint2 r[U][4];
    auto weights = [&](int32_t c) {
#pragma unroll
        for (int i = 0; i < U; ++i) {
            const int32_t k = (c + i) * 16 + 4 * t;
            const bool in = c + i < c1 && k < K && n < N;
#pragma unroll
            for (int q = 0; q < 4; ++q)
                r[i][q] = in ? __ldg(reinterpret_cast<const uint2*>(w + (int64_t)(k + q) * ld_w + n)) : zero;
        }
    };
    weights(c0);
    if (dependent) asm volatile("griddepcontrol.wait;" ::: "memory");
    for (int32_t c = c0; c < c1; c += U) {
        if (c > c0) weights(c);
#pragma unroll
        for (int i = 0; i < U; ++i) {
            const int32_t k = (c + i) * 16 + 4 * t;
            const bool in = c + i < c1 && k < K;
            uint2 a[MT][2];
#pragma unroll
            for (int m = 0; m < MT; ++m)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int row = 16 * m + 8 * h + g;
                    a[m][h] = in && row < T ? *reinterpret_cast<const uint2*>(x + row * ld_x + k) : zero;
                }
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const uint32_t b0 = pair_up(word(r[i][0], e / 2), word(r[i][1], e / 2), e & 1);
                const uint32_t b1 = pair_up(word(r[i][2], e / 2), word(r[i][3], e / 2), e & 1);
#pragma unroll
                for (int m = 0; m < MT; ++m) mma(acc[m][e], a[m][0].x, a[m][1].x, a[m][0].y, a[m][1].y, b0, b1);
            }
        }
    }
    // accumulator e: rows g, g + 8; the columns of groups 2t, 2t + 1
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int e = 0; e < 4; ++e)
#pragma unroll
            for (int v = 0; v < 4; ++v) red[warp][16 * m + g + 8 * (v >> 1)][8 * t + 4 * (v & 1) + e] = acc[m][e][v];
    __syncthreads();
    if (!SPLIT) return;
    // this CTA's sum, over its first warp's, for the cluster to read
    for (int row = warp; row < T; row += BACK_WARPS) {
        float v = 0.f;
#pragma unroll
        for (int s = 0; s < BACK_WARPS; ++s) v += red[s][row][lane];
        red[0][row][lane] = v;
    }
    tc::cluster_sync();
}
// An output's value, the sums in the order of k.
template <int MT, bool SPLIT> __device__ __forceinline__ float summed(Red<MT>& red, int row, int col, int split)
{
    float v = 0.f;
    if (!SPLIT) {
#pragma unroll
        for (int s = 0; s < BACK_WARPS; ++s) v += red[s][row][col];
    } else {
        for (int r = 0; r < split; ++r) v += peer(red[0][row][col], r);
    }
    return v;
}

// d_act = dy . W_down, and from it and u: du and act.
template <int MT, bool SPLIT> __global__ void __launch_bounds__(32 * BACK_WARPS) k_back_act(const __grid_constant__ Back p)
{
    const int32_t split = SPLIT ? 1 << p.split_log : 1, rank = (int)blockIdx.x & (split - 1);
    __shared__ Red<MT> red;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    constexpr int OWN = 16 * MT * BACK_N / (32 * BACK_WARPS);  // values of a thread
    const int32_t t0 = blockIdx.y * 16 * MT, T = min(p.T - t0, 16 * MT);  // this CTA's tokens
    const int32_t n0 = (SPLIT ? (int)blockIdx.x >> p.split_log : (int)blockIdx.x) * BACK_N, n = n0 + (threadIdx.x & 31);
    float a[OWN] = {}, b[OWN] = {};
#pragma unroll
    for (int i = 0; i < OWN; ++i) {
        const int row = (threadIdx.x >> 5) + i * BACK_WARPS;
        if (row < T && n < p.inner && (row & (split - 1)) == rank) {
            a[i] = __bfloat162float(p.u[(t0 + row) * p.ld_u + n]);
            b[i] = __bfloat162float(p.u[(t0 + row) * p.ld_u + p.inner + n]);
        }
    }
    rows_by_weights<MT, SPLIT>(red, p.w_down, p.ld_wd, p.inner, n0, p.dy + t0 * p.ld_dy, p.ld_dy, T, p.d, rank, split, false);
#pragma unroll
    for (int i = 0; i < OWN; ++i) {
        const int row = (threadIdx.x >> 5) + i * BACK_WARPS;
        if (row >= T || n >= p.inner || (row & (split - 1)) != rank) continue;
        const float d = summed<MT, SPLIT>(red, row, threadIdx.x & 31, split);
        const float s = 1.f / (1.f + __expf(-a[i])), as = a[i] * s;
        const int64_t at = (int64_t)(t0 + row) * p.inner;
        p.du[2 * at + n] = __float2bfloat16_rn(d * b[i] * s * fmaf(a[i], 1.f - s, 1.f));
        p.du[2 * at + p.inner + n] = __float2bfloat16_rn(d * as);
        p.act[at + n] = __float2bfloat16_rn(as * b[i]);
    }
    if (SPLIT) tc::cluster_sync();  // the others may still be reading this CTA's sum
}

// Eight values of a weight gradient's row, from `at` on.
__device__ __forceinline__ void put_grad(const Back& p, void* out, int64_t at, const float* v)
{
    float s[8];
    if (p.out_f32) {
        float* dst = static_cast<float*>(out) + at;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            unpack<float>(p.accumulate ? ld_plain(dst + 4 * h) : make_uint4(0, 0, 0, 0), s);
            *reinterpret_cast<float4*>(dst + 4 * h) =
                make_float4(s[0] + v[4 * h], s[1] + v[4 * h + 1], s[2] + v[4 * h + 2], s[3] + v[4 * h + 3]);
        }
    } else {
        bf16* dst = static_cast<bf16*>(out) + at;
        unpack<bf16>(p.accumulate ? ld_plain(dst) : make_uint4(0, 0, 0, 0), s);  // added in fp32, rounded once
#pragma unroll
        for (int e = 0; e < 8; ++e) s[e] += v[e];
        *reinterpret_cast<uint4*>(dst) = pack<bf16>(s);
    }
}

// One warp: a tile of GRAD_M x GRAD_N of a^T . b over the tokens; a [T, M], b [T, N].
__device__ __forceinline__ void grad_tile(const Back& p, int32_t tile, const bf16* a, int64_t ld_a, int32_t M, const bf16* b,
                                          int64_t ld_b, int32_t N, void* out, int64_t ld_out)
{
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const int32_t across = (N + GRAD_N - 1) / GRAD_N;
    const int32_t m0 = tile / across * GRAD_M + 8 * g, n0 = tile % across * GRAD_N;
    const bool in_m = m0 < M, in_n = n0 + 4 * g < N;
    float acc[4][4][4] = {};
    for (int32_t k0 = 0; k0 < p.T; k0 += 16) {
        uint4 ra[4];
        uint2 rb[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const int32_t k = k0 + 4 * t + q;
            ra[q] = k < p.T && in_m ? *reinterpret_cast<const uint4*>(a + k * ld_a + m0) : make_uint4(0, 0, 0, 0);
            rb[q] = k < p.T && in_n ? *reinterpret_cast<const uint2*>(b + k * ld_b + n0 + 4 * g) : make_uint2(0, 0);
        }
#pragma unroll
        for (int f = 0; f < 4; ++f) {  // row groups: rows 8 * group + 2f, and 8 * group + 2f + 1 as the upper eight
            const uint32_t a0 = pair_up(word(ra[0], f), word(ra[1], f), 0), a1 = pair_up(word(ra[0], f), word(ra[1], f), 1);
            const uint32_t a2 = pair_up(word(ra[2], f), word(ra[3], f), 0), a3 = pair_up(word(ra[2], f), word(ra[3], f), 1);
#pragma unroll
            for (int e = 0; e < 4; ++e)
                mma(acc[f][e], a0, a1, a2, a3, pair_up(word(rb[0], e / 2), word(rb[1], e / 2), e & 1),
                    pair_up(word(rb[2], e / 2), word(rb[3], e / 2), e & 1));
        }
    }
    // a lane ends up with columns [8t, 8t + 8) of its eight rows
    const int32_t n = n0 + 8 * t;
    if (!in_m || n >= N) return;
#pragma unroll
    for (int f = 0; f < 4; ++f)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            float v[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] = acc[f][e & 3][2 * h + (e >> 2)];
            put_grad(p, out, (m0 + 2 * f + h) * ld_out + n, v);
        }
}

// dx = du . W_up by the first CTAs; a tile of dW_up = du^T . x or dW_down = dy^T . act by each warp of the others.
template <int MT, bool SPLIT> __global__ void __launch_bounds__(32 * BACK_WARPS) k_back_grads(const __grid_constant__ Back p)
{
    __shared__ Red<MT> red;
    if ((int)blockIdx.x < p.dx_ctas) {
        const int32_t split = SPLIT ? 1 << p.split_log : 1, rank = (int)blockIdx.x & (split - 1);
        const int32_t at = SPLIT ? (int)blockIdx.x >> p.split_log : (int)blockIdx.x;
        const int32_t groups = (p.T + 16 * MT - 1) / (16 * MT), t0 = at % groups * 16 * MT, T = min(p.T - t0, 16 * MT);
        const int32_t n0 = at / groups * BACK_N, n = n0 + (threadIdx.x & 31);
        const int64_t ld_du = 2 * (int64_t)p.inner;
        rows_by_weights<MT, SPLIT>(red, p.w_up, p.ld_wu, p.d, n0, p.du + t0 * ld_du, ld_du, T, 2 * p.inner, rank, split, true);
        for (int row = threadIdx.x >> 5; row < T; row += BACK_WARPS) {
            if ((row & (split - 1)) != rank) continue;
            const float v = summed<MT, SPLIT>(red, row, threadIdx.x & 31, split);
            if (n < p.d) p.dx[(t0 + row) * p.ld_dx + n] = __float2bfloat16_rn(v);
        }
        if (SPLIT) tc::cluster_sync();
        return;
    }
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int32_t tile = ((int)blockIdx.x - p.dx_ctas) * BACK_WARPS + (threadIdx.x >> 5);
    if (tile < p.up_tiles)
        grad_tile(p, tile, p.du, 2 * (int64_t)p.inner, 2 * p.inner, p.x, p.ld_x, p.d, p.dw_up, p.ld_dwu);
    else if (tile < p.up_tiles + p.down_tiles)
        grad_tile(p, tile - p.up_tiles, p.dy, p.ld_dy, p.d, p.act, p.inner, p.inner, p.dw_down, p.ld_dwd);
}

template <int MT> cudaError_t launch_back(Back p, cudaStream_t s)
{
    const int32_t groups = (p.T + 16 * MT - 1) / (16 * MT);
    cudaLaunchAttribute la[2];
    la[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    la[0].val.programmaticStreamSerializationAllowed = 1;
    la[1].id = cudaLaunchAttributeClusterDimension;
    la[1].val.clusterDim.y = la[1].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.blockDim = dim3(32 * BACK_WARPS);
    cfg.stream = s;
    int32_t across = (p.inner + BACK_N - 1) / BACK_N;
    p.split_log = split_of((int64_t)across * groups, BACK_FEW, p.d, 16 * 4 * BACK_WARPS);
    la[1].val.clusterDim.x = 1u << p.split_log;
    cfg.gridDim = dim3((unsigned)across << p.split_log, (unsigned)groups);
    cfg.attrs = la + 1;
    cfg.numAttrs = p.split_log ? 1 : 0;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, p.split_log ? k_back_act<MT, true> : k_back_act<MT, false>, p);
    if (e != cudaSuccess) return e;
    across = p.dx ? (p.d + BACK_N - 1) / BACK_N : 0;
    p.split_log = across ? split_of((int64_t)across * groups, BACK_FEW, 2 * (int64_t)p.inner, 16 * 4 * BACK_WARPS) : 0;
    p.dx_ctas = across * groups << p.split_log;
    const int32_t grads = (p.up_tiles + p.down_tiles + BACK_WARPS - 1) / BACK_WARPS;
    la[1].val.clusterDim.x = 1u << p.split_log;
    cfg.gridDim = dim3((unsigned)(p.dx_ctas + (grads + (1 << p.split_log) - 1 >> p.split_log << p.split_log)));
    cfg.attrs = la;
    cfg.numAttrs = p.split_log ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, p.split_log ? k_back_grads<MT, true> : k_back_grads<MT, false>, p);
}

}  // namespace ffn_small

cudaError_t launch_ffn_small_backward(const FfnSmallBackward& f, cudaStream_t s)
{
    using namespace ffn_small;
    const auto tiles = [](int32_t m, int32_t n) { return (m + GRAD_M - 1) / GRAD_M * ((n + GRAD_N - 1) / GRAD_N); };
    Back p{};
    p.dy = static_cast<const bf16*>(f.dy);
    p.x = static_cast<const bf16*>(f.x);
    p.u = static_cast<const bf16*>(f.u);
    p.w_up = static_cast<const bf16*>(f.w_up);
    p.w_down = static_cast<const bf16*>(f.w_down);
    p.ld_dy = f.ld_dy;
    p.ld_x = f.ld_x;
    p.ld_u = f.ld_u;
    p.ld_wu = f.ld_wu;
    p.ld_wd = f.ld_wd;
    p.act = static_cast<bf16*>(f.act);
    p.du = static_cast<bf16*>(f.du);
    p.dx = static_cast<bf16*>(f.dx);
    p.dw_up = f.dw_up;
    p.dw_down = f.dw_down;
    p.ld_dx = f.ld_dx;
    p.ld_dwu = f.ld_dwu;
    p.ld_dwd = f.ld_dwd;
    p.T = f.T;
    p.d = f.d;
    p.inner = f.inner;
    p.out_f32 = f.out_f32;
    p.accumulate = f.accumulate;
    p.up_tiles = f.dw_up ? tiles(2 * f.inner, f.d) : 0;
    p.down_tiles = f.dw_down ? tiles(f.d, f.inner) : 0;
    return f.T <= 16 ? launch_back<1>(p, s) : launch_back<2>(p, s);
}

cudaError_t launch_ffn_small(const FfnSmall& f, cudaStream_t s)
{
    ffn_small::Params p{};
    p.x = static_cast<const bf16*>(f.x);
    p.ld_x = f.ld_x;
    p.w = static_cast<const bf16*>(f.w_up);
    p.ld_w = f.ld_wu;
    p.out = static_cast<bf16*>(f.act);
    p.ld_out = f.inner;
    p.u = static_cast<bf16*>(f.u);
    p.ld_u = f.ld_u;
    p.T = f.T;
    p.rows = f.inner;
    p.K = f.d;
    const cudaError_t e = ffn_small::launch<true>(p, false, s);
    if (e != cudaSuccess) return e;
    p.x = p.out;
    p.ld_x = f.inner;
    p.w = static_cast<const bf16*>(f.w_down);
    p.ld_w = f.ld_wd;
    p.out = static_cast<bf16*>(f.y);
    p.ld_out = f.ld_y;
    p.u = nullptr;
    p.rows = f.d;
    p.K = f.inner;
    return ffn_small::launch<false>(p, true, s);
}

}  // namespace sol
