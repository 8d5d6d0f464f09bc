// k_ffn_small.cu -- the gated feed-forward block for a few tokens (a denoising server's
// smallest batches, single tokens): y = (silu(x Wg^T) * (x Wu^T)) Wd^T.
//
// Bound by the weights' bytes: 6 * d * inner of them against some tens of kilobytes of
// everything else.  The weights are streamed once, straight from HBM to registers in rows of
// consecutive 16-byte vectors (the tiles of k_ffn.cu would read each row 128 bytes at a time
// and multiply 128 rows of mostly nothing), and multiplied by m16n8k16 tensor instructions:
// 16 rows of weights by 8 tokens.  Which k of a 32-wide chunk a register stands for does not
// matter as long as both operands agree, so that a lane's 16-byte vector of a weight row and
// of a token's row are used as they come.
//
// A CTA takes 16 rows of weights (up projection: 8 of the gated half and the 8 of the other
// half that they meet, so that a thread ends up with a and b of the same value), its warps a
// share of K each; the shares are added through shared memory in the order of the warps.
// The second kernel is launched to overlap the first one's end (programmatic dependent
// launch) and starts by loading weights, which do not depend on it.
#include <cuda_bf16.h>

#include "common.cuh"
#include "launch.h"
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
};

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

template <bool UP, int NT, int WARPS>
__global__ void __launch_bounds__(32 * WARPS, (NT > 2 ? SM_WARPS / 2 : SM_WARPS) / WARPS) k_small(const __grid_constant__ Params p)
{
    constexpr int OUT = UP ? 8 : 16;  // outputs a token of this CTA
    __shared__ float red[WARPS][16][8 * NT + 1];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const int32_t j0 = blockIdx.x * OUT;
    // rows g and g + 8 of the tensor instruction
    const int32_t ra = j0 + g, rb = UP ? p.rows + j0 + g : j0 + 8 + g;
    const bool la = ra < p.rows, lb = UP ? la : rb < p.rows;
    const int32_t chunks = (p.K + CHUNK - 1) / CHUNK, share = (chunks + WARPS - 1) / WARPS;
    const int32_t c0 = min(warp * share, chunks), c1 = min(c0 + share, chunks);
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
                const uint4 x = c + i < c1 && k < p.K && 8 * n + g < p.T
                                    ? *reinterpret_cast<const uint4*>(p.x + (8 * n + g) * p.ld_x + k)
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
    for (int i = threadIdx.x; i < OUT * p.T; i += 32 * WARPS) {
        const int j = i % OUT, n = i / OUT;
        if (j0 + j >= p.rows) continue;
        float v = 0.f, v2 = 0.f;
#pragma unroll
        for (int s = 0; s < WARPS; ++s) {
            v += red[s][j][n];
            if (UP) v2 += red[s][j + 8][n];
        }
        if (UP) {
            if (p.u) {
                p.u[n * p.ld_u + j0 + j] = __float2bfloat16_rn(v);
                p.u[n * p.ld_u + p.rows + j0 + j] = __float2bfloat16_rn(v2);
            }
            v = v / (1.f + __expf(-v)) * v2;
        }
        p.out[n * p.ld_out + j0 + j] = __float2bfloat16_rn(v);
    }
}

template <bool UP, int WARPS> cudaError_t launch(const Params& p, bool after, cudaStream_t s)
{
    cudaLaunchAttribute la[1];
    la[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    la[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.blockDim = dim3(32 * WARPS);
    cfg.gridDim = dim3((unsigned)((p.rows + (UP ? 7 : 15)) / (UP ? 8 : 16)));
    cfg.stream = s;
    cfg.attrs = la;
    cfg.numAttrs = after ? 1 : 0;
    return p.T <= 8    ? cudaLaunchKernelEx(&cfg, k_small<UP, 1, WARPS>, p)
           : p.T <= 16 ? cudaLaunchKernelEx(&cfg, k_small<UP, 2, WARPS>, p)
                       : cudaLaunchKernelEx(&cfg, k_small<UP, 4, WARPS>, p);
}

// Sixteen warps a CTA where there is at most one CTA an SM, else eight.
template <bool UP> cudaError_t launch(const Params& p, bool after, cudaStream_t s)
{
    return (p.rows + (UP ? 7 : 15)) / (UP ? 8 : 16) <= 148 ? launch<UP, 16>(p, after, s) : launch<UP, 8>(p, after, s);
}

}  // namespace ffn_small

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
