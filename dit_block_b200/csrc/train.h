// train.h -- host-side launchers of the training kernels (internal to the library).
// Arguments reach these only after sol_train.cu validated them.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "sol_train.h"

namespace sol {

// ---- gated feed-forward block (k_ffn.cu)

// One matrix operand as it lies in memory: `rows` rows of `cols` bf16, row stride ld.
struct Mat {
    const void* p;
    int64_t rows, cols, ld;
};

// What a product's epilogue does with the accumulator.
enum FfnEpi {
    FFN_STORE = 0,  // out = acc (bf16 or f32; optionally added to what out holds)
    FFN_UP = 1,     // acc = [a | b]: act = silu(a) * b, u = [a | b] if kept
    FFN_DACT = 2,   // acc = d_act, with u = [a | b]: du, act
};

struct FfnProduct {
    FfnEpi epi;
    int64_t M, N, K;   // FFN_UP: N = inner (2 * inner rows of B)
    Mat a, b;
    bool a_mn, b_mn;   // operand stored with M (N) contiguous instead of K
    void* out;         // FFN_STORE: the product; FFN_UP, FFN_DACT: act (FFN_DACT: may be NULL)
    int64_t ld_out;
    bool out_f32, accumulate;
    void* u;           // FFN_UP: kept u or NULL; FFN_DACT: u (read)
    int64_t ld_u;
    void* du;          // FFN_DACT
    int64_t ld_du;
    float* slots;      // workspace of ffn_slot_bytes (of a launch's products one and the same)
};

// Bytes of f32 slots for the tiles that several workers share, for products of up to `rows` rows.
size_t ffn_slot_bytes(int64_t rows);
// One launch (and one to join what several workers share) of n products: one FFN_UP or FFN_DACT, or up to three
// FFN_STORE with B of one layout that do not depend on each other.  Reorders g.  after: the kernel
// before on the stream is one of the same call, which may still be ending.
cudaError_t launch_ffn_products(FfnProduct* g, int n, bool after, cudaStream_t s);

// The whole forward pass for a few tokens (k_ffn_small.cu).  Measured against k_ffn.cu, us, u kept:
//     tokens      1           16          32          64          96          128         160         192         300
//     64 x 64     3.2 : 8.2   3.8 : 8.3   4.7 : 8.4   4.8 : 8.6   5.0 : 8.8   4.9 : 9.1   5.0 : 8.7   5.0 : 8.7   5.0 : 8.7
//     256 x 512   3.4 : 10.4  4.6 : 10.5  5.7 : 10.5  6.1 : 10.7  7.8 : 11.0  8.1 : 11.3  9.9 : 11.5  10.4 : 11.5 15.5 : 11.7
//     568 x 936   3.9 : 14.0  5.4 : 14.1  7.0 : 14.1  9.6 : 15.0  11.7 : 16.3 14.1 : 17.8 17.4 : 18.1 19.9 : 18.1 29.7 : 18.2
//     1000 x 2504 6.4 : 18.0  9.4 : 18.2  12.9 : 18.3 16.6 : 20.0 24.7 : 21.8 28.9 : 23.2 36.8 : 22.6 42.0 : 22.6
//     3000 x 4000 18.1 : 28.7 26.3 : 29.0 31.8 : 29.6 57.5 : 31.1 -           94 : 38     117 : 41
//     5120 x 13824 70 : 87    101 : 87    141 : 88
// k_ffn.cu takes 8 to 14 us beside its k-blocks and the weights' bytes at 6.2 TB/s; this one 3 us, with 6 TB/s
// for up to 8 tokens, and less the more of them, whose values cost as many loads as the weights.  Long rows of
// W_down are few CTAs' work: 200 x 13000 takes 20.0 : 20.9 with 32 tokens, 33.5 : 23.6 with 64.  The rule has no
// budget between the one up to 128 tokens and the one of the smallest blocks, which leaves 256 x 512 from 129 to some 200
// tokens, and 568 x 936 to some 165, to k_ffn.cu: 1 to 3 us more than here.
inline bool ffn_small_fits(int64_t T, int64_t d, int64_t inner)
{
    if (T <= 8) return true;
    const int64_t most = (T <= 64 ? 200000000 : T <= 128 ? 128000000 : 6000000) / T;
    return T <= 512 && d * inner <= most && (T <= 32 || inner <= 8192);
}
struct FfnSmall {
    int32_t T, d, inner;
    const void *x, *w_up, *w_down;
    int64_t ld_x, ld_wu, ld_wd;
    void *y, *u, *act;  // u may be NULL; act [T, inner] is workspace
    int64_t ld_y, ld_u;
};
cudaError_t launch_ffn_small(const FfnSmall& f, cudaStream_t s);

// The whole backward pass for a few tokens (k_ffn_small.cu), in two launches.  Measured as above, all gradients:
//     tokens      1           16          32          64          96          128         200         256         300
//     64 x 64     4.0 : 10.5  4.5 : 10.3  5.7 : 10.3  6.7 : 10.4  7.5 : 10.5  8.8 : 10.8  10.5 : 10.7 11.8 : 10.9 13.8 : 11.2
//     256 x 512   5.1 : 15.9  6.1 : 15.8  8.1 : 15.8  8.5 : 16.0  10.0 : 16.4 11.5 : 17.0 13.3 : 16.9 17.6 : 17.3 20.6 : 17.2
//     568 x 936   7.5 : 22.4  8.6 : 22.6  11.0 : 22.8 12.4 : 23.3 13.6 : 22.7 15.7 : 23.9 18.9 : 24.2 22.7 : 25.0 25.3 : 25.7
//     1000 x 2504 13.3 : 38.5 14.8 : 38.6 19.1 : 38.7 25.3 : 39.2 30.9 : 33.7 35.9 : 35.2 53.2 : 37.5
//     640 x 8800  20.8 : 56.8 25.0 : 57.0 33.3 : 57.2 50.9 : 57.9 91.5 : 46.8
//     3000 x 4000 44 : 94     48 : 93     59 : 94     84 : 96     123 : 74
//     5120 x 13824 181 : 288  214 : 290   293 : 291   464 : 292
// The rule's ends leave 568 x 936 past 224 tokens and 1000 x 2504 from 80 to some 125 to k_ffn.cu: up to 2 and 3 us more
// than here.
inline bool ffn_small_backward_fits(int64_t T, int64_t d, int64_t inner)
{
    if (T <= 16) return d * inner < (int64_t)1 << 40;  // tiles of the gradients below 2^31
    return T <= 224 && d * inner <= (T <= 64 ? 800000000 : 200000000) / T;
}
struct FfnSmallBackward {
    int32_t T, d, inner;
    const void *dy, *x, *u, *w_up, *w_down;
    int64_t ld_dy, ld_x, ld_u, ld_wu, ld_wd;
    void *act, *du;                // workspace [T, inner], [T, 2 * inner]
    void *dx, *dw_up, *dw_down;    // each may be NULL
    int64_t ld_dx, ld_dwu, ld_dwd;
    bool out_f32, accumulate;      // of dw_up and dw_down
};
cudaError_t launch_ffn_small_backward(const FfnSmallBackward& f, cudaStream_t s);

// Error flags raised by these kernels' bounded waits; optionally cleared.  Synchronous.
uint32_t ffn_device_error(bool clear);

// ---- AdamW (k_adamw.cu)

constexpr int kAdamwChunk = 4096;  // values of one CTA, a multiple of SOL_ADAMW_BLOCK

struct AdamwTensor {
    float* p;
    void* copy;
    const void* g;
    void *m, *v;
    float *ms, *vs;
    int64_t n;
    float wd;
    uint32_t ordinal;  // place in the plan, for the rounding hash
};
struct AdamwChunk {
    int32_t tensor;
    int32_t index;     // chunk inside the tensor
};
struct AdamwCount {  // of a step counted on the device
    float inv_bc1, inv_bc2;
    uint32_t step;
};
struct AdamwTable {
    const AdamwTensor* tensors;
    const AdamwChunk* chunks;
    int64_t n_chunks;
    AdamwCount* count;  // the steps of a plan run one after another
};

cudaError_t launch_adamw_step(const AdamwTable& t, sol_dtype grad_dt, int state_bits, const sol_adamw_scalars& h,
                              cudaStream_t s);
cudaError_t launch_adamw_grad_norm(float* out, const AdamwTable& t, sol_dtype grad_dt, float max_norm, void* workspace,
                                   cudaStream_t s);
cudaError_t launch_adamw_decode(void* m_out, void* v_out, sol_dtype out_dt, const void* m, const void* v,
                                const float* ms, const float* vs, int64_t n, cudaStream_t s);

}  // namespace sol
