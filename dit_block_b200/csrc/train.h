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

// The whole forward pass for a few tokens (k_ffn_small.cu).  Measured at d x inner, us, against
// k_ffn.cu:   1 token   5120 x 13824  69.8 : 83.5    1000 x 2504   6.0 : 19.0
//            16 tokens  5120 x 13824  93 : 82.5      3000 x 8000  47 : 37     1000 x 2504   8.5 : 20
//            32 tokens  5120 x 13824 142 : 85.6      1024 x 4096  15 : 20      256 x 512    5.7 : 9.2
// k_ffn.cu takes some 14 us beside the weights' bytes at 6.2 TB/s; this one 3 us, with 6 TB/s for
// up to 8 tokens, and about 3.3 and 2.2 TB/s for up to 16 and 32, where the tokens' values cost as
// many loads as the weights: the two meet at 78 and 38 MB of weights.
inline bool ffn_small_fits(int64_t T, int64_t d, int64_t inner)
{
    return T <= 8 || (T <= 16 && d * inner <= 13000000) || (T <= 32 && d * inner <= 6300000);
}
struct FfnSmall {
    int32_t T, d, inner;
    const void *x, *w_up, *w_down;
    int64_t ld_x, ld_wu, ld_wd;
    void *y, *u, *act;  // u may be NULL; act [T, inner] is workspace
    int64_t ld_y, ld_u;
};
cudaError_t launch_ffn_small(const FfnSmall& f, cudaStream_t s);

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
