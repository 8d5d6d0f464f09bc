// k_adamw.cu -- the optimizer step over many tensors at once: AdamW with f32 or 8-bit
// moments, the global gradient norm with its clip factor, and reading 8-bit moments back.
//
// All are bound by HBM: per value 8 bytes of parameter, 2 or 4 of gradient, 16 of f32 (4 of
// 8-bit) moments and 2 of a bf16 copy against some 20 (60) instructions.  One CTA takes one
// chunk of 4096 values of one tensor, found through a table that the plan holds; every load
// of a thread is in flight before the first is used.
#include <algorithm>
#include <cmath>

#include <cuda_bf16.h>

#include "common.cuh"
#include "launch.h"
#include "train.h"

namespace sol {
namespace adamw {

constexpr int THREADS = 256;
constexpr int BLOCK = SOL_ADAMW_BLOCK;
constexpr int CHUNK = kAdamwChunk;
constexpr int NORM_CTAS = 148 * 8;  // partial sums of the gradient norm
static_assert((NORM_CTAS) * sizeof(double) <= SOL_ADAMW_NORM_WORKSPACE, "the norm's partial sums must fit its workspace");

// The step's scalars as the kernels use them.
struct Scalars {
    float lr, beta1, beta2, one_minus1, one_minus2, eps, inv_bc1, inv_bc2;
    double b1, b2;  // for steps counted on the device
    uint32_t seed_lo, seed_hi, step;
    const float* lr_device;
    const int64_t* step_device;
    const float* grad_factor;
};

struct Live {  // scalars of this launch, lr / step from the device where asked
    float lr, inv_bc1, inv_bc2, factor;
    uint32_t step;
};

// Called by every thread of the CTA.
__device__ __forceinline__ Live live_scalars(const Scalars& h)
{
    Live l{h.lr, h.inv_bc1, h.inv_bc2, 1.f, h.step};
    if (h.lr_device) l.lr = __ldg(h.lr_device);
    if (h.grad_factor) l.factor = __ldg(h.grad_factor);
    if (h.step_device) {
        __shared__ float bc[2];
        const int64_t step = max(*h.step_device, (int64_t)1);
        if (threadIdx.x == 0) {
            bc[0] = (float)(1.0 / (1.0 - pow(h.b1, (double)step)));
            bc[1] = (float)(1.0 / (1.0 - pow(h.b2, (double)step)));
        }
        __syncthreads();
        l.inv_bc1 = bc[0];
        l.inv_bc2 = bc[1];
        l.step = (uint32_t)step;
    }
    return l;
}

// One value: p, m, v in and out (fp32), g already widened.
__device__ __forceinline__ void update(float& p, float& m, float& v, float g, float wd, const Scalars& h, const Live& l)
{
    g *= l.factor;
    m = h.beta1 * m + h.one_minus1 * g;
    v = h.beta2 * v + h.one_minus2 * (g * g);
    p -= l.lr * (wd * p + (m * l.inv_bc1) / (sqrtf(v * l.inv_bc2) + h.eps));
}

__device__ __forceinline__ void load4(const float* p, float* f) { unpack<float>(ld_stream(p), f); }
__device__ __forceinline__ void load4(const bf16* p, float* f)
{
    const uint2 r = __ldcs(reinterpret_cast<const uint2*>(p));
    f[0] = __uint_as_float(r.x << 16);
    f[1] = __uint_as_float(r.x & 0xffff0000u);
    f[2] = __uint_as_float(r.y << 16);
    f[3] = __uint_as_float(r.y & 0xffff0000u);
}
__device__ __forceinline__ float widen(float x) { return x; }
__device__ __forceinline__ float widen(bf16 x) { return __bfloat162float(x); }

// f32 moments: a thread takes four vectors of four values, a CTA's threads side by side.
template <typename G>
__global__ void __launch_bounds__(THREADS) k_step32(const AdamwTable t, const __grid_constant__ Scalars h)
{
    const AdamwChunk c = t.chunks[blockIdx.x];
    const AdamwTensor x = t.tensors[c.tensor];
    const Live l = live_scalars(h);
    const int64_t base = (int64_t)c.index * CHUNK;
    const G* grad = static_cast<const G*>(x.g);
    float *pm = static_cast<float*>(x.m), *pv = static_cast<float*>(x.v);
    bf16* copy = static_cast<bf16*>(x.copy);
    constexpr int U = CHUNK / (4 * THREADS);
    float p[U][4], m[U][4], v[U][4], g[U][4];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int64_t i = base + 4 * (u * THREADS + threadIdx.x);
        if (i + 4 <= x.n) {
            load4(x.p + i, p[u]);
            load4(pm + i, m[u]);
            load4(pv + i, v[u]);
            load4(grad + i, g[u]);
        }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int64_t i = base + 4 * (u * THREADS + threadIdx.x);
        if (i + 4 <= x.n) {
#pragma unroll
            for (int e = 0; e < 4; ++e) update(p[u][e], m[u][e], v[u][e], g[u][e], x.wd, h, l);
            st_stream(x.p + i, pack<float>(p[u]));
            st_stream(pm + i, pack<float>(m[u]));
            st_stream(pv + i, pack<float>(v[u]));
            if (copy)
                *reinterpret_cast<uint2*>(copy + i) = make_uint2(pack2_bf16(p[u][0], p[u][1]), pack2_bf16(p[u][2], p[u][3]));
        } else {
            for (int64_t j = i; j < x.n; ++j) {  // the tensor's last one to three values
                float pp = x.p[j], mm = pm[j], vv = pv[j];
                update(pp, mm, vv, widen(grad[j]), x.wd, h, l);
                x.p[j] = pp;
                pm[j] = mm;
                pv[j] = vv;
                if (copy) copy[j] = __float2bfloat16_rn(pp);
            }
        }
    }
}

// ---------------------------------------------------------------------------------
// 8-bit moments.

// The finalizer of MurmurHash3 (Appleby 2011).
__device__ __forceinline__ uint32_t mixed(uint32_t h)
{
    h = (h ^ (h >> 16)) * 0x85EBCA6Bu;
    h = (h ^ (h >> 13)) * 0xC2B2AE35u;
    return h ^ (h >> 16);
}

__device__ __forceinline__ float decode_first(int q, float s)
{
    return (float)(q * abs(q)) * (1.f / 16129.f) * s;  // off by at most 3 * 2^-24
}
__device__ __forceinline__ float decode_second(uint32_t q, float s)
{
    const float k2 = (float)(q * q) * (1.f / 65025.f);
    return k2 * k2 * s;  // off by at most 6 * 2^-24
}

// Code of |x| (first) or x (second) in a block of scale s > 0, rounded up where the 16-bit
// fraction r is below the place between the two neighbours.
__device__ __forceinline__ int encode_first(float x, float s, float r)
{
    const float t = fabsf(x) / s * 16129.f;
    float k = floorf(sqrtf(t));
    if (r * fmaf(2.f, k, 1.f) < t - k * k) k += 1.f;
    const int q = (int)fminf(k, 127.f);
    return x < 0.f ? -q : q;
}
__device__ __forceinline__ uint32_t encode_second(float x, float s, float r)
{
    const float t = x / s * 4228250625.f;
    float k = floorf(sqrtf(sqrtf(t)));
    const float width = fmaf(fmaf(fmaf(4.f, k, 6.f), k, 4.f), k, 1.f), k2 = k * k;
    if (r * width < t - k2 * k2) k += 1.f;
    const uint32_t q = (uint32_t)fminf(k, 255.f);
    return x > 0.f ? max(q, 1u) : 0u;
}

// Largest magnitude over a warp by the bits of |x| (NaN above infinity above all numbers),
// as the block's scale: NaN where it is not finite.
__device__ __forceinline__ float block_scale(uint32_t bits)
{
    bits = __reduce_max_sync(0xffffffffu, bits);
    return __uint_as_float(bits >= 0x7f800000u ? 0x7fffffffu : bits);
}

// A warp takes one block of 256 values, eight a lane; a CTA its 16 blocks in two rounds.
template <typename G>
__global__ void __launch_bounds__(THREADS) k_step8(const AdamwTable t, const __grid_constant__ Scalars h)
{
    const AdamwChunk c = t.chunks[blockIdx.x];
    const AdamwTensor x = t.tensors[c.tensor];
    const Live l = live_scalars(h);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const G* grad = static_cast<const G*>(x.g);
    int8_t* pm = static_cast<int8_t*>(x.m);
    uint8_t* pv = static_cast<uint8_t*>(x.v);
    bf16* copy = static_cast<bf16*>(x.copy);
    const uint32_t key = mixed(mixed(mixed(x.ordinal * 0x9E3779B9u + l.step) ^ h.seed_hi) ^ h.seed_lo);
    for (int b = warp; b < CHUNK / BLOCK; b += THREADS / 32) {
        const int64_t start = (int64_t)c.index * CHUNK + b * BLOCK;
        if (start >= x.n) break;
        const int64_t i = start + 8 * lane, blk = start / BLOCK;
        const int live = (int)min((int64_t)8, max((int64_t)0, x.n - i));
        float p[8], g[8], m[8], v[8];
        const float s1 = x.ms[blk], s2 = x.vs[blk];
        if (live == 8) {
            load4(x.p + i, p);
            load4(x.p + i + 4, p + 4);
            load4(grad + i, g);
            load4(grad + i + 4, g + 4);
            const uint2 q1 = __ldcs(reinterpret_cast<const uint2*>(pm + i));
            const uint2 q2 = __ldcs(reinterpret_cast<const uint2*>(pv + i));
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                m[e] = decode_first((int)(int8_t)((e < 4 ? q1.x : q1.y) >> (8 * (e & 3))), s1);
                v[e] = decode_second(((e < 4 ? q2.x : q2.y) >> (8 * (e & 3))) & 255u, s2);
            }
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                p[e] = g[e] = m[e] = v[e] = 0.f;
                if (e < live) {
                    p[e] = x.p[i + e];
                    g[e] = widen(grad[i + e]);
                    m[e] = decode_first(pm[i + e], s1);
                    v[e] = decode_second(pv[i + e], s2);
                }
            }
        }
        uint32_t top1 = 0, top2 = 0;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            update(p[e], m[e], v[e], g[e], x.wd, h, l);
            if (e < live) {  // values past the tensor's end count for nothing
                top1 = max(top1, __float_as_uint(m[e]) & 0x7fffffffu);
                top2 = max(top2, __float_as_uint(v[e]) & 0x7fffffffu);
            }
        }
        const float n1 = block_scale(top1), n2 = block_scale(top2);
        uint2 q1 = make_uint2(0, 0), q2 = make_uint2(0, 0);
        const uint32_t at = mixed(key + (uint32_t)((uint64_t)start >> 32)) + (uint32_t)i;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const uint32_t r = mixed(at + e);
            const uint32_t a = n1 > 0.f ? (uint32_t)encode_first(m[e], n1, (float)(r >> 16) * (1.f / 65536.f)) & 255u : 0u;
            const uint32_t w = n2 > 0.f ? encode_second(v[e], n2, (float)(r & 0xffffu) * (1.f / 65536.f)) : 0u;
            (e < 4 ? q1.x : q1.y) |= a << (8 * (e & 3));
            (e < 4 ? q2.x : q2.y) |= w << (8 * (e & 3));
        }
        if (live == 8) {
            st_stream(x.p + i, pack<float>(p));
            st_stream(x.p + i + 4, pack<float>(p + 4));
            *reinterpret_cast<uint2*>(pm + i) = q1;
            *reinterpret_cast<uint2*>(pv + i) = q2;
            if (copy) st_stream(copy + i, pack<bf16>(p));
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e)
                if (e < live) {
                    x.p[i + e] = p[e];
                    pm[i + e] = (int8_t)((e < 4 ? q1.x : q1.y) >> (8 * (e & 3)));
                    pv[i + e] = (uint8_t)((e < 4 ? q2.x : q2.y) >> (8 * (e & 3)));
                    if (copy) copy[i + e] = __float2bfloat16_rn(p[e]);
                }
        }
        if (lane == 0) {
            x.ms[blk] = n1;
            x.vs[blk] = n2;
        }
    }
}

// ---------------------------------------------------------------------------------
// Global gradient norm.

// Sum of squares of 16 values: scaled by a power of two near their largest magnitude,
// squared and added in fp32, then brought back in fp64, so that neither 1e30 nor 1e-30 is
// lost.  A non-finite value makes the sum infinite or NaN.
__device__ __forceinline__ double squares16(const float* g)
{
    uint32_t top = 0;
#pragma unroll
    for (int e = 0; e < 16; ++e) top = max(top, __float_as_uint(g[e]) & 0x7fffffffu);
    if (top >= 0x7f800000u) return top == 0x7f800000u ? INFINITY : NAN;
    const uint32_t ex = min(max(top >> 23, 1u), 253u);  // biased exponent of the scale's inverse
    const float scale = __uint_as_float((254u - ex) << 23);
    float s = 0.f;
#pragma unroll
    for (int e = 0; e < 16; ++e) {
        const float y = g[e] * scale;
        s = fmaf(y, y, s);
    }
    return (double)s * __longlong_as_double((long long)(1023 + 2 * ((int)ex - 127)) << 52);
}

__device__ __forceinline__ double cta_sum(double v, double* buf)
{
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
    if ((threadIdx.x & 31) == 0) buf[threadIdx.x >> 5] = v;
    __syncthreads();
    double s = 0.0;
    for (int i = 0; i < (int)blockDim.x / 32; ++i) s += buf[i];
    return s;
}

// CTA b sums chunks b, b + gridDim.x, ...: the order depends on the plan alone.
template <typename G>
__global__ void __launch_bounds__(THREADS) k_norm_partial(const AdamwTable t, double* partial)
{
    __shared__ double buf[THREADS / 32];
    double sum = 0.0;
    for (int64_t b = blockIdx.x; b < t.n_chunks; b += gridDim.x) {
        const AdamwChunk c = t.chunks[b];
        const AdamwTensor* x = t.tensors + c.tensor;
        const G* grad = static_cast<const G*>(x->g);
        const int64_t n = x->n, base = (int64_t)c.index * CHUNK;
        float g[16];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const int64_t i = base + 4 * (u * THREADS + threadIdx.x);
            if (i + 4 <= n) {
                load4(grad + i, g + 4 * u);
            } else {
#pragma unroll
                for (int e = 0; e < 4; ++e) g[4 * u + e] = i + e < n ? widen(grad[i + e]) : 0.f;
            }
        }
        sum += squares16(g);
    }
    sum = cta_sum(sum, buf);
    if (threadIdx.x == 0) partial[blockIdx.x] = sum;
}

__global__ void __launch_bounds__(THREADS) k_norm_final(float* out, const double* partial, int n, float max_norm)
{
    __shared__ double buf[THREADS / 32];
    double sum = 0.0;
    for (int i = threadIdx.x; i < n; i += THREADS) sum += partial[i];
    sum = cta_sum(sum, buf);
    if (threadIdx.x == 0) {
        const double norm = sqrt(sum), f = (double)max_norm / (norm + 1e-6);
        out[0] = (float)norm;
        out[1] = f > 1.0 ? 1.f : (float)f;  // a NaN stays
    }
}

// Eight values a thread; the last thread's share may be smaller.
template <typename T>
__global__ void __launch_bounds__(THREADS)
    k_decode(T* m_out, T* v_out, const int8_t* m, const uint8_t* v, const float* ms, const float* vs, int64_t n)
{
    const int64_t i = 8 * ((int64_t)blockIdx.x * THREADS + threadIdx.x);
    if (i >= n) return;
    const bool whole = i + 8 <= n;
    float f[8];
    if (m_out) {
        const float s = ms[i / BLOCK];
        if (whole) {
            const uint2 q = __ldcs(reinterpret_cast<const uint2*>(m + i));
#pragma unroll
            for (int e = 0; e < 8; ++e) f[e] = decode_first((int)(int8_t)((e < 4 ? q.x : q.y) >> (8 * (e & 3))), s);
#pragma unroll
            for (int e = 0; e < 8; e += Vec<T>::N) st_stream(m_out + i + e, pack<T>(f + e));
        } else {
            for (int64_t j = i; j < n; ++j) m_out[j] = (T)decode_first(m[j], s);
        }
    }
    if (v_out) {
        const float s = vs[i / BLOCK];
        if (whole) {
            const uint2 q = __ldcs(reinterpret_cast<const uint2*>(v + i));
#pragma unroll
            for (int e = 0; e < 8; ++e) f[e] = decode_second(((e < 4 ? q.x : q.y) >> (8 * (e & 3))) & 255u, s);
#pragma unroll
            for (int e = 0; e < 8; e += Vec<T>::N) st_stream(v_out + i + e, pack<T>(f + e));
        } else {
            for (int64_t j = i; j < n; ++j) v_out[j] = (T)decode_second(v[j], s);
        }
    }
}

}  // namespace adamw

cudaError_t launch_adamw_step(const AdamwTable& t, sol_dtype grad_dt, int state_bits, const sol_adamw_scalars& a,
                              cudaStream_t s)
{
    if (t.n_chunks == 0) return cudaSuccess;
    adamw::Scalars h{};
    h.lr = (float)a.lr;
    h.beta1 = (float)a.beta1;
    h.beta2 = (float)a.beta2;
    h.one_minus1 = (float)(1.0 - a.beta1);
    h.one_minus2 = (float)(1.0 - a.beta2);
    h.eps = (float)a.eps;
    h.b1 = a.beta1;
    h.b2 = a.beta2;
    h.inv_bc1 = (float)(1.0 / (1.0 - std::pow(a.beta1, (double)a.step)));
    h.inv_bc2 = (float)(1.0 / (1.0 - std::pow(a.beta2, (double)a.step)));
    h.seed_lo = (uint32_t)a.seed;
    h.seed_hi = (uint32_t)(a.seed >> 32);
    h.step = (uint32_t)a.step;
    h.lr_device = a.lr_device;
    h.step_device = a.step_device;
    h.grad_factor = a.grad_factor;
    const unsigned grid = (unsigned)t.n_chunks;
    if (state_bits == 32) {
        if (grad_dt == SOL_DTYPE_BF16)
            adamw::k_step32<bf16><<<grid, adamw::THREADS, 0, s>>>(t, h);
        else
            adamw::k_step32<float><<<grid, adamw::THREADS, 0, s>>>(t, h);
    } else {
        if (grad_dt == SOL_DTYPE_BF16)
            adamw::k_step8<bf16><<<grid, adamw::THREADS, 0, s>>>(t, h);
        else
            adamw::k_step8<float><<<grid, adamw::THREADS, 0, s>>>(t, h);
    }
    return cudaGetLastError();
}

cudaError_t launch_adamw_grad_norm(float* out, const AdamwTable& t, sol_dtype grad_dt, float max_norm, void* workspace,
                                   cudaStream_t s)
{
    double* partial = static_cast<double*>(workspace);
    const int grid = (int)std::min<int64_t>(t.n_chunks, adamw::NORM_CTAS);
    if (grid > 0) {
        if (grad_dt == SOL_DTYPE_BF16)
            adamw::k_norm_partial<bf16><<<grid, adamw::THREADS, 0, s>>>(t, partial);
        else
            adamw::k_norm_partial<float><<<grid, adamw::THREADS, 0, s>>>(t, partial);
        const cudaError_t e = cudaGetLastError();
        if (e != cudaSuccess) return e;
    }
    adamw::k_norm_final<<<1, adamw::THREADS, 0, s>>>(out, partial, grid, max_norm);
    return cudaGetLastError();
}

cudaError_t launch_adamw_decode(void* m_out, void* v_out, sol_dtype out_dt, const void* m, const void* v,
                                const float* ms, const float* vs, int64_t n, cudaStream_t s)
{
    if (n == 0) return cudaSuccess;
    const unsigned grid = (unsigned)((n + 8 * adamw::THREADS - 1) / (8 * adamw::THREADS));
    if (out_dt == SOL_DTYPE_BF16)
        adamw::k_decode<bf16><<<grid, adamw::THREADS, 0, s>>>((bf16*)m_out, (bf16*)v_out, (const int8_t*)m,
                                                              (const uint8_t*)v, ms, vs, n);
    else
        adamw::k_decode<float><<<grid, adamw::THREADS, 0, s>>>((float*)m_out, (float*)v_out, (const int8_t*)m,
                                                               (const uint8_t*)v, ms, vs, n);
    return cudaGetLastError();
}

}  // namespace sol
