// k_adamw.cu -- the optimizer step over many tensors at once: AdamW with f32 or 8-bit
// moments, the global gradient norm with its clip factor, and reading 8-bit moments back.
//
// Per value 8 bytes of parameter, 2 or 4 of gradient, 16 of f32 (4 of 8-bit) moments and 2 of a
// bf16 copy.  One CTA takes one chunk of 4096 values of one tensor, found through a table that
// the plan holds.  212 M values, bf16 gradients and copies: with f32 moments 28 bytes a value in 914 us,
// 6.5 TB/s, the rate of a plain copy (with the norm, which reads the gradients once more: 30 bytes,
// 0.99 ms); with 8-bit moments 16.06 bytes in 558 us, 6.1 TB/s (with the norm 0.64 to 0.72 ms), as long as eight CTAs of
// four warps an SM hide the latencies of its 77 instructions a value (the codes, the roots, the random
// rounding): that is what keeps it 7% from a copy.
#include <algorithm>
#include <cmath>

#include <cuda_bf16.h>

#include "common.cuh"
#include "launch.h"
#include "train.h"

namespace sol {
namespace adamw {

constexpr int THREADS = 256;
constexpr int BLOCK = SOL_ADAMW_BLOCK, HALF = BLOCK / 2;
constexpr int CHUNK = kAdamwChunk;
constexpr int STEP8_THREADS = 128, STEP8_SPLIT = THREADS / STEP8_THREADS;
constexpr int STEP8_CTAS = 8;       // 64 registers (one spilled): 559 us, 590 with 7 CTAs of 72, 620 with 6 of 80
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
    const AdamwCount* count;  // of k_count, where the step is counted on the device
};

struct Live {  // scalars of this launch, lr / step from the device where asked
    float lr, inv_bc1, inv_bc2, factor;
    uint32_t step;
};

// What a step counted on the device needs of its number, by the first threads of two warps.
__device__ __forceinline__ void count_step(const Scalars& h, AdamwCount* out)
{
    const int64_t step = max(*h.step_device, (int64_t)1);
    if (threadIdx.x == 0) {
        out->inv_bc1 = (float)(1.0 / (1.0 - pow(h.b1, (double)step)));
        out->step = (uint32_t)step;
    }
    if (threadIdx.x == 32) out->inv_bc2 = (float)(1.0 / (1.0 - pow(h.b2, (double)step)));
}
__global__ void __launch_bounds__(64) k_count(const __grid_constant__ Scalars h, AdamwCount* out)
{
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    count_step(h, out);
}

// Called by every thread of the CTA.
__device__ __forceinline__ Live live_scalars(const Scalars& h)
{
    __shared__ AdamwCount here;
    Live l{h.lr, h.inv_bc1, h.inv_bc2, 1.f, h.step};
    if (h.lr_device) l.lr = __ldg(h.lr_device);
    if (h.grad_factor) l.factor = __ldg(h.grad_factor);
    if (h.count) {
        asm volatile("griddepcontrol.wait;" ::: "memory");
        l.inv_bc1 = __ldcg(&h.count->inv_bc1);
        l.inv_bc2 = __ldcg(&h.count->inv_bc2);
        l.step = __ldcg(&h.count->step);
    } else if (h.step_device) {
        count_step(h, &here);
        __syncthreads();
        l.inv_bc1 = here.inv_bc1;
        l.inv_bc2 = here.inv_bc2;
        l.step = here.step;
    }
    return l;
}

// sqrt with one MUFU operation, off by at most 2^-23 of itself; subnormal arguments count.
__device__ __forceinline__ float sqrt_fast(float x)
{
    float y;
    asm("sqrt.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// One value: p, m, v in and out (fp32), g already widened.  The quotient is off by some
// 2^-22 of the update, which is far below the rounding of p; its divisor stays below 2^65, as
// __fdividef wants it.
__device__ __forceinline__ void update(float& p, float& m, float& v, float g, float wd, const Scalars& h, const Live& l)
{
    g *= l.factor;
    m = h.beta1 * m + h.one_minus1 * g;
    v = h.beta2 * v + h.one_minus2 * (g * g);
    p -= l.lr * (wd * p + __fdividef(m * l.inv_bc1, sqrt_fast(v * l.inv_bc2) + h.eps));
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

// Small whole numbers to fp32 and back without conversion instructions (which run at an
// eighth of the rate of additions): 2^23 + q has q in its low mantissa bits.
// Byte e of w, as 2^23 + byte; halfword e of w, as 2^23 + halfword (one byte permutation each).
__device__ __forceinline__ float magic_byte(uint32_t w, int e)
{
    return __uint_as_float(__byte_perm(w, 0x4B000000u, 0x7540u + e));
}
__device__ __forceinline__ float magic_half(uint32_t w, int e)
{
    return __uint_as_float(__byte_perm(w, 0x4B000000u, e ? 0x7532u : 0x7510u));
}

__device__ __forceinline__ float2 both(float x) { return make_float2(x, x); }

// A block's scale s as the decoders use it: k^power * unit, or, where s is so small that
// unit would be subnormal, (k^power * step) * s.
__device__ __forceinline__ float2 decode_unit(float s, float step)
{
    return s < 1e-28f ? make_float2(step, s) : make_float2(step * s, 1.f);
}
// k * |k| and k^4 are formed with at most one rounding, the products add three more
__device__ __forceinline__ float2 decode_first2(float2 z, float u)  // z: 2^23 + (code ^ 0x80)
{
    const float2 k = __fadd2_rn(z, both(-(8388608.f + 128.f)));
    return __fmul2_rn(make_float2(k.x * fabsf(k.x), k.y * fabsf(k.y)), both(u));
}
__device__ __forceinline__ float2 decode_second2(float2 z, float u)  // z: 2^23 + code
{
    const float2 k = __fadd2_rn(z, both(-8388608.f)), k2 = __fmul2_rn(k, k);
    return __fmul2_rn(__fmul2_rn(k2, k2), both(u));
}
constexpr float STEP1 = 1.f / 16129.f, STEP2 = (float)(1.0 / 4228250625.0);  // 127^-2, 255^-4

__device__ __forceinline__ void scale8(float2* x, float f)
{
#pragma unroll
    for (int e = 0; e < 4; ++e) x[e] = __fmul2_rn(x[e], both(f));
}

// Eight codes (two words) of a block to values.
__device__ __forceinline__ void decode_first8(uint2 q, float s, float2* m)
{
    const float2 u = decode_unit(s, STEP1);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const uint32_t w = (e < 2 ? q.x : q.y) ^ 0x80808080u;
        m[e] = decode_first2(make_float2(magic_byte(w, 2 * (e & 1)), magic_byte(w, 2 * (e & 1) + 1)), u.x);
    }
    if (u.y != 1.f) scale8(m, u.y);
}
__device__ __forceinline__ void decode_second8(uint2 q, float s, float2* v)
{
    const float2 u = decode_unit(s, STEP2);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const uint32_t w = e < 2 ? q.x : q.y;
        v[e] = decode_second2(make_float2(magic_byte(w, 2 * (e & 1)), magic_byte(w, 2 * (e & 1) + 1)), u.x);
    }
    if (u.y != 1.f) scale8(v, u.y);
}

__device__ __forceinline__ float root_ftz(float x)
{
    float y;
    asm("sqrt.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float rcp_ftz(float x)
{
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// update() on two values: move = -lr / (1 - beta1^step), shrink = -lr * weight_decay.  ROOT_FTZ: the root of a subnormal v counts as zero.
template <bool ROOT_FTZ>
__device__ __forceinline__ void update2(float2& p, float2& m, float2& v, float2 g, float move, float shrink,
                                        const Scalars& h, const Live& l)
{
    g = __fmul2_rn(g, both(l.factor));
    m = __ffma2_rn(both(h.beta1), m, __fmul2_rn(both(h.one_minus1), g));
    v = __ffma2_rn(both(h.beta2), v, __fmul2_rn(both(h.one_minus2), __fmul2_rn(g, g)));
    const float2 x = __fmul2_rn(v, both(l.inv_bc2));
    const float2 d = __fadd2_rn(
        ROOT_FTZ ? make_float2(root_ftz(x.x), root_ftz(x.y)) : make_float2(sqrt_fast(x.x), sqrt_fast(x.y)), both(h.eps));
    const float2 up = __ffma2_rn(__fmul2_rn(m, both(move)), make_float2(rcp_ftz(d.x), rcp_ftz(d.y)), p);
    p = __ffma2_rn(both(shrink), p, up);
}

// Codes of two values.  t is a value in units of the table's first step.  Its root, made
// smaller by 2^-20 of itself, minus a half, rounded to a whole number, is k: the root's floor, or one
// less where the root is within 2^-20 above a whole number (so that the block's largest value
// has k one below the table's end).  The value is stored as k + 1 where the 16-bit fraction h / 65536
// is below (t - k^power) / ((k + 1)^power - k^power); at a k one too low that is always.
// z holds k in its low byte (1.5 * 2^23 + k); the sign of s says whether to take k + 1.
constexpr float MAGIC = 12582912.f, SHY = 1.f - 0x1p-20f;

__device__ __forceinline__ void encode_first2(float2 x, float inv, uint32_t r0, uint32_t r1, float2& z, float2& s)
{
    const float2 minus_t = make_float2(fabsf(x.x) * -inv, fabsf(x.y) * -inv);
    const float2 c = make_float2(root_ftz(-minus_t.x), root_ftz(-minus_t.y));
    z = __fadd2_rn(__ffma2_rn(c, both(SHY), both(-0.5f)), both(MAGIC));
    const float2 k = __fadd2_rn(z, both(-MAGIC));
    const float2 h = __fadd2_rn(make_float2(magic_half(r0, 1), magic_half(r1, 1)), both(-8388608.f));
    const float2 width = __ffma2_rn(both(2.f / 65536.f), k, both(1.f / 65536.f));
    s = __ffma2_rn(h, width, __ffma2_rn(k, k, minus_t));
}
__device__ __forceinline__ void encode_second2(float2 x, float inv, uint32_t r0, uint32_t r1, float2& z, float2& s)
{
    float2 t = __fmul2_rn(x, both(inv));
    t = make_float2(fmaxf(t.x, x.x > 0.f ? 1.f : 0.f), fmaxf(t.y, x.y > 0.f ? 1.f : 0.f));  // 1 at least
    const float2 c = make_float2(root_ftz(root_ftz(t.x)), root_ftz(root_ftz(t.y)));
    z = __fadd2_rn(__ffma2_rn(c, both(SHY), both(-0.5f)), both(MAGIC));
    const float2 k = __fadd2_rn(z, both(-MAGIC)), k2 = __fmul2_rn(k, k);
    const float2 h = __fadd2_rn(make_float2(magic_half(r0, 0), magic_half(r1, 0)), both(-8388608.f));
    float2 width = __ffma2_rn(both(4.f / 65536.f), k, both(6.f / 65536.f));
    width = __ffma2_rn(width, k, both(4.f / 65536.f));
    width = __ffma2_rn(width, k, both(1.f / 65536.f));
    s = __ffma2_rn(h, width, __ffma2_rn(k2, k2, make_float2(-t.x, -t.y)));
}

// The low bytes of four words; 0xff or 0 in each byte by the words' signs.
__device__ __forceinline__ uint32_t low_bytes(float2 a, float2 b)
{
    return __byte_perm(__byte_perm(__float_as_uint(a.x), __float_as_uint(a.y), 0x0040),
                       __byte_perm(__float_as_uint(b.x), __float_as_uint(b.y), 0x0040), 0x5410);
}
__device__ __forceinline__ uint32_t prmt_sign(uint32_t a, uint32_t b)  // bytes 0 and 1: the signs of a and b
{
    uint32_t r;
    asm("prmt.b32 %0, %1, %2, 0x00fb;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
__device__ __forceinline__ uint32_t sign_bytes(float2 a, float2 b)
{
    return __byte_perm(prmt_sign(__float_as_uint(a.x), __float_as_uint(a.y)),
                       prmt_sign(__float_as_uint(b.x), __float_as_uint(b.y)), 0x5410);
}
// k or k + 1 of four values, a byte each (no byte can overflow); then negated where x < 0.
__device__ __forceinline__ uint32_t four_codes(float2 z0, float2 z1, float2 s0, float2 s1)
{
    return low_bytes(z0, z1) + (sign_bytes(s0, s1) & 0x01010101u);
}
__device__ __forceinline__ uint32_t four_signed(uint32_t q, float2 x0, float2 x1)
{
    const uint32_t n = sign_bytes(x0, x1);
    return (((q ^ n) & 0x7f7f7f7fu) + (n & 0x01010101u)) ^ (n & 0x80808080u);
}

// Largest magnitude of three, NaN if one is NaN.
__device__ __forceinline__ float max_abs_nan(float a, float b, float c)
{
    float y;
    asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(y) : "f"(a), "f"(b), "f"(c));
    return y;
}

// A block's scale from its lanes' largest magnitudes: by their bits (NaN above infinity above all
// numbers), NaN where it is not finite.
__device__ __forceinline__ float block_scale(float top)
{
    const uint32_t bits = __reduce_max_sync(0xffffffffu, __float_as_uint(top) & 0x7fffffffu);
    return __uint_as_float(bits >= 0x7f800000u ? 0x7fffffffu : bits);
}

// How a block's values are brought to units of the table's first step (`most` of them make up the
// scale s): x * inv; for a small s, where most / s would overflow, x * 2^100 first.  What is inverted is s * down:
// the reciprocal of an s above 2^126 would be flushed.  A scale of zero or NaN gives zero codes.
struct Unit {
    float down, inv;
    __device__ __forceinline__ bool small() const { return down > 1.f; }
};
constexpr float SMALL = 0x1p100f, DOWN = 0x1p-24f;
__device__ __forceinline__ Unit unit_of(float s, float most)
{
    Unit u;
    u.down = s < 1e-28f ? SMALL * DOWN : DOWN;
    u.inv = s > 0.f ? (most * DOWN) * rcp_ftz(s * u.down) : 0.f;  // off by 2^-22: the margin of 2^-20 covers it
    return u;
}
// The codes of a lane's eight new moments (two runs of four, HALF apart; `at`: the hash's argument for the
// first) and the scales of their block.
__device__ __forceinline__ void encode8(float2* m, float2* v, uint32_t at, uint2& q1, uint2& q2, float& n1, float& n2)
{
    float top1 = 0.f, top2 = 0.f;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        top1 = max_abs_nan(top1, m[e].x, m[e].y);
        top2 = max_abs_nan(top2, v[e].x, v[e].y);
    }
    n1 = block_scale(top1);
    n2 = block_scale(top2);
    const Unit u1 = unit_of(n1, 16129.f), u2 = unit_of(n2, 4228250625.f);
    if (u1.small()) scale8(m, SMALL);
    if (u2.small()) scale8(v, SMALL);
#pragma unroll
    for (int w = 0; w < 2; ++w) {
        float2 z[4], up[4];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const uint32_t r0 = mixed(at + HALF * w + 2 * e), r1 = mixed(at + HALF * w + 2 * e + 1);
            encode_first2(m[2 * w + e], u1.inv, r0, r1, z[e], up[e]);
            encode_second2(v[2 * w + e], u2.inv, r0, r1, z[2 + e], up[2 + e]);
        }
        (w ? q1.y : q1.x) = four_signed(four_codes(z[0], z[1], up[0], up[1]), m[2 * w], m[2 * w + 1]);
        (w ? q2.y : q2.x) = four_codes(z[2], z[3], up[2], up[3]);
    }
}

// A block on its way through shared memory: the next one's loads are in flight while a block is
// worked on, without registers for them.  A lane takes values [4 * lane, + 4) of either half, so that
// every load and store of a warp is one run of bytes.
template <typename G> struct alignas(16) BlockIn {
    float p[BLOCK];
    G g[BLOCK];
    uint8_t mv[2][BLOCK];
};

__device__ __forceinline__ void copy16(void* dst, const void* src)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
}
__device__ __forceinline__ void load4s(const float* p, float2* f)
{
    unpack2<float>(*reinterpret_cast<const uint4*>(p), f);
}
__device__ __forceinline__ void load4s(const bf16* p, float2* f)
{
    const uint2 r = *reinterpret_cast<const uint2*>(p);
    f[0] = make_float2(__uint_as_float(r.x << 16), __uint_as_float(r.x & 0xffff0000u));
    f[1] = make_float2(__uint_as_float(r.y << 16), __uint_as_float(r.y & 0xffff0000u));
}

// A warp takes one block of 256 values at a time, eight a lane, two blocks in flight.  A CTA is small
// so that its warps need not wait for each other's end, and is done after two blocks a warp, so that reads and
// writes stay close together in memory.  212 M values, bf16 gradients and copies: 558 us = 6.1 TB/s (a lane on
// eight values in a row, CTAs of 256 threads: 718, of 128: 679; four blocks a warp instead of two: 984).
template <typename G, bool ROOT_FTZ>
__global__ void __launch_bounds__(STEP8_THREADS, STEP8_CTAS) k_step8(const AdamwTable t, const __grid_constant__ Scalars h)
{
    __shared__ BlockIn<G> in[2][STEP8_THREADS / 32];
    const AdamwChunk c = t.chunks[blockIdx.x / STEP8_SPLIT];
    const AdamwTensor x = t.tensors[c.tensor];
    const int warp = blockIdx.x % STEP8_SPLIT * (STEP8_THREADS / 32) + (threadIdx.x >> 5), lane = threadIdx.x & 31;
    const G* grad = static_cast<const G*>(x.g);
    uint8_t *pm = static_cast<uint8_t*>(x.m), *pv = static_cast<uint8_t*>(x.v);
    bf16* copy = static_cast<bf16*>(x.copy);
    const int64_t base = (int64_t)c.index * CHUNK, end = min(x.n, base + CHUNK);
    int64_t start = base + warp * BLOCK;
    constexpr int STRIDE = THREADS / 32 * BLOCK;

    auto fetch = [&](int64_t from, int stage) {  // whole blocks only
        if (from + BLOCK <= end) {
            BlockIn<G>& d = in[stage][threadIdx.x >> 5];
            constexpr int V = 16 / sizeof(G);
            copy16(d.p + 4 * lane, x.p + from + 4 * lane);
            copy16(d.p + HALF + 4 * lane, x.p + from + HALF + 4 * lane);
#pragma unroll
            for (int e = 0; e < BLOCK; e += 32 * V) copy16(d.g + e + V * lane, grad + from + e + V * lane);
            copy16(&d.mv[0][16 * lane], (lane < 16 ? pm : pv) + from + 16 * (lane & 15));
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    float s1 = 0.f, s2 = 0.f;
    if (start < end) {
        s1 = x.ms[start / BLOCK];
        s2 = x.vs[start / BLOCK];
    }
    fetch(start, 0);
    const Live l = live_scalars(h);
    const uint32_t key = mixed(mixed(mixed(x.ordinal * 0x9E3779B9u + l.step) ^ h.seed_hi) ^ h.seed_lo);
    const uint32_t from = mixed(key + (uint32_t)((uint64_t)c.index * CHUNK >> 32));  // a chunk's upper halves agree
    for (int stage = 0; start < end; start += STRIDE, stage ^= 1) {
        fetch(start + STRIDE, stage ^ 1);
        const int64_t blk = start / BLOCK, i = start + 4 * lane;
        float n1 = s1, n2 = s2;
        if (start + STRIDE < end) {
            s1 = x.ms[blk + THREADS / 32];
            s2 = x.vs[blk + THREADS / 32];
        }
        const uint32_t at = from + (uint32_t)i;
        float2 p[4], g[4], m[4], v[4];
        uint2 q1, q2;
        if (start + BLOCK <= end) {
            asm volatile("cp.async.wait_group 1;" ::: "memory");
            __syncwarp();
            const BlockIn<G>& d = in[stage][threadIdx.x >> 5];
            uint32_t w[2][2];
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                load4s(d.p + r * HALF + 4 * lane, p + 2 * r);
                load4s(d.g + r * HALF + 4 * lane, g + 2 * r);
#pragma unroll
                for (int k = 0; k < 2; ++k) w[k][r] = *reinterpret_cast<const uint32_t*>(&d.mv[k][r * HALF + 4 * lane]);
            }
            __syncwarp();  // read before the next block but one is copied here
            decode_first8(make_uint2(w[0][0], w[0][1]), n1, m);
            decode_second8(make_uint2(w[1][0], w[1][1]), n2, v);
#pragma unroll
            for (int e = 0; e < 4; ++e) update2<ROOT_FTZ>(p[e], m[e], v[e], g[e], -l.lr * l.inv_bc1, -l.lr * x.wd, h, l);
            // the parameters leave first: their registers are free for the codes
            st_stream(x.p + i, pack2<float>(p));
            st_stream(x.p + i + HALF, pack2<float>(p + 2));
            if (copy) {
                const uint4 r = pack2<bf16>(p);
                __stcs(reinterpret_cast<uint2*>(copy + i), make_uint2(r.x, r.y));
                __stcs(reinterpret_cast<uint2*>(copy + i + HALF), make_uint2(r.z, r.w));
            }
            encode8(m, v, at, q1, q2, n1, n2);
            *reinterpret_cast<uint32_t*>(pm + i) = q1.x;
            *reinterpret_cast<uint32_t*>(pm + i + HALF) = q1.y;
            *reinterpret_cast<uint32_t*>(pv + i) = q2.x;
            *reinterpret_cast<uint32_t*>(pv + i + HALF) = q2.y;
        } else {
            // the tensor's last block: value e of the lane is i + e, or i + HALF + e - 4 from e = 4 on
            const auto index = [&](int e) { return i + e + (e < 4 ? 0 : HALF - 4); };
            float fp[8] = {}, fg[8] = {};
            uint32_t w1[2] = {}, w2[2] = {};
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const int64_t j = index(e);
                if (j >= x.n) continue;
                fp[e] = x.p[j];
                fg[e] = widen(grad[j]);
                w1[e >> 2] |= (uint32_t)pm[j] << (8 * (e & 3));
                w2[e >> 2] |= (uint32_t)pv[j] << (8 * (e & 3));
            }
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                p[e] = make_float2(fp[2 * e], fp[2 * e + 1]);
                g[e] = make_float2(fg[2 * e], fg[2 * e + 1]);
            }
            decode_first8(make_uint2(w1[0], w1[1]), n1, m);
            decode_second8(make_uint2(w2[0], w2[1]), n2, v);
#pragma unroll
            for (int e = 0; e < 4; ++e) update2<ROOT_FTZ>(p[e], m[e], v[e], g[e], -l.lr * l.inv_bc1, -l.lr * x.wd, h, l);
#pragma unroll
            for (int e = 0; e < 8; ++e)  // values past the tensor's end count for nothing
                if (index(e) >= x.n) (e & 1 ? m[e / 2].y : m[e / 2].x) = (e & 1 ? v[e / 2].y : v[e / 2].x) = 0.f;
            encode8(m, v, at, q1, q2, n1, n2);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const int64_t j = index(e);
                if (j >= x.n) continue;
                const float pe = e & 1 ? p[e / 2].y : p[e / 2].x;
                x.p[j] = pe;
                pm[j] = (uint8_t)((e < 4 ? q1.x : q1.y) >> (8 * (e & 3)));
                pv[j] = (uint8_t)((e < 4 ? q2.x : q2.y) >> (8 * (e & 3)));
                if (copy) copy[j] = __float2bfloat16_rn(pe);
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

// Sum of squares of 16 values.  Where the plain fp32 sum is neither close to overflow nor so
// small that squares may have been lost (below 2^-126 each, nothing next to 2^-80), it is
// taken; else the values are scaled by a power of two near their largest magnitude and the
// sum is brought back in fp64, so that neither 1e30 nor 1e-30 is lost.  A non-finite value makes
// the sum infinite or NaN.
__device__ __forceinline__ double squares16(const float* g)
{
    float s = 0.f;
#pragma unroll
    for (int e = 0; e < 16; ++e) s = fmaf(g[e], g[e], s);
    if (s > 8.3e-25f && s < 1e38f) return (double)s;
    uint32_t top = 0;
#pragma unroll
    for (int e = 0; e < 16; ++e) top = max(top, __float_as_uint(g[e]) & 0x7fffffffu);
    if (top >= 0x7f800000u) return top == 0x7f800000u ? INFINITY : NAN;
    const uint32_t ex = min(max(top >> 23, 1u), 253u);  // biased exponent of the scale's inverse
    const float scale = __uint_as_float((254u - ex) << 23);
    s = 0.f;
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

// The 16 values of a thread in a chunk, by 16-byte vectors, as 16 fp32 registers; zeros behind
// the tensor's end.
template <typename G> __device__ __forceinline__ void load16(const G* grad, int64_t base, int64_t n, float* g)
{
    constexpr int V = Vec<G>::N;
#pragma unroll
    for (int u = 0; u < 16 / V; ++u) {
        const int64_t i = base + V * (u * THREADS + threadIdx.x);
        if (i + V <= n) {
            unpack<G>(ld_stream(grad + i), g + V * u);
        } else {
#pragma unroll
            for (int e = 0; e < V; ++e) g[V * u + e] = i + e < n ? widen(grad[i + e]) : 0.f;
        }
    }
}

// CTA b sums chunks b, b + gridDim.x, ...: the order depends on the plan alone.
template <typename G>
__global__ void __launch_bounds__(THREADS, 8) k_norm_partial(const AdamwTable t, double* partial)
{
    __shared__ double buf[THREADS / 32];
    double sum = 0.0;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    for (int64_t b = blockIdx.x; b < t.n_chunks; b += gridDim.x) {
        const AdamwChunk c = t.chunks[b];
        const AdamwTensor* x = t.tensors + c.tensor;
        float g[16];
        load16(static_cast<const G*>(x->g), (int64_t)c.index * CHUNK, x->n, g);
        sum += squares16(g);
    }
    sum = cta_sum(sum, buf);
    if (threadIdx.x == 0) partial[blockIdx.x] = sum;
}

__global__ void __launch_bounds__(THREADS) k_norm_final(float* out, const double* partial, int n, float max_norm)
{
    __shared__ double buf[THREADS / 32];
    double sum = 0.0;
    asm volatile("griddepcontrol.wait;" ::: "memory");  // set up while k_norm_partial ends
    for (int i = threadIdx.x; i < n; i += THREADS) sum += partial[i];
    sum = cta_sum(sum, buf);
    if (threadIdx.x == 0) {
        const double norm = sqrt(sum);
        // without a limit nothing is clipped, not by infinity / infinity either; a NaN stays
        const double f = isinf(max_norm) && isinf(norm) ? 1.0 : (double)max_norm / (norm + 1e-6);
        out[0] = (float)norm;
        out[1] = f > 1.0 ? 1.f : (float)f;
    }
}

// Eight values a thread; the last thread's share may be smaller.
template <typename T> __device__ __forceinline__ void put8(T* out, const float2* f, int live)
{
    if (live == 8) {
#pragma unroll
        for (int e = 0; e < 8; e += Vec<T>::N) st_stream(out + e, pack2<T>(f + e / 2));
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e)
            if (e < live) out[e] = (T)(e & 1 ? f[e / 2].y : f[e / 2].x);
    }
}
__device__ __forceinline__ uint2 codes8(const uint8_t* q, int live)
{
    if (live == 8) return __ldcs(reinterpret_cast<const uint2*>(q));
    uint32_t w[2] = {};
    for (int e = 0; e < live; ++e) w[e >> 2] |= (uint32_t)q[e] << (8 * (e & 3));
    return make_uint2(w[0], w[1]);
}
template <typename T>
__global__ void __launch_bounds__(THREADS)
    k_decode(T* m_out, T* v_out, const uint8_t* m, const uint8_t* v, const float* ms, const float* vs, int64_t n)
{
    const int64_t i = 8 * ((int64_t)blockIdx.x * THREADS + threadIdx.x);
    if (i >= n) return;
    const int live = (int)min((int64_t)8, n - i);
    uint2 q1, q2;
    float s1, s2;
    if (m_out) {
        q1 = codes8(m + i, live);
        s1 = __ldg(ms + i / BLOCK);
    }
    if (v_out) {
        q2 = codes8(v + i, live);
        s2 = __ldg(vs + i / BLOCK);
    }
    float2 f[4];
    if (m_out) {
        decode_first8(q1, s1, f);
        put8(m_out + i, f, live);
    }
    if (v_out) {
        decode_second8(q2, s2, f);
        put8(v_out + i, f, live);
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
    // The powers of a step counted on the device: in each CTA where all run at once, which costs 1 us and the
    // launch of k_count 5 (20,000 values, 8 bits: 7.9 against 13.2 us a call); else k_count, once for all (212 M
    // values: 573 to 597 against 626 us, 558 with the host's step).
    const bool counted = a.step_device && t.n_chunks > 148 * 3;
    if (counted) {
        h.count = t.count;
        adamw::k_count<<<1, 64, 0, s>>>(h, t.count);
        const cudaError_t e = cudaGetLastError();
        if (e != cudaSuccess) return e;
    }
    // the root of a subnormal v (below 1e-19) is nothing next to an eps of 1e-12 or more
    const bool bf = grad_dt == SOL_DTYPE_BF16, ftz = a.eps >= 1e-12;
    const auto kern = state_bits == 32 ? (bf ? adamw::k_step32<bf16> : adamw::k_step32<float>)
                      : bf             ? (ftz ? adamw::k_step8<bf16, true> : adamw::k_step8<bf16, false>)
                                       : (ftz ? adamw::k_step8<float, true> : adamw::k_step8<float, false>);
    cudaLaunchAttribute la[1];
    la[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    la[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    const int split = state_bits == 32 ? 1 : adamw::STEP8_SPLIT;
    cfg.gridDim = dim3((unsigned)(t.n_chunks * split));
    cfg.blockDim = dim3(adamw::THREADS / split);
    cfg.stream = s;
    cfg.attrs = la;
    cfg.numAttrs = counted ? 1 : 0;  // behind k_count alone
    return cudaLaunchKernelEx(&cfg, kern, t, h);
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
    cudaLaunchAttribute la[1];
    la[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    la[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(1);
    cfg.blockDim = dim3(adamw::THREADS);
    cfg.stream = s;
    cfg.attrs = la;
    cfg.numAttrs = grid > 0 ? 1 : 0;  // behind k_norm_partial alone
    return cudaLaunchKernelEx(&cfg, adamw::k_norm_final, out, (const double*)partial, grid, max_norm);
}

cudaError_t launch_adamw_decode(void* m_out, void* v_out, sol_dtype out_dt, const void* m, const void* v,
                                const float* ms, const float* vs, int64_t n, cudaStream_t s)
{
    if (n == 0) return cudaSuccess;
    const unsigned grid = (unsigned)((n + 8 * adamw::THREADS - 1) / (8 * adamw::THREADS));
    if (out_dt == SOL_DTYPE_BF16)
        adamw::k_decode<bf16><<<grid, adamw::THREADS, 0, s>>>((bf16*)m_out, (bf16*)v_out, (const uint8_t*)m,
                                                              (const uint8_t*)v, ms, vs, n);
    else
        adamw::k_decode<float><<<grid, adamw::THREADS, 0, s>>>((float*)m_out, (float*)v_out, (const uint8_t*)m,
                                                               (const uint8_t*)v, ms, vs, n);
    return cudaGetLastError();
}

}  // namespace sol
