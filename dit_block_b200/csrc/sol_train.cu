// sol_train.cu -- the C ABI of the training operators (declared in include/sol_train.h):
// argument validation, workspace layout, the AdamW plan, and the calls' launches.  Every
// check runs on the host before anything is launched.
#include <algorithm>
#include <cmath>
#include <cstdarg>
#include <cstdio>
#include <limits>
#include <new>
#include <utility>
#include <vector>

#include "common.cuh"
#include "launch.h"
#include "train.h"

struct sol_adamw_plan {
    void* dev;  // the tables below, one allocation
    int device;
    sol::AdamwTable table;
    sol_dtype grad_dt;
    int32_t state_bits;
};

namespace {

sol_status fail(sol_status st, const char* fmt, ...)
{
    char buf[384];
    va_list ap;
    va_start(ap, fmt);
    std::vsnprintf(buf, sizeof buf, fmt, ap);
    va_end(ap);
    sol::record_error(buf);
    return st;
}

sol_status cuda_status(cudaError_t e, const char* what)
{
    return e == cudaSuccess ? SOL_OK : fail(SOL_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e));
}

#define CHECK(cond, st, ...)                       \
    do {                                           \
        if (!(cond)) return fail(st, __VA_ARGS__); \
    } while (0)

#define TRY(expr)                      \
    do {                               \
        const sol_status st_ = (expr); \
        if (st_ != SOL_OK) return st_; \
    } while (0)

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }
size_t up256(size_t x) { return (x + 255) & ~(size_t)255; }

// A row-strided tensor as a span of bytes, for the overlap checks.
struct Span {
    const char* name;
    const void* p;
    int64_t rows, ld, width;
    size_t esz;
    const char* begin() const { return (const char*)p; }
    const char* end() const { return begin() + (size_t)((rows - 1) * ld + width) * esz; }
};

bool meet(const Span& a, const Span& b)
{
    if (!a.p || !b.p || a.rows <= 0 || b.rows <= 0) return false;
    return a.begin() < b.end() && b.begin() < a.end();
}

sol_status check_rows(const Span& t)
{
    CHECK(t.p, SOL_ERR_INVALID_ARGUMENT, "%s is NULL", t.name);
    CHECK(aligned(t.p, 16), SOL_ERR_MISALIGNED, "%s is not 16-byte aligned", t.name);
    CHECK(t.ld >= t.width, SOL_ERR_INVALID_ARGUMENT, "ld of %s (%lld) is below the row width %lld", t.name,
          (long long)t.ld, (long long)t.width);
    CHECK(t.ld % (int64_t)(16 / t.esz) == 0, SOL_ERR_MISALIGNED, "ld of %s (%lld) is not a multiple of %d elements (16 bytes)",
          t.name, (long long)t.ld, (int)(16 / t.esz));
    CHECK(t.ld < ((int64_t)1 << 38), SOL_ERR_UNSUPPORTED, "ld of %s (%lld) must be below 2^38", t.name, (long long)t.ld);
    return SOL_OK;
}

// Written tensors must not meet each other or anything read.
sol_status check_apart(const Span* written, int n_written, const Span* read, int n_read)
{
    for (int i = 0; i < n_written; ++i) {
        for (int j = i + 1; j < n_written; ++j)
            CHECK(!meet(written[i], written[j]), SOL_ERR_INVALID_ARGUMENT, "%s overlaps %s", written[i].name,
                  written[j].name);
        for (int j = 0; j < n_read; ++j)
            CHECK(!meet(written[i], read[j]), SOL_ERR_INVALID_ARGUMENT, "%s overlaps %s", written[i].name,
                  read[j].name);
    }
    return SOL_OK;
}

bool ffn_sizes_ok(int64_t n_tokens, int64_t d, int64_t inner)
{
    const int64_t most = (int64_t)1 << 28;
    return n_tokens >= 0 && n_tokens < ((int64_t)1 << 30) && d >= 8 && d < most && d % 8 == 0 && inner >= 8 &&
           inner < most && inner % 8 == 0;
}

sol_status check_ffn_sizes(int64_t n_tokens, int64_t d, int64_t inner, sol_dtype dt)
{
    CHECK(dt == SOL_DTYPE_BF16, SOL_ERR_UNSUPPORTED, "the feed-forward calls take bf16 only");
    CHECK(n_tokens >= 0, SOL_ERR_INVALID_ARGUMENT, "n_tokens (%lld) is negative", (long long)n_tokens);
    CHECK(n_tokens < ((int64_t)1 << 30), SOL_ERR_UNSUPPORTED, "n_tokens (%lld) must be below 2^30", (long long)n_tokens);
    CHECK(d >= 8 && inner >= 8, SOL_ERR_INVALID_ARGUMENT, "d (%lld) and inner (%lld) must be at least 8", (long long)d,
          (long long)inner);
    CHECK(ffn_sizes_ok(n_tokens, d, inner), SOL_ERR_UNSUPPORTED,
          "d (%lld) and inner (%lld) must be multiples of 8 below 2^28", (long long)d, (long long)inner);
    return SOL_OK;
}

// Workspace: act [T, inner], du [T, 2 * inner] (bf16), then the f32 slots of one launch (the
// launches run one after another).
struct FfnWorkspace {
    size_t act, du, slots, total;
};

FfnWorkspace ffn_layout(int64_t T, int64_t d, int64_t inner)
{
    FfnWorkspace w;
    w.act = 0;
    w.du = up256((size_t)T * (size_t)inner * 2);
    w.slots = up256(w.du + (size_t)T * (size_t)inner * 4);
    const size_t most = T > 0 ? sol::ffn_slot_bytes(std::max({T, d, 2 * inner})) : 0;
    w.total = up256(w.slots + most);
    return w;
}

sol_status check_workspace(const void* p, size_t bytes, const FfnWorkspace& lay)
{
    CHECK(p, SOL_ERR_INVALID_ARGUMENT, "workspace is NULL");
    CHECK(aligned(p, 256), SOL_ERR_MISALIGNED, "workspace is not 256-byte aligned");
    CHECK(bytes >= lay.total, SOL_ERR_INVALID_ARGUMENT, "workspace of %zu bytes is below the %zu needed", bytes, lay.total);
    return SOL_OK;
}

sol::FfnProduct product(sol::FfnEpi epi, int64_t M, int64_t N, int64_t K, sol::Mat a, bool a_mn, sol::Mat b, bool b_mn,
                        void* out, int64_t ld_out, void* ws, const FfnWorkspace& lay)
{
    sol::FfnProduct g{};
    g.epi = epi;
    g.M = M;
    g.N = N;
    g.K = K;
    g.a = a;
    g.b = b;
    g.a_mn = a_mn;
    g.b_mn = b_mn;
    g.out = out;
    g.ld_out = ld_out;
    g.slots = reinterpret_cast<float*>((char*)ws + lay.slots);
    return g;
}

}  // namespace

extern "C" {

size_t sol_ffn_workspace_bytes(int64_t n_tokens, int64_t d, int64_t inner)
{
    if (!ffn_sizes_ok(n_tokens, d, inner)) return 0;
    return std::max<size_t>(ffn_layout(n_tokens, d, inner).total, 256);
}

sol_status sol_ffn(const sol_ffn_desc* desc, sol_stream_t stream)
{
    CHECK(desc, SOL_ERR_INVALID_ARGUMENT, "desc is NULL");
    const sol_ffn_desc& f = *desc;
    const int64_t T = f.n_tokens, d = f.d, inner = f.inner;
    TRY(check_ffn_sizes(T, d, inner, f.dt));
    const Span sw[2] = {{"w_up", f.w_up, 2 * inner, f.ld_wu, d, 2}, {"w_down", f.w_down, d, f.ld_wd, inner, 2}};
    TRY(check_rows(sw[0]));
    TRY(check_rows(sw[1]));
    if (T == 0) return SOL_OK;
    const FfnWorkspace lay = ffn_layout(T, d, inner);
    TRY(check_workspace(f.workspace, f.workspace_bytes, lay));
    const Span written[3] = {{"y", f.y, T, f.ld_y, d, 2}, {"u", f.u, T, f.ld_u, 2 * inner, 2},
                             {"workspace", f.workspace, 1, 0, (int64_t)lay.total, 1}};
    const Span read[3] = {sw[0], sw[1], {"x", f.x, T, f.ld_x, d, 2}};
    TRY(check_rows(written[0]));
    if (f.u) TRY(check_rows(written[1]));
    TRY(check_rows(read[2]));
    TRY(check_apart(written, 3, read, 3));
    const cudaStream_t s = (cudaStream_t)stream;
    void* act = (char*)f.workspace + lay.act;
    if (sol::ffn_small_fits(T, d, inner)) {
        const sol::FfnSmall small{(int32_t)T, (int32_t)d, (int32_t)inner, f.x, f.w_up, f.w_down, f.ld_x, f.ld_wu, f.ld_wd,
                                  f.y, f.u, act, f.ld_y, f.ld_u};
        return cuda_status(sol::launch_ffn_small(small, s), "sol_ffn launch");
    }
    sol::FfnProduct g = product(sol::FFN_UP, T, inner, d, {f.x, T, d, f.ld_x}, false, {f.w_up, 2 * inner, d, f.ld_wu}, false,
                                act, inner, f.workspace, lay);
    g.u = f.u;
    g.ld_u = f.ld_u;
    TRY(cuda_status(sol::launch_ffn_products(&g, 1, false, s), "sol_ffn up projection launch"));
    g = product(sol::FFN_STORE, T, d, inner, {act, T, inner, inner}, false, {f.w_down, d, inner, f.ld_wd}, false, f.y, f.ld_y,
                f.workspace, lay);
    return cuda_status(sol::launch_ffn_products(&g, 1, true, s), "sol_ffn down projection launch");
}

sol_status sol_ffn_backward(const sol_ffn_backward_desc* desc, sol_stream_t stream)
{
    CHECK(desc, SOL_ERR_INVALID_ARGUMENT, "desc is NULL");
    const sol_ffn_backward_desc& f = *desc;
    const int64_t T = f.n_tokens, d = f.d, inner = f.inner;
    TRY(check_ffn_sizes(T, d, inner, f.dt));
    CHECK(f.grad_dt == SOL_DTYPE_F32 || f.grad_dt == SOL_DTYPE_BF16, SOL_ERR_UNSUPPORTED,
          "grad_dt %d is not SOL_DTYPE_F32 or SOL_DTYPE_BF16", (int)f.grad_dt);
    const size_t ge = f.grad_dt == SOL_DTYPE_F32 ? 4 : 2;
    const cudaStream_t s = (cudaStream_t)stream;
    const FfnWorkspace lay = ffn_layout(T, d, inner);
    const Span written[4] = {{"dw_up", f.dw_up, 2 * inner, f.ld_dwu, d, ge}, {"dw_down", f.dw_down, d, f.ld_dwd, inner, ge},
                             {"dx", T ? f.dx : nullptr, T, f.ld_dx, d, 2},
                             {"workspace", T ? f.workspace : nullptr, 1, 0, (int64_t)lay.total, 1}};
    const Span read[5] = {{"dy", f.dy, T, f.ld_dy, d, 2}, {"u", f.u, T, f.ld_u, 2 * inner, 2}, {"x", f.x, T, f.ld_x, d, 2},
                          {"w_up", f.w_up, 2 * inner, f.ld_wu, d, 2}, {"w_down", f.w_down, d, f.ld_wd, inner, 2}};
    for (int i = 0; i < 3; ++i)
        if (written[i].p) TRY(check_rows(written[i]));
    TRY(check_rows(read[3]));
    TRY(check_rows(read[4]));
    if (T > 0) {
        for (int i = 0; i < 3; ++i) TRY(check_rows(read[i]));
        TRY(check_workspace(f.workspace, f.workspace_bytes, lay));
    }
    TRY(check_apart(written, 4, read, 5));
    if (T == 0) {
        // a sum over no tokens
        for (int i = 0; i < 2 && !f.accumulate; ++i)
            if (written[i].p)
                TRY(cuda_status(cudaMemset2DAsync(const_cast<void*>(written[i].p), (size_t)written[i].ld * ge, 0,
                                                  (size_t)written[i].width * ge, (size_t)written[i].rows, s),
                                "sol_ffn_backward"));
        return SOL_OK;
    }
    if (!f.dx && !f.dw_up && !f.dw_down) return SOL_OK;
    void* act = (char*)f.workspace + lay.act;
    void* du = (char*)f.workspace + lay.du;
    if (sol::ffn_small_backward_fits(T, d, inner)) {
        const sol::FfnSmallBackward small{(int32_t)T, (int32_t)d, (int32_t)inner, f.dy, f.x, f.u, f.w_up, f.w_down,
                                          f.ld_dy, f.ld_x, f.ld_u, f.ld_wu, f.ld_wd, act, du, f.dx, f.dw_up, f.dw_down,
                                          f.ld_dx, f.ld_dwu, f.ld_dwd, f.grad_dt == SOL_DTYPE_F32, f.accumulate != 0};
        return cuda_status(sol::launch_ffn_small_backward(small, s), "sol_ffn_backward launch");
    }
    // d_act, and in its epilogue du and act
    sol::FfnProduct g = product(sol::FFN_DACT, T, inner, d, {f.dy, T, d, f.ld_dy}, false, {f.w_down, d, inner, f.ld_wd}, true,
                                f.dw_down ? act : nullptr, inner, f.workspace, lay);
    g.u = const_cast<void*>(f.u);
    g.ld_u = f.ld_u;
    g.du = du;
    g.ld_du = 2 * inner;
    TRY(cuda_status(sol::launch_ffn_products(&g, 1, false, s), "sol_ffn_backward d_act launch"));
    sol::FfnProduct all[3];
    int n = 0;
    if (f.dx)
        all[n++] = product(sol::FFN_STORE, T, d, 2 * inner, {du, T, 2 * inner, 2 * inner}, false, {f.w_up, 2 * inner, d, f.ld_wu},
                           true, f.dx, f.ld_dx, f.workspace, lay);
    if (f.dw_up)
        all[n++] = product(sol::FFN_STORE, 2 * inner, d, T, {du, T, 2 * inner, 2 * inner}, true, {f.x, T, d, f.ld_x}, true,
                           f.dw_up, f.ld_dwu, f.workspace, lay);
    if (f.dw_down)
        all[n++] = product(sol::FFN_STORE, d, inner, T, {f.dy, T, d, f.ld_dy}, true, {act, T, inner, inner}, true, f.dw_down,
                           f.ld_dwd, f.workspace, lay);
    for (int i = f.dx ? 1 : 0; i < n; ++i) {
        all[i].out_f32 = f.grad_dt == SOL_DTYPE_F32;
        all[i].accumulate = f.accumulate != 0;
    }
    return cuda_status(sol::launch_ffn_products(all, n, true, s), "sol_ffn_backward gradients launch");
}

// ---------------------------------------------------------------------------------

sol_status sol_adamw_plan_create(sol_adamw_plan** plan, const sol_adamw_tensor* tensors, int32_t n_tensors,
                                 sol_dtype grad_dt, int32_t state_bits)
try {
    CHECK(plan, SOL_ERR_INVALID_ARGUMENT, "plan is NULL");
    *plan = nullptr;
    CHECK(n_tensors >= 0, SOL_ERR_INVALID_ARGUMENT, "n_tensors (%d) is negative", (int)n_tensors);
    CHECK(tensors || n_tensors == 0, SOL_ERR_INVALID_ARGUMENT, "tensors is NULL");
    CHECK(grad_dt == SOL_DTYPE_F32 || grad_dt == SOL_DTYPE_BF16, SOL_ERR_UNSUPPORTED,
          "grad_dt %d is not SOL_DTYPE_F32 or SOL_DTYPE_BF16", (int)grad_dt);
    CHECK(state_bits == 32 || state_bits == 8, SOL_ERR_UNSUPPORTED, "state_bits (%d) is not 32 or 8", (int)state_bits);
    struct Buffer {
        const char *begin, *end, *name;
        int32_t tensor;
        bool written;
    };
    std::vector<Buffer> bufs;
    std::vector<sol::AdamwTensor> rows;
    std::vector<sol::AdamwChunk> chunks;
    for (int32_t i = 0; i < n_tensors; ++i) {
        const sol_adamw_tensor& t = tensors[i];
        CHECK(t.n >= 0 && t.n < ((int64_t)1 << 40), SOL_ERR_INVALID_ARGUMENT, "tensor %d: n (%lld) must be in [0, 2^40)",
              (int)i, (long long)t.n);
        CHECK(std::isfinite(t.weight_decay) && t.weight_decay >= 0.f, SOL_ERR_INVALID_ARGUMENT,
              "tensor %d: weight_decay must be finite and >= 0", (int)i);
        if (t.n == 0) continue;
        const size_t n = (size_t)t.n, st = state_bits == 8 ? 1 : 4, blocks = (n + SOL_ADAMW_BLOCK - 1) / SOL_ADAMW_BLOCK;
        const struct {
            const char* name;
            const void* p;
            size_t bytes;
            bool needed, written;
        } f[7] = {{"param", t.param, n * 4, true, true},
                  {"copy", t.copy, n * 2, false, true},
                  {"grad", t.grad, n * (grad_dt == SOL_DTYPE_F32 ? 4 : 2), true, false},
                  {"m", t.m, n * st, true, true},
                  {"v", t.v, n * st, true, true},
                  {"m_scale", t.m_scale, blocks * 4, state_bits == 8, true},
                  {"v_scale", t.v_scale, blocks * 4, state_bits == 8, true}};
        for (const auto& b : f) {
            CHECK(b.p || !b.needed, SOL_ERR_INVALID_ARGUMENT, "tensor %d: %s is NULL", (int)i, b.name);
            if (!b.p) continue;
            // scales are read one by one; the others by 16-byte vectors
            const bool scale = b.p == t.m_scale || b.p == t.v_scale;
            CHECK(!scale || state_bits == 8, SOL_ERR_INVALID_ARGUMENT, "tensor %d: %s is given for 32-bit moments", (int)i,
                  b.name);
            CHECK(aligned(b.p, scale ? 4 : 16), SOL_ERR_MISALIGNED, "tensor %d: %s is not %d-byte aligned", (int)i, b.name,
                  scale ? 4 : 16);
            bufs.push_back({(const char*)b.p, (const char*)b.p + b.bytes, b.name, i, b.written});
        }
        const int64_t nc = (t.n + sol::kAdamwChunk - 1) / sol::kAdamwChunk;
        CHECK((int64_t)chunks.size() + nc < ((int64_t)1 << 31), SOL_ERR_UNSUPPORTED, "the plan has more than 2^43 values");
        for (int64_t c = 0; c < nc; ++c) chunks.push_back({(int32_t)rows.size(), (int32_t)c});
        rows.push_back({t.param, t.copy, t.grad, t.m, t.v, t.m_scale, t.v_scale, t.n, t.weight_decay, (uint32_t)i});
    }
    // buffers in order of address: one that begins before an earlier one ended meets it
    std::sort(bufs.begin(), bufs.end(), [](const Buffer& a, const Buffer& b) { return a.begin < b.begin; });
    const Buffer *far = nullptr, *far_written = nullptr;  // reaching furthest so far: of all, of the written
    for (const Buffer& b : bufs) {
        const Buffer* hit = b.written && far && b.begin < far->end ? far
                            : far_written && b.begin < far_written->end ? far_written : nullptr;
        CHECK(!hit, SOL_ERR_INVALID_ARGUMENT, "%s of tensor %d overlaps %s of tensor %d", b.name, (int)b.tensor, hit->name,
              (int)hit->tensor);
        if (!far || b.end > far->end) far = &b;
        if (b.written && (!far_written || b.end > far_written->end)) far_written = &b;
    }
    sol_adamw_plan* r = new sol_adamw_plan{};
    r->grad_dt = grad_dt;
    r->state_bits = state_bits;
    const size_t at = up256(rows.size() * sizeof(sol::AdamwTensor)), count = up256(at + chunks.size() * sizeof(sol::AdamwChunk)),
                 total = count + sizeof(sol::AdamwCount);
    cudaError_t e = cudaGetDevice(&r->device);
    if (e == cudaSuccess && !rows.empty()) {
        e = cudaMalloc(&r->dev, total);
        if (e == cudaSuccess)
            e = cudaMemcpy(r->dev, rows.data(), rows.size() * sizeof(sol::AdamwTensor), cudaMemcpyHostToDevice);
        if (e == cudaSuccess)
            e = cudaMemcpy((char*)r->dev + at, chunks.data(), chunks.size() * sizeof(sol::AdamwChunk),
                           cudaMemcpyHostToDevice);
        // a copy from pageable memory may still be on its way, and steps may run on any stream
        if (e == cudaSuccess) e = cudaStreamSynchronize(cudaStreamLegacy);
    }
    if (e != cudaSuccess) {
        if (r->dev) cudaFree(r->dev);
        delete r;
        return cuda_status(e, "sol_adamw_plan_create");
    }
    r->table = {static_cast<const sol::AdamwTensor*>(r->dev),
                reinterpret_cast<const sol::AdamwChunk*>((const char*)r->dev + at), (int64_t)chunks.size(),
                reinterpret_cast<sol::AdamwCount*>((char*)r->dev + count)};
    *plan = r;
    return SOL_OK;
} catch (const std::bad_alloc&) {
    return fail(SOL_ERR_INVALID_ARGUMENT, "out of host memory for the plan's tables");
}

sol_status sol_adamw_plan_destroy(sol_adamw_plan* plan)
{
    if (!plan) return SOL_OK;
    cudaError_t e = cudaSuccess;
    if (plan->dev) {
        // a plan may be let go of while some stream is captured, which has nothing to do with it: without this the
        // capture would be spoilt
        cudaStreamCaptureMode mode = cudaStreamCaptureModeRelaxed;
        e = cudaThreadExchangeStreamCaptureMode(&mode);
        if (e == cudaSuccess) {
            e = cudaFree(plan->dev);
            cudaThreadExchangeStreamCaptureMode(&mode);
        }
    }
    delete plan;
    return cuda_status(e, "sol_adamw_plan_destroy");
}

static sol_status check_plan(const sol_adamw_plan* plan)
{
    CHECK(plan, SOL_ERR_INVALID_ARGUMENT, "plan is NULL");
    int dev = 0;
    TRY(cuda_status(cudaGetDevice(&dev), "cudaGetDevice"));
    CHECK(dev == plan->device, SOL_ERR_INVALID_ARGUMENT, "the plan was made on device %d, the current device is %d",
          plan->device, dev);
    return SOL_OK;
}

sol_status sol_adamw_step(const sol_adamw_plan* plan, const sol_adamw_scalars* h, sol_stream_t stream)
{
    CHECK(h, SOL_ERR_INVALID_ARGUMENT, "scalars is NULL");
    CHECK(std::isfinite(h->lr) && std::isfinite(h->eps) && h->eps >= 0, SOL_ERR_INVALID_ARGUMENT,
          "lr must be finite, eps finite and >= 0");
    // a divisor below fp32's normal numbers is taken for zero, which makes 0 / (0 + eps) NaN
    CHECK(h->eps == 0 || h->eps >= std::numeric_limits<float>::min(), SOL_ERR_INVALID_ARGUMENT,
          "eps (%g) must be 0 or at least 2^-126", h->eps);
    CHECK(h->beta1 >= 0 && h->beta1 < 1 && h->beta2 >= 0 && h->beta2 < 1, SOL_ERR_INVALID_ARGUMENT,
          "beta1 and beta2 must be in [0, 1)");
    CHECK(h->step >= 1, SOL_ERR_INVALID_ARGUMENT, "step (%lld) must be at least 1", (long long)h->step);
    CHECK(aligned(h->lr_device, 4) && aligned(h->step_device, 8) && aligned(h->grad_factor, 4), SOL_ERR_MISALIGNED,
          "lr_device, step_device or grad_factor is not aligned to its type");
    TRY(check_plan(plan));
    return cuda_status(sol::launch_adamw_step(plan->table, plan->grad_dt, plan->state_bits, *h, (cudaStream_t)stream),
                       "sol_adamw_step launch");
}

sol_status sol_adamw_grad_norm(float* out, const sol_adamw_plan* plan, float max_norm, void* workspace,
                               size_t workspace_bytes, sol_stream_t stream)
{
    CHECK(out, SOL_ERR_INVALID_ARGUMENT, "out is NULL");
    CHECK(aligned(out, 8), SOL_ERR_MISALIGNED, "out is not 8-byte aligned");
    CHECK(max_norm > 0.f, SOL_ERR_INVALID_ARGUMENT, "max_norm must be above 0");
    CHECK(workspace, SOL_ERR_INVALID_ARGUMENT, "workspace is NULL");
    CHECK(aligned(workspace, 16), SOL_ERR_MISALIGNED, "workspace is not 16-byte aligned");
    CHECK(workspace_bytes >= SOL_ADAMW_NORM_WORKSPACE, SOL_ERR_INVALID_ARGUMENT,
          "workspace of %zu bytes is below the %d needed", workspace_bytes, SOL_ADAMW_NORM_WORKSPACE);
    CHECK(!meet({"out", out, 1, 0, 2, 4}, {"workspace", workspace, 1, 0, SOL_ADAMW_NORM_WORKSPACE, 1}),
          SOL_ERR_INVALID_ARGUMENT, "out overlaps workspace");
    TRY(check_plan(plan));
    return cuda_status(
        sol::launch_adamw_grad_norm(out, plan->table, plan->grad_dt, max_norm, workspace, (cudaStream_t)stream),
        "sol_adamw_grad_norm launch");
}

sol_status sol_adamw_state_decode(void* m_out, void* v_out, sol_dtype out_dt, const void* m, const void* v,
                                  const float* m_scale, const float* v_scale, int64_t n, sol_stream_t stream)
{
    CHECK(out_dt == SOL_DTYPE_F32 || out_dt == SOL_DTYPE_BF16, SOL_ERR_UNSUPPORTED,
          "out_dt %d is not SOL_DTYPE_F32 or SOL_DTYPE_BF16", (int)out_dt);
    CHECK(n >= 0 && n < ((int64_t)1 << 40), SOL_ERR_INVALID_ARGUMENT, "n (%lld) must be in [0, 2^40)", (long long)n);
    if (n == 0 || (!m_out && !v_out)) return SOL_OK;
    const int64_t es = out_dt == SOL_DTYPE_F32 ? 4 : 2, blocks = (n + SOL_ADAMW_BLOCK - 1) / SOL_ADAMW_BLOCK;
    const Span written[2] = {{"m_out", m_out, 1, 0, n, (size_t)es}, {"v_out", v_out, 1, 0, n, (size_t)es}};
    const Span read[4] = {{"m", m_out ? m : nullptr, 1, 0, n, 1}, {"m_scale", m_out ? m_scale : nullptr, 1, 0, blocks, 4},
                          {"v", v_out ? v : nullptr, 1, 0, n, 1}, {"v_scale", v_out ? v_scale : nullptr, 1, 0, blocks, 4}};
    for (int i = 0; i < 2; ++i) {
        if (!written[i].p) continue;
        CHECK(read[2 * i].p && read[2 * i + 1].p, SOL_ERR_INVALID_ARGUMENT, "%s or %s is NULL", i ? "v" : "m",
              i ? "v_scale" : "m_scale");
        CHECK(aligned(written[i].p, 16) && aligned(read[2 * i].p, 16) && aligned(read[2 * i + 1].p, 4), SOL_ERR_MISALIGNED,
              "%s or its codes are not 16-byte aligned", written[i].name);
    }
    TRY(check_apart(written, 2, read, 4));
    return cuda_status(sol::launch_adamw_decode(m_out, v_out, out_dt, m, v, m_scale, v_scale, n, (cudaStream_t)stream),
                       "sol_adamw_state_decode launch");
}

}  // extern "C"
