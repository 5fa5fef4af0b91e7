// C-ABI layer of the layer steps around the token mixers: the gated linear
// recurrence, the RMS norm and the matrix product.  Argument validation and dispatch; contracts
// in include/cpdr.h.
#include <cuda_runtime.h>

#include <cstdint>
#include <initializer_list>
#include <string>

#include "cpdr_internal.hpp"

namespace {

using cpdr::check_device_ptr;
using cpdr::check_launch_ctx;
using cpdr::check_launched;
using cpdr::fail_with;

#define CPDR_TRY(x)                   \
    do {                              \
        cpdr_status _s = (x);         \
        if (_s != CPDR_OK) return _s; \
    } while (0)

// One tensor argument: its bytes in memory.
struct Span {
    const void *p;
    size_t bytes;
    const char *name;
};

bool overlap(const Span &a, const Span &b) {
    if (!a.p || !b.p || a.bytes == 0 || b.bytes == 0) return false;
    const char *x = (const char *)a.p, *y = (const char *)b.p;
    return x < y + b.bytes && y < x + a.bytes;
}

// Refuses outputs that overlap an input or one another.  An output may be
// the whole of one of the tensors of `same` (the in-place forms).
cpdr_status check_outputs(const char *what, std::initializer_list<Span> outs, std::initializer_list<Span> ins,
                          std::initializer_list<std::pair<const void *, const void *>> same = {}) {
    auto allowed = [&](const Span &a, const Span &b) {
        if (a.p != b.p || a.bytes != b.bytes) return false;
        for (const auto &s : same)
            if (s.first == a.p && s.second == b.p) return true;
        return false;
    };
    for (const Span *o = outs.begin(); o != outs.end(); o++) {
        for (const Span &i : ins)
            if (overlap(*o, i) && !allowed(*o, i))
                return fail_with(CPDR_ERR_INVALID, std::string(what) + ": " + o->name + " overlaps " + i.name);
        for (const Span *q = outs.begin(); q != o; q++)
            if (overlap(*o, *q))
                return fail_with(CPDR_ERR_INVALID, std::string(what) + ": " + o->name + " overlaps " + q->name);
    }
    return CPDR_OK;
}

size_t elem_bytes(const cpdr_ctx *c) { return c->plan.in_dtype == CPDR_DTYPE_F32 ? 4 : 2; }

cpdr_status check_channels(const char *what, int32_t channels) {
    if (channels < 1 || channels % 8 != 0)
        return fail_with(CPDR_ERR_INVALID, std::string(what) + ": channels must be a positive multiple of 8");
    if (channels > (1 << 24)) return fail_with(CPDR_ERR_UNSUPPORTED, std::string(what) + ": channels are at most 2^24");
    return CPDR_OK;
}

cpdr_status check_norm(const char *what, int64_t rows, int32_t width, float eps) {
    if (rows < 0 || rows > INT32_MAX) return fail_with(CPDR_ERR_INVALID, std::string(what) + ": rows must be 0 .. 2^31 - 1");
    if (width < 1 || width % 8 != 0)
        return fail_with(CPDR_ERR_INVALID, std::string(what) + ": width must be a positive multiple of 8");
    if (width > cpdr::kMaxNormWidth)
        return fail_with(CPDR_ERR_UNSUPPORTED, std::string(what) + ": width is at most 16384");
    if (!(eps >= 0.f) || eps > 1.f) return fail_with(CPDR_ERR_INVALID, std::string(what) + ": eps must be in [0, 1]");
    return CPDR_OK;
}

size_t round256(size_t x) { return (x + 255) & ~size_t(255); }

cpdr_status check_linear(const char *what, const cpdr_ctx *c, int64_t rows, int32_t K, int32_t N, int32_t act, bool e4m3) {
    if (c->plan.in_dtype != CPDR_DTYPE_BF16)
        return fail_with(CPDR_ERR_UNSUPPORTED, std::string(what) + ": only bf16 contexts (the products run on the tensor cores)");
    if (rows < 0 || rows > (int64_t)INT32_MAX - 512)
        return fail_with(CPDR_ERR_INVALID, std::string(what) + ": rows must be 0 .. 2^31 - 513");
    const int mult = e4m3 ? 16 : 8;
    if (K < 1 || K % mult != 0)
        return fail_with(CPDR_ERR_INVALID, std::string(what) + ": K must be a positive multiple of " + std::to_string(mult));
    if (N < 1 || N % 8 != 0) return fail_with(CPDR_ERR_INVALID, std::string(what) + ": N must be a positive multiple of 8");
    if (K > (1 << 23) || N > (1 << 23)) return fail_with(CPDR_ERR_UNSUPPORTED, std::string(what) + ": K and N are at most 2^23");
    if (act < 0 || act > 2)
        return fail_with(CPDR_ERR_INVALID, std::string(what) + ": activation must be 0 (none), 1 (SiLU) or 2 (GELU)");
    return CPDR_OK;
}

// The backward's workspace: dz (with an activation), then the row blocks' column sums.
size_t linear_dz_bytes(int64_t rows, int32_t N, int32_t act) { return act ? round256((size_t)rows * (size_t)N * 2) : 0; }
size_t linear_workspace(const cpdr_ctx *c, int64_t rows, int32_t N, int32_t act) {
    return linear_dz_bytes(rows, N, act) + cpdr::linear_dz_parts(c, rows, N) * (size_t)N * sizeof(float);
}

size_t norm_workspace(const cpdr_ctx *c, int64_t rows, int width) {
    return (size_t)cpdr::rmsnorm_bwd_grid(c, rows, width) * (size_t)width * sizeof(float);
}

}  // namespace

extern "C" {

cpdr_status cpdr_glr_carry_bytes(const cpdr_ctx *c, int32_t channels, size_t *bytes) {
    if (!c || !bytes) return fail_with(CPDR_ERR_INVALID, "null argument");
    CPDR_TRY(check_channels("cpdr_glr_carry_bytes", channels));
    *bytes = (size_t)c->plan.glr_groups * (size_t)channels * sizeof(float);
    return CPDR_OK;
}

cpdr_status cpdr_plan_glr(const cpdr_ctx *c, int32_t channels, int32_t backward, int32_t out[3]) {
    if (!c || !out) return fail_with(CPDR_ERR_INVALID, "null argument");
    if (c->has_device) CPDR_TRY(check_launch_ctx(c));
    CPDR_TRY(check_channels("cpdr_plan_glr", channels));
    return check_launched(cpdr::glr_plan(c, channels, backward != 0, out), "cpdr_plan_glr");
}

cpdr_status cpdr_glr_fwd(const cpdr_ctx *c, const void *x, const float *gate, const float *h0, int32_t channels,
                         void *y, float *hT, float *carry, void *stream) {
    CPDR_TRY(check_launch_ctx(c));
    CPDR_TRY(check_channels("cpdr_glr_fwd", channels));
    CPDR_TRY(check_device_ptr(x, "x"));
    CPDR_TRY(check_device_ptr(gate, "gate"));
    CPDR_TRY(check_device_ptr(h0, "h0", true));
    CPDR_TRY(check_device_ptr(y, "y"));
    CPDR_TRY(check_device_ptr(hT, "hT", true));
    CPDR_TRY(check_device_ptr(carry, "carry", true));
    const size_t n = (size_t)c->plan.B * (size_t)c->plan.T * (size_t)channels, es = elem_bytes(c);
    const size_t st = (size_t)c->plan.N * (size_t)channels * 4;
    // hT may be h0: a sequence's state is read by its first step and written by its last
    CPDR_TRY(check_outputs("cpdr_glr_fwd",
                           {{y, n * es, "y"}, {hT, st, "hT"},
                            {carry, (size_t)c->plan.glr_groups * (size_t)channels * 4, "carry"}},
                           {{x, n * es, "x"}, {gate, n * 4, "gate"}, {h0, st, "h0"}}, {{hT, h0}}));
    return check_launched(cpdr::launch_glr_fwd(c, x, gate, h0, channels, y, hT, carry, stream), "cpdr_glr_fwd");
}

cpdr_status cpdr_glr_bwd(const cpdr_ctx *c, const void *x, const float *gate, const float *carry, const void *dy,
                         const float *dhT, int32_t channels, void *dx, float *dgate, float *dh0, void *stream) {
    CPDR_TRY(check_launch_ctx(c));
    CPDR_TRY(check_channels("cpdr_glr_bwd", channels));
    CPDR_TRY(check_device_ptr(x, "x"));
    CPDR_TRY(check_device_ptr(gate, "gate"));
    CPDR_TRY(check_device_ptr(carry, "carry"));
    CPDR_TRY(check_device_ptr(dy, "dy"));
    CPDR_TRY(check_device_ptr(dhT, "dhT", true));
    CPDR_TRY(check_device_ptr(dx, "dx"));
    CPDR_TRY(check_device_ptr(dgate, "dgate"));
    CPDR_TRY(check_device_ptr(dh0, "dh0", true));
    const size_t n = (size_t)c->plan.B * (size_t)c->plan.T * (size_t)channels, es = elem_bytes(c);
    const size_t st = (size_t)c->plan.N * (size_t)channels * 4;
    CPDR_TRY(check_outputs("cpdr_glr_bwd", {{dx, n * es, "dx"}, {dgate, n * 4, "dgate"}, {dh0, st, "dh0"}},
                           {{x, n * es, "x"}, {gate, n * 4, "gate"}, {dy, n * es, "dy"}, {dhT, st, "dhT"},
                            {carry, (size_t)c->plan.glr_groups * (size_t)channels * 4, "carry"}},
                           {{dh0, dhT}}));
    return check_launched(cpdr::launch_glr_bwd(c, x, gate, carry, dy, dhT, channels, dx, dgate, dh0, stream),
                          "cpdr_glr_bwd");
}

cpdr_status cpdr_glr_step(const cpdr_ctx *c, const void *x, const float *gate, const float *state, float *state_out,
                          const int32_t *slots, int32_t n, int32_t num_slots, int32_t channels, void *y, void *stream) {
    CPDR_TRY(check_launch_ctx(c));
    CPDR_TRY(check_channels("cpdr_glr_step", channels));
    if (n < 0 || n > 65535) return fail_with(CPDR_ERR_INVALID, "cpdr_glr_step: n must be 0 .. 65535");
    if (num_slots < 1) return fail_with(CPDR_ERR_INVALID, "cpdr_glr_step: num_slots must be positive");
    if (!slots && n > num_slots)
        return fail_with(CPDR_ERR_INVALID, "cpdr_glr_step: without slots, row i's state is slot i: n must be at most num_slots");
    if (n == 0) return CPDR_OK;
    CPDR_TRY(check_device_ptr(x, "x"));
    CPDR_TRY(check_device_ptr(gate, "gate"));
    CPDR_TRY(check_device_ptr(state, "state"));
    CPDR_TRY(check_device_ptr(state_out, "state_out"));
    if (slots && ((uintptr_t)slots & 3u) != 0)
        return fail_with(CPDR_ERR_INVALID, "cpdr_glr_step: slots not 4-byte aligned");
    CPDR_TRY(check_device_ptr(y, "y"));
    const size_t e = (size_t)n * (size_t)channels, es = elem_bytes(c);
    const size_t st = (size_t)num_slots * (size_t)channels * 4;
    CPDR_TRY(check_outputs("cpdr_glr_step", {{y, e * es, "y"}, {state_out, st, "state_out"}},
                           {{x, e * es, "x"}, {gate, e * 4, "gate"}, {state, st, "state"}, {slots, (size_t)n * 4, "slots"}},
                           {{state_out, state}}));
    return check_launched(cpdr::launch_glr_step(c, x, gate, state, state_out, slots, n, num_slots, channels, y, stream),
                          "cpdr_glr_step");
}

cpdr_status cpdr_rmsnorm_fwd(const cpdr_ctx *c, int64_t rows, int32_t width, const void *x, const void *residual,
                             const float *weight, float eps, void *sum_out, void *y, void *y8, float *scale,
                             void *stream) {
    CPDR_TRY(check_launch_ctx(c));
    CPDR_TRY(check_norm("cpdr_rmsnorm_fwd", rows, width, eps));
    if (rows == 0) return CPDR_OK;
    if (!y && !y8) return fail_with(CPDR_ERR_INVALID, "cpdr_rmsnorm_fwd: neither y nor y8 is given");
    if ((y8 == nullptr) != (scale == nullptr))
        return fail_with(CPDR_ERR_INVALID, "cpdr_rmsnorm_fwd: y8 and scale come together");
    CPDR_TRY(check_device_ptr(x, "x"));
    CPDR_TRY(check_device_ptr(residual, "residual", true));
    CPDR_TRY(check_device_ptr(weight, "weight"));
    CPDR_TRY(check_device_ptr(sum_out, "sum_out", true));
    CPDR_TRY(check_device_ptr(y, "y", true));
    CPDR_TRY(check_device_ptr(y8, "y8", true));
    CPDR_TRY(check_device_ptr(scale, "scale", true));
    const size_t n = (size_t)rows * (size_t)width, es = elem_bytes(c);
    CPDR_TRY(check_outputs("cpdr_rmsnorm_fwd",
                           {{sum_out, n * es, "sum_out"}, {y, n * es, "y"}, {y8, n, "y8"}, {scale, (size_t)rows * 4, "scale"}},
                           {{x, n * es, "x"}, {residual, n * es, "residual"}, {weight, (size_t)width * 4, "weight"}},
                           {{sum_out, x}, {sum_out, residual}, {y, x}, {y, residual}}));
    return check_launched(cpdr::launch_rmsnorm_fwd(c, rows, width, x, residual, weight, eps, sum_out, y, y8, scale, stream),
                          "cpdr_rmsnorm_fwd");
}

cpdr_status cpdr_rmsnorm_bwd_workspace_bytes(const cpdr_ctx *c, int64_t rows, int32_t width, size_t *bytes) {
    CPDR_TRY(check_launch_ctx(c));
    if (!bytes) return fail_with(CPDR_ERR_INVALID, "null argument");
    CPDR_TRY(check_norm("cpdr_rmsnorm_bwd_workspace_bytes", rows, width, 0.f));
    *bytes = norm_workspace(c, rows, width);
    return CPDR_OK;
}

cpdr_status cpdr_rmsnorm_bwd(const cpdr_ctx *c, int64_t rows, int32_t width, const void *s, const float *weight,
                             float eps, const void *dy, const void *dsum, void *ds, float *dweight, void *ws,
                             size_t ws_bytes, void *stream) {
    CPDR_TRY(check_launch_ctx(c));
    CPDR_TRY(check_norm("cpdr_rmsnorm_bwd", rows, width, eps));
    CPDR_TRY(check_device_ptr(s, "s", rows == 0));
    CPDR_TRY(check_device_ptr(weight, "weight"));
    CPDR_TRY(check_device_ptr(dy, "dy", rows == 0));
    CPDR_TRY(check_device_ptr(dsum, "dsum", true));
    CPDR_TRY(check_device_ptr(ds, "ds", rows == 0));
    CPDR_TRY(check_device_ptr(dweight, "dweight"));
    CPDR_TRY(check_device_ptr(ws, "workspace"));
    const size_t n = (size_t)rows * (size_t)width, es = elem_bytes(c), need = norm_workspace(c, rows, width);
    if (ws_bytes < need) return fail_with(CPDR_ERR_WORKSPACE, "cpdr_rmsnorm_bwd: workspace too small");
    CPDR_TRY(check_outputs("cpdr_rmsnorm_bwd",
                           {{ds, n * es, "ds"}, {dweight, (size_t)width * 4, "dweight"}, {ws, need, "workspace"}},
                           {{s, n * es, "s"}, {weight, (size_t)width * 4, "weight"}, {dy, n * es, "dy"}, {dsum, n * es, "dsum"}},
                           {{ds, dy}, {ds, dsum}}));
    return check_launched(cpdr::launch_rmsnorm_bwd(c, rows, width, s, weight, eps, dy, dsum, ds, dweight, (float *)ws, stream),
                          "cpdr_rmsnorm_bwd");
}

cpdr_status cpdr_plan_linear(const cpdr_ctx *c, int64_t rows, int32_t K, int32_t N, int32_t e4m3, int32_t out[2]) {
    if (!c || !out) return fail_with(CPDR_ERR_INVALID, "null argument");
    CPDR_TRY(check_linear("cpdr_plan_linear", c, rows, K, N, 0, e4m3 != 0));
    if (rows == 0) return fail_with(CPDR_ERR_INVALID, "cpdr_plan_linear: no rows");
    cpdr::linear_plan(c, rows, K, N, e4m3 != 0, out);
    return CPDR_OK;
}

cpdr_status cpdr_linear_fwd(const cpdr_ctx *c, int64_t rows, int32_t K, int32_t N, const void *x, const void *w,
                            const float *x_scale, const float *w_scale, const float *bias, int32_t activation,
                            const void *residual, void *z, void *y, void *stream) {
    CPDR_TRY(check_launch_ctx(c));
    if ((x_scale == nullptr) != (w_scale == nullptr) && rows > 0)
        return fail_with(CPDR_ERR_INVALID, "cpdr_linear_fwd: x_scale and w_scale come together");
    const bool e4m3 = w_scale != nullptr;
    CPDR_TRY(check_linear("cpdr_linear_fwd", c, rows, K, N, activation, e4m3));
    if (rows == 0) return CPDR_OK;
    CPDR_TRY(check_device_ptr(x, "x"));
    CPDR_TRY(check_device_ptr(w, "w"));
    CPDR_TRY(check_device_ptr(x_scale, "x_scale", true));
    CPDR_TRY(check_device_ptr(w_scale, "w_scale", true));
    CPDR_TRY(check_device_ptr(bias, "bias", true));
    CPDR_TRY(check_device_ptr(residual, "residual", true));
    CPDR_TRY(check_device_ptr(z, "z", true));
    CPDR_TRY(check_device_ptr(y, "y"));
    const size_t es = e4m3 ? 1 : 2, ny = (size_t)rows * (size_t)N * 2;
    CPDR_TRY(check_outputs("cpdr_linear_fwd", {{y, ny, "y"}, {z, ny, "z"}},
                           {{x, (size_t)rows * (size_t)K * es, "x"}, {w, (size_t)N * (size_t)K * es, "w"},
                            {x_scale, (size_t)rows * 4, "x_scale"}, {w_scale, (size_t)N * 4, "w_scale"},
                            {bias, (size_t)N * 4, "bias"}, {residual, ny, "residual"}},
                           {{y, residual}}));
    return check_launched(cpdr::launch_linear_fwd(c, rows, K, N, x, w, x_scale, w_scale, bias, activation, residual, z, y, stream),
                          "cpdr_linear_fwd");
}

cpdr_status cpdr_linear_bwd_workspace_bytes(const cpdr_ctx *c, int64_t rows, int32_t K, int32_t N, int32_t activation,
                                            size_t *bytes) {
    CPDR_TRY(check_launch_ctx(c));
    if (!bytes) return fail_with(CPDR_ERR_INVALID, "null argument");
    CPDR_TRY(check_linear("cpdr_linear_bwd_workspace_bytes", c, rows, K, N, activation, false));
    *bytes = linear_workspace(c, rows, N, activation);
    return CPDR_OK;
}

cpdr_status cpdr_linear_bwd(const cpdr_ctx *c, int64_t rows, int32_t K, int32_t N, const void *x, const void *w,
                            const void *z, const void *dy, int32_t activation, void *dx, void *dw, float *dbias,
                            void *ws, size_t ws_bytes, void *stream) {
    CPDR_TRY(check_launch_ctx(c));
    CPDR_TRY(check_linear("cpdr_linear_bwd", c, rows, K, N, activation, false));
    const bool none = rows == 0;
    CPDR_TRY(check_device_ptr(x, "x", none || !dw));
    CPDR_TRY(check_device_ptr(w, "w", !dx));
    CPDR_TRY(check_device_ptr(z, "z", none || activation == 0));
    CPDR_TRY(check_device_ptr(dy, "dy", none));
    CPDR_TRY(check_device_ptr(dx, "dx", true));
    CPDR_TRY(check_device_ptr(dw, "dw", true));
    CPDR_TRY(check_device_ptr(dbias, "dbias", true));
    const size_t need = linear_workspace(c, rows, N, activation);
    CPDR_TRY(check_device_ptr(ws, "workspace", need == 0));
    if (ws_bytes < need) return fail_with(CPDR_ERR_WORKSPACE, "cpdr_linear_bwd: workspace too small");
    const size_t nx = (size_t)rows * (size_t)K * 2, nw = (size_t)N * (size_t)K * 2, ny = (size_t)rows * (size_t)N * 2;
    CPDR_TRY(check_outputs("cpdr_linear_bwd", {{dx, nx, "dx"}, {dw, nw, "dw"}, {dbias, (size_t)N * 4, "dbias"}, {ws, need, "workspace"}},
                           {{x, nx, "x"}, {w, nw, "w"}, {activation ? z : nullptr, ny, "z"}, {dy, ny, "dy"}}));
    if (none) {   // sums over no rows
        cudaStream_t st = (cudaStream_t)stream;
        cudaError_t e = dw ? cudaMemsetAsync(dw, 0, nw, st) : cudaSuccess;
        if (e == cudaSuccess && dbias) e = cudaMemsetAsync(dbias, 0, (size_t)N * 4, st);
        return check_launched((int)e, "cpdr_linear_bwd: zero fill");
    }
    float *part = (float *)((char *)ws + linear_dz_bytes(rows, N, activation));
    return check_launched(cpdr::launch_linear_bwd(c, rows, K, N, x, w, z, dy, activation, dx, dw, dbias, ws, part, stream),
                          "cpdr_linear_bwd");
}

}  // extern "C"
