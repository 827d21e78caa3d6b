// ops.cpp -- the C ABI declared in include/sparseloco_ops.h: host-side
// argument checks and launches.  No allocation and no synchronisation.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <cmath>

#include "ops_internal.h"
#include "sparseloco_ops.h"

namespace {

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

bool overlap(const void* a, size_t na, const void* b, size_t nb) {
    const uintptr_t x = reinterpret_cast<uintptr_t>(a);
    const uintptr_t y = reinterpret_cast<uintptr_t>(b);
    return na && nb && x < y + nb && y < x + na;
}

sl_status from_hip(hipError_t e) { return e == hipSuccess ? SL_OK : SL_ERR_HIP; }

bool known_type(int32_t t) { return t == SL_F32 || t == SL_BF16 || t == SL_F16; }
size_t bytes_of(int32_t t) { return t == SL_F32 ? 4 : 2; }

constexpr int64_t kMaxBytes = int64_t(1) << 46;  // of any one operand

// a * b, or -1 where it passes kMaxBytes (both >= 0).
int64_t product(int64_t a, int64_t b) { return a < 0 || b < 0 || (b && a > kMaxBytes / b) ? -1 : a * b; }

// Elements from the first to the last of a strided batch of matrices (none
// empty), or -1 if it is too large.
int64_t extent(int64_t rows, int64_t cols, int64_t count, int64_t ld, int64_t stride) {
    const int64_t one = product(rows - 1, ld), all = product(count - 1, stride);
    if (one < 0 || all < 0 || one + all + cols > kMaxBytes / 4) return -1;
    return one + all + cols;
}

// The largest |a s + b s^3 + c s^5| for s in [0, top]: at top or where the
// derivative a + 3 b q + 5 c q^2 (q = s^2) is zero.
double largest_value(double a, double b, double c, double top) {
    auto f = [&](double q) { return std::fabs(std::sqrt(q) * (a + b * q + c * q * q)); };
    double most = f(top * top);
    auto meet = [&](double q) { if (q > 0 && q < top * top) most = std::max(most, f(q)); };
    if (c == 0) {
        if (b != 0) meet(-a / (3 * b));
    } else {
        const double d = 9 * b * b - 20 * a * c;
        if (d >= 0) {
            meet((-3 * b + std::sqrt(d)) / (10 * c));
            meet((-3 * b - std::sqrt(d)) / (10 * c));
        }
    }
    return most;
}

// The largest |b q + c q^2| for q in [0, top].
double largest_poly(double b, double c, double top) {
    auto f = [&](double q) { return std::fabs(b * q + c * q * q); };
    double most = f(top);
    if (c != 0 && -b / (2 * c) > 0 && -b / (2 * c) < top) most = std::max(most, f(-b / (2 * c)));
    return most;
}

// The largest |a + b q + c q^2| for q in [0, top].
double largest_factor(double a, double b, double c, double top) {
    auto f = [&](double q) { return std::fabs(a + b * q + c * q * q); };
    double most = std::max(f(0), f(top));
    if (c != 0 && -b / (2 * c) > 0 && -b / (2 * c) < top) most = std::max(most, f(-b / (2 * c)));
    return most;
}

// Reads the steps and refuses those whose fp16 operands could overflow.
sl_status read_steps(const float* coefficients, int32_t n, sl::Quintic* steps, sl::UpdateArgs* u) {
    if (n < 1 || n > SL_MAX_STEPS || !coefficients) return SL_ERR_INVALID_ARG;
    double product = 1, grown = 1;
    double top = 1.01;  // the start's largest singular value is at most 1, up to rounding
    for (int32_t k = 0; k < n; ++k) {
        const float a = coefficients[3 * k], b = coefficients[3 * k + 1], c = coefficients[3 * k + 2];
        if (!std::isfinite(a) || !std::isfinite(b) || !std::isfinite(c)) return SL_ERR_INVALID_ARG;
        if (!(top <= 3.8) || !(largest_poly(b, c, top * top) <= 30)) return SL_ERR_INVALID_ARG;
        const double factor = largest_factor(a, b, c, top * top);
        if (!(factor <= 1e4)) return SL_ERR_INVALID_ARG;
        product *= factor;
        u->factors[k] = (float)factor;
        grown = std::max(grown, factor > 100 ? 1e30 : product);
        top = largest_value(a, b, c, top);
        steps[k] = {a, b, c};
    }
    u->growth = (float)std::min(grown, 1e30);
    return SL_OK;
}

// Sizes of sl_orthogonalize and sl_muon_step; *noop where there is nothing to do.
sl_status check_sizes(int64_t rows, int64_t cols, int64_t count, int32_t products, bool* noop) {
    *noop = false;
    if (products != SL_PRODUCTS_F16 && products != SL_PRODUCTS_SPLIT) return SL_ERR_INVALID_ARG;
    if (rows < 0 || cols < 0 || count < 0 || rows > SL_MAX_SIDE || cols > SL_MAX_SIDE) return SL_ERR_SHAPE;
    if (rows == 0 || cols == 0 || count == 0) {
        *noop = true;
        return SL_OK;
    }
    // Beyond this a launch's blocks would not fit 31 bits (and no memory would hold the operands).
    const int64_t one = product(rows, cols);
    if (count > 65535 || product(one, count) < 0 || product(one, count) > (int64_t(1) << 40)) return SL_ERR_SHAPE;
    const int64_t side = std::min(rows, cols);
    if (product(product(side, side), count) > (int64_t(1) << 40)) return SL_ERR_SHAPE;
    return SL_OK;
}

int64_t update_workspace(int64_t rows, int64_t cols, int64_t count, int32_t products, bool update) {
    bool noop = false;
    if (check_sizes(rows, cols, count, products, &noop) != SL_OK) return -1;
    return noop ? 0 : (int64_t)sl::update_workspace_bytes(rows, cols, count, products == SL_PRODUCTS_SPLIT, update);
}

sl_status check_workspace(const void* workspace, int64_t bytes, int64_t need) {
    if (need == 0) return SL_OK;
    if (!workspace || bytes < need) return SL_ERR_INVALID_ARG;
    return aligned(workspace, 256) ? SL_OK : SL_ERR_ALIGN;
}

}  // namespace

extern "C" {

int64_t sl_orthogonalize_workspace(int64_t rows, int64_t cols, int64_t count, int32_t products) {
    return update_workspace(rows, cols, count, products, false);
}

int64_t sl_muon_step_workspace(int64_t rows, int64_t cols, int64_t count, int32_t products) {
    return update_workspace(rows, cols, count, products, true);
}

sl_status sl_orthogonalize(const void* x, int32_t x_type, int64_t x_ld, int64_t x_stride, void* out,
                           int32_t out_type, int64_t out_ld, int64_t out_stride, int64_t rows, int64_t cols,
                           int64_t count, const float* coefficients, int32_t n_steps, float eps, int32_t products,
                           void* workspace, int64_t workspace_bytes, void* stream) {
    bool noop = false;
    sl_status st = check_sizes(rows, cols, count, products, &noop);
    if (st != SL_OK) return st;
    if (!known_type(x_type) || !known_type(out_type) || !std::isfinite(eps) || eps < 0) return SL_ERR_INVALID_ARG;
    sl::Quintic steps[SL_MAX_STEPS];
    sl::UpdateArgs u = {};
    st = read_steps(coefficients, n_steps, steps, &u);
    if (st != SL_OK || noop) return st;
    if (!x || !out) return SL_ERR_INVALID_ARG;
    if (x_ld < cols || out_ld < cols) return SL_ERR_SHAPE;
    if (count > 1 && (x_stride < 0 || out_stride < (rows - 1) * out_ld + cols)) return SL_ERR_SHAPE;
    if (count == 1) x_stride = out_stride = 0;
    const int64_t nx = extent(rows, cols, count, x_ld, x_stride), no = extent(rows, cols, count, out_ld, out_stride);
    if (nx < 0 || no < 0) return SL_ERR_SHAPE;
    if (!aligned(x, bytes_of(x_type)) || !aligned(out, bytes_of(out_type))) return SL_ERR_ALIGN;
    const int64_t need = update_workspace(rows, cols, count, products, false);
    st = check_workspace(workspace, workspace_bytes, need);
    if (st != SL_OK) return st;
    const size_t bx = nx * bytes_of(x_type), bo = no * bytes_of(out_type);
    if (overlap(x, bx, out, bo) || overlap(workspace, need, x, bx) || overlap(workspace, need, out, bo))
        return SL_ERR_INVALID_ARG;
    u.rows = rows, u.cols = cols, u.count = count;
    u.x = {const_cast<void*>(x), x_type, x_ld, x_stride};
    u.out = {out, out_type, out_ld, out_stride};
    u.steps = steps, u.n_steps = n_steps, u.eps = eps, u.split = products == SL_PRODUCTS_SPLIT;
    return from_hip(sl::launch_update(u, workspace, static_cast<hipStream_t>(stream)));
}

sl_status sl_muon_step(void* theta, int32_t theta_type, float* momentum, const void* grad, int32_t grad_type,
                       int64_t rows, int64_t cols, int64_t count, float grad_scale, float decay, int32_t nesterov,
                       float lr, float weight_decay, float update_scale, const float* coefficients, int32_t n_steps,
                       float eps, int32_t products, void* workspace, int64_t workspace_bytes, void* stream) {
    bool noop = false;
    sl_status st = check_sizes(rows, cols, count, products, &noop);
    if (st != SL_OK) return st;
    if ((theta_type != SL_F32 && theta_type != SL_BF16) || (grad_type != SL_F32 && grad_type != SL_BF16))
        return SL_ERR_INVALID_ARG;
    for (float v : {grad_scale, decay, lr, weight_decay, update_scale, eps})
        if (!std::isfinite(v)) return SL_ERR_INVALID_ARG;
    const float keep = (float)(1.0 - (double)lr * weight_decay), move = (float)((double)lr * update_scale);
    if (eps < 0 || !std::isfinite(keep) || !std::isfinite(move)) return SL_ERR_INVALID_ARG;
    sl::Quintic steps[SL_MAX_STEPS];
    sl::UpdateArgs u = {};
    st = read_steps(coefficients, n_steps, steps, &u);
    if (st != SL_OK || noop) return st;
    if (!theta || !momentum || !grad) return SL_ERR_INVALID_ARG;
    if (!aligned(theta, 16) || !aligned(momentum, 16) || !aligned(grad, 16)) return SL_ERR_ALIGN;
    const int64_t need = update_workspace(rows, cols, count, products, true);
    st = check_workspace(workspace, workspace_bytes, need);
    if (st != SL_OK) return st;
    const int64_t one = rows * cols;
    const size_t n = (size_t)(one * count);
    const void* bufs[4] = {theta, momentum, grad, workspace};
    const size_t lens[4] = {n * bytes_of(theta_type), n * 4, n * bytes_of(grad_type), (size_t)need};
    for (int a = 0; a < 4; ++a)
        for (int b = 0; b < a; ++b)
            if (overlap(bufs[a], lens[a], bufs[b], lens[b])) return SL_ERR_INVALID_ARG;
    u.rows = rows, u.cols = cols, u.count = count;
    u.x = {const_cast<void*>(grad), grad_type, cols, one};
    u.momentum = momentum;
    u.grad_scale = grad_scale, u.decay = decay, u.nesterov = nesterov != 0;
    u.out = {theta, theta_type, cols, one};
    u.keep = keep, u.move = move;
    u.steps = steps, u.n_steps = n_steps, u.eps = eps, u.split = products == SL_PRODUCTS_SPLIT;
    return from_hip(sl::launch_update(u, workspace, static_cast<hipStream_t>(stream)));
}

int64_t sl_token_logprobs_workspace(int64_t rows, int64_t vocab, int32_t type, int32_t n_top) {
    if (!known_type(type) || n_top < 0 || n_top > SL_MAX_ALTERNATIVES) return -1;
    if (rows < 0 || rows > 0x7fffffff || vocab < 1 || vocab > SL_MAX_VOCAB) return -1;
    return rows == 0 ? 0 : (int64_t)sl::logprob_workspace_bytes(rows, vocab, type, n_top);
}

sl_status sl_token_logprobs(const void* logits, int32_t type, int64_t ld, const int64_t* targets, int64_t rows,
                            int64_t vocab, int32_t n_top, float* logprob, float* entropy, float* top_logprob,
                            int32_t* top_index, void* workspace, int64_t workspace_bytes, void* stream) {
    if (!known_type(type) || n_top < 0 || n_top > SL_MAX_ALTERNATIVES) return SL_ERR_INVALID_ARG;
    if (rows < 0 || rows > 0x7fffffff || vocab < 1 || vocab > SL_MAX_VOCAB) return SL_ERR_SHAPE;
    if (rows == 0) return SL_OK;
    if (ld < vocab) return SL_ERR_SHAPE;
    if (!logits || (logprob && !targets) || (n_top && (!top_logprob || !top_index))) return SL_ERR_INVALID_ARG;
    if (!aligned(logits, bytes_of(type)) || !aligned(targets, 8) || !aligned(logprob, 4) || !aligned(entropy, 4) ||
        !aligned(top_logprob, 4) || !aligned(top_index, 4))
        return SL_ERR_ALIGN;
    const int64_t elements = extent(rows, vocab, 1, ld, 0);
    if (elements < 0) return SL_ERR_SHAPE;
    const int64_t need = sl_token_logprobs_workspace(rows, vocab, type, n_top);
    const sl_status st = check_workspace(workspace, workspace_bytes, need);
    if (st != SL_OK) return st;
    if (!n_top) top_logprob = nullptr, top_index = nullptr;
    // Everything written against everything.
    const void* bufs[7] = {logprob, entropy, top_logprob, top_index, workspace, logits, targets};
    const size_t n = (size_t)rows;
    const size_t lens[7] = {logprob ? n * 4 : 0, entropy ? n * 4 : 0, top_logprob ? n * n_top * 4 : 0,
                            top_index ? n * n_top * 4 : 0, (size_t)need, (size_t)elements * bytes_of(type),
                            targets ? n * 8 : 0};
    for (int a = 0; a < 5; ++a)
        for (int b = a + 1; b < 7; ++b)
            if (overlap(bufs[a], lens[a], bufs[b], lens[b])) return SL_ERR_INVALID_ARG;
    const sl::LogprobArgs args = {logits, type, ld, targets, rows, vocab, n_top, logprob, entropy, top_logprob, top_index};
    return from_hip(sl::launch_logprobs(args, workspace, static_cast<hipStream_t>(stream)));
}

}  // extern "C"
