// rotary_api.cu -- C entry points of the rotary positions, with or without a norm
// of the head: argument checks, the host-side frequency rules, dispatch to
// rotary.cu and norm_rotary.cu.
#include <cmath>

#include "internal.cuh"

namespace orthros {
namespace {

bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

constexpr double kTwoPi = 6.283185307179586476925286766559;

// freq / 2 pi modulo a turn, to the nearest 2^-64 turn. The quotient needs more than a
// double's 53 bits (at position 2^31 those leave 4e-7 rad): freq times 1 / 2 pi, held as the sum
// of two doubles, with the product's own rounding recovered by a fused multiply-add
// (Dekker's two-term product). std::fma throughout, so that every machine gives the same steps.
uint64_t turn_units(double freq) {
    constexpr double kHigh = 0x1.45f306dc9c883p-3, kLow = -0x1.6b01ec5417056p-57;  // 1 / 2 pi
    if (freq < 0) return ~turn_units(-freq) + 1u;  // the opposite (q - floor(q) is exact for q >= 0 only)
    const double q = freq * kHigh;
    double rest = std::fma(freq, kLow, std::fma(freq, kHigh, -q));  // freq / 2 pi - q
    rest = std::fmod(rest, 1.0);
    const double a = std::ldexp(q - std::floor(q), 64);  // [0, 2^64)
    const double b = std::ldexp(std::fabs(rest), 64);    // [0, 2^64)
    const double ai = std::floor(a), bi = std::floor(b);
    const double left = (a - ai) + (rest < 0 ? bi - b : b - bi);  // (-1, 2)
    uint64_t u = static_cast<uint64_t>(ai);
    u += rest < 0 ? ~static_cast<uint64_t>(bi) + 1u : static_cast<uint64_t>(bi);
    return u + static_cast<uint64_t>(static_cast<int64_t>(std::floor(left + 0.5)));
}

int elem_bytes(orthros_dtype t) { return t == ORTHROS_F32 ? 4 : 2; }

// What every rotating call has in common.
orthros_status check_rotation(int n, int H, int d, orthros_dtype dtype, const uint64_t *steps, int rot_dim, orthros_rope_layout layout,
                              float amplitude) {
    if (n < 0) return report_error(ORTHROS_EINVAL, "token count %d must be >= 0", n);
    if (H < 1) return report_error(ORTHROS_EINVAL, "head count %d must be >= 1", H);
    if (dtype != ORTHROS_BF16 && dtype != ORTHROS_F32) return report_error(ORTHROS_EINVAL, "unknown dtype %d", (int)dtype);
    if (d != 64 && d != 128) return report_error(ORTHROS_EUNSUPPORTED, "head size d = %d (supported: 64, 128)", d);
    if (H > 65536) return report_error(ORTHROS_EUNSUPPORTED, "head count %d exceeds 65536", H);
    if (rot_dim < 2 || rot_dim > d || rot_dim % 2 != 0)
        return report_error(ORTHROS_EINVAL, "rot_dim = %d must be even and lie in [2, d = %d]", rot_dim, d);
    if (rot_dim % 16 != 0) return report_error(ORTHROS_EUNSUPPORTED, "rot_dim = %d must be a multiple of 16", rot_dim);
    if (layout != ORTHROS_ROPE_HALF && layout != ORTHROS_ROPE_INTERLEAVED)
        return report_error(ORTHROS_EINVAL, "unknown rotary layout %d", (int)layout);
    if (!std::isfinite(amplitude)) return report_error(ORTHROS_EINVAL, "amplitude must be finite");
    if (n > 0 && !steps) return report_error(ORTHROS_EINVAL, "steps must not be NULL");
    if (reinterpret_cast<uintptr_t>(steps) & 7u) return report_error(ORTHROS_EINVAL, "steps must be 8-byte aligned");
    return ORTHROS_OK;
}

// A [n, H, d] tensor read (or written, `out`) with a token stride.
orthros_status check_rows(const char *name, const void *p, long long stride, int H, int d, orthros_dtype dtype, bool out) {
    if (!p) return report_error(ORTHROS_EINVAL, "%s must not be NULL", name);
    if (!aligned16(p)) return report_error(ORTHROS_EINVAL, "%s must be 16-byte aligned", name);
    if (stride < (out ? (long long)H * d : 0LL) || stride > (1LL << 40) || (stride * elem_bytes(dtype)) % 16 != 0)
        return report_error(ORTHROS_EINVAL, "%s: token stride %lld (a multiple of 16 bytes%s)", name, stride,
                            out ? ", at least H * d" : ", at least 0");
    return ORTHROS_OK;
}

orthros_status check_affine(const char *name, const float *alpha, const float *beta) {
    if ((alpha == nullptr) != (beta == nullptr)) return report_error(ORTHROS_EINVAL, "alpha%s and beta%s: both or neither", name, name);
    if (!aligned16(alpha) || !aligned16(beta)) return report_error(ORTHROS_EINVAL, "alpha%s and beta%s must be 16-byte aligned", name, name);
    return ORTHROS_OK;
}

#define ORTHROS_TRY(expr)                                  \
    do {                                                   \
        const orthros_status st_ = (expr);                 \
        if (st_ != ORTHROS_OK) return st_;                 \
    } while (0)

orthros_status cuda_error(cudaError_t e, const char *what) {
    return report_error(ORTHROS_ECUDA, "%s: %s", what, cudaGetErrorString(e));
}

// The norm of a call that has one.
orthros_status check_norm(const char *name, const float *weight, float eps) {
    if (!std::isfinite(eps) || !(eps > 0.f)) return report_error(ORTHROS_EINVAL, "eps must be finite and > 0");
    if (!aligned16(weight)) return report_error(ORTHROS_EINVAL, "%s must be 16-byte aligned", name);
    return ORTHROS_OK;
}

// orthros_rotate, or with eps > 0 orthros_norm_rotate.
orthros_status rotate_rows(const void *x, long long x_stride, const int32_t *positions, const float *weight, float eps,
                           const float *alpha, const float *beta, const uint64_t *steps, int rot_dim, orthros_rope_layout layout,
                           float amplitude, int n, int H, int d, orthros_dtype dtype, void *y, long long y_stride,
                           cudaStream_t stream, const char *name) {
    ORTHROS_TRY(check_rotation(n, H, d, dtype, steps, rot_dim, layout, amplitude));
    ORTHROS_TRY(check_affine("", alpha, beta));
    if (n == 0) return ORTHROS_OK;
    ORTHROS_TRY(check_rows("x", x, x_stride, H, d, dtype, false));
    ORTHROS_TRY(check_rows("y", y, y_stride, H, d, dtype, true));
    if (x == y && x_stride != y_stride) return report_error(ORTHROS_EINVAL, "in place, x_stride and y_stride must agree");
    if (!positions) return report_error(ORTHROS_EINVAL, "positions must not be NULL");
    RotateParams p{};
    p.x = x;
    p.y = y;
    p.x_stride = x_stride;
    p.y_stride = y_stride;
    p.positions = positions;
    p.alpha = alpha;
    p.beta = beta;
    p.steps = steps;
    p.n = n;
    p.H = H;
    p.rot = rot_dim;
    p.interleaved = layout == ORTHROS_ROPE_INTERLEAVED;
    p.amplitude = amplitude;
    p.eps = eps;
    p.weight = weight;
    ProfScope ps(name, stream);
    const cudaError_t e = eps > 0.f ? launch_norm_rotate(p, d, dtype, stream) : launch_rotate(p, d, dtype, stream);
    return e == cudaSuccess ? ORTHROS_OK : cuda_error(e, name);
}

// Where the gradient sums of a backward call lie in its workspace.
struct GradLayout {
    int parts;
    size_t weight_off, total;
};
GradLayout grad_layout(int n, int H, int d, orthros_dtype dtype, bool norm) {
    GradLayout L;
    L.parts = rotate_grad_parts(n, H, d, elem_bytes(dtype));
    L.weight_off = L.total = align_up((size_t)L.parts * 2 * H * d * sizeof(float), 256);
    if (norm) L.total += align_up((size_t)rotate_grad_groups(H, d, elem_bytes(dtype)) * L.parts * d * sizeof(float), 256);
    return L;
}
bool grad_shape_ok(int n, int H, int d, orthros_dtype dtype) {
    return n >= 0 && H >= 1 && H <= 65536 && (d == 64 || d == 128) && (dtype == ORTHROS_BF16 || dtype == ORTHROS_F32);
}

// orthros_rotate_backward, or with eps > 0 orthros_norm_rotate_backward.
orthros_status rotate_rows_backward(const void *dy, long long dy_stride, const void *x, long long x_stride,
                                    const int32_t *positions, const float *weight, float eps, const float *alpha,
                                    const uint64_t *steps, int rot_dim, orthros_rope_layout layout, float amplitude, int n,
                                    int H, int d, orthros_dtype dtype, void *dx, long long dx_stride, float *d_weight,
                                    float *d_alpha, float *d_beta, void *workspace, size_t workspace_bytes, cudaStream_t stream) {
    const bool norm = eps > 0.f, grads = d_alpha || d_weight;
    ORTHROS_TRY(check_rotation(n, H, d, dtype, steps, rot_dim, layout, amplitude));
    if (!aligned16(alpha)) return report_error(ORTHROS_EINVAL, "alpha must be 16-byte aligned");
    if ((d_alpha == nullptr) != (d_beta == nullptr)) return report_error(ORTHROS_EINVAL, "d_alpha and d_beta: both or neither");
    const GradLayout L = grad_layout(n, H, d, dtype, norm);
    if (grads && (!workspace || workspace_bytes < L.total))
        return report_error(ORTHROS_EWORKSPACE, "workspace needs %zu bytes, got %zu", L.total, workspace ? workspace_bytes : (size_t)0);
    if (grads && (reinterpret_cast<uintptr_t>(workspace) & 255u) != 0)
        return report_error(ORTHROS_EINVAL, "workspace must be 256-byte aligned");
    if (n == 0) {
        cudaError_t e = cudaSuccess;
        if (d_alpha) e = cudaMemsetAsync(d_alpha, 0, sizeof(float) * (size_t)H * d, stream);
        if (d_beta && e == cudaSuccess) e = cudaMemsetAsync(d_beta, 0, sizeof(float) * (size_t)H * d, stream);
        if (d_weight && e == cudaSuccess) e = cudaMemsetAsync(d_weight, 0, sizeof(float) * (size_t)d, stream);
        return e == cudaSuccess ? ORTHROS_OK : cuda_error(e, "empty gradient");
    }
    ORTHROS_TRY(check_rows("dy", dy, dy_stride, H, d, dtype, false));
    ORTHROS_TRY(check_rows("dx", dx, dx_stride, H, d, dtype, true));
    if (norm || d_alpha) ORTHROS_TRY(check_rows("x", x, x_stride, H, d, dtype, false));
    if (dx == dy && dx_stride != dy_stride) return report_error(ORTHROS_EINVAL, "in place, dy_stride and dx_stride must agree");
    if (!positions) return report_error(ORTHROS_EINVAL, "positions must not be NULL");
    RotateBwdParams p{};
    p.dy = dy;
    p.x = x;
    p.dx = dx;
    p.dy_stride = dy_stride;
    p.x_stride = x_stride;
    p.dx_stride = dx_stride;
    p.positions = positions;
    p.alpha = alpha;
    p.steps = steps;
    p.n = n;
    p.H = H;
    p.rot = rot_dim;
    p.interleaved = layout == ORTHROS_ROPE_INTERLEAVED;
    p.amplitude = amplitude;
    p.partial = static_cast<float *>(workspace);
    p.n_part = L.parts;
    p.d_alpha = d_alpha;
    p.d_beta = d_beta;
    p.eps = eps;
    p.weight = weight;
    p.d_weight = d_weight;
    if (d_weight) p.partial_w = reinterpret_cast<float *>(static_cast<uint8_t *>(workspace) + L.weight_off);
    {
        ProfScope ps(norm ? "norm_rotate_backward" : "rotate_backward", stream);
        const cudaError_t e = norm ? launch_norm_rotate_backward(p, d, dtype, stream) : launch_rotate_backward(p, d, dtype, stream);
        if (e != cudaSuccess) return cuda_error(e, "rotate backward launch");
    }
    if (grads) {
        ProfScope ps(norm ? "norm_grad_sum" : "rotate_grad_sum", stream);
        const cudaError_t e = norm ? launch_norm_grad_sum(p, d, elem_bytes(dtype), stream) : launch_rotate_grad_sum(p, d, stream);
        if (e != cudaSuccess) return cuda_error(e, "gradient sum launch");
    }
    return ORTHROS_OK;
}

// What the two appends have in common. Token slots come from `slots`, or, when that is
// null, from token_seq, token_pos and the block table.
struct AppendArgs {
    const void *q, *q_out, *k, *v;
    long long q_stride, q_out_stride, k_stride, v_stride;
    const float *q_weight, *k_weight;
    float eps;
    const float *alpha_base, *beta_base, *alpha_out, *beta_out;
    const uint64_t *steps;
    int rot_dim;
    orthros_rope_layout layout;
    float amplitude;
    const int32_t *slots, *token_seq, *token_pos, *out_positions;
    int n_new, n_out, Hq, Hkv, d;
    orthros_dtype dtype;
    void *q_rot, *q_out_rot, *k_cache, *v_cache;
    const int32_t *block_table;
    int B, max_pages, page_size, num_pages;
    void *workspace;
    size_t workspace_bytes;
};
orthros_status append_rows(const AppendArgs &a, bool by_slot, cudaStream_t stream, const char *name) {
    if (a.n_out < 0) return report_error(ORTHROS_EINVAL, "n_out = %d must be >= 0", a.n_out);
    if (a.Hkv < 1 || a.Hkv > 65536) return report_error(ORTHROS_EINVAL, "Hkv = %d must lie in [1, 65536]", a.Hkv);
    ORTHROS_TRY(check_rotation(a.n_new, a.Hq, a.d, a.dtype, a.n_new + (long long)a.n_out > 0 ? a.steps : nullptr, a.rot_dim,
                               a.layout, a.amplitude));
    if (a.n_out > 0 && !a.steps) return report_error(ORTHROS_EINVAL, "steps must not be NULL");
    if ((long long)a.n_new + a.n_out > 0x7fffffffLL)
        return report_error(ORTHROS_EUNSUPPORTED, "%lld rows exceed 2^31 - 1", (long long)a.n_new + a.n_out);
    ORTHROS_TRY(check_affine("_base", a.alpha_base, a.beta_base));
    ORTHROS_TRY(check_affine("_out", a.alpha_out, a.beta_out));
    if (!a.workspace || a.workspace_bytes < kStatusBytes)
        return report_error(ORTHROS_EWORKSPACE, "workspace needs %zu bytes", kStatusBytes);
    if ((reinterpret_cast<uintptr_t>(a.workspace) & 255u) != 0)
        return report_error(ORTHROS_EINVAL, "workspace must be 256-byte aligned");
    if (a.n_new > 0) {
        ORTHROS_TRY(check_rows("k_new", a.k, a.k_stride, a.Hkv, a.d, a.dtype, false));
        ORTHROS_TRY(check_rows("v_new", a.v, a.v_stride, a.Hkv, a.d, a.dtype, false));
        if (a.q) {
            ORTHROS_TRY(check_rows("q", a.q, a.q_stride, a.Hq, a.d, a.dtype, false));
            if (!a.q_rot || !aligned16(a.q_rot)) return report_error(ORTHROS_EINVAL, "q_rot must not be NULL and 16-byte aligned");
        }
        if (by_slot) {
            if (!a.slots || !a.token_pos || !a.k_cache || !a.v_cache)
                return report_error(ORTHROS_EINVAL, "k_cache, v_cache, token_slots and token_pos must not be NULL");
        } else if (!a.token_seq || !a.token_pos || !a.block_table || !a.k_cache || !a.v_cache) {
            return report_error(ORTHROS_EINVAL, "k_cache, v_cache, block_table, token_seq and token_pos must not be NULL");
        }
        if (!aligned16(a.k_cache) || !aligned16(a.v_cache))
            return report_error(ORTHROS_EINVAL, "k_cache and v_cache must be 16-byte aligned");
        if ((!by_slot && (a.B < 1 || a.max_pages < 1)) || a.page_size < 1 || a.num_pages < 1)
            return report_error(ORTHROS_EINVAL, by_slot ? "page_size and num_pages must be >= 1"
                                                        : "B, max_pages, page_size and num_pages must be >= 1");
    }
    if (a.n_out > 0) {
        ORTHROS_TRY(check_rows("q_out", a.q_out, a.q_out_stride, a.Hq, a.d, a.dtype, false));
        if (!a.q_out_rot || !aligned16(a.q_out_rot)) return report_error(ORTHROS_EINVAL, "q_out_rot must not be NULL and 16-byte aligned");
        if (!a.out_positions) return report_error(ORTHROS_EINVAL, "out_positions must not be NULL when n_out > 0");
    }
    uint32_t *status = static_cast<uint32_t *>(a.workspace);
    if (a.n_new == 0 && a.n_out == 0) {
        const cudaError_t e = cudaMemsetAsync(status, 0, sizeof(uint32_t), stream);
        return e == cudaSuccess ? ORTHROS_OK : cuda_error(e, "status reset");
    }
    RotateParams p{};
    p.x = a.q;
    p.y = a.q_rot;
    p.x_stride = a.q_stride;
    p.y_stride = (long long)a.Hq * a.d;
    p.positions = a.token_pos;
    p.alpha = a.alpha_base;
    p.beta = a.beta_base;
    p.steps = a.steps;
    p.n = a.n_new;
    p.H = a.Hq;
    p.rot = a.rot_dim;
    p.interleaved = a.layout == ORTHROS_ROPE_INTERLEAVED;
    p.amplitude = a.amplitude;
    p.eps = a.eps;
    p.weight = a.q_weight;
    p.k_weight = a.k_weight;
    p.x_out = a.q_out;
    p.y_out = a.q_out_rot;
    p.x_out_stride = a.q_out_stride;
    p.alpha_out = a.alpha_out;
    p.beta_out = a.beta_out;
    p.out_positions = a.out_positions;
    p.n_out = a.n_out;
    p.k = a.k;
    p.v = a.v;
    p.k_stride = a.k_stride;
    p.v_stride = a.v_stride;
    p.slots = a.slots;
    p.token_seq = a.token_seq;
    p.block_table = a.block_table;
    p.k_cache = a.k_cache;
    p.v_cache = a.v_cache;
    p.Hkv = a.Hkv;
    p.B = a.B;
    p.max_pages = a.max_pages;
    p.page_size = a.page_size;
    p.num_pages = a.num_pages;
    p.status = status;
    ProfScope ps(name, stream);
    const cudaError_t e = a.eps > 0.f ? launch_norm_rotate(p, a.d, a.dtype, stream) : launch_rotate_append(p, a.d, a.dtype, stream);
    return e == cudaSuccess ? ORTHROS_OK : cuda_error(e, name);
}

}  // namespace
}  // namespace orthros

using namespace orthros;

extern "C" {

orthros_status orthros_rotary_frequencies(int rot_dim, double base, orthros_rope_scaling rule, double factor,
                                          double original_length, double low_turns, double high_turns, double *freq,
                                          float *amplitude) {
    clear_error();
    if (rot_dim < 2 || rot_dim % 2 != 0) return report_error(ORTHROS_EINVAL, "rot_dim = %d must be even and >= 2", rot_dim);
    if (!(base > 1.0) || !std::isfinite(base)) return report_error(ORTHROS_EINVAL, "base must be finite and > 1");
    if (!freq || !amplitude) return report_error(ORTHROS_EINVAL, "freq and amplitude must not be NULL");
    const int r = (int)rule;
    if (r < ORTHROS_ROPE_PLAIN || r > ORTHROS_ROPE_BANDS_TEMPERED)
        return report_error(ORTHROS_EINVAL, "unknown scaling rule %d", r);
    const bool bands = r == ORTHROS_ROPE_BANDS || r == ORTHROS_ROPE_BANDS_TEMPERED;
    if (r != ORTHROS_ROPE_PLAIN && (!(factor >= 1.0) || !std::isfinite(factor)))
        return report_error(ORTHROS_EINVAL, "factor must be finite and >= 1");
    if (r == ORTHROS_ROPE_STRETCH && rot_dim < 4) return report_error(ORTHROS_EINVAL, "STRETCH needs rot_dim >= 4");
    if (bands && (!(original_length > 0.0) || !std::isfinite(original_length) || !(low_turns >= 0.0) ||
                  !(high_turns > low_turns) || !std::isfinite(high_turns)))
        return report_error(ORTHROS_EINVAL, "BANDS needs original_length > 0 and 0 <= low_turns < high_turns, all finite");
    if (r == ORTHROS_ROPE_STRETCH) base *= std::pow(factor, (double)rot_dim / (rot_dim - 2));
    for (int i = 0; i < rot_dim / 2; ++i) {
        const double f = std::pow(base, -2.0 * i / rot_dim);
        freq[i] = f;
        if (r == ORTHROS_ROPE_LINEAR) freq[i] = f / factor;
        if (bands) {
            const double turns = original_length * f / kTwoPi;
            const double s = std::fmin(1.0, std::fmax(0.0, (turns - low_turns) / (high_turns - low_turns)));
            freq[i] = (1.0 - s) * f / factor + s * f;
        }
    }
    *amplitude = r == ORTHROS_ROPE_BANDS_TEMPERED ? (float)(0.1 * std::log(factor) + 1.0) : 1.f;
    return ORTHROS_OK;
}

orthros_status orthros_rotary_steps(const double *freq, int n, uint64_t *steps) {
    clear_error();
    if (n < 0) return report_error(ORTHROS_EINVAL, "n = %d must be >= 0", n);
    if (n > 0 && (!freq || !steps)) return report_error(ORTHROS_EINVAL, "freq and steps must not be NULL");
    for (int i = 0; i < n; ++i)
        if (!std::isfinite(freq[i])) return report_error(ORTHROS_EINVAL, "freq[%d] is not finite", i);
    for (int i = 0; i < n; ++i) steps[i] = turn_units(freq[i]);
    return ORTHROS_OK;
}

orthros_status orthros_rotate(const void *x, long long x_stride, const int32_t *positions, const float *alpha,
                              const float *beta, const uint64_t *steps, int rot_dim, orthros_rope_layout layout,
                              float amplitude, int n, int H, int d, orthros_dtype dtype, void *y, long long y_stride,
                              orthros_stream_t stream) {
    clear_error();
    return rotate_rows(x, x_stride, positions, nullptr, 0.f, alpha, beta, steps, rot_dim, layout, amplitude, n, H, d, dtype, y,
                       y_stride, reinterpret_cast<cudaStream_t>(stream), "rotate");
}

orthros_status orthros_norm_rotate(const void *x, long long x_stride, const int32_t *positions, const float *weight, float eps,
                                   const float *alpha, const float *beta, const uint64_t *steps, int rot_dim,
                                   orthros_rope_layout layout, float amplitude, int n, int H, int d, orthros_dtype dtype,
                                   void *y, long long y_stride, orthros_stream_t stream) {
    clear_error();
    ORTHROS_TRY(check_norm("weight", weight, eps));
    return rotate_rows(x, x_stride, positions, weight, eps, alpha, beta, steps, rot_dim, layout, amplitude, n, H, d, dtype, y,
                       y_stride, reinterpret_cast<cudaStream_t>(stream), "norm_rotate");
}

size_t orthros_rotate_backward_workspace_size(int n, int H, int d, orthros_dtype dtype) {
    return grad_shape_ok(n, H, d, dtype) ? grad_layout(n, H, d, dtype, false).total : 0;
}

size_t orthros_norm_rotate_backward_workspace_size(int n, int H, int d, orthros_dtype dtype) {
    return grad_shape_ok(n, H, d, dtype) ? grad_layout(n, H, d, dtype, true).total : 0;
}

orthros_status orthros_rotate_backward(const void *dy, long long dy_stride, const void *x, long long x_stride,
                                       const int32_t *positions, const float *alpha, const uint64_t *steps, int rot_dim,
                                       orthros_rope_layout layout, float amplitude, int n, int H, int d,
                                       orthros_dtype dtype, void *dx, long long dx_stride, float *d_alpha,
                                       float *d_beta, void *workspace, size_t workspace_bytes, orthros_stream_t stream) {
    clear_error();
    return rotate_rows_backward(dy, dy_stride, x, x_stride, positions, nullptr, 0.f, alpha, steps, rot_dim, layout, amplitude, n,
                                H, d, dtype, dx, dx_stride, nullptr, d_alpha, d_beta, workspace, workspace_bytes,
                                reinterpret_cast<cudaStream_t>(stream));
}

orthros_status orthros_norm_rotate_backward(const void *dy, long long dy_stride, const void *x, long long x_stride,
                                            const int32_t *positions, const float *weight, float eps, const float *alpha,
                                            const uint64_t *steps, int rot_dim, orthros_rope_layout layout, float amplitude,
                                            int n, int H, int d, orthros_dtype dtype, void *dx, long long dx_stride,
                                            float *d_weight, float *d_alpha, float *d_beta, void *workspace,
                                            size_t workspace_bytes, orthros_stream_t stream) {
    clear_error();
    ORTHROS_TRY(check_norm("weight", weight, eps));
    return rotate_rows_backward(dy, dy_stride, x, x_stride, positions, weight, eps, alpha, steps, rot_dim, layout, amplitude, n, H,
                                d, dtype, dx, dx_stride, d_weight, d_alpha, d_beta, workspace, workspace_bytes,
                                reinterpret_cast<cudaStream_t>(stream));
}

orthros_status orthros_rotate_append(
    const void *q, long long q_stride, const void *q_out, long long q_out_stride, const void *k_new, long long k_stride,
    const void *v_new, long long v_stride, const float *alpha_base, const float *beta_base, const float *alpha_out,
    const float *beta_out, const uint64_t *steps, int rot_dim, orthros_rope_layout layout, float amplitude,
    const int32_t *token_seq, const int32_t *token_pos, const int32_t *out_positions, int n_new, int n_out, int Hq,
    int Hkv, int d, orthros_dtype dtype, void *q_rot, void *q_out_rot, void *k_cache, void *v_cache,
    const int32_t *block_table, int B, int max_pages, int page_size, int num_pages, void *workspace,
    size_t workspace_bytes, orthros_stream_t stream) {
    clear_error();
    const AppendArgs a{q, q_out, k_new, v_new, q_stride, q_out_stride, k_stride, v_stride, nullptr, nullptr, 0.f, alpha_base,
                       beta_base, alpha_out, beta_out, steps, rot_dim, layout, amplitude, nullptr, token_seq, token_pos,
                       out_positions, n_new, n_out, Hq, Hkv, d, dtype, q_rot, q_out_rot, k_cache, v_cache, block_table, B,
                       max_pages, page_size, num_pages, workspace, workspace_bytes};
    return append_rows(a, false, reinterpret_cast<cudaStream_t>(stream), "rotate_append");
}

orthros_status orthros_norm_rotate_append(
    const void *q, long long q_stride, const void *q_out, long long q_out_stride, const void *k_new, long long k_stride,
    const void *v_new, long long v_stride, const float *q_weight, const float *k_weight, float eps, const float *alpha_base,
    const float *beta_base, const float *alpha_out, const float *beta_out, const uint64_t *steps, int rot_dim,
    orthros_rope_layout layout, float amplitude, const int32_t *token_slots, const int32_t *token_pos,
    const int32_t *out_positions, int n_new, int n_out, int Hq, int Hkv, int d, orthros_dtype dtype, void *q_rot,
    void *q_out_rot, void *k_cache, void *v_cache, int page_size, int num_pages, void *workspace, size_t workspace_bytes,
    orthros_stream_t stream) {
    clear_error();
    if (eps == 0.f) {
        if (q_weight || k_weight) return report_error(ORTHROS_EINVAL, "eps = 0 (no norm): q_weight and k_weight must be NULL");
    } else {
        ORTHROS_TRY(check_norm("q_weight", q_weight, eps));
        ORTHROS_TRY(check_norm("k_weight", k_weight, eps));
    }
    const AppendArgs a{q, q_out, k_new, v_new, q_stride, q_out_stride, k_stride, v_stride, q_weight, k_weight, eps, alpha_base,
                       beta_base, alpha_out, beta_out, steps, rot_dim, layout, amplitude, token_slots, nullptr, token_pos,
                       out_positions, n_new, n_out, Hq, Hkv, d, dtype, q_rot, q_out_rot, k_cache, v_cache, nullptr, 0,
                       0, page_size, num_pages, workspace, workspace_bytes};
    return append_rows(a, true, reinterpret_cast<cudaStream_t>(stream), "norm_rotate_append");
}

}  // extern "C"
