// rotary_api.cu -- C entry points of the rotary positions: argument checks,
// the host-side frequency rules, dispatch to rotary.cu.
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
                              orthros_stream_t stream_) {
    clear_error();
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
    cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_);
    ProfScope ps("rotate", stream);
    const cudaError_t e = launch_rotate(p, d, dtype, stream);
    return e == cudaSuccess ? ORTHROS_OK : cuda_error(e, "rotate launch");
}

size_t orthros_rotate_backward_workspace_size(int n, int H, int d, orthros_dtype dtype) {
    if (n < 0 || H < 1 || H > 65536 || (d != 64 && d != 128) || (dtype != ORTHROS_BF16 && dtype != ORTHROS_F32)) return 0;
    return align_up((size_t)rotate_grad_parts(n, H, d, elem_bytes(dtype)) * 2 * H * d * sizeof(float), 256);
}

orthros_status orthros_rotate_backward(const void *dy, long long dy_stride, const void *x, long long x_stride,
                                       const int32_t *positions, const float *alpha, const uint64_t *steps, int rot_dim,
                                       orthros_rope_layout layout, float amplitude, int n, int H, int d,
                                       orthros_dtype dtype, void *dx, long long dx_stride, float *d_alpha,
                                       float *d_beta, void *workspace, size_t workspace_bytes,
                                       orthros_stream_t stream_) {
    clear_error();
    ORTHROS_TRY(check_rotation(n, H, d, dtype, steps, rot_dim, layout, amplitude));
    if (!aligned16(alpha)) return report_error(ORTHROS_EINVAL, "alpha must be 16-byte aligned");
    if ((d_alpha == nullptr) != (d_beta == nullptr)) return report_error(ORTHROS_EINVAL, "d_alpha and d_beta: both or neither");
    const size_t need = orthros_rotate_backward_workspace_size(n, H, d, dtype);
    if (d_alpha && (!workspace || workspace_bytes < need))
        return report_error(ORTHROS_EWORKSPACE, "workspace needs %zu bytes, got %zu", need, workspace ? workspace_bytes : (size_t)0);
    if (d_alpha && (reinterpret_cast<uintptr_t>(workspace) & 255u) != 0)
        return report_error(ORTHROS_EINVAL, "workspace must be 256-byte aligned");
    cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_);
    if (n == 0) {
        if (d_alpha) {
            cudaError_t e = cudaMemsetAsync(d_alpha, 0, sizeof(float) * (size_t)H * d, stream);
            if (e == cudaSuccess) e = cudaMemsetAsync(d_beta, 0, sizeof(float) * (size_t)H * d, stream);
            if (e != cudaSuccess) return cuda_error(e, "empty gradient");
        }
        return ORTHROS_OK;
    }
    ORTHROS_TRY(check_rows("dy", dy, dy_stride, H, d, dtype, false));
    ORTHROS_TRY(check_rows("dx", dx, dx_stride, H, d, dtype, true));
    if (d_alpha) ORTHROS_TRY(check_rows("x", x, x_stride, H, d, dtype, false));
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
    p.n_part = rotate_grad_parts(n, H, d, elem_bytes(dtype));
    p.d_alpha = d_alpha;
    p.d_beta = d_beta;
    {
        ProfScope ps("rotate_backward", stream);
        const cudaError_t e = launch_rotate_backward(p, d, dtype, stream);
        if (e != cudaSuccess) return cuda_error(e, "rotate backward launch");
    }
    if (d_alpha) {
        ProfScope ps("rotate_grad_sum", stream);
        const cudaError_t e = launch_rotate_grad_sum(p, d, stream);
        if (e != cudaSuccess) return cuda_error(e, "affine gradient launch");
    }
    return ORTHROS_OK;
}

orthros_status orthros_rotate_append(
    const void *q, long long q_stride, const void *q_out, long long q_out_stride, const void *k_new, long long k_stride,
    const void *v_new, long long v_stride, const float *alpha_base, const float *beta_base, const float *alpha_out,
    const float *beta_out, const uint64_t *steps, int rot_dim, orthros_rope_layout layout, float amplitude,
    const int32_t *token_seq, const int32_t *token_pos, const int32_t *out_positions, int n_new, int n_out, int Hq,
    int Hkv, int d, orthros_dtype dtype, void *q_rot, void *q_out_rot, void *k_cache, void *v_cache,
    const int32_t *block_table, int B, int max_pages, int page_size, int num_pages, void *workspace,
    size_t workspace_bytes, orthros_stream_t stream_) {
    clear_error();
    if (n_out < 0) return report_error(ORTHROS_EINVAL, "n_out = %d must be >= 0", n_out);
    if (Hkv < 1 || Hkv > 65536) return report_error(ORTHROS_EINVAL, "Hkv = %d must lie in [1, 65536]", Hkv);
    ORTHROS_TRY(check_rotation(n_new, Hq, d, dtype, n_new + (long long)n_out > 0 ? steps : nullptr, rot_dim, layout, amplitude));
    if (n_out > 0 && !steps) return report_error(ORTHROS_EINVAL, "steps must not be NULL");
    if ((long long)n_new + n_out > 0x7fffffffLL)
        return report_error(ORTHROS_EUNSUPPORTED, "%lld rows exceed 2^31 - 1", (long long)n_new + n_out);
    ORTHROS_TRY(check_affine("_base", alpha_base, beta_base));
    ORTHROS_TRY(check_affine("_out", alpha_out, beta_out));
    if (!workspace || workspace_bytes < kStatusBytes)
        return report_error(ORTHROS_EWORKSPACE, "workspace needs %zu bytes", kStatusBytes);
    if ((reinterpret_cast<uintptr_t>(workspace) & 255u) != 0)
        return report_error(ORTHROS_EINVAL, "workspace must be 256-byte aligned");
    if (n_new > 0) {
        ORTHROS_TRY(check_rows("k_new", k_new, k_stride, Hkv, d, dtype, false));
        ORTHROS_TRY(check_rows("v_new", v_new, v_stride, Hkv, d, dtype, false));
        if (q) {
            ORTHROS_TRY(check_rows("q", q, q_stride, Hq, d, dtype, false));
            if (!q_rot || !aligned16(q_rot)) return report_error(ORTHROS_EINVAL, "q_rot must not be NULL and 16-byte aligned");
        }
        if (!token_seq || !token_pos || !block_table || !k_cache || !v_cache)
            return report_error(ORTHROS_EINVAL, "k_cache, v_cache, block_table, token_seq and token_pos must not be NULL");
        if (!aligned16(k_cache) || !aligned16(v_cache))
            return report_error(ORTHROS_EINVAL, "k_cache and v_cache must be 16-byte aligned");
        if (B < 1 || max_pages < 1 || page_size < 1 || num_pages < 1)
            return report_error(ORTHROS_EINVAL, "B, max_pages, page_size and num_pages must be >= 1");
    }
    if (n_out > 0) {
        ORTHROS_TRY(check_rows("q_out", q_out, q_out_stride, Hq, d, dtype, false));
        if (!q_out_rot || !aligned16(q_out_rot)) return report_error(ORTHROS_EINVAL, "q_out_rot must not be NULL and 16-byte aligned");
        if (!out_positions) return report_error(ORTHROS_EINVAL, "out_positions must not be NULL when n_out > 0");
    }
    cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_);
    uint32_t *status = static_cast<uint32_t *>(workspace);
    if (n_new == 0 && n_out == 0) {
        const cudaError_t e = cudaMemsetAsync(status, 0, sizeof(uint32_t), stream);
        return e == cudaSuccess ? ORTHROS_OK : cuda_error(e, "status reset");
    }
    RotateParams p{};
    p.x = q;
    p.y = q_rot;
    p.x_stride = q_stride;
    p.y_stride = (long long)Hq * d;
    p.positions = token_pos;
    p.alpha = alpha_base;
    p.beta = beta_base;
    p.steps = steps;
    p.n = n_new;
    p.H = Hq;
    p.rot = rot_dim;
    p.interleaved = layout == ORTHROS_ROPE_INTERLEAVED;
    p.amplitude = amplitude;
    p.x_out = q_out;
    p.y_out = q_out_rot;
    p.x_out_stride = q_out_stride;
    p.alpha_out = alpha_out;
    p.beta_out = beta_out;
    p.out_positions = out_positions;
    p.n_out = n_out;
    p.k = k_new;
    p.v = v_new;
    p.k_stride = k_stride;
    p.v_stride = v_stride;
    p.token_seq = token_seq;
    p.block_table = block_table;
    p.k_cache = k_cache;
    p.v_cache = v_cache;
    p.Hkv = Hkv;
    p.B = B;
    p.max_pages = max_pages;
    p.page_size = page_size;
    p.num_pages = num_pages;
    p.status = status;
    ProfScope ps("rotate_append", stream);
    const cudaError_t e = launch_rotate_append(p, d, dtype, stream);
    return e == cudaSuccess ? ORTHROS_OK : cuda_error(e, "rotated append launch");
}

}  // extern "C"
