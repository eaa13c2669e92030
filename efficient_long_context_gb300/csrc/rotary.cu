// rotary.cu -- rotary positions: the affine of a query stream followed by the
// rotation of its channel pairs, the gradient of both, and the paged append
// that rotates new keys on their way into the cache.
//
// Mathematics. Pair i of a head at position t turns by the angle t * f_i:
//   (y_a, y_b) = m (u_a cos - u_b sin, u_a sin + u_b cos),  u = alpha (.) x + beta,
// over the first `rot` channels (pairs (i, i + rot/2) or (2i, 2i + 1)); the
// other channels leave as u. The rotation is orthogonal, so its gradient is the
// rotation by the opposite angle: g = m R(-t) dy, dx = alpha (.) g,
// d_alpha = sum_t g (.) x, d_beta = sum_t g.
//
// Angles. t * f_i in fp32 loses its fraction at long positions (an ulp at
// t = 131072, f = 1 is 0.008 rad), so frequencies arrive as 64-bit fixed-point
// fractions of a turn: the phase of position t is the low 64 bits of t * step,
// an integer product that wraps as the angle does. Its top 32 bits (2^-32 turn,
// 1.5e-9 rad) go through sincospif; sin and cos are good to about 1e-7 at every
// 32-bit position, negative ones included.
//
// Arithmetic is fp32 throughout, rounded once to the element type on the store;
// the affine's gradients are accumulated and returned in fp32.
#include "internal.cuh"

namespace orthros {
namespace {

// A row (one head of one token) is moved in work items of two 16-byte vectors:
// a rotated item holds VEC pairs (vectors i and i + rot/2/VEC in the half
// layout, vectors 2i and 2i + 1 in the interleaved one); the channels past
// `rot` are items of two consecutive vectors. rot is a multiple of 16, so no
// vector is split between the two kinds.
template <typename T> struct Vec {
    static constexpr int kN = 16 / (int)sizeof(T);
};

template <typename T> __device__ __forceinline__ void unpack(const uint4 &r, float (&f)[Vec<T>::kN]);
template <> __device__ __forceinline__ void unpack<float>(const uint4 &r, float (&f)[4]) {
    f[0] = __uint_as_float(r.x);
    f[1] = __uint_as_float(r.y);
    f[2] = __uint_as_float(r.z);
    f[3] = __uint_as_float(r.w);
}
template <> __device__ __forceinline__ void unpack<__nv_bfloat16>(const uint4 &r, float (&f)[8]) {
    const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        f[2 * i] = __uint_as_float(w[i] << 16);
        f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
}
template <typename T> __device__ __forceinline__ uint4 pack(const float (&f)[Vec<T>::kN]);
template <> __device__ __forceinline__ uint4 pack<float>(const float (&f)[4]) {
    return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
}
template <> __device__ __forceinline__ uint4 pack<__nv_bfloat16>(const float (&f)[8]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t *>(&h);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// cos and sin of position t's angle for one frequency step, times the amplitude.
__device__ __forceinline__ void angle(int t, uint64_t step, float amp, float &c, float &s) {
    const uint64_t phase = static_cast<uint64_t>(static_cast<int64_t>(t)) * step;  // modulo one turn
    const int hi = static_cast<int>(static_cast<uint32_t>(phase >> 32));           // in units of 2^-32 turn
    sincospif(static_cast<float>(hi) * 4.656612873077393e-10f, &s, &c);            // 2 pi hi 2^-32 = pi (hi 2^-31)
    c *= amp;
    s *= amp;
}

// Where the two vectors of item i start, in channels.
template <int VEC>
__device__ __forceinline__ void item_channels(int i, int rot, bool interleaved, int &ca, int &cb) {
    const bool split = !interleaved && 2 * VEC * i < rot;  // a rotated item of the half layout
    ca = split ? VEC * i : 2 * VEC * i;
    cb = split ? VEC * i + (rot >> 1) : 2 * VEC * i + VEC;
}

// Rotates the pairs of an item in place: (a[j], b[j]) in the half layout,
// neighbours of the 2 VEC channels in the interleaved one.
template <int VEC>
__device__ __forceinline__ void turn(float (&a)[VEC], float (&b)[VEC], const float (&c)[VEC], const float (&s)[VEC],
                                     bool interleaved) {
    if (!interleaved) {
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
            const float x = a[j], y = b[j];
            a[j] = fmaf(x, c[j], -y * s[j]);
            b[j] = fmaf(x, s[j], y * c[j]);
        }
    } else {
#pragma unroll
        for (int j = 0; j < VEC / 2; ++j) {
            const float x = a[2 * j], y = a[2 * j + 1];
            a[2 * j] = fmaf(x, c[j], -y * s[j]);
            a[2 * j + 1] = fmaf(x, s[j], y * c[j]);
        }
#pragma unroll
        for (int j = 0; j < VEC / 2; ++j) {
            const float x = b[2 * j], y = b[2 * j + 1];
            b[2 * j] = fmaf(x, c[VEC / 2 + j], -y * s[VEC / 2 + j]);
            b[2 * j + 1] = fmaf(x, s[VEC / 2 + j], y * c[VEC / 2 + j]);
        }
    }
}

template <int VEC>
__device__ __forceinline__ void load_affine(const float *p, int ca, int cb, float (&a)[VEC], float (&b)[VEC]) {
#pragma unroll
    for (int j = 0; j < VEC; j += 4) {
        const float4 x = __ldg(reinterpret_cast<const float4 *>(p + ca + j));
        const float4 y = __ldg(reinterpret_cast<const float4 *>(p + cb + j));
        a[j] = x.x, a[j + 1] = x.y, a[j + 2] = x.z, a[j + 3] = x.w;
        b[j] = y.x, b[j + 1] = y.y, b[j + 2] = y.z, b[j + 3] = y.w;
    }
}

// ---------------------------------------------------------------------------
// Forward. A thread owns one (token, item) and walks heads, so the item's
// cosines and sines stay in registers; a warp's lanes are the items of a few
// tokens at the same head, so its affine loads are shared. Bound by HBM: every
// element read once and written once.
// ---------------------------------------------------------------------------
constexpr int kFwdThreads = 128;
constexpr int kHeadsInFlight = 4;  // heads whose loads a thread has in flight

// Heads [h0, h1) of one token's item: src and dst point at the token's head 0.
template <typename T, int D>
__device__ __forceinline__ void rotate_heads(const T *src, T *dst, int h0, int h1, int ca, int cb, bool rotated,
                                             bool interleaved, const float *alpha, const float *beta,
                                             const float (&c)[Vec<T>::kN], const float (&s)[Vec<T>::kN]) {
    constexpr int VEC = Vec<T>::kN;
    for (int hb = h0; hb < h1; hb += kHeadsInFlight) {
        uint4 ra[kHeadsInFlight], rb[kHeadsInFlight];
#pragma unroll
        for (int u = 0; u < kHeadsInFlight; ++u) {
            if (hb + u < h1) {
                ra[u] = __ldcs(reinterpret_cast<const uint4 *>(src + (hb + u) * D + ca));
                rb[u] = __ldcs(reinterpret_cast<const uint4 *>(src + (hb + u) * D + cb));
            }
        }
#pragma unroll
        for (int u = 0; u < kHeadsInFlight; ++u) {
            if (hb + u >= h1) break;
            float a[VEC], b[VEC];
            unpack<T>(ra[u], a);
            unpack<T>(rb[u], b);
            if (alpha) {
                float ka[VEC], kb[VEC];
                load_affine<VEC>(alpha + (hb + u) * D, ca, cb, ka, kb);
#pragma unroll
                for (int j = 0; j < VEC; ++j) a[j] *= ka[j], b[j] *= kb[j];
                load_affine<VEC>(beta + (hb + u) * D, ca, cb, ka, kb);
#pragma unroll
                for (int j = 0; j < VEC; ++j) a[j] += ka[j], b[j] += kb[j];
            }
            if (rotated) turn<VEC>(a, b, c, s, interleaved);
            *reinterpret_cast<uint4 *>(dst + (hb + u) * D + ca) = pack<T>(a);
            *reinterpret_cast<uint4 *>(dst + (hb + u) * D + cb) = pack<T>(b);
        }
    }
}

template <typename T, int D>
__global__ void __launch_bounds__(kFwdThreads) rotate_kernel(const RotateParams p) {
    constexpr int VEC = Vec<T>::kN, IPR = D / (2 * VEC);
    const long long gid = (long long)blockIdx.x * kFwdThreads + threadIdx.x;
    const long long tok = gid / IPR;
    const int item = (int)(gid % IPR);
    if (tok >= p.n) return;
    const bool rotated = 2 * VEC * item < p.rot;
    int ca, cb;
    item_channels<VEC>(item, p.rot, p.interleaved, ca, cb);
    float c[VEC], s[VEC];
    if (rotated) {
        const int t = p.positions[tok];
#pragma unroll
        for (int j = 0; j < VEC; ++j) angle(t, __ldg(p.steps + VEC * item + j), p.amplitude, c[j], s[j]);
    }
    const int h0 = blockIdx.y * p.heads_per_block, h1 = min(p.H, h0 + p.heads_per_block);
    rotate_heads<T, D>(static_cast<const T *>(p.x) + tok * p.x_stride, static_cast<T *>(p.y) + tok * p.y_stride, h0, h1,
                       ca, cb, rotated, p.interleaved, p.alpha, p.beta, c, s);
}

// ---------------------------------------------------------------------------
// Append. Rows 0 .. n_new - 1 are the new tokens: their queries (base stream)
// are rotated to q_rot, their keys rotated into the page slot, their values
// copied there. Rows n_new .. n_new + n_out - 1 are the output stream's
// queries. The virtual heads of a token are its Hq query heads, Hkv key heads
// and Hkv value heads, cut over blockIdx.y.
// ---------------------------------------------------------------------------
template <typename T, int D>
__global__ void __launch_bounds__(kFwdThreads) rotate_append_kernel(const RotateAppendParams p) {
    constexpr int VEC = Vec<T>::kN, IPR = D / (2 * VEC);
    const long long gid = (long long)blockIdx.x * kFwdThreads + threadIdx.x;
    const long long row = gid / IPR;
    const int item = (int)(gid % IPR);
    if (row >= (long long)p.n_new + p.n_out) return;
    const bool out = row >= p.n_new;
    const int nq = (out ? p.q_out : p.q) ? p.Hq : 0;
    const int v0 = blockIdx.y * p.heads_per_block, v1 = v0 + p.heads_per_block;  // virtual heads
    const int nv = nq + (out ? 0 : 2 * p.Hkv);
    if (v0 >= nv) return;
    const bool rotated = 2 * VEC * item < p.rot;
    int ca, cb;
    item_channels<VEC>(item, p.rot, p.interleaved, ca, cb);
    const int t = out ? p.out_positions[row - p.n_new] : p.token_pos[row];
    float c[VEC], s[VEC];
    if (rotated && v0 < nq + p.Hkv) {
#pragma unroll
        for (int j = 0; j < VEC; ++j) angle(t, __ldg(p.steps + VEC * item + j), p.amplitude, c[j], s[j]);
    }
    if (v0 < nq) {
        const int h1 = min(nq, v1);
        if (out) {
            const long long r = row - p.n_new;
            rotate_heads<T, D>(static_cast<const T *>(p.q_out) + r * p.q_out_stride,
                               static_cast<T *>(p.q_out_rot) + r * p.Hq * D, v0, h1, ca, cb, rotated, p.interleaved,
                               p.alpha_out, p.beta_out, c, s);
        } else {
            rotate_heads<T, D>(static_cast<const T *>(p.q) + row * p.q_stride,
                               static_cast<T *>(p.q_rot) + row * p.Hq * D, v0, h1, ca, cb, rotated, p.interleaved,
                               p.alpha_base, p.beta_base, c, s);
        }
    }
    if (out || v1 <= nq) return;
    // the token's page slot
    const int b = p.token_seq[row];
    if (b < 0 || b >= p.B || t < 0 || t / p.page_size >= p.max_pages) {
        if (item == 0) set_status(p.status, ORTHROS_DEV_BAD_POSITION);
        return;
    }
    const int pg = p.block_table[(long long)b * p.max_pages + t / p.page_size];
    if (pg < 0 || pg >= p.num_pages) {
        if (item == 0) set_status(p.status, ORTHROS_DEV_BAD_PAGE);
        return;
    }
    const long long slot = ((long long)pg * p.page_size + t % p.page_size) * p.Hkv * D;
    const int k0 = max(v0 - nq, 0), k1 = min(v1 - nq, p.Hkv);
    if (k0 < k1)
        rotate_heads<T, D>(static_cast<const T *>(p.k) + row * p.k_stride, static_cast<T *>(p.k_cache) + slot, k0, k1,
                           ca, cb, rotated, p.interleaved, nullptr, nullptr, c, s);
    const T *vs = static_cast<const T *>(p.v) + row * p.v_stride;
    T *vd = static_cast<T *>(p.v_cache) + slot;
    for (int h = max(v0 - nq - p.Hkv, 0); h < min(v1 - nq - p.Hkv, p.Hkv); ++h) {
        const uint4 a = __ldcs(reinterpret_cast<const uint4 *>(vs + h * D + ca));
        const uint4 b2 = __ldcs(reinterpret_cast<const uint4 *>(vs + h * D + cb));
        *reinterpret_cast<uint4 *>(vd + h * D + ca) = a;
        *reinterpret_cast<uint4 *>(vd + h * D + cb) = b2;
    }
}

// ---------------------------------------------------------------------------
// Backward. A block covers a range of tokens and a group of heads; a thread
// owns one (head, item) and walks the block's tokens with the affine's gradient
// in registers, so d_alpha and d_beta cost no traffic per token. The angles of
// kTabTokens tokens at a time are computed once by the block and shared by its
// heads. The block's sums go to the workspace as one partial each, and
// rotate_grad_sum_kernel adds the partials in a fixed order (no atomics: the
// same call gives the same bits). Bound by HBM: dy and x read once, dx written.
// ---------------------------------------------------------------------------
constexpr int kBwdThreads = 256;
constexpr int kTabTokens = 32;

template <typename T, int D, bool kGrads>
__global__ void __launch_bounds__(kBwdThreads, 2) rotate_backward_kernel(const RotateBwdParams p) {
    constexpr int VEC = Vec<T>::kN, IPR = D / (2 * VEC);
    // table entry (token, quarter q, item): two (cos, sin) pairs, so that the
    // lanes of a row read consecutive 16-byte words
    constexpr int kQ = VEC / 2;
    __shared__ float4 tab[kTabTokens][kQ][IPR];
    __shared__ float red[kBwdThreads * 2];
    const int tid = threadIdx.x;
    const int hb = p.heads_per_block;            // heads of this block
    const int lanes = kBwdThreads / (hb * IPR);  // tokens handled side by side
    const int tl = tid / (hb * IPR);
    const int h = blockIdx.y * hb + (tid / IPR) % hb;
    const int item = tid % IPR;
    const bool active = tl < lanes && h < p.H;
    const bool rotated = 2 * VEC * item < p.rot;
    int ca, cb;
    item_channels<VEC>(item, p.rot, p.interleaved, ca, cb);
    const long long n0 = p.n * blockIdx.x / gridDim.x, n1 = p.n * (blockIdx.x + 1) / gridDim.x;
    float al[2][VEC], da[2][VEC], db[2][VEC];
#pragma unroll
    for (int j = 0; j < VEC; ++j) {
        al[0][j] = al[1][j] = 1.f;
        da[0][j] = da[1][j] = db[0][j] = db[1][j] = 0.f;
    }
    if (active && p.alpha) load_affine<VEC>(p.alpha + h * D, ca, cb, al[0], al[1]);
    const int half = p.rot >> 1;
    for (long long base = n0; base < n1; base += kTabTokens) {
        const int cnt = (int)min((long long)kTabTokens, n1 - base);
        __syncthreads();
        for (int e = tid; e < cnt * half; e += kBwdThreads) {
            const int k = e / half, pr = e % half;  // token of the table, pair
            float c, s;
            angle(p.positions[base + k], __ldg(p.steps + pr), p.amplitude, c, s);
            float2 *dst = reinterpret_cast<float2 *>(&tab[k][(pr % VEC) / 2][pr / VEC]);
            dst[pr & 1] = make_float2(c, -s);  // the opposite angle
        }
        __syncthreads();
        if (!active) continue;
#pragma unroll 2
        for (int k = tl; k < cnt; k += lanes) {
            const long long tok = base + k;
            const T *dy = static_cast<const T *>(p.dy) + tok * p.dy_stride + h * D;
            uint4 ra = __ldcs(reinterpret_cast<const uint4 *>(dy + ca));
            uint4 rb = __ldcs(reinterpret_cast<const uint4 *>(dy + cb));
            uint4 xa, xb;
            if constexpr (kGrads) {
                const T *x = static_cast<const T *>(p.x) + tok * p.x_stride + h * D;
                xa = __ldcs(reinterpret_cast<const uint4 *>(x + ca));
                xb = __ldcs(reinterpret_cast<const uint4 *>(x + cb));
            }
            float a[VEC], b[VEC];
            unpack<T>(ra, a);
            unpack<T>(rb, b);
            if (rotated) {
                float c[VEC], s[VEC];
#pragma unroll
                for (int q = 0; q < kQ; ++q) {
                    const float4 v = tab[k][q][item];
                    c[2 * q] = v.x, s[2 * q] = v.y, c[2 * q + 1] = v.z, s[2 * q + 1] = v.w;
                }
                turn<VEC>(a, b, c, s, p.interleaved);
            }
            if constexpr (kGrads) {
                float x0[VEC], x1[VEC];
                unpack<T>(xa, x0);
                unpack<T>(xb, x1);
#pragma unroll
                for (int j = 0; j < VEC; ++j) {
                    da[0][j] = fmaf(a[j], x0[j], da[0][j]);
                    da[1][j] = fmaf(b[j], x1[j], da[1][j]);
                    db[0][j] += a[j];
                    db[1][j] += b[j];
                }
            }
#pragma unroll
            for (int j = 0; j < VEC; ++j) a[j] *= al[0][j], b[j] *= al[1][j];
            T *dx = static_cast<T *>(p.dx) + tok * p.dx_stride + h * D;
            *reinterpret_cast<uint4 *>(dx + ca) = pack<T>(a);
            *reinterpret_cast<uint4 *>(dx + cb) = pack<T>(b);
        }
    }
    if constexpr (kGrads) {
        // sum over the token lanes of the block, one channel of every thread at a time
        float *part = p.partial + (long long)blockIdx.x * 2 * p.H * D;
#pragma unroll
        for (int v = 0; v < 2; ++v) {
#pragma unroll
            for (int j = 0; j < VEC; ++j) {
                __syncthreads();
                red[tid] = da[v][j];
                red[kBwdThreads + tid] = db[v][j];
                __syncthreads();
                if (tl == 0 && active) {
                    float sa = 0.f, sb = 0.f;
                    for (int l = 0; l < lanes; ++l) {
                        sa += red[l * hb * IPR + tid];
                        sb += red[kBwdThreads + l * hb * IPR + tid];
                    }
                    const int ch = h * D + (v ? cb : ca) + j;
                    part[ch] = sa;
                    part[p.H * D + ch] = sb;
                }
            }
        }
    }
}

// d_alpha and d_beta: column sums over the n_part partials [n_part, 2, H d].
// A block takes 32 columns; its 8 warps stride over the partials.
__global__ void __launch_bounds__(256) rotate_grad_sum_kernel(const float *__restrict__ partial, int n_part, int cols,
                                                              float *__restrict__ d_alpha, float *__restrict__ d_beta) {
    __shared__ float red[8][32];
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    const int col = blockIdx.x * 32 + lane;  // cols (= H d) is a multiple of 32: no block straddles the two
    float s0 = 0.f, s1 = 0.f, s2 = 0.f, s3 = 0.f;
    int i = w;
    for (; i + 24 < n_part; i += 32) {
        s0 += partial[(long long)i * 2 * cols + col];
        s1 += partial[(long long)(i + 8) * 2 * cols + col];
        s2 += partial[(long long)(i + 16) * 2 * cols + col];
        s3 += partial[(long long)(i + 24) * 2 * cols + col];
    }
    for (; i < n_part; i += 8) s0 += partial[(long long)i * 2 * cols + col];
    red[w][lane] = (s0 + s1) + (s2 + s3);
    __syncthreads();
    if (w == 0) {
        float s = 0.f;
#pragma unroll
        for (int k = 0; k < 8; ++k) s += red[k][lane];
        if (col < cols) d_alpha[col] = s;
        else d_beta[col - cols] = s;
    }
}

// Heads a thread walks: as many as leave at least four blocks per SM, so that
// its angles are shared by many heads on long inputs while a decoding step
// still spreads over the GPU.
int heads_per_block(long long token_blocks, int heads) {
    const long long want = 4LL * device_sm_count();
    int hp = heads;
    while (hp > 1 && token_blocks * ((heads + hp - 1) / hp) < want) hp = (hp + 1) / 2;
    return hp;
}

template <typename T, int D> cudaError_t rotate_t(RotateParams p, cudaStream_t s) {
    constexpr int IPR = D / (2 * Vec<T>::kN);
    const long long tb = (p.n * IPR + kFwdThreads - 1) / kFwdThreads;
    p.heads_per_block = heads_per_block(tb, p.H);
    const dim3 grid((unsigned)tb, (p.H + p.heads_per_block - 1) / p.heads_per_block);
    rotate_kernel<T, D><<<grid, kFwdThreads, 0, s>>>(p);
    return cudaGetLastError();
}

template <typename T, int D> cudaError_t append_t(RotateAppendParams p, cudaStream_t s) {
    constexpr int IPR = D / (2 * Vec<T>::kN);
    const long long tb = (((long long)p.n_new + p.n_out) * IPR + kFwdThreads - 1) / kFwdThreads;
    const int heads = (p.q || p.q_out ? p.Hq : 0) + 2 * p.Hkv;
    p.heads_per_block = heads_per_block(tb, heads);
    const dim3 grid((unsigned)tb, (heads + p.heads_per_block - 1) / p.heads_per_block);
    rotate_append_kernel<T, D><<<grid, kFwdThreads, 0, s>>>(p);
    return cudaGetLastError();
}

template <typename T, int D> cudaError_t backward_t(RotateBwdParams p, cudaStream_t s) {
    constexpr int IPR = D / (2 * Vec<T>::kN);
    p.heads_per_block = p.H < kBwdThreads / IPR ? p.H : kBwdThreads / IPR;
    const dim3 grid(p.n_part, (p.H + p.heads_per_block - 1) / p.heads_per_block);
    if (p.d_alpha) rotate_backward_kernel<T, D, true><<<grid, kBwdThreads, 0, s>>>(p);
    else rotate_backward_kernel<T, D, false><<<grid, kBwdThreads, 0, s>>>(p);
    return cudaGetLastError();
}

}  // namespace

// Partials of the affine's gradient (blocks along the tokens): two blocks per
// SM over all head groups, but no fewer than 16 tokens a block.
int rotate_grad_parts(long long n, int H, int d, int elem_bytes) {
    const int per = kBwdThreads / (d * elem_bytes / 32);  // heads of a block
    const int groups = (H + per - 1) / per;
    long long parts = 2LL * device_sm_count() / groups;
    if (parts > (n + 15) / 16) parts = (n + 15) / 16;
    return parts < 1 ? 1 : (int)parts;
}

#define ORTHROS_BY_TYPE(FN, P)                                                                          \
    (dtype == ORTHROS_F32 ? (d == 128 ? FN<float, 128>(P, stream) : FN<float, 64>(P, stream))           \
                          : (d == 128 ? FN<__nv_bfloat16, 128>(P, stream) : FN<__nv_bfloat16, 64>(P, stream)))

cudaError_t launch_rotate(const RotateParams &p, int d, orthros_dtype dtype, cudaStream_t stream) {
    return ORTHROS_BY_TYPE(rotate_t, p);
}
cudaError_t launch_rotate_append(const RotateAppendParams &p, int d, orthros_dtype dtype, cudaStream_t stream) {
    return ORTHROS_BY_TYPE(append_t, p);
}
cudaError_t launch_rotate_backward(const RotateBwdParams &p, int d, orthros_dtype dtype, cudaStream_t stream) {
    return ORTHROS_BY_TYPE(backward_t, p);
}
cudaError_t launch_rotate_grad_sum(const RotateBwdParams &p, int d, cudaStream_t stream) {
    const int cols = p.H * d;
    rotate_grad_sum_kernel<<<2 * cols / 32, 256, 0, stream>>>(p.partial, p.n_part, cols, p.d_alpha, p.d_beta);
    return cudaGetLastError();
}
#undef ORTHROS_BY_TYPE

}  // namespace orthros
