// norm_rotary.cu -- rotary positions behind a norm of each head (models that norm
// queries and keys): the rotation of rotary.cu, its gradient and the append, with
//   u = a (.) xh + beta,  xh = r x,  r = (mean_c x_c^2 + eps)^(-1/2),  a = alpha (.) w,
// where the weight w [d] is shared by the heads. The gradient: with g = m R(-t) dy,
//   dx = r (a (.) g - xh mean_c(a g xh)),  S = sum_t g (.) xh (per head),
//   d_alpha = w (.) S,  d_w = sum_h alpha (.) S,  d_beta = sum_t g.
//
// Norm and rotation share one pass over the rows: a row lies on neighbouring lanes
// of a warp, two vectors each, so that its sums are a few exchanges between them.
// What bounds the kernels is HBM as long as the arithmetic keeps up; the norm adds a
// half to the rotation's, so everything runs on pairs of channels (packed fp32
// instructions), and the layout of the pairs is fixed at compile time: with one kernel for
// both layouts the batch's loads and the affine did not fit the registers beside it
// (32768 x 32 x 128 bf16: 98 to 130 us instead of 89).
#include "ptx.cuh"
#include "rotary.cuh"

namespace orthros {

using namespace rope;

namespace {

// Two floats of one packed instruction.
using F2 = uint64_t;
__device__ __forceinline__ F2 f2(float a, float b) { return ptx::f32x2(a, b); }
__device__ __forceinline__ void split(F2 x, float &a, float &b) { asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(x)); }
__device__ __forceinline__ F2 mul(F2 a, F2 b) {
    F2 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ F2 add(F2 a, F2 b) {
    F2 r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ F2 sub(F2 a, F2 b) {
    F2 r;
    asm("sub.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ F2 fma(F2 a, F2 b, F2 c) {
    F2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ float sum(F2 x) {
    float a, b;
    split(x, a, b);
    return a + b;
}

// A work item's 2 VEC channels as VEC / 2 steps of two channel pairs: the pairs' first
// channels X = (x_0, x_1) and second ones Y. Half layout: X are channels 2q, 2q + 1 of vector
// a, Y of vector b. Interleaved: step q takes four consecutive channels of vector a (the first
// half of the steps) or b, X the even ones.
template <typename T, bool kInter> struct Steps {
    static constexpr int VEC = Vec<T>::kN, kN = VEC / 2;
    // vector (0: a, 1: b) and channel of X's element e (second = 0) or Y's (1) of step q
    static __device__ __forceinline__ constexpr int vec(int q, int second) { return kInter ? q / (VEC / 4) : second; }
    static __device__ __forceinline__ constexpr int ch(int q, int second, int e) {
        return kInter ? 4 * (q % (VEC / 4)) + 2 * e + second : 2 * q + e;
    }
    static __device__ __forceinline__ uint32_t word(const uint4 &v, int i) { return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w; }
    static __device__ __forceinline__ float value(const uint4 &v, int c) {
        if constexpr (sizeof(T) == 4) return __uint_as_float(word(v, c));
        const uint32_t w = word(v, c / 2);
        return __uint_as_float(c & 1 ? w & 0xffff0000u : w << 16);
    }
    static __device__ __forceinline__ F2 get(const uint4 &a, const uint4 &b, int q, int second) {
        const uint4 &v = vec(q, second) ? b : a;
        return f2(value(v, ch(q, second, 0)), value(v, ch(q, second, 1)));
    }
    // the rounded vectors of all steps' X and Y
    static __device__ __forceinline__ void put(const F2 (&x)[kN], const F2 (&y)[kN], uint4 &a, uint4 &b) {
        float f[2][VEC];
#pragma unroll
        for (int q = 0; q < kN; ++q) {
            split(x[q], f[vec(q, 0)][ch(q, 0, 0)], f[vec(q, 0)][ch(q, 0, 1)]);
            split(y[q], f[vec(q, 1)][ch(q, 1, 0)], f[vec(q, 1)][ch(q, 1, 1)]);
        }
        uint32_t w[2][4];
#pragma unroll
        for (int v = 0; v < 2; ++v) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if constexpr (sizeof(T) == 4) w[v][i] = __float_as_uint(f[v][i]);
                else w[v][i] = ptx::pack_bf16(f[v][2 * i], f[v][2 * i + 1]);
            }
        }
        a = make_uint4(w[0][0], w[0][1], w[0][2], w[0][3]);
        b = make_uint4(w[1][0], w[1][1], w[1][2], w[1][3]);
    }
    // the item's channels of a [d] vector in steps
    static __device__ __forceinline__ void load(const float *p, int ca, int cb, F2 (&x)[kN], F2 (&y)[kN]) {
        float f[2][VEC];
        load_affine<VEC>(p, ca, cb, f[0], f[1]);
#pragma unroll
        for (int q = 0; q < kN; ++q) {
            x[q] = f2(f[vec(q, 0)][ch(q, 0, 0)], f[vec(q, 0)][ch(q, 0, 1)]);
            y[q] = f2(f[vec(q, 1)][ch(q, 1, 0)], f[vec(q, 1)][ch(q, 1, 1)]);
        }
    }
    // item, step and element of pair pr
    static __device__ __forceinline__ void find(int pr, int quarter, int &item, int &q, int &e) {
        if constexpr (kInter) {
            const int v = pr >= quarter, left = pr - v * quarter;  // quarter = D / 4: pairs of the vectors a
            item = left / (VEC / 2), q = v * (VEC / 4) + left % (VEC / 2) / 2, e = left % 2;
        } else {
            item = pr / VEC, q = pr % VEC / 2, e = pr % 2;
        }
    }
};

// Cosines and sines of a few tokens, computed once by the block: entry (token, step, item) has
// the cosines of the step's two pairs, then their sines. Pairs past `rot` stay: 1 and 0.
template <typename T, int D, bool kInter> struct Angles {
    static constexpr int IPR = D / (2 * Vec<T>::kN), kN = Steps<T, kInter>::kN;
    float4 e[kTabTokens][kN][IPR];
    // angles of cnt positions; sign -1 for the transposed rotation
    __device__ __forceinline__ void fill(const int *pos, int cnt, const uint64_t *steps, int rot, float amp, float sign) {
        for (int x = threadIdx.x; x < cnt * (D / 2); x += blockDim.x) {
            const int k = x / (D / 2), pr = x % (D / 2);
            float c = 1.f, s = 0.f;
            if (pr < rot >> 1) angle(pos[k], __ldg(steps + pr), amp, c, s);
            int i, q, el;
            Steps<T, kInter>::find(pr, D / 4, i, q, el);
            float *to = reinterpret_cast<float *>(&e[k][q][i]) + el;
            to[0] = c;
            to[2] = sign * s;
        }
    }
    __device__ __forceinline__ void read(int k, int q, int item, F2 &c, F2 &s) const {
        const float4 v = e[k][q][item];
        c = f2(v.x, v.y), s = f2(v.z, v.w);
    }
};

// Sum over the kLanes neighbouring lanes that hold a row (they run together).
template <int kLanes> __device__ __forceinline__ float row_sum(float x) {
    const uint32_t mask = ((1u << kLanes) - 1) << (threadIdx.x & 31 & ~(kLanes - 1));
#pragma unroll
    for (int o = 1; o < kLanes; o <<= 1) x += __shfl_xor_sync(mask, x, o);
    return x;
}

// ---------------------------------------------------------------------------
// Forward and append: rotary.cu's moving kernel (its threads, tables, runs of tokens and
// virtual heads) with the norm on the way. One kernel is both, a forward an append without
// keys, output rows and status word: compiled for it alone, the compiler works on a
// batch's tokens side by side and spills (160 bytes a thread). Bound by HBM: 32768 x 32 x 128
// bf16 with weight and affine 89 us, 6.1 TB/s (91 % of the measured copy rate; the rotation alone
// 86); 8000 tokens of GQA 32/8 appended in 35 us (5.3 TB/s: start and end of a 28 us kernel).
// ---------------------------------------------------------------------------
constexpr int kTokens = 4;  // of a thread's batch of loads

template <typename T, int D, bool kInter>
__global__ void __launch_bounds__(kMoveThreads) norm_move_kernel(const RotateParams p) {
    using S = Steps<T, kInter>;
    constexpr int VEC = S::VEC, IPR = D / (2 * VEC), N = S::kN;
    __shared__ Angles<T, D, kInter> tab[2];
    __shared__ int pos[kRunTokens];
    __shared__ long long slot[kRunTokens];  // append: first element of the token's page slot, or -1
    const bool append = p.status != nullptr;
    if (append && blockIdx.x == gridDim.x - 1) {
        if (blockIdx.y == 0) write_status(p);
        return;
    }
    const int tid = threadIdx.x;
    const int hb = p.heads_per_block;
    const int lanes = blockDim.x / (hb * IPR);  // tokens handled side by side
    const int tl = tid / (hb * IPR);
    const int h = blockIdx.y * hb + (tid / IPR) % hb;
    const int item = tid % IPR;
    const bool out = (int)blockIdx.x >= p.blocks;
    const int bx = out ? blockIdx.x - p.blocks : blockIdx.x, nbx = out ? gridDim.x - 1 - p.blocks : p.blocks;
    const long long n = out ? p.n_out : p.n;
    const int32_t *positions = out ? p.out_positions : p.positions;
    // what this thread's virtual head moves
    const T *src = static_cast<const T *>(out ? p.x_out : p.x);
    T *dst = static_cast<T *>(out ? p.y_out : p.y);
    long long ss = out ? p.x_out_stride : p.x_stride, ds = p.y_stride;
    const float *alpha = out ? p.alpha_out : p.alpha, *beta = out ? p.beta_out : p.beta, *weight = p.weight;
    int hh = h;  // head within its tensor
    bool paged = false, copies = false;
    if (append && h >= p.H) {
        hh = h - p.H;
        paged = true;
        copies = hh >= p.Hkv;  // a value head
        if (copies) hh -= p.Hkv;
        src = static_cast<const T *>(copies ? p.v : p.k);
        dst = static_cast<T *>(copies ? p.v_cache : p.k_cache);
        ss = copies ? p.v_stride : p.k_stride;
        alpha = beta = nullptr;
        weight = p.k_weight;
    }
    const bool active = tl < lanes && (paged ? !out && h < p.H + 2 * p.Hkv : h < p.H && src != nullptr);
    const Item<VEC, D> it(item, p.rot, kInter);
    src += hh * D;
    dst += hh * D;
    F2 ax[N], ay[N], bx_[N], by[N];
#pragma unroll
    for (int q = 0; q < N; ++q) ax[q] = ay[q] = f2(1.f, 1.f), bx_[q] = by[q] = f2(0.f, 0.f);
    if (active && alpha) {
        S::load(alpha + hh * D, it.ca, it.cb, ax, ay);
        S::load(beta + hh * D, it.ca, it.cb, bx_, by);
    }
    if (active && weight && !copies) {  // the norm's weight goes into alpha
        F2 wx[N], wy[N];
        S::load(weight, it.ca, it.cb, wx, wy);
#pragma unroll
        for (int q = 0; q < N; ++q) ax[q] = mul(ax[q], wx[q]), ay[q] = mul(ay[q], wy[q]);
    }
    const long long n0 = n * bx / nbx, n1 = n * (bx + 1) / nbx;
    const int step = table_tokens(lanes);
    int buf = 0;
    for (long long base = n0; base < n1; base += step, buf ^= 1) {
        const int cnt = (int)min((long long)step, n1 - base);
        const int run = (int)((base - n0) % kRunTokens);  // first entry of these tokens in pos and slot
        // the first batch's loads are under way while the angles are computed
        uint4 ra[kTokens], rb[kTokens];
        auto load = [&](int k0) {
#pragma unroll
            for (int u = 0; u < kTokens; ++u) {
                const int k = k0 + u * lanes;
                ra[u] = rb[u] = make_uint4(0, 0, 0, 0);  // (past the tokens: summed, not used)
                if (k < cnt) {
                    ra[u] = __ldcs(reinterpret_cast<const uint4 *>(src + (base + k) * ss + it.ca));
                    rb[u] = __ldcs(reinterpret_cast<const uint4 *>(src + (base + k) * ss + it.cb));
                }
            }
        };
        if (active) load(tl);
        if (run == 0) {
            __syncthreads();  // the last run's entries have been used
            for (int k = tid; k < kRunTokens && base + k < n1; k += blockDim.x) {
                pos[k] = positions[base + k];
                if (append && !out) {
                    const long long at = page_slot(p, base + k);
                    slot[k] = at < 0 ? -1 : at * p.Hkv * D;
                }
            }
            __syncthreads();
        }
        tab[buf].fill(pos + run, cnt, p.steps, p.rot, p.amplitude, 1.f);
        __syncthreads();
        if (!active) continue;
        for (int k0 = tl; k0 < cnt; k0 += kTokens * lanes) {
            if (k0 != tl) load(k0);
            float r[kTokens];  // 1 / rms of the batch's rows, their exchanges side by side
            if (!copies) {
#pragma unroll
                for (int u = 0; u < kTokens; ++u) {
                    F2 sx = f2(0.f, 0.f), sy = sx;
#pragma unroll
                    for (int q = 0; q < N; ++q) {
                        const F2 x = S::get(ra[u], rb[u], q, 0), y = S::get(ra[u], rb[u], q, 1);
                        sx = fma(x, x, sx), sy = fma(y, y, sy);
                    }
                    r[u] = sum(add(sx, sy));
                }
#pragma unroll
                for (int u = 0; u < kTokens; ++u) r[u] = rsqrtf(fmaf(row_sum<IPR>(r[u]), 1.f / D, p.eps));
            }
#pragma unroll
            for (int u = 0; u < kTokens; ++u) {
                const int k = k0 + u * lanes;
                if (k >= cnt) break;
                T *to = paged ? dst + slot[run + k] : dst + (base + k) * ds;
                if (paged && slot[run + k] < 0) continue;
                if (!copies) {
                    const F2 rr = f2(r[u], r[u]);
                    F2 ox[N], oy[N];
#pragma unroll
                    for (int q = 0; q < N; ++q) {
                        const F2 x = fma(mul(S::get(ra[u], rb[u], q, 0), rr), ax[q], bx_[q]);
                        const F2 y = fma(mul(S::get(ra[u], rb[u], q, 1), rr), ay[q], by[q]);
                        F2 c, s;
                        tab[buf].read(k, q, item, c, s);
                        ox[q] = sub(mul(x, c), mul(y, s));
                        oy[q] = fma(x, s, mul(y, c));
                    }
                    S::put(ox, oy, ra[u], rb[u]);
                }
                *reinterpret_cast<uint4 *>(to + it.ca) = ra[u];
                *reinterpret_cast<uint4 *>(to + it.cb) = rb[u];
            }
        }
    }
}

// ---------------------------------------------------------------------------
// Backward: rotary.cu's gradient kernel (rows through shared memory, kDepth tokens ahead of
// the thread that takes them, partials of a block added in a fixed order) with both sums of
// a row, of x^2 and of a g x, taken in one exchange. The weight's gradient is the block's sums per
// head, weighed by alpha, added over its heads. Bound by HBM: 32768 x 32 x 128 bf16 with all
// gradients 134 us, 6.0 TB/s (90 %), and 6 us of sum (with alpha read in the loop over the heads
// that summed the weight's gradient the kernel took 8 us longer).
// ---------------------------------------------------------------------------
constexpr int kDepth = 6;

template <typename T, int D, bool kGrads, bool kInter>
__global__ void __launch_bounds__(kBwdThreads, kBwdBlocks) norm_backward_kernel(const RotateBwdParams p) {
    using S = Steps<T, kInter>;
    constexpr int VEC = S::VEC, IPR = D / (2 * VEC), N = S::kN;
    extern __shared__ uint4 fifo[];  // [kDepth][dy a, dy b, x a, x b][thread]
    __shared__ Angles<T, D, kInter> tab[2];
    __shared__ int pos[kRunTokens];
    const int tid = threadIdx.x;
    const int hb = p.heads_per_block;            // heads of this block
    const int lanes = kBwdThreads / (hb * IPR);  // tokens handled side by side
    const int tl = tid / (hb * IPR);
    const int h = blockIdx.y * hb + (tid / IPR) % hb;
    const int item = tid % IPR;
    const bool active = tl < lanes && h < p.H;
    const Item<VEC, D> it(item, p.rot, kInter);
    const int ca = it.ca, cb = it.cb;
    const long long n0 = p.n * blockIdx.x / gridDim.x, n1 = p.n * (blockIdx.x + 1) / gridDim.x;
    constexpr int step = kTabTokens;
    const int n = (int)(n1 - n0);
    // this thread's tokens, kDepth of them ahead
    int ahead = 0, ahead_k = tl, wr = 0;
    auto fetch = [&]() {
        if (active && ahead_k < step && ahead + ahead_k < n) {
            uint4 *to = fifo + wr * 4 * kBwdThreads + tid;
            const long long i = n0 + ahead + ahead_k;
            const T *dy = static_cast<const T *>(p.dy) + i * p.dy_stride + h * D;
            const T *x = static_cast<const T *>(p.x) + i * p.x_stride + h * D;
            copy16(to, dy + ca);
            copy16(to + kBwdThreads, dy + cb);
            copy16(to + 2 * kBwdThreads, x + ca);
            copy16(to + 3 * kBwdThreads, x + cb);
            ahead_k += lanes;
            if (ahead_k >= step) ahead += step, ahead_k = tl;
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
        wr = wr + 1 == kDepth ? 0 : wr + 1;
    };
    for (int i = 0; i < kDepth; ++i) fetch();
    F2 ax[N], ay[N], dax[N], day[N], dbx[N], dby[N];
#pragma unroll
    for (int q = 0; q < N; ++q) {
        ax[q] = ay[q] = f2(1.f, 1.f);
        dax[q] = day[q] = dbx[q] = dby[q] = f2(0.f, 0.f);
    }
    if (active && p.alpha) S::load(p.alpha + h * D, ca, cb, ax, ay);
    if (active && p.weight) {
        F2 wx[N], wy[N];
        S::load(p.weight, ca, cb, wx, wy);
#pragma unroll
        for (int q = 0; q < N; ++q) ax[q] = mul(ax[q], wx[q]), ay[q] = mul(ay[q], wy[q]);
    }
    int buf = 0, rd = 0;
    for (int base = 0; base < n; base += step, buf ^= 1) {
        const int cnt = min(step, n - base);
        const int run = base % kRunTokens;  // first entry of these tokens in pos
        if (run == 0) {
            __syncthreads();
            for (int k = tid; k < kRunTokens && base + k < n; k += kBwdThreads) pos[k] = p.positions[n0 + base + k];
            __syncthreads();
        }
        tab[buf].fill(pos + run, cnt, p.steps, p.rot, p.amplitude, -1.f);  // the opposite angle
        __syncthreads();
        if (!active) continue;
        for (int k = tl; k < cnt; k += lanes) {
            asm volatile("cp.async.wait_group %0;" ::"n"(kDepth - 1) : "memory");
            const uint4 *from = fifo + rd * 4 * kBwdThreads + tid;
            rd = rd + 1 == kDepth ? 0 : rd + 1;
            const uint4 ga = from[0], gb = from[kBwdThreads], xa = from[2 * kBwdThreads], xb = from[3 * kBwdThreads];
            F2 gx[N], gy[N], s0 = f2(0.f, 0.f), s1 = s0;
#pragma unroll
            for (int q = 0; q < N; ++q) {
                const F2 u = S::get(ga, gb, q, 0), v = S::get(ga, gb, q, 1);
                F2 c, s;
                tab[buf].read(k, q, item, c, s);
                gx[q] = sub(mul(u, c), mul(v, s));
                gy[q] = fma(u, s, mul(v, c));
                const F2 x = S::get(xa, xb, q, 0), y = S::get(xa, xb, q, 1);
                s0 = fma(x, x, fma(y, y, s0));
                s1 = fma(mul(gx[q], ax[q]), x, fma(mul(gy[q], ay[q]), y, s1));
            }
            const float r = rsqrtf(fmaf(row_sum<IPR>(sum(s0)), 1.f / D, p.eps));
            // (a row whose squares overflow has r = 0 and xh = 0, while its sum of a g x may be inf or NaN)
            const float dot = row_sum<IPR>(sum(s1)), mean = r > 0.f ? dot * r * (1.f / D) : 0.f;
            const F2 rr = f2(r, r), mm = f2(-mean * r, -mean * r);
            F2 ox[N], oy[N];
#pragma unroll
            for (int q = 0; q < N; ++q) {
                const F2 x = mul(S::get(xa, xb, q, 0), rr), y = mul(S::get(xa, xb, q, 1), rr);
                if constexpr (kGrads) {
                    dax[q] = fma(gx[q], x, dax[q]), day[q] = fma(gy[q], y, day[q]);
                    dbx[q] = add(gx[q], dbx[q]), dby[q] = add(gy[q], dby[q]);
                }
                ox[q] = fma(x, mm, mul(mul(gx[q], ax[q]), rr));
                oy[q] = fma(y, mm, mul(mul(gy[q], ay[q]), rr));
            }
            uint4 oa, ob;
            S::put(ox, oy, oa, ob);
            T *dx = static_cast<T *>(p.dx) + (n0 + base + k) * p.dx_stride + h * D;
            *reinterpret_cast<uint4 *>(dx + ca) = oa;
            *reinterpret_cast<uint4 *>(dx + cb) = ob;
            fetch();  // into the slot this thread has just read
        }
    }
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    if constexpr (kGrads) {
        // sums over the token lanes of the block, through the shared memory that the loads have left:
        // [channel of a thread][thread], vector a's channels first
        float *red = reinterpret_cast<float *>(fifo);
        __syncthreads();
#pragma unroll
        for (int q = 0; q < N; ++q) {
            const F2 all[4] = {dax[q], day[q], dbx[q], dby[q]};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                float f[2];
                split(all[i], f[0], f[1]);
#pragma unroll
                for (int e = 0; e < 2; ++e)
                    red[((i / 2 * 2 + S::vec(q, i & 1)) * VEC + S::ch(q, i & 1, e)) * kBwdThreads + tid] = f[e];
            }
        }
        __syncthreads();
        const int row = hb * IPR;  // threads of a token lane
        float *by_head = red + 4 * VEC * kBwdThreads;  // [head of the block][channel]: alpha (.) the block's S
        if (active) {
            float *part = p.partial + (long long)blockIdx.x * 2 * p.H * D;
            const int last = p.d_alpha ? 4 * VEC : 2 * VEC;
            for (int v = tl; v < last; v += lanes) {  // this thread's channels, shared with its fellows of other lanes
                const float *from = red + v * kBwdThreads + tid - tl * row;
                const int j = v % VEC, at = (v / VEC & 1 ? cb : ca) + j;
                const float al = p.alpha && p.partial_w && v < 2 * VEC ? __ldg(p.alpha + h * D + at) : 1.f;
                float total = 0.f;
                for (int l = 0; l < lanes; ++l) total += from[l * row];
                if (p.d_alpha) part[(v < 2 * VEC ? 0 : p.H * D) + h * D + at] = total;
                if (p.partial_w && v < 2 * VEC) by_head[(h - (int)blockIdx.y * hb) * D + at] = al * total;
            }
        }
        if (!p.partial_w) return;
        // the weight's gradient: the heads of the block, a quarter (d = 128) or an eighth of them a thread
        constexpr int kParts = kBwdThreads / D;
        __syncthreads();
        const int heads = min(hb, p.H - (int)blockIdx.y * hb), c = tid % D;
        float total = 0.f;
        for (int hh = tid / D; hh < heads; hh += kParts) total += by_head[hh * D + c];
        red[tid] = total;
        __syncthreads();
        if (tid >= D) return;
#pragma unroll
        for (int i = 1; i < kParts; ++i) total += red[i * D + tid];
        p.partial_w[((long long)blockIdx.y * gridDim.x + blockIdx.x) * D + tid] = total;
    }
}

// The gradients from the blocks' sums: d_alpha = w (.) S and d_beta from the n_part partials
// [n_part, 2, H d], and d_w from the n_w block sums [n_w, d] of alpha (.) S. Blocks of 32 columns:
// 2 H d / 32 for the affine's (none when they are not wanted), then d / 32 for the weight's.
constexpr int kSumWarps = 32;  // of a block: a partial a lane and a few loads each, all in flight at once

__global__ void __launch_bounds__(kSumWarps * 32) norm_grad_sum_kernel(const RotateBwdParams p, int cols, int d, int n_w) {
    __shared__ float red[kSumWarps][33];
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    const int affine = p.d_alpha ? 2 * cols / 32 : 0;
    const bool weight = (int)blockIdx.x >= affine;
    const int col0 = (weight ? blockIdx.x - affine : blockIdx.x) * 32;
    const float *from = (weight ? p.partial_w : p.partial) + col0 + lane;
    const int n = weight ? n_w : p.n_part;
    const long long step = weight ? d : 2 * cols;
    asm volatile("griddepcontrol.wait;" ::: "memory");  // (a dependent launch: the partials are there now)
    constexpr int kLoads = 8;
    float s = 0.f;
    for (int i0 = w; i0 < n; i0 += kLoads * kSumWarps) {
        float x[kLoads];
#pragma unroll
        for (int u = 0; u < kLoads; ++u) x[u] = i0 + u * kSumWarps < n ? from[(i0 + u * kSumWarps) * step] : 0.f;
#pragma unroll
        for (int u = 0; u < kLoads; ++u) s += x[u];
    }
    red[w][lane] = s;
    __syncthreads();
    // warp w adds up column w
    s = red[lane][w];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    if (lane == 0) {
        const int col = col0 + w;
        if (weight) p.d_weight[col] = s;
        else if (col < cols) p.d_alpha[col] = p.weight ? s * p.weight[col % d] : s;
        else p.d_beta[col - cols] = s;
    }
}

template <typename T, int D, bool kInter> cudaError_t move_k(RotateParams p, cudaStream_t s) {
    static std::atomic<int> resident{0};
    int per_sm = 0;
    const auto kernel = norm_move_kernel<T, D, kInter>;
    const bool append = p.status != nullptr;
    if (cudaError_t e = resident_threads((const void *)kernel, resident, per_sm); e != cudaSuccess) return e;
    const MoveGrid m = move_grid(p.H + (append ? 2 * p.Hkv : 0), D / (2 * Vec<T>::kN), per_sm, p.n, p.n_out, append);
    p.heads_per_block = m.heads_per_block;
    p.blocks = m.blocks;
    const dim3 grid((unsigned)(m.blocks + m.out_blocks + (append ? 1 : 0)), m.groups);
    kernel<<<grid, m.threads, 0, s>>>(p);
    return cudaGetLastError();
}
template <typename T, int D> cudaError_t move_t(const RotateParams &p, cudaStream_t s) {
    return p.interleaved ? move_k<T, D, true>(p, s) : move_k<T, D, false>(p, s);
}

template <typename T, int D, bool kGrads, bool kInter> cudaError_t backward_k(RotateBwdParams p, cudaStream_t s) {
    constexpr int IPR = D / (2 * Vec<T>::kN), kSlot = kBwdThreads * 16;
    p.heads_per_block = p.H < kBwdThreads / IPR ? p.H : kBwdThreads / IPR;
    const dim3 grid(p.n_part, (p.H + p.heads_per_block - 1) / p.heads_per_block);
    const auto kernel = norm_backward_kernel<T, D, kGrads, kInter>;
    static SmemLimit limit;
    if (cudaError_t e = limit.ensure((const void *)kernel, kDepth * 4 * kSlot); e != cudaSuccess) return e;
    // slots for the tokens of a thread, where those are few
    const int lanes = kBwdThreads / (p.heads_per_block * IPR), step = kTabTokens;
    const long long m = (p.n + p.n_part - 1) / p.n_part, most = (m + step - 1) / step * ((step + lanes - 1) / lanes);
    int bytes = (int)(most < kDepth ? most : kDepth) * 4 * kSlot;
    const int sums = Vec<T>::kN * kSlot * 3 / 2;  // the sums' exchange: 4 VEC floats a thread, 2 VEC for the weight's
    if (kGrads && bytes < sums) bytes = sums;
    kernel<<<grid, kBwdThreads, bytes, s>>>(p);
    return cudaGetLastError();
}
template <typename T, int D> cudaError_t backward_t(const RotateBwdParams &p, cudaStream_t s) {
    if (p.d_alpha || p.d_weight) return p.interleaved ? backward_k<T, D, true, true>(p, s) : backward_k<T, D, true, false>(p, s);
    return p.interleaved ? backward_k<T, D, false, true>(p, s) : backward_k<T, D, false, false>(p, s);
}

}  // namespace

#define ORTHROS_BY_TYPE(FN, P)                                                                          \
    (dtype == ORTHROS_F32 ? (d == 128 ? FN<float, 128>(P, stream) : FN<float, 64>(P, stream))           \
                          : (d == 128 ? FN<__nv_bfloat16, 128>(P, stream) : FN<__nv_bfloat16, 64>(P, stream)))

cudaError_t launch_norm_rotate(const RotateParams &p, int d, orthros_dtype dtype, cudaStream_t stream) {
    return ORTHROS_BY_TYPE(move_t, p);
}
cudaError_t launch_norm_rotate_backward(const RotateBwdParams &p, int d, orthros_dtype dtype, cudaStream_t stream) {
    return ORTHROS_BY_TYPE(backward_t, p);
}
#undef ORTHROS_BY_TYPE

cudaError_t launch_norm_grad_sum(const RotateBwdParams &p, int d, int elem_bytes, cudaStream_t stream) {
    const int cols = p.H * d;
    const int blocks = (p.d_alpha ? 2 * cols / 32 : 0) + (p.d_weight ? d / 32 : 0);
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(blocks);
    cfg.blockDim = dim3(kSumWarps * 32);
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, norm_grad_sum_kernel, p, cols, d, p.n_part * rotate_grad_groups(p.H, d, elem_bytes));
}

}  // namespace orthros
