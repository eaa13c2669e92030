// rotary.cu -- rotary positions: the affine of a query stream followed by the
// rotation of its channel pairs, the gradient of both, and the paged append
// that rotates new keys on their way into the cache.
//
// Mathematics. Pair i of a head at position t turns by the angle t * f_i:
//   (y_a, y_b) = m (u_a cos - u_b sin, u_a sin + u_b cos),  u = alpha (.) x + beta,
// over the first `rot` channels (pairs (i, i + rot/2) or (2i, 2i + 1)); the
// other channels leave as u. The rotation is orthogonal, so its gradient is the
// rotation by the opposite angle: g = m R(-t) dy, dx = alpha (.) g,
// d_alpha = sum_t g (.) x, d_beta = sum_t g. Angles and precision: rotary.cuh.
#include "rotary.cuh"

namespace orthros {

using namespace rope;

namespace {

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

// Rotates the pairs of an item in place: (a[j], b[j]) in the half layout,
// neighbours of the 2 VEC channels in the interleaved one.
template <int VEC, int D>
__device__ __forceinline__ void turn(float (&a)[VEC], float (&b)[VEC], const float (&c)[VEC], const float (&s)[VEC],
                                     const Item<VEC, D> &it, bool interleaved) {
    if (!interleaved) {
        if (!it.ra) return;
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
            const float x = a[j], y = b[j];
            a[j] = fmaf(x, c[j], -y * s[j]);
            b[j] = fmaf(x, s[j], y * c[j]);
        }
        return;
    }
    if (it.ra) {
#pragma unroll
        for (int j = 0; j < VEC / 2; ++j) {
            const float x = a[2 * j], y = a[2 * j + 1];
            a[2 * j] = fmaf(x, c[j], -y * s[j]);
            a[2 * j + 1] = fmaf(x, s[j], y * c[j]);
        }
    }
    if (it.rb) {
#pragma unroll
        for (int j = 0; j < VEC / 2; ++j) {
            const float x = b[2 * j], y = b[2 * j + 1];
            b[2 * j] = fmaf(x, c[VEC / 2 + j], -y * s[VEC / 2 + j]);
            b[2 * j + 1] = fmaf(x, s[VEC / 2 + j], y * c[VEC / 2 + j]);
        }
    }
}

// Cosines and sines of a few tokens, computed once by the block and shared by its
// heads: entry (token, j / 2, item) holds angles j and j + 1 of the item, so the
// lanes of a row read consecutive 16-byte words.
template <typename T, int D> struct Table {
    static constexpr int VEC = Vec<T>::kN, IPR = D / (2 * VEC), kQ = VEC / 2;
    float4 e[kTabTokens][kQ][IPR];
    // angles of cnt positions; sign -1 for the transposed rotation
    __device__ __forceinline__ void fill(const int *pos, int cnt, const uint64_t *steps, int rot, bool interleaved, float amp,
                                         float sign) {
        const int half = rot >> 1;
        for (int x = threadIdx.x; x < cnt * half; x += blockDim.x) {
            const int k = x / half, pr = x % half;
            float c, s;
            angle(pos[k], __ldg(steps + pr), amp, c, s);
            int i, j;  // the item and its angle that pair pr is
            if (!interleaved) i = pr / VEC, j = pr % VEC;
            else i = (pr % (D / 4)) / kQ, j = pr % kQ + (pr >= D / 4 ? kQ : 0);
            reinterpret_cast<float2 *>(&e[k][j / 2][i])[j & 1] = make_float2(c, sign * s);
        }
    }
    __device__ __forceinline__ void read(int k, int item, float (&c)[VEC], float (&s)[VEC]) const {
#pragma unroll
        for (int q = 0; q < kQ; ++q) {
            const float4 v = e[k][q][item];
            c[2 * q] = v.x, s[2 * q] = v.y, c[2 * q + 1] = v.z, s[2 * q + 1] = v.w;
        }
    }
};

// ---------------------------------------------------------------------------
// Forward and append: one kernel moves rows. A thread owns one (head, item) with
// the affine's channels in registers and walks the tokens of its block, kBatch
// tokens' loads in flight; the angles come from the block's table. Blocks take
// equal runs of tokens, as many as fit the GPU at once. Bound by HBM: every
// element read once and written once. 32768 x 32 x 128 bf16 with the affine: 86 us,
// 6.2 TB/s (92 % of the measured copy rate). Threads that owned a token and
// walked its heads read the affine from L1 for every head (116 us, L1 70 % busy);
// two tokens in flight instead of four, 117 us; eight do not fit the registers.
//
// The virtual heads of a token are its Hq query heads, then (append) its Hkv key
// heads and Hkv value heads. Blocks from p.blocks on (along x) move the output
// stream's rows; an append's last one writes the status word.
// ---------------------------------------------------------------------------
template <typename T, int D, bool kAppend>
__global__ void __launch_bounds__(kMoveThreads) rotate_move_kernel(const RotateParams p) {
    constexpr int VEC = Vec<T>::kN, IPR = D / (2 * VEC);
    __shared__ Table<T, D> tab[2];
    __shared__ int pos[kRunTokens];
    __shared__ long long slot[kRunTokens];  // append: first element of the token's page slot, or -1
    if (kAppend && blockIdx.x == gridDim.x - 1) {
        if (blockIdx.y == 0) write_status(p);
        return;
    }
    const int tid = threadIdx.x;
    const int hb = p.heads_per_block;
    const int lanes = blockDim.x / (hb * IPR);  // tokens handled side by side
    const int tl = tid / (hb * IPR);
    const int h = blockIdx.y * hb + (tid / IPR) % hb;
    const int item = tid % IPR;
    const bool out = kAppend && (int)blockIdx.x >= p.blocks;
    const int bx = out ? blockIdx.x - p.blocks : blockIdx.x, nbx = out ? gridDim.x - 1 - p.blocks : p.blocks;
    const long long n = out ? p.n_out : p.n;
    const int32_t *positions = out ? p.out_positions : p.positions;
    // what this thread's virtual head moves
    const T *src = static_cast<const T *>(out ? p.x_out : p.x);
    T *dst = static_cast<T *>(out ? p.y_out : p.y);
    long long ss = out ? p.x_out_stride : p.x_stride, ds = p.y_stride;
    const float *alpha = out ? p.alpha_out : p.alpha, *beta = out ? p.beta_out : p.beta;
    int hh = h;                  // head within its tensor
    bool paged = false, value = false;
    if (kAppend && h >= p.H) {
        hh = h - p.H;
        paged = true;
        value = hh >= p.Hkv;
        if (value) hh -= p.Hkv;
        src = static_cast<const T *>(value ? p.v : p.k);
        dst = static_cast<T *>(value ? p.v_cache : p.k_cache);
        ss = value ? p.v_stride : p.k_stride;
        alpha = beta = nullptr;
    }
    const bool active = tl < lanes && (kAppend ? (paged ? !out && h < p.H + 2 * p.Hkv : src != nullptr) : h < p.H);
    Item<VEC, D> it(item, p.rot, p.interleaved);
    if (value) it.ra = it.rb = false;
    src += hh * D;
    dst += hh * D;
    float al[2][VEC], be[2][VEC];
    const bool affine = active && alpha;
    if (affine) {
        load_affine<VEC>(alpha + hh * D, it.ca, it.cb, al[0], al[1]);
        load_affine<VEC>(beta + hh * D, it.ca, it.cb, be[0], be[1]);
    }
    const long long n0 = n * bx / nbx, n1 = n * (bx + 1) / nbx;
    const int step = table_tokens(lanes);
    int buf = 0;
    for (long long base = n0; base < n1; base += step, buf ^= 1) {
        const int cnt = (int)min((long long)step, n1 - base);
        const int run = (int)((base - n0) % kRunTokens);  // first entry of these tokens in pos and slot
        // the first batch's loads are under way while the angles are computed
        uint4 ra[kBatch], rb[kBatch];
        auto load = [&](int k0) {
#pragma unroll
            for (int u = 0; u < kBatch; ++u) {
                const int k = k0 + u * lanes;
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
                if (kAppend && !out) {
                    const long long at = page_slot(p, base + k);
                    slot[k] = at < 0 ? -1 : at * p.Hkv * D;
                }
            }
            __syncthreads();
        }
        tab[buf].fill(pos + run, cnt, p.steps, p.rot, p.interleaved, p.amplitude, 1.f);
        __syncthreads();
        if (!active) continue;
        for (int k0 = tl; k0 < cnt; k0 += kBatch * lanes) {
            if (k0 != tl) load(k0);
#pragma unroll
            for (int u = 0; u < kBatch; ++u) {
                const int k = k0 + u * lanes;
                if (k >= cnt) break;
                T *to = kAppend && paged ? dst + slot[run + k] : dst + (base + k) * ds;
                if (kAppend && paged && slot[run + k] < 0) continue;
                if (value) {
                    *reinterpret_cast<uint4 *>(to + it.ca) = ra[u];
                    *reinterpret_cast<uint4 *>(to + it.cb) = rb[u];
                    continue;
                }
                float a[VEC], b[VEC], c[VEC], s[VEC];
                unpack<T>(ra[u], a);
                unpack<T>(rb[u], b);
                if (affine) {
#pragma unroll
                    for (int j = 0; j < VEC; ++j) {
                        a[j] = fmaf(a[j], al[0][j], be[0][j]);
                        b[j] = fmaf(b[j], al[1][j], be[1][j]);
                    }
                }
                tab[buf].read(k, item, c, s);
                turn<VEC, D>(a, b, c, s, it, p.interleaved);
                *reinterpret_cast<uint4 *>(to + it.ca) = pack<T>(a);
                *reinterpret_cast<uint4 *>(to + it.cb) = pack<T>(b);
            }
        }
    }
}

// ---------------------------------------------------------------------------
// Backward. A block covers a run of tokens and a group of heads; a thread owns one
// (head, item) and walks the block's tokens with the affine's gradient in
// registers, so d_alpha and d_beta cost no traffic per token. The block's sums go
// to the workspace as one partial each, and rotate_grad_sum_kernel adds the
// partials in a fixed order (no atomics: the same call gives the same bits).
// Rows reach a thread through slots of its own in shared memory, kBwdDepth tokens
// ahead: no other thread touches them, so they need no barrier.
// Bound by HBM: dy and x read once, dx written. 32768 x 32 x 128 bf16: 133 us,
// 6.0 TB/s (89 % of the measured copy rate; the sum of the partials is 5 us of
// it). 138 us with four tokens in flight in registers (which they filled with 256
// threads), 138 with three ahead instead of six, 143 as two blocks of 256
// threads. The moving kernel above keeps its loads in registers: through
// shared memory it took 84 to 110 us by the depth, and its append 38 to 46.
// ---------------------------------------------------------------------------
constexpr int kBwdDepth = 6;   // tokens a thread has in flight

template <typename T, int D, bool kGrads>
__global__ void __launch_bounds__(kBwdThreads, kBwdBlocks) rotate_backward_kernel(const RotateBwdParams p) {
    constexpr int VEC = Vec<T>::kN, IPR = D / (2 * VEC), kV = kGrads ? 4 : 2;
    extern __shared__ uint4 fifo[];  // [kBwdDepth][kV][thread]
    __shared__ Table<T, D> tab[2];
    __shared__ int pos[kRunTokens];
    const int tid = threadIdx.x;
    const int hb = p.heads_per_block;            // heads of this block
    const int lanes = kBwdThreads / (hb * IPR);  // tokens handled side by side
    const int tl = tid / (hb * IPR);
    const int h = blockIdx.y * hb + (tid / IPR) % hb;
    const int item = tid % IPR;
    const bool active = tl < lanes && h < p.H;
    const Item<VEC, D> it(item, p.rot, p.interleaved);
    const int ca = it.ca, cb = it.cb;
    const long long n0 = p.n * blockIdx.x / gridDim.x, n1 = p.n * (blockIdx.x + 1) / gridDim.x;
    constexpr int step = kTabTokens;
    const int n = (int)(n1 - n0);
    // this thread's tokens, kBwdDepth of them ahead
    int ahead = 0, ahead_k = tl, wr = 0;
    auto fetch = [&]() {
        if (active && ahead_k < step && ahead + ahead_k < n) {
            uint4 *to = fifo + wr * kV * kBwdThreads + tid;
            const long long i = n0 + ahead + ahead_k;
            const T *dy = static_cast<const T *>(p.dy) + i * p.dy_stride + h * D;
            copy16(to, dy + ca);
            copy16(to + kBwdThreads, dy + cb);
            if constexpr (kGrads) {
                const T *x = static_cast<const T *>(p.x) + i * p.x_stride + h * D;
                copy16(to + 2 * kBwdThreads, x + ca);
                copy16(to + 3 * kBwdThreads, x + cb);
            }
            ahead_k += lanes;
            if (ahead_k >= step) ahead += step, ahead_k = tl;
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
        wr = wr + 1 == kBwdDepth ? 0 : wr + 1;
    };
    for (int i = 0; i < kBwdDepth; ++i) fetch();
    float al[2][VEC], da[2][VEC], db[2][VEC];
#pragma unroll
    for (int j = 0; j < VEC; ++j) {
        al[0][j] = al[1][j] = 1.f;
        da[0][j] = da[1][j] = db[0][j] = db[1][j] = 0.f;
    }
    if (active && p.alpha) load_affine<VEC>(p.alpha + h * D, ca, cb, al[0], al[1]);
    int buf = 0, rd = 0;
    for (int base = 0; base < n; base += step, buf ^= 1) {
        const int cnt = min(step, n - base);
        const int run = base % kRunTokens;  // first entry of these tokens in pos
        if (run == 0) {
            __syncthreads();
            for (int k = tid; k < kRunTokens && base + k < n; k += kBwdThreads) pos[k] = p.positions[n0 + base + k];
            __syncthreads();
        }
        tab[buf].fill(pos + run, cnt, p.steps, p.rot, p.interleaved, p.amplitude, -1.f);  // the opposite angle
        __syncthreads();
        if (!active) continue;
        for (int k = tl; k < cnt; k += lanes) {
            asm volatile("cp.async.wait_group %0;" ::"n"(kBwdDepth - 1) : "memory");
            const uint4 *from = fifo + rd * kV * kBwdThreads + tid;
            rd = rd + 1 == kBwdDepth ? 0 : rd + 1;
            float a[VEC], b[VEC], c[VEC], s[VEC];
            float x0[VEC], x1[VEC];
            unpack<T>(from[0], a);
            unpack<T>(from[kBwdThreads], b);
            if constexpr (kGrads) {
                unpack<T>(from[2 * kBwdThreads], x0);
                unpack<T>(from[3 * kBwdThreads], x1);
            }
            tab[buf].read(k, item, c, s);
            turn<VEC, D>(a, b, c, s, it, p.interleaved);
            if constexpr (kGrads) {
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
            T *dx = static_cast<T *>(p.dx) + (n0 + base + k) * p.dx_stride + h * D;
            *reinterpret_cast<uint4 *>(dx + ca) = pack<T>(a);
            *reinterpret_cast<uint4 *>(dx + cb) = pack<T>(b);
            fetch();  // into the slot this thread has just read
        }
    }
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    if constexpr (kGrads) {
        // sums over the token lanes of the block, through the shared memory that the loads have left:
        // [value of a thread][thread]
        float *red = reinterpret_cast<float *>(fifo);
        __syncthreads();
#pragma unroll
        for (int v = 0; v < 2; ++v) {
#pragma unroll
            for (int j = 0; j < VEC; ++j) {
                red[(v * VEC + j) * kBwdThreads + tid] = da[v][j];
                red[((2 + v) * VEC + j) * kBwdThreads + tid] = db[v][j];
            }
        }
        __syncthreads();
        float *part = p.partial + (long long)blockIdx.x * 2 * p.H * D;
        const int row = hb * IPR;  // threads of a token lane
        if (!active) return;
        for (int v = tl; v < 4 * VEC; v += lanes) {  // this thread's channels, shared with its fellows of other lanes
            const float *from = red + v * kBwdThreads + tid - tl * row;
            float sum = 0.f;
            for (int l = 0; l < lanes; ++l) sum += from[l * row];
            const int j = v % VEC, ch = h * D + (v / VEC & 1 ? cb : ca) + j;
            part[(v < 2 * VEC ? 0 : p.H * D) + ch] = sum;
        }
    }
}

// d_alpha and d_beta: column sums over the n_part partials [n_part, 2, H d].
// A block takes 32 columns; its 8 warps stride over the partials.
__global__ void __launch_bounds__(256) rotate_grad_sum_kernel(const float *partial, int n_part, int cols, float *d_alpha,
                                                              float *d_beta) {
    __shared__ float red[8][32];
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    const int col = blockIdx.x * 32 + lane;  // cols (= H d) is a multiple of 32: no block straddles the two
    float s0 = 0.f, s1 = 0.f, s2 = 0.f, s3 = 0.f;
    asm volatile("griddepcontrol.wait;" ::: "memory");  // (a dependent launch: the partials are there now)
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

template <typename T, int D, bool kAppend> cudaError_t move_t(RotateParams p, int heads, cudaStream_t s) {
    static std::atomic<int> resident{0};
    int per_sm = 0;
    if (cudaError_t e = resident_threads((const void *)rotate_move_kernel<T, D, kAppend>, resident, per_sm); e != cudaSuccess) return e;
    const MoveGrid m = move_grid(heads, D / (2 * Vec<T>::kN), per_sm, p.n, p.n_out, kAppend);
    p.heads_per_block = m.heads_per_block;
    p.blocks = m.blocks;
    const dim3 grid((unsigned)(m.blocks + m.out_blocks + (kAppend ? 1 : 0)), m.groups);
    rotate_move_kernel<T, D, kAppend><<<grid, m.threads, 0, s>>>(p);
    return cudaGetLastError();
}

template <typename T, int D> cudaError_t rotate_t(const RotateParams &p, cudaStream_t s) {
    return move_t<T, D, false>(p, p.H, s);
}
template <typename T, int D> cudaError_t append_t(const RotateParams &p, cudaStream_t s) {
    return move_t<T, D, true>(p, p.H + 2 * p.Hkv, s);
}

template <typename T, int D> cudaError_t backward_t(RotateBwdParams p, cudaStream_t s) {
    constexpr int IPR = D / (2 * Vec<T>::kN);
    p.heads_per_block = p.H < kBwdThreads / IPR ? p.H : kBwdThreads / IPR;
    const dim3 grid(p.n_part, (p.H + p.heads_per_block - 1) / p.heads_per_block);
    const bool grads = p.d_alpha != nullptr;
    const auto kernel = grads ? rotate_backward_kernel<T, D, true> : rotate_backward_kernel<T, D, false>;
    constexpr int kSlot = kBwdThreads * 16;
    static SmemLimit limit[2];
    if (cudaError_t e = limit[grads].ensure((const void *)kernel, kBwdDepth * (grads ? 4 : 2) * kSlot); e != cudaSuccess) return e;
    // slots for the tokens of a thread, where those are few
    const int lanes = kBwdThreads / (p.heads_per_block * IPR), step = kTabTokens;
    const long long m = (p.n + p.n_part - 1) / p.n_part, most = (m + step - 1) / step * ((step + lanes - 1) / lanes);
    int fifo = (int)(most < kBwdDepth ? most : kBwdDepth) * (grads ? 4 : 2) * kSlot;
    if (grads && fifo < Vec<T>::kN * kSlot) fifo = Vec<T>::kN * kSlot;  // the sums' exchange
    kernel<<<grid, kBwdThreads, fifo, s>>>(p);
    return cudaGetLastError();
}

}  // namespace

// Groups of heads that the gradient's blocks take (one where a block holds all heads).
int rotate_grad_groups(int H, int d, int elem_bytes) {
    const int per = kBwdThreads / (d * elem_bytes / 32);  // heads of a block
    return (H + per - 1) / per;
}

// Partials of the affine's gradient (blocks along the tokens): kBwdBlocks per
// SM over all head groups, but no fewer than 16 tokens a block.
int rotate_grad_parts(long long n, int H, int d, int elem_bytes) {
    const int groups = rotate_grad_groups(H, d, elem_bytes);
    long long parts = (long long)kBwdBlocks * device_sm_count() / groups;
    if (parts > (n + 15) / 16) parts = (n + 15) / 16;
    return parts < 1 ? 1 : (int)parts;
}

#define ORTHROS_BY_TYPE(FN, P)                                                                          \
    (dtype == ORTHROS_F32 ? (d == 128 ? FN<float, 128>(P, stream) : FN<float, 64>(P, stream))           \
                          : (d == 128 ? FN<__nv_bfloat16, 128>(P, stream) : FN<__nv_bfloat16, 64>(P, stream)))

cudaError_t launch_rotate(const RotateParams &p, int d, orthros_dtype dtype, cudaStream_t stream) {
    return ORTHROS_BY_TYPE(rotate_t, p);
}
cudaError_t launch_rotate_append(const RotateParams &p, int d, orthros_dtype dtype, cudaStream_t stream) {
    return ORTHROS_BY_TYPE(append_t, p);
}
cudaError_t launch_rotate_backward(const RotateBwdParams &p, int d, orthros_dtype dtype, cudaStream_t stream) {
    return ORTHROS_BY_TYPE(backward_t, p);
}
cudaError_t launch_rotate_grad_sum(const RotateBwdParams &p, int d, cudaStream_t stream) {
    const int cols = p.H * d;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(2 * cols / 32);
    cfg.blockDim = dim3(256);
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, rotate_grad_sum_kernel, (const float *)p.partial, p.n_part, cols, p.d_alpha, p.d_beta);
}
#undef ORTHROS_BY_TYPE

}  // namespace orthros
