// rotary.cuh -- what the rotary kernels have in common, with and without a norm of
// the head (rotary.cu, norm_rotary.cu): work items, angles, token slots, the grid
// of a moving kernel.
//
// Mathematics. Pair i of a head at position t turns by the angle t * f_i:
//   (y_a, y_b) = m (u_a cos - u_b sin, u_a sin + u_b cos)
// over the first `rot` channels (pairs (i, i + rot/2) or (2i, 2i + 1)); the
// other channels leave as u.
//
// Angles. t * f_i in fp32 loses its fraction at long positions (an ulp at
// t = 131072, f = 1 is 0.008 rad), so frequencies arrive as 64-bit fixed-point
// fractions of a turn, rounded to half a unit: the phase of position t is the low
// 64 bits of t * step, an integer product that wraps as the angle does, off by
// 2^-34 turn at most. Its top 32 bits (2^-32 turn, 1.5e-9 rad), as a float (pi 2^-24),
// go through sincospif (2^-23): sin and cos are off by less than 4e-7 at every 32-bit
// position, negative ones included.
//
// Arithmetic is fp32 throughout, rounded once to the element type on the store;
// the affine's gradients are accumulated and returned in fp32.
#pragma once
#include "internal.cuh"

namespace orthros {
namespace rope {

// A row (one head of one token) is moved in work items of two 16-byte vectors.
// Half layout: a rotated item holds the two vectors of VEC pairs, i and i +
// rot/2/VEC; the channels past `rot` are items of two consecutive vectors.
// Interleaved layout: pairs lie within a vector, so item i takes vectors i and
// i + D/2/VEC, and neighbouring lanes move neighbouring vectors (two consecutive
// vectors per lane left every 32-byte sector to two instructions: 189 against
// 133 us for 32768 x 32 x 128 bf16). rot is a multiple of 16, so every vector is
// rotated or not as a whole.
template <typename T> struct Vec {
    static constexpr int kN = 16 / (int)sizeof(T);
};

// 16 bytes from global to shared memory, not through registers.
__device__ __forceinline__ void copy16(uint4 *to, const void *from) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"((uint32_t)__cvta_generic_to_shared(to)), "l"(from) : "memory");
}

// cos and sin of position t's angle for one frequency step, times the amplitude.
__device__ __forceinline__ void angle(int t, uint64_t step, float amp, float &c, float &s) {
    const uint64_t phase = static_cast<uint64_t>(static_cast<int64_t>(t)) * step;  // modulo one turn
    const int hi = static_cast<int>(static_cast<uint32_t>(phase >> 32));           // in units of 2^-32 turn
    sincospif(static_cast<float>(hi) * 4.656612873077393e-10f, &s, &c);            // 2 pi hi 2^-32 = pi (hi 2^-31)
    c *= amp;
    s *= amp;
}

// The two vectors of a work item: first channels, and which of them rotate.
// Pair j of the item's angles is pair first_a + j (vector a and, in the half
// layout, b) for j < n_a, and first_b + j - VEC/2 for an interleaved vector b.
template <int VEC, int D> struct Item {
    int ca, cb;
    bool ra, rb;
    __device__ __forceinline__ Item(int i, int rot, bool interleaved) {
        const bool split = !interleaved && 2 * VEC * i < rot;  // a rotated item of the half layout
        ca = interleaved || split ? VEC * i : 2 * VEC * i;
        cb = interleaved ? ca + D / 2 : split ? ca + (rot >> 1) : ca + VEC;
        ra = interleaved ? ca < rot : split;
        rb = interleaved ? cb < rot : split;
    }
    // pair of the item's j-th angle (interleaved: the first VEC/2 are vector a's, the others b's)
    __device__ __forceinline__ int pair(int j, bool interleaved) const {
        return !interleaved ? ca + j : j < VEC / 2 ? ca / 2 + j : cb / 2 + j - VEC / 2;
    }
    __device__ __forceinline__ bool turns(int j, bool interleaved) const {
        return !interleaved || j < VEC / 2 ? ra : rb;
    }
};

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

// Cosines and sines of a few tokens are computed once by a block and shared by its heads.
constexpr int kTabTokens = 16;  // at most
constexpr int kRunTokens = 128;  // positions (and page slots) a block looks up at a time
constexpr int kBatch = 4;        // tokens whose loads a thread of the moving kernel has in flight
// Tokens of a table (a divisor of kRunTokens), for so many handled side by side: one
// batch of loads a thread, which are under way while the angles are computed. Two
// batches leave the second one's trip to memory bare: 16384 x 32 x 128 fp32 96 us
// instead of 86, 32768 x 8 x 128 53 instead of 46.
__device__ __forceinline__ int table_tokens(int lanes) { return lanes > 2 ? kTabTokens : kBatch * lanes; }

constexpr int kMoveThreads = 512;  // of a moving kernel's block, at most
constexpr int kBwdThreads = 512;   // of a gradient kernel's block
constexpr int kBwdBlocks = 1;      // its blocks per SM

// Token slot of new token i in the page pool, or -1 when it has none.
__device__ __forceinline__ long long page_slot(const RotateParams &p, long long i) {
    if (p.slots) {  // given by the caller
        const int s = p.slots[i];
        return s >= 0 && s < (long long)p.num_pages * p.page_size ? s : -1;
    }
    const int b = p.token_seq[i], t = p.positions[i];
    if (b < 0 || b >= p.B || t < 0 || t / p.page_size >= p.max_pages) return -1;
    const int pg = p.block_table[(long long)b * p.max_pages + t / p.page_size];
    if (pg < 0 || pg >= p.num_pages) return -1;
    return (long long)pg * p.page_size + t % p.page_size;
}

// The status word of an append, written by a block of its own that checks every new
// token beside the moving ones: no reset launch before the kernel, no atomics.
__device__ __forceinline__ void write_status(const RotateParams &p) {
    constexpr int kBatchS = 8;  // tokens a thread looks up at once
    uint32_t wrong = 0;
    if (p.slots)  // -1: a token that is not cached
        for (long long i = threadIdx.x; i < p.n; i += blockDim.x) {
            const int s = p.slots[i];
            if (s < -1 || s >= (long long)p.num_pages * p.page_size) wrong |= ORTHROS_DEV_BAD_PAGE;
        }
    for (long long i0 = threadIdx.x; !p.slots && i0 < p.n; i0 += (long long)kBatchS * blockDim.x) {
        int b[kBatchS], t[kBatchS];
#pragma unroll
        for (int u = 0; u < kBatchS; ++u) {
            const long long i = i0 + (long long)u * blockDim.x;
            b[u] = i < p.n ? p.token_seq[i] : 0;
            t[u] = i < p.n ? p.positions[i] : -1;
        }
#pragma unroll
        for (int u = 0; u < kBatchS; ++u) {
            if (i0 + (long long)u * blockDim.x >= p.n) break;
            if (b[u] < 0 || b[u] >= p.B || t[u] < 0 || t[u] / p.page_size >= p.max_pages) {
                wrong |= ORTHROS_DEV_BAD_POSITION;
            } else {
                const int pg = p.block_table[(long long)b[u] * p.max_pages + t[u] / p.page_size];
                if (pg < 0 || pg >= p.num_pages) wrong |= ORTHROS_DEV_BAD_PAGE;
            }
        }
    }
    const int pos = __syncthreads_or(wrong & ORTHROS_DEV_BAD_POSITION), pg = __syncthreads_or(wrong & ORTHROS_DEV_BAD_PAGE);
    if (threadIdx.x == 0) *p.status = (pos ? ORTHROS_DEV_BAD_POSITION : 0u) | (pg ? ORTHROS_DEV_BAD_PAGE : 0u);
}

// The grid of a moving kernel. The heads of a token are cut into equal groups, a block per group: as few groups
// as fill the SM's registers with threads to within a tenth (a token's 48
// virtual heads of 8 items in one group are a block of 384 threads where 512
// fit, three groups of 16 fill them), since every group computes the token's
// angles again. Several tokens go side by side when a group is narrow. Blocks
// along the tokens: as many as run at once, with equal runs of tokens.
struct MoveGrid {
    int heads_per_block, threads, blocks, out_blocks, groups;  // blocks along the new tokens, the output rows
};
inline MoveGrid move_grid(int heads, int items, int per_sm, long long n, long long n_out, bool append) {
    MoveGrid m{};
    int best = 0;
    const int g0 = (heads * items + kMoveThreads - 1) / kMoveThreads;
    for (int g = g0; g <= g0 + 3 && g <= heads; ++g) {
        const int h = (heads + g - 1) / g, row = h * items;
        const int side = row >= 256 ? 1 : 256 / row < kTabTokens ? 256 / row : kTabTokens;
        const int t = (row * side + 31) / 32 * 32;
        const int busy = (int)((long long)(per_sm / t) * (side * row) * heads / ((long long)h * g));  // threads with work
        if (busy > best + best / 10) m.groups = g, m.heads_per_block = h, m.threads = t, best = busy;
    }
    const int lanes = m.threads / (m.heads_per_block * items);  // (the kernel's)
    // blocks that run at once (append: one of them, in each group's row, for the status
    // word), shared between the new tokens and the output stream's rows by their
    // number: a second wave of a few short blocks cost 3 us
    const int fit = device_sm_count() * (per_sm / m.threads < 32 ? per_sm / m.threads : 32) / m.groups - (append ? 1 : 0);
    const long long most = (n + lanes - 1) / lanes, most_out = (n_out + lanes - 1) / lanes;
    long long out = n_out == 0 ? 0 : fit * n_out / (n + n_out);
    out = out > most_out ? most_out : out < 1 && n_out > 0 ? 1 : out;
    long long blocks = fit - out;
    blocks = blocks > most ? most : blocks < 1 && n > 0 ? 1 : blocks < 0 ? 0 : blocks;
    m.blocks = (int)blocks;
    m.out_blocks = (int)out;
    return m;
}
// Threads of a kernel that an SM's registers hold (looked up once per kernel, kept in `resident`).
inline cudaError_t resident_threads(const void *kernel, std::atomic<int> &resident, int &per_sm) {
    per_sm = resident.load(std::memory_order_relaxed);
    if (per_sm != 0) return cudaSuccess;
    cudaFuncAttributes at;
    if (cudaError_t e = cudaFuncGetAttributes(&at, kernel); e != cudaSuccess) return e;
    per_sm = 65536 / ((at.numRegs + 7) / 8 * 8);
    resident.store(per_sm, std::memory_order_relaxed);
    return cudaSuccess;
}

}  // namespace rope
}  // namespace orthros
