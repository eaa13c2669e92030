// step_plan.cu -- what a serving step needs from its lengths, made on the GPU:
// pages for the sequences that grow, the sequence, position and slot of every
// new token, and the ancestor masks of drafted trees; and the move of an accepted
// path to its places in the cache.
//
// Plan. With L_b cached and m_b new tokens, sequence b needs ceil((L_b + m_b) / P)
// pages; what it lacks it takes from the top of the free stack, the sequences in
// order, so that its share is an exclusive prefix sum of the lacks. Ended
// sequences (m_b = -1) push theirs before, if all their ids are the pool's. A
// token's sequence is found by a binary search in the prefix sums of m_b, its page
// in the table or, if it is a new one, on the stack: no thread waits for another's
// table entry.
//
// One launch of one cluster: every CTA computes all prefix sums in shared memory
// (a few microseconds of loads whatever the CTAs), then a cluster barrier stands
// between the last read of the inputs and the first write of the outputs, so that
// a length, a page count or the height of the stack may be updated in place. Bound by
// the latency of that chain (load, scan, barrier, table look-up, store), not by
// bytes: a step's arrays are a few hundred KB. 64 decoding sequences: 4.5 us; 500
// trees of up to 64 tokens, 18000 rows, 31 ended sequences: 11.3 us, 0.9 of them the look at
// the ended ones' page ids (16.7 without it, but with one CTA's threads returning a sequence's
// pages each and the lengths read again for every pass).
#include "internal.cuh"

namespace orthros {
namespace {

constexpr int kThreads = 1024, kWarps = kThreads / 32;
constexpr int kMaxCluster = 8;

__device__ __forceinline__ long long warp_scan(long long v, int lane) {  // inclusive
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long u = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o) v += u;
    }
    return v;
}

// Last index i of a non-decreasing a[0 .. n-1] with a[i] <= x (a[0] <= x).
__device__ __forceinline__ int last_at_most(const int *a, int n, int x) {
    int lo = 0, hi = n;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (a[mid] <= x) lo = mid;
        else hi = mid;
    }
    return lo;
}

// One sequence's part of the plan.
struct Need {
    int rows, cached, held;  // tokens of the step, cached ones, pages held
    int lack, back;          // pages to take, pages to give back
    bool ends, wrong;        // has ended; lengths that cannot be
};
__device__ __forceinline__ Need need_of(const StepPlanParams &p, int b) {
    Need s;
    s.cached = p.cache_lens[b];
    s.held = p.held_in[b];
    const int m = p.new_lens[b];
    s.rows = max(m, 0);
    const long long total = (long long)s.cached + s.rows;
    s.wrong = m < -1 || s.held < 0 || s.held > p.max_pages ||
              (m >= 0 && (s.cached < 0 || total > (long long)p.max_pages * p.page_size || (p.parents && m > p.max_tree)));
    s.lack = s.back = 0;
    s.ends = !s.wrong && m < 0;
    if (s.wrong) return s;
    if (s.ends) s.back = s.held;
    else s.lack = max(s.held, (int)((total + p.page_size - 1) / p.page_size)) - s.held;
    return s;
}

// Whether this lane finds an id from outside the pool among the first n pages of sequence b (each lane looks at its own).
__device__ __forceinline__ bool foreign_page(const StepPlanParams &p, int b, int n, int lane) {
    const int32_t *row = p.block_table + (long long)b * p.max_pages;
    constexpr int kPages = 16;  // of a lane at a time
    bool foreign = false;
    for (int i0 = lane; i0 < n; i0 += 32 * kPages) {
        int id[kPages];
#pragma unroll
        for (int u = 0; u < kPages; ++u) id[u] = i0 + 32 * u < n ? row[i0 + 32 * u] : 0;
#pragma unroll
        for (int u = 0; u < kPages; ++u) foreign |= id[u] < 0 || id[u] >= p.num_pages;
    }
    return foreign;
}

// (aligned: every thread of a warp at once, which a branch of one lane just before does not leave for certain)
__device__ __forceinline__ void cluster_arrive_wait() {
    __syncwarp();
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// kWords: 32-bit words that hold a token's mask (0: no trees), at least p.words.
template <int kWords> __global__ void __launch_bounds__(kThreads) step_plan_kernel(const StepPlanParams p) {
    extern __shared__ int sm[];
    int *start = sm;                  // [B + 1] first token row
    int *off = start + p.B + 1;       // [B + 1] pages taken by the sequences before it
    int *cached = off + p.B + 1;      // [B] cached tokens, or -1: the sequence has no place in this step
    int *held = cached + p.B;         // [B] pages held before, or -1: it has ended
    __shared__ long long wsum[3][kWarps], carry[3];
    __shared__ int s_taken;
    __shared__ uint32_t s_flags;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int rank = blockIdx.x, ctas = gridDim.x;  // one cluster
    if (tid == 0) {
        carry[0] = carry[1] = carry[2] = 0;
        s_taken = 0;
        s_flags = 0;
    }
    const int count = *p.count_in;
    __syncthreads();
    // prefix sums over the sequences, 1024 at a time: token rows, pages to take, pages to give back
    uint32_t flags = 0;
    for (int base = 0; base < p.B; base += kThreads) {
        const int b = base + tid;
        Need s{};
        if (b < p.B) s = need_of(p, b);
        if (s.wrong) flags |= ORTHROS_DEV_BAD_LENGTH;
        // an id from outside the pool on the stack would come to another sequence, steps later: one that has
        // such an id among its pages keeps them all
        for (unsigned ends = __ballot_sync(0xffffffffu, s.back > 0); ends; ends &= ends - 1) {
            const int src = __ffs(ends) - 1;
            if (__any_sync(0xffffffffu, foreign_page(p, base + warp * 32 + src, __shfl_sync(0xffffffffu, s.back, src), lane)) && lane == src) {
                s.wrong = true;
                s.ends = false;
                s.back = 0;
                flags |= ORTHROS_DEV_BAD_PAGE;
            }
        }
        long long v[3] = {s.rows, s.lack, s.back};
#pragma unroll
        for (int k = 0; k < 3; ++k) {
            v[k] = warp_scan(v[k], lane);
            if (lane == 31) wsum[k][warp] = v[k];
        }
        __syncthreads();
        if (warp < 3) wsum[warp][lane] = warp_scan(wsum[warp][lane], lane);
        __syncthreads();
#pragma unroll
        for (int k = 0; k < 3; ++k) v[k] += carry[k] + (warp ? wsum[k][warp - 1] : 0);
        if (b < p.B) {
            // (held to 32 bits: sums past the tokens or the pool refuse the step below)
            start[b + 1] = (int)min(v[0], 0x7fffffffLL);
            off[b + 1] = (int)min(v[1], 0x7fffffffLL);
            cached[b] = s.wrong ? -1 : s.ends ? 0 : s.cached;
            held[b] = s.ends ? -1 : s.held;
            if (b == 0) start[0] = off[0] = 0;
        }
        // ended sequences' pages go back, the lanes' of a warp one after the other by all of it, the warps
        // shared out over the ranks; nobody reads the stack or these table rows yet
        const long long to = count + v[2] - s.back;
        unsigned gives = __ballot_sync(0xffffffffu, warp % ctas == rank && s.back > 0 && count >= 0 && to + s.back <= p.num_pages);
        for (; gives; gives &= gives - 1) {
            const int src = __ffs(gives) - 1;
            const int n = __shfl_sync(0xffffffffu, s.back, src);
            int32_t *at = p.free_pages + __shfl_sync(0xffffffffu, to, src);
            const int32_t *row = p.block_table + (long long)(base + warp * 32 + src) * p.max_pages;
            constexpr int kPages = 8;  // of a lane at a time, loaded before the first is stored
            for (int i0 = lane; i0 < n; i0 += 32 * kPages) {
                int id[kPages];
#pragma unroll
                for (int u = 0; u < kPages; ++u)
                    if (i0 + 32 * u < n) id[u] = row[i0 + 32 * u];
#pragma unroll
                for (int u = 0; u < kPages; ++u)
                    if (i0 + 32 * u < n) at[i0 + 32 * u] = id[u];
            }
        }
        __syncthreads();
        if (tid < 3) carry[tid] += wsum[tid][kWarps - 1];
        __syncthreads();
    }
    const long long rows = carry[0], avail = count + carry[2];
    // nothing of the step can be: more tokens than rows, or a stack that cannot hold these pages
    const bool none = rows > p.n || count < 0 || avail > p.num_pages;
    if (none) flags |= ORTHROS_DEV_BAD_LENGTH;
    // a sequence whose pages are not all there takes none
    int taken = 0;
    for (int b = tid; b < p.B && !none; b += kThreads) {
        if (cached[b] < 0 || off[b + 1] == off[b]) continue;
        if (off[b + 1] <= avail) {
            taken = off[b + 1];  // (they ascend)
        } else {
            cached[b] = -1;
            flags |= ORTHROS_DEV_NO_PAGES;
        }
    }
    if (taken) atomicMax(&s_taken, taken);
    if (flags) atomicOr(&s_flags, flags);
    // lengths and pages of sequences that change nothing, before they may be written over
    constexpr int kMine = kPlanMaxSeqs / kThreads;
    int len[kMine], own[kMine];
    if (rank == 0) {
#pragma unroll
        for (int k = 0; k < kMine; ++k) {
            const int b = tid + k * kThreads;
            if (b >= p.B) break;
            if (none || cached[b] < 0) len[k] = p.cache_lens[b], own[k] = p.held_in[b];
        }
    }
    __syncthreads();
    taken = s_taken;
    if (rank == 0 && tid == 0) *p.status = s_flags;
    if (ctas > 1) cluster_arrive_wait();
    else __syncthreads();

    // ---- outputs ----
    if (rank == 0) {
#pragma unroll
        for (int k = 0; k < kMine; ++k) {
            const int b = tid + k * kThreads;
            if (b >= p.B) break;
            int kv = -1;
            if (!none && cached[b] >= 0) {
                const bool ends = held[b] < 0;
                kv = len[k] = ends ? 0 : cached[b] + start[b + 1] - start[b];
                own[k] = ends ? 0 : held[b] + off[b + 1] - off[b];
            }
            p.q_indptr[b] = none ? -1 : start[b];
            p.kv_lens[b] = kv;
            p.held_out[b] = own[k];
            if (p.lens_out) p.lens_out[b] = len[k];
        }
        if (tid == 0) {
            p.q_indptr[p.B] = none ? -1 : (int)rows;
            *p.count_out = none ? count : (int)avail - taken;
        }
    }
    const int at0 = rank * kThreads + tid, step = ctas * kThreads;
    auto on_stack = [&](int i) { return __ldcg(p.free_pages + (int)avail - 1 - i); };  // i-th page taken
    uint32_t found = 0;
    for (long long e = at0; e < taken; e += step) {  // (none: taken is 0)
        const int j = (int)e, b = last_at_most(off, p.B, j);
        const int id = on_stack(j);
        if (id < 0 || id >= p.num_pages) found |= ORTHROS_DEV_BAD_PAGE;
        p.block_table[(long long)b * p.max_pages + held[b] + j - off[b]] = id;
    }
    const int real = none ? 0 : (int)rows;
    for (long long e = at0; e < p.n; e += step) {
        const int i = (int)e;
        int seq = -1, pos = 0, slot = -1;
        uint32_t m[kWords > 0 ? kWords : 1];
#pragma unroll
        for (int w = 0; w < kWords; ++w) m[w] = 0;
        if (i < real) {
            const int b = last_at_most(start, p.B, i);
            if (cached[b] >= 0) {
                const int j = i - start[b];
                seq = b;
                pos = cached[b] + j;
                const int pg = pos / p.page_size, in = pos - pg * p.page_size;
                const int id = pg < held[b] ? p.block_table[(long long)b * p.max_pages + pg] : on_stack(off[b] + pg - held[b]);
                if constexpr (kWords > 0) {  // up the tree
                    int at = j, depth = 0;
                    while (true) {
#pragma unroll
                        for (int w = 0; w < kWords; ++w)
                            if (at >> 5 == w) m[w] |= 1u << (at & 31);
                        const int up = __ldg(p.parents + start[b] + at);
                        if (up < -1 || up >= at) found |= ORTHROS_DEV_BAD_POSITION;
                        if (up < 0 || up >= at) break;
                        at = up;
                        ++depth;
                    }
                    pos = cached[b] + depth;
                }
                if (id >= 0 && id < p.num_pages) slot = id * p.page_size + in;
                else found |= ORTHROS_DEV_BAD_PAGE;
            }
        }
        p.token_seq[i] = seq;
        p.token_pos[i] = pos;
        p.token_slots[i] = slot;
#pragma unroll
        for (int w = 0; w < kWords; ++w)
            if (w < p.words) p.tree_mask[(long long)i * p.words + w] = m[w];
    }
    if (found) atomicOr(p.status, found);
}

// ---------------------------------------------------------------------------
// Commit: token acc[i] of sequence b's tree goes from place L + acc[i] to L + i, in every
// layer's keys and values. The path ascends (acc[i] >= i), so a thread that owns 16 bytes of
// the rows may move them in order, kMoves loads in flight before their stores: what a store
// overwrites has been read. A block takes a sequence in one layer or a few,
// its moves laid end to end; one block past the sequences checks all paths and writes the status word, as
// the moving blocks of the first layer write the lengths. Bound by latency: lengths, path, pages and
// rows are four loads that wait for one another. One layer of 32 sequences: 3.4 us; 48 sequences
// in 32 layers (44 MB read and written): 11 us, 60 % of the copy rate, with eight moves in flight
// instead of four 0.9 us more (registers: three blocks an SM). With many places to check (sequences
// times `most`) the status block is the last to end, 256 places a turn: 500 sequences with most = 8
// take 18 us, with most = 64 110 us.
// ---------------------------------------------------------------------------
constexpr int kCommitThreads = 256, kMoves = 4;

struct Path {
    int first, n;  // cached tokens before the tree, accepted ones (0 if the path cannot be)
    bool known;    // the lengths can be: first counts
    uint32_t flags;
};
__device__ __forceinline__ Path path_of(const TreeCommitParams &p, int b) {
    Path a{0, 0, false, 0};
    const int nb = p.q_indptr[b + 1] - p.q_indptr[b], len = p.kv_lens[b], k = p.n_accepted[b];
    if (nb < 0 || len < nb || (long long)len > (long long)p.max_pages * p.page_size) {
        a.flags = ORTHROS_DEV_BAD_LENGTH;
        return a;
    }
    a.first = len - nb;
    a.known = true;
    if (k < 0 || k > p.most || k > nb) {
        a.flags = ORTHROS_DEV_BAD_LENGTH;
        return a;
    }
    a.n = k;
    return a;
}
// Token i of the path: its status bits, and the slots it moves between (long long: a row's bytes follow).
__device__ __forceinline__ uint32_t place_of(const TreeCommitParams &p, int b, const Path &a, int i, long long &from, long long &to) {
    const int32_t *acc = p.accepted + (long long)b * p.most;
    const int nb = p.kv_lens[b] - a.first, x = acc[i];
    from = to = 0;
    if (x < i || x >= nb || (i > 0 && acc[i - 1] >= x)) return ORTHROS_DEV_BAD_POSITION;
    const int32_t *bt = p.block_table + (long long)b * p.max_pages;
    const int s = a.first + x, t = a.first + i;
    const int ps = bt[s / p.page_size], pt = bt[t / p.page_size];
    if (ps < 0 || ps >= p.num_pages || pt < 0 || pt >= p.num_pages) return ORTHROS_DEV_BAD_PAGE;
    from = (long long)ps * p.page_size + s % p.page_size;
    to = (long long)pt * p.page_size + t % p.page_size;
    return 0;
}

__global__ void __launch_bounds__(kCommitThreads) tree_commit_kernel(const TreeCommitParams p) {
    __shared__ long long from[kTreeMaxTokens], to[kTreeMaxTokens];
    const int tid = threadIdx.x, b = blockIdx.x;
    const int layer0 = blockIdx.y * p.layers_per_block, layers = min(p.layers_per_block, p.layers - layer0);
    if (b == p.B) {  // the status word
        if (layer0 > 0) return;
        uint32_t flags = 0;
        const long long places = (long long)p.B * p.most;
#pragma unroll 4
        for (long long e = tid; e < places; e += kCommitThreads) {
            const int s = (int)(e / p.most), i = (int)(e % p.most);
            const Path a = path_of(p, s);
            flags |= a.flags;
            long long x, y;
            if (i < a.n) flags |= place_of(p, s, a, i, x, y);
        }
        uint32_t all = 0;
#pragma unroll
        for (uint32_t bit = ORTHROS_DEV_BAD_POSITION; bit <= ORTHROS_DEV_BAD_LENGTH; bit <<= 1)
            if (__syncthreads_or(flags & bit)) all |= bit;
        if (tid == 0) *p.status = all;
        return;
    }
    const Path a = path_of(p, b);
    uint32_t wrong = a.flags;
    for (int i = tid; i < a.n; i += kCommitThreads) wrong |= place_of(p, b, a, i, from[i], to[i]);
    wrong = __syncthreads_or(wrong);
    if (layer0 == 0 && tid == 0 && a.known) p.cache_lens[b] = a.first + (wrong ? 0 : a.n);
    if (wrong) return;  // nothing of this sequence moves
    const int chunks = p.row_bytes / 16;
    const long long pool = (long long)p.num_pages * p.page_size * p.row_bytes;
    for (int c = tid; c < 2 * chunks; c += kCommitThreads) {
        uint8_t *at = (c < chunks ? p.k_cache : p.v_cache) + layer0 * pool + (c < chunks ? c : c - chunks) * 16LL;
        // (a batch may span layers: their moves do not touch one another)
        int i = 0, left = layers * a.n;
        while (left > 0) {
            uint4 r[kMoves];
            uint8_t *dst[kMoves];
#pragma unroll
            for (int u = 0; u < kMoves; ++u) {
                dst[u] = nullptr;
                if (u < left) {
                    if (from[i] != to[i]) {
                        r[u] = *reinterpret_cast<const uint4 *>(at + from[i] * p.row_bytes);
                        dst[u] = at + to[i] * p.row_bytes;
                    }
                    if (++i == a.n) i = 0, at += pool;
                }
            }
#pragma unroll
            for (int u = 0; u < kMoves; ++u)
                if (dst[u]) *reinterpret_cast<uint4 *>(dst[u]) = r[u];
            left -= kMoves;
        }
    }
}

}  // namespace

cudaError_t launch_step_plan(const StepPlanParams &p, cudaStream_t stream) {
    const auto kernel = p.words == 0 ? step_plan_kernel<0> : p.words <= 2 ? step_plan_kernel<2> : step_plan_kernel<kTreeMaxTokens / 32>;
    static SmemLimit limit[3];
    const int which = p.words == 0 ? 0 : p.words <= 2 ? 1 : 2;
    auto bytes = [](int B) { return (4 * B + 2) * (int)sizeof(int); };
    if (cudaError_t e = limit[which].ensure((const void *)kernel, bytes(kPlanMaxSeqs)); e != cudaSuccess) return e;
    int ctas = 1;  // CTAs of the cluster: 1024 tokens each, up to the portable eight
    while (ctas < kMaxCluster && p.n > ctas * kThreads) ctas *= 2;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = ctas;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(ctas);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = bytes(p.B);
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, p);
}

cudaError_t launch_tree_commit(TreeCommitParams p, cudaStream_t stream) {
    // eight blocks an SM, five of which run at once (five an SM: 48 sequences x 32 layers 1.1 us longer)
    const int fit = 8 * device_sm_count();
    p.layers_per_block = (int)(((long long)p.layers * p.B + fit - 1) / fit);
    if (p.layers_per_block > p.layers) p.layers_per_block = p.layers;
    const int groups = (p.layers + p.layers_per_block - 1) / p.layers_per_block;
    tree_commit_kernel<<<dim3(p.B + 1, groups), kCommitThreads, 0, stream>>>(p);
    return cudaGetLastError();
}

}  // namespace orthros
