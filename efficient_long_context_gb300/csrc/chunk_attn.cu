// chunk_attn.cu -- attention of new tokens over a paged cache that already
// holds their keys: one token per sequence (decoding), chunks of a prompt, or
// both mixed, on the tensor cores (tcgen05, TMEM, TMA).
//
// What it computes. Token i of a sequence's n_b new ones sits at position
// t = kv_len - n_b + i and sees keys max(0, t - w + 1) .. t:
//   o = sum_j p_j v_j / l,  p_j = exp(scale q.k_j - m),  l = sum_j p_j,
// one pass over the keys with a running maximum m and sum l per row.
//
// Rows. The g query heads that share a kv head are rows of one product: a
// 128-row tile holds 128 / g consecutive tokens, all their g heads (row = token
// * g + head), so a key/value tile staged once serves g times as many rows and a
// decoding token fills g rows instead of one.
//
// Units and the split of the key axis. A unit is up to two row tiles of one
// sequence and the key tiles (128 tokens) they see. The plan kernel lists the
// units with the running count of their key tiles (at most 32 units are listed by
// every CTA itself); all kv heads have the same list. The CTAs form lanes = gcd(Hkv, CTAs) lanes; lane c % lanes serves kv
// heads c % lanes, + lanes, ..., and its CTAs cut the lane's key tiles, laid end
// to end, into equal shares. So every CTA gets the same number of key tiles
// whatever the batch looks like, a long history of one sequence is spread over
// the whole GPU, and neighbouring CTAs (one per lane) read the same token rows
// of the cache at the same time. A unit cut by a share's border leaves partials
// (m, l, unnormalised o; fp32) that the merge kernel joins; a CTA has at most
// two of those, so the workspace does not grow with the batch.
//
// Two ways through a unit. With two row tiles, slot s works on row tile s and
// both read each key tile. With one (decoding and short chunks), both slots work
// on the same rows, slot s on every second key tile, with accumulators of their
// own that the epilogue adds up, so that the softmax of one tile still runs
// beside the products of the other.
//
// Roles (352 threads, one persistent CTA per SM): warps 0-7 softmax (slot w >> 2,
// one thread per row), warp 8 copies (page lookups by its lanes, TMA boxes of
// up to 128 tokens within a page), warp 9 issues tcgen05.mma, warp 10 clears value
// rows that no row of the unit sees. S = Q K^T (bf16,
// M = 128, N = 128) goes to TMEM, P returns there as bf16 over S, O += P V. TMEM:
// S0 [0,128) S1 [128,256) O0 [256,256+d) O1 [384,384+d).
//
// Precision: products of bf16 values accumulate in fp32; m, l and o are fp32;
// P is rounded to bf16 for the product with V (the sum l takes it unrounded),
// at most half a bf16 step of each term; over the keys of a row that is 0.0015 of o
// (relative, measured with independent values), beside 0.0017 of o's own rounding.
//
// Bound and measured (GQA 32/8, d = 128): decoding by HBM, 32 sequences over 16K-32K
// keys in 480 us, 6.6 TB/s, 97 % of the measured copy rate; chunks by the softmax that
// has to run beside the products, 2 x 4000 tokens over 24K keys at 1484 TFLOP/s (76 %
// of the measured bf16 rate; 1375 once the power limit lowers the clock), 2048
// tokens at window 4096 in 110 us, 5 of them the merge.
//
// Keys outside the sequence's length or before every row's window are never
// read into a result: their copy boxes are skipped (zero fill), their logits
// replaced by -inf and, where a page reaches past them, their value rows
// cleared in shared memory, so whatever a stale page holds does not matter.
#include "ptx.cuh"

namespace orthros {

using namespace ptx;

namespace {

constexpr int kRows = 128;  // rows of a tile
constexpr int kKeys = 128;  // keys of a tile
constexpr int kSoftmaxWarps = 8, kCopyWarp = 8, kMmaWarp = 9, kClearWarp = 10;
constexpr int kThreads = 352;
// At most three of the eleven warps sit on a scheduler: 168 registers a thread
// fit (3 x 32 x 168 of 16K), so the bound is taken for 384 threads.
constexpr int kBound = 384;
constexpr int kFlagRing = 16;
// A share of fewer key tiles than this is not worth a CTA of its own.
constexpr int kMinTiles = 2;

template <int D> struct Cfg {
    static constexpr int kNumK = D == 128 ? 3 : 6, kNumV = D == 128 ? 2 : 4;  // stages: 160 KB in flight
    static constexpr int kSub = D / 64;             // 128-byte swizzle atoms per row
    static constexpr int kTile = kRows * D * 2;     // one 128 x D bf16 tile
    static constexpr int kQ0 = 0;
    static constexpr int kK0 = 2 * kTile;
    static constexpr int kV0 = kK0 + kNumK * kTile;
    static constexpr int kMeta = kV0 + kNumV * kTile;
    static constexpr int kSmem = kMeta + 2048 + 1024;  // + alignment slack
    static constexpr int kTmemO = 256;
};

// One run of key tiles of one unit, as the roles need it.
struct Segment {
    int end;                 // no more segments
    int b, kv, tok0, cnt;    // sequence, kv head, first token and tokens of the unit
    int pos0;                // position of the unit's first token
    int kt0, nkt;            // key tiles kt0 .. kt0 + nkt - 1
    int pair;                // two row tiles (else both slots share one)
    int partial;             // partial index, or -1: the unit is complete here
    int lo[2], hi[2];        // pair: tiles of the run that slot s works on (lo > hi: none)
};

constexpr int kSegRing = 2;

constexpr int kMaxK = 6, kMaxV = 4;
struct Meta {
    uint64_t k_full[kMaxK], k_empty[kMaxK], v_full[kMaxV], v_empty[kMaxV];
    uint64_t q_full[2], q_empty[2];
    uint64_t ve_full[kMaxV];  // a value tile with unseen rows arrived: warp 10 clears them, then completes v_full
    uint64_t s_full[2], o_free[2];
    uint64_t p_half[2], p_full[2];  // the first 64 keys of a P tile are stored (and O rescaled); all are
    uint64_t o_full[2];  // slot s's O complete, for slot s's threads
    uint64_t ox_full;    // slot 1's O of a shared row tile complete, for slot 0's threads
    uint64_t ml_full, ml_free;
    uint64_t g_full[kSegRing], g_empty[kSegRing];
    uint64_t mma_done;
    uint32_t tmem_base;
    int abort;
    volatile int bad[kFlagRing];  // per key tile (running count): its keys [bad >> 8, bad & 255) had page ids outside the pool
    Segment seg[kSegRing];
    float2 ml[kRows];             // slot 1's running max and sum, for slot 0 (shared row tile)
};
static_assert(sizeof(Meta) <= 2048, "barriers and metadata must fit their shared-memory region");

__device__ __forceinline__ void tma_load_5d(void *smem_dst, const CUtensorMap *map, uint64_t *bar, int c0, int c1, int c2,
                                            int c3, int c4) {
    asm volatile(
        "cp.async.bulk.tensor.5d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %4, %5, %6, %7}], [%2];" ::"r"(smem_u32(smem_dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(c4)
        : "memory");
}

// The products are issued under a predicate by a whole warp rather than inside a
// one-lane branch: warp-uniform descriptors stay in uniform registers.
template <typename T> __device__ __forceinline__ T uniform(T x) { return __shfl_sync(0xffffffffu, x, 0); }
__device__ __forceinline__ uint32_t elect_one() {
    uint32_t e;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(e));
    return e;
}
__device__ __forceinline__ void mma_ss_if(uint32_t el, uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
    asm volatile(
        "{\n\t.reg .pred p, e;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "setp.ne.b32 e, %5, 0;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(acc), "r"(el)
        : "memory");
}
__device__ __forceinline__ void mma_ts_if(uint32_t el, uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
    asm volatile(
        "{\n\t.reg .pred p, e;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "setp.ne.b32 e, %5, 0;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
        "r"(a), "l"(b), "r"(idesc), "r"(acc), "r"(el)
        : "memory");
}
__device__ __forceinline__ void tc_commit_if(uint32_t el, uint64_t *bar) {
    asm volatile(
        "{\n\t.reg .pred e;\n\tsetp.ne.b32 e, %1, 0;\n\t"
        "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(smem_u32(bar)),
        "r"(el)
        : "memory");
}

__device__ __forceinline__ void st_global_32b(void *dst, const uint32_t (&w)[8]) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(dst), "r"(w[0]), "r"(w[1]), "r"(w[2]),
                 "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                 : "memory");
}

__device__ __forceinline__ void reg_fence(uint32_t (&r)[32]) {
    asm volatile(""
                 : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]),
                   "+r"(r[7]), "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]),
                   "+r"(r[14]), "+r"(r[15]), "+r"(r[16]), "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]),
                   "+r"(r[21]), "+r"(r[22]), "+r"(r[23]), "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]),
                   "+r"(r[28]), "+r"(r[29]), "+r"(r[30]), "+r"(r[31]));
}

// Key and value tiles lie in groups of 8 tokens, a 1 KB swizzle atom of 64 channels
// after the other within a group, so that one copy box brings whole rows of any
// multiple of 8 tokens. Byte offset of (token, 16-byte chunk c):
template <int D> __device__ __forceinline__ uint32_t kv_offset(int row, int c) {
    return (row >> 3) * (D * 16) + (c >> 3) * 1024 + (row & 7) * 128 + (((c & 7) ^ (row & 7)) << 4);
}

// Token of a row within its tile: row / g for rows and groups up to 128.
__device__ __forceinline__ int row_token(const ChunkParams &p, int row) { return row * p.g_inv >> 16; }

// Key tiles a run of tokens at positions [first, last] sees.
__device__ __forceinline__ void key_tiles(int first, int last, int window, int &lo, int &hi) {
    lo = max(0, first - window + 1) / kKeys;
    hi = last / kKeys;
}

// What a row's output is scaled by. Every row sees a key (its own), so a sum that is 0 had
// only logits of -inf: such a row has no softmax and is NaN, as is one whose sum is.
__device__ __forceinline__ float inverse_sum(float l) { return l > 0.f ? 1.f / l : __int_as_float(0x7fc00000); }

// New tokens of a sequence that has nb of them among len in the cache, or 0 when there
// are none or its lengths are impossible (wrong).
__device__ __forceinline__ int new_tokens(const ChunkParams &p, int nb, int len, bool &wrong) {
    wrong = nb > 0 && (nb > p.max_new || len < nb || (long long)len > (long long)p.max_pages * p.page_size);
    return wrong ? 0 : nb;
}

// The same for sequence b: its first row of q and cached tokens.
__device__ __forceinline__ int new_tokens(const ChunkParams &p, int b, int &tok0, int &len, bool &wrong) {
    tok0 = p.q_indptr[b];
    len = p.kv_lens[b];
    return new_tokens(p, p.q_indptr[b + 1] - tok0, len, wrong);
}

// The unit that begins at token i of a sequence's nb (i < nb).
__device__ __forceinline__ ChunkUnit unit_at(const ChunkParams &p, int b, int tok0, int nb, int len, int i) {
    ChunkUnit u;
    u.b = b;
    u.tok0 = tok0 + i;
    u.cnt = min(2 * p.tile_tokens, nb - i);
    u.pos0 = len - nb + i;
    int hi;
    key_tiles(u.pos0, u.pos0 + u.cnt - 1, p.window, u.kt_lo, hi);
    u.n_kt = hi - u.kt_lo + 1;
    u.start = 0;
    return u;
}

// ---------------------------------------------------------------------------
// Plan: one block. Checks the lengths, lists the units and their key tiles.
// ---------------------------------------------------------------------------
constexpr int kPlanThreads = 1024;

__device__ __forceinline__ long long warp_scan(long long v, int lane) {  // inclusive
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long u = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o) v += u;
    }
    return v;
}

__device__ void fill_nan(const ChunkParams &p, long long tok0, long long tok1, int d, int tid, int nthreads) {
    const long long e0 = tok0 * p.Hq * d, e1 = tok1 * p.Hq * d;
    for (long long i = e0 + tid; i < e1; i += nthreads) p.o[i] = __float2bfloat16_rn(__int_as_float(0x7fc00000));
    if (p.lse)
        for (long long i = tok0 * p.Hq + tid; i < tok1 * p.Hq; i += nthreads) p.lse[i] = __int_as_float(0x7fc00000);
}

__global__ void __launch_bounds__(kPlanThreads) chunk_plan_kernel(const ChunkParams p, int d) {
    __shared__ long long wsum[2][32];
    __shared__ long long carry[2];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    if (tid == 0) {
        p.plan->flags = 0;
        carry[0] = carry[1] = 0;
    }
    int bad = 0;
    for (int b = tid; b < p.B; b += kPlanThreads) bad |= p.q_indptr[b + 1] < p.q_indptr[b];
    if (tid == 0) bad |= p.q_indptr[0] != 0 || p.q_indptr[p.B] != p.n;
    if (__syncthreads_or(bad)) {  // no token's sequence is known
        if (tid == 0) *p.plan = ChunkPlan{0, ORTHROS_DEV_BAD_LENGTH, 0};
        fill_nan(p, 0, p.n, d, tid, kPlanThreads);
        return;
    }
    const int ut = 2 * p.tile_tokens;
    for (int b = warp; b < p.B; b += kPlanThreads / 32) {
        int tok0, len;
        bool wrong;
        const int nb = new_tokens(p, b, tok0, len, wrong);
        if (wrong) {
            if (lane == 0) set_status(&p.plan->flags, ORTHROS_DEV_BAD_LENGTH);
            fill_nan(p, tok0, p.q_indptr[b + 1], d, lane, 32);
        }
        long long tiles = 0;
        for (int i = lane * ut; i < nb; i += 32 * ut) tiles += unit_at(p, b, tok0, nb, len, i).n_kt;
        tiles = warp_scan(tiles, lane);
        if (lane == 31) {
            p.seq_units[b] = (nb + ut - 1) / ut;
            p.seq_tiles[b] = tiles;
        }
    }
    __syncthreads();
    // exclusive prefix sums over the sequences, 1024 at a time
    for (int base = 0; base < p.B; base += kPlanThreads) {
        const int b = base + tid;
        const long long u = b < p.B ? p.seq_units[b] : 0, t = b < p.B ? p.seq_tiles[b] : 0;
        long long su = warp_scan(u, lane), st = warp_scan(t, lane);
        if (lane == 31) {
            wsum[0][warp] = su;
            wsum[1][warp] = st;
        }
        __syncthreads();
        if (warp == 0) {
            wsum[0][lane] = warp_scan(wsum[0][lane], lane);
            wsum[1][lane] = warp_scan(wsum[1][lane], lane);
        }
        __syncthreads();
        su += carry[0] + (warp ? wsum[0][warp - 1] : 0);
        st += carry[1] + (warp ? wsum[1][warp - 1] : 0);
        if (b < p.B) {
            p.seq_units[b] = (int)(su - u);
            p.seq_tiles[b] = st - t;
        }
        __syncthreads();
        if (tid == 0) {
            carry[0] += wsum[0][31];
            carry[1] += wsum[1][31];
        }
        __syncthreads();
    }
    if (tid == 0) {
        p.plan->units = (int)carry[0];
        p.plan->tiles = carry[1];
    }
    for (int b = warp; b < p.B; b += kPlanThreads / 32) {
        int tok0, len;
        bool wrong;
        const int nb = new_tokens(p, b, tok0, len, wrong);
        const int u0 = p.seq_units[b];
        long long at = p.seq_tiles[b];
        for (int i0 = 0; i0 < nb; i0 += 32 * ut) {
            const int i = i0 + lane * ut;
            ChunkUnit u{};
            if (i < nb) u = unit_at(p, b, tok0, nb, len, i);
            const long long sum = warp_scan(u.n_kt, lane);
            u.start = at + sum - u.n_kt;
            if (i < nb) p.units[u0 + i / ut] = u;
            at += __shfl_sync(0xffffffffu, sum, 31);
        }
    }
}

// ---------------------------------------------------------------------------
// Main kernel
// ---------------------------------------------------------------------------
// The shares of a lane: `total` key tiles over `eff` CTAs, equal up to borders that
// move to a unit's end within kSnap key tiles (a quarter of a share at most): a
// cut costs two partial epilogues and a merge, as much as a few tiles.
constexpr int kSnap = 3;
struct Shares {
    long long total;
    int eff, snap;
    __device__ long long border(int j) const {  // before it moves
        // (a 64-bit division takes the copy warp, which starts with two, half a microsecond)
        if (total * eff <= 0xffffffffLL) return (uint32_t)total * (uint32_t)j / (uint32_t)eff;
        return total * j / eff;
    }
    // border x, which falls into the unit [u0, u0 + n), where it ends up
    __device__ long long moved(long long x, long long u0, int n) const {
        return x - u0 <= snap ? u0 : u0 + n - x <= snap ? u0 + n : x;
    }
};
__device__ __forceinline__ Shares shares_of(const ChunkParams &p, const ChunkPlan &pl) {
    Shares s;
    s.total = (long long)(p.Hkv / p.lanes) * pl.tiles;
    s.eff = (int)max(1LL, min((long long)p.per_lane, s.total / kMinTiles));
    s.snap = 0;  // the largest with 4 snap eff <= total, up to kSnap
    while (s.snap < kSnap && 4LL * (s.snap + 1) * s.eff <= s.total) ++s.snap;
    return s;
}

// Last unit whose start is <= x (all 32 lanes; units are sorted by start).
__device__ int find_unit(const ChunkUnit *units, int n, long long x, int lane) {
    int lo = 0, len = n;
    while (len > 1) {
        const int step = (len + 31) / 32;
        const int i = lo + lane * step;
        const bool le = i < lo + len && units[i].start <= x;
        const int k = 31 - __clz(__ballot_sync(0xffffffffu, le));  // lane 0 always holds
        const int at = k * step;
        lo += at;
        len = min(step, len - at);
    }
    return lo;
}

// Whether key tile `it` of a segment has rows that none of its unit's tokens sees:
// all but rows [r0, r1).
__device__ __forceinline__ bool unseen_rows(const Segment &sg, int window, int it, int &r0, int &r1) {
    const int key0 = (sg.kt0 + it) * kKeys;
    r0 = max(0, max(0, sg.pos0 - window + 1) - key0);  // (in this order: a window may be INT_MAX)
    r1 = min(kKeys, sg.pos0 + sg.cnt - key0);
    return r0 > 0 || r1 < kKeys;
}

template <int D>
__global__ void __launch_bounds__(kBound, 1)
    chunk_attn_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                      const __grid_constant__ CUtensorMap tm_v, const ChunkParams p) {
    using C = Cfg<D>;
    constexpr int kNumK = C::kNumK, kNumV = C::kNumV;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    Meta &mt = *reinterpret_cast<Meta *>(smem + C::kMeta);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    volatile int *abort = &mt.abort;
    const int g = p.Hq / p.Hkv;
    const int tt = p.tile_tokens;
    uint32_t *status = &p.heads[blockIdx.x].flags;  // this CTA's; the merge collects them

    if (tid == 0) {
        *status = 0;
        for (int i = 0; i < kNumK; ++i) {
            mbar_init(&mt.k_full[i], 1);
            mbar_init(&mt.k_empty[i], 1);
        }
        for (int i = 0; i < kNumV; ++i) {
            mbar_init(&mt.v_full[i], 1);
            mbar_init(&mt.v_empty[i], 1);
            mbar_init(&mt.ve_full[i], 1);
        }
        for (int s = 0; s < 2; ++s) {
            mbar_init(&mt.q_full[s], 1);
            mbar_init(&mt.q_empty[s], 1);
            mbar_init(&mt.s_full[s], 1);
            mbar_init(&mt.p_half[s], kRows);
            mbar_init(&mt.p_full[s], kRows);
            mbar_init(&mt.o_full[s], 1);
            mbar_init(&mt.o_free[s], kRows);
        }
        mbar_init(&mt.ox_full, 1);
        mbar_init(&mt.ml_full, kRows);
        mbar_init(&mt.ml_free, kRows);
        for (int r = 0; r < kSegRing; ++r) {
            mbar_init(&mt.g_full[r], 1);
            mbar_init(&mt.g_empty[r], kSoftmaxWarps + 2);
        }
        mbar_init(&mt.mma_done, 1);
        mt.abort = 0;
        fence_mbar_init();
    }
    if (warp == kCopyWarp && lane == 0) {
        prefetch_tmap(&tm_q);
        prefetch_tmap(&tm_k);
        prefetch_tmap(&tm_v);
    }
    if (warp == kMmaWarp) {
        tmem_alloc(&mt.tmem_base, 512);
        tmem_relinquish();
    }
    // lengths of the sequence that this lane of the copy warp lists (no plan: no launch to wait for)
    int tok0 = 0, tok1 = 0, len = 0, tok_first = 0, tok_last = p.n;
    if (warp == kCopyWarp && p.direct) {
        const int b = p.B == 1 ? 0 : lane;
        if (b < p.B) tok0 = p.q_indptr[b], tok1 = p.q_indptr[b + 1], len = p.kv_lens[b];
        tok_first = p.q_indptr[0], tok_last = p.q_indptr[p.B];
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = mt.tmem_base;
    // the merge may be launched; the plan's kernel, where there is one, must have finished
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");

    if (warp == kCopyWarp) {
        // ---------------- segments and copies ----------------
        // The batch's units: from the plan, or, when there are at most 32 (one per
        // sequence, or those of a single sequence), one per lane of this warp.
        ChunkPlan pl;
        ChunkUnit own{};
        if (p.direct) {
            const int ut = 2 * tt;
            const bool one = p.B == 1;  // lane = unit of the sequence, else lane = sequence
            const int b = one ? 0 : lane;
            bool wrong;
            const int nb = new_tokens(p, tok1 - tok0, len, wrong);
            const bool order = __all_sync(0xffffffffu, tok1 >= tok0 && tok_first == 0 && tok_last == p.n);
            if (!order || __any_sync(0xffffffffu, wrong)) {
                // impossible lengths: NaN for their rows, or for all rows when no token's sequence is known
                if (lane == 0 && blockIdx.x == 0) set_status(status, ORTHROS_DEV_BAD_LENGTH);
                for (int k = 0; k < (one || !order ? 1 : p.B); ++k) {
                    if (order && !__shfl_sync(0xffffffffu, (int)wrong, k)) continue;
                    fill_nan(p, order ? p.q_indptr[k] : 0, order ? p.q_indptr[k + 1] : p.n, D,
                             (int)blockIdx.x * 32 + lane, (int)gridDim.x * 32);
                }
            }
            const int i = one ? lane * ut : 0;
            if (order && i < nb) own = unit_at(p, b, tok0, nb, len, i);
            const long long sum = warp_scan(own.n_kt, lane);
            own.start = sum - own.n_kt;
            pl.units = 32;
            pl.tiles = __shfl_sync(0xffffffffu, sum, 31);
        } else {
            pl = *p.plan;
        }
        auto get_unit = [&](int u) -> ChunkUnit {
            if (!p.direct) return p.units[u];
            ChunkUnit r;
            r.b = __shfl_sync(0xffffffffu, own.b, u);
            r.tok0 = __shfl_sync(0xffffffffu, own.tok0, u);
            r.cnt = __shfl_sync(0xffffffffu, own.cnt, u);
            r.pos0 = __shfl_sync(0xffffffffu, own.pos0, u);
            r.kt_lo = __shfl_sync(0xffffffffu, own.kt_lo, u);
            r.n_kt = __shfl_sync(0xffffffffu, own.n_kt, u);
            r.start = __shfl_sync(0xffffffffu, own.start, u);
            return r;
        };
        // unit that holds key tile x of the list
        auto find = [&](long long x) -> int {
            if (!p.direct) return find_unit(p.units, pl.units, x, lane);
            return 31 - __clz(__ballot_sync(0xffffffffu, own.n_kt > 0 && own.start <= x));
        };
        const int ln = blockIdx.x % p.lanes, j = blockIdx.x / p.lanes;
        ChunkHead head{};
        long long head_u0 = 0;  // first key tile and key tiles of the unit it names
        int head_n = 0;
        uint32_t gk = 0, gv = 0;  // key and value copies issued
        uint32_t nq[2] = {0, 0};  // query tiles issued per slot
        int ring = 0;
        bool alive = true;
        auto publish = [&](const Segment &sg) -> bool {
            const int r = ring % kSegRing;
            if (ring >= kSegRing && !mbar_wait_warp(&mt.g_empty[r], ((ring / kSegRing) - 1) & 1, abort, status))
                return false;
            if (lane == 0) {
                mt.seg[r] = sg;
                mbar_arrive(&mt.g_full[r]);
            }
            __syncwarp();
            ++ring;
            return true;
        };
        if (pl.tiles > 0) {
            const Shares sh = shares_of(p, pl);
            if (j < sh.eff) {
                // both borders of the share, moved, the end first (one body for both: this code runs
                // once, from a cold instruction cache); the unit that it begins with
                long long x = 0, x1 = 0;
                int kvo = 0, u = 0;  // which of the lane's kv heads (few: counted, not divided), unit
                bool past = false;
#pragma unroll 1
                for (int k = 1; k >= 0; --k) {
                    x1 = x;
                    x = sh.border(j + k);
                    if (x >= sh.total) continue;  // the lane's end stays
                    kvo = 0;
                    while (x >= (kvo + 1) * pl.tiles) ++kvo;
                    u = find(x - kvo * pl.tiles);
                    const ChunkUnit e = get_unit(u);
                    const long long u0 = kvo * pl.tiles + e.start;
                    x = sh.moved(x, u0, e.n_kt);
                    past = x == u0 + e.n_kt;
                }
                auto next_unit = [&]() {  // (a lane without a unit is passed over)
                    do {
                        if (++u == pl.units) {
                            u = 0;
                            ++kvo;
                        }
                    } while (p.direct && __shfl_sync(0xffffffffu, own.n_kt, u) == 0);
                };
                if (past) next_unit();
                while (x < x1 && alive) {
                    const ChunkUnit un = get_unit(u);
                    const int a = (int)(x - kvo * pl.tiles - un.start);
                    const int n_tiles = (int)min((long long)(un.n_kt - a), x1 - x);
                    Segment sg;
                    sg.end = 0;
                    sg.b = un.b;
                    sg.kv = ln + kvo * p.lanes;
                    sg.tok0 = un.tok0;
                    sg.cnt = un.cnt;
                    sg.pos0 = un.pos0;
                    sg.kt0 = un.kt_lo + a;
                    sg.nkt = n_tiles;
                    sg.pair = un.cnt > tt;
                    const bool starts = a == 0, ends = a + n_tiles == un.n_kt;
                    sg.partial = starts && ends ? -1 : 2 * (int)blockIdx.x + (starts ? 1 : 0);
                    if (starts && !ends) {
                        head_u0 = x;
                        head_n = un.n_kt;
                        head.tok0 = un.tok0;
                        head.cnt = un.cnt;
                        head.kv = sg.kv;
                    }
#pragma unroll
                    for (int s = 0; s < 2; ++s) {
                        int lo = 0, hi = n_tiles - 1;
                        if (sg.pair) {
                            const int c0 = s * tt, c1 = s ? un.cnt : tt;
                            int kl, kh;
                            key_tiles(un.pos0 + c0, un.pos0 + c1 - 1, p.window, kl, kh);
                            lo = max(lo, kl - sg.kt0);
                            hi = min(hi, kh - sg.kt0);
                        }
                        sg.lo[s] = lo;
                        sg.hi[s] = hi;
                    }
                    if (!(alive = publish(sg))) break;
                    // query tiles (rows past the tile's tokens keep whatever was there: their results are dropped)
                    for (int s = 0; alive && s < (sg.pair ? 2 : 1); ++s) {
                        if (nq[s] > 0 && !mbar_wait_warp(&mt.q_empty[s], (nq[s] - 1) & 1, abort, status)) {
                            alive = false;
                            break;
                        }
                        if (lane == 0) {
                            mbar_arrive_expect_tx(&mt.q_full[s], C::kSub * 128 * g * tt);
                            for (int h = 0; h < C::kSub; ++h)
                                tma_load_3d(smem + C::kQ0 + s * C::kTile + h * (kRows * 128), &tm_q, &mt.q_full[s],
                                            64 * h, sg.kv * g, sg.tok0 + s * tt);
                        }
                        __syncwarp();
                        ++nq[s];
                    }
                    if (!alive) break;
                    // key/value tiles: keys [key_lo, key_hi] exist for this unit
                    const int32_t *bt = p.block_table + (long long)sg.b * p.max_pages;
                    const int key_hi = un.pos0 + un.cnt - 1;
                    const int key_lo = max(0, un.pos0 - p.window + 1);
                    const int oob = p.num_pages * p.page_size;  // past the pool: the copy fills zeros
                    const int box = p.box;
                    const int n_box = box ? kKeys / box : 0;
                    // first token row of this lane's box of a tile (TMA), or oob; bad: page id outside the pool
                    // (The page is awaited here, a tile before its use: awaited at its use, decoding took 1 %
                    // longer, its copies less in step with those of the other heads.)
                    auto look = [&](int kt, int &bad) -> int {
                        bad = 0;
                        if (lane >= n_box) return oob;
                        const int key = kt * kKeys + lane * box;
                        if (key > key_hi || key + box - 1 < key_lo) return oob;
                        const int pg = bt[key / p.page_size];
                        if (pg < 0 || pg >= p.num_pages) {
                            bad = 1;
                            return oob;
                        }
                        return pg * p.page_size + key % p.page_size;
                    };
                    int bad_next = 0, tok_next = look(sg.kt0, bad_next);
                    for (int it = 0; it < sg.nkt; ++it) {
                        const uint32_t gi = gk;
                        const int sk = gi % kNumK, sv = gi % kNumV;
                        const int tok = tok_next, bad = bad_next;
                        if (it + 1 < sg.nkt) tok_next = look(sg.kt0 + it + 1, bad_next);
                        if (gi >= (uint32_t)kNumK &&
                            !mbar_wait_warp(&mt.k_empty[sk], ((gi / kNumK) - 1) & 1, abort, status)) {
                            alive = false;
                            break;
                        }
                        uint8_t *ks = smem + C::kK0 + sk * C::kTile, *vs = smem + C::kV0 + sv * C::kTile;
                        if (box) {
                            const unsigned wrong = __ballot_sync(0xffffffffu, bad);
                            if (lane == 0) {
                                if (wrong) set_status(status, ORTHROS_DEV_BAD_PAGE);
                                mt.bad[gi % kFlagRing] = wrong ? (__ffs(wrong) - 1) * box << 8 | (32 - __clz(wrong)) * box : 0;
                                mbar_arrive_expect_tx(&mt.k_full[sk], C::kTile);
                            }
                            __syncwarp();
                            if (lane < n_box)
                                tma_load_5d(ks + lane * box * D * 2, &tm_k, &mt.k_full[sk], 0, 0, 0, tok >> 3, sg.kv);
                            if (gi >= (uint32_t)kNumV &&
                                !mbar_wait_warp(&mt.v_empty[sv], ((gi / kNumV) - 1) & 1, abort, status)) {
                                ++gk;
                                alive = false;
                                break;
                            }
                            int r0, r1;
                            const bool edge = unseen_rows(sg, p.window, it, r0, r1);
                            uint64_t *full = edge ? &mt.ve_full[sv] : &mt.v_full[sv];
                            if (lane == 0) mbar_arrive_expect_tx(full, C::kTile);
                            __syncwarp();
                            if (lane < n_box)
                                tma_load_5d(vs + lane * box * D * 2, &tm_v, full, 0, 0, 0, tok >> 3, sg.kv);
                            ++gv;
                        } else {
                            // page sizes without a copy box: the lanes gather the rows, 16 bytes at a time
                            if (gi >= (uint32_t)kNumV &&
                                !mbar_wait_warp(&mt.v_empty[sv], ((gi / kNumV) - 1) & 1, abort, status)) {
                                alive = false;
                                break;
                            }
                            unsigned bad0 = kKeys, bad1 = 0;  // first and past the last key without a page
                            constexpr int kCh = D / 8;
                            for (int e = lane; e < kRows * kCh; e += 32) {
                                const int row = e / kCh, c = e % kCh;
                                const int key = (sg.kt0 + it) * kKeys + row;
                                long long src = -1;
                                if (key >= key_lo && key <= key_hi) {
                                    const int pg = bt[key / p.page_size];
                                    if (pg < 0 || pg >= p.num_pages) bad0 = min(bad0, (unsigned)row), bad1 = max(bad1, (unsigned)row + 1);
                                    else src = (((long long)pg * p.page_size + key % p.page_size) * p.Hkv + sg.kv) * D + 8 * c;
                                }
                                const uint32_t dk = smem_u32(ks + kv_offset<D>(row, c)), dv = smem_u32(vs + kv_offset<D>(row, c));
                                const uint32_t bytes = src >= 0 ? 16 : 0;  // 0: zero fill
                                const __nv_bfloat16 *a = p.k + max(src, 0LL), *b2 = p.v + max(src, 0LL);
                                asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dk), "l"(a), "r"(bytes) : "memory");
                                asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dv), "l"(b2), "r"(bytes) : "memory");
                            }
                            asm volatile("cp.async.wait_all;" ::: "memory");
                            fence_proxy_async_smem();
                            bad0 = __reduce_min_sync(0xffffffffu, bad0);
                            bad1 = __reduce_max_sync(0xffffffffu, bad1);
                            __syncwarp();  // (the reductions order no memory: lane 0 arrives for every lane's rows)
                            if (lane == 0) {
                                if (bad1) set_status(status, ORTHROS_DEV_BAD_PAGE);
                                mt.bad[gi % kFlagRing] = bad1 ? (int)(bad0 << 8 | bad1) : 0;
                                mbar_arrive(&mt.k_full[sk]);
                                mbar_arrive(&mt.v_full[sv]);
                            }
                            __syncwarp();
                        }
                        ++gk;
                    }
                    x += n_tiles;
                    next_unit();
                }
            }
        }
        if (alive) {
            Segment sg{};
            sg.end = 1;
            publish(sg);
        }
        if (head_n > 0) {
            // the CTAs whose share begins inside the unit hold its other parts
            const Shares sh = shares_of(p, pl);
            head.n_parts = 1;
            for (int k0 = j + 1; k0 < sh.eff; k0 += 32) {  // (a lane looks at one border)
                const int k = k0 + lane;
                const unsigned in = __ballot_sync(0xffffffffu, k < sh.eff && sh.moved(sh.border(k), head_u0, head_n) < head_u0 + head_n);
                head.n_parts += __popc(in);
                if (in != 0xffffffffu) break;
            }
        }
        if (lane == 0) {
            ChunkHead &to = p.heads[blockIdx.x];
            to.n_parts = head.n_parts;
            to.tok0 = head.tok0;
            to.cnt = head.cnt;
            to.kv = head.kv;
            // nothing may be in flight when the CTA leaves
            if (p.box) {
                for (uint32_t i = gk > (uint32_t)kNumK ? gk - kNumK : 0; i < gk; ++i)
                    mbar_wait_drain(&mt.k_full[i % kNumK], (i / kNumK) & 1, status);
                for (uint32_t i = gv > (uint32_t)kNumV ? gv - kNumV : 0; i < gv; ++i)
                    mbar_wait_drain(&mt.v_full[i % kNumV], (i / kNumV) & 1, status);
            }
            for (int s = 0; s < 2; ++s)
                if (nq[s] > 0) mbar_wait_drain(&mt.q_full[s], (nq[s] - 1) & 1, status);
        }
    } else if (warp == kMmaWarp) {
        // ---------------- tcgen05.mma issuer ----------------
        {
            const uint32_t el = elect_one();
            const uint32_t tm = uniform(tmem);
            constexpr uint32_t kIdescS = idesc_f16(1, 1, 0, 0, kRows, kKeys);  // bf16, both K-major
            constexpr uint32_t kIdescO = idesc_f16(1, 1, 0, 1, kRows, D);      // bf16, V MN-major
            constexpr uint32_t kTileU = C::kTile >> 4;
            const uint64_t dq = desc_sw128(smem_u32(smem + C::kQ0), 16, 1024);
            const uint64_t dk = desc_sw128(smem_u32(smem + C::kK0), 16, D * 16);
            const uint64_t dv = desc_sw128(smem_u32(smem + C::kV0), 1024, D * 16);
            auto issue_s = [&](int s, uint64_t qd, uint64_t kd) {
#pragma unroll
                for (int ks = 0; ks < D / 16; ++ks) {
                    const uint32_t qo = ((ks >> 2) * (kRows * 128) + (ks & 3) * 32) >> 4;
                    const uint32_t ko = ((ks >> 2) * 1024 + (ks & 3) * 32) >> 4;
                    mma_ss_if(el, tm + s * 128, qd + qo, kd + ko, kIdescS, ks > 0);
                }
                tc_commit_if(el, &mt.s_full[s]);
            };
            // O += P V over half h of the tile's keys
            auto issue_pv = [&](int s, int h, uint64_t vd, uint32_t acc0) {
#pragma unroll
                for (int k = 0; k < kKeys / 32; ++k) {
                    const int kk = h * (kKeys / 32) + k;
                    mma_ts_if(el, tm + C::kTmemO + s * 128, tm + s * 128 + kk * 8, vd + (uint64_t)((kk * 16 * D * 2) >> 4),
                              kIdescO, kk > 0 ? 1u : acc0);
                }
            };
            // stage and phase of the next key tile, the next value tile (counted, not divided: this
            // warp's instructions are on the critical path)
            uint32_t ks = 0, kph = 0, vs = 0, vph = 0;
            auto next_k = [&]() {
                if (++ks == kNumK) ks = 0, kph ^= 1;
            };
            auto next_v = [&]() {
                if (++vs == kNumV) vs = 0, vph ^= 1;
            };
            uint32_t nq0 = 0, nq1 = 0;         // phase of the next query tile per slot
            uint32_t pc0 = 0, pc1 = 0;         // of the next P tile
            uint32_t oc0 = 0, oc1 = 0;         // segments in which the slot had tiles
            bool ok = true;
            for (int i = 0; ok; ++i) {
                const int r = i % kSegRing;
                if (!(ok = mbar_wait_warp(&mt.g_full[r], (i / kSegRing) & 1, abort, status))) break;
                // (broadcast: known to be the same in every lane, as everything that follows from them)
                const Segment &sr = mt.seg[r];
                const bool end = uniform(sr.end) != 0, pair = uniform(sr.pair) != 0;
                const int n = uniform(sr.nkt);
                const int lo0 = uniform(sr.lo[0]), hi0 = uniform(sr.hi[0]), lo1 = uniform(sr.lo[1]), hi1 = uniform(sr.hi[1]);
                __syncwarp();
                if (lane == 0) mbar_arrive(&mt.g_empty[r]);
                if (end) break;
                auto key_tile = [&]() -> bool {
                    if (!mbar_wait_warp(&mt.k_full[ks], kph, abort, status)) return false;
                    tc_fence_after();
                    return true;
                };
                auto value_tile = [&]() -> bool { return mbar_wait_warp(&mt.v_full[vs], vph, abort, status); };
                // the slot's next P V: the first half of the keys goes while the softmax finishes the second;
                // before the slot's first product of the segment, its O is free
                auto pv_tile = [&](int s, uint32_t &pc, uint32_t &oc, bool first) -> bool {
                    const uint64_t vd = dv + (uint64_t)(vs * kTileU);
                    if (first) {
                        if (oc > 0 && !mbar_wait_warp(&mt.o_free[s], (oc - 1) & 1, abort, status)) return false;
                        ++oc;
                    }
                    if (!mbar_wait_warp(&mt.p_half[s], pc, abort, status)) return false;
                    tc_fence_after();
                    issue_pv(s, 0, vd, !first);
                    if (!mbar_wait_warp(&mt.p_full[s], pc, abort, status)) return false;
                    tc_fence_after();
                    issue_pv(s, 1, vd, 1);
                    pc ^= 1;
                    return true;
                };
                if (pair) {
                    // first tile's S of both slots
                    if (!(ok = mbar_wait_warp(&mt.q_full[0], nq0, abort, status) && key_tile())) break;
                    if (lo0 <= 0 && hi0 >= 0) issue_s(0, dq, dk + (uint64_t)(ks * kTileU));
                    if (n == 1) tc_commit_if(el, &mt.q_empty[0]);
                    if (!(ok = mbar_wait_warp(&mt.q_full[1], nq1, abort, status))) break;
                    tc_fence_after();
                    if (lo1 <= 0 && hi1 >= 0) issue_s(1, dq + kTileU, dk + (uint64_t)(ks * kTileU));
                    if (n == 1) tc_commit_if(el, &mt.q_empty[1]);
                    tc_commit_if(el, &mt.k_empty[ks]);
                    next_k();
                    // per tile and slot: P V, then the next tile's S into the columns that held P
                    int it = 0;
                    // both: both slots work on tiles it and it + 1, neither for the first or the last time
                    auto tile = [&](bool both) -> bool {
                        const bool more = both || it + 1 < n;
                        if (!value_tile()) return false;
                        if (both || (it >= lo0 && it <= hi0)) {
                            if (!pv_tile(0, pc0, oc0, !both && it == lo0)) return false;
                            if (!both && it == hi0) tc_commit_if(el, &mt.o_full[0]);
                        }
                        if (more) {
                            if (!key_tile()) return false;
                            if (both || (it + 1 >= lo0 && it + 1 <= hi0)) issue_s(0, dq, dk + (uint64_t)(ks * kTileU));
                            if (it + 2 == n) tc_commit_if(el, &mt.q_empty[0]);
                        }
                        if (both || (it >= lo1 && it <= hi1)) {
                            if (!pv_tile(1, pc1, oc1, !both && it == lo1)) return false;
                            if (!both && it == hi1) tc_commit_if(el, &mt.o_full[1]);
                        }
                        tc_commit_if(el, &mt.v_empty[vs]);
                        next_v();
                        if (more) {
                            if (both || (it + 1 >= lo1 && it + 1 <= hi1)) issue_s(1, dq + kTileU, dk + (uint64_t)(ks * kTileU));
                            if (it + 2 == n) tc_commit_if(el, &mt.q_empty[1]);
                            tc_commit_if(el, &mt.k_empty[ks]);
                            next_k();
                        }
                        ++it;
                        return true;
                    };
                    const int mid0 = max(lo0, lo1) + 1, mid1 = min(hi0, hi1);  // tiles mid0 .. mid1 - 1 in full
                    while (ok && it < n) {
                        while (ok && it >= mid0 && it < mid1) ok = tile(true);
                        if (ok && it < n) ok = tile(false);
                    }
                    nq0 ^= 1;
                    nq1 ^= 1;
                } else {
                    if (!(ok = mbar_wait_warp(&mt.q_full[0], nq0, abort, status))) break;
                    nq0 ^= 1;
                    // tile it's S into slot s
                    auto s_tile = [&](int it, int s) -> bool {
                        if (!key_tile()) return false;
                        issue_s(s, dq, dk + (uint64_t)(ks * kTileU));
                        if (it + 1 == n) tc_commit_if(el, &mt.q_empty[0]);
                        tc_commit_if(el, &mt.k_empty[ks]);
                        next_k();
                        return true;
                    };
                    ok = s_tile(0, 0) && (n < 2 || s_tile(1, 1));
                    // (one body for both slots: these segments are short, their code mostly cold)
                    uint32_t pc[2] = {pc0, pc1}, oc[2] = {oc0, oc1};
                    for (int it = 0; ok && it < n; ++it) {
                        const int s = it & 1;
                        if (!(ok = value_tile() && pv_tile(s, pc[s], oc[s], it < 2))) break;
                        if (it + 2 >= n) tc_commit_if(el, s ? &mt.ox_full : &mt.o_full[0]);
                        tc_commit_if(el, &mt.v_empty[vs]);
                        next_v();
                        if (it + 2 < n) ok = s_tile(it + 2, s);
                    }
                    pc0 = pc[0], pc1 = pc[1], oc0 = oc[0], oc1 = oc[1];
                }
            }
            // every product issued must be complete before tensor memory is freed
            tc_commit_if(el, &mt.mma_done);
            if (lane == 0) mbar_wait_drain(&mt.mma_done, 0, status);
        }
        __syncwarp();
    } else if (warp == kClearWarp) {
        // ---------------- unseen value rows: a page that reaches past the unit's keys holds
        // anything there, and 0 * NaN is NaN ----------------
        uint32_t gk = 0;
        uint32_t ne = 0;  // bit per stage: parity of such tiles handled
        bool ok = true;
        for (int i = 0; ok; ++i) {
            const int r = i % kSegRing;
            if (!mbar_wait_warp(&mt.g_full[r], (i / kSegRing) & 1, abort, status)) break;
            const Segment sg = mt.seg[r];
            __syncwarp();
            if (lane == 0) mbar_arrive(&mt.g_empty[r]);
            if (sg.end) break;
            if (!p.box) continue;  // gathered rows come clean
            for (int it = 0; it < sg.nkt; ++it) {
                int r0, r1;
                if (!unseen_rows(sg, p.window, it, r0, r1)) continue;
                const uint32_t sv = (gk + it) % kNumV;
                if (!(ok = mbar_wait_warp(&mt.ve_full[sv], (ne >> sv) & 1, abort, status))) break;
                ne ^= 1u << sv;
                uint8_t *vs = smem + C::kV0 + sv * C::kTile;
                constexpr int kCh = D / 8;
                for (int e = lane; e < (r0 + kKeys - r1) * kCh; e += 32) {
                    const int k = e / kCh, row = k < r0 ? k : r1 + k - r0;
                    *reinterpret_cast<uint4 *>(vs + kv_offset<D>(row, e % kCh)) = make_uint4(0, 0, 0, 0);
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(&mt.v_full[sv]);
            }
            gk += sg.nkt;
        }
    } else {
        // ---------------- softmax: one thread per row ----------------
        const int s = warp >> 2;
        const int row = ((warp & 3) << 5) | lane;
        const uint32_t lane_off = static_cast<uint32_t>((warp & 3) * 32) << 16;
        const uint32_t t_s = tmem + lane_off + s * 128;
        const uint32_t t_o = tmem + lane_off + C::kTmemO;  // slot 0's O (slot 1's: + 128)
        const float c2 = p.scale_log2;
        uint32_t cnt = 0;              // S tiles of this slot handled
        uint32_t oc = 0, ox = 0;       // phases of o_full[s] and ox_full waited for
        uint32_t shared = 0;           // segments with one row tile
        uint32_t gk = 0;               // key tiles of earlier segments
        for (int i = 0;; ++i) {
            const int r = i % kSegRing;
            if (!mbar_wait_warp(&mt.g_full[r], (i / kSegRing) & 1, abort, status)) break;
            const Segment sg = mt.seg[r];
            __syncwarp();
            if (lane == 0) mbar_arrive(&mt.g_empty[r]);
            if (sg.end) break;
            const int c0 = sg.pair && s ? tt : 0;                    // first token of this slot's row tile
            const int n_tok = min(tt, sg.cnt - c0);
            const bool mine = row < n_tok * g;                       // a real row
            const bool idle = (warp & 3) * 32 >= n_tok * g;          // no real row in this warp
            const int t_first = sg.pos0 + c0, t_last = t_first + n_tok - 1;
            const int t_row = mine ? t_first + row_token(p, row) : t_last;
            const int lo_row = max(0, t_row - p.window + 1);
            const int lo_max = max(0, t_last - p.window + 1);
            const int it0 = sg.pair ? sg.lo[s] : s, step = sg.pair ? 1 : 2, it1 = sg.pair ? sg.hi[s] : sg.nkt - 1;
            const int tiles = it0 <= it1 ? (it1 - it0) / step + 1 : 0;
            float m_ref = -INFINITY, l = 0.f;
            bool ok = true, bad = false;
            for (int it = it0; it <= it1; it += step) {
                if (!(ok = mbar_wait_warp(&mt.s_full[s], cnt & 1, abort, status))) break;
                ++cnt;
                if (idle) {
                    mbar_arrive(&mt.p_half[s]);
                    mbar_arrive(&mt.p_full[s]);
                    continue;
                }
                tc_fence_after();
                const int key0 = (sg.kt0 + it) * kKeys;
                const int no_page = mt.bad[(gk + it) % kFlagRing];
                if (no_page && key0 + (no_page >> 8) <= t_row && key0 + (no_page & 255) > lo_row) bad = true;
                uint32_t xr[kKeys];
                using Cols = uint32_t[32];
                const float *x = reinterpret_cast<const float *>(xr);
                for (int pass = 0;; ++pass) {
#pragma unroll
                    for (int q = 0; q < kKeys / 32; ++q) tmem_ld32(t_s + 32 * q, *reinterpret_cast<Cols *>(xr + 32 * q));
                    tmem_ld_wait();
#pragma unroll
                    for (int q = 0; q < kKeys / 32; ++q) reg_fence(*reinterpret_cast<Cols *>(xr + 32 * q));
                    // A loop of no or one turn, so that the compiler keeps a branch around the mask: as 128
                    // predicated selects it ran for every tile (ALU instructions 2.8-fold, the kernel 1.5-fold).
                    int turns = key0 + kKeys - 1 > t_first || key0 < lo_max;  // warp-uniform
                    asm volatile("" : "+r"(turns));
                    for (; turns > 0; --turns) {
                        const int first = key0 - lo_row;
                        const unsigned span = t_row - lo_row;
#pragma unroll
                        for (int c = 0; c < kKeys; ++c)
                            if ((unsigned)(first + c) > span) xr[c] = __float_as_uint(-INFINITY);
                    }
                    if (pass) break;
                    float mq[16];
#pragma unroll
                    for (int q = 0; q < 16; ++q)
                        mq[q] = max3(max3(x[8 * q], x[8 * q + 1], x[8 * q + 2]), max3(x[8 * q + 3], x[8 * q + 4], x[8 * q + 5]),
                                     fmaxf(x[8 * q + 6], x[8 * q + 7]));
                    const float m_tile = max3(max3(max3(mq[0], mq[1], mq[2]), max3(mq[3], mq[4], mq[5]), max3(mq[6], mq[7], mq[8])),
                                              max3(mq[9], mq[10], mq[11]), max3(mq[12], mq[13], fmaxf(mq[14], mq[15])));
                    // the shift follows the maximum only when it grew by more than 2^8 (P stays finite in bf16)
                    const float m_new = fmaxf(m_ref, m_tile);
                    const bool resc = (m_new - m_ref) * c2 > 8.f;  // true on the first finite maximum
                    const float alpha = resc ? ex2((m_ref - m_new) * c2) : 1.f;
                    if (resc) {
                        l *= alpha;
                        m_ref = m_new;
                    }
                    if (!__any_sync(0xffffffffu, resc) || it == it0) break;
                    // Rescales O, which is idle here (the product of the slot's previous tile completed
                    // before this S); the logits are loaded again after it rather than held beside it.
#pragma unroll
                    for (int j = 0; j < D / 32; ++j) {
                        uint32_t o[32];
                        tmem_ld32(t_o + s * 128 + 32 * j, o);
                        tmem_ld_wait();
                        reg_fence(o);
#pragma unroll
                        for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha);
                        tmem_st32(t_o + s * 128 + 32 * j, o);
                    }
                    tmem_st_wait();
                }
                const float mb = m_ref == -INFINITY ? 0.f : m_ref * c2;
                float ls[4] = {0.f, 0.f, 0.f, 0.f};
                const uint64_t cv = f32x2(c2, c2), mv = f32x2(-mb, -mb);
#pragma unroll
                for (int j = 0; j < kKeys / 32; ++j) {
                    const float *xj = x + 32 * j;
                    uint32_t pk[16];
#pragma unroll
                    for (int e = 0; e < 16; ++e) {
                        float a0, a1;
                        fma_f32x2(xj[2 * e], xj[2 * e + 1], cv, mv, a0, a1);
                        const float p0 = ex2(a0), p1 = ex2(a1);
                        add_f32x2(ls[2 * (e & 1)], ls[2 * (e & 1) + 1], p0, p1);
                        pk[e] = pack_bf16(p0, p1);
                    }
                    tmem_st16(t_s + 16 * j, pk);
                    if (j == 2) {
                        tmem_st_wait();
                        tc_fence_before();
                        mbar_arrive(&mt.p_half[s]);
                    }
                }
                l += (ls[0] + ls[1]) + (ls[2] + ls[3]);
                tmem_st_wait();
                tc_fence_before();
                mbar_arrive(&mt.p_full[s]);
            }
            if (!ok) break;
            if (bad) l = __int_as_float(0x7fc00000);  // the row saw a page that does not exist: NaN

            // ---- epilogue ----
            const int n0 = sg.pair ? (s == 0 ? tiles : 0) : (sg.nkt + 1) / 2;  // slot 0's tiles
            const int n1 = sg.pair ? (s == 1 ? tiles : 0) : sg.nkt / 2;        // slot 1's
            gk += sg.nkt;
            if (!sg.pair && s == 1) {
                // slot 0 finishes the shared rows
                if (shared > 0 && !mbar_wait_warp(&mt.ml_free, (shared - 1) & 1, abort, status)) break;
                mt.ml[row] = make_float2(m_ref, l);
                mbar_arrive(&mt.ml_full);
                ++shared;
                continue;
            }
            // weights of the two accumulators (a slot with its own row tile: 1 and 0)
            float w0 = 1.f, w1 = 0.f, m = m_ref;
            bool two = false;
            if (n0 + n1 > 0 && !mbar_wait_warp(&mt.o_full[s], oc++ & 1, abort, status)) break;
            if (!sg.pair) {
                two = n1 > 0;
                if (two && !mbar_wait_warp(&mt.ox_full, ox++ & 1, abort, status)) break;
                if (!mbar_wait_warp(&mt.ml_full, shared & 1, abort, status)) break;
                ++shared;
                const float2 o = mt.ml[row];
                mbar_arrive(&mt.ml_free);
                if (two) {
                    m = fmaxf(m_ref, o.x);
                    const float mb = m == -INFINITY ? 0.f : m * c2;
                    w0 = ex2(m_ref * c2 - mb);
                    w1 = ex2(o.x * c2 - mb);
                    l = l * w0 + o.y * w1;
                }
            }
            if (!idle) {
                tc_fence_after();
                const int rt = row_token(p, row);
                const long long tok = sg.tok0 + c0 + rt;
                const int h = sg.kv * g + row - rt * g;
                const uint32_t t_a = t_o + (sg.pair ? s * 128 : 0);
                const bool fin = sg.partial < 0;
                const long long out = tok * p.Hq + h;  // row of o, or of the partials
                const long long at = ((long long)sg.partial * p.slots_cap + (sg.pair ? s : 0)) * p.rows_cap + row;
                if (fin) {
                    const float inv = inverse_sum(l);
                    w0 *= inv;
                    w1 *= inv;
                    if (mine && p.lse) p.lse[out] = m * p.scale + logf(l);
                } else if (mine) {
                    p.part_ml[at] = make_float2(m, l);
                }
                // 32 channels a turn, not unrolled: this code runs once per segment, mostly from a cold
                // instruction cache
                if (n0 + n1 > 0)
#pragma unroll 1
                    for (int j = 0; j < D / 32; ++j) {
                        uint32_t o[32];
                        tmem_ld32(t_a + 32 * j, o);
                        tmem_ld_wait();
                        reg_fence(o);
                        float f[32];
#pragma unroll
                        for (int e = 0; e < 32; ++e) f[e] = __uint_as_float(o[e]) * w0;
                        if (two) {
                            tmem_ld32(t_a + 128 + 32 * j, o);
                            tmem_ld_wait();
                            reg_fence(o);
#pragma unroll
                            for (int e = 0; e < 32; ++e) f[e] = fmaf(__uint_as_float(o[e]), w1, f[e]);
                        }
                        if (!mine) continue;
                        if (fin) {
                            __nv_bfloat16 *dst = p.o + out * D + 32 * j;
#pragma unroll
                            for (int e = 0; e < 2; ++e) {
                                uint32_t w[8];
#pragma unroll
                                for (int i = 0; i < 8; ++i) w[i] = pack_bf16(f[16 * e + 2 * i], f[16 * e + 2 * i + 1]);
                                if (p.o_aligned32) {
                                    st_global_32b(dst + 16 * e, w);
                                } else {
                                    uint4 *to = reinterpret_cast<uint4 *>(dst + 16 * e);
                                    to[0] = make_uint4(w[0], w[1], w[2], w[3]);
                                    to[1] = make_uint4(w[4], w[5], w[6], w[7]);
                                }
                            }
                        } else {
                            float *dst = p.part_o + at * D + 32 * j;
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                uint32_t w[8];
#pragma unroll
                                for (int i = 0; i < 8; ++i) w[i] = __float_as_uint(f[8 * e + i]);
                                st_global_32b(dst + 8 * e, w);
                            }
                        }
                    }
                tc_fence_before();
            }
            if (n0) mbar_arrive(&mt.o_free[0]);
            if (n1) mbar_arrive(&mt.o_free[1]);
        }
    }

    tc_fence_before();
    __syncthreads();
    if (warp == kMmaWarp) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

// ---------------------------------------------------------------------------
// Merge of the units that a share's border cut: o = sum_k w_k o_k / sum_k w_k l_k with
// w_k = exp(scale (m_k - max m)), the parts in a fixed order with a running maximum.
// Many rows: 8 lanes join a row (addresses and weights cost every lane the same, and a
// warp per row was bound by its instructions: 11 us of the 2048-token call instead of
// 5). Few rows may have many parts: a block joins a row, its warps every fourth part
// each, and adds their results up (a warp that walked the parts alone took 7 us longer
// for the 152 of one token over a single kv head).
// ---------------------------------------------------------------------------
constexpr int kMergeWarps = 4;
constexpr int kMergeRows = 32;    // a block per row up to so many rows of a partial
constexpr int kMergeBlocks = 16;  // blocks of a unit beyond

// Running joint of parts of one row: kLanes lanes, lane l with channels 4 kLanes i + 4 l .. + 3, i < V.
template <int V> struct Joint {
    float M, L;
    float4 acc[V];
    __device__ __forceinline__ void clear() {
        M = -INFINITY, L = 0.f;
#pragma unroll
        for (int i = 0; i < V; ++i) acc[i] = make_float4(0.f, 0.f, 0.f, 0.f);
    }
    template <int kParts> __device__ __forceinline__ void add(const float2 (&ml)[kParts], const float4 (&x)[kParts][V], float c2) {
        float m = M;
#pragma unroll
        for (int k = 0; k < kParts; ++k) m = fmaxf(m, ml[k].x);
        const float mb = m == -INFINITY ? 0.f : m * c2;
        const float w0 = ex2(M * c2 - mb);
        M = m;
        L *= w0;
#pragma unroll
        for (int i = 0; i < V; ++i) acc[i].x *= w0, acc[i].y *= w0, acc[i].z *= w0, acc[i].w *= w0;
#pragma unroll
        for (int k = 0; k < kParts; ++k) {
            if (ml[k].x == -INFINITY) {  // no finite logit: no output, and a sum of 0 or NaN
                L += ml[k].y;
                continue;
            }
            const float w = ex2(ml[k].x * c2 - mb);
            L = fmaf(w, ml[k].y, L);
#pragma unroll
            for (int i = 0; i < V; ++i) {
                acc[i].x = fmaf(w, x[k][i].x, acc[i].x);
                acc[i].y = fmaf(w, x[k][i].y, acc[i].y);
                acc[i].z = fmaf(w, x[k][i].z, acc[i].z);
                acc[i].w = fmaf(w, x[k][i].w, acc[i].w);
            }
        }
    }
};

template <int D, bool kRowBlocks>
__global__ void __launch_bounds__(kMergeWarps * 32) chunk_merge_kernel(const ChunkParams p) {
    const int tid = threadIdx.x, g = p.Hq / p.Hkv;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const ChunkHead hd = p.heads[blockIdx.x];
    if (blockIdx.x == 0 && blockIdx.y == 0) {
        // the call's status word, from the CTAs' (and the plan's)
        __shared__ uint32_t all;
        if (tid == 0) all = p.direct ? 0u : p.plan->flags;
        __syncthreads();
        uint32_t f = 0;
        for (int i = tid; i < (int)gridDim.x; i += kMergeWarps * 32) f |= p.heads[i].flags;
        if (f) atomicOr(&all, f);
        __syncthreads();
        if (tid == 0) *p.status = all;
    }
    if (hd.n_parts == 0) return;
    const float c2 = p.scale_log2;
    const int cap = p.slots_cap * p.rows_cap;  // rows of a partial, slot-major
    // row r's token and head: its row of o, or -1 when no token stands there
    auto out_row = [&](int r) -> long long {
        const int slot = r / p.rows_cap, row = r % p.rows_cap;
        if (row >= min(p.tile_tokens, hd.cnt - slot * p.tile_tokens) * g) return -1;
        const int rt = row_token(p, row);
        return ((long long)hd.tok0 + slot * p.tile_tokens + rt) * p.Hq + hd.kv * g + row - rt * g;
    };
    // row r of part k: the head's own (second) partial, then the first partial of the lane's next CTAs
    auto part_row = [&](int k, int r) -> long long {
        const int id = k == 0 ? 2 * blockIdx.x + 1 : 2 * (blockIdx.x + k * p.lanes);
        return (long long)id * cap + r;
    };
    auto store = [&](long long out, int chunk, const float4 &a, float inv) {
        reinterpret_cast<uint2 *>(p.o + out * D)[chunk] = make_uint2(pack_bf16(a.x * inv, a.y * inv), pack_bf16(a.z * inv, a.w * inv));
    };
    if constexpr (!kRowBlocks) {
        constexpr int kLanes = 8, V = D / (4 * kLanes), kParts = 2;
        const int lane = tid % kLanes;
        for (int r = (blockIdx.y * kMergeWarps * 32 + tid) / kLanes; r < cap; r += gridDim.y * kMergeWarps * (32 / kLanes)) {
            const long long out = out_row(r);
            if (out < 0) continue;
            Joint<V> jt;
            jt.clear();
            for (int k0 = 0; k0 < hd.n_parts; k0 += kParts) {
                float2 ml[kParts];
                float4 x[kParts][V];
#pragma unroll
                for (int k = 0; k < kParts; ++k) {
                    ml[k] = make_float2(-INFINITY, 0.f);
                    if (k0 + k >= hd.n_parts) continue;
                    const long long at = part_row(k0 + k, r);
                    ml[k] = p.part_ml[at];
                    const float4 *src = reinterpret_cast<const float4 *>(p.part_o + at * D) + lane;
#pragma unroll
                    for (int i = 0; i < V; ++i) x[k][i] = src[i * kLanes];
                }
                jt.add(ml, x, c2);
            }
            const float inv = inverse_sum(jt.L);
#pragma unroll
            for (int i = 0; i < V; ++i) store(out, lane + i * kLanes, jt.acc[i], inv);
            if (lane == 0 && p.lse) p.lse[out] = jt.M * p.scale + logf(jt.L);
        }
    } else {
        // a block per row: kLanes threads hold a row, kSub parts are walked side by side
        constexpr int kLanes = D / 4, kSub = kMergeWarps * 32 / kLanes, kParts = 8;
        __shared__ float2 sub_ml[kSub];
        __shared__ float4 sub_x[kSub][kLanes];
        const int lane = tid % kLanes, sub = tid / kLanes;
        const int r = blockIdx.y;
        const long long out = out_row(r);
        if (out >= 0) {
            Joint<1> jt;
            jt.clear();
            for (int k0 = sub; k0 < hd.n_parts; k0 += kSub * kParts) {
                float2 ml[kParts];
                float4 x[kParts][1];
#pragma unroll
                for (int k = 0; k < kParts; ++k) {
                    ml[k] = make_float2(-INFINITY, 0.f);
                    if (k0 + k * kSub >= hd.n_parts) continue;
                    const long long at = part_row(k0 + k * kSub, r);
                    ml[k] = p.part_ml[at];
                    x[k][0] = reinterpret_cast<const float4 *>(p.part_o + at * D)[lane];
                }
                jt.add(ml, x, c2);
            }
            if (lane == 0) sub_ml[sub] = make_float2(jt.M, jt.L);
            sub_x[sub][lane] = jt.acc[0];
            __syncthreads();
            if (sub == 0) {
                float2 ml[kSub];
                float4 x[kSub][1];
#pragma unroll
                for (int k = 0; k < kSub; ++k) ml[k] = sub_ml[k], x[k][0] = sub_x[k][lane];
                jt.clear();
                jt.add(ml, x, c2);
                const float inv = inverse_sum(jt.L);
                store(out, lane, jt.acc[0], inv);
                if (lane == 0 && p.lse) p.lse[out] = jt.M * p.scale + logf(jt.L);
            }
        }
    }
}

template <int D> cudaError_t launch_d(const ChunkParams &p, cudaStream_t stream) {
    CUtensorMap tq, tk, tv;
    const long long tokens = p.box ? (long long)p.num_pages * p.page_size : 8;  // (unused maps are valid ones)
    const int box = p.box ? p.box : 8;
    if (!encode_rows_map_3d(&tq, p.q, p.n, p.Hq, D, p.Hq / p.Hkv, p.tile_tokens) ||
        !encode_kv_groups_map(&tk, p.k, tokens, p.Hkv, D, box) || !encode_kv_groups_map(&tv, p.v, tokens, p.Hkv, D, box))
        return cudaErrorInvalidValue;
    static SmemLimit limit;
    if (cudaError_t e = limit.ensure((const void *)chunk_attn_kernel<D>, Cfg<D>::kSmem); e != cudaSuccess) return e;
    if (!p.direct) {
        ProfScope ps("chunk_plan", stream);
        chunk_plan_kernel<<<1, kPlanThreads, 0, stream>>>(p, D);
        if (cudaError_t e = cudaGetLastError(); e != cudaSuccess) return e;
    }
    // the attention's set-up overlaps the plan, the merge's launch the attention
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(p.lanes * p.per_lane);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = Cfg<D>::kSmem;
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = p.direct ? 0 : 1;
    {
        ProfScope ps("chunk_attn", stream);
        if (cudaError_t e = cudaLaunchKernelEx(&cfg, chunk_attn_kernel<D>, tq, tk, tv, p); e != cudaSuccess) return e;
    }
    const int rows = p.slots_cap * p.rows_cap;
    cudaLaunchConfig_t mc = {};
    mc.gridDim = dim3(p.lanes * p.per_lane, rows <= kMergeRows ? rows : kMergeBlocks);
    mc.blockDim = dim3(kMergeWarps * 32);
    mc.stream = stream;
    mc.attrs = attr;
    mc.numAttrs = 1;
    ProfScope ps("chunk_merge", stream);
    if (cudaError_t e = cudaLaunchKernelEx(&mc, rows <= kMergeRows ? chunk_merge_kernel<D, true> : chunk_merge_kernel<D, false>, p); e != cudaSuccess) return e;
    return cudaGetLastError();
}

}  // namespace

long long chunk_max_units(long long n, int B, int tile_tokens) { return n / (2 * tile_tokens) + B; }

cudaError_t launch_chunk_attention(const ChunkParams &p, int d, cudaStream_t stream) {
    return d == 128 ? launch_d<128>(p, stream) : launch_d<64>(p, stream);
}

}  // namespace orthros
