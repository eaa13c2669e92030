// chunk_api.cu -- C entry points of the attention of new tokens over the paged
// cache, consecutive ones or drafted trees: argument checks, workspace carving,
// dispatch to chunk_attn.cu.
#include <algorithm>
#include <cmath>
#include <numeric>

#include "internal.cuh"

namespace orthros {
namespace {

bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

struct ChunkLayout {
    size_t plan_off, seq_units_off, seq_tiles_off, units_off, heads_off, ml_off, o_off, total;
    int tile_tokens, ctas, slots_cap, rows_cap;
};

ChunkLayout chunk_layout(int B, int n, int max_new, int Hq, int Hkv, int d) {
    ChunkLayout L{};
    const int g = Hq / Hkv;
    L.tile_tokens = 128 / g;
    L.ctas = device_sm_count();
    // a partial holds one row tile of a short chunk's tokens, or both tiles of a long one's
    L.slots_cap = max_new <= L.tile_tokens ? 1 : 2;
    L.rows_cap = std::min(max_new, L.tile_tokens) * g;
    size_t at = kStatusBytes;
    auto take = [&](size_t bytes) {
        const size_t o = at;
        at += align_up(bytes, 256);
        return o;
    };
    L.plan_off = take(sizeof(ChunkPlan));
    L.seq_units_off = take(sizeof(int32_t) * (size_t)B);
    L.seq_tiles_off = take(sizeof(long long) * (size_t)B);
    L.units_off = take(sizeof(ChunkUnit) * (size_t)chunk_max_units(n, B, L.tile_tokens));
    L.heads_off = take(sizeof(ChunkHead) * (size_t)L.ctas);
    const size_t rows = 2 * (size_t)L.ctas * L.slots_cap * L.rows_cap;
    L.ml_off = take(sizeof(float2) * rows);
    L.o_off = take(sizeof(float) * rows * d);
    L.total = at;
    return L;
}

// Shapes that both entry points refuse.
orthros_status check_shape(int B, int n, int max_new, int Hq, int Hkv, int d, int max_pages, int page_size, orthros_dtype dtype) {
    if (B < 0 || n < 0) return report_error(ORTHROS_EINVAL, "B = %d and n = %d must be >= 0", B, n);
    if (n > 0 && B < 1) return report_error(ORTHROS_EINVAL, "n = %d tokens with B = 0", n);
    if (max_new < (n > 0 ? 1 : 0)) return report_error(ORTHROS_EINVAL, "max_new = %d must be >= 1", max_new);
    if (Hq < 1 || Hkv < 1 || Hq % Hkv != 0)
        return report_error(ORTHROS_EINVAL, "Hq = %d must be a positive multiple of Hkv = %d", Hq, Hkv);
    if (max_pages < 1 || page_size < 1) return report_error(ORTHROS_EINVAL, "max_pages and page_size must be >= 1");
    if (dtype != ORTHROS_BF16 && dtype != ORTHROS_F32) return report_error(ORTHROS_EINVAL, "unknown dtype %d", (int)dtype);
    if (dtype != ORTHROS_BF16) return report_error(ORTHROS_EUNSUPPORTED, "the attention of new tokens over the cache takes bf16 only");
    if (d != 64 && d != 128) return report_error(ORTHROS_EUNSUPPORTED, "head size d = %d (supported: 64, 128)", d);
    if (Hq / Hkv > 128) return report_error(ORTHROS_EUNSUPPORTED, "%d query heads per kv head (at most 128)", Hq / Hkv);
    if (Hkv > 65536) return report_error(ORTHROS_EUNSUPPORTED, "Hkv = %d exceeds 65536", Hkv);
    return ORTHROS_OK;
}

// Both attentions: consecutive new tokens, or (tree) drafted trees with their masks.
orthros_status attend(const void *q, const int32_t *q_indptr, const int32_t *kv_lens, const int32_t *tree_mask, bool tree, int words,
                      const void *k_cache, const void *v_cache, const int32_t *block_table, int B, int n, int max_new, int Hq,
                      int Hkv, int d, int window, float scale, orthros_dtype dtype, int max_pages, int page_size, int num_pages,
                      void *o, float *lse, void *workspace, size_t workspace_bytes, cudaStream_t stream) {
    if (const orthros_status st = check_shape(B, n, max_new, Hq, Hkv, d, max_pages, page_size, dtype); st != ORTHROS_OK)
        return st;
    max_new = std::min(max_new, n);
    if (tree) max_new = std::min(max_new, 32 * words);
    if (window < 1) return report_error(ORTHROS_EINVAL, "window = %d must be >= 1", window);
    if (!std::isfinite(scale) || !(scale > 0.f)) return report_error(ORTHROS_EINVAL, "scale must be finite and > 0");
    if (num_pages < 1) return report_error(ORTHROS_EINVAL, "num_pages = %d must be >= 1", num_pages);
    if ((long long)num_pages * page_size > 0x7fffffffLL - 128 || (long long)max_pages * page_size > 0x7fffffffLL - 128)
        return report_error(ORTHROS_EUNSUPPORTED, "a pool or block table of 2^31 token slots");
    const ChunkLayout L = chunk_layout(B, n, max_new, Hq, Hkv, d);
    if (!workspace || workspace_bytes < L.total)
        return report_error(ORTHROS_EWORKSPACE, "workspace needs %zu bytes, got %zu", L.total, workspace ? workspace_bytes : (size_t)0);
    if ((reinterpret_cast<uintptr_t>(workspace) & 255u) != 0)
        return report_error(ORTHROS_EINVAL, "workspace must be 256-byte aligned");
    if (n > 0) {
        if (!q || !o || !k_cache || !v_cache) return report_error(ORTHROS_EINVAL, "q, o, k_cache and v_cache must not be NULL");
        if (!q_indptr || !kv_lens || !block_table)
            return report_error(ORTHROS_EINVAL, "q_indptr, kv_lens and block_table must not be NULL");
        if (tree && (!tree_mask || (reinterpret_cast<uintptr_t>(tree_mask) & 3u)))
            return report_error(ORTHROS_EINVAL, "tree_mask must not be NULL and 4-byte aligned");
        if (!aligned16(q) || !aligned16(o) || !aligned16(k_cache) || !aligned16(v_cache))
            return report_error(ORTHROS_EINVAL, "q, o, k_cache and v_cache must be 16-byte aligned");
    }
    uint8_t *ws = static_cast<uint8_t *>(workspace);
    if (n == 0) {
        const cudaError_t e = cudaMemsetAsync(ws, 0, sizeof(uint32_t), stream);
        return e == cudaSuccess ? ORTHROS_OK : report_error(ORTHROS_ECUDA, "status reset: %s", cudaGetErrorString(e));
    }
    ChunkParams p{};
    p.q = static_cast<const __nv_bfloat16 *>(q);
    p.k = static_cast<const __nv_bfloat16 *>(k_cache);
    p.v = static_cast<const __nv_bfloat16 *>(v_cache);
    p.q_indptr = q_indptr;
    p.kv_lens = kv_lens;
    p.block_table = block_table;
    p.B = B;
    p.n = n;
    p.max_new = max_new;
    p.tree_mask = reinterpret_cast<const uint32_t *>(tree_mask);
    p.words = words;
    p.Hq = Hq;
    p.Hkv = Hkv;
    p.window = window;
    p.max_pages = max_pages;
    p.page_size = page_size;
    p.num_pages = num_pages;
    p.tile_tokens = L.tile_tokens;
    p.g_inv = 65536 / (Hq / Hkv) + 1;
    // the largest copy box of whole 8-row swizzle atoms that never crosses a page
    p.box = 128;
    while (page_size % p.box != 0) p.box /= 2;
    if (p.box < 8) p.box = 0;
    p.lanes = std::gcd(Hkv, L.ctas);
    p.per_lane = L.ctas / p.lanes;
    p.rows_cap = L.rows_cap;
    p.slots_cap = L.slots_cap;
    p.direct = (B <= 32 && p.max_new <= 2 * p.tile_tokens) || (B == 1 && n <= 32 * 2 * p.tile_tokens);
    p.scale = scale;
    p.scale_log2 = scale * 1.4426950408889634f;
    p.o = static_cast<__nv_bfloat16 *>(o);
    p.o_aligned32 = (reinterpret_cast<uintptr_t>(o) & 31u) == 0;
    p.lse = lse;
    p.status = reinterpret_cast<uint32_t *>(ws);
    p.plan = reinterpret_cast<ChunkPlan *>(ws + L.plan_off);
    p.seq_units = reinterpret_cast<int32_t *>(ws + L.seq_units_off);
    p.seq_tiles = reinterpret_cast<long long *>(ws + L.seq_tiles_off);
    p.units = reinterpret_cast<ChunkUnit *>(ws + L.units_off);
    p.heads = reinterpret_cast<ChunkHead *>(ws + L.heads_off);
    p.part_ml = reinterpret_cast<float2 *>(ws + L.ml_off);
    p.part_o = reinterpret_cast<float *>(ws + L.o_off);
    const cudaError_t e = launch_chunk_attention(p, d, stream);
    return e == cudaSuccess ? ORTHROS_OK : report_error(ORTHROS_ECUDA, "attention launch: %s", cudaGetErrorString(e));
}

}  // namespace
}  // namespace orthros

using namespace orthros;

extern "C" {

size_t orthros_chunk_attention_workspace_size(int B, int n, int max_new, int Hq, int Hkv, int d, int max_pages,
                                              int page_size, orthros_dtype dtype) {
    if (check_shape(B, n, max_new, Hq, Hkv, d, max_pages, page_size, dtype) != ORTHROS_OK) return 0;
    return chunk_layout(B, n, std::min(max_new, n), Hq, Hkv, d).total;
}

orthros_status orthros_chunk_attention(const void *q, const int32_t *q_indptr, const int32_t *kv_lens,
                                       const void *k_cache, const void *v_cache, const int32_t *block_table, int B,
                                       int n, int max_new, int Hq, int Hkv, int d, int window, float scale,
                                       orthros_dtype dtype, int max_pages, int page_size, int num_pages, void *o,
                                       float *lse, void *workspace, size_t workspace_bytes, orthros_stream_t stream) {
    clear_error();
    return attend(q, q_indptr, kv_lens, nullptr, false, 0, k_cache, v_cache, block_table, B, n, max_new, Hq, Hkv, d, window, scale,
                  dtype, max_pages, page_size, num_pages, o, lse, workspace, workspace_bytes,
                  reinterpret_cast<cudaStream_t>(stream));
}

size_t orthros_tree_attention_workspace_size(int B, int n, int max_new, int Hq, int Hkv, int d, int max_pages, int page_size,
                                             orthros_dtype dtype) {
    return orthros_chunk_attention_workspace_size(B, n, std::min(max_new, kTreeMaxTokens), Hq, Hkv, d, max_pages, page_size, dtype);
}

orthros_status orthros_tree_attention(const void *q, const int32_t *q_indptr, const int32_t *kv_lens, const int32_t *tree_mask,
                                      int mask_words, const void *k_cache, const void *v_cache, const int32_t *block_table,
                                      int B, int n, int max_new, int Hq, int Hkv, int d, int window, float scale,
                                      orthros_dtype dtype, int max_pages, int page_size, int num_pages, void *o, float *lse,
                                      void *workspace, size_t workspace_bytes, orthros_stream_t stream) {
    clear_error();
    if (mask_words < 1 || mask_words > kTreeMaxTokens / 32)
        return report_error(ORTHROS_EINVAL, "mask_words = %d must lie in [1, %d]", mask_words, kTreeMaxTokens / 32);
    return attend(q, q_indptr, kv_lens, tree_mask, true, mask_words, k_cache, v_cache, block_table, B, n, max_new, Hq, Hkv, d,
                  window, scale, dtype, max_pages, page_size, num_pages, o, lse, workspace, workspace_bytes,
                  reinterpret_cast<cudaStream_t>(stream));
}

}  // extern "C"
