// step_api.cu -- C entry points of a serving step's plan and of the commit of a
// tree's accepted path: argument checks, dispatch to step_plan.cu.
#include "internal.cuh"

namespace orthros {
namespace {

bool aligned(const void *p, unsigned bytes) { return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) == 0; }

orthros_status check_workspace(const void *workspace, size_t bytes) {
    if (!workspace || bytes < kStatusBytes)
        return report_error(ORTHROS_EWORKSPACE, "workspace needs %zu bytes, got %zu", kStatusBytes, workspace ? bytes : (size_t)0);
    if (!aligned(workspace, 256)) return report_error(ORTHROS_EINVAL, "workspace must be 256-byte aligned");
    return ORTHROS_OK;
}

orthros_status check_pool(int B, int max_pages, int page_size, int num_pages) {
    if (B < 1) return report_error(ORTHROS_EINVAL, "B = %d must be >= 1", B);
    if (max_pages < 1 || page_size < 1 || num_pages < 1)
        return report_error(ORTHROS_EINVAL, "max_pages, page_size and num_pages must be >= 1");
    if ((long long)num_pages * page_size > 0x7fffffffLL || (long long)max_pages * page_size > 0x7fffffffLL)
        return report_error(ORTHROS_EUNSUPPORTED, "a pool or block table of 2^31 token slots");
    return ORTHROS_OK;
}

// int32 arrays of a call: none NULL, all 4-byte aligned.
struct Array {
    const char *name;
    const void *p;
};
template <int N> orthros_status check_arrays(const Array (&a)[N]) {
    for (const Array &x : a) {
        if (!x.p) return report_error(ORTHROS_EINVAL, "%s must not be NULL", x.name);
        if (!aligned(x.p, 4)) return report_error(ORTHROS_EINVAL, "%s must be 4-byte aligned", x.name);
    }
    return ORTHROS_OK;
}

}  // namespace
}  // namespace orthros

using namespace orthros;

extern "C" {

orthros_status orthros_plan_step(const int32_t *cache_lens, const int32_t *new_lens, const int32_t *pages_held,
                                 const int32_t *free_count, const int32_t *parents, int max_tree, int32_t *free_pages,
                                 int32_t *block_table, int B, int n, int max_pages, int page_size, int num_pages,
                                 int32_t *q_indptr, int32_t *kv_lens, int32_t *cache_lens_out, int32_t *pages_held_out, int32_t *free_count_out,
                                 int32_t *token_seq, int32_t *token_pos, int32_t *token_slots, int32_t *tree_mask,
                                 void *workspace, size_t workspace_bytes, orthros_stream_t stream_) {
    clear_error();
    if (orthros_status st = check_pool(B, max_pages, page_size, num_pages); st != ORTHROS_OK) return st;
    if (B > kPlanMaxSeqs) return report_error(ORTHROS_EUNSUPPORTED, "B = %d exceeds %d", B, kPlanMaxSeqs);
    if (n < 0) return report_error(ORTHROS_EINVAL, "n = %d must be >= 0", n);
    if (max_tree < 0 || max_tree > kTreeMaxTokens)
        return report_error(ORTHROS_EINVAL, "max_tree = %d must lie in [0, %d]", max_tree, kTreeMaxTokens);
    if (orthros_status st = check_workspace(workspace, workspace_bytes); st != ORTHROS_OK) return st;
    const Array all[] = {{"cache_lens", cache_lens}, {"new_lens", new_lens}, {"pages_held", pages_held}, {"free_count", free_count},
                         {"free_pages", free_pages}, {"block_table", block_table}, {"q_indptr", q_indptr}, {"kv_lens", kv_lens},
                         {"pages_held_out", pages_held_out}, {"free_count_out", free_count_out}};
    if (orthros_status st = check_arrays(all); st != ORTHROS_OK) return st;
    if (kv_lens == cache_lens || kv_lens == cache_lens_out)
        return report_error(ORTHROS_EINVAL, "kv_lens is a buffer of its own (-1 for a sequence that has no place in the step)");
    if (!aligned(cache_lens_out, 4)) return report_error(ORTHROS_EINVAL, "cache_lens_out must be 4-byte aligned");
    if (n > 0) {
        const Array rows[] = {{"token_seq", token_seq}, {"token_pos", token_pos}, {"token_slots", token_slots}};
        if (orthros_status st = check_arrays(rows); st != ORTHROS_OK) return st;
        if (max_tree > 0) {
            const Array tree[] = {{"parents", parents}, {"tree_mask", tree_mask}};
            if (orthros_status st = check_arrays(tree); st != ORTHROS_OK) return st;
        }
    }
    StepPlanParams p{};
    p.cache_lens = cache_lens;
    p.new_lens = new_lens;
    p.held_in = pages_held;
    p.count_in = free_count;
    p.parents = max_tree > 0 ? parents : nullptr;
    p.free_pages = free_pages;
    p.block_table = block_table;
    p.q_indptr = q_indptr;
    p.kv_lens = kv_lens;
    p.lens_out = cache_lens_out;
    p.held_out = pages_held_out;
    p.count_out = free_count_out;
    p.token_seq = token_seq;
    p.token_pos = token_pos;
    p.token_slots = token_slots;
    p.tree_mask = reinterpret_cast<uint32_t *>(tree_mask);
    p.B = B;
    p.n = n;
    p.max_pages = max_pages;
    p.page_size = page_size;
    p.num_pages = num_pages;
    p.max_tree = max_tree;
    p.words = (max_tree + 31) / 32;
    p.status = static_cast<uint32_t *>(workspace);
    cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_);
    ProfScope ps("plan_step", stream);
    const cudaError_t e = launch_step_plan(p, stream);
    return e == cudaSuccess ? ORTHROS_OK : report_error(ORTHROS_ECUDA, "step plan launch: %s", cudaGetErrorString(e));
}

orthros_status orthros_tree_commit(void *k_cache, void *v_cache, int layers, const int32_t *block_table, const int32_t *q_indptr,
                                   const int32_t *kv_lens, const int32_t *accepted, const int32_t *n_accepted, int most, int B,
                                   int Hkv, int d, orthros_dtype dtype, int max_pages, int page_size, int num_pages,
                                   int32_t *cache_lens, void *workspace, size_t workspace_bytes, orthros_stream_t stream_) {
    clear_error();
    if (orthros_status st = check_pool(B, max_pages, page_size, num_pages); st != ORTHROS_OK) return st;
    if (layers < 1 || layers > 65535) return report_error(ORTHROS_EINVAL, "layers = %d must lie in [1, 65535]", layers);
    if (most < 1 || most > kTreeMaxTokens) return report_error(ORTHROS_EINVAL, "most = %d must lie in [1, %d]", most, kTreeMaxTokens);
    if (Hkv < 1 || Hkv > 65536) return report_error(ORTHROS_EINVAL, "Hkv = %d must lie in [1, 65536]", Hkv);
    if (dtype != ORTHROS_BF16 && dtype != ORTHROS_F32) return report_error(ORTHROS_EINVAL, "unknown dtype %d", (int)dtype);
    if (d != 64 && d != 128) return report_error(ORTHROS_EUNSUPPORTED, "head size d = %d (supported: 64, 128)", d);
    if (orthros_status st = check_workspace(workspace, workspace_bytes); st != ORTHROS_OK) return st;
    const Array all[] = {{"block_table", block_table}, {"q_indptr", q_indptr}, {"kv_lens", kv_lens}, {"accepted", accepted},
                         {"n_accepted", n_accepted}, {"cache_lens", cache_lens}};
    if (orthros_status st = check_arrays(all); st != ORTHROS_OK) return st;
    if (!k_cache || !v_cache || !aligned(k_cache, 16) || !aligned(v_cache, 16))
        return report_error(ORTHROS_EINVAL, "k_cache and v_cache must not be NULL and 16-byte aligned");
    if (cache_lens == kv_lens || cache_lens == n_accepted || cache_lens == q_indptr)
        return report_error(ORTHROS_EINVAL, "cache_lens is written while kv_lens, n_accepted and q_indptr are read: a buffer of its own");
    TreeCommitParams p{};
    p.k_cache = static_cast<uint8_t *>(k_cache);
    p.v_cache = static_cast<uint8_t *>(v_cache);
    p.block_table = block_table;
    p.q_indptr = q_indptr;
    p.kv_lens = kv_lens;
    p.accepted = accepted;
    p.n_accepted = n_accepted;
    p.cache_lens = cache_lens;
    p.layers = layers;
    p.B = B;
    p.most = most;
    p.max_pages = max_pages;
    p.page_size = page_size;
    p.num_pages = num_pages;
    p.row_bytes = Hkv * d * (dtype == ORTHROS_F32 ? 4 : 2);
    p.status = static_cast<uint32_t *>(workspace);
    cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_);
    ProfScope ps("tree_commit", stream);
    const cudaError_t e = launch_tree_commit(p, stream);
    return e == cudaSuccess ? ORTHROS_OK : report_error(ORTHROS_ECUDA, "tree commit launch: %s", cudaGetErrorString(e));
}

}  // extern "C"
