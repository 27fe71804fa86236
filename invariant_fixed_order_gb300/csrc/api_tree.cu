// C ABI of the operators that serve a tree of drafted tokens: argument
// validation, before any launch.
#include <math.h>

#include <string>

#include "common.cuh"
#include "internal.h"

using namespace bi;

namespace {
bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
bool aligned16(const void* p) { return aligned(p, 16); }
constexpr int32_t kMaxPages = 0x7fffffff / BI_PAGE;  // a slot (16 * page + offset) is an int32
constexpr int32_t kMaxTreeHeads = 65535;              // KV heads are a grid's y extent
}  // namespace

static bi_status run_build_slots(const char* name, bool pad, const int32_t* q_len, const int32_t* pos0,
                                 int32_t* page_table, const int32_t* free_pages, int32_t n_free,
                                 const int32_t* free_head, int32_t* free_head_out, const int32_t* depth, int32_t* cu_q,
                                 int32_t* tok_req, int32_t* tok_pos, int32_t* slots, int32_t B, int32_t T,
                                 int32_t max_pages, int32_t num_pages, int32_t* dev_status, bi_stream stream) {
    const auto bad = [name](bi_status st, const char* what) { return fail(st, std::string(name) + what); };
    if (B < 0 || T < 0 || n_free < 0) return bad(BI_ERR_SHAPE, ": negative size");
    if (max_pages <= 0 || num_pages <= 0 || max_pages > kMaxPages || num_pages > kMaxPages)
        return bad(BI_ERR_SHAPE, ": need 0 < max_pages, num_pages < 2^27");
    if (!free_head || !free_head_out || !cu_q || (n_free > 0 && !free_pages) || (B > 0 && (!q_len || !pos0 || !page_table)) ||
        (T > 0 && (!tok_req || !tok_pos || !slots)))
        return bad(BI_ERR_INVALID, ": null pointer");
    const void* all[] = {q_len, pos0, page_table, free_pages, free_head, free_head_out, depth, cu_q, tok_req, tok_pos, slots};
    for (const void* p : all)
        if (!aligned(p, 4)) return bad(BI_ERR_INVALID, ": pointers must be 4-byte aligned");
    cudaError_t e = launch_build_slots(q_len, pos0, page_table, free_pages, n_free, free_head, free_head_out, depth, cu_q,
                                       tok_req, tok_pos, slots, pad, B, T, max_pages, num_pages, dev_status,
                                       static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? BI_OK : cuda_fail(e, (std::string(name) + " launch").c_str());
}

extern "C" bi_status bi_build_slots(const int32_t* q_len, const int32_t* pos0, int32_t* page_table,
                                    const int32_t* free_pages, int32_t n_free, const int32_t* free_head,
                                    int32_t* free_head_out, const int32_t* depth, int32_t* cu_q, int32_t* tok_req,
                                    int32_t* tok_pos, int32_t* slots, int32_t B, int32_t T, int32_t max_pages,
                                    int32_t num_pages, int32_t* dev_status, bi_stream stream) {
    return run_build_slots("bi_build_slots", false, q_len, pos0, page_table, free_pages, n_free, free_head, free_head_out,
                           depth, cu_q, tok_req, tok_pos, slots, B, T, max_pages, num_pages, dev_status, stream);
}

extern "C" bi_status bi_build_slots_padded(const int32_t* q_len, const int32_t* pos0, int32_t* page_table,
                                           const int32_t* free_pages, int32_t n_free, const int32_t* free_head,
                                           int32_t* free_head_out, const int32_t* depth, int32_t* cu_q, int32_t* tok_req,
                                           int32_t* tok_pos, int32_t* slots, int32_t B, int32_t T, int32_t max_pages,
                                           int32_t num_pages, int32_t* dev_status, bi_stream stream) {
    return run_build_slots("bi_build_slots_padded", true, q_len, pos0, page_table, free_pages, n_free, free_head,
                           free_head_out, depth, cu_q, tok_req, tok_pos, slots, B, T, max_pages, num_pages, dev_status,
                           stream);
}

extern "C" bi_status bi_qk_norm_rope_append(const void* qkv, bi_dtype qkv_dtype, const bi_bf16* q_gamma,
                                            const bi_bf16* k_gamma, float eps, const int32_t* tok_pos,
                                            const int32_t* slots, const float* rope_cos, const float* rope_sin,
                                            int32_t max_pos, bi_bf16* q_out, bi_bf16* k_cache, bi_bf16* v_cache,
                                            int32_t num_pages, int32_t T, int32_t H, int32_t Hkv, int32_t Dh,
                                            int32_t* dev_status, bi_stream stream) {
    if (T < 0 || H <= 0 || Hkv <= 0 || max_pos <= 0 || num_pages <= 0 || num_pages > kMaxPages)
        return fail(BI_ERR_SHAPE, "bi_qk_norm_rope_append: bad shape");
    if (Dh <= 0 || Dh % 16 || Dh > 256) return fail(BI_ERR_SHAPE, "bi_qk_norm_rope_append: need Dh % 16 == 0, Dh <= 256");
    if (H > (1 << 20) || Hkv > (1 << 20)) return fail(BI_ERR_SHAPE, "bi_qk_norm_rope_append: too many heads");
    if (qkv_dtype != BI_BF16 && qkv_dtype != BI_F32) return fail(BI_ERR_INVALID, "bi_qk_norm_rope_append: bad dtype");
    if (!(eps >= 0.0f)) return fail(BI_ERR_INVALID, "bi_qk_norm_rope_append: need eps >= 0");
    if (T == 0) return BI_OK;
    if (!qkv || !tok_pos || !slots || !rope_cos || !rope_sin || !q_out || !k_cache || !v_cache)
        return fail(BI_ERR_INVALID, "bi_qk_norm_rope_append: null pointer");
    if (!aligned16(qkv) || !aligned16(q_gamma) || !aligned16(k_gamma) || !aligned16(rope_cos) || !aligned16(rope_sin) ||
        !aligned16(q_out) || !aligned16(k_cache) || !aligned16(v_cache))
        return fail(BI_ERR_INVALID, "bi_qk_norm_rope_append: pointers must be 16-byte aligned");
    cudaError_t e = launch_qk_norm_rope_append(qkv, qkv_dtype == BI_F32, q_gamma, k_gamma, eps, tok_pos, slots, rope_cos,
                                               rope_sin, max_pos, q_out, k_cache, v_cache, num_pages, T, H, Hkv, Dh,
                                               dev_status, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? BI_OK : cuda_fail(e, "bi_qk_norm_rope_append launch");
}

extern "C" size_t bi_tree_attention_workspace_size(int32_t B, int32_t T, int32_t H, int32_t Hkv, int32_t Dh,
                                                   int32_t max_nodes, int32_t max_seq_len) {
    if (B <= 0 || T <= 0 || max_nodes <= 0 || max_nodes > BI_TREE_MAX_NODES || max_seq_len <= 0 ||
        !attention_supported(H, Hkv, Dh))
        return 0;
    return tree_ws_bytes(B, T, H, Hkv, Dh, max_nodes, max_seq_len);
}

extern "C" int32_t bi_tree_attention_segment(int32_t positions, int32_t nodes, int32_t H, int32_t Hkv) {
    if (positions <= 0 || positions > 0x7fffff00 || nodes <= 0 || nodes > BI_TREE_MAX_NODES || nodes > positions ||
        !attention_supported(H, Hkv, 128))
        return 0;
    return tree_segment(positions, nodes, H, Hkv);
}

static bi_status run_tree_attention(const bi_bf16* q, const int32_t* cu_q, const int32_t* pos0,
                                    const uint32_t* tree_mask, int32_t mask_words, const bi_bf16* k_cache,
                                    const bi_bf16* v_cache, const int32_t* page_table, void* out,
                                    bi_dtype out_dtype, int32_t B, int32_t T, int32_t H, int32_t Hkv, int32_t Dh,
                                    int32_t max_pages, int32_t num_pages, int32_t max_nodes, int32_t max_seq_len,
                                    float scale, void* ws, size_t ws_bytes, int32_t* dev_status, bi_stream stream,
                                    uint64_t wait_ns, int32_t skip_copy) {
    if (B < 0 || T < 0) return fail(BI_ERR_SHAPE, "bi_tree_attention: negative size");
    if (!attention_supported(H, Hkv, Dh))
        return fail(BI_ERR_UNSUPPORTED, "bi_tree_attention: need Dh in {64,128} and H/Hkv in {1,2,4,8}");
    if (Hkv > kMaxTreeHeads) return fail(BI_ERR_SHAPE, "bi_tree_attention: need Hkv <= 65535");
    if (max_nodes <= 0 || max_nodes > BI_TREE_MAX_NODES || mask_words < (max_nodes + 31) / 32)
        return fail(BI_ERR_SHAPE, "bi_tree_attention: need 0 < max_nodes <= 256 and mask_words * 32 >= max_nodes");
    if (max_pages <= 0 || num_pages <= 0 || max_pages > kMaxPages || num_pages > kMaxPages)
        return fail(BI_ERR_SHAPE, "bi_tree_attention: need 0 < max_pages, num_pages < 2^27");
    if (static_cast<int64_t>(num_pages) * Hkv * BI_PAGE > 0x7fffffffLL)
        return fail(BI_ERR_SHAPE, "bi_tree_attention: a cache of 2^31 or more rows (pages x KV heads x 16)");
    if (max_seq_len <= 0 || max_seq_len > max_pages * BI_PAGE)
        return fail(BI_ERR_SHAPE, "bi_tree_attention: need 0 < max_seq_len <= max_pages * 16");
    if (out_dtype != BI_BF16 && out_dtype != BI_F32) return fail(BI_ERR_INVALID, "bi_tree_attention: bad dtype");
    if (B == 0 || T == 0) return BI_OK;
    if (!q || !cu_q || !pos0 || !tree_mask || !k_cache || !v_cache || !page_table || !out)
        return fail(BI_ERR_INVALID, "bi_tree_attention: null pointer");
    if (!aligned16(q) || !aligned16(k_cache) || !aligned16(v_cache) || !aligned16(out))
        return fail(BI_ERR_INVALID, "bi_tree_attention: pointers must be 16-byte aligned");
    const size_t need = tree_ws_bytes(B, T, H, Hkv, Dh, max_nodes, max_seq_len);
    if (need > 0 && (!ws || ws_bytes < need)) return fail(BI_ERR_WORKSPACE, "bi_tree_attention: workspace too small");
    if (!aligned16(ws)) return fail(BI_ERR_INVALID, "bi_tree_attention: workspace must be 16-byte aligned");
    const TreeArgs a{q, k_cache, v_cache, cu_q, pos0, page_table, tree_mask, out, out_dtype == BI_F32, mask_words, B, T,
                     H, Hkv, Dh, max_pages, num_pages, max_nodes, max_seq_len, default_scale(scale, Dh), dev_status,
                     wait_ns, skip_copy};
    cudaError_t e = launch_tree_attention(a, ws, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? BI_OK : cuda_fail(e, "bi_tree_attention launch");
}

extern "C" bi_status bi_tree_attention(const bi_bf16* q, const int32_t* cu_q, const int32_t* pos0,
                                       const uint32_t* tree_mask, int32_t mask_words, const bi_bf16* k_cache,
                                       const bi_bf16* v_cache, const int32_t* page_table, void* out,
                                       bi_dtype out_dtype, int32_t B, int32_t T, int32_t H, int32_t Hkv, int32_t Dh,
                                       int32_t max_pages, int32_t num_pages, int32_t max_nodes, int32_t max_seq_len,
                                       float scale, void* ws, size_t ws_bytes, int32_t* dev_status, bi_stream stream) {
    return run_tree_attention(q, cu_q, pos0, tree_mask, mask_words, k_cache, v_cache, page_table, out, out_dtype, B, T, H,
                              Hkv, Dh, max_pages, num_pages, max_nodes, max_seq_len, scale, ws, ws_bytes, dev_status,
                              stream, kWaitLimitNs, -1);
}

extern "C" bi_status bi_tree_attention_wait_test(const bi_bf16* q, const int32_t* cu_q, const int32_t* pos0,
                                                 const uint32_t* tree_mask, int32_t mask_words, const bi_bf16* k_cache,
                                                 const bi_bf16* v_cache, const int32_t* page_table, void* out,
                                                 bi_dtype out_dtype, int32_t B, int32_t T, int32_t H, int32_t Hkv,
                                                 int32_t Dh, int32_t max_pages, int32_t num_pages, int32_t max_nodes,
                                                 int32_t max_seq_len, float scale, void* ws, size_t ws_bytes,
                                                 uint64_t wait_limit_ns, int32_t skip_copy, int32_t* dev_status,
                                                 bi_stream stream) {
    if (!dev_status) return fail(BI_ERR_INVALID, "bi_tree_attention_wait_test: needs dev_status");
    if (wait_limit_ns < 1000000ull || wait_limit_ns > kWaitLimitNs)
        return fail(BI_ERR_INVALID, "bi_tree_attention_wait_test: wait limit outside [1 ms, 2 s]");
    return run_tree_attention(q, cu_q, pos0, tree_mask, mask_words, k_cache, v_cache, page_table, out, out_dtype, B, T, H,
                              Hkv, Dh, max_pages, num_pages, max_nodes, max_seq_len, scale, ws, ws_bytes, dev_status,
                              stream, wait_limit_ns, skip_copy);
}

extern "C" size_t bi_token_logprobs_workspace_size(int32_t R, int32_t V, int32_t K) {
    return token_logprobs_ws_bytes(R, V, K);
}

extern "C" bi_status bi_token_logprobs(const void* logits, bi_dtype logits_dtype, int64_t row_stride,
                                       const int32_t* tokens, float* logprobs, float* entropy, int32_t* top_ids,
                                       float* top_logprobs, int32_t R, int32_t V, int32_t P, int32_t K, void* ws,
                                       size_t ws_bytes, int32_t* dev_status, bi_stream stream) {
    if (R < 0 || V <= 0 || P < 0) return fail(BI_ERR_SHAPE, "bi_token_logprobs: need R >= 0, V > 0, P >= 0");
    if (row_stride < V) return fail(BI_ERR_SHAPE, "bi_token_logprobs: row stride below V");
    if (K < 0 || K > BI_LOGPROBS_MAX_TOP || K > V) return fail(BI_ERR_SHAPE, "bi_token_logprobs: need 0 <= K <= min(32, V)");
    if (static_cast<int64_t>(K) * ((static_cast<int64_t>(V) + 4095) / 4096) > 4096)
        return fail(BI_ERR_SHAPE, "bi_token_logprobs: need K * ceil(V / 4096) <= 4096");
    if (logits_dtype != BI_BF16 && logits_dtype != BI_F32) return fail(BI_ERR_INVALID, "bi_token_logprobs: bad dtype");
    if (R == 0) return BI_OK;
    if (!logits || (P > 0 && (!tokens || !logprobs)) || (K > 0 && (!top_ids || !top_logprobs)))
        return fail(BI_ERR_INVALID, "bi_token_logprobs: null pointer");
    if (!aligned(logits, logits_dtype == BI_F32 ? 4 : 2)) return fail(BI_ERR_INVALID, "bi_token_logprobs: misaligned logits");
    if (!ws || ws_bytes < token_logprobs_ws_bytes(R, V, K) || !aligned16(ws))
        return fail(BI_ERR_WORKSPACE, "bi_token_logprobs: workspace too small or not 16-byte aligned");
    cudaError_t e = launch_token_logprobs(logits, logits_dtype == BI_F32, row_stride, tokens, logprobs, entropy, top_ids,
                                          top_logprobs, R, V, P, K, ws, dev_status, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? BI_OK : cuda_fail(e, "bi_token_logprobs launch");
}
