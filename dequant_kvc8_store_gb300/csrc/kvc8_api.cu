// kvc8_api.cu -- the extern "C" entry points of libkvc8 (declared in kvc8.h):
// host-side argument checks, then the launches in kvc8_store.cu,
// kvc8_gather.cu, kvc8_bf16.cu, kvc8_attention.cu, kvc8_rope.cu, kvc8_prefix.cu, kvc8_blocks.cu,
// kvc8_tree.cu and kvc8_compact.cu.  Nothing here allocates device memory or synchronises,
// except kvc8_get_error, whose purpose is to synchronise.
#include <cmath>
#include <cstdint>

#include "kvc8_internal.cuh"

namespace kvc8 {

int sm_count() {
    static std::atomic<int> cached[kMaxDevices];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return 1;
    const bool in_range = dev >= 0 && dev < kMaxDevices;
    if (in_range) {
        const int c = cached[dev].load(std::memory_order_relaxed);
        if (c > 0) return c;
    }
    int n = 0;
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n < 1)
        n = 1;
    if (in_range) cached[dev].store(n, std::memory_order_relaxed);
    return n;
}

namespace {

constexpr int kMaxHeadDim = 256;
constexpr int kMaxRopeHeads = 1 << 16;  // heads of a token: row indices stay far inside 32 bits
// Appended rows (tokens x 2 x kv_heads) up to which the fused append + gather
// beats the store followed by a gather (measured on decode-shaped batches:
// 16 384 rows still won, 65 536 lost).
constexpr int64_t kFusedAppendMaxRows = 16384;

bool aligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

kvc8_status check_workspace(const kvc8_geom *g, const void *ws, size_t bytes) {
    if (ws == nullptr || !aligned(ws, kAlign)) return KVC8_ERR_WORKSPACE;
    if (bytes < plan_bytes(g->num_seqs)) return KVC8_ERR_WORKSPACE;
    return KVC8_OK;
}

}  // namespace

kvc8_status check_geom(const kvc8_geom *g) {
    if (g == nullptr) return KVC8_ERR_INVALID_ARG;
    if (g->num_seqs < 0 || g->kv_heads < 1 || g->block_size < 1 || g->num_blocks < 1 ||
        g->max_blocks_per_seq < 1 || g->head_dim < 16)
        return KVC8_ERR_INVALID_ARG;
    if (g->quant_mode < 0 || g->quant_mode > 2) return KVC8_ERR_INVALID_ARG;
    if (g->head_dim % 16 != 0) return KVC8_ERR_INVALID_ARG;
    if (g->head_dim > kMaxHeadDim) return KVC8_ERR_UNSUPPORTED;
    // tile and unit counters are 32/64-bit; keep B * MB * 2H well inside int64
    if ((int64_t)g->num_seqs * g->max_blocks_per_seq > (int64_t)INT32_MAX) return KVC8_ERR_UNSUPPORTED;
    return KVC8_OK;
}

kvc8_status check_gather_args(const kvc8_geom *g, const int8_t *kc, const int8_t *vc,
                              const float *ks, const float *vs, const int32_t *bt,
                              const int32_t *lens, const void *ko, const void *vo,
                              int64_t out_rows, int64_t tok_stride, int64_t head_stride) {
    if (kc == nullptr || vc == nullptr || ks == nullptr || vs == nullptr || bt == nullptr ||
        lens == nullptr || ko == nullptr || vo == nullptr)
        return KVC8_ERR_INVALID_ARG;
    if (out_rows < 0 || tok_stride < 0 || head_stride < 0) return KVC8_ERR_INVALID_ARG;
    if (tok_stride % 8 != 0 || head_stride % 8 != 0) return KVC8_ERR_INVALID_ARG;
    if (!aligned(ko, 16) || !aligned(vo, 16) || !aligned(kc, 16) || !aligned(vc, 16))
        return KVC8_ERR_INVALID_ARG;
    if (!aligned(ks, 16) || !aligned(vs, 16)) return KVC8_ERR_INVALID_ARG;
    return KVC8_OK;
}

}  // namespace kvc8

using namespace kvc8;

extern "C" {

const char *kvc8_status_str(kvc8_status s) {
    switch (s) {
        case KVC8_OK: return "ok";
        case KVC8_ERR_INVALID_ARG: return "invalid argument";
        case KVC8_ERR_UNSUPPORTED: return "unsupported geometry";
        case KVC8_ERR_CUDA: return "CUDA error";
        case KVC8_ERR_DEVICE_BOUNDS: return "device-side bounds error";
        case KVC8_ERR_WORKSPACE: return "workspace missing, too small or misaligned";
    }
    return "unknown status";
}

int32_t kvc8_version(void) { return 10200; }

kvc8_status kvc8_store(const kvc8_geom *g, int64_t num_tokens, const void *key_states,
                       const void *value_states, int64_t x_tok_stride, int64_t x_head_stride,
                       int8_t *key_cache, int8_t *value_cache, float *key_scale,
                       float *value_scale, const int32_t *block_table, const int32_t *cu_q_lens,
                       const int32_t *context_kv_lens, int32_t *dev_error, cudaStream_t stream) {
    kvc8_status st = check_geom(g);
    if (st != KVC8_OK) return st;
    if (num_tokens < 0) return KVC8_ERR_INVALID_ARG;
    if (num_tokens > INT32_MAX) return KVC8_ERR_UNSUPPORTED;  // token indices are 32-bit
    if (cu_q_lens == nullptr && num_tokens != g->num_seqs) return KVC8_ERR_INVALID_ARG;
    if (num_tokens == 0 || g->num_seqs == 0) return num_tokens == 0 ? KVC8_OK : KVC8_ERR_INVALID_ARG;
    if (key_states == nullptr || value_states == nullptr || key_cache == nullptr ||
        value_cache == nullptr || key_scale == nullptr || value_scale == nullptr ||
        block_table == nullptr || context_kv_lens == nullptr)
        return KVC8_ERR_INVALID_ARG;
    if (x_tok_stride < 0 || x_head_stride < 0 || x_tok_stride % 8 != 0 || x_head_stride % 8 != 0)
        return KVC8_ERR_INVALID_ARG;
    if (!aligned(key_states, 16) || !aligned(value_states, 16) || !aligned(key_cache, 16) ||
        !aligned(value_cache, 16))
        return KVC8_ERR_INVALID_ARG;
    if (!aligned(key_scale, 16) || !aligned(value_scale, 16)) return KVC8_ERR_INVALID_ARG;
    StoreArgs a;
    a.g = *g;
    a.num_tokens = num_tokens;
    a.k_states = static_cast<const uint16_t *>(key_states);
    a.v_states = static_cast<const uint16_t *>(value_states);
    a.x_tok_stride = x_tok_stride;
    a.x_head_stride = x_head_stride;
    a.k_cache = key_cache;
    a.v_cache = value_cache;
    a.k_scale = key_scale;
    a.v_scale = value_scale;
    a.block_table = block_table;
    a.cu_q_lens = cu_q_lens;
    a.context_kv_lens = context_kv_lens;
    a.dev_error = dev_error;
    a.bs_magic = g->block_size >= 2 ? ~0ull / (unsigned long long)g->block_size + 1ull : 0ull;
    return cuda_status(launch_store(a, stream));
}

// The plan, then room for one int32 per sequence (the spans of a long
// append, which kvc8_append_gather gathers in a second pass).
size_t kvc8_gather_workspace_bytes(const kvc8_geom *g) {
    if (g == nullptr || g->num_seqs < 0) return 0;
    return plan_bytes(g->num_seqs) +
           align_up(sizeof(int32_t) * (size_t)(g->num_seqs > 0 ? g->num_seqs : 1), kAlign);
}

kvc8_status kvc8_build_metadata(const kvc8_geom *g, const int32_t *context_lengths,
                                const int64_t *context_seq_offset, int64_t *offsets_out,
                                void *workspace, size_t workspace_bytes, int32_t *dev_error,
                                cudaStream_t stream) {
    kvc8_status st = check_geom(g);
    if (st != KVC8_OK) return st;
    if (context_lengths == nullptr && g->num_seqs > 0) return KVC8_ERR_INVALID_ARG;
    st = check_workspace(g, workspace, workspace_bytes);
    if (st != KVC8_OK) return st;
    return cuda_status(launch_plan(*g, context_lengths, context_seq_offset, offsets_out,
                                   workspace, dev_error, stream));
}

kvc8_status kvc8_dequant_gather(const kvc8_geom *g, const int8_t *key_cache,
                                const int8_t *value_cache, const float *key_scale,
                                const float *value_scale, const int32_t *block_table,
                                const int32_t *context_lengths,
                                const int64_t *context_seq_offset, void *key_out,
                                void *value_out, int64_t out_rows, int64_t out_tok_stride,
                                int64_t out_head_stride, void *workspace,
                                size_t workspace_bytes, int32_t *dev_error,
                                cudaStream_t stream) {
    kvc8_status st = check_geom(g);
    if (st != KVC8_OK) return st;
    if (g->num_seqs == 0) return KVC8_OK;
    st = check_gather_args(g, key_cache, value_cache, key_scale, value_scale, block_table,
                           context_lengths, key_out, value_out, out_rows, out_tok_stride,
                           out_head_stride);
    if (st != KVC8_OK) return st;
    st = check_workspace(g, workspace, workspace_bytes);
    if (st != KVC8_OK) return st;
    cudaError_t e = launch_plan(*g, context_lengths, context_seq_offset, nullptr, workspace,
                                dev_error, stream);
    if ((st = cuda_status(e)) != KVC8_OK) return st;
    GatherArgs a;
    a.g = *g;
    a.k_cache = key_cache;
    a.v_cache = value_cache;
    a.k_scale = key_scale;
    a.v_scale = value_scale;
    a.block_table = block_table;
    a.context_lengths = context_lengths;
    a.k_out = static_cast<uint16_t *>(key_out);
    a.v_out = static_cast<uint16_t *>(value_out);
    a.out_rows = out_rows;
    a.out_tok_stride = out_tok_stride;
    a.out_head_stride = out_head_stride;
    a.plan = workspace;
    a.dev_error = dev_error;
    return cuda_status(launch_gather(a, /*use_pdl=*/true, stream));
}

kvc8_status kvc8_dequant_gather_planned(const kvc8_geom *g, const int8_t *key_cache,
                                        const int8_t *value_cache, const float *key_scale,
                                        const float *value_scale, const int32_t *block_table,
                                        const int32_t *context_lengths, void *key_out,
                                        void *value_out, int64_t out_rows,
                                        int64_t out_tok_stride, int64_t out_head_stride,
                                        void *workspace, size_t workspace_bytes,
                                        int32_t *dev_error, cudaStream_t stream) {
    kvc8_status st = check_geom(g);
    if (st != KVC8_OK) return st;
    if (g->num_seqs == 0) return KVC8_OK;
    st = check_gather_args(g, key_cache, value_cache, key_scale, value_scale, block_table,
                           context_lengths, key_out, value_out, out_rows, out_tok_stride,
                           out_head_stride);
    if (st != KVC8_OK) return st;
    st = check_workspace(g, workspace, workspace_bytes);
    if (st != KVC8_OK) return st;
    GatherArgs a;
    a.g = *g;
    a.k_cache = key_cache;
    a.v_cache = value_cache;
    a.k_scale = key_scale;
    a.v_scale = value_scale;
    a.block_table = block_table;
    a.context_lengths = context_lengths;
    a.k_out = static_cast<uint16_t *>(key_out);
    a.v_out = static_cast<uint16_t *>(value_out);
    a.out_rows = out_rows;
    a.out_tok_stride = out_tok_stride;
    a.out_head_stride = out_head_stride;
    a.plan = workspace;
    a.dev_error = dev_error;
    if ((st = cuda_status(reset_plan_counter(workspace, stream))) != KVC8_OK) return st;
    return cuda_status(launch_gather(a, /*use_pdl=*/false, stream));
}

// Shared checks and argument packing of the append + gather entry points.
static kvc8_status append_args(const kvc8_geom *g, int64_t num_tokens, const void *key_states,
                               const void *value_states, int64_t x_tok_stride,
                               int64_t x_head_stride, int8_t *key_cache, int8_t *value_cache,
                               float *key_scale, float *value_scale,
                               const int32_t *block_table, const int32_t *cu_q_lens,
                               const int32_t *context_kv_lens, void *key_out, void *value_out,
                               int64_t out_rows, int64_t out_tok_stride,
                               int64_t out_head_stride, void *workspace,
                               size_t workspace_bytes, int32_t *dev_error, GatherArgs *a,
                               AppendArgs *p) {
    kvc8_status st = check_geom(g);
    if (st != KVC8_OK) return st;
    if (num_tokens < 0) return KVC8_ERR_INVALID_ARG;
    if (num_tokens > INT32_MAX) return KVC8_ERR_UNSUPPORTED;  // token indices are 32-bit
    if (cu_q_lens == nullptr && num_tokens != g->num_seqs) return KVC8_ERR_INVALID_ARG;
    // the fused kernel indexes its work items and appended rows in 32 bits
    if ((int64_t)g->num_seqs * g->max_blocks_per_seq * g->kv_heads > (int64_t)INT32_MAX ||
        num_tokens * 2 * g->kv_heads > (int64_t)INT32_MAX)
        return KVC8_ERR_UNSUPPORTED;
    st = check_gather_args(g, key_cache, value_cache, key_scale, value_scale, block_table,
                           context_kv_lens, key_out, value_out, out_rows, out_tok_stride,
                           out_head_stride);
    if (st != KVC8_OK) return st;
    if (num_tokens > 0) {
        if (key_states == nullptr || value_states == nullptr) return KVC8_ERR_INVALID_ARG;
        if (x_tok_stride < 0 || x_head_stride < 0 || x_tok_stride % 8 != 0 ||
            x_head_stride % 8 != 0)
            return KVC8_ERR_INVALID_ARG;
        if (!aligned(key_states, 16) || !aligned(value_states, 16)) return KVC8_ERR_INVALID_ARG;
    }
    st = check_workspace(g, workspace, workspace_bytes);
    if (st != KVC8_OK) return st;
    a->g = *g;
    a->k_cache = key_cache;
    a->v_cache = value_cache;
    a->k_scale = key_scale;
    a->v_scale = value_scale;
    a->block_table = block_table;
    a->context_lengths = context_kv_lens;  // the gather part reads the cached positions
    a->k_out = static_cast<uint16_t *>(key_out);
    a->v_out = static_cast<uint16_t *>(value_out);
    a->out_rows = out_rows;
    a->out_tok_stride = out_tok_stride;
    a->out_head_stride = out_head_stride;
    a->plan = workspace;
    a->dev_error = dev_error;
    p->num_tokens = num_tokens;
    const int64_t rows = num_tokens * 2 * g->kv_heads;
    p->items = (rows + kAppendRowsPerItem - 1) / kAppendRowsPerItem;
    p->k_states = static_cast<const uint16_t *>(key_states);
    p->v_states = static_cast<const uint16_t *>(value_states);
    p->x_tok_stride = x_tok_stride;
    p->x_head_stride = x_head_stride;
    p->k_cache = key_cache;
    p->v_cache = value_cache;
    p->k_scale = key_scale;
    p->v_scale = value_scale;
    p->cu_q_lens = cu_q_lens;
    p->context_kv_lens = context_kv_lens;
    return KVC8_OK;
}

kvc8_status kvc8_append_gather(const kvc8_geom *g, int64_t num_tokens, const void *key_states,
                               const void *value_states, int64_t x_tok_stride,
                               int64_t x_head_stride, int8_t *key_cache, int8_t *value_cache,
                               float *key_scale, float *value_scale,
                               const int32_t *block_table, const int32_t *cu_q_lens,
                               const int32_t *context_kv_lens,
                               const int64_t *context_seq_offset, void *key_out,
                               void *value_out, int64_t out_rows, int64_t out_tok_stride,
                               int64_t out_head_stride, void *workspace,
                               size_t workspace_bytes, int32_t *dev_error, cudaStream_t stream) {
    if (g != nullptr && g->num_seqs == 0 && check_geom(g) == KVC8_OK)
        return num_tokens == 0 ? KVC8_OK : KVC8_ERR_INVALID_ARG;
    GatherArgs a;
    AppendArgs p;
    kvc8_status st = append_args(g, num_tokens, key_states, value_states, x_tok_stride,
                                 x_head_stride, key_cache, value_cache, key_scale, value_scale,
                                 block_table, cu_q_lens, context_kv_lens, key_out, value_out,
                                 out_rows, out_tok_stride, out_head_stride, workspace,
                                 workspace_bytes, dev_error, &a, &p);
    if (st != KVC8_OK) return st;
    // A long append (a prompt rather than a decode step) is faster as the
    // store kernel followed by a gather of every position: the fused kernel's
    // append rows follow the definition with one division per value.
    const size_t span_at = plan_bytes(g->num_seqs);
    const bool long_append =
        num_tokens * 2 * g->kv_heads > kFusedAppendMaxRows &&
        workspace_bytes >= span_at + sizeof(int32_t) * (size_t)g->num_seqs;
    if (long_append) {
        StoreArgs s;
        s.g = *g;
        s.num_tokens = num_tokens;
        s.k_states = p.k_states;
        s.v_states = p.v_states;
        s.x_tok_stride = x_tok_stride;
        s.x_head_stride = x_head_stride;
        s.k_cache = key_cache;
        s.v_cache = value_cache;
        s.k_scale = key_scale;
        s.v_scale = value_scale;
        s.block_table = block_table;
        s.cu_q_lens = cu_q_lens;
        s.context_kv_lens = context_kv_lens;
        s.dev_error = dev_error;
        s.bs_magic = g->block_size >= 2 ? ~0ull / (unsigned long long)g->block_size + 1ull : 0ull;
        if ((st = cuda_status(launch_store(s, stream))) != KVC8_OK) return st;
        int32_t *spans = reinterpret_cast<int32_t *>(static_cast<char *>(workspace) + span_at);
        st = cuda_status(launch_plan_span(*g, context_kv_lens, cu_q_lens, context_seq_offset, workspace, spans,
                                          dev_error, stream));
        if (st != KVC8_OK) return st;
        a.context_lengths = spans;
        return cuda_status(launch_gather(a, /*use_pdl=*/true, stream));
    }
    st = cuda_status(launch_plan_append(*g, context_kv_lens, cu_q_lens, context_seq_offset, nullptr,
                                        workspace, dev_error, stream));
    if (st != KVC8_OK) return st;
    return cuda_status(launch_append_gather(a, p, /*use_pdl=*/true, stream));
}

kvc8_status kvc8_build_append_metadata(const kvc8_geom *g, const int32_t *cu_q_lens,
                                       const int32_t *context_kv_lens,
                                       const int64_t *context_seq_offset, int64_t *offsets_out,
                                       void *workspace, size_t workspace_bytes,
                                       int32_t *dev_error, cudaStream_t stream) {
    kvc8_status st = check_geom(g);
    if (st != KVC8_OK) return st;
    if (context_kv_lens == nullptr && g->num_seqs > 0) return KVC8_ERR_INVALID_ARG;
    st = check_workspace(g, workspace, workspace_bytes);
    if (st != KVC8_OK) return st;
    return cuda_status(launch_plan_append(*g, context_kv_lens, cu_q_lens, context_seq_offset,
                                          offsets_out, workspace, dev_error, stream));
}

kvc8_status kvc8_append_gather_planned(const kvc8_geom *g, int64_t num_tokens,
                                       const void *key_states, const void *value_states,
                                       int64_t x_tok_stride, int64_t x_head_stride,
                                       int8_t *key_cache, int8_t *value_cache, float *key_scale,
                                       float *value_scale, const int32_t *block_table,
                                       const int32_t *cu_q_lens, const int32_t *context_kv_lens,
                                       void *key_out, void *value_out, int64_t out_rows,
                                       int64_t out_tok_stride, int64_t out_head_stride,
                                       void *workspace, size_t workspace_bytes,
                                       int32_t *dev_error, cudaStream_t stream) {
    if (g != nullptr && g->num_seqs == 0 && check_geom(g) == KVC8_OK)
        return num_tokens == 0 ? KVC8_OK : KVC8_ERR_INVALID_ARG;
    GatherArgs a;
    AppendArgs p;
    kvc8_status st = append_args(g, num_tokens, key_states, value_states, x_tok_stride,
                                 x_head_stride, key_cache, value_cache, key_scale, value_scale,
                                 block_table, cu_q_lens, context_kv_lens, key_out, value_out,
                                 out_rows, out_tok_stride, out_head_stride, workspace,
                                 workspace_bytes, dev_error, &a, &p);
    if (st != KVC8_OK) return st;
    if ((st = cuda_status(reset_plan_counter(workspace, stream))) != KVC8_OK) return st;
    return cuda_status(launch_append_gather(a, p, /*use_pdl=*/false, stream));
}

size_t kvc8_attention_workspace_bytes(const kvc8_geom *g, int32_t num_q_heads) {
    if (g == nullptr || g->num_seqs < 0 || g->kv_heads < 1 || num_q_heads < g->kv_heads) return 0;
    return attention_workspace_bytes(*g, num_q_heads / g->kv_heads);
}

kvc8_status kvc8_paged_decode_attention(const kvc8_geom *g, int32_t num_q_heads,
                                        const void *query, int64_t q_seq_stride,
                                        int64_t q_head_stride, const int8_t *key_cache,
                                        const int8_t *value_cache, const float *key_scale,
                                        const float *value_scale, const int32_t *block_table,
                                        const int32_t *context_lengths, float softmax_scale,
                                        void *out, int64_t out_seq_stride,
                                        int64_t out_head_stride, void *workspace,
                                        size_t workspace_bytes, int32_t *dev_error,
                                        cudaStream_t stream) {
    kvc8_status st = check_geom(g);
    if (st != KVC8_OK) return st;
    if (num_q_heads < 1 || num_q_heads % g->kv_heads != 0) return KVC8_ERR_INVALID_ARG;
    const int group = num_q_heads / g->kv_heads;
    if (group > 8 || (g->head_dim != 64 && g->head_dim != 128) || g->block_size % 16 != 0)
        return KVC8_ERR_UNSUPPORTED;
    if (!std::isfinite(softmax_scale)) return KVC8_ERR_INVALID_ARG;
    const int64_t splits =
        ((int64_t)g->max_blocks_per_seq * g->block_size + kAttnChunk - 1) / kAttnChunk;
    if ((int64_t)g->num_seqs * g->kv_heads * splits > (int64_t)INT32_MAX) return KVC8_ERR_UNSUPPORTED;
    if (g->num_seqs == 0) return KVC8_OK;
    if (query == nullptr || key_cache == nullptr || value_cache == nullptr ||
        key_scale == nullptr || value_scale == nullptr || block_table == nullptr ||
        context_lengths == nullptr || out == nullptr)
        return KVC8_ERR_INVALID_ARG;
    if (q_seq_stride < 0 || q_head_stride < 0 || q_seq_stride % 8 != 0 || q_head_stride % 8 != 0 ||
        out_seq_stride < 0 || out_head_stride < 0)
        return KVC8_ERR_INVALID_ARG;
    if (!aligned(query, 16) || !aligned(key_cache, 16) || !aligned(value_cache, 16) ||
        !aligned(key_scale, 16) || !aligned(value_scale, 16) || !aligned(out, 2))
        return KVC8_ERR_INVALID_ARG;
    if (workspace == nullptr || !aligned(workspace, kAlign) ||
        workspace_bytes < attention_workspace_bytes(*g, group))
        return KVC8_ERR_WORKSPACE;
    AttnArgs a = {};
    a.g = *g;
    a.group = group;
    a.q = static_cast<const uint16_t *>(query);
    a.q_seq_stride = q_seq_stride;
    a.q_head_stride = q_head_stride;
    a.k_cache = key_cache;
    a.v_cache = value_cache;
    a.k_scale = key_scale;
    a.v_scale = value_scale;
    a.block_table = block_table;
    a.context_lengths = context_lengths;
    a.scale_log2 = (float)((double)softmax_scale * 1.4426950408889634);  // log2(e)
    a.out = static_cast<uint16_t *>(out);
    a.out_seq_stride = out_seq_stride;
    a.out_head_stride = out_head_stride;
    a.dev_error = dev_error;
    return cuda_status(launch_attention(a, workspace, stream));
}

// Geometry checks for the bf16 cache (quant_mode is not used there).
static kvc8_status check_geom_bf16(const kvc8_geom *g) {
    if (g == nullptr) return KVC8_ERR_INVALID_ARG;
    kvc8_geom q = *g;
    q.quant_mode = 0;
    return check_geom(&q);
}

kvc8_status kvc8_store_bf16(const kvc8_geom *g, int64_t num_tokens, const void *key_states,
                            const void *value_states, int64_t x_tok_stride, int64_t x_head_stride,
                            void *key_cache, void *value_cache, const int32_t *block_table,
                            const int32_t *cu_q_lens, const int32_t *context_kv_lens,
                            int32_t *dev_error, cudaStream_t stream) {
    kvc8_status st = check_geom_bf16(g);
    if (st != KVC8_OK) return st;
    if (num_tokens < 0) return KVC8_ERR_INVALID_ARG;
    if (num_tokens > INT32_MAX) return KVC8_ERR_UNSUPPORTED;
    if (cu_q_lens == nullptr && num_tokens != g->num_seqs) return KVC8_ERR_INVALID_ARG;
    if (num_tokens == 0 || g->num_seqs == 0) return num_tokens == 0 ? KVC8_OK : KVC8_ERR_INVALID_ARG;
    if (key_states == nullptr || value_states == nullptr || key_cache == nullptr ||
        value_cache == nullptr || block_table == nullptr || context_kv_lens == nullptr)
        return KVC8_ERR_INVALID_ARG;
    if (x_tok_stride < 0 || x_head_stride < 0 || x_tok_stride % 8 != 0 || x_head_stride % 8 != 0)
        return KVC8_ERR_INVALID_ARG;
    if (!aligned(key_states, 16) || !aligned(value_states, 16) || !aligned(key_cache, 16) ||
        !aligned(value_cache, 16))
        return KVC8_ERR_INVALID_ARG;
    StoreBf16Args a;
    a.g = *g;
    a.num_tokens = num_tokens;
    a.k_states = static_cast<const uint16_t *>(key_states);
    a.v_states = static_cast<const uint16_t *>(value_states);
    a.x_tok_stride = x_tok_stride;
    a.x_head_stride = x_head_stride;
    a.k_cache = static_cast<uint16_t *>(key_cache);
    a.v_cache = static_cast<uint16_t *>(value_cache);
    a.block_table = block_table;
    a.cu_q_lens = cu_q_lens;
    a.context_kv_lens = context_kv_lens;
    a.dev_error = dev_error;
    return cuda_status(launch_store_bf16(a, stream));
}

kvc8_status kvc8_gather_bf16(const kvc8_geom *g, const void *key_cache, const void *value_cache,
                             const int32_t *block_table, const int32_t *context_lengths,
                             const int64_t *context_seq_offset, void *key_out, void *value_out,
                             int64_t out_rows, int64_t out_tok_stride, int64_t out_head_stride,
                             void *workspace, size_t workspace_bytes, int32_t *dev_error,
                             cudaStream_t stream) {
    kvc8_status st = check_geom_bf16(g);
    if (st != KVC8_OK) return st;
    if (g->num_seqs == 0) return KVC8_OK;
    if (key_cache == nullptr || value_cache == nullptr || block_table == nullptr ||
        context_lengths == nullptr || key_out == nullptr || value_out == nullptr)
        return KVC8_ERR_INVALID_ARG;
    if (out_rows < 0 || out_tok_stride < 0 || out_head_stride < 0 || out_tok_stride % 8 != 0 ||
        out_head_stride % 8 != 0)
        return KVC8_ERR_INVALID_ARG;
    if (!aligned(key_out, 16) || !aligned(value_out, 16) || !aligned(key_cache, 16) ||
        !aligned(value_cache, 16))
        return KVC8_ERR_INVALID_ARG;
    kvc8_geom q = *g;
    q.quant_mode = 0;
    st = check_workspace(&q, workspace, workspace_bytes);
    if (st != KVC8_OK) return st;
    st = cuda_status(launch_plan(q, context_lengths, context_seq_offset, nullptr, workspace, dev_error,
                                 stream));
    if (st != KVC8_OK) return st;
    GatherBf16Args a;
    a.g = q;
    a.k_cache = static_cast<const uint16_t *>(key_cache);
    a.v_cache = static_cast<const uint16_t *>(value_cache);
    a.block_table = block_table;
    a.context_lengths = context_lengths;
    a.k_out = static_cast<uint16_t *>(key_out);
    a.v_out = static_cast<uint16_t *>(value_out);
    a.out_rows = out_rows;
    a.out_tok_stride = out_tok_stride;
    a.out_head_stride = out_head_stride;
    a.plan = workspace;
    a.dev_error = dev_error;
    return cuda_status(launch_gather_bf16(a, /*use_pdl=*/true, stream));
}

kvc8_status kvc8_rope_frequencies(const kvc8_rope_scaling *s, int32_t rotary_dim, uint64_t *freqs,
                                  float *attention_factor) {
    if (s == nullptr || rotary_dim < 0 || rotary_dim % 2 != 0) return KVC8_ERR_INVALID_ARG;
    if (rotary_dim > 0 && freqs == nullptr) return KVC8_ERR_INVALID_ARG;
    if (s->kind < KVC8_ROPE_PLAIN || s->kind > KVC8_ROPE_BY_PARTS) return KVC8_ERR_INVALID_ARG;
    if (!std::isfinite(s->base) || !(s->base > 0.0)) return KVC8_ERR_INVALID_ARG;
    if (s->kind != KVC8_ROPE_PLAIN && (!std::isfinite(s->factor) || !(s->factor > 0.0)))
        return KVC8_ERR_INVALID_ARG;
    if (s->kind == KVC8_ROPE_BASE && rotary_dim == 2) return KVC8_ERR_INVALID_ARG;  // one pair
    const bool parts = s->kind == KVC8_ROPE_BY_PARTS;
    if (parts && (!std::isfinite(s->original_positions) || !(s->original_positions > 0.0) ||
                  !std::isfinite(s->low) || !std::isfinite(s->high) || !(s->low < s->high)))
        return KVC8_ERR_INVALID_ARG;
    const double two_pi = 6.283185307179586;
    const double R = rotary_dim;
    double base = s->base;
    if (s->kind == KVC8_ROPE_BASE && rotary_dim > 2) base *= std::pow(s->factor, R / (R - 2.0));
    for (int i = 0; i < rotary_dim / 2; ++i) {
        double f = std::pow(base, -2.0 * i / R);
        if (s->kind == KVC8_ROPE_LINEAR) f /= s->factor;
        if (parts) {
            const double r = s->original_positions * f / two_pi;
            const double g = std::fmin(1.0, std::fmax(0.0, (r - s->low) / (s->high - s->low)));
            f = f / s->factor * (1.0 - g) + f * g;
        }
        if (!std::isfinite(f)) return KVC8_ERR_INVALID_ARG;
        double turns = f / two_pi;
        turns -= std::floor(turns);  // whole turns per position change nothing
        const double scaled = std::rint(std::ldexp(turns, 64));
        freqs[i] = scaled < 18446744073709551616.0 ? (uint64_t)scaled : 0;
    }
    if (attention_factor != nullptr)
        *attention_factor = parts && s->factor > 1.0 ? (float)(0.1 * std::log(s->factor) + 1.0) : 1.0f;
    return KVC8_OK;
}

// Checks of a rotation over heads of D channels, packed into the kernel's
// arguments.
static kvc8_status rope_args(const kvc8_rope *r, int32_t head_dim, RopeArgs *a) {
    if (r == nullptr) return KVC8_ERR_INVALID_ARG;
    if (r->rotary_dim < 0 || r->rotary_dim > head_dim || r->rotary_dim % 2 != 0)
        return KVC8_ERR_INVALID_ARG;
    if (r->rotary_dim % 16 != 0) return KVC8_ERR_UNSUPPORTED;
    if (r->interleaved != 0 && r->interleaved != 1) return KVC8_ERR_INVALID_ARG;
    if (!std::isfinite(r->attention_factor)) return KVC8_ERR_INVALID_ARG;
    if (r->rotary_dim > 0 && (r->freqs == nullptr || !aligned(r->freqs, 8)))
        return KVC8_ERR_INVALID_ARG;
    if (!aligned(r->q_norm_weight, 16) || !aligned(r->k_norm_weight, 16) ||
        !aligned(r->positions, 4))
        return KVC8_ERR_INVALID_ARG;
    if ((r->q_norm_weight != nullptr || r->k_norm_weight != nullptr) &&
        (!std::isfinite(r->norm_eps) || r->norm_eps < 0.0f))
        return KVC8_ERR_INVALID_ARG;
    a->rotary_dim = r->rotary_dim;
    a->interleaved = r->interleaved;
    a->factor = r->attention_factor;
    a->eps = r->norm_eps;
    a->freqs = r->freqs;
    a->q_weight = static_cast<const uint16_t *>(r->q_norm_weight);
    a->k_weight = static_cast<const uint16_t *>(r->k_norm_weight);
    a->positions = r->positions;
    return KVC8_OK;
}

// A side of bf16 rows in and out: both given, aligned, strides multiples of 8.
static kvc8_status rope_rows(const void *in, int64_t ts, int64_t hs, const void *out, int64_t ots,
                             int64_t ohs) {
    if (in == nullptr || out == nullptr || !aligned(in, 16) || !aligned(out, 16))
        return KVC8_ERR_INVALID_ARG;
    for (int64_t s : {ts, hs, ots, ohs})
        if (s < 0 || s % 8 != 0) return KVC8_ERR_INVALID_ARG;
    return KVC8_OK;
}

// Checks and packing shared by the two rotating stores (everything but the scales).
static kvc8_status rope_store_args(const kvc8_geom *g, const kvc8_rope *r, int64_t num_tokens,
                                   int32_t num_q_heads, const void *query, int64_t q_tok_stride,
                                   int64_t q_head_stride, void *q_out, int64_t qo_tok_stride,
                                   int64_t qo_head_stride, const void *key_states,
                                   const void *value_states, int64_t x_tok_stride,
                                   int64_t x_head_stride, void *key_cache, void *value_cache,
                                   const int32_t *block_table, const int32_t *cu_q_lens,
                                   const int32_t *context_kv_lens, int32_t *dev_error,
                                   RopeArgs *a) {
    kvc8_status st = rope_args(r, g->head_dim, a);
    if (st != KVC8_OK) return st;
    if (num_tokens < 0 || num_q_heads < 0) return KVC8_ERR_INVALID_ARG;
    if (num_tokens > INT32_MAX) return KVC8_ERR_UNSUPPORTED;  // token indices are 32-bit
    if (num_q_heads > kMaxRopeHeads || g->kv_heads > kMaxRopeHeads) return KVC8_ERR_UNSUPPORTED;
    if (cu_q_lens == nullptr && num_tokens != g->num_seqs) return KVC8_ERR_INVALID_ARG;
    if (num_tokens > 0 && g->num_seqs == 0) return KVC8_ERR_INVALID_ARG;
    a->num_tokens = num_tokens;
    if (num_tokens == 0) return KVC8_OK;
    if (key_states == nullptr || value_states == nullptr || key_cache == nullptr ||
        value_cache == nullptr || block_table == nullptr || context_kv_lens == nullptr)
        return KVC8_ERR_INVALID_ARG;
    if (x_tok_stride < 0 || x_head_stride < 0 || x_tok_stride % 8 != 0 || x_head_stride % 8 != 0)
        return KVC8_ERR_INVALID_ARG;
    if (!aligned(key_states, 16) || !aligned(value_states, 16) || !aligned(key_cache, 16) ||
        !aligned(value_cache, 16))
        return KVC8_ERR_INVALID_ARG;
    if (num_q_heads > 0) {
        st = rope_rows(query, q_tok_stride, q_head_stride, q_out, qo_tok_stride, qo_head_stride);
        if (st != KVC8_OK) return st;
    }
    a->g = *g;
    a->q_heads = num_q_heads;
    a->q = static_cast<const uint16_t *>(query);
    a->q_tok_stride = q_tok_stride;
    a->q_head_stride = q_head_stride;
    a->q_out = static_cast<uint16_t *>(q_out);
    a->qo_tok_stride = qo_tok_stride;
    a->qo_head_stride = qo_head_stride;
    a->k = static_cast<const uint16_t *>(key_states);
    a->v = static_cast<const uint16_t *>(value_states);
    a->x_tok_stride = x_tok_stride;
    a->x_head_stride = x_head_stride;
    a->k_cache = key_cache;
    a->v_cache = value_cache;
    a->block_table = block_table;
    a->cu_q_lens = cu_q_lens;
    a->context_kv_lens = context_kv_lens;
    a->dev_error = dev_error;
    return KVC8_OK;
}

kvc8_status kvc8_rope_store(const kvc8_geom *g, const kvc8_rope *r, int64_t num_tokens,
                            int32_t num_q_heads, const void *query, int64_t q_tok_stride,
                            int64_t q_head_stride, void *q_out, int64_t qo_tok_stride,
                            int64_t qo_head_stride, const void *key_states,
                            const void *value_states, int64_t x_tok_stride,
                            int64_t x_head_stride, int8_t *key_cache, int8_t *value_cache,
                            float *key_scale, float *value_scale, const int32_t *block_table,
                            const int32_t *cu_q_lens, const int32_t *context_kv_lens,
                            int32_t *dev_error, cudaStream_t stream) {
    kvc8_status st = check_geom(g);
    if (st != KVC8_OK) return st;
    RopeArgs a = {};
    st = rope_store_args(g, r, num_tokens, num_q_heads, query, q_tok_stride, q_head_stride, q_out,
                         qo_tok_stride, qo_head_stride, key_states, value_states, x_tok_stride,
                         x_head_stride, key_cache, value_cache, block_table, cu_q_lens,
                         context_kv_lens, dev_error, &a);
    if (st != KVC8_OK || num_tokens == 0) return st;
    if (key_scale == nullptr || value_scale == nullptr || !aligned(key_scale, 16) ||
        !aligned(value_scale, 16))
        return KVC8_ERR_INVALID_ARG;
    a.k_scale = key_scale;
    a.v_scale = value_scale;
    return cuda_status(launch_rope(a, static_cast<RopeSink>(g->quant_mode), stream));
}

kvc8_status kvc8_rope_store_bf16(const kvc8_geom *g, const kvc8_rope *r, int64_t num_tokens,
                                 int32_t num_q_heads, const void *query, int64_t q_tok_stride,
                                 int64_t q_head_stride, void *q_out, int64_t qo_tok_stride,
                                 int64_t qo_head_stride, const void *key_states,
                                 const void *value_states, int64_t x_tok_stride,
                                 int64_t x_head_stride, void *key_cache, void *value_cache,
                                 const int32_t *block_table, const int32_t *cu_q_lens,
                                 const int32_t *context_kv_lens, int32_t *dev_error,
                                 cudaStream_t stream) {
    kvc8_status st = check_geom_bf16(g);
    if (st != KVC8_OK) return st;
    RopeArgs a = {};
    st = rope_store_args(g, r, num_tokens, num_q_heads, query, q_tok_stride, q_head_stride, q_out,
                         qo_tok_stride, qo_head_stride, key_states, value_states, x_tok_stride,
                         x_head_stride, key_cache, value_cache, block_table, cu_q_lens,
                         context_kv_lens, dev_error, &a);
    if (st != KVC8_OK || num_tokens == 0) return st;
    return cuda_status(launch_rope(a, kSinkBf16, stream));
}

kvc8_status kvc8_qk_norm_rope(const kvc8_rope *r, int64_t num_tokens, int32_t head_dim,
                              int32_t num_q_heads, const void *query, int64_t q_tok_stride,
                              int64_t q_head_stride, void *q_out, int64_t qo_tok_stride,
                              int64_t qo_head_stride, int32_t kv_heads, const void *key,
                              int64_t k_tok_stride, int64_t k_head_stride, void *k_out,
                              int64_t ko_tok_stride, int64_t ko_head_stride,
                              cudaStream_t stream) {
    if (head_dim < 16 || head_dim % 16 != 0) return KVC8_ERR_INVALID_ARG;
    if (head_dim > kMaxHeadDim) return KVC8_ERR_UNSUPPORTED;
    RopeArgs a = {};
    kvc8_status st = rope_args(r, head_dim, &a);
    if (st != KVC8_OK) return st;
    if (num_tokens < 0 || num_q_heads < 0 || kv_heads < 0) return KVC8_ERR_INVALID_ARG;
    if (num_tokens > INT32_MAX || num_q_heads > kMaxRopeHeads || kv_heads > kMaxRopeHeads)
        return KVC8_ERR_UNSUPPORTED;
    if (num_tokens == 0 || (num_q_heads == 0 && kv_heads == 0)) return KVC8_OK;
    if (r->rotary_dim > 0 && r->positions == nullptr) return KVC8_ERR_INVALID_ARG;
    if (num_q_heads > 0) {
        st = rope_rows(query, q_tok_stride, q_head_stride, q_out, qo_tok_stride, qo_head_stride);
        if (st != KVC8_OK) return st;
    }
    if (kv_heads > 0) {
        st = rope_rows(key, k_tok_stride, k_head_stride, k_out, ko_tok_stride, ko_head_stride);
        if (st != KVC8_OK) return st;
    }
    a.g.kv_heads = kv_heads;
    a.g.head_dim = head_dim;
    a.num_tokens = num_tokens;
    a.q_heads = num_q_heads;
    a.q = static_cast<const uint16_t *>(query);
    a.q_tok_stride = q_tok_stride;
    a.q_head_stride = q_head_stride;
    a.q_out = static_cast<uint16_t *>(q_out);
    a.qo_tok_stride = qo_tok_stride;
    a.qo_head_stride = qo_head_stride;
    a.k = static_cast<const uint16_t *>(key);
    a.x_tok_stride = k_tok_stride;
    a.x_head_stride = k_head_stride;
    a.k_out = static_cast<uint16_t *>(k_out);
    a.ko_tok_stride = ko_tok_stride;
    a.ko_head_stride = ko_head_stride;
    return cuda_status(launch_rope(a, kSinkRows, stream));
}

// What kvc8_paged_decode_attention supports, for the prefix form: beside it a
// prefix table, whose positions are 32-bit, as are the query rows of a kv head.
static kvc8_status check_prefix_geom(const kvc8_geom *g, int32_t num_q_heads,
                                     int32_t max_prefix_blocks) {
    kvc8_status st = check_geom(g);
    if (st != KVC8_OK) return st;
    if (num_q_heads < 1 || num_q_heads % g->kv_heads != 0) return KVC8_ERR_INVALID_ARG;
    if (num_q_heads / g->kv_heads > 8 || (g->head_dim != 64 && g->head_dim != 128) ||
        g->block_size % 16 != 0)
        return KVC8_ERR_UNSUPPORTED;
    const int64_t splits =
        ((int64_t)g->max_blocks_per_seq * g->block_size + kAttnChunk - 1) / kAttnChunk;
    if ((int64_t)g->num_seqs * g->kv_heads * splits > (int64_t)INT32_MAX) return KVC8_ERR_UNSUPPORTED;
    if (max_prefix_blocks < 1) return KVC8_ERR_INVALID_ARG;
    // (with room for a step's overhang past the end)
    if ((int64_t)max_prefix_blocks * g->block_size > (int64_t)INT32_MAX - 4096 ||
        (int64_t)g->num_seqs * num_q_heads > (int64_t)INT32_MAX / 2)
        return KVC8_ERR_UNSUPPORTED;
    // units of 128 query rows and 128 positions are counted in 32 bits
    const int64_t rows = (int64_t)g->num_seqs * (num_q_heads / g->kv_heads);
    const int64_t tiles = (rows + 127) / 128 * g->kv_heads;
    const int64_t steps = ((int64_t)max_prefix_blocks * g->block_size + 127) / 128;
    if (tiles > (int64_t)INT32_MAX / steps) return KVC8_ERR_UNSUPPORTED;
    return KVC8_OK;
}

size_t kvc8_shared_prefix_workspace_bytes(const kvc8_geom *g, int32_t num_q_heads,
                                          int32_t max_prefix_blocks) {
    if (check_prefix_geom(g, num_q_heads, max_prefix_blocks) != KVC8_OK) return 0;
    return shared_prefix_workspace_bytes(*g, num_q_heads / g->kv_heads);
}

kvc8_status kvc8_shared_prefix_attention(const kvc8_geom *g, int32_t num_q_heads,
                                         const void *query, int64_t q_seq_stride,
                                         int64_t q_head_stride, const int8_t *key_cache,
                                         const int8_t *value_cache, const float *key_scale,
                                         const float *value_scale, const int32_t *prefix_table,
                                         int32_t max_prefix_blocks,
                                         const int32_t *prefix_length,
                                         const int32_t *block_table,
                                         const int32_t *context_lengths, float softmax_scale,
                                         void *out, int64_t out_seq_stride,
                                         int64_t out_head_stride, void *workspace,
                                         size_t workspace_bytes, int32_t *dev_error,
                                         cudaStream_t stream) {
    kvc8_status st = check_prefix_geom(g, num_q_heads, max_prefix_blocks);
    if (st != KVC8_OK) return st;
    if (!std::isfinite(softmax_scale)) return KVC8_ERR_INVALID_ARG;
    if (g->num_seqs == 0) return KVC8_OK;
    if (query == nullptr || key_cache == nullptr || value_cache == nullptr ||
        key_scale == nullptr || value_scale == nullptr || prefix_table == nullptr ||
        prefix_length == nullptr || block_table == nullptr || context_lengths == nullptr ||
        out == nullptr)
        return KVC8_ERR_INVALID_ARG;
    if (q_seq_stride < 0 || q_head_stride < 0 || q_seq_stride % 8 != 0 || q_head_stride % 8 != 0 ||
        out_seq_stride < 0 || out_head_stride < 0)
        return KVC8_ERR_INVALID_ARG;
    if (!aligned(query, 16) || !aligned(key_cache, 16) || !aligned(value_cache, 16) ||
        !aligned(key_scale, 16) || !aligned(value_scale, 16) || !aligned(out, 2))
        return KVC8_ERR_INVALID_ARG;
    const int group = num_q_heads / g->kv_heads;
    if (workspace == nullptr || !aligned(workspace, kAlign) ||
        workspace_bytes < shared_prefix_workspace_bytes(*g, group))
        return KVC8_ERR_WORKSPACE;
    PrefixArgs p = {};
    AttnArgs &a = p.own;
    a.g = *g;
    a.group = group;
    a.q = static_cast<const uint16_t *>(query);
    a.q_seq_stride = q_seq_stride;
    a.q_head_stride = q_head_stride;
    a.k_cache = key_cache;
    a.v_cache = value_cache;
    a.k_scale = key_scale;
    a.v_scale = value_scale;
    a.block_table = block_table;
    a.context_lengths = context_lengths;
    a.scale_log2 = (float)((double)softmax_scale * 1.4426950408889634);  // log2(e)
    a.out = static_cast<uint16_t *>(out);
    a.out_seq_stride = out_seq_stride;
    a.out_head_stride = out_head_stride;
    a.dev_error = dev_error;
    p.prefix_table = prefix_table;
    p.max_prefix_blocks = max_prefix_blocks;
    p.prefix_length = prefix_length;
    return cuda_status(launch_shared_prefix(p, workspace, stream));
}

kvc8_status kvc8_assign_blocks(const kvc8_geom *g, const int32_t *held_lens,
                               const int32_t *want_lens, int32_t *free_blocks,
                               const int32_t *free_count, int32_t *free_count_out,
                               int32_t *block_table, int32_t *lens_out, int64_t *slot_map,
                               int64_t slot_rows, int32_t *dev_error, cudaStream_t stream) {
    kvc8_status st = check_geom(g);
    if (st != KVC8_OK) return st;
    if (g->num_seqs > KVC8_ASSIGN_MAX_SEQS) return KVC8_ERR_UNSUPPORTED;
    if (free_blocks == nullptr || free_count == nullptr || free_count_out == nullptr || slot_rows < 0)
        return KVC8_ERR_INVALID_ARG;
    if (g->num_seqs > 0 && (held_lens == nullptr || want_lens == nullptr || block_table == nullptr ||
                            lens_out == nullptr))
        return KVC8_ERR_INVALID_ARG;
    if (!aligned(slot_map, 8)) return KVC8_ERR_INVALID_ARG;
    AssignArgs a = {};
    a.num_seqs = g->num_seqs;
    a.block_size = g->block_size;
    a.num_blocks = g->num_blocks;
    a.max_blocks_per_seq = g->max_blocks_per_seq;
    a.held = held_lens;
    a.want = want_lens;
    a.free_blocks = free_blocks;
    a.free_count = free_count;
    a.free_count_out = free_count_out;
    a.block_table = block_table;
    a.lens_out = lens_out;
    a.slot_map = slot_map;
    a.slot_rows = slot_map == nullptr ? 0 : slot_rows;
    a.dev_error = dev_error;
    return cuda_status(launch_assign(a, stream));
}

// What the tree attention supports: kvc8_paged_decode_attention's geometries, with
// units of 128 query rows and 128 positions counted in 32 bits.
static kvc8_status check_tree_geom(const kvc8_geom *g, int32_t num_q_heads, int64_t num_tokens,
                                   int32_t max_drafts) {
    kvc8_status st = check_geom(g);
    if (st != KVC8_OK) return st;
    if (num_q_heads < 1 || num_q_heads % g->kv_heads != 0 || num_tokens < 0 || max_drafts < 1)
        return KVC8_ERR_INVALID_ARG;
    const int group = num_q_heads / g->kv_heads;
    if (group > 8 || (g->head_dim != 64 && g->head_dim != 128) || g->block_size % 16 != 0 ||
        max_drafts > KVC8_MAX_DRAFTS || num_tokens > INT32_MAX)
        return KVC8_ERR_UNSUPPORTED;
    // A tile of query rows may have all its steps in one CTA, at about 1.4 us each: 2^26 positions take 0.7 s, which
    // keeps clear of the two seconds that its waits are allowed.
    const int64_t cap = (int64_t)g->max_blocks_per_seq * g->block_size;
    if (cap > (int64_t)1 << 26) return KVC8_ERR_UNSUPPORTED;
    const int64_t tiles = (int64_t)g->num_seqs * ((max_drafts * group + 127) / 128);  // < 2^36
    const int64_t steps = (cap + 127) / 128;
    if (tiles > (int64_t)INT32_MAX / steps / g->kv_heads) return KVC8_ERR_UNSUPPORTED;
    return KVC8_OK;
}

size_t kvc8_tree_attention_workspace_bytes(const kvc8_geom *g, int32_t num_q_heads,
                                           int64_t num_tokens, int32_t max_drafts) {
    if (check_tree_geom(g, num_q_heads, num_tokens, max_drafts) != KVC8_OK) return 0;
    return tree_workspace_bytes(*g);
}

kvc8_status kvc8_tree_attention(const kvc8_geom *g, int32_t num_q_heads, int64_t num_tokens,
                                int32_t max_drafts, const void *query, int64_t q_tok_stride,
                                int64_t q_head_stride, const int8_t *key_cache,
                                const int8_t *value_cache, const float *key_scale,
                                const float *value_scale, const int32_t *block_table,
                                const int32_t *cu_q_lens, const int32_t *context_kv_lens,
                                const uint64_t *tree_mask, int32_t mask_words,
                                float softmax_scale, void *out, int64_t out_tok_stride,
                                int64_t out_head_stride, void *workspace,
                                size_t workspace_bytes, int32_t *dev_error,
                                cudaStream_t stream) {
    kvc8_status st = check_tree_geom(g, num_q_heads, num_tokens, max_drafts);
    if (st != KVC8_OK) return st;
    if (!std::isfinite(softmax_scale)) return KVC8_ERR_INVALID_ARG;
    if (cu_q_lens == nullptr && num_tokens != g->num_seqs) return KVC8_ERR_INVALID_ARG;
    if (tree_mask != nullptr && mask_words < (max_drafts + 63) / 64) return KVC8_ERR_INVALID_ARG;
    if (tree_mask != nullptr && mask_words > 1 << 20) return KVC8_ERR_UNSUPPORTED;  // bits are counted in 32 bits
    if (num_tokens == 0 || g->num_seqs == 0) return num_tokens == 0 ? KVC8_OK : KVC8_ERR_INVALID_ARG;
    if (query == nullptr || key_cache == nullptr || value_cache == nullptr ||
        key_scale == nullptr || value_scale == nullptr || block_table == nullptr ||
        context_kv_lens == nullptr || out == nullptr || out == query)
        return KVC8_ERR_INVALID_ARG;
    if (q_tok_stride < 0 || q_head_stride < 0 || q_tok_stride % 8 != 0 || q_head_stride % 8 != 0 ||
        out_tok_stride < 0 || out_head_stride < 0)
        return KVC8_ERR_INVALID_ARG;
    if (!aligned(query, 16) || !aligned(key_cache, 16) || !aligned(value_cache, 16) ||
        !aligned(key_scale, 16) || !aligned(value_scale, 16) || !aligned(out, 2) ||
        !aligned(tree_mask, 8))
        return KVC8_ERR_INVALID_ARG;
    if (workspace == nullptr || !aligned(workspace, kAlign) || workspace_bytes < tree_workspace_bytes(*g))
        return KVC8_ERR_WORKSPACE;
    TreeArgs t = {};
    AttnArgs &a = t.base;
    a.g = *g;
    a.group = num_q_heads / g->kv_heads;
    a.q = static_cast<const uint16_t *>(query);
    a.q_seq_stride = q_tok_stride;
    a.q_head_stride = q_head_stride;
    a.k_cache = key_cache;
    a.v_cache = value_cache;
    a.k_scale = key_scale;
    a.v_scale = value_scale;
    a.block_table = block_table;
    a.context_lengths = context_kv_lens;
    a.scale_log2 = (float)((double)softmax_scale * 1.4426950408889634);  // log2(e)
    a.out = static_cast<uint16_t *>(out);
    a.out_seq_stride = out_tok_stride;
    a.out_head_stride = out_head_stride;
    a.dev_error = dev_error;
    t.num_tokens = num_tokens;
    t.max_drafts = max_drafts;
    t.cu_q_lens = cu_q_lens;
    t.mask = tree_mask;
    t.mask_words = mask_words;
    return cuda_status(launch_tree(t, workspace, stream));
}

static kvc8_status compact(const kvc8_geom *g, int32_t value_bytes, void *key_cache,
                           void *value_cache, float *key_scale, float *value_scale,
                           const int32_t *block_table, const int32_t *context_kv_lens,
                           const int32_t *accepted, int32_t max_accepted,
                           const int32_t *num_accepted, int32_t *lens_out, int32_t *dev_error,
                           cudaStream_t stream) {
    if (max_accepted < 1) return KVC8_ERR_INVALID_ARG;
    if (max_accepted > KVC8_MAX_DRAFTS) return KVC8_ERR_UNSUPPORTED;
    if (g->num_seqs == 0) return KVC8_OK;
    if (key_cache == nullptr || value_cache == nullptr || block_table == nullptr ||
        context_kv_lens == nullptr || accepted == nullptr || num_accepted == nullptr)
        return KVC8_ERR_INVALID_ARG;
    if (!aligned(key_cache, 16) || !aligned(value_cache, 16)) return KVC8_ERR_INVALID_ARG;
    CompactArgs a = {};
    a.g = *g;
    a.row_bytes = g->head_dim * value_bytes;
    a.k_cache = static_cast<char *>(key_cache);
    a.v_cache = static_cast<char *>(value_cache);
    a.k_scale = key_scale;
    a.v_scale = value_scale;
    a.block_table = block_table;
    a.context_kv_lens = context_kv_lens;
    a.accepted = accepted;
    a.max_accepted = max_accepted;
    a.num_accepted = num_accepted;
    a.lens_out = lens_out;
    a.dev_error = dev_error;
    return cuda_status(launch_compact(a, stream));
}

kvc8_status kvc8_compact_drafts(const kvc8_geom *g, int8_t *key_cache, int8_t *value_cache,
                                float *key_scale, float *value_scale,
                                const int32_t *block_table, const int32_t *context_kv_lens,
                                const int32_t *accepted, int32_t max_accepted,
                                const int32_t *num_accepted, int32_t *lens_out,
                                int32_t *dev_error, cudaStream_t stream) {
    kvc8_status st = check_geom(g);
    if (st != KVC8_OK) return st;
    if (g->num_seqs > 0 && (key_scale == nullptr || value_scale == nullptr || !aligned(key_scale, 16) ||
                            !aligned(value_scale, 16)))
        return KVC8_ERR_INVALID_ARG;
    return compact(g, 1, key_cache, value_cache, key_scale, value_scale, block_table,
                   context_kv_lens, accepted, max_accepted, num_accepted, lens_out, dev_error,
                   stream);
}

kvc8_status kvc8_compact_drafts_bf16(const kvc8_geom *g, void *key_cache, void *value_cache,
                                     const int32_t *block_table,
                                     const int32_t *context_kv_lens, const int32_t *accepted,
                                     int32_t max_accepted, const int32_t *num_accepted,
                                     int32_t *lens_out, int32_t *dev_error,
                                     cudaStream_t stream) {
    kvc8_status st = check_geom_bf16(g);
    if (st != KVC8_OK) return st;
    return compact(g, 2, key_cache, value_cache, nullptr, nullptr, block_table, context_kv_lens,
                   accepted, max_accepted, num_accepted, lens_out, dev_error, stream);
}

kvc8_status kvc8_get_error(int32_t *dev_error, int32_t *host_code, int32_t reset,
                           cudaStream_t stream) {
    if (dev_error == nullptr || host_code == nullptr) return KVC8_ERR_INVALID_ARG;
    int32_t v = 0;
    kvc8_status st = cuda_status(cudaMemcpyAsync(&v, dev_error, sizeof v, cudaMemcpyDeviceToHost, stream));
    if (st != KVC8_OK) return st;
    if ((st = cuda_status(cudaStreamSynchronize(stream))) != KVC8_OK) return st;
    *host_code = v;
    if (reset) {
        if ((st = cuda_status(cudaMemsetAsync(dev_error, 0, sizeof(int32_t), stream))) != KVC8_OK) return st;
        if ((st = cuda_status(cudaStreamSynchronize(stream))) != KVC8_OK) return st;
    }
    return v == 0 ? KVC8_OK : KVC8_ERR_DEVICE_BOUNDS;
}

}  // extern "C"
