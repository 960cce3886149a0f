// Entry points around the attention of a bounded cache: norm + rotation +
// append, attention with per-key weight totals, and eviction.  Argument checks
// on the host first, then launches only, as for every call of the library.

#include <algorithm>
#include <cmath>
#include <cstdio>
#include <new>
#include <vector>

#include "plan_host.h"

namespace pa {

namespace {

size_t align256(size_t n) { return (n + 255) / 256 * 256; }

// Longest history (in keys) any tile's query of the plan's host copy may see.
int64_t longest_tile_seq(const pa_plan *plan) {
    const int32_t *w = plan->words.data();
    int32_t longest = 0;
    for (int32_t t = 0; t < plan->n_tiles; ++t)
        longest = std::max(longest, w[plan->off_seqlen + w[plan->off_tiles + 4 * (size_t)t]]);
    return longest;
}

}  // namespace

pa_status spans_disjoint(const Span *written, int n_written, const Span *read, int n_read, const char *call) {
    auto meet = [](const Span &a, const Span &b) {
        const uintptr_t x = reinterpret_cast<uintptr_t>(a.at), y = reinterpret_cast<uintptr_t>(b.at);
        return a.at && b.at && a.bytes && b.bytes && x < y + b.bytes && y < x + a.bytes;
    };
    for (int i = 0; i < n_written; ++i)
        for (int j = i + 1; j < n_written + n_read; ++j) {
            const Span &b = j < n_written ? written[j] : read[j - n_written];
            if (!meet(written[i], b)) continue;
            char msg[256];
            std::snprintf(msg, sizeof msg, "%s: %s overlaps %s", call, written[i].name, b.name);
            return fail(PA_ERR_ARG, msg);
        }
    return PA_OK;
}

bool mass_rows_fit(const pa_plan *plan, int32_t hq, int32_t splits) {
    return (int64_t)plan->queries * hq <= INT32_MAX / splits;
}

MassLayout mass_layout(const pa_plan *plan, int32_t hq, int32_t dv, int32_t splits, int32_t window, int64_t max_keys) {
    MassLayout l{};
    const size_t rows = (size_t)plan->queries * hq;
    const size_t part = splits > 1 ? align256((size_t)splits * rows * dv * sizeof(float)) : 0;
    l.lse = part;
    l.lse_final = l.lse + align256((size_t)splits * rows * sizeof(float));
    l.items = l.lse_final + (splits > 1 && plan->n_tiles > 0 ? align256(rows * sizeof(float)) : 0);
    // work lists: [sequences + 1] starts and the records; for tiles also the key
    // blocks of as many sequences as can have some, and the laid out log-sum-exps
    const size_t seqs = (size_t)plan->sequences + 1;
    l.tiles = l.items + align256((seqs + plan->n_decode) * sizeof(int32_t));
    l.blocks = l.tiles + (plan->n_tiles > 0 ? align256((seqs + plan->queries) * sizeof(int32_t)) : 0);
    const int64_t per_seq = ((int64_t)plan->width * plan->page_size + 127) / 128;
    const int64_t blocks = std::min<int64_t>(std::min(plan->sequences, plan->n_tiles) * per_seq, INT32_MAX);
    l.max_blocks = (int32_t)blocks;
    l.tile_lse = l.blocks + (plan->n_tiles > 0 ? align256(((size_t)blocks + 1) * sizeof(int4)) : 0);
    l.scores = l.tile_lse + align256((size_t)plan->n_tiles * hq * 128 * sizeof(float));
    int64_t keys = std::max<int64_t>(max_keys, plan->max_seq_len);
    if (window > 0 && keys > window) keys = (int64_t)window + 3;      // a row starts up to three keys early
    l.cap = plan->n_decode > 0 ? (keys + 31) / 32 * 32 : 0;
    // rows and keys are below 2^31 each, so their product fits; its bytes may not
    const uint64_t scores = (uint64_t)plan->n_decode * (uint64_t)hq * (uint64_t)l.cap;
    l.bytes = scores >> 60 ? SIZE_MAX : l.scores + align256((size_t)scores * sizeof(float));
    return l;
}

namespace {

MassArgs mass_args(const AttnArgs &a, const MassLayout &lay, char *ws, float *key_mass, size_t lists) {
    MassArgs m{};
    m.plan = a.plan;
    m.q = a.q; m.k = a.k;
    m.key_mass = key_mass;
    m.lse = a.ws_lse;
    m.lse_final = a.splits > 1 ? reinterpret_cast<float *>(ws + lay.lse_final) : a.ws_lse;
    m.scores = a.scores;
    m.cap = a.score_cap;
    m.group_start = reinterpret_cast<int32_t *>(ws + lists);
    m.hq = a.hq; m.hkv = a.hkv; m.d = a.d;
    m.splits = a.splits; m.causal = a.causal; m.window = a.window;
    m.scale = a.scale;
    m.dtype = a.dtype;
    m.status = a.status;
    return m;
}

}  // namespace

cudaError_t add_item_mass(const pa_plan *plan, const AttnArgs &a, const MassLayout &lay, char *ws, float *key_mass, bool merge,
                          bool use_list, cudaStream_t st) {
    MassArgs m = mass_args(a, lay, ws, key_mass, lay.items);
    m.group_list = m.group_start + plan->sequences + 1;
    m.longest = (int32_t)plan->max_seq_len;
    const bool repeated = (plan_facts(plan) & kFactRepeatedItems) != 0;
    cudaError_t e = mass_items_grouped(m, repeated) ? launch_mass_index(m, kMassItems, st) : cudaSuccess;
    if (e == cudaSuccess) e = launch_mass_items(m, repeated, merge ? &a : nullptr, use_list, st);
    return e;
}

cudaError_t add_tile_mass(const pa_plan *plan, const AttnArgs &a, const MassLayout &lay, char *ws, float *key_mass,
                          cudaStream_t st) {
    MassArgs m = mass_args(a, lay, ws, key_mass, lay.tiles);
    m.group_list = m.group_start + plan->sequences + 1;
    m.longest = (int32_t)std::max(longest_tile_seq(plan), plan->max_seq_len);
    if (prefill_supported(a)) {
        m.n_blocks = reinterpret_cast<int32_t *>(ws + lay.blocks);           // its own 16 bytes, then the list
        m.blocks = reinterpret_cast<int4 *>(ws + lay.blocks) + 1;
        m.max_blocks = lay.max_blocks;
        m.tile_lse = reinterpret_cast<float *>(ws + lay.tile_lse);
        cudaError_t e = launch_mass_tiles_prepare(m, st);
        return e == cudaSuccess ? launch_mass_tiles(m, st) : e;
    }
    cudaError_t e = launch_mass_index(m, kMassQueries, st);
    if (e == cudaSuccess && a.splits > 1) e = launch_lse_final(m, reinterpret_cast<float *>(ws + lay.lse_final), st);
    return e == cudaSuccess ? launch_mass_recompute(m, st) : e;
}

}  // namespace pa

using pa::fail;

extern "C" {

size_t pa_mass_workspace_bytes(const pa_plan *plan, int32_t num_heads, int32_t num_kv_heads, int32_t value_dim,
                               int32_t splits, int32_t window, int64_t max_keys) {
    if (!plan || num_heads < 1 || num_heads > 65535 || num_kv_heads < 1 || num_heads % num_kv_heads || value_dim < 1 ||
        value_dim > PA_MAX_HEAD_DIM || splits < 1 || splits > PA_MAX_SPLITS || window < 0 || max_keys < 0 ||
        max_keys > INT32_MAX || !pa::mass_rows_fit(plan, num_heads, splits))
        return 0;
    const size_t bytes = pa::mass_layout(plan, num_heads, value_dim, splits, window, max_keys).bytes;
    return bytes == SIZE_MAX ? 0 : bytes;
}

pa_status paged_attn_forward_mass(const pa_plan *plan, const void *q, const void *k_cache, const void *v_cache, void *out,
                                  float *key_mass, int32_t num_heads, int32_t num_kv_heads, int32_t head_dim,
                                  int32_t value_dim, float scale, int32_t causal, int32_t window, pa_dtype dtype,
                                  void *workspace, size_t workspace_bytes, int32_t splits, pa_stream_t stream) {
    static const char kName[] = "paged_attn_forward_mass";
    pa_status st = pa::check_attention_args(plan, num_heads, num_kv_heads, head_dim, value_dim, 0, scale, causal, window,
                                            dtype, false, kName);
    if (st != PA_OK) return st;
    if (!key_mass) return fail(PA_ERR_ARG, "paged_attn_forward_mass: key_mass is null");
    if (reinterpret_cast<uintptr_t>(key_mass) % sizeof(float))
        return fail(PA_ERR_ARG, "paged_attn_forward_mass: key_mass not 4-byte aligned");
    if (splits >= 1 && splits <= PA_MAX_SPLITS && !pa::mass_rows_fit(plan, num_heads, splits))
        return fail(PA_ERR_LIMIT, "paged_attn_forward_mass: more than 2^31 - 1 (query, head, split) rows");
    if (std::max<int64_t>(plan->max_seq_len, pa::longest_tile_seq(plan)) > pa::kMaxCountedKeys)
        return fail(PA_ERR_LIMIT, "paged_attn_forward_mass: history above 2^30 keys");
    try {
        if (pa::plan_facts(plan) & pa::kFactSharedPages)
            return fail(PA_ERR_WRITE_CONFLICT, "paged_attn_forward_mass: two sequences hold one page, its totals would have two owners");
        return pa::attention_with_mass(plan, q, k_cache, v_cache, out, key_mass, num_heads, num_kv_heads, head_dim,
                                       value_dim, scale, causal, window, dtype, workspace, workspace_bytes, splits,
                                       (cudaStream_t)stream, kName);
    } catch (const std::bad_alloc &) {
        return fail(PA_ERR_LIMIT, "paged_attn_forward_mass: out of host memory");
    }
}

pa_status paged_qk_norm_rope_store(const pa_plan *plan, const void *q, int64_t q_stride, const void *new_k,
                                   int64_t k_stride, const void *new_v, int64_t v_stride, void *q_out, void *k_cache,
                                   void *v_cache, float *key_mass, const float *rope_table, int32_t max_positions,
                                   int32_t rope_dim, int32_t interleaved, const int32_t *positions, const void *q_weight,
                                   const void *k_weight, float eps, int32_t num_heads, int32_t num_kv_heads,
                                   int32_t head_dim, int32_t value_dim, pa_dtype dtype, pa_stream_t stream) {
#define BAD(status, what) return fail(status, "paged_qk_norm_rope_store: " what)
    if (!plan) BAD(PA_ERR_ARG, "plan is null");
    if (!pa::valid_dtype(dtype)) BAD(PA_ERR_DTYPE, "dtype must be F32, F16 or BF16");
    if (num_heads < 1 || num_kv_heads < 1 || head_dim < 1 || value_dim < 1)
        BAD(PA_ERR_SHAPE, "heads, head_dim and value_dim must be >= 1");
    if (head_dim > PA_MAX_HEAD_DIM || value_dim > PA_MAX_HEAD_DIM) BAD(PA_ERR_LIMIT, "head dim above 1024");
    if (num_heads > 65535 || num_kv_heads > 65535) BAD(PA_ERR_LIMIT, "num_heads above the launch grid limit");
    if (interleaved != 0 && interleaved != 1) BAD(PA_ERR_ARG, "interleaved must be 0 or 1");
    if (rope_table) {
        if (rope_dim < 2 || rope_dim % 2 || rope_dim > head_dim) BAD(PA_ERR_SHAPE, "rope_dim must be even and in 2..head_dim");
        if (max_positions < 1) BAD(PA_ERR_SHAPE, "the rope table has no rows");
    } else if (positions) {
        BAD(PA_ERR_ARG, "positions without a rope table");
    }
    if ((q_weight || k_weight) && (!std::isfinite(eps) || eps < 0.f)) BAD(PA_ERR_SHAPE, "eps must be finite and >= 0");
    if (q_stride < 0 || k_stride < 0 || v_stride < 0) BAD(PA_ERR_SHAPE, "negative stride");
    const int64_t most = (int64_t)1 << 40;
    if ((int64_t)plan->pages * plan->page_size * num_kv_heads * std::max(head_dim, value_dim) > most ||
        (int64_t)plan->queries * num_heads * head_dim > most ||
        std::max(q_stride, std::max(k_stride, v_stride)) > most / std::max(plan->queries, 1))
        BAD(PA_ERR_RANGE, "tensor too large");
    if (plan->queries == 0) return PA_OK;
    if (!plan->dev) BAD(PA_ERR_STATE, "plan not uploaded");
    if (!q || !new_k || !new_v || !q_out || !k_cache || !v_cache) BAD(PA_ERR_ARG, "null tensor");
    const void *ptrs[] = {q, new_k, new_v, q_out, k_cache, v_cache, key_mass, rope_table, positions, q_weight, k_weight};
    const char *names[] = {"q", "new_k", "new_v", "q_out", "k_cache", "v_cache", "key_mass", "the rope table",
                           "positions", "q_weight", "k_weight"};
    pa_status on_dev = pa::operands_on_device(ptrs, names, 11, "paged_qk_norm_rope_store");
    if (on_dev != PA_OK) return on_dev;
    for (const void *p : {(const void *)key_mass, (const void *)rope_table, (const void *)positions})
        if (reinterpret_cast<uintptr_t>(p) % 4) BAD(PA_ERR_ARG, "32-bit operand not 4-byte aligned");
    for (const void *p : {q, new_k, new_v, (const void *)q_out, (const void *)k_cache, (const void *)v_cache, q_weight, k_weight})
        if (reinterpret_cast<uintptr_t>(p) % pa::elem_bytes(dtype)) BAD(PA_ERR_ARG, "operand not aligned to its element");
    {
        const size_t es = (size_t)pa::elem_bytes(dtype), n = (size_t)plan->queries,
                     slots = (size_t)plan->pages * plan->page_size * num_kv_heads;
        auto rows = [&](int64_t stride, int32_t heads, int32_t dim) {
            return ((n - 1) * (size_t)stride + (size_t)heads * dim) * es;
        };
        const pa::Span written[] = {{k_cache, slots * head_dim * es, "k_cache"}, {v_cache, slots * value_dim * es, "v_cache"},
                                    {key_mass, slots * sizeof(float), "key_mass"},
                                    {q_out, n * num_heads * head_dim * es, "q_out"}};
        // q may be its own output when it is dense: every row is read before it is written
        const bool own = q == q_out && (n == 1 || q_stride == (int64_t)num_heads * head_dim);
        const pa::Span read[] = {{new_k, rows(k_stride, num_kv_heads, head_dim), "new_k"},
                                 {new_v, rows(v_stride, num_kv_heads, value_dim), "new_v"},
                                 {rope_table, (size_t)max_positions * rope_dim * sizeof(float), "the rope table"},
                                 {positions, n * sizeof(int32_t), "positions"},
                                 {q_weight, (size_t)head_dim * es, "q_weight"},
                                 {k_weight, (size_t)head_dim * es, "k_weight"},
                                 {own ? nullptr : q, rows(q_stride, num_heads, head_dim), "q"}};
        const pa_status apart = pa::spans_disjoint(written, 4, read, 7, "paged_qk_norm_rope_store");
        if (apart != PA_OK) return apart;
    }
    pa::NormRopeArgs a{};
    a.plan = pa::view_of(plan);
    a.q = q; a.k = new_k; a.v = new_v;
    a.q_stride = q_stride; a.k_stride = k_stride; a.v_stride = v_stride;
    a.q_out = q_out; a.k_cache = k_cache; a.v_cache = v_cache;
    a.key_mass = key_mass;
    a.table = rope_table;
    a.positions = positions;
    a.q_weight = q_weight; a.k_weight = k_weight;
    a.eps = eps;
    a.max_positions = max_positions;
    a.rot = rope_table ? rope_dim : 0;
    a.interleaved = interleaved;
    a.hq = num_heads; a.hkv = num_kv_heads; a.d = head_dim; a.dv = value_dim;
    a.dtype = dtype;
    a.status = pa::device_status_ptr();
    if (!a.status) BAD(PA_ERR_CUDA, "device status word unavailable");
    cudaError_t e = pa::launch_norm_rope_store(a, (cudaStream_t)stream);
    if (e != cudaSuccess) return pa::fail_cuda(e, "paged_qk_norm_rope_store launch");
    return PA_OK;
#undef BAD
}

pa_status paged_kv_evict(const pa_plan *plan, const pa_plan *kept_plan, float *key_mass, void *k_cache, void *v_cache,
                         int32_t *kept, int32_t kept_stride, int32_t sink, int32_t recent, int32_t num_kv_heads,
                         int32_t head_dim, int32_t value_dim, pa_dtype dtype, pa_stream_t stream) {
#define BAD(status, what) return fail(status, "paged_kv_evict: " what)
    if (!plan || !kept_plan) BAD(PA_ERR_ARG, "plan is null");
    if (!pa::valid_dtype(dtype)) BAD(PA_ERR_DTYPE, "dtype must be F32, F16 or BF16");
    if (num_kv_heads < 1 || head_dim < 1 || value_dim < 1) BAD(PA_ERR_SHAPE, "heads, head_dim and value_dim must be >= 1");
    if (head_dim > PA_MAX_HEAD_DIM || value_dim > PA_MAX_HEAD_DIM) BAD(PA_ERR_LIMIT, "head dim above 1024");
    if (num_kv_heads > 65535) BAD(PA_ERR_LIMIT, "num_kv_heads above the launch grid limit");
    if (sink < 0 || recent < 0) BAD(PA_ERR_ARG, "sink and recent must be >= 0");
    if ((int64_t)sink + recent > INT32_MAX) BAD(PA_ERR_RANGE, "sink + recent too large");
    if (plan->sequences != kept_plan->sequences || plan->page_size != kept_plan->page_size || plan->pages != kept_plan->pages)
        BAD(PA_ERR_SHAPE, "the plans differ in sequences, page size or pool");
    if ((int64_t)plan->pages * plan->page_size * num_kv_heads * std::max(head_dim, value_dim) > (int64_t)1 << 40)
        BAD(PA_ERR_RANGE, "cache too large");
    int32_t longest = 0, longest_src = 0;
    bool in_place = false;
    try {
        const int32_t *w = plan->words.data(), *d = kept_plan->words.data();
        const int32_t ps = plan->page_size;
        // Rows are written into a page that nothing else reads or writes: a page no
        // entry of the source schedule holds (those that its device copy may have
        // advanced onto among them), named once, or the sequence's own page of the same
        // index, held by nobody else.  Pages inside the sink keep every row where it is
        // and may be shared.
        const bool src_shared = (pa::plan_facts(plan) & pa::kFactSharedReach) != 0;
        const bool dst_shared = (pa::plan_facts(kept_plan) & pa::kFactSharedPages) != 0;
        std::vector<int32_t> written, all;      // filled only when some page is shared
        for (int32_t s = 0; s < plan->sequences; ++s) {
            const int32_t n = w[plan->off_seqlen + s], m = d[kept_plan->off_seqlen + s];
            // a source that can advance may be longer on the device, up to what its pages hold
            const int64_t most = pa::can_advance(plan, s) ? (int64_t)plan->reach[(size_t)s] * ps : n;
            if (m > most) BAD(PA_ERR_SHAPE, "a sequence would keep more keys than it has");
            if (m < n && m < (int64_t)sink + recent) BAD(PA_ERR_SHAPE, "a sequence's budget is below sink + recent");
            longest = std::max(longest, m);
            longest_src = std::max(longest_src, n);
            const int32_t *from = w + plan->off_table + (size_t)s * plan->width;
            const int32_t *to = d + kept_plan->off_table + (size_t)s * kept_plan->width;
            const int64_t kept_pages = ((int64_t)m + ps - 1) / ps;
            for (int64_t g = 0; g < kept_pages; ++g) {
                const bool fresh = to[g] != from[g];
                if (fresh && (plan->held[(size_t)to[g] / 64] >> (to[g] % 64) & 1))
                    BAD(PA_ERR_WRITE_CONFLICT, "the kept schedule writes a page that the source schedule reads or reserves");
                in_place |= !fresh;
                // (rows may move even where the host copies' lengths agree: the source
                // may have been advanced on the device)
                if ((src_shared || dst_shared) && (fresh || (g + 1) * ps > sink)) written.push_back(to[g]);
            }
            if (src_shared) all.insert(all.end(), from, from + plan->reach[(size_t)s]);
        }
        if (src_shared || dst_shared) {
            std::sort(written.begin(), written.end());
            if (std::adjacent_find(written.begin(), written.end()) != written.end())
                BAD(PA_ERR_WRITE_CONFLICT, "two sequences of the kept schedule write one page");
            std::sort(all.begin(), all.end());
            for (int32_t pg : written) {
                auto range = std::equal_range(all.begin(), all.end(), pg);
                if (range.second - range.first > 1)
                    BAD(PA_ERR_WRITE_CONFLICT, "the kept schedule writes a page that two sequences hold");
            }
        }
        if (kept_stride < longest) BAD(PA_ERR_SHAPE, "kept has fewer columns than the longest kept history");
    } catch (const std::bad_alloc &) {
        BAD(PA_ERR_LIMIT, "out of host memory");
    }
    if (kept_stride > pa::kMaxCountedKeys || longest_src > pa::kMaxCountedKeys)
        BAD(PA_ERR_LIMIT, "more than 2^30 keys or columns of kept");
    pa::EvictArgs a{};
    a.src.sequences = plan->sequences;
    a.key_mass = key_mass;
    a.k_cache = k_cache;
    a.v_cache = v_cache;
    a.kept = kept;
    a.kept_stride = kept_stride;
    a.sink = sink; a.recent = recent;
    a.hkv = num_kv_heads; a.d = head_dim; a.dv = value_dim;
    a.elem = pa::elem_bytes(dtype);
    if (!pa::evict_fits_grid(a, in_place)) BAD(PA_ERR_LIMIT, "more lists of keys than a launch can number");
    if (plan->sequences == 0 || kept_stride == 0) return PA_OK;
    if (!plan->dev || !kept_plan->dev) BAD(PA_ERR_STATE, "plan not uploaded");
    if (!key_mass || !k_cache || !v_cache || !kept) BAD(PA_ERR_ARG, "null tensor");
    const void *ptrs[] = {key_mass, k_cache, v_cache, kept};
    const char *names[] = {"key_mass", "k_cache", "v_cache", "kept"};
    pa_status on_dev = pa::operands_on_device(ptrs, names, 4, "paged_kv_evict");
    if (on_dev != PA_OK) return on_dev;
    for (const void *p : {(const void *)key_mass, (const void *)kept})
        if (reinterpret_cast<uintptr_t>(p) % 4) BAD(PA_ERR_ARG, "32-bit operand not 4-byte aligned");
    for (const void *p : {(const void *)k_cache, (const void *)v_cache})
        if (reinterpret_cast<uintptr_t>(p) % pa::elem_bytes(dtype)) BAD(PA_ERR_ARG, "operand not aligned to its element");
    const size_t slots = (size_t)plan->pages * plan->page_size * num_kv_heads, es = (size_t)pa::elem_bytes(dtype);
    const pa::Span written[] = {{key_mass, slots * sizeof(float), "key_mass"}, {k_cache, slots * head_dim * es, "k_cache"},
                                {v_cache, slots * value_dim * es, "v_cache"},
                                {kept, (size_t)plan->sequences * num_kv_heads * kept_stride * sizeof(int32_t), "kept"}};
    const pa_status apart = pa::spans_disjoint(written, 4, nullptr, 0, "paged_kv_evict");
    if (apart != PA_OK) return apart;
    a.src = pa::view_of(plan);
    a.dst = pa::view_of(kept_plan);
    a.status = pa::device_status_ptr();
    if (!a.status) BAD(PA_ERR_CUDA, "device status word unavailable");
    cudaError_t e = pa::launch_evict(a, longest_src, longest, in_place, (cudaStream_t)stream);
    if (e != cudaSuccess) return pa::fail_cuda(e, "paged_kv_evict launch");
    return PA_OK;
#undef BAD
}

}  // extern "C"
