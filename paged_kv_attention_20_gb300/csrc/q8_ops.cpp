// Entry points of the 8-bit cache: the append that quantises, the read-back into a
// paged cache of wider elements, and attention over the 8-bit rows.  Argument checks
// on the host first, then launches only, as for every call of the library.

#include <algorithm>
#include <cstdio>
#include <new>

#include "per_device.h"
#include "plan_host.h"

namespace pa {

namespace {

size_t align256(size_t n) { return (n + 255) / 256 * 256; }

// Workspace of paged_attn_forward_q8: the split partials, and where prefill tiles run on
// the tensor cores a paged 16-bit copy of the tiles' histories (byte offsets).  The copy has
// pages of 128 rows whatever the cache's: the prefill kernel loads a key tile with the fewest
// boxes then (1149 TFLOP/s on the mixed step's chunks, 1030 with pages of 16).
constexpr int32_t kCopyPage = 128;

// Of the histories of sequences with tiles, from the first block of 128 keys that a tile's query
// sees: their blocks, and the keys of the longest.
struct CopiedKeys {
    int64_t blocks = 0, longest = 0;
};

CopiedKeys copied_keys(const pa_plan *plan, int32_t window) {
    CopiedKeys c;
    for (const auto &[seq, pos] : plan->tile_starts) {
        const int64_t len = plan->words[plan->off_seqlen + seq];
        const int64_t first = window > 0 ? std::max<int64_t>(0, (int64_t)pos - window + 1) / kCopyPage : 0;
        c.blocks += (len + kCopyPage - 1) / kCopyPage - first;
        c.longest = std::max(c.longest, len - first * kCopyPage);
    }
    return c;
}

struct Q8Layout {
    bool tiles;
    int32_t width;                        // of the copy's block table
    size_t places, table, k, bytes;       // the values follow the keys
    size_t page_bytes;                    // of one page of one tensor
    int64_t room;                         // pages
    CopiedKeys copied;
};

bool tiles_on_tensor_cores(const pa_plan *plan, int32_t d, int32_t dv, pa_dtype dtype) {
    return plan->n_tiles > 0 && dtype != PA_F32 && d == 128 && dv == 128;
}

// max_keys: keys the copy holds at least, over all sequences with tiles; 0: the host copy's.
Q8Layout q8_layout(const pa_plan *plan, int32_t hq, int32_t hkv, int32_t d, int32_t dv, pa_dtype dtype, int32_t splits,
                   int32_t window, int64_t max_keys) {
    Q8Layout l{};
    l.tiles = tiles_on_tensor_cores(plan, d, dv, dtype);
    l.bytes = splits > 1 ? align256(pa_workspace_bytes(plan->queries, hq, dv, splits)) : 0;
    if (!l.tiles) return l;
    l.copied = copied_keys(plan, window);
    l.places = l.bytes;
    l.table = l.places + align256((size_t)plan->sequences * sizeof(int2));
    l.width = (int32_t)((std::min<int64_t>((int64_t)plan->width * plan->page_size, INT32_MAX) + kCopyPage - 1) / kCopyPage);
    l.k = l.table + align256((size_t)plan->sequences * l.width * sizeof(int32_t));
    l.page_bytes = (size_t)kCopyPage * hkv * 128 * 2;
    l.room = std::max<int64_t>(l.copied.blocks, (max_keys + kCopyPage - 1) / kCopyPage + (int64_t)plan->tile_starts.size());
    l.bytes = l.k + 2 * (size_t)l.room * l.page_bytes;
    return l;
}

// Rows of a cache of the plan's pool.
size_t slots_of(const pa_plan *plan, int32_t heads) { return (size_t)plan->pages * plan->page_size * heads; }

pa_status cache_shape(const pa_plan *plan, int32_t heads, int32_t d, int32_t dv, const char *name) {
    auto bad = [&](pa_status status, const char *what) {
        char msg[256];
        std::snprintf(msg, sizeof msg, "%s: %s", name, what);
        return fail(status, msg);
    };
    if (heads < 1 || d < 1 || dv < 1) return bad(PA_ERR_SHAPE, "heads, head_dim and value_dim must be >= 1");
    if (d > PA_MAX_HEAD_DIM || dv > PA_MAX_HEAD_DIM) return bad(PA_ERR_LIMIT, "head dim above 1024");
    if (heads > 65535) return bad(PA_ERR_LIMIT, "num_heads above the launch grid limit");
    if ((int64_t)plan->pages * plan->page_size > ((int64_t)1 << 40) / ((int64_t)heads * std::max(d, dv)))
        return bad(PA_ERR_RANGE, "cache too large");
    return PA_OK;
}

}  // namespace

namespace {

// SMs to give to a mixed call's decode items while its tiles run on the others (0: one after
// the other).  The persistent 8-bit decode reads 48 GB/s on each SM of its own beside the
// prefill kernel but no more than HBM gives, the prefill kernel does 6.5 TFLOP/s on each; the
// share is taken that ends both soonest, when it saves at least 5 % and both are long enough
// for the fork and join to be noise (the mixed step: 282 us with 52 SMs, 311 one after the
// other).
int q8_sms_beside_prefill(const pa_plan *plan, const AttnArgs &a, int64_t copied_blocks, int sms) {
    constexpr double kFlopsPerSm = 6.5e12, kBytesPerSm = 4.8e10, kHbmBytes = 6.0e12, kCopyBytes = 4.0e12;
    if (plan->n_decode == 0 || plan->n_tiles == 0 || sms < 8) return 0;
    double keys_p = plan->keys_tiles[a.causal], keys_d = plan->keys_decode[a.causal];
    if (a.window > 0) visible_key_sums(plan, a.causal, a.window, keys_p, keys_d);
    const double flops = keys_p * a.hq * 4.0 * 128, bytes = keys_d * a.hkv * 258.0;
    // the copy comes before the tiles, beside the decode items: a byte read and two written
    const double t_copy = (double)copied_blocks * kCopyPage * a.hkv * 256.0 * 3 / kCopyBytes;
    const double t_prefill = flops / (kFlopsPerSm * sms), t_decode = bytes / kHbmBytes;
    if (t_prefill < 20e-6 || t_decode < 20e-6) return 0;
    double best = t_copy + t_prefill + t_decode;
    const double serial = best;
    int best_n = 0;
    for (int n = 1; n < sms; ++n) {
        const double t = std::max(t_copy + flops / (kFlopsPerSm * (sms - n)), bytes / std::min(kBytesPerSm * n, kHbmBytes));
        if (t < best) {
            best = t;
            best_n = n;
        }
    }
    return best < 0.95 * serial ? best_n : 0;
}

// Splits that the tensor-core decode kernel takes, of at most a.splits: those that end soonest.
// It is persistent and has some 12 us from the launch to the end of a unit's first tile; a tile
// of 32 KB takes 0.56 us (0.68 with up to eight columns, 0.9 with sixteen), or its share of HBM
// where more SMs read; a unit costs two tiles more; units sorted by length leave a fifth of the
// longest one uneven; and partials cost a merge.  Within 2 % of the best count over 32 batches, 15 %
// at worst.  The split heuristic's counts are those of a kernel whose blocks share an SM: with them
// 4 histories to 2000 keys (8 KV heads) take 27 us for 18, 16 to 500 25 for 14, 4 to 8000 33 for
// 25, 64 to 8000 117 for 111.
// The kernel for other shapes takes the caller's count, but for one or two tiles of 128 keys a query:
// a second tile takes as long as a merge (4 histories to 200 keys, fp32: 14-18 us either way, and a
// launch less).
// A captured call is replayed for lengths that are not known here; it takes its histories to grow,
// all by one factor, until the longest fills its row of the block table (one history captured at 200
// keys with 16 splits and replayed at 32768: 32 us, 161 in the one split that 200 keys need; fp32
// 128, 1650).
int32_t q8_splits(const pa_plan *plan, const Q8AttnArgs &x, int sms, bool captured) {
    const AttnArgs &a = x.a;
    int64_t visible = most_visible_keys(plan, a.causal, a.window);
    double grown = 1;
    if (captured) {
        const int64_t reach = std::min<int64_t>((int64_t)plan->width * plan->page_size, kMaxCountedKeys);
        const int64_t most = a.window > 0 && a.causal ? std::min<int64_t>(reach, a.window) : reach;
        grown = (double)most / (double)std::max<int64_t>(visible, 1);
        visible = most;
    }
    if (!q8_decode_tc_supported(x)) return visible <= 256 ? 1 : a.splits;
    const int32_t pair = a.d == 64 ? 2 : 1, group = a.hq / a.hkv;
    const int64_t columns = (int64_t)pair * group * plan->longest_run;
    const int64_t per = std::min<int64_t>(group, 16 / pair);
    const double items = columns <= 16 ? plan->decode_runs : plan->n_decode;
    const double units = items * ((a.hkv + pair - 1) / pair) * (double)((group + per - 1) / per);
    const double tile = columns <= 4 ? 0.56e-6 : columns <= 8 ? 0.68e-6 : 0.9e-6;
    // (under a window a unit of several queries reads a few keys more than one of them sees)
    const double longest = (double)visible + (a.window > 0 ? plan->longest_run - 1 : 0);
    double keys = plan->keys_decode[a.causal], none = 0;
    if (a.window > 0) visible_key_sums(plan, a.causal, a.window, none, keys);
    const double most = longest / 128, mean = grown * keys / plan->n_decode / 128;
    const double merge = (double)plan->queries * a.hq * a.dv * 8 / 4e12;
    int32_t best = 1;
    double best_t = 0;
    for (int32_t s = 1; s <= a.splits; ++s) {
        const double all = units * s, t = std::max(tile, 32768 * std::min<double>(all, sms) / 6.3e12);
        const double longest_unit = std::max(1.0, most / s), sm = all / sms * (std::max(1.0, mean / s + 0.3) + 2);
        const double uneven = all > sms ? 0.2 * longest_unit : 0;
        const double time = t * (std::max(longest_unit + 2, sm) + uneven) + (s > 1 ? 5e-6 + merge * s : 0);
        if (s == 1 || time < best_t) {
            best = s;
            best_t = time;
        }
    }
    return best;
}

}  // namespace

cudaError_t launch_q8_decode(const Q8AttnArgs &q, bool use_decode_list, int longest_run, cudaStream_t st) {
    return q8_decode_tc_supported(q) ? launch_q8_decode_tc(q, use_decode_list, longest_run, st)
                                     : launch_q8_decode_any(q, use_decode_list, st);
}

}  // namespace pa

using pa::fail;

extern "C" {

pa_status paged_kv_store_q8(const pa_plan *plan, const void *new_k, int64_t k_stride, const void *new_v, int64_t v_stride,
                            uint8_t *k_cache, uint8_t *v_cache, uint8_t *k_scale, uint8_t *v_scale, int32_t num_heads,
                            int32_t head_dim, int32_t value_dim, pa_dtype dtype, pa_stream_t stream) {
#define BAD(status, what) return fail(status, "paged_kv_store_q8: " what)
    if (!plan) BAD(PA_ERR_ARG, "plan is null");
    if (!pa::valid_dtype(dtype)) BAD(PA_ERR_DTYPE, "dtype must be F32, F16 or BF16");
    const pa_status shape = pa::cache_shape(plan, num_heads, head_dim, value_dim, "paged_kv_store_q8");
    if (shape != PA_OK) return shape;
    if (k_stride < 0 || v_stride < 0) BAD(PA_ERR_SHAPE, "negative stride");
    const int64_t most = (int64_t)1 << 40;
    if (std::max(k_stride, v_stride) > most / std::max(plan->queries, 1)) BAD(PA_ERR_RANGE, "tensor too large");
    if (plan->queries == 0) return PA_OK;
    if (!plan->dev) BAD(PA_ERR_STATE, "plan not uploaded");
    if (!new_k || !new_v || !k_cache || !v_cache || !k_scale || !v_scale) BAD(PA_ERR_ARG, "null tensor");
    const void *ptrs[] = {new_k, new_v, k_cache, v_cache, k_scale, v_scale};
    const char *names[] = {"new_k", "new_v", "k_cache", "v_cache", "k_scale", "v_scale"};
    const pa_status on_dev = pa::operands_on_device(ptrs, names, 6, "paged_kv_store_q8");
    if (on_dev != PA_OK) return on_dev;
    for (const void *p : {new_k, new_v})
        if (reinterpret_cast<uintptr_t>(p) % pa::elem_bytes(dtype)) BAD(PA_ERR_ARG, "operand not aligned to its element");
    const size_t es = (size_t)pa::elem_bytes(dtype), n = (size_t)plan->queries, slots = pa::slots_of(plan, num_heads);
    const pa::Span written[] = {{k_cache, slots * head_dim, "k_cache"}, {v_cache, slots * value_dim, "v_cache"},
                                {k_scale, slots, "k_scale"}, {v_scale, slots, "v_scale"}};
    const pa::Span read[] = {{new_k, ((n - 1) * (size_t)k_stride + (size_t)num_heads * head_dim) * es, "new_k"},
                             {new_v, ((n - 1) * (size_t)v_stride + (size_t)num_heads * value_dim) * es, "new_v"}};
    const pa_status apart = pa::spans_disjoint(written, 4, read, 2, "paged_kv_store_q8");
    if (apart != PA_OK) return apart;
    pa::Q8StoreArgs a{};
    a.plan = pa::view_of(plan);
    a.k = new_k; a.v = new_v;
    a.k_stride = k_stride; a.v_stride = v_stride;
    a.k_cache = k_cache; a.v_cache = v_cache; a.k_scale = k_scale; a.v_scale = v_scale;
    a.hkv = num_heads; a.d = head_dim; a.dv = value_dim;
    a.dtype = dtype;
    const cudaError_t e = pa::launch_q8_store(a, (cudaStream_t)stream);
    if (e != cudaSuccess) return pa::fail_cuda(e, "paged_kv_store_q8 launch");
    return PA_OK;
#undef BAD
}

pa_status paged_kv_load_q8(const pa_plan *plan, const pa_plan *to_plan, const uint8_t *k_cache, const uint8_t *v_cache,
                           const uint8_t *k_scale, const uint8_t *v_scale, void *k_to, void *v_to, int32_t num_heads,
                           int32_t head_dim, int32_t value_dim, pa_dtype dtype, pa_stream_t stream) {
#define BAD(status, what) return fail(status, "paged_kv_load_q8: " what)
    if (!plan || !to_plan) BAD(PA_ERR_ARG, "plan is null");
    if (!pa::valid_dtype(dtype)) BAD(PA_ERR_DTYPE, "dtype must be F32, F16 or BF16");
    for (const pa_plan *p : {plan, to_plan}) {
        const pa_status shape = pa::cache_shape(p, num_heads, head_dim, value_dim, "paged_kv_load_q8");
        if (shape != PA_OK) return shape;
    }
    if (plan->sequences != to_plan->sequences) BAD(PA_ERR_SHAPE, "the plans differ in their number of sequences");
    int32_t longest = 0;
    try {
        pa::plan_facts(plan);
        // the device copy of either plan may be ahead of the host's: pages that are only
        // reserved count as held
        if (pa::plan_facts(to_plan) & pa::kFactSharedReach)
            BAD(PA_ERR_WRITE_CONFLICT, "two sequences of the destination hold one page");
        const int32_t *w = plan->words.data(), *d = to_plan->words.data();
        for (int32_t s = 0; s < plan->sequences; ++s) {
            const int64_t n = w[plan->off_seqlen + s], m = d[to_plan->off_seqlen + s];
            const int64_t most = pa::can_advance(plan, s) ? (int64_t)plan->reach[(size_t)s] * plan->page_size : n;
            if (m > most) BAD(PA_ERR_SHAPE, "a sequence of the destination is longer than its source");
            longest = std::max<int32_t>(longest, (int32_t)m);
        }
        if (longest > pa::kMaxCountedKeys) BAD(PA_ERR_LIMIT, "history above 2^30 keys");
    } catch (const std::bad_alloc &) {
        BAD(PA_ERR_LIMIT, "out of host memory");
    }
    if (plan->sequences == 0) return PA_OK;
    if (!plan->dev || !to_plan->dev) BAD(PA_ERR_STATE, "plan not uploaded");
    if (!k_cache || !v_cache || !k_scale || !v_scale || !k_to || !v_to) BAD(PA_ERR_ARG, "null tensor");
    const void *ptrs[] = {k_cache, v_cache, k_scale, v_scale, k_to, v_to};
    const char *names[] = {"k_cache", "v_cache", "k_scale", "v_scale", "k_to", "v_to"};
    const pa_status on_dev = pa::operands_on_device(ptrs, names, 6, "paged_kv_load_q8");
    if (on_dev != PA_OK) return on_dev;
    const size_t es = (size_t)pa::elem_bytes(dtype);
    for (const void *p : {(const void *)k_to, (const void *)v_to})
        if (reinterpret_cast<uintptr_t>(p) % es) BAD(PA_ERR_ARG, "operand not aligned to its element");
    const size_t slots = pa::slots_of(plan, num_heads), to = pa::slots_of(to_plan, num_heads);
    const pa::Span written[] = {{k_to, to * head_dim * es, "k_to"}, {v_to, to * value_dim * es, "v_to"}};
    const pa::Span read[] = {{k_cache, slots * head_dim, "k_cache"}, {v_cache, slots * value_dim, "v_cache"},
                             {k_scale, slots, "k_scale"}, {v_scale, slots, "v_scale"}};
    const pa_status apart = pa::spans_disjoint(written, 2, read, 4, "paged_kv_load_q8");
    if (apart != PA_OK) return apart;
    pa::Q8LoadArgs a{};
    a.plan = pa::view_of(plan);
    const pa::PlanView v = pa::view_of(to_plan);
    a.k = k_cache; a.v = v_cache; a.k_scale = k_scale; a.v_scale = v_scale;
    a.k_to = k_to; a.v_to = v_to;
    a.to_table = v.table; a.to_lens = v.seq_lens;
    a.to_width = v.width; a.to_page_size = v.page_size;
    a.hkv = num_heads; a.d = head_dim; a.dv = value_dim;
    a.dtype = dtype;
    a.status = pa::device_status_ptr();
    if (!a.status) BAD(PA_ERR_CUDA, "device status word unavailable");
    const cudaError_t e = pa::launch_q8_load(a, longest, (cudaStream_t)stream);
    if (e != cudaSuccess) return pa::fail_cuda(e, "paged_kv_load_q8 launch");
    return PA_OK;
#undef BAD
}

size_t pa_q8_workspace_bytes(const pa_plan *plan, int32_t num_heads, int32_t num_kv_heads, int32_t head_dim, int32_t value_dim,
                             pa_dtype dtype, int32_t splits, int64_t max_keys) {
    return pa_q8_window_workspace_bytes(plan, num_heads, num_kv_heads, head_dim, value_dim, dtype, splits, 0, max_keys);
}

size_t pa_q8_window_workspace_bytes(const pa_plan *plan, int32_t num_heads, int32_t num_kv_heads, int32_t head_dim,
                                    int32_t value_dim, pa_dtype dtype, int32_t splits, int32_t window, int64_t max_keys) {
    if (!plan || !pa::valid_dtype(dtype) || num_heads < 1 || num_heads > 65535 || num_kv_heads < 1 ||
        num_heads % num_kv_heads || head_dim < 1 || head_dim > PA_MAX_HEAD_DIM || value_dim < 1 ||
        value_dim > PA_MAX_HEAD_DIM || splits < 1 || splits > PA_MAX_SPLITS || window < 0 || max_keys < 0 || max_keys > INT32_MAX ||
        !pa::mass_rows_fit(plan, num_heads, splits))
        return 0;
    return pa::q8_layout(plan, num_heads, num_kv_heads, head_dim, value_dim, dtype, splits, window, max_keys).bytes;
}

pa_status paged_attn_forward_q8(const pa_plan *plan, const void *q, const uint8_t *k_cache, const uint8_t *v_cache,
                                const uint8_t *k_scale, const uint8_t *v_scale, void *out, int32_t num_heads,
                                int32_t num_kv_heads, int32_t head_dim, int32_t value_dim, float scale, int32_t causal,
                                int32_t window, pa_dtype dtype, void *workspace, size_t workspace_bytes, int32_t splits,
                                pa_stream_t stream) {
    static const char kName[] = "paged_attn_forward_q8";
#define BAD(status, what) return fail(status, "paged_attn_forward_q8: " what)
    pa_status ok = pa::check_attention_args(plan, num_heads, num_kv_heads, head_dim, value_dim, 0, scale, causal, window, dtype,
                                            false, kName);
    if (ok != PA_OK) return ok;
    ok = pa::cache_shape(plan, num_kv_heads, head_dim, value_dim, kName);
    if (ok != PA_OK) return ok;
    if (splits < 1 || splits > PA_MAX_SPLITS) BAD(PA_ERR_SPLITS, "splits must be in 1..64");
    if (!pa::mass_rows_fit(plan, num_heads, splits)) BAD(PA_ERR_LIMIT, "more than 2^31 - 1 (query, head, split) rows");
    const pa::Q8Layout lay =
        pa::q8_layout(plan, num_heads, num_kv_heads, head_dim, value_dim, dtype, splits, window, 0);
    if (std::max(plan->max_seq_len, plan->tile_longest) > pa::kMaxCountedKeys) BAD(PA_ERR_LIMIT, "history above 2^30 keys");
    if (splits > 1 && pa_workspace_bytes(plan->queries, num_heads, value_dim, splits) > PA_WORKSPACE_LIMIT_BYTES)
        BAD(PA_ERR_WORKSPACE, "split partials above the 1 GiB limit");
    if (plan->queries > 0 && lay.bytes > 0) {
        if (!workspace) BAD(PA_ERR_WORKSPACE, "workspace is null");
        if (workspace_bytes < lay.bytes) BAD(PA_ERR_WORKSPACE, "workspace too small");
        if (!pa::aligned16(workspace)) BAD(PA_ERR_WORKSPACE, "workspace not 16-byte aligned");
    }
    if (plan->queries == 0) return PA_OK;
    if (!plan->dev) BAD(PA_ERR_STATE, "plan not uploaded");
    if (!q || !k_cache || !v_cache || !k_scale || !v_scale || !out) BAD(PA_ERR_ARG, "null tensor");
    void *const ws = lay.bytes > 0 ? workspace : nullptr;
    const void *ptrs[] = {q, k_cache, v_cache, k_scale, v_scale, out, ws};
    const char *names[] = {"q", "k_cache", "v_cache", "k_scale", "v_scale", "out", "the workspace"};
    ok = pa::operands_on_device(ptrs, names, 7, kName);
    if (ok != PA_OK) return ok;
    const size_t es = (size_t)pa::elem_bytes(dtype), rows = (size_t)plan->queries * num_heads,
                 slots = pa::slots_of(plan, num_kv_heads);
    for (const void *p : {q, (const void *)out})
        if (reinterpret_cast<uintptr_t>(p) % es) BAD(PA_ERR_ARG, "operand not aligned to its element");
    const pa::Span written[] = {{out, rows * value_dim * es, "out"}, {ws, workspace_bytes, "the workspace"}};
    const pa::Span read[] = {{q, rows * head_dim * es, "q"}, {k_cache, slots * head_dim, "k_cache"},
                             {v_cache, slots * value_dim, "v_cache"}, {k_scale, slots, "k_scale"}, {v_scale, slots, "v_scale"}};
    ok = pa::spans_disjoint(written, 2, read, 5, kName);
    if (ok != PA_OK) return ok;

    pa::Q8AttnArgs x{};
    pa::AttnArgs &a = x.a;
    a.plan = pa::view_of(plan);
    a.q = q; a.k = k_cache; a.v = v_cache; a.out = out;
    x.k_scale = k_scale; x.v_scale = v_scale;
    a.hq = num_heads; a.hkv = num_kv_heads; a.d = head_dim; a.dv = value_dim;
    a.scale = scale; a.causal = causal; a.window = window; a.splits = splits; a.dtype = dtype;
    a.status = pa::device_status_ptr();
    if (!a.status) BAD(PA_ERR_CUDA, "device status word unavailable");
    char *const base = static_cast<char *>(ws);
    int sms = 0;
    if (pa::device_sms(sms) != cudaSuccess) sms = 0;
    if (plan->n_tiles == 0 && splits > 1 && sms > 0) {
        cudaStreamCaptureStatus capture = cudaStreamCaptureStatusNone;
        const bool asked = cudaStreamIsCapturing((cudaStream_t)stream, &capture) == cudaSuccess;
        if (!asked) (void)cudaGetLastError();        // (the launch says what is wrong with the stream)
        a.splits = pa::q8_splits(plan, x, sms, !asked || capture != cudaStreamCaptureStatusNone);
    }
    if (a.splits > 1) {
        a.ws_o = reinterpret_cast<float *>(base);
        a.ws_lse = reinterpret_cast<float *>(base + (splits * rows * value_dim * sizeof(float) + 255) / 256 * 256);
    }
    cudaStream_t st = (cudaStream_t)stream;
    cudaEvent_t t0, t1;
    pa::take_timing(t0, t1);
    cudaError_t e = cudaSuccess;
    auto mark = [&](cudaEvent_t ev) {
        if (ev && e == cudaSuccess) e = cudaEventRecord(ev, st);
    };
    // The tiles' histories as 16-bit pages for the tensor-core prefill kernel, which then
    // reads them once per query head and tile; what the caller gave beyond the need makes
    // room for longer ones (staged plans).
    pa::AttnArgs wide = a;
    if (lay.tiles) {
        const int64_t more = (int64_t)((workspace_bytes - lay.bytes) / (2 * lay.page_bytes));
        const int64_t room = std::min<int64_t>(lay.room + more, INT32_MAX / pa::kCopyPage);
        wide.k = base + lay.k;
        wide.v = base + lay.k + (size_t)room * lay.page_bytes;
        wide.plan.table = reinterpret_cast<const int32_t *>(base + lay.table);
        wide.plan.width = lay.width;
        wide.plan.page_size = pa::kCopyPage;
        wide.plan.pages = (int32_t)room;
    }
    if (lay.tiles && pa::prefill_supported(wide)) {
        int2 *const places = reinterpret_cast<int2 *>(base + lay.places);
        // the decode items beside the copy and the tiles, on SMs of their own
        const int beside = pa::q8_sms_beside_prefill(plan, a, lay.copied.blocks, sms);
        pa::SideStream *side = beside > 0 ? pa::side_stream(st) : nullptr;
        bool forked = false;
        if (side) {
            x.a.max_ctas = beside;
            wide.max_ctas = sms - beside;
            e = pa::fork_side(*side, st);
            forked = e == cudaSuccess;
            if (e == cudaSuccess) e = pa::launch_q8_decode(x, true, plan->longest_run, side->stream);
        }
        if (e == cudaSuccess) e = pa::launch_q8_places(a.plan, places, window, pa::kCopyPage, wide.plan.pages, a.status, st);
        pa::Q8LoadArgs c{};
        c.plan = a.plan;
        c.k = k_cache; c.v = v_cache; c.k_scale = k_scale; c.v_scale = v_scale;
        c.k_to = const_cast<void *>(wide.k); c.v_to = const_cast<void *>(wide.v);
        c.places = places;
        c.to_table_out = reinterpret_cast<int32_t *>(base + lay.table);
        c.to_width = lay.width;
        c.to_page_size = pa::kCopyPage;
        c.hkv = num_kv_heads; c.d = head_dim; c.dv = value_dim;
        c.dtype = dtype;
        c.status = a.status;
        if (e == cudaSuccess) e = pa::launch_q8_load(c, (int)lay.copied.longest, st);
        mark(t0);
        if (e == cudaSuccess) e = pa::launch_prefill(wide, st);
        mark(t1);
        if (forked)
            e = pa::join_side(*side, st, e);
        else if (e == cudaSuccess && plan->n_decode > 0)
            e = pa::launch_q8_decode(x, true, plan->longest_run, st);
        if (e == cudaSuccess && splits > 1) e = pa::launch_merge(a, false, st);
    } else {
        const bool all_decode = plan->n_tiles == 0;
        mark(t0);
        if (e == cudaSuccess) e = pa::launch_q8_decode(x, all_decode, plan->longest_run, st);
        mark(t1);
        if (e == cudaSuccess && a.splits > 1) e = pa::launch_merge(a, all_decode, st);
    }
    if (e != cudaSuccess) return pa::fail_cuda(e, kName);
    return PA_OK;
#undef BAD
}

}  // extern "C"
