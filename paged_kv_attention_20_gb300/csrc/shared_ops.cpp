// Attention of a batch whose sequences begin with the same pages: the prefix is attended
// once for all queries, each sequence's own keys as always, and the partials are merged.

#include <algorithm>

#include "per_device.h"
#include "plan_host.h"

using pa::fail;

namespace {

// SMs that the prefix's kernel takes while the own keys are attended on the others (0: one after
// the other), and how long the call is thought to take with them, in seconds.
struct Beside {
    int32_t sms;
    double time;
};

// For the splits that a call is given.  The prefix's units, (128 rows of queries and heads, KV head,
// split), take 9 us to start and end and 1 us a tile of 128 keys, in rounds on the SMs that they
// have; a split's partials are written and read again.  The own keys of groups of up to seven heads
// are read by many blocks at 34 GB/s an SM, 3.3 TB/s in all beside the prefix, and at 4.4 TB/s on the
// whole GPU where the prefix has ended.  Those of larger groups have a persistent kernel that keeps
// to its SMs: 3.2 us a unit and 1.35 us a tile of it.  The SMs are those that make 1 to 8 rounds.
// Against sweeps of the share (16 to 256 queries, 7 or 8 split counts each, groups of 4 and 8) the one
// taken is the best or within 5 % of it, 12 % where a call has far more splits than it should.  64
// queries behind 16384 keys, 9 splits: with 1, 512 and 2048 own keys 44, 81 and 168 us; on the SMs of
// the best split count, which the call does not run with, 45, 86 and 200 (groups of 8: 83, 105 and
// 160; 123, 120 and 191).
Beside beside_of(const pa_plan *plan, int32_t hq, int32_t hkv, int32_t shared, int32_t prefix_splits, int32_t splits, int32_t sms) {
    const int64_t group = hq / hkv, per_tile = std::max<int64_t>(1, 128 / group);
    const int64_t units = (plan->queries + per_tile - 1) / per_tile * hkv * prefix_splits;
    const double tiles = shared / 128.0 / prefix_splits;
    const double own_keys = std::max(0.0, plan->keys_decode[1] + plan->keys_tiles[1] - (double)plan->queries * shared);
    const double own_bytes = own_keys * hkv * 512.0;
    const double partials = (double)plan->queries * hq * 128 * 4 * 2 / 4e12 * prefix_splits;
    auto prefix = [&](int64_t n) { return 9e-6 + (double)((units + n - 1) / n) * (1e-6 + 1e-6 * tiles); };
    const bool persistent = group >= 8 && group <= 128;
    const int64_t own_units = std::max<int64_t>(1, (int64_t)plan->n_decode * hkv * splits);
    const double unit = 3.2e-6 + 1.35e-6 * std::max(1.0, own_keys * hkv / (double)own_units / 128);
    auto rounds = [&](int64_t n) { return std::max((double)((own_units + n - 1) / n) * unit, own_bytes / 4.4e12); };
    Beside best{0, prefix(sms) + (persistent ? rounds(sms) : 5e-6 + own_bytes / 4.4e12) + partials};
    if (plan->n_tiles > 0) return best;
    for (int64_t r = 1; r <= 8; ++r) {
        const int64_t n = (units + r - 1) / r;
        if (n > sms - 8) continue;
        const double t = prefix(n), rate = std::min(3.4e10 * (double)(sms - n), 3.3e12);
        const double own = persistent ? rounds(sms - n) : 5e-6 + std::min(own_bytes / rate, t + std::max(0.0, own_bytes - rate * t) / 4.4e12);
        const double time = std::max(t, own) + partials + 3e-6;          // a fork and a join more
        if (time < best.time) best = Beside{(int32_t)n, time};
    }
    return best;
}

// Splits of the prefix, those that end soonest, and of the sequences' own keys, the split heuristic's
// for what is left of the sequences.
struct Layout {
    int32_t prefix_splits, splits;
};

Layout layout_of(const pa_plan *plan, int32_t hq, int32_t hkv, int32_t shared, int32_t sms) {
    Layout best{1, 1};
    if (plan->queries == 0) return best;
    const int64_t group = hq / hkv;
    const int64_t longest = std::max<int64_t>(0, std::max(plan->max_seq_len, plan->tile_longest) - shared);
    const int64_t blocks = std::max<int64_t>(1, (int64_t)plan->n_decode * hkv * ((group + 3) / 4) + (int64_t)plan->n_tiles * hq);
    int64_t own = (blocks >= sms ? 4 : 8) * (int64_t)sms / blocks;
    own = std::min<int64_t>(own, std::max<int64_t>(1, longest / (4 * (int64_t)plan->page_size)));
    best.splits = (int32_t)std::max<int64_t>(1, std::min<int64_t>(own, PA_MAX_SPLITS / 2));
    const int64_t most = std::max<int64_t>(1, std::min<int64_t>(PA_MAX_SPLITS / 2, shared / 128));
    double best_t = -1;
    for (int32_t s = 1; s <= most; ++s) {
        const double t = beside_of(plan, hq, hkv, shared, s, best.splits, sms).time;
        if (best_t >= 0 && t >= 0.97 * best_t) continue;           // (more splits have to be worth it)
        best_t = t;
        best.prefix_splits = s;
    }
    return best;
}

void shared_splits(const pa_plan *plan, int32_t hq, int32_t hkv, int32_t shared, int32_t sms, int32_t out[2]) {
    const Layout l = layout_of(plan, hq, hkv, shared, sms);
    out[0] = l.prefix_splits;
    out[1] = l.splits;
    // A prefix that all queries together read in less than 20 MB (of 16-bit heads of 128) is not
    // worth a launch and partials of its own: 8 sequences behind 512 keys of 8 KV heads, 17 MB,
    // take 16 us that way and 24 with it; 8 behind 1024 and 16 behind 512, 34 MB, 23-25 and 24.
    if (plan->queries > 0 && (double)plan->queries * shared * hkv * 512.0 < 20e6) {
        out[1] += out[0];
        out[0] = 0;
    }
}

}  // namespace

extern "C" {

pa_status paged_attn_shared_splits(const pa_plan *plan, int32_t num_heads, int32_t num_kv_heads, int32_t shared,
                                   int32_t num_sms, int32_t out[2]) {
#define BAD(status, what) return fail(status, "paged_attn_shared_splits: " what)
    if (!plan || !out) BAD(PA_ERR_ARG, "null argument");
    if (num_heads < 1 || num_kv_heads < 1 || num_heads % num_kv_heads)
        BAD(PA_ERR_SHAPE, "num_heads must be a positive multiple of num_kv_heads");
    if (shared < 0 || num_sms < 1) BAD(PA_ERR_ARG, "shared must be >= 0 and num_sms >= 1");
    shared_splits(plan, num_heads, num_kv_heads, shared, num_sms, out);
    return PA_OK;
#undef BAD
}

pa_status paged_attn_forward_shared(const pa_plan *plan, const void *q, const void *k_cache, const void *v_cache, void *out,
                                    int32_t num_heads, int32_t num_kv_heads, int32_t head_dim, int32_t value_dim, float scale,
                                    int32_t causal, int32_t shared, pa_dtype dtype, void *workspace, size_t workspace_bytes,
                                    int32_t prefix_splits, int32_t splits, pa_stream_t stream) {
    static const char kName[] = "paged_attn_forward_shared";
#define BAD(status, what) return fail(status, "paged_attn_forward_shared: " what)
    pa_status ok = pa::check_attention_args(plan, num_heads, num_kv_heads, head_dim, value_dim, 0, scale, causal, 0, dtype,
                                            false, kName);
    if (ok != PA_OK) return ok;
    if (shared < 0) BAD(PA_ERR_ARG, "shared must be >= 0");
    if (prefix_splits < 0 || splits < 1 || prefix_splits > PA_MAX_SPLITS || splits > PA_MAX_SPLITS ||
        prefix_splits + splits > PA_MAX_SPLITS)
        BAD(PA_ERR_SPLITS, "prefix_splits must be at least 0, splits 1, and 64 in all");
    const int32_t all = prefix_splits + splits;
    if (!pa::mass_rows_fit(plan, num_heads, all)) BAD(PA_ERR_LIMIT, "more than 2^31 - 1 (query, head, split) rows");
    const size_t need = pa_workspace_bytes(plan->queries, num_heads, value_dim, all);
    if (need > PA_WORKSPACE_LIMIT_BYTES) BAD(PA_ERR_WORKSPACE, "workspace above the 1 GiB limit");
    if (plan->queries > 0) {
        if (!workspace) BAD(PA_ERR_WORKSPACE, "workspace is null");
        if (workspace_bytes < need) BAD(PA_ERR_WORKSPACE, "workspace too small");
        if (!pa::aligned16(workspace)) BAD(PA_ERR_WORKSPACE, "workspace not 16-byte aligned");
        if (shared % plan->page_size) BAD(PA_ERR_SHAPE, "shared must be a multiple of the page size");
        int32_t pages = 0, lowest = 0;
        pa::plan_prefix(plan, pages, lowest);
        if (shared / plan->page_size > pages) BAD(PA_ERR_SHAPE, "the queried sequences do not begin with that many shared pages");
        if (causal && lowest < shared) BAD(PA_ERR_SHAPE, "a query lies within the shared keys");
        // without a causal end a sequence's keys are all seen; none may end inside the prefix
        const int32_t *w = plan->words.data();
        if (!causal)
            for (int32_t i = 0; i < plan->queries; ++i)
                if (w[plan->off_seqlen + w[plan->off_qmeta + 4 * (size_t)i]] < shared)
                    BAD(PA_ERR_SHAPE, "a sequence ends within the shared keys");
    }
    if (plan->queries == 0) return PA_OK;
    if (!plan->dev) BAD(PA_ERR_STATE, "plan not uploaded");
    if (!q || !k_cache || !v_cache || !out) BAD(PA_ERR_ARG, "null tensor");
    const void *ptrs[] = {q, k_cache, v_cache, out, workspace};
    const char *names[] = {"q", "the key cache", "the value cache", "out", "the workspace"};
    ok = pa::operands_on_device(ptrs, names, 5, kName);
    if (ok != PA_OK) return ok;
    const size_t es = (size_t)pa::elem_bytes(dtype), rows = (size_t)plan->queries * num_heads,
                 slots = (size_t)plan->pages * plan->page_size * num_kv_heads;
    for (const void *p : {q, k_cache, v_cache, (const void *)out})
        if (reinterpret_cast<uintptr_t>(p) % es) BAD(PA_ERR_ARG, "operand not aligned to its element");
    const pa::Span written[] = {{out, rows * value_dim * es, "out"}, {workspace, workspace_bytes, "the workspace"}};
    const pa::Span read[] = {{q, rows * head_dim * es, "q"}, {k_cache, slots * head_dim * es, "the key cache"},
                             {v_cache, slots * value_dim * es, "the value cache"}};
    ok = pa::spans_disjoint(written, 2, read, 3, kName);
    if (ok != PA_OK) return ok;

    pa::AttnArgs a{};
    a.plan = pa::view_of(plan);
    a.q = q; a.k = k_cache; a.v = v_cache; a.out = out;
    a.hq = num_heads; a.hkv = num_kv_heads; a.d = head_dim; a.dv = value_dim;
    a.scale = scale; a.causal = causal; a.dtype = dtype;
    a.status = pa::device_status_ptr();
    if (!a.status) BAD(PA_ERR_CUDA, "device status word unavailable");
    a.ws_o = static_cast<float *>(workspace);
    a.ws_lse = reinterpret_cast<float *>(static_cast<char *>(workspace) + (all * rows * value_dim * sizeof(float) + 255) / 256 * 256);
    cudaStream_t st = (cudaStream_t)stream;
    cudaEvent_t t0, t1;
    pa::take_timing(t0, t1);
    cudaError_t e = cudaSuccess;
    auto mark = [&](cudaEvent_t ev) {
        if (ev && e == cudaSuccess) e = cudaEventRecord(ev, st);
    };
    pa::SideStream *side = nullptr;
    bool forked = false;
    pa::AttnArgs own = a, merged = a;
    own.splits = merged.splits = all;
    if (shared > 0 && prefix_splits > 0 && pa::prefix_supported(a)) {
        // partials: the prefix's splits, then each sequence's own
        pa::AttnArgs prefix = a;
        prefix.splits = prefix_splits;
        own.splits = splits;
        own.skip = shared;
        own.ws_o = a.ws_o + (size_t)prefix_splits * rows * value_dim;
        own.ws_lse = a.ws_lse + (size_t)prefix_splits * rows;
        int sms = 0;
        const int share = pa::device_sms(sms) == cudaSuccess
                              ? beside_of(plan, num_heads, num_kv_heads, shared, prefix_splits, splits, sms).sms
                              : 0;
        side = share > 0 ? pa::side_stream(st) : nullptr;
        if (side) {
            // the prefix first, so that its CTAs hold their SMs; the own keys from the side stream
            prefix.max_ctas = share;
            own.max_ctas = sms - share;
            e = pa::fork_side(*side, st);
            forked = e == cudaSuccess;
        }
        mark(t0);
        if (e == cudaSuccess) e = pa::launch_prefix(prefix, shared, st);
        mark(t1);
        t0 = t1 = nullptr;
    }
    // (else every sequence attends to all of its keys)
    const bool tiles = plan->n_tiles > 0 && pa::prefill_supported(own);
    cudaStream_t to = side ? side->stream : st;
    mark(t0);
    if (e == cudaSuccess && tiles) e = pa::launch_prefill(own, to);
    if (e == cudaSuccess && (!tiles || plan->n_decode > 0)) e = pa::launch_decode(own, tiles || plan->n_tiles == 0, to);
    mark(t1);
    if (forked) e = pa::join_side(*side, st, e);
    if (e == cudaSuccess) e = pa::launch_merge(merged, false, st);
    if (e != cudaSuccess) return pa::fail_cuda(e, kName);
    return PA_OK;
#undef BAD
}

}  // extern "C"
