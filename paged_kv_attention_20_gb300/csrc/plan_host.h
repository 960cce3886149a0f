// Host-side internals shared by the entry points: the plan object, error
// reporting and the operand checks that come before every launch.
#pragma once

#include <atomic>
#include <cstdint>
#include <mutex>
#include <vector>

#include "pa_internal.h"

struct pa_plan {
    int32_t queries = 0, sequences = 0, width = 0, page_size = 0, pages = 0;
    int32_t n_decode = 0, n_tiles = 0, n_tile_queries = 0;
    int64_t max_seq_len = 0;          // longest sequence any decode item reads
    int64_t tile_longest = 0;         // keys of the longest sequence with prefill tiles
    std::vector<std::pair<int32_t, int32_t>> tile_starts;   // sequences with prefill tiles, the lowest position of their queries
    int32_t longest_run = 1, decode_runs = 0;    // of decode items at consecutive positions of a sequence
    std::vector<int32_t> words;       // host copy of the device metadata
    size_t off_qmeta = 0, off_seqlen = 0, off_table = 0, off_decode = 0, off_tiles = 0, off_order = 0;
    const int32_t *dev = nullptr;     // caller's device copy (after upload)
    // visible keys of the prefill tiles' queries and of the decode items, without
    // a window, non-causal [0] and causal [1] (the mixed call's SM share needs them)
    double keys_tiles[2] = {0, 0}, keys_decode[2] = {0, 0};
    // facts of the host copy that only some calls need, worked out on first use
    // (plan_facts): 0 = not yet, else kFactsKnown | flags.  `reach` then has the
    // entries of each row that hold the sequence's keys or may come to hold some
    // without the host's knowledge (graph replays of pa_plan_advance move the device
    // copy alone): the used ones and, where the plan can advance, those after them up
    // to the first that names no page or a page in use (padding).  `held` has a bit
    // for every page that such an entry names.
    mutable std::atomic<int32_t> facts{0};
    mutable std::mutex facts_mutex;
    mutable std::vector<uint64_t> held;
    mutable std::vector<int32_t> reach;
    mutable std::vector<uint8_t> moves;   // per sequence: pa_plan_advance moves it on
    // what the queried sequences begin with (plan_prefix), worked out on first use and again
    // after an advance: pages that all of them hold first, the lowest query position
    mutable std::atomic<int32_t> prefix_known{0};
    mutable int32_t prefix_pages = 0, prefix_lowest = 0;
};

namespace pa {

constexpr int32_t kFactsKnown = 1;
constexpr int32_t kFactSharedPages = 2;     // some page is held by two used block-table entries
constexpr int32_t kFactRepeatedItems = 4;   // some sequence has more than one decode item
constexpr int32_t kFactSharedReach = 8;     // some page is held by two entries within `reach`

// Facts about the plan's host copy (kFact* flags); std::bad_alloc when the host
// has no memory for them.
int32_t plan_facts(const pa_plan *plan);
// Leading pages that every queried sequence of the host copy holds, and the lowest query position.
void plan_prefix(const pa_plan *plan, int32_t &pages, int32_t &lowest);
// Whether sequence s of the plan may have advanced on the device (after plan_facts).
inline bool can_advance(const pa_plan *plan, int32_t s) { return plan->moves[(size_t)s] != 0; }

// Visible keys summed over the prefill tiles' queries and over the decode items.
void visible_key_sums(const pa_plan *plan, int causal, int window, double &keys_tiles, double &keys_decode);
// Most keys that a decode item sees.
int64_t most_visible_keys(const pa_plan *plan, int causal, int window);

// A mixed call's decode items can run beside its prefill tiles: the tiles are
// bound by the tensor core and the softmax, the decode items by HBM, and one
// after the other they leave one of the two idle for the whole of the other.
// The decode kernel then runs on a second stream of the caller's thread (one
// per device, created on first use outside stream capture), forked from and
// joined back into the caller's stream with events, so the call stays one
// ordered step of that stream and can be captured into a graph.
struct SideStream {
    cudaStream_t stream = nullptr;
    cudaEvent_t fork = nullptr, join = nullptr;
    bool failed = false;
};
// The calling thread's on the current device; null where there is none yet and `st` is being captured,
// and where it belongs to a capture that is not `st`'s.
SideStream *side_stream(cudaStream_t st);
// What is put on the side stream from here on comes after what `st` holds.
cudaError_t fork_side(SideStream &side, cudaStream_t st);
// And what `st` gets from here on after that; also where a launch in between failed with `e`, as
// the work beside still writes the caller's tensors.  The first error.
cudaError_t join_side(SideStream &side, cudaStream_t st, cudaError_t e);

// The events of pa_time_next_kernel, for the one call that takes them.
void take_timing(cudaEvent_t &start, cudaEvent_t &stop);

pa_status fail(pa_status st, const char *msg);
pa_status fail_cuda(cudaError_t e, const char *what);
bool valid_dtype(pa_dtype d);
int elem_bytes(pa_dtype d);
bool aligned16(const void *ptr);
PlanView view_of(const pa_plan *p);
// PA_OK when every non-null pointer of `ptrs` is device memory of the current
// device, else PA_ERR_ARG naming the operand.
pa_status operands_on_device(const void *const *ptrs, const char *const *names, int n, const char *call);

// A byte range of an operand.
struct Span {
    const void *at;
    size_t bytes;
    const char *name;
};
// PA_OK when none of the `written` ranges meets another of them or one of the
// `read` ranges, else PA_ERR_ARG naming the two.  Null and empty ranges meet nothing.
pa_status spans_disjoint(const Span *written, int n_written, const Span *read, int n_read, const char *call);

// Workspace of paged_attn_forward_mass: byte offsets of its parts.
struct MassLayout {
    size_t lse, lse_final, items, tiles, blocks, tile_lse, scores, bytes;   // the split partials start at 0
    int32_t max_blocks;                                    // key blocks of sequences with tiles
    int64_t cap;                                           // keys of one score row
};
// Whether the (query, head, split) rows can be counted in 32 bits, as the kernels' grids do.
bool mass_rows_fit(const pa_plan *plan, int32_t hq, int32_t splits);
// For rows that fit; bytes: SIZE_MAX when the score rows pass 2^62 bytes.
// max_keys: keys the score rows hold at least; 0: the longest history of the host copy.
// window: the call's, 0 when it is not causal (a causal query sees at most `window` keys).
MassLayout mass_layout(const pa_plan *plan, int32_t hq, int32_t dv, int32_t splits, int32_t window, int64_t max_keys);
// The kernels that follow the attention of `a` and add its weights to key_mass:
// the decode items with stored scores (merging the split outputs in the same
// launch when `merge`), and the tiles -- or, where the tiles have no tensor-core
// kernel, every query -- with recomputed ones.
cudaError_t add_item_mass(const pa_plan *plan, const AttnArgs &a, const MassLayout &lay, char *ws, float *key_mass, bool merge,
                          bool use_list, cudaStream_t st);
cudaError_t add_tile_mass(const pa_plan *plan, const AttnArgs &a, const MassLayout &lay, char *ws, float *key_mass,
                          cudaStream_t st);
// Attention entry body with totals; key_mass is not null.
pa_status attention_with_mass(const pa_plan *plan, const void *q, const void *k, const void *v, void *out,
                              float *key_mass, int32_t hq, int32_t hkv, int32_t d, int32_t dv, float scale,
                              int32_t causal, int32_t window, pa_dtype dtype, void *ws, size_t ws_bytes, int32_t splits,
                              cudaStream_t st, const char *name);

}  // namespace pa
