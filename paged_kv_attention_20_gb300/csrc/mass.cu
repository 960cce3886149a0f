// Per-key totals of the softmax weights (paged_attn_forward_mass).
//
// For key j of a sequence and KV head kv the call adds
//   sum over the sequence's queries q and the heads h of group kv of
//   softmax_j = 2^(s_qhj - lse_qh)            (s and lse in log2 units)
// to key_mass[page, kv, row].  The log-sum-exp is only known once a query's
// whole history has been seen, so the attention kernels run first and this pass
// follows:
//  * decode items: the decode kernels leave their scores (4 bytes per key and
//    head, against 2*(D+Dv)/G bytes of cache per key and head) in the workspace,
//    and `mass_items_kernel` turns them into weights: the cache is read once;
//  * prefill tiles: the scores are recomputed from K and Q, tile by tile.
// Every key has one owner that adds its terms in a fixed order: no atomics, and
// the same bits on every run.  Sequences do not share pages (checked on the
// host).

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <type_traits>

#include "merge.cuh"
#include "pa_internal.h"

namespace pa {
namespace {

constexpr float kLog2e = 1.4426950408889634f;

template <typename T> __device__ __forceinline__ float to_f(T x);
template <> __device__ __forceinline__ float to_f<float>(float x) { return x; }
template <> __device__ __forceinline__ float to_f<__half>(__half x) { return __half2float(x); }
template <> __device__ __forceinline__ float to_f<__nv_bfloat16>(__nv_bfloat16 x) { return __bfloat162float(x); }

// Log-sum-exp of a row over its splits, in log2 units.
__device__ __forceinline__ float merged_lse2(const MassArgs &a, int64_t row) {
    const int64_t rows = (int64_t)a.plan.queries * a.hq;
    float m = -INFINITY;
    for (int s = 0; s < a.splits; ++s) m = fmaxf(m, a.lse[s * rows + row]);
    if (a.splits == 1 || m == -INFINITY) return m * kLog2e;
    float t = 0.f;
    for (int s = 0; s < a.splits; ++s) t += exp2f((a.lse[s * rows + row] - m) * kLog2e);
    return m * kLog2e + log2f(t);
}

__global__ void lse_final_kernel(MassArgs a, float *out) {
    griddep_wait();
    griddep_launch();
    const int64_t row = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
    if (row < (int64_t)a.plan.queries * a.hq) out[row] = merged_lse2(a, row) / kLog2e;
}

// ---------------------------------------------------------------- grouping --
__device__ __forceinline__ int record_seq(const PlanView &p, int kind, int i) {
    if (kind == kMassTiles) return p.tiles[i].x;
    return p.qmeta[kind == kMassItems ? p.decode[i] : i].x;
}

constexpr int kIndexThreads = 1024;

// Inclusive prefix sum over the CTA (32 warps); `sums` is scratch of 32 ints.
__device__ __forceinline__ int block_prefix(int c, int *sums) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int x = c;
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
    }
    if (lane == 31) sums[warp] = x;
    __syncthreads();
    int before = 0;
    for (int w = 0; w < warp; ++w) before += sums[w];
    __syncthreads();
    return before + x;
}

// One CTA of 1024 threads: group_start[s] .. group_start[s+1] delimit the records of sequence s
// in group_list, in ascending record order (a stable counting sort).
__device__ __forceinline__ void group_records(const MassArgs &a, int kind, int n) {
    __shared__ __align__(16) int seqs[kIndexThreads];
    __shared__ int carry, sums[32];
    const int S = a.plan.sequences, tid = threadIdx.x;
    if (n <= kIndexThreads && S < kIndexThreads) {
        // the usual sizes: one pass in shared memory, a sequence and a record per thread
        __shared__ int count[kIndexThreads];
        count[tid] = 0;
        const int mine = tid < n ? record_seq(a.plan, kind, tid) : -1;
        seqs[tid] = mine;
        __syncthreads();
        if (mine >= 0) atomicAdd(&count[mine], 1);
        __syncthreads();
        const int c = count[tid];
        const int upto = block_prefix(c, sums);
        if (tid <= S) a.group_start[tid] = upto - c;
        count[tid] = upto - c;
        __syncthreads();
        if (mine >= 0) {
            // records of the same sequence before mine
            int before = 0, t = 0;
            for (; t + 4 <= tid; t += 4) {
                const int4 v = *reinterpret_cast<const int4 *>(seqs + t);
                before += (v.x == mine) + (v.y == mine) + (v.z == mine) + (v.w == mine);
            }
            for (; t < tid; ++t) before += seqs[t] == mine;
            a.group_list[count[mine] + before] = tid;
        }
        return;
    }
    for (int s = tid; s <= S; s += kIndexThreads) a.group_start[s] = 0;
    __syncthreads();
    for (int i = tid; i < n; i += kIndexThreads) atomicAdd(&a.group_start[record_seq(a.plan, kind, i)], 1);
    if (tid == 0) carry = 0;
    __syncthreads();
    // exclusive prefix sums of the counts, 1024 sequences a step; the entry of s
    // then serves as the cursor of its records and ends at its upper bound
    for (int base = 0; base <= S; base += kIndexThreads) {
        const int s = base + tid;
        const int c = s < S ? a.group_start[s] : 0;
        const int x = block_prefix(c, sums);
        if (s <= S) a.group_start[s] = carry + x - c;
        __syncthreads();
        if (tid == kIndexThreads - 1) carry += x;
        __syncthreads();
    }
    for (int base = 0; base < n; base += kIndexThreads) {
        const int i = base + tid, cnt = min(n - base, kIndexThreads);
        const int mine = i < n ? record_seq(a.plan, kind, i) : -1;
        seqs[tid] = mine;
        __syncthreads();
        int before = 0, after = 0;
        for (int t = 0; t < cnt; ++t) {
            const bool same = seqs[t] == mine;
            before += same && t < tid;
            after += same && t > tid;
        }
        const int at = i < n ? a.group_start[mine] : 0;
        __syncthreads();
        if (i < n) {
            a.group_list[at + before] = i;
            if (after == 0) a.group_start[mine] = at + before + 1;
        }
        __syncthreads();
    }
    // the cursors stand at the upper bounds: shift them into place, from the end
    for (int base = (S / kIndexThreads) * kIndexThreads; base >= 0; base -= kIndexThreads) {
        const int s = base + tid;
        const int v = s <= S ? (s == 0 ? 0 : a.group_start[s - 1]) : 0;
        __syncthreads();
        if (s <= S) a.group_start[s] = v;
        __syncthreads();
    }
}

__global__ void __launch_bounds__(kIndexThreads) mass_index_kernel(MassArgs a, int kind, int n) {
    griddep_wait();
    griddep_launch();
    group_records(a, kind, n);
}

// ------------------------------------------------------------------- tiles --
// Block 0 groups the tiles by sequence and lists the key blocks of the sequences
// that have some: blocks[i] = {sequence, first key, its tiles [z, w) in the
// list}.  Every other block lays out one tile's log-sum-exps: [Hq][128], merged
// over the splits, negated and in log2 units, 0 past the tile's queries.
__global__ void __launch_bounds__(kIndexThreads) mass_tiles_prepare_kernel(MassArgs a) {
    griddep_wait();
    griddep_launch();
    const int tid = threadIdx.x;
    if (blockIdx.x == 0) {
        group_records(a, kMassTiles, a.plan.n_tiles);
        __syncthreads();                       // group_start is read below by other threads than wrote it
        __shared__ int sums[32], upto[kIndexThreads];
        int before = 0;                        // blocks of the sequences before this step's 1024
        const int S = a.plan.sequences;
        for (int base = 0; base < S; base += kIndexThreads) {
            const int s = base + tid;
            const int z = s < S ? a.group_start[s] : 0, w = s < S ? a.group_start[s + 1] : 0;
            int c = w > z ? a.plan.seq_lens[s] : 0;
            if (c > kMaxCountedKeys) {         // (only a device copy's length: the host refuses it)
                atomicCAS(a.status, 0, PA_DEVICE_RANGE);
                c = 0;
            }
            c = (c + 127) / 128;
            upto[tid] = block_prefix(c, sums);
            __syncthreads();
            const int total = upto[kIndexThreads - 1];
            for (int i = tid; i < total; i += kIndexThreads) {
                int lo = 0, hi = kIndexThreads - 1;    // first entry whose inclusive sum passes i
                while (lo < hi) {
                    const int mid = (lo + hi) / 2;
                    if (upto[mid] > i)
                        hi = mid;
                    else
                        lo = mid + 1;
                }
                const int first = lo ? upto[lo - 1] : 0, q = base + lo;
                if (before + i < a.max_blocks)
                    a.blocks[before + i] = make_int4(q, 128 * (i - first), a.group_start[q], a.group_start[q + 1]);
            }
            before += total;
            __syncthreads();
        }
        if (tid == 0) {
            if (before > a.max_blocks) atomicCAS(a.status, 0, PA_DEVICE_RANGE);
            *a.n_blocks = min(before, a.max_blocks);
        }
        return;
    }
    const int tile_id = (int)blockIdx.x - 1;
    const int4 tile = a.plan.tiles[tile_id];
    __shared__ float part[128][33];
    float *out = a.tile_lse + (int64_t)tile_id * a.hq * 128;
    for (int h0 = 0; h0 < a.hq; h0 += 32) {
        __syncthreads();
        for (int i = tid; i < 128 * 32; i += kIndexThreads) {
            const int c = i >> 5, h = h0 + (i & 31);
            part[c][i & 31] = c < tile.z && h < a.hq ? -merged_lse2(a, (int64_t)(tile.y + c) * a.hq + h) : 0.f;
        }
        __syncthreads();
        for (int i = tid; i < 128 * 32; i += kIndexThreads) {
            const int h = h0 + (i >> 7), c = i & 127;
            if (h < a.hq) out[(int64_t)h * 128 + c] = part[c][i >> 7];
        }
    }
}

// ------------------------------------------------------------ decode items --
constexpr int kItemThreads = 256, kItemWarps = kItemThreads / 32;
constexpr int kItemKeys = 4 * kItemThreads;     // four keys a thread and step
constexpr int kHeadsAtOnce = 4;                 // score rows in flight
constexpr int kMaxStagedHeads = 64;

// A quad at the ends of the visible range loads its four scores all the same
// (score_origin keeps them inside the row; entries no key has may hold anything and are
// not added) and its totals before any is written: an end costs no chain of loads
// (24 sequences of four drafted tokens, window 1000: the pass 14.8 us, so 12.4, and
// 10.8 with as many blocks as the window touches).
template <bool kQuads>
__device__ __forceinline__ void add_to_part(const MassArgs &a, const int32_t *trow, int kvh, int ps_shift, int j, int in,
                                            const float (&p)[4]) {
    const int ps = a.plan.page_size;
    if constexpr (kQuads) {
        const int pg = ps_shift >= 0 ? j >> ps_shift : j / ps;
        float *at = a.key_mass + ((int64_t)trow[pg] * a.hkv + kvh) * ps + (j - pg * ps), old[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) old[k] = in >> k & 1 ? at[k] : 0.f;
#pragma unroll
        for (int k = 0; k < 4; ++k)
            if (in >> k & 1) at[k] = old[k] + p[k];
    } else {
#pragma unroll
        for (int k = 0; k < 4; ++k)
            if (in >> k & 1) {
                const int pg = (j + k) / ps;
                a.key_mass[((int64_t)trow[pg] * a.hkv + kvh) * ps + (j + k - pg * ps)] += p[k];
            }
    }
}

// The keys of [lo, hi) among j .. j + 3, a bit each.
__device__ __forceinline__ int quad_mask(int j, int lo, int hi) {
    const int below = min(max(lo - j, 0), 4), past = min(max(j + 4 - hi, 0), 4);
    return (15 << below) & (15 >> past);
}

// Sequences of one item: a CTA per (item, KV head, block of keys), four consecutive
// keys per thread and step, the group's heads in turn.  The scores come from L2 when
// they fit there (4 bytes a key and head), the totals are read and written once.
// The pass is latency-bound (metadata, then scores, table and log-sum-exps, then
// the totals): the first step's scores are asked for before the log-sum-exps are
// merged.
// Four CTAs of 64 registers an SM, or three of 80 where the merge rides along: four
// histories of 32-128K keys at G = 8 take 254 us a call so and 260 at four, 64 of
// 0.5-8K at G = 4 the same 215; without the merge 18 us at four and 23 at three.
// kQuads: pages hold whole aligned fours of keys and the totals are 16-byte
// aligned.
template <bool kQuads>
__device__ __forceinline__ void add_item(const MassArgs &a, int blocks, int ps_shift, int block, float *lse) {
    const int blk = block % blocks;
    const int rest = block / blocks;
    const int kvh = rest % a.hkv, item = rest / a.hkv;
    const int G = a.hq / a.hkv, ps = a.plan.page_size;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t rows = (int64_t)a.plan.queries * a.hq;
    const int qi = a.plan.decode[item];
    // what hangs on the query alone is asked for at once: its metadata and the
    // first of this warp's log-sum-exps (over the splits, two a lane)
    const int64_t row0 = (int64_t)qi * a.hq + kvh * G;
    const bool mine = warp < G;
    float l0 = mine && lane < a.splits ? a.lse[lane * rows + row0 + warp] : -INFINITY;
    float l1 = mine && lane + 32 < a.splits ? a.lse[(lane + 32) * rows + row0 + warp] : -INFINITY;
    const int4 meta = a.plan.qmeta[qi];
    int64_t lo64, hi64;
    visible_range(meta.y, a.causal ? 0 : a.plan.seq_lens[meta.x], a.causal, a.window, lo64, hi64);
    const int lo = (int)lo64, hi = (int)hi64;       // positions fit 32 bits
    const int origin = (int)score_origin(lo);
    if (hi - origin > a.cap || hi > kMaxCountedKeys) {
        // the workspace holds no scores past cap: this item adds nothing (nor does
        // one whose steps could leave 32 bits)
        if (threadIdx.x == 0) atomicCAS(a.status, 0, PA_DEVICE_RANGE);
        return;
    }
    const int step = blocks * kItemKeys;             // at most about the longest history
    const int start = lo / step * step + blk * kItemKeys;
    if (start >= hi || (start + kItemKeys <= lo && start + step >= hi)) return;   // nothing here (uniform)
    const int32_t *trow = a.plan.table + (int64_t)meta.x * a.plan.width;
    for (int g0 = 0; g0 < G; g0 += kMaxStagedHeads) {
        const int gn = min(G - g0, kMaxStagedHeads);
        const float *head0 = a.scores + ((int64_t)item * a.hq + kvh * G + g0) * a.cap - origin;
        float4 early[kHeadsAtOnce];
        int page = 0;
        auto ask = [&](int j) {                     // the page and the first heads' scores of four keys
            if (j + 4 > lo && j < hi) {
                if (kQuads) page = trow[ps_shift >= 0 ? j >> ps_shift : j / ps];
#pragma unroll
                for (int g = 0; g < kHeadsAtOnce; ++g)
                    if (g < gn) early[g] = *reinterpret_cast<const float4 *>(head0 + j + g * a.cap);
            }
        };
        int j = start + 4 * (int)threadIdx.x;
        ask(j);
        __syncthreads();
        for (int g = warp; g < gn; g += kItemWarps) {
            if (g0 + g != warp) {
                l0 = lane < a.splits ? a.lse[lane * rows + row0 + g0 + g] : -INFINITY;
                l1 = lane + 32 < a.splits ? a.lse[(lane + 32) * rows + row0 + g0 + g] : -INFINITY;
            }
            float m = fmaxf(l0, l1);
            for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
            float t = (l0 == -INFINITY ? 0.f : exp2f((l0 - m) * kLog2e)) + (l1 == -INFINITY ? 0.f : exp2f((l1 - m) * kLog2e));
            for (int o = 16; o; o >>= 1) t += __shfl_xor_sync(0xffffffffu, t, o);
            if (lane == 0) lse[g] = a.splits == 1 ? l0 * kLog2e : m * kLog2e + log2f(t);
        }
        __syncthreads();
        for (; j < hi; j += step) {
            if (j + 4 <= lo) {
                ask(j + step);
                continue;
            }
            const float *sc = head0 + j;
            const bool all = j >= lo && j + 4 <= hi;
            float4 *m = nullptr;
            float4 old;
            if (kQuads && all) {
                m = reinterpret_cast<float4 *>(a.key_mass + ((int64_t)page * a.hkv + kvh) * ps +
                                               (ps_shift >= 0 ? j & (ps - 1) : j % ps));
                old = *m;
            }
            float p[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int g = 0; g < kHeadsAtOnce; ++g)
                if (g < gn) {
                    const float4 v = early[g];
                    const float l = lse[g];
                    p[0] += exp2f(v.x - l); p[1] += exp2f(v.y - l); p[2] += exp2f(v.z - l); p[3] += exp2f(v.w - l);
                }
            ask(j + step);
#pragma unroll 4
            for (int g = kHeadsAtOnce; g < gn; ++g) {
                const float4 v = *reinterpret_cast<const float4 *>(sc + g * a.cap);
                const float l = lse[g];
                p[0] += exp2f(v.x - l); p[1] += exp2f(v.y - l); p[2] += exp2f(v.z - l); p[3] += exp2f(v.w - l);
            }
            if (kQuads && all) {
                old.x += p[0]; old.y += p[1]; old.z += p[2]; old.w += p[3];
                *m = old;
            } else {
                add_to_part<kQuads>(a, trow, kvh, ps_shift, j, quad_mask(j, lo, hi), p);
            }
        }
    }
}

// Sequences of several items (drafted tokens, short runs): a CTA per (sequence,
// KV head, block of keys).  It finds the sequence's items among the plan's (or
// takes them from the grouped list when those are many), stages their ranges and
// log-sum-exps, eight items at a time, and adds all their weights to a key before
// it touches the key's total.  Key j always falls to block (j / kItemKeys) % blocks
// and to one thread of it, whatever an item's own range: no two CTAs meet on a key.
constexpr int kScanItems = 1024;               // more items in the plan: grouped list
constexpr int kStagedItems = 8;

struct RepeatedShared {
    int item[kScanItems], lo[kScanItems], hi[kScanItems];
    float lse[kStagedItems][kMaxStagedHeads];
    int count[kItemWarps];
};

template <bool kQuads>
__device__ __forceinline__ void add_repeated(const MassArgs &a, int grouped, int blocks, int ps_shift, int block,
                                             RepeatedShared &sh) {
    const int blk = block % blocks;
    const int rest = block / blocks;
    const int kvh = rest % a.hkv, seq = rest / a.hkv;
    const int G = a.hq / a.hkv, ps = a.plan.page_size;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int64_t rows = (int64_t)a.plan.queries * a.hq;
    const int seq_len = a.plan.seq_lens[seq];
    const int32_t *trow = a.plan.table + (int64_t)seq * a.plan.width;
    const int step = blocks * kItemKeys;
    auto stage = [&](int at, int item, int pos) {
        int64_t lo, hi;
        visible_range(pos, seq_len, a.causal, a.window, lo, hi);
        if (hi - score_origin(lo) > a.cap || hi > kMaxCountedKeys) {
            atomicCAS(a.status, 0, PA_DEVICE_RANGE);    // no scores past cap: adds nothing
            lo = hi = 0;
        }
        sh.item[at] = item;
        sh.lo[at] = (int)lo;
        sh.hi[at] = (int)hi;
    };
    const int g_first = grouped ? a.group_start[seq] : 0, g_last = grouped ? a.group_start[seq + 1] : 0;
    for (int base = g_first; grouped ? base < g_last : base == 0; base += kScanItems) {
        // this round's items, in the order of the plan's list
        int cnt = 0;
        __syncthreads();
        if (grouped) {
            cnt = min(kScanItems, g_last - base);
            for (int i = tid; i < cnt; i += kItemThreads) {
                const int item = a.group_list[base + i];
                stage(i, item, a.plan.qmeta[a.plan.decode[item]].y);
            }
        } else {
            for (int i0 = 0; i0 < a.plan.n_decode; i0 += kItemThreads) {
                const int i = i0 + tid;
                int4 meta = make_int4(-1, 0, 0, 0);
                if (i < a.plan.n_decode) meta = a.plan.qmeta[a.plan.decode[i]];
                const unsigned hit = __ballot_sync(0xffffffffu, meta.x == seq);
                if (lane == 0) sh.count[warp] = __popc(hit);
                __syncthreads();
                int at = cnt + __popc(hit & ((1u << lane) - 1u));
                for (int w = 0; w < kItemWarps; ++w) {
                    at += w < warp ? sh.count[w] : 0;
                    cnt += sh.count[w];
                }
                if (meta.x == seq) stage(at, i, meta.y);
                __syncthreads();
            }
        }
        __syncthreads();
        for (int e0 = 0; e0 < cnt; e0 += kStagedItems) {
            const int items = min(kStagedItems, cnt - e0);
            int lo_all = 0x7fffffff, hi_all = 0;
            for (int i = 0; i < items; ++i) {
                lo_all = min(lo_all, sh.lo[e0 + i]);
                hi_all = max(hi_all, sh.hi[e0 + i]);
            }
            const int start = lo_all / step * step + blk * kItemKeys;
            if (start >= hi_all || (start + kItemKeys <= lo_all && start + step >= hi_all)) continue;   // uniform
            for (int g0 = 0; g0 < G; g0 += kMaxStagedHeads) {
                const int gn = min(G - g0, kMaxStagedHeads);
                __syncthreads();
                for (int k = warp; k < items * gn; k += kItemWarps) {
                    const int i = k / gn, g = k - i * gn;
                    const int64_t row = (int64_t)a.plan.decode[sh.item[e0 + i]] * a.hq + kvh * G + g0 + g;
                    const float l0 = lane < a.splits ? a.lse[lane * rows + row] : -INFINITY;
                    const float l1 = lane + 32 < a.splits ? a.lse[(lane + 32) * rows + row] : -INFINITY;
                    float m = fmaxf(l0, l1);
                    for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
                    float t = (l0 == -INFINITY ? 0.f : exp2f((l0 - m) * kLog2e)) +
                              (l1 == -INFINITY ? 0.f : exp2f((l1 - m) * kLog2e));
                    for (int o = 16; o; o >>= 1) t += __shfl_xor_sync(0xffffffffu, t, o);
                    if (lane == 0) sh.lse[i][g] = a.splits == 1 ? l0 * kLog2e : m * kLog2e + log2f(t);
                }
                __syncthreads();
                for (int j = start + 4 * tid; j < hi_all; j += step) {
                    float p[4] = {0.f, 0.f, 0.f, 0.f};
                    int any = 0;
#pragma unroll 2
                    for (int i = 0; i < items; ++i) {
                        const int lo = sh.lo[e0 + i], hi = sh.hi[e0 + i];
                        if (j + 4 <= lo || j >= hi) continue;
                        const float *sc = a.scores + ((int64_t)sh.item[e0 + i] * a.hq + kvh * G + g0) * a.cap + (j - (int)score_origin(lo));
                        const int in = quad_mask(j, lo, hi);
                        float w[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
                        for (int g = 0; g < gn; ++g) {
                            const float4 v = *reinterpret_cast<const float4 *>(sc + g * a.cap);
                            const float l = sh.lse[i][g];
                            w[0] += exp2f(v.x - l); w[1] += exp2f(v.y - l); w[2] += exp2f(v.z - l); w[3] += exp2f(v.w - l);
                        }
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            if (in >> k & 1) p[k] += w[k];
                        any |= in;
                    }
                    if (kQuads && any == 15) {
                        const int pg = ps_shift >= 0 ? j >> ps_shift : j / ps;
                        float4 *m = reinterpret_cast<float4 *>(a.key_mass + ((int64_t)trow[pg] * a.hkv + kvh) * ps + (j - pg * ps));
                        float4 v = *m;
                        v.x += p[0]; v.y += p[1]; v.z += p[2]; v.w += p[3];
                        *m = v;
                    } else {
                        add_to_part<kQuads>(a, trow, kvh, ps_shift, j, any, p);
                    }
                }
            }
        }
    }
}

// kRepeated: some sequence has several items (units are sequences, else items).
template <bool kQuads, bool kRepeated>
__global__ void __launch_bounds__(kItemThreads, 4) mass_items_kernel(MassArgs a, int grouped, int blocks, int ps_shift) {
    griddep_wait();
    griddep_launch();
    if constexpr (kRepeated) {
        __shared__ RepeatedShared sh;
        add_repeated<kQuads>(a, grouped, blocks, ps_shift, blockIdx.x, sh);
    } else {
        __shared__ float lse[kMaxStagedHeads];
        add_item<kQuads>(a, blocks, ps_shift, blockIdx.x, lse);
    }
}

// The merge of the split outputs and the totals in one launch: both follow the
// decode kernel and neither needs the other.  The first merge_blocks CTAs merge.
template <typename T, int VEC, bool kQuads, bool kRepeated>
__global__ void __launch_bounds__(kItemThreads, 3) merge_and_items_kernel(AttnArgs attn, MassArgs a, int use_list, int nrows,
                                                                          int wide, int merge_blocks, int grouped, int blocks,
                                                                          int ps_shift) {
    griddep_wait();
    griddep_launch();
    extern __shared__ float part[];
    if ((int)blockIdx.x < merge_blocks) {
        if (wide)
            merge_row_wide<T, VEC>(attn, use_list, blockIdx.x, part);
        else
            merge_rows<T, VEC>(attn, use_list, nrows, blockIdx.x);
        return;
    }
    const int block = (int)blockIdx.x - merge_blocks;
    if constexpr (kRepeated) {
        __shared__ RepeatedShared sh;
        add_repeated<kQuads>(a, grouped, blocks, ps_shift, block, sh);
    } else {
        __shared__ float lse[kMaxStagedHeads];
        add_item<kQuads>(a, blocks, ps_shift, block, lse);
    }
}

// ------------------------------------------------------- recomputed scores --
constexpr int kReThreads = 256, kReKeys = 32, kReRows = kReThreads / kReKeys;

// One CTA per (sequence, KV head, block of 32 keys): the keys stay in shared
// memory (fp32), the sequence's queries stream past, eight (query, head) rows at
// a time, one dot product per thread.
template <typename T>
__global__ void __launch_bounds__(kReThreads) mass_recompute_kernel(MassArgs a, int blocks) {
    griddep_wait();
    griddep_launch();
    extern __shared__ float sm[];
    const int stride = a.d | 1;                        // odd: the 32 keys of a warp hit 32 banks
    float *keys = sm;                                   // [32][stride]
    float *rows = keys + kReKeys * stride;              // [8][d]
    __shared__ float part[kReRows][kReKeys];
    const int blk = blockIdx.x % blocks;
    const int rest = blockIdx.x / blocks;
    const int kvh = rest % a.hkv, s = rest / a.hkv;
    const int G = a.hq / a.hkv, ps = a.plan.page_size;
    const int first = a.group_start[s], last = a.group_start[s + 1];
    if (first == last) return;
    const int n = a.plan.seq_lens[s];
    if (n > kMaxCountedKeys) {                          // (only a device copy's length: the host refuses it)
        if (threadIdx.x == 0) atomicCAS(a.status, 0, PA_DEVICE_RANGE);
        return;
    }
    const int32_t *trow = a.plan.table + (int64_t)s * a.plan.width;
    const T *kc = static_cast<const T *>(a.k), *qc = static_cast<const T *>(a.q);
    const int key = threadIdx.x % kReKeys, slot = threadIdx.x / kReKeys;
    for (int j0 = blk * kReKeys; j0 < n; j0 += blocks * kReKeys) {
        __syncthreads();
        for (int i = threadIdx.x; i < kReKeys * a.d; i += kReThreads) {
            const int t = i / a.d, e = i - t * a.d, j = j0 + t;
            keys[t * stride + e] =
                j < n ? to_f<T>(kc[(((int64_t)trow[j / ps] * ps + j % ps) * a.hkv + kvh) * a.d + e]) : 0.f;
        }
        float sum = 0.f;
        for (int e = first; e < last; ++e) {
            const int q0 = a.group_list[e], nrows = G;
            for (int r0 = 0; r0 < nrows; r0 += kReRows) {
                // any row of these eight that sees a key of the block?
                const int r = r0 + slot;
                const bool live = r < nrows;
                const int qi = q0 + (live ? r : r0) / G, h = kvh * G + (live ? r : r0) % G;
                int64_t lo, hi;
                visible_range(a.plan.qmeta[qi].y, n, a.causal, a.window, lo, hi);
                const bool sees = live && lo < j0 + kReKeys && hi > j0;
                if (!__syncthreads_or(sees)) continue;
                for (int i = threadIdx.x; i < kReRows * a.d; i += kReThreads) {
                    const int t = i / a.d, c = i - t * a.d, rr = r0 + t;
                    rows[i] = rr < nrows
                                  ? to_f<T>(qc[((int64_t)(q0 + rr / G) * a.hq + kvh * G + rr % G) * a.d + c]) *
                                        (a.scale * kLog2e)
                                  : 0.f;
                }
                __syncthreads();
                const int64_t j = j0 + key;
                if (sees && j >= lo && j < hi) {
                    float dot = 0.f;
                    for (int c = 0; c < a.d; ++c) dot = fmaf(rows[slot * a.d + c], keys[key * stride + c], dot);
                    sum += exp2f(dot - a.lse_final[(int64_t)qi * a.hq + h] * kLog2e);
                }
            }
        }
        __syncthreads();
        part[slot][key] = sum;
        __syncthreads();
        if (slot == 0 && j0 + key < n) {
            float t = 0.f;
            for (int w = 0; w < kReRows; ++w) t += part[w][key];
            const int64_t page = trow[(j0 + key) / ps];
            a.key_mass[(page * a.hkv + kvh) * ps + (j0 + key) % ps] += t;
        }
    }
}

int blocks_for(int64_t units, int64_t want) {
    const int64_t most = INT32_MAX / (units > 0 ? units : 1);
    const int64_t b = want < most ? want : most;
    return (int)(b < 1 ? 1 : b);
}

template <typename T> cudaError_t launch_re(const MassArgs &a, cudaStream_t st) {
    const size_t smem = (size_t)(kReKeys * (a.d | 1) + kReRows * a.d) * sizeof(float);
    cudaError_t e = cudaFuncSetAttribute(mass_recompute_kernel<T>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    const int64_t units = (int64_t)a.plan.sequences * a.hkv;
    const int blocks = blocks_for(units, ((int64_t)a.longest + kReKeys - 1) / kReKeys);
    return launch_pdl(mass_recompute_kernel<T>, dim3((unsigned)(units * blocks)), dim3(kReThreads), smem, st, a, blocks);
}

}  // namespace

cudaError_t launch_mass_index(const MassArgs &a, MassRecords kind, cudaStream_t st) {
    const int n = kind == kMassItems ? a.plan.n_decode : (kind == kMassTiles ? a.plan.n_tiles : a.plan.queries);
    return launch_pdl(mass_index_kernel, dim3(1), dim3(kIndexThreads), 0, st, a, (int)kind, n);
}

cudaError_t launch_mass_tiles_prepare(const MassArgs &a, cudaStream_t st) {
    return launch_pdl(mass_tiles_prepare_kernel, dim3((unsigned)(1 + a.plan.n_tiles)), dim3(kIndexThreads), 0, st, a);
}

cudaError_t launch_lse_final(const MassArgs &a, float *out, cudaStream_t st) {
    const int64_t rows = (int64_t)a.plan.queries * a.hq;
    return launch_pdl(lse_final_kernel, dim3((unsigned)((rows + 255) / 256)), dim3(256), 0, st, a, out);
}

bool mass_items_grouped(const MassArgs &a, bool repeated) { return repeated && a.plan.n_decode > kScanItems; }

cudaError_t launch_mass_items(const MassArgs &a, bool repeated, const AttnArgs *merge, bool use_list, cudaStream_t st) {
    const int64_t units = (int64_t)(repeated ? a.plan.sequences : a.plan.n_decode) * a.hkv;
    // blocks a unit: one per 1024 keys of the longest history, or of what a window can
    // touch, but no more than fill the GPU once (a CTA's start costs three dependent
    // loads, its further keys one)
    int64_t keys = a.longest;
    if (a.causal && a.window > 0 && (int64_t)a.window + kItemKeys < keys) keys = (int64_t)a.window + kItemKeys;
    const int64_t most = (keys + kItemKeys - 1) / kItemKeys, fill = (152 * 4 + units - 1) / units;
    const int blocks = blocks_for(units, most < fill ? most : fill);
    const int ps = a.plan.page_size;
    int shift = -1;
    if ((ps & (ps - 1)) == 0)
        for (shift = 0; (1 << shift) < ps; ++shift) {}
    const bool quads = ps % 4 == 0 && reinterpret_cast<uintptr_t>(a.key_mass) % 16 == 0;
    const dim3 block(kItemThreads);
    const int grouped = mass_items_grouped(a, repeated) ? 1 : 0;
    cudaError_t e;
    if (!merge) {
        const dim3 grid((unsigned)(units * blocks));
        auto launch = [&](auto kernel) { return launch_pdl(kernel, grid, block, 0, st, a, grouped, blocks, shift); };
        if (repeated)
            e = quads ? launch(mass_items_kernel<true, true>) : launch(mass_items_kernel<false, true>);
        else
            e = quads ? launch(mass_items_kernel<true, false>) : launch(mass_items_kernel<false, false>);
    } else {
        const int nrows = (use_list ? a.plan.n_decode : a.plan.queries) * a.hq;
        const bool wide = merge_is_wide(*merge, nrows);
        const int64_t mb = wide ? nrows : (nrows + 7) / 8;
        if (mb + units * blocks > INT32_MAX) return cudaErrorInvalidValue;
        const dim3 grid((unsigned)(mb + units * blocks));
        const size_t smem = wide ? (size_t)8 * merge->dv * sizeof(float) : 0;
        auto launch = [&](auto kernel) {
            return launch_pdl(kernel, grid, block, smem, st, *merge, a, use_list ? 1 : 0, nrows, wide ? 1 : 0, (int)mb,
                              grouped, blocks, shift);
        };
        auto by_kind = [&](auto t, auto vec) {
            using T = decltype(t);
            constexpr int VEC = decltype(vec)::value;
            if (repeated)
                return quads ? launch(merge_and_items_kernel<T, VEC, true, true>)
                             : launch(merge_and_items_kernel<T, VEC, false, true>);
            return quads ? launch(merge_and_items_kernel<T, VEC, true, false>)
                         : launch(merge_and_items_kernel<T, VEC, false, false>);
        };
        auto by_vec = [&](auto t) {
            const int vec = merge_vec(*merge);
            return vec == 4   ? by_kind(t, std::integral_constant<int, 4>())
                   : vec == 2 ? by_kind(t, std::integral_constant<int, 2>())
                              : by_kind(t, std::integral_constant<int, 1>());
        };
        e = a.dtype == PA_F32 ? by_vec(float()) : (a.dtype == PA_F16 ? by_vec(__half()) : by_vec(__nv_bfloat16()));
    }
    if (e != cudaSuccess) return e;
    return cudaGetLastError();
}

cudaError_t launch_mass_recompute(const MassArgs &a, cudaStream_t st) {
    cudaError_t e;
    switch (a.dtype) {
        case PA_F32: e = launch_re<float>(a, st); break;
        case PA_F16: e = launch_re<__half>(a, st); break;
        default: e = launch_re<__nv_bfloat16>(a, st); break;
    }
    if (e != cudaSuccess) return e;
    return cudaGetLastError();
}

}  // namespace pa
