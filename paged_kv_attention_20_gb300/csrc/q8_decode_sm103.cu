// Attention over the 8-bit cache on tcgen05 tensor cores, for decode items with 16-bit
// queries and heads of 128 or 64.
//
// Halving the bytes of a key doubles the multiply-adds per byte, and CUDA cores, which
// keep up with a 16-bit cache for groups of up to four query heads, no longer do.  The
// e4m3 rows go to the tensor core as they are (kind::f8f6f4), keys as MMA rows:
//   S^T = K . Q^T   (M = 128 keys, N = query columns, K = 128 dims)
//   O^T += V^T . P  (M = 128 dims, N = weight columns, K = 128 keys; V is MN-major)
// so that N, not M, is padded to the few query heads, each of 128 threads owns one key of
// a tile, and the accumulators are a few columns wide.
//
// The other operands are 16-bit or fp32 numbers and become sums of short floats, one
// column each; products with e4m3 are exact and sums are fp32:
//   Q: a row times a power of two, as e4m3 pieces q1 + q2/16 (+ q3/256): exact for bf16
//      with two and for fp16 with three, but for elements 2^-17 (2^-21) below the row's
//      largest, which are off by 2^-23 (2^-27) of that.
//   P: weights 2^(u_j - R + 7) as e5m2 pieces p1 + p2/8 + p3/128, 2^-10 of a weight.
//      e5m2, whose numbers span 2^32, and not e4m3: a long tail of weights 2^-20 of the
//      largest must not vanish, and here one is lost only below 2^-31 of it.
// Two heads of 64 lie side by side in a slot and are taken as one of 128: a query row is
// zero over the other head's dims, and of an O^T column only its own head's 64 lanes count
// (behind an odd last head the box reads zeros, past the slot's end).
// Queries of one sequence at consecutive positions (drafted tokens) share a unit as far as
// its columns go, and with it their keys; each column masks its own range.
// A key's scale multiplies its score.  A value's cannot be applied after the sum over
// keys, so it goes into the weight: u_j = s_j + log2(scale of V_j), whose reference
// maximum R is kept apart from the scores' r; the row sum takes 2^(s_j - r).
//
// The kernel is bound by HBM: a 128-key tile is 32 KB, six are in flight.  It is
// persistent, one CTA per SM walking (item, split, KV head, chunk of up to 16 heads) units
// in serpentine rounds.  Two groups of four softmax warps (thread = key of a tile, then
// dim of the output) take units in turn, each with its own query, S^T, P and O^T buffers,
// so that a unit's start (queries, first references) and end (row sums, output), 2.7 us of
// latencies, pass beside the other group's tiles.  Units of more than eight columns are bound
// by the softmax (3000 cycles a tile with a group alone) and have both groups, eight columns
// each (the decode layer with groups of 16 in two splits: 143 us, 158 with a group a unit).
// Warp 8 loads tiles by TMA and works out the units, warp 11 fetches scales, warps 9 and 10
// issue S^T and O^T.
// References move only when a score passes them by a few binades, which all 128 threads
// learn from one barrier a tile; O^T is rescaled then.  Every wait is bounded: a role that
// waited in vain records it and goes on without waiting, so that a group's warps meet at
// every barrier, and they leave together at the end of the unit.

#include <cuda.h>

#include "per_device.h"
#include "q8_format.cuh"
#include "sm103_tc.cuh"
#include "tma_host.h"

namespace pa {
namespace {

using namespace tc;
using namespace q8;

constexpr int kN = 128;                  // keys per tile
constexpr int kD = 128;                  // head dim = value dim
constexpr int kTile = kN * kD;           // bytes of a tile of K or V
constexpr int kBuf = 3;                  // S^T buffers of a group, in TMEM
constexpr int kPBuf = 2;                 // P buffers of a group, in shared memory
constexpr int kUnits = 8;                // units whose parameters are on hand
constexpr int kThreads = 384;
constexpr int kListed = 8192;            // items among which the first queries of units are counted
constexpr uint32_t kTmemCols = 512;      // S^T of the groups at 0 and 192, 64 columns each; O^T at 384, 448
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kTop = 7.f;              // a fresh reference puts its weight at 2^7 ...
constexpr float kSlack = 8.f;            // ... and weights up to 2^15 leave it (e5m2 ends at 1.75 * 2^15)
constexpr float kSumSlack = 32.f;

constexpr int round16(int n) { return (n + 15) / 16 * 16; }

struct Unit {
    int qi, nq, pos;                    // first query, queries (0: another unit has them), its position
    int kvh, g0, heads;                 // KV head (of 128 dims), first query head of a group, heads
    int split, seq_len, n_kt, j0, j1, jb;
    int first;                          // the CTA's tiles before it
    const int32_t *trow;
};

// What column g of a unit holds: query k, head `real` of a pair, head h of its group.
struct Column {
    int k, real, h;
};

// Up to eight columns a softmax thread; a unit of sixteen has both groups, eight columns each,
// where smaller ones have a group each.
template <int GH, int QP, int RH> struct Shared {
    static constexpr bool kJoin = GH > 8;
    static constexpr int GC = kJoin ? 8 : GH, SETS = kJoin ? 1 : 2;
    static constexpr int NS = round16(QP * GH), NP = round16(3 * GH);
    static constexpr int kStages = 6;
    uint8_t kv[kStages][2 * kTile];                  // 128-byte swizzle; eights of rows (TcParams)
    uint8_t q[SETS][NS * 128];                       // of the group's unit: its GC columns' first pieces, second, ..; then the other group's
    uint8_t p[SETS][kPBuf][NP * 128];                // the same, 128 keys each
    uint8_t scale[kStages][2 * RH][kN];              // scale bytes of the tile's keys and values
    uint64_t kv_full[kStages], kv_empty[kStages], scale_full[kStages];
    uint64_t s_full[SETS][kBuf], s_read[SETS][kBuf], p_ready[SETS][kPBuf], o_done[SETS][kPBuf];
    uint64_t q_ready[SETS], o_free[SETS];
    uint64_t up_full[kUnits], up_empty[kUnits];
    Unit unit[kUnits];
    float red[2][4][GC][2];                          // a group's warps: maxima of a tile
    float sum[2][4][GC];                             // and row sums of a unit (a warp may be here while another still reads red)
    struct Out {
        int64_t at;                                  // row of a column's output, -1: none
        float inv, up;                               // what its sum is multiplied by, one after the other
        int real;
        uint32_t nan[4];
    } out[2][GC];
    uint32_t nan[2][GC][4];                          // dims of the tile whose value is NaN for the column (units of several queries)
    // per column: reference of the weights with the values' scales, of the scores, and the
    // scale of the query row (with the softmax scale, log2); factors of a change of reference;
    // the keys it sees, where they differ between columns
    float4 ref[2][GC];
    float2 change[2][GC];
    int2 range[2][GC];
    Column column[GH];
    uint32_t first[kListed / 32];                    // bit of an item: a unit's first query
    uint16_t before[kListed / 32];                   // such items before a word's
    int firsts;
    uint32_t tmem_base;
};

__device__ __forceinline__ void mma_f8_ss(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
        " tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n}\n" ::"r"(d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}

// Instruction descriptor of kind::f8f6f4 with fp32 accumulation: A e4m3, B e4m3 or e5m2 (K-major).
__host__ __device__ constexpr uint32_t idesc_f8(int M, int N, bool b_e5m2, bool a_mn) {
    return (1u << 4) | ((b_e5m2 ? 1u : 0u) << 10) | ((a_mn ? 1u : 0u) << 15) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}

__device__ __forceinline__ void tmem_ld8(uint32_t taddr, uint32_t *r) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];\n"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                 : "r"(taddr));
}
__device__ __forceinline__ void tmem_st8(uint32_t taddr, const uint32_t *r) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};\n" ::"r"(taddr), "r"(r[0]), "r"(r[1]),
                 "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
                 : "memory");
}

// N columns from `at` on, a multiple of eight.
template <int N> __device__ __forceinline__ void tmem_load(uint32_t at, uint32_t (&r)[N]);
template <> __device__ __forceinline__ void tmem_load<8>(uint32_t at, uint32_t (&r)[8]) { tmem_ld8(at, r); }
template <> __device__ __forceinline__ void tmem_load<16>(uint32_t at, uint32_t (&r)[16]) { tmem_ld16(at, r); }
template <> __device__ __forceinline__ void tmem_load<24>(uint32_t at, uint32_t (&r)[24]) {
#pragma unroll
    for (int c = 0; c < 24; c += 8) tmem_ld8(at + c, r + c);
}

// Barriers of one group's 128 threads.  They want whole warps: lanes that a branch before has
// parted meet first.
__device__ __forceinline__ void group_bar(int group) {
    __syncwarp();
    asm volatile("bar.sync %0, 128;\n" ::"r"(group + 1) : "memory");
}
__device__ __forceinline__ bool group_any(int group, bool pred) {
    uint32_t r;
    __syncwarp();
    asm volatile("{\n .reg .pred p, q;\n setp.ne.u32 p, %1, 0;\n bar.red.or.pred q, %2, 128, p;\n selp.u32 %0, 1, 0, q;\n}\n"
                 : "=r"(r)
                 : "r"((uint32_t)pred), "r"(group + 1)
                 : "memory");
    return r != 0;
}

__device__ __forceinline__ void cp_async16(void *dst, const void *src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;\n" ::"r"(smem_u32(dst)), "l"(src) : "memory");
}
// Arrives on `bar` once this thread's copies so far have landed.
__device__ __forceinline__ void cp_async_arrive(uint64_t *bar) {
    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];\n" ::"r"(smem_u32(bar)) : "memory");
}
__device__ __forceinline__ void cp_async_wait_all() { asm volatile("cp.async.wait_all;\n" ::: "memory"); }

// fp32 maximum over a warp by the integer reduction; NaN counts as the largest.
__device__ __forceinline__ float warp_max(float x) {
    int i = __float_as_int(x);
    i = __reduce_max_sync(0xffffffffu, i ^ ((i >> 31) & 0x7fffffff));
    return __int_as_float(i ^ ((i >> 31) & 0x7fffffff));
}

template <typename T> __device__ __forceinline__ T rounded(float x);
template <> __device__ __forceinline__ __half rounded<__half>(float x) { return __float2half_rn(x); }
template <> __device__ __forceinline__ __nv_bfloat16 rounded<__nv_bfloat16>(float x) { return __float2bfloat16_rn(x); }

// Two weights to two e5m2 bytes and back.
__device__ __forceinline__ uint32_t to_e5m2(float x, float y) {
    return __nv_cvt_float2_to_fp8x2(make_float2(x, y), __NV_SATFINITE, __NV_E5M2);
}
__device__ __forceinline__ float2 from_e5m2(uint32_t two) {
    const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)two, __NV_E5M2);
    return __half22float2(*reinterpret_cast<const __half2 *>(&h));
}

// Bit 7 of every e4m3 byte that is NaN.
__device__ __forceinline__ uint32_t nan_bytes(uint32_t four) { return ((four & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u; }

struct TcParams {
    int group, chunks;     // query heads per KV head, chunks of `per` of them
    int per, rq;           // heads of a KV head and queries of a unit
    int ps_shift, box_rows;
    // Where a tile's K and V start, and from eight rows to the next: eights of K and V in turn
    // where one box loads both, else V behind K.
    uint32_t k_at, v_at, eight;
    int together;
    float scale_log2;
};

template <typename T, int GH, int QP, int RH>
__global__ void __launch_bounds__(kThreads, 1)
    q8_decode_tc_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v, Q8AttnArgs q8a,
                        int use_list, TcParams tp) {
    using S = Shared<GH, QP, RH>;
    constexpr int D = kD / RH;
    constexpr int NS = S::NS, NP = S::NP, kStages = S::kStages, GC = S::GC;
    constexpr bool kJoin = S::kJoin;
    constexpr int kWarps = kJoin ? 8 : 4;              // softmax warps of a unit
    griddep_wait();
    const AttnArgs &a = q8a.a;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    if ((smem_u32(smem_raw) & 1023u) != 0u) {
        if (threadIdx.x == 0) atomicCAS(a.status, 0, PA_DEVICE_LAYOUT);
        return;
    }
    S &s = *reinterpret_cast<S *>(smem_raw);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int ps = a.plan.page_size;
    const int items = use_list ? a.plan.n_decode : a.plan.queries;
    const int hv = (a.hkv + RH - 1) / RH;      // heads of 128 dims (the last pair may lack its second)
    // How many of the queries after q (way 1) or before it (way -1), up to `most`, carry on the
    // run of consecutive positions of its sequence; four loads are in flight at a time.
    auto carries_on = [&](int q, int4 meta, int way, int most) -> int {
        int n = 0;
        while (n < most) {
            int4 m[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const int at = q + way * (n + k + 1);
                m[k] = at >= 0 && at < a.plan.queries ? a.plan.qmeta[at] : make_int4(-1, 0, 0, 0);
            }
            int k = 0;
            while (k < 4 && m[k].x == meta.x && m[k].y == meta.y + way * (n + k + 1)) ++k;
            n += k;
            if (k < 4) break;
        }
        return n < most ? n : most;
    };
    // A run of consecutive positions is cut every rq queries from its start on, at its seventeenth,
    // and from there where the position is a multiple of rq: no piece is longer than rq, and every
    // query of a run, looking back no further, finds the same cuts.  `at`: queries of the run
    // before this one (17: as many or more).
    auto cut = [&](int at, int4 meta, int k) -> bool {
        const int i = at + k;
        return i == 16 || (i < 16 ? i : meta.y + k) % tp.rq == 0;
    };
    auto query_of = [&](int item) -> int { return use_list ? a.plan.decode[item] : item; };
    // Where runs share units, every CTA counts the first queries of units before it starts (2 us):
    // units without a query, three of four with runs of four, cost each CTA a step and leave some
    // CTAs more work than others (four tokens a sequence over the decode layer's histories: 129 us,
    // 184 with such units).  Beyond kListed items they stay in.
    const bool listed = tp.rq > 1 && items <= kListed;
    if (listed) {
        const int words = (items + 31) / 32;
        for (int w = warp; w < words; w += kThreads / 32) {
            const int item = w * 32 + lane;
            bool is_first = false;
            if (item < items) {
                const int q = query_of(item);
                const int4 meta = a.plan.qmeta[q];
                is_first = cut(carries_on(q, meta, -1, 17), meta, 0);
            }
            __syncwarp();
            const uint32_t bits = __ballot_sync(0xffffffffu, is_first);
            if (lane == 0) s.first[w] = bits;
        }
        __syncthreads();
        if (warp == 0) {
            int before = 0;
            for (int w0 = 0; w0 < words; w0 += 32) {
                const int n = w0 + lane < words ? __popc(s.first[w0 + lane]) : 0;
                int sum = n;
                for (int o = 1; o < 32; o <<= 1) {
                    const int y = __shfl_up_sync(0xffffffffu, sum, o);
                    if (lane >= o) sum += y;
                }
                if (w0 + lane < words) s.before[w0 + lane] = (uint16_t)(before + sum - n);
                before += __shfl_sync(0xffffffffu, sum, 31);
            }
            if (lane == 0) s.firsts = before;
        }
        __syncthreads();
    }
    const int units = (listed ? s.firsts : items) * a.splits * hv * tp.chunks;
    // the item of the n-th first query
    auto first_item = [&](int n) -> int {
        int lo = 0, hi = (items + 31) / 32;              // before[lo] <= n < before[hi]
        while (hi - lo > 1) {
            const int mid = (lo + hi) / 2;
            if (s.before[mid] <= n) lo = mid; else hi = mid;
        }
        uint32_t bits = s.first[lo];
        for (int k = n - s.before[lo]; k > 0; --k) bits &= bits - 1;
        return lo * 32 + __ffs(bits) - 1;
    };
    auto unit_at = [&](int u) -> Unit {
        Unit x;
        x.first = 0;
        x.g0 = u % tp.chunks * tp.per;
        int rest = u / tp.chunks;
        x.kvh = rest % hv;
        rest /= hv;
        x.split = rest % a.splits;
        x.heads = tp.group - x.g0 < tp.per ? tp.group - x.g0 : tp.per;
        x.qi = query_of(listed ? first_item(rest / a.splits) : rest / a.splits);
        const int4 meta = a.plan.qmeta[x.qi];
        x.nq = 1;
        x.pos = meta.y;
        if (tp.rq > 1) {
            const int at = carries_on(x.qi, meta, -1, 17);
            if (cut(at, meta, 0)) {
                const int after = carries_on(x.qi, meta, 1, tp.rq - 1);
                while (x.nq <= after && !cut(at, meta, x.nq)) ++x.nq;
            } else {
                x.nq = 0;
            }
        }
        x.seq_len = a.plan.seq_lens[meta.x];
        int64_t lo, hi, last, j0, j1;
        visible_range(meta.y, x.seq_len, a.causal, a.window, lo, hi);
        if (x.nq > 1) visible_range(meta.y + x.nq - 1, x.seq_len, a.causal, a.window, last, hi);
        split_bounds(lo, hi, a.splits, x.split, ps, j0, j1);
        if (x.nq == 0) j1 = j0;
        x.j0 = (int)j0;
        x.j1 = (int)j1;
        // tiles start where a TMA box does (no box crosses a page)
        x.jb = x.j0 < x.j1 ? x.j0 / tp.box_rows * tp.box_rows : x.j0;
        x.n_kt = (x.j1 - x.jb + kN - 1) / kN;
        x.trow = a.plan.table + (int64_t)meta.x * a.plan.width;
        return x;
    };
    // the CTA's i-th unit: rounds in serpentine order, so that units sorted by size even out
    auto unit_of = [&](int i) -> int {
        const int64_t g = gridDim.x, b = blockIdx.x;
        const int64_t u = i * g + ((i & 1) ? g - 1 - b : b);
        return u < units ? (int)u : units;
    };

    if (tid == 0) {
        for (int i = 0; i < kStages; ++i) {
            mbar_init(&s.kv_full[i], 1);
            mbar_init(&s.kv_empty[i], 1);
            mbar_init(&s.scale_full[i], 32);
        }
        for (int i = 0; i < S::SETS; ++i) {
            for (int b = 0; b < kBuf; ++b) {
                mbar_init(&s.s_full[i][b], 1);
                mbar_init(&s.s_read[i][b], kWarps);
            }
            for (int b = 0; b < kPBuf; ++b) {
                mbar_init(&s.p_ready[i][b], kWarps);
                mbar_init(&s.o_done[i][b], 1);
            }
            mbar_init(&s.q_ready[i], kWarps);
            mbar_init(&s.o_free[i], kWarps);
        }
        for (int i = 0; i < kUnits; ++i) {
            mbar_init(&s.up_full[i], 1);
            mbar_init(&s.up_empty[i], 3 + kWarps);   // two issuers, the scales' warp, the softmax warps
        }
        fence_mbar_init();
    }
    if (tid < GH) {
        const int columns = RH * tp.per, k = tid / columns, rest = tid - k * columns;
        s.column[tid] = k < tp.rq ? Column{k, rest / tp.per, rest % tp.per} : Column{GH, 0, 0};   // GH: no query
    }
    // the first units, one a lane, while the rest is set up: a chain of dependent loads
    Unit mine{};
    if (warp == 8 && unit_of(lane) < units) mine = unit_at(unit_of(lane));
    __syncwarp();
    if (warp == 0) {
        tmem_alloc(&s.tmem_base, kTmemCols);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = s.tmem_base;
    auto tmem_s = [tmem](int set, int b) -> uint32_t { return tmem + 192u * (uint32_t)set + 64u * (uint32_t)b; };
    auto tmem_o = [tmem](int set) -> uint32_t { return tmem + 384u + 64u * (uint32_t)set; };

    if (warp == 8 || warp == 11) {
        // ------------------------------------------------------ producers --
        // Warp 8 loads the tiles, warp 11 the scales.  A lane loads a page's rows, of K and V with
        // one box where it can (lanes 0-7), else of K or V (8-15); the page of the next tile, the
        // next unit's first among them, is looked up before the wait.  Warp 8 works units out, one
        // a lane and 32 at a time (a chain of dependent loads), and publishes unit i + 1 before it
        // loads unit i.
        const bool tiles = warp == 8;
        const int step = tiles ? tp.box_rows : 16;    // keys a lane looks the page up for
        const int oob = a.plan.pages * (ps >> 3);     // past the cache: zeros (in eights of rows)
        const CUtensorMap *map = lane < 8 ? &tm_k : &tm_v;
        if (tiles && (lane == 0 || lane == 8)) tma_prefetch_desc(map);
        int gt = 0;
        bool ok = true;
        auto unit = [&](int i, int first) -> Unit {
            const int slot = i % kUnits;
            if (tiles) {
                if (i > 0 && i % 32 == 0 && unit_of(i + lane) < units) mine = unit_at(unit_of(i + lane));
                if (lane == i % 32) {
                    if (i >= kUnits) ok = mbar_wait(&s.up_empty[slot], ((i / kUnits) - 1) & 1);
                    if (ok) {
                        mine.first = first;
                        s.unit[slot] = mine;
                        mbar_arrive(&s.up_full[slot]);
                    }
                }
                ok = __all_sync(0xffffffffu, ok);
                __syncwarp();
                return s.unit[slot];                  // (its slot is written again by this warp alone)
            }
            ok = __all_sync(0xffffffffu, mbar_wait(&s.up_full[slot], (i / kUnits) & 1));
            const Unit x = s.unit[slot];
            __syncwarp();
            if (lane == 0) mbar_arrive(&s.up_empty[slot]);
            return x;
        };
        // Page of piece lane % 8 of a tile (`step` keys), -1 past the unit's keys.
        auto page_of = [&](const Unit &x, int kt) -> int {
            const int lp = (x.jb + kt * kN + (lane & 7) * step) >> tp.ps_shift;
            return lane < (tiles ? 16 : 16 * RH) && (lane & 7) * step < kN && lp <= (x.j1 - 1) >> tp.ps_shift ? x.trow[lp] : -1;
        };
        Unit x{}, nx{};
        int next = -1;
        if (unit_of(0) < units) {
            x = unit(0, 0);
            if (ok && x.n_kt > 0) next = page_of(x, 0);
        }
        for (int i = 0; ok && unit_of(i) < units; ++i, x = nx) {
            nx.n_kt = 0;
            if (unit_of(i + 1) < units) nx = unit(i + 1, gt + x.n_kt);
            for (int kt = 0; ok && kt < x.n_kt; ++kt, ++gt) {
                const int j = x.jb + kt * kN + (lane & 7) * step, page = next, st = gt % kStages;
                const bool last = kt + 1 == x.n_kt;
                if (!last || nx.n_kt > 0) next = page_of(last ? nx : x, last ? 0 : kt + 1);
                if (gt >= kStages) ok = __all_sync(0xffffffffu, mbar_wait(&s.kv_empty[st], ((gt / kStages) - 1) & 1));
                if (!ok) break;
                if (tiles) {
                    if (lane == 0) mbar_arrive_expect_tx(&s.kv_full[st], 2 * kTile);
                    __syncwarp();
                    if ((lane & 7) * step < kN && lane < (tp.together ? 8 : 16))
                        tma_load_4d(s.kv[st] + (lane >> 3) * tp.v_at + ((lane & 7) * step >> 3) * tp.eight, map, x.kvh * kD, 0, 0,
                                    page < 0 ? oob : page * (ps >> 3) + ((j & (ps - 1)) >> 3), &s.kv_full[st]);
                } else {
                    // Eight lanes a head and tensor, keys' first.  By cp.async: loads of the softmax
                    // threads' own would be waited for at their fence before every P (159 us for the
                    // decode layer, 110 without them).  Keys past the unit's pages are masked,
                    // whatever their bytes.
                    const int h = x.kvh * RH + (lane >> 3) % RH;
                    if (page >= 0 && (RH == 1 || h < a.hkv))
                        cp_async16(&s.scale[st][lane >> 3][(lane & 7) * 16],
                                   ((lane >> 3) < RH ? q8a.k_scale : q8a.v_scale) + ((int64_t)page * a.hkv + h) * ps + (j & (ps - 1)));
                    cp_async_arrive(&s.scale_full[st]);
                }
            }
            // (after an empty unit the next one's first pages are looked up here)
            if (ok && x.n_kt == 0 && nx.n_kt > 0) next = page_of(nx, 0);
        }
        if (!ok && lane == 0) atomicCAS(a.status, 0, PA_DEVICE_TIMEOUT_TMA);
        // no load may still be landing when the CTA leaves
        cp_async_wait_all();
        if (tiles)
            for (int t = gt > kStages ? gt - kStages : 0; t < gt; ++t) mbar_wait(&s.kv_full[t % kStages], (t / kStages) & 1, 2000000ll);
    } else if (warp == 9 || warp == 10) {
        // -------------------------------------------------------- issuers --
        if (lane == 0) {
            bool ok = true;
            int gt = 0;
            const bool scores = warp == 9;
            int done[2] = {0, 0}, begun[2] = {0, 0};   // tiles and units (that have some) of each set of buffers
            constexpr uint32_t idesc_s = idesc_f8(kN, NS, false, false), idesc_o = idesc_f8(kD, NP, true, true);
            for (int i = 0; ok && unit_of(i) < units; ++i) {
                if (!mbar_wait(&s.up_full[i % kUnits], (i / kUnits) & 1)) { ok = false; break; }
                const int n_kt = s.unit[i % kUnits].n_kt;
                mbar_arrive(&s.up_empty[i % kUnits]);
                // Empty units take no part in these barriers: a group could finish two of them
                // before an issuer has looked once.
                if (n_kt == 0) continue;
                const int set = kJoin ? 0 : i & 1, n = begun[set]++;
                if (scores) {
                    if (!mbar_wait(&s.q_ready[set], n & 1)) { ok = false; break; }
                } else if (n > 0 && !mbar_wait(&s.o_free[set], (n - 1) & 1)) {
                    ok = false;
                    break;
                }
                for (int kt = 0; kt < n_kt; ++kt, ++gt, ++done[set]) {
                    const int t = done[set], st = gt % kStages;
                    if (!mbar_wait(&s.kv_full[st], (gt / kStages) & 1)) { ok = false; break; }
                    if (scores) {
                        // the buffer's last tile has been read by the softmax
                        const int b = t % kBuf;
                        if (t >= kBuf && !mbar_wait(&s.s_read[set][b], ((t / kBuf) - 1) & 1)) { ok = false; break; }
                        tc_fence_after();
                        const uint64_t kd = smem_desc(smem_u32(s.kv[st]) + tp.k_at, 16, tp.eight, kLayoutSwizzle128B);
                        const uint64_t qd = smem_desc(smem_u32(s.q[set]), 16, 1024, kLayoutSwizzle128B);
#pragma unroll
                        for (int ks = 0; ks < kD / 32; ++ks)
                            mma_f8_ss(tmem_s(set, b), kd + 2 * ks, qd + 2 * ks, idesc_s, ks > 0 ? 1u : 0u);
                        mma_commit(&s.s_full[set][b]);
                    } else {
                        const int b = t % kPBuf;
                        if (!mbar_wait(&s.p_ready[set][b], (t / kPBuf) & 1)) { ok = false; break; }
                        tc_fence_after();
                        // 32 keys are four eights of V, and 32 bytes of every row of P
                        const uint64_t vd = smem_desc(smem_u32(s.kv[st]) + tp.v_at, 16, tp.eight, kLayoutSwizzle128B);
                        const uint64_t four = tp.eight * 4 >> 4;
                        const uint64_t pd = smem_desc(smem_u32(s.p[set][b]), 16, 1024, kLayoutSwizzle128B);
#pragma unroll
                        for (int ks = 0; ks < kN / 32; ++ks)
                            mma_f8_ss(tmem_o(set), vd + ks * four, pd + 2 * ks, idesc_o, kt > 0 || ks > 0 ? 1u : 0u);
                        mma_commit(&s.o_done[set][b]);
                        mma_commit(&s.kv_empty[st]);
                    }
                }
            }
            if (!ok) atomicCAS(a.status, 0, PA_DEVICE_TIMEOUT_MMA);
        }
    } else {
        // -------------------------------------------------------- softmax --
        const int grp = warp >> 2, w4 = warp & 3, row = tid & 127;   // row: key of a tile, dim of the output
        const int set = kJoin ? 0 : grp, g_at = kJoin ? grp * GC : 0;  // buffers; first of the group's columns of a unit
        const int s_at = QP * g_at, p_at = 3 * g_at;                   // and of its rows of Q and P
        const uint32_t lane_off = (uint32_t)(32 * w4) << 16;
        const int64_t rows = (int64_t)a.plan.queries * a.hq;
        bool ok = true;
        int t = 0;                                   // tiles of this group's units
        auto wait = [&](uint64_t *bar, uint32_t parity, long long limit = 2000000000ll) {
            if (ok) ok = __all_sync(0xffffffffu, mbar_wait(bar, parity, limit));
        };
        constexpr long long kUnitLimit = 20000000000ll;   // where the other group's whole unit, of 2^30 keys at most, comes before
        // one arrival a warp, for what its lanes have done and fenced
        auto warp_arrive = [&](uint64_t *bar) {
            __syncwarp();
            if (lane == 0) mbar_arrive(bar);
        };
        auto read_unit = [&](int i) -> Unit {
            wait(&s.up_full[i % kUnits], (i / kUnits) & 1, kUnitLimit);
            const Unit x = s.unit[i % kUnits];
            __syncwarp();
            if (lane == 0) mbar_arrive(&s.up_empty[i % kUnits]);
            return x;
        };
        // first element of a column's row in q and the output, of the 64 or 128 it has
        auto row_of = [&](const Unit &x, const Column &c) -> int64_t {
            return (int64_t)(x.qi + c.k) * a.hq + (int64_t)(x.kvh * RH + c.real) * tp.group + x.g0 + c.h;
        };
        auto held = [&](const Unit &x, const Column &c) -> bool {
            return c.k < x.nq && c.h < x.heads && (RH == 1 || x.kvh * RH + c.real < a.hkv);
        };
        uint32_t second = 0;                         // columns of the second head of a pair
        if (RH == 2)
#pragma unroll
            for (int g = 0; g < GC; ++g) second |= (uint32_t)s.column[g_at + g].real << g;
        // Query rows: the group's warp w holds its columns w * GC/4 .., four dims a lane.
        struct Q4 { uint2 w[GC / 4]; };
        auto load_q = [&](const Unit &x) -> Q4 {
            Q4 r;
#pragma unroll
            for (int k = 0; k < GC / 4; ++k) {
                const Column c = s.column[g_at + w4 * (GC / 4) + k];
                const bool mine = held(x, c) && (RH == 1 || lane >> 4 == c.real);
                r.w[k] = mine ? reinterpret_cast<const uint2 *>(static_cast<const T *>(a.q) + row_of(x, c) * D)[lane % (32 / RH)]
                              : make_uint2(0u, 0u);
            }
            return r;
        };
        auto store_q = [&](const Q4 &r) {
#pragma unroll
            for (int k = 0; k < GC / 4; ++k) {
                const int g = w4 * (GC / 4) + k;
                union { uint2 w; T t[4]; } in;
                in.w = r.w[k];
                float x[4];
                uint32_t top = 0;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    x[e] = to_f32<T>(in.t[e]);
                    top = max(top, finite_bits(x[e]));
                }
                const uint32_t b = scale_byte(__reduce_max_sync(0xffffffffu, top));
                if (lane == 0) s.ref[grp][g].z = power_of(b) * tp.scale_log2;
                float inv = power_of(254u - b);
#pragma unroll
                for (int piece = 0; piece < QP; ++piece) {
                    const uint32_t lo = pack2_e4m3(x[0], x[1], inv), hi = pack2_e4m3(x[2], x[3], inv);
                    const int n = s_at + piece * GC + g;
                    *reinterpret_cast<uint32_t *>(s.q[set] + n * 128 + (((lane >> 2) ^ (n & 7)) << 4) + (lane & 3) * 4) = lo | hi << 16;
                    // what is left, sixteen times as large
                    const float2 u = unpack2_e4m3(lo), v = unpack2_e4m3(hi);
                    x[0] = (x[0] * inv - u.x) * 16.f;
                    x[1] = (x[1] * inv - u.y) * 16.f;
                    x[2] = (x[2] * inv - v.x) * 16.f;
                    x[3] = (x[3] * inv - v.y) * 16.f;
                    inv = 1.f;
                }
            }
            fence_proxy_async_smem();
            warp_arrive(&s.q_ready[set]);
        };
        // References of a unit to come, and its columns' keys.  A column without a query head has
        // references that nothing passes, and weights of 0.
        auto begin = [&](const Unit &x) {
            if (row < GC) {
                const Column c = s.column[g_at + row];
                s.ref[grp][row].x = s.ref[grp][row].y = held(x, c) ? -INFINITY : INFINITY;
                if (x.nq > 1) {
                    int64_t lo, hi;
                    visible_range(x.pos + c.k, x.seq_len, a.causal, a.window, lo, hi);
                    s.range[grp][row] = make_int2(lo > x.j0 ? (int)lo : x.j0, hi < x.j1 ? (int)hi : x.j1);
                    for (int w = 0; w < 4; ++w) s.nan[grp][row][w] = 0;
                }
            }
            __syncwarp();
        };
        Unit x{};
        const int first = kJoin ? 0 : grp, stride = kJoin ? 1 : 2;      // the group's units
        if (unit_of(first) < units) {
            x = read_unit(first);
            begin(x);
            if (ok && x.n_kt > 0) store_q(load_q(x));
        }
        for (int i = first; unit_of(i) < units; i += stride) {
            // the group's warps know the unit and see its queries' scales, or leave together
            if (group_any(grp, !ok)) {
                ok = false;
                break;
            }
            float l[GC];
#pragma unroll
            for (int g = 0; g < GC; ++g) l[g] = 0.f;
            int2 inner = make_int2(0, 0);        // keys that every query of the unit sees
            if (x.nq > 1) {
                int64_t lo, hi, none;
                visible_range(x.pos, x.seq_len, a.causal, a.window, none, hi);
                visible_range(x.pos + x.nq - 1, x.seq_len, a.causal, a.window, lo, none);
                inner = make_int2((int)lo, (int)hi);
            }
            // references and query scales, in registers (read from shared memory for every tile they
            // cost the decode layer 10 us)
            float ref_u[GC], ref_s[GC], scale_q[GC];
            auto take = [&] {
#pragma unroll
                for (int g = 0; g < GC; ++g) {
                    ref_u[g] = s.ref[grp][g].x;
                    ref_s[g] = s.ref[grp][g].y;
                }
            };
            take();
#pragma unroll
            for (int g = 0; g < GC; ++g) scale_q[g] = s.ref[grp][g].z;
            for (int kt = 0; kt < x.n_kt; ++kt, ++t) {
                const int b = t % kBuf, pb = t % kPBuf;
                const int gt = x.first + kt, st = gt % kStages;
                const int j = x.jb + kt * kN + row;
                const bool seen = j >= x.j0 && j < x.j1;
                // S^T first: a stage's barriers serve both groups' tiles, and only once this tile has
                // been scored is its stage's phase the one meant
                __syncwarp();                 // (tensor memory is read by whole warps, after a wait in vain too)
                wait(&s.s_full[set][b], (t / kBuf) & 1, kt == 0 ? kUnitLimit : 2000000000ll);
                tc_fence_after();
                wait(&s.scale_full[st], (gt / kStages) & 1);
                float kf[RH], ev[RH];
#pragma unroll
                for (int h = 0; h < RH; ++h) {
                    kf[h] = power_of(s.scale[st][h][row]);
                    ev[h] = (float)s.scale[st][RH + h][row] - 127.f;
                }
                auto kf_of = [&](int g) -> float { return RH == 2 && (second >> g & 1u) ? kf[RH - 1] : kf[0]; };
                auto ev_of = [&](int g) -> float { return RH == 2 && (second >> g & 1u) ? ev[RH - 1] : ev[0]; };
                uint32_t c[QP * GC < 16 && QP * GC > 8 ? 16 : QP * GC];
                tmem_load(tmem_s(set, b) + lane_off + s_at, c);
                tmem_wait_ld();
                tc_fence_before();
                warp_arrive(&s.s_read[set][b]);
                float sco[GC];
                bool past = false;
                const bool masks = x.nq > 1 && (x.jb + kt * kN < inner.x || x.jb + kt * kN + kN > inner.y);
#pragma unroll
                for (int g = 0; g < GC; ++g) {
                    float y = __uint_as_float(c[(QP - 1) * GC + g]);
#pragma unroll
                    for (int piece = QP - 2; piece >= 0; --piece) y = fmaf(y, 0.0625f, __uint_as_float(c[piece * GC + g]));
                    sco[g] = seen ? y * kf_of(g) * scale_q[g] : -INFINITY;
                    past |= sco[g] + ev_of(g) > ref_u[g] + kSlack || sco[g] > ref_s[g] + kSumSlack;
                }
                if (masks) {
                    // (a score that is not seen after all may have raised the alarm in vain)
#pragma unroll
                    for (int g = 0; g < GC; ++g) {
                        const int2 range = s.range[grp][g];
                        if (j < range.x || j >= range.y) sco[g] = -INFINITY;
                    }
                }
                if (group_any(grp, past)) {
                    // new references: the maxima of the tile where they are above the old ones
#pragma unroll
                    for (int g = 0; g < GC; ++g) {
                        const float mu = warp_max(sco[g] + ev_of(g)), ms = warp_max(sco[g]);
                        if (lane == 0) {
                            s.red[grp][w4][g][0] = mu;
                            s.red[grp][w4][g][1] = ms;
                        }
                    }
                    group_bar(grp);
                    if (row < GC) {
                        const float4 old = s.ref[grp][row];
                        float mu = old.x, ms = old.y;
#pragma unroll
                        for (int w = 0; w < 4; ++w) {
                            mu = fmaxf(mu, s.red[grp][w][row][0]);
                            ms = fmaxf(ms, s.red[grp][w][row][1]);
                        }
                        s.change[grp][row] = make_float2(mu > old.x ? ex2(old.x - mu) : 1.f, ms > old.y ? ex2(old.y - ms) : 1.f);
                        s.ref[grp][row].x = mu;
                        s.ref[grp][row].y = ms;
                    }
                    group_bar(grp);
#pragma unroll
                    for (int g = 0; g < GC; ++g) l[g] *= s.change[grp][g].y;
                    take();
                    if (kt > 0) {
                        wait(&s.o_done[set][(t - 1) % kPBuf], ((t - 1) / kPBuf) & 1);
                        tc_fence_after();
#pragma unroll
                        for (int c0 = 0; c0 < 3 * GC; c0 += 8) {
                            uint32_t o[8];
                            tmem_ld8(tmem_o(set) + lane_off + p_at + c0, o);
                            tmem_wait_ld();
#pragma unroll
                            for (int e = 0; e < 8; ++e)
                                if (c0 + e < 3 * GC) o[e] = __float_as_uint(__uint_as_float(o[e]) * s.change[grp][(c0 + e) % GC].x);
                            tmem_st8(tmem_o(set) + lane_off + p_at + c0, o);
                        }
                        tmem_wait_st();
                    }
                }
                // the P buffer's last tile has been through the tensor core
                if (t >= kPBuf) wait(&s.o_done[set][pb], ((t / kPBuf) - 1) & 1);
                uint8_t *const prow = s.p[set][pb] + p_at * 128 + (row & 15);
                const int chunk = row >> 4;
#pragma unroll
                for (int g = 0; g < GC; g += 2) {
                    float p[2];
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        p[e] = ex2(sco[g + e] + ev_of(g + e) - (ref_u[g + e] == -INFINITY ? 0.f : ref_u[g + e]) + kTop);
                        l[g + e] += ex2(sco[g + e] - (ref_s[g + e] == -INFINITY ? 0.f : ref_s[g + e]));
                    }
                    float up = 1.f;
#pragma unroll
                    for (int piece = 0; piece < 3; ++piece) {
                        const uint32_t two = to_e5m2(p[0], p[1]);
                        const int n0 = piece * GC + g, n1 = n0 + 1;   // (p_at is a multiple of eight)
                        prow[n0 * 128 + ((chunk ^ (n0 & 7)) << 4)] = (uint8_t)two;
                        prow[n1 * 128 + ((chunk ^ (n1 & 7)) << 4)] = (uint8_t)(two >> 8);
                        if (piece < 2) {
                            const float2 f = from_e5m2(two);
                            up = piece == 0 ? 8.f : 16.f;
                            p[0] = (p[0] - f.x) * up;
                            p[1] = (p[1] - f.y) * up;
                        }
                    }
                }
                // value rows that the unit does not see must not reach O^T (tail slots may hold NaN)
                if ((!kJoin || grp == 0) && (masks || x.jb + kt * kN + kN > x.j1 || x.jb + kt * kN < x.j0)) {
                    wait(&s.kv_full[st], (gt / kStages) & 1);
                    uint8_t *const v = s.kv[st] + tp.v_at + (row >> 3) * tp.eight + (row & 7) * 128;
                    if (!seen) {
#pragma unroll
                        for (int e = 0; e < 8; ++e) *reinterpret_cast<uint4 *>(v + e * 16) = make_uint4(0u, 0u, 0u, 0u);
                    } else if (masks && (j < inner.x || j >= inner.y)) {
                        // a row for some of the unit's queries, which weighs 0 for the others: NaN
                        // in it is taken out here and given to those it belongs to at the end
                        uint32_t some = 0;               // bit 7 of the bytes that are NaN
#pragma unroll
                        for (int e = 0; e < 8; ++e) {
                            const uint4 w = *reinterpret_cast<const uint4 *>(v + ((e + row) & 7) * 16);
                            some |= nan_bytes(w.x) | nan_bytes(w.y) | nan_bytes(w.z) | nan_bytes(w.w);
                        }
                        for (int e = 0; some != 0 && e < 32; ++e) {
                            uint32_t *const word = reinterpret_cast<uint32_t *>(v) + e;
                            const uint32_t is_nan = nan_bytes(*word);
                            if (is_nan == 0) continue;
                            *word &= ~(is_nan | (is_nan - (is_nan >> 7)));
                            const int dim = ((e >> 2) ^ (row & 7)) * 16 + (e & 3) * 4;
                            const uint32_t bits = (is_nan >> 7 & 1u) | (is_nan >> 14 & 2u) | (is_nan >> 21 & 4u) | (is_nan >> 28 & 8u);
                            for (int g = 0; g < GH; ++g) {
                                const int2 range = s.range[grp + g / GC][g % GC];
                                if (j >= range.x && j < range.y) atomicOr(&s.nan[grp + g / GC][g % GC][dim >> 5], bits << (dim & 31));
                            }
                        }
                    }
                }
                fence_proxy_async_smem();       // the generic stores before the tensor core reads them
                tc_fence_before();
                warp_arrive(&s.p_ready[set][pb]);
            }
            // ------------------------------------------------------ epilogue --
            // the group's next unit: its queries are on their way during the rest
            const bool more = unit_of(i + stride) < units;
            Unit nx = x;
            Q4 qn{};
            if (more) {
                nx = read_unit(i + stride);
                if (ok) qn = load_q(nx);
            }
            const int part = row / D, col = row % D;         // the head of a pair this dim belongs to
            if (x.n_kt == 0) {
                if (a.ws_o) {        // an empty split
                    for (int g = 0; g < GC; ++g) {
                        const Column c = s.column[g_at + g];
                        if (!held(x, c) || part != c.real) continue;
                        const int64_t at = (int64_t)x.split * rows + row_of(x, c);
                        a.ws_o[at * D + col] = 0.f;
                        if (col == 0) a.ws_lse[at] = -INFINITY;
                    }
                }
            } else {
                // a thread a column sums the warps and works out what its output is multiplied by
#pragma unroll
                for (int g = 0; g < GC; ++g) {
                    for (int o = 16; o; o >>= 1) l[g] += __shfl_xor_sync(0xffffffffu, l[g], o);
                    if (lane == 0) s.sum[grp][w4][g] = l[g];
                }
                // (the first group notes NaN for both until it hands over its last weights)
                if (kJoin) wait(&s.o_done[set][(t - 1) % kPBuf], ((t - 1) / kPBuf) & 1);
                group_bar(grp);
                if (row < GC) {
                    const Column c = s.column[g_at + row];
                    const float4 ref = s.ref[grp][row];
                    const float L = (s.sum[grp][0][row] + s.sum[grp][1][row]) + (s.sum[grp][2][row] + s.sum[grp][3][row]);
                    const bool there = held(x, c);
                    const int64_t at = there ? row_of(x, c) + (a.ws_o ? (int64_t)x.split * rows : 0) : -1;
                    // L is 0 only where no key was seen; NaN stays NaN.  Two factors: the power goes down to
                    // 2^-126 with the values' scales, and divided by L (2^16 for as many equal scores) it
                    // would leave fp32's range where the output does not.
                    s.out[grp][row].at = at;
                    s.out[grp][row].inv = L == 0.f ? 0.f : exp2f(-kTop) / L;
                    s.out[grp][row].up = exp2f(ref.x - ref.y);
                    s.out[grp][row].real = c.real;
                    for (int w = 0; w < 4; ++w) s.out[grp][row].nan[w] = x.nq > 1 ? s.nan[grp][row][w] : 0u;
                    if (there && a.ws_o) a.ws_lse[at] = L == 0.f ? -INFINITY : (ref.y + log2f(L)) * kLn2;
                }
                group_bar(grp);
                wait(&s.o_done[set][(t - 1) % kPBuf], ((t - 1) / kPBuf) & 1);
                tc_fence_after();
                uint32_t o[GC == 8 ? 24 : 16];
                tmem_load(tmem_o(set) + lane_off + p_at, o);
                tmem_wait_ld();
#pragma unroll
                for (int g = 0; g < GC; ++g) {
                    const int64_t at = s.out[grp][g].at;
                    const float inv = s.out[grp][g].inv;
                    const float v = fmaf(fmaf(__uint_as_float(o[2 * GC + g]), 0.0625f, __uint_as_float(o[GC + g])), 0.125f, __uint_as_float(o[g]));
                    const bool is_nan = s.out[grp][g].nan[w4] >> lane & 1u;
                    const float y = is_nan ? __uint_as_float(0x7fffffffu) : inv == 0.f ? 0.f : v * inv * s.out[grp][g].up;
                    if (at >= 0 && (RH == 1 || part == s.out[grp][g].real)) {
                        if (a.ws_o)
                            a.ws_o[at * D + col] = y;
                        else
                            static_cast<T *>(a.out)[at * D + col] = rounded<T>(y);
                    }
                }
            }
            if (x.n_kt > 0) {
                tc_fence_before();
                warp_arrive(&s.o_free[set]);
            }
            if (more) {
                begin(nx);                             // (the group has read this unit's references)
                if (nx.n_kt > 0) store_q(qn);          // S^T of the unit is done: its queries may go
            }
            x = nx;
        }
        if (!ok && lane == 0) atomicCAS(a.status, 0, PA_DEVICE_TIMEOUT_SOFTMAX);
    }
    griddep_launch();
    tc_fence_before();
    __syncthreads();
    if (warp == 0) {
        tc_fence_after();
        tmem_dealloc(tmem, kTmemCols);
    }
}

bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

int log2_exact(int v) {
    if (v <= 0 || (v & (v - 1))) return -1;
    int s = 0;
    while ((1 << s) < v) ++s;
    return s;
}

template <typename T, int GH, int QP, int RH>
cudaError_t launch_gh(const Q8AttnArgs &q, int items, int use_list, int run, cudaStream_t st) {
    const AttnArgs &a = q.a;
    using S = Shared<GH, QP, RH>;
    static_assert(sizeof(S) <= 232448, "shared memory above the per-block limit");
    TcParams tp{};
    tp.group = a.hq / a.hkv;
    tp.per = RH * tp.group <= GH ? tp.group : GH / RH;
    tp.chunks = (tp.group + tp.per - 1) / tp.per;
    tp.rq = run > 1 && tp.chunks == 1 ? GH / (RH * tp.per) : 1;
    tp.ps_shift = log2_exact(a.plan.page_size);
    tp.box_rows = a.plan.page_size < kN ? a.plan.page_size : kN;
    tp.scale_log2 = a.scale * kLog2e;
    // K and V as one tensor, the distance of their buffers being a stride: {bytes of a slot,
    // eight rows, the two tensors, eights of rows}.  A box of a page's rows of one head, of
    // both, takes the TMA unit as long as one of K alone: about 100 cycles, which with pages
    // of 16 rows and a box for each left HBM waiting (5.8 TB/s; 6.4 with pages of 64).
    // Buffers further apart than a stride may be (2^40 bytes; the allocator places some so)
    // have a box each.
    const uintptr_t ka = reinterpret_cast<uintptr_t>(a.k), va = reinterpret_cast<uintptr_t>(a.v);
    const uint64_t apart = ka < va ? va - ka : ka - va;
    tp.together = apart > 0 && apart < (uint64_t)1 << 40;
    tp.eight = tp.together ? 2048 : 1024;
    tp.k_at = tp.together && ka > va ? 1024 : 0;
    tp.v_at = !tp.together ? kTile : ka > va ? 0 : 1024;
    const uint64_t slot = (uint64_t)a.d * a.hkv, rows = (uint64_t)a.plan.pages * a.plan.page_size;
    const uint64_t dims[4] = {slot, 8, tp.together ? 2u : 1u, rows / 8}, strides[3] = {slot, tp.together ? apart : slot, 8 * slot};
    const uint32_t box[4] = {kD, 8, tp.together ? 2u : 1u, (uint32_t)tp.box_rows / 8};
    CUtensorMap tk, tv;
    if (!encode_map(&tk, kTmaBytes, tp.together && ka > va ? a.v : a.k, 4, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B))
        return cudaErrorInvalidValue;
    tv = tk;
    if (!tp.together && !encode_map(&tv, kTmaBytes, a.v, 4, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B)) return cudaErrorInvalidValue;
    static PerDevice known;
    int resident = 0;
    cudaError_t e = resident_ctas(known, q8_decode_tc_kernel<T, GH, QP, RH>, kThreads, sizeof(S), resident);
    if (e != cudaSuccess) return e;
    const int64_t units = (int64_t)items * a.splits * ((a.hkv + RH - 1) / RH) * tp.chunks;
    if (units > INT32_MAX) return cudaErrorInvalidValue;
    int64_t ctas = units;
    if (ctas > resident) ctas = resident;
    if (a.max_ctas > 0 && a.max_ctas < ctas) ctas = a.max_ctas;
    return launch_pdl(q8_decode_tc_kernel<T, GH, QP, RH>, dim3((unsigned)ctas), dim3(kThreads), sizeof(S), st, tk, tv, q, use_list, tp);
}

// Columns of a unit: the smallest of 4, 8 and 16 that holds the heads of the longest run of
// consecutive queries.
template <typename T, int QP, int RH>
cudaError_t launch_t(const Q8AttnArgs &q, int items, int use_list, int run, cudaStream_t st) {
    const int64_t columns = (int64_t)RH * (q.a.hq / q.a.hkv) * run;
    return columns <= 4 ? launch_gh<T, 4, QP, RH>(q, items, use_list, run, st)
           : columns <= 8 ? launch_gh<T, 8, QP, RH>(q, items, use_list, run, st)
                          : launch_gh<T, 16, QP, RH>(q, items, use_list, run, st);
}

}  // namespace

bool q8_decode_tc_supported(const Q8AttnArgs &q) {
    const AttnArgs &a = q.a;
    return a.dtype != PA_F32 && a.d == a.dv && (a.d == kD || a.d == kD / 2) &&
           log2_exact(a.plan.page_size) >= 4 && aligned16(a.q) && aligned16(a.k) && aligned16(a.v) && aligned16(q.k_scale) &&
           aligned16(q.v_scale) && tma_available();
}

cudaError_t launch_q8_decode_tc(const Q8AttnArgs &q, bool use_decode_list, int longest_run, cudaStream_t st) {
    const int items = use_decode_list ? q.a.plan.n_decode : q.a.plan.queries;
    if (items == 0) return cudaSuccess;
    const int ul = use_decode_list ? 1 : 0, run = use_decode_list ? longest_run : 16;
    if (q.a.d == kD)
        return q.a.dtype == PA_BF16 ? launch_t<__nv_bfloat16, 2, 1>(q, items, ul, run, st) : launch_t<__half, 3, 1>(q, items, ul, run, st);
    return q.a.dtype == PA_BF16 ? launch_t<__nv_bfloat16, 2, 2>(q, items, ul, run, st) : launch_t<__half, 3, 2>(q, items, ul, run, st);
}

}  // namespace pa
