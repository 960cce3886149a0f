// Eviction from a paged cache by accumulated attention weight.
//
// Per (sequence, KV head) with n keys and a budget of `keep` of them: the first
// `sink` and the last `recent` keys stay, and of the others the keep - sink -
// recent with the largest totals (equal totals: the lower index stays; a NaN
// total counts below every number).  The kept keys move, in cache order, to the
// rows 0 .. keep-1 of the destination schedule: its pages are the sequence's own
// ones or fresh ones.
//
// Two kernels.  `select_kernel` finds the keep-th largest total by narrowing an
// interval of order-preserving 32-bit keys, up to 11 bits a round, and writes the
// kept indices in ascending order.  `move_kernel` moves the rows; in place that is safe without
// any ordering between CTAs: a CTA owns a column slice of one (sequence, head)
// and walks the ranks upwards, rank i reads row src(i) >= i and writes row i, so
// what a chunk of ranks writes has been read by this or an earlier chunk, and a
// barrier between the reads and the writes of a chunk is all it takes.

#include <algorithm>
#include <type_traits>

#include "pa_internal.h"
#include "per_device.h"
#include "sm103_tc.cuh"

namespace pa {
namespace {

// Physical row of key j of sequence s, -1 when the table maps none.
// ps_shift: log2(page size), -1 when it is no power of two.
__device__ __forceinline__ int64_t slot_of(const PlanView &p, int s, int j, int ps_shift) {
    const int g = ps_shift >= 0 ? j >> ps_shift : j / p.page_size;
    if (g >= p.width) return -1;
    const int pg = p.table[(int64_t)s * p.width + g];
    return pg < 0 || pg >= p.pages ? -1 : (int64_t)pg * p.page_size + (j - g * p.page_size);
}

__device__ __forceinline__ int64_t mass_at(int64_t slot, int h, int hkv, int ps, int ps_shift) {
    const int64_t pg = ps_shift >= 0 ? slot >> ps_shift : slot / ps;
    return (pg * hkv + h) * ps + (slot - pg * ps);
}

// Keys whose unsigned order is the order of the totals: 0 is no key at all, NaN
// counts below every number, -0 = +0.
__device__ __forceinline__ uint32_t order_key(float x) {
    if (x != x) return 1u;
    const uint32_t u = __float_as_uint(x == 0.f ? 0.f : x);
    return ((u & 0x80000000u) ? ~u : (u | 0x80000000u)) + 1u;    // -inf: 0x00800000, +inf: 0xff800001
}

struct Budget {
    int n, keep, first, last, want;   // candidates [first, last), `want` of them stay
};

__device__ __forceinline__ Budget budget_of(const EvictArgs &a, int s) {
    Budget b;
    b.n = a.src.seq_lens[s];
    if (b.n > kMaxCountedKeys) b.n = 0;       // (only a device copy's length: select_kernel reports it)
    b.keep = min(min(a.dst.seq_lens[s], b.n), a.kept_stride);
    b.first = min(a.sink, b.keep);
    const int r = min(a.recent, b.keep - b.first);
    b.last = b.n - r;
    b.want = b.keep - b.first - r;
    return b;
}

// ------------------------------------------------------------------ choice --
// One cluster of C CTAs per (sequence, head); CTA r holds the r-th part of the
// candidates' order keys in shared memory (they are re-read from global memory
// when a part is longer than fits).  The keep-th largest key is found by
// narrowing an interval [lo, hi] of keys: 2048 equal bins over it, counted with
// shared-memory atomics, the bin that holds the threshold becomes the interval
// (11 bits a round, so at most three; bins follow the data's own range, which
// spreads the counts: totals crowd into a few exponents).  Each CTA adds up the
// cluster's histograms itself, through distributed shared memory.
constexpr int kBins = 2048;
constexpr int kMaxSelectWarps = 32;
constexpr uint32_t kMaxCluster = 8;

struct SelectShared {
    int hist[kBins];
    int warp_a[kMaxSelectWarps], warp_b[kMaxSelectWarps];
    uint32_t lo, hi;          // this CTA's smallest and largest key
    int above, equal;         // this CTA's keys above / at the threshold
    int found_bin, found_above, found_count;
};

template <typename V> __device__ __forceinline__ const V *peer(const V *p, uint32_t rank) {
    uint64_t out;
    asm("mapa.u64 %0, %1, %2;\n" : "=l"(out) : "l"(reinterpret_cast<uint64_t>(p)), "r"(rank));
    return reinterpret_cast<const V *>(out);
}

// room: fours of keys the dynamic shared memory holds.  A part that is longer
// (the device lengths can exceed the host's that sized the launch) is re-read
// instead.  quads: the totals of four keys at a multiple of four lie together.
// A lone CTA has 512 threads, three of them fit an SM; the CTAs of a cluster have
// an SM each and 1024 threads.
template <bool kCluster>
__global__ void __launch_bounds__(kCluster ? 1024 : 512, kCluster ? 1 : 3) select_kernel(EvictArgs a, int ps_shift, int room, int quads) {
    griddep_wait();
    griddep_launch();
    constexpr int kSelectThreads = kCluster ? 1024 : 512, kSelectWarps = kSelectThreads / 32;
    constexpr int kPer = kBins / kSelectThreads;       // bins a thread
    using Bins = typename std::conditional<kPer == 2, int2, int4>::type;
    union Pack {
        Bins v;
        int i[kPer];
    };
    extern __shared__ uint4 staged[];
    __shared__ __align__(16) SelectShared sh;
    const uint32_t C = kCluster ? tc::cluster_nctarank() : 1u, rank = kCluster ? tc::cluster_ctarank() : 0u;
    const int pair = (int)(blockIdx.x / C);
    const int h = pair % a.hkv, s = pair / a.hkv;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const Budget b = budget_of(a, s);
    int32_t *kept = a.kept + ((int64_t)s * a.hkv + h) * a.kept_stride;
    const int all = (int)C * kSelectThreads, me = (int)rank * kSelectThreads + tid;
    // what needs no choice: the sink, the recent keys, the places past the budget
    auto write_fixed = [&]() {
        for (int i = me; i < b.first; i += all) kept[i] = i;
        for (int i = me; i < b.n - b.last; i += all) kept[b.first + b.want + i] = b.last + i;
        for (int i = b.keep + me; i < a.kept_stride; i += all) kept[i] = -1;
    };
    // what the host could not see of a source that advanced on the device: a budget
    // above the length (every key stays), or one too small for the sink and the recent
    // keys of a sequence that was to stay as it is
    if (me == 0 && h == 0 && (a.dst.seq_lens[s] > b.n || (b.keep < b.n && b.keep < a.sink + a.recent)))
        atomicCAS(a.status, 0, PA_DEVICE_RANGE);
    if (b.keep == b.n) {                      // the whole cluster leaves here together
        for (int i = me; i < a.kept_stride; i += all) kept[i] = i < b.n ? i : -1;
        return;
    }
    if (b.want == 0) {
        write_fixed();
        return;
    }
    // a cluster barrier's release waits for every earlier store and costs ~2000
    // cycles a time where __syncthreads costs tens: no store comes before the last
    // one, and a CTA alone uses the latter
    auto barrier = [&]() {
        if (kCluster)
            tc::cluster_barrier();
        else
            __syncthreads();
    };

    // the candidates as aligned fours (places outside [first, last) hold no key), my
    // part of them
    const int j0 = b.first & ~3, fours = (b.last - j0 + 3) / 4;
    const int span = (fours + (int)C - 1) / (int)C;
    const int part0 = min(fours, (int)rank * span), cnt = min(fours, part0 + span) - part0;
    bool mapped = true;                        // every place seen had a page (no branch: loads stay in flight)
    auto fetch = [&](int q) -> uint4 {
        const int j = j0 + 4 * (part0 + q);
        float m[4];
        if (quads) {
            const int64_t slot = slot_of(a.src, s, j, ps_shift);
            mapped &= slot >= 0;
            const float4 v = *reinterpret_cast<const float4 *>(
                a.key_mass + mass_at(slot < 0 ? 0 : slot, h, a.hkv, a.src.page_size, ps_shift));
            m[0] = v.x; m[1] = v.y; m[2] = v.z; m[3] = v.w;
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int64_t slot = slot_of(a.src, s, min(max(j + i, b.first), b.last - 1), ps_shift);
                mapped &= slot >= 0;
                m[i] = a.key_mass[mass_at(slot < 0 ? 0 : slot, h, a.hkv, a.src.page_size, ps_shift)];
            }
        }
        auto k = [&](int i) { return j + i >= b.first && j + i < b.last ? order_key(m[i]) : 0u; };
        return make_uint4(k(0), k(1), k(2), k(3));
    };
    const bool fits = span <= room;
    auto key4 = [&](int q) -> uint4 { return fits ? staged[q] : fetch(q); };

    uint32_t lo = 0xffffffffu, hi = 0u;
#pragma unroll 8
    for (int q = tid; q < cnt; q += kSelectThreads) {
        const uint4 k = fetch(q);
        if (fits) staged[q] = k;
        // 0 wraps to the top for the minimum and is never the maximum
        lo = min(min(lo, min(k.x - 1u, k.y - 1u)), min(k.z - 1u, k.w - 1u));
        hi = max(max(hi, max(k.x, k.y)), max(k.z, k.w));
    }
    lo = lo == 0xffffffffu ? lo : lo + 1u;
    lo = __reduce_min_sync(0xffffffffu, lo);
    hi = __reduce_max_sync(0xffffffffu, hi);
    if (lane == 0) {
        sh.warp_a[warp] = (int)lo;
        sh.warp_b[warp] = (int)hi;
    }
    __syncthreads();
    if (kCluster) {
        if (tid == 0) {
#pragma unroll
            for (int w = 0; w < kSelectWarps; ++w) {
                lo = min(lo, (uint32_t)sh.warp_a[w]);
                hi = max(hi, (uint32_t)sh.warp_b[w]);
            }
            sh.lo = lo;
            sh.hi = hi;
        }
        barrier();
        lo = __reduce_min_sync(0xffffffffu, lane < (int)C ? *peer(&sh.lo, lane) : 0xffffffffu);
        hi = __reduce_max_sync(0xffffffffu, lane < (int)C ? *peer(&sh.hi, lane) : 0u);
    } else {
        lo = __reduce_min_sync(0xffffffffu, lane < kSelectWarps ? (uint32_t)sh.warp_a[lane] : 0xffffffffu);
        hi = __reduce_max_sync(0xffffffffu, lane < kSelectWarps ? (uint32_t)sh.warp_b[lane] : 0u);
    }
    // invariant: exactly b.want - need keys lie above hi, and need >= 1 of those in [lo, hi] stay
    int need = b.want;
    bool whole = false;                        // every key of [lo, hi] stays
    while (true) {
        const int width_bits = 32 - __clz((int)(hi - lo));     // 0 when lo == hi
        const int shift = width_bits > 11 ? width_bits - 11 : 0;
        Pack c;
#pragma unroll
        for (int i = 0; i < kPer; ++i) c.i[i] = 0;
        reinterpret_cast<Bins *>(sh.hist)[tid] = c.v;
        __syncthreads();
        const uint32_t width = hi - lo;
        for (int q = tid; q < cnt; q += kSelectThreads) {
            const uint4 k = key4(q);
            if (k.x - lo <= width) atomicAdd(&sh.hist[(k.x - lo) >> shift], 1);
            if (k.y - lo <= width) atomicAdd(&sh.hist[(k.y - lo) >> shift], 1);
            if (k.z - lo <= width) atomicAdd(&sh.hist[(k.z - lo) >> shift], 1);
            if (k.w - lo <= width) atomicAdd(&sh.hist[(k.w - lo) >> shift], 1);
        }
        barrier();
        // bins from the top: thread t holds bins kBins - kPer * (t + 1) .. kBins - 1 - kPer * t
        const int first = kBins - kPer * (tid + 1);
        if (!kCluster) {
            c.v = *reinterpret_cast<const Bins *>(&sh.hist[first]);
        } else {
            Pack x[kMaxCluster];
#pragma unroll
            for (uint32_t r = 0; r < kMaxCluster; ++r)
                x[r].v = *reinterpret_cast<const Bins *>(peer(&sh.hist[first], r < C ? r : rank));
#pragma unroll
            for (uint32_t r = 0; r < kMaxCluster; ++r)
#pragma unroll
                for (int i = 0; i < kPer; ++i) c.i[i] += r < C ? x[r].i[i] : 0;
        }
        int mine = 0;
#pragma unroll
        for (int i = 0; i < kPer; ++i) mine += c.i[i];
        int x = mine;
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, x, o);
            if (lane >= o) x += y;
        }
        if (lane == 31) sh.warp_a[warp] = x;
        __syncthreads();
        int before = x - mine;
#pragma unroll
        for (int w = 0; w < kSelectWarps; ++w) before += w < warp ? sh.warp_a[w] : 0;
        if (before < need && before + mine >= need) {
            int acc = before, bin = 0, in_bin = 0;
            bool found = false;
#pragma unroll
            for (int i = kPer - 1; i >= 0; --i) {          // from the top bin down
                if (!found && acc + c.i[i] >= need) {
                    found = true;
                    bin = first + i;
                    in_bin = c.i[i];
                }
                if (!found) acc += c.i[i];
            }
            sh.found_bin = bin;
            sh.found_above = acc;
            sh.found_count = in_bin;
        }
        // also: no CTA clears its histogram while another still reads it
        barrier();
        need -= sh.found_above;
        const uint32_t bin_lo = lo + ((uint32_t)sh.found_bin << shift);
        hi = (uint32_t)min((unsigned long long)hi, (unsigned long long)bin_lo + ((1ull << shift) - 1ull));   // the last bin may be cut
        lo = bin_lo;
        whole = sh.found_count == need;
        if (shift == 0 || whole) break;
        __syncthreads();
    }
    // a key stays when it is above hi, or in [lo, hi] and among the first `need`
    // of those (all of them when whole; else lo == hi: ties, the lowest indices)
    const uint32_t width = hi - lo;
    auto count = [&](uint32_t k) -> int { return k > hi ? 1 : (k - lo <= width ? 1 << 16 : 0); };
    int gt = 0, eq = 0;
    const int per_warp = ((cnt + kSelectWarps - 1) / kSelectWarps + 31) / 32 * 32;
    const int w0 = min(cnt, warp * per_warp), w1 = min(cnt, w0 + per_warp);
    for (int q = w0 + lane; q < w1; q += 32) {
        const uint4 k = key4(q);
        const int c = count(k.x) + count(k.y) + count(k.z) + count(k.w);
        gt += c & 0xffff;
        eq += c >> 16;
    }
    gt = __reduce_add_sync(0xffffffffu, gt);
    eq = __reduce_add_sync(0xffffffffu, eq);
    if (lane == 0) {
        sh.warp_a[warp] = gt;
        sh.warp_b[warp] = eq;
    }
    __syncthreads();
    int g0 = 0, e0 = 0, g_all = 0, e_all = 0;
#pragma unroll
    for (int w = 0; w < kSelectWarps; ++w) {
        const int g = sh.warp_a[w], e = sh.warp_b[w];
        g0 += w < warp ? g : 0;
        e0 += w < warp ? e : 0;
        g_all += g;
        e_all += e;
    }
    if (kCluster) {
        if (tid == 0) {
            sh.above = g_all;
            sh.equal = e_all;
        }
        barrier();
        g0 += __reduce_add_sync(0xffffffffu, lane < (int)rank ? *peer(&sh.above, lane) : 0);
        e0 += __reduce_add_sync(0xffffffffu, lane < (int)rank ? *peer(&sh.equal, lane) : 0);
        barrier();                             // no CTA leaves while another reads its counts
    }
    write_fixed();
    if (!mapped) atomicCAS(a.status, 0, PA_DEVICE_RANGE);
    for (int base = w0; base < w1; base += 32) {
        const int q = base + lane;
        const uint4 k4 = q < w1 ? key4(q) : make_uint4(0u, 0u, 0u, 0u);
        const uint32_t k[4] = {k4.x, k4.y, k4.z, k4.w};
        // above | equal << 16 of my four and of the lanes before me
        const int mine = count(k[0]) + count(k[1]) + count(k[2]) + count(k[3]);
        int x = mine;
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, x, o);
            if (lane >= o) x += y;
        }
        int g = g0 + ((x - mine) & 0xffff), e = e0 + ((x - mine) >> 16);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int c = count(k[i]);
            if (c == 1 || (c && e < need)) kept[b.first + g + min(e, need)] = j0 + 4 * (part0 + q) + i;
            g += c & 0xffff;
            e += c >> 16;
        }
        const int sum = __shfl_sync(0xffffffffu, x, 31);
        g0 += sum & 0xffff;
        e0 += sum >> 16;
    }
}

// -------------------------------------------------------------------- move --
constexpr int kMoveThreads = 256, kMoveRanks = 128, kMoveUnroll = 4;

__device__ __forceinline__ int2 lds_move(uint32_t addr) {
    int2 m;
    asm volatile("ld.shared.v2.s32 {%0, %1}, [%2];\n" : "=r"(m.x), "=r"(m.y) : "r"(addr));
    return m;
}

// Copies one column of kMoveUnroll rows of a chunk, `per` ranks apart: `at` is
// the thread's column of row 0, the rows are moves[r].x -> moves[r].y (y < 0:
// stays), looked up again for the stores so that registers hold little but the
// data in flight.
template <typename U, bool kOrdered>
__device__ __forceinline__ void move_column(U *at, uint32_t moves, int per, int64_t stride) {
    U v[kMoveUnroll];
#pragma unroll
    for (int u = 0; u < kMoveUnroll; ++u) {
        const int2 m = lds_move(moves + (uint32_t)(u * per) * 8u);
        if (m.y >= 0) v[u] = at[m.x * stride];
    }
    if (kOrdered) __syncthreads();           // every read of these ranks before any write of them
#pragma unroll
    for (int u = 0; u < kMoveUnroll; ++u) {
        const int2 m = lds_move(moves + (uint32_t)(u * per) * 8u);
        if (m.y >= 0) at[m.y * stride] = v[u];
    }
}

// kOrdered (some page is written in place): part p of a (sequence, head) owns
// column slice p of all its ranks and walks them upwards.  Otherwise nothing
// written is read, and part p takes every parts-th chunk of ranks, all columns.
// The ordered walk is bound by its own length, a barrier every 64 ranks: 64 histories
// of 0.5-8K to half (1024 CTAs) take 271 us a call in place and 185 into fresh pages, two
// of 100-131K to a quarter (two slices a list, 32 CTAs) 753 against 115.
template <typename U, bool kOrdered>
__global__ void __launch_bounds__(kMoveThreads, kOrdered ? 4 : 5)
    move_kernel(EvictArgs a, int ps_shift, int uk, int uv, int w_shift, int nk, int parts) {
    griddep_wait();
    griddep_launch();
    // source and destination rows of the chunk's ranks; past them nothing moves
    __shared__ int2 moves[kMoveRanks + kMoveThreads * kMoveUnroll];
    // heads fastest: the CTAs that run together write neighbouring rows of the same slots
    const int h = blockIdx.x % a.hkv;
    const int part = (int)(blockIdx.x / a.hkv) % parts, s = (int)(blockIdx.x / a.hkv) / parts;
    const int32_t *kept = a.kept + ((int64_t)s * a.hkv + h) * a.kept_stride;
    const int keep = budget_of(a, s).keep, ps = a.src.page_size;
    const int w = 1 << w_shift, lane = threadIdx.x & (w - 1), sub = threadIdx.x >> w_shift, per = kMoveThreads >> w_shift;
    U *kc = static_cast<U *>(a.k_cache) + (int64_t)h * uk + lane, *vc = static_cast<U *>(a.v_cache) + (int64_t)h * uv + lane;
    const int64_t sk = (int64_t)a.hkv * uk, sv = (int64_t)a.hkv * uv;
    for (int r = kMoveRanks + threadIdx.x; r < kMoveRanks + per * kMoveUnroll; r += kMoveThreads) moves[r] = make_int2(-1, -1);
    for (int base = kOrdered ? 0 : part * kMoveRanks; base < keep; base += kOrdered ? kMoveRanks : parts * kMoveRanks) {
        float m = 0.f;
        int64_t m_to = -1;
        bool moving = false;
        __syncthreads();                     // the last chunk's rows are done with
        if (threadIdx.x < kMoveRanks) {
            int2 mv = make_int2(-1, -1);
            const int i = base + threadIdx.x;
            if (i < keep) {
                const int64_t f = slot_of(a.src, s, kept[i], ps_shift), t = slot_of(a.dst, s, i, ps_shift);
                if (f < 0 || t < 0)
                    atomicCAS(a.status, 0, PA_DEVICE_RANGE);
                else if (f != t)
                    mv = make_int2((int)f, (int)t);
                if (mv.y >= 0 && (!kOrdered || part == 0)) {
                    m = a.key_mass[mass_at(f, h, a.hkv, ps, ps_shift)];
                    m_to = mass_at(t, h, a.hkv, ps, ps_shift);
                }
            }
            moving = mv.y >= 0;
            moves[threadIdx.x] = mv;
        }
        if (!__syncthreads_or(moving)) continue;
        if (m_to >= 0) a.key_mass[m_to] = m;
#pragma unroll 1
        for (int r0 = 0; r0 < kMoveRanks; r0 += per * kMoveUnroll) {
            uint32_t mv = tc::smem_u32(moves + r0 + sub);
            if (kOrdered) {
                const bool is_k = part < nk;
                const int c0 = (is_k ? part : part - nk) << w_shift;
                if (c0 + lane >= (is_k ? uk : uv)) mv = tc::smem_u32(moves + kMoveRanks + sub);     // no such column
                move_column<U, true>((is_k ? kc : vc) + c0, mv, per, is_k ? sk : sv);
            } else {
                // one loop over the columns of both tensors: a single copy of the body
#pragma unroll 1
                for (int c = lane; c < uk + uv; c += w) {
                    U *at = c < uk ? kc + (c - lane) : vc + (c - lane - uk);
                    move_column<U, false>(at, mv, per, c < uk ? sk : sv);
                }
            }
        }
    }
}

int ps_shift_of(int ps) {
    if (ps & (ps - 1)) return -1;
    int s = 0;
    while ((1 << s) < ps) ++s;
    return s;
}

// Lanes of a column slice (log2) and, in place, the slices of K and of V, for rows moved
// in units of `unit` bytes.
struct Slices {
    int uk, uv, w_shift, nk, parts;
};
Slices slices_of(const EvictArgs &a, int unit) {
    Slices c{};
    c.uk = (int)((int64_t)a.d * a.elem / unit);
    c.uv = (int)((int64_t)a.dv * a.elem / unit);
    while (c.w_shift < 4 && (1 << c.w_shift) < std::max(c.uk, c.uv)) ++c.w_shift;
    const int w = 1 << c.w_shift;
    c.nk = (c.uk + w - 1) / w;
    c.parts = c.nk + (c.uv + w - 1) / w;
    return c;
}

// Bytes of a row that move at a time.
int move_unit(const EvictArgs &a) {
    const int64_t kb = (int64_t)a.d * a.elem, vb = (int64_t)a.dv * a.elem;
    const uintptr_t bases = reinterpret_cast<uintptr_t>(a.k_cache) | reinterpret_cast<uintptr_t>(a.v_cache);
    return kb % 16 == 0 && vb % 16 == 0 && bases % 16 == 0 ? 16 : a.elem;
}

template <typename U> cudaError_t launch_move(const EvictArgs &a, bool in_place, int longest, cudaStream_t st) {
    const Slices c = slices_of(a, (int)sizeof(U));
    const int64_t pairs = (int64_t)a.src.sequences * a.hkv;
    int64_t parts = c.parts;
    if (!in_place) {
        parts = (longest + kMoveRanks - 1) / kMoveRanks;
        if (parts < 1) parts = 1;
        if (parts * pairs > INT32_MAX) parts = INT32_MAX / pairs;
    }
    const dim3 grid((unsigned)(pairs * parts)), block(kMoveThreads);
    const int sh = ps_shift_of(a.src.page_size);
    return in_place
               ? launch_pdl(move_kernel<U, true>, grid, block, 0, st, a, sh, c.uk, c.uv, c.w_shift, c.nk, (int)parts)
               : launch_pdl(move_kernel<U, false>, grid, block, 0, st, a, sh, c.uk, c.uv, c.w_shift, 0, (int)parts);
}

// Fours of keys a CTA holds in shared memory at most (half of an SM's; the CTAs of
// clusters have an SM each).
constexpr int kStagedFours = 6144, kClusterStagedFours = 12288;
// What the CTA of a cluster asks for at least: more than half of an SM's shared memory.
constexpr size_t kAlone = 120 * 1024;

cudaLaunchConfig_t cluster_config(cudaLaunchAttribute (&attr)[2], unsigned grid, int cluster, size_t smem) {
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)cluster;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(cluster > 1 ? 1024 : 512);
    cfg.dynamicSmemBytes = smem;
    cfg.attrs = attr;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
    return cfg;
}

// Clusters of a size that the current device runs at once, an SM a CTA: fewer than
// its SMs over the size, since a cluster stays in one group of SMs and the groups'
// sizes differ (of eight CTAs a GB300 holds 15, not 19).  0 when unknown.
int clusters_at_once(int cluster) {
    static PerDevice known[kMaxCluster + 1];
    int n = 0;
    const cudaError_t e = known[cluster].get(n, [&](int, int &v) {
        cudaLaunchAttribute attr[2];
        const cudaLaunchConfig_t cfg = cluster_config(attr, (unsigned)cluster, cluster, kAlone);
        const cudaError_t set = cudaFuncSetAttribute(select_kernel<true>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                     (int)(kClusterStagedFours * sizeof(uint4)));
        return set == cudaSuccess ? cudaOccupancyMaxActiveClusters(&v, select_kernel<true>, &cfg) : set;
    });
    if (e == cudaSuccess) return n;
    cudaGetLastError();
    return 0;
}

// Fours of keys a CTA of `cluster` stages, whatever the sink's alignment; 0: more than
// it holds, they are re-read.
int staged_fours(int cluster, int longest) {
    const int span = (longest / 4 + 2 + cluster - 1) / cluster;
    return span <= (cluster > 1 ? kClusterStagedFours : kStagedFours) ? span : 0;
}

// CTAs per (sequence, head).  A round of clusters of c takes about 10 + c + 0.8 k / c
// microseconds for k thousand keys (barriers, then the passes over a CTA's part), a
// lone CTA 10 + 1.1 k and about twice the passes where its keys do not fit; the
// rounds are what decides, so that more CTAs to a list are no gain once they cost one.
// Measured, microseconds by cluster size 1, 2, 4, 6, 8:
//   16 lists of 131K keys   -, -, 39, 34, 50      32 lists of 32K   73, 21, 19, 37, 55
//   64 lists of 16K        28, 19, 33, 53, 88     128 lists of 16K  28, 34, 59, 95, 158
// No part is below 2048 keys.
int select_ctas(int64_t pairs, int longest) {
    int best_c = 1;
    double best = 0.;
    for (int c = 1; c <= (int)kMaxCluster && (c == 1 || longest / c >= 2048); ++c) {
        const int room = staged_fours(c, longest);
        const double k = 1e-3 * longest * (room ? 1. : 2.);
        double rounds, each;
        if (c == 1) {
            const int per_sm = std::min(3, 227 * 1024 / (room * 16 + 9 * 1024));
            rounds = std::max(1., (double)pairs / (152 * per_sm));
            each = 10. + 1.1 * k;
        } else {
            const int at_once = clusters_at_once(c);
            if (!at_once) continue;
            rounds = (double)((pairs + at_once - 1) / at_once);
            each = 10. + c + 0.8 * k / c;
        }
        if (c == 1 || rounds * each < best) {
            best = rounds * each;
            best_c = c;
        }
    }
    return best_c;
}

cudaError_t launch_select(const EvictArgs &a, int cluster, int room, cudaStream_t st) {
    size_t smem = (size_t)room * sizeof(uint4);
    if (cluster > 1 && smem < kAlone) smem = kAlone;
    auto kernel = cluster > 1 ? select_kernel<true> : select_kernel<false>;
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         (int)((cluster > 1 ? kClusterStagedFours : kStagedFours) * sizeof(uint4)));
    if (e != cudaSuccess) return e;
    cudaLaunchAttribute attr[2];
    cudaLaunchConfig_t cfg = cluster_config(attr, (unsigned)(a.src.sequences * a.hkv * cluster), cluster, smem);
    cfg.stream = st;
    const int quads = a.src.page_size % 4 == 0 && reinterpret_cast<uintptr_t>(a.key_mass) % 16 == 0;
    return cudaLaunchKernelEx(&cfg, kernel, a, ps_shift_of(a.src.page_size), room, quads);
}

}  // namespace

bool evict_fits_grid(const EvictArgs &a, bool in_place) {
    const int64_t pairs = (int64_t)a.src.sequences * a.hkv;
    return pairs <= INT32_MAX / (int)kMaxCluster && (!in_place || pairs * slices_of(a, move_unit(a)).parts <= INT32_MAX);
}

cudaError_t launch_evict(const EvictArgs &a, int longest, int longest_kept, bool in_place, cudaStream_t st) {
    const int cluster = select_ctas((int64_t)a.src.sequences * a.hkv, longest);
    cudaError_t e = launch_select(a, cluster, staged_fours(cluster, longest), st);
    if (e != cudaSuccess) return e;
    switch (move_unit(a)) {
        case 16: e = launch_move<uint4>(a, in_place, longest_kept, st); break;
        case 4: e = launch_move<uint32_t>(a, in_place, longest_kept, st); break;
        default: e = launch_move<uint16_t>(a, in_place, longest_kept, st); break;
    }
    if (e != cudaSuccess) return e;
    return cudaGetLastError();
}

}  // namespace pa
