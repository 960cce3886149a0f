// Eviction from a paged cache by accumulated attention weight.
//
// Per (sequence, KV head) with n keys and a budget of `keep` of them: the first
// `sink` and the last `recent` keys stay, and of the others the keep - sink -
// recent with the largest totals (equal totals: the lower index stays; a NaN
// total counts below every number).  The kept keys move, in cache order, to the
// rows 0 .. keep-1 of the destination schedule: its pages are the sequence's own
// ones or fresh ones.
//
// Two kernels.  `select_kernel` finds the keep-th largest total by radix
// selection over order-preserving 32-bit keys and writes the kept indices in
// ascending order.  `move_kernel` moves the rows; in place that is safe without
// any ordering between CTAs: a CTA owns a column slice of one (sequence, head)
// and walks the ranks upwards, rank i reads row src(i) >= i and writes row i, so
// what a chunk of ranks writes has been read by this or an earlier chunk, and a
// barrier between the reads and the writes of a chunk is all it takes.

#include "pa_internal.h"

namespace pa {
namespace {

// Physical row of key j of sequence s, -1 when the table maps none.
__device__ __forceinline__ int64_t slot_of(const PlanView &p, int s, int j) {
    const int g = j / p.page_size;
    if (g >= p.width) return -1;
    const int pg = p.table[(int64_t)s * p.width + g];
    return pg < 0 || pg >= p.pages ? -1 : (int64_t)pg * p.page_size + (j - g * p.page_size);
}

__device__ __forceinline__ int64_t mass_at(int64_t slot, int h, int hkv, int ps) {
    const int64_t pg = slot / ps;
    return (pg * hkv + h) * ps + (slot - pg * ps);
}

// Keys whose unsigned order is the order of the totals: NaN lowest, -0 = +0.
__device__ __forceinline__ uint32_t order_key(float x) {
    if (x != x) return 0u;
    const uint32_t u = __float_as_uint(x == 0.f ? 0.f : x);
    return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

struct Budget {
    int n, keep, first, last, want;   // candidates [first, last), `want` of them stay
};

__device__ __forceinline__ Budget budget_of(const EvictArgs &a, int s) {
    Budget b;
    b.n = a.src.seq_lens[s];
    b.keep = min(min(a.dst.seq_lens[s], b.n), a.kept_stride);
    b.first = min(a.sink, b.keep);
    const int r = min(a.recent, b.keep - b.first);
    b.last = b.n - r;
    b.want = b.keep - b.first - r;
    return b;
}

constexpr int kSelectThreads = 1024;

__global__ void __launch_bounds__(kSelectThreads) select_kernel(EvictArgs a) {
    griddep_wait();
    griddep_launch();
    __shared__ int hist[256];
    __shared__ uint32_t s_prefix;
    __shared__ int s_need;
    __shared__ int warp_gt[32], warp_eq[32];
    const int h = blockIdx.x % a.hkv, s = blockIdx.x / a.hkv;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const Budget b = budget_of(a, s);
    int32_t *kept = a.kept + ((int64_t)s * a.hkv + h) * a.kept_stride;
    for (int i = b.keep + tid; i < a.kept_stride; i += kSelectThreads) kept[i] = -1;
    if (b.keep == b.n) {
        for (int i = tid; i < b.keep; i += kSelectThreads) kept[i] = i;
        return;
    }
    for (int i = tid; i < b.first; i += kSelectThreads) kept[i] = i;
    for (int i = tid; i < b.n - b.last; i += kSelectThreads) kept[b.first + b.want + i] = b.last + i;
    if (b.want == 0) return;
    auto key = [&](int j) -> uint32_t {
        const int64_t slot = slot_of(a.src, s, j);
        if (slot < 0) {
            atomicCAS(a.status, 0, PA_DEVICE_RANGE);
            return 0u;
        }
        return order_key(a.key_mass[mass_at(slot, h, a.hkv, a.src.page_size)]);
    };
    // the want-th largest key, eight bits a pass
    uint32_t prefix = 0u, mask = 0u;
    int need = b.want;
    for (int shift = 24; shift >= 0; shift -= 8) {
        for (int i = tid; i < 256; i += kSelectThreads) hist[i] = 0;
        __syncthreads();
        for (int j = b.first + tid; j < b.last; j += kSelectThreads) {
            const uint32_t k = key(j);
            if ((k & mask) == prefix) atomicAdd(&hist[(k >> shift) & 255u], 1);
        }
        __syncthreads();
        if (tid == 0) {
            int d = 255, above = 0;
            while (d > 0 && above + hist[d] < need) above += hist[d--];
            s_prefix = prefix | ((uint32_t)d << shift);
            s_need = need - above;
        }
        __syncthreads();
        prefix = s_prefix;
        need = s_need;
        mask |= 255u << shift;
        __syncthreads();
    }
    // every key above the threshold and the first `need` equal to it, in order
    int gt0 = 0, eq0 = 0;
    for (int base = b.first; base < b.last; base += kSelectThreads) {
        const int j = base + tid;
        const uint32_t k = j < b.last ? key(j) : 0u;
        const bool gt = j < b.last && k > prefix, eq = j < b.last && k == prefix;
        const unsigned bg = __ballot_sync(0xffffffffu, gt), be = __ballot_sync(0xffffffffu, eq);
        if (lane == 0) {
            warp_gt[warp] = __popc(bg);
            warp_eq[warp] = __popc(be);
        }
        __syncthreads();
        int g = gt0, e = eq0, gs = 0, es = 0;
        for (int w = 0; w < kSelectThreads / 32; ++w) {
            if (w == warp) {
                g += gs;
                e += es;
            }
            gs += warp_gt[w];
            es += warp_eq[w];
        }
        gt0 += gs;
        eq0 += es;
        const unsigned below = (1u << lane) - 1u;
        g += __popc(bg & below);
        e += __popc(be & below);
        if (gt || (eq && e < need)) kept[b.first + g + min(e, need)] = j;
        __syncthreads();
    }
}

constexpr int kMoveThreads = 256, kMoveUnroll = 8;

// One CTA: a slice of `w` units of the rows of one (sequence, head), of K, of V
// or the totals.
template <typename U> __device__ __forceinline__ void move_slice(const EvictArgs &a, U *cache, int units, int c0, int w,
                                                                 int s, int h, bool totals) {
    const int lane = threadIdx.x % w, sub = threadIdx.x / w, per = kMoveThreads / w;
    const Budget b = budget_of(a, s);
    const int32_t *kept = a.kept + ((int64_t)s * a.hkv + h) * a.kept_stride;
    const int c = c0 + lane;
    const bool col = c < units;
    const int ps = a.src.page_size;
    for (int base = 0; base < b.keep; base += per * kMoveUnroll) {
        U v[kMoveUnroll];
        int64_t to[kMoveUnroll];
#pragma unroll
        for (int u = 0; u < kMoveUnroll; ++u) {
            const int i = base + u * per + sub;
            to[u] = -1;
            if (i < b.keep && col) {
                const int64_t from = slot_of(a.src, s, kept[i]), dst = slot_of(a.dst, s, i);
                if (from < 0 || dst < 0) {
                    atomicCAS(a.status, 0, PA_DEVICE_RANGE);
                } else if (from != dst) {
                    v[u] = cache[totals ? mass_at(from, h, a.hkv, ps) : (from * a.hkv + h) * units + c];
                    to[u] = totals ? mass_at(dst, h, a.hkv, ps) : (dst * a.hkv + h) * units + c;
                }
            }
        }
        __syncthreads();       // every read of this chunk before any write of it
#pragma unroll
        for (int u = 0; u < kMoveUnroll; ++u)
            if (to[u] >= 0) cache[to[u]] = v[u];
    }
}

template <typename U>
__global__ void __launch_bounds__(kMoveThreads) move_kernel(EvictArgs a, int uk, int uv, int w, int nk, int nv) {
    griddep_wait();
    griddep_launch();
    const int parts = nk + nv + 1;
    const int part = blockIdx.x % parts;
    const int64_t sh = blockIdx.x / parts;
    const int h = (int)(sh % a.hkv), s = (int)(sh / a.hkv);
    if (part < nk)
        move_slice<U>(a, static_cast<U *>(a.k_cache), uk, part * w, w, s, h, false);
    else if (part < nk + nv)
        move_slice<U>(a, static_cast<U *>(a.v_cache), uv, (part - nk) * w, w, s, h, false);
    else
        move_slice<float>(a, a.key_mass, 1, 0, 1, s, h, true);
}

template <typename U> cudaError_t launch_move(const EvictArgs &a, cudaStream_t st) {
    const int uk = (int)((int64_t)a.d * a.elem / sizeof(U)), uv = (int)((int64_t)a.dv * a.elem / sizeof(U));
    int w = 1;
    while (w < 16 && w < (uk > uv ? uk : uv)) w *= 2;
    const int nk = (uk + w - 1) / w, nv = (uv + w - 1) / w;
    const int64_t blocks = (int64_t)a.src.sequences * a.hkv * (nk + nv + 1);
    if (blocks > INT32_MAX) return cudaErrorInvalidValue;
    return launch_pdl(move_kernel<U>, dim3((unsigned)blocks), dim3(kMoveThreads), 0, st, a, uk, uv, w, nk, nv);
}

}  // namespace

cudaError_t launch_evict(const EvictArgs &a, cudaStream_t st) {
    const int64_t blocks = (int64_t)a.src.sequences * a.hkv;
    if (blocks > INT32_MAX) return cudaErrorInvalidValue;
    cudaError_t e = launch_pdl(select_kernel, dim3((unsigned)blocks), dim3(kSelectThreads), 0, st, a);
    if (e != cudaSuccess) return e;
    auto al = [](const void *p, int n) { return (reinterpret_cast<uintptr_t>(p) % n) == 0; };
    const int64_t kb = (int64_t)a.d * a.elem, vb = (int64_t)a.dv * a.elem;
    if (kb % 16 == 0 && vb % 16 == 0 && al(a.k_cache, 16) && al(a.v_cache, 16))
        e = launch_move<uint4>(a, st);
    else if (a.elem == 4)
        e = launch_move<uint32_t>(a, st);
    else
        e = launch_move<uint16_t>(a, st);
    if (e != cudaSuccess) return e;
    return cudaGetLastError();
}

}  // namespace pa
