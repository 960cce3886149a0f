// The 8-bit cache's append (paged_kv_store_q8) and its read-back into a paged cache
// of wider elements (paged_kv_load_q8).
//
// Both move rows and are bound by HBM: an append reads each new row once and writes
// D + 1 bytes, a read-back reads D + 1 bytes and writes the row.  The append needs a
// row's maximum before its first element can be written; a group of lanes holds the
// row in registers meanwhile, 16 elements a lane, so that a lane writes 16 bytes.

#include <climits>
#include <type_traits>

#include "per_device.h"
#include "q8_format.cuh"

namespace pa {
namespace {

using namespace q8;

constexpr int kThreads = 256;

// Maximum over the aligned groups of `lanes` lanes (a power of two).
__device__ __forceinline__ uint32_t group_max(uint32_t v, int lanes) {
    for (int o = lanes >> 1; o; o >>= 1) v = max(v, __shfl_xor_sync(0xffffffffu, v, o));
    return v;
}

struct NewRow {
    const void *src;
    uint8_t *dst, *scale;
    int dim;
};

// The key or value row of (token, head), given the token's slot.
template <typename T>
__device__ __forceinline__ NewRow new_row(const Q8StoreArgs &a, bool value, uint32_t token, uint32_t h, uint32_t slot) {
    const uint32_t ps = a.plan.page_size, page = slot / ps;
    NewRow r;
    r.dim = value ? a.dv : a.d;
    r.src = static_cast<const T *>(value ? a.v : a.k) + (int64_t)token * (value ? a.v_stride : a.k_stride) + (int64_t)h * r.dim;
    r.dst = (value ? a.v_cache : a.k_cache) + ((int64_t)slot * a.hkv + h) * r.dim;
    r.scale = (value ? a.v_scale : a.k_scale) + ((int64_t)page * a.hkv + h) * ps + (slot - page * ps);
    return r;
}

// The fp32 bits of the largest |x| of 16 elements, or of NaN or infinity where one of them is:
// two elements an instruction (an append of finite rows issues a third of what element by
// element takes).
template <typename T> __device__ __forceinline__ uint32_t largest_bits(const uint4 *w);
template <> __device__ __forceinline__ uint32_t largest_bits<float>(const uint4 *w) {
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i)
        top = max(max(max(top, w[i].x & 0x7fffffffu), max(w[i].y & 0x7fffffffu, w[i].z & 0x7fffffffu)), w[i].w & 0x7fffffffu);
    return top;
}
template <typename P> __device__ __forceinline__ P largest_pair(const uint4 *w) {
    P m{};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const uint32_t u = (i % 4 == 0 ? w[i / 4].x : i % 4 == 1 ? w[i / 4].y : i % 4 == 2 ? w[i / 4].z : w[i / 4].w) & 0x7fff7fffu;
        m = __hmax2_nan(m, *reinterpret_cast<const P *>(&u));
    }
    return m;
}
template <> __device__ __forceinline__ uint32_t largest_bits<__nv_bfloat16>(const uint4 *w) {
    const __nv_bfloat162 m = largest_pair<__nv_bfloat162>(w);
    return max(__float_as_uint(__low2float(m)) & 0x7fffffffu, __float_as_uint(__high2float(m)) & 0x7fffffffu);
}
template <> __device__ __forceinline__ uint32_t largest_bits<__half>(const uint4 *w) {
    const __half2 m = largest_pair<__half2>(w);
    return max(__float_as_uint(__low2float(m)) & 0x7fffffffu, __float_as_uint(__high2float(m)) & 0x7fffffffu);
}

// Rows of a multiple of 16 elements, up to 16 * 32: `lanes` lanes for the key and the value
// row of one (token, head), both in flight at once (one row a lane took 25 us for 16384
// tokens of 8 heads of 128).
template <typename T>
__global__ void __launch_bounds__(kThreads) store_rows_kernel(Q8StoreArgs a, uint32_t rows, int lanes) {
    constexpr int kLoads = 16 * sizeof(T) / 16;
    griddep_wait();
    griddep_launch();
    const uint32_t l = threadIdx.x % lanes, idx0 = blockIdx.x * (kThreads / lanes) + threadIdx.x / lanes;
    const bool live = idx0 < rows;
    const uint32_t idx = live ? idx0 : 0u, token = idx / a.hkv, h = idx - token * a.hkv;
    const uint32_t slot = (uint32_t)a.plan.qmeta[token].z;
    union { uint4 w[kLoads]; T t[16]; } in[2];
    NewRow r[2];
    bool mine[2];
#pragma unroll
    for (int v = 0; v < 2; ++v) {
        r[v] = new_row<T>(a, v == 1, token, h, slot);
        mine[v] = live && (int)l * 16 < r[v].dim;
#pragma unroll
        for (int i = 0; i < kLoads; ++i)
            in[v].w[i] = mine[v] ? reinterpret_cast<const uint4 *>(static_cast<const T *>(r[v].src) + l * 16)[i] : make_uint4(0u, 0u, 0u, 0u);
    }
#pragma unroll
    for (int v = 0; v < 2; ++v) {
        // the largest |x| of all elements; where that is not finite, of the finite ones
        uint32_t top = largest_bits<T>(in[v].w);
        const bool finite = !__any_sync(0xffffffffu, top >= 0x7f800000u);
        if (!finite) {
            top = 0;
#pragma unroll
            for (int i = 0; i < 16; ++i) top = max(top, finite_bits(to_f32<T>(in[v].t[i])));
        }
        const uint32_t b = scale_byte(group_max(top, lanes));
        if (!mine[v]) continue;
        const float inv = power_of(254u - b);
        uint32_t out[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float x[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) x[e] = to_f32<T>(in[v].t[4 * i + e]);
            out[i] = finite ? pack2_finite(x[0], x[1], inv) | pack2_finite(x[2], x[3], inv) << 16
                            : pack2_e4m3(x[0], x[1], inv) | pack2_e4m3(x[2], x[3], inv) << 16;
        }
        *reinterpret_cast<uint4 *>(r[v].dst + l * 16) = make_uint4(out[0], out[1], out[2], out[3]);
        if (l == 0) *r[v].scale = (uint8_t)b;
    }
}

// Any row: a warp each, one element a lane, read twice (the second time from L1 or L2).
template <typename T>
__global__ void __launch_bounds__(kThreads) store_any_kernel(Q8StoreArgs a, int64_t rows) {
    griddep_wait();
    griddep_launch();
    const int lane = threadIdx.x & 31;
    for (int64_t idx = blockIdx.x * (int64_t)(kThreads / 32) + threadIdx.x / 32; idx < rows;
         idx += (int64_t)gridDim.x * (kThreads / 32)) {
        const uint32_t token = (uint32_t)(idx / (2 * a.hkv));
        uint32_t h = (uint32_t)(idx - (int64_t)token * (2 * a.hkv));
        const bool value = h >= (uint32_t)a.hkv;
        if (value) h -= a.hkv;
        const NewRow r = new_row<T>(a, value, token, h, (uint32_t)a.plan.qmeta[token].z);
        const T *src = static_cast<const T *>(r.src);
        uint32_t top = 0;
        for (int i = lane; i < r.dim; i += 32) top = max(top, finite_bits(to_f32<T>(src[i])));
        const uint32_t b = scale_byte(group_max(top, 32));
        const float inv = power_of(254u - b);
        for (int i = lane; i < r.dim; i += 32) r.dst[i] = (uint8_t)pack2_e4m3(to_f32<T>(src[i]), 0.f, inv);
        if (lane == 0) *r.scale = (uint8_t)b;
    }
}

bool aligned(const void *p, int n) { return (reinterpret_cast<uintptr_t>(p) % n) == 0; }

template <typename T> cudaError_t launch_store(const Q8StoreArgs &a, cudaStream_t st) {
    const int64_t rows = (int64_t)a.plan.queries * a.hkv;
    const int64_t es = sizeof(T);
    const int widest = a.d > a.dv ? a.d : a.dv;
    const bool wide = a.d % 16 == 0 && a.dv % 16 == 0 && widest <= 512 && aligned(a.k, 16) && aligned(a.v, 16) &&
                      aligned(a.k_cache, 16) && aligned(a.v_cache, 16) && a.k_stride * es % 16 == 0 && a.v_stride * es % 16 == 0;
    int64_t blocks;
    if (wide) {
        int lanes = 1;
        while (lanes * 16 < widest) lanes *= 2;
        blocks = (rows + kThreads / lanes - 1) / (kThreads / lanes);
        if (rows <= INT32_MAX)
            return launch_pdl(store_rows_kernel<T>, dim3((unsigned)blocks), dim3(kThreads), 0, st, a, (uint32_t)rows, lanes);
    }
    blocks = (2 * rows + kThreads / 32 - 1) / (kThreads / 32);
    if (blocks > 152 * 64) blocks = 152 * 64;
    return launch_pdl(store_any_kernel<T>, dim3((unsigned)blocks), dim3(kThreads), 0, st, a, 2 * rows);
}

// ---------------------------------------------------------------- read-back --

constexpr int kKeys = 64;      // keys a block takes at a time, at most

// Units of one tensor's rows: eight elements, or one where rows are no multiple of eight.
template <typename T, int E>
__device__ __forceinline__ void read_rows(const uint8_t *cache, const uint8_t *scale, T *to, int hkv, int dim, int ps,
                                          const int64_t *from_row, const int64_t *scale_at, const int64_t *to_row, int keys) {
    const int per_head = dim / E, per_key = hkv * per_head;
    const int across = per_key < kThreads ? per_key : kThreads;
    const int lanes = kThreads / across;               // keys side by side
    const int kl = (int)threadIdx.x / across;
    if (kl >= lanes) return;
    for (int u = (int)threadIdx.x - kl * across; u < per_key; u += across) {
        const int h = u / per_head;
#pragma unroll 2
        for (int k = kl; k < keys; k += lanes) {
            const uint32_t b = scale[scale_at[k] + (int64_t)h * ps];
            const float s = power_of(b);
            const uint8_t *src = cache + from_row[k] * hkv * dim + (int64_t)u * E;
            T *dst = to + to_row[k] * hkv * dim + (int64_t)u * E;
            if constexpr (E == 8) {
                const uint2 w = *reinterpret_cast<const uint2 *>(src);
                union { T t[8]; uint32_t u[8 * sizeof(T) / 4]; uint4 o[sizeof(T) / 2]; } x;
                if (std::is_same<T, __half>::value && in_half_range(b)) {
                    const __half2 m = half_power_of(b);
#pragma unroll
                    for (int i = 0; i < 4; ++i) x.u[i] = times_half((i < 2 ? w.x : w.y) >> (16 * (i & 1)), m);
                } else {
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float2 f = unpack2_e4m3((i < 2 ? w.x : w.y) >> (16 * (i & 1)));
                        x.t[2 * i] = read_back<T>(f.x * s);
                        x.t[2 * i + 1] = read_back<T>(f.y * s);
                    }
                }
#pragma unroll
                for (int i = 0; i < (int)sizeof(T) / 2; ++i) reinterpret_cast<uint4 *>(dst)[i] = x.o[i];
            } else {
                *dst = read_back<T>(unpack_e4m3(*src) * s);
            }
        }
    }
}

// Eight blocks an SM hide the loads: 291 us for the batch of 64 histories (6.1 TB/s, 90 % of
// the copy rate), 350 with five blocks and twice the loads in flight in each.
template <typename T, int E>
__global__ void __launch_bounds__(kThreads, 8) load_kernel(Q8LoadArgs a, int block_keys) {
    __shared__ int64_t from_row[kKeys], scale_at[kKeys], to_row[kKeys];
    griddep_wait();
    griddep_launch();
    const int ps = a.plan.page_size;
    for (int s = blockIdx.y; s < a.plan.sequences; s += gridDim.y) {
        int n = a.plan.seq_lens[s];
        int2 place = make_int2(0, 0);
        if (a.places) {
            place = a.places[s];
            if (place.x == kQ8NoTiles) continue;
        } else {
            const int m = a.to_lens[s];
            if (m > n && blockIdx.x == 0 && threadIdx.x == 0) atomicCAS(a.status, 0, PA_DEVICE_RANGE);
            n = m < n ? m : n;
        }
        const int32_t *row = a.plan.table + (int64_t)s * a.plan.width;
        for (int64_t j0 = (int64_t)place.y * a.to_page_size + (int64_t)blockIdx.x * block_keys; j0 < n; j0 += (int64_t)gridDim.x * block_keys) {
            const int keys = n - j0 < block_keys ? (int)(n - j0) : block_keys;
            __syncthreads();               // the rows of the round before are read
            if ((int)threadIdx.x < keys) {
                const int j = (int)j0 + threadIdx.x;
                const int g = j / ps, r = j - g * ps;
                const int64_t page = row[g];
                from_row[threadIdx.x] = page * ps + r;
                scale_at[threadIdx.x] = page * a.hkv * ps + r;
                const int tg = j / a.to_page_size, tr = j - tg * a.to_page_size;
                int32_t to;
                if (a.places) {
                    // without room for the sequence nothing is written and its table names the first page
                    to = place.x == kQ8NoRoom ? 0 : place.x + (tg - place.y);
                    if (tr == 0 || j == (int)j0) a.to_table_out[(int64_t)s * a.to_width + tg] = to;
                } else {
                    to = a.to_table[(int64_t)s * a.to_width + tg];
                }
                to_row[threadIdx.x] = (int64_t)to * a.to_page_size + tr;
            }
            __syncthreads();
            if (place.x == kQ8NoRoom) continue;
            read_rows<T, E>(a.k, a.k_scale, static_cast<T *>(a.k_to), a.hkv, a.d, ps, from_row, scale_at, to_row, keys);
            read_rows<T, E>(a.v, a.v_scale, static_cast<T *>(a.v_to), a.hkv, a.dv, ps, from_row, scale_at, to_row, keys);
        }
    }
}

// Place of every sequence with prefill tiles in a run of pages that holds what their queries see:
// one block, sequences in their order.  (The places are read around L1, which the atomics pass.)
__global__ void __launch_bounds__(1024) places_kernel(PlanView plan, int2 *places, int32_t window, int32_t page_size, int32_t room,
                                                      int32_t *status) {
    __shared__ int32_t warp_sum[32];
    griddep_wait();
    griddep_launch();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    for (int s = tid; s < plan.sequences; s += 1024) places[s].y = INT_MAX;
    __syncthreads();
    for (int t = tid; t < plan.n_tiles; t += 1024) atomicMin(&places[plan.tiles[t].x].y, plan.tiles[t].w);
    __syncthreads();
    int64_t before = 0;
    for (int s0 = 0; s0 < plan.sequences; s0 += 1024) {
        const int s = s0 + tid;
        const int lowest = s < plan.sequences ? __ldcg(&places[s].y) : INT_MAX;
        const bool tiles = lowest != INT_MAX;
        const int first = tiles && window > 0 && lowest >= window ? (lowest - window + 1) / page_size : 0;
        const int pages = tiles ? (int)(((int64_t)plan.seq_lens[s] + page_size - 1) / page_size) - first : 0;
        int sum = pages;
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, sum, o);
            if (lane >= o) sum += y;
        }
        if (lane == 31) warp_sum[warp] = sum;
        __syncthreads();
        int64_t at = before, all = 0;
        for (int w = 0; w < 32; ++w) {
            if (w < warp) at += warp_sum[w];
            all += warp_sum[w];
        }
        at += sum - pages;
        if (s < plan.sequences) {
            const bool fits = at + pages <= room;
            places[s] = make_int2(!tiles ? kQ8NoTiles : fits ? (int32_t)at : kQ8NoRoom, first);
            if (tiles && !fits) atomicCAS(status, 0, PA_DEVICE_RANGE);
        }
        before += all;
        __syncthreads();
    }
}

template <typename T> cudaError_t launch_load_t(const Q8LoadArgs &a, int longest, cudaStream_t st) {
    const bool wide = a.d % 8 == 0 && a.dv % 8 == 0 && aligned(a.k, 8) && aligned(a.v, 8) && aligned(a.k_to, 16) && aligned(a.v_to, 16);
    // Blocks of 64 keys, or of 32 or 16 where those would be few: 152 * 8 are resident at once, and
    // with unequal histories the last round shows until there are four (16 histories to 12K keys, 8
    // heads of 128: 109 us in blocks of 32, 121 of 64; a mixed step's eight chunks 32 us in blocks
    // of 16, 41 of 64).  Rows of under 512 bytes make blocks whose start is most of their time; two
    // rounds suffice there (64 histories to 2760, one head of 80: 16 us of 64, 20 of 32).
    const int64_t all = (int64_t)a.plan.sequences * longest, want = (int64_t)152 * 8 * (a.hkv * (a.d + a.dv) >= 512 ? 4 : 2);
    const int keys = all >= want * 64 ? 64 : all >= want * 32 ? 32 : 16;
    int64_t x = ((int64_t)longest + keys - 1) / keys;
    if (x < 1) x = 1;
    if (x > 65535) x = 65535;
    const int y = a.plan.sequences < 65535 ? a.plan.sequences : 65535;
    const dim3 grid((unsigned)x, (unsigned)y);
    return wide ? launch_pdl(load_kernel<T, 8>, grid, dim3(kThreads), 0, st, a, keys)
                : launch_pdl(load_kernel<T, 1>, grid, dim3(kThreads), 0, st, a, keys);
}

}  // namespace

cudaError_t launch_q8_store(const Q8StoreArgs &a, cudaStream_t st) {
    switch (a.dtype) {
        case PA_F32: return launch_store<float>(a, st);
        case PA_F16: return launch_store<__half>(a, st);
        default: return launch_store<__nv_bfloat16>(a, st);
    }
}

cudaError_t launch_q8_load(const Q8LoadArgs &a, int longest, cudaStream_t st) {
    switch (a.dtype) {
        case PA_F32: return launch_load_t<float>(a, longest, st);
        case PA_F16: return launch_load_t<__half>(a, longest, st);
        default: return launch_load_t<__nv_bfloat16>(a, longest, st);
    }
}

cudaError_t launch_q8_places(const PlanView &plan, int2 *places, int32_t window, int32_t page_size, int32_t room, int32_t *status,
                             cudaStream_t st) {
    return launch_pdl(places_kernel, dim3(1), dim3(1024), 0, st, plan, places, window, page_size, room, status);
}

}  // namespace pa
