// Merge of split partials, for the merge kernels and for the kernel that also
// adds up the per-key totals.  Blocks of 256 threads.
//
// out = sum_s w_s o_s / sum_s w_s with w_s = exp(lse_s - max_s lse_s); empty
// splits (lse = -inf) weigh 0.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "pa_internal.h"

namespace pa {

template <typename T> __device__ __forceinline__ T from_float(float x);
template <> __device__ __forceinline__ float from_float<float>(float x) { return x; }
template <> __device__ __forceinline__ __half from_float<__half>(float x) { return __float2half_rn(x); }
template <> __device__ __forceinline__ __nv_bfloat16 from_float<__nv_bfloat16>(float x) { return __float2bfloat16_rn(x); }

// One warp per (query, head) row, eight rows per 256-thread block.  Every
// lane derives the split weights e^(lse_s - M) itself (M = max over splits,
// empty splits weigh 0) and holds VEC consecutive value columns of each
// 32*VEC-column chunk, read as one vector per split.
template <typename T, int VEC> struct OutVec;
template <typename T> struct OutVec<T, 1> {
    static __device__ __forceinline__ void store(T *p, const float *v) { p[0] = from_float<T>(v[0]); }
};
template <typename T> struct OutVec<T, 2> {
    static __device__ __forceinline__ void store(T *p, const float *v) {
        p[0] = from_float<T>(v[0]);
        p[1] = from_float<T>(v[1]);
    }
};
template <> struct OutVec<float, 4> {
    static __device__ __forceinline__ void store(float *p, const float *v) {
        *reinterpret_cast<float4 *>(p) = make_float4(v[0], v[1], v[2], v[3]);
    }
};
template <typename T> struct OutVec<T, 4> {
    static __device__ __forceinline__ void store(T *p, const float *v) {
        union { T h[4]; uint2 u; } x;
#pragma unroll
        for (int i = 0; i < 4; ++i) x.h[i] = from_float<T>(v[i]);
        *reinterpret_cast<uint2 *>(p) = x.u;
    }
};

template <int VEC> __device__ __forceinline__ void load_vec(const float *p, float *v) {
    if constexpr (VEC == 4) {
        const float4 x = *reinterpret_cast<const float4 *>(p);
        v[0] = x.x; v[1] = x.y; v[2] = x.z; v[3] = x.w;
    } else if constexpr (VEC == 2) {
        const float2 x = *reinterpret_cast<const float2 *>(p);
        v[0] = x.x; v[1] = x.y;
    } else {
        v[0] = p[0];
    }
}

template <typename T, int VEC>
__device__ __forceinline__ void merge_rows(const AttnArgs &a, int use_list, int nrows, int block) {
    const int wid = (int)((block * 256 + threadIdx.x) >> 5);
    const int lane = threadIdx.x & 31;
    if (wid >= nrows) return;
    const int item = wid / a.hq, h = wid - item * a.hq;
    const int qi = use_list ? a.plan.decode[item] : item;
    const int S = a.splits;
    const int64_t rows = (int64_t)a.plan.queries * a.hq;
    const int64_t row = (int64_t)qi * a.hq + h;
    // lane l holds the weights of splits l and l + 32 (at most PA_MAX_SPLITS = 64)
    float m = -INFINITY;
    for (int s = lane; s < S; s += 32) m = fmaxf(m, a.ws_lse[s * rows + row]);
    for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    float wl[2];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        const int s = lane + 32 * k;
        const float l = s < S ? a.ws_lse[s * rows + row] : -INFINITY;
        wl[k] = l == -INFINITY ? 0.f : __expf(l - m);
    }
    float tot = wl[0] + wl[1];
    for (int o = 16; o; o >>= 1) tot += __shfl_xor_sync(0xffffffffu, tot, o);
    const float inv = 1.f / tot;
    T *out = static_cast<T *>(a.out) + row * a.dv;
    // every lane runs every chunk (the weights are shuffled in the loop); a lane
    // past the last column reads column 0 and stores nothing
    for (int c0 = 0; c0 < a.dv; c0 += 32 * VEC) {
        const bool live = c0 + lane * VEC < a.dv;
        const int c = live ? c0 + lane * VEC : 0;
        float acc[VEC];
#pragma unroll
        for (int i = 0; i < VEC; ++i) acc[i] = 0.f;
        // no branch on empty splits (their weight is 0 and their partial 0), so the
        // loads of several splits are in flight at once
#pragma unroll 8
        for (int s = 0; s < S; ++s) {
            const float ws = __shfl_sync(0xffffffffu, s < 32 ? wl[0] : wl[1], s & 31);
            float v[VEC];
            load_vec<VEC>(a.ws_o + (s * rows + row) * a.dv + c, v);
#pragma unroll
            for (int i = 0; i < VEC; ++i) acc[i] += ws * v[i];
        }
#pragma unroll
        for (int i = 0; i < VEC; ++i) acc[i] *= inv;
        if (live) OutVec<T, VEC>::store(out + c, acc);
    }
}

// Few rows or many splits: one 8-warp block per (query, head) row, warp w
// taking splits w, w + 8, ...; the eight partial sums meet in shared memory.
// Rows spread over every SM and all splits of a row are in flight at once,
// where one warp per row would walk its splits one after another.
template <typename T, int VEC>
__device__ __forceinline__ void merge_row_wide(const AttnArgs &a, int use_list, unsigned block, float *part) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;   // part: [8][dv]
    const int item = block / a.hq, h = block - item * a.hq;
    const int qi = use_list ? a.plan.decode[item] : item;
    const int S = a.splits;
    const int64_t rows = (int64_t)a.plan.queries * a.hq;
    const int64_t row = (int64_t)qi * a.hq + h;
    float m = -INFINITY;
    for (int s = lane; s < S; s += 32) m = fmaxf(m, a.ws_lse[s * rows + row]);
    for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    float wl[2];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        const int s = lane + 32 * k;
        const float l = s < S ? a.ws_lse[s * rows + row] : -INFINITY;
        wl[k] = l == -INFINITY ? 0.f : __expf(l - m);
    }
    float tot = wl[0] + wl[1];
    for (int o = 16; o; o >>= 1) tot += __shfl_xor_sync(0xffffffffu, tot, o);
    for (int c0 = 0; c0 < a.dv; c0 += 32 * VEC) {
        const bool live = c0 + lane * VEC < a.dv;
        const int c = live ? c0 + lane * VEC : 0;
        float acc[VEC];
#pragma unroll
        for (int i = 0; i < VEC; ++i) acc[i] = 0.f;
#pragma unroll 4
        for (int s = warp; s < S; s += 8) {
            const float ws = __shfl_sync(0xffffffffu, s < 32 ? wl[0] : wl[1], s & 31);
            float v[VEC];
            load_vec<VEC>(a.ws_o + (s * rows + row) * a.dv + c, v);
#pragma unroll
            for (int i = 0; i < VEC; ++i) acc[i] += ws * v[i];
        }
        if (live) {
#pragma unroll
            for (int i = 0; i < VEC; ++i) part[warp * a.dv + c + i] = acc[i];
        }
    }
    __syncthreads();
    const float inv = 1.f / tot;
    T *out = static_cast<T *>(a.out) + row * a.dv;
    for (int c = threadIdx.x; c < a.dv; c += 256) {
        float x = 0.f;
#pragma unroll
        for (int w = 0; w < 8; ++w) x += part[w * a.dv + c];
        out[c] = from_float<T>(x * inv);
    }
}

// Few rows or long split chains: a block per row.  Else eight rows a block.
inline bool merge_is_wide(const AttnArgs &a, int nrows) { return nrows < 1024 || a.splits >= 16; }

// Columns a lane handles at a time: the workspace is 16-byte aligned and rows are
// dv floats apart; the output takes 4-wide stores only when its base allows them.
inline int merge_vec(const AttnArgs &a) {
    const uintptr_t ob = reinterpret_cast<uintptr_t>(a.out);
    const uintptr_t esz = a.dtype == PA_F32 ? 4 : 2;
    return a.dv % 4 == 0 && ob % (4 * esz) == 0 ? 4 : (a.dv % 2 == 0 ? 2 : 1);
}

}  // namespace pa
