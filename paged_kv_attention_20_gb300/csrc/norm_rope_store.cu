// Per-head RMS norm of queries and keys, position rotation and cache append in
// one pass over the step's new rows.
//
// For every head row x of Q and of the new K (D elements, fp32 arithmetic):
//   y = x / sqrt(mean(x^2) + eps) * w                  (no w: y = x)
// and for the first `rot` dims the pairs (a, b) = (y_i, y_{i + rot/2}), or
// (y_2i, y_2i+1) when interleaved, turn by their position's angle:
//   a' = a cos - b sin,   b' = b cos + a sin
// with cos_i | sin_i read from the row of the caller's table.  Q goes to a
// dense output, K and V rows (V unchanged) to the plan's cache slots, each
// element rounded once.  A key's accumulated attention weight starts at 0.
//
// The pass reads and writes each row once: it is bound by HBM for prompt
// chunks and by launch latency for single tokens.  A row is spread over
// L = D / (2 * 16 bytes) lanes, each holding two 16-byte chunks that contain
// whole pairs, so the rotation needs no exchange between lanes and the norm
// only log2(L) shuffles.

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "pa_internal.h"

namespace pa {
namespace {

constexpr int kThreads = 256;

template <typename T> __device__ __forceinline__ float to_f(T x);
template <> __device__ __forceinline__ float to_f<float>(float x) { return x; }
template <> __device__ __forceinline__ float to_f<__half>(__half x) { return __half2float(x); }
template <> __device__ __forceinline__ float to_f<__nv_bfloat16>(__nv_bfloat16 x) { return __bfloat162float(x); }

template <typename T> __device__ __forceinline__ T from_f(float x);
template <> __device__ __forceinline__ float from_f<float>(float x) { return x; }
template <> __device__ __forceinline__ __half from_f<__half>(float x) { return __float2half_rn(x); }
template <> __device__ __forceinline__ __nv_bfloat16 from_f<__nv_bfloat16>(float x) { return __float2bfloat16_rn(x); }

// 16 bytes of T as floats and back.
template <typename T> struct Chunk {
    static constexpr int V = 16 / sizeof(T);
    union U {
        uint4 u;
        T t[V];
    };
    static __device__ __forceinline__ void unpack(const uint4 &w, float (&f)[V]) {
        U x;
        x.u = w;
#pragma unroll
        for (int i = 0; i < V; ++i) f[i] = to_f<T>(x.t[i]);
    }
    static __device__ __forceinline__ uint4 pack(const float (&f)[V]) {
        U x;
#pragma unroll
        for (int i = 0; i < V; ++i) x.t[i] = from_f<T>(f[i]);
        return x.u;
    }
};

// Row r of a token: query heads, then key heads, then value heads.
struct RowId {
    int token, head, part;     // part 0: Q, 1: K, 2: V
};

__device__ __forceinline__ RowId row_id(const NormRopeArgs &a, int64_t idx) {
    const int per = a.hq + 2 * a.hkv;
    RowId r;
    r.token = (int)(idx / per);
    const int h = (int)(idx - (int64_t)r.token * per);
    r.part = h < a.hq ? 0 : (h < a.hq + a.hkv ? 1 : 2);
    r.head = h - (r.part == 0 ? 0 : (r.part == 1 ? a.hq : a.hq + a.hkv));
    return r;
}

// Position of a token, or -1 (recorded once per row) when the table has no row for it.
__device__ __forceinline__ int table_position(const NormRopeArgs &a, int token, int plan_pos) {
    const int pos = a.positions ? a.positions[token] : plan_pos;
    return a.table && (pos < 0 || pos >= a.max_positions) ? -1 : pos;
}

template <typename T, int L>
__global__ void __launch_bounds__(kThreads) norm_rope_kernel(NormRopeArgs a, int64_t rows) {
    constexpr int V = Chunk<T>::V;
    griddep_wait();
    griddep_launch();
    const int64_t idx = (int64_t)blockIdx.x * (kThreads / L) + threadIdx.x / L;
    const int l = threadIdx.x % L;
    const bool live = idx < rows;
    const RowId r = row_id(a, live ? idx : rows - 1);
    const int4 meta = a.plan.qmeta[r.token];
    const int pos = table_position(a, r.token, meta.y);
    const int64_t slot = meta.z;
    const bool ok = live && (pos >= 0 || !a.table);
    if (live && !ok && l == 0) atomicCAS(a.status, 0, PA_DEVICE_RANGE);
    if (r.part == 2) {
        // value rows: a copy
        if (!ok) return;
        const uint4 *src = reinterpret_cast<const uint4 *>(static_cast<const T *>(a.v) + (int64_t)r.token * a.v_stride +
                                                           (int64_t)r.head * a.dv);
        uint4 *dst = reinterpret_cast<uint4 *>(static_cast<T *>(a.v_cache) + (slot * a.hkv + r.head) * a.dv);
        for (int c = l; c < a.dv / V; c += L) dst[c] = src[c];
        return;
    }
    const T *src = r.part == 0 ? static_cast<const T *>(a.q) + (int64_t)r.token * a.q_stride
                               : static_cast<const T *>(a.k) + (int64_t)r.token * a.k_stride;
    src += (int64_t)r.head * a.d;
    const T *w = static_cast<const T *>(r.part == 0 ? a.q_weight : a.k_weight);
    // my two chunks: a pair of halves (or of neighbours) inside the rotated dims,
    // neighbours past them
    const int turned = a.rot / (2 * V);           // lanes that rotate
    const bool mine = l * 2 * V < a.d;
    int c0 = l * 2 * V, c1 = c0 + V;
    if (!a.interleaved && l < turned) {
        c0 = l * V;
        c1 = a.rot / 2 + l * V;
    }
    float x0[V], x1[V];
#pragma unroll
    for (int i = 0; i < V; ++i) x0[i] = x1[i] = 0.f;
    if (mine) {
        Chunk<T>::unpack(*reinterpret_cast<const uint4 *>(src + c0), x0);
        Chunk<T>::unpack(*reinterpret_cast<const uint4 *>(src + c1), x1);
    }
    if (w) {
        float ss = 0.f;
#pragma unroll
        for (int i = 0; i < V; ++i) ss += x0[i] * x0[i] + x1[i] * x1[i];
        // the lanes of a row sit in one aligned group of a warp; all 32 lanes are here
        // or have left as whole value rows, so the group's own mask is named
        const unsigned group = L == 32 ? 0xffffffffu : ((1u << (L & 31)) - 1u) << ((threadIdx.x & 31) / L * L);
#pragma unroll
        for (int o = L / 2; o; o >>= 1) ss += __shfl_xor_sync(group, ss, o);
        const float inv = rsqrtf(ss / (float)a.d + a.eps);
        if (mine) {
            float w0[V], w1[V];
            Chunk<T>::unpack(*reinterpret_cast<const uint4 *>(w + c0), w0);
            Chunk<T>::unpack(*reinterpret_cast<const uint4 *>(w + c1), w1);
#pragma unroll
            for (int i = 0; i < V; ++i) {
                x0[i] *= inv * w0[i];
                x1[i] *= inv * w1[i];
            }
        }
    }
    if (!ok || !mine) return;
    if (a.table && l < turned) {
        const float *cs = a.table + (int64_t)pos * a.rot + l * V;
        float c[V], s[V];
#pragma unroll
        for (int i = 0; i < V; i += 4) {
            const float4 cc = *reinterpret_cast<const float4 *>(cs + i);
            const float4 sn = *reinterpret_cast<const float4 *>(cs + a.rot / 2 + i);
            c[i] = cc.x; c[i + 1] = cc.y; c[i + 2] = cc.z; c[i + 3] = cc.w;
            s[i] = sn.x; s[i + 1] = sn.y; s[i + 2] = sn.z; s[i + 3] = sn.w;
        }
        if (a.interleaved) {
            // pairs (2i, 2i + 1) of my 2V consecutive elements
#pragma unroll
            for (int i = 0; i < V / 2; ++i) {
                const float p = x0[2 * i], q = x0[2 * i + 1];
                x0[2 * i] = p * c[i] - q * s[i];
                x0[2 * i + 1] = q * c[i] + p * s[i];
                const float u = x1[2 * i], v = x1[2 * i + 1];
                x1[2 * i] = u * c[V / 2 + i] - v * s[V / 2 + i];
                x1[2 * i + 1] = v * c[V / 2 + i] + u * s[V / 2 + i];
            }
        } else {
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const float p = x0[i], q = x1[i];
                x0[i] = p * c[i] - q * s[i];
                x1[i] = q * c[i] + p * s[i];
            }
        }
    }
    T *dst = r.part == 0 ? static_cast<T *>(a.q_out) + ((int64_t)r.token * a.hq + r.head) * a.d
                         : static_cast<T *>(a.k_cache) + (slot * a.hkv + r.head) * a.d;
    *reinterpret_cast<uint4 *>(dst + c0) = Chunk<T>::pack(x0);
    *reinterpret_cast<uint4 *>(dst + c1) = Chunk<T>::pack(x1);
    if (r.part == 1 && a.key_mass && l == 0) {
        const int ps = a.plan.page_size;
        a.key_mass[(slot / ps * a.hkv + r.head) * ps + slot % ps] = 0.f;
    }
}

// Any head dim, stride and alignment: one warp per row, one element per lane
// and step.
template <typename T>
__global__ void __launch_bounds__(kThreads) norm_rope_any_kernel(NormRopeArgs a, int64_t rows) {
    griddep_wait();
    griddep_launch();
    const int64_t idx = (int64_t)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
    const int lane = threadIdx.x & 31;
    if (idx >= rows) return;
    const RowId r = row_id(a, idx);
    const int4 meta = a.plan.qmeta[r.token];
    const int pos = table_position(a, r.token, meta.y);
    const int64_t slot = meta.z;
    if (a.table && pos < 0) {
        if (lane == 0) atomicCAS(a.status, 0, PA_DEVICE_RANGE);
        return;
    }
    if (r.part == 2) {
        const T *src = static_cast<const T *>(a.v) + (int64_t)r.token * a.v_stride + (int64_t)r.head * a.dv;
        T *dst = static_cast<T *>(a.v_cache) + (slot * a.hkv + r.head) * a.dv;
        for (int i = lane; i < a.dv; i += 32) dst[i] = src[i];
        return;
    }
    const T *src = r.part == 0 ? static_cast<const T *>(a.q) + (int64_t)r.token * a.q_stride
                               : static_cast<const T *>(a.k) + (int64_t)r.token * a.k_stride;
    src += (int64_t)r.head * a.d;
    T *dst = r.part == 0 ? static_cast<T *>(a.q_out) + ((int64_t)r.token * a.hq + r.head) * a.d
                         : static_cast<T *>(a.k_cache) + (slot * a.hkv + r.head) * a.d;
    const T *w = static_cast<const T *>(r.part == 0 ? a.q_weight : a.k_weight);
    float inv = 1.f;
    if (w) {
        float ss = 0.f;
        for (int i = lane; i < a.d; i += 32) {
            const float x = to_f<T>(src[i]);
            ss += x * x;
        }
        for (int o = 16; o; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
        inv = rsqrtf(ss / (float)a.d + a.eps);
    }
    auto normed = [&](int i) { return w ? to_f<T>(src[i]) * (inv * to_f<T>(w[i])) : to_f<T>(src[i]); };
    const int half = a.table ? a.rot / 2 : 0;
    const float *cs = a.table ? a.table + (int64_t)pos * a.rot : nullptr;
    for (int i = lane; i < half; i += 32) {
        const int ia = a.interleaved ? 2 * i : i, ib = a.interleaved ? 2 * i + 1 : i + half;
        const float p = normed(ia), q = normed(ib), c = cs[i], s = cs[half + i];
        dst[ia] = from_f<T>(p * c - q * s);
        dst[ib] = from_f<T>(q * c + p * s);
    }
    for (int i = 2 * half + lane; i < a.d; i += 32) dst[i] = from_f<T>(normed(i));
    if (r.part == 1 && a.key_mass && lane == 0) {
        const int ps = a.plan.page_size;
        a.key_mass[(slot / ps * a.hkv + r.head) * ps + slot % ps] = 0.f;
    }
}

template <typename T, int L> cudaError_t launch_l(const NormRopeArgs &a, int64_t rows, cudaStream_t st) {
    const int64_t blocks = (rows + kThreads / L - 1) / (kThreads / L);
    return launch_pdl(norm_rope_kernel<T, L>, dim3((unsigned)blocks), dim3(kThreads), 0, st, a, rows);
}

template <typename T> cudaError_t launch_t(const NormRopeArgs &a, cudaStream_t st) {
    constexpr int V = Chunk<T>::V;
    const int64_t rows = (int64_t)a.plan.queries * (a.hq + 2 * a.hkv);
    auto al = [](const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; };
    // 16-byte chunks throughout: whole pairs of chunks per row, rotated dims a
    // whole number of them, rows and bases aligned
    const bool wide = a.d % (2 * V) == 0 && a.d <= 64 * V && a.dv % V == 0 && a.rot % (2 * V) == 0 &&
                      a.q_stride % V == 0 && a.k_stride % V == 0 && a.v_stride % V == 0 && al(a.q) && al(a.k) &&
                      al(a.v) && al(a.q_out) && al(a.k_cache) && al(a.v_cache) && al(a.table) && al(a.q_weight) &&
                      al(a.k_weight);
    if (!wide) {
        const int64_t blocks = (rows + kThreads / 32 - 1) / (kThreads / 32);
        if (blocks > INT32_MAX) return cudaErrorInvalidValue;
        return launch_pdl(norm_rope_any_kernel<T>, dim3((unsigned)blocks), dim3(kThreads), 0, st, a, rows);
    }
    const int lanes = a.d / (2 * V);
    if (rows / (kThreads / 32) > INT32_MAX) return cudaErrorInvalidValue;
    if (lanes <= 4) return launch_l<T, 4>(a, rows, st);
    if (lanes <= 8) return launch_l<T, 8>(a, rows, st);
    if (lanes <= 16) return launch_l<T, 16>(a, rows, st);
    return launch_l<T, 32>(a, rows, st);
}

}  // namespace

cudaError_t launch_norm_rope_store(const NormRopeArgs &a, cudaStream_t st) {
    cudaError_t e;
    switch (a.dtype) {
        case PA_F32: e = launch_t<float>(a, st); break;
        case PA_F16: e = launch_t<__half>(a, st); break;
        default: e = launch_t<__nv_bfloat16>(a, st); break;
    }
    if (e != cudaSuccess) return e;
    return cudaGetLastError();
}

}  // namespace pa
