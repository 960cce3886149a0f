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
#include "per_device.h"
#include "sm103_tc.cuh"

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

__device__ __forceinline__ RowId row_id(const NormRopeArgs &a, uint32_t idx) {
    const uint32_t per = (uint32_t)(a.hq + 2 * a.hkv);
    RowId r;
    r.token = (int)(idx / per);
    const int h = (int)(idx - (uint32_t)r.token * per);
    r.part = h < a.hq ? 0 : (h < a.hq + a.hkv ? 1 : 2);
    r.head = h - (r.part == 0 ? 0 : (r.part == 1 ? a.hq : a.hq + a.hkv));
    r.token += a.first_token;
    return r;
}

// Position of a token, or -1 when the table has no row for it.
__device__ __forceinline__ int table_position(const NormRopeArgs &a, int token, int plan_pos) {
    const int pos = a.positions ? a.positions[token] : plan_pos;
    return a.table && (pos < 0 || pos >= a.max_positions) ? -1 : pos;
}

// 1 / sqrt(mean of the row's squares + eps); a row's L lanes call together.
template <int V, int L>
__device__ __forceinline__ float row_scale(const float (&x0)[V], const float (&x1)[V], int d, float eps, unsigned group) {
    float ss = 0.f;
#pragma unroll
    for (int e = 0; e < V; ++e) ss += x0[e] * x0[e] + x1[e] * x1[e];
#pragma unroll
    for (int o = L / 2; o; o >>= 1) ss += __shfl_xor_sync(group, ss, o);
    return rsqrtf(ss / (float)d + eps);
}

// Turns a thread's pairs: (x0[i], x1[i]), or interleaved the neighbours of its 2V
// consecutive elements.
template <int V>
__device__ __forceinline__ void turn(float (&x0)[V], float (&x1)[V], const float (&c)[V], const float (&s)[V], bool interleaved) {
    if (interleaved) {
#pragma unroll
        for (int e = 0; e < V / 2; ++e) {
            const float p = x0[2 * e], q = x0[2 * e + 1];
            x0[2 * e] = p * c[e] - q * s[e];
            x0[2 * e + 1] = q * c[e] + p * s[e];
            const float u = x1[2 * e], v = x1[2 * e + 1];
            x1[2 * e] = u * c[V / 2 + e] - v * s[V / 2 + e];
            x1[2 * e + 1] = v * c[V / 2 + e] + u * s[V / 2 + e];
        }
    } else {
#pragma unroll
        for (int e = 0; e < V; ++e) {
            const float p = x0[e], q = x1[e];
            x0[e] = p * c[e] - q * s[e];
            x1[e] = q * c[e] + p * s[e];
        }
    }
}

// One row per group of L lanes: single tokens and small batches, where a launch's
// latency counts and the rows spread over as many CTAs as there are.
template <typename T, int L>
__global__ void __launch_bounds__(kThreads) norm_rope_kernel(NormRopeArgs a, uint32_t rows) {
    constexpr int V = Chunk<T>::V;
    griddep_wait();
    griddep_launch();
    const uint32_t idx0 = blockIdx.x * (uint32_t)(kThreads / L) + threadIdx.x / L;
    const int l = threadIdx.x % L;
    const int turned = a.rot / (2 * V);           // lanes that rotate
    // my two chunks: a pair of halves (or of neighbours) inside the rotated dims,
    // neighbours past them
    int c0 = l * 2 * V, c1 = c0 + V;
    if (!a.interleaved && l < turned) {
        c0 = l * V;
        c1 = a.rot / 2 + l * V;
    }
    const bool mine = l * 2 * V < a.d;
    const bool live = idx0 < rows;
    const RowId r = row_id(a, live ? idx0 : 0u);
    const int4 meta = a.plan.qmeta[r.token];
    uint4 w0 = make_uint4(0u, 0u, 0u, 0u), w1 = w0;
    if (r.part < 2 && mine) {
        const T *src = r.part == 0 ? static_cast<const T *>(a.q) + (int64_t)r.token * a.q_stride
                                   : static_cast<const T *>(a.k) + (int64_t)r.token * a.k_stride;
        src += (int64_t)r.head * a.d;
        w0 = *reinterpret_cast<const uint4 *>(src + c0);
        w1 = *reinterpret_cast<const uint4 *>(src + c1);
    }
    const int pos = table_position(a, r.token, meta.y);
    const int64_t slot = meta.z;
    const bool ok = live && (pos >= 0 || !a.table);
    if (live && !ok && l == 0) atomicCAS(a.status, 0, PA_DEVICE_RANGE);
    if (r.part == 2) {
        // value rows: a copy
        if (ok) {
            const uint4 *src = reinterpret_cast<const uint4 *>(
                static_cast<const T *>(a.v) + (int64_t)r.token * a.v_stride + (int64_t)r.head * a.dv);
            uint4 *dst = reinterpret_cast<uint4 *>(static_cast<T *>(a.v_cache) + (slot * a.hkv + r.head) * a.dv);
#pragma unroll 2
            for (int c = l; c < a.dv / V; c += L) dst[c] = src[c];
        }
        return;
    }
    float x0[V], x1[V], c[V], s[V];
    const bool turns = ok && a.table && l < turned;
    if (turns) {
        const float *cs = a.table + (int64_t)pos * a.rot + l * V;
#pragma unroll
        for (int e = 0; e < V; e += 4) {
            const float4 cc = *reinterpret_cast<const float4 *>(cs + e);
            const float4 sn = *reinterpret_cast<const float4 *>(cs + a.rot / 2 + e);
            c[e] = cc.x; c[e + 1] = cc.y; c[e + 2] = cc.z; c[e + 3] = cc.w;
            s[e] = sn.x; s[e + 1] = sn.y; s[e + 2] = sn.z; s[e + 3] = sn.w;
        }
    }
    Chunk<T>::unpack(w0, x0);
    Chunk<T>::unpack(w1, x1);
    const T *w = static_cast<const T *>(r.part == 0 ? a.q_weight : a.k_weight);
    if (w) {
        // a row's lanes are one aligned group of a warp and take the same branches;
        // other groups may be elsewhere, so the group names only itself
        const unsigned group = L == 32 ? 0xffffffffu : ((1u << (L & 31)) - 1u) << ((threadIdx.x & 31) / L * L);
        const float inv = row_scale<V, L>(x0, x1, a.d, a.eps, group);
        if (mine) {
            float g0[V], g1[V];
            Chunk<T>::unpack(*reinterpret_cast<const uint4 *>(w + c0), g0);
            Chunk<T>::unpack(*reinterpret_cast<const uint4 *>(w + c1), g1);
#pragma unroll
            for (int e = 0; e < V; ++e) {
                x0[e] *= inv * g0[e];
                x1[e] *= inv * g1[e];
            }
        }
    }
    if (!ok || !mine) return;
    if (turns) turn<V>(x0, x1, c, s, a.interleaved);
    T *dst = r.part == 0 ? static_cast<T *>(a.q_out) + ((int64_t)r.token * a.hq + r.head) * a.d
                            : static_cast<T *>(a.k_cache) + (slot * a.hkv + r.head) * a.d;
    *reinterpret_cast<uint4 *>(dst + c0) = Chunk<T>::pack(x0);
    *reinterpret_cast<uint4 *>(dst + c1) = Chunk<T>::pack(x1);
    if (r.part == 1 && a.key_mass && l == 0) {
        const int ps = a.plan.page_size;
        a.key_mass[(slot / ps * a.hkv + r.head) * ps + slot % ps] = 0.f;
    }
}

// ------------------------------------------------------------- many tokens --
// A prompt's tokens stream through shared memory: each warp has its own stages,
// lane 0 brings a token's Q, K, V and table row in with bulk copies, and the warp
// norms, turns and writes the rows from there.  The bytes in flight no longer
// hang on registers: with one row a thread an SM has 32 KB of loads in flight,
// too little for the HBM's latency.  A large token gets one stage and the SM up
// to 16 warps, whose loads, arithmetic and stores overlap one another's; small
// tokens get three stages a warp.  16384 tokens of 32 + 8 + 8 heads of 128 (bf16,
// 411 MB): one row a thread 98 us, three stages and five warps 123 us, one stage
// and 16 warps with bulk stores 82 us (a stage waited for its stores to be
// read), weights and turn folded into packed coefficients 79 us, stores from
// registers 75 us (5.5 TB/s).
constexpr int kManyTokens = 2048;
constexpr size_t kTokenSmem = 216 * 1024;

struct StageLayout {
    int q_bytes, k_bytes, v_bytes, t_bytes;    // of one token; t: the table row
    int stage;                                  // bytes of a stage
    int stages;                                 // of a warp
    int warps;                                  // a CTA's (0: a token is too large)
};

template <typename T> StageLayout stage_layout(const NormRopeArgs &a) {
    StageLayout l{};
    const int64_t q = (int64_t)a.hq * a.d * sizeof(T), k = (int64_t)a.hkv * a.d * sizeof(T),
                  v = (int64_t)a.hkv * a.dv * sizeof(T), t = a.table ? (int64_t)a.rot * 4 : 0;
    const int64_t stage = (q + k + v + t + 127) / 128 * 128;
    const int64_t room = (int64_t)kTokenSmem - 2 * a.d * (int64_t)sizeof(T);        // the weights' copy
    l.stages = room / (stage * 3 + 64) >= 16 ? 3 : 1;
    const int64_t warps = room / (stage * l.stages + 64);                            // 64: a warp's barriers
    if (warps < 1) return l;
    l.warps = (int)(warps > 16 ? 16 : warps);
    l.q_bytes = (int)q;
    l.k_bytes = (int)k;
    l.v_bytes = (int)v;
    l.t_bytes = (int)t;
    l.stage = (int)stage;
    return l;
}

__device__ __forceinline__ void bulk_load(void *dst, const void *src, int bytes, uint64_t *bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];\n" ::"r"(
                     tc::smem_u32(dst)),
                 "l"(src), "r"(bytes), "r"(tc::smem_u32(bar))
                 : "memory");
}

// 16 bytes of T as V / 2 float pairs and back.
template <typename T> struct Pairs {
    static constexpr int N = 8 / sizeof(T);
    static __device__ __forceinline__ float2 pair(uint32_t w);
    static __device__ __forceinline__ uint32_t word(float2 x);
    static __device__ __forceinline__ void unpack(const uint4 &w, float2 *p) {
        p[0] = pair(w.x); p[1] = pair(w.y); p[2] = pair(w.z); p[3] = pair(w.w);
    }
    static __device__ __forceinline__ uint4 pack(const float2 *p) {
        return make_uint4(word(p[0]), word(p[1]), word(p[2]), word(p[3]));
    }
};
template <> __device__ __forceinline__ float2 Pairs<__nv_bfloat16>::pair(uint32_t w) {
    return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}
template <> __device__ __forceinline__ uint32_t Pairs<__nv_bfloat16>::word(float2 x) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(x.x, x.y);
    return *reinterpret_cast<const uint32_t *>(&h);
}
template <> __device__ __forceinline__ float2 Pairs<__half>::pair(uint32_t w) {
    return __half22float2(*reinterpret_cast<const __half2 *>(&w));
}
template <> __device__ __forceinline__ uint32_t Pairs<__half>::word(float2 x) {
    const __half2 h = __floats2half2_rn(x.x, x.y);
    return *reinterpret_cast<const uint32_t *>(&h);
}
template <> struct Pairs<float> {
    static constexpr int N = 2;
    static __device__ __forceinline__ void unpack(const uint4 &w, float2 *p) {
        p[0] = make_float2(__uint_as_float(w.x), __uint_as_float(w.y));
        p[1] = make_float2(__uint_as_float(w.z), __uint_as_float(w.w));
    }
    static __device__ __forceinline__ uint4 pack(const float2 *p) {
        return make_uint4(__float_as_uint(p[0].x), __float_as_uint(p[0].y), __float_as_uint(p[1].x), __float_as_uint(p[1].y));
    }
};

__device__ __forceinline__ float2 fmul2(float2 a, float2 b) {
    unsigned long long r;
    asm("mul.rn.f32x2 %0, %1, %2;\n"
        : "=l"(r)
        : "l"(*reinterpret_cast<unsigned long long *>(&a)), "l"(*reinterpret_cast<unsigned long long *>(&b)));
    return *reinterpret_cast<float2 *>(&r);
}
__device__ __forceinline__ uint4 lds16(uint32_t addr) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];\n" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr));
    return v;
}
// The norm's weights and the turn of a token folded into 2 * 2N coefficient pairs
// for my 2N element pairs p (chunk c0: p[0..N), chunk c1: p[N..2N)).  The turn is
// linear, so with p scaled by the norm a row becomes
//   halves:     out[i] = p[i] cf[i] + p[N+i] cf[N+i],  out[N+i] = p[N+i] cf[2N+i] + p[i] cf[3N+i]
//   neighbours: out[i] = p[i] cf[i] + swapped(p[i]) cf[2N+i]
template <typename T>
__device__ __forceinline__ void coefficients(float2 (&cf)[4 * Pairs<T>::N], uint32_t weights, bool weighted, int c0, int c1,
                                             bool mine, uint32_t table_row, int half_bytes, int l, bool turns, bool interleaved) {
    constexpr int N = Pairs<T>::N, V = 2 * N;
    float2 g[2 * N];
#pragma unroll
    for (int i = 0; i < 2 * N; ++i) g[i] = make_float2(1.f, 1.f);
    if (weighted && mine) {
        Pairs<T>::unpack(lds16(weights + (uint32_t)(c0 * sizeof(T))), g);
        Pairs<T>::unpack(lds16(weights + (uint32_t)(c1 * sizeof(T))), g + N);
    }
    float2 c[N], sn[N];
#pragma unroll
    for (int i = 0; i < N; ++i) {
        c[i] = make_float2(1.f, 1.f);
        sn[i] = make_float2(0.f, 0.f);
    }
    if (turns) {
#pragma unroll
        for (int e = 0; e < V; e += 4) {
            Pairs<float>::unpack(lds16(table_row + (uint32_t)(4 * (l * V + e))), c + e / 2);
            Pairs<float>::unpack(lds16(table_row + (uint32_t)half_bytes + (uint32_t)(4 * (l * V + e))), sn + e / 2);
        }
    }
    if (interleaved) {
        // pair i of my 2N turns by angle i: (c, c) and (-s, s) for (x, y) and (y, x)
#pragma unroll
        for (int i = 0; i < 2 * N; ++i) {
            const float ci = i & 1 ? c[i / 2].y : c[i / 2].x, si = i & 1 ? sn[i / 2].y : sn[i / 2].x;
            cf[i] = make_float2(g[i].x * ci, g[i].y * ci);
            cf[2 * N + i] = make_float2(-g[i].y * si, g[i].x * si);
        }
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i) {
            cf[i] = fmul2(g[i], c[i]);
            cf[N + i] = fmul2(g[N + i], make_float2(-sn[i].x, -sn[i].y));
            cf[2 * N + i] = fmul2(g[N + i], c[i]);
            cf[3 * N + i] = fmul2(g[i], sn[i]);
        }
    }
}

template <typename T, int L, int kStages>
__global__ void __launch_bounds__(512, 1) norm_rope_tokens_kernel(NormRopeArgs a, StageLayout lay, int tokens) {
    constexpr int V = Chunk<T>::V, kRowsAtOnce = 32 / L;
    griddep_wait();
    extern __shared__ __align__(128) uint8_t smem[];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, l = lane % L;
    uint8_t *ring = smem + (size_t)warp * kStages * lay.stage;
    uint8_t *tail = smem + (size_t)lay.warps * kStages * lay.stage;
    uint64_t *full = reinterpret_cast<uint64_t *>(tail + warp * 64);
    T *weights = reinterpret_cast<T *>(tail + (size_t)lay.warps * 64);              // q_weight, k_weight
    for (int i = threadIdx.x; i < a.d; i += blockDim.x) {
        if (a.q_weight) weights[i] = static_cast<const T *>(a.q_weight)[i];
        if (a.k_weight) weights[a.d + i] = static_cast<const T *>(a.k_weight)[i];
    }
    if (lane == 0) {
        for (int i = 0; i < kStages; ++i) tc::mbar_init(&full[i], 1);
        tc::fence_mbar_init();
    }
    __syncthreads();

    const int turned = a.rot / (2 * V);
    int c0 = l * 2 * V, c1 = c0 + V;
    if (!a.interleaved && l < turned) {
        c0 = l * V;
        c1 = a.rot / 2 + l * V;
    }
    const bool mine = l * 2 * V < a.d;
    const int walkers = (int)gridDim.x * lay.warps, me = (int)blockIdx.x * lay.warps + warp;
    struct Token {
        int slot, pos;       // pos < 0 with a table: it has no such row
    };
    auto look_up = [&](int i) -> Token {         // my i-th token
        const int64_t t = me + (int64_t)i * walkers;
        if (t >= tokens) return Token{0, 0};
        const int4 m = a.plan.qmeta[a.first_token + t];
        return Token{m.z, table_position(a, a.first_token + (int)t, m.y)};
    };
    // lane 0 starts the loads of my i-th token into stage i % kStages
    auto load = [&](int i, const Token &k) {
        const int64_t t = me + (int64_t)i * walkers;
        if (t >= tokens || lane != 0) return;
        const int64_t at = a.first_token + t;
        uint8_t *st = ring + (size_t)(i % kStages) * lay.stage;
        uint64_t *bar = &full[i % kStages];
        const bool row = a.table && k.pos >= 0;
        tc::mbar_arrive_expect_tx(bar, (uint32_t)(lay.q_bytes + lay.k_bytes + lay.v_bytes + (row ? lay.t_bytes : 0)));
        bulk_load(st, static_cast<const T *>(a.q) + at * a.q_stride, lay.q_bytes, bar);
        bulk_load(st + lay.q_bytes, static_cast<const T *>(a.k) + at * a.k_stride, lay.k_bytes, bar);
        bulk_load(st + lay.q_bytes + lay.k_bytes, static_cast<const T *>(a.v) + at * a.v_stride, lay.v_bytes, bar);
        if (row) bulk_load(st + lay.q_bytes + lay.k_bytes + lay.v_bytes, a.table + (int64_t)k.pos * a.rot, lay.t_bytes, bar);
    };
    const int steps = me < tokens ? (tokens - me + walkers - 1) / walkers : 0;
    // tokens i .. i + kStages - 1 of step i, the last of them about to be loaded; a
    // token's metadata is looked up a step before its loads start
    Token queue[kStages + 1];
#pragma unroll
    for (int k = 0; k < kStages; ++k) {
        queue[k] = look_up(k);
        if (k < kStages - 1) load(k, queue[k]);
    }
    bool ok = true;
    int i = 0;
    for (; i < steps; ++i) {
        // the stage of token i + kStages - 1 held token i - 1, which every lane is done with
        queue[kStages] = look_up(i + kStages);
        load(i + kStages - 1, queue[kStages - 1]);
        const Token cur = queue[0];
        ok = __all_sync(0xffffffffu, tc::mbar_wait(&full[i % kStages], (uint32_t)((i / kStages) & 1)));
        if (!ok) break;
        uint8_t *st = ring + (size_t)(i % kStages) * lay.stage;
        const int64_t at = a.first_token + me + (int64_t)i * walkers;
        if (!a.table || cur.pos >= 0) {
            constexpr int N = Pairs<T>::N;
            const uint32_t stage = tc::smem_u32(st);
            const bool turns = a.table && l < turned;
            // the Q rows with Q's weights, then the K rows with K's (they follow in the stage)
#pragma unroll 1
            for (int part = 0; part < 2; ++part) {
                const int rows = part == 0 ? a.hq : a.hkv;
                const bool weighted = (part == 0 ? a.q_weight : a.k_weight) != nullptr;
                float2 cf[4 * N];
                coefficients<T>(cf, tc::smem_u32(weights + (part == 0 ? 0 : a.d)), weighted, c0, c1, mine,
                                stage + (uint32_t)(lay.q_bytes + lay.k_bytes + lay.v_bytes), 2 * a.rot, l, turns,
                                a.interleaved && turns);
                T *dst = part == 0 ? static_cast<T *>(a.q_out) + at * a.hq * a.d
                                   : static_cast<T *>(a.k_cache) + (int64_t)cur.slot * a.hkv * a.d;
                const uint32_t base = stage + (uint32_t)(part == 0 ? 0 : lay.q_bytes);
#pragma unroll 2
                for (int r0 = 0; r0 < rows; r0 += kRowsAtOnce) {
                    const int r = r0 + lane / L;
                    const bool live = r < rows && mine;
                    const uint32_t row = base + (uint32_t)((live ? r : 0) * a.d * (int)sizeof(T));
                    float2 p[2 * N], o[2 * N];
                    Pairs<T>::unpack(lds16(row + (uint32_t)((live ? c0 : 0) * sizeof(T))), p);
                    Pairs<T>::unpack(lds16(row + (uint32_t)((live ? c1 : 0) * sizeof(T))), p + N);
                    if (weighted) {
                        float2 ss = make_float2(0.f, 0.f);
#pragma unroll
                        for (int i = 0; i < 2 * N; ++i) ss = tc::ffma2(p[i], p[i], ss);
                        float sum = live ? ss.x + ss.y : 0.f;
#pragma unroll
                        for (int o2 = L / 2; o2; o2 >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o2);
                        const float inv = rsqrtf(sum / (float)a.d + a.eps);
#pragma unroll
                        for (int i = 0; i < 2 * N; ++i) p[i] = fmul2(p[i], make_float2(inv, inv));
                    }
                    if (!turns) {
                        // no partner's value enters, not even times 0
#pragma unroll
                        for (int i = 0; i < N; ++i) {
                            o[i] = fmul2(p[i], cf[i]);
                            o[N + i] = fmul2(p[N + i], cf[2 * N + i]);
                        }
                    } else if (a.interleaved) {
#pragma unroll
                        for (int i = 0; i < 2 * N; ++i)
                            o[i] = tc::ffma2(p[i], cf[i], fmul2(make_float2(p[i].y, p[i].x), cf[2 * N + i]));
                    } else {
#pragma unroll
                        for (int i = 0; i < N; ++i) {
                            o[i] = tc::ffma2(p[i], cf[i], fmul2(p[N + i], cf[N + i]));
                            o[N + i] = tc::ffma2(p[N + i], cf[2 * N + i], fmul2(p[i], cf[3 * N + i]));
                        }
                    }
                    if (live) {
                        *reinterpret_cast<uint4 *>(dst + (int64_t)r * a.d + c0) = Pairs<T>::pack(o);
                        *reinterpret_cast<uint4 *>(dst + (int64_t)r * a.d + c1) = Pairs<T>::pack(o + N);
                    }
                }
            }
            const int64_t slot = cur.slot;
            if (a.key_mass) {
                const int ps = a.plan.page_size;
                for (int h = lane; h < a.hkv; h += 32) a.key_mass[(slot / ps * a.hkv + h) * ps + slot % ps] = 0.f;
            }
            uint4 *vd = reinterpret_cast<uint4 *>(static_cast<T *>(a.v_cache) + slot * a.hkv * a.dv);
            const uint32_t vs = stage + (uint32_t)(lay.q_bytes + lay.k_bytes);
#pragma unroll 4
            for (int c = lane; c < lay.v_bytes / 16; c += 32) vd[c] = lds16(vs + (uint32_t)(16 * c));
        } else if (lane == 0) {
            atomicCAS(a.status, 0, PA_DEVICE_RANGE);
        }
        __syncwarp();
#pragma unroll
        for (int k = 0; k < kStages; ++k) queue[k] = queue[k + 1];
    }
    if (!ok && lane == 0) {
        atomicCAS(a.status, 0, PA_DEVICE_TIMEOUT_TMA);
        // tokens i .. i + kStages - 1 may still be landing in shared memory: wait for them, briefly
        for (int k = i; k < i + kStages && k < steps; ++k)
            tc::mbar_wait(&full[k % kStages], (uint32_t)((k / kStages) & 1), 2000000ll);
    }
    griddep_launch();
}

// Any head dim, stride and alignment: one warp per row, one element per lane
// and step.
template <typename T>
__global__ void __launch_bounds__(kThreads) norm_rope_any_kernel(NormRopeArgs a, uint32_t rows) {
    griddep_wait();
    griddep_launch();
    const uint32_t idx = blockIdx.x * (uint32_t)(kThreads / 32) + (threadIdx.x >> 5);
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

template <typename T, int L, int kStages>
cudaError_t launch_tokens(const NormRopeArgs &a, const StageLayout &lay, int tokens, cudaStream_t st) {
    static PerDevice configured;
    cudaError_t e = allow_smem(configured, norm_rope_tokens_kernel<T, L, kStages>, kTokenSmem);
    int sms = 0;
    if (e == cudaSuccess) e = device_sms(sms);
    if (e != cudaSuccess) return e;
    return launch_pdl(norm_rope_tokens_kernel<T, L, kStages>, dim3((unsigned)sms), dim3(32u * (unsigned)lay.warps),
                      kTokenSmem, st, a, lay, tokens);
}

template <typename T, int L> cudaError_t launch_l(const NormRopeArgs &a, uint32_t rows, cudaStream_t st) {
    constexpr uint32_t per = kThreads / L;                // rows a CTA and step
    const StageLayout lay = stage_layout<T>(a);
    if (a.plan.queries >= kManyTokens && lay.warps >= 4) {
        const int tokens = (int)(rows / (uint32_t)(a.hq + 2 * a.hkv));
        return lay.stages == 3 ? launch_tokens<T, L, 3>(a, lay, tokens, st) : launch_tokens<T, L, 1>(a, lay, tokens, st);
    }
    return launch_pdl(norm_rope_kernel<T, L>, dim3((rows + per - 1) / per), dim3(kThreads), 0, st, a, rows);
}

template <typename T> cudaError_t launch_t(const NormRopeArgs &a, uint32_t rows, cudaStream_t st) {
    constexpr int V = Chunk<T>::V;
    auto al = [](const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; };
    // 16-byte chunks throughout: whole pairs of chunks per row, rotated dims a
    // whole number of them, rows and bases aligned
    const bool wide = a.d % (2 * V) == 0 && a.d <= 64 * V && a.dv % V == 0 && a.rot % (2 * V) == 0 &&
                      a.q_stride % V == 0 && a.k_stride % V == 0 && a.v_stride % V == 0 && al(a.q) && al(a.k) &&
                      al(a.v) && al(a.q_out) && al(a.k_cache) && al(a.v_cache) && al(a.table) && al(a.q_weight) &&
                      al(a.k_weight);
    if (!wide)
        return launch_pdl(norm_rope_any_kernel<T>, dim3((rows + kThreads / 32 - 1) / (kThreads / 32)), dim3(kThreads), 0, st,
                          a, rows);
    const int lanes = a.d / (2 * V);
    if (lanes <= 4) return launch_l<T, 4>(a, rows, st);
    if (lanes <= 8) return launch_l<T, 8>(a, rows, st);
    if (lanes <= 16) return launch_l<T, 16>(a, rows, st);
    return launch_l<T, 32>(a, rows, st);
}

}  // namespace

cudaError_t launch_norm_rope_store(const NormRopeArgs &args, cudaStream_t st) {
    // rows are counted in 32 bits: a launch takes at most 2^30 of them (one launch,
    // but for batches of many millions of tokens)
    const int per = args.hq + 2 * args.hkv, most = (1 << 30) / per;
    for (int t = 0; t < args.plan.queries; t += most) {
        NormRopeArgs a = args;
        a.first_token = t;
        const int left = args.plan.queries - t;
        const uint32_t rows = (uint32_t)(left < most ? left : most) * (uint32_t)per;
        cudaError_t e;
        switch (a.dtype) {
            case PA_F32: e = launch_t<float>(a, rows, st); break;
            case PA_F16: e = launch_t<__half>(a, rows, st); break;
            default: e = launch_t<__nv_bfloat16>(a, rows, st); break;
        }
        if (e != cudaSuccess) return e;
        if (left <= most) break;
    }
    return cudaGetLastError();
}

}  // namespace pa
