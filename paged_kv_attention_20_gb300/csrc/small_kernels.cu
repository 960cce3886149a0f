// Cache append, split merge and the device status word.
//
// Append: ruDNN 0.1.7, src/paged_attention/mod.rs, `append_with_report` --
// new rows [queries, heads, d|dv] land in the caches at the plan's positions,
// an elementwise kernel over queries * heads * max(d, dv).  Here each thread
// moves one 16-byte chunk (or one element when rows are not 16-byte multiples
// or not aligned); the destination slot comes precomputed in the plan.
//
// Merge: same page, `execute_attention_into` (merge launch when splits > 1)
// and `attention_into_split` (FP32 statistics): out = sum_s w_s o_s / sum_s w_s
// with w_s = exp(lse_s - max_s lse_s); empty splits (lse = -inf) weigh 0.

#include <atomic>

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "merge.cuh"
#include "pa_internal.h"

namespace pa {

__device__ int32_t g_device_status = 0;

template <typename U>
__global__ void kv_store_kernel(PlanView plan, const U *__restrict__ new_k, const U *__restrict__ new_v,
                                U *__restrict__ kc, U *__restrict__ vc, int heads, int uk, int uv,
                                int64_t total) {
    // One work unit = one U-sized piece of one row; K pieces then V pieces per (query, head).
    griddep_wait();
    griddep_launch();
    const int per_row = uk + uv;
    for (int64_t idx = blockIdx.x * (int64_t)blockDim.x + threadIdx.x; idx < total;
         idx += (int64_t)gridDim.x * blockDim.x) {
        int64_t row = idx / per_row;          // (query, head)
        int u = (int)(idx - row * per_row);
        int64_t qi = row / heads;
        int h = (int)(row - qi * heads);
        int64_t slot = plan.qmeta[qi].z;
        if (u < uk) {
            kc[(slot * heads + h) * uk + u] = new_k[row * uk + u];
        } else {
            u -= uk;
            vc[(slot * heads + h) * uv + u] = new_v[row * uv + u];
        }
    }
}

cudaError_t launch_kv_store(const PlanView &plan, const void *new_k, const void *new_v, void *k_cache,
                            void *v_cache, int heads, int d, int dv, int elem_bytes, cudaStream_t st) {
    const int64_t kb = (int64_t)d * elem_bytes, vb = (int64_t)dv * elem_bytes;
    auto al = [](const void *p, int a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; };
    int unit = elem_bytes;
    if (kb % 16 == 0 && vb % 16 == 0 && al(new_k, 16) && al(new_v, 16) && al(k_cache, 16) && al(v_cache, 16))
        unit = 16;
    const int uk = (int)(kb / unit), uv = (int)(vb / unit);
    const int64_t total = (int64_t)plan.queries * heads * (uk + uv);
    const int threads = 256;
    int64_t blocks = (total + threads - 1) / threads;
    if (blocks > 152 * 32) blocks = 152 * 32;
    if (blocks < 1) blocks = 1;
    const dim3 grid((unsigned)blocks), block(threads);
    cudaError_t e;
    if (unit == 16)
        e = launch_pdl(kv_store_kernel<uint4>, grid, block, 0, st, plan, (const uint4 *)new_k, (const uint4 *)new_v,
                       (uint4 *)k_cache, (uint4 *)v_cache, heads, uk, uv, total);
    else if (unit == 4)
        e = launch_pdl(kv_store_kernel<uint32_t>, grid, block, 0, st, plan, (const uint32_t *)new_k,
                       (const uint32_t *)new_v, (uint32_t *)k_cache, (uint32_t *)v_cache, heads, uk, uv, total);
    else
        e = launch_pdl(kv_store_kernel<uint16_t>, grid, block, 0, st, plan, (const uint16_t *)new_k,
                       (const uint16_t *)new_v, (uint16_t *)k_cache, (uint16_t *)v_cache, heads, uk, uv, total);
    if (e != cudaSuccess) return e;
    return cudaGetLastError();
}

template <typename T, int VEC>
__global__ void __launch_bounds__(256) merge_kernel(AttnArgs a, int use_list, int nrows) {
    griddep_wait();
    griddep_launch();
    merge_rows<T, VEC>(a, use_list, nrows, blockIdx.x);
}

template <typename T, int VEC>
__global__ void __launch_bounds__(256) merge_wide_kernel(AttnArgs a, int use_list) {
    griddep_wait();
    griddep_launch();
    extern __shared__ float part[];
    merge_row_wide<T, VEC>(a, use_list, blockIdx.x, part);
}

template <int VEC> cudaError_t launch_merge_vec(const AttnArgs &a, bool use_list, int nrows, cudaStream_t st) {
    const int ul = use_list ? 1 : 0;
    if (merge_is_wide(a, nrows)) {
        const dim3 grid((unsigned)nrows), block(256);
        const size_t smem = (size_t)8 * a.dv * sizeof(float);
        switch (a.dtype) {
            case PA_F32: return launch_pdl(merge_wide_kernel<float, VEC>, grid, block, smem, st, a, ul);
            case PA_F16: return launch_pdl(merge_wide_kernel<__half, VEC>, grid, block, smem, st, a, ul);
            default: return launch_pdl(merge_wide_kernel<__nv_bfloat16, VEC>, grid, block, smem, st, a, ul);
        }
    }
    const dim3 grid((unsigned)((nrows + 7) / 8)), block(256);
    switch (a.dtype) {
        case PA_F32: return launch_pdl(merge_kernel<float, VEC>, grid, block, 0, st, a, ul, nrows);
        case PA_F16: return launch_pdl(merge_kernel<__half, VEC>, grid, block, 0, st, a, ul, nrows);
        default: return launch_pdl(merge_kernel<__nv_bfloat16, VEC>, grid, block, 0, st, a, ul, nrows);
    }
}

cudaError_t launch_merge(const AttnArgs &a, bool use_list, cudaStream_t st) {
    const int items = use_list ? a.plan.n_decode : a.plan.queries;
    if (items == 0) return cudaSuccess;
    const int nrows = items * a.hq;
    const int vec = merge_vec(a);
    cudaError_t e = vec == 4   ? launch_merge_vec<4>(a, use_list, nrows, st)
                    : vec == 2 ? launch_merge_vec<2>(a, use_list, nrows, st)
                               : launch_merge_vec<1>(a, use_list, nrows, st);
    if (e != cudaSuccess) return e;
    return cudaGetLastError();
}

// Every query moves to the next position of its sequence: pos + 1, the write
// slot of that position from the block table, and a sequence length covering
// it.  A position the table does not map (past the row, or a negative or
// out-of-pool entry) leaves the query unchanged and records PA_DEVICE_RANGE.
__global__ void plan_advance_kernel(PlanView plan, int32_t *status) {
    griddep_wait();           // the previous kernel may still read the plan
    griddep_launch();
    const int q = blockIdx.x * blockDim.x + threadIdx.x;
    if (q >= plan.queries) return;
    int4 *meta = const_cast<int4 *>(plan.qmeta) + q;
    const int4 m = *meta;
    const int64_t np = (int64_t)m.y + 1;
    if (np >= (int64_t)plan.width * plan.page_size) {
        atomicCAS(status, 0, PA_DEVICE_RANGE);
        return;
    }
    const int32_t pg = plan.table[(int64_t)m.x * plan.width + np / plan.page_size];
    if (pg < 0 || pg >= plan.pages) {
        atomicCAS(status, 0, PA_DEVICE_RANGE);
        return;
    }
    *meta = make_int4(m.x, (int)np, pg * plan.page_size + (int)(np % plan.page_size), 0);
    atomicMax(const_cast<int32_t *>(plan.seq_lens) + m.x, (int)(np + 1));
}

cudaError_t launch_plan_advance(const PlanView &plan, int32_t *status, cudaStream_t st) {
    const int threads = 128;
    cudaError_t e = launch_pdl(plan_advance_kernel, dim3((unsigned)((plan.queries + threads - 1) / threads)),
                               dim3(threads), 0, st, plan, status);
    if (e != cudaSuccess) return e;
    return cudaGetLastError();
}

int32_t *device_status_ptr() {
    static std::atomic<int32_t *> cached[64];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return nullptr;
    int32_t *at = cached[dev].load(std::memory_order_acquire);
    if (!at) {
        void *p = nullptr;
        if (cudaGetSymbolAddress(&p, g_device_status) != cudaSuccess) return nullptr;
        at = static_cast<int32_t *>(p);
        cached[dev].store(at, std::memory_order_release);
    }
    return at;
}

cudaError_t read_device_status(int32_t *code, bool clear) {
    cudaError_t e = cudaDeviceSynchronize();
    if (e != cudaSuccess) return e;
    e = cudaMemcpyFromSymbol(code, g_device_status, sizeof(int32_t));
    if (e != cudaSuccess) return e;
    if (clear) {
        int32_t zero = 0;
        e = cudaMemcpyToSymbol(g_device_status, &zero, sizeof(int32_t));
    }
    return e;
}

}  // namespace pa
