// Per-key totals of prefill tiles on tcgen05 tensor cores.
//
// The attention has run and left every query's log-sum-exp.  For a block of 128
// keys of one sequence and KV head this kernel recomputes the scores against all
// the sequence's tile queries and adds up the weights:
//   total_j += sum over (query n, head h of the group) of 2^(scale_log2 * k_j . q_n - lse_n)
// The keys are the M rows of the MMA (S^T = K Q^T: K stays in shared memory, Q
// tiles of 128 queries of one head stream past), so a key is a TMEM lane and its
// sum lives in registers of one or two threads: no atomics, one fixed order, one
// add to memory per key.  A step (128 keys x 128 queries of one head) costs 2 * 128^3
// flops on the tensor core (512 cycles at its rate) and 128^2 exponentials (512 cycles
// at 32 a cycle and SM); P is never written and V never read.
//
// `mass_tiles_prepare_kernel` runs before it: it lists the key blocks of every
// sequence with tiles and lays the log-sum-exps out tile by tile, negated and in
// log2 units, so that a step's 128 arrive with one bulk copy.
//
// Roles, two CTAs per SM: warps 0-7 add up, in two groups that take every second
// step each; warp 8 walks the CTA's units and starts the loads of K (one box per
// page and 64-column half), Q (two stages) and the log-sum-exps; warp 9 issues the
// MMAs into two S buffers.  A ring of step descriptors in shared memory tells warps
// 0-7 and 9 what each step is.  All waits are bounded (timeout -> device status word).
//
// Eight chunks of 512 queries over 0.5-4.6K keys, 32 heads (15,600 steps, 65 GFLOP):
// one thread a key, log-sum-exps gathered by the producer 85 us; producer a step
// ahead 85 us; log-sum-exps by bulk copy, 64 columns a thread 78 us; two groups on
// alternate steps 71 us (0.92 PFLOP/s).  Units of 256 keys, each Q tile serving two
// MMAs, four Q stages in one CTA per SM: 80 us, as no second CTA then covers the load
// of a unit's keys.  What is left is latency (a Q tile arrives ~1500 cycles after its
// stage is free; two stages a CTA are all the shared memory holds) and the last round
// of units, which fills half of the GPU.

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "pa_internal.h"
#include "per_device.h"
#include "sm103_tc.cuh"
#include "tma_host.h"

namespace pa {
namespace {

using namespace tc;

constexpr int kKeys = 128;              // keys per unit: MMA rows
constexpr int kQ = 128;                 // queries per step: MMA columns
constexpr int kD = 128;                 // head dim
constexpr int kHalf = 128 * 128;        // bytes of 128 rows x 64 columns
constexpr int kTile = 2 * kHalf;
constexpr int kStages = 2;              // Q ring and S buffers
constexpr int kSlots = 8;               // step descriptors
constexpr int kAdders = 8;              // adding warps: two groups of four
constexpr int kThreads = 32 * (kAdders + 2);
constexpr uint32_t kTmemCols = kStages * kQ;
constexpr float kLog2e = 1.4426950408889634f;

enum StepKind { kWork = 0, kUnitEnd = 1, kExit = 2 };

struct alignas(16) Step {
    int kind, first;        // first: this step opens a unit (its K tile is new)
    int buf;                // S buffer, and so the group of warps, that takes it
    int key0;
    int pos0, nq;           // position of column 0, live columns
    int seq_len, kvh;
    int trow_lo, trow_hi;   // block-table row
};

struct Smem {
    uint8_t k[kTile];
    uint8_t q[kStages][kTile];
    // 16-byte aligned: bulk copies land here
    float lse[kSlots][kQ];                    // of the step's columns: negated, log2 units, 0 past the tile
    Step step[kSlots];
    float part[2][kKeys];                     // the second group's sums at the end of a unit
    uint64_t k_full, k_empty;
    uint64_t q_full[kStages], q_empty[kStages];
    uint64_t s_full[kStages], s_empty[kStages];
    uint64_t d_full[kSlots], d_empty[kSlots];
    uint64_t part_full[2], part_empty[2];
    uint32_t tmem_base;
};

struct TileParams {
    PlanView plan;
    float *key_mass;
    const float *lse;                         // [tiles, Hq, 128]
    const int32_t *group_list;                // tiles by sequence
    const int4 *blocks;                       // key blocks: {seq, first key, list entries [z, w)}
    const int32_t *n_blocks;
    int hq, hkv, causal, window, bf16;
    float scale_log2;
    int32_t *status;
};

__device__ __forceinline__ void bulk_load(void *dst, const void *src, uint32_t bytes, uint64_t *bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];\n" ::"r"(smem_u32(dst)),
                 "l"(src), "r"(bytes), "r"(smem_u32(bar))
                 : "memory");
}

__global__ void __launch_bounds__(kThreads, 2)
    mass_tiles_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k, TileParams prm) {
    griddep_wait();
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    if ((smem_u32(smem_raw) & 1023u) != 0u) {
        if (threadIdx.x == 0) atomicCAS(prm.status, 0, PA_DEVICE_LAYOUT);
        return;
    }
    Smem &s = *reinterpret_cast<Smem *>(smem_raw);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int ps = prm.plan.page_size, G = prm.hq / prm.hkv;

    if (tid == 0) {
        mbar_init(&s.k_full, 1);
        mbar_init(&s.k_empty, 1);
        for (int i = 0; i < kStages; ++i) {
            mbar_init(&s.q_full[i], 1);
            mbar_init(&s.q_empty[i], 1);
            mbar_init(&s.s_full[i], 1);
            mbar_init(&s.s_empty[i], 128);       // one group
        }
        for (int i = 0; i < kSlots; ++i) {
            mbar_init(&s.d_full[i], 1);
            mbar_init(&s.d_empty[i], kAdders + 1);      // the adding warps and the MMA issuer
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&s.part_full[i], 128);
            mbar_init(&s.part_empty[i], 128);
        }
        fence_mbar_init();
    }
    if (warp == 0) {
        tmem_alloc(&s.tmem_base, kTmemCols);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = s.tmem_base;

    if (warp == kAdders) {
        // ---------------------------------------------------- producer --
        if (lane == 0) {
            tma_prefetch_desc(&tm_q);
            tma_prefetch_desc(&tm_k);
        }
        const int units = *prm.n_blocks * prm.hkv;
        const int oob_row = prm.plan.pages * ps;
        const int n_boxes = kKeys / ps;
        int t = 0, d = 0, u_open = 0;          // steps, descriptors and units (K loads) so far
        bool go = true;
        // lane 0 waits, the warp follows
        auto wait = [&](uint64_t *bar, uint32_t parity) -> bool {
            int ok = 1;
            if (lane == 0) ok = mbar_wait(bar, parity) ? 1 : 0;
            return __shfl_sync(0xffffffffu, ok, 0) != 0;
        };
        auto slot_free = [&]() -> bool { return d < kSlots || wait(&s.d_empty[d % kSlots], (uint32_t)((d / kSlots - 1) & 1)); };
        auto tell = [&](const Step &st) -> bool {          // a descriptor without log-sum-exps
            if (!slot_free()) return false;
            if (lane == 0) {
                s.step[d % kSlots] = st;
                mbar_arrive(&s.d_full[d % kSlots]);
            }
            ++d;
            return true;
        };
        auto block_of = [&](int u) -> int4 { return u < units ? prm.blocks[u / prm.hkv] : make_int4(0, 0, 0, 0); };
        // Walk over the CTA's units, their tiles and the group's heads.  Nothing the
        // loop carries is a load still on its way, but for the next unit's record and
        // the next tile's number.
        int u = (int)blockIdx.x;
        int4 rec = block_of(u);
        while (go && u < units) {
            const int4 blk = rec;
            rec = block_of(u + (int)gridDim.x);
            Step st{};
            st.kind = kWork;
            st.kvh = u % prm.hkv;
            st.key0 = blk.y;
            st.seq_len = prm.plan.seq_lens[blk.x];
            const int32_t *trow = prm.plan.table + (int64_t)blk.x * prm.plan.width;
            st.trow_lo = (int32_t)(uint32_t)reinterpret_cast<uint64_t>(trow);
            st.trow_hi = (int32_t)(uint32_t)(reinterpret_cast<uint64_t>(trow) >> 32);
            // first and one-past-last tile entry that sees the unit's keys, 32 entries at a time
            auto sees = [&](const int4 &tile) {
                const int hi = prm.causal ? tile.w + tile.z : st.seq_len;
                const int64_t lo = prm.window > 0 ? (int64_t)tile.w - prm.window + 1 : 0;
                return st.key0 < hi && (int64_t)st.key0 + kKeys > lo;
            };
            bool open = false;
            st.buf = 0;
            for (int e0 = blk.z; go && e0 < blk.w; e0 += 32) {
                // a lane looks at one entry; the warp then takes those that count, in order
                const int id = e0 + lane < blk.w ? prm.group_list[e0 + lane] : -1;
                const int4 mine = id >= 0 ? prm.plan.tiles[id] : make_int4(0, 0, 0, 0);
                unsigned todo = __ballot_sync(0xffffffffu, id >= 0 && sees(mine));
                if (!open && todo) {
                    // the unit's keys
                    if (u_open > 0 && !wait(&s.k_empty, (uint32_t)((u_open - 1) & 1))) { go = false; break; }
                    ++u_open;
                    if (lane == 0) mbar_arrive_expect_tx(&s.k_full, kTile);
                    __syncwarp();
                    if (lane < n_boxes) {
                        const int lp = st.key0 / ps + lane, used_pages = (st.seq_len + ps - 1) / ps;
                        const int row = lp < used_pages ? trow[lp] * ps : oob_row;
                        tma_load_3d(s.k + lane * ps * 128, &tm_k, 0, st.kvh, row, &s.k_full);
                        tma_load_3d(s.k + kHalf + lane * ps * 128, &tm_k, 64, st.kvh, row, &s.k_full);
                    }
                    open = true;
                    st.first = 1;
                }
                while (go && todo) {
                    const int from = __ffs(todo) - 1;
                    todo &= todo - 1;
                    const int tile_id = __shfl_sync(0xffffffffu, id, from);
                    const int q0 = __shfl_sync(0xffffffffu, mine.y, from);
                    st.nq = __shfl_sync(0xffffffffu, mine.z, from);
                    st.pos0 = __shfl_sync(0xffffffffu, mine.w, from);
                    for (int g = 0; g < G; ++g) {
                        const int b = t % kStages, sl = d % kSlots, h = st.kvh * G + g;
                        if (!slot_free()) { go = false; break; }
                        if (lane == 0) {
                            s.step[sl] = st;
                            mbar_arrive_expect_tx(&s.d_full[sl], kQ * sizeof(float));
                            bulk_load(s.lse[sl], prm.lse + ((int64_t)tile_id * prm.hq + h) * kQ, kQ * sizeof(float), &s.d_full[sl]);
                        }
                        ++d;
                        st.first = 0;
                        st.buf ^= 1;
                        if (t >= kStages && !wait(&s.q_empty[b], (uint32_t)((t / kStages - 1) & 1))) { go = false; break; }
                        if (lane == 0) {
                            mbar_arrive_expect_tx(&s.q_full[b], kTile);
                            tma_load_3d(s.q[b], &tm_q, 0, h, q0, &s.q_full[b]);
                            tma_load_3d(s.q[b] + kHalf, &tm_q, 64, h, q0, &s.q_full[b]);
                        }
                        ++t;
                    }
                }
            }
            if (go && open) {
                st.kind = kUnitEnd;
                go = tell(st);
            }
            u += (int)gridDim.x;
        }
        {
            Step st{};
            st.kind = kExit;
            if (go) go = tell(st);
        }
        if (!go && lane == 0) atomicCAS(prm.status, 0, PA_DEVICE_TIMEOUT_TMA);
        // leave only when the last loads have landed (on a timeout some may be unread)
        if (lane == 0) {
            for (int i = t > kStages ? t - kStages : 0; i < t; ++i)
                mbar_wait(&s.q_full[i % kStages], (uint32_t)((i / kStages) & 1), 2000000ll);
            if (u_open > 0) mbar_wait(&s.k_full, (uint32_t)((u_open - 1) & 1), 2000000ll);
            for (int i = d > kSlots ? d - kSlots : 0; i < d; ++i)
                mbar_wait(&s.d_full[i % kSlots], (uint32_t)((i / kSlots) & 1), 2000000ll);
        }
    } else if (warp == kAdders + 1) {
        // -------------------------------------------------- MMA issuer --
        if (lane == 0) {
            const uint32_t idesc = idesc_f16(kKeys, kQ, prm.bf16 != 0, false, false);
            const uint64_t k_desc = smem_desc(smem_u32(s.k), 16, 1024, kLayoutSwizzle128B);
            int t = 0, units = 0, used[2] = {0, 0};      // used: steps of an S buffer so far
            bool ok = true;
            for (int d = 0;; ++d) {
                if (!mbar_wait(&s.d_full[d % kSlots], (uint32_t)((d / kSlots) & 1))) { ok = false; break; }
                const int4 st = *reinterpret_cast<const int4 *>(&s.step[d % kSlots]);
                const int kind = st.x, first = st.y, sb = st.z;
                mbar_arrive(&s.d_empty[d % kSlots]);
                if (kind == kExit) break;
                if (kind == kUnitEnd) {
                    mma_commit(&s.k_empty);          // K is free once the unit's MMAs are done
                    continue;
                }
                const int b = t % kStages;
                if (first && !mbar_wait(&s.k_full, (uint32_t)(units++ & 1))) { ok = false; break; }
                if (!mbar_wait(&s.q_full[b], (uint32_t)((t / kStages) & 1))) { ok = false; break; }
                const int n = sb ? used[1]++ : used[0]++;
                if (n > 0 && !mbar_wait(&s.s_empty[sb], (uint32_t)((n - 1) & 1))) { ok = false; break; }
                tc_fence_after();
                const uint64_t q_desc = smem_desc(smem_u32(s.q[b]), 16, 1024, kLayoutSwizzle128B);
#pragma unroll
                for (int ks = 0; ks < kD / 16; ++ks) {
                    const uint64_t o = (uint64_t)(((ks / 4) * kHalf + (ks % 4) * 32) >> 4);
                    mma_f16_ss(tmem + (uint32_t)(sb * kQ), k_desc + o, q_desc + o, idesc, ks > 0 ? 1u : 0u);
                }
                mma_commit(&s.s_full[sb]);
                mma_commit(&s.q_empty[b]);
                ++t;
            }
            if (!ok) atomicCAS(prm.status, 0, PA_DEVICE_TIMEOUT_MMA);
        }
    } else {
        // ------------------------------------------------ adding warps --
        // Group g = warps 4g .. 4g + 3 takes the steps of S buffer g, every second one
        // of a unit, so that one group's waits and start of a step lie under the
        // other's exponentials.  A thread is a key row (TMEM lane 32 * (warp % 4) + lane).
        const int row = 32 * (warp & 3) + lane, group = warp >> 2;
        const uint32_t sb = tmem + ((uint32_t)(32 * (warp & 3)) << 16) + (uint32_t)(group * kQ);
        const float2 sc2 = make_float2(prm.scale_log2, prm.scale_log2);
        float total = 0.f;
        int n = 0, unit = 0;                            // my steps and units so far
        bool ok = true;
        for (int d = 0;; ++d) {
            const int sl = d % kSlots;
            ok = __all_sync(0xffffffffu, mbar_wait(&s.d_full[sl], (uint32_t)((d / kSlots) & 1)));
            if (!ok) break;
            const int4 what = *reinterpret_cast<const int4 *>(&s.step[sl]);
            if (what.x == kExit) break;
            const int j = what.w + row;                // my key
            if (what.x == kUnitEnd) {
                const Step st = s.step[sl];
                // the second group hands its sums to the first (bounded waits: a named
                // barrier would hold the others if one warp had given up)
                const int slot = unit & 1;
                if (group == 1) {
                    if (unit >= 2)
                        ok = __all_sync(0xffffffffu, mbar_wait(&s.part_empty[slot], (uint32_t)((unit / 2 - 1) & 1)));
                    if (!ok) break;
                    s.part[slot][row] = total;
                    mbar_arrive(&s.part_full[slot]);
                } else {
                    ok = __all_sync(0xffffffffu, mbar_wait(&s.part_full[slot], (uint32_t)((unit / 2) & 1)));
                    if (!ok) break;
                    total += s.part[slot][row];
                    mbar_arrive(&s.part_empty[slot]);
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(&s.d_empty[sl]);
                if (group == 0 && j < st.seq_len && !(total == 0.f)) {
                    const int32_t *trow = reinterpret_cast<const int32_t *>((uint64_t)(uint32_t)st.trow_lo |
                                                                            ((uint64_t)(uint32_t)st.trow_hi << 32));
                    const int64_t page = trow[j / ps];
                    prm.key_mass[(page * prm.hkv + st.kvh) * ps + j % ps] += total;
                }
                total = 0.f;
                ++unit;
                continue;
            }
            if (what.z != group) {                     // the other group's step
                if (lane == 0) mbar_arrive(&s.d_empty[sl]);
                continue;
            }
            const int2 cols = *reinterpret_cast<const int2 *>(&s.step[sl].pos0);    // pos0, nq
            ok = __all_sync(0xffffffffu, mbar_wait(&s.s_full[group], (uint32_t)(n & 1)));
            if (!ok) break;
            ++n;
            tc_fence_after();
            float v[2][32];
            tmem_ld32f(sb, v[0]);
            // columns (queries) that see my key: an interval
            int n0 = prm.causal ? j - cols.x : 0, n1 = cols.y - 1;
            if (prm.window > 0) n1 = (int)min((int64_t)n1, (int64_t)j - cols.x + prm.window - 1);
            const bool edge = __any_sync(0xffffffffu, n0 > 0 || n1 < kQ - 1);
            const float4 *ls = reinterpret_cast<const float4 *>(s.lse[sl]);
            float2 acc[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) acc[i] = make_float2(0.f, 0.f);
            // 32 columns at a time, the next ones on their way
#pragma unroll
            for (int c = 0; c < kQ / 32; ++c) {
                tmem_wait_ld();
                if (c + 1 < kQ / 32) {
                    tmem_ld32f(sb + (uint32_t)(32 * (c + 1)), v[(c + 1) & 1]);
                } else {
                    // all of S is in registers: the next MMA may have the buffer
                    tc_fence_before();
                    mbar_arrive(&s.s_empty[group]);
                }
                const float *x = v[c & 1];
                if (!edge) {
#pragma unroll
                    for (int i = 0; i < 32; i += 4) {
                        const float4 l = ls[8 * c + i / 4];
                        const float2 p = ffma2(make_float2(x[i], x[i + 1]), sc2, make_float2(l.x, l.y));
                        const float2 q = ffma2(make_float2(x[i + 2], x[i + 3]), sc2, make_float2(l.z, l.w));
                        acc[(i / 2) & 3] = fadd2(acc[(i / 2) & 3], make_float2(ex2(p.x), ex2(p.y)));
                        acc[(i / 2 + 1) & 3] = fadd2(acc[(i / 2 + 1) & 3], make_float2(ex2(q.x), ex2(q.y)));
                    }
                } else {
#pragma unroll
                    for (int i = 0; i < 32; i += 2) {
                        const int col = 32 * c + i;
                        const float2 l = reinterpret_cast<const float2 *>(ls)[col / 2];
                        const float2 p = ffma2(make_float2(x[i], x[i + 1]), sc2, l);
                        // columns outside the interval hold other queries' scores, NaN included
                        acc[(i / 2) & 3] = fadd2(acc[(i / 2) & 3], make_float2(col >= n0 && col <= n1 ? ex2(p.x) : 0.f,
                                                                               col + 1 >= n0 && col + 1 <= n1 ? ex2(p.y) : 0.f));
                    }
                }
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&s.d_empty[sl]);
            const float2 sum = fadd2(fadd2(acc[0], acc[1]), fadd2(acc[2], acc[3]));
            total += sum.x + sum.y;
        }
        if (!ok && lane == 0) atomicCAS(prm.status, 0, PA_DEVICE_TIMEOUT_SOFTMAX);
    }
    griddep_launch();
    tc_fence_before();
    __syncthreads();
    if (warp == 0) {
        tc_fence_after();
        tmem_dealloc(tmem, kTmemCols);
    }
}

bool make_map(CUtensorMap *m, const void *base, int heads, int64_t rows, int box_rows, bool bf16) {
    return encode_map_3d(m, base, bf16, kD, (uint64_t)heads, (uint64_t)rows, (uint64_t)kD * 2, (uint64_t)kD * 2 * heads, 64,
                         1, (uint32_t)box_rows, CU_TENSOR_MAP_SWIZZLE_128B);
}

}  // namespace

cudaError_t launch_mass_tiles(const MassArgs &a, cudaStream_t st) {
    const bool bf16 = a.dtype == PA_BF16;
    CUtensorMap tq, tk;
    if (!make_map(&tq, a.q, a.hq, a.plan.queries, kQ, bf16) ||
        !make_map(&tk, a.k, a.hkv, (int64_t)a.plan.pages * a.plan.page_size, a.plan.page_size, bf16))
        return cudaErrorInvalidValue;
    static PerDevice configured;
    cudaError_t e = allow_smem(configured, mass_tiles_kernel, sizeof(Smem));
    int sms = 0;
    if (e == cudaSuccess) e = device_sms(sms);
    if (e != cudaSuccess) return e;
    TileParams prm{};
    prm.plan = a.plan;
    prm.key_mass = a.key_mass;
    prm.lse = a.tile_lse;
    prm.group_list = a.group_list;
    prm.blocks = a.blocks;
    prm.n_blocks = a.n_blocks;
    prm.hq = a.hq; prm.hkv = a.hkv;
    prm.causal = a.causal; prm.window = a.window;
    prm.bf16 = bf16 ? 1 : 0;
    prm.scale_log2 = a.scale * kLog2e;
    prm.status = a.status;
    e = launch_pdl(mass_tiles_kernel, dim3((unsigned)(2 * sms)), dim3(kThreads), sizeof(Smem), st, tq, tk, prm);
    if (e != cudaSuccess) return e;
    return cudaGetLastError();
}

}  // namespace pa
