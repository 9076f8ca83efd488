// bf16 attention backward on the sm_103a tensor cores (tcgen05 + TMA + tensor memory).
//
// The pages keep P out of device memory in the backward pass too: it is recomputed from Q, K and the
// saved statistic ("账房先生的奔命：Flash Attention 与内存 I/O 革命" §七 重计算).  The gradient formulas
// themselves are the textbook derivative of O = softmax(scale Q K^T) V:
//     P = exp(scale S - LSE),  dV = P^T dO,  dP = dO V^T,  dS = P o (dP - D),  D_i = dO_i . O_i,
//     dK = scale dS^T Q,  dQ = scale dS K.
//
// Three kernels per call:
//   bwd_prep_kernel   -D_i and -LSE_i * log2(e) per query row (padded to a multiple of 128 rows per head;
//                     pad rows get 0 and -inf so they contribute nothing), and zeroes the fp32 dQ
//                     accumulator.  Negated so that the main kernel applies them with packed-pair adds.
//   bwd_tc_kernel     one CTA per (head, block of 128 keys).  K_j, V_j stay in shared memory; the CTA
//                     walks every block of 128 queries i:
//                         S^T  = K_j Q_i^T              fp32 in tensor memory
//                         dP^T = V_j dO_i^T
//                         P^T  = exp2(S^T scale log2e - LSE2_i)    thread = key row; packed fp32
//                                                       pairs (f32x2) for the element-wise work
//                         dS^T = P^T o (dP^T - D_i)
//                         dV_j += P^T dO_i              P^T as bf16 from tensor memory
//                         dK_j += dS^T Q_i              dS^T as bf16 from tensor memory
//                         dQ_i = dS K_j                 dS as bf16 from shared memory (the slot's dS^T
//                                                       read MN-major), queries as tensor-memory lanes
//                     and adds dQ_i into the fp32 accumulator with tensor reduce-add copies.
//   bwd_dq_convert    dQ = bf16(scale * accumulator).
// The main and conversion kernels are programmatic dependents of the kernel before them: the prep kernel
// releases the main kernel at its start, whose TMA thread loads K and V and only then waits for the prep
// kernel's results; the conversion kernel launches as the main kernel's CTAs finish and waits for them.  The
// backward measured 0.8 % faster at N = 8192 d = 128, 2.6 % at N = 2048 and 2.3 % at B=4 H=16 N=2048 d = 64.
//
// At d = 128 every product is 128 x 128 x 128 (M = 128 keys or queries, N = 128 queries or head
// dimensions): N = 128 is the narrowest tcgen05 shape that runs at the full rate, which 64-query steps
// (three of five products at N = 64) did not reach.  Tensor memory then holds exactly S^T, dP^T, dV and
// dK (4 x 128 columns at d = 128), with dQ reusing the columns of dP^T; at d = 64 dQ has 64 columns of its
// own.  The MMAs of step i run in the order dV(i), S^T(i+1), dK(i), dQ(i), dP^T(i+1): the next S^T goes
// right behind dV (its columns held P^T, which dV has just read), so forming P(i+1) overlaps dK and dQ on
// the tensor core.
//
// Warp roles (320 threads): warps 0-3 and 4-7 are two warpgroups that own the same 128 key rows
// (tensor-memory lanes) and split each step's queries, 64 each, for P^T and dS^T; for dQ the lanes are
// the step's 128 queries and the warpgroups split the head dimension, d / 2 columns each, which they move
// out of tensor memory (thread = query row) and stage.  At the end warps 0-3 write dV and warps 4-7 dK.
// Warp 8 issues the TMA loads and every reduce-add, warp 9 allocates tensor memory and issues the MMAs.
//
// Shared memory (d = 128: 226 KB): K and V resident, two Q stages, and two slots that each hold a step's dO
// tile, then its dS^T (once dV has read dO), then the first warpgroup's fp32 dQ columns (once dQ has read
// dS^T) as d / 64 [128][32] blocks, 128-byte swizzled and written with 16-byte stores; the TMA thread adds
// each block into the accumulator with one tensor reduce and loads the dO tile of step i + 2 there by
// 64-column chunks, each once the block under it has been read (one barrier for the whole tile).  The
// second warpgroup's blocks have a buffer of their own, which the TMA thread adds only after it has issued
// that dO load: with the second half's reduce issued first (from that warpgroup's own leader thread) the dO
// tile queued behind it in the copy unit, which cost 11 % of the backward at d = 128.  At the end the K and V
// tiles' space takes the bf16 rows of dK and dV, so that they leave in whole-row stores.  The kernel has no static
// shared memory, so its dynamic region starts aligned and needs no slack.
//
// kCross (fa_cross_bwd): N counts keys, the queries are Tq blocks of their own length, and an entry has klen <= N
// keys.  Grouped query heads that share a key head are rows of one head here, so dK and dV sum over the group
// in tensor memory.  Key blocks past klen only write zeros; in the block that klen cuts, the rows past it are
// cleared in the K and V tiles (whatever lies there, 0 * NaN is NaN) before the first product.  Where there are few
// key blocks (a short prompt under many query rows), `parts` CTAs share the query blocks of each and leave fp32 dK and
// dV for bwd_join_kernel, which adds them up in a fixed order.  Over a single key block a step's dQ is complete: it
// leaves as bf16 from the registers, and there is no accumulator to clear, add to and convert.
//
// (An earlier layout formed dQ^T = K^T dS^T at d = 128, thread = head-dimension index, each warp staging a
// [64][32] stripe with scalar stores: once the tensor-memory loads were widened to 64 columns, the present
// layout measured 0.6-0.7 % faster, and it serves both head sizes.)

#include <cuda_bf16.h>
#include <math.h>
#include <type_traits>

#include "fa_internal.h"
#include "fa_ptx.cuh"

namespace fa {
namespace {

using namespace ptx;

__device__ int g_bwd_status;

constexpr int BK = 128;  // keys per CTA
constexpr int BQ = 128;  // queries per step
constexpr int HQ = 64;   // queries per warpgroup half of a step
constexpr int kThreads = 320;
constexpr int kTmaWarp = 8;
constexpr int kMmaWarp = 9;

struct BwdBarriers {
    uint64_t kv_full;
    uint64_t q_full[2];            // Q tile + LSE2 and -D rows of a step
    uint64_t q_empty[2];           // dK of that step has read the Q tile
    uint64_t do_full[2];           // a step's dO tile is in its slot
    uint64_t dv_done[2];           // dV of that step has read dO: the slot takes dS^T
    uint64_t staged_a[2];          // the first warpgroup's dQ columns are staged in the slot
    uint64_t s_full;
    uint64_t dp_full;
    uint64_t p_ready;              // both halves' P^T of a step are in tensor memory (256 arrivals)
    uint64_t ds_ready[2];          // a half's dS^T is in tensor memory (d = 128: and in the step's slot)
    uint64_t ds_smem;              // d = 64: both halves' dS^T are in the step's slot (what dQ reads)
    uint64_t dq_full;
    uint64_t dq_empty;
    uint64_t staged_b;             // the second warpgroup's dQ columns are in their staging buffer
    uint64_t stage_b_free;         // ... and their reduce has read them (arrived by the TMA thread)
    uint64_t dkdv_full;
    uint64_t mma_done;
    uint64_t kv_clean;             // kCross: K and V rows past the entry's keys are cleared (256 arrivals)
    uint32_t tmem_base;
    WaitCtl wait;
};

// Shared memory.  K and V stay resident; Q has two stages.  Each step's dO tile lives in one of two
// slots, and the slot is reused within the step: once dV has read dO it takes the step's dS^T (the A
// operand of dQ), and once dQ has read that it takes the first warpgroup's fp32 dQ columns, which the
// TMA thread adds into the accumulator before loading the dO tile of step i + 2 there.  The second
// warpgroup's columns have a buffer of their own.
template <int D>
struct BwdCfg {
    static constexpr int kChunks = D / 64;
    static constexpr uint32_t kChunkK = BK * 128;          // one 64-column chunk of a K or V tile
    static constexpr uint32_t kChunkQ = BQ * 128;          // one 64-column chunk of a Q or dO tile
    static constexpr uint32_t kKBytes = BK * D * 2;
    static constexpr uint32_t kQBytes = BQ * D * 2;
    static constexpr uint32_t kDSChunk = BK * 128;         // dS^T of one half: 128 key rows x 64 queries
    // dQ = dS K is formed with the step's queries as tensor-memory lanes (M = 128, N = d); the two
    // warpgroups split its d columns, and each stages [128 queries][d / 2] fp32.
    static constexpr uint32_t kHalfDQBytes = BQ * (D / 2) * 4;   // fp32 dQ of one warpgroup (16 or 32 KB)
    static constexpr uint32_t kSlotBytes = 2 * kDSChunk;   // holds a dO tile, dS^T or a half's dQ rows
    static constexpr uint32_t kOffK = 0;
    static constexpr uint32_t kOffV = kOffK + kKBytes;
    static constexpr uint32_t kOffQ = kOffV + kKBytes;
    static constexpr uint32_t kOffSlot = kOffQ + 2 * kQBytes;
    static constexpr uint32_t kOffStageB = kOffSlot + 2 * kSlotBytes;   // the second half's dQ rows
    // A warpgroup's dQ columns are staged as [BQ][32] fp32 blocks (128-byte swizzled, written by 16-byte
    // stores), d / 64 of them, each added into the accumulator by one tensor reduce.
    static constexpr int kDqBlocks = D / 64;
    // d = 64: dS ready for dK (tensor memory) is signalled before the shared-memory copy for dQ, which
    // waits for dV to have read the slot; a barrier of its own covers that copy.  At d = 128 one signal
    // after both measured as fast (and 0.7 % faster at N = 32768).
    static constexpr bool kEarlyDsReady = D == 64;
    static constexpr uint32_t kDqBlockBytes = BQ * 32 * 4;
    static constexpr uint32_t kRowBytes = BQ * 4;          // LSE2 or -D of one query block
    static constexpr uint32_t kOffRows = kOffStageB + kHalfDQBytes;    // [q stage][LSE2 | -D][BQ] floats
    static constexpr uint32_t kOffBar = kOffRows + 2 * 2 * kRowBytes;
    static constexpr uint32_t kSmemNeed = kOffBar + sizeof(BwdBarriers);
    // Room to align the region to 1024 bytes if the dynamic shared memory does not start aligned (it
    // does when the kernel has no static shared memory, which is the case here).
    static constexpr uint32_t kAlignSlack = kSmemNeed + 1024 <= 232448 ? 1024 : 232448 - kSmemNeed;
    static constexpr uint32_t kSmemBytes = kSmemNeed + kAlignSlack;
    static constexpr uint32_t kColS = 0, kColDP = 128, kColDV = 256, kColDK = 256 + D;
    // dQ reuses the columns of dP^T at d = 128 (all 512 are taken); at d = 64 it has spare columns of its
    // own, so the next dP^T need not wait for it to be moved out.
    static constexpr bool kOwnDQ = D == 64;
    static constexpr uint32_t kColDQ = kOwnDQ ? 256 + 2 * D : kColDP;
    static_assert(kColDQ + D <= 512, "tensor memory columns");
    static constexpr uint32_t kTmemCols = 512;
    static_assert(kQBytes <= kSlotBytes && kHalfDQBytes <= kSlotBytes, "slot contents");
    static_assert(kDqBlocks * kDqBlockBytes == kHalfDQBytes && kDqBlocks == kChunks, "one block per dO chunk");
    static_assert(kSmemNeed <= 232448, "shared memory per CTA");
};

// Query block visited at step i by a CTA whose walk starts at block `rot`.
__device__ __forceinline__ int qblock(int i, int rot, int Tq) {
    const int b = i + rot % Tq;
    return b < Tq ? b : b - Tq;
}
// The same for a CTA that takes the Tq blocks from `base` on (kCross; base 0 otherwise).
template <bool kCross>
__device__ __forceinline__ int qblock_from(int i, int rot, int Tq, int base) {
    return kCross ? base + qblock(i, rot, Tq) : qblock(i, rot, Tq);
}

template <int D, bool kCross, bool kDirect>
__device__ void bwd_producer(const CUtensorMap* tm_q, const CUtensorMap* tm_k, const CUtensorMap* tm_v,
                             const CUtensorMap* tm_do, const CUtensorMap* tm_dq, const float* lse2, const float* row_d,
                             float* __restrict__ dq_acc, uint8_t* smem, BwdBarriers* bars, int head, int k0, int N,
                             int Tq, int Npad, int rot, int qbase, int starve) {
    using C = BwdCfg<D>;
    WaitCtl* wc = &bars->wait;
    const uint64_t pol_keep = policy_evict_last();
    mbar_expect_tx(&bars->kv_full, 2 * C::kKBytes);
    for (int c = 0; c < C::kChunks; ++c) {
        tma_load_3d(smem + C::kOffK + c * C::kChunkK, tm_k, &bars->kv_full, c * 64, k0, head, pol_keep);
        tma_load_3d(smem + C::kOffV + c * C::kChunkK, tm_v, &bars->kv_full, c * 64, k0, head, pol_keep);
    }
    // The kernel may start while the prep kernel is still running: K and V are inputs of the call, but the
    // row terms and the zeroed accumulator are the prep kernel's, and only this thread touches them.
    griddep_wait();
    // The first warpgroup's dQ columns of step j end up in slot j % 2 as d / 64 [BQ][32] blocks.  This
    // thread adds each block into the accumulator once the warpgroup has staged them (rows past N are
    // clipped by the tensor map) and reloads the slot once the reduces have read it, so it owns the slot's
    // whole cycle.  Block c lies under chunk c of the dO tile that reloads the slot and is its own bulk
    // group, so that chunk c can load as soon as that block has been read.
    auto reduce_first_half = [&](int j) -> bool {
        const int t = j & 1;
        const int q0 = qblock_from<kCross>(j, rot, Tq, qbase) * BQ;
        if (!mbar_wait(&bars->staged_a[t], (j >> 1) & 1, wc)) return false;
        // (kDirect: nothing is staged, the arrival says that dQ has read the slot.)
        for (int w = 0; w < (kDirect ? 0 : C::kDqBlocks); ++w) {
            tma_reduce_add_3d(tm_dq, smem + C::kOffSlot + t * C::kSlotBytes + w * C::kDqBlockBytes, 32 * w, q0, head);
            bulk_commit_group();
        }
        return true;
    };
    // The second warpgroup's dQ columns of step j, from their own buffer, added after the dO loads so that
    // those do not queue behind them; the buffer is handed back once the reduce has read it.
    auto reduce_second_half = [&](int j) -> bool {
        // (kDirect: nothing arrives; without waits on stage_b_free nothing would hold the next arrival back.)
        if (!kDirect && !mbar_wait(&bars->staged_b, j & 1, wc)) return false;
        const int q0 = qblock_from<kCross>(j, rot, Tq, qbase) * BQ;
        for (int b = 0; b < (kDirect ? 0 : C::kDqBlocks); ++b)
            tma_reduce_add_3d(tm_dq, smem + C::kOffStageB + b * C::kDqBlockBytes, D / 2 + 32 * b, q0, head);
        bulk_commit_group();
        return true;
    };
    auto free_stage_b = [&]() {
        bulk_wait_group_read<0>();
        mbar_arrive(&bars->stage_b_free);
    };
    int q_issued = 0, do_issued = 0;
    bool ok = true;
    for (int i = 0; i < Tq && ok; ++i) {
        const int s = i & 1;
        const int qb = qblock_from<kCross>(i, rot, Tq, qbase);
        if (i >= 2 && !(ok = mbar_wait(&bars->q_empty[s], ((i >> 1) - 1) & 1, wc))) break;
        // starve != 0 withholds the Q loads so that the first waits on them run out: the failure path of
        // the bounded waits, exercised by the tests with a short budget.
        if (!starve) {
            uint64_t* bar = &bars->q_full[s];
            mbar_expect_tx(bar, C::kQBytes + 2 * C::kRowBytes);
            for (int c = 0; c < C::kChunks; ++c)
                tma_load_3d(smem + C::kOffQ + s * C::kQBytes + c * C::kChunkQ, tm_q, bar, c * 64, qb * BQ, head,
                            pol_keep);
            float* rows = reinterpret_cast<float*>(smem + C::kOffRows) + s * 2 * BQ;
            const size_t r0 = (size_t)head * Npad + (size_t)qb * BQ;
            bulk_load(rows, lse2 + r0, C::kRowBytes, bar);
            bulk_load(rows + BQ, row_d + r0, C::kRowBytes, bar);
            q_issued = i + 1;
        }

        if (i >= 2) {
            if (i >= 3) free_stage_b();
            if (!(ok = reduce_first_half(i - 2))) break;
        }
        for (int c = 0; c < C::kChunks; ++c) {
            // Chunk c overwrites the block of reduce group c (the groups are read in order).
            if (i >= 2) {
                if (C::kChunks == 2 && c == 0) bulk_wait_group_read<1>();
                else bulk_wait_group_read<0>();
            }
            if (c == 0) mbar_expect_tx(&bars->do_full[s], C::kQBytes);
            tma_load_3d(smem + C::kOffSlot + s * C::kSlotBytes + c * C::kChunkQ, tm_do, &bars->do_full[s], c * 64,
                        qb * BQ, head, pol_keep);
        }
        do_issued = i + 1;
        if (i >= 2 && !(ok = reduce_second_half(i - 2))) break;
    }
    for (int j = (Tq > 2 ? Tq - 2 : 0); ok && j < Tq; ++j) {
        if (j >= 1) free_stage_b();
        ok = reduce_first_half(j) && reduce_second_half(j);
    }
    bulk_wait_group<0>();
    // Copies still in flight must land before the CTA can exit.
    drain_wait(&bars->kv_full, 0, wc);
    for (int i = (q_issued > 2 ? q_issued - 2 : 0); i < q_issued; ++i) drain_wait(&bars->q_full[i & 1], (i >> 1) & 1, wc);
    for (int i = (do_issued > 2 ? do_issued - 2 : 0); i < do_issued; ++i)
        drain_wait(&bars->do_full[i & 1], (i >> 1) & 1, wc);
}

// MMA order of step i: dV(i), S^T(i+1), dK(i), dQ(i), dP^T(i+1).  S^T of the next step goes right
// behind dV (its columns held P^T, which dV has just read), so the softmax warps can form P(i+1) while
// the tensor core works on dK and dQ; at d = 128 dP^T(i+1) waits until dQ(i) has left its columns.
template <int D, bool kCross>
__device__ void bwd_mma(uint8_t* smem, BwdBarriers* bars, uint32_t tmem, int Tq, bool cut) {
    using C = BwdCfg<D>;
    WaitCtl* wc = &bars->wait;
    constexpr uint32_t idS = idesc_bf16_f32(BK, BQ, 0, 0);   // S^T, dP^T: A and B K-major over the head dimension
    constexpr uint32_t idG = idesc_bf16_f32(BK, D, 0, 1);    // dV, dK: A from TMEM, B MN-major [q][d]
    // dQ: A = dS read MN-major from the slot's dS^T, B = K (MN-major over d).
    constexpr uint32_t idQ = idesc_bf16_f32(BQ, D, 1, 1);
    // Operand descriptors are built once; each use only adds a constant byte offset.  K-major views
    // serve S^T and dP^T; MN-major views of the same tiles serve dV, dK and dQ.
    const uint64_t kK = sdesc_sw128(smem_u32(smem + C::kOffK), 16, 1024);
    const uint64_t kV = sdesc_sw128(smem_u32(smem + C::kOffV), 16, 1024);
    const uint64_t kQ = sdesc_sw128(smem_u32(smem + C::kOffQ), 16, 1024);
    const uint64_t kDO = sdesc_sw128(smem_u32(smem + C::kOffSlot), 16, 1024);
    const uint64_t mQ = sdesc_sw128(smem_u32(smem + C::kOffQ), C::kChunkQ, 1024);
    const uint64_t mDO = sdesc_sw128(smem_u32(smem + C::kOffSlot), C::kChunkQ, 1024);
    const uint64_t mK = sdesc_sw128(smem_u32(smem + C::kOffK), C::kChunkK, 1024);
    const uint64_t mDS = sdesc_sw128(smem_u32(smem + C::kOffSlot), C::kDSChunk, 1024);

    // X^T = A B^T over the head dimension, both tiles K-major (S^T = K Q^T, dP^T = V dO^T).
    auto qk_like = [&](uint64_t a0, uint64_t b0, uint32_t dst) {
        const uint32_t d = tmem + dst;
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk)
            mma_ss(d, sdesc_advance(a0, (kk / 4) * C::kChunkK + (kk % 4) * 32),
                   sdesc_advance(b0, (kk / 4) * C::kChunkQ + (kk % 4) * 32), idS, kk > 0);
    };
    // G += A[tmem] B_tile over one half's 64 queries, B MN-major over the head dimension (dV or dK).
    auto grad = [&](uint32_t a_col, uint64_t b0, int half, uint32_t dst, bool acc) {
        const uint32_t d = tmem + dst, a = tmem + a_col + half * HQ;
#pragma unroll
        for (int kk = 0; kk < HQ / 16; ++kk)
            mma_ts(d, a + kk * 8, sdesc_advance(b0, (half * (HQ / 16) + kk) * 16 * 128), idG,
                   (acc || kk > 0) ? 1u : 0u);
    };
    // dQ = dS K over the 128 keys: at d = 128 into the columns of dP^T (free once dK used dS^T), at d = 64
    // into columns of its own.
    auto dq = [&](uint64_t ds0) {
        const uint32_t d = tmem + C::kColDQ;
#pragma unroll
        for (int kk = 0; kk < BK / 16; ++kk)
            mma_ss(d, sdesc_advance(ds0, kk * 16 * 128), sdesc_advance(mK, kk * 16 * 128), idQ, kk > 0);
    };

    bool ok = mbar_wait_poll(&bars->kv_full, 0, wc) && mbar_wait_poll(&bars->q_full[0], 0, wc);
    if (kCross && cut) ok = ok && mbar_wait_poll(&bars->kv_clean, 0, wc);
    if (ok) {
        tc_fence_after();
        qk_like(kK, kQ, C::kColS);
        mma_commit(&bars->s_full);
        if ((ok = mbar_wait_poll(&bars->do_full[0], 0, wc))) {
            tc_fence_after();
            qk_like(kV, kDO, C::kColDP);
            mma_commit(&bars->dp_full);
        }
    }
    for (int i = 0; ok && i < Tq; ++i) {
        const int s = i & 1, s1 = s ^ 1;
        const uint64_t bdo = sdesc_advance(mDO, s * C::kSlotBytes), bq = sdesc_advance(mQ, s * C::kQBytes);
        // dV waits for both halves' P^T at once: one barrier test fewer per step for this thread, whose
        // every test costs the tensor core idle cycles, measured faster than starting on the first half
        // (1.3 % at d = 128, N = 8192; 2.4 % at N = 32768; 0.8 % at d = 64, N = 2048).
        if (!(ok = mbar_wait_poll(&bars->p_ready, i & 1, wc))) break;
        tc_fence_after();
        for (int h = 0; h < 2; ++h) grad(C::kColS, bdo, h, C::kColDV, i > 0 || h > 0);
        mma_commit(&bars->dv_done[s]);
        if (i + 1 < Tq) {
            if (!(ok = mbar_wait_poll(&bars->q_full[s1], ((i + 1) >> 1) & 1, wc))) break;
            tc_fence_after();
            qk_like(kK, sdesc_advance(kQ, s1 * C::kQBytes), C::kColS);
            mma_commit(&bars->s_full);
        }
        for (int h = 0; h < 2; ++h) {
            if (!(ok = mbar_wait_poll(&bars->ds_ready[h], i & 1, wc))) break;
            tc_fence_after();
            grad(C::kColDP, bq, h, C::kColDK, i > 0 || h > 0);
        }
        if (!ok) break;
        mma_commit(&bars->q_empty[s]);
        // dQ reads both halves' dS^T from the slot (at d = 128 ds_ready already covered it).
        if constexpr (C::kEarlyDsReady) {
            if (!(ok = mbar_wait_poll(&bars->ds_smem, i & 1, wc))) break;
            tc_fence_after();
        }
        // At d = 64 dQ has its own columns, which dQ of step i-1 must have left: each warpgroup arrives on
        // ds_smem(i) only after it has moved dQ(i-1) out (program order, behind that drain's tcgen05 fence),
        // so the wait on ds_smem above covers it and this thread saves a barrier test per step.
        static_assert(!C::kOwnDQ || C::kEarlyDsReady, "dQ's own columns are freed through ds_smem");
        dq(sdesc_advance(mDS, s * C::kSlotBytes));
        mma_commit(&bars->dq_full);
        if (i + 1 < Tq) {
            // One test for the whole dO tile: testing its two 64-column chunks separately, so that dP^T
            // could start on the first, measured 1.1-1.5 % slower at d = 128.
            if (!(ok = mbar_wait_poll(&bars->do_full[s1], ((i + 1) >> 1) & 1, wc))) break;
            // At d = 128 the columns of dP^T hold dQ of step i until it has been moved out.
            if (!C::kOwnDQ && !(ok = mbar_wait_poll(&bars->dq_empty, i & 1, wc))) break;
            tc_fence_after();
            qk_like(kV, sdesc_advance(kDO, s1 * C::kSlotBytes), C::kColDP);
            mma_commit(&bars->dp_full);
        }
    }
    if (ok) mma_commit(&bars->dkdv_full);
    mma_commit(&bars->mma_done);
    drain_wait(&bars->mma_done, 0, wc);
}

// What fa_cross_bwd adds to the kernel's arguments.
struct BwdCross {
    const int* key_lens;   // [B], or null: every entry has N keys
    int Hk, parts;         // parts: CTAs that share the query blocks of a key block
    float* part;           // parts > 1: [head][key block][part][dV, dK][128][D] fp32, dK not scaled
    __nv_bfloat16* dq;     // kDirect: where dQ goes
    int R;                 // query rows of a head
};

// Warps 0-7 write this CTA's share of dV (0-3) and dK (4-7): whole rows of fp32, a thread a row.
template <int D>
__device__ __noinline__ void bwd_write_parts(uint32_t tmem, float* __restrict__ part) {
    using C = BwdCfg<D>;
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int half = warp / 4, quarter = warp % 4;
    const uint32_t lane_off = (uint32_t)(quarter * 32) << 16;
    const uint32_t col = half == 0 ? C::kColDV : C::kColDK;
    float* row = part + ((size_t)blockIdx.x * 2 + half) * (BK * D) + (quarter * 32 + lane) * D;
#pragma unroll
    for (int q = 0; q < D / 32; ++q) {
        uint32_t y[32];
        tmem_ld32(tmem + lane_off + col + q * 32, y);
        tmem_ld_wait();
#pragma unroll
        for (int c = 0; c < 8; ++c)
            reinterpret_cast<uint4*>(row + q * 32)[c] = make_uint4(y[4 * c], y[4 * c + 1], y[4 * c + 2], y[4 * c + 3]);
    }
}

// Warps 0-7 write dV (0-3) and dK (4-7, scaled) once every MMA has completed.  The K and V tiles are free
// by then: each thread converts its key row to bf16 and puts it in the V (dV) or K (dK) tile's space,
// 16-byte chunks XOR-swizzled by the row; then each warp copies its own 32 rows out, a warp's 16-byte
// stores covering whole rows (two at d = 128, four at d = 64), where one row per thread would touch 32
// rows of memory per store.  A call rather than inlined code: inlined, its registers shaped the step loop
// of bwd_softgrad (this copy inlined made the d = 64 backward 2.4 % slower; called, it is 1.5-1.8 % faster
// than the one-row-per-thread stores at every N, and at d = 128 0.3 % faster at N = 8192, 1.8 % at 2048).
template <int D, bool kCross>
__device__ __noinline__ void bwd_write_dkdv(uint8_t* smem, uint32_t tmem, __nv_bfloat16* __restrict__ dk,
                                                   __nv_bfloat16* __restrict__ dv, int head, int k0, int N, int klen,
                                                   float scale) {
    using C = BwdCfg<D>;
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int half = warp / 4, quarter = warp % 4;
    const int r = quarter * 32 + lane;
    const uint32_t lane_off = (uint32_t)(quarter * 32) << 16;
    const uint32_t col = half == 0 ? C::kColDV : C::kColDK;
    const float mul = half == 0 ? 1.f : scale;
    __nv_bfloat16* out = half == 0 ? dv : dk;
    uint8_t* tile = smem + (half == 0 ? C::kOffV : C::kOffK);
    constexpr int kRowChunks = D / 8;                 // 16-byte chunks in a bf16 row
    constexpr int kRowsPerStore = 32 / kRowChunks;    // rows one warp store covers
#pragma unroll
    for (int q2 = 0; q2 < D / 64; ++q2) {
        uint32_t y[2][32];
        tmem_ld64(tmem + lane_off + col + q2 * 64, y);
        tmem_ld_wait();
#pragma unroll
        for (int b = 0; b < 2; ++b)
#pragma unroll
            for (int c4 = 0; c4 < 4; ++c4) {
                const int c = q2 * 8 + b * 4 + c4;
                uint32_t w[4];
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    w[e] = pack_bf16(__uint_as_float(y[b][8 * c4 + 2 * e]) * mul,
                                     __uint_as_float(y[b][8 * c4 + 2 * e + 1]) * mul);
                *reinterpret_cast<uint4*>(tile + r * (D * 2) + ((c ^ (r & (kRowChunks - 1))) << 4)) =
                    make_uint4(w[0], w[1], w[2], w[3]);
            }
    }
    __syncwarp();
    const int sub = lane / kRowChunks, c = lane % kRowChunks;
#pragma unroll
    for (int it = 0; it < 32 / kRowsPerStore; ++it) {
        const int rr = quarter * 32 + it * kRowsPerStore + sub;
        uint4 v = *reinterpret_cast<const uint4*>(tile + rr * (D * 2) + ((c ^ (rr & (kRowChunks - 1))) << 4));
        if (kCross && k0 + rr >= klen) v = make_uint4(0, 0, 0, 0);
        if (k0 + rr < N)
            *reinterpret_cast<uint4*>(out + ((size_t)head * N + k0 + rr) * D + c * 8) = v;
    }
}

// Warps 0-7.  Thread = key row r of the CTA (tensor-memory lane) in the softmax-gradient part, where
// `half` selects queries [64 half, 64 half + 64) of each step, and query row r of the step in the dQ
// part, where `half` selects head-dimension columns [d/2 half, d/2 half + d/2).
// Order of step i: dS(i), P(i+1), then dQ(i) out of tensor memory (P(0) comes first).
template <int D, bool kCross, bool kDirect>
__device__ void bwd_softgrad(uint8_t* smem, BwdBarriers* bars, uint32_t tmem, float* __restrict__ dq_acc,
                             const CUtensorMap* tm_dq, __nv_bfloat16* __restrict__ dk, __nv_bfloat16* __restrict__ dv,
                             int head, int k0, int N, int klen, int Tq, int rot, int qbase, float scale, float scale_log2,
                             const BwdCross& ca) {
    using C = BwdCfg<D>;
    WaitCtl* wc = &bars->wait;
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int half = warp / 4, quarter = warp % 4;
    const int r = quarter * 32 + lane;                    // key row in the block, = TMEM lane
    const uint32_t lane_off = (uint32_t)(quarter * 32) << 16;
    const bool valid_key = k0 + r < klen;
    const bool all_keys_valid = k0 + BK <= klen;   // CTA-uniform: only the head's last key block masks
    const float* rows_base = reinterpret_cast<const float*>(smem + C::kOffRows);
    const uint64_t sl2 = f2_pack(scale_log2, scale_log2);

    // P(j) for this half: P^T as bf16 pairs over the first 32 of the half's 64 columns of S^T; the fp32
    // values stay in p2 for dS(j).
    uint64_t p2[HQ / 2];
    auto form_p = [&](int j) -> bool {
        if (!warp_wait(&bars->s_full, j & 1, wc)) return false;
        if (!warp_wait(&bars->q_full[j & 1], (j >> 1) & 1, wc)) return false;
        tc_fence_after();
        const float* lse2 = rows_base + (j & 1) * 2 * BQ + half * HQ;
        uint32_t sr[2][32];
        tmem_ld64(tmem + lane_off + C::kColS + half * HQ, sr);
        tmem_ld_wait();
        uint32_t pk[32];
        // The row terms come in 16-byte loads (two query pairs each), and key rows past N are masked only in
        // the head's last key block: with both the backward measured 2 % faster at d = 128 and 4-6 % at d = 64.
        const float4* lse4 = reinterpret_cast<const float4*>(lse2);
        auto body = [&](auto all_valid) {
#pragma unroll
            for (int c2 = 0; c2 < HQ / 4; ++c2) {
                const float4 l = lse4[c2];
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    const int c = 2 * c2 + u;
                    const int q = (2 * c) / 32, e = (2 * c) % 32;
                    const uint64_t x2 = ffma2(f2_pack(__uint_as_float(sr[q][e]), __uint_as_float(sr[q][e + 1])), sl2,
                                              u == 0 ? f2_pack(l.x, l.y) : f2_pack(l.z, l.w));
                    float x0, x1;
                    f2_unpack(x2, x0, x1);
                    float p0 = ex2(x0), p1 = ex2(x1);
                    if constexpr (!decltype(all_valid)::value) {
                        p0 = valid_key ? p0 : 0.f;
                        p1 = valid_key ? p1 : 0.f;
                    }
                    p2[c] = f2_pack(p0, p1);
                    pk[c] = pack_bf16(p0, p1);
                }
            }
        };
        if (all_keys_valid) body(std::true_type{});
        else body(std::false_type{});
        tmem_st32(tmem + lane_off + C::kColS + half * HQ, pk);
        tmem_st_wait();
        tc_fence_before();
        // A warpgroup cannot arrive for step j + 1 before the phase of step j completes: P(j + 1) needs
        // S^T(j + 1), which the MMA thread issues only after that phase.
        mbar_arrive(&bars->p_ready);
        return true;
    };

    if (kCross && !all_keys_valid && klen < N) {
        if (!warp_wait(&bars->kv_full, 0, wc)) return;
        const int from = klen - k0, chunks = (BK - from) * 8;   // 16-byte pieces of a 64-column chunk's rows
        for (int i = threadIdx.x; i < 2 * C::kChunks * chunks; i += 256)
            *reinterpret_cast<uint4*>(smem + C::kOffK + (i / chunks) * C::kChunkK + from * 128 + (i % chunks) * 16) =
                make_uint4(0, 0, 0, 0);
        fence_proxy_async_smem();
        mbar_arrive(&bars->kv_clean);
    }
    bool ok = Tq > 0 && form_p(0);
    for (int i = 0; ok && i < Tq; ++i) {
        const int s = i & 1;
        // dS(i) = P(i) o (dP(i) - D).
        if (!(ok = warp_wait(&bars->dp_full, i & 1, wc))) break;
        tc_fence_after();
        const float4* drow4 = reinterpret_cast<const float4*>(rows_base + s * 2 * BQ + BQ + half * HQ);
        uint32_t pk[32];
        {
            uint32_t dr[2][32];
            tmem_ld64(tmem + lane_off + C::kColDP + half * HQ, dr);
            tmem_ld_wait();
#pragma unroll
            for (int c2 = 0; c2 < HQ / 4; ++c2) {
                const float4 dv4 = drow4[c2];
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    const int c = 2 * c2 + u;
                    const int q = (2 * c) / 32, e = (2 * c) % 32;
                    const uint64_t g2 = fadd2(f2_pack(__uint_as_float(dr[q][e]), __uint_as_float(dr[q][e + 1])),
                                              u == 0 ? f2_pack(dv4.x, dv4.y) : f2_pack(dv4.z, dv4.w));
                    float d0, d1;
                    f2_unpack(fmul2(p2[c], g2), d0, d1);
                    pk[c] = pack_bf16(d0, d1);
                }
            }
        }
        tmem_st32(tmem + lane_off + C::kColDP + half * HQ, pk);
        if constexpr (C::kEarlyDsReady) {
            // dK reads dS^T from tensor memory: signal it now, not after the shared-memory copy below,
            // which has to wait until dV has read the dO tile in the slot.
            tmem_st_wait();
            tc_fence_before();
            mbar_arrive(&bars->ds_ready[half]);
        }
        // dS^T row r into this half's chunk of the step's slot (128-byte rows, 16-byte chunks XOR-swizzled
        // by r % 8) for dQ, once dV has read the dO tile there.
        if (!(ok = warp_wait(&bars->dv_done[s], (i >> 1) & 1, wc))) break;
        uint8_t* row = smem + C::kOffSlot + s * C::kSlotBytes + half * C::kDSChunk + r * 128;
#pragma unroll
        for (int ch = 0; ch < 8; ++ch)
            *reinterpret_cast<uint4*>(row + ((ch ^ (r & 7)) << 4)) =
                make_uint4(pk[4 * ch], pk[4 * ch + 1], pk[4 * ch + 2], pk[4 * ch + 3]);
        fence_proxy_async_smem();
        if constexpr (C::kEarlyDsReady) {
            mbar_arrive(&bars->ds_smem);
        } else {
            tmem_st_wait();
            tc_fence_before();
            mbar_arrive(&bars->ds_ready[half]);
        }

        if (i + 1 < Tq && !(ok = form_p(i + 1))) break;

        // dQ_i: thread = query row r of the step, this warpgroup's d / 2 columns, staged as row r of d / 64
        // [BQ][32] fp32 blocks with 16-byte stores, 16-byte chunks XOR-swizzled by r % 8 (the tensor map's
        // 128-byte swizzle): the first warpgroup's in the step's slot (dQ has read its dS^T), the second's in
        // its own buffer once the previous step's reduce has read it.
        if (!(ok = warp_wait(&bars->dq_full, i & 1, wc))) break;
        tc_fence_after();
        uint32_t x[D / 64][32];
        if constexpr (D == 128) tmem_ld64(tmem + lane_off + C::kColDQ + (D / 2) * half, x);
        else tmem_ld32(tmem + lane_off + C::kColDQ + (D / 2) * half, x[0]);
        tmem_ld_wait();
        tc_fence_before();
        if constexpr (!C::kOwnDQ) mbar_arrive(&bars->dq_empty);
        if constexpr (kDirect) {
            const int row = qblock_from<kCross>(i, rot, Tq, qbase) * BQ + r;
            if (row < ca.R) {
                uint4* dst = reinterpret_cast<uint4*>(ca.dq + ((size_t)head * ca.R + row) * D + (D / 2) * half);
#pragma unroll
                for (int b = 0; b < D / 64; ++b)
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        uint32_t w[4];
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            w[e] = pack_bf16(__uint_as_float(x[b][8 * j + 2 * e]) * scale, __uint_as_float(x[b][8 * j + 2 * e + 1]) * scale);
                        dst[4 * b + j] = make_uint4(w[0], w[1], w[2], w[3]);
                    }
            }
            if (half == 0) mbar_arrive(&bars->staged_a[s]);
            continue;
        }
        if (half == 1 && i > 0 && !(ok = warp_wait(&bars->stage_b_free, (i - 1) & 1, wc))) break;
        uint8_t* rowp = smem + (half == 0 ? C::kOffSlot + s * C::kSlotBytes : C::kOffStageB) + r * 128;
#pragma unroll
        for (int b = 0; b < D / 64; ++b)
#pragma unroll
            for (int j = 0; j < 8; ++j)
                *reinterpret_cast<uint4*>(rowp + b * C::kDqBlockBytes + ((j ^ (lane & 7)) << 4)) =
                    make_uint4(x[b][4 * j], x[b][4 * j + 1], x[b][4 * j + 2], x[b][4 * j + 3]);
        fence_proxy_async_smem();
        mbar_arrive(half == 0 ? &bars->staged_a[s] : &bars->staged_b);
    }
    if (!ok) return;
    if (!warp_wait(&bars->dkdv_full, 0, wc)) return;
    tc_fence_after();
    if (kCross && ca.parts > 1) bwd_write_parts<D>(tmem, ca.part);
    else bwd_write_dkdv<D, kCross>(smem, tmem, dk, dv, head, k0, N, klen, scale);
}

// kDirect (kCross, one key block): dQ leaves as bf16 at once.
template <int D, bool kCross, bool kDirect>
__global__ void __launch_bounds__(kThreads, 1)
bwd_tc_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
              const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ CUtensorMap tm_do,
              const __grid_constant__ CUtensorMap tm_dq, const float* lse2, const float* row_d, float* __restrict__ dq_acc,
              __nv_bfloat16* __restrict__ dk, __nv_bfloat16* __restrict__ dv, int N, int Npad,
              int blocks_per_head, float scale, float scale_log2, long long wait_budget, int starve, BwdCross ca) {
    using C = BwdCfg<D>;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t pad = (1024 - (smem_u32(smem_raw) & 1023)) & 1023;
    if (pad > C::kAlignSlack) {   // cannot happen without static shared memory; never touch memory past the end
        if (threadIdx.x == 0) atomicCAS(&g_bwd_status, 0, (int)FA_ERR_CUDA);
        return;
    }
    uint8_t* smem = smem_raw + pad;
    BwdBarriers* bars = reinterpret_cast<BwdBarriers*>(smem + C::kOffBar);
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    // 1-D grid, head-major: the CTAs of one head walk the same Q/dO blocks, which stay in L2.
    const int parts = kCross ? ca.parts : 1;
    const int block = kCross ? (int)blockIdx.x / parts : (int)blockIdx.x;
    const int head = block / blocks_per_head;
    const int k0 = (block % blocks_per_head) * BK;
    int Tq = Npad / BQ, qbase = 0;
    if (kCross && parts > 1) {   // every part has a block: there are at most as many parts
        const int part = (int)blockIdx.x % parts, all = Tq;
        qbase = (int)((long long)all * part / parts);
        Tq = (int)((long long)all * (part + 1) / parts) - qbase;
    }
    // Every CTA of a head walks the query blocks starting at its own key-block index, so that at any time
    // the CTAs add into different dQ rows instead of all contending for the same ones in L2.
    const int rot = block % blocks_per_head;
    int klen = N;
    if (kCross) {
        if (ca.key_lens) klen = min(max(ca.key_lens[head / ca.Hk], 0), N);
        if (k0 >= klen) {   // no keys here: the gradients are zero
            const int64_t n16 = (int64_t)min(BK, N - k0) * (D / 8);
            const size_t at = ((size_t)head * N + k0) * D;
            for (int64_t i = threadIdx.x; parts == 1 && i < n16; i += kThreads) {   // (else bwd_join_kernel does)
                reinterpret_cast<uint4*>(dk + at)[i] = make_uint4(0, 0, 0, 0);
                reinterpret_cast<uint4*>(dv + at)[i] = make_uint4(0, 0, 0, 0);
            }
            if (kDirect) {
                const int q0 = qbase * BQ, rows = min(Tq * BQ, ca.R - q0);
                for (int64_t i = threadIdx.x; i < (int64_t)rows * (D / 8); i += kThreads)
                    reinterpret_cast<uint4*>(ca.dq + ((size_t)head * ca.R + q0) * D)[i] = make_uint4(0, 0, 0, 0);
            }
            griddep_wait();   // the conversion kernel counts on this grid ending after the prep kernel
            return;
        }
    }

    if (threadIdx.x == 0) {
        bars->wait.budget = wait_budget;
        mbar_init(&bars->kv_full, 1);
        for (int t = 0; t < 2; ++t) {
            mbar_init(&bars->q_full[t], 1);
            mbar_init(&bars->q_empty[t], 1);
            mbar_init(&bars->do_full[t], 1);
            mbar_init(&bars->dv_done[t], 1);
            mbar_init(&bars->staged_a[t], 128);
            mbar_init(&bars->ds_ready[t], 128);
        }
        mbar_init(&bars->staged_b, 128);
        mbar_init(&bars->p_ready, 256);
        mbar_init(&bars->s_full, 1);
        mbar_init(&bars->dp_full, 1);
        mbar_init(&bars->dq_full, 1);
        mbar_init(&bars->dq_empty, 256);
        mbar_init(&bars->ds_smem, 256);
        mbar_init(&bars->stage_b_free, 1);
        mbar_init(&bars->dkdv_full, 1);
        mbar_init(&bars->mma_done, 1);
        if (kCross) mbar_init(&bars->kv_clean, 256);
        bars->wait.abort = 0;
        fence_mbar_init();
    }
    if (warp == kTmaWarp && lane == 0) {
        tma_prefetch_desc(&tm_q);
        tma_prefetch_desc(&tm_k);
        tma_prefetch_desc(&tm_v);
        tma_prefetch_desc(&tm_do);
        tma_prefetch_desc(&tm_dq);
    }
    if (warp == kMmaWarp) {
        tmem_alloc(&bars->tmem_base, C::kTmemCols);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = bars->tmem_base;

    if (warp == kTmaWarp) {
        if (lane == 0)
            bwd_producer<D, kCross, kDirect>(&tm_q, &tm_k, &tm_v, &tm_do, &tm_dq, lse2, row_d, dq_acc, smem, bars, head, k0, N, Tq, Npad,
                                    rot, qbase, starve);
    } else if (warp == kMmaWarp) {
        if (lane == 0) bwd_mma<D, kCross>(smem, bars, tmem, Tq, k0 + BK > klen && klen < N);
    } else {
        bwd_softgrad<D, kCross, kDirect>(smem, bars, tmem, dq_acc, &tm_dq, dk, dv, head, k0, N, klen, Tq, rot, qbase, scale,
                                scale_log2, ca);
    }

    tc_fence_before();
    __syncthreads();
    if (warp == kMmaWarp) {
        tc_fence_after();
        tmem_dealloc(tmem, C::kTmemCols);
    }
    if (threadIdx.x == 0 && bars->wait.abort) atomicCAS(&g_bwd_status, 0, (int)FA_ERR_TIMEOUT);
}

// ------------------------------------------------------------------------------------------------ one query block
// kCross heads of one query block (128 rows or fewer; d = 64: or two) over many keys: queries and keys change places.  A
// CTA keeps the head's Q and dO in shared memory and walks key blocks: a block's dV and dK are complete and leave as bf16
// from the V and K tiles' space by tensor stores, and dQ adds up in tensor memory until the end.  With a CTA a key block
// (above) 0.7 us of work came with 5 us of set-up and write-out.  At d = 64 the tensor core forms the next S^T behind dV,
// as above; at d = 128 tensor memory is full, dK takes the columns of S^T, and the next S^T waits until dK has left them.
// Bound by HBM and, at d = 128, by that chain: 1024 heads of 128 rows over 2000 keys take 252 us at d = 64 (4.4 TB/s; a
// CTA a key block 650) and 421 at d = 128 (5.3 TB/s; 893); of 200 rows at d = 64 415 (826).  With the gradients copied
// out by the threads instead of tensor stores 288 and 547.
struct WalkBarriers {
    uint64_t q_full;               // Q, dO and the row terms
    uint64_t kv_full[4];
    uint64_t staged[4];            // a block's dK and dV are in its K and V tiles (256 arrivals)
    uint64_t s_full;
    uint64_t dp_full;
    uint64_t p_ready;              // P^T is in tensor memory (256 arrivals)
    uint64_t ds_ready;             // dS^T is in tensor and shared memory (256 arrivals)
    uint64_t grad_full;            // a step's products are done
    uint64_t drained[2];           // ... and its dV and its dK are out of tensor memory (128 arrivals)
    uint64_t mma_done;
    uint64_t kv_clean;             // K and V rows past the entry's keys are cleared (256 arrivals)
    uint32_t tmem_base;
    WaitCtl wait;
};

// kNq: query blocks of a head.  d = 64 leaves room for two; a step is then a key block and one of them.
template <int D, int kNq>
struct WalkCfg {
    static constexpr int kStages = D == 64 ? 4 : 2;
    static constexpr int kChunks = D / 64;
    static constexpr uint32_t kChunk = 128 * 128;          // 64 columns of a tile
    static constexpr uint32_t kTile = 128 * D * 2;
    static constexpr uint32_t kOffQ = 0, kOffKV = kNq * 2 * kTile;   // query block: Q, then dO; stage: K, then V
    static constexpr uint32_t kOffDS = kOffKV + kStages * 2 * kTile;           // dS^T, 128 keys x 64 queries a half
    static constexpr uint32_t kOffRows = kOffDS + 2 * kChunk;                  // LSE2 | -D
    static constexpr uint32_t kRowBytes = kNq * BQ * 4;
    static constexpr uint32_t kOffBar = kOffRows + 2 * kRowBytes;
    static constexpr uint32_t kSmemNeed = kOffBar + sizeof(WalkBarriers);
    static constexpr uint32_t kAlignSlack = kSmemNeed + 1024 <= 232448 ? 1024 : 232448 - kSmemNeed;   // as BwdCfg's
    static constexpr uint32_t kSmemBytes = kSmemNeed + kAlignSlack;
    static constexpr bool kOwnDK = D == 64;
    static constexpr uint32_t kColS = 0, kColDP = 128, kColDV = 256, kColDK = kOwnDK ? 320 : kColS, kColDQ = 384;
    static constexpr uint32_t kTmemCols = 512;
    static_assert(kSmemNeed <= 232448, "shared memory per CTA");
    static_assert(kColDQ + kNq * D <= 512, "tensor memory columns");
    static_assert(kOwnDK || kNq == 1, "the next S^T waits until dK is out");
};

template <int D, int kNq>
__device__ void walk_producer(const CUtensorMap* tm_q, const CUtensorMap* tm_k, const CUtensorMap* tm_v,
                              const CUtensorMap* tm_do, const CUtensorMap* tm_dk, const CUtensorMap* tm_dv,
                              const float* lse2, const float* row_d, uint8_t* smem, WalkBarriers* bars, int head, int b0,
                              int T, int Npad, int starve) {
    using C = WalkCfg<D, kNq>;
    WaitCtl* wc = &bars->wait;
    const uint64_t pol = policy_evict_first();
    auto load_kv = [&](int j) {
        const int s = j % C::kStages;
        uint8_t* tile = smem + C::kOffKV + s * 2 * C::kTile;
        mbar_expect_tx(&bars->kv_full[s], 2 * C::kTile);
        for (int c = 0; c < C::kChunks; ++c) {
            tma_load_3d(tile + c * C::kChunk, tm_k, &bars->kv_full[s], c * 64, (b0 + j) * BK, head, pol);
            tma_load_3d(tile + C::kTile + c * C::kChunk, tm_v, &bars->kv_full[s], c * 64, (b0 + j) * BK, head, pol);
        }
    };
    int issued = 0;
    load_kv(issued++);
    griddep_wait();   // the row terms are the prep kernel's
    if (!starve) {
        mbar_expect_tx(&bars->q_full, kNq * 2 * C::kTile + 2 * C::kRowBytes);
        for (int i = 0; i < kNq * C::kChunks; ++i) {
            const int c = i % C::kChunks, b = i / C::kChunks;
            uint8_t* tile = smem + C::kOffQ + b * 2 * C::kTile + c * C::kChunk;
            tma_load_3d(tile, tm_q, &bars->q_full, c * 64, b * BQ, head, pol);
            tma_load_3d(tile + C::kTile, tm_do, &bars->q_full, c * 64, b * BQ, head, pol);
        }
        bulk_load(smem + C::kOffRows, lse2 + (size_t)head * Npad, C::kRowBytes, &bars->q_full);
        bulk_load(smem + C::kOffRows + C::kRowBytes, row_d + (size_t)head * Npad, C::kRowBytes, &bars->q_full);
    }
    while (issued < T && issued < C::kStages) load_kv(issued++);
    for (int j = 0; j < T; ++j) {   // a block's gradients leave (rows past N are clipped), then its stage is filled again
        if (!mbar_wait(&bars->staged[j % C::kStages], (j / C::kStages) & 1, wc)) break;
        uint8_t* tile = smem + C::kOffKV + (j % C::kStages) * 2 * C::kTile;
        for (int c = 0; c < C::kChunks; ++c) {
            tma_store_3d(tm_dk, tile + c * C::kChunk, c * 64, (b0 + j) * BK, head);
            tma_store_3d(tm_dv, tile + C::kTile + c * C::kChunk, c * 64, (b0 + j) * BK, head);
        }
        bulk_commit_group();
        if (issued < T) {
            bulk_wait_group_read<0>();
            load_kv(issued++);
        }
    }
    bulk_wait_group<0>();
    // Copies still in flight must land before the CTA can exit.
    if (!starve) drain_wait(&bars->q_full, 0, wc);
    for (int j = (issued > C::kStages ? issued - C::kStages : 0); j < issued; ++j)
        drain_wait(&bars->kv_full[j % C::kStages], (j / C::kStages) & 1, wc);
}

template <int D, int kNq>
__device__ void walk_mma(uint8_t* smem, WalkBarriers* bars, uint32_t tmem, int T, bool cut) {
    using C = WalkCfg<D, kNq>;
    WaitCtl* wc = &bars->wait;
    constexpr uint32_t idS = idesc_bf16_f32(BK, BQ, 0, 0);   // as in bwd_mma
    constexpr uint32_t idG = idesc_bf16_f32(BK, D, 0, 1);
    constexpr uint32_t idQ = idesc_bf16_f32(BQ, D, 1, 1);
    const uint64_t kK = sdesc_sw128(smem_u32(smem + C::kOffKV), 16, 1024);
    const uint64_t kQ = sdesc_sw128(smem_u32(smem + C::kOffQ), 16, 1024);
    const uint64_t mQ = sdesc_sw128(smem_u32(smem + C::kOffQ), C::kChunk, 1024);
    const uint64_t mK = sdesc_sw128(smem_u32(smem + C::kOffKV), C::kChunk, 1024);
    const uint64_t mDS = sdesc_sw128(smem_u32(smem + C::kOffDS), C::kChunk, 1024);
    // S^T = K Q^T and dP^T = V dO^T of step u: `other` 0 or 1 takes the second tile of each pair (V, dO).
    auto scores = [&](int u, int other, uint32_t dst) {
        const uint64_t a0 = sdesc_advance(kK, (2 * (u / kNq % C::kStages) + other) * C::kTile);
        const uint64_t q0 = sdesc_advance(kQ, (2 * (u % kNq) + other) * C::kTile);
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk)
            mma_ss(tmem + dst, sdesc_advance(a0, (kk / 4) * C::kChunk + (kk % 4) * 32),
                   sdesc_advance(q0, (kk / 4) * C::kChunk + (kk % 4) * 32), idS, kk > 0);
    };
    // dV += P^T dO and dK += dS^T Q over the 128 queries, each half's 64 in 32 columns at the half's start.
    auto grad = [&](int u, uint32_t a_col, int other, uint32_t dst) {
        const uint64_t q0 = sdesc_advance(mQ, (2 * (u % kNq) + other) * C::kTile);
#pragma unroll
        for (int kk = 0; kk < BQ / 16; ++kk)
            mma_ts(tmem + dst, tmem + a_col + (kk / 4) * HQ + (kk % 4) * 8, sdesc_advance(q0, kk * 16 * 128), idG,
                   (u % kNq > 0 || kk > 0) ? 1u : 0u);
    };
    auto wait_kv = [&](int u) -> bool {
        const int j = u / kNq;
        if (u % kNq) return true;
        return mbar_wait_poll(&bars->kv_full[j % C::kStages], (j / C::kStages) & 1, wc) &&
               (!(cut && j == T - 1) || mbar_wait_poll(&bars->kv_clean, 0, wc));
    };
    const int steps = T * kNq;
    bool ok = mbar_wait_poll(&bars->q_full, 0, wc) && wait_kv(0);
    if (ok) {
        tc_fence_after();
        scores(0, 0, C::kColS);
        mma_commit(&bars->s_full);
        scores(0, 1, C::kColDP);
        mma_commit(&bars->dp_full);
    }
    for (int u = 0; ok && u < steps; ++u) {
        const int j = u / kNq;
        const bool next = u + 1 < steps, drained = u % kNq == 0 && j > 0;   // drained: the last block's gradients must be out
        if (!(ok = mbar_wait_poll(&bars->p_ready, u & 1, wc))) break;
        if (drained && !(ok = mbar_wait_poll(&bars->drained[0], (j - 1) & 1, wc))) break;
        tc_fence_after();
        grad(u, C::kColS, 1, C::kColDV);
        if (C::kOwnDK && next) {
            if (!(ok = wait_kv(u + 1))) break;
            tc_fence_after();
            scores(u + 1, 0, C::kColS);
            mma_commit(&bars->s_full);
        }
        if (!(ok = mbar_wait_poll(&bars->ds_ready, u & 1, wc))) break;
        if (C::kOwnDK && drained && !(ok = mbar_wait_poll(&bars->drained[1], (j - 1) & 1, wc))) break;
        tc_fence_after();
        grad(u, C::kColDP, 0, C::kColDK);
        const uint64_t k0 = sdesc_advance(mK, 2 * (j % C::kStages) * C::kTile);
#pragma unroll
        for (int kk = 0; kk < BK / 16; ++kk)   // dQ += dS K
            mma_ss(tmem + C::kColDQ + (u % kNq) * D, sdesc_advance(mDS, kk * 16 * 128), sdesc_advance(k0, kk * 16 * 128), idQ,
                   (j > 0 || kk > 0) ? 1u : 0u);
        mma_commit(&bars->grad_full);
        if (next) {
            if (!C::kOwnDK && !(ok = wait_kv(u + 1))) break;
            tc_fence_after();
            scores(u + 1, 1, C::kColDP);
            mma_commit(&bars->dp_full);
            if (!C::kOwnDK) {
                if (!(ok = mbar_wait_poll(&bars->drained[1], j & 1, wc))) break;
                tc_fence_after();
                scores(u + 1, 0, C::kColS);
                mma_commit(&bars->s_full);
            }
        }
    }
    mma_commit(&bars->mma_done);
    drain_wait(&bars->mma_done, 0, wc);
}

// Warps 0-7.  Thread = key row r of the block; `half` selects queries for P^T and dS^T, dV (0) or dK (1) when they leave,
// and columns of dQ at the end (thread = query row).
template <int D, int kNq>
__device__ void walk_softgrad(uint8_t* smem, WalkBarriers* bars, uint32_t tmem, float* __restrict__ dq_acc,
                              int head, int b0, int N, int klen, int T, float scale, float scale_log2, const BwdCross& ca) {
    using C = WalkCfg<D, kNq>;
    WaitCtl* wc = &bars->wait;
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int half = warp / 4, quarter = warp % 4;
    const int r = quarter * 32 + lane;
    const uint32_t lane_off = (uint32_t)(quarter * 32) << 16;
    const float* rows = reinterpret_cast<const float*>(smem + C::kOffRows);
    const uint64_t sl2 = f2_pack(scale_log2, scale_log2);
    uint64_t p2[HQ / 2];

    auto form_p = [&](int u) -> bool {
        const int j = u / kNq, k0 = (b0 + j) * BK;
        if (u % kNq == 0 && k0 + BK > klen && klen < N) {   // the block that the length cuts: clear what lies behind it
            const int s = j % C::kStages, from = klen - k0, chunks = (BK - from) * 8;
            if (!warp_wait(&bars->kv_full[s], (j / C::kStages) & 1, wc)) return false;
            uint8_t* tile = smem + C::kOffKV + s * 2 * C::kTile;
            for (int i = threadIdx.x; i < 2 * C::kChunks * chunks; i += 256)
                *reinterpret_cast<uint4*>(tile + (i / chunks) * C::kChunk + from * 128 + (i % chunks) * 16) = make_uint4(0, 0, 0, 0);
            fence_proxy_async_smem();
            mbar_arrive(&bars->kv_clean);
        }
        if (u == 0 && !warp_wait(&bars->q_full, 0, wc)) return false;
        if (!warp_wait(&bars->s_full, u & 1, wc)) return false;
        tc_fence_after();
        uint32_t sr[2][32];
        tmem_ld64(tmem + lane_off + C::kColS + half * HQ, sr);
        tmem_ld_wait();
        uint32_t pk[32];
        const float4* lse4 = reinterpret_cast<const float4*>(rows + (u % kNq) * BQ + half * HQ);
        const float keep = k0 + r < klen ? 0.f : -INFINITY;
#pragma unroll
        for (int c2 = 0; c2 < HQ / 4; ++c2) {
            const float4 l = lse4[c2];
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                const int c = 2 * c2 + u;
                const int q = (2 * c) / 32, e = (2 * c) % 32;
                const uint64_t x2 = ffma2(f2_pack(__uint_as_float(sr[q][e]), __uint_as_float(sr[q][e + 1])), sl2,
                                          u == 0 ? f2_pack(l.x, l.y) : f2_pack(l.z, l.w));
                float x0, x1;
                f2_unpack(x2, x0, x1);
                const float p0 = keep == 0.f ? ex2(x0) : 0.f, p1 = keep == 0.f ? ex2(x1) : 0.f;
                p2[c] = f2_pack(p0, p1);
                pk[c] = pack_bf16(p0, p1);
            }
        }
        tmem_st32(tmem + lane_off + C::kColS + half * HQ, pk);
        tmem_st_wait();
        tc_fence_before();
        mbar_arrive(&bars->p_ready);
        return true;
    };

    const int steps = T * kNq;
    bool ok = form_p(0);
    for (int u = 0; ok && u < steps; ++u) {
        // dS(u) = P(u) o (dP(u) - D).  The slot is free: this thread has waited for grad_full of the step before.
        if (!(ok = warp_wait(&bars->dp_full, u & 1, wc))) break;
        tc_fence_after();
        {
            const float4* drow4 = reinterpret_cast<const float4*>(rows + (kNq + u % kNq) * BQ + half * HQ);
            uint32_t pk[32];
            uint32_t dr[2][32];
            tmem_ld64(tmem + lane_off + C::kColDP + half * HQ, dr);
            tmem_ld_wait();
#pragma unroll
            for (int c2 = 0; c2 < HQ / 4; ++c2) {
                const float4 d4 = drow4[c2];
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    const int c = 2 * c2 + u;
                    const int q = (2 * c) / 32, e = (2 * c) % 32;
                    const uint64_t g2 = fadd2(f2_pack(__uint_as_float(dr[q][e]), __uint_as_float(dr[q][e + 1])),
                                              u == 0 ? f2_pack(d4.x, d4.y) : f2_pack(d4.z, d4.w));
                    float d0, d1;
                    f2_unpack(fmul2(p2[c], g2), d0, d1);
                    pk[c] = pack_bf16(d0, d1);
                }
            }
            tmem_st32(tmem + lane_off + C::kColDP + half * HQ, pk);
            uint8_t* row = smem + C::kOffDS + half * C::kChunk + r * 128;
#pragma unroll
            for (int ch = 0; ch < 8; ++ch)
                *reinterpret_cast<uint4*>(row + ((ch ^ (r & 7)) << 4)) =
                    make_uint4(pk[4 * ch], pk[4 * ch + 1], pk[4 * ch + 2], pk[4 * ch + 3]);
        }
        fence_proxy_async_smem();
        tmem_st_wait();
        tc_fence_before();
        mbar_arrive(&bars->ds_ready);

        if (C::kOwnDK && u + 1 < steps && !(ok = form_p(u + 1))) break;

        // dV and dK of the block, bf16, into the V and K tile's space as the tensor map has it: 64-column chunks of
        // 128-byte rows, 16-byte pieces XOR-swizzled by the row.  Zeros behind the entry's keys.
        if (!(ok = warp_wait(&bars->grad_full, u & 1, wc))) break;
        if (u % kNq < kNq - 1) continue;
        tc_fence_after();
        const int j = u / kNq;
        uint8_t* tile = smem + C::kOffKV + (j % C::kStages) * 2 * C::kTile + (half == 0 ? C::kTile : 0) + r * 128;
        const float mul = (b0 + j) * BK + r >= klen ? 0.f : half == 0 ? 1.f : scale;
        uint32_t w[D / 2];
#pragma unroll
        for (int q = 0; q < D / 32; ++q) {
            uint32_t y[32];
            tmem_ld32(tmem + lane_off + (half == 0 ? C::kColDV : C::kColDK) + q * 32, y);
            tmem_ld_wait();
#pragma unroll
            for (int e = 0; e < 16; ++e)
                w[q * 16 + e] = mul == 0.f ? 0u : pack_bf16(__uint_as_float(y[2 * e]) * mul, __uint_as_float(y[2 * e + 1]) * mul);
        }
        tc_fence_before();
        mbar_arrive(&bars->drained[half]);
#pragma unroll
        for (int c = 0; c < D / 8; ++c)
            *reinterpret_cast<uint4*>(tile + (c / 8) * C::kChunk + (((c % 8) ^ (r & 7)) << 4)) =
                make_uint4(w[4 * c], w[4 * c + 1], w[4 * c + 2], w[4 * c + 3]);
        fence_proxy_async_smem();
        mbar_arrive(&bars->staged[j % C::kStages]);

        if (!C::kOwnDK && u + 1 < steps && !(ok = form_p(u + 1))) break;
    }
    if (!ok) return;
    // dQ: complete (bf16), or added to the other CTAs' of this head.
    griddep_wait();   // the prep kernel has cleared the accumulator
#pragma unroll
    for (int n = 0; n < kNq; ++n) {
        uint32_t x[D / 64][32];
        const uint32_t col = C::kColDQ + n * D + (D / 2) * half;
        if constexpr (D == 128) tmem_ld64(tmem + lane_off + col, x);
        else tmem_ld32(tmem + lane_off + col, x[0]);
        tmem_ld_wait();
        if (n * BQ + r >= ca.R) continue;
        const size_t at = ((size_t)head * ca.R + n * BQ + r) * D + (D / 2) * half;
        if (ca.parts > 1) {
#pragma unroll
            for (int b = 0; b < D / 64; ++b)
#pragma unroll
                for (int e = 0; e < 32; e += 4)
                    red_add_f32x4(dq_acc + at + 32 * b + e, __uint_as_float(x[b][e]), __uint_as_float(x[b][e + 1]),
                                  __uint_as_float(x[b][e + 2]), __uint_as_float(x[b][e + 3]));
            continue;
        }
        uint4* dst = reinterpret_cast<uint4*>(ca.dq + at);
#pragma unroll
        for (int b = 0; b < D / 64; ++b)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                uint32_t w[4];
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    w[e] = pack_bf16(__uint_as_float(x[b][8 * i + 2 * e]) * scale, __uint_as_float(x[b][8 * i + 2 * e + 1]) * scale);
                dst[4 * b + i] = make_uint4(w[0], w[1], w[2], w[3]);
            }
    }
}

// ca.parts CTAs share the key blocks of a head: those below its entry's length, and those behind, which only get zeros.
template <int D, int kNq>
__global__ void __launch_bounds__(kThreads, 1)
bwd_walk_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ CUtensorMap tm_do,
                const __grid_constant__ CUtensorMap tm_dk, const __grid_constant__ CUtensorMap tm_dv,
                const float* lse2, const float* row_d, float* __restrict__ dq_acc,
                __nv_bfloat16* __restrict__ dk, __nv_bfloat16* __restrict__ dv, int N, int Npad, float scale,
                float scale_log2, long long wait_budget, int starve, BwdCross ca) {
    using C = WalkCfg<D, kNq>;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t pad = (1024 - (smem_u32(smem_raw) & 1023)) & 1023;
    if (pad > C::kAlignSlack) {   // as in bwd_tc_kernel
        if (threadIdx.x == 0) atomicCAS(&g_bwd_status, 0, (int)FA_ERR_CUDA);
        return;
    }
    uint8_t* smem = smem_raw + pad;
    WalkBarriers* bars = reinterpret_cast<WalkBarriers*>(smem + C::kOffBar);
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int head = (int)blockIdx.x / ca.parts, part = (int)blockIdx.x % ca.parts;
    const int klen = ca.key_lens ? min(max(ca.key_lens[head / ca.Hk], 0), N) : N;
    const int live = (klen + BK - 1) / BK, all = (N + BK - 1) / BK;
    const int b0 = (int)((long long)live * part / ca.parts);
    const int T = (int)((long long)live * (part + 1) / ca.parts) - b0;
    {
        const int dead = all - live;
        const int64_t r0 = (int64_t)(live + (int)((long long)dead * part / ca.parts)) * BK;
        const int64_t r1 = (int64_t)(live + (int)((long long)dead * (part + 1) / ca.parts)) * BK;
        const int64_t n16 = (min(r1, (int64_t)N) - r0) * (D / 8);   // negative where there are none
        const size_t at = ((size_t)head * N + r0) * D;
        for (int64_t i = threadIdx.x; i < n16; i += kThreads) {
            reinterpret_cast<uint4*>(dk + at)[i] = make_uint4(0, 0, 0, 0);
            reinterpret_cast<uint4*>(dv + at)[i] = make_uint4(0, 0, 0, 0);
        }
        if (ca.parts == 1 && live == 0)
            for (int64_t i = threadIdx.x; i < (int64_t)ca.R * (D / 8); i += kThreads)
                reinterpret_cast<uint4*>(ca.dq + (size_t)head * ca.R * D)[i] = make_uint4(0, 0, 0, 0);
        if (T == 0) {
            griddep_wait();   // the conversion kernel counts on this grid ending after the prep kernel
            return;
        }
    }
    if (threadIdx.x == 0) {
        bars->wait.budget = wait_budget;
        mbar_init(&bars->q_full, 1);
        for (int t = 0; t < 4; ++t) {
            mbar_init(&bars->kv_full[t], 1);
            mbar_init(&bars->staged[t], 256);
        }
        mbar_init(&bars->s_full, 1);
        mbar_init(&bars->dp_full, 1);
        mbar_init(&bars->p_ready, 256);
        mbar_init(&bars->ds_ready, 256);
        mbar_init(&bars->grad_full, 1);
        for (int t = 0; t < 2; ++t) mbar_init(&bars->drained[t], 128);
        mbar_init(&bars->mma_done, 1);
        mbar_init(&bars->kv_clean, 256);
        bars->wait.abort = 0;
        fence_mbar_init();
    }
    if (warp == kTmaWarp && lane == 0) {
        tma_prefetch_desc(&tm_q);
        tma_prefetch_desc(&tm_k);
        tma_prefetch_desc(&tm_v);
        tma_prefetch_desc(&tm_do);
    }
    if (warp == kMmaWarp) {
        tmem_alloc(&bars->tmem_base, C::kTmemCols);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = bars->tmem_base;

    if (warp == kTmaWarp) {
        if (lane == 0)
            walk_producer<D, kNq>(&tm_q, &tm_k, &tm_v, &tm_do, &tm_dk, &tm_dv, lse2, row_d, smem, bars, head, b0, T, Npad, starve);
    } else if (warp == kMmaWarp) {
        if (lane == 0) walk_mma<D, kNq>(smem, bars, tmem, T, (b0 + T) * BK > klen && klen < N);
    } else {
        walk_softgrad<D, kNq>(smem, bars, tmem, dq_acc, head, b0, N, klen, T, scale, scale_log2, ca);
    }

    tc_fence_before();
    __syncthreads();
    if (warp == kMmaWarp) {
        tc_fence_after();
        tmem_dealloc(tmem, C::kTmemCols);
    }
    if (threadIdx.x == 0 && bars->wait.abort) atomicCAS(&g_bwd_status, 0, (int)FA_ERR_TIMEOUT);
}

// -D_i = -(dO_i . O_i) and -LSE2_i = -LSE_i log2(e) into [head][Npad] arrays (pad rows: 0 and -inf);
// zeroes n4 times four floats of the dQ accumulator (all of it, or none).  D/8 threads share a row (16-byte loads of O and
// dO), each warp takes 2 * 32 / (D/8) rows per pass, so enough bytes are in flight to stream at HBM speed.
template <int D>
__global__ void bwd_prep_kernel(const __nv_bfloat16* __restrict__ o, const __nv_bfloat16* __restrict__ dout,
                                const float* __restrict__ lse, float* __restrict__ row_d, float* __restrict__ lse2,
                                float* __restrict__ dq_acc, int N, int Npad, int64_t heads, int64_t n4) {
    griddep_launch_dependents();
    constexpr int kTpr = D / 8;          // threads per row
    constexpr int kRpw = 32 / kTpr;      // rows per warp and pass
    const int lane = threadIdx.x & 31;
    const int sub = lane / kTpr, part = lane % kTpr;
    const int64_t nwarps = (int64_t)gridDim.x * (blockDim.x >> 5);
    const int64_t warp_id = (int64_t)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5);
    const int64_t rows = heads * Npad;
    for (int64_t base = warp_id * 2 * kRpw; base < rows; base += nwarps * 2 * kRpw) {
        float acc[2];
        int64_t w[2];
        bool valid[2];
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            w[u] = base + u * kRpw + sub;
            const int64_t h = w[u] / Npad;
            const int r = (int)(w[u] - h * Npad);
            valid[u] = w[u] < rows && r < N;
            acc[u] = 0.f;
            if (valid[u]) {
                const size_t off = ((size_t)h * N + r) * D + part * 8;
                const uint4 a = *reinterpret_cast<const uint4*>(o + off);
                const uint4 g = *reinterpret_cast<const uint4*>(dout + off);
                const __nv_bfloat162* a2 = reinterpret_cast<const __nv_bfloat162*>(&a);
                const __nv_bfloat162* g2 = reinterpret_cast<const __nv_bfloat162*>(&g);
#pragma unroll
                for (int t = 0; t < 4; ++t) {
                    const float2 fa = __bfloat1622float2(a2[t]), fg = __bfloat1622float2(g2[t]);
                    acc[u] = fmaf(fa.x, fg.x, fmaf(fa.y, fg.y, acc[u]));
                }
            }
        }
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
            for (int off = kTpr / 2; off; off >>= 1) acc[u] += __shfl_xor_sync(0xffffffffu, acc[u], off);
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            if (part != 0 || w[u] >= rows) continue;
            const int64_t h = w[u] / Npad;
            const int r = (int)(w[u] - h * Npad);
            row_d[w[u]] = valid[u] ? -acc[u] : 0.f;
            lse2[w[u]] = valid[u] ? -lse[(size_t)h * N + r] * 1.4426950408889634f : -INFINITY;
        }
    }
    float4* z = reinterpret_cast<float4*>(dq_acc);
    for (int64_t idx = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; idx < n4; idx += (int64_t)gridDim.x * blockDim.x)
        z[idx] = make_float4(0.f, 0.f, 0.f, 0.f);
}

// dK and dV of every key from the parts' shares, added in order: four columns a thread.  Keys past an entry's length: zeros.
template <int D>
__global__ void __launch_bounds__(256) bwd_join_kernel(const __grid_constant__ BwdCross ca, __nv_bfloat16* __restrict__ dk,
                                                       __nv_bfloat16* __restrict__ dv, int N, int blocks_per_head,
                                                       int64_t n4, float scale) {
    griddep_wait();
    const int64_t idx = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (idx >= n4) return;
    const int64_t row = idx / (D / 4);
    const int c = (int)(idx - row * (D / 4)) * 4;
    const int64_t head = row / N;
    const int key = (int)(row - head * N);
    const int klen = ca.key_lens ? ca.key_lens[head / ca.Hk] : N;
    float4 s[2] = {make_float4(0.f, 0.f, 0.f, 0.f), make_float4(0.f, 0.f, 0.f, 0.f)};
    if (key < klen) {
        const float* src = ca.part + (size_t)(head * blocks_per_head + key / BK) * ca.parts * (2 * BK * D) + (key % BK) * D + c;
        for (int p = 0; p < ca.parts; ++p, src += 2 * BK * D)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const float4 x = *reinterpret_cast<const float4*>(src + h * (BK * D));
                s[h].x += x.x;
                s[h].y += x.y;
                s[h].z += x.z;
                s[h].w += x.w;
            }
    }
    const uint2 v = make_uint2(pack_bf16(s[0].x, s[0].y), pack_bf16(s[0].z, s[0].w));
    const uint2 k = make_uint2(pack_bf16(s[1].x * scale, s[1].y * scale), pack_bf16(s[1].z * scale, s[1].w * scale));
    reinterpret_cast<uint2*>(dv)[idx] = v;
    reinterpret_cast<uint2*>(dk)[idx] = k;
}

// dQ = bf16(scale * accumulator), four elements per thread and load, grid-stride.  The kernel ahead still adds to the
// accumulator when this one starts, so it is not read-only memory: no __restrict__, plain loads from L2, and kLoads of them in
// flight by hand.
__global__ void bwd_dq_convert_kernel(const float* dq_acc, __nv_bfloat16* __restrict__ dq, float scale, int64_t n4) {
    constexpr int kLoads = 4;
    griddep_wait();   // launched to start while the main kernel finishes: its reduce-adds must be complete
    const int64_t step = (int64_t)gridDim.x * blockDim.x;
    for (int64_t i0 = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i0 < n4; i0 += kLoads * step) {
        float4 a[kLoads];
#pragma unroll
        for (int u = 0; u < kLoads; ++u)
            if (i0 + u * step < n4) a[u] = __ldcg(reinterpret_cast<const float4*>(dq_acc) + i0 + u * step);
#pragma unroll
        for (int u = 0; u < kLoads; ++u) {
            uint2 out;
            out.x = pack_bf16(a[u].x * scale, a[u].y * scale);
            out.y = pack_bf16(a[u].z * scale, a[u].w * scale);
            if (i0 + u * step < n4) reinterpret_cast<uint2*>(dq)[i0 + u * step] = out;
        }
    }
}

// s: the queries' rows; Nk keys (kCross: of another number, with the lengths in ca).
template <int D, bool kCross, bool kDirect>
cudaError_t launch(const void* q, const void* k, const void* v, const void* o, const void* dout, const float* lse,
                   void* dq, void* dk, void* dv, const Shape& s, int Nk, float scale, void* workspace, cudaStream_t st,
                   BwdTiming timing, BwdCross ca = {}) {
    using C = BwdCfg<D>;
    const BwdWorkspace w = bwd_workspace_layout(s);
    char* ws = (char*)workspace;
    float* dq_acc = (float*)(ws + w.dq_acc);
    float* row_d = (float*)(ws + w.row_d);
    float* lse2 = (float*)(ws + w.lse2);
    const int Npad = bwd_padded_rows(s.N);
    const int blocks = device_sm_count() * 4;
    const int bph = (Nk + BK - 1) / BK;
    ca.dq = (__nv_bfloat16*)dq;
    const int64_t n4 = s.heads() * (int64_t)s.N * D / 4;
    bwd_prep_kernel<D><<<blocks, 256, 0, st>>>((const __nv_bfloat16*)o, (const __nv_bfloat16*)dout, lse, row_d,
                                               lse2, dq_acc, s.N, Npad, s.heads(), kDirect ? 0 : n4);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    count_launches(1);

    CUtensorMap tq, tk, tv, tdo, tdq;
    constexpr auto make_map = kCross ? encode_tmap_bf16_3d : make_tmap_bf16_3d;
    constexpr auto make_map_f32 = kCross ? encode_tmap_f32_3d : make_tmap_f32_3d;
    if ((e = make_map(&tq, q, s.d, s.N, s.heads(), BQ)) != cudaSuccess) return e;
    if ((e = make_map(&tdo, dout, s.d, s.N, s.heads(), BQ)) != cudaSuccess) return e;
    if ((e = make_map(&tk, k, s.d, Nk, s.heads(), BK)) != cudaSuccess) return e;
    if ((e = make_map(&tv, v, s.d, Nk, s.heads(), BK)) != cudaSuccess) return e;
    // The dQ staging boxes: [BQ rows][32 columns], 128-byte swizzled.
    if ((e = make_map_f32(&tdq, dq_acc, s.d, s.N, s.heads(), 32, BQ, true)) != cudaSuccess)
        return e;
    e = set_max_dynamic_smem((const void*)bwd_tc_kernel<D, kCross, kDirect>, (int)C::kSmemBytes);
    if (e != cudaSuccess) return e;
    if ((long long)bph * s.heads() > INT32_MAX) return cudaErrorInvalidConfiguration;
    const int parts = kCross ? ca.parts : 1;
    if ((long long)bph * s.heads() * parts > INT32_MAX) return cudaErrorInvalidConfiguration;
    const unsigned grid = (unsigned)(bph * s.heads() * parts);
    const WaitPolicy wp = wait_policy();
    if (timing.start && (e = cudaEventRecord(timing.start, st)) != cudaSuccess) return e;
    if ((e = launch_dependent(bwd_tc_kernel<D, kCross, kDirect>, dim3(grid), dim3(kThreads), C::kSmemBytes, st, tq, tk, tv, tdo, tdq,
                              lse2, row_d, dq_acc, (__nv_bfloat16*)dk, (__nv_bfloat16*)dv, Nk, Npad, bph, scale,
                              scale * 1.4426950408889634f, wp.budget_cycles, wp.starve, ca)) != cudaSuccess)
        return e;
    count_launches(1);
    if (timing.stop && (e = cudaEventRecord(timing.stop, st)) != cudaSuccess) return e;
    if (!kDirect) {
        if ((e = launch_dependent(bwd_dq_convert_kernel, dim3(blocks), dim3(256), 0, st, dq_acc, (__nv_bfloat16*)dq, scale,
                                  n4)) != cudaSuccess)
            return e;
        count_launches(1);
    }
    if (parts > 1) {
        // An ordinary launch, behind both kernels.
        const int64_t k4 = s.heads() * (int64_t)Nk * (D / 4);
        bwd_join_kernel<D><<<(unsigned)((k4 + 255) / 256), 256, 0, st>>>(ca, (__nv_bfloat16*)dk, (__nv_bfloat16*)dv, Nk, bph,
                                                                         k4, scale);
        if ((e = cudaGetLastError()) != cudaSuccess) return e;
        count_launches(1);
    }
    return cudaSuccess;
}

// Heads of one query block (d = 64: of two) over many keys.
template <int D, int kNq>
cudaError_t launch_walk(const CrossBwd& c, void* workspace, cudaStream_t st, BwdCross ca) {
    using C = WalkCfg<D, kNq>;
    const Shape s{c.f.B, c.f.Hk, c.f.rows(), c.f.d};
    const BwdWorkspace w = bwd_workspace_layout(s);
    char* ws = (char*)workspace;
    float* dq_acc = (float*)(ws + w.dq_acc);
    float* row_d = (float*)(ws + w.row_d);
    float* lse2 = (float*)(ws + w.lse2);
    const int Npad = bwd_padded_rows(s.N);
    const int blocks = device_sm_count() * 4;
    const int64_t n4 = ca.parts > 1 ? s.heads() * (int64_t)s.N * D / 4 : 0;
    ca.dq = (__nv_bfloat16*)c.dq;
    if (s.heads() * ca.parts > INT32_MAX) return cudaErrorInvalidConfiguration;
    bwd_prep_kernel<D><<<blocks, 256, 0, st>>>((const __nv_bfloat16*)c.f.o, (const __nv_bfloat16*)c.dout, c.f.lse, row_d, lse2,
                                               dq_acc, s.N, Npad, s.heads(), n4);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    count_launches(1);
    CUtensorMap tq, tk, tv, tdo, tdk, tdv;
    if ((e = encode_tmap_bf16_3d(&tq, c.f.q, D, s.N, s.heads(), BQ)) != cudaSuccess) return e;
    if ((e = encode_tmap_bf16_3d(&tdo, c.dout, D, s.N, s.heads(), BQ)) != cudaSuccess) return e;
    if ((e = encode_tmap_bf16_3d(&tk, c.f.k, D, c.f.Nk, s.heads(), BK)) != cudaSuccess) return e;
    if ((e = encode_tmap_bf16_3d(&tv, c.f.v, D, c.f.Nk, s.heads(), BK)) != cudaSuccess) return e;
    if ((e = encode_tmap_bf16_3d(&tdk, c.dk, D, c.f.Nk, s.heads(), BK)) != cudaSuccess) return e;
    if ((e = encode_tmap_bf16_3d(&tdv, c.dv, D, c.f.Nk, s.heads(), BK)) != cudaSuccess) return e;
    if ((e = set_max_dynamic_smem((const void*)bwd_walk_kernel<D, kNq>, (int)C::kSmemBytes)) != cudaSuccess) return e;
    const WaitPolicy wp = wait_policy();
    if ((e = launch_dependent(bwd_walk_kernel<D, kNq>, dim3((unsigned)(s.heads() * ca.parts)), dim3(kThreads), C::kSmemBytes, st, tq, tk,
                              tv, tdo, tdk, tdv, lse2, row_d, dq_acc, (__nv_bfloat16*)c.dk, (__nv_bfloat16*)c.dv, c.f.Nk, Npad,
                              c.f.scale, c.f.scale * 1.4426950408889634f, wp.budget_cycles, wp.starve, ca)) != cudaSuccess)
        return e;
    count_launches(1);
    if (ca.parts > 1) {
        if ((e = launch_dependent(bwd_dq_convert_kernel, dim3(blocks), dim3(256), 0, st, dq_acc, ca.dq, c.f.scale, n4)) !=
            cudaSuccess)
            return e;
        count_launches(1);
    }
    return cudaSuccess;
}

}  // namespace

cudaError_t launch_bwd_tc(const void* q, const void* k, const void* v, const void* o, const void* dout,
                          const float* lse, void* dq, void* dk, void* dv, const Shape& s, float scale,
                          void* workspace, cudaStream_t st, BwdTiming timing) {
    return s.d == 128 ? launch<128, false, false>(q, k, v, o, dout, lse, dq, dk, dv, s, s.N, scale, workspace, st, timing)
                      : launch<64, false, false>(q, k, v, o, dout, lse, dq, dk, dv, s, s.N, scale, workspace, st, timing);
}

BwdCrossPlan bwd_cross_plan(int64_t heads, int R, int d, int Nk) {
    const Shape s{1, (int)heads, R, d};
    BwdCrossPlan p = {1, 0, 0, bwd_workspace_layout(s).total};
    // Less than half a wave of key blocks: as many parts of the query axis as fill one, of four steps each or more.
    const int64_t ctas = heads * ((Nk + BK - 1) / BK);
    const int steps = bwd_padded_rows(R) / BQ;
    if (2 * ctas <= kPlanSms) {
        const int64_t fill = kPlanSms / ctas, most = steps / 4;
        p.parts = (int)(fill < most ? fill : most);
        if (p.parts < 1) p.parts = 1;
    }
    // Few query blocks and more key blocks than SMs: as many CTAs a head as is estimated shortest.  A CTA's set-up takes 5 us,
    // a key block what block_us says, converting dQ 2.  64 heads of 64 rows, us with a CTA a key block and so, d = 64: 600 keys
    // 19.8, 14.1; 2000 40.8, 23.7; 8000 155, 69; d = 128: 25.1, 18.1; 61.6, 36.2; 202, 111.  At one key block dQ leaves at once
    // (13.1 against 13.5 us, 200 heads of 64 rows over 64 keys).
    if (R <= (d == 64 ? 2 : 1) * BQ && Nk > BK && ctas > kPlanSms) {
        const int64_t blocks = (Nk + BK - 1) / BK;
        const double block_us = d == 128 ? 3.8 : R <= BQ ? 1.95 : 3.5;
        double best = 1e30;
        for (int n = 1; n <= 64 && n <= blocks; ++n) {
            const double us = (double)((heads * n + kPlanSms - 1) / kPlanSms) *
                                  (5 + (double)((blocks + n - 1) / n) * block_us) + (n > 1 ? 2 : 0);
            if (us < best) {
                best = us;
                p.walk = n;
            }
        }
    }
    if (p.parts > 1) {
        p.part_offset = p.bytes;
        p.bytes += (size_t)ctas * p.parts * (2 * BK * sizeof(float)) * d;
    }
    return p;
}

cudaError_t launch_cross_bwd(const CrossBwd& c, void* workspace, cudaStream_t st) {
    const Shape s{c.f.B, c.f.Hk, c.f.rows(), c.f.d};
    const BwdCrossPlan p = bwd_cross_plan(c.f.heads(), c.f.rows(), c.f.d, c.f.Nk);
    BwdCross ca{c.f.key_lens, c.f.Hk, p.parts, (float*)((char*)workspace + p.part_offset), nullptr, c.f.rows()};
    if (p.walk) {
        ca.parts = p.walk;
        auto* f = c.f.d == 128 ? launch_walk<128, 1> : c.f.rows() <= BQ ? launch_walk<64, 1> : launch_walk<64, 2>;
        return f(c, workspace, st, ca);
    }
    const bool direct = c.f.Nk <= BK;
    auto* f = c.f.d == 128 ? (direct ? launch<128, true, true> : launch<128, true, false>)
                           : (direct ? launch<64, true, true> : launch<64, true, false>);
    return f(c.f.q, c.f.k, c.f.v, c.f.o, c.dout, c.f.lse, c.dq, c.dk, c.dv, s, c.f.Nk, c.f.scale, workspace, st,
             BwdTiming{nullptr, nullptr}, ca);
}

int bwd_tc_read_and_clear_status(cudaStream_t st) {
    int v = 0, zero = 0;
    if (cudaMemcpyFromSymbolAsync(&v, g_bwd_status, sizeof(int), 0, cudaMemcpyDeviceToHost, st) != cudaSuccess)
        return -1;
    if (cudaMemcpyToSymbolAsync(g_bwd_status, &zero, sizeof(int), 0, cudaMemcpyHostToDevice, st) != cudaSuccess)
        return -1;
    if (cudaStreamSynchronize(st) != cudaSuccess) return -1;
    return v;
}

}  // namespace fa
