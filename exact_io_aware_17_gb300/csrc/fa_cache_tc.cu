// Attention of 33 and more query rows a key head over the paged 8-bit cache (fa_cache_fwd): wide groups of query heads, or
// several tokens a step.
//
//     S = scale Q K^T,  m = max S,  l = sum exp(S - m),  O = sum exp(S - m) V / l,  LSE = m + ln l
//
// The warps' streams of fa_rows.cu read and unpack the cache once for every 16 rows and are bound by that.  Here a CTA takes
// up to 128 rows of a key head as the M of tcgen05 products: the cache is read and unpacked once, so the bound is HBM
// again, nearly.  64 requests of 8192 tokens each x 8 heads (1.07 GB), d = 128, us in streams and here: 48 rows 425, 296
// (3.6 TB/s), 64 rows 535, 299, 128 rows 1019, 424.  A tile takes 1.0 us, the row warps' chain from S to P, where HBM would
// take 0.73; set-up and write-out of a CTA take 7 us, which only one CTA an SM does not overlap.
//
// Eight warps convert: each loads the codes of 32 of a tile's 128 keys or values two tiles ahead into registers, turns them
// into f16 (exact) and writes them to shared memory in the products' layout, three tiles of 64 KB (K and V, d = 128).  A
// thread forms S of the next tile before P V of this one.  Four warps hold a row a lane: running maximum and sum, P to
// tensor memory as f16.  Up to 64 rows stand in the lanes twice, and each copy takes half of a tile's keys (P of the others
// is zero), with a maximum, sum and O of its own until the end, so that four warps share the softmax and not two.  Q is f16
// too, scaled by a power of two per row, so that elements down to 2^-29 of the row's largest are exact.
//
// A key block's scale multiplies its scores, a value block's its probabilities: P is 2^(s + log2 scale - u), with the row's
// running maximum u of s + log2 scale over the keys that it sees, as in fa_rows.cu.  O is rescaled only when u has grown by
// more than 8 (P then stays within f16's range with 2^7 to spare for small ones; f16 drops what is below 2^-32 of the row's
// largest).

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <math.h>

#include "fa_internal.h"
#include "fa_ptx.cuh"

namespace fa {
namespace {

using namespace ptx;

__device__ int g_cache_status;

constexpr int BM = 128;           // query rows of a CTA (tensor-memory lanes)
constexpr int BN = 128;           // keys of a tile
constexpr int kMmaWarp = 4, kFirstConverter = 5, kConverters = 8;   // warps; 0-3 are the rows'; four convert K, four V
constexpr int kStages = 3;        // tiles of K, and of V, in shared memory
constexpr int kScaleSlots = 8;    // of tiles' scales: those of K are up to four tiles ahead of the softmax
constexpr int kThreads = 32 * (kFirstConverter + kConverters);
constexpr float kGrowth = 8.f;    // log2 units by which a maximum may grow before l or O follows
constexpr float kPScale = 128.f;  // of probabilities in f16: with 2^8 for the growth at most 2^15
constexpr float kMaxFloat = 3.402823466e38f;

struct CacheBarriers {
    uint64_t q_full;              // 128 arrivals
    uint64_t full[2][kStages];    // a tile of K, of V is in its buffer (128 arrivals)
    uint64_t free[2][kStages];    // the product that reads it is done
    uint64_t s_full[2];
    uint64_t p_full[2];           // P is in tensor memory (32 arrivals for each warp with rows)
    uint64_t pv_done[2];          // P V is done: its P buffer is free, O is complete so far
    uint64_t joined;              // the copies' results are in shared memory (128 arrivals)
    uint64_t mma_done;
    uint32_t tmem_base;
    int new_nan;                  // a value of the newest tokens is NaN
    WaitCtl wait;
};

template <int D>
struct CacheCfg {
    static constexpr int kChunks = D / 64;
    static constexpr uint32_t kChunk = 128 * 128;             // 64 columns of a tile
    static constexpr uint32_t kTile = kChunks * kChunk;
    static constexpr uint32_t kOffQ = 0, kOffKV = kTile;   // stages of K, then of V
    static constexpr uint32_t kOffScale = kOffKV + 2 * kStages * kTile;   // [K, V][slot][group of 16 keys]
    static constexpr uint32_t kOffBar = kOffScale + 2 * kScaleSlots * 8 * 4;
    static constexpr uint32_t kSmemNeed = kOffBar + sizeof(CacheBarriers);
    static constexpr uint32_t kSmemBytes = kSmemNeed + (kSmemNeed + 1024 <= 232448 ? 1024 : 232448 - kSmemNeed);   // room to align
    static_assert(kSmemNeed <= 232448, "shared memory per CTA");
    static constexpr uint32_t kColP = 256, kColO = 384;       // S: 0 and 128
};

struct CacheTcArgs {
    const __nv_bfloat16* q;           // [BH][R][D]
    __nv_bfloat16* o;
    float* lse;                       // [BH][R]
    const uint8_t *k, *v;             // [block][head][token][D] e4m3
    const float *k_scale, *v_scale;   // [block][head]
    const int *table, *lens;
    float* part_o;                    // [BH][row tile][split][tile_rows][D]
    float2* part_ml;
    int R, N, Hk, cap, bs_log2, max_blocks, n_blocks, splits, row_tiles, tile_rows;
    float scale_log2;
    long long wait_budget;
    int starve;
};

// Two e4m3 codes (the low or high half of w) as two f16.
__device__ __forceinline__ uint32_t codes_f16(uint32_t w, int high) {
    uint32_t r;
    if (high) asm("{.reg .b16 l, h;\n\tmov.b32 {l, h}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, h;\n\t}" : "=r"(r) : "r"(w));
    else asm("{.reg .b16 l, h;\n\tmov.b32 {l, h}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, l;\n\t}" : "=r"(r) : "r"(w));
    return r;
}
// log2 of a power of two (of 0: -127), from its exponent bits: 2^23 + them is exact.
__device__ __forceinline__ float log2_scale(float x) {
    return __uint_as_float(0x4b000000u | __float_as_uint(x) >> 23) - (8388608.f + 127.f);
}
__device__ __forceinline__ uint32_t f16x2(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
// (Not the read-only path: an append ahead on the stream may still be writing when this kernel starts.)
__device__ __forceinline__ uint4 load_codes(const uint8_t* p) {
    uint4 r;
    asm volatile("ld.global.L1::no_allocate.v4.b32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w)
                 : "l"(p)
                 : "memory");
    return r;
}
// Codes that are NaN (all bits but the sign) become zero; *any says that there was one.
__device__ __forceinline__ uint32_t drop_nan(uint32_t w, uint32_t* any) {
    const uint32_t nan = ((w & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u;
    *any |= nan;
    return w & ~((nan >> 7) * 255u);
}

// A converter warp of K (kv = 0) or V: keys 32 part .. 32 part + 31 of each tile from i0 to i1 - 1.
template <int D>
__device__ void cache_convert(const CacheTcArgs& a, uint8_t* smem, CacheBarriers* bars, int kv, int part, int b, int hk, int len,
                              int limit_all, int i0, int i1) {
    using C = CacheCfg<D>;
    constexpr int kPieces = D / 16, kRows = 32 / kPieces, kLoads = 32 / kRows;   // 16-byte pieces of a row; rows of a load
    WaitCtl* wc = &bars->wait;
    // Row and piece of a lane: eight lanes that store together have four pieces of an even row and the next one's, which
    // the swizzle puts into different banks.
    const int lane = threadIdx.x & 31;
    const int sub = D == 128 ? (lane >> 2 & 1) + 2 * (lane >> 4) : lane >> 2;
    const int piece = D == 128 ? (lane & 3) + (lane >> 1 & 4) : lane & 3;
    const int* trow = a.table + (size_t)b * a.max_blocks;
    const uint8_t* codes = kv ? a.v : a.k;
    const float* block_scales = kv ? a.v_scale : a.k_scale;
    float* scales = reinterpret_cast<float*>(smem + C::kOffScale) + kv * kScaleSlots * 8 + 2 * part;
    auto block_of = [&](int i, int u) -> int {
        const int key = min(i, i1) * BN + 32 * part + 16 * u;
        const int p = i < i1 && key < len ? trow[key >> a.bs_log2] : -1;
        return (unsigned)p < (unsigned)a.n_blocks ? p : -1;
    };
    struct Held {
        uint4 c[kLoads];
        float scale;   // of the half that the lane stands for: lanes 0 and 1
    } held[2];
    int next[2][2];   // blocks of the next two tiles to load
#pragma unroll
    for (int n = 0; n < 2; ++n)
#pragma unroll
        for (int u = 0; u < 2; ++u) next[n][u] = block_of(i0 + n, u);
    int first[4];     // and of those to ask for at the start
    // Further ahead, a lane a 128-byte line (d = 64: every other lane), the codes are asked into L2.
    constexpr int kAhead = 6, kLines = 16 * D / 128;   // lines of 16 keys
    auto ahead_of = [&](int i) { return block_of(i, lane / 16); };
    auto ask = [&](int block, int i) {
        const int key = (min(i, i1) * BN + 32 * part + 16 * (lane / 16)) & ((1 << a.bs_log2) - 1);
        if (block >= 0 && lane % 16 < kLines) {
            const uint8_t* p = codes + ((((size_t)block * a.Hk + hk) << a.bs_log2) + key) * D + lane % 16 * 128;
            asm volatile("prefetch.global.L2 [%0];" ::"l"(p));
        }
    };
    static_assert(kAhead == 6, "two tiles load at once, four are asked for");
#pragma unroll
    for (int n = 0; n < 4; ++n) first[n] = ahead_of(i0 + 2 + n);
    int ahead = ahead_of(i0 + kAhead);
    auto load = [&](Held& h, int i, const int (&block)[2]) {   // the codes of tile i, zeros where there is no token
        const int key = min(i, i1) * BN + 32 * part, mine = lane & 1 ? block[1] : block[0];
        h.scale = mine >= 0 ? block_scales[(size_t)mine * a.Hk + hk] : kv ? 0.f : -1.f;
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            const int at_key = key + 16 * u;
            const uint8_t* src = codes + ((((size_t)max(block[u], 0) * a.Hk + hk) << a.bs_log2) +
                                          (at_key & ((1 << a.bs_log2) - 1)) + sub) * D + piece * 16;
#pragma unroll
            for (int n = 0; n < kLoads / 2; ++n)
                h.c[u * (kLoads / 2) + n] = block[u] >= 0 && at_key + sub + n * kRows < len ? load_codes(src + n * kRows * D)
                                                                                        : make_uint4(0, 0, 0, 0);
        }
    };
    auto step = [&](Held& h, int i) -> bool {
        const int j = i - i0, s = j % kStages;
        if (j >= kStages && !warp_wait(&bars->free[kv][s], (j / kStages - 1) & 1, wc)) return false;
        const int key = i * BN + 32 * part;
        if (kv && key + 32 > limit_all && limit_all < len) {
            // Newest tokens, which not every row sees: an unseen NaN would reach every row as 0 * NaN.
            uint32_t any = 0;
#pragma unroll
            for (int n = 0; n < kLoads; ++n)
                if (key + sub + n * kRows >= limit_all) {
                    h.c[n].x = drop_nan(h.c[n].x, &any);
                    h.c[n].y = drop_nan(h.c[n].y, &any);
                    h.c[n].z = drop_nan(h.c[n].z, &any);
                    h.c[n].w = drop_nan(h.c[n].w, &any);
                }
            if (any) bars->new_nan = 1;
        }
        uint8_t* tile = smem + C::kOffKV + (kv * kStages + s) * C::kTile + (piece / 4) * C::kChunk;
#pragma unroll
        for (int n = 0; n < kLoads; ++n) {
            const int row = 32 * part + sub + n * kRows;
            const uint32_t w[4] = {h.c[n].x, h.c[n].y, h.c[n].z, h.c[n].w};
#pragma unroll
            for (int e = 0; e < 2; ++e)
                *reinterpret_cast<uint4*>(tile + row * 128 + ((((piece % 4) * 2 + e) ^ (row & 7)) << 4)) =
                    make_uint4(codes_f16(w[2 * e], 0), codes_f16(w[2 * e], 1), codes_f16(w[2 * e + 1], 0),
                               codes_f16(w[2 * e + 1], 1));
        }
        if (lane < 2) scales[j % kScaleSlots * 8 + lane] = h.scale;
        fence_proxy_async_smem();
        mbar_arrive(&bars->full[kv][s]);
        load(h, i + 2, next[0]);
        next[0][0] = block_of(i + 3, 0);
        next[0][1] = block_of(i + 3, 1);
        ask(ahead, i + kAhead);
        ahead = ahead_of(i + kAhead + 1);
        return true;
    };
    load(held[0], i0, next[0]);
    load(held[1], i0 + 1, next[1]);
#pragma unroll
    for (int n = 0; n < 4; ++n) ask(first[n], i0 + 2 + n);
    next[0][0] = block_of(i0 + 2, 0);
    next[0][1] = block_of(i0 + 2, 1);
    for (int i = i0; i < i1; i += 2) {
        if (!step(held[0], i)) return;
        if (i + 1 < i1 && !step(held[1], i + 1)) return;
    }
}

template <int D>
__device__ void cache_mma(uint8_t* smem, CacheBarriers* bars, uint32_t tmem, int T) {
    using C = CacheCfg<D>;
    WaitCtl* wc = &bars->wait;
    constexpr uint32_t kF16 = ~((1u << 7) | (1u << 10));   // f16 operands in the place of bf16
    constexpr uint32_t idS = idesc_bf16_f32(BM, BN, 0, 0) & kF16, idPV = idesc_bf16_f32(BM, D, 0, 1) & kF16;
    const uint64_t q0 = sdesc_sw128(smem_u32(smem + C::kOffQ), 16, 1024);
    const uint64_t k0 = sdesc_sw128(smem_u32(smem + C::kOffKV), 16, 1024);
    const uint64_t v0 = sdesc_sw128(smem_u32(smem + C::kOffKV + kStages * C::kTile), C::kChunk, 1024);
    auto scores = [&](int j) {
        const int s = j & 1, stage = j % kStages;
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
            const uint32_t at = (kk / 4) * C::kChunk + (kk % 4) * 32;
            mma_ss(tmem + 128 * s, sdesc_advance(q0, at), sdesc_advance(k0, stage * C::kTile + at), idS, kk > 0);
        }
        mma_commit(&bars->s_full[s]);
        mma_commit(&bars->free[0][stage]);
    };
    bool ok = mbar_wait_poll(&bars->q_full, 0, wc) && mbar_wait_poll(&bars->full[0][0], 0, wc);
    if (ok) {
        tc_fence_after();
        scores(0);
    }
    for (int j = 0; ok && j < T; ++j) {
        const int s = j & 1;
        if (j + 1 < T) {
            if (!(ok = mbar_wait_poll(&bars->full[0][(j + 1) % kStages], ((j + 1) / kStages) & 1, wc))) break;
            tc_fence_after();
            scores(j + 1);
        }
        const int stage = j % kStages;
        if (!(ok = mbar_wait_poll(&bars->full[1][stage], (j / kStages) & 1, wc))) break;
        if (!(ok = mbar_wait_poll(&bars->p_full[s], (j >> 1) & 1, wc))) break;
        tc_fence_after();
#pragma unroll
        for (int kk = 0; kk < BN / 16; ++kk)
            mma_ts(tmem + C::kColO, tmem + C::kColP + 64 * s + kk * 8, sdesc_advance(v0, stage * C::kTile + kk * 16 * 128), idPV,
                   (j > 0 || kk > 0) ? 1u : 0u);
        mma_commit(&bars->free[1][stage]);
        mma_commit(&bars->pv_done[s]);
    }
    mma_commit(&bars->mma_done);
    drain_wait(&bars->mma_done, 0, wc);
}

// Row r of the tile, a lane of tensor memory: loads and scales its Q, then the softmax, then its output.
// kCopies: the rows stand once or twice among the lanes.
template <int D, int kCopies>
__device__ void cache_row(const CacheTcArgs& a, uint8_t* smem, CacheBarriers* bars, uint32_t tmem, int b, int hk, int row0,
                          int len, int limit_all, int i0, int i1) {
    using C = CacheCfg<D>;
    WaitCtl* wc = &bars->wait;
    const int r = threadIdx.x, bh = b * a.Hk + hk, T = i1 - i0;
    constexpr int copy_rows = BM / kCopies, chunks = 4 / kCopies;   // of 32 keys, that this warp takes
    const int row = row0 + r % copy_rows, c0 = r / copy_rows * chunks;
    const uint32_t lane_off = (uint32_t)(r & ~31) << 16;
    const bool mine = row < a.R;

    float qscale;
    {
        const __nv_bfloat16* src = a.q + ((size_t)bh * a.R + row) * D;
        float amax = 0.f;
#pragma unroll
        for (int i = 0; i < D / 8; ++i) {
            const uint4 w4 = mine ? *reinterpret_cast<const uint4*>(src + 8 * i) : make_uint4(0, 0, 0, 0);
            const uint32_t w[4] = {w4.x, w4.y, w4.z, w4.w};
#pragma unroll
            for (int j = 0; j < 4; ++j)
                amax = max3(amax, fabsf(__uint_as_float(w[j] << 16)), fabsf(__uint_as_float(w[j] & 0xffff0000u)));
        }
        // mul = 2^(14 - exponent of amax), kept a normal number.  A NaN among the elements is one in f16 too.
        const int ex = min(max((int)(__float_as_uint(amax) >> 23) - 127, -100), 127);
        const float mul = __uint_as_float((uint32_t)(min(14 - ex, 100) + 127) << 23);
        qscale = amax <= kMaxFloat ? a.scale_log2 / mul : __int_as_float(0x7fc00000);
#pragma unroll
        for (int i = 0; i < D / 8; ++i) {
            const uint4 w4 = mine ? *reinterpret_cast<const uint4*>(src + 8 * i) : make_uint4(0, 0, 0, 0);
            const uint32_t w[4] = {w4.x, w4.y, w4.z, w4.w};
            uint32_t h[4];
#pragma unroll
            for (int j = 0; j < 4; ++j)
                h[j] = f16x2(__uint_as_float(w[j] << 16) * mul, __uint_as_float(w[j] & 0xffff0000u) * mul);
            *reinterpret_cast<uint4*>(smem + C::kOffQ + (i / 8) * C::kChunk + r * 128 + (((i % 8) ^ (r & 7)) << 4)) =
                make_uint4(h[0], h[1], h[2], h[3]);
        }
        fence_proxy_async_smem();
        if (!a.starve) mbar_arrive(&bars->q_full);
    }
    if (kCopies == 1 && row0 + (r & ~31) >= a.R) return;   // no row of this warp
    if (kCopies > 1) {   // P of the other copies' keys stays zero
        uint32_t z[32];
#pragma unroll
        for (int e = 0; e < 32; ++e) z[e] = 0;
#pragma unroll
        for (int c = 0; c < 4; ++c) tmem_st32(tmem + lane_off + C::kColP + 32 * c, z);
        tmem_st_wait();
    }

    const int limit = len - (a.N - 1 - row % a.N);   // keys that the row sees
    float m = -INFINITY, l = 0.f, u = -INFINITY;   // l in units of 2^m, O in units of 2^u / kPScale
    constexpr bool kHold = chunks <= 2;   // the scores stay in registers between the maximum and the probabilities
    for (int j = 0; j < T; ++j) {
        const int s = j & 1, key0 = (i0 + j) * BN;
        if (!warp_wait(&bars->full[1][j % kStages], (j / kStages) & 1, wc)) return;   // its scales
        if (!warp_wait(&bars->s_full[s], (j >> 1) & 1, wc)) return;
        tc_fence_after();
        const float* ks = reinterpret_cast<const float*>(smem + C::kOffScale) + j % kScaleSlots * 8;
        const float* vs = ks + kScaleSlots * 8;
        const uint32_t tS = tmem + lane_off + 128 * s;
        float mx = m, ux = u;
        bool whole = key0 + BN <= limit_all;
#pragma unroll
        for (int i = 0; i < 8; ++i) whole = whole && ks[i] >= 0.f;
        // Scores are x * cs; in a tile that masks something, -inf or the scaled score, and cs is 1.
        auto group_scale = [&](int i) { return whole ? qscale * ks[i] : 1.f; };
        auto mask = [&](uint32_t (&x)[32], int c) {
#pragma unroll
            for (int e = 0; e < 32; ++e) {
                const float f = ks[2 * c + e / 16];
                x[e] = key0 + 32 * c + e < limit && f >= 0.f ? __float_as_uint(__uint_as_float(x[e]) * (qscale * f)) : 0xff800000u;
            }
        };
        auto largest = [&](const uint32_t (&x)[32], int c) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                float g[2] = {-INFINITY, -INFINITY};
#pragma unroll
                for (int e = 0; e < 16; e += 4)
#pragma unroll
                    for (int k = 0; k < 2; ++k)
                        g[k] = max3(g[k], __uint_as_float(x[16 * i + e + 2 * k]), __uint_as_float(x[16 * i + e + 2 * k + 1]));
                const float s = fmaxf(g[0], g[1]) * group_scale(2 * c + i);
                mx = fmaxf(mx, s);
                ux = fmaxf(ux, s + log2_scale(vs[2 * c + i]));
            }
        };
        uint32_t held[kHold ? chunks : 1][32];
        if constexpr (kHold) {
#pragma unroll
            for (int c = 0; c < chunks; ++c) tmem_ld32(tS + 32 * (c0 + c), held[c]);
            tmem_ld_wait();
#pragma unroll
            for (int c = 0; c < chunks; ++c) {
                if (!whole) mask(held[c], c0 + c);
                largest(held[c], c0 + c);
            }
        } else {
#pragma unroll 1
            for (int c = 0; c < chunks; ++c) {
                tmem_ld32(tS + 32 * c, held[0]);
                tmem_ld_wait();
                if (!whole) mask(held[0], c);
                largest(held[0], c);
            }
        }
        if (mx > m + kGrowth || (m == -INFINITY && mx > -INFINITY)) {
            l *= m == -INFINITY ? 0.f : ex2(m - mx);
            m = mx;
        }
        const bool grown = ux > u + kGrowth || (u == -INFINITY && ux > -INFINITY);
        if (__any_sync(0xffffffffu, grown)) {   // O follows its unit
            if (j > 0) {
                if (!warp_wait(&bars->pv_done[s ^ 1], ((j - 1) >> 1) & 1, wc)) return;
                tc_fence_after();
                const float f = !grown ? 1.f : u == -INFINITY ? 0.f : ex2(u - ux);
#pragma unroll 1
                for (int c = 0; c < D / 32; ++c) {
                    uint32_t x[32];
                    tmem_ld32(tmem + lane_off + C::kColO + 32 * c, x);
                    tmem_ld_wait();
#pragma unroll
                    for (int e = 0; e < 32; ++e) x[e] = __float_as_uint(__uint_as_float(x[e]) * f);
                    tmem_st32(tmem + lane_off + C::kColO + 32 * c, x);
                }
                tmem_st_wait();
            }
            if (grown) u = ux;
        }
        const float pscale = u == -INFINITY ? 0.f : ex2(m - u) * kPScale;
        // P's buffer is free: S of this tile was formed behind P V of the tile before the last.
        const float nm = m == -INFINITY ? 0.f : -m;
        const uint64_t nm2 = f2_pack(nm, nm);
        uint64_t l2 = 0;
        auto probabilities = [&](const uint32_t (&x)[32], int c) {
            uint32_t pk[16];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                // (pv is beyond fp32 only where a probability that would matter is 0 in fp32.)
                const float cs = group_scale(2 * c + i), pv = fminf(vs[2 * c + i] * pscale, kMaxFloat);
                const uint64_t cs2 = f2_pack(cs, cs), pv2 = f2_pack(pv, pv);
#pragma unroll
                for (int e = 0; e < 16; e += 2) {
                    float x0, x1;
                    f2_unpack(ffma2(f2_pack(__uint_as_float(x[16 * i + e]), __uint_as_float(x[16 * i + e + 1])), cs2, nm2), x0, x1);
                    const uint64_t p2 = f2_pack(ex2(x0), ex2(x1));
                    l2 = fadd2(l2, p2);
                    float p0, p1;
                    f2_unpack(fmul2(p2, pv2), p0, p1);
                    pk[8 * i + e / 2] = f16x2(p0, p1);
                }
            }
            tmem_st16(tmem + lane_off + C::kColP + 64 * s + 16 * c, pk);
        };
        if constexpr (kHold) {
#pragma unroll
            for (int c = 0; c < chunks; ++c) probabilities(held[c], c0 + c);
        } else {
#pragma unroll 1
            for (int c = 0; c < chunks; ++c) {
                tmem_ld32(tS + 32 * c, held[0]);
                tmem_ld_wait();
                if (!whole) mask(held[0], c);
                probabilities(held[0], c);
            }
        }
        float l0, l1;
        f2_unpack(l2, l0, l1);
        l += l0 + l1;
        tmem_st_wait();
        tc_fence_before();
        mbar_arrive(&bars->p_full[s]);
    }

    if (T > 0) {
        if (!warp_wait(&bars->pv_done[(T - 1) & 1], ((T - 1) >> 1) & 1, wc)) return;
        tc_fence_after();
    }
    const int split = blockIdx.x / a.row_tiles % a.splits, rt = blockIdx.x % a.row_tiles;
    // The copies of a row join through the K and V buffers, which are free by now.
    const float unit = u == -INFINITY ? 0.f : ex2(u - m) / kPScale;
    constexpr int kPitch = D + 4;
    float* joint = reinterpret_cast<float*>(smem + C::kOffKV);
    float2* joint_ml = reinterpret_cast<float2*>(joint + BM * kPitch);
    static_assert(BM * (kPitch * 4 + 8) <= 2 * kStages * C::kTile, "the copies' results fit");
    if (kCopies > 1) {
        joint_ml[r] = make_float2(m, l);
#pragma unroll 1
        for (int c = 0; c < D / 32; ++c) {
            uint32_t x[32];
            if (T > 0) {
                tmem_ld32(tmem + lane_off + C::kColO + 32 * c, x);
                tmem_ld_wait();
            }
#pragma unroll
            for (int e = 0; e < 32; e += 4)
                *reinterpret_cast<float4*>(joint + r * kPitch + 32 * c + e) =
                    T > 0 ? make_float4(__uint_as_float(x[e]) * unit, __uint_as_float(x[e + 1]) * unit,
                                                      __uint_as_float(x[e + 2]) * unit, __uint_as_float(x[e + 3]) * unit)
                                        : make_float4(0.f, 0.f, 0.f, 0.f);
        }
        mbar_arrive(&bars->joined);
        if (!warp_wait(&bars->joined, 0, wc)) return;
        float mm = -INFINITY;
        for (int k = 0; k < kCopies; ++k) mm = fmaxf(mm, joint_ml[r % copy_rows + k * copy_rows].x);
        m = mm;
        l = 0.f;
        for (int k = 0; k < kCopies; ++k) {
            const float2 ml = joint_ml[r % copy_rows + k * copy_rows];
            l = fmaf(ex2(ml.x - (mm == -INFINITY ? 0.f : mm)), ml.y, l);
        }
    }
    const bool whole = a.splits == 1;
    const float inv = !whole ? 1.f : l > 0.f ? 1.f / l : (l == 0.f ? 0.f : l);   // NaN stays NaN
    const size_t out = (size_t)bh * a.R + row;
    const size_t at = (((size_t)bh * a.row_tiles + rt) * a.splits + split) * a.tile_rows + r % copy_rows;
    // A copy writes its share of the columns, 32 at a time.
#pragma unroll 1
    for (int c = c0 * D / 128; c < (c0 + chunks) * D / 128; ++c) {
        uint32_t x[32];
        if (kCopies > 1) {
            float y[32];
#pragma unroll
            for (int e = 0; e < 32; ++e) y[e] = 0.f;
            for (int k = 0; k < kCopies; ++k) {
                const int from = r % copy_rows + k * copy_rows;
                const float f = ex2(joint_ml[from].x - (m == -INFINITY ? 0.f : m)) * inv;
#pragma unroll
                for (int e = 0; e < 32; e += 4) {
                    const float4 v = *reinterpret_cast<const float4*>(joint + from * kPitch + 32 * c + e);
                    y[e] = fmaf(f, v.x, y[e]);
                    y[e + 1] = fmaf(f, v.y, y[e + 1]);
                    y[e + 2] = fmaf(f, v.z, y[e + 2]);
                    y[e + 3] = fmaf(f, v.w, y[e + 3]);
                }
            }
#pragma unroll
            for (int e = 0; e < 32; ++e) x[e] = __float_as_uint(y[e]);
        } else {
            if (T > 0) {
                tmem_ld32(tmem + lane_off + C::kColO + 32 * c, x);
                tmem_ld_wait();
            }
#pragma unroll
            for (int e = 0; e < 32; ++e) x[e] = T > 0 ? __float_as_uint(__uint_as_float(x[e]) * (unit * inv)) : 0u;
        }
        if (bars->new_nan) {   // the newest tokens' NaN, where this row sees them
            for (int key = max(limit_all, i0 * BN); key < min(limit, i1 * BN); ++key) {
                const int p = a.table[(size_t)b * a.max_blocks + (key >> a.bs_log2)];
                if ((unsigned)p >= (unsigned)a.n_blocks) continue;
                const uint8_t* v = a.v + (((((size_t)p * a.Hk + hk) << a.bs_log2) + (key & ((1 << a.bs_log2) - 1))) * D + 32 * c);
#pragma unroll
                for (int e = 0; e < 32; ++e)
                    if ((v[e] & 127) == 127) x[e] = 0x7fc00000u;
            }
        }
        if (!mine) continue;
        if (whole) {
            uint4* dst = reinterpret_cast<uint4*>(a.o + out * D + 32 * c);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                uint32_t w[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) w[e] = pack_bf16(__uint_as_float(x[8 * i + 2 * e]), __uint_as_float(x[8 * i + 2 * e + 1]));
                dst[i] = make_uint4(w[0], w[1], w[2], w[3]);
            }
        } else {
            uint4* dst = reinterpret_cast<uint4*>(a.part_o + at * D + 32 * c);
#pragma unroll
            for (int i = 0; i < 8; ++i) dst[i] = make_uint4(x[4 * i], x[4 * i + 1], x[4 * i + 2], x[4 * i + 3]);
        }
    }
    if (!mine || c0 > 0) return;
    if (whole) a.lse[out] = l == 0.f ? -INFINITY : (m + log2f(l)) * 0.69314718055994531f;
    else a.part_ml[at] = make_float2(m, l);
}

template <int D, int kCopies>
__global__ void __launch_bounds__(kThreads, 1) cache_tc_kernel(const __grid_constant__ CacheTcArgs a) {
    using C = CacheCfg<D>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
    CacheBarriers* bars = reinterpret_cast<CacheBarriers*>(smem + C::kOffBar);
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    griddep_wait();
    griddep_launch_dependents();
    int x = blockIdx.x;
    const int row0 = x % a.row_tiles * BM;
    x /= a.row_tiles;
    const int split = x % a.splits, bh = x / a.splits;
    const int b = bh / a.Hk, hk = bh - b * a.Hk;
    const int len = min(max(a.lens[b], 0), a.cap), limit_all = len - (a.N - 1);   // keys that every row sees
    const int tiles = (len + BN - 1) / BN;
    const int i0 = (int)((long long)tiles * split / a.splits), i1 = (int)((long long)tiles * (split + 1) / a.splits);
    if (threadIdx.x == 0) {
        bars->wait.budget = a.wait_budget;
        mbar_init(&bars->q_full, 128);
        const int warps = kCopies > 1 ? 4 : (min(a.R - row0, BM) + 31) / 32;
        for (int t = 0; t < 2; ++t) {
            for (int k = 0; k < kStages; ++k) {
                mbar_init(&bars->full[t][k], 16 * kConverters);
                mbar_init(&bars->free[t][k], 1);
            }
            mbar_init(&bars->s_full[t], 1);
            mbar_init(&bars->p_full[t], 32 * warps);
            mbar_init(&bars->pv_done[t], 1);
        }
        mbar_init(&bars->joined, 128);
        mbar_init(&bars->mma_done, 1);
        bars->new_nan = 0;
        bars->wait.abort = 0;
        fence_mbar_init();
    }
    if (warp == kMmaWarp) {
        tmem_alloc(&bars->tmem_base, 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = bars->tmem_base;

    if (warp < kMmaWarp) cache_row<D, kCopies>(a, smem, bars, tmem, b, hk, row0, len, limit_all, i0, i1);
    else if (warp == kMmaWarp) {
        if (lane == 0 && i1 > i0) cache_mma<D>(smem, bars, tmem, i1 - i0);
    } else if (i1 > i0) {
        const int part = warp - kFirstConverter;
        cache_convert<D>(a, smem, bars, part / 4, part % 4, b, hk, len, limit_all, i0, i1);
    }

    tc_fence_before();
    __syncthreads();
    if (warp == kMmaWarp) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
    if (threadIdx.x == 0 && bars->wait.abort) atomicCAS(&g_cache_status, 0, (int)FA_ERR_TIMEOUT);
}

template <int D, int kCopies>
cudaError_t launch_tc(const CacheTcArgs& a, int64_t bh, cudaStream_t st) {
    using C = CacheCfg<D>;
    constexpr auto kernel = cache_tc_kernel<D, kCopies>;
    cudaError_t e = set_max_dynamic_smem((const void*)kernel, (int)C::kSmemBytes);
    if (e != cudaSuccess) return e;
    e = launch_dependent(kernel, dim3((unsigned)(bh * a.row_tiles * a.splits)), dim3(kThreads), C::kSmemBytes, st, a);
    if (e == cudaSuccess) count_launches(1);
    return e;
}

}  // namespace

RowsPlan cache_tiles_plan(int64_t bh, int R, int d, int64_t keys) {
    RowsPlan p;
    p.tiles = true;
    p.tile_rows = R < BM ? (R + 15) / 16 * 16 : BM;
    p.row_tiles = (R + BM - 1) / BM;
    const int64_t items = bh * p.row_tiles, tiles = (keys + BN - 1) / BN;
    // A CTA's set-up and write-out take 7 us, a tile about 1 (d = 64: 0.9), joining the splits 4.  Many waves overlap.
    const double tile_us = d == 128 ? 1.0 : 0.9;
    double best = 1e30;
    for (int64_t n = 1; n <= kPlanSms && (n == 1 || n * 4 <= tiles); ++n) {
        const double waves = (double)(items * n) / kPlanSms;
        const double us = (waves > 3 ? waves : ceil(waves)) * (7 + (double)((tiles + n - 1) / n) * tile_us) + (n > 1 ? 4 : 0);
        if (us < best) {
            best = us;
            p.splits = (int)n;
        }
    }
    p.ml_offset = p.splits == 1 ? 0 : ((size_t)items * p.splits * p.tile_rows * d * sizeof(float) + 255) & ~(size_t)255;
    p.bytes = p.splits == 1 ? 0 : p.ml_offset + (size_t)items * p.splits * p.tile_rows * sizeof(float2);
    return p;
}

cudaError_t launch_cache_fwd_tiles(const CacheFwd& c, const RowsPlan& p, void* workspace, cudaStream_t st) {
    CacheTcArgs a = {};
    a.q = (const __nv_bfloat16*)c.q;
    a.o = (__nv_bfloat16*)c.o;
    a.lse = c.lse;
    a.k = (const uint8_t*)c.k_cache;
    a.v = (const uint8_t*)c.v_cache;
    a.k_scale = c.k_scale;
    a.v_scale = c.v_scale;
    a.table = c.table;
    a.lens = c.lens;
    a.part_o = (float*)workspace;
    a.part_ml = (float2*)((char*)workspace + p.ml_offset);
    a.R = c.Hq / c.Hk * c.N;
    a.N = c.N;
    a.Hk = c.Hk;
    a.cap = c.max_blocks * c.bs;
    a.bs_log2 = c.bs == 16 ? 4 : c.bs == 32 ? 5 : c.bs == 64 ? 6 : 7;
    a.max_blocks = c.max_blocks;
    a.n_blocks = c.n_blocks;
    a.splits = p.splits;
    a.row_tiles = p.row_tiles;
    a.tile_rows = p.tile_rows;
    a.scale_log2 = c.scale * 1.4426950408889634f;
    const WaitPolicy wp = wait_policy();
    a.wait_budget = wp.budget_cycles;
    a.starve = wp.starve;
    const int64_t bh = (int64_t)c.B * c.Hk;
    auto* f = c.d == 128 ? (a.R <= 64 ? launch_tc<128, 2> : launch_tc<128, 1>) : (a.R <= 64 ? launch_tc<64, 2> : launch_tc<64, 1>);
    const cudaError_t e = f(a, bh, st);
    if (e != cudaSuccess || p.splits == 1) return e;
    return launch_rows_combine(a.part_o, a.part_ml, c.o, c.lse, a.R, p.tile_rows, p.row_tiles, 0, bh * p.row_tiles, p.splits, c.d,
                               st);
}

int cache_tc_read_and_clear_status(cudaStream_t st) {
    int v = 0, zero = 0;
    if (cudaMemcpyFromSymbolAsync(&v, g_cache_status, sizeof(int), 0, cudaMemcpyDeviceToHost, st) != cudaSuccess) return -1;
    if (cudaMemcpyToSymbolAsync(g_cache_status, &zero, sizeof(int), 0, cudaMemcpyHostToDevice, st) != cudaSuccess) return -1;
    if (cudaStreamSynchronize(st) != cudaSuccess) return -1;
    return v;
}

}  // namespace fa
