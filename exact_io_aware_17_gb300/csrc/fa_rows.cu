// Attention of a few query rows over a long key axis: the decoding step.  Serves the paged 8-bit cache
// (fa_cache_fwd) and, for few rows, cross attention over bf16 keys (fa_cross_fwd).
//
// Per (batch, key/value head) the G grouped query heads x N tokens are R = G N rows over the same keys:
//     S = scale Q K^T,  m = max S,  l = sum exp(S - m),  O = sum exp(S - m) V / l,  LSE = m + ln l
// with the running maximum and sum of "账房先生的奔命：Flash Attention 与内存 I/O 革命" §六 (Online Softmax).
//
// With up to 16 rows a key there are at most 32 flops a byte, far below what the tensor cores need to be
// the bound: the keys and values have to stream at HBM speed, with few instructions a byte.  So a warp is a stream of
// its own: it walks a contiguous range of keys through a private ring of tiles in shared memory, filled by asynchronous
// copies a tile or more ahead (8 KB in flight a warp, 96 KB or more an SM), feeds mma.sync from it and keeps its own m, l and O;
// nothing in the loop waits for another warp.  Warps merge at the end through shared memory, CTAs (the splits of a
// long key axis) through fp32 partials and a second kernel, by the same exp-sum factorisation as the online rescale.
//
// The products.  Up to 8 rows (kSmall): S = Q K^T with the rows in M, then O^T = V^T P^T with 16 output columns in M
// and the 8 rows in N: P's accumulator layout is the B operand's, and no half of an instruction is empty.  9 to 16
// rows: S = Q K^T and O = P V, rows in M.
// bf16 keys: mma m16n8k16 throughout, P rounded to bf16.
// Cache: up to 8 rows, Q K^T runs on the e4m3 codes as they are (m16n8k32), with Q as hi + lo / 32, two e4m3 pieces after
// a power-of-two scale per row: 4 + 4 significant bits hold a bf16 exactly, but for elements below 2^-14 of the row's
// largest, which are off by up to 2^-22 of it.  Its sums measured exact to 2^-21 of their terms' magnitudes.  The two pieces
// are the two halves of M.  9 to 16 rows would need both products, so K's codes become f16 (exact) and Q too, scaled by a
// power of two per row (exact down to 2^-29 of the row's largest): 64 requests of 4096 to 8192 tokens x 8 heads (806 MB),
// d = 128, took 168 us with two e4m3 products and 140 so (5.7 TB/s), and of 8192 tokens each, d = 64, 127 and 107.  V's codes
// become f16 (exact) for P V.  The scale of a key block multiplies its scores, that of a value block its probabilities: the
// product takes 2^(s + log2 scale - u) as f16, with the row's running maximum u of s + log2 scale over the keys that it sees,
// so that a block counts by what it adds to the row, however far the scales lie apart and whatever other rows see.  f16 rounds
// this to 11 bits and drops what is below 2^-37 of the row's largest.

#include <cuda_bf16.h>
#include <math.h>

#include "fa_internal.h"
#include "fa_ptx.cuh"

namespace fa {
namespace {

using namespace ptx;

constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
// CTAs an SM, as the registers allow, and the ring of each of their warps, which together fill its shared memory.  Measured at
// 2 (24 KB), 3 (16 KB) and 4 (12 KB) CTAs, us, for 64 x 4096 to 8192 tokens x 8 heads: d = 128, 4 rows a head 130, 126, -; 16
// rows 140, 136, -; d = 64, 4 rows 91, 78, 73; 16 rows over 8192 tokens each -, 107, 103, but one request of 131072 tokens x 4 heads 21.2,
// 22.9.  Bf16 keys, 64 heads x 32768, d = 128: 153, 150; 16 rows: 128 heads x 1000 13.0, 15.5, 512 x 8192 309, 305; 32 x 4096 x
// 16 heads, d = 64: 45.3, 43.9, 43.4.
__host__ __device__ constexpr int ctas_per_sm(int d, bool small, bool cache) {
    return d == 128 ? (small || cache ? 3 : 2) : small ? 4 : 3;
}
__host__ __device__ constexpr int ring_bytes(int d, bool small, bool cache) {
    return ctas_per_sm(d, small, cache) == 2 ? 24576 : ctas_per_sm(d, small, cache) == 3 ? 16384 : 12288;
}
constexpr float kLoScale = 32.f;      // hi's last place is at most 16, so lo is at most 8 before this scale (codes reach 448)
constexpr float kPScale = 4096.f;     // probabilities in f16: 2^12 keeps them out of the subnormals
constexpr float kMaxFloat = 3.402823466e38f;

struct RowsArgs {
    const __nv_bfloat16* q;           // [BH][R][D]
    __nv_bfloat16* o;
    float* lse;                       // [BH][R]
    const uint8_t *k, *v;             // cache: [block][head][token][D] e4m3; dense: [BH][cap][D] bf16
    const float *k_scale, *v_scale;   // cache: [block][head]
    const int* table;                 // cache: [B][max_blocks]
    const int* lens;                  // [B]; dense: null for Nk
    float* part_o;                    // [BH][row tile][split][rows of a tile][D]
    float2* part_ml;                  // [BH][row tile][split][rows of a tile]  (m in log2 units, l)
    int R, N, Hk, cap, bs_log2, max_blocks, n_blocks, splits, row_tiles;
    float scale_log2;
};

// Asynchronous copies into shared memory past L1.  With `on` false they write zeros and read nothing.
__device__ __forceinline__ void copy16(uint32_t dst, const void* src, uint64_t policy) {
    asm volatile("cp.async.cg.shared.global.L2::cache_hint [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "l"(policy) : "memory");
}
__device__ __forceinline__ void copy16(uint32_t dst, const void* src, bool on) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(on ? 16 : 0) : "memory");
}
__device__ __forceinline__ void copy4(uint32_t dst, const void* src, bool on) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(on ? 4 : 0) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void lds16(uint32_t* r, uint32_t addr) {
    asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];" : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void lds8(uint32_t* r, uint32_t addr) {
    asm volatile("ld.shared.v2.b32 {%0,%1}, [%2];" : "=r"(r[0]), "=r"(r[1]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void sts_u16(uint32_t addr, uint32_t v) {
    asm volatile("st.shared.u16 [%0], %1;" ::"r"(addr), "h"((uint16_t)v) : "memory");
}
__device__ __forceinline__ float lds_f16(uint32_t addr) {
    float f;
    asm volatile("{.reg .b16 h;\n\tld.shared.b16 h, [%1];\n\tcvt.f32.f16 %0, h;\n\t}" : "=f"(f) : "r"(addr) : "memory");
    return f;
}
__device__ __forceinline__ void sts16_zero(uint32_t addr) {
    asm volatile("st.shared.v4.b32 [%0], {%1,%1,%1,%1};" ::"r"(addr), "r"(0) : "memory");
}

__device__ __forceinline__ void mma_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_bf16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_e4m3(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k32.row.col.f32.e4m3.e4m3.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// Two e4m3 codes (the low or high half of w) as two f16.
__device__ __forceinline__ uint32_t e4m3x2_f16(uint32_t w, int high) {
    uint32_t r;
    if (high) asm("{.reg .b16 l, h;\n\tmov.b32 {l, h}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, h;\n\t}" : "=r"(r) : "r"(w));
    else asm("{.reg .b16 l, h;\n\tmov.b32 {l, h}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, l;\n\t}" : "=r"(r) : "r"(w));
    return r;
}
__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
__device__ __forceinline__ uint32_t prmt(uint32_t a, uint32_t b, uint32_t sel) {
    uint32_t r;
    asm("prmt.b32 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(b), "r"(sel));
    return r;
}
// log2 of a power of two (of 0: -127), from its exponent bits: 2^23 + them is exact.
__device__ __forceinline__ float log2_scale(float x) {
    return __uint_as_float(0x4b000000u | __float_as_uint(x) >> 23) - (8388608.f + 127.f);
}
// Code i of w as a float.
__device__ __forceinline__ float e4m3_f32(uint32_t w, int i) {
    const uint32_t f2 = e4m3x2_f16(w, i >> 1);
    float f;
    if (i & 1) asm("{.reg .b16 l, h;\n\tmov.b32 {l, h}, %1;\n\tcvt.f32.f16 %0, h;\n\t}" : "=f"(f) : "r"(f2));
    else asm("{.reg .b16 l, h;\n\tmov.b32 {l, h}, %1;\n\tcvt.f32.f16 %0, l;\n\t}" : "=f"(f) : "r"(f2));
    return f;
}
// Four values as e4m3: the nearest codes, and the codes of kLoScale times what those leave.
__device__ __forceinline__ void split_e4m3(const float (&x)[4], uint32_t& hi, uint32_t& lo) {
    const uint32_t h01 = e4m3x2(x[0], x[1]), h23 = e4m3x2(x[2], x[3]);
    float r[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        r[i] = (x[i] - e4m3_f32(i < 2 ? h01 : h23, i & 1)) * kLoScale;
    }
    hi = h01 | h23 << 16;
    lo = e4m3x2(r[0], r[1]) | e4m3x2(r[2], r[3]) << 16;
}

// A warp's key tile in shared memory and how its lanes read it.  g = lane / 4, t = lane % 4.  Pieces are 16 bytes; piece c of
// row r lies at c ^ (r % 8) of 128-byte rows (rows of 256 bytes are two blocks of them), at c ^ (r / 2 % 4) of 64-byte ones.
//   K: column n of the 8-key tile j of S is key 8 j + key(n); lane (g, t) reads pieces t + 4 s of the row of key(g).  The
//      order of the head dimension in the product is theirs.
//   V: lane (g, t) reads the piece of its output columns (its half piece of 64-byte rows; two pieces of 256-byte ones)
//      in the rows of the four keys of which it holds the scores, 16 u + key(2t), key(2t + 1) and 8 further on.
// Eight lanes of a 16-byte access read pieces t of two rows (K), or two pieces of four rows (V).  With 128-byte rows
// key(n) makes the two rows differ by 4 and lanes of odd t take their two V rows in the other order, so that the
// eight always meet eight different pieces of the swizzle.
template <int D, bool kCache, bool kSmall>
struct Tile {
    static constexpr int kKeys = kCache ? kCacheTileKeys : kDenseTileKeys;
    static constexpr int kElt = kCache ? 1 : 2;
    static constexpr int kNT = kKeys / 8;                       // 8-key column tiles of S
    static constexpr int kRow = D * kElt;                       // bytes of a row: 64, 128 or 256
    static constexpr int kBytes = kKeys * kRow;                 // of K, and of V
    static constexpr int kRingBytes = ring_bytes(D, kSmall, kCache);
    static constexpr int kStages = kRingBytes / (2 * kBytes);   // 2 to 4
    static constexpr int kVW = kRow / 32;                       // words of V a lane holds for one key
    static constexpr bool kSwap = kRow >= 128;
    __device__ static int key(int n) { return kSwap ? (n >> 1) | (n & 1) << 2 : n; }
    // First head dimension of the 8 that steps 2 i and 2 i + 1 (cache: step i) of the product take from lane t.
    __device__ static int dk(int t, int i) { return kCache ? 16 * (t + 4 * (i / 2)) + 8 * (i % 2) : 8 * (t + 4 * i); }
    // Output columns of a lane: its word w of V (4 codes or 2 bf16) starts at column(w, g).
    __device__ static int column(int w, int g) {
        return kCache ? (D / 8) * g + 4 * w : kRow == 256 ? 64 * (w / 4) + 8 * g + 2 * (w % 4) : 8 * g + 2 * w;
    }
    // Byte offset of piece c of a row.
    __device__ static int at(int row, int c) {
        if (kRow == 64) return row * 64 + ((c ^ ((row >> 1) & 3)) << 4);
        return (c >> 3) * (kKeys * 128) + row * 128 + (((c & 7) ^ (row & 7)) << 4);
    }
};

template <int D, bool kCache, bool kSmall>
__global__ void __launch_bounds__(kThreads, ctas_per_sm(D, kSmall, kCache))
rows_kernel(const __grid_constant__ RowsArgs a) {
    using T = Tile<D, kCache, kSmall>;
    constexpr int kTileRows = kSmall ? 8 : 16;
    constexpr int kE = kSmall ? 1 : 2;               // rows whose scores a lane holds: g (and g + 8)
    extern __shared__ __align__(128) uint8_t smem[];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int g = lane >> 2, t = lane & 3;
    // The kernel may start while the one ahead of it on the stream is finishing: nothing of memory is touched before this.
    griddep_wait();
    griddep_launch_dependents();
    int x = blockIdx.x;
    const int rt = x % a.row_tiles;
    x /= a.row_tiles;
    const int split = x % a.splits;
    const int bh = x / a.splits;
    const int b = bh / a.Hk, hk = bh - b * a.Hk;
    const int len = a.lens ? min(max(a.lens[b], 0), a.cap) : a.cap;
    const int row0 = rt * kTileRows;

    // This warp's tiles, and its ring of them in shared memory.
    const int tiles = (len + T::kKeys - 1) / T::kKeys;
    const int W = a.splits * kWarps, wi = split * kWarps + warp;
    const int per = tiles / W, more = tiles - per * W;   // the first `more` warps take one tile more
    const int i0 = wi * per + min(wi, more), i1 = i0 + per + (wi < more ? 1 : 0);
    const uint32_t ring = smem_u32(smem) + warp * T::kRingBytes;
    const uint32_t scales = smem_u32(smem) + kWarps * T::kRingBytes + warp * (T::kStages * 16);   // ks ks vs vs a stage

    const int* trow = kCache ? a.table + (size_t)b * a.max_blocks : nullptr;
    // Blocks of the two 16-key halves of the next tile to start: -1 where there are no keys or the table names no block.
    int next[2] = {-1, -1};
    auto fetch = [&](int i) {
        if constexpr (kCache) {
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                const int key = i * T::kKeys + 16 * u;
                const int p = i < i1 && key < len ? trow[key >> a.bs_log2] : -1;
                next[u] = (unsigned)p < (unsigned)a.n_blocks ? p : -1;
            }
        }
    };
    const uint64_t policy = policy_evict_first();
    uint32_t there = 0;   // cache: two bits a tile, the latest tile's lowest: which halves have a block
    // A copy instruction moves 512 bytes: kRpc rows, a lane a piece; kCopies of them 16 rows.  Where a lane's piece goes:
    // its place in the swizzle for the first rows, which the others' row numbers XOR.
    constexpr int kPieces = T::kRow / 16, kRpc = 32 / kPieces, kCopies = 16 / kRpc;
    const int my_row = lane / kPieces, my_piece = lane % kPieces;
    const int my_at = T::at(my_row, my_piece);
    int load_stage = 0;
    auto issue = [&](int i) {   // starts the copies of tile i, if there is one
        if (i < i1) {
            const int s = load_stage, key0 = i * T::kKeys;
            load_stage = s + 1 == T::kStages ? 0 : s + 1;
            const uint32_t kd = ring + s * (2 * T::kBytes);
            // Byte offset of the 16 keys 16 u of the tile.
            auto source = [&](int u) {
                const size_t row = kCache ? (((size_t)max(next[u], 0) * a.Hk + hk) << a.bs_log2) +
                                                ((key0 + 16 * u) & ((1 << a.bs_log2) - 1))
                                          : (size_t)bh * a.cap + key0;
                return row * T::kRow + lane * 16;
            };
            if (key0 + T::kKeys <= len && (!kCache || (next[0] >= 0 && next[1] >= 0))) {
#pragma unroll
                for (int u = 0; u < T::kKeys / 16; ++u) {
                    const uint8_t *ksrc = a.k + source(u), *vsrc = a.v + source(u);
#pragma unroll
                    for (int n = 0; n < kCopies; ++n) {
                        // Rows n kRpc on: further by their bytes, and by their low bits in the swizzle (64-byte rows: 8 rows
                        // on is the same place).
                        const int flip = T::kRow == 64 ? 0 : ((n * kRpc) & 7) << 4;
                        const uint32_t dst = kd + (my_at ^ flip) + (16 * u + n * kRpc) * (T::kRow < 128 ? T::kRow : 128);
                        copy16(dst, ksrc + n * 512, policy);
                        copy16(dst + T::kBytes, vsrc + n * 512, policy);
                    }
                }
            } else {   // rows without a token become zeros (rolled: unrolled, it would be predicated into every tile)
#pragma unroll
                for (int u = 0; u < T::kKeys / 16; ++u) {
                    const size_t src = source(u) - lane * 16;
#pragma unroll 1
                    for (int n = 0; n < kCopies; ++n) {
                        const int row = n * kRpc + my_row;
                        const bool on = key0 + 16 * u + row < len && (!kCache || next[u] >= 0);
                        const uint32_t dst = kd + T::at(16 * u + row, my_piece);
                        const size_t off = on ? src + row * T::kRow + my_piece * 16 : 0;
                        copy16(dst, a.k + off, on);
                        copy16(dst + T::kBytes, a.v + off, on);
                    }
                }
            }
            if (kCache && lane < 4) {
                const int bl = lane & 1 ? next[1] : next[0];
                const float* src = lane < 2 ? a.k_scale : a.v_scale;
                copy4(scales + s * 16 + lane * 4, bl >= 0 ? src + ((size_t)bl * a.Hk + hk) : src, bl >= 0);
            }
        }
        copy_commit();
        if (kCache) there = there << 2 | (next[0] >= 0 ? 1u : 0u) | (next[1] >= 0 ? 2u : 0u);
        fetch(i + 1);
    };
    fetch(i0);
#pragma unroll
    for (int s = 0; s < T::kStages - 1; ++s) issue(i0 + s);

    // Q fragments.  Cache: rows scaled by a power of two, as two e4m3 pieces or f16.
    constexpr int kQ8 = D / 32;                      // groups of 8 head dimensions of a lane
    uint32_t qa[kCache ? (kSmall ? kQ8 : 2 * kQ8) : 2 * kQ8][4];
    float qscale[kE];
    {
        uint4 raw[2][kQ8];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int r = row0 + g + 8 * e;
            const bool on = e < kE && r < a.R;
            const __nv_bfloat16* src = a.q + ((size_t)bh * a.R + r) * D;
#pragma unroll
            for (int i = 0; i < kQ8; ++i)
                raw[e][i] = on ? *reinterpret_cast<const uint4*>(src + T::dk(t, i)) : make_uint4(0, 0, 0, 0);
        }
        if constexpr (kCache) {
#pragma unroll
            for (int e = 0; e < kE; ++e) {
                float amax = 0.f;
#pragma unroll
                for (int i = 0; i < kQ8; ++i) {
                    const uint32_t w[4] = {raw[e][i].x, raw[e][i].y, raw[e][i].z, raw[e][i].w};
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        amax = max3(amax, fabsf(__uint_as_float(w[j] << 16)), fabsf(__uint_as_float(w[j] & 0xffff0000u)));
                }
                amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
                amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
                // mul = 2^(7 - exponent of amax), with f16 2^(14 - it), kept a normal number.
                const int ex = min(max((int)(__float_as_uint(amax) >> 23) - 127, -100), 127);
                const float mul = __uint_as_float((uint32_t)(min((kSmall ? 7 : 14) - ex, 100) + 127) << 23);
                // An infinity or NaN in the row makes all of its scores NaN, as the product would (but for zeros).
                qscale[e] = amax <= kMaxFloat ? a.scale_log2 / mul : __int_as_float(0x7fc00000);
#pragma unroll
                for (int i = 0; i < kQ8; ++i) {
                    const uint32_t w[4] = {raw[e][i].x, raw[e][i].y, raw[e][i].z, raw[e][i].w};
#pragma unroll
                    for (int p = 0; p < 2; ++p) {
                        const float v[4] = {__uint_as_float(w[2 * p] << 16) * mul, __uint_as_float(w[2 * p] & 0xffff0000u) * mul,
                                            __uint_as_float(w[2 * p + 1] << 16) * mul,
                                            __uint_as_float(w[2 * p + 1] & 0xffff0000u) * mul};
                        if constexpr (kSmall) {
                            split_e4m3(v, qa[i][2 * p], qa[i][2 * p + 1]);
                        } else {
                            qa[2 * i + p][e] = pack_f16(v[0], v[1]);
                            qa[2 * i + p][2 + e] = pack_f16(v[2], v[3]);
                        }
                    }
                }
            }
        } else {
#pragma unroll
            for (int e = 0; e < kE; ++e) qscale[e] = a.scale_log2;
#pragma unroll
            for (int e = 0; e < 2; ++e)
#pragma unroll
                for (int i = 0; i < kQ8; ++i) {
                    qa[2 * i][e] = raw[e][i].x;
                    qa[2 * i][2 + e] = raw[e][i].y;
                    qa[2 * i + 1][e] = raw[e][i].z;
                    qa[2 * i + 1][2 + e] = raw[e][i].w;
                }
        }
    }
    // Keys that the lane's rows see: token n of N sees the keys before lens - (N - 1 - n).
    int limit[kE];
#pragma unroll
    for (int e = 0; e < kE; ++e) limit[e] = len - (a.N - 1 - (row0 + g + 8 * e) % a.N);
    const int limit_all = len - (a.N - 1);   // keys that every row sees

    // O: kSmall: O^T, tile w is columns column(w / 2, g) + 2 (w % 2) (c0, c1) and one further (c2, c3) of rows 2t, 2t + 1 (bf16:
    // columns column(w, g)).  Else: tile s is the column s of each lane group's share, c0, c1 of row g, c2, c3 of g + 8.
    constexpr int kAcc = kSmall ? D / 16 : D / 8;
    float acc[kAcc][4];
#pragma unroll
    for (int s = 0; s < kAcc; ++s)
#pragma unroll
        for (int c = 0; c < 4; ++c) acc[s][c] = 0.f;
    float m[kE], l[kE];
#pragma unroll
    for (int e = 0; e < kE; ++e) {
        m[e] = -INFINITY;
        l[e] = 0.f;
    }
    // Cache: um, the running maximum of score + log2 of the value scale (O is in units of 2^um / kPScale), and kPScale 2^(m - um).
    float um[kE], pscale[kE];
#pragma unroll
    for (int e = 0; e < kE; ++e) {
        um[e] = -INFINITY;
        pscale[e] = 0.f;
    }
    const bool odd = t & 1;
    // Byte pairs of two keys side by side, whichever order a lane loaded them in.
    const uint32_t sel_lo = kCache ? (odd ? 0x1504u : 0x5140u) : (odd ? 0x1054u : 0x5410u);
    const uint32_t sel_hi = kCache ? (odd ? 0x3726u : 0x7362u) : (odd ? 0x3276u : 0x7632u);
    // Byte offsets of the lane's first piece of K (row key(g)), and of V in rows key(2t) and key(2t + 1), in the other
    // order where t is odd; the rest are constants away (8 rows on is the same place of the swizzle).
    const int kat = T::at(T::key(g), t);
    int vat[2];
#pragma unroll
    for (int k = 0; k < 2; ++k)
        vat[k] = T::kRow == 64 ? T::at(T::key(2 * t + (k ^ (t & 1))), g >> 1) + (g & 1) * 8 : T::at(T::key(2 * t + (k ^ (t & 1))), g);

    int stage = 0;
    for (int i = i0; i < i1; ++i) {
        const int key0 = i * T::kKeys;
        copy_wait<T::kStages - 2>();
        __syncwarp();   // every lane's copies of tile i have landed, and every lane is done with tile i - 1
        const uint32_t has = kCache ? there >> (2 * (T::kStages - 2)) & 3 : 3;
        issue(i + T::kStages - 1);
        const uint32_t kd = ring + stage * (2 * T::kBytes), vd = kd + T::kBytes;
        float ks[2] = {1.f, 1.f}, vs[2] = {1.f, 1.f};
        if (kCache) {
            uint32_t w[4];
            lds16(w, scales + stage * 16);
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                ks[u] = __uint_as_float(w[u]);
                vs[u] = __uint_as_float(w[2 + u]);
            }
        }
        stage = stage + 1 == T::kStages ? 0 : stage + 1;

        float sc[T::kNT][2 * kE];
#pragma unroll
        for (int j = 0; j < T::kNT; ++j) {
            uint32_t kr[T::kRow / 16];
            // Rows 8 j further on: a whole swizzle pattern away.
#pragma unroll
            for (int s = 0; s < T::kRow / 64; ++s)
                lds16(kr + 4 * s, kd + j * 8 * (T::kRow < 128 ? T::kRow : 128) +
                                      (T::kRow == 64 ? kat : (s >> 1) * (T::kKeys * 128) + (kat ^ ((s & 1) << 6))));
            float c[4] = {0.f, 0.f, 0.f, 0.f};
            if constexpr (kCache) {
                if constexpr (kSmall) {
#pragma unroll
                    for (int i8 = 0; i8 < kQ8; ++i8) mma_e4m3(c, qa[i8], kr[2 * i8], kr[2 * i8 + 1]);
                } else {
#pragma unroll
                    for (int w = 0; w < 2 * kQ8; ++w)
                        mma_f16(c, qa[w][0], qa[w][1], qa[w][2], qa[w][3], e4m3x2_f16(kr[w], 0), e4m3x2_f16(kr[w], 1));
                }
            } else {
#pragma unroll
                for (int i = 0; i < 2 * kQ8; ++i)
                    mma_bf16(c, qa[i][0], qa[i][1], qa[i][2], qa[i][3], kr[2 * i], kr[2 * i + 1]);
            }
            if constexpr (kSmall) {
                sc[j][0] = kCache ? fmaf(c[2], 1.f / kLoScale, c[0]) : c[0];
                sc[j][1] = kCache ? fmaf(c[3], 1.f / kLoScale, c[1]) : c[1];
            } else {
#pragma unroll
                for (int k = 0; k < 4; ++k) sc[j][k] = c[k];
            }
        }
        // Scores are sc * cs; in a tile that masks something, -inf or the scaled score, and cs is 1.
        float cs[kE][2];
#pragma unroll
        for (int e = 0; e < kE; ++e)
#pragma unroll
            for (int u = 0; u < 2; ++u) cs[e][u] = kCache ? qscale[e] * ks[u] : qscale[e];
        const bool whole = key0 + T::kKeys <= limit_all && has == 3;
        if (!whole) {
#pragma unroll
            for (int j = 0; j < T::kNT; ++j)
#pragma unroll
                for (int c = 0; c < 2 * kE; ++c) {
                    const int key = key0 + 8 * j + T::key(2 * t + (c & 1));
                    const bool on = key < limit[c >> 1] && (has >> (j / 2) & 1);
                    sc[j][c] = on ? sc[j][c] * cs[c >> 1][j / 2] : -INFINITY;
                }
#pragma unroll
            for (int e = 0; e < kE; ++e) cs[e][0] = cs[e][1] = 1.f;
        }
        float m_new[kE], um_new[kE];
        bool moved = false;
#pragma unroll
        for (int e = 0; e < kE; ++e) {
            float mu[2] = {-INFINITY, -INFINITY};
#pragma unroll
            for (int j = 0; j < T::kNT; ++j) mu[j / 2] = max3(mu[j / 2], sc[j][2 * e], sc[j][2 * e + 1]);
            m_new[e] = T::kNT > 2 ? max3(m[e], mu[0] * cs[e][0], mu[1] * cs[e][1]) : fmaxf(m[e], mu[0] * cs[e][0]);
            um_new[e] = um[e];
            if (kCache)
                um_new[e] = max3(um[e], fmaf(mu[0], cs[e][0], log2_scale(vs[0])), fmaf(mu[1], cs[e][1], log2_scale(vs[1])));
            moved |= m_new[e] != m[e] || (kCache && um_new[e] != um[e]);
        }
        if (__any_sync(0xffffffffu, moved)) {   // l follows the maximum, O its unit (bf16 keys: the maximum)
            float fall[kE];
#pragma unroll
            for (int e = 0; e < kE; ++e) {
#pragma unroll
                for (int o = 1; o <= 2; ++o) {   // the other keys' lanes of the row
                    m_new[e] = fmaxf(m_new[e], __shfl_xor_sync(0xffffffffu, m_new[e], o));
                    if (kCache) um_new[e] = fmaxf(um_new[e], __shfl_xor_sync(0xffffffffu, um_new[e], o));
                }
                const float alpha = m[e] == -INFINITY ? 0.f : ex2(m[e] - m_new[e]);
                l[e] *= alpha;
                m[e] = m_new[e];
                fall[e] = alpha;
                if (kCache) {
                    fall[e] = um[e] == -INFINITY ? 0.f : ex2(um[e] - um_new[e]);
                    um[e] = um_new[e];
                    pscale[e] = um[e] == -INFINITY ? 0.f : ex2(m[e] - um[e]) * kPScale;
                }
            }
            float al[2];
            if constexpr (kSmall) {   // O's rows are 2t and 2t + 1; lane 4 r holds row r's
                al[0] = __shfl_sync(0xffffffffu, fall[0], 8 * t);
                al[1] = __shfl_sync(0xffffffffu, fall[0], 8 * t + 4);
            } else {
                al[0] = fall[0];
                al[1] = fall[kE - 1];
            }
#pragma unroll
            for (int s = 0; s < kAcc; ++s)
#pragma unroll
                for (int c = 0; c < 4; ++c) acc[s][c] *= al[kSmall ? c & 1 : c >> 1];
        }
        uint32_t pa[T::kKeys / 16][2 * kE];   // [.][2 (8-key half) + e] as the A operand, or [8-key half] as the B operand
#pragma unroll
        for (int e = 0; e < kE; ++e) {
            const float nm = m[e] == -INFINITY ? 0.f : -m[e];
            const uint64_t nm2 = f2_pack(nm, nm);
            // (Beyond fp32 only where a probability that would matter is 0 in fp32.)
            const float pv[2] = {kCache ? fminf(vs[0] * pscale[e], kMaxFloat) : 1.f,
                                 kCache ? fminf(vs[1] * pscale[e], kMaxFloat) : 1.f};
            uint64_t l2 = 0;
#pragma unroll
            for (int j = 0; j < T::kNT; ++j) {
                const float c = cs[e][j / 2];
                float x0, x1;
                f2_unpack(ffma2(f2_pack(sc[j][2 * e], sc[j][2 * e + 1]), f2_pack(c, c), nm2), x0, x1);
                const uint64_t p2 = f2_pack(ex2(x0), ex2(x1));
                l2 = fadd2(l2, p2);
                float p0, p1;
                if (kCache) {
                    f2_unpack(fmul2(p2, f2_pack(pv[j / 2], pv[j / 2])), p0, p1);
                    pa[j / 2][kE * (j & 1) + e] = pack_f16(p0, p1);
                } else {
                    f2_unpack(p2, p0, p1);
                    pa[j / 2][kE * (j & 1) + e] = pack_bf16(p0, p1);
                }
            }
            float s0, s1;
            f2_unpack(l2, s0, s1);
            l[e] += s0 + s1;
        }
        if constexpr (kCache) {
            if (!whole && a.N > 1 && key0 + T::kKeys > limit_all) {
                // The newest tokens, which some rows see and others do not: added row by row, and their V rows cleared
                // for the product, in which an unseen NaN would reach every row.  P goes through the K tile's space.
                const int r0 = max(limit_all - key0, 0), r1 = min(len - key0, T::kKeys);
                __syncwarp();
#pragma unroll
                for (int j = 0; j < T::kNT; ++j)
#pragma unroll
                    for (int e = 0; e < kE; ++e) {
                        const uint32_t p2 = pa[j / 2][kE * (j & 1) + e], row = kd + ((g + 8 * e) * T::kKeys + 8 * j) * 2;
                        sts_u16(row + T::key(2 * t) * 2, p2);
                        sts_u16(row + T::key(2 * t + 1) * 2, p2 >> 16);
                    }
                __syncwarp();
                for (int r = r0; r < r1; ++r) {
                    if (!(has >> (r >> 4) & 1)) continue;
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        // kSmall: row 2t + c over the columns of share g; else rows g, g + 8 over those of share 2t + c.
                        const int share = kSmall ? g : 2 * t + c;
                        uint32_t vw[T::kVW];
                        if constexpr (T::kRow == 64) lds8(vw, vd + T::at(r, share >> 1) + (share & 1) * 8);
                        else lds16(vw, vd + T::at(r, share));
#pragma unroll
                        for (int e = 0; e < kE; ++e) {
                            const int row = kSmall ? 2 * t + c : g + 8 * e;
                            if (key0 + r >= len - (a.N - 1 - (row0 + row) % a.N)) continue;
                            const float p = lds_f16(kd + (row * T::kKeys + r) * 2);
#pragma unroll
                            for (int w = 0; w < T::kVW; ++w)
#pragma unroll
                                for (int i4 = 0; i4 < 4; ++i4) {
                                    float& o = kSmall ? acc[2 * w + (i4 >> 1)][2 * (i4 & 1) + c] : acc[(kSmall ? 0 : 4 * w + i4)][2 * e + c];
                                    o = fmaf(p, e4m3_f32(vw[w], i4), o);
                                }
                        }
                    }
                }
                __syncwarp();
                for (int r = r0 + lane; r < r1; r += 32) {
#pragma unroll
                    for (int c = 0; c < T::kRow / 16; ++c) sts16_zero(vd + T::at(r, c));
                }
                __syncwarp();
            }
        }
#pragma unroll
        for (int u = 0; u < T::kKeys / 16; ++u) {
            uint32_t vr[4][T::kVW];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const uint32_t at = vd + vat[k & 1] + (16 * u + 8 * (k >> 1)) * (T::kRow < 128 ? T::kRow : 128);
                if constexpr (T::kRow == 64) {
                    lds8(vr[k], at);
                } else {
#pragma unroll
                    for (int s = 0; s < T::kRow / 128; ++s) lds16(vr[k] + 4 * s, at + s * (T::kKeys * 128));
                }
            }
#pragma unroll
            for (int w = 0; w < T::kVW; ++w) {
                const uint32_t a01 = prmt(vr[0][w], vr[1][w], sel_lo), a23 = prmt(vr[0][w], vr[1][w], sel_hi);
                const uint32_t b01 = prmt(vr[2][w], vr[3][w], sel_lo), b23 = prmt(vr[2][w], vr[3][w], sel_hi);
                if constexpr (kCache && kSmall) {
                    mma_f16(acc[2 * w], e4m3x2_f16(a01, 0), e4m3x2_f16(a01, 1), e4m3x2_f16(b01, 0), e4m3x2_f16(b01, 1), pa[u][0],
                            pa[u][1]);
                    mma_f16(acc[2 * w + 1], e4m3x2_f16(a23, 0), e4m3x2_f16(a23, 1), e4m3x2_f16(b23, 0), e4m3x2_f16(b23, 1),
                            pa[u][0], pa[u][1]);
                } else if constexpr (kCache) {
                    const uint32_t (&p)[2 * kE] = pa[u];
                    mma_f16(acc[4 * w + 0], p[0], p[1], p[2], p[3], e4m3x2_f16(a01, 0), e4m3x2_f16(b01, 0));
                    mma_f16(acc[4 * w + 1], p[0], p[1], p[2], p[3], e4m3x2_f16(a01, 1), e4m3x2_f16(b01, 1));
                    mma_f16(acc[4 * w + 2], p[0], p[1], p[2], p[3], e4m3x2_f16(a23, 0), e4m3x2_f16(b23, 0));
                    mma_f16(acc[4 * w + 3], p[0], p[1], p[2], p[3], e4m3x2_f16(a23, 1), e4m3x2_f16(b23, 1));
                } else if constexpr (kSmall) {
                    mma_bf16(acc[w], a01, a23, b01, b23, pa[u][0], pa[u][1]);
                } else {
                    const uint32_t (&p)[2 * kE] = pa[u];
                    mma_bf16(acc[2 * w + 0], p[0], p[1], p[2], p[3], a01, b01);
                    mma_bf16(acc[2 * w + 1], p[0], p[1], p[2], p[3], a23, b23);
                }
            }
        }
    }
    copy_wait<0>();
#pragma unroll
    for (int e = 0; e < kE; ++e) {
        l[e] += __shfl_xor_sync(0xffffffffu, l[e], 1);
        l[e] += __shfl_xor_sync(0xffffffffu, l[e], 2);
    }
    __syncthreads();   // the rings are free

    // Merge the warps: [warp][rows][D] fp32.  Rows and 16-column pieces are padded so that the lanes' stores spread over
    // the banks.
    constexpr int kRowPitch = D + D / 4 + 4, kWarpPitch = kTileRows * kRowPitch;
    auto col = [](int d) { return d + 4 * (d / 16); };
    float* so = reinterpret_cast<float*>(smem);
    float2* sml = reinterpret_cast<float2*>(so + kWarps * kWarpPitch);
    float unit[2] = {1.f, 1.f};   // of O's rows, as fall above
    if constexpr (kCache) {
        float own[kE];
#pragma unroll
        for (int e = 0; e < kE; ++e) own[e] = um[e] == -INFINITY ? 0.f : ex2(um[e] - m[e]) / kPScale;
        unit[0] = kSmall ? __shfl_sync(0xffffffffu, own[0], 8 * t) : own[0];
        unit[1] = kSmall ? __shfl_sync(0xffffffffu, own[0], 8 * t + 4) : own[kE - 1];
    }
    float* mine = so + warp * kWarpPitch;
    if constexpr (kSmall) {
        constexpr int kTilesPerWord = kCache ? 2 : 1;
#pragma unroll
        for (int w = 0; w < kAcc; ++w)
#pragma unroll
            for (int c = 0; c < 2; ++c)
                *reinterpret_cast<float2*>(mine + (2 * t + c) * kRowPitch +
                                           col(T::column(w / kTilesPerWord, g) + 2 * (w % kTilesPerWord))) =
                    make_float2(acc[w][c] * unit[c], acc[w][2 + c] * unit[c]);
    } else {
        constexpr int kCols = 4 / T::kElt;   // columns of a word of V
#pragma unroll
        for (int e = 0; e < 2; ++e)
#pragma unroll
            for (int c = 0; c < 2; ++c)
#pragma unroll
                for (int s = 0; s < kAcc; s += 2)
                    *reinterpret_cast<float2*>(mine + (g + 8 * e) * kRowPitch + col(T::column(s / kCols, 2 * t + c) + s % kCols)) =
                        make_float2(acc[s][2 * e + c] * unit[e], acc[s + 1][2 * e + c] * unit[e]);
    }
    if (t == 0) {
#pragma unroll
        for (int e = 0; e < kE; ++e) sml[warp * kTileRows + g + 8 * e] = make_float2(m[e], l[e]);
    }
    __syncthreads();
    constexpr int kPairs = D / 2;   // a thread takes two adjacent columns of a row
    const int rows = min(kTileRows, a.R - row0);
    for (int idx = threadIdx.x; idx < rows * kPairs; idx += kThreads) {
        const int r = idx / kPairs, d = 2 * (idx % kPairs);
        const int row = row0 + r;
        float mm = -INFINITY;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) mm = fmaxf(mm, sml[w * kTileRows + r].x);
        const float m0 = mm == -INFINITY ? 0.f : mm;
        float ll = 0.f, o0 = 0.f, o1 = 0.f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            const float2 ml = sml[w * kTileRows + r];
            const float c = ex2(ml.x - m0);
            const float2 v = *reinterpret_cast<const float2*>(so + w * kWarpPitch + r * kRowPitch + col(d));
            ll = fmaf(c, ml.y, ll);
            o0 = fmaf(c, v.x, o0);
            o1 = fmaf(c, v.y, o1);
        }
        if (a.splits == 1) {
            const float inv = ll > 0.f ? 1.f / ll : (ll == 0.f ? 0.f : ll);   // NaN stays NaN
            *reinterpret_cast<uint32_t*>(a.o + ((size_t)bh * a.R + row) * D + d) = pack_bf16(o0 * inv, o1 * inv);
            if (d == 0) a.lse[(size_t)bh * a.R + row] = ll == 0.f ? -INFINITY : (m0 + log2f(ll)) * 0.69314718055994531f;
        } else {
            const size_t at = (((size_t)bh * a.row_tiles + rt) * a.splits + split) * kTileRows + r;
            *reinterpret_cast<float2*>(a.part_o + at * D + d) = make_float2(o0, o1);
            if (d == 0) a.part_ml[at] = make_float2(mm, ll);
        }
    }
}

// Joins the splits of a row.  Partials are [group][split][rows of a group] for the row groups `first` onwards, groups
// counted over the heads.  kWarps warps share a row's splits (one warp where there are few splits and many rows; many
// where a few rows' chains of loads would take long) and add up in shared memory, in a fixed order.
struct CombineArgs {
    const float* part_o;
    const float2* part_ml;
    __nv_bfloat16* o;
    float* lse;
    int R, group, groups, splits;   // rows and groups of a head
    int64_t first, slots;           // slots: groups * rows of a group to join
};

template <int D, int kW>
__global__ void __launch_bounds__(kW == 1 ? 128 : kW * 32) rows_combine_kernel(const __grid_constant__ CombineArgs a) {
    constexpr int kC = D / 32, kRows = kW == 1 ? 4 : 1;   // rows of a CTA
    __shared__ float so[kW][D];
    __shared__ float sl[kW];
    griddep_wait();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t slot = (int64_t)blockIdx.x * kRows + (kW == 1 ? warp : 0);
    if (slot >= a.slots) return;
    const int64_t gi = slot / a.group, head = (gi + a.first) / a.groups;
    const int r = (int)(slot - gi * a.group), row = (int)(gi + a.first - head * a.groups) * a.group + r;
    if (row >= a.R) return;
    const size_t at0 = (size_t)gi * a.splits * a.group + r;
    float mm = -INFINITY;
    for (int s = lane; s < a.splits; s += 32) mm = fmaxf(mm, a.part_ml[at0 + (size_t)s * a.group].x);
#pragma unroll
    for (int o = 16; o; o >>= 1) mm = fmaxf(mm, __shfl_xor_sync(0xffffffffu, mm, o));
    const float m0 = mm == -INFINITY ? 0.f : mm;
    float ll = 0.f, o[kC];
#pragma unroll
    for (int c = 0; c < kC; ++c) o[c] = 0.f;
#pragma unroll 8
    for (int s = kW == 1 ? 0 : warp; s < a.splits; s += kW) {
        const size_t at = at0 + (size_t)s * a.group;
        const float2 ml = a.part_ml[at];
        const float c = ex2(ml.x - m0);
        ll = fmaf(c, ml.y, ll);
        const float* src = a.part_o + at * D + lane * kC;
#pragma unroll
        for (int i = 0; i < kC; i += 2) {
            const float2 v = *reinterpret_cast<const float2*>(src + i);
            o[i] = fmaf(c, v.x, o[i]);
            o[i + 1] = fmaf(c, v.y, o[i + 1]);
        }
    }
    if constexpr (kW > 1) {
#pragma unroll
        for (int c = 0; c < kC; ++c) so[warp][lane * kC + c] = o[c];
        if (lane == 0) sl[warp] = ll;
        __syncthreads();
        if (warp > 0) return;
        ll = 0.f;
#pragma unroll
        for (int c = 0; c < kC; ++c) o[c] = 0.f;
#pragma unroll
        for (int k = 0; k < kW; ++k) {
            ll += sl[k];
#pragma unroll
            for (int c = 0; c < kC; ++c) o[c] += so[k][lane * kC + c];
        }
    }
    const float inv = ll > 0.f ? 1.f / ll : (ll == 0.f ? 0.f : ll);   // NaN stays NaN
    const size_t out = (size_t)head * a.R + row;
    uint32_t* dst = reinterpret_cast<uint32_t*>(a.o + out * D + lane * kC);
#pragma unroll
    for (int i = 0; i < kC; i += 2) dst[i / 2] = pack_bf16(o[i] * inv, o[i + 1] * inv);
    if (lane == 0) a.lse[out] = ll == 0.f ? -INFINITY : (m0 + log2f(ll)) * 0.69314718055994531f;
}

template <int D, bool kCache, bool kSmall>
cudaError_t launch_rows(const RowsArgs& a, int64_t bh, cudaStream_t st) {
    // The rings, which the merge reuses, and their scales.
    using T = Tile<D, kCache, kSmall>;
    constexpr int smem = kWarps * (T::kRingBytes + T::kStages * 16);
    static_assert((kSmall ? 8 : 16) * (D + D / 4 + 4 + 2) * (int)sizeof(float) <= T::kRingBytes, "the merge fits the rings");
    cudaError_t e = set_max_dynamic_smem((const void*)rows_kernel<D, kCache, kSmall>, smem);
    if (e != cudaSuccess) return e;
    e = launch_dependent(rows_kernel<D, kCache, kSmall>, dim3((unsigned)(bh * a.row_tiles * a.splits)), dim3(kThreads), smem, st,
                         a);
    if (e == cudaSuccess) count_launches(1);
    return e;
}

template <bool kCache>
cudaError_t launch(RowsArgs a, int d, int64_t bh, const RowsPlan& p, void* workspace, cudaStream_t st) {
    a.splits = p.splits;
    a.row_tiles = p.row_tiles;
    a.part_o = (float*)workspace;
    a.part_ml = (float2*)((char*)workspace + p.ml_offset);
    const bool small = p.tile_rows == 8;
    cudaError_t e;
    if (d == 128) e = small ? launch_rows<128, kCache, true>(a, bh, st) : launch_rows<128, kCache, false>(a, bh, st);
    else e = small ? launch_rows<64, kCache, true>(a, bh, st) : launch_rows<64, kCache, false>(a, bh, st);
    if (e != cudaSuccess || p.splits == 1) return e;
    return launch_rows_combine(a.part_o, a.part_ml, a.o, a.lse, a.R, p.tile_rows, p.row_tiles, 0, bh * p.row_tiles, p.splits, d,
                               st);
}

}  // namespace

cudaError_t launch_rows_combine(const float* part_o, const float2* part_ml, void* o, float* lse, int R, int group, int groups,
                                int64_t first, int64_t count, int splits, int d, cudaStream_t st) {
    const CombineArgs a{part_o, part_ml, (__nv_bfloat16*)o, lse, R, group, groups, splits, first, count * group};
    // Warps a row.  The calls took, us: 76 splits of 16 rows 31.8 with 4 warps, 29.7 with 8, 28.5 with 16; 32 splits of 32 rows
    // 19.4 with one, 14.2 with 4; 4 splits of 256 rows 13.1 with one, 12.0 with 4; 4 splits of 26624 rows (the tiles' last
    // wave) are a warp each: four would be as many idle ones.
    const int warps = a.slots > 2048 ? 1 : splits > 16 ? 16 : 4;
    auto* f = d == 128 ? (warps == 16  ? rows_combine_kernel<128, 16>
                          : warps == 4 ? rows_combine_kernel<128, 4>
                                       : rows_combine_kernel<128, 1>)
                       : (warps == 16  ? rows_combine_kernel<64, 16>
                          : warps == 4 ? rows_combine_kernel<64, 4>
                                       : rows_combine_kernel<64, 1>);
    const int64_t ctas = warps > 1 ? a.slots : (a.slots + 3) / 4;
    if (ctas > INT32_MAX) return cudaErrorInvalidConfiguration;
    const cudaError_t e = launch_dependent(f, dim3((unsigned)ctas), dim3(warps > 1 ? 32 * warps : 128), 0, st, a);
    if (e == cudaSuccess) count_launches(1);
    return e;
}

RowsPlan rows_plan(int64_t bh, int R, int d, int64_t keys, int tile_keys) {
    RowsPlan p;
    p.tiles = false;
    p.tile_rows = R <= 8 ? 8 : 16;
    p.row_tiles = (R + p.tile_rows - 1) / p.tile_rows;
    const int64_t items = bh * p.row_tiles;
    // Few items: one wave of splits, of 128 KB of keys and values or more (16 heads x 512 bf16 keys of d =
    // 64 took 5 us either way, and a second kernel costs the host 6); where they leave slots idle and the splits stay
    // long, two to four fuller waves.  Many items: a few waves, which balance ragged lengths, of at least 32 tiles a CTA.
    // Measured with two CTAs an SM, us at splits for 1, 2, 4 and 8 waves: one request of 131072 tokens x 4 heads (4 items)
    // 31, 39, 56, 74; 8 x 2000 tokens x 8 heads (64 items) 15.4, 15.8, 15.7, 16.0 (19.6 at 32 tiles a CTA or more); 32 x 8191
    // bf16 keys x 4 heads (128 items) 48.5, 47.5, 46.4, 49.8; 64 x 4096 to 8192 tokens x 8 heads (512 items) 147, 139, 134, 140.
    const int64_t slots = ctas_per_sm(d, p.tile_rows == 8, tile_keys == kCacheTileKeys) * kPlanSms;
    int64_t splits;
    if (4 * items <= slots) {
        const int64_t bytes = keys * 2 * d * (tile_keys == kCacheTileKeys ? 1 : 2);   // of an item
        splits = slots / items;
        for (int waves = 2; waves <= 4 && splits * items * 100 < slots * (waves - 1) * 93; ++waves) {
            if (bytes / (waves * slots / items) < 512 << 10) break;
            splits = waves * slots / items;
        }
        if (splits > bytes / (128 << 10)) splits = bytes / (128 << 10);
    } else {
        splits = (4 * slots + items - 1) / items;
        if (splits > keys / (32 * tile_keys)) splits = keys / (32 * tile_keys);
    }
    p.splits = (int)splits;
    if (p.splits < 1) p.splits = 1;
    p.ml_offset = p.splits == 1 ? 0 : ((size_t)items * p.splits * p.tile_rows * d * sizeof(float) + 255) & ~(size_t)255;
    p.bytes = p.splits == 1 ? 0 : p.ml_offset + (size_t)items * p.splits * p.tile_rows * sizeof(float2);
    return p;
}

cudaError_t launch_cache_fwd(const CacheFwd& c, const RowsPlan& p, void* workspace, cudaStream_t st) {
    RowsArgs a = {};
    a.q = (const __nv_bfloat16*)c.q;
    a.o = (__nv_bfloat16*)c.o;
    a.lse = c.lse;
    a.k_scale = c.k_scale;
    a.v_scale = c.v_scale;
    a.table = c.table;
    a.lens = c.lens;
    a.R = c.Hq / c.Hk * c.N;
    a.N = c.N;
    a.Hk = c.Hk;
    a.cap = c.max_blocks * c.bs;
    a.max_blocks = c.max_blocks;
    a.n_blocks = c.n_blocks;
    a.bs_log2 = c.bs == 16 ? 4 : c.bs == 32 ? 5 : c.bs == 64 ? 6 : 7;
    a.scale_log2 = c.scale * 1.4426950408889634f;
    a.k = (const uint8_t*)c.k_cache;
    a.v = (const uint8_t*)c.v_cache;
    return launch<true>(a, c.d, (int64_t)c.B * c.Hk, p, workspace, st);
}

cudaError_t launch_cross_fwd_rows(const CrossFwd& c, const RowsPlan& p, void* workspace, cudaStream_t st) {
    RowsArgs a = {};
    a.q = (const __nv_bfloat16*)c.q;
    a.o = (__nv_bfloat16*)c.o;
    a.lse = c.lse;
    a.lens = c.key_lens;
    a.R = c.rows();
    a.N = 1;   // every row sees all of its keys
    a.Hk = c.Hk;
    a.cap = c.Nk;
    a.scale_log2 = c.scale * 1.4426950408889634f;
    a.k = (const uint8_t*)c.k;
    a.v = (const uint8_t*)c.v;
    return launch<false>(a, c.d, c.heads(), p, workspace, st);
}

}  // namespace fa
