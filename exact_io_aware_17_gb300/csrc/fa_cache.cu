// The paged 8-bit key/value cache: the plan of a step (block tables and slots from the requests' lengths)
// and the append of new tokens (fa_cache_plan, fa_cache_append; contracts in include/fa.h).
//
// A cache block holds `bs` tokens of every key/value head as e4m3 codes, [block][head][token][d], and one
// fp32 scale for each block and head.  Scales are powers of two: e4m3 is a floating-point format, so another
// scale would gain range but no precision, and with powers of two dividing by a scale and moving a block to a
// larger one are exact (but for codes that reach e4m3's subnormals), whatever the order of the appends.

#include <cuda_bf16.h>
#include <limits.h>
#include <stdint.h>

#include "fa_internal.h"
#include "fa_ptx.cuh"

namespace fa {
namespace {

using namespace ptx;

// ------------------------------------------------------------------------------------------------ plan
// Every CTA scans all requests (two prefix sums: packed tokens, then new blocks) and then writes its own
// share of the slots and of the table rows, so that one launch does it all and no CTA waits for another.
// The scan reads 8 bytes a request from L2 and is repeated by at most one CTA an SM.
constexpr int kPlanThreads = 512;   // = requests per scan step

struct PlanArgs {
    const int* lens;
    const int* new_lens;
    int* table;
    const int* free_blocks;
    const int* used;
    int64_t* slots;
    int* starts;
    int* total;
    int* used_out;
    int B, max_blocks, n_free, max_tokens, bs;
};

// Exclusive prefix sum of x over the CTA's threads; *sum gets the total.  All threads call it.
__device__ __forceinline__ long long cta_scan(long long x, long long* warp_sums, long long* sum) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    long long y = x;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long z = __shfl_up_sync(0xffffffffu, y, o);
        if (lane >= o) y += z;
    }
    __syncthreads();   // the previous scan's readers are done with warp_sums
    if (lane == 31) warp_sums[warp] = y;
    __syncthreads();
    long long before = 0, all = 0;
#pragma unroll
    for (int w = 0; w < kPlanThreads / 32; ++w) {
        if (w < warp) before += warp_sums[w];
        all += warp_sums[w];
    }
    *sum = all;
    return before + y - x;
}

__global__ void __launch_bounds__(kPlanThreads) cache_plan_kernel(PlanArgs a) {
    __shared__ long long warp_sums[kPlanThreads / 32];
    __shared__ int s_start[kPlanThreads + 1], s_len[kPlanThreads], s_total[kPlanThreads], s_old[kPlanThreads],
        s_need[kPlanThreads];
    __shared__ long long s_base[kPlanThreads];
    const int tid = threadIdx.x;
    griddep_wait();   // the kernel ahead on the stream may have written the lengths
    griddep_launch_dependents();
    const long long cap = (long long)a.max_blocks * a.bs;
    // This CTA's share of the packed tokens.
    const long long share = ((long long)a.max_tokens + gridDim.x - 1) / gridDim.x;
    const int t0 = (int)min((long long)a.max_tokens, share * blockIdx.x);
    const int t1 = (int)min((long long)a.max_tokens, share * (blockIdx.x + 1));
    const long long used0 = a.used ? max(*a.used, 0) : 0;
    long long tokens = 0, blocks = used0;   // before this step's requests
    for (int b0 = 0; b0 < a.B; b0 += kPlanThreads) {
        const int b = b0 + tid;
        const bool live = b < a.B;
        const long long n = live ? max(a.new_lens[b], 0) : 0;
        const long long len = live ? min((long long)max(a.lens[b], 0), cap) : 0;
        long long sum;
        const long long before = tokens + cta_scan(n, warp_sums, &sum);
        const int start = (int)min(before, (long long)a.max_tokens);
        const int stop = (int)min(before + n, (long long)a.max_tokens);
        tokens += sum;
        const long long end = min(len + (stop - start), cap);
        const int old = (int)((len + a.bs - 1) / a.bs);
        const int need = (int)((end + a.bs - 1) / a.bs) - old;
        const long long base = blocks + cta_scan(need, warp_sums, &sum);
        blocks += sum;
        const int got = (int)min(max((long long)a.n_free - base, 0LL), (long long)need);
        const int total = (int)min(end, (long long)(old + got) * a.bs);
        s_start[tid] = start;
        if (tid == kPlanThreads - 1) s_start[kPlanThreads] = stop;
        s_len[tid] = (int)len;
        s_total[tid] = total;
        s_old[tid] = old;
        s_need[tid] = need;
        s_base[tid] = base;
        if (live && blockIdx.x == 0) {
            a.starts[b] = start;
            a.total[b] = total;
        }
        __syncthreads();
        const int count = min(kPlanThreads, a.B - b0);
        // Slots of this CTA's tokens among these requests: the request by bisection in shared memory.
        const int u0 = max(t0, s_start[0]), u1 = min(t1, s_start[kPlanThreads]);
        for (int t = u0 + tid; t < u1; t += kPlanThreads) {
            int lo = 0, hi = count - 1;   // the last request with start <= t (empty ones share their start)
            while (lo < hi) {
                const int mid = (lo + hi + 1) >> 1;
                if (s_start[mid] <= t) lo = mid;
                else hi = mid - 1;
            }
            const long long pos = (long long)s_len[lo] + (t - s_start[lo]);
            int64_t slot = -1;
            if (pos < s_total[lo]) {
                const int j = (int)(pos / a.bs), old = s_old[lo];
                const int block = j < old ? a.table[(size_t)(b0 + lo) * a.max_blocks + j]
                                          : a.free_blocks[s_base[lo] + (j - old)];
                if (block >= 0) slot = (int64_t)block * a.bs + pos % a.bs;
            }
            a.slots[t] = slot;
        }
        // New table entries, one warp a request.  Entries of earlier blocks are only read (above), so the
        // CTAs' reads and writes of the table never meet.
        const int warps = gridDim.x * (kPlanThreads / 32);
        for (int i = blockIdx.x * (kPlanThreads / 32) + (tid >> 5); i < count; i += warps) {
            const int need_i = s_need[i];
            int* row = a.table + (size_t)(b0 + i) * a.max_blocks + s_old[i];
            for (int j = tid & 31; j < need_i; j += 32) {
                const long long at = s_base[i] + j;
                row[j] = at < a.n_free ? a.free_blocks[at] : -1;
            }
        }
        __syncthreads();
    }
    const int planned = (int)min(tokens, (long long)a.max_tokens);
    for (int t = max(t0, planned) + tid; t < t1; t += kPlanThreads) a.slots[t] = -1;
    if (blockIdx.x == 0 && tid == 0) {
        a.starts[a.B] = planned;
        *a.used_out = (int)min(blocks, (long long)INT_MAX);
    }
}

// ---------------------------------------------------------------------------------------------- append
constexpr int kAppendThreads = 128;
constexpr int kAppendHold = 8;       // 16-byte loads of a lane that stay in registers between a run's two passes
constexpr int kAppendWarps = 6000;   // warps that fill the GPU a little more than once (152 SMs, 24 resident)
struct AppendArgs {
    const __nv_bfloat16* x[2];       // keys, values
    uint8_t* cache[2];
    float* scale[2];
    int64_t token_stride[2], head_stride[2];
    const int64_t* slots;
    int T, H, bs, window;            // window: packed tokens whose runs one warp takes, 1 .. 32
    int64_t n_slots, items;          // items: windows * H * 2
};

__device__ __forceinline__ uint32_t pack_e4m3x4(float a, float b, float c, float d) {
    uint16_t lo, hi;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(b), "f"(a));
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(d), "f"(c));
    return (uint32_t)lo | ((uint32_t)hi << 16);
}
__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }
// The larger magnitudes of two pairs of bf16, NaN left out.
__device__ __forceinline__ uint32_t max_abs2(uint32_t m, uint32_t w) {
    uint32_t r;
    asm("max.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(m), "r"(w & 0x7fff7fffu));
    return r;
}
// A pair of bf16 with zeros in the place of infinities and NaN.
__device__ __forceinline__ uint32_t finite2(uint32_t w) {
    return ((w & 0x7f80u) == 0x7f80u ? 0u : w & 0xffffu) | ((w & 0x7f800000u) == 0x7f800000u ? 0u : w & 0xffff0000u);
}

// The least power of two s >= 2^-100 with amax <= 448 s; 448 = 1.75 * 2^8.
__device__ __forceinline__ float block_scale(float amax) {
    const uint32_t u = __float_as_uint(amax);
    const int e = (int)(u >> 23) - 127 - 8 + ((u & 0x7fffffu) > 0x600000u ? 1 : 0);
    return __uint_as_float((uint32_t)(max(e, -100) + 127) << 23);
}

// One warp takes one run (tokens next to each other in the packed order and in one block) of one head, keys or
// values: the largest magnitude first, then the codes; the values of short runs stay in registers between the two
// passes, longer ones are read again from L2.  Lanes hold 8 values each (16-byte loads).  Bound by HBM: prompts of 65536
// tokens x 8 heads of 128 in blocks of 16 take 66 us (6.1 TB/s read and written), of 131072 128 us (6.3; blocks of 32, 64 and
// 128: 142, 131, 182), 16 ragged ones of up to 2048 tokens 21 to 28 us for blocks of 16 to 128 tokens (4.8 to 3.6 TB/s), 256
// single tokens 5.8 us.  Holding 16 loads instead of 8 (24.0 against 22.5
// us in blocks of 32) and a CTA a run instead of a warp (26.7 against 28.4 us in blocks of 128, 26.2 against 24.6 in
// blocks of 64) were not worth it.
template <int D>
__device__ void append_run(const AppendArgs& a, int which, int h, int t, int64_t slot, int rows) {
    constexpr int kLpr = D / 8, kRpp = 32 / kLpr;   // lanes per row, rows per pass
    constexpr int kHold = kAppendHold, kStep = kHold * kRpp;
    const int lane = threadIdx.x & 31, sub = lane / kLpr, part = lane % kLpr;
    const int64_t block = slot / a.bs;
    const int off = (int)(slot - block * a.bs);
    const __nv_bfloat16* x = a.x[which] + (int64_t)t * a.token_stride[which] + (int64_t)h * a.head_stride[which] + part * 8;
    const int64_t ts = a.token_stride[which];
    uint8_t* out = a.cache[which] + ((block * a.H + h) * a.bs) * D + part * 8;

    uint4 held[kHold];
    float amax;
    // The largest finite magnitude.  Infinities are rare: found, they are left out in a second pass.
    auto largest = [&](bool leave_out) {
        uint32_t m2 = 0;
        for (int r0 = 0; r0 < rows; r0 += kStep) {
#pragma unroll
            for (int i = 0; i < kHold; ++i) {
                const int r = r0 + i * kRpp + sub;
                held[i] = r < rows ? *reinterpret_cast<const uint4*>(x + r * ts) : make_uint4(0, 0, 0, 0);
            }
#pragma unroll
            for (int i = 0; i < kHold; ++i) {
                const uint32_t w[4] = {held[i].x, held[i].y, held[i].z, held[i].w};
#pragma unroll
                for (int j = 0; j < 4; ++j) m2 = max_abs2(m2, leave_out ? finite2(w[j]) : w[j]);
            }
        }
#pragma unroll
        for (int o = 16; o; o >>= 1) m2 = max_abs2(m2, __shfl_xor_sync(0xffffffffu, m2, o));
        amax = fmaxf(bf16_lo(m2), bf16_hi(m2));
    };
    largest(false);
    if (!(amax <= 3.402823466e38f)) largest(true);
    float* sp = a.scale[which] + block * a.H + h;
    float s = block_scale(amax);
    if (off > 0) {   // earlier tokens in the block: its scale never shrinks
        const float old = *sp;
        if (old >= s) {
            s = old;
        } else {
            const float ratio = old / s;
            for (int r = sub; r < off; r += kRpp) {
                uint2* p = reinterpret_cast<uint2*>(out + (int64_t)r * D);
                const uint2 c = *p;
                float f[8];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const uint32_t w = j < 2 ? c.x : c.y;
                    uint32_t h2;
                    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h2) : "h"((uint16_t)(w >> (16 * (j & 1)))));
                    float2 v;
                    asm("{.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\tcvt.f32.f16 %0, l;\n\tcvt.f32.f16 %1, h;\n\t}"
                        : "=f"(v.x), "=f"(v.y) : "r"(h2));
                    f[2 * j] = v.x * ratio;
                    f[2 * j + 1] = v.y * ratio;
                }
                *p = make_uint2(pack_e4m3x4(f[0], f[1], f[2], f[3]), pack_e4m3x4(f[4], f[5], f[6], f[7]));
            }
        }
    }
    __syncwarp();
    if (lane == 0) *sp = s;
    const float inv = 1.f / s;   // exact, a power of two (a caller's own scale need not be one)
    out += (int64_t)off * D;
    const bool all_held = rows <= kStep;
    for (int r0 = 0; r0 < rows; r0 += kStep) {
#pragma unroll
        for (int i = 0; i < kHold; ++i) {
            const int r = r0 + i * kRpp + sub;
            if (!all_held && r < rows) held[i] = *reinterpret_cast<const uint4*>(x + r * ts);
        }
#pragma unroll
        for (int i = 0; i < kHold; ++i) {
            const int r = r0 + i * kRpp + sub;
            if (r >= rows) continue;
            const uint4 w = held[i];
            *reinterpret_cast<uint2*>(out + (int64_t)r * D) =
                make_uint2(pack_e4m3x4(bf16_lo(w.x) * inv, bf16_hi(w.x) * inv, bf16_lo(w.y) * inv, bf16_hi(w.y) * inv),
                           pack_e4m3x4(bf16_lo(w.z) * inv, bf16_hi(w.z) * inv, bf16_lo(w.w) * inv, bf16_hi(w.w) * inv));
        }
    }
}

// A warp takes the runs of one head, keys or values, that begin in its window of packed tokens.  Neighbouring warps
// take neighbouring heads, whose rows lie next to each other.  A step of single tokens wants windows of one token
// (its runs are one token each, and a warp takes its runs one after another), a long prompt wide ones: most of its
// tokens follow in another's run.
template <int D>
__global__ void __launch_bounds__(kAppendThreads) cache_append_kernel(const __grid_constant__ AppendArgs a) {
    const int lane = threadIdx.x & 31;
    griddep_wait();   // the kernel ahead on the stream may have written the slots or the values
    griddep_launch_dependents();
    const int64_t item = (int64_t)blockIdx.x * (kAppendThreads / 32) + (threadIdx.x >> 5);
    if (item >= a.items) return;
    const int64_t pair = item / a.H;
    const int h = (int)(item - pair * a.H), which = (int)(pair & 1);
    const int w0 = (int)(pair >> 1) * a.window, t = w0 + lane;
    const bool mine = lane < a.window && t < a.T;
    const int64_t slot = mine ? a.slots[t] : -1;
    const int64_t prev = mine && t > 0 ? a.slots[t - 1] : -1;
    const bool valid = slot >= 0 && slot < a.n_slots;
    const bool follows = valid && t > 0 && prev == slot - 1 && slot % a.bs != 0;
    uint32_t starts = __ballot_sync(0xffffffffu, valid && !follows);
    const uint32_t cont = __ballot_sync(0xffffffffu, follows);
    while (starts) {
        const int first = __ffs(starts) - 1;
        starts &= starts - 1;
        const int64_t s0 = __shfl_sync(0xffffffffu, slot, first);
        // Tokens that follow within the window, then past it (a block holds at most bs tokens).
        int rows = first == 31 ? 1 : __ffs(~(cont >> (first + 1)));
        if (first + rows == a.window) {
            while (true) {   // 32 slots at a time: the first that does not go on ends the run
                const int u = w0 + first + rows + lane;
                const int64_t s = s0 + rows + lane;
                const bool on = u < a.T && s / a.bs == s0 / a.bs && a.slots[u] == s;
                const uint32_t stop = ~__ballot_sync(0xffffffffu, on);
                rows += stop ? __ffs(stop) - 1 : 32;
                if (stop) break;
            }
        }
        append_run<D>(a, which, h, w0 + first, s0, rows);
    }
}

}  // namespace

cudaError_t launch_cache_plan(const int* lens, const int* new_lens, int* table, const int* free_blocks, const int* used,
                              int64_t* slots, int* starts, int* total, int* used_out, int B, int max_blocks, int n_free,
                              int max_tokens, int bs, cudaStream_t st) {
    PlanArgs a{lens, new_lens, table, free_blocks, used, slots, starts, total, used_out, B, max_blocks, n_free, max_tokens, bs};
    const int work = max_tokens / 1024 + 1;
    const int grid = work < device_sm_count() ? work : device_sm_count();
    const cudaError_t e = launch_dependent(cache_plan_kernel, dim3(grid), dim3(kPlanThreads), 0, st, a);
    if (e == cudaSuccess) count_launches(1);
    return e;
}

cudaError_t launch_cache_append(const CacheAppend& c, cudaStream_t st) {
    AppendArgs a;
    a.x[0] = (const __nv_bfloat16*)c.k;
    a.x[1] = (const __nv_bfloat16*)c.v;
    a.cache[0] = (uint8_t*)c.k_cache;
    a.cache[1] = (uint8_t*)c.v_cache;
    a.scale[0] = c.k_scale;
    a.scale[1] = c.v_scale;
    for (int i = 0; i < 2; ++i) {
        a.token_stride[i] = c.token_stride[i];
        a.head_stride[i] = c.head_stride[i];
    }
    a.slots = c.slots;
    a.T = c.T;
    a.H = c.H;
    a.bs = c.bs;
    a.n_slots = (int64_t)c.n_blocks * c.bs;
    const int64_t wide = (int64_t)c.T * c.H * 2 / kAppendWarps;
    a.window = wide < 1 ? 1 : wide > 32 ? 32 : (int)wide;
    a.items = ((int64_t)c.T + a.window - 1) / a.window * c.H * 2;
    const int64_t ctas = (a.items + kAppendThreads / 32 - 1) / (kAppendThreads / 32);
    if (ctas > INT32_MAX) return cudaErrorInvalidConfiguration;
    const unsigned grid = (unsigned)ctas;
    const cudaError_t e = launch_dependent(c.d == 128 ? cache_append_kernel<128> : cache_append_kernel<64>, dim3(grid),
                                           dim3(kAppendThreads), 0, st, a);
    if (e == cudaSuccess) count_launches(1);
    return e;
}

}  // namespace fa
