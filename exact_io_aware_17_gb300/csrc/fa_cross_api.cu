// C entry points of attention over keys of another length and over the paged 8-bit cache: argument checks,
// workspace sizes, dispatch.  The declarations and their contracts are in include/fa.h.

#include <math.h>

#include "fa_internal.h"

namespace fa {
namespace {

fa_status check_cross(const char* fn, int B, int Hq, int Hk, int Nq, int Nk, int d, float scale) {
    if (B < 1 || Hq < 1 || Hk < 1 || Nq < 1 || Nk < 1 || d < 1)
        return set_error(FA_ERR_INVALID_ARG, "%s: B, Hq, Hk, Nq, Nk, d must be >= 1 (got B=%d Hq=%d Hk=%d Nq=%d Nk=%d d=%d)",
                         fn, B, Hq, Hk, Nq, Nk, d);
    if (Hq % Hk) return set_error(FA_ERR_INVALID_ARG, "%s: Hq must be a multiple of Hk (got %d, %d)", fn, Hq, Hk);
    if ((int64_t)B * Hq > INT32_MAX || (int64_t)(Hq / Hk) * Nq * d > INT32_MAX || (int64_t)Nk * d > INT32_MAX)
        return set_error(FA_ERR_INVALID_ARG, "%s: B*Hq, Hq/Hk*Nq*d and Nk*d must fit in int32", fn);
    return check_scale(fn, scale);
}

fa_status check_head_size(const char* fn, int d) {
    if (d != 64 && d != 128) return set_error(FA_ERR_UNSUPPORTED, "%s: d must be 64 or 128 (got %d)", fn, d);
    return FA_OK;
}

fa_status check_workspace(const char* fn, const void* workspace, size_t have, size_t need) {
    if (!need) return FA_OK;
    if (!workspace) return set_error(FA_ERR_INVALID_ARG, "%s: workspace is NULL", fn);
    if ((uintptr_t)workspace & 255u) return set_error(FA_ERR_INVALID_ARG, "%s: workspace is not 256-byte aligned", fn);
    if (have < need)
        return set_error(FA_ERR_INVALID_ARG, "%s: workspace holds %zu bytes, needs %zu", fn, have, need);
    return FA_OK;
}

fa_status check_int_ptr(const char* fn, const void* p, const char* name, unsigned align) {
    const void* ptrs[] = {p};
    const char* names[] = {name};
    return check_ptrs(fn, ptrs, names, 1, align);
}

// Few rows a key head stream through fa_rows.cu, more of them go to the tensor-core tiles.  Streamed and tiled, us, at
// rows 1, 8, 16, 24, 32, 48: 32 x 4 key heads of 4096 keys, d = 128: 47, 58; 48, 59; 54, 59; 65, 59; 66, 59; 91, 59;
// 2 x 8 of 1024, d = 64: 7.7, 9.0 at 1 row, 8.5, 9.1 at 16; 4 of 65536, d = 128: 27, 39 at 8 rows, 30, 40 at 16 and 32.
constexpr int kMaxStreamRows = 16;
struct CrossPlan {
    bool stream;
    RowsPlan rows;
    TilesPlan tiles;
    size_t bytes() const { return stream ? rows.bytes : tiles.bytes; }
};
CrossPlan cross_plan(int B, int Hq, int Hk, int Nq, int Nk, int d) {
    CrossPlan p = {};
    const int R = Hq / Hk * Nq;
    p.stream = R <= kMaxStreamRows;
    if (p.stream) p.rows = rows_plan((int64_t)B * Hk, R, d, Nk, kDenseTileKeys);
    else p.tiles = tiles_plan((int64_t)B * Hk, R, d, Nk);
    return p;
}

// Shape of a cache: blocks of 16, 32, 64 or 128 tokens.
fa_status check_cache(const char* fn, int H, int d, int n_blocks, int bs) {
    if (H < 1 || d < 1 || n_blocks < 1)
        return set_error(FA_ERR_INVALID_ARG, "%s: H, d, n_blocks must be >= 1 (got H=%d d=%d n_blocks=%d)", fn, H, d, n_blocks);
    if ((int64_t)n_blocks * H > INT32_MAX)
        return set_error(FA_ERR_INVALID_ARG, "%s: n_blocks*H must fit in int32 (got %d, %d)", fn, n_blocks, H);
    if (bs != 16 && bs != 32 && bs != 64 && bs != 128)
        return set_error(FA_ERR_UNSUPPORTED, "%s: block_size must be 16, 32, 64 or 128 (got %d)", fn, bs);
    return check_head_size(fn, d);
}

fa_status check_cache_fwd(const char* fn, int B, int Hq, int Hk, int N, int d, int n_blocks, int bs, int max_blocks) {
    if (B < 1 || Hq < 1 || N < 1 || max_blocks < 1)
        return set_error(FA_ERR_INVALID_ARG, "%s: B, Hq, N, max_blocks must be >= 1 (got B=%d Hq=%d N=%d max_blocks=%d)", fn,
                         B, Hq, N, max_blocks);
    fa_status st = check_cache(fn, Hk, d, n_blocks, bs);
    if (st) return st;
    if (Hq % Hk) return set_error(FA_ERR_INVALID_ARG, "%s: Hq must be a multiple of Hk (got %d, %d)", fn, Hq, Hk);
    if ((int64_t)B * Hq > INT32_MAX || (int64_t)(Hq / Hk) * N * d > INT32_MAX || (int64_t)max_blocks * bs > INT32_MAX - 256)
        return set_error(FA_ERR_INVALID_ARG, "%s: B*Hq, Hq/Hk*N*d and max_blocks*block_size must fit in int32", fn);
    return FA_OK;
}

// More rows a key head than two of a stream's 16 go to the tensor-core tiles where there are two tiles of 128 keys an SM or
// more.  Streamed and tiled, us, at rows 32, 48, 64, 128 of query heads (one token a request, requests of equal length): 64
// requests x 8192 tokens x 8 heads, d = 128: 288, 293; 425, 296; 535, 299; 1019, 424; d = 64: 186, 240; 274, 241; 338, 243; 643,
// 388; 16 x 1024 x 8, d = 128: 21.4, 15.8; 22.2, 16.5; 32.0, 17.0; 50.3, 21.1; 1 x 16384 x 4: 13.2, 15.4; 16.7, 16.2; 18.5,
// 16.8; 27.4, 21.7; 64 x 512 x 8: 34.0, 43.9; 47.8, 46.7; 60.2, 48.8; 111, 56.5; 1 x 1000 x 8 (64 tiles): 10.2, 15.1; 10.3,
// 15.8; 10.6, 16.2; 11.2, 20.6.  (The rule looks at rows and keys; rows that are new tokens have not been measured apart.)
bool cache_in_tiles(int64_t bh, int R, int64_t keys) {
    return R > 2 * kMaxStreamRows && bh * ((keys + 127) / 128) >= 2 * kPlanSms;
}

RowsPlan cache_plan_rows(int B, int Hq, int Hk, int N, int d, int bs, int max_blocks) {
    const int R = Hq / Hk * N;
    const int64_t keys = (int64_t)max_blocks * bs;
    return cache_in_tiles((int64_t)B * Hk, R, keys) ? cache_tiles_plan((int64_t)B * Hk, R, d, keys)
                                                    : rows_plan((int64_t)B * Hk, R, d, keys, kCacheTileKeys);
}

fa_status check_grid(const char* fn, int64_t bh, const RowsPlan& p) {
    if (bh * p.row_tiles * p.splits > INT32_MAX)
        return set_error(FA_ERR_INVALID_ARG, "%s: too many rows for one call", fn);
    return FA_OK;
}

}  // namespace
}  // namespace fa

using namespace fa;

extern "C" {

size_t fa_cross_fwd_workspace_size(int B, int Hq, int Hk, int Nq, int Nk, int d) {
    const fa_status st = check_cross("", B, Hq, Hk, Nq, Nk, d, 1.f);
    clear_error();
    if (st || (d != 64 && d != 128)) return 0;
    return cross_plan(B, Hq, Hk, Nq, Nk, d).bytes();
}

fa_status fa_cross_fwd(const void* q, const void* k, const void* v, const int* key_lens, void* o, float* lse, int B, int Hq,
                       int Hk, int Nq, int Nk, int d, float scale, void* workspace, size_t workspace_bytes, void* stream) {
    const char* fn = "fa_cross_fwd";
    clear_error();
    fa_status st = check_cross(fn, B, Hq, Hk, Nq, Nk, d, scale);
    if (st) return st;
    const void* ptrs[] = {q, k, v, o, lse};
    const char* names[] = {"q", "k", "v", "o", "lse"};
    if ((st = check_ptrs(fn, ptrs, names, 5))) return st;
    if ((st = check_head_size(fn, d))) return st;
    if (key_lens && (st = check_int_ptr(fn, key_lens, "key_lens", 4))) return st;
    const CrossPlan p = cross_plan(B, Hq, Hk, Nq, Nk, d);
    if ((st = check_workspace(fn, workspace, workspace_bytes, p.bytes()))) return st;
    if (p.stream && (st = check_grid(fn, (int64_t)B * Hk, p.rows))) return st;
    const CrossFwd c{q, k, v, key_lens, o, lse, B, Hq, Hk, Nq, Nk, d, scale};
    return launch_result(fn, p.stream ? launch_cross_fwd_rows(c, p.rows, workspace, (cudaStream_t)stream)
                                      : launch_cross_fwd_tiles(c, p.tiles, workspace, (cudaStream_t)stream));
}

size_t fa_cross_bwd_workspace_size(int B, int Hq, int Hk, int Nq, int Nk, int d) {
    const fa_status st = check_cross("", B, Hq, Hk, Nq, Nk, d, 1.f);
    clear_error();
    if (st || (d != 64 && d != 128)) return 0;
    return bwd_cross_plan((int64_t)B * Hk, Hq / Hk * Nq, d, Nk).bytes;
}

fa_status fa_cross_bwd(const void* q, const void* k, const void* v, const int* key_lens, const void* o, const void* dout,
                       const float* lse, void* dq, void* dk, void* dv, int B, int Hq, int Hk, int Nq, int Nk, int d,
                       float scale, void* workspace, size_t workspace_bytes, void* stream) {
    const char* fn = "fa_cross_bwd";
    clear_error();
    fa_status st = check_cross(fn, B, Hq, Hk, Nq, Nk, d, scale);
    if (st) return st;
    const void* ptrs[] = {q, k, v, o, dout, lse, dq, dk, dv};
    const char* names[] = {"q", "k", "v", "o", "dout", "lse", "dq", "dk", "dv"};
    if ((st = check_ptrs(fn, ptrs, names, 9))) return st;
    if ((st = check_head_size(fn, d))) return st;
    if (key_lens && (st = check_int_ptr(fn, key_lens, "key_lens", 4))) return st;
    const size_t need = bwd_cross_plan((int64_t)B * Hk, Hq / Hk * Nq, d, Nk).bytes;
    if ((st = check_workspace(fn, workspace, workspace_bytes, need))) return st;
    const CrossBwd c{{q, k, v, key_lens, const_cast<void*>(o), const_cast<float*>(lse), B, Hq, Hk, Nq, Nk, d, scale},
                     dout, dq, dk, dv};
    return launch_result(fn, launch_cross_bwd(c, workspace, (cudaStream_t)stream));
}

fa_status fa_cache_plan(const int* lens, const int* new_lens, int* block_table, const int* free_blocks, const int* used,
                        long long* slots, int* starts, int* total_lens, int* used_out, int B, int max_blocks, int n_free,
                        int max_tokens, int block_size, void* stream) {
    const char* fn = "fa_cache_plan";
    clear_error();
    if (B < 1 || max_blocks < 1 || n_free < 0 || max_tokens < 0 || max_tokens > INT32_MAX - 1024)
        return set_error(FA_ERR_INVALID_ARG, "%s: B, max_blocks must be >= 1, n_free >= 0, max_tokens in [0, 2^31 - 1025] (got "
                         "B=%d max_blocks=%d n_free=%d max_tokens=%d)", fn, B, max_blocks, n_free, max_tokens);
    fa_status st = check_cache(fn, 1, 64, 1, block_size);
    if (st) return st;
    if ((int64_t)max_blocks * block_size > INT32_MAX - 256 || B > INT32_MAX - 1024)
        return set_error(FA_ERR_INVALID_ARG, "%s: B and max_blocks*block_size must fit in int32", fn);
    const void* ptrs[] = {lens, new_lens, block_table, starts, total_lens, used_out};
    const char* names[] = {"lens", "new_lens", "block_table", "starts", "total_lens", "used_out"};
    if ((st = check_ptrs(fn, ptrs, names, 6, 4))) return st;
    if (n_free && (st = check_int_ptr(fn, free_blocks, "free_blocks", 4))) return st;
    if (used && (st = check_int_ptr(fn, used, "used", 4))) return st;
    if (max_tokens && (st = check_int_ptr(fn, slots, "slots", 8))) return st;
    // Thread blocks read lengths, table and free blocks while others write, so no output may share memory with an input
    // or another output.
    const struct { const void* p; size_t bytes; } at[] = {
        {block_table, (size_t)B * max_blocks * 4}, {slots, (size_t)max_tokens * 8}, {starts, ((size_t)B + 1) * 4},
        {total_lens, (size_t)B * 4}, {used_out, 4},                                    // outputs, then inputs
        {lens, (size_t)B * 4}, {new_lens, (size_t)B * 4}, {free_blocks, (size_t)n_free * 4}, {used, used ? (size_t)4 : 0}};
    for (int i = 0; i < 5; ++i)
        for (int j = i + 1; j < 9; ++j)
            if (at[i].bytes && at[j].bytes && (uintptr_t)at[i].p < (uintptr_t)at[j].p + at[j].bytes &&
                (uintptr_t)at[j].p < (uintptr_t)at[i].p + at[i].bytes)
                return set_error(FA_ERR_INVALID_ARG, "%s: an output overlaps an input or another output", fn);
    return launch_result(fn, launch_cache_plan(lens, new_lens, block_table, free_blocks, used, (int64_t*)slots, starts,
                                               total_lens, used_out, B, max_blocks, n_free, max_tokens, block_size,
                                               (cudaStream_t)stream));
}

fa_status fa_cache_append(const void* k, const void* v, const long long* slots, void* k_cache, void* v_cache, float* k_scale,
                          float* v_scale, int T, int H, int d, long long k_token_stride, long long k_head_stride,
                          long long v_token_stride, long long v_head_stride, int n_blocks, int block_size, void* stream) {
    const char* fn = "fa_cache_append";
    clear_error();
    if (T < 0 || T > INT32_MAX - 1024) return set_error(FA_ERR_INVALID_ARG, "%s: T must be in [0, 2^31 - 1025] (got %d)", fn, T);
    fa_status st = check_cache(fn, H, d, n_blocks, block_size);
    if (st) return st;
    // Strides of a single token or head are never used.
    if (T <= 1) k_token_stride = v_token_stride = 0;
    if (H == 1) k_head_stride = v_head_stride = 0;
    const long long strides[] = {k_token_stride, k_head_stride, v_token_stride, v_head_stride};
    for (long long s : strides)
        if (s < 0 || s % 8) return set_error(FA_ERR_INVALID_ARG, "%s: strides must be >= 0 and multiples of 8 (got %lld)", fn, s);
    if (T == 0) return FA_OK;
    const void* ptrs[] = {k, v, k_cache, v_cache};
    const char* names[] = {"k", "v", "k_cache", "v_cache"};
    if ((st = check_ptrs(fn, ptrs, names, 4))) return st;
    if ((st = check_int_ptr(fn, slots, "slots", 8))) return st;
    if ((st = check_int_ptr(fn, k_scale, "k_scale", 4)) || (st = check_int_ptr(fn, v_scale, "v_scale", 4))) return st;
    const CacheAppend c{k, v, (const int64_t*)slots, k_cache, v_cache, k_scale, v_scale, {k_token_stride, v_token_stride},
                        {k_head_stride, v_head_stride}, T, H, d, n_blocks, block_size};
    return launch_result(fn, launch_cache_append(c, (cudaStream_t)stream));
}

size_t fa_cache_fwd_workspace_size(int B, int Hq, int Hk, int N, int d, int block_size, int max_blocks) {
    const fa_status st = check_cache_fwd("", B, Hq, Hk, N, d, 1, block_size, max_blocks);
    clear_error();
    if (st) return 0;
    return cache_plan_rows(B, Hq, Hk, N, d, block_size, max_blocks).bytes;
}

fa_status fa_cache_fwd(const void* q, const void* k_cache, const void* v_cache, const float* k_scale, const float* v_scale,
                       const int* block_table, const int* lens, void* o, float* lse, int B, int Hq, int Hk, int N, int d,
                       int n_blocks, int block_size, int max_blocks, float scale, void* workspace, size_t workspace_bytes,
                       void* stream) {
    const char* fn = "fa_cache_fwd";
    clear_error();
    fa_status st = check_cache_fwd(fn, B, Hq, Hk, N, d, n_blocks, block_size, max_blocks);
    if (st || (st = check_scale(fn, scale))) return st;
    const void* ptrs[] = {q, k_cache, v_cache, o, lse};
    const char* names[] = {"q", "k_cache", "v_cache", "o", "lse"};
    if ((st = check_ptrs(fn, ptrs, names, 5))) return st;
    const void* words[] = {k_scale, v_scale, block_table, lens};
    const char* word_names[] = {"k_scale", "v_scale", "block_table", "lens"};
    if ((st = check_ptrs(fn, words, word_names, 4, 4))) return st;
    const RowsPlan p = cache_plan_rows(B, Hq, Hk, N, d, block_size, max_blocks);
    if ((st = check_workspace(fn, workspace, workspace_bytes, p.bytes))) return st;
    if ((st = check_grid(fn, (int64_t)B * Hk, p))) return st;
    const CacheFwd c{q, k_cache, v_cache, k_scale, v_scale, block_table, lens, o, lse, B, Hq, Hk, N, d, n_blocks, block_size,
                     max_blocks, scale};
    return launch_result(fn, p.tiles ? launch_cache_fwd_tiles(c, p, workspace, (cudaStream_t)stream)
                                     : launch_cache_fwd(c, p, workspace, (cudaStream_t)stream));
}

}  // extern "C"
