// C ABI of the 8-bit key/value cache (include/mlora.h): argument checks, the handle's
// workspace, and launches.  Host side only; the caller owns the pages.
#include <cuda_runtime.h>

#include <cstdarg>
#include <cstdio>
#include <new>

#include "../../include/mlora.h"
#include "attend.h"
#include "tc.h"

using namespace mlora;

struct mlora_cache {
    int device = 0;
    CachePages pages{};
    int q_heads = 0;
    char* ws = nullptr;       // the status word, the join counters, the partial results
    AttendWs attend{};
    Divide page_div{}, group_div{};
};

namespace {

mlora_status fail(mlora_status s, const char* fmt, ...) {
    char buf[512];
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(buf, sizeof buf, fmt, ap);
    va_end(ap);
    set_last_error(buf);
    return s;
}

mlora_status cuda_fail(cudaError_t e, const char* what) {
    cudaGetLastError();   // reported here: not the next launch's error
    return fail(MLORA_ERR_CUDA, "%s: %s (%s)", what, cudaGetErrorName(e), cudaGetErrorString(e));
}

#define CU_TRY(expr)                                              \
    do {                                                          \
        cudaError_t e_ = (expr);                                  \
        if (e_ != cudaSuccess) return cuda_fail(e_, #expr);       \
    } while (0)

// Makes the cache's device current for the scope of one call and restores the caller's.
struct DeviceGuard {
    int prev = -1;
    bool moved = false;
    cudaError_t err = cudaSuccess;
    explicit DeviceGuard(int dev) {
        err = cudaGetDevice(&prev);
        if (err == cudaSuccess && prev != dev) {
            err = cudaSetDevice(dev);
            moved = err == cudaSuccess;
        }
    }
    ~DeviceGuard() {
        if (moved) cudaSetDevice(prev);
    }
};

bool aligned16(const void* p) { return ((uintptr_t)p & 15u) == 0; }

// The arguments that append, read and attend share.  `run` is false where the call has
// nothing to do (no rows or no sequences).
mlora_status check_step(mlora_cache_t c, mlora_dtype dtype, int T, const int32_t* offsets, const int32_t* lengths,
                        const int32_t* pages, int n_seqs, int width, int max_new, CacheStep* step, bool* run) {
    if (!c) return fail(MLORA_ERR_INVALID_ARG, "cache is NULL");
    if (dtype != MLORA_F32 && dtype != MLORA_BF16) return fail(MLORA_ERR_INVALID_ARG, "dtype %d", (int)dtype);
    if (T < 0 || n_seqs < 0 || width < 0 || max_new < 0)
        return fail(MLORA_ERR_INVALID_ARG, "T %d, n_seqs %d, width %d or max_new %d is negative", T, n_seqs, width,
                    max_new);
    if (n_seqs > 65535 || (long long)width * c->pages.page > 1 << 30)
        return fail(MLORA_ERR_INVALID_ARG, "n_seqs %d exceeds 65535, or width %d holds more than 2^30 tokens", n_seqs,
                    width);
    if (!offsets && T != n_seqs)
        return fail(MLORA_ERR_INVALID_ARG, "without offsets T %d must equal n_seqs %d", T, n_seqs);
    *run = T > 0 && n_seqs > 0 && max_new > 0;
    if (!*run) return MLORA_OK;
    if (!lengths || (!pages && width > 0)) return fail(MLORA_ERR_INVALID_ARG, "lengths/pages is NULL");
    *step = CacheStep{offsets, lengths, pages, n_seqs, width, T, max_new < T ? max_new : T};
    return MLORA_OK;
}

mlora_status check_rows(const char* name, const void* p, int64_t row, int64_t head, mlora_dtype dtype) {
    const int64_t unit = dtype == MLORA_BF16 ? 8 : 4;   // elements per 16 bytes
    if (!p) return fail(MLORA_ERR_INVALID_ARG, "%s is NULL", name);
    if (!aligned16(p) || row % unit || head % unit || row < 0 || head < 0)
        return fail(MLORA_ERR_INVALID_ARG, "%s: 16-byte alignment (strides %lld, %lld elements)", name, (long long)row,
                    (long long)head);
    return MLORA_OK;
}

// The codes as [n_pages x heads x page] rows of `dim` bytes, in boxes of 16 tokens; a box
// is 64 or 128 columns wide, its columns past `dim` and rows past the end read as zero.
bool encode_codes(CUtensorMap* map, const void* codes, const CachePages& c) {
    const bool narrow = c.dim <= 64;
    cuuint64_t dims[2] = {(cuuint64_t)c.dim, (cuuint64_t)c.n_pages * c.heads * c.page};
    cuuint64_t strides[1] = {(cuuint64_t)c.dim};
    cuuint32_t box[2] = {narrow ? 64u : 128u, 16};
    return tc_encode_typed(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, codes, 2, dims, strides, box,
                           narrow ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B);
}

}  // namespace

extern "C" {

mlora_status mlora_cache_create(void* k_codes, float* k_scale, void* v_codes, float* v_scale, int n_pages,
                                int page_size, int kv_heads, int head_dim, int q_heads, uint64_t prompt_bytes,
                                mlora_cache_t* out) {
    if (!out) return fail(MLORA_ERR_INVALID_ARG, "out is NULL");
    *out = nullptr;
    if (!k_codes || !k_scale || !v_codes || !v_scale) return fail(MLORA_ERR_INVALID_ARG, "codes/scale is NULL");
    if (!aligned16(k_codes) || !aligned16(v_codes)) return fail(MLORA_ERR_INVALID_ARG, "codes must be 16-byte aligned");
    if (((uintptr_t)k_scale | (uintptr_t)v_scale) & 3u) return fail(MLORA_ERR_INVALID_ARG, "scales must be 4-byte aligned");
    if (n_pages < 1 || kv_heads < 1 || q_heads < 1 || q_heads > 32767 || q_heads % kv_heads)
        return fail(MLORA_ERR_INVALID_ARG, "n_pages %d, kv_heads %d, q_heads %d", n_pages, kv_heads, q_heads);
    if (page_size < 16 || page_size > 256 || page_size % 16 || head_dim < 16 || head_dim > 256 || head_dim % 16)
        return fail(MLORA_ERR_UNSUPPORTED, "page_size %d and head_dim %d must be multiples of 16 in [16, 256]", page_size,
                    head_dim);
    if ((long long)n_pages * kv_heads >= (1ll << 31) / page_size)
        return fail(MLORA_ERR_UNSUPPORTED, "n_pages %d x kv_heads %d x page_size %d exceeds 2^31", n_pages, kv_heads,
                    page_size);
    mlora_cache* c = new (std::nothrow) mlora_cache;
    if (!c) return fail(MLORA_ERR_OOM, "host memory");
    c->pages = CachePages{(int8_t*)k_codes, (int8_t*)v_codes, k_scale, v_scale, n_pages, page_size, kv_heads, head_dim};
    c->q_heads = q_heads;
    c->page_div = divide_by(page_size);
    c->group_div = divide_by(q_heads / kv_heads);
    cudaError_t e = cudaGetDevice(&c->device);
    int sms = 0;
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, c->device);
    const size_t ctas = (size_t)sms * ATTEND_OCC, head = 256 + (ctas * sizeof(int) + 255) / 256 * 256;
    const size_t split = 2 * ctas * ATTEND_SLOT * sizeof(float), prompt = (size_t)sms * PROMPT_SLOT * sizeof(float);
    const size_t slots = split > prompt ? split : prompt, table = 65536 * sizeof(int);
    // converted prompt tiles: no more than all pages' tokens (and a tile's rest per page)
    const size_t most = attend_prompt_bytes(c->pages, (long long)n_pages * page_size + 128);
    const size_t operands = (size_t)prompt_bytes < most ? (size_t)prompt_bytes : most;
    if (e == cudaSuccess) e = cudaMalloc((void**)&c->ws, head + slots + table + operands);
    if (e == cudaSuccess) e = cudaMemset(c->ws, 0, head);
    if (e == cudaSuccess) e = attend_split_init();
    if (e == cudaSuccess) e = attend_prompt_init();
    if (e == cudaSuccess && !(encode_codes(&c->attend.k16, k_codes, c->pages) && encode_codes(&c->attend.v16, v_codes, c->pages)))
        e = cudaErrorInvalidValue;
    // the memset is queued on the legacy stream, which other streams need not wait for
    if (e == cudaSuccess) e = cudaDeviceSynchronize();
    c->attend.counters = (int*)(c->ws + 256);
    c->attend.partial = (float*)(c->ws + head);
    c->attend.sms = sms;
    c->attend.operand_at = (int*)(c->ws + head + slots);
    c->attend.operands = (uint8_t*)(c->ws + head + slots + table);
    c->attend.operand_bytes = operands;
    if (e != cudaSuccess) {
        cudaGetLastError();   // (as in cuda_fail)
        if (c->ws) cudaFree(c->ws);
        delete c;
        return e == cudaErrorMemoryAllocation ? fail(MLORA_ERR_OOM, "workspace: %s", cudaGetErrorString(e))
                                              : cuda_fail(e, "mlora_cache_create");
    }
    *out = c;
    return MLORA_OK;
}

mlora_status mlora_cache_destroy(mlora_cache_t c) {
    if (!c) return MLORA_OK;
    DeviceGuard g(c->device);
    cudaError_t e = g.err;
    if (e == cudaSuccess) e = cudaDeviceSynchronize();
    if (c->ws) cudaFree(c->ws);
    delete c;
    return e == cudaSuccess ? MLORA_OK : cuda_fail(e, "mlora_cache_destroy");
}

mlora_status mlora_cache_append(mlora_cache_t c, const void* K, int64_t k_row, int64_t k_head, const void* V,
                                int64_t v_row, int64_t v_head, mlora_dtype dtype, int T, const int32_t* offsets,
                                const int32_t* lengths, const int32_t* pages, int n_seqs, int width, int max_new,
                                mlora_stream_t stream) {
    CacheStep s;
    bool run;
    mlora_status st = check_step(c, dtype, T, offsets, lengths, pages, n_seqs, width, max_new, &s, &run);
    if (st != MLORA_OK || !run) return st;
    if ((st = check_rows("K", K, k_row, k_head, dtype)) != MLORA_OK) return st;
    if ((st = check_rows("V", V, v_row, v_head, dtype)) != MLORA_OK) return st;
    DeviceGuard g(c->device);
    if (g.err != cudaSuccess) return cuda_fail(g.err, "cudaSetDevice");
    CU_TRY(launch_append(dtype == MLORA_BF16, c->pages, s, RowsIn{K, k_row, k_head}, RowsIn{V, v_row, v_head},
                         (uint32_t*)c->ws, (cudaStream_t)stream));
    return MLORA_OK;
}

mlora_status mlora_cache_read(mlora_cache_t c, void* K, int64_t k_row, int64_t k_head, void* V, int64_t v_row,
                              int64_t v_head, mlora_dtype dtype, int T, const int32_t* offsets, const int32_t* lengths,
                              const int32_t* pages, int n_seqs, int width, int max_new, mlora_stream_t stream) {
    CacheStep s;
    bool run;
    mlora_status st = check_step(c, dtype, T, offsets, lengths, pages, n_seqs, width, max_new, &s, &run);
    if (st != MLORA_OK || !run) return st;
    if ((st = check_rows("K", K, k_row, k_head, dtype)) != MLORA_OK) return st;
    if ((st = check_rows("V", V, v_row, v_head, dtype)) != MLORA_OK) return st;
    DeviceGuard g(c->device);
    if (g.err != cudaSuccess) return cuda_fail(g.err, "cudaSetDevice");
    CU_TRY(launch_read(dtype == MLORA_BF16, c->pages, s, RowsOut{K, k_row, k_head}, RowsOut{V, v_row, v_head},
                       (uint32_t*)c->ws, (cudaStream_t)stream));
    return MLORA_OK;
}

mlora_status mlora_cache_attend(mlora_cache_t c, const void* Q, int64_t q_row, int64_t q_head, void* O, int64_t o_row,
                                int64_t o_head, mlora_dtype dtype, int T, const int32_t* offsets,
                                const int32_t* lengths, const int32_t* pages, int n_seqs, int width, int max_new,
                                float scale, int window, mlora_stream_t stream) {
    CacheStep s;
    bool run;
    mlora_status st = check_step(c, dtype, T, offsets, lengths, pages, n_seqs, width, max_new, &s, &run);
    if (st != MLORA_OK) return st;
    if (!(scale > 0.f && scale < 3.0e38f)) return fail(MLORA_ERR_INVALID_ARG, "scale %g", scale);
    if (window < 0) return fail(MLORA_ERR_INVALID_ARG, "window %d is negative", window);
    if (!run) return MLORA_OK;
    if ((long long)s.max_new * (c->q_heads / c->pages.heads) > 1 << 30)
        return fail(MLORA_ERR_UNSUPPORTED, "%d rows of %d heads per key head", s.max_new, c->q_heads / c->pages.heads);
    if ((long long)s.max_new * c->q_heads > 1ll << 34)   // (row tiles x heads are counted in 32 bits)
        return fail(MLORA_ERR_UNSUPPORTED, "%d rows of %d heads", s.max_new, c->q_heads);
    if ((st = check_rows("Q", Q, q_row, q_head, dtype)) != MLORA_OK) return st;
    if ((st = check_rows("O", O, o_row, o_head, dtype)) != MLORA_OK) return st;
    DeviceGuard g(c->device);
    if (g.err != cudaSuccess) return cuda_fail(g.err, "cudaSetDevice");
    AttendArgs a{c->pages, s, RowsIn{Q, q_row, q_head}, RowsOut{O, o_row, o_head}, c->q_heads, c->page_div,
                 c->group_div, scale, window, (uint32_t*)c->ws};
    const bool bf16 = dtype == MLORA_BF16;
    CU_TRY(attend_prompt_takes(bf16, a) ? launch_attend_prompt(bf16, a, c->attend, (cudaStream_t)stream)
                                        : launch_attend_split(bf16, a, c->attend, (cudaStream_t)stream));
    return MLORA_OK;
}

mlora_status mlora_cache_status(mlora_cache_t c, mlora_stream_t stream) {
    if (!c) return fail(MLORA_ERR_INVALID_ARG, "cache is NULL");
    DeviceGuard g(c->device);
    if (g.err != cudaSuccess) return cuda_fail(g.err, "cudaSetDevice");
    cudaStream_t st = (cudaStream_t)stream;
    uint32_t word = 0;
    CU_TRY(cudaMemcpyAsync(&word, c->ws, sizeof word, cudaMemcpyDeviceToHost, st));
    CU_TRY(cudaMemsetAsync(c->ws, 0, sizeof word, st));
    CU_TRY(cudaStreamSynchronize(st));
    if (word & STATUS_TIMEOUT) return fail(MLORA_ERR_DEVICE_TIMEOUT, "a kernel pipeline wait gave up");
    if (word & STATUS_BAD_STEP) return fail(MLORA_ERR_DEVICE_STEP, "a step named rows, lengths or pages out of range");
    return MLORA_OK;
}

mlora_status mlora_debug_cache_expire_wait(mlora_cache_t c, long long cycles, mlora_stream_t stream) {
    if (!c) return fail(MLORA_ERR_INVALID_ARG, "cache is NULL");
    if (cycles < 1 || cycles > (1ll << 31)) return fail(MLORA_ERR_INVALID_ARG, "cycles not in [1, 2^31]");
    DeviceGuard g(c->device);
    if (g.err != cudaSuccess) return cuda_fail(g.err, "cudaSetDevice");
    CU_TRY(launch_expired_wait((uint32_t*)c->ws, cycles, (cudaStream_t)stream));
    return MLORA_OK;
}

}  // extern "C"
