// The cache's append and read (include/mlora.h): rows to int8 codes with one scale per
// page and head, and back.
//
// A step touches the blocks of each sequence that hold positions start .. len - 1.  One CTA takes one (sequence, block, head,
// keys or values): the block's codes are contiguous, its rows are strided.
#include <cuda_bf16.h>

#include "cache.h"

namespace mlora {

namespace {

constexpr float TINY_SCALE = 0x1p-120f;   // below it the codes are 0 (1 / s stays finite above)

// 8 elements of a row, 16-byte aligned
template <typename T>
__device__ __forceinline__ void load8(const T* p, float* x);
template <>
__device__ __forceinline__ void load8<__nv_bfloat16>(const __nv_bfloat16* p, float* x) {
    const uint4 u = *reinterpret_cast<const uint4*>(p);
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[2 * i] = __uint_as_float(w[i] << 16);
        x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
}
template <>
__device__ __forceinline__ void load8<float>(const float* p, float* x) {
    const float4 a = *reinterpret_cast<const float4*>(p), b = *reinterpret_cast<const float4*>(p + 4);
    x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w, x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
}
template <typename T>
__device__ __forceinline__ void store8(T* p, const float* x);
template <>
__device__ __forceinline__ void store8<__nv_bfloat16>(__nv_bfloat16* p, const float* x) {
    uint4 u;
    __nv_bfloat162* h = reinterpret_cast<__nv_bfloat162*>(&u);
#pragma unroll
    for (int i = 0; i < 4; ++i) h[i] = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
    *reinterpret_cast<uint4*>(p) = u;
}
template <>
__device__ __forceinline__ void store8<float>(float* p, const float* x) {
    *reinterpret_cast<float4*>(p) = make_float4(x[0], x[1], x[2], x[3]);
    *reinterpret_cast<float4*>(p + 4) = make_float4(x[4], x[5], x[6], x[7]);
}

// rint(clamp(x * inv)) as a byte: adding 1.5 * 2^23 leaves the integer (ties to even) in
// the sum's low mantissa bits.  fminf/fmaxf drop a NaN, so it is sent to 0 first.
__device__ __forceinline__ uint32_t code_of(float x, float inv) {
    float t = __fmul_rn(x, inv);
    t = t != t ? 0.f : fminf(fmaxf(t, -127.f), 127.f);
    return __float_as_uint(__fadd_rn(t, 12582912.f)) & 0xFFu;
}
__device__ __forceinline__ uint32_t pack4(const float* x, float inv) {
    return code_of(x[0], inv) | code_of(x[1], inv) << 8 | code_of(x[2], inv) << 16 | code_of(x[3], inv) << 24;
}
// code i of a word as a float
__device__ __forceinline__ float value_of(uint32_t word, int i) { return (float)(int8_t)(word >> (8 * i)); }

__device__ __forceinline__ int floor_div(int a, int b) { return a >= 0 ? a / b : -((b - 1 - a) / b); }

constexpr int APPEND_THREADS = 256;

template <typename T>
__global__ void __launch_bounds__(APPEND_THREADS) append_kernel(CachePages c, CacheStep s, RowsIn K, RowsIn V,
                                                                uint32_t* status) {
    const int b = blockIdx.z, h = blockIdx.y >> 1;
    const bool is_v = blockIdx.y & 1;
    const SeqRec q = load_seq(s, c.page, b, status);
    const int start = q.start < 0 ? 0 : q.start, skip = start - q.start;   // rows at negative positions
    const int j = start / c.page + (int)blockIdx.x;
    const int lo = max(start - j * c.page, 0);                              // tokens of the block held before
    const int hi = min(q.start + q.rows - j * c.page, c.page);              // and after
    if (hi <= lo || q.rows <= skip) return;
    const int id = load_page(s, c, b, j, status);
    if (id < 0) return;
    const RowsIn& R = is_v ? V : K;
    const T* src = (const T*)R.ptr + (q.row0 + (j * c.page + lo - q.start)) * R.row + h * R.head;
    const size_t at = (size_t)id * c.heads + h;
    float* scale = (is_v ? c.v_scale : c.k_scale) + at;
    int8_t* dst = (is_v ? c.v_codes : c.k_codes) + at * c.page * c.dim;
    const float held = lo > 0 ? *scale : 0.f;
    const int vr = c.dim / 8, n = (hi - lo) * vr;   // vectors of 8 per row, and in all
    float m = 0.f;
    for (int i = threadIdx.x; i < n; i += APPEND_THREADS) {
        float x[8];
        load8(src + (size_t)(i / vr) * R.row + i % vr * 8, x);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const float a = fabsf(x[e]);
            m = fmaxf(m, a <= 3.402823466e38f ? a : 0.f);
        }
    }
    __shared__ float top[APPEND_THREADS / 32];
#pragma unroll
    for (int d = 16; d; d >>= 1) m = fmaxf(m, __shfl_xor_sync(~0u, m, d));
    if ((threadIdx.x & 31) == 0) top[threadIdx.x >> 5] = m;
    __syncthreads();
    for (int w = 0; w < APPEND_THREADS / 32; ++w) m = fmaxf(m, top[w]);
    const float now = fmaxf(held, __fdiv_rn(m, 127.f));
    const float inv = now >= TINY_SCALE ? __fdiv_rn(1.f, now) : 0.f;
    if (threadIdx.x == 0) *scale = now;
    if (now != held)   // the scale grew: what the block held is restored and quantised again
        for (int i = threadIdx.x; i < lo * vr; i += APPEND_THREADS) {
            uint2* p = reinterpret_cast<uint2*>(dst + (size_t)i * 8);
            const uint2 u = *p;
            float x[8];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                x[e] = __fmul_rn(value_of(u.x, e), held);
                x[4 + e] = __fmul_rn(value_of(u.y, e), held);
            }
            *p = make_uint2(pack4(x, inv), pack4(x + 4, inv));
        }
    for (int i = threadIdx.x; i < n; i += APPEND_THREADS) {
        float x[8];
        load8(src + (size_t)(i / vr) * R.row + i % vr * 8, x);
        *reinterpret_cast<uint2*>(dst + ((size_t)lo * vr + i) * 8) = make_uint2(pack4(x, inv), pack4(x + 4, inv));
    }
}

constexpr int READ_THREADS = 256;

template <typename T>
__global__ void __launch_bounds__(READ_THREADS) read_kernel(CachePages c, CacheStep s, RowsOut K, RowsOut V,
                                                            uint32_t* status) {
    const int b = blockIdx.z, h = blockIdx.y >> 1;
    const bool is_v = blockIdx.y & 1;
    const SeqRec q = load_seq(s, c.page, b, status);
    const int j = floor_div(q.start, c.page) + (int)blockIdx.x;   // negative: rows that name no token
    const int lo = max(q.start - j * c.page, 0), hi = min(q.start + q.rows - j * c.page, c.page);
    if (hi <= lo) return;
    const int id = j >= 0 ? load_page(s, c, b, j, status) : -1;
    const RowsOut& R = is_v ? V : K;
    T* dst = (T*)R.ptr + (q.row0 + (j * c.page + lo - q.start)) * R.row + h * R.head;
    const size_t at = (size_t)(id < 0 ? 0 : id) * c.heads + h;
    const float sc = id < 0 ? 0.f : (is_v ? c.v_scale : c.k_scale)[at];
    const int8_t* src = (is_v ? c.v_codes : c.k_codes) + (at * c.page + lo) * c.dim;
    const int vr = c.dim / 8, n = (hi - lo) * vr;
    for (int i = threadIdx.x; i < n; i += READ_THREADS) {
        const uint2 u = id < 0 ? make_uint2(0u, 0u) : *reinterpret_cast<const uint2*>(src + (size_t)i * 8);
        float x[8];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            x[e] = __fmul_rn(value_of(u.x, e), sc);
            x[4 + e] = __fmul_rn(value_of(u.y, e), sc);
        }
        store8((T*)dst + (size_t)(i / vr) * R.row + i % vr * 8, x);
    }
}

// Blocks that max_new consecutive positions can touch.
int most_blocks(int max_new, int page) { return (max_new + page - 2) / page + 1; }

}  // namespace

cudaError_t launch_append(bool bf16, const CachePages& c, const CacheStep& s, const RowsIn& k, const RowsIn& v,
                          uint32_t* status, cudaStream_t st) {
    const dim3 grid(most_blocks(s.max_new, c.page), 2 * c.heads, s.n_seqs);
    if (bf16) append_kernel<__nv_bfloat16><<<grid, APPEND_THREADS, 0, st>>>(c, s, k, v, status);
    else append_kernel<float><<<grid, APPEND_THREADS, 0, st>>>(c, s, k, v, status);
    return cudaGetLastError();
}

cudaError_t launch_read(bool bf16, const CachePages& c, const CacheStep& s, const RowsOut& k, const RowsOut& v,
                        uint32_t* status, cudaStream_t st) {
    const dim3 grid(most_blocks(s.max_new, c.page), 2 * c.heads, s.n_seqs);
    if (bf16) read_kernel<__nv_bfloat16><<<grid, READ_THREADS, 0, st>>>(c, s, k, v, status);
    else read_kernel<float><<<grid, READ_THREADS, 0, st>>>(c, s, k, v, status);
    return cudaGetLastError();
}

}  // namespace mlora
