// Causal attention over the 8-bit cache (include/mlora.h), one CTA per (row, query head):
// each warp takes every fourth token, its lanes share the head's elements; the softmax
// keeps a running maximum and sum per warp, and the warps join at the end.
#include <cuda_bf16.h>

#include "cache.h"

namespace mlora {

namespace {

constexpr int ROW_WARPS = 4;

template <typename T>
__global__ void __launch_bounds__(32 * ROW_WARPS) attend_row_kernel(AttendArgs a) {
    const CachePages& c = a.pages;
    const int i = blockIdx.x, b = blockIdx.z, hq = blockIdx.y;
    const int h = hq / (a.q_heads / c.heads);
    const SeqRec s = load_seq(a.step, c.page, b, a.status);
    if (i >= s.rows) return;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const T* q = (const T*)a.q.ptr + (int64_t)(s.row0 + i) * a.q.row + hq * a.q.head;
    T* o = (T*)a.o.ptr + (int64_t)(s.row0 + i) * a.o.row + hq * a.o.head;
    float qr[8], acc[8];
    bool fine = true;   // a query that holds a NaN or an infinity gives NaN
    for (int e = 0; e < 8; ++e) {
        const int d = lane + 32 * e;
        qr[e] = d < c.dim ? (float)q[d] * a.scale : 0.f;
        acc[e] = 0.f;
        fine &= fabsf(qr[e]) <= 3.402823466e38f;
    }
    fine = __all_sync(~0u, fine);
    const int pos = s.start + i;
    const int lo = a.window > 0 ? max(0, pos - a.window + 1) : 0;
    float m = -INFINITY, l = 0.f;
    for (int t = lo + warp; t <= pos; t += ROW_WARPS) {
        const int id = load_page(a.step, c, b, t / c.page, a.status);
        const size_t at = (size_t)(id < 0 ? 0 : id) * c.heads + h;
        const size_t base = (at * c.page + t % c.page) * c.dim;
        const float ks = id < 0 ? 0.f : c.k_scale[at], vs = id < 0 ? 0.f : c.v_scale[at];
        float x = 0.f;
        for (int e = 0; e < 8; ++e) {
            const int d = lane + 32 * e;
            if (d < c.dim) x += qr[e] * (float)c.k_codes[base + d];
        }
        for (int d = 16; d; d >>= 1) x += __shfl_xor_sync(~0u, x, d);
        x *= ks;
        const float mn = fmaxf(m, x), f = expf(m - mn), p = expf(x - mn);
        m = mn;
        l = l * f + p;
        for (int e = 0; e < 8; ++e) {
            const int d = lane + 32 * e;
            if (d < c.dim) acc[e] = acc[e] * f + p * vs * (float)c.v_codes[base + d];
        }
    }
    __shared__ float sm[ROW_WARPS], sl[ROW_WARPS], so[ROW_WARPS][256];
    sm[warp] = m;
    sl[warp] = l;
    for (int e = 0; e < 8; ++e) so[warp][lane + 32 * e] = acc[e];
    __syncthreads();
    float top = -INFINITY, sum = 0.f;
    for (int w = 0; w < ROW_WARPS; ++w) top = fmaxf(top, sm[w]);
    for (int w = 0; w < ROW_WARPS; ++w) sum += sm[w] == -INFINITY ? 0.f : sl[w] * expf(sm[w] - top);
    if (!fine) sum = pos >= 0 ? NAN : 0.f;
    for (int d = threadIdx.x; d < c.dim; d += 32 * ROW_WARPS) {
        float v = 0.f;
        for (int w = 0; w < ROW_WARPS; ++w) v += sm[w] == -INFINITY ? 0.f : so[w][d] * expf(sm[w] - top);
        o[d] = (T)(sum == 0.f ? 0.f : fine ? v / sum : NAN);
    }
}

}  // namespace

cudaError_t launch_attend(bool bf16, const AttendArgs& a, cudaStream_t st) {
    const dim3 grid(a.step.max_new, a.q_heads, a.step.n_seqs);
    if (bf16) attend_row_kernel<__nv_bfloat16><<<grid, 32 * ROW_WARPS, 0, st>>>(a);
    else attend_row_kernel<float><<<grid, 32 * ROW_WARPS, 0, st>>>(a);
    return cudaGetLastError();
}

}  // namespace mlora
