// The cache's append and read (include/mlora.h): rows to int8 codes with one scale per
// page and head, and back.
//
// A step touches the blocks of each sequence that hold positions start .. len - 1.  A group
// of threads takes one tile: one (sequence, block, head, keys or values), whose codes are
// contiguous and whose rows are strided, in vectors of 16 elements.
//
// Bound: HBM, 3 bytes per bf16 element each way: 106k tokens of 8 heads of 128 are read in 103 us,
// 6.3 TB/s (fp32 231 us, 4.7 TB/s); 30k tokens written and read back take 63 us, 5.8 TB/s (fp32 123 us,
// 4.9 TB/s); the rows of 256 sequences, 32 heads, written and the pages that they lie in read back
// take 46 us, 4.5 TB/s (fp32 80 us).  A tile's loads
// depend on the sequence's length, then on its page: small groups, each with all its loads in
// flight at once, cover that chain.  A step of few rows (decode) gives a tile to a warp: it is one
// row, and its time is the chain's.
#include <cuda_bf16.h>

#include "cache.h"

namespace mlora {

namespace {

constexpr int THREADS = 128;
// CTAs per SM (register limits): of 1 to 16 each, those that measured best at 100k tokens read and
// at 28k tokens appended
constexpr int READ_CTAS = 10;
template <typename T, int HELD>
constexpr int APPEND_CTAS = HELD == 1 ? (sizeof(T) == 2 ? 12 : 8) : sizeof(T) == 2 ? 9 : 4;
constexpr int HELD = 4;                    // vectors per thread kept in registers at most

// 16 elements of a row as they lie in memory
template <typename T>
struct Vec {
    static constexpr int W = sizeof(T) * 4;   // words
    uint32_t w[W];
    __device__ __forceinline__ void load(const T* p) {
#pragma unroll
        for (int i = 0; i < W; i += 4) *reinterpret_cast<uint4*>(w + i) = __ldg(reinterpret_cast<const uint4*>(p) + i / 4);
    }
    __device__ __forceinline__ void clear() {
#pragma unroll
        for (int i = 0; i < W; ++i) w[i] = 0u;
    }
    __device__ __forceinline__ float at(int e) const {
        if (sizeof(T) == 4) return __uint_as_float(w[e]);
        return __uint_as_float(e & 1 ? w[e / 2] & 0xFFFF0000u : w[e / 2] << 16);
    }
};

__device__ __forceinline__ float max_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}
// The largest |x| of a vector; NaN if one is NaN.
__device__ __forceinline__ float largest(const Vec<float>& v) {
    float m = 0.f;
#pragma unroll
    for (int e = 0; e < 16; ++e) m = max_nan(m, fabsf(__uint_as_float(v.w[e])));
    return m;
}
__device__ __forceinline__ float largest(const Vec<__nv_bfloat16>& v) {
    __nv_bfloat162 m = __float2bfloat162_rn(0.f);
#pragma unroll
    for (int i = 0; i < 8; ++i) m = __hmax2_nan(m, __habs2(*reinterpret_cast<const __nv_bfloat162*>(&v.w[i])));
    return max_nan(__low2float(m), __high2float(m));
}
// The largest finite |x|.
template <typename T>
__device__ __forceinline__ float largest_finite(const Vec<T>& v) {
    float m = 0.f;
#pragma unroll
    for (int e = 0; e < 16; ++e) {
        const float a = fabsf(v.at(e));
        m = fmaxf(m, a <= 3.402823466e38f ? a : 0.f);
    }
    return m;
}

// rint(x * inv) in the low byte: adding 1.5 * 2^23 leaves the integer (ties to even) in the
// sum's low mantissa bits.  Without CLAMP, |x * inv| rounds to at most 127.
template <bool CLAMP>
__device__ __forceinline__ uint32_t code_of(float x, float inv) {
    float t = __fmul_rn(x, inv);
    if (CLAMP) t = t != t ? 0.f : fminf(fmaxf(t, -127.f), 127.f);
    return __float_as_uint(__fadd_rn(t, 12582912.f));
}
__device__ __forceinline__ uint32_t low_bytes(uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    return __byte_perm(__byte_perm(a, b, 0x0040), __byte_perm(c, d, 0x0040), 0x5410);
}
template <bool CLAMP, typename F>
__device__ __forceinline__ uint4 codes16(F&& at, float inv) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
        w[i] = low_bytes(code_of<CLAMP>(at(4 * i), inv), code_of<CLAMP>(at(4 * i + 1), inv),
                         code_of<CLAMP>(at(4 * i + 2), inv), code_of<CLAMP>(at(4 * i + 3), inv));
    return make_uint4(w[0], w[1], w[2], w[3]);
}
// code e of 16 as a float: code + 128 under the exponent of 2^23, exactly
__device__ __forceinline__ float value_of(const uint32_t (&w)[4], int e) {
    return __uint_as_float(__byte_perm(w[e / 4] ^ 0x80808080u, 0x4B000000u, 0x7650 | (e & 3))) - 8388736.f;
}

__device__ __forceinline__ int floor_div(int a, int b) { return a / b - (a % b < 0 ? 1 : 0); }

// The largest value over a group of threads (a warp or the CTA); NaN if one is NaN.
template <int GROUP>
__device__ __forceinline__ float group_max(float m) {
#pragma unroll
    for (int d = 16; d; d >>= 1) m = max_nan(m, __shfl_xor_sync(~0u, m, d));
    if (GROUP > 32) {
        __shared__ float top[THREADS / 32];
        __syncthreads();
        if ((threadIdx.x & 31) == 0) top[threadIdx.x >> 5] = m;
        __syncthreads();
#pragma unroll
        for (int w = 0; w < THREADS / 32; ++w) m = max_nan(m, top[w]);
    }
    return m;
}

template <typename T, int GROUP, int HELD>
__global__ void __launch_bounds__(THREADS, (APPEND_CTAS<T, HELD>)) append_kernel(CachePages c, CacheStep s, RowsIn K, RowsIn V, Divide per_row,
                                                         uint32_t* status) {
    const int part = blockIdx.y * (THREADS / GROUP) + threadIdx.x / GROUP, t = threadIdx.x % GROUP;
    const int b = blockIdx.z, h = part >> 1;
    const bool is_v = part & 1;
    if (h >= c.heads) return;
    const SeqRec q = load_seq(s, c.page, b, status);
    const int start = q.start < 0 ? 0 : q.start, skip = start - q.start;   // rows at negative positions
    const int j = start / c.page + (int)blockIdx.x, end = q.start + q.rows;
    if ((long long)j * c.page >= end) return;   // (the launch covers max_new rows, of up to 2^31)
    const int lo = max(start - j * c.page, 0);                              // tokens of the block held before
    const int hi = min(end - j * c.page, c.page);                           // and after
    if (hi <= lo || q.rows <= skip) return;
    const int id = load_page(s, c, b, j, status);
    if (id < 0) return;
    const RowsIn& R = is_v ? V : K;
    const T* src = (const T*)R.ptr + (q.row0 + (j * c.page + lo - q.start)) * R.row + h * R.head;
    const size_t at = (size_t)id * c.heads + h;
    float* scale = (is_v ? c.v_scale : c.k_scale) + at;
    int8_t* dst = (is_v ? c.v_codes : c.k_codes) + at * c.page * c.dim;
    const float held = lo > 0 ? *scale : 0.f;
    const int n = (hi - lo) * per_row.d;
    auto load = [&](int i) {
        Vec<T> v;
        const int r = quotient(per_row, i);
        v.load(src + (int64_t)r * R.row + (i - r * per_row.d) * 16);
        return v;
    };
    Vec<T> x[HELD];
#pragma unroll
    for (int k = 0; k < HELD; ++k) {
        if (t + k * GROUP < n) x[k] = load(t + k * GROUP);
        else x[k].clear();
    }
    float m = 0.f;
#pragma unroll
    for (int k = 0; k < HELD; ++k) m = max_nan(m, largest(x[k]));
    for (int i = t + HELD * GROUP; i < n; i += GROUP) m = max_nan(m, largest(load(i)));
    m = group_max<GROUP>(m);
    const bool finite = m <= 3.402823466e38f;
    if (!finite) {   // infinities and NaN do not enter the maximum
        m = 0.f;
#pragma unroll
        for (int k = 0; k < HELD; ++k) m = fmaxf(m, largest_finite(x[k]));
        for (int i = t + HELD * GROUP; i < n; i += GROUP) m = fmaxf(m, largest_finite(load(i)));
        m = group_max<GROUP>(m);
    }
    const float now = fmaxf(held, __fdiv_rn(m, 127.f));
    const float inv = now >= TINY_SCALE ? __fdiv_rn(1.f, now) : 0.f;
    if (t == 0) *scale = now;
    if (now != held && lo > 0) {   // the scale grew: what the block held is restored and quantised again
        const int was = lo * per_row.d;
#pragma unroll 4
        for (int i = t; i < was; i += GROUP) {
            uint4* p = reinterpret_cast<uint4*>(dst + (size_t)i * 16);
            const uint4 u = *p;
            const uint32_t w[4] = {u.x, u.y, u.z, u.w};
            *p = codes16<true>([&](int e) { return __fmul_rn(value_of(w, e), held); }, inv);
        }
    }
    int8_t* out = dst + (size_t)lo * c.dim;
    auto store = [&](int i, const Vec<T>& v) {
        auto value = [&](int e) { return v.at(e); };
        *reinterpret_cast<uint4*>(out + (size_t)i * 16) = finite ? codes16<false>(value, inv) : codes16<true>(value, inv);
    };
#pragma unroll
    for (int k = 0; k < HELD; ++k)
        if (t + k * GROUP < n) store(t + k * GROUP, x[k]);
    for (int i = t + HELD * GROUP; i < n; i += GROUP) store(i, load(i));
}

template <typename T>
__device__ __forceinline__ void store16(T* p, const uint32_t (&w)[4], float sc);
template <>
__device__ __forceinline__ void store16<__nv_bfloat16>(__nv_bfloat16* p, const uint32_t (&w)[4], float sc) {
    uint32_t y[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(__fmul_rn(value_of(w, 2 * i), sc), __fmul_rn(value_of(w, 2 * i + 1), sc));
        y[i] = *reinterpret_cast<const uint32_t*>(&h);
    }
    reinterpret_cast<uint4*>(p)[0] = make_uint4(y[0], y[1], y[2], y[3]);
    reinterpret_cast<uint4*>(p)[1] = make_uint4(y[4], y[5], y[6], y[7]);
}
template <>
__device__ __forceinline__ void store16<float>(float* p, const uint32_t (&w)[4], float sc) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
        reinterpret_cast<float4*>(p)[i] = make_float4(__fmul_rn(value_of(w, 4 * i), sc), __fmul_rn(value_of(w, 4 * i + 1), sc),
                                                      __fmul_rn(value_of(w, 4 * i + 2), sc), __fmul_rn(value_of(w, 4 * i + 3), sc));
}

// Restores the x-th block that sequence b's rows may touch.
template <typename T, int GROUP>
__device__ __forceinline__ void read_block(const CachePages& c, const CacheStep& s, const SeqRec& q, const RowsOut& R,
                                           bool is_v, int b, int h, int x, const Divide& per_row, uint32_t* status) {
    const int t = threadIdx.x % GROUP;
    const int j = floor_div(q.start, c.page) + x;   // negative: rows that name no token
    const long long first = (long long)j * c.page;  // its first position, perhaps outside 32 bits
    const int lo = (int)max(q.start - first, 0ll), hi = (int)min(q.start + q.rows - first, (long long)c.page);
    if (hi <= lo) return;
    const int id = j >= 0 ? load_page(s, c, b, j, status) : -1;
    T* dst = (T*)R.ptr + (q.row0 + (first + lo - q.start)) * R.row + h * R.head;
    const size_t at = (size_t)(id < 0 ? 0 : id) * c.heads + h;
    const int8_t* src = (is_v ? c.v_codes : c.k_codes) + (at * c.page + lo) * c.dim;
    const int n = (hi - lo) * per_row.d;
    const float sc = id < 0 ? 0.f : (is_v ? c.v_scale : c.k_scale)[at];
    for (int i0 = 0; i0 < n; i0 += HELD * GROUP) {
        uint4 u[HELD];
#pragma unroll
        for (int k = 0; k < HELD; ++k) {
            const int i = i0 + k * GROUP + t;
            u[k] = id >= 0 && i < n ? __ldcs(reinterpret_cast<const uint4*>(src + (size_t)i * 16)) : make_uint4(0u, 0u, 0u, 0u);
        }
#pragma unroll
        for (int k = 0; k < HELD; ++k) {
            const int i = i0 + k * GROUP + t;
            if (i >= n) break;
            const uint32_t w[4] = {u[k].x, u[k].y, u[k].z, u[k].w};
            const int r = quotient(per_row, i);
            store16<T>(dst + (int64_t)r * R.row + (i - r * per_row.d) * 16, w, sc);
        }
    }
}

// TWO: rows that touch two blocks at most, mostly one of them; one CTA looks at both (a CTA
// that finds nothing costs a third of one that does).
template <typename T, int GROUP, bool TWO>
__global__ void __launch_bounds__(THREADS, READ_CTAS) read_kernel(CachePages c, CacheStep s, RowsOut K, RowsOut V,
                                                                  Divide per_row, uint32_t* status) {
    const int part = blockIdx.y * (THREADS / GROUP) + threadIdx.x / GROUP, b = blockIdx.z, h = part >> 1;
    if (h >= c.heads) return;
    const SeqRec q = load_seq(s, c.page, b, status);
#pragma unroll 1
    for (int x = blockIdx.x; x < (TWO ? 2 : (int)blockIdx.x + 1); ++x)
        read_block<T, GROUP>(c, s, q, part & 1 ? V : K, part & 1, b, h, x, per_row, status);
}

// Blocks that max_new consecutive positions can touch.
int most_blocks(int max_new, int page) { return (int)(((long long)max_new + page - 2) / page) + 1; }

template <int GROUP, typename Rows, typename Kernel>
cudaError_t launch(Kernel kernel, int blocks, const CachePages& c, const CacheStep& s, const Rows& k, const Rows& v,
                   uint32_t* status, cudaStream_t st) {
    constexpr int PARTS = THREADS / GROUP;
    const dim3 grid(blocks, (2 * c.heads + PARTS - 1) / PARTS, s.n_seqs);
    kernel<<<grid, THREADS, 0, st>>>(c, s, k, v, divide_by(c.dim / 16), status);
    return cudaGetLastError();
}

// A warp per tile where a sequence's rows are at most what a warp holds, else the CTA.
bool few_rows(const CachePages& c, const CacheStep& s) { return (long long)s.max_new * (c.dim / 16) <= 32 * HELD; }

}  // namespace

cudaError_t launch_append(bool bf16, const CachePages& c, const CacheStep& s, const RowsIn& k, const RowsIn& v,
                          uint32_t* status, cudaStream_t st) {
    const int blocks = most_blocks(s.max_new, c.page);
    // decode: a row's vectors are one per lane at most, and more warps fit an SM with them alone (256
    // rows of 32 heads, and their pages read back: 47 us, 50 us with room for HELD; fp32 81, 87 us)
    if ((long long)s.max_new * (c.dim / 16) <= 32)
        return bf16 ? launch<32>(append_kernel<__nv_bfloat16, 32, 1>, blocks, c, s, k, v, status, st)
                    : launch<32>(append_kernel<float, 32, 1>, blocks, c, s, k, v, status, st);
    if (few_rows(c, s))
        return bf16 ? launch<32>(append_kernel<__nv_bfloat16, 32, HELD>, blocks, c, s, k, v, status, st)
                    : launch<32>(append_kernel<float, 32, HELD>, blocks, c, s, k, v, status, st);
    return bf16 ? launch<THREADS>(append_kernel<__nv_bfloat16, THREADS, HELD>, blocks, c, s, k, v, status, st)
                : launch<THREADS>(append_kernel<float, THREADS, HELD>, blocks, c, s, k, v, status, st);
}

template <typename T>
static cudaError_t read_by_shape(const CachePages& c, const CacheStep& s, const RowsOut& k, const RowsOut& v,
                                 uint32_t* status, cudaStream_t st) {
    const int blocks = most_blocks(s.max_new, c.page);
    if (few_rows(c, s)) return launch<32>(read_kernel<T, 32, false>, blocks, c, s, k, v, status, st);
    if (blocks == 2) return launch<THREADS>(read_kernel<T, THREADS, true>, 1, c, s, k, v, status, st);
    return launch<THREADS>(read_kernel<T, THREADS, false>, blocks, c, s, k, v, status, st);
}

cudaError_t launch_read(bool bf16, const CachePages& c, const CacheStep& s, const RowsOut& k, const RowsOut& v,
                        uint32_t* status, cudaStream_t st) {
    return bf16 ? read_by_shape<__nv_bfloat16>(c, s, k, v, status, st) : read_by_shape<float>(c, s, k, v, status, st);
}

}  // namespace mlora
