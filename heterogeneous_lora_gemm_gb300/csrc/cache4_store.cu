// The 4-bit cache's append and read (include/mlora.h): rows to 4-bit codes with a scale per 16
// elements of a token, and back.
//
// Every atom (16 elements of a token) is a value of its own: nothing that the block held is read.
// Steps of many rows take a block of 16 tokens of a head per warp, a lane two atoms that lie
// together in the block: 16 bytes to a lane and 512 to a warp of codes, whose 32 bytes of row
// elements are gathered or scattered in L1.  Steps of few rows take an atom per thread, along the row.
//
// Bound: HBM, 2 + 9/16 bytes per bf16 element: 28k prompt tokens of 8 heads of 128 are appended in 30 us,
// 5.2 TB/s, and 29.6k read back in 30 us, 5.1 TB/s (floors 23 us each); the rows of 256 sequences, 32
// heads, take 3.2 us and the pages that they lie in 34 us to read (floor 26); 29k fp32 rows are appended in 46 us and read in 67 (together 0.70 of the floor).  Both wait for the chain of
// length, page and rows more than for memory; the read's 32-byte pieces of rows keep L1 busy at three
// quarters of its rate.  What measured slower: a lane per 16 bytes of a row, side by side (prompts read in
// 36 us); lanes that trade halves so that a store fills 32 bytes (30 us, and 39 for the decode pages);
// keys and values of a block in two warps (appended in 37 us).
#include <cuda_bf16.h>

#include "block4.cuh"
#include "cache.h"

namespace mlora {

namespace {

constexpr int THREADS = 64;
constexpr int FEW = 8;   // rows of a sequence up to which a thread takes an atom

// 16 elements of a row as they lie in memory
template <typename T>
struct Row16 {
    static constexpr int W = sizeof(T) * 4;   // words
    uint32_t w[W];
    __device__ __forceinline__ void load(const T* p) {
#pragma unroll
        for (int i = 0; i < W; i += 4) {
            const uint4 v = __ldg(reinterpret_cast<const uint4*>(p) + i / 4);
            w[i] = v.x, w[i + 1] = v.y, w[i + 2] = v.z, w[i + 3] = v.w;
        }
    }
    __device__ __forceinline__ void store(T* p) const {
#pragma unroll
        for (int i = 0; i < W; i += 4) reinterpret_cast<uint4*>(p)[i / 4] = make_uint4(w[i], w[i + 1], w[i + 2], w[i + 3]);
    }
    __device__ __forceinline__ float at(int e) const {
        if (sizeof(T) == 4) return __uint_as_float(w[e]);
        return __uint_as_float(e & 1 ? w[e / 2] & 0xFFFF0000u : w[e / 2] << 16);
    }
};

struct Atom {
    uint2 codes;
    uint32_t scale;   // e4m3
};

__device__ __forceinline__ float max_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}
// The largest |x|; NaN if one is NaN.
__device__ __forceinline__ float largest(const Row16<float>& x) {
    float m = 0.f;
#pragma unroll
    for (int e = 0; e < 16; ++e) m = max_nan(m, fabsf(x.at(e)));
    return m;
}
__device__ __forceinline__ float largest(const Row16<__nv_bfloat16>& x) {
    __nv_bfloat162 m = __float2bfloat162_rn(0.f);
#pragma unroll
    for (int i = 0; i < 8; ++i) m = __hmax2_nan(m, __habs2(*reinterpret_cast<const __nv_bfloat162*>(&x.w[i])));
    return max_nan(__low2float(m), __high2float(m));
}

// rint(x * inv) + 8 for 16 x, a nibble each.  Adding 1.5 * 2^23 + 8 leaves the integer (ties to even) in
// the sum's low mantissa bits; the sums' bits in a number to the base 16 are the nibbles once the
// constant is taken off.
template <bool CLAMP, typename T>
__device__ __forceinline__ uint2 codes16(const Row16<T>& x, float inv) {
    uint32_t w[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        w[i] = 0u - 0x4B400000u * 0x11111111u;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            float t = __fmul_rn(x.at(8 * i + e), inv);
            if (CLAMP) t = t != t ? 0.f : fminf(fmaxf(t, -7.f), 7.f);
            w[i] += __float_as_uint(__fadd_rn(t, 12582920.f)) * (1u << (4 * e));
        }
    }
    return make_uint2(w[0], w[1]);
}

// `grow` is 1 / (7 unit).
template <typename T>
__device__ __forceinline__ Atom quantise(const Row16<T>& x, float unit, float grow) {
    float top = largest(x);
    const bool finite = top <= 3.402823466e38f;
    if (!finite) {   // infinities and NaN do not enter the maximum
        top = 0.f;
#pragma unroll
        for (int e = 0; e < 16; ++e) {
            const float a = fabsf(x.at(e));
            top = fmaxf(top, a <= 3.402823466e38f ? a : 0.f);
        }
    }
    uint16_t s;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(s) : "f"(0.f), "f"(__fmul_rn(top, grow)));
    const float step = __fmul_rn(scale_f32(s), unit), inv = s ? __fdiv_rn(1.f, step) : 0.f;
    // a scale that is rounded to nearest leaves the largest code below 7.5, unless it is below the
    // least normal one or at the end of its range
    const bool inside = finite && s >= 8 && s < 0x7E;
    return Atom{inside ? codes16<false>(x, inv) : codes16<true>(x, inv), s};
}

__device__ __forceinline__ uint8_t* block_of(const CachePages& c, int id, int h, int at) {
    return c.blocks + (((size_t)id * c.heads + h) * (c.page >> 4) + at) * block4_bytes(c.dim);
}

// A lane's `it`-th pair of atoms of a block: tokens t and t + next, their group (may lie past the
// head), and the first one's place.
struct PairOf {
    int t, next, group, atom;
};
__device__ __forceinline__ PairOf pair_of(bool is_v, int it, int lane, int groups) {
    PairOf p;
    if (is_v) {
        p.t = (it & 1) * 8 + (lane & 3) * 2, p.next = 1, p.group = (it >> 1) * 8 + (lane >> 2);
        p.atom = value_atom(p.t, p.group, groups);
    } else {
        p.t = lane >> 2, p.next = 8, p.group = it * 4 + (lane & 3);
        p.atom = key_atom(p.t, p.group, groups);
    }
    return p;
}
__device__ __forceinline__ int pairs_of(bool is_v, int groups) { return is_v ? (groups + 7) / 8 * 2 : (groups + 3) / 4; }

// A warp per block and head; a lane's rows do not wait for the page that they go to.
template <typename T>
__global__ void __launch_bounds__(THREADS) append_blocks_kernel(CachePages c, CacheStep s, RowsIn K, RowsIn V, uint32_t* status) {
    const int h = blockIdx.y * (THREADS / 32) + threadIdx.x / 32, lane = threadIdx.x & 31, b = blockIdx.z;
    if (h >= c.heads) return;
    const SeqRec q = load_seq(s, c.page, b, status);
    const int start = max(q.start, 0), end = q.start + q.rows;
    const int j = (start >> 4) + (int)blockIdx.x;   // 16-token block of the sequence
    if ((long long)j * 16 >= end) return;           // (the launch covers max_new rows, of up to 2^31)
    const int lo = max(start - j * 16, 0), hi = min(end - j * 16, 16);
    if (hi <= lo) return;
    const int page = j * 16 / c.page;
    const int id = load_page(s, c, b, page, status);
    const int64_t row = q.row0 + (int64_t)j * 16 - q.start;   // of the block's first token
    const T* k_src = (const T*)K.ptr + row * K.row + h * K.head;
    const T* v_src = (const T*)V.ptr + row * V.row + h * V.head;
    const int groups = c.dim >> 4, keys = pairs_of(false, groups), n = keys + pairs_of(true, groups);
    const float k_grow = __fdiv_rn(1.f, __fmul_rn(7.f, c.k_unit)), v_grow = __fdiv_rn(1.f, __fmul_rn(7.f, c.v_unit));
    for (int i = 0; i < n; ++i) {
        const bool is_v = i >= keys;
        const PairOf p = pair_of(is_v, is_v ? i - keys : i, lane, groups);
        if (p.group >= groups) continue;
        const T* src = (is_v ? v_src : k_src) + p.group * 16;
        const int64_t stride = is_v ? V.row : K.row;
        const bool in0 = p.t >= lo && p.t < hi, in1 = p.t + p.next >= lo && p.t + p.next < hi;
        Row16<T> x0, x1;
        if (in0) x0.load(src + p.t * stride);
        if (in1) x1.load(src + (p.t + p.next) * stride);
        if (id < 0) return;
        const float unit = is_v ? c.v_unit : c.k_unit, grow = is_v ? v_grow : k_grow;
        uint8_t* block = block_of(c, id, h, j - page * (c.page >> 4));
        uint8_t* codes = block + (is_v ? 8 * c.dim : 0);
        uint8_t* scales = block + (is_v ? 17 * c.dim : 16 * c.dim);
        Atom a0, a1;
        if (in0) a0 = quantise(x0, unit, grow);
        if (in1) a1 = quantise(x1, unit, grow);
        if (in0 && in1) {
            *reinterpret_cast<uint4*>(codes + p.atom * 8) = make_uint4(a0.codes.x, a0.codes.y, a1.codes.x, a1.codes.y);
            *reinterpret_cast<uint16_t*>(scales + p.atom) = (uint16_t)(a0.scale | a1.scale << 8);
        } else if (in0 || in1) {
            const int at = p.atom + (in0 ? 0 : 1);
            *reinterpret_cast<uint2*>(codes + at * 8) = in0 ? a0.codes : a1.codes;
            scales[at] = (uint8_t)(in0 ? a0.scale : a1.scale);
        }
    }
}

template <typename T>
__global__ void __launch_bounds__(THREADS) append_rows_kernel(CachePages c, CacheStep s, RowsIn K, RowsIn V, Divide groups,
                                                              uint32_t* status) {
    const int i = blockIdx.x * THREADS + threadIdx.x, part = quotient(groups, i), group = i - part * groups.d;
    const int h = part >> 1, b = blockIdx.z, row = blockIdx.y;
    const bool is_v = part & 1;
    if (h >= c.heads) return;
    const SeqRec q = load_seq(s, c.page, b, status);
    const int pos = q.start + row;
    if (row >= q.rows || pos < 0) return;
    const RowsIn& R = is_v ? V : K;
    Row16<T> x;
    x.load((const T*)R.ptr + (int64_t)(q.row0 + row) * R.row + h * R.head + group * 16);
    const int page = pos / c.page, t = pos & 15;
    const int id = load_page(s, c, b, page, status);
    if (id < 0) return;
    uint8_t* block = block_of(c, id, h, (pos - page * c.page) >> 4);
    const float unit = is_v ? c.v_unit : c.k_unit;
    const Atom a = quantise(x, unit, __fdiv_rn(1.f, __fmul_rn(7.f, unit)));
    const int at = is_v ? value_atom(t, group, groups.d) : key_atom(t, group, groups.d);
    *reinterpret_cast<uint2*>(block + (is_v ? 8 * c.dim : 0) + at * 8) = a.codes;
    block[(is_v ? 17 * c.dim : 16 * c.dim) + at] = (uint8_t)a.scale;
}

// the halves of a bf16 pair, each times f
__device__ __forceinline__ void unpack_times(uint32_t w, float f, float& a, float& b) {
    asm("{\n .reg .b64 x, y;\n mov.b64 x, {%2, %3};\n mov.b64 y, {%4, %4};\n mul.rn.f32x2 x, x, y;\n mov.b64 {%0, %1}, x;\n}"
        : "=f"(a), "=f"(b)
        : "r"(w << 16), "r"(w & 0xFFFF0000u), "f"(f));
}
// (code * scale) * unit, the first product exact: 16 elements as they lie in memory
template <typename T>
__device__ __forceinline__ Row16<T> restored(uint2 codes, uint32_t scale, float unit) {
    const Scale2 s = scale_bf16(scale * 0x00010001u);
    Row16<T> r;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const uint32_t w = i ? codes.y : codes.x;
        const uint32_t y[4] = {codes_bf16<0>(w, s), codes_bf16<1>(w, s), codes_bf16<2>(w, s), codes_bf16<3>(w, s)};
        float v[8];
#pragma unroll
        for (int e = 0; e < 4; ++e) unpack_times(y[e], unit, v[e], v[4 + e]);
        if constexpr (sizeof(T) == 4) {
#pragma unroll
            for (int e = 0; e < 8; ++e) r.w[8 * i + e] = __float_as_uint(v[e]);
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const __nv_bfloat162 z = __floats2bfloat162_rn(v[2 * e], v[2 * e + 1]);
                r.w[4 * i + e] = *reinterpret_cast<const uint32_t*>(&z);
            }
        }
    }
    return r;
}

// A warp per block and head.
template <typename T>
__global__ void __launch_bounds__(THREADS) read_blocks_kernel(CachePages c, CacheStep s, RowsOut K, RowsOut V, uint32_t* status) {
    constexpr int AHEAD = 2;   // pairs that are loaded together
    const int h = blockIdx.y * (THREADS / 32) + threadIdx.x / 32, lane = threadIdx.x & 31, b = blockIdx.z;
    if (h >= c.heads) return;
    const SeqRec q = load_seq(s, c.page, b, status);
    const int j = (q.start >> 4) + (int)blockIdx.x;   // (rounded down) negative: rows that name no token
    const long long first = (long long)j * 16;        // its first position, perhaps outside 32 bits
    const int lo = (int)max(q.start - first, 0ll), hi = (int)min(q.start + q.rows - first, 16ll);
    if (hi <= lo) return;
    const int page = j >= 0 ? j * 16 / c.page : 0, id = j >= 0 ? load_page(s, c, b, page, status) : -1;
    const int64_t row = q.row0 + first - q.start;   // of the block's first token
    T* k_dst = (T*)K.ptr + row * K.row + h * K.head;
    T* v_dst = (T*)V.ptr + row * V.row + h * V.head;
    const uint8_t* block = block_of(c, max(id, 0), h, id < 0 ? 0 : j - page * (c.page >> 4));
    const int groups = c.dim >> 4, keys = pairs_of(false, groups), n = keys + pairs_of(true, groups);
    for (int i0 = 0; i0 < n; i0 += AHEAD) {
        uint4 w[AHEAD];
        uint32_t sc[AHEAD];
#pragma unroll
        for (int z = 0; z < AHEAD; ++z) {
            const bool is_v = i0 + z >= keys;
            const PairOf p = pair_of(is_v, is_v ? i0 + z - keys : i0 + z, lane, groups);
            w[z] = make_uint4(0u, 0u, 0u, 0u);
            sc[z] = 0u;
            if (id >= 0 && i0 + z < n && p.group < groups) {
                w[z] = __ldcs(reinterpret_cast<const uint4*>(block + (is_v ? 8 * c.dim : 0) + p.atom * 8));
                sc[z] = *reinterpret_cast<const uint16_t*>(block + (is_v ? 17 * c.dim : 16 * c.dim) + p.atom);
            }
        }
#pragma unroll
        for (int z = 0; z < AHEAD; ++z) {
            const bool is_v = i0 + z >= keys;
            const PairOf p = pair_of(is_v, is_v ? i0 + z - keys : i0 + z, lane, groups);
            if (i0 + z >= n || p.group >= groups) continue;
            T* dst = (is_v ? v_dst : k_dst) + p.group * 16;
            const int64_t stride = is_v ? V.row : K.row;
            const float unit = is_v ? c.v_unit : c.k_unit;
            const int t1 = p.t + p.next;
            if (p.t >= lo && p.t < hi) restored<T>(make_uint2(w[z].x, w[z].y), sc[z] & 0xFFu, unit).store(dst + p.t * stride);
            if (t1 >= lo && t1 < hi) restored<T>(make_uint2(w[z].z, w[z].w), sc[z] >> 8, unit).store(dst + t1 * stride);
        }
    }
}

template <typename T>
__global__ void __launch_bounds__(THREADS) read_rows_kernel(CachePages c, CacheStep s, RowsOut K, RowsOut V, Divide groups,
                                                            uint32_t* status) {
    const int i = blockIdx.x * THREADS + threadIdx.x, part = quotient(groups, i), group = i - part * groups.d;
    const int h = part >> 1, b = blockIdx.z, row = blockIdx.y;
    const bool is_v = part & 1;
    if (h >= c.heads) return;
    const SeqRec q = load_seq(s, c.page, b, status);
    if (row >= q.rows) return;
    const int pos = q.start + row, page = pos < 0 ? 0 : pos / c.page, t = pos & 15;
    const int id = pos < 0 ? -1 : load_page(s, c, b, page, status);
    uint2 w = make_uint2(0u, 0u);
    uint32_t sc = 0u;
    if (id >= 0) {
        const uint8_t* block = block_of(c, id, h, (pos - page * c.page) >> 4);
        const int at = is_v ? value_atom(t, group, groups.d) : key_atom(t, group, groups.d);
        w = *reinterpret_cast<const uint2*>(block + (is_v ? 8 * c.dim : 0) + at * 8);
        sc = block[(is_v ? 17 * c.dim : 16 * c.dim) + at];
    }
    const RowsOut& R = is_v ? V : K;
    restored<T>(w, sc, is_v ? c.v_unit : c.k_unit).store((T*)R.ptr + (int64_t)(q.row0 + row) * R.row + h * R.head + group * 16);
}

// 16-token blocks that max_new consecutive positions can touch.
int most_blocks(int max_new) { return (int)(((long long)max_new + 14) / 16) + 1; }

// Steps of few rows: a thread per atom, [heads, keys or values, groups] x rows x sequences.
template <typename Rows, typename Kernel>
cudaError_t launch_rows(Kernel kernel, const CachePages& c, const CacheStep& s, const Rows& k, const Rows& v, uint32_t* status,
                        cudaStream_t st) {
    const int groups = c.dim / 16;
    const dim3 grid((2 * c.heads * groups + THREADS - 1) / THREADS, s.max_new, s.n_seqs);
    kernel<<<grid, THREADS, 0, st>>>(c, s, k, v, divide_by(groups), status);
    return cudaGetLastError();
}
constexpr int WARPS = THREADS / 32;

template <typename T>
cudaError_t append(const CachePages& c, const CacheStep& s, const RowsIn& k, const RowsIn& v, uint32_t* status, cudaStream_t st) {
    if (s.max_new <= FEW) return launch_rows(append_rows_kernel<T>, c, s, k, v, status, st);
    const dim3 grid(most_blocks(s.max_new), (c.heads + WARPS - 1) / WARPS, s.n_seqs);
    append_blocks_kernel<T><<<grid, THREADS, 0, st>>>(c, s, k, v, status);
    return cudaGetLastError();
}

template <typename T>
cudaError_t read(const CachePages& c, const CacheStep& s, const RowsOut& k, const RowsOut& v, uint32_t* status, cudaStream_t st) {
    if (s.max_new <= FEW) return launch_rows(read_rows_kernel<T>, c, s, k, v, status, st);
    const dim3 grid(most_blocks(s.max_new), (c.heads + WARPS - 1) / WARPS, s.n_seqs);
    read_blocks_kernel<T><<<grid, THREADS, 0, st>>>(c, s, k, v, status);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_append4(bool bf16, const CachePages& c, const CacheStep& s, const RowsIn& k, const RowsIn& v,
                           uint32_t* status, cudaStream_t st) {
    return bf16 ? append<__nv_bfloat16>(c, s, k, v, status, st) : append<float>(c, s, k, v, status, st);
}

cudaError_t launch_read4(bool bf16, const CachePages& c, const CacheStep& s, const RowsOut& k, const RowsOut& v,
                         uint32_t* status, cudaStream_t st) {
    return bf16 ? read<__nv_bfloat16>(c, s, k, v, status, st) : read<float>(c, s, k, v, status, st);
}

}  // namespace mlora
