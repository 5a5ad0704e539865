// The 4-bit cache's append and read (include/mlora.h): rows to 4-bit codes with a scale per 16
// elements of a token, and back.
//
// Every atom (16 elements of a token) is a value of its own: nothing that the block held is read.
// Steps of many rows take a block of 16 tokens of a head's keys or values per warp, a lane two
// atoms that lie together in the block; steps of few rows an atom per thread, along the row.
#include <cuda_bf16.h>

#include "block4.cuh"
#include "cache.h"

namespace mlora {

namespace {

constexpr int THREADS = 128;
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
    __device__ __forceinline__ float at(int e) const {
        if (sizeof(T) == 4) return __uint_as_float(w[e]);
        return __uint_as_float(e & 1 ? w[e / 2] & 0xFFFF0000u : w[e / 2] << 16);
    }
};

struct Atom {
    uint2 codes;
    uint32_t scale;   // e4m3
};

// rint(x * inv) + 8 in the low byte: adding 1.5 * 2^23 + 8 leaves the integer (ties to even) in the
// sum's low mantissa bits.
template <bool CLAMP>
__device__ __forceinline__ uint32_t code_of(float x, float inv) {
    float t = __fmul_rn(x, inv);
    if (CLAMP) t = t != t ? 0.f : fminf(fmaxf(t, -7.f), 7.f);
    return __float_as_uint(__fadd_rn(t, 12582920.f));
}
template <bool CLAMP, typename T>
__device__ __forceinline__ uint2 codes16(const Row16<T>& x, float inv) {
    uint32_t w[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        uint32_t c[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) c[e] = code_of<CLAMP>(x.at(8 * i + e), inv);
        auto bytes = [&](int e) {   // codes e, e + 2, e + 4, e + 6
            return __byte_perm(__byte_perm(c[e], c[e + 2], 0x0040), __byte_perm(c[e + 4], c[e + 6], 0x0040), 0x5410);
        };
        w[i] = bytes(0) | bytes(1) << 4;
    }
    return make_uint2(w[0], w[1]);
}

// `grow` is 1 / (7 unit).
template <typename T>
__device__ __forceinline__ Atom quantise(const Row16<T>& x, float unit, float grow) {
    float top = 0.f;
    bool finite = true;
#pragma unroll
    for (int e = 0; e < 16; ++e) {   // infinities and NaN do not enter the maximum
        const float a = fabsf(x.at(e));
        const bool ok = a <= 3.402823466e38f;
        finite &= ok;
        top = fmaxf(top, ok ? a : 0.f);
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

template <typename T>
__global__ void __launch_bounds__(THREADS) append_blocks_kernel(CachePages c, CacheStep s, RowsIn K, RowsIn V, uint32_t* status) {
    const int part = blockIdx.y * (THREADS / 32) + threadIdx.x / 32, lane = threadIdx.x & 31;
    const int b = blockIdx.z, h = part >> 1;
    const bool is_v = part & 1;
    if (h >= c.heads) return;
    const SeqRec q = load_seq(s, c.page, b, status);
    const int start = max(q.start, 0), end = q.start + q.rows;
    const int j = (start >> 4) + (int)blockIdx.x;   // 16-token block of the sequence
    if ((long long)j * 16 >= end) return;           // (the launch covers max_new rows, of up to 2^31)
    const int lo = max(start - j * 16, 0), hi = min(end - j * 16, 16);
    if (hi <= lo) return;
    const int page = j * 16 / c.page;
    const int id = load_page(s, c, b, page, status);
    if (id < 0) return;
    const RowsIn& R = is_v ? V : K;
    const T* src = (const T*)R.ptr + (q.row0 + (int64_t)j * 16 - q.start) * R.row + h * R.head;
    uint8_t* block = block_of(c, id, h, j - page * (c.page >> 4));
    const int groups = c.dim >> 4;
    uint8_t* codes = block + (is_v ? 8 * c.dim : 0);
    uint8_t* scales = block + (is_v ? 17 * c.dim : 16 * c.dim);
    const float unit = is_v ? c.v_unit : c.k_unit, grow = __fdiv_rn(1.f, __fmul_rn(7.f, unit));
    const int n = pairs_of(is_v, groups);
#pragma unroll 2
    for (int it = 0; it < n; ++it) {
        const PairOf p = pair_of(is_v, it, lane, groups);
        if (p.group >= groups) continue;
        const int t1 = p.t + p.next;
        const bool in0 = p.t >= lo && p.t < hi, in1 = t1 >= lo && t1 < hi;
        Atom a0, a1;
        Row16<T> x;
        if (in0) {
            x.load(src + p.t * R.row + p.group * 16);
            a0 = quantise(x, unit, grow);
        }
        if (in1) {
            x.load(src + t1 * R.row + p.group * 16);
            a1 = quantise(x, unit, grow);
        }
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

// (code * scale) * unit, the first product exact
template <typename T>
__device__ __forceinline__ void restore(T* p, uint2 codes, uint32_t scale, float unit) {
    const Scale2 s = scale_bf16(scale * 0x00010001u);
    float v[16];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const uint32_t w = i ? codes.y : codes.x;
        const uint32_t y[4] = {codes_bf16<0>(w, s), codes_bf16<1>(w, s), codes_bf16<2>(w, s), codes_bf16<3>(w, s)};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            v[8 * i + e] = __fmul_rn(__uint_as_float(y[e] << 16), unit);
            v[8 * i + 4 + e] = __fmul_rn(__uint_as_float(y[e] & 0xFFFF0000u), unit);
        }
    }
    if constexpr (sizeof(T) == 4) {
#pragma unroll
        for (int i = 0; i < 4; ++i) reinterpret_cast<float4*>(p)[i] = make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
    } else {
        uint32_t y[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const __nv_bfloat162 z = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
            y[i] = *reinterpret_cast<const uint32_t*>(&z);
        }
        reinterpret_cast<uint4*>(p)[0] = make_uint4(y[0], y[1], y[2], y[3]);
        reinterpret_cast<uint4*>(p)[1] = make_uint4(y[4], y[5], y[6], y[7]);
    }
}

template <typename T>
__global__ void __launch_bounds__(THREADS) read_blocks_kernel(CachePages c, CacheStep s, RowsOut K, RowsOut V, uint32_t* status) {
    const int part = blockIdx.y * (THREADS / 32) + threadIdx.x / 32, lane = threadIdx.x & 31;
    const int b = blockIdx.z, h = part >> 1;
    const bool is_v = part & 1;
    if (h >= c.heads) return;
    const SeqRec q = load_seq(s, c.page, b, status);
    const int j = (q.start >> 4) + (int)blockIdx.x;   // (rounded down) negative: rows that name no token
    const long long first = (long long)j * 16;        // its first position, perhaps outside 32 bits
    const int lo = (int)max(q.start - first, 0ll), hi = (int)min(q.start + q.rows - first, 16ll);
    if (hi <= lo) return;
    const int page = j >= 0 ? j * 16 / c.page : 0, id = j >= 0 ? load_page(s, c, b, page, status) : -1;
    const RowsOut& R = is_v ? V : K;
    T* dst = (T*)R.ptr + (q.row0 + first - q.start) * R.row + h * R.head;
    const uint8_t* block = block_of(c, max(id, 0), h, id < 0 ? 0 : j - page * (c.page >> 4));
    const int groups = c.dim >> 4;
    const uint8_t* codes = block + (is_v ? 8 * c.dim : 0);
    const uint8_t* scales = block + (is_v ? 17 * c.dim : 16 * c.dim);
    const float unit = is_v ? c.v_unit : c.k_unit;
    const int n = pairs_of(is_v, groups);
#pragma unroll 2
    for (int it = 0; it < n; ++it) {
        const PairOf p = pair_of(is_v, it, lane, groups);
        if (p.group >= groups) continue;
        uint4 w = make_uint4(0u, 0u, 0u, 0u);
        uint32_t sc = 0u;
        if (id >= 0) {
            w = __ldcs(reinterpret_cast<const uint4*>(codes + p.atom * 8));
            sc = *reinterpret_cast<const uint16_t*>(scales + p.atom);
        }
        const int t1 = p.t + p.next;
        if (p.t >= lo && p.t < hi) restore(dst + p.t * R.row + p.group * 16, make_uint2(w.x, w.y), sc & 0xFFu, unit);
        if (t1 >= lo && t1 < hi) restore(dst + t1 * R.row + p.group * 16, make_uint2(w.z, w.w), sc >> 8, unit);
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
    restore((T*)R.ptr + (int64_t)(q.row0 + row) * R.row + h * R.head + group * 16, w, sc, is_v ? c.v_unit : c.k_unit);
}

// 16-token blocks that max_new consecutive positions can touch.
int most_blocks(int max_new) { return (int)(((long long)max_new + 14) / 16) + 1; }

template <typename Rows, typename Blocks, typename Single>
cudaError_t launch(Blocks blocks, Single single, const CachePages& c, const CacheStep& s, const Rows& k, const Rows& v,
                   uint32_t* status, cudaStream_t st) {
    if (s.max_new <= FEW) {
        const int groups = c.dim / 16;
        const dim3 grid((2 * c.heads * groups + THREADS - 1) / THREADS, s.max_new, s.n_seqs);
        single<<<grid, THREADS, 0, st>>>(c, s, k, v, divide_by(groups), status);
    } else {
        const dim3 grid(most_blocks(s.max_new), (2 * c.heads + THREADS / 32 - 1) / (THREADS / 32), s.n_seqs);
        blocks<<<grid, THREADS, 0, st>>>(c, s, k, v, status);
    }
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_append4(bool bf16, const CachePages& c, const CacheStep& s, const RowsIn& k, const RowsIn& v,
                           uint32_t* status, cudaStream_t st) {
    return bf16 ? launch(append_blocks_kernel<__nv_bfloat16>, append_rows_kernel<__nv_bfloat16>, c, s, k, v, status, st)
                : launch(append_blocks_kernel<float>, append_rows_kernel<float>, c, s, k, v, status, st);
}

cudaError_t launch_read4(bool bf16, const CachePages& c, const CacheStep& s, const RowsOut& k, const RowsOut& v,
                         uint32_t* status, cudaStream_t st) {
    return bf16 ? launch(read_blocks_kernel<__nv_bfloat16>, read_rows_kernel<__nv_bfloat16>, c, s, k, v, status, st)
                : launch(read_blocks_kernel<float>, read_rows_kernel<float>, c, s, k, v, status, st);
}

}  // namespace mlora
