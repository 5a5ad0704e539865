// Norms and rotation of query and key heads ahead of attention (include/mlora.h): C ABI and kernel.
//
// Mathematics.  A head x of D elements at position p:  y = w x / sqrt(mean(x^2) + eps)  (left out
// without weights), then pairs (a, b) of the first R elements turn by p f_i:
//     a' = a cos - b sin,  b' = a sin + b cos.
// Angles are held in turns: f / 2 pi as a 64-bit fraction, so that p times it, in wrapping
// integers, is the angle modulo a turn with no loss at any position; its nearest quarter turn is
// taken off before it becomes a float (of 24 bits: off by up to 2^-28 of a turn).
//
// A warp takes a row and some heads of its queries and keys.  A lane takes 16 elements of a head, in
// runs of 16 bytes that lie side by side with its neighbours'; sines and cosines are computed once for
// all the warp's heads and go, with the weights, into factors that the lane keeps: x' = x k0 + o k1, o
// being x's partner.  16 lanes at most share a head and its sum of squares.  Arithmetic is in pairs.
//
// Bound: HBM, each element read and written once: 29.6k rows of 32/8 heads of 128 in bf16 take 105 us,
// 5.8 TB/s (a plain copy of as many bytes 89 us), half of each head 108 us, of neighbours 109, in fp32 178 us, 6.8 TB/s; 4000 rows of 15 heads of
// 80 in fp32 11.5 us and 8 rows 2.9 us, a launch and the chain of offsets, length and sines.  What
// measured slower: two groups of heads on their way (117 us), rows without the factors (120 us).
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cmath>
#include <new>
#include <type_traits>

#include "abi.h"
#include "cache.h"
#include "f32x2.cuh"

using namespace mlora;

struct mlora_rotary {
    int device = 0, sms = 0;
    int dim = 0, turned = 0;      // head size, elements that turn
    bool interleaved = false;
    uint32_t* ws = nullptr;       // the status word, then the table
    uint64_t* turns = nullptr;    // [turned / 2] turns per position, in 2^-64
};

namespace {

constexpr int WARPS = 4, THREADS = 32 * WARPS;
constexpr int MOST = 16;   // groups of heads that a warp takes at most
// CTAs per SM (register limits): bf16 rows spill at 6 (a word; neighbours 4, of part of a head 8) and are faster all
// the same (30k rows of 32/8 heads 109 us, 113 us at 5, before whole heads had a form), fp32 rows would spill 20
template <typename T>
constexpr int CTAS = sizeof(T) == 2 ? 6 : 5;

struct RotaryArgs {
    RowsIn q, k;
    RowsOut qo, ko;
    int q_heads, kv_heads, dim, turned;
    const uint64_t* turns;
    const float* q_weight;
    const float* k_weight;
    float eps;
    CacheStep step;
    int q_groups, k_groups, per;   // groups of heads that a warp takes at a time, and how many of them a warp takes
    uint32_t* status;
};

__device__ __forceinline__ uint64_t swapped(uint64_t a) {
    const float2 v = unpair(a);
    return pair(v.y, v.x);
}

// 16 elements as they lie in memory, 16 bytes at each of the places `at`; eight pairs of adjacent ones.
template <typename T>
struct Raw {
    static constexpr int VEC = 16 / sizeof(T), N = 16 / VEC, W = 4 * N;   // elements in 16 bytes, such runs, words
    uint32_t w[W];
    __device__ __forceinline__ void clear() {
#pragma unroll
        for (int i = 0; i < W; ++i) w[i] = 0u;
    }
    __device__ __forceinline__ void load(const T* p, const int (&at)[N]) {
#pragma unroll
        for (int k = 0; k < N; ++k) {
            const uint4 v = *reinterpret_cast<const uint4*>(p + at[k]);
            w[4 * k] = v.x, w[4 * k + 1] = v.y, w[4 * k + 2] = v.z, w[4 * k + 3] = v.w;
        }
    }
    __device__ __forceinline__ void store(T* p, const int (&at)[N]) const {
#pragma unroll
        for (int k = 0; k < N; ++k)
            *reinterpret_cast<uint4*>(p + at[k]) = make_uint4(w[4 * k], w[4 * k + 1], w[4 * k + 2], w[4 * k + 3]);
    }
    __device__ __forceinline__ void get(uint64_t (&x)[8]) const {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            x[i] = sizeof(T) == 4 ? pair(__uint_as_float(w[2 * i % W]), __uint_as_float(w[(2 * i + 1) % W]))
                                  : pair(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xFFFF0000u));
    }
    __device__ __forceinline__ void put(int i, uint64_t x) {
        const float2 v = unpair(x);
        if (sizeof(T) == 4) {
            w[2 * i % W] = __float_as_uint(v.x);
            w[(2 * i + 1) % W] = __float_as_uint(v.y);
        } else {
            const __nv_bfloat162 h = __floats2bfloat162_rn(v.x, v.y);
            w[i] = *reinterpret_cast<const uint32_t*>(&h);
        }
    }
};
// Sine and cosine of an angle in turns, 2^-64 each.
__device__ __forceinline__ float2 cos_sin(uint64_t turns) {
    const uint32_t quarter = (uint32_t)((turns + (1ull << 61)) >> 62);
    const int rest = (int)((int64_t)(turns - ((uint64_t)quarter << 62)) >> 30);   // within an eighth of a turn, 2^-34 each
    float s, c;
    sincospif(__int2float_rn(rest) * 0x1p-33f, &s, &c);
    if (quarter & 1) {
        const float t = c;
        c = -s;
        s = t;
    }
    return quarter & 2 ? make_float2(-c, -s) : make_float2(c, s);
}

// The sequence that holds a row: the last whose range begins at or before it (32 looks at a time).
__device__ __forceinline__ int sequence_of(const CacheStep& s, int row, int lane) {
    int lo = 0, hi = s.n_seqs;
    while (hi - lo > 1) {
        const int step = (hi - lo + 31) / 32, at = lo + lane * step;
        const int n = __popc(__ballot_sync(~0u, at < hi && s.offsets[min(at, hi - 1)] <= row));
        lo += max(n - 1, 0) * step;
        hi = min(lo + step, hi);
    }
    return min(lo, s.n_seqs - 1);
}

// LANES: of a head (its 16-element slots, rounded up to a power of two).  ALL: every element turns.
template <typename T, int LANES, bool INTERLEAVED, bool ALL>
__global__ void __launch_bounds__(THREADS, CTAS<T>) rotary_kernel(const RotaryArgs a) {
    constexpr int HEADS = 32 / LANES;   // at a time
    __shared__ float2 turn[WARPS][128];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    // lengths and limits of the sequences are as load_seq checks them, up to 2^30 tokens
    constexpr int PAGE = 1 << 15;
    if (a.step.offsets && blockIdx.x == 0 && blockIdx.y == 0)   // ranges that hold no row are looked at here
        for (int b = threadIdx.x; b < a.step.n_seqs; b += THREADS) load_seq(a.step, PAGE, b, a.status);
    const int row = blockIdx.x * WARPS + warp;
    if (row >= a.step.T) return;
    const int sub = lane / LANES, slot = lane % LANES;
    const bool mine = slot * 16 < a.dim, turns = ALL || slot * 16 < a.turned;
    // the slot's runs of 16 bytes, such that those of a head's slots lie side by side: of the elements that
    // turn, or of the others; the second half of the runs are the first half's partners
    using Row = Raw<T>;
    const int base = turns ? 0 : a.turned, length = turns ? a.turned : a.dim - a.turned;
    int at[Row::N];
#pragma unroll
    for (int k = 0; k < Row::N; ++k) at[k] = base + (slot - base / 16) * Row::VEC + k * (length / Row::N);

    // groups of heads [g0, g1): the queries' first, then the keys'.  The next group's elements are on
    // their way while one is turned.
    const int g0 = blockIdx.y * a.per, g1 = min(g0 + a.per, a.q_groups + a.k_groups);
    Row next;
    const T* src = nullptr;   // the lane's head of the group that is fetched next
    int64_t src_step = 0;
    auto seek = [&](int g) {
        const bool is_k = g >= a.q_groups;
        const int64_t head = is_k ? a.k.head : a.q.head;
        src = (const T*)(is_k ? a.k.ptr : a.q.ptr) + row * (is_k ? a.k.row : a.q.row) + ((is_k ? g - a.q_groups : g) * HEADS + sub) * head;
        src_step = HEADS * head;
    };
    auto there = [&](int g) { return mine && (g < a.q_groups ? g * HEADS + sub < a.q_heads : (g - a.q_groups) * HEADS + sub < a.kv_heads); };
    auto fetch = [&](int g) {
        if (g == a.q_groups) seek(g);
        if (g < g1 && there(g)) next.load(src, at);
        else next.clear();
        src += src_step;
    };
    seek(g0);
    fetch(g0);   // (before the row's position is known: that is a chain of loads)

    const int b = a.step.offsets ? sequence_of(a.step, row, lane) : row;
    const SeqRec s = load_seq(a.step, PAGE, b, a.status);
    const int i = row - s.row0;
    if (i < 0 || i >= s.rows) return;   // of no sequence
    const int pos = s.start + i;
    for (int p = lane; p < a.turned / 2; p += 32) turn[warp][p] = cos_sin((uint64_t)(int64_t)pos * a.turns[p]);
    __syncwarp();
    const float inv_dim = 1.f / (float)a.dim;
    for (int g = g0; g < g1;) {
        // the queries' groups, or the keys'
        const bool is_k = g >= a.q_groups;
        const int last = is_k ? g1 : min(g1, a.q_groups);
        const float* weight = is_k ? a.k_weight : a.q_weight;
        const int64_t dst_head = is_k ? a.ko.head : a.qo.head;
        T* dst = (T*)(is_k ? a.ko.ptr : a.qo.ptr) + row * (is_k ? a.ko.row : a.qo.row) + ((is_k ? g - a.q_groups : g) * HEADS + sub) * dst_head;
        // A pair x of adjacent elements, and its partner o (the other half's pair, or x itself swapped):
        // x' = x k0 + o k1 holds the weights and the turn (x' = x k0 for elements that do not turn)
        uint64_t k0[8], k1[8];
        {
            float w[16];
#pragma unroll
            for (int e = 0; e < 16; e += 4) {
                const float4 v = weight && mine ? *reinterpret_cast<const float4*>(weight + at[e / Row::VEC] + e % Row::VEC)
                                                : make_float4(1.f, 1.f, 1.f, 1.f);
                w[e] = v.x, w[e + 1] = v.y, w[e + 2] = v.z, w[e + 3] = v.w;
            }
            float2 v[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) {   // of the lane's pairs
                const int i = INTERLEAVED ? 2 * e : e, p = at[i / Row::VEC] + i % Row::VEC;
                v[e] = turns && (!ALL || mine) ? turn[warp][INTERLEAVED ? p / 2 : p] : make_float2(1.f, 0.f);
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                if (INTERLEAVED) {
                    k0[i] = pair(v[i].x * w[2 * i], v[i].x * w[2 * i + 1]);
                    k1[i] = pair(-v[i].y * w[2 * i + 1], v[i].y * w[2 * i]);
                } else {
                    const int c = i % 4 * 2, o = (2 * i) ^ 8;   // (the partner's first element)
                    const float sign = i < 4 ? -1.f : 1.f;
                    k0[i] = pair(v[c].x * w[2 * i], v[c + 1].x * w[2 * i + 1]);
                    k1[i] = pair(sign * v[c].y * w[o], sign * v[c + 1].y * w[o + 1]);
                }
            }
        }
#pragma unroll 1
        for (; g < last; ++g) {
            uint64_t x[8];
            if (pos < 0) next.clear();
            next.get(x);
            fetch(g + 1);
            float inv = 1.f;
            if (weight && pos >= 0) {
                auto squares = [&]() {
                    uint64_t t = mul2(x[0], x[0]);
#pragma unroll
                    for (int i = 1; i < 8; ++i) t = fma2(x[i], x[i], t);
                    const float2 v = unpair(t);
                    float r = v.x + v.y;
#pragma unroll
                    for (int d = 1; d < LANES; d <<= 1) r += __shfl_xor_sync(~0u, r, d);
                    return r;
                };
                float sum = squares(), eps = a.eps;
                // squares that leave fp32, or are lost beside no eps: the head by a power of two
                const bool far = !(sum <= 0x1p120f) || (sum < 0x1p-90f && eps < 0x1p-70f);
                if (__any_sync(~0u, far)) {
                    const float f = !far ? 1.f : !(sum <= 0x1p120f) ? 0x1p-70f : 0x1p60f;
#pragma unroll
                    for (int i = 0; i < 8; ++i) x[i] = mul2(x[i], pair(f, f));
                    sum = squares();
                    eps = eps * f * f;
                }
                const float mean = fmaf(sum, inv_dim, eps), r = rsqrtf(mean);
                inv = mean == 0.f || mean > 3.4e38f ? 0.f : fmaf(r * 0.5f, fmaf(-mean * r, r, 1.f), r);   // (a Newton step)
            }
            Row out;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                uint64_t y = mul2(x[i], k0[i]);
                if (turns) y = fma2(INTERLEAVED ? swapped(x[i]) : x[i ^ 4], k1[i], y);
                out.put(i, mul2(y, pair(inv, inv)));   // (exact where there is no norm)
            }
            if (there(g)) out.store(dst, at);
            dst += HEADS * dst_head;
        }
    }
}

template <typename T, int LANES>
cudaError_t launch(RotaryArgs a, bool interleaved, int sms, cudaStream_t st) {
    constexpr int HEADS = 32 / LANES;
    a.q_groups = (a.q_heads + HEADS - 1) / HEADS;
    a.k_groups = (a.kv_heads + HEADS - 1) / HEADS;
    // groups of heads per warp: as many as leave some 32 warps to an SM, MOST at most
    const int all = a.q_groups + a.k_groups;
    const long long groups = (long long)a.step.T * all / (32ll * sms);
    a.per = groups < 1 ? 1 : groups > MOST ? MOST : (int)groups;
    a.per = (all + (all + a.per - 1) / a.per - 1) / ((all + a.per - 1) / a.per);   // (as equal as they can be)
    const dim3 grid((unsigned)(((long long)a.step.T + WARPS - 1) / WARPS), (all + a.per - 1) / a.per);
    const bool whole = a.turned == a.dim;
    const auto kernel = interleaved ? (whole ? rotary_kernel<T, LANES, true, true> : rotary_kernel<T, LANES, true, false>)
                                    : (whole ? rotary_kernel<T, LANES, false, true> : rotary_kernel<T, LANES, false, false>);
    kernel<<<grid, THREADS, 0, st>>>(a);
    return cudaGetLastError();
}

template <typename T>
cudaError_t launch_by_dim(const RotaryArgs& a, bool interleaved, int sms, cudaStream_t st) {
    const int slots = a.dim / 16;
    return slots == 1 ? launch<T, 1>(a, interleaved, sms, st)
         : slots == 2 ? launch<T, 2>(a, interleaved, sms, st)
         : slots <= 4 ? launch<T, 4>(a, interleaved, sms, st)
         : slots <= 8 ? launch<T, 8>(a, interleaved, sms, st)
                      : launch<T, 16>(a, interleaved, sms, st);
}

// A frequency in radians per position as turns per position, modulo 1, in 2^-64: 1 / 2 pi in two
// doubles, the product's rounding kept.
uint64_t turns_of(double f) {
    constexpr double hi = 0x1.45f306dc9c883p-3, lo = -0x1.6b01ec5417056p-57;
    if (f < 0) return 0u - turns_of(-f);
    const double t = f * hi, rest = std::fma(f, hi, -t) + f * lo;
    return (uint64_t)((t - std::floor(t)) * 0x1p64) + (uint64_t)(int64_t)std::llrint(rest * 0x1p64);   // (the difference is exact)
}

// Whether two of rows x heads runs of `dim` elements, at i row + j head (strides >= 0), have an element
// in common: whether |i row - j head| < dim for some i < rows and j < heads that are not both 0.
bool heads_overlap(int rows, int64_t row, int heads, int64_t head, int dim) {
    if ((rows > 1 && row < dim) || (heads > 1 && head < dim)) return true;
    if (rows == 1 || heads == 1) return false;
    // rows that end before the next begins, heads that do
    if ((__int128)(heads - 1) * head + dim <= row || (__int128)(rows - 1) * row + dim <= head) return false;
    for (int j = 1; j < heads; ++j) {   // the rows to both sides of head j of row 0
        const __int128 at = (__int128)j * head, i = at / row, past = at - i * row;
        if (i >= rows) return false;
        if (i > 0 && past < dim) return true;
        if (i + 1 < rows && row - past < dim) return true;
    }
    return false;
}

}  // namespace

extern "C" {

mlora_status mlora_rotary_create(int head_dim, int rotary_dim, const double* freq, int interleaved, mlora_rotary_t* out) {
    if (!out) return fail(MLORA_ERR_INVALID_ARG, "out is NULL");
    *out = nullptr;
    if (head_dim < 16 || head_dim > 256 || head_dim % 16)
        return fail(MLORA_ERR_UNSUPPORTED, "head_dim %d must be a multiple of 16 in [16, 256]", head_dim);
    if (rotary_dim < 0 || rotary_dim > head_dim || rotary_dim % 16)
        return fail(MLORA_ERR_UNSUPPORTED, "rotary_dim %d must be a multiple of 16 in [0, head_dim]", rotary_dim);
    if (rotary_dim && !freq) return fail(MLORA_ERR_INVALID_ARG, "freq is NULL");
    uint64_t table[128];
    for (int i = 0; i < rotary_dim / 2; ++i) {
        if (!(std::fabs(freq[i]) <= 1024.0))
            return fail(MLORA_ERR_INVALID_ARG, "freq[%d] = %g is not a number of radians per position in [-1024, 1024]", i, freq[i]);
        table[i] = turns_of(freq[i]);
    }
    mlora_rotary* r = new (std::nothrow) mlora_rotary;
    if (!r) return fail(MLORA_ERR_OOM, "host memory");
    r->dim = head_dim;
    r->turned = rotary_dim;
    r->interleaved = interleaved != 0;
    cudaError_t e = cudaGetDevice(&r->device);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&r->sms, cudaDevAttrMultiProcessorCount, r->device);
    if (e == cudaSuccess) e = cudaMalloc((void**)&r->ws, 256 + sizeof table);
    if (e == cudaSuccess) {
        r->turns = (uint64_t*)((char*)r->ws + 256);
        e = cudaMemset(r->ws, 0, 256);
    }
    if (e == cudaSuccess && rotary_dim)
        e = cudaMemcpy(r->turns, table, rotary_dim / 2 * sizeof(uint64_t), cudaMemcpyHostToDevice);
    // both are queued on the legacy stream, which other streams need not wait for
    if (e == cudaSuccess) e = cudaDeviceSynchronize();
    if (e != cudaSuccess) {
        cudaGetLastError();   // (as in cuda_fail)
        if (r->ws) cudaFree(r->ws);
        delete r;
        return e == cudaErrorMemoryAllocation ? fail(MLORA_ERR_OOM, "workspace: %s", cudaGetErrorString(e))
                                              : cuda_fail(e, "mlora_rotary_create");
    }
    *out = r;
    return MLORA_OK;
}

mlora_status mlora_rotary_destroy(mlora_rotary_t r) {
    if (!r) return MLORA_OK;
    DeviceGuard g(r->device);
    cudaError_t e = g.err;
    if (e == cudaSuccess) e = cudaDeviceSynchronize();
    if (r->ws) cudaFree(r->ws);
    delete r;
    return e == cudaSuccess ? MLORA_OK : cuda_fail(e, "mlora_rotary_destroy");
}

mlora_status mlora_rotary_apply(mlora_rotary_t r, const void* Q, int64_t q_row, int64_t q_head, void* Qo, int64_t qo_row,
                                int64_t qo_head, int q_heads, const void* K, int64_t k_row, int64_t k_head, void* Ko,
                                int64_t ko_row, int64_t ko_head, int kv_heads, mlora_dtype dtype, int T,
                                const float* q_weight, const float* k_weight, float eps, const int32_t* offsets,
                                const int32_t* lengths, int n_seqs, int max_new, mlora_stream_t stream) {
    if (!r) return fail(MLORA_ERR_INVALID_ARG, "rotary is NULL");
    if (dtype != MLORA_F32 && dtype != MLORA_BF16) return fail(MLORA_ERR_INVALID_ARG, "dtype %d", (int)dtype);
    if (T < 0 || n_seqs < 0 || max_new < 0)
        return fail(MLORA_ERR_INVALID_ARG, "T %d, n_seqs %d or max_new %d is negative", T, n_seqs, max_new);
    if (n_seqs > 65535) return fail(MLORA_ERR_INVALID_ARG, "n_seqs %d exceeds 65535", n_seqs);
    if (!offsets && T != n_seqs)
        return fail(MLORA_ERR_INVALID_ARG, "without offsets T %d must equal n_seqs %d", T, n_seqs);
    if (q_heads < 1 || q_heads > 32767 || kv_heads < 1 || kv_heads > 32767)
        return fail(MLORA_ERR_INVALID_ARG, "q_heads %d and kv_heads %d must lie in [1, 32767]", q_heads, kv_heads);
    if (!(eps >= 0.f && eps < 3.0e38f)) return fail(MLORA_ERR_INVALID_ARG, "eps %g", eps);
    if (((uintptr_t)q_weight | (uintptr_t)k_weight) & 15u)
        return fail(MLORA_ERR_INVALID_ARG, "weights must be 16-byte aligned");
    if (!(T > 0 && n_seqs > 0 && max_new > 0)) return MLORA_OK;
    if (!lengths) return fail(MLORA_ERR_INVALID_ARG, "lengths is NULL");
    mlora_status st = check_rows("Q", Q, q_row, q_head, dtype);
    if (st == MLORA_OK) st = check_rows("Q_out", Qo, qo_row, qo_head, dtype);
    if (st == MLORA_OK) st = check_rows("K", K, k_row, k_head, dtype);
    if (st == MLORA_OK) st = check_rows("K_out", Ko, ko_row, ko_head, dtype);
    if (st != MLORA_OK) return st;
    if (Qo == Ko) return fail(MLORA_ERR_INVALID_ARG, "Q_out and K_out are the same memory");
    // (heads of an output that lie in one another would be written by several warps)
    if (heads_overlap(T, qo_row, q_heads, qo_head, r->dim) || heads_overlap(T, ko_row, kv_heads, ko_head, r->dim))
        return fail(MLORA_ERR_INVALID_ARG, "an output's heads of %d elements overlap (strides %lld, %lld and %lld, %lld)", r->dim,
                    (long long)qo_row, (long long)qo_head, (long long)ko_row, (long long)ko_head);
    DeviceGuard g(r->device);
    if (g.err != cudaSuccess) return cuda_fail(g.err, "cudaSetDevice");
    const CacheStep step{offsets, lengths, nullptr, n_seqs, 1 << 15, T, max_new < T ? max_new : T};
    const RotaryArgs a{RowsIn{Q, q_row, q_head}, RowsIn{K, k_row, k_head}, RowsOut{Qo, qo_row, qo_head},
                       RowsOut{Ko, ko_row, ko_head}, q_heads, kv_heads, r->dim, r->turned, r->turns, q_weight, k_weight,
                       eps, step, 0, 0, 0, r->ws};
    const cudaError_t e = dtype == MLORA_BF16
                              ? launch_by_dim<__nv_bfloat16>(a, r->interleaved, r->sms, (cudaStream_t)stream)
                              : launch_by_dim<float>(a, r->interleaved, r->sms, (cudaStream_t)stream);
    return e == cudaSuccess ? MLORA_OK : cuda_fail(e, "mlora_rotary_apply");
}

mlora_status mlora_rotary_status(mlora_rotary_t r, mlora_stream_t stream) {
    if (!r) return fail(MLORA_ERR_INVALID_ARG, "rotary is NULL");
    DeviceGuard g(r->device);
    cudaError_t e = g.err;
    cudaStream_t st = (cudaStream_t)stream;
    uint32_t word = 0;
    if (e == cudaSuccess) e = cudaMemcpyAsync(&word, r->ws, sizeof word, cudaMemcpyDeviceToHost, st);
    if (e == cudaSuccess) e = cudaMemsetAsync(r->ws, 0, sizeof word, st);
    if (e == cudaSuccess) e = cudaStreamSynchronize(st);
    if (e != cudaSuccess) return cuda_fail(e, "mlora_rotary_status");
    if (word & STATUS_BAD_STEP) return fail(MLORA_ERR_DEVICE_STEP, "a step named rows or lengths out of range");
    return MLORA_OK;
}

}  // extern "C"
