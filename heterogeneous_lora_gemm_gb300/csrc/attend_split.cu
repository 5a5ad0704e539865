// Causal attention over the 8-bit cache for sequences with few rows in the step (decode:
// one token), any row and head count (include/mlora.h).
//
// Mathematics.  With codes kc, vc and page scales ks, vs, row r (query token i, query head
// g of the key/value head's group) has  x_t = scale ks_t (q_r . kc_t),  and
//     o_r = sum_t 2^(x'_t - m) vs_t vc_t / sum_t 2^(x'_t - m),   x' = x log2 e,
// with a running m: only a lower bound of the maximum is needed, so m moves (and the
// accumulators are rescaled) only when some x' exceeds m + 8.
//
// Products run on mma.sync m16n8k16 with fp32 sums, transposed: tokens (S^T = K Q^T) and
// head elements (O^T = V^T P^T) are the 16-row side, query rows the 8-column side, so that
// a group of up to 8 heads wastes nothing.  S^T takes fp16: a code is exact in it (byte ^
// 0x80 under the exponent of 1024, minus 1152: the cheapest conversion), and so is a bf16
// query that a power of two per row has brought below 1 (its elements under 2^-14 of the
// row's largest round to 2^-25 of it).  O^T takes bf16: the weights, times vs, need its
// range (a heavy token may hold a zero where light ones do not), as the sum of two terms (16
// bits: one term's 8 would be off by as much as the rounded output; the tensor pipe has room
// under the codes' stream).  fp32 rows run the same products with the query as the sum of two
// fp16 terms (22 bits) and the weights as three bf16 terms (24 bits).
//
// Bound: HBM (the codes are read once per row tile): 32 sequences of 32k tokens, 32/8 heads of
// 128, bf16, take 328 us, 6.5 TB/s; 4 sequences 150 us, 5.9 TB/s; 32 of 3 to 4k with as many key
// heads as query heads 83 us, 5.1 TB/s; one short sequence 9.7 us, the chain of a CTA's start, a
// range's loads and the join.  Each warp streams 32-token chunks
// of its own through a private ring of TMA copies: no CTA-wide barrier in the loop.
// Work split: all (sequence, row tile, head) items' tokens in one line, cut into equal
// ranges, one per resident CTA; every CTA finds its range from the lengths.  An item is as
// long as its tokens plus what its start costs (LEAD).  An item cut between CTAs is joined,
// in range order, by the CTA that finishes it last, so results do not depend on timing.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "attend.h"
#include "attend_mma.cuh"
#include "tc_ptx.cuh"

namespace mlora {

using namespace ptx;

namespace {

constexpr int WARPS = 4, THREADS = 32 * WARPS;
constexpr int PIECE = 16;                 // tokens of a copied box and of a product
constexpr int LEAD = 1;                   // units (of WARPS chunks) that starting an item costs
constexpr int MIN_UNITS = LEAD + 1;       // a CTA's range is at least so long
constexpr float SLACK = 8.f;              // m moves when x > m + 8: weights stay below 2^8
constexpr float NO_MAX = -1e38f;          // m before anything is seen (finite: -inf - m stays -inf)

template <bool F32, int DP, int NT>
struct Shape {
    static constexpr int TERMS = F32 ? 2 : 1;          // of a query
    static constexpr int PTERMS = F32 ? 3 : 2;         // of a weight
    static constexpr int KS = DP / 16;                 // k steps of q . k = 16-row tiles of O^T
    static constexpr int RT = 8 * NT;                  // query rows per tile
    static constexpr int CB = DP == 256 ? 2 : 1;       // column boxes
    static constexpr int ROWB = DP / CB;               // bytes of a box row
    static constexpr int BOX = PIECE * ROWB;
    // a warp takes a chunk of two pieces at a time: waits, votes and issues are per chunk
    // (one where the accumulators leave no registers for two)
    static constexpr int SUB = DP == 256 ? 1 : 2;
    static constexpr int CHUNK_T = PIECE * SUB;
    static constexpr int PART = 2 * CB * BOX;          // keys and values of a piece
    static constexpr int STAGE = SUB * PART;
    // CTAs per SM: three where the accumulators of 8 rows leave the registers, else two
    static constexpr int OCC = !F32 && DP <= 128 && NT == 1 ? 3 : 2;
    // (64 KB of ring also where the queries' fragments leave no more, 16 fp32 rows of up to 256 elements: 2 x
    // 300 rows after 1000, 16/8 heads, 124 us, 188 us with the 96 KB that one CTA per SM has room for)
    static constexpr int STAGES = (OCC == 3 || (F32 && DP == 256 && NT == 2) ? 64 : 96) * 1024 / WARPS / STAGE;
    static constexpr int RING = WARPS * STAGES * STAGE;
    static constexpr int QWORDS = KS * NT * TERMS * 64;    // query fragments, 32-bit words
    static constexpr int SMEM = 1024 + RING + QWORDS * 4;
    static constexpr int SLOT = RT * (DP + 2);             // floats of a partial result: O, then m, l per row
    static_assert(WARPS * RT * DP * 4 <= RING, "the join buffer lies in the ring");
};

// shared-memory offset of 16-byte chunk `c` of box row `r`
template <int ROWB>
__device__ __forceinline__ int swz(int r, int c) {
    return ROWB == 128 ? r * 128 + ((c ^ (r & 7)) << 4) : r * 64 + ((c ^ ((r >> 1) & 3)) << 4);
}

__device__ __forceinline__ uint32_t prmt(uint32_t a, uint32_t b, uint32_t s) { return __byte_perm(a, b, s); }
// two bytes (code + 128) under 0x64 -> two codes in fp16
__device__ __forceinline__ uint32_t minus1152(uint32_t u) {
    const __half2 h = __hsub2(*reinterpret_cast<__half2*>(&u), __half2half2(__ushort_as_half(0x6480)));
    return *reinterpret_cast<const uint32_t*>(&h);
}
// two bytes under 0x43 -> two codes in bf16: 128 + low 7 bits, minus 128 or (sign bit) 256
__device__ __forceinline__ uint32_t bf16_codes(uint32_t u) {
    const uint32_t a = u & 0xFF7FFF7Fu, b = u & 0xFF80FF80u;
    const __nv_bfloat162 h = __hsub2(*reinterpret_cast<const __nv_bfloat162*>(&a), *reinterpret_cast<const __nv_bfloat162*>(&b));
    return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ void mma_bf(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                       uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, "
        "%2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// A sequence's share of the work line: tiles x heads items, each LEAD + units long (1 where the
// rows see nothing: zeros are written).
struct Line {
    SeqRec s;
    int c0, c1;       // chunks [c0, c1) that its rows see
    int tiles, units; // row tiles, units of tokens per item
    __device__ int length() const { return units ? LEAD + units : 1; }
    __device__ long long total(int heads) const { return (long long)tiles * heads * length(); }
};
template <int RT, int CHUNK_T>
__device__ __forceinline__ Line line_of(const AttendArgs& a, int G, int b) {
    Line n;
    n.s = load_seq(a.step, a.pages.page, b, a.status);
    const int last = n.s.start + n.s.rows - 1;   // position of the last processed row
    n.c0 = first_seen(n.s.start, a.window) / CHUNK_T;
    n.c1 = last >= 0 ? last / CHUNK_T + 1 : n.c0;
    n.tiles = (n.s.rows * G + RT - 1) / RT;
    n.units = (n.c1 - n.c0 + WARPS - 1) / WARPS;
    return n;
}

struct Tail {
    uint64_t full[WARPS][8];
    int abort_flag;
    int first_b, last_of;
    long long first_at;
    Line first;
    long long scan[WARPS];
    float qf[32];
    float m[WARPS][32], l[WARPS][32];
};

// N adjacent elements as floats (N x their size: 4 to 32 bytes, aligned), zeros unless `there`
template <int N>
__device__ __forceinline__ void load_elements(const float* p, bool there, float* x) {
#pragma unroll
    for (int e = 0; e < N; e += 2) {
        const float2 v = there ? *reinterpret_cast<const float2*>(p + e) : make_float2(0.f, 0.f);
        x[e] = v.x, x[e + 1] = v.y;
    }
}
template <int N>
__device__ __forceinline__ void load_elements(const __nv_bfloat16* p, bool there, float* x) {
    uint32_t w[N / 2];
    if (N == 2) w[0] = there ? *reinterpret_cast<const uint32_t*>(p) : 0u;
    if (N == 4) {
        const uint2 u = there ? *reinterpret_cast<const uint2*>(p) : make_uint2(0u, 0u);
        w[0] = u.x, w[N / 2 - 1] = u.y;
    }
    if (N == 8) {
        const uint4 u = there ? *reinterpret_cast<const uint4*>(p) : make_uint4(0u, 0u, 0u, 0u);
        w[0] = u.x, w[1 % (N / 2)] = u.y, w[2 % (N / 2)] = u.z, w[3 % (N / 2)] = u.w;
    }
#pragma unroll
    for (int i = 0; i < N / 2; ++i) {
        x[2 * i] = __uint_as_float(w[i] << 16);
        x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
}

template <bool F32, int DP, int NT>
__global__ void __launch_bounds__(THREADS, (Shape<F32, DP, NT>::OCC))
attend_split_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV, const AttendArgs a,
                    float* __restrict__ partial, int* __restrict__ counters) {
    using Sh = Shape<F32, DP, NT>;
    using E = typename std::conditional<F32, float, __nv_bfloat16>::type;
    constexpr int KS = Sh::KS, RT = Sh::RT, SUB = Sh::SUB, CHUNK_T = Sh::CHUNK_T, TERMS = Sh::TERMS, PTERMS = Sh::PTERMS, CB = Sh::CB;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t* smem = (uint8_t*)(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
    uint32_t* qfrag = reinterpret_cast<uint32_t*>(smem + Sh::RING);
    float* join = reinterpret_cast<float*>(smem);
    __shared__ Tail tl;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, tig = lane & 3;
    const CachePages& c = a.pages;
    const int H = c.heads, G = a.q_heads / H, D = c.dim;

    // ---- this CTA's range of the line
    if (lane == 0) {
        for (int s = 0; s < Sh::STAGES; ++s) mbar_init(&tl.full[warp][s], 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (tid == 0) tl.abort_flag = 0;
    if (tid == 0) {
        asm volatile("prefetch.tensormap [%0];" ::"l"(&tmK) : "memory");
        asm volatile("prefetch.tensormap [%0];" ::"l"(&tmV) : "memory");
    }
    const int per = (a.step.n_seqs + THREADS - 1) / THREADS;
    const int b_lo = min(tid * per, a.step.n_seqs), b_hi = min(b_lo + per, a.step.n_seqs);
    Line n;
    long long mine = 0;
    for (int b = b_lo; b < b_hi; ++b) {
        n = line_of<RT, Sh::CHUNK_T>(a, G, b);
        mine += n.total(H);
    }
    long long incl = mine;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const long long v = __shfl_up_sync(~0u, incl, d);
        if (lane >= d) incl += v;
    }
    if (lane == 31) tl.scan[warp] = incl;
    __syncthreads();
    long long total = 0, before = 0;
#pragma unroll
    for (int w = 0; w < WARPS; ++w) {
        if (w < warp) before += tl.scan[w];
        total += tl.scan[w];
    }
    before += incl - mine;
    const int cta = blockIdx.x;
    const int ctas = total >= (long long)MIN_UNITS * gridDim.x ? (int)gridDim.x : ((int)total + MIN_UNITS - 1) / MIN_UNITS;
    if (cta >= ctas) return;
    // ranges: the first `over` of them one longer than the others
    const long long each = total >> 31 ? total / ctas : (uint32_t)total / (uint32_t)ctas;
    const int over = (int)(total - each * ctas);
    auto range_at = [&](int i) { return each * i + min(i, over); };
    auto cta_of = [&](long long u) {   // the CTA whose range holds position u
        const long long cut = (each + 1) * over, v = u < cut ? u : u - cut, w = u < cut ? each + 1 : each;
        return (u < cut ? 0 : over) + (int)(total >> 31 ? v / w : (uint32_t)v / (uint32_t)w);
    };
    long long at = range_at(cta);
    const long long end = range_at(cta + 1);
    if (at >= before && at < before + mine) {
        long long p = before;
        int b = b_lo;
        if (per > 1)
            for (; b < b_hi; ++b) {
                n = line_of<RT, Sh::CHUNK_T>(a, G, b);
                if (at < p + n.total(H)) break;
                p += n.total(H);
            }
        tl.first_b = b;
        tl.first_at = p;
        tl.first = n;
    }
    __syncthreads();
    int b = tl.first_b;
    long long b_at = tl.first_at;   // where sequence b begins on the line
    n = tl.first;

    uint32_t issued = 0, used = 0;     // chunks copied and consumed by this warp, over all items
    uint8_t* ring = smem + warp * Sh::STAGES * Sh::STAGE;
    volatile int* abort_flag = &tl.abort_flag;
    bool alive = true;

    while (at < end) {
        while (at >= b_at + n.total(H)) {
            b_at += n.total(H);
            n = line_of<RT, Sh::CHUNK_T>(a, G, ++b);
        }
        const long long into = at - b_at;
        const int item = (int)(into >> 31 ? into / n.length() : (uint32_t)into / (uint32_t)n.length());
        const long long item_at = b_at + (long long)item * n.length();
        const int tile = item / H, h = item - tile * H;
        const int r0 = tile * RT, rows = min(RT, n.s.rows * G - r0);
        const int i0 = quotient(a.group, r0);   // the tile's first query token, and its head in the group
        const int g0 = r0 - i0 * G;
        auto token_of = [&](int r) { return quotient(a.group, g0 + r); };   // row r's query token, from i0 on
        auto out_of = [&](int r) {
            const int i = token_of(r);
            return (E*)a.o.ptr + (int64_t)(n.s.row0 + i0 + i) * a.o.row + (int64_t)(h * G + g0 + r - i * G) * a.o.head;
        };
        if (!n.units) {   // the rows see nothing
            for (int i = tid; i < rows * (D / 4); i += THREADS) {
                const int r = i / (D / 4);
                store4<E>(out_of(r) + (i - r * (D / 4)) * 4, make_float4(0.f, 0.f, 0.f, 0.f));
            }
            at = item_at + 1;
            continue;
        }
        const int u0 = (int)max(at - item_at - LEAD, 0ll), u1 = (int)(min((long long)n.length(), end - item_at) - LEAD);
        at = item_at + n.length();
        if (u1 <= u0) break;   // only the lead is in this range: the item is the next CTA's
        // positions that the tile's rows may see: row r at start + i0 + token_of(r)
        const int pos_lo = n.s.start + i0, pos_hi = pos_lo + token_of(rows - 1);
        const int seen_from = first_seen(pos_lo, a.window);
        const int ca = max(n.c0 + u0 * WARPS, seen_from / CHUNK_T);
        const int cb = min(min(n.c0 + u1 * WARPS, n.c1), pos_hi >= 0 ? pos_hi / CHUNK_T + 1 : 0);
        const int count = max(0, (cb - ca - warp + WARPS - 1) / WARPS);   // this warp's chunks: ca + warp, + WARPS, ...

        // ---- the tile's queries, a row per warp at a time: their loads first
        constexpr int EL = DP / 32;
        float x[RT / WARPS][EL];
#pragma unroll
        for (int k = 0; k < RT / WARPS; ++k) {
            const int r = warp + k * WARPS, i = token_of(r);
            const E* q = (const E*)a.q.ptr + (int64_t)(n.s.row0 + i0 + i) * a.q.row +
                         (int64_t)(h * G + g0 + r - i * G) * a.q.head + lane * EL;
            load_elements<EL>(q, r < rows && lane * EL < D, x[k]);
        }

        // ---- page ids and scales of 32 pieces, one per lane, a batch ahead
        constexpr int BATCH = 32 / SUB;   // chunks
        auto token_at = [&](int k) { return (ca + warp + k * WARPS) * CHUNK_T; };   // of this warp's chunk k
        auto id_at = [&](int k, int t) {   // nothing is read past the last token that the tile sees
            return k < count && t <= pos_hi ? load_page(a.step, c, b, quotient(a.page, t), a.status) : -1;
        };
        auto row_of = [&](int id, int t) {   // first code row of the piece; past the tensor for a bad page
            return id < 0 ? c.n_pages * H * c.page : (id * H + h) * c.page + t - quotient(a.page, t) * c.page;
        };
        const int my_k = lane / SUB, my_off = lane % SUB * PIECE;
        int id1;
        int row, row1;
        float ks, vs, ks1 = 0.f, vs1 = 0.f;
        {
            const int t = token_at(my_k) + my_off, t1 = token_at(BATCH + my_k) + my_off;
            // (nor before the first that it sees: where a window begins, in the first chunk)
            const int id = t + PIECE > seen_from ? id_at(my_k, t) : -1;
            id1 = id_at(BATCH + my_k, t1);
            row = row_of(id, t), row1 = row_of(id1, t1);
            ks = id >= 0 ? c.k_scale[(size_t)id * H + h] : 0.f;
            vs = id >= 0 ? c.v_scale[(size_t)id * H + h] : 0.f;
        }
        // copies chunk k of the item, a box per lane; `row` holds batch `batch`
        const int box = lane % (2 * CB * SUB), box_sub = box / (2 * CB), box_v = box / CB & 1, box_q = box % CB;
        auto issue = [&](int k, int batch) {
            const int r = __shfl_sync(~0u, k / BATCH == batch ? row : row1, k % BATCH * SUB + box_sub);
            const uint32_t st = issued % Sh::STAGES;
            uint64_t* bar = &tl.full[warp][st];
            if (lane == 0) mbar_expect_tx(bar, Sh::STAGE);
            __syncwarp();
            if (lane < 2 * CB * SUB)
                tma_2d(ring + st * Sh::STAGE + box_sub * Sh::PART + (box_v * CB + box_q) * Sh::BOX, box_v ? &tmV : &tmK, bar,
                       box_q * 128, r);
            ++issued;
        };
        int next = 0;   // next chunk to copy
        if (alive)
            for (; next < min(count, Sh::STAGES); ++next) issue(next, 0);

        // ---- queries as fp16 fragments
#pragma unroll
        for (int kk = 0; kk < RT / WARPS; ++kk) {
            const int r = warp + kk * WARPS;
            float top = 0.f;
            bool fine = true;
#pragma unroll
            for (int e = 0; e < EL; ++e) {
                fine &= fabsf(x[kk][e]) <= 3.402823466e38f;
                top = fmaxf(top, fabsf(x[kk][e]));
            }
            fine = __all_sync(~0u, fine);
            top = __uint_as_float(__reduce_max_sync(~0u, __float_as_uint(top)));   // (>= 0: ordered like its bits)
            // 2^-k with top 2^-k in [1/2, 1); top below 2^-100 counts as 2^-100, and one above 2^114
            // stays below 2^14 (within fp16, where a factor of 2^128 would leave fp32)
            const int k = fine ? min(max((int)(__float_as_uint(top) >> 23) - 126, -100), 114) : 0;
            const float down = __uint_as_float((uint32_t)(127 - k) << 23);
            if (lane == 0)
                tl.qf[r] = fine ? a.scale * (1.4426950408889634f * __uint_as_float((uint32_t)(127 + k) << 23)) : NAN;
#pragma unroll
            for (int e = 0; e < EL; e += 2) {
                const int d = lane * EL + e, ch = d % 128 / 16, w = d % 16 / 4;
                const int s = DP == 64 ? w : d / 128 * 8 + ch % 2 * 4 + w, t = DP == 64 ? ch : ch / 2;
                const float v0 = fine ? x[kk][e] * down : 0.f, v1 = fine ? x[kk][e + 1] * down : 0.f;
                const __half2 hi = __floats2half2_rn(v0, v1);
                uint32_t* dst = qfrag + (((s * NT + r / 8) * TERMS) * 32 + r % 8 * 4 + t) * 2 + d % 4 / 2;
                *dst = *reinterpret_cast<const uint32_t*>(&hi);
                if (TERMS == 2) {
                    const float2 f = __half22float2(hi);
                    const __half2 lo = __floats2half2_rn(v0 - f.x, v1 - f.y);
                    dst[64] = *reinterpret_cast<const uint32_t*>(&lo);
                }
            }
        }
        __syncthreads();
        uint2 qreg[KS][NT][TERMS];
        constexpr bool QREG = KS * NT * TERMS <= 16;
        auto qf_at = [&](int s, int t, int term) {
            return *reinterpret_cast<const uint2*>(qfrag + (((s * NT + t) * TERMS + term) * 32 + lane) * 2);
        };
        if (QREG)
#pragma unroll
            for (int s = 0; s < KS; ++s)
#pragma unroll
                for (int t = 0; t < NT; ++t)
#pragma unroll
                    for (int term = 0; term < TERMS; ++term) qreg[s][t][term] = qf_at(s, t, term);
        float qf[NT][2], m[NT][2], l[NT][2], o[KS][NT][4];
        int hi[NT][2];   // tokens first_seen(hi - 1) .. hi - 1 are seen
        int hi_min = 0x7fffffff, hi_max = -0x7fffffff;
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int r = t * 8 + 2 * tig + e;
                qf[t][e] = tl.qf[r];
                m[t][e] = NO_MAX;
                l[t][e] = 0.f;
                hi[t][e] = pos_lo + token_of(min(r, rows - 1)) + 1;
#pragma unroll
                for (int s = 0; s < KS; ++s) o[s][t][e] = o[s][t][2 + e] = 0.f;
            }
        hi_min = pos_lo + 1;
        hi_max = pos_hi + 1;
        const int lo_max = first_seen(pos_hi, a.window);

        // ---- this warp's chunks
        for (int k = 0; k < count && alive; ++k) {
            if (k && k % BATCH == 0) {
                row = row1, ks = ks1, vs = vs1;
                const int t = token_at(k + BATCH + my_k) + my_off;
                id1 = id_at(k + BATCH + my_k, t);
                row1 = row_of(id1, t);
            }
            if (k % BATCH == BATCH / 4) {   // the next batch's scales, well before they are used
                ks1 = id1 >= 0 ? c.k_scale[(size_t)id1 * H + h] : 0.f;
                vs1 = id1 >= 0 ? c.v_scale[(size_t)id1 * H + h] : 0.f;
            }
            float ksk[SUB], vsk[SUB];
#pragma unroll
            for (int u = 0; u < SUB; ++u) {
                ksk[u] = __shfl_sync(~0u, ks, k % BATCH * SUB + u);
                vsk[u] = __shfl_sync(~0u, vs, k % BATCH * SUB + u);
            }
            const uint32_t st = used % Sh::STAGES;
            alive = __all_sync(~0u, mbar_wait(&tl.full[warp][st], (used / Sh::STAGES) & 1, abort_flag, a.status));
            if (!alive) break;
            const uint8_t* stage = ring + st * Sh::STAGE;

            constexpr int CH = 2 / SUB;                  // independent sums per piece (even and odd k steps)
            float sc[SUB][CH][NT][4] = {};
            constexpr int J = Sh::ROWB == 128 ? 2 : 1;   // 16-byte chunks of a box row per thread
#pragma unroll
            for (int q = 0; q < CB; ++q)
#pragma unroll
                for (int j = 0; j < J; ++j)
#pragma unroll
                    for (int u = 0; u < SUB; ++u) {
                        const uint8_t* kb = stage + u * Sh::PART + q * Sh::BOX;
                        const int ch = J * tig + j;
                        const uint4 ra = *reinterpret_cast<const uint4*>(kb + swz<Sh::ROWB>(g, ch));
                        const uint4 rb = *reinterpret_cast<const uint4*>(kb + swz<Sh::ROWB>(g + 8, ch));
                        const uint32_t wa[4] = {ra.x, ra.y, ra.z, ra.w}, wb[4] = {rb.x, rb.y, rb.z, rb.w};
#pragma unroll
                        for (int w = 0; w < 4; ++w) {
                            const int s = (q * J + j) * 4 + w;
                            const uint32_t xa = wa[w] ^ 0x80808080u, xb = wb[w] ^ 0x80808080u;
                            const uint32_t a0 = minus1152(prmt(xa, 0x64646464u, 0x4140)),
                                           a1 = minus1152(prmt(xb, 0x64646464u, 0x4140)),
                                           a2 = minus1152(prmt(xa, 0x64646464u, 0x4342)),
                                           a3 = minus1152(prmt(xb, 0x64646464u, 0x4342));
#pragma unroll
                            for (int t = 0; t < NT; ++t)
#pragma unroll
                                for (int term = 0; term < TERMS; ++term) {
                                    const uint2 f = QREG ? qreg[s][t][term] : qf_at(s, t, term);
                                    mma_f16(sc[u][s % CH][t], a0, a1, a2, a3, f.x, f.y);
                                }
                        }
                    }
            // scores -> x log2 e; tokens g and g + 8 of each piece, rows 2 tig and 2 tig + 1 of each tile
            const int t0 = token_at(k);
            const bool edge = t0 + CHUNK_T > hi_min || t0 < lo_max;
            bool above = false;
            float top[NT][2];
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    top[t][e] = -INFINITY;
#pragma unroll
                    for (int u = 0; u < SUB; ++u) {
                        const float f = qf[t][e] * ksk[u];
                        float& x0 = sc[u][0][t][e];
                        float& x1 = sc[u][0][t][2 + e];
                        x0 = (CH == 2 ? x0 + sc[u][CH - 1][t][e] : x0) * f;
                        x1 = (CH == 2 ? x1 + sc[u][CH - 1][t][2 + e] : x1) * f;
                        if (edge) {
                            const int at = t0 + u * PIECE + g, from = first_seen(hi[t][e] - 1, a.window);
                            if (at >= hi[t][e] || at < from) x0 = -INFINITY;
                            if (at + 8 >= hi[t][e] || at + 8 < from) x1 = -INFINITY;
                        }
                        top[t][e] = fmaxf(top[t][e], fmaxf(x0, x1));
                    }
                    above |= top[t][e] > m[t][e] + SLACK;
                }
            if (__any_sync(~0u, above)) {
#pragma unroll
                for (int t = 0; t < NT; ++t)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        float x = top[t][e];
#pragma unroll
                        for (int d = 4; d < 32; d <<= 1) x = fmaxf(x, __shfl_xor_sync(~0u, x, d));
                        x = fmaxf(x, m[t][e]);
                        const float f = ex2(m[t][e] - x);
                        m[t][e] = x;
                        l[t][e] *= f;
#pragma unroll
                        for (int s = 0; s < KS; ++s) {
                            o[s][t][e] *= f;
                            o[s][t][2 + e] *= f;
                        }
                    }
            }
#pragma unroll
            for (int u = 0; u < SUB; ++u) {
                uint32_t p[NT][PTERMS][2];   // weights times vs as the B operand: tokens x rows
#pragma unroll
                for (int t = 0; t < NT; ++t) {
                    float w[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) w[e] = ex2(sc[u][0][t][e] - m[t][e & 1]);
                    l[t][0] += w[0] + w[2];
                    l[t][1] += w[1] + w[3];
#pragma unroll
                    for (int z = 0; z < 2; ++z) {
                        float x0 = w[2 * z] * vsk[u], x1 = w[2 * z + 1] * vsk[u];
#pragma unroll
                        for (int term = 0; term < PTERMS; ++term) {
                            const uint32_t y = bf2_of(x0, x1);
                            p[t][term][z] = transpose8(y);
                            x0 -= __uint_as_float(y << 16);
                            x1 -= __uint_as_float(y & 0xFFFF0000u);
                        }
                    }
                }
                // O^T += V^T P^T; thread's elements: 16 (DP 64: 8) adjacent ones, of tokens 2 tig, + 1, + 8, + 9
                constexpr int W = Sh::ROWB / 32;   // words of a box row per thread
#pragma unroll
                for (int q = 0; q < CB; ++q) {
                    const uint8_t* vb = stage + u * Sh::PART + (CB + q) * Sh::BOX;
                    uint32_t v[4][W];
#pragma unroll
                    for (int z = 0; z < 4; ++z) {
                        const int r = 2 * tig + (z & 1) + (z >> 1) * 8;
                        if (W == 4) {
                            const uint4 y = *reinterpret_cast<const uint4*>(vb + swz<Sh::ROWB>(r, g));
                            v[z][0] = y.x, v[z][1] = y.y, v[z][W - 2] = y.z, v[z][W - 1] = y.w;
                        } else {
                            const uint2 y = *reinterpret_cast<const uint2*>(vb + swz<Sh::ROWB>(r, g >> 1) + (g & 1) * 8);
                            v[z][0] = y.x, v[z][1] = y.y;
                        }
                    }
#pragma unroll
                    for (int w = 0; w < W; ++w) {
                        uint32_t y[2][4];   // [token pair][element of the word]
#pragma unroll
                        for (int z = 0; z < 2; ++z) {
                            const uint32_t e0 = prmt(v[2 * z][w], v[2 * z + 1][w], 0x5140),
                                           e1 = prmt(v[2 * z][w], v[2 * z + 1][w], 0x7362);
                            y[z][0] = bf16_codes(prmt(e0, 0x43434343u, 0x4140));
                            y[z][1] = bf16_codes(prmt(e0, 0x43434343u, 0x4342));
                            y[z][2] = bf16_codes(prmt(e1, 0x43434343u, 0x4140));
                            y[z][3] = bf16_codes(prmt(e1, 0x43434343u, 0x4342));
                        }
#pragma unroll
                        for (int z = 0; z < 2; ++z)
#pragma unroll
                            for (int t = 0; t < NT; ++t) {
                                float(&to)[4] = o[q * (KS / CB) + w * 2 + z][t];
                                float part[4] = {0.f, 0.f, 0.f, 0.f};
                                // fp32 rows: the tensor cores' sums drop bits, so that 16 tokens are summed
                                // there, the small terms first, and rounded into the long sum here (152
                                // sequences of 16000 tokens: error against 64 bits 7.0e-6 without, 0.9e-6
                                // with, 2.2e-6 in plain fp32; 16 x 8000 tokens, 32/8 heads: 61 and 67 us when
                                // measured, 65 us now)
#pragma unroll
                                for (int term = PTERMS - 1; term >= 0; --term)
                                    mma_bf(F32 ? part : to, y[0][2 * z], y[0][2 * z + 1], y[1][2 * z], y[1][2 * z + 1],
                                           p[t][term][0], p[t][term][1]);
                                if (F32)
#pragma unroll
                                    for (int e = 0; e < 4; ++e) to[e] += part[e];
                            }
                    }
                }
            }
            ++used;
            __syncwarp();
            if (next < count) {
                issue(next, k / BATCH);
                ++next;
            }
        }
        if (!alive)   // copies in flight land before the ring is used for anything else
            for (; used != issued; ++used) {
                const long long t0 = clock64();
                while (!mbar_try_wait(&tl.full[warp][used % Sh::STAGES], (used / Sh::STAGES) & 1) &&
                       clock64() - t0 < 200000000ll) {
                }
            }

        // ---- join the warps: rows' m and l, then O through shared memory
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
#pragma unroll
                for (int d = 4; d < 32; d <<= 1) l[t][e] += __shfl_xor_sync(~0u, l[t][e], d);
                if (g == 0) {
                    tl.m[warp][t * 8 + 2 * tig + e] = m[t][e];
                    tl.l[warp][t * 8 + 2 * tig + e] = l[t][e];
                }
            }
        __syncthreads();   // every warp is done with its ring
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int r = t * 8 + 2 * tig + e;
                float top = tl.m[0][r];
#pragma unroll
                for (int w = 1; w < WARPS; ++w) top = fmaxf(top, tl.m[w][r]);
                const float f = ex2(m[t][e] - top);
                float* dst = join + (warp * RT + r) * DP;
#pragma unroll
                for (int q = 0; q < CB; ++q) {
                    constexpr int SB = KS / CB;
                    // elements q * 128 + g * EPT + 2 s + {0, 1}; rows of 16-byte pieces rotated by the row
                    // pair so that the four tig of a quarter warp meet different banks
#pragma unroll
                    for (int s = 0; s < SB; s += 2) {
                        const int d = q * 128 + g * (2 * SB) + 2 * s;
                        float4 v = make_float4(o[q * SB + s][t][e] * f, o[q * SB + s][t][2 + e] * f,
                                               o[q * SB + s + 1][t][e] * f, o[q * SB + s + 1][t][2 + e] * f);
                        *reinterpret_cast<float4*>(dst + (d ^ (tig << 2))) = v;
                    }
                }
            }
        __syncthreads();
        const bool whole = u0 == 0 && u1 == n.units;
        const int first = whole ? cta : cta_of(item_at + LEAD), lastc = whole ? cta : cta_of(item_at + n.length() - 1);
        float* slot = partial + (size_t)(2 * cta + (u0 == 0 ? 1 : 0)) * Sh::SLOT;
        for (int i = tid; i < RT * DP / 4; i += THREADS) {
            const int r = i / (DP / 4), d = i % (DP / 4) * 4;
            float top = tl.m[0][r], sum = 0.f;
#pragma unroll
            for (int w = 1; w < WARPS; ++w) top = fmaxf(top, tl.m[w][r]);
            float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int w = 0; w < WARPS; ++w) {
                const float4 y = *reinterpret_cast<const float4*>(join + (w * RT + r) * DP + (d ^ ((r >> 1 & 3) << 2)));
                v.x += y.x, v.y += y.y, v.z += y.z, v.w += y.w;
                sum += tl.l[w][r] * ex2(tl.m[w][r] - top);
            }
            if (whole) {
                if (r < rows && d < D) {
                    const float inv = sum == 0.f ? 0.f : 1.f / sum;
                    store4<E>(out_of(r) + d, make_float4(v.x * inv, v.y * inv, v.z * inv, v.w * inv));
                }
            } else {
                *reinterpret_cast<float4*>(slot + r * DP + d) = v;
                if (d == 0) {
                    slot[RT * DP + r] = top;
                    slot[RT * DP + RT + r] = sum;
                }
            }
        }
        if (!whole) {
            // the item's CTAs first .. lastc: the last to arrive joins their slots in order
            __syncthreads();
            if (tid == 0) {   // (release and acquire for the whole CTA, around its barriers)
                int seen;
                asm volatile("atom.acq_rel.gpu.global.add.s32 %0, [%1], 1;" : "=r"(seen) : "l"(counters + first) : "memory");
                tl.last_of = seen == lastc - first;
                if (tl.last_of) counters[first] = 0;
            }
            __syncthreads();
            if (tl.last_of) {
                auto slot_of = [&](int i) { return partial + (size_t)(2 * i + (i == first ? 1 : 0)) * Sh::SLOT; };
                for (int i = tid; i < RT * DP / 4; i += THREADS) {
                    const int r = i / (DP / 4), d = i % (DP / 4) * 4;
                    if (r >= rows || d >= D) continue;
                    float top = NO_MAX;
                    for (int k = first; k <= lastc; ++k) top = fmaxf(top, __ldcg(slot_of(k) + RT * DP + r));
                    float sum = 0.f;
                    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
                    for (int k = first; k <= lastc; ++k) {
                        const float* p = slot_of(k);
                        const float f = ex2(__ldcg(p + RT * DP + r) - top);
                        const float4 y = __ldcg(reinterpret_cast<const float4*>(p + r * DP + d));
                        sum = fmaf(__ldcg(p + RT * DP + RT + r), f, sum);
                        v.x = fmaf(y.x, f, v.x), v.y = fmaf(y.y, f, v.y), v.z = fmaf(y.z, f, v.z), v.w = fmaf(y.w, f, v.w);
                    }
                    const float inv = sum == 0.f ? 0.f : 1.f / sum;
                    store4<E>(out_of(r) + d, make_float4(v.x * inv, v.y * inv, v.z * inv, v.w * inv));
                }
            }
        }
        if (at < end) {
            fence_proxy_async_smem();   // the join buffer's generic accesses before the next item's copies
            __syncthreads();
        }
    }
}

template <bool F32, int DP, int NT>
cudaError_t launch(const AttendArgs& a, const AttendWs& ws, cudaStream_t st) {
    using Sh = Shape<F32, DP, NT>;
    static_assert(Sh::SLOT <= ATTEND_SLOT, "workspace slot");
    static_assert(Sh::OCC <= ATTEND_OCC, "workspace slots");
    // ranges are cut for OCC CTAs on each SM (of 228 KB, 1 KB of it the system's per CTA)
    static_assert(Sh::OCC * (Sh::SMEM + (int)sizeof(Tail) + 1024) <= 228 * 1024, "resident CTAs");
    attend_split_kernel<F32, DP, NT><<<ws.sms * Sh::OCC, THREADS, Sh::SMEM, st>>>(ws.k16, ws.v16, a, ws.partial, ws.counters);
    return cudaGetLastError();
}

template <bool F32, int DP, int NT>
cudaError_t init() {
    return cudaFuncSetAttribute(attend_split_kernel<F32, DP, NT>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                Shape<F32, DP, NT>::SMEM);
}

}  // namespace

cudaError_t attend_split_init() {
    cudaError_t e = cudaSuccess;
    auto one = [&](cudaError_t x) { e = e == cudaSuccess ? x : e; };
    one(init<false, 64, 1>()), one(init<false, 64, 2>()), one(init<false, 128, 1>()), one(init<false, 128, 2>());
    one(init<false, 256, 1>()), one(init<false, 256, 2>());
    one(init<true, 64, 1>()), one(init<true, 64, 2>()), one(init<true, 128, 1>()), one(init<true, 128, 2>());
    one(init<true, 256, 1>()), one(init<true, 256, 2>());
    return e;
}

// Rows per tile: 8, or 16 where a sequence and head has more (past 16 only fp32 rows of more than
// 128 elements come here, in tiles of 16; the rest are attend_prompt.cu's).
template <bool F32, int DP>
static cudaError_t by_rows(const AttendArgs& a, const AttendWs& ws, cudaStream_t st) {
    const long long rows = (long long)a.step.max_new * (a.q_heads / a.pages.heads);
    return rows <= 8 ? launch<F32, DP, 1>(a, ws, st) : launch<F32, DP, 2>(a, ws, st);
}

template <bool F32>
static cudaError_t by_shape(const AttendArgs& a, const AttendWs& ws, cudaStream_t st) {
    const int D = a.pages.dim;
    return D <= 64 ? by_rows<F32, 64>(a, ws, st) : D <= 128 ? by_rows<F32, 128>(a, ws, st) : by_rows<F32, 256>(a, ws, st);
}

cudaError_t launch_attend_split(bool bf16, const AttendArgs& a, const AttendWs& ws, cudaStream_t st) {
    return bf16 ? by_shape<false>(a, ws, st) : by_shape<true>(a, ws, st);
}

}  // namespace mlora
