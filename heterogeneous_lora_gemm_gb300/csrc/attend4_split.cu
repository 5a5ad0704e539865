// Causal attention over the 4-bit cache for sequences with few rows in the step (decode: one
// token), any row and head count (include/mlora.h).
//
// Mathematics.  With values kc, vc (code times scale) and units ku, vu, row r (query token i, query
// head g of the key/value head's group) has raw scores  y_t = q_r . kc_t,  and
//     o_r = vu sum_t w_t vc_t / sum_t w_t,   w_t = 2^(f (y_t - ref) + OFF),   f = scale ku log2 e,
// with a running ref: only a lower bound of the largest y is needed, so ref moves (and the accumulators
// are rescaled) only when some f (y - ref) exceeds SLACK.  The difference is taken before the factor: near
// the row's largest it is exact, however large f y is, so that the largest weight is always
// 2^OFF to 2^(OFF + SLACK).  (As f y - (f ref - OFF) it would be off by the rounding of the latter: past a score
// of 2^24 weights left fp16 at both ends.)  ku is in `scale`, vu is taken at the end.
//
// Products run on mma.sync m16n8k16 in fp16 with fp32 sums, transposed: tokens (S^T = K Q^T) and
// head elements (O^T = V^T P^T) are the 16-row side, query rows the 8-column side, so that a group
// of up to 8 heads wastes nothing.  A code times its scale is exact in fp16 (block4.cuh), and so is
// a bf16 query that a power of two per row has brought below 1 (its elements under 2^-14 of the
// row's largest round to 2^-25 of it).  Weights have 11 bits, down to 2^-26 of the row's largest, and
// the row's sum is that of the rounded ones: an error of 0.0002 against 64 bits beside the rounded
// output's 0.0017.  fp32 rows run the same products with queries and weights as the sum of two terms
// (22 bits), and sum 16 tokens on the tensor cores, the long sum outside: those cut sums off.
//
// A warp works alone: it streams chunks of 16-token blocks, one copy each, through a private ring,
// holds its rows' queries as fragments (a lane's share of a row is 32 adjacent bytes of it, 64 where
// rows are fp32) and writes an item that is its own from registers.
// Work split: all (sequence, row tile, head) items' chunks in one line, cut into equal ranges, one
// per resident warp; every CTA finds its warps' ranges from the lengths (Shape, below: what an item's
// length is).  An item cut between warps is joined at their CTA's end,
// one cut between CTAs then by the CTA that gets there last; either in range order, so that results do
// not depend on timing.
//
// Bound: the conversions, 9 instructions per 16 codes and lane, beside HBM: 32 sequences of 32k tokens,
// 32/8 heads of 128, bf16, take 210 us, 5.7 TB/s, where the copies alone take 180 us and everything
// but the copies 195 us; of 300 instructions per block and warp 145 convert, the vector units' integer
// pipe is busy 46% of the time, half-precision 30%, mma.sync 24%.  32 of 129 to 4096 with as many key heads as
// query heads take 57 us, 4.1 TB/s, one of 777 tokens 9.0 us (13.4 under a page table for 32k: by_rows below): a CTA's
// start, a range's loads, a join.
//
// What measured slower (32 sequences of 32k): weights in two terms, 22 bits, for bf16 rows as well (248 us, the 57 us
// above 66; the error stays 0.0017), as bf16 with bf16 values 347 us;
// a chunk's scores taken with the last one's values (233 against 230 at the time); four CTAs per SM
// (233), two (270); a CTA per range, its warps in turns over the chunks, joined per item (221 us, and
// 50 against 39 us for 81 sequences of 194 tokens, 64/32 heads, fp32); parts joined through global memory
// alone (215 us, one short sequence 17 us).
#include <cuda_fp16.h>

#include <type_traits>

#include "attend.h"
#include "attend_mma.cuh"
#include "block4.cuh"
#include "f32x2.cuh"
#include "tc_ptx.cuh"

namespace mlora {

using namespace ptx;

namespace {

constexpr int WARPS = 4, THREADS = 32 * WARPS;
constexpr int PIECE = 16;                 // tokens of a block and of a product
// ref is the largest y when it is set, of weight 2^OFF, and moves when one's weight would exceed 2^(OFF + SLACK):
// weights stay below 2^15, within fp16, and their 11 bits reach down to 2^-26 of the largest
constexpr float OFF = 12.f, SLACK = 3.f;
// Items of up to this length are taken by a CTA each where CTAs are left over (8 key heads of 200 tokens, 8
// long, 8.0 us, cut between CTAs 8.8; of 400 tokens, 16 long, 9.7 and 9.1 us)
constexpr int ALONE = 2 * WARPS;
// ref before anything is seen: far below any score, finite (-inf less it stays -inf), and so that the bound set
// from it (SLACK / f is 2.6e38 at the most) lies below any score as well
constexpr float NO_MAX = -3e38f;
constexpr int EXTRA = 3;                  // of a partial result beside O, per row: ref, the weights' sum, f

template <bool F32, int DP, int NT, bool LONG>
struct Shape {
    static constexpr int TERMS = F32 ? 2 : 1;          // of a query and of a weight
    static constexpr int KS = DP / 16;                 // k steps of q . k = 16-row tiles of O^T
    static constexpr int RT = 8 * NT;                  // query rows per tile
    static constexpr int CB = DP == 256 ? 2 : 1;       // 128-element units of values
    static constexpr int W = DP == 64 ? 2 : 4;         // words of four elements per lane and unit
    // CTAs per SM: three where the accumulators of 8 rows leave the registers, else two
    static constexpr int OCC = !F32 && DP <= 128 && NT == 1 ? 3 : 2;
    // pieces that a warp takes at a time: waits, votes and issues are per chunk.  (32 sequences of 32k tokens
    // 210 us with four, 226 us with two; one sequence of 777 tokens 13.4 and 9.0 us)
    static constexpr int SUB = DP == 256 ? 1 : LONG ? 4 : 2;
    static_assert(!LONG || OCC == 3, "long ranges");
    static constexpr int CHUNK_T = PIECE * SUB;
    static constexpr int PART = 18 * DP;               // bytes of a piece
    static constexpr int STAGE = SUB * PART;
    // query fragments: in registers where they are few, else a lane's own words of shared memory
    static constexpr int QUERY = KS * NT * TERMS * 256;    // bytes per warp
    static constexpr bool QREG = QUERY <= 16 * 256;
    static constexpr int ROOM = (228 * 1024 / OCC - 3 * 1024) / WARPS - (QREG ? 0 : QUERY);
    static constexpr int STAGES = ROOM / STAGE < 8 ? ROOM / STAGE : 8;
    static constexpr int OWN = STAGES * STAGE + (QREG ? 0 : QUERY);   // of a warp: ring, fragments
    static_assert(STAGES >= 2 && OWN >= RT * (DP + EXTRA) * 4, "ring; a partial result in its place");
    static constexpr int SMEM = 128 + WARPS * OWN;
    static constexpr int SLOT = RT * (DP + EXTRA);     // floats of a partial result: O, then ref, l, f per row
    // How the line is cut.  Long ranges: starting an item costs as much as LEAD chunks, and a range has at least
    // LEAST.  Short ones: an item of more than one chunk is brought to a multiple of WARPS, so that the CTAs'
    // ranges begin where items do as far as can be; every end of one inside an item is a join more.  (8 key heads
    // of 777 tokens 9.0 us, 10.3 us with starts of a chunk; of 100 tokens 7.5 and 10.5 us)
    static constexpr int LEAD = LONG ? 2 : 0, LEAST = LONG ? 2 : 1;
};

// A sequence's share of the work line: tiles x heads items, each lead + units long (1 where the
// rows see nothing: zeros are written).
struct Line {
    SeqRec s;
    int c0;           // first chunk that its rows see
    int tiles, units; // row tiles, chunks per item
    int length;       // 1 where the rows see nothing: zeros are written
    __device__ long long total(int heads) const { return (long long)tiles * heads * length; }
};
template <typename Sh>
__device__ __forceinline__ Line line_of(const AttendArgs& a, int G, int b) {
    constexpr int RT = Sh::RT, CHUNK_T = Sh::CHUNK_T;
    Line n;
    n.s = load_seq(a.step, a.pages.page, b, a.status);
    const int last = n.s.start + n.s.rows - 1;   // position of the last processed row
    n.c0 = first_seen(n.s.start, a.window) / CHUNK_T;
    n.tiles = (n.s.rows * G + RT - 1) / RT;
    n.units = last >= 0 ? last / CHUNK_T + 1 - n.c0 : 0;
    n.length = n.units == 0 ? 1 : Sh::LEAD ? Sh::LEAD + n.units : n.units == 1 ? 1 : (n.units + WARPS - 1) / WARPS * WARPS;
    return n;
}

// What a warp has of an item that it does not have whole: at most the item its range begins in, and
// the one that it ends in.
struct Part {
    long long item_at;     // the item's place on the line
    const float* slot;
    int length;            // of the item
    int row, g0, h, rows;  // its rows: first output row and head in the group, key head, how many
};
struct Tail {
    uint64_t full[WARPS][8];
    long long scan[WARPS], first_at[WARPS];
    int longest[WARPS];
    Part parts[WARPS][2];
    int first_b[WARPS], count[WARPS], order[2 * WARPS + 1];
    int abort_flag, last_of;
};

__device__ __forceinline__ float reciprocal(float x) {   // to 2^-22; 0 past 2^126
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// 16 adjacent elements as floats, zeros unless `there`
__device__ __forceinline__ void load16(const float* p, bool there, float* x) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float4 v = there ? reinterpret_cast<const float4*>(p)[i] : make_float4(0.f, 0.f, 0.f, 0.f);
        x[4 * i] = v.x, x[4 * i + 1] = v.y, x[4 * i + 2] = v.z, x[4 * i + 3] = v.w;
    }
}
__device__ __forceinline__ void load16(const __nv_bfloat16* p, bool there, float* x) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const uint4 v = there ? reinterpret_cast<const uint4*>(p)[i] : make_uint4(0u, 0u, 0u, 0u);
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            x[8 * i + 2 * k] = __uint_as_float(w[k] << 16);
            x[8 * i + 2 * k + 1] = __uint_as_float(w[k] & 0xFFFF0000u);
        }
    }
}

// `zeros`: a block of zeros, in the place of one that cannot be read.  FULL: heads of DP elements, so
// that a block's offsets are constants.
template <bool F32, int DP, int NT, bool LONG, bool FULL>
__global__ void __launch_bounds__(THREADS, (Shape<F32, DP, NT, LONG>::OCC))
attend4_split_kernel(const AttendArgs a, float* __restrict__ partial, int* __restrict__ counters, const uint8_t* __restrict__ zeros) {
    using Sh = Shape<F32, DP, NT, LONG>;
    using E = typename std::conditional<F32, float, __nv_bfloat16>::type;
    constexpr int KS = Sh::KS, RT = Sh::RT, SUB = Sh::SUB, CHUNK_T = Sh::CHUNK_T, TERMS = Sh::TERMS, CB = Sh::CB, W = Sh::W;
    extern __shared__ __align__(128) uint8_t smem4[];
    uint8_t* smem = (uint8_t*)(((uintptr_t)smem4 + 127) & ~(uintptr_t)127);
    __shared__ Tail tl;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, tig = lane & 3;
    const CachePages& c = a.pages;
    const int H = c.heads, G = a.q_heads / H, D = FULL ? DP : c.dim, groups = D / 16;
    const int bytes = block4_bytes(D);

    // ---- this warp's range of the line
    if (lane == 0) {
        for (int s = 0; s < Sh::STAGES; ++s) mbar_init(&tl.full[warp][s], SUB);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (tid == 0) tl.abort_flag = 0;
    const int per = (a.step.n_seqs + THREADS - 1) / THREADS;
    const int b_lo = min(tid * per, a.step.n_seqs), b_hi = min(b_lo + per, a.step.n_seqs);
    long long mine = 0;
    int longest = 0;   // item
    for (int b = b_lo; b < b_hi; ++b) {
        const Line n = line_of<Sh>(a, G, b);
        mine += n.total(H);
        longest = max(longest, n.length);
    }
    if (!LONG) longest = __reduce_max_sync(~0u, longest);
    long long incl = mine;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const long long v = __shfl_up_sync(~0u, incl, d);
        if (lane >= d) incl += v;
    }
    if (lane == 31) {
        tl.scan[warp] = incl;
        if (!LONG) tl.longest[warp] = longest;
    }
    __syncthreads();
    long long total = 0, before = 0;
#pragma unroll
    for (int w = 0; w < WARPS; ++w) {
        if (w < warp) before += tl.scan[w];
        total += tl.scan[w];
        if (!LONG) longest = max(longest, tl.longest[w]);
    }
    before += incl - mine;
    const int all = gridDim.x * WARPS;
    const int least = !LONG && longest > WARPS && longest <= ALONE ? longest / WARPS : Sh::LEAST;
    const int workers = total >= (long long)least * all ? all : (int)((total + least - 1) / least);
    const int cta = blockIdx.x, worker = cta * WARPS + warp;
    if (cta * WARPS >= workers) return;
    // ranges: the first `over` of them one longer than the others
    const long long each = total >> 31 ? total / workers : (uint32_t)total / (uint32_t)workers;
    const int over = (int)(total - each * workers);
    auto range_at = [&](int i) { return each * i + min(i, over); };
    auto worker_of = [&](long long u) {   // the one whose range holds position u
        const long long mark = (each + 1) * over, v = u < mark ? u : u - mark, w = u < mark ? each + 1 : each;
        return (u < mark ? 0 : over) + (int)(total >> 31 ? v / w : (uint32_t)v / (uint32_t)w);
    };
#pragma unroll 1
    for (int w = 0; w < WARPS; ++w) {   // where each of the CTA's ranges begins
        const int i = cta * WARPS + w;
        const long long from = range_at(i);
        if (i >= workers || from < before || from >= before + mine) continue;
        long long p = before;
        int b = b_lo;
        for (; per > 1 && b < b_hi - 1; ++b) {
            const long long length = line_of<Sh>(a, G, b).total(H);
            if (from < p + length) break;
            p += length;
        }
        tl.first_b[w] = b;
        tl.first_at[w] = p;
    }
    __syncthreads();
    const bool works = worker < workers;
    long long at = works ? range_at(worker) : 0;
    const long long end = works ? range_at(worker + 1) : 0;
    int b = works ? tl.first_b[warp] : 0;
    long long b_at = works ? tl.first_at[warp] : 0;   // where sequence b begins on the line
    Line n = line_of<Sh>(a, G, b);
    int parts = 0;

    uint8_t* ring = smem + warp * Sh::OWN;
    uint2* query = reinterpret_cast<uint2*>(ring + Sh::STAGES * Sh::STAGE);
    volatile int* abort_flag = &tl.abort_flag;
    uint32_t fill = 0, drain = 0, turn = 0;   // stages to copy to and to consume, and the latter's phase
    int flying = 0;                           // chunks copied and not consumed
    bool alive = true;

    while (at < end) {
        while (at >= b_at + n.total(H)) {
            b_at += n.total(H);
            n = line_of<Sh>(a, G, ++b);
        }
        const long long into = at - b_at;
        const int item = (int)(into >> 31 ? into / n.length : (uint32_t)into / (uint32_t)n.length);
        const long long item_at = b_at + (long long)item * n.length;
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
            for (int i = lane; i < rows * (D / 4); i += 32) {
                const int r = i / (D / 4);
                store4<E>(out_of(r) + (i - r * (D / 4)) * 4, make_float4(0.f, 0.f, 0.f, 0.f));
            }
            at = item_at + 1;
            continue;
        }
        const int u0 = (int)max(at - item_at - Sh::LEAD, 0ll), u1 = (int)(min((long long)n.length, end - item_at) - Sh::LEAD);
        at = item_at + n.length;
        if (u1 <= u0) break;   // only the lead is in this range: the item is the next warp's
        // positions that the tile's rows may see: row r at start + i0 + token_of(r)
        const int pos_lo = n.s.start + i0, pos_hi = pos_lo + token_of(rows - 1);
        const int seen_from = first_seen(pos_lo, a.window);
        const int ca = max(n.c0 + u0, seen_from / CHUNK_T);
        const int cb = min(n.c0 + u1, pos_hi >= 0 ? pos_hi / CHUNK_T + 1 : 0);
        const int count = max(0, cb - ca);   // this warp's chunks: ca, ca + 1, ...

        // ---- pages of 32 blocks, one per lane, a batch ahead
        constexpr int BATCH = 32 / SUB;   // chunks
        const int my_k = lane / SUB, my_off = lane % SUB * PIECE;
        auto block_at = [&](int k) {   // of this lane's piece of chunk k, -1 for a bad page; nothing is read
                                       // past the last token that the tile sees, or before the first
            const int t = (ca + k) * CHUNK_T + my_off;
            if (k >= count || t > pos_hi || t + PIECE <= seen_from) return -1;
            const int j = quotient(a.page, t), id = load_page(a.step, c, b, j, a.status);
            return id < 0 ? -1 : (id * H + h) * (c.page >> 4) + ((t - j * c.page) >> 4);
        };
        int block = block_at(my_k), block1 = block_at(BATCH + my_k);
        // copies chunk k of the item, a block by the lane that looked its page up; `block` holds batch `batch`
        auto issue = [&](int k, int batch) {
            if (lane / SUB == k % BATCH) {
                const int r = k / BATCH == batch ? block : block1;
                uint64_t* bar = &tl.full[warp][fill];
                mbar_expect_tx(bar, bytes);
                bulk_g2s(ring + fill * Sh::STAGE + lane % SUB * Sh::PART, r < 0 ? zeros : c.blocks + (size_t)(uint32_t)r * (uint32_t)bytes,
                         bytes, bar);
            }
            fill = fill + 1 == Sh::STAGES ? 0 : fill + 1;
            ++flying;
        };

        // ---- the tile's queries: a lane holds, of row g (and 8 + g), 16 elements in each 64.  K step s takes
        // of them the pairs (x, x + 4): codes that lie in one nibble of a word's halves, the even ones over 16
        uint2 qreg[Sh::QREG ? KS : 1][NT][TERMS];
        float factor[NT];
        int next = 0;   // next chunk to copy
        {
            float x[NT][DP / 64][16];
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                const int r = t * 8 + g, i = token_of(min(r, rows - 1));
                const E* q = (const E*)a.q.ptr + (int64_t)(n.s.row0 + i0 + i) * a.q.row + (int64_t)(h * G + g0 + min(r, rows - 1) - i * G) * a.q.head;
#pragma unroll
                for (int u = 0; u < DP / 64; ++u) load16(q + u * 64 + tig * 16, r < rows && (FULL || u * 4 + tig < groups), x[t][u]);
            }
            if (alive)
                for (; next < min(count, Sh::STAGES); ++next) issue(next, 0);
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                float top = 0.f;
                bool fine = true;
#pragma unroll
                for (int u = 0; u < DP / 64; ++u)
#pragma unroll
                    for (int e = 0; e < 16; ++e) {
                        fine &= fabsf(x[t][u][e]) <= 3.402823466e38f;
                        top = fmaxf(top, fabsf(x[t][u][e]));
                    }
                top = fine ? top : INFINITY;
#pragma unroll
                for (int d = 1; d < 4; d <<= 1) top = fmaxf(top, __shfl_xor_sync(~0u, top, d));
                fine = top <= 3.402823466e38f;
                // 2^-k with top 2^-k in [1/2, 1); top below 2^-100 counts as 2^-100, and one above 2^118 stays
                // below 2^10 (16 times it within fp16, where a factor of 2^128 would leave fp32)
                const int k = fine ? min(max((int)(__float_as_uint(top) >> 23) - 126, -100), 118) : 0;
                const float down = fine ? __uint_as_float((uint32_t)(127 - k) << 23) : 0.f;
                const float f = a.scale * (1.4426950408889634f * __uint_as_float((uint32_t)(127 + k) << 23));
                factor[t] = fine ? fminf(fmaxf(f, 0x1p-126f), 0x1.fffffep127f) : NAN;   // (-inf times it stays -inf, 0 times it 0)
#pragma unroll
                for (int u = 0; u < DP / 64; ++u)
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        float v[2][2];
#pragma unroll
                        for (int z = 0; z < 2; ++z)
#pragma unroll
                            for (int y = 0; y < 2; ++y) {
                                const float e = x[t][u][j / 2 * 8 + j % 2 * 2 + z + 4 * y];
                                v[z][y] = fine ? e * down * (z ? 1.f : 16.f) : 0.f;
                            }
#pragma unroll
                        for (int term = 0; term < TERMS; ++term) {
                            uint32_t w[2];
#pragma unroll
                            for (int z = 0; z < 2; ++z) {
                                const __half2 y = __floats2half2_rn(v[z][0], v[z][1]);
                                w[z] = *reinterpret_cast<const uint32_t*>(&y);
                                const float2 back = __half22float2(y);
                                v[z][0] -= back.x, v[z][1] -= back.y;
                            }
                            if (Sh::QREG) qreg[u * 4 + j][t][term] = make_uint2(w[0], w[1]);
                            else query[(((u * 4 + j) * NT + t) * TERMS + term) * 32 + lane] = make_uint2(w[0], w[1]);
                        }
                    }
            }
        }
        float qf[NT][2], ref[NT][2], l[NT][2], bound[NT][2], sum[NT][4], o[KS][NT][4];
        int hi[NT][2];   // tokens first_seen(hi - 1) .. hi - 1 are seen
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                ref[t][e] = NO_MAX;
                bound[t][e] = NO_MAX;   // ref + SLACK / qf, or a little less
                l[t][e] = sum[t][e] = sum[t][2 + e] = 0.f;
                hi[t][e] = pos_lo + token_of(min(t * 8 + 2 * tig + e, rows - 1)) + 1;
                // (a row that sees nothing may hold anything: its factor would make masked scores NaN)
                const float f = __shfl_sync(~0u, factor[t], (2 * tig + e) * 4);
                qf[t][e] = hi[t][e] > 0 ? f : 1.f;
#pragma unroll
                for (int s = 0; s < KS; ++s) o[s][t][e] = o[s][t][2 + e] = 0.f;
            }
        const int hi_min = pos_lo + 1, lo_max = first_seen(pos_hi, a.window);

        // ---- this warp's chunks
        for (int k = 0; k < count && alive; ++k) {
            if (k && k % BATCH == 0) {
                block = block1;
                block1 = block_at(k + BATCH + my_k);
            }
            alive = __all_sync(~0u, mbar_wait(&tl.full[warp][drain], turn, abort_flag, a.status));
            if (!alive) break;
            const uint8_t* stage = ring + drain * Sh::STAGE;
            drain = drain + 1 == Sh::STAGES ? 0 : drain + 1;
            turn ^= drain == 0;

            // a lane's two atoms of a block and their scales (zeros where the head has no such group)
            auto atoms_at = [&](const uint8_t* codes, const uint8_t* scales, int at, bool there, uint4& w, uint32_t& s16) {
                w = make_uint4(0u, 0u, 0u, 0u);
                s16 = 0u;
                if (FULL || there) {
                    w = *reinterpret_cast<const uint4*>(codes + at * 8);
                    s16 = *reinterpret_cast<const uint16_t*>(scales + at);
                }
            };
            // scores of tokens g and g + 8 of each piece, rows 2 tig and 2 tig + 1 of each tile: 64 elements at
            // a time, the lane's atoms of the two tokens, group tig of the four
            constexpr int CH = SUB == 1 ? 2 : 1;   // independent sums per piece (even and odd k steps)
            float sc[SUB][CH][NT][4] = {};
#pragma unroll
            for (int q = 0; q < DP / 64; ++q)
#pragma unroll
                for (int u = 0; u < SUB; ++u) {
                    const uint8_t* kb = stage + u * Sh::PART;
                    const int n = min(4, groups - 4 * q);
                    uint4 w;
                    uint32_t s16;
                    atoms_at(kb, kb + 16 * D, q * 64 + (g * n + tig) * 2, tig < n, w, s16);
                    const Scale3 sa = scale_f16(__byte_perm(s16, 0u, 0x4040)), sb = scale_f16(__byte_perm(s16, 0u, 0x4141));
                    auto step = [&](int s, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3) {
#pragma unroll
                        for (int t = 0; t < NT; ++t)
#pragma unroll
                            for (int term = 0; term < TERMS; ++term) {
                                const uint2 f = Sh::QREG ? qreg[Sh::QREG ? s : 0][t][term] : query[((s * NT + t) * TERMS + term) * 32 + lane];
                                mma_f16(sc[u][s % CH][t], a0, a1, a2, a3, f.x, f.y);
                            }
                    };
                    step(4 * q, codes_f16<0>(w.x, sa), codes_f16<0>(w.z, sb), codes_f16<1>(w.x, sa), codes_f16<1>(w.z, sb));
                    step(4 * q + 1, codes_f16<2>(w.x, sa), codes_f16<2>(w.z, sb), codes_f16<3>(w.x, sa), codes_f16<3>(w.z, sb));
                    step(4 * q + 2, codes_f16<0>(w.y, sa), codes_f16<0>(w.w, sb), codes_f16<1>(w.y, sa), codes_f16<1>(w.w, sb));
                    step(4 * q + 3, codes_f16<2>(w.y, sa), codes_f16<2>(w.w, sb), codes_f16<3>(w.y, sa), codes_f16<3>(w.w, sb));
                }
            // the largest score itself, against the bound
            const int t0 = (ca + k) * CHUNK_T;
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
                        float& x0 = sc[u][0][t][e];
                        float& x1 = sc[u][0][t][2 + e];
                        if (CH == 2) x0 += sc[u][CH - 1][t][e], x1 += sc[u][CH - 1][t][2 + e];
                        if (edge) {
                            const int at = t0 + u * PIECE + g, from = first_seen(hi[t][e] - 1, a.window);
                            if (at >= hi[t][e] || at < from) x0 = -INFINITY;
                            if (at + 8 >= hi[t][e] || at + 8 < from) x1 = -INFINITY;
                        }
                        top[t][e] = fmaxf(top[t][e], fmaxf(x0, x1));
                    }
                    above |= top[t][e] > bound[t][e];
                }
            if (__any_sync(~0u, above)) {
#pragma unroll
                for (int t = 0; t < NT; ++t)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        float x = top[t][e];
#pragma unroll
                        for (int d = 4; d < 32; d <<= 1) x = fmaxf(x, __shfl_xor_sync(~0u, x, d));
                        x = fmaxf(x, ref[t][e]);
                        const float f = ex2((ref[t][e] - x) * qf[t][e]);
                        ref[t][e] = x;
                        bound[t][e] = __fadd_rd(x, SLACK * 0.9999f * reciprocal(qf[t][e]));
                        sum[t][e] *= f;
                        l[t][e] *= f;
#pragma unroll
                        for (int s = 0; s < KS; ++s) {
                            o[s][t][e] *= f;
                            o[s][t][2 + e] *= f;
                        }
                    }
            }
            constexpr uint32_t ONES = 0x3C003C00u;
#pragma unroll
            for (int u = 0; u < SUB; ++u) {
                uint32_t p[NT][TERMS][2];   // weights as the B operand: tokens x rows
#pragma unroll
                for (int t = 0; t < NT; ++t) {
#pragma unroll
                    for (int z = 0; z < 2; ++z) {
                        const float2 x = unpair(fma2(add2(pair(sc[u][0][t][2 * z], sc[u][0][t][2 * z + 1]), pair(-ref[t][0], -ref[t][1])),
                                                     pair(qf[t][0], qf[t][1]), pair(OFF, OFF)));
                        const float w0 = ex2(x.x), w1 = ex2(x.y);
                        const __half2 y = __floats2half2_rn(w0, w1);
                        p[t][0][z] = transpose8(*reinterpret_cast<const uint32_t*>(&y));
                        if (F32) {
                            const float2 f = __half22float2(y);
                            const __half2 low = __floats2half2_rn(w0 - f.x, w1 - f.y);
                            p[t][TERMS - 1][z] = transpose8(*reinterpret_cast<const uint32_t*>(&low));
                            l[t][0] += w0;
                            l[t][1] += w1;
                        }
                    }
                    // bf16 rows: the sum of all tokens' weights, in every row of the result
                    if (!F32) mma_f16(sum[t], ONES, ONES, ONES, ONES, p[t][0][0], p[t][0][1]);
                }
                // O^T += V^T P^T; a lane's elements: 16 (DP 64: 8) adjacent ones of each 128
#pragma unroll
                for (int q = 0; q < CB; ++q) {
                    // atoms of tokens 2 tig and + 1, + 8 and + 9, of the lane's group (DP 64: half a group), as words
                    // of four elements, token 2 tig in the low half
                    const uint8_t* vb = stage + u * Sh::PART + 8 * D;
                    const int n = min(8, groups - 8 * q), gr = DP == 64 ? g >> 1 : g;
                    uint32_t v[2][W];
                    Scale3 vs[2];
#pragma unroll
                    for (int z = 0; z < 2; ++z) {
                        uint4 w;
                        uint32_t s16;
                        atoms_at(vb, vb + 9 * D, q * 128 + (z * n + gr) * 8 + tig * 2, gr < n, w, s16);
                        vs[z] = scale_f16(__byte_perm(s16 & 0x7F7Fu, 0u, 0x4140));
                        const uint32_t lo = DP == 64 && (g & 1) ? w.y : w.x, hi = DP == 64 && (g & 1) ? w.w : w.z;
                        v[z][0] = __byte_perm(lo, hi, 0x5410), v[z][1] = __byte_perm(lo, hi, 0x7632);
                        if (W == 4) v[z][W - 2] = __byte_perm(w.y, w.w, 0x5410), v[z][W - 1] = __byte_perm(w.y, w.w, 0x7632);
                    }
#pragma unroll
                    for (int w = 0; w < W; ++w) {
                        auto values = [&](int z, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3) {
#pragma unroll
                            for (int t = 0; t < NT; ++t) {
                                float(&to)[4] = o[q * (KS / CB) + w * 2 + z][t];
                                if (!F32) {
                                    mma_f16(to, a0, a1, a2, a3, p[t][0][0], p[t][0][1]);
                                    continue;
                                }
                                // fp32 rows: the tensor cores' sums drop bits, so that 16 tokens are summed there, the
                                // small term first, and rounded into the long sum here
                                float part[4] = {0.f, 0.f, 0.f, 0.f};
                                mma_f16(part, a0, a1, a2, a3, p[t][TERMS - 1][0], p[t][TERMS - 1][1]);
                                mma_f16(part, a0, a1, a2, a3, p[t][0][0], p[t][0][1]);
#pragma unroll
                                for (int e = 0; e < 4; ++e) to[e] += part[e];
                            }
                        };
                        values(0, codes_f16<0>(v[0][w], vs[0]), codes_f16<1>(v[0][w], vs[0]), codes_f16<0>(v[1][w], vs[1]),
                               codes_f16<1>(v[1][w], vs[1]));
                        values(1, codes_f16<2>(v[0][w], vs[0]), codes_f16<3>(v[0][w], vs[0]), codes_f16<2>(v[1][w], vs[1]),
                               codes_f16<3>(v[1][w], vs[1]));
                    }
                }
            }
            --flying;
            __syncwarp();
            if (next < count) {
                issue(next, k / BATCH);
                ++next;
            }
        }

        // ---- the rows: a lane holds 16 (DP 64: 8) adjacent elements in each 128, the even ones over 16
        constexpr int EPL = 2 * KS / CB;   // elements per lane and unit
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                if (!F32) l[t][e] = sum[t][e];
                else
#pragma unroll
                    for (int d = 4; d < 32; d <<= 1) l[t][e] += __shfl_xor_sync(~0u, l[t][e], d);
            }
        // row r's elements 4 i .. of the lane's in unit q, times f
        auto four = [&](int t, int e, int q, int i, float f) {
            const int s = q * (KS / CB) + 2 * i;
            return make_float4(o[s][t][e] * 16.f * f, o[s][t][2 + e] * f, o[s + 1][t][e] * 16.f * f, o[s + 1][t][2 + e] * f);
        };
        auto put_row = [&](int t, int e, float f) {
            const int r = t * 8 + 2 * tig + e;
            if (r >= rows) return;
            E* to = out_of(r);
#pragma unroll
            for (int q = 0; q < CB; ++q) {
                const int d = q * 128 + g * EPL;
                if (!FULL && d >= D) continue;
#pragma unroll
                for (int i = 0; i < EPL / 4; i += F32 ? 1 : 2) {
                    const float4 x = four(t, e, q, i, f);
                    if (F32) store4<E>(to + d + 4 * i, x);
                    else {
                        const float4 y = four(t, e, q, i + 1, f);
                        *reinterpret_cast<uint4*>(to + d + 4 * i) = make_uint4(bf2_of(x.x, x.y), bf2_of(x.z, x.w), bf2_of(y.x, y.y), bf2_of(y.z, y.w));
                    }
                }
            }
        };
        if (u0 == 0 && u1 == n.length - Sh::LEAD) {
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
                for (int e = 0; e < 2; ++e) put_row(t, e, l[t][e] == 0.f ? 0.f : c.v_unit / l[t][e]);
            continue;
        }
        // (into the warp's ring where nothing more of the range comes: every copy has been consumed)
        float* slot = at >= end ? reinterpret_cast<float*>(ring) : partial + (size_t)worker * Sh::SLOT;
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int r = t * 8 + 2 * tig + e;
#pragma unroll
                for (int q = 0; q < CB; ++q)
#pragma unroll
                    for (int i = 0; i < EPL / 4; ++i)
                        *reinterpret_cast<float4*>(slot + r * DP + q * 128 + g * EPL + 4 * i) = four(t, e, q, i, 1.f);
                if (g == 0) {
                    slot[RT * DP + r] = ref[t][e];
                    slot[RT * DP + RT + r] = l[t][e];
                    slot[RT * DP + 2 * RT + r] = qf[t][e];
                }
            }
        if (lane == 0) tl.parts[warp][parts] = Part{item_at, slot, n.length, n.s.row0 + i0, g0, h, rows};
        ++parts;
    }
    // copies in flight land before the warp goes
    for (; flying > 0; --flying) {
        const long long t0 = clock64();
        while (!mbar_try_wait(&tl.full[warp][drain], turn) && clock64() - t0 < 200000000ll) {
        }
        drain = drain + 1 == Sh::STAGES ? 0 : drain + 1;
        turn ^= drain == 0;
    }
    if (lane == 0) tl.count[warp] = parts;
    __syncthreads();

    // ---- the CTA's parts, in range order: those of one item stand together
    if (tid == 0) {
        int i = 0;
        for (int w = 0; w < WARPS; ++w)
            for (int z = 0; z < tl.count[w]; ++z) tl.order[i++] = 2 * w + z;
        tl.order[i] = -1;
    }
    __syncthreads();
    auto part = [&](int i) -> const Part& { return tl.parts[tl.order[i] >> 1][tl.order[i] & 1]; };
    // joins slots slot_at(0 .. k - 1), a batch of loads at a time: rows of item p, or (`to`) a slot again
    auto join = [&](auto batch, const Part& p, int k, auto slot_at, float* to) {
        constexpr int BATCH = decltype(batch)::value;
        for (int i = tid; i < RT * DP / 4; i += THREADS) {
            const int r = i / (DP / 4), d = i % (DP / 4) * 4;
            if (!to && (r >= p.rows || d >= D)) continue;
            float top = NO_MAX, total = 0.f, factor;
            float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
            asm volatile("ld.relaxed.gpu.f32 %0, [%1];" : "=f"(factor) : "l"(slot_at(0) + RT * DP + 2 * RT + r) : "memory");
            for (int z0 = 0; z0 < k; z0 += BATCH) {
                float mz[BATCH], lz[BATCH];
                float4 y[BATCH];
#pragma unroll
                for (int z = 0; z < BATCH; ++z) {
                    mz[z] = NO_MAX, lz[z] = 0.f;
                    y[z] = make_float4(0.f, 0.f, 0.f, 0.f);
                    if (z0 + z < k) {   // (other threads' results, of this CTA or another)
                        const float* from = slot_at(z0 + z);
                        asm volatile("ld.relaxed.gpu.f32 %0, [%1];" : "=f"(mz[z]) : "l"(from + RT * DP + r) : "memory");
                        asm volatile("ld.relaxed.gpu.f32 %0, [%1];" : "=f"(lz[z]) : "l"(from + RT * DP + RT + r) : "memory");
                        asm volatile("ld.relaxed.gpu.v4.f32 {%0, %1, %2, %3}, [%4];"
                                     : "=f"(y[z].x), "=f"(y[z].y), "=f"(y[z].z), "=f"(y[z].w)
                                     : "l"(from + r * DP + d)
                                     : "memory");
                    }
                }
                float now = top;
#pragma unroll
                for (int z = 0; z < BATCH; ++z) now = fmaxf(now, mz[z]);
                const float f = ex2((top - now) * factor);
                top = now;
                total *= f, v.x *= f, v.y *= f, v.z *= f, v.w *= f;
#pragma unroll
                for (int z = 0; z < BATCH; ++z) {
                    const float w = ex2((mz[z] - now) * factor);   // (times 0 where there is none)
                    total = fmaf(lz[z], w, total);
                    v.x = fmaf(y[z].x, w, v.x), v.y = fmaf(y[z].y, w, v.y), v.z = fmaf(y[z].z, w, v.z), v.w = fmaf(y[z].w, w, v.w);
                }
            }
            if (to) {
                *reinterpret_cast<float4*>(to + r * DP + d) = v;
                if (d == 0) {
                    to[RT * DP + r] = top;
                    to[RT * DP + RT + r] = total;
                    to[RT * DP + 2 * RT + r] = factor;
                }
            } else {
                const float inv = total == 0.f ? 0.f : c.v_unit / total;
                const int token = quotient(a.group, p.g0 + r);
                E* row = (E*)a.o.ptr + (int64_t)(p.row + token) * a.o.row + (int64_t)(p.h * G + p.g0 + r - token * G) * a.o.head;
                store4<E>(row + d, make_float4(v.x * inv, v.y * inv, v.z * inv, v.w * inv));
            }
        }
    };
#pragma unroll 1
    for (int i = 0; tl.order[i] >= 0;) {
        const Part p = part(i);
        int k = 1;
        while (tl.order[i + k] >= 0 && part(i + k).item_at == p.item_at) ++k;
        auto warp_slot = [&](int z) { return part(i + z).slot; };
        // the item's CTAs first .. last
        const int first = worker_of(p.item_at + Sh::LEAD) / WARPS, last = worker_of(p.item_at + p.length - 1) / WARPS;
        using Warps = std::integral_constant<int, WARPS>;
        if (first == last) join(Warps(), p, k, warp_slot, nullptr);
        else {
            auto cta_slot = [&](int z) { return partial + (size_t)(all + 2 * (first + z) + (z == 0 ? 1 : 0)) * Sh::SLOT; };
            join(Warps(), p, k, warp_slot, cta_slot(cta - first));
            __syncthreads();
            if (tid == 0) {   // (release and acquire for the whole CTA, around its barriers)
                int seen;
                asm volatile("atom.acq_rel.gpu.global.add.s32 %0, [%1], 1;" : "=r"(seen) : "l"(counters + first) : "memory");
                tl.last_of = seen == last - first;
                if (tl.last_of) counters[first] = 0;
            }
            __syncthreads();
            if (tl.last_of) join(std::integral_constant<int, 8>(), p, last - first + 1, cta_slot, nullptr);
            __syncthreads();
        }
        i += k;
    }
}

template <bool F32, int DP, int NT, bool LONG, bool FULL>
cudaError_t launch(const AttendArgs& a, const AttendWs& ws, cudaStream_t st) {
    using Sh = Shape<F32, DP, NT, LONG>;
    static_assert(Sh::OCC <= ATTEND_OCC, "workspace counters");
    static_assert(sizeof(Tail) <= 1024 && Sh::OCC * (Sh::SMEM + 1024 + 1024) <= 228 * 1024, "resident CTAs");
    // as many CTAs as are resident, or as the longest line that the page tables allow has ranges for
    const double tiles = (double)a.step.max_new * (a.q_heads / a.pages.heads) / Sh::RT + 1;
    const double chunks = (double)a.step.width * a.pages.page / Sh::CHUNK_T + WARPS + Sh::LEAD;
    const double ctas = a.step.n_seqs * tiles * a.pages.heads * chunks / (WARPS * Sh::LEAST) + 1, most = ws.sms * Sh::OCC;
    attend4_split_kernel<F32, DP, NT, LONG, FULL><<<(int)(ctas < most ? ctas : most), THREADS, Sh::SMEM, st>>>(a, ws.partial, ws.counters, ws.zeros);
    return cudaGetLastError();
}

template <bool F32, int DP, int NT, bool LONG = false>
cudaError_t allow() {
    constexpr int bytes = Shape<F32, DP, NT, LONG>::SMEM;
    cudaError_t e = cudaFuncSetAttribute(attend4_split_kernel<F32, DP, NT, LONG, false>, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e == cudaSuccess)
        e = cudaFuncSetAttribute(attend4_split_kernel<F32, DP, NT, LONG, true>, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    return e;
}
template <int DP, int NT>
constexpr size_t slot_bytes() {   // one per warp, two per CTA (fp32 rows need no more)
    return (size_t)(WARPS + 2) * sizeof(float) * Shape<false, DP, NT, false>::OCC * Shape<false, DP, NT, false>::SLOT;
}
template <int DP>
constexpr size_t most_bytes() {
    return slot_bytes<DP, 1>() > slot_bytes<DP, 2>() ? slot_bytes<DP, 1>() : slot_bytes<DP, 2>();
}

}  // namespace

cudaError_t attend4_split_init() {
    cudaError_t e = cudaSuccess;
    auto one = [&](cudaError_t x) { e = e == cudaSuccess ? x : e; };
    one(allow<false, 64, 1>()), one(allow<false, 64, 2>()), one(allow<false, 128, 1>()), one(allow<false, 128, 2>());
    one(allow<false, 64, 1, true>()), one(allow<false, 128, 1, true>());
    one(allow<false, 256, 1>()), one(allow<false, 256, 2>());
    one(allow<true, 64, 1>()), one(allow<true, 64, 2>()), one(allow<true, 128, 1>()), one(allow<true, 128, 2>());
    one(allow<true, 256, 1>()), one(allow<true, 256, 2>());
    return e;
}

size_t attend4_split_bytes(int dim) { return dim <= 64 ? most_bytes<64>() : dim <= 128 ? most_bytes<128>() : most_bytes<256>(); }

// Rows per tile: 8, or 16 where a sequence and head has more (past 16 only fp32 rows of more than
// 128 elements come here, in tiles of 16; the rest are attend_prompt.cu's).
template <bool F32, int DP, bool FULL>
static cudaError_t by_rows(const AttendArgs& a, const AttendWs& ws, cudaStream_t st) {
    const bool few = (long long)a.step.max_new * (a.q_heads / a.pages.heads) <= 8;
    if constexpr (!F32 && DP <= 128) {
        // By the tokens that the page tables hold (lengths are not known here), from 128 for each of 12 warps
        // per SM on, long ranges: 32 sequences of 32k tokens take 210 us so and 226 us with short ones, one of
        // 777 tokens 13.4 us and 9.0 us.
        const long long most = (long long)a.step.n_seqs * a.step.width * a.pages.page * a.pages.heads;
        if (few && most >= 128ll * 12 * ws.sms) return launch<F32, DP, 1, true, FULL>(a, ws, st);
    }
    return few ? launch<F32, DP, 1, false, FULL>(a, ws, st) : launch<F32, DP, 2, false, FULL>(a, ws, st);
}
template <bool F32, int DP>
static cudaError_t by_width(const AttendArgs& a, const AttendWs& ws, cudaStream_t st) {
    return a.pages.dim == DP ? by_rows<F32, DP, true>(a, ws, st) : by_rows<F32, DP, false>(a, ws, st);
}

template <bool F32>
static cudaError_t by_shape(const AttendArgs& a, const AttendWs& ws, cudaStream_t st) {
    const int D = a.pages.dim;
    return D <= 64 ? by_width<F32, 64>(a, ws, st) : D <= 128 ? by_width<F32, 128>(a, ws, st) : by_width<F32, 256>(a, ws, st);
}

cudaError_t launch_attend4_split(bool bf16, const AttendArgs& a, const AttendWs& ws, cudaStream_t st) {
    return bf16 ? by_shape<false>(a, ws, st) : by_shape<true>(a, ws, st);
}

}  // namespace mlora
