// Causal attention over the 8-bit cache for sequences with many rows in the step
// (prompts), bf16, head_dim <= 128 (include/mlora.h).
//
// Mathematics as in attend_split.cu: x = scale ks (q . kc) log2 e, o = sum 2^(x - m) vs vc /
// sum 2^(x - m), m a running bound that moves when some x exceeds m + 8.  Rows are (query
// token, query head of the group) pairs of one key/value head, 256 per CTA as two tiles of
// 128: a converted key/value tile serves both, and one tile's softmax runs under the other
// tile's products.
//
// Products run on tcgen05.mma, 128 rows x 128 tokens: S = Q K^T in fp16 (codes exact,
// queries below 1 after a power of two per row), O += P V in bf16 with P = 2^(x - m) vs
// (one rounding) from tensor memory.  Tensor memory: S of the two tiles (P lies over S)
// and O of the two tiles, all 512 columns.
//
// Roles: warps 0-3 and 4-7 softmax and output of tile 0 and 1 (a thread per row), 8-11
// convert code tiles into fp16 keys (row-major rows of head elements) and bf16 values
// (tokens as rows: the product reads them column-major), 12 issues products, 13 copies
// code tiles (16-token boxes, so that pages of any multiple of 16 tokens do).
// Bound: the tensor pipe's 2 x 4 x 128^3 operations per token tile, closely followed by
// the softmax and the conversion (about 3.5 and 2 instructions per element).
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "attend.h"
#include "tc_ptx.cuh"

namespace mlora {

using namespace ptx;

namespace {

constexpr int TILE = 128;                  // rows per tile and tokens per tile
constexpr int PROMPT_ROWS = 2 * TILE;      // rows per CTA
constexpr int PROMPT_THREADS = 14 * 32;
constexpr float SLACK = 8.f, NO_MAX = -1e38f;

template <int DP>
struct PShape {
    static constexpr int BLK = DP / 64;                 // 64-element column blocks (128-byte rows)
    static constexpr int OPER = BLK * TILE * 128;       // bytes of a Q, K or V operand tile
    static constexpr int CODES = TILE * DP;             // bytes of a code tile
    static constexpr int SMEM = 1024 + 6 * OPER + 2 * CODES + 512;
};

struct PTail {
    uint64_t cfull[2], cempty[2];     // code tiles (keys, values)
    uint64_t kfull[2], kempty[2], vfull[2], vempty[2];
    uint64_t scfull[4], sfull[2], pfull[2], qfull, ofull;
    float scales[4][16];              // of a tile's 16-token pieces: 8 of keys, 8 of values
    uint32_t tmem;
    int abort_flag;
};
static_assert(sizeof(PTail) <= 512, "barriers and scales");

__device__ __forceinline__ void mbar_arrive(uint64_t* bar) {
    asm volatile("mbarrier.arrive.release.cta.shared::cta.b64 _, [%0];" ::"r"(smem_u32(bar)) : "memory");
}
__device__ __forceinline__ void tmem_ld32(uint32_t addr, uint32_t* r) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
          "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
          "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(addr));
}
// Waits for the thread's loads; the loaded registers are operands, so that no use of them
// moves above the wait.
__device__ __forceinline__ void tmem_wait_ld(uint32_t* r) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                   "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]),
                   "+r"(r[16]), "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]), "+r"(r[22]), "+r"(r[23]),
                   "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]), "+r"(r[29]), "+r"(r[30]), "+r"(r[31])
                 :
                 : "memory");
}
__device__ __forceinline__ void tmem_st32(uint32_t addr, const uint32_t* r) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
        "%15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};" ::"r"(addr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
        "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]),
        "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]),
        "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
        : "memory");
}
__device__ __forceinline__ void tmem_st16(uint32_t addr, const uint32_t* r) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
        "%15, %16};" ::"r"(addr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
        "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
}
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
// D += A B with A in tensor memory
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
    asm volatile(
        "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}\n" ::"r"(
            d),
        "r"(a), "l"(b), "r"(idesc), "r"(acc)
        : "memory");
}
__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// pairs of fp32
__device__ __forceinline__ uint64_t pair(float a, float b) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ float2 unpair(uint64_t a) {
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(a));
    return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ uint32_t bf2_of(float a, float b) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
}
// 4 codes of a word as fp16 or bf16 (two words); see attend_split.cu
__device__ __forceinline__ uint32_t minus1152(uint32_t u) {
    const __half2 h = __hsub2(*reinterpret_cast<__half2*>(&u), __half2half2(__ushort_as_half(0x6480)));
    return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ uint32_t bf16_codes(uint32_t u) {
    const uint32_t a = u & 0xFF7FFF7Fu, b = u & 0xFF80FF80u;
    const __nv_bfloat162 h = __hsub2(*reinterpret_cast<const __nv_bfloat162*>(&a), *reinterpret_cast<const __nv_bfloat162*>(&b));
    return *reinterpret_cast<const uint32_t*>(&h);
}
template <bool BF>
__device__ __forceinline__ uint2 widen(uint32_t w) {
    if (BF) return make_uint2(bf16_codes(__byte_perm(w, 0x43434343u, 0x4140)), bf16_codes(__byte_perm(w, 0x43434343u, 0x4342)));
    w ^= 0x80808080u;
    return make_uint2(minus1152(__byte_perm(w, 0x64646464u, 0x4140)), minus1152(__byte_perm(w, 0x64646464u, 0x4342)));
}

// One code tile (128 tokens x DP, as 16-token boxes) into an operand tile: DP / 64 blocks of
// 128 rows of 128 bytes under the 128-byte swizzle.  A warp takes 8 tokens x 64 elements at a
// time; lanes pair token t with t ^ 5, so that neither the reads (16-byte chunks at c ^ t)
// nor the writes (at (2 c + z) ^ t) of a quarter warp meet in a bank.
template <int DP, bool BF>
__device__ __forceinline__ void convert_tile(const uint8_t* codes, uint8_t* dst, int warp, int lane) {
    constexpr int N = 16 * (DP / 64) / 4;   // (8-token group, block) pairs per warp
    const int c = lane & 3, t8 = (lane >> 3) ^ ((lane & 4) ? 5 : 0);
#pragma unroll
    for (int u = 0; u < N; ++u) {
        const int combo = warp * N + u, blk = combo % (DP / 64), t = combo / (DP / 64) * 8 + t8;
        const int from = DP == 64 ? t * 64 + ((c ^ ((t >> 1) & 3)) << 4) : t * 128 + (((blk * 4 + c) ^ (t & 7)) << 4);
        const uint4 x = *reinterpret_cast<const uint4*>(codes + from);
        const uint2 a = widen<BF>(x.x), b = widen<BF>(x.y), d = widen<BF>(x.z), e = widen<BF>(x.w);
        uint8_t* row = dst + blk * (TILE * 128) + t * 128;
        *reinterpret_cast<uint4*>(row + (((2 * c) ^ (t & 7)) << 4)) = make_uint4(a.x, a.y, b.x, b.y);
        *reinterpret_cast<uint4*>(row + (((2 * c + 1) ^ (t & 7)) << 4)) = make_uint4(d.x, d.y, e.x, e.y);
    }
}

// Bits e of [lo, hi) of 32 columns.
__device__ __forceinline__ uint32_t column_mask(int lo, int hi) {
    const uint32_t below = hi >= 32 ? ~0u : hi <= 0 ? 0u : (1u << hi) - 1u;
    return lo <= 0 ? below : lo >= 32 ? 0u : below & ~((1u << lo) - 1u);
}

// The row's largest x over a tile (columns [lo, hi) of it if EDGE): the maximum of the raw
// scores of each 16-token piece, times its factor.
template <bool EDGE>
__device__ __forceinline__ float row_max(uint32_t sbase, const float* sc, float qf, int lo, int hi) {
    float mx = -INFINITY;
    uint32_t x[2][32];   // quarters of the row's 128 scores, the next one on its way
    tmem_ld32(sbase, x[0]);
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        uint32_t* y = x[q & 1];
        tmem_wait_ld(y);
        if (q < 3) tmem_ld32(sbase + (q + 1) * 32, x[(q + 1) & 1]);
        const uint32_t seen = EDGE ? column_mask(lo - q * 32, hi - q * 32) : ~0u;
#pragma unroll
        for (int g = 0; g < 2; ++g) {
            float a = -INFINITY, b = -INFINITY;
#pragma unroll
            for (int e = 0; e < 16; e += 2) {
                const int i = g * 16 + e;
                a = fmaxf(a, !EDGE || (seen >> i & 1) ? __uint_as_float(y[i]) : -INFINITY);
                b = fmaxf(b, !EDGE || (seen >> (i + 1) & 1) ? __uint_as_float(y[i + 1]) : -INFINITY);
            }
            a = fmaxf(a, b);
            const float v = a * (qf * sc[q * 2 + g]);
            mx = fmaxf(mx, EDGE && a == -INFINITY ? -INFINITY : v);
        }
    }
    return mx;
}

// Weights of a row over a tile: their sum into l2, times the value scales in bf16 over the
// scores that are read (32 columns of scores are 16 of weights).
template <bool EDGE>
__device__ __forceinline__ void weigh(uint32_t sbase, const float* sc, float qf, float m, int lo, int hi, uint64_t& l2) {
    const uint64_t nm = pair(-m, -m);
    uint32_t x[2][32];
    tmem_ld32(sbase, x[0]);
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        uint32_t* y = x[q & 1];
        uint32_t p[16];
        tmem_wait_ld(y);
        if (q < 3) tmem_ld32(sbase + (q + 1) * 32, x[(q + 1) & 1]);
        const uint32_t seen = EDGE ? column_mask(lo - q * 32, hi - q * 32) : ~0u;
#pragma unroll
        for (int g = 0; g < 2; ++g) {
            const float f = qf * sc[q * 2 + g], v = sc[8 + q * 2 + g];
            const uint64_t f2 = pair(f, f), v2 = pair(v, v);
#pragma unroll
            for (int e = 0; e < 16; e += 2) {
                const int i = g * 16 + e;
                const float2 z = unpair(fma2(pair(__uint_as_float(y[i]), __uint_as_float(y[i + 1])), f2, nm));
                float p0 = ex2(z.x), p1 = ex2(z.y);
                if (EDGE) {
                    p0 = seen >> i & 1 ? p0 : 0.f;
                    p1 = seen >> (i + 1) & 1 ? p1 : 0.f;
                }
                const uint64_t pp = pair(p0, p1);
                l2 = add2(l2, pp);
                const float2 w = unpair(mul2(pp, v2));
                p[i / 2] = bf2_of(w.x, w.y);
            }
        }
        tmem_st16(sbase + q * 16, p);
    }
}

template <int DP>
__global__ void __launch_bounds__(PROMPT_THREADS, 1)
attend_prompt_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV, const AttendArgs a,
                     int tiles) {
    using Sh = PShape<DP>;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t* smem = (uint8_t*)(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
    uint8_t* qs = smem;                              // [2 tiles]
    uint8_t* kb = smem + 2 * Sh::OPER;               // [2]
    uint8_t* vb = smem + 4 * Sh::OPER;               // [2]
    uint8_t* codes = smem + 6 * Sh::OPER;            // keys, values
    PTail& tl = *reinterpret_cast<PTail*>(codes + 2 * Sh::CODES);
    volatile int* abort_flag = &tl.abort_flag;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const CachePages& c = a.pages;
    const int H = c.heads, G = a.q_heads / H, D = c.dim;
    const int b = blockIdx.y, h = blockIdx.x % H, tile = tiles - 1 - blockIdx.x / H;   // the longest first

    const SeqRec s = load_seq(a.step, c.page, b, a.status);
    const int R = s.rows * G, r0 = tile * PROMPT_ROWS;
    if (r0 >= R) return;
    const int rows = min(PROMPT_ROWS, R - r0);
    const bool two = rows > TILE;
    const int pos_lo = s.start + r0 / G, pos_hi = s.start + (r0 + rows - 1) / G;
    const int ta = a.window > 0 ? max(0, pos_lo - a.window + 1) / 16 * 16 : 0;
    const int tb = pos_hi + 1;
    const int nt = tb > ta ? (tb - ta + TILE - 1) / TILE : 0;

    if (tid == 0) {
        for (int i = 0; i < 2; ++i) {
            mbar_init(&tl.cfull[i], 1);
            mbar_init(&tl.cempty[i], 128);
            mbar_init(&tl.kfull[i], 128);
            mbar_init(&tl.kempty[i], 1);
            mbar_init(&tl.vfull[i], 128);
            mbar_init(&tl.vempty[i], 1);
            mbar_init(&tl.sfull[i], 1);
            mbar_init(&tl.pfull[i], 128);
        }
        for (int i = 0; i < 4; ++i) mbar_init(&tl.scfull[i], 1);
        mbar_init(&tl.qfull, 256);
        mbar_init(&tl.ofull, 1);
        tl.abort_flag = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 12) {
        __syncwarp();
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&tl.tmem)), "r"(512)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = tl.tmem;

    if (warp < 8) {
        // ---- softmax and output: a thread per row
        const int t = warp >> 2, q4 = warp & 3;
        const int r = r0 + t * TILE + q4 * 32 + lane, rl = q4 * 32 + lane;
        const bool live = r < R;
        const int64_t row = s.row0 + (live ? r : r0) / G, head = h * G + (live ? r : r0) % G;
        // the query: fp16 scaled by a power of two, NaN statistics for a row that is not finite
        float qf;
        {
            const __nv_bfloat16* q = (const __nv_bfloat16*)a.q.ptr + row * a.q.row + head * a.q.head;
            auto load = [&](int i) {
                return live && i * 8 < D ? *reinterpret_cast<const uint4*>(q + i * 8) : make_uint4(0u, 0u, 0u, 0u);
            };
            float top = 0.f;
            bool fine = true;
#pragma unroll 4
            for (int i = 0; i < DP / 8; ++i) {
                const uint4 w = load(i);
                const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float x = fabsf(__uint_as_float(u[e] << 16)), y = fabsf(__uint_as_float(u[e] & 0xFFFF0000u));
                    fine &= x <= 3.402823466e38f && y <= 3.402823466e38f;
                    top = fmaxf(top, fmaxf(x, y));
                }
            }
            const int k = fine ? min(max((int)(__float_as_uint(top) >> 23) - 126, -100), 127) : 0;
            const float down = __uint_as_float((uint32_t)(127 - min(k, 126)) << 23) * (k > 126 ? 0.5f : 1.f);
            qf = fine ? a.scale * 1.4426950408889634f * __uint_as_float((uint32_t)(127 + k) << 23) : NAN;
#pragma unroll 4
            for (int i = 0; i < DP / 8; ++i) {
                const uint4 w = load(i);
                const uint32_t u[4] = {w.x, w.y, w.z, w.w};
                uint32_t v[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const __half2 p = __floats2half2_rn(__uint_as_float(u[e] << 16) * down,
                                                        __uint_as_float(u[e] & 0xFFFF0000u) * down);
                    v[e] = fine ? *reinterpret_cast<const uint32_t*>(&p) : 0u;
                }
                *reinterpret_cast<uint4*>(qs + t * Sh::OPER + i / 8 * (TILE * 128) + rl * 128 + (((i & 7) ^ (rl & 7)) << 4)) =
                    make_uint4(v[0], v[1], v[2], v[3]);
            }
            fence_proxy_async_smem();
            mbar_arrive(&tl.qfull);
        }
        const uint32_t lane_base = tmem + ((uint32_t)(q4 * 32) << 16);
        const uint32_t sbase = lane_base + t * TILE, obase = lane_base + 256 + t * TILE;
        const int hi = s.start + r / G + 1, lo = a.window > 0 ? hi - a.window : 0;   // tokens [lo, hi) are seen
        // limits of the tile's rows, for the tiles that no limit cuts
        const int rt = r0 + t * TILE;
        const int hi_min = s.start + rt / G + 1, hi_max = s.start + min(R - 1, rt + TILE - 1) / G + 1;
        const int lo_max = a.window > 0 ? hi_max - a.window : 0;
        float m = NO_MAX;
        uint64_t l2 = pair(0.f, 0.f);
        bool ok = true;
        if (t == 0 || two)
            for (int j = 0; j < nt; ++j) {
                ok = mbar_wait(&tl.scfull[j & 3], (j >> 2) & 1, abort_flag, a.status) &&
                     mbar_wait(&tl.sfull[t], j & 1, abort_flag, a.status);
                ok = __all_sync(~0u, ok);
                if (!ok) break;
                tc_fence_after();
                const float* sc = tl.scales[j & 3];
                const int t0 = ta + j * TILE;
                const bool edge = t0 + TILE > hi_min || t0 < lo_max;
                const float mx = edge ? row_max<true>(sbase, sc, qf, lo - t0, hi - t0) : row_max<false>(sbase, sc, qf, 0, 0);
                const bool above = mx > m + SLACK;
                if (__any_sync(~0u, above)) {   // the products so far are complete: S came after them
                    const float now = above ? mx : m, f = ex2(m - now);
                    m = now;
                    l2 = mul2(l2, pair(f, f));
                    if (j > 0)
#pragma unroll 1
                        for (int q = 0; q < DP / 32; ++q) {
                            uint32_t y[32];
                            tmem_ld32(obase + q * 32, y);
                            tmem_wait_ld(y);
#pragma unroll
                            for (int e = 0; e < 32; ++e) y[e] = __float_as_uint(__uint_as_float(y[e]) * f);
                            tmem_st32(obase + q * 32, y);
                        }
                }
                if (edge) weigh<true>(sbase, sc, qf, m, lo - t0, hi - t0, l2);
                else weigh<false>(sbase, sc, qf, m, 0, 0, l2);
                tmem_wait_st();
                tc_fence_before();
                mbar_arrive(&tl.pfull[t]);
            }
        if (t == 0 || two) {
            if (ok && nt > 0) ok = mbar_wait(&tl.ofull, 0, abort_flag, a.status);
            ok = __all_sync(~0u, ok);
            tc_fence_after();
            const float2 ls = unpair(l2);
            const float l = ls.x + ls.y, inv = l == 0.f ? 0.f : 1.f / l;
            __nv_bfloat16* o = (__nv_bfloat16*)a.o.ptr + row * a.o.row + head * a.o.head;
#pragma unroll
            for (int q = 0; q < DP / 32; ++q) {
                uint32_t x[32];
                if (nt > 0) {
                    tmem_ld32(obase + q * 32, x);
                    tmem_wait_ld(x);
                } else {
#pragma unroll
                    for (int e = 0; e < 32; ++e) x[e] = 0u;
                }
                if (!live) continue;
#pragma unroll
                for (int e = 0; e < 32; e += 8) {
                    if (q * 32 + e >= D) break;
                    uint32_t y[4];
#pragma unroll
                    for (int z = 0; z < 4; ++z)
                        y[z] = bf2_of(__uint_as_float(x[e + 2 * z]) * inv, __uint_as_float(x[e + 2 * z + 1]) * inv);
                    *reinterpret_cast<uint4*>(o + q * 32 + e) = make_uint4(y[0], y[1], y[2], y[3]);
                }
            }
        }
    } else if (warp < 12) {
        // ---- conversion
        for (int j = 0; j < nt; ++j) {
            const uint32_t par = j & 1, use = (j >> 1) & 1;
            if (!mbar_wait(&tl.cfull[0], par, abort_flag, a.status) ||
                !mbar_wait(&tl.kempty[j & 1], use ^ 1, abort_flag, a.status))
                break;
            convert_tile<DP, false>(codes, kb + (j & 1) * Sh::OPER, warp - 8, lane);
            mbar_arrive(&tl.cempty[0]);
            fence_proxy_async_smem();
            mbar_arrive(&tl.kfull[j & 1]);
            if (!mbar_wait(&tl.cfull[1], par, abort_flag, a.status) ||
                !mbar_wait(&tl.vempty[j & 1], use ^ 1, abort_flag, a.status))
                break;
            convert_tile<DP, true>(codes + Sh::CODES, vb + (j & 1) * Sh::OPER, warp - 8, lane);
            mbar_arrive(&tl.cempty[1]);
            fence_proxy_async_smem();
            mbar_arrive(&tl.vfull[j & 1]);
        }
    } else if (warp == 12) {
        if (lane == 0 && nt > 0) {
            // ---- products
            const uint32_t idesc_s = (1u << 4) | ((uint32_t)(TILE >> 3) << 17) | ((uint32_t)(TILE >> 4) << 24);   // fp16
            const uint32_t idesc_o = idesc_bf16(TILE, DP) | (1u << 16);                                           // B column-major
            auto scores = [&](int t, int j) {
#pragma unroll
                for (int k = 0; k < DP / 16; ++k) {
                    const uint32_t off = k / 4 * (TILE * 128) + k % 4 * 32;
                    mma_bf16(tmem + t * TILE, sdesc(smem_u32(qs + t * Sh::OPER) + off, 1024, SW128),
                             sdesc(smem_u32(kb + (j & 1) * Sh::OPER) + off, 1024, SW128), idesc_s, k > 0);
                }
                mma_commit(&tl.sfull[t]);
            };
            auto values = [&](int t, int j) {
#pragma unroll
                for (int k = 0; k < TILE / 16; ++k)
                    mma_ts(tmem + 256 + t * TILE, tmem + t * TILE + k * 8,
                           sdesc_lbo(smem_u32(vb + (j & 1) * Sh::OPER) + k * 2048, TILE * 128, 1024, SW128), idesc_o,
                           j > 0 || k > 0);
            };
            auto wait = [&](uint64_t* bar, int parity) {
                const bool ok = mbar_wait(bar, parity, abort_flag, a.status);
                tc_fence_after();
                return ok;
            };
            bool ok = wait(&tl.qfull, 0);
            for (int j = 0; ok && j < nt; ++j) {
                if (!(ok = wait(&tl.kfull[j & 1], (j >> 1) & 1))) break;
                scores(0, j);
                if (two) {
                    if (j > 0) {
                        if (!(ok = wait(&tl.pfull[1], (j - 1) & 1))) break;
                        values(1, j - 1);
                        mma_commit(&tl.vempty[(j - 1) & 1]);
                    }
                    scores(1, j);
                }
                mma_commit(&tl.kempty[j & 1]);
                if (!(ok = wait(&tl.vfull[j & 1], (j >> 1) & 1) && wait(&tl.pfull[0], j & 1))) break;
                values(0, j);
                if (!two) mma_commit(&tl.vempty[j & 1]);
            }
            if (ok && two) {
                ok = wait(&tl.pfull[1], (nt - 1) & 1);
                if (ok) values(1, nt - 1);
            }
            mma_commit(&tl.ofull);
            const long long t0 = clock64();   // the products are complete before the CTA goes
            while (!mbar_try_wait(&tl.ofull, 0) && clock64() - t0 < 200000000ll) {
            }
        }
    } else {
        // ---- code tiles and scales: lanes 0-7 the keys' 16-token pieces, 8-15 the values'
        const int piece = lane & 7;
        const bool is_v = lane & 8;
        int done = 0;
        bool ok = true;
        for (int j = 0; j < nt; ++j) {
            const int tk = ta + j * TILE + piece * 16;
            int crow = c.n_pages * H * c.page;   // past the end: reads as zero
            float sc = 0.f;
            if (lane < 16 && tk < tb) {
                const int id = load_page(a.step, c, b, tk / c.page, a.status);
                if (id >= 0) {
                    crow = (id * H + h) * c.page + tk % c.page;
                    sc = (is_v ? c.v_scale : c.k_scale)[(size_t)id * H + h];
                }
            }
            ok = mbar_wait(&tl.cempty[0], (j & 1) ^ 1, abort_flag, a.status);
            if (!__all_sync(~0u, ok)) break;
            if (lane < 16) tl.scales[j & 3][lane] = sc;
            if (lane == 0) mbar_expect_tx(&tl.cfull[0], Sh::CODES);
            __syncwarp();
            if (lane == 0) mbar_arrive(&tl.scfull[j & 3]);
            if (lane < 8) tma_2d(codes + piece * 16 * DP, &tmK, &tl.cfull[0], 0, crow);
            done = 2 * j + 1;
            ok = mbar_wait(&tl.cempty[1], (j & 1) ^ 1, abort_flag, a.status);
            if (!__all_sync(~0u, ok)) break;
            if (lane == 8) mbar_expect_tx(&tl.cfull[1], Sh::CODES);
            __syncwarp();
            if (lane >= 8 && lane < 16) tma_2d(codes + Sh::CODES + piece * 16 * DP, &tmV, &tl.cfull[1], 0, crow);
            done = 2 * j + 2;
        }
        // copies in flight land before the CTA goes
        for (int i = 0; i < 2; ++i) {
            const int n = (done + 1 - i) / 2;
            const long long t0 = clock64();
            while (n > 0 && !mbar_try_wait(&tl.cfull[i], (n - 1) & 1) && clock64() - t0 < 200000000ll) {
            }
        }
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    if (warp == 12) {
        __syncwarp();
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512) : "memory");
    }
}

template <int DP>
cudaError_t launch(const AttendArgs& a, const AttendWs& ws, cudaStream_t st) {
    const long long rows = (long long)a.step.max_new * (a.q_heads / a.pages.heads);
    const int tiles = (int)((rows + PROMPT_ROWS - 1) / PROMPT_ROWS);
    attend_prompt_kernel<DP><<<dim3((unsigned)tiles * a.pages.heads, a.step.n_seqs), PROMPT_THREADS, PShape<DP>::SMEM, st>>>(
        ws.k16, ws.v16, a, tiles);
    return cudaGetLastError();
}

}  // namespace

cudaError_t attend_prompt_init() {
    cudaError_t e = cudaFuncSetAttribute(attend_prompt_kernel<64>, cudaFuncAttributeMaxDynamicSharedMemorySize, PShape<64>::SMEM);
    if (e == cudaSuccess)
        e = cudaFuncSetAttribute(attend_prompt_kernel<128>, cudaFuncAttributeMaxDynamicSharedMemorySize, PShape<128>::SMEM);
    return e;
}

bool attend_prompt_takes(bool bf16, const AttendArgs& a) {
    return bf16 && a.pages.dim <= 128 && (long long)a.step.max_new * (a.q_heads / a.pages.heads) > 64;
}

cudaError_t launch_attend_prompt(const AttendArgs& a, const AttendWs& ws, cudaStream_t st) {
    return a.pages.dim <= 64 ? launch<64>(a, ws, st) : launch<128>(a, ws, st);
}

}  // namespace mlora
