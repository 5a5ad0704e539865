// Causal attention over the 8-bit and the 4-bit cache for sequences with many rows in the step
// (prompts) (include/mlora.h).
//
// Mathematics as in attend_split.cu: x = scale ks (q . kc) log2 e, o = sum 2^(x - m) vs vc /
// sum 2^(x - m).  The value scale goes into the exponent, 2^(x - m + log2 vs), and out of the
// sum again per 16 tokens.  Weights under 2^-126 are lost, so that vs has to stay well above: a block of
// vs < 2^-64 has its codes brought down by 2^-64 (exact in bf16) under a scale of 2^64 vs, and one of
// vs < 2^-120, whose codes append stores as 0, is converted to zeros under a scale of 1.  m is a
// row's largest x when it was last set; a step whose weights sum to more than 2^14 sets it
// again (no maximum is taken otherwise; bf16 and fp32 hold weights above 1 as well as below).
// x - m takes the exact product and the rounded m, so that the largest weight is 2^d, d up to half of m's
// last bit.  From 2^31 on that leaves fp32: a row whose m would reach 2^30 has all its x's divided by a
// power of two.  (Unequal scores then lie 2^5 apart at the least: 2^-32 of the weight, where it was 2^-64 or less.)
// Rows are (query token, query head of the group) pairs of one key/value head, 256 per CTA as
// two tiles of 128 (one, where heads have more than 128 elements or rows are fp32): a converted
// key/value tile serves both.
//
// Products run on tcgen05.mma in bf16, 128 rows x 64 tokens a step: S = Q K^T (queries and
// codes exact), O += P V with P = 2^(x - m) vs from tensor memory, rounded once to bf16: 8 bits,
// where attend_split.cu has the room under its codes' stream for 16.  The row's sum takes the
// rounded weights, so that an error of theirs is none of scale: 0.0019 against 64 bits, of which
// rounding the output is 0.0017; a second term would add half of the products again, and a subtraction
// and a conversion per weight to the softmax warps, whose chain is the bound.  The tensor cores also cut the sums of O off at every 16 tokens, which bf16
// rows leave at that: of a sum of one sign 0.25% over 2^20 tokens, 0.9% over 2^21.  Tensor
// memory, all 512 columns: two S of 64 columns per tile, so that a step's scores are ready
// before the last step's weights are done (P lies over its S), and O of the two tiles (or of
// one, of up to 256 columns).  fp32 rows run the same products over three bf16 terms of the
// queries and of the weights (24 bits): 2 x 1000 rows of 16/8 heads of 128 after 100 take 57 us (266 us
// in attend_split.cu), 8192 tokens of 32/8 heads 1640 us, 335 TFLOP/s or 1000 of the terms' products.
// Their O is taken out of the tensor cores every FOLD steps (118 x 6000 tokens: error against 64 bits
// 1.1e-6, 2.0e-6 with twice the steps, 5.6e-6 without, 1.4e-6 in plain fp32; 8192 tokens 1670, 1485 and
// 1335 us, when measured).
//
// Bound: the products, 2 x 2 x 128 x 64 x head_dim operations per tile and step.  8192 tokens of
// 32/8 heads of 128 take 380 us, 1450 TFLOP/s; 4096 take 121 us, 1130 TFLOP/s (the tensor pipe is
// busy 55% of the time, tensor memory 61%, the issue slots 47%).  A step takes 1500
// cycles, of which the products could do with 1280: half of the exponentials or half of the
// products left out changes it by 2%, the weights' sum left out by 6%: what counts is a softmax
// warp's own chain of some 300 instructions.  A row tile's start and end take 9000 cycles.
//
// What measured slower (8192 tokens): scores of 128 tokens a product, without a second buffer
// (487 us); two threads per row (423); the sums by mma.sync (570); one arrival per warp (396);
// the tiles' products in turns (426); waits that sleep (389).
//
// Conversion: a sequence of many row tiles (PRE_TILES) has its codes converted once, by a kernel
// before, into operand tiles (as they lie in shared memory) in the handle's workspace, which
// the attention copies in bulk; converted per row tile the work takes half of the issue slots
// (8192 tokens: 496 us against 572 at the time).  One of fewer, or one for which the workspace
// has no room left, is converted inside the attention.
//
// Where row tiles are fewer than half the SMs, each one's tokens are cut into equal parts, a CTA
// each; the CTA that finishes a row tile last joins the parts, in their order (300 tokens after
// 5000 of one sequence: 46 us).
//
// The 4-bit cache (BITS 4, block4.cuh): a code times its scale is exact in bf16, so that the operand
// tiles hold the values themselves, over a unit that goes into the scores' factor (on the host) and
// into the output; tokens have no scales left (8192 tokens 360 us, 382 us over 8 bits; 4 prompts of
// 6000 rows after 1024 134 and 140 us).  Values and weights of bf16 rows could be fp16 (weights in 11 bits: error
// 0.0017, in bf16 0.0021), but fp16 holds no weight under 2^-24: with m 12 below the largest, so that the weights
// reach as far as attend4_split.cu's, it moves often (442 and 152 us; scores of three times the size 615 us,
// 407 in bf16); with m 6 below, 495 us at that size, and tokens under 2^-31 of the largest are lost.
//
// Roles: warps 0-3 and 4-7 softmax and output of tile 0 and 1 (a thread per row), 8 copies
// operand tiles or 8-15 read codes and convert them into keys and values in bf16 (tokens as rows; the
// second product reads them column-major), a warp per 16 tokens of 128 with the next 128
// tokens' codes on their way in registers, 16 and 17 issue the products of tile 0 and 1 (one
// warp's waits would outlast both tiles' products).
#include <cuda_bf16.h>

#include <climits>
#include <type_traits>

#include "attend.h"
#include "block4.cuh"
#include "f32x2.cuh"
#include "tc_ptx.cuh"

namespace mlora {

using namespace ptx;

namespace {

constexpr int TILE = 128;                  // rows per tile
constexpr int STEP = 64;                   // tokens per product
constexpr int PART = 512;                  // a part of a row tile's tokens is at least so long
constexpr int SOFT = 8, CONV = 8;          // softmax and conversion warps
constexpr int PROMPT_THREADS = 32 * (SOFT + CONV + 4);   // (two warps only complete a warpgroup)
// Registers per thread: 96 at launch, then the softmax warps take what the others leave; the
// sum may not exceed the launch's.
constexpr int REGS_SOFT = 128, REGS_REST = 72;
static_assert(32 * (SOFT * REGS_SOFT + (CONV + 4) * REGS_REST) <= PROMPT_THREADS * 96, "register split");
constexpr int FOLD = 16;                   // steps of fp32 rows between roundings of O into fp32 outside
constexpr float MOST = 16384.f;            // sum of a step's weights over which m moves
constexpr int FAR = 30;                    // a row's x's are divided so that |m| stays below 2^FAR
constexpr float NO_MAX = -1e38f;           // m of a row that has seen nothing
constexpr int MOST_DOWN = 114;             // queries are divided by 2^MOST_DOWN at most (scale 2^128 would leave fp32)
constexpr float SMALL_SCALE = 0x1p-64f;    // value scales below it are brought up by 1 / SMALL_SCALE

template <int DP, bool F32 = false>
struct PShape {
    // elements up to 256 leave tensor memory for one row tile, and shared memory for key and value
    // tiles of 64 tokens; so do fp32 rows' terms for one row tile
    static_assert(!F32 || DP <= 128, "queries in three terms");
    static constexpr int TERMS = F32 ? 3 : 1;           // bf16 terms of a query and of a weight
    static constexpr int TILES = DP == 256 || F32 ? 1 : 2;   // row tiles per CTA
    // columns of tensor memory: scores at 0, and a step's weights over them; of fp32 rows their
    // lower two terms at P_AT; O, and after it (fp32) that of the lower terms: the tensor cores'
    // sums drop bits, those of the full size one in 16 tokens rather than three
    static constexpr int P_AT = 2 * STEP, P_COLS = (TERMS - 1) * STEP / 2;
    static constexpr int O_AT = 256, O_COLS = (F32 ? 2 : 1) * DP;
    static_assert(!F32 || P_AT + 2 * P_COLS <= O_AT, "lower terms");
    static constexpr int ROWS = TILES * TILE;
    static constexpr int KT = DP == 256 ? 64 : 128;     // tokens converted at a time
    static constexpr int SPT = KT / STEP;               // steps per token tile
    static constexpr int BLK = DP / 64;                 // 64-element column blocks (128-byte rows)
    static constexpr int QOPER = BLK * TILE * 128;      // bytes of a Q operand tile
    static constexpr int OPER = BLK * KT * 128;         // of a K or V operand tile
    static constexpr int SMEM = 1024 + TILES * TERMS * QOPER + 4 * OPER + 2048;
    static_assert(SMEM <= 232448 && O_AT + TILES * O_COLS <= 512, "shared and tensor memory");
    static constexpr int PIECES = KT / 16;              // of 16 tokens
    static_assert(PROMPT_SLOT >= ROWS * (DP + 2), "workspace slot");
};

struct PTail {
    uint64_t kfull[2], kempty[2], vfull[2], vempty[2];
    uint64_t scfull[4], sfull[2][2], pfull[2][2], odone[2][2], qfull[2], alldone[2];   // [tile][S buffer]
    float qf[2][TILE];                // per row: scale log2 e over the query's power of two
    float scales[4][24];              // of a token tile's 16-token pieces: ks, log2 vs, 1 / vs (8 each)
    uint32_t tmem;
    int abort_flag, last;
};
static_assert(sizeof(PTail) <= 2048, "barriers, scales and row factors");

__device__ __forceinline__ bool elect_one() {
    uint32_t p;
    asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}\n" : "=r"(p));
    return p != 0;
}
__device__ __forceinline__ void mbar_arrive(uint64_t* bar) {
    asm volatile("mbarrier.arrive.release.cta.shared::cta.b64 _, [%0];" ::"r"(smem_u32(bar)) : "memory");
}
// whether the phase is complete, without a wait
__device__ __forceinline__ bool mbar_done(uint64_t* bar, uint32_t parity) {
    uint32_t ok;
    asm volatile("{\n .reg .pred p;\n mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n selp.u32 %0, 1, 0, p;\n}\n"
                 : "=r"(ok)
                 : "r"(smem_u32(bar)), "r"(parity)
                 : "memory");
    return ok != 0;
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
__device__ __forceinline__ void tmem_ld16(uint32_t addr, uint32_t* r) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, "
        "[%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(addr));
}
__device__ __forceinline__ void tmem_st16(uint32_t addr, const uint32_t* r) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
        "%15, %16};" ::"r"(addr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
        "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
}
__device__ __forceinline__ void tmem_loaded16(uint32_t* r) {
    asm volatile(""
                 : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                   "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15])
                 :
                 : "memory");
}
__device__ __forceinline__ void tmem_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
// Names loaded registers as operands after the wait, so that no use of them moves above it.
__device__ __forceinline__ void tmem_loaded(uint32_t* r) {
    asm volatile(""
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
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
// One product of 16 elements of K: D += A B, A in shared (SS) or tensor memory (TS).  The
// descriptors' low words are made in place from the loop's base and a constant: hoisted out of
// the loop they would spill, and the reloads would outlast the products.
template <int A_OFF, int B_OFF>
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
    asm volatile(
        "{\n .reg .pred p;\n .reg .b64 a, b;\n setp.ne.b32 p, %4, 0;\n add.s64 a, %1, %5;\n add.s64 b, %2, %6;\n"
        " tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, p;\n}\n" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(acc), "n"(A_OFF >> 4), "n"(B_OFF >> 4)
        : "memory");
}
template <int A_COL, int B_OFF>
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
    asm volatile(
        "{\n .reg .pred p;\n .reg .b64 b;\n .reg .b32 a;\n setp.ne.b32 p, %4, 0;\n add.s32 a, %1, %5;\n add.s64 b, %2, "
        "%6;\n tcgen05.mma.cta_group::1.kind::f16 [%0], [a], b, %3, p;\n}\n" ::"r"(d),
        "r"(a), "l"(b), "r"(idesc), "r"(acc), "n"(A_COL), "n"(B_OFF >> 4)
        : "memory");
}
// K steps [0, N): SS in 64-element blocks of 128 (A) and B_ROWS rows of 128 bytes, TS over rows
// of tokens.
template <int N, int B_ROWS, int K = 0>
__device__ __forceinline__ void product_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
    mma_ss<K / 4 * (128 * 128) + K % 4 * 32, K / 4 * (B_ROWS * 128) + K % 4 * 32>(d, a, b, idesc, K > 0 ? 1u : acc);
    if constexpr (K + 1 < N) product_ss<N, B_ROWS, K + 1>(d, a, b, idesc, acc);
}
template <int N, int K = 0>
__device__ __forceinline__ void product_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
    mma_ts<K * 8, K * 2048>(d, a, b, idesc, K > 0 ? 1u : acc);
    if constexpr (K + 1 < N) product_ts<N, K + 1>(d, a, b, idesc, acc);
}
__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ uint32_t bf2_of(float a, float b) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
}
// the halves of a bf16 pair onto two fp32 sums
__device__ __forceinline__ void add_bf16(float& a, float& b, uint32_t w) {
    asm("{\n .reg .b16 l, h;\n mov.b32 {l, h}, %2;\n add.rn.f32.bf16 %0, l, %0;\n add.rn.f32.bf16 %1, h, %1;\n}"
        : "+f"(a), "+f"(b)
        : "r"(w));
}
// 4 codes of a word as bf16 (two words); see attend_split.cu
__device__ __forceinline__ uint32_t bf16_codes(uint32_t u) {
    const uint32_t a = u & 0xFF7FFF7Fu, b = u & 0xFF80FF80u;
    const __nv_bfloat162 h = __hsub2(*reinterpret_cast<const __nv_bfloat162*>(&a), *reinterpret_cast<const __nv_bfloat162*>(&b));
    return *reinterpret_cast<const uint32_t*>(&h);
}
// The upper byte, 0x43 for the codes themselves, holds seven bits of the exponent: 0x23 gives them
// times SMALL_SCALE.
constexpr uint32_t OVER = 0x43434343u, OVER_SMALL = 0x23232323u;
__device__ __forceinline__ uint2 widen(uint32_t w, uint32_t over) {
    return make_uint2(bf16_codes(__byte_perm(w, over, 0x4140)), bf16_codes(__byte_perm(w, over, 0x4342)));
}
// 16 bytes of global memory (zeros where `in` is false) into shared memory
__device__ __forceinline__ void cp_async16_or_zero(uint32_t dst, const void* src, bool in) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(in ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp_async_wait_all() { asm volatile("cp.async.wait_all;" ::: "memory"); }

// 16 codes of token t, elements 16 c .. of 64-element block blk, into an operand tile: DP / 64
// blocks of KT rows of 128 bytes under the 128-byte swizzle.  (Lanes pair token t with t ^ 5,
// so that the writes of a quarter warp, at (2 c + z) ^ t, do not meet in a bank.)
template <int KT>
__device__ __forceinline__ void convert16(uint4 x, uint8_t* dst, int t, int blk, int c, uint32_t over) {
    const uint2 a = widen(x.x, over), b = widen(x.y, over), d = widen(x.z, over), e = widen(x.w, over);
    uint8_t* row = dst + blk * (KT * 128) + t * 128;
    *reinterpret_cast<uint4*>(row + (((2 * c) ^ (t & 7)) << 4)) = make_uint4(a.x, a.y, b.x, b.y);
    *reinterpret_cast<uint4*>(row + (((2 * c + 1) ^ (t & 7)) << 4)) = make_uint4(d.x, d.y, e.x, e.y);
}

template <int N>
__device__ __forceinline__ void registers_up() {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void registers_down() {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

// Barrier of the softmax warps.
__device__ __forceinline__ void soft_sync() {
    __syncwarp();
    asm volatile("bar.sync 1, %0;" ::"n"(32 * SOFT) : "memory");
}

// Bits e of [lo, hi) of 32 columns.
__device__ __forceinline__ uint32_t column_mask(int lo, int hi) {
    const uint32_t below = hi >= 32 ? ~0u : hi <= 0 ? 0u : (1u << hi) - 1u;
    return lo <= 0 ? below : lo >= 32 ? 0u : below & ~((1u << lo) - 1u);
}

// The largest x of a row's 64 scores, of columns [lo, hi) of them: the maximum of the raw
// scores of each 16-token piece, times its factor.
template <bool BARE>
__device__ __forceinline__ float row_max(uint32_t sat, const float* sc, float qf, int lo, int hi) {
    float mx = -INFINITY;
#pragma unroll 1
    for (int g = 0; g < STEP / 16; ++g) {
        uint32_t y[16];
        tmem_ld16(sat + g * 16, y);
        tmem_wait_ld();
        tmem_loaded16(y);
        const uint32_t seen = column_mask(lo - g * 16, hi - g * 16);
        float a = -INFINITY;
#pragma unroll
        for (int e = 0; e < 16; ++e) a = fmaxf(a, seen >> e & 1 ? __uint_as_float(y[e]) : -INFINITY);
        mx = fmaxf(mx, a == -INFINITY ? -INFINITY : a * (BARE ? qf : qf * sc[g]));
    }
    return mx;
}

// Weights of a row's 64 scores: times the value scales into y[0, 32) (bf16 pairs); returns
// the sum of what was rounded (without the value scales), so that a heavy token's rounding is
// divided out again.  PG tokens share their scales: 16, or 64 where pages are multiples of it
// (8192 tokens, 32/8 heads, pages of 64: 466 us with PG 64, 474 us with PG 16, when measured).
// BARE: tokens have no scales (4 bits).
template <bool EDGE, int PG, bool BARE>
__device__ __forceinline__ uint64_t weigh(uint32_t sat, const float* sc, float qf, float m, int lo, int hi,
                                          uint32_t (&y)[STEP]) {
    tmem_ld32(sat, y);
    tmem_ld32(sat + 32, y + 32);
    tmem_wait_ld();
    tmem_loaded(y);
    tmem_loaded(y + 32);
    uint64_t sum = pair(0.f, 0.f);
#pragma unroll
    for (int g = 0; g < STEP / PG; ++g) {
        const float f = BARE ? qf : qf * sc[g * (PG / 16)], c = BARE ? -m : sc[8 + g * (PG / 16)] - m;
        const float v = BARE ? 1.f : sc[16 + g * (PG / 16)];
        const uint64_t f2 = pair(f, f), c2 = pair(c, c);
        float l[2] = {0.f, 0.f};
#pragma unroll
        for (int k = 0; k < PG; k += 32) {
            const uint32_t seen = EDGE ? column_mask(lo - g * PG - k, hi - g * PG - k) : 0u;
#pragma unroll
            for (int e = 0; e < (PG < 32 ? PG : 32); e += 2) {
                const int i = g * PG + k + e;
                const float2 z = unpair(fma2(pair(__uint_as_float(y[i]), __uint_as_float(y[i + 1])), f2, c2));
                float p0 = ex2(z.x), p1 = ex2(z.y);
                if (EDGE) {
                    p0 = seen >> e & 1 ? p0 : 0.f;
                    p1 = seen >> (e + 1) & 1 ? p1 : 0.f;
                }
                const uint32_t w = bf2_of(p0, p1);
                add_bf16(l[0], l[1], w);
                y[i / 2] = w;
            }
        }
        sum = BARE ? add2(pair(l[0], l[1]), sum) : fma2(pair(l[0], l[1]), pair(v, v), sum);
    }
    return sum;
}

// The same for fp32 rows, the weights as three bf16 terms (24 bits): the first into y, the others
// into columns pat and pat + 32; the sum is that of the weights themselves.
template <bool EDGE, int PG, bool BARE>
__device__ __forceinline__ uint64_t weigh3(uint32_t sat, uint32_t pat, const float* sc, float qf, float m, int lo, int hi,
                                           uint32_t (&y)[STEP]) {
    constexpr int N = PG < 32 ? PG : 32;
    uint64_t sum = pair(0.f, 0.f);
#pragma unroll
    for (int half = 0; half < 2; ++half) {
        uint32_t x[32], w2[16], w3[16];
        tmem_ld32(sat + half * 32, x);
        tmem_wait_ld();
        tmem_loaded(x);
        const uint32_t seen = EDGE ? column_mask(lo - half * 32, hi - half * 32) : 0u;
#pragma unroll
        for (int g = 0; g < 32; g += N) {
            const float* at = sc + half * 2 + g / 16;
            const float f = BARE ? qf : qf * at[0], c = BARE ? -m : at[8] - m, v = BARE ? 1.f : at[16];
            const uint64_t f2 = pair(f, f), c2 = pair(c, c);
            uint64_t l = pair(0.f, 0.f);
#pragma unroll
            for (int i = g; i < g + N; i += 2) {
                const float2 z = unpair(fma2(pair(__uint_as_float(x[i]), __uint_as_float(x[i + 1])), f2, c2));
                float p0 = ex2(z.x), p1 = ex2(z.y);
                if (EDGE) {
                    p0 = seen >> i & 1 ? p0 : 0.f;
                    p1 = seen >> (i + 1) & 1 ? p1 : 0.f;
                }
                l = add2(l, pair(p0, p1));
                const uint32_t u = bf2_of(p0, p1);
                p0 -= __uint_as_float(u << 16);
                p1 -= __uint_as_float(u & 0xFFFF0000u);
                const uint32_t t = bf2_of(p0, p1);
                y[half * 16 + i / 2] = u;
                w2[i / 2] = t;
                w3[i / 2] = bf2_of(p0 - __uint_as_float(t << 16), p1 - __uint_as_float(t & 0xFFFF0000u));
            }
            sum = BARE ? add2(l, sum) : fma2(l, pair(v, v), sum);
        }
        tmem_st16(pat + half * 16, w2);
        tmem_st16(pat + 32 + half * 16, w3);
    }
    return sum;
}

// Whether a block of value scale vs counts as zeros, and the byte over its codes (see put_scales).
__device__ __forceinline__ bool no_values(float vs) { return fabsf(vs) < TINY_SCALE; }
__device__ __forceinline__ uint32_t values_over(float vs) { return vs < SMALL_SCALE ? OVER_SMALL : OVER; }

// A conversion warp's share of a token tile of one operand, 16 tokens and WB column
// blocks, as codes in registers.  (VALUES is the 4-bit cache's: its keys and values lie apart.)
template <int BITS, int DP, bool VALUES>
struct Piece {
    using Sh = PShape<DP>;
    // a warp per 16 tokens, or two with half of the blocks each; 16-byte loads per thread
    static constexpr int WB = Sh::BLK * Sh::PIECES / CONV, N = 2 * WB;
    // warp w's 16-token piece and first column block
    static __device__ __forceinline__ int piece(int w) { return Sh::PIECES == CONV ? w : w % Sh::PIECES; }
    static __device__ __forceinline__ int blk0(int w) { return Sh::PIECES == CONV ? 0 : w / Sh::PIECES * WB; }
    uint4 x[N];
    // tokens `place` .. + 15 of page `id`; zeros where id < 0
    __device__ __forceinline__ void load(const CachePages& c, int id, int h, int place, int w, int lane) {
        const int8_t* codes = VALUES ? c.v_codes : c.k_codes;
        const int c4 = lane & 3, t8 = (lane >> 3) ^ ((lane & 4) ? 5 : 0), b0 = blk0(w);
        const int8_t* from = codes + ((size_t)(id < 0 ? 0 : id * c.heads + h) * c.page + place + t8) * c.dim + b0 * 64 + c4 * 16;
#pragma unroll
        for (int u = 0; u < N; ++u)
            x[u] = id >= 0 && ((b0 + u % WB) * 4 + c4) * 16 < c.dim
                       ? __ldg(reinterpret_cast<const uint4*>(from + u / WB * 8 * c.dim + u % WB * 64))
                       : make_uint4(0u, 0u, 0u, 0u);
    }
    __device__ __forceinline__ void zero() {
#pragma unroll
        for (int u = 0; u < N; ++u) x[u] = make_uint4(0u, 0u, 0u, 0u);
    }
    // into operand tile `dst` (generic address)
    __device__ __forceinline__ void store(uint8_t* dst, int w, int lane, uint32_t over = OVER) const {
        const int c4 = lane & 3, t8 = (lane >> 3) ^ ((lane & 4) ? 5 : 0), b0 = blk0(w);
#pragma unroll
        for (int u = 0; u < N; ++u)
            convert16<Sh::KT>(x[u], dst, piece(w) * 16 + u / WB * 8 + t8, b0 + u % WB, c4, over);
    }
};
// In 4 bits a lane takes two atoms (16 elements of a token) that lie together in the block: of keys,
// tokens g and g + 8 of each 64 elements; of values, tokens 2 tig and 2 tig + 1 of each 8 tokens and 128
// elements.
template <int DP, bool VALUES>
struct Piece<4, DP, VALUES> {
    using Sh = PShape<DP>;
    static constexpr int WB = Sh::BLK * Sh::PIECES / CONV, N = VALUES ? (DP == 64 ? 1 : 2) : WB;
    static __device__ __forceinline__ int piece(int w) { return Sh::PIECES == CONV ? w : w % Sh::PIECES; }
    static __device__ __forceinline__ int blk0(int w) { return Sh::PIECES == CONV ? 0 : w / Sh::PIECES * WB; }
    static_assert(!VALUES || DP == 64 || WB == 2, "values are taken 128 elements at a time");
    uint4 x[N];
    uint32_t s[N];   // the two scales
    // the lane's u-th pair: its group (of 16 elements) and first token, and the second's distance
    static __device__ __forceinline__ int group_of(int u, int w, int lane) {
        return VALUES ? blk0(w) * 4 + (DP == 64 ? lane >> 2 & 3 : lane >> 2) : (blk0(w) + u) * 4 + (lane & 3);
    }
    static __device__ __forceinline__ int token_of(int u, int lane) {
        return VALUES ? (DP == 64 ? lane >> 4 : u) * 8 + (lane & 3) * 2 : lane >> 2;
    }
    __device__ __forceinline__ void load(const CachePages& c, int id, int h, int place, int w, int lane) {
        const int groups = c.dim >> 4;
        const uint8_t* block =
            c.blocks + ((size_t)(id < 0 ? 0 : id * c.heads + h) * (c.page >> 4) + (place >> 4)) * block4_bytes(c.dim);
#pragma unroll
        for (int u = 0; u < N; ++u) {
            const int gr = group_of(u, w, lane), t = token_of(u, lane);
            const int at = VALUES ? value_atom(t, gr, groups) : key_atom(t, gr, groups);
            x[u] = make_uint4(0u, 0u, 0u, 0u);
            s[u] = 0u;
            if (id >= 0 && gr < groups) {
                x[u] = __ldg(reinterpret_cast<const uint4*>(block + (VALUES ? 8 * c.dim : 0) + at * 8));
                s[u] = __ldg(reinterpret_cast<const uint16_t*>(block + (VALUES ? 17 * c.dim : 16 * c.dim) + at));
            }
        }
    }
    __device__ __forceinline__ void zero() {}   // (no scale is too small)
    // 16 values of a token, as 32 bytes of the tile
    static __device__ __forceinline__ void put(uint8_t* dst, int t, int gr, uint2 codes, uint32_t scale) {
        const Scale2 sc = scale_bf16(scale);
        uint8_t* row = dst + (gr >> 2) * (Sh::KT * 128) + t * 128;
#pragma unroll
        for (int z = 0; z < 2; ++z) {
            const uint32_t w = z ? codes.y : codes.x;
            const uint32_t a = codes_bf16<0>(w, sc), b = codes_bf16<1>(w, sc), d = codes_bf16<2>(w, sc), e = codes_bf16<3>(w, sc);
            *reinterpret_cast<uint4*>(row + (((2 * (gr & 3) + z) ^ (t & 7)) << 4)) =
                make_uint4(__byte_perm(a, b, 0x5410), __byte_perm(d, e, 0x5410), __byte_perm(a, b, 0x7632), __byte_perm(d, e, 0x7632));
        }
    }
    // (values: lanes of odd groups store their second token first, so that the stores of a quarter
    // warp, at (2 group + z) ^ token, do not meet in a bank)
    __device__ __forceinline__ void store(uint8_t* dst, int w, int lane, uint32_t = 0u) const {
#pragma unroll
        for (int u = 0; u < N; ++u) {
            const int gr = group_of(u, w, lane), t = piece(w) * 16 + token_of(u, lane);
            const bool swap = VALUES && (gr & 1);
            const uint2 a = make_uint2(x[u].x, x[u].y), b = make_uint2(x[u].z, x[u].w);
            const uint32_t sa = __byte_perm(s[u], 0u, 0x4040), sb = __byte_perm(s[u], 0u, 0x4141);
            const int next = VALUES ? 1 : 8;
            put(dst, t + (swap ? next : 0), gr, swap ? b : a, swap ? sb : sa);
            put(dst, t + (swap ? 0 : next), gr, swap ? a : b, swap ? sa : sb);
        }
    }
};
// Scales of 16 tokens as the softmax takes them (see the top of the file).
__device__ __forceinline__ void put_scales(float* sc, int w, float ks, float vs) {
    const bool none = no_values(vs);
    const float up = vs < SMALL_SCALE ? vs * (1.f / SMALL_SCALE) : vs;
    sc[w] = ks;
    sc[8 + w] = none ? 0.f : log2f(up);
    sc[16 + w] = none ? 1.f : 1.f / up;
}

// Token tiles of a sequence that its rows see, from token `lo` on.
struct Span {
    int j0, j1, lo;
};
template <int KT>
__device__ __forceinline__ Span span_of(const SeqRec& s, int window) {
    const int tb = s.start + s.rows, ta = first_seen(s.start, window);
    return tb > ta ? Span{ta / KT, (tb + KT - 1) / KT, ta} : Span{0, 0, 0};
}

constexpr int PRE_THREADS = 32 * CONV;
// Row tiles over which a sequence is converted before: 64 KB written and read again per 128 tokens
// and head (of 128) cost more than to convert 16 KB for each of a few row tiles.  32/8 heads of 128, before
// and in place: 16 x 128 tokens after 4000, 2 row tiles, 220 and 146 us; 32 x 600, 10 tiles, 228 and
// 220 us; 8 x 1200, 19 tiles, 145 and 144 us; 1024 after 6000, 16 tiles, 104 and 116 us; 4 prompts
// of 14 to 32 tiles 139 and 150 us; heads of 256, 2 x 1000 rows, 16 tiles, 49 and 53 us.
constexpr int PRE_TILES = 12;
constexpr int NOT_HERE = INT_MIN;   // at[b] of a sequence that is converted inside the attention

// Operand tiles in the workspace: at[b] + j is the place of tile j of sequence b (each place
// holds every head's keys and values, then their scales).
template <int BITS, int DP, bool F32>
__global__ void __launch_bounds__(PRE_THREADS) convert_kernel(const AttendArgs a, uint8_t* __restrict__ operands, int room,
                                                              int* __restrict__ at) {
    using Sh = PShape<DP, F32>;
    const CachePages& c = a.pages;
    const int H = c.heads, G = a.q_heads / H, b = blockIdx.y;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    auto need = [&](int i) {
        const SeqRec s = load_seq(a.step, c.page, i, a.status);
        const Span p = span_of<Sh::KT>(s, a.window);
        return s.rows * G > PRE_TILES * Sh::ROWS ? p.j1 - p.j0 : 0;
    };
    const SeqRec s = load_seq(a.step, c.page, b, a.status);
    const Span p = span_of<Sh::KT>(s, a.window);
    const int mine = need(b);
    long long before = 0;
    for (int i = tid; i < b; i += PRE_THREADS) before += need(i);
    __shared__ long long part[CONV];
#pragma unroll
    for (int d = 16; d; d >>= 1) before += __shfl_xor_sync(~0u, before, d);
    if (lane == 0) part[warp] = before;
    __syncthreads();
    before = 0;
    for (int w = 0; w < CONV; ++w) before += part[w];
    const bool here = mine > 0 && before + mine <= room;
    if (blockIdx.x == 0 && tid == 0) at[b] = here ? (int)before - p.j0 : NOT_HERE;
    if (!here) return;
    for (int i = blockIdx.x; i < mine * H; i += gridDim.x) {
        const int j = p.j0 + i / H, h = i % H, tk = j * Sh::KT + Piece<BITS, DP, false>::piece(warp) * 16;
        // (no page is looked up that holds no token that is seen)
        const int blk = tk / c.page, place = tk % c.page;
        const int id = tk < s.start + s.rows && blk >= p.lo / c.page ? load_page(a.step, c, b, blk, a.status) : -1;
        float ks = 0.f, vs = 1.f;
        if constexpr (BITS == 8) ks = id >= 0 ? c.k_scale[(size_t)id * H + h] : 0.f, vs = id >= 0 ? c.v_scale[(size_t)id * H + h] : 0.f;
        const size_t slot = (size_t)(before + j - p.j0) * H + h;
        uint8_t* to = operands + slot * 2 * Sh::OPER;
        Piece<BITS, DP, false> k;
        Piece<BITS, DP, true> v;
        k.load(c, id, h, place, warp, lane);
        v.load(c, id, h, place, warp, lane);
        if (no_values(vs)) v.zero();   // (ahead of the keys' store: 48 registers, 56 after it; 2 x 1000 rows of 256 44.0, 45.4 us)
        k.store(to, warp, lane);
        v.store(to + Sh::OPER, warp, lane, values_over(vs));
        if (BITS == 8 && lane == 0 && warp < Sh::PIECES)
            put_scales(reinterpret_cast<float*>(operands + (size_t)room * H * 2 * Sh::OPER) + slot * 24, warp, ks, vs);
    }
}

template <int BITS, int DP, int PG, bool F32>
__global__ void __launch_bounds__(PROMPT_THREADS, 1) attend_prompt_kernel(const AttendArgs a, int tiles,
                                                                           float* __restrict__ partial,
                                                                           int* __restrict__ counters,
                                                                           const uint8_t* __restrict__ operands,
                                                                           int room, const int* __restrict__ at) {
    using Sh = PShape<DP, F32>;
    using E = std::conditional_t<F32, float, __nv_bfloat16>;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t* smem = (uint8_t*)(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
    constexpr int KT = Sh::KT, SPT = Sh::SPT;
    uint8_t* qs = smem;                              // [TILES][TERMS]
    uint8_t* kb = smem + Sh::TILES * Sh::TERMS * Sh::QOPER;   // [2]
    uint8_t* vb = kb + 2 * Sh::OPER;                 // [2]
    PTail& tl = *reinterpret_cast<PTail*>(vb + 2 * Sh::OPER);
    volatile int* abort_flag = &tl.abort_flag;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const CachePages& c = a.pages;
    const int H = c.heads, G = a.q_heads / H, D = c.dim;
    const int b = blockIdx.y, h = blockIdx.x % H, tile = tiles - 1 - blockIdx.x / H;   // the longest first
    const int part = blockIdx.z, item = blockIdx.y * gridDim.x + blockIdx.x;

    const SeqRec s = load_seq(a.step, c.page, b, a.status);
    const int R = s.rows * G, r0 = tile * Sh::ROWS;
    if (r0 >= R) return;
    const int rows = min(Sh::ROWS, R - r0);
    const bool two = rows > TILE;
    const int pos_lo = s.start + r0 / G, pos_hi = s.start + (r0 + rows - 1) / G;
    const int first = at ? at[b] : NOT_HERE;   // place of the sequence's tile 0 in the workspace
    const bool pre = first != NOT_HERE;
    // tokens [ta, tb), whole tiles wherever they are converted: the sums' order is the same
    int ta = first_seen(pos_lo, a.window) / KT * KT;
    int tb = pos_hi + 1;
    const int all = tb > ta ? (tb - ta + KT - 1) / KT : 0;
    const int parts = max(1, min((int)gridDim.z, all * KT / PART));
    if (part >= parts) return;
    if (parts > 1) {   // this CTA's part of them
        auto edge = [&](int z) { return ta + (all / parts * z + all % parts * z / parts) * KT; };   // all z / parts: past 2^31
        const int from = edge(part);
        tb = min(tb, edge(part + 1));
        ta = from;
    }
    const int nt = tb > ta ? (tb - ta + KT - 1) / KT : 0;      // conversions
    const int steps = tb > ta ? (tb - ta + STEP - 1) / STEP : 0;   // products

    if (tid == 0) {
        for (int i = 0; i < 2; ++i) {
            mbar_init(&tl.kfull[i], pre ? 1 : 32 * CONV);
            mbar_init(&tl.kempty[i], two ? 2 : 1);
            mbar_init(&tl.vfull[i], pre ? 1 : 32 * CONV);
            mbar_init(&tl.vempty[i], two ? 2 : 1);
            mbar_init(&tl.qfull[i], TILE);
            mbar_init(&tl.alldone[i], 1);
            for (int u = 0; u < 2; ++u) {
                mbar_init(&tl.sfull[i][u], 1);
                mbar_init(&tl.pfull[i][u], TILE);
                mbar_init(&tl.odone[i][u], 1);
            }
        }
        for (int i = 0; i < 4; ++i) mbar_init(&tl.scfull[i], pre ? 1 : Sh::PIECES);
        tl.abort_flag = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == SOFT + CONV) {
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

    if (warp >= SOFT) registers_down<REGS_REST>();
    if (warp < SOFT) {
        registers_up<REGS_SOFT>();
        // ---- softmax and output: a thread per row
        const int t = warp >> 2, q4 = warp & 3;
        const int rl = q4 * 32 + lane, r = r0 + t * TILE + rl;
        const bool live = r < R;
        // A warp's 32 rows lie 16 bytes to a lane: row and 16-byte chunk of its k-th access (of CH)
        constexpr int EPC = 16 / sizeof(E), CH = DP / EPC, PER = CH < 32 ? 32 / CH : 1;   // chunks per row, rows at a time
        auto row_at = [&](int k) { return q4 * 32 + k * PER + lane / CH; };
        const int chunk = lane % CH;
        auto place = [&](int row) {   // of the lane's chunk in tile t of the queries
            return qs + t * Sh::QOPER + chunk / 8 * (TILE * 128) + row * 128 + (((chunk & 7) ^ (row & 7)) << 4);
        };
        // the chunk's address in rows with the given strides, and from access k to the next
        const int rr0 = r0 + t * TILE + row_at(0), tok0 = quotient(a.group, rr0), g0 = rr0 - tok0 * G;
        const int per_tok = quotient(a.group, PER), per_g = PER - per_tok * G;
        struct Walk {
            int64_t at, step, wrap;
            int g;
        };
        auto walk = [&](int64_t row, int64_t head) {
            return Walk{(int64_t)(s.row0 + tok0) * row + (int64_t)(h * G + g0) * head + chunk * EPC, per_tok * row + per_g * head,
                        row - G * head, g0};
        };
        auto advance_row = [&](Walk& v) {
            v.at += v.step;
            v.g += per_g;
            if (v.g >= G) {
                v.g -= G;
                v.at += v.wrap;
            }
        };
        auto there = [&](int k) { return rr0 + k * PER < R && chunk * EPC < D; };
        if constexpr (F32) {
            // the queries below 1 by a power of two per row, as three bf16 terms; a row that is not
            // finite zeros under NaN statistics
            if (t == 0) {
                constexpr int BATCH = 8;   // rows' loads in flight
                Walk at = walk(a.q.row, a.q.head);
#pragma unroll 1
                for (int k0 = 0; k0 < 32 / PER; k0 += BATCH) {
                    uint4 w[BATCH];
#pragma unroll
                    for (int k = 0; k < BATCH; ++k) {
                        w[k] = there(k0 + k) ? *reinterpret_cast<const uint4*>((const E*)a.q.ptr + at.at) : make_uint4(0u, 0u, 0u, 0u);
                        advance_row(at);
                    }
#pragma unroll
                    for (int k = 0; k < BATCH; ++k) {
                        const uint32_t u[4] = {w[k].x, w[k].y, w[k].z, w[k].w};
                        uint32_t top = 0u;   // largest |bits| of the row (ordered like the values)
#pragma unroll
                        for (int e = 0; e < 4; ++e) top = max(top, u[e] & 0x7FFFFFFFu);
#pragma unroll
                        for (int d = 1; d < CH; d <<= 1) top = max(top, __shfl_xor_sync(~0u, top, d));
                        const bool fine = top < 0x7F800000u;
                        const int x = fine ? min(max((int)(top >> 23) - 126, -100), MOST_DOWN) : 0;
                        const float down = fine ? __uint_as_float((uint32_t)(127 - x) << 23) : 0.f;
                        float v[4];
#pragma unroll
                        for (int e = 0; e < 4; ++e) v[e] = fine ? __uint_as_float(u[e]) * down : 0.f;
                        const int row = row_at(k0 + k);
                        uint8_t* to = qs + chunk / 16 * (TILE * 128) + row * 128 + (((chunk % 16 / 2) ^ (row & 7)) << 4) + chunk % 2 * 8;
#pragma unroll
                        for (int z = 0; z < Sh::TERMS; ++z) {
                            const uint2 y = make_uint2(bf2_of(v[0], v[1]), bf2_of(v[2], v[3]));
                            *reinterpret_cast<uint2*>(to + z * Sh::QOPER) = y;
                            v[0] -= __uint_as_float(y.x << 16);
                            v[1] -= __uint_as_float(y.x & 0xFFFF0000u);
                            v[2] -= __uint_as_float(y.y << 16);
                            v[3] -= __uint_as_float(y.y & 0xFFFF0000u);
                        }
                        if (chunk == 0)
                            tl.qf[t][row] = fine ? a.scale * (1.4426950408889634f * __uint_as_float((uint32_t)(127 + x) << 23)) : NAN;
                    }
                }
                fence_proxy_async_smem();
                mbar_arrive(&tl.qfull[t]);
            }
        } else {
            // the queries as they are, but a row outside 2^+-64 brought below 1 by a power of two, and one
            // that is not finite zeros under NaN statistics
            tl.qf[t][rl] = a.scale * 1.4426950408889634f;
            if (Sh::TILES == 2 || t == 0) {
                Walk at = walk(a.q.row, a.q.head);
#pragma unroll 4
                for (int k = 0; k < 32 / PER; ++k) {
                    const bool in = there(k);   // (zeros elsewhere)
                    cp_async16_or_zero(smem_u32(place(row_at(k))), (const __nv_bfloat16*)a.q.ptr + (in ? at.at : 0), in);
                    advance_row(at);
                }
                cp_async_wait_all();
                __syncwarp();
                // largest |bits| of a chunk (ordered like the values)
                auto top_of = [](const uint4& w) {
                    const uint32_t u = __vmaxu2(__vmaxu2(w.x & 0x7FFF7FFFu, w.y & 0x7FFF7FFFu),
                                                __vmaxu2(w.z & 0x7FFF7FFFu, w.w & 0x7FFF7FFFu));
                    return max(u >> 16, u & 0xFFFFu);
                };
                bool wild = false;
#pragma unroll 4
                for (int k = 0; k < 32 / PER; ++k) {
                    const uint32_t top = top_of(*reinterpret_cast<const uint4*>(place(row_at(k))));
                    wild |= top != 0u && (top >> 7) - 63u > 128u;
                }
                if (__any_sync(~0u, wild)) {
#pragma unroll 1
                    for (int k = 0; k < 32 / PER; ++k) {
                        uint4* to = reinterpret_cast<uint4*>(place(row_at(k)));
                        const uint4 w = *to;
                        uint32_t top = top_of(w);
#pragma unroll
                        for (int d = 1; d < CH; d <<= 1) top = max(top, __shfl_xor_sync(~0u, top, d));
                        const bool fine = top < 0x7F80u;
                        const int x = fine ? min(max((int)(top >> 7) - 126, -100), MOST_DOWN) : 0;
                        const float down = fine ? __uint_as_float((uint32_t)(127 - x) << 23) : 0.f;
                        auto scaled = [&](uint32_t u) {
                            return fine ? bf2_of(__uint_as_float(u << 16) * down, __uint_as_float(u & 0xFFFF0000u) * down) : 0u;
                        };
                        *to = make_uint4(scaled(w.x), scaled(w.y), scaled(w.z), scaled(w.w));
                        if (chunk == 0)
                            tl.qf[t][row_at(k)] = fine ? a.scale * (1.4426950408889634f * __uint_as_float((uint32_t)(127 + x) << 23)) : NAN;
                    }
                }
                fence_proxy_async_smem();
                mbar_arrive(&tl.qfull[t]);
            }
        }
        __syncwarp();
        float qf = tl.qf[t][rl];
        const uint32_t lane_base = tmem + ((uint32_t)(q4 * 32) << 16);
        const uint32_t sbase = lane_base + t * TILE, obase = lane_base + Sh::O_AT + t * TILE;
        const int hi = s.start + r / G + 1, lo = first_seen(hi - 1, a.window);   // tokens [lo, hi) are seen
        // limits of the tile's rows, for the token tiles that no limit cuts
        const int rt = r0 + t * TILE;
        const int hi_min = s.start + rt / G + 1, hi_max = s.start + min(R - 1, rt + TILE - 1) / G + 1;
        const int lo_max = first_seen(hi_max - 1, a.window);
        float m = NO_MAX;
        // what the row's x's are divided by, a power of two (tl.qf holds their factor before that)
        auto divisor = [&]() { return __uint_as_float(__float_as_uint(tl.qf[t][rl]) - __float_as_uint(qf) + 0x3F800000u); };
        uint64_t l2 = pair(0.f, 0.f);
        bool ok = true;
        // 32 elements of the row, from 32 q on, times f, into the queries' place (the products that read
        // it are complete), and the warp's rows from there
        auto put32 = [&](const uint32_t (&x)[32], float f, int q) {
#pragma unroll
            for (int e = 0; e < 32; e += EPC) {
                uint32_t y[4];
#pragma unroll
                for (int z = 0; z < 4; ++z)
                    y[z] = F32 ? __float_as_uint(__uint_as_float(x[e + z]) * f)
                               : bf2_of(__uint_as_float(x[e + 2 * z % EPC]) * f, __uint_as_float(x[e + (2 * z + 1) % EPC]) * f);
                const int ch = (q * 32 + e) / EPC;
                *reinterpret_cast<uint4*>(qs + t * Sh::QOPER + ch / 8 * (TILE * 128) + rl * 128 + (((ch & 7) ^ (rl & 7)) << 4)) =
                    make_uint4(y[0], y[1], y[2], y[3]);
            }
        };
        auto put_rows = [&]() {
            __syncwarp();
            Walk at = walk(a.o.row, a.o.head);
#pragma unroll 4
            for (int k = 0; k < 32 / PER; ++k) {
                const uint4 y = *reinterpret_cast<const uint4*>(place(row_at(k)));
                if (there(k)) *reinterpret_cast<uint4*>((E*)a.o.ptr + at.at) = y;
                advance_row(at);
            }
        };
        // the row in its part's slot: O as [DP / 4][256 rows] of 16 bytes, then m and l
        float* slot = partial + ((size_t)item * gridDim.z + part) * PROMPT_SLOT;
        uint4* mine = reinterpret_cast<uint4*>(slot) + t * TILE + rl;
        float* ml = slot + DP * Sh::ROWS + t * TILE + rl;
        // fp32 rows: the tensor cores' sums cut off, so that O is taken out every FOLD steps and added,
        // rounded to nearest, to the row's sum of before, which waits in the output row (or the part's
        // slot) under the bound `under`
        float under = m;
        float* held = nullptr;
        const int group4 = parts == 1 ? 4 : 4 * Sh::ROWS;   // floats from 4 elements to the next
        if constexpr (F32) {
            const int tok = quotient(a.group, r), g = r - tok * G;
            held = parts == 1 ? (float*)a.o.ptr + (int64_t)(s.row0 + tok) * a.o.row + (int64_t)(h * G + g) * a.o.head : (float*)mine;
        }
        // 4 elements of that sum, times f
        auto held_at = [&](int k) { return live && (parts > 1 || k * 4 < D) ? reinterpret_cast<float4*>(held + k * group4) : nullptr; };
        // 32 elements of O, from 32 q on
        auto sum_of = [&](int q, uint32_t (&x)[32], bool more, float f) {
            uint32_t low[32];
            __syncwarp();
            tmem_ld32(obase + q * 32, x);
            tmem_ld32(obase + DP + q * 32, low);
            tmem_wait_ld();
            tmem_loaded(x);
            tmem_loaded(low);
#pragma unroll
            for (int e = 0; e < 32; e += 4) {
                const float4* p = held_at(q * 8 + e / 4);
                const float4 y = more && p ? *p : make_float4(0.f, 0.f, 0.f, 0.f);
                const float z[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    x[e + k] = __float_as_uint(fmaf(z[k], f, __uint_as_float(x[e + k]) + __uint_as_float(low[e + k])));
            }
        };
        if (t == 0 || two) {
            for (int i = 0; i < steps; ++i) {
                if constexpr (F32)
                    if (i > 0 && i % FOLD == 0) {   // (the wait: as where the bound moves, below)
                        ok = __all_sync(~0u, mbar_wait(&tl.odone[t][(i - 1) & 1], ((i - 1) >> 1) & 1, abort_flag, a.status));
                        if (!ok) break;
                        tc_fence_after();
#pragma unroll 1
                        for (int q = 0; q < DP / 32; ++q) {
                            uint32_t x[32];
                            sum_of(q, x, i > FOLD, ex2(under - m));
#pragma unroll
                            for (int e = 0; e < 32; e += 4)
                                if (float4* p = held_at(q * 8 + e / 4))
                                    *p = make_float4(__uint_as_float(x[e]), __uint_as_float(x[e + 1]), __uint_as_float(x[e + 2]),
                                                     __uint_as_float(x[e + 3]));
                        }
                        under = m;
                    }
                // (the look at the scales' barrier is under way during the wait for the scores)
                const bool scales = BITS == 4 || i % SPT != 0 || mbar_done(&tl.scfull[i / SPT & 3], i / SPT >> 2 & 1);
                ok = mbar_wait(&tl.sfull[t][i & 1], (i >> 1) & 1, abort_flag, a.status);
                if (!scales) ok = ok && mbar_wait(&tl.scfull[i / SPT & 3], i / SPT >> 2 & 1, abort_flag, a.status);
                ok = __all_sync(~0u, ok);
                if (!ok) break;
                tc_fence_after();
                const float* sc = tl.scales[i / SPT & 3] + i % SPT * 4;
                const int t0 = ta + i * STEP;
                const bool edge = t0 + STEP > hi_min || t0 < lo_max;
                const uint32_t sat = sbase + (i & 1) * STEP;
                uint32_t y[STEP];
                // P (of fp32 rows its first term) over the scores
                auto put_weights = [&](float2 sum) {
                    l2 = add2(l2, pair(sum.x, sum.y));
                    tmem_st32(sat, y);
                    tmem_wait_st();
                };
                const uint32_t pat = lane_base + Sh::P_AT + (i & 1) * Sh::P_COLS;
                // with the bound so far, which usually holds; else the bound moves.  The usual step has a
                // path of its own: joined with the other's, it took 70 moves of registers (5% of the time).
                bool above = true, done = false;
                if (!edge && i > 0) {
                    float2 sum;
                    if constexpr (F32) sum = unpair(weigh3<false, PG, BITS == 4>(sat, pat, sc, qf, m, 0, 0, y));
                    else sum = unpair(weigh<false, PG, BITS == 4>(sat, sc, qf, m, 0, 0, y));
                    above = sum.x + sum.y > MOST;
                    done = !__any_sync(~0u, above);
                    if (done) put_weights(sum);
                }
                for (bool move = !edge || i == 0; !done; move = true) {
                    if (move) {
                        // (fp32 rows: the lower terms of weights that are dropped land before the next ones')
                        if constexpr (F32) tmem_wait_st();
                        const float q = tl.qf[t][rl], up = divisor(), was = m * up;
                        const float mx = row_max<BITS == 4>(sat, sc, q, lo - t0, hi - t0);
                        const float now = above ? fmaxf(mx, was) : was, f = ex2(was - now);
                        const uint32_t far = max((__float_as_uint(now) >> 23 & 0xFFu), 126u + FAR) - (126u + FAR);
                        const float down = now == NO_MAX ? 1.f : __uint_as_float((127u - far) << 23);
                        m = now * down;
                        qf = q * down;
                        if constexpr (F32) under *= up * down;
                        l2 = mul2(l2, pair(f, f));
                        if (i > 0) {
                            // O, once the last step's product is complete (the one before it is: these
                            // scores came after it, so the barrier is at this phase or past it)
                            ok = __all_sync(~0u, mbar_wait(&tl.odone[t][(i - 1) & 1], ((i - 1) >> 1) & 1, abort_flag, a.status));
                            if (!ok) break;
                            tc_fence_after();
#pragma unroll 1
                            for (int q = 0; q < Sh::O_COLS / 16; ++q) {
                                uint32_t x[16];
                                tmem_ld16(obase + q * 16, x);
                                tmem_wait_ld();
                                tmem_loaded16(x);
#pragma unroll
                                for (int e = 0; e < 16; ++e) x[e] = __float_as_uint(__uint_as_float(x[e]) * f);
                                tmem_st16(obase + q * 16, x);
                            }
                        }
                    }
                    float2 sum;
                    if constexpr (F32) sum = unpair(weigh3<true, PG, BITS == 4>(sat, pat, sc, qf, m, lo - t0, hi - t0, y));
                    else sum = unpair(weigh<true, PG, BITS == 4>(sat, sc, qf, m, lo - t0, hi - t0, y));
                    above = sum.x + sum.y > MOST;
                    done = move || !__any_sync(~0u, above);
                    if (done) put_weights(sum);
                }
                if (!ok) break;
                tc_fence_before();
                mbar_arrive(&tl.pfull[t][i & 1]);
            }
            if (ok && steps > 0) ok = mbar_wait(&tl.odone[t][(steps - 1) & 1], ((steps - 1) >> 1) & 1, abort_flag, a.status);
            __syncwarp();
            tc_fence_after();
            const float2 ls = unpair(l2);
            const float l = ls.x + ls.y, inv = parts > 1 ? 1.f : l == 0.f ? 0.f : (BITS == 4 ? c.v_unit : 1.f) / l;
#pragma unroll
            for (int q = 0; q < DP / 32; ++q) {
                uint32_t x[32];
                if (nt > 0) {
                    if constexpr (F32) sum_of(q, x, steps > FOLD, ex2(under - m));
                    else {
                        __syncwarp();
                        tmem_ld32(obase + q * 32, x);
                        tmem_wait_ld();
                        tmem_loaded(x);
                    }
                } else {
#pragma unroll
                    for (int e = 0; e < 32; ++e) x[e] = 0u;
                }
                if (parts == 1) put32(x, inv, q);
                else if (live)
#pragma unroll
                    for (int e = 0; e < 32; e += 4)
                        mine[(q * 8 + e / 4) * Sh::ROWS] = make_uint4(x[e], x[e + 1], x[e + 2], x[e + 3]);
            }
            if (parts == 1) put_rows();
            else if (live) {
                ml[0] = m * divisor();
                ml[Sh::ROWS] = l;
            }
        }
        if (parts > 1) {
            // the last CTA to finish joins the row tile's parts (release and acquire for all its
            // softmax threads, around their barrier)
            soft_sync();
            if (tid == 0) {
                int seen;
                asm volatile("atom.acq_rel.gpu.global.add.s32 %0, [%1], 1;" : "=r"(seen) : "l"(counters + item) : "memory");
                tl.last = seen == parts - 1;
                if (tl.last) counters[item] = 0;
            }
            soft_sync();
            if (tl.last && (t == 0 || two)) {   // (a dead row's slot holds what it holds: nothing of it is stored)
                const size_t next = PROMPT_SLOT / 4;   // from a part to the next, in 16 bytes
                const uint4* first4 = mine - part * next;
                const float* first_ml = ml - (size_t)part * PROMPT_SLOT;
                float top = NO_MAX, sum = 0.f;
                for (int z = 0; z < parts; ++z) top = fmaxf(top, __ldcg(first_ml + (size_t)z * PROMPT_SLOT));
                for (int z = 0; z < parts; ++z) {
                    const float* p = first_ml + (size_t)z * PROMPT_SLOT;
                    sum = fmaf(__ldcg(p + Sh::ROWS), ex2(__ldcg(p) - top), sum);
                }
                const float inv = sum == 0.f ? 0.f : (BITS == 4 ? c.v_unit : 1.f) / sum;
#pragma unroll 1
                for (int q = 0; q < DP / 32; ++q) {
                    float o[32] = {};
#pragma unroll 1
                    for (int z = 0; z < parts; ++z) {
                        const float f = ex2(__ldcg(first_ml + (size_t)z * PROMPT_SLOT) - top);
                        uint4 y[8];
#pragma unroll
                        for (int e = 0; e < 8; ++e) y[e] = __ldcg(first4 + z * next + (q * 8 + e) * Sh::ROWS);
#pragma unroll
                        for (int e = 0; e < 8; ++e) {
                            o[4 * e] = fmaf(__uint_as_float(y[e].x), f, o[4 * e]);
                            o[4 * e + 1] = fmaf(__uint_as_float(y[e].y), f, o[4 * e + 1]);
                            o[4 * e + 2] = fmaf(__uint_as_float(y[e].z), f, o[4 * e + 2]);
                            o[4 * e + 3] = fmaf(__uint_as_float(y[e].w), f, o[4 * e + 3]);
                        }
                    }
                    uint32_t x[32];
#pragma unroll
                    for (int e = 0; e < 32; ++e) x[e] = __float_as_uint(o[e]);
                    put32(x, inv, q);
                }
                put_rows();
            }
        }
    } else if (warp < SOFT + CONV && pre) {
        // ---- copies of converted tiles
        if (warp == SOFT) {
            int done = 0;
            for (int j = 0; j < nt; ++j) {
                const uint32_t use = (j >> 1) & 1;
                const size_t slot = (size_t)(first + ta / KT + j) * H + h;
                const uint8_t* from = operands + slot * 2 * Sh::OPER;
                const float* scales = reinterpret_cast<const float*>(operands + (size_t)room * H * 2 * Sh::OPER) + slot * 24;
                const float sc = BITS == 8 && lane < 24 ? scales[lane] : 0.f;
                if (!__all_sync(~0u, mbar_wait(&tl.kempty[j & 1], use ^ 1, abort_flag, a.status))) break;
                if (BITS == 8 && lane < 24) tl.scales[j & 3][lane] = sc;
                __syncwarp();
                if (lane == 0) {
                    if (BITS == 8) mbar_arrive(&tl.scfull[j & 3]);
                    mbar_expect_tx(&tl.kfull[j & 1], Sh::OPER);
                    bulk_g2s(kb + (j & 1) * Sh::OPER, from, Sh::OPER, &tl.kfull[j & 1]);
                }
                done = 2 * j + 1;
                if (!__all_sync(~0u, mbar_wait(&tl.vempty[j & 1], use ^ 1, abort_flag, a.status))) break;
                if (lane == 0) {
                    mbar_expect_tx(&tl.vfull[j & 1], Sh::OPER);
                    bulk_g2s(vb + (j & 1) * Sh::OPER, from + Sh::OPER, Sh::OPER, &tl.vfull[j & 1]);
                }
                done = 2 * j + 2;
            }
            // copies in flight land before the CTA goes: each barrier's last phase
            for (int i = 0; i < 4; ++i) {
                const int copies = (done + 1 - (i >> 1)) / 2;          // of keys or values
                const int n = (copies + 1 - (i & 1)) / 2;              // through this buffer
                uint64_t* bar = (i >> 1 ? tl.vfull : tl.kfull) + (i & 1);
                const long long t0 = clock64();
                while (n > 0 && !mbar_try_wait(bar, (n - 1) & 1) && clock64() - t0 < 200000000ll) {
                }
            }
        }
    } else if (warp < SOFT + CONV) {
        // ---- conversion: the warp's 16 tokens of each tile
        const int w = warp - SOFT;
        // the warp's tokens of the tile that is loaded next: block and place in the sequence's table
        int tk = ta + Piece<BITS, DP, false>::piece(w) * 16, blk = tk / c.page, place = tk % c.page;
        const int dblk = KT / c.page, dplace = KT % c.page;
        auto next_id = [&]() { return tk < tb ? load_page(a.step, c, b, blk, a.status) : -1; };   // -1: nothing to read
        auto advance = [&]() {
            tk += KT;
            blk += dblk;
            place += dplace;
            if (place >= c.page) place -= c.page, ++blk;
        };
        auto scale = [&](const float* p, int id) { return BITS == 4 ? 1.f : id >= 0 ? p[(size_t)id * H + h] : 0.f; };
        Piece<BITS, DP, false> k;
        Piece<BITS, DP, true> v;
        int id = blk >= first_seen(pos_lo, a.window) / c.page ? next_id() : -1;   // (pages that no row sees: of the first tile)
        k.load(c, id, h, place, w, lane);
        v.load(c, id, h, place, w, lane);
        float ks = scale(c.k_scale, id), vs = scale(c.v_scale, id);
        advance();
        id = next_id();
        for (int j = 0; j < nt; ++j) {
            const uint32_t use = (j >> 1) & 1;
            if (!mbar_wait(&tl.kempty[j & 1], use ^ 1, abort_flag, a.status)) break;
            if (BITS == 8 && lane == 0 && (Sh::PIECES == CONV || w < Sh::PIECES)) {
                put_scales(tl.scales[j & 3], w, ks, vs);
                mbar_arrive(&tl.scfull[j & 3]);
            }
            k.store(kb + (j & 1) * Sh::OPER, w, lane);
            fence_proxy_async_smem();
            mbar_arrive(&tl.kfull[j & 1]);
            k.load(c, id, h, place, w, lane);
            if (!mbar_wait(&tl.vempty[j & 1], use ^ 1, abort_flag, a.status)) break;
            if (no_values(vs)) v.zero();
            v.store(vb + (j & 1) * Sh::OPER, w, lane, values_over(vs));
            fence_proxy_async_smem();
            mbar_arrive(&tl.vfull[j & 1]);
            v.load(c, id, h, place, w, lane);
            ks = scale(c.k_scale, id);
            vs = scale(c.v_scale, id);
            advance();
            id = next_id();
        }
    } else if (steps > 0 && (warp == SOFT + CONV || (two && warp == SOFT + CONV + 1))) {
        // ---- products of a tile: a step's scores go ahead of the last step's weights
        const int t = warp - SOFT - CONV;
        const uint32_t idesc_s = idesc_bf16(TILE, STEP), idesc_o = idesc_bf16(TILE, DP) | (1u << 16);   // (O: B column-major)
        const uint64_t dq = sdesc(smem_u32(qs + t * Sh::QOPER), 1024, SW128), dk = sdesc(smem_u32(kb), 1024, SW128),
                       dv = sdesc_lbo(smem_u32(vb), KT * 128, 1024, SW128);
        const uint32_t tm = tmem + t * TILE;
        // operand tile of step i, and the step's 64 rows (tokens) of it
        auto half_of = [](int i) { return (uint64_t)((i / SPT & 1) * (Sh::OPER >> 4) + i % SPT * (STEP * 128 >> 4)); };
        auto ends = [&](int i) { return i % SPT == SPT - 1 || i + 1 == steps; };   // step i is its token tile's last
        auto wait = [&](uint64_t* bar, int parity) {
            return __all_sync(~0u, mbar_wait(bar, parity, abort_flag, a.status));
        };
        auto scores = [&](int i) {
#pragma unroll
            for (int z = Sh::TERMS - 1; z >= 0; --z)   // (the smallest first: fewer sums of the full size)
                product_ss<DP / 16, KT>(tm + (i & 1) * STEP, dq + z * (Sh::QOPER >> 4), dk + half_of(i), idesc_s,
                                        z < Sh::TERMS - 1);
            mma_commit(&tl.sfull[t][i & 1]);
            if (ends(i)) mma_commit(&tl.kempty[i / SPT & 1]);
        };
        // steps 0 and 1 have a score buffer each; from then on a step's values free the buffer of
        // the scores two steps on
        bool ok = wait(&tl.qfull[t], 0) && wait(&tl.kfull[0], 0);
        if (SPT == 1 && steps > 1) ok = ok && wait(&tl.kfull[1], 0);
        tc_fence_after();
        if (ok && elect_one()) {
            scores(0);
            if (steps > 1) scores(1);
        }
        __syncwarp();
        for (int i = 0; ok && i < steps; ++i) {
            if (i % SPT == 0) {   // operand tiles of this step's values and of the scores two steps on
                const int j = (i + 2) / SPT;
                ok = wait(&tl.vfull[i / SPT & 1], i / SPT >> 1 & 1);
                if (ok && i + 2 < steps) ok = wait(&tl.kfull[j & 1], j >> 1 & 1);
            }
            ok = ok && wait(&tl.pfull[t][i & 1], (i >> 1) & 1);
            if (!ok) break;
            tc_fence_after();
            if (elect_one()) {
                product_ts<STEP / 16>(tm + Sh::O_AT, tm + (i & 1) * STEP, dv + half_of(i), idesc_o,
                                      F32 ? i % FOLD > 0 : i > 0);
#pragma unroll
                for (int z = 0; z < Sh::TERMS - 1; ++z)
                    product_ts<STEP / 16>(tm + Sh::O_AT + DP, tm + Sh::P_AT + (i & 1) * Sh::P_COLS + z * (STEP / 2),
                                          dv + half_of(i), idesc_o, i % FOLD > 0 || z > 0);
                mma_commit(&tl.odone[t][i & 1]);
                if (ends(i)) mma_commit(&tl.vempty[i / SPT & 1]);
                if (i + 2 < steps) scores(i + 2);
            }
            __syncwarp();
        }
        if (elect_one()) mma_commit(&tl.alldone[t]);
        __syncwarp();
        const long long t0 = clock64();   // the products are complete before the CTA goes
        while (!mbar_try_wait(&tl.alldone[t], 0) && clock64() - t0 < 200000000ll) {
        }
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    if (warp == SOFT + CONV) {
        __syncwarp();
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512) : "memory");
    }
}

template <int BITS, int DP, int PG, bool F32>
cudaError_t launch(const AttendArgs& a, const AttendWs& ws, cudaStream_t st) {
    using Sh = PShape<DP, F32>;
    const long long rows = (long long)a.step.max_new * (a.q_heads / a.pages.heads);
    const int tiles = (int)((rows + Sh::ROWS - 1) / Sh::ROWS);
    const int room = (int)(ws.operand_bytes / ((size_t)a.pages.heads * (2 * Sh::OPER + 96)));
    const bool pre = tiles > PRE_TILES && room > 0;
    if (pre) {
        // a few thousand warps in all, as many blocks for each sequence
        const int blocks = a.step.n_seqs >= 8 * ws.sms ? 1 : (8 * ws.sms + a.step.n_seqs - 1) / a.step.n_seqs;
        convert_kernel<BITS, DP, F32><<<dim3(blocks, a.step.n_seqs), PRE_THREADS, 0, st>>>(a, ws.operands, room, ws.operand_at);
        const cudaError_t e = cudaGetLastError();
        if (e != cudaSuccess) return e;
    }
    // fewer row tiles than half the SMs: as many parts of each as give every SM a CTA
    const long long ctas = (long long)tiles * a.pages.heads * a.step.n_seqs;
    const int parts = ctas * 2 <= ws.sms ? (int)(ws.sms / ctas) : 1;
    const dim3 grid((unsigned)tiles * a.pages.heads, a.step.n_seqs, parts);
    attend_prompt_kernel<BITS, DP, PG, F32><<<grid, PROMPT_THREADS, Sh::SMEM, st>>>(
        a, tiles, ws.partial, ws.counters, ws.operands, room, pre ? ws.operand_at : nullptr);
    return cudaGetLastError();
}

}  // namespace

template <int BITS, int DP, bool F32>
static cudaError_t init() {
    constexpr int bytes = PShape<DP, F32>::SMEM;
    cudaError_t e = cudaFuncSetAttribute(attend_prompt_kernel<BITS, DP, STEP, F32>, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (BITS == 8 && e == cudaSuccess)
        e = cudaFuncSetAttribute(attend_prompt_kernel<8, DP, 16, F32>, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    return e;
}
template <int BITS>
static cudaError_t init_shapes() {
    cudaError_t e = init<BITS, 64, false>();
    if (e == cudaSuccess) e = init<BITS, 128, false>();
    if (e == cudaSuccess) e = init<BITS, 256, false>();
    if (e == cudaSuccess) e = init<BITS, 64, true>();
    if (e == cudaSuccess) e = init<BITS, 128, true>();
    return e;
}

cudaError_t attend_prompt_init(int bits) { return bits == 4 ? init_shapes<4>() : init_shapes<8>(); }

template <int DP>
static size_t operand_bytes(const CachePages& c, long long tokens) {
    return (size_t)((tokens + PShape<DP>::KT - 1) / PShape<DP>::KT) * c.heads * (2 * PShape<DP>::OPER + 96);
}

size_t attend_prompt_bytes(const CachePages& c, long long tokens) {
    return c.dim <= 64 ? operand_bytes<64>(c, tokens) : c.dim <= 128 ? operand_bytes<128>(c, tokens) : operand_bytes<256>(c, tokens);
}

// From 17 rows of a sequence and head on (fp32 rows of more than 128 elements excepted: their
// terms outgrow shared memory).  32/8 heads after 4000 tokens (2000 where they are 64 sequences), this
// kernel against attend_split.cu, for 1, 16 and 64 sequences: bf16 rows at 6 tokens 25, 60, 127 us
// against 22, 79, 145, at 4 tokens 25, 61, 127 against 22, 46, 81; fp32 rows at 6 tokens 38, 133, 267
// against 49, 140, 255, at 12 tokens 134 against 243 (16 sequences), at 4 tokens 35, 100, 220 against
// 24, 59, 104.  The rule knows neither the number of sequences nor the type: it costs one sequence of
// bf16 rows 3 us and 64 of fp32 rows 12 us at 6 tokens.  Over 4 bits it is the same rule, this kernel against
// attend4_split.cu, for 1 (after 5000), 16 (after 4000) and 64 (after 1000) sequences: bf16 rows at 5 tokens
// 27, 55, 73 us against 21, 54, 63, at 12 tokens 27, 56, 75 against 25, 74, 84; fp32 rows at 5 tokens 39, 115, 136
// against 25, 77, 86, at 12 tokens 39, 117, 142 against 30, 106, 119, at 16 tokens 39, 119, 144 against 25, 135, 153:
// from 17 to 32 rows fp32 rows pay up to 60%, bf16 rows of heads of 256 50% (160 against 106 us).
bool attend_prompt_takes(bool bf16, const AttendArgs& a) {
    return (bf16 || a.pages.dim <= 128) && (long long)a.step.max_new * (a.q_heads / a.pages.heads) > 16;
}

template <int BITS, int PG>
static cudaError_t launch_by_dim(bool bf16, const AttendArgs& a, const AttendWs& ws, cudaStream_t st) {
    const int D = a.pages.dim;
    if (!bf16) return D <= 64 ? launch<BITS, 64, PG, true>(a, ws, st) : launch<BITS, 128, PG, true>(a, ws, st);
    return D <= 64 ? launch<BITS, 64, PG, false>(a, ws, st)
                   : D <= 128 ? launch<BITS, 128, PG, false>(a, ws, st) : launch<BITS, 256, PG, false>(a, ws, st);
}

cudaError_t launch_attend_prompt(bool bf16, const AttendArgs& a, const AttendWs& ws, cudaStream_t st) {
    if (a.pages.blocks) return launch_by_dim<4, STEP>(bf16, a, ws, st);
    return a.pages.page % STEP ? launch_by_dim<8, 16>(bf16, a, ws, st) : launch_by_dim<8, STEP>(bf16, a, ws, st);
}

}  // namespace mlora
