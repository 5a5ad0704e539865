// Key/value cache in 8 bits (int8 pages, one fp32 scale per page and head) and the
// attention over it: declarations shared by cache.cu, cache_store.cu and attend*.cu.
#pragma once
#include <cuda.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "internal.h"

namespace mlora {

constexpr float TINY_SCALE = 0x1p-120f;   // codes under a smaller scale are 0 (1 / s stays finite above)

// The caller's pages: codes [n_pages][heads][page][dim], scales [n_pages][heads].
struct CachePages {
    int8_t* k_codes;
    int8_t* v_codes;
    float* k_scale;
    float* v_scale;
    int n_pages, page, heads, dim;
};

// One step's rows, lengths and page table (see include/mlora.h).
struct CacheStep {
    const int32_t* offsets;   // NULL: one row per sequence
    const int32_t* lengths;
    const int32_t* pages;
    int n_seqs, width, T, max_new;
};

// Rows [T][heads][dim] with element strides.
template <typename P>
struct RowsOf {
    P ptr;
    int64_t row, head;
};
using RowsIn = RowsOf<const void*>;
using RowsOut = RowsOf<void*>;

// n / d for 0 <= n < 2^31 by a multiplication: with 2^(s-1) < d <= 2^s and
// mul = ceil(2^(31+s) / d), n mul exceeds n 2^(31+s) / d by less than 2^(31+s) / d.
struct Divide {
    uint32_t mul;   // 0: d = 1
    int shift;
    int d;
};
inline Divide divide_by(int d) {
    int s = 0;
    while ((1ll << s) < d) ++s;
    if (s == 0) return Divide{0u, 0, 1};
    return Divide{(uint32_t)(((1ull << (31 + s)) + d - 1) / d), s - 1, d};
}

// One sequence of a step, checked: rows row0 .. row0 + rows - 1 are processed and lie at
// positions start, start + 1, ... (start may be negative), of `len` tokens held.
struct SeqRec {
    int row0, rows, start, len;
};

#ifdef __CUDACC__
__device__ __forceinline__ int quotient(const Divide& v, int n) {
    return v.mul ? (int)(__umulhi((uint32_t)n, v.mul) >> v.shift) : n;
}
__device__ __forceinline__ SeqRec load_seq(const CacheStep& s, int page, int b, uint32_t* status) {
    SeqRec r;
    int n = 1;
    r.row0 = b;
    bool bad = false;
    if (s.offsets) {
        const int o0 = s.offsets[b], o1 = s.offsets[b + 1];
        r.row0 = o0;
        n = o1 - o0;
        if (o0 < 0 || o1 < o0 || o1 > s.T) {
            r.row0 = 0;
            n = 0;
            bad = true;
        }
    }
    const int len = s.lengths[b];
    const long long cap = (long long)s.width * page;
    r.len = len < 0 ? 0 : (len > cap ? (int)cap : len);
    bad |= r.len != len;
    r.start = r.len - n;
    r.rows = n < s.max_new ? n : s.max_new;
    bad |= r.rows != n;
    if (bad) atomicOr(status, STATUS_BAD_STEP);
    return r;
}

// Page of block j of sequence b, -1 (and the status bit) if it is out of range.
__device__ __forceinline__ int load_page(const CacheStep& s, const CachePages& c, int b, int j, uint32_t* status) {
    const int id = s.pages[(size_t)b * s.width + j];
    if (id >= 0 && id < c.n_pages) return id;
    atomicOr(status, STATUS_BAD_STEP);
    return -1;
}

// First token that a row at position pos sees; window 0: all of them.  (A difference is taken only
// where it is not negative: pos reaches -2^31, and the window 2^31 - 1.)
__device__ __forceinline__ int first_seen(int pos, int window) {
    return window > 0 && pos >= window ? pos - window + 1 : 0;
}
#endif

struct AttendArgs {
    CachePages pages;
    CacheStep step;
    RowsIn q;
    RowsOut o;
    int q_heads;
    Divide page, group;   // by pages.page, by query heads per key/value head
    float scale;
    int window;
    uint32_t* status;
};

cudaError_t launch_append(bool bf16, const CachePages& c, const CacheStep& s, const RowsIn& k, const RowsIn& v,
                          uint32_t* status, cudaStream_t st);
cudaError_t launch_read(bool bf16, const CachePages& c, const CacheStep& s, const RowsOut& k, const RowsOut& v,
                        uint32_t* status, cudaStream_t st);

}  // namespace mlora
