// paged.cuh -- what the paged cache's sources share: error bits, argument checks, types.
#pragma once

#include <cmath>
#include <type_traits>

#include "common.cuh"
#include "dfl.h"

namespace dfl {

// error bits (dfl_paged.err)
constexpr int kPgCapacity = 1, kPgState = 2, kPgArg = 4, kPgTimeout = 8;
constexpr int kPgMaxGroup = 16;          // query heads per key/value head
constexpr int kPgMaxRows = 1 << 30;      // rows of a call's buffers, tokens of a pool or a sequence: places some tiles behind the last one are numbers too
constexpr int64_t kPgMaxLd = 1 << 22;    // elements between rows: what a tile of 128 rows spans fits 31 bits of bytes

inline bool pg_aligned(const void *p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

inline int pg_check(const dfl_paged *c) {
    if (!c || c->n_seq < 1 || c->n_seq > DFL_PAGED_MAX_SEQ || c->n_kv < 1 || c->n_kv > 1024 || c->n_pages < 1 || c->max_pages < 1)
        return DFL_E_INVALID_ARG;
    if (c->head_dim != 64 && c->head_dim != 128 && c->head_dim != 256) return DFL_E_UNSUPPORTED;
    if (c->page != 16 && c->page != 32 && c->page != 64 && c->page != 128) return DFL_E_UNSUPPORTED;
    if (c->type != DFL_BF16 && c->type != DFL_F16) return DFL_E_UNSUPPORTED;
    if ((int64_t)c->n_pages * c->page > kPgMaxRows || (int64_t)c->max_pages * c->page > kPgMaxRows) return DFL_E_INVALID_ARG;
    if (!c->k || !c->v || !pg_aligned(c->k, 16) || !pg_aligned(c->v, 16)) return DFL_E_INVALID_ARG;
    const void *p[] = {c->table, c->held, c->ring, c->queue, c->err};
    for (const void *q : p)
        if (!q || !pg_aligned(q, 4)) return DFL_E_INVALID_ARG;
    return DFL_OK;
}

inline int pg_check_rows(const dfl_paged *c, const void *p, int64_t ld, int heads) {
    if (!p || !pg_aligned(p, 16) || ld % 8 || ld < (int64_t)heads * c->head_dim) return DFL_E_INVALID_ARG;
    return ld <= kPgMaxLd ? DFL_OK : DFL_E_UNSUPPORTED;
}

// Whether two ranges of bytes, or two sets of rows [n][width] of 16-bit numbers, share memory. Rows the same distance apart may lie in
// the gaps between each other; others are taken for overlapping where their whole ranges do.
inline bool pg_overlap(const void *p, int64_t n, const void *q, int64_t m) {
    const uintptr_t x = reinterpret_cast<uintptr_t>(p), y = reinterpret_cast<uintptr_t>(q);
    return p && q && n && m && x < y + uintptr_t(m) && y < x + uintptr_t(n);
}
inline bool pg_rows_overlap(const void *p, int64_t ldp, int64_t wp, const void *q, int64_t ldq, int64_t wq, int64_t n) {
    if (!pg_overlap(p, ((n - 1) * ldp + wp) * 2, q, ((n - 1) * ldq + wq) * 2)) return false;
    if (ldp != ldq) return true;
    const uintptr_t x = reinterpret_cast<uintptr_t>(p), y = reinterpret_cast<uintptr_t>(q);
    const int64_t off = int64_t((x < y ? y - x : x - y) / 2) % ldp;              // of the later one's rows in the earlier one's
    return off < (x < y ? wp : wq) || off + (x < y ? wq : wp) > ldp;
}

inline int pg_check_heads(const dfl_paged *c, int n_q, int window, float scale) {
    if (n_q < 1 || n_q % c->n_kv || window < 0 || !(scale > 0) || !std::isfinite(scale * 1.5f)) return DFL_E_INVALID_ARG;
    return n_q / c->n_kv > kPgMaxGroup ? DFL_E_UNSUPPORTED : DFL_OK;
}

inline int pg_shift(const dfl_paged *c) {
    int shift = 4;
    while (1 << shift < c->page) ++shift;
    return shift;
}

inline int pg_launched(cudaError_t e) { return e == cudaSuccess ? DFL_OK : DFL_E_CUDA; }

__device__ __forceinline__ void pg_report(int *err, int bits) {
    if (bits) atomicOr(err, bits);
}

// ---- what both attentions use -------------------------------------------------------------------------
__device__ __forceinline__ float exp2_fast(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// two numbers rounded to the type, the first in the low half
template <typename T>
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
    if constexpr (std::is_same<T, __nv_bfloat16>::value) {
        const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
        return *reinterpret_cast<const uint32_t *>(&v);
    } else {
        const __half2 v = __floats2half2_rn(lo, hi);
        return *reinterpret_cast<const uint32_t *>(&v);
    }
}

// 16 bytes into shared memory, asynchronously, or zeros
__device__ __forceinline__ void cp_async16_or_zeros(unsigned to, const void *from, bool there) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to), "l"(from), "r"(there ? 16 : 0) : "memory");
}

// Arguments of both attentions
struct PagedAttnArgs {
    dfl_paged c;
    const void *q, *k, *v;     // k, v: packed rows of prompts; the pages are c.k, c.v
    void *out;
    int64_t ldq, ldk, ldv, ldo;
    int n_q, group, total;     // rows of the packed buffers
    const int32_t *cu, *len;
    int rows, window, causal;
    int shift;                 // page = 1 << shift
    int inverse;               // r / group is (r * inverse) >> 12 for r < 256
    float scale_log2;          // scale * log2(e): weights are powers of two
    int stall;                 // dfl_paged_test_stall
};

// a DFL_* code each
int launch_paged_prompt(const PagedAttnArgs &a, cudaStream_t s);                 // prompt.cu
int launch_paged_attn(const PagedAttnArgs &a, void *scratch, cudaStream_t s);    // pagedattn.cu
size_t paged_attn_scratch(const dfl_paged *c, int n_q, int rows);

}  // namespace dfl
