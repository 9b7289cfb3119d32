// kv8.cu -- a key/value cache in 8 bits (include/dfl.h, dfl_kv8): rows in, attention over it, eviction by
// accumulated attention weight, rows out.
//
// A block is 32 tokens of one key/value head. Its keys (and, apart from them, its values) share one fp32
// scale: value = (code - 128) * scale with |code - 128| <= 127, so a value is off by at most scale / 2 =
// amax / 254. The newest tokens stay fp32 in a tail of 48 rows until their block is complete and
// committed: 31 tokens of an open block and the 16 rows of a verify fit, and rolling rows back is index
// arithmetic. Code layouts follow the attention's matrix fragments (keys in chunks of 64 along the head
// dimension, values with the tokens innermost).
#include <algorithm>
#include <cmath>
#include <type_traits>

#include "common.cuh"
#include "dfl.h"

namespace dfl {
namespace {

constexpr int kBlk = DFL_KV8_BLOCK;
constexpr int kTail = DFL_KV8_TAIL;
constexpr int kMaxGroup = 16;            // query heads per key/value head
// error bits (dfl_kv8.err)
constexpr int kErrCapacity = 1, kErrState = 2, kErrTable = 4;

struct KvView {                          // one head of one sequence
    uint8_t *k, *v;
    float *ks, *vs, *kt, *vt, *score;
    const int32_t *table;
    int32_t *sealed;
    int nb;
};

__device__ __forceinline__ KvView view(const dfl_kv8 &c, int s, int h) {
    const size_t u = (size_t)s * c.n_kv + h, blk = (size_t)kBlk * c.head_dim;
    KvView w;
    w.k = c.k + u * c.n_blocks * blk;
    w.v = c.v + u * c.n_blocks * blk;
    w.ks = c.k_scale + u * c.n_blocks;
    w.vs = c.v_scale + u * c.n_blocks;
    w.kt = c.k_tail + u * kTail * c.head_dim;
    w.vt = c.v_tail + u * kTail * c.head_dim;
    w.table = c.table + u * c.n_blocks;
    w.score = c.score ? c.score + u * c.n_blocks : nullptr;
    w.sealed = c.sealed + u;
    w.nb = c.n_blocks;
    return w;
}

// code offsets inside a block: token t, channel d
__host__ __device__ __forceinline__ int k_at(int t, int d) { return ((d >> 6) * kBlk + t) * 64 + (d & 63); }
__host__ __device__ __forceinline__ int v_at(int t, int d) { return d * kBlk + t; }

__device__ __forceinline__ float expand(uint8_t c, float scale) { return float(int(c) - 128) * scale; }

__device__ __forceinline__ int rows_of(const int32_t *cnt, int s, int rows) {
    return cnt ? min(max(cnt[s], 0), rows) : rows;
}

// The codes of x at `scale` >= kTiny, 128 + the integer nearest to x / scale, exactly: in the low byte of each result. With
// inv = 1 / scale rounded, x inv is off by at most 127 2^-24 < 2^-17. Adding 1.5 * 2^23 + 128 rounds it to an integer c; the
// rest f = x inv - c, rounded once, tells where c might not be the nearest: |f| > 1/2 - 2^-15, for one value in some 16,000.
// There c is off by one at most, and the remainder r = x - c scale, which is exact in fp32 (it is a multiple of the smaller
// unit in the last place of x and scale, and no larger than about scale / 2), is held against scale / 2.
constexpr float kTiny = 1e-30f;
constexpr float kRound = 12582912.f + 128.f;
template <int N>
__device__ __forceinline__ void codes_of(const float (&x)[N], float scale, float inv, uint32_t (&code)[N]) {
    float far = 0.f;
#pragma unroll
    for (int k = 0; k < N; ++k) {
        const float t = fmaf(x[k], inv, kRound);
        far = fmaxf(far, fabsf(fmaf(x[k], inv, kRound - t)));
        code[k] = __float_as_uint(t);
    }
    if (far <= 0.5f - 3.0517578125e-05f) return;
#pragma unroll
    for (int k = 0; k < N; ++k) {
        const float c = __uint_as_float(code[k]) - kRound, r = fmaf(-c, scale, x[k]);
        const bool off = 2.f * fabsf(r) > scale || (2.f * fabsf(r) == scale && (code[k] & 1));   // a tie goes to the even one
        code[k] += !off ? 0 : r > 0.f ? 1 : -1;
    }
}
// for scales whose reciprocal or remainders would leave fp32's normal range: the quotient in fp64
__device__ __noinline__ uint32_t code_of_tiny(float x, float scale) {
    return uint32_t(int(fmin(fmax(rint((double)x / (double)scale), -127.0), 127.0)) + 128);
}

// ---------------------------------------------------------------------------------------------------
// append and stage
// ---------------------------------------------------------------------------------------------------
struct WriteArgs {
    dfl_kv8 c;
    const int32_t *len, *cnt;
    const float *k, *v;
    int64_t ld;
    int rows, commit;
    int run;                 // blocks that a CTA of many rows' seals
};

// What a call does to one head: tokens from 32 z on are `have` rows of the tail (or, after a cut, of block
// z's codes) and n new rows; the first `full` blocks of them are sealed, the rest goes to the tail.
struct Plan {
    int z, have, n, full, cut, bad;
};
__device__ __forceinline__ Plan plan_of(const WriteArgs &a, int s, const KvView &w) {
    Plan p{};
    const int L = a.len[s], zs = *w.sealed;
    p.n = rows_of(a.cnt, s, a.rows);
    if (zs < 0 || zs > w.nb) {
        p.bad = kErrTable;
    } else if (L < 0 || L > kBlk * w.nb - p.n) {
        p.bad = kErrCapacity;
    } else if (L > kBlk * zs + kTail) {
        p.bad = kErrState;
    } else {
        p.z = min(zs, L / kBlk);
        p.cut = zs > p.z;
        p.have = L - kBlk * p.z;
        p.full = (p.have + (a.commit ? p.n : 0)) / kBlk;
    }
    return p;
}

// Channels d..d+3 of token 32 z + r of a head, keys (V = false) or values.
template <bool V, int HD>
struct Rows {
    const float *src;        // the call's rows of this head
    int64_t ld;
    const float *tail;
    const uint8_t *old;      // after a cut: block z's codes and scale
    float old_scale;
    int have, cut;
    __device__ __forceinline__ float4 get(int r, int d) const {
        if (r >= have) return *reinterpret_cast<const float4 *>(src + (size_t)(r - have) * ld + d);
        float y[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) y[k] = cut ? expand(old[V ? v_at(r, d + k) : k_at(r, d + k)], old_scale) : V ? tail[(d + k) * kTail + r] : tail[r * HD + d + k];
        return make_float4(y[0], y[1], y[2], y[3]);
    }
};
template <bool V, int HD>
__device__ __forceinline__ Rows<V, HD> rows_from(const WriteArgs &a, int s, int h, const KvView &w, const Plan &p, bool old) {
    const int phys = old ? w.table[p.z] : 0;      // old: rows before the call's own are wanted after a cut
    return {(V ? a.v : a.k) + (size_t)s * a.rows * a.ld + (size_t)h * HD, a.ld, V ? w.vt : w.kt, (V ? w.v : w.k) + (size_t)phys * kBlk * HD,
            old ? (V ? w.vs : w.ks)[phys] : 0.f, p.have, p.cut};
}

constexpr int kWriteThreads = 256;
constexpr int kVPitch = 40;

// the low bytes of four words as one
__device__ __forceinline__ uint32_t low_bytes(uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    return __byte_perm(__byte_perm(a, b, 0x0040), __byte_perm(c, d, 0x0040), 0x5410);
}

// Seals block b of the plan: a thread holds 4 tokens x 4 channels at a time, kPieces times. The codes go through shared
// memory, so that they leave in 16-byte stores whatever their layout.
template <bool V, int HD, int kThreads>
struct Seal {
    static constexpr int kPieces = (2 * HD + kThreads - 1) / kThreads, dq = HD / 4;
    float y[kPieces][16];                                            // [token][channel]
    // piece e: tokens t.. and channels d.. of it, so that a warp's words of shared memory lie in different banks: values with
    // the tokens innermost, a channel's 32 tokens 40 bytes apart
    static __device__ __forceinline__ int piece_t(int e) { return V ? 4 * (e & 7) : 4 * (e / dq); }
    static __device__ __forceinline__ int piece_d(int e) { return V ? 4 * (e >> 3) : 4 * (e % dq); }
    __device__ __forceinline__ void load(const Rows<V, HD> &x, int b) {
#pragma unroll
        for (int i = 0; i < kPieces; ++i) {
            const int e = i * kThreads + int(threadIdx.x), r = kBlk * b + piece_t(e), d = piece_d(e);   // of 8 * hd / 4 pieces
            if (e >= 8 * dq) break;
            if (kBlk * b >= x.have) {                                // all of the block is the call's
                const float *at = x.src + (size_t)(r - x.have) * x.ld + d;
#pragma unroll
                for (int k = 0; k < 4; ++k) put(i, k, *reinterpret_cast<const float4 *>(at + k * x.ld));
            } else {
#pragma unroll
                for (int k = 0; k < 4; ++k) put(i, k, x.get(r + k, d));
            }
        }
    }
    __device__ __forceinline__ void put(int i, int k, const float4 &v) { y[i][4 * k] = v.x, y[i][4 * k + 1] = v.y, y[i][4 * k + 2] = v.z, y[i][4 * k + 3] = v.w; }
    // Nothing is written if `bad` anywhere in the CTA. Two barriers: what a call reads of red and code is read before the next one's.
    __device__ __forceinline__ bool store(const KvView &w, int phys, int bad, uint32_t *red, uint8_t *code) const {
        const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
        float most = 0.f;
#pragma unroll
        for (int i = 0; i < kPieces; ++i)
            if (i * kThreads + tid < 8 * dq)
#pragma unroll
                for (int k = 0; k < 16; ++k) asm("max.NaN.f32 %0, %0, %1;" : "+f"(most) : "f"(fabsf(y[i][k])));
        uint32_t top = __reduce_max_sync(0xffffffffu, __float_as_uint(most) & 0x7fffffffu);   // as bits: infinities and NaN come last
        if (lane == 0) red[warp] = top;
        if (__syncthreads_or(bad)) return false;
#pragma unroll
        for (int i = 0; i < kThreads / 32; ++i) top = max(top, red[i]);
        const float scale = top < 0x7f800000u ? __fdiv_rn(__uint_as_float(top), 127.f) : NAN;
        const bool tiny = scale < kTiny, none = !(scale > 0.f);
        const float inv = none || tiny ? 0.f : 1.f / scale;
#pragma unroll
        for (int i = 0; i < kPieces; ++i) {
            const int e = i * kThreads + tid, t = piece_t(e), d = piece_d(e);
            if (e >= 8 * dq) break;
            uint32_t q[16];
            if (!none && !tiny) {
                codes_of(y[i], scale, inv, q);
            } else {
#pragma unroll
                for (int k = 0; k < 16; ++k) q[k] = none ? 128u : code_of_tiny(y[i][k], scale);
            }
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const uint32_t word = V ? low_bytes(q[k], q[4 + k], q[8 + k], q[12 + k]) : low_bytes(q[4 * k], q[4 * k + 1], q[4 * k + 2], q[4 * k + 3]);
                *reinterpret_cast<uint32_t *>(code + (V ? (d + k) * kVPitch + t : k_at(t + k, d))) = word;
            }
        }
        __syncthreads();
        uint4 *dst = reinterpret_cast<uint4 *>((V ? w.v : w.k) + (size_t)phys * kBlk * HD);
        for (int e = tid; e < 2 * HD; e += kThreads) {
            const uint2 *from = reinterpret_cast<const uint2 *>(code + (V ? (e >> 1) * kVPitch + 16 * (e & 1) : 16 * e));
            const uint2 lo = from[0], hi = from[1];
            dst[e] = make_uint4(lo.x, lo.y, hi.x, hi.y);
        }
        if (tid == 0) (V ? w.vs : w.ks)[phys] = scale;
        return true;
    }
};

// A head whose plan follows a table entry out of range is left alone.
__device__ __forceinline__ bool bad_table(const KvView &w, const Plan &p) {
    int bad = 0;
    for (int b = threadIdx.x; b < max(p.full, p.cut); b += blockDim.x) bad |= unsigned(w.table[p.z + b]) >= unsigned(w.nb);
    return __syncthreads_or(bad);
}

// What is left of a call behind its full blocks moves to the tail's front, one CTA for a head's keys or values. A row that
// comes from the tail lies 32 * full >= 32 rows further back than its place, behind all rows written here, or is where it
// belongs. Every load is under way before the first store.
constexpr int kTurn = 64;
using Turn = float[kTurn][kTail + 1];   // values turn through shared memory, so that a channel's tokens are stored together
template <bool V, int HD, int kThreads>
__device__ __forceinline__ void keep_rest(const Rows<V, HD> &x, const KvView &w, const Plan &p, Turn &turn) {
    const int tid = threadIdx.x, left = p.have + p.n - kBlk * p.full, first = !p.cut && p.full == 0 ? p.have : 0;
    constexpr int kSome = (kTail * (kTurn / 4) + kThreads - 1) / kThreads;   // at most 47 rows of 16 pieces a turn
    float4 y[HD / kTurn][kSome];
#pragma unroll
    for (int c = 0; c < HD / kTurn; ++c)
#pragma unroll
        for (int i = 0; i < kSome; ++i) {
            const int e = tid + i * kThreads;
            if (e < (left - first) * (kTurn / 4)) y[c][i] = x.get(kBlk * p.full + first + e / (kTurn / 4), c * kTurn + 4 * (e % (kTurn / 4)));
        }
    __syncthreads();
#pragma unroll
    for (int c = 0; c < HD / kTurn; ++c) {
        if (V) __syncthreads();
#pragma unroll
        for (int i = 0; i < kSome; ++i) {
            const int e = tid + i * kThreads, t = e / (kTurn / 4), d = 4 * (e % (kTurn / 4));
            if (e >= (left - first) * (kTurn / 4)) continue;
            if (V)
                turn[d][t] = y[c][i].x, turn[d + 1][t] = y[c][i].y, turn[d + 2][t] = y[c][i].z, turn[d + 3][t] = y[c][i].w;
            else
                *reinterpret_cast<float4 *>(w.kt + (size_t)(first + t) * HD + c * kTurn + d) = y[c][i];
        }
        if (!V) continue;
        __syncthreads();
        for (int d = tid >> 5; d < kTurn; d += kThreads / 32)
            for (int t = tid & 31; t < left - first; t += 32) w.vt[(size_t)(c * kTurn + d) * kTail + first + t] = turn[d][t];
    }
}

// Scores of the blocks that begin among the new rows, and the count of sealed ones. All threads of the CTA call it.
__device__ __forceinline__ void settle(const WriteArgs &a, int s, const KvView &w, const Plan &p) {
    if (w.score) {
        const int L = a.len[s];
        for (int b = (L + kBlk - 1) / kBlk + threadIdx.x; b * kBlk < L + p.n; b += blockDim.x) w.score[b] = 0.f;
    }
    __syncthreads();   // every thread has read the count
    if (threadIdx.x == 0) *w.sealed = p.z + p.full;
}

// One launch for a call of few rows, one CTA per head: latency, of the counts, then the rows, then the stores. 8 staged rows
// for 4 sequences of 8 heads of 128 take 4.0 us.
template <int HD>
__global__ void __launch_bounds__(kWriteThreads) k_kv8_write(WriteArgs a) {
    __shared__ uint32_t red[kWriteThreads / 32];
    __shared__ __align__(16) uint8_t code[kVPitch * HD];
    __shared__ Turn turn;
    const int h = blockIdx.x, s = blockIdx.y;
    const KvView w = view(a.c, s, h);
    pdl_wait();
    Plan p = plan_of(a, s, w);
    if (!p.bad && bad_table(w, p)) p.bad = kErrTable;
    if (p.bad) {
        if (threadIdx.x == 0) atomicOr(a.c.err, p.bad);
        return;
    }
    const Rows<false, HD> xk = rows_from<false, HD>(a, s, h, w, p, p.cut);
    const Rows<true, HD> xv = rows_from<true, HD>(a, s, h, w, p, p.cut);
    for (int b = 0; b < p.full; ++b) {
        const int phys = w.table[p.z + b];
        Seal<false, HD, kWriteThreads> k;
        k.load(xk, b);
        k.store(w, phys, 0, red, code);
        Seal<true, HD, kWriteThreads> v;
        v.load(xv, b);
        v.store(w, phys, 0, red, code);
    }
    keep_rest<false, HD, kWriteThreads>(xk, w, p, turn);
    keep_rest<true, HD, kWriteThreads>(xv, w, p, turn);
    settle(a, s, w, p);
}

// Many rows: a CTA for the keys or the values of a.run consecutive blocks, the next block's rows asked for as soon as the codes
// of the one before are out of the registers; grid (2 x runs, heads, sequences). The first one, which alone reads rows held
// before the call's first whole block, also keeps the rest. k_kv8_count behind it settles the call and reports what is bad.
// 4 bytes in and one out a value, some 15 instructions: 8 x 8192 rows of 8 heads of 128 take 142 us, 4.7 TB/s, 70 % of a
// plain copy's; what is missing is loads in flight while the codes are made (asking for a block ahead into registers of
// its own, or more CTAs of fewer registers, took longer: 151 and 179 us). A short call is latency: 1024 rows 7 us, 2 of them the second launch.
template <bool V, int HD, int kThreads>
__device__ __forceinline__ void append_blocks(const WriteArgs &a, int s, int h, const KvView &w, const Plan &p, int b0, uint32_t *red, uint8_t *code, Turn &turn) {
    const Rows<V, HD> x = rows_from<V, HD>(a, s, h, w, p, p.cut && b0 == 0);
    const int b1 = min(b0 + a.run, p.full);
    if (b0 < b1) {
        int bad = 0;
        for (int i = threadIdx.x; i < p.full; i += kThreads) bad |= unsigned(w.table[p.z + i]) >= unsigned(w.nb);
        Seal<V, HD, kThreads> seal;
        seal.load(x, b0);
        for (int b = b0; b < b1; ++b) {
            if (!seal.store(w, w.table[p.z + b], bad, red, code)) return;
            if (b + 1 < b1) seal.load(x, b + 1);
        }
        __syncthreads();
    }
    if (b0 == 0) keep_rest<V, HD, kThreads>(x, w, p, turn);
}
template <int HD>
__global__ void __launch_bounds__(2 * HD, 512 / HD) k_kv8_append(WriteArgs a) {
    constexpr int kThreads = 2 * HD;                                 // one piece of a block each
    __shared__ uint32_t red[kThreads / 32];
    __shared__ __align__(16) uint8_t code[kVPitch * HD];
    __shared__ Turn turn;
    const int b = (blockIdx.x >> 1) * a.run, h = blockIdx.y, s = blockIdx.z;
    const KvView w = view(a.c, s, h);
    pdl_wait();
    const Plan p = plan_of(a, s, w);
    pdl_trigger();
    if (p.bad || (b > 0 && b >= p.full) || (p.cut && b == 0 && bad_table(w, p))) return;   // a cut reads through the entry
    if (blockIdx.x & 1)
        append_blocks<true, HD, kThreads>(a, s, h, w, p, b, red, code, turn);
    else
        append_blocks<false, HD, kThreads>(a, s, h, w, p, b, red, code, turn);
}
__global__ void __launch_bounds__(64) k_kv8_count(WriteArgs a) {
    const int s = blockIdx.y;
    const KvView w = view(a.c, s, blockIdx.x);
    Plan p = plan_of(a, s, w);
    if (!p.bad && bad_table(w, p)) p.bad = kErrTable;
    pdl_wait();
    if (!p.bad)
        settle(a, s, w, p);
    else if (threadIdx.x == 0)
        atomicOr(a.c.err, p.bad);
}

// ---------------------------------------------------------------------------------------------------
// rows out
// ---------------------------------------------------------------------------------------------------
struct ReadArgs {
    dfl_kv8 c;
    const int32_t *len, *first;
    float *k, *v;
    int rows;
};

// One CTA per 32-token block of the range and head: grid (blocks, heads, sequences). A code is expanded by one subtraction and
// one product, rounded once; values turn through shared memory, so that all stores are of 16 bytes. Bound by its stores, 4 of
// the 5 bytes that a value costs: 8 x 8192 rows of 8 heads of 128 in 118 us, 5.7 TB/s, 84 % of a plain copy's.
__global__ void __launch_bounds__(256) k_kv8_read(ReadArgs a) {
    __shared__ uint32_t vcode[256 * 9];
    const int h = blockIdx.y, s = blockIdx.z, hd = a.c.head_dim;
    const KvView w = view(a.c, s, h);
    pdl_wait();
    const int L = a.len[s], first = a.first ? a.first[s] : 0, z = *w.sealed;
    int bad = 0;
    if (z < 0 || z > w.nb)
        bad = kErrTable;
    else if (L < 0 || L > kBlk * w.nb || first < 0)
        bad = kErrCapacity;
    else if (L > kBlk * z + kTail)
        bad = kErrState;
    const int hi = int(min((long long)L, (long long)first + a.rows)), b = bad ? 0 : first / kBlk + blockIdx.x;
    if (!bad && (first >= hi || kBlk * b >= hi)) return;             // no token of the range: the entry is nobody's business
    if (!bad && b < z && unsigned(w.table[b]) >= unsigned(w.nb)) bad = kErrTable;
    if (bad) {
        if (threadIdx.x == 0) atomicOr(a.c.err, bad);
        return;
    }
    const int dq = hd / 4, pos0 = kBlk * b;
    const size_t blk = (size_t)kBlk * hd, row = (size_t)a.c.n_kv * hd, out0 = ((size_t)s * a.rows * a.c.n_kv + h) * hd;
    auto put = [&](float *out, int t, int d, const float4 &y) {      // token t of the block, channels d..
        const int pos = pos0 + t;
        if (pos >= first && pos < hi) *reinterpret_cast<float4 *>(out + out0 + (size_t)(pos - first) * row + d) = y;
    };
    if (b < z) {
        const int phys = w.table[b];
        const float ks = w.ks[phys], vs = w.vs[phys];
        const uint4 *kc = reinterpret_cast<const uint4 *>(w.k + phys * blk), *vc = reinterpret_cast<const uint4 *>(w.v + phys * blk);
        for (int e = threadIdx.x; e < 2 * hd; e += blockDim.x) {     // a channel's 32 tokens, 36 bytes apart
            const uint4 y = vc[e];
            uint32_t *dst = vcode + (e >> 1) * 9 + 4 * (e & 1);
            dst[0] = y.x, dst[1] = y.y, dst[2] = y.z, dst[3] = y.w;
        }
        auto four = [](uint32_t x, float f) {
            return make_float4(expand(x & 255, f), expand(x >> 8 & 255, f), expand(x >> 16 & 255, f), expand(x >> 24, f));
        };
        for (int e = threadIdx.x; e < kBlk * dq; e += blockDim.x) {  // four channels of a token
            const int t = e / dq, d = 4 * (e % dq);
            put(a.k, t, d, four(reinterpret_cast<const uint32_t *>(kc)[k_at(t, d) >> 2], ks));
        }
        __syncthreads();
        for (int e = threadIdx.x; e < 8 * dq; e += blockDim.x) {     // four tokens of four channels
            const int t = 4 * (e / dq), d = 4 * (e % dq);
            uint32_t x[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) x[k] = vcode[(d + k) * 9 + (t >> 2)];
#pragma unroll
            for (int k = 0; k < 4; ++k)
                put(a.v, t + k, d, make_float4(expand(x[0] >> 8 * k & 255, vs), expand(x[1] >> 8 * k & 255, vs), expand(x[2] >> 8 * k & 255, vs), expand(x[3] >> 8 * k & 255, vs)));
        }
    } else {
        for (int e = threadIdx.x; e < kBlk * dq; e += blockDim.x) {
            const int t = e / dq, d = 4 * (e % dq), r = pos0 + t - kBlk * z;
            if (pos0 + t >= hi) break;
            put(a.k, t, d, *reinterpret_cast<const float4 *>(w.kt + (size_t)r * hd + d));
            put(a.v, t, d, make_float4(w.vt[(size_t)d * kTail + r], w.vt[(size_t)(d + 1) * kTail + r], w.vt[(size_t)(d + 2) * kTail + r], w.vt[(size_t)(d + 3) * kTail + r]));
        }
    }
}

// ---------------------------------------------------------------------------------------------------
// attention
// ---------------------------------------------------------------------------------------------------
struct AttnKvArgs {
    dfl_kv8 c;
    const float *q;
    float *out;
    int64_t ldq, ldo;
    int n_q, rows, window, causal, score;
    const int32_t *len, *cnt;
    float scale;
    int groups;           // row groups of a head
    // How the work is cut (see attn_cut). share == 0: `splits` CTAs at most for a unit's coded blocks, and with `apart` one
    // more for its tail (grid x 0; else the last split's CTA takes it). share != 0: `ctas` CTAs share all units evenly.
    int splits, apart, share, ctas;
    float *part_o;        // [part][rows of a group][head_dim]
    float *part_ml;       // [part][rows of a group][2]: running maximum (base 2) and sum
    int *part_bad;        // [part]: a table entry was out of range
    float *blk_lse;       // [sequence][head][n_blocks][2][16]: log2 of the shares of a block's halves in row 0's sums
};

// A unit is one row group of a head: unit (s * n_kv + h) * groups + rg. The sums of each CTA that has some of it are a part,
// merged by k_kv8_merge. Part ids: with splits, unit by unit (the tail's own CTA first); with shares, CTA + unit, which no
// two (CTA, unit) have in common, as both only grow along the work.
__device__ __forceinline__ size_t part_of(const AttnKvArgs &a, size_t unit, int i) {   // i: CTA of the unit, or CTA
    return a.share ? unit + i : unit * (a.splits + a.apart) + i;
}

struct Span {
    int z, L, n, bad;   // sealed blocks, committed tokens, staged rows
    int b0, nb;         // blocks that some row sees: b0 .. b0 + nb - 1
    int coded;          // the first so many of them are held as codes, the others lie in the tail
    int groups;         // row groups that have rows
};
__device__ __forceinline__ Span span_of(const AttnKvArgs &a, int s, int sealed, int rows_per_group) {
    Span p{sealed, a.len[s], rows_of(a.cnt, s, a.rows), 0, 0, 0, 0, 0};
    if (p.z < 0 || p.z > a.c.n_blocks)
        p.bad = kErrTable;
    else if (p.L < 0 || p.L > kBlk * a.c.n_blocks - p.n)
        p.bad = kErrCapacity;
    else if (p.L < kBlk * p.z || p.L + p.n > kBlk * p.z + kTail)
        p.bad = kErrState;
    if (p.bad || p.n == 0) return p;
    const int at = a.causal ? p.L : p.L - 1;
    p.b0 = (a.window > 0 ? max(0, at - a.window + 1) : 0) / kBlk;
    p.nb = (p.L + p.n - 1) / kBlk + 1 - p.b0;   // every row sees its own token, so the tail is never empty
    p.coded = min(p.nb, max(0, p.z - p.b0));
    p.groups = (p.n * (a.n_q / a.c.n_kv) + rows_per_group - 1) / rows_per_group;
    return p;
}
// The span of a sequence by its first head. The heads of a sequence have equal sealed counts, but where a bad table entry has kept
// one from going on with the others, or a caller has set them: heads that differ from the first are left alone (kErrState).
__device__ __forceinline__ Span span_of_seq(const AttnKvArgs &a, int s, int rows_per_group) {
    return span_of(a, s, a.c.sealed[(size_t)s * a.c.n_kv], rows_per_group);
}
// the tokens lo..hi-1 that row m sees
__device__ __forceinline__ void seen(const AttnKvArgs &a, const Span &p, int m, int &lo, int &hi) {
    const int at = a.causal ? p.L + m : p.L - 1;   // the last token that the window counts from
    lo = a.window > 0 ? max(0, at - a.window + 1) : 0;
    hi = a.causal ? p.L + m + 1 : p.L + p.n;
}

// Both products run on the tensor cores (m16n8k16, fp16 in, fp32 sums), keys and value channels as the
// 16-row operand, query rows as the 8 columns: S^T = K Q^T and O^T = V^T P^T, so rows that a call does not
// have cost at most 7 columns. Codes are whole numbers of at most 7 bits and exact in fp16; the block's
// key scale multiplies the fp32 logits. A query row (scaled by a power of two to 2^14..2^15) and the weights
// (2^7 and more for the row's largest) enter as two fp16 halves, hi + lo, which hold 22 bits, and nothing below
// 2^-25. A block's value scale multiplies the fp32 sums of its own products, so that the size of one block's
// values, seen by a row or not, takes nothing from another's.
//
// These are the older tensor instructions on purpose. The fifth generation's take their operands from shared or tensor
// memory, so every code would be written there a second time at twice its size; a unit has 1 to 16 rows (32 columns with both
// halves), for which the time is loads, expansion and the softmax between the products. Their rate comes near to a bound
// only where 16 rows share each code: 8 clocks an instruction of 256 codes, 8 rows and one half are 74 % of the time that HBM
// takes for the codes (8 sequences of 16384 tokens and 16 heads of 128: 59 of 80 us).
//
// Fragment order. A thread (g = lane / 4, t = lane % 4) loads 16 consecutive channels of a key at once, so
// channel 64 c + 16 t + 4 j + e is input 2t + e (e < 2) or 2t + 6 + e of the product's step 4 c + j, and
// the query halves are laid out to match. Row r of 8-key matrix j holds key 8 (r / 2) + 2 j + r % 2 of a block: the
// transposed weights of matrices 2 s and 2 s + 1 are then the inputs of step s of the second product, whose
// thread t takes the keys 8 t + 4 s .. + 3, 8 consecutive codes of a value channel for both steps. A warp with half a
// block's keys has the matrices 0 and 1, or 2 and 3.
constexpr float kLog2e = 1.44269504088896340736f;
constexpr float kTop = 7.f;    // log2 of the weight at a row's maximum

template <int HD, int NT, bool PK = false>
struct AttnShape {
    // Groups of four warps, 16 warps an SM of 128 registers a thread. A warp takes kM tiles of 16 keys at a time: two, which
    // halves what a turn costs besides its products and the reads of the query halves, or one where the rings would not fit.
    static constexpr int kM = HD == 256 ? 1 : 2;
    static constexpr int kTurn = 2 * kM;                             // blocks that a group takes at a time
    static constexpr int kUnit = 16 * kM * HD;                       // bytes of a warp's keys, or values, of a turn
    static constexpr int kCtas = HD == 256 && NT == 2 ? 1 : 2;
    static constexpr int kGroups = HD == 256 && NT == 2 ? 4 : 2;
    static constexpr int kWarps = 4 * kGroups;
    static constexpr int kStep = kGroups * kTurn;                    // blocks that a CTA takes at a time
    // Units under way, as many as the CTAs of an SM have room for: two CTAs, or in shares of up to 4 rows three (80 registers).
    static constexpr int kShareCtas = PK && HD < 256 ? 3 : kCtas;
    static constexpr int kRing = (HD == 64 ? 5 : 3) - (HD < 256 && (NT == 2 || PK) ? 1 : 0);
    static constexpr int kQBytes = NT * 8 * HD * (PK ? 2 : 4);                  // query halves
    static constexpr int kPBytes = kGroups * 2 * kTurn * NT * (PK ? 256 : 512);   // a turn's weights, for each group
    static constexpr int kSmem = kQBytes + kPBytes + kWarps * kRing * kUnit;
    static_assert(kGroups * 8 * NT * (HD + 4) * 4 <= kSmem, "the merge's use of the shared memory");
    static constexpr int kTailPitch = kTail + 4;                     // of the tail's weights [rows][48 tokens], fp32
    static_assert(kTail * HD * 4 <= 4 * kRing * kUnit && (PK ? 4 : 8 * NT) * kTailPitch * 4 <= kPBytes / kGroups, "the tail's: keys or values in a group's rings");
};

// the four warps of a group: a barrier, and one that also tells whether x holds anywhere in the group
__device__ __forceinline__ void group_sync(int grp) { asm volatile("barrier.cta.sync.aligned %0, 128;" ::"r"(grp + 1) : "memory"); }
__device__ __forceinline__ bool group_or(int grp, bool x) {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\tbarrier.cta.red.or.aligned.pred q, %2, 128, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(r)
        : "r"(uint32_t(x)), "r"(grp + 1)
        : "memory");
    return r;
}

template <bool FIRST = false>   // FIRST: d = a b
__device__ __forceinline__ void mma_f16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    if constexpr (FIRST)
        asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
            : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
    else
        asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// 2^x by the hardware's instruction: off by 2 units in the last place, results below 2^-126 are 0
__device__ __forceinline__ float ex2(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
    uint32_t r;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
    return r;
}
// codes of bytes 0, 1 (or 2, 3) of w as two fp16: 0x6400 | c is 1024 + c, less 1152
__device__ __forceinline__ uint32_t codes_lo(uint32_t w) {
    uint32_t r;
    asm("{\n\t.reg .b32 x;\n\tprmt.b32 x, %1, 0x64646464, 0x4140;\n\tadd.rn.f16x2 %0, x, %2;\n\t}" : "=r"(r) : "r"(w), "r"(0xE480E480u));
    return r;
}
__device__ __forceinline__ uint32_t codes_hi(uint32_t w) {
    uint32_t r;
    asm("{\n\t.reg .b32 x;\n\tprmt.b32 x, %1, 0x64646464, 0x4342;\n\tadd.rn.f16x2 %0, x, %2;\n\t}" : "=r"(r) : "r"(w), "r"(0xE480E480u));
    return r;
}

// two fp32 as fp16 halves hi + lo, the first in the low half of a word
__device__ __forceinline__ void halves2(float x0, float x1, uint32_t &hi, uint32_t &lo) {
    const __half2 h = __floats2half2_rn(x0, x1);
    const float2 f = __half22float2(h);
    const __half2 l = __floats2half2_rn(x0 - f.x, x1 - f.y);
    hi = *reinterpret_cast<const uint32_t *>(&h);
    lo = *reinterpret_cast<const uint32_t *>(&l);
}
// two fp32 as three bf16 each: 24 bits over fp32's whole range
__device__ __forceinline__ void thirds2(float x0, float x1, uint32_t (&w)[3]) {
#pragma unroll
    for (int i = 0; i < 3; ++i) {
        const __nv_bfloat162 b = __floats2bfloat162_rn(x0, x1);
        const float2 f = __bfloat1622float2(b);
        w[i] = *reinterpret_cast<const uint32_t *>(&b);
        x0 -= f.x;
        x1 -= f.y;
    }
}
// 2^(14 - floor(log2 x)) for x > 0, within the normal range; 1 for 0
__device__ __forceinline__ float lift(float x) {
    const int e = int(__float_as_uint(x) >> 23);           // biased exponent; 0 for subnormals
    if (x == 0.f) return 1.f;
    return __uint_as_float(uint32_t(min(127 + 14 + 127 - max(e, 1), 253)) << 23);
}
__device__ __forceinline__ float group_max(float x) {      // over the eight g of a t
    x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 4));
    x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 8));
    return fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 16));
}
__device__ __forceinline__ float group_sum(float x) {
    x += __shfl_xor_sync(0xffffffffu, x, 4);
    x += __shfl_xor_sync(0xffffffffu, x, 8);
    return x + __shfl_xor_sync(0xffffffffu, x, 16);
}
template <int N>
__device__ __forceinline__ void cp_async_wait_groups() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

// the splits that coded blocks are worth: at least a turn each
template <int W>
__device__ __forceinline__ int splits_of(int splits, int coded) { return min(splits, (coded + W - 1) / W); }

// Shares: the work in the order of its units, each weighing its coded blocks and, behind them, its tail as
// kTailWeight: what a unit costs besides its blocks, the tail, its first loads and the groups' merge, in blocks. (64 sequences
// of some 5000 tokens, 8 heads of 128, one token, and 8 of 16384 and 16 heads, 8 rows: 126 and 136 us at 8, 119 and 129 at 40,
// 122 and 135 at 64.) CTA b of G takes the weights [W b / G, W (b + 1) / G).
constexpr int kTailWeight = 40;
__device__ __forceinline__ long weight_of(const AttnKvArgs &a, const Span &p) { return (long)a.c.n_kv * p.groups * (p.coded + kTailWeight); }
template <int W>
__device__ __forceinline__ int shares_of(const AttnKvArgs &a, long work) { return int(min((long)a.ctas, (work + W - 1) / W)); }

// block-wide sums of two numbers (all threads call it and get them)
__device__ __forceinline__ void block_sums(long &x, long &y, long (*sm)[2]) {
    x = warp_sum(x);
    y = warp_sum(y);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) sm[threadIdx.x >> 5][0] = x, sm[threadIdx.x >> 5][1] = y;
    __syncthreads();
    x = y = 0;
    for (int i = 0; i < int(blockDim.x >> 5); ++i) x += sm[i][0], y += sm[i][1];
}

// What a CTA does of a unit: its coded blocks x0..x1-1 (of the span's), and its tail or not.
struct Piece {
    int s, h, rg, x0, x1;
    bool tail, whole;   // whole: all of the unit, which then needs no merge
    int index;          // of its part: the split (the tail's own CTA counts as one behind them), or the CTA
};
template <int HD, int NT>
struct AttnShared {
    float q_scale[8 * NT], top[AttnShape<HD, NT>::kGroups][4][8 * NT], m[AttnShape<HD, NT>::kGroups][8 * NT], l[AttnShape<HD, NT>::kWarps][8 * NT];
    int bad;
    uint32_t poisoned;   // bit r: row r of the group sees a value that is not finite: its outputs are NaN, its weights what they are
};
template <int HD, int NT>
struct QueryRows {      // a warp takes every kWarps-th row of the group; `n` of the call's rows count, the others are not read
    static constexpr int kW = AttnShape<HD, NT>::kWarps, kRows = (8 * NT + kW - 1) / kW;
    float2 x[kRows][HD / 64];
    __device__ __forceinline__ void load(const AttnKvArgs &a, int s, int h, int rg, int n) {
        const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, per = a.n_q / a.c.n_kv;
#pragma unroll
        for (int i = 0; i < kRows; ++i) {
            const int r = warp + i * kW, rid = rg * 8 * NT + r;
            const bool on = r < 8 * NT && rid < n * per;
            const float *q = a.q + ((size_t)s * a.rows + rid / per) * a.ldq + (size_t)(h * per + rid % per) * HD + 2 * lane;
#pragma unroll
            for (int k = 0; k < HD / 64; ++k) x[i][k] = on ? *reinterpret_cast<const float2 *>(q + 64 * k) : make_float2(0.f, 0.f);
        }
    }
};

// One CTA's piece of a unit: 8 NT query rows (row r = m * group + i of the head's rows), its coded blocks and perhaps the
// tail. Groups of four warps take every kGroups-th turn of blocks, each group with a running softmax of its own, merged at
// the end. In a turn of two or four blocks each warp takes a quarter of the keys for the first product and, for the second,
// a quarter of the value channels over all keys; the weights pass through shared memory between them. So a warp's sums are
// small, its code is short (a short call spends much of its time on fetching code), and each code is read from shared
// memory and expanded once in the CTA. Keys and values come through a ring of the warp's own (16-byte asynchronous copies):
// what a warp copies only it reads.
// What bounds it: with many sequences the issue of instructions and the latency between the steps of a turn at 16 or 24 warps an SM
// (32 query heads over 8 of 128, one token of 64 sequences of some 5000: 119 us, 5.6 TB/s, 83 % of a plain copy's; verifies of
// 8 rows of 8 sequences of 16384 and 16 heads of 128, two halves of 16 columns: 128 us, 4.2 TB/s, 62 %). With one
// sequence a CTA has one to three turns, and the time is the launch, the first loads (table, then scales and codes), some
// 3 us a turn and the merge: 16384 tokens of 2 heads of 256 take 12.2 us for a token, 27 us for 8 rows of 6 heads each.
//
// PK, for up to 4 rows: the query's lo halves take the columns 4..7 that no row needs, so one product does for both halves, in
// both products. The thread pairs t and t + 2 then hold the same two rows: after the first product each adds up the halves of
// one of the tile's two keys a thread, so that the softmax's work is halved too. The 64 sequences above: 132 us without, 129
// with, 126 with the third CTA an SM that its fewer registers allow (120 since units count their tails rightly).
template <int HD, int NT, bool PK>
__device__ __forceinline__ void attn_piece(const AttnKvArgs &a, const Span &p, const Piece &u, QueryRows<HD, NT> &qr, uint8_t *smem, AttnShared<HD, NT> &sh) {
    using S = AttnShape<HD, NT, PK>;
    constexpr int RG = 8 * NT, kW = S::kWarps, kG = S::kGroups, kRing = S::kRing, kUnit = S::kUnit, kPitch = HD + 4, kMt = HD / 64, kM = S::kM, kTurn = S::kTurn, kWin = 32 / kTurn;
    const int s = u.s, h = u.h, rg = u.rg;
    static_assert(!PK || NT == 1, "one tile of columns holds both halves");
    constexpr int kE = PK ? 2 : 4;                                   // logits a thread has of a tile
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t = lane & 3;
    const int t2 = PK ? 2 * (t & 1) : 2 * t, low = PK ? t >> 1 : 0;  // this thread's rows t2 and t2 + 1 of a tile, and (PK) its key of two
    // first product: block `mine` of the turn, all its keys (kM = 2) or those with bit 2 = key_half
    const int grp = warp >> 2, wq = warp & 3, mine = kM == 2 ? wq : wq >> 1, key_half = kM == 2 ? 0 : wq & 1;
    const size_t head = (size_t)s * a.c.n_kv + h, head_blocks = head * a.c.n_blocks;
    const int per = a.n_q / a.c.n_kv, live = p.n * per - rg * RG;    // rows of this group that exist
    const int n = u.x1 - u.x0, first = p.b0 + u.x0 + kTurn * grp;    // coded blocks; turn i of this group begins with first + kTurn kG i
    const int turns = (n - kTurn * grp + kTurn * kG - 1) / (kTurn * kG);   // <= 0: none
    uint8_t *ring = smem + S::kQBytes + S::kPBytes + warp * kRing * kUnit;
    using Weights = typename std::conditional<PK, uint2, uint4>::type;   // a thread's of a step
    constexpr int kQ = PK ? 2 : 4;                                   // pieces of 16 query inputs: hi, and (not PK) lo
    Weights *pbuf = reinterpret_cast<Weights *>(smem + S::kQBytes + grp * (S::kPBytes / kG)) + lane;
    const uint4 *qf = reinterpret_cast<const uint4 *>(smem) + lane;
    const bool keep_lse = a.score && rg == 0;

    int bad = 0;
    auto load_phys = [&](int i0) {                                   // lane l: where block l % kTurn of turn i0 + l / kTurn is stored
        const int b = first + kTurn * kG * (i0 + lane / kTurn) + lane % kTurn;
        int at = 0;
        if (b < p.b0 + u.x1) {
            at = a.c.table[head_blocks + b];
            if (unsigned(at) >= unsigned(a.c.n_blocks)) at = 0, bad = 1;
        }
        return at;
    };
    int phys = load_phys(0), phys_next = load_phys(kWin);            // of the kWin turns that are being asked for, and the next
    float ks = a.c.k_scale[head_blocks + phys], vs = a.c.v_scale[head_blocks + phys], ks_next = 0.f, vs_next = 0.f;

    // unit 2 i is turn i's keys (of this warp), unit 2 i + 1 its values (of this warp's channels)
    uint8_t *put = ring;                                             // the slot that the next unit goes to
    const uint8_t *take = ring;                                      // the slot that is read next
    auto issue = [&](int v) {
        const int i = v >> 1;
        if (i < turns) {
            if (v % (2 * kWin) == 0 && v > 0) {
                phys = phys_next;
                phys_next = load_phys(i + kWin);
            }
            const int lane0 = kTurn * (i % kWin), left = n - kTurn * (grp + kG * i);   // blocks of the turn: up to kTurn
            if (v & 1) {
#pragma unroll
                for (int j = 0; j < kTurn; ++j) {
                    const size_t off = (head_blocks + __shfl_sync(0xffffffffu, phys, lane0 + j)) * (kBlk * HD) + wq * (8 * HD) + 16 * lane;
                    if (j < left)
#pragma unroll
                        for (int k = 0; k < HD / 64; ++k) cp_async16(put + j * (8 * HD) + 512 * k + 16 * lane, a.c.v + off + 512 * k);
                }
            } else {
                const size_t off = (head_blocks + __shfl_sync(0xffffffffu, phys, lane0 + mine)) * (kBlk * HD);
                if (mine < left) {
                    if (kM == 2) {
#pragma unroll
                        for (int k = 0; k < HD / 16; ++k) cp_async16(put + 512 * k + 16 * lane, a.c.k + off + 512 * k + 16 * lane);
                    } else {
                        const uint8_t *src = a.c.k + off + key_half * 256 + (lane >> 4) * 512 + (lane & 15) * 16;
#pragma unroll
                        for (int c = 0; c < HD / 64; ++c) {
                            cp_async16(put + c * 1024 + 16 * lane, src + c * 2048);
                            cp_async16(put + c * 1024 + 512 + 16 * lane, src + c * 2048 + 1024);
                        }
                    }
                }
            }
            put = put == ring + (kRing - 1) * kUnit ? ring : put + kUnit;
        }
        cp_async_commit();
    };
    auto taken = [&]() { take = take == ring + (kRing - 1) * kUnit ? ring : take + kUnit; };
#pragma unroll
    for (int v = 0; v < kRing; ++v) issue(v);

    // The tail's rows, keys or values, into the first group's rings (by its 128 threads), 16 bytes at a time. The pieces of a key
    // change places so that a warp's reads of it lie in different banks.
    const int trows = p.L + p.n - kBlk * p.z;
    float *tail_rows = reinterpret_cast<float *>(smem + S::kQBytes + S::kPBytes);
    auto key_piece = [&](int key, int q) { return key * (HD / 4) + (q ^ ((q >> 3) & 1) ^ ((key & 1) << 1)); };
    auto copy_tail = [&](bool values) {
        const float *src = values ? a.c.v_tail + head * HD * kTail : a.c.k_tail + head * kTail * HD;
        if (values) {
            for (int e = tid; e < HD * (kTail / 4); e += 128)
                if (4 * (e % (kTail / 4)) < trows) cp_async16(tail_rows + 4 * e, src + 4 * e);
        } else {
            for (int e = tid; e < trows * (HD / 4); e += 128) cp_async16(tail_rows + 4 * key_piece(e / (HD / 4), e % (HD / 4)), src + 4 * e);
        }
        cp_async_commit();
    };
    const bool tail_only = u.tail && n == 0;
    if (tail_only && grp == 0) copy_tail(false);

    // ---- query rows into their fragments ----
    if (tid == 0) sh.bad = 0, sh.poisoned = 0;
#pragma unroll
    for (int j = 0; j < QueryRows<HD, NT>::kRows; ++j) {
        const int r = warp + j * kW;
        if (r >= RG) break;
        float amax = 0.f;
        bool fin = true;
#pragma unroll
        for (int i = 0; i < HD / 64; ++i) {
            if (r >= live) qr.x[j][i] = make_float2(0.f, 0.f);
            fin = fin && isfinite(qr.x[j][i].x) && isfinite(qr.x[j][i].y);
            amax = fmaxf(amax, fmaxf(fabsf(qr.x[j][i].x), fabsf(qr.x[j][i].y)));
        }
        fin = __all_sync(0xffffffffu, fin);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
        const float f = fin ? lift(amax) : 0.f;
        if (lane == 0) sh.q_scale[r] = fin ? a.scale * kLog2e / f : NAN;
#pragma unroll
        for (int i = 0; i < HD / 64; ++i) {
            uint32_t hi = 0, lo = 0;
            if (fin) halves2(qr.x[j][i].x * f, qr.x[j][i].y * f, hi, lo);
            const int d = 2 * lane;                                  // of chunk i
            uint32_t *dst = reinterpret_cast<uint32_t *>(smem) + (((i * NT + r / 8) * kQ + ((d & 15) >> 3)) * 32 + (r & 7) * 4 + (d >> 4)) * 4 + ((d & 7) >> 1);
            if (PK && r >= 4) continue;
            dst[0] = hi;
            dst[PK ? 4 * 4 * 4 : 2 * 32 * 4] = lo;
        }
    }
    __syncthreads();
    auto scale_of = [&](int nt) { return *reinterpret_cast<const float2 *>(&sh.q_scale[8 * nt + t2]); };
    // the tokens lo..hi-1 that row 8 nt + 2 t + e sees; all, if it does not exist: nothing reads its sums
    auto row_sees = [&](int nt, int e, int &lo, int &hi) {
        const int r = 8 * nt + t2 + e;
        lo = 0, hi = 1 << 30;
        if (r < live) seen(a, p, (rg * RG + r) / per, lo, hi);
    };
    // PK: both halves of two of a tile's logits, x[0..1] of key 2 low (the other two go to the thread that has their other half)
    auto join = [&](float (&x)[4]) {
        const float y0 = __shfl_xor_sync(0xffffffffu, low ? x[0] : x[2], 2), y1 = __shfl_xor_sync(0xffffffffu, low ? x[1] : x[3], 2);
        x[0] = (low ? x[2] : x[0]) + y0;
        x[1] = (low ? x[3] : x[1]) + y1;
    };
    auto rows_sum = [&](float x) {                                   // over all threads that have the row
        if (PK) x += __shfl_xor_sync(0xffffffffu, x, 2);
        return group_sum(x);
    };
    // tokens all_lo..all_hi-1 are seen by every row of the group that exists
    int all_lo, all_hi, dummy;
    seen(a, p, min(p.n - 1, (rg * RG + RG - 1) / per), all_lo, dummy);
    seen(a, p, rg * RG / per, dummy, all_hi);

    // A row's weights are 2^(logit - mx + kTop), for all four warps of the group. mx is a maximum that is only renewed when a
    // weight would pass 2^15, so most pairs need no maximum across the lanes and rescale nothing: the row's largest weight
    // lies in 2^7..2^15.
    float o[kMt][NT][4], mx[NT][2], l[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
        for (int e = 0; e < 2; ++e) mx[nt][e] = -INFINITY, l[nt][e] = 0.f;
#pragma unroll
        for (int mt = 0; mt < kMt; ++mt) o[mt][nt][0] = o[mt][nt][1] = o[mt][nt][2] = o[mt][nt][3] = 0.f;
    }
    // Renews mx by the logits y of the group (y == -inf: not seen), and rescales the sums. The four warps call it together.
    auto renew = [&](const float (&y)[kM][NT][kE]) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            float t0 = -INFINITY, t1 = -INFINITY;
#pragma unroll
            for (int m = 0; m < kM; ++m)
#pragma unroll
                for (int k = 0; k < kE; k += 2) t0 = fmaxf(t0, y[m][nt][k]), t1 = fmaxf(t1, y[m][nt][k + 1]);
            if (PK) t0 = fmaxf(t0, __shfl_xor_sync(0xffffffffu, t0, 2)), t1 = fmaxf(t1, __shfl_xor_sync(0xffffffffu, t1, 2));
            t0 = group_max(t0);
            t1 = group_max(t1);
            if (g == 0 && low == 0) sh.top[grp][wq][8 * nt + t2] = t0, sh.top[grp][wq][8 * nt + t2 + 1] = t1;
        }
        group_sync(grp);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                float now = mx[nt][e];
#pragma unroll
                for (int i = 0; i < 4; ++i) now = fmaxf(now, sh.top[grp][i][8 * nt + t2 + e]);
                const float f = mx[nt][e] == now ? 1.f : ex2(mx[nt][e] - now);
                mx[nt][e] = now;
                l[nt][e] *= f;
#pragma unroll
                for (int mt = 0; mt < kMt; ++mt) o[mt][nt][e] *= f, o[mt][nt][2 + e] *= f;
            }
    };
    auto put_lse = [&](int b, int half, int r, float total, float top) {   // row r's sum over half a block, of weights at `top`
        a.blk_lse[((head_blocks + b) * 2 + half) * 16 + r] = total == 0.f ? -INFINITY : top - kTop + log2f(total);
    };

    for (int i = 0; i < turns; ++i) {
        if (i % kWin == 0) {                                         // the next kWin turns' scales
            if (i > 0) ks = ks_next, vs = vs_next;
            const int at = first + kTurn * kG * (i + lane / kTurn) + lane % kTurn;
            if (at >= p.b0 + u.x1) ks = vs = 0.f;                    // what is read in place of a block that is not there
            for (uint32_t nan = __ballot_sync(0xffffffffu, isnan(vs)); nan; nan &= nan - 1) {   // lane r asks for row r
                const int from = kBlk * __shfl_sync(0xffffffffu, at, __ffs(nan) - 1);
                int lo = 0, hi = 0;
                if (lane < min(live, RG)) seen(a, p, (rg * RG + lane) / per, lo, hi);
                if (lo < from + kBlk && hi > from) atomicOr(&sh.poisoned, 1u << lane);
            }
            if (isnan(vs)) vs = 0.f;
        }
        if (i % kWin == kWin / 2) {                                  // the next window's, half a window ahead
            ks_next = a.c.k_scale[head_blocks + phys_next];
            vs_next = a.c.v_scale[head_blocks + phys_next];
        }
        const int from = kTurn * (i % kWin) + mine, b = first + kTurn * kG * i + mine;   // this warp's block of the turn
        const float bks = __shfl_sync(0xffffffffu, ks, from);
        const bool there = b < p.b0 + u.x1;
        cp_async_wait_groups<kRing - 1>();
        __syncwarp();
        // consecutive products go to at least four sums: the query's halves have sums of their own where tiles and rows give fewer
        constexpr int kParts = kM * NT < 4 ? 2 : 1;
        float xs[kParts][kM][NT][4];
#pragma unroll
        for (int k = 0; k < kParts * kM * NT * 4; ++k) (&xs[0][0][0][0])[k] = 0.f;
        float(&x)[kM][NT][4] = xs[0];
        const uint8_t *K = take + (kM == 2 ? 8 * (g >> 1) + (g & 1) : 4 * (g >> 1) + (g & 1)) * 64 + 16 * t;
#pragma unroll
        for (int c = 0; c < HD / 64; ++c) {
            uint32_t kw[2 * kM][4];                                  // of matrix j: this thread's key of it, 128 bytes behind matrix j - 1's
#pragma unroll
            for (int j = 0; j < 2 * kM; ++j) *reinterpret_cast<uint4 *>(kw[j]) = *reinterpret_cast<const uint4 *>(K + c * (1024 * kM) + 128 * j);
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                uint32_t qh[NT][4], ql[NT][4];
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    *reinterpret_cast<uint4 *>(qh[nt]) = qf[((c * NT + nt) * kQ + half) * 32];
                    if (!PK) *reinterpret_cast<uint4 *>(ql[nt]) = qf[((c * NT + nt) * kQ + 2 + half) * 32];
                }
#pragma unroll
                for (int jj = 0; jj < 2; ++jj) {
                    const int j = 2 * half + jj;
                    uint32_t af[kM][4];
#pragma unroll
                    for (int m = 0; m < kM; ++m) {
                        af[m][0] = codes_lo(kw[2 * m][j]), af[m][1] = codes_lo(kw[2 * m + 1][j]);
                        af[m][2] = codes_hi(kw[2 * m][j]), af[m][3] = codes_hi(kw[2 * m + 1][j]);
                    }
#pragma unroll
                    for (int part = 0; part < (PK ? 1 : 2); ++part)
#pragma unroll
                        for (int m = 0; m < kM; ++m)
#pragma unroll
                            for (int nt = 0; nt < NT; ++nt)
                                mma_f16(xs[(PK ? j : part) % kParts][m][nt], af[m], part ? ql[nt][2 * jj] : qh[nt][2 * jj], part ? ql[nt][2 * jj + 1] : qh[nt][2 * jj + 1]);
                }
            }
        }
        __syncwarp();
        taken();
        issue(2 * i + kRing);
        if (kParts == 2)
#pragma unroll
            for (int k = 0; k < kM * NT * 4; ++k) (&x[0][0][0])[k] += (&xs[kParts - 1][0][0][0])[k];
        if (PK)
#pragma unroll
            for (int m = 0; m < kM; ++m) join(x[m][0]);
        float y[kM][NT][kE], peak = -INFINITY;                       // exponents of the weights
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const float z = bks * (e ? scale_of(nt).y : scale_of(nt).x), less = kTop - mx[nt][e];   // +inf before a row's first key
#pragma unroll
                for (int m = 0; m < kM; ++m)
#pragma unroll
                    for (int k = e; k < kE; k += 2) y[m][nt][k] = fmaf(x[m][nt][k], z, less);
            }
        const int pos0 = kBlk * b;
        if (!there || pos0 < all_lo || pos0 + kBlk > all_hi) {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    int lo, hi;
                    row_sees(nt, e, lo, hi);
#pragma unroll
                    for (int m = 0; m < kM; ++m)
#pragma unroll
                        for (int k = e; k < kE; k += 2) {
                            const int pos = pos0 + 8 * (g >> 1) + 4 * (m + key_half) + 2 * (k >> 1 | low) + (g & 1);
                            if (!there || pos < lo || pos >= hi) y[m][nt][k] = -INFINITY;
                        }
                }
        }
#pragma unroll
        for (int m = 0; m < kM; ++m)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int k = 0; k < kE; ++k) peak = fmaxf(peak, y[m][nt][k]);
        if (group_or(grp, peak > 15.f)) {                            // seldom, once the maxima have been met
#pragma unroll
            for (int m = 0; m < kM; ++m)
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int k = 0; k < kE; ++k) y[m][nt][k] = y[m][nt][k] == -INFINITY ? -INFINITY : x[m][nt][k] * (bks * (k & 1 ? scale_of(nt).y : scale_of(nt).x));
            renew(y);
#pragma unroll
            for (int m = 0; m < kM; ++m)
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int k = 0; k < kE; ++k) y[m][nt][k] += mx[nt][k & 1] == -INFINITY ? 0.f : kTop - mx[nt][k & 1];
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
            for (int m = 0; m < kM; ++m)
#pragma unroll
                for (int k = 0; k < kE; ++k) y[m][nt][k] = ex2(y[m][nt][k]);
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                float sum = PK ? y[0][nt][e] : y[0][nt][e] + y[0][nt][kE - 2 + e];
                if (kM == 2) sum += PK ? y[kM - 1][nt][e] : y[kM - 1][nt][e] + y[kM - 1][nt][kE - 2 + e];
                l[nt][e] += sum;
                if (keep_lse) {
                    const float total = rows_sum(sum);
                    const int r = 8 * nt + t2 + e;
                    if (g == 0 && low == 0 && r < per && there) {
                        put_lse(b, key_half, r, total, mx[nt][e]);
                        if (kM == 2) put_lse(b, 1, r, 0.f, 0.f);     // the block's sum is one
                    }
                }
            }
#pragma unroll
            for (int m = 0; m < kM; ++m) {
                uint4 w;                                             // hi and lo halves of the step's two input pairs
                halves2(y[m][nt][0], y[m][nt][1], w.x, w.z);
                Weights &to = pbuf[((kM * wq + m) * NT + nt) * 32];
                if constexpr (PK) {                                  // hi in columns 0..3 and lo in 4..7, of both keys
                    const uint32_t other = __shfl_xor_sync(0xffffffffu, low ? w.x : w.z, 2);
                    to = make_uint2(transpose8x8(low ? other : w.x), transpose8x8(low ? w.z : other));
                } else {
                    halves2(y[m][nt][2], y[m][nt][3], w.y, w.w);
                    to = make_uint4(transpose8x8(w.x), transpose8x8(w.y), transpose8x8(w.z), transpose8x8(w.w));
                }
            }
        }
        cp_async_wait_groups<kRing - 1>();
        group_sync(grp);
        const uint8_t *V = take + g * kBlk + 8 * t;
        // A block's products have sums of their own, which its value scale takes to the running ones in fp32. (The tensor cores cut
        // off what they add below the last place; over a long context that would add up: 16384 tokens 5e-6 to 8e-6 of the outputs.)
        constexpr int kMs = kMt < 2 ? kMt : 2;                       // channel tiles at once
#pragma unroll
        for (int m0 = 0; m0 < kMt; m0 += kMs) {
#pragma unroll
            for (int j = 0; j < kTurn; ++j) {                        // block of the turn
                const float bvs = __shfl_sync(0xffffffffu, vs, kTurn * (i % kWin) + j);
                float d[kMs][NT][4];
                uint32_t af[kMs][2][4];
#pragma unroll
                for (int m = 0; m < kMs; ++m) {
                    const uint8_t *from = V + j * (8 * HD) + 16 * (m0 + m) * kBlk;
                    const uint2 v0 = *reinterpret_cast<const uint2 *>(from), v1 = *reinterpret_cast<const uint2 *>(from + 8 * kBlk);
                    af[m][0][0] = codes_lo(v0.x), af[m][0][1] = codes_lo(v1.x), af[m][0][2] = codes_hi(v0.x), af[m][0][3] = codes_hi(v1.x);
                    af[m][1][0] = codes_lo(v0.y), af[m][1][1] = codes_lo(v1.y), af[m][1][2] = codes_hi(v0.y), af[m][1][3] = codes_hi(v1.y);
                }
#pragma unroll
                for (int st = 0; st < 2; ++st) {
                    uint4 w[NT];
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
                        const Weights &from = pbuf[((2 * j + st) * NT + nt) * 32];
                        if constexpr (PK)
                            w[nt].x = from.x, w[nt].y = from.y;
                        else
                            w[nt] = from;
                    }
#pragma unroll
                    for (int part = 0; part < (PK ? 1 : 2); ++part)
#pragma unroll
                        for (int m = 0; m < kMs; ++m)
#pragma unroll
                            for (int nt = 0; nt < NT; ++nt) {
                                if (st + part == 0)
                                    mma_f16<true>(d[m][nt], af[m][st], w[nt].x, w[nt].y);
                                else
                                    mma_f16(d[m][nt], af[m][st], part ? w[nt].z : w[nt].x, part ? w[nt].w : w[nt].y);
                            }
                }
#pragma unroll
                for (int k = 0; k < kMs * NT * 4; ++k) (&o[m0][0][0])[k] = fmaf((&d[0][0][0])[k], bvs, (&o[m0][0][0])[k]);
            }
        }
        __syncwarp();
        taken();
        issue(2 * i + 1 + kRing);
    }
    cp_async_wait_groups<0>();

    // ---- the tail (at most 48 fp32 rows), by the first group: warps 0..2 take 16 keys each, then every warp its channels of
    // the values. Keys enter as two fp16 halves, each key's 64 channels scaled by a power of two of their own; values and
    // weights as three bf16 parts (fp32's range, so that no token's size touches another's precision). A token that
    // holds an infinity or a NaN makes the rows that see it NaN; its own numbers enter as 0. ----
    if (u.tail && grp == 0) {
        const int base = kBlk * p.z;
        if (!tail_only) {
            group_sync(0);                                           // every warp is done with its ring
            copy_tail(false);
        }
        cp_async_wait_groups<0>();
        group_sync(0);
        float x[NT][4];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int k = 0; k < 4; ++k) x[nt][k] = 0.f;
        const int key0 = 16 * wq + 4 * (g >> 1) + (g & 1);           // and key0 + 2
        if (wq < 3) {
            const float4 *K = reinterpret_cast<const float4 *>(tail_rows);
#pragma unroll 1
            for (int c = 0; c < HD / 64; ++c) {
                float4 kr[2][4];
                float up[2], back[2];
#pragma unroll
                for (int m = 0; m < 2; ++m)
#pragma unroll
                    for (int j = 0; j < 4; ++j) kr[m][j] = key0 + 2 * m < trows ? K[key_piece(key0 + 2 * m, 16 * c + 4 * t + j)] : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                for (int m = 0; m < 2; ++m) {
                    uint32_t top = 0;                                // magnitudes as bits: infinities and NaN come last
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const float4 y = kr[m][j];
                        top = max(max(top, __float_as_uint(y.x) & 0x7fffffffu), __float_as_uint(y.y) & 0x7fffffffu);
                        top = max(max(top, __float_as_uint(y.z) & 0x7fffffffu), __float_as_uint(y.w) & 0x7fffffffu);
                    }
                    top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
                    top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
                    const bool fin = top < 0x7f800000u;
                    up[m] = fin ? lift(__uint_as_float(top)) : 0.f;
                    back[m] = fin ? 1.f / up[m] : NAN;
                }
                float xc[NT][4];
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) xc[nt][0] = xc[nt][1] = xc[nt][2] = xc[nt][3] = 0.f;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    uint32_t ah[4], al[4];
#pragma unroll
                    for (int m = 0; m < 2; ++m) {
                        const float4 y = up[m] == 0.f ? make_float4(0.f, 0.f, 0.f, 0.f) : kr[m][j];
                        halves2(y.x * up[m], y.y * up[m], ah[m], al[m]);
                        halves2(y.z * up[m], y.w * up[m], ah[2 + m], al[2 + m]);
                    }
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
                        const uint2 *f = reinterpret_cast<const uint2 *>(qf + ((c * NT + nt) * kQ + (j >> 1)) * 32) + (j & 1);
                        const uint2 qh = f[0];
                        mma_f16(xc[nt], al, qh.x, qh.y);
                        if (!PK) {
                            const uint2 ql = f[2 * 32 * 2];
                            mma_f16(xc[nt], ah, ql.x, ql.y);
                        }
                        mma_f16(xc[nt], ah, qh.x, qh.y);
                    }
                }
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int k = 0; k < 4; ++k) x[nt][k] = fmaf(xc[nt][k], back[k >> 1], x[nt][k]);
            }
        }
        if (PK) join(x[0]);
        group_sync(0);                                               // the keys are read, and sh.top is free
        copy_tail(true);
        float y[kM][NT][kE];
        if (kM == 2)
#pragma unroll
            for (int k = 0; k < NT * kE; ++k) (&y[kM - 1][0][0])[k] = -INFINITY;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                int lo, hi;
                row_sees(nt, e, lo, hi);
#pragma unroll
                for (int k = e; k < kE; k += 2) {
                    const int pos = base + key0 + 2 * (k >> 1 | low);
                    y[0][nt][k] = wq == 3 || pos < lo || pos >= hi ? -INFINITY : x[nt][k] * (e ? scale_of(nt).y : scale_of(nt).x);
                }
            }
        renew(y);
        float *weight = reinterpret_cast<float *>(smem + S::kQBytes);   // [row][token], in the group's buffer
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const float ref = mx[nt][e] == -INFINITY ? 0.f : mx[nt][e] - kTop;
                const int r = 8 * nt + t2 + e;
                float sum = 0.f;
#pragma unroll
                for (int k = e; k < kE; k += 2) {
                    sum += y[0][nt][k] = ex2(y[0][nt][k] - ref);
                    if (wq < 3) weight[r * S::kTailPitch + key0 + 2 * (k >> 1 | low)] = y[0][nt][k];
                }
                l[nt][e] += sum;
                if (keep_lse) {
                    const float total = rows_sum(sum);
                    const int b = p.z + (wq >> 1);
                    if (g == 0 && low == 0 && r < per && b < p.b0 + p.nb) put_lse(b, wq & 1, r, total, mx[nt][e]);
                }
            }
        cp_async_wait_groups<0>();
        group_sync(0);
#pragma unroll 1
        for (int st = 0; st < 3; ++st) {
            if (16 * st >= trows) break;
            uint32_t wf[NT][2][3], poison = 0;                       // of this step's four tokens of the thread, not finite
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                float4 y = make_float4(0.f, 0.f, 0.f, 0.f);          // PK: columns 4..7 hold no rows
                if (!PK || g < 4) y = *reinterpret_cast<const float4 *>(weight + (8 * nt + g) * S::kTailPitch + 16 * st + 4 * t);
                thirds2(y.x, y.y, wf[nt][0]);
                thirds2(y.z, y.w, wf[nt][1]);
            }
#pragma unroll
            for (int mt = 0; mt < kMt; ++mt) {
                uint32_t af[3][4];
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const int key = 16 * st + 4 * t;
                    float4 vr = make_float4(0.f, 0.f, 0.f, 0.f);
                    if (key < trows) vr = *reinterpret_cast<const float4 *>(tail_rows + (wq * (HD / 4) + 16 * mt + g + 8 * k) * kTail + key);
                    float v[4] = {vr.x, vr.y, vr.z, vr.w};
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        if (key + e >= trows || !isfinite(v[e])) {
                            if (key + e < trows) poison |= 1u << e;
                            v[e] = 0.f;
                        }
                    }
                    uint32_t y0[3], y1[3];
                    thirds2(v[0], v[1], y0);
                    thirds2(v[2], v[3], y1);
#pragma unroll
                    for (int i = 0; i < 3; ++i) af[i][k] = y0[i], af[i][2 + k] = y1[i];
                }
#pragma unroll
                for (int i = 2; i >= 0; --i)                         // the small products first
#pragma unroll
                    for (int k = 2 - i; k >= 0; --k)
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) mma_bf16(o[mt][nt], af[i][0], af[i][1], af[i][2], af[i][3], wf[nt][0][k], wf[nt][1][k]);
            }
            for (; poison; poison &= poison - 1) {
                const int pos = base + 16 * st + 4 * t + __ffs(poison) - 1;
#pragma unroll 1
                for (int r = 0; r < min(live, RG); ++r) {
                    int lo, hi;
                    seen(a, p, (rg * RG + r) / per, lo, hi);
                    if (lo <= pos && hi > pos) atomicOr(&sh.poisoned, 1u << r);
                }
            }
        }
    }

    // ---- the groups' sums, merged in their order ----
    if (bad) sh.bad = 1;
    __syncthreads();                                                 // also: the shared memory may be reused
    float *om = reinterpret_cast<float *>(smem) + grp * RG * kPitch;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int r = 8 * nt + t2 + e;
            const float sum = rows_sum(l[nt][e]);
            if (g == 0) {
                sh.l[warp][r] = sum;
                if (wq == 0) sh.m[grp][r] = mx[nt][e];
            }
#pragma unroll
            for (int mt = 0; mt < kMt; ++mt) {
                float o0 = o[mt][nt][e], o1 = o[mt][nt][2 + e];
                if (PK) {                                            // the halves' sums
                    o0 += __shfl_xor_sync(0xffffffffu, o0, 2);
                    o1 += __shfl_xor_sync(0xffffffffu, o1, 2);
                }
                om[r * kPitch + wq * (HD / 4) + 16 * mt + g] = o0;
                om[r * kPitch + wq * (HD / 4) + 16 * mt + g + 8] = o1;
            }
        }
    __syncthreads();
    const size_t part = part_of(a, size_t(head) * a.groups + rg, u.index);
    if (tid == 0) {
        if (sh.bad) atomicOr(a.c.err, kErrTable);
        a.part_bad[part] = sh.bad;
    }
    if (sh.bad) return;
    if (tid < (PK ? 4 : RG)) {   // each group's factor, in place of its maximum
        float top = -INFINITY, total = 0.f;
#pragma unroll
        for (int i = 0; i < kG; ++i) top = fmaxf(top, sh.m[i][tid]);
#pragma unroll
        for (int i = 0; i < kG; ++i) {
            const float f = sh.m[i][tid] == top ? 1.f : ex2(sh.m[i][tid] - top);
            sh.m[i][tid] = f;
            total = fmaf((sh.l[4 * i][tid] + sh.l[4 * i + 1][tid]) + (sh.l[4 * i + 2][tid] + sh.l[4 * i + 3][tid]), f, total);
        }
        sh.l[0][tid] = total;
        *reinterpret_cast<float2 *>(a.part_ml + (part * RG + tid) * 2) = make_float2(top, total);
    }
    __syncthreads();
    for (int e = tid; e < min(live, RG) * (HD / 4); e += kW * 32) {
        const int r = e / (HD / 4), d = 4 * (e % (HD / 4));
        float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int i = 0; i < kG; ++i) {
            const float4 y = *reinterpret_cast<const float4 *>(reinterpret_cast<const float *>(smem) + (i * RG + r) * kPitch + d);
            const float f = sh.m[i][r];
            sum.x = fmaf(y.x, f, sum.x), sum.y = fmaf(y.y, f, sum.y), sum.z = fmaf(y.z, f, sum.z), sum.w = fmaf(y.w, f, sum.w);
        }
        if (sh.poisoned >> r & 1) sum = make_float4(NAN, NAN, NAN, NAN);
        if (u.whole) {
            const int rid = rg * RG + r;
            const float total = sh.l[0][r];
            *reinterpret_cast<float4 *>(a.out + ((size_t)s * a.rows + rid / per) * a.ldo + (size_t)(h * per + rid % per) * HD + d) =
                make_float4(sum.x / total, sum.y / total, sum.z / total, sum.w / total);
        } else {
            *reinterpret_cast<float4 *>(a.part_o + (part * RG + r) * HD + d) = sum;
        }
    }
}

// Splits: grid (splits, heads x row groups, sequences).
template <int HD, int NT, bool PK>
__global__ void __launch_bounds__(AttnShape<HD, NT, PK>::kWarps * 32, AttnShape<HD, NT, PK>::kCtas) k_kv8_attn(AttnKvArgs a) {
    constexpr int RG = 8 * NT;
    extern __shared__ __align__(16) uint8_t kv_smem[];
    __shared__ AttnShared<HD, NT> sh;
    const int split = int(blockIdx.x) - a.apart;
    Piece u{int(blockIdx.z), int(blockIdx.y) / a.groups, int(blockIdx.y) % a.groups};
    pdl_wait();
    const int sealed = a.c.sealed[(size_t)u.s * a.c.n_kv + u.h];
    Span p = span_of_seq(a, u.s, RG);
    pdl_trigger();
    if (p.z != sealed) p.bad = kErrState;
    if (p.bad) {
        if (threadIdx.x == 0 && blockIdx.x == 0) atomicOr(a.c.err, p.bad);
        return;
    }
    const int nsplit = splits_of<AttnShape<HD, NT, PK>::kStep>(a.splits, p.coded);
    u.tail = a.apart ? split < 0 : split == max(nsplit - 1, 0);
    if (u.rg >= p.groups || (split >= nsplit && !u.tail)) return;
    const bool codes = split >= 0 && split < nsplit;
    u.x0 = codes ? int((long)p.coded * split / nsplit) : 0;
    u.x1 = codes ? int((long)p.coded * (split + 1) / nsplit) : 0;
    u.whole = nsplit == 0 || (nsplit == 1 && !a.apart);
    u.index = split + a.apart;
    QueryRows<HD, NT> q;
    q.load(a, u.s, u.h, u.rg, p.n);
    attn_piece<HD, NT, PK>(a, p, u, q, kv_smem, sh);
}

// Shares: a.ctas CTAs.
template <int HD, int NT, bool PK>
__global__ void __launch_bounds__(AttnShape<HD, NT, PK>::kWarps * 32, AttnShape<HD, NT, PK>::kShareCtas) k_kv8_attn_share(AttnKvArgs a) {
    constexpr int RG = 8 * NT, kW = AttnShape<HD, NT, PK>::kWarps;
    extern __shared__ __align__(16) uint8_t kv_smem[];
    __shared__ AttnShared<HD, NT> sh;
    __shared__ long sm_sums[kW][2], sm_off;
    __shared__ int sm_seq;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, cta = blockIdx.x;
    pdl_wait();
    pdl_trigger();
    // the work in all, this CTA's share of it, and the sequence that the share begins in
    long work = 0, none = 0;
    for (int i = tid; i < a.c.n_seq; i += kW * 32) {
        const Span p = span_of_seq(a, i, RG);
        if (p.bad && cta == 0) atomicOr(a.c.err, p.bad);
        work += weight_of(a, p);
    }
    block_sums(work, none, sm_sums);
    const int G = shares_of<AttnShape<HD, NT, PK>::kStep>(a, work);
    if (cta >= G) return;
    long pos = work * cta / G, off = 0;
    const long pos_end = work * (cta + 1) / G;
    for (int base = 0; base < a.c.n_seq; base += kW * 32) {
        const long x = base + tid < a.c.n_seq ? weight_of(a, span_of_seq(a, base + tid, RG)) : 0;
        long upto = x;                                               // of the warp, then of the chunk
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long y = __shfl_up_sync(0xffffffffu, upto, o);
            if (lane >= o) upto += y;
        }
        __syncthreads();
        if (lane == 31) sm_sums[warp][0] = upto;
        if (tid == 0) sm_seq = -1;
        __syncthreads();
        long chunk = 0;
        for (int i = 0; i < kW; ++i) {
            if (i < warp) upto += sm_sums[i][0];
            chunk += sm_sums[i][0];
        }
        if (pos < off + upto && pos >= off + upto - x) sm_seq = base + tid, sm_off = off + upto - x;
        __syncthreads();
        if (sm_seq >= 0) break;
        off += chunk;
    }
    off = sm_off;
    for (int s = sm_seq; pos < pos_end;) {
        const Span p = span_of_seq(a, s, RG);
        const long mine = weight_of(a, p);
        if (pos >= off + mine) {                                     // the next sequence
            off += mine;
            ++s;
            continue;
        }
        const int weight = p.coded + kTailWeight, ui = int((pos - off) / weight), from = int(pos - off - (long)ui * weight);
        const int to = int(min((long)weight, from + pos_end - pos));
        pos += to - from;
        Piece u{s, ui / p.groups, ui % p.groups, min(from, p.coded), min(to, p.coded)};
        u.tail = from <= p.coded && to > p.coded;
        u.whole = from == 0 && u.tail;
        u.index = cta;
        if (a.c.sealed[(size_t)s * a.c.n_kv + u.h] != p.z) {         // a head that differs from the first
            if (tid == 0) atomicOr(a.c.err, kErrState);
            continue;
        }
        if (!u.tail && u.x0 == u.x1) continue;
        QueryRows<HD, NT> q;
        q.load(a, s, u.h, u.rg, p.n);
        __syncthreads();                                             // the piece before is done with the shared memory
        attn_piece<HD, NT, PK>(a, p, u, q, kv_smem, sh);
    }
}

// Latency: some 5 us behind the attention, the parts' states, then their sums, with all loads of a kind at once.
// Merges the parts of a unit's rows in a fixed order (grid x < row_ctas), and adds row 0's share of 256 blocks to the
// scores (grid x behind them, row group 0). HD / 4 threads take four channels each of a row; with `apart_rows` all threads of
// a CTA take one row and share out its parts (few units of many parts), else each such group takes a row of its own.
constexpr int kMergeThreads = 256;
constexpr int kMaxCtas = 456;   // of a launch that share or split units: three for each SM at most
template <int HD, int NT>
__global__ void __launch_bounds__(kMergeThreads) k_kv8_merge(AttnKvArgs a, int row_ctas, int apart_rows) {
    constexpr int RG = 8 * NT, kLanes = kMergeThreads / (HD / 4), kSome = 4;
    __shared__ float4 acc[kLanes][HD / 4];
    __shared__ float fac[kMaxCtas + 1], top_s[16], total_s[16];
    __shared__ long sums[kMergeThreads / 32][2];
    const int h = blockIdx.y / a.groups, rg = blockIdx.y % a.groups, s = blockIdx.z, tid = threadIdx.x, lane = tid & 31;
    const bool row_part = int(blockIdx.x) < row_ctas;
    const KvView w = view(a.c, s, h);
    const int sealed = *w.sealed;
    const Span p = span_of(a, s, sealed, RG);
    const int per = a.n_q / a.c.n_kv, live = p.n * per - rg * RG, row0 = blockIdx.x * (apart_rows ? 1 : kLanes);
    const int b0 = p.b0 + (int(blockIdx.x) - row_ctas) * kMergeThreads;
    bool off_duty = p.bad || a.c.sealed[(size_t)s * a.c.n_kv] != sealed || live <= 0 || (row_part ? row0 >= live : rg || b0 >= p.b0 + p.nb);
    long W = 0, before = 0;                                          // the work in all, and that of the sequences before s
    if (a.share && !off_duty) {
        for (int i = tid; i < a.c.n_seq; i += kMergeThreads) {
            const long x = weight_of(a, span_of_seq(a, i, RG));
            W += x;
            before += i < s ? x : 0;
        }
        block_sums(W, before, sums);
    }
    // the parts: those of the unit's CTAs
    const size_t unit = ((size_t)s * a.c.n_kv + h) * a.groups + rg;
    const int nsplit = splits_of<AttnShape<HD, NT>::kStep>(a.splits, p.coded);
    int first = 0, parts = a.apart + (a.apart ? nsplit : max(nsplit, 1));
    if (a.share && !off_duty) {
        const int G = shares_of<AttnShape<HD, NT>::kStep>(a, W);
        const long start = before + (long)(h * p.groups + rg) * (p.coded + kTailWeight);
        first = int(cta_of(start, W, G));
        parts = 1 + int(cta_of(start + p.coded, W, G)) - first;
    }
    pdl_wait();   // by every CTA, so that this grid does not end before the one it follows
    if (off_duty || (parts == 1 && row_part)) return;                // one CTA had the whole unit and has written it
    const size_t part1 = part_of(a, unit, first);
    auto id = [&](int i) { return part1 + i; };
    int bad = 0;
    for (int i = tid; i < parts; i += kMergeThreads) bad |= a.part_bad[id(i)];
    auto put = [&](int r, int d4, const float4 &sum, float total) {
        const int rid = rg * RG + r;
        *reinterpret_cast<float4 *>(a.out + ((size_t)s * a.rows + rid / per) * a.ldo + (size_t)(h * per + rid % per) * HD + 4 * d4) =
            make_float4(sum.x / total, sum.y / total, sum.z / total, sum.w / total);
    };
    auto add = [](float4 &sum, const float4 &y, float f) {
        sum.x = fmaf(y.x, f, sum.x), sum.y = fmaf(y.y, f, sum.y), sum.z = fmaf(y.z, f, sum.z), sum.w = fmaf(y.w, f, sum.w);
    };
    const int d4 = tid % (HD / 4), i0 = tid / (HD / 4);
    if (row_part && !apart_rows) {
        const int r = row0 + i0;
        const bool on = r < min(live, RG);
        float2 ml[kSome];
        float4 y[kSome];
#pragma unroll
        for (int i = 0; i < kSome; ++i)                              // the first parts' loads all at once
            if (on && i < parts) {
                ml[i] = *reinterpret_cast<const float2 *>(a.part_ml + (id(i) * RG + r) * 2);
                y[i] = *reinterpret_cast<const float4 *>(a.part_o + (id(i) * RG + r) * HD + 4 * d4);
            }
        if (__syncthreads_or(bad) || !on) return;
        float top = -INFINITY, total = 0.f;
        float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int i = 0; i < kSome; ++i)
            if (i < parts) top = fmaxf(top, ml[i].x);
        for (int i = kSome; i < parts; ++i) top = fmaxf(top, a.part_ml[(id(i) * RG + r) * 2]);
        auto take = [&](const float2 &x, const float4 &v) {
            const float f = x.x == top ? 1.f : ex2(x.x - top);
            total = fmaf(x.y, f, total);
            add(sum, v, f);
        };
#pragma unroll
        for (int i = 0; i < kSome; ++i)
            if (i < parts) take(ml[i], y[i]);
        for (int i = kSome; i < parts; ++i)
            take(*reinterpret_cast<const float2 *>(a.part_ml + (id(i) * RG + r) * 2), *reinterpret_cast<const float4 *>(a.part_o + (id(i) * RG + r) * HD + 4 * d4));
        put(r, d4, sum, total);
        return;
    }
    // A warp's view of row r: the largest maximum and the sum, and each part's factor to f. `some` holds the first 128 parts'
    // states, four a lane, asked for before.
    struct Some {
        float2 v[4];
    };
    auto ask = [&](int r) {
        Some x;
#pragma unroll
        for (int k = 0; k < 4; ++k) x.v[k] = lane + 32 * k < parts ? *reinterpret_cast<const float2 *>(a.part_ml + (id(lane + 32 * k) * RG + r) * 2) : make_float2(-INFINITY, 0.f);
        return x;
    };
    auto state = [&](int r, const Some &some, float &top, float &total, float *f) {
        top = fmaxf(fmaxf(some.v[0].x, some.v[1].x), fmaxf(some.v[2].x, some.v[3].x));
        for (int i = 128 + lane; i < parts; i += 32) top = fmaxf(top, a.part_ml[(id(i) * RG + r) * 2]);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
        total = 0.f;
        auto take = [&](int i, const float2 &y) {
            const float x = y.x == top ? 1.f : ex2(y.x - top);
            total = fmaf(y.y, x, total);
            if (f) f[i] = x;
        };
#pragma unroll
        for (int k = 0; k < 4; ++k)
            if (lane + 32 * k < parts) take(lane + 32 * k, some.v[k]);
        for (int i = 128 + lane; i < parts; i += 32) take(i, *reinterpret_cast<const float2 *>(a.part_ml + (id(i) * RG + r) * 2));
        total = warp_sum(total);
    };
    float top, total;
    if (row_part) {
        constexpr int kMany = 8;
        float4 y[kMany], sum = make_float4(0.f, 0.f, 0.f, 0.f);
        const Some some = ask(row0);
#pragma unroll
        for (int k = 0; k < kMany; ++k)                              // on their way while the factors are found
            if (i0 + k * kLanes < parts) y[k] = *reinterpret_cast<const float4 *>(a.part_o + (id(i0 + k * kLanes) * RG + row0) * HD + 4 * d4);
        if (__syncthreads_or(bad)) return;
        if (tid < 32) {
            state(row0, some, top, total, fac);
            if (lane == 0) total_s[0] = total;
        }
        __syncthreads();
#pragma unroll
        for (int k = 0; k < kMany; ++k)
            if (i0 + k * kLanes < parts) add(sum, y[k], fac[i0 + k * kLanes]);
#pragma unroll 4
        for (int i = i0 + kMany * kLanes; i < parts; i += kLanes) add(sum, *reinterpret_cast<const float4 *>(a.part_o + (id(i) * RG + row0) * HD + 4 * d4), fac[i]);
        acc[i0][d4] = sum;
        __syncthreads();
        if (i0 == 0) {
#pragma unroll
            for (int i = 1; i < kLanes; ++i) {
                const float4 v = acc[i][d4];
                sum.x += v.x, sum.y += v.y, sum.z += v.z, sum.w += v.w;
            }
            put(row0, d4, sum, total_s[0]);
        }
        return;
    }
    const int b = b0 + tid;
    float4 lse[2][4];                                                // of the halves, for up to 16 rows
    const bool on = b < p.b0 + p.nb;
    const float4 *x = reinterpret_cast<const float4 *>(a.blk_lse + (((size_t)s * a.c.n_kv + h) * w.nb + (on ? b : b0)) * 32);
#pragma unroll
    for (int k = 0; k < 2; ++k)
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (4 * i < per) lse[k][i] = x[4 * k + i];
    const float old = on ? w.score[b] : 0.f;
    for (int r = tid >> 5; r < per; r += kMergeThreads / 32) {
        state(r, ask(r), top, total, nullptr);
        if (lane == 0) top_s[r] = top - kTop, total_s[r] = total;
    }
    if (__syncthreads_or(bad) || !on) return;
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float v[2][4] = {{lse[0][i].x, lse[0][i].y, lse[0][i].z, lse[0][i].w}, {lse[1][i].x, lse[1][i].y, lse[1][i].z, lse[1][i].w}};
#pragma unroll
        for (int k = 0; k < 4; ++k)
            if (4 * i + k < per) sum += (ex2(v[0][k] - top_s[4 * i + k]) + ex2(v[1][k] - top_s[4 * i + k])) / total_s[4 * i + k];
    }
    w.score[b] = old + sum;
}

// ---- host side ----
// How a call's work is cut: row groups of 8 rows, or of 16 (whose codes are expanded once for two products) where a head
// has more than 8. Up to as many units as half the CTAs that fit the part's 152 SMs at once: splits of a unit's blocks, and
// a CTA of its own for the tail or not; all in one wave (CTAs of a second one were measured to wait for tens of microseconds
// although slots were free). Costs are in turns; a tail inside a CTA is worth about 2. More units: shares, which leave no slot
// idle but cost a little more (finding the share, pieces of two or three units, their parts' merge). So shares also take long
// contexts where whole splits leave slots idle: 128 units of 512 blocks on 304 slots take 97 us in shares and 115 in splits
// (16 rows of 128: 130 and 159), 96 units 101 and 114; but 72 units took 71 and 64, 128 units of 128 blocks 41 and 40.
constexpr int kFewRows = 4;              // rows for which both halves fit one tile of columns
struct AttnCut {
    int nt, groups, splits, apart, share, ctas;
    size_t units, o_bytes, ml_bytes, bad_bytes, lse_bytes, total;
};
size_t up256(size_t n) { return (n + 255) / 256 * 256; }
constexpr int kMaxSplits = 127;
AttnCut attn_cut(const dfl_kv8 *c, int n_q, int rows, int window, int score) {
    AttnCut t{};
    const int r = rows * (n_q / c->n_kv);
    t.nt = r > 8 ? 2 : 1;
    t.groups = (r + 8 * t.nt - 1) / (8 * t.nt);
    t.units = (size_t)c->n_seq * c->n_kv * t.groups;
    const bool wide = c->head_dim == 256 && t.nt == 2;
    const int step = wide ? AttnShape<256, 2>::kStep : c->head_dim == 256 ? AttnShape<256, 1>::kStep : AttnShape<128, 1>::kStep;
    const int slots = wide ? 152 : 2 * 152, blocks = window ? std::min(c->n_blocks, window / kBlk + 2) : c->n_blocks;
    t.splits = 1;
    t.share = t.units > (size_t)slots / 2;
    if (!t.share) {
        const int most = std::min(kMaxSplits, (blocks + step - 1) / step);
        int best = 0;
        for (int apart = 0; apart < 2; ++apart)
            for (int n = 1; n <= most && t.units * (n + apart) <= (size_t)slots; ++n) {
                const int cost = (blocks + step * n - 1) / (step * n) + (apart ? 0 : 2);
                if (!best || cost < best) best = cost, t.splits = n, t.apart = apart;
            }
        // a CTA's blocks in splits, and in shares: long ones only, and what is saved
        const size_t whole = (size_t)best * step, even = t.units * (blocks + kTailWeight) / slots;
        t.share = even >= 160 && whole >= even + 16;
    }
    if (t.share) t.splits = 1, t.apart = 0, t.ctas = r <= kFewRows && c->head_dim < 256 ? 3 * 152 : slots;
    const size_t parts = t.share ? t.units + t.ctas : t.units * (t.splits + t.apart);
    t.o_bytes = up256(parts * 8 * t.nt * c->head_dim * 4);
    t.ml_bytes = up256(parts * 8 * t.nt * 8);
    t.bad_bytes = up256(parts * 4);
    t.lse_bytes = score ? up256((size_t)c->n_seq * c->n_kv * c->n_blocks * 128) : 0;
    t.total = t.o_bytes + t.ml_bytes + t.bad_bytes + t.lse_bytes;
    return t;
}

// the kernels' shared memory, once per device
template <int HD, int NT, bool PK>
cudaError_t allow_smem() {
    const int smem = AttnShape<HD, NT, PK>::kSmem;
    const cudaError_t e = cudaFuncSetAttribute(k_kv8_attn<HD, NT, PK>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    return e != cudaSuccess ? e : cudaFuncSetAttribute(k_kv8_attn_share<HD, NT, PK>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
}
template <int HD, int NT>
cudaError_t prepare_kv8_attn() {
    static bool done[kMaxDevices] = {};
    const int dev = current_device();
    if (dev < 0) return cudaErrorInvalidDevice;
    if (done[dev]) return cudaSuccess;
    cudaError_t e = allow_smem<HD, NT, false>();
    if (e == cudaSuccess && NT == 1) e = allow_smem<HD, NT, NT == 1>();
    done[dev] = e == cudaSuccess;
    return e;
}

template <int HD, int NT, bool PK>
cudaError_t launch_kv8_pieces(const AttnKvArgs &a, cudaStream_t s) {
    const int smem = AttnShape<HD, NT, PK>::kSmem, threads = AttnShape<HD, NT, PK>::kWarps * 32;
    return a.share ? launch_pdl(k_kv8_attn_share<HD, NT, PK>, dim3(a.ctas), dim3(threads), smem, s, a)
                   : launch_pdl(k_kv8_attn<HD, NT, PK>, dim3(a.splits + a.apart, a.c.n_kv * a.groups, a.c.n_seq), dim3(threads), smem, s, a);
}
template <int HD, int NT>
cudaError_t launch_kv8_attn(const AttnKvArgs &a, cudaStream_t s) {
    cudaError_t e = prepare_kv8_attn<HD, NT>();
    if (e != cudaSuccess) return e;
    const unsigned heads = unsigned(a.c.n_kv * a.groups);
    const bool few = NT == 1 && a.rows * (a.n_q / a.c.n_kv) <= kFewRows;
    e = few ? launch_kv8_pieces<HD, NT, NT == 1>(a, s) : launch_kv8_pieces<HD, NT, false>(a, s);
    if (e != cudaSuccess) return e;
    const int apart_rows = !a.share && a.splits > 8, lanes = kMergeThreads / (HD / 4);
    const int row_ctas = apart_rows ? 8 * NT : (8 * NT + lanes - 1) / lanes;
    const unsigned x = row_ctas + (a.score ? (a.c.n_blocks + kMergeThreads - 1) / kMergeThreads : 0);
    return launch_pdl(k_kv8_merge<HD, NT>, dim3(x, heads, a.c.n_seq), dim3(kMergeThreads), 0, s, a, row_ctas, apart_rows);
}

// ---------------------------------------------------------------------------------------------------
// eviction
// ---------------------------------------------------------------------------------------------------
struct EvictArgs {
    dfl_kv8 c;
    const int32_t *len;
    int keep, sink, recent;
    int32_t *table;
    float *score;
    int32_t *sealed, *len_out;
};

// fp32 -> an unsigned key of the same order; a NaN comes first, -0 equals 0
__device__ __forceinline__ uint32_t order_key(float x) {
    if (isnan(x)) return 0u;
    const uint32_t u = __float_as_uint(x + 0.f);
    return u & 0x80000000u ? ~u : u | 0x80000000u;
}

// exclusive prefix sum over the CTA's 1024 threads
__device__ __forceinline__ int block_scan(int v, int *sums) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int x = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
    }
    __syncthreads();
    if (lane == 31) sums[warp] = x;
    __syncthreads();
    int before = lane < warp ? sums[lane] : 0;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) before += __shfl_xor_sync(0xffffffffu, before, o);
    return before + x - v;
}

// One CTA per head; a call reads and writes a few bytes a block, so its time is the latency of the steps: 5.3 us at 512 blocks,
// 10.3 us at 4096 (64 heads). The score of
// the last block kept by choice is found digit by digit (8 bits at a time, by a histogram of the candidates that agree
// so far); blocks above it are kept, and as many of those equal to it as there is room for, the lowest indexes first.
// Then the table is partitioned in order: a thread takes a run of consecutive blocks, so two prefix sums over the
// threads place them all.
constexpr int kEvictThreads = 1024;
__global__ void __launch_bounds__(kEvictThreads) k_kv8_evict(EvictArgs a) {
    __shared__ int hist[256], sums[32], pick[2];
    const int h = blockIdx.x, s = blockIdx.y, tid = threadIdx.x;
    const KvView w = view(a.c, s, h);
    const size_t base = ((size_t)s * a.c.n_kv + h) * w.nb;
    pdl_wait();
    const int n = *w.sealed, L = a.len[s];
    // the heads of a sequence thin alike, or its len would not fit them all
    const bool differ = tid < a.c.n_kv && a.c.sealed[(size_t)s * a.c.n_kv + tid] != n;
    const int bad = __syncthreads_or(n < 0 || n > w.nb) ? kErrTable : __syncthreads_or(differ) || L < kBlk * n || L > kBlk * n + kTail ? kErrState : 0;
    if (bad) {                                                   // the outputs are the inputs
        for (int b = tid; b < w.nb; b += kEvictThreads) a.table[base + b] = w.table[b], a.score[base + b] = w.score[b];
        if (tid == 0) {
            atomicOr(a.c.err, bad);
            a.sealed[(size_t)s * a.c.n_kv + h] = n;
            if (h == 0) a.len_out[s] = L;
        }
        return;
    }
    const int keep = min(n, a.keep);
    const int c0 = min(a.sink, n), c1 = max(c0, n - a.recent);   // candidates c0..c1-1
    int room = keep - (c0 + n - c1);                             // how many of them stay
    const bool all = room >= c1 - c0, some = !all && room > 0;
    uint32_t prefix = 0;
    if (some) {
        for (int shift = 24; shift >= 0; shift -= 8) {
            if (tid < 256) hist[tid] = 0;
            __syncthreads();
            for (int b = c0 + tid; b < c1; b += kEvictThreads) {
                const uint32_t key = order_key(w.score[b]);
                if (shift == 24 || (key >> (shift + 8)) == (prefix >> (shift + 8))) atomicAdd(&hist[(key >> shift) & 255], 1);
            }
            __syncthreads();
            if (tid < 32) {                                      // lane l: digits 255 - 8 l .. 248 - 8 l, from the top
                int c[8], mine = 0;
#pragma unroll
                for (int k = 0; k < 8; ++k) mine += c[k] = hist[255 - 8 * tid - k];
                int upto = mine;
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const int y = __shfl_up_sync(0xffffffffu, upto, o);
                    if (tid >= o) upto += y;
                }
                int above = upto - mine;
                if (above < room && upto >= room) {
                    int k = 0;
                    while (above + c[k] < room) above += c[k++];
                    pick[0] = 255 - 8 * tid - k;
                    pick[1] = above;
                }
            }
            __syncthreads();
            prefix |= uint32_t(pick[0]) << shift;
            room -= pick[1];
        }
    }
    // kept: outside the candidates, or above the last one kept, or equal to it and among the first `room`
    const int run = (w.nb + kEvictThreads - 1) / kEvictThreads, b0 = min(w.nb, tid * run), b1 = min(w.nb, b0 + run);
    int equal = 0, over = 0;
    for (int b = b0; b < b1; ++b) {
        const bool cand = b >= c0 && b < c1;
        const uint32_t key = some && cand ? order_key(w.score[b]) : 0;
        equal += some && cand && key == prefix;
        over += b < n && (!cand || all || (some && key > prefix));
    }
    int left = room - block_scan(equal, sums);                   // equal ones that this run may still keep
    const int kept_here = over + min(max(left, 0), equal);
    int rank = block_scan(kept_here, sums);
    for (int b = b0; b < b1; ++b) {
        const bool cand = b >= c0 && b < c1;
        const float score = w.score[b];
        const uint32_t key = some && cand ? order_key(score) : 0;
        bool kept = b < n && (!cand || all || (some && key > prefix));
        if (some && cand && key == prefix) kept = left-- > 0;
        a.table[base + (kept ? rank : b < n ? keep + (b - rank) : b)] = w.table[b];
        if (kept) a.score[base + rank] = score;
        if (b >= keep) {   // the tail's two blocks follow the kept ones; nothing is held behind them
            const int from = b + n - keep;
            a.score[base + b] = b < keep + 2 && from < w.nb ? w.score[from] : 0.f;
        }
        rank += kept;
    }
    if (tid == 0) {
        a.sealed[(size_t)s * a.c.n_kv + h] = keep;
        if (h == 0) a.len_out[s] = L - kBlk * (n - keep);
    }
}

__global__ void k_kv8_init(dfl_kv8 c) {
    const size_t heads = (size_t)c.n_seq * c.n_kv, n = heads * c.n_blocks;
    const size_t i0 = blockIdx.x * (size_t)blockDim.x + threadIdx.x, step = (size_t)gridDim.x * blockDim.x;
    for (size_t i = i0; i < n; i += step) {
        c.table[i] = int32_t(i % c.n_blocks);
        if (c.score) c.score[i] = 0.f;
        if (i < heads) c.sealed[i] = 0;
    }
    if (i0 == 0) *c.err = 0;
}

// ---------------------------------------------------------------------------------------------------
// argument checks
// ---------------------------------------------------------------------------------------------------
bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

int check_cache(const dfl_kv8 *c) {
    if (!c || c->n_seq < 1 || c->n_seq > 65535 || c->n_kv < 1 || c->n_kv > 1024 || c->n_blocks < 1 || c->n_blocks > (1 << 20))
        return DFL_E_INVALID_ARG;
    if (c->head_dim != 64 && c->head_dim != 128 && c->head_dim != 256) return DFL_E_UNSUPPORTED;
    const void *p[] = {c->k, c->v, c->k_scale, c->v_scale, c->k_tail, c->v_tail, c->table, c->sealed, c->err};
    for (const void *q : p)
        if (!q || !aligned16(q)) return DFL_E_INVALID_ARG;
    return aligned16(c->score) ? DFL_OK : DFL_E_INVALID_ARG;
}

int check_rows(const dfl_kv8 *c, const void *p, int64_t ld, int heads) {
    return p && aligned16(p) && ld % 4 == 0 && ld >= (int64_t)heads * c->head_dim ? DFL_OK : DFL_E_INVALID_ARG;
}

struct Range {
    const void *p;
    size_t bytes;
};
bool overlap(const Range &a, const Range &b) {
    const uintptr_t x = reinterpret_cast<uintptr_t>(a.p), y = reinterpret_cast<uintptr_t>(b.p);
    return x < y + b.bytes && y < x + a.bytes;
}

int launched(cudaError_t e) { return e == cudaSuccess ? DFL_OK : DFL_E_CUDA; }

int write_rows(const dfl_kv8 *c, const int32_t *len, const int32_t *cnt, int rows, const float *k, const float *v, int64_t ld,
               int commit, cudaStream_t s) {
    int rc = check_cache(c);
    if (rc) return rc;
    if (!len || rows < 1) return DFL_E_INVALID_ARG;
    if ((rc = check_rows(c, k, ld, c->n_kv)) || (rc = check_rows(c, v, ld, c->n_kv))) return rc;
    if (!commit && rows > DFL_MAX_ROWS) return DFL_E_UNSUPPORTED;
    if (rows > kBlk * c->n_blocks) return DFL_E_CAPACITY;
    WriteArgs a{*c, len, cnt, k, v, ld, rows, commit, 1};
    // Up to 64 rows complete three blocks at most: one launch. More rows take a launch with a CTA for each run of blocks and a
    // short one behind it: at 1024 rows of 8 heads of 128 they take 7 us, one CTA a head alone 260 us.
    if (!commit || rows <= 64) {
        const dim3 grid(c->n_kv, c->n_seq);
        return launched(c->head_dim == 64    ? launch_pdl(k_kv8_write<64>, grid, dim3(kWriteThreads), 0, s, a)
                        : c->head_dim == 128 ? launch_pdl(k_kv8_write<128>, grid, dim3(kWriteThreads), 0, s, a)
                                             : launch_pdl(k_kv8_write<256>, grid, dim3(kWriteThreads), 0, s, a));
    }
    const int blocks = (kTail + rows) / kBlk;
    // runs of up to 4 blocks, as long as the part's 152 SMs still get four CTAs each (8 x 8192 rows of 8 heads of 128: 142 us,
    // with a block a CTA 173)
    a.run = int(std::min<size_t>(4, std::max<size_t>(1, (size_t)2 * blocks * c->n_kv * c->n_seq / (4 * 152))));
    const dim3 grid(2 * ((blocks + a.run - 1) / a.run), c->n_kv, c->n_seq);
    const int l = launched(c->head_dim == 64    ? launch_pdl(k_kv8_append<64>, grid, dim3(128), 0, s, a)
                           : c->head_dim == 128 ? launch_pdl(k_kv8_append<128>, grid, dim3(256), 0, s, a)
                                                : launch_pdl(k_kv8_append<256>, grid, dim3(512), 0, s, a));
    return l ? l : launched(launch_pdl(k_kv8_count, dim3(c->n_kv, c->n_seq), dim3(64), 0, s, a));
}

}  // namespace

cudaError_t kv8_attn_prepare() {
    cudaError_t e;
    if ((e = prepare_kv8_attn<64, 1>()) || (e = prepare_kv8_attn<64, 2>()) || (e = prepare_kv8_attn<128, 1>()) || (e = prepare_kv8_attn<128, 2>()) ||
        (e = prepare_kv8_attn<256, 1>()))
        return e;
    return prepare_kv8_attn<256, 2>();
}

}  // namespace dfl

using namespace dfl;

extern "C" {

int dfl_kv8_init(const dfl_kv8 *c, void *stream) {
    const int rc = check_cache(c);
    if (rc) return rc;
    const size_t n = (size_t)c->n_seq * c->n_kv * c->n_blocks;
    k_kv8_init<<<unsigned(std::min<size_t>((n + 255) / 256, 1024)), 256, 0, static_cast<cudaStream_t>(stream)>>>(*c);
    return launched(cudaGetLastError());
}

int dfl_kv8_status(const dfl_kv8 *c, void *stream) {
    const int rc = check_cache(c);
    if (rc) return rc;
    int bits = 0;
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (cudaMemcpyAsync(&bits, c->err, 4, cudaMemcpyDeviceToHost, s) != cudaSuccess || cudaStreamSynchronize(s) != cudaSuccess)
        return DFL_E_CUDA;
    if (!bits) return DFL_OK;
    if (cudaMemsetAsync(c->err, 0, 4, s) != cudaSuccess) return DFL_E_CUDA;
    return bits & kErrTable ? DFL_E_INVALID_ARG : bits & kErrState ? DFL_E_STATE : DFL_E_CAPACITY;
}

int dfl_kv8_append(const dfl_kv8 *c, const int32_t *len, const int32_t *cnt, int rows, const float *k, const float *v, int64_t ld,
                   void *stream) {
    return write_rows(c, len, cnt, rows, k, v, ld, 1, static_cast<cudaStream_t>(stream));
}

int dfl_kv8_stage(const dfl_kv8 *c, const int32_t *len, const int32_t *cnt, int rows, const float *k, const float *v, int64_t ld,
                  void *stream) {
    return write_rows(c, len, cnt, rows, k, v, ld, 0, static_cast<cudaStream_t>(stream));
}

int64_t dfl_kv8_attn_scratch_bytes(const dfl_kv8 *c, int n_q, int rows, int window, int score) {
    if (!c || c->n_seq < 1 || c->n_kv < 1 || c->n_blocks < 1 || n_q < 1 || n_q % c->n_kv || n_q / c->n_kv > kMaxGroup || rows < 1 ||
        rows > DFL_MAX_ROWS || window < 0 || (c->head_dim != 64 && c->head_dim != 128 && c->head_dim != 256))
        return -1;
    return (int64_t)attn_cut(c, n_q, rows, window, score).total;
}

int dfl_kv8_attn(const dfl_kv8 *c, const float *q, int64_t ldq, int n_q, int rows, const int32_t *len, const int32_t *cnt, int window,
                 int causal, float scale, int score, float *out, int64_t ldo, void *scratch, size_t scratch_bytes, void *stream) {
    int rc = check_cache(c);
    if (rc) return rc;
    if (n_q < 1 || n_q % c->n_kv || rows < 1 || window < 0 || !len || !std::isfinite(scale)) return DFL_E_INVALID_ARG;
    if (n_q / c->n_kv > kMaxGroup || rows > DFL_MAX_ROWS) return DFL_E_UNSUPPORTED;
    if ((rc = check_rows(c, q, ldq, n_q)) || (rc = check_rows(c, out, ldo, n_q))) return rc;
    if (score && !c->score) return DFL_E_INVALID_ARG;
    const AttnCut t = attn_cut(c, n_q, rows, window, score);
    if (!scratch || (reinterpret_cast<uintptr_t>(scratch) & 255) || scratch_bytes < t.total) return DFL_E_INVALID_ARG;
    AttnKvArgs a{*c, q, out, ldq, ldo, n_q, rows, window, causal != 0, score != 0, len, cnt, scale, t.groups, t.splits, t.apart, t.share, t.ctas};
    uint8_t *at = static_cast<uint8_t *>(scratch);
    a.part_o = reinterpret_cast<float *>(at);
    a.part_ml = reinterpret_cast<float *>(at += t.o_bytes);
    a.part_bad = reinterpret_cast<int *>(at += t.ml_bytes);
    a.blk_lse = reinterpret_cast<float *>(at += t.bad_bytes);
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    cudaError_t e;
    if (c->head_dim == 64)
        e = t.nt == 1 ? launch_kv8_attn<64, 1>(a, st) : launch_kv8_attn<64, 2>(a, st);
    else if (c->head_dim == 128)
        e = t.nt == 1 ? launch_kv8_attn<128, 1>(a, st) : launch_kv8_attn<128, 2>(a, st);
    else
        e = t.nt == 1 ? launch_kv8_attn<256, 1>(a, st) : launch_kv8_attn<256, 2>(a, st);
    return e == cudaSuccess ? DFL_OK : DFL_E_CUDA;
}

int dfl_kv8_evict(const dfl_kv8 *c, const int32_t *len, int keep, int sink, int recent, int32_t *table_out, float *score_out,
                  int32_t *sealed_out, int32_t *len_out, void *stream) {
    const int rc = check_cache(c);
    if (rc) return rc;
    if (!c->score || !len || !table_out || !score_out || !sealed_out || !len_out || keep < 0 || sink < 0 || recent < 0 ||
        (int64_t)sink + recent > keep)
        return DFL_E_INVALID_ARG;
    const size_t heads = (size_t)c->n_seq * c->n_kv * 4, all = heads * c->n_blocks, seqs = (size_t)c->n_seq * 4;
    const Range r[] = {{table_out, all}, {score_out, all}, {sealed_out, heads}, {len_out, seqs},      // written
                       {c->table, all},  {c->score, all},  {c->sealed, heads},  {len, seqs},     {c->err, 4}};
    for (int i = 0; i < 4; ++i)
        for (int j = i + 1; j < 9; ++j)
            if (overlap(r[i], r[j])) return DFL_E_INVALID_ARG;
    EvictArgs a{*c, len, keep, sink, recent, table_out, score_out, sealed_out, len_out};
    return launched(launch_pdl(k_kv8_evict, dim3(c->n_kv, c->n_seq), dim3(kEvictThreads), 0, static_cast<cudaStream_t>(stream), a));
}

int dfl_kv8_read(const dfl_kv8 *c, const int32_t *len, const int32_t *first, int rows, float *k_out, float *v_out, void *stream) {
    const int rc = check_cache(c);
    if (rc) return rc;
    if (!len || !k_out || !v_out || !aligned16(k_out) || !aligned16(v_out) || rows < 1) return DFL_E_INVALID_ARG;
    const int blocks = std::min(rows / kBlk + 2, c->n_blocks + 2);   // that the range can touch
    ReadArgs a{*c, len, first, k_out, v_out, rows};
    return launched(launch_pdl(k_kv8_read, dim3(blocks, c->n_kv, c->n_seq), dim3(256), 0, static_cast<cudaStream_t>(stream), a));
}

}  // extern "C"
