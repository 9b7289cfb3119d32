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

// The code of x at `scale` > 0, 128 + the integer nearest to x / scale, exactly: away from a border between
// two codes the fp32 quotient (off by less than 2^-15 at |quotient| <= 128) decides; within 2^-10 of one,
// and for scales whose reciprocal leaves the normal range, the quotient is taken in fp64, which tells the
// quotient of two fp32 numbers from a border.
__device__ __forceinline__ uint32_t code_of(float x, float scale, float inv) {
    const float y = x * inv;
    float c = rintf(y);
    if (scale < 1e-30f || fabsf(fabsf(y - c) - 0.5f) < 0.0009765625f) c = float(rint((double)x / (double)scale));
    return uint32_t(int(fminf(fmaxf(c, -127.f), 127.f)) + 128);
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
};

// What a call does to one head: tokens from 32 z on are `have` rows of the tail (or, after a cut, of block
// z's codes) and n new rows; the first `full` blocks of them are sealed, the rest goes to the tail.
struct Plan {
    int z, have, n, full, cut, bad;
};
__device__ __forceinline__ Plan plan_of(const WriteArgs &a, int s, const KvView &w, int *err) {
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

constexpr int kWriteThreads = 512;       // 256 for the keys, 256 for the values

// One CTA per head: it seals the head's blocks one after another, then moves the rest to the tail.
__global__ void __launch_bounds__(kWriteThreads) k_kv8_write(WriteArgs a) {
    __shared__ float red[2][8];
    __shared__ int bad[2];
    __shared__ int tab_bad;
    const int h = blockIdx.x, s = blockIdx.y, hd = a.c.head_dim;
    const bool is_v = threadIdx.x >= 256;
    const int tid = threadIdx.x & 255, lane = tid & 31, warp = tid >> 5;
    KvView w = view(a.c, s, h);
    Plan p = plan_of(a, s, w, a.c.err);
    if (threadIdx.x == 0) tab_bad = 0;
    __syncthreads();
    if (!p.bad)   // every table entry that the call follows
        for (int b = threadIdx.x; b < max(p.full, p.cut); b += blockDim.x)
            if (unsigned(w.table[p.z + b]) >= unsigned(w.nb)) tab_bad = 1;
    __syncthreads();
    if (tab_bad) p.bad = kErrTable;
    if (p.bad) {
        if (threadIdx.x == 0) atomicOr(a.c.err, p.bad);
        return;
    }
    const float *src = (is_v ? a.v : a.k) + (size_t)s * a.rows * a.ld + (size_t)h * hd;
    float *tail = is_v ? w.vt : w.kt;
    uint8_t *codes = is_v ? w.v : w.k;
    float *scales = is_v ? w.vs : w.ks;
    const size_t blk = (size_t)kBlk * hd;
    const int cut_phys = p.cut ? w.table[p.z] : 0;
    const uint8_t *old = codes + cut_phys * blk;
    const float old_scale = p.cut ? scales[cut_phys] : 0.f;
    auto row = [&](int r, int d) -> float {   // token 32 z + r, channel d
        if (r >= p.have) return src[(size_t)(r - p.have) * a.ld + d];
        if (p.cut) return expand(old[is_v ? v_at(r, d) : k_at(r, d)], old_scale);
        return is_v ? tail[(size_t)d * kTail + r] : tail[(size_t)r * hd + d];
    };
    const int dgroups = hd / 4;              // a thread takes 4 channels (keys) or 4 tokens (values) at a time
    for (int b = 0; b < p.full; ++b) {
        float x[8][4];
        float amax = 0.f;
        int nonfinite = 0;
        for (int i = 0; i < hd / 32; ++i) {
            const int e = i * 256 + tid;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int t = is_v ? 4 * (e / hd) + j : e / dgroups;
                const int d = is_v ? e % hd : 4 * (e % dgroups) + j;
                const float f = row(kBlk * b + t, d);
                x[i][j] = f;
                if (isfinite(f))
                    amax = fmaxf(amax, fabsf(f));
                else
                    nonfinite = 1;
            }
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
        __syncthreads();
        if (tid == 0) bad[is_v] = 0;
        if (lane == 0) red[is_v][warp] = amax;
        __syncthreads();
        if (nonfinite) bad[is_v] = 1;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < 8; ++i) amax = fmaxf(amax, red[is_v][i]);
        const float scale = bad[is_v] ? NAN : __fdiv_rn(amax, 127.f);
        const float inv = scale > 0.f ? 1.f / scale : 0.f;
        const int phys = w.table[p.z + b];
        uint8_t *dst = codes + phys * blk;
        for (int i = 0; i < hd / 32; ++i) {
            const int e = i * 256 + tid;
            uint32_t word = 0;
#pragma unroll
            for (int j = 0; j < 4; ++j) word |= (scale > 0.f ? code_of(x[i][j], scale, inv) : 128u) << (8 * j);
            const int at = is_v ? v_at(4 * (e / hd), e % hd) : k_at(e / dgroups, 4 * (e % dgroups));
            *reinterpret_cast<uint32_t *>(dst + at) = word;
        }
        if (tid == 0) scales[phys] = scale;
    }
    __syncthreads();   // block 0 has read the tail's first rows
    // The rest moves to the tail's front. A row that comes from the tail lies 32 * full >= 32 rows further
    // back, behind all rows written here, or is where it belongs.
    const int left = p.have + p.n - kBlk * p.full;
    for (int e = tid; e < left * hd; e += 256) {
        const int t = e / hd, d = e % hd, r = kBlk * p.full + t;
        if (!p.cut && p.full == 0 && r < p.have) continue;
        const float f = row(r, d);
        if (is_v)
            tail[(size_t)d * kTail + t] = f;
        else
            tail[(size_t)t * hd + d] = f;
    }
    if (w.score) {
        const int L = a.len[s];
        for (int b = (L + kBlk - 1) / kBlk + threadIdx.x; b * kBlk < L + p.n; b += blockDim.x) w.score[b] = 0.f;
    }
    if (threadIdx.x == 0) *w.sealed = p.z + p.full;
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

// One CTA per 32-token block of the range and head: grid (blocks, heads, sequences).
__global__ void __launch_bounds__(256) k_kv8_read(ReadArgs a) {
    const int h = blockIdx.y, s = blockIdx.z, hd = a.c.head_dim;
    const KvView w = view(a.c, s, h);
    const int L = a.len[s], first = a.first ? a.first[s] : 0, z = *w.sealed;
    int bad = 0;
    if (z < 0 || z > w.nb)
        bad = kErrTable;
    else if (L < 0 || L > kBlk * w.nb || first < 0)
        bad = kErrCapacity;
    else if (L > kBlk * z + kTail)
        bad = kErrState;
    if (!bad && first >= L) return;
    const int b = bad ? 0 : first / kBlk + blockIdx.x;
    if (!bad && b < z && unsigned(w.table[b]) >= unsigned(w.nb)) bad = kErrTable;
    if (bad) {
        if (threadIdx.x == 0) atomicOr(a.c.err, bad);
        return;
    }
    const int hi = int(min((long long)L, (long long)first + a.rows));
    const size_t blk = (size_t)kBlk * hd;
    const int phys = b < z ? w.table[b] : 0;
    const float ks = b < z ? w.ks[phys] : 0.f, vs = b < z ? w.vs[phys] : 0.f;
    for (int e = threadIdx.x; e < kBlk * hd; e += blockDim.x) {
        const int t = e / hd, d = e % hd, pos = kBlk * b + t;
        if (pos < first || pos >= hi) continue;
        const size_t o = (((size_t)s * a.rows + (pos - first)) * a.c.n_kv + h) * hd + d;
        if (b < z) {
            a.k[o] = expand(w.k[phys * blk + k_at(t, d)], ks);
            a.v[o] = expand(w.v[phys * blk + v_at(t, d)], vs);
        } else {
            const int r = pos - kBlk * z;
            a.k[o] = w.kt[(size_t)r * hd + d];
            a.v[o] = w.vt[(size_t)d * kTail + r];
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
};

struct Span {
    int z, L, n, bad;   // sealed blocks, committed tokens, staged rows
};
__device__ __forceinline__ Span span_of(const AttnKvArgs &a, int s, const KvView &w) {
    Span p{*w.sealed, a.len[s], rows_of(a.cnt, s, a.rows), 0};
    if (p.z < 0 || p.z > w.nb)
        p.bad = kErrTable;
    else if (p.L < 0 || p.L > kBlk * w.nb - p.n)
        p.bad = kErrCapacity;
    else if (p.L < kBlk * p.z || p.L + p.n > kBlk * p.z + kTail)
        p.bad = kErrState;
    return p;
}
// the tokens lo..hi-1 that row m sees
__device__ __forceinline__ void seen(const AttnKvArgs &a, const Span &p, int m, int &lo, int &hi) {
    const int at = a.causal ? p.L + m : p.L - 1;   // the last token that the window counts from
    lo = a.window > 0 ? max(0, at - a.window + 1) : 0;
    hi = a.causal ? p.L + m + 1 : p.L + p.n;
}

// One CTA per head of a sequence: its warps share out the keys of one query row after another, a lane takes
// every 32nd channel.
constexpr int kSimpleThreads = 256;
__global__ void __launch_bounds__(kSimpleThreads) k_kv8_attn_simple(AttnKvArgs a) {
    __shared__ float sm_o[8][256], sm_m[8], sm_l[8];
    __shared__ int tab_bad;
    const int h = blockIdx.x, s = blockIdx.y, hd = a.c.head_dim, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const KvView w = view(a.c, s, h);
    Span p = span_of(a, s, w);
    const int group = a.n_q / a.c.n_kv;
    if (threadIdx.x == 0) tab_bad = 0;
    __syncthreads();
    if (!p.bad)
        for (int b = threadIdx.x; b < p.z; b += blockDim.x)
            if (unsigned(w.table[b]) >= unsigned(w.nb)) tab_bad = 1;
    __syncthreads();
    if (tab_bad) p.bad = kErrTable;
    if (p.bad) {
        if (threadIdx.x == 0) atomicOr(a.c.err, p.bad);
        return;
    }
    const size_t blk = (size_t)kBlk * hd;
    auto key = [&](int j, int d) {
        const int b = j / kBlk, t = j % kBlk;
        if (b >= p.z) return w.kt[(size_t)(j - kBlk * p.z) * hd + d];
        const int phys = w.table[b];
        return expand(w.k[phys * blk + k_at(t, d)], w.ks[phys]);
    };
    auto value = [&](int j, int d) {
        const int b = j / kBlk, t = j % kBlk;
        if (b >= p.z) return w.vt[(size_t)d * kTail + (j - kBlk * p.z)];
        const int phys = w.table[b];
        return expand(w.v[phys * blk + v_at(t, d)], w.vs[phys]);
    };
    for (int r = 0; r < p.n * group; ++r) {
        const int m = r / group, qh = h * group + r % group;
        int lo, hi;
        seen(a, p, m, lo, hi);
        const float *q = a.q + ((size_t)s * a.rows + m) * a.ldq + (size_t)qh * hd;
        float qr[8], o[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) qr[i] = 32 * i + lane < hd ? q[32 * i + lane] : 0.f, o[i] = 0.f;
        auto logit = [&](int j) {
            float x = 0.f;
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (32 * i < hd) x = fmaf(qr[i], key(j, 32 * i + lane), x);
            return warp_sum(x) * a.scale;
        };
        float mx = -INFINITY, l = 0.f;
        for (int j = lo + warp; j < hi; j += 8) {
            const float x = logit(j), mn = fmaxf(mx, x);
            const float f = mx == mn ? 1.f : expf(mx - mn), e = expf(x - mn);
            l = fmaf(l, f, e);
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (32 * i < hd) o[i] = fmaf(o[i], f, e * value(j, 32 * i + lane));
            mx = mn;
        }
        if (lane == 0) sm_m[warp] = mx, sm_l[warp] = l;
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (32 * i < hd) sm_o[warp][32 * i + lane] = o[i];
        __syncthreads();
        float top = -INFINITY, total = 0.f;
        for (int i = 0; i < 8; ++i) top = fmaxf(top, sm_m[i]);
        for (int i = 0; i < 8; ++i) total += sm_m[i] == -INFINITY ? 0.f : sm_l[i] * expf(sm_m[i] - top);
        for (int d = threadIdx.x; d < hd; d += blockDim.x) {
            float x = 0.f;
            for (int i = 0; i < 8; ++i) x += sm_m[i] == -INFINITY ? 0.f : sm_o[i][d] * expf(sm_m[i] - top);
            a.out[((size_t)s * a.rows + m) * a.ldo + (size_t)qh * hd + d] = x / total;
        }
        if (a.score && m == 0)
            for (int b = lo / kBlk + warp; b * kBlk < hi; b += 8) {
                float x = 0.f;
                for (int j = max(lo, b * kBlk); j < min(hi, (b + 1) * kBlk); ++j) x += expf(logit(j) - top) / total;
                if (lane == 0) w.score[b] += x;
            }
        __syncthreads();
    }
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

// exclusive prefix sum over the CTA's threads (blockDim.x = 1024); *total = the sum
__device__ __forceinline__ int block_scan(int v, int *sums, int *total) {
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
    int before = 0, all = 0;
    for (int i = 0; i < 32; ++i) {
        if (i < warp) before += sums[i];
        all += sums[i];
    }
    *total = all;
    return before + x - v;
}

// One CTA per head. The score of the last block kept by choice is found digit by digit (8 bits at a time, by a
// histogram of the candidates that agree so far); blocks above it are kept, and as many of those equal to
// it as there is room for, the lowest indexes first. Then the table is partitioned in order.
constexpr int kEvictThreads = 1024;
__global__ void __launch_bounds__(kEvictThreads) k_kv8_evict(EvictArgs a) {
    __shared__ int hist[256], sums[32], pick[2];
    const int h = blockIdx.x, s = blockIdx.y, tid = threadIdx.x;
    const KvView w = view(a.c, s, h);
    const size_t base = ((size_t)s * a.c.n_kv + h) * w.nb;
    const int n = *w.sealed;
    if (n < 0 || n > w.nb) {
        if (tid == 0) atomicOr(a.c.err, kErrTable);
        return;
    }
    const int keep = min(n, a.keep);
    const int c0 = min(a.sink, n), c1 = max(c0, n - a.recent);   // candidates c0..c1-1
    int room = keep - (c0 + n - c1);                             // how many of them stay
    const bool all = room >= c1 - c0, none = room <= 0;
    uint32_t prefix = 0;
    if (!all && !none) {
        for (int shift = 24; shift >= 0; shift -= 8) {
            if (tid < 256) hist[tid] = 0;
            __syncthreads();
            for (int b = c0 + tid; b < c1; b += kEvictThreads) {
                const uint32_t key = order_key(w.score[b]);
                if (shift == 24 || (key >> (shift + 8)) == (prefix >> (shift + 8))) atomicAdd(&hist[(key >> shift) & 255], 1);
            }
            __syncthreads();
            if (tid == 0) {
                int above = 0, d = 255;
                while (above + hist[d] < room) above += hist[d--];
                pick[0] = d;
                pick[1] = above;
            }
            __syncthreads();
            prefix |= uint32_t(pick[0]) << shift;
            room -= pick[1];
        }
    }
    // kept: outside the candidates, or above the last one kept, or equal to it and among the first `room`
    int kept_before = 0, equal_before = 0;
    for (int b0 = 0; b0 < w.nb; b0 += kEvictThreads) {
        const int b = b0 + tid;
        const bool held = b < n, cand = b >= c0 && b < c1;
        const uint32_t key = cand && !all && !none ? order_key(w.score[b]) : 0;
        const int eq = cand && !all && !none && key == prefix;
        int total_eq = 0;
        const int rank_eq = equal_before + block_scan(eq, sums, &total_eq);
        const bool kept = held && (!cand || all || (!none && (key > prefix || (eq && rank_eq < room))));
        int total_kept = 0;
        const int rank = kept_before + block_scan(kept, sums, &total_kept);
        if (b < w.nb) {
            const int to = kept ? rank : held ? keep + (b - rank) : b;
            a.table[base + to] = w.table[b];
            if (kept) a.score[base + to] = w.score[b];
            if (b >= keep) {   // the tail's two blocks follow the kept ones; nothing is held behind them
                const int from = b + n - keep;
                a.score[base + b] = b < keep + 2 && from < w.nb ? w.score[from] : 0.f;
            }
        }
        kept_before += total_kept;
        equal_before += total_eq;
    }
    if (tid == 0) {
        a.sealed[(size_t)s * a.c.n_kv + h] = keep;
        if (h == 0) a.len_out[s] = a.len[s] - kBlk * (n - keep);
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
    if (!c || c->n_seq < 1 || c->n_seq > 65535 || c->n_kv < 1 || c->n_kv > 65535 || c->n_blocks < 1 || c->n_blocks > (1 << 20))
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

int launched() { return cudaGetLastError() == cudaSuccess ? DFL_OK : DFL_E_CUDA; }

int write_rows(const dfl_kv8 *c, const int32_t *len, const int32_t *cnt, int rows, const float *k, const float *v, int64_t ld,
               int commit, cudaStream_t s) {
    int rc = check_cache(c);
    if (rc) return rc;
    if (!len || rows < 1) return DFL_E_INVALID_ARG;
    if ((rc = check_rows(c, k, ld, c->n_kv)) || (rc = check_rows(c, v, ld, c->n_kv))) return rc;
    if (!commit && rows > DFL_MAX_ROWS) return DFL_E_UNSUPPORTED;
    if (rows > kBlk * c->n_blocks) return DFL_E_CAPACITY;
    WriteArgs a{*c, len, cnt, k, v, ld, rows, commit};
    k_kv8_write<<<dim3(c->n_kv, c->n_seq), kWriteThreads, 0, s>>>(a);
    return launched();
}

}  // namespace
}  // namespace dfl

using namespace dfl;

extern "C" {

int dfl_kv8_init(const dfl_kv8 *c, void *stream) {
    const int rc = check_cache(c);
    if (rc) return rc;
    const size_t n = (size_t)c->n_seq * c->n_kv * c->n_blocks;
    k_kv8_init<<<unsigned(std::min<size_t>((n + 255) / 256, 1024)), 256, 0, static_cast<cudaStream_t>(stream)>>>(*c);
    return launched();
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

int64_t dfl_kv8_attn_scratch_bytes(const dfl_kv8 *c, int n_q, int rows, int score) {
    if (!c || c->n_seq < 1 || c->n_kv < 1 || c->n_blocks < 1 || n_q < 1 || n_q % c->n_kv || n_q / c->n_kv > kMaxGroup || rows < 1 ||
        rows > DFL_MAX_ROWS || (c->head_dim != 64 && c->head_dim != 128 && c->head_dim != 256))
        return -1;
    (void)score;
    return 256;
}

int dfl_kv8_attn(const dfl_kv8 *c, const float *q, int64_t ldq, int n_q, int rows, const int32_t *len, const int32_t *cnt, int window,
                 int causal, float scale, int score, float *out, int64_t ldo, void *scratch, size_t scratch_bytes, void *stream) {
    int rc = check_cache(c);
    if (rc) return rc;
    if (n_q < 1 || n_q % c->n_kv || rows < 1 || window < 0 || !len || !std::isfinite(scale)) return DFL_E_INVALID_ARG;
    if (n_q / c->n_kv > kMaxGroup || rows > DFL_MAX_ROWS) return DFL_E_UNSUPPORTED;
    if ((rc = check_rows(c, q, ldq, n_q)) || (rc = check_rows(c, out, ldo, n_q))) return rc;
    if (score && !c->score) return DFL_E_INVALID_ARG;
    if (!scratch || (reinterpret_cast<uintptr_t>(scratch) & 255) || (int64_t)scratch_bytes < dfl_kv8_attn_scratch_bytes(c, n_q, rows, score))
        return DFL_E_INVALID_ARG;
    AttnKvArgs a{*c, q, out, ldq, ldo, n_q, rows, window, causal != 0, score != 0, len, cnt, scale};
    k_kv8_attn_simple<<<dim3(c->n_kv, c->n_seq), kSimpleThreads, 0, static_cast<cudaStream_t>(stream)>>>(a);
    return launched();
}

int dfl_kv8_evict(const dfl_kv8 *c, const int32_t *len, int keep, int sink, int recent, int32_t *table_out, float *score_out,
                  int32_t *sealed_out, int32_t *len_out, void *stream) {
    const int rc = check_cache(c);
    if (rc) return rc;
    if (!c->score || !len || !table_out || !score_out || !sealed_out || !len_out || keep < 0 || sink < 0 || recent < 0 ||
        (int64_t)sink + recent > keep)
        return DFL_E_INVALID_ARG;
    if (table_out == c->table || score_out == c->score || sealed_out == c->sealed || len_out == len) return DFL_E_INVALID_ARG;
    EvictArgs a{*c, len, keep, sink, recent, table_out, score_out, sealed_out, len_out};
    k_kv8_evict<<<dim3(c->n_kv, c->n_seq), kEvictThreads, 0, static_cast<cudaStream_t>(stream)>>>(a);
    return launched();
}

int dfl_kv8_read(const dfl_kv8 *c, const int32_t *len, const int32_t *first, int rows, float *k_out, float *v_out, void *stream) {
    const int rc = check_cache(c);
    if (rc) return rc;
    if (!len || !k_out || !v_out || !aligned16(k_out) || !aligned16(v_out) || rows < 1) return DFL_E_INVALID_ARG;
    const int blocks = std::min(rows / kBlk + 2, c->n_blocks + 2);   // that the range can touch
    ReadArgs a{*c, len, first, k_out, v_out, rows};
    k_kv8_read<<<dim3(blocks, c->n_kv, c->n_seq), 256, 0, static_cast<cudaStream_t>(stream)>>>(a);
    return launched();
}

}  // extern "C"
