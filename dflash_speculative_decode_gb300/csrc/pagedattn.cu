// pagedattn.cu -- attention of one token, or of a verify's rows, over the paged cache (include/dfl.h, dfl_paged_attn).
//
// The call reads every visible key and value once for each chunk of up to 64 query rows x heads, so it is bound by HBM as long
// as few rows share them. The keys
// of all units (a sequence, a key/value head, a chunk of query rows) lie one after another on a line of granules of
// 64, which is cut evenly among the CTAs: the lengths of a batch, which the host does not know, decide nothing but
// where the cuts fall. A unit that a cut goes through leaves a part (sums, maximum, weight) for each CTA, and a
// second launch adds the parts in their order.
//
// A CTA is four warps with a ring of tiles of 64 keys (32 of 256 channels), brought in by 16-byte asynchronous
// copies. Each warp brings its quarter of a tile's keys, takes their scores S = Q K^T (mma.m16n8k16, a token's heads
// of one group beside each other as the rows) as soon as they are there, and puts its weights P into shared memory;
// after the tile's one barrier each warp adds P V for a quarter of the channels. So no score or sum is computed
// twice, and at the end of a unit nothing but the weights' sums has to be joined. Weights are relative to a maximum
// that all warps hold, renewed only when one of them meets a score that passes it by more than 16 powers of two (12, fp16; the
// barrier says so, and the tile's weights are taken again). Up to 16 rows a weight goes to its product in two parts of the type
// (rounded, and what the rounding left), so that the output's own rounding is all that shows: the outputs are as near the formulas
// as those of fp32 weights, and calls 1 to 9 % slower (token batch 203 us, 201 with one part; one sequence of 16384 tokens 13.1 and
// 12.7; 64 of up to 300 15.6 and 14.5). Units of more rows, whose products count, take it rounded. mma.sync and not tcgen05: with 16
// rows a tile the products are a small part of what even these units do while the keys arrive. They are not with more rows: 8 rows
// of 12 heads over 1 of 256 are 96 a unit, two chunks that each read all keys, through a ring of two stages with queries
// read from shared memory for each tile, and take 24 us over 16384 tokens (floor 2.5), 189 us for 64 sequences of 5000 (49); 8 rows
// of 4 heads a group of 128 channels (32 a unit) 20 us (9.9) and 225 us (195).
//
// Measured: one token of 64 sequences of up to 8191 tokens (8 heads of 128) in 203 us, 6.6 TB/s, 97 % of measured; verifies of 8
// rows over 8 x 16384 tokens (16 heads) in 167 us, 95 %. One sequence is bound by latency: 16384 tokens of 2 heads of 256 in
// 13 to 14.5 us in a graph, of which the merge is 2.5 (floor 5.0). Before: a key group a warp, each with a softmax and all channels of its own,
// 209, 182 and 21 us; the next tile's scores beside the products in the same warp's stream 2 to 4 % slower than now.
#include <algorithm>

#include "paged.cuh"

namespace dfl {
namespace {

constexpr int kWarps = 4, kThreads = 32 * kWarps;
constexpr int kGranule = 64;                    // keys of a granule
constexpr int kStep = 16;                       // a unit's keys begin at a multiple of it: a page at least
// Units of so many bytes at most are taken whole, one CTA each: a cut of many short units costs more (parts to write and to
// add, a second unit to begin in most CTAs) than a last unit that others wait for. One token, 8 heads of 128, sequences
// of up to 400 tokens: 64 of them 18.8 us (24.5 cut), 256 of them 60 us (73); 8 of up to 1000: 18.7 us (12.4 cut).
__host__ __device__ inline long long whole_bytes(long long units) { return min(96ll * 1024 + 2560 * units, 1024ll * 1024); }
constexpr int kMaxCtas = 304;                   // two an SM
// Shared memory of a CTA, two an SM. The granules before each sequence's lie behind it, so above some 1180 sequences (64 channels 1690;
// units of 17 to 32 rows: 95 of 128 channels, 1120 of 64) one CTA fits, and the line's 304 shares go in two turns: 1150 sequences of
// 100 tokens, 8 heads of 128, take 124 ns each, 1200 220 ns; 8 rows of 32 heads over 2000 tokens 1.65 us each for 90, 2.4 for 100.
constexpr int kBudget = 112 * 1024;
constexpr int kMergeThreads = 256;
constexpr int kMostGranules = (1 << 30) - 1;    // of all sequences, 2^36 tokens: what is added up below stays a 32-bit number

struct AttnWork {
    PagedAttnArgs a;
    int chunks;                                 // of query rows
    int *pre;                                   // [n_seq + 1] granules before each sequence's, of one unit each; then the CTAs in use, 0 without cuts
    int4 *first;                                // [CTA] the unit that its share begins in (sequence, unit) and whether inside it
    float *ml, *o;                              // parts: [CTA][2][rows][2], [CTA][2][rows][HD]
    int by_cut;                                 // merge: a CTA a cut, not a unit
    int solo;                                   // the capacity alone says that units are taken whole: a CTA has one
};

// MT tiles of 16 query rows
template <int HD, int MT_>
struct Shape {
    static constexpr int MT = MT_, kKeys = HD == 256 ? 32 : 64;   // keys of a tile
    static constexpr int kMine = kKeys / kWarps;                  // of a warp
    static constexpr int kRows = 16 * MT;
    static constexpr int kParts = MT == 1 ? 2 : 1;                // of a weight: rounded, and what the rounding left
    static constexpr int kQ = kRows * HD * 2, kHalf = kRows * kKeys * 2, kP = kParts * kHalf;
    static constexpr int kTile = kKeys * HD * 2 * 2;
    static constexpr int kStages = (kBudget - kQ - 2 * kP) / kTile;
    static constexpr int kBytes = kQ + 2 * kP + kStages * kTile;
    static_assert(kStages >= 2 && kGranule % kKeys == 0 && kStep % kMine == 0, "");
};

template <typename T>
__device__ __forceinline__ void mma16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    if constexpr (std::is_same<T, __nv_bfloat16>::value)
        mma_bf16(d, a[0], a[1], a[2], a[3], b0, b1);
    else
        asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], unsigned addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t (&r)[4], unsigned addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
template <int N>
__device__ __forceinline__ void cp_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

// What a sequence brings to a call
struct SeqWork {
    int n, row0, len, seen, lo, hi, granules;   // rows, the first of them, tokens before them, keys that some row sees: seen .. hi - 1; lo: seen rounded down to a step
};
__device__ __forceinline__ SeqWork seq_work(const PagedAttnArgs &a, int r0, int r1, int len, int held, int *bits) {
    SeqWork w{0, 0, 0, 0, 0, 0, 0};
    if (r0 < 0 || r1 < r0 || r1 > a.total || len < 0 || r1 - r0 > a.rows) {
        *bits |= kPgArg;
        return w;
    }
    if (r1 == r0) return w;
    const int n = r1 - r0;
    if (held > a.c.max_pages || (long long)len + n > (long long)held * a.c.page) {
        *bits |= kPgState;
        return w;
    }
    w.n = n;
    w.row0 = r0;
    w.len = len;
    w.hi = len + n;
    w.seen = !a.window ? 0 : max(0, a.causal ? len - a.window + 1 : len - a.window);
    w.lo = w.seen / kStep * kStep;
    w.granules = (w.hi - w.lo + kGranule - 1) / kGranule;
    return w;
}

__device__ __forceinline__ SeqWork seq_work(const PagedAttnArgs &a, int s, int *bits) {
    return seq_work(a, a.cu[s], a.cu[s + 1], a.len[s], a.c.held[s], bits);
}

// The first granule of CTA i of n over `all`, and the CTA that has granule x (in 32 bits where they do: the divisions are on the way
// to a call's first loads)
__device__ __forceinline__ long long cut(long long all, int i, int n) {
    return all <= 0xffffffffu / kMaxCtas ? (long long)(unsigned(all) * unsigned(i) / unsigned(n)) : all * i / n;
}
__device__ __forceinline__ int cta_at(long long x, long long all, int n) {
    return all <= 0xffffffffu / kMaxCtas ? int((unsigned(x + 1) * unsigned(n) - 1u) / unsigned(all)) : int(((x + 1) * n - 1) / all);
}

// Outputs. Those of finite values lie between the largest and the smallest value, but where weights are rounded and the sum that divides is not, by
// up to 2^-11 (fp16) further out: at the type's end, where that would be infinite, they are its largest number. (For bf16 the header's limit on
// values is far below it.)
template <typename T>
__device__ __forceinline__ float held(float x) {
    if constexpr (std::is_same<T, __half>::value) x = fabsf(x) < 65600.f ? fminf(fmaxf(x, -65504.f), 65504.f) : x;
    return x;
}
template <typename T>
__device__ __forceinline__ uint32_t pack2_out(float lo, float hi) { return pack2<T>(held<T>(lo), held<T>(hi)); }
template <typename T>
__device__ __forceinline__ void unpack2(uint32_t x, float &lo, float &hi) {
    if constexpr (std::is_same<T, __nv_bfloat16>::value) {
        lo = __uint_as_float(x << 16), hi = __uint_as_float(x & 0xFFFF0000u);
    } else {
        const float2 v = __half22float2(*reinterpret_cast<const __half2 *>(&x));
        lo = v.x, hi = v.y;
    }
}
// The halves of x that are an infinity or a NaN, as masks
template <typename T>
__device__ __forceinline__ uint32_t odd_halves(uint32_t x) {
    const uint32_t e = std::is_same<T, __nv_bfloat16>::value ? 0x7F80u : 0x7C00u;
    return ((x & e) == e ? 0xFFFFu : 0u) | ((x >> 16 & e) == e ? 0xFFFF0000u : 0u);
}

template <typename T, int HD, int MT>
__global__ void __launch_bounds__(kThreads, 2) k_paged_attn(const AttnWork w) {
    using Sh = Shape<HD, MT>;
    constexpr int kStages = Sh::kStages, kRows = Sh::kRows, kKeys = Sh::kKeys, kMine = Sh::kMine;
    constexpr int kCh = HD / 8;                                  // 16-byte pieces of a row
    constexpr int kNt = kMine / 8;                               // tiles of 8 keys of a warp's scores
    constexpr int kN = HD / kWarps / 8;                          // tiles of 8 channels of a warp's sums
    // fp16 weights are held times 2^kShift (what is lost lies 2^-28 below the largest); the maximum in use may fall behind by kBehind powers of two
    constexpr bool kBf16 = std::is_same<T, __nv_bfloat16>::value;
    constexpr float kShift = kBf16 ? 0.f : 3.f, kBehind = kBf16 ? 16.f : 12.f;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ int s_sum[kWarps], s_most[kWarps], s_some[kWarps];
    __shared__ float s_row[kWarps][kRows];                       // maxima, and at the end the weights' sums
    const PagedAttnArgs &a = w.a;
    const dfl_paged &c = a.c;
    uint8_t *qs = smem, *ps = qs + Sh::kQ, *ring = ps + 2 * Sh::kP;
    int *pre = reinterpret_cast<int *>(smem + Sh::kBytes);
    const int t = threadIdx.x, warp = t >> 5, lane = t & 31, g = a.group, S = c.n_seq;
    const unsigned q_at = saddr(qs), p_at = saddr(ps), ring_at = saddr(ring);
    pdl_wait();
    pdl_trigger();

    // ---- granules before each sequence's, of one unit a sequence ----
    const int units = c.n_kv * w.chunks;
    bool whole_units = w.solo;
    long long x = blockIdx.x, end = (long long)S * units;
    if (!w.solo) {
        int bits = 0;
        const int each = (S + kThreads - 1) / kThreads, s0 = min(t * each, S), s1 = min(s0 + each, S);
        int sum = 0, most = 0, some = 0;
        constexpr int kBatch = 4;                                // sequences whose numbers a thread asks for together
        for (int s = t; s < S; s += kBatch * kThreads) {
            int r0[kBatch], r1[kBatch], len[kBatch], held[kBatch];
#pragma unroll
            for (int i = 0; i < kBatch; ++i) {
                const int at = min(s + i * kThreads, S - 1);
                r0[i] = a.cu[at], r1[i] = a.cu[at + 1], len[i] = a.len[at], held[i] = c.held[at];
            }
#pragma unroll
            for (int i = 0; i < kBatch; ++i)
                if (s + i * kThreads < S) {
                    const int n = seq_work(a, r0[i], r1[i], len[i], held[i], &bits).granules;
                    pre[s + i * kThreads + 1] = n;
                    most = max(most, n), some += n != 0;
                }
        }
        __syncthreads();
        for (int s = s0; s < s1; ++s) sum += pre[s + 1];
        int upto = sum;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int u = __shfl_up_sync(0xffffffffu, upto, o);
            if (lane >= o) upto = min(upto + u, kMostGranules);  // (a thread's own are fewer than 2^30)
        }
        most = __reduce_max_sync(0xffffffffu, most), some = __reduce_add_sync(0xffffffffu, some);
        if (lane == 31) s_sum[warp] = upto, s_most[warp] = most, s_some[warp] = some;
        __syncthreads();
        int at = upto - sum;
        for (int i = 0; i < warp; ++i) at = min(at + s_sum[i], kMostGranules);
        for (int s = s0; s < s1; ++s) pre[s + 1] = at += pre[s + 1];
        if (t == 0) pre[0] = 0;
        most = 0, some = 0;
        long long total = 0;
        for (int i = 0; i < kWarps; ++i) most = max(most, s_most[i]), some += s_some[i], total += s_sum[i];
        __syncthreads();
        // a table whose rows name the same pages over and over can hold more than a pool: nothing of the call is done
        const bool far = total >= kMostGranules;
        if (far) bits |= kPgState;
        const long long all = far ? 0 : (long long)pre[S] * units;
        // (of few sequences among many, the line has them side by side)
        whole_units = (long long)most * kGranule * HD * 4 <= whole_bytes((long long)some * units) && 4 * some >= S && !far;
        // 256 channels: as many granules each as the fullest of all CTAs would have, so that fewer of the larger parts are to be added
        // (16384 tokens of 2 heads in 13.1 us, 15.8 with all CTAs). Below, all CTAs (2 heads of 64 in 9.8 us, 10.6; 8 of 128 17.1, 18.5)
        const long long least = HD == 256 ? max((all + gridDim.x - 1) / gridDim.x, 1ll) : 1;
        const int ctas = int(min((long long)gridDim.x, max(1ll, (all + least - 1) / least)));
        if (blockIdx.x == 0) {
            pg_report(c.err, bits);
            for (int s = t; s <= S; s += kThreads) w.pre[s] = pre[s];
            if (t == 0) w.pre[S + 1] = whole_units || far ? 0 : ctas;
        }
        if (!whole_units) {
            if (int(blockIdx.x) >= ctas) return;
            x = cut(all, blockIdx.x, ctas);
            end = cut(all, blockIdx.x + 1, ctas);
        }
    }

    for (int slot = 0; x < end;) {
        // ---- the piece: granules g0 .. g1 - 1 of a unit ----
        int s = 0, u, g0 = 0, g1, bits = 0;
        SeqWork sw;
        if (whole_units) {
            s = int(unsigned(x) / unsigned(units)), u = int(unsigned(x) % unsigned(units));
            sw = seq_work(a, s, &bits);
            g1 = sw.granules;
            if (w.solo && u == 0 && t == 0) pg_report(c.err, bits);
            x += gridDim.x;
        } else {
            for (int hi = S - 1; s < hi;) {                      // the last sequence that begins at or before x, of those with granules
                const int mid = (s + hi) >> 1;
                if ((long long)pre[mid + 1] * units > x) hi = mid;
                else s = mid + 1;
            }
            sw = seq_work(a, s, &bits);
            const long long at = x - (long long)pre[s] * units;
            u = at <= 0xffffffffu ? int(unsigned(at) / unsigned(sw.granules)) : int(at / sw.granules);
            g0 = int(at - (long long)u * sw.granules), g1 = int(min((long long)sw.granules, g0 + (end - x)));
            x += g1 - g0;
        }
        const int h = u / w.chunks, first = u % w.chunks * kRows, live = min(kRows, sw.n * g - first);
        const bool whole = g0 == 0 && g1 == sw.granules;
        if (!whole_units && slot == 0 && t == 0) w.first[blockIdx.x] = make_int4(s, u, g0 > 0, 0);
        const int part = slot;
        slot = 1;                                                // a CTA's first piece, or the one that its cut ends in
        if (live <= 0) continue;
        const int row0 = sw.row0;
        const int base = sw.lo + g0 * kGranule, stop = min(sw.hi, sw.lo + g1 * kGranule);
        const int tiles = (stop - base + kKeys - 1) / kKeys;
        const int32_t *table = c.table + (size_t)s * c.max_pages;

        // the pages of the warp's keys in the next 32 tiles, a tile a lane; asked for 32 tiles ahead
        const auto pages = [&](int i) {
            const int key = base + kKeys * (i + lane) + kMine * warp;
            return key < stop ? table[key >> a.shift] : 0;
        };
        int page_now = pages(0), page_next = pages(32);
        const auto fetch = [&](int i) {                          // the warp's keys of tile i into its stage
            if (i < tiles) {
                if (i && i % 32 == 0) page_now = page_next, page_next = pages(i + 32);
                const int id = __shfl_sync(0xffffffffu, page_now, i % 32), key0 = base + kKeys * i + kMine * warp;
                const bool ok = id >= 0 && id < c.n_pages;
                const size_t from = ((((size_t)(ok ? id : 0) * c.n_kv + h) << a.shift) + (key0 & (c.page - 1))) * HD;
                const unsigned to = ring_at + i % kStages * Sh::kTile + kMine * warp * HD * 2;
#pragma unroll
                for (int y = 0; y < 2 * kMine * kCh / 32; ++y) {
                    const int p = y * 32 + lane, kv = p / (kMine * kCh), key = p / kCh % kMine, ch = p % kCh;
                    const unsigned dst = to + kv * (kKeys * HD * 2) + key * HD * 2 + ((ch ^ (key & 7)) << 4);
                    const T *src = static_cast<const T *>(kv ? c.v : c.k) + from + key * HD + ch * 8;
                    if (ok || kv) cp_async16_or_zeros(dst, src, ok && key0 + key < stop && key0 + key >= sw.seen);
                    else                                         // a page that is none: keys that make NaN of what sees them
                        asm volatile("st.shared.v4.u32 [%0], {%1,%1,%1,%1};" ::"r"(dst), "r"(0x7FFF7FFFu) : "memory");
                }
                if (!ok && key0 < stop && lane == 0) pg_report(c.err, kPgArg);
            }
            asm volatile("cp.async.commit_group;" ::: "memory");
        };
        __syncthreads();                                         // the memory of the piece before is free
        // queries, with the first tile's copies; rows behind the last one are zeros
#pragma unroll
        for (int i = 0; i < kRows * kCh / kThreads; ++i) {
            const int at = i * kThreads + t, r = at / kCh, ch = at % kCh, p = first + min(r, live - 1), token = p * a.inverse >> 12;
            cp_async16_or_zeros(q_at + r * HD * 2 + ((ch ^ (r & 7)) << 4), static_cast<const T *>(a.q) + (int64_t)(row0 + token) * a.ldq + (h * g + p - token * g) * HD + ch * 8, r < live);
        }
#pragma unroll
        for (int i = 0; i < kStages - 1; ++i) fetch(i);
        cp_wait<kStages - 2>();
        __syncthreads();
        const auto q_tile = [&](int mt, int ks) {                // a lane's row address of a 16 x 16 tile of queries
            const int r = mt * 16 + lane % 16, ch = 2 * ks + lane / 16;
            return q_at + r * HD * 2 + ((ch ^ (r & 7)) << 4);
        };
        uint32_t qf[MT == 1 ? HD / 16 : 1][4];
        if constexpr (MT == 1)
#pragma unroll
            for (int ks = 0; ks < HD / 16; ++ks) ldsm4(qf[ks], q_tile(0, ks));
        // what each of the lane's rows sees: keys lo .. hi - 1, counted from base
        int lo[MT][2], hi[MT][2];
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int b = 0; b < 2; ++b) {
                const int p = first + min(mt * 16 + lane / 4 + 8 * b, live - 1), pos = sw.len + (p * a.inverse >> 12);
                hi[mt][b] = (a.causal ? pos + 1 : sw.hi) - base;
                lo[mt][b] = (!a.window ? 0 : max(0, a.causal ? pos - a.window + 1 : sw.len - a.window)) - base;
            }
        const int p0 = sw.len + first / g, p1 = sw.len + (first + live - 1) / g;      // positions of the first and last row
        const int all_hi = (a.causal ? p0 + 1 : sw.hi) - base;                        // keys below it, from all_lo on, are seen by all rows
        const int all_lo = (!a.window ? 0 : max(0, a.causal ? p1 - a.window + 1 : sw.len - a.window)) - base;
        const bool differ = a.causal && sw.n > 1;                // a row may see less than what is loaded

        float o[MT][kN][4], top[MT][2], sum[MT][2];
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
            top[mt][0] = top[mt][1] = -INFINITY;
            sum[mt][0] = sum[mt][1] = 0.f;
#pragma unroll
            for (int i = 0; i < kN; ++i) o[mt][i][0] = o[mt][i][1] = o[mt][i][2] = o[mt][i][3] = 0.f;
        }
        for (int i = 0; i < tiles; ++i) {
            cp_wait<kStages - 2>();
            __syncwarp();
            const unsigned kt = ring_at + i % kStages * Sh::kTile, vt = kt + kKeys * HD * 2;
            const int k0 = kKeys * i, mine = k0 + kMine * warp;  // the tile's first key, the warp's
            // S: rows x the warp's keys. One tile of rows: even and odd steps in sums of their own, so that fewer wait for each other
            constexpr int kChains = MT == 1 ? 2 : 1;
            float sc[MT][kNt][4];
            {
                float part[kChains][MT][kNt][4] = {};
                if constexpr (kNt == 2) {
#pragma unroll
                    for (int ks = 0; ks < HD / 16; ++ks) {
                        uint32_t kf[4];                          // keys 0-7: channels 0-7, 8-15; keys 8-15: the same
                        const int key = kMine * warp + (lane / 16) * 8 + lane % 8, ch = 2 * ks + lane / 8 % 2;
                        ldsm4(kf, kt + key * HD * 2 + ((ch ^ (key & 7)) << 4));
#pragma unroll
                        for (int mt = 0; mt < MT; ++mt) {
                            uint32_t q[4];
                            if constexpr (MT > 1) ldsm4(q, q_tile(mt, ks));
                            mma16<T>(part[ks % kChains][mt][0], MT == 1 ? qf[ks % (HD / 16)] : q, kf[0], kf[1]);
                            mma16<T>(part[ks % kChains][mt][1], MT == 1 ? qf[ks % (HD / 16)] : q, kf[2], kf[3]);
                        }
                    }
                } else {
#pragma unroll
                    for (int ks = 0; ks < HD / 16; ks += 2) {
                        uint32_t kf[4];                          // 8 keys: channels 0-7, 8-15, 16-23, 24-31
                        const int key = kMine * warp + lane % 8, ch = 2 * ks + lane / 8;
                        ldsm4(kf, kt + key * HD * 2 + ((ch ^ (key & 7)) << 4));
#pragma unroll
                        for (int z = 0; z < 2; ++z)
#pragma unroll
                            for (int mt = 0; mt < MT; ++mt) {
                                uint32_t q[4];
                                if constexpr (MT > 1) ldsm4(q, q_tile(mt, ks + z));
                                mma16<T>(part[z % kChains][mt][0], MT == 1 ? qf[(ks + z) % (HD / 16)] : q, kf[2 * z], kf[2 * z + 1]);
                            }
                    }
                }
#pragma unroll
                for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                    for (int b = 0; b < kNt; ++b)
#pragma unroll
                        for (int e = 0; e < 4; ++e) sc[mt][b][e] = kChains == 2 ? part[0][mt][b][e] + part[kChains - 1][mt][b][e] : part[0][mt][b][e];
            }
            const bool masked = k0 < all_lo || k0 + kKeys > all_hi;
            if (masked)
#pragma unroll
                for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                    for (int b = 0; b < kNt; ++b)
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const int key = mine + 8 * b + 2 * (lane % 4) + (e & 1);
                            if (key < lo[mt][e >> 1] || key >= hi[mt][e >> 1]) sc[mt][b][e] = -INFINITY;
                        }
            float most[MT][2], add[MT][2];
            bool renew = false;
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                for (int b = 0; b < 2; ++b) {
                    float m = fmaxf(sc[mt][0][2 * b], sc[mt][0][2 * b + 1]);
                    if constexpr (kNt == 2) m = fmaxf(m, fmaxf(sc[mt][1][2 * b], sc[mt][1][2 * b + 1]));
                    most[mt][b] = m;
                    renew |= (m - top[mt][b]) * a.scale_log2 > kBehind;
                }
            const auto weigh = [&] {                             // the tile's weights into shared memory
#pragma unroll
                for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                    for (int b = 0; b < 2; ++b) {
                        // (the maximum is taken off before the scale: the product of a large one is rounded by many powers of two, and parts have
                        // maxima of their own)
                        const float base = top[mt][b] == -INFINITY ? 0.f : top[mt][b];
                        add[mt][b] = 0.f;
                        const int r = mt * 16 + lane / 4 + 8 * b;
#pragma unroll
                        for (int y = 0; y < kNt; ++y) {
                            const float e0 = exp2_fast(fmaf(sc[mt][y][2 * b] - base, a.scale_log2, kShift)), e1 = exp2_fast(fmaf(sc[mt][y][2 * b + 1] - base, a.scale_log2, kShift));
                            add[mt][b] += e0 + e1;
                            const int ch = warp * kNt + y;
                            uint32_t *to = reinterpret_cast<uint32_t *>(ps + (i & 1) * Sh::kP + r * kKeys * 2 + ((ch ^ (kKeys == 64 ? r & 7 : r >> 1 & 3)) << 4) + 4 * (lane % 4));
                            const uint32_t both = pack2<T>(e0, e1);
                            to[0] = both;
                            if constexpr (Sh::kParts == 2) {
                                float r0, r1;
                                unpack2<T>(both, r0, r1);
                                to[Sh::kHalf / 4] = pack2<T>(e0 - r0, e1 - r1);
                            }
                        }
                    }
            };
            if (i > 0) weigh();                                  // (the first tile has no maximum yet)
            if (i == 0 || __syncthreads_or(renew)) {
#pragma unroll
                for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                    for (int b = 0; b < 2; ++b) {
                        float m = most[mt][b];
                        m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 1));
                        m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 2));
                        if (lane % 4 == 0) s_row[warp][mt * 16 + lane / 4 + 8 * b] = m;
                    }
                __syncthreads();
#pragma unroll
                for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                    for (int b = 0; b < 2; ++b) {
                        const int r = mt * 16 + lane / 4 + 8 * b;
                        const float m = fmaxf(fmaxf(s_row[0][r], s_row[1][r]), fmaxf(s_row[2][r], s_row[3][r]));
                        if (m > top[mt][b]) {
                            const float keep = exp2_fast((top[mt][b] - m) * a.scale_log2);
                            top[mt][b] = m;
                            sum[mt][b] *= keep;
#pragma unroll
                            for (int y = 0; y < kN; ++y) o[mt][y][2 * b] *= keep, o[mt][y][2 * b + 1] *= keep;
                        }
                    }
                weigh();
                __syncthreads();
            }
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) sum[mt][0] += add[mt][0], sum[mt][1] += add[mt][1];
            fetch(i + kStages - 1);                              // where tile i - 1 was: all warps are past its products
            // O += P V. Where a row does not see all keys of the tile, a value that is not finite counts for none in the product,
            // and makes NaN of the sums of the rows that see it
            const bool mixed = masked && differ;
            uint32_t odd = 0;
#pragma unroll
            for (int ks = 0; ks < kKeys / 16; ++ks) {
                uint32_t pf[MT][4], pl[4];
#pragma unroll
                for (int mt = 0; mt < MT; ++mt) {
                    const int r = mt * 16 + lane % 16, ch = 2 * ks + lane / 16;
                    const unsigned at = p_at + (i & 1) * Sh::kP + r * kKeys * 2 + ((ch ^ (kKeys == 64 ? r & 7 : r >> 1 & 3)) << 4);
                    ldsm4(pf[mt], at);
                    if constexpr (Sh::kParts == 2) ldsm4(pl, at + Sh::kHalf);
                }
#pragma unroll
                for (int y = 0; y < kN / 2; ++y) {
                    uint32_t vf[4];                              // channels 0-7: keys 0-7, 8-15; channels 8-15: the same
                    const int key = 16 * ks + lane % 16, ch = warp * kN + 2 * y + lane / 16;
                    ldsm4t(vf, vt + key * HD * 2 + ((ch ^ (key & 7)) << 4));
                    if (mixed)
#pragma unroll
                        for (int z = 0; z < 4; ++z) {
                            const uint32_t m = odd_halves<T>(vf[z]);
                            odd |= m;
                            vf[z] &= ~m;
                        }
#pragma unroll
                    for (int mt = 0; mt < MT; ++mt) {
                        mma16<T>(o[mt][2 * y], pf[mt], vf[0], vf[1]);
                        mma16<T>(o[mt][2 * y + 1], pf[mt], vf[2], vf[3]);
                    }
                    if constexpr (Sh::kParts == 2) {
                        mma16<T>(o[0][2 * y], pl, vf[0], vf[1]);
                        mma16<T>(o[0][2 * y + 1], pl, vf[2], vf[3]);
                    }
                }
            }
            if (mixed && __any_sync(0xffffffffu, odd)) {
                const uint16_t *v = reinterpret_cast<const uint16_t *>(ring + i % kStages * Sh::kTile + kKeys * HD * 2);
                for (int key = 0; key < kKeys; ++key)
#pragma unroll
                    for (int y = 0; y < kN; ++y)
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            const int ch = warp * kN + y, x16 = 2 * (lane % 4) + e;
                            if (odd_halves<T>(v[key * HD + ((ch ^ (key & 7)) << 3) + x16]) & 0xFFFFu)
#pragma unroll
                                for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                                    for (int b = 0; b < 2; ++b)
                                        if (k0 + key >= lo[mt][b] && k0 + key < hi[mt][b]) o[mt][y][2 * b + e] = NAN;
                        }
            }
        }
        cp_wait<0>();
        // ---- the weights' sums joined; out, or into the parts ----
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int b = 0; b < 2; ++b) {
                sum[mt][b] += __shfl_xor_sync(0xffffffffu, sum[mt][b], 1);
                sum[mt][b] += __shfl_xor_sync(0xffffffffu, sum[mt][b], 2);
                if (lane % 4 == 0) s_row[warp][mt * 16 + lane / 4 + 8 * b] = sum[mt][b];
            }
        __syncthreads();
        const size_t slot_at = (size_t)blockIdx.x * 2 + part;
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int b = 0; b < 2; ++b) {
                const int r = mt * 16 + lane / 4 + 8 * b;
                if (r >= live) continue;
                const float l = (s_row[0][r] + s_row[1][r]) + (s_row[2][r] + s_row[3][r]);
                if (whole) {
                    const float d = 1.f / l;
                    const int p = first + r, token = p * a.inverse >> 12;
                    T *to = static_cast<T *>(a.out) + (int64_t)(row0 + token) * a.ldo + (h * g + p - token * g) * HD + warp * kN * 8 + 2 * (lane % 4);
#pragma unroll
                    for (int y = 0; y < kN; ++y) *reinterpret_cast<uint32_t *>(to + 8 * y) = pack2_out<T>(o[mt][y][2 * b] * d, o[mt][y][2 * b + 1] * d);
                } else {
                    float *to = w.o + (slot_at * kRows + r) * HD + warp * kN * 8 + 2 * (lane % 4);
#pragma unroll
                    for (int y = 0; y < kN; ++y) *reinterpret_cast<float2 *>(to + 8 * y) = make_float2(o[mt][y][2 * b], o[mt][y][2 * b + 1]);
                    if (warp == 0 && lane % 4 == 0) *reinterpret_cast<float2 *>(w.ml + (slot_at * kRows + r) * 2) = make_float2(top[mt][b], l);
                }
            }
    }
}

// The parts of units that cuts went through, added in the order of their CTAs. A half warp takes 64 channels of a row, 16 bytes a
// lane; SHARE half warps share them where rows are few and parts many, each every SHARE-th part.
template <typename T, int HD, int SHARE>
__global__ void __launch_bounds__(kMergeThreads) k_paged_merge(const AttnWork w, int kRows) {
    constexpr int kHalves = kMergeThreads / 16, kSlices = HD / 64;
    __shared__ float s_o[SHARE > 1 ? kHalves : 1][64], s_ml[SHARE > 1 ? kHalves : 1][2];
    const PagedAttnArgs &a = w.a;
    const dfl_paged &c = a.c;
    const int half = threadIdx.x >> 4, lane = threadIdx.x & 15, g = a.group, units = c.n_kv * w.chunks;
    pdl_wait();
    const int total = w.pre[c.n_seq], ctas = w.pre[c.n_seq + 1];
    int u = blockIdx.y, s = blockIdx.z;
    if (w.by_cut) {                                              // the unit that the share of CTA blockIdx.y + 1 begins inside of
        if (int(blockIdx.y) + 1 >= ctas) return;
        const int4 at = w.first[blockIdx.y + 1];
        if (!at.z) return;
        s = at.x, u = at.y;
    }
    const int h = u / w.chunks, first = u % w.chunks * kRows;
    const int id = blockIdx.x * (kHalves / SHARE) + half / SHARE, r = id / kSlices, ch = id % kSlices * 64 + 4 * lane;
    const int begin = w.pre[s], granules = w.pre[s + 1] - begin;
    const int row0 = a.cu[s], live = min(kRows, (a.cu[s + 1] - row0) * g - first);
    if (!granules || !ctas) return;
    const long long all = (long long)total * units, from = (long long)begin * units + (long long)u * granules;
    const int c0 = cta_at(from, all, ctas), parts = cta_at(from + granules - 1, all, ctas) - c0 + 1;
    if (parts == 1 || (w.by_cut && c0 != int(blockIdx.y))) return;                // (of a unit's cuts, the first one's CTA adds)
    const bool mine = r < live;
    const int head = cut(all, c0, ctas) < from;                  // the first part is its CTA's second piece
    float m = -INFINITY, l = 0.f, v[4] = {0.f, 0.f, 0.f, 0.f};
    constexpr int kBatch = 4;
    for (int p0 = half % SHARE; mine && p0 < parts; p0 += SHARE * kBatch) {
        float2 ml[kBatch];
        float4 o[kBatch];
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            const int p = min(p0 + i * SHARE, parts - 1);
            const size_t at = ((size_t)(c0 + p) * 2 + (p == 0 ? head : 0)) * kRows + r;
            ml[i] = *reinterpret_cast<const float2 *>(w.ml + at * 2);
            o[i] = *reinterpret_cast<const float4 *>(w.o + at * HD + ch);
            if (p0 + i * SHARE >= parts) ml[i] = make_float2(-INFINITY, 0.f), o[i] = make_float4(0.f, 0.f, 0.f, 0.f);
        }
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            const float next = fmaxf(m, ml[i].x), keep = m == next ? 1.f : exp2_fast((m - next) * a.scale_log2);
            const float f = ml[i].x == next ? 1.f : exp2_fast((ml[i].x - next) * a.scale_log2);
            m = next;
            l = l * keep + ml[i].y * f;
            v[0] = v[0] * keep + o[i].x * f, v[1] = v[1] * keep + o[i].y * f, v[2] = v[2] * keep + o[i].z * f, v[3] = v[3] * keep + o[i].w * f;
        }
    }
    if constexpr (SHARE > 1) {
        *reinterpret_cast<float4 *>(&s_o[half][4 * lane]) = make_float4(v[0], v[1], v[2], v[3]);
        if (lane == 0) s_ml[half][0] = m, s_ml[half][1] = l;
        __syncthreads();
        if (half % SHARE) return;
        m = -INFINITY, l = 0.f, v[0] = v[1] = v[2] = v[3] = 0.f;
#pragma unroll
        for (int i = 0; i < SHARE; ++i) m = fmaxf(m, s_ml[half + i][0]);
#pragma unroll
        for (int i = 0; i < SHARE; ++i) {
            const float f = s_ml[half + i][0] == m ? 1.f : exp2_fast((s_ml[half + i][0] - m) * a.scale_log2);
            const float4 o = *reinterpret_cast<const float4 *>(&s_o[half + i][4 * lane]);
            l = fmaf(s_ml[half + i][1], f, l);
            v[0] = fmaf(o.x, f, v[0]), v[1] = fmaf(o.y, f, v[1]), v[2] = fmaf(o.z, f, v[2]), v[3] = fmaf(o.w, f, v[3]);
        }
    }
    if (!mine) return;
    const float d = 1.f / l;
    const int p = first + r;
    *reinterpret_cast<uint2 *>(static_cast<T *>(a.out) + (int64_t)(row0 + p / g) * a.ldo + (h * g + p % g) * HD + ch) =
        make_uint2(pack2_out<T>(v[0] * d, v[1] * d), pack2_out<T>(v[2] * d, v[3] * d));
}

// Rows of a chunk: the fewest of 16, 32 and 64 that hold all, or the most
int chunk_rows(int rows) { return rows <= 16 ? 16 : rows <= 32 ? 32 : 64; }

struct Scratch {
    size_t pre, first, ml, o, total;
};
Scratch scratch_of(const dfl_paged *c, int n_q, int rows) {
    const size_t r = (size_t)kMaxCtas * 2 * chunk_rows(rows * (n_q / c->n_kv));
    Scratch s;
    s.pre = ((size_t)(c->n_seq + 2) * 4 + 255) / 256 * 256;
    s.first = (size_t)kMaxCtas * sizeof(int4);
    s.ml = r * 2 * 4;
    s.o = r * c->head_dim * 4;
    s.total = s.pre + s.first + s.ml + s.o;
    return s;
}

template <typename T, int HD, int MT>
int launch_shape(const AttnWork &w, cudaStream_t st) {
    using Sh = Shape<HD, MT>;
    const int dev = current_device();
    if (dev < 0) return DFL_E_CUDA;
    static int sms[kMaxDevices] = {};
    if (!sms[dev]) {
        int n = 0;
        if (cudaFuncSetAttribute(k_paged_attn<T, HD, MT>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 Sh::kBytes + (DFL_PAGED_MAX_SEQ + 1) * 4) != cudaSuccess ||
            cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
            return DFL_E_CUDA;
        sms[dev] = n;
    }
    const dfl_paged &c = w.a.c;
    const int64_t granules = ((int64_t)c.max_pages * c.page + kGranule - 1) / kGranule + 1;   // of a unit at most
    const int units = c.n_kv * w.chunks, rows = std::min(Sh::kRows, w.a.rows * w.a.group) * (HD / 64);
    AttnWork m = w;
    // (more CTAs than that are not launched for units of which many may be without rows)
    m.solo = granules * kGranule * HD * 4 <= whole_bytes((long long)c.n_seq * units) && (int64_t)c.n_seq * units <= 8 * kMaxCtas;
    const int64_t ctas = m.solo ? (int64_t)c.n_seq * units : std::min<int64_t>(std::min(2 * sms[dev], kMaxCtas), c.n_seq * units * granules);
    const cudaError_t e = launch_pdl(k_paged_attn<T, HD, MT>, dim3(unsigned(ctas)), dim3(kThreads), Sh::kBytes + (m.solo ? 0 : (c.n_seq + 1) * 4), st, m);
    if (e != cudaSuccess || m.solo) return pg_launched(e);
    // A CTA a unit, or where these are more than the cuts, a cut; half warps share a row's parts: 16 where rows are few in all, 4 of
    // cuts, as one sequence among many may have most of them
    constexpr int kHalves = kMergeThreads / 16, kFew = 4;
    if ((int64_t)c.n_seq * units * rows < 8 * sms[dev])
        return pg_launched(launch_pdl(k_paged_merge<T, HD, kHalves>, dim3(rows, units, c.n_seq), dim3(kMergeThreads), 0, st, m, int(Sh::kRows)));
    m.by_cut = (int64_t)c.n_seq * units >= ctas;
    if (m.by_cut)
        return pg_launched(launch_pdl(k_paged_merge<T, HD, kFew>, dim3((rows * kFew + kHalves - 1) / kHalves, unsigned(std::max<int64_t>(ctas - 1, 1))),
                                      dim3(kMergeThreads), 0, st, m, int(Sh::kRows)));
    return pg_launched(launch_pdl(k_paged_merge<T, HD, 1>, dim3((rows + kHalves - 1) / kHalves, units, c.n_seq), dim3(kMergeThreads), 0, st, m, int(Sh::kRows)));
}

template <typename T, int HD>
int launch_rows(const AttnWork &w, int rows, cudaStream_t st) {
    return rows == 16 ? launch_shape<T, HD, 1>(w, st) : rows == 32 ? launch_shape<T, HD, 2>(w, st) : launch_shape<T, HD, 4>(w, st);
}

template <typename T>
int launch_type(const AttnWork &w, int rows, cudaStream_t st) {
    const int hd = w.a.c.head_dim;
    return hd == 64 ? launch_rows<T, 64>(w, rows, st) : hd == 128 ? launch_rows<T, 128>(w, rows, st) : launch_rows<T, 256>(w, rows, st);
}

}  // namespace

size_t paged_attn_scratch(const dfl_paged *c, int n_q, int rows) { return scratch_of(c, n_q, rows).total; }

int launch_paged_attn(const PagedAttnArgs &a, void *scratch, cudaStream_t st) {
    const Scratch s = scratch_of(&a.c, a.n_q, a.rows);
    const int rows = chunk_rows(a.rows * a.group);
    uint8_t *at = static_cast<uint8_t *>(scratch);
    const AttnWork w{a, (a.rows * a.group + rows - 1) / rows, reinterpret_cast<int *>(at), reinterpret_cast<int4 *>(at + s.pre),
                     reinterpret_cast<float *>(at + s.pre + s.first), reinterpret_cast<float *>(at + s.pre + s.first + s.ml), 0, 0};
    return a.c.type == DFL_BF16 ? launch_type<__nv_bfloat16>(w, rows, st) : launch_type<__half>(w, rows, st);
}

}  // namespace dfl
