// pagedattn.cu -- attention of one token, or of a verify's rows, over the paged cache (include/dfl.h, dfl_paged_attn).
//
// The call reads every visible key and value once, so it is bound by HBM as long as few rows share them. The keys
// of all units (a sequence, a key/value head, a chunk of query rows) lie one after another on a line of granules of
// 64, which is cut evenly among the CTAs: the lengths of a batch, which the host does not know, decide nothing but
// where the cuts fall. A unit that a cut goes through leaves a part (sums, maximum, weight) for each CTA, and a
// second launch adds the parts in their order.
//
// A CTA is four warps. A step is 16 keys, which lie in one page: the warps of a key group bring its keys and values
// into a ring of their own (16-byte asynchronous copies, no other warp waits), the scores S = Q K^T and sums P V go
// through mma.m16n8k16 with 16 query rows (a token's heads of one group beside each other) as the rows, and the
// group keeps a softmax of its own over its steps; groups are joined when the CTA is done with the unit. mma.sync
// and not tcgen05: with 16 rows a tile the products are a fifth of what even these units can do while the keys
// arrive, and each warp goes at its own pace.
#include <algorithm>

#include "paged.cuh"

namespace dfl {
namespace {

constexpr int kWarps = 4, kThreads = 32 * kWarps;
constexpr int kGranule = 64;                    // keys of a granule
constexpr int kStep = 16;                       // keys of a step
constexpr int kLeast = 4;                       // granules of a CTA at least
constexpr int kMaxCtas = 304;                   // two an SM
constexpr int kBudget = 108 * 1024;             // shared memory of a CTA's queries and rings
constexpr int kMergeThreads = 256;

struct AttnWork {
    PagedAttnArgs a;
    int chunks;                                 // of query rows
    int *pre;                                   // [n_seq + 1] granules before each sequence's, of one unit each; then the CTAs in use
    float *ml, *o;                              // parts: [CTA][2][rows][2], [CTA][2][rows][HD]
    int ways;                                   // merge: warps that share a row
};

// MT tiles of 16 rows a warp, MW warps beside each other along the rows, CW along the channels of the values
template <int HD, int MT_, int MW_>
struct Shape {
    static constexpr int MT = MT_, MW = MW_, CW = HD == 256 ? 2 : 1;
    static constexpr int GW = MW * CW, KW = kWarps / GW;      // warps of a key group, key groups
    static constexpr int kRows = 16 * MT * MW;
    static constexpr int kQ = kRows * HD * 2;
    static constexpr int kStage = kStep * HD * 2 * 2;
    static constexpr int kStages = (kBudget - kQ) / (KW * kStage);
    static constexpr int kRing = KW * kStages * kStage;
    static_assert(KW >= 1 && kStages >= 2 && KW * kRows * HD * 4 <= kRing, "");
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
// 16 bytes into shared memory, or zeros
__device__ __forceinline__ void cp16(unsigned dst, const void *src, bool there) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(there ? 16 : 0) : "memory");
}
template <int N>
__device__ __forceinline__ void cp_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

__device__ __forceinline__ float exp2_fast(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// What a sequence brings to a call
struct SeqWork {
    int n, len, seen, lo, hi, granules;         // rows, tokens before them, keys that some row sees: seen .. hi - 1; lo: seen rounded down to a step
};
__device__ SeqWork seq_work(const PagedAttnArgs &a, int s, int *bits) {
    SeqWork w{0, 0, 0, 0, 0, 0};
    const int r0 = a.cu[s], r1 = a.cu[s + 1], len = a.len[s], held = a.c.held[s];
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
    w.len = len;
    w.hi = len + n;
    w.seen = !a.window ? 0 : max(0, a.causal ? len - a.window + 1 : len - a.window);
    w.lo = w.seen / kStep * kStep;
    w.granules = (w.hi - w.lo + kGranule - 1) / kGranule;
    return w;
}

// The first granule of CTA i of n over `all`, and the CTA that has granule x
__device__ __forceinline__ long long cut(long long all, int i, int n) { return all * i / n; }
__device__ __forceinline__ int cta_at(long long x, long long all, int n) { return int(((x + 1) * n - 1) / all); }

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
// The halves of x that are an infinity or a NaN, as masks
template <typename T>
__device__ __forceinline__ uint32_t odd_halves(uint32_t x) {
    const uint32_t e = std::is_same<T, __nv_bfloat16>::value ? 0x7F80u : 0x7C00u;
    return ((x & e) == e ? 0xFFFFu : 0u) | ((x >> 16 & e) == e ? 0xFFFF0000u : 0u);
}

template <typename T, int HD, int MT, int MW>
__global__ void __launch_bounds__(kThreads, 2) k_paged_attn(const AttnWork w) {
    using Sh = Shape<HD, MT, MW>;
    constexpr int KW = Sh::KW, GW = Sh::GW, CW = Sh::CW, kStages = Sh::kStages, kRows = Sh::kRows;
    constexpr int kCh = HD / 8;                                  // 16-byte pieces of a row
    constexpr int kN = HD / CW / 8;                              // tiles of 8 channels of a warp's sums
    constexpr float kShift = std::is_same<T, __nv_bfloat16>::value ? 0.f : 10.f;   // fp16 weights are held times 2^10: lost below 2^-35
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ int s_sum[kWarps];
    __shared__ float s_ml[KW][kRows][2];
    const PagedAttnArgs &a = w.a;
    const dfl_paged &c = a.c;
    uint8_t *qs = smem, *ring0 = smem + Sh::kQ;
    int *pre = reinterpret_cast<int *>(smem + Sh::kQ + Sh::kRing);
    const int t = threadIdx.x, warp = t >> 5, lane = t & 31, g = a.group, S = c.n_seq;
    const int kg = warp / GW, mw = warp % GW / CW, cw = warp % CW;
    pdl_wait();

    // ---- granules before each sequence's, of one unit a sequence ----
    int bits = 0;
    {
        int *mine = pre;
        const int each = (S + kThreads - 1) / kThreads, s0 = min(t * each, S), s1 = min(s0 + each, S);
        int sum = 0;
        for (int s = s0; s < s1; ++s) {
            const int n = seq_work(a, s, &bits).granules;
            mine[s + 1] = n;
            sum += n;
        }
        int upto = sum;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int u = __shfl_up_sync(0xffffffffu, upto, o);
            if (lane >= o) upto += u;
        }
        if (lane == 31) s_sum[warp] = upto;
        __syncthreads();
        int at = upto - sum;
        for (int i = 0; i < warp; ++i) at += s_sum[i];
        for (int s = s0; s < s1; ++s) mine[s + 1] = at += mine[s + 1];
        if (t == 0) mine[0] = 0;
        __syncthreads();
    }
    const int units = c.n_kv * w.chunks;
    const long long all = (long long)pre[S] * units;
    const int ctas = int(min((long long)gridDim.x, max(1ll, (all + kLeast - 1) / kLeast)));
    if (blockIdx.x == 0) {
        pg_report(c.err, bits);
        for (int s = t; s <= S; s += kThreads) w.pre[s] = pre[s];
        if (t == 0) w.pre[S + 1] = ctas;
    }
    if (int(blockIdx.x) >= ctas) return;
    long long x = cut(all, blockIdx.x, ctas);
    const long long end = cut(all, blockIdx.x + 1, ctas);

    for (int slot = 0; x < end;) {
        // ---- the piece: granules g0 .. g1 - 1 of a unit ----
        int s = 0;
        for (int hi = S - 1; s < hi;) {                          // the last sequence that begins at or before x, of those with granules
            const int mid = (s + hi) >> 1;
            if ((long long)pre[mid + 1] * units > x) hi = mid;
            else s = mid + 1;
        }
        int none = 0;
        const SeqWork sw = seq_work(a, s, &none);
        const long long at = x - (long long)pre[s] * units;
        const int u = int(at / sw.granules), g0 = int(at % sw.granules), g1 = int(min((long long)sw.granules, g0 + (end - x)));
        const int h = u / w.chunks, first = u % w.chunks * kRows, live = min(kRows, sw.n * g - first);
        x += g1 - g0;
        const bool whole = g0 == 0 && g1 == sw.granules;
        const int part = slot;
        slot = 1;                                                // a CTA's first piece, or the one that its cut ends in
        if (live <= 0) continue;
        const int row0 = a.cu[s];
        const int base = sw.lo + g0 * kGranule, stop = min(sw.hi, sw.lo + g1 * kGranule);
        const int steps = (stop - base + kStep - 1) / kStep, mine = (steps - kg + KW - 1) / KW;
        const int32_t *table = c.table + (size_t)s * c.max_pages;
        uint8_t *ring = ring0 + kg * kStages * Sh::kStage;
        const unsigned ring_at = saddr(ring);

        // the pages of the group's next 32 steps, a step a lane; asked for 32 steps ahead
        const auto pages = [&](int i) {
            const int key = base + kStep * (kg + KW * (i + lane));
            return key < stop ? table[key / c.page] : 0;
        };
        int page_now = pages(0), page_next = pages(32);
        const auto fetch = [&](int i) {                          // step i of the group into its stage
            if (i < mine) {
                if (i && i % 32 == 0) page_now = page_next, page_next = pages(i + 32);
                const int id = __shfl_sync(0xffffffffu, page_now, i % 32), key0 = base + kStep * (kg + KW * i);
                const bool ok = id >= 0 && id < c.n_pages;
                const size_t from = (((size_t)(ok ? id : 0) * c.n_kv + h) * c.page + key0 % c.page) * HD;
                const unsigned to = ring_at + i % kStages * Sh::kStage;
#pragma unroll
                for (int y = 0; y < 2 * kStep * kCh / 32 / GW; ++y) {
                    const int p = (y * GW + warp % GW) * 32 + lane, kv = p / (kStep * kCh), key = p / kCh % kStep, ch = p % kCh;
                    const unsigned dst = to + kv * (kStep * HD * 2) + key * HD * 2 + ((ch ^ (key & 7)) << 4);
                    const T *src = static_cast<const T *>(kv ? c.v : c.k) + from + key * HD + ch * 8;
                    if (ok || kv) cp16(dst, src, ok && key0 + key < stop && key0 + key >= sw.seen);
                    else                                         // a page that is none: keys that make NaN of what sees them
                        asm volatile("st.shared.v4.u32 [%0], {%1,%1,%1,%1};" ::"r"(dst), "r"(0x7FFF7FFFu) : "memory");
                }
                if (!ok && lane == 0) pg_report(c.err, kPgArg);
            }
            asm volatile("cp.async.commit_group;" ::: "memory");
        };
        const auto group_sync = [&] {
            if constexpr (GW == 1) __syncwarp();
            else asm volatile("bar.sync %0, %1;" ::"r"(1 + kg), "n"(32 * GW) : "memory");
        };
        __syncthreads();                                         // the memory of the piece before is free
#pragma unroll
        for (int i = 0; i < kStages - 1; ++i) fetch(i);
        // queries: rows behind the last one are zeros
        for (int i = t; i < kRows * kCh; i += kThreads) {
            const int r = i / kCh, ch = i % kCh, p = first + r;
            uint4 v = make_uint4(0, 0, 0, 0);
            if (r < live) v = *reinterpret_cast<const uint4 *>(static_cast<const T *>(a.q) + (int64_t)(row0 + p / g) * a.ldq + (h * g + p % g) * HD + ch * 8);
            *reinterpret_cast<uint4 *>(qs + r * HD * 2 + ((ch ^ (r & 7)) << 4)) = v;
        }
        __syncthreads();
        const auto q_at = [&](int mt, int ks) {                  // a lane's row address of a 16 x 16 tile of queries
            const int r = (mw * MT + mt) * 16 + lane % 16, ch = 2 * ks + lane / 16;
            return saddr(qs) + r * HD * 2 + ((ch ^ (r & 7)) << 4);
        };
        uint32_t qf[MT == 1 ? HD / 16 : 1][4];
        if constexpr (MT == 1)
#pragma unroll
            for (int ks = 0; ks < HD / 16; ++ks) ldsm4(qf[ks], q_at(0, ks));
        // what each of the lane's rows sees: keys lo .. hi - 1, counted from base
        int lo[MT][2], hi[MT][2];
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int b = 0; b < 2; ++b) {
                const int p = first + min((mw * MT + mt) * 16 + lane / 4 + 8 * b, live - 1), pos = sw.len + p / g;
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
        for (int i = 0; i < mine; ++i) {
            cp_wait<kStages - 2>();
            group_sync();
            fetch(i + kStages - 1);
            const unsigned kt = ring_at + i % kStages * Sh::kStage, vt = kt + kStep * HD * 2;
            const int k0 = kStep * (kg + KW * i);
            // S: rows x 16 keys
            float sc[MT][2][4];
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                for (int b = 0; b < 2; ++b) sc[mt][b][0] = sc[mt][b][1] = sc[mt][b][2] = sc[mt][b][3] = 0.f;
#pragma unroll
            for (int ks = 0; ks < HD / 16; ++ks) {
                uint32_t kf[4];                                  // keys 0-7: channels 0-7, 8-15; keys 8-15: the same
                const int key = (lane / 16) * 8 + lane % 8, ch = 2 * ks + lane / 8 % 2;
                ldsm4(kf, kt + key * HD * 2 + ((ch ^ (key & 7)) << 4));
#pragma unroll
                for (int mt = 0; mt < MT; ++mt) {
                    if constexpr (MT == 1) {
                        mma16<T>(sc[0][0], qf[ks], kf[0], kf[1]);
                        mma16<T>(sc[0][1], qf[ks], kf[2], kf[3]);
                    } else {
                        uint32_t q[4];
                        ldsm4(q, q_at(mt, ks));
                        mma16<T>(sc[mt][0], q, kf[0], kf[1]);
                        mma16<T>(sc[mt][1], q, kf[2], kf[3]);
                    }
                }
            }
            const bool masked = k0 < all_lo || k0 + kStep > all_hi;
            if (masked)
#pragma unroll
                for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                    for (int b = 0; b < 2; ++b)
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const int key = k0 + 8 * b + 2 * (lane % 4) + (e & 1);
                            if (key < lo[mt][e >> 1] || key >= hi[mt][e >> 1]) sc[mt][b][e] = -INFINITY;
                        }
            uint32_t pf[MT][4];
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) {
                float next[2];
#pragma unroll
                for (int b = 0; b < 2; ++b) {
                    float m = fmaxf(fmaxf(sc[mt][0][2 * b], sc[mt][0][2 * b + 1]), fmaxf(sc[mt][1][2 * b], sc[mt][1][2 * b + 1]));
                    m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 1));
                    m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 2));
                    next[b] = fmaxf(m, top[mt][b]);
                }
                if (__any_sync(0xffffffffu, next[0] > top[mt][0] || next[1] > top[mt][1])) {
#pragma unroll
                    for (int b = 0; b < 2; ++b) {
                        const float keep = next[b] > top[mt][b] ? exp2_fast((top[mt][b] - next[b]) * a.scale_log2) : 1.f;
                        top[mt][b] = next[b];
                        sum[mt][b] *= keep;
#pragma unroll
                        for (int y = 0; y < kN; ++y) o[mt][y][2 * b] *= keep, o[mt][y][2 * b + 1] *= keep;
                    }
                }
#pragma unroll
                for (int b = 0; b < 2; ++b) {
                    const float off = top[mt][b] == -INFINITY ? 0.f : kShift - top[mt][b] * a.scale_log2;
#pragma unroll
                    for (int y = 0; y < 2; ++y) {
                        const float e0 = exp2_fast(fmaf(sc[mt][y][2 * b], a.scale_log2, off)), e1 = exp2_fast(fmaf(sc[mt][y][2 * b + 1], a.scale_log2, off));
                        sum[mt][b] += e0 + e1;
                        pf[mt][2 * y + b] = pack2<T>(e0, e1);
                    }
                }
            }
            // O += P V. Where a row does not see all keys of the step, a value that is not finite counts for none in the product,
            // and makes NaN of the sums of the rows that see it
            const bool mixed = masked && differ;
            uint32_t odd = 0;
#pragma unroll
            for (int y = 0; y < kN / 2; ++y) {
                uint32_t vf[4];                                  // channels 0-7: keys 0-7, 8-15; channels 8-15: the same
                const int key = lane % 16, ch = cw * kN + 2 * y + lane / 16;
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
            }
            if (mixed && __any_sync(0xffffffffu, odd)) {
                const uint16_t *v = reinterpret_cast<const uint16_t *>(ring + i % kStages * Sh::kStage + kStep * HD * 2);
                for (int key = 0; key < kStep; ++key)
#pragma unroll
                    for (int y = 0; y < kN; ++y)
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            const int ch = cw * kN + y, x16 = 2 * (lane % 4) + e;
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
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int b = 0; b < 2; ++b) {
                sum[mt][b] += __shfl_xor_sync(0xffffffffu, sum[mt][b], 1);
                sum[mt][b] += __shfl_xor_sync(0xffffffffu, sum[mt][b], 2);
            }
        // ---- the groups' sums through shared memory, then out or into the parts ----
        __syncthreads();
        float *all_o = reinterpret_cast<float *>(ring0);         // [group][row][HD], 8 channels of a row turned by its number
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int b = 0; b < 2; ++b) {
                const int r = (mw * MT + mt) * 16 + lane / 4 + 8 * b;
                if (r >= live) continue;
                float *to = all_o + ((size_t)kg * kRows + r) * HD;
#pragma unroll
                for (int y = 0; y < kN; ++y)
                    *reinterpret_cast<float2 *>(to + (((cw * kN + y) ^ (r & 3)) << 3) + 2 * (lane % 4)) = make_float2(o[mt][y][2 * b], o[mt][y][2 * b + 1]);
                if (cw == 0 && lane % 4 == 0) s_ml[kg][r][0] = top[mt][b], s_ml[kg][r][1] = sum[mt][b];
            }
        __syncthreads();
        float *part_o = w.o + ((size_t)blockIdx.x * 2 + part) * kRows * HD, *part_ml = w.ml + ((size_t)blockIdx.x * 2 + part) * kRows * 2;
        for (int i = t; i < live * kCh; i += kThreads) {
            const int r = i / kCh, ch = i % kCh;
            float m = -INFINITY, l = 0.f, v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int k = 0; k < KW; ++k) m = fmaxf(m, s_ml[k][r][0]);
#pragma unroll
            for (int k = 0; k < KW; ++k) {
                const float mk = s_ml[k][r][0], f = mk == m ? 1.f : exp2_fast((mk - m) * a.scale_log2);
                l = fmaf(s_ml[k][r][1], f, l);
                const float4 *from = reinterpret_cast<const float4 *>(all_o + ((size_t)k * kRows + r) * HD + ((ch ^ (r & 3)) << 3));
                const float4 p = from[0], q = from[1];
                v[0] = fmaf(p.x, f, v[0]), v[1] = fmaf(p.y, f, v[1]), v[2] = fmaf(p.z, f, v[2]), v[3] = fmaf(p.w, f, v[3]);
                v[4] = fmaf(q.x, f, v[4]), v[5] = fmaf(q.y, f, v[5]), v[6] = fmaf(q.z, f, v[6]), v[7] = fmaf(q.w, f, v[7]);
            }
            if (whole) {
                const float d = 1.f / l;
                const int p = first + r;
                T *to = static_cast<T *>(a.out) + (int64_t)(row0 + p / g) * a.ldo + (h * g + p % g) * HD + ch * 8;
                *reinterpret_cast<uint4 *>(to) = make_uint4(pack2<T>(v[0] * d, v[1] * d), pack2<T>(v[2] * d, v[3] * d), pack2<T>(v[4] * d, v[5] * d),
                                                            pack2<T>(v[6] * d, v[7] * d));
            } else {
                float4 *to = reinterpret_cast<float4 *>(part_o + (size_t)r * HD + ch * 8);
                to[0] = make_float4(v[0], v[1], v[2], v[3]);
                to[1] = make_float4(v[4], v[5], v[6], v[7]);
                if (ch == 0) part_ml[2 * r] = m, part_ml[2 * r + 1] = l;
            }
        }
    }
}

// The parts of units that cuts went through, added in the order of their CTAs. `ways` warps share a row.
template <typename T, int HD>
__global__ void __launch_bounds__(kMergeThreads) k_paged_merge(const AttnWork w, int kRows) {
    constexpr int kW = kMergeThreads / 32, kV = HD / 32;         // a lane's channels
    __shared__ float s_o[kW][HD];
    const PagedAttnArgs &a = w.a;
    const dfl_paged &c = a.c;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = a.group, units = c.n_kv * w.chunks;
    const int u = blockIdx.y, s = blockIdx.z, h = u / w.chunks, first = u % w.chunks * kRows;
    pdl_wait();
    const int begin = w.pre[s], granules = w.pre[s + 1] - begin;
    if (!granules) return;
    const int ctas = w.pre[c.n_seq + 1], row0 = a.cu[s], live = min(kRows, (a.cu[s + 1] - row0) * g - first);
    const long long all = (long long)w.pre[c.n_seq] * units, from = (long long)begin * units + (long long)u * granules;
    const int c0 = cta_at(from, all, ctas), c1 = cta_at(from + granules - 1, all, ctas), parts = c1 - c0 + 1;
    if (parts == 1) return;
    const int head = cut(all, c0, ctas) < from;                  // the first part is its CTA's second piece
    const int share = w.ways, way = warp % share;
    for (int r = blockIdx.x * (kW / share) + warp / share; r - warp / share < live; r += gridDim.x * (kW / share)) {
        const bool mine = r < live;
        const auto slot = [&](int p) { return (size_t)(c0 + p) * 2 + (p == 0 ? head : 0); };
        float m = -INFINITY, l = 0.f, v[kV];
#pragma unroll
        for (int i = 0; i < kV; ++i) v[i] = 0.f;
        if (mine) {
            for (int p = lane; p < parts; p += 32) m = fmaxf(m, w.ml[(slot(p) * kRows + r) * 2]);
#pragma unroll
            for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
            for (int p = lane; p < parts; p += 32) {
                const float2 ml = *reinterpret_cast<const float2 *>(w.ml + (slot(p) * kRows + r) * 2);
                l = fmaf(ml.y, ml.x == m ? 1.f : exp2_fast((ml.x - m) * a.scale_log2), l);
            }
#pragma unroll
            for (int o = 16; o; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
#pragma unroll 4
            for (int p = way; p < parts; p += share) {
                const float mp = w.ml[(slot(p) * kRows + r) * 2], f = mp == m ? 1.f : exp2_fast((mp - m) * a.scale_log2);
                const float *src = w.o + (slot(p) * kRows + r) * HD + lane * kV;
#pragma unroll
                for (int i = 0; i < kV; i += 2) {
                    const float2 x = *reinterpret_cast<const float2 *>(src + i);
                    v[i] = fmaf(x.x, f, v[i]), v[i + 1] = fmaf(x.y, f, v[i + 1]);
                }
            }
        }
        if (share > 1) {
            __syncthreads();
#pragma unroll
            for (int i = 0; i < kV; ++i) s_o[warp][lane * kV + i] = v[i];
            __syncthreads();
            if (way) continue;
            for (int k = 1; k < share; ++k)
#pragma unroll
                for (int i = 0; i < kV; ++i) v[i] += s_o[warp + k][lane * kV + i];
        }
        if (!mine) continue;
        const float d = 1.f / l;
        const int p = first + r;
        uint32_t *to = reinterpret_cast<uint32_t *>(static_cast<T *>(a.out) + (int64_t)(row0 + p / g) * a.ldo + (h * g + p % g) * HD + lane * kV);
#pragma unroll
        for (int i = 0; i < kV; i += 2) to[i / 2] = pack2<T>(v[i] * d, v[i + 1] * d);
    }
}

// Rows of a chunk: the fewest of 16, 32, 64 (and 128 below 256 channels, whose sums fit the registers) that hold all, or the most
int chunk_rows(int hd, int rows) { return rows <= 16 ? 16 : rows <= 32 ? 32 : rows <= 64 || hd == 256 ? 64 : 128; }

struct Scratch {
    size_t pre, ml, o, total;
};
Scratch scratch_of(const dfl_paged *c, int n_q, int rows) {
    const size_t r = (size_t)kMaxCtas * 2 * chunk_rows(c->head_dim, rows * (n_q / c->n_kv));
    Scratch s;
    s.pre = ((size_t)(c->n_seq + 2) * 4 + 255) / 256 * 256;
    s.ml = r * 2 * 4;
    s.o = r * c->head_dim * 4;
    s.total = s.pre + s.ml + s.o;
    return s;
}

template <typename T, int HD, int MT, int MW>
int launch_shape(const AttnWork &w, cudaStream_t st) {
    using Sh = Shape<HD, MT, MW>;
    const int dev = current_device();
    if (dev < 0) return DFL_E_CUDA;
    static int sms[kMaxDevices] = {};
    if (!sms[dev]) {
        int n = 0;
        if (cudaFuncSetAttribute(k_paged_attn<T, HD, MT, MW>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 Sh::kQ + Sh::kRing + (DFL_PAGED_MAX_SEQ + 1) * 4) != cudaSuccess ||
            cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
            return DFL_E_CUDA;
        sms[dev] = n;
    }
    const dfl_paged &c = w.a.c;
    const int64_t most = (int64_t)c.n_seq * c.n_kv * w.chunks * (((int64_t)c.max_pages * c.page + kGranule - 1) / kGranule + 1);
    const int ctas = int(std::min<int64_t>(std::min(2 * sms[dev], kMaxCtas), (most + kLeast - 1) / kLeast));
    const cudaError_t e = launch_pdl(k_paged_attn<T, HD, MT, MW>, dim3(ctas), dim3(kThreads), Sh::kQ + Sh::kRing + (c.n_seq + 1) * 4, st, w);
    if (e != cudaSuccess) return DFL_E_CUDA;
    const int units = c.n_kv * w.chunks, rows = std::min(Sh::kRows, w.a.rows * w.a.group);
    AttnWork m = w;
    m.ways = (int64_t)c.n_seq * units * rows >= 8 * sms[dev] ? 1 : kMergeThreads / 32;
    const dim3 grid(m.ways > 1 ? rows : (rows + 7) / 8, units, c.n_seq);
    return pg_launched(launch_pdl(k_paged_merge<T, HD>, grid, dim3(kMergeThreads), 0, st, m, int(Sh::kRows)));
}

template <typename T, int HD>
int launch_rows(const AttnWork &w, int rows, cudaStream_t st) {
    if constexpr (HD == 256)
        return rows == 16 ? launch_shape<T, HD, 1, 1>(w, st) : rows == 32 ? launch_shape<T, HD, 1, 2>(w, st) : launch_shape<T, HD, 2, 2>(w, st);
    else
        return rows == 16   ? launch_shape<T, HD, 1, 1>(w, st)
               : rows == 32 ? launch_shape<T, HD, 2, 1>(w, st)
               : rows == 64 ? launch_shape<T, HD, 2, 2>(w, st)
                            : launch_shape<T, HD, 2, 4>(w, st);
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
    const int rows = chunk_rows(a.c.head_dim, a.rows * a.group);
    uint8_t *at = static_cast<uint8_t *>(scratch);
    const AttnWork w{a, (a.rows * a.group + rows - 1) / rows, reinterpret_cast<int *>(at), reinterpret_cast<float *>(at + s.pre),
                     reinterpret_cast<float *>(at + s.pre + s.ml), 1};
    return a.c.type == DFL_BF16 ? launch_type<__nv_bfloat16>(w, rows, st) : launch_type<__half>(w, rows, st);
}

}  // namespace dfl
