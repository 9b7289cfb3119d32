// paged.cu -- a paged key/value cache in 16 bits (include/dfl.h, dfl_paged): plans, rows into pages, and the entry points.
#include <algorithm>
#include <atomic>

#include "paged.cuh"

namespace dfl {
namespace {

// ---------------------------------------------------------------------------------------------------
// plan
// ---------------------------------------------------------------------------------------------------
// Sums over the sequences give each one's rows, the pages it gives back and those it takes. A CTA reads all
// lengths and scans them itself, so that one launch of many CTAs can share the writing: slots, table entries
// and ring places of a plan follow from the state before it alone. Pages taken that the ring did not hold yet
// are those given back in this call, found by the sums. The CTA that comes last writes what all read. Its bytes are a
// few microseconds' at most (1.4 MB for 512 prompts); what it takes is the chain of loads, two scans and the last CTA.
// THREADS: 512 where there are many rows to write (328 thousand of 512 sequences in 9.4 us, 11.2 with 256), 256 where
// the call is short (64 sequences in 5.0 us, 5.8 with 512).
constexpr int kPlanMany = 32768;

struct PlanArgs {
    dfl_paged c;
    const int32_t *len, *cnt;
    int32_t *cu, *slots;
    int rows, shift;           // page = 1 << shift
};

// Sums over the CTA's threads of two numbers, up to each thread's own; *all gets the whole ones'.
template <int THREADS>
__device__ longlong2 plan_scan(longlong2 v, longlong2 *red, longlong2 *all) {
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    constexpr int kW = THREADS / 32;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long x = __shfl_up_sync(0xffffffffu, v.x, o), y = __shfl_up_sync(0xffffffffu, v.y, o);
        if (lane >= o) v.x += x, v.y += y;
    }
    if (lane == 31) red[w] = v;
    __syncthreads();
    longlong2 total{0, 0};
#pragma unroll
    for (int i = 0; i < kW; ++i) {
        const longlong2 r = red[i];
        if (i == w) v.x += total.x, v.y += total.y;
        total.x += r.x, total.y += r.y;
    }
    *all = total;
    return v;
}

// the first sequence whose sum lies above x (sums ascend; one does)
__device__ __forceinline__ int plan_find(const int *sum, int n, int x) {
    int lo = 0, hi = n - 1;
    while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (sum[mid] > x) hi = mid;
        else lo = mid + 1;
    }
    return lo;
}

template <int THREADS, int EACH>               // EACH: sequences of a thread at most
__global__ void __launch_bounds__(THREADS) k_paged_plan(PlanArgs a) {
    extern __shared__ int plan_smem[];
    __shared__ longlong2 red[2][THREADS / 32];
    __shared__ int s_bits, s_used, s_last;
    const dfl_paged &c = a.c;
    const int S = c.n_seq, N = c.n_pages, P = c.page, t = threadIdx.x;
    int *row_end = plan_smem, *give_end = row_end + S, *take_end = give_end + S, *want = take_end + S, *had = want + S, *got = had + S, *lens = got + S;
    pdl_wait();
    pdl_trigger();
    if (t == 0) s_bits = s_used = 0;
    const int first = c.queue[0], count = c.queue[1];
    // the sequences of a thread follow each other, so that its own sums add up in place
    const int each = (S + THREADS - 1) / THREADS, s0 = min(t * each, S), s1 = min(s0 + each, S);
    int bits = 0, n[EACH], len[EACH], held[EACH];
    longlong2 sum{0, 0}, total, moved;
#pragma unroll
    for (int i = 0; i < EACH; ++i)
        if (s0 + i < s1) len[i] = a.len[s0 + i], n[i] = a.cnt[s0 + i], held[i] = c.held[s0 + i];
#pragma unroll
    for (int i = 0; i < EACH; ++i)
        if (s0 + i < s1) {
            if (len[i] < 0 || n[i] < 0) len[i] = -1, n[i] = 0, bits |= kPgArg;
            sum.x += n[i];
        }
    long long at = plan_scan<THREADS>(sum, red[0], &total).x - sum.x;
    longlong2 move{0, 0};      // pages given back, pages taken
#pragma unroll
    for (int i = 0; i < EACH; ++i)
        if (s0 + i < s1) {
            const int s = s0 + i;
            at += n[i];
            row_end[s] = int(min(at, (long long)INT32_MAX));
            lens[s] = len[i];
            bool fine = len[i] >= 0;
            if (fine && ((long long)len[i] + n[i] > (long long)c.max_pages * P || at > a.rows)) fine = false, bits |= kPgCapacity;
            if (held[i] < 0 || held[i] > c.max_pages) fine = false, held[i] = 0, bits |= kPgState;
            want[s] = fine ? int(((long long)len[i] + n[i] + P - 1) >> a.shift) : held[i];
            had[s] = held[i];
            got[s] = fine;
            move.x += max(held[i] - want[s], 0);
            move.y += max(want[s] - held[i], 0);
        }
    const longlong2 upto = plan_scan<THREADS>(move, red[1], &moved);
    long long give = upto.x - move.x, take = upto.y - move.y;
    const bool sound = first >= 0 && first < N && count >= 0 && count <= N && count + moved.x <= N;
    const int have = sound ? int(count + moved.x) : 0;
    for (int s = s0; s < s1; ++s) {
        give += max(had[s] - want[s], 0);
        const int need = max(want[s] - had[s], 0);
        take += need;
        if (!sound) got[s] = 0, bits |= kPgState;
        if (got[s] && need && take > have) got[s] = 0, bits |= kPgCapacity;
        give_end[s] = int(min(give, (long long)INT32_MAX));
        take_end[s] = int(min(take, (long long)INT32_MAX));
        if (got[s] && need) atomicMax(&s_used, int(take));
    }
    if (bits) atomicOr(&s_bits, bits);
    __syncthreads();
    const int used = s_used, G = gridDim.x * THREADS, me = blockIdx.x * THREADS + t;
    const int given = sound ? int(moved.x) : 0;
    // page i of those that the plan takes, in their order
    const auto taken = [&](int i) {
        if (i < count) return c.ring[i < N - first ? first + i : first + i - N];
        const int s = plan_find(give_end, S, i - count), j = i - count - (give_end[s] - (had[s] - want[s]));
        return c.table[(size_t)s * c.max_pages + want[s] + j];
    };
    const auto wrap = [&](int i) { return i < N ? i : i < 2 * N ? i - N : i - 2 * N; };   // (N is below 2^27)
    // a thread's first page taken and first page given back, asked for before the rows are looked at
    const int taker = me < used ? plan_find(take_end, S, me) : 0, giver = me < given ? plan_find(give_end, S, me) : 0;
    const int first_taken = me < used ? taken(me) : 0;
    const auto back = [&](int j, int s) { return c.table[(size_t)s * c.max_pages + want[s] + j - (give_end[s] - (had[s] - want[s]))]; };
    const int first_given = me < given ? back(me, giver) : 0;
    int worse = 0;
    // four rows a thread: they mostly lie in one page, which is looked up once
    for (int r0 = 4 * me; r0 < a.rows; r0 += 4 * G) {
        int slot[4] = {-1, -1, -1, -1}, s = -1, page = -1, id = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int r = r0 + i;
            if (r >= total.x) break;
            if (s < 0) s = plan_find(row_end, S, r);
            while (row_end[s] <= r) ++s, page = -1;
            if (!got[s]) continue;
            const int pos = lens[s] + r - (s ? row_end[s - 1] : 0), p = pos >> a.shift;
            if (p != page) {
                page = p;
                id = p < had[s] ? c.table[(size_t)s * c.max_pages + p] : taken(take_end[s] - (want[s] - had[s]) + p - had[s]);
            }
            if (id >= 0 && id < N) slot[i] = (id << a.shift) + (pos & (P - 1));
            else worse = kPgArg;
        }
        if (r0 + 4 <= a.rows && (reinterpret_cast<uintptr_t>(a.slots) & 15) == 0)
            *reinterpret_cast<int4 *>(a.slots + r0) = make_int4(slot[0], slot[1], slot[2], slot[3]);
        else
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (r0 + i < a.rows) a.slots[r0 + i] = slot[i];
    }
    for (int i = me; i < used; i += G) {
        const int s = i == me ? taker : plan_find(take_end, S, i);
        c.table[(size_t)s * c.max_pages + had[s] + i - (take_end[s] - (want[s] - had[s]))] = i == me ? first_taken : taken(i);
    }
    for (int j = me; j < given; j += G) c.ring[wrap(first + count + j)] = j == me ? first_given : back(j, plan_find(give_end, S, j));
    if (blockIdx.x == 0)
        for (int s = t; s <= S; s += THREADS) a.cu[s] = s ? min(row_end[s - 1], a.rows) : 0;
    if (worse) atomicOr(&s_bits, worse);
    __syncthreads();
    if (t == 0) {
        if (s_bits) atomicOr(c.err, s_bits);
        s_last = 1;
        if (gridDim.x > 1) {
            __threadfence();
            s_last = atomicInc(reinterpret_cast<unsigned *>(c.queue + 2), gridDim.x - 1) == gridDim.x - 1;
        }
    }
    __syncthreads();
    if (!s_last || !sound) return;
    for (int s = t; s < S; s += THREADS)
        if (got[s]) c.held[s] = want[s];
    if (t == 0) {
        c.queue[0] = wrap(first + used);
        c.queue[1] = have - used;
    }
}

template <int THREADS, int EACH>
int launch_plan(const PlanArgs &a, cudaStream_t s) {
    const int dev = current_device();
    if (dev < 0) return DFL_E_CUDA;
    static bool done[kMaxDevices] = {};
    if (!done[dev]) {
        if (cudaFuncSetAttribute(k_paged_plan<THREADS, EACH>, cudaFuncAttributeMaxDynamicSharedMemorySize, 7 * 4 * DFL_PAGED_MAX_SEQ) != cudaSuccess)
            return DFL_E_CUDA;
        done[dev] = true;
    }
    const int ctas = std::min(std::max(int(((int64_t)a.rows + 4 * THREADS - 1) / (4 * THREADS)), std::max(1, std::min(16, a.c.n_pages / 16384))), 304);
    return pg_launched(launch_pdl(k_paged_plan<THREADS, EACH>, dim3(ctas), dim3(THREADS), (size_t)7 * 4 * a.c.n_seq, s, a));
}
template <int THREADS>
int launch_plan(const PlanArgs &a, cudaStream_t s) {
    return a.c.n_seq <= THREADS ? launch_plan<THREADS, 1>(a, s) : launch_plan<THREADS, DFL_PAGED_MAX_SEQ / THREADS>(a, s);
}

__global__ void k_paged_init(dfl_paged c) {
    const int i = blockIdx.x * blockDim.x + threadIdx.x;
    if (i < c.n_pages) c.ring[i] = i;
    if (i < c.n_seq) c.held[i] = 0;
    if (i < 4) c.queue[i] = i == 1 ? c.n_pages : 0;
    if (i == 0) *c.err = 0;
}

// ---------------------------------------------------------------------------------------------------
// append
// ---------------------------------------------------------------------------------------------------
struct AppendArgs {
    dfl_paged c;
    const int32_t *slots;
    int rows;
    const uint8_t *k, *v;
    int64_t ldk, ldv;          // bytes
};

// One thread moves 16 bytes of a key and of the value beside it: bound by HBM (14.6 thousand rows of 16 heads of 128 in 38.8 us, 6.2
// TB/s, 91 % of measured), or for few rows by the launch (64 rows in 1.6 us in a graph, 5.2 with the host).
__global__ void __launch_bounds__(256) k_paged_append(AppendArgs a) {
    const dfl_paged &c = a.c;
    const int hc = c.head_dim / 8, chunks = c.n_kv * hc;       // 16-byte pieces of a head, of a row
    pdl_wait();
    pdl_trigger();
    const long long i = (long long)blockIdx.x * 256 + threadIdx.x;
    const int r = int(i / chunks), at = int(i % chunks), h = at / hc, x = at % hc;
    if (r >= a.rows) return;
    const int slot = a.slots[r];
    if (slot < 0) return;
    const int page = slot / c.page;
    if (page >= c.n_pages) {
        pg_report(c.err, kPgArg);
        return;
    }
    const size_t to = (((size_t)page * c.n_kv + h) * c.page + slot % c.page) * hc + x;
    const uint4 k = ldg_stream(a.k + r * a.ldk + at * 16), v = ldg_stream(a.v + r * a.ldv + at * 16);
    static_cast<uint4 *>(c.k)[to] = k;
    static_cast<uint4 *>(c.v)[to] = v;
}

constexpr float kLog2e = 1.4426950408889634f;

std::atomic<int> test_stall{0};

}  // namespace
}  // namespace dfl

using namespace dfl;

extern "C" {

int dfl_paged_init(const dfl_paged *c, void *stream) {
    const int rc = pg_check(c);
    if (rc) return rc;
    const int n = std::max(std::max(c->n_pages, c->n_seq), 4);
    k_paged_init<<<unsigned((n + 255) / 256), 256, 0, static_cast<cudaStream_t>(stream)>>>(*c);
    return pg_launched(cudaGetLastError());
}

int dfl_paged_status(const dfl_paged *c, void *stream) {
    const int rc = pg_check(c);
    if (rc) return rc;
    int bits = 0;
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (cudaMemcpyAsync(&bits, c->err, 4, cudaMemcpyDeviceToHost, s) != cudaSuccess || cudaStreamSynchronize(s) != cudaSuccess)
        return DFL_E_CUDA;
    if (!bits) return DFL_OK;
    if (cudaMemsetAsync(c->err, 0, 4, s) != cudaSuccess) return DFL_E_CUDA;
    return bits & kPgTimeout ? DFL_E_TIMEOUT : bits & kPgArg ? DFL_E_INVALID_ARG : bits & kPgState ? DFL_E_STATE : DFL_E_CAPACITY;
}

int dfl_paged_plan(const dfl_paged *c, const int32_t *len, const int32_t *cnt, int32_t *cu, int32_t *slots, int rows, void *stream) {
    const int rc = pg_check(c);
    if (rc) return rc;
    if (!len || !cnt || !cu || rows < 0 || (rows && !slots)) return DFL_E_INVALID_ARG;
    if (rows > kPgMaxRows) return DFL_E_UNSUPPORTED;
    const void *p[] = {len, cnt, cu, slots};
    for (const void *q : p)
        if (!pg_aligned(q, 4)) return DFL_E_INVALID_ARG;
    // what is written shares memory with nothing else
    const struct {
        const void *p;
        int64_t bytes;
    } all[] = {{cu, (c->n_seq + 1) * 4ll}, {slots, rows * 4ll}, {len, c->n_seq * 4ll}, {cnt, c->n_seq * 4ll}, {c->held, c->n_seq * 4ll},
               {c->table, (int64_t)c->n_seq * c->max_pages * 4}, {c->ring, c->n_pages * 4ll}, {c->queue, 16}};
    for (int i = 0; i < 2; ++i)
        for (int j = i + 1; j < 8; ++j)
            if (pg_overlap(all[i].p, all[i].bytes, all[j].p, all[j].bytes)) return DFL_E_INVALID_ARG;
    for (int i = 4; i < 8; ++i)
        if (pg_overlap(len, all[2].bytes, all[i].p, all[i].bytes) || pg_overlap(cnt, all[3].bytes, all[i].p, all[i].bytes)) return DFL_E_INVALID_ARG;
    const PlanArgs a{*c, len, cnt, cu, slots, rows, pg_shift(c)};
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    return rows > kPlanMany ? launch_plan<512>(a, s) : launch_plan<256>(a, s);
}

int dfl_paged_append(const dfl_paged *c, const int32_t *slots, int rows, const void *k, int64_t ldk, const void *v, int64_t ldv,
                     void *stream) {
    int rc = pg_check(c);
    if (rc) return rc;
    if (rows == 0) return DFL_OK;
    if (rows < 0 || !slots || !pg_aligned(slots, 4)) return DFL_E_INVALID_ARG;
    if (rows > kPgMaxRows) return DFL_E_UNSUPPORTED;
    if ((rc = pg_check_rows(c, k, ldk, c->n_kv)) || (rc = pg_check_rows(c, v, ldv, c->n_kv))) return rc;
    const int64_t w = (int64_t)c->n_kv * c->head_dim, pool = (int64_t)c->n_pages * c->page * w * 2;
    for (const void *p : {static_cast<const void *>(c->k), static_cast<const void *>(c->v)})
        if (pg_overlap(p, pool, k, ((rows - 1) * ldk + w) * 2) || pg_overlap(p, pool, v, ((rows - 1) * ldv + w) * 2)) return DFL_E_INVALID_ARG;
    const AppendArgs a{*c, slots, rows, static_cast<const uint8_t *>(k), static_cast<const uint8_t *>(v), ldk * 2, ldv * 2};
    const int64_t blocks = ((int64_t)rows * c->n_kv * (c->head_dim / 8) + 255) / 256;
    if (blocks > INT32_MAX) return DFL_E_UNSUPPORTED;
    return pg_launched(launch_pdl(k_paged_append, dim3(unsigned(blocks)), dim3(256), 0, static_cast<cudaStream_t>(stream), a));
}

int dfl_paged_prompt(const dfl_paged *c, const void *q, int64_t ldq, int n_q, const void *k, int64_t ldk, const void *v, int64_t ldv,
                     const int32_t *cu, int rows, int window, float scale, void *out, int64_t ldo, void *stream) {
    int rc = pg_check(c);
    if (rc || (rc = pg_check_heads(c, n_q, window, scale))) return rc;
    if (rows == 0) return DFL_OK;
    if (rows < 0 || !cu || !pg_aligned(cu, 4)) return DFL_E_INVALID_ARG;
    if (rows > kPgMaxRows) return DFL_E_UNSUPPORTED;
    if ((rc = pg_check_rows(c, q, ldq, n_q)) || (rc = pg_check_rows(c, k, ldk, c->n_kv)) || (rc = pg_check_rows(c, v, ldv, c->n_kv)) ||
        (rc = pg_check_rows(c, out, ldo, n_q)))
        return rc;
    const int64_t wq = (int64_t)n_q * c->head_dim, wk = (int64_t)c->n_kv * c->head_dim;
    if (pg_rows_overlap(out, ldo, wq, q, ldq, wq, rows) || pg_rows_overlap(out, ldo, wq, k, ldk, wk, rows) ||
        pg_rows_overlap(out, ldo, wq, v, ldv, wk, rows))
        return DFL_E_INVALID_ARG;
    const int g = n_q / c->n_kv;
    const PagedAttnArgs a{*c, q, k, v, out, ldq, ldk, ldv, ldo, n_q, g, rows, cu, nullptr, 0, window, 1, pg_shift(c), (4096 + g - 1) / g, scale * kLog2e,
                          test_stall.load(std::memory_order_relaxed)};
    return launch_paged_prompt(a, static_cast<cudaStream_t>(stream));
}

int dfl_paged_test_stall(int copies) {
    test_stall.store(copies, std::memory_order_relaxed);
    return DFL_OK;
}

int64_t dfl_paged_attn_scratch_bytes(const dfl_paged *c, int n_q, int rows) {
    if (!c || c->n_seq < 1 || c->n_seq > DFL_PAGED_MAX_SEQ || c->n_kv < 1 || n_q < 1 || n_q % c->n_kv || n_q / c->n_kv > kPgMaxGroup ||
        rows < 1 || rows > DFL_MAX_ROWS || (c->head_dim != 64 && c->head_dim != 128 && c->head_dim != 256))
        return -1;
    return (int64_t)paged_attn_scratch(c, n_q, rows);
}

int dfl_paged_attn(const dfl_paged *c, const void *q, int64_t ldq, int n_q, int total, const int32_t *cu, const int32_t *len, int rows,
                   int window, int causal, float scale, void *out, int64_t ldo, void *scratch, size_t scratch_bytes, void *stream) {
    int rc = pg_check(c);
    if (rc || (rc = pg_check_heads(c, n_q, window, scale))) return rc;
    if (rows < 1 || total < 0 || !cu || !len || !pg_aligned(cu, 4) || !pg_aligned(len, 4)) return DFL_E_INVALID_ARG;
    if (rows > DFL_MAX_ROWS || total > kPgMaxRows) return DFL_E_UNSUPPORTED;
    if (!scratch || !pg_aligned(scratch, 256) || (int64_t)scratch_bytes < dfl_paged_attn_scratch_bytes(c, n_q, rows)) return DFL_E_INVALID_ARG;
    if (total == 0) return DFL_OK;
    if ((rc = pg_check_rows(c, q, ldq, n_q)) || (rc = pg_check_rows(c, out, ldo, n_q))) return rc;
    const int64_t wq = (int64_t)n_q * c->head_dim, pool = (int64_t)c->n_pages * c->page * c->n_kv * c->head_dim * 2, all = ((total - 1) * ldo + wq) * 2;
    if (pg_rows_overlap(out, ldo, wq, q, ldq, wq, total) || pg_overlap(out, all, c->k, pool) || pg_overlap(out, all, c->v, pool)) return DFL_E_INVALID_ARG;
    const int g = n_q / c->n_kv;
    const PagedAttnArgs a{*c, q, nullptr, nullptr, out, ldq, 0, 0, ldo, n_q, g, total, cu, len, rows, window, causal != 0, pg_shift(c), (4096 + g - 1) / g, scale * kLog2e, 0};
    return launch_paged_attn(a, scratch, static_cast<cudaStream_t>(stream));
}

}  // extern "C"
