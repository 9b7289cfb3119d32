// prompt.cu -- causal grouped-query attention of packed prompts (include/dfl.h, dfl_paged_prompt) on the tcgen05
// tensor cores.
//
// A tile's 128 rows are tokens x query heads: 128 / g tokens, the g heads of one key/value head beside each other
// (row r = token r / g, head r % g), so a group's heads read their keys and values once and a short prompt fills
// one tile. A CTA takes kTiles tiles that follow each other and walks over the keys they see, kKeys at a time:
//     S = Q K^T (tensor memory), P = 2^(c S - m) rounded to the type (tensor memory, over S), O += P V
// with c = scale * log2(e). A thread owns one row: it holds the row's maximum and sum and needs no other thread's
// values. The maximum in use is renewed only where a tile's passes it by more than 16 powers of two (12, fp16); until then P
// is larger than 1 and no sum changes scale, so O in tensor memory is seldom touched.
//
// P is rounded to the type of the values, as the tensor cores take their operands: a relative 2^-8 (bf16) or 2^-11
// (fp16) of each weight at most, the size of the output's own rounding; the sum that divides is of the unrounded
// weights, in fp32. fp16 weights are held times 2^3, so that what is lost below its smallest number lies 2^-28
// below the largest weight.
//
// Masked places. A masked score is replaced, so what a key holds there shows nowhere. A masked weight is 0, and 0
// times a value that is not finite would make NaN of rows that do not see it; that shows in the sums at the end
// (one that is not finite where the weights' sum is). Then the CTA does its tiles once more, taking what is not finite out
// of each tile of values before the product, and notes for each row which channels it saw such a value in. So a
// prompt without such values pays nothing for them. One in 16384 tokens costs 1.1 to 3 times the price (32 heads of 128: 1.39 ms, 1.51 to
// 1.61; 12 of 256: 1.16, 2.3 to 2.8; 4 of 64: 0.16, 0.51), a prompt of nothing else ten times as much.
// What bounds it (measured in cycles of one CTA). Long rows of keys, 128 channels: a pair of tiles takes 128 keys in some
// 2900, of which the products are 2200 at full rate: a tile's softmax (1250: the maximum 400, the weights 750, the rest
// tensor memory) and its products (1100) follow each other, and two tiles in turn hide one behind the other. 256 channels:
// 64 keys in 1600, as the scores' products of 64 columns run at half rate (128 would need S or Q somewhere else).
// 64 channels: a tile's softmax costs as much beside half the products, and with 2 key/value heads 256 items of 1 to 128 pairs on 152
// SMs take as long as the longest one (an even share were 109).
// 16384 tokens: 1.39 to 1.44 ms for 32 heads of 128 (1530 to 1580 TFLOP/s, 79 to 82 % of measured; 1.45 to 1.5 ms over seconds,
// where the card's power counts), 1.15 to 1.18 ms for 12 of 256 (1400 to 1430), 0.16 ms for 4 of 64 (860). Short rows: an item begins and ends in some
// 10 thousand cycles (its place 1000 to 3000, queries and first keys 4000, sums out 3000 to 5000), as much as 3 pairs.
// What was measured on the way (the 16384 tokens above): one lane issuing its products under `lane == 0` 2.23 ms, under
// elect 1.58; queries by a thread a row 18 thousand cycles a tile, by asynchronous copies 3 thousand; weights handed over in
// halves 1.43 -> 1.39 ms (256 channels: 6 % slower, not done); CTAs that stay and take items in turn 1.53 ms (a short
// prompt 7.6 us, 4.9 with a CTA an item; packed prompts 3 % faster); one tile a CTA, two CTAs an SM 1.56 ms.
// The kernel of 128 channels spills 120 bytes a thread at its 168 registers (148 loaded back).
#include <algorithm>

#include "paged.cuh"
#include "tc.cuh"

namespace dfl {
namespace {

constexpr int kPromptQ = 128;    // tensor memory column of Q (256 channels alone)

template <int HD>
struct PromptShape {
    // 256 channels: one tile's sums take half of the tensor memory, so S is held twice instead of two tiles, and Q is
    // in tensor memory too, where the product reads it beside the keys from shared memory
    static constexpr int kTiles = HD == 256 ? 1 : 2;
    static constexpr int kKeys = HD == 256 ? 64 : 128;
    static constexpr int kStage = kKeys * HD * 2;
    static constexpr int kStages = HD == 64 ? 8 : 5;
    // Q of each tile; afterwards, and with 256 channels from the start, a place where each warp turns its rows round
    static constexpr int kQBytes = kTiles * 128 * HD * 2;
    static constexpr int kSmem = kQBytes + kStages * kStage + 1024;   // + slack to align to 1024 bytes
    static constexpr int kThreads = kTiles * 128 + 128;   // softmax; copies, products and two idle warps
    // (two tiles: a launch of 384 threads x 168 registers; 2 x 128 x 208 + 128 x 80 are fewer)
    // tensor memory columns
    static constexpr int kS = 0, kSPitch = kKeys;                      // two of them: a tile's each, or two in turn
    static constexpr int kO = 256;
};

struct PromptArgs {
    dfl_paged c;
    const uint8_t *q;
    uint8_t *out;
    int64_t ldq, ldo;          // bytes
    int group, inverse, total, window;            // r / group is (r * inverse) >> 12 for rows of a tile
    const int32_t *cu;
    float scale_log2;
    int stall;                 // test of the give-up path: the most copies of an item in its first pass, or, negative, its second
};

// Instruction descriptor of kind::f16 with an fp32 accumulator of 128 rows and N columns: operands of the type, A
// along its inputs, B along them or (transposed) along its columns.
template <typename T>
__device__ constexpr uint32_t prompt_idesc(int N, bool transposed) {
    const uint32_t fmt = std::is_same<T, __nv_bfloat16>::value ? 1u : 0u;
    return (1u << 4) | (fmt << 7) | (fmt << 10) | (transposed ? 1u << 16 : 0u) | (uint32_t(N >> 3) << 17) | (128u >> 4 << 24);
}

__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}"
        ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
        : "memory");
}
// A from tensor memory: 128 lanes, two inputs a column
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}"
        ::"r"(d), "r"(a), "l"(b), "r"(idesc), "r"(accumulate)
        : "memory");
}

// One lane of a warp whose lanes are all here. The products are issued under it and not under a lane's number: the compiler then
// knows that one thread is active, and keeps descriptors and addresses in uniform registers.
__device__ __forceinline__ bool elect_one() {
    uint32_t ok;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(ok));
    return ok != 0;
}
template <typename X>
__device__ __forceinline__ X uniform(X x) { return __shfl_sync(0xffffffffu, x, 0); }

// Descriptor of a tile [keys][64-channel blocks of 128 bytes] read along its channels (the product's columns): 8 keys
// are 1024 bytes, the next 64 channels `block` bytes further.
__device__ __forceinline__ uint64_t values_desc(const void *tile, int block) {
    const uint64_t a = saddr(tile);
    return ((a >> 4) & 0x3FFFull) | ((uint64_t)(block >> 4) << 16) | ((uint64_t)(1024 >> 4) << 32) | (1ull << 46) | (2ull << 61);
}

__device__ __forceinline__ void tma_load_3d(void *dst, const CUtensorMap *map, int x, int y, int z, uint64_t *b) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];"
        ::"r"(saddr(dst)), "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(saddr(b))
        : "memory");
}

// mbar_wait with what mostly happens first: the phase is over
__device__ __forceinline__ bool wait_for(uint64_t *b, unsigned parity, volatile int *bad) {
    return mbar_test(b, parity) || mbar_wait(b, parity, bad);
}

// A place in the ring and the parity of the phase there, moved on without divisions
struct Place {
    int s;
    unsigned phase;
    __device__ void go(int by, int stages) {
        s += by;
        if (s >= stages) s -= stages, phase ^= 1u;
    }
};

__device__ __forceinline__ void st_shared(unsigned at, uint4 v) {
    asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}
__device__ __forceinline__ uint4 ld_shared(unsigned at) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(at) : "memory");
    return v;
}

// two numbers in a register pair
__device__ __forceinline__ uint64_t pair(uint32_t lo, uint32_t hi) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "r"(lo), "r"(hi));
    return r;
}
__device__ __forceinline__ void halves(uint64_t p, float &lo, float &hi) { asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(p)); }
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}

// Outputs of finite values. They lie between the largest and the smallest value, but as weights are rounded and the sum that divides is not, by
// up to 2^-11 (fp16) further out: at the type's end, where that would be infinite, they are its largest number. A NaN stays one.
template <typename T>
__device__ __forceinline__ uint32_t pack2_out(float lo, float hi) {
    if constexpr (std::is_same<T, __nv_bfloat16>::value) return pack2<T>(lo, hi);   // (the header's limit on values is far below its end)
    uint32_t r;
    asm("cvt.rn.satfinite.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

// Whether a 16-bit number is an infinity or a NaN
template <typename T>
__device__ __forceinline__ bool odd16(uint32_t x) {
    const uint32_t e = std::is_same<T, __nv_bfloat16>::value ? 0x7F80u : 0x7C00u;
    return (x & e) == e;
}

__device__ __forceinline__ void mbar_inval(uint64_t *b) { asm volatile("mbarrier.inval.shared::cta.b64 [%0];" ::"r"(saddr(b)) : "memory"); }

// The keys that tile w of the item sees, as tiles of kKeys
struct KeyRange {
    int begin, end;
};

// Items: kTiles tiles of a sequence. Of all sequences together the last ones, which see most keys, come first, so that what the
// grid's end is made of is short: item number x has the largest index i for which more than x items have an index of i or above.
struct Item {
    int row0, rows, at;                          // the sequence's first row and rows; the item's index in it
};
constexpr int kItemLanes = 8;                    // sequences of a lane at most

__device__ __forceinline__ int items_of(const PromptArgs &a, int per, int s, int h, int number, int *row0, int *rows) {
    const int b = a.cu[s], e = a.cu[s + 1];
    if (b < 0 || e < b || e > a.total) {
        if (number == 0 && h == 0) pg_report(a.c.err, kPgArg);
        return 0;
    }
    *row0 = b, *rows = e - b;
    return (e - b + per - 1) / per;
}

// Every warp for itself, up to 32 * LANES sequences
template <int LANES>
__device__ __forceinline__ bool find_item(const PromptArgs &a, int per, int number, int h, Item &item) {
    const int lane = threadIdx.x & 31, S = a.c.n_seq;
    if (S == 1) {
        const int n = items_of(a, per, 0, h, number, &item.row0, &item.rows);
        item.at = n - 1 - number;
        return number < n;
    }
    int n[LANES], row0[LANES], rows[LANES], most = 0;
#pragma unroll
    for (int v = 0; v < LANES; ++v) {
        n[v] = 0;
        if (32 * v < S) {                        // (the warp together)
            const int s = min(32 * v + lane, S - 1), count = items_of(a, per, s, h, number, &row0[v], &rows[v]);
            n[v] = 32 * v + lane < S ? count : 0;
            most = max(most, n[v]);
        }
    }
    const auto from = [&](int i) {               // items with an index of i or above
        int sum = 0;
#pragma unroll
        for (int v = 0; v < LANES; ++v)
            if (32 * v < S) sum += max(0, n[v] - i);
        return __reduce_add_sync(0xffffffffu, sum);
    };
    int lo = 0, hi = __reduce_max_sync(0xffffffffu, most);       // from(lo) > number >= from(hi)
    if (number >= from(0)) return false;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (from(mid) > number) lo = mid;
        else hi = mid;
    }
    int left = number - from(hi);                // of the sequences that have an item of index lo, the left-th
#pragma unroll
    for (int v = 0; v < LANES; ++v) {
        if (32 * v >= S || left < 0) break;
        const uint32_t has = __ballot_sync(0xffffffffu, n[v] > lo);
        const int count = __popc(has);
        if (left < count) {
            const uint32_t who = __ballot_sync(0xffffffffu, (has >> lane & 1u) && __popc(has & ((1u << lane) - 1u)) == left);
            const int from_lane = __ffs(who) - 1;
            item.row0 = __shfl_sync(0xffffffffu, row0[v], from_lane);
            item.rows = __shfl_sync(0xffffffffu, rows[v], from_lane);
        }
        left -= count;
    }
    item.at = lo;
    return true;
}

// The CTA together, any number of sequences: one after another, the last items of each first
template <int THREADS>
__device__ bool find_item_wide(const PromptArgs &a, int per, int number, int h, int *sums, Item *item) {
    const int t = threadIdx.x, warp = t >> 5, lane = t & 31, S = a.c.n_seq;
    const int each = (S + THREADS - 1) / THREADS, s0 = min(t * each, S), s1 = min(s0 + each, S);
    int mine = 0, row0 = 0, rows = 0;
    for (int s = s0; s < s1; ++s) mine += items_of(a, per, s, h, number, &row0, &rows);
    int sum = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(0xffffffffu, sum, o);
        if (lane >= o) sum += u;
    }
    if (t == 0) item->rows = 0;
    if (lane == 31) sums[warp] = sum;
    __syncthreads();
    for (int w = 0; w < warp; ++w) sum += sums[w];
    int left = number - (sum - mine);
    if (left >= 0 && left < mine)
        for (int s = s0; s < s1; ++s) {
            const int n = items_of(a, per, s, h, 1, &row0, &rows);
            if (left < n) {
                *item = Item{row0, rows, n - 1 - left};
                break;
            }
            left -= n;
        }
    __syncthreads();
    return item->rows > 0;
}

template <typename T, int HD>
__global__ void __launch_bounds__(PromptShape<HD>::kThreads, 1)
    k_prompt(const __grid_constant__ CUtensorMap tk, const __grid_constant__ CUtensorMap tv, const PromptArgs a) {
    using Sh = PromptShape<HD>;
    constexpr int kTiles = Sh::kTiles, kKeys = Sh::kKeys, kSoft = kTiles * 128, kMaxStages = Sh::kStages;
    extern __shared__ uint8_t prompt_smem_raw[];
    __shared__ __align__(8) uint64_t full[kMaxStages], empty[kMaxStages], b_q, b_s[2], b_p[2], b_h[2], b_o[2], b_meet[3], b_done;
    __shared__ uint32_t s_tmem, s_odd[3][kKeys / 32];
    __shared__ int s_issued, s_again, s_sum[Sh::kThreads / 32];
    __shared__ Item s_item;
    __shared__ volatile int s_bad;
    uint8_t *base = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(prompt_smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t *qs = base, *ring = base + Sh::kQBytes;
    const int t = threadIdx.x, warp = t >> 5, lane = t & 31, g = a.group;
    const int tokens = 128 / g;                                  // of a tile
    const int h = blockIdx.x % a.c.n_kv, number = blockIdx.x / a.c.n_kv;
    if (warp == kTiles * 4 && lane == 0) {
        asm volatile("prefetch.tensormap [%0];" ::"l"(&tk) : "memory");
        asm volatile("prefetch.tensormap [%0];" ::"l"(&tv) : "memory");
    }
    pdl_wait();
    pdl_trigger();

    // ---- the CTA's item: tiles item * kTiles .. of a sequence ----
    Item item;
    if (a.c.n_seq <= 32) {
        if (!find_item<1>(a, kTiles * tokens, number, h, item)) return;          // each warp by itself
    } else if (a.c.n_seq <= 32 * kItemLanes) {
        if (!find_item<kItemLanes>(a, kTiles * tokens, number, h, item)) return;
    } else {
        if (!find_item_wide<Sh::kThreads>(a, kTiles * tokens, number, h, s_sum, &s_item)) return;
        item = s_item;
    }
    const int row0 = item.row0, n = item.rows, tok0 = item.at * kTiles * tokens;
    const auto range = [&](int w) {
        const int lo = tok0 + w * tokens, hi = min(lo + tokens, n);
        KeyRange r{0, 0};
        if (lo < n) {
            r.begin = a.window ? max(0, lo - a.window + 1) / kKeys : 0;
            r.end = (hi + kKeys - 1) / kKeys;
        }
        return r;
    };
    const KeyRange r0 = range(0), r1 = kTiles == 2 ? range(1) : KeyRange{0, 0};
    const int jb = r0.begin, je = max(r0.end, r1.end);           // tiles of keys that any row sees
    if (warp == kTiles * 4 + 1) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(saddr(&s_tmem)), "r"(512) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }

    // What each pass begins and ends with; the warps of a kind go through both of their passes by themselves, so that each kind has its
    // registers.
    const auto init_pass = [&](int again) {      // by the thread that copies: its first copies need not wait for the others
        if (again) {
            for (int i = 0; i < kMaxStages; ++i) mbar_inval(&full[i]), mbar_inval(&empty[i]);
            for (int i = 0; i < 2; ++i) mbar_inval(&b_s[i]), mbar_inval(&b_p[i]), mbar_inval(&b_h[i]), mbar_inval(&b_o[i]);
            for (int i = 0; i < 3; ++i) mbar_inval(&b_meet[i]);
            mbar_inval(&b_q), mbar_inval(&b_done);
        }
        for (int i = 0; i < kMaxStages; ++i) {
            mbar_init(&full[i], 1);              // the producer's arrival (with the stage's bytes)
            mbar_init(&empty[i], 1);             // the MMA thread's commit
        }
        mbar_init(&b_q, kSoft);                  // Q lies where the products read it
        for (int i = 0; i < 2; ++i) {
            mbar_init(&b_s[i], 1);               // S is complete: the MMA thread's commit
            mbar_init(&b_h[i], 128);             // two tiles: the first half of P lies in tensor memory, and O may be added to
            mbar_init(&b_p[i], 128);             // all of it does
            mbar_init(&b_o[i], 1);               // P V is added: a tile's, or of every other tile of keys
        }
        for (int i = 0; i < 3; ++i) mbar_init(&b_meet[i], i ? 128 : kSoft);   // the threads of both tiles, of one
        mbar_init(&b_done, 1);                   // the MMA thread's last commit
        s_issued = s_again = 0;
        s_bad = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    };
    const auto begin_pass = [&] {
        tc_fence_before();
        __syncthreads();
        tc_fence_after();
    };
    const auto end_pass = [&](int stages) {
        tc_fence_before();
        __syncthreads();
        if (t == 0) {
            // every commit has landed before anything is used again; after a wait gave up, every copy issued too
            if (s_bad)
                for (int k = max(0, s_issued - stages); k < s_issued; ++k) mbar_drain(&full[k % stages], unsigned(k / stages) & 1u);
            if (!mbar_drain(&b_done, 0u)) s_bad = 1;
            if (s_bad) pg_report(a.c.err, kPgTimeout);
        }
        __syncthreads();
        tc_fence_after();
        const bool done = s_bad || !s_again;
        __syncthreads();
        return done;
    };

    if (warp >= kTiles * 4) {
        if constexpr (kTiles == 2) asm volatile("setmaxnreg.dec.sync.aligned.u32 80;");
        for (int again = 0; again < 2; ++again) {
            const int stages = kMaxStages - again;     // the second time the last stage holds the notes on values that are not finite
            if (warp == kTiles * 4) {
                // ---- copies: K and V of each tile in turn through the ring ----
                const int limit = again ? -a.stall : a.stall, all = limit > 0 ? min(limit, 2 * (je - jb)) : 2 * (je - jb);
                int k = 0;
                Place at{0, 1u};                       // (the first round's stages are free: the phase before counts as over)
                const auto copy = [&] {
                    mbar_expect(&full[at.s], unsigned(Sh::kStage));
                    for (int x = 0; x < HD / 64; ++x)
                        tma_load_3d(ring + at.s * Sh::kStage + x * kKeys * 128, k & 1 ? &tv : &tk, 64 * x, h, row0 + (jb + (k >> 1)) * kKeys, &full[at.s]);
                    at.go(1, stages);
                    ++k;
                };
                if (lane == 0) {
                    init_pass(again);
                    copy();                        // (the others would stand in the queries' way)
                }
                __syncwarp();
                begin_pass();
                if (lane == 0) {
                    while (k < all && wait_for(&empty[at.s], at.phase, &s_bad) && !s_bad) copy();
                    s_issued = k;
                }
                __syncwarp();
            } else if (warp == kTiles * 4 + 1) {
                begin_pass();
                const uint32_t tmem = s_tmem;
                // ---- products: the whole warp waits, one lane issues ----
                constexpr uint32_t id_s = prompt_idesc<T>(kKeys, false), id_o = prompt_idesc<T>(HD, true);
                const uint64_t q_desc = uniform(sw128_desc(qs)), k_desc = uniform(sw128_desc(ring)), v_desc = uniform(values_desc(ring, kKeys * 128));
                const uint32_t tm = uniform(tmem);
                const int begin = uniform(jb), end = uniform(je);
                const KeyRange rs[2] = {{uniform(r0.begin), uniform(r0.end)}, {uniform(r1.begin), uniform(r1.end)}};
                const auto scores = [&](int w, int at, int stage) {        // tile w, S number `at`, keys in the stage
                    const uint64_t b = k_desc + uint64_t(stage * (Sh::kStage >> 4)), q = q_desc + uint64_t(w * (HD / 64) * (16384 >> 4));
                    const uint32_t d = tm + Sh::kS + at * Sh::kSPitch;
#pragma unroll
                    for (int i = 0; i < HD / 16; ++i) {
                        const uint64_t bi = b + uint64_t((i / 4) * (kKeys * 128 >> 4) + 2 * (i % 4));
                        if constexpr (HD == 256) mma_ts(d, tm + kPromptQ + 8 * i, bi, id_s, i > 0);
                        else mma_ss(d, q + uint64_t((i / 4) * (16384 >> 4) + 2 * (i % 4)), bi, id_s, i > 0);
                    }
                };
                const auto values = [&](int w, int at, int stage, bool add, int half) {      // of the tile's keys the first or second half

                    const uint64_t b = v_desc + uint64_t(stage * (Sh::kStage >> 4));
                    const uint32_t d = tm + Sh::kO + w * HD, p = tm + Sh::kS + at * Sh::kSPitch;
#pragma unroll
                    for (int y = 0; y < kKeys / 32; ++y) {
                        const int i = half * (kKeys / 32) + y;
                        mma_ts(d, p + 8 * i, b + uint64_t(i * (2048 >> 4)), id_o, add || i > 0);
                    }
                };
                const auto over = [&](uint64_t *b, unsigned parity) { return __all_sync(0xffffffffu, wait_for(b, parity, &s_bad)) != 0; };
                bool ok = over(&b_q, 0u);
                tc_fence_after();
                Place k{0, 0u}, v{1, 0u};              // the stages of K j and of V j - 1
                unsigned p_phase[2] = {0u, 0u};
                // a thread's products run in the order of issue: S may be written over P as soon as P V has been issued
                for (int j = begin; ok && j <= end; ++j) {
                    if constexpr (kTiles == 1) {
                        if (j < end) {
                            if (!(ok = over(&full[k.s], k.phase))) break;
                            tc_fence_after();
                            if (elect_one()) {
                                scores(0, j & 1, k.s);
                                tc_commit(&b_s[j & 1]);
                                tc_commit(&empty[k.s]);
                            }
                            k.go(2, stages);
                        }
                        if (j > begin) {
                            const int at = (j - 1) & 1;
                            if (!(ok = over(&full[v.s], v.phase) && over(&b_p[at], p_phase[at]))) break;
                            p_phase[at] ^= 1u;
                            tc_fence_after();
                            if (elect_one()) {
                                values(0, at, v.s, j - 1 > begin, 0);
                                values(0, at, v.s, true, 1);
                                tc_commit(&b_o[(j - 1 - begin) & 1]);
                                tc_commit(&empty[v.s]);
                            }
                            v.go(2, stages);
                        }
                    } else {
                        bool has_k = false, has_v = false;
#pragma unroll
                        for (int w = 0; w < 2; ++w) {
                            const KeyRange r = rs[w];
                            const bool adds = j - 1 >= r.begin && j - 1 < r.end, takes = j >= r.begin && j < r.end;
                            if (adds) {
                                if (!(ok = (has_v || over(&full[v.s], v.phase)) && over(&b_h[w], p_phase[w]))) break;
                                has_v = true;
                                tc_fence_after();
                                if (elect_one()) values(w, w, v.s, j - 1 > r.begin, 0);
                                if (!(ok = over(&b_p[w], p_phase[w]))) break;
                                p_phase[w] ^= 1u;
                            }
                            if (takes) {
                                if (!(ok = has_k || over(&full[k.s], k.phase))) break;
                                has_k = true;
                            }
                            tc_fence_after();
                            if (elect_one()) {
                                if (adds) {
                                    values(w, w, v.s, true, 1);
                                    tc_commit(&b_o[w]);
                                }
                                if (w == 1 && j > begin) tc_commit(&empty[v.s]);
                                if (takes) {
                                    scores(w, w, k.s);
                                    tc_commit(&b_s[w]);
                                }
                                if (w == 1 && j < end) tc_commit(&empty[k.s]);
                            }
                        }
                        if (!ok) break;
                        if (j > begin) v.go(2, stages);
                        k.go(2, stages);
                    }
                }
                if (elect_one()) tc_commit(&b_done);
                __syncwarp();
            } else {
                begin_pass();
            }
            if (end_pass(stages)) break;
        }
    } else {
        if constexpr (kTiles == 2) asm volatile("setmaxnreg.inc.sync.aligned.u32 208;");
        for (int again = 0; again < 2; ++again) {
            const int stages = kMaxStages - again;     // the second time the last stage holds the notes on values that are not finite
            // ---- softmax: tile w, a row a thread ----
            const int w = warp >> 2, r = t & 127;
            const KeyRange rg = w ? r1 : r0;
            const int t0 = tok0 + w * tokens;                          // the tile's first token
            const auto token_of = [&](int row) { return row * a.inverse >> 12; };
            const bool live = r < tokens * g && t0 + token_of(r) < n;
            const int tok = min(t0 + min(token_of(r), tokens - 1), n - 1), hi = tok + 1, lo = a.window ? max(0, tok - a.window + 1) : 0;
            const int full_lo = a.window ? max(0, min(t0 + tokens, n) - a.window) : 0;   // keys from here to t0 are seen by all rows
            const uint32_t lanes = uint32_t(32 * (warp & 3)) << 16;
            // Rows cross between memory, where a row's pieces of 16 bytes go by lanes beside each other, and tensor memory, where a lane
            // has a row, through the warp's part of the shared memory (pieces turned by the row's number)
            constexpr int kPieces = HD / 8;            // of a row
            const unsigned q_at = saddr(qs), turn = q_at + (w * 4 + (warp & 3)) * 32 * kPieces * 16;
            const auto turn_at = [&](int row, int piece) { return turn + (row * kPieces + (piece ^ (row & 7))) * 16; };
            // The rows that a lane meets there, from the warp's first ones on, in a buffer of packed rows
            constexpr int kRowStep = 32 / kPieces, kEach = kPieces;
            const int step_t = kRowStep / g, step_h = kRowStep - step_t * g, tokens_here = min(tokens, n - t0);
            struct Walk {
                unsigned at;                           // bytes from the tile's first row on
                int token, head;
            };
            const auto walk = [&](unsigned ld) {
                int row = 32 * (warp & 3) + lane / kPieces;
                asm volatile("" : "+r"(row));          // (each walk is to be made where it is used, not all of its places kept in registers)
                const int token = token_of(row), head = row - token * g;
                return Walk{token * ld + head * HD * 2 + lane % kPieces * 16, token, head};
            };
            const auto walk_on = [&](Walk &x, unsigned ld) {
                x.at += step_t * ld + step_h * HD * 2, x.token += step_t, x.head += step_h;
                if (x.head >= g) x.at += ld - g * HD * 2, ++x.token, x.head -= g;
            };
            const int64_t first = row0 + min(t0, n - 1), head0 = h * g * HD * 2;   // (a tile without tokens reads a row that is there, and writes none)
            // Q, asked for before the CTA's threads meet; rows of tokens behind the sequence's last one are zeros
            {
                const uint8_t *from = a.q + first * a.ldq + head0;
                Walk x = walk(unsigned(a.ldq));
#pragma unroll
                for (int i = 0; i < kEach; ++i) {
                    const bool there = x.token < tokens_here;
                    const int row = i * kRowStep + lane / kPieces, ch = lane % kPieces, all = 32 * (warp & 3) + row;
                    const unsigned to = HD == 256 ? turn_at(row, ch) : q_at + (w * (HD / 64) + ch / 8) * 16384 + all * 128 + (((ch & 7) ^ (all & 7)) << 4);
                    cp_async16_or_zeros(to, from + (there ? x.at : 0u), there);
                    walk_on(x, unsigned(a.ldq));
                }
            }
            begin_pass();
            const uint32_t tmem = s_tmem, t_o = tmem + Sh::kO + w * HD + lanes;
            cp_async_wait_all();
            if constexpr (HD == 256) {
                __syncwarp();
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                    uint32_t v[32];
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const uint4 p = ld_shared(turn_at(lane, 8 * x + i));
                        v[4 * i] = p.x, v[4 * i + 1] = p.y, v[4 * i + 2] = p.z, v[4 * i + 3] = p.w;
                    }
                    tc_st32(tmem + kPromptQ + 32 * x + lanes, v);
                }
                tc_wait_st();
                tc_fence_before();
            } else {
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            }
            mbar_arrive(&b_q);

            // fp16 weights are held times 2^kShift; the maximum in use may fall behind by kBehind powers of two
            constexpr bool kBf16 = std::is_same<T, __nv_bfloat16>::value;
            constexpr float kShift = kBf16 ? 0.f : 3.f, kBehind = kBf16 ? 16.f : 12.f, kFar = 1024.f;
            const float c = a.scale_log2;
            float top = -INFINITY, sum = 0.f;      // the maximum in use and the weights' sum
            uint32_t seen[HD / 32];                // channels in which the row saw a value that is not finite
#pragma unroll
            for (int i = 0; i < HD / 32; ++i) seen[i] = 0;
            int met[2] = {0, 0};                   // meetings of both tiles' threads, of this one's
            bool ok = true;
            for (int j = rg.begin; j < rg.end; ++j) {
                const int it = j - rg.begin, at = kTiles == 1 ? (j & 1) : w;
                const int phase = kTiles == 1 ? (j - jb) >> 1 : it;
                // A wait names a phase by its parity: it must not be possible that the next but one has begun, and none may be left out.
                // With S held twice the sums of tile it - 1 may or may not be there, so they tick on two barriers in turn, of which one
                // goes on only after the tile's own P; those of the tile before (or before that) are there already and are ticked off
                constexpr int kAhead = kTiles == 1 ? 2 : 1;
                const auto added = [&](int i) {
                    return kTiles == 1 ? wait_for(&b_o[i & 1], unsigned(i >> 1) & 1u, &s_bad) : wait_for(&b_o[w], unsigned(i) & 1u, &s_bad);
                };
                ok = wait_for(&b_s[at], unsigned(phase) & 1u, &s_bad) && (it < kAhead || added(it - kAhead));
                if (!__all_sync(0xffffffffu, ok)) break;               // tcgen05.ld takes the whole warp
                tc_fence_after();
                uint32_t s[kKeys / 32][32];
                const uint32_t t_s = tmem + Sh::kS + at * Sh::kSPitch + lanes;
#pragma unroll
                for (int x = 0; x < kKeys / 32; ++x) tc_ld32_async(t_s + 32 * x, s[x]);
                tc_wait_ld();
#pragma unroll
                for (int x = 0; x < kKeys / 32; ++x) tc_tie32(s[x]);
                const int k0 = j * kKeys;
                if (k0 + kKeys > t0 + 1 || k0 < full_lo) {
#pragma unroll
                    for (int x = 0; x < kKeys / 32; ++x) {
                        const int up = min(max(hi - k0 - 32 * x, 0), 32), down = min(max(lo - k0 - 32 * x, 0), 32);
                        const uint32_t seen_by = (up == 32 ? 0xffffffffu : (1u << up) - 1u) & ~(down == 32 ? 0xffffffffu : (1u << down) - 1u);
#pragma unroll
                        for (int i = 0; i < 32; ++i)
                            if (!(seen_by >> i & 1u)) s[x][i] = __float_as_uint(-INFINITY);
                    }
                }
                float m[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                for (int x = 0; x < kKeys; x += 8)
#pragma unroll
                    for (int y = 0; y < 4; ++y)
                        m[y] = fmaxf(fmaxf(m[y], __uint_as_float(s[x / 32][x % 32 + y])), __uint_as_float(s[x / 32][x % 32 + y + 4]));
                const float best = fmaxf(fmaxf(m[0], m[1]), fmaxf(m[2], m[3]));
                // a row that has seen nothing yet has no sums that a new maximum would change
                const bool renew = (best - top) * c > kBehind, scale = renew && top != -INFINITY;
                float keep = 1.f;
                if (scale) keep = exp2_fast((top - best) * c);
                if (renew) top = best;
                if (__any_sync(0xffffffffu, scale)) {
                    if constexpr (kAhead == 2) {
                        ok = added(it - 1);
                        if (!__all_sync(0xffffffffu, ok)) break;
                        tc_fence_after();
                    }
#pragma unroll 1
                    for (int x = 0; x < HD; x += 32) {
                        uint32_t o[32];
                        tc_ld32(t_o + x, o);
#pragma unroll
                        for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * keep);
                        tc_st32(t_o + x, o);
                    }
                }
                // Where the maximum is so large that the rounding of its product with c is worth 2^-15 of a power of two and more (16 of them at
                // 2^28, which fp16 weights have no room for), it leaves the scores before they are scaled. (Always: packed prompts 269.6 us, 266.5 so;
                // where all scores are of that size, 294)
                const float base = top != -INFINITY && fabsf(top) * c > kFar ? top : 0.f;
                if (__any_sync(0xffffffffu, base != 0.f)) {
#pragma unroll
                    for (int x = 0; x < kKeys / 32; ++x)
#pragma unroll
                        for (int i = 0; i < 32; ++i) s[x][i] = __float_as_uint(__uint_as_float(s[x][i]) - base);
                }
                const float off = top == -INFINITY ? 0.f : kShift - (top - base) * c;
                const uint64_t c2 = pair(__float_as_uint(c), __float_as_uint(c)), off2 = pair(__float_as_uint(off), __float_as_uint(off));
                uint64_t add[4] = {0, 0, 0, 0};
#pragma unroll
                for (int x = 0; x < 2; ++x) {              // half of the keys: with two tiles their products need not wait for the others
                    uint32_t p[kKeys / 4];
#pragma unroll
                    for (int i = 0; i < kKeys / 4; ++i) {
                        const int k = x * (kKeys / 2) + 2 * i;
                        float p0, p1;
                        halves(fma2(pair(s[k / 32][k % 32], s[k / 32][k % 32 + 1]), c2, off2), p0, p1);
                        p0 = exp2_fast(p0), p1 = exp2_fast(p1);
                        add[i & 3] = add2(add[i & 3], pair(__float_as_uint(p0), __float_as_uint(p1)));
                        p[i] = pack2<T>(p0, p1);
                    }
                    if constexpr (kTiles == 2) {
                        tc_st32(t_s + 32 * x, p);
                        if (x == 0 && !again) {
                            tc_wait_st();
                            tc_fence_before();
                            mbar_arrive(&b_h[at]);
                        }
                    } else {
                        tc_st16(t_s + 16 * x, p);
                    }
                }
                float a0, a1;
                halves(add2(add2(add[0], add[1]), add2(add[2], add[3])), a0, a1);
                sum = sum * keep + (a0 + a1);
                if (again) {
                    // what is not finite leaves the tile of values, and each row notes what it saw of it
                    const bool both = kTiles == 2 && j >= r0.begin && j < r0.end && j >= r1.begin && j < r1.end;
                    const int who = both ? t : r, count = both ? 256 : 128, id = both ? 0 : 1 + w;
                    const int k = 2 * (j - jb) + 1, parts = count / kKeys, key = who / parts, part = who % parts;
                    uint32_t *notes = reinterpret_cast<uint32_t *>(ring + (kMaxStages - 1) * Sh::kStage) + id * kKeys * (HD / 32), *odd = s_odd[id];
                    const auto meet = [&] {
                        mbar_arrive(&b_meet[id]);
                        return __all_sync(0xffffffffu, wait_for(&b_meet[id], unsigned(met[id != 0]++) & 1u, &s_bad)) != 0;
                    };
                    ok = wait_for(&full[k % stages], unsigned(k / stages) & 1u, &s_bad);
                    if (!__all_sync(0xffffffffu, ok)) break;
                    if (!(ok = meet())) break;     // the notes of the tile before have been read
                    if (who < kKeys / 32) odd[who] = 0;
                    if (!(ok = meet())) break;
                    uint8_t *vt = ring + (k % stages) * Sh::kStage;
                    bool any = false;
                    for (int word = part * (HD / 32) / parts; word < (part + 1) * (HD / 32) / parts; ++word) {
                        uint32_t bits = 0;
                        for (int i = 0; i < 4; ++i) {
                            const int ch = word * 4 + i;               // 16-byte pieces of the key's channels
                            uint4 *p = reinterpret_cast<uint4 *>(vt + (ch / 8) * kKeys * 128 + key * 128 + (((ch & 7) ^ (key & 7)) << 4));
                            uint32_t v[4] = {p->x, p->y, p->z, p->w}, hit = 0;
                            for (int y = 0; y < 4; ++y) {
                                if (odd16<T>(v[y] & 0xFFFFu)) hit |= 1u << (2 * y), v[y] &= 0xFFFF0000u;
                                if (odd16<T>(v[y] >> 16)) hit |= 2u << (2 * y), v[y] &= 0xFFFFu;
                            }
                            if (hit) *p = make_uint4(v[0], v[1], v[2], v[3]);
                            bits |= hit << (8 * i);
                        }
                        notes[key * (HD / 32) + word] = bits;
                        any |= bits != 0;
                    }
                    if (any) atomicOr(&odd[key / 32], 1u << (key % 32));
                    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                    if (!(ok = meet())) break;
                    for (int x = 0; x < kKeys / 32; ++x)
                        for (uint32_t left = odd[x]; left; left &= left - 1) {
                            const int kr = 32 * x + __ffs(left) - 1;
                            if (k0 + kr >= lo && k0 + kr < hi)
#pragma unroll
                                for (int i = 0; i < HD / 32; ++i) seen[i] |= notes[kr * (HD / 32) + i];
                        }
                }
                tc_wait_st();
                tc_fence_before();
                if (kTiles == 2 && again) mbar_arrive(&b_h[at]);
                mbar_arrive(&b_p[at]);
            }
            // ---- the sums, divided and rounded ----
            const int last = rg.end - rg.begin - 1;
            if (last >= 0) {
                if (ok) ok = kTiles == 1 ? wait_for(&b_o[last & 1], unsigned(last >> 1) & 1u, &s_bad) : wait_for(&b_o[w], unsigned(last) & 1u, &s_bad);
                if (__all_sync(0xffffffffu, ok)) {
                    tc_fence_after();
                    const float part = 1.f / sum;
                    float odd = 0.f;                   // NaN where a sum is not finite
#pragma unroll
                    for (int x = 0; x < HD / 32; ++x) {
                        uint32_t o[32];
                        tc_ld32(t_o + 32 * x, o);
#pragma unroll
                        for (int i = 0; i < 32; ++i) odd = fmaf(__uint_as_float(o[i]), 0.f, odd);
                        if (again) {
#pragma unroll
                            for (int i = 0; i < 32; ++i)
                                if (seen[x] >> i & 1u) o[i] = 0x7FFFFFFFu;
                        }
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            uint32_t p[4];
#pragma unroll
                            for (int y = 0; y < 4; ++y) p[y] = pack2_out<T>(__uint_as_float(o[8 * i + 2 * y]) * part, __uint_as_float(o[8 * i + 2 * y + 1]) * part);
                            st_shared(turn_at(lane, 4 * x + i), make_uint4(p[0], p[1], p[2], p[3]));
                        }
                    }
                    __syncwarp();
                    uint8_t *rows = a.out + first * a.ldo + head0;
                    Walk to = walk(unsigned(a.ldo));
#pragma unroll
                    for (int half = 0; half < kEach; half += 8) {
                        uint4 v[8];
#pragma unroll
                        for (int i = 0; i < 8; ++i) v[i] = ld_shared(turn_at((half + i) * kRowStep + lane / kPieces, lane % kPieces));
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            if (to.token < tokens_here) *reinterpret_cast<uint4 *>(rows + to.at) = v[i];
                            walk_on(to, unsigned(a.ldo));
                        }
                    }
                    __syncwarp();
                    if (live && isnan(odd) && !isnan(sum)) s_again = 1;
                }
            }
            if (end_pass(stages)) break;
        }
    }
    if (warp == kTiles * 4 + 1)
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(s_tmem), "r"(512) : "memory");
}

// Rows [rows][n_kv][HD] of the type, ld elements apart, as boxes of 64 channels x 1 head x `keys` rows in the 128-byte
// swizzle; rows past the end read as zero.
bool rows_map(CUtensorMap *map, const dfl_paged &c, const void *p, int64_t ld, int rows, int keys) {
    const EncodeTiled enc = encoder();
    if (!enc) return false;
    const cuuint64_t dims[3] = {cuuint64_t(c.head_dim), cuuint64_t(c.n_kv), cuuint64_t(rows)};
    const cuuint64_t strides[2] = {cuuint64_t(c.head_dim) * 2, cuuint64_t(ld) * 2};
    const cuuint32_t box[3] = {64u, 1u, cuuint32_t(keys)}, estr[3] = {1u, 1u, 1u};
    return enc(map, c.type == DFL_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3, const_cast<void *>(p), dims, strides,
               box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <typename T, int HD>
int launch_prompt(const PagedAttnArgs &a, cudaStream_t s) {
    using Sh = PromptShape<HD>;
    const int dev = current_device();
    if (dev < 0) return DFL_E_CUDA;
    static bool done[kMaxDevices] = {};
    if (!done[dev]) {
        if (cudaFuncSetAttribute(k_prompt<T, HD>, cudaFuncAttributeMaxDynamicSharedMemorySize, Sh::kSmem) != cudaSuccess) return DFL_E_CUDA;
        done[dev] = true;
    }
    CUtensorMap tk, tv;
    if (!rows_map(&tk, a.c, a.k, a.ldk, a.total, Sh::kKeys) || !rows_map(&tv, a.c, a.v, a.ldv, a.total, Sh::kKeys)) return DFL_E_CUDA;
    const PromptArgs p{a.c, static_cast<const uint8_t *>(a.q), static_cast<uint8_t *>(a.out), a.ldq * 2, a.ldo * 2, a.group, a.inverse, a.total, a.window, a.cu,
                       a.scale_log2, a.stall};
    const int per = Sh::kTiles * (128 / a.group);                // tokens of an item
    const int64_t items = (int64_t)a.total / per + std::min(a.c.n_seq, a.total);
    if (items * a.c.n_kv > INT32_MAX) return DFL_E_UNSUPPORTED;
    return pg_launched(launch_pdl(k_prompt<T, HD>, dim3(unsigned(items * a.c.n_kv)), dim3(Sh::kThreads), Sh::kSmem, s, tk, tv, p));
}

}  // namespace

int launch_paged_prompt(const PagedAttnArgs &a, cudaStream_t s) {
    const int hd = a.c.head_dim;
    if (a.c.type == DFL_BF16)
        return hd == 64 ? launch_prompt<__nv_bfloat16, 64>(a, s) : hd == 128 ? launch_prompt<__nv_bfloat16, 128>(a, s) : launch_prompt<__nv_bfloat16, 256>(a, s);
    return hd == 64 ? launch_prompt<__half, 64>(a, s) : hd == 128 ? launch_prompt<__half, 128>(a, s) : launch_prompt<__half, 256>(a, s);
}

}  // namespace dfl
