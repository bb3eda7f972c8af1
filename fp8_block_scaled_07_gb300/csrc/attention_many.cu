// attention_many.cu -- attention over the paged 8-bit cache for requests with
// many rows of queries: prompts (attention.cuh).
//
// An item is 256 rows (queries x heads that share a cache head) of a request:
// two tiles of 128 rows, which share the stream of K and V tiles of 128 tokens
// and go through it in steps of 64 tokens:
//   S = Q K^T  (rows on the 128-row side, Q and K e4m3 in shared memory),
//   O += P V   (P fp16 in tensor memory, V fp16 in shared memory, MN-major).
// CTAs take items from a counter, a request's longest first.
//
// K's codes are read by the tensor core as they are; q is split, and both
// halves go to one accumulator, so lo has no factor of its own: it is e5m2,
// whose 3 significant bits still hold the rest of a bf16 (an integer of at
// most 8 in units of its last bit) exactly.
// V's codes become fp16 (exactly) on their way: a warpgroup converts a tile
// that 256 rows then use, and a probability costs one conversion instead of a
// split (hi + lo in e4m3: seven instructions for two probabilities, and the
// softmax took 4700 cycles of a tile's 6700; the products take the same tensor
// time either way).  It converts two rows of a lane at a time: more at once
// hold up the tensor core's reads of shared memory (1 / 2 / 4 / 8 rows: 558 /
// 543 / 556 / 591 us for a prompt of 4096 with 128 heads of 192/128).
//
// A step's S has a buffer of its own (two of 64 columns a row tile, P over S),
// so the softmax of one step runs beside the products of the others.  With
// steps of 128 and one buffer the chain S, softmax, P V was serial: 4600
// cycles a tile; the price of 64 is 48 cycles for 32 of K's bytes instead of
// 32 (N = 64 against 128, shared memory's rate).
// A thread of the softmax has a whole row: with two to a row the exchange of
// the maximum took 230 cycles of a step's 1000.  P is written over S.
// Probabilities are 2^(x - M + 8) in fp16, and M follows the true maximum once
// that has passed it by 2^7: after a request's first tiles O is hardly ever
// rescaled.  (P made with the M there is while the maximum is still looked
// for, and made again when that fails: 600 us against 555 us.)
// Each row tile has an issuing warp of its own, and that warp runs as a whole
// (see warp_mma_e4m3).
//
// 128 tokens for 256 rows take 1.73 us with dk = 128 (1.29 us is what the
// products take alone, 2480 cycles) and 2.01 us with dk = 192 (1.73 us); a
// call has some 21 us more for its start, first loads and last results.
//   prompt of 4096, 128 heads of 192/128: 572 us, 1201 TFLOP/s (tensor pipe 56% busy)
//   chunks of 2048, 1437 and 1552 with a past, 32 heads on 8 of 128: 201 us, 1040 TFLOP/s
//   (640 items on 152 SMs: 9% of the time is the last round's)
// (in a long run of calls; under a profiler, cold, the prompt takes 538 us)
#include "attention.cuh"

namespace fp8bs {
namespace {

// warps: 0 producer, 1-2 MMA (a row tile each), 3 scales, 4-11 softmax, 12-15 V's conversion
constexpr int kThreads = 512;
// registers of a thread: of the warpgroups 0 and 3, and of the softmax's two
constexpr int kRegsLow = 96, kRegsHigh = 160, kRegsLaunch = 128;
static_assert(2 * kRegsLow + 2 * kRegsHigh == 4 * kRegsLaunch, "what some give, others take");
constexpr int kItems = 4;           // items announced ahead
constexpr int kNotes = 8;           // items whose notes of NaNs in V are kept: the last one's are read once the next has begun
static_assert(kNotes > kItems + 1, "the results of an item are written before the item kItems + 1 on is announced");
constexpr int kNanBits = 9;         // tokens of an item that only some rows see, and those to the end of their tile: 383 at most
constexpr float kPBits = 8.0f, kSlack = 7.0f;   // 2^15 < 65504
constexpr uint32_t kOdd = 1u << 31;             // of a tile: some page's scale of K is not at least kLeast
constexpr float kLeast = 0x1p-60f;              // (two factors of so much have a product above 0)

template <int DK, int DV>
struct Many {
    static constexpr bool kWide = DK >= 128, kHalf = DK % 128 == 64;
    static constexpr int kKBytes = 128 * DK, kVBytes = 128 * DV, kFBytes = 2 * kVBytes;
    static constexpr int kQTile = 128 * DK;                    // hi or lo of 128 rows
    static constexpr int kSK = DK == 192 ? 2 : 3;              // stages of K, of V's codes, of V in fp16
    static constexpr int kSV = 2;
    static constexpr int kSF = DK == 192 ? 1 : 2;
    static constexpr int kMisc = kManyB * 20 + 16 + kRing * 8 * 16 + kRing * 4 + 256 * 4 + kItems * 48 + kNotes * (DV + 2) * 4 + 1024;
    static constexpr int kSmem = 1024 + 4 * kQTile + kSK * kKBytes + kSV * kVBytes + kSF * kFBytes + kMisc;
    static_assert(kSmem <= 227 * 1024, "shared memory");
};

// What a role has to know of an item, as the producer announces it.
struct ManyItem {
    int nmax;            // tiles of K and V (-1: no more items)
    int steps[2];        // of 64 tokens, of each row tile
    int b, h, n, len, first, rows, row0, pad[2];
};

// The warp that issues the products runs as a whole, and one elected thread
// issues: then addresses and descriptors are the warp's, not a thread's, and an
// instruction costs no copies to uniform registers (issued by a branch of one
// thread, eight products of 48 cycles each took 1000 cycles to issue).
// N products of e4m3 (K 32), their operands 32 bytes further on each; the
// first one starts the sum unless `add`.
template <int N>
__device__ __forceinline__ void warp_mma_e4m3(uint32_t d_tmem, uint64_t a, uint64_t b, uint32_t idesc, uint32_t add) {
    static_assert(N == 4 || N == 2, "products of one call");
    if constexpr (N == 4)
        asm volatile(
            "{\n\t.reg .pred p, e;\n\t"
            "setp.ne.b32 p, %4, 0;\n\t"
            "elect.sync _|e, 0xFFFFFFFF;\n\t"
            "@e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t"
            "@e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %5, %6, %3, 1;\n\t"
            "@e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %7, %8, %3, 1;\n\t"
            "@e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %9, %10, %3, 1;\n\t}" ::"r"(d_tmem),
            "l"(a), "l"(b), "r"(idesc), "r"(add), "l"(a + 2), "l"(b + 2), "l"(a + 4), "l"(b + 4), "l"(a + 6), "l"(b + 6)
            : "memory");
    else
        asm volatile(
            "{\n\t.reg .pred p, e;\n\t"
            "setp.ne.b32 p, %4, 0;\n\t"
            "elect.sync _|e, 0xFFFFFFFF;\n\t"
            "@e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t"
            "@e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %5, %6, %3, 1;\n\t}" ::"r"(d_tmem),
            "l"(a), "l"(b), "r"(idesc), "r"(add), "l"(a + 2), "l"(b + 2)
            : "memory");
}
// Four products of P (fp16 in tensor memory, 16 tokens each: 8 columns) and V
// (2048 bytes each).
__device__ __forceinline__ void warp_mma_pv(uint32_t d_tmem, uint32_t p_tmem, uint64_t v, uint32_t idesc, uint32_t add) {
    asm volatile(
        "{\n\t.reg .pred p, e;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "elect.sync _|e, 0xFFFFFFFF;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%5], %6, %3, 1;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%7], %8, %3, 1;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%9], %10, %3, 1;\n\t}" ::"r"(d_tmem),
        "r"(p_tmem), "l"(v), "r"(idesc), "r"(add), "r"(p_tmem + 8), "l"(v + 128), "r"(p_tmem + 16), "l"(v + 256),
        "r"(p_tmem + 24), "l"(v + 384)
        : "memory");
}
__device__ __forceinline__ void warp_commit(uint64_t* bar) {
    asm volatile(
        "{\n\t.reg .pred e;\n\t"
        "elect.sync _|e, 0xFFFFFFFF;\n\t"
        "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(smem_u32(bar))
        : "memory");
}

// Instruction descriptor: D f32, A and B fp16, A K-major, B MN-major.
__host__ __device__ constexpr uint32_t idesc_f16_mn(int M, int N) {
    return (1u << 4) | (1u << 16) | (static_cast<uint32_t>(N >> 3) << 17) | (static_cast<uint32_t>(M >> 4) << 24);
}

// V in fp16, MN-major: panels of 64 values (128-byte rows, one per token,
// 128-byte swizzle), 16 KB apart; groups of 8 tokens every 1024 bytes.
__device__ __forceinline__ uint64_t smem_desc_v16(uint32_t saddr) {
    uint64_t d = 0;
    d |= static_cast<uint64_t>((saddr & 0x3FFFFu) >> 4);
    d |= static_cast<uint64_t>(16384 >> 4) << 16;
    d |= static_cast<uint64_t>(1024 >> 4) << 32;
    d |= static_cast<uint64_t>(1) << 46;
    d |= static_cast<uint64_t>(2) << 61;
    return d;
}

__device__ __forceinline__ void tmem_st16u(uint32_t taddr, const uint32_t* v) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
        "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]),
        "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
        : "memory");
}

__device__ __forceinline__ uint32_t f32x2_to_f16x2(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint32_t two) {
    uint32_t r;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(static_cast<uint16_t>(two)));
    return r;
}
// 32 bytes (32-byte aligned) to global memory.
__device__ __forceinline__ void st_global_32(void* dst, const uint32_t (&w)[8]) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(dst), "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]),
                 "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                 : "memory");
}
__device__ __forceinline__ float max3(float a, float b, float c) {
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}

template <int DK, int DV>
__global__ void __launch_bounds__(kThreads, 1)
    attn_many_kernel(const __grid_constant__ CUtensorMap tm_k0, const __grid_constant__ CUtensorMap tm_k1,
                     const __grid_constant__ CUtensorMap tm_v, const AttnParams p) {
    using F = Many<DK, DV>;
    constexpr int SK = F::kSK, SV = F::kSV, SF = F::kSF;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    uint8_t* sK = smem;
    uint8_t* sV = sK + SK * F::kKBytes;              // codes
    uint8_t* sF = sV + SV * F::kVBytes;              // fp16
    uint8_t* sQ = sF + SF * F::kFBytes;              // [tile][hi, lo]
    ManyItem* s_item = reinterpret_cast<ManyItem*>(sQ + 4 * F::kQTile);     // [kItems]
    long long* s_cum = reinterpret_cast<long long*>(s_item + kItems);       // [kManyB + 1] items before each request
    float4* s_page = reinterpret_cast<float4*>(s_cum + kManyB + 2);         // [kRing][8] K's scale, log2 of V's, 1 / V's
    int* s_len = reinterpret_cast<int*>(s_page + kRing * 8);
    int* s_n = s_len + kManyB;
    int* s_first = s_n + kManyB;
    uint32_t* s_dead = reinterpret_cast<uint32_t*>(s_first + kManyB);       // [kRing] pages that are left out, as bits; kOdd
    float* s_qf = reinterpret_cast<float*>(s_dead + kRing);                 // [256] factor of a row's S
    uint32_t* s_nan = reinterpret_cast<uint32_t*>(s_qf + 256);              // [kNotes][DV] NaNs in V (nan_key), as offsets from
    int* s_base = reinterpret_cast<int*>(s_nan + kNotes * DV);              // [kNotes] the tokens that all of the item's rows see
    uint32_t* s_nans = reinterpret_cast<uint32_t*>(s_base + kNotes);        // [kNotes] the last item with such a NaN, plus 1
    uint64_t* bars = reinterpret_cast<uint64_t*>(s_nans + kNotes);
    uint64_t* kfull = bars;
    uint64_t* kempty = kfull + SK;
    uint64_t* vfull = kempty + SK;
    uint64_t* vempty = vfull + SV;     // (4 converting warps)
    uint64_t* ffull = vempty + SV;     // [SF][2 halves of 64 tokens] (2 converting warps)
    uint64_t* fempty = ffull + 2 * SF;
    uint64_t* sfull = fempty + 2 * SF; // [2 tiles][2 buffers]: S of the tile's rows is in TMEM
    uint64_t* pfull = sfull + 4;       // [2][2]: P is (4 warps)
    uint64_t* odone = pfull + 4;       // [2][2]: P V has been added to O
    uint64_t* qfull = odone + 4;       // 2: Q is in shared memory (4 warps)
    uint64_t* qread = qfull + 2;       // 2: its factors have been read (4 warps)
    uint64_t* cfull = qread + 2;       // kRing: page constants
    uint64_t* cempty = cfull + kRing;  // (8 softmax warps, 4 converting)
    uint64_t* ifull = cempty + kRing;  // kItems
    uint64_t* iempty = ifull + kItems; // (2 MMA, 1 scales, 4 converting, 8 softmax)
    uint64_t* mma_done = iempty + kItems;
    uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(mma_done + 1);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_holder + 1);
    __shared__ long long s_scan[kThreads / 32];
    static_assert((2 * SK + 2 * SV + 4 * SF + 16 + 2 * kRing + 2 * kItems + 1) * 8 + 8 <= 1024, "barrier block");

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    for (int i = threadIdx.x; i < kNotes * (DV + 2); i += kThreads) s_nan[i] = 0;
    if (threadIdx.x == 0) {
        for (int i = 0; i < SK; ++i) {
            mbar_init(&kfull[i], 1);
            mbar_init(&kempty[i], 2);
        }
        for (int i = 0; i < SV; ++i) {
            mbar_init(&vfull[i], 1);
            mbar_init(&vempty[i], 4);
        }
        for (int i = 0; i < 2 * SF; ++i) {
            mbar_init(&ffull[i], 2);
            mbar_init(&fempty[i], 2);
        }
        for (int i = 0; i < 4; ++i) {
            mbar_init(&sfull[i], 1);
            mbar_init(&pfull[i], 4);
            mbar_init(&odone[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&qfull[i], 4);
            mbar_init(&qread[i], 4);
        }
        for (int i = 0; i < kRing; ++i) {
            mbar_init(&cfull[i], 1);
            mbar_init(&cempty[i], 12);
        }
        for (int i = 0; i < kItems; ++i) {
            mbar_init(&ifull[i], 1);
            mbar_init(&iempty[i], 15);
        }
        mbar_init(mma_done, 2);
        *abort_flag = 0;
        fence_mbar_init();
        tma_prefetch_desc(&tm_k0);
        tma_prefetch_desc(&tm_k1);
        tma_prefetch_desc(&tm_v);
    }
    if (warp == 1) {
        tmem_alloc(tmem_holder, 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_holder;
    griddep_launch_dependents();
    griddep_wait();

    const int cap = p.width << p.bs_log2;
    {   // items of each request, as a running sum
        const int b = threadIdx.x;
        static_assert(kManyB <= kThreads, "a thread per request");
        long long mine = 0;
        if (b < p.B) {
            const int len = max(0, min(p.lens[b], cap)), first = p.offsets[b], n = p.offsets[b + 1] - first;
            const int64_t rows = min(static_cast<int64_t>(n), p.T - first) * p.G;   // (q may end before the request)
            s_len[b] = len;
            s_n[b] = n;
            s_first[b] = first;
            if (len > 0 && first >= 0 && rows > p.few_rows && rows < (1LL << 31) - 512) mine = (rows + 255) / 256 * p.Hkv;
        }
        long long inc = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long up = __shfl_up_sync(0xFFFFFFFFu, inc, o);
            if (lane >= o) inc += up;
        }
        if (lane == 31) s_scan[warp] = inc;
        __syncthreads();
        long long run = inc - mine;
        for (int w = 0; w < warp; ++w) run += s_scan[w];
        if (b < p.B) s_cum[b] = run;
        if (b == p.B - 1) s_cum[p.B] = run + mine;
        __syncthreads();
    }
    const int pages_per_tile = 128 >> p.bs_log2, bs = 1 << p.bs_log2;
    // tokens that the query of row r sees
    auto limit = [&](const ManyItem& m, int r) { return max(0, min(m.len, m.len - m.n + r / p.G + 1)); };
    // The k-th item of this CTA; false: there is none, or the wait gave up.
    auto item_of = [&](int k, ManyItem& m) {
        if (!mbar_wait(&ifull[k % kItems], (k / kItems) & 1, abort_flag)) return false;
        m = s_item[k % kItems];
        return m.nmax >= 0;
    };
    auto page_of = [&](const ManyItem& m, int tile) {
        const int idx = tile * pages_per_tile + lane;
        const bool on = lane < pages_per_tile && (idx << p.bs_log2) < m.len;
        return on ? p.tables[static_cast<int64_t>(m.b) * p.width + idx] : -1;
    };

    // whole warpgroups change their register budgets: 0 and 3 give, 1 and 2 take
    if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsLow));
    if (warp == 0) {
        // ------------------------------------------------ producer: items from the counter, their tiles by TMA
        // (lane i loads page i of a tile)
        const long long total = s_cum[p.B];
        int g = 0;
        bool ok = true;
        long long idx = blockIdx.x;
        for (int k = 0; ok; ++k) {
            ManyItem m{};
            m.nmax = -1;
            int ticket = 0;
            if (idx < total) {
                if (lane == 0) ticket = atomicAdd(p.next, 1);   // the item after this one
                int l = 0, r = p.B;
                while (r - l > 1) {
                    const int mid = (l + r) >> 1;
                    if (s_cum[mid] <= idx) l = mid; else r = mid;
                }
                m.b = l;
                m.len = s_len[l];
                m.n = s_n[l];
                m.first = s_first[l];
                m.rows = static_cast<int>(min(static_cast<int64_t>(m.n), p.T - m.first)) * p.G;
                const int rem = static_cast<int>(idx - s_cum[l]), at = rem / p.Hkv;
                m.h = rem - at * p.Hkv;
                m.row0 = ((m.rows + 255) / 256 - 1 - at) * 256;   // longest first
                m.nmax = 0;
#pragma unroll
                for (int t = 0; t < 2; ++t) {
                    const int r0 = m.row0 + t * 128, r1 = min(m.rows, r0 + 128);
                    m.steps[t] = r1 > r0 ? (limit(m, r1 - 1) + 63) >> 6 : 0;
                    m.nmax = max(m.nmax, (m.steps[t] + 1) >> 1);
                }
            }
            ok = __all_sync(0xFFFFFFFFu, mbar_wait(&iempty[k % kItems], ((k / kItems) & 1) ^ 1, abort_flag)) != 0;
            if (!ok) break;
            if (lane == 0) {
                s_item[k % kItems] = m;
                mbar_arrive(&ifull[k % kItems]);
            }
            __syncwarp();
            if (m.nmax < 0) break;
            // the queries on their way to L2
            for (int r = lane; r < min(256, m.rows - m.row0); r += 32) {
                const int rr = m.row0 + r, j = rr / p.G;
                const uint16_t* q = p.q + (m.first + static_cast<int64_t>(j)) * p.q_ts + (m.h * p.G + rr - j * p.G) * p.q_hs;
#pragma unroll
                for (int c = 0; c < DK; c += 64) asm volatile("prefetch.global.L2 [%0];" ::"l"(q + c));
            }
            int page = page_of(m, 0);
            for (int i = 0; i < m.nmax; ++i, ++g) {
                const int next_page = i + 1 < m.nmax ? page_of(m, i + 1) : -1;
                const int np = min(pages_per_tile, (m.len - i * 128 + bs - 1) >> p.bs_log2);
                {
                    const int st = g % SK;
                    uint8_t* kt = sK + st * F::kKBytes;
                    ok = __all_sync(0xFFFFFFFFu, mbar_wait(&kempty[st], ((g / SK) & 1) ^ 1, abort_flag)) != 0;
                    if (!ok) break;
                    if (lane == 0) mbar_arrive_expect_tx(&kfull[st], static_cast<uint32_t>(np * bs * DK));
                    __syncwarp();
                    if (lane < np) {
                        if constexpr (F::kWide) tma_load_page(kt + lane * bs * 128, &tm_k0, &kfull[st], 0, m.h * bs, page);
                        if constexpr (F::kHalf)
                            tma_load_page(kt + (F::kWide ? 128 * 128 : 0) + lane * bs * 64, &tm_k1, &kfull[st],
                                          F::kWide ? 128 : 0, m.h * bs, page);
                    }
                }
                {
                    const int st = g % SV;
                    ok = __all_sync(0xFFFFFFFFu, mbar_wait(&vempty[st], ((g / SV) & 1) ^ 1, abort_flag)) != 0;
                    const bool skip = p.debug_skip != 0 && g == 0;
                    if (lane == 0 && !skip) mbar_arrive_expect_tx(&vfull[st], static_cast<uint32_t>(np * bs * DV));
                    __syncwarp();
                    if (lane < np && !skip)
                        tma_load_page(sV + st * F::kVBytes + lane * bs * DV, &tm_v, &vfull[st], 0, m.h * bs, page);
                }
                page = next_page;
                if (!ok) {   // (both of the tile's loads are on their way)
                    ++g;
                    break;
                }
            }
            ticket = __shfl_sync(0xFFFFFFFFu, ticket, 0);
            idx = static_cast<long long>(gridDim.x) + ticket;
            // every CTA that had an item asks once in vain; the last to ask leaves the counter as it was found
            if (lane == 0 && ticket == total - 1) *p.next = 0;
        }
        if (!ok) attn_abort(abort_flag);
        const volatile int never = 0;   // every load issued must land before the CTA may exit
        for (int st = 0; st < SK && st < g; ++st) {
            const int uses = g / SK + (st < g % SK ? 1 : 0);
            if (!mbar_wait(&kfull[st], (uses - 1) & 1, &never)) attn_abort(abort_flag);
        }
        for (int st = 0; st < SV && st < g; ++st) {
            const int uses = g / SV + (st < g % SV ? 1 : 0);
            if (!mbar_wait(&vfull[st], (uses - 1) & 1, &never)) attn_abort(abort_flag);
        }
    } else if (warp == 1 || warp == 2) {
        // ------------------------------------------------ MMA issuers, one for each row tile
        // (one warp for both did not keep up: 650 cycles to issue a step's twelve products
        // beside four busy warps, which take the tensor core 620)
        constexpr uint32_t id_hi = idesc_e4m3_f32(128, 64);
        constexpr uint32_t id_lo = idesc_e4m3_f32(128, 64) | (1u << 7);    // A e5m2
        constexpr uint32_t id_o = idesc_f16_mn(128, DV);
        bool ok = true;
        ManyItem m;
        // A wait that gave up is looked at once a tile: the products issued meanwhile read and write what they always do.
        auto wait = [&](uint64_t* bar, int phase) {
            ok = mbar_wait(bar, phase, abort_flag) && ok;
            __syncwarp();
        };
        auto same = [](uint32_t x) { return __reduce_or_sync(0xFFFFFFFFu, x); };   // (known to the compiler as the warp's)
        const uint32_t t = same(warp - 1);
        const uint32_t dS = same(tmem) + t * 128, dO = same(tmem) + 256 + t * DV;
        const uint32_t q0 = same(smem_u32(sQ)) + t * 2 * F::kQTile, k0 = same(smem_u32(sK)), f0 = same(smem_u32(sF));
        int kst = 0, kph = 0, fst = 0, fph = 0, qph = 0, ph0 = 0, ph1 = 0;   // stages; phases of their barriers, of Q's and of P's
        // S of 64 tokens (half hv of stage kst) into buffer hv
        auto qk = [&](int hv) {
            const uint32_t d = dS + hv * 64, k = k0 + kst * F::kKBytes;
#pragma unroll
            for (int part = 0; part < 2; ++part) {
                const uint32_t q = q0 + part * F::kQTile;
                const uint32_t id = part == 0 ? id_hi : id_lo;
                if constexpr (F::kWide)
                    warp_mma_e4m3<4>(d, smem_desc_sw128(q), smem_desc_sw128(k + hv * 64 * 128), id, part);
                if constexpr (F::kHalf)
                    warp_mma_e4m3<2>(d, smem_desc_sw64(q + (F::kWide ? 128 * 128 : 0)),
                                     smem_desc_sw64(k + (F::kWide ? 128 * 128 : 0) + hv * 64 * 64), id, part || F::kWide ? 1u : 0u);
            }
            warp_commit(&sfull[t * 2 + hv]);
        };
        auto k_done = [&]() {
            warp_commit(&kempty[kst]);
            if (++kst == SK) {
                kst = 0;
                kph ^= 1;
            }
        };
        for (int k = 0; __all_sync(0xFFFFFFFFu, ok && item_of(k, m)); ++k) {
            __syncwarp();
            if (lane == 0) mbar_arrive(&iempty[k % kItems]);
            __syncwarp();
            const int steps = same(t ? m.steps[1] : m.steps[0]), nmax = same(m.nmax);
            if (nmax == 0) continue;
            wait(&kfull[kst], kph);
            if (steps > 0) {
                wait(&qfull[t], qph);
                qph ^= 1;
                tc_fence_after();
                qk(0);
                if (steps > 1) qk(1);
            }
            k_done();
            // (both warps wait for every tile and half, used or not, and release it)
            for (int i = 0; i < nmax; ++i) {
                if (!__all_sync(0xFFFFFFFFu, ok)) break;
                const bool more = i + 1 < nmax;
                if (more) wait(&kfull[kst], kph);
#pragma unroll
                for (int hv = 0; hv < 2; ++hv) {
                    const int step = 2 * i + hv;
                    wait(&ffull[fst * 2 + hv], fph);
                    if (step < steps) {
                        wait(&pfull[t * 2 + hv], hv ? ph1 : ph0);
                        if (hv) ph1 ^= 1; else ph0 ^= 1;
                        tc_fence_after();
                        warp_mma_pv(dO, dS + hv * 64, smem_desc_v16(f0 + fst * F::kFBytes) + hv * (64 * 128 >> 4), id_o, step);
                        warp_commit(&odone[t * 2 + hv]);
                    }
                    warp_commit(&fempty[fst * 2 + hv]);
                    if (step + 2 < steps) qk(hv);
                }
                if (more) k_done();
                if (++fst == SF) {
                    fst = 0;
                    fph ^= 1;
                }
            }
        }
        ok = __all_sync(0xFFFFFFFFu, ok) != 0;
        if (!ok) attn_abort(abort_flag);
        warp_commit(mma_done);
        const volatile int never = 0;
        if (!mbar_wait(mma_done, 0, &never)) attn_abort(abort_flag);
    } else {
        // ------------------------------------------------ scales of the tiles' pages, fetched two tiles ahead
        int g = 0;
        bool ok = true;
        ManyItem m;
        for (int k = 0; __all_sync(0xFFFFFFFFu, ok && item_of(k, m)); ++k) {
            __syncwarp();
            if (lane == 0) mbar_arrive(&iempty[k % kItems]);
            float ks = 0.0f, vs = 0.0f, ks1 = 0.0f, vs1 = 0.0f;   // of the next tile to write, and of the one after
            auto scales_of = [&](int page, float& a, float& b) {
                const bool on = page >= 0 && page < p.n_pages;
                const int64_t at = static_cast<int64_t>(page) * p.Hkv + m.h;
                a = on ? __ldg(p.k_scale + at) : 0.0f;
                b = on ? __ldg(p.v_scale + at) : 0.0f;
            };
            const int all_see = limit(m, m.row0), note = k % kNotes;
            if (m.nmax > 0) scales_of(page_of(m, 0), ks, vs);
            if (m.nmax > 1) scales_of(page_of(m, 1), ks1, vs1);
            int page2 = m.nmax > 2 ? page_of(m, 2) : -1;
            for (int i = 0; i < m.nmax; ++i, ++g) {
                const int slot = g % kRing;
                ok = __all_sync(0xFFFFFFFFu, mbar_wait(&cempty[slot], ((g / kRing) & 1) ^ 1, abort_flag)) != 0;
                if (!ok) break;
                const bool on = is_scale(vs);
                const bool there = lane < pages_per_tile && i * 128 + lane * bs < m.len;
                uint32_t dead = __ballot_sync(0xFFFFFFFFu, there && !on);
                if (__any_sync(0xFFFFFFFFu, there && on && !(ks >= kLeast))) dead |= kOdd;
                if (i * 128 + 128 > all_see) {
                    // NaNs in V of tokens that only some of the item's rows see: taken out and noted (note_nans) before
                    // the conversion, which waits for these constants.  Here, in the codes, they cost 0 to 2% of a
                    // prompt's time; looked for by the warps that convert, 3 to 7%.
                    // (The stage's tile before it must be done with first: a phase is told from the next, not from the
                    // one after that.)
                    const int st = g % SV, was = g - SV;
                    ok = was < 0 || mbar_wait(&cempty[was % kRing], (was / kRing) & 1, abort_flag);
                    ok = __all_sync(0xFFFFFFFFu, ok && mbar_wait(&vfull[st], (g / SV) & 1, abort_flag)) != 0;
                    if (!ok) break;
                    uint8_t* v = sV + st * F::kVBytes;
                    constexpr int kCh = DV / 16;   // 16 codes each
#pragma unroll 1
                    for (int x0 = lane; x0 < 128 * kCh; x0 += 128) {
                        uint32_t nans = 0;
#pragma unroll
                        for (int u = 0; u < 4; ++u) nans |= e4m3_nans(*reinterpret_cast<const uint4*>(v + (x0 + u * 32) * 16));
                        if (nans == 0) continue;
#pragma unroll 1
                        for (int x = x0; x < x0 + 128; x += 32) {
                            const int r = x / kCh, c = (x % kCh) ^ (DV == 128 ? r & 7 : (r >> 1) & 3), tok = i * 128 + r;
                            uint4* at = reinterpret_cast<uint4*>(v + x * 16);
                            const uint4 codes = *at;
                            if (tok < all_see || tok >= m.len || ((dead >> (r >> p.bs_log2)) & 1) || e4m3_nans(codes) == 0) continue;
                            *at = without_nans(codes);
                            note_nans(codes, s_nan + note * DV + c * 16, nan_key<kNanBits>(k + 1, tok - all_see));
                            s_base[note] = all_see;
                            s_nans[note] = k + 1;
                        }
                    }
                    fence_proxy_async_smem();
                }
                if (lane < 8) s_page[slot * 8 + lane] = on ? make_float4(ks, log2f(vs), 1.0f / vs, 0.0f) : make_float4(1.0f, 0.0f, 0.0f, 0.0f);
                if (lane == 0) s_dead[slot] = dead;
                __syncwarp();
                if (lane == 0) mbar_arrive(&cfull[slot]);
                ks = ks1;
                vs = vs1;
                if (i + 2 < m.nmax) scales_of(page2, ks1, vs1);
                if (i + 3 < m.nmax) page2 = page_of(m, i + 3);
            }
        }
        if (!ok) attn_abort(abort_flag);
    }
    } else if (warp >= 12) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsLow));
        // ------------------------------------------------ V to fp16: each warp 32 tokens of a tile
        // A token that is not there becomes zeros: its codes may be anything, a NaN too.
        const int part = warp - 12, hv = part >> 1;
        constexpr int kChunks = DV / 16;              // 16 codes, 32 bytes of fp16
        constexpr int kIter = 32 * kChunks / 32;
        // Chunk and row of a lane in step u.  A quarter-warp reads 8 chunks of
        // 16 bytes and writes 8 twice, all in different banks: dv = 128: four
        // chunks of the rows r and r ^ 5 (the swizzles differ in bit 2 for the
        // reads, in bit 0 for the writes); dv = 64: of two neighbouring rows.
        const int c = DV == 128 ? (lane & 3) + ((lane >> 4) & 1) * 4 : lane & 3;
        auto row_of = [&](int u) {
            if constexpr (DV == 128)
                return part * 32 + (u >> 1) * 8 + ((((u & 1) * 2 + ((lane >> 3) & 1))) ^ (((lane >> 2) & 1) * 5));
            else
                return part * 32 + u * 8 + (lane >> 2);
        };
        int g = 0;
        bool ok = true;
        ManyItem m;
        for (int k = 0; ok && item_of(k, m); ++k) {
            __syncwarp();
            if (lane == 0) mbar_arrive(&iempty[k % kItems]);
            for (int i = 0; i < m.nmax && ok; ++i, ++g) {
                const int slot = g % kRing, st = g % SV, sf = g % SF;
                ok = ok && mbar_wait(&cfull[slot], (g / kRing) & 1, abort_flag) &&
                     mbar_wait(&vfull[st], (g / SV) & 1, abort_flag) &&
                     mbar_wait(&fempty[sf * 2 + hv], ((g / SF) & 1) ^ 1, abort_flag);
                ok = __all_sync(0xFFFFFFFFu, ok) != 0;
                if (!ok) break;
                const uint32_t dead = s_dead[slot];
                const bool whole = dead == 0 && i * 128 + 128 <= m.len;
                const uint8_t* src = sV + st * F::kVBytes;
                uint8_t* dst = sF + sf * F::kFBytes;
                constexpr int kFly = 2;   // rows' chunks in flight together
#pragma unroll 1
                for (int k0 = 0; k0 < kIter; k0 += kFly) {
                    uint4 v[kFly];
#pragma unroll
                    for (int u = 0; u < kFly; ++u) {
                        const int r = row_of(k0 + u);
                        v[u] = DV == 128 ? *reinterpret_cast<const uint4*>(src + r * 128 + ((c ^ (r & 7)) << 4))
                                         : *reinterpret_cast<const uint4*>(src + r * 64 + ((c ^ ((r >> 1) & 3)) << 4));
                    }
                    if (!whole) {
#pragma unroll
                        for (int u = 0; u < kFly; ++u) {
                            const int r = row_of(k0 + u);
                            if (i * 128 + r >= m.len || ((dead >> (r >> p.bs_log2)) & 1)) v[u] = make_uint4(0, 0, 0, 0);
                        }
                    }
#pragma unroll
                    for (int u = 0; u < kFly; ++u) {
                        const int r = row_of(k0 + u);
                        const uint4 a = make_uint4(e4m3x2_to_f16x2(v[u].x), e4m3x2_to_f16x2(v[u].x >> 16),
                                                   e4m3x2_to_f16x2(v[u].y), e4m3x2_to_f16x2(v[u].y >> 16));
                        const uint4 b = make_uint4(e4m3x2_to_f16x2(v[u].z), e4m3x2_to_f16x2(v[u].z >> 16),
                                                   e4m3x2_to_f16x2(v[u].w), e4m3x2_to_f16x2(v[u].w >> 16));
                        const int j = (c & 3) * 2;
                        uint8_t* row = dst + (c >> 2) * 16384 + r * 128;
                        *reinterpret_cast<uint4*>(row + ((j ^ (r & 7)) << 4)) = a;
                        *reinterpret_cast<uint4*>(row + (((j + 1) ^ (r & 7)) << 4)) = b;
                    }
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(&ffull[sf * 2 + hv]);
                    mbar_arrive(&vempty[st]);
                    mbar_arrive(&cempty[slot]);
                }
            }
        }
        if (!ok) attn_abort(abort_flag);
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsHigh));
        // ------------------------------------------------ softmax: a thread per row
        const int s8 = warp - 4, tile = s8 >> 2, t = (s8 & 3) * 32 + lane;
        const uint32_t lane_off = static_cast<uint32_t>((s8 & 3) * 32) << 16;
        const uint32_t tS = tmem + lane_off + tile * 128, tO = tmem + lane_off + 256 + tile * DV;
        int g = 0, nq = 0;               // tiles; the row tile's items so far
        int nb[2] = {0, 0};              // uses of its buffers so far
        bool ok = true;                  // (a wait that gave up is acted on where the warp meets)
        float M = -INFINITY, l = 0.0f;
        int pn = 0, lim = 0;               // of the item before: steps, where its row goes
        int64_t row = -1;
        for (int k = 0;; ++k) {
            ManyItem m;
            const bool there = __all_sync(0xFFFFFFFFu, item_of(k, m) && ok) != 0;
            if (there && (tile ? m.steps[1] : m.steps[0]) > 0) {
                // ---- this item's queries: its products start while the last one's results are written
                // (the last one's reads of Q are done: their S has been read)
                if (nq > 0) ok = mbar_wait(&qread[tile], (nq - 1) & 1, abort_flag) && ok;
                // a warp takes its 32 rows, 4 at a time, 8 lanes a row: a lane has the
                // row's 8 values at 8 lane, and those 64 and 128 further on
                constexpr int kCh = DK / 64;
                const int sub = lane >> 3, el = lane & 7;
                uint8_t* qh = sQ + tile * 2 * F::kQTile;
                // lane r places row r
                int64_t src = -1;
                {
                    const int rr = m.row0 + tile * 128 + t, j = rr / p.G;
                    if (rr < m.rows)
                        src = (m.first + static_cast<int64_t>(j)) * p.q_ts + (m.h * p.G + rr - j * p.G) * p.q_hs;
                }
                constexpr int kFly = kCh == 3 ? 2 : 4;   // passes whose loads are in flight together
#pragma unroll 1
                for (int pass0 = 0; pass0 < 8; pass0 += kFly) {
                    uint4 v[kFly][kCh];
#pragma unroll
                    for (int k2 = 0; k2 < kFly; ++k2) {
                        const int64_t at = __shfl_sync(0xFFFFFFFFu, src, (pass0 + k2) * 4 + sub);
#pragma unroll
                        for (int c = 0; c < kCh; ++c)
                            v[k2][c] = at >= 0 ? __ldg(reinterpret_cast<const uint4*>(p.q + at) + c * 8 + el) : make_uint4(0, 0, 0, 0);
                    }
#pragma unroll
                    for (int k2 = 0; k2 < kFly; ++k2) {
                        const int r = (s8 & 3) * 32 + (pass0 + k2) * 4 + sub;
                        // the largest magnitude, as bf16 bits: above 0x7F7F it is not a number
                        uint32_t m2 = 0;
#pragma unroll
                        for (int c = 0; c < kCh; ++c)
                            m2 = __vmaxu2(m2, __vmaxu2(__vmaxu2(v[k2][c].x & 0x7FFF7FFFu, v[k2][c].y & 0x7FFF7FFFu),
                                                       __vmaxu2(v[k2][c].z & 0x7FFF7FFFu, v[k2][c].w & 0x7FFF7FFFu)));
#pragma unroll
                        for (int o = 4; o >= 1; o >>= 1) m2 = __vmaxu2(m2, __shfl_xor_sync(0xFFFFFFFFu, m2, o));
                        const uint32_t top = max(m2 & 0xFFFFu, m2 >> 16);
                        // 2^e <= it < 2^(e + 1); elements times 2^(7 - e)
                        const int e = max(-100, static_cast<int>(top >> 7) - 127);
                        const float up = __uint_as_float(static_cast<uint32_t>(127 + 7 - e) << 23);
                        const float down = __uint_as_float(static_cast<uint32_t>(127 - 7 + e) << 23);
#pragma unroll
                        for (int c = 0; c < kCh; ++c) {
                            const uint32_t w[4] = {v[k2][c].x, v[k2][c].y, v[k2][c].z, v[k2][c].w};
                            uint16_t hi[4];
                            uint32_t lo[4];
#pragma unroll
                            for (int i2 = 0; i2 < 4; ++i2) {
                                const float2 f = __fmul2_rn(make_float2(__uint_as_float(w[i2] << 16), __uint_as_float(w[i2] & 0xFFFF0000u)),
                                                            make_float2(up, up));
                                hi[i2] = f32x2_to_e4m3x2(f.x, f.y);
                                // the rest in fp16: an e5m2 is its high byte, rounded (3 significant bits
                                // are there unless hi is subnormal)
                                asm("sub.f16x2 %0, %1, %2;" : "=r"(lo[i2]) : "r"(f32x2_to_f16x2(f.x, f.y)), "r"(e4m3x2_to_f16x2(hi[i2])));
                                lo[i2] += 0x00800080u;
                            }
                            int at;
                            if (F::kWide && c < 2) {
                                const int byte = c * 64 + el * 8;
                                at = r * 128 + (((byte >> 4) ^ (r & 7)) << 4) + (byte & 15);
                            } else {
                                const int byte = el * 8;
                                at = (F::kWide ? 128 * 128 : 0) + r * 64 + (((byte >> 4) ^ ((r >> 1) & 3)) << 4) + (byte & 15);
                            }
                            *reinterpret_cast<uint2*>(qh + at) = make_uint2(hi[0] | (static_cast<uint32_t>(hi[1]) << 16),
                                                                            hi[2] | (static_cast<uint32_t>(hi[3]) << 16));
                            *reinterpret_cast<uint2*>(qh + F::kQTile + at) = make_uint2(__byte_perm(lo[0], lo[1], 0x7531),
                                                                                       __byte_perm(lo[2], lo[3], 0x7531));
                        }
                        if (el == 0) s_qf[tile * 128 + r] = top > 0x7F7Fu ? __uint_as_float(0x7FC00000u) : down * p.scale;
                    }
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(&qfull[tile]);
            }
            // ---- the last item's results
            if (k > 0) {
                uint4* dst = reinterpret_cast<uint4*>(p.out + row * DV);
                if (pn > 0) {
                    const int b = (pn - 1) & 1;
                    ok = mbar_wait(&odone[tile * 2 + b], ((b ? nb[1] : nb[0]) - 1) & 1, abort_flag) && ok;
                    __syncwarp();
                    tc_fence_after();
                    const float inv = l == 0.0f ? 0.0f : __frcp_rn(l);
#pragma unroll 1
                    for (int c = 0; c < DV; c += 32) {
                        uint32_t r[32];
                        __syncwarp();
                        tmem_ld32(tO + c, r);
                        tmem_wait_ld();
                        if (row >= 0) {
#pragma unroll
                            for (int k2 = 0; k2 < 2; ++k2) {   // 32 bytes at a time: half as many lines touched as with 16
                                uint32_t w[8];
#pragma unroll
                                for (int u = 0; u < 8; ++u) {
                                    const __nv_bfloat162 b2 = __floats2bfloat162_rn(__uint_as_float(r[16 * k2 + 2 * u]) * inv,
                                                                                    __uint_as_float(r[16 * k2 + 2 * u + 1]) * inv);
                                    w[u] = *reinterpret_cast<const uint32_t*>(&b2);
                                }
                                st_global_32(dst + c / 8 + 2 * k2, w);
                            }
                        }
                    }
                    tc_fence_before();
                    const uint32_t last = k - 1, note = last % kNotes;
                    if (s_nans[note] == last + 1 && row >= 0) {   // (rare)
#pragma unroll 1
                        for (int d = 0; d < DV; ++d)
                            if (sees_nan<kNanBits>(s_nan[note * DV + d], last + 1, lim - s_base[note]))
                                p.out[row * DV + d] = __float2bfloat16_rn(__uint_as_float(0x7FC00000u));
                    }
                } else if (row >= 0) {
#pragma unroll
                    for (int k2 = 0; k2 < DV / 8; ++k2) dst[k2] = make_uint4(0, 0, 0, 0);
                }
                if (row >= 0 && p.lse) p.lse[row] = l == 0.0f ? -INFINITY : (M - kPBits + log2f(l)) * kLn2;
            }
            if (!there) break;
            // ---- this item's tiles
            const int steps = (tile ? m.steps[1] : m.steps[0]), nmax = m.nmax;
            const int min_lim = limit(m, m.row0 + tile * 128);   // the tile's first row sees least
            {
                const int rr = m.row0 + tile * 128 + t, j = rr / p.G;
                const bool valid = rr < m.rows;
                lim = valid ? limit(m, rr) : 0x7FFFFFFF;
                row = valid ? (m.first + static_cast<int64_t>(j)) * p.Hq + m.h * p.G + rr - j * p.G : -1;
            }
            pn = steps;
            __syncwarp();
            if (lane == 0) mbar_arrive(&iempty[k % kItems]);
            float qf = 1.0f;
            bool odd_rows = false;   // (of the warp's)
            if (steps > 0) {
                ok = mbar_wait(&qfull[tile], nq & 1, abort_flag) && ok;
                ++nq;
                qf = s_qf[tile * 128 + t];
                odd_rows = __any_sync(0xFFFFFFFFu, row >= 0 && !(qf >= kLeast)) != 0;
                __syncwarp();
                if (lane == 0) mbar_arrive(&qread[tile]);
            }
            M = -INFINITY;
            l = 0.0f;
            for (int i = 0; i < nmax; ++i, ++g) {
                const int slot = g % kRing;
                ok = mbar_wait(&cfull[slot], (g / kRing) & 1, abort_flag) && ok;
                const uint32_t dead = s_dead[slot];
#pragma unroll 1
                for (int hv = 0; hv < 2; ++hv) {   // (and the buffer of that step)
                    const int step = 2 * i + hv;
                    if (step >= steps) break;
                    const bool masked = (step + 1) * 64 > min_lim || dead != 0;   // (the same in the whole tile)
                    const int col0 = hv * 64;
                    float ck[4], lv[4], iv[4];   // constants of 16 columns each
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        const float4 of = s_page[slot * 8 + ((col0 + q * 16) >> p.bs_log2)];
                        ck[q] = of.x * qf;
                        lv[q] = of.y;
                        iv[q] = of.z;
                    }
                    ok = mbar_wait(&sfull[tile * 2 + hv], (hv ? nb[1] : nb[0]) & 1, abort_flag) && ok;
                    __syncwarp();
                    tc_fence_after();
                    // ---- S; columns that the row does not see are -inf
                    uint32_t r[64];
                    tmem_ld32(tS + hv * 64, *reinterpret_cast<uint32_t(*)[32]>(r));
                    tmem_ld32(tS + hv * 64 + 32, *reinterpret_cast<uint32_t(*)[32]>(r + 32));
                    tmem_wait_ld();
                    if (masked) {
                        // A factor that is zero (K's scale may be, or the product) would make NaN of an -inf, and
                        // a negative one turns round the order that the maximum below goes by: then x itself.
                        if (odd_rows || (dead & kOdd) != 0) {
#pragma unroll
                            for (int k2 = 0; k2 < 64; ++k2)
                                r[k2] = __float_as_uint(fmaf(__uint_as_float(r[k2]), ck[k2 / 16], lv[k2 / 16]));
#pragma unroll
                            for (int q = 0; q < 4; ++q) {
                                ck[q] = 1.0f;
                                lv[q] = 0.0f;
                            }
                        }
                        const int left = lim - i * 128 - col0;
#pragma unroll
                        for (int q = 0; q < 4; ++q) {
                            const int lf = (dead >> ((col0 + q * 16) >> p.bs_log2)) & 1 ? 0 : left - q * 16;
#pragma unroll
                            for (int k2 = 0; k2 < 16; ++k2)
                                if (k2 >= lf) r[q * 16 + k2] = 0xFF800000u;
                        }
                    }
                    // ---- the row's maximum of x = S c + log2(v_scale)
                    float mx = -INFINITY;
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        const uint32_t* x = r + q * 16;
                        float a = __uint_as_float(x[0]), c = __uint_as_float(x[1]);
#pragma unroll
                        for (int k2 = 2; k2 < 16; k2 += 4) {
                            a = max3(a, __uint_as_float(x[k2]), __uint_as_float(x[k2 + 1]));
                            if (k2 + 2 < 16) c = max3(c, __uint_as_float(x[k2 + 2]), __uint_as_float(x[k2 + 3]));
                        }
                        mx = fmaxf(mx, fmaf(fmaxf(a, c), ck[q], lv[q]));
                    }
                    const bool grows = mx > M + kSlack || (M == -INFINITY && mx > M);
                    if (__any_sync(0xFFFFFFFFu, grows)) {
                        const float fac = grows ? ex2(M - mx) : 1.0f;
                        if (grows) M = mx;
                        l *= fac;
                        if (step > 0) {   // O, once the products of the step before are done
                            ok = mbar_wait(&odone[tile * 2 + (hv ^ 1)], ((hv ? nb[0] : nb[1]) - 1) & 1, abort_flag) && ok;
                            __syncwarp();
                            tc_fence_after();
#pragma unroll 1
                            for (int c = 0; c < DV; c += 16) {
                                float o[16];
                                tmem_ld<16>(tO + c, o);
                                tmem_wait_ld();
#pragma unroll
                                for (int e = 0; e < 16; ++e) o[e] *= fac;
                                tmem_st16(tO + c, o);
                            }
                        }
                    }
                    // ---- P = 2^(x - M + 8)
                    const float off = M == -INFINITY ? 0.0f : kPBits - M;
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        const float2 c2 = make_float2(ck[q], ck[q]), l2 = make_float2(lv[q] + off, lv[q] + off);
                        float2 sum = make_float2(0.0f, 0.0f);
#pragma unroll
                        for (int k2 = 0; k2 < 16; k2 += 2) {
                            const int at = q * 16 + k2;
                            const float2 y = __ffma2_rn(make_float2(__uint_as_float(r[at]), __uint_as_float(r[at + 1])), c2, l2);
                            const float2 e2 = make_float2(ex2(y.x), ex2(y.y));
                            sum = __fadd2_rn(sum, e2);
                            r[at / 2] = f32x2_to_f16x2(e2.x, e2.y);
                        }
                        l = fmaf(sum.x + sum.y, iv[q], l);
                    }
                    // ---- P over S
                    tmem_st16u(tS + hv * 64, r);
                    tmem_st16u(tS + hv * 64 + 16, r + 16);
                    tmem_wait_st();
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&pfull[tile * 2 + hv]);
                    if (hv) ++nb[1]; else ++nb[0];
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(&cempty[slot]);
                if (!__all_sync(0xFFFFFFFFu, ok)) break;
            }
        }
        if (!ok) attn_abort(abort_flag);
    }

    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 1) tmem_dealloc(tmem, 512);
}

template <int DK, int DV>
cudaError_t launch(const AttnMaps& m, const AttnParams& p, int sms, cudaStream_t st) {
    using F = Many<DK, DV>;
    static int configured[64] = {};
    int dev = 0;
    cudaGetDevice(&dev);
    if (dev >= 64 || !configured[dev]) {
        const cudaError_t e = cudaFuncSetAttribute(attn_many_kernel<DK, DV>, cudaFuncAttributeMaxDynamicSharedMemorySize, F::kSmem);
        if (e != cudaSuccess) return e;
        cudaFuncAttributes a{};   // (the registers that change hands are the launch's)
        if (cudaFuncGetAttributes(&a, attn_many_kernel<DK, DV>) != cudaSuccess || a.numRegs != kRegsLaunch)
            return cudaErrorInvalidConfiguration;
        if (dev < 64) configured[dev] = 1;
    }
    return launch_pdl(attn_many_kernel<DK, DV>, dim3(sms), dim3(kThreads), F::kSmem, st, m.k0, m.k1, m.v, p);
}

}  // namespace

cudaError_t launch_many(int dk, const AttnMaps& m, const AttnParams& p, int sms, cudaStream_t st) {
    return dk == 64 ? launch<64, 64>(m, p, sms, st) : dk == 128 ? launch<128, 128>(m, p, sms, st) : launch<192, 128>(m, p, sms, st);
}
int many_read_and_clear_status(cudaStream_t st) { return read_and_clear_attention_status(st); }
bool many_set_wait_limit(long long cycles) { return set_attention_wait_limit(cycles); }

}  // namespace fp8bs
