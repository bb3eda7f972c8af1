// attention_few.cu -- attention over the paged 8-bit cache for requests with
// few rows of queries: single tokens, a few of them, a group of heads
// (attention.cuh).
//
// A tile is 128 tokens of one cache head; the MMA has the tokens on its
// 128-row side and the rows of queries, hi and lo, on its N side:
//   S^T [token, row] = K (K-major) x Q,   O^T [dv, row] = V^T (V as it lies,
//   MN-major) x P.
// So the tensor core reads each byte of the cache once, whatever the number
// of rows, and a thread of the softmax owns one token.
// dv = 64: two tokens share a 128-byte row of V, so the 128 M rows are the
// dims of the even and of the odd tokens, K counts pairs, and P has separate
// columns for the two; the halves of O are added at the end.
//
// The tiles of all requests and heads form one sequence, which is cut into as
// many ranges of equal cost as there are CTAs: ragged lengths load the GPU
// evenly, and few requests are split over it.  A segment (the tiles of one request, cache
// head and chunk of rows) that a cut goes through leaves parts, which
// attn_join_kernel adds.
//
// A CTA's warps: 0 loads the tiles by TMA, 1 issues the MMAs, 2 splits the
// next segment's queries, 3 fetches the scales of the tiles' pages, 4-7 are
// the softmax.
//
// A tile is in the pipeline for some 7000 cycles: 2500 for HBM under load, 700
// for S, 2200 for the softmax's chain (TMEM read, maximum over the tokens,
// exponentials, P to shared memory), the rest for O.  Bandwidth is what fits
// in shared memory over that time, so K and V have rings of their own: K's
// stage is free after S, V's only after O, and V gets twice the stages.
#include "attention.cuh"

#include <type_traits>

namespace fp8bs {
namespace {

constexpr float kPBits = 4.0f;      // probabilities are 2^(x - M + 4): at most 16 with the true maximum M,
constexpr float kMostBits = 8.0f;   // and at most 256 with one that has since been passed: 32 x the half unit of
                                    // hi that lo has to hold is 256 there, below e4m3's 448
constexpr int kThreads = 256;
constexpr int kJoinThreads = 256;
constexpr int kNanBits = 8;         // a segment's rows are at most 32 queries, and what none of them sees need not be told apart

// A part: O of each row, then (M, l) of each; a multiple of 16 bytes.
__host__ __device__ constexpr int part_floats(int ru, int dv) { return ru * dv + (ru < 2 ? 4 : 2 * ru); }
// A range's record: first and last range of the segment that crosses its
// begin (-1: none), two unused, that segment's output rows (64 bits each).
__host__ __device__ constexpr int info_ints(int ru) { return 4 + (ru < 2 ? 4 : 2 * ru); }
// CTAs per SM: rows cost registers.
__host__ __device__ constexpr int few_blocks(int ru) { return ru > 16 ? 1 : 2; }

// RU: the rows that are computed; the MMA has at least NR = 8.  kSeveral: a
// request may have several queries, and then tokens that only some rows see,
// whose V is looked over for NaNs.  (Kernels of their own: with the search in
// those of single tokens too, 8 rows of 64 values took 69.5 us against 66.8,
// 32 rows of 128 62.5 against 60.6.)
template <int DK, int DV, int RU, bool kSeveral>
struct Few {
    static constexpr int NR = RU < 8 ? 8 : RU;
    static constexpr bool kWide = DK >= 128;                  // a 128-byte slab of K ...
    static constexpr bool kHalf = DK % 128 == 64;             // ... and a 64-byte one
    static constexpr int kN = 2 * NR;                         // columns of S: hi, lo
    static constexpr int kPair = DV == 64 ? 2 : 1;
    static constexpr int kON = kN * kPair;                    // columns of O
    static constexpr int kKBytes = 128 * DK, kVBytes = 128 * DV;
    static constexpr int kQBytes = kN * DK, kPBytes = kON * 128;
    static constexpr int kCols = 2 * kN + 2 * kON;
    static constexpr int kTmem = kCols <= 64 ? 64 : kCols <= 128 ? 128 : kCols <= 256 ? 256 : 512;
    static constexpr int kBlocks = few_blocks(RU);
    static constexpr int kBars = 448;
    static constexpr int kPairX = DV == 64 ? RU * 64 : 0;     // the odd tokens' half of O (floats)
    static constexpr int kMisc = 2 * NR * 8 + (3 * kFewB + 12) * 4 + (4 * RU + 8 * RU + 2 * RU + 2 * NR + 2 * NR) * 4 +
                                 kRing * 8 * 12 + kPairX * 4 + (kSeveral ? (2 * DV + 2) * 4 : 0) + 8 + kBars;
    static constexpr int kFixed = 1024 + 2 * kQBytes + 2 * kPBytes + kMisc;
    static constexpr int kBudget = (kBlocks == 1 ? 227 : 113) * 1024 - 64;   // (64: s_scan)
    // K's stages are a third of the space (2 at least), V's the rest.  (A KB more for K's: 4 rows of 64 values with 4
    // and 7 stages 57.3 us, with 3 and 8 58.2.)
    static constexpr int kSK = (kBudget - kFixed + 1024) / 3 / kKBytes < 2 ? 2 : (kBudget - kFixed + 1024) / 3 / kKBytes > 4 ? 4 : (kBudget - kFixed + 1024) / 3 / kKBytes;
    static constexpr int kFitV = (kBudget - kFixed - kSK * kKBytes) / kVBytes;
    static constexpr int kSV = kFitV > 8 ? 8 : kFitV;
    static constexpr int kSmem = kFixed + kSK * kKBytes + kSV * kVBytes;
    static constexpr int kPartFloats = part_floats(RU, DV);
    static constexpr int kSegment = RU >= 16 ? 3 : 2;   // cost of a segment in tiles (see TileWalk)
    static_assert(kSK >= 2 && kSV >= 2, "pipeline depth");
};

// a / b of not negative numbers, in 32 bits where a has no more (a 64-bit
// division takes some 100 instructions, and a launch begins with several).
__device__ __forceinline__ long long quotient(long long a, long long b) {
    return ((a | b) >> 32) == 0 ? static_cast<long long>(static_cast<uint32_t>(a) / static_cast<uint32_t>(b)) : a / b;
}

// A segment costs more than its tiles: its first tile takes the long way to
// the maxima, and its results are written.  Ranges are equal in tiles plus
// kSegment of them for each segment: position v of a segment is its tile
// v - kSegment, or, before that, nothing.  (Equal in tiles alone, the CTAs
// that got the short requests of a ragged batch ended last: 64 requests of
// 100 to 8192, SMs busy 69% of the time.  1 / 2 / 3 tiles for a segment: 16
// rows 97 / 76 / 73 us, 8 rows of 64 values 68 / 65 / 66 us.)
//
// Walks a CTA's tiles: requests in order, their segments (cache head, chunk
// of RU rows), a segment's tiles.  It runs for every tile in every warp, so a
// division is done per request only.
template <int kSegment>
struct TileWalk {
    const int* seg;   // [B + 1] segments of one cache head before each request
    const int* len;   // [B]
    int B, Hkv, b, h, c, tile, nt, chunks;
    __device__ void enter() {
        nt = (len[b] + 127) >> 7;
        chunks = seg[b + 1] - seg[b];
    }
    // To position v (cum: positions of one cache head before each request);
    // returns the tiles before it.
    __device__ long long start(const int* cum, const int* seg_, const int* len_, int B_, int Hkv_, long long v) {
        seg = seg_;
        len = len_;
        B = B_;
        Hkv = Hkv_;
        int l = 0, r = B;
        while (r - l > 1) {
            const int m = (l + r) >> 1;
            if (static_cast<long long>(cum[m]) * Hkv <= v) l = m; else r = m;
        }
        b = l;
        enter();
        const long long rem = v - static_cast<long long>(cum[b]) * Hkv;
        const int s = static_cast<int>(quotient(rem, nt + kSegment));
        const int at = static_cast<int>(rem - static_cast<long long>(s) * (nt + kSegment));
        tile = max(0, at - kSegment);
        h = s / chunks;
        c = s - h * chunks;
        return v - (static_cast<long long>(seg[b]) * Hkv + s) * kSegment - min(at, kSegment);
    }
    __device__ void next() {
        if (++tile == nt) next_segment();
    }
    __device__ void next_segment() {
        tile = 0;
        if (++c < chunks) return;
        c = 0;
        if (++h < Hkv) return;
        h = 0;
        do ++b; while (b < B && seg[b + 1] == seg[b]);
        if (b < B) enter();
        else b = B - 1;   // past the last tile
    }
};

// A bounded wait for the roles that watch several barriers: false once
// nothing has moved for the limit, or somebody gave up.
struct Patience {
    long long since = 0;
    uint32_t idle = 0;
    __device__ bool left(bool moved, const volatile int* abort_flag) {
        if (moved) idle = 0;
        else if (++idle == 1) since = clock64();
        else if ((idle & 63u) == 0u) return !*abort_flag && clock64() - since <= g_wait_limit_cycles;
        return true;
    }
};

template <int DK, int DV, int RU, bool kSeveral>
__global__ void __launch_bounds__(kThreads, (Few<DK, DV, RU, kSeveral>::kBlocks))
    attn_few_kernel(const __grid_constant__ CUtensorMap tm_k0, const __grid_constant__ CUtensorMap tm_k1,
                    const __grid_constant__ CUtensorMap tm_v, const AttnParams p) {
    using F = Few<DK, DV, RU, kSeveral>;
    using Walk = TileWalk<F::kSegment>;
    constexpr int kSegment = F::kSegment;
    constexpr int SK = F::kSK, SV = F::kSV, NR = F::NR, N = F::kN, ON = F::kON;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    uint8_t* sK = smem;                              // SK tiles of K: the 128-byte slab, then the 64-byte one
    uint8_t* sV = sK + SK * F::kKBytes;              // SV tiles of V
    uint8_t* sQ = sV + SV * F::kVBytes;              // 2 segments' queries
    uint8_t* sP = sQ + 2 * F::kQBytes;               // 2 tiles' probabilities
    long long* s_row = reinterpret_cast<long long*>(sP + 2 * F::kPBytes);    // [2][NR] output row (token * Hq + head) or -1
    int* s_cum = reinterpret_cast<int*>(s_row + 2 * NR);                     // [kFewB + 1] positions before each request
    int* s_seg = s_cum + kFewB + 4;                  // [kFewB + 1] segments before it (of one cache head, both)
    int* s_len = s_seg + kFewB + 4;                  // [kFewB]
    int* s_min = s_len + kFewB;                      // [2] tokens that every row sees
    float* s_qf = reinterpret_cast<float*>(s_min + 4);                       // [2][NR] factor of a row's S
    int* s_lim = reinterpret_cast<int*>(s_qf + 2 * NR);                      // [2][NR] tokens a row sees
    float* s_max = reinterpret_cast<float*>(s_lim + 2 * NR);                 // [4 warps][RU]
    float* s_l = s_max + 4 * RU;                     // [2 segments][4 warps][RU]
    float* s_M = s_l + 8 * RU;                       // [2][RU]
    float* s_ck = s_M + 2 * RU;                      // [kRing][8] k_scale of the tile's pages
    float* s_lv = s_ck + kRing * 8;                  // log2(v_scale), -inf: the page is left out
    float* s_iv = s_lv + kRing * 8;                  // 1 / v_scale, or 0
    float* s_x = s_iv + kRing * 8;                   // dv = 64: [RU][64]
    uint32_t* s_nan = reinterpret_cast<uint32_t*>(s_x + F::kPairX);          // [2 segments][DV] NaNs in V (nan_key)
    uint32_t* s_nans = s_nan + 2 * DV;               // [2] the last segment that has one
    uint64_t* bars = reinterpret_cast<uint64_t*>((reinterpret_cast<uintptr_t>(s_nan + (kSeveral ? 2 * DV + 2 : 0)) + 7) & ~static_cast<uintptr_t>(7));
    uint64_t* kfull = bars;
    uint64_t* kempty = kfull + SK;
    uint64_t* vfull = kempty + SK;
    uint64_t* vempty = vfull + SV;
    uint64_t* sfull = vempty + SV;     // 2: S of a tile is in TMEM
    uint64_t* sempty = sfull + 2;      // 2: and has been read (4 warps)
    uint64_t* pfull = sempty + 2;      // 2: P of a tile is in shared memory (4 warps)
    uint64_t* pvdone = pfull + 2;      // 2: O holds the tile
    uint64_t* cfull = pvdone + 2;      // kRing: page constants
    uint64_t* cempty = cfull + kRing;
    uint64_t* qfull = cempty + kRing;  // 2: a segment's queries
    uint64_t* qempty = qfull + 2;      // 2: (the MMAs, 4 softmax warps)
    uint64_t* mma_done = qempty + 2;
    uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(mma_done + 1);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_holder + 1);
    __shared__ int2 s_scan[kThreads / 32];
    static_assert((2 * SK + 2 * SV + 8 + 2 * kRing + 4 + 1) * 8 + 16 + 8 <= F::kBars, "barrier block");

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (int i = 0; i < SK; ++i) {
            mbar_init(&kfull[i], 1);
            mbar_init(&kempty[i], 1);
        }
        for (int i = 0; i < SV; ++i) {
            mbar_init(&vfull[i], 1);
            mbar_init(&vempty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&sfull[i], 1);
            mbar_init(&sempty[i], 4);
            mbar_init(&pfull[i], 4);
            mbar_init(&pvdone[i], 1);
            mbar_init(&qfull[i], 1);
            mbar_init(&qempty[i], 5);
        }
        for (int i = 0; i < kRing; ++i) {
            mbar_init(&cfull[i], 1);
            mbar_init(&cempty[i], 4);
        }
        mbar_init(mma_done, 1);
        *abort_flag = 0;
        fence_mbar_init();
        tma_prefetch_desc(&tm_k0);
        tma_prefetch_desc(&tm_k1);
        tma_prefetch_desc(&tm_v);
    }
    if (warp == 1) {
        tmem_alloc(tmem_holder, F::kTmem);
        tmem_relinquish();
    }
    if constexpr (kSeveral)
        for (int i = threadIdx.x; i < 2 * DV + 2; i += kThreads) s_nan[i] = 0;
    if constexpr (RU < NR) {   // rows that are only there for the MMA stay zero
        uint4* z = reinterpret_cast<uint4*>(sQ);
        for (int i = threadIdx.x; i < (2 * F::kQBytes + 2 * F::kPBytes) / 16; i += kThreads) z[i] = make_uint4(0, 0, 0, 0);
        fence_proxy_async_smem();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_holder;
    const uint32_t tS = tmem, tO = tmem + 2 * N;
    griddep_launch_dependents();
    griddep_wait();

    // ---- the work: positions and segments of every request of few rows, as
    // running sums (both within 31 bits: the host sees to it)
    const int cap = p.width << p.bs_log2;
    {
        const int b = threadIdx.x;
        static_assert(kFewB <= kThreads, "a thread per request");
        int segs = 0, tiles = 0;
        if (b < p.B) {
            const int len = max(0, min(p.lens[b], cap));
            const int64_t n = p.offsets ? min(static_cast<int64_t>(p.offsets[b + 1] - p.offsets[b]), p.T - p.offsets[b]) : 1;
            const int64_t rows = n * p.G;   // (q may end before the request)
            s_len[b] = len;
            tiles = (len + 127) >> 7;
            if (len > 0 && rows > 0 && rows <= p.few_rows) segs = (static_cast<int>(rows) + RU - 1) / RU;
        }
        const int mine = segs * (tiles + kSegment);
        int inc = mine, sinc = segs;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int up = __shfl_up_sync(0xFFFFFFFFu, inc, o), sup = __shfl_up_sync(0xFFFFFFFFu, sinc, o);
            if (lane >= o) {
                inc += up;
                sinc += sup;
            }
        }
        if (lane == 31) s_scan[warp] = make_int2(inc, sinc);
        __syncthreads();
        int run = inc - mine, srun = sinc - segs;
        for (int w = 0; w < warp; ++w) {
            run += s_scan[w].x;
            srun += s_scan[w].y;
        }
        if (b < p.B) {
            s_cum[b] = run;
            s_seg[b] = srun;
        }
        if (b == p.B - 1) {
            s_cum[p.B] = run + mine;
            s_seg[p.B] = srun + segs;
        }
        __syncthreads();
    }
    // range r: `each` positions, and one more for the first `more` ranges
    const long long total = static_cast<long long>(s_cum[p.B]) * p.Hkv;
    const long long ctas = total < static_cast<long long>(gridDim.x) ? total : static_cast<long long>(gridDim.x);
    const long long me = blockIdx.x;
    const long long each = ctas > 0 ? quotient(total, ctas) : 0, more = total - each * ctas;
    auto begin_of = [&](long long r) { return r * each + min(r, more); };
    Walk it;
    int ntiles = 0;
    if (me < ctas) {
        const long long v0 = begin_of(me), v1 = begin_of(me + 1);
        const long long first = it.start(s_cum, s_seg, s_len, p.B, p.Hkv, v0);
        Walk end;
        ntiles = static_cast<int>((v1 == total ? total - static_cast<long long>(s_seg[p.B]) * p.Hkv * kSegment
                                               : end.start(s_cum, s_seg, s_len, p.B, p.Hkv, v1)) - first);
        if (threadIdx.x == 0) {
            if (me == 0) p.info[0] = static_cast<int>(ctas);
            // did the range's first segment begin before it? in which range, and where does it end?
            auto range_of = [&](long long v) {
                return static_cast<int>(v < more * (each + 1) ? quotient(v, each + 1) : more + quotient(v - more * (each + 1), each));
            };
            const long long t0 = v0 - it.tile;
            *reinterpret_cast<int2*>(p.info + 4 + me * info_ints(RU)) =
                ntiles > 0 && it.tile > 0 ? make_int2(range_of(t0), range_of(t0 + it.nt - 1)) : make_int2(-1, -1);
        }
    } else if (total == 0 && me == 0 && threadIdx.x == 0) {
        p.info[0] = 0;
    }

    // ---- rows that no tile reaches: requests without tokens, rows past the last request
    {
        auto zero_rows = [&](int64_t r0, int64_t r1) {
            uint4* o = reinterpret_cast<uint4*>(p.out) + r0 * p.Hq * (DV / 8);
            for (int64_t i = threadIdx.x; i < (r1 - r0) * p.Hq * (DV / 8); i += kThreads) o[i] = make_uint4(0, 0, 0, 0);
            if (p.lse)
                for (int64_t i = threadIdx.x; i < (r1 - r0) * p.Hq; i += kThreads) p.lse[r0 * p.Hq + i] = -INFINITY;
        };
        for (int b = blockIdx.x; b < p.B; b += gridDim.x) {
            if (s_len[b] != 0) continue;
            if (p.offsets) {
                const int64_t r0 = max(0, p.offsets[b]), r1 = min(static_cast<int64_t>(p.offsets[b + 1]), p.T);
                if (r0 < r1) zero_rows(r0, r1);
            } else {
                zero_rows(p.row0 + b, p.row0 + b + 1);
            }
        }
        if (p.offsets && p.fill_tail) {
            const int64_t end = max(0, p.offsets[p.B]);
            for (int64_t r = end + blockIdx.x; r < p.T; r += gridDim.x) zero_rows(r, r + 1);
        }
    }

    const int pages_per_tile = 128 >> p.bs_log2, bs = 1 << p.bs_log2;
    if (warp == 0) {
        // ------------------------------------------------ producer: lane i loads page i of the tile
        auto page_of = [&](const Walk& w) {
            const int idx = w.tile * pages_per_tile + lane;
            const bool on = lane < pages_per_tile && (idx << p.bs_log2) < w.len[w.b];
            return on ? p.tables[static_cast<int64_t>(w.b) * p.width + idx] : -1;
        };
        // K and V go their own ways: a stage of V that is not free yet must
        // not hold back the next K.
        struct Stream {
            Walk w;
            int i, page;
        } k, v;
        k.w = it;
        k.i = 0;
        k.page = ntiles > 0 ? page_of(it) : -1;
        v = k;
        auto advance = [&](Stream& s) {
            ++s.i;
            if (s.i < ntiles) {
                s.w.next();
                s.page = page_of(s.w);
            }
        };
        auto pages = [&](const Walk& w) { return min(pages_per_tile, ((w.len[w.b] - w.tile * 128) + bs - 1) >> p.bs_log2); };
        Patience patience;
        bool ok = true;
        while (v.i < ntiles) {   // (V does not overtake K, so K is done then)
            bool moved = false;
            if (k.i < ntiles && __all_sync(0xFFFFFFFFu, mbar_test(&kempty[k.i % SK], ((k.i / SK) & 1) ^ 1))) {
                const int st = k.i % SK, np = pages(k.w);
                if (lane == 0) mbar_arrive_expect_tx(&kfull[st], static_cast<uint32_t>(np * bs * DK));
                __syncwarp();
                uint8_t* dst = sK + st * F::kKBytes;
                if (lane < np) {
                    if constexpr (F::kWide) tma_load_page(dst + lane * bs * 128, &tm_k0, &kfull[st], 0, k.w.h * bs, k.page);
                    if constexpr (F::kHalf)
                        tma_load_page(dst + (F::kWide ? 128 * 128 : 0) + lane * bs * 64, &tm_k1, &kfull[st],
                                      F::kWide ? 128 : 0, k.w.h * bs, k.page);
                }
                advance(k);
                moved = true;
            }
            __syncwarp();
            if (v.i < k.i && __all_sync(0xFFFFFFFFu, mbar_test(&vempty[v.i % SV], ((v.i / SV) & 1) ^ 1))) {
                const int st = v.i % SV, np = pages(v.w);
                const bool skip = p.debug_skip != 0 && v.i == 0;
                if (lane == 0 && !skip) mbar_arrive_expect_tx(&vfull[st], static_cast<uint32_t>(np * bs * DV));
                __syncwarp();
                if (lane < np && !skip)
                    tma_load_page(sV + st * F::kVBytes + lane * bs * DV, &tm_v, &vfull[st], 0, v.w.h * bs / F::kPair, v.page);
                advance(v);
                moved = true;
            }
            __syncwarp();
            if (!__all_sync(0xFFFFFFFFu, patience.left(moved, abort_flag))) {
                ok = false;
                break;
            }
        }
        if (!ok) attn_abort(abort_flag);
        // every load issued must land before the CTA may exit
        const volatile int never = 0;
        for (int st = 0; st < SK && st < k.i; ++st) {
            const int uses = k.i / SK + (st < k.i % SK ? 1 : 0);
            if (!mbar_wait(&kfull[st], (uses - 1) & 1, &never)) attn_abort(abort_flag);
        }
        for (int st = 0; st < SV && st < v.i; ++st) {
            const int uses = v.i / SV + (st < v.i % SV ? 1 : 0);
            if (!mbar_wait(&vfull[st], (uses - 1) & 1, &never)) attn_abort(abort_flag);
        }
    } else if (warp == 1) {
        // ------------------------------------------------ MMA issuer
        if (lane == 0) {
            constexpr uint32_t id_s = idesc_e4m3_f32(128, N);
            constexpr uint32_t id_o = idesc_e4m3_f32(128, ON) | (1u << 15);   // A (V) is MN-major
            // Two tiles may be between their S and their O.  Whichever product
            // has its operands goes next: waiting for a K that is still on
            // its way must not hold back a P that is there.
            int sg = -1, iq = 0, ip = 0;
            uint32_t first_bits = 0;   // bit i & 1: tile i is its segment's first here; bit 2 + (i & 1): its segment is odd
            Patience patience;
            while (ip < ntiles) {
                bool moved = false;
                if (iq < ntiles && iq - ip < 2) {
                    const int st = iq % SK, buf = iq & 1;
                    const bool fresh = iq == 0 || it.tile == 0;
                    const int sq = fresh ? sg + 1 : sg;
                    if (mbar_test(&kfull[st], (iq / SK) & 1) && mbar_test(&sempty[buf], ((iq >> 1) & 1) ^ 1) &&
                        (!fresh || mbar_test(&qfull[sq & 1], (sq >> 1) & 1))) {
                        sg = sq;
                        tc_fence_after();
                        const uint32_t k = smem_u32(sK + st * F::kKBytes), q = smem_u32(sQ + (sg & 1) * F::kQBytes);
                        const uint32_t d = tS + buf * N;
                        if constexpr (F::kWide) {
                            const uint64_t da = smem_desc_sw128(k), db = smem_desc_sw128(q);
#pragma unroll
                            for (int kk = 0; kk < 4; ++kk) mma_e4m3(d, da + 2 * kk, db + 2 * kk, id_s, kk > 0 ? 1u : 0u);
                        }
                        if constexpr (F::kHalf) {
                            const uint64_t da = smem_desc_sw64(k + (F::kWide ? 128 * 128 : 0));
                            const uint64_t db = smem_desc_sw64(q + (F::kWide ? N * 128 : 0));
#pragma unroll
                            for (int kk = 0; kk < 2; ++kk)
                                mma_e4m3(d, da + 2 * kk, db + 2 * kk, id_s, F::kWide || kk > 0 ? 1u : 0u);
                        }
                        mma_commit(&kempty[st]);
                        mma_commit(&sfull[buf]);
                        if (iq == ntiles - 1 || it.tile == it.nt - 1) mma_commit(&qempty[sg & 1]);
                        first_bits = (first_bits & ~(5u << buf)) | (fresh ? 1u << buf : 0u) | (sg & 1 ? 4u << buf : 0u);
                        it.next();
                        ++iq;
                        moved = true;
                    }
                }
                if (ip < iq) {
                    const int st = ip % SV, buf = ip & 1;
                    if (mbar_test(&pfull[buf], (ip >> 1) & 1) && mbar_test(&vfull[st], (ip / SV) & 1)) {
                        tc_fence_after();
                        const uint64_t da = smem_desc_mn128(smem_u32(sV + st * F::kVBytes));
                        const uint64_t db = smem_desc_sw128(smem_u32(sP + buf * F::kPBytes));
                        const bool fresh = (first_bits >> buf) & 1;
                        const uint32_t d = tO + ((first_bits >> buf) & 4 ? ON : 0);
#pragma unroll
                        for (int kk = 0; kk < 4 / F::kPair; ++kk)   // 32 tokens (or pairs): 32 rows of V, 32 bytes of P
                            mma_e4m3(d, da + kk * (4096 >> 4), db + 2 * kk, id_o, fresh && kk == 0 ? 0u : 1u);
                        mma_commit(&vempty[st]);
                        mma_commit(&pvdone[buf]);
                        ++ip;
                        moved = true;
                    }
                }
                if (!patience.left(moved, abort_flag)) {
                    attn_abort(abort_flag);
                    break;
                }
            }
            mma_commit(mma_done);
            const volatile int never = 0;
            if (!mbar_wait(mma_done, 0, &never)) attn_abort(abort_flag);
        }
    } else if (warp == 2) {
        // ------------------------------------------------ queries of each segment, split into e4m3 hi and lo
        int sg = -1;
        for (int i = 0; i < ntiles; ++i, it.next()) {
            if (i > 0 && it.tile != 0) continue;
            ++sg;
            const int buf = sg & 1;
            const int h = it.h, chunk = it.c;
            const int64_t first = p.offsets ? p.offsets[it.b] : p.row0 + it.b;
            const int n = p.offsets ? p.offsets[it.b + 1] - p.offsets[it.b] : 1;
            const int len = it.len[it.b];
            // lane r places row r: row chunk * RU + r of the segment is query
            // (that) / G, head (that) % G
            int64_t src = -1, row = -1;
            int lim = len;
            {
                const int rr = chunk * RU + lane, j = rr / p.G;
                const int64_t tok = first + j;
                const int head = h * p.G + rr - j * p.G;
                if (lane < RU && j < n && tok >= 0 && tok < p.T) {
                    src = tok * p.q_ts + head * p.q_hs;
                    row = tok * p.Hq + head;
                    lim = max(0, min(len, len - n + j + 1));
                }
            }
            const int least = __reduce_min_sync(0xFFFFFFFFu, lim);
            // kLanes lanes take a row, 8 values each
            constexpr int kLanes = DK / 8, kRows = 32 / kLanes, kPasses = (RU + kRows - 1) / kRows;
            constexpr int kFly = kPasses < 4 ? kPasses : 4;   // passes whose loads are in flight together
            const int sub = lane / kLanes, el = lane - sub * kLanes;
            uint4 v[kFly];
            auto load_rows = [&](int pass0) {
#pragma unroll
                for (int k = 0; k < kFly; ++k) {
                    const int r = (pass0 + k) * kRows + sub;
                    const int64_t at = __shfl_sync(0xFFFFFFFFu, src, r & 31);
                    v[k] = sub < kRows && r < RU && at >= 0 ? __ldg(reinterpret_cast<const uint4*>(p.q + at) + el)
                                                            : make_uint4(0, 0, 0, 0);
                }
            };
            load_rows(0);
            if (!__all_sync(0xFFFFFFFFu, mbar_wait(&qempty[buf], ((sg >> 1) & 1) ^ 1, abort_flag))) {
                attn_abort(abort_flag);
                break;
            }
            uint8_t* q = sQ + buf * F::kQBytes;
            if (lane < RU) {
                s_row[buf * NR + lane] = row;
                s_lim[buf * NR + lane] = lim;
            }
            if (lane == 0) s_min[buf] = least;
            for (int pass0 = 0; pass0 < kPasses; pass0 += kFly) {
                if (pass0 > 0) load_rows(pass0);
#pragma unroll
                for (int k = 0; k < kFly; ++k) {
                    const int r = (pass0 + k) * kRows + sub;
                    // the largest magnitude, as bf16 bits: above 0x7F7F it is not a number
                    const uint32_t m2 = __vmaxu2(__vmaxu2(v[k].x & 0x7FFF7FFFu, v[k].y & 0x7FFF7FFFu),
                                                 __vmaxu2(v[k].z & 0x7FFF7FFFu, v[k].w & 0x7FFF7FFFu));
                    uint32_t top = max(m2 & 0xFFFFu, m2 >> 16);
                    if constexpr (kRows == 1) {
                        top = __reduce_max_sync(0xFFFFFFFFu, top);
                    } else {
#pragma unroll
                        for (int o = kLanes / 2; o >= 1; o >>= 1) top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
                    }
                    // 2^e <= it < 2^(e + 1); elements times 2^(7 - e)
                    const int e = max(-100, static_cast<int>(top >> 7) - 127);
                    const float up = __uint_as_float(static_cast<uint32_t>(127 + 7 - e) << 23);
                    const float down = __uint_as_float(static_cast<uint32_t>(127 - 7 + e) << 23);
                    float f[8];
                    unpack_bf16x8(v[k], f);
                    uint16_t hi[4], lo[4];
#pragma unroll
                    for (int i2 = 0; i2 < 4; ++i2) split_e4m3x2(f[2 * i2] * up, f[2 * i2 + 1] * up, hi[i2], lo[i2]);
                    if (sub < kRows && r < RU) {
                        const uint2 ph = make_uint2(hi[0] | (static_cast<uint32_t>(hi[1]) << 16), hi[2] | (static_cast<uint32_t>(hi[3]) << 16));
                        const uint2 pl = make_uint2(lo[0] | (static_cast<uint32_t>(lo[1]) << 16), lo[2] | (static_cast<uint32_t>(lo[3]) << 16));
                        const int byte = el * 8;
                        uint8_t* dst;   // (NR rows on, the same swizzle: NR is a multiple of 8)
                        int step;
                        if (F::kWide && byte < 128) {
                            dst = q + r * 128 + (((byte >> 4) ^ (r & 7)) << 4) + (byte & 15);
                            step = NR * 128;
                        } else {
                            const int b2 = byte & 63;
                            dst = q + (F::kWide ? N * 128 : 0) + r * 64 + (((b2 >> 4) ^ ((r >> 1) & 3)) << 4) + (b2 & 15);
                            step = NR * 64;
                        }
                        *reinterpret_cast<uint2*>(dst) = ph;
                        *reinterpret_cast<uint2*>(dst + step) = pl;
                        if (el == 0) s_qf[buf * NR + r] = top > 0x7F7Fu ? __uint_as_float(0x7FC00000u) : down * p.scale;
                    }
                }
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(&qfull[buf]);
        }
    } else if (warp == 3) {
        // ------------------------------------------------ scales of each tile's pages
        // Eight lanes take a tile, the warp four at a time, and the next
        // four's are loaded before these are written: the loads of a table
        // entry and then of a scale that it names cost two latencies of HBM.
        const int sub = lane & 7, grp = lane >> 3;
        Walk w = it;
        int ahead = grp;   // the tile that w stands at
        auto load = [&](float& ks, float& vs) {
            ks = 0.0f;
            vs = 0.0f;
            if (ahead < ntiles) {
                const int idx = w.tile * pages_per_tile + sub;
                if (sub < pages_per_tile && (idx << p.bs_log2) < w.len[w.b]) {
                    const int page = p.tables[static_cast<int64_t>(w.b) * p.width + idx];
                    if (page >= 0 && page < p.n_pages) {
                        const int64_t at = static_cast<int64_t>(page) * p.Hkv + w.h;
                        ks = __ldg(p.k_scale + at);
                        vs = __ldg(p.v_scale + at);
                    }
                }
                for (int i = 0; i < 4; ++i) w.next();
                ahead += 4;
            }
            __syncwarp();
        };
        if (ntiles > 0)
            for (int i = 0; i < grp; ++i) w.next();
        float ks, vs;
        load(ks, vs);
        for (int i0 = 0; i0 < ntiles; i0 += 4) {
            const int i = i0 + grp, slot = i % kRing;
            float ks1, vs1;
            load(ks1, vs1);
            const bool got = i >= ntiles || mbar_wait(&cempty[slot], ((i / kRing) & 1) ^ 1, abort_flag);
            if (!__all_sync(0xFFFFFFFFu, got)) {
                attn_abort(abort_flag);
                break;
            }
            if (i < ntiles) {
                const bool on = is_scale(vs);
                s_ck[slot * 8 + sub] = on ? ks : 0.0f;
                s_lv[slot * 8 + sub] = on ? log2f(vs) : -INFINITY;
                s_iv[slot * 8 + sub] = on ? 1.0f / vs : 0.0f;
            }
            __syncwarp();
            if (i < ntiles && sub == 0) mbar_arrive(&cfull[slot]);
            ks = ks1;
            vs = vs1;
        }
    } else {
        // ------------------------------------------------ softmax: a thread per token of the tile
        const int w4 = warp & 3, t = threadIdx.x - 128;
        const uint32_t lane_off = static_cast<uint32_t>(w4 * 32) << 16;
        const int kb = t / F::kPair;   // P's byte and V's row of the token
        bool ok = true;
        // A segment's results are written after the first tile of the next:
        // its last O is complete by then, and the MMAs have work meanwhile.
        struct {
            int last, sg;         // its last tile (-1: there is none to write)
            bool began, whole;    // it began in an earlier range; it is all in this one
        } done;
        done.last = -1;
        auto finish = [&]() {   // (after a barrier: s_l and s_M are there)
            const int par = done.sg & 1;
            bool good = mbar_wait(&pvdone[done.last & 1], (done.last >> 1) & 1, abort_flag);
            __syncwarp();
            tc_fence_after();
            float o[RU];
            {
                float raw[N];
                tmem_ld<N>(tO + lane_off + par * ON + (F::kPair == 2 ? (w4 >> 1) * N : 0), raw);
                tmem_wait_ld();
                tc_fence_before();
#pragma unroll
                for (int r = 0; r < RU; ++r) o[r] = fmaf(raw[NR + r], kLoInv, raw[r]);
            }
            if constexpr (F::kPair == 2) {   // even and odd tokens' halves
                if (w4 >= 2) {
#pragma unroll
                    for (int r = 0; r < RU; ++r) s_x[r * 64 + (t & 63)] = o[r];
                }
                good = bar_all(1, 128, good);
                if (w4 < 2) {
#pragma unroll
                    for (int r = 0; r < RU; ++r) o[r] += s_x[r * 64 + t];
                }
            }
            const bool writes = F::kPair == 1 || w4 < 2;
            const int d = t;
            if constexpr (kSeveral) {
                if (s_nans[par] == static_cast<uint32_t>(done.sg + 1) && writes) {   // (rare)
                    const uint32_t key = s_nan[par * DV + d];
#pragma unroll
                    for (int r = 0; r < RU; ++r)
                        if (sees_nan<kNanBits>(key, done.sg + 1, s_lim[par * NR + r] - s_min[par]))
                            o[r] = __uint_as_float(0x7FC00000u);
                }
            }
            // lane r knows row r: its sum, its place
            const float* sl = s_l + par * 4 * RU;
            const int mr = lane % RU;
            const float sum = sl[mr] + sl[RU + mr] + sl[2 * RU + mr] + sl[3 * RU + mr];
            const float inv = sum == 0.0f ? 0.0f : __frcp_rn(sum);
            const long long row = s_row[par * NR + mr];
            // whole: the results; else a part, which attn_join_kernel takes from here
            if (done.whole) {
#pragma unroll
                for (int r = 0; r < RU; ++r) {
                    const long long at = __shfl_sync(0xFFFFFFFFu, row, r);
                    const float f = __shfl_sync(0xFFFFFFFFu, inv, r);
                    if (at >= 0 && writes) p.out[at * DV + d] = __float2bfloat16_rn(o[r] * f);
                }
                if (p.lse && t < RU && row >= 0)
                    p.lse[row] = sum == 0.0f ? -INFINITY : (s_M[par * RU + mr] - kPBits + log2f(sum)) * kLn2;
            } else {
                float* part = p.parts + (me * 2 + (done.began ? 0 : 1)) * F::kPartFloats;
                if (writes) {
#pragma unroll
                    for (int r = 0; r < RU; ++r) part[r * DV + d] = o[r];
                }
                if (t < RU) {
                    *reinterpret_cast<float2*>(part + RU * DV + 2 * t) = make_float2(s_M[par * RU + t], sum);
                    if (done.began) reinterpret_cast<long long*>(p.info + 4 + me * info_ints(RU) + 4)[t] = row;
                }
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&qempty[par]);   // the rows' constants have been read
            done.last = -1;
            return good;
        };
        // A wait that gave up in one thread only must not take that thread out:
        // the others would wait at the next barrier for good.  All 128 leave
        // together, on what a barrier says.
        bool left = false;
        for (int i = 0, sg = 0; i < ntiles || done.last >= 0; it.next_segment(), ++sg) {
        // ---- a segment, or what this range has of it; at the end a round without tiles
        const bool over = i >= ntiles;
        const int tile0 = it.tile, count = over ? 1 : min(it.nt - tile0, ntiles - i), len = it.len[it.b];
        const int qb = (sg & 1) * NR;
        if (!over) ok = mbar_wait(&qfull[sg & 1], (sg >> 1) & 1, abort_flag) && ok;
        const int least = s_min[sg & 1];
        float top_m = -INFINITY;       // the maximum of row lane % RU
        bool settled = false;          // every row has one (the same in all threads)
        float ref[RU], l[RU];          // M - kPBits of each row (0 before there is one), the token's sums
#pragma unroll
        for (int r = 0; r < RU; ++r) {
            ref[r] = 0.0f;
            l[r] = 0.0f;
        }
        for (int u = 0; u < count; ++u, ++i) {
            const int buf = i & 1, slot = i % kRing;
            if (over) {
                ok = bar_all(1, 128, ok);
            } else {
            ok = mbar_wait(&cfull[slot], (i / kRing) & 1, abort_flag) && ok;
            const int pg = slot * 8 + (t >> p.bs_log2);
            const float ck = s_ck[pg], lv = s_lv[pg], iv = s_iv[pg];
            ok = mbar_wait(&sfull[buf], (i >> 1) & 1, abort_flag) && ok;
            __syncwarp();
            tc_fence_after();
            const int tok = (tile0 + u) * 128 + t;
            float y[RU];   // the exponents x - ref
            {
                float s[N];
                tmem_ld<N>(tS + lane_off + buf * N, s);
                tmem_wait_ld();
#pragma unroll
                for (int r = 0; r < RU; ++r) y[r] = fmaf(fmaf(s[NR + r], kLoInv, s[r]), s_qf[qb + r] * ck, lv - ref[r]);
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(&sempty[buf]);
                mbar_arrive(&cempty[slot]);
            }
            if ((tile0 + u) * 128 + 128 > least) {   // some row sees only part of the tile
#pragma unroll
                for (int r = 0; r < RU; ++r)
                    if (tok >= s_lim[qb + r]) y[r] = -INFINITY;
            }
            if (lv == -INFINITY) {
#pragma unroll
                for (int r = 0; r < RU; ++r) y[r] = -INFINITY;
            }
            // The last place of hi + lo / 32 is 2^-14, and thousands of probabilities below half of that, next to a
            // large one, would all become 0 (or, a little above, be rounded the same way).  So what lo is rounded
            // from is shifted by up to half a place either way, by the golden ratio's multiples modulo 1, which lie
            // evenly in any run of tokens: the errors of like probabilities cancel.  (A 0 stays 0.)
            uint32_t dither;   // ten bits of the multiple m in [0, 1) as (1 + m) 2^-9, less 1.5 * 2^-9
            asm("sub.f16x2 %0, %1, %2;" : "=r"(dither) : "r"(((static_cast<uint32_t>(tok) * 0x9E3779B9u) >> 22) * 0x10001u + 0x18001800u), "r"(0x1A001A00u));
            // The maxima stay while every probability fits: then one barrier,
            // which also says so, is all that the warps share of a tile.  Not
            // before every row has a maximum, though: one that has seen nothing
            // so far (its tiles' pages are left out) has to get it with the
            // first token that it sees, however small that one's exponent.
            float most = y[0];
#pragma unroll
            for (int r = 1; r < RU; ++r) most = fmaxf(most, y[r]);
            if (!bar_all(1, 128, ok && settled && !(most > kMostBits))) {
                // the true maxima: lane r of each warp gives its warp's, lane l
                // of every warp then joins those of row l % RU
                float mine = 0.0f;
#pragma unroll
                for (int r = 0; r < RU; ++r) {
                    const float m = warp_max(y[r] + ref[r]);
                    if (lane == r) mine = m;
                }
                if (lane < RU) s_max[w4 * RU + lane] = mine;
                ok = bar_all(1, 128, ok);
                if (!ok) {
                    left = true;
                    break;
                }
                float top = s_max[lane % (4 * RU)];
#pragma unroll
                for (int k = 32; k < 4 * RU; k += 32) top = fmaxf(top, s_max[k + lane]);
#pragma unroll
                for (int o = RU; o < 4 * RU && o < 32; o <<= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
                const bool grows = top > top_m;
                const float my_fac = grows ? ex2(top_m - top) : 1.0f;   // 0 for the first
                if (grows) top_m = top;
                settled = __all_sync(0xFFFFFFFFu, top_m != -INFINITY) != 0;
                float fac[RU];
#pragma unroll
                for (int r = 0; r < RU; ++r) {
                    fac[r] = __shfl_sync(0xFFFFFFFFu, my_fac, r);
                    const float m = __shfl_sync(0xFFFFFFFFu, top_m, r);
                    const float now = m == -INFINITY ? 0.0f : m - kPBits;
                    y[r] += ref[r] - now;
                    ref[r] = now;
                    l[r] *= fac[r];
                }
                if (u > 0) {   // O in the old unit: bring it to the new one
                    ok = mbar_wait(&pvdone[buf ^ 1], ((i - 1) >> 1) & 1, abort_flag) && ok;
                    __syncwarp();
                    tc_fence_after();
#pragma unroll
                    for (int c = 0; c < ON; c += 16) {
                        float o[16];
                        tmem_ld<16>(tO + lane_off + (sg & 1) * ON + c, o);
                        tmem_wait_ld();
#pragma unroll
                        for (int e = 0; e < 16; ++e)
                            if ((c + e) % NR < RU) o[e] *= fac[(c + e) % NR % RU];
                        tmem_st16(tO + lane_off + (sg & 1) * ON + c, o);
                    }
                    tmem_wait_st();
                }
            }
            if (i >= 2) ok = mbar_wait(&pvdone[buf], ((i - 2) >> 1) & 1, abort_flag) && ok;   // P is free
            uint8_t* P = sP + buf * F::kPBytes + (F::kPair == 2 ? (t & 1) * N * 128 : 0);
            int kx = kb;   // (new for the compiler at each tile: the rows' eight addresses, kept through the loop, spill)
            asm volatile("" : "+r"(kx));
            // P, split, in the layout the MMA reads: row n of 128 bytes, byte = token (or pair)
#pragma unroll
            for (int r = 0; r < RU; r += 2) {
                const bool two = r + 1 < RU;
                const int r1 = two ? r + 1 : r;
                const float p0 = ex2(y[r]);
                const float p1 = two ? ex2(y[r1]) : 0.0f;
                uint16_t hi, lo;
                split_e4m3x2(p0, p1, hi, lo, dither);
                const int a0 = r * 128 + (kx ^ ((r & 7) << 4));
                l[r] = fmaf(p0, iv, l[r]);
                P[a0] = static_cast<uint8_t>(hi);
                P[NR * 128 + a0] = static_cast<uint8_t>(lo);
                if (two) {
                    const int a1 = r1 * 128 + (kx ^ ((r1 & 7) << 4));
                    l[r1] = fmaf(p1, iv, l[r1]);
                    P[a1] = static_cast<uint8_t>(hi >> 8);
                    P[NR * 128 + a1] = static_cast<uint8_t>(lo >> 8);
                }
            }
            // V of a token that is not there may hold anything, a NaN too: zero it.  One that only some rows see
            // keeps its numbers (note_nans).
            if (tok >= (kSeveral ? least : len) || lv == -INFINITY) {
                const int st = i % SV;
                ok = mbar_wait(&vfull[st], (i / SV) & 1, abort_flag) && ok;
                uint8_t* vr = sV + st * F::kVBytes + kb * 128;
                auto chunk = [&](int c) {
                    return reinterpret_cast<uint4*>(vr + (((c + (F::kPair == 2 ? (t & 1) * 4 : 0)) ^ (kb & 7)) << 4));
                };
                if (!kSeveral || tok >= len || lv == -INFINITY) {
#pragma unroll
                    for (int c = 0; c < DV / 16; ++c) *chunk(c) = make_uint4(0, 0, 0, 0);
                } else {
#pragma unroll 1
                    for (int c = 0; c < DV / 16; ++c) {
                        const uint4 v = *chunk(c);
                        if (e4m3_nans(v) == 0) continue;
                        *chunk(c) = without_nans(v);
                        note_nans(v, s_nan + (sg & 1) * DV + c * 16, nan_key<kNanBits>(sg + 1, min(tok - least, (1 << kNanBits) - 1)));
                        s_nans[sg & 1] = sg + 1;
                    }
                }
            }
            fence_proxy_async_smem();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&pfull[buf]);
            }
            if (u == 0 && done.last >= 0) ok = finish() && ok;
        }
        if (left || over) break;

        // ---- the segment's end: sums over the tokens
        int row = 0;
#pragma unroll
        for (int o = 16, c = RU; o >= 1; o >>= 1) {
            if (c > 1) {   // half the rows stay here, the others' sums go to the partner lane
                c >>= 1;
                const bool up = (lane & o) != 0;
#pragma unroll
                for (int r = 0; r < RU / 2; ++r) {
                    if (r < c) {
                        const float give = up ? l[r] : l[r + c];
                        const float keep = up ? l[r + c] : l[r];
                        l[r] = keep + __shfl_xor_sync(0xFFFFFFFFu, give, o);
                    }
                }
                row += up ? c : 0;
            } else {
                l[0] += __shfl_xor_sync(0xFFFFFFFFu, l[0], o);
            }
        }
        s_l[((sg & 1) * 4 + w4) * RU + row] = l[0];   // (lanes that share a row hold the same sum)
        if (w4 == 0 && lane < RU) s_M[(sg & 1) * RU + lane] = top_m;
        done.last = i - 1;
        done.sg = sg;
        done.began = tile0 > 0;
        done.whole = tile0 == 0 && count == it.nt;
        }
        if (!ok) attn_abort(abort_flag);
    }

    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 1) tmem_dealloc(tmem, F::kTmem);
}

// Joins the parts of the segments that the cut went through:
//   out = sum_i 2^(M_i - M) O_i / sum_i 2^(M_i - M) l_i,  M = max_i M_i,
// in the order of the ranges, so that results do not depend on timing.  It is
// a launch of its own because a part's epilogue must not wait: publishing a
// part and finding out whether it was the last (a fence, an atomic, two more
// loads) cost the softmax warps 6 us of loaded HBM latency each.
// A CTA stands at the begin of range r, for up to 8 of the rows (the CTAs are few:
// starting them costs more than what they do, 512 threads for each 4 rows 3 us); the segment
// that crosses it is joined by the first such range's.  Its warps share the
// parts of a row; the loads of a part's M, l and O are issued together, so the
// kernel is three latencies long: the record, the parts, the store.
template <int DV, int RU>
__global__ void __launch_bounds__(kJoinThreads) attn_join_kernel(const AttnParams p) {
    griddep_launch_dependents();
    griddep_wait();
    constexpr int kPart = part_floats(RU, DV);
    constexpr int W = kJoinThreads / 32;
    constexpr int kRows = RU < 8 ? RU : 8;      // rows of a CTA
    constexpr int kSplit = W / kRows;           // warps that share a row, each with every kSplit-th part
    constexpr int kV = DV / 32;                 // values per lane
    constexpr int kU = 16;                      // parts whose loads are in flight together
    __shared__ float s_m[W], s_l[W], s_o[W][DV];
    const int r1 = blockIdx.x + 1, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int32_t* info = p.info + 4 + static_cast<int64_t>(r1) * info_ints(RU);
    const int r = blockIdx.y * kRows + warp % kRows, share = warp / kRows;
    const int2 span = __ldcg(reinterpret_cast<const int2*>(info));
    const long long at = __ldcg(reinterpret_cast<const long long*>(info + 4) + r);
    const int ranges = __ldcg(p.info);
    if (r1 >= ranges || span.x != r1 - 1) return;
    const int n = span.y - span.x + 1;
    const float* first = p.parts + (static_cast<int64_t>(span.x) * 2 + 1) * kPart;   // the segment's begin: its range's last slot
    const float* rest = p.parts + static_cast<int64_t>(r1) * 2 * kPart;             // then the first slots of the next ranges
    auto part = [&](int c) { return c == 0 ? first : rest + static_cast<int64_t>(c - 1) * 2 * kPart; };
    float m = -INFINITY, l = 0.0f, o[kV];
#pragma unroll
    for (int e = 0; e < kV; ++e) o[e] = 0.0f;
    auto merge = [&](float m2, float l2, const float (&o2)[kV]) {
        const float top = fmaxf(m, m2), ref = top == -INFINITY ? 0.0f : top;
        const float a = ex2(m - ref), b = ex2(m2 - ref);
        l = l * a + l2 * b;
#pragma unroll
        for (int e = 0; e < kV; ++e) o[e] = o[e] * a + o2[e] * b;
        m = top;
    };
    for (int c0 = share; c0 < n; c0 += kSplit * kU) {
        float2 ml[kU];
        float v[kU][kV];
#pragma unroll
        for (int u = 0; u < kU; ++u) {
            if (c0 + u * kSplit >= n) break;
            const float* src = part(c0 + u * kSplit);
            ml[u] = __ldcg(reinterpret_cast<const float2*>(src + RU * DV) + r);
            if constexpr (kV == 4) {
                const float4 q = __ldcg(reinterpret_cast<const float4*>(src + r * DV) + lane);
                v[u][0] = q.x; v[u][1] = q.y; v[u][2] = q.z; v[u][3] = q.w;
            } else {
                const float2 q = __ldcg(reinterpret_cast<const float2*>(src + r * DV) + lane);
                v[u][0] = q.x; v[u][1] = q.y;
            }
        }
#pragma unroll
        for (int u = 0; u < kU; ++u) {
            if (c0 + u * kSplit >= n) break;
            merge(ml[u].x, ml[u].y, v[u]);
        }
    }
    if (lane == 0) {
        s_m[warp] = m;
        s_l[warp] = l;
    }
#pragma unroll
    for (int e = 0; e < kV; ++e) s_o[warp][lane * kV + e] = o[e];
    __syncthreads();
    // (after a wait that gave up, the record may be another call's)
    if (share != 0 || at < 0 || at >= p.T * p.Hq) return;
#pragma unroll
    for (int k = 1; k < kSplit; ++k) {
        float v[kV];
#pragma unroll
        for (int e = 0; e < kV; ++e) v[e] = s_o[warp + k * kRows][lane * kV + e];
        merge(s_m[warp + k * kRows], s_l[warp + k * kRows], v);
    }
    const float inv = l == 0.0f ? 0.0f : __frcp_rn(l);
    uint32_t* dst = reinterpret_cast<uint32_t*>(p.out + at * DV) + lane * (kV / 2);
#pragma unroll
    for (int e = 0; e < kV; e += 2) {
        const __nv_bfloat162 b = __floats2bfloat162_rn(o[e] * inv, o[e + 1] * inv);
        dst[e / 2] = *reinterpret_cast<const uint32_t*>(&b);
    }
    if (p.lse && lane == 0) p.lse[at] = l == 0.0f ? -INFINITY : (m - kPBits + log2f(l)) * kLn2;
}

template <int DK, int DV, int RU, bool kSeveral>
cudaError_t launch(const AttnMaps& m, const AttnParams& p, int sms, cudaStream_t st) {
    using F = Few<DK, DV, RU, kSeveral>;
    static int configured[64] = {};
    int dev = 0;
    cudaGetDevice(&dev);
    if (dev >= 64 || !configured[dev]) {
        const cudaError_t e = cudaFuncSetAttribute(attn_few_kernel<DK, DV, RU, kSeveral>, cudaFuncAttributeMaxDynamicSharedMemorySize, F::kSmem);
        if (e != cudaSuccess) return e;
        if (dev < 64) configured[dev] = 1;
    }
    const int ctas = sms * F::kBlocks;
    const cudaError_t e = launch_pdl(attn_few_kernel<DK, DV, RU, kSeveral>, dim3(ctas), dim3(kThreads), F::kSmem, st, m.k0, m.k1, m.v, p);
    if (e != cudaSuccess) return e;
    // at most so many ranges: those of the longest lengths the tables can hold
    const int64_t positions = static_cast<int64_t>(p.B) * ((static_cast<int64_t>(p.width) << p.bs_log2) / 128 + 1 + F::kSegment) * p.Hkv *
                          ((p.few_rows + RU - 1) / RU);
    const int64_t ranges = std::min<int64_t>(positions, ctas);
    if (ranges < 2) return cudaSuccess;
    return launch_pdl(attn_join_kernel<DV, RU>, dim3(static_cast<unsigned>(ranges - 1), RU < 8 ? 1 : RU / 8), dim3(kJoinThreads), 0, st, p);
}

template <int DK, int DV, bool kSeveral>
cudaError_t launch_rows(int ru, const AttnMaps& m, const AttnParams& p, int sms, cudaStream_t st) {
    switch (ru) {
        case 1: return launch<DK, DV, 1, kSeveral>(m, p, sms, st);
        case 4: return launch<DK, DV, 4, kSeveral>(m, p, sms, st);
        case 8: return launch<DK, DV, 8, kSeveral>(m, p, sms, st);
        case 16: return launch<DK, DV, 16, kSeveral>(m, p, sms, st);
    }
    return launch<DK, DV, 32, kSeveral>(m, p, sms, st);
}

size_t info_bytes(int ru, int sms) { return (4 + static_cast<size_t>(sms) * few_blocks(ru) * info_ints(ru)) * sizeof(int32_t); }

}  // namespace

// The heads that share a cache head, or twice those where requests may have
// several queries.
int few_rows_per_tile(int G, bool ragged) {
    const int rows = ragged ? 2 * G : G;
    return rows <= 1 ? 1 : rows <= 4 ? 4 : rows <= 8 ? 8 : rows <= 16 ? 16 : 32;
}

size_t few_workspace(int ru, int dv, int sms) {
    return info_bytes(ru, sms) + static_cast<size_t>(sms) * few_blocks(ru) * 2 * part_floats(ru, dv) * sizeof(float);
}

void few_workspace_split(AttnParams& p, void* base, int ru, int sms) {
    p.info = static_cast<int32_t*>(base);
    p.parts = reinterpret_cast<float*>(static_cast<uint8_t*>(base) + info_bytes(ru, sms));
}

cudaError_t launch_few(int dk, int ru, const AttnMaps& m, const AttnParams& p, int sms, cudaStream_t st) {
    auto of = [&](auto several) {
        constexpr bool S = decltype(several)::value;
        return dk == 64    ? launch_rows<64, 64, S>(ru, m, p, sms, st)
               : dk == 128 ? launch_rows<128, 128, S>(ru, m, p, sms, st)
                           : launch_rows<192, 128, S>(ru, m, p, sms, st);
    };
    return p.offsets ? of(std::true_type()) : of(std::false_type());
}
int few_read_and_clear_status(cudaStream_t st) { return read_and_clear_attention_status(st); }
bool few_set_wait_limit(long long cycles) { return set_attention_wait_limit(cycles); }

}  // namespace fp8bs
