// kvcache.cu -- the paged 8-bit key/value cache between the FP8 projections:
//   kv_plan     block tables, slot maps and positions of one step, built on
//               the GPU from the requests' lengths (no host round trip)
//   kv_append   bf16 keys and values -> e4m3 codes in the requests' pages,
//               one fp32 scale per (page, head)
//
// A page holds block_size tokens (a power of two) of every head: codes
// [n_pages, H, block_size, d], scales [n_pages, H].  Token position p of
// request b lives in page tables[b, p / block_size] at p % block_size; its
// slot is page * block_size + p % block_size (64 bits: a cache of one narrow
// head passes 2^31 tokens).
#include "common.cuh"

#include <algorithm>
#include <type_traits>

namespace fp8bs {
namespace {

// ---------------------------------------------------------------- plan
constexpr int kPlanThreads = 1024;
constexpr int kPlanWarps = kPlanThreads / 32;
constexpr int kPlanMaxB = 8192;
constexpr int kPlanPer = kPlanMaxB / kPlanThreads;   // requests of a thread, at most
constexpr int kPlanTok = 4;   // consecutive tokens per thread (16-byte stores)

struct PlanParams {
    const int32_t *past, *fresh, *free_pages, *used;
    int32_t *tables, *lens, *offsets, *positions, *used_out;
    int64_t* slots;
    int64_t T;
    int32_t B, n_free, width, bs_log2, vec;
};

// The two 32-bit sums of a pair, each held at 2^31 - 1 (lengths are device
// data: whatever they hold, the sums stay monotone and every index below
// stays within its array).
__device__ __forceinline__ unsigned long long pack_sums(int pages, int tokens) {
    return (static_cast<unsigned long long>(static_cast<uint32_t>(pages)) << 32) | static_cast<uint32_t>(tokens);
}
__device__ __forceinline__ unsigned long long add_sums(unsigned long long a, unsigned long long b) {
    const uint32_t lo = static_cast<uint32_t>(a) + static_cast<uint32_t>(b);
    const uint32_t hi = static_cast<uint32_t>(a >> 32) + static_cast<uint32_t>(b >> 32);
    return pack_sums(static_cast<int>(min(hi, 0x7FFFFFFFu)), static_cast<int>(min(lo, 0x7FFFFFFFu)));
}

// Every CTA scans the requests itself (B <= 8192: two small arrays, read from
// L2) and then serves its slice of the tokens and of the newly taken pages,
// so one launch with no communication between CTAs does it all.  Latency is
// what it costs (lengths, sums over the CTA, a page's number, the stores): a
// thread's loads are issued together (read one after the other between stores,
// 4096 requests took 29.8 us), and a call takes 9.3 us for 64 requests and for
// 4096, which is the host's time for it; alone on the GPU, 4 us.
//   need[b]  = pages(past + new) - pages(past), 0 where the table row is too narrow
//   granted  = the running sum of needs up to b is within the free list
//              (monotone, so the granted requests' pages are consecutive in it)
// The smem arrays hold the running sums: s_tok (tokens before b) and s_need
// (pages before b); a request that is not granted has the sign bit of
// s_state set.
__global__ void __launch_bounds__(kPlanThreads) kv_plan_kernel(const PlanParams p) {
    griddep_launch_dependents();
    griddep_wait();
    extern __shared__ int32_t plan_smem[];
    int32_t* s_tok = plan_smem;                 // [B + 1]
    int32_t* s_need = s_tok + p.B + 1;          // [B + 1]
    int32_t* s_past = s_need + p.B + 1;         // [B]: past length, or -1 - past where not granted
    __shared__ unsigned long long s_warp[kPlanWarps];
    __shared__ int s_granted;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int bs_mask = (1 << p.bs_log2) - 1;
    const int per = (p.B + kPlanThreads - 1) / kPlanThreads;   // requests per thread, consecutive
    const int lo = min(p.B, tid * per), n = min(p.B, lo + per) - lo;
    // Everything of a thread's requests stays in registers, all loads issued together.
    int past[kPlanPer], fresh[kPlanPer], need[kPlanPer];
#pragma unroll
    for (int i = 0; i < kPlanPer; ++i) {
        past[i] = i < n ? p.past[lo + i] : 0;
        fresh[i] = i < n ? p.fresh[lo + i] : 0;
    }
    const int used = max(0, min(*p.used, p.n_free));
    const int avail = p.n_free - used;
    if (tid == 0) s_granted = 0;
    // sums of this thread's requests (tokens in the low word, pages in the high)
    unsigned long long sum = 0;
#pragma unroll
    for (int i = 0; i < kPlanPer; ++i) {
        past[i] = max(0, past[i]);
        fresh[i] = max(0, fresh[i]);
        const int64_t total = static_cast<int64_t>(past[i]) + fresh[i];
        const int64_t now = (total + bs_mask) >> p.bs_log2, old = (static_cast<int64_t>(past[i]) + bs_mask) >> p.bs_log2;
        const bool fits = now <= p.width;
        need[i] = fits ? static_cast<int>(now - old) : 0;
        if (!fits) past[i] = -1 - past[i];
        if (i < n) sum = add_sums(sum, pack_sums(need[i], fresh[i]));
    }
    unsigned long long inc = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const unsigned long long up = __shfl_up_sync(0xFFFFFFFFu, inc, o);
        if (lane >= o) inc = add_sums(inc, up);
    }
    if (lane == 31) s_warp[warp] = inc;
    __syncthreads();
    unsigned long long run = __shfl_up_sync(0xFFFFFFFFu, inc, 1);
    if (lane == 0) run = 0;
    for (int w = 0; w < warp; ++w) run = add_sums(run, s_warp[w]);
    int granted = 0;
#pragma unroll
    for (int i = 0; i < kPlanPer; ++i) {
        if (i >= n) break;
        const int b = lo + i;
        s_tok[b] = static_cast<int>(run & 0xFFFFFFFFu);
        s_need[b] = static_cast<int>(run >> 32);
        if (blockIdx.x == 0) p.offsets[b] = s_tok[b];
        run = add_sums(run, pack_sums(need[i], fresh[i]));
        const int incl = static_cast<int>(run >> 32);
        const bool room = incl <= avail;
        if (room) granted = incl;
        if (past[i] >= 0 && !room && need[i] != 0) past[i] = -1 - past[i];
        s_past[b] = past[i];
        if (blockIdx.x == 0) p.lens[b] = past[i] >= 0 ? past[i] + fresh[i] : -1 - past[i];
        if (b == p.B - 1) {
            s_tok[p.B] = static_cast<int>(run & 0xFFFFFFFFu);
            s_need[p.B] = static_cast<int>(run >> 32);
        }
    }
    atomicMax(&s_granted, granted);
    __syncthreads();
    const int total_tok = s_tok[p.B], total_need = min(s_need[p.B], s_granted);
    if (blockIdx.x == 0 && tid == 0) {
        p.offsets[p.B] = total_tok;
        *p.used_out = used + s_granted;
    }
    // last request b with a[b] <= i (requests with nothing are skipped over)
    auto owner = [&](const int32_t* a, int i) {
        int l = 0, r = p.B;
        while (r - l > 1) {
            const int m = (l + r) >> 1;
            if (a[m] <= i) l = m; else r = m;
        }
        return l;
    };
    const int64_t stride = static_cast<int64_t>(gridDim.x) * kPlanThreads;
    const int64_t me = static_cast<int64_t>(blockIdx.x) * kPlanThreads + tid;
    // the pages taken from the free list: entry e goes to its request's row
    for (int64_t e = me; e < total_need; e += stride) {
        const int b = owner(s_need, static_cast<int>(e));
        const int past = s_past[b];
        const int old = (past + bs_mask) >> p.bs_log2;
        p.tables[static_cast<int64_t>(b) * p.width + old + (static_cast<int>(e) - s_need[b])] = p.free_pages[used + e];
    }
    // the tokens
    for (int64_t t0 = me * kPlanTok; t0 < p.T; t0 += stride * kPlanTok) {
        long long slot[kPlanTok];
        int pos[kPlanTok];
        int b = t0 < total_tok ? owner(s_tok, static_cast<int>(t0)) : p.B;
        int last = -1, last_page = 0;   // the page of the previous token
#pragma unroll
        for (int i = 0; i < kPlanTok; ++i) {
            const int64_t t = t0 + i;
            slot[i] = -1;
            pos[i] = -1;
            if (t >= total_tok || t >= p.T) continue;
            while (b + 1 < p.B && s_tok[b + 1] <= t) {
                ++b;
                last = -1;
            }
            const int past = s_past[b];
            if (past < 0) continue;
            const int at = past + static_cast<int>(t - s_tok[b]), idx = at >> p.bs_log2;
            if (idx != last) {
                const int old = (past + bs_mask) >> p.bs_log2;
                last_page = idx < old ? p.tables[static_cast<int64_t>(b) * p.width + idx]
                                      : p.free_pages[used + s_need[b] + idx - old];
                last = idx;
            }
            slot[i] = (static_cast<long long>(last_page) << p.bs_log2) + (at & bs_mask);
            pos[i] = at;
        }
        if (p.vec && t0 + kPlanTok <= p.T) {
            longlong2* d = reinterpret_cast<longlong2*>(p.slots + t0);
            d[0] = make_longlong2(slot[0], slot[1]);
            d[1] = make_longlong2(slot[2], slot[3]);
            if (p.positions) *reinterpret_cast<int4*>(p.positions + t0) = make_int4(pos[0], pos[1], pos[2], pos[3]);
        } else {
            for (int i = 0; i < kPlanTok && t0 + i < p.T; ++i) {
                p.slots[t0 + i] = slot[i];
                if (p.positions) p.positions[t0 + i] = pos[i];
            }
        }
    }
}

// ---------------------------------------------------------------- append
constexpr int kAppThreads = 128;
constexpr int kAppRows = 8;   // rows of heads that a warp takes together of a run of few tokens
constexpr int kAppFill = 3;

struct AppendParams {
    const uint16_t* x[2];     // K, V
    int64_t ts[2], hs[2];     // token and head strides (elements)
    uint8_t* cache[2];
    float* scale[2];
    const int64_t* slots;
    int64_t T, n_slots;
    int32_t H, d[2], inv[2], bs_log2, window, shares, ctas, rows_log2, ue8m0;
};

struct Run {   // a stretch of tokens in consecutive slots of one page
    int64_t t;         // its first token
    int64_t page;
    int off, n;
};

__device__ __forceinline__ uint32_t quant_div2(float a, float b, float s) {
    return f32x2_to_e4m3x2(__fdiv_rn(a, s), __fdiv_rn(b, s));
}

// The larger of each half (bf16, a NaN loses), of magnitudes.
__device__ __forceinline__ uint32_t max_bf16x2(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("max.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}
__device__ __forceinline__ uint32_t max_abs_bf16x8(uint32_t m, const uint4& v) {
    constexpr uint32_t kAbs = 0x7FFF7FFFu;
    return max_bf16x2(max_bf16x2(m, max_bf16x2(v.x & kAbs, v.y & kAbs)), max_bf16x2(v.z & kAbs, v.w & kAbs));
}

// 8 codes of 8 bf16.  kFp32, kUe8m0: by the scale's reciprocal, exact for
// finite values; kDivide: the division itself, which takes +-inf to +-448.
enum { kFp32, kUe8m0, kDivide };
template <int MODE>
__device__ __forceinline__ uint2 codes8(const uint4& v, float s, float r) {
    if (MODE == kDivide) {
        float f[8];
        unpack_bf16x8(v, f);
        return make_uint2(quant_div2(f[0], f[1], s) | (quant_div2(f[2], f[3], s) << 16),
                          quant_div2(f[4], f[5], s) | (quant_div2(f[6], f[7], s) << 16));
    }
    float nx[8];
    unpack_bf16x8_neg(v, nx);
    return quant8n<MODE == kUe8m0>(nx, s, r);
}

// The chunks (16 bytes of x) of one head's run, as one lane meets them: 32
// chunks further at each step, without a division.
struct ChunkWalk {
    const uint16_t* at;
    int64_t step, wrap;   // elements: a step, and what a step into the next token adds
    int rem, by, chunks;
    __device__ __forceinline__ uint4 next(bool on) {
        const uint4 v = on ? __ldg(reinterpret_cast<const uint4*>(at)) : make_uint4(0, 0, 0, 0);
        at += step;
        rem += by;
        if (rem >= chunks) {
            rem -= chunks;
            at += wrap;
        }
        return v;
    }
};

// One warp appends a run for up to ROWS << sub_log2 heads from h0 on (nh of
// them).  A head's chunks lie over 32 >> sub_log2 lanes, R chunks a lane;
// with kLong a run may pass the registers, and what does is
// read again.  Lane j holds the amax
// and the scale of head h0 + j.
// The scale: block_scale of the run's largest finite magnitude, and at least
// the page's scale when the page holds earlier tokens; if that grows the
// scale, the earlier tokens' codes are written again for it.
template <int R, int ROWS, bool kLong>
__device__ __forceinline__ void append_heads(const AppendParams& p, int which, const Run& run, int h0, int nh,
                                             int sub_log2) {
    const int lane = threadIdx.x & 31;
    const int d = p.d[which], chunks = d >> 3, total = run.n * chunks;
    const int lanes = 32 >> sub_log2, mine = lane >> (5 - sub_log2), c_lane = lane & (lanes - 1);
    const int64_t ts = p.ts[which], hs = p.hs[which];
    const uint16_t* x = p.x[which] + run.t * ts + h0 * hs;
    float* scale = p.scale[which] + run.page * p.H + h0;
    uint8_t* tiles = p.cache[which] + ((run.page * p.H + h0) << p.bs_log2) * d;   // a head's tile after the other's
    const int64_t tile = static_cast<int64_t>(d) << p.bs_log2;
    const float held = run.off > 0 && lane < nh ? scale[lane] : 0.0f;
    // chunk c of a head: token c / chunks (by the reciprocal: c < 2^14)
    auto walk = [&](int h, int c) {
        const int tok = static_cast<int>((static_cast<uint32_t>(c) * static_cast<uint32_t>(p.inv[which])) >> 21);
        const int rem = c - tok * chunks, q = static_cast<int>((32u * static_cast<uint32_t>(p.inv[which])) >> 21);
        return ChunkWalk{x + h * hs + tok * ts + rem * 8, q * ts + (32 - q * chunks) * 8, ts - chunks * 8, rem,
                         32 - q * chunks, chunks};
    };
    uint4 reg[ROWS][R];
    if (R == 1) {
        const uint16_t* at = x + mine * hs + (walk(0, c_lane).at - x);
        const int64_t step = hs << sub_log2;
#pragma unroll
        for (int i = 0; i < ROWS; ++i) {
            const bool on = (i << sub_log2) + mine < nh && c_lane < total;
            reg[i][0] = on ? __ldg(reinterpret_cast<const uint4*>(at)) : make_uint4(0, 0, 0, 0);
            at += step;
        }
    } else {
#pragma unroll
        for (int i = 0; i < ROWS; ++i) {
            ChunkWalk w = walk(i, lane);
#pragma unroll
            for (int j = 0; j < R; ++j) reg[i][j] = w.next(i < nh && j * 32 + lane < total);
        }
    }
    float amax = 0.0f;
    if constexpr (R == 1) {
        // all rows' maxima together: each step hands half of the rows to the other lanes, until a lane has one row
        static_assert(ROWS == 8, "three steps");
        uint32_t m[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) m[i] = max_abs_bf16x8(0, reg[i][0]);
        int o = lanes >> 1;
#pragma unroll
        for (int n = 4; n >= 1; n >>= 1, o >>= 1) {
            const bool up = (lane & o) != 0;
#pragma unroll
            for (int i = 0; i < n; ++i) {
                const uint32_t give = up ? m[i] : m[i + n], keep = up ? m[i + n] : m[i];
                m[i] = max_bf16x2(keep, __shfl_xor_sync(0xFFFFFFFFu, give, o));
            }
        }
        for (; o >= 1; o >>= 1) m[0] = max_bf16x2(m[0], __shfl_xor_sync(0xFFFFFFFFu, m[0], o));
        // row i's is with the lanes from i lanes / 8 on
        const uint32_t mine_max = __shfl_sync(0xFFFFFFFFu, m[0], ((lane & ((1 << sub_log2) - 1)) << (5 - sub_log2)) +
                                                                     (((lane >> sub_log2) & 7) << (2 - sub_log2)));
        if ((lane >> sub_log2) < 8) amax = __uint_as_float(max(mine_max >> 16, mine_max & 0xFFFFu) << 16);
    }
#pragma unroll
    for (int i = 0; i < (R == 1 ? 0 : ROWS); ++i) {
        uint32_t m = 0;
#pragma unroll
        for (int j = 0; j < R; ++j) m = max_abs_bf16x8(m, reg[i][j]);
        if (kLong && total > R * 32) {
            ChunkWalk w = walk(i, R * 32 + lane);
            for (int c0 = R * 32 + lane; c0 < total; c0 += 32 * 8) {
                uint4 v[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) v[j] = w.next(c0 + j * 32 < total);
#pragma unroll
                for (int j = 0; j < 8; ++j) m = max_abs_bf16x8(m, v[j]);
            }
        }
#pragma unroll
        for (int o = 16; o >= 1; o >>= 1)
            if (o < lanes) m = max_bf16x2(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
        m = __shfl_sync(0xFFFFFFFFu, m, (lane & ((1 << sub_log2) - 1)) << (5 - sub_log2));
        if ((lane >> sub_log2) == i) amax = __uint_as_float(max(m >> 16, m & 0xFFFFu) << 16);
    }
    const unsigned infs = __ballot_sync(0xFFFFFFFFu, isinf(amax));
    for (unsigned left = infs; left; left &= left - 1) {   // an infinity does not set the scale: the finite values only
        const int h = __ffs(left) - 1;
        float a = 0.0f;
        ChunkWalk w = walk(h, lane);
        for (int c = lane; c < total; c += 32) {
            float f[8];
            unpack_bf16x8(w.next(true), f);
#pragma unroll
            for (int i = 0; i < 8; ++i) a = fmaxf(a, isinf(f[i]) ? 0.0f : fabsf(f[i]));
        }
#pragma unroll
        for (int o = 16; o >= 1; o >>= 1) a = fmaxf(a, __shfl_xor_sync(0xFFFFFFFFu, a, o));
        if (lane == h) amax = a;
    }
    const float want = block_scale(amax, p.ue8m0 != 0);
    const bool grow = want > held;
    const float s = grow ? want : held;
    if (lane < nh && (grow || run.off == 0)) scale[lane] = s;
    // the earlier tokens' codes for a scale that grew
    for (unsigned left = __ballot_sync(0xFFFFFFFFu, lane < nh && run.off > 0 && grow); left; left &= left - 1) {
        const int h = __ffs(left) - 1;
        const float was = __shfl_sync(0xFFFFFFFFu, held, h), now = __shfl_sync(0xFFFFFFFFu, s, h);
        uint4* w = reinterpret_cast<uint4*>(tiles + h * tile);
        const int n16 = run.off * d / 16;
        for (int c0 = lane; c0 < n16; c0 += 32 * 4) {
            uint4 v[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) v[j] = c0 + j * 32 < n16 ? w[c0 + j * 32] : make_uint4(0, 0, 0, 0);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                uint32_t u[4] = {v[j].x, v[j].y, v[j].z, v[j].w};
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float2 a = e4m3x2_to_f32x2(static_cast<uint16_t>(u[i] & 0xFFFFu));
                    const float2 b = e4m3x2_to_f32x2(static_cast<uint16_t>(u[i] >> 16));
                    u[i] = quant_div2(__fmul_rn(a.x, was), __fmul_rn(a.y, was), now) |
                           (quant_div2(__fmul_rn(b.x, was), __fmul_rn(b.y, was), now) << 16);
                }
                if (c0 + j * 32 < n16) w[c0 + j * 32] = make_uint4(u[0], u[1], u[2], u[3]);
            }
        }
    }
    const float r = __frcp_rn(s);
    auto store = [&](auto mode) {
        constexpr int MODE = decltype(mode)::value;
        uint8_t* dst = tiles + mine * tile + static_cast<int64_t>(run.off) * d + c_lane * 8;
        const int64_t step = tile << sub_log2;
#pragma unroll
        for (int i = 0; i < ROWS; ++i) {
            const int h = (i << sub_log2) + mine;
            const float s_h = __shfl_sync(0xFFFFFFFFu, s, h & 31), r_h = __shfl_sync(0xFFFFFFFFu, r, h & 31);
#pragma unroll
            for (int j = 0; j < R; ++j)
                if (h < nh && j * 32 + c_lane < total)
                    *reinterpret_cast<uint2*>(dst + j * 256) = codes8<MODE>(reg[i][j], s_h, r_h);
            if (kLong && total > R * 32) {
                ChunkWalk w = walk(i, R * 32 + lane);
                for (int c0 = R * 32 + lane; c0 < total; c0 += 32 * 8) {
                    uint4 v[8];
#pragma unroll
                    for (int j = 0; j < 8; ++j) v[j] = w.next(c0 + j * 32 < total);
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        if (c0 + j * 32 < total)
                            *reinterpret_cast<uint2*>(dst + (c0 - lane + j * 32) * 8) = codes8<MODE>(v[j], s_h, r_h);
                }
            }
            dst += step;
        }
    };
    if (infs)
        store(std::integral_constant<int, kDivide>());
    else if (p.ue8m0 && __all_sync(0xFFFFFFFFu, lane >= nh || (__float_as_uint(s) & 0x007FFFFFu) == 0u))
        // (a page's scale that stays need not be a power of two)
        store(std::integral_constant<int, kUe8m0>());
    else
        store(std::integral_constant<int, kFp32>());
}

// Bound by HBM, or by what is in flight: a warp first needs its slots, then
// the values and the page's scale, and only then has something to store.  So
// every warp asks for as much as its registers hold at once: the run of a long
// prompt, or eight rows of heads of a single token.  Prompts (18000 tokens,
// 8 heads of 128, pages of 32): 33 us, 4.6 TB/s; 64-token windows of one warp
// each, read twice: 55 us.  256 single tokens of 128 heads of 192/128: 11.5 us
// (9.3 us is the host's time), by instructions rather than bytes; one head
// after the other in a warp: 57.7 us.
//
// The runs that start in a window of tokens are shared out over `shares`
// warps: a run is a list of units (K or V, some heads), and unit u of the
// window belongs to warp u mod shares.
// A long run keeps REG chunks a lane between its two uses.
template <int REG, int CTAS>
__global__ void __launch_bounds__(kAppThreads, CTAS) kv_append_kernel(const AppendParams p) {
    griddep_launch_dependents();
    griddep_wait();
    const int lane = threadIdx.x & 31;
    const uint32_t win = blockIdx.x / static_cast<uint32_t>(p.ctas);   // (a window's warps: `ctas` blocks)
    const int share = static_cast<int>(blockIdx.x - win * p.ctas) * (kAppThreads / 32) + (threadIdx.x >> 5);
    const int64_t t0 = static_cast<int64_t>(win) * p.window;
    const int bs_mask = (1 << p.bs_log2) - 1;
    // lane i has the slot of token t0 + i: where runs start, and where they go on
    const long long cur = t0 + lane < p.T ? p.slots[t0 + lane] : -1;
    long long prev = __shfl_up_sync(0xFFFFFFFFu, cur, 1);
    if (lane == 0) prev = t0 > 0 ? p.slots[t0 - 1] : -2;
    const bool valid = cur >= 0 && cur < p.n_slots, goes_on = valid && prev + 1 == cur && (cur & bs_mask) != 0;
    const unsigned more = __ballot_sync(0xFFFFFFFFu, goes_on);
    unsigned starts = __ballot_sync(0xFFFFFFFFu, valid && !goes_on && lane < p.window);
    int base = 0;   // units before this run, mod shares
    while (starts) {
        const int src = __ffs(starts) - 1;
        starts &= starts - 1;
        const long long slot = __shfl_sync(0xFFFFFFFFu, cur, src);
        Run run;
        run.t = t0 + src;
        run.off = static_cast<int>(slot & bs_mask);
        run.page = slot >> p.bs_log2;
        const int room = bs_mask + 1 - run.off;   // (a run ends with its page)
        const unsigned after = src < 31 ? ~more >> (src + 1) : 0u;
        if (after) {
            run.n = __ffs(after);
        } else {
            run.n = 32 - src;
        }
        if (src + run.n == 32) {
            for (; run.n < room; run.n += 32) {
                const int64_t tt = run.t + run.n + lane;
                const bool on = run.n + lane < room && tt < p.T && p.slots[tt] == slot + run.n + lane;
                const unsigned m = __ballot_sync(0xFFFFFFFFu, on);
                if (m != 0xFFFFFFFFu) {
                    run.n += __ffs(~m) - 1;
                    break;
                }
            }
        }
#pragma unroll 1
        for (int which = 0; which < 2; ++which) {
            const int total = run.n * (p.d[which] >> 3);
            const int sub_log2 = total <= 8 ? 2 : total <= 16 ? 1 : 0;
            const int per_log2 = total <= 32 ? p.rows_log2 + sub_log2 : total <= 128 ? min(p.rows_log2, REG == 16 ? 2 : 1) : 0;
            const int per = 1 << per_log2, units = (p.H + per - 1) >> per_log2;
            int u = share - base;
            if (u < 0) u += p.shares;
            for (; u < units; u += p.shares) {
                const int h0 = u * per, nh = min(per, p.H - h0);
                if (total <= 32)
                    append_heads<1, kAppRows, false>(p, which, run, h0, nh, sub_log2);
                else if (total <= 128)
                    append_heads<4, REG / 4, false>(p, which, run, h0, nh, 0);
                else
                    append_heads<REG, 1, true>(p, which, run, h0, nh, 0);
            }
            base += units;
            if (base >= p.shares) base %= p.shares;
        }
    }
}

// A call's array, for the check that none of its results overlaps another of its arrays.
struct Span {
    const void* at;
    int64_t bytes;
};
bool overlap(const Span& a, const Span& b) {
    const uintptr_t x = reinterpret_cast<uintptr_t>(a.at), y = reinterpret_cast<uintptr_t>(b.at);
    return a.at && b.at && a.bytes > 0 && b.bytes > 0 && x < y + static_cast<uintptr_t>(b.bytes) && y < x + static_cast<uintptr_t>(a.bytes);
}

bool block_size_ok(int32_t bs) { return bs == 16 || bs == 32 || bs == 64 || bs == 128; }
int log2_of(int32_t bs) {
    int l = 0;
    while ((1 << l) < bs) ++l;
    return l;
}

}  // namespace
}  // namespace fp8bs

using namespace fp8bs;

extern "C" fp8_status fp8_kv_plan(const int32_t* past, const int32_t* fresh, int32_t B, int32_t block_size,
                                  const int32_t* free_pages, int32_t n_free, const int32_t* used, int32_t* tables,
                                  int32_t width, int32_t* lens, int32_t* offsets, int64_t T, int64_t* slots,
                                  int32_t* positions, int32_t* used_out, void* stream) {
    if (B < 0 || T < 0 || n_free < 0 || width <= 0 || !block_size_ok(block_size)) return FP8_ERR_INVALID_ARG;
    if (static_cast<int64_t>(width) * block_size > (1LL << 31) - 1) return FP8_ERR_INVALID_ARG;
    if (B > kPlanMaxB || T > (1LL << 31) - 1) return FP8_ERR_UNSUPPORTED;
    if (B == 0) return T == 0 ? FP8_OK : FP8_ERR_INVALID_ARG;
    if (!past || !fresh || !used || !tables || !lens || !offsets || !used_out) return FP8_ERR_INVALID_ARG;
    if ((n_free > 0 && !free_pages) || (T > 0 && !slots)) return FP8_ERR_INVALID_ARG;
    // Every CTA reads the inputs while others write results already.
    const Span arrays[10] = {{tables, 4LL * B * width}, {lens, 4LL * B}, {offsets, 4LL * B + 4}, {slots, 8 * T},
                             {positions, 4 * T}, {used_out, 4}, {past, 4LL * B}, {fresh, 4LL * B},
                             {free_pages, 4LL * n_free}, {used, 4}};
    for (int i = 0; i < 6; ++i)
        for (int j = i + 1; j < 10; ++j)
            if (overlap(arrays[i], arrays[j])) return FP8_ERR_INVALID_ARG;
    PlanParams p{};
    p.past = past;
    p.fresh = fresh;
    p.free_pages = free_pages;
    p.used = used;
    p.tables = tables;
    p.lens = lens;
    p.offsets = offsets;
    p.positions = positions;
    p.used_out = used_out;
    p.slots = slots;
    p.T = T;
    p.B = B;
    p.n_free = n_free;
    p.width = width;
    p.bs_log2 = log2_of(block_size);
    p.vec = aligned16(slots) && (!positions || aligned16(positions)) ? 1 : 0;
    const size_t smem = (3 * static_cast<size_t>(B) + 2) * sizeof(int32_t);
    static int configured[64] = {};
    int dev = 0;
    cudaGetDevice(&dev);
    if (dev >= 64 || !configured[dev]) {
        FP8_CUDA_TRY(cudaFuncSetAttribute(kv_plan_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                          (3 * kPlanMaxB + 2) * 4));
        if (dev < 64) configured[dev] = 1;
    }
    const int64_t per_cta = static_cast<int64_t>(kPlanThreads) * kPlanTok;
    int64_t grid = (T + per_cta - 1) / per_cta;
    if (grid > device_sm_count()) grid = device_sm_count();
    if (grid < 1) grid = 1;
    const cudaError_t e = launch_pdl(kv_plan_kernel, dim3(static_cast<unsigned>(grid)), dim3(kPlanThreads), smem,
                                     static_cast<cudaStream_t>(stream), p);
    return e == cudaSuccess ? FP8_OK : FP8_ERR_CUDA;
}

extern "C" fp8_status fp8_kv_append(const void* k, int64_t k_token_stride, int64_t k_head_stride, const void* v,
                                    int64_t v_token_stride, int64_t v_head_stride, const int64_t* slots, int64_t T,
                                    int32_t H, int32_t dk, int32_t dv, void* k_cache, float* k_scale, void* v_cache,
                                    float* v_scale, int64_t n_pages, int32_t block_size, int scale_fmt, void* stream) {
    auto dim_ok = [](int32_t d) { return d > 0 && d <= 1024 && d % 16 == 0; };
    if (T < 0 || H <= 0 || !dim_ok(dk) || !dim_ok(dv) || n_pages < 0 || !block_size_ok(block_size))
        return FP8_ERR_INVALID_ARG;
    if (scale_fmt != FP8_SCALE_FP32 && scale_fmt != FP8_SCALE_UE8M0) return FP8_ERR_INVALID_ARG;
    if (T > (1LL << 31) - 1 || H > 65535 || n_pages > (1LL << 31) - 1) return FP8_ERR_UNSUPPORTED;
    if (T == 0) return FP8_OK;
    if (!k || !v || !slots || !k_cache || !k_scale || !v_cache || !v_scale) return FP8_ERR_INVALID_ARG;
    if (!aligned16(k) || !aligned16(v) || !aligned16(k_cache) || !aligned16(v_cache)) return FP8_ERR_INVALID_ARG;
    if (k_token_stride % 8 || k_head_stride % 8 || v_token_stride % 8 || v_head_stride % 8 || k_token_stride < 0 ||
        k_head_stride < 0 || v_token_stride < 0 || v_head_stride < 0)
        return FP8_ERR_INVALID_ARG;
    AppendParams p{};
    p.x[0] = static_cast<const uint16_t*>(k);
    p.x[1] = static_cast<const uint16_t*>(v);
    p.ts[0] = k_token_stride;
    p.ts[1] = v_token_stride;
    p.hs[0] = k_head_stride;
    p.hs[1] = v_head_stride;
    p.cache[0] = static_cast<uint8_t*>(k_cache);
    p.cache[1] = static_cast<uint8_t*>(v_cache);
    p.scale[0] = k_scale;
    p.scale[1] = v_scale;
    p.slots = slots;
    p.T = T;
    p.H = H;
    p.d[0] = dk;
    p.d[1] = dv;
    p.bs_log2 = log2_of(block_size);
    p.n_slots = n_pages << p.bs_log2;
    p.ue8m0 = scale_fmt;
    for (int i = 0; i < 2; ++i) p.inv[i] = ((1 << 21) + p.d[i] / 8 - 1) / (p.d[i] / 8);
    // Windows of one token while that gives the machine few enough warps, else
    // of 32; then as many warps to a window, and as few heads at a time in a
    // warp, as fill the machine about kAppFill times.  Few tokens are single
    // ones more often than not: then more warps with fewer registers, which
    // take a long run in more loads (256 tokens of 128 heads 14.0 us against
    // 15.7 us; prompts the other way, 33 us against 49 us).
    const int sms = device_sm_count();
    const bool few = T <= static_cast<int64_t>(sms) * 16;
    const int64_t fill = static_cast<int64_t>(sms) * (kAppThreads / 32) * (few ? 5 : 4);
    const int64_t w = few ? 1 : 32, windows = (T + w - 1) / w;
    int64_t rows = 1;
    while (rows < kAppRows && windows * 2 * ((H + rows - 1) / rows) > kAppFill * fill) rows *= 2;
    const int64_t most = (2 * ((H + rows - 1) / rows) + kAppThreads / 32 - 1) / (kAppThreads / 32);
    const int64_t ctas = std::max<int64_t>(1, std::min(kAppFill * fill / windows / (kAppThreads / 32), most));
    p.window = static_cast<int32_t>(w);
    p.rows_log2 = log2_of(static_cast<int32_t>(rows));
    p.ctas = static_cast<int32_t>(ctas);
    p.shares = static_cast<int32_t>(ctas) * (kAppThreads / 32);
    const int64_t grid = windows * ctas;
    if (grid > (1LL << 31) - 1) return FP8_ERR_UNSUPPORTED;
    const cudaError_t e = launch_pdl(few ? kv_append_kernel<8, 5> : kv_append_kernel<16, 4>, dim3(static_cast<unsigned>(grid)), dim3(kAppThreads), 0,
                                     static_cast<cudaStream_t>(stream), p);
    return e == cudaSuccess ? FP8_OK : FP8_ERR_CUDA;
}
