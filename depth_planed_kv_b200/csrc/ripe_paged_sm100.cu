// ripe_paged_sm100.cu -- ripe_paged_attn on the tensor cores: chunks of new tokens
// (prompts, chunks of prompts, draft blocks with many rows) over a paged cache; bf16,
// head size 32, 64, 96 or 128.
//
// Per item (row tile of tokens x the query heads of one key/value head, see
// ripe_paged.cuh): S = Q K^T and O += P V with the online softmax
//   m' = max(m, max_k S), P = 2^(c S - m'), l' = l 2^(m - m') + sum P, O' = O 2^(m - m') + P V
// (c = scale * log2 e).  m moves only when a row's maximum grew by more than 2^8: until
// then P stays below 2^8, which fp32 sums and bf16's exponent hold without loss, and the
// accumulator need not be read back.  l sums the unrounded P; P is rounded to bf16 for
// the second product (2^-8 of a weight at most, below the rounding of O itself).
//
// One persistent CTA per SM, 12 warps: two groups of four softmax warps (a row per
// thread), the MMA warp, three TMA warps.  Two streams s = 0, 1, one per softmax group,
// each with two S buffers (64 keys each) and its own O in tensor memory:
//   two M tiles (more than 128 rows): stream s is M tile s, both over the same key tile;
//   one M tile: stream s takes every second key tile, joined at the item's end.
// S of a stream's next key tile is already there when its softmax ends a tile, so neither
// the exponentials nor the tensor pipe wait for the other's latency.  (With one S buffer
// of 128 keys per stream the chain softmax -> P V -> Q K^T -> softmax took 4400 cycles a
// pair of tiles, of which the exponential unit and the tensor pipe were each busy 2100.)
// Keys and values arrive in 64-key tiles through one ring of shared-memory stages, 64-byte
// swizzle (the boxes: see paged_tc_kernel).
//
// Measured with the join of cut items: 2048 tokens behind 32768, 32 query heads over 8,
// head size 128: 963 us after a rest, 1.18 PFLOP/s, and 1110 us in a long run under the power
// cap, 1.02 PFLOP/s (cuBLAS 1.65 in a burst and near 1.4 under the cap).  A pair of 64-key
// tiles takes 1740 cycles there, where the products need 1133 (64 columns a product: 49
// cycles instead of 32, the queries' reads from shared memory bind) and the exponential unit
// 1060; the softmax's serial parts are the rest (two of its warps a scheduler, 46% of the
// issue slots used).  64 draft blocks of 8 tokens behind 512 to 4096, pages of 16: 130 us
// for 654 MB, 5.0 TB/s (146 in a long run): TMA issue and the items' ends.
// 2048 tokens alone, 55 heads of size 96: 91 us, 0.49 PFLOP/s: items of 2 to 32 tiles, half
// of their time their own beginnings and ends (the masked tiles, the last rows' way out).
#include <cuda.h>
#include <cudaTypedefs.h>
#include <math.h>
#include <string.h>

#include <type_traits>

#include "ripe_launch.h"
#include "ripe_paged.cuh"
#include "ripe_paged_launch.h"
#include "sm100_ptx.cuh"

using namespace sm100;

namespace {

constexpr int kKT = 64;  // keys per tile
constexpr int kThreads = 384;  // softmax warps 0-7 (4 a stream), the MMA warp, three TMA warps
constexpr int kMmaWarp = 8, kTmaWarp = 9, kTmaWarps = 3;
// Where there is less than kMinCost (key tiles x M tiles) a CTA, items are cut into pieces of
// 2^kPieces key tiles.  (Stretches of 8 whatever the items: 4 sequences of 1 to 16 tokens
// behind 19 took 34 us, one CTA all eight items; now 11.  Stretches of 1: 10, but 33 against 20
// for one chunk of 673 tokens of one head, cut into halves of tiles; now 22.)
constexpr int kMinCost = 8, kPieces = 2;

struct alignas(64) PagedMaps {
    CUtensorMap q, k, v;
};

template <int D, int ST>
struct Lay {
    static constexpr int NCH = D / 32;         // 32-channel chunks
    static constexpr int QTILE = NCH * 8192;   // 128 rows of bf16
    static constexpr int TILE = NCH * 4096;    // 64 keys of bf16
    static constexpr int Q = 0;
    static constexpr int KV = 2 * QTILE;
    static constexpr int BARS = KV + ST * TILE;
    static constexpr int NBAR = 2 * ST + 2 * 4 + 6 * 2 + 3;
    static constexpr int ML = BARS + ((NBAR * 8 + 15) / 16) * 16;  // [2][128] (m, l) of stream 1
    static constexpr int SEG = ML + 2 * 128 * 8;  // the segments under way, as the TMA warp found them
    static constexpr int MISC = SEG + 2 * 64;
    static constexpr int TOTAL = MISC + 32;
    // The plan is read before the first item, by the one warp that goes on with it; the joined
    // (m, l) come after.
    static constexpr int PLAN = ML;
    static_assert(sizeof(PagedPlanHead) <= 2 * 128 * 8, "plan over (m, l)");
    static_assert(sizeof(PagedSeg) <= 64, "segment slots");
    static_assert(sizeof(PagedPlanSmem) <= (size_t)ST * TILE, "plan arrays over the stages");
    static_assert(ST >= 8, "the first products of an item need four key tiles, and its first values");
    static_assert(TOTAL + 512 <= 232448, "shared memory of one CTA");
};

// Waits with the whole warp: true only if every lane saw the phase complete.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, volatile int* abort, int32_t* err) {
    return __all_sync(0xffffffffu, mbar_wait_idle(bar, parity, abort, err));
}

__device__ __forceinline__ bool elect_one() {
    uint32_t p;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
    return p != 0;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
    float d;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}
// Two lanes of fp32 in a register pair.
__device__ __forceinline__ uint64_t pair(float lo, float hi) {
    uint64_t d;
    asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "f"(lo), "f"(hi));
    return d;
}
__device__ __forceinline__ void unpair(uint64_t d, float& lo, float& hi) { asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(d)); }
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
// Arithmetic that stays where it is written.
__device__ __forceinline__ void fma2_here(float& lo, float& hi, uint64_t b, uint64_t c) {
    uint64_t d = pair(lo, hi);
    asm volatile("fma.rn.f32x2 %0, %0, %1, %2;" : "+l"(d) : "l"(b), "l"(c));
    unpair(d, lo, hi);
}
__device__ __forceinline__ float ex2_here(float x) {
    float y;
    asm volatile("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ uint32_t pack_here(float lo, float hi) {
    uint32_t y;
    asm volatile("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(y) : "f"(hi), "f"(lo));
    return y;
}
// The lowest n bits (all for n >= 32, none for n <= 0).
__device__ __forceinline__ uint32_t below(int n) { return n >= 32 ? ~0u : n <= 0 ? 0u : (1u << n) - 1; }
// -inf where `see` has no bit.
__device__ __forceinline__ void hide(float* v, uint32_t see) {
    if (__all_sync(0xffffffffu, see == ~0u)) return;
#pragma unroll
    for (int j = 0; j < 32; ++j) v[j] = (see >> j) & 1 ? v[j] : -INFINITY;
}

// s + 0 * w, two bf16 each.
__device__ __forceinline__ uint32_t zero_times(uint32_t w, uint32_t s) {
    uint32_t d;
    asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(d) : "r"(w), "r"(0u), "r"(s));
    return d;
}
// Zeros the values the matrix product must not see in a key tile that some row sees
// only in part: keys from `end` (of the tile) on, whose slots hold anything, and values
// that are not finite (`flag` then holds `mark`; paged_nonfinite puts them back
// where they are seen).  128 threads, 16 bytes at a time in the order they lie.  With two
// M tiles both streams clean the tile, each before its own product: what the later one
// still writes is what the earlier one wrote, and the flag is set before a value goes, so
// that a stream which finds a value gone already finds the flag too.
template <int NCH, bool GROUPS>
__device__ __forceinline__ void clean_values(char* sv, int t, int end, volatile int* flag, int mark) {
    if (end >= kKT) {
        // 0 * x adds up to 0 if x are all finite, else to NaN: an instruction a pair
        uint4 x[NCH * 2];
        uint32_t s0 = 0, s1 = 0;
#pragma unroll
        for (int i = 0; i < NCH * 2; ++i) x[i] = reinterpret_cast<const uint4*>(sv)[t + i * 128];
#pragma unroll
        for (int i = 0; i < NCH * 2; ++i) {
            s0 = zero_times(x[i].x, s0);
            s1 = zero_times(x[i].y, s1);
            s0 = zero_times(x[i].z, s0);
            s1 = zero_times(x[i].w, s1);
        }
        if ((s0 | s1) == 0) return;
    }
#pragma unroll 2
    for (int i = t; i < NCH * 256; i += 128) {
        uint4* at = reinterpret_cast<uint4*>(sv) + i;
        uint4 x = *at;
        const int key = GROUPS ? i / (NCH * 32) * 8 + ((i & 31) >> 2) : (i & 255) >> 2;  // four 16-byte units a key and chunk
        if (key >= end) {
            if (x.x | x.y | x.z | x.w) *at = make_uint4(0, 0, 0, 0);
            continue;
        }
        // an exponent of all ones carries into its sign bit
        auto top = [](uint32_t w) { return ((w & 0x7F807F80u) + 0x00800080u) & 0x80008000u; };
        if (top(x.x) | top(x.y) | top(x.z) | top(x.w)) {
            auto finite = [&](uint32_t w) {
                const uint32_t b = top(w);
                return w & ~((b >> 15 & 1u) * 0x0000FFFFu | (b >> 31) * 0xFFFF0000u);
            };
            *flag = mark;
            __threadfence_block();
            *at = make_uint4(finite(x.x), finite(x.y), finite(x.z), finite(x.w));
        }
    }
}

// One key tile of one row: S (64 columns, on their way into x and y) -> P over its first
// 32 columns (at s_col), the running maximum m (log2 units) and sum l, and O (at o_col)
// rescaled where the maximum moved, once the product before (`pv_done`) has left it.  n:
// tiles of the item before this one.  PART: keys past `hi`, or up to `lo` and not below
// `first` (from the tile's first key), are hidden.  Two code paths, because the test alone
// costs the full tiles a third of their time once the compiler turns it into selects.
// False if a wait gave up.
template <int D, bool PART>
__device__ __forceinline__ bool softmax_step(float* x, float* y, uint32_t s_col, uint32_t o_col, float c2, int hi, int lo,
                                             int first, bool valid, int n, float& m, float& l, uint64_t* pv_done,
                                             uint32_t parity, volatile int* abort, int32_t* err) {
    tmem_wait_ld32(x);
    tmem_wait_ld32(y);
    if (PART) {
        hide(x, below(hi + 1) & (~below(lo + 1) | below(first)));
        hide(y, below(hi - 31) & (~below(lo - 31) | below(first - 32)));
    }
    float m0 = x[0], m1 = x[1], m2 = y[0], m3 = y[1];
#pragma unroll
    for (int j = 2; j < 30; j += 4) {
        m0 = max3(m0, x[j], x[j + 1]);
        m1 = max3(m1, x[j + 2], x[j + 3]);
        m2 = max3(m2, y[j], y[j + 1]);
        m3 = max3(m3, y[j + 2], y[j + 3]);
    }
    m0 = max3(m0, x[30], x[31]);
    m2 = max3(m2, y[30], y[31]);
    const float mx = max3(m0, m1, fmaxf(m2, m3)) * c2;
    const bool grow = valid && mx > m + 8.f;  // m = -inf: any finite maximum
    if (__any_sync(0xffffffffu, grow)) {
        const float mn = grow ? mx : m;
        const float f = m == mn ? 1.f : ex2(m - mn);  // 0 from m = -inf
        m = mn;
        l *= f;
        if (n > 0) {
            if (!warp_wait(pv_done, parity, abort, err)) return false;
            tc_fence_after();
#pragma unroll 1  // seldom run, and the loop around it is better small (2048 tokens alone: 99 us, rolled 89)
            for (int c = 0; c < D; c += 16) {
                float o[16];
                tmem_ld16(o_col + c, o);
                tmem_wait_ld16(o);
#pragma unroll
                for (int j = 0; j < 16; ++j) o[j] *= f;
                tmem_st16(o_col + c, reinterpret_cast<const uint32_t*>(o));
            }
        }
    }
    const float mref = m == -INFINITY ? 0.f : -m;
    // The exponential unit takes a warp 8 cycles an instruction, and a warp that waits for
    // each result idles it: the other work is written out between the exponentials (the
    // asm statements keep their order), the second half's scaling beside the first half's
    // exponentials, the first half's sums and packing beside the second's, two fp32 lanes an
    // instruction.  (Every fourth exponential as a polynomial on the FMA pipe: 1240 us against
    // 1080 for 2048 tokens at 32768; issue slots are as scarce as the exponential unit.)
    const uint64_t cc = pair(c2, c2), mm = pair(mref, mref);
    uint64_t la = 0, lb = 0;  // pairs of partial sums
    uint32_t w[16];
#pragma unroll
    for (int j = 0; j < 8; j += 2) fma2_here(x[j], x[j + 1], cc, mm);
#pragma unroll
    for (int j = 0; j < 32; j += 4) {
        x[j] = ex2_here(x[j]);
        if (j < 24) fma2_here(x[j + 8], x[j + 9], cc, mm);
        else fma2_here(y[j - 24], y[j - 23], cc, mm);
        x[j + 1] = ex2_here(x[j + 1]);
        if (j < 24) fma2_here(x[j + 10], x[j + 11], cc, mm);
        else fma2_here(y[j - 22], y[j - 21], cc, mm);
        x[j + 2] = ex2_here(x[j + 2]);
        x[j + 3] = ex2_here(x[j + 3]);
    }
#pragma unroll
    for (int j = 0; j < 32; j += 4) {
        y[j] = ex2_here(y[j]);
        if (j < 24) fma2_here(y[j + 8], y[j + 9], cc, mm);
        la = add2(la, pair(x[j], x[j + 1]));
        w[j / 2] = pack_here(x[j], x[j + 1]);
        y[j + 1] = ex2_here(y[j + 1]);
        if (j < 24) fma2_here(y[j + 10], y[j + 11], cc, mm);
        lb = add2(lb, pair(x[j + 2], x[j + 3]));
        w[j / 2 + 1] = pack_here(x[j + 2], x[j + 3]);
        y[j + 2] = ex2_here(y[j + 2]);
        y[j + 3] = ex2_here(y[j + 3]);
    }
    tmem_st16(s_col, w);
#pragma unroll
    for (int j = 0; j < 32; j += 4) {
        w[j / 2] = pack_here(y[j], y[j + 1]);
        w[j / 2 + 1] = pack_here(y[j + 2], y[j + 3]);
        la = add2(la, pair(y[j], y[j + 1]));
        lb = add2(lb, pair(y[j + 2], y[j + 3]));
    }
    tmem_st16(s_col + 16, w);
    float l0, l1, l2, l3;
    unpair(la, l0, l1);
    unpair(lb, l2, l3);
    l += (l0 + l1) + (l2 + l3);
    return true;
}

// Key tiles of a stretch that M tile 0 of two needs: those up to its own last token (the
// rest are M tile 1's alone).
__device__ __forceinline__ int first_tiles(const PagedArgs& a, const PagedSeg& s) {
    const int end = (s.c + s.t0 + a.tok1 - 1) / kKT + 1 - (s.tiles.tlo - s.tiles.ts);
    return max(0, min(s.tb, end) - s.ta);
}

// Where O's channel c of row r lies in a slot: eight rows' pieces of 16 bytes side by side,
// so that a warp's store, a piece of 32 rows, fills four lines rather than a sector in each
// of 32 (the last item's end, of a CTA that leaves a partial, took 10000 cycles of 154000
// for 2048 tokens of 55 heads).
template <int D>
__device__ __forceinline__ constexpr int slot_at(int r, int c) {
    return ((r >> 3) * (D / 4) + (c >> 2)) * 32 + (r & 7) * 4 + (c & 3);
}

// A key tile lies in its stage as 32-channel chunks of 64 keys one behind the other, or, by
// GROUPS, as groups of eight keys one behind the other, all chunks of a group together.  A
// box brings what one page holds of that: all 64 keys and chunks, or one chunk of a smaller
// page; by groups, eight keys of all chunks.  Groups are taken for pages of 16 keys: 8 boxes
// a tile instead of 16 (12 for head size 96, 8 for 64), and boxes are what such pages cost
// (64 draft blocks of 8 tokens, head size 128: 139 us with chunks, 130 with groups).
template <int D, int ST, bool GROUPS>
__global__ void __launch_bounds__(kThreads, 1) paged_tc_kernel(const __grid_constant__ PagedMaps tm,
                                                               const __grid_constant__ PagedArgs a) {
    using L = Lay<D, ST>;
    constexpr int NCH = L::NCH;
    extern __shared__ char smem_raw[];
    char* smem = reinterpret_cast<char*>((reinterpret_cast<uintptr_t>(smem_raw) + 511) & ~(uintptr_t)511);
    char* sQ = smem + L::Q;
    char* sKV = smem + L::KV;
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + L::BARS);
    // s_full, p_full: [stream][S buffer]; the others with two: [stream] or [parity of the segment]
    uint64_t *kv_full = bars, *kv_empty = bars + ST, *s_full = bars + 2 * ST, *p_full = s_full + 4, *pv_done = p_full + 4,
             *o_full = pv_done + 2, *o_free = o_full + 2, *seg_full = o_free + 2, *seg_empty = seg_full + 2,
             *q_full = seg_empty + 2, *q_free = q_full + 1, *ml_full = q_free + 1, *drain = ml_full + 1;
    float2* s_ml = reinterpret_cast<float2*>(smem + L::ML);
    uint32_t* s_tmem = reinterpret_cast<uint32_t*>(smem + L::MISC);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + L::MISC + 4);
    PagedSeg* s_seg[2] = {reinterpret_cast<PagedSeg*>(smem + L::SEG), reinterpret_cast<PagedSeg*>(smem + L::SEG + 64)};
    volatile int* s_bad = reinterpret_cast<volatile int*>(smem + L::MISC + 16);  // [4] item with non-finite values

    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    if (threadIdx.x == 0) {
        for (int i = 0; i < ST; ++i) {
            mbar_init(kv_full + i, 1);
            mbar_init(kv_empty + i, 1);
        }
        for (int i = 0; i < 4; ++i) {
            mbar_init(s_full + i, 1);
            mbar_init(p_full + i, 128);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(pv_done + i, 1);
            mbar_init(o_full + i, 1);
            mbar_init(o_free + i, 128);
            mbar_init(seg_full + i, 1);
            mbar_init(seg_empty + i, 8 + kTmaWarps);  // all but the warp that fills it
        }
        mbar_init(q_full, 1);
        mbar_init(q_free, 1);
        mbar_init(ml_full, 128);
        mbar_init(drain, 1);
        fence_barrier_init();
        *abort_flag = 0;
        for (int i = 0; i < 4; ++i) s_bad[i] = 0;
    }
    if (warp == kMmaWarp) {
        tmem_alloc(s_tmem, 512);
        tmem_relinquish();
    }
    if (warp == kTmaWarp && lane < 3) prefetch_tmap(lane == 0 ? &tm.q : lane == 1 ? &tm.k : &tm.v);
    PagedPlan<kKT> plan;  // carried on by the first TMA warp alone
    plan.template begin<kThreads>(a, *reinterpret_cast<PagedPlanHead*>(smem + L::PLAN), *reinterpret_cast<PagedPlanSmem*>(sKV),
                                  kMinCost, kPieces);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *s_tmem;

    if (warp >= kTmaWarp) {
        // ------------------------------------------------------------ TMA producers
        // A tile is one box where a page holds it (64 keys), else nsub pages x NCH chunks of 32
        // channels, a box per lane.  A lane's copy takes its warp about 70 cycles to issue, and a
        // load another 250 for its barriers, so three warps take the loads in turn: with pages of
        // 16 keys one warp alone brings 11 bytes per cycle (HBM gives an SM 23).  Each waits for
        // its own stages only; that cannot be off by a round, because stages are freed in the
        // order of use and a warp comes round every kTmaWarps < ST loads.
        static_assert(kTmaWarps < ST, "see above");
        const int pw = warp - kTmaWarp;
        const int pb = GROUPS ? 8 : a.page < kKT ? a.page : kKT, nsub = kKT / pb;
        const int nch = GROUPS || nsub == 1 ? 1 : NCH;  // boxes of pb keys
        const int sub = lane / nch, ch = lane % nch;
        const uint32_t box = (uint32_t)pb * 64;  // bytes of a chunk of pb keys
        char* dst = sKV + (GROUPS ? sub * NCH * 512 : ch * 4096 + sub * (int)box);
        int st = 0, ph = 1, turn = 0, n = 0;  // stage, its empty parity (the first round passes), whose load, segments begun
        bool ok = true;
        for (;; ++n) {
            PagedSeg* slot = s_seg[n & 1];
            if (pw == 0) {
                // The next segment, for the other warps too; one without keys ends the work.
                PagedSeg s;
                if (!plan.next(a, s)) s.ta = s.tb = 0;
                if (!(ok = warp_wait(seg_empty + (n & 1), ((n >> 1) & 1) ^ 1, abort_flag, a.err))) break;
                if (lane == 0) {
                    *slot = s;
                    mbar_arrive(seg_full + (n & 1));
                }
                __syncwarp();
            } else if (!(ok = warp_wait(seg_full + (n & 1), (n >> 1) & 1, abort_flag, a.err))) {
                break;
            }
            const int ta = slot->ta, tb = slot->tb;
            if (ta == tb) break;
            const int p0 = slot->c + slot->t0, end = p0 + slot->ntok, head = slot->head, seq = slot->seq, slot_w = slot->w;
            const PagedTiles tiles = slot->tiles;
            if (pw == 0) {
                if (!(ok = warp_wait(q_free, (n & 1) ^ 1, abort_flag, a.err))) break;
                if (lane == 0) {
                    mbar_expect_tx(q_full, slot->w * NCH * ((uint32_t)a.tok1 * a.G * 64));
                    for (int mt = 0; mt < slot->w; ++mt)
                        for (int c = 0; c < NCH; ++c)
                            tma_load_3d(sQ + mt * L::QTILE + c * 8192, &tm.q, 32 * c, head * a.G,
                                        slot->r + slot->t0 + mt * a.tok1, q_full);
                }
                __syncwarp();
            } else {
                __syncwarp();
                if (lane == 0) mbar_arrive(seg_empty + (n & 1));
            }
            // The order of use: the first `ahead` key tiles, then each tile's values and the
            // keys `ahead` tiles on.
            const int ahead = slot_w == 2 ? 2 : 4;
            auto on = [&](int t) { return t < tb && sub < nsub && tiles.tile(t) * kKT + sub * pb < end; };
            // Behind the window a page may be gone, whatever the table says: a box that no row
            // sees is read as zeros, by a page id past the last.
            const int gone_to = a.window > 0 ? p0 - a.window - pb + 1 : -1;  // paged_any_seen in two comparisons
            auto gone = [&](int t) {
                const int k = tiles.tile(t) * kKT + sub * pb;
                return k <= gone_to && k >= a.sinks;
            };
            auto entry = [&](int t) { return on(t) && !gone(t) ? paged_entry(a, seq, tiles.tile(t) * kKT + sub * pb) : 0; };
            auto load = [&](int t, int id, const CUtensorMap* map) {
                const int k0 = tiles.tile(t) * kKT, y = (k0 + sub * pb) & (a.page - 1);
                if (turn == pw) {
                    if (!warp_wait(kv_empty + st, ph, abort_flag, a.err)) return false;
                    if (lane == 0) mbar_expect_tx(kv_full + st, min(nsub, (end - k0 + pb - 1) / pb) * NCH * box);
                    __syncwarp();
                    if (on(t))
                        tma_load_5d(dst + st * L::TILE, map, 0, y, ch, head, gone(t) ? a.npages : paged_checked(a, id),
                                    kv_full + st);
                    __syncwarp();
                }
                if (++turn == kTmaWarps) turn = 0;
                if (++st == ST) {
                    st = 0;
                    ph ^= 1;
                }
                return true;
            };
            int ids[4];  // table entries of tiles t .. t + 3, for this lane's box
#pragma unroll
            for (int i = 0; i < 4; ++i) ids[i] = entry(ta + i);
            ok = load(ta, ids[0], &tm.k);
            for (int i = 1; i < ahead && ta + i < tb && ok; ++i)
                ok = load(ta + i, i == 1 ? ids[1] : i == 2 ? ids[2] : ids[3], &tm.k);
            for (int t = ta; t < tb && ok; ++t) {
                const int next = entry(t + 4);
                if (!(ok = load(t, ids[0], &tm.v))) break;
                if (t + ahead < tb) ok = load(t + ahead, ahead == 2 ? ids[2] : next, &tm.k);
                ids[0] = ids[1];
                ids[1] = ids[2];
                ids[2] = ids[3];
                ids[3] = next;
            }
            if (!ok) break;
        }
        // Every copy has landed before the CTA's shared memory goes away: on the ordinary
        // way out the MMA warp waited for all of them.  Otherwise give those in flight time
        // (a stage may be one that nobody loads any more).
        if (!ok || *abort_flag) {
            const long long t0 = clock64();
            while (clock64() - t0 < (1 << 20)) {}
        }
    } else if (warp == kMmaWarp) {
        // ------------------------------------------------------------ MMA issuer
        if (elect_one()) {
            constexpr uint32_t IDESC_QK = idesc_bf16(128, kKT, 0), IDESC_PV = idesc_bf16(128, D, 1);
            const uint64_t dq = smem_desc(smem_u32(sQ), 16, 512, kLayoutSwizzle64B);
            // bytes from a chunk to the next, and from eight keys to the next eight
            constexpr uint32_t chunk = GROUPS ? 512 : 4096, group = GROUPS ? NCH * 512 : 512;
            const uint64_t dk = smem_desc(smem_u32(sKV), 16, group, kLayoutSwizzle64B);
            const uint64_t dv = smem_desc(smem_u32(sKV), chunk, group, kLayoutSwizzle64B);
            int seg = 0, st = 0;
            uint32_t ph = 0;                                         // the next stage in the order of use
            uint32_t nqk[2] = {0, 0}, npv[2] = {0, 0}, uses[2] = {0, 0};  // products and segments of each stream so far
            bool ok = true;
            auto stage = [&]() -> bool {  // waits for it
                return mbar_wait_idle(kv_full + st, ph, abort_flag, a.err);
            };
            auto next_stage = [&]() {  // frees it once the products issued so far are done
                mma_commit(kv_empty + st);
                if (++st == ST) {
                    st = 0;
                    ph ^= 1;
                }
            };
            // S of stream s (its next buffer) = Q tile `qt` x K in the current stage
            auto qk = [&](auto s, int qt) {
                const uint32_t b = nqk[s.value]++ & 1;
#pragma unroll
                for (int ks = 0; ks < D / 16; ++ks)
                    mma_bf16(tmem + 128 * s.value + 64 * b, dq + qt * (L::QTILE / 16) + ((ks >> 1) * 8192 + (ks & 1) * 32) / 16,
                             dk + st * (L::TILE / 16) + (ks >> 1) * (chunk / 16) + (ks & 1) * 2, IDESC_QK, ks > 0 ? 1u : 0u);
                mma_commit(s_full + 2 * s.value + b);
            };
            // O of stream s += P x V in the current stage; waits for P, and for O before its first use
            auto pv = [&](auto s, bool first, bool last) -> bool {
                const uint32_t n = npv[s.value]++, b = n & 1;
                if (!mbar_wait_idle(p_full + 2 * s.value + b, (n >> 1) & 1, abort_flag, a.err)) return false;
                if (first && !mbar_wait_idle(o_free + s.value, (uses[s.value]++ & 1) ^ 1, abort_flag, a.err)) return false;
                tc_fence_after();
#pragma unroll
                for (int ks = 0; ks < kKT / 16; ++ks)
                    mma_bf16_ts(tmem + 256 + D * s.value, tmem + 128 * s.value + 64 * b + ks * 8,
                                dv + st * (L::TILE / 16) + ks * (group / 8), IDESC_PV, (!first || ks > 0) ? 1u : 0u);
                mma_commit(pv_done + s.value);
                if (last) mma_commit(o_full + s.value);
                return true;
            };
            const std::integral_constant<int, 0> s0{};
            const std::integral_constant<int, 1> s1{};
            while ((ok = mbar_wait_idle(seg_full + (seg & 1), (seg >> 1) & 1, abort_flag, a.err))) {
                const PagedSeg& s = *s_seg[seg & 1];
                const int T = s.tb - s.ta;
                const bool two = s.w == 2;
                const int T0 = two ? first_tiles(a, s) : 0;
                mbar_arrive(seg_empty + (seg & 1));
                if (T == 0) break;
                if (!(ok = mbar_wait_idle(q_full, seg & 1, abort_flag, a.err))) break;
                ++seg;
                if (two) {
                    for (int i = 0; i < 2 && i < T && (ok = stage()); ++i) {
                        if (i < T0) qk(s0, 0);
                        qk(s1, 1);
                        next_stage();
                    }
                    if (T <= 2) mma_commit(q_free);
                    for (int i = 0; i < T && ok; ++i) {
                        if (!(ok = stage())) break;
                        const int vst = st;
                        if (i < T0 && !(ok = pv(s0, i == 0, i + 1 == T0))) break;
                        if (i + 2 < T) {
                            // the keys two tiles on lie in the next stage
                            const uint32_t vph = ph;
                            if (++st == ST) {
                                st = 0;
                                ph ^= 1;
                            }
                            const int kst = st;
                            const uint32_t kph = ph;
                            if (!(ok = stage())) break;
                            if (i + 2 < T0) qk(s0, 0);
                            st = vst;
                            ph = vph;
                            if (!(ok = pv(s1, i == 0, false))) break;
                            mma_commit(kv_empty + vst);
                            st = kst;
                            ph = kph;
                            qk(s1, 1);
                            next_stage();
                            if (i + 3 == T) mma_commit(q_free);
                        } else {
                            if (!(ok = pv(s1, i == 0, i + 1 == T))) break;
                            next_stage();
                        }
                    }
                } else {
                    for (int i = 0; i < 4 && i < T && (ok = stage()); ++i) {
                        if (i & 1) qk(s1, 0); else qk(s0, 0);
                        next_stage();
                    }
                    if (T <= 4) mma_commit(q_free);
                    for (int i = 0; i < T && ok; ++i) {
                        if (!(ok = stage())) break;
                        if (!(ok = i & 1 ? pv(s1, i == 1, i + 2 >= T) : pv(s0, i == 0, i + 2 >= T))) break;
                        next_stage();
                        if (i + 4 < T) {
                            if (!(ok = stage())) break;
                            if (i & 1) qk(s1, 0); else qk(s0, 0);
                            next_stage();
                            if (i + 5 == T) mma_commit(q_free);
                        }
                    }
                }
                if (!ok) break;
            }
            // Every MMA issued so far has completed before TMEM is released.
            volatile int no_abort = 0;
            mma_commit(drain);
            mbar_wait_idle(drain, 0, &no_abort, a.err);
        }
        __syncwarp();
    } else {
        // ------------------------------------------------------------ softmax and epilogue
        const int wg = warp / 4, t = threadIdx.x % 128;  // stream; TMEM lane = row of the M tile
        const uint32_t lane_addr = (uint32_t)((warp % 4) * 32) << 16;
        const uint32_t s_col = tmem + 128 * wg + lane_addr, o_col1 = tmem + 256 + D + lane_addr, o_col = wg ? o_col1 : o_col1 - D;
        const float c2 = a.scale_log2;
        const int tok = t / a.G, g = t - tok * a.G;
        int base = 0, seg = 0, joins = 0, uses = 0, uses1 = 0;  // uses: of this stream, and of stream 1, as in the MMA warp
        uint32_t steps = 0;                                     // key tiles of this stream so far
        if (threadIdx.x == 0) a.hdr[blockIdx.x].kind = 0;
        bool ok = true;
        while (ok && (ok = warp_wait(seg_full + (seg & 1), (seg >> 1) & 1, abort_flag, a.err))) {
            const PagedSeg& s = *s_seg[seg & 1];
            // what the loop over key tiles uses, in registers: it must not wait for loads
            const int ta = s.ta, T = s.tb - ta, sw = s.w, ts = s.tiles.ts, skip = s.tiles.tlo - ts;
            if (T == 0) break;
            const int ahead = sw == 2 ? 2 : 4;
            const int mytok = s.t0 + (sw == 2 ? wg * a.tok1 : 0) + tok;  // this row's token
            const bool valid = tok < a.tok1 && mytok < s.t0 + s.ntok;
            const int pos = s.c + mytok;
            const int p0 = s.c + s.t0, p1 = p0 + s.ntok - 1;
            const int nsteps = sw == 1 ? (T + 1 - wg) / 2 : wg ? T : first_tiles(a, s);
            float m = -INFINITY, l = 0.f;
            // paged_all_seen of a tile in three comparisons
            const int full_hi = p0 - (kKT - 1), full_lo = a.window > 0 ? p1 - a.window : -1, full_first = a.sinks - kKT;
            int tile = ta + (sw == 2 ? 0 : wg);
            float x[32], y[32];
            auto scores = [&](uint32_t step) -> bool {  // waits for the stream's S of `step` and begins to load it
                const uint32_t b = step & 1;
                if (!warp_wait(s_full + 2 * wg + b, (step >> 1) & 1, abort_flag, a.err)) return false;
                tc_fence_after();
                tmem_ld32(s_col + 64 * b, x);
                tmem_ld32(s_col + 64 * b + 32, y);
                return true;
            };
            if (nsteps > 0) ok = scores(steps);
            for (int n = 0; n < nsteps && ok; ++n, ++steps, tile += sw == 2 ? 1 : 2) {
                const int k0 = (tile < ts ? tile : tile + skip) * kKT;
                const bool part = k0 > full_hi || (k0 <= full_lo && k0 > full_first);
                const uint32_t b = steps & 1;
                if (part) {
                    // The tile's values, in the order the TMA warps load.  Only once the scores are
                    // there: their product was issued when every load up to `ahead` tiles back had
                    // arrived, so the parity cannot be that of the stage's earlier round.
                    const int i = tile - ta, k = base + min(T, ahead) + i + min(i, max(T - ahead, 0)), st = k % ST;
                    if (!(ok = warp_wait(kv_full + st, (k / ST) & 1, abort_flag, a.err))) break;
                    clean_values<NCH, GROUPS>(sKV + st * L::TILE, t, p1 + 1 - k0, s_bad + (seg & 3), seg + 1);
                    __threadfence_block();
                    fence_proxy_async_smem();
                    __syncwarp();
                    ok = softmax_step<D, true>(x, y, s_col + 64 * b, o_col, c2, pos - k0, a.window > 0 ? pos - a.window - k0 : -1,
                                               a.sinks - k0, valid, n, m, l, pv_done + wg, (steps + 1) & 1, abort_flag, a.err);
                } else {
                    ok = softmax_step<D, false>(x, y, s_col + 64 * b, o_col, c2, 0, 0, 0, valid, n, m, l, pv_done + wg,
                                                (steps + 1) & 1, abort_flag, a.err);
                }
                if (!ok) break;
                // the next scores are on their way while P is
                const bool more = n + 1 == nsteps || scores(steps + 1);
                tmem_wait_st();
                tc_fence_before();
                mbar_arrive(p_full + 2 * wg + b);
                ok = more;
                if (!ok) break;
            }
            if (!ok) break;
            // -------------------------------------------------------- the item's end
            const bool whole = paged_whole(s);
            const int slot = s.ta > 0 ? 0 : 1;
            if (threadIdx.x == 0 && !whole && s.ta > 0) {
                PagedHdr h;
                h.kind = s.tb == s.tiles.nt ? 2 : 1;
                h.row0 = s.r + s.t0;
                h.ntok = s.ntok;
                h.head = s.head;
                h.c0 = s.c0;
                h.gaps = s.gaps;
                a.hdr[blockIdx.x] = h;
            }
            const bool two = s.w == 1 && T > 1;  // both streams hold a part of the one M tile
            if (two && wg == 1) {
                // not before the other stream has read the join before: it then left this one's O
                if (uses1 > 0 && !(ok = warp_wait(o_free + 1, (uses1 - 1) & 1, abort_flag, a.err))) break;
                s_ml[(joins & 1) * 128 + t] = make_float2(m, l);
                mbar_arrive(ml_full);
            }
            if (s.w == 2 || wg == 0) {
                float f0 = 1.f, f1 = 0.f;
                const bool any = nsteps > 0;  // else these rows have nothing in this stretch
                if (any && !(ok = warp_wait(o_full + wg, uses & 1, abort_flag, a.err))) break;
                if (two) {
                    if (!(ok = warp_wait(ml_full, joins & 1, abort_flag, a.err))) break;
                    if (!(ok = warp_wait(o_full + 1, uses1 & 1, abort_flag, a.err))) break;
                    const float2 x = s_ml[(joins & 1) * 128 + t];
                    const float mn = fmaxf(m, x.x);
                    f0 = m == mn ? 1.f : ex2(m - mn);
                    f1 = x.x == mn ? 1.f : ex2(x.x - mn);
                    m = mn;
                    l = l * f0 + x.y * f1;
                }
                tc_fence_after();
                const bool bad = s_bad[seg & 3] == seg + 1;
                const int head = s.head * a.G + g;
                const int64_t row = s.r + mytok;
                const int prow = (s.w == 2 ? wg * 128 : 0) + t;
                float* part = paged_slot(a, blockIdx.x, slot);
                if (valid && !whole) {
                    part[prow] = m;
                    part[a.slot_rows + prow] = l;
                } else if (valid && a.lse) {
                    a.lse[row * a.H + head] = (m + log2f(l)) * 0.693147180559945309f;
                }
                const float inv = whole ? 1.f / l : 1.f;
                // where this lane's row goes (0: nowhere)
                const uint64_t dst = !valid ? 0
                                     : whole ? (uint64_t)(a.o + (row * a.o_rs + (int64_t)head * D) * 2)
                                             : (uint64_t)(part + 2 * a.slot_rows + slot_at<D>(prow, 0));
                auto store = [&](uint4 (&v)[4], int at, int step) {
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        if (dst) *reinterpret_cast<uint4*>(dst + at + k * step) = v[k];
                };
#pragma unroll
                for (int c = 0; c < D; c += 32) {
                    float o[32];
                    tmem_ld32(o_col + c, o);
                    if (two) {
                        float o1[32];
                        tmem_ld32(o_col1 + c, o1);
                        tmem_wait_ld32(o);
                        tmem_wait_ld32(o1);
#pragma unroll
                        for (int j = 0; j < 32; ++j) o[j] = o[j] * f0 + o1[j] * f1;
                    } else {
                        tmem_wait_ld32(o);
                    }
                    if (!any) {
#pragma unroll
                        for (int j = 0; j < 32; ++j) o[j] = 0.f;
                    } else if (c + 32 == D) {
                        tc_fence_before();
                        mbar_arrive(o_free + wg);
                        if (two) mbar_arrive(o_free + 1);
                    }
                    uint4 v[4];
                    if (whole) {
#pragma unroll
                        for (int j = 0; j < 32; j += 8)
                            v[j / 8] = make_uint4(pack_bf16(o[j] * inv, o[j + 1] * inv), pack_bf16(o[j + 2] * inv, o[j + 3] * inv),
                                                  pack_bf16(o[j + 4] * inv, o[j + 5] * inv), pack_bf16(o[j + 6] * inv, o[j + 7] * inv));
                        store(v, 2 * c, 16);
                    } else {
#pragma unroll
                        for (int q = 0; q < 32; q += 16) {
#pragma unroll
                            for (int j = 0; j < 16; j += 4)
                                v[j / 4] = make_uint4(__float_as_uint(o[q + j]), __float_as_uint(o[q + j + 1]),
                                                      __float_as_uint(o[q + j + 2]), __float_as_uint(o[q + j + 3]));
                            store(v, 4 * slot_at<D>(0, c + q), 4 * slot_at<D>(0, 4));
                        }
                    }
                    __syncwarp();
                }
                if (bad && valid) {  // onto what the warp has just written
                    for (int c = 0; c < D; ++c) {
                        const float x = paged_nonfinite<kKT>(a, s, pos, c);
                        if (x == 0.f) continue;
                        __nv_bfloat16* at = reinterpret_cast<__nv_bfloat16*>(a.o) + row * a.o_rs + (int64_t)head * D + c;
                        if (whole) *at = __float2bfloat16_rn(__bfloat162float(*at) + x);
                        else part[2 * a.slot_rows + slot_at<D>(prow, c)] += x;
                    }
                }
            }
            uses1 += s.w == 2 || two;
            uses = wg ? uses1 : uses + (nsteps > 0);
            joins += two;
            base += 2 * T;
            __syncwarp();
            if (lane == 0) mbar_arrive(seg_empty + (seg & 1));
            ++seg;
        }
    }
    grid_launch_dependents();
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == kMmaWarp) tmem_dealloc(tmem, 512);
}

// Joins the partials of an item that was cut, as paged_merge_kernel does, from this
// kernel's slots: a warp takes four rows, eight lanes a row, and carries on maximum, sum
// and O from partial to partial (a partial's loads wait for nothing but the header).
constexpr int kMergeWarps = 4, kMergeRows = 4 * kMergeWarps;

template <int D>
__global__ void __launch_bounds__(32 * kMergeWarps) paged_tc_merge_kernel(const __grid_constant__ PagedArgs a) {
    grid_dependency_wait();
    const int c1 = blockIdx.x;
    const PagedHdr h = a.hdr[c1];
    const int lane = threadIdx.x % 32, piece = lane / 4;
    const int row = blockIdx.y * kMergeRows + threadIdx.x / 32 * 4 + lane % 4;  // of the slot
    // the item's row: an M tile's rows past its last token are empty
    const int per = a.tok1 * a.G, i = row < 128 ? row : row - 128 + per;
    if (h.kind != 2) return;
    const int n = c1 - h.c0 + 1;
    // of the first 32 CTAs, those that left something
    unsigned some = 0;
    if (h.gaps) some = __ballot_sync(0xffffffffu, lane < n && (lane == 0 || a.hdr[h.c0 + lane].kind != 0));
    if ((row & 127) >= per || i >= h.ntok * a.G) return;
    const int64_t stride = 2 * (int64_t)a.slot_rows * (D + 2);
    // partial k: slot B of CTA c0, then slot A of c0 + 1 ... c1
    const float* first = paged_slot(a, h.c0, 1);
    const float* rest = paged_slot(a, h.c0, 0);
    float m = -INFINITY, l = 0.f;
    float4 o[D / 32];
#pragma unroll
    for (int j = 0; j < D / 32; ++j) o[j] = make_float4(0.f, 0.f, 0.f, 0.f);
    auto join = [&](int k) {
        const float* p = k == 0 ? first : rest + k * stride;
        const float mk = p[row], lk = p[a.slot_rows + row];
        const float mn = fmaxf(m, mk);
        const float f = m == mn ? 1.f : exp2f(m - mn), w = mk == mn ? 1.f : exp2f(mk - mn);
        m = mn;
        l = l * f + lk * w;
#pragma unroll
        for (int j = 0; j < D / 32; ++j) {
            const float4 x = *reinterpret_cast<const float4*>(p + 2 * a.slot_rows + slot_at<D>(row, 32 * j + 4 * piece));
            o[j].x = o[j].x * f + x.x * w;
            o[j].y = o[j].y * f + x.y * w;
            o[j].z = o[j].z * f + x.z * w;
            o[j].w = o[j].w * f + x.w * w;
        }
    };
    if (h.gaps) {
        while (some) {
            const int k = __ffs(some) - 1;
            some &= some - 1;
            if (some) {  // two at a time, their loads together
                const int k2 = __ffs(some) - 1;
                some &= some - 1;
                join(k);
                join(k2);
            } else {
                join(k);
            }
        }
        for (int k = 32; k < n; ++k)
            if (a.hdr[h.c0 + k].kind != 0) join(k);
    } else {
#pragma unroll 2
        for (int k = 0; k < n; ++k) join(k);
    }
    const int tok = i / a.G, head = h.head * a.G + i - tok * a.G;
    const int64_t orow = h.row0 + tok;
    if (piece == 0 && a.lse) a.lse[orow * a.H + head] = m * 0.693147180559945309f + logf(l);
    const float inv = 1.f / l;
    char* dst = a.o + (orow * a.o_rs + (int64_t)head * D + 4 * piece) * 2;
#pragma unroll
    for (int j = 0; j < D / 32; ++j)
        *reinterpret_cast<uint2*>(dst + 64 * j) =
            make_uint2(pack_bf16(o[j].x * inv, o[j].y * inv), pack_bf16(o[j].z * inv, o[j].w * inv));
}

PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
    static PFN_cuTensorMapEncodeTiled_v12000 fn = [] {
        void* p = nullptr;
        cudaDriverEntryPointQueryResult r;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &r) != cudaSuccess ||
            r != cudaDriverEntryPointSuccess)
            p = nullptr;
        return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
    }();
    return fn;
}

template <int D, int ST, bool GROUPS>
cudaError_t launch(const PagedMaps& tm, const PagedArgs& a, int grid, cudaStream_t st) {
    static PerDeviceOnce once;
    constexpr int smem = Lay<D, ST>::TOTAL + 512;
    cudaError_t e = per_device_once(once, [] {
        return cudaFuncSetAttribute(paged_tc_kernel<D, ST, GROUPS>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    });
    if (e != cudaSuccess) return e;
    paged_tc_kernel<D, ST, GROUPS><<<grid, kThreads, smem, st>>>(tm, a);
    ripe_count_launch();
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    // rows of the items: M tile 1 begins at slot row 128
    const int most = a.max_ntok <= a.tok1 ? a.max_ntok * a.G : 128 + (min(a.max_ntok, a.tpt) - a.tok1) * a.G;
    return launch_paged_dependent(paged_tc_merge_kernel<D>, dim3((unsigned)grid, (unsigned)((most + kMergeRows - 1) / kMergeRows)),
                                  32 * kMergeWarps, st, a);
}

}  // namespace

// Maps of the pages ([pages][heads][positions][d], any strides) in boxes of `rows`
// positions of one page and head and `chunks` times 32 channels, which land one chunk
// behind the other.
bool paged_kv_map(void* map, const void* base, const PagedArgs& a, int rows, int chunks) {
    const auto encode = encode_fn();
    if (!encode) return false;
    const cuuint64_t dims[5] = {32, (cuuint64_t)a.page, (cuuint64_t)a.d / 32, (cuuint64_t)a.Hkv, (cuuint64_t)a.npages};
    const cuuint64_t strides[4] = {(cuuint64_t)a.pos_stride * 2, 64, (cuuint64_t)a.head_stride * 2, (cuuint64_t)a.page_stride * 2};
    const cuuint32_t box[5] = {32, (cuuint32_t)rows, (cuuint32_t)chunks, 1, 1};
    const cuuint32_t estr[5] = {1, 1, 1, 1, 1};
    return encode(reinterpret_cast<CUtensorMap*>(map), CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 5, const_cast<void*>(base), dims,
                  strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_64B,
                  CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

cudaError_t launch_paged_tc(PagedArgs a, int grid, cudaStream_t st) {
    PagedMaps tm;
    const auto encode = encode_fn();
    if (!encode) return cudaErrorNotSupported;
    const cuuint64_t dims[3] = {(cuuint64_t)a.d, (cuuint64_t)a.H, (cuuint64_t)a.nrows};
    const cuuint64_t strides[2] = {(cuuint64_t)a.d * 2, (cuuint64_t)a.q_rs * 2};
    const cuuint32_t box[3] = {32, (cuuint32_t)a.G, (cuuint32_t)a.tok1};
    const cuuint32_t estr[3] = {1, 1, 1};
    if (encode(&tm.q, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<char*>(a.q), dims, strides, box, estr,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_64B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
        return cudaErrorInvalidValue;
    const bool groups = a.page == 16;
    const int rows = groups ? 8 : a.page < kKT ? a.page : kKT, chunks = groups || rows == kKT ? a.d / 32 : 1;
    if (!paged_kv_map(&tm.k, a.k, a, rows, chunks) || !paged_kv_map(&tm.v, a.v, a, rows, chunks)) return cudaErrorInvalidValue;
    if (a.d == 32) return groups ? launch<32, 40, true>(tm, a, grid, st) : launch<32, 40, false>(tm, a, grid, st);
    if (a.d == 64) return groups ? launch<64, 22, true>(tm, a, grid, st) : launch<64, 22, false>(tm, a, grid, st);
    if (a.d == 96) return groups ? launch<96, 14, true>(tm, a, grid, st) : launch<96, 14, false>(tm, a, grid, st);
    if (a.d == 128) return groups ? launch<128, 10, true>(tm, a, grid, st) : launch<128, 10, false>(tm, a, grid, st);
    return cudaErrorInvalidValue;
}
