// ripe_paged_sm100.cu -- ripe_paged_attn on the tensor cores: chunks of new tokens
// (prompts, chunks of prompts, draft blocks with many rows) over a paged cache; bf16,
// head size 64, 96 or 128.
//
// Per item (row tile of tokens x the query heads of one key/value head, see
// ripe_paged.cuh): S = Q K^T and O += P V with the online softmax
//   m' = max(m, max_k S), P = 2^(c S - m'), l' = l 2^(m - m') + sum P, O' = O 2^(m - m') + P V
// (c = scale * log2 e).  m moves only when a row's maximum grew by more than 2^8: until
// then P stays below 2^8, which fp32 sums and bf16's exponent hold without loss, and the
// accumulator need not be read back.  l sums the unrounded P; P is rounded to bf16 for
// the second product (2^-8 of a weight at most, below the rounding of O itself).
//
// One persistent CTA per SM, 10 warps: two softmax warpgroups (one row per thread), a
// TMA warp, an MMA warp.  Two streams s = 0, 1, each with its own S and O in tensor
// memory (S 2 x 128 columns, P over S, O 2 x d columns), keep the tensor pipe busy with
// one stream's products while the other's softmax runs:
//   two M tiles (more than 128 rows): stream s is M tile s, both over the same key tile;
//   one M tile: stream s takes every second key tile, joined at the item's end.
// Keys and values arrive in 128-key tiles through one ring of shared-memory stages (K
// and V in turn), one TMA box per page (or 128 rows of it) and 32 channels, 64-byte
// swizzle.
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

constexpr int kKT = 128;       // keys per tile
constexpr int kThreads = 640;  // softmax warps 0-15 (8 a stream), the MMA warp, three TMA warps
constexpr int kMmaWarp = 16, kTmaWarp = 17, kTmaWarps = 3;
constexpr int kMinCost = 4;    // key tiles x M tiles a CTA takes at least (two key tiles of two M tiles)

struct alignas(64) PagedMaps {
    CUtensorMap q, k, v;
};

template <int D, int ST>
struct Lay {
    static constexpr int NCH = D / 32;         // 32-channel chunks
    static constexpr int TILE = NCH * 8192;    // 128 rows of bf16
    static constexpr int Q = 0;
    static constexpr int KV = 2 * TILE;
    static constexpr int BARS = KV + ST * TILE;
    static constexpr int NBAR = 2 * ST + 7 * 2 + 3 + 16;
    static constexpr int MX = BARS + ((NBAR * 8 + 15) / 16) * 16;  // [stream][half][128] maximum of a row's half
    static constexpr int ML = MX + 4 * 128 * 4;                    // [2][stream][half][128] l at an item's end, then [2][128] m of stream 1
    static constexpr int SEG = ML + 10 * 128 * 4;  // the segments under way, as the TMA warp found them
    static constexpr int MISC = SEG + 2 * 64;
    static constexpr int TOTAL = MISC + 64;
    static_assert(sizeof(PagedSeg) <= 64, "segment slots");
    static_assert(sizeof(PagedPlanSmem) <= (size_t)ST * TILE, "plan arrays over the stages");
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
// Exponential and packing that stay where they are written.
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
template <int N>
__device__ __forceinline__ void hide(float* v, uint32_t see) {
    constexpr uint32_t kAll = N == 32 ? ~0u : (1u << N) - 1;
    if (__all_sync(0xffffffffu, (see & kAll) == kAll)) return;
#pragma unroll
    for (int j = 0; j < N; ++j) v[j] = (see >> j) & 1 ? v[j] : -INFINITY;
}

// Zeros the values the matrix product must not see in a key tile that some row sees
// only in part: keys from `end` (of the tile) on, whose slots hold anything, and values
// that are not finite (returns whether there were any; paged_nonfinite puts them back
// where they are seen).  256 threads, 16 bytes at a time in the order they lie.  With two
// M tiles both streams clean the tile, each before its own product: what the later one
// still writes is what the earlier one wrote.
template <int NCH>
__device__ __forceinline__ bool clean_values(char* sv, int t, int end) {
    bool found = false;
#pragma unroll 4
    for (int i = t; i < NCH * 512; i += 256) {
        uint4* at = reinterpret_cast<uint4*>(sv) + i;
        uint4 x = *at;
        if (((i & 511) >> 2) >= end) {  // four 16-byte units a key
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
            *at = make_uint4(finite(x.x), finite(x.y), finite(x.z), finite(x.w));
            found = true;
        }
    }
    return found;
}

// Half a key tile of one row: S (64 columns at s_col) -> P over its first 32 columns, the
// running maximum m (log2 units; the whole row's, the other half's warp tells its own
// through `mx_mine`/`mx_other`) and this half's sum l, and half of O (D/2 columns at
// o_col) rescaled where the maximum moved.  PART: keys past `hi`, or up to `lo` and not
// below `first` (from the first of the 64), are hidden.  Two code paths, because the test
// alone costs the full tiles a third of their time once the compiler turns it into
// selects.  False if the wait for the other half gave up.
template <int D, bool PART>
__device__ __forceinline__ bool softmax_step(uint32_t s_col, uint32_t o_col, float c2, int hi, int lo, int first, bool valid,
                                             bool have_o, float& m, float& l, float* mx_mine, volatile float* mx_other,
                                             uint64_t* bar_mine, uint64_t* bar_other, uint32_t parity, int lane,
                                             volatile int* abort, int32_t* err) {
    // Two passes over S: the second read costs less than holding the scores.
    uint32_t see[2] = {~0u, ~0u};
    if (PART) {
#pragma unroll
        for (int c = 0; c < 2; ++c)
            see[c] = below(hi + 1 - 32 * c) & (~below(lo + 1 - 32 * c) | below(first - 32 * c));
    }
    float mx;
    {
        float x[32], y[32];
        tmem_ld32(s_col, x);
        tmem_ld32(s_col + 32, y);
        tmem_wait_ld32(x);
        tmem_wait_ld32(y);
        if (PART) {
            hide<32>(x, see[0]);
            hide<32>(y, see[1]);
        }
        float m0 = x[0], m1 = y[0];
#pragma unroll
        for (int j = 1; j < 31; j += 2) {
            m0 = max3(m0, x[j], x[j + 1]);
            m1 = max3(m1, y[j], y[j + 1]);
        }
        mx = fmaxf(max3(m0, x[31], y[31]), m1);
    }
    *mx_mine = mx;
    __syncwarp();
    if (lane == 0) mbar_arrive(bar_other);
    if (!__all_sync(0xffffffffu, mbar_wait_idle(bar_mine, parity, abort, err))) return false;
    mx = fmaxf(mx, *mx_other) * c2;
    const bool grow = valid && mx > m + 8.f;  // m = -inf: any finite maximum
    if (__any_sync(0xffffffffu, grow)) {
        const float mn = grow ? mx : m;
        const float f = m == mn ? 1.f : ex2(m - mn);  // 0 from m = -inf
        m = mn;
        l *= f;
        if (have_o) {
            // The stream's earlier P V are complete: s_full came after them.
#pragma unroll
            for (int c = 0; c < D / 2; c += 16) {
                float o[16];
                tmem_ld16(o_col + c, o);
                tmem_wait_ld16(o);
#pragma unroll
                for (int j = 0; j < 16; ++j) o[j] *= f;
                tmem_st16(o_col + c, reinterpret_cast<const uint32_t*>(o));
            }
        }
    }
    const float mref = m == -INFINITY ? 0.f : m;
    // Exponentials of chunk c while chunk c - 1 is summed and packed: written out in
    // that order (the asm statements keep it), because the exponential unit takes a
    // warp 8 cycles an instruction and a warp that waits for each result idles it.
    float l0 = 0.f, l1 = 0.f;
    float v[3][16];
    tmem_ld16(s_col, v[0]);
#pragma unroll
    for (int c = 0; c <= 4; ++c) {
        float *x = v[c % 3], *y = v[(c + 2) % 3];
        uint32_t w[8];
        if (c < 4) {
            tmem_wait_ld16(x);
            if (c < 3) tmem_ld16(s_col + 16 * (c + 1), v[(c + 1) % 3]);
            if (PART) hide<16>(x, see[c / 2] >> (c % 2 * 16));
#pragma unroll
            for (int j = 0; j < 16; ++j) x[j] = fmaf(x[j], c2, -mref);
        }
#pragma unroll
        for (int j = 0; j < 16; j += 2) {
            if (c < 4) x[j] = ex2_here(x[j]);
            if (c > 0) {
                l0 += y[j];
                l1 += y[j + 1];
            }
            if (c < 4) x[j + 1] = ex2_here(x[j + 1]);
            if (c > 0) w[j / 2] = pack_here(y[j], y[j + 1]);
        }
        if (c > 0) tmem_st8(s_col + 8 * (c - 1), w);  // over columns read before
    }
    l += l0 + l1;
    return true;
}

template <int D, int ST>
__global__ void __launch_bounds__(kThreads, 1) paged_tc_kernel(const __grid_constant__ PagedMaps tm,
                                                               const __grid_constant__ PagedArgs a) {
    using L = Lay<D, ST>;
    constexpr int NCH = L::NCH;
    extern __shared__ char smem_raw[];
    char* smem = reinterpret_cast<char*>((reinterpret_cast<uintptr_t>(smem_raw) + 511) & ~(uintptr_t)511);
    char* sQ = smem + L::Q;
    char* sKV = smem + L::KV;
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + L::BARS);
    uint64_t *kv_full = bars, *kv_empty = bars + ST, *s_full = bars + 2 * ST, *p_full = s_full + 2, *o_full = p_full + 2,
             *o_free = o_full + 2, *seg_full = o_free + 2, *seg_empty = seg_full + 2, *ml_full = seg_empty + 2, *q_full = ml_full + 2,
             *q_free = q_full + 1, *drain = q_free + 1, *mx_full = drain + 1;
    float* s_mx = reinterpret_cast<float*>(smem + L::MX);
    float *s_l = reinterpret_cast<float*>(smem + L::ML), *s_m1 = s_l + 8 * 128;
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
        for (int i = 0; i < 2; ++i) {
            mbar_init(s_full + i, 1);
            mbar_init(p_full + i, 256);
            mbar_init(o_full + i, 1);
            mbar_init(o_free + i, 256);
            mbar_init(ml_full + i, 256);
            mbar_init(seg_full + i, 1);
            mbar_init(seg_empty + i, 16 + kTmaWarps);  // all but the warp that fills it
        }
        mbar_init(q_full, 1);
        mbar_init(q_free, 1);
        for (int i = 0; i < 16; ++i) mbar_init(mx_full + i, 1);
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
    plan.template begin<kThreads>(a, *reinterpret_cast<PagedPlanSmem*>(sKV), kMinCost);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *s_tmem;

    if (warp >= kTmaWarp) {
        // ------------------------------------------------------------ TMA producers
        // A tile is nsub (pages, or 128 keys of one) x NCH boxes, dealt to the lanes of three
        // warps: a lane's copy takes the warp about 64 cycles to issue, so with pages of 16
        // keys one warp alone would hold a tile back for 4100 cycles (measured: 15 bytes per
        // cycle and SM instead of the 23 that HBM gives).
        const int pw = warp - kTmaWarp, b = lane * kTmaWarps + pw;
        const int pb = a.page < kKT ? a.page : kKT, nsub = kKT / pb;
        const int sub = b / NCH, ch = b % NCH;
        const uint32_t box = (uint32_t)pb * 64;
        char* dst = sKV + ch * 8192 + sub * (int)box;
        int st = 0, ph = 1, n = 0;  // stage, its empty parity (the first round passes), segments begun
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
            const int end = slot->c + slot->t0 + slot->ntok, head = slot->head, seq = slot->seq;
            const PagedTiles tiles = slot->tiles;
            if (pw == 0) {
                if (!(ok = warp_wait(q_free, (n & 1) ^ 1, abort_flag, a.err))) break;
                if (lane == 0) {
                    mbar_expect_tx(q_full, slot->w * NCH * ((uint32_t)a.tok1 * a.G * 64));
                    for (int mt = 0; mt < slot->w; ++mt)
                        for (int c = 0; c < NCH; ++c)
                            tma_load_3d(sQ + (mt * NCH + c) * 8192, &tm.q, 32 * c, head * a.G,
                                        slot->r + slot->t0 + mt * a.tok1, q_full);
                }
                __syncwarp();
            } else {
                __syncwarp();
                if (lane == 0) mbar_arrive(seg_empty + (n & 1));
            }
            auto page_of = [&](int t) {
                const int key = tiles.tile(t) * kKT + sub * pb;
                return t < tb && sub < nsub && key < end ? paged_page(a, seq, key) : -1;
            };
            int id = page_of(ta);
            for (int t = ta; t < tb && ok; ++t) {
                const int next_id = page_of(t + 1);
                const int k0 = tiles.tile(t) * kKT, y = (k0 + sub * pb) & (a.page - 1);
#pragma unroll
                for (int kv = 0; kv < 2; ++kv) {
                    if (!(ok = warp_wait(kv_empty + st, ph, abort_flag, a.err))) break;
                    if (pw == 0 && lane == 0)
                        mbar_expect_tx(kv_full + st, min(nsub, (end - k0 + pb - 1) / pb) * NCH * box);
                    if (id >= 0) tma_load_4d(dst + st * L::TILE, kv ? &tm.v : &tm.k, 32 * ch, y, head, id, kv_full + st);
                    __syncwarp();
                    if (++st == ST) {
                        st = 0;
                        ph ^= 1;
                    }
                }
                id = next_id;
            }
        }
        // Every copy has landed before the CTA's shared memory goes away: on the ordinary
        // way out the MMA warp waited for all of them.  Otherwise a stage may lack the first
        // warp's share of the bytes it expects, so give the copies time instead of waiting on it.
        if (!ok || *abort_flag) {
            const long long t0 = clock64();
            while (clock64() - t0 < (1 << 20)) {}
        }
    } else if (warp == kMmaWarp) {
        // ------------------------------------------------------------ MMA issuer
        if (elect_one()) {
            constexpr uint32_t IDESC_QK = idesc_bf16(128, kKT, 0), IDESC_PV = idesc_bf16(128, D, 1);
            const uint64_t dq = smem_desc(smem_u32(sQ), 16, 512, kLayoutSwizzle64B);
            const uint64_t dk = smem_desc(smem_u32(sKV), 16, 512, kLayoutSwizzle64B);
            const uint64_t dv = smem_desc(smem_u32(sKV), 8192, 512, kLayoutSwizzle64B);
            int seg = 0, st0 = 0, ph0 = 0;  // the segment's first stage
            uint32_t steps[2] = {0, 0}, uses[2] = {0, 0};
            bool ok = true;
            // stage `k` places after (st0, ph0); k < 2 * ST
            auto at = [&](int k, int& st, uint32_t& ph) {
                st = st0 + k;
                ph = ph0;
                while (st >= ST) {
                    st -= ST;
                    ph ^= 1;
                }
            };
            // S of stream s = Q tile `qt` x K in stage st
            auto qk = [&](auto s, int qt, int st) {
#pragma unroll
                for (int ks = 0; ks < D / 16; ++ks) {
                    constexpr uint32_t u = 1;  // 16-byte units
                    const uint32_t o = ((ks >> 1) * 8192 + (ks & 1) * 32) / 16 * u;
                    mma_bf16(tmem + 128 * s.value, dq + qt * (L::TILE / 16) + o, dk + st * (L::TILE / 16) + o, IDESC_QK,
                             ks > 0 ? 1u : 0u);
                }
                mma_commit(s_full + s.value);
            };
            // O of stream s += P x V in stage st; waits for P, and for O before its first use
            auto pv = [&](auto s, bool first, int st, uint32_t ph) -> bool {
                if (!mbar_wait_idle(p_full + s.value, steps[s.value]++ & 1, abort_flag, a.err)) return false;
                if (first && !mbar_wait_idle(o_free + s.value, (uses[s.value]++ & 1) ^ 1, abort_flag, a.err)) return false;
                if (!mbar_wait_idle(kv_full + st, ph, abort_flag, a.err)) return false;
                tc_fence_after();
#pragma unroll
                for (int ks = 0; ks < kKT / 16; ++ks)
                    mma_bf16_ts(tmem + 256 + D * s.value, tmem + 128 * s.value + (ks & 3) * 8 + (ks >> 2) * 64,
                                dv + st * (L::TILE / 16) + ks * 64, IDESC_PV, (!first || ks > 0) ? 1u : 0u);
                return true;
            };
            const std::integral_constant<int, 0> s0{};
            const std::integral_constant<int, 1> s1{};
            while ((ok = mbar_wait_idle(seg_full + (seg & 1), (seg >> 1) & 1, abort_flag, a.err))) {
                const PagedSeg& s = *s_seg[seg & 1];
                const int T = s.tb - s.ta;
                const bool two = s.w == 2;
                mbar_arrive(seg_empty + (seg & 1));
                if (T == 0) break;
                if (!(ok = mbar_wait_idle(q_full, seg & 1, abort_flag, a.err))) break;
                ++seg;
                int st, kst;
                uint32_t ph, kph;
                // stages in order: K 0, V 0, K 1, V 1, ...
                at(0, st, ph);
                if (!(ok = mbar_wait_idle(kv_full + st, ph, abort_flag, a.err))) break;
                if (two) {
                    qk(s0, 0, st);
                    qk(s1, 1, st);
                    mma_commit(kv_empty + st);
                    if (T == 1) mma_commit(q_free);
                    for (int i = 0; i < T; ++i) {
                        at(1, st, ph);
                        at(2, kst, kph);
                        const bool last = i + 1 == T;
                        if (!(ok = pv(s0, i == 0, st, ph))) break;
                        if (last) {
                            mma_commit(o_full);
                        } else {
                            if (!(ok = mbar_wait_idle(kv_full + kst, kph, abort_flag, a.err))) break;
                            qk(s0, 0, kst);
                        }
                        if (!(ok = pv(s1, i == 0, st, ph))) break;
                        mma_commit(kv_empty + st);
                        if (last) {
                            mma_commit(o_full + 1);
                        } else {
                            qk(s1, 1, kst);
                            mma_commit(kv_empty + kst);
                            if (i + 2 == T) mma_commit(q_free);
                        }
                        at(2, st0, kph);
                        ph0 = kph;
                    }
                } else {
                    qk(s0, 0, st);
                    mma_commit(kv_empty + st);
                    if (T > 1) {
                        at(2, st, ph);
                        if (!(ok = mbar_wait_idle(kv_full + st, ph, abort_flag, a.err))) break;
                        qk(s1, 0, st);
                        mma_commit(kv_empty + st);
                    }
                    if (T <= 2) mma_commit(q_free);
                    for (int i = 0; i < T; ++i) {
                        at(1, st, ph);
                        if (!(ok = i & 1 ? pv(s1, i == 1, st, ph) : pv(s0, i == 0, st, ph))) break;
                        mma_commit(kv_empty + st);
                        if (i + 2 < T) {
                            at(4, kst, kph);
                            if (!(ok = mbar_wait_idle(kv_full + kst, kph, abort_flag, a.err))) break;
                            if (i & 1) qk(s1, 0, kst); else qk(s0, 0, kst);
                            mma_commit(kv_empty + kst);
                            if (i + 3 == T) mma_commit(q_free);
                        } else {
                            mma_commit(o_full + (i & 1));
                        }
                        at(2, st0, kph);
                        ph0 = kph;
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
        // Warp: stream warp / 8, columns (of S and of O) of half (warp / 4) % 2, rows of
        // quarter warp % 4.  Two warps a row, because one warp per scheduler and stream left
        // the exponential unit half idle (2600 cycles a tile against 1060 at its rate).
        const int wg = warp / 8, half = (warp / 4) % 2, t = threadIdx.x % 128;  // t: TMEM lane = row of the M tile
        const uint32_t lane_addr = (uint32_t)((warp % 4) * 32) << 16;
        const uint32_t s_col = tmem + 128 * wg + 64 * half + lane_addr, o_col1 = tmem + 256 + D + D / 2 * half + lane_addr,
                       o_col = wg ? o_col1 : o_col1 - D;
        float* mx_mine = s_mx + (wg * 2 + half) * 128 + t;
        float* mx_other = s_mx + (wg * 2 + (half ^ 1)) * 128 + t;
        const float c2 = a.scale_log2;
        const int tok = t / a.G, g = t - tok * a.G;
        int base = 0, seg = 0, steps = 0, uses = 0, uses1 = 0;  // uses: of this stream, and of stream 1, as in the MMA warp
        if (threadIdx.x == 0) a.hdr[blockIdx.x].kind = 0;
        bool ok = true;
        while (ok && (ok = warp_wait(seg_full + (seg & 1), (seg >> 1) & 1, abort_flag, a.err))) {
            const PagedSeg& s = *s_seg[seg & 1];
            const int T = s.tb - s.ta;
            if (T == 0) break;
            const int mytok = s.t0 + (s.w == 2 ? wg * a.tok1 : 0) + tok;  // this row's token
            const bool valid = tok < a.tok1 && mytok < s.t0 + s.ntok;
            const int pos = s.c + mytok;
            const int p0 = s.c + s.t0, p1 = p0 + s.ntok - 1;
            const int nsteps = s.w == 2 ? T : (T + 1 - wg) / 2;
            float m = -INFINITY, l = 0.f;
            for (int n = 0; n < nsteps && ok; ++n, ++steps) {
                const int i = s.w == 2 ? n : 2 * n + wg;
                const int k0 = s.tiles.tile(s.ta + i) * kKT;
                const bool part = !paged_all_seen(a, k0, kKT, p0, p1);
                if (!(ok = warp_wait(s_full + wg, steps & 1, abort_flag, a.err))) break;
                tc_fence_after();
                if (part) {
                    // Only once the scores are there: they come after the products that used
                    // the stage before, so the parity cannot be that of an earlier round.
                    const int k = base + 2 * i + 1, st = k % ST;
                    if (!(ok = warp_wait(kv_full + st, (k / ST) & 1, abort_flag, a.err))) break;
                    if (clean_values<NCH>(sKV + st * L::TILE, threadIdx.x % 256, p1 + 1 - k0)) {
                        s_bad[seg & 3] = seg + 1;
                        __threadfence_block();
                    }
                    fence_proxy_async_smem();
                    __syncwarp();
                }
                const int kh = k0 + 64 * half;
                if (part)
                    ok = softmax_step<D, true>(s_col, o_col, c2, pos - kh, a.window > 0 ? pos - a.window - kh : -1,
                                               a.sinks - kh, valid, n > 0, m, l, mx_mine, mx_other, mx_full + warp,
                                               mx_full + (warp ^ 4), steps & 1, lane, abort_flag, a.err);
                else
                    ok = softmax_step<D, false>(s_col, o_col, c2, 0, 0, 0, valid, n > 0, m, l, mx_mine, mx_other,
                                                mx_full + warp, mx_full + (warp ^ 4), steps & 1, lane, abort_flag, a.err);
                if (!ok) break;
                tmem_wait_st();
                tc_fence_before();
                mbar_arrive(p_full + wg);
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
                a.hdr[blockIdx.x] = h;
            }
            const bool two = s.w == 1 && T > 1;  // both streams hold a part of the one M tile
            if (s.w == 2 || two || wg == 0) {
                s_l[((uses & 1) * 4 + wg * 2 + half) * 128 + t] = l;
                if (two && wg == 1 && half == 0) s_m1[(uses & 1) * 128 + t] = m;
                mbar_arrive(ml_full + wg);
            }
            if (s.w == 2 || wg == 0) {
                if (!(ok = warp_wait(ml_full + wg, uses & 1, abort_flag, a.err))) break;
                l += s_l[((uses & 1) * 4 + wg * 2 + (half ^ 1)) * 128 + t];
                if (!(ok = warp_wait(o_full + wg, uses & 1, abort_flag, a.err))) break;
                float f0 = 1.f, f1 = 0.f;
                if (two) {
                    if (!(ok = warp_wait(ml_full + 1, uses1 & 1, abort_flag, a.err))) break;
                    if (!(ok = warp_wait(o_full + 1, uses1 & 1, abort_flag, a.err))) break;
                    const float* l1 = s_l + ((uses1 & 1) * 4 + 2) * 128 + t;
                    const float m1 = s_m1[(uses1 & 1) * 128 + t], mn = fmaxf(m, m1);
                    f0 = m == mn ? 1.f : ex2(m - mn);
                    f1 = m1 == mn ? 1.f : ex2(m1 - mn);
                    m = mn;
                    l = l * f0 + (l1[0] + l1[128]) * f1;
                }
                tc_fence_after();
                const bool bad = s_bad[seg & 3] == seg + 1;
                const int head = s.head * a.G + g;
                const int64_t row = s.r + mytok;
                const int prow = (s.w == 2 ? wg * 128 : 0) + t;
                float* part = paged_slot(a, blockIdx.x, slot);
                if (valid && half == 0) {
                    if (!whole) {
                        part[prow] = m;
                        part[a.slot_rows + prow] = l;
                    } else if (a.lse) {
                        a.lse[row * a.H + head] = (m + log2f(l)) * 0.693147180559945309f;
                    }
                }
                const float inv = whole ? 1.f / l : 1.f;
                const int c0 = D / 2 * half;
#pragma unroll
                for (int c = 0; c < D / 2; c += 16) {
                    float o[16];
                    tmem_ld16(o_col + c, o);
                    if (two) {
                        float o1[16];
                        tmem_ld16(o_col1 + c, o1);
                        tmem_wait_ld16(o);
                        tmem_wait_ld16(o1);
#pragma unroll
                        for (int j = 0; j < 16; ++j) o[j] = o[j] * f0 + o1[j] * f1;
                    } else {
                        tmem_wait_ld16(o);
                    }
                    if (c + 16 == D / 2) {
                        tc_fence_before();
                        mbar_arrive(o_free + wg);
                        if (two) mbar_arrive(o_free + 1);
                    }
                    if (valid && whole) {
                        uint4* dst = reinterpret_cast<uint4*>(a.o + (row * a.o_rs + (int64_t)head * D + c0 + c) * 2);
#pragma unroll
                        for (int j = 0; j < 16; j += 8)
                            dst[j / 8] = make_uint4(pack_bf16(o[j] * inv, o[j + 1] * inv), pack_bf16(o[j + 2] * inv, o[j + 3] * inv),
                                                    pack_bf16(o[j + 4] * inv, o[j + 5] * inv), pack_bf16(o[j + 6] * inv, o[j + 7] * inv));
                    } else if (valid) {
                        float4* dst = reinterpret_cast<float4*>(part + 2 * a.slot_rows + (int64_t)prow * D + c0 + c);
#pragma unroll
                        for (int j = 0; j < 16; j += 4) dst[j / 4] = make_float4(o[j], o[j + 1], o[j + 2], o[j + 3]);
                    }
                    __syncwarp();
                }
                if (bad && valid) {  // onto what this thread has just written
                    for (int c = c0; c < c0 + D / 2; ++c) {
                        const float x = paged_nonfinite<kKT>(a, s, pos, c);
                        if (x == 0.f) continue;
                        __nv_bfloat16* at = reinterpret_cast<__nv_bfloat16*>(a.o) + row * a.o_rs + (int64_t)head * D + c;
                        if (whole) *at = __float2bfloat16_rn(__bfloat162float(*at) + x);
                        else part[2 * a.slot_rows + (int64_t)prow * D + c] += x;
                    }
                }
            }
            uses1 += s.w == 2 || two;
            uses = wg ? uses1 : uses + 1;
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

template <int D, int ST>
cudaError_t launch(const PagedMaps& tm, const PagedArgs& a, int grid, cudaStream_t st) {
    static PerDeviceOnce once;
    constexpr int smem = Lay<D, ST>::TOTAL + 512;
    cudaError_t e = per_device_once(once, [] {
        return cudaFuncSetAttribute(paged_tc_kernel<D, ST>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    });
    if (e != cudaSuccess) return e;
    paged_tc_kernel<D, ST><<<grid, kThreads, smem, st>>>(tm, a);
    ripe_count_launch();
    return cudaGetLastError();
}

}  // namespace

// Maps of the pages ([pages][heads][positions][d], any strides) in boxes of `rows`
// positions of one page and head and 32 channels.
bool paged_kv_map(void* map, const void* base, const PagedArgs& a, int rows) {
    const auto encode = encode_fn();
    if (!encode) return false;
    const cuuint64_t dims[4] = {(cuuint64_t)a.d, (cuuint64_t)a.page, (cuuint64_t)a.Hkv, (cuuint64_t)a.npages};
    const cuuint64_t strides[3] = {(cuuint64_t)a.pos_stride * 2, (cuuint64_t)a.head_stride * 2, (cuuint64_t)a.page_stride * 2};
    const cuuint32_t box[4] = {32, (cuuint32_t)rows, 1, 1};
    const cuuint32_t estr[4] = {1, 1, 1, 1};
    return encode(reinterpret_cast<CUtensorMap*>(map), CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(base), dims,
                  strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_64B,
                  CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

int paged_tc_slot_rows() { return 256; }

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
    const int rows = a.page < kKT ? a.page : kKT;
    if (!paged_kv_map(&tm.k, a.k, a, rows) || !paged_kv_map(&tm.v, a.v, a, rows)) return cudaErrorInvalidValue;
    if (a.d == 64) return launch<64, 11>(tm, a, grid, st);
    if (a.d == 96) return launch<96, 7>(tm, a, grid, st);
    if (a.d == 128) return launch<128, 4>(tm, a, grid, st);
    return cudaErrorInvalidValue;
}
