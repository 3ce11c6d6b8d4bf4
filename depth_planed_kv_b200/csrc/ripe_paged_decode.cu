// ripe_paged_decode.cu -- ripe_paged_attn for few rows: at most 16 rows per key/value
// head and sequence (single tokens, short draft blocks); bf16, head size 32, 64, 96 or 128.
//
// The keys and values are read once and each feeds at most 16 rows, so the bytes are
// what counts: a row tile of 128 in the tensor-memory kernel would be 7/8 empty, and
// its pipeline's hand-overs cost more than the loads.  Here each warp streams its own
// 16 keys of every 64-key tile through its own ring of stages (one TMA box for the keys
// and one for the values; the warp that waits is the one that reuses the stage, so there
// is no other hand-over) and keeps its own running maximum, sum and output in registers:
//   S^T = K Q^T (keys on the 16-row side of m16n8k16, rows on its 8-column side),
//   P^T by an 8x8 transpose in registers, O^T += V^T P^T.
// The four warps of a CTA join at an item's end through shared memory; the running
// maximum moves only when it grew by more than 2^8 (as in ripe_paged_sm100.cu), so most
// blocks need no exchange between lanes at all.
//
// Measured with the merge: 16 sequences of 32768 keys, 32 query heads over 8, head size
// 128, one token each: 340 us for 2.15 GB, 6.3 TB/s (a plain copy reaches 6.55).  One
// sequence of 1024 keys and 55 heads of size 96: 14.0 us for 21.6 MB, bound by the chain of
// latencies (plan, table, keys and values, join, then the merge kernel).  DRAM 77% and 17%
// of peak.
#include <cuda.h>
#include <math.h>

#include "ripe_launch.h"
#include "ripe_paged.cuh"
#include "ripe_paged_launch.h"
#include "sm100_ptx.cuh"

using namespace sm100;

namespace {

constexpr int kWarps = 4, kThreads = 32 * kWarps;
constexpr int kKT = 16 * kWarps;  // keys per tile: 16 per warp
constexpr int kMinCost = 1;       // key tiles a CTA takes at least (2: 5 short sequences 11 us, 1: 8)

struct alignas(64) DecodeMaps {
    CUtensorMap k, v;
};

template <int D, int NS>
struct Lay {
    static constexpr int NCH = D / 32;
    static constexpr int BLK = NCH * 1024;  // 16 keys of bf16
    static constexpr int HC = D / 2, PITCH = HC + 4;
    static constexpr int STAGES = 0;        // [warp][NS][K, V]
    static constexpr int BUF = STAGES + kWarps * NS * 2 * BLK;     // [warp][8][PITCH] floats
    static constexpr int ML = BUF + kWarps * 8 * PITCH * 4;        // [warp][16] (m, l)
    static constexpr int BARS = ML + kWarps * 16 * 8;              // [warp][NS]
    static constexpr int MISC = BARS + kWarps * NS * 8;            // bad [warp], abort
    static constexpr int PLAN = MISC + 32;
    static constexpr int TOTAL = PLAN + (int)sizeof(PagedPlanHead);
    static_assert(sizeof(PagedPlanSmem) <= (size_t)BUF, "plan arrays over the stages");
    static_assert(TOTAL + 512 + 1024 <= 116736, "two CTAs per SM");
};

template <int D, int NR, int NS>
__global__ void __launch_bounds__(kThreads, 2) paged_decode_kernel(const __grid_constant__ DecodeMaps tm,
                                                                   const __grid_constant__ PagedArgs a) {
    using L = Lay<D, NS>;
    constexpr int NCH = L::NCH, KS = D / 16;
    extern __shared__ char smem_raw[];
    char* smem = reinterpret_cast<char*>((reinterpret_cast<uintptr_t>(smem_raw) + 511) & ~(uintptr_t)511);
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    char* st_base = smem + L::STAGES + warp * NS * 2 * L::BLK;
    float* buf = reinterpret_cast<float*>(smem + L::BUF);
    float2* s_ml = reinterpret_cast<float2*>(smem + L::ML);
    uint64_t* full = reinterpret_cast<uint64_t*>(smem + L::BARS) + warp * NS;
    volatile int* s_bad = reinterpret_cast<volatile int*>(smem + L::MISC);
    volatile int* abort_flag = s_bad + kWarps;

    if (threadIdx.x == 0) {
        for (int i = 0; i < kWarps * NS; ++i) mbar_init(reinterpret_cast<uint64_t*>(smem + L::BARS) + i, 1);
        fence_barrier_init();
        *abort_flag = 0;
        a.hdr[blockIdx.x].kind = 0;
        prefetch_tmap(&tm.k);
        prefetch_tmap(&tm.v);
    }
    PagedPlan<kKT> plan;
    plan.template begin<kThreads>(a, *reinterpret_cast<PagedPlanHead*>(smem + L::PLAN),
                                  *reinterpret_cast<PagedPlanSmem*>(smem + L::STAGES), kMinCost);

    // ---- the warp's loads: its live blocks of all items in order, NS ahead
    PagedPlan<kKT> iplan = plan;
    PagedSeg is;
    int it_t = 0, issued = 0, first = 0, ent = 0;  // ent: lane i, the table's entry for tile first + i of the item
    bool more = iplan.next(a, is);
    // One load for 32 tiles' pages (a load per tile would hold each issue for its latency).
    auto look_up = [&]() {
        first = it_t;
        const int t = it_t + lane, kb = is.tiles.tile(is.ta + t) * kKT + warp * 16;
        ent = t < is.tb - is.ta && kb < is.c + is.t0 + is.ntok ? paged_entry(a, is.seq, kb) : 0;
    };
    if (more) look_up();
    // Moves to the next block with a key some row sees.
    auto seek = [&]() {
        while (more) {
            while (it_t < is.tb - is.ta) {
                const int kb = is.tiles.tile(is.ta + it_t) * kKT + warp * 16, p0 = is.c + is.t0;
                if (paged_any_seen(a, kb, 16, p0, p0 + is.ntok - 1)) {
                    if (it_t - first >= 32) look_up();
                    return;
                }
                ++it_t;
            }
            it_t = 0;
            more = iplan.next(a, is);
            if (more) look_up();
        }
    };
    auto issue = [&]() {
        if (!more) return;
        const int st = issued % NS;
        char* dst = st_base + st * 2 * L::BLK;
        const int y = (is.tiles.tile(is.ta + it_t) * kKT + warp * 16) & (a.page - 1);
        const int page = paged_checked(a, __shfl_sync(0xffffffffu, ent, it_t - first));
        if (lane == 0) mbar_expect_tx(full + st, 2 * L::BLK);
        __syncwarp();
        if (lane < 2) tma_load_5d(dst + lane * L::BLK, lane ? &tm.v : &tm.k, 0, y, 0, is.head, page, full + st);
        ++issued;
        ++it_t;
        seek();
    };
    seek();
    for (int i = 0; i < NS; ++i) issue();

    const float c2 = a.scale_log2;
    const int gq = lane / 4, tq = lane % 4;
    PagedSeg s;
    int used = 0;
    while (plan.next(a, s)) {
        const int rows = s.ntok * a.G, p0 = s.c + s.t0, p1 = p0 + s.ntok - 1;
        // Q as the B operand: row gq of each 8, channels 2 tq and 2 tq + 8 of each 16.
        uint32_t qf[NR][KS][2];
        int pos[NR][2];
#pragma unroll
        for (int nr = 0; nr < NR; ++nr) {
            const int row = nr * 8 + gq, tok = row / a.G;
            const bool on = row < rows;
            const char* src = a.q + ((s.r + s.t0 + tok) * a.q_rs + (int64_t)(s.head * a.G + row - tok * a.G) * D + 2 * tq) * 2;
#pragma unroll
            for (int ks = 0; ks < KS; ++ks)
#pragma unroll
                for (int j = 0; j < 2; ++j)
                    qf[nr][ks][j] = on ? __ldg(reinterpret_cast<const uint32_t*>(src + (ks * 16 + j * 8) * 2)) : 0u;
            pos[nr][0] = p0 + (nr * 8 + 2 * tq) / a.G;
            pos[nr][1] = p0 + (nr * 8 + 2 * tq + 1) / a.G;
        }
        float o[NR][KS][4], m[NR][2], l[NR][2];
#pragma unroll
        for (int nr = 0; nr < NR; ++nr) {
#pragma unroll
            for (int mt = 0; mt < KS; ++mt)
#pragma unroll
                for (int j = 0; j < 4; ++j) o[nr][mt][j] = 0.f;
            m[nr][0] = m[nr][1] = -INFINITY;
            l[nr][0] = l[nr][1] = 0.f;
        }
        bool bad = false;
        for (int t = s.ta; t < s.tb; ++t) {
            const int kb = s.tiles.tile(t) * kKT + warp * 16;
            if (!paged_any_seen(a, kb, 16, p0, p1)) continue;
            const int st = used % NS;
            char* sk = st_base + st * 2 * L::BLK;
            if (!__all_sync(0xffffffffu, mbar_wait(full + st, (used / NS) & 1, abort_flag, a.err))) break;
            ++used;
            const uint32_t ka = smem_u32(sk), va = ka + L::BLK;
            float sc[NR][4];
#pragma unroll
            for (int nr = 0; nr < NR; ++nr)
#pragma unroll
                for (int j = 0; j < 4; ++j) sc[nr][j] = 0.f;
            {
                const int key = ((lane >> 3) & 1) * 8 + (lane & 7), sw = (key >> 1) & 3, hi = lane >> 4;
#pragma unroll
                for (int ks = 0; ks < KS; ++ks) {
                    uint32_t a0, a1, a2, a3;
                    ldsm_x4(ka + (ks >> 1) * 1024 + key * 64 + ((((ks & 1) * 2 + hi) ^ sw) << 4), a0, a1, a2, a3);
#pragma unroll
                    for (int nr = 0; nr < NR; ++nr) mma_16816(sc[nr], a0, a1, a2, a3, qf[nr][ks][0], qf[nr][ks][1]);
                }
            }
            if (!paged_all_seen(a, kb, 16, p0, p1)) {
#pragma unroll
                for (int nr = 0; nr < NR; ++nr)
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        if (!paged_seen(a, kb + gq + (j >> 1) * 8, pos[nr][j & 1])) sc[nr][j] = -INFINITY;
                // What the second product must not see: slots past the last token, and
                // values that are not finite (put back where they are seen at the item's end).
                const int key = lane >> 1;
                bool found = false;
#pragma unroll
                for (int c = 0; c < NCH; ++c) {
#pragma unroll
                    for (int u = 0; u < 2; ++u) {
                        uint4* p = reinterpret_cast<uint4*>(sk + L::BLK + c * 1024 + key * 64 + ((lane & 1) * 2 + u) * 16);
                        uint4 x = *p;
                        uint32_t* w = reinterpret_cast<uint32_t*>(&x);
                        bool ch = false;
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            if ((w[j] & 0x7F80u) == 0x7F80u) {
                                w[j] &= 0xFFFF0000u;
                                ch = true;
                            }
                            if ((w[j] & 0x7F800000u) == 0x7F800000u) {
                                w[j] &= 0xFFFFu;
                                ch = true;
                            }
                        }
                        if (kb + key > p1) {
                            *p = make_uint4(0, 0, 0, 0);
                        } else if (ch) {
                            *p = x;
                            found = true;
                        }
                    }
                }
                bad |= __any_sync(0xffffffffu, found);
                fence_proxy_async_smem();  // before a copy lands there again
                __syncwarp();
            }
            // scaled maxima of this lane's rows; m moves when one outgrows it by 2^8
            bool grow = false;
            float mx[NR][2];
#pragma unroll
            for (int nr = 0; nr < NR; ++nr)
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    mx[nr][j] = fmaxf(sc[nr][j], sc[nr][j + 2]) * c2;
                    grow |= mx[nr][j] > m[nr][j] + 8.f;
                }
            if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
                for (int nr = 0; nr < NR; ++nr)
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        float x = mx[nr][j];
#pragma unroll
                        for (int d = 4; d < 32; d <<= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, d));
                        const float mn = fmaxf(m[nr][j], x);
                        const float f = m[nr][j] == mn ? 1.f : ex2(m[nr][j] - mn);
                        m[nr][j] = mn;
                        l[nr][j] *= f;
#pragma unroll
                        for (int mt = 0; mt < KS; ++mt) {
                            o[nr][mt][j] *= f;
                            o[nr][mt][j + 2] *= f;
                        }
                    }
            }
            uint32_t pf[NR][2];
#pragma unroll
            for (int nr = 0; nr < NR; ++nr) {
                const float r0 = m[nr][0] == -INFINITY ? 0.f : m[nr][0], r1 = m[nr][1] == -INFINITY ? 0.f : m[nr][1];
                const float e0 = ex2(fmaf(sc[nr][0], c2, -r0)), e1 = ex2(fmaf(sc[nr][1], c2, -r1));
                const float e2 = ex2(fmaf(sc[nr][2], c2, -r0)), e3 = ex2(fmaf(sc[nr][3], c2, -r1));
                l[nr][0] += e0 + e2;
                l[nr][1] += e1 + e3;
                pf[nr][0] = movmatrix_t(pack_bf16(e0, e1));
                pf[nr][1] = movmatrix_t(pack_bf16(e2, e3));
            }
            {
                const int key = (lane >> 4) * 8 + (lane & 7), sw = (key >> 1) & 3, hi = (lane >> 3) & 1;
#pragma unroll
                for (int mt = 0; mt < KS; ++mt) {
                    uint32_t a0, a1, a2, a3;
                    ldsm_x4_t(va + (mt >> 1) * 1024 + key * 64 + ((((mt & 1) * 2 + hi) ^ sw) << 4), a0, a1, a2, a3);
#pragma unroll
                    for (int nr = 0; nr < NR; ++nr) mma_16816(o[nr][mt], a0, a1, a2, a3, pf[nr][0], pf[nr][1]);
                }
            }
            __syncwarp();
            issue();
        }
        // ---------------------------------------------------------------- the item's end
#pragma unroll
        for (int nr = 0; nr < NR; ++nr)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
#pragma unroll
                for (int d = 4; d < 32; d <<= 1) l[nr][j] += __shfl_xor_sync(0xffffffffu, l[nr][j], d);
                if (gq == 0) s_ml[warp * 16 + nr * 8 + 2 * tq + j] = make_float2(m[nr][j], l[nr][j]);
            }
        if (lane == 0) s_bad[warp] = bad;
        const bool whole = paged_whole(s);
        const int slot = s.ta > 0 ? 0 : 1;
        if (threadIdx.x == 0 && !whole && s.ta > 0) {
            PagedHdr h;
            h.kind = s.tb == s.tiles.nt ? 2 : 1;
            h.row0 = s.r + s.t0;
            h.ntok = s.ntok;
            h.head = s.head;
            h.c0 = s.c0;
            a.hdr[blockIdx.x] = h;
        }
        float* part = paged_slot(a, blockIdx.x, slot);
        const int rr = threadIdx.x / 16, cc = threadIdx.x % 16;  // row of 8, pair of channels
#pragma unroll
        for (int nr = 0; nr < NR; ++nr) {
            if (nr * 8 >= rows) break;
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                __syncthreads();
#pragma unroll
                for (int mt = 0; mt < KS / 2; ++mt) {
                    const float* x = o[nr][half * (KS / 2) + mt];
                    float* p = buf + (warp * 8 + 2 * tq) * L::PITCH + mt * 16 + gq;
                    p[0] = x[0];
                    p[L::PITCH] = x[1];
                    p[8] = x[2];
                    p[L::PITCH + 8] = x[3];
                }
                __syncthreads();
                const int row = nr * 8 + rr;
                if (row >= rows) continue;
                float mw = -INFINITY, lw = 0.f, f[kWarps];
#pragma unroll
                for (int w = 0; w < kWarps; ++w) mw = fmaxf(mw, s_ml[w * 16 + row].x);
#pragma unroll
                for (int w = 0; w < kWarps; ++w) {
                    const float2 x = s_ml[w * 16 + row];
                    f[w] = x.x == mw ? 1.f : ex2(x.x - mw);
                    lw += f[w] * x.y;
                }
                const int tok = row / a.G, head = s.head * a.G + row - tok * a.G;
                const int64_t orow = s.r + s.t0 + tok;
                const bool any_bad = s_bad[0] | s_bad[1] | s_bad[2] | s_bad[3];
                if (half == 0 && cc == 0) {
                    if (!whole) {
                        part[row] = mw;
                        part[a.slot_rows + row] = lw;
                    } else if (a.lse) {
                        a.lse[orow * a.H + head] = (mw + log2f(lw)) * 0.693147180559945309f;
                    }
                }
                const float inv = whole ? 1.f / lw : 1.f;
                for (int p = cc; p < L::HC / 2; p += 16) {
                    float v[2] = {0.f, 0.f};
#pragma unroll
                    for (int w = 0; w < kWarps; ++w) {
                        const float2 x = *reinterpret_cast<const float2*>(buf + (w * 8 + rr) * L::PITCH + 2 * p);
                        v[0] += f[w] * x.x;
                        v[1] += f[w] * x.y;
                    }
                    const int c = half * L::HC + 2 * p;
                    if (any_bad) {
                        v[0] += paged_nonfinite<kKT>(a, s, s.c + s.t0 + tok, c);
                        v[1] += paged_nonfinite<kKT>(a, s, s.c + s.t0 + tok, c + 1);
                    }
                    if (whole)
                        *reinterpret_cast<uint32_t*>(a.o + (orow * a.o_rs + (int64_t)head * D + c) * 2) =
                            pack_bf16(v[0] * inv, v[1] * inv);
                    else
                        *reinterpret_cast<float2*>(part + 2 * a.slot_rows + row * D + c) = make_float2(v[0], v[1]);
                }
            }
        }
        __syncthreads();
    }
    // Copies still in flight land before the CTA's shared memory goes away (only after a
    // wait gave up; otherwise every block was used).
    volatile int no_abort = 0;
    for (int i = used; i < issued; ++i) mbar_wait(full + i % NS, (i / NS) & 1, &no_abort, a.err);
    grid_launch_dependents();
}

template <int D, int NR, int NS>
cudaError_t launch(const DecodeMaps& tm, const PagedArgs& a, int grid, cudaStream_t st) {
    static PerDeviceOnce once;
    constexpr int smem = Lay<D, NS>::TOTAL + 512;
    cudaError_t e = per_device_once(once, [] {
        return cudaFuncSetAttribute(paged_decode_kernel<D, NR, NS>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    });
    if (e != cudaSuccess) return e;
    paged_decode_kernel<D, NR, NS><<<grid, kThreads, smem, st>>>(tm, a);
    ripe_count_launch();
    return cudaGetLastError();
}

template <int NR>
cudaError_t launch_d(const DecodeMaps& tm, const PagedArgs& a, int grid, cudaStream_t st) {
    if (a.d == 32) return launch<32, NR, 8>(tm, a, grid, st);
    if (a.d == 64) return launch<64, NR, 6>(tm, a, grid, st);
    if (a.d == 96) return launch<96, NR, 4>(tm, a, grid, st);
    if (a.d == 128) return launch<128, NR, 3>(tm, a, grid, st);
    return cudaErrorInvalidValue;
}

}  // namespace

cudaError_t launch_paged_decode(PagedArgs a, int grid, cudaStream_t st) {
    DecodeMaps tm;
    if (!paged_kv_map(&tm.k, a.k, a, 16, a.d / 32) || !paged_kv_map(&tm.v, a.v, a, 16, a.d / 32)) return cudaErrorInvalidValue;
    return a.slot_rows <= 8 ? launch_d<1>(tm, a, grid, st) : launch_d<2>(tm, a, grid, st);
}
