// ripe_paged.cu -- the paged cache beside the tensor-core attention kernels: the write
// of new tokens (ripe_paged_append), the attention of chunks in 32 bits or at head sizes
// the tensor-core kernels have no form for, and the kernel that joins cut items.
#include <math.h>

#include <type_traits>

#include "ripe_launch.h"
#include "ripe_paged.cuh"
#include "ripe_paged_launch.h"
#include "sm100_ptx.cuh"

using namespace sm100;

namespace {

__device__ int32_t g_error_word;

// ------------------------------------------------------------------ append
// Row r of K and V goes to slot pos % page of page table[seq][pos / page], pos = ctx +
// r - row0[seq].  A copy: bound by HBM (read once, written once).  One block per row and
// share of its 16-byte vectors; the row's sequence comes from a 32-way search of row0
// (two rounds of loads by one warp; 1024 sequences at most), beside which the other warps
// check that the offsets ascend, as the search takes them to.  Three prompts of 1500 to 4000
// tokens, 55 heads of size 96: 46 us for 247 MB, 5.4 TB/s (a plain copy reaches 6.55); 64
// ragged draft blocks: 3.3 us, a launch and three dependent loads.
constexpr int kAppendThreads = 128, kAppendVecs = 4;

__global__ void __launch_bounds__(kAppendThreads) paged_append_kernel(const __grid_constant__ PagedArgs a,
                                                                      const char* __restrict__ K,
                                                                      const char* __restrict__ V, int64_t row_stride,
                                                                      int esize) {
    const int64_t row = blockIdx.x;
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    __shared__ int64_t s_off;  // elements from the pages' base to the token's head 0, or -1
    __shared__ int s_fall[kAppendThreads / 32 - 1];
    // Where the row goes, by the last of the first n sequences with row0 <= row (warp 0).
    auto place = [&](int n) {
        const int per = (n + 31) / 32, i = min(lane * per, n);
        const unsigned c = __ballot_sync(0xffffffffu, i < n && __ldg(a.row0 + i) <= row);
        const int lo = c ? (31 - __clz(c)) * per : 0;
        const int j = lo + lane;
        const unsigned f = __ballot_sync(0xffffffffu, lane < per && j < n && __ldg(a.row0 + j) <= row);
        const int seq = f ? lo + 31 - __clz(f) : -1;
        if (lane != 0) return;
        int64_t off = -1;
        if (seq >= 0) {
            const PagedSeq q = paged_seq(a, seq);
            if (row - q.r < q.n) {
                const int64_t pos = q.c + (row - q.r);
                const int id = __ldg(a.table + seq * a.table_stride + (pos >> a.page_shift));
                off = (unsigned)id < (unsigned)a.npages ? id * a.page_stride + (pos & (a.page - 1)) * a.pos_stride : -2;
            }
        }
        s_off = off;
    };
    int bad = 0, code = 0;
    if (warp == 0) {
        place(a.nseq);
    } else {
        // The other warps look for offsets that descend, and at the block's share of all
        // sequences: a bad one may own no row that a block would find it by.
        constexpr int kOthers = kAppendThreads - 32, kAhead = 4;
        const int t = threadIdx.x - 32;
        int fall = a.nseq;
        for (int i0 = t; i0 < a.nseq; i0 += kOthers * kAhead) {
            int lo[kAhead], hi[kAhead];
#pragma unroll
            for (int j = 0; j < kAhead; ++j) {
                const int i = min(i0 + j * kOthers, a.nseq - 1);
                lo[j] = __ldg(a.row0 + i);
                hi[j] = __ldg(a.row0 + i + 1);
            }
#pragma unroll
            for (int j = 0; j < kAhead; ++j)
                if (hi[j] < lo[j]) fall = min(fall, min(i0 + j * kOthers, a.nseq - 1));
        }
        if (blockIdx.y == 0)
            for (int64_t i = blockIdx.x + (int64_t)gridDim.x * t; i < a.nseq && code == 0; i += (int64_t)gridDim.x * kOthers) {
                bad = (int)i;
                code = paged_seq(a, bad).code;
            }
        fall = __reduce_min_sync(0xffffffffu, fall);
        if (lane == 0) s_fall[warp - 1] = fall;
    }
    __syncthreads();
    int fall = s_fall[0];
    for (int i = 1; i < kAppendThreads / 32 - 1; ++i) fall = min(fall, s_fall[i]);
    if (code && bad <= fall) set_device_error(a.err, code);
    if (fall < a.nseq) {  // the sequences from there on are skipped
        if (warp == 0) place(fall);
        __syncthreads();
    }
    const int64_t off = s_off;
    if (off < 0) {
        if (off == -2 && threadIdx.x == 0) set_device_error(a.err, RIPE_DEVERR_PAGE);
        return;
    }
    const int per_head = a.d * esize / 16, total = a.Hkv * per_head;
    const uint4* src[2] = {reinterpret_cast<const uint4*>(K + row * row_stride * esize),
                           reinterpret_cast<const uint4*>(V + row * row_stride * esize)};
    char* dst[2] = {const_cast<char*>(a.k) + off * esize, const_cast<char*>(a.v) + off * esize};
    uint4 x[2][kAppendVecs];
    const int i0 = blockIdx.y * kAppendThreads * kAppendVecs + threadIdx.x;
#pragma unroll
    for (int kv = 0; kv < 2; ++kv)
#pragma unroll
        for (int j = 0; j < kAppendVecs; ++j) {
            const int i = i0 + j * kAppendThreads;
            if (i < total) x[kv][j] = __ldcs(src[kv] + i);
        }
#pragma unroll
    for (int j = 0; j < kAppendVecs; ++j) {
        const int i = i0 + j * kAppendThreads;
        if (i >= total) break;
        const int h = i / per_head;
        const int64_t at = h * a.head_stride * esize + (int64_t)(i - h * per_head) * 16;
        *reinterpret_cast<uint4*>(dst[0] + at) = x[0][j];
        *reinterpret_cast<uint4*>(dst[1] + at) = x[1][j];
    }
}

// ------------------------------------------------------------------ attention on CUDA cores
// Items of 16 rows (tokens x heads of the group), 32 keys at a time, double-buffered in
// shared memory by cp.async as they lie in the cache; fp32 arithmetic (FFMA).  Eight
// lanes share a row: four of the 32 scores each, then d/8 channels of O each.  Bound by the
// latency of shared memory at few warps (0.5 to 0.9 instructions a cycle and SM), so as many
// CTAs as fit: 55 single tokens behind 1900 to 3200, 64 heads over 32 of size 80, bf16: 1.97
// ms (two CTAs an SM 4.04; 1.4 GB, 0.72 TB/s).  4 tokens behind 48, two heads of size 16: 10 us.
constexpr int kSimtThreads = 128, kRows = 16, kKT = 32;
constexpr int kSimtMinCost = 1;  // key tiles a CTA takes at least (2: 26 short sequences 27 us, 1: 17)

template <typename Elem>
__device__ __forceinline__ float4 load4(const char* p);
template <>
__device__ __forceinline__ float4 load4<float>(const char* p) {
    return *reinterpret_cast<const float4*>(p);
}
template <>
__device__ __forceinline__ float4 load4<__nv_bfloat16>(const char* p) {
    const uint2 x = *reinterpret_cast<const uint2*>(p);
    return make_float4(__uint_as_float(x.x << 16), __uint_as_float(x.x & 0xFFFF0000u), __uint_as_float(x.y << 16),
                       __uint_as_float(x.y & 0xFFFF0000u));
}

// Shared-memory row pitch: 16 bytes more than the row, so that eight rows' vectors at one
// channel fall into different banks.
__host__ __device__ inline int simt_pitch(int d, int esize) { return d * esize + 16; }

template <typename Elem>
__global__ void __launch_bounds__(kSimtThreads) paged_simt_kernel(const __grid_constant__ PagedArgs a) {
    constexpr int ES = sizeof(Elem);
    extern __shared__ __align__(16) char smem[];
    __shared__ float s_p[kRows][kKT + 1];
    __shared__ PagedPlanHead s_plan;
    const int pitch = simt_pitch(a.d, ES), tile = kKT * pitch;
    char* sQ = smem;                 // [16] rows
    char* sKV = smem + kRows * pitch;  // [2 buffers][K, V][32] rows
    const int tid = threadIdx.x, row = tid / 8, sub = tid % 8;
    const int nv = a.d * ES / 16, n4 = a.d / 4;

    if (tid == 0) a.hdr[blockIdx.x].kind = 0;
    PagedPlan<kKT> plan;
    plan.template begin<kSimtThreads>(a, s_plan, *reinterpret_cast<PagedPlanSmem*>(smem), kSimtMinCost);
    PagedSeg s;
    while (plan.next(a, s)) {
        const int p0 = s.c + s.t0, p1 = p0 + s.ntok - 1, rows = s.ntok * a.G;
        const int tok = row / a.G, pos = p0 + tok;
        const bool valid = row < rows;
        const bool live = tid / 32 * 4 < rows;  // the warp has rows; a single token leaves three idle
        __syncthreads();  // the previous item's tiles and Q are no longer read
        for (int i = tid; i < kRows * nv; i += kSimtThreads) {
            const int r = i / nv, v = i - r * nv, tk = r / a.G;
            const bool on = r < rows;
            cp_async16_zfill(sQ + r * pitch + v * 16,
                             a.q + (on ? ((s.r + s.t0 + tk) * a.q_rs + (int64_t)(s.head * a.G + r - tk * a.G) * a.d) * ES + v * 16
                                       : 0),
                             on);
        }
        // Four threads a key; its page is looked up a tile ahead of its copies.
        const int lr = tid / 4, lv = tid % 4;
        const int gone_to = a.window > 0 ? p0 - a.window : -1;
        // Later slots hold anything, and behind the window the page may be gone: read as zeros.
        auto needed = [&](int key) { return key <= p1 && (key > gone_to || key < a.sinks); };
        auto entry = [&](int t) {
            const int key = s.tiles.tile(t) * kKT + lr;
            return t < s.tb && needed(key) ? paged_entry(a, s.seq, key) : 0;
        };
        int ent = entry(s.ta);
        auto load = [&](int t, int b) {
            const int key = s.tiles.tile(t) * kKT + lr;
            const bool on = needed(key);
            const int64_t off = on ? (paged_checked(a, ent) * a.page_stride + s.head * a.head_stride +
                                      (key & (a.page - 1)) * a.pos_stride) * ES
                                   : 0;
            ent = entry(t + 1);
            char* dk = sKV + b * 2 * tile + lr * pitch;
            for (int v = lv; v < nv; v += 4) {
                cp_async16_zfill(dk + v * 16, a.k + off + (on ? v * 16 : 0), on);
                cp_async16_zfill(dk + tile + v * 16, a.v + off + (on ? v * 16 : 0), on);
            }
            cp_async_commit();
        };
        float m = -INFINITY, l = 0.f;
        float4 o[4];  // channels 4 (sub + 8 j)
#pragma unroll
        for (int j = 0; j < 4; ++j) o[j] = make_float4(0.f, 0.f, 0.f, 0.f);
        load(s.ta, 0);
        for (int t = s.ta; t < s.tb; ++t) {
            const int b = (t - s.ta) & 1, k0 = s.tiles.tile(t) * kKT;
            if (t + 1 < s.tb) {
                load(t + 1, b ^ 1);
                cp_async_wait_group<1>();
            } else {
                cp_async_wait_group<0>();
            }
            __syncthreads();
            const char* K = sKV + b * 2 * tile;
            const char* V = K + tile;
            if (live) {
                const bool part = !paged_all_seen(a, k0, kKT, p0, p1);
                float sc[4] = {0.f, 0.f, 0.f, 0.f};
                for (int i = 0; i < n4; ++i) {
                    const float4 q = load4<Elem>(sQ + row * pitch + i * 4 * ES);
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const float4 k = load4<Elem>(K + (sub + 8 * j) * pitch + i * 4 * ES);
                        sc[j] = fmaf(q.x, k.x, fmaf(q.y, k.y, fmaf(q.z, k.z, fmaf(q.w, k.w, sc[j]))));
                    }
                }
                float mx = -INFINITY;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    sc[j] = part && !paged_seen(a, k0 + sub + 8 * j, pos) ? -INFINITY : sc[j] * a.scale_log2;
                    mx = fmaxf(mx, sc[j]);
                }
#pragma unroll
                for (int d = 1; d < 8; d <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, d));
                const float mn = fmaxf(m, mx), f = m == mn ? 1.f : exp2f(m - mn), ref = mn == -INFINITY ? 0.f : mn;
                m = mn;
                l *= f;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    o[j].x *= f;
                    o[j].y *= f;
                    o[j].z *= f;
                    o[j].w *= f;
                    const float e = exp2f(sc[j] - ref);
                    l += e;
                    s_p[row][sub + 8 * j] = e;
                }
                // Hidden keys get -0, so that the second product can leave them out: a weight that is 0
                // because it is small still meets its value, as the formula has it.
                if (part) {
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        if (!paged_seen(a, k0 + sub + 8 * j, pos)) s_p[row][sub + 8 * j] = -0.f;
                }
                __syncwarp();  // a row's eight lanes sit in one warp
                auto add = [&](int key, auto partial) {
                    const float p = s_p[row][key];
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        if (sub + 8 * j < n4) {
                            const float4 v = load4<Elem>(V + key * pitch + (sub + 8 * j) * 4 * ES);
                            // a hidden key's value may be anything: it must not meet the zero weight
                            const bool skip = partial.value && __float_as_uint(p) == 0x80000000u;
                            o[j].x = skip ? o[j].x : fmaf(p, v.x, o[j].x);
                            o[j].y = skip ? o[j].y : fmaf(p, v.y, o[j].y);
                            o[j].z = skip ? o[j].z : fmaf(p, v.z, o[j].z);
                            o[j].w = skip ? o[j].w : fmaf(p, v.w, o[j].w);
                        }
                    }
                };
                if (part) {
#pragma unroll 8
                    for (int key = 0; key < kKT; ++key) add(key, std::true_type());
                } else {
#pragma unroll 8
                    for (int key = 0; key < kKT; ++key) add(key, std::false_type());
                }
            }
            __syncthreads();  // before the next load into this buffer
        }
#pragma unroll
        for (int d = 1; d < 8; d <<= 1) l += __shfl_xor_sync(0xffffffffu, l, d);
        const bool whole = paged_whole(s);
        if (tid == 0 && !whole && s.ta > 0) {
            PagedHdr h;
            h.kind = s.tb == s.tiles.nt ? 2 : 1;
            h.row0 = s.r + s.t0;
            h.ntok = s.ntok;
            h.head = s.head;
            h.c0 = s.c0;
            a.hdr[blockIdx.x] = h;
        }
        if (!valid) continue;
        const int64_t orow = s.r + s.t0 + tok;
        const int head = s.head * a.G + row - tok * a.G;
        float* part = paged_slot(a, blockIdx.x, s.ta > 0 ? 0 : 1);
        if (sub == 0) {
            if (!whole) {
                part[row] = m;
                part[a.slot_rows + row] = l;
            } else if (a.lse) {
                a.lse[orow * a.H + head] = m * 0.693147180559945309f + logf(l);
            }
        }
        const float inv = whole ? 1.f / l : 1.f;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            if (sub + 8 * j >= n4) break;
            const int c = 4 * (sub + 8 * j);
            if (!whole) {
                float2* dst = reinterpret_cast<float2*>(part + 2 * a.slot_rows + row * a.d + c);
                dst[0] = make_float2(o[j].x, o[j].y);
                dst[1] = make_float2(o[j].z, o[j].w);
            } else if constexpr (ES == 4) {
                *reinterpret_cast<float4*>(a.o + (orow * a.o_rs + (int64_t)head * a.d + c) * 4) =
                    make_float4(o[j].x * inv, o[j].y * inv, o[j].z * inv, o[j].w * inv);
            } else {
                *reinterpret_cast<uint2*>(a.o + (orow * a.o_rs + (int64_t)head * a.d + c) * 2) =
                    make_uint2(pack_bf16(o[j].x * inv, o[j].y * inv), pack_bf16(o[j].z * inv, o[j].w * inv));
            }
        }
    }
    grid_launch_dependents();
}

// ------------------------------------------------------------------ merge
// One block column per CTA of the attention kernel; a CTA that ended an item it did not
// begin joins that item's partials, from the CTA that began it (its slot B) over the ones
// in the middle to itself (slot A):
//   m = max m_k, l = sum 2^(m_k - m) l_k, O = sum 2^(m_k - m) O_k / l.
// A warp per row: lane k holds partial k's m and l (32 at a time), then the lanes take
// channel pairs and the partials' loads go out together.  Bound by latency, three rounds
// of L2 (the partials were written just before).
constexpr int kMergeWarps = 4, kMergeThreads = 32 * kMergeWarps;

template <typename Elem>
__global__ void __launch_bounds__(kMergeThreads) paged_merge_kernel(const __grid_constant__ PagedArgs a) {
    grid_dependency_wait();
    const int c1 = blockIdx.x;
    const PagedHdr h = a.hdr[c1];
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int row = blockIdx.y * kMergeWarps + warp;  // the item's
    if (h.kind != 2 || row >= h.ntok * a.G) return;
    const int64_t stride = 2 * (int64_t)a.slot_rows * (a.d + 2);
    // partial k: slot B of CTA c0, then slot A of c0 + 1 ... c1
    const float* first = paged_slot(a, h.c0, 1);
    const float* rest = paged_slot(a, h.c0, 0);
    const int n = c1 - h.c0 + 1, np = a.d / 2;
    float m = -INFINITY, l = 0.f, o[4] = {0.f, 0.f, 0.f, 0.f};
    for (int k0 = 0; k0 < n; k0 += 32) {
        const int k = k0 + lane;
        float mk = -INFINITY, lk = 0.f;
        if (k < n) {
            const float* p = k == 0 ? first : rest + k * stride;
            mk = p[row];
            lk = p[a.slot_rows + row];
        }
        float mn = mk;
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) mn = fmaxf(mn, __shfl_xor_sync(0xffffffffu, mn, d));
        mn = fmaxf(mn, m);
        const float f = m == mn ? 1.f : exp2f(m - mn), fk = mk == mn ? 1.f : exp2f(mk - mn);
        m = mn;
        l *= f;
        float ls = fk * lk;
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) ls += __shfl_xor_sync(0xffffffffu, ls, d);
        l += ls;
#pragma unroll
        for (int j = 0; j < 4; ++j) o[j] *= f;
        const int kn = min(32, n - k0);
#pragma unroll 4
        for (int q = 0; q < kn; ++q) {
            const float* p = k0 + q == 0 ? first : rest + (k0 + q) * stride;
            const float w = __shfl_sync(0xffffffffu, fk, q);
            const float2* v = reinterpret_cast<const float2*>(p + 2 * a.slot_rows + (int64_t)row * a.d);
#pragma unroll
            for (int j = 0; j < 2; ++j)
                if (lane + 32 * j < np) {
                    const float2 x = v[lane + 32 * j];
                    o[2 * j] += w * x.x;
                    o[2 * j + 1] += w * x.y;
                }
        }
    }
    const int tok = row / a.G, head = h.head * a.G + row - tok * a.G;
    const int64_t orow = h.row0 + tok;
    if (lane == 0 && a.lse) a.lse[orow * a.H + head] = m * 0.693147180559945309f + logf(l);
    const float inv = 1.f / l;
#pragma unroll
    for (int j = 0; j < 2; ++j)
        if (lane + 32 * j < np) {
            char* dst = a.o + (orow * a.o_rs + (int64_t)head * a.d + 2 * (lane + 32 * j)) * sizeof(Elem);
            if constexpr (sizeof(Elem) == 4)
                *reinterpret_cast<float2*>(dst) = make_float2(o[2 * j] * inv, o[2 * j + 1] * inv);
            else
                *reinterpret_cast<uint32_t*>(dst) = pack_bf16(o[2 * j] * inv, o[2 * j + 1] * inv);
        }
}

template <typename Elem>
cudaError_t simt_t(const PagedArgs& a, int grid, cudaStream_t st) {
    static PerDeviceOnce once;
    const int smem = (kRows + 4 * kKT) * simt_pitch(a.d, sizeof(Elem));
    cudaError_t e = per_device_once(once, [] {
        return cudaFuncSetAttribute(paged_simt_kernel<Elem>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                    (kRows + 4 * kKT) * simt_pitch(128, sizeof(Elem)));
    });
    if (e != cudaSuccess) return e;
    // the plan's arrays share the tiles' memory
    paged_simt_kernel<Elem><<<grid, kSimtThreads, smem > (int)sizeof(PagedPlanSmem) ? smem : (int)sizeof(PagedPlanSmem), st>>>(a);
    ripe_count_launch();
    return cudaGetLastError();
}

}  // namespace

cudaError_t paged_error_word(int32_t** word) {
    static PerDeviceOnce once;
    static int32_t* words[64];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    e = per_device_once(once, [dev] {
        void* p = nullptr;
        const cudaError_t found = cudaGetSymbolAddress(&p, g_error_word);
        words[dev & 63] = (int32_t*)p;
        return found;
    });
    *word = words[dev & 63];
    return e;
}

cudaError_t launch_paged_simt(PagedArgs a, int dtype, int grid, cudaStream_t st) {
    return dtype == RIPE_F32 ? simt_t<float>(a, grid, st) : simt_t<__nv_bfloat16>(a, grid, st);
}

cudaError_t launch_paged_merge(const PagedArgs& a, int dtype, int grid, cudaStream_t st) {
    const int most = a.tpt < a.max_ntok ? a.tpt : a.max_ntok;
    const int y = (most * a.G + kMergeWarps - 1) / kMergeWarps;
    const dim3 g((unsigned)grid, (unsigned)y);
    return dtype == RIPE_F32 ? launch_paged_dependent(paged_merge_kernel<float>, g, kMergeThreads, st, a)
                             : launch_paged_dependent(paged_merge_kernel<__nv_bfloat16>, g, kMergeThreads, st, a);
}

cudaError_t launch_paged_append(const PagedArgs& a, const char* K, const char* V, int64_t row_stride, int esize,
                                cudaStream_t st) {
    const int vecs = a.Hkv * a.d * esize / 16, per = kAppendThreads * kAppendVecs;
    paged_append_kernel<<<dim3((unsigned)a.nrows, (unsigned)((vecs + per - 1) / per)), kAppendThreads, 0, st>>>(
        a, K, V, row_stride, esize);
    ripe_count_launch();
    return cudaGetLastError();
}
