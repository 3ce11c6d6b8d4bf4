// ripe_paged.cuh -- argument block and device-side work plan shared by the kernels
// of ripe_paged_attn (attention of chunks of new tokens over a paged cache).
//
// Work.  The new tokens of a sequence are cut into row tiles of `tpt` tokens; a row
// tile and one key/value head are an item, whose rows are (token, query head of the
// group).  An item's keys are cut into tiles of KT; those no row can see (past the
// last token, or behind the window and past the first `sinks` tokens) are left out.
// An item costs its key tiles times its M tiles.  All items of the call, in the
// order (sequence, head, row tile), form one line of that cost, and each CTA takes an
// equal stretch of it, whatever the mix of lengths: the lengths are on the device
// only, so each CTA finds its own stretch from ctx_len and row0 (block-wide scans,
// about 2.5 us).  An item inside one stretch is finished by its CTA; one that
// is cut leaves partials (m, l, unnormalised O) for paged_merge_kernel, at most two
// per CTA: the item its stretch begins inside (slot A), and the one it ends inside
// (slot B).  The order of the merge follows the CTA numbers, so results repeat bit
// for bit.
#pragma once

#include <stdint.h>

#include "ripe_internal.cuh"

constexpr int kPagedMaxSeqs = 1024;

// What a CTA left in its slot A: 0 nothing, 1 a middle stretch of an item, 2 the end
// of an item (then the item follows).
struct PagedHdr {
    int kind, row0, ntok, head, c0;  // c0: the CTA that began the item
    int gaps;                        // CTAs between may have left nothing (kind 0)
    int pad[2];
};

struct PagedArgs {
    const char *q, *k, *v;
    char* o;
    float* lse;
    int64_t q_rs, o_rs;                           // elements between tokens' rows
    int64_t page_stride, head_stride, pos_stride;  // elements
    const int32_t *table, *ctx, *row0;
    int64_t table_stride;
    int table_width, nseq, nrows, H, Hkv, G, d, page, page_shift, npages;
    int window, sinks;  // window 0: none
    int max_ntok;       // longer sequences are skipped
    int tok1, tpt;      // tokens of one M tile and of one row tile (1 or 2 M tiles)
    float scale_log2;
    float* part;        // [CTA][2] slots of slot_rows x (d + 2) floats
    PagedHdr* hdr;      // [CTA]
    int slot_rows;
    int32_t* err;       // never NULL
};

// The chunk of sequence i: `n` tokens behind `c` cached ones, rows from `r`.  n = 0
// for a sequence that is skipped (bad offsets, or past its pages), code says why.  falls:
// its offsets descend; then those behind it are skipped too, so that no row belongs to two,
// and what code says of them means nothing.
struct PagedSeq {
    int c, n, r, code;
    bool falls;
};

__device__ __forceinline__ PagedSeq paged_seq(const PagedArgs& a, int i) {
    PagedSeq s;
    s.r = __ldg(a.row0 + i);
    s.c = __ldg(a.ctx + i);
    const int e = __ldg(a.row0 + i + 1);
    s.n = s.code = 0;
    s.falls = e < s.r;
    if (s.r < 0 || e < s.r || e > a.nrows || e - s.r > a.max_ntok) {
        s.code = RIPE_DEVERR_ROWS;
    } else if (e > s.r && (s.c < 0 || (int64_t)s.c + (e - s.r) > (int64_t)a.table_width * a.page)) {
        s.code = RIPE_DEVERR_CAPACITY;
    } else {
        s.n = e - s.r;
    }
    return s;
}

// Key tiles of tokens [t0, t0 + nt) of a chunk: tiles [0, ts) hold the first tokens,
// then tiles from `tlo` on (the same line where the two meet).
struct PagedTiles {
    int nt, ts, tlo;
    __device__ __forceinline__ int tile(int t) const { return t < ts ? t : t - ts + tlo; }
};

template <int KT>
__device__ __forceinline__ PagedTiles paged_tiles(const PagedArgs& a, int c, int t0, int ntok) {
    PagedTiles p;
    const int p0 = c + t0, hi = p0 + ntok;
    p.nt = (hi + KT - 1) / KT;
    p.ts = 0;
    p.tlo = 0;
    if (a.window > 0 && a.window <= p0) {
        const int lo = (p0 + 1 - a.window) / KT, ts = (min(a.sinks, hi) + KT - 1) / KT;
        if (ts < lo) {
            p.nt += ts - lo;
            p.ts = ts;
            p.tlo = lo;
        }
    }
    return p;
}

// Every key of [k0, k0 + nk) is seen by every token of positions [p0, p1].
__device__ __forceinline__ bool paged_all_seen(const PagedArgs& a, int k0, int nk, int p0, int p1) {
    return k0 + nk - 1 <= p0 && (a.window <= 0 || k0 > p1 - a.window || k0 + nk <= a.sinks);
}
// Some key of [k0, k0 + nk) may be seen by some token of positions [p0, p1].
__device__ __forceinline__ bool paged_any_seen(const PagedArgs& a, int k0, int nk, int p0, int p1) {
    return k0 <= p1 && (a.window <= 0 || k0 + nk - 1 > p0 - a.window || k0 < a.sinks);
}
__device__ __forceinline__ bool paged_seen(const PagedArgs& a, int key, int pos) {
    return key <= pos && (a.window <= 0 || key > pos - a.window || key < a.sinks);
}

// The table's entry for key `key` of sequence `seq`, to be passed through paged_checked
// before use (apart, so that a load far ahead of its use waits for nothing).
__device__ __forceinline__ int paged_entry(const PagedArgs& a, int seq, int key) {
    return __ldg(a.table + seq * a.table_stride + (key >> a.page_shift));
}
// An id outside the pool is reported and read as page 0 (that sequence's rows then mean
// nothing).
__device__ __forceinline__ int paged_checked(const PagedArgs& a, int id) {
    if ((unsigned)id >= (unsigned)a.npages) {
        set_device_error(a.err, RIPE_DEVERR_PAGE);
        id = 0;
    }
    return id;
}
__device__ __forceinline__ int paged_page(const PagedArgs& a, int seq, int key) {
    return paged_checked(a, paged_entry(a, seq, key));
}

// A stretch of one item: key tiles [ta, tb) of its `nt`.
struct PagedSeg {
    int seq, c, r, n;       // the sequence (PagedSeq)
    int t0, ntok, head, w;  // the row tile's tokens, the key/value head, M tiles
    int ta, tb;
    int c0, gaps;           // the CTA that began the item, for a stretch that does not (PagedHdr)
    PagedTiles tiles;
};

// What the plan needs of shared memory: a little of its own, and arrays for calls with many
// row tiles, which may lie where copies land later.
struct PagedPlanHead {
    int64_t warp[32];
    PagedSeg s;  // where the CTA's stretch begins, as one thread finds it
    int qt, off;
    int fall;               // the first sequence whose offsets descend
};
struct PagedPlanSmem {
    int64_t cp[kPagedMaxSeqs + 1];  // one head's cost before each sequence
    int64_t tp[1024 + 1];           // one head's cost before each thread's run of row tiles
    int sq[kPagedMaxSeqs + 1];      // row tiles before each sequence
};

// Inclusive block-wide scan of one value per thread (all threads call it; one barrier).
// *flag, if given, becomes whether it was set in any thread.
template <int THREADS, typename T>
__device__ __forceinline__ T paged_scan(T v, T* warp_sums, T& total, bool* flag = nullptr) {
    const int lane = threadIdx.x % 32, w = threadIdx.x / 32;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const T y = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o) v += y;
    }
    if (lane == 31) warp_sums[w] = v;
    if (flag) *flag = __syncthreads_or(*flag);
    else __syncthreads();
    total = 0;
#pragma unroll
    for (int i = 0; i < THREADS / 32; ++i) {
        if (i < w) v += warp_sums[i];
        total += warp_sums[i];
    }
    return v;
}

// a / b for a >= 0, b > 0: the 32-bit division where it fits (most calls), a fraction of
// the other's cost.
__device__ __forceinline__ int64_t paged_div(int64_t a, int64_t b) {
    return ((a | b) >> 31) == 0 ? (int64_t)((uint32_t)a / (uint32_t)b) : a / b;
}

template <int KT>
struct PagedPlan {
    int64_t x, x_end;  // this CTA's stretch of the line (x moves)
    int64_t stretch;   // its length, before the line's end cuts it
    int nseq;          // sequences before the first whose offsets descend (while the plan is made)
    int qt;            // row tile within the sequence
    int off;           // cost already behind x within the item
    int cut;           // an item is cut at multiples of 2^cut key tiles
    PagedSeg s;        // the current item (s.head included)

    __device__ __forceinline__ int item(const PagedArgs& a) {  // s.seq, qt -> the row tile; its cost
        s.t0 = qt * a.tpt;
        s.ntok = min(a.tpt, s.n - s.t0);
        s.w = s.ntok > a.tok1 ? 2 : 1;
        s.tiles = paged_tiles<KT>(a, s.c, s.t0, s.ntok);
        return s.tiles.nt * s.w;
    }
    __device__ __forceinline__ void load(const PagedArgs& a, int i) {
        const PagedSeq q = paged_seq(a, i);
        s.seq = i;
        s.c = q.c;
        s.n = q.n;
        s.r = q.r;
    }

    // A stretch shorter than min_cost is not worth its partials, so the CTAs take min_cost
    // each, and not all work; or, with `pieces` and less than half of min_cost, items are cut
    // into pieces of 2^pieces key tiles only, each taken whole by the CTA that its last key
    // tile falls to, so that small items still spread over all CTAs.
    __device__ __forceinline__ void share(const PagedArgs& a, int64_t one_head, int min_cost, int pieces) {
        const int64_t total = one_head * a.Hkv;
        int64_t len = paged_div(total + gridDim.x - 1, gridDim.x);
        cut = 0;
        if (len < min_cost) {
            if (pieces > 0 && len * 2 < min_cost) {
                cut = pieces;
                len = len < 1 ? 1 : len;
            } else {
                len = min_cost;
            }
        }
        s.c0 = 0;
        stretch = len;
        x = len * blockIdx.x;
        x_end = x + len < total ? x + len : total;
    }
    // The head that holds x, of the current sequence (one head of it costs `c`, `before`
    // lies ahead of it); returns how far x is into that head's row tiles.
    __device__ __forceinline__ int64_t head_of(const PagedArgs& a, int64_t before, int64_t c) {
        const int64_t rem = x - before * a.Hkv;
        s.head = (int)paged_div(rem, c);
        return rem - s.head * c;
    }
    // The row tile that holds cost `y`, of those from the current one (after `p`).
    __device__ __forceinline__ void tile_of(const PagedArgs& a, int64_t p, int64_t y) {
        int c = item(a);
        while (p + c <= y) {
            p += c;
            ++qt;
            c = item(a);
        }
        off = (int)(y - p);
    }

    // The thread that found the CTA's place tells the others.
    __device__ __forceinline__ void tell(PagedPlanHead& h) {
        // The item begins where its first piece's cost ends up: a CTA that ends inside that piece
        // leaves it to the next.
        s.c0 = (int)paged_div(x - off + (min(s.tiles.nt, 1 << cut) * s.w - 1), stretch);
        s.gaps = cut > 0;
        h.s = s;
        h.qt = qt;
        h.off = off;
    }

    // All threads of the block; ends with a barrier, after which `sm` may be reused.  This
    // runs before anything else of the kernel, once and from a cold instruction cache, so the
    // usual cases have short ways of their own, few row tiles per sequence or a thread per row
    // tile (about 4500 cycles each, where the way for any number takes 9000: 38 us against 36
    // for 23 single tokens beside a chunk of 509).
    template <int THREADS>
    __device__ void begin(const PagedArgs& a, PagedPlanHead& h, PagedPlanSmem& sm, int min_cost, int pieces = 0) {
        static_assert(THREADS <= 1024, "one scan value per warp");
        const int tid = threadIdx.x;
        bool falls = false;
        if (tid == 0) h.fall = a.nseq;  // seen by the others behind a scan
        nseq = a.nseq;
        if (a.nseq <= THREADS && a.max_ntok <= 4 * a.tpt) {
            // few row tiles per sequence: a thread per sequence, one scan
            s.n = 0;
            int64_t cost = 0;
            int code = 0;
            if (tid < a.nseq) {
                const PagedSeq q = paged_seq(a, tid);
                s.seq = tid;
                s.c = q.c;
                s.n = q.n;
                s.r = q.r;
                falls = q.falls;
                code = q.code;
                for (qt = 0; qt * a.tpt < s.n; ++qt) cost += item(a);
            }
            int64_t total;
            const bool mine = falls;
            int64_t incl = paged_scan<THREADS>(cost, h.warp, total, &falls);
            if (falls) {
                if (mine) atomicMin(&h.fall, tid);
                __syncthreads();
                if (tid >= h.fall) cost = 0;
                if (tid > h.fall) code = 0;
                incl = paged_scan<THREADS>(cost, h.warp, total);
            }
            if (code && blockIdx.x == 0) set_device_error(a.err, code);
            share(a, total, min_cost, pieces);
            if (x < x_end && (incl - cost) * a.Hkv <= x && x < incl * a.Hkv) {  // one thread's sequence
                const int64_t y = head_of(a, incl - cost, cost);
                qt = 0;
                tile_of(a, 0, y);
                tell(h);
            }
        } else {
            // row tiles before each sequence
            unsigned sum = 0;  // behind a sequence whose offsets descend it may be anything
            int bad = 0, code = 0;  // this thread's first sequence with a code
            for (int i0 = 0; i0 < a.nseq; i0 += THREADS) {
                const int i = i0 + tid;
                unsigned nq = 0, add;
                falls = false;
                if (i < a.nseq) {
                    const PagedSeq q = paged_seq(a, i);
                    if (code == 0) {
                        bad = i;
                        code = q.code;
                    }
                    nq = (unsigned)((q.n + a.tpt - 1) / a.tpt);
                    falls = q.falls;
                }
                const unsigned incl = sum + paged_scan<THREADS>(nq, reinterpret_cast<unsigned*>(h.warp), add);
                if (i < a.nseq) sm.sq[i + 1] = (int)incl;
                if (falls) atomicMin(&h.fall, i);
                sum += add;
                __syncthreads();
            }
            if (tid == 0) sm.sq[0] = 0;
            __syncthreads();
            nseq = h.fall;
            if (code && bad <= nseq && blockIdx.x == 0) set_device_error(a.err, code);
            const int base = sm.sq[nseq];
            if (base <= THREADS) {
                // a thread per row tile
                int64_t cost = 0, total;
                if (tid < base) {
                    find(a, sm, tid);
                    cost = item(a);
                }
                const int64_t incl = paged_scan<THREADS>(cost, h.warp, total);
                sm.tp[tid] = incl - cost;
                if (tid == 0) sm.tp[THREADS] = total;
                __syncthreads();
                share(a, total, min_cost, pieces);
                if (x < x_end && tid < base) {
                    const int64_t before = sm.tp[sm.sq[s.seq]], one = sm.tp[sm.sq[s.seq + 1]] - before;
                    if (before * a.Hkv <= x && x < (before + one) * a.Hkv) {  // in this sequence
                        const int64_t y = head_of(a, before, one) - (incl - cost - before);
                        if (y >= 0 && y < cost) {  // one thread's row tile
                            off = (int)y;
                            tell(h);
                        }
                    }
                }
            } else {
                // cost before each thread's run of row tiles, and before each sequence
                const int per = max(1, (base + THREADS - 1) / THREADS);
                const int q0 = min(base, tid * per), q1 = min(base, q0 + per);
                int64_t cost = 0, total;
                if (q0 < q1) {
                    find(a, sm, q0);
                    for (int q = q0; q < q1; ++q) {
                        cost += item(a);
                        step(a);
                    }
                }
                const int64_t incl = paged_scan<THREADS>(cost, h.warp, total);
                sm.tp[tid] = incl - cost;
                __syncthreads();
                for (int i = tid; i <= nseq; i += THREADS) {
                    const int q = sm.sq[i], run = q / per;
                    int64_t p = q < base ? sm.tp[run] : total;
                    if (q < base) {
                        find(a, sm, run * per);
                        for (int j = run * per; j < q; ++j) {
                            p += item(a);
                            step(a);
                        }
                    }
                    sm.cp[i] = p;
                }
                __syncthreads();
                share(a, total, min_cost, pieces);
                if (x < x_end && tid == 0) {
                    int lo = 0, hi = nseq;  // the last sequence with cp * Hkv <= x: it has tiles
                    while (hi - lo > 1) {
                        const int mid = (lo + hi) / 2;
                        if (sm.cp[mid] * a.Hkv <= x) lo = mid; else hi = mid;
                    }
                    load(a, lo);
                    const int64_t y = sm.cp[lo] + head_of(a, sm.cp[lo], sm.cp[lo + 1] - sm.cp[lo]);
                    int r0 = 0, r1 = THREADS;  // the last run that begins at or before y
                    while (r1 - r0 > 1) {
                        const int mid = (r0 + r1) / 2;
                        if (mid * per < base && sm.tp[mid] <= y) r0 = mid; else r1 = mid;
                    }
                    // from there, or from the sequence's first row tile
                    qt = r0 * per - sm.sq[lo];
                    int64_t p = sm.tp[r0];
                    if (qt < 0) {
                        qt = 0;
                        p = sm.cp[lo];
                    }
                    tile_of(a, p, y);
                    tell(h);
                }
            }
        }
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");  // asynchronous copies may land on `sm` next
        __syncthreads();
        s = h.s;
        qt = h.qt;
        off = h.off;
    }
    // The sequence and row tile of global row tile q.
    __device__ __forceinline__ void find(const PagedArgs& a, const PagedPlanSmem& sm, int q) {
        int lo = 0, hi = nseq;  // the last sequence with sq <= q has tiles: sq[lo + 1] > q
        while (hi - lo > 1) {
            const int mid = (lo + hi) / 2;
            if (sm.sq[mid] <= q) lo = mid; else hi = mid;
        }
        load(a, lo);
        qt = q - sm.sq[lo];
    }
    // The next row tile (a sequence without tokens has none); stays put after the last.
    __device__ __forceinline__ void step(const PagedArgs& a) {
        ++qt;
        if (qt * (int64_t)a.tpt >= s.n) {
            int i = s.seq + 1;
            while (i < nseq) {
                load(a, i);
                if (s.n > 0) break;
                ++i;
            }
            qt = 0;
            if (i >= nseq) s.n = 0;
        }
    }

    // The next stretch of an item; false when the CTA's share is done.
    __device__ __forceinline__ bool next(const PagedArgs& a, PagedSeg& out) {
        while (x < x_end) {
            const int c = item(a);
            const int64_t room = x_end - x;
            const int end = (int)(room < c - off ? off + room : c);
            out = s;
            out.ta = (off >> (s.w - 1)) & -(1 << cut);
            out.tb = end == c ? s.tiles.nt : (end >> (s.w - 1)) & -(1 << cut);
            x += end - off;
            off = 0;
            if (++qt * (int64_t)a.tpt >= s.n) {
                qt = 0;
                if (++s.head == a.Hkv) {
                    s.head = 0;
                    if (x < x_end) {
                        do load(a, s.seq + 1);
                        while (s.n == 0);
                    }
                }
            }
            if (out.tb > out.ta) return true;
        }
        return false;
    }
};

// Whether a stretch leaves a partial, and where: slot A when it begins inside its
// item, slot B when it only ends inside.
__device__ __forceinline__ bool paged_whole(const PagedSeg& s) { return s.ta == 0 && s.tb == s.tiles.nt; }

__device__ __forceinline__ float* paged_slot(const PagedArgs& a, int cta, int slot) {
    return a.part + ((int64_t)cta * 2 + slot) * a.slot_rows * (a.d + 2);
}
// A slot holds m [slot_rows] (log2 units), l [slot_rows], then O [slot_rows][d] (in the
// tensor-memory kernel's own order).

// Launches a kernel that begins beside the one before it and waits for its end.
template <typename Kernel>
cudaError_t launch_paged_dependent(Kernel kernel, dim3 grid, int threads, cudaStream_t st, const PagedArgs& a) {
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3((unsigned)threads);
    cfg.stream = st;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    ripe_count_launch();
    return cudaLaunchKernelEx(&cfg, kernel, a);
}

// The sum of the values of V in channel c that are not finite, of keys the row sees in
// key tiles that are not seen whole by all rows (0 if there are none): the kernels read
// such values as zeros there, because a matrix product would carry them (0 * inf) into
// rows whose mask hides them.
template <int KT>
__device__ __noinline__ float paged_nonfinite(const PagedArgs& a, const PagedSeg& s, int pos, int c) {
    const int p0 = s.c + s.t0, p1 = p0 + s.ntok - 1;
    float sum = 0.f;
    for (int t = s.ta; t < s.tb; ++t) {
        const int k0 = s.tiles.tile(t) * KT;
        if (paged_all_seen(a, k0, KT, p0, p1)) continue;
        for (int key = k0; key < k0 + KT && key <= pos; ++key) {
            if (!paged_seen(a, key, pos)) continue;
            const int64_t row = paged_page(a, s.seq, key) * a.page_stride + s.head * a.head_stride +
                                (key & (a.page - 1)) * a.pos_stride;
            const float f = __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(a.v)[row + c]);
            if (!isfinite(f)) sum += f;
        }
    }
    return sum;
}
