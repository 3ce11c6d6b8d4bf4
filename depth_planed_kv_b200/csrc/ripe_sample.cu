// ripe_sample.cu -- the draw of one token per row of logits, with temperature, top-k,
// top-p and min-p, from given uniforms.
//
// With m = max_v z_v and w_v = exp((z_v - m) / T), and the tokens in the order (z
// descending, v ascending), the kept set is a prefix of that order:
//   top-k   the first k tokens;
//   top-p   those with (mass before them) < p * (mass of the first k), at least one;
//   min-p   those with w_v >= min_p (w of the first token is 1).
// The token is the smallest v whose running sum of kept w, in index order, exceeds u
// times the kept mass; its log probability is log(w_v / kept mass).
//
// A draw is a comparison of running sums with a border, so the sums must not depend on
// the order of additions, and a weight's error must be small against the borders of a
// flat row, 1/V apart: weights are integers of 2^-46 of the largest (2^-(63 - ceil(log2 V))
// above 2^17 tokens, so that a sum of V of them stays within 2^63), which add up exactly in
// any order.  Each is right to 2^-30 of itself and half a unit; V half units are below
// 2^-24 of the largest weight, u's own resolution, up to 2^20 tokens (2^-18 for 2^23).
// (With 32-bit exponentials and sums about one row in 10^4 of 10^5 near-equal tokens would
// draw its neighbour.)
//
// One cluster of 1 to 8 CTAs per row; each CTA holds a contiguous slice of the row in
// shared memory, so the logits are read from memory once.
//   top-k up to a few hundred: each CTA's threads have the largest logit
//     of their share; the ceil(k / CTAs)-th largest of those is a bound that so many of the
//     CTA's tokens reach, so the least such bound of the CTAs is reached by k tokens of the
//     row, and by few more where large logits lie all over the row.  Those alone are gathered
//     in the first CTA, sorted and drawn from; the other CTAs are done.  Where they lie close
//     together (rising or falling with the index, or a slice of -inf), the bound is too low, a
//     CTA has more than its part of the list holds, and the row goes the last way below.
//   top-p: 1024 bins of tokens and mass, linear in z below the maximum, which the CTAs
//     read from one another through distributed shared memory, give the bin where the mass
//     passes p.  The tokens down to it, if few, are gathered as above; else the border's
//     bin alone is gathered and sorted, and then all CTAs sum what is kept.
//   else (many tokens in that bin, a large k, or as above): bins of the ordered bit pattern in
//     the border's bin, until it holds one token or one value.
//
// Measured, normal logits: 1 x 32000 fp32, all filters: 10.7 us, a chain of load, maximum, two
// cluster barriers and one CTA's sort (clusters of 2 to 8 CTAs all take 10.5 to 11.4).
// 48 x 65537 bf16, top-p and min-p: 38 us (6 CTAs a row: 36, 4: 43, 2: 56).  256 x 131072
// fp32, three rows in ten without top-k: 149 us, 0.90 TB/s of 134 MB.  Instructions bind the
// large ones; by the kind of row (256 x 131072, every row alike), a warp's instructions for 32
// tokens: top-k alone 36 (102 us), temperature alone 92 (160 us), top-p 165 (296 us: bin,
// weight and its atomics, the weight again for what is kept), top-k with the large logits in
// one eighth of the row 145 (310 us; with top-p and min-p besides 570, where they lie all over
// the row 102).
#include <math.h>

#include "ripe_internal.cuh"
#include "ripe_launch.h"

namespace {

constexpr int kThreads = 512, kWarps = kThreads / 32;
constexpr int kBins = 1024;
constexpr int kMaxCluster = 8;
constexpr int kList = kThreads;  // tokens sorted in one CTA
constexpr float kRange = 28.f;  // the bins reach this many units of T below the maximum
constexpr int kPow = 512;       // table of 2^(-i / 512)

typedef unsigned long long u64;

struct SampleArgs {
    const void* z;
    int64_t row_stride;
    int nrows, V, per, seg;  // per: tokens of one CTA; seg: tokens of one warp (a multiple of 32)
    const float *u, *temperature, *top_p, *min_p;
    const int32_t* top_k;
    int32_t* token;
    float* logprob;
    int bits;  // the largest weight is 2^bits
};

// What a CTA tells the others of its cluster; two of them in turn, so that one cluster
// barrier per exchange is enough.
struct alignas(16) Msg {
    u64 sum;  // or a key
    float mx;
    int idx;
};

// 2^31 * 2^(-i / 512), by repeated multiplication with 2^(-1/512) in 64 bits.
struct PowTable {
    unsigned v[kPow];
};
constexpr u64 mul_high(u64 a, u64 b) {
    const u64 al = a & 0xffffffffull, ah = a >> 32, bl = b & 0xffffffffull, bh = b >> 32;
    const u64 mid = ah * bl + ((al * bl) >> 32), mid2 = al * bh + (mid & 0xffffffffull);
    return ah * bh + (mid >> 32) + (mid2 >> 32);
}
constexpr PowTable make_pow_table() {
    PowTable t{};
    const u64 step = 18421787711448657618ull;  // 2^64 * 2^(-1/512)
    u64 x = step;
    t.v[0] = 0x80000000u;
    for (int i = 1; i < kPow; ++i) {
        t.v[i] = (unsigned)((x + (1ull << 32)) >> 33);
        x = mul_high(x, step);
    }
    return t;
}
__device__ const PowTable kPowTable = make_pow_table();

struct Shared {
    unsigned cnt[2][kBins], lo[2][kBins], hi[2][kBins];  // bins: tokens, mass (low and high words)
    u64 list[kList];      // gathered tokens: (key, ~index), so that larger comes first
    u64 swap[2 * kList];
    unsigned mine[kList];  // this CTA's tokens for the list
    unsigned pow2[kPow];  // 2^31 * 2^(-i / 512)
    Msg msg[2][kMaxCluster];
    u64 wsum[kWarps], scan[kWarps];
    float wmax[kWarps];
    int widx[kWarps];
    u64 pick[6];
    unsigned listed, token;
    unsigned count[2][kMaxCluster];  // tokens each CTA lists
    double it, c, low;               // the row's settings, see Row
};

__device__ __forceinline__ unsigned cluster_size() {
    unsigned n;
    asm("mov.u32 %0, %%cluster_nctaid.x;" : "=r"(n));
    return n;
}
__device__ __forceinline__ unsigned cluster_rank() {
    unsigned n;
    asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(n));
    return n;
}
// Without .aligned: the loops before a barrier may leave a warp's lanes apart.
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire;" ::: "memory"); }
__device__ __forceinline__ void cluster_sync() {
    cluster_arrive();
    cluster_wait();
}
// The address of `p` (shared memory of this CTA) in CTA `rank` of the cluster.
__device__ __forceinline__ uint32_t peer(const void* p, unsigned rank) {
    uint32_t a;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"((uint32_t)__cvta_generic_to_shared(p)), "r"(rank));
    return a;
}
__device__ __forceinline__ uint2 peer_ld2(uint32_t a) {
    uint2 x;
    asm volatile("ld.shared::cluster.v2.u32 {%0, %1}, [%2];" : "=r"(x.x), "=r"(x.y) : "r"(a));
    return x;
}
__device__ __forceinline__ void peer_st(uint32_t a, unsigned x) {
    asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(a), "r"(x) : "memory");
}

// NaN is never drawn; -0 is 0; +inf counts as the largest finite value.
__device__ __forceinline__ float to_logit(float x) { return x != x ? -INFINITY : fminf(x, 3.402823466e38f) + 0.f; }
__device__ __forceinline__ float load_logit(const float* z, int64_t i) { return to_logit(__ldg(z + i)); }
__device__ __forceinline__ float load_logit(const __nv_bfloat16* z, int64_t i) { return to_logit(__bfloat162float(z[i])); }
// The logits of 16 bytes.
__device__ __forceinline__ void unpack(const uint4& v, const float*, float* x) {
    x[0] = __uint_as_float(v.x);
    x[1] = __uint_as_float(v.y);
    x[2] = __uint_as_float(v.z);
    x[3] = __uint_as_float(v.w);
}
__device__ __forceinline__ void unpack(const uint4& v, const __nv_bfloat16*, float* x) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[2 * i] = __uint_as_float(w[i] << 16);
        x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
}

// The bit pattern of a logit as an integer of the same order.
__device__ __forceinline__ unsigned key_of(float x) {
    const unsigned b = __float_as_uint(x);
    return b & 0x80000000u ? ~b : b | 0x80000000u;
}

__device__ __forceinline__ float logit_of(unsigned key) {
    return __uint_as_float(key & 0x80000000u ? key & 0x7FFFFFFFu : ~key);
}

struct Row {
    float m, scale0;       // maximum; bins per unit of z at the first level
    float c_hi, c_lo, c_512;  // log2(e) / T as a sum of two floats, and 512 times it
    double dm, it;         // maximum, 1 / T
    int bits;
    const unsigned* pow2;
    // 2^bits * exp((x - m) / T), rounded.  t = (m - x) * c (the difference with its rounding
    // error, the product through fused operations), t = k / 512 + r; 2^-t = 2^(-k / 512) (1 - q),
    // q = 1 - 2^-r = r (ln2 - r (ln2^2 / 2 - r ln2^3 / 6)) for |r| < 2^-9.9: the next term is
    // below 2^-46, q is right to 2^-31 (its fp32 steps 2^-33, its rounding 2^-32) and the table
    // to 2^-31.
    __device__ __forceinline__ u64 weight(float x) const {
        const float hi = m - x, bb = hi - m, lo = (m - (hi - bb)) - (x + bb);
        const float kMagic = 12582912.f;  // 1.5 * 2^23: adding it leaves the rounded integer in the low bits
        const float p = hi * c_512;
        if (!(p < (float)(kPow * (bits + 1)))) return 0ull;  // also -inf
        const float y = p + kMagic, kf = (y - kMagic) * (-1.f / kPow);
        const float r = fmaf(lo, c_hi, fmaf(hi, c_lo, fmaf(hi, c_hi, kf)));
        const float q = r * (0.693147181f - r * (0.240226507f - r * 0.0555041087f));
        const int qi = __float_as_int(fmaf(q, 2147483648.f, kMagic)) - __float_as_int(kMagic);
        const int k = __float_as_int(y) - __float_as_int(kMagic);
        const unsigned T = pow2[k & (kPow - 1)];
        const u64 w = ((u64)T << 31) - (u64)((long long)qi * (long long)T);  // 2^62 * 2^-frac
        const int sh = 62 - bits + (k >> 9);  // k <= 512 * (bits + 1): sh <= 63
        return (w + (1ull << (sh - 1))) >> sh;
    }
    // first-level bin: linear in z, largest first; monotone
    __device__ __forceinline__ int bin0(float x) const {
        return __float_as_int(fminf((m - x) * scale0, (float)(kBins - 1)) + 8388608.f) & (kBins - 1);
    }
};

template <typename Elem, bool RES>
struct Cta {
    const SampleArgs& a;
    Shared& sh;
    float* sx;
    const Elem* z;
    int n;  // tokens of this CTA's slice
    unsigned rank, size;
    int tid, warp, lane, phase = 0;  // phase: which Msg buffer is next

    __device__ __forceinline__ float get(int i) const { return RES ? sx[i] : load_logit(z, i); }

    // f(i, x) for every token of the slice, each warp its contiguous segment in order.
    template <typename F>
    __device__ __forceinline__ void each(F&& f) const {
        const int e = min(n, (warp + 1) * a.seg);
#pragma unroll 4
        for (int i = warp * a.seg + lane; i < e; i += 32) f(i, get(i));
    }

    // The same in any order, 16 bytes of shared memory at a time (a: where the slice's first
    // token lies against 16 bytes).
    template <typename F>
    __device__ __forceinline__ void each_any(F&& f) const {
        if (!RES) {
            each(f);
            return;
        }
        const int off = (int)(((uintptr_t)sx & 15) / 4), i0 = min(n, (4 - off) & 3), nq = (n - i0) / 4;
#pragma unroll 2
        for (int q = tid; q < nq; q += kThreads) {
            const int i = i0 + 4 * q;
            const float4 v = *reinterpret_cast<const float4*>(sx + i);
            f(i, v.x);
            f(i + 1, v.y);
            f(i + 2, v.z);
            f(i + 3, v.w);
        }
        if (tid < n - 4 * nq) {
            const int i = tid < i0 ? tid : tid + 4 * nq;
            f(i, sx[i]);
        }
    }

    // Gathers tokens (each CTA's `count` slice indexes in sh.mine) in the first CTA: each CTA
    // has its own part of the list there, so that one barrier of the cluster does.  False (to
    // all CTAs) if one has more than its part holds.  In the first CTA the tokens end up in
    // sh.list[0 .. n).
    __device__ __forceinline__ bool gather(unsigned count, int v0, int use, int& n) {
        const unsigned part = 2 * kList / size, most = part < kList ? part : kList;  // sh.mine holds kList
        if (tid < (int)size) peer_st(peer(&sh.count[use][rank], tid), count);
        if (count <= most)
            for (unsigned j = tid; j < count; j += kThreads) {
                const int i = sh.mine[j];
                const uint32_t d = peer(sh.swap + rank * part + j, 0);
                peer_st(d + 4, key_of(get(i)));
                peer_st(d, ~(unsigned)(v0 + i));
            }
        cluster_sync();
        bool fit = true;
        n = 0;
        for (unsigned i = 0; i < size; ++i) {
            const unsigned c = sh.count[use][i];
            fit &= c <= most;
            n += (int)c;
        }
        fit &= n <= kList;
        if (rank == 0 && fit) {
            for (unsigned q = tid; q < 2 * kList; q += kThreads) {
                const unsigned from = q / part, j = q % part;
                unsigned at = 0;
                for (unsigned i = 0; i < from; ++i) at += sh.count[use][i];
                if (j < sh.count[use][from]) sh.list[at + j] = sh.swap[q];
            }
            __syncthreads();
        }
        return fit;
    }

    // How many of sh.list[0 .. n) are larger than this thread's v: its rank.
    __device__ __forceinline__ int rank_of(u64 v, int n) const {
        int k = 0;
        if (warp * 32 < n) {
#pragma unroll 8
            for (int i = 0; i < n; ++i) k += sh.list[i] > v;
        }
        return k;
    }

    // Sum over the threads before and up to this one.
    __device__ __forceinline__ u64 inclusive(u64 v) {
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const u64 x = __shfl_up_sync(0xffffffffu, v, o);
            if (lane >= o) v += x;
        }
        __syncthreads();
        if (lane == 31) sh.wsum[warp] = v;
        __syncthreads();
        static_assert(kWarps == 16, "half a warp adds them");
        u64 s = (lane & 15) < warp ? sh.wsum[lane & 15] : 0ull;
#pragma unroll
        for (int o = 8; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
        return v + s;
    }

    // Tells every CTA of the cluster this CTA's (sum, mx, idx), and returns all of them.
    __device__ __forceinline__ const Msg* exchange(u64 sum, float mx, int idx) {
        Msg* buf = sh.msg[phase];
        phase ^= 1;
        if (tid < (int)size) {
            const uint32_t d = peer(buf + rank, tid);
            peer_st(d, (unsigned)sum);
            peer_st(d + 4, (unsigned)(sum >> 32));
            peer_st(d + 8, __float_as_uint(mx));
            peer_st(d + 12, (unsigned)idx);
        }
        cluster_sync();
        return buf;
    }

    __device__ __forceinline__ u64 block_sum(u64 v) {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
        __syncthreads();
        if (lane == 0) sh.wsum[warp] = v;
        __syncthreads();
        u64 t = 0;
        for (int w = 0; w < kWarps; ++w) t += sh.wsum[w];
        return t;
    }

    // Bins of one level, of all CTAs: finds the bin where the running count (mass == false)
    // or mass passes `target`: the first bin with before < target <= before + own.  share > 0:
    // the target is that share of all the mass of these bins (returned in `target`).  Returns
    // the bin; before_cnt, before_mass grow by what lies in the bins ahead of it; own: its
    // count and mass.
    __device__ int find_bin(int b, bool mass, bool with_mass, double share, double& target, u64& before_cnt,
                            u64& before_mass, u64& own_cnt, u64& own_mass) {
        constexpr int kPer = kBins / kThreads;
        u64 c[kPer], s[kPer], ct = 0, st = 0;
#pragma unroll
        for (int j = 0; j < kPer; ++j) c[j] = s[j] = 0;
        // all loads on their way before the first is added
        static_assert(kPer == 2, "8-byte loads");
        uint2 v[kMaxCluster];
        auto read = [&](const unsigned* from) {
#pragma unroll
            for (unsigned r = 0; r < kMaxCluster; ++r) v[r] = r < size ? peer_ld2(peer(from + tid * kPer, r)) : make_uint2(0, 0);
        };
        read(sh.cnt[b]);
#pragma unroll
        for (unsigned r = 0; r < kMaxCluster; ++r) {
            c[0] += v[r].x;
            c[1] += v[r].y;
        }
        if (with_mass) {
            read(sh.lo[b]);
#pragma unroll
            for (unsigned r = 0; r < kMaxCluster; ++r) {
                s[0] += v[r].x;
                s[1] += v[r].y;
            }
            read(sh.hi[b]);
#pragma unroll
            for (unsigned r = 0; r < kMaxCluster; ++r) {
                s[0] += (u64)v[r].x << 32;
                s[1] += (u64)v[r].y << 32;
            }
        }
#pragma unroll
        for (int j = 0; j < kPer; ++j) {
            ct += c[j];
            st += s[j];
        }
        // exclusive prefix over the threads
        u64 ci = ct, si = st;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const u64 x = __shfl_up_sync(0xffffffffu, ci, o), y = __shfl_up_sync(0xffffffffu, si, o);
            if (lane >= o) {
                ci += x;
                si += y;
            }
        }
        __syncthreads();
        if (lane == 31) {
            sh.wsum[warp] = ci;
            sh.scan[warp] = si;
        }
        if (tid == 0) sh.pick[0] = kBins;
        __syncthreads();
        u64 cb = before_cnt + ci - ct, sb = before_mass + si - st, all = 0;
        for (int w = 0; w < kWarps; ++w) {
            if (w < warp) {
                cb += sh.wsum[w];
                sb += sh.scan[w];
            }
            all += sh.scan[w];
        }
        if (share > 0.0) target = share * (double)all;
#pragma unroll
        for (int j = 0; j < kPer; ++j) {
            const double lo = mass ? (double)sb : (double)cb, up = mass ? (double)(sb + s[j]) : (double)(cb + c[j]);
            if (lo < target && target <= up) {
                sh.pick[0] = tid * kPer + j;
                sh.pick[1] = cb;
                sh.pick[2] = sb;
                sh.pick[3] = c[j];
                sh.pick[4] = s[j];
            }
            cb += c[j];
            sb += s[j];
        }
        __syncthreads();
        const int bin = (int)sh.pick[0];
        if (bin < kBins) {
            before_cnt = sh.pick[1];
            before_mass = sh.pick[2];
            own_cnt = sh.pick[3];
            own_mass = sh.pick[4];
        }
        __syncthreads();
        return bin;
    }

    __device__ __forceinline__ void clear_bins(int b) {
        for (int i = tid; i < kBins; i += kThreads) sh.cnt[b][i] = sh.lo[b][i] = sh.hi[b][i] = 0u;
    }
    __device__ __forceinline__ void add_bin(int b, int i, u64 w) {
        atomicAdd(&sh.cnt[b][i], 1u);
        if (w) {
            const unsigned l = (unsigned)w, old = atomicAdd(&sh.lo[b][i], l);
            const unsigned h = (unsigned)(w >> 32) + (old + l < old ? 1u : 0u);
            if (h) atomicAdd(&sh.hi[b][i], h);
        }
    }
};

// The border of a prefix of the order: tokens with key > kt are in, and the first `c` (in
// index order) of those with key == kt.
struct Border {
    unsigned kt;
    u64 c;      // 0: none
    u64 equal;  // tokens with key == kt (known when c > 0)
    u64 mass;   // of the prefix
};

// From the first level's bins (buffer 0, complete) to the border; later levels use buffer 1.
template <typename Elem, bool RES>
__device__ Border find_border(Cta<Elem, RES>& t, const Row& row, bool mass, double target, bool with_mass) {
    u64 bc = 0, bm = 0, oc = 0, om = 0;
    const int b0 = t.find_bin(0, mass, with_mass, 0.0, target, bc, bm, oc, om);
    Border r;
    r.kt = 0;
    r.c = 0;
    r.equal = 0;
    r.mass = bm + om;
    // the keys that can lie in the bin (its edges, widened by the rounding of bin0)
    const double w = 1.0 / (double)row.scale0, e = (1e-5 * (b0 + 1) + 0.51) * w + 1e-6 * fabs(row.dm);
    unsigned khi = b0 == 0 ? key_of(row.m) : min(key_of(row.m), key_of((float)(row.dm - b0 * w + e)));
    unsigned klo = b0 == kBins - 1 ? key_of(-INFINITY) : key_of((float)(row.dm - b0 * w - e));
    if (klo > khi) klo = khi;
    auto inside = [&](float x, unsigned k) { return k >= klo && k <= khi && row.bin0(x) == b0; };
    while (true) {
        const bool all = mass ? oc == 1 : (double)(bc + oc) == target;
        if (all) {  // the whole bin is in: the border lies below its last token
            r.mass = bm + om;
            r.kt = klo - 1;
            r.c = 0;
            // tokens of a neighbouring first-level bin may share the widened range; the bin's own
            // smallest key is the border
            unsigned least = 0xffffffffu;
            t.each([&](int, float x) {
                const unsigned k = key_of(x);
                if (inside(x, k)) least = min(least, k);
            });
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) least = min(least, __shfl_xor_sync(0xffffffffu, least, o));
            __syncthreads();
            if (t.lane == 0) t.sh.widx[t.warp] = (int)least;
            __syncthreads();
            for (int i = 0; i < kWarps; ++i) least = min(least, (unsigned)t.sh.widx[i]);
            const Msg* g = t.exchange(0, 0.f, (int)least);
            for (unsigned i = 0; i < t.size; ++i) least = min(least, (unsigned)g[i].idx);
            r.kt = least - 1;
            return r;
        }
        if (klo == khi) {
            r.kt = klo;
            r.equal = oc;
            const u64 w1 = oc ? om / oc : 0;
            double c = mass ? ceil((target - (double)bm) / (double)(w1 ? w1 : 1)) : target - (double)bc;
            r.c = (u64)fmin(fmax(c, 1.0), (double)oc);
            r.mass = bm + r.c * w1;
            return r;
        }
        // bins of the ordered bit pattern over [klo, khi], largest first
        int shift = 0;
        while (((khi - klo) >> shift) >= kBins) ++shift;
        const int b = 1;
        cluster_sync();  // nobody reads the bins of the level before any more
        t.clear_bins(b);
        __syncthreads();
        t.each([&](int, float x) {
            const unsigned k = key_of(x);
            if (inside(x, k)) t.add_bin(b, (int)((khi - k) >> shift), with_mass ? row.weight(x) : 0ull);
        });
        cluster_sync();
        const int i = t.find_bin(b, mass, with_mass, 0.0, target, bc, bm, oc, om);
        const unsigned top = khi - ((unsigned)i << shift);
        const unsigned span = (1u << shift) - 1;
        if (i >= kBins) {  // cannot be: the bins hold what the bin before held
            r.kt = klo - 1;
            return r;
        }
        klo = top - klo > span ? top - span : klo;
        khi = top;
    }
}

template <typename Elem, bool RES>
__global__ void __launch_bounds__(kThreads, 2) sample_kernel(const __grid_constant__ SampleArgs a) {
    extern __shared__ __align__(16) char smem[];
    Shared& sh = *reinterpret_cast<Shared*>(smem);
    const unsigned size = cluster_size();
    const int r = blockIdx.x / size;
    Cta<Elem, RES> t{a, sh, reinterpret_cast<float*>(smem + sizeof(Shared)), nullptr, 0, cluster_rank(), size,
                     (int)threadIdx.x, (int)threadIdx.x / 32, (int)threadIdx.x % 32};
    if (t.tid == 0) sh.listed = 0;
    cluster_arrive();  // waited for before the first word to another CTA: by then all have started
    const int v0 = t.rank * a.per;
    t.z = reinterpret_cast<const Elem*>(a.z) + r * a.row_stride + v0;
    t.n = max(0, min(a.per, a.V - v0));

    const float T = a.temperature ? __ldg(a.temperature + r) : 1.f;
    const int k = a.top_k ? __ldg(a.top_k + r) : 0;
    const float p = a.top_p ? __ldg(a.top_p + r) : 1.f;
    const float mp = a.min_p ? __ldg(a.min_p + r) : 0.f;
    if (t.tid == kThreads - 1) {  // 64-bit divisions and logarithms once, beside the loads
        sh.it = 1.0 / (double)T;
        sh.c = 1.4426950408889634074 * sh.it;
        sh.low = mp > 0.f ? log((double)mp) * (double)T : -INFINITY;  // min-p, as a bound on z - m
    }

    // ---- the slice, and the largest logit (lowest index on ties)
    float mx = -INFINITY;
    int mi = 0x7fffffff;
    auto better = [&](float x, int i) {
        if (x > mx || (x == mx && i < mi)) {
            mx = x;
            mi = i;
        }
    };
    if (RES) {
        // 16 bytes at a time from the first aligned address; token i goes to sx[i], which is
        // laid so that an aligned 16 bytes of logits meets aligned shared memory
        constexpr int kV = 16 / sizeof(Elem);
        const int pad = (int)(((uintptr_t)t.z & 15) / sizeof(Elem)), i0 = min(t.n, (kV - pad) % kV), nv = (t.n - i0) / kV;
        t.sx += pad;
        const uint4* src = reinterpret_cast<const uint4*>(t.z + i0);
        auto take = [&](const uint4& q, int j) {
            float x[kV];
            unpack(q, (const Elem*)nullptr, x);
#pragma unroll
            for (int e = 0; e < kV; ++e) {
                x[e] = to_logit(x[e]);
                if (x[e] > mx) {
                    mx = x[e];
                    mi = i0 + j * kV + e;
                }
            }
#pragma unroll
            for (int e = 0; e < kV; e += 4)
                *reinterpret_cast<float4*>(t.sx + i0 + j * kV + e) = make_float4(x[e], x[e + 1], x[e + 2], x[e + 3]);
        };
        int j = t.tid;
        for (; j + 3 * kThreads < nv; j += 4 * kThreads) {
            const uint4 q0 = __ldg(src + j), q1 = __ldg(src + j + kThreads), q2 = __ldg(src + j + 2 * kThreads),
                        q3 = __ldg(src + j + 3 * kThreads);
            take(q0, j);
            take(q1, j + kThreads);
            take(q2, j + 2 * kThreads);
            take(q3, j + 3 * kThreads);
        }
        for (; j < nv; j += kThreads) take(__ldg(src + j), j);
        const int rest = t.n - nv * kV;  // before the first and after the last 16 bytes
        if (t.tid < rest) {
            const int i = t.tid < i0 ? t.tid : t.tid + nv * kV;
            const float x = load_logit(t.z, i);
            t.sx[i] = x;
            better(x, i);
        }
    } else {
        t.each([&](int i, float x) {
            if (x > mx) {
                mx = x;
                mi = i;
            }
        });
    }
    t.clear_bins(0);
    for (int i = t.tid; i < kPow; i += kThreads) sh.pow2[i] = kPowTable.v[i];
    const unsigned top = key_of(mx);  // of this thread's tokens
    mi = mi == 0x7fffffff ? mi : mi + v0;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        const float x = __shfl_xor_sync(0xffffffffu, mx, o);
        const int i = __shfl_xor_sync(0xffffffffu, mi, o);
        better(x, i);
    }
    if (t.lane == 0) {
        sh.wmax[t.warp] = mx;
        sh.widx[t.warp] = mi;
    }
    __syncthreads();
    // ---- top-k: the bound that enough of this CTA's tokens reach (see above), to 16 bits of its key
    const bool need_k = k > 0 && k < a.V, need_p = p < 1.f, few_k = need_k && k <= kList * 3 / 4;
    unsigned bound = 0;
    if (few_k) {
        reinterpret_cast<unsigned short*>(sh.mine)[t.tid] = (unsigned short)(top >> 16);
        __syncthreads();
    }
    {
        mx = sh.wmax[t.lane & (kWarps - 1)];
        mi = sh.widx[t.lane & (kWarps - 1)];
#pragma unroll
        for (int o = kWarps / 2; o > 0; o >>= 1) {
            const float x = __shfl_xor_sync(0xffffffffu, mx, o);
            const int i = __shfl_xor_sync(0xffffffffu, mi, o);
            better(x, i);
        }
    }
    if (few_k) {
        // one warp looks for the bound: 16 maxima a lane, in eight words
        if (t.warp == 0) {
            const int want = (k + (int)size - 1) / (int)size;
            unsigned v[8], least16 = 0xffffu;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                v[i] = sh.mine[t.lane + 32 * i];
                least16 = min(least16, min(v[i] & 0xffffu, v[i] >> 16));
            }
            // all of the threads' maxima reach lo, none reaches hi
            unsigned lo = __reduce_min_sync(0xffffffffu, least16), hi = (key_of(mx) >> 16) + 1;
            if (want > kThreads) hi = lo + 1;
            while (hi - lo > 1) {
                const unsigned mid = (lo + hi) / 2;
                int c = 0;
#pragma unroll
                for (int i = 0; i < 8; ++i) c += ((v[i] & 0xffffu) >= mid) + ((v[i] >> 16) >= mid);
                if (__reduce_add_sync(0xffffffffu, c) >= want) lo = mid; else hi = mid;
            }
            bound = lo;  // t.tid < size tells the others
        }
    }
    cluster_wait();
    {
        const Msg* g = t.exchange(bound, mx, mi);
        bound = 0xffffu;
        for (unsigned i = 0; i < size; ++i) {
            better(g[i].mx, g[i].idx);
            bound = min(bound, (unsigned)g[i].sum);
        }
    }
    // Every CTA of the cluster takes the same way out; a CTA leaves only when no other will
    // read or write its shared memory any more.
    if (mx == -INFINITY || !(T > 0.f) || k == 1 || mp > 1.f || p <= 0.f) {
        if (t.rank == 0 && t.tid == 0) {
            a.token[r] = mx == -INFINITY ? -1 : mi;
            if (a.logprob) a.logprob[r] = mx == -INFINITY ? -INFINITY : 0.f;
        }
        return;  // the exchange's barrier was the last word to any CTA
    }
    Row row;
    row.m = mx;
    row.dm = mx;
    row.it = sh.it;
    const double c = sh.c;
    row.c_hi = fminf((float)c, 1e30f);
    row.c_512 = row.c_hi * kPow;
    row.c_lo = c < 1e30 ? (float)(c - (double)row.c_hi) : 0.f;
    row.scale0 = fminf(fmaxf((float)kBins / (kRange * T), 1e-30f), 1e30f);
    row.bits = a.bits;
    row.pow2 = sh.pow2;
    const double one = (double)(1ull << a.bits);
    const float least = mp > 0.f ? fminf(__double2float_ru(row.dm + sh.low), row.m) : -INFINITY;
    auto min_p_keeps = [&](float x) { return x >= least; };
    const float u = __ldg(a.u + r);
    // u outside [0, 1) is taken as its nearer end (at 1: the last token with weight)
    const double uu = fmin(u > 0.f ? (double)u : 0.0, 1.0 - 0x1p-50);
    auto logprob_of = [&](float x, double W) {
        return (x == row.m ? 0.f : (float)(((double)x - row.dm) * row.it)) - logf((float)(W / one));
    };
    // at u below the resolution, the first kept token of any weight at all
    auto any_weight = [&](float x) { return x == row.m || ((double)x - row.dm) * row.it > -745.0; };

    // The first CTA's end of a row whose tokens of interest (n of them) are all in its list.
    auto draw_from_list = [&](int n, double target) {
        const u64 mine = t.tid < n ? sh.list[t.tid] : 0ull;
        const int at = t.rank_of(mine, n);
        if (t.tid == 0) sh.token = 0xffffffffu;
        if (t.tid < n) sh.swap[at] = mine;
        __syncthreads();
        // in the order of the logits
        const u64 v = t.tid < n ? sh.swap[t.tid] : 0ull;
        const float x = logit_of((unsigned)(v >> 32));
        const u64 w = t.tid < n ? row.weight(x) : 0ull;
        bool in = t.tid < n && (!need_k || t.tid < k);
        const u64 upto = t.inclusive(in ? w : 0ull);
        if (need_k && need_p) {
            if (t.tid == min(n, k) - 1) sh.pick[0] = upto;
            __syncthreads();
            target = (double)p * (double)sh.pick[0];
        }
        in = in && (!need_p || t.tid == 0 || (double)(upto - w) < target) && min_p_keeps(x);
        const int kept = __syncthreads_count(in);  // the first `kept` tokens
        if (t.tid == kept - 1) sh.pick[1] = upto;
        // in the order of the indexes: the low words are ~index, so smaller is later
        if (t.tid < kept) sh.list[t.tid] = (u64)(unsigned)v;
        __syncthreads();
        const u64 W = sh.pick[1];
        const int place = t.rank_of((unsigned)v, kept);
        if (t.tid < kept) sh.swap[place] = w;
        __syncthreads();
        const double goal = uu * (double)W;
        const u64 run = t.inclusive(t.tid < kept ? sh.swap[t.tid] : 0ull);
        // the place where the running sum passes the goal; u below the resolution: the first token
        // of any weight
        if (t.tid < kept) {
            if (goal < 1.0 ? false : (double)run > goal) atomicMin(&sh.token, (unsigned)t.tid);
            if (goal < 1.0 && any_weight(x)) atomicMin(&sh.token, (unsigned)place);
        }
        __syncthreads();
        if (t.tid < kept && (unsigned)place == sh.token) {
            a.token[r] = (int)~(unsigned)v;
            if (a.logprob) a.logprob[r] = logprob_of(x, (double)W);
        }
    };

    // ---- the border of top-k and top-p
    Border bd;
    bd.kt = 0;
    bd.c = 0;
    bd.equal = 0;
    int last_equal = 0x7fffffff;  // of the tokens at the border, the last index that is in
    // Slice indexes of the tokens for which f(x), in sh.mine (as many as fit); returns how many.
    auto collect = [&](auto&& f) -> unsigned {
        t.each_any([&](int i, float x) {
            if (f(x)) {
                const unsigned at = atomicAdd(&sh.listed, 1u);
                if (at < kList) sh.mine[at] = (unsigned)i;
            }
        });
        __syncthreads();
        return sh.listed;
    };
    if (few_k) {
        const float from = bound <= 0x007fu ? -INFINITY : logit_of(bound << 16);
        int n;
        if (t.gather(collect([&](float x) { return x >= from; }), v0, 0, n)) {
            if (t.rank == 0) draw_from_list(n, 0.0);
            return;
        }
    }
    if (need_k || need_p) {
        const bool mass0 = need_p && !need_k;  // with top-k, weights count among the first k only
        auto fill = [&](bool with_mass) {
            unsigned last = 0;  // tokens of the last bin, most of them: counted apart
            t.each_any([&](int, float x) {
                const int b = row.bin0(x);
                const u64 w = with_mass ? row.weight(x) : 0ull;
                if (b == kBins - 1 && w == 0) ++last;
                else t.add_bin(0, b, w);
            });
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) last += __shfl_xor_sync(0xffffffffu, last, o);
            if (t.lane == 0 && last) atomicAdd(&sh.cnt[0][kBins - 1], last);
        };
        fill(mass0);
        cluster_sync();
        u64 bc = 0, bm = 0, oc = 0, om = 0;
        double target = (double)k;
        const int b0 = t.find_bin(0, !need_k, mass0, need_k ? 0.0 : (double)p, target, bc, bm, oc, om);
        const bool whole = bc + oc <= kList;  // all tokens down to the border's bin fit the list
        bool listed_all = false;
        if (mass0 && (whole || oc <= kList)) {
            // a first test that is cheaper than the bin: half a bin and the rounding below it
            const float from = b0 == kBins - 1 ? -INFINITY
                                               : (float)(row.dm - (b0 + 0.51 + 1e-5 * b0) / (double)row.scale0 - 1e-6 * fabs(row.dm));
            int n;
            listed_all = t.gather(collect([&](float x) {
                if (!(x >= from)) return false;
                const int b = row.bin0(x);
                return b == b0 || (whole && b < b0);
            }), v0, 1, n);
            if (listed_all && whole) {
                if (t.rank == 0) draw_from_list(n, target);
                return;
            }
            // -------- the last token kept, of the border's bin, to all CTAs
            if (listed_all && t.rank == 0) {
                const u64 mine = t.tid < n ? sh.list[t.tid] : 0ull;
                const int at = t.rank_of(mine, n);
                if (t.tid < n) sh.swap[at] = mine;
                __syncthreads();
                const u64 v = t.tid < n ? sh.swap[t.tid] : 0ull;
                const u64 w = t.tid < n ? row.weight(logit_of((unsigned)(v >> 32))) : 0ull;
                const u64 ahead = bm + t.inclusive(w) - w;
                const int in = __syncthreads_count(t.tid < n && (bc + t.tid == 0 || (double)ahead < target));
                if (t.tid == in - 1)
                    for (unsigned i = 0; i < size; ++i) {
                        const uint32_t d = peer(&sh.pick[5], i);
                        peer_st(d, (unsigned)(v >> 32));
                        peer_st(d + 4, ~(unsigned)v);
                    }
            }
            if (listed_all) {
                cluster_sync();
                bd.kt = (unsigned)sh.pick[5];
                bd.c = 1;
                last_equal = (int)(sh.pick[5] >> 32);
            }
        }
        if (!listed_all) {
            // -------- many tokens in the border's bin, or a large k
            if (need_k && need_p) {  // now with the weights
                cluster_sync();
                t.clear_bins(0);
                __syncthreads();
                fill(true);
                cluster_sync();
            }
            if (need_k) bd = find_border(t, row, false, (double)k, need_p);
            if (need_p) bd = find_border(t, row, true, need_k ? (double)p * (double)bd.mass : target, true);
            if (bd.c > 0 && bd.c < bd.equal) {
                u64 n = 0;
                t.each([&](int, float x) { n += key_of(x) == bd.kt; });
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) n += __shfl_xor_sync(0xffffffffu, n, o);
                const u64 mine = n;
                const u64 all = t.block_sum(t.lane == 0 ? n : 0ull);
                const Msg* g = t.exchange(all, 0.f, 0);
                u64 before = 0;
                for (unsigned i = 0; i < t.rank; ++i) before += g[i].sum;
                for (int w = 0; w < t.warp; ++w) before += sh.wsum[w];
                int found = 0x7fffffff;
                if (before < bd.c && bd.c <= before + mine) {
                    const int e = min(t.n, (t.warp + 1) * a.seg);
                    for (int i0 = t.warp * a.seg; i0 < e; i0 += 32) {
                        const int i = i0 + t.lane;
                        const unsigned hit = __ballot_sync(0xffffffffu, i < e && key_of(t.get(i)) == bd.kt);
                        const u64 want = bd.c - before;  // >= 1
                        if (want <= (u64)__popc(hit)) {
                            unsigned rest = hit;
                            for (u64 j = 1; j < want; ++j) rest &= rest - 1;
                            found = v0 + i0 + __ffs(rest) - 1;
                            break;
                        }
                        before += __popc(hit);
                    }
                }
                __syncthreads();
                if (t.lane == 0) sh.widx[t.warp] = found;
                __syncthreads();
                for (int w = 0; w < kWarps; ++w) found = min(found, sh.widx[w]);
                const Msg* h = t.exchange(0, 0.f, found);
                for (unsigned i = 0; i < size; ++i) last_equal = min(last_equal, h[i].idx);
            }
        }
    }
    // the border as a logit (nothing lies between the keys of -0, which no token has, and of
    // the negative number nearest 0; tokens at -inf weigh nothing)
    const float border = bd.kt == 0x7fffffffu ? __uint_as_float(0x80000001u) : bd.kt <= 0x007fffffu ? -INFINITY : logit_of(bd.kt);
    auto kept = [&](int i, float x) {
        const bool in = !(need_k || need_p) || x > border || (bd.c > 0 && x == border && v0 + i <= last_equal);
        return in && min_p_keeps(x);
    };
    // ---- the draw: all CTAs sum what is kept, in index order
    u64 s = 0;
    t.each([&](int i, float x) {
        if (kept(i, x)) s += row.weight(x);
    });
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    const u64 mine = s;
    const u64 cta = t.block_sum(t.lane == 0 ? s : 0ull);
    const Msg* g = t.exchange(cta, 0.f, 0);
    u64 before = 0, W = 0;
    for (unsigned i = 0; i < size; ++i) {
        if (i < t.rank) before += g[i].sum;
        W += g[i].sum;
    }
    for (int w = 0; w < t.warp; ++w) before += sh.wsum[w];
    const double goal = uu * (double)W;
    auto emit = [&](int i) {
        a.token[r] = v0 + i;
        if (a.logprob) a.logprob[r] = logprob_of(t.get(i), (double)W);
    };
    if (goal < 1.0) {
        int first = 0x7fffffff;
        t.each([&](int i, float x) {
            if (kept(i, x) && any_weight(x)) first = min(first, i);
        });
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) first = min(first, __shfl_xor_sync(0xffffffffu, first, o));
        __syncthreads();
        if (t.lane == 0) sh.widx[t.warp] = first;
        __syncthreads();
        for (int w = 0; w < kWarps; ++w) first = min(first, sh.widx[w]);
        const Msg* h = t.exchange(0, 0.f, first);
        int owner = -1;
        for (int i = (int)size - 1; i >= 0; --i)
            if (h[i].idx != 0x7fffffff) owner = i;
        if (owner == (int)t.rank && t.tid == 0) emit(first);
    } else if ((double)before <= goal && (double)(before + mine) > goal) {
        const int e = min(t.n, (t.warp + 1) * a.seg);
        for (int i0 = t.warp * a.seg; i0 < e; i0 += 32) {
            const int i = i0 + t.lane;
            u64 w = 0;
            if (i < e) {
                const float x = t.get(i);
                if (kept(i, x)) w = row.weight(x);
            }
            u64 inc = w;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const u64 y = __shfl_up_sync(0xffffffffu, inc, o);
                if (t.lane >= o) inc += y;
            }
            const unsigned over = __ballot_sync(0xffffffffu, (double)(before + inc) > goal);
            if (over) {
                if (t.lane == __ffs(over) - 1) emit(i);
                break;
            }
            before += __shfl_sync(0xffffffffu, inc, 31);
        }
    }
}

template <typename Elem, bool RES>
cudaError_t launch_t(SampleArgs a, int cluster, cudaStream_t st) {
    static PerDeviceOnce once;
    constexpr int kMost = 232448;
    cudaError_t e = per_device_once(once, [] {
        return cudaFuncSetAttribute(sample_kernel<Elem, RES>, cudaFuncAttributeMaxDynamicSharedMemorySize, kMost);
    });
    if (e != cudaSuccess) return e;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = (unsigned)cluster;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(a.nrows * cluster));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = sizeof(Shared) + (RES ? (size_t)a.per * 4 + 32 : 0);
    cfg.stream = st;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    ripe_count_launch();
    return cudaLaunchKernelEx(&cfg, sample_kernel<Elem, RES>, a);
}

}  // namespace

cudaError_t launch_sample(int nrows, int V, const void* z, int bf16, int64_t row_stride, const float* u,
                          const float* temperature, const int32_t* top_k, const float* top_p, const float* min_p,
                          int32_t* token, float* logprob, cudaStream_t st) {
    SampleArgs a;
    a.z = z;
    a.row_stride = row_stride;
    a.nrows = nrows;
    a.V = V;
    a.u = u;
    a.temperature = temperature;
    a.top_k = top_k;
    a.top_p = top_p;
    a.min_p = min_p;
    a.token = token;
    a.logprob = logprob;
    a.bits = 46;
    while (V > 1ll << (63 - a.bits)) --a.bits;
    int cluster = 1;
    while (cluster < kMaxCluster && V > cluster * 2048) cluster *= 2;
    a.per = ((V + cluster - 1) / cluster + 7) / 8 * 8;  // slices begin alike against 16 bytes
    a.seg = (a.per + 32 * kWarps - 1) / (32 * kWarps) * 32;
    const bool res = sizeof(Shared) + (size_t)a.per * 4 + 32 <= 232448;
    if (bf16) return res ? launch_t<__nv_bfloat16, true>(a, cluster, st) : launch_t<__nv_bfloat16, false>(a, cluster, st);
    return res ? launch_t<float, true>(a, cluster, st) : launch_t<float, false>(a, cluster, st);
}
