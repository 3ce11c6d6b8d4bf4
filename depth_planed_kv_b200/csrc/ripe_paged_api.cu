// ripe_paged_api.cu -- C entry points of the paged single-plane cache: argument checks,
// the choice of kernel and its workspace.
#include <math.h>
#include <string.h>

#include "ripe_launch.h"
#include "ripe_paged.cuh"
#include "ripe_paged_launch.h"

namespace {

bool aligned(const void* p, uintptr_t n) { return ((uintptr_t)p & (n - 1)) == 0; }

int check_pages(const ripe_pages_t* p) {
    if (!p) return ripe_fail(RIPE_ERR_INVALID_ARG, "pages is NULL");
    if (p->dtype != RIPE_BF16 && p->dtype != RIPE_F32) return ripe_fail(RIPE_ERR_INVALID_ARG, "dtype=%d", p->dtype);
    const int es = p->dtype == RIPE_BF16 ? 2 : 4;
    if (p->Hkv < 1 || p->Hkv > 256) return ripe_fail(RIPE_ERR_INVALID_ARG, "Hkv=%d outside [1,256]", p->Hkv);
    if (p->d < 8 || p->d > 128) return ripe_fail(RIPE_ERR_UNSUPPORTED, "d=%d outside [8,128]", p->d);
    if ((p->d * es) % 16)
        return ripe_fail(RIPE_ERR_UNALIGNED, "d*sizeof(element)=%d not a multiple of 16", p->d * es);
    if (p->page < 16 || p->page > 1024 || (p->page & (p->page - 1)))
        return ripe_fail(RIPE_ERR_INVALID_ARG, "page=%d is not a power of two in [16,1024]", p->page);
    if (p->npages < 1) return ripe_fail(RIPE_ERR_INVALID_ARG, "npages=%d < 1", p->npages);
    if (p->reserved[0] || p->reserved[1] || p->reserved[2])
        return ripe_fail(RIPE_ERR_INVALID_ARG, "reserved fields must be 0");
    const struct { int64_t stride; int n; const char* name; } dims[3] = {{p->page_stride, p->npages, "page_stride"},
                                                                         {p->head_stride, p->Hkv, "head_stride"},
                                                                         {p->pos_stride, p->page, "pos_stride"}};
    for (const auto& x : dims) {
        if (x.n == 1) continue;
        if (x.stride < p->d || x.stride > (1ll << 37) / es)
            return ripe_fail(RIPE_ERR_INVALID_ARG, "%s=%lld outside [d, 2^37 bytes]", x.name, (long long)x.stride);
        if ((x.stride * es) % 16)
            return ripe_fail(RIPE_ERR_UNALIGNED, "%s=%lld elements is not a multiple of 16 bytes", x.name, (long long)x.stride);
    }
    return RIPE_OK;
}

int check_batch(const ripe_pages_t* p, const ripe_paged_batch_t* b) {
    if (!b) return ripe_fail(RIPE_ERR_INVALID_ARG, "batch is NULL");
    if (b->nseq < 0 || b->nseq > kPagedMaxSeqs)
        return ripe_fail(RIPE_ERR_INVALID_ARG, "nseq=%d outside [0,%d]", b->nseq, kPagedMaxSeqs);
    if (b->nrows < 0 || b->nrows > (1 << 24)) return ripe_fail(RIPE_ERR_INVALID_ARG, "nrows=%d outside [0,2^24]", b->nrows);
    if (b->nseq == 0 || b->nrows == 0) return RIPE_OK;
    if (b->table_width < 1 || (int64_t)b->table_width * p->page > (1 << 30))
        return ripe_fail(RIPE_ERR_INVALID_ARG, "table_width=%d: at least 1, and at most 2^30 positions", b->table_width);
    if (b->nseq > 1 && b->table_stride < b->table_width)
        return ripe_fail(RIPE_ERR_INVALID_ARG, "table_stride=%lld < table_width=%d", (long long)b->table_stride, b->table_width);
    if (!p->K || !p->V || !b->table || !b->ctx_len || !b->row0)
        return ripe_fail(RIPE_ERR_INVALID_ARG, "NULL pointer argument");
    if (!aligned(p->K, 16) || !aligned(p->V, 16)) return ripe_fail(RIPE_ERR_UNALIGNED, "the pages must be 16-byte aligned");
    if (!aligned(b->table, 4) || !aligned(b->ctx_len, 4) || !aligned(b->row0, 4) || !aligned(b->err_dev, 4))
        return ripe_fail(RIPE_ERR_UNALIGNED, "int32 arrays must be 4-byte aligned");
    return RIPE_OK;
}

int check_rows(const void* x, int64_t stride, int64_t least, int es, const char* name) {
    if (!x) return ripe_fail(RIPE_ERR_INVALID_ARG, "%s is NULL", name);
    if (!aligned(x, 16)) return ripe_fail(RIPE_ERR_UNALIGNED, "%s must be 16-byte aligned", name);
    if (stride < least || stride > (1ll << 37) / es)
        return ripe_fail(RIPE_ERR_INVALID_ARG, "%s: row stride %lld outside [%lld, 2^37 bytes]", name, (long long)stride,
                         (long long)least);
    if ((stride * es) % 16)
        return ripe_fail(RIPE_ERR_UNALIGNED, "%s: row stride %lld is not a multiple of 16 bytes", name, (long long)stride);
    return RIPE_OK;
}

// Which kernel serves a call, on how many CTAs, and its workspace.
//   decode: at most 16 rows per key/value head and sequence, what its registers hold (tc on
//           such calls: 64 sequences of 512 to 4096 keys with 16 rows each 135 us against
//           124, with 8 rows 131 against 117, one of 1024 keys 19.4 against 13.8, 16 of 32768
//           keys with 4 rows 340 both).
//   tc:     tcgen05; simt: CUDA cores (f32, other head sizes).
struct Plan {
    enum { DECODE, TC, SIMT } kind;
    int G, grid, tok1, tpt, slot_rows;
    size_t bytes;
};

int make_plan(const ripe_pages_t* p, int H, int max_ntok, Plan& q) {
    if (H < 1 || H > 256 || H % p->Hkv)
        return ripe_fail(RIPE_ERR_INVALID_ARG, "H=%d is not a multiple of Hkv=%d in [1,256]", H, p->Hkv);
    if (max_ntok < 1) return ripe_fail(RIPE_ERR_INVALID_ARG, "max_ntok=%d < 1", max_ntok);
    q.G = H / p->Hkv;
    const bool many = fused_supported(p->dtype, p->d);  // heads per key/value head
    const bool tc = many || (p->dtype == RIPE_BF16 && p->d == 32);
    if (q.G > (many ? 128 : 16))
        return ripe_fail(RIPE_ERR_UNSUPPORTED, "%d query heads per key/value head: at most %d here", q.G, many ? 128 : 16);
    const int sms = device_sm_count();
    if (sms < 1) return ripe_fail(RIPE_ERR_CUDA, "no current CUDA device");
    if (tc && (int64_t)max_ntok * q.G <= 16) {
        q.kind = Plan::DECODE;
        q.grid = 2 * sms;
        q.slot_rows = (int64_t)max_ntok * q.G <= 8 ? 8 : 16;
        q.tok1 = q.tpt = q.slot_rows / q.G;
    } else if (tc) {
        q.kind = Plan::TC;
        q.grid = sms;
        q.slot_rows = 256;
        q.tok1 = 128 / q.G;
        q.tpt = 2 * q.tok1;
    } else {
        q.kind = Plan::SIMT;
        q.grid = (p->d * (p->dtype == RIPE_BF16 ? 2 : 4) <= 256 ? 4 : 2) * sms;  // what shared memory holds
        q.slot_rows = 16;
        q.tok1 = q.tpt = 16 / q.G;
    }
    const size_t part = ((size_t)q.grid * sizeof(PagedHdr) + 255) / 256 * 256;
    q.bytes = part + (size_t)q.grid * 2 * q.slot_rows * (p->d + 2) * sizeof(float);
    return RIPE_OK;
}

int fill(PagedArgs& a, const ripe_pages_t* p, const ripe_paged_batch_t* b) {
    a.k = (const char*)p->K;
    a.v = (const char*)p->V;
    a.page_stride = p->npages == 1 ? p->d : p->page_stride;
    a.head_stride = p->Hkv == 1 ? p->d : p->head_stride;
    a.pos_stride = p->pos_stride;
    a.table = b->table;
    a.table_stride = b->table_stride;
    a.ctx = b->ctx_len;
    a.row0 = b->row0;
    a.table_width = b->table_width;
    a.nseq = b->nseq;
    a.nrows = b->nrows;
    a.Hkv = p->Hkv;
    a.d = p->d;
    a.page = p->page;
    for (a.page_shift = 4; (1 << a.page_shift) < p->page;) ++a.page_shift;
    a.npages = p->npages;
    a.err = b->err_dev;
    const cudaError_t e = a.err ? cudaSuccess : paged_error_word(&a.err);
    return e == cudaSuccess ? RIPE_OK : ripe_fail(RIPE_ERR_CUDA, "device error word: %s", cudaGetErrorString(e));
}

}  // namespace

extern "C" {

int ripe_paged_append(const ripe_pages_t* pages, const ripe_paged_batch_t* batch, const void* K, const void* V,
                      int64_t row_stride, ripe_stream_t stream) {
    int rc = check_pages(pages);
    if (rc != RIPE_OK || (rc = check_batch(pages, batch)) != RIPE_OK) return rc;
    if (batch->nseq == 0 || batch->nrows == 0) return RIPE_OK;
    const int es = pages->dtype == RIPE_BF16 ? 2 : 4;
    const int64_t least = (int64_t)pages->Hkv * pages->d;
    if ((rc = check_rows(K, row_stride, least, es, "K")) != RIPE_OK) return rc;
    if ((rc = check_rows(V, row_stride, least, es, "V")) != RIPE_OK) return rc;
    PagedArgs a;
    memset(&a, 0, sizeof a);
    if ((rc = fill(a, pages, batch)) != RIPE_OK) return rc;
    a.max_ntok = batch->nrows;
    const cudaError_t e = launch_paged_append(a, (const char*)K, (const char*)V, row_stride, es, (cudaStream_t)stream);
    return e == cudaSuccess ? RIPE_OK : ripe_fail(RIPE_ERR_CUDA, "paged append launch: %s", cudaGetErrorString(e));
}

int ripe_paged_attn_workspace(const ripe_pages_t* pages, int H, int max_ntok, size_t* bytes) {
    int rc = check_pages(pages);
    if (rc != RIPE_OK) return rc;
    if (!bytes) return ripe_fail(RIPE_ERR_INVALID_ARG, "bytes is NULL");
    Plan q;
    if ((rc = make_plan(pages, H, max_ntok, q)) != RIPE_OK) return rc;
    *bytes = q.bytes;
    return RIPE_OK;
}

int ripe_paged_attn(const ripe_pages_t* pages, const ripe_paged_batch_t* batch, int H, const void* Q, int64_t q_stride,
                    int window, int sinks, float scale, void* O, int64_t o_stride, float* lse, void* work,
                    size_t work_bytes, ripe_stream_t stream) {
    int rc = check_pages(pages);
    if (rc != RIPE_OK || (rc = check_batch(pages, batch)) != RIPE_OK) return rc;
    if (window < 0 || sinks < 0) return ripe_fail(RIPE_ERR_INVALID_ARG, "window=%d and sinks=%d must be >= 0", window, sinks);
    if (!(scale >= 0.f) || isinf(scale)) return ripe_fail(RIPE_ERR_INVALID_ARG, "scale must be finite and >= 0");
    if (batch->nseq == 0 || batch->nrows == 0) return RIPE_OK;
    Plan q;
    if ((rc = make_plan(pages, H, batch->max_ntok, q)) != RIPE_OK) return rc;
    const int es = pages->dtype == RIPE_BF16 ? 2 : 4;
    if ((rc = check_rows(Q, q_stride, (int64_t)H * pages->d, es, "Q")) != RIPE_OK) return rc;
    if ((rc = check_rows(O, o_stride, (int64_t)H * pages->d, es, "O")) != RIPE_OK) return rc;
    if (!aligned(lse, 4)) return ripe_fail(RIPE_ERR_UNALIGNED, "lse must be 4-byte aligned");
    if (!work || work_bytes < q.bytes)
        return ripe_fail(RIPE_ERR_CAPACITY, "work holds %zu bytes, the call needs %zu", work ? work_bytes : (size_t)0, q.bytes);
    if (!aligned(work, 256)) return ripe_fail(RIPE_ERR_UNALIGNED, "work must be 256-byte aligned");
    PagedArgs a;
    memset(&a, 0, sizeof a);
    if ((rc = fill(a, pages, batch)) != RIPE_OK) return rc;
    a.q = (const char*)Q;
    a.o = (char*)O;
    a.lse = lse;
    a.q_rs = q_stride;
    a.o_rs = o_stride;
    a.H = H;
    a.G = q.G;
    constexpr int kMost = 1 << 30;  // positions are below it: differences stay within 32 bits
    a.window = window < kMost ? window : kMost;
    a.sinks = sinks < kMost ? sinks : kMost;
    a.max_ntok = batch->max_ntok;
    a.tok1 = q.tok1;
    a.tpt = q.tpt;
    a.slot_rows = q.slot_rows;
    a.scale_log2 = (scale == 0.f ? 1.0f / sqrtf((float)pages->d) : scale) * 1.4426950408889634f;
    char* w = (char*)work;
    a.hdr = (PagedHdr*)w;
    a.part = (float*)(w + q.bytes - (size_t)q.grid * 2 * q.slot_rows * (pages->d + 2) * sizeof(float));
    const cudaStream_t st = (cudaStream_t)stream;
    cudaError_t e = q.kind == Plan::DECODE ? launch_paged_decode(a, q.grid, st)
                    : q.kind == Plan::TC   ? launch_paged_tc(a, q.grid, st)
                                           : launch_paged_simt(a, pages->dtype, q.grid, st);
    if (e == cudaSuccess && q.kind != Plan::TC) e = launch_paged_merge(a, pages->dtype, q.grid, st);
    return e == cudaSuccess ? RIPE_OK : ripe_fail(RIPE_ERR_CUDA, "paged attention launch: %s", cudaGetErrorString(e));
}

int ripe_paged_get_device_error(int32_t* code_host, ripe_stream_t stream) {
    if (!code_host) return ripe_fail(RIPE_ERR_INVALID_ARG, "code_host is NULL");
    const cudaStream_t st = (cudaStream_t)stream;
    int32_t* word = nullptr;
    cudaError_t e = paged_error_word(&word);
    if (e == cudaSuccess) e = cudaMemcpyAsync(code_host, word, sizeof(int32_t), cudaMemcpyDeviceToHost, st);
    if (e == cudaSuccess) e = cudaMemsetAsync(word, 0, sizeof(int32_t), st);
    if (e == cudaSuccess) e = cudaStreamSynchronize(st);
    return e == cudaSuccess ? RIPE_OK : ripe_fail(RIPE_ERR_CUDA, "paged device error: %s", cudaGetErrorString(e));
}

}  // extern "C"
