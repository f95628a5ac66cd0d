// The paged operators' C entry points: checks of arguments, tensor maps and launches.  No
// state is kept but, per device, the address of the error word and the kernels' attributes.
#include "paged.h"

#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdarg>
#include <cstdio>
#include <cstring>
#include <mutex>

namespace dflash {
namespace {

__device__ uint32_t g_paged_err;

constexpr int kMaxDevices = 64;
// (set_up: of the attention kernels, by kind: bf16 + 2 * wide)
struct DeviceInfo {
    bool ready, set_up[4];
    int sms;
    uint32_t *err;
};
std::mutex g_mu;
DeviceInfo g_dev[kMaxDevices];
thread_local char g_msg[512] = "no error";

int fail(int code, const char *fmt, ...) {
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(g_msg, sizeof g_msg, fmt, ap);
    va_end(ap);
    return code;
}

// Once per device, with it current; later calls only look.
int device_info(const char *who, DeviceInfo *out) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess || dev < 0 || dev >= kMaxDevices)
        return fail(RING_ECUDA, "%s: cudaGetDevice: %s", who, cudaGetErrorString(e));
    std::lock_guard<std::mutex> lock(g_mu);
    DeviceInfo &d = g_dev[dev];
    if (!d.ready) {
        void *p = nullptr;
        e = cudaGetSymbolAddress(&p, g_paged_err);
        if (e == cudaSuccess) e = cudaDeviceGetAttribute(&d.sms, cudaDevAttrMultiProcessorCount, dev);
        if (e != cudaSuccess) return fail(RING_ECUDA, "%s: set-up: %s", who, cudaGetErrorString(e));
        d.err = static_cast<uint32_t *>(p);
        d.ready = true;
    }
    *out = d;
    return RING_OK;
}

// The kernels of a kind, once per device and when first called for: one that a device cannot run fails the
// calls that want it and no others.
int set_up_attend(const char *who, int kind) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess || dev < 0 || dev >= kMaxDevices)
        return fail(RING_ECUDA, "%s: cudaGetDevice: %s", who, cudaGetErrorString(e));
    std::lock_guard<std::mutex> lock(g_mu);
    switch (kind) {
    case 0: e = paged_attend_setup_t<PAGED_F16>(); break;
    case 1: e = paged_attend_setup_t<PAGED_BF16>(); break;
    case 2: e = paged_prefill_setup_t<PAGED_F16>(); break;
    default: e = paged_prefill_setup_t<PAGED_BF16>(); break;
    }
    if (e != cudaSuccess) return fail(RING_ECUDA, "%s: set-up: %s", who, cudaGetErrorString(e));
    g_dev[dev].set_up[kind] = true;
    return RING_OK;
}

using EncodeTiled = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                                 const cuuint64_t *, const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave,
                                 CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiled encode_fn() {
    static const EncodeTiled fn = [] {
        void *p = nullptr;
        cudaDriverEntryPointQueryResult st;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &st) !=
                cudaSuccess ||
            st != cudaDriverEntryPointSuccess)
            p = nullptr;
        return reinterpret_cast<EncodeTiled>(p);
    }();
    return fn;
}

bool is16(int t) { return t == PAGED_F16 || t == PAGED_BF16; }
bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

// rows tensors: given (where there are rows: an empty tensor may have no address), 16-byte alignment
// of every head, and strides that say something where there is more than one of a kind
bool rows_ok(const void *p, int64_t rs, int64_t hs, int esize, int64_t n_rows, int heads) {
    return (p || n_rows == 0) && aligned16(p) && (rs * esize) % 16 == 0 && (hs * esize) % 16 == 0 && rs >= (n_rows > 1) && hs >= (heads > 1) &&
           rs < (int64_t)1 << 38 && hs < (int64_t)1 << 38;
}

// an output that is its input's tensor has its strides (a head's lanes read it whole before they write)
bool in_place_ok(const void *in, const void *out, int64_t rs, int64_t hs, int64_t ors, int64_t ohs, int64_t n_rows, int heads) {
    return in != out || n_rows == 0 || ((n_rows == 1 || rs == ors) && (heads <= 1 || hs == ohs));
}

int check_cache(const char *who, const paged_cache *c) {
    if (!c) return fail(RING_EINVAL, "%s: cache is NULL", who);
    if (!is16(c->format) && c->format != PAGED_INT8 && c->format != PAGED_E4M3)
        return fail(RING_EINVAL, "%s: unknown page format %d", who, c->format);
    if (c->head_dim != 64 && c->head_dim != 128)
        return fail(RING_EINVAL, "%s: head_dim %d (64 or 128)", who, c->head_dim);
    if (c->page_size < 16 || c->page_size > 256 || (c->page_size & (c->page_size - 1)))
        return fail(RING_EINVAL, "%s: page_size %d (16, 32, 64, 128 or 256)", who, c->page_size);
    if (c->n_pages <= 0 || c->n_head_kv <= 0) return fail(RING_EINVAL, "%s: the cache is empty", who);
    if (c->n_head_kv > 65536) return fail(RING_EINVAL, "%s: more than 65536 kv heads", who);
    if (!c->k || !c->v || !aligned16(c->k) || !aligned16(c->v))
        return fail(RING_EINVAL, "%s: pools must be given and 16-byte aligned", who);
    const int es = is16(c->format) ? 2 : 1;
    const int64_t st[3] = {c->page_stride, c->head_stride, c->row_stride};
    for (int64_t s : st)
        if (s <= 0 || (s * es) % 16 || s * es >= (int64_t)1 << 40)
            return fail(RING_EINVAL, "%s: pool strides must be positive multiples of 16 bytes", who);
    if (!is16(c->format)) {
        if (!c->k_scale || !c->v_scale || !aligned16(c->k_scale) || !aligned16(c->v_scale))
            return fail(RING_EINVAL, "%s: quantised pages need 16-byte aligned scales", who);
        if (c->scale_page_stride <= 0 || c->scale_head_stride <= 0 || c->scale_page_stride % 4 || c->scale_head_stride % 4)
            return fail(RING_EINVAL, "%s: scale strides must be positive multiples of 4", who);
    }
    return RING_OK;
}

int check_batch(const char *who, const paged_cache *c, const paged_batch *b, int64_t n_rows) {
    if (!b) return fail(RING_EINVAL, "%s: batch is NULL", who);
    if (b->n_seq < 0 || b->max_pages < 0 || b->max_q < 0 || b->max_kv < 0 || b->pages_stride < 0)
        return fail(RING_EINVAL, "%s: negative batch dimension", who);
    if (n_rows < 0 || n_rows > INT32_MAX / 2) return fail(RING_EINVAL, "%s: n_rows out of range", who);
    if (b->max_q > INT32_MAX / 2) return fail(RING_EINVAL, "%s: max_q out of range", who);
    if (b->n_seq > 0 && (!b->q_start || !b->kv_len || (!b->pages && b->max_pages)))
        return fail(RING_EINVAL, "%s: NULL batch array", who);
    if (b->n_seq > 65536) return fail(RING_EINVAL, "%s: more than 65536 sequences", who);
    const int64_t cap = (int64_t)b->max_pages * c->page_size;
    if (cap > INT32_MAX / 2) return fail(RING_EINVAL, "%s: block table spans more than 2^30 positions", who);
    if (b->max_kv > cap) return fail(RING_EINVAL, "%s: max_kv %d above the block table's %lld positions", who, b->max_kv,
                                     (long long)cap);
    return RING_OK;
}

int check_rope(const char *who, const paged_rope *r, int head_dim) {
    if (!r) return RING_OK;
    if (r->rotary_dim <= 0 || r->rotary_dim % 16 || r->rotary_dim > head_dim)
        return fail(RING_EINVAL, "%s: rotary_dim %d (a multiple of 16 up to head_dim)", who, r->rotary_dim);
    if ((r->layout != PAGED_HALF && r->layout != PAGED_INTERLEAVED) || !std::isfinite(r->magnitude))
        return fail(RING_EINVAL, "%s: the rotation is not paged_rope_init's", who);
    return RING_OK;
}

// inv_freq / 2 pi modulo one turn, in 2^-64: the product with a two-part 1 / 2 pi, whose second
// part is what double precision leaves of it
uint64_t turns_of(double f) {
    const double hi_c = 0.15915494309189535, lo_c = -9.839338337591243e-18;
    const double p = f * hi_c;
    const double rest = std::fma(f, hi_c, -p) + f * lo_c;
    const double frac = p - std::floor(p);
    // 2^64 * frac in two halves, each exact in double
    const double top = std::floor(std::ldexp(frac, 32));
    const double low = std::ldexp(frac, 64) - std::ldexp(top, 32);
    return ((uint64_t)top << 32) + (uint64_t)low + (uint64_t)(int64_t)std::llrint(std::ldexp(rest, 64));
}

void set_rope(PagedRowsArgs &a, const paged_rope *r) {
    a.rot = r ? r->rotary_dim : 0;
    a.layout = r ? r->layout : 0;
    a.magnitude = r ? r->magnitude : 1.f;
    if (r) std::memcpy(a.turn, r->turns, sizeof(uint64_t) * (r->rotary_dim / 2));
}

PagedPool pool_of(const paged_cache *c) {
    PagedPool p{};
    p.k = static_cast<uint8_t *>(c->k);
    p.v = static_cast<uint8_t *>(c->v);
    p.ks = c->k_scale;
    p.vs = c->v_scale;
    p.page_stride = c->page_stride;
    p.head_stride = c->head_stride;
    p.row_stride = c->row_stride;
    p.s_page_stride = c->scale_page_stride;
    p.s_head_stride = c->scale_head_stride;
    p.n_pages = c->n_pages;
    p.page_shift = __builtin_ctz((unsigned)c->page_size);
    p.n_head_kv = c->n_head_kv;
    p.format = c->format;
    return p;
}

PagedBatchDev batch_of(const paged_batch *b, int64_t n_rows) {
    PagedBatchDev d{};
    d.q_start = b->q_start;
    d.kv_len = b->kv_len;
    d.pages = b->pages;
    d.pages_stride = b->pages_stride;
    d.n_rows = n_rows;
    d.n_seq = b->n_seq;
    d.max_pages = b->max_pages;
    return d;
}

// K or V pools as [n_pages][n_head_kv][page_size][head_dim] boxes of up to 128 bytes by
// `rows` tokens of one head and page
bool encode_pool(CUtensorMap *tm, const paged_cache *c, void *base, int rows) {
    const EncodeTiled fn = encode_fn();
    if (!fn) return false;
    const int es = is16(c->format) ? 2 : 1;
    const int inner = std::min(c->head_dim, 128 / es);
    cuuint64_t dims[4] = {(cuuint64_t)c->head_dim, (cuuint64_t)c->page_size, (cuuint64_t)c->n_head_kv,
                          (cuuint64_t)c->n_pages};
    cuuint64_t strides[3] = {(cuuint64_t)(c->row_stride * es), (cuuint64_t)(c->head_stride * es),
                             (cuuint64_t)(c->page_stride * es)};
    cuuint32_t box[4] = {(cuuint32_t)inner, (cuuint32_t)std::min(rows, c->page_size), 1, 1};
    cuuint32_t unit[4] = {1, 1, 1, 1};
    return fn(tm, es == 2 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_UINT8, 4, base, dims, strides, box,
              unit, CU_TENSOR_MAP_INTERLEAVE_NONE, inner * es == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
              CU_TENSOR_MAP_L2_PROMOTION_L2_128B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Queries as [n_rows][n_head][head_dim], boxes of 64 values by the heads of one kv head by tokens
bool encode_queries(CUtensorMap *tm, const paged_attend_args *g, int head_dim, int group, int tokens) {
    const EncodeTiled fn = encode_fn();
    if (!fn) return false;
    // a stride of a dimension of one entry is never walked, but has to be one
    const int64_t hs = g->n_head > 1 ? g->q_head_stride : head_dim;
    const int64_t rs = g->n_rows > 1 ? g->q_row_stride : (int64_t)head_dim * g->n_head;
    cuuint64_t dims[3] = {(cuuint64_t)head_dim, (cuuint64_t)g->n_head, (cuuint64_t)g->n_rows};
    cuuint64_t strides[2] = {(cuuint64_t)hs * 2, (cuuint64_t)rs * 2};
    cuuint32_t box[3] = {64, (cuuint32_t)group, (cuuint32_t)tokens};
    cuuint32_t unit[3] = {1, 1, 1};
    return fn(tm, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3, const_cast<void *>(g->q), dims, strides, box, unit,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Which kernel serves a batch, its rows per item and its CTAs: what the workspace and the launch
// go by.  The streaming kernel up to a number of query rows per kv head, the tensor-core one above it,
// whose items are one or two blocks of as many whole tokens as 128 rows take.
// The border, measured on 64 sequences of up to 1,024 / 16,384 tokens, 8 kv heads of 128 (us):
//   bf16 pages  16 rows: streaming 54 / 367, tensor-core 63 / 373;  32 rows: 69 / 382 and 62 / 371
//   int8 pages  16 rows: streaming 47 / 291, tensor-core 75 / 416;  32 rows: 70 / 454 and 74 / 415
//   (e4m3, bf16 queries, 32 rows: 66 / 401 and 73 / 400)
// so 16 rows over 16-bit pages and 32 over quantised ones, more than the streaming kernel has.
// No more CTAs than the bounds leave work for.
struct AttendPlan {
    int rows, tokens, ctas, min_tiles, item_cost;
    bool wide;
};
AttendPlan plan_of(const paged_cache *c, const paged_batch *b, int group, int sms) {
    const int64_t rows = (int64_t)b->max_q * group;
    AttendPlan p{};
    p.wide = rows > (is16(c->format) ? 16 : 32);
    const int block = 128 / group;                                 // whole tokens of a tensor-core block
    p.rows = p.wide ? (b->max_q <= block ? 1 : 2) * block * group : (rows <= 16 ? 16 : 32);
    p.tokens = p.wide ? p.rows / group : std::max(1, b->max_q);
    // What an item's beginning and end cost, in tiles: without it a share of many short items takes
    // longer than one of as many tiles of a long item.  Tensor-core kernel: two prompts of 4,097 tokens 248
    // us at 0, 214 at 2 and 3; int8 trees 130 us at 2, 126 at 3, 127 at 4 (123 at 3 now).  Streaming kernel, 64 sequences of up to 1,024 / 16,384 tokens, int8, 4 tokens
    // each: 94 / 321 us at 0, 56 / 292 at 4, 53 / 286 at 6, 53 / 288 at 8; bf16 85 / 370 and 54 / 367 at 6.
    p.item_cost = p.wide ? 3 : 6;
    // (fewest units of a share; one token over 1,024 positions: 16 us with 2, 22 with 2 + item_cost)
    p.min_tiles = 2;
    const int64_t keys = b->max_kv > 0 ? b->max_kv : (int64_t)b->max_pages * c->page_size;
    const int64_t tiles = keys / (p.wide ? 128 : 64) + 2 + p.item_cost;   // of an item, wherever it begins
    const int64_t items = (int64_t)b->n_seq * c->n_head_kv * ((b->max_q + p.tokens - 1) / p.tokens);
    // an item has min_tiles units or more
    const int64_t fit = p.wide ? sms : 2 * sms;
    const int64_t most = items >= fit ? fit : (items * tiles + p.min_tiles - 1) / p.min_tiles;
    p.ctas = (int)std::max<int64_t>(1, std::min(most, fit));
    return p;
}

int64_t up256(int64_t x) { return (x + 255) & ~(int64_t)255; }

int64_t workspace_of(const AttendPlan &p, int head_dim) {
    const int64_t parts = (int64_t)p.ctas * 2 * p.rows;
    return up256(parts * head_dim * 4) + up256(parts * 8) + up256((int64_t)p.ctas * 16);
}

int check_heads(const char *who, const paged_cache *c, int n_head) {
    if (n_head <= 0 || n_head % c->n_head_kv || n_head / c->n_head_kv > kPagedMaxGroup)
        return fail(RING_EINVAL, "%s: n_head %d (a multiple of n_head_kv %d, up to %d times)", who, n_head, c->n_head_kv,
                    kPagedMaxGroup);
    return RING_OK;
}

}  // namespace
}  // namespace dflash

using namespace dflash;

#define TRY(x)                         \
    do {                               \
        const int rc_ = (x);           \
        if (rc_ != RING_OK) return rc_; \
    } while (0)

extern "C" int paged_rope_init(paged_rope *r, const double *inv_freq, double magnitude, int32_t rotary_dim, int32_t layout) {
    static const char *who = "paged_rope_init";
    if (!r || !inv_freq) return fail(RING_EINVAL, "%s: NULL argument", who);
    paged_rope x{};
    x.magnitude = (float)magnitude;
    x.rotary_dim = rotary_dim;
    x.layout = layout;
    TRY(check_rope(who, &x, kPagedMaxDim));
    for (int i = 0; i < rotary_dim / 2; ++i) {
        if (!(inv_freq[i] >= 0.0) || !(inv_freq[i] < 1e6)) return fail(RING_EINVAL, "%s: inv_freq[%d] out of range", who, i);
        x.turns[i] = turns_of(inv_freq[i]);
    }
    *r = x;
    return RING_OK;
}

extern "C" int paged_norm_rope(const paged_norm_rope_args *g, void *stream) {
    static const char *who = "paged_norm_rope";
    if (!g) return fail(RING_EINVAL, "%s: args is NULL", who);
    if (!is16(g->dtype) && g->dtype != PAGED_F32) return fail(RING_EINVAL, "%s: unknown type %d", who, g->dtype);
    if (g->head_dim != 64 && g->head_dim != 128) return fail(RING_EINVAL, "%s: head_dim %d (64 or 128)", who, g->head_dim);
    if (g->n_rows < 0 || g->n_rows > INT32_MAX / 2 || g->n_head_q < 0 || g->n_head_k < 0 || g->n_head_q > 65536 ||
        g->n_head_k > 65536)
        return fail(RING_EINVAL, "%s: dimension out of range", who);
    if (!(g->eps >= 0.f)) return fail(RING_EINVAL, "%s: eps must not be negative", who);
    TRY(check_rope(who, g->rope, g->head_dim));
    const int es = g->dtype == PAGED_F32 ? 4 : 2;
    if (g->n_head_q && (!rows_ok(g->q, g->q_row_stride, g->q_head_stride, es, g->n_rows, g->n_head_q) ||
                        !rows_ok(g->q_out, g->qo_row_stride, g->qo_head_stride, es, g->n_rows, g->n_head_q)))
        return fail(RING_EINVAL, "%s: q and q_out must be given with every head 16-byte aligned", who);
    if (g->n_head_k && (!rows_ok(g->k, g->k_row_stride, g->k_head_stride, es, g->n_rows, g->n_head_k) ||
                        !rows_ok(g->k_out, g->ko_row_stride, g->ko_head_stride, es, g->n_rows, g->n_head_k)))
        return fail(RING_EINVAL, "%s: k and k_out must be given with every head 16-byte aligned", who);
    if ((g->n_head_q && !in_place_ok(g->q, g->q_out, g->q_row_stride, g->q_head_stride, g->qo_row_stride, g->qo_head_stride,
                                     g->n_rows, g->n_head_q)) ||
        (g->n_head_k && !in_place_ok(g->k, g->k_out, g->k_row_stride, g->k_head_stride, g->ko_row_stride, g->ko_head_stride,
                                     g->n_rows, g->n_head_k)))
        return fail(RING_EINVAL, "%s: an output in its input's place must have its strides", who);
    if ((g->q_norm && !aligned16(g->q_norm)) || (g->k_norm && !aligned16(g->k_norm)))
        return fail(RING_EINVAL, "%s: norm weights must be 16-byte aligned", who);
    if (g->rope && !g->positions && g->n_rows) return fail(RING_EINVAL, "%s: a rotation needs positions", who);
    if (g->n_rows == 0 || g->n_head_q + g->n_head_k == 0) return RING_OK;
    DeviceInfo d;
    TRY(device_info(who, &d));
    PagedRowsArgs a{};
    a.q = g->q;
    a.k = g->k;
    a.qo = g->q_out;
    a.ko = g->k_out;
    a.q_rs = g->q_row_stride; a.q_hs = g->q_head_stride;
    a.k_rs = g->k_row_stride; a.k_hs = g->k_head_stride;
    a.qo_rs = g->qo_row_stride; a.qo_hs = g->qo_head_stride;
    a.ko_rs = g->ko_row_stride; a.ko_hs = g->ko_head_stride;
    a.q_norm = g->q_norm;
    a.k_norm = g->k_norm;
    a.positions = g->positions;
    a.err = d.err;
    a.n_rows = g->n_rows;
    a.eps = g->eps;
    a.nq = g->n_head_q;
    a.nk = g->n_head_k;
    set_rope(a, g->rope);
    const cudaError_t e = launch_paged_rows(a, g->dtype, g->head_dim, false, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? RING_OK : fail(RING_ECUDA, "%s: launch: %s", who, cudaGetErrorString(e));
}

extern "C" int paged_append(const paged_append_args *g, void *stream) {
    static const char *who = "paged_append";
    if (!g) return fail(RING_EINVAL, "%s: args is NULL", who);
    TRY(check_cache(who, g->cache));
    TRY(check_batch(who, g->cache, g->batch, g->n_rows));
    if (!is16(g->dtype)) return fail(RING_EINVAL, "%s: rows must be F16 or BF16", who);
    if (is16(g->cache->format) && g->cache->format != g->dtype)
        return fail(RING_EINVAL, "%s: rows and 16-bit pages must have one type", who);
    if (g->n_head_q < 0 || g->n_head_q > 65536) return fail(RING_EINVAL, "%s: n_head_q out of range", who);
    if (!(g->eps >= 0.f)) return fail(RING_EINVAL, "%s: eps must not be negative", who);
    TRY(check_rope(who, g->rope, g->cache->head_dim));
    if (!rows_ok(g->k, g->k_row_stride, g->k_head_stride, 2, g->n_rows, g->cache->n_head_kv) ||
        !rows_ok(g->v, g->v_row_stride, g->v_head_stride, 2, g->n_rows, g->cache->n_head_kv))
        return fail(RING_EINVAL, "%s: k and v must be given with every head 16-byte aligned", who);
    if (g->n_head_q && (!rows_ok(g->q, g->q_row_stride, g->q_head_stride, 2, g->n_rows, g->n_head_q) ||
                        !rows_ok(g->q_out, g->qo_row_stride, g->qo_head_stride, 2, g->n_rows, g->n_head_q)))
        return fail(RING_EINVAL, "%s: q and q_out must be given with every head 16-byte aligned", who);
    if (g->n_head_q && !in_place_ok(g->q, g->q_out, g->q_row_stride, g->q_head_stride, g->qo_row_stride, g->qo_head_stride,
                                    g->n_rows, g->n_head_q))
        return fail(RING_EINVAL, "%s: an output in its input's place must have its strides", who);
    if ((g->q_norm && !aligned16(g->q_norm)) || (g->k_norm && !aligned16(g->k_norm)))
        return fail(RING_EINVAL, "%s: norm weights must be 16-byte aligned", who);
    if (g->n_rows == 0 || g->batch->n_seq == 0) return RING_OK;
    DeviceInfo d;
    TRY(device_info(who, &d));
    PagedRowsArgs a{};
    a.q = g->q;
    a.k = g->k;
    a.v = g->v;
    a.qo = g->q_out;
    a.q_rs = g->q_row_stride; a.q_hs = g->q_head_stride;
    a.k_rs = g->k_row_stride; a.k_hs = g->k_head_stride;
    a.v_rs = g->v_row_stride; a.v_hs = g->v_head_stride;
    a.qo_rs = g->qo_row_stride; a.qo_hs = g->qo_head_stride;
    a.q_norm = g->q_norm;
    a.k_norm = g->k_norm;
    a.positions = g->positions;
    a.pool = pool_of(g->cache);
    a.batch = batch_of(g->batch, g->n_rows);
    a.err = d.err;
    a.n_rows = g->n_rows;
    a.eps = g->eps;
    a.nq = g->n_head_q;
    a.nk = a.nv = g->cache->n_head_kv;
    set_rope(a, g->rope);
    const cudaError_t e = launch_paged_rows(a, g->dtype, g->cache->head_dim, true, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? RING_OK : fail(RING_ECUDA, "%s: launch: %s", who, cudaGetErrorString(e));
}

extern "C" int paged_gather(const paged_gather_args *g, void *stream) {
    static const char *who = "paged_gather";
    if (!g) return fail(RING_EINVAL, "%s: args is NULL", who);
    TRY(check_cache(who, g->cache));
    TRY(check_batch(who, g->cache, g->batch, g->n_rows));
    if (!is16(g->dtype)) return fail(RING_EINVAL, "%s: rows must be F16 or BF16", who);
    if (is16(g->cache->format) && g->cache->format != g->dtype)
        return fail(RING_EINVAL, "%s: rows and 16-bit pages must have one type", who);
    if (!rows_ok(g->k, g->k_row_stride, g->k_head_stride, 2, g->n_rows, g->cache->n_head_kv) ||
        !rows_ok(g->v, g->v_row_stride, g->v_head_stride, 2, g->n_rows, g->cache->n_head_kv))
        return fail(RING_EINVAL, "%s: k and v must be given with every head 16-byte aligned", who);
    if (g->n_rows == 0 || g->batch->n_seq == 0) return RING_OK;
    DeviceInfo d;
    TRY(device_info(who, &d));
    PagedGatherArgs a{};
    a.k = g->k;
    a.v = g->v;
    a.k_rs = g->k_row_stride; a.k_hs = g->k_head_stride;
    a.v_rs = g->v_row_stride; a.v_hs = g->v_head_stride;
    a.pool = pool_of(g->cache);
    a.batch = batch_of(g->batch, g->n_rows);
    a.err = d.err;
    const cudaError_t e = launch_paged_gather(a, g->dtype, g->cache->head_dim, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? RING_OK : fail(RING_ECUDA, "%s: launch: %s", who, cudaGetErrorString(e));
}

// Of each of two passes: the states of its items that are not cut, where its items' states are, and a word.
static int64_t level_bytes(const paged_cache *c, int64_t n_rows, int n_head) {
    return up256(n_rows * n_head * c->head_dim * 4) + up256(n_rows * n_head * 8) + up256(n_rows * c->n_head_kv * 8) +
           up256(4);
}

extern "C" int paged_attend_workspace(const paged_cache *cache, const paged_batch *batch, int32_t n_head, int64_t *bytes) {
    static const char *who = "paged_attend_workspace";
    if (!bytes) return fail(RING_EINVAL, "%s: bytes is NULL", who);
    TRY(check_cache(who, cache));
    TRY(check_batch(who, cache, batch, 0));
    TRY(check_heads(who, cache, n_head));
    DeviceInfo d;
    TRY(device_info(who, &d));
    *bytes = workspace_of(plan_of(cache, batch, n_head / cache->n_head_kv, d.sms), cache->head_dim);
    return RING_OK;
}

extern "C" int paged_attend_shared_workspace(const paged_cache *cache, const paged_batch *batch, const paged_batch *prefix,
                                             int64_t n_rows, int32_t n_head, int64_t *bytes) {
    static const char *who = "paged_attend_shared_workspace";
    if (!bytes) return fail(RING_EINVAL, "%s: bytes is NULL", who);
    TRY(check_cache(who, cache));
    TRY(check_batch(who, cache, batch, n_rows));
    TRY(check_batch(who, cache, prefix, n_rows));
    TRY(check_heads(who, cache, n_head));
    DeviceInfo d;
    TRY(device_info(who, &d));
    const int group = n_head / cache->n_head_kv;
    *bytes = 2 * level_bytes(cache, n_rows, n_head) + workspace_of(plan_of(cache, batch, group, d.sms), cache->head_dim) +
             workspace_of(plan_of(cache, prefix, group, d.sms), cache->head_dim);
    return RING_OK;
}

// One pass: what the kernels take of it, and its launch.  a: as filled from the call.
static int attend_pass(const char *who, const paged_attend_args *g, const paged_batch *b, const AttendPlan &p, PagedAttendArgs &a,
                       uint8_t *ws, cudaStream_t st) {
    const int64_t parts = (int64_t)p.ctas * 2 * p.rows;
    const int dim = g->cache->head_dim;
    a.batch = batch_of(b, g->n_rows);
    a.part_acc = reinterpret_cast<float *>(ws);
    ws += up256(parts * dim * 4);
    a.part_ml = reinterpret_cast<float2 *>(ws);
    ws += up256(parts * 8);
    a.desc = reinterpret_cast<int4 *>(ws);
    if (a.level != kOnly) {
        ws += up256((int64_t)p.ctas * 16);
        a.level_acc = reinterpret_cast<float *>(ws);
        ws += up256(g->n_rows * g->n_head * dim * 4);
        a.level_ml = reinterpret_cast<float2 *>(ws);
        ws += up256(g->n_rows * g->n_head * 8);
        a.level_items = reinterpret_cast<int2 *>(ws);
        ws += up256(g->n_rows * g->cache->n_head_kv * 8);
        a.level_broken = reinterpret_cast<int *>(ws);
    }
    a.max_q = b->max_q;
    a.ctas = p.ctas;
    a.min_tiles = p.min_tiles;
    a.item_cost = p.item_cost;
    a.tile_tokens = p.tokens;
    a.tile_rows = p.rows;
    CUtensorMap tk, tv, tq;
    const int box = p.wide ? 128 : 64;
    if (!encode_pool(&tk, g->cache, g->cache->k, box) || !encode_pool(&tv, g->cache, g->cache->v, box) ||
        (p.wide && !encode_queries(&tq, g, dim, a.group, 128 / a.group)))
        return fail(RING_ECUDA, "%s: cuTensorMapEncodeTiled failed", who);
    const bool f16 = g->dtype == PAGED_F16;
    const cudaError_t e = p.wide ? (f16 ? launch_paged_prefill_t<PAGED_F16>(a, tk, tv, tq, dim, st)
                                        : launch_paged_prefill_t<PAGED_BF16>(a, tk, tv, tq, dim, st))
                                 : (f16 ? launch_paged_attend_t<PAGED_F16>(a, tk, tv, dim, st)
                                        : launch_paged_attend_t<PAGED_BF16>(a, tk, tv, dim, st));
    return e == cudaSuccess ? RING_OK : fail(RING_ECUDA, "%s: launch: %s", who, cudaGetErrorString(e));
}

// prefix: NULL, or what paged_attend_shared has beside the arguments.
static int attend(const char *who, const paged_attend_args *g, const paged_batch *prefix, void *stream) {
    TRY(check_cache(who, g->cache));
    TRY(check_batch(who, g->cache, g->batch, g->n_rows));
    if (prefix) TRY(check_batch(who, g->cache, prefix, g->n_rows));
    TRY(check_heads(who, g->cache, g->n_head));
    if (!is16(g->dtype)) return fail(RING_EINVAL, "%s: q and o must be F16 or BF16", who);
    if (is16(g->cache->format) && g->cache->format != g->dtype)
        return fail(RING_EINVAL, "%s: queries and 16-bit pages must have one type", who);
    if (g->mask != PAGED_CAUSAL && g->mask != PAGED_FULL && g->mask != PAGED_TREE)
        return fail(RING_EINVAL, "%s: unknown mask %d", who, g->mask);
    if ((g->mask == PAGED_TREE) != (g->tree != nullptr))
        return fail(RING_EINVAL, "%s: tree words go with the tree mask", who);
    if (g->mask == PAGED_TREE && g->batch->max_q > 64)
        return fail(RING_EINVAL, "%s: a token tree has at most 64 nodes, max_q is %d", who, g->batch->max_q);
    if (g->window < 0) return fail(RING_EINVAL, "%s: negative window", who);
    if (prefix && g->window) return fail(RING_EINVAL, "%s: no windows over shared beginnings", who);
    // (in log2 units it has to be finite too)
    if (!(g->scale >= 0.f) || !std::isfinite(g->scale * 1.5f)) return fail(RING_EINVAL, "%s: scale must be finite and not negative", who);
    if (!rows_ok(g->q, g->q_row_stride, g->q_head_stride, 2, g->n_rows, g->n_head) ||
        !rows_ok(g->o, g->o_row_stride, g->o_head_stride, 2, g->n_rows, g->n_head))
        return fail(RING_EINVAL, "%s: q and o must be given with every head 16-byte aligned", who);
    if (g->q == g->o && g->n_rows > 0) return fail(RING_EINVAL, "%s: o may not be q", who);
    if (g->n_rows == 0 || g->batch->n_seq == 0 || g->batch->max_q == 0) return RING_OK;
    DeviceInfo d;
    TRY(device_info(who, &d));
    const int group = g->n_head / g->cache->n_head_kv, dim = g->cache->head_dim;
    const AttendPlan p = plan_of(g->cache, g->batch, group, d.sms);
    const AttendPlan pp = prefix ? plan_of(g->cache, prefix, group, d.sms) : p;
    for (const AttendPlan *x : {&p, &pp}) {
        const int kind = (g->dtype == PAGED_BF16) + 2 * x->wide;
        if (!d.set_up[kind]) TRY(set_up_attend(who, kind));
        d.set_up[kind] = true;
    }
    const int64_t level = prefix ? level_bytes(g->cache, g->n_rows, g->n_head) : 0, first = workspace_of(pp, dim) + level;
    const int64_t need = workspace_of(p, dim) + level + (prefix ? first : 0);
    if (!g->workspace || (reinterpret_cast<uintptr_t>(g->workspace) & 255) || g->workspace_bytes < need)
        return fail(RING_EINVAL, "%s: needs %lld bytes of 256-byte aligned workspace", who, (long long)need);
    PagedAttendArgs a{};
    a.q = static_cast<const uint16_t *>(g->q);
    a.o = static_cast<uint16_t *>(g->o);
    a.lse = g->lse;
    a.tree = g->tree;
    a.q_rs = g->q_row_stride; a.q_hs = g->q_head_stride;
    a.o_rs = g->o_row_stride; a.o_hs = g->o_head_stride;
    a.pool = pool_of(g->cache);
    a.err = d.err;
    a.n_head = g->n_head;
    a.group = group;
    a.mask = g->mask;
    // one that reaches back past any position is none (and sums of positions and windows stay in 32 bits)
    a.window = g->window > INT32_MAX / 2 ? 0 : g->window;
    const double scale = g->scale > 0.f ? (double)g->scale : 1.0 / std::sqrt((double)dim);
    a.scale_log2 = (float)(scale * 1.4426950408889634);
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    uint8_t *ws = static_cast<uint8_t *>(g->workspace);
    if (!prefix || prefix->n_seq == 0) return attend_pass(who, g, g->batch, p, a, ws, st);
    PagedAttendArgs b = a;
    b.level = kPrefix;
    b.mask = PAGED_FULL;
    a.level = kOwn;
    TRY(attend_pass(who, g, prefix, pp, b, ws, st));
    a.first = &b;
    a.sms = d.sms;
    return attend_pass(who, g, g->batch, p, a, ws + first, st);
}

extern "C" int paged_attend(const paged_attend_args *g, void *stream) {
    static const char *who = "paged_attend";
    if (!g) return fail(RING_EINVAL, "%s: args is NULL", who);
    return attend(who, g, nullptr, stream);
}

extern "C" int paged_attend_shared(const paged_attend_args *g, const paged_batch *prefix, void *stream) {
    static const char *who = "paged_attend_shared";
    if (!g) return fail(RING_EINVAL, "%s: args is NULL", who);
    if (!prefix) return fail(RING_EINVAL, "%s: prefix is NULL", who);
    return attend(who, g, prefix, stream);
}

extern "C" int paged_device_error(uint32_t *bits) {
    static const char *who = "paged_device_error";
    DeviceInfo d;
    TRY(device_info(who, &d));
    uint32_t w = 0;
    cudaError_t e = cudaDeviceSynchronize();
    if (e == cudaSuccess) e = cudaMemcpy(&w, d.err, 4, cudaMemcpyDeviceToHost);
    if (e == cudaSuccess && w) e = cudaMemset(d.err, 0, 4);
    if (e != cudaSuccess) return fail(RING_ECUDA, "%s: %s", who, cudaGetErrorString(e));
    if (bits) *bits = w;
    return w ? fail(RING_EDEVICE, "%s: device error word 0x%x", who, w) : RING_OK;
}

extern "C" const char *paged_last_error(void) { return g_msg; }
