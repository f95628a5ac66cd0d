// The gated delta rule's C entry points: checks of arguments and launches.  No state is kept
// but, per device, the address of the error word.
#include "delta.h"

#include <cmath>
#include <cstdarg>
#include <cstdio>
#include <mutex>

namespace dflash {
namespace {

__device__ uint32_t g_delta_err;

constexpr int kMaxDevices = 64;
struct DeviceInfo {
    bool ready, chunk;                   // chunk: the kernels of many tokens are set up
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
        e = cudaGetSymbolAddress(&p, g_delta_err);
        if (e == cudaSuccess) e = cudaDeviceGetAttribute(&d.sms, cudaDevAttrMultiProcessorCount, dev);
        if (e != cudaSuccess) return fail(RING_ECUDA, "%s: set-up: %s", who, cudaGetErrorString(e));
        d.err = static_cast<uint32_t *>(p);
        d.ready = true;
    }
    *out = d;
    return RING_OK;
}

// The kernels of many tokens, once per device and when first called for.
int set_up_chunk(const char *who) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess) {
        std::lock_guard<std::mutex> lock(g_mu);
        e = delta_chunk_setup();
        if (e == cudaSuccess) g_dev[dev].chunk = true;
    }
    return e == cudaSuccess ? RING_OK : fail(RING_ECUDA, "%s: set-up: %s", who, cudaGetErrorString(e));
}

bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

// rows of 16-bit values: given (where there are rows), 16-byte alignment of every head, and strides
// that say something where there is more than one of a kind
bool rows_ok(const void *p, int64_t rs, int64_t hs, int64_t n_rows, int heads) {
    return (p || n_rows == 0) && aligned16(p) && (rs * 2) % 16 == 0 && (hs * 2) % 16 == 0 && rs >= (n_rows > 1) &&
           hs >= (heads > 1) && rs < (int64_t)1 << 38 && hs < (int64_t)1 << 38;
}

int check_state(const char *who, const delta_state *s) {
    if (!s) return fail(RING_EINVAL, "%s: state is NULL", who);
    if ((s->dim_k != 64 && s->dim_k != 128) || (s->dim_v != 64 && s->dim_v != 128))
        return fail(RING_EINVAL, "%s: state of %d x %d (64 or 128 each)", who, s->dim_v, s->dim_k);
    if (s->n_slots <= 0 || s->n_head <= 0) return fail(RING_EINVAL, "%s: the pool is empty", who);
    if (s->n_head > 65536) return fail(RING_EINVAL, "%s: more than 65536 heads", who);
    if (!s->data || !aligned16(s->data)) return fail(RING_EINVAL, "%s: the pool must be given and 16-byte aligned", who);
    for (int64_t x : {s->slot_stride, s->head_stride})
        if (x <= 0 || x % 4 || x >= (int64_t)1 << 38)
            return fail(RING_EINVAL, "%s: state strides must be positive multiples of 4", who);
    return RING_OK;
}

int check_batch(const char *who, const delta_state *s, const delta_batch *b, int64_t n_rows, int n_head_k) {
    if (!b) return fail(RING_EINVAL, "%s: batch is NULL", who);
    if (b->n_seq < 0 || b->n_seq > 65536 || b->max_q < 0 || b->max_q > INT32_MAX / 2)
        return fail(RING_EINVAL, "%s: batch dimension out of range", who);
    if (b->n_seq > 0 && (!b->q_start || !b->slot_in || !b->slot_out)) return fail(RING_EINVAL, "%s: NULL batch array", who);
    if ((int64_t)b->n_seq * s->n_head > INT32_MAX / 16) return fail(RING_EINVAL, "%s: more than 2^27 sequences times heads", who);
    if (n_rows < 0 || n_rows > INT32_MAX / 2) return fail(RING_EINVAL, "%s: n_rows out of range", who);
    if (n_head_k <= 0 || s->n_head % n_head_k)
        return fail(RING_EINVAL, "%s: %d key heads (a divisor of the %d heads)", who, n_head_k, s->n_head);
    if (delta_chunks(n_rows, b->n_seq) * s->n_head > INT32_MAX)
        return fail(RING_EINVAL, "%s: more than 2^31 chunks of 32 rows times heads", who);
    return RING_OK;
}

int64_t up256(int64_t x) { return (x + 255) & ~(int64_t)255; }

// Which kernels serve a batch: token by token alone where no sequence is longer than kDeltaTokens, and where states are
// kept behind single tokens.
bool by_chunks(const delta_batch *b) { return b->max_q > kDeltaTokens && !b->save; }

int64_t tile_bytes(const delta_state *s, int64_t chunks, int n_head_k) {
    return up256(chunks * n_head_k * 2 * kDeltaChunk * s->dim_k * 2);
}
int64_t workspace_of(const delta_state *s, const delta_batch *b, int64_t n_rows, int n_head_k) {
    if (!by_chunks(b) || b->n_seq == 0) return 0;
    const int64_t chunks = delta_chunks(n_rows, b->n_seq);
    return tile_bytes(s, chunks, n_head_k) + up256(chunks * s->n_head * kDeltaHeadBytes);
}

}  // namespace
}  // namespace dflash

using namespace dflash;

#define TRY(x)                         \
    do {                               \
        const int rc_ = (x);           \
        if (rc_ != RING_OK) return rc_; \
    } while (0)

extern "C" int delta_rule_workspace(const delta_state *state, const delta_batch *batch, int64_t n_rows, int32_t n_head_k,
                                    int64_t *bytes) {
    static const char *who = "delta_rule_workspace";
    if (!bytes) return fail(RING_EINVAL, "%s: bytes is NULL", who);
    TRY(check_state(who, state));
    TRY(check_batch(who, state, batch, n_rows, n_head_k));
    *bytes = workspace_of(state, batch, n_rows, n_head_k);
    return RING_OK;
}

extern "C" int delta_rule(const delta_rule_args *g, void *stream) {
    static const char *who = "delta_rule";
    if (!g) return fail(RING_EINVAL, "%s: args is NULL", who);
    TRY(check_state(who, g->state));
    TRY(check_batch(who, g->state, g->batch, g->n_rows, g->n_head_k));
    const delta_state *s = g->state;
    const delta_batch *b = g->batch;
    if (g->dtype != PAGED_F16 && g->dtype != PAGED_BF16) return fail(RING_EINVAL, "%s: rows must be F16 or BF16", who);
    if (!(g->scale >= 0.f) || !std::isfinite(g->scale)) return fail(RING_EINVAL, "%s: scale must be finite and not negative", who);
    if (!(g->eps >= 0.f) || !std::isfinite(g->eps)) return fail(RING_EINVAL, "%s: eps must be finite and not negative", who);
    if (!rows_ok(g->q, g->q_row_stride, g->q_head_stride, g->n_rows, g->n_head_k) ||
        !rows_ok(g->k, g->k_row_stride, g->k_head_stride, g->n_rows, g->n_head_k) ||
        !rows_ok(g->v, g->v_row_stride, g->v_head_stride, g->n_rows, s->n_head) ||
        !rows_ok(g->o, g->o_row_stride, g->o_head_stride, g->n_rows, s->n_head))
        return fail(RING_EINVAL, "%s: q, k, v and o must be given with every head 16-byte aligned", who);
    if (g->n_rows > 0 && (g->o == g->q || g->o == g->k || g->o == g->v)) return fail(RING_EINVAL, "%s: o may not be an input", who);
    if (g->n_rows > 0 && (!g->g || !g->beta || (reinterpret_cast<uintptr_t>(g->g) & 3) || (reinterpret_cast<uintptr_t>(g->beta) & 3)))
        return fail(RING_EINVAL, "%s: g and beta must be given", who);
    for (int64_t x : {g->g_row_stride, g->beta_row_stride})
        if (x < (g->n_rows > 1) || x >= (int64_t)1 << 38) return fail(RING_EINVAL, "%s: strides of g and beta must be positive", who);
    const int64_t need = workspace_of(s, b, g->n_rows, g->n_head_k);
    if (need > 0 && (!g->workspace || (reinterpret_cast<uintptr_t>(g->workspace) & 255) || g->workspace_bytes < need))
        return fail(RING_EINVAL, "%s: needs %lld bytes of 256-byte aligned workspace", who, (long long)need);
    if (b->n_seq == 0) return RING_OK;
    DeviceInfo d;
    TRY(device_info(who, &d));
    DeltaArgs a{};
    a.q = static_cast<const uint16_t *>(g->q);
    a.k = static_cast<const uint16_t *>(g->k);
    a.v = static_cast<const uint16_t *>(g->v);
    a.o = static_cast<uint16_t *>(g->o);
    a.q_rs = g->q_row_stride; a.q_hs = g->q_head_stride;
    a.k_rs = g->k_row_stride; a.k_hs = g->k_head_stride;
    a.v_rs = g->v_row_stride; a.v_hs = g->v_head_stride;
    a.o_rs = g->o_row_stride; a.o_hs = g->o_head_stride;
    a.g = g->g;
    a.beta = g->beta;
    a.g_rs = g->g_row_stride; a.beta_rs = g->beta_row_stride;
    a.state = s->data;
    a.slot_stride = s->slot_stride; a.head_stride = s->head_stride;
    a.q_start = b->q_start;
    a.slot_in = b->slot_in;
    a.slot_out = b->slot_out;
    a.save = b->save;
    a.err = d.err;
    a.n_rows = g->n_rows;
    a.scale = g->scale > 0.f ? g->scale : (float)(1.0 / std::sqrt((double)s->dim_k));
    a.eps = g->eps;
    a.n_seq = b->n_seq;
    a.max_q = b->max_q;
    a.n_slots = s->n_slots;
    a.n_head = s->n_head;
    a.n_head_k = g->n_head_k;
    a.group = s->n_head / g->n_head_k;
    a.normalise = g->normalise;
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    cudaError_t e;
    if (by_chunks(b)) {
        if (!d.chunk) TRY(set_up_chunk(who));
        a.tiles = static_cast<uint8_t *>(g->workspace);
        a.heads = a.tiles + tile_bytes(s, delta_chunks(g->n_rows, b->n_seq), g->n_head_k);
        // (few tokens are a matter of bytes, what is done before the longer ones' walk is not: side by side)
        a.split = 1;
        e = launch_delta_prep(a, g->dtype, s->dim_k, st);
        if (e == cudaSuccess) e = launch_delta_step(a, g->dtype, s->dim_k, s->dim_v, st);
        if (e == cudaSuccess) e = launch_delta_scan(a, g->dtype, s->dim_k, s->dim_v, d.sms, st);
    } else {
        e = launch_delta_step(a, g->dtype, s->dim_k, s->dim_v, st);
    }
    return e == cudaSuccess ? RING_OK : fail(RING_ECUDA, "%s: launch: %s", who, cudaGetErrorString(e));
}

extern "C" int delta_device_error(uint32_t *bits) {
    static const char *who = "delta_device_error";
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

extern "C" const char *delta_last_error(void) { return g_msg; }
