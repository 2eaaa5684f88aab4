// C ABI of the 8-bit key/value cache: argument checks and launches (layouts and semantics in
// include/qlin.h).  Nothing here allocates or throws.
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>

#include "../../include/qlin.h"
#include "qlin_kv_internal.h"

using namespace qlin;

static_assert(kKvBlock == QLIN_KV_BLOCK, "block size");

static bool aligned(const void* p, size_t n) { return ((uintptr_t)p & (n - 1)) == 0; }

static qlin_status check_cache(const qlin_kv_cache* c, KvView* v) {
  if (!c || !c->codes || !c->scales || !aligned(c->codes, 16) || !aligned(c->scales, 16)) return QLIN_ERR_INVALID_ARG;
  if (c->code != QLIN_KV_INT8 && c->code != QLIN_KV_E4M3) return QLIN_ERR_INVALID_ARG;
  if (c->n_pages < 1 || c->n_heads < 1 || c->head_dim < 1 || c->page_tokens < 1 || c->page_tokens % kKvBlock)
    return QLIN_ERR_INVALID_ARG;
  if (c->head_dim != 64 && c->head_dim != 128) return QLIN_ERR_UNSUPPORTED;
  const int blocks = c->page_tokens / kKvBlock;
  // cells (one block's keys or values) are counted in 32 bits: 2 TB of codes at least
  if ((double)c->n_pages * c->n_heads * 2.0 * blocks >= 2147483648.0) return QLIN_ERR_UNSUPPORTED;
  *v = KvView{(uint8_t*)c->codes, c->scales, c->n_pages, c->n_heads, blocks};
  return QLIN_OK;
}

static qlin_status check_batch(const qlin_kv_cache* c, const qlin_kv_batch* b, void* ws, KvBatch* v) {
  if (!b || !ws || !aligned(ws, 256)) return QLIN_ERR_INVALID_ARG;
  if (b->n_seqs < 0 || b->total_q < 0 || b->max_q < 0 || b->max_kv < 0 || b->pages_width < 0 ||
      b->pages_stride < b->pages_width)
    return QLIN_ERR_INVALID_ARG;
  if (b->n_seqs > kKvMaxSeqs) return QLIN_ERR_UNSUPPORTED;
  if (b->n_seqs > 0 && (!b->q_start || !b->kv_len || !b->pages || !aligned(b->q_start, 4) || !aligned(b->kv_len, 4) ||
                        !aligned(b->pages, 4)))
    return QLIN_ERR_INVALID_ARG;
  *v = KvBatch{b->q_start, b->kv_len,  b->pages, b->pages_stride, b->n_seqs,
               b->total_q, b->max_q,   b->pages_width, c->page_tokens, (int32_t*)ws};
  return QLIN_OK;
}

static bool check_heads(const qlin_heads* h, KvHeads* v) {
  if (!h || !h->data || !aligned(h->data, 16) || h->token_stride < 0 || h->head_stride < 0 || h->token_stride % 8 ||
      h->head_stride % 8)
    return false;
  *v = KvHeads{(const uint16_t*)h->data, h->token_stride, h->head_stride};
  return true;
}

// query heads per key/value head, or 0
static int head_group(const qlin_kv_cache* c, int n_q_heads) {
  if (n_q_heads < 1 || n_q_heads % c->n_heads || n_q_heads > 65536) return 0;
  return n_q_heads / c->n_heads;
}

static int attend_sms() { return std::min(qlin_sm_count(), kMaxSms); }

// status and counters, then the partial results of the two attention kernels
static size_t decode_partials(int head_dim) { return (kv_decode_partial_bytes(head_dim, attend_sms()) + 255) & ~(size_t)255; }
static size_t workspace_bytes(int head_dim) {
  return kKvPartialsOffset + decode_partials(head_dim) + kv_prefill_partial_bytes(head_dim, attend_sms());
}

extern "C" {

qlin_status qlin_kv_workspace_bytes(const qlin_kv_cache* c, size_t* bytes) {
  KvView v;
  if (!bytes) return QLIN_ERR_INVALID_ARG;
  const qlin_status st = check_cache(c, &v);
  if (st != QLIN_OK) return st;
  *bytes = workspace_bytes(c->head_dim);
  return QLIN_OK;
}

qlin_status qlin_kv_init_workspace(void* ws, size_t bytes, qlin_stream stream) {
  if (!ws || !aligned(ws, 256)) return QLIN_ERR_INVALID_ARG;
  if (bytes < kKvPartialsOffset) return QLIN_ERR_WORKSPACE;
  return cudaMemsetAsync(ws, 0, kKvPartialsOffset, (cudaStream_t)stream) == cudaSuccess ? QLIN_OK : QLIN_ERR_CUDA;
}

qlin_status qlin_kv_append(const qlin_kv_cache* c, const qlin_kv_batch* b, const qlin_heads* K, const qlin_heads* V,
                           const qlin_heads* Q, int n_q_heads, void* Q_out, const qlin_rope* rope, void* ws,
                           qlin_stream stream) {
  KvView cv;
  KvBatch bv;
  qlin_status st = check_cache(c, &cv);
  if (st == QLIN_OK) st = check_batch(c, b, ws, &bv);
  if (st != QLIN_OK) return st;
  KvRope r{nullptr, nullptr, 0, 0, 0};
  if (rope && rope->rot_dim != 0) {
    if (rope->rot_dim < 0 || rope->rot_dim % 16 || rope->rot_dim > c->head_dim || rope->n_pos < 1 || !rope->cos ||
        !rope->sin || !aligned(rope->cos, 16) || !aligned(rope->sin, 16))
      return QLIN_ERR_INVALID_ARG;
    r = KvRope{rope->cos, rope->sin, rope->n_pos, rope->rot_dim, rope->interleaved != 0};
  }
  KvHeads kv, vv, qv{nullptr, 0, 0};
  int nq = 0;
  if (bv.n_seqs == 0 || bv.total_q == 0) return QLIN_OK;
  if (!check_heads(K, &kv) || !check_heads(V, &vv)) return QLIN_ERR_INVALID_ARG;
  if (Q) {
    if (!check_heads(Q, &qv) || n_q_heads < 1 || n_q_heads > 65536 || !Q_out || !aligned(Q_out, 16)) return QLIN_ERR_INVALID_ARG;
    nq = n_q_heads;
  }
  return launch_kv_append(c->code, c->head_dim, cv, bv, kv, vv, qv, nq, (uint16_t*)Q_out, r, stream) ? QLIN_ERR_CUDA
                                                                                                   : QLIN_OK;
}

qlin_status qlin_kv_read(const qlin_kv_cache* c, const qlin_kv_batch* b, void* K_out, void* V_out, void* ws,
                         qlin_stream stream) {
  KvView cv;
  KvBatch bv;
  qlin_status st = check_cache(c, &cv);
  if (st == QLIN_OK) st = check_batch(c, b, ws, &bv);
  if (st != QLIN_OK) return st;
  if (bv.n_seqs == 0 || bv.total_q == 0) return QLIN_OK;
  if (!K_out || !V_out || !aligned(K_out, 16) || !aligned(V_out, 16)) return QLIN_ERR_INVALID_ARG;
  return launch_kv_read(c->code, c->head_dim, cv, bv, (uint16_t*)K_out, (uint16_t*)V_out, stream) ? QLIN_ERR_CUDA
                                                                                                : QLIN_OK;
}

qlin_status qlin_kv_attend(const qlin_kv_cache* c, const qlin_kv_batch* b, const qlin_heads* Q, int n_q_heads,
                           float scale, int window, int sinks, void* O, float* lse, void* ws, size_t ws_bytes,
                           qlin_stream stream) {
  KvAttendArgs a{};
  qlin_status st = check_cache(c, &a.cache);
  if (st == QLIN_OK) st = check_batch(c, b, ws, &a.batch);
  if (st != QLIN_OK) return st;
  a.group = head_group(c, n_q_heads);
  if (a.group == 0 || !(scale > 0.f) || !std::isfinite(scale) || window < 0 || sinks < 0) return QLIN_ERR_INVALID_ARG;
  if (ws_bytes < workspace_bytes(c->head_dim)) return QLIN_ERR_WORKSPACE;
  if (a.batch.n_seqs == 0 || a.batch.total_q == 0) return QLIN_OK;
  // a window, or sinks, as long as the table hide nothing; shorter ones leave the kernels' differences of
  // positions room in 32 bits up to 2^30
  const int64_t positions = (int64_t)a.batch.pages_width * a.batch.page_tokens;
  const bool hides = window > 0 && window < positions && sinks < positions;
  if (hides && (window > 1 << 30 || sinks > 1 << 30)) return QLIN_ERR_UNSUPPORTED;
  a.window = hides ? window : 0;
  a.sinks = hides ? sinks : 0;
  if (!check_heads(Q, &a.q) || !O || !aligned(O, 16) || !aligned(lse, 4)) return QLIN_ERR_INVALID_ARG;
  a.o = (uint16_t*)O;
  a.lse = lse;
  a.scale = (float)((double)scale * 1.4426950408889634);
  a.counters = (uint32_t*)((uint8_t*)ws + kKvCountersOffset);
  a.partials = (float*)((uint8_t*)ws + kKvPartialsOffset);
  // Sequences with up to 16 query rows per key/value head go to the decoding kernel, the others
  // to the tensor-core one; a step that can hold both kinds launches both.
  const int sms = attend_sms();
  const bool uniform = a.batch.n_seqs == 1 || (int64_t)a.batch.max_q * a.batch.n_seqs == a.batch.total_q;
  const int64_t most = (int64_t)std::min(a.batch.max_q, a.batch.total_q) * a.group;
  // (a step may have rows that no sequence has: total_q says nothing of a sequence's rows)
  const int64_t least = uniform ? most : 1;
  // rows of a sequence, and (row block, head) items of a step, are counted in 32 bits
  if (most > INT32_MAX ||
      (most > kKvDecodeRows &&
       ((int64_t)a.batch.total_q * a.group / kKvPrefillRows + a.batch.n_seqs) * a.cache.n_heads > INT32_MAX))
    return QLIN_ERR_UNSUPPORTED;
  a.min_rows = 1;
  a.max_rows = most <= kKvDecodeRows ? INT32_MAX : kKvDecodeRows;
  int e = 0;
  if (least <= kKvDecodeRows) {
    e = launch_kv_decode(c->code, c->head_dim, a, (int)std::min<int64_t>(most, kKvDecodeRows), sms, stream);
    a.min_rows = kKvDecodeRows + 1;
  }
  if (!e && most > kKvDecodeRows) {
    a.partials = (float*)((uint8_t*)a.partials + decode_partials(c->head_dim));
    e = launch_kv_prefill(c->code, c->head_dim, a, (int)std::min<int64_t>(most, INT32_MAX), sms, stream);
  }
  return e ? QLIN_ERR_CUDA : QLIN_OK;
}

qlin_status qlin_kv_poll_status(void* ws, qlin_stream stream) {
  if (!ws || !aligned(ws, 256)) return QLIN_ERR_INVALID_ARG;
  cudaStream_t s = (cudaStream_t)stream;
  int32_t v = 0;
  if (cudaMemcpyAsync(&v, ws, 4, cudaMemcpyDeviceToHost, s) != cudaSuccess || cudaStreamSynchronize(s) != cudaSuccess)
    return QLIN_ERR_CUDA;
  if (v == 0) return QLIN_OK;
  // a call that gave up may have left counters behind
  if (cudaMemsetAsync(ws, 0, kKvPartialsOffset, s) != cudaSuccess || cudaStreamSynchronize(s) != cudaSuccess)
    return QLIN_ERR_CUDA;
  return v == kStatusTimeout ? QLIN_ERR_TIMEOUT : v == kStatusInvalid ? QLIN_ERR_INVALID_ARG : QLIN_ERR_CUDA;
}

}  // extern "C"
