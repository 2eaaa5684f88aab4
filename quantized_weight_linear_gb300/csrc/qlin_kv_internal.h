// Declarations of the 8-bit key/value cache shared by its host file and kernels (layouts and
// semantics in include/qlin.h).
#pragma once
#include "qlin_internal.h"

namespace qlin {

// device status word: a bad index in the batch's device arrays; a fault of the library's own
constexpr int kStatusInvalid = 1, kStatusInternal = 3;

constexpr int kKvBlock = 16;      // tokens that share a scale
constexpr int kKvMaxSeqs = 2048;  // sequences of a step

struct KvView {
  uint8_t* codes;
  float* scales;
  int n_pages, n_heads, page_blocks;  // page_blocks: blocks of 16 tokens in a page
};

struct KvBatch {
  const int32_t* q_start;
  const int32_t* kv_len;
  const int32_t* pages;
  int64_t pages_stride;
  int n_seqs, total_q, max_q, pages_width, page_tokens;
  int32_t* status;
};

struct KvHeads {
  const uint16_t* data;
  int64_t token_stride, head_stride;
};

struct KvRope {
  const float* cos;
  const float* sin;
  int n_pos, rot, interleaved;  // rot = 0: no rotation
};

struct KvAttendArgs {
  KvView cache;
  KvBatch batch;
  KvHeads q;
  uint16_t* o;
  float* lse;     // or null
  int group;      // query heads per key/value head
  float scale;    // of q . k, times log2(e)
  int window, sinks;
  int min_rows, max_rows;  // the launch takes the sequences with that many query rows a key/value head
  uint32_t* counters;  // [kMaxSms] arrival counters of split rows, zero between calls
  float* partials;     // partial results of split rows
};

// Workspace of the cache calls: [status, 256 bytes][counters][partials]
constexpr int kMaxSms = 192;  // CTAs that may share a row
constexpr size_t kKvCountersOffset = 256;
constexpr size_t kKvPartialsOffset = kKvCountersOffset + kMaxSms * 4;
size_t kv_decode_partial_bytes(int head_dim, int sms);

int launch_kv_append(int code, int head_dim, const KvView& c, const KvBatch& b, const KvHeads& k, const KvHeads& v,
                     const KvHeads& q, int n_q_heads, uint16_t* q_out, const KvRope& r, void* stream);
int launch_kv_read(int code, int head_dim, const KvView& c, const KvBatch& b, uint16_t* k_out, uint16_t* v_out,
                   void* stream);
// Up to so many rows: kern_kv_decode.cu (whose variants hold 8 and 16), more: kern_kv_prefill.cu.  us of
// either, 8 key heads of 128, int8, at 4 / 8 / 16 rows: 64 sequences of 8192 177 / 180 / 259 against 335 /
// 335 / 338; 16 of 4096 36 / 39 / 54 against 59 / 59 / 60; one of 4096 13.4 / 16.0 / 23.8 against 18.9 /
// 19.0 / 19.3, the one case that it loses.
constexpr int kKvDecodeRows = 16;
// rows: most query rows per key/value head of a sequence
int launch_kv_decode(int code, int head_dim, const KvAttendArgs& a, int rows, int sms, void* stream);
constexpr int kKvPrefillRows = 256;  // rows of a row block of the latter
size_t kv_prefill_partial_bytes(int head_dim, int sms);
int launch_kv_prefill(int code, int head_dim, const KvAttendArgs& a, int rows, int sms, void* stream);

}  // namespace qlin
