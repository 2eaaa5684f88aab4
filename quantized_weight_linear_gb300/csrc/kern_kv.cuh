// Device view and helpers of the 8-bit key/value cache (layouts in include/qlin.h): addressing
// of (block, head) cells, the ragged batch, exact byte -> fp16 conversion, rounding to codes.
//
// Codes and scales are read past L1 (__ldcg or bulk copies): a kernel launched early by
// programmatic dependent launch may share its SM with the append that is rewriting them, and a
// line that append put into L1 must not be what the reader sees.
#pragma once
#include <cuda_fp8.h>

#include "kern_common.cuh"
#include "qlin_kv_internal.h"

namespace qlin {

enum KvCode { kKvInt8 = 1, kKvE4m3 = 2 };

__host__ __device__ constexpr float kv_qmax(int code) { return code == kKvInt8 ? 127.f : 448.f; }
// The reciprocal is a constant, so a block's scale is one product: absmax * fl(1 / Q)
__host__ __device__ constexpr float kv_qmax_inv(int code) { return code == kKvInt8 ? (float)(1.0 / 127.0) : (float)(1.0 / 448.0); }
// Smallest block scale, 2^-60: an all-zero block still has a reciprocal and a logarithm, and
// nothing the attention multiplies leaves the fp32 range on the small side
constexpr float kKvMinScale = 8.673617379884035e-19f;

// A value scale as the attention uses it: one under the smallest (0, in caches from elsewhere) has
// neither logarithm nor reciprocal that the sums can take.  Such a block's values count as 0: its codes
// are replaced by 0, which kv_no_values() tells, under half the smallest scale, whose reciprocal is exact
// too.  Negative scales and NaN stay what they are and give NaN.
__device__ __forceinline__ float kv_value_scale(float s) { return s >= 0.f && s < kKvMinScale ? 0.5f * kKvMinScale : s; }
__device__ __forceinline__ bool kv_no_values(float inverse) { return inverse > 1.f / kKvMinScale; }
// Four bytes of code 0
__host__ __device__ constexpr uint32_t kv_zero_codes(int code) { return code == kKvInt8 ? 0x80808080u : 0u; }

// Bytes of the K (or V) cell of one (block, head)
template <int D>
constexpr int kKvCellBytes = kKvBlock * D;

__device__ __forceinline__ void kv_report(int32_t* status, int32_t what) { atomicCAS(status, 0, what); }

// The K cell of block r of page p, head h; the V cell is page_tokens * D bytes further
template <int D>
__device__ __forceinline__ const uint8_t* kv_cell(const KvView& c, int64_t p, int h, int r) {
  return c.codes + ((p * c.n_heads + h) * 2 * c.page_blocks + r) * kKvCellBytes<D>;
}
__device__ __forceinline__ int64_t kv_scale_index(const KvView& c, int64_t p, int h, int r) {
  return ((p * c.n_heads + h) * c.page_blocks + r) * 2;
}

// The table's entry for block blk of a sequence, unchecked; -1 where the table ends before
__device__ __forceinline__ int kv_page_entry(const KvView& c, const KvBatch& b, int seq, int blk) {
  const int col = blk / c.page_blocks;
  return col < b.pages_width ? __ldg(b.pages + (int64_t)seq * b.pages_stride + col) : -1;
}
// Whether an entry is a page (reported if not)
__device__ __forceinline__ bool kv_page_there(const KvView& c, const KvBatch& b, int entry) {
  if (entry >= 0 && entry < c.n_pages) return true;
  kv_report(b.status, kStatusInvalid);
  return false;
}
// The page of block blk of sequence b, or -1 (reported) where the table or the page is out of range
__device__ __forceinline__ int kv_page(const KvView& c, const KvBatch& b, int seq, int blk) {
  const int p = kv_page_entry(c, b, seq, blk);
  return kv_page_there(c, b, p) ? p : -1;
}

// A sequence of the step: its first row in Q / K / V, its tokens, its position of row 0
struct KvSeq {
  int row0, n, pos0, kv;
};
// n = 0 (reported) where the index arrays make no sense
__device__ __forceinline__ KvSeq kv_seq(const KvBatch& b, int seq) {
  KvSeq s;
  s.row0 = __ldg(b.q_start + seq);
  const int end = __ldg(b.q_start + seq + 1);
  s.kv = __ldg(b.kv_len + seq);
  s.n = (int)((uint32_t)end - (uint32_t)s.row0);  // wraps where the two are far out of range
  if (s.row0 < 0 || end < s.row0 || end > b.total_q || s.n > b.max_q) {
    kv_report(b.status, kStatusInvalid);
    s.row0 = s.n = s.kv = 0;
  }
  if ((int64_t)s.kv > (int64_t)b.pages_width * b.page_tokens) {
    kv_report(b.status, kStatusInvalid);
    s.n = s.kv = 0;
  }
  if (s.kv < 0) s.kv = 0;
  s.pos0 = s.kv - s.n;
  return s;
}

// Whether q_start falls after entry s.  The searches below, and the walks that stand for them, give one
// answer only where it does nowhere.
__device__ __forceinline__ bool kv_falls(const KvBatch& b, int s) {
  return s < b.n_seqs && __ldg(b.q_start + s + 1) < __ldg(b.q_start + s);
}

// Largest seq with first(seq) <= u, for the non-decreasing first(s) = q_start[s] / div + mul * s
// (the whole warp searches, 32 probes a round)
__device__ __forceinline__ int kv_find_seq(const KvBatch& b, int64_t u, int div, int mul, int lane) {
  int lo = 0, hi = b.n_seqs;  // the answer is in [lo, hi)
  while (hi - lo > 1) {
    const int step = (hi - lo + 31) / 32;
    const int s = lo + lane * step;
    const bool le = s < hi && (int64_t)(__ldg(b.q_start + s) / div) + (int64_t)mul * s <= u;
    const unsigned m = __ballot_sync(0xffffffffu, le);
    const int k = m ? 31 - __clz(m) : 0;  // probe 0 (s = lo) always qualifies unless u < first(0)
    lo += k * step;
    hi = min(lo + step, hi);
  }
  return lo;
}

// fp16 pairs of the codes in bytes (0, 1) and (2, 3) of w, exact.  int8 is stored as u = code +
// 128: 0x6400 | u is 1024 + u in fp16, minus 1152 the code.  e4m3 has a conversion instruction
// (moving the bits into place and a product by 2^8 took twice the instructions: 142 against 99 us
// for 537 MB of cache).  It turns the two NaN patterns, which the append never writes but memory
// that was never written may hold, into NaN: where a tile has such bytes they are cleared first.
template <int CODE>
__device__ __forceinline__ void kv_to_half(uint32_t w, uint32_t& h01, uint32_t& h23) {
  if constexpr (CODE == kKvInt8) {
    uint32_t a, b;
    asm("prmt.b32 %0, %1, %2, 0x4140;" : "=r"(a) : "r"(w), "r"(0x64646464u));
    asm("prmt.b32 %0, %1, %2, 0x4342;" : "=r"(b) : "r"(w), "r"(0x64646464u));
    h01 = f16x2_sub(a, 0x64806480u);
    h23 = f16x2_sub(b, 0x64806480u);
  } else {
    asm("{\n .reg .b16 lo, hi;\n mov.b32 {lo, hi}, %2;\n cvt.rn.f16x2.e4m3x2 %0, lo;\n cvt.rn.f16x2.e4m3x2 %1, hi;\n}"
        : "=r"(h01), "=r"(h23)
        : "r"(w));
  }
}

// The same as bf16 pairs (8 significant bits hold both kinds of codes), with the work on the FMA
// pipe where it can be: the softmax next to it needs the ALU.  int8: 0x4300 | u is f = 128 + u for
// u = code + 128 under 128 and 2 u from there, so h = f / 2 - 128 is code / 2 or code, and code =
// h - max(-h, 0).  e4m3: the bits after the sign four places up, and the sign at the top, are a
// bf16 number 2^-120 of the value (16 byte + 240 (byte & 128) puts both there); NaN patterns come
// out as +-480.
template <int CODE>
__device__ __forceinline__ uint32_t kv_pair_to_bf16(uint32_t bytes) {
  uint32_t r;
  if constexpr (CODE == kKvInt8) {
    uint32_t h;
    asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(h) : "r"(bytes), "r"(0x3F003F00u), "r"(0xC300C300u));
    asm("{\n .reg .b32 m;\n fma.rn.relu.bf16x2 m, %1, %2, %3;\n sub.rn.bf16x2 %0, %4, m;\n}"
        : "=r"(r)
        : "r"(bytes), "r"(0xBF00BF00u), "r"(0x43004300u), "r"(h));
  } else {
    const uint32_t moved = bytes * 16u + (bytes & 0x00800080u) * 240u;
    asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(moved), "r"(0x7B807B80u));  // by 2^120
  }
  return r;
}
template <int CODE>
__device__ __forceinline__ void kv_to_bf16(uint32_t w, uint32_t& b01, uint32_t& b23) {
  uint32_t a, b;
  asm("prmt.b32 %0, %1, %2, 0x4140;" : "=r"(a) : "r"(w), "r"(CODE == kKvInt8 ? 0x43434343u : 0u));
  asm("prmt.b32 %0, %1, %2, 0x4342;" : "=r"(b) : "r"(w), "r"(CODE == kKvInt8 ? 0x43434343u : 0u));
  b01 = kv_pair_to_bf16<CODE>(a);
  b23 = kv_pair_to_bf16<CODE>(b);
}

// The first n of the 16 bytes of w (n <= 0: none), the others 0
__device__ __forceinline__ uint4 kv_first_bytes(uint4 w, int n) {
  auto keep = [&](uint32_t x, int k) { return k <= 0 ? 0u : k >= 4 ? x : x & ((1u << (8 * k)) - 1u); };
  return make_uint4(keep(w.x, n), keep(w.y, n - 4), keep(w.z, n - 8), keep(w.w, n - 12));
}

// The value of one stored byte
template <int CODE>
__device__ __forceinline__ float kv_byte_value(uint32_t byte) {
  if constexpr (CODE == kKvInt8) {
    return (float)((int)byte - 128);
  } else {
    const uint32_t h = ((byte & 0x80u) << 8) | ((byte & 0x7Fu) << 7);
    return __half2float(__ushort_as_half((unsigned short)h)) * 256.f;
  }
}

// The byte of y = value / scale: round half to even, saturating, NaN -> 0
template <int CODE>
__device__ __forceinline__ uint32_t kv_byte(float y) {
  if (y != y) y = 0.f;
  if constexpr (CODE == kKvInt8) {
    return (uint32_t)(__float2int_rn(fminf(fmaxf(y, -127.f), 127.f)) + 128);
  } else {
    return (uint32_t)__nv_cvt_float_to_fp8(y, __NV_SATFINITE, __NV_E4M3);
  }
}

// ---- attention ---------------------------------------------------------------------------

// A row's weights 2^(t - M) go to fp16, which has 2^-24 as its smallest step and ends at 2^16.  M is
// set 10 under the largest t, and raised only when a weight would pass 2^15: sums are rescaled a few
// times a row instead of once a tile, and a weight is off by 2^-12 of itself, or, under 2^-24 of the
// row's largest, by up to 2^-35 of that one.  (With M at the largest t it was 2^-25: behind a first
// token of 99.9% of the weight and a small value, 131072 tokens lost 6% of the output in an emulation.)
constexpr float kKvTopLog2 = 10.f, kKvGrowLog2 = 15.f;

// (off by 2 ulp at most, and 0 under 2^-126: nothing beside a weight's rounding to fp16)
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// Two weights in fp16.  They are under 2^15 but for the rounding of t, half a unit from |t| = 2^22 on:
// scores so far out saturate instead of becoming infinite.
__device__ __forceinline__ uint32_t pack_weights(float lo, float hi) {
  uint32_t d;
  asm("cvt.rn.satfinite.f16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
  return d;
}

// The blocks that some row of a sequence sees: blocks [0, sb) and [wb, wb + n - sb)
struct Visible {
  int n, sb, wb;
  __device__ __forceinline__ int block(int i) const { return i < sb ? i : wb + i - sb; }
};
__device__ __forceinline__ Visible visible_blocks(const KvSeq& s, int window, int sinks) {
  Visible v{0, 0, 0};
  if (s.n == 0 || s.kv == 0) return v;
  if (window > 0) {
    const int64_t first = (int64_t)max(s.pos0, 0) - window + 1;
    v.wb = first > 0 ? (int)(first / kKvBlock) : 0;
    const int sink_blocks = (int)(((int64_t)min(sinks, s.kv) + kKvBlock - 1) / kKvBlock);
    v.sb = min(sink_blocks, v.wb);
  }
  v.n = v.sb + (s.kv - 1) / kKvBlock - v.wb + 1;
  return v;
}

// One row of the result from its joined sums
__device__ __forceinline__ float row_inverse(float l) { return l == 0.f ? 0.f : 1.f / l; }
__device__ __forceinline__ float row_lse(float m, float l) { return l == 0.f ? -INFINITY : (m + log2f(l)) * 0.6931471805599453f; }

// 2^floor(log2 am) as bits, kept to normal numbers with a normal reciprocal: queries are divided
// by it, so that a row's largest element is in [1, 2) (exact, and fp16 cannot overflow)
__device__ __forceinline__ uint32_t row_exponent(float am) {
  uint32_t e = __float_as_uint(am) & 0x7F800000u;
  if (e == 0u) e = 127u << 23;
  return e > (253u << 23) ? 253u << 23 : e;
}

}  // namespace qlin
