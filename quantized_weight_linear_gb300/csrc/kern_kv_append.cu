// Appending a step's keys and values to the paged 8-bit cache, with the position rotation and
// the quantization on the way, and reading cached values back.
//
// A warp, or two, per work item, so that a block's new values stay in registers between its
// absolute maximum and its codes:
//  * a (block of 16 tokens, head, K or V) that gets tokens: one warp at head_dim 64, two at 128
//    (32 values a lane) hold them, take their maximum, the scale and the codes -- one read of the
//    activations, one write of the codes;
//  * 1024 elements of one token's queries (rotated only): a lane meets the same element of the
//    heads every 256 elements, so it loads its part of the table's row once.
// The sequence of a block is found by a 32-way search over q_start: sequence s owns the block
// items from q_start[s] / 16 + 2 s on, at least as many as it can touch ((n + 14) / 16 + 1), so
// the host needs no lengths to size the grid; items past a sequence's last block end at once.  Where no
// sequence has more than a token, sequence s owns block item s (128 sequences,
// with their read-back: 14.7 -> 13.2 us).
// A block that already holds tokens is read and requantized only if its scale grows.
//
// The arithmetic that decides a code is fp32, one rounding per operation (no fused
// multiply-add), so codes and scales are reproducible bit for bit; the only division is one
// reciprocal per block.  At prompt sizes the queries run at the memory's rate and the blocks at the
// latency of their loads (16751 tokens of 32 + 2 x 8 heads of 128: 377 MB in 86 us, 4.4 TB/s; DRAM at 50%,
// issue at 58%); one
// token per sequence is launch and load latency (3 us for one, 7 us for 128 sequences).
#include "kern_kv.cuh"

namespace qlin {
namespace {

constexpr int kThreads = 256;
constexpr int kQSlab = 1024;  // query elements per item (512: 132 us for the prompts above with their reading, 1024: 111)

struct AppendArgs {
  KvView cache;
  KvBatch batch;
  KvHeads k, v, q;
  uint16_t* q_out;
  KvRope rope;
  int q_elems;          // query elements of a token (0: no queries)
  int64_t block_items;  // items before the query items
};

// Loads that are issued where they stand (the compiler would move them behind the checks that their
// results wait for)
__device__ __forceinline__ uint4 load_now16(const uint16_t* p) {
  uint4 v;
  asm volatile("ld.global.nc.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
  return v;
}
__device__ __forceinline__ uint32_t load_now4(const uint16_t* p) {
  uint32_t v;
  asm volatile("ld.global.nc.u32 %0, [%1];" : "=r"(v) : "l"(p));
  return v;
}

__device__ __forceinline__ void unpack8(const uint4 w, float (&x)[8]) {
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(u[i] << 16);
    x[2 * i + 1] = __uint_as_float(u[i] & 0xFFFF0000u);
  }
}

// The part of the tables' row pos that elements d0 .. d0 + 7 of a head need: of a split pair both
// halves use the same eight entries, of neighbouring pairs there are four
struct Turn {
  float c[8], s[8];
  bool second;  // the elements are the second ones of split pairs
};
__device__ __forceinline__ Turn load_turn(const KvRope& r, int d0, int pos) {
  Turn t;
  const int half = r.rot >> 1;
  t.second = !r.interleaved && d0 >= half;
  const int i0 = r.interleaved ? d0 >> 1 : t.second ? d0 - half : d0;
  const float4* cp = reinterpret_cast<const float4*>(r.cos + (int64_t)pos * half + i0);
  const float4* sp = reinterpret_cast<const float4*>(r.sin + (int64_t)pos * half + i0);
  const float4 c0 = __ldg(cp), s0 = __ldg(sp);
  float4 c1 = c0, s1 = s0;
  if (!r.interleaved) {
    c1 = __ldg(cp + 1);
    s1 = __ldg(sp + 1);
  }
  t.c[0] = c0.x; t.c[1] = c0.y; t.c[2] = c0.z; t.c[3] = c0.w;
  t.c[4] = c1.x; t.c[5] = c1.y; t.c[6] = c1.z; t.c[7] = c1.w;
  t.s[0] = s0.x; t.s[1] = s0.y; t.s[2] = s0.z; t.s[3] = s0.w;
  t.s[4] = s1.x; t.s[5] = s1.y; t.s[6] = s1.z; t.s[7] = s1.w;
  return t;
}
// Where the partners of elements d0 .. d0 + 7 of a split pair are (0: none are needed)
__device__ __forceinline__ int partner_offset(const KvRope& r, int d0) {
  if (d0 >= r.rot || r.interleaved) return 0;
  return d0 >= (r.rot >> 1) ? -(r.rot >> 1) : r.rot >> 1;
}
// Turns eight elements (y: their partners, of split pairs), one rounding per operation
__device__ __forceinline__ void turn8(float (&x)[8], const float (&y)[8], const Turn& t, bool interleaved) {
  if (interleaved) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float a = x[2 * i], b = x[2 * i + 1];
      x[2 * i] = __fsub_rn(__fmul_rn(a, t.c[i]), __fmul_rn(b, t.s[i]));
      x[2 * i + 1] = __fadd_rn(__fmul_rn(b, t.c[i]), __fmul_rn(a, t.s[i]));
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float u = __fmul_rn(x[i], t.c[i]), w = __fmul_rn(y[i], t.s[i]);
      x[i] = t.second ? __fadd_rn(u, w) : __fsub_rn(u, w);
    }
  }
}

__device__ __forceinline__ float finite_abs(float x) {
  const float a = fabsf(x);
  return a <= 3.402823466e38f ? a : 0.f;  // infinities and NaN do not enter a scale
}
// Maxima that keep a NaN
__device__ __forceinline__ float max_nan(float a, float b) {
  float m;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(m) : "f"(a), "f"(b));
  return m;
}
__device__ __forceinline__ uint32_t max_nan2(uint32_t a, uint32_t b) {
  uint32_t m;
  asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(m) : "r"(a), "r"(b));
  return m;
}

// Four bytes at once: kv_byte of each, or, when every y is finite (so |y| is at most the largest
// code and an ulp or two), the same bytes with less work: adding 1.5 * 2^23 + 128 rounds to an
// integer, half to even, and leaves the offset code in the low byte
template <int CODE, bool kFinite>
__device__ __forceinline__ uint32_t kv_byte4(float y0, float y1, float y2, float y3) {
  if constexpr (!kFinite) {
    return kv_byte<CODE>(y0) | kv_byte<CODE>(y1) << 8 | kv_byte<CODE>(y2) << 16 | kv_byte<CODE>(y3) << 24;
  } else if constexpr (CODE == kKvInt8) {
    auto at = [](float y) { return __float_as_uint(__fadd_rn(y, 12583040.f)); };
    return __byte_perm(__byte_perm(at(y0), at(y1), 0x0040), __byte_perm(at(y2), at(y3), 0x0040), 0x5410);
  } else {
    const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(y0, y1), __NV_SATFINITE, __NV_E4M3);
    const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(y2, y3), __NV_SATFINITE, __NV_E4M3);
    return lo | hi << 16;
  }
}

// Rescaled byte of an older code: code * (old / new)
template <int CODE>
__device__ __forceinline__ uint32_t requant(uint32_t byte, float f) {
  return kv_byte<CODE>(__fmul_rn(kv_byte_value<CODE>(byte), f));
}
template <int CODE>
__device__ __forceinline__ uint32_t requant4(uint32_t w, float f) {
  return requant<CODE>(w & 255u, f) | requant<CODE>((w >> 8) & 255u, f) << 8 | requant<CODE>((w >> 16) & 255u, f) << 16 |
         requant<CODE>(w >> 24, f) << 24;
}

template <bool B>
struct Known {
  static constexpr bool value = B;
};

// Rows [r0, r1) of the block are the step's, rows [0, r0) were there before
struct BlockRows {
  int r0, r1;
};

// The warps that hold a block between them (one at head_dim 64, two at 128) and their maxima
template <int D>
constexpr int kBlockWarps = D / 64;
struct Team {
  float* cell;  // one per warp, in shared memory
  int bar, warp, lane;
};
template <int D>
__device__ __forceinline__ float team_max(const Team& t, float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = max_nan(v, __shfl_xor_sync(0xffffffffu, v, o));
  if constexpr (kBlockWarps<D> == 2) {
    if (t.lane == 0) t.cell[t.warp] = v;
    asm volatile("bar.sync %0, 64;" ::"r"(t.bar) : "memory");
    v = max_nan(t.cell[0], t.cell[1]);
  }
  return v;
}

// The block's scale from the new values' maximum; f = old * (1 / scale)
template <int CODE>
__device__ __forceinline__ float block_scale(float amax, float old, float& inv) {
  const float s = fmaxf(fmaxf(old, __fmul_rn(amax, kv_qmax_inv(CODE))), kKvMinScale);
  inv = __frcp_rn(s);
  return s;
}

// Where a block is, from its entry of the page table: looked at after the rows' loads went out
struct Place {
  int entry, head, block;  // block of the page
  template <int D>
  __device__ __forceinline__ bool find(const AppendArgs& a, int which, uint8_t*& cell, float*& scale) const {
    if (!kv_page_there(a.cache, a.batch, entry)) return false;
    cell = const_cast<uint8_t*>(kv_cell<D>(a.cache, entry, head, block + which * a.cache.page_blocks));
    scale = a.cache.scales + kv_scale_index(a.cache, entry, head, block) + which;
    return true;
  }
};

// Keys: 16-byte pieces of 8 elements; D / 8 lanes a token; a warp has 8 or 16 of the tokens
template <int CODE, int D>
__device__ void append_keys(const AppendArgs& a, const uint16_t* src, int64_t stride, int pos, BlockRows br, const Place& place,
                            const Team& team) {
  constexpr int C = D / 8, TP = 32 / C, IT = kKvBlock / TP / kBlockWarps<D>;
  const int d0 = (team.lane % C) * 8, tr = team.warp * (kKvBlock / kBlockWarps<D>) + team.lane / C;
  const bool turned = d0 < a.rope.rot;
  const int off = partner_offset(a.rope, d0);
  const bool split = a.rope.rot > 0 && !a.rope.interleaved;
  // All rows' loads before the first use and without branches: a row that is not the step's reads
  // one that is and counts as zero
  uint4 raw[IT], mate[IT];
#pragma unroll
  for (int it = 0; it < IT; ++it) {
    const int n = min(max(it * TP + tr, br.r0), br.r1 - 1) - br.r0;
    const uint16_t* row = src + (int64_t)n * stride + d0;
    raw[it] = load_now16(row);
    mate[it] = split ? load_now16(row + off) : raw[it];
  }
  uint8_t* cell;
  float* scale;
  if (!place.find<D>(a, 0, cell, scale)) return;
  float x[IT][8];
  float amax = 0.f;
  const float old = br.r0 > 0 ? __ldcg(scale) : 0.f;
#pragma unroll
  for (int it = 0; it < IT; ++it) {
    const int r = it * TP + tr;
    unpack8(raw[it], x[it]);
    if (turned) {
      float y[8];
      unpack8(mate[it], y);
      turn8(x[it], y, load_turn(a.rope, d0, pos + min(max(r, br.r0), br.r1 - 1) - br.r0), a.rope.interleaved);
    }
    const bool own = r >= br.r0 && r < br.r1;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      x[it][i] = own ? x[it][i] : 0.f;
      amax = max_nan(amax, fabsf(x[it][i]));
    }
  }
  amax = team_max<D>(team, amax);
  const bool finite = amax <= 3.402823466e38f;
  if (!finite) {
    amax = 0.f;
#pragma unroll
    for (int it = 0; it < IT; ++it)
#pragma unroll
      for (int i = 0; i < 8; ++i) amax = fmaxf(amax, finite_abs(x[it][i]));
    __syncwarp();
    if (kBlockWarps<D> == 2) asm volatile("bar.sync %0, 64;" ::"r"(team.bar) : "memory");  // the maxima are read
    amax = team_max<D>(team, amax);
  }
  float inv;
  const float s = block_scale<CODE>(amax, old, inv);
  const float f = __fmul_rn(old, inv);
  auto encode = [&](auto all_finite) {
#pragma unroll
    for (int it = 0; it < IT; ++it) {
      const int r = it * TP + tr;
      uint2* p = reinterpret_cast<uint2*>(cell + r * D + d0);
      if (r >= br.r0 && r < br.r1) {
        uint32_t w[2];
#pragma unroll
        for (int h = 0; h < 2; ++h)
          w[h] = kv_byte4<CODE, all_finite.value>(__fmul_rn(x[it][4 * h], inv), __fmul_rn(x[it][4 * h + 1], inv),
                                                  __fmul_rn(x[it][4 * h + 2], inv), __fmul_rn(x[it][4 * h + 3], inv));
        *p = make_uint2(w[0], w[1]);
      } else if (r < br.r0 && s > old) {
        const uint2 w = __ldcg(p);
        *p = make_uint2(requant4<CODE>(w.x, f), requant4<CODE>(w.y, f));
      }
    }
  };
  if (finite)
    encode(Known<true>{});
  else
    encode(Known<false>{});
  if (team.lane == 0 && team.warp == 0) *scale = s;
}

// Values: a lane takes two neighbouring elements of all 16 tokens, so that it writes each
// element's 16 tokens (adjacent in the cache) at once
template <int CODE, int D>
__device__ void append_values(const AppendArgs& a, const uint16_t* src, int64_t stride, BlockRows br, const Place& place,
                              const Team& team) {
  const int d0 = team.warp * 64 + team.lane * 2;
  uint32_t raw[kKvBlock];
  uint32_t amax2 = 0u;
#pragma unroll
  for (int r = 0; r < kKvBlock; ++r) {
    raw[r] = 0u;
    if (r >= br.r0 && r < br.r1) raw[r] = load_now4(src + (int64_t)(r - br.r0) * stride + d0);
  }
  uint8_t* cell;
  float* scale;
  if (!place.find<D>(a, 1, cell, scale)) return;
  const float old = br.r0 > 0 ? __ldcg(scale) : 0.f;
#pragma unroll
  for (int r = 0; r < kKvBlock; ++r) amax2 = max_nan2(amax2, raw[r] & 0x7FFF7FFFu);
  auto value = [&](int r, int e) -> float { return __uint_as_float(e ? raw[r] & 0xFFFF0000u : raw[r] << 16); };
  float amax = team_max<D>(team, max_nan(__uint_as_float(amax2 << 16), __uint_as_float(amax2 & 0xFFFF0000u)));
  const bool finite = amax <= 3.402823466e38f;
  if (!finite) {
    amax = 0.f;
#pragma unroll
    for (int r = 0; r < kKvBlock; ++r) amax = fmaxf(amax, fmaxf(finite_abs(value(r, 0)), finite_abs(value(r, 1))));
    __syncwarp();
    if (kBlockWarps<D> == 2) asm volatile("bar.sync %0, 64;" ::"r"(team.bar) : "memory");  // the maxima are read
    amax = team_max<D>(team, amax);
  }
  float inv;
  const float s = block_scale<CODE>(amax, old, inv);
  const float f = __fmul_rn(old, inv);
  const bool grow = br.r0 > 0 && s > old;
  if (br.r0 == 0 && br.r1 == kKvBlock && finite) {  // a whole block, the most of a prompt's
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      uint32_t w[4];
#pragma unroll
      for (int i = 0; i < 4; ++i)
        w[i] = kv_byte4<CODE, true>(__fmul_rn(value(4 * i, e), inv), __fmul_rn(value(4 * i + 1, e), inv),
                                    __fmul_rn(value(4 * i + 2, e), inv), __fmul_rn(value(4 * i + 3, e), inv));
      *reinterpret_cast<uint4*>(cell + (d0 + e) * kKvBlock) = make_uint4(w[0], w[1], w[2], w[3]);
    }
  } else if (br.r1 - br.r0 == 1 && !grow) {  // one token and nothing to requantize: single bytes
#pragma unroll
    for (int r = 0; r < kKvBlock; ++r)
      if (r == br.r0)
#pragma unroll
        for (int e = 0; e < 2; ++e)
          cell[(d0 + e) * kKvBlock + r] = (uint8_t)kv_byte<CODE>(__fmul_rn(value(r, e), inv));
  } else {
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      uint4* p = reinterpret_cast<uint4*>(cell + (d0 + e) * kKvBlock);
      const uint4 o = __ldcg(p);
      const uint32_t was[4] = {o.x, o.y, o.z, o.w};
      uint32_t w[4] = {0u, 0u, 0u, 0u};
#pragma unroll
      for (int r = 0; r < kKvBlock; ++r) {
        uint32_t byte = (was[r >> 2] >> (8 * (r & 3))) & 255u;
        if (r < br.r0) {
          if (grow) byte = requant<CODE>(byte, f);
        } else if (r < br.r1) {
          byte = kv_byte<CODE>(__fmul_rn(value(r, e), inv));
        }
        w[r >> 2] |= byte << (8 * (r & 3));
      }
      *p = make_uint4(w[0], w[1], w[2], w[3]);
    }
  }
  if (team.lane == 0 && team.warp == 0) *scale = s;
}

// The item's block of a sequence of the batch; false if there is none
struct BlockItem {
  KvSeq s;
  int entry, blk, head, which;  // entry of the page table, unchecked
  BlockRows br;
};
__device__ __forceinline__ bool find_block(const KvView& c, const KvBatch& b, int64_t item, int lane, BlockItem& it) {
  it.which = (int)(item & 1);
  it.head = (int)((item >> 1) % c.n_heads);
  const int64_t u = (item >> 1) / c.n_heads;
  const bool single = b.max_q <= 1;  // a sequence's token is in one block: its number is the item's
  const int seq = single ? (int)u : kv_find_seq(b, u, kKvBlock, 2, lane);
  it.s = kv_seq(b, seq);
  const int lo = it.s.pos0 > 0 ? it.s.pos0 : 0;  // first position stored
  const int64_t j = single ? 0 : u - (__ldg(b.q_start + seq) / kKvBlock + 2 * (int64_t)seq);
  if (it.s.n == 0 || j < 0 || lo / kKvBlock + j > (it.s.kv - 1) / kKvBlock || lo >= it.s.kv) return false;
  it.blk = lo / kKvBlock + (int)j;
  it.br.r0 = lo > it.blk * kKvBlock ? lo - it.blk * kKvBlock : 0;
  it.br.r1 = it.s.kv - it.blk * kKvBlock < kKvBlock ? it.s.kv - it.blk * kKvBlock : kKvBlock;
  it.entry = kv_page_entry(c, b, seq, it.blk);
  return true;
}

// An item for every 32 sequences: whether q_start falls (the items of a sequence that the search passes
// over would not tell; where every sequence has its item, the launch has none of these)
__device__ __forceinline__ void check_order(const KvBatch& b, int64_t item, int lane) {
  if (item * 32 < b.n_seqs && kv_falls(b, (int)item * 32 + lane)) kv_report(b.status, kStatusInvalid);
}

// One query item, or one of those behind them
template <int D>
__device__ __forceinline__ void rotate_query(const AppendArgs& a, int64_t qi, int lane) {
  const int slabs = (a.q_elems + kQSlab - 1) / kQSlab;
  if (qi >= (int64_t)a.batch.total_q * slabs) {
    if (a.batch.max_q > 1) check_order(a.batch, qi - (int64_t)a.batch.total_q * slabs, lane);
    return;
  }
  const int t = (int)(qi / slabs), e0 = (int)(qi % slabs) * kQSlab, e1 = min(e0 + kQSlab, a.q_elems);
  const int d0 = (lane * 8) % D;  // the lane's elements of a head, every 256 / D heads
  const int off = partner_offset(a.rope, d0);
  const bool split = a.rope.rot > 0 && !a.rope.interleaved;
  const uint16_t* src = a.q.data + (int64_t)t * a.q.token_stride + d0;
  uint4 w[kQSlab / 256], v[kQSlab / 256];  // the elements and their partners, on their way while the rest is looked up
#pragma unroll
  for (int i = 0; i < kQSlab / 256; ++i) {
    const int e = min(e0 + lane * 8 + 256 * i, e1 - 8);
    const uint16_t* row = src + (int64_t)(e / D) * a.q.head_stride;
    w[i] = load_now16(row);
    v[i] = split ? load_now16(row + off) : w[i];
  }
  const int seq = kv_find_seq(a.batch, t, 1, 0, lane);
  const KvSeq s = kv_seq(a.batch, seq);
  const int pos = s.pos0 + t - s.row0;
  const bool real = t >= s.row0 && t < s.row0 + s.n && pos >= 0;
  if (real && a.rope.rot > 0 && pos >= a.rope.n_pos) {
    kv_report(a.batch.status, kStatusInvalid);
    return;
  }
  const bool turned = real && d0 < a.rope.rot;
  Turn turn{};
  if (turned) turn = load_turn(a.rope, d0, pos);
  uint16_t* dst = a.q_out + (int64_t)t * a.q_elems;
#pragma unroll
  for (int i = 0; i < kQSlab / 256; ++i) {
    const int e = e0 + lane * 8 + 256 * i;
    if (e >= e1) break;
    if (turned) {
      float x[8], y[8];
      unpack8(w[i], x);
      unpack8(v[i], y);
      turn8(x, y, turn, a.rope.interleaved);
      w[i] = make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]), pack_bf16x2(x[6], x[7]));
    } else if (!real) {
      w[i] = make_uint4(0u, 0u, 0u, 0u);
    }
    *reinterpret_cast<uint4*>(dst + e) = w[i];
  }
}

// A block item is a chain of loads (sequence, lengths, page, rows, table), so what counts is how many
// warps wait at once: four CTAs of an SM, at 64 registers with a few spilled, take 113 us where two
// without spills take 131 (append and read of 16751 prompt tokens, 8 heads of 128, caches warm, queries apart)
template <int CODE, int D>
__global__ void __launch_bounds__(kThreads, 4) kv_append_kernel(AppendArgs a) {
  constexpr int W = kBlockWarps<D>;
  __shared__ float maxima[kThreads / 32];
  pdl_wait();
  pdl_launch_dependents();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t item = (int64_t)blockIdx.x * (kThreads / 32) + warp;
  if (item < a.block_items * W) {
    const Team team{maxima + warp / W * W, 1 + warp / W, warp % W, lane};
    BlockItem it;
    if (!find_block(a.cache, a.batch, item / W, lane, it)) return;
    const int pos = it.blk * kKvBlock + it.br.r0;  // of the first new row
    if (a.rope.rot > 0 && it.blk * kKvBlock + it.br.r1 > a.rope.n_pos) {
      kv_report(a.batch.status, kStatusInvalid);
      return;
    }
    const int t = it.s.row0 + pos - it.s.pos0;
    const KvHeads& h = it.which ? a.v : a.k;
    const uint16_t* src = h.data + (int64_t)t * h.token_stride + (int64_t)it.head * h.head_stride;
    const Place place{it.entry, it.head, it.blk % a.cache.page_blocks};
    if (it.which)
      append_values<CODE, D>(a, src, h.token_stride, it.br, place, team);
    else
      append_keys<CODE, D>(a, src, h.token_stride, pos, it.br, place, team);
    return;
  }
  rotate_query<D>(a, item - a.block_items * W, lane);
}

struct ReadArgs {
  KvView cache;
  KvBatch batch;
  uint16_t* k_out;
  uint16_t* v_out;
  int64_t block_items;
};

// A warp takes the keys and the values of a (block, head), whose loads wait together; then one item per
// token that zeroes a padding token's rows.  16751 tokens of 8 heads of 128: 103 MB in 18 us, 5.7 TB/s; bound by the
// items' chains of loads.
template <int CODE, int D>
__global__ void __launch_bounds__(kThreads) kv_read_kernel(ReadArgs a) {
  pdl_wait();
  pdl_launch_dependents();
  const int lane = threadIdx.x & 31;
  const int64_t item = (int64_t)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
  const int H = a.cache.n_heads;
  if (item < a.block_items) {
    BlockItem it;
    if (!find_block(a.cache, a.batch, 2 * item, lane, it) || !kv_page_there(a.cache, a.batch, it.entry)) return;
    const int r = it.blk % a.cache.page_blocks;
    const uint8_t* cell = kv_cell<D>(a.cache, it.entry, it.head, r);
    const uint8_t* vcell = kv_cell<D>(a.cache, it.entry, it.head, r + a.cache.page_blocks);
    // keys: 8 elements of every TP-th row; values: E elements of all rows
    constexpr int C = D / 8, TP = 32 / C, IT = kKvBlock / TP, E = D / 32;
    const int d0 = (lane % C) * 8, tr = lane / C, e0 = lane * E;
    uint2 kw[IT];
    uint32_t w[E][4];
#pragma unroll
    for (int i = 0; i < IT; ++i) kw[i] = __ldcg(reinterpret_cast<const uint2*>(cell + (i * TP + tr) * D + d0));
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const uint4 q = __ldcg(reinterpret_cast<const uint4*>(vcell + (e0 + e) * kKvBlock));
      w[e][0] = q.x; w[e][1] = q.y; w[e][2] = q.z; w[e][3] = q.w;
    }
    const float2 s = __ldcg(reinterpret_cast<const float2*>(a.cache.scales + kv_scale_index(a.cache, it.entry, it.head, r)));
    // output row of block row r0
    const int64_t t0 = it.s.row0 + it.blk * kKvBlock + it.br.r0 - it.s.pos0, row = (int64_t)H * D;
    uint16_t* out = a.k_out + (t0 * H + it.head) * D;
#pragma unroll
    for (int i = 0; i < IT; ++i) {
      const int br = i * TP + tr;
      if (br < it.br.r0 || br >= it.br.r1) continue;
      uint32_t o[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint32_t two = ((j & 2) ? kw[i].y : kw[i].x) >> (16 * (j & 1));
        o[j] = pack_bf16x2(__fmul_rn(kv_byte_value<CODE>(two & 255u), s.x), __fmul_rn(kv_byte_value<CODE>((two >> 8) & 255u), s.x));
      }
      *reinterpret_cast<uint4*>(out + (br - it.br.r0) * row + d0) = make_uint4(o[0], o[1], o[2], o[3]);
    }
    out = a.v_out + (t0 * H + it.head) * D;
#pragma unroll
    for (int br = 0; br < kKvBlock; ++br) {
      if (br < it.br.r0 || br >= it.br.r1) continue;
      uint32_t o[E / 2];
#pragma unroll
      for (int j = 0; j < E / 2; ++j)
        o[j] = pack_bf16x2(__fmul_rn(kv_byte_value<CODE>((w[2 * j][br >> 2] >> (8 * (br & 3))) & 255u), s.y),
                           __fmul_rn(kv_byte_value<CODE>((w[2 * j + 1][br >> 2] >> (8 * (br & 3))) & 255u), s.y));
      uint32_t* p = reinterpret_cast<uint32_t*>(out + (br - it.br.r0) * row + e0);
      if constexpr (E == 4)
        *reinterpret_cast<uint2*>(p) = make_uint2(o[0], o[1]);
      else
        *p = o[0];
    }
    return;
  }
  const int64_t t = item - a.block_items;
  if (t >= a.batch.total_q) {
    if (a.batch.max_q > 1) check_order(a.batch, t - a.batch.total_q, lane);
    return;
  }
  const int seq = kv_find_seq(a.batch, t, 1, 0, lane);
  const KvSeq s = kv_seq(a.batch, seq);
  if (s.n == 0 || t < s.row0 || t >= s.row0 + s.n || s.pos0 + (int)(t - s.row0) >= 0) return;
  for (int e = lane * 8; e < H * D; e += 256) {
    *reinterpret_cast<uint4*>(a.k_out + t * H * D + e) = make_uint4(0u, 0u, 0u, 0u);
    *reinterpret_cast<uint4*>(a.v_out + t * H * D + e) = make_uint4(0u, 0u, 0u, 0u);
  }
}

template <typename Args>
int launch_items(void (*kernel)(Args), const Args& a, int64_t items, void* stream) {
  if (items <= 0) return 0;
  const int64_t ctas = (items + kThreads / 32 - 1) / (kThreads / 32);
  if (ctas > INT32_MAX) return (int)cudaErrorInvalidConfiguration;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)ctas);
  cfg.blockDim = dim3(kThreads);
  cfg.stream = (cudaStream_t)stream;
  cudaLaunchAttribute at{};
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = QLIN_USE_PDL;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  return (int)cudaLaunchKernelEx(&cfg, kernel, a);
}

int order_items(const KvBatch& b) { return b.max_q > 1 ? (b.n_seqs + 31) / 32 : 0; }
int64_t block_items(const KvView& c, const KvBatch& b) {
  const int64_t blocks = b.max_q <= 1 ? b.n_seqs : (int64_t)b.total_q / kKvBlock + 2 * (int64_t)b.n_seqs;
  return blocks * c.n_heads * 2;
}

}  // namespace

int launch_kv_append(int code, int head_dim, const KvView& c, const KvBatch& b, const KvHeads& k, const KvHeads& v,
                     const KvHeads& q, int n_q_heads, uint16_t* q_out, const KvRope& r, void* stream) {
  AppendArgs a{c, b, k, v, q, q_out, r, n_q_heads * head_dim, block_items(c, b)};
  const int64_t items = a.block_items * (head_dim / 64) + (int64_t)b.total_q * ((a.q_elems + kQSlab - 1) / kQSlab) + order_items(b);
  if (head_dim == 128)
    return launch_items(code == kKvInt8 ? kv_append_kernel<kKvInt8, 128> : kv_append_kernel<kKvE4m3, 128>, a, items, stream);
  return launch_items(code == kKvInt8 ? kv_append_kernel<kKvInt8, 64> : kv_append_kernel<kKvE4m3, 64>, a, items, stream);
}

int launch_kv_read(int code, int head_dim, const KvView& c, const KvBatch& b, uint16_t* k_out, uint16_t* v_out,
                   void* stream) {
  ReadArgs a{c, b, k_out, v_out, block_items(c, b) / 2};
  const int64_t items = a.block_items + b.total_q + order_items(b);
  if (head_dim == 128)
    return launch_items(code == kKvInt8 ? kv_read_kernel<kKvInt8, 128> : kv_read_kernel<kKvE4m3, 128>, a, items, stream);
  return launch_items(code == kKvInt8 ? kv_read_kernel<kKvInt8, 64> : kv_read_kernel<kKvE4m3, 64>, a, items, stream);
}

}  // namespace qlin
