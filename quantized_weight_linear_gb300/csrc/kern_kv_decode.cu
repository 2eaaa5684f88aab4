// Attention over the paged 8-bit cache for up to 16 query rows per key/value head (decoding).
//
// O_i = sum_j e^(w_ij) v_j / sum_j e^(w_ij), w_ij = scale q_i . k_j, k_j = ks_b ck_j, v_j = vs_b
// cv_j for the codes ck, cv and the scales of j's block of 16 tokens.  The products run on the
// bare codes, exact in fp16 (m16n8k16 MMAs, fp32 accumulators), and both scales ride on the
// exponent: with t_ij = (q_i . ck_j) (scale log2(e) ks_b) + log2(vs_b),
//   p_ij = 2^(t_ij - M_i),  O_i = sum p_ij cv_j / L_i,  L_i = sum p_ij / vs_b,
// one FMA and one exponential an element.  p < 2^15 goes to fp16 (11 bits; kern_kv.cuh says where M is
// and what that does to small weights); M, L and O stay in fp32.  Queries are scaled by a power of two per row
// so that the row's largest element is in [1, 2): bf16 to fp16 is then exact but for elements
// under 2^-14 of the largest, and cannot overflow.
//
// Work: an item is (sequence, head); four of its blocks (64 tokens) are a unit, and the units of
// all items form one line that is cut into equal ranges, one per warp of a grid of one CTA per SM,
// so ragged batches balance by themselves and one long sequence uses the whole GPU.  A warp
// streams its units (K and V cells, by cp.async.bulk into a ring of its own) and keeps the softmax
// state of the current item in registers.  Items that a range cuts are put together through
// shared memory inside a CTA, then through the workspace: the last CTA to arrive joins the partial
// results in CTA order, so the result does not depend on the order of arrival.
//
// The tokens are the MMA rows (S^T = K Q^T, O^T = V^T P^T): 8 query rows, the usual number, fill
// the N = 8 columns, where as MMA rows they would leave half of every MMA empty and double the
// accumulators.  Neither layout of the cache needs a transposition: a lane's 16 bytes of a key
// are four k-steps of its A operand (the queries are loaded in the same order of elements), and
// its 16 bytes of a value element are the tokens of one block, four for each of four MMAs -- in an
// MMA the lanes t = 0..3 of a row cover four tokens of the blocks t.  The weights go from the
// first product's accumulators to the second's B operand by an 8 x 8 transposition (movmatrix).
// The conversion of the bytes is most of the instructions: two a pair of codes.
//
// Bound by memory: 4 sequences of 524288 tokens (4.3 GB) take 647 us, 6.65 TB/s, 0.98 of the
// measured copy; 64 ragged ones (600 MB) 115 us, of which 3 us before the first keys, 85 at the
// memory's rate and the rest the spread of the CTAs' ends and two joins of 3 us; one sequence of
// 4100 tokens (8 MB) 13 us, all of it latency.  Six warps with two units of 16 KB in flight each fill
// the shared memory; with 16 rows (NT = 2) five leave room for the larger partial results.  Heads of 64
// are bound by the latency of those six warps instead: 64 sequences of 8192 tokens (537 MB) take 133 us,
// 4.0 TB/s, with DRAM at 46%, issue at 29% and the tensor pipe at 9% in a capture: twice the softmax a
// byte, and no unit full.
#include "kern_kv.cuh"

namespace qlin {
namespace {

constexpr int kUnitBlocks = 4;

// NT: tiles of 8 query rows
template <int D, int NT>
struct DecCfg {
  static constexpr int kWarps = NT == 1 ? 6 : 5, kThreads = kWarps * 32;
  static constexpr int kStages = 2 * (128 / D);
  static constexpr int kRows = 8 * NT;
  // the lanes of a row read the same value element of four blocks: 32 bytes between the cells
  // spread them over the banks
  static constexpr int kVCell = kKvCellBytes<D> + 32;
  static constexpr int kK = kUnitBlocks * kKvCellBytes<D>, kStage = kK + (kUnitBlocks - 1) * kVCell + kKvCellBytes<D>;
  static constexpr int kPart = kRows * D + 2 * kRows;  // floats of a partial result: O, M, L
  static constexpr int kRing = kWarps * kStages * kStage;
  static constexpr int kHead = kWarps * kPart * 4;
  static_assert(kRing >= kHead + kMaxSms * kRows * 4 + kThreads * 16, "what the joins put into the idle ring");
  static_assert(kRing + kHead + kWarps * kStages * 16 + (kKvMaxSeqs + 1) * 4 + 128 + 1024 <= 232448, "shared memory");
  static_assert(kStage % 16 == 0 && kHead % 16 == 0, "alignment of the bulk copies");
};

template <int D, int NT>
size_t smem_bytes(int n_seqs) {
  using C = DecCfg<D, NT>;
  return (size_t)C::kRing + C::kHead + C::kWarps * C::kStages * 16 + (size_t)(n_seqs + 1) * 4 + 128;
}

// 8 x 8 fp16 transposition over a warp
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

// A sequence of this launch, or n = 0
__device__ __forceinline__ KvSeq decode_seq(const KvAttendArgs& a, int seq) {
  KvSeq s = kv_seq(a.batch, seq);
  if (s.n * a.group > a.max_rows) s.n = 0;
  return s;
}

// An item: a sequence's head, and the line's units [u0, u0 + units)
struct Item {
  KvSeq s;
  Visible vis;
  int u0, units, head, rows, seq;
};

// Units of an item: its blocks', and an empty one for what it takes beside them (queries, start, end:
// about a unit's time), so that ranges with many short sequences are not the last to finish
__device__ __forceinline__ int item_units(const Visible& v) { return v.n ? (v.n + kUnitBlocks - 1) / kUnitBlocks + 1 : 0; }

__device__ __forceinline__ Item item_at(const KvAttendArgs& a, const int* prefix, int u) {
  int lo = 0, hi = a.batch.n_seqs;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (prefix[mid] <= u) lo = mid; else hi = mid;
  }
  Item it;
  it.seq = lo;
  it.s = decode_seq(a, lo);
  it.vis = visible_blocks(it.s, a.window, a.sinks);
  it.units = item_units(it.vis);
  it.head = (u - prefix[lo]) / it.units;
  it.u0 = prefix[lo] + it.head * it.units;
  it.rows = it.s.n * a.group;
  return it;
}

// split_owner of the line's units over G CTAs, in 32 bits where the product fits
__device__ __forceinline__ int owner_of(int u, uint32_t U, uint32_t G) {
  if (U < 0xFFFFFFFFu / G) return (int)(((uint32_t)(u + 1) * G - 1u) / U);
  return (int)split_owner(u, U, G);
}

// What joining the parts of an item needs of it
struct Cut {
  int u0, units, rows, row0, head;  // u0 = -1: no item
};

// Output row of row r of an item (row0: its sequence's first token)
__device__ __forceinline__ int64_t row_out(const KvAttendArgs& a, int row0, int head, int r) {
  return (int64_t)(row0 + r / a.group) * (a.cache.n_heads * a.group) + head * a.group + r % a.group;
}

template <int CODE, int D, int NT>
__global__ void __launch_bounds__(DecCfg<D, NT>::kThreads, 1) kv_decode_kernel(const KvAttendArgs a) {
  using C = DecCfg<D, NT>;
  constexpr int KS = D / 16, kWarps = C::kWarps, kThreads = C::kThreads, kRows = C::kRows;
  extern __shared__ __align__(128) uint8_t smem_raw[];
  uint8_t* ring_all = smem_align128(smem_raw);
  float* heads = reinterpret_cast<float*>(ring_all + C::kRing);
  uint64_t* bars = reinterpret_cast<uint64_t*>(ring_all + C::kRing + C::kHead);
  int* prefix = reinterpret_cast<int*>(bars + 2 * kWarps * C::kStages);
  __shared__ int64_t scan[kWarps];
  // the cut items: entry 2 w of warp w's first one, entry 2 w + 1 of its last one
  __shared__ Cut cuts[2 * kWarps];
  __shared__ float weight[2 * kWarps][kRows], row_l[kWarps][kRows];
  __shared__ int complete[2 * kWarps];  // an entry's item, joined from here, is the last part to arrive

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
  uint8_t* ring = ring_all + warp * C::kStages * C::kStage;
  uint64_t* kbar = bars + warp * 2 * C::kStages;
  uint64_t* vbar = kbar + C::kStages;
  if (lane == 0) {
    for (int s = 0; s < 2 * C::kStages; ++s) mbar_init(&kbar[s], 1);
    fence_mbar_init();
    cuts[2 * warp].u0 = cuts[2 * warp + 1].u0 = -1;
    complete[2 * warp] = complete[2 * warp + 1] = 0;
  }
  pdl_wait();
  pdl_launch_dependents();

  // prefix[s]: units before sequence s
  int64_t carry = 0;
  for (int b = 0; b < a.batch.n_seqs; b += kThreads) {
    int64_t n = 0;
    if (b + tid < a.batch.n_seqs)
      n = (int64_t)item_units(visible_blocks(decode_seq(a, b + tid), a.window, a.sinks)) * a.cache.n_heads;
    int64_t x = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += y;
    }
    if (lane == 31) scan[warp] = x;
    __syncthreads();
    int64_t before = carry, all = 0;
    for (int w = 0; w < kWarps; ++w) {
      if (w < warp) before += scan[w];
      all += scan[w];
    }
    if (b + tid < a.batch.n_seqs) prefix[b + tid] = (int)min(before + x - n, (int64_t)INT_MAX);
    carry += all;
    __syncthreads();
  }

  // sequences that see nothing: zeros
  for (int s = blockIdx.x; s < a.batch.n_seqs; s += (int)gridDim.x) {
    const KvSeq q = decode_seq(a, s);
    if (q.n == 0 || q.kv > 0) continue;
    const int64_t hq = (int64_t)a.cache.n_heads * a.group;
    uint4* o = reinterpret_cast<uint4*>(a.o + q.row0 * hq * D);
    for (int64_t i = tid; i < q.n * hq * (D / 8); i += kThreads) o[i] = make_uint4(0u, 0u, 0u, 0u);
    if (a.lse)
      for (int64_t i = tid; i < q.n * hq; i += kThreads) a.lse[q.row0 * hq + i] = -INFINITY;
  }
  if (carry > INT_MAX) {  // 1.4e11 tokens x heads
    kv_report(a.batch.status, kStatusInvalid);
    return;
  }

  // A unit a warp, if there are no more (17 units for each of 8 heads: 11.7 us, rounded down to six a
  // CTA, so that some warps have two, 14.0); no CTA of the line is without one, since those that an
  // item spans all take part in joining it
  const int64_t U = carry, G = max((int64_t)1, min((int64_t)gridDim.x, (U + kWarps - 1) / kWarps));
  if (blockIdx.x >= G) return;
  const int cs = (int)split_start(blockIdx.x, U, G), ce = (int)split_start(blockIdx.x + 1, U, G);
  const int ws = cs + (ce - cs) * warp / kWarps, we = cs + (ce - cs) * (warp + 1) / kWarps;
  const int n = we - ws;
  bool ok = true;
  float o[NT][D / 16][4];  // lane (g, t): elements 16 m + g (+ 8) of rows 8 nt + 2 t, + 1
  float m[NT][2], l[NT][2];
  Item it{};

  auto stash = [&](float* part) {  // this warp's state of the item
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int k = 0; k < D / 16; ++k)
#pragma unroll
        for (int i = 0; i < 4; ++i) part[(8 * nt + 2 * t + (i & 1)) * D + 16 * k + 8 * (i >> 1) + g] = o[nt][k][i];
      if (g == 0)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          part[kRows * D + 8 * nt + 2 * t + h] = m[nt][h];
          part[kRows * D + kRows + 8 * nt + 2 * t + h] = l[nt][h];
        }
    }
  };

  if (n > 0) {
    // Batches of 8 units: lane 4 (j % 8) + b holds the cell (in units of 16 D bytes) of block b
    // of unit j, or -1, and its scales.  Pages are looked up two batches ahead and scales one, so
    // that neither load is waited for
    auto cell_of = [&](int j) -> int {
      if (j >= n) return -1;
      const Item x = item_at(a, prefix, ws + j);
      const int i = (ws + j - x.u0) * kUnitBlocks + t;
      if (i >= x.vis.n) return -1;
      const int blk = x.vis.block(i);
      const int p = max(kv_page(a.cache, a.batch, x.seq, blk), 0);
      return ((p * a.cache.n_heads + x.head) * 2) * a.cache.page_blocks + blk % a.cache.page_blocks;
    };
    auto scales_of = [&](int cell) -> float2 {
      if (cell < 0) return make_float2(1.f, 1.f);
      const int ph = cell / (2 * a.cache.page_blocks), r = cell % (2 * a.cache.page_blocks);
      return __ldcg(reinterpret_cast<const float2*>(a.cache.scales) + (int64_t)ph * a.cache.page_blocks + r);
    };
    int cell0 = cell_of(g), cell1 = -1, cell2 = -1;

    // the K or V cells of unit j into its stage; batch: that of the unit being consumed
    auto issue = [&](int j, int batch, int v) {
      const int c = __shfl_sync(0xffffffffu, (j >> 3) == batch ? cell0 : cell1, 4 * (j & 7) + t);
      const int s = j % C::kStages;
      uint64_t* bar = (v ? vbar : kbar) + s;
      const unsigned have = __ballot_sync(0xffffffffu, c >= 0) & 15u;
      if (lane == 0) mbar_arrive_expect_tx(bar, (uint32_t)__popc(have) * kKvCellBytes<D>);
      __syncwarp();
      if (lane < kUnitBlocks && c >= 0)
        bulk_g2s(ring + s * C::kStage + (v ? C::kK + lane * C::kVCell : lane * kKvCellBytes<D>),
                 a.cache.codes + ((int64_t)c + (v ? a.cache.page_blocks : 0)) * kKvCellBytes<D>, kKvCellBytes<D>, bar);
    };
    const int ahead = min(C::kStages, n);
    for (int j = 0; j < ahead; ++j) {
      issue(j, 0, 0);
      issue(j, 0, 1);
    }
    const float2 sc0 = scales_of(cell0);
    if (n > 8) {
      cell1 = cell_of(8 + g);
      cell2 = cell_of(16 + g);
    }
    float2 sc1 = scales_of(cell1);
    float ks = 1.f, lvs = 0.f, ivs = 1.f;
    bool zeros = false;  // some block of the batch has no values
    auto take = [&](const float2& sc) {
      const float vs = kv_value_scale(sc.y);
      ks = sc.x;
      lvs = log2f(vs);
      ivs = 1.f / vs;
      zeros = __any_sync(0xffffffffu, kv_no_values(ivs));
    };

    uint32_t qb[NT][KS][2];
    float rf[NT][2];
    int item_end = -1, k_issued = ahead, v_issued = ahead;
    for (int j = 0; j < n; ++j) {
      const int u = ws + j;
      if (j > 0 && (j & 7) == 0) {  // next batch of 8 units
        cell0 = cell1;
        take(sc1);
        cell1 = cell2;
        sc1 = scales_of(cell1);
        cell2 = cell_of(j + 16 + g);
      }
      if (u >= item_end) {  // first unit of an item (or of the range)
        it = item_at(a, prefix, u);
        item_end = it.u0 + it.units;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
          for (int k = 0; k < D / 16; ++k)
#pragma unroll
            for (int i = 0; i < 4; ++i) o[nt][k][i] = 0.f;
          m[nt][0] = m[nt][1] = -INFINITY;
          l[nt][0] = l[nt][1] = 0.f;
          // queries: lane (g, t) takes the elements of row g that its words of a key hold
          const int r = 8 * nt + g;
          const uint16_t* src = a.q.data + (int64_t)(it.s.row0 + r / a.group) * a.q.token_stride +
                                (int64_t)(it.head * a.group + r % a.group) * a.q.head_stride;
          uint2 raw[KS];
          float am = 0.f;
#pragma unroll
          for (int s = 0; s < KS; ++s) {
            raw[s] = r < it.rows ? __ldg(reinterpret_cast<const uint2*>(src + 64 * (s >> 2) + 16 * t + 4 * (s & 3)))
                                 : make_uint2(0u, 0u);
            am = fmaxf(am, fmaxf(fmaxf(fabsf(__uint_as_float(raw[s].x << 16)), fabsf(__uint_as_float(raw[s].x & 0xFFFF0000u))),
                                 fmaxf(fabsf(__uint_as_float(raw[s].y << 16)), fabsf(__uint_as_float(raw[s].y & 0xFFFF0000u)))));
          }
          am = fmaxf(am, __shfl_xor_sync(0xffffffffu, am, 1));
          am = fmaxf(am, __shfl_xor_sync(0xffffffffu, am, 2));
          const uint32_t e = row_exponent(am);
          const float f = __uint_as_float(e) * a.scale, inv = __uint_as_float((254u << 23) - e);
#pragma unroll
          for (int h = 0; h < 2; ++h) rf[nt][h] = __shfl_sync(0xffffffffu, f, 4 * (2 * t + h));
#pragma unroll
          for (int s = 0; s < KS; ++s) {
            qb[nt][s][0] = pack_f16x2(__uint_as_float(raw[s].x << 16) * inv, __uint_as_float(raw[s].x & 0xFFFF0000u) * inv);
            qb[nt][s][1] = pack_f16x2(__uint_as_float(raw[s].y << 16) * inv, __uint_as_float(raw[s].y & 0xFFFF0000u) * inv);
          }
        }
      }
      if (j == 0) take(sc0);  // after the first queries' loads went out
      const int stage = j % C::kStages;
      const uint32_t phase = (uint32_t)(j / C::kStages) & 1u;
      const uint8_t* kc = ring + stage * C::kStage;
      ok = __all_sync(0xffffffffu, mbar_wait(&kbar[stage], phase, a.batch.status));
      if (!ok) break;
      if ((u - it.u0) * kUnitBlocks >= it.vis.n) {  // the empty one
        if (j + C::kStages < n) {
          issue(j + C::kStages, j >> 3, 0);
          issue(j + C::kStages, j >> 3, 1);
          k_issued = v_issued = j + C::kStages + 1;
        }
      } else {
        // S^T = K Q^T: row g (g + 8) of tile i is token 4 i + g % 2 (+ 2) of block g / 2, so that
        // after the transposition a lane (row, t) holds tokens 4 i .. 4 i + 3 of block t
        float x[NT][4][4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 4; ++e) x[nt][i][e] = 0.f;
          const uint8_t* row = kc + (g >> 1) * kKvCellBytes<D> + (4 * i + (g & 1)) * D + 16 * t;
#pragma unroll
          for (int c = 0; c < KS / 4; ++c) {
            const uint4 w0 = *reinterpret_cast<const uint4*>(row + 64 * c);
            const uint4 w1 = *reinterpret_cast<const uint4*>(row + 2 * D + 64 * c);
            const uint32_t a0[4] = {w0.x, w0.y, w0.z, w0.w}, a1[4] = {w1.x, w1.y, w1.z, w1.w};
#pragma unroll
            for (int s = 0; s < 4; ++s) {
              uint32_t af[4];
              kv_to_half<CODE>(a0[s], af[0], af[2]);
              kv_to_half<CODE>(a1[s], af[1], af[3]);
#pragma unroll
              for (int nt = 0; nt < NT; ++nt) mma_f16(x[nt][i], af, qb[nt][4 * c + s][0], qb[nt][4 * c + s][1]);
            }
          }
        }
        __syncwarp();  // every lane has read the keys
        if (j + C::kStages < n) {
          issue(j + C::kStages, j >> 3, 0);
          k_issued = j + C::kStages + 1;
        }
        // the lane's block of the unit: its scales and tokens
        const int from = 4 * (j & 7) + (g >> 1);
        const float bks = __shfl_sync(0xffffffffu, ks, from), blv = __shfl_sync(0xffffffffu, lvs, from),
                    biv = __shfl_sync(0xffffffffu, ivs, from);
        const int bi = (u - it.u0) * kUnitBlocks + (g >> 1);
        const int tok = it.vis.block(bi) * kKvBlock;
        const int p_last = it.s.kv - 1;
        const bool partial = bi >= it.vis.n || tok + kKvBlock - 1 > it.s.pos0 ||
                             (a.window > 0 && tok <= p_last - a.window && tok + kKvBlock > a.sinks);
        const bool any_partial = __any_sync(0xffffffffu, partial);
        if (any_partial) {  // some element is masked
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const int pos = it.s.pos0 + (8 * nt + 2 * t + h) / a.group;
#pragma unroll
              for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                  const int k = tok + 4 * i + (g & 1) + 2 * e;
                  if (bi >= it.vis.n || k > pos || (a.window > 0 && k <= pos - a.window && k >= a.sinks))
                    x[nt][i][2 * e + h] = -INFINITY;
                }
            }
        }
        float kb[NT][2], top[NT][2];
        bool grow = false;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            kb[nt][h] = fmaxf(bks * rf[nt][h], 1e-37f);  // positive, so that it keeps -inf
            float v = -INFINITY;
#pragma unroll
            for (int i = 0; i < 4; ++i) v = fmaxf(v, fmaxf(x[nt][i][h], x[nt][i][2 + h]));
            top[nt][h] = fmaf(v, kb[nt][h], blv);
            grow |= top[nt][h] > m[nt][h] + kKvGrowLog2;
          }
        if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              float v = top[nt][h];
#pragma unroll
              for (int s = 4; s < 32; s <<= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, s));
              v = fmaxf(v - kKvTopLog2, m[nt][h]);
              const float f = m[nt][h] == -INFINITY ? 0.f : ex2(m[nt][h] - v);
              m[nt][h] = v;
              l[nt][h] *= f;
#pragma unroll
              for (int k = 0; k < D / 16; ++k) {
                o[nt][k][h] *= f;
                o[nt][k][2 + h] *= f;
              }
            }
        }
        uint32_t pb[NT][4][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          const float off0 = blv - (m[nt][0] == -INFINITY ? 0.f : m[nt][0]), off1 = blv - (m[nt][1] == -INFINITY ? 0.f : m[nt][1]);
          float s0 = 0.f, s1 = 0.f;
#pragma unroll
          for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const float p0 = ex2(fmaf(x[nt][i][2 * e], kb[nt][0], off0)), p1 = ex2(fmaf(x[nt][i][2 * e + 1], kb[nt][1], off1));
              s0 += p0;
              s1 += p1;
              pb[nt][i][e] = transpose8(pack_weights(p0, p1));
            }
          l[nt][0] = fmaf(s0, biv, l[nt][0]);
          l[nt][1] = fmaf(s1, biv, l[nt][1]);
        }
        // O^T += V^T P^T
        ok = __all_sync(0xffffffffu, mbar_wait(&vbar[stage], phase, a.batch.status));
        if (!ok) break;
        if (CODE == kKvE4m3 && any_partial) {  // bytes that were never written may be NaN: clear them
          for (int i = lane; i < kUnitBlocks * D; i += 32) {
            const int b = i / D, vb = (u - it.u0) * kUnitBlocks + b;
            const int have = vb < it.vis.n ? it.s.kv - it.vis.block(vb) * kKvBlock : 0;
            if (have >= kKvBlock) continue;
            uint4* v = reinterpret_cast<uint4*>(ring + stage * C::kStage + C::kK + b * C::kVCell + (i % D) * kKvBlock);
            *v = kv_first_bytes(*v, have);
          }
          fence_proxy_async_smem();  // before the next copy into these bytes
          __syncwarp();
        }
        if (zeros) {
          for (int b = 0; b < kUnitBlocks; ++b) {
            if (!kv_no_values(__shfl_sync(0xffffffffu, ivs, 4 * (j & 7) + b))) continue;
            constexpr uint32_t z = kv_zero_codes(CODE);
            uint4* v = reinterpret_cast<uint4*>(ring + stage * C::kStage + C::kK + b * C::kVCell);
            for (int i = lane; i < D; i += 32) v[i] = make_uint4(z, z, z, z);
          }
          fence_proxy_async_smem();  // as above
          __syncwarp();
        }
        const uint8_t* vc = kc + C::kK + t * C::kVCell;
#pragma unroll
        for (int k = 0; k < D / 16; ++k) {
          const uint4 w0 = *reinterpret_cast<const uint4*>(vc + (16 * k + g) * kKvBlock);
          const uint4 w1 = *reinterpret_cast<const uint4*>(vc + (16 * k + 8 + g) * kKvBlock);
          const uint32_t a0[4] = {w0.x, w0.y, w0.z, w0.w}, a1[4] = {w1.x, w1.y, w1.z, w1.w};
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            uint32_t af[4];
            kv_to_half<CODE>(a0[i], af[0], af[2]);
            kv_to_half<CODE>(a1[i], af[1], af[3]);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) mma_f16(o[nt][k], af, pb[nt][i][0], pb[nt][i][1]);
          }
        }
        __syncwarp();  // every lane has read the values
        if (j + C::kStages < n) {
          issue(j + C::kStages, j >> 3, 1);
          v_issued = j + C::kStages + 1;
        }
      }
      if (u + 1 == item_end || j + 1 == n) {  // the item, or the warp's part of it, is done
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int s = 4; s < 32; s <<= 1) l[nt][h] += __shfl_xor_sync(0xffffffffu, l[nt][h], s);
        if (it.u0 >= ws && item_end <= we) {  // whole: straight to the output
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            const float i0 = row_inverse(l[nt][0]), i1 = row_inverse(l[nt][1]);
            const int r = 8 * nt + g;
            uint32_t* dst = reinterpret_cast<uint32_t*>(a.o + row_out(a, it.s.row0, it.head, r) * D);
#pragma unroll
            for (int k = 0; k < D / 16; ++k)
#pragma unroll
              for (int e = 0; e < 2; ++e) {  // a lane gets elements 16 k + 8 e + 2 t, + 1 of row g
                const uint32_t w = transpose8(pack_bf16x2(o[nt][k][2 * e] * i0, o[nt][k][2 * e + 1] * i1));
                if (r < it.rows) dst[8 * k + 4 * e + t] = w;
              }
            if (a.lse && g == 0)
#pragma unroll
              for (int h = 0; h < 2; ++h)
                if (8 * nt + 2 * t + h < it.rows) a.lse[row_out(a, it.s.row0, it.head, 8 * nt + 2 * t + h)] = row_lse(m[nt][h], l[nt][h]);
          }
        } else if (u + 1 < we) {  // began before this warp, ends in it: kept until the rings are idle
          stash(heads + warp * C::kPart);
          if (lane == 0) cuts[2 * warp] = Cut{it.u0, it.units, it.rows, it.s.row0, it.head};
        }
      }
    }
    if (!ok) {  // a wait gave up: the copies in flight must land before the ring is reused
      for (int j = max(0, k_issued - C::kStages); j < k_issued; ++j)
        mbar_wait(&kbar[j % C::kStages], (uint32_t)(j / C::kStages) & 1u, a.batch.status, kWaitLimitNs / 8);
      for (int j = max(0, v_issued - C::kStages); j < v_issued; ++j)
        mbar_wait(&vbar[j % C::kStages], (uint32_t)(j / C::kStages) & 1u, a.batch.status, kWaitLimitNs / 8);
    }
  }
  __syncthreads();  // all rings are idle: the partial results of the warps' last items go there
  float* tails = reinterpret_cast<float*>(ring_all);
  if (n > 0 && ok && !(it.u0 >= ws && it.u0 + it.units <= we)) {
    stash(tails + warp * C::kPart);
    if (lane == 0) cuts[2 * warp + 1] = Cut{it.u0, it.units, it.rows, it.s.row0, it.head};
  }
  __syncthreads();

  // Join the cut items, in range order: the entries of an item are neighbours, and the items'
  // groups of entries go to the warps in turn.  (All of the CTA's threads on one item after
  // another took 2-3 us an item.)
  auto part_of = [&](int e) -> const float* { return ((e & 1) ? tails : heads) + (e >> 1) * C::kPart; };
  {
    const int key = lane < 2 * kWarps ? cuts[lane].u0 : -1;
    const unsigned used = __ballot_sync(0xffffffffu, key >= 0);
    const unsigned before = used & ((1u << lane) - 1u);
    const int prev = __shfl_sync(0xffffffffu, key, before ? 31 - __clz(before) : lane);
    unsigned starts = __ballot_sync(0xffffffffu, key >= 0 && (!before || prev != key));
    for (int k = 0; starts; ++k) {
      const int e = __ffs(starts) - 1;
      starts &= starts - 1u;
      if (k % kWarps != warp) continue;
      const unsigned mine_mask = used & ~((1u << e) - 1u) & (starts ? (1u << (__ffs(starts) - 1)) - 1u : 0xffffffffu);
      const Cut x = cuts[e];
      const bool whole = x.u0 >= cs && x.u0 + x.units <= ce;
      float* mine = a.partials + (2 * (int64_t)blockIdx.x + (x.u0 < cs ? 0 : 1)) * C::kPart;
      if (lane < x.rows) {
        float mm = -INFINITY, ll = 0.f;
        for (unsigned s = mine_mask; s; s &= s - 1u) mm = fmaxf(mm, part_of(__ffs(s) - 1)[kRows * D + lane]);
        for (unsigned s = mine_mask; s; s &= s - 1u) {
          const float* p = part_of(__ffs(s) - 1) + kRows * D + lane;
          const float f = p[0] == -INFINITY && mm == -INFINITY ? 1.f : ex2(p[0] - mm);
          weight[__ffs(s) - 1][lane] = f;
          ll = fmaf(p[kRows], f, ll);
        }
        if (whole) {
          row_l[warp][lane] = ll;
          if (a.lse) a.lse[row_out(a, x.row0, x.head, lane)] = row_lse(mm, ll);
        } else {
          mine[kRows * D + lane] = mm;
          mine[kRows * D + kRows + lane] = ll;
        }
      }
      __syncwarp();
      const int pieces = x.rows * (D / 4);  // of four elements
      for (int i0 = lane; i0 < pieces; i0 += 128) {
        float4 v[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) v[q] = make_float4(0.f, 0.f, 0.f, 0.f);
        for (unsigned s = mine_mask; s; s &= s - 1u) {
          const int en = __ffs(s) - 1;
          const float4* p = reinterpret_cast<const float4*>(part_of(en));
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const int i = min(i0 + 32 * q, pieces - 1);
            const float4 w = p[i];
            const float f = weight[en][i / (D / 4)];
            v[q].x = fmaf(w.x, f, v[q].x);
            v[q].y = fmaf(w.y, f, v[q].y);
            v[q].z = fmaf(w.z, f, v[q].z);
            v[q].w = fmaf(w.w, f, v[q].w);
          }
        }
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const int i = i0 + 32 * q, r = i / (D / 4);
          if (i >= pieces) break;
          if (whole) {
            const float inv = row_inverse(row_l[warp][r]);
            reinterpret_cast<uint2*>(a.o + row_out(a, x.row0, x.head, r) * D)[i % (D / 4)] =
                make_uint2(pack_bf16x2(v[q].x * inv, v[q].y * inv), pack_bf16x2(v[q].z * inv, v[q].w * inv));
          } else {
            reinterpret_cast<float4*>(mine)[i] = v[q];
          }
        }
      }
      if (!whole) {  // the warp's stores, then its arrival (release; acquire for the last to arrive)
        __syncwarp();
        if (lane == 0) {
          const int c0 = owner_of(x.u0, (uint32_t)U, (uint32_t)G), c1 = owner_of(x.u0 + x.units - 1, (uint32_t)U, (uint32_t)G);
          complete[e] = atom_add_acq_rel_gpu(a.counters + c0, 1u) == (unsigned)(c1 - c0);
        }
      }
    }
  }
  __syncthreads();

  // items whose last part came from here: the whole CTA joins the CTAs' parts
  float* cta_weight = reinterpret_cast<float*>(ring_all + C::kHead);       // [kRows][kMaxSms]
  float4* sums = reinterpret_cast<float4*>(cta_weight + kRows * kMaxSms);  // [kThreads]
  for (int e = 0; e < 2 * kWarps; ++e) {
    if (!complete[e]) continue;
    const Cut x = cuts[e];
    const int c0 = owner_of(x.u0, (uint32_t)U, (uint32_t)G), c1 = owner_of(x.u0 + x.units - 1, (uint32_t)U, (uint32_t)G);
    if (tid == 0) a.counters[c0] = 0u;
    auto cta_part = [&](int c) -> const float* { return a.partials + (2 * (int64_t)c + (c == c0 ? 1 : 0)) * C::kPart; };
    // as many threads as fit share a piece of four elements, each every `share`-th part; the first
    // parts are on their way while the weights are made
    const int pieces = x.rows * (D / 4), share = pieces < kThreads ? kThreads / pieces : 1, per = kThreads / share;
    constexpr int kEarly = 8;
    float4 early[kEarly];
    {
      const int i = tid % per, k0 = tid / per;
#pragma unroll
      for (int s = 0; s < kEarly; ++s) {
        const int c = c0 + k0 + s * share;
        early[s] = i < pieces && k0 < share && c <= c1 ? __ldcg(reinterpret_cast<const float4*>(cta_part(c)) + i)
                                                       : make_float4(0.f, 0.f, 0.f, 0.f);
      }
    }
    // weights of the parts: a warp takes a row, its lanes the parts
    for (int r = warp; r < x.rows; r += kWarps) {
      constexpr int kSlots = kMaxSms / 32;
      float pm[kSlots], pl[kSlots], mm = -INFINITY, ll = 0.f;
#pragma unroll
      for (int s = 0; s < kSlots; ++s) {
        const int c = c0 + lane + 32 * s;
        pm[s] = c <= c1 ? __ldcg(cta_part(c) + kRows * D + r) : -INFINITY;
        pl[s] = c <= c1 ? __ldcg(cta_part(c) + kRows * D + kRows + r) : 0.f;
      }
#pragma unroll
      for (int s = 0; s < kSlots; ++s) mm = fmaxf(mm, pm[s]);
#pragma unroll
      for (int s = 16; s > 0; s >>= 1) mm = fmaxf(mm, __shfl_xor_sync(0xffffffffu, mm, s));
#pragma unroll
      for (int s = 0; s < kSlots; ++s) {
        const float f = pm[s] == -INFINITY && mm == -INFINITY ? 1.f : ex2(pm[s] - mm);
        cta_weight[r * kMaxSms + lane + 32 * s] = f;
        ll = fmaf(pl[s], f, ll);
      }
#pragma unroll
      for (int s = 16; s > 0; s >>= 1) ll += __shfl_xor_sync(0xffffffffu, ll, s);
      if (lane == 0) {
        row_l[0][r] = ll;
        if (a.lse) a.lse[row_out(a, x.row0, x.head, r)] = row_lse(mm, ll);
      }
    }
    __syncthreads();
    for (int i0 = 0; i0 < pieces; i0 += per) {
      const int i = i0 + tid % per, k0 = tid / per, r = i / (D / 4);
      float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
      if (i < pieces && k0 < share) {
        auto add = [&](const float4& p, int c) {
          const float f = cta_weight[r * kMaxSms + c - c0];
          v.x = fmaf(p.x, f, v.x);
          v.y = fmaf(p.y, f, v.y);
          v.z = fmaf(p.z, f, v.z);
          v.w = fmaf(p.w, f, v.w);
        };
        int c = c0 + k0;
        if (i0 == 0) {
#pragma unroll
          for (int s = 0; s < kEarly; ++s)
            if (c + s * share <= c1) add(early[s], c + s * share);
          c += kEarly * share;
        }
#pragma unroll 8
        for (; c <= c1; c += share) add(__ldcg(reinterpret_cast<const float4*>(cta_part(c)) + i), c);
      }
      if (share > 1) {
        sums[tid] = v;
        __syncthreads();
        if (i < pieces && k0 == 0)
          for (int k = 1; k < share; ++k) {
            const float4 p = sums[tid + k * per];
            v.x += p.x;
            v.y += p.y;
            v.z += p.z;
            v.w += p.w;
          }
      }
      if (i < pieces && k0 == 0) {
        const float inv = row_inverse(row_l[0][r]);
        reinterpret_cast<uint2*>(a.o + row_out(a, x.row0, x.head, r) * D)[i % (D / 4)] =
            make_uint2(pack_bf16x2(v.x * inv, v.y * inv), pack_bf16x2(v.z * inv, v.w * inv));
      }
    }
    __syncthreads();  // before the next item's weights
  }
}

template <int CODE, int D, int NT>
int launch(const KvAttendArgs& a, int sms, void* stream) {
  static std::atomic<uint64_t> done{0};
  auto kernel = kv_decode_kernel<CODE, D, NT>;
  static const size_t most = smem_bytes<D, NT>(kKvMaxSeqs);
  if (const int e = smem_attr_once(kernel, most, done)) return e;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)sms);
  cfg.blockDim = dim3(DecCfg<D, NT>::kThreads);
  cfg.dynamicSmemBytes = smem_bytes<D, NT>(a.batch.n_seqs);
  cfg.stream = (cudaStream_t)stream;
  cudaLaunchAttribute at{};
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = QLIN_USE_PDL;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  return (int)cudaLaunchKernelEx(&cfg, kernel, a);
}

template <int CODE, int D>
int launch_rows(const KvAttendArgs& a, int rows, int sms, void* stream) {
  return rows <= 8 ? launch<CODE, D, 1>(a, sms, stream) : launch<CODE, D, 2>(a, sms, stream);
}

}  // namespace

size_t kv_decode_partial_bytes(int head_dim, int sms) {
  return (size_t)sms * 2 * (size_t)(head_dim == 128 ? DecCfg<128, 2>::kPart : DecCfg<64, 2>::kPart) * 4;
}

int launch_kv_decode(int code, int head_dim, const KvAttendArgs& a, int rows, int sms, void* stream) {
  if (head_dim == 128)
    return code == kKvInt8 ? launch_rows<kKvInt8, 128>(a, rows, sms, stream) : launch_rows<kKvE4m3, 128>(a, rows, sms, stream);
  return code == kKvInt8 ? launch_rows<kKvInt8, 64>(a, rows, sms, stream) : launch_rows<kKvE4m3, 64>(a, rows, sms, stream);
}

}  // namespace qlin
