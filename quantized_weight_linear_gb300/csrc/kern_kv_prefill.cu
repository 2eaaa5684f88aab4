// Attention over the paged 8-bit cache for many query rows per key/value head (prompts, drafts),
// on the 5th-generation tensor cores.  The mathematics is that of kern_kv_decode.cu: products on
// the bare codes, both block scales on the exponent.  Here the keys' codes become bf16 (exact too),
// so that the queries are operands as they are; the values' codes fp16, like the weights.
//
// An item is 256 rows (tokens x query heads of one key/value head) against the tiles of eight blocks
// that they see.  The tiles of all items form one line that is cut into equal ranges, one per CTA
// of a grid of one per SM: causal, ragged and windowed work balances by itself, and few rows over
// many keys use the whole GPU.  A CTA walks its range; the pieces of an item that a cut leaves in
// several CTAs are put together by a second kernel, in CTA order.  The warps are specialised and
// run ahead of one another across items, so that an item's start (queries, first keys) hides
// behind the end of the one before:
//  * warp 0, scout: looks up the pages of the tiles ahead and puts their blocks' places and scales
//    into a table;
//  * warps 4-7 (keys) and 8-11 (values), converters: bytes from global memory to registers a tile
//    ahead, then 16-bit operands in shared memory, K-major with the 128-byte swizzle: keys
//    [128 tokens][D], values [D][128 tokens] (they are transposed in the cache already); once per
//    256 rows.  They bring an item's queries too (cp.async into the swizzled operand);
//  * warp 2: describes the next items;
//  * warps 1 and 3, MMA: S = Q K^T and O += P V in two lanes of work, so that the tensor cores are
//    busy with one while the softmax warps are with the other; P is read from TMEM.  With over 128
//    rows the lanes are the item's two tiles of 128 rows; with fewer they are its even and odd
//    tiles of keys, joined at the end;
//  * warps 12-15 and 16-19, softmax of the lanes: a thread owns a row: its scores from TMEM, the
//    running maximum, the exponentials, fp16 weights back to TMEM over the scores' own columns.  A
//    row's sums are rescaled only when its maximum grows by more than 2^8, in TMEM by the thread.
//
// TMEM columns: scores of the two lanes (128 each), sums (D each).  Shared memory at D = 128:
// queries 64 KB, five operand stages 160 KB.
//
// Bound by each lane's chain.  A tile of 128 keys and 256 rows takes 2048 tensor cycles; its MMAs read
// 192 KB of operands (1536 cycles of shared memory) and the converters write 64 KB more (512); but a
// lane's scores, softmax (2350 cycles) and product follow one another, since the weights take the scores'
// place: 4500 cycles in all, with no unit full.  4096 queries over 32768 tokens, 32 heads, 8 key heads of
// 128 (2.06 TFLOP): 1.75 ms, 1175 TFLOP/s, 0.62 of the bf16 rate (ncu: tensor pipe 45% active, issue
// 51%); the exponentials are not in the way (without them: 2% less).  Eight warps for the
// conversion, two 64-key halves for the weights and one range of tiles a CTA are what measured
// best against four warps, quarters, a tile of rows a CTA (ragged prompts 89 -> 77 us).
#include <cstddef>

#include "kern_kv.cuh"
#include "kern_umma.cuh"

namespace qlin {
namespace {

constexpr int kThreads = 640;
constexpr int kTileRows = 128;
constexpr int kCtaRows = 2 * kTileRows;
static_assert(kCtaRows == kKvPrefillRows, "row blocks");
constexpr int kTileKeys = 128;
constexpr int kTileBlocks = kTileKeys / kKvBlock;
constexpr int kSlots = 4;  // tiles in the table
constexpr int kSegs = 3;   // items in the table
constexpr int kItemCost = 2;  // what an item takes beside its tiles, in tiles (4: ragged prompts 4% slower)

// A block of a tile: its keys' scale times the softmax's, log2 and reciprocal of its values' scale, its cell of keys
// (in units of 16 D bytes; -1: no row needs the block)
struct BlockInfo {
  float ks, lvs, ivs;
  int cell;
};

// The part of an item in a CTA's range
struct Seg {
  int nt, t0;               // its tiles: t0, t0 + 1, ... of the item's
  int rows, row0;           // rows of the item, the first one's place among its sequence's rows
  int head, tok0, pos0;     // key/value head; first row in Q and position of the sequence's first token
  int sink_blocks, shift;  // tile t of the item holds blocks 8 t .. 8 t + 7, from sink_blocks on `shift` blocks later
  int part;                 // 0: the whole item, 1: its first piece, 2: another piece
};

// FEW: no sequence has over 128 rows a head.  Then the way of the keys' bytes into operands is the
// longest part of the chain: the registers go to the converters, and the softmax warps read the
// scores in two halves (five drafts of 16 sequences: 97 -> 78 us; the same split costs a prompt chunk
// 11%).  Now 75 us, with no unit full: DRAM 31%, tensor pipe 25%, issue 38%, 40 of a tile's 128 rows used.
template <int D, bool FEW>
struct PreSmem {
  static constexpr int kOps = D == 128 ? 5 : 8;  // 16-bit operand stages
  __align__(1024) uint8_t q[FEW ? 1 : 2][D / 64][kTileRows * 128];
  __align__(1024) uint8_t op[kOps][D * kTileKeys * 2];
  __align__(16) BlockInfo info[kSlots][kTileBlocks];
  __align__(16) Seg seg[kSegs];
  float2 other[kTileRows];            // M and L of the lane with the odd tiles
  int tail[kSlots];                   // tokens of the tile that the sequence has, | its blocks without values << 16
  uint64_t op_full[kOps], op_empty[kOps], info_full[kSlots], info_empty[kSlots];
  uint64_t q_full[kSegs], q_empty, seg_full[kSegs], seg_empty[kSegs], s_full[2], p_full[2][2], o_full[2], o_empty[2], other_full;  // p_full: halves of 64 keys
  int start[3];  // row block, head, tile where the CTA's range begins
  int64_t tiles_at[2];  // tiles of the line before the range, and up to its end
  uint32_t tmem;
};
// (sizeof is rounded up to the alignment)
template <int D, bool FEW>
constexpr size_t pre_smem_bytes() {
  using S = PreSmem<D, FEW>;
  return offsetof(S, tmem) + 4;
}

// A cut item, described by the CTA that has its first piece, for the joining kernel
struct PreCut {
  int rows, row0, head, tok0, last_cta;  // rows = 0: none
};

struct PreArgs {
  KvAttendArgs a;
  PreCut* cuts;    // [grid]
  float* parts;    // [grid][2]: pieces of the CTA's first and last item, each O [256][D], M [256], L [256]
  int row_blocks;  // upper bound of the row blocks of all sequences
};

// Registers: the launch gives every warp 96; the softmax warps hold a row's scores.  (-Xptxas -v, spill
// stores at head size 128: 128 bytes for int8, 148 for e4m3, 16 and 32 with FEW; at 64 up to 24.  Other
// splits of the registers measured slower.)
template <int N>
__device__ __forceinline__ void regs_inc() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N)); }
template <int N>
__device__ __forceinline__ void regs_dec() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N)); }
template <bool FEW>
struct Regs {  // warps 0-3, 4-11, 12-19
  static constexpr int kIssue = FEW ? 64 : 56, kConvert = FEW ? 72 : 48, kSoftmax = FEW ? 104 : 160;
  static_assert(128 * kIssue + 256 * kConvert + 256 * kSoftmax <= kThreads * 96, "registers of the launch");
};

// 32 columns of the warp's TMEM lanes, without waiting
__device__ __forceinline__ void tmem_ld32_start(uint32_t taddr, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
        "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
        "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr));
}
// Waits for the warp's TMEM loads; the values pass through, so that no use moves above the wait
__device__ __forceinline__ void tmem_ld32_wait(uint32_t* r) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
      : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
        "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]),
        "+r"(r[16]), "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]), "+r"(r[22]), "+r"(r[23]),
        "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]), "+r"(r[29]), "+r"(r[30]), "+r"(r[31])
      :: "memory");
}
// 16 columns, without waiting
__device__ __forceinline__ void tmem_st16_start(uint32_t taddr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// 32 bytes, aligned to 32
__device__ __forceinline__ void store32(void* at, const uint32_t* r) {
  asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(at), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]),
               "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
               : "memory");
}

// One lane of a converged warp.  (The MMAs are issued under this, not under lane == 0: with the
// warp's control flow uniform their operands stay in uniform registers.  Issuing eight MMAs from
// a lane == 0 branch took 1300 cycles, twice what they take to run.)
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}" : "=r"(p));
  return p != 0;
}

// mbarrier arrival that counts for n
__device__ __forceinline__ void mbar_arrive_n(uint64_t* bar, uint32_t n) {
  asm volatile("{\n .reg .b64 st;\n mbarrier.arrive.shared::cta.b64 st, [%0], %1;\n}" ::"r"(smem_u32(bar)), "r"(n) : "memory");
}

// The bits under n (none for n <= 0, all from 32 on)
__device__ __forceinline__ uint32_t bits_below(int n) { return n <= 0 ? 0u : n >= 32 ? 0xFFFFFFFFu : (1u << n) - 1u; }

// Two fp32 operations in one instruction
__device__ __forceinline__ uint64_t pack2(float lo, float hi) {
  uint64_t d;
  asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "f"(lo), "f"(hi));
  return d;
}
__device__ __forceinline__ void unpack2(uint64_t d, float& lo, float& hi) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(d));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

// 256 rows of a sequence
struct RowBlock {
  KvSeq s;  // kv: visible keys end there for these rows
  Visible vis;
  int tiles;            // of eight visible blocks, in order (the sinks' and the window's may share one)
  int seq, row0, rows;  // rows = 0: none, or a sequence of another launch
};

// Sequence s owns the row blocks from q_start[s] * group / 256 + s on
__device__ __forceinline__ int64_t first_row_block(const KvAttendArgs& a, int s) {
  return (int64_t)__ldg(a.batch.q_start + s) * a.group / kCtaRows + s;
}

__device__ __forceinline__ RowBlock row_block(const KvAttendArgs& a, int seq, int ub) {
  RowBlock b;
  b.seq = seq;
  b.s = kv_seq(a.batch, seq);
  b.rows = b.row0 = b.tiles = 0;
  b.vis = Visible{0, 0, 0};
  const int64_t j = ub - first_row_block(a, seq);
  const int all = b.s.n * a.group;
  if (all < a.min_rows || j < 0 || j * kCtaRows >= all) return b;
  b.row0 = (int)j * kCtaRows;
  b.rows = min(kCtaRows, all - b.row0);
  // the keys that these rows see
  KvSeq rows = b.s;
  const int t0 = b.row0 / a.group, t1 = (b.row0 + b.rows - 1) / a.group;
  rows.pos0 = b.s.pos0 + t0;
  rows.kv = max(b.s.pos0 + t1 + 1, 0);
  rows.n = t1 - t0 + 1;
  b.vis = visible_blocks(rows, a.window, a.sinks);
  b.tiles = (b.vis.n + kTileBlocks - 1) / kTileBlocks;
  b.s.kv = rows.kv;
  return b;
}

// Walks the items of a CTA's range of the line (a whole warp)
struct Walk {
  RowBlock b;
  int ub, head, t0, t1;  // the current item, its tiles in the range
  int64_t left;          // tiles of the range after these
  __device__ __forceinline__ void load(const KvAttendArgs& a, int lane) {
    int lo = 0, hi = a.batch.n_seqs;
    while (hi - lo > 1) {
      const int step = (hi - lo + 31) / 32, s = lo + lane * step;
      const unsigned m = __ballot_sync(0xffffffffu, s < hi && first_row_block(a, s) <= ub);
      const int k = m ? 31 - __clz(m) : 0;
      lo += k * step;
      hi = min(lo + step, hi);
    }
    b = row_block(a, lo, ub);
  }
  __device__ __forceinline__ void start(const KvAttendArgs& a, int ub_, int head_, int tile, int64_t tiles, int lane) {
    ub = ub_;
    head = head_;
    t0 = tile;
    load(a, lane);
    t1 = (int)min((int64_t)b.tiles, tile + tiles);
    left = tiles - (t1 - t0);
  }
  __device__ __forceinline__ bool next(const PreArgs& p, int lane) {
    if (left == 0) return false;
    if (++head == p.a.cache.n_heads) {
      head = 0;
      do {
        if (++ub >= p.row_blocks) return false;  // (the range ends before)
        load(p.a, lane);
      } while (b.tiles == 0);
    }
    t0 = 0;
    t1 = (int)min((int64_t)b.tiles, left);
    left -= t1;
    return true;
  }
};

__device__ __forceinline__ int64_t pre_row_out(const KvAttendArgs& a, int tok0, int head, int q) {
  return (int64_t)(tok0 + q / a.group) * (a.cache.n_heads * a.group) + head * a.group + q % a.group;
}

template <int CODE, int D, bool FEW>
__global__ void __launch_bounds__(kThreads, 1) kv_prefill_kernel(const PreArgs p) {
  using SM = PreSmem<D, FEW>;
  using R = Regs<FEW>;
  constexpr int kOps = SM::kOps;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  SM& sm = *reinterpret_cast<SM*>(smem_raw);
  const KvAttendArgs& a = p.a;
  int32_t* status = a.batch.status;
  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
  const int H = a.cache.n_heads;
  int64_t* scan = reinterpret_cast<int64_t*>(sm.other);  // [20][2] (before it holds anything else)
  int* start = sm.start;

  if (tid == 0) {
    for (int s = 0; s < kOps; ++s) {
      mbar_init(&sm.op_full[s], 4);
      mbar_init(&sm.op_empty[s], 2);
    }
    for (int s = 0; s < kSlots; ++s) {
      mbar_init(&sm.info_full[s], 1);
      mbar_init(&sm.info_empty[s], 8 + 8);  // converters; softmax warps of both lanes, or of one for two each
    }
    for (int s = 0; s < kSegs; ++s) {
      mbar_init(&sm.q_full[s], 8);
      mbar_init(&sm.seg_full[s], 1);
      mbar_init(&sm.seg_empty[s], 8 + 8 + 2);  // converters, softmax and MMA warps
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sm.s_full[i], 1);
      mbar_init(&sm.p_full[i][0], 4);
      mbar_init(&sm.p_full[i][1], 4);
      mbar_init(&sm.o_empty[i], 4);
      mbar_init(&sm.o_full[i], 1);
    }
    mbar_init(&sm.q_empty, 2);
    mbar_init(&sm.other_full, 4);
    fence_mbar_init();
    sm.tmem = 0xffffffffu;
  }
  pdl_wait();
  if (tid == 0) pdl_launch_dependents();

  // ---- the line: a thread counts `per` neighbouring row blocks
  const int per = (p.row_blocks + kThreads - 1) / kThreads, u0 = min(tid * per, p.row_blocks), u1 = min(u0 + per, p.row_blocks);
  auto seq_at = [&](int ub) {
    int lo = 0, hi = a.batch.n_seqs;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (first_row_block(a, mid) <= ub) lo = mid; else hi = mid;
    }
    return lo;
  };
  const int seq0 = u0 < u1 ? seq_at(u0) : 0;
  // places of the line and tiles: an item takes kItemCost places before its tiles'
  int64_t places = 0, tiles = 0;
  bool blind = false;  // rows that see no key
  for (int ub = u0, seq = seq0; ub < u1; ++ub) {
    while (seq + 1 < a.batch.n_seqs && first_row_block(a, seq + 1) <= ub) ++seq;
    const RowBlock b = row_block(a, seq, ub);
    if (b.tiles) places += (int64_t)(b.tiles + kItemCost) * H;
    tiles += (int64_t)b.tiles * H;
    blind |= b.rows > 0 && b.tiles == 0;
  }
  int64_t x = places, xt = tiles;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t y = __shfl_up_sync(0xffffffffu, x, o), yt = __shfl_up_sync(0xffffffffu, xt, o);
    if (lane >= o) {
      x += y;
      xt += yt;
    }
  }
  // where q_start falls, the line and the items would not match: the sum of the tiles becomes negative
  // (a return from here instead cost registers: a prompt chunk 1760 -> 2360 us)
  bool falls = false;
  for (int s = tid; s < a.batch.n_seqs; s += kThreads) falls |= kv_falls(a.batch, s);
  if (__any_sync(0xffffffffu, falls)) {
    kv_report(status, kStatusInvalid);
    xt = -((int64_t)1 << 57);
  }
  if (lane == 31) {
    scan[2 * warp] = x;
    scan[2 * warp + 1] = xt;
  }
  const bool any_blind = __syncthreads_or(blind);
  int64_t before = x - places, tiles_before = xt - tiles, U = 0, all_tiles = 0;
  for (int w = 0; w < kThreads / 32; ++w) {
    if (w < warp) {
      before += scan[2 * w];
      tiles_before += scan[2 * w + 1];
    }
    U += scan[2 * w];
    all_tiles += scan[2 * w + 1];
  }
  // at least two tiles a CTA
  const int64_t G = all_tiles < 0 ? 0 : max((int64_t)1, min((int64_t)gridDim.x, U / (kItemCost + 2)));
  if (blockIdx.x < G) {
    for (int e = 0; e < 2; ++e) {  // the range's begin and end
      const int64_t at = split_start(blockIdx.x + e, U, G);
      if (at == U && tid == 0) sm.tiles_at[e] = all_tiles;
      if (at < before || at >= before + places) continue;
      int64_t b = before, bt = tiles_before;
      for (int ub = u0, seq = seq0; ub < u1; ++ub) {
        while (seq + 1 < a.batch.n_seqs && first_row_block(a, seq + 1) <= ub) ++seq;
        const int n = row_block(a, seq, ub).tiles;
        if (n == 0) continue;
        const int64_t len = n + kItemCost;
        if (at < b + len * H) {
          const int head = (int)((at - b) / len), tile = max((int)((at - b) % len) - kItemCost, 0);
          sm.tiles_at[e] = bt + (int64_t)head * n + tile;
          if (e == 0) {
            sm.start[0] = ub;
            sm.start[1] = head;
            sm.start[2] = tile;
          }
          break;
        }
        b += len * H;
        bt += (int64_t)n * H;
      }
    }
  }
  __syncthreads();
  const int64_t ce = blockIdx.x < G ? split_start(blockIdx.x + 1, U, G) : U;
  const int total = blockIdx.x < G ? (int)(sm.tiles_at[1] - sm.tiles_at[0]) : 0;  // tiles of this CTA
  if (tid == 0) p.cuts[blockIdx.x].rows = 0;
  if (any_blind)
    for (int ub = blockIdx.x; ub < p.row_blocks; ub += (int)gridDim.x) {
      const RowBlock b = row_block(a, seq_at(ub), ub);
      if (b.rows == 0 || b.tiles > 0) continue;
      for (int64_t i = tid; i < (int64_t)b.rows * H * (D / 8); i += kThreads) {
        const int64_t row = pre_row_out(a, b.s.row0, (int)(i / (D / 8) % H), b.row0 + (int)(i / (D / 8) / H));
        reinterpret_cast<uint4*>(a.o + row * D)[i % (D / 8)] = make_uint4(0u, 0u, 0u, 0u);
        if (a.lse && i % (D / 8) == 0) a.lse[row] = -INFINITY;
      }
    }
  if (total == 0) return;
  if (smem_u32(smem_raw) & 1023u) {  // the operands' swizzle needs it; dynamic shared memory starts so
    if (tid == 0) kv_report(status, kStatusInternal);
    return;
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&sm.tmem)), "r"(512u)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sm.tmem;
  bool ok = true;

  if (warp < 4) regs_dec<R::kIssue>();
  if (warp == 0) {
    // ------------------------------------------------------------------ scout
    // lane i < 8 looks after block i of a tile
    Walk w;
    w.start(a, start[0], start[1], start[2], total, lane);
    int t = w.t0;
    bool more = true;
    struct Ahead {
      int blk, page, head, tail;
    };
    auto look = [&]() -> Ahead {  // the next tile
      Ahead h{-1, -1, 0, 0};
      if (more && t == w.t1) {
        more = w.next(p, lane);
        t = w.t0;
      }
      if (!more) return h;
      const int first = t++ * kTileBlocks, i = first + (lane & 7);
      h.head = w.head;
      h.tail = w.b.s.kv - (first + w.b.vis.wb - w.b.vis.sb) * kKvBlock;
      if (i < w.b.vis.n) {
        h.blk = w.b.vis.block(i);
        const int col = h.blk / a.cache.page_blocks;
        if (col < a.batch.pages_width) h.page = __ldg(a.batch.pages + (int64_t)w.b.seq * a.batch.pages_stride + col);
      }
      return h;
    };
    auto cell_at = [&](const Ahead& h) -> int {
      if (h.blk < 0) return -1;
      int page = h.page;
      if (page < 0 || page >= a.cache.n_pages) {
        kv_report(status, kStatusInvalid);
        page = 0;
      }
      return (page * H + h.head) * 2 * a.cache.page_blocks + h.blk % a.cache.page_blocks;
    };
    auto scales_at = [&](int cell) -> float2 {
      if (cell < 0) return make_float2(1.f, 1.f);
      const int ph = cell / (2 * a.cache.page_blocks), r = cell % (2 * a.cache.page_blocks);
      return __ldcg(reinterpret_cast<const float2*>(a.cache.scales) + (int64_t)ph * a.cache.page_blocks + r);
    };
    // Step j writes tile j's entry; the scales of tile j + 1 and the page of tile j + 3 are asked for, and the
    // cells of tile j + 2 are brought into L2 for the converters' loads
    Ahead h[3];
    int cell[3];
    for (int k = 0; k < 3; ++k) h[k] = look();
    cell[0] = cell_at(h[0]);
    cell[1] = cell_at(h[1]);
    float2 sc = scales_at(cell[0]);
    for (int j = 0; j < total && ok; ++j) {
      const int slot = j % kSlots;
      const Ahead next = look();
      const float2 sc1 = scales_at(cell[1]);
      cell[2] = cell_at(h[2]);
      if (cell[2] >= 0 && lane < kTileBlocks) {
        const uint8_t* src = a.cache.codes + (int64_t)cell[2] * kKvCellBytes<D>;
        asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(src), "r"(kKvCellBytes<D>));
        asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(src + (int64_t)a.cache.page_blocks * kKvCellBytes<D>),
                     "r"(kKvCellBytes<D>));
      }
      ok = mbar_wait(&sm.info_empty[slot], ((uint32_t)(j / kSlots) & 1u) ^ 1u, status);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      const float vs = kv_value_scale(sc.y), ivs = 1.f / vs;
      const unsigned none = __ballot_sync(0xffffffffu, kv_no_values(ivs)) & ((1u << kTileBlocks) - 1u);
      if (lane < kTileBlocks) sm.info[slot][lane] = BlockInfo{fmaxf(sc.x * a.scale, 1e-37f), log2f(vs), ivs, cell[0]};
      if (lane == 0) sm.tail[slot] = min(max(h[0].tail, 0), kTileKeys) | (int)none << 16;
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm.info_full[slot]);
      h[0] = h[1];
      h[1] = h[2];
      h[2] = next;
      cell[0] = cell[1];
      cell[1] = cell[2];
      sc = sc1;
    }
  } else if (warp == 1 || warp == 3) {
    // ------------------------------------------------------------------ MMA issuers, one a lane of work
    // (The whole warp waits and counts, one elected lane issues.  Issuing blocks while the tensor
    // cores have work queued, so with one warp for both lanes its waits between the MMAs left them
    // idle.)  A job is a tile of keys for one lane: its scores, then its product, whose weights the
    // next job's scores overwrite.  Of an item of over 128 rows both lanes take every tile, else in
    // turn, going on across items.
    constexpr uint32_t idesc_s = idesc_f16(1, kTileKeys, kTileRows), idesc_o = idesc_f16(0, D, kTileRows);
    const int ln = warp >> 1;
    const uint32_t s_at = tmem + 128u * ln, o_at = tmem + 256u + (uint32_t)D * ln;
    const uint64_t dq0 = umma_desc_sw128(sm.q[0][0]), dop = umma_desc_sw128(sm.op[0]);
    auto wait = [&](uint64_t* bar, int phase) -> bool {
      return __all_sync(0xffffffffu, mbar_wait(bar, (uint32_t)phase & 1u, status));
    };
    uint32_t p_phase = 0;
    int parity = 0;  // lane of the item's first job
    for (int seg = 0, done = 0; done < total && ok; ++seg) {
      const int slot = seg % kSegs;
      ok = wait(&sm.q_full[slot], seg / kSegs);
      if (!ok) break;
      const int nt = sm.seg[slot].nt;
      const bool dual = !FEW && sm.seg[slot].rows > kTileRows;
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm.seg_empty[slot]);
      const int mine = ln ^ parity, step = dual ? 1 : 2, first = dual ? 0 : mine;
      const uint64_t dq = dq0 + (uint64_t)(dual ? mine * (int)(sizeof(sm.q[0]) >> 4) : 0);
      for (int j = first; j < nt && ok; j += step) {
        const bool last = j + step >= nt;
        const int ku = 2 * (done + j), vu = ku + 1, ks = ku % kOps, vs = vu % kOps;
        ok = wait(&sm.op_full[ks], ku / kOps);
        if (!ok) break;
        tc_fence_after();
        if (elect_one()) {
          const uint64_t dk = dop + (uint64_t)(ks * (int)(sizeof(sm.op[0]) >> 4));
#pragma unroll
          for (int h = 0; h < D / 64; ++h)
#pragma unroll
            for (int k = 0; k < 4; ++k)
              umma_f16(s_at, dq + (uint64_t)(h * (kTileRows * 128 >> 4) + 2 * k), dk + (uint64_t)(h * (kTileKeys * 128 >> 4) + 2 * k),
                       idesc_s, (h | k) ? 1u : 0u);
          umma_commit(&sm.s_full[ln]);
          umma_commit(&sm.op_empty[ks]);
          if (!dual) umma_commit(&sm.op_empty[ks]);  // for the other lane, which skips the tile
          if (last) umma_commit(&sm.q_empty);
        }
        __syncwarp();
        // the lane's sums of the item before have been read
        ok = wait(&sm.op_full[vs], vu / kOps) && (j > first || seg == 0 || wait(&sm.o_empty[ln], seg - 1));
        if (!ok) break;
#pragma unroll
        for (int h = 0; h < 2; ++h) {  // as soon as the weights of 64 keys are there
          ok = wait(&sm.p_full[ln][h], (int)p_phase);
          if (!ok) break;
          tc_fence_after();
          if (elect_one()) {
            const uint64_t dv = dop + (uint64_t)(vs * (int)(sizeof(sm.op[0]) >> 4));
#pragma unroll
            for (int k = 0; k < 4; ++k)
              umma_f16_ta(o_at, s_at + 32u * h + 8u * k, dv + (uint64_t)(h * (D * 128 >> 4) + 2 * k), idesc_o,
                          j == first && (h | k) == 0 ? 0u : 1u);
            if (h == 1) {
              umma_commit(&sm.op_empty[vs]);
              if (!dual) umma_commit(&sm.op_empty[vs]);
              if (last) umma_commit(&sm.o_full[ln]);
            }
          }
          __syncwarp();
        }
        p_phase ^= 1u;
      }
      if (ok && first >= nt) {  // one tile, and the other lane has it
        ok = seg == 0 || wait(&sm.o_empty[ln], seg - 1);
        if (lane == 0) {
          mbar_arrive(&sm.q_empty);
          mbar_arrive(&sm.o_full[ln]);
        }
        __syncwarp();
      }
      done += nt;
      if (!dual) parity ^= nt & 1;
    }
    if (!ok) {  // what was issued must not outlive the kernel
      if (elect_one()) umma_commit(&sm.o_full[ln]);
      __syncwarp();
      const uint64_t t0 = global_ns();
      while (global_ns() - t0 < kWaitLimitNs / 100) {}
    }
  } else if (warp == 2) {
    // ------------------------------------------------------------------ items
    Walk w;
    w.start(a, start[0], start[1], start[2], total, lane);
    bool more = true;
    for (int seg = 0; ok && more; ++seg) {
      const int slot = seg % kSegs;
      ok = seg < kSegs || mbar_wait(&sm.seg_empty[slot], (uint32_t)(seg / kSegs - 1) & 1u, status);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      if (lane == 0) {
        Seg& g = sm.seg[slot];
        g.nt = w.t1 - w.t0;
        g.t0 = w.t0;
        g.rows = w.b.rows;
        g.row0 = w.b.row0;
        g.head = w.head;
        g.tok0 = w.b.s.row0;
        g.pos0 = w.b.s.pos0;
        g.shift = w.b.vis.wb - w.b.vis.sb;
        g.sink_blocks = g.shift ? w.b.vis.sb : 0;
        g.part = w.t0 == 0 ? (w.t1 == w.b.tiles ? 0 : 1) : 2;
        if (g.part == 1)
          // the range ends before its tile t1, so its last tile's place is ce + n - t1 - 1
          p.cuts[blockIdx.x] = PreCut{w.b.rows, w.b.row0, w.head, w.b.s.row0,
                                      (int)min(split_owner(ce + w.b.tiles - w.t1 - 1, U, G), G - 1)};
        mbar_arrive(&sm.seg_full[slot]);
      }
      more = w.next(p, lane);
    }
  } else if (warp < 12) {
    // ------------------------------------------------------------------ converters
    // A piece is 16 bytes: 16 elements of a key, or the 16 tokens of a value element; it becomes
    // two 16-byte chunks of its operand row.  Thread ct takes pieces ct, ct + 128, ...
    regs_dec<R::kConvert>();
    const bool values = warp >= 8;
    const int ct = tid & 127;
    constexpr int kPieces = kTileKeys * D / 16 / 128;
    constexpr uint32_t kZero = kv_zero_codes(CODE);
    // Key pieces: four lanes take 64 bytes of a key, so that the eight lanes of a store's phase are
    // two neighbouring keys, whose swizzles differ in the lowest bit: all banks, no conflicts.
    constexpr int kHalves = D / 64;
    const int krow = ct / 4, kc = ct % 4;
    const uint32_t kd0 = (uint32_t)(krow * 128 + (((2 * kc) ^ (krow & 7)) << 4));
    const uint32_t kd1 = (uint32_t)(krow * 128 + (((2 * kc + 1) ^ (krow & 7)) << 4));
    auto half8 = [&](uint32_t x, uint32_t y) -> uint4 {
      uint4 h;
      kv_to_half<CODE>(x, h.x, h.y);
      kv_to_half<CODE>(y, h.z, h.w);
      return h;
    };
    auto bf8 = [&](uint32_t x, uint32_t y) -> uint4 {
      uint4 h;
      kv_to_bf16<CODE>(x, h.x, h.y);
      kv_to_bf16<CODE>(y, h.z, h.w);
      return h;
    };
    // block of piece i of a tile: the pieces of a cell are neighbours
    auto block_at = [&](int i) { return (i * 128 + ct) / D; };
    uint4 w[kPieces];
    int tail = kTileKeys;
    auto load = [&](int j) -> bool {  // tile j's bytes; then its entry of the table is through
      const int slot = j % kSlots;
      if (!__all_sync(0xffffffffu, mbar_wait(&sm.info_full[slot], (uint32_t)(j / kSlots) & 1u, status))) return false;
#pragma unroll
      for (int i = 0; i < kPieces; ++i) {
        // keys: piece i is half i % kHalves of key krow + 32 (i / kHalves)
        const int cell = sm.info[slot][values ? block_at(i) : 2 * (i / kHalves) + krow / 16].cell;
        const int at = values ? (i * 128 + ct) % D : (krow % 16) * (D / 16) + 4 * (i % kHalves) + kc;
        w[i] = cell < 0 ? make_uint4(0u, 0u, 0u, 0u)
                        : __ldcg(reinterpret_cast<const uint4*>(a.cache.codes + ((int64_t)cell + (values ? a.cache.page_blocks : 0)) *
                                                                                     kKvCellBytes<D>) + at);
      }
      // blocks without values: cleared here, or with the tail's bytes (each where it measured better: as below
      // for both codes a prompt chunk of int8 takes 1780 us instead of 1747, as here a window prompt of e4m3
      // 233 instead of 209)
      if constexpr (CODE == kKvE4m3) {
        tail = sm.tail[slot];
      } else if (const int none = sm.tail[slot] >> 16; values && none) {
#pragma unroll
        for (int i = 0; i < kPieces; ++i)
          if (none >> block_at(i) & 1) w[i] = make_uint4(kZero, kZero, kZero, kZero);
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm.info_empty[slot]);
      return true;
    };
    auto convert = [&](int j) -> bool {
      const int n = 2 * j + (values ? 1 : 0);  // unit
      if (!__all_sync(0xffffffffu, mbar_wait(&sm.op_empty[n % kOps], ((uint32_t)(n / kOps) & 1u) ^ 1u, status))) return false;
      uint8_t* op = sm.op[n % kOps];
      if (!values) {
#pragma unroll
        for (int i = 0; i < kPieces; ++i) {
          const uint4 lo = bf8(w[i].x, w[i].y), hi = bf8(w[i].z, w[i].w);
          uint8_t* dst = op + (i % kHalves) * kTileKeys * 128 + (i / kHalves) * 32 * 128;
          *reinterpret_cast<uint4*>(dst + kd0) = lo;
          *reinterpret_cast<uint4*>(dst + kd1) = hi;
        }
      } else {
        // e4m3: bytes behind the sequence's end may be NaN and are cleared (a NaN key is masked)
        if (CODE == kKvE4m3 && tail != kTileKeys) {
#pragma unroll
          for (int i = 0; i < kPieces; ++i) {
            w[i] = kv_first_bytes(w[i], (tail & 0xFFFF) - block_at(i) * kKvBlock);
            if (tail >> (16 + block_at(i)) & 1) w[i] = make_uint4(kZero, kZero, kZero, kZero);
          }
        }
#pragma unroll
        for (int i = 0; i < kPieces; ++i) {
          const int row = (i * 128 + ct) % D, b = block_at(i);  // element, block of the tile
          uint8_t* dst = op + (b / 4) * D * 128 + row * 128;
          *reinterpret_cast<uint4*>(dst + (((2 * (b % 4)) ^ (row & 7)) << 4)) = half8(w[i].x, w[i].y);
          *reinterpret_cast<uint4*>(dst + (((2 * (b % 4) + 1) ^ (row & 7)) << 4)) = half8(w[i].z, w[i].w);
        }
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm.op_full[n % kOps]);  // the warp's part of the unit is written
      return true;
    };
    // The next item's queries, by all converters (one warp alone took 8 us for 64 KB, which nothing
    // hid): a thread copies one 16-byte piece of every kRowsAtOnce-th row; its source moves on by a
    // step, and by another where the row passes the last head of a token
    int seg = 0, next_item = 0;  // items so far, the tile where the next one begins
    auto queries = [&]() -> bool {
      const int slot = seg % kSegs;
      const bool there = mbar_wait(&sm.seg_full[slot], (uint32_t)(seg / kSegs) & 1u, status) &&
                         (seg == 0 || mbar_wait(&sm.q_empty, (uint32_t)(seg - 1) & 1u, status));  // the item before has its scores
      if (!__all_sync(0xffffffffu, there)) return false;
      const Seg& g = sm.seg[slot];
      constexpr int kPieces = D / 8, kRowsAtOnce = 256 / kPieces;
      const int piece = (tid - 128) % kPieces, first_row = (tid - 128) / kPieces;
      const int rows = g.rows, tiles = !FEW && rows > kTileRows ? 2 : 1, q0 = g.row0 + first_row;
      int head = q0 % a.group;
      const uint16_t* src = a.q.data + (int64_t)(g.tok0 + q0 / a.group) * a.q.token_stride +
                            (int64_t)(g.head * a.group + head) * a.q.head_stride + 8 * piece;
      const int dhead = kRowsAtOnce % a.group;
      const int64_t step = (int64_t)(kRowsAtOnce / a.group) * a.q.token_stride + (int64_t)dhead * a.q.head_stride;
      const int64_t wrap = a.q.token_stride - (int64_t)a.group * a.q.head_stride;
      uint32_t dst = smem_u32(sm.q[0][piece / 8]) + (uint32_t)(first_row * 128 + (((piece % 8) ^ (first_row & 7)) << 4));
      int left = rows - first_row;  // rows from here on are zeros
#pragma unroll 1
      for (int tile = 0; tile < tiles; ++tile) {
#pragma unroll 4
        for (int k = 0; k < kTileRows / kRowsAtOnce; ++k) {
          asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst + (uint32_t)(k * kRowsAtOnce * 128)),
                       "l"(left > 0 ? src : a.q.data), "r"(left > 0 ? 16 : 0)
                       : "memory");
          left -= kRowsAtOnce;
          src += step;
          head += dhead;
          if (head >= a.group) {
            head -= a.group;
            src += wrap;
          }
        }
        dst += (uint32_t)sizeof(sm.q[0]);
      }
      next_item += g.nt;
      ++seg;
      return true;
    };
    auto queries_there = [&]() {
      asm volatile("cp.async.wait_all;" ::: "memory");
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(&sm.q_full[(seg - 1) % kSegs]);
        mbar_arrive(&sm.seg_empty[(seg - 1) % kSegs]);
      }
    };
    ok = queries() && load(0);
    if (ok) queries_there();
    // An item's queries follow its first tile: by then the stages are full, and the tensor cores
    // are about to be through with the queries before
    for (int j = 0; j < total && ok; ++j) {
      ok = convert(j);
      const bool item = j == next_item;
      if (ok && item) ok = queries();
      if (ok && j + 1 < total) ok = load(j + 1);
      if (ok && item) queries_there();
    }
  } else {
    // ------------------------------------------------------------------ softmax
    regs_inc<R::kSoftmax>();
    const int ln = (warp - 12) >> 2, quad = warp & 3;  // lane of work, TMEM lane quadrant
    const uint32_t tm = tmem + ((uint32_t)(32 * quad) << 16);
    const uint32_t s_col = tm + 128u * ln, o_col = tm + 256u + (uint32_t)D * ln;
    uint32_t s_phase = 0, other_phase = 0;
    int parity = 0;  // lane of the item's first job
    for (int seg = 0, done = 0; done < total && ok; ++seg) {
      ok = __all_sync(0xffffffffu, mbar_wait(&sm.seg_full[seg % kSegs], (uint32_t)(seg / kSegs) & 1u, status));
      if (!ok) break;
      const Seg& g = sm.seg[seg % kSegs];
      const bool dual = !FEW && g.rows > kTileRows;
      const int mine = ln ^ parity;  // 256 rows: tile of rows; else: first tile of keys
      const int warp_row = (dual ? mine * kTileRows : 0) + 32 * quad, r = warp_row + lane;
      const bool live = warp_row < g.rows;  // some row of the warp exists
      float m = -INFINITY, l = 0.f;
      const int pos = g.pos0 + (g.row0 + r) / a.group;
      const int p_first = g.pos0 + (g.row0 + warp_row) / a.group;
      const int p_last = g.pos0 + (g.row0 + min(warp_row + 31, g.rows - 1)) / a.group;
      const int lo = a.window > 0 ? pos - a.window : -1;  // keys up to lo are outside the window
      bool first = true;
      for (int j = dual ? 0 : mine; j < g.nt && ok; j += dual ? 1 : 2) {
        const int slot = (done + j) % kSlots;
        ok = mbar_wait(&sm.info_full[slot], (uint32_t)((done + j) / kSlots) & 1u, status) &&
             mbar_wait(&sm.s_full[ln], s_phase, status);
        ok = __all_sync(0xffffffffu, ok);  // the TMEM accesses below are the whole warp's
        if (!ok) break;
        s_phase ^= 1u;
        tc_fence_after();
        if (live) {
          const float4* info = reinterpret_cast<const float4*>(sm.info[slot]);
          // position of the tile's column c: c < split: sink_tok + c, else tok + c
          const int sink_tok = (g.t0 + j) * kTileKeys, tok = sink_tok + g.shift * kKvBlock;
          const int split = min(max(g.sink_blocks * kKvBlock - sink_tok, 0), kTileKeys);
          const bool masked = split > 0 || tok + kTileKeys - 1 > p_first ||
                              (a.window > 0 && tok <= p_last - a.window && tok + kTileKeys > a.sinks);
          // which of the 32 columns from c0 on the row sees: those up to pos, inside the window or sinks
          auto seen = [&](int c0) -> uint32_t {
            auto at = [&](int first) -> uint32_t {
              return bits_below(pos + 1 - first) & (~bits_below(lo + 1 - first) | bits_below(a.sinks - first));
            };
            // (without a window the first term alone: a prompt chunk 1826 -> 1753 us; the branch costs
            // the variant for few rows 6%, which masks a tile in dozens)
            if (!FEW && a.window == 0) return bits_below(pos + 1 - tok - c0);
            uint32_t see = at(tok + c0);
            if (split > c0) {
              const uint32_t sink = bits_below(split - c0);
              see = (see & ~sink) | (at(sink_tok + c0) & sink);
            }
            return see;
          };
          if constexpr (!FEW) {
            uint32_t x[128];
#pragma unroll
            for (int c = 0; c < 4; ++c) tmem_ld32_start(s_col + 32u * c, x + 32 * c);
#pragma unroll
            for (int c = 0; c < 4; ++c) tmem_ld32_wait(x + 32 * c);
            if (masked) {
#pragma unroll
              for (int q = 0; q < 4; ++q) {
                const uint32_t see = seen(32 * q);
#pragma unroll
                for (int e = 0; e < 32; ++e)
                  if (!(see & (1u << e))) x[32 * q + e] = 0xFF800000u;  // -inf
              }
            }
            // the largest t = raw * kb + log2(vs) of the tile
            float top = -INFINITY;
#pragma unroll
            for (int b = 0; b < kTileBlocks; ++b) {
              const float4 k = info[b];
              float v = __uint_as_float(x[16 * b]);
#pragma unroll
              for (int e = 1; e < 15; e += 2) v = max3(v, __uint_as_float(x[16 * b + e]), __uint_as_float(x[16 * b + e + 1]));
              v = fmaxf(v, __uint_as_float(x[16 * b + 15]));
              top = fmaxf(top, fmaf(v, k.x, k.y));
            }
            if (__any_sync(0xffffffffu, top > m + kKvGrowLog2)) {
              const float mn = fmaxf(m, top - kKvTopLog2);
              const float f = m == -INFINITY ? 0.f : ex2(m - mn);
              m = mn;
              l *= f;
              if (!first) {  // the sums so far: the lane's last product came before these scores
#pragma unroll 1
                for (int c = 0; c < D / 16; ++c) {
                  uint32_t y[16];
                  tmem_ld16(o_col + 16u * c, y);
#pragma unroll
                  for (int e = 0; e < 16; ++e) y[e] = __float_as_uint(__uint_as_float(y[e]) * f);
                  tmem_st16(o_col + 16u * c, y);
                }
              }
            }
            const float base = m == -INFINITY ? 0.f : m;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
#pragma unroll
              for (int c = 2 * h; c < 2 * h + 2; ++c) {
                uint32_t w[16];
#pragma unroll
                for (int b = 0; b < 2; ++b) {
                  const float4 k = info[2 * c + b];
                  const float kb = k.x, off = k.y - base;
                  const uint64_t kb2 = pack2(kb, kb), off2 = pack2(off, off);
                  uint64_t sum2 = 0ull;
#pragma unroll
                  for (int e = 0; e < 8; ++e) {
                    const int at = 32 * c + 16 * b + 2 * e;
                    float p0, p1;
                    unpack2(fma2(pack2(__uint_as_float(x[at]), __uint_as_float(x[at + 1])), kb2, off2), p0, p1);
                    p0 = ex2(p0);
                    p1 = ex2(p1);
                    sum2 = add2(sum2, pack2(p0, p1));
                    w[8 * b + e] = pack_weights(p0, p1);
                  }
                  float s0, s1;
                  unpack2(sum2, s0, s1);
                  l = fmaf(s0 + s1, k.z, l);
                }
                tmem_st16_start(s_col + 16u * c, w);  // over the scores, which are all in registers
              }
              tmem_st_wait();
              tc_fence_before();
              __syncwarp();
              if (lane == 0) mbar_arrive(&sm.p_full[ln][h]);  // the product over these 64 keys may start
            }
          } else {
            uint32_t x[64];
            auto scores = [&](int h) {  // of 64 keys, masked
              tmem_ld32_start(s_col + 64u * h, x);
              tmem_ld32_start(s_col + 64u * h + 32u, x + 32);
              tmem_ld32_wait(x);
              tmem_ld32_wait(x + 32);
              if (masked) {
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                  const uint32_t see = seen(64 * h + 32 * q);
#pragma unroll
                  for (int e = 0; e < 32; ++e)
                    if (!(see & (1u << e))) x[32 * q + e] = 0xFF800000u;  // -inf
                }
              }
            };
            // the largest t = raw * kb + log2(vs) of the tile
            float top = -INFINITY;
#pragma unroll 1
            for (int h = 1; h >= 0; --h) {
              scores(h);
#pragma unroll
              for (int b = 0; b < 4; ++b) {
                auto v = [&](int e) { return __uint_as_float(x[16 * b + e]); };
                const float u0 = max3(v(0), v(1), v(2)), u1 = max3(v(3), v(4), v(5)), u2 = max3(v(6), v(7), v(8));
                const float u3 = max3(v(9), v(10), v(11)), u4 = max3(v(12), v(13), v(14));
                const float4 k = info[4 * h + b];
                top = fmaxf(top, fmaf(max3(max3(u0, u1, u2), u3, fmaxf(u4, v(15))), k.x, k.y));
              }
            }
            if (__any_sync(0xffffffffu, top > m + kKvGrowLog2)) {
              const float mn = fmaxf(m, top - kKvTopLog2);
              const float f = m == -INFINITY ? 0.f : ex2(m - mn);
              m = mn;
              l *= f;
              if (!first) {  // the sums so far: the lane's last product came before these scores
#pragma unroll 1
                for (int c = 0; c < D / 16; ++c) {
                  uint32_t y[16];
                  tmem_ld16(o_col + 16u * c, y);
#pragma unroll
                  for (int e = 0; e < 16; ++e) y[e] = __float_as_uint(__uint_as_float(y[e]) * f);
                  tmem_st16(o_col + 16u * c, y);
                }
              }
            }
            const float base = m == -INFINITY ? 0.f : m;
#pragma unroll 1
            for (int h = 0; h < 2; ++h) {
              if (h) scores(1);  // (the first half is still here; its weights went over the scores 0 .. 31)
              uint32_t w[32];
#pragma unroll
              for (int b = 0; b < 4; ++b) {
                const float4 k = info[4 * h + b];
                const float off = k.y - base;
                const uint64_t kb2 = pack2(k.x, k.x), off2 = pack2(off, off);
                uint64_t sum2 = 0ull;
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                  float p0, p1;
                  unpack2(fma2(pack2(__uint_as_float(x[16 * b + 2 * e]), __uint_as_float(x[16 * b + 2 * e + 1])), kb2, off2), p0, p1);
                  p0 = ex2(p0);
                  p1 = ex2(p1);
                  sum2 = add2(sum2, pack2(p0, p1));
                  w[8 * b + e] = pack_weights(p0, p1);
                }
                float s0, s1;
                unpack2(sum2, s0, s1);
                l = fmaf(s0 + s1, k.z, l);
              }
              tmem_st16_start(s_col + 32u * h, w);
              tmem_st16_start(s_col + 32u * h + 16u, w + 16);
              tmem_st_wait();
              tc_fence_before();
              __syncwarp();
              if (lane == 0) mbar_arrive(&sm.p_full[ln][h]);  // the product over these 64 keys may start
            }
          }
        } else {
          __syncwarp();
          if (lane == 0) {
            mbar_arrive(&sm.p_full[ln][0]);
            mbar_arrive(&sm.p_full[ln][1]);
          }
        }
        if (lane == 0) mbar_arrive_n(&sm.info_empty[slot], dual ? 1u : 2u);
        first = false;
      }
      // ---- the item's results, once the tensor cores are through with it
      if (ok) ok = mbar_wait(&sm.o_full[ln], (uint32_t)seg & 1u, status);
      const bool second = !dual && mine == 1;  // the lane with the odd tiles hands its sums over
      if (ok && !dual && !second) ok = mbar_wait(&sm.other_full, other_phase, status);
      if (!dual) other_phase ^= 1u;
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      tc_fence_after();
      if (second) {
        sm.other[32 * quad + lane] = make_float2(m, l);
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm.other_full);
      } else {
        float fa = 1.f, fb = 0.f;
        const bool both = !dual && g.nt > 1;  // the other lane has sums
        if (both) {
          const float2 o = sm.other[32 * quad + lane];
          const float mn = fmaxf(m, o.x);
          fa = m == -INFINITY ? 0.f : ex2(m - mn);
          fb = o.x == -INFINITY ? 0.f : ex2(o.x - mn);
          l = l * fa + o.y * fb;
          m = mn;
        }
        if (live) {
          const bool valid = r < g.rows, whole = g.part == 0;
          const uint32_t b_col = tm + 256u + (uint32_t)D * (ln ^ 1);
          float* part = p.parts + (2 * (int64_t)blockIdx.x + (g.part == 1 ? 1 : 0)) * kCtaRows * (D + 2);
          if (whole) {
            const float inv = row_inverse(l);
            fa *= inv;
            fb *= inv;
            if (valid && a.lse) a.lse[pre_row_out(a, g.tok0, g.head, g.row0 + r)] = row_lse(m, l);
          } else if (valid) {
            part[kCtaRows * D + r] = m;
            part[kCtaRows * (D + 1) + r] = l;
          }
          const bool wide = ((uintptr_t)a.o & 31u) == 0;  // whole sectors, in half the stores
          const int64_t row = valid ? pre_row_out(a, g.tok0, g.head, g.row0 + r) : 0;
#pragma unroll 1
          for (int c = 0; c < D; c += 32) {
            uint32_t y[32];
            tmem_ld32_start(o_col + (uint32_t)c, y);
            tmem_ld32_wait(y);
#pragma unroll
            for (int e = 0; e < 32; ++e) y[e] = __float_as_uint(__uint_as_float(y[e]) * fa);
            if (both) {
              uint32_t z[32];
              tmem_ld32_start(b_col + (uint32_t)c, z);
              tmem_ld32_wait(z);
#pragma unroll
              for (int e = 0; e < 32; ++e) y[e] = __float_as_uint(fmaf(__uint_as_float(z[e]), fb, __uint_as_float(y[e])));
            }
            if (!valid) continue;
            if (whole) {
              uint32_t w[16];
#pragma unroll
              for (int e = 0; e < 16; ++e) w[e] = pack_bf16x2(__uint_as_float(y[2 * e]), __uint_as_float(y[2 * e + 1]));
              uint16_t* o = a.o + row * D + c;
              if (wide) {
                store32(o, w);
                store32(o + 16, w + 8);
              } else {
#pragma unroll
                for (int v = 0; v < 4; ++v)
                  reinterpret_cast<uint4*>(o)[v] = make_uint4(w[4 * v], w[4 * v + 1], w[4 * v + 2], w[4 * v + 3]);
              }
            } else {
#pragma unroll
              for (int v = 0; v < 4; ++v) store32(part + r * D + c + 8 * v, y + 8 * v);
            }
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {  // the sums have been read
          mbar_arrive(&sm.o_empty[ln]);
          if (!dual) mbar_arrive(&sm.o_empty[ln ^ 1]);
        }
      }
      done += g.nt;
      if (!dual) parity ^= g.nt & 1;
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm.seg_empty[seg % kSegs]);  // the entry has been read
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512u));
  }
}

// Joins N rows, every `apart`-th from r on, of the pieces of a cut item, in CTA order; C pieces' loads
// wait together
template <int D, int N, int C>
__device__ __forceinline__ void join_rows(const PreArgs& p, const PreCut& cut, int cta, int r, int apart, int lane) {
  const KvAttendArgs& a = p.a;
  constexpr int E = D / 32;
  float m[N], l[N], o[N][E];
#pragma unroll
  for (int i = 0; i < N; ++i) {
    m[i] = -INFINITY;
    l[i] = 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e) o[i][e] = 0.f;
  }
#pragma unroll 1
  for (int c0 = cta; c0 <= cut.last_cta; c0 += C) {
    float pm[C][N], pl[C][N], x[C][N][E];
#pragma unroll
    for (int k = 0; k < C; ++k) {
      const bool there = c0 + k <= cut.last_cta;
      const float* part = p.parts + (2 * (int64_t)(c0 + k) + (c0 + k == cta ? 1 : 0)) * kCtaRows * (D + 2);
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const int q = min(r + i * apart, cut.rows - 1);  // (a row past the end is read as the last)
        pm[k][i] = there ? __ldcg(part + kCtaRows * D + q) : -INFINITY;
        pl[k][i] = there ? __ldcg(part + kCtaRows * (D + 1) + q) : 0.f;
        if constexpr (E == 4) {
          const float4 v = there ? __ldcg(reinterpret_cast<const float4*>(part + q * D) + lane) : make_float4(0.f, 0.f, 0.f, 0.f);
          x[k][i][0] = v.x; x[k][i][1] = v.y; x[k][i][2] = v.z; x[k][i][3] = v.w;
        } else {
          const float2 v = there ? __ldcg(reinterpret_cast<const float2*>(part + q * D) + lane) : make_float2(0.f, 0.f);
          x[k][i][0] = v.x; x[k][i][1] = v.y;
        }
      }
    }
#pragma unroll
    for (int k = 0; k < C; ++k)
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const float mn = fmaxf(m[i], pm[k][i]);
        const float f = m[i] == -INFINITY ? 0.f : ex2(m[i] - mn);
        const float g = pm[k][i] == -INFINITY && mn == -INFINITY ? 1.f : ex2(pm[k][i] - mn);
        m[i] = mn;
        l[i] = fmaf(l[i], f, pl[k][i] * g);
#pragma unroll
        for (int e = 0; e < E; ++e) o[i][e] = fmaf(o[i][e], f, x[k][i][e] * g);
      }
  }
#pragma unroll
  for (int i = 0; i < N; ++i) {
    if (r + i * apart >= cut.rows) return;
    const float inv = row_inverse(l[i]);
    const int64_t row = pre_row_out(a, cut.tok0, cut.head, cut.row0 + r + i * apart);
    uint32_t w[E / 2];
#pragma unroll
    for (int e = 0; e < E; e += 2) w[e / 2] = pack_bf16x2(o[i][e] * inv, o[i][e + 1] * inv);
    if constexpr (E == 4)
      reinterpret_cast<uint2*>(a.o + row * D)[lane] = make_uint2(w[0], w[1]);
    else
      reinterpret_cast<uint32_t*>(a.o + row * D)[lane] = w[0];
    if (lane == 0 && a.lse) a.lse[row] = row_lse(m[i], l[i]);
  }
}

// Joins the pieces of the cut items.  An item in two or three pieces: a warp takes two rows; in
// more: one.
template <int D>
__global__ void __launch_bounds__(256) kv_join_kernel(const PreArgs p) {
  pdl_wait();
  pdl_launch_dependents();
  const int lane = threadIdx.x & 31, cta = blockIdx.y, at = blockIdx.x * 8 + (threadIdx.x >> 5);
  const PreCut cut = p.cuts[cta];
  if (cut.last_cta - cta < 3) {
    const int apart = (cut.rows + 1) / 2;
    if (at < apart) join_rows<D, 2, 2>(p, cut, cta, at, apart, lane);
  } else if (at < cut.rows) {
    join_rows<D, 1, 4>(p, cut, cta, at, 1, lane);
  }
}

template <typename Kernel>
int launch_one(Kernel kernel, dim3 grid, int threads, size_t smem, const PreArgs& p, void* stream) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = dim3((unsigned)threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = (cudaStream_t)stream;
  cudaLaunchAttribute at{};
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = QLIN_USE_PDL;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  return (int)cudaLaunchKernelEx(&cfg, kernel, p);
}

template <int CODE, int D, bool FEW>
int launch(const PreArgs& p, int rows, int sms, void* stream) {
  static std::atomic<uint64_t> done{0};
  auto kernel = kv_prefill_kernel<CODE, D, FEW>;
  constexpr size_t smem = pre_smem_bytes<D, FEW>();
  static_assert(smem <= 232448, "shared memory");
  if (const int e = smem_attr_once(kernel, smem, done)) return e;
  if (const int e = launch_one(kernel, dim3((unsigned)sms), kThreads, smem, p, stream)) return e;
  const int groups = (std::min(rows, kCtaRows) + 7) / 8;  // of rows of a cut item
  return launch_one(kv_join_kernel<D>, dim3((unsigned)groups, (unsigned)sms), 256, 0, p, stream);
}

template <int CODE, int D>
int launch_rows(const PreArgs& p, int rows, int sms, void* stream) {
  return rows <= kTileRows ? launch<CODE, D, true>(p, rows, sms, stream) : launch<CODE, D, false>(p, rows, sms, stream);
}

constexpr size_t kCutBytes = (kMaxSms * sizeof(PreCut) + 255) / 256 * 256;

}  // namespace

size_t kv_prefill_partial_bytes(int head_dim, int sms) {
  return kCutBytes + (size_t)sms * 2 * kCtaRows * (head_dim + 2) * 4;
}

int launch_kv_prefill(int code, int head_dim, const KvAttendArgs& a, int rows, int sms, void* stream) {
  const int64_t blocks = (int64_t)a.batch.total_q * a.group / kCtaRows + a.batch.n_seqs;  // (the host checked that it fits)
  const PreArgs p{a, (PreCut*)a.partials, (float*)((uint8_t*)a.partials + kCutBytes), (int)blocks};
  if (head_dim == 128) return code == kKvInt8 ? launch_rows<kKvInt8, 128>(p, rows, sms, stream) : launch_rows<kKvE4m3, 128>(p, rows, sms, stream);
  return code == kKvInt8 ? launch_rows<kKvInt8, 64>(p, rows, sms, stream) : launch_rows<kKvE4m3, 64>(p, rows, sms, stream);
}

}  // namespace qlin
