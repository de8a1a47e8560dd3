// fg_paged_attention.cu -- softmax attention of query rows over the paged 4-bit KV cache, split
// over the cache's length and joined, and the accumulation of its probabilities in the slots'
// weights.
//
// "FlexGen Guide: High-Throughput LLM Offloading on One GPU", section 3: the KV cache is held as
// 4-bit groups and dequantised on the fly for the attention dot products.
//
// Bound: the cache's bytes (D + 8 D/G per slot and key-value head: 144 for heads of 128 in groups
// of 64).  The query rows of a sequence that share a key-value head -- its new tokens' rows times
// the query heads of the head's group -- are columns of one product, 8 (the width of an mma.sync n8
// operand) or two times 8 to a tile, so that the codes are read and unpacked once for all of them.
// One column alone has a kernel of its own (below).
//
// Work is cut in blocks of 32 slots of one (sequence, key-value head, column tile), an item.  A warp
// streams its blocks through two stages of its own shared memory by bulk copies (cp.async.bulk, an
// mbarrier per stage) and meets no other warp before it is done.  A block lies in one or two pages
// (page_size % 16 == 0), six copies each, issued by as many lanes; the lanes look the page table up
// for 32 blocks at a time.  Two unrolled stages measured 210 us where three in a ring, whose
// addresses are computed, took 219 (512 sequences of 513 to 544 slots, 32 heads of 128: 1.26 GB; 227
// us since the sums are exact, 5.5 TB/s of 6.46 measured for a copy; up to 265 on other cards and
// power states).  Which warp takes which blocks: make_plan below.
//
// Both products run on the tensor cores straight from the codes (the group decomposition):
//     q . k_t = sum_g ( min_tg * sum_{d in g} q_d  +  scale_tg * sum_{d in g} q_d c_td )
//     o_d     = sum_t p_t min_tg  +  sum_t w_tg c_td,  w_tg = p_t scale_tg
// The operands are fp16; w goes in as its rounding and the rest, 22 bits together: a row whose
// weight lies on a few slots would otherwise carry their rounding in all of its values (half a step,
// 2.4e-4, against the output's own).  Both are of w times a power of two F that brings the largest V
// scale met so far to 2^12 .. 2^13 (Fit below; undone where a block's products are added in fp32), so
// that what the pair's last place, 2^-24, drops is 2^-37 of that scale for every slot: without F a
// slot with w below 2^-25 lost its codes and kept its minimum, and thousands of them beside one slot
// with most of the weight were 2 to 30 % of an output (16384 slots, 2 % of the weight off that slot, V
// scales of 0.03 and 0.001).  A nibble in bits 4-7 of a 16-bit half is the fp16 subnormal
// c * 2^-20, exact, so that an AND, and for some a shift or a multiplication, unpacks a pair of codes,
// and the fp32 results are rescaled.  Not bits 0-3, which two of four nibbles would reach without a
// shift: the tensor core aligns a product by its operands' exponents, -14 for every subnormal, and
// drops what lies some 24 bits below; with c * 2^-24 that was 3e-5 of a code's weight, with c * 2^-20
// it is 6e-7 (codes of 1 under minima of -scale).  Scores, softmax state and sums are fp32.
//   scores: A = codes of 16 slots x 16 dims of one group, B = q (16 dims x 8 columns)
//   output: A = codes of 16 dims x 16 slots (ldmatrix.trans), B = w of the dims' group (16 slots x 8
//           columns), which is the score tile's layout transposed (movmatrix)
// Both score and output fragments give a lane the columns 2c, 2c+1 (c = lane % 4), so the softmax
// state of a column never leaves its lanes.  A block's output products start from zero and are added
// in fp32 registers: the tensor core's additions truncate, which grows with a sum.
// What the tile kernel costs beyond the bytes is the fixed part of a launch (7 us from its start to
// the first block's arrival, 6 us of join) and instructions: 24 sequences of 8192 slots and 8 heads of
// 8 columns take 69 us for 214 MB.  Rows beyond a tile's 8 columns unpack the codes again: 512 rows of
// 8 prompts of 512 over 8 heads of 128 take 125 us.
#include <math.h>

#include <type_traits>

#include "fg_paged.cuh"

namespace {

constexpr int kWarps = 4;
constexpr int kBlock = 32;              // slots per warp step
constexpr int kCta = kWarps * kBlock;   // slots per CTA step
constexpr int kCols = 8;                // columns per tile
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kSlack = 2.0f;
constexpr uint32_t kLowNibble = 0x000F000Fu;  // bits 0-3 of both halves: c * 2^-24
constexpr uint32_t kNibble = 0x00F000F0u;     // bits 4-7 of both halves: c * 2^-20
constexpr float kUnit = 1048576.0f;           // 2^20: sums of products with codes, back to their size
constexpr float kScore = kUnit * kLog2e;      // and to log2 units

// Pairs of fp16 numbers c * 2^-20 from nibbles 0, and from nibbles 1, of a word's 16-bit halves.  The
// multiplication by 16 (exact) is the FMA pipe's, which has room; a shift would be the ALU's.
__device__ __forceinline__ uint32_t nibble0(uint32_t x) {
  const uint32_t n = x & kLowNibble;
  const __half2 h = __hmul2(*reinterpret_cast<const __half2 *>(&n), __float2half2_rn(16.0f));
  return *reinterpret_cast<const uint32_t *>(&h);
}
__device__ __forceinline__ uint32_t nibble1(uint32_t x) { return x & kNibble; }

// The four nibbles of a word's halves: nibble i is bits 4i .. 4i+3 of the low and of the high half.
struct Nibbles {
  uint32_t n[4];
  __device__ __forceinline__ explicit Nibbles(uint32_t x) {
    const uint32_t y = x >> 8;
    n[0] = nibble0(x);
    n[1] = nibble1(x);
    n[2] = nibble0(y);
    n[3] = nibble1(y);
  }
};

// CTAs (of four warps) resident per SM, which is what the register budgets are cut for.  Tile kernel:
// 168 registers a thread hold one tile of D <= 128 (at 128, four CTAs, three tracked sequences of up
// to 40000 slots and 8 heads of 4 columns took 69 us instead of 58); two tiles, or D = 256, need 255.
// Single-column kernel: 128 registers (five CTAs spill: 242 us instead of 225 for 512 sequences of 513
// to 544 slots and 32 heads of 128).
__host__ __device__ constexpr int tile_ctas(int D, int cols) { return cols <= kCols && D <= 128 ? 3 : 2; }
__host__ __device__ constexpr int one_ctas(int D) { return D <= 128 ? 4 : 3; }

struct Part {  // a unit's part of a cut item: the units that have it, the part's slots
  int item, u0, u1, t0, t1;
};

struct PagedAttnArgs {
  PagedArgs kv;
  const __half *q;
  int64_t ldq;
  __half *out;
  int64_t ldo;
  int R, rows_per_seq, limit;
  int tile0, tiles;  // column tiles of this launch: tile0 .. tile0 + tiles - 1
  int pcols;         // columns per item: 1 (single-column launches), 8 or 16
  int items, seqs;
  int units;         // partitioned launches: warps that share the blocks of all items; else 0
  bool shared_unit;  // otherwise: the CTA's warps share an item, or have one each
  const int32_t *positions, *counts;
  // partitioned launches: per unit two parts of cut items (Walk)
  float2 *ml;        // [units][2][pcols]: running maximum (log2 units) and sum; sum < 0: a bad page
  float *po;         // [units][2][pcols][D] unnormalised outputs
  Part *parts;       // [units][2] (accumulate)
  int2 *cut;         // [items]: first and last unit of a cut item; first < 0: whole in one unit
  float *scores;     // [items][pcols][score_ld] (accumulate)
  int64_t score_ld;
};

// One (sequence, key-value head, column tile); ht = head * tiles + tile, item = s * heads * tiles + ht.
struct Item {
  int s, h, n0, ncols;  // columns n0 .. n0 + ncols - 1 of the head (column n: row n / R, query head n % R)
  int pos, live;        // first new slot; rows of the sequence that see anything
  __device__ __forceinline__ int len(int n, int R) const {  // slots that column n sees
    const int i = n / R;
    return i < live ? pos + i + 1 : 0;
  }
};

__device__ __forceinline__ Item load_item(const PagedAttnArgs &a, int s, int ht, bool flag) {
  Item it;
  it.h = a.tiles == 1 ? ht : ht / a.tiles;
  const int tile = a.tile0 + ht - it.h * a.tiles;
  it.s = s;
  it.n0 = tile * a.pcols;
  it.ncols = min(a.pcols, a.rows_per_seq * a.R - it.n0);
  const int pos = a.positions[it.s], count = a.counts ? a.counts[it.s] : a.rows_per_seq;
  const bool range = pos < -1 || count < 0 || count > a.rows_per_seq ||
                     (pos >= 0 && static_cast<int64_t>(pos) + count > a.limit);
  if (range && flag) atomicOr(a.kv.err, FG_DEVERR_RANGE);
  it.pos = pos;
  it.live = range || pos < 0 ? 0 : count;
  return it;
}

// Blocks of 32 slots that a sequence's rows see together.
__device__ __forceinline__ int seq_blocks(const PagedAttnArgs &a, int s) {
  const int pos = a.positions[s], count = a.counts ? a.counts[s] : a.rows_per_seq;
  const bool on = pos >= 0 && count > 0 && count <= a.rows_per_seq && static_cast<int64_t>(pos) + count <= a.limit;
  return on ? (pos + count + kBlock - 1) / kBlock : 0;
}

// A warp's way through its share of the work.  Partitioned launches lay the blocks of all items in
// a row (sequence, then head and tile, then block) and cut it into `units` runs that differ by a
// block at most, no more than one for every kMinBlocks blocks: a run is up to two parts of cut items,
// the first and the last, with whole items in between.  A part is number 2 * unit + 1 if it begins
// its item, else 2 * unit.
constexpr int kMinBlocks = 4;

// x / d; the 64-bit division only where 32 bits do not hold x (both are not negative, d > 0).
__device__ __forceinline__ int64_t divide(int64_t x, int d) {
  return x <= 0xFFFFFFFFll ? static_cast<int64_t>(static_cast<uint32_t>(x) / static_cast<uint32_t>(d)) : x / d;
}

struct Walk {
  int s, ht, b, nblk;  // at block b of head and tile ht of sequence s, which has nblk blocks
  int longer;          // the units 0 .. longer - 1 have one block more than `per`
  int64_t per, g, end; // place in the row of all blocks, and where this unit's run ends

  __device__ __forceinline__ int64_t start_of(int unit) const { return unit * per + min(unit, longer); }
  __device__ __forceinline__ int unit_of(int64_t block) const {
    const int64_t head = longer * (per + 1);
    const int64_t x = block < head ? block : block - head;
    const int64_t d = block < head ? per + 1 : per;
    const int64_t u = x <= 0xFFFFFFFFll && d <= 0xFFFFFFFFll
                          ? static_cast<int64_t>(static_cast<uint32_t>(x) / static_cast<uint32_t>(d)) : x / d;
    return static_cast<int>(block < head ? u : longer + u);
  }
  __device__ __forceinline__ bool begin(const PagedAttnArgs &a, int unit, int lane) {
    const int HT = a.kv.H * a.tiles;
    if (!a.units) {
      if (unit >= a.items) return false;
      s = unit / HT;
      ht = unit - s * HT;
      b = 0;
      return true;
    }
    int64_t sum = 0;
    for (int i = lane; i < a.seqs; i += 32) sum += seq_blocks(a, i);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    const int64_t total = sum * HT;
    const int64_t most = (total + kMinBlocks - 1) / kMinBlocks;
    const int units = static_cast<int>(most < a.units ? most : a.units);
    if (unit >= units) return false;
    per = divide(total, units);
    longer = static_cast<int>(total - per * units);
    g = start_of(unit);
    end = start_of(unit + 1);
    nblk = 0;
    int64_t base = 0;  // blocks of one head and tile before the chunk of 32 sequences
    for (int i = 0; i < a.seqs; i += 32) {
      const uint32_t n = i + lane < a.seqs ? seq_blocks(a, i + lane) : 0u;
      uint32_t incl = n;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const uint32_t v = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += v;
      }
      const uint32_t after = __ballot_sync(0xffffffffu, (base + incl) * HT > g);
      if (after) {  // the first sequence that ends behind g
        const int l = __ffs(after) - 1;
        nblk = __shfl_sync(0xffffffffu, n, l);
        base += __shfl_sync(0xffffffffu, incl, l) - nblk;
        s = i + l;
        break;
      }
      base += __shfl_sync(0xffffffffu, incl, 31);
    }
    if (nblk == 0) return false;
    const int64_t rest = g - base * HT;
    ht = static_cast<int>(divide(rest, nblk));
    b = static_cast<int>(rest - static_cast<int64_t>(ht) * nblk);
    return true;
  }
  __device__ __forceinline__ int run() const {  // blocks of the segment at b
    const int64_t left = end - g;
    return left < nblk - b ? static_cast<int>(left) : nblk - b;
  }
  __device__ __forceinline__ bool next(const PagedAttnArgs &a, int ran) {
    g += ran;
    if (g >= end) return false;
    b = 0;
    if (++ht == a.kv.H * a.tiles) {
      ht = 0;
      do {
        if (++s >= a.seqs) return false;  // (not with blocks left)
        nblk = seq_blocks(a, s);
      } while (nblk == 0);
    }
    return true;
  }
};

// A warp's walk (in shared memory) one segment on; the stages' last reads and writes come before the
// next segment's copies.
__device__ __forceinline__ bool advance(const PagedAttnArgs &a, Walk *shared, int lane) {
  Walk w = *shared;
  const bool more = w.next(a, w.run());
  fence_proxy_async_smem();
  __syncwarp();
  if (lane == 0) *shared = w;
  __syncwarp();
  return more;
}

__device__ __forceinline__ void flag_bad_sequences(const PagedAttnArgs &a, int lane) {
  bool range = false;
  for (int i = lane; i < a.seqs; i += 32) {
    const int pos = a.positions[i], count = a.counts ? a.counts[i] : a.rows_per_seq;
    range |= pos < -1 || count < 0 || count > a.rows_per_seq ||
             (pos >= 0 && static_cast<int64_t>(pos) + count > a.limit);
  }
  if (range) atomicOr(a.kv.err, FG_DEVERR_RANGE);
}

// What a segment's outputs are: an item's whole rows, or part `index` of a cut item.
struct Target {
  bool whole;
  int64_t index;
};

__device__ __forceinline__ Target target_of(const PagedAttnArgs &a, const Walk &w, int unit, int item, int ran,
                                            bool leader) {
  Target t;
  t.whole = !a.units || ran == w.nblk;
  t.index = 2 * static_cast<int64_t>(unit) + (w.b == 0);
  if (a.units && leader) {
    if (t.whole) {
      a.cut[item] = make_int2(-1, -1);
    } else {
      const int64_t g0 = w.g - w.b;
      const int u1 = w.b == 0 || a.scores ? w.unit_of(g0 + w.nblk - 1) : 0;
      if (w.b == 0) a.cut[item] = make_int2(unit, u1);
      if (a.scores)
        a.parts[t.index] = Part{item, w.b == 0 ? unit : w.unit_of(g0), u1, w.b * kBlock, (w.b + ran) * kBlock};
    }
  }
  return t;
}

template <int D, int G, int NT>  // NT: column tiles of 8 per unit
struct Shape {
  static constexpr int NG = D / G;
  static constexpr int RB = D / 2;                 // code bytes per slot
  static constexpr int KW = G / 32;                // K code words per lane, slot and group
  static constexpr int CH = D / 32;                // 32-dim chunks (16 bytes of codes)
  static constexpr int CODE_B = kBlock * RB, META_B = kBlock * NG * 2;
  static constexpr int STAGE_B = 2 * CODE_B + 4 * META_B;
  static constexpr int WARP_B = 2 * STAGE_B > NT * kCols * D * 4 ? 2 * STAGE_B : NT * kCols * D * 4;
  static constexpr int SMEM = kWarps * WARP_B;  // a warp's two stages, at the end its outputs
  static constexpr int kCtas = tile_ctas(D, NT * kCols);
};

__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// d = A * B (fresh accumulators)
__device__ __forceinline__ void mma_f16_z(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                          uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}

__device__ __forceinline__ uint32_t transpose_8x8(uint32_t x) {
  uint32_t y;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

__device__ __forceinline__ float fast_exp2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ uint32_t pack_h2(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t *>(&h);
}

template <int N>
__device__ __forceinline__ void load_words(const uint8_t *p, uint32_t (&w)[N]) {
  if constexpr (N == 1) {
    w[0] = *reinterpret_cast<const uint32_t *>(p);
  } else if constexpr (N == 2) {
    const uint2 v = *reinterpret_cast<const uint2 *>(p);
    w[0] = v.x;
    w[1] = v.y;
  } else {
    const uint4 v = *reinterpret_cast<const uint4 *>(p);
    w[0] = v.x;
    w[1] = v.y;
    w[2] = v.z;
    w[3] = v.w;
  }
}

__device__ __forceinline__ void ldmatrix_x4_trans(uint32_t (&r)[4], uint32_t addr) {
  // volatile: stays between the wait for its stage and the fence before the stage's next copy
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr));
}

// A warp's copies of its blocks: what never changes for a lane, and the pool places of the next 32
// blocks, block i's in lane i, in units of 16 slots.
constexpr uint32_t kNoSecond = 0xFFFFFFFFu, kJoined = 0xFFFFFFFEu;

template <int RB, int NG, int CODE_B, int META_B>
struct Copies {
  const uint8_t *pool;  // lanes 0-5 (first 16 slots) and 8-13 (second): the array of lane % 8
  uint32_t dst, per16;  // shared address in stage 0; bytes of 16 slots
  uint32_t a16, b16;    // block `lane`: first half; second half, kJoined (it follows) or kNoSecond
  bool bad;

  __device__ __forceinline__ void init(const PagedAttnArgs &a, uint32_t base, int lane) {
    const int arr = lane & 7, run = lane >> 3;
    const bool codes = arr < 2;
    const void *const ptr = arr == 0   ? static_cast<const void *>(a.kv.kc)
                            : arr == 1 ? static_cast<const void *>(a.kv.vc)
                            : arr == 2 ? static_cast<const void *>(a.kv.km)
                            : arr == 3 ? static_cast<const void *>(a.kv.ks)
                            : arr == 4 ? static_cast<const void *>(a.kv.vm)
                                       : static_cast<const void *>(a.kv.vs);
    pool = arr < 6 && run < 2 ? static_cast<const uint8_t *>(ptr) : nullptr;
    per16 = 16u * (codes ? RB : NG * 2);
    dst = base + (codes ? arr * CODE_B : 2 * CODE_B + (arr - 2) * META_B) + (run & 1) * per16;
    a16 = b16 = 0;
    bad = false;
  }
  // the places of blocks t + lane * step (slots below t_end)
  __device__ __forceinline__ void look_up(const PagedAttnArgs &a, int s, int h, int t, int step, int t_end, int lane) {
    const int64_t tl = t + static_cast<int64_t>(lane) * step;
    int64_t x = 0, y = 0;
    if (tl < t_end) x = paged_slot(a.kv, s, h, static_cast<int>(tl));
    if (tl + 16 < t_end) y = paged_slot(a.kv, s, h, static_cast<int>(tl) + 16);
    bad |= x < 0 || y < 0;  // flagged at the end; the pool's first slots are read instead
    x = x < 0 ? 0 : x;
    y = y < 0 ? 0 : y;
    a16 = static_cast<uint32_t>(x >> 4);
    b16 = tl + 16 >= t_end ? kNoSecond : y == x + 16 ? kJoined : static_cast<uint32_t>(y >> 4);
  }
  // block `i` of the table into the stage at byte offset `off`, completion on `bar`
  __device__ __forceinline__ void issue(int i, uint32_t off, uint32_t bar, int lane) {
    const uint32_t x = __shfl_sync(0xffffffffu, a16, i), y = __shfl_sync(0xffffffffu, b16, i);
    if (lane == 0) mbar_arrive_expect_tx(bar, (y == kNoSecond ? 16 : 32) * (2 * RB + 8 * NG));
    __syncwarp();
    const bool run = lane >> 3;
    if (pool && (!run || y < kJoined))
      bulk_g2s(dst + off, pool + static_cast<uint64_t>(run ? y : x) * per16, y == kJoined ? 2 * per16 : per16, bar);
  }
};

// The power of two by which a run's weights w = p * scale are multiplied on their way into fp16.  It
// starts where the smallest scale, 2^-24, wants it and falls when a scale does not fit: scale * f <=
// kFits and p <= 2^kSlack leave w * f <= 2^15.  Uniform in the warp.  The check of every block's scales
// costs 1 to 3 % (512 sequences of 513 to 544 slots, 32 heads of 128: 225.2 to 227.5 us; 24 ragged ones
// of up to 16384, 8 columns a head: 77.5 to 79.7); the scales kept in registers from the check to their
// use, and compared in fp16 pairs, measured the same or up to 1.6 % more.
constexpr float kFits = 8192.0f;

struct Fit {
  float f, inv;
  __device__ __forceinline__ Fit() : f(68719476736.0f), inv(1.0f / 68719476736.0f) {}  // 2^36
  // `scale`: the warp's largest, above kFits / f.  Its exponent e gives f = 2^(12 - e); fp16's largest
  // is taken for an infinite one.
  __device__ __forceinline__ void fall(float scale) {
    const uint32_t e = min(__float_as_uint(scale) >> 23, 127u + 15u);
    f = __uint_as_float((127u + 12u + 127u - e) << 23);
    inv = __uint_as_float((e - 12u) << 23);
  }
};

// The weights of the 4 slots t .. t + 3 (t % 4 == 0, so that they lie in one page), of which those
// below `end` grow.
__device__ __forceinline__ void grow4(const PagedAttnArgs &a, int s, int h, int t, int end, float4 add) {
  const int64_t slot = paged_slot(a.kv, s, h, t);
  if (slot < 0) return;
  float *w = a.kv.weights + slot;
  float4 v = *reinterpret_cast<float4 *>(w);
  v.x += add.x;
  v.y += t + 1 < end ? add.y : 0.f;
  v.z += t + 2 < end ? add.z : 0.f;
  v.w += t + 3 < end ? add.w : 0.f;
  if (t + 3 < end) {
    *reinterpret_cast<float4 *>(w) = v;
  } else {  // the slots behind stay as they are
    w[0] = v.x;
    if (t + 1 < end) w[1] = v.y;
    if (t + 2 < end) w[2] = v.z;
  }
}

// A column's probabilities of slots t .. t + 3 (those below its length `end`), added to *add.
__device__ __forceinline__ void grow_by(float4 *add, const float *scores, int t, int end, float m, float inv) {
  if (t >= end) return;
  const float4 v = *reinterpret_cast<const float4 *>(scores + t);  // (behind `end`: anything)
  add->x += fast_exp2(v.x - m) * inv;
  add->y += t + 1 < end ? fast_exp2(v.y - m) * inv : 0.f;
  add->z += t + 2 < end ? fast_exp2(v.z - m) * inv : 0.f;
  add->w += t + 3 < end ? fast_exp2(v.w - m) * inv : 0.f;
}

// The weights of a single-column item's slots begin .. end - 1, once its maximum and 1 / sum are
// known, by `n` threads of which this is number i.
__device__ __forceinline__ void grow_row(const PagedAttnArgs &a, int s, int h, const float *scores, int begin, int end,
                                         float m, float inv, int i, int n) {
  for (int t = begin + 4 * i; t < end; t += 4 * n) {
    float4 add = make_float4(0.f, 0.f, 0.f, 0.f);
    grow_by(&add, scores, t, end, m, inv);
    grow4(a, s, h, t, end, add);
  }
}

// A slot's numbers of one array (its groups' minima, or scales), loaded at once.
template <int NG>
struct Nums {
  uint32_t w[(NG + 1) / 2];
  __device__ __forceinline__ explicit Nums(const __half *p) {
    if constexpr (NG == 1) w[0] = *reinterpret_cast<const uint16_t *>(p);
    else if constexpr (NG == 2) w[0] = *reinterpret_cast<const uint32_t *>(p);
    else {
      const uint2 v = *reinterpret_cast<const uint2 *>(p);
      w[0] = v.x;
      w[1] = v.y;
    }
  }
  __device__ __forceinline__ float get(int g) const {
    const __half2 h = *reinterpret_cast<const __half2 *>(&w[g / 2]);
    return g & 1 ? __high2float(h) : __low2float(h);
  }
};

// The B operands of 8 dims of q (v): dims (0, 4) and (2, 6), the A operands' nibbles 0 and 2, then
// (1, 5) and (3, 7), nibbles 1 and 3.
__device__ __forceinline__ void q_operands(uint32_t (&f)[4], const uint4 &v) {
  f[0] = __byte_perm(v.x, v.z, 0x5410);
  f[1] = __byte_perm(v.y, v.w, 0x5410);
  f[2] = __byte_perm(v.x, v.z, 0x7632);
  f[3] = __byte_perm(v.y, v.w, 0x7632);
}

template <int D, int G, int NT, bool TRACK>
__global__ void __launch_bounds__(kWarps * 32, Shape<D, G, NT>::kCtas) paged_attn_kernel(const PagedAttnArgs a) {
  using S = Shape<D, G, NT>;
  constexpr int NG = S::NG, RB = S::RB, KW = S::KW, CH = S::CH, NC = NT * kCols;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ __align__(8) uint64_t full_bar[kWarps][2];
  __shared__ float red_m[kWarps][NC], red_l[kWarps][NC];
  __shared__ int bad_page;

  griddep_launch();  // the join may be scheduled once every CTA runs
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int gid = lane >> 2, c = lane & 3;
  const int unit = a.shared_unit ? blockIdx.x : blockIdx.x * kWarps + warp;
  const int first = a.shared_unit ? warp : 0;
  const int step = a.shared_unit ? kCta : kBlock;  // slots from one of this warp's blocks to the next
  if (TRACK && a.units && lane < 2 && unit < a.units) a.parts[2 * unit + lane].item = -1;
  if (a.units && unit == 0) flag_bad_sequences(a, lane);
  __shared__ Walk walks[kWarps];  // (out of the registers: used once per segment)
  {
    Walk w;
    if (!w.begin(a, unit, lane)) return;
    if (lane == 0) walks[warp] = w;
    __syncwarp();
  }

  const uint32_t bar0 = smem_u32(&full_bar[warp][0]);
  if (lane == 0) {
    mbar_init(bar0, 1);
    mbar_init(bar0 + 8, 1);
    fence_mbar_init();
    fence_proxy_async_smem();
  }
  if (a.shared_unit) {
    if (tid == 0) bad_page = 0;
    __syncthreads();
  } else {
    __syncwarp();
  }
  uint8_t *const wbase = smem + warp * S::WARP_B;
  Copies<RB, NG, S::CODE_B, S::META_B> cp;
  cp.init(a, smem_u32(wbase), lane);
  bool ok = true;
  uint32_t phase = 0;  // bit i: the parity of stage i's next phase

  while (true) {  // segments
    const Walk walk = walks[warp];
    const int ht = walk.ht, item = walk.s * a.kv.H * a.tiles + ht;
    const Item it = load_item(a, walk.s, ht, !a.units && first == 0 && lane == 0);
    // live columns' lengths: rows ascend with the column, so the last live one sees most
    int lmin = 0, lmax = 0;
    {
      const int last = min(it.n0 + it.ncols, it.live * a.R) - 1;
      if (last >= it.n0) {
        lmin = it.len(it.n0, a.R);
        lmax = it.len(last, a.R);
      }
    }
    const int ran = a.units ? walk.run() : 0;
    const int t_begin = a.units ? walk.b * kBlock : 0;
    const int t_end = a.units ? min(lmax, t_begin + ran * kBlock) : lmax;
    const int t_first = t_begin + first * kBlock;
    const int steps = ok && t_end > t_first ? (t_end - t_first + step - 1) / step : 0;
    cp.bad = false;
    if (steps > 0) {
      cp.look_up(a, it.s, it.h, t_first, step, t_end, lane);
      cp.issue(0, 0, bar0, lane);
      if (steps > 1) cp.issue(1, S::STAGE_B, bar0 + 8, lane);
    }
    const Target target = target_of(a, walk, unit, item, ran, lane == 0);

    // ---- q of column n0 + 8 nt + gid as the B operand of the score MMAs ----
    // Word j of group g of lane class c: dims 2o .. 2o+7, o = g*G/2 + c*G/8 + 4j.  Low-nibble MMA
    // (nibbles 0 and 2 of the halves): k slots (2c, 2c+1) = dims (2o, 2o+4), (2c+8, 2c+9) = (2o+2,
    // 2o+6); high-nibble MMA: the same + 1.
    uint32_t qf[NT][NG][KW][4];
    float qsum[NT][2][NG];  // columns 2c, 2c+1: sum of q over the group, over kUnit
    int len[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; nt++) {
      const int col = nt * kCols + gid, n = it.n0 + col;
      const bool on = col < it.ncols && it.len(n, a.R) > 0;
      const __half *qrow = a.q + (static_cast<int64_t>(it.s) * a.rows_per_seq + n / a.R) * a.ldq +
                           (static_cast<int64_t>(it.h) * a.R + n % a.R) * D;
#pragma unroll
      for (int g = 0; g < NG; g++) {
        float sum = 0.f;
#pragma unroll
        for (int j = 0; j < KW; j++) {
          uint4 v = make_uint4(0, 0, 0, 0);
          if (on) v = *reinterpret_cast<const uint4 *>(qrow + g * G + c * (G / 4) + 8 * j);
          const __half *e = reinterpret_cast<const __half *>(&v);
          q_operands(qf[nt][g][j], v);
#pragma unroll
          for (int i = 0; i < 8; i++) sum += __half2float(e[i]);
        }
        sum += __shfl_xor_sync(0xffffffffu, sum, 1);
        sum += __shfl_xor_sync(0xffffffffu, sum, 2);
        sum *= 1.0f / kUnit;
        qsum[nt][0][g] = __shfl_sync(0xffffffffu, sum, 8 * c);
        qsum[nt][1][g] = __shfl_sync(0xffffffffu, sum, 8 * c + 4);
      }
#pragma unroll
      for (int e = 0; e < 2; e++) {
        const int m = nt * kCols + 2 * c + e;
        len[nt][e] = m < it.ncols ? it.len(it.n0 + m, a.R) : 0;
      }
    }
    float *const srow = TRACK ? a.scores + static_cast<int64_t>(item) * NC * a.score_ld : nullptr;
    // this lane's places in a stage: K code rows, group numbers, ldmatrix rows of V codes
    const uint8_t *const kbase = wbase + gid * RB + c * (G / 8);
    const __half *const nbase = reinterpret_cast<const __half *>(wbase + 2 * S::CODE_B) + gid * NG;
    const uint32_t vbase = smem_u32(wbase) + S::CODE_B + ((lane >> 3 & 1) * 8 + (lane & 7)) * RB + (lane >> 4) * 16;

    Fit fit;
    float m[NT][2], l[NT][2];
    float vacc[NT][2][NG];   // sum of p min over this lane's slots
    float ov[NT][CH][2][4];  // chunk ch, x: dims 32 ch + 4 gid + 2x ([0], [1]: columns 2c, 2c+1) and + 1 ([2], [3])
#pragma unroll
    for (int nt = 0; nt < NT; nt++) {
      m[nt][0] = m[nt][1] = -INFINITY;
      l[nt][0] = l[nt][1] = 0.f;
#pragma unroll
      for (int g = 0; g < NG; g++) {
        vacc[nt][0][g] = vacc[nt][1][g] = 0.f;
      }
#pragma unroll
      for (int i = 0; i < CH; i++)
#pragma unroll
        for (int x = 0; x < 2; x++) ov[nt][i][x][0] = ov[nt][i][x][1] = ov[nt][i][x][2] = ov[nt][i][x][3] = 0.f;
    }

    // one block of 32 slots at t, in stage ST; EDGE: some live column does not see all of them
    auto block = [&](auto stage, auto edge, int t) {
      constexpr int OFF = decltype(stage)::value * S::STAGE_B;
      constexpr bool EDGE = decltype(edge)::value;
      // ---- scores (over kUnit) of slots t + 16u + gid + 8x, columns 2c + e ----
      float sc[NT][2][2][2];
#pragma unroll
      for (int u = 0; u < 2; u++) {
        const __half *const n0 = nbase + OFF / 2 + 16 * u * NG, *const n1 = n0 + 8 * NG;
        const Nums<NG> km[2] = {Nums<NG>(n0), Nums<NG>(n1)};
        const Nums<NG> ks[2] = {Nums<NG>(n0 + kBlock * NG), Nums<NG>(n1 + kBlock * NG)};
#pragma unroll
        for (int g = 0; g < NG; g++) {
          uint32_t k0[KW], k1[KW];
          load_words<KW>(kbase + OFF + 16 * u * RB + g * (G / 2), k0);
          load_words<KW>(kbase + OFF + (16 * u + 8) * RB + g * (G / 2), k1);
          float lo[NT][4], hi[NT][4];  // two chains of MMAs
#pragma unroll
          for (int j = 0; j < KW; j++) {
            const Nibbles x0(k0[j]), x1(k1[j]);
#pragma unroll
            for (int nt = 0; nt < NT; nt++) {
              if (j == 0) {
                mma_f16_z(lo[nt], x0.n[0], x1.n[0], x0.n[2], x1.n[2], qf[nt][g][j][0], qf[nt][g][j][1]);
                mma_f16_z(hi[nt], x0.n[1], x1.n[1], x0.n[3], x1.n[3], qf[nt][g][j][2], qf[nt][g][j][3]);
              } else {
                mma_f16(lo[nt], x0.n[0], x1.n[0], x0.n[2], x1.n[2], qf[nt][g][j][0], qf[nt][g][j][1]);
                mma_f16(hi[nt], x0.n[1], x1.n[1], x0.n[3], x1.n[3], qf[nt][g][j][2], qf[nt][g][j][3]);
              }
            }
          }
#pragma unroll
          for (int x = 0; x < 2; x++) {
            const float mn = km[x].get(g), sl = ks[x].get(g);
#pragma unroll
            for (int nt = 0; nt < NT; nt++)
#pragma unroll
              for (int e = 0; e < 2; e++) {
                const float v = g == 0 ? mn * qsum[nt][e][g] : fmaf(mn, qsum[nt][e][g], sc[nt][u][x][e]);
                sc[nt][u][x][e] = fmaf(sl, lo[nt][2 * x + e] + hi[nt][2 * x + e], v);
              }
          }
        }
      }
      if constexpr (EDGE) {
#pragma unroll
        for (int nt = 0; nt < NT; nt++)
#pragma unroll
          for (int u = 0; u < 2; u++)
#pragma unroll
            for (int x = 0; x < 2; x++)
#pragma unroll
              for (int e = 0; e < 2; e++)
                if (t + 16 * u + gid + 8 * x >= min(len[nt][e], t_end)) sc[nt][u][x][e] = -INFINITY;
      }
      if constexpr (TRACK) {
#pragma unroll
        for (int nt = 0; nt < NT; nt++)
#pragma unroll
          for (int e = 0; e < 2; e++)
            if (len[nt][e] > 0)
#pragma unroll
              for (int u = 0; u < 2; u++)
#pragma unroll
                for (int x = 0; x < 2; x++) {
                  const int ts = t + 16 * u + gid + 8 * x;
                  if (!EDGE || ts < len[nt][e])
                    srow[(nt * kCols + 2 * c + e) * a.score_ld + ts] = sc[nt][u][x][e] * kScore;
                }
      }
      // ---- running maximum: moves only when a score exceeds it by more than kSlack, so that
      //      p = 2^(s - m) <= 2^kSlack and w = p * scale * fit.f stays inside fp16 ----
      const __half *const vs0 = nbase + OFF / 2 + 3 * kBlock * NG;  // V scales of slots gid, gid + 8, ..
      float vmax = 0.f;
#pragma unroll
      for (int i = 0; i < 4; i++) {
        const Nums<NG> v(vs0 + 8 * i * NG);
#pragma unroll
        for (int g = 0; g < NG; g++)
          if (!EDGE || t + 8 * i + gid < t_end) vmax = fmaxf(vmax, fabsf(v.get(g)));
      }
      float cmax[NT][2];
      bool moves = vmax * fit.f > kFits;
#pragma unroll
      for (int nt = 0; nt < NT; nt++)
#pragma unroll
        for (int e = 0; e < 2; e++) {
          cmax[nt][e] =
              fmaxf(fmaxf(sc[nt][0][0][e], sc[nt][0][1][e]), fmaxf(sc[nt][1][0][e], sc[nt][1][1][e])) * kScore;
          moves |= cmax[nt][e] > m[nt][e] + kSlack;
        }
      if (__any_sync(0xffffffffu, moves)) {
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) vmax = fmaxf(vmax, __shfl_xor_sync(0xffffffffu, vmax, o));
        if (vmax * fit.f > kFits) fit.fall(vmax);
#pragma unroll
        for (int nt = 0; nt < NT; nt++) {
          float al[2];
#pragma unroll
          for (int e = 0; e < 2; e++) {
            float mn = cmax[nt][e];
#pragma unroll
            for (int o = 4; o < 32; o <<= 1) mn = fmaxf(mn, __shfl_xor_sync(0xffffffffu, mn, o));
            mn = fmaxf(m[nt][e], mn);
            al[e] = mn == -INFINITY ? 1.f : fast_exp2(m[nt][e] - mn);
            m[nt][e] = mn;
            l[nt][e] *= al[e];
          }
#pragma unroll
          for (int g = 0; g < NG; g++) {
            vacc[nt][0][g] *= al[0];
            vacc[nt][1][g] *= al[1];
          }
#pragma unroll
          for (int ch = 0; ch < CH; ch++)
#pragma unroll
            for (int x = 0; x < 2; x++)
#pragma unroll
              for (int i = 0; i < 4; i++) ov[nt][ch][x][i] *= al[i & 1];
        }
      }
      // ---- p and the sums ----
      uint32_t b[2][NT][NG][2], bl[2][NT][NG][2];  // w rounded, and the rest
#pragma unroll
      for (int u = 0; u < 2; u++) {
        float p[NT][2][2];
#pragma unroll
        for (int nt = 0; nt < NT; nt++)
#pragma unroll
          for (int x = 0; x < 2; x++)
#pragma unroll
            for (int e = 0; e < 2; e++) {
              const float v = sc[nt][u][x][e];
              p[nt][x][e] = EDGE && v == -INFINITY ? 0.f : fast_exp2(fmaf(v, kScore, -m[nt][e]));
              l[nt][e] += p[nt][x][e];
            }
        const __half *const n0 = nbase + OFF / 2 + (2 * kBlock + 16 * u) * NG, *const n1 = n0 + 8 * NG;
        const Nums<NG> vm[2] = {Nums<NG>(n0), Nums<NG>(n1)};
        const Nums<NG> vsc[2] = {Nums<NG>(n0 + kBlock * NG), Nums<NG>(n1 + kBlock * NG)};
#pragma unroll
        for (int g = 0; g < NG; g++)
#pragma unroll
          for (int x = 0; x < 2; x++) {
            const float vs = vsc[x].get(g) * fit.f, vb = vm[x].get(g);
#pragma unroll
            for (int nt = 0; nt < NT; nt++) {
              float w0 = p[nt][x][0] * vs, w1 = p[nt][x][1] * vs, o0 = p[nt][x][0] * vb, o1 = p[nt][x][1] * vb;
              if constexpr (EDGE) {  // masked slots may hold anything
                if (p[nt][x][0] == 0.f) w0 = o0 = 0.f;
                if (p[nt][x][1] == 0.f) w1 = o1 = 0.f;
              }
              vacc[nt][0][g] += o0;
              vacc[nt][1][g] += o1;
              const uint32_t w = pack_h2(w0, w1);
              const float2 r = __half22float2(*reinterpret_cast<const __half2 *>(&w));
              b[u][nt][g][x] = transpose_8x8(w);
              bl[u][nt][g][x] = transpose_8x8(pack_h2(w0 - r.x, w1 - r.y));
            }
          }
      }
      // ---- the output product: a block's MMAs start from zero and are added in fp32 registers (the
      //      tensor core's own additions truncate, and what they lose grows with the sum) ----
#pragma unroll
      for (int ch = 0; ch < CH; ch += 2) {
        uint32_t r[2][4];  // [u]: slots 0-7 and 8-15 of chunk ch, then of chunk ch + 1
        ldmatrix_x4_trans(r[0], vbase + OFF + ch * 16);
        ldmatrix_x4_trans(r[1], vbase + OFF + 16 * RB + ch * 16);
        const int g = ch * 32 / G;
#pragma unroll
        for (int y = 0; y < 2; y++)
#pragma unroll
          for (int x = 0; x < 2; x++) {
            uint32_t lo[2][2], hi[2][2];  // dims 2x (rows gid) and 2x + 1 (rows gid + 8) of the four
#pragma unroll
            for (int u = 0; u < 2; u++)
#pragma unroll
              for (int z = 0; z < 2; z++) {
                const uint32_t w = x ? r[u][2 * y + z] >> 8 : r[u][2 * y + z];
                lo[u][z] = nibble0(w);
                hi[u][z] = nibble1(w);
              }
#pragma unroll
            for (int nt = 0; nt < NT; nt++) {
              float d[4];
              mma_f16_z(d, lo[0][0], hi[0][0], lo[0][1], hi[0][1], b[0][nt][g][0], b[0][nt][g][1]);
              mma_f16(d, lo[1][0], hi[1][0], lo[1][1], hi[1][1], b[1][nt][g][0], b[1][nt][g][1]);
              mma_f16(d, lo[0][0], hi[0][0], lo[0][1], hi[0][1], bl[0][nt][g][0], bl[0][nt][g][1]);
              mma_f16(d, lo[1][0], hi[1][0], lo[1][1], hi[1][1], bl[1][nt][g][0], bl[1][nt][g][1]);
              float(&o)[4] = ov[nt][ch + y][x];
#pragma unroll
              for (int i = 0; i < 4; i++) o[i] = fmaf(d[i], fit.inv, o[i]);
            }
          }
      }
    };

    int t = t_first;
    // one step: wait for stage ST, its block, and the copy of the block two steps on
    auto run = [&](auto stage, int k) -> bool {
      constexpr int ST = decltype(stage)::value;
      if (!mbar_wait_bounded(bar0 + 8 * ST, phase >> ST & 1, nullptr, a.kv.err)) {
        // gave up: the copy in flight lands (or times out) before the stages are written again
        if (k + 1 < steps) mbar_wait_bounded(bar0 + 8 * (ST ^ 1), phase >> (ST ^ 1) & 1, nullptr, a.kv.err);
        ok = false;
        return false;
      }
      phase ^= 1u << ST;
      if (t + kBlock > min(lmin, t_end)) block(stage, std::true_type{}, t);
      else block(stage, std::false_type{}, t);
      if (k + 2 < steps) {
        fence_proxy_async_smem();  // every lane has used the stage before the copy that refills it
        __syncwarp();
        if (((k + 2) & 31) == 0) cp.look_up(a, it.s, it.h, t + 2 * step, step, t_end, lane);
        cp.issue((k + 2) & 31, ST * S::STAGE_B, bar0 + 8 * ST, lane);
      }
      t += step;
      return true;
    };
    for (int k = 0; k < steps; k += 2) {
      if (!run(std::integral_constant<int, 0>{}, k)) break;
      if (k + 1 < steps && !run(std::integral_constant<int, 1>{}, k + 1)) break;
    }
    const bool any_bad = __any_sync(0xffffffffu, cp.bad);
    if (any_bad && lane == 0) {
      atomicOr(a.kv.err, FG_DEVERR_RANGE);
      if (a.shared_unit) bad_page = 1;
    }

    // ---- this warp's columns: totals, and outputs ----
    float *const wo = reinterpret_cast<float *>(wbase);  // [NC][D], in the (drained) stages, for the join below
    const bool good_warp = ok && !any_bad;
#pragma unroll
    for (int nt = 0; nt < NT; nt++) {
#pragma unroll
      for (int e = 0; e < 2; e++) {
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) l[nt][e] += __shfl_xor_sync(0xffffffffu, l[nt][e], o);
#pragma unroll
        for (int g = 0; g < NG; g++)
#pragma unroll
          for (int o = 4; o < 32; o <<= 1) vacc[nt][e][g] += __shfl_xor_sync(0xffffffffu, vacc[nt][e][g], o);
        const int n = nt * kCols + 2 * c + e;
        if (gid == 0) {
          red_m[warp][n] = m[nt][e];
          red_l[warp][n] = l[nt][e];
        }
        if (n >= it.ncols) continue;
        const int cn = it.n0 + n;
        const float inv = len[nt][e] > 0 && good_warp ? 1.0f / l[nt][e] : 0.f;
        const int64_t pi = target.index * NC + n;
        if (!a.shared_unit && !target.whole && gid == 0) a.ml[pi] = make_float2(m[nt][e], good_warp ? l[nt][e] : -1.f);
        __half *const orow = a.out + (static_cast<int64_t>(it.s) * a.rows_per_seq + cn / a.R) * a.ldo +
                             (static_cast<int64_t>(it.h) * a.R + cn % a.R) * D + 4 * gid;
#pragma unroll
        for (int ch = 0; ch < CH; ch++) {
          const float base = vacc[nt][e][ch * 32 / G];
          float v[4];
#pragma unroll
          for (int x = 0; x < 2; x++) {
            v[2 * x] = ov[nt][ch][x][e] * kUnit + base;
            v[2 * x + 1] = ov[nt][ch][x][2 + e] * kUnit + base;
          }
          if (a.shared_unit) {
            *reinterpret_cast<float4 *>(wo + n * D + ch * 32 + 4 * gid) = make_float4(v[0], v[1], v[2], v[3]);
          } else if (!target.whole) {
            *reinterpret_cast<float4 *>(a.po + pi * D + ch * 32 + 4 * gid) = make_float4(v[0], v[1], v[2], v[3]);
          } else {
            uint2 r = make_uint2(0u, 0u);  // (a row that sees nothing, or a bad page: zero, whatever v is)
            if (inv != 0.f) r = make_uint2(pack_h2(v[0] * inv, v[1] * inv), pack_h2(v[2] * inv, v[3] * inv));
            *reinterpret_cast<uint2 *>(orow + ch * 32) = r;
          }
        }
      }
    }
    bool good = good_warp;
    const int w0 = a.shared_unit ? 0 : warp, w1 = a.shared_unit ? kWarps : warp + 1;
    const int me = a.shared_unit ? tid : lane, all = a.shared_unit ? kWarps * 32 : 32;
    if (a.shared_unit) {  // the CTA's warps joined
      good = __syncthreads_and(ok) && !bad_page;
      for (int i = tid; i < it.ncols * (D / 4); i += kWarps * 32) {
        const int n = i / (D / 4), d = 4 * (i % (D / 4));
        float M = -INFINITY, den = 0.f;
        float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int w = 0; w < kWarps; w++) M = fmaxf(M, red_m[w][n]);
#pragma unroll
        for (int w = 0; w < kWarps; w++) {
          const float f = red_m[w][n] == -INFINITY ? 0.f : exp2f(red_m[w][n] - M);
          const float4 v = *reinterpret_cast<const float4 *>(smem + w * S::WARP_B + (n * D + d) * 4);
          den += f * red_l[w][n];
          if (f != 0.f) o = make_float4(o.x + f * v.x, o.y + f * v.y, o.z + f * v.z, o.w + f * v.w);
        }
        const int cn = it.n0 + n;
        const float inv = 1.0f / den;
        uint2 r = make_uint2(0u, 0u);
        if (it.len(cn, a.R) > 0 && good) r = make_uint2(pack_h2(o.x * inv, o.y * inv), pack_h2(o.z * inv, o.w * inv));
        *reinterpret_cast<uint2 *>(a.out + (static_cast<int64_t>(it.s) * a.rows_per_seq + cn / a.R) * a.ldo +
                                   (static_cast<int64_t>(it.h) * a.R + cn % a.R) * D + d) = r;
      }
    } else {
      __syncwarp();
    }
    if (TRACK && target.whole && good) {  // the unit saw whole rows: its slots' weights
      for (int i = 4 * me; i < lmax; i += 4 * all) {
        float4 add = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int n = 0; n < it.ncols; n++) {
          const int end = it.len(it.n0 + n, a.R);
          float M = -INFINITY, den = 0.f;
          for (int w = w0; w < w1; w++) M = fmaxf(M, red_m[w][n]);
          for (int w = w0; w < w1; w++) den += red_m[w][n] == -INFINITY ? 0.f : exp2f(red_m[w][n] - M) * red_l[w][n];
          grow_by(&add, srow + n * a.score_ld, i, end, M, 1.0f / den);
        }
        grow4(a, it.s, it.h, i, lmax, add);
      }
    }
    if (!a.units || !advance(a, &walks[warp], lane)) return;
  }
}

// ------------------------------------------------------------------------------------------------
// One column (one new token, a key-value head of its own): the tile's eight columns hold what one
// column has to offer instead.
//   scores: column 2c of q is zero outside group c % 2, so that lane (gid, c) finds the dot product
//           of slot gid + 8 (c / 2) with group c % 2 in its own fragment; the two lanes of a slot
//           add their groups' shares.
//   output: lane (gid, c) holds w of that slot and group as two fp16 numbers, w's rounding and the
//           rest (22 bits together), in columns 2c and 2c+1 of a matrix whose transpose is the B
//           operand: columns 0-3 for slots 0-7 of the 16, columns 4-7 for slots 8-15.
// A = V codes transposed comes from ldmatrix.trans on 16-bit elements (4 codes of a slot): a lane
// gets two slots' codes of dims 4 gid .. 4 gid + 3, in operand order.
// ------------------------------------------------------------------------------------------------
template <int D, int G>
struct One {
  static constexpr int NG = D / G;  // 1 or 2
  static constexpr int RB = D / 2;
  static constexpr int KW = D / 32;  // K code words per lane and slot
  static constexpr int CH = D / 32;  // 32-dim chunks (16 bytes of codes)
  static constexpr int CODE_B = kBlock * RB, META_B = kBlock * NG * 2;
  static constexpr int STAGE_B = 2 * CODE_B + 4 * META_B;
  static constexpr int WARP_B = 2 * STAGE_B;  // two stages; >= D * 4, the warp's outputs at the end
  static constexpr int SMEM = kWarps * WARP_B;
  static constexpr int kCtas = one_ctas(D);
};

template <int D, int G, bool TRACK>
__global__ void __launch_bounds__(kWarps * 32, One<D, G>::kCtas) paged_attn_one_kernel(const PagedAttnArgs a) {
  using S = One<D, G>;
  constexpr int NG = S::NG, RB = S::RB, KW = S::KW, CH = S::CH;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ __align__(8) uint64_t full_bar[kWarps][2];
  __shared__ float red_m[kWarps], red_l[kWarps];
  __shared__ int bad_page;

  griddep_launch();  // the join may be scheduled once every CTA runs
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int gid = lane >> 2, c = lane & 3;
  const int unit = a.shared_unit ? blockIdx.x : blockIdx.x * kWarps + warp;
  const int first = a.shared_unit ? warp : 0;
  const int step = a.shared_unit ? kCta : kBlock;  // slots from one of this warp's blocks to the next
  if (TRACK && a.units && lane < 2 && unit < a.units) a.parts[2 * unit + lane].item = -1;
  if (a.units && unit == 0) flag_bad_sequences(a, lane);
  __shared__ Walk walks[kWarps];  // (out of the registers: used once per segment)
  {
    Walk w;
    if (!w.begin(a, unit, lane)) return;
    if (lane == 0) walks[warp] = w;
    __syncwarp();
  }

  const uint32_t bar0 = smem_u32(&full_bar[warp][0]);
  if (lane == 0) {
    mbar_init(bar0, 1);
    mbar_init(bar0 + 8, 1);
    fence_mbar_init();
    fence_proxy_async_smem();
  }
  if (a.shared_unit) {
    if (tid == 0) bad_page = 0;
    __syncthreads();
  } else {
    __syncwarp();
  }
  uint8_t *const wbase = smem + warp * S::WARP_B;
  Copies<RB, NG, S::CODE_B, S::META_B> cp;
  cp.init(a, smem_u32(wbase), lane);
  bool ok = true;
  uint32_t phase = 0;  // bit i: the parity of stage i's next phase

  while (true) {  // segments
    const Walk walk = walks[warp];
    const int s = walk.s, h = walk.ht, item = s * a.kv.H + h;
    const int len = load_item(a, s, h, !a.units && first == 0 && lane == 0).len(0, 1);
    const int ran = a.units ? walk.run() : 0;
    const int t_begin = a.units ? walk.b * kBlock : 0;
    const int t_end = a.units ? min(len, t_begin + ran * kBlock) : len;
    const int t_first = t_begin + first * kBlock;
    const int steps = ok && t_end > t_first ? (t_end - t_first + step - 1) / step : 0;
    cp.bad = false;
    if (steps > 0) {
      cp.look_up(a, s, h, t_first, step, t_end, lane);
      cp.issue(0, 0, bar0, lane);
      if (steps > 1) cp.issue(1, S::STAGE_B, bar0 + 8, lane);
    }
    const Target target = target_of(a, walk, unit, item, ran, lane == 0);

    // ---- q as the B operand; word j of lane class c: dims 2o .. 2o+7 ----
    const __half *qrow = a.q + static_cast<int64_t>(s) * a.ldq + static_cast<int64_t>(h) * D;
    uint32_t qf[KW][4];
    float ql;  // sum of q over this lane's group, over kUnit
    const int g = NG == 2 ? c & 1 : 0;
    {
      float part[NG];
#pragma unroll
      for (int i = 0; i < NG; i++) part[i] = 0.f;
#pragma unroll
      for (int j = 0; j < KW; j++) {
        const int o = D == 64 ? 8 * c + 4 * j : 64 * (j >> 2) + 16 * c + 4 * (j & 3);
        uint4 v = make_uint4(0, 0, 0, 0);
        if (len > 0) v = *reinterpret_cast<const uint4 *>(qrow + 2 * o);
        const __half *e = reinterpret_cast<const __half *>(&v);
        float sum = 0.f;
#pragma unroll
        for (int i = 0; i < 8; i++) sum += __half2float(e[i]);
#pragma unroll
        for (int i = 0; i < NG; i++) part[i] += o / (G / 2) == i ? sum : 0.f;
        const bool on = !(gid & 1) && (NG == 1 || o / (G / 2) == ((gid >> 1) & 1));
        if (!on) v = make_uint4(0, 0, 0, 0);
        q_operands(qf[j], v);
      }
#pragma unroll
      for (int i = 0; i < NG; i++) {
        part[i] += __shfl_xor_sync(0xffffffffu, part[i], 1);
        part[i] += __shfl_xor_sync(0xffffffffu, part[i], 2);
      }
      ql = (NG == 2 && g ? part[NG - 1] : part[0]) * (1.0f / kUnit);
    }
    const bool upper = c & 2;  // this lane's slot is gid + 8 of the 16
    const int tq = gid + (upper ? 8 : 0);
    float *const srow = TRACK ? a.scores + static_cast<int64_t>(item) * a.score_ld : nullptr;
    // this lane's places in a stage: K code rows, group numbers, ldmatrix rows of V codes
    const uint8_t *const kbase = wbase + gid * RB + (D == 64 ? 8 : 16) * c;
    const __half *const nbase = reinterpret_cast<const __half *>(wbase + 2 * S::CODE_B) + tq * NG + g;
    const uint32_t vbase = smem_u32(wbase) + S::CODE_B + ((lane >> 3 & 1) * 8 + (lane & 7)) * RB + (lane >> 4) * 16;

    Fit fit;
    float m = -INFINITY, l = 0.f, vacc = 0.f;
    float ov[CH][2][2];  // chunk ch, x: dims 32 ch + 4 gid + 2x and + 1
#pragma unroll
    for (int i = 0; i < CH; i++)
#pragma unroll
      for (int x = 0; x < 2; x++) ov[i][x][0] = ov[i][x][1] = 0.f;

    // one block of 32 slots at t, in stage ST; EDGE: some of them are not seen
    auto block = [&](auto stage, auto edge, int t) {
      constexpr int OFF = decltype(stage)::value * S::STAGE_B;
      constexpr bool EDGE = decltype(edge)::value;
      float sc[2];
#pragma unroll
      for (int u = 0; u < 2; u++) {
        uint32_t k0[KW], k1[KW];
#pragma unroll
        for (int j = 0; j < KW; j += (D == 64 ? 2 : 4)) {
          const uint8_t *p = kbase + OFF + 16 * u * RB + (D == 64 ? 0 : 16 * j);
          if constexpr (D == 64) {
            const uint2 x = *reinterpret_cast<const uint2 *>(p), y = *reinterpret_cast<const uint2 *>(p + 8 * RB);
            k0[j] = x.x, k0[j + 1] = x.y, k1[j] = y.x, k1[j + 1] = y.y;
          } else {
            const uint4 x = *reinterpret_cast<const uint4 *>(p), y = *reinterpret_cast<const uint4 *>(p + 8 * RB);
            k0[j] = x.x, k0[j + 1] = x.y, k0[j + 2] = x.z, k0[j + 3] = x.w;
            k1[j] = y.x, k1[j + 1] = y.y, k1[j + 2] = y.z, k1[j + 3] = y.w;
          }
        }
        float lo[4], hi[4];  // two chains of MMAs
#pragma unroll
        for (int j = 0; j < KW; j++) {
          const Nibbles x0(k0[j]), x1(k1[j]);
          if (j == 0) {
            mma_f16_z(lo, x0.n[0], x1.n[0], x0.n[2], x1.n[2], qf[j][0], qf[j][1]);
            mma_f16_z(hi, x0.n[1], x1.n[1], x0.n[3], x1.n[3], qf[j][2], qf[j][3]);
          } else {
            mma_f16(lo, x0.n[0], x1.n[0], x0.n[2], x1.n[2], qf[j][0], qf[j][1]);
            mma_f16(hi, x0.n[1], x1.n[1], x0.n[3], x1.n[3], qf[j][2], qf[j][3]);
          }
        }
        const __half *n = nbase + OFF / 2 + 16 * u * NG;
        float part = fmaf(__half2float(n[kBlock * NG]), upper ? lo[2] + hi[2] : lo[0] + hi[0], __half2float(n[0]) * ql);
        if constexpr (NG == 2) part += __shfl_xor_sync(0xffffffffu, part, 1);
        sc[u] = part;
      }
      if constexpr (EDGE) {
#pragma unroll
        for (int u = 0; u < 2; u++)
          if (t + 16 * u + tq >= t_end) sc[u] = -INFINITY;
      }
      if constexpr (TRACK) {
        if (!(c & 1))
#pragma unroll
          for (int u = 0; u < 2; u++)
            if (!EDGE || t + 16 * u + tq < t_end) srow[t + 16 * u + tq] = sc[u] * kScore;
      }
      float cmax = fmaxf(sc[0], sc[1]) * kScore;  // scores are held over kUnit
      float vs[2];
#pragma unroll
      for (int u = 0; u < 2; u++) {
        vs[u] = __half2float(nbase[OFF / 2 + (3 * kBlock + 16 * u) * NG]);
        if (EDGE && t + 16 * u + tq >= t_end) vs[u] = 0.f;  // masked slots may hold anything
      }
      const float vmax = fmaxf(fabsf(vs[0]), fabsf(vs[1]));
      if (__any_sync(0xffffffffu, cmax > m + kSlack || vmax * fit.f > kFits)) {  // the running maximum moves, or F falls
        float v = vmax;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
        if (v * fit.f > kFits) fit.fall(v);
#pragma unroll
        for (int o = 2; o < 32; o <<= 1) cmax = fmaxf(cmax, __shfl_xor_sync(0xffffffffu, cmax, o));
        cmax = fmaxf(m, cmax);
        const float al = cmax == -INFINITY ? 1.f : fast_exp2(m - cmax);
        m = cmax;
        l *= al;
        vacc *= al;
#pragma unroll
        for (int i = 0; i < CH; i++)
#pragma unroll
          for (int x = 0; x < 2; x++) {
            ov[i][x][0] *= al;
            ov[i][x][1] *= al;
          }
      }
      uint32_t b[2][2];
#pragma unroll
      for (int u = 0; u < 2; u++) {
        const __half *n = nbase + OFF / 2 + (2 * kBlock + 16 * u) * NG;
        const float p = fast_exp2(fmaf(sc[u], kScore, -m));
        float w = p * (vs[u] * fit.f), pm = p * __half2float(n[0]);
        if (EDGE && t + 16 * u + tq >= t_end) w = pm = 0.f;  // (their p is 0)
        l += p;
        vacc += pm;
        // w rounded, and the rest, in columns 2c and 2c+1 of the slot's row
        uint32_t wp = pack_h2(w, w - __half2float(__float2half_rn(w)));
        if (NG == 1 && (c & 1)) wp = 0u;
        const uint32_t wt = transpose_8x8(wp);
        b[u][0] = gid < 4 ? wt : 0u;
        b[u][1] = gid < 4 ? 0u : wt;
      }
      // the block's MMAs start from zero and are added in fp32 registers (the tensor core's own
      // additions truncate, and what they lose grows with the sum)
#pragma unroll
      for (int ch = 0; ch < CH; ch += 2) {
        uint32_t r[2][4];  // [u]: slots 0-7 and 8-15 of chunk ch, then of chunk ch + 1
        ldmatrix_x4_trans(r[0], vbase + OFF + ch * 16);
        ldmatrix_x4_trans(r[1], vbase + OFF + 16 * RB + ch * 16);
#pragma unroll
        for (int y = 0; y < 2; y++)
#pragma unroll
          for (int x = 0; x < 2; x++) {
            uint32_t lo[2][2], hi[2][2];  // dims 2x (rows gid) and 2x + 1 (rows gid + 8) of the four
#pragma unroll
            for (int u = 0; u < 2; u++)
#pragma unroll
              for (int z = 0; z < 2; z++) {
                const uint32_t w = x ? r[u][2 * y + z] >> 8 : r[u][2 * y + z];
                lo[u][z] = nibble0(w);
                hi[u][z] = nibble1(w);
              }
            float d[4];
            mma_f16_z(d, lo[0][0], hi[0][0], lo[0][1], hi[0][1], b[0][0], b[0][1]);
            mma_f16(d, lo[1][0], hi[1][0], lo[1][1], hi[1][1], b[1][0], b[1][1]);
            ov[ch + y][x][0] = fmaf(d[0] + d[1], fit.inv, ov[ch + y][x][0]);  // both columns of w
            ov[ch + y][x][1] = fmaf(d[2] + d[3], fit.inv, ov[ch + y][x][1]);
          }
      }
    };

    int t = t_first;
    // one step: wait for stage ST, its block, and the copy of the block two steps on
    auto run = [&](auto stage, int k) -> bool {
      constexpr int ST = decltype(stage)::value;
      if (!mbar_wait_bounded(bar0 + 8 * ST, phase >> ST & 1, nullptr, a.kv.err)) {
        // gave up: the copy in flight lands (or times out) before the stages are written again
        if (k + 1 < steps) mbar_wait_bounded(bar0 + 8 * (ST ^ 1), phase >> (ST ^ 1) & 1, nullptr, a.kv.err);
        ok = false;
        return false;
      }
      phase ^= 1u << ST;
      if (t + kBlock > t_end) block(stage, std::true_type{}, t);
      else block(stage, std::false_type{}, t);
      if (k + 2 < steps) {
        fence_proxy_async_smem();  // every lane has used the stage before the copy that refills it
        __syncwarp();
        if (((k + 2) & 31) == 0) cp.look_up(a, s, h, t + 2 * step, step, t_end, lane);
        cp.issue((k + 2) & 31, ST * S::STAGE_B, bar0 + 8 * ST, lane);
      }
      t += step;
      return true;
    };
    for (int k = 0; k < steps; k += 2) {
      if (!run(std::integral_constant<int, 0>{}, k)) break;
      if (k + 1 < steps && !run(std::integral_constant<int, 1>{}, k + 1)) break;
    }
    const bool any_bad = __any_sync(0xffffffffu, cp.bad);
    if (any_bad && lane == 0) {
      atomicOr(a.kv.err, FG_DEVERR_RANGE);
      if (a.shared_unit) bad_page = 1;
    }

    // ---- totals of the warp: every slot was counted by two lanes; group i's min sum in lane i ----
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
    l *= 0.5f;
#pragma unroll
    for (int o = 2; o < 32; o <<= 1) vacc += __shfl_xor_sync(0xffffffffu, vacc, o);
    float o4[CH / NG][4];  // lanes c = group: dims 4 gid .. 4 gid + 3 of its chunks
#pragma unroll
    for (int i = 0; i < CH; i++) {
      const int cg = i / (CH / NG);
      float v[4];
#pragma unroll
      for (int x = 0; x < 2; x++) {
        v[2 * x] = ov[i][x][0] * kUnit;
        v[2 * x + 1] = ov[i][x][1] * kUnit;
      }
#pragma unroll
      for (int x = 0; x < 4; x++) {
        v[x] += __shfl_xor_sync(0xffffffffu, v[x], 2);
        if (NG == 1 || c == cg) o4[i % (CH / NG)][x] = v[x] + vacc;
      }
    }
    const int64_t pi = target.index;
    __half *const orow = a.out + static_cast<int64_t>(s) * a.ldo + static_cast<int64_t>(h) * D;
    if (!a.shared_unit) {
      const bool good = ok && !any_bad;
      if (!target.whole && lane == 0) a.ml[pi] = make_float2(m, good ? l : -1.f);
      const float inv = 1.0f / l;
      const bool on = len > 0 && good;
      if (c < NG) {
#pragma unroll
        for (int i = 0; i < CH / NG; i++) {
          const int d = (c * (CH / NG) + i) * 32 + 4 * gid;
          if (!target.whole) {
            *reinterpret_cast<float4 *>(a.po + pi * D + d) = make_float4(o4[i][0], o4[i][1], o4[i][2], o4[i][3]);
          } else {
            uint2 r = make_uint2(0u, 0u);
            if (on) r = make_uint2(pack_h2(o4[i][0] * inv, o4[i][1] * inv), pack_h2(o4[i][2] * inv, o4[i][3] * inv));
            *reinterpret_cast<uint2 *>(orow + d) = r;
          }
        }
      }
      if (TRACK && target.whole && on) {  // this warp saw the whole row: its slots' weights
        __syncwarp();
        grow_row(a, s, h, srow, 0, t_end, m, inv, lane, 32);
      }
      if (!a.units || !advance(a, &walks[warp], lane)) return;
      continue;
    }
    float *wo = reinterpret_cast<float *>(wbase);
    if (c < NG)
#pragma unroll
      for (int i = 0; i < CH / NG; i++)
        *reinterpret_cast<float4 *>(wo + (c * (CH / NG) + i) * 32 + 4 * gid) =
            make_float4(o4[i][0], o4[i][1], o4[i][2], o4[i][3]);
    if (lane == 0) {
      red_m[warp] = m;
      red_l[warp] = l;
    }
    const bool good = __syncthreads_and(ok) && !bad_page;
    float M = -INFINITY, den = 0.f, f[kWarps];
#pragma unroll
    for (int w = 0; w < kWarps; w++) M = fmaxf(M, red_m[w]);
#pragma unroll
    for (int w = 0; w < kWarps; w++) {
      f[w] = red_m[w] == -INFINITY ? 0.f : exp2f(red_m[w] - M);
      den += f[w] * red_l[w];
    }
    const float inv = 1.0f / den;
    const bool on = len > 0 && good;
    for (int d = 2 * tid; d < D; d += 2 * kWarps * 32) {
      float o0 = 0.f, o1 = 0.f;
#pragma unroll
      for (int w = 0; w < kWarps; w++)
        if (f[w] != 0.f) {
          const float2 v = *reinterpret_cast<const float2 *>(smem + w * S::WARP_B + d * 4);
          o0 += f[w] * v.x;
          o1 += f[w] * v.y;
        }
      *reinterpret_cast<__half2 *>(orow + d) = on ? __floats2half2_rn(o0 * inv, o1 * inv) : __floats2half2_rn(0.f, 0.f);
    }
    if (TRACK && on)  // (the CTA's scores were published by the barrier above)
      grow_row(a, s, h, srow, 0, t_end, M, inv, tid, kWarps * 32);
    return;
  }
}

// Column n of a cut item over the parts that units u0 .. u1 have of it (the first one's begins the
// item), by one warp: maximum and sum; sum 0: nothing seen, or a bad page.
__device__ __forceinline__ float2 join_ml(const PagedAttnArgs &a, int n, int u0, int u1) {
  const int lane = threadIdx.x & 31;
  float M = -INFINITY, den = 0.f;
  bool bad = false;
  for (int u = u0 + lane; u <= u1; u += 32) {
    const float2 v = a.ml[(2 * static_cast<int64_t>(u) + (u == u0)) * a.pcols + n];
    bad |= v.y < 0.f;
    const float mx = fmaxf(M, v.x);
    if (v.x != -INFINITY) den = (M == -INFINITY ? 0.f : den * exp2f(M - mx)) + v.y * exp2f(v.x - mx);
    M = mx;
  }
  float top = M;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
  den = M == -INFINITY ? 0.f : den * exp2f(M - top);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) den += __shfl_xor_sync(0xffffffffu, den, o);
  return make_float2(top, __any_sync(0xffffffffu, bad) ? 0.f : den);
}

constexpr int kJoinWarps = 8;
constexpr int kPartsPerBlock = 2;  // of those whose slots' weights grow
constexpr int kMaxCols = 16;  // columns per item: at most two tiles

// A column's parts number w, w + warps, .. joined by a warp, V dims a lane: their maximum and sum
// (sum < 0: a bad page among them) and outputs.  Parts are read four at a time.
template <int D>
__device__ __forceinline__ float2 join_parts(const PagedAttnArgs &a, int n, int u0, int u1, int w, int warps,
                                             float (&o)[D / 32]) {
  constexpr int V = D / 32, U = 4;
  const int lane = threadIdx.x & 31;
  float M = -INFINITY, den = 0.f;
  bool bad = false;
#pragma unroll
  for (int e = 0; e < V; e++) o[e] = 0.f;
  for (int u = u0 + w; u <= u1; u += U * warps) {
    float2 t[U];
    float v[U][V];
#pragma unroll
    for (int i = 0; i < U; i++) {
      const int x = u + i * warps;
      t[i] = make_float2(-INFINITY, 0.f);
      if (x <= u1) {
        const int64_t pi = (2 * static_cast<int64_t>(x) + (x == u0)) * a.pcols + n;
        t[i] = a.ml[pi];
        const float *p = a.po + pi * D + lane * V;
        if constexpr (V == 2) {
          *reinterpret_cast<float2 *>(v[i]) = *reinterpret_cast<const float2 *>(p);
        } else {
#pragma unroll
          for (int e = 0; e < V; e += 4) *reinterpret_cast<float4 *>(v[i] + e) = *reinterpret_cast<const float4 *>(p + e);
        }
      }
    }
    float mx = M;
#pragma unroll
    for (int i = 0; i < U; i++) {
      mx = fmaxf(mx, t[i].x);
      bad |= t[i].y < 0.f;
    }
    const float keep = M == -INFINITY ? 0.f : exp2f(M - mx);
    den *= keep;
#pragma unroll
    for (int e = 0; e < V; e++) o[e] *= keep;
#pragma unroll
    for (int i = 0; i < U; i++) {
      if (t[i].x == -INFINITY) continue;  // a part that saw nothing of the column
      const float f = exp2f(t[i].x - mx);
      den += f * t[i].y;
#pragma unroll
      for (int e = 0; e < V; e++) o[e] += f * v[i][e];
    }
    M = mx;
  }
  return make_float2(M, bad ? -1.f : den);
}

template <int V>
__device__ __forceinline__ void store_row(__half *dst, const float (&o)[V], float inv) {
  uint32_t r[V / 2];
#pragma unroll
  for (int e = 0; e < V; e += 2) r[e / 2] = pack_h2(o[e] * inv, o[e + 1] * inv);
  if constexpr (V == 2) *reinterpret_cast<uint32_t *>(dst) = r[0];
  else if constexpr (V == 4) *reinterpret_cast<uint2 *>(dst) = make_uint2(r[0], r[1]);
  else *reinterpret_cast<uint4 *>(dst) = make_uint4(r[0], r[1], r[2], r[3]);
}

// The first blocks: a column of an item to a warp, or (wide) to a block: a cut item's parts joined
// into the column's output row, and zeros for items without blocks, which no unit meets.  Behind
// them (accumulate) the weights of the parts' slots, kPartsPerBlock to a block.
template <int D>
__global__ void __launch_bounds__(kJoinWarps * 32) paged_join_kernel(const PagedAttnArgs a, int out_cols, int out_blocks,
                                                                     bool wide) {
  constexpr int V = D / 32;  // dims per lane
  __shared__ float2 col[kPartsPerBlock][kMaxCols];
  __shared__ float part[kJoinWarps][D];
  __shared__ float2 part_ml[kJoinWarps];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, HT = a.kv.H * a.tiles;
  if (static_cast<int>(blockIdx.x) < out_blocks) {
    const int i = wide ? blockIdx.x : blockIdx.x * kJoinWarps + warp;
    if (i >= a.items * out_cols) return;
    const int item = i / out_cols, n = i - item * out_cols;
    const Item it = load_item(a, item / HT, item % HT, false);
    if (n >= it.ncols) return;
    const int cn = it.n0 + n;
    griddep_wait();
    const int2 c = it.live ? a.cut[item] : make_int2(0, 0);
    if (c.x < 0) return;
    float o[V];
    float2 t = make_float2(-INFINITY, 0.f);
#pragma unroll
    for (int e = 0; e < V; e++) o[e] = 0.f;
    const bool sees = it.len(cn, a.R) > 0;
    if (sees) t = join_parts<D>(a, n, c.x, c.y, wide ? warp : 0, wide ? kJoinWarps : 1, o);
    __half *const dst = a.out + (static_cast<int64_t>(it.s) * a.rows_per_seq + cn / a.R) * a.ldo +
                        (static_cast<int64_t>(it.h) * a.R + cn % a.R) * D;
    if (wide && sees) {
#pragma unroll
      for (int e = 0; e < V; e++) part[warp][lane * V + e] = o[e];
      if (lane == 0) part_ml[warp] = t;
      __syncthreads();
      if (warp > 0) return;
      float M = -INFINITY, den = 0.f;
      bool bad = false;
#pragma unroll
      for (int w = 0; w < kJoinWarps; w++) M = fmaxf(M, part_ml[w].x);
#pragma unroll
      for (int e = 0; e < V; e++) o[e] = 0.f;
      for (int w = 0; w < kJoinWarps; w++) {
        bad |= part_ml[w].y < 0.f;
        if (part_ml[w].x == -INFINITY) continue;
        const float f = exp2f(part_ml[w].x - M);
        den += f * part_ml[w].y;
#pragma unroll
        for (int e = 0; e < V; e++) o[e] += f * part[w][lane * V + e];
      }
      t = make_float2(M, bad ? -1.f : den);
    } else if (wide && warp > 0) {
      return;
    }
    const bool good = sees && !(t.y < 0.f);
    if (!good)
#pragma unroll
      for (int e = 0; e < V; e++) o[e] = 0.f;
    const float inv = good ? 1.0f / t.y : 0.f;
    store_row<V>(dst + lane * V, o, inv);
    return;
  }
  constexpr int P = kPartsPerBlock, WP = kJoinWarps / P;  // warps per part
  const int k = warp / WP, w = warp % WP, i = tid % (32 * WP);
  const int number = (blockIdx.x - out_blocks) * P + k;
  griddep_wait();
  Part p;
  p.item = -1;
  if (number < 2 * a.units) p = a.parts[number];
  Item it;
  it.ncols = 0;
  if (p.item >= 0) {
    it = load_item(a, p.item / HT, p.item % HT, false);
    for (int n = w; n < it.ncols; n += WP) {
      const float2 v = it.len(it.n0 + n, a.R) > 0 ? join_ml(a, n, p.u0, p.u1) : make_float2(0.f, 0.f);
      if (lane == 0) col[k][n] = make_float2(v.x, v.y != 0.f ? 1.0f / v.y : 0.f);
    }
  }
  __syncthreads();
  if (p.item < 0) return;
  const float *sc = a.scores + static_cast<int64_t>(p.item) * a.pcols * a.score_ld;
  const int last = min(it.n0 + it.ncols, it.live * a.R) - 1;
  const int end = min(p.t1, last >= it.n0 ? it.len(last, a.R) : 0);
  if (a.pcols == 1) {
    if (col[k][0].y != 0.f) grow_row(a, it.s, it.h, sc, p.t0, end, col[k][0].x, col[k][0].y, i, 32 * WP);
    return;
  }
  for (int t = p.t0 + 4 * i; t < end; t += 4 * 32 * WP) {
    float4 add = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int n = 0; n < it.ncols; n++) {
      const float2 c = col[k][n];
      if (c.y != 0.f) grow_by(&add, sc + n * a.score_ld, t, it.len(it.n0 + n, a.R), c.x, c.y);
    }
    grow4(a, it.s, it.h, t, end, add);
  }
}

struct Plan {
  int tiles, pcols;  // column tiles of pcols columns
  int units;         // of a partitioned launch; 0: an item per warp or CTA
  bool one, shared_unit;
  size_t ml, po, parts, cut, scores, total;  // bytes, each part 256-byte aligned
  int64_t score_ld;
};

size_t align256(size_t x) { return (x + 255) & ~size_t(255); }

void plan_bytes(Plan *p, int64_t items, int D, int limit, bool accumulate) {
  const size_t n = 2 * static_cast<size_t>(p->units);
  p->score_ld = (static_cast<int64_t>(limit) + 31) / 32 * 32;
  p->ml = align256(n * p->pcols * sizeof(float2));
  p->po = align256(n * p->pcols * D * sizeof(float));
  p->parts = accumulate ? align256(n * sizeof(Part)) : 0;
  p->cut = p->units ? align256(static_cast<size_t>(items) * sizeof(int2)) : 0;
  p->scores = accumulate ? align256(static_cast<size_t>(items) * p->pcols * p->score_ld * sizeof(float)) : 0;
  p->total = p->ml + p->po + p->parts + p->cut + p->scores;
}

// Direct launches (units = 0) give an item to a CTA, or to a warp once there are several items for
// each resident one, and write its rows at once.  Partitioned launches run one wave of warps that
// share all blocks evenly (Walk) and a join.  Direct is for short items, and for somewhat longer
// ones where there are many: 30 sequences of 2000 slots and 32 heads of 128 took 58.8 us direct and
// 62.3 partitioned, 8 of them 23.9 and 26.0, one 21.4 and 19.5; 64 tracked ones of 1500 to 2112
// slots 120 and 133; 24 ragged ones of up to 16384 slots and 8 shared heads 95 and 79.  The tile
// kernel wants nearly the same limits (4 columns, heads of 128, half to all of the length; us direct
// and partitioned): 500 slots, 8 items 10.6 and 13.7, 1200 items 42 and 50; 1000 slots, 8 items 15.2
// and 14.3, 240 items 18 and 25; 2000 slots, 64 items 24 and 20, 240 items 30 and 34, 1200 items 94
// and 96; 4000 slots, 240 items 51 and 44.  They are off by 11 % at 4000 slots and 1200 items (162 and
// 146; tracked 259 and 213) and, tracked, by 15 to 21 % for a few items of 1000 slots (20.3 and 17.5); a
// single column's by 4 to 15 % from 1200 items on (500 slots, 4800 items: 89 and 78).
// Two column tiles to an item halve the unpacking; heads of 64 have the registers for it (24
// sequences of 8192 slots, 8 heads of 16 columns: 77 us instead of 89).
// Accumulating launches take the column tiles one after the other, so that a slot's weight is grown
// by one CTA at a time and in a fixed order; each reads the cache again (16 sequences of 4096 slots, 8
// heads of 12 columns: 111 us, of 8 columns 60; the 512 prompt rows above, 64 tiles: 1.07 ms).
Plan make_plan(int64_t pairs, int cols, int D, int G, int limit, bool accumulate, int64_t *items) {
  Plan p;
  p.one = cols == 1 && D / G <= 2;
  p.pcols = p.one ? 1 : cols > kCols && D == 64 ? 2 * kCols : kCols;
  p.tiles = (cols + p.pcols - 1) / p.pcols;
  const int per_sm = p.one ? one_ctas(D) : tile_ctas(D, p.pcols);
  *items = pairs * (accumulate ? 1 : p.tiles);
  const int warps = per_sm * kWarps * fg_sm_count();
  const bool many = *items >= 4LL * warps;
  const int sms = fg_sm_count();
  const bool direct = limit <= 1024 || (limit <= 2048 && *items >= sms) || (limit <= 4096 && *items >= 8LL * sms);
  p.units = direct ? 0 : warps;
  p.shared_unit = !p.units && !many;
  plan_bytes(&p, *items, D, limit, accumulate);
  return p;
}

int plan_limit(const fg_paged_kv *kv, int max_len) {
  const int cap = fg_paged_capacity(kv);
  return max_len && max_len < cap ? max_len : cap;
}

template <typename K>
fg_status set_smem(K kernel, int bytes, bool (&done)[64]) {
  int dev = 0;
  cudaGetDevice(&dev);
  if (dev < 0 || dev >= 64 || done[dev]) return FG_OK;
  const fg_status rc = fg_cuda_check(cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes));
  done[dev] = rc == FG_OK;
  return rc;
}

template <int D, int G, int NT>
fg_status launch_tiles(const PagedAttnArgs &a, unsigned grid, bool accumulate, cudaStream_t st) {
  using S = Shape<D, G, NT>;
  static bool done[2][64] = {{false}};
  const auto kernel = accumulate ? paged_attn_kernel<D, G, NT, true> : paged_attn_kernel<D, G, NT, false>;
  const fg_status rc = set_smem(kernel, S::SMEM, done[accumulate]);
  if (rc != FG_OK) return rc;
  kernel<<<grid, kWarps * 32, S::SMEM, st>>>(a);
  return FG_OK;
}

template <int D, int G>
fg_status launch(PagedAttnArgs a, const Plan &p, int cols, bool accumulate, cudaStream_t st) {
  const int rounds = accumulate ? p.tiles : 1;
  const unsigned grid = p.units         ? p.units / kWarps
                        : p.shared_unit ? a.items
                                        : (static_cast<unsigned>(a.items) + kWarps - 1) / kWarps;
  for (int r = 0; r < rounds; r++) {
    a.tile0 = r;
    fg_status rc = FG_OK;
    if constexpr (D / G <= 2) {
      if (p.one) {
        static bool done[2][64] = {{false}};
        const auto kernel = accumulate ? paged_attn_one_kernel<D, G, true> : paged_attn_one_kernel<D, G, false>;
        if ((rc = set_smem(kernel, One<D, G>::SMEM, done[accumulate])) != FG_OK) return rc;
        kernel<<<grid, kWarps * 32, One<D, G>::SMEM, st>>>(a);
      }
    }
    if (!p.one && p.pcols == kCols) rc = launch_tiles<D, G, 1>(a, grid, accumulate, st);
    if constexpr (D == 64) {
      if (!p.one && p.pcols == 2 * kCols) rc = launch_tiles<D, G, 2>(a, grid, accumulate, st);
    }
    if (rc != FG_OK || (rc = fg_launch_check()) != FG_OK) return rc;
    if (!p.units) continue;
    const int left = cols - r * p.pcols, out_cols = left < p.pcols ? left : p.pcols;
    // a programmatic dependent: its blocks start while the last units run and wait for them
    cudaLaunchConfig_t lc = {};
    // few items have many parts each
    const bool wide = p.units >= 16LL * a.items;
    const int out_blocks = wide ? a.items * out_cols : (a.items * out_cols + kJoinWarps - 1) / kJoinWarps;
    lc.gridDim = dim3(out_blocks + (accumulate ? (2 * p.units + kPartsPerBlock - 1) / kPartsPerBlock : 0));
    lc.blockDim = dim3(kJoinWarps * 32);
    lc.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    lc.attrs = attr;
    lc.numAttrs = 1;
    if ((rc = fg_cuda_check(cudaLaunchKernelEx(&lc, paged_join_kernel<D>, a, out_cols, out_blocks, wide))) != FG_OK) return rc;
    if ((rc = fg_launch_check()) != FG_OK) return rc;
  }
  return FG_OK;
}

}  // namespace

extern "C" size_t fg_paged_attention_workspace_bytes(const fg_paged_kv *kv, int num_q_heads, int rows, int rows_per_seq,
                                                     int max_len, int accumulate) {
  if (fg_paged_validate(kv) != FG_OK || rows <= 0 || rows_per_seq < 1 || num_q_heads < 1 || num_q_heads % kv->num_heads ||
      max_len < 0)
    return 0;
  const int64_t cols = static_cast<int64_t>(num_q_heads / kv->num_heads) * rows_per_seq;
  if (cols > INT32_MAX) return 0;
  int64_t items;
  return make_plan(static_cast<int64_t>(rows / rows_per_seq) * kv->num_heads, static_cast<int>(cols), kv->head_dim,
                   fg_kv_group(kv->group), plan_limit(kv, max_len), accumulate != 0, &items).total;
}

extern "C" fg_status fg_paged_attention(const fg_paged_kv *kv, const fg_half *q, int64_t ldq, int num_q_heads,
                                        fg_half *out, int64_t ldo, int rows, int rows_per_seq,
                                        const int32_t *positions, const int32_t *row_counts, int max_len,
                                        int accumulate, void *workspace, size_t workspace_bytes, void *stream) {
  fg_status rc = fg_paged_validate(kv);
  if (rc != FG_OK) return rc;
  if (num_q_heads < 1 || num_q_heads % kv->num_heads) return FG_ERR_SHAPE;
  if (rows < 0 || rows_per_seq < 1 || rows % rows_per_seq || rows / rows_per_seq > kv->num_seqs) return FG_ERR_SHAPE;
  if (max_len < 0 || (accumulate != 0 && accumulate != 1)) return FG_ERR_INVALID;
  if (accumulate && !kv->weights) return FG_ERR_INVALID;
  if (rows == 0) return FG_OK;
  if (!q || !out || !positions || !fg_aligned16(q) || !fg_aligned16(out) || !fg_aligned16(workspace))
    return FG_ERR_INVALID;
  const int64_t hD = static_cast<int64_t>(num_q_heads) * kv->head_dim;
  if (ldq < hD || ldo < hD || ldq % 8 || ldo % 8) return FG_ERR_SHAPE;
  const int64_t pairs = static_cast<int64_t>(rows / rows_per_seq) * kv->num_heads;
  const int64_t cols = static_cast<int64_t>(num_q_heads / kv->num_heads) * rows_per_seq;
  if (pairs > INT32_MAX || cols > INT32_MAX) return FG_ERR_SHAPE;
  const int limit = plan_limit(kv, max_len);
  int64_t items;
  Plan p = make_plan(pairs, static_cast<int>(cols), kv->head_dim, fg_kv_group(kv->group), limit, accumulate != 0, &items);
  if (items * p.pcols > INT32_MAX / 2) return FG_ERR_SHAPE;
  const size_t have = workspace ? workspace_bytes : 0;
  if (p.total > have && p.units) {  // less scratch: items stay whole, a CTA each
    p.units = 0;
    p.shared_unit = true;
    plan_bytes(&p, items, kv->head_dim, limit, accumulate != 0);
  }
  if (p.total > have) return FG_ERR_WORKSPACE;
  PagedAttnArgs a;
  if (!fg_paged_args(kv, &a.kv)) return FG_ERR_CUDA;
  a.q = reinterpret_cast<const __half *>(q);
  a.ldq = ldq;
  a.out = reinterpret_cast<__half *>(out);
  a.ldo = ldo;
  a.R = num_q_heads / kv->num_heads;
  a.rows_per_seq = rows_per_seq;
  a.limit = limit;
  a.tiles = accumulate ? 1 : p.tiles;
  a.tile0 = 0;
  a.pcols = p.pcols;
  a.items = static_cast<int>(items);
  a.seqs = rows / rows_per_seq;
  a.units = p.units;
  a.shared_unit = p.shared_unit;
  a.positions = positions;
  a.counts = row_counts;
  uint8_t *ws = static_cast<uint8_t *>(workspace);
  a.ml = reinterpret_cast<float2 *>(ws);
  a.po = reinterpret_cast<float *>(ws + p.ml);
  a.parts = reinterpret_cast<Part *>(ws + p.ml + p.po);
  a.cut = reinterpret_cast<int2 *>(ws + p.ml + p.po + p.parts);
  a.scores = accumulate ? reinterpret_cast<float *>(ws + p.ml + p.po + p.parts + p.cut) : nullptr;
  a.score_ld = p.score_ld;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const int n = static_cast<int>(cols);
  const bool acc = accumulate != 0;
  if (fg_kv_group(kv->group) == 64) {
    switch (kv->head_dim) {
      case 64: return launch<64, 64>(a, p, n, acc, st);
      case 128: return launch<128, 64>(a, p, n, acc, st);
      case 256: return launch<256, 64>(a, p, n, acc, st);
    }
  } else {
    switch (kv->head_dim) {
      case 128: return launch<128, 128>(a, p, n, acc, st);
      case 256: return launch<256, 128>(a, p, n, acc, st);
    }
  }
  return FG_ERR_UNSUPPORTED;
}
