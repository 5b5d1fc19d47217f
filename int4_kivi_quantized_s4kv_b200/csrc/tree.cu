// s4kv_tree_attention device side: attention of a tree of drafted tokens over
// the paged cache, its ancestors and itself ("KV-Cache-Optimierung --
// PagedAttention, quantisierter KV, Speculative Cache", "Kernpunkte").
//
// For node i of sequence b and query head j (kv head j / G):
//   out = softmax(sm_scale * q K^T) V
// over the cached tokens (full pages dequantized, code * scale + zero; the
// partial page from the fp16 residual), the node's ancestors and the node.
//
// Work.  A unit is 64 query rows (node, head of the group) of a (sequence, kv
// head); its keys come in tiles of 128: tile 0 holds the drafted tokens (64) and the
// residual rows (16), tile t >= 1 the pages 8(t-1) .. 8t-1.  The tiles of all units
// are laid end to end and cut into one contiguous range a CTA (one persistent CTA
// an SM) -- or, with fewer units than CTAs, each unit into parts -- so that one
// long sequence fills the card; a unit cut between CTAs leaves partial results, which
// its CTAs merge at their end, each a share of the rows.
//
// Tile.  Everything stands transposed: tokens (keys) or channels (values) on the
// MMA's M = 128, query rows on N = 64, so that few rows cost little and both
// dequantized operands are A operands, which live in tensor memory:
//   S^T[token][row]   = K Q^T       K: lane = token,   from 4 K warps
//   O^T[channel][row] += V^T P^T    V: lane = channel, from 4 V warps
// A page's code words are mma fragments, and tcgen05.st's 16-lane shape lays a
// fragment's registers down as they come, so unpacking a page is the same
// straight-line code as in decode attention and no dequantized byte goes through
// shared memory.  Keys: S = sum q (code scale) + sum q zero.  code/4 * scale is kept as
// its fp16 rounding and the exact remainder, cut to e5m2 (a second, fp8 MMA
// against an e5m2 copy of q): the factor 1/4 keeps any fp16 range finite.  Of a product
// code * scale above 1 the cut loses less than 2^-14, and q's rounding 2^-3 of the remainder, at
// most 2^-14 more; below 1 the cut loses less than 2^-14 itself (e5m2's smallest step 2^-16, times 4),
// and below 1/8 there is no remainder left: the product is its fp16 rounding (2^-11 of it).  The zero
// points' share is one number a (page, row): two helper warps compute it with
// mma.sync (8 pages x 64 rows) and hand it over as a tf32 hi + lo pair (21 bits and fp32's
// range: the sum of 128 products of fp16 numbers may be 2^39), which two more MMAs with a
// constant one-hot operand (token -> page) add to S.  Values:
// code * scale + zero, rounded once to fp16.  Weights enter as fp16 hi + lo.
// What is left of the error is the values' rounding, as large as the output's own.
//
// Softmax.  Two groups of 4 warps take 32 query rows each; a thread is a token.  The
// reference of a row is the largest logit of a piece's first tile in which one is above
// -infinity, and moves only when a weight would pass 2^14 (still finite in fp16): a vote of the
// group decides, and moving it (a maximum over the 128 tokens, the sums and O rescaled) is rare.
//
// What bounds it: 176 bytes of int4 cache a token feed 512 R operations (R = nodes x G), so that HBM would for few rows
// and the tensor pipe for many; in fact it is the warps' instruction issue (8100 to 8600 warp instructions a tile, of them
// softmax 2800, keys 1850, values 1270, the rest waiting and issuing; 60 to 69% of the issue slots) and the chain S, softmax,
// O, which one set of accumulators leaves no second of.  Measured, captured and warm: 64 sequences of 8192 tokens, 16 nodes,
// group 4: 402 us, 1.9 TB/s of cache, 0.34 PFLOP/s; 8 of 32768, 64 nodes, group 8: 1480 to 1590 us with the clock, 0.35 to
// 0.37 PFLOP/s; one of 32768: 43 us; two of 50 tokens: 11.4 us.  For short contexts a unit's beginning and end count for more than its tiles,
// and the code that they alone run is fetched each time, so that it is kept small: rolled loops, one copy (64 sequences
// of 300 tokens: 59 us, 75 with loops unrolled; of 20 warps 4 waited for instructions at 61 us, 6 at 75).
#include <cfloat>
#include <type_traits>

#include "kernels.cuh"
#include "tc05.cuh"

namespace s4kv {

namespace {

// warps: K 0-3, V 4-7 and softmax 8-15 (their number mod 4 is the quarter of the
// tensor-memory lanes that they reach), then the single ones
constexpr int kVWarp0 = 4, kSoftmaxWarp0 = 8, kPageWarp = 16, kMmaWarp = 17, kHelpWarp0 = 18;
constexpr int kTreeThreads = 32 * 20;  // 5 warps a scheduler: 96 registers a thread
constexpr int kTile = 128;                 // keys a tile
constexpr int kTilePages = kTile / kPage;  // 8
constexpr int kGroupRows = 32;             // query rows of a softmax group
// Where there are more CTAs than units (TreeSplit).  A unit of fewer than kWholeTiles tiles is not cut: the merge costs as
// much as 4 or 5 tiles, whether its CTAs are two or one a tile.  (Whole below 2 / 6 / 8 tiles, and at least 3 tiles a part:
// one sequence of 300, 500, 700, 900 tokens, 8 kv heads, 17.4, 18.7, 18.3, 17.7 / 15.8, 17.1, 18.1, 17.7 / 15.7, 17.1, 25.3,
// 17.7, and 15.7, 17.1, 22.4, 22.2 us.)  It has kMaxPieces parts at most, one more for each kTilesAPiece of its tiles: a
// row's merge reads them all.  (One unit: with 40, 40 + tiles / 16, 40 + tiles / 4 parts 22.0, 20.7, 20.7 us at 16K tokens,
// 26.1, 24.4, 26.0 at 32K.)
constexpr int kWholeTiles = 6, kMaxPieces = 40, kTilesAPiece = 16;
// In consecutive ranges, the beginning and end of a unit count as so many tiles.  (0 / 3 / 4 / 6 / 8: 128 sequences of 16 to
// 2000 tokens, 8 kv heads, 242 / 191 / 187 / 188 / 179 us; 64 of 300 71.5 / 67.1 / 65.3 / 60.9 / 63.1; 24 of 100 to 4000,
// group 8, 141.7 / 107.4 / 105.3 / 109.3 / 112.0; 64 of 8192 all alike.)  Parts leave CTAs without work, ranges give a CTA
// two units to begin and end: parts are taken while the longest has no more than this many tiles above an even share.
// (Parts / ranges: 100 units of 2048, 5120, 10240 tokens 39.4 / 47.6, 72.1 / 70.3, 127.3 / 106.8 us, 2, 9 and 22 tiles
// above; 76 of them 39.6 / 40.8, 69.7 / 57.5, 126.2 / 87.5, 5, 17 and 36 above.)
constexpr int kUnitTiles = 6;
constexpr float kRefSlack = 14.0f;         // log2 slack of the softmax reference: weights up to 2^14, finite in fp16

constexpr uint32_t kIdescTS = tc05::idesc_f16_f32(128, kTreeRows);
constexpr uint32_t kIdescTZ = tc05::idesc_tf32_f32(128, kTreeRows);
constexpr uint32_t kIdescTS8 = tc05::idesc_e5m2_f32(128, kTreeRows);
constexpr uint32_t kIdescTO = tc05::idesc_f16_f32(128, 2 * kTreeRows) | tc05::kIdescMnB;  // weights hi | lo

// tensor memory, all 512 columns: S, O (hi | lo), K hi [2], V [2], K lo [2]
constexpr uint32_t kTmS = 0, kTmO = 64, kTmKhi = 192, kTmV = 320, kTmKlo = 448;

// shared memory
constexpr uint32_t kQHiBytes = kTreeRows * 256, kQ8Bytes = kTreeRows * 128, kPBytes = kTile * kTreeRows * 2;
constexpr uint32_t kOffQHi = 0;                              // [2]
constexpr uint32_t kOffP = kOffQHi + 2 * kQHiBytes;          // [2][hi, lo]
constexpr uint32_t kOffQ8 = kOffP + 4 * kPBytes;             // [2]
constexpr uint32_t kOffHot = kOffQ8 + 2 * kQ8Bytes;          // one-hot operand [128][8]
constexpr uint32_t kZeroBytes = kTreeRows * 32;               // zero-point operand [64][8]
constexpr uint32_t kOffZero = kOffHot + kTile * 32;          // [2][hi, lo]
constexpr uint32_t kOffRef = kOffZero + 4 * kZeroBytes;      // minus the reference, [2][32] fp32
constexpr uint32_t kOffRed = kOffRef + 2 * 32 * 4;           // [2][4][32] fp32
constexpr uint32_t kOffFlag = kOffRed + 2 * 4 * 32 * 4;      // [2] last-piece flags, tensor memory's address, abort
constexpr uint32_t kOffSplit = kOffFlag + 16;                  // the TreeSplit
constexpr uint32_t kOffCut = kOffSplit + 32;                    // [2][2] the cut units' pieces, TreeCut
constexpr uint32_t kOffOdd = kOffCut + 4 * 32;                 // [4 pieces][4 V warps] drafted values that are not finite
constexpr uint32_t kOffSeen = kOffOdd + 64;                     // [2][group][drafted token] the group's rows that see it
constexpr uint32_t kOffBar = kOffSeen + 2 * 2 * 64 * 4;
constexpr uint32_t kBars = 38;  // (an even number: the ring behind them is aligned)
constexpr uint32_t kOffRing = kOffBar + 8 * kBars;
static_assert(Fmt<4>::kVZero - Fmt<4>::kVScale == 128 && Fmt<2>::kVZero - Fmt<2>::kVScale == 128 &&
                  Fmt<8>::kVZero - Fmt<8>::kVScale == 128, "missing pages: 256 bytes of value scales and zero points");
static_assert(kOffQ8 % 1024 == 0 && kOffRing % 16 == 0, "operand alignment");

template <int kBits>
struct Ring {
  // pages 16 bytes apart, so that the same word of the 8 pages lies in 8 banks
  static constexpr uint32_t kPageStride = Fmt<kBits>::kBlock + 16;
  static constexpr uint32_t kStage = kTilePages * kPageStride;
  static constexpr int kStages = kBits == 8 ? 2 : kBits == 2 ? 6 : 4;
  static constexpr uint32_t kSmem = kOffRing + kStages * kStage + 1024;
};
static_assert(Ring<4>::kSmem <= 227 * 1024 && Ring<8>::kSmem <= 227 * 1024 && Ring<2>::kSmem <= 227 * 1024, "smem");

// A sequence's share of the work; n = 0 where it has none.
struct TreeSeq {
  int c0, n, L, tiles, blocks;
  uint32_t bad;
};
__device__ __forceinline__ TreeSeq tree_seq(const TreeParams &p, int b) {
  TreeSeq s;
  s.c0 = __ldg(p.cu_nodes + b);
  const int c1 = __ldg(p.cu_nodes + b + 1);
  s.L = __ldg(p.seq_lens + b);
  s.bad = 0;
  s.n = 0;
  if (s.c0 < 0 || c1 < s.c0 || c1 > p.n_nodes || c1 - s.c0 > p.max_nodes) s.bad = S4KV_EFLAG_TREE;
  else if (c1 > s.c0 && (s.L < 0 || s.L > p.max_pages * kPage)) s.bad = S4KV_EFLAG_SEQ_LEN;
  else s.n = c1 - s.c0;
  s.tiles = s.n > 0 ? 1 + (s.L / kPage + kTilePages - 1) / kTilePages : 0;
  s.blocks = (s.n * p.group + kTreeRows - 1) / kTreeRows;
  return s;
}

// A warp's place in the flattened (sequence, kv head, row block, tile) order.
struct TreeWalk {
  TreeSeq s;
  int b, h, rb;
  int tile, rem;    // first tile of the current piece, tiles (with kUnitTiles before each further unit) left from it on
  long long start;  // flattened index of the unit's tile 0 (ranges only)
  __device__ __forceinline__ int take() const { return min(rem, s.tiles - tile); }
  __device__ __forceinline__ int pages(int t) const { return min(kTilePages, s.L / kPage - kTilePages * (t - 1)); }
  __device__ __forceinline__ void next(const TreeParams &p) {
    const int t = take();
    rem -= t + kUnitTiles;
    start += s.tiles + kUnitTiles;
    tile = 0;
    if (rem <= 0) return;
    if (++rb < s.blocks) return;
    rb = 0;
    if (++h < p.num_kv_heads) return;
    h = 0;
    do {
      s = tree_seq(p, ++b);
    } while (s.n == 0 && b + 1 < p.batch);
  }
};

// A unit that is cut between CTAs: where it lies, its CTAs, and this group's rows.
struct TreeCut {
  long long out;  // offset of the sequence's kv head in out
  int first, last, odd, row0, rows, ticket;
};
static_assert(sizeof(TreeCut) == 32, "kOffCut");

// How the units' tiles are dealt out.  With at least as many CTAs as units, a CTA takes a part of one unit (first ..
// last: its unit's CTAs), so that none has two beginnings and ends; the CTAs that units leave over are shared out by
// tiles.  With fewer CTAs, or where that would leave too much to one of them, W CTAs take consecutive ranges of all
// units' positions, the first `extra` of `each` + 1, the others of `each` > kUnitTiles: a unit has kUnitTiles positions
// for its beginning and end, then one a tile (so that every range has a tile).
struct TreeSplit {
  long long each;  // 0: parts of one unit
  int extra, first, last;
  // first position of CTA c's range, CTA of a position
  __device__ __forceinline__ long long begin(int c) const { return c * each + min(c, extra); }
  __device__ __forceinline__ int cta_of(long long x) const {
    const long long longer = extra * (each + 1);
    return static_cast<int>(x < longer ? div(x, each + 1) : extra + div(x - longer, each));
  }
  // 64-bit quotients are slow and next to never needed
  static __device__ __forceinline__ long long div(long long x, long long y) {
    return ((x | y) >> 32) == 0 ? static_cast<long long>(static_cast<uint32_t>(x) / static_cast<uint32_t>(y)) : x / y;
  }
  // CTAs of a unit of `tiles` tiles; `spare` = (CTAs - units) / tiles of all units, less 2^-20 of it for the roundings, so
  // that all units' together are no more than there are
  static __device__ __forceinline__ int parts(int tiles, float spare) {
    const uint32_t t = tiles, c = 1 + static_cast<uint32_t>(static_cast<float>(t) * spare);
    return t < kWholeTiles ? 1 : min(min(c, t), kMaxPieces + t / kTilesAPiece);
  }
};

__device__ __forceinline__ void group_sync(int id) { asm volatile("barrier.cta.sync %0, 128;" ::"r"(id) : "memory"); }
__device__ __forceinline__ bool group_any(int id, bool x) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\tbarrier.cta.red.or.pred q, %2, 128, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"(x ? 1u : 0u), "r"(id)
      : "memory");
  return r != 0;
}
// Lane j's v[0] becomes the reduction over the warp's lanes of every lane's v[j];
// the rest of v is used up.
template <typename Op>
__device__ __forceinline__ float warp_reduce_rows(float (&v)[32], int lane, Op op) {
#pragma unroll
  for (int s = 16; s > 0; s >>= 1) {
    const bool up = lane & s;
#pragma unroll
    for (int j = 0; j < s; ++j) {
      const float keep = up ? v[j + s] : v[j], send = up ? v[j] : v[j + s];
      v[j] = op(keep, __shfl_xor_sync(0xFFFFFFFFu, send, s));
    }
  }
  return v[0];
}

__device__ __forceinline__ uint32_t hmul2_u32(uint32_t a, uint32_t b) { return h2_as_u32(__hmul2(u32_as_h2(a), u32_as_h2(b))); }

// Exactly code / 4 from tile_codes' units, and the codes themselves.
template <int kBits>
__device__ __forceinline__ uint32_t quarter_unit() { return kBits == 4 ? 0x58005800u : 0x34003400u; }  // 128 (codes come as code / 512), 1/4
template <int kBits>
__device__ __forceinline__ void tile_codes(uint32_t w0, uint32_t w1, int parity, uint32_t (&a)[4]) {
  if (kBits == 4) unpack_codes_s9(w0, a[0], a[1], a[2], a[3]);
  else if (kBits == 8) unpack_codes8(w0, w1, a[0], a[1], a[2], a[3]);
  else if (parity) unpack_codes2<1>(w0, a[0], a[1], a[2], a[3]);
  else unpack_codes2<0>(w0, a[0], a[1], a[2], a[3]);
}

}  // namespace

template <int kBits>
__global__ void __launch_bounds__(kTreeThreads, 1) tree_kernel(const TreeParams p) {
  using F = Fmt<kBits>;
  using R = Ring<kBits>;
  constexpr unsigned kAll = 0xFFFFFFFFu;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_addr(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t *sm = smem_raw + (base - raw);
  volatile int *abort_flag = reinterpret_cast<volatile int *>(sm + kOffFlag + 12);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int H = p.num_kv_heads, G = p.group, B = p.batch;

  // barriers: a count of uses gives each its phase
  auto bar = [&](int i) { return base + kOffBar + 8u * i; };
  auto full = [&](int s) { return bar(s); };          // page stages: the page warp and its copies
  auto empty = [&](int s) { return bar(6 + s); };     // (10: K, V and helper warps)
  auto k_ready = [&](int x) { return bar(12 + x); };  // K and the zero-point operand written (6: K and helper warps)
  auto k_free = [&](int x) { return bar(14 + x); };
  auto v_ready = [&](int x) { return bar(16 + x); };
  auto v_free = [&](int x) { return bar(18 + x); };
  const uint32_t s_full = bar(20), s_free = bar(22);
  auto merged = [&](int g) { return bar(21 + 2 * g); };  // a group's items to merge have come
  auto p_full = [&](int x) { return bar(24 + x); };
  auto p_free = [&](int x) { return bar(26 + x); };
  auto q_full = [&](int x) { return bar(28 + x); };
  auto q_free = [&](int x) { return bar(30 + x); };
  auto seen_full = [&](int x) { return bar(32 + x); };
  auto seen_free = [&](int x) { return bar(34 + x); };
  const uint32_t mma_done = bar(36);  // every product has completed

  // ---- barriers and the one-hot operand, while the plan's first loads come
  const int per = (B + 31) >> 5, b_lo = min(B, lane * per), b_hi = min(B, b_lo + per);
  // (a batch of up to 32 has one sequence a lane, read once)
  const TreeSeq mine0 = tree_seq(p, min(b_lo, B - 1));
  if (warp == 0) {
    for (int i = lane; i < static_cast<int>(kBars); i += 32) {
      // their arrivals, 4 bits a barrier
      const unsigned long long counts = i < 16 ? 0x1166AAAAAA111111ull : i < 32 ? 0x1122118818111144ull : 0x118811ull;
      mbar_init(bar(i), static_cast<uint32_t>(counts >> (4 * (i & 15))) & 15u);
    }
    if (lane == 0) *abort_flag = 0;
    fence_barrier_init();
  }
  // the one-hot operand: token t counts the share of page t / 16, in quarters as the keys
#pragma unroll 1
  for (int i = tid; i < kTile * 8; i += kTreeThreads) {
    const int t = i >> 3, k = i & 7;
    sts32(base + kOffHot + tc05::plain_tf32_offset(t, k), k == t / kPage ? __float_as_uint(0.25f) : 0u);
  }

  // ---- plan: every warp finds this CTA's range for itself
  TreeWalk w;
  {
    long long sum = 0;
    uint32_t units = 0;  // at most 2^30
    uint32_t bad = 0;
    auto seq = [&](int b) { return b == b_lo ? mine0 : tree_seq(p, b); };
#pragma unroll 1
    for (int b = b_lo; b < b_hi; ++b) {
      const TreeSeq s = seq(b);
      bad |= s.bad;
      sum += static_cast<long long>(s.tiles) * s.blocks * H;
      units += s.blocks * H;
    }
    if (blockIdx.x == 0 && warp == 0 && bad) flag_error(p.err, bad);
    units = __reduce_add_sync(kAll, units);
    // tiles, at most 2^24 a unit
    const long long T = (static_cast<long long>(__reduce_add_sync(kAll, static_cast<uint32_t>(sum >> 24))) << 24) +
                        __reduce_add_sync(kAll, static_cast<uint32_t>(sum) & 0xFFFFFFu);
    if (T == 0) return;
    const long long all = T + static_cast<long long>(kUnitTiles) * units;  // positions
    const long long even = TreeSplit::div(all, p.num_ctas);
    bool parts = units <= static_cast<uint32_t>(p.num_ctas);
    const float spare = __fdividef(static_cast<float>(p.num_ctas - static_cast<int>(units)), static_cast<float>(T)) * (1.0f - 0x1p-20f);
    if (parts) {
      bool fits = true;  // the longest part
#pragma unroll 1
      for (int b = b_lo; b < b_hi; ++b) {
        const TreeSeq s = seq(b);
        if (s.tiles > 0) fits = fits && s.tiles <= TreeSplit::parts(s.tiles, spare) * (kUnitTiles + even);
      }
      parts = __all_sync(kAll, fits);
    }
    // what is scanned: a sequence's CTAs or its positions, and a unit's
    auto share_of = [&](const TreeSeq &s) {
      return parts ? TreeSplit::parts(s.tiles, spare) : s.tiles + kUnitTiles;
    };
    sum = 0;
#pragma unroll 1
    for (int b = b_lo; b < b_hi; ++b) {
      const TreeSeq s = seq(b);
      sum += static_cast<long long>(s.blocks) * H * share_of(s);
    }
    long long incl = sum;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const long long t = __shfl_up_sync(kAll, incl, off);
      if (lane >= off) incl += t;
    }
    int W = p.num_ctas;
    if (parts) W = static_cast<int>(__shfl_sync(kAll, incl, 31));
    else if (even <= kUnitTiles) W = static_cast<int>(TreeSplit::div(all, kUnitTiles + 1));
    if (static_cast<int>(blockIdx.x) >= W) return;  // the whole CTA
    TreeSplit split = {0, 0, 0, 0};
    long long s0 = blockIdx.x;
    w.rem = 0;
    if (!parts) {
      split.each = TreeSplit::div(all, W);
      split.extra = static_cast<int>(all - split.each * W);
      s0 = split.begin(blockIdx.x);
      w.rem = static_cast<int>(split.begin(blockIdx.x + 1) - s0);
    }
    const long long excl = incl - sum;
    const unsigned hit = __ballot_sync(kAll, excl <= s0 && s0 < incl);
    const int src = __ffs(hit) - 1;
    int bs = 0;
    long long pre = excl;
    if (lane == src) {
#pragma unroll 1
      for (bs = b_lo; bs < b_hi; ++bs) {
        const TreeSeq s = seq(bs);
        const long long mine = static_cast<long long>(s.blocks) * H * share_of(s);
        if (s0 < pre + mine) break;
        pre += mine;
      }
    }
    w.b = __shfl_sync(kAll, bs, src);
    pre = __shfl_sync(kAll, pre, src);
    w.s = tree_seq(p, w.b);
    const int each = share_of(w.s);
    const int u = static_cast<int>(TreeSplit::div(s0 - pre, each)), k = static_cast<int>(s0 - pre - static_cast<long long>(u) * each);
    w.h = u / w.s.blocks;
    w.rb = u - w.h * w.s.blocks;
    w.start = pre + static_cast<long long>(u) * each + kUnitTiles;
    w.tile = max(0, k - kUnitTiles);
    w.rem -= max(0, kUnitTiles - k);
    if (parts) {  // part k of the unit
      split.first = static_cast<int>(blockIdx.x) - k;
      split.last = split.first + each - 1;
      const uint32_t t = w.s.tiles;  // t (k + 1) < 2^32
      w.tile = static_cast<int>(t * k / each);
      w.rem = static_cast<int>(t * (k + 1) / each) - w.tile;
    }
    if (tid == 0) *reinterpret_cast<TreeSplit *>(sm + kOffSplit) = split;  // for the merge of cut units
  }

  // ---- setup
  if (warp == kMmaWarp) {
    tc05::tmem_alloc(base + kOffFlag + 8, 512);
    tc05::tmem_relinquish();
    tc05::fence_before_sync();
  }
  fence_proxy_async();
  __syncthreads();
  tc05::fence_after_sync();
  const uint32_t tmem = lds32_at(base + kOffFlag + 8);
  bool failed = false;
  auto fail = [&]() {
    failed = true;
    *abort_flag = 1;
  };
  auto wait_warp = [&](uint32_t b_, uint32_t parity) { return wait_warp_abort(b_, parity, abort_flag); };
  // the phase of the use before the one of count k, of two buffers in turn
  auto prev2 = [](int k) { return static_cast<uint32_t>(((k >> 1) - 1) & 1); };

  if (warp == kPageWarp) {
    // ------------------------------------------------- pages into the ring
    // and who sees whom: the rows of either group that see a drafted token
    auto see = [&](int su, int (&up)[2]) {
      const int n = w.s.n;
      if (su >= 2 && !wait_warp(seen_free(su & 1), prev2(su))) return false;
      // ancestors of nodes lane and lane + 32, themselves among them, by pointer doubling
      unsigned long long anc[2];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int a = lane + 32 * e;
        if (up[e] < -1 || up[e] >= a) {
          if (a < n) flag_error(p.err, S4KV_EFLAG_TREE);
          up[e] = -1;
        }
        anc[e] = 1ull << a;
      }
#pragma unroll 1
      for (int s = 1; s < n; s <<= 1) {
        unsigned long long m[2];
        int u[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const unsigned long long m0 = __shfl_sync(kAll, anc[0], up[e] & 31), m1 = __shfl_sync(kAll, anc[1], up[e] & 31);
          const int u0 = __shfl_sync(kAll, up[0], up[e] & 31), u1 = __shfl_sync(kAll, up[1], up[e] & 31);
          m[e] = up[e] < 0 ? 0ull : up[e] < 32 ? m0 : m1;
          u[e] = up[e] < 0 ? -1 : up[e] < 32 ? u0 : u1;
        }
        anc[0] |= m[0];
        anc[1] |= m[1];
        up[0] = u[0];
        up[1] = u[1];
        if (!__any_sync(kAll, up[0] >= 0 || up[1] >= 0)) break;
      }
      // turned round, node by node: its rows (of all 64) see the tokens lane and lane + 32 if these are among its ancestors;
      // rows that the unit does not have see token 0, so that their sums are finite
      const int first = kTreeRows * w.rb, rows = min(kTreeRows, n * G - first);
      unsigned long long seen[2] = {lane == 0 && rows < kTreeRows ? ~0ull << rows : 0ull, 0ull};
#pragma unroll 1
      for (int node = first / G; node * G < first + rows; ++node) {
        const unsigned long long m = node < 32 ? __shfl_sync(kAll, anc[0], node) : __shfl_sync(kAll, anc[1], node - 32);
        const int from = max(node * G - first, 0), to = min(node * G + G - first, rows);  // 0 <= from < to <= 64
        const unsigned long long mine = ~0ull >> (64 - (to - from)) << from;
        if (m >> lane & 1) seen[0] |= mine;
        if (m >> (lane + 32) & 1) seen[1] |= mine;
      }
      const uint32_t at = base + kOffSeen + 4 * (128 * (su & 1) + lane);
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        sts32(at + 128 * e, static_cast<uint32_t>(seen[e]));
        sts32(at + 128 * e + 256, static_cast<uint32_t>(seen[e] >> 32));
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(seen_full(su & 1));
      return true;
    };
    int k = 0, su = 0;  // stages filled, pieces with a tile 0
    while (w.rem > 0 && !failed) {
      const int t1 = w.tile + w.take();
      const int32_t *bt = p.block_tables + static_cast<long>(w.b) * p.max_pages;
      const uint8_t *head = p.pool + static_cast<long long>(w.h) * F::kBlock;
      const int t0 = max(w.tile, 1);
      // masks are made while the ring is full, but the first piece's behind the copies of its first pages
      const int t_see = w.tile > 0 ? t1 + 1 : k > 0 ? t0 : min(t0 + 1, t1);
      // the ids of 4 tiles are read at once, before the 4 tiles ahead of them are fetched
      const int last = min(w.s.L / kPage, kTilePages * (t1 - 1));
      auto ids_of = [&](int t) { return kTilePages * (t - 1) + lane < last ? __ldg(bt + kTilePages * (t - 1) + lane) : 0; };
      int ids = t0 < t1 ? ids_of(t0) : 0, ids_next = t0 + 4 < t1 ? ids_of(t0 + 4) : 0;
      int up[2];
#pragma unroll
      for (int e = 0; e < 2; ++e)
        up[e] = w.tile == 0 && lane + 32 * e < w.s.n ? __ldg(p.parents + w.s.c0 + lane + 32 * e) : -1;
#pragma unroll 1
      for (int t = t0;; ++t, ++k) {
        if (t == t_see && !see(su++, up)) {
          fail();
          break;
        }
        if (t >= t1) break;
        const int np = w.pages(t), st = k % R::kStages;
        int phys = __shfl_sync(kAll, ids, (kTilePages * (t - t0) + lane) & 31);
        if (((t - t0) & 3) == 3) {
          ids = ids_next;
          ids_next = t + 5 < t1 ? ids_of(t + 5) : 0;
        }
        if (k >= R::kStages && !wait_warp(empty(st), (k / R::kStages - 1) & 1)) {
          fail();
          break;
        }
        // missing pages: value = code * 0 + 0, which a weight of 0 leaves alone (what the stage held might not be finite)
#pragma unroll 1
        for (int y = 16 * np + lane; y < 16 * kTilePages; y += 32)
          sts128(base + kOffRing + st * R::kStage + (y >> 4) * R::kPageStride + F::kVScale + 16 * (y & 15), make_uint4(0, 0, 0, 0));
        if (np < kTilePages) fence_proxy_async();
        __syncwarp();
        if (lane == 0) mbar_arrive_expect_tx(full(st), np * F::kBlock);
        __syncwarp();
        if (lane < np) {
          if (static_cast<unsigned>(phys) >= static_cast<unsigned>(p.num_pages)) {
            flag_error(p.err, S4KV_EFLAG_PAGE_RANGE);
            phys = 0;
          }
          bulk_copy_g2s(base + kOffRing + st * R::kStage + lane * R::kPageStride,
                        head + static_cast<long long>(phys) * H * F::kBlock, F::kBlock, full(st));
        }
      }
      w.next(p);
    }
    // before the CTA exits the copies in flight must have landed, after an abort too
    for (int j = max(0, k - R::kStages); j < k; ++j) wait_landed(full(j % R::kStages), (j / R::kStages) & 1);
  } else if (warp < kSoftmaxWarp0 || warp >= kHelpWarp0) {
    // ------------------------- K warps, V warps, helpers: a tile's operands
    const int n = lane >> 2, i = lane & 3;
    const bool is_v = warp >= kVWarp0 && warp < kSoftmaxWarp0, is_help = warp >= kHelpWarp0;
    const int wq = warp & 3;                  // K, V: quarter of the lanes
    const int hw = warp - kHelpWarp0;         // helpers: rows 32 hw ..
    const uint32_t lane_base = static_cast<uint32_t>(32 * wq) << 16;
    int k = 0, kt = 0, uc = 0;  // stages read, tiles, pieces
    while (w.rem > 0 && !failed) {
      const int t1 = w.tile + w.take();
      if (is_help) {
        // the unit's queries into shared memory, in the MMA's channel order (fp16: position 16 j + 8 e + 2 i + x holds
        // channel 32 i + 4 j + 2 e + x; e5m2: position 16 j + 4 i + y channel 32 i + 4 j + y)
        if (uc >= 2 && !wait_warp(q_free(uc & 1), prev2(uc))) {
          fail();
          break;
        }
        const int r = 32 * hw + lane, row = kTreeRows * w.rb + r;
        const bool real = row < w.s.n * G;
        const uint4 *src = reinterpret_cast<const uint4 *>(
            p.q + (static_cast<long>(w.s.c0 + (real ? row / G : 0)) * p.num_q_heads + w.h * G + (real ? row % G : 0)) * kHeadDim);
        const uint32_t qh = base + kOffQHi + (uc & 1) * kQHiBytes, q8 = base + kOffQ8 + (uc & 1) * kQ8Bytes;
        uint4 x[16];
#pragma unroll
        for (int c = 0; c < 16; ++c) x[c] = real ? __ldg(src + c) : make_uint4(0, 0, 0, 0);
#pragma unroll
        for (int t = 0; t < 4; ++t) {
          // words of channels 32 c + 8 t ..: tiles 2t (x, y) and 2t + 1 (z, w)
          const uint4 &a = x[t], &b = x[4 + t], &c = x[8 + t], &d = x[12 + t];
          sts128(qh + tc05::sw128_offset(r, 32 * t, kTreeRows), make_uint4(a.x, b.x, c.x, d.x));
          sts128(qh + tc05::sw128_offset(r, 32 * t + 8, kTreeRows), make_uint4(a.y, b.y, c.y, d.y));
          sts128(qh + tc05::sw128_offset(r, 32 * t + 16, kTreeRows), make_uint4(a.z, b.z, c.z, d.z));
          sts128(qh + tc05::sw128_offset(r, 32 * t + 24, kTreeRows), make_uint4(a.w, b.w, c.w, d.w));
          auto e5 = [](uint32_t lo, uint32_t hi) {
            return e5m2x2_of_f16x2(lo) | static_cast<uint32_t>(e5m2x2_of_f16x2(hi)) << 16;
          };
          sts128(q8 + tc05::sw128_offset_b8(r, 32 * t), make_uint4(e5(a.x, a.y), e5(b.x, b.y), e5(c.x, c.y), e5(d.x, d.y)));
          sts128(q8 + tc05::sw128_offset_b8(r, 32 * t + 16), make_uint4(e5(a.z, a.w), e5(b.z, b.w), e5(c.z, c.w), e5(d.z, d.w)));
        }
        fence_proxy_async();
        __syncwarp();
        if (lane == 0) mbar_arrive(q_full(uc & 1));
      }
      for (int t = w.tile; t < t1; ++t, ++kt) {
        const int x2 = kt & 1;
        if (kt >= 2 && !wait_warp(is_v ? v_free(x2) : k_free(x2), prev2(kt))) {
          fail();
          break;
        }
        tc05::fence_after_sync();
        const uint32_t tKhi = tmem + kTmKhi + 64u * x2, tKlo = tmem + kTmKlo + 32u * x2, tV = tmem + kTmV + 64u * x2;
        if (t > 0) {
          const int np = w.pages(t), st = k % R::kStages;
          const uint32_t stage = base + kOffRing + st * R::kStage;
          if (!wait_warp(full(st), (k / R::kStages) & 1)) {
            fail();
            break;
          }
          ++k;
          if (is_help) {
            // rows 32 hw .. + 31 (two 16-row A tiles, by ldmatrix from the queries' shared-memory tile) times the zero
            // points of the 8 pages (B: page n), which lie in the same channel order
            float acc[2][4] = {};
            const uint32_t z = stage + n * R::kPageStride + F::kKZero + 4 * i;
            const uint32_t qh = base + kOffQHi + (uc & 1) * kQHiBytes;
            const int r = 32 * hw + (lane & 15);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              uint32_t b0 = lds32_at(z + 32 * j), b1 = lds32_at(z + 32 * j + 16);
              if (n >= np) b0 = b1 = 0;
              const uint32_t qr = qh + tc05::sw128_offset(r, 16 * j + 8 * (lane >> 4), kTreeRows);
              uint32_t a[4], c[4];
              ldmatrix_x4<0>(qr, a[0], a[1], a[2], a[3]);
              ldmatrix_x4<16 * 128>(qr, c[0], c[1], c[2], c[3]);
              mma16816(acc[0], a[0], a[1], a[2], a[3], b0, b1);
              mma16816(acc[1], c[0], c[1], c[2], c[3], b0, b1);
            }
            // shares of pages 2i, 2i + 1 for rows n, n + 8, hi and what it leaves, of which the MMA takes 11 bits (rounded by
            // integer instructions: with cvt.rna.tf32 for both 64 sequences of 300 tokens took 59.8 us for 58.7)
            const uint32_t zo = base + kOffZero + x2 * (2 * kZeroBytes);
#pragma unroll
            for (int m = 0; m < 2; ++m) {
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                const float v0 = acc[m][2 * e], v1 = acc[m][2 * e + 1];
                const float h0 = tc05::round_tf32(v0), h1 = tc05::round_tf32(v1);
                const uint32_t at = zo + tc05::plain_tf32_offset(32 * hw + 16 * m + 8 * e + n, 2 * i);
                sts64(at, __float_as_uint(h0), __float_as_uint(h1));
                sts64(at + kZeroBytes, __float_as_uint(v0 - h0), __float_as_uint(v1 - h1));
              }
            }
          } else if (is_v) {
            // pages in batches of 4 (missing ones have scale and zero point 0); lanes 0-15 of the quarter: channels 32 wq + 4n + {0, 1}, 16-31: + {2, 3}
            const uint32_t sv = stage + F::kVScale + 32 * i + 4 * wq, zv = stage + F::kVZero + 32 * wq + 4 * i;
            const uint32_t cv = stage + F::kVCode + (kBits == 8 ? 512 * wq + 16 * lane
                                                     : kBits == 4 ? 512 * (wq >> 1) + 16 * lane + 8 * (wq & 1) : 16 * lane + 4 * wq);
            auto page = [&](int pg, uint32_t *a, uint32_t *c) {
              const uint32_t off = pg * R::kPageStride;
              const uint32_t s0 = lds32_at(sv + off), s1 = lds32_at(sv + off + 16), z0 = lds32_at(zv + off), z1 = lds32_at(zv + off + 16);
              uint32_t x[4], y[4];
              if (kBits == 8) {
                const uint4 cw = lds128_at(cv + off);
                tile_codes<kBits>(cw.x, cw.y, 0, x);
                tile_codes<kBits>(cw.z, cw.w, 1, y);
              } else if (kBits == 4) {
                const uint2 cw = lds64_at(cv + off);
                tile_codes<kBits>(cw.x, 0, 0, x);
                tile_codes<kBits>(cw.y, 0, 1, y);
              } else {
                const uint32_t cw = lds32_at(cv + off);
                tile_codes<kBits>(cw, 0, 0, x);
                tile_codes<kBits>(cw, 0, 1, y);
              }
#pragma unroll
              for (int r = 0; r < 4; ++r) {
                if (kBits == 4) {
                  x[r] = hmul2_u32(x[r], 0x60006000u);  // * 512: the codes
                  y[r] = hmul2_u32(y[r], 0x60006000u);
                }
                a[r] = hfma2_u32(x[r], r < 2 ? s0 : s1, r < 2 ? z0 : z1);
                c[r] = hfma2_u32(y[r], r < 2 ? s0 : s1, r < 2 ? z0 : z1);
              }
            };
#pragma unroll 1
            for (int pb = 0; pb < kTilePages; pb += 4) {
              uint32_t o0[16], o1[16];
#pragma unroll
              for (int j = 0; j < 4; ++j) page(pb + j, o0 + 4 * j, o1 + 4 * j);
              tc05::tmem_st_frag16(tV + lane_base + 8 * pb, o0);
              tc05::tmem_st_frag16(tV + lane_base + (16u << 16) + 8 * pb, o1);
            }
          } else {
            // two pages a warp, half of a page's tiles at a time (unrolled by 2 64 sequences of 300 tokens took 61.6 us for
            // 57.3, 64 of 8192 395.4 for 396.2)
#pragma unroll 1
            for (int ph = 0; ph < 4; ++ph) {
              const int pg = 2 * wq + (ph >> 1), hf = ph & 1;
              if (pg >= np) break;  // the lanes of missing pages hold what they held: their logits are masked
              const uint32_t blk = stage + pg * R::kPageStride, sc = blk + F::kKScale + 64 * i + 32 * hf;
              const uint4 sa = lds128_at(sc), sb = lds128_at(sc + 16);
              const uint32_t s[8] = {sa.x, sa.y, sa.z, sa.w, sb.x, sb.y, sb.z, sb.w};
              uint32_t cw[8];
              if (kBits == 4) {
                const uint4 c = lds128_at(blk + F::kKCode + 512 * hf + 16 * lane);
                cw[0] = c.x; cw[1] = c.y; cw[2] = c.z; cw[3] = c.w;
              } else if (kBits == 8) {
                const uint4 c = lds128_at(blk + F::kKCode + 1024 * hf + 16 * lane), d = lds128_at(blk + F::kKCode + 1024 * hf + 512 + 16 * lane);
                cw[0] = c.x; cw[1] = c.y; cw[2] = c.z; cw[3] = c.w;
                cw[4] = d.x; cw[5] = d.y; cw[6] = d.z; cw[7] = d.w;
              } else {
                const uint2 c = lds64_at(blk + F::kKCode + 16 * lane + 8 * hf);
                cw[0] = c.x; cw[1] = c.y;
              }
              uint32_t hi[16], lo[8];
#pragma unroll
              for (int q = 0; q < 4; ++q) {
                uint32_t a[4];
                tile_codes<kBits>(kBits == 8 ? cw[2 * q] : kBits == 4 ? cw[q] : cw[q >> 1], kBits == 8 ? cw[2 * q + 1] : 0, q & 1, a);
                uint32_t rem[4];
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                  const uint32_t c4 = hmul2_u32(a[r], quarter_unit<kBits>()), sr = s[2 * q + (r >> 1)];
                  const uint32_t hr = hmul2_u32(c4, sr);
                  hi[4 * q + r] = hr;
                  rem[r] = h2_as_u32(__hfma2(u32_as_h2(c4), u32_as_h2(sr), __hneg2(u32_as_h2(hr))));  // exact (above fp16's smallest step)
                }
                // an fp16 number's upper byte is its e5m2 truncation (3 significant bits of the remainder)
                lo[2 * q] = __byte_perm(rem[0], rem[2], 0x7531);
                lo[2 * q + 1] = __byte_perm(rem[1], rem[3], 0x7531);
              }
              const uint32_t at = lane_base + (static_cast<uint32_t>(16 * (ph >> 1)) << 16);
              tc05::tmem_st_frag16(tKhi + at + 32 * hf, hi);
              tc05::tmem_st_frag8(tKlo + at + 16 * hf, lo);
            }
          }
          // the stage has been read
          fence_proxy_async();
          __syncwarp();
          if (lane == 0) mbar_arrive(empty(st));
        } else if (!is_help) {
          // tile 0: tokens 0-63 the drafted ones, 64-79 the residual rows
          const int r = w.s.L % kPage;
          const long res_base = (static_cast<long>(w.b) * H + w.h) * kPage * kHeadDim;
          auto rows_of = [&](int grp, const __half *x, const __half *res, int &count, long &stride) -> const __half * {
            if (grp < 4) {
              count = w.s.n - kPage * grp;
              stride = static_cast<long>(H) * kHeadDim;
              return x + (static_cast<long>(w.s.c0 + kPage * grp) * H + w.h) * kHeadDim;
            }
            count = grp == 4 ? r : 0;
            stride = kHeadDim;
            return res + res_base;
          };
          if (is_v) {
            // a drafted value that is not finite must not reach the rows that do not see it, and 0 * infinity would: it
            // is taken as 0 here and added at the end to the rows that do
            bool odd = false;
            auto finite = [&](uint32_t x) {
              const uint32_t e = x & 0x7C007C00u;
              if ((e & 0xFFFFu) == 0x7C00u) x &= 0xFFFF0000u, odd = true;
              if ((e >> 16) == 0x7C00u) x &= 0x0000FFFFu, odd = true;
              return x;
            };
#pragma unroll 1
            for (int pg = 0; pg < kTilePages; ++pg) {
              int count;
              long stride;
              const __half *rv = rows_of(pg, p.v, p.res_v, count, stride) + 32 * wq + 4 * n;
              uint2 x[4];
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const int tk = 2 * i + (e & 1) + 8 * (e >> 1);
                x[e] = tk < count ? *reinterpret_cast<const uint2 *>(rv + tk * stride) : make_uint2(0, 0);
                if (pg < 4) x[e] = make_uint2(finite(x[e].x), finite(x[e].y));
              }
              uint32_t o0[4], o1[4];
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                o0[2 * e] = __byte_perm(x[2 * e].x, x[2 * e + 1].x, 0x5410);
                o0[2 * e + 1] = __byte_perm(x[2 * e].x, x[2 * e + 1].x, 0x7632);
                o1[2 * e] = __byte_perm(x[2 * e].y, x[2 * e + 1].y, 0x5410);
                o1[2 * e + 1] = __byte_perm(x[2 * e].y, x[2 * e + 1].y, 0x7632);
              }
              tc05::tmem_st_frag4(tV + lane_base + 8 * pg, o0);
              tc05::tmem_st_frag4(tV + lane_base + (16u << 16) + 8 * pg, o1);
            }
            odd = __any_sync(kAll, odd);
            if (lane == 0) reinterpret_cast<volatile int *>(sm + kOffOdd)[4 * (uc & 3) + wq] = odd;
          } else {
#pragma unroll 1
            for (int e = 0; e < 2; ++e) {
              int count;
              long stride;
              const __half *rk = rows_of(2 * wq + e, p.k, p.res_k, count, stride) + 32 * i;
              if (count <= 0) break;  // and none in the groups behind it but the residual's, which is no odd one
              uint4 x[4], y[4];
#pragma unroll
              for (int c = 0; c < 4; ++c) {
                x[c] = y[c] = make_uint4(0, 0, 0, 0);
                if (n < count) x[c] = *reinterpret_cast<const uint4 *>(rk + n * stride + 8 * c);
                if (n + 8 < count) y[c] = *reinterpret_cast<const uint4 *>(rk + (n + 8) * stride + 8 * c);
              }
#pragma unroll
              for (int hf = 0; hf < 2; ++hf) {
                uint32_t hi[16];
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                  const uint4 &u = x[2 * hf + c], &v = y[2 * hf + c];
                  const uint32_t us[4] = {u.x, u.y, u.z, u.w}, vs[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                  for (int q = 0; q < 4; ++q) {  // in quarters, as the quantized keys
                    hi[8 * c + 2 * q] = hmul2_u32(us[q], 0x34003400u);
                    hi[8 * c + 2 * q + 1] = hmul2_u32(vs[q], 0x34003400u);
                  }
                }
                tc05::tmem_st_frag16(tKhi + lane_base + (static_cast<uint32_t>(16 * e) << 16) + 32 * hf, hi);
              }
            }
          }
        }
        if (is_help) {
          fence_proxy_async();
        } else {
          tc05::tmem_wait_st();
          tc05::fence_before_sync();
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(is_v ? v_ready(x2) : k_ready(x2));
      }
      ++uc;
      w.next(p);
    }
  } else if (warp == kMmaWarp) {
    // ------------------- S^T(kt) = K Q^T, then O^T += V^T P^T of tile kt - 1
    const uint64_t dhot = tc05::smem_desc_plain32b(base + kOffHot);
    int kt = 0, uc = 0;
    bool fresh = true;  // tile kt - 1 starts a piece
    auto issue_pv = [&](int k1) {
      const int x2 = k1 & 1;
      if (!wait_warp(v_ready(x2), (k1 >> 1) & 1) || !wait_warp(p_full(x2), (k1 >> 1) & 1)) return false;
      tc05::fence_after_sync();
      const uint64_t dp = tc05::smem_desc_mn64(base + kOffP + (2 * x2) * kPBytes, kPBytes);
      const uint32_t tV = tmem + kTmV + 64u * x2;
      if (tc05::elect_one()) {
#pragma unroll
        for (int j = 0; j < 8; ++j)
          tc05::issue_f16_ts(tmem + kTmO, tV + 8 * j, dp + ((2048 * j) >> 4), kIdescTO, (!fresh || j > 0) ? 1u : 0u);
        tc05::issue_commit(p_free(x2));
        tc05::issue_commit(v_free(x2));
      }
      __syncwarp();
      return true;
    };
    while (w.rem > 0 && !failed) {
      const int t1 = w.tile + w.take();
      const uint64_t dq = tc05::smem_desc_sw128(base + kOffQHi + (uc & 1) * kQHiBytes);
      const uint64_t dq8 = tc05::smem_desc_sw128(base + kOffQ8 + (uc & 1) * kQ8Bytes);
      // the last product of the piece before first: its sums wait for it, and nobody yet for this piece's logits
      for (int t = w.tile; t < t1; ++t, ++kt) {
        const int x2 = kt & 1;
        if ((t == w.tile && !wait_warp(q_full(uc & 1), (uc >> 1) & 1)) || !wait_warp(k_ready(x2), (kt >> 1) & 1) ||
            (kt >= 1 && !wait_warp(s_free, (kt - 1) & 1))) {
          fail();
          break;
        }
        tc05::fence_after_sync();
        const uint32_t tS = tmem + kTmS, tKhi = tmem + kTmKhi + 64u * x2, tKlo = tmem + kTmKlo + 32u * x2;
        if (tc05::elect_one()) {
#pragma unroll
          for (int j = 0; j < 8; ++j)
            tc05::issue_f16_ts(tS, tKhi + 8 * j, dq + (((j >> 2) * (kQHiBytes / 2) + (j & 3) * 32) >> 4), kIdescTS, j > 0 ? 1u : 0u);
          if (t > 0) {
#pragma unroll
            for (int j = 0; j < 4; ++j) tc05::issue_e5m2_ts(tS, tKlo + 8 * j, dq8 + ((32 * j) >> 4), kIdescTS8, 1u);
            const uint64_t dzero = tc05::smem_desc_plain32b(base + kOffZero + x2 * (2 * kZeroBytes));
            tc05::issue_tf32_ss(tS, dhot, dzero, kIdescTZ, 1u);
            tc05::issue_tf32_ss(tS, dhot, dzero + (kZeroBytes >> 4), kIdescTZ, 1u);
          }
          tc05::issue_commit(s_full);
          tc05::issue_commit(k_free(x2));
          if (t + 1 == t1) tc05::issue_commit(q_free(uc & 1));
        }
        __syncwarp();
        if (kt > 0 && !issue_pv(kt - 1)) {
          fail();
          break;
        }
        fresh = t == w.tile;
      }
      ++uc;
      w.next(p);
    }
    if (!failed && !issue_pv(kt - 1)) fail();
    // no product may be under way, nor signal a barrier, once the CTA gives its tensor memory back and leaves: after an
    // abort nobody else has waited for the last ones
    if (tc05::elect_one()) tc05::issue_commit(mma_done);
    __syncwarp();
    wait_landed(mma_done, 0);
  } else {
    // ------------------------------------------- softmax and the output
    const int g = (warp - kSoftmaxWarp0) >> 2, wq = warp & 3, tl = 32 * wq + lane;
    const uint32_t lane_base = static_cast<uint32_t>(32 * wq) << 16;
    const uint32_t s_ref = base + kOffRef + 128 * g;
    float *red = reinterpret_cast<float *>(sm + kOffRed) + 128 * g;
    volatile int *last_flag = reinterpret_cast<volatile int *>(sm + kOffFlag) + g;
    const int bid = 1 + g;
    const float sc = 4.0f * p.scale_log2;
    const uint32_t tO = tmem + kTmO + 32u * g + lane_base;
    bool ok = true;  // the group leaves together: a failed wait is told at the next vote
    TreeCut *cuts = reinterpret_cast<TreeCut *>(sm + kOffCut) + 2 * g;
    bool first_piece = true;
    int kt = 0, uc = 0, su = 0, num_cuts = 0, merges = 0;  // (su: pieces with a tile 0)
    while (w.rem > 0 && !failed) {
      const int t0 = w.tile, t1 = w.tile + w.take();
      const int rows = min(kGroupRows, w.s.n * G - kTreeRows * w.rb - kGroupRows * g);  // of this group
      float l[32];
#pragma unroll
      for (int j = 0; j < 32; ++j) l[j] = 0.f;
      float myref = -INFINITY;  // lane j: the reference of row j (every warp of the group holds the same); none yet
      bool without = true;      // a row of the group has none
      if (rows > 0) {
        if (wq == 0) reinterpret_cast<float *>(sm + kOffRef)[32 * g + lane] = 0.f;
        group_sync(bid);
      }
      uint32_t seen = 0;  // tile 0: the rows that see this token
      if (t0 == 0) {
        if (rows > 0 && wq < 2) {
          ok = ok && wait_warp(seen_full(su & 1), (su >> 1) & 1);
          seen = lds32_at(base + kOffSeen + 4 * (64 * (2 * (su & 1) + g) + tl));
        } else if (wq >= 2) {
          seen = tl - 64 < w.s.L % kPage ? 0xFFFFFFFFu : 0u;  // the residual rows
        }
        __syncwarp();
        ++su;
      }
      for (int t = t0; t < t1; ++t, ++kt) {
        const int x2 = kt & 1;
        ok = ok && wait_warp(s_full, kt & 1);
        if (rows <= 0) {  // nothing to do but to keep the barriers' counts
          ok = ok && (kt < 2 || wait_warp(p_free(x2), prev2(kt)));
          if (!ok) *abort_flag = 1;  // the group leaves at its next vote
          if (lane == 0) {
            if (t == 0) mbar_arrive(seen_free((su - 1) & 1));
            mbar_arrive(s_free);
            mbar_arrive(p_full(x2));
          }
          continue;
        }
        tc05::fence_after_sync();
        float sv[32];
        auto load = [&]() {
          tc05::tmem_ld32(tmem + kTmS + 32u * g + lane_base, reinterpret_cast<uint32_t (&)[32]>(sv));
          tc05::tmem_wait_ld();
        };
        // logits in log2 units minus the reference; -inf where this token is not seen
        const uint32_t mask = t == 0 ? seen : (tl / kPage < w.pages(t) ? 0xFFFFFFFFu : 0u);
        const bool masked = __any_sync(kAll, mask != 0xFFFFFFFFu);
        auto shift_as = [&](auto with_mask) {
          float m0 = -INFINITY, m1 = -INFINITY;
#pragma unroll
          for (int j = 0; j < 32; j += 4) {
            const uint4 r = lds128_at(s_ref + 4 * j);
            float2 a = make_float2(sv[j], sv[j + 1]), b = make_float2(sv[j + 2], sv[j + 3]);
            a = fma2(a, make_float2(sc, sc), make_float2(__uint_as_float(r.x), __uint_as_float(r.y)));
            b = fma2(b, make_float2(sc, sc), make_float2(__uint_as_float(r.z), __uint_as_float(r.w)));
            if (with_mask.value) {
              a.x = mask >> j & 1 ? a.x : -INFINITY;
              a.y = mask >> (j + 1) & 1 ? a.y : -INFINITY;
              b.x = mask >> (j + 2) & 1 ? b.x : -INFINITY;
              b.y = mask >> (j + 3) & 1 ? b.y : -INFINITY;
            }
            m0 = fmax3(m0, a.x, a.y);
            m1 = fmax3(m1, b.x, b.y);
            sv[j] = a.x;
            sv[j + 1] = a.y;
            sv[j + 2] = b.x;
            sv[j + 3] = b.y;
          }
          return fmaxf(m0, m1);
        };
        auto shift = [&]() { return masked ? shift_as(std::true_type()) : shift_as(std::false_type()); };
        load();
        const float top = shift();
        if (group_any(bid, top > kRefSlack || without || !ok)) {
          if (group_any(bid, !ok)) {
            fail();
            break;
          }
          // move references: lane j finds the tile's maximum of row j
          red[32 * wq + lane] = warp_reduce_rows(sv, lane, [](float a, float b) { return fmaxf(a, b); });
          group_sync(bid);
          const float up = fmaxf(fmaxf(red[lane], red[32 + lane]), fmaxf(red[64 + lane], red[96 + lane]));
          const bool none = myref == -INFINITY;  // the sums so far are 0 (or NaN)
          const float by = none || up > kRefSlack ? up : 0.f;
          const float f = none ? 1.0f : fast_exp2(-by);
          myref = none ? by : myref + by;
          without = __any_sync(kAll, myref == -INFINITY && lane < rows);
          if (wq == 0) reinterpret_cast<float *>(sm + kOffRef)[32 * g + lane] = myref == -INFINITY ? 0.f : -myref;
          group_sync(bid);
          if (t > t0) {
            // the sums so far, and O once every product before this tile's is in it
            ok = ok && wait_warp(p_free(x2 ^ 1), ((kt - 1) >> 1) & 1);
            tc05::fence_after_sync();
#pragma unroll
            for (int j = 0; j < 32; ++j) l[j] *= __shfl_sync(kAll, f, j);
#pragma unroll 1
            for (int part = 0; part < 2; ++part) {
              uint32_t o[32];
              tc05::tmem_ld32(tO + kTreeRows * part, o);
              tc05::tmem_wait_ld();
#pragma unroll
              for (int j = 0; j < 32; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * __shfl_sync(kAll, f, j));
              tc05::tmem_st32(tO + kTreeRows * part, o);
            }
            tc05::tmem_wait_st();
          }
          load();
          shift();
        }
        // S has been read
        tc05::fence_before_sync();
        __syncwarp();
        if (lane == 0) {
          if (t == 0) mbar_arrive(seen_free((su - 1) & 1));
          mbar_arrive(s_free);
        }
        ok = ok && (kt < 2 || wait_warp(p_free(x2), prev2(kt)));
        const uint32_t ph = base + kOffP + (2 * x2) * kPBytes + (tl >> 3) * 1024 + (tl & 7) * 128;
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          uint32_t hi[4], lo[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int j = 8 * c + 2 * e;
            const float2 x = make_float2(fast_exp2(sv[j]), fast_exp2(sv[j + 1]));
            const float2 ls = add2(make_float2(l[j], l[j + 1]), x);
            l[j] = ls.x;
            l[j + 1] = ls.y;
            const __half2 hh = __floats2half2_rn(x.x, x.y);
            const float2 d = sub2(x, __half22float2(hh));
            hi[e] = h2_as_u32(hh);
            lo[e] = h2_as_u32(__floats2half2_rn(d.x, d.y));
          }
          const uint32_t at = ph + (((4 * g + c) ^ (tl & 7)) << 4);
          sts128(at, make_uint4(hi[0], hi[1], hi[2], hi[3]));
          sts128(at + kPBytes, make_uint4(lo[0], lo[1], lo[2], lo[3]));
        }
        fence_proxy_async();
        __syncwarp();
        if (lane == 0) mbar_arrive(p_full(x2));
      }
      if (failed) break;

      // ---- the piece's end: sums over the tokens (lane j: row j), O once its last product is in it
      if (rows > 0) {
        red[32 * wq + lane] = warp_reduce_rows(l, lane, [](float a, float b) { return a + b; });
        ok = ok && wait_warp(p_free((kt - 1) & 1), ((kt - 1) >> 1) & 1);
        if (group_any(bid, !ok)) {
          fail();
          break;
        }
        const float lsum = red[lane] + red[32 + lane] + red[64 + lane] + red[96 + lane];
        tc05::fence_after_sync();
        const int row0 = kTreeRows * w.rb + kGroupRows * g;
        const int ch = 32 * wq + 4 * (lane & 7) + 2 * (lane >> 4) + (lane >> 3 & 1);
        // drafted values that are not finite, to the rows that see them: +infinity in `more`, -infinity in `less`, NaN in both
        uint32_t more = 0, less = 0;
        if (t0 == 0 && *(reinterpret_cast<volatile int *>(sm + kOffOdd) + 4 * (uc & 3) + wq)) {
#pragma unroll 1
          for (int j = 0; j < rows; ++j)
            for (int a = (row0 + j) / G; a >= 0;) {
              const float x = __half2float(p.v[(static_cast<long>(w.s.c0 + a) * H + w.h) * kHeadDim + ch]);
              if (!(x <= FLT_MAX)) more |= 1u << j;
              if (!(x >= -FLT_MAX)) less |= 1u << j;
              const int up = __ldg(p.parents + w.s.c0 + a);
              a = up < a ? up : -1;
            }
        }
        // 8 rows at a time (the loop is short: a unit's end is run once in a while, and would be fetched each time)
        const bool whole = t0 == 0 && t1 == w.s.tiles;
        const long long slot = 2ll * blockIdx.x + (first_piece ? 0 : 1);
        const float factor = 1.0f / lsum;
        int head = row0 % G;
        __half *dst = p.out + (static_cast<long>(w.s.c0 + row0 / G) * p.num_q_heads + w.h * G + head) * kHeadDim + ch;
        float *part = p.part + (slot * kTreeRows + kGroupRows * g) * kHeadDim + ch;
#pragma unroll 1
        for (int c = 0; c < rows; c += 8) {
          float o[8], lo[8];
          tc05::tmem_ld8(tO + c, o);
          tc05::tmem_ld8(tO + kTreeRows + c, lo);
          tc05::tmem_wait_ld();
#pragma unroll
          for (int j = 0; j < 8; ++j) o[j] += lo[j];
          if (__any_sync(kAll, (more | less) != 0)) {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              if (more >> (c + j) & 1) o[j] += INFINITY;
              if (less >> (c + j) & 1) o[j] -= INFINITY;
            }
          }
          if (whole) {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              const __half x = __float2half_rn(o[j] * __shfl_sync(kAll, factor, c + j));
              if (c + j < rows) *dst = x;
              dst += kHeadDim;
              if (++head == G) {
                head = 0;
                dst += static_cast<long>(p.num_q_heads - G) * kHeadDim;
              }
            }
          } else {
#pragma unroll
            for (int j = 0; j < 8; ++j)
              if (c + j < rows) part[(c + j) * kHeadDim] = o[j];
          }
        }
        if (!whole) {
          if (wq == 0) p.part_ml[slot * kTreeRows + kGroupRows * g + lane] = make_float2(myref, lsum);
          __threadfence();
          group_sync(bid);
          if (wq == 0 && lane == 0) {
            const TreeSplit split = *reinterpret_cast<const TreeSplit *>(sm + kOffSplit);
            TreeCut c;
            c.out = (static_cast<long long>(w.s.c0) * p.num_q_heads + w.h * G) * kHeadDim;
            c.first = split.each ? split.cta_of(w.start) : split.first;
            c.last = split.each ? split.cta_of(w.start + w.s.tiles - 1) : split.last;
            c.odd = split.each && split.begin(c.first) < w.start - kUnitTiles;
            c.row0 = row0;
            c.rows = rows;
            c.ticket = ((w.b * H + w.h) * ((p.max_nodes * G + kTreeRows - 1) / kTreeRows) + w.rb) * 2 + g;
            cuts[num_cuts] = c;
            atomicAdd(p.tickets + c.ticket, 1u);
          }
          ++num_cuts;
        }
      }
      first_piece = false;
      ++uc;
      w.next(p);
    }

    // ---- units that are cut between CTAs: each of a unit's CTAs merges its share of the rows once all pieces are
    // there (all CTAs are resident, and each has told of its pieces before it waits here)
    // (a group without rows in the last unit has not waited for that unit's last product, which reads both groups' weights)
    ok = ok && wait_warp(p_free((kt - 1) & 1), ((kt - 1) >> 1) & 1);
    if (!failed && group_any(bid, !ok)) fail();
    for (int x = 0; x < num_cuts && !failed; ++x) {
      const TreeCut c = cuts[x];
      const int pieces = c.last - c.first + 1, mine = static_cast<int>(blockIdx.x) - c.first;
      uint32_t *ticket = p.tickets + c.ticket;
      if (wq == 0 && lane == 0) {
        const long long begun = clock64();
        uint32_t there;
        while (true) {
          asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(there) : "l"(ticket) : "memory");
          if (static_cast<int>(there & 0xFFFFu) >= pieces || clock64() - begun > kAbortWaitCycles) break;
          __nanosleep(100);  // the counter's line is everybody's
        }
        *last_flag = static_cast<int>(there & 0xFFFFu) >= pieces;
      }
      group_sync(bid);
      if (!*last_flag) {
        fail();
        break;
      }
      __threadfence();
      const int ch = 32 * wq + 4 * (lane & 7) + 2 * (lane >> 4) + (lane >> 3 & 1);
      auto slot_of = [&](int k) { return (2ll * (c.first + k) + (k == 0 ? c.odd : 0)) * kTreeRows + kGroupRows * g; };
      // its items, (row, piece) pairs with the pieces of a row in their order, come by bulk copies, 64 at a time into the
      // 32 KB where the weights were: one wait for other SMs' writes, whether they are few rows of many pieces or many of few
      const int lo = c.rows * mine / pieces, items = (c.rows * (mine + 1) / pieces - lo) * pieces;
      const uint32_t s_items = base + kOffP + 2 * g * kPBytes;
      float *ml = reinterpret_cast<float *>(sm + kOffQ8 + g * kQ8Bytes);  // [items], fewer than 32 + pieces of them
      const float *vals = reinterpret_cast<const float *>(sm + kOffP + 2 * g * kPBytes);
      auto fetch = [&](int y0) {
        const int count = min(64, items - y0);
        if (wq == 0 && count > 0) {
          asm volatile("fence.proxy.async;" ::: "memory");  // plain stores (other SMs' to the pieces, this one's to the weights) before the copies
          if (lane == 0) mbar_arrive_expect_tx(merged(g), count * kHeadDim * 4);
          __syncwarp();
          for (int y = lane; y < count; y += 32)
            bulk_copy_g2s(s_items + y * kHeadDim * 4, p.part + (slot_of((y0 + y) % pieces) + lo + (y0 + y) / pieces) * kHeadDim,
                          kHeadDim * 4, merged(g));
        }
      };
      fetch(0);
      // ml[row][piece] = the piece's weight: many rows of few pieces a thread each, few rows of many pieces a warp each
      if (pieces <= 4) {
        if (tl * pieces < items) {
          float2 x[4];
          float top = -INFINITY, sum = 0.f;
#pragma unroll
          for (int k = 0; k < 4; ++k)
            x[k] = k < pieces ? __ldcg(p.part_ml + slot_of(k) + lo + tl) : make_float2(-INFINITY, 0.f);
#pragma unroll
          for (int k = 0; k < 4; ++k) top = fmaxf(top, x[k].x);
#pragma unroll
          for (int k = 0; k < 4; ++k) sum += (x[k].x = fast_exp2(x[k].x - top)) * x[k].y;
#pragma unroll
          for (int k = 0; k < 4; ++k)
            if (k < pieces) ml[tl * pieces + k] = x[k].x / sum;
        }
      } else for (int r = wq; r * pieces < items; r += 4) {
        float M = -INFINITY, sum = 0.f;
        for (int y = lane; y < pieces; y += 32) {
          const float2 x = __ldcg(p.part_ml + slot_of(y) + lo + r);
          const float top = fmaxf(M, x.x), at = top == -INFINITY ? 0.f : top;  // (a piece without weight has no reference)
          sum = sum * fast_exp2(M - at) + x.y * fast_exp2(x.x - at);
          M = top;
          ml[r * pieces + y] = x.x;
        }
        float top = M;
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) top = fmaxf(top, __shfl_xor_sync(kAll, top, off));
        sum = lane < pieces ? sum * fast_exp2(M - top) : 0.f;
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) sum += __shfl_xor_sync(kAll, sum, off);
        for (int y = lane; y < pieces; y += 32) ml[r * pieces + y] = fast_exp2(ml[r * pieces + y] - top) / sum;
      }
      group_sync(bid);
      int k = 0, row = c.row0 + lo;
      float acc = 0.f;
      for (int y0 = 0; y0 < items; y0 += 64) {
        ok = ok && wait_warp(merged(g), merges & 1);
        const int count = ok ? min(64, items - y0) : 0;
#pragma unroll 4
        for (int y = 0; y < count; ++y) {
          acc += ml[y0 + y] * vals[y * kHeadDim + ch];
          if (++k == pieces) {
            const int node = row / G;
            p.out[c.out + (static_cast<long long>(node) * p.num_q_heads + (row - node * G)) * kHeadDim + ch] = __float2half_rn(acc);
            acc = 0.f;
            k = 0;
            ++row;
          }
        }
        if (group_any(bid, !ok)) {
          // the items on their way must have landed before the CTA leaves, and no more are sent for
          wait_landed(merged(g), merges & 1);
          fail();
          break;
        }
        ++merges;
        fetch(y0 + 64);  // the items have been read
      }
      if (failed) break;
      group_sync(bid);
      // the last of them leaves the counter at zero
      if (wq == 0 && lane == 0 && (atomicAdd(ticket, 0x10000u) >> 16) + 1 == static_cast<uint32_t>(pieces)) *ticket = 0u;
    }
  }

  if (failed) flag_error(p.err, S4KV_EFLAG_TIMEOUT);
  tc05::fence_before_sync();
  __syncthreads();
  if (warp == kMmaWarp) {
    tc05::fence_after_sync();
    tc05::tmem_dealloc(tmem, 512);
  }
}

template <int kBits>
static cudaError_t launch_tree_for(const TreeParams &p, cudaStream_t stream) {
  const cudaError_t e = cudaFuncSetAttribute(tree_kernel<kBits>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             static_cast<int>(Ring<kBits>::kSmem));
  if (e != cudaSuccess) return e;
  // a cooperative launch: CTAs that share a unit wait for one another at its end
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeCooperative;
  attr[0].val.cooperative = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(p.num_ctas));
  cfg.blockDim = dim3(kTreeThreads);
  cfg.dynamicSmemBytes = Ring<kBits>::kSmem;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, tree_kernel<kBits>, p);
}

cudaError_t launch_tree(const TreeParams &p, cudaStream_t stream) {
  return p.bits == 8 ? launch_tree_for<8>(p, stream) : p.bits == 2 ? launch_tree_for<2>(p, stream) : launch_tree_for<4>(p, stream);
}

}  // namespace s4kv
