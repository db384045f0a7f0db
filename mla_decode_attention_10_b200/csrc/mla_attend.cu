// mla_attend.cu -- decode attention over the paged latent cache with shared
// prefixes, on the tcgen05 tensor cores (contract in mla_epilogue.h).
//
//   s = scale * q . key (576 terms),  p = exp(s - m),  out = (sum_k p key[0:512]) / (sum_k p)
//
// Work.  A unit is a prefix group (all rows (token, head) of the group against
// the prefix's keys) or a token (its H rows against its own keys).  A unit's
// rows are taken 64 at a time (row tile) and its keys 64 at a time (key tile).
// All (unit, row tile, key tile) triples, in this order, are dealt out to one
// CTA per SM in contiguous runs of equal cost, whatever the lengths are; lengths
// stay in device memory (each CTA adds them up itself).  A CTA's piece of one row
// tile is a segment; it ends with the segment's unnormalised sum, maximum and
// denominator in the workspace, and a second kernel joins a row's segments.
//
// Tensor cores.  A CTA holds 64 rows because TMEM holds their fp32 sums, 64 x 512,
// in half of its 512 columns (128 rows would fill it and leave no room for the
// scores).  M = 64 in the weight-stationary form (.ws) spreads a row over two TMEM
// lanes (columns 0 .. N/2-1 on lanes 0..63, the rest on lanes 64..127).  Measured
// on B200: N = 256 in 80 cycles, against 128 for the plain M = 64 form; N = 64 in
// 32, or in 28 with the q rows in TMEM.  S = Q K^T is 36 such products a key tile
// (N = 64, K = 16), O += P V is 8 (N = 256; V is the K tile itself, read with the
// key index as the contraction): 1697 cycles in all.  With e4m3 q and cache the
// codes are multiplied as they are (kind::f8f6f4, K = 32): 18 + 12 products (the
// weights are three e5m2 terms), 1493 cycles.
//
// Warps (16, one CTA an SM):
//   softmax (8, or 4 where rows are decoded): scores from TMEM, running maximum
//          and sum, weights to shared memory, the sums' rescaling (only when a
//          row's maximum has grown by more than a margin since the last time), the
//          segment's result;
//   scores, sums (1 each): issue the products.  The queue of issued products is
//          short: what one warp waits for between two products is lost time unless
//          the other has some under way (one warp for both: 538 us instead of 492
//          for 256 tokens over 32 K keys, all else the same);
//   finder (1): looks up the CTA's segments for all the others;
//   loaders (4, or 8 where rows are decoded) fill a ring of tile halves:
//     - whole tiles of rows kept as they are (bf16; e4m3 with e4m3 q): tensor
//       copies of 128 bytes x 8 to 64 rows, or of half a tile where a page has 64
//       rows; one loader warp a tile, in turn;
//     - tiles with a ragged end, or pages that tensor copies cannot follow:
//       16-byte asynchronous copies, zeros where there is no key;
//     - rows to be decoded: loads, integer arithmetic, stores;
//     - prefixes of many rows that need decoding (or odd pages): decoded once by a
//       kernel before this one, into images of tiles as they lie in shared memory,
//       which come by two or three bulk copies.
// S of tile i+1 is issued before O of tile i, so the softmax of i overlaps it.
// Every wait is bounded: on timeout a status bit is set, all roles stop, TMEM
// is freed and the kernel returns.  Each CTA leaves word of it in the workspace,
// and rows that it had a part in come out as NaN.
//
// What bounds it (cycles of a key tile, in the kernel): images and bf16 prefixes
// 2070 to 2120, of which the products take 1697: the tile's way through the ring
// (copy 1300, scores 1000, softmax 1300, sums 700) is longer than 2.5 tiles'
// products; codes 1750 to 1850 of 1493, the softmax (one tile at a time, 900 for the
// weights' three terms and 900 for the rest of the way round); a CTA's first bf16
// tiles from HBM 2800.  Rows decoded by the loaders take 5100 (e4m3) to 6000 (mx):
// the loads' latency (1200), which an arrival on a barrier does not let overlap the
// stores of the tile before, then twice 1500 for a half's arithmetic and stores.

#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_runtime.h>

#include <atomic>
#include <climits>
#include <cmath>
#include <cstdint>

#include "latent_math.cuh"
#include "latent_rows.cuh"
#include "mla_epilogue.h"
#include "mla_harness.h"
#include "mla_runtime.h"

namespace mla {
namespace attend {

constexpr int kRowsTile = 64;   // rows of a CTA (MMA M)
constexpr int kKeys = 64;       // keys of a tile
constexpr int kDv = 512;        // values
constexpr uint32_t kSlabBytes = 64 * 128;  // one 128-byte column slab of 64 rows, 128-byte swizzle

// Operand forms.  kBf16: q and keys as bf16, weights as bf16.  kF8: q and keys as
// the e4m3 codes they are stored in, weights as three e5m2 terms (hi + mid + lo:
// each takes three of the weight's bits, nine in all against bf16's eight).
enum Op { kBf16 = 0, kF8 = 1 };

// A key tile is 128-byte slabs of its rows: the 512 values, then the rotary slab
// (in kF8 half full).  In shared memory it lies in two halves of a ring of
// halves, which are filled, used and freed one by one, and its rotary slab, which
// comes with the first half, in a slot of its own.  A segment's q rows pass
// through the ring like a tile, on their way to TMEM; what has no room there
// (bf16: the last two value slabs and the rotary slab) stays in shared memory.
// Freed of the q rows, shared memory holds 2.5 tiles instead of 2, or in kF8 4.5
// instead of 3.
template <int OP>
struct Shape {
  static constexpr int kElem = OP == kF8 ? 1 : 2;
  static constexpr int kHalfSlabs = OP == kF8 ? 2 : 4;
  static constexpr int kPeSlab = 2 * kHalfSlabs;
  static constexpr int kPeSteps = OP == kF8 ? 2 : 4;        // MMAs over the rotary slab, 32 bytes of a row each
  static constexpr int kQSlab0 = OP == kF8 ? kPeSlab + 1 : 6;  // q slabs from here on stay in shared memory
  static constexpr int kQSlabs = kPeSlab + 1 - kQSlab0;
  static constexpr int kTerms = OP == kF8 ? 3 : 1;          // weights
  static constexpr int kKeySteps = OP == kF8 ? 2 : 4;       // MMAs over a tile's keys, 32 or 16 keys each
  static constexpr uint32_t kHalf = kHalfSlabs * kSlabBytes;
  static constexpr int kHalves = OP == kF8 ? 9 : 5;
  // A tile's first half follows, in its place, the second half of the tile kSlots
  // before: that tile's rotary slab and flags have been used by then.
  static constexpr int kSlots = (kHalves + 1) / 2;
  static constexpr uint32_t kP = OP == kF8 ? 2 * kSlabBytes : kSlabBytes;
  static constexpr int kPBufs = OP == kF8 ? 2 : 1;
  static constexpr uint32_t kPeAt = kHalves * kHalf;
  static constexpr uint32_t kQAt = kPeAt + kSlots * kSlabBytes;
  static constexpr uint32_t kPAt = kQAt + kQSlabs * kSlabBytes;
  static constexpr uint32_t kSmem = kPAt + kP * kPBufs + 1024;
  static constexpr uint32_t kTile = (kPeSlab + 1) * kSlabBytes;
  static constexpr uint32_t kImage = kTile + 128;           // a tile as it lies in shared memory, then its 64 flags
};
constexpr int kMaxHalves = 9, kMaxSlots = 5;

// A role's place in the ring: the half it is at, how often it has been round, and
// the tile's rotary slot.
template <int OP>
struct Ring {
  uint32_t half = 0, lap = 0, slot = 0;
  __device__ __forceinline__ void next_half() {
    if (++half == Shape<OP>::kHalves) {
      half = 0;
      ++lap;
    }
  }
  __device__ __forceinline__ void next_tile() {  // both halves passed
    if (++slot == Shape<OP>::kSlots) slot = 0;
  }
  __device__ __forceinline__ void skip_tile() {
    next_half();
    next_half();
    next_tile();
  }
};

// Roles.  Rows that need no decoding are copied, which four warps issue easily,
// and leave eight warps for the softmax (130 us with four, 115 with eight for 590 K
// e4m3 keys, at the time); decoding rows takes eight warps.
template <int FMT, int OP>
struct Roles {
  static constexpr bool kDecode = OP == kBf16 && FMT != MLA_CACHE_BF16;
  static constexpr int kSoft = kDecode ? 4 : 8;
  static constexpr int kLoad0 = kSoft;
  static constexpr int kLoad = kDecode ? 8 : 4;
  static constexpr int kScores = 12;          // the warp that issues the scores' products
  static constexpr int kSums = 13;            // and the sums'
  static constexpr int kFinds = 14;           // and the one that finds the segments
  static constexpr int kTakers = 14;          // warps that take them up
  static constexpr int kLoadRegs = kDecode ? 152 : 176;     // with kIssueRegs and the softmax's 128: 512 for four times four warps
  static constexpr int kRows = kRowsTile / kLoad;           // rows of a loader warp
};
// Sixteen warps (one without work) of 128 registers; the last four hand on to the loaders
// what issuing products does not need.
constexpr int kThreads = 32 * 16;
constexpr int kIssueRegs = 80;
constexpr uint32_t kArrivals = 33;     // a loader warp's on a half's barrier: its own and its threads' copies'

constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kTmemS = 256;       // score buffers: columns 256 + 32 b
constexpr uint32_t kTmemQ = 320;       // q rows: 32 bytes of each in 8 columns
constexpr uint32_t kWaitSpins = 1u << 22;  // tries of a wait
constexpr uint32_t kFindTimes = 16;        // that many more for the next segment, behind millions of tokens without keys
constexpr uint32_t kLandSpins = 1u << 14;  // for copies under way to land
constexpr float kRescale = 8.0f;       // the reference maximum moves when a score passes it by 2^8
constexpr int kChunks = kDv / 4;       // 16-byte pieces of a row's fp32 sums
// What the deal counts (measured cycles, in hundreds): a key tile, by how it comes,
// and a segment's start and end, by its rows (their sums are written out).
constexpr int kCostPrefix = 21, kCostRows = 28, kCostE4m3 = 51, kCostMx = 60, kCostF8 = 18, kCostSegment = 25, kCostRow = 1;

struct Params {
  const uint8_t* q;
  int64_t q_st, q_sh;  // bytes
  const float* q_scale;
  const uint8_t* cache;
  const float* kv_scale;
  int64_t cache_blocks;
  int32_t block_size;
  const int32_t* prefix_table;
  int64_t prefix_stride, prefix_keys;
  const int32_t* prefix_lens;
  const int32_t* group_offsets;
  const int32_t* block_table;
  int64_t table_stride, table_keys;
  const int32_t* seq_lens;
  int32_t T, H, G;
  int32_t q_fp8;
  float sm_scale;
  uint16_t* out;
  float* lse;
  int64_t* plan;      // [0] each CTA's run, [1 + u] where unit u starts
  uint32_t* gave_up;  // by CTA: 1 if one of its waits ran out, and its segments are not to be trusted
  uint8_t* image;     // decoded prefix tiles, or null: prefixes are read from the cache
  int64_t image_tiles;  // tiles of one group's image
  uint8_t* prefix_part;
  uint8_t* own_part;
  int32_t own_rows;   // rows of an own segment: min(H, 64)
  int32_t ctas;       // CTAs of the attention kernel
  int32_t image_bytes;  // of one tile's image
  int32_t box_rows;     // cache rows of one tensor copy (8, 16, 32 or 64), or 0: none are made
  int32_t tile_cost, prefix_cost;  // of a tile of own keys, of a prefix
  uint32_t spins;     // tries of a wait: kWaitSpins, or fewer in tests
  int32_t* status;
};

// kF8 weights are 2^lift times p, at most 2^15: e5m2 reaches 57344, and down to
// 2^-16, so each is off by up to 2^-17 / 2^lift of the largest.  All of n keys
// that is n times as much, and the denominator does not share it: the lift is the
// one at which it stays below 2^-11, 7 up to 2^13 keys and one more for each
// doubling, up to 13 (2^19 keys).  The reference may lag behind a row's maximum by
// what is left of 15.  (Not 13 for all: 590 K e4m3 keys, 4 K a CTA, take 98 us with
// 7 and 8 left, 101 with 12 and 3, 103 with 13 and 2.)
constexpr float kF8Top = 15.0f;
// A score's scale and its difference to the reference are one rounding, but the
// reference has been rounded too, by half a unit: that far the largest weight may
// be from 1.  Where the unit passes 1, kF8 weights go without lift and margin; where
// it would lead out of a weight's type, weights are zero while the maximum is there,
// and a row whose maximum stays there is NaN: by its infinite reference, or, of low
// scores, because it has a maximum but no denominator.
constexpr float kF8Large = 4194304.0f;                       // 2^22
constexpr float kF8Most = 268435456.0f;                       // 2^28: off by 2^8 at most
constexpr float kMost = 2147483648.0f;                       // 2^31: by 2^64
__device__ __forceinline__ float f8_lift(int tiles) {
  return fminf(static_cast<float>(7 + 32 - __clz(max(tiles - 1, 0) >> 7)), 13.0f);
}

// ---- a segment's result: fp32 sums as [chunk of 4 columns][row] 16-byte
// pieces (neighbouring rows, on neighbouring lanes, are contiguous), then the
// rows' maxima (in powers of two) and denominators; whole 128-byte lines
__host__ __device__ constexpr int64_t part_bytes(int rows) {
  return (static_cast<int64_t>(rows) * (kChunks * 16 + 8) + 127) / 128 * 128;
}

__device__ __forceinline__ uint32_t smem_u32(const void* p) { return static_cast<uint32_t>(__cvta_generic_to_shared(p)); }

__device__ __forceinline__ void report(int32_t* status, int32_t bit) {
  if (status != nullptr) atomicOr(status, bit);
}

__device__ __forceinline__ void pdl_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void pdl_trigger() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

__device__ __forceinline__ int uniform(int v) { return __shfl_sync(0xffffffffu, v, 0); }

// a / b; 64-bit divisions are slow
__device__ __forceinline__ int64_t quotient(int64_t a, int64_t b) {
  if (((a | b) >> 32) == 0) return static_cast<uint32_t>(a) / static_cast<uint32_t>(b);
  return a / b;
}

// ---- units ---------------------------------------------------------------------

struct Unit {
  int64_t rows0;  // first (token, head) row
  int64_t rows;
  int64_t len;    // keys
  const int32_t* table;
  const uint8_t* image;  // its decoded tiles, or null
  bool prefix;
  int64_t part0;  // number of the first row tile, within the unit's kind

  __device__ __forceinline__ int64_t row_tiles() const { return (rows + kRowsTile - 1) / kRowsTile; }
  __device__ __forceinline__ int64_t key_tiles() const { return (len + kKeys - 1) / kKeys; }
  int32_t tile_cost, start_cost;
  // what one row tile counts for in the deal: its start, then its key tiles
  __device__ __forceinline__ int64_t row_cost() const { return len > 0 ? key_tiles() * tile_cost + start_cost : 0; }
  // the first key tile that starts at or behind position x of the row tile
  __device__ __forceinline__ int64_t tile_at(int64_t x) const {
    return x > start_cost ? quotient(x - start_cost + tile_cost - 1, tile_cost) : 0;
  }
  __device__ __forceinline__ int64_t cost() const { return row_tiles() * row_cost(); }
};

__device__ __forceinline__ int64_t cut(int64_t v, int64_t lo, int64_t hi) { return v < lo ? lo : v > hi ? hi : v; }

// Tokens [lo, hi) of group g.
__device__ __forceinline__ void group_tokens(const Params& p, int64_t g, int64_t& lo, int64_t& hi, bool& bad) {
  if (p.group_offsets == nullptr) {
    lo = 0;
    hi = p.T;
    bad = false;
    return;
  }
  const int64_t a = __ldcg(p.group_offsets + g), b = __ldcg(p.group_offsets + g + 1);
  lo = cut(a, 0, p.T);
  hi = cut(b, lo, p.T);
  bad = lo != a || hi != b;
}

// A token's own keys, given their number.
__device__ __forceinline__ Unit token_unit(const Params& p, int64_t t, int64_t len, bool& bad) {
  Unit x;
  x.rows0 = t * p.H;
  x.rows = p.H;
  x.table = p.block_table + t * p.table_stride;
  x.image = nullptr;
  x.prefix = false;
  x.part0 = t * ((p.H + kRowsTile - 1) / kRowsTile);
  bad = len > p.table_keys;
  x.len = cut(len, 0, p.table_keys);
  x.tile_cost = p.tile_cost;
  x.start_cost = kCostSegment + kCostRow * p.own_rows;
  return x;
}

// Unit u: group u for u < G, else token u - G.  `bad`: something had to be cut.
// Row tiles are numbered from rows0 / 64 + g on for a group: floor(x) + 1 >=
// ceil(x), so the numbers of consecutive groups do not meet.
__device__ __forceinline__ Unit unit_at(const Params& p, int64_t u, bool& bad) {
  if (u >= p.G) return token_unit(p, u - p.G, p.table_keys > 0 ? __ldcg(p.seq_lens + (u - p.G)) : 0, bad);
  Unit x;
  int64_t lo, hi;
  group_tokens(p, u, lo, hi, bad);
  const int64_t len = __ldcg(p.prefix_lens + u);
  x.rows0 = lo * p.H;
  x.rows = (hi - lo) * p.H;
  x.table = p.prefix_table + u * p.prefix_stride;
  x.image = p.image != nullptr ? p.image + u * p.image_tiles * p.image_bytes : nullptr;
  x.prefix = true;
  x.part0 = x.rows0 / kRowsTile + u;
  bad = bad || len > p.prefix_keys;
  x.len = cut(len, 0, p.prefix_keys);
  x.tile_cost = p.prefix_cost;
  x.start_cost = kCostSegment + kCostRow * kRowsTile;
  return x;
}

// One segment: rows [row0, row0 + rows) against key tiles [k0, k1) of `len` keys.
struct Segment {
  const int32_t* table;
  const uint8_t* image;
  uint8_t* part;
  int32_t row0, rows;
  int32_t k0, k1;  // equal: there are no more segments
  int32_t len;
  int32_t part_rows;
};

// A place in the CTA's run.
struct Cursor {
  int64_t pos, end;  // this CTA's run
  int64_t base, u;   // where unit u starts
  const Unit* known;  // unit u, if it has been looked up already
  int64_t window;    // lane i knows the number of keys of token `window` + i
  int32_t window_len;
};

// The next segment, by a whole warp.
__device__ __forceinline__ bool next_segment(const Params& p, Cursor& c, Segment& s) {
  while (c.pos < c.end) {
    bool bad;
    Unit x;
    if (c.known != nullptr) {
      x = *c.known;
    } else if (c.u < p.G) {
      x = unit_at(p, c.u, bad);
    } else {
      int64_t t = c.u - p.G;
      if (t >= p.T) return false;  // (only if lengths change under the call)
      if (t - c.window >= 32) {
        const int64_t mine = t + (threadIdx.x & 31u);
        c.window = t;
        c.window_len = p.table_keys > 0 && mine < p.T ? __ldcg(p.seq_lens + mine) : 0;
      }
      // to the next token that has keys of its own: the others count for nothing
      const uint32_t some = __ballot_sync(0xffffffffu, c.window_len > 0) >> static_cast<int>(t - c.window);
      if (some == 0u) {
        c.u = p.G + c.window + 32;
        continue;
      }
      t += __ffs(static_cast<int>(some)) - 1;
      c.u = p.G + t;
      x = token_unit(p, t, __shfl_sync(0xffffffffu, c.window_len, static_cast<int>(t - c.window)), bad);
    }
    const int64_t per = x.row_cost(), n = x.row_tiles() * per;
    if (c.pos >= c.base + n) {
      c.base += n;
      c.known = nullptr;
      uint32_t u = static_cast<uint32_t>(c.u) + 1u;
      const uint32_t groups = static_cast<uint32_t>(p.G);
      if (n == 0 && u < groups) {  // past groups without keys or tokens, 32 at a time (so there are offsets)
        const uint32_t mine = u + (threadIdx.x & 31u);
        bool works = true;
        if (mine < groups)
          works = __ldcg(p.prefix_lens + mine) > 0 && __ldcg(p.group_offsets + mine) < __ldcg(p.group_offsets + mine + 1);
        const uint32_t some = __ballot_sync(0xffffffffu, works);
        u += some != 0u ? static_cast<uint32_t>(__ffs(static_cast<int>(some)) - 1) : 32u;
      }
      c.u = u;
      continue;
    }
    const int64_t off = c.pos - c.base, r = off < per ? 0 : quotient(off, per), from = off - r * per;
    const int64_t to = per - from < c.end - c.pos ? per : from + (c.end - c.pos);
    c.pos += to - from;
    // the key tiles that start in this run
    const int64_t k = x.tile_at(from), k_end = to < per ? x.tile_at(to) : x.key_tiles();
    if (k >= k_end) continue;
    s.row0 = static_cast<int32_t>(x.rows0 + r * kRowsTile);
    s.rows = static_cast<int32_t>(x.rows - r * kRowsTile < kRowsTile ? x.rows - r * kRowsTile : kRowsTile);
    s.k0 = static_cast<int32_t>(k);
    s.k1 = static_cast<int32_t>(k_end);
    s.len = static_cast<int32_t>(x.len);
    s.table = x.table;
    s.image = x.image;
    s.part_rows = x.prefix ? kRowsTile : p.own_rows;
    // segments ascend in (CTA, row tile), so CTA + row tile numbers each one
    s.part = (x.prefix ? p.prefix_part : p.own_part) +
             (static_cast<int64_t>(blockIdx.x) + x.part0 + r) * part_bytes(s.part_rows);
    return true;
  }
  return false;
}

// ---- tensor cores and barriers -----------------------------------------------------

// Shared-memory matrix descriptor, 128-byte swizzle.  K-major operand (rows
// of 64 values): 8-row groups `sbo` = 1024 bytes apart, lbo unused.  MN-major
// operand (V: rows are keys): 64-column slabs `lbo` bytes apart, 8-key groups
// `sbo` = 1024 bytes apart.
__device__ __forceinline__ uint64_t smem_desc(uint32_t addr, uint32_t lbo, uint32_t sbo) {
  return static_cast<uint64_t>((addr >> 4) & 0x3fffu) | (static_cast<uint64_t>(lbo >> 4) << 16) |
         (static_cast<uint64_t>(sbo >> 4) << 32) | (static_cast<uint64_t>(1) << 46) | (static_cast<uint64_t>(2) << 61);
}

// Instruction descriptor, fp32 accumulator, M = 64.  kBf16: both operands bf16
// (kind::f16).  kF8 (kind::f8f6f4): B e4m3, A e4m3 (q) or e5m2 (weights).
// b_mn: B is MN-major.
template <int OP>
__device__ __forceinline__ constexpr uint32_t instr_desc(int n, bool b_mn) {
  const uint32_t at = OP == kBf16 ? 1u : (b_mn ? 1u : 0u), bt = OP == kBf16 ? 1u : 0u;
  return (1u << 4) | (at << 7) | (bt << 10) | ((b_mn ? 1u : 0u) << 16) | (static_cast<uint32_t>(n >> 3) << 17) |
         (static_cast<uint32_t>(kRowsTile >> 4) << 24);
}

// One MMA, issued by one lane of the warp.  The warp stays converged, and
// everything that decides the addresses is uniform over it (broadcast where it
// comes from memory), so the compiler keeps the descriptors in uniform
// registers.  Issued from a branch on the lane, each MMA first moved its
// descriptors there: 50 to 160 cycles, where the N = 64 form takes 32 (the 4 KB
// of its operands at 128 bytes a cycle).
template <int OP>
__device__ __forceinline__ void mma_ws(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
  if constexpr (OP == kBf16) {
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "elect.sync _|q, 0xffffffff;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "@q tcgen05.mma.ws.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
        : "memory");
  } else {
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "elect.sync _|q, 0xffffffff;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "@q tcgen05.mma.ws.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
        : "memory");
  }
}

// The same with A in TMEM.
template <int OP>
__device__ __forceinline__ void mma_ws_tmem(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
  if constexpr (OP == kBf16) {
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "elect.sync _|q, 0xffffffff;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "@q tcgen05.mma.ws.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
        "r"(a), "l"(b), "r"(idesc), "r"(accumulate)
        : "memory");
  } else {
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "elect.sync _|q, 0xffffffff;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "@q tcgen05.mma.ws.cta_group::1.kind::f8f6f4 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
        "r"(a), "l"(b), "r"(idesc), "r"(accumulate)
        : "memory");
  }
}

// 16 bytes of each of 64 rows to four columns of TMEM lanes 0..63 and again of
// lanes 64..127: a .ws product reads its A rows in both places.
__device__ __forceinline__ void tmem_copy(uint32_t taddr, uint64_t desc) {
  asm volatile(
      "{\n\t.reg .pred q;\n\t"
      "elect.sync _|q, 0xffffffff;\n\t"
      "@q tcgen05.cp.cta_group::1.64x128b.warpx2::02_13 [%0], %1;\n\t}" ::"r"(taddr),
      "l"(desc)
      : "memory");
}

__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(p));
  return p != 0u;
}

// All MMAs issued so far arrive on the barrier when they have completed.
__device__ __forceinline__ void commit(uint32_t bar) {
  if (elect_one())
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
  __syncwarp();
}


__device__ __forceinline__ void fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }

__device__ __forceinline__ void arrive(uint32_t bar, uint32_t count = 1) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(count) : "memory");
}

__device__ __forceinline__ void fence_async() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

// 32 or 16 columns of this warp's TMEM lanes, one lane's per thread; the wait names
// the registers, so no use of them can be scheduled before it.
template <int N>
__device__ __forceinline__ void tmem_ld(uint32_t taddr, uint32_t (&v)[N]);

template <>
__device__ __forceinline__ void tmem_ld<32>(uint32_t taddr, uint32_t (&v)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
      "%15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]), "=r"(v[8]),
        "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15]), "=r"(v[16]),
        "=r"(v[17]), "=r"(v[18]), "=r"(v[19]), "=r"(v[20]), "=r"(v[21]), "=r"(v[22]), "=r"(v[23]), "=r"(v[24]),
        "=r"(v[25]), "=r"(v[26]), "=r"(v[27]), "=r"(v[28]), "=r"(v[29]), "=r"(v[30]), "=r"(v[31])
      : "r"(taddr)
      : "memory");
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(v[0]), "+r"(v[1]), "+r"(v[2]), "+r"(v[3]), "+r"(v[4]), "+r"(v[5]), "+r"(v[6]), "+r"(v[7]),
                 "+r"(v[8]), "+r"(v[9]), "+r"(v[10]), "+r"(v[11]), "+r"(v[12]), "+r"(v[13]), "+r"(v[14]),
                 "+r"(v[15]), "+r"(v[16]), "+r"(v[17]), "+r"(v[18]), "+r"(v[19]), "+r"(v[20]), "+r"(v[21]),
                 "+r"(v[22]), "+r"(v[23]), "+r"(v[24]), "+r"(v[25]), "+r"(v[26]), "+r"(v[27]), "+r"(v[28]),
                 "+r"(v[29]), "+r"(v[30]), "+r"(v[31])
               :
               : "memory");
}

template <>
__device__ __forceinline__ void tmem_ld<16>(uint32_t taddr, uint32_t (&v)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, "
      "[%16];"
      : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]), "=r"(v[8]),
        "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15])
      : "r"(taddr)
      : "memory");
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(v[0]), "+r"(v[1]), "+r"(v[2]), "+r"(v[3]), "+r"(v[4]), "+r"(v[5]), "+r"(v[6]), "+r"(v[7]),
                 "+r"(v[8]), "+r"(v[9]), "+r"(v[10]), "+r"(v[11]), "+r"(v[12]), "+r"(v[13]), "+r"(v[14]),
                 "+r"(v[15])
               :
               : "memory");
}

__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t (&v)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%32], {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, "
      "%14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31};" ::"r"(v[0]),
      "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]), "r"(v[10]),
      "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15]), "r"(v[16]), "r"(v[17]), "r"(v[18]), "r"(v[19]),
      "r"(v[20]), "r"(v[21]), "r"(v[22]), "r"(v[23]), "r"(v[24]), "r"(v[25]), "r"(v[26]), "r"(v[27]), "r"(v[28]),
      "r"(v[29]), "r"(v[30]), "r"(v[31]), "r"(taddr)
      : "memory");
}

// Waits for the phase, until `spins` tries (looked at every sixteenth) or another role's giving up.
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, volatile uint32_t* abort_flag, uint32_t spins) {
  for (uint32_t i = 0;; ++i) {
    uint32_t done;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.b32 p, 0, 0;\n\t"
        "elect.sync _|q, 0xffffffff;\n\t"
        "@q mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(done)
        : "r"(bar), "r"(parity)
        : "memory");
    if (__any_sync(0xffffffffu, done != 0u)) return true;
    if ((i & 15u) == 15u && __any_sync(0xffffffffu, i >= spins || *abort_flag != 0u)) return false;
  }
}

// barrier `id` over `n` threads, returning the OR of `pred` over them
__device__ __forceinline__ bool bar_or(int id, int n, bool pred) {
  uint32_t out;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.u32 p, %1, 0;\n\t"
      "barrier.red.or.pred q, %2, %3, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(out)
      : "r"(pred ? 1u : 0u), "r"(id), "r"(n)
      : "memory");
  return out != 0u;
}

__device__ __forceinline__ void bar_sync(int id, int n) { asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(n) : "memory"); }

__device__ __forceinline__ float exp2_fast(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// Two fp16 rounded to the nearest e5m2 (ties away from zero), as fp16: an e5m2 is
// the upper byte of an fp16.  Integer arithmetic, since conversions share a unit of
// a quarter of the rate with the exponentials.  (No finite value here is near
// e5m2's largest; a NaN may turn into 0, but the row's denominator is a NaN then.)
__device__ __forceinline__ uint32_t near_e5m2(uint32_t h) { return (h + 0x00800080u) & 0xff00ff00u; }

__device__ __forceinline__ uint32_t sub_f16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

__device__ __forceinline__ void st_shared(uint32_t addr, const uint4& v) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w)
               : "memory");
}

__device__ __forceinline__ uint4 ld_shared(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr) : "memory");
  return v;
}

// 16 bytes global -> shared without registers; `ok` false writes zeros and reads nothing.
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool ok) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(ok ? 16 : 0) : "memory");
}

// The barrier gets one arrival of this thread when its copies so far have landed.
__device__ __forceinline__ void cp_async_arrive(uint32_t bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
}

// `bytes` contiguous bytes global -> shared by the copy engine, counted on the barrier.
__device__ __forceinline__ void bulk_copy(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
               "l"(src), "r"(bytes), "r"(bar)
               : "memory");
}

// A box of the cache (128 bytes of `box_rows` rows) into swizzled rows, counted on the barrier.
__device__ __forceinline__ void tensor_copy(uint32_t dst, const CUtensorMap* map, int x, int row, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(
          dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(row), "r"(bar)
      : "memory");
}

// The same of several slabs, each 64 rows below the one before it: a half of a tile at once.
__device__ __forceinline__ void tensor_copy_half(uint32_t dst, const CUtensorMap* map, int row, int slab, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(
          dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(0), "r"(row), "r"(slab), "r"(bar)
      : "memory");
}

__device__ __forceinline__ void arrive_expect(uint32_t bar, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes) : "memory");
}

// Segments known ahead: more than the roles are ever apart would be of no use.
constexpr uint32_t kSegments = 8;

struct Bars {
  uint64_t full[kMaxHalves], empty[kMaxHalves];
  uint64_t q_empty;
  uint64_t s_full[2], s_empty[2];
  uint64_t p_full[2], pv_done[2], o_empty;  // [tile & 1]
  uint64_t drained[2];
  uint64_t seg_full[kSegments], seg_empty[kSegments];
};

struct Shared {
  Bars bars;
  Segment segments[kSegments];
  uint32_t tmem;
  uint32_t abort_flag;
  uint32_t never;  // stays 0
  alignas(16) uint8_t valid[kMaxSlots][kKeys];  // 1: the key counts, by rotary slot
  float xch[4][kRowsTile];
  int64_t warp_sum[kThreads / 32];
  int64_t first_unit, first_base;
  Unit unit;  // the first unit: every role starts with it
};

// ---- the loaders' pieces --------------------------------------------------------
//
// A warp has eight or sixteen rows of a tile.  Its lanes read along the rows (256
// or 512 contiguous bytes at a time): with a few lanes on each of eight rows the
// same loads took four times as many passes through the load pipe.

// Piece `c` (0..7) of slab `s` of row r in a tile at `base`.
__device__ __forceinline__ uint32_t piece_addr(uint32_t base, int s, int r, int c) {
  return base + static_cast<uint32_t>(s) * kSlabBytes + static_cast<uint32_t>(r) * 128u +
         (static_cast<uint32_t>(c ^ (r & 7)) << 4);
}

// The address of row i of the warp's rows from the lane that holds it; null: no key.
__device__ __forceinline__ const uint8_t* row_at(const uint8_t* mine, int i) {
  return reinterpret_cast<const uint8_t*>(__shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(mine), i));
}

// ROWS rows that need no decoding, as a lane copies them, 16 bytes at a time: of
// step i it copies one piece of row `of`.  (All rows' addresses are had before the
// first copy: a shuffle between two copies waits for the first.)
template <int OP, int ROWS>
struct Pieces {
  static constexpr int kHalf = 8 * Shape<OP>::kHalfSlabs;  // pieces of a row's half: 32 or 16
  static constexpr int kAtOnce = 32 / kHalf;               // rows a warp covers at once
  static constexpr int kPe = 4 * Shape<OP>::kElem;         // pieces of the rotary values: 8 or 4
  const uint8_t* of[ROWS / kAtOnce];
  const uint8_t* of_pe[ROWS * kPe / 32];

  __device__ __forceinline__ Pieces(const uint8_t* mine, int lane) {
#pragma unroll
    for (int i = 0; i < ROWS / kAtOnce; ++i) of[i] = row_at(mine, kAtOnce * i + lane / kHalf);
#pragma unroll
    for (int i = 0; i < ROWS * kPe / 32; ++i) of_pe[i] = row_at(mine, (32 / kPe) * i + lane / kPe);
  }
  // Half h's values, or the rotary values, piece by piece: f(slab, row, piece, address of the piece or null).
  template <class F>
  __device__ __forceinline__ void values(int h, int lane, const F& f) const {
#pragma unroll
    for (int i = 0; i < ROWS / kAtOnce; ++i) {
      const int c = lane % kHalf;
      f(Shape<OP>::kHalfSlabs * h + (c >> 3), kAtOnce * i + lane / kHalf, c & 7,
        of[i] != nullptr ? of[i] + 16 * (kHalf * h + c) : nullptr);
    }
  }
  template <class F>
  __device__ __forceinline__ void rotary(int lane, const F& f) const {
#pragma unroll
    for (int i = 0; i < ROWS * kPe / 32; ++i) {
      const int c = lane % kPe;
      f(Shape<OP>::kPeSlab, (32 / kPe) * i + lane / kPe, c, of_pe[i] != nullptr ? of_pe[i] + 16 * (2 * kHalf + c) : nullptr);
    }
  }
};

// What a lane holds of its warp's eight quantised rows.  Half h of rows 2 j and
// 2 j + 1 (lanes 0..15 and 16..31): codes[4 h + j], 16 codes a lane.  The rest
// of the rows: the rotary values.
template <int FMT>
struct Raw {
  uint4 codes[8];
  uint4 rest[FMT == MLA_CACHE_MX ? 2 : 1];
  uint4 scales;  // mx: the 16 scale bytes of row `lane` (lanes 0..7)
};

template <int FMT>
__device__ __forceinline__ void load_rows(Raw<FMT>& raw, const uint8_t* mine, int lane) {
  const uint8_t* rows[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) rows[j] = row_at(mine, 2 * j + (lane >> 4));
  if constexpr (FMT == MLA_CACHE_MX) {
    const uint8_t* rest[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) rest[i] = row_at(mine, 4 * i + (lane >> 3));
    raw.scales = load16(mine, kMxScales);
#pragma unroll
    for (int i = 0; i < 2; ++i) raw.rest[i] = load16(rest[i], kMxPe + 16 * (lane & 7));
  } else {
    raw.rest[0] = load16(row_at(mine, lane >> 2), 512 + 16 * (lane & 3));
  }
#pragma unroll
  for (int h = 0; h < 2; ++h)
#pragma unroll
    for (int j = 0; j < 4; ++j) raw.codes[4 * h + j] = load16(rows[j], 256 * h + 16 * (lane & 15));
}

// Sixteen codes -> two pieces of bf16 values.
template <int FMT>
__device__ __forceinline__ void decode(const uint4& w, uint32_t byte, uint4& a, uint4& b) {
  if ((FMT == MLA_CACHE_MX && byte > kMxPlain) || any_nan_code(w)) {
    codes_to_bf16(w, FMT == MLA_CACHE_MX ? mx_scale(byte) : 1.0f, a, b);
  } else {
    plain_codes_to_bf16(w, FMT == MLA_CACHE_MX ? mx_mul2(byte) : kBf16Pow120, a, b);
  }
}

// Half h of the warp's rows, decoded, through `put(slab, row, piece, value)`.
// A lane's two pieces swap places in odd slabs, so that eight lanes' stores
// fall on different banks.
template <int FMT, class Put>
__device__ __forceinline__ void store_half(const Raw<FMT>& raw, int h, int row0, int lane, const Put& put) {
  const int slab = 4 * h + ((lane & 15) >> 2), piece = 2 * (lane & 3), odd = (lane >> 2) & 1;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int r = row0 + 2 * j + (lane >> 4);
    uint32_t byte = 0;
    if constexpr (FMT == MLA_CACHE_MX) {  // of group 8 h + (lane & 15) / 2
      const int from = 2 * j + (lane >> 4);
      const uint32_t lo = __shfl_sync(0xffffffffu, h == 0 ? raw.scales.x : raw.scales.z, from);
      const uint32_t hi = __shfl_sync(0xffffffffu, h == 0 ? raw.scales.y : raw.scales.w, from);
      byte = (((lane & 8) != 0 ? hi : lo) >> (8 * ((lane >> 1) & 3))) & 0xffu;
    }
    uint4 a, b;
    decode<FMT>(raw.codes[4 * h + j], byte, a, b);
    put(slab, r, piece + odd, odd ? b : a);
    put(slab, r, piece + (odd ^ 1), odd ? a : b);
  }
  if (h == 0) {
    if constexpr (FMT == MLA_CACHE_MX) {
#pragma unroll
      for (int i = 0; i < 2; ++i) put(8, row0 + 4 * i + (lane >> 3), lane & 7, raw.rest[i]);
    } else {
      uint4 a, b;
      decode<FMT>(raw.rest[0], 0u, a, b);
      put(8, row0 + (lane >> 2), 2 * (lane & 3), a);
      put(8, row0 + (lane >> 2), 2 * (lane & 3) + 1, b);
    }
  }
}

// ---- the roles ---------------------------------------------------------------------

// On a wait that ran out (not on another role's): says so, and that all roles stop.
__device__ __forceinline__ void give_up(const Params& p, uint32_t* abort_flag) {
  volatile uint32_t* ab = abort_flag;
  if ((threadIdx.x & 31u) == 0u && *ab == 0u) {
    *ab = 1u;
    report(p.status, MLA_STATUS_TIMEOUT);
  }
}

// One warp finds the CTA's segments for all the others.  Found by each of them
// for itself, a segment cost every role some 2000 cycles (lengths to be fetched,
// 64-bit divisions), one role behind the other.
__device__ __forceinline__ bool find_segments(const Params& p, Cursor cur, Shared& sh) {
  for (uint32_t n = 0;; ++n) {
    Segment s;
    if (!next_segment(p, cur, s)) s.k0 = s.k1 = 0;
    if (n >= kSegments &&
        !warp_wait(smem_u32(&sh.bars.seg_empty[n % kSegments]), (n / kSegments - 1) & 1u, &sh.abort_flag, p.spins))
      return false;
    if ((threadIdx.x & 31u) == 0u) {
      sh.segments[n % kSegments] = s;
      arrive(smem_u32(&sh.bars.seg_full[n % kSegments]));
    }
    __syncwarp();
    if (s.k0 == s.k1) return true;
  }
}

// Segment n, when it is known; and the warp's leave of it.
__device__ __forceinline__ bool segment_known(const Params& p, Shared& sh, uint32_t n) {
  return warp_wait(smem_u32(&sh.bars.seg_full[n % kSegments]), (n / kSegments) & 1u, &sh.abort_flag, kFindTimes * p.spins);
}
__device__ __forceinline__ void segment_done(Shared& sh, uint32_t n) {
  __syncwarp();
  if ((threadIdx.x & 31u) == 0u) arrive(smem_u32(&sh.bars.seg_empty[n % kSegments]));
}

// A walk over this CTA's key tiles, one at a time.  A tile that comes by copies of
// many bytes each (an image's, or a whole one by tensor copies) is one loader
// warp's work, in turn; of the others each warp has some rows.
struct TileWalk {
  const int32_t* table = nullptr;
  int32_t len = 0, kt = 0, k0 = 0, k1 = 0;
  uint32_t seg = 0;    // segments begun
  int32_t number = -1;  // of the tile, in the CTA's run
  int32_t owned = 0;   // tiles of the segment before this one are one warp's each
  bool copied = false;  // the segment's tiles come from an image
  bool any = true;     // not yet behind the last

  // To the next tile; false: a wait ran out.  `boxes`: tensor copies are made.
  __device__ __forceinline__ bool next(const Params& p, Shared& sh, bool boxes) {
    ++number;
    if (!any || ++kt < k1) return true;
    if (!segment_known(p, sh, seg)) return false;
    const Segment& s = sh.segments[seg % kSegments];
    kt = k0 = uniform(s.k0);
    k1 = uniform(s.k1);
    any = k0 < k1;
    table = s.table;
    len = uniform(s.len);
    copied = uniform(s.image != nullptr ? 1 : 0) != 0;
    owned = copied ? k1 : boxes ? len / kKeys : 0;
    ++seg;
    return true;
  }
};

struct Tile {
  int32_t kt;
  uint32_t seg;
  bool copied, first, any;
  bool whole;  // one warp's work
  bool mine;   // this warp has work with it

  __device__ __forceinline__ Tile(const TileWalk& w, int warp, int warps)
      : kt(w.kt),
        seg(w.seg),
        copied(w.copied),
        first(w.kt == w.k0),
        any(w.any),
        whole(w.kt < w.owned),
        mine(!(w.kt < w.owned) || w.number % warps == warp) {}
};

// Where the key of row r of a tile lies.  The page number is fetched a tile
// ahead and not looked at before address().
struct KeyAt {
  int32_t page;
  uint32_t in_page;
  bool key;

  __device__ __forceinline__ void fetch(const Params& p, const int32_t* table, int32_t len, int32_t kt, int r, bool any) {
    const uint32_t k = static_cast<uint32_t>(kt) * kKeys + static_cast<uint32_t>(r);
    key = any && k < static_cast<uint32_t>(len);
    page = 0;
    in_page = 0;
    if (key) {
      const uint32_t bs = static_cast<uint32_t>(p.block_size), pg = k / bs;
      in_page = k - pg * bs;
      page = __ldcg(table + pg);
    }
  }
  // null: no key, or no such page (`bad`)
  __device__ __forceinline__ const uint8_t* address(const Params& p, int bytes, bool& bad) const {
    const bool ok = key && page >= 0 && page < p.cache_blocks;
    bad = bad || (key && !ok);
    return ok ? p.cache + (static_cast<int64_t>(page) * p.block_size + in_page) * bytes : nullptr;
  }
};

// q row `i` of the `rows` from `row0` on.
__device__ __forceinline__ const uint8_t* q_row(const Params& p, int32_t row0, int32_t rows, int i, bool& ok) {
  ok = i < rows;
  const int32_t row = ok ? row0 + i : 0, t = row / p.H;
  return p.q + static_cast<int64_t>(t) * p.q_st + static_cast<int64_t>(row - t * p.H) * p.q_sh;
}

// A loader warp's part of the segment's 64 q rows, to `to(slab, row, piece)`; the
// two halves' barriers get the warp's arrivals.  What stays in shared memory is
// written once `free()` has waited for the previous segment's scores.
template <int FMT, int OP, class To, class Free>
__device__ __forceinline__ bool load_q(const Params& p, int32_t row0, int32_t rows, const To& to, const Free& free,
                                       uint32_t full0, uint32_t full1, int warp, int lane) {
  constexpr int kRows = Roles<FMT, OP>::kRows;
  constexpr bool kStay = Shape<OP>::kQSlabs > 0;
  bool ok;
  const uint8_t* mine = q_row(p, row0, rows, kRows * warp + lane % kRows, ok);
  if (!ok || lane >= kRows) mine = nullptr;
  if (OP == kBf16 && p.q_fp8) {
    if (!free()) return false;
#pragma unroll
    for (int i = 0; i < kRows / 8; ++i) {
      const uint8_t* eight = row_at(mine, 8 * i + (lane & 7));
      Raw<MLA_CACHE_E4M3> raw;
      load_rows<MLA_CACHE_E4M3>(raw, lane < 8 ? eight : nullptr, lane);
      auto put = [&](int s, int r, int c, const uint4& v) { st_shared(to(s, r, c), v); };
      store_half<MLA_CACHE_E4M3>(raw, 0, kRows * warp + 8 * i, lane, put);
      store_half<MLA_CACHE_E4M3>(raw, 1, kRows * warp + 8 * i, lane, put);
    }
    __syncwarp();
    if (lane == 0) {
      arrive(full0, kArrivals);
      arrive(full1, kArrivals);
    }
  } else {
    const Pieces<OP, kRows> pieces(mine, lane);
    auto copy = [&](int s, int r, int c, const uint8_t* src) {
      cp_async16(to(s, kRows * warp + r, c), src != nullptr ? src : p.q, src != nullptr);
    };
    pieces.values(0, lane, copy);
    if (!kStay) pieces.rotary(lane, copy);
    cp_async_arrive(full0);
    if (lane == 0) arrive(full0);
    if (kStay && !free()) return false;
    pieces.values(1, lane, copy);
    if (kStay) pieces.rotary(lane, copy);
    cp_async_arrive(full1);
    if (lane == 0) arrive(full1);
  }
  return true;
}

// The cache as seen by tensor copies: 128 bytes of box_rows rows; and where that is
// a whole tile, half a tile's slabs of 64 rows.
struct Maps {
  const CUtensorMap *slab, *half;
};

// Loader warps fill the ring: for each segment its q rows, then tile by tile.  A
// half's barrier counts kArrivals of each warp: one of its own, and one of each
// thread's asynchronous copies where there are any.
template <int FMT, int OP>
struct Filler {
  using S = Shape<OP>;
  using R = Roles<FMT, OP>;
  const Params& p;
  Shared& sh;
  uint32_t smem;
  int warp, lane;
  Ring<OP> ring;

  // The ring's next half, when it is free.
  __device__ __forceinline__ bool acquire() const {
    return ring.lap == 0 || warp_wait(smem_u32(&sh.bars.empty[ring.half]), (ring.lap - 1) & 1u, &sh.abort_flag, p.spins);
  }
  // Past a tile that is other warps' work.  Waits and arrives all the same: a wait on a
  // barrier tells a phase from its neighbours only, so no warp may come to lag two
  // phases behind the others.  (Without its arrivals a tile, the work of one warp,
  // went its whole way without the rest.)
  __device__ __forceinline__ bool skip_tile() {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      if (!acquire()) return false;
      if (lane == 0) arrive(smem_u32(&sh.bars.full[ring.half]), kArrivals);
      __syncwarp();
      ring.next_half();
    }
    ring.next_tile();
    return true;
  }
  // The q rows of segment seg - 1.
  __device__ __forceinline__ bool fill_q(uint32_t seg) {
    const Segment& info = sh.segments[(seg - 1) % kSegments];
    const uint32_t full0 = smem_u32(&sh.bars.full[ring.half]), base0 = smem + ring.half * S::kHalf;
    if (!acquire()) return false;
    ring.next_half();
    const uint32_t full1 = smem_u32(&sh.bars.full[ring.half]), base1 = smem + ring.half * S::kHalf;
    if (!acquire()) return false;
    ring.next_half();
    const uint32_t rest = smem + S::kQAt, pe = smem + S::kPeAt + ring.slot * kSlabBytes;
    ring.next_tile();
    auto to = [&](int s, int r, int c) {
      return s >= S::kQSlab0      ? piece_addr(rest, s - S::kQSlab0, r, c)
             : s == S::kPeSlab    ? piece_addr(pe, 0, r, c)
             : s >= S::kHalfSlabs ? piece_addr(base1, s - S::kHalfSlabs, r, c)
                                  : piece_addr(base0, s, r, c);
    };
    auto free = [&]() {
      return seg <= 1 || warp_wait(smem_u32(&sh.bars.q_empty), (seg - 2) & 1u, &sh.abort_flag, p.spins);
    };
    return load_q<FMT, OP>(p, info.row0, info.rows, to, free, full0, full1, warp, lane);
  }
  // A tile, half by half: put(h, place of a piece, barrier, place of the rotary slab, flags).
  template <class Put>
  __device__ __forceinline__ bool fill(const Put& put) {
    const uint32_t pe = smem + S::kPeAt + ring.slot * kSlabBytes;
    uint8_t* valid = sh.valid[ring.slot];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const uint32_t full = smem_u32(&sh.bars.full[ring.half]), base = smem + ring.half * S::kHalf;
      if (!acquire()) return false;
      ring.next_half();
      put(h, base, full, pe, valid);
    }
    ring.next_tile();
    return true;
  }
  // A tile of an image.
  __device__ __forceinline__ bool fill_image(const Tile& t) {
    return fill([&](int h, uint32_t base, uint32_t full, uint32_t pe, uint8_t* valid) {
      if (elect_one()) {
        const uint8_t* image = sh.segments[(t.seg - 1) % kSegments].image + static_cast<int64_t>(t.kt) * S::kImage;
        arrive(full, kArrivals - 1);
        arrive_expect(full, S::kHalf + (h == 0 ? kSlabBytes + kKeys : 0));
        bulk_copy(base, image + h * S::kHalf, S::kHalf, full);
        if (h == 0) {
          bulk_copy(pe, image + S::kPeSlab * kSlabBytes, kSlabBytes, full);
          bulk_copy(smem_u32(valid), image + S::kTile, kKeys, full);
        }
      }
      __syncwarp();
    });
  }
};

// Piece `c` of slab `s`, row r of half h of a tile.
template <int OP>
__device__ __forceinline__ uint32_t half_addr(uint32_t base, uint32_t pe, int h, int s, int r, int c) {
  return s == Shape<OP>::kPeSlab ? piece_addr(pe, 0, r, c) : piece_addr(base, s - h * Shape<OP>::kHalfSlabs, r, c);
}

// Rows kept as they are.
template <int FMT, int OP>
__device__ __forceinline__ bool copy_tiles(const Params& p, const Maps& maps, Filler<FMT, OP>& f, bool& bad_page) {
  using S = Shape<OP>;
  using R = Roles<FMT, OP>;
  const int warp = f.warp, lane = f.lane, row0 = R::kRows * warp;
  // Of a tile that all warps fill, lane i < kRows looks after row i of the warp's;
  // of one that comes by tensor copies, lane i after box i, which is copied slab
  // by slab.  Page numbers are fetched two tiles ahead.
  TileWalk w;  // two tiles ahead of the one being stored
  KeyAt at;
  const int boxes = p.box_rows > 0 ? kKeys / p.box_rows : 0;
  auto fetch = [&](const Tile& t) {
    if (!t.any || !t.mine || t.copied) return;
    const int look = !t.whole ? (lane < R::kRows ? row0 + lane : -1) : lane < boxes ? lane * p.box_rows : -1;
    at.fetch(p, w.table, w.len, t.kt, look, look >= 0);
  };
  // where the tile's rows lie that this lane looks after
  const uint8_t* mine = nullptr;
  int32_t box = 0;
  auto locate = [&](const Tile& t) {
    mine = nullptr;
    if (!t.any || !t.mine || t.copied) return;
    mine = at.address(p, row_bytes(FMT), bad_page);
    box = static_cast<int32_t>(static_cast<uint32_t>(at.page) * static_cast<uint32_t>(p.block_size) + at.in_page);
  };
  auto rows = [&](int h, uint32_t base, uint32_t full, uint32_t pe, uint8_t* valid) {
    if (h == 0 && lane < R::kRows) valid[row0 + lane] = mine != nullptr ? 1 : 0;
    const Pieces<OP, R::kRows> pieces(mine, lane);
    auto copy = [&](int s, int r, int c, const uint8_t* src) {
      cp_async16(half_addr<OP>(base, pe, h, s, row0 + r, c), src != nullptr ? src : p.q, src != nullptr);
    };
    pieces.values(h, lane, copy);
    if (h == 0) pieces.rotary(lane, copy);
    cp_async_arrive(full);
    __syncwarp();
    if (lane == 0) arrive(full);
  };
  auto whole = [&](int h, uint32_t base, uint32_t full, uint32_t pe, uint8_t* valid) {
    // a box in a page that does not exist: no keys
    const uint32_t gone = __ballot_sync(0xffffffffu, lane < boxes && mine == nullptr);
    const uint32_t box_bytes = static_cast<uint32_t>(p.box_rows) * 128u;
    const int slabs = S::kHalfSlabs + (h == 0 ? 1 : 0);
    if (h == 0 && lane < kKeys / 4) reinterpret_cast<uint32_t*>(valid)[lane] = 0x01010101u;
    if (gone != 0u) {
      __syncwarp();
      if (h == 0 && lane < boxes && mine == nullptr)
        for (int i = 0; i < p.box_rows; ++i) valid[lane * p.box_rows + i] = 0;
      for (int i = lane; i < slabs * kKeys * 8; i += 32) {
        const int s = i / (kKeys * 8), r = (i >> 3) % kKeys;
        if ((gone >> (r / p.box_rows)) & 1u)
          st_shared(half_addr<OP>(base, pe, h, s < S::kHalfSlabs ? h * S::kHalfSlabs + s : S::kPeSlab, r, i & 7),
                    make_uint4(0, 0, 0, 0));
      }
      fence_async();
    }
    __syncwarp();
    if (lane == 0) {
      arrive(full, kArrivals - 1);
      arrive_expect(full, static_cast<uint32_t>(slabs * (boxes - __popc(gone))) * box_bytes);
    }
    __syncwarp();
    if (lane < boxes && mine != nullptr) {
      constexpr int kX = 128 / S::kElem;
      const uint32_t row = static_cast<uint32_t>(lane) * box_bytes;
      if (h == 0) tensor_copy(pe + row, maps.slab, S::kPeSlab * kX, box, full);
      if (boxes == 1) {
        tensor_copy_half(base, maps.half, box, h * S::kHalfSlabs, full);
      } else {
#pragma unroll
        for (int s = 0; s < S::kHalfSlabs; ++s)
          tensor_copy(base + static_cast<uint32_t>(s) * kSlabBytes + row, maps.slab, (h * S::kHalfSlabs + s) * kX, box, full);
      }
    }
    __syncwarp();
  };
  auto next = [&]() { return w.next(p, f.sh, boxes > 0); };
  auto tile = [&]() { return Tile(w, warp, R::kLoad); };
  if (!next()) return false;
  Tile now = tile();
  fetch(now);
  // the first segment's q rows go out while page numbers are under way
  if (now.any && !f.fill_q(now.seg)) return false;
  locate(now);
  if (!next()) return false;
  Tile then = tile();
  fetch(then);
  while (now.any) {
    if (now.first && now.seg > 1 && !f.fill_q(now.seg)) return false;
    if (!now.mine) {
      if (!f.skip_tile()) return false;
    } else if (now.copied) {
      if (!f.fill_image(now)) return false;
    } else if (now.whole) {
      if (!f.fill(whole)) return false;
    } else {
      if (!f.fill(rows)) return false;
    }
    locate(then);
    if (!then.any || then.first) segment_done(f.sh, now.seg - 1);
    now = then;
    if (!next()) return false;
    then = tile();
    fetch(then);
  }
  return true;
}

// Rows to be decoded, eight a warp.  An arrival on a barrier waits for the loads
// before it, so the next tile's go out behind this one's last arrival.  (Two groups
// of four warps that take tiles in turn, sixteen rows a warp, so as to load and
// decode at the same time, took 7200 and 6900 cycles a tile, against 6000 and 5100:
// they too have to arrive for one another's tiles.)
template <int FMT, int OP>
__device__ __forceinline__ bool decode_tiles(const Params& p, Filler<FMT, OP>& f, bool& bad_page) {
  using R = Roles<FMT, OP>;
  constexpr int kRows = R::kRows;
  const int warp = f.warp, lane = f.lane, row0 = kRows * warp;
  TileWalk w;  // two tiles ahead of the one being stored
  KeyAt at;
  Raw<FMT> raw;
  const uint8_t* mine = nullptr;  // the row that lane < kRows looks after
  auto take = [&]() {
    const Tile t(w, warp, R::kLoad);
    if (t.any && !t.copied) at.fetch(p, w.table, w.len, t.kt, lane < kRows ? row0 + lane : -1, lane < kRows);
    return t;
  };
  auto load = [&](const Tile& t) {
    mine = t.any && !t.copied ? at.address(p, row_bytes(FMT), bad_page) : nullptr;
    load_rows<FMT>(raw, mine, lane);
  };
  auto rows = [&](int h, uint32_t base, uint32_t full, uint32_t pe, uint8_t* valid) {
    if (h == 0 && lane < kRows) valid[row0 + lane] = mine != nullptr ? 1 : 0;
    store_half<FMT>(raw, h, row0, lane,
                    [&](int s, int r, int c, const uint4& v) { st_shared(half_addr<OP>(base, pe, h, s, r, c), v); });
    __syncwarp();
    if (lane == 0) arrive(full, kArrivals);
  };
  if (!w.next(p, f.sh, false)) return false;
  Tile now = take();
  if (now.any && !f.fill_q(now.seg)) return false;
  load(now);
  if (!w.next(p, f.sh, false)) return false;
  Tile then = take();
  while (now.any) {
    if (now.first && now.seg > 1 && !f.fill_q(now.seg)) return false;
    if (!now.mine) {
      if (!f.skip_tile()) return false;
    } else if (now.copied) {
      if (!f.fill_image(now)) return false;
    } else {
      if (!f.fill(rows)) return false;
    }
    load(then);
    if (!then.any || then.first) segment_done(f.sh, now.seg - 1);
    now = then;
    if (!w.next(p, f.sh, false)) return false;
    then = take();
  }
  return true;
}

template <int FMT, int OP>
__device__ __forceinline__ void loader(const Params& p, const Maps& maps, Shared& sh, uint32_t smem) {
  bool bad_page = false;
  using R = Roles<FMT, OP>;
  Filler<FMT, OP> f{p, sh, smem, uniform((static_cast<int>(threadIdx.x) >> 5) - R::kLoad0),
                    static_cast<int>(threadIdx.x) & 31, {}};
  bool good;
  if constexpr (R::kDecode) {
    good = decode_tiles<FMT, OP>(p, f, bad_page);
  } else {
    good = copy_tiles<FMT, OP>(p, maps, f, bad_page);
  }
  // no copy may be under way when the CTA ends: on the way out after a timeout
  // (else every copy's tile has been used) give the copy engine's theirs
  asm volatile("cp.async.wait_all;" ::: "memory");
  if (!good) {
    give_up(p, &sh.abort_flag);
    for (int i = 0; i < Shape<OP>::kHalves; ++i)
      for (uint32_t parity = 0; parity < 2; ++parity) (void)warp_wait(smem_u32(&sh.bars.full[i]), parity, &sh.never, kLandSpins);
  }
  if (bad_page) report(p.status, MLA_STATUS_SLOT_RANGE);
}

// The products of one tile's weights with half of its values, into 256 columns of
// the sums, which they add to (`more`) or begin.
template <int OP>
__device__ __forceinline__ void pv_half(uint64_t p, uint64_t v, uint32_t d, uint32_t more) {
  using S = Shape<OP>;
  constexpr uint32_t id = instr_desc<OP>(256, true);
  constexpr uint64_t kStep = static_cast<uint64_t>(kSlabBytes / S::kKeySteps) >> 4;  // that many keys further down the tile
#pragma unroll
  for (int t = 0; t < S::kTerms; ++t) {
    // weights: 32-byte steps along a row; kF8 terms at bytes 0 and 64 of the first slab, 0 of the second
    const uint64_t pt = p + static_cast<uint64_t>(t == 1 ? 4 : t == 2 ? kSlabBytes >> 4 : 0);
#pragma unroll
    for (int j = 0; j < S::kKeySteps; ++j)
      mma_ws<OP>(d, pt + static_cast<uint64_t>(j * 2), v + static_cast<uint64_t>(j) * kStep, id, t == 0 && j == 0 ? more : 1u);
  }
}

// Scores over `slabs` slabs of the keys at `k` and of the q rows, in TMEM or in
// shared memory.  (Unrolled over the slabs too, the compiler kept every product's
// addresses in registers, and where it ran out of them fetched some from memory
// before each product.)
template <int OP>
__device__ __forceinline__ void qk_tmem(uint32_t q, uint64_t k, uint32_t d, int slabs) {
#pragma unroll 1
  for (int s = 0; s < slabs; ++s) {
#pragma unroll
    for (int j = 0; j < 4; ++j)
      mma_ws_tmem<OP>(d, q + 8u * static_cast<uint32_t>(j), k + static_cast<uint64_t>(2 * j), instr_desc<OP>(kKeys, false), 1u);
    q += 32u;
    k += kSlabBytes >> 4;
  }
}

template <int OP>
__device__ __forceinline__ void qk_smem(uint64_t q, uint64_t k, uint32_t d, int slabs) {
#pragma unroll 1
  for (int s = 0; s < slabs; ++s) {
#pragma unroll
    for (int j = 0; j < 4; ++j)
      mma_ws<OP>(d, q + static_cast<uint64_t>(2 * j), k + static_cast<uint64_t>(2 * j), instr_desc<OP>(kKeys, false), 1u);
    q += kSlabBytes >> 4;
    k += kSlabBytes >> 4;
  }
}

// Scores over the rotary slab: the first of a tile.
template <int OP>
__device__ __forceinline__ void qk_rotary(uint32_t q_tmem, uint64_t q_smem, uint64_t k, uint32_t d) {
  using S = Shape<OP>;
#pragma unroll
  for (int j = 0; j < S::kPeSteps; ++j) {
    if constexpr (S::kPeSlab < S::kQSlab0) {
      mma_ws_tmem<OP>(d, q_tmem + 8u * static_cast<uint32_t>(j), k + static_cast<uint64_t>(2 * j), instr_desc<OP>(kKeys, false),
                      j > 0 ? 1u : 0u);
    } else {
      mma_ws<OP>(d, q_smem + static_cast<uint64_t>(2 * j), k + static_cast<uint64_t>(2 * j), instr_desc<OP>(kKeys, false),
                 j > 0 ? 1u : 0u);
    }
  }
}

// STEPS 32-byte pieces of the q rows, at `q`, to TMEM from piece J0 on.
template <int J0, int STEPS>
__device__ __forceinline__ void q_copy(uint64_t q, uint32_t tmem) {
  constexpr int kPieces = STEPS < 4 ? STEPS : 4;  // of a slab
  uint32_t to = tmem + kTmemQ + 8u * J0;
#pragma unroll 1
  for (int s = 0; s < STEPS / kPieces; ++s) {
#pragma unroll
    for (int i = 0; i < 2 * kPieces; ++i) tmem_copy(to + 4u * static_cast<uint32_t>(i), q + static_cast<uint64_t>(i));
    to += 32u;
    q += kSlabBytes >> 4;
  }
}

// Products issued by this warp have completed before TMEM is freed.
__device__ __forceinline__ void drain(uint64_t* bar, uint32_t* never) {
  commit(smem_u32(bar));
  (void)warp_wait(smem_u32(bar), 0u, never, kWaitSpins);
}

// Issues the copies of every segment's q rows to TMEM and the scores' products of every tile.
template <int OP>
__device__ __forceinline__ bool issue_scores(const Params& p, Shared& sh, uint32_t smem, uint32_t tmem) {
  using S = Shape<OP>;
  volatile uint32_t* ab = &sh.abort_flag;
  const uint64_t d_half = smem_desc(smem, 16, 1024), d_pe = smem_desc(smem + S::kPeAt, 16, 1024);
  const uint64_t d_q = smem_desc(smem + S::kQAt, 16, 1024);  // the q rows' slabs from kQSlab0 on
  const uint32_t q = tmem + kTmemQ;
  uint32_t it = 0, segs = 0;
  Ring<OP> ring;
  // The half has come, and the tensor cores may read it.  (The fence between plain
  // stores or asynchronous copies and the tensor cores' reads is made here: made by
  // the warps that decode rows, it waited for the next rows' loads.)
  auto come = [&]() {
    if (!warp_wait(smem_u32(&sh.bars.full[ring.half]), ring.lap & 1u, ab, p.spins)) return false;
    fence_async();
    fence_after();
    return true;
  };
  while (true) {
    if (!segment_known(p, sh, segs)) return false;
    const Segment& x = sh.segments[segs % kSegments];
    const int tiles = uniform(x.k1 - x.k0);
    if (tiles == 0) return true;
    segment_done(sh, segs);
    if (!come()) return false;
    // The products that read the previous segment's q rows have completed.  Those
    // that read these run behind the copies.
    if (segs > 0 && !warp_wait(smem_u32(&sh.bars.q_empty), (segs - 1) & 1u, ab, p.spins)) return false;
    ++segs;
    q_copy<0, 4 * S::kHalfSlabs>(smem_desc(smem + ring.half * S::kHalf, 16, 1024), tmem);
    if (S::kPeSlab < S::kQSlab0)
      q_copy<4 * S::kPeSlab, S::kPeSteps>(smem_desc(smem + S::kPeAt + ring.slot * kSlabBytes, 16, 1024), tmem);
    commit(smem_u32(&sh.bars.empty[ring.half]));
    ring.next_half();
    if (!come()) return false;
    constexpr int kSlabs = (S::kQSlab0 < S::kPeSlab ? S::kQSlab0 : S::kPeSlab) - S::kHalfSlabs;
    q_copy<4 * S::kHalfSlabs, 4 * kSlabs>(smem_desc(smem + ring.half * S::kHalf, 16, 1024), tmem);
    commit(smem_u32(&sh.bars.empty[ring.half]));
    ring.next_half();
    ring.next_tile();
    for (int i = 0; i < tiles; ++i, ++it) {
      const uint32_t buf = it & 1u;
      const uint32_t d = tmem + kTmemS + 32u * buf;
      if (it >= 2 && !warp_wait(smem_u32(&sh.bars.s_empty[buf]), (it / 2 - 1) & 1u, ab, p.spins)) return false;
      if (!come()) return false;
      qk_rotary<OP>(q + 32u * S::kPeSlab, d_q + static_cast<uint64_t>(S::kQSlabs > 0 ? (S::kQSlabs - 1) * (kSlabBytes >> 4) : 0),
                    d_pe + ring.slot * (kSlabBytes >> 4), d);
      qk_tmem<OP>(q, d_half + ring.half * (S::kHalf >> 4), d, S::kHalfSlabs);
      ring.next_half();
      if (!come()) return false;
      const uint64_t k = d_half + ring.half * (S::kHalf >> 4);
      qk_tmem<OP>(q + 32u * S::kHalfSlabs, k, d, kSlabs);
      if (kSlabs < S::kHalfSlabs) qk_smem<OP>(d_q, k + kSlabs * (kSlabBytes >> 4), d, S::kHalfSlabs - kSlabs);
      commit(smem_u32(&sh.bars.s_full[buf]));
      ring.next_half();
      ring.next_tile();
    }
    commit(smem_u32(&sh.bars.q_empty));
  }
}

// Issues the sums' products of every tile.
template <int OP>
__device__ __forceinline__ bool issue_sums(const Params& p, Shared& sh, uint32_t smem, uint32_t tmem) {
  using S = Shape<OP>;
  volatile uint32_t* ab = &sh.abort_flag;
  const uint64_t d_p = smem_desc(smem + S::kPAt, 16, 1024), d_v = smem_desc(smem, kSlabBytes, 1024);
  uint32_t it = 0, segs = 0;
  Ring<OP> ring;
  while (true) {
    if (!segment_known(p, sh, segs)) return false;
    const Segment& x = sh.segments[segs % kSegments];
    const int tiles = uniform(x.k1 - x.k0);
    if (tiles == 0) return true;
    segment_done(sh, segs);
    ring.skip_tile();  // the q rows
    if (segs > 0 && !warp_wait(smem_u32(&sh.bars.o_empty), (segs - 1) & 1u, ab, p.spins)) return false;
    ++segs;
    for (int i = 0; i < tiles; ++i, ++it) {
      const uint32_t buf = it & 1u;
      if (!warp_wait(smem_u32(&sh.bars.p_full[buf]), (it / 2) & 1u, ab, p.spins)) return false;
      fence_async();  // the weights came by plain stores (and the rows may have)
      fence_after();
      const uint64_t w = d_p + (S::kPBufs > 1 ? buf * (S::kP >> 4) : 0u);
#pragma unroll 1
      for (uint32_t h = 0; h < 2; ++h) {
        pv_half<OP>(w, d_v + ring.half * (S::kHalf >> 4), tmem + 128u * h, i > 0 ? 1u : 0u);
        commit(smem_u32(&sh.bars.empty[ring.half]));
        ring.next_half();
      }
      commit(smem_u32(&sh.bars.pv_done[buf]));
      ring.next_tile();
    }
  }
}

// The softmax of WARPS warps.  A thread has one row (TMEM lane), and of a tile's
// scores half `half` of the keys, of that (8 warps) half `sub`; of the sums the
// same half of each 256 columns and half `sub` of the TMEM columns.
template <int OP, int WARPS>
__device__ __forceinline__ void softmax_role(const Params& p, Shared& sh, uint32_t sP, uint32_t tmem,
                                             float scale2) {
  constexpr int kN = 32 * 4 / WARPS;           // keys of a thread: 32 or 16
  constexpr int kParts = WARPS / 2;            // threads to a row
  const int warp = static_cast<int>(threadIdx.x) >> 5, lane = static_cast<int>(threadIdx.x) & 31;
  const int r = (warp & 1) * 32 + lane;
  const int half = (warp >> 1) & 1, sub = warp >> 2;
  const int part = half * (kParts / 2) + sub;  // keys part * kN ..
  // the warps that share rows with this one: their barriers, their threads
  const int bar_a = 1 + 2 * (warp & 1), bar_b = bar_a + 1;
  constexpr int kShare = 16 * WARPS;
  const uint32_t lanes = static_cast<uint32_t>(warp & 3) << 21;
  const bool negative = scale2 < 0.0f;  // then the scores change sign, and the scale
  scale2 = fabsf(scale2);
  volatile uint32_t* ab = &sh.abort_flag;
  uint32_t it = 0;
  Ring<OP> ring;
  bool good = true;   // no wait has run out in this warp
  bool left = false;  // the warps that share rows have left the walk together
  for (uint32_t segs = 0; good; ++segs) {
    good = segment_known(p, sh, segs);
    if (bar_or(bar_a, kShare, !good)) {  // the warps that share rows leave together
      good = false;
      break;
    }
    const Segment seg = sh.segments[segs % kSegments];
    if (seg.k0 == seg.k1) break;
    segment_done(sh, segs);
    constexpr float kMostOf = OP == kF8 ? kF8Most : kMost;
    const float lift = OP == kF8 ? f8_lift(seg.k1 - seg.k0) : 0.0f;
    float m = -INFINITY;      // the row's maximum when the reference last moved, in powers of two
    float ref = 0.0f;         // the reference
    float limit = -INFINITY;  // it moves when a score passes this
    float l = 0.0f;       // this thread's share of the denominator
    ring.skip_tile();     // the q rows
    for (int kt = seg.k0; kt < seg.k1; ++kt, ++it) {
      const uint32_t buf = it & 1u;
      // the flags first: they are there before the scores, and may have come by the copy engine
      good = warp_wait(smem_u32(&sh.bars.full[ring.half]), ring.lap & 1u, ab, p.spins) && good;
      uint32_t ok[kN / 4];
#pragma unroll
      for (int j = 0; j < kN / 16; ++j) {
        const uint4 f = ld_shared(smem_u32(&sh.valid[ring.slot][part * kN + 16 * j]));
        ok[4 * j] = f.x;
        ok[4 * j + 1] = f.y;
        ok[4 * j + 2] = f.z;
        ok[4 * j + 3] = f.w;
      }
      uint32_t all = ok[0];
#pragma unroll
      for (int j = 1; j < kN / 4; ++j) all &= ok[j];
      const bool whole = all == 0x01010101u;
      good = warp_wait(smem_u32(&sh.bars.s_full[buf]), (it / 2) & 1u, ab, p.spins) && good;
      fence_after();
      uint32_t v[kN];
      tmem_ld<kN>(tmem + kTmemS + 32u * buf + lanes + static_cast<uint32_t>(sub * kN), v);
      fence_before();
      __syncwarp();
      if (lane == 0) arrive(smem_u32(&sh.bars.s_empty[buf]));
      ring.skip_tile();
      if (negative) {
#pragma unroll
        for (int j = 0; j < kN; ++j) v[j] ^= 0x80000000u;
      }
      if (!whole) {
#pragma unroll
        for (int j = 0; j < kN; ++j) v[j] = (ok[j >> 2] >> (8 * (j & 3))) & 1u ? v[j] : 0xff800000u;
      }
      float t[kN / 4];
#pragma unroll
      for (int j = 0; j < kN / 4; ++j)
        t[j] = fmaxf(fmaxf(__uint_as_float(v[4 * j]), __uint_as_float(v[4 * j + 1])),
                     fmaxf(__uint_as_float(v[4 * j + 2]), __uint_as_float(v[4 * j + 3])));
#pragma unroll
      for (int n = kN / 8; n > 0; n /= 2)
#pragma unroll
        for (int j = 0; j < n; ++j) t[j] = fmaxf(t[j], t[j + n]);
      const float top = t[0] == -INFINITY ? -INFINITY : t[0] * scale2;  // scale2 >= 0: the largest score
      const bool first = kt == seg.k0;
      // One vote a tile: whether a row's reference must move, or a wait ran out
      // (then all the warps leave together).
      const bool moved = bar_or(bar_a, kShare, first || top > limit || !good);
      float factor = 1.0f;
      if (moved) {
        if (bar_or(bar_b, kShare, !good)) {
          good = false;
          left = true;
          break;
        }
        sh.xch[part][r] = top;
        bar_sync(bar_b, kShare);
        float next = m;
#pragma unroll
        for (int i = 0; i < kParts; ++i) next = fmaxf(next, sh.xch[i][r]);
        if (next > m) {
          float next_ref = next;
          limit = next + kRescale;
          if constexpr (OP == kF8) {
            const bool large = fabsf(next) >= kF8Large;
            next_ref = large ? next : next - lift;
            limit = large ? next : next + (kF8Top - lift);
          }
          if (fabsf(next) >= kMostOf) next_ref = INFINITY;
          if (!first) factor = m <= -kMostOf ? 0.0f : exp2_fast(ref - next_ref);
          m = next;
          ref = next_ref;
        }
        l *= factor;
      }
      float sum[4] = {0.0f, 0.0f, 0.0f, 0.0f};
      uint32_t w[kN / 2], mid[kN / 4], lo[kN / 4];
#pragma unroll
      for (int j = 0; j < kN / 2; ++j) {
        float a = exp2_fast(fmaf(__uint_as_float(v[2 * j]), scale2, -ref));
        float b = exp2_fast(fmaf(__uint_as_float(v[2 * j + 1]), scale2, -ref));
        if (!whole) {  // (a zero scale makes no weight of a masked score)
          a = (ok[j >> 1] >> (16 * (j & 1))) & 1u ? a : 0.0f;
          b = (ok[j >> 1] >> (16 * (j & 1) + 8)) & 1u ? b : 0.0f;
        }
        sum[j & 3] += a + b;
        if constexpr (OP == kF8) {
          uint32_t h, x;
          asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(h) : "f"(b), "f"(a));
          // each remainder is exact in fp16: it has the bits the term left over
          const uint32_t t0 = near_e5m2(h), r0 = sub_f16x2(h, t0);
          const uint32_t t1 = near_e5m2(r0), r1 = sub_f16x2(r0, t1);
          x = near_e5m2(r1);
          if ((j & 1) == 0) {
            w[j >> 1] = t0;
            mid[j >> 1] = t1;
            lo[j >> 1] = x;
          } else {  // the upper bytes of four
            w[j >> 1] = __byte_perm(w[j >> 1], t0, 0x7531);
            mid[j >> 1] = __byte_perm(mid[j >> 1], t1, 0x7531);
            lo[j >> 1] = __byte_perm(lo[j >> 1], x, 0x7531);
          }
        } else {
          w[j] = pack_bf16x2(a, b);
        }
      }
      l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
      // the weights that were in this buffer have been read
      constexpr uint32_t kBack = Shape<OP>::kPBufs;
      if (it >= kBack) good = warp_wait(smem_u32(&sh.bars.pv_done[(it - kBack) & 1u]), ((it - kBack) / 2) & 1u, ab, p.spins);
      if (moved && !first) {
        // the previous tile's products are in the sums (all threads move or none)
        if (kBack > 1) good = warp_wait(smem_u32(&sh.bars.pv_done[(it - 1) & 1u]), ((it - 1) / 2) & 1u, ab, p.spins) && good;
        fence_after();
#pragma unroll 1
        for (uint32_t c = 0; c < 1024u / WARPS; c += 32) {
          uint32_t o[32];
          const uint32_t at = tmem + lanes + static_cast<uint32_t>(sub) * 128u + c;
          tmem_ld<32>(at, o);
#pragma unroll
          for (int j = 0; j < 32; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * factor);
          tmem_st32(at, o);
        }
        asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
      }
      const uint32_t dst = sP + (kBack > 1 ? buf * Shape<OP>::kP : 0u);
      if constexpr (OP == kF8) {
#pragma unroll
        for (int j = 0; j < kN / 16; ++j) {
          const int c = part * (kN / 16) + j;
          st_shared(piece_addr(dst, 0, r, c), make_uint4(w[4 * j], w[4 * j + 1], w[4 * j + 2], w[4 * j + 3]));
          st_shared(piece_addr(dst, 0, r, 4 + c), make_uint4(mid[4 * j], mid[4 * j + 1], mid[4 * j + 2], mid[4 * j + 3]));
          st_shared(piece_addr(dst, 1, r, c), make_uint4(lo[4 * j], lo[4 * j + 1], lo[4 * j + 2], lo[4 * j + 3]));
        }
      } else {
#pragma unroll
        for (int j = 0; j < kN / 8; ++j)
          st_shared(piece_addr(dst, 0, r, part * (kN / 8) + j), make_uint4(w[4 * j], w[4 * j + 1], w[4 * j + 2], w[4 * j + 3]));
      }
      fence_before();
      __syncwarp();
      if (lane == 0) arrive(smem_u32(&sh.bars.p_full[buf]));
    }
    if (left) break;
    // ---- the segment's result
    good = warp_wait(smem_u32(&sh.bars.pv_done[(it - 1) & 1u]), ((it - 1) / 2) & 1u, ab, p.spins) && good;
    if (bar_or(bar_a, kShare, !good)) {
      good = false;
      break;
    }
    fence_after();
    const bool keep = r < seg.rows;
    uint4* out = reinterpret_cast<uint4*>(seg.part) + r;
#pragma unroll 1
    for (int i = 0; i < 1024 / WARPS; i += 32) {
      const int c = sub * 128 + i;
      uint32_t v[32];
      tmem_ld<32>(tmem + lanes + static_cast<uint32_t>(c), v);
      // TMEM column c of this lane: output column (c / 128) 256 + half 128 + c % 128
      const int chunk0 = ((c >> 7) * 256 + half * 128 + (c & 127)) / 4;
      if (keep) {
#pragma unroll
        for (int j = 0; j < 8; ++j)
          __stcg(out + static_cast<int64_t>(chunk0 + j) * seg.part_rows,
                 make_uint4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]));
      }
    }
    fence_before();
    __syncwarp();
    if (lane == 0) arrive(smem_u32(&sh.bars.o_empty));
    sh.xch[part][r] = l;
    bar_sync(bar_b, kShare);
    if (part == 0 && keep) {
      float* stat = reinterpret_cast<float*>(seg.part + static_cast<int64_t>(seg.part_rows) * kChunks * 16);
      float den = l;
#pragma unroll
      for (int i = 1; i < kParts; ++i) den += sh.xch[i][r];
      __stcg(stat + r, m <= -kMostOf ? m : ref);
      __stcg(stat + seg.part_rows + r, den);
    }
    bar_sync(bar_b, kShare);
  }
  if (!good && *ab == 0u && lane == 0) {
    *ab = 1u;
    report(p.status, MLA_STATUS_TIMEOUT);
  }
}

// Adds up the units' tiles: this CTA's run of tiles and the unit it starts in.
// Thread i takes the units [i n, (i + 1) n).
__device__ __forceinline__ Cursor plan_run(const Params& p, Shared& sh) {
  const int64_t units = static_cast<int64_t>(p.G) + p.T;
  const int64_t per = (units + kThreads - 1) / kThreads;
  const int64_t u0 = static_cast<int64_t>(threadIdx.x) * per;
  const int64_t u1 = u0 + per < units ? u0 + per : units;
  const int lane = static_cast<int>(threadIdx.x) & 31, warp = static_cast<int>(threadIdx.x) >> 5;
  int64_t sum = 0;
  bool any_bad = false;
  Unit last{};  // the thread's last unit: its only one as a rule, and then not looked up again
  for (int64_t u = u0; u < u1; ++u) {
    bool bad;
    last = unit_at(p, u, bad);
    sum += last.cost();
    any_bad = any_bad || bad;
  }
  if (any_bad && blockIdx.x == 0) report(p.status, MLA_STATUS_LEN_RANGE);
  int64_t incl = sum;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int64_t o = __shfl_up_sync(0xffffffffu, incl, d);
    if (lane >= d) incl += o;
  }
  if (lane == 31) sh.warp_sum[warp] = incl;
  __syncthreads();
  int64_t before = 0, total = 0;
  for (int w = 0; w < kThreads / 32; ++w) {
    if (w < warp) before += sh.warp_sum[w];
    total += sh.warp_sum[w];
  }
  // at least a tile's cost, so that every CTA between a row tile's first and last has one of its key tiles
  const int64_t least = p.tile_cost > p.prefix_cost ? p.tile_cost : p.prefix_cost;
  const int64_t even = quotient(total + p.ctas - 1, p.ctas), each = even > least ? even : least;
  Cursor c;
  c.pos = each * blockIdx.x;
  c.end = c.pos + each < total ? c.pos + each : total;
  int64_t base = before + incl - sum;
  if (blockIdx.x == 0 && threadIdx.x == 0) p.plan[0] = each;
  const bool mine = c.pos >= base && c.pos < base + sum;
  if (mine || blockIdx.x == 0) {
    for (int64_t u = u0; u < u1; ++u) {
      bool bad;
      const Unit x = u + 1 == u1 ? last : unit_at(p, u, bad);
      if (blockIdx.x == 0) p.plan[1 + u] = base;
      if (c.pos >= base && c.pos < base + x.cost()) {
        sh.first_unit = u;
        sh.first_base = base;
        sh.unit = x;
      }
      base += x.cost();
    }
  }
  __syncthreads();
  c.u = sh.first_unit;
  c.base = sh.first_base;
  c.known = &sh.unit;
  c.window = -64;  // none
  c.window_len = 0;
  return c;
}

template <int FMT, int OP>
__global__ void __launch_bounds__(kThreads, 1)
    attend_kernel(const __grid_constant__ CUtensorMap slab_map, const __grid_constant__ CUtensorMap half_map,
                  const Params p) {
  using S = Shape<OP>;
  using R = Roles<FMT, OP>;
  extern __shared__ uint8_t dsmem[];
  __shared__ Shared sh;
  const int warp = uniform(static_cast<int>(threadIdx.x) >> 5);
  const uint32_t smem = (smem_u32(dsmem) + 1023u) & ~1023u;
  if (warp == R::kScores) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&sh.tmem)),
                 "r"(kTmemCols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  if (threadIdx.x == 0) {
    sh.abort_flag = 0u;
    sh.never = 0u;
    sh.first_unit = 0;
    sh.first_base = 0;
    auto init = [](uint64_t* b, uint32_t n) {
      asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(smem_u32(b)), "r"(n) : "memory");
    };
    for (int i = 0; i < S::kHalves; ++i) {
      init(&sh.bars.full[i], kArrivals * R::kLoad);
      init(&sh.bars.empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      init(&sh.bars.s_full[i], 1);
      init(&sh.bars.s_empty[i], R::kSoft);
      init(&sh.bars.p_full[i], R::kSoft);
      init(&sh.bars.pv_done[i], 1);
    }
    init(&sh.bars.q_empty, 1);
    init(&sh.bars.o_empty, R::kSoft);
    for (uint32_t i = 0; i < kSegments; ++i) {
      init(&sh.bars.seg_full[i], 1);
      init(&sh.bars.seg_empty[i], R::kTakers);
    }
    init(&sh.bars.drained[0], 1);
    init(&sh.bars.drained[1], 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (threadIdx.x == 32 && p.box_rows > 0) {
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&slab_map)) : "memory");
    if (p.box_rows == kKeys) asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&half_map)) : "memory");
  }
  pdl_wait();     // the lengths, q and the cache rows may come from the upstream kernel
  pdl_trigger();  // the joining kernel waits for this grid's end itself
  fence_before();
  __syncthreads();
  fence_after();
  const uint32_t tmem = static_cast<uint32_t>(uniform(static_cast<int>(sh.tmem)));
  const Cursor cur = plan_run(p, sh);
  if (uniform(cur.pos < cur.end ? 1 : 0) != 0) {  // a branch that the compiler sees is uniform
    if (warp < R::kSoft) {
      float scale2 = p.sm_scale * 1.4426950408889634f;  // powers of two: log2(e)
      if (p.q_fp8) scale2 *= __ldcg(p.q_scale);
      if (FMT == MLA_CACHE_E4M3) scale2 *= __ldcg(p.kv_scale);
      softmax_role<OP, R::kSoft>(p, sh, smem + S::kPAt, tmem, scale2);
    } else if (warp < R::kScores) {
      asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(R::kLoadRegs));
      loader<FMT, OP>(p, Maps{&slab_map, &half_map}, sh, smem);
    } else {
      asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kIssueRegs));
      if (warp == R::kScores) {
        if (!issue_scores<OP>(p, sh, smem, tmem)) give_up(p, &sh.abort_flag);
        drain(&sh.bars.drained[0], &sh.never);
      } else if (warp == R::kSums) {
        if (!issue_sums<OP>(p, sh, smem, tmem)) give_up(p, &sh.abort_flag);
        drain(&sh.bars.drained[1], &sh.never);
      } else if (warp == R::kFinds) {
        if (!find_segments(p, cur, sh)) give_up(p, &sh.abort_flag);
      }
    }
  }
  fence_before();
  __syncthreads();
  if (threadIdx.x == 0) p.gave_up[blockIdx.x] = sh.abort_flag;
  if (warp == R::kScores) {
    fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTmemCols) : "memory");
  }
}

// ---- decoded prefix tiles -------------------------------------------------------------
//
// A prefix of a group with many rows is read by many CTAs, 64 rows at a time.
// It is decoded once, into tiles as they lie in shared memory (swizzled 16-bit
// values, zeros where there is no key, and a flag for each key); the attention
// kernel then fetches a tile half with two or three bulk copies.  One block a
// tile; blocks behind a prefix's end leave.
template <int FMT, int OP>
__global__ void __launch_bounds__(256) image_kernel(const Params p) {
  pdl_wait();
  const int64_t g = blockIdx.y;
  bool bad;
  const Unit x = unit_at(p, g, bad);
  const int64_t kt = blockIdx.x;
  if (kt < x.key_tiles() && x.rows > 0) {
    const int warp = static_cast<int>(threadIdx.x) >> 5, lane = static_cast<int>(threadIdx.x) & 31;
    const int row0 = 8 * warp;
    uint8_t* dst = p.image + (g * p.image_tiles + kt) * Shape<OP>::kImage;
    KeyAt at;
    bool bad_page = false;
    at.fetch(p, x.table, static_cast<int32_t>(x.len), static_cast<int32_t>(kt), row0 + lane, lane < 8);
    const uint8_t* mine = at.address(p, row_bytes(FMT), bad_page);
    auto put = [&](int s, int r, int c, const uint4& v) {
      *reinterpret_cast<uint4*>(dst + piece_addr(0, s, r, c)) = v;
    };
    if constexpr (Roles<FMT, OP>::kDecode) {
      Raw<FMT> raw;
      load_rows<FMT>(raw, mine, lane);
      store_half<FMT>(raw, 0, row0, lane, put);
      store_half<FMT>(raw, 1, row0, lane, put);
    } else {
      const Pieces<OP, 8> pieces(mine, lane);
      auto copy = [&](int s, int r, int c, const uint8_t* src) {
        put(s, row0 + r, c, src != nullptr ? __ldcg(reinterpret_cast<const uint4*>(src)) : make_uint4(0, 0, 0, 0));
      };
      pieces.values(0, lane, copy);
      pieces.values(1, lane, copy);
      pieces.rotary(lane, copy);
    }
    if (lane < 8) dst[Shape<OP>::kTile + row0 + lane] = mine != nullptr ? 1 : 0;
    if (bad_page) report(p.status, MLA_STATUS_SLOT_RANGE);
  }
  pdl_trigger();
}

// ---- joining a row's segments ----------------------------------------------------------
//
// out = sum_i 2^(m_i - M) O_i / sum_i 2^(m_i - M) l_i.  A block takes one token,
// 16 of its heads and a slice of the columns; thread (row, worker), CH chunks of
// four columns at a time.  A thread's first sums are loaded before the weights
// they need are known, so the chain is plan, statistics and sums: few trips to
// memory, whatever n is (5 us: 1.9 for the plan, 1.3 for the statistics, the rest
// for weights and sums).  With few tokens the columns are cut into more slices and
// a row's segments shared out to classes of workers; all blocks run at once where
// they can (1024 rows of 12 segments: in two waves 12 us, in one 6).

constexpr int kJoinRows = 16, kJoinWorkers = 16, kJoinThreads = kJoinRows * kJoinWorkers;

template <int CH>
__global__ void __launch_bounds__(kJoinThreads, 3) join_kernel(const Params p, int slices) {
  constexpr int kAhead = 8 / CH;      // segments loaded ahead
  extern __shared__ float weights[];  // [segments][16]
  __shared__ float red[2][kJoinWorkers][kJoinRows];
  __shared__ float4 sums[kJoinWorkers][kJoinRows];
  pdl_wait();
  const int row = static_cast<int>(threadIdx.x) % kJoinRows, wk = static_cast<int>(threadIdx.x) / kJoinRows;
  const int head_blocks = (p.H + kJoinRows - 1) / kJoinRows;
  int64_t b = blockIdx.x;
  const int slice = static_cast<int>(b % slices);
  b /= slices;
  const int h = static_cast<int>(b % head_blocks) * kJoinRows + row;
  const int64_t t = b / head_blocks;
  const bool live = h < p.H;

  // the row's segments: n1 of its group's prefix, n2 of its own keys
  const int64_t each = __ldcg(p.plan);
  int n1 = 0, n2 = 0;
  const uint8_t* part1 = p.prefix_part;  // its first segment of either kind, and the row in it
  const uint8_t* part2 = p.own_part;
  int row1 = 0;
  const int row2 = h % kRowsTile;
  int cta1 = 0, cta2 = 0;  // the CTA that has its first segment of either kind; the others follow
  if (live) {
    int64_t g = -1;
    if (p.G > 0 && p.group_offsets == nullptr) {
      g = 0;
    } else if (p.G > 0) {
      int64_t lo = 0, hi = p.G;  // the last group that starts at or before t
      while (lo < hi) {
        const int64_t mid = (lo + hi) / 2;
        if (static_cast<int64_t>(__ldcg(p.group_offsets + mid)) <= t) lo = mid + 1; else hi = mid;
      }
      g = lo - 1;
    }
    // all that the numbers of segments need is fetched before any is worked out
    bool bad;
    const Unit own = unit_at(p, p.G + t, bad);
    const int64_t own_at = __ldcg(p.plan + 1 + p.G + t);
    Unit x = own;
    int64_t at = 0;
    if (g >= 0) {
      x = unit_at(p, g, bad);
      at = __ldcg(p.plan + 1 + g);
    }
    // CTAs c0 .. c1 have the row's key tiles
    auto span = [&](const Unit& x, int64_t at, int64_t tile, int rows, const uint8_t*& part, int& cta, int& n) {
      const int64_t per = x.row_cost();
      if (per == 0) return;
      const int64_t f = at + tile * per;
      // (cut, lest lengths that change under the call lead out of the workspace)
      const int64_t c0 = cut(quotient(f + x.start_cost, each), 0, p.ctas - 1);
      const int64_t c1 = cut(quotient(f + per - x.tile_cost, each), c0, p.ctas - 1);
      part += (c0 + x.part0 + tile) * part_bytes(rows);
      cta = static_cast<int>(c0);
      n = static_cast<int>(c1 - c0) + 1;
    };
    span(own, own_at, h / kRowsTile, p.own_rows, part2, cta2, n2);
    const int64_t i = t * p.H + h - x.rows0;
    if (g >= 0 && i >= 0 && i < x.rows) {
      span(x, at, i / kRowsTile, kRowsTile, part1, cta1, n1);
      row1 = static_cast<int>(i % kRowsTile);
    }
  }
  const int n = n1 + n2;
  // segment i, its rows and the row in it
  auto part_of = [&](int i, int& rows, int& r) -> const uint8_t* {
    const bool pre = i < n1;
    rows = pre ? kRowsTile : p.own_rows;
    r = pre ? row1 : row2;
    return pre ? part1 + i * part_bytes(kRowsTile) : part2 + (i - n1) * part_bytes(p.own_rows);
  };
  auto stats_of = [&](int i, float& m, float& l) {
    int rows, r;
    const uint8_t* part = part_of(i, rows, r);
    const float* s = reinterpret_cast<const float*>(part + static_cast<int64_t>(rows) * kChunks * 16) + r;
    m = __ldcg(s);
    l = __ldcg(s + rows);
  };

  // `per` chunks in this slice; workers: cw columns of chunks, 16 / cw segment classes
  const int per = kChunks / slices;
  const int cw = per / CH < kJoinWorkers ? per / CH : kJoinWorkers;
  const int classes = kJoinWorkers / cw;
  const int cls = wk / cw;
  const int chunk0 = slice * per + wk % cw;
  auto load = [&](int i, int c0, float4 (&o)[CH]) {
    int rows, r;
    const float4* part = reinterpret_cast<const float4*>(part_of(i, rows, r)) + r;
#pragma unroll
    for (int k = 0; k < CH; ++k) o[k] = __ldcg(part + (chunk0 + c0 + k * cw) * rows);
  };
  float4 ahead[kAhead][CH];
#pragma unroll
  for (int j = 0; j < kAhead; ++j) {
    const int i = cls + j * classes;
    if (i < n) load(i, 0, ahead[j]);
  }

  // ---- weights
  float m0 = -INFINITY, l0 = 0.0f;
  if (wk < n) stats_of(wk, m0, l0);
  for (int i = wk; i < n; i += kJoinWorkers)  // what a CTA left that gave up may be an earlier call's: the row is NaN
    if (__ldcg(p.gave_up + (i < n1 ? cta1 + i : cta2 + i - n1)) != 0u) l0 = __uint_as_float(0x7fffffffu);
  float top = m0;
  for (int i = wk + kJoinWorkers; i < n; i += kJoinWorkers) {
    float m, l;
    stats_of(i, m, l);
    top = fmaxf(top, m);
  }
  red[0][wk][row] = top;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kJoinWorkers; ++i) top = fmaxf(top, red[0][i][row]);
  const float ref = top == -INFINITY ? 0.0f : top;
  float den = 0.0f;
  for (int i = wk; i < n; i += kJoinWorkers) {
    float m = m0, l = l0;
    if (i != wk) stats_of(i, m, l);
    const float w = exp2f(m - ref);
    weights[i * kJoinRows + row] = w;
    den += w * l;
  }
  red[1][wk][row] = den;
  __syncthreads();
  den = 0.0f;
#pragma unroll
  for (int i = 0; i < kJoinWorkers; ++i) den += red[1][i][row];
  if (den == 0.0f && top > -INFINITY) den = __uint_as_float(0x7fffffffu);
  const bool some = den > 0.0f || den != den;
  if (live && slice == 0 && wk == 0 && p.lse != nullptr)
    p.lse[t * p.H + h] = some ? (ref + log2f(den)) * 0.6931471805599453f : -INFINITY;
  float mul = some ? 1.0f / den : 0.0f;
  if (p.kv_scale != nullptr) mul *= __ldcg(p.kv_scale);

  // ---- sums
  for (int c0 = 0; c0 < per; c0 += cw * CH) {
    float4 acc[CH];
#pragma unroll
    for (int k = 0; k < CH; ++k) acc[k] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    auto add = [&](int i, const float4 (&o)[CH]) {
      const float w = weights[i * kJoinRows + row];
#pragma unroll
      for (int k = 0; k < CH; ++k) {
        acc[k].x += w * o[k].x;
        acc[k].y += w * o[k].y;
        acc[k].z += w * o[k].z;
        acc[k].w += w * o[k].w;
      }
    };
    for (int i = cls; i < n; i += kAhead * classes) {
      if (c0 > 0 || i != cls) {
#pragma unroll
        for (int j = 0; j < kAhead; ++j)
          if (i + j * classes < n) load(i + j * classes, c0, ahead[j]);
      }
#pragma unroll
      for (int j = 0; j < kAhead; ++j)
        if (i + j * classes < n) add(i + j * classes, ahead[j]);
    }
    if (CH == 1 && classes > 1) {
      __syncthreads();
      sums[wk][row] = acc[0];
      __syncthreads();
      if (cls == 0) {
        for (int k = 1; k < classes; ++k) {
          const float4 o = sums[k * cw + wk % cw][row];
          acc[0].x += o.x;
          acc[0].y += o.y;
          acc[0].z += o.z;
          acc[0].w += o.w;
        }
      }
    }
    if (live && cls == 0) {
#pragma unroll
      for (int k = 0; k < CH; ++k) {
        uint2 o = make_uint2(pack_bf16x2(acc[k].x * mul, acc[k].y * mul), pack_bf16x2(acc[k].z * mul, acc[k].w * mul));
        if (n == 0) o = make_uint2(0, 0);
        *reinterpret_cast<uint2*>(p.out + (t * p.H + h) * kDv + 4 * (chunk0 + c0 + k * cw)) = o;
      }
    }
  }
  pdl_trigger();
}

// ---- host ------------------------------------------------------------------------------

// A prefix is decoded once, into the workspace, when its rows need decoding (or
// pages are too small for tensor copies), its group has at least kImageRows rows
// on average and the images fit kImageLimit; else its tiles are read from the
// cache.  Measured with images and without: 128 rows behind 8 K mx keys 30 and 31
// us, behind 32 K 54 and 47; 256 rows 33 and 37, 60 and 68; 1024 rows 45 and 69,
// 107 and 189.
constexpr int64_t kImageRows = 4 * kRowsTile;
constexpr int kLeastBox = 8;  // rows of a tensor copy at least: the swizzle's period
constexpr int64_t kImageLimit = INT64_C(1) << 31;

struct Layout {
  int64_t gave_up, prefix_part, own_part, image, image_tiles, bytes;
};

// `image_bytes`: of a tile's image, 0 where a call makes none.  (How many tiles may
// be imaged goes by the largest images, whatever a call's are, so that a workspace
// for those is enough for every call.)
constexpr int32_t kMostImageBytes = static_cast<int32_t>(Shape<kBf16>::kImage);
Layout layout_of(int64_t T, int64_t H, int64_t G, int64_t prefix_keys, int64_t ctas, int64_t image_bytes) {
  auto up = [](int64_t v) { return (v + 255) / 256 * 256; };
  Layout l;
  l.gave_up = 8 * (1 + G + T);
  l.prefix_part = up(l.gave_up + 4 * ctas);
  const int64_t prefix_parts = G > 0 ? T * H / kRowsTile + G + 1 + ctas : 0;
  l.own_part = up(l.prefix_part + prefix_parts * part_bytes(kRowsTile));
  const int64_t own_parts = T * ((H + kRowsTile - 1) / kRowsTile) + ctas;
  l.image = up(l.own_part + own_parts * part_bytes(static_cast<int>(H < kRowsTile ? H : kRowsTile)));
  l.image_tiles = (prefix_keys + kKeys - 1) / kKeys;
  if (image_bytes == 0 || G < 1 || G > 65535 || T * H < kImageRows * G || l.image_tiles > kImageLimit / kMostImageBytes / G)
    l.image_tiles = 0;
  l.bytes = up(l.image + G * l.image_tiles * image_bytes);
  return l;
}

// The kernels of a call: by format, and with both q and cache in e4m3 on the codes themselves.
struct Kernels {
  const void* attend;
  const void* image;
  uint32_t smem;
  int32_t image_bytes, tile_cost, prefix_cost;
};

template <int FMT, int OP>
Kernels kernels_of(int32_t tile_cost) {
  return Kernels{reinterpret_cast<const void*>(&attend_kernel<FMT, OP>),
                 reinterpret_cast<const void*>(&image_kernel<FMT, OP>), Shape<OP>::kSmem,
                 static_cast<int32_t>(Shape<OP>::kImage), tile_cost, OP == kF8 ? kCostF8 : kCostPrefix};
}

const Kernels kKernels[4] = {kernels_of<MLA_CACHE_BF16, kBf16>(kCostRows), kernels_of<MLA_CACHE_E4M3, kBf16>(kCostE4m3),
                             kernels_of<MLA_CACHE_MX, kBf16>(kCostMx), kernels_of<MLA_CACHE_E4M3, kF8>(kCostF8)};

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) % n) == 0; }

std::atomic<bool> g_smem_ready[kMaxDevices][4];
std::atomic<uint32_t> g_spins{kWaitSpins};  // (mla_harness_attend_spins)

PFN_cuTensorMapEncodeTiled_v12000 tensor_map_encoder() {
  static std::atomic<PFN_cuTensorMapEncodeTiled_v12000> known{nullptr};
  PFN_cuTensorMapEncodeTiled_v12000 fn = known.load(std::memory_order_acquire);
  if (fn == nullptr) {
    void* ptr = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &ptr, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess) {
      fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(ptr);
      known.store(fn, std::memory_order_release);
    } else {
      (void)cudaGetLastError();
    }
  }
  return fn;
}

// The largest power of two up to 64 that divides a block's rows, so that a box
// of that many rows, at a multiple of it in the sequence, lies in one page.
int box_rows_of(int64_t block_size) {
  int r = kKeys;
  while (block_size % r != 0) r /= 2;
  return r >= kLeastBox ? r : 0;
}

// The kernels a call takes, and whether they fetch whole tiles by tensor copies: rows of
// 16-bit values or codes as they are, in pages of a multiple of eight rows.
int kernels_at(int32_t format, bool q8) { return format == MLA_CACHE_E4M3 && q8 ? 3 : format; }
bool needs_decoding(int k) { return k == MLA_CACHE_MX || k == MLA_CACHE_E4M3; }
bool by_tensor_copies(int k, int64_t block_size, int64_t num_blocks) {
  const int64_t cache_rows = num_blocks * block_size;
  return !needs_decoding(k) && box_rows_of(block_size) > 0 && cache_rows > 0 && cache_rows < INT_MAX;
}
int64_t image_bytes_of(int k, int64_t block_size, int64_t num_blocks) {
  return by_tensor_copies(k, block_size, num_blocks) ? 0 : kKernels[k].image_bytes;
}

bool cache_ok(int32_t format, int64_t block_size, int64_t num_blocks) {
  return format >= MLA_CACHE_BF16 && format <= MLA_CACHE_MX && block_size >= 1 && block_size <= INT_MAX && num_blocks >= 0 &&
         num_blocks <= (INT64_C(1) << 50) / block_size;
}

bool sizes_ok(int64_t T, int64_t H, int64_t G) {
  return T >= 0 && H >= 1 && H <= 65535 && T <= (static_cast<int64_t>(INT_MAX) - kRowsTile) / H && G >= 0 && G <= T;
}

mla_status launch(const void* fn, dim3 grid, int threads, size_t smem, bool pdl, mla_stream_t stream, void** args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(static_cast<unsigned>(threads), 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = reinterpret_cast<cudaStream_t>(stream);
  cudaLaunchAttribute attr[1];
  if (pdl) {
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
  }
  const cudaError_t e = cudaLaunchKernelExC(&cfg, fn, args);
  return e == cudaSuccess ? MLA_OK : cuda_failure(e);
}

}  // namespace attend
}  // namespace mla

extern "C" {

void mla_harness_attend_spins(int64_t spins) {
  using namespace mla::attend;
  g_spins.store(spins < 0 || spins > kWaitSpins ? kWaitSpins : static_cast<uint32_t>(spins), std::memory_order_relaxed);
}

mla_status mla_prefix_attend_workspace(int64_t T, int64_t H, int64_t G, int64_t prefix_keys, int32_t sm_count,
                                       int64_t* bytes) {
  using namespace mla::attend;
  if (bytes == nullptr || !sizes_ok(T, H, G) || prefix_keys < 0 || prefix_keys > (INT64_C(1) << 62))
    return MLA_ERR_INVALID_ARG;
  if (sm_count <= 0) {
    const mla_status s = mla::current_device(nullptr, &sm_count);
    if (s != MLA_OK) return s;
  }
  *bytes = layout_of(T, H, G, prefix_keys, sm_count, kMostImageBytes).bytes;
  return MLA_OK;
}

mla_status mla_prefix_attend_workspace_for(int64_t T, int64_t H, int64_t G, int64_t prefix_keys, int32_t format, uint32_t flags,
                                           int64_t block_size, int64_t num_blocks, int32_t sm_count, int64_t* bytes) {
  using namespace mla::attend;
  if ((flags & ~(MLA_FLAG_Q_FP8 | MLA_FLAG_PDL)) != 0 || format < MLA_CACHE_BF16 || format > MLA_CACHE_MX)
    return MLA_ERR_UNSUPPORTED;
  if (bytes == nullptr || !sizes_ok(T, H, G) || prefix_keys < 0 || prefix_keys > (INT64_C(1) << 62) ||
      !cache_ok(format, block_size, num_blocks))
    return MLA_ERR_INVALID_ARG;
  if (sm_count <= 0) {
    const mla_status s = mla::current_device(nullptr, &sm_count);
    if (s != MLA_OK) return s;
  }
  const int k = kernels_at(format, (flags & MLA_FLAG_Q_FP8) != 0);
  *bytes = layout_of(T, H, G, prefix_keys, sm_count, image_bytes_of(k, block_size, num_blocks)).bytes;
  return MLA_OK;
}

mla_status mla_prefix_attend_launch(
    const void* q, int64_t q_stride_t, int64_t q_stride_h, const float* q_scale,
    const void* cache, int32_t format, int64_t block_size, int64_t num_blocks, const float* kv_scale,
    const int32_t* prefix_table, int64_t prefix_stride, int64_t prefix_cols,
    const int32_t* prefix_lens, const int32_t* group_offsets, int64_t G,
    const int32_t* block_table, int64_t table_stride, int64_t table_cols, const int32_t* seq_lens,
    int64_t T, int64_t H, float sm_scale, uint32_t flags,
    void* out, float* lse, void* workspace, int64_t workspace_bytes, int32_t* status, mla_stream_t stream) {
  using namespace mla::attend;
  if ((flags & ~(MLA_FLAG_Q_FP8 | MLA_FLAG_PDL)) != 0) return MLA_ERR_UNSUPPORTED;
  if (format < MLA_CACHE_BF16 || format > MLA_CACHE_MX) return MLA_ERR_UNSUPPORTED;
  if (!sizes_ok(T, H, G) || !cache_ok(format, block_size, num_blocks) || table_cols < 0 || table_cols > INT_MAX ||
      table_stride < 0 || prefix_cols < 0 || prefix_cols > INT_MAX || prefix_stride < 0)
    return MLA_ERR_INVALID_ARG;
  if (!std::isfinite(sm_scale)) return MLA_ERR_INVALID_ARG;
  if (T == 0) return MLA_OK;
  const bool q8 = (flags & MLA_FLAG_Q_FP8) != 0;
  if (q == nullptr || (cache == nullptr && num_blocks > 0) || out == nullptr || workspace == nullptr) return MLA_ERR_INVALID_ARG;
  if ((q8 && q_scale == nullptr) || (format == MLA_CACHE_E4M3 && kv_scale == nullptr)) return MLA_ERR_INVALID_ARG;
  if (G > 0 && (prefix_table == nullptr || prefix_lens == nullptr || prefix_cols < 1)) return MLA_ERR_INVALID_ARG;
  if (G > 1 && group_offsets == nullptr) return MLA_ERR_INVALID_ARG;
  if (table_cols > 0 && (block_table == nullptr || seq_lens == nullptr)) return MLA_ERR_INVALID_ARG;
  if (q_stride_t < 0 || q_stride_h < 0) return MLA_ERR_INVALID_ARG;
  const int64_t unit = q8 ? 16 : 8;
  if (!aligned(q, 16) || !aligned(cache, 16) || !aligned(out, 16) || !aligned(workspace, 256) ||
      (T > 1 && q_stride_t % unit != 0) || (H > 1 && q_stride_h % unit != 0))
    return MLA_ERR_ALIGNMENT;
  if (!aligned(q_scale, 4) || !aligned(kv_scale, 4) || !aligned(prefix_table, 4) || !aligned(prefix_lens, 4) ||
      !aligned(group_offsets, 4) || !aligned(block_table, 4) || !aligned(seq_lens, 4) || !aligned(lse, 4) ||
      !aligned(status, 4))
    return MLA_ERR_ALIGNMENT;

  int dev = 0;
  int32_t sms = 0;
  mla_status s = mla::current_device(&dev, &sms);
  if (s != MLA_OK) return s;
  const int k = kernels_at(format, q8);
  const Layout lay = layout_of(T, H, G, prefix_cols * block_size, sms, image_bytes_of(k, block_size, num_blocks));
  if (workspace_bytes < lay.bytes) return MLA_ERR_INVALID_ARG;

  Params p;
  const int64_t esz = q8 ? 1 : 2;
  p.q = static_cast<const uint8_t*>(q);
  p.q_st = q_stride_t * esz;
  p.q_sh = q_stride_h * esz;
  p.q_scale = q8 ? q_scale : nullptr;
  p.cache = static_cast<const uint8_t*>(cache);
  p.kv_scale = format == MLA_CACHE_E4M3 ? kv_scale : nullptr;
  p.cache_blocks = num_blocks;
  p.block_size = static_cast<int32_t>(block_size);
  p.prefix_table = prefix_table;
  p.prefix_stride = prefix_stride;
  p.prefix_keys = prefix_cols * block_size;
  p.prefix_lens = prefix_lens;
  p.group_offsets = group_offsets;
  p.block_table = block_table;
  p.table_stride = table_stride;
  p.table_keys = table_cols * block_size;
  p.seq_lens = seq_lens;
  p.T = static_cast<int32_t>(T);
  p.H = static_cast<int32_t>(H);
  p.G = static_cast<int32_t>(G);
  p.q_fp8 = q8 ? 1 : 0;
  p.sm_scale = sm_scale;
  p.out = static_cast<uint16_t*>(out);
  p.lse = lse;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  p.plan = reinterpret_cast<int64_t*>(ws);
  p.gave_up = reinterpret_cast<uint32_t*>(ws + lay.gave_up);
  p.image = lay.image_tiles > 0 ? ws + lay.image : nullptr;
  p.image_tiles = lay.image_tiles;
  p.prefix_part = ws + lay.prefix_part;
  p.own_part = ws + lay.own_part;
  p.own_rows = static_cast<int32_t>(H < kRowsTile ? H : kRowsTile);
  p.ctas = sms;
  p.spins = g_spins.load(std::memory_order_relaxed);
  p.status = status;

  const Kernels& ks = kKernels[k];
  p.image_bytes = ks.image_bytes;
  p.tile_cost = ks.tile_cost;
  if (!g_smem_ready[dev][k].load(std::memory_order_acquire)) {
    // idempotent: two threads racing here both set the same attribute
    const cudaError_t e =
        cudaFuncSetAttribute(ks.attend, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(ks.smem));
    if (e != cudaSuccess) return mla::cuda_failure(e);
    g_smem_ready[dev][k].store(true, std::memory_order_release);
  }
  CUtensorMap slab_map{}, half_map{};
  p.box_rows = 0;
  if (by_tensor_copies(k, block_size, num_blocks)) {
    const int64_t cache_rows = num_blocks * block_size;
    const int box = box_rows_of(block_size);
    PFN_cuTensorMapEncodeTiled_v12000 encode = tensor_map_encoder();
    if (encode == nullptr) return mla::cuda_failure(cudaErrorNotSupported);
    const cuuint64_t elem = k == 3 ? 1 : 2;
    const cuuint64_t dims[2] = {576, static_cast<cuuint64_t>(cache_rows)};
    const cuuint64_t strides[1] = {576 * elem};
    const cuuint32_t size[2] = {static_cast<cuuint32_t>(128 / elem), static_cast<cuuint32_t>(box)};
    const cuuint32_t step[2] = {1, 1};
    const CUtensorMapDataType type = k == 3 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
    CUresult r = encode(&slab_map, type, 2, const_cast<void*>(cache), dims, strides, size, step, CU_TENSOR_MAP_INTERLEAVE_NONE,
                        CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_128B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r == CUDA_SUCCESS && box == kKeys) {
      const cuuint64_t dims3[3] = {size[0], dims[1], kDv / size[0]};  // bytes of a slab, rows, value slabs
      const cuuint64_t strides3[2] = {strides[0], 128};
      const cuuint32_t size3[3] = {size[0], kKeys, static_cast<cuuint32_t>(kDv / size[0] / 2)};
      const cuuint32_t step3[3] = {1, 1, 1};
      r = encode(&half_map, type, 3, const_cast<void*>(cache), dims3, strides3, size3, step3, CU_TENSOR_MAP_INTERLEAVE_NONE,
                 CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_128B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    }
    if (r != CUDA_SUCCESS) return MLA_ERR_INVALID_ARG;
    p.box_rows = box;
  }
  p.prefix_cost = needs_decoding(k) && p.image == nullptr ? ks.tile_cost : ks.prefix_cost;
  void* args[] = {&p};
  void* attend_args[] = {&slab_map, &half_map, &p};
  bool pdl = (flags & MLA_FLAG_PDL) != 0;
  if (p.image != nullptr) {
    s = launch(ks.image, dim3(static_cast<unsigned>(lay.image_tiles), static_cast<unsigned>(G), 1), 256, 0, pdl, stream,
               args);
    if (s != MLA_OK) return s;
    pdl = true;
  }
  s = launch(ks.attend, dim3(static_cast<unsigned>(sms), 1, 1), kThreads, ks.smem, pdl, stream, attend_args);
  if (s != MLA_OK) return s;

  // slices: as many blocks as run at once, three to an SM, a thread not below one chunk of columns
  const int64_t rows = T * ((H + kJoinRows - 1) / kJoinRows);
  int32_t slices = 1;
  while (slices < 32 && rows * slices * 2 <= 3 * sms) slices *= 2;
  void* jargs[] = {&p, &slices};
  const void* join = slices <= 2   ? reinterpret_cast<const void*>(&join_kernel<4>)
                     : slices == 4 ? reinterpret_cast<const void*>(&join_kernel<2>)
                                   : reinterpret_cast<const void*>(&join_kernel<1>);
  return launch(join, dim3(static_cast<unsigned>(rows * slices), 1, 1), kJoinThreads,
                static_cast<size_t>(2 * sms) * kJoinRows * sizeof(float), true, stream, jargs);
}

}  // extern "C"
