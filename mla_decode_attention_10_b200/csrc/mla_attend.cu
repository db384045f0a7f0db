// mla_attend.cu -- decode attention over the paged latent cache with shared
// prefixes, on the tcgen05 tensor cores (contract in mla_epilogue.h).
//
//   s = scale * q . key (576 terms),  p = exp(s - m),  out = (sum_k p key[0:512]) / (sum_k p)
//
// Work.  A unit is a prefix group (all rows (token, head) of the group against
// the prefix's keys) or a token (its H rows against its own keys).  A unit's
// rows are taken 64 at a time (row tile) and its keys 64 at a time (key tile).
// All (unit, row tile, key tile) triples, in this order, are dealt out to one
// CTA per SM in equal contiguous runs: every CTA gets the same number of
// tiles whatever the lengths are, and lengths stay in device memory (each CTA
// adds them up itself).  A CTA's piece of one row tile is a segment; it ends
// with the segment's unnormalised sum, maximum and denominator in the
// workspace, and a second small kernel joins a row's segments.
//
// A CTA holds 64 rows because TMEM holds their fp32 sums, 64 x 512, in half of
// its 512 columns (128 rows would fill it and leave no room for the scores).
// M = 64 in the weight-stationary form (.ws) spreads a row over two TMEM lanes
// (columns 0 .. N/2-1 on lanes 0..63, the rest on lanes 64..127).  Measured on
// B200: N = 256 in 80 cycles, against 128 for the plain M = 64 form; N = 64 in
// 50 for both.
//
// Roles (13 warps):
//   warps 0..3   softmax: scores from TMEM, running maximum and sum, weights
//                to shared memory, the sums' rescaling, the segment's result;
//   warp 4       issues the MMAs: per key tile 36 of S = Q K^T (M 64, N 64,
//                K 16) and 8 of O += P V (M 64, N 256, K 16; V is the K tile
//                itself, read with the key index as the contraction);
//   warps 5..12  load q and the cache rows, decode them to bf16 (or fp16 when
//                both are e4m3: one conversion instead of four) and store
//                them in the 128-byte swizzle.  The next tile's loads are in
//                flight in registers while the tensor cores work on the two
//                tiles in shared memory.  Plain loads take any block size,
//                page order and row format, and zero what lies behind a
//                sequence's end or in a page that does not exist.
// S of tile i+1 is issued before O of tile i, so the softmax of i overlaps it.
// Every wait is bounded: on timeout a status bit is set, all roles stop, TMEM
// is freed and the kernel returns.

#include <cuda_runtime.h>

#include <atomic>
#include <climits>
#include <cmath>
#include <cstdint>

#include "latent_math.cuh"
#include "latent_rows.cuh"
#include "mla_epilogue.h"
#include "mla_runtime.h"

namespace mla {
namespace attend {

constexpr int kRowsTile = 64;   // rows of a CTA (MMA M)
constexpr int kKeys = 64;       // keys of a tile
constexpr int kD = 576;         // score contraction
constexpr int kDv = 512;        // values
constexpr int kSlabs = 9;       // 64-wide column slabs of a 576-wide row
constexpr uint32_t kSlabBytes = 64 * 128;               // 64 rows x 64 values of 16 bits
constexpr uint32_t kTileBytes = kSlabs * kSlabBytes;    // 72 KB
constexpr uint32_t kPBytes = kRowsTile * kKeys * 2;     // 8 KB
constexpr int kStages = 2;
constexpr int kSoftWarps = 4, kMmaWarp = 4, kLoadWarp0 = 5, kLoadWarps = 8;
constexpr int kThreads = 32 * (kLoadWarp0 + kLoadWarps);  // 416
constexpr uint32_t kSmemBytes = kTileBytes * (1 + kStages) + kPBytes + 1024;
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kTmemS = 256;       // score buffers: columns 256 + 32 b
constexpr uint32_t kWaitSpins = 1u << 22;
constexpr float kRescale = 8.0f;       // the reference maximum moves when a score passes it by 2^8
constexpr int kChunks = kDv / 4;       // 16-byte pieces of a row's fp32 sums
constexpr int kSegCost = 2;            // what a segment's start and end cost, in key tiles (see plan_run)

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
  int64_t* plan;      // [0] tiles per CTA, [1 + u] first tile of unit u
  uint8_t* prefix_part;
  uint8_t* own_part;
  int32_t own_rows;   // rows of an own segment: min(H, 64)
  int32_t ctas;       // CTAs of the attention kernel
  int32_t* status;
};

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

// ---- units ---------------------------------------------------------------------

struct Unit {
  int64_t rows0;  // first (token, head) row
  int64_t rows;
  int64_t len;    // keys
  const int32_t* table;
  bool prefix;
  int64_t part0;  // number of the first row tile, within the unit's kind

  __device__ __forceinline__ int64_t row_tiles() const { return (rows + kRowsTile - 1) / kRowsTile; }
  __device__ __forceinline__ int64_t key_tiles() const { return (len + kKeys - 1) / kKeys; }
  // what one row tile counts for in the deal: kSegCost for its start, then its key tiles
  __device__ __forceinline__ int64_t row_cost() const { return len > 0 ? key_tiles() + kSegCost : 0; }
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

// Unit u: group u for u < G, else token u - G.  `bad`: something had to be cut.
// Row tiles are numbered from rows0 / 64 + g on for a group: floor(x) + 1 >=
// ceil(x), so the numbers of consecutive groups do not meet.
__device__ __forceinline__ Unit unit_at(const Params& p, int64_t u, bool& bad) {
  Unit x;
  int64_t len, keys;
  if (u < p.G) {
    int64_t lo, hi;
    group_tokens(p, u, lo, hi, bad);
    len = __ldcg(p.prefix_lens + u);
    keys = p.prefix_keys;
    x.rows0 = lo * p.H;
    x.rows = (hi - lo) * p.H;
    x.table = p.prefix_table + u * p.prefix_stride;
    x.prefix = true;
    x.part0 = x.rows0 / kRowsTile + u;
  } else {
    const int64_t t = u - p.G;
    bad = false;
    len = p.table_keys > 0 ? __ldcg(p.seq_lens + t) : 0;
    keys = p.table_keys;
    x.rows0 = t * p.H;
    x.rows = p.H;
    x.table = p.block_table + t * p.table_stride;
    x.prefix = false;
    x.part0 = t * ((p.H + kRowsTile - 1) / kRowsTile);
  }
  bad = bad || len > keys;
  x.len = cut(len, 0, keys);
  return x;
}

// One segment: rows [row0, row0 + rows) against key tiles [k0, k1).
struct Segment {
  int64_t row0;
  int32_t rows;
  int32_t k0, k1;
  int64_t len;
  const int32_t* table;
  uint8_t* part;
  int32_t part_rows;
};

struct Cursor {
  int64_t pos, end;  // this CTA's run
  int64_t base, u;   // where unit u starts
};

__device__ __forceinline__ bool next_segment(const Params& p, Cursor& c, Segment& s) {
  while (c.pos < c.end) {
    bool bad;
    const Unit x = unit_at(p, c.u, bad);
    const int64_t per = x.row_cost(), n = x.row_tiles() * per;
    if (c.pos >= c.base + n) {
      c.base += n;
      ++c.u;
      continue;
    }
    const int64_t off = c.pos - c.base, r = off / per, from = off - r * per;
    const int64_t to = per - from < c.end - c.pos ? per : from + (c.end - c.pos);
    c.pos += to - from;
    if (to <= kSegCost) continue;  // only the row tile's start: its keys are the next CTA's
    const int64_t k = from > kSegCost ? from - kSegCost : 0;
    s.row0 = x.rows0 + r * kRowsTile;
    s.rows = static_cast<int32_t>(x.rows - r * kRowsTile < kRowsTile ? x.rows - r * kRowsTile : kRowsTile);
    s.k0 = static_cast<int32_t>(k);
    s.k1 = static_cast<int32_t>(to - kSegCost);
    s.len = x.len;
    s.table = x.table;
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

// Instruction descriptor of kind::f16, fp32 accumulator: operands fp16 (0) or
// bf16 (1), M = 64; b_mn: B is MN-major.
__device__ __forceinline__ constexpr uint32_t instr_desc(bool f16, int n, bool b_mn) {
  return (1u << 4) | ((f16 ? 0u : 1u) << 7) | ((f16 ? 0u : 1u) << 10) | ((b_mn ? 1u : 0u) << 16) |
         (static_cast<uint32_t>(n >> 3) << 17) | (static_cast<uint32_t>(kRowsTile >> 4) << 24);
}

// One MMA, issued by one lane of the warp.  The warp stays converged, and
// everything that decides the addresses is uniform over it (broadcast where it
// comes from memory), so the compiler keeps the descriptors in uniform
// registers.  Issued from a branch on the lane, each MMA first moved its
// descriptors there: 50 to 65 cycles, where the N = 64 form takes 32 (the 4 KB
// of its operands at 128 bytes a cycle).
template <bool ACCUMULATE>
__device__ __forceinline__ void mma_ws(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "elect.sync _|q, 0xffffffff;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "@q tcgen05.mma.ws.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "n"(ACCUMULATE ? 1 : 0)
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

__device__ __forceinline__ int uniform(int v) { return __shfl_sync(0xffffffffu, v, 0); }

__device__ __forceinline__ void fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }

__device__ __forceinline__ void arrive(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}

// 32 columns of this warp's TMEM lanes, one lane's per thread; the wait names
// the registers, so no use of them can be scheduled before it.
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, uint32_t (&v)[32]) {
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

// Whether the phase of `parity` has completed.  One lane asks (32 lanes' asking
// costs 32 times as much of the shared-memory pipe, which the operands and the
// loaders need), the warp stays converged and gets one answer.
__device__ __forceinline__ bool warp_test(uint32_t bar, uint32_t parity) {
  uint32_t done;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.b32 p, 0, 0;\n\t"
      "elect.sync _|q, 0xffffffff;\n\t"
      "@q mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(done)
      : "r"(bar), "r"(parity)
      : "memory");
  return __any_sync(0xffffffffu, done != 0u) != 0;
}

// Waits for the phase, at most kWaitSpins tries or until another role gave up.
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, volatile uint32_t* abort_flag) {
  for (uint32_t i = 0; i < kWaitSpins; ++i) {
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
    if ((i & 15u) == 15u && __any_sync(0xffffffffu, *abort_flag != 0u)) return false;
  }
  return false;
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

struct Bars {
  uint64_t kv_full[kStages], kv_empty[kStages];
  uint64_t q_full, q_empty;
  uint64_t s_full[2], s_empty[2];
  uint64_t p_full, pv_done, o_empty;
  uint64_t drained;
};

struct Shared {
  Bars bars;
  uint32_t tmem;
  uint32_t abort_flag;
  uint32_t never;  // stays 0
  alignas(16) uint8_t valid[kStages][kKeys];  // 1: the key counts, by stage
  float xch[2][kRowsTile];
  int64_t warp_sum[kThreads / 32];
  int64_t first_unit, first_base;
};

// ---- the loaders' pieces --------------------------------------------------------

// A thread's share of a quantised row (four threads to a row): its words by format.
template <int FMT>
struct Raw {
  static constexpr int kWords = FMT == MLA_CACHE_MX ? 11 : 9;
  uint4 w[kWords];
};

// Word j: e4m3, piece 4 j + quarter.  mx: the same for the 8 slabs of codes, then
// the scale bytes, then two pieces of rotary values (the flip keeps two rows'
// stores on different banks).
template <int FMT>
__device__ __forceinline__ uint4 load_word(const uint8_t* row, int j, int r, int quarter, bool ok) {
  const uint4* s = reinterpret_cast<const uint4*>(row);
  int piece = 4 * j + quarter;
  if constexpr (FMT == MLA_CACHE_MX) {
    if (j == 8) piece = kMxScales / 16;
    if (j > 8) piece = kMxPe / 16 + (((j - 9) ^ (r & 1)) << 2) + quarter;
  }
  return ok ? __ldcg(s + piece) : make_uint4(0, 0, 0, 0);
}

template <int FMT>
__device__ __forceinline__ void load_row(Raw<FMT>& raw, const uint8_t* row, int r, int quarter, bool ok) {
#pragma unroll
  for (int j = 0; j < Raw<FMT>::kWords; ++j) raw.w[j] = load_word<FMT>(row, j, r, quarter, ok);
}

// Piece `c` (0..7) of slab `s` of row r in a tile at `base`.
__device__ __forceinline__ uint32_t piece_addr(uint32_t base, int s, int r, int c) {
  return base + static_cast<uint32_t>(s) * kSlabBytes + static_cast<uint32_t>(r) * 128u +
         (static_cast<uint32_t>(c ^ (r & 7)) << 4);
}

// Word j of a row, decoded, into the tile at `base` (`scales`: word 8 of an mx row).
template <int FMT, bool F16>
__device__ __forceinline__ void store_word(const uint4& w, const uint4& scales, int j, uint32_t base, int r, int quarter) {
  if (FMT == MLA_CACHE_MX && j > 8) {
    st_shared(piece_addr(base, 8, r, (((j - 9) ^ (r & 1)) << 2) + quarter), w);
  } else if (FMT == MLA_CACHE_E4M3 || j < 8) {
    uint4 a, b;
    if constexpr (FMT == MLA_CACHE_E4M3) {
      if (any_nan_code(w)) {
        if constexpr (F16) {
          codes_to_f16(w, a, b);
        } else {
          codes_to_bf16(w, 1.0f, a, b);
        }
      } else if constexpr (F16) {
        plain_codes_to_f16(w, a, b);
      } else {
        plain_codes_to_bf16(w, kBf16Pow120, a, b);
      }
    } else {
      // the scale byte of latents 64 j + 16 quarter ..: group 2 j + quarter / 2
      const uint32_t word = (j >> 1) == 0 ? scales.x : (j >> 1) == 1 ? scales.y : (j >> 1) == 2 ? scales.z : scales.w;
      const uint32_t byte = (word >> (16 * (j & 1) + 8 * (quarter >> 1))) & 0xffu;
      if (byte > kMxPlain || any_nan_code(w)) {
        codes_to_bf16(w, mx_scale(byte), a, b);
      } else {
        plain_codes_to_bf16(w, mx_mul2(byte), a, b);
      }
    }
    st_shared(piece_addr(base, j, r, 2 * quarter), a);
    st_shared(piece_addr(base, j, r, 2 * quarter + 1), b);
  }
}

template <int FMT, bool F16>
__device__ __forceinline__ void store_row(const Raw<FMT>& raw, uint32_t base, int r, int quarter) {
#pragma unroll
  for (int j = 0; j < Raw<FMT>::kWords; ++j)
    store_word<FMT, F16>(raw.w[j], raw.w[FMT == MLA_CACHE_MX ? 8 : 0], j, base, r, quarter);
}

// One q row's share of a thread among `LANES` to a row: 16-bit values straight to
// shared memory, or codes through registers.
template <int LANES, bool F16>
__device__ __forceinline__ void load_q16(const uint8_t* row, uint32_t base, int r, int lane, bool ok) {
#pragma unroll
  for (int s = 0; s < kSlabs; ++s) {
#pragma unroll
    for (int c = 0; c < 8; c += LANES)
      cp_async16(piece_addr(base, s, r, c + lane), row + (s * 8 + c + lane) * 16, ok);
  }
}

template <bool F16>
__device__ __forceinline__ void load_q8(const uint8_t* row, uint32_t base, int r, int quarter, bool ok) {
  uint4 w[kSlabs];
#pragma unroll
  for (int j = 0; j < kSlabs; ++j) w[j] = load_word<MLA_CACHE_E4M3>(row, j, r, quarter, ok);
#pragma unroll
  for (int j = 0; j < kSlabs; ++j) store_word<MLA_CACHE_E4M3, F16>(w[j], w[j], j, base, r, quarter);
}

// ---- the roles ---------------------------------------------------------------------

// A walk over this CTA's key tiles, one at a time.
struct TileWalk {
  Cursor cur;
  const int32_t* table;
  int32_t len, kt, k1;
  int32_t row0, rows;  // q rows of the segment
  int32_t seg;         // segments begun
  bool first;          // the tile is its segment's first

  __device__ __forceinline__ void start(const Cursor& c) {
    cur = c;
    kt = k1 = seg = 0;
    first = false;
  }
  // To the next tile; false behind the last.
  __device__ __forceinline__ bool next(const Params& p) {
    first = ++kt >= k1;
    if (!first) return true;
    Segment s;
    if (!next_segment(p, cur, s)) {
      kt = k1 = 0;
      return false;
    }
    table = s.table;
    len = static_cast<int32_t>(s.len);
    kt = s.k0;
    k1 = s.k1;
    row0 = static_cast<int32_t>(s.row0);
    rows = s.rows;
    ++seg;
    return true;
  }
};

// Where a thread finds the key of its row r in a tile.  The page number is
// fetched a tile ahead and not looked at before address().
struct KeyAt {
  int32_t page;
  uint32_t in_page;
  bool key;

  __device__ __forceinline__ void fetch(const Params& p, const TileWalk& w, int r, bool any) {
    const uint32_t k = static_cast<uint32_t>(w.kt) * kKeys + static_cast<uint32_t>(r);
    key = any && k < static_cast<uint32_t>(w.len);
    page = 0;
    in_page = 0;
    if (key) {
      const uint32_t bs = static_cast<uint32_t>(p.block_size), pg = k / bs;
      in_page = k - pg * bs;
      page = __ldcg(w.table + pg);
    }
  }
  __device__ __forceinline__ const uint8_t* address(const Params& p, int bytes, bool& ok, bool& bad) const {
    ok = key && page >= 0 && page < p.cache_blocks;
    bad = bad || (key && !ok);
    return ok ? p.cache + (static_cast<int64_t>(page) * p.block_size + in_page) * bytes : p.cache;
  }
};

// q row `i` of the `rows` from `row0` on.
__device__ __forceinline__ const uint8_t* q_row(const Params& p, int32_t row0, int32_t rows, int i, bool& ok) {
  ok = i < rows;
  const int32_t row = ok ? row0 + i : 0, t = row / p.H;
  return p.q + static_cast<int64_t>(t) * p.q_st + static_cast<int64_t>(row - t * p.H) * p.q_sh;
}

__device__ __forceinline__ void publish(uint32_t bar) {
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  __syncwarp();
  if ((threadIdx.x & 31u) == 0u) arrive(bar);
}

// bf16 rows: asynchronous copies straight into the tile, eight threads to a
// row (whole 128-byte lines), rows r and r + 32 of a thread.  Up to two tiles
// are under way; a tile is published when its copies have landed, at the
// latest before this warp waits for a free stage.
__device__ __forceinline__ bool load_bf16(const Params& p, const Cursor& cur, Shared& sh, uint32_t sQ, uint32_t sK,
                                          bool& bad_page) {
  const int tid = static_cast<int>(threadIdx.x) - 32 * kLoadWarp0;
  const int r = tid >> 3, c = tid & 7;
  volatile uint32_t* ab = &sh.abort_flag;
  TileWalk w;
  w.start(cur);
  bool any = w.next(p), good = true;
  KeyAt at[2];
  at[0].fetch(p, w, r, any);
  at[1].fetch(p, w, r + 32, any);
  uint32_t it = 0, published = 0;
  bool q_out = false;  // q copies under way with tile it - 1
  auto publish_tile = [&]() {
    if (q_out) {
      publish(smem_u32(&sh.bars.q_full));
      q_out = false;
    }
    publish(smem_u32(&sh.bars.kv_full[published & 1u]));
    ++published;
  };
  while (uniform(any ? 1 : 0) != 0) {
    const uint32_t st = it & 1u, base = sK + st * kTileBytes;
    const bool first = uniform(w.first ? 1 : 0) != 0;
    if (it >= kStages) {
      const uint32_t bar = smem_u32(&sh.bars.kv_empty[st]), parity = (it / kStages - 1) & 1u;
      if (published < it && (first || !warp_test(bar, parity))) {
        asm volatile("cp.async.wait_group 0;" ::: "memory");
        while (published < it) publish_tile();
      }
      if (!warp_wait(bar, parity, ab)) good = false;
    } else if (first && published < it) {
      asm volatile("cp.async.wait_group 0;" ::: "memory");
      while (published < it) publish_tile();
    }
    if (first) {  // the segment's q rows, once the previous segment's scores have been computed
      if (good && w.seg > 1) good = warp_wait(smem_u32(&sh.bars.q_empty), (w.seg - 2) & 1u, ab);
      if (p.q_fp8) {
        bool ok;
        const uint8_t* src = q_row(p, w.row0, w.rows, tid >> 2, ok);
        load_q8<false>(src, sQ, tid >> 2, tid & 3, ok);
      } else {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          bool ok;
          const uint8_t* src = q_row(p, w.row0, w.rows, r + 32 * h, ok);
          load_q16<8, false>(src, sQ, r + 32 * h, c, ok);
        }
      }
      q_out = true;
    }
    if (!good) break;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      bool ok;
      const uint8_t* src = at[h].address(p, row_bytes(MLA_CACHE_BF16), ok, bad_page);
#pragma unroll
      for (int s = 0; s < kSlabs; ++s) cp_async16(piece_addr(base, s, r + 32 * h, c), src + (s * 8 + c) * 16, ok);
      if (c == 0) sh.valid[st][r + 32 * h] = ok ? 1 : 0;
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
    ++it;
    any = w.next(p);
    at[0].fetch(p, w, r, any);
    at[1].fetch(p, w, r + 32, any);
    if (published + 1 < it) {
      asm volatile("cp.async.wait_group 1;" ::: "memory");
      publish_tile();
    }
  }
  asm volatile("cp.async.wait_group 0;" ::: "memory");
  while (good && published < it) publish_tile();
  return good;
}

// Quantised rows: the eight warps form two groups of four, group g has the
// tiles of stage g.  A tile's rows wait in registers (rows r and r + 32 of a
// thread, four threads to a row) while the other group's tile is stored, and
// are decoded on their way to shared memory.
template <int FMT, bool F16>
__device__ __forceinline__ bool load_codes(const Params& p, const Cursor& cur, Shared& sh, uint32_t sQ, uint32_t sK,
                                           bool& bad_page) {
  const int tid = (static_cast<int>(threadIdx.x) - 32 * kLoadWarp0) & 127;
  const uint32_t st = static_cast<uint32_t>(uniform((static_cast<int>(threadIdx.x) - 32 * kLoadWarp0) >> 7));
  const int r = tid >> 2, quarter = tid & 3;
  const uint32_t base = sK + st * kTileBytes;
  volatile uint32_t* ab = &sh.abort_flag;
  TileWalk w;
  w.start(cur);
  bool any = w.next(p);
  if (st == 1 && any) any = w.next(p);
  KeyAt at[2];
  Raw<FMT> raw[2];
  bool ok[2];
  auto issue = [&]() {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const uint8_t* src = at[h].address(p, row_bytes(FMT), ok[h], bad_page);
      load_row<FMT>(raw[h], src, r + 32 * h, quarter, ok[h]);
    }
  };
  at[0].fetch(p, w, r, any);
  at[1].fetch(p, w, r + 32, any);
  issue();
  for (uint32_t n = 0; uniform(any ? 1 : 0) != 0; ++n) {
    // what this tile's q rows need; then the walk goes on to this group's next tile
    const bool first = uniform(w.first ? 1 : 0) != 0;
    const int32_t row0 = w.row0, rows = w.rows, seg = w.seg;
    any = w.next(p);
    if (any) any = w.next(p);
    at[0].fetch(p, w, r, any);
    at[1].fetch(p, w, r + 32, any);
    if (n > 0 && !warp_wait(smem_u32(&sh.bars.kv_empty[st]), (n - 1) & 1u, ab)) return false;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
#pragma unroll
      for (int j = 0; j < Raw<FMT>::kWords; ++j)
        store_word<FMT, F16>(raw[h].w[j], raw[h].w[FMT == MLA_CACHE_MX ? 8 : 0], j, base, r + 32 * h, quarter);
      if (quarter == 0) sh.valid[st][r + 32 * h] = ok[h] ? 1 : 0;
    }
    publish(smem_u32(&sh.bars.kv_full[st]));
    if (first) {
      // the segment's q rows, once the previous segment's scores have been computed
      if (seg > 1 && !warp_wait(smem_u32(&sh.bars.q_empty), (seg - 2) & 1u, ab)) return false;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        bool q_ok;
        const uint8_t* src = q_row(p, row0, rows, r + 32 * h, q_ok);
        if (p.q_fp8) {
          load_q8<F16>(src, sQ, r + 32 * h, quarter, q_ok);
        } else if constexpr (!F16) {
          load_q16<4, F16>(src, sQ, r + 32 * h, quarter, q_ok);
        }
      }
      asm volatile("cp.async.commit_group;" ::: "memory");
      asm volatile("cp.async.wait_group 0;" ::: "memory");
      publish(smem_u32(&sh.bars.q_full));
    }
    // the next tile's loads go out behind the fences, which would wait for them
    issue();
  }
  return true;
}

template <int FMT, bool F16>
__device__ __forceinline__ void loader(const Params& p, const Cursor& cur, Shared& sh, uint32_t sQ, uint32_t sK) {
  bool bad_page = false, good;
  if constexpr (FMT == MLA_CACHE_BF16) {
    good = load_bf16(p, cur, sh, sQ, sK, bad_page);
  } else {
    good = load_codes<FMT, F16>(p, cur, sh, sQ, sK, bad_page);
  }
  if (!good && (threadIdx.x & 31u) == 0u && sh.abort_flag == 0u) {
    *reinterpret_cast<volatile uint32_t*>(&sh.abort_flag) = 1u;
    report(p.status, MLA_STATUS_TIMEOUT);
  }
  if (bad_page) report(p.status, MLA_STATUS_SLOT_RANGE);
}

// The products of one tile's weights with its values, into the sums.
template <bool F16, bool FIRST>
__device__ __forceinline__ void pv_products(uint64_t p, uint64_t v, uint32_t tmem) {
  constexpr uint32_t id = instr_desc(F16, 256, true);
#pragma unroll
  for (int half = 0; half < 2; ++half) {
    const uint32_t d = tmem + static_cast<uint32_t>(half) * 128u;
    const uint64_t vh = v + static_cast<uint64_t>(half * 4 * (kSlabBytes >> 4));
    mma_ws<!FIRST>(d, p, vh, id);
#pragma unroll
    for (int j = 1; j < kKeys / 16; ++j)
      mma_ws<true>(d, p + static_cast<uint64_t>(j * 2), vh + static_cast<uint64_t>(j * 128), id);
  }
}

template <bool F16>
__device__ __forceinline__ void mma_role(const Params& p, Cursor cur, Shared& sh, uint32_t sQ, uint32_t sK, uint32_t sP,
                                         uint32_t tmem) {
  volatile uint32_t* ab = &sh.abort_flag;
  const uint64_t dQ = smem_desc(sQ, 16, 1024), dK = smem_desc(sK, 16, 1024);
  const uint64_t dP = smem_desc(sP, 16, 1024), dV = smem_desc(sK, kSlabBytes, 1024);
  uint32_t s = 0, v = 0;        // the next tile to get scores, and sums: v <= s <= v + 2
  uint32_t seg = 0;             // segments begun
  int left = 0;                 // tiles of the current segment without scores
  bool more = true, first = false;
  uint32_t first_bits = 0;      // bit (i & 1): tile i is its segment's first
  uint32_t v_seg = 0;           // segments whose sums have begun
  uint32_t idle = 0;
  // whichever has its operands goes: the sums of the oldest tile (they free its
  // stage), else the scores of the next.  Waiting for a certain one of the two
  // would let the loaders and the tensor cores wait for each other in turn.
  while (true) {
    if (left == 0 && more) {
      Segment x;
      left = uniform(next_segment(p, cur, x) ? x.k1 - x.k0 : 0);
      more = left > 0;
      first = true;
      if (more) ++seg;
    }
    if (left == 0 && v == s) break;
    if (v < s && warp_test(smem_u32(&sh.bars.p_full), v & 1u)) {
      const bool opens = ((first_bits >> (v & 1u)) & 1u) != 0u;
      if (!opens || v_seg == 0 || warp_test(smem_u32(&sh.bars.o_empty), (v_seg - 1) & 1u)) {
        fence_after();
        const uint64_t vd = dV + (v & 1u) * (kTileBytes >> 4);
        if (opens) {
          pv_products<F16, true>(dP, vd, tmem);
          ++v_seg;
        } else {
          pv_products<F16, false>(dP, vd, tmem);
        }
        commit(smem_u32(&sh.bars.kv_empty[v & 1u]));
        commit(smem_u32(&sh.bars.pv_done));
        ++v;
        idle = 0;
        continue;
      }
    }
    const uint32_t st = s & 1u;
    if (left > 0 && s < v + 2 && warp_test(smem_u32(&sh.bars.kv_full[st]), (s / kStages) & 1u) &&
        (!first || warp_test(smem_u32(&sh.bars.q_full), (seg - 1) & 1u)) &&
        (s < 2 || warp_test(smem_u32(&sh.bars.s_empty[st]), (s / 2 - 1) & 1u))) {
      fence_after();
      constexpr uint32_t id = instr_desc(F16, kKeys, false);
      const uint64_t k = dK + st * (kTileBytes >> 4);
#pragma unroll
      for (int j = 0; j < kD / 16; ++j) {
        const uint64_t off = static_cast<uint64_t>((j >> 2) * (kSlabBytes >> 4) + (j & 3) * 2);
        if (j == 0) {
          mma_ws<false>(tmem + kTmemS + 32u * st, dQ + off, k + off, id);
        } else {
          mma_ws<true>(tmem + kTmemS + 32u * st, dQ + off, k + off, id);
        }
      }
      commit(smem_u32(&sh.bars.s_full[st]));
      --left;
      if (left == 0) commit(smem_u32(&sh.bars.q_empty));
      first_bits = (first_bits & ~(1u << st)) | ((first ? 1u : 0u) << st);
      first = false;
      ++s;
      idle = 0;
      continue;
    }
    if (++idle > kWaitSpins || ((idle & 15u) == 15u && __any_sync(0xffffffffu, *ab != 0u))) {
      if ((threadIdx.x & 31u) == 0u && *ab == 0u) {
        *ab = 1u;
        report(p.status, MLA_STATUS_TIMEOUT);
      }
      break;
    }
  }
  // every product issued has completed before TMEM is freed
  commit(smem_u32(&sh.bars.drained));
  (void)warp_wait(smem_u32(&sh.bars.drained), 0u, &sh.never);
}

template <bool F16>
__device__ __forceinline__ void softmax_role(const Params& p, Cursor cur, Shared& sh, uint32_t sP, uint32_t tmem,
                                             float scale2) {
  const int warp = static_cast<int>(threadIdx.x) >> 5, lane = static_cast<int>(threadIdx.x) & 31;
  const int r = (warp & 1) * 32 + lane;  // this thread's row
  const int half = warp >> 1;            // its half of the keys (scores) and of each 256 columns (sums)
  const uint32_t lanes = static_cast<uint32_t>(warp) << 21;
  volatile uint32_t* ab = &sh.abort_flag;
  Segment seg;
  uint32_t it = 0;
  bool good = true;
  while (good && next_segment(p, cur, seg)) {
    float m = -INFINITY;  // the reference maximum of the row, in powers of two
    float l = 0.0f;       // this thread's share of the denominator
    for (int kt = seg.k0; kt < seg.k1; ++kt, ++it) {
      const uint32_t st = it & 1u;
      good = warp_wait(smem_u32(&sh.bars.s_full[st]), (it / 2) & 1u, ab) && good;
      // all four warps leave together: a wait that ran out in one is seen by all here
      if (bar_or(1, 32 * kSoftWarps, !good)) {
        good = false;
        break;
      }
      fence_after();
      uint32_t v[32];
      tmem_ld32(tmem + kTmemS + 32u * st + lanes, v);
      const uint4 va = ld_shared(smem_u32(&sh.valid[st][32 * half])), vb = ld_shared(smem_u32(&sh.valid[st][32 * half + 16]));
      fence_before();
      __syncwarp();
      if (lane == 0) arrive(smem_u32(&sh.bars.s_empty[st]));
      float s[32];
      float top = -INFINITY;
#pragma unroll
      for (int j = 0; j < 32; ++j) s[j] = __uint_as_float(v[j]) * scale2;
      if ((va.x & va.y & va.z & va.w & vb.x & vb.y & vb.z & vb.w) != 0x01010101u) {
        const uint32_t ok[8] = {va.x, va.y, va.z, va.w, vb.x, vb.y, vb.z, vb.w};
#pragma unroll
        for (int j = 0; j < 32; ++j) s[j] = (ok[j >> 2] >> (8 * (j & 3))) & 1u ? s[j] : -INFINITY;
      }
#pragma unroll
      for (int j = 0; j < 32; ++j) top = fmaxf(top, s[j]);
      const bool first = kt == seg.k0;
      // products into the sums run until pv_done of the previous tile
      const bool moved = bar_or(1, 32 * kSoftWarps, first || top > m + kRescale);
      float factor = 1.0f;
      if (moved) {
        sh.xch[half][r] = top;
        bar_sync(2, 32 * kSoftWarps);
        const float next = fmaxf(m, fmaxf(top, sh.xch[half ^ 1][r]));
        if (!first && next > m) factor = m == -INFINITY ? 0.0f : exp2_fast(m - next);
        m = next;
        l *= factor;
      }
      const float ref = m == -INFINITY ? 0.0f : m;
      uint32_t w[16];
#pragma unroll
      for (int j = 0; j < 16; ++j) {
        const float a = exp2_fast(s[2 * j] - ref), b = exp2_fast(s[2 * j + 1] - ref);
        l += a + b;
        if constexpr (F16) {
          asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(w[j]) : "f"(b), "f"(a));
        } else {
          w[j] = pack_bf16x2(a, b);
        }
      }
      if (it > 0) {  // the previous tile's weights have been read, its products are in the sums
        good = warp_wait(smem_u32(&sh.bars.pv_done), (it - 1) & 1u, ab);
      }
      if (good && moved && !first) {
        fence_after();
#pragma unroll 1
        for (uint32_t c = 0; c < 256; c += 32) {
          tmem_ld32(tmem + lanes + c, v);
#pragma unroll
          for (int j = 0; j < 32; ++j) v[j] = __float_as_uint(__uint_as_float(v[j]) * factor);
          tmem_st32(tmem + lanes + c, v);
        }
        asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
      }
#pragma unroll
      for (int j = 0; j < 4; ++j)
        st_shared(sP + static_cast<uint32_t>(r) * 128u + (static_cast<uint32_t>((half * 4 + j) ^ (r & 7)) << 4),
                  make_uint4(w[4 * j], w[4 * j + 1], w[4 * j + 2], w[4 * j + 3]));
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      fence_before();
      __syncwarp();
      if (lane == 0) arrive(smem_u32(&sh.bars.p_full));
    }
    if (!good) break;
    // ---- the segment's result
    good = warp_wait(smem_u32(&sh.bars.pv_done), (it - 1) & 1u, ab);
    if (bar_or(1, 32 * kSoftWarps, !good)) {
      good = false;
      break;
    }
    fence_after();
    const bool keep = r < seg.rows;
    uint4* dst = reinterpret_cast<uint4*>(seg.part) + r;
#pragma unroll 1
    for (int c = 0; c < 256; c += 32) {
      uint32_t v[32];
      tmem_ld32(tmem + lanes + static_cast<uint32_t>(c), v);
      // TMEM column c of this lane: output column (c / 128) 256 + half 128 + c % 128
      const int chunk0 = ((c >> 7) * 256 + half * 128 + (c & 127)) / 4;
      if (keep) {
#pragma unroll
        for (int j = 0; j < 8; ++j)
          __stcg(dst + static_cast<int64_t>(chunk0 + j) * seg.part_rows,
                 make_uint4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]));
      }
    }
    fence_before();
    __syncwarp();
    if (lane == 0) arrive(smem_u32(&sh.bars.o_empty));
    sh.xch[half][r] = l;
    bar_sync(2, 32 * kSoftWarps);
    if (half == 0 && keep) {
      float* stat = reinterpret_cast<float*>(seg.part + static_cast<int64_t>(seg.part_rows) * kChunks * 16);
      __stcg(stat + r, m);
      __stcg(stat + seg.part_rows + r, l + sh.xch[1][r]);
    }
    bar_sync(2, 32 * kSoftWarps);
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
  for (int64_t u = u0; u < u1; ++u) {
    bool bad;
    sum += unit_at(p, u, bad).cost();
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
  const int64_t each = total > p.ctas ? (total + p.ctas - 1) / p.ctas : 1;
  Cursor c;
  c.pos = each * blockIdx.x;
  c.end = c.pos + each < total ? c.pos + each : total;
  int64_t base = before + incl - sum;
  if (blockIdx.x == 0 && threadIdx.x == 0) p.plan[0] = each;
  const bool mine = c.pos >= base && c.pos < base + sum;
  if (mine || blockIdx.x == 0) {
    for (int64_t u = u0; u < u1; ++u) {
      bool bad;
      const int64_t n = unit_at(p, u, bad).cost();
      if (blockIdx.x == 0) p.plan[1 + u] = base;
      if (c.pos >= base && c.pos < base + n) {
        sh.first_unit = u;
        sh.first_base = base;
      }
      base += n;
    }
  }
  __syncthreads();
  c.u = sh.first_unit;
  c.base = sh.first_base;
  return c;
}

template <int FMT, bool F16>
__global__ void __launch_bounds__(kThreads, 1) attend_kernel(const Params p) {
  constexpr uint32_t kFillWarps = FMT == MLA_CACHE_BF16 ? kLoadWarps : kLoadWarps / 2;  // that fill one tile
  extern __shared__ uint8_t dsmem[];
  __shared__ Shared sh;
  const int warp = uniform(static_cast<int>(threadIdx.x) >> 5);
  const uint32_t sQ = (smem_u32(dsmem) + 1023u) & ~1023u;
  const uint32_t sK = sQ + kTileBytes;
  const uint32_t sP = sK + kStages * kTileBytes;
  if (warp == kMmaWarp) {
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
    for (int i = 0; i < 2; ++i) {
      init(&sh.bars.kv_full[i], kFillWarps);
      init(&sh.bars.kv_empty[i], 1);
      init(&sh.bars.s_full[i], 1);
      init(&sh.bars.s_empty[i], kSoftWarps);
    }
    init(&sh.bars.q_full, kFillWarps);
    init(&sh.bars.q_empty, 1);
    init(&sh.bars.p_full, kSoftWarps);
    init(&sh.bars.pv_done, 1);
    init(&sh.bars.o_empty, kSoftWarps);
    init(&sh.bars.drained, 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  pdl_wait();     // the lengths, q and the cache rows may come from the upstream kernel
  pdl_trigger();  // the joining kernel waits for this grid's end itself
  fence_before();
  __syncthreads();
  fence_after();
  const uint32_t tmem = static_cast<uint32_t>(uniform(static_cast<int>(sh.tmem)));
  const Cursor cur = plan_run(p, sh);
  if (uniform(cur.pos < cur.end ? 1 : 0) != 0) {  // a branch that the compiler sees is uniform
    if (warp < kSoftWarps) {
      float scale2 = p.sm_scale * 1.4426950408889634f;  // powers of two: log2(e)
      if (p.q_fp8) scale2 *= __ldcg(p.q_scale);
      if (FMT == MLA_CACHE_E4M3) scale2 *= __ldcg(p.kv_scale);
      softmax_role<F16>(p, cur, sh, sP, tmem, scale2);
    } else if (warp == kMmaWarp) {
      mma_role<F16>(p, cur, sh, sQ, sK, sP, tmem);
    } else {
      loader<FMT, F16>(p, cur, sh, sQ, sK);
    }
  }
  fence_before();
  __syncthreads();
  if (warp == kMmaWarp) {
    fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTmemCols) : "memory");
  }
}

// ---- joining a row's segments ----------------------------------------------------------
//
// out = sum_i 2^(m_i - M) O_i / sum_i 2^(m_i - M) l_i.  A block takes one token,
// 16 of its heads and a slice of the columns; thread (row, worker).  The
// workers of a row first share out its segments for the weights, then its
// (column chunk, segment class) pairs for the sum.  With few tokens the
// columns are cut into more slices and the segments into classes, so that a
// single row's many segments are still read by many threads.

constexpr int kJoinRows = 16, kJoinWorkers = 16, kJoinThreads = kJoinRows * kJoinWorkers;

__global__ void __launch_bounds__(kJoinThreads) join_kernel(const Params p, int slices) {
  extern __shared__ float weights[];  // [segments][16]
  __shared__ float red[kJoinWorkers][kJoinRows];
  __shared__ uint4 sums[kJoinWorkers][kJoinRows];
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
  int64_t n1 = 0, n2 = 0, at1 = 0, at2 = 0;
  int prow = 0;
  const int orow = h % kRowsTile;
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
    bool bad;
    if (g >= 0) {
      const Unit x = unit_at(p, g, bad);
      const int64_t i = t * p.H + h - x.rows0, per = x.row_cost();
      if (i >= 0 && i < x.rows && per > 0) {
        const int64_t tile = i / kRowsTile, f = __ldcg(p.plan + 1 + g) + tile * per;
        const int64_t c0 = (f + kSegCost) / each;  // the CTA that has the first key tile
        at1 = c0 + x.part0 + tile;
        n1 = (f + per - 1) / each - c0 + 1;
        prow = static_cast<int>(i % kRowsTile);
      }
    }
    const Unit x = unit_at(p, p.G + t, bad);
    const int64_t per = x.row_cost(), tile = h / kRowsTile;
    if (per > 0) {
      const int64_t f = __ldcg(p.plan + 1 + p.G + t) + tile * per;
      const int64_t c0 = (f + kSegCost) / each;
      at2 = c0 + x.part0 + tile;
      n2 = (f + per - 1) / each - c0 + 1;
    }
  }
  const int n = static_cast<int>(n1 + n2);
  auto part_of = [&](int i, int& rows, int& r) -> const uint8_t* {
    if (i < n1) {
      rows = kRowsTile;
      r = prow;
      return p.prefix_part + (at1 + i) * part_bytes(kRowsTile);
    }
    rows = p.own_rows;
    r = orow;
    return p.own_part + (at2 + i - n1) * part_bytes(p.own_rows);
  };

  // ---- weights
  float top = -INFINITY;
  for (int i = wk; i < n; i += kJoinWorkers) {
    int rows, r;
    const uint8_t* part = part_of(i, rows, r);
    const float m = __ldcg(reinterpret_cast<const float*>(part + static_cast<int64_t>(rows) * kChunks * 16) + r);
    weights[i * kJoinRows + row] = m;
    top = fmaxf(top, m);
  }
  red[wk][row] = top;
  __syncthreads();
  for (int i = 0; i < kJoinWorkers; ++i) top = fmaxf(top, red[i][row]);
  __syncthreads();
  const float ref = top == -INFINITY ? 0.0f : top;
  float den = 0.0f;
  for (int i = wk; i < n; i += kJoinWorkers) {
    int rows, r;
    const uint8_t* part = part_of(i, rows, r);
    const float l = __ldcg(reinterpret_cast<const float*>(part + static_cast<int64_t>(rows) * kChunks * 16) + rows + r);
    const float w = exp2f(weights[i * kJoinRows + row] - ref);
    weights[i * kJoinRows + row] = w;
    den += w * l;
  }
  red[wk][row] = den;
  __syncthreads();
  den = 0.0f;
  for (int i = 0; i < kJoinWorkers; ++i) den += red[i][row];
  if (live && slice == 0 && wk == 0 && p.lse != nullptr)
    p.lse[t * p.H + h] = den > 0.0f || den != den ? (ref + log2f(den)) * 0.6931471805599453f : -INFINITY;
  float mul = den > 0.0f || den != den ? 1.0f / den : 0.0f;
  if (p.kv_scale != nullptr) mul *= __ldcg(p.kv_scale);

  // ---- sums: `per` chunks of 4 columns in this slice, cw of them at a time, 16 / cw segment classes
  const int per = kChunks / slices;
  const int cw = per < kJoinWorkers ? per : kJoinWorkers;
  const int classes = kJoinWorkers / cw;
  const int cls = wk / cw;
  for (int c0 = 0; c0 < per; c0 += cw) {
    const int chunk = slice * per + c0 + wk % cw;
    float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 4
    for (int i = cls; i < n; i += classes) {
      int rows, r;
      const uint8_t* part = part_of(i, rows, r);
      const float4 o = __ldcg(reinterpret_cast<const float4*>(part) + static_cast<int64_t>(chunk) * rows + r);
      const float w = weights[i * kJoinRows + row];
      acc.x += w * o.x;
      acc.y += w * o.y;
      acc.z += w * o.z;
      acc.w += w * o.w;
    }
    if (classes > 1) {
      __syncthreads();
      sums[wk][row] = make_uint4(__float_as_uint(acc.x), __float_as_uint(acc.y), __float_as_uint(acc.z),
                                 __float_as_uint(acc.w));
      __syncthreads();
      if (cls == 0) {
        for (int i = 1; i < classes; ++i) {
          const uint4 o = sums[i * cw + wk % cw][row];
          acc.x += __uint_as_float(o.x);
          acc.y += __uint_as_float(o.y);
          acc.z += __uint_as_float(o.z);
          acc.w += __uint_as_float(o.w);
        }
      }
    }
    if (live && cls == 0) {
      uint2 o = make_uint2(pack_bf16x2(acc.x * mul, acc.y * mul), pack_bf16x2(acc.z * mul, acc.w * mul));
      if (n == 0) o = make_uint2(0, 0);
      *reinterpret_cast<uint2*>(p.out + (t * p.H + h) * kDv + 4 * chunk) = o;
    }
  }
  pdl_trigger();
}

// ---- host ------------------------------------------------------------------------------

struct Layout {
  int64_t prefix_part, own_part, bytes;
};

Layout layout_of(int64_t T, int64_t H, int64_t G, int64_t ctas) {
  auto up = [](int64_t v) { return (v + 255) / 256 * 256; };
  Layout l;
  l.prefix_part = up(8 * (1 + G + T));
  const int64_t prefix_parts = G > 0 ? T * H / kRowsTile + G + 1 + ctas : 0;
  l.own_part = up(l.prefix_part + prefix_parts * part_bytes(kRowsTile));
  const int64_t own_parts = T * ((H + kRowsTile - 1) / kRowsTile) + ctas;
  l.bytes = up(l.own_part + own_parts * part_bytes(static_cast<int>(H < kRowsTile ? H : kRowsTile)));
  return l;
}

template <int FMT, bool F16>
const void* kernel_for() {
  return reinterpret_cast<const void*>(&attend_kernel<FMT, F16>);
}

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) % n) == 0; }

std::atomic<bool> g_smem_ready[kMaxDevices][4];

bool sizes_ok(int64_t T, int64_t H, int64_t G) {
  return T >= 0 && H >= 1 && H <= 65535 && T <= (static_cast<int64_t>(INT_MAX) - kRowsTile) / H && G >= 0 && G <= T;
}

mla_status launch(const void* fn, int64_t blocks, int threads, size_t smem, bool pdl, mla_stream_t stream,
                  void** args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(blocks), 1, 1);
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

mla_status mla_prefix_attend_workspace(int64_t T, int64_t H, int64_t G, int32_t sm_count, int64_t* bytes) {
  using namespace mla::attend;
  if (bytes == nullptr || !sizes_ok(T, H, G)) return MLA_ERR_INVALID_ARG;
  if (sm_count <= 0) {
    const mla_status s = mla::current_device(nullptr, &sm_count);
    if (s != MLA_OK) return s;
  }
  *bytes = layout_of(T, H, G, sm_count).bytes;
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
  if (!sizes_ok(T, H, G) || block_size < 1 || block_size > INT_MAX || num_blocks < 0 || table_cols < 0 ||
      table_cols > INT_MAX || table_stride < 0 || prefix_cols < 0 || prefix_cols > INT_MAX || prefix_stride < 0)
    return MLA_ERR_INVALID_ARG;
  if (num_blocks > (INT64_C(1) << 50) / block_size) return MLA_ERR_INVALID_ARG;
  if (!std::isfinite(sm_scale)) return MLA_ERR_INVALID_ARG;
  if (T == 0) return MLA_OK;
  const bool q8 = (flags & MLA_FLAG_Q_FP8) != 0;
  if (q == nullptr || cache == nullptr || out == nullptr || workspace == nullptr) return MLA_ERR_INVALID_ARG;
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
  const Layout lay = layout_of(T, H, G, sms);
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
  p.prefix_part = ws + lay.prefix_part;
  p.own_part = ws + lay.own_part;
  p.own_rows = static_cast<int32_t>(H < kRowsTile ? H : kRowsTile);
  p.ctas = sms;
  p.status = status;

  static const void* const kernels[4] = {kernel_for<MLA_CACHE_BF16, false>(), kernel_for<MLA_CACHE_E4M3, false>(),
                                         kernel_for<MLA_CACHE_MX, false>(), kernel_for<MLA_CACHE_E4M3, true>()};
  const int k = format == MLA_CACHE_E4M3 && q8 ? 3 : format;
  if (!g_smem_ready[dev][k].load(std::memory_order_acquire)) {
    // idempotent: two threads racing here both set the same attribute
    const cudaError_t e =
        cudaFuncSetAttribute(kernels[k], cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(kSmemBytes));
    if (e != cudaSuccess) return mla::cuda_failure(e);
    g_smem_ready[dev][k].store(true, std::memory_order_release);
  }
  void* args[] = {&p};
  s = launch(kernels[k], sms, kThreads, kSmemBytes, (flags & MLA_FLAG_PDL) != 0, stream, args);
  if (s != MLA_OK) return s;

  const int64_t rows = T * ((H + kJoinRows - 1) / kJoinRows);
  int32_t slices = 1;
  while (slices < 32 && rows * slices < 8 * sms) slices *= 2;
  void* jargs[] = {&p, &slices};
  return launch(reinterpret_cast<const void*>(&join_kernel), rows * slices, kJoinThreads,
                static_cast<size_t>(2 * sms) * kJoinRows * sizeof(float), true, stream, jargs);
}

}  // extern "C"
