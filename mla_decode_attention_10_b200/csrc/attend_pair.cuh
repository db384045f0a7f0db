// attend_pair.cuh -- prefixes of groups with many rows, on pairs of CTAs
// (included by mla_attend.cu, inside its namespace).
//
// Two CTAs of a cluster share one tensor-core product of M = 128 rows
// (cta_group::2): each holds 64 of the rows with their sums, and half of the
// other operand.  In a step of 128 keys CTA r reads the keys of tile 2 i + r for
// the scores, and 128 of each 256 value columns of both tiles for the sums.
// Per 64 keys and SM that is 1090 cycles of products (measured; 1794 on one SM,
// where every operand is read for 64 rows only) and 70 KB of copies, like one
// SM's 72 KB for half the work.
//
// Rows and keys come from the decoded tiles in the workspace, so the loaders
// are bulk copies: the keys' slabs, and the values' again in another cut
// (the products read their operands from one CTA's shared memory each, and
// the two cuts share a quarter of the data only).
//
// Shared memory holds q (72 KB), one step's keys (72 KB) and values (64 KB), and
// the weights (16 KB).  Keys are freed by halves as their products complete
// and refilled while softmax and sums run; values the other way round.
//
// Roles as in the single kernel: 8 softmax warps, an MMA warp (the leader's
// issues; the other CTA's forwards "filled" to the leader), 4 loader warps.
// Barriers that the MMA waits on count both CTAs and are the leader's; what it
// commits arrives in both CTAs.

constexpr uint32_t kPairV = 4 * 2 * kSlabBytes;   // four 64-column slabs of 128 keys
constexpr uint32_t kPairP = 2 * kSlabBytes;       // 64 rows x 128 keys
constexpr uint32_t kPairSmem = 2 * Shape<kBf16>::kTile + kPairV + kPairP + 1024;

struct PairBars {
  uint64_t k_full[2], k_empty[2];  // by half: slabs 0..3 and the rotary slab, slabs 4..7
  uint64_t v_full, v_empty[2];     // by half of the value columns
  uint64_t f_full[4];              // a step's key flags, by step
  uint64_t q_full, q_empty;
  uint64_t s_full[2], s_empty[2];
  uint64_t p_full[2], pv_done[2], o_empty;
  uint64_t drained;
};

struct PairShared {
  PairBars bars;
  uint32_t tmem;
  uint32_t abort_flag;
  uint32_t never;  // stays 0
  alignas(16) uint8_t valid[4][2 * kKeys];  // 1: the key counts, by step
  float xch[4][kRowsTile];
  int64_t warp_sum[kThreads / 32];
  int64_t first_unit, first_base;
  Unit unit;
};

__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// One MMA of the pair, issued by one lane of the leader's warp.
template <bool ACCUMULATE>
__device__ __forceinline__ void mma_pair(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "elect.sync _|q, 0xffffffff;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "@q tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "n"(ACCUMULATE ? 1 : 0)
      : "memory");
}

// All the pair's MMAs issued so far arrive on the barrier of both CTAs when they have completed.
__device__ __forceinline__ void commit_pair(uint32_t bar) {
  if (elect_one())
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(bar),
        "h"(static_cast<uint16_t>(3))
        : "memory");
  __syncwarp();
}

// Which of seven phases have completed, as bits (see ask); arrivals of the other CTA are acquired.
__device__ __forceinline__ uint32_t ask_pair(const uint32_t (&bar)[7], const uint32_t (&parity)[7]) {
  uint32_t bits;
  asm volatile(
      "{\n\t.reg .pred q, p0, p1, p2, p3, p4, p5, p6;\n\t"
      ".reg .b32 a, b, c;\n\t"
      "setp.ne.b32 p0, 0, 0;\n\t"
      "setp.ne.b32 p1, 0, 0;\n\t"
      "setp.ne.b32 p2, 0, 0;\n\t"
      "setp.ne.b32 p3, 0, 0;\n\t"
      "setp.ne.b32 p4, 0, 0;\n\t"
      "setp.ne.b32 p5, 0, 0;\n\t"
      "setp.ne.b32 p6, 0, 0;\n\t"
      "elect.sync _|q, 0xffffffff;\n\t"
      "@q mbarrier.test_wait.parity.acquire.cluster.shared::cta.b64 p0, [%1], %8;\n\t"
      "@q mbarrier.test_wait.parity.acquire.cluster.shared::cta.b64 p1, [%2], %9;\n\t"
      "@q mbarrier.test_wait.parity.acquire.cluster.shared::cta.b64 p2, [%3], %10;\n\t"
      "@q mbarrier.test_wait.parity.acquire.cluster.shared::cta.b64 p3, [%4], %11;\n\t"
      "@q mbarrier.test_wait.parity.acquire.cluster.shared::cta.b64 p4, [%5], %12;\n\t"
      "@q mbarrier.test_wait.parity.acquire.cluster.shared::cta.b64 p5, [%6], %13;\n\t"
      "@q mbarrier.test_wait.parity.acquire.cluster.shared::cta.b64 p6, [%7], %14;\n\t"
      "selp.u32 a, 1, 0, p0;\n\t"
      "selp.u32 b, 2, 0, p1;\n\t"
      "or.b32 a, a, b;\n\t"
      "selp.u32 b, 4, 0, p2;\n\t"
      "selp.u32 c, 8, 0, p3;\n\t"
      "or.b32 b, b, c;\n\t"
      "or.b32 a, a, b;\n\t"
      "selp.u32 b, 16, 0, p4;\n\t"
      "selp.u32 c, 32, 0, p5;\n\t"
      "or.b32 b, b, c;\n\t"
      "selp.u32 c, 64, 0, p6;\n\t"
      "or.b32 b, b, c;\n\t"
      "or.b32 %0, a, b;\n\t}"
      : "=r"(bits)
      : "r"(bar[0]), "r"(bar[1]), "r"(bar[2]), "r"(bar[3]), "r"(bar[4]), "r"(bar[5]), "r"(bar[6]), "r"(parity[0]),
        "r"(parity[1]), "r"(parity[2]), "r"(parity[3]), "r"(parity[4]), "r"(parity[5]), "r"(parity[6])
      : "memory");
  return __reduce_or_sync(0xffffffffu, bits);
}

// Whether an event loop must give up: too many rounds without an event, or another role did.
__device__ __forceinline__ bool gave_up(const Params& p, uint32_t& idle, volatile uint32_t* ab) {
  const bool out = ++idle > kWaitSpins;
  if (!out && ((idle & 15u) != 15u || !__any_sync(0xffffffffu, *ab != 0u))) return false;
  if ((threadIdx.x & 31u) == 0u && *ab == 0u) {
    *ab = 1u;
    report(p.status, MLA_STATUS_TIMEOUT);
  }
  return true;
}

// The leader's MMA warp.
__device__ __forceinline__ void pair_mma(const Params& p, Cursor cur, PairShared& sh, uint32_t sQ, uint32_t sK,
                                         uint32_t sV, uint32_t sP, uint32_t tmem) {
  constexpr uint32_t kM = (128u >> 4) << 24;
  constexpr uint32_t kQk = (instr_desc<kBf16>(2 * kKeys, false) & 0x00ffffffu) | kM;
  constexpr uint32_t kPv = (instr_desc<kBf16>(256, true) & 0x00ffffffu) | kM;
  volatile uint32_t* ab = &sh.abort_flag;
  const uint64_t dQ = smem_desc(sQ, 16, 1024), dK = smem_desc(sK, 16, 1024);
  const uint64_t dP = smem_desc(sP, 16, 1024), dV = smem_desc(sV, 2 * kSlabBytes, 1024);
  uint32_t s = 0, v = 0;        // the next step to get scores, and sums: v <= s <= v + 2
  bool begun = false;           // step s has its first half's scores
  uint32_t seg = 0, v_seg = 0;  // segments begun, and whose sums have begun
  int left = 0;                 // steps of the current segment without scores
  bool more = true, first = false;
  uint32_t first_bits = 0;      // bit (i & 1): step i is its segment's first
  uint32_t idle = 0;
  while (true) {
    if (left == 0 && more) {
      Segment x;
      left = uniform(next_segment<true>(p, cur, x) ? x.k1 - x.k0 : 0);
      more = left > 0;
      first = true;
      if (more) ++seg;
    }
    if (left == 0 && v == s) break;
    const uint32_t buf = s & 1u;
    const uint32_t bars[7] = {smem_u32(&sh.bars.p_full[v & 1u]), smem_u32(&sh.bars.o_empty),
                              smem_u32(&sh.bars.k_full[0]),      smem_u32(&sh.bars.k_full[1]),
                              smem_u32(&sh.bars.q_full),         smem_u32(&sh.bars.s_empty[buf]),
                              smem_u32(&sh.bars.v_full)};
    const uint32_t parities[7] = {(v / 2) & 1u,   (v_seg - 1) & 1u,   s & 1u, s & 1u,
                                  (seg - 1) & 1u, (s / 2 - 1) & 1u, v & 1u};
    const uint32_t got = ask_pair(bars, parities);
    const bool opens = ((first_bits >> (v & 1u)) & 1u) != 0u;
    if (v < s && (got & 1u) != 0u && (got & 64u) != 0u && (!opens || v_seg == 0 || (got & 2u) != 0u)) {
      fence_after();
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        const uint32_t d = tmem + static_cast<uint32_t>(half) * 128u;
        const uint64_t vh = dV + static_cast<uint64_t>(half) * (4 * kSlabBytes >> 4);
        if (opens) {
          mma_pair<false>(d, dP, vh, kPv);
        } else {
          mma_pair<true>(d, dP, vh, kPv);
        }
#pragma unroll
        for (int j = 1; j < 8; ++j)
          mma_pair<true>(d, dP + static_cast<uint64_t>((j >> 2) * (kSlabBytes >> 4) + (j & 3) * 2),
                         vh + static_cast<uint64_t>(j * 128), kPv);
        commit_pair(smem_u32(&sh.bars.v_empty[half]));
      }
      commit_pair(smem_u32(&sh.bars.pv_done[v & 1u]));
      if (opens) ++v_seg;
      ++v;
      idle = 0;
      continue;
    }
    const uint32_t d = tmem + kTmemS + 64u * buf;
    bool went = false;
    if (left > 0 && !begun && s < v + 2 && (got & 4u) != 0u && (!first || (got & 16u) != 0u) &&
        (s < 2 || (got & 32u) != 0u)) {
      fence_async();
      fence_after();
#pragma unroll
      for (int j = 0; j < 20; ++j) {  // the rotary slab, then slabs 0..3
        const int slab = j < 4 ? 8 : (j >> 2) - 1;
        const uint64_t off = static_cast<uint64_t>(slab * (kSlabBytes >> 4) + (j & 3) * 2);
        if (j == 0) {
          mma_pair<false>(d, dQ + off, dK + off, kQk);
        } else {
          mma_pair<true>(d, dQ + off, dK + off, kQk);
        }
      }
      commit_pair(smem_u32(&sh.bars.k_empty[0]));
      begun = went = true;
    }
    if (begun && (got & 8u) != 0u) {
      fence_async();
      fence_after();
#pragma unroll
      for (int j = 16; j < 32; ++j) {
        const uint64_t off = static_cast<uint64_t>((j >> 2) * (kSlabBytes >> 4) + (j & 3) * 2);
        mma_pair<true>(d, dQ + off, dK + off, kQk);
      }
      commit_pair(smem_u32(&sh.bars.k_empty[1]));
      commit_pair(smem_u32(&sh.bars.s_full[buf]));
      --left;
      if (left == 0) commit_pair(smem_u32(&sh.bars.q_empty));
      first_bits = (first_bits & ~(1u << buf)) | ((first ? 1u : 0u) << buf);
      first = false;
      begun = false;
      went = true;
      ++s;
    }
    if (went) {
      idle = 0;
      continue;
    }
    if (gave_up(p, idle, ab)) break;
  }
  // every product issued has completed before TMEM is freed
  commit_pair(smem_u32(&sh.bars.drained));
}

// The other CTA's MMA warp: tells the leader what has been filled here.
__device__ __forceinline__ void pair_relay(const Params& p, Cursor cur, PairShared& sh) {
  volatile uint32_t* ab = &sh.abort_flag;
  uint32_t steps = 0, segs = 0;
  while (true) {
    Segment x;
    const int n = uniform(next_segment<true>(p, cur, x, 1) ? x.k1 - x.k0 : 0);
    if (n == 0) break;
    steps += static_cast<uint32_t>(n);
    ++segs;
  }
  uint32_t k0 = 0, k1 = 0, v = 0, q = 0, idle = 0;
  while (k0 < steps || k1 < steps || v < steps || q < segs) {
    const uint32_t bars[6] = {smem_u32(&sh.bars.k_full[0]), smem_u32(&sh.bars.k_full[1]), smem_u32(&sh.bars.v_full),
                              smem_u32(&sh.bars.q_full),    smem_u32(&sh.bars.q_full),    smem_u32(&sh.bars.q_full)};
    const uint32_t parities[6] = {k0 & 1u, k1 & 1u, v & 1u, q & 1u, q & 1u, q & 1u};
    const uint32_t got = ask(bars, parities);
    bool went = false;
    auto pass = [&](bool ready, uint64_t* bar, uint32_t& n) {
      if (!ready) return;
      fence_async();  // q rows may have come by plain stores and copies
      if (elect_one()) arrive_leader(smem_u32(bar));
      __syncwarp();
      ++n;
      went = true;
    };
    pass(q < segs && (got & 8u) != 0u, &sh.bars.q_full, q);
    pass(k0 < steps && (got & 1u) != 0u, &sh.bars.k_full[0], k0);
    pass(k1 < steps && (got & 2u) != 0u, &sh.bars.k_full[1], k1);
    pass(v < steps && (got & 4u) != 0u, &sh.bars.v_full, v);
    if (went) {
      idle = 0;
    } else if (gave_up(p, idle, ab)) {
      break;
    }
  }
}

// Loader warps: warp 0 fills the keys, warp 1 the values, all four the q rows.
__device__ __forceinline__ bool pair_load(const Params& p, Cursor cur, PairShared& sh, uint32_t sQ, uint32_t sK,
                                          uint32_t sV, int rank, int warp) {
  using S = Shape<kBf16>;
  const int lane = static_cast<int>(threadIdx.x) & 31;
  volatile uint32_t* ab = &sh.abort_flag;
  uint32_t it = 0, nseg = 0;
  Segment seg;
  while (uniform(next_segment<true>(p, cur, seg, rank) ? 1 : 0) != 0) {
    // the segment's q rows, once the previous segment's scores have been computed
    if (nseg > 0 && !warp_wait(smem_u32(&sh.bars.q_empty), (nseg - 1) & 1u, ab)) return false;
    load_q<MLA_CACHE_BF16, kBf16>(p, static_cast<int32_t>(seg.row0), seg.rows, sQ, smem_u32(&sh.bars.q_full), warp, lane);
    ++nseg;
    if (warp > 1) continue;
    const uint8_t* tiles = p.image + seg.u * p.image_tiles * kImage;
    const int steps = uniform(seg.k1 - seg.k0);
    for (int i = 0; i < steps; ++i, ++it) {
      const uint8_t* t0 = tiles + 2 * static_cast<int64_t>(seg.k0 + i) * kImage;  // the step's two tiles
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        constexpr uint32_t kHalf = S::kHalfSlabs * kSlabBytes;
        const uint32_t empty = smem_u32(warp == 0 ? &sh.bars.k_empty[h] : &sh.bars.v_empty[h]);
        if (it > 0 && !warp_wait(empty, (it - 1) & 1u, ab)) return false;
        if (elect_one()) {
          if (warp == 0) {
            const uint32_t full = smem_u32(&sh.bars.k_full[h]);
            const uint8_t* mine = t0 + rank * kImage;
            arrive_expect(full, kHalf + (h == 0 ? kSlabBytes : 0));
            bulk_copy(sK + h * kHalf, mine + h * kHalf, kHalf, full);
            if (h == 0) {
              bulk_copy(sK + S::kPeSlab * kSlabBytes, mine + S::kPeSlab * kSlabBytes, kSlabBytes, full);
              // Flags have four slots: step i + 4's keys are fetched only behind the scores of
              // i + 3, which wait for the softmax of i + 1, so the slot's reader is done.
              const uint32_t flags = smem_u32(&sh.bars.f_full[it & 3u]);
              arrive_expect(flags, 2 * kKeys);
              bulk_copy(smem_u32(sh.valid[it & 3u]), t0 + S::kTile, kKeys, flags);
              bulk_copy(smem_u32(sh.valid[it & 3u]) + kKeys, t0 + kImage + S::kTile, kKeys, flags);
            }
          } else {
            // value columns 256 h + 128 rank ..: slabs 4 h + 2 rank and the next, of both tiles
            const uint32_t full = smem_u32(&sh.bars.v_full);
            if (h == 0) {
              asm volatile("mbarrier.expect_tx.relaxed.cta.shared::cta.b64 [%0], %1;" ::"r"(full), "r"(kPairV / 2) : "memory");
            } else {
              arrive_expect(full, kPairV / 2);
            }
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              const uint32_t slab = static_cast<uint32_t>(4 * h + 2 * rank + j) * kSlabBytes;
              const uint32_t dst = sV + static_cast<uint32_t>(2 * h + j) * 2u * kSlabBytes;
              bulk_copy(dst, t0 + slab, kSlabBytes, full);
              bulk_copy(dst + kSlabBytes, t0 + kImage + slab, kSlabBytes, full);
            }
          }
        }
        __syncwarp();
      }
    }
  }
  return true;
}

__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1) pair_kernel(const Params p, int e4m3) {
  using S = Shape<kBf16>;
  using R = Roles<MLA_CACHE_BF16, kBf16>;
  extern __shared__ uint8_t dsmem[];
  __shared__ PairShared sh;
  const int warp = uniform(static_cast<int>(threadIdx.x) >> 5);
  const int rank = static_cast<int>(blockIdx.x) & 1;  // clusters are neighbouring blocks
  const uint32_t sQ = (smem_u32(dsmem) + 1023u) & ~1023u;
  const uint32_t sK = sQ + S::kTile;
  const uint32_t sV = sK + S::kTile;
  const uint32_t sP = sV + kPairV;
  if (warp == R::kMma) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&sh.tmem)),
                 "r"(kTmemCols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  }
  if (threadIdx.x == 0) {
    sh.abort_flag = 0u;
    sh.never = 0u;
    sh.first_unit = 0;
    sh.first_base = 0;
    auto init = [](uint64_t* b, uint32_t n) {
      asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(smem_u32(b)), "r"(n) : "memory");
    };
    // filled: the leader's also count the other CTA's
    const uint32_t peer = rank == 0 ? 1 : 0;
    for (int i = 0; i < 2; ++i) {
      init(&sh.bars.k_full[i], 1 + peer);
      init(&sh.bars.k_empty[i], 1);
      init(&sh.bars.v_empty[i], 1);
      init(&sh.bars.s_full[i], 1);
      init(&sh.bars.s_empty[i], 2 * R::kSoft);
      init(&sh.bars.p_full[i], 2 * R::kSoft);
      init(&sh.bars.pv_done[i], 1);
    }
    for (int i = 0; i < 4; ++i) init(&sh.bars.f_full[i], 1);
    init(&sh.bars.v_full, 1 + peer);
    init(&sh.bars.q_full, 32 * R::kLoad + peer);
    init(&sh.bars.q_empty, 1);
    init(&sh.bars.o_empty, 2 * R::kSoft);
    init(&sh.bars.drained, 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  pdl_wait();
  pdl_trigger();
  fence_before();
  __syncwarp();
  cluster_sync();
  fence_after();
  const uint32_t tmem = static_cast<uint32_t>(uniform(static_cast<int>(sh.tmem)));
  const Cursor cur = plan_run(p, sh, 0, p.G, blockIdx.x / 2, gridDim.x / 2, 1);
  const bool work = uniform(cur.pos < cur.end ? 1 : 0) != 0;
  if (work) {
    if (warp < R::kSoft) {
      float scale2 = p.sm_scale * 1.4426950408889634f;  // powers of two: log2(e)
      if (p.q_fp8) scale2 *= __ldcg(p.q_scale);
      if (e4m3 != 0) scale2 *= __ldcg(p.kv_scale);
      softmax_role<kBf16, R::kSoft, true>(p, cur, sh, sP, tmem, scale2, rank);
    } else if (warp == R::kMma) {
      if (rank == 0) {
        pair_mma(p, cur, sh, sQ, sK, sV, sP, tmem);
      } else {
        pair_relay(p, cur, sh);
      }
      (void)warp_wait(smem_u32(&sh.bars.drained), 0u, &sh.never);
    } else {
      const bool good = pair_load(p, cur, sh, sQ, sK, sV, rank, warp - R::kLoad0);
      // no copy may be under way when the CTA ends: on the way out after a timeout
      // (else every copy has been used) give the copy engine's theirs
      asm volatile("cp.async.wait_all;" ::: "memory");
      if (!good) {
        for (uint32_t parity = 0; parity < 2; ++parity) {
          (void)warp_wait(smem_u32(&sh.bars.k_full[0]), parity, &sh.never);
          (void)warp_wait(smem_u32(&sh.bars.k_full[1]), parity, &sh.never);
          (void)warp_wait(smem_u32(&sh.bars.v_full), parity, &sh.never);
          for (int i = 0; i < 4; ++i) (void)warp_wait(smem_u32(&sh.bars.f_full[i]), parity, &sh.never);
        }
        if ((threadIdx.x & 31u) == 0u && *reinterpret_cast<volatile uint32_t*>(&sh.abort_flag) == 0u) {
          *reinterpret_cast<volatile uint32_t*>(&sh.abort_flag) = 1u;
          report(p.status, MLA_STATUS_TIMEOUT);
        }
      }
    }
  }
  fence_before();
  __syncwarp();
  cluster_sync();  // neither CTA ends while the other may still arrive on its barriers
  if (warp == R::kMma) {
    fence_after();
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTmemCols) : "memory");
  }
}
