// mla_latent.cu -- latent cache rows written with a norm, the rotation and
// microscaled codes in one pass, and read back as bf16 rows (contracts in
// mla_epilogue.h).
//
// Both kernels move bytes: a row costs 1.2 + 0.6 to 1.2 KB of traffic and a
// few operations per value, so they are bound by HBM at large sizes and by the
// chain of dependent loads at decode sizes.

#include <atomic>
#include <climits>
#include <cmath>
#include <cstdint>
#include <cuda_runtime.h>

#include "epilogue_device.cuh"
#include "latent_rows.cuh"
#include "mla_runtime.h"

namespace mla {
namespace latent {

// ------------------------------------------------------------------------------------
// insert: one warp per token.  Lane l holds the latents 16 l .. 16 l + 15 (32
// contiguous bytes in, 16 codes out) and the rotary pair (l, l + 32), so a
// group of 32 latents is a pair of lanes and the norm's sum one warp reduction.
// ------------------------------------------------------------------------------------

struct InsertArgs {
  const uint16_t* kv_c;
  int64_t kv_st;
  const uint16_t* k_pe;
  int64_t kp_st;
  const int64_t* slots;
  const uint16_t* norm_w;
  double eps;
  const int32_t* positions;
  const float* cos_sin;
  int64_t rope_rows;
  const float* kv_scale;
  int64_t T;
  int64_t cache_rows;
  uint8_t* cache;
  int32_t* status;
};

// The least e with a <= 448 * 2^e for a >= 0 finite, kept within the format's
// range: a = m * 2^x with m in [1, 2) needs e = x - 8 while m <= 1.75 (448 =
// 1.75 * 2^8), else x - 7.
__device__ __forceinline__ int mx_exponent(float a) {
  const uint32_t u = __float_as_uint(a);
  const int e = static_cast<int>(u >> 23) - 127 - 8 + ((u & 0x7fffffu) > 0x600000u ? 1 : 0);
  return min(max(e, kMxMinExp), kMxMaxExp);  // zero and subnormals fall to the minimum
}

// x rounded to e4m3 after a product with a power of two (exact unless it
// leaves the normal range, and then far below the smallest code).
__device__ __forceinline__ uint32_t codes4(const float* y, float mul) {
  return pack_e4m3x2(__fmul_rn(y[0], mul), __fmul_rn(y[1], mul)) |
         (pack_e4m3x2(__fmul_rn(y[2], mul), __fmul_rn(y[3], mul)) << 16);
}

template <int FMT, bool ROPE>
__global__ void __launch_bounds__(128, 6) insert_kernel(const InsertArgs a) {
  const int lane = static_cast<int>(threadIdx.x) & 31;
  const int64_t t = static_cast<int64_t>(blockIdx.x) * (blockDim.x >> 5) + (threadIdx.x >> 5);
  if (t >= a.T) {
    pdl_trigger();
    return;
  }
  // what no upstream kernel writes: slot, position, table row, scale, norm weights
  const int64_t slot = __ldg(a.slots + t);
  Rot rot{1.0f, 0.0f, false};
  if constexpr (ROPE) rot = load_rotation(a.positions, a.cos_sin, a.rope_rows, t, lane);
  float scale = 1.0f;
  if constexpr (FMT == MLA_CACHE_E4M3) scale = __ldg(a.kv_scale);
  uint4 w0 = make_uint4(0, 0, 0, 0), w1 = w0;
  if (a.norm_w != nullptr) {
    w0 = __ldg(reinterpret_cast<const uint4*>(a.norm_w) + 2 * lane);
    w1 = __ldg(reinterpret_cast<const uint4*>(a.norm_w) + 2 * lane + 1);
  }
  pdl_wait();
  const uint16_t* src = a.kv_c + t * a.kv_st;
  const uint4 v0 = ld_chunk(src, 2 * lane);
  const uint4 v1 = ld_chunk(src, 2 * lane + 1);
  const uint32_t pe = ld_pair(a.k_pe + t * a.kp_st, lane);
  if (lane == 0) {
    if (slot >= a.cache_rows) report(a.status, MLA_STATUS_SLOT_RANGE);
    if (ROPE && !rot.on) report(a.status, MLA_STATUS_POS_RANGE);
  }
  if (slot >= 0 && slot < a.cache_rows) {
    const uint32_t xw[8] = {v0.x, v0.y, v0.z, v0.w, v1.x, v1.y, v1.z, v1.w};
    const uint32_t ww[8] = {w0.x, w0.y, w0.z, w0.w, w1.x, w1.y, w1.z, w1.w};
    float y[16];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      y[2 * i] = bf16_lo(xw[i]);
      y[2 * i + 1] = bf16_hi(xw[i]);
    }
    if (a.norm_w != nullptr) {
      // The sum of squares, its root and the products are held in 64 bits and
      // y is rounded once to fp32: a code next to a rounding border is then
      // the one of the exact formula, whatever the order of the sum.
      double s = 0.0;
#pragma unroll
      for (int i = 0; i < 16; ++i) s = fma(static_cast<double>(y[i]), static_cast<double>(y[i]), s);
#pragma unroll
      for (int m = 16; m > 0; m >>= 1) s += __shfl_xor_sync(0xffffffffu, s, m);
      const double r = 1.0 / sqrt(s * (1.0 / 512.0) + a.eps);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        y[2 * i] = static_cast<float>(static_cast<double>(y[2 * i]) * r * static_cast<double>(bf16_lo(ww[i])));
        y[2 * i + 1] =
            static_cast<float>(static_cast<double>(y[2 * i + 1]) * r * static_cast<double>(bf16_hi(ww[i])));
      }
    }
    uint8_t* dst = a.cache + slot * row_bytes(FMT);
    if constexpr (FMT == MLA_CACHE_BF16) {
      uint4 o0 = v0, o1 = v1;  // without a norm: the input bits
      if (a.norm_w != nullptr) {
        o0 = make_uint4(pack_bf16x2(y[0], y[1]), pack_bf16x2(y[2], y[3]), pack_bf16x2(y[4], y[5]),
                        pack_bf16x2(y[6], y[7]));
        o1 = make_uint4(pack_bf16x2(y[8], y[9]), pack_bf16x2(y[10], y[11]), pack_bf16x2(y[12], y[13]),
                        pack_bf16x2(y[14], y[15]));
      }
      reinterpret_cast<uint4*>(dst)[2 * lane] = o0;
      reinterpret_cast<uint4*>(dst)[2 * lane + 1] = o1;
      store_pe<false, ROPE, true>(dst, lane, pe, rot, Divisor{});
    } else if constexpr (FMT == MLA_CACHE_E4M3) {
      const Divisor d = make_divisor(scale);
      uint32_t o[4];
      if (d.fast) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
          o[i] = e4m3x2_of_f32<true>(y[4 * i], y[4 * i + 1], d) |
                 (e4m3x2_of_f32<true>(y[4 * i + 2], y[4 * i + 3], d) << 16);
        store_pe<true, ROPE, true>(dst, lane, pe, rot, d);
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
          o[i] = e4m3x2_of_f32<false>(y[4 * i], y[4 * i + 1], d) |
                 (e4m3x2_of_f32<false>(y[4 * i + 2], y[4 * i + 3], d) << 16);
        store_pe<true, ROPE, false>(dst, lane, pe, rot, d);
      }
      reinterpret_cast<uint4*>(dst)[lane] = make_uint4(o[0], o[1], o[2], o[3]);
    } else {
      float amax = 0.0f;
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const float m = fabsf(y[i]);
        if (m < INFINITY) amax = fmaxf(amax, m);  // NaN and infinities set no scale
      }
      amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
      const int e = mx_exponent(amax);
      const float mul = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);  // 2^-e, normal for e in [-117, 119]
      reinterpret_cast<uint4*>(dst)[lane] =
          make_uint4(codes4(y, mul), codes4(y + 4, mul), codes4(y + 8, mul), codes4(y + 12, mul));
      if ((lane & 1) == 0) dst[kMxScales + (lane >> 1)] = static_cast<uint8_t>(e + 127);
      // the rotary pair goes where a bf16 row has it, relative to its values 512..575
      store_pe<false, ROPE, true>(dst + kMxPe - 2 * kNope, lane, pe, rot, Divisor{});
    }
  }
  pdl_trigger();
}

// ------------------------------------------------------------------------------------
// gather
// ------------------------------------------------------------------------------------

struct GatherArgs {
  const uint8_t* cache;
  int64_t cache_blocks;
  int32_t block_size;
  const float* kv_scale;
  const int32_t* table;
  int64_t table_stride;
  int64_t table_keys;  // table_cols * block_size
  const int32_t* cu;
  const int32_t* first;
  int64_t B;
  int64_t N;
  uint8_t* out;
  int64_t out_stride;  // bytes
  bool wide;           // rows of out start on 32-byte boundaries
  int32_t* status;
};

// The last b < B with cu[b] <= r, or -1 (32-ary search over the ascending cu:
// each round the warp looks at 32 evenly spaced entries).
__device__ __forceinline__ int64_t sequence_of(const int32_t* cu, int64_t B, int64_t r, int lane) {
  int64_t lo = 0, n = B;  // the count of entries <= r among cu[lo .. lo + n)
  while (n > 0) {
    const int64_t step = (n + 31) / 32;
    const int64_t i = lo + static_cast<int64_t>(lane) * step;
    const bool le = i < lo + n && static_cast<int64_t>(__ldcg(cu + i)) <= r;
    const int c = __popc(__ballot_sync(0xffffffffu, le));
    if (c == 0) return lo - 1;
    const int64_t at = lo + static_cast<int64_t>(c - 1) * step;  // cu[at] <= r
    const int64_t end = lo + n;
    lo = at + 1;
    n = min(step - 1, end - lo);
  }
  return lo - 1;
}

// A warp takes kGatherRows consecutive rows: one search for the first, then lane
// i < kGatherRows finds row i's sequence, page and address, and every row's
// loads are issued before any is stored.  (One row per warp, each with its own
// chain of search, table and row, ran at a third of the copy bandwidth.)
constexpr int kGatherRows = 8;
constexpr int kGatherSteps = 8;  // sequences passed one by one; eight rows lie in eight unless some are empty

// Sixteen values to 32 contiguous bytes.
__device__ __forceinline__ void store32(uint8_t* dst, bool wide, const uint4& a, const uint4& b) {
  if (wide) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(dst), "r"(a.x), "r"(a.y), "r"(a.z),
                 "r"(a.w), "r"(b.x), "r"(b.y), "r"(b.z), "r"(b.w)
                 : "memory");
  } else {
    reinterpret_cast<uint4*>(dst)[0] = a;
    reinterpret_cast<uint4*>(dst)[1] = b;
  }
}

template <int FMT>
__global__ void __launch_bounds__(256) gather_kernel(const GatherArgs a) {
  pdl_wait();
  const int lane = static_cast<int>(threadIdx.x) & 31;
  const int64_t r0 = (static_cast<int64_t>(blockIdx.x) * (blockDim.x >> 5) + (threadIdx.x >> 5)) * kGatherRows;
  if (r0 < a.N) {
    // this lane's row: its address, or null
    const uint8_t* src = nullptr;
    const int64_t r = r0 + lane;
    int64_t b = sequence_of(a.cu, a.B, r0, lane);
    if (lane < kGatherRows && r < a.N) {
      // on from the first row's sequence to the last one that starts at or before r: step by
      // step, and behind many empty ones by bisection (150 K of them one by one: 37 ms)
      int64_t hi = min(b + kGatherSteps, a.B - 1);
      while (b < hi && static_cast<int64_t>(__ldcg(a.cu + b + 1)) <= r) ++b;
      if (b == hi) {
        hi = a.B - 1;
        while (b < hi) {
          const int64_t mid = b + (hi - b + 1) / 2;
          if (static_cast<int64_t>(__ldcg(a.cu + mid)) <= r) b = mid; else hi = mid - 1;
        }
      }
      const int64_t end = b >= 0 ? static_cast<int64_t>(__ldcg(a.cu + b + 1)) : 0;
      if (b >= 0 && r < end) {
        const int64_t k = (a.first != nullptr ? static_cast<int64_t>(__ldcg(a.first + b)) : 0) + r - __ldcg(a.cu + b);
        if (k < 0 || k >= a.table_keys) {
          report(a.status, MLA_STATUS_LEN_RANGE);
        } else {
          const int64_t page = __ldcg(a.table + b * a.table_stride + k / a.block_size);
          if (page < 0 || page >= a.cache_blocks) {
            report(a.status, MLA_STATUS_SLOT_RANGE);
          } else {
            src = a.cache + (page * a.block_size + k % a.block_size) * row_bytes(FMT);
          }
        }
      }
    }
    const uint8_t* rows[kGatherRows];
#pragma unroll
    for (int i = 0; i < kGatherRows; ++i)
      rows[i] = reinterpret_cast<const uint8_t*>(
          __shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(src), i));
    uint8_t* out = a.out + r0 * a.out_stride;
    if constexpr (FMT == MLA_CACHE_BF16) {
      // 72 pieces a row: 64 by all lanes, the other 8 of four rows at a time
#pragma unroll
      for (int h = 0; h < kGatherRows; h += 4) {
        const uint8_t* t = reinterpret_cast<const uint8_t*>(
            __shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(src), h + (lane >> 3)));
        uint4 x[8];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          x[2 * i] = load16(rows[h + i], 16 * lane);
          x[2 * i + 1] = load16(rows[h + i], 512 + 16 * lane);
        }
        const uint4 y = load16(t, 1024 + 16 * (lane & 7));
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          if (rows[h + i] != nullptr) {
            uint4* d = reinterpret_cast<uint4*>(out + (h + i) * a.out_stride);
            d[lane] = x[2 * i];
            d[32 + lane] = x[2 * i + 1];
          }
        }
        if (t != nullptr) reinterpret_cast<uint4*>(out + (h + (lane >> 3)) * a.out_stride)[64 + (lane & 7)] = y;
      }
    } else {
      uint4 c[kGatherRows];
      float scale = 1.0f;
      uint4 scales = make_uint4(0, 0, 0, 0);  // mx: the 16 scale bytes of this lane's row
      if constexpr (FMT == MLA_CACHE_E4M3) scale = __ldcg(a.kv_scale);
      if constexpr (FMT == MLA_CACHE_MX) scales = load16(src, kMxScales);
#pragma unroll
      for (int i = 0; i < kGatherRows; ++i)
        c[i] = load16(rows[i], 16 * lane);
      if constexpr (FMT == MLA_CACHE_E4M3) {
        // the four last pieces of all eight rows
        const uint8_t* t = reinterpret_cast<const uint8_t*>(
            __shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(src), lane >> 2));
        const uint4 p = load16(t, 512 + 16 * (lane & 3));
        uint4 x, y;
        codes_to_bf16(p, scale, x, y);
        if (t != nullptr) store32(out + (lane >> 2) * a.out_stride + 1024 + 32 * (lane & 3), a.wide, x, y);
      } else {
        uint4 p[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const uint8_t* t = reinterpret_cast<const uint8_t*>(
              __shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(src), 4 * h + (lane >> 3)));
          p[h] = load16(t, kMxPe + 16 * (lane & 7));
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int i = 4 * h + (lane >> 3);
          const bool there = __shfl_sync(0xffffffffu, src != nullptr ? 1 : 0, i) != 0;
          if (there) reinterpret_cast<uint4*>(out + i * a.out_stride)[64 + (lane & 7)] = p[h];
        }
      }
#pragma unroll
      for (int i = 0; i < kGatherRows; ++i) {
        float mul = scale;
        if constexpr (FMT == MLA_CACHE_MX) {  // of group lane / 2: word lane / 8, byte lane / 2 % 4
          const uint32_t w0 = __shfl_sync(0xffffffffu, scales.x, i), w1 = __shfl_sync(0xffffffffu, scales.y, i);
          const uint32_t w2 = __shfl_sync(0xffffffffu, scales.z, i), w3 = __shfl_sync(0xffffffffu, scales.w, i);
          const uint32_t word = lane < 16 ? (lane < 8 ? w0 : w1) : (lane < 24 ? w2 : w3);
          mul = mx_scale(word >> (8 * ((lane >> 1) & 3)));
        }
        uint4 x, y;
        codes_to_bf16(c[i], mul, x, y);
        if (rows[i] != nullptr) store32(out + i * a.out_stride + 32 * lane, a.wide, x, y);
      }
    }
  }
  pdl_trigger();
}

template <int FMT, bool ROPE>
const void* insert_for() {
  return reinterpret_cast<const void*>(&insert_kernel<FMT, ROPE>);
}

const void* const kInsertKernels[3][2] = {{insert_for<0, false>(), insert_for<0, true>()},
                                          {insert_for<1, false>(), insert_for<1, true>()},
                                          {insert_for<2, false>(), insert_for<2, true>()}};
const void* const kGatherKernels[3] = {reinterpret_cast<const void*>(&gather_kernel<0>),
                                       reinterpret_cast<const void*>(&gather_kernel<1>),
                                       reinterpret_cast<const void*>(&gather_kernel<2>)};

mla_status launch(const void* fn, int64_t blocks, int threads, bool pdl, mla_stream_t stream, void* arg) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(blocks), 1, 1);
  cfg.blockDim = dim3(static_cast<unsigned>(threads), 1, 1);
  cfg.stream = reinterpret_cast<cudaStream_t>(stream);
  cudaLaunchAttribute attr[1];
  if (pdl) {
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
  }
  void* args[] = {arg};
  const cudaError_t e = cudaLaunchKernelExC(&cfg, fn, args);
  return e == cudaSuccess ? MLA_OK : cuda_failure(e);
}

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) % n) == 0; }

}  // namespace latent
}  // namespace mla

extern "C" {

mla_status mla_latent_insert_launch(const void* kv_c, int64_t kv_c_stride_t, const void* k_pe, int64_t k_pe_stride_t,
                                    const int64_t* slot_mapping, const void* norm_weight, float eps,
                                    const int32_t* positions, const float* cos_sin, int64_t rope_rows,
                                    const float* kv_scale, int64_t T, int64_t block_size, int64_t num_blocks,
                                    int32_t format, uint32_t flags, void* cache, int32_t* status,
                                    mla_stream_t stream) {
  using namespace mla::latent;
  if ((flags & ~(MLA_FLAG_ROPE | MLA_FLAG_PDL)) != 0) return MLA_ERR_UNSUPPORTED;
  if (format < MLA_CACHE_BF16 || format > MLA_CACHE_MX) return MLA_ERR_UNSUPPORTED;
  if (T < 0 || T > INT_MAX || block_size < 1 || num_blocks < 0) return MLA_ERR_INVALID_ARG;
  if (num_blocks > (INT64_C(1) << 50) / block_size) return MLA_ERR_INVALID_ARG;
  if (!(eps >= 0.0f) || !std::isfinite(eps)) return MLA_ERR_INVALID_ARG;
  const bool rope = (flags & MLA_FLAG_ROPE) != 0;
  if (rope && (rope_rows < 1 || rope_rows > (INT64_C(1) << 40))) return MLA_ERR_INVALID_ARG;
  if (T == 0) return MLA_OK;
  const int64_t cache_rows = num_blocks * block_size;
  if (kv_c == nullptr || k_pe == nullptr || slot_mapping == nullptr || (cache == nullptr && cache_rows > 0))
    return MLA_ERR_INVALID_ARG;
  if (rope && (positions == nullptr || cos_sin == nullptr)) return MLA_ERR_INVALID_ARG;
  if (format == MLA_CACHE_E4M3 && kv_scale == nullptr) return MLA_ERR_INVALID_ARG;
  if (kv_c_stride_t < 0 || k_pe_stride_t < 0) return MLA_ERR_INVALID_ARG;
  if (!aligned(kv_c, 16) || (cache != nullptr && !aligned(cache, 16)) || (T > 1 && kv_c_stride_t % 8 != 0) ||
      !aligned(norm_weight, 16))
    return MLA_ERR_ALIGNMENT;
  if (!aligned(k_pe, 2) || !aligned(slot_mapping, 8) || (rope && (!aligned(positions, 4) || !aligned(cos_sin, 4))) ||
      (format == MLA_CACHE_E4M3 && !aligned(kv_scale, 4)) || !aligned(status, 4))
    return MLA_ERR_ALIGNMENT;

  int32_t sms = 0;
  const mla_status s = mla::current_device(nullptr, &sms);
  if (s != MLA_OK) return s;
  InsertArgs a;
  a.kv_c = static_cast<const uint16_t*>(kv_c);
  a.kv_st = kv_c_stride_t;
  a.k_pe = static_cast<const uint16_t*>(k_pe);
  a.kp_st = k_pe_stride_t;
  a.slots = slot_mapping;
  a.norm_w = static_cast<const uint16_t*>(norm_weight);
  a.eps = static_cast<double>(eps);
  a.positions = positions;
  a.cos_sin = cos_sin;
  a.rope_rows = rope ? rope_rows : 0;
  a.kv_scale = kv_scale;
  a.T = T;
  a.cache_rows = cache_rows;
  a.cache = static_cast<uint8_t*>(cache);
  a.status = status;
  // as in the epilogue: one row per block until every SM has one, at most 4 (8192 tokens with norm, rotation and
  // microscaling: 6.2 us with 4 rows a block, 6.8 with 8, 6.6 with 2; six blocks an SM)
  const int64_t per_sm = (T + sms - 1) / sms;
  const int warps = static_cast<int>(per_sm < 4 ? per_sm : 4);
  return launch(kInsertKernels[format][rope ? 1 : 0], (T + warps - 1) / warps, 32 * warps,
                (flags & MLA_FLAG_PDL) != 0, stream, &a);
}

mla_status mla_latent_gather_launch(const void* cache, int32_t format, int64_t block_size, int64_t num_blocks,
                                    const float* kv_scale, const int32_t* block_table, int64_t table_stride,
                                    int64_t table_cols, const int32_t* cu_rows, const int32_t* first, int64_t B,
                                    int64_t N, uint32_t flags, void* out, int64_t out_stride, int32_t* status,
                                    mla_stream_t stream) {
  using namespace mla::latent;
  if ((flags & ~MLA_FLAG_PDL) != 0) return MLA_ERR_UNSUPPORTED;
  if (format < MLA_CACHE_BF16 || format > MLA_CACHE_MX) return MLA_ERR_UNSUPPORTED;
  if (B < 0 || N < 0 || B > INT_MAX || N > INT_MAX || block_size < 1 || block_size > INT_MAX || num_blocks < 0 ||
      table_cols < 0 || table_cols > INT_MAX || table_stride < 0 || out_stride < 0)
    return MLA_ERR_INVALID_ARG;
  if (num_blocks > (INT64_C(1) << 50) / block_size) return MLA_ERR_INVALID_ARG;
  if (B == 0 || N == 0) return MLA_OK;
  if ((cache == nullptr && num_blocks > 0) || block_table == nullptr || cu_rows == nullptr || out == nullptr)
    return MLA_ERR_INVALID_ARG;
  if (format == MLA_CACHE_E4M3 && kv_scale == nullptr) return MLA_ERR_INVALID_ARG;
  if (N > 1 && out_stride < 576) return MLA_ERR_INVALID_ARG;
  if (!aligned(cache, 16) || !aligned(out, 16) || (N > 1 && out_stride % 8 != 0)) return MLA_ERR_ALIGNMENT;
  if (!aligned(block_table, 4) || !aligned(cu_rows, 4) || !aligned(first, 4) || !aligned(status, 4) ||
      (format == MLA_CACHE_E4M3 && !aligned(kv_scale, 4)))
    return MLA_ERR_ALIGNMENT;
  int32_t sms = 0;
  const mla_status s = mla::current_device(nullptr, &sms);
  if (s != MLA_OK) return s;
  GatherArgs a;
  a.cache = static_cast<const uint8_t*>(cache);
  a.cache_blocks = num_blocks;
  a.block_size = static_cast<int32_t>(block_size);
  a.kv_scale = kv_scale;
  a.table = block_table;
  a.table_stride = table_stride;
  a.table_keys = table_cols * block_size;
  a.cu = cu_rows;
  a.first = first;
  a.B = B;
  a.N = N;
  a.out = static_cast<uint8_t*>(out);
  a.out_stride = 2 * out_stride;
  a.wide = aligned(out, 32) && (N == 1 || out_stride % 16 == 0);
  a.status = status;
  // 8 warps a block; while that leaves SMs without one, one warp a block
  const int64_t warps = (N + kGatherRows - 1) / kGatherRows;
  const int per = warps <= sms ? 1 : 8;
  return launch(kGatherKernels[format], (warps + per - 1) / per, 32 * per, (flags & MLA_FLAG_PDL) != 0, stream, &a);
}

}  // extern "C"
