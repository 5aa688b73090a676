// The router's gradient: through the gates, the sigmoid, the balance loss and
// the logits product.  "DeepSeek_V3_Report：Annotation", eqs. (13), (15) and
// (17)-(20).
//
//  1. dlogits_kernel -- one warp per token.  With s = sigmoid(z),
//     g_k = s_k / sum of the chosen s and s' = s / sum of all s, both
//     normalisations have the same gradient,
//       d(sum_k a_k g_k)/dz_i = g_i (1 - s_i) (a_i - sum_j g_j a_j),
//     with a = dgate for the gates and a = dloss alpha f / S for the balance
//     loss.  The gates are given, so their sum is not needed; that of all s
//     is, and where it is tiny the s' come from e^(z - max z).  1 - s is
//     1 / (1 + e^z).
//  2. products_kernel -- du = du_base + dz C and dC = dz^T u on the tensor
//     cores.  u and C are bf16 as they are; dz is fp32, so it is split into
//     three bf16 terms (hi + mid + lo holds its 24 bits) and every 16 deep step
//     of the product takes three MMAs.  Two terms would lose 2^-17 of a
//     gradient, which the router keeps in high precision.  For many tokens and
//     experts (half_operands) du takes scaled half operands and two terms
//     instead (half_centroids_kernel).
//     The two products run side by side in one launch, each on its share of
//     the SMs (make_plan): du waits for memory while dC waits for the tensor
//     cores.
//  3. reduce_kernel -- where the depth T of dC's tiles is split over CTAs, their
//     parts are added in a fixed order.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>

#include "epi_math.cuh"
#include "moe_common.cuh"

namespace moe {
namespace {

constexpr int kRgThreads = 128;
constexpr int kRgMaxK = 32;

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) v = __fadd_rn(v, __shfl_xor_sync(0xffffffffu, v, off));
  return v;
}

// The kernels of a call are launched to overlap: the next one's CTAs come in
// (and set up their barriers and TMEM) as soon as there is room, and wait for
// results where they need them (and read them past L1).
__device__ __forceinline__ void launch_dependents() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void wait_predecessor() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// What a product takes of dz: bf16 terms [3][T][E] (hi + mid + lo = dz), and
// for du half terms [2][T][E] of dz 2^-k_e 2^m_t (see half_centroids_kernel).
struct Terms {
  uint16_t* bf16;         // NULL: not wanted
  uint16_t* half;
  const float* cent_inv;  // [E] 2^-k_e
  float* row_scale;       // [T] 2^-m_t
};

// 2^(14 - floor(log2 max)): scales values of magnitude up to max below 2^15.
__device__ __forceinline__ float scale_to_2_14(float max) {
  const int e = static_cast<int>(__float_as_uint(max) >> 23) - 127;
  const int m = max > 0.f ? min(126, 14 - e) : 0;  // 14 - 128 at least
  return __uint_as_float(static_cast<uint32_t>(m + 127) << 23);
}
// The inverse of a power of two between 2^-126 and 2^126.
__device__ __forceinline__ float pow2_inverse(float p) { return __uint_as_float(0x7F000000u - __float_as_uint(p)); }

// du with half operands: half has three more mantissa bits than bf16, so two
// terms of dz hold 22 bits and more, where bf16 takes three terms for 24 -- a
// third of the tensor core's work less.  Half's narrow exponent is met by exact
// powers of two: centroid e is scaled by 2^k_e so that its largest element
// reaches [2^14, 2^15), which dz[.][e] undoes, and token t's row of dz by 2^m_t
// in the same way, which the epilogue undoes.  What half's smallest step then
// loses is 2^-39 of the centroid's, or the row's, largest element.  One CTA an
// expert.
__global__ void __launch_bounds__(256) half_centroids_kernel(const uint16_t* __restrict__ cent, int d,
                                                             uint16_t* __restrict__ out,
                                                             float* __restrict__ cent_inv) {
  __shared__ float part[8];
  launch_dependents();
  const uint4* row = reinterpret_cast<const uint4*>(cent + static_cast<int64_t>(blockIdx.x) * d);
  uint4* dst = reinterpret_cast<uint4*>(out + static_cast<int64_t>(blockIdx.x) * d);
  float m = 0.f;
  for (int v = threadIdx.x; v < d / 8; v += 256) {
    const uint4 w = __ldg(row + v);
    const uint32_t x[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      // an infinite element does not set the scale: the others would vanish
      const float lo = fabsf(__uint_as_float(x[i] << 16)), hi = fabsf(__uint_as_float(x[i] & 0xFFFF0000u));
      m = fmaxf(m, fmaxf(lo < INFINITY ? lo : 0.f, hi < INFINITY ? hi : 0.f));
    }
  }
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, off));
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = m;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 8; ++i) m = fmaxf(m, part[i]);
  const float k = scale_to_2_14(m);
  for (int v = threadIdx.x; v < d / 8; v += 256) {
    const uint4 w = __ldg(row + v);
    uint32_t x[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __half2 h = __floats2half2_rn(__fmul_rn(k, __uint_as_float(x[i] << 16)), __fmul_rn(k, __uint_as_float(x[i] & 0xFFFF0000u)));
      x[i] = *reinterpret_cast<const uint32_t*>(&h);
    }
    dst[v] = make_uint4(x[0], x[1], x[2], x[3]);
  }
  if (threadIdx.x == 0) cent_inv[blockIdx.x] = pow2_inverse(k);
}

// Lane l owns experts 4 l + 128 i .. + 3, i < Q: 16-byte accesses (E % 16 == 0).
template <int Q>
__global__ void __launch_bounds__(kRgThreads) dlogits_kernel(
    const float* __restrict__ dgate, const float* __restrict__ logits,
    const int32_t* __restrict__ idx, const float* __restrict__ gate, int T, int E, int K,
    const float* __restrict__ f, const float* __restrict__ dloss, int seq_len, float alpha,
    float* __restrict__ dz, const Terms terms, int32_t* dev_err) {
  __shared__ float gate_sm[kRgThreads / 32 * 128 * Q];
  const int lane = threadIdx.x & 31;
  const int64_t t = static_cast<int64_t>(blockIdx.x) * (kRgThreads / 32) + (threadIdx.x >> 5);
  launch_dependents();
  if (t >= T) return;
  float4 z[Q];
#pragma unroll
  for (int i = 0; i < Q; ++i) {
    const int e = 128 * i + 4 * lane;
    z[i] = e < E ? __ldg(reinterpret_cast<const float4*>(logits + t * E + e)) : make_float4(0.f, 0.f, 0.f, 0.f);
  }
  float g = 0.f, a = 0.f;
  int mine = -1;
  if (dgate && lane < K) {
    g = __ldg(gate + t * K + lane);
    a = __ldg(dgate + t * K + lane);
    mine = __ldg(idx + t * K + lane);
    if (mine < 0 || mine >= E) {
      set_dev_err(dev_err, MOE_DEVERR_BAD_INDEX);
      mine = -1;
      g = a = 0.f;  // whatever dgate holds there
    }
  }
  // s and 1 - s from one exponential: e^-|z| / (1 + e^-|z|) and 1 / (1 + e^-|z|)
  float s[4 * Q], rest[4 * Q], out[4 * Q];
#pragma unroll
  for (int i = 0; i < Q; ++i) {
    const float v[4] = {z[i].x, z[i].y, z[i].z, z[i].w};
    const bool in = 128 * i + 4 * lane < E;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float em = expf(-fabsf(v[j]));
      const float big = __frcp_rn(__fadd_rn(1.0f, em)), small = __fmul_rn(em, big);
      s[4 * i + j] = in ? (v[j] >= 0.f ? big : small) : 0.f;
      rest[4 * i + j] = v[j] >= 0.f ? small : big;
      out[4 * i + j] = 0.f;
    }
  }
  if (f) {
    const int64_t q = t / seq_len;
    const float c0 = __fmul_rn(alpha, dloss ? __ldg(dloss + q) : 1.0f) / static_cast<float>(seq_len);
    float c[4 * Q], sum = 0.f, mean = 0.f;
#pragma unroll
    for (int i = 0; i < Q; ++i) {
      const int e = 128 * i + 4 * lane;
      const float4 w = e < E ? __ldg(reinterpret_cast<const float4*>(f + q * E + e)) : make_float4(0.f, 0.f, 0.f, 0.f);
      c[4 * i] = __fmul_rn(c0, w.x);
      c[4 * i + 1] = __fmul_rn(c0, w.y);
      c[4 * i + 2] = __fmul_rn(c0, w.z);
      c[4 * i + 3] = __fmul_rn(c0, w.w);
#pragma unroll
      for (int j = 4 * i; j < 4 * i + 4; ++j) {
        sum = __fadd_rn(sum, s[j]);
        mean = fmaf(s[j], c[j], mean);
      }
    }
    sum = warp_sum(sum);
    mean = warp_sum(mean);
    if (sum < 0x1p-25f) {
      // Every s is below 2^-25, where it is e^z to the last bit: the shares are
      // those of e^(z - max z), which cannot all underflow.
      float top = -INFINITY;
#pragma unroll
      for (int i = 0; i < Q; ++i) {
        const int e = 128 * i + 4 * lane;
        if (e >= E) continue;
        const float4 v = __ldg(reinterpret_cast<const float4*>(logits + t * E + e));
        s[4 * i] = v.x;
        s[4 * i + 1] = v.y;
        s[4 * i + 2] = v.z;
        s[4 * i + 3] = v.w;
        top = fmaxf(top, fmaxf(fmaxf(v.x, v.y), fmaxf(v.z, v.w)));
      }
#pragma unroll
      for (int off = 16; off > 0; off >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
      sum = mean = 0.f;
#pragma unroll
      for (int j = 0; j < 4 * Q; ++j) {
        s[j] = 128 * (j / 4) + 4 * lane < E ? expf(__fsub_rn(s[j], top)) : 0.f;
        sum = __fadd_rn(sum, s[j]);
        mean = fmaf(s[j], c[j], mean);
      }
      sum = warp_sum(sum);
      mean = warp_sum(mean);
    }
    const float inv = __fdiv_rn(1.0f, sum);
    mean = __fmul_rn(mean, inv);
#pragma unroll
    for (int j = 0; j < 4 * Q; ++j)
      out[j] = __fmul_rn(__fmul_rn(__fmul_rn(s[j], inv), rest[j]), __fsub_rn(c[j], mean));
  }
  if (dgate) {
    const float mean = warp_sum(__fmul_rn(g, a));
    const float part = __fmul_rn(g, __fsub_rn(a, mean));
    // to their experts through shared memory; an index given twice adds in k order
    float* at = gate_sm + (threadIdx.x >> 5) * 128 * Q;
#pragma unroll
    for (int i = 0; i < Q; ++i) *reinterpret_cast<float4*>(at + 128 * i + 4 * lane) = make_float4(0.f, 0.f, 0.f, 0.f);
    __syncwarp();
    const uint32_t same = __match_any_sync(0xffffffffu, mine < 0 ? -1 - lane : mine);
    if (__all_sync(0xffffffffu, (same & (same - 1)) == 0)) {
      if (mine >= 0) at[mine] = part;
      __syncwarp();
    } else {
      for (int k = 0; k < K; ++k) {
        if (lane == k && mine >= 0) at[mine] += part;
        __syncwarp();
      }
    }
#pragma unroll
    for (int i = 0; i < Q; ++i) {
      const float4 v = *reinterpret_cast<const float4*>(at + 128 * i + 4 * lane);
      out[4 * i] = fmaf(v.x, rest[4 * i], out[4 * i]);
      out[4 * i + 1] = fmaf(v.y, rest[4 * i + 1], out[4 * i + 1]);
      out[4 * i + 2] = fmaf(v.z, rest[4 * i + 2], out[4 * i + 2]);
      out[4 * i + 3] = fmaf(v.w, rest[4 * i + 3], out[4 * i + 3]);
    }
  }
  const int64_t plane = static_cast<int64_t>(T) * E;
#pragma unroll
  for (int i = 0; i < Q; ++i) {
    const int e = 128 * i + 4 * lane;
    if (e >= E) continue;
    float r[4] = {out[4 * i], out[4 * i + 1], out[4 * i + 2], out[4 * i + 3]};
    if (dz) *reinterpret_cast<float4*>(dz + t * E + e) = make_float4(r[0], r[1], r[2], r[3]);
    if (terms.bf16) {
      // hi + mid + lo = out: each difference is exact
#pragma unroll
      for (int m = 0; m < 3; ++m) {
        const __nv_bfloat162 h0 = __floats2bfloat162_rn(r[0], r[1]), h1 = __floats2bfloat162_rn(r[2], r[3]);
        *reinterpret_cast<uint2*>(terms.bf16 + m * plane + t * E + e) =
            make_uint2(*reinterpret_cast<const uint32_t*>(&h0), *reinterpret_cast<const uint32_t*>(&h1));
        r[0] = __fsub_rn(r[0], __low2float(h0));
        r[1] = __fsub_rn(r[1], __high2float(h0));
        r[2] = __fsub_rn(r[2], __low2float(h1));
        r[3] = __fsub_rn(r[3], __high2float(h1));
      }
    }
  }
  if (!terms.half) return;
  wait_predecessor();  // half_centroids_kernel's scales
  float top = 0.f;
#pragma unroll
  for (int i = 0; i < Q; ++i) {
    const int e = 128 * i + 4 * lane;
    const float4 c = e < E ? __ldcg(reinterpret_cast<const float4*>(terms.cent_inv + e)) : make_float4(0.f, 0.f, 0.f, 0.f);
    out[4 * i] = __fmul_rn(out[4 * i], c.x);
    out[4 * i + 1] = __fmul_rn(out[4 * i + 1], c.y);
    out[4 * i + 2] = __fmul_rn(out[4 * i + 2], c.z);
    out[4 * i + 3] = __fmul_rn(out[4 * i + 3], c.w);
#pragma unroll
    for (int j = 4 * i; j < 4 * i + 4; ++j) top = fmaxf(top, fabsf(out[j]));
  }
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
  const float m_t = scale_to_2_14(top);
  if (lane == 0) terms.row_scale[t] = pow2_inverse(m_t);
#pragma unroll
  for (int i = 0; i < Q; ++i) {
    const int e = 128 * i + 4 * lane;
    if (e >= E) continue;
    float r[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) r[j] = __fmul_rn(m_t, out[4 * i + j]);
#pragma unroll
    for (int m = 0; m < 2; ++m) {
      const __half2 h0 = __floats2half2_rn(r[0], r[1]), h1 = __floats2half2_rn(r[2], r[3]);
      *reinterpret_cast<uint2*>(terms.half + m * plane + t * E + e) =
          make_uint2(*reinterpret_cast<const uint32_t*>(&h0), *reinterpret_cast<const uint32_t*>(&h1));
      r[0] = __fsub_rn(r[0], __low2float(h0));
      r[1] = __fsub_rn(r[1], __high2float(h0));
      r[2] = __fsub_rn(r[2], __low2float(h1));
      r[3] = __fsub_rn(r[3], __high2float(h1));
    }
  }
}

// ------------------------------------------------------------- products --
// D [M][N] = (base) + A [M][L] B [L][N] with A the terms of dz (TERMS: three in
// bf16, two in half) and B of the same type, N contiguous (the tensor core reads
// it as an MN-major operand).
//   du: A = dz as stored (M = tokens, depth = experts), B = the centroids
//   dC: A = dz transposed, also MN-major (M = experts, depth = tokens), B = u
// Tiles of 128 x 256 over depth blocks of 32.  One thread issues the TMA
// loads of a ring of stages (the terms of A in one box or two, 8 KB each, and
// 16 KB of B), one thread issues the MMAs, eight warps add finished
// accumulators in registers: the two TMEM accumulators alternate every 128
// deep, so that a tensor-core sum, whose additions may truncate, stays 24
// steps long and the rest is rounded fp32 additions.  The depth blocks of all
// tiles form one line that is cut over the CTAs as make_plan says, for du at
// tile borders.  An epilogue warp has 32 x 32 patches of its own in
// shared memory, which TMA fills with the base ahead of time and empties into
// the result.
// A depth block of dC takes a CTA 0.64 us, 87% of the measured tensor peak.  du
// reads the base and writes du besides (4096 x 7168 fp32: 36 us at the copy rate)
// and takes 58 us there on the whole GPU: its operand loads wait behind those
// streams; deeper patches, contiguous operands, narrower tiles, L2 prefetches and
// pairs of CTAs (cta_group::2) gave nothing more, dC at its side did.
constexpr uint32_t kFmtF16 = 0;  // kind::f16
constexpr int kPrM = 128, kPrN = 256, kPrK = 32;
constexpr int kPrChunk = 4;                       // depth blocks per accumulator
constexpr int kPrTerm = kPrM * kPrK * 2;          // bytes of one term's A block
constexpr int kPrSlab = 64 * kPrK * 2;            // 64 columns of an MN-major operand
constexpr int kPrB = kPrK * kPrN * 2;
constexpr int kPrEpiWarps = 8;
constexpr int kPrThreads = 128 + 32 * kPrEpiWarps;  // TMA, MMA and two spare warps; the epilogue
// launched with 168 registers a thread; 128 x 72 + 256 x 216 = 384 x 168
constexpr int kPrRegsCtl = 72, kPrRegsEpi = 216;
constexpr int kPrPatch = 32 * 32 * 4;
constexpr uint32_t kPrTmemCols = 2 * kPrN;
// du keeps three patches a warp (two loads of the base in flight while one is
// used) and, with three terms, a stage less than dC.
template <bool A_MN, int TERMS>
struct Ring {
  static constexpr int kStage = TERMS * kPrTerm + kPrB;
  static constexpr int kStages = A_MN || TERMS == 2 ? 4 : 3;
  static constexpr int kPatches = A_MN ? 2 : 3;
  static constexpr int kSmem = 1024 + kStages * kStage + kPatches * kPrEpiWarps * kPrPatch + 512;
};

// The parts of dC's tiles, n of each: tile * n + i, [kPrM][kPrN] fp32.
struct Parts {
  const float* part;
  float* out;
  int tiles, n, mt, M, N;
};

struct ProductArgs {
  int M, N, KB;  // KB: depth blocks of a tile
  int mt;        // m tiles (the faster tile index)
  int units;     // depth blocks of all tiles
  int per;       // depth blocks of a CTA; 0: whole tiles, evenly
  int first, share;  // whole tiles: the first CTAs take this many, the others the rest
  int has_base;
  const float* row_scale;  // of half terms
  int32_t* dev_err;
};

// MN-major operand with the 128-byte swizzle: TMA boxes of 64 (contiguous)
// x 32 (depth) elements are 4 KB slabs of 128-byte rows.  8 depth rows are a
// 1024-byte atom (stride byte offset), the next 64 elements are the next slab
// (leading byte offset).
__device__ __forceinline__ uint64_t smem_desc_mn_sw128(uint32_t smem_addr, uint32_t slab_stride) {
  uint64_t d = 0;
  d |= static_cast<uint64_t>((smem_addr >> 4) & 0x3FFFu);
  d |= static_cast<uint64_t>(slab_stride >> 4) << 16;
  d |= static_cast<uint64_t>(1024u >> 4) << 32;
  d |= static_cast<uint64_t>(1u) << 46;
  d |= static_cast<uint64_t>(2u) << 61;
  return d;
}

// TMA store of a patch; the waits: for all but the last N stores to have read
// theirs, and for all to have written.
__device__ __forceinline__ void tma_store_2d(const CUtensorMap* map, const void* src, int32_t c0,
                                             int32_t c1) {
  asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.tile.bulk_group [%0, {%2, %3}], [%1];" ::"l"(
                   reinterpret_cast<uint64_t>(map)),
               "r"(smem_u32(src)), "r"(c0), "r"(c1)
               : "memory");
  asm volatile("cp.async.bulk.commit_group;" ::: "memory");
}
template <int N>
__device__ __forceinline__ void tma_store_wait_read() {
  asm volatile("cp.async.bulk.wait_group.read %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void tma_store_wait_done() {
  asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
}

struct Segment {
  int m0, n0, k0, k1;
  bool whole;  // covers the tile's depth
};

// The next stretch of one tile in [pos, end).
__device__ __forceinline__ Segment next_segment(const ProductArgs& a, int pos, int end) {
  Segment s;
  const int tile = pos / a.KB;
  s.k0 = pos - tile * a.KB;
  s.k1 = min(a.KB, s.k0 + (end - pos));
  s.m0 = tile % a.mt * kPrM;
  s.n0 = tile / a.mt * kPrN;
  s.whole = s.k0 == 0 && s.k1 == a.KB;
  return s;
}

__device__ __forceinline__ void add4(float4& a, const float4& b) {
  a.x = __fadd_rn(a.x, b.x);
  a.y = __fadd_rn(a.y, b.y);
  a.z = __fadd_rn(a.z, b.z);
  a.w = __fadd_rn(a.w, b.w);
}

// Adds the parts of every tile in turn: a CTA takes a row of a tile at a time
// and reads eight parts ahead.
__global__ void __launch_bounds__(64) reduce_kernel(const Parts a) {
  constexpr int kAhead = 8;
  wait_predecessor();
  for (int g = blockIdx.x; g < a.tiles * kPrM; g += gridDim.x) {
    const int tile = g / kPrM, row = g % kPrM;
    const int m = tile % a.mt * kPrM + row, n = tile / a.mt * kPrN + 4 * threadIdx.x;
    if (m >= a.M || n >= a.N) continue;
    const float4* p = reinterpret_cast<const float4*>(a.part + (static_cast<int64_t>(tile) * a.n * kPrM + row) * kPrN) + threadIdx.x;
    float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int i = 0; i < a.n; i += kAhead) {
      float4 v[kAhead];
#pragma unroll
      for (int j = 0; j < kAhead; ++j)
        v[j] = i + j < a.n ? __ldcg(p + static_cast<int64_t>(i + j) * (kPrM * kPrN / 4)) : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int j = 0; j < kAhead; ++j) add4(sum, v[j]);
    }
    *reinterpret_cast<float4*>(a.out + static_cast<int64_t>(m) * a.N + n) = sum;
  }
}

// One product and where it reads and writes.
struct Product {
  CUtensorMap a, b, base, out, part;
  ProductArgs args;
};

// CTA `cta` of the product's `ctas`.
template <bool A_MN, int TERMS>
__device__ __forceinline__ void run_product(const Product& pr, const int cta, const int ctas) {
  const ProductArgs& args = pr.args;
  using R = Ring<A_MN, TERMS>;
  constexpr int kStages = R::kStages, kPatches = R::kPatches;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  uint8_t* ring = smem_raw + (((raw + 1023u) & ~1023u) - raw);
  uint8_t* patches = ring + kStages * R::kStage;
  uint64_t* full = reinterpret_cast<uint64_t*>(patches + kPatches * kPrEpiWarps * kPrPatch);
  uint64_t* empty = full + kStages;
  uint64_t* acc_full = empty + kStages;
  uint64_t* acc_empty = acc_full + 2;
  uint64_t* done = acc_empty + 2;
  uint64_t* base_full = done + 1;  // [epilogue warp][patch]
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(base_full + kPatches * kPrEpiWarps);
  int* abort_flag = reinterpret_cast<int*>(tmem_slot + 1);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int p = 0; p < 2; ++p) {
      mbar_init(&acc_full[p], 1);
      mbar_init(&acc_empty[p], kPrEpiWarps);
    }
    for (int p = 0; p < kPatches * kPrEpiWarps; ++p) mbar_init(&base_full[p], 1);
    mbar_init(done, 1);
    *abort_flag = 0;
    fence_barrier_init();
    prefetch_tmap(&pr.a);
    prefetch_tmap(&pr.b);
    prefetch_tmap(&pr.out);
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, kPrTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  volatile int* abort_v = abort_flag;
  wait_predecessor();  // dz's terms
  if (A_MN) launch_dependents();
  int start, end;
  if (args.per) {
    start = min(args.units, cta * args.per);
    end = min(args.units, start + args.per);
  } else {
    const int64_t tiles = args.units / args.KB;
    const bool early = cta < args.first;
    const int64_t b = early ? cta : cta - args.first, n = early ? args.first : ctas - args.first;
    const int64_t t0 = early ? 0 : args.share, nt = early ? args.share : tiles - args.share;
    start = static_cast<int>(t0 + nt * b / n) * args.KB;
    end = static_cast<int>(t0 + nt * (b + 1) / n) * args.KB;
  }

  if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kPrRegsCtl));
    if (warp == 0 && lane == 0) {
      // --------------------------------------------------------- TMA producer
      int it = 0;
      bool live = true;
      for (int pos = start; pos < end && live;) {
        const Segment g = next_segment(args, pos, end);
        pos += g.k1 - g.k0;
        for (int kb = g.k0; kb < g.k1; ++kb, ++it) {
          const int s = it % kStages;
          if (!mbar_wait(&empty[s], ((it / kStages) & 1) ^ 1, abort_v, args.dev_err)) {
            live = false;
            break;
          }
          uint8_t* sA = ring + s * R::kStage;
          uint8_t* sB = sA + TERMS * kPrTerm;
          mbar_arrive_expect_tx(&full[s], R::kStage);
          if (A_MN) {  // [64 experts][term][depth][64]
            tma_load_3d(sA, &pr.a, &full[s], g.m0, kb * kPrK, 0);
            tma_load_3d(sA + TERMS * kPrSlab, &pr.a, &full[s], g.m0 + 64, kb * kPrK, 0);
          } else {     // [term][row][depth]
            tma_load_3d(sA, &pr.a, &full[s], kb * kPrK, g.m0, 0);
          }
#pragma unroll
          for (int j = 0; j < kPrN / 64; ++j)
            tma_load_2d(sB + j * kPrSlab, &pr.b, &full[s], g.n0 + 64 * j, kb * kPrK);
        }
      }
      // every issued copy lands before the CTA can exit
      for (int i = it > kStages ? it - kStages : 0; i < it; ++i)
        mbar_wait(&full[i % kStages], (i / kStages) & 1, nullptr, args.dev_err);
    } else if (warp == 1 && lane == 0) {
      // ----------------------------------------------------------- MMA issuer
      constexpr uint32_t kFmt = TERMS == 2 ? kFmtF16 : kFmtBF16;
      const uint32_t idesc = instr_desc(kFmt, kFmt, kPrM, kPrN) | (A_MN ? 1u << 15 : 0u) | (1u << 16);
      constexpr uint64_t kStepA = A_MN ? 2048 >> 4 : 32 >> 4;  // 16 deep
      constexpr uint64_t kStepB = 2048 >> 4;
      int it = 0, ch = 0;
      bool live = true;
      for (int pos = start; pos < end && live;) {
        const Segment g = next_segment(args, pos, end);
        pos += g.k1 - g.k0;
        for (int kc = g.k0; kc < g.k1 && live; kc += kPrChunk, ++ch) {
          const int p = ch & 1;
          if (!mbar_wait(&acc_empty[p], ((ch >> 1) & 1) ^ 1, abort_v, args.dev_err)) {
            live = false;
            break;
          }
          tc_fence_after();
          const uint32_t acc = tmem + static_cast<uint32_t>(p * kPrN);
          const int kend = min(kc + kPrChunk, g.k1);
          for (int kb = kc; kb < kend; ++kb, ++it) {
            const int s = it % kStages;
            if (!mbar_wait(&full[s], (it / kStages) & 1, abort_v, args.dev_err)) {
              live = false;
              break;
            }
            tc_fence_after();
            const uint32_t sA = smem_u32(ring + s * R::kStage);
            const uint64_t bd = smem_desc_mn_sw128(sA + TERMS * kPrTerm, kPrSlab);
#pragma unroll
            for (int k = 0; k < kPrK / 16; ++k)
#pragma unroll
              for (int j = TERMS - 1; j >= 0; --j) {  // the smallest term first
                const uint64_t ad = A_MN ? smem_desc_mn_sw128(sA + j * kPrSlab, TERMS * kPrSlab)
                                         : smem_desc_sw64(sA + j * kPrTerm);
                mma_f16(acc, ad + k * kStepA, bd + k * kStepB, idesc, (kb > kc || k > 0 || j < TERMS - 1) ? 1u : 0u);
              }
            mma_commit(&empty[s]);
          }
          if (live) mma_commit(&acc_full[p]);
        }
      }
      mma_commit(done);
      mbar_wait(done, 0, nullptr, args.dev_err);
    }
    __syncwarp();
  } else {
    // --------------------------------------------------------------- epilogue
    // a warp reads the TMEM lanes of its quarter (warp % 4): 32 rows, 128 columns
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kPrRegsEpi));
    const int quarter = warp & 3, half = (warp - 4) >> 2;
    const uint32_t tq = tmem + (static_cast<uint32_t>(quarter * 32) << 16) + half * 128;
    uint8_t* patch = patches + (warp - 4) * kPatches * kPrPatch;
    uint64_t* landed = base_full + kPatches * (warp - 4);
    // the base's patches, loaded ahead of their use: tile and patch of the
    // next load, loads issued (all of lane 0), patches used
    const int t1 = end / args.KB;
    int lt = start / args.KB, lb = 0, loads = 0, used = 0;
    auto load_next = [&]() {
      while (lt < t1 && (lt / args.mt * kPrN + half * 128 >= args.N || lt % args.mt * kPrM + quarter * 32 >= args.M)) ++lt;
      if (lt >= t1) return;
      const int b = loads % kPatches;
      mbar_arrive_expect_tx(&landed[b], kPrPatch);
      tma_load_2d(patch + b * kPrPatch, &pr.base, &landed[b], lt / args.mt * kPrN + half * 128 + 32 * lb,
                  lt % args.mt * kPrM + quarter * 32);
      ++loads;
      if (++lb == 4) {
        lb = 0;
        ++lt;
      }
    };
    const bool has_base = !A_MN && args.has_base;
    if (has_base && lane == 0) {
#pragma unroll
      for (int i = 0; i < kPatches; ++i) load_next();
    }
    int ch = 0;
    bool ok = true;
    for (int pos = start; pos < end && ok;) {
      const Segment g = next_segment(args, pos, end);
      pos += g.k1 - g.k0;
      // the row's power of two back
      float row_scale = 1.f;
      if (TERMS == 2 && g.m0 + quarter * 32 + lane < args.M) row_scale = __ldcg(args.row_scale + g.m0 + quarter * 32 + lane);
      float acc[128];
#pragma unroll
      for (int i = 0; i < 128; ++i) acc[i] = 0.f;
      for (int kc = g.k0; kc < g.k1; kc += kPrChunk, ++ch) {
        const int p = ch & 1;
        ok = __all_sync(0xffffffffu, mbar_wait(&acc_full[p], (ch >> 1) & 1, abort_v, args.dev_err));
        if (!ok) break;
        tc_fence_after();
#pragma unroll
        for (int c = 0; c < 128; c += 32) {
          float v[32];
          tmem_ld32(tq + p * kPrN + c, v);
          tmem_ld_wait();
#pragma unroll
          for (int i = 0; i < 32; ++i) acc[c + i] = __fadd_rn(acc[c + i], v[i]);
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&acc_empty[p]);
      }
      if (!ok) break;
      // whole tiles go to the result, the part of one to the CTA's place
      const bool direct = !A_MN || g.whole;
      if (direct && (g.n0 + half * 128 >= args.N || g.m0 + quarter * 32 >= args.M)) continue;
      const CUtensorMap* dst = direct ? &pr.out : &pr.part;
      const int row0 = direct ? g.m0 + quarter * 32 : cta * kPrM + quarter * 32;
      const int col0 = direct ? g.n0 + half * 128 : half * 128;
#pragma unroll
      for (int b = 0; b < 4; ++b, ++used) {
        uint8_t* buf = patch + used % kPatches * kPrPatch;
        if (has_base) {
          ok = __all_sync(0xffffffffu, mbar_wait(&landed[used % kPatches], (used / kPatches) & 1, abort_v, args.dev_err));
          if (!ok) break;
        } else {
          if (lane == 0) tma_store_wait_read<kPatches - 1>();  // this patch's last store has read it
          __syncwarp();
        }
        // lane = row of 128 bytes, 16-byte pieces swizzled as TMA does
#pragma unroll
        for (int c = 0; c < 8; ++c) {
          float4* at = reinterpret_cast<float4*>(buf + lane * 128 + ((c ^ (lane & 7)) << 4));
          float4 v = make_float4(acc[32 * b + 4 * c], acc[32 * b + 4 * c + 1], acc[32 * b + 4 * c + 2], acc[32 * b + 4 * c + 3]);
          if (TERMS == 2) {
            v.x = __fmul_rn(row_scale, v.x);
            v.y = __fmul_rn(row_scale, v.y);
            v.z = __fmul_rn(row_scale, v.z);
            v.w = __fmul_rn(row_scale, v.w);
          }
          if (has_base) add4(v, *at);
          *at = v;
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          tma_store_2d(dst, buf, col0 + 32 * b, row0);
          if (has_base && used > 0) {  // the patch before this one has been stored: load ahead into it
            tma_store_wait_read<1>();
            load_next();
          }
        }
      }
    }
    // every copy of this warp has landed or left before the CTA can exit
    if (lane == 0) {
      for (int i = used; i < loads; ++i) mbar_wait(&landed[i % kPatches], (i / kPatches) & 1, nullptr, args.dev_err);
      tma_store_wait_done();
    }
    __syncwarp();
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) tmem_dealloc(tmem, kPrTmemCols);
}

// Both products in one launch: dC's CTAs come first, du's take the other SMs and
// those that dC leaves.  (As two launches du would read terms that only dC has
// waited for.)
template <int DU_TERMS>
__global__ void __launch_bounds__(kPrThreads, 1) products_kernel(const __grid_constant__ Product dc,
                                                                 const __grid_constant__ Product du,
                                                                 const int dc_ctas) {
  const int cta = blockIdx.x;
  if (cta < dc_ctas) run_product<true, 3>(dc, cta, dc_ctas);
  else run_product<false, DU_TERMS>(du, cta - dc_ctas, static_cast<int>(gridDim.x) - dc_ctas);
}
template <int DU_TERMS>
constexpr int kPrSmem = std::max(Ring<true, 3>::kSmem, Ring<false, DU_TERMS>::kSmem);

// Launches a kernel, behind: before the one ahead of it has ended.
template <typename... P, typename... A>
bool launch(void (*kern)(P...), int64_t grid, int block, int smem, bool behind, cudaStream_t st, const A&... args) {
  cudaLaunchAttribute at;
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(grid));
  cfg.blockDim = dim3(block);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cfg.attrs = &at;
  cfg.numAttrs = behind ? 1 : 0;
  if (cudaLaunchKernelEx(&cfg, kern, args...) == cudaSuccess) return true;
  cudaGetLastError();
  return false;
}

// When du takes half operands: above 4096 tokens, with more than 256 experts or
// where tokens x experts, the work saved, outweigh converting the centroids.  A
// call from one graph, three bf16 terms / two half terms, us, rows of 7168:
//   experts     128        160        256        304        384        512        1024
//   4100     79 /  83  100 / 103   91 /  99  112 / 107  124 / 121  175 / 164  322 / 293
//   8192    131 / 135  175 / 175  182 / 184  208 / 230  222 / 205  305 / 284  589 / 514
//   16384   260 / 260  330 / 327  332 / 315  440 / 416  452 / 426  608 / 537 1183 / 1016
// (4608 for 4100 with 128, 160, 512 and 1024 experts.)  Up to 128 experts du waits
// for memory either way.  At 4096 tokens and fewer the halves gain little (384
// experts: 117 / 114 at 4096, 68 / 64 at 2048, 41 / 44 at 1024), and three terms
// hold two bits more.
bool half_operands(int T, int E) {
  return T > 4096 && (E > 256 || (E > 128 && static_cast<int64_t>(T) * E > 1 << 21));
}

struct Plan {
  // workspace bytes: dz in bf16 and in half terms, the centroids in half, the
  // scales of both, dC's parts
  size_t bf16, half, cent, cent_inv, row_scale, parts, all;
  bool half_du;
  int du_units, du_kb, du_mt, du_ctas, du_first, du_share;
  int dc_units, dc_kb, dc_mt, dc_per, dc_ctas;
  bool fits;   // 32-bit arithmetic
};

// How the products are cut, and which SMs they get.  dC's tiles, each tk depth
// blocks deep, are taken whole (one, two, .. by a CTA) or cut into n equal parts
// (one CTA each, the depth padded with blocks of zeros).  du's CTAs have the
// other SMs from the start, with so many tiles each that they end with those that
// get in when dC's CTAs leave.  Of all these the one that ends first by the
// following times (in 10 ns, measured at full clock) is taken.
// From one graph 4096 tokens x 256 experts x 7168 take 87 us so and 99 with each
// product on the whole GPU in turn, 16384 x 384 405 and 437, 1024 x 256 29 and 39,
// 6000 x 64 x 2048 35 and 72.  Under the power cap the clock falls and dC, bound by
// the tensor cores, slows more than du, bound by memory: 16384 x 384 in a long loop
// takes 430 to 450.
constexpr int kDcBlock = 64, kDcPart = 250;     // a depth block; a tile's or a part's result
constexpr int kDuTile = 150, kDuBlock3 = 85, kDuBlock2 = 57, kDuLeast = 600;  // a tile; HBM's share of it
constexpr int kAdd = 500, kAddPart = 16;        // reduce_kernel; each part of a tile

void plan_products(Plan& p, bool du, bool dc, int64_t sms, int64_t tiles, int64_t tk, int64_t du_tiles) {
  const int64_t du_cost = std::max(kDuLeast, kDuTile + (p.half_du ? kDuBlock2 : kDuBlock3) * p.du_kb);
  p.dc_kb = p.dc_per = p.dc_units = p.dc_ctas = p.du_first = p.du_share = 0;
  p.du_ctas = static_cast<int>(std::min(sms, du_tiles));
  p.fits = true;
  if (!dc || tk == 0) return;
  int64_t best = INT64_MAX;
  // tiles of kb blocks (padded), per blocks of their line a CTA, each tile in so many parts
  auto take = [&](int64_t kb, int64_t per, int64_t parts) {
    const int64_t dc_end = per * kDcBlock + (parts > 1 ? 1 : per / kb) * kDcPart;
    const int64_t add = parts > 1 ? kAdd + kAddPart * parts : 0;
    if (dc_end + add >= best) return;
    const int64_t units = tiles * kb, ctas = (units + per - 1) / per, free = sms - ctas;
    int64_t end = dc_end, first = 0, share = 0, on = 0;
    if (du) {
      // late tiles by each CTA that comes after dC's, early ones by the others
      const int64_t ideal = (du_tiles * du_cost + ctas * dc_end) / sms;
      const int64_t guess = std::max<int64_t>(0, (ideal - dc_end) / du_cost);
      end = INT64_MAX;  // with no free SM, guess + 1 late tiles a CTA are all there are
      for (int64_t late = guess; late <= guess + 1; ++late) {
        const int64_t rest = std::max<int64_t>(0, du_tiles - late * ctas);
        if (free == 0 && rest > 0) continue;
        const int64_t early = free ? (rest + free - 1) / free : 0;
        const int64_t e = std::max(early * du_cost, dc_end + late * du_cost);
        if (e >= end) continue;
        end = e;
        first = rest == du_tiles ? 0 : std::min(free, rest);
        share = first ? rest : 0;
        on = first ? first + std::min(ctas, du_tiles - rest) : std::min(late ? ctas : free, du_tiles);
      }
    }
    if (end + add >= best) return;
    best = end + add;
    p.fits = units < (1ll << 31) && per < (1ll << 31);
    p.dc_kb = static_cast<int>(kb);
    p.dc_per = static_cast<int>(per);
    p.dc_units = static_cast<int>(units);
    p.dc_ctas = static_cast<int>(ctas);
    if (!du) return;
    p.du_ctas = static_cast<int>(on);
    p.du_first = static_cast<int>(first);
    p.du_share = static_cast<int>(share);
  };
  const int64_t least = (tiles + sms - 1) / sms;
  for (int64_t m = least; m < least + 4; ++m) take(tk, tk * m, 1);
  for (int64_t n = 2; n <= 32 && n * tiles <= sms && n <= tk; n += n < 4 ? 1 : n / 4) {
    const int64_t part = (tk + n - 1) / n;
    take(part * n, part, n);
  }
}

Plan make_plan(int T, int d, int E, bool du, bool dc) {
  Plan p;
  const int64_t sms = moe_num_sms();
  const int64_t nt = (d + kPrN - 1) / kPrN;
  const int64_t tm = (static_cast<int64_t>(T) + kPrM - 1) / kPrM, tk = (static_cast<int64_t>(T) + kPrK - 1) / kPrK;
  const int64_t em = (E + kPrM - 1) / kPrM, ek = (E + kPrK - 1) / kPrK;
  const int64_t units = tm * nt * ek;
  p.half_du = du && half_operands(T, E);
  p.du_units = static_cast<int>(units);
  p.du_kb = static_cast<int>(ek);
  p.du_mt = static_cast<int>(tm);
  p.dc_mt = static_cast<int>(em);
  plan_products(p, du, dc, sms, em * nt, tk, tm * nt);
  p.fits = units < (1ll << 31) && p.fits;
  auto bytes = [](int64_t a, int64_t b, int64_t c) { return (static_cast<size_t>(a) * b * c + 255) / 256 * 256; };
  p.bf16 = dc || (du && !p.half_du) ? bytes(T, E, 3 * 2) : 0;
  p.half = p.half_du ? bytes(T, E, 2 * 2) : 0;
  p.cent = p.half_du ? bytes(E, d, 2) : 0;
  p.cent_inv = p.half_du ? bytes(E, 4, 1) : 0;
  p.row_scale = p.half_du ? bytes(T, 4, 1) : 0;
  p.parts = p.dc_per < p.dc_kb ? static_cast<size_t>(p.dc_ctas) * kPrM * kPrN * sizeof(float) : 0;
  p.all = p.bf16 + p.half + p.cent + p.cent_inv + p.row_scale + p.parts;
  return p;
}

// Shared memory beyond 48 KB has to be granted once per kernel and device.
bool grant_smem() {
  static bool done[64] = {};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return false;
  if (dev >= 0 && dev < 64 && done[dev]) return true;
  const auto attr = cudaFuncAttributeMaxDynamicSharedMemorySize;
  if (cudaFuncSetAttribute(products_kernel<3>, attr, kPrSmem<3>) != cudaSuccess ||
      cudaFuncSetAttribute(products_kernel<2>, attr, kPrSmem<2>) != cudaSuccess)
    return false;
  if (dev >= 0 && dev < 64) done[dev] = true;
  return true;
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

moe_status check_sizes(int T, int d, int E) {
  if (T < 0 || d <= 0 || E <= 0) return MOE_ERR_INVALID_ARG;
  if (d % 128 != 0 || E % 16 != 0) return MOE_ERR_SHAPE;
  if (E > 1024) return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

}  // namespace
}  // namespace moe

extern "C" moe_status moe_route_backward_workspace_size(int T, int d, int E, size_t* bytes) {
  if (!bytes) return MOE_ERR_INVALID_ARG;
  const moe_status s = moe::check_sizes(T, d, E);
  if (s != MOE_OK) return s;
  // enough for a call with either or both products
  const moe::Plan both = moe::make_plan(T, d, E, true, true), dc = moe::make_plan(T, d, E, false, true);
  if (!both.fits || !dc.fits) return MOE_ERR_UNSUPPORTED;
  *bytes = std::max(both.all, dc.all);
  return MOE_OK;
}

extern "C" moe_status moe_route_backward_launches(int T, int d, int E, int du, int dcentroids, int* launches) {
  if (!launches) return MOE_ERR_INVALID_ARG;
  const moe_status s = moe::check_sizes(T, d, E);
  if (s != MOE_OK) return s;
  const moe::Plan plan = moe::make_plan(T, d, E, du != 0, dcentroids != 0);
  if (!plan.fits) return MOE_ERR_UNSUPPORTED;
  *launches = T == 0 ? 0 : plan.half_du + 1 + (du || dcentroids) + (plan.parts != 0);
  return MOE_OK;
}

extern "C" moe_status moe_route_backward(
    const float* dgate, const float* logits, const int32_t* topk_idx, const float* topk_gate,
    const uint16_t* u, int64_t ldu, const uint16_t* centroids, int T, int d, int E, int K,
    const float* f, const float* dloss, int seq_len, float alpha, const float* du_base,
    float* dlogits, float* du, float* dcentroids, void* ws, size_t ws_bytes, int32_t* dev_err,
    moe_stream_t stream) {
  using namespace moe;
  const moe_status s = check_sizes(T, d, E);
  if (s != MOE_OK) return s;
  if (K <= 0 || (f && seq_len <= 0)) return MOE_ERR_INVALID_ARG;
  if (K > E || ldu < d || (f && T % seq_len != 0)) return MOE_ERR_SHAPE;
  if (K > kRgMaxK) return MOE_ERR_UNSUPPORTED;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (T == 0) {
    if (dcentroids && cudaMemsetAsync(dcentroids, 0, static_cast<size_t>(E) * d * 4, st) != cudaSuccess)
      return MOE_ERR_CUDA;
    return MOE_OK;
  }
  if (!logits || (dgate && (!topk_idx || !topk_gate)) || (du && !centroids) || (dcentroids && !u))
    return MOE_ERR_INVALID_ARG;
  if (!aligned16(logits) || !aligned16(u) || !aligned16(centroids) || ldu % 8 != 0 ||
      !aligned16(du_base) || !aligned16(du) || !aligned16(dcentroids) || !aligned16(dlogits) ||
      !aligned16(f) || !aligned4(dgate) || !aligned4(topk_idx) || !aligned4(topk_gate) || !aligned4(dloss))
    return MOE_ERR_ALIGN;
  const Plan plan = make_plan(T, d, E, du, dcentroids);
  if (!plan.fits) return MOE_ERR_UNSUPPORTED;
  if (ws_bytes < plan.all || !ws) return MOE_ERR_WORKSPACE;
  if (!aligned16(ws)) return MOE_ERR_ALIGN;
  uint8_t* at = static_cast<uint8_t*>(ws);
  auto take = [&](size_t n) {
    uint8_t* p = at;
    at += n;
    return p;
  };
  uint16_t* bf16_terms = reinterpret_cast<uint16_t*>(take(plan.bf16));
  uint16_t* half_terms = reinterpret_cast<uint16_t*>(take(plan.half));
  uint16_t* half_cent = reinterpret_cast<uint16_t*>(take(plan.cent));
  float* cent_inv = reinterpret_cast<float*>(take(plan.cent_inv));
  float* row_scale = reinterpret_cast<float*>(take(plan.row_scale));
  float* parts = reinterpret_cast<float*>(take(plan.parts));
  const bool half_du = plan.half_du;
  if ((du || dcentroids) && !grant_smem()) return MOE_ERR_CUDA;
  if (half_du && !launch(half_centroids_kernel, E, 256, 0, false, st, centroids, d, half_cent, cent_inv))
    return MOE_ERR_CUDA;
  const Terms terms{dcentroids || (du && !half_du) ? bf16_terms : nullptr, half_du ? half_terms : nullptr, cent_inv,
                    row_scale};
  const int Q = (E + 127) / 128;
  auto dlogits_q = Q <= 1 ? dlogits_kernel<1> : Q <= 2 ? dlogits_kernel<2> : Q <= 3 ? dlogits_kernel<3>
                 : Q <= 4 ? dlogits_kernel<4> : dlogits_kernel<8>;
  constexpr int kWarps = kRgThreads / 32;
  if (!launch(dlogits_q, (static_cast<int64_t>(T) + kWarps - 1) / kWarps, kRgThreads, 0, half_du, st, dgate, logits,
              topk_idx, topk_gate, T, E, K, f, dloss, seq_len, alpha, dlogits, terms, dev_err))
    return MOE_ERR_CUDA;

  const auto bf16 = CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, fp32 = CU_TENSOR_MAP_DATA_TYPE_FLOAT32;
  const auto fp16 = CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
  const uint64_t rd = static_cast<uint64_t>(d) * 4, rz = static_cast<uint64_t>(E) * 2;
  const uint64_t stride[2] = {rz, rz * T};
  Product pc{}, pu{};
  const int dc_ctas = dcentroids ? plan.dc_ctas : 0, du_ctas = du ? plan.du_ctas : 0;
  if (dcentroids) {
    const uint64_t extent[3] = {static_cast<uint64_t>(E), static_cast<uint64_t>(T), 3};
    const uint32_t box[3] = {64, kPrK, 3};
    if (!moe_make_tmap_3d(&pc.a, bf16_terms, bf16, extent, stride, box, 128) ||
        !moe_make_tmap_2d(&pc.b, u, bf16, d, T, static_cast<uint64_t>(ldu) * 2, 64, kPrK) ||
        !moe_make_tmap_2d(&pc.out, dcentroids, fp32, d, E, rd, 32, 32) ||
        (plan.parts && !moe_make_tmap_2d(&pc.part, parts, fp32, kPrN, static_cast<uint64_t>(plan.dc_ctas) * kPrM, kPrN * 4, 32, 32)))
      return MOE_ERR_CUDA;
    pc.args = {E, d, plan.dc_kb, plan.dc_mt, plan.dc_units, plan.dc_per, 0, 0, 0, nullptr, dev_err};
  }
  if (du) {
    const uint32_t n = half_du ? 2 : 3;
    const uint64_t extent[3] = {static_cast<uint64_t>(E), static_cast<uint64_t>(T), n};
    const uint32_t box[3] = {kPrK, kPrM, n};
    if (!moe_make_tmap_3d(&pu.a, half_du ? half_terms : bf16_terms, half_du ? fp16 : bf16, extent, stride, box, 64) ||
        !moe_make_tmap_2d(&pu.b, half_du ? half_cent : centroids, half_du ? fp16 : bf16, d, E, static_cast<uint64_t>(d) * 2, 64, kPrK) ||
        !moe_make_tmap_2d(&pu.base, du_base ? du_base : du, fp32, d, T, rd, 32, 32) ||
        !moe_make_tmap_2d(&pu.out, du, fp32, d, T, rd, 32, 32))
      return MOE_ERR_CUDA;
    pu.args = {T, d, plan.du_kb, plan.du_mt, plan.du_units, 0, plan.du_first, plan.du_share, du_base ? 1 : 0, row_scale, dev_err};
  }
  if (dc_ctas + du_ctas > 0) {
    const bool ok = half_du
        ? launch(products_kernel<2>, dc_ctas + du_ctas, kPrThreads, kPrSmem<2>, true, st, pc, pu, dc_ctas)
        : launch(products_kernel<3>, dc_ctas + du_ctas, kPrThreads, kPrSmem<3>, true, st, pc, pu, dc_ctas);
    if (!ok) return MOE_ERR_CUDA;
  }
  if (plan.parts) {
    const Parts all{parts, dcentroids, plan.dc_units / plan.dc_kb, plan.dc_kb / plan.dc_per, plan.dc_mt, E, d};
    const int64_t rows = static_cast<int64_t>(all.tiles) * kPrM;
    if (!launch(reduce_kernel, std::min<int64_t>(rows, 16 * moe_num_sms()), 64, 0, true, st, all)) return MOE_ERR_CUDA;
  }
  return MOE_OK;
}
