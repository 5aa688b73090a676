// The router's gradient: through the gates, the sigmoid, the balance loss and
// the logits product.  "DeepSeek_V3_Report：Annotation", eqs. (13), (15) and
// (17)-(20).
//
//  1. dlogits_kernel -- one warp per token.  With s = sigmoid(z),
//     g_k = s_k / sum of the chosen s and s' = s / sum of all s, both
//     normalisations have the same gradient,
//       d(sum_k a_k g_k)/dz_i = g_i (1 - s_i) (a_i - sum_j g_j a_j),
//     with a = dgate for the gates and a = dloss alpha f / S for the balance
//     loss.  No division by a sum that may be tiny; 1 - s is 1 / (1 + e^z).
//  2. product_kernel -- du = du_base + dz C and dC = dz^T u on the tensor
//     cores.  u and C are bf16 as they are; dz is fp32, so it is split into
//     three bf16 terms (hi + mid + lo holds its 24 bits) and every 64 deep
//     block of the product takes three MMAs.  Two terms would lose 2^-17 of a
//     gradient, which the router keeps in high precision.
//  3. reduce_kernel -- adds the partial tiles of dC, whose depth T is split
//     over the CTAs, in a fixed order.
#include <cuda_bf16.h>

#include <algorithm>

#include "epi_math.cuh"
#include "moe_common.cuh"

namespace moe {
namespace {

constexpr int kRgThreads = 256;
constexpr int kRgMaxK = 32;

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) v = __fadd_rn(v, __shfl_xor_sync(0xffffffffu, v, off));
  return v;
}

// P = experts per lane; lane l owns experts 32 i + l.
template <int P>
__global__ void __launch_bounds__(kRgThreads) dlogits_kernel(
    const float* __restrict__ dgate, const float* __restrict__ logits,
    const int32_t* __restrict__ idx, const float* __restrict__ gate, int T, int E, int K,
    const float* __restrict__ f, const float* __restrict__ dloss, int seq_len, float alpha,
    float* __restrict__ dz, uint16_t* __restrict__ terms, int32_t* dev_err) {
  const int lane = threadIdx.x & 31;
  const int64_t t = static_cast<int64_t>(blockIdx.x) * (kRgThreads / 32) + (threadIdx.x >> 5);
  if (t >= T) return;
  float rest[P], out[P], s[P];
#pragma unroll
  for (int i = 0; i < P; ++i) {
    const int e = 32 * i + lane;
    out[i] = rest[i] = s[i] = 0.f;
    if (e < E) {
      const float z = __ldg(logits + t * E + e);
      rest[i] = __fdiv_rn(1.0f, __fadd_rn(1.0f, expf(z)));
      s[i] = __fdiv_rn(1.0f, __fadd_rn(1.0f, expf(-z)));
    }
  }
  if (f) {
    const int64_t q = t / seq_len;
    const float c0 = __fmul_rn(alpha, dloss ? __ldg(dloss + q) : 1.0f) / static_cast<float>(seq_len);
    float c[P], sum = 0.f, mean = 0.f;
#pragma unroll
    for (int i = 0; i < P; ++i) {
      const int e = 32 * i + lane;
      c[i] = e < E ? __fmul_rn(c0, __ldg(f + q * E + e)) : 0.f;
      sum = __fadd_rn(sum, s[i]);
      mean = fmaf(s[i], c[i], mean);
    }
    sum = warp_sum(sum);
    mean = __fdiv_rn(warp_sum(mean), sum);
#pragma unroll
    for (int i = 0; i < P; ++i)
      out[i] = __fmul_rn(__fmul_rn(__fdiv_rn(s[i], sum), rest[i]), __fsub_rn(c[i], mean));
  }
  if (dgate) {
    float g = 0.f, a = 0.f;
    int e = -1;
    if (lane < K) {
      g = __ldg(gate + t * K + lane);
      a = __ldg(dgate + t * K + lane);
      e = __ldg(idx + t * K + lane);
      if (e < 0 || e >= E) {
        set_dev_err(dev_err, MOE_DEVERR_BAD_INDEX);
        e = -1;
        g = 0.f;
      }
    }
    const float mean = warp_sum(__fmul_rn(g, a));
    const float part = __fmul_rn(g, __fsub_rn(a, mean));
    for (int k = 0; k < K; ++k) {
      const int ek = __shfl_sync(0xffffffffu, e, k);
      const float pk = __shfl_sync(0xffffffffu, part, k);
#pragma unroll
      for (int i = 0; i < P; ++i)
        if (ek == 32 * i + lane) out[i] = fmaf(pk, rest[i], out[i]);
    }
  }
  const int64_t plane = static_cast<int64_t>(T) * E;
#pragma unroll
  for (int i = 0; i < P; ++i) {
    const int e = 32 * i + lane;
    if (e >= E) continue;
    if (dz) dz[t * E + e] = out[i];
    if (terms) {
      // hi + mid + lo = out: each difference is exact
      float r = out[i];
#pragma unroll
      for (int j = 0; j < 3; ++j) {
        const __nv_bfloat16 h = __float2bfloat16_rn(r);
        terms[j * plane + t * E + e] = __bfloat16_as_ushort(h);
        r = __fsub_rn(r, __bfloat162float(h));
      }
    }
  }
}

// ------------------------------------------------------------- products --
// D [M][N] = (base) + A [M][L] B [L][N] with A the three bf16 terms of dz and
// B bf16, N contiguous (the tensor core reads it as an MN-major operand).
//   du: A = dz as stored (M = tokens, depth = experts), B = the centroids
//   dC: A = dz transposed, also MN-major (M = experts, depth = tokens), B = u
// Tiles of 128 x 256 over depth blocks of 64.  One warp issues TMA loads into
// a two-stage ring (80 KB a stage: 3 x 16 KB of A, 32 KB of B), one thread
// issues the MMAs, eight warps add finished accumulators in registers: the
// two TMEM accumulators alternate every 128 deep, so that a tensor-core sum,
// whose additions may truncate, stays 24 steps long and the rest is rounded
// fp32 additions.  The depth blocks of all tiles form one line that is cut
// evenly over the CTAs (for du at tile borders): every SM gets the same work
// whatever the shape, and dC's few tiles still fill the GPU.
constexpr int kPrM = 128, kPrN = 256, kPrK = 64;
constexpr int kPrStages = 2;
constexpr int kPrChunk = 2;                       // depth blocks per accumulator
constexpr int kPrTerm = kPrM * kPrK * 2;          // bytes of one term's A block
constexpr int kPrB = kPrK * kPrN * 2;
constexpr int kPrStage = 3 * kPrTerm + kPrB;
constexpr int kPrEpiWarps = 8;
constexpr int kPrThreads = 128 + 32 * kPrEpiWarps;  // TMA, MMA and two idle warps; the epilogue
// launched with 168 registers a thread; 128 x 56 + 256 x 224 = 384 x 168
constexpr int kPrRegsCtl = 56, kPrRegsEpi = 224;
constexpr int kPrPatch = 32 * 32 * 4;             // a warp's 32 x 32 transpose patch
constexpr int kPrSmem = 1024 + kPrStages * kPrStage + kPrEpiWarps * kPrPatch + 256;
constexpr uint32_t kPrTmemCols = 2 * kPrN;

struct ProductArgs {
  int M, N, KB;        // KB: depth blocks of a tile
  int mt;              // m tiles (the faster tile index)
  int64_t units;       // depth blocks of all tiles
  int whole;           // cut at tile borders only
  const float* base;   // may be out
  float* out;
  float* part;         // partial tiles [2 * CTAs][128][256]
  int32_t* dev_err;
};

// First depth block of CTA c of G.
__host__ __device__ inline int64_t cut(int64_t units, int KB, int whole, int c, int G) {
  return whole ? units / KB * c / G * KB : units * c / G;
}

// MN-major operand with the 128-byte swizzle: TMA boxes of 64 (contiguous)
// x 64 (depth) elements are 8 KB slabs of 128-byte rows.  8 depth rows are a
// 1024-byte atom (stride byte offset), the next 64 elements are the next slab
// (leading byte offset).
__device__ __forceinline__ uint64_t smem_desc_mn_sw128(uint32_t smem_addr) {
  uint64_t d = 0;
  d |= static_cast<uint64_t>((smem_addr >> 4) & 0x3FFFu);
  d |= static_cast<uint64_t>(8192u >> 4) << 16;
  d |= static_cast<uint64_t>(1024u >> 4) << 32;
  d |= static_cast<uint64_t>(1u) << 46;
  d |= static_cast<uint64_t>(2u) << 61;
  return d;
}

struct Segment {
  int m0, n0, k0, k1;
  bool whole;  // covers the tile's depth
  bool first;  // the CTA's first tile
};

// The next stretch of one tile in [pos, end).
__device__ __forceinline__ Segment next_segment(const ProductArgs& a, int64_t start, int64_t pos,
                                                int64_t end) {
  Segment s;
  const int64_t tile = pos / a.KB;
  s.k0 = static_cast<int>(pos - tile * a.KB);
  s.k1 = static_cast<int>(min(static_cast<int64_t>(a.KB), s.k0 + (end - pos)));
  s.m0 = static_cast<int>(tile % a.mt) * kPrM;
  s.n0 = static_cast<int>(tile / a.mt) * kPrN;
  s.whole = s.k0 == 0 && s.k1 == a.KB;
  s.first = pos == start;
  return s;
}

template <bool A_MN>
__global__ void __launch_bounds__(kPrThreads, 1) product_kernel(
    const __grid_constant__ CUtensorMap tmHi, const __grid_constant__ CUtensorMap tmMid,
    const __grid_constant__ CUtensorMap tmLo, const __grid_constant__ CUtensorMap tmB,
    const ProductArgs args) {
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  uint8_t* ring = smem_raw + (((raw + 1023u) & ~1023u) - raw);
  uint8_t* patches = ring + kPrStages * kPrStage;
  uint64_t* full = reinterpret_cast<uint64_t*>(patches + kPrEpiWarps * kPrPatch);
  uint64_t* empty = full + kPrStages;
  uint64_t* acc_full = empty + kPrStages;
  uint64_t* acc_empty = acc_full + 2;
  uint64_t* done = acc_empty + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(done + 1);
  int* abort_flag = reinterpret_cast<int*>(tmem_slot + 1);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int s = 0; s < kPrStages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int p = 0; p < 2; ++p) {
      mbar_init(&acc_full[p], 1);
      mbar_init(&acc_empty[p], kPrEpiWarps);
    }
    mbar_init(done, 1);
    *abort_flag = 0;
    fence_barrier_init();
    prefetch_tmap(&tmHi);
    prefetch_tmap(&tmMid);
    prefetch_tmap(&tmLo);
    prefetch_tmap(&tmB);
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
  const int64_t start = cut(args.units, args.KB, args.whole, blockIdx.x, gridDim.x);
  const int64_t end = cut(args.units, args.KB, args.whole, blockIdx.x + 1, gridDim.x);

  if (warp < 4) {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kPrRegsCtl));
    if (warp == 0 && lane == 0) {
      // --------------------------------------------------------- TMA producer
      const CUtensorMap* tmA[3] = {&tmLo, &tmMid, &tmHi};
      int it = 0;
      bool live = true;
      for (int64_t pos = start; pos < end && live;) {
        const Segment g = next_segment(args, start, pos, end);
        pos += g.k1 - g.k0;
        for (int kb = g.k0; kb < g.k1; ++kb, ++it) {
          const int s = it % kPrStages;
          if (!mbar_wait(&empty[s], ((it / kPrStages) & 1) ^ 1, abort_v, args.dev_err)) {
            live = false;
            break;
          }
          uint8_t* sA = ring + s * kPrStage;
          uint8_t* sB = sA + 3 * kPrTerm;
          mbar_arrive_expect_tx(&full[s], kPrStage);
#pragma unroll
          for (int j = 0; j < 3; ++j) {
            if (A_MN) {
              tma_load_2d(sA + j * kPrTerm, tmA[j], &full[s], g.m0, kb * kPrK);
              tma_load_2d(sA + j * kPrTerm + 8192, tmA[j], &full[s], g.m0 + 64, kb * kPrK);
            } else {
              tma_load_2d(sA + j * kPrTerm, tmA[j], &full[s], kb * kPrK, g.m0);
            }
          }
#pragma unroll
          for (int j = 0; j < kPrN / 64; ++j)
            tma_load_2d(sB + j * 8192, &tmB, &full[s], g.n0 + 64 * j, kb * kPrK);
        }
      }
      // every issued copy lands before the CTA can exit
      for (int i = it > kPrStages ? it - kPrStages : 0; i < it; ++i)
        mbar_wait(&full[i % kPrStages], (i / kPrStages) & 1, nullptr, args.dev_err);
    } else if (warp == 1 && lane == 0) {
      // ----------------------------------------------------------- MMA issuer
      const uint32_t idesc = instr_desc(kFmtBF16, kFmtBF16, kPrM, kPrN) | (A_MN ? 1u << 15 : 0u) | (1u << 16);
      constexpr uint64_t kStepA = A_MN ? 2048 >> 4 : 32 >> 4;  // 16 deep
      constexpr uint64_t kStepB = 2048 >> 4;
      int it = 0, ch = 0;
      bool live = true;
      for (int64_t pos = start; pos < end && live;) {
        const Segment g = next_segment(args, start, pos, end);
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
            const int s = it % kPrStages;
            if (!mbar_wait(&full[s], (it / kPrStages) & 1, abort_v, args.dev_err)) {
              live = false;
              break;
            }
            tc_fence_after();
            const uint32_t sA = smem_u32(ring + s * kPrStage);
            const uint64_t bd = smem_desc_mn_sw128(sA + 3 * kPrTerm);
#pragma unroll
            for (int k = 0; k < kPrK / 16; ++k)
#pragma unroll
              for (int j = 0; j < 3; ++j) {
                const uint64_t ad = A_MN ? smem_desc_mn_sw128(sA + j * kPrTerm) : smem_desc_sw128(sA + j * kPrTerm);
                mma_f16(acc, ad + k * kStepA, bd + k * kStepB, idesc, (kb > kc || k > 0 || j > 0) ? 1u : 0u);
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
    // ------------------------------------------------------------- epilogue
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kPrRegsEpi));
    // a warp reads the TMEM lanes of its quarter (warp % 4): 32 rows, 128 columns
    const int quarter = warp & 3, half = (warp - 4) >> 2;
    const uint32_t tq = tmem + (static_cast<uint32_t>(quarter * 32) << 16) + half * 128;
    float4* patch = reinterpret_cast<float4*>(patches + (warp - 4) * kPrPatch);
    const int pr = lane >> 3, pc = lane & 7;  // row group and 16-byte column when reading a patch
    int ch = 0;
    bool ok = true;
    for (int64_t pos = start; pos < end && ok;) {
      const Segment g = next_segment(args, start, pos, end);
      pos += g.k1 - g.k0;
      float acc[128];
#pragma unroll
      for (int i = 0; i < 128; ++i) acc[i] = 0.f;
      for (int kc = g.k0; kc < g.k1; kc += kPrChunk, ++ch) {
        const int p = ch & 1;
        ok = __all_sync(0xffffffffu, mbar_wait(&acc_full[p], (ch >> 1) & 1, abort_v, args.dev_err));
        if (!ok) break;
        tc_fence_after();
#pragma unroll
        for (int c = 0; c < 128; c += 16) {
          float v[16];
          tmem_ld16(tq + p * kPrN + c, v);
          tmem_ld_wait();
#pragma unroll
          for (int i = 0; i < 16; ++i) acc[c + i] = __fadd_rn(acc[c + i], v[i]);
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&acc_empty[p]);
      }
      if (!ok) break;
      // whole tiles go to the result, a part of a tile to the CTA's slot of
      // its first or its last tile
      const bool direct = g.whole;
      const int row0 = direct ? g.m0 + quarter * 32 : quarter * 32;
      const int col0 = direct ? g.n0 + half * 128 : half * 128;
      const int rows = direct ? min(32, args.M - row0) : 32;
      const int64_t ld = direct ? args.N : kPrN;
      float* dst = direct ? args.out
                          : args.part + (2 * static_cast<int64_t>(blockIdx.x) + (g.first ? 0 : 1)) * (kPrM * kPrN);
      const float* base = direct ? args.base : nullptr;
      if (direct && col0 >= args.N) continue;
#pragma unroll
      for (int b = 0; b < 4; ++b) {
        // lane = row into the patch (chunks swizzled by the row), then rows of 128 bytes out
#pragma unroll
        for (int c = 0; c < 8; ++c)
          patch[lane * 8 + (c ^ (lane & 7))] =
              make_float4(acc[32 * b + 4 * c], acc[32 * b + 4 * c + 1], acc[32 * b + 4 * c + 2], acc[32 * b + 4 * c + 3]);
        __syncwarp();
        float4 add[8];
        if (base) {
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const int r = 4 * i + pr;
            if (r < rows)
              add[i] = *reinterpret_cast<const float4*>(base + (row0 + r) * ld + col0 + 32 * b + 4 * pc);
          }
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int r = 4 * i + pr;
          float4 v = patch[r * 8 + (pc ^ (r & 7))];
          if (r < rows) {
            if (base) {
              v.x = __fadd_rn(v.x, add[i].x);
              v.y = __fadd_rn(v.y, add[i].y);
              v.z = __fadd_rn(v.z, add[i].z);
              v.w = __fadd_rn(v.w, add[i].w);
            }
            *reinterpret_cast<float4*>(dst + (row0 + r) * ld + col0 + 32 * b + 4 * pc) = v;
          }
        }
        __syncwarp();
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) tmem_dealloc(tmem, kPrTmemCols);
}

// The CTA whose share holds depth block x.
__host__ __device__ inline int owner(int64_t x, int64_t units, int G) {
  int c = static_cast<int>((x * G) / units);
  while (c + 1 < G && units * (c + 1) / G <= x) ++c;
  while (c > 0 && units * c / G > x) --c;
  return c;
}

// Adds the parts of every tile that more than one CTA worked on, CTA by CTA.
__global__ void __launch_bounds__(256) reduce_kernel(const float* __restrict__ part, int64_t units,
                                                     int KB, int mt, int G, int M, int N,
                                                     float* __restrict__ out) {
  const int tile = blockIdx.x;
  const int c0 = owner(static_cast<int64_t>(tile) * KB, units, G);
  const int c1 = owner(static_cast<int64_t>(tile + 1) * KB - 1, units, G);
  if (c0 == c1) return;
  const int m0 = tile % mt * kPrM, n0 = tile / mt * kPrN;
  // 8 rows of 256 columns a block
  const int v = threadIdx.x & 63;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int r = blockIdx.y * 8 + i * 4 + (threadIdx.x >> 6);
    if (m0 + r >= M || n0 + 4 * v >= N) continue;
    float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int c = c0; c <= c1; ++c) {
      const int slot = 2 * c + (units * c / G / KB == tile ? 0 : 1);
      const float4 p = __ldg(reinterpret_cast<const float4*>(part + static_cast<int64_t>(slot) * (kPrM * kPrN) + r * kPrN) + v);
      sum.x = __fadd_rn(sum.x, p.x);
      sum.y = __fadd_rn(sum.y, p.y);
      sum.z = __fadd_rn(sum.z, p.z);
      sum.w = __fadd_rn(sum.w, p.w);
    }
    *reinterpret_cast<float4*>(out + static_cast<int64_t>(m0 + r) * N + n0 + 4 * v) = sum;
  }
}

template <int P>
void launch_dlogits(cudaStream_t st, const float* dgate, const float* logits, const int32_t* idx,
                    const float* gate, int T, int E, int K, const float* f, const float* dloss,
                    int seq_len, float alpha, float* dz, uint16_t* terms, int32_t* dev_err) {
  const int blocks = (T + kRgThreads / 32 - 1) / (kRgThreads / 32);
  dlogits_kernel<P><<<blocks, kRgThreads, 0, st>>>(dgate, logits, idx, gate, T, E, K, f, dloss,
                                                   seq_len, alpha, dz, terms, dev_err);
}

struct Plan {
  size_t terms, parts;  // workspace bytes
  int64_t du_units, dc_units;
  int du_kb, du_mt, du_ctas, dc_kb, dc_mt, dc_ctas;
};

Plan make_plan(int T, int d, int E) {
  Plan p;
  const int sms = moe_num_sms();
  const int64_t nt = (d + kPrN - 1) / kPrN;
  p.du_mt = (T + kPrM - 1) / kPrM;
  p.du_kb = (E + kPrK - 1) / kPrK;
  p.du_units = p.du_mt * nt * p.du_kb;
  p.du_ctas = static_cast<int>(std::min<int64_t>(sms, p.du_mt * nt));
  p.dc_mt = (E + kPrM - 1) / kPrM;
  p.dc_kb = (T + kPrK - 1) / kPrK;
  p.dc_units = p.dc_mt * nt * p.dc_kb;
  p.dc_ctas = static_cast<int>(std::min<int64_t>(sms, p.dc_units));
  p.terms = (static_cast<size_t>(T) * E * 2 * 3 + 255) / 256 * 256;
  p.parts = static_cast<size_t>(2) * p.dc_ctas * kPrM * kPrN * sizeof(float);
  return p;
}

// Shared memory beyond 48 KB has to be granted once per kernel and device.
bool grant_smem() {
  static bool done[64] = {};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return false;
  if (dev >= 0 && dev < 64 && done[dev]) return true;
  if (cudaFuncSetAttribute(product_kernel<true>, cudaFuncAttributeMaxDynamicSharedMemorySize, kPrSmem) != cudaSuccess ||
      cudaFuncSetAttribute(product_kernel<false>, cudaFuncAttributeMaxDynamicSharedMemorySize, kPrSmem) != cudaSuccess)
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
  const moe::Plan p = moe::make_plan(T, d, E);
  *bytes = p.terms + p.parts;
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
      !aligned4(dgate) || !aligned4(topk_idx) || !aligned4(topk_gate) || !aligned4(f) || !aligned4(dloss))
    return MOE_ERR_ALIGN;
  size_t need = 0;
  moe_route_backward_workspace_size(T, d, E, &need);
  if (ws_bytes < need || !ws) return MOE_ERR_WORKSPACE;
  if (!aligned16(ws)) return MOE_ERR_ALIGN;
  const Plan plan = make_plan(T, d, E);
  uint16_t* terms = static_cast<uint16_t*>(ws);
  float* parts = reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + plan.terms);
  const bool products = du || dcentroids;
  if (products && !grant_smem()) return MOE_ERR_CUDA;
  const int P = (E + 31) / 32;
  auto go = P <= 1 ? launch_dlogits<1> : P <= 2 ? launch_dlogits<2> : P <= 4 ? launch_dlogits<4>
          : P <= 8 ? launch_dlogits<8> : P <= 12 ? launch_dlogits<12> : P <= 16 ? launch_dlogits<16>
          : launch_dlogits<32>;
  go(st, dgate, logits, topk_idx, topk_gate, T, E, K, f, dloss, seq_len, alpha, dlogits,
     products ? terms : nullptr, dev_err);
  MOE_CUDA_CHECK_LAUNCH();

  const auto bf16 = CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
  const size_t plane = static_cast<size_t>(T) * E;
  CUtensorMap a[3], b;
  if (du) {
    for (int j = 0; j < 3; ++j)
      if (!moe_make_tmap_2d(&a[j], terms + j * plane, bf16, E, T, static_cast<uint64_t>(E) * 2, kPrK, kPrM))
        return MOE_ERR_CUDA;
    if (!moe_make_tmap_2d(&b, centroids, bf16, d, E, static_cast<uint64_t>(d) * 2, 64, kPrK)) return MOE_ERR_CUDA;
    const ProductArgs args{T, d, plan.du_kb, plan.du_mt, plan.du_units, 1, du_base, du, nullptr, dev_err};
    product_kernel<false><<<plan.du_ctas, kPrThreads, kPrSmem, st>>>(a[0], a[1], a[2], b, args);
    MOE_CUDA_CHECK_LAUNCH();
  }
  if (dcentroids) {
    for (int j = 0; j < 3; ++j)
      if (!moe_make_tmap_2d(&a[j], terms + j * plane, bf16, E, T, static_cast<uint64_t>(E) * 2, 64, kPrK))
        return MOE_ERR_CUDA;
    if (!moe_make_tmap_2d(&b, u, bf16, d, T, static_cast<uint64_t>(ldu) * 2, 64, kPrK)) return MOE_ERR_CUDA;
    const ProductArgs args{E, d, plan.dc_kb, plan.dc_mt, plan.dc_units, 0, nullptr, dcentroids, parts, dev_err};
    product_kernel<true><<<plan.dc_ctas, kPrThreads, kPrSmem, st>>>(a[0], a[1], a[2], b, args);
    MOE_CUDA_CHECK_LAUNCH();
    const int64_t tiles = plan.dc_units / plan.dc_kb;
    if (plan.dc_kb > 1) {  // a tile of one depth block has one owner
      reduce_kernel<<<dim3(static_cast<unsigned>(tiles), kPrM / 8), 256, 0, st>>>(
          parts, plan.dc_units, plan.dc_kb, plan.dc_mt, plan.dc_ctas, E, d, dcentroids);
      MOE_CUDA_CHECK_LAUNCH();
    }
  }
  return MOE_OK;
}
