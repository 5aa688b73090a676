// The combine with an 8-bit checkpoint of the expert outputs, and its
// backward from the checkpoint.
// "DeepSeek_V3_Report：Annotation", eq. (12), "Fine-Grained Quantization",
// "Low-Precision Activation" (activations kept for the backward in FP8) and
// "Low-Precision Communication" (gradients quantised with power-of-two scales).
//
//   moe_combine_checkpoint           out = u + Ys + sum_k gate_k Y[r_k];  yq, ys = Q(Y[r_k])
//   moe_combine_checkpoint_backward  dy[r_k] = Q2(gate_k dout);  dgate_k = dout . (yq ys)[r_k]
//
// Both are streaming kernels.  A warp takes four 128-column tiles of a token at a
// time through all of its K rows, eight lanes a tile: lane l of a tile holds the
// columns 32 s + 4 l .. + 3 (s = 0..3), so that every fp32 access is a coalesced
// 16-byte one and a tile's maximum takes three shuffles for 16 values a lane
// (one lane per 4 values would take five).  The forward's pieces are CTAs' warps
// in any order; the backward's share a CTA a token, for the sums of dgate.
// One B200, 4096 tokens x 8 experts x 7168, one of several launches in a graph: the
// combine with its checkpoint 238 us, 96% of the measured copy rate (HBM bound); its
// backward 109 us, 90%, and 284 us, 92%, with the fp32 rows as well (in a loop 2 to
// 6 us more).
#include <cuda_fp8.h>

#include "epi_math.cuh"
#include "moe_common.cuh"

namespace moe {
namespace {

constexpr int kCkWarps = 4;      // warps of a CTA with much to do besides
constexpr int kCkMaxWarps = 16;  // most warps of a CTA whose warps share a token
constexpr int kCkMaxK = 32;
constexpr int kCkTiles = 4;  // tiles of one warp step

struct Shape {
  dim3 block;  // (32 * warps of a token, tokens)
  unsigned grid;
  size_t smem;
};

// Four warps a token where that gives an SM 24 warps, more where the tokens are
// few, up to 16 (x 8 experts x 7168: 200 tokens 8.9 us with 14 against 9.7 with
// seven, 700 tokens 20.8 with five against 22.6 with four); several tokens a CTA
// where a token has fewer pieces.
Shape ck_shape(int T, int K, int tiles) {
  const int items = (tiles + kCkTiles - 1) / kCkTiles;
  const int64_t want = (static_cast<int64_t>(moe_num_sms()) * 24 + T - 1) / T;
  const int most = static_cast<int>(want < kCkWarps ? kCkWarps : (want > kCkMaxWarps ? kCkMaxWarps : want));
  const int steps = (items + most - 1) / most;
  const int warps = (items + steps - 1) / steps;
  const int tokens = warps >= kCkWarps ? 1 : kCkWarps / warps;
  return {dim3(32 * warps, tokens), static_cast<unsigned>((static_cast<int64_t>(T) + tokens - 1) / tokens),
          static_cast<size_t>(tokens) * warps * (K * 8 + 256) * sizeof(float)};
}

// Two E4M3 bytes -> two floats (exact: every E4M3 value is a half value).
__device__ __forceinline__ float2 codes_to_float2(uint32_t w) {
  return __half22float2(__half2(__nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(w), __NV_E4M3)));
}

// Largest magnitude of a tile: this lane's 16 values, then its eight lanes.
__device__ __forceinline__ float tile_amax(const float4 (&v)[4]) {
  float m = 0.f;
#pragma unroll
  for (int s = 0; s < 4; ++s)
    m = fmaxf(m, fmaxf(fmaxf(fabsf(v[s].x), fabsf(v[s].y)), fmaxf(fabsf(v[s].z), fabsf(v[s].w))));
#pragma unroll
  for (int off = 4; off > 0; off >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, off));
  return m;
}

// pow2_ceil(quant_scale(x)) for x >= 1e-4 without the division: 448 = 1.75 *
// 2^8, so with x = m 2^e the quotient is at most 2^(e-8) when m <= 1.75 (and
// above 2^(e-9), which rounding cannot undercut), and the next larger m is
// already rounded above 2^(e-8).  Adding 0x1fffff to the bits carries into the
// exponent exactly when the mantissa is above 1.75's.
__device__ __forceinline__ float pow2_quant_scale(float amax) {
  const float x = fmaxf(amax, kQuantEps);
  const uint32_t b = ((__float_as_uint(x) + 0x1FFFFFu) & 0x7F800000u) - (8u << 23);
  return x < INFINITY ? __uint_as_float(b) : x;
}

// Two fp32 values as one 64-bit register pair: the packed instructions round
// each half as the single ones do, at half the issue slots.
__device__ __forceinline__ uint64_t pack2(float lo, float hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ float2 unpack2(uint64_t v) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
  return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}

// The token's pairs, one a lane: sorted row (-1 dropped) and gate.
__device__ __forceinline__ void load_pair(const int32_t* __restrict__ dst_of,
                                          const float* __restrict__ gate, int64_t t, int K, int lane,
                                          int64_t rows, bool live, int& row, float& g,
                                          int32_t* dev_err) {
  row = -1;
  g = 0.f;
  if (live && lane < K) {
    row = __ldg(dst_of + t * K + lane);
    g = __ldg(gate + t * K + lane);
    if (row >= rows) {
      set_dev_err(dev_err, MOE_DEVERR_BAD_INDEX);
      row = -1;
    }
  }
}

template <bool POW2>
__global__ void __launch_bounds__(32 * kCkWarps) combine_checkpoint_kernel(
    const float* __restrict__ Y, int64_t rows, const int32_t* __restrict__ dst_of,
    const float* __restrict__ gate, const float* __restrict__ Ysh, const uint16_t* __restrict__ u,
    int T, int K, int d, float* __restrict__ out, uint8_t* __restrict__ yq, float* __restrict__ ys,
    int32_t* dev_err) {
  const int lane = threadIdx.x & 31;
  const int tiles = d / 128, items = (tiles + kCkTiles - 1) / kCkTiles;
  const int64_t unit = static_cast<int64_t>(blockIdx.x) * kCkWarps + (threadIdx.x >> 5);
  const int64_t t = unit / items;
  if (t >= T) return;
  int row;
  float g;
  load_pair(dst_of, gate, t, K, lane, rows, true, row, g, dev_err);
  const uint32_t kept = __ballot_sync(0xffffffffu, row >= 0);
  const int j = static_cast<int>(unit - t * items) * kCkTiles + (lane >> 3);
  const bool in = j < tiles;               // a token's last piece may hold fewer tiles
  const int64_t col = static_cast<int64_t>(j) * 128 + 4 * (lane & 7);
  float4 acc[4];
#pragma unroll
  for (int s = 0; s < 4; ++s) {
    acc[s] = make_float4(0.f, 0.f, 0.f, 0.f);
    if (in) {
      const uint2 ub = __ldg(reinterpret_cast<const uint2*>(u + t * d + col + 32 * s));
      acc[s] = make_float4(bf16_bits_to_float(ub.x & 0xFFFFu), bf16_bits_to_float(ub.x >> 16),
                           bf16_bits_to_float(ub.y & 0xFFFFu), bf16_bits_to_float(ub.y >> 16));
      if (Ysh) {
        const float4 a = __ldg(reinterpret_cast<const float4*>(Ysh + t * d + col + 32 * s));
        acc[s].x += a.x;
        acc[s].y += a.y;
        acc[s].z += a.z;
        acc[s].w += a.w;
      }
    }
  }
  float4 next[4];
  auto fetch = [&](uint32_t left) {
    const int64_t r = __shfl_sync(0xffffffffu, row, __ffs(left) - 1);
#pragma unroll
    for (int s = 0; s < 4; ++s)
      next[s] = in ? __ldg(reinterpret_cast<const float4*>(Y + r * d + col + 32 * s)) : make_float4(0.f, 0.f, 0.f, 0.f);
  };
  if (kept) fetch(kept);
  for (uint32_t left = kept; left;) {
    const int k = __ffs(left) - 1;
    left &= left - 1;
    float4 v[4];
#pragma unroll
    for (int s = 0; s < 4; ++s) v[s] = next[s];
    if (left) fetch(left);                 // the next row's loads overlap this row's arithmetic
    const int64_t r = __shfl_sync(0xffffffffu, row, k);
    const float w = __shfl_sync(0xffffffffu, g, k);
    const float s0 = quant_scale(tile_amax(v));
    const float scale = POW2 ? pow2_ceil(s0) : s0;
    const float rs = __frcp_rn(scale);
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      acc[s].x = fmaf(w, v[s].x, acc[s].x);
      acc[s].y = fmaf(w, v[s].y, acc[s].y);
      acc[s].z = fmaf(w, v[s].z, acc[s].z);
      acc[s].w = fmaf(w, v[s].w, acc[s].w);
      if (in)
        *reinterpret_cast<uint32_t*>(yq + r * d + col + 32 * s) =
            e4m3x4(div_by_scale(v[s].x, scale, rs), div_by_scale(v[s].y, scale, rs),
                   div_by_scale(v[s].z, scale, rs), div_by_scale(v[s].w, scale, rs));
    }
    if (in && (lane & 7) == 0) ys[r * tiles + j] = scale;
  }
  if (in) {
#pragma unroll
    for (int s = 0; s < 4; ++s) *reinterpret_cast<float4*>(out + t * d + col + 32 * s) = acc[s];
  }
}

// dout is read once a tile (and ROWS experts) and gives all gradient tiles.  Its
// largest magnitude is found once: rounding is monotone, so the largest |fl(g x)| is
// fl(|g| max |x|).  The 32 scales of four tiles and eight experts are computed by
// the 32 lanes at once and handed out by shuffles.  Power-of-two scales divide
// exactly: a product with the inverse gives the quotient, and folded into the gate
// it gives the same bits with one product (a gate beyond 1e30 keeps the two).
// Without dy a lane holds 16 neighbouring columns, so that a row's codes are one
// 16-byte access a lane; with it the columns 32 s + 4 l, so that the fp32 rows' are.
// What counts besides is that the codes are asked for three rows ahead: without
// the conversions the kernel took as long, one row ahead with 40 warps an SM took
// 123 us for 4096 x 8 rows of 7168, three ahead with 28 (72 registers a thread)
// takes 109.  ROWS is 8, 4 or 2 by K, with more than 8 in turns of 8 (lane l
// has expert l % 8 of a turn, so fewer ROWS are for K <= ROWS alone); 4096 x 4
// rows take 67 us with four and 70 with eight, 4096 x 2 of 5120 35 with two
// and 42.  At most WARPS warps a CTA.
template <bool WITH_DY, int WARPS, int ROWS>
__global__ void __launch_bounds__(32 * WARPS, WARPS > kCkWarps ? 2 : (ROWS == 2 ? 8 : 7)) combine_checkpoint_backward_kernel(
    const float* __restrict__ dout, const int32_t* __restrict__ dst_of,
    const float* __restrict__ gate, const uint8_t* __restrict__ yq, const float* __restrict__ ys,
    int64_t rows, int T, int K, int d, uint8_t* __restrict__ dyq, float* __restrict__ dys,
    float* __restrict__ dy, float* __restrict__ dgate, int32_t* dev_err) {
  extern __shared__ float dot[];  // [tokens][warps][K][8], then [tokens][warps][8][32]
  constexpr int kLane = WITH_DY ? 4 : 16, kStep = WITH_DY ? 32 : 4;
  constexpr int kAhead = ROWS < 3 ? ROWS : 3;
  const int64_t t = static_cast<int64_t>(blockIdx.x) * blockDim.y + threadIdx.y;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  const int64_t P = static_cast<int64_t>(T) * K;
  int row;
  float g;
  load_pair(dst_of, gate, t, K, lane, rows, t < T, row, g, dev_err);
  if (row < 0) g = 0.f;  // whatever a dropped pair's gate holds
  const int tiles = d / 128, end = t < T ? tiles : 0;
  float* mine = dot + blockDim.y * warps * K * 8 + (threadIdx.y * warps + warp) * 8 * 32 + lane;  // one lane's sums
  int k0 = 0;
  do {  // ROWS experts at a time (K == 0: the shared expert's rows alone)
    const int my_row = __shfl_sync(0xffffffffu, row, k0 + (lane & 7));
    const float my_gate = __shfl_sync(0xffffffffu, g, k0 + (lane & 7));
    const bool plain = !WITH_DY && __all_sync(0xffffffffu, fabsf(my_gate) <= 1e30f);
#pragma unroll
    for (int m = 0; m < ROWS; ++m) mine[32 * m] = 0.f;
    for (int item = warp; item * kCkTiles < end; item += warps) {
      const int j = item * kCkTiles + (lane >> 3);
      const bool in = j < tiles;
      const int64_t col = static_cast<int64_t>(j) * 128 + kLane * (lane & 7);
      float4 a[4];
#pragma unroll
      for (int s = 0; s < 4; ++s)
        a[s] = in ? __ldg(reinterpret_cast<const float4*>(dout + t * d + col + kStep * s)) : make_float4(0.f, 0.f, 0.f, 0.f);
      uint4 next[kAhead];
#pragma unroll
      for (int i = 0; i < kAhead; ++i) next[i] = make_uint4(0u, 0u, 0u, 0u);
      auto fetch = [&](int m, uint4& to) {
        const int r = __shfl_sync(0xffffffffu, row, k0 + m);
        if (r < 0 || !in) return;
        const uint8_t* p = yq + static_cast<int64_t>(r) * d + col;
        if (WITH_DY)
          to = make_uint4(__ldg(reinterpret_cast<const uint32_t*>(p)), __ldg(reinterpret_cast<const uint32_t*>(p + 32)),
                          __ldg(reinterpret_cast<const uint32_t*>(p + 64)), __ldg(reinterpret_cast<const uint32_t*>(p + 96)));
        else
          to = __ldg(reinterpret_cast<const uint4*>(p));
      };
#pragma unroll
      for (int i = 0; i < kAhead; ++i) fetch(i, next[i]);
      const int64_t my_tile = static_cast<int64_t>(my_row) * tiles + j;
      const float my_ys = my_row >= 0 && in ? __ldg(ys + my_tile) : 0.f;
      const float amax = tile_amax(a);
      uint64_t a2[8];
#pragma unroll
      for (int s = 0; s < 4; ++s) {
        a2[2 * s] = pack2(a[s].x, a[s].y);
        a2[2 * s + 1] = pack2(a[s].z, a[s].w);
      }
      // 1 / 2^e by its exponent; an infinite maximum leaves no finite scale: every code is NaN
      auto inverse = [](float scale) { return scale < INFINITY ? __uint_as_float(0x7F000000u - __float_as_uint(scale)) : NAN; };
      auto write_codes = [&](int64_t r, const uint32_t (&q)[4]) {
        uint8_t* p = dyq + r * d + col;
        if (WITH_DY) {
#pragma unroll
          for (int s = 0; s < 4; ++s) *reinterpret_cast<uint32_t*>(p + 32 * s) = q[s];
        } else {
          *reinterpret_cast<uint4*>(p) = make_uint4(q[0], q[1], q[2], q[3]);
        }
      };
      auto write_folded = [&](int64_t r, float wi) {  // wi = w / scale
        const uint64_t wi2 = pack2(wi, wi);
        uint32_t q[4];
#pragma unroll
        for (int s = 0; s < 4; ++s) {
          const float2 ql = unpack2(mul2(wi2, a2[2 * s])), qh = unpack2(mul2(wi2, a2[2 * s + 1]));
          q[s] = e4m3x4(ql.x, ql.y, qh.x, qh.y);
        }
        write_codes(r, q);
      };
      auto write_row = [&](int64_t r, float w, float inv) {
        const uint64_t w2 = pack2(w, w), inv2 = pack2(inv, inv);
        uint32_t q[4];
#pragma unroll
        for (int s = 0; s < 4; ++s) {
          const uint64_t lo = mul2(w2, a2[2 * s]), hi = mul2(w2, a2[2 * s + 1]);
          const float2 ql = unpack2(mul2(lo, inv2)), qh = unpack2(mul2(hi, inv2));
          q[s] = e4m3x4(ql.x, ql.y, qh.x, qh.y);
          if (WITH_DY) {
            const float2 vl = unpack2(lo), vh = unpack2(hi);
            *reinterpret_cast<float4*>(dy + r * d + col + kStep * s) = make_float4(vl.x, vl.y, vh.x, vh.y);
          }
        }
        write_codes(r, q);
      };
      if (k0 == 0 && in) {
        const float scale = pow2_quant_scale(amax), inv = inverse(scale);
        if (WITH_DY) write_row(P + t, 1.0f, inv);
        else write_folded(P + t, inv);
        if ((lane & 7) == 0) dys[(P + t) * tiles + j] = scale;
      }
      const float my_scale = pow2_quant_scale(__fmul_rn(fabsf(my_gate), amax));
      const float my_wi = __fmul_rn(my_gate, inverse(my_scale));
      if (my_row >= 0 && in) dys[my_tile] = my_scale;
#pragma unroll
      for (int m = 0; m < ROWS; ++m) {
        const int r = __shfl_sync(0xffffffffu, row, k0 + m);
        const int from = (lane & 24) | m;
        const uint32_t code[4] = {next[m % kAhead].x, next[m % kAhead].y, next[m % kAhead].z, next[m % kAhead].w};
        if (m + kAhead < ROWS) fetch(m + kAhead, next[m % kAhead]);
        if (r < 0) continue;
        if (plain) {
          const float wi = __shfl_sync(0xffffffffu, my_wi, from);
          if (in) write_folded(r, wi);
        } else {
          const float w = __shfl_sync(0xffffffffu, g, k0 + m);
          if (in) write_row(r, w, inverse(pow2_quant_scale(__fmul_rn(fabsf(w), amax))));
        }
        const float scale = __shfl_sync(0xffffffffu, my_ys, from);
        uint64_t sum2 = pack2(0.f, 0.f);
#pragma unroll
        for (int s = 0; s < 4; ++s) {
          const float2 fl = codes_to_float2(code[s] & 0xFFFFu), fh = codes_to_float2(code[s] >> 16);
          sum2 = fma2(a2[2 * s], pack2(fl.x, fl.y), sum2);
          sum2 = fma2(a2[2 * s + 1], pack2(fh.x, fh.y), sum2);
        }
        const float2 sum = unpack2(sum2);
        mine[32 * m] = fmaf(__fadd_rn(sum.x, sum.y), scale, mine[32 * m]);
      }
    }
#pragma unroll
    for (int m = 0; m < ROWS; ++m) {
      float p = mine[32 * m];
      p += __shfl_xor_sync(0xffffffffu, p, 16);
      p += __shfl_xor_sync(0xffffffffu, p, 8);
      // the rest of the sum over the lanes is left to the end
      if (lane < 8 && k0 + m < K) dot[((threadIdx.y * warps + warp) * K + k0 + m) * 8 + lane] = p;
    }
    k0 += ROWS;
  } while (k0 < K);
  __syncthreads();
  if (t < T && threadIdx.x < K) {
    float sum = 0.f;
    for (int w = 0; w < warps; ++w)
#pragma unroll
      for (int i = 0; i < 8; ++i) sum += dot[((threadIdx.y * warps + w) * K + threadIdx.x) * 8 + i];
    dgate[t * K + threadIdx.x] = sum;
  }
}

template <int ROWS>
auto pick_backward(bool with_dy, bool many) {
  return with_dy ? (many ? combine_checkpoint_backward_kernel<true, kCkMaxWarps, ROWS> : combine_checkpoint_backward_kernel<true, kCkWarps, ROWS>)
                 : (many ? combine_checkpoint_backward_kernel<false, kCkMaxWarps, ROWS> : combine_checkpoint_backward_kernel<false, kCkWarps, ROWS>);
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

}  // namespace
}  // namespace moe

extern "C" moe_status moe_combine_checkpoint(const float* Y, int64_t rows, const int32_t* dst_of,
                                             const float* topk_gate, const float* Y_shared,
                                             const uint16_t* u, int T, int K, int d, int pow2,
                                             float* out, uint8_t* yq, float* ys, int32_t* dev_err,
                                             moe_stream_t stream) {
  using namespace moe;
  if (T < 0 || K < 0 || d <= 0 || rows < 0) return MOE_ERR_INVALID_ARG;
  if (d % 128 != 0) return MOE_ERR_SHAPE;
  if (K > kCkMaxK || rows > 0x7FFFFFFFll) return MOE_ERR_UNSUPPORTED;
  if (T == 0) return MOE_OK;
  if (!u || !out || (K > 0 && (!dst_of || !topk_gate || (rows > 0 && (!Y || !yq || !ys)))))
    return MOE_ERR_INVALID_ARG;
  if (!aligned16(Y) || !aligned16(Y_shared) || !aligned16(u) || !aligned16(out) || !aligned16(yq) ||
      !aligned4(ys) || !aligned4(dst_of) || !aligned4(topk_gate))
    return MOE_ERR_ALIGN;
  auto kern = pow2 ? combine_checkpoint_kernel<true> : combine_checkpoint_kernel<false>;
  const int64_t items = (d / 128 + kCkTiles - 1) / kCkTiles;
  const int64_t blocks = (T * items + kCkWarps - 1) / kCkWarps;
  if (blocks > 0x7FFFFFFFll) return MOE_ERR_UNSUPPORTED;
  kern<<<static_cast<unsigned>(blocks), 32 * kCkWarps, 0, static_cast<cudaStream_t>(stream)>>>(
      Y, rows, dst_of, topk_gate, Y_shared, u, T, K, d, out, yq, ys, dev_err);
  MOE_CUDA_CHECK_LAUNCH();
  return MOE_OK;
}

extern "C" moe_status moe_combine_checkpoint_backward(const float* dout, const int32_t* dst_of,
                                                      const float* topk_gate, const uint8_t* yq,
                                                      const float* ys, int64_t rows, int T, int K,
                                                      int d, uint8_t* dyq, float* dys, float* dy,
                                                      float* dgate, int32_t* dev_err,
                                                      moe_stream_t stream) {
  using namespace moe;
  if (T < 0 || K < 0 || d <= 0 || rows < 0) return MOE_ERR_INVALID_ARG;
  if (d % 128 != 0) return MOE_ERR_SHAPE;
  const int64_t P = static_cast<int64_t>(T) * K;
  if (K > kCkMaxK || rows > 0x7FFFFFFFll || P + T > 0x7FFFFFFFll) return MOE_ERR_UNSUPPORTED;
  if (T == 0) return MOE_OK;
  if (K > 0 && rows > P) return MOE_ERR_SHAPE;  // no gradient row for a pair behind the T*K-th
  if (!dout || !dyq || !dys ||
      (K > 0 && (!dst_of || !topk_gate || !dgate || (rows > 0 && (!yq || !ys)))))
    return MOE_ERR_INVALID_ARG;
  if (!aligned16(dout) || !aligned16(yq) || !aligned16(dyq) || !aligned16(dy) || !aligned4(ys) ||
      !aligned4(dys) || !aligned4(dgate) || !aligned4(dst_of) || !aligned4(topk_gate))
    return MOE_ERR_ALIGN;
  const Shape sh = ck_shape(T, K, d / 128);
  const bool many = sh.block.x * sh.block.y > 32 * kCkWarps;
  auto kern = K > 4 ? pick_backward<8>(dy, many) : (K > 2 ? pick_backward<4>(dy, many) : pick_backward<2>(dy, many));
  kern<<<sh.grid, sh.block, sh.smem, static_cast<cudaStream_t>(stream)>>>(
      dout, dst_of, topk_gate, yq, ys, rows, T, K, d, dyq, dys, dy, dgate, dev_err);
  MOE_CUDA_CHECK_LAUNCH();
  return MOE_OK;
}
