// The combine with an 8-bit checkpoint of the expert outputs, and its
// backward from the checkpoint.
// "DeepSeek_V3_Report：Annotation", eq. (12), "Fine-Grained Quantization",
// "Low-Precision Activation" (activations kept for the backward in FP8) and
// "Low-Precision Communication" (gradients quantised with power-of-two scales).
//
//   moe_combine_checkpoint           out = u + Ys + sum_k gate_k Y[r_k];  yq, ys = Q(Y[r_k])
//   moe_combine_checkpoint_backward  dy[r_k] = Q2(gate_k dout);  dgate_k = dout . (yq ys)[r_k]
//
// Both are HBM-bound streaming kernels, one CTA per token.  A warp takes four
// 128-column tiles at a time, eight lanes a tile: lane l of a tile holds the
// columns 32 s + 4 l .. + 3 (s = 0..3), so that every fp32 access is a
// coalesced 16-byte one and a tile's maximum takes three shuffles for 16
// values a lane (one lane per 4 values would take five).
#include <cuda_fp8.h>

#include "epi_math.cuh"
#include "moe_common.cuh"

namespace moe {
namespace {

constexpr int kCkMaxWarps = 16;
constexpr int kCkMaxK = 32;
constexpr int kCkTiles = 4;  // tiles of one warp step

// Warps of a CTA and steps of a warp for a row of so many tiles.
inline int ck_warps(int tiles) {
  const int items = (tiles + kCkTiles - 1) / kCkTiles;
  const int steps = (items + kCkMaxWarps - 1) / kCkMaxWarps;
  return (items + steps - 1) / steps;
}

__device__ __forceinline__ void codes_to_float(uint32_t w, float (&f)[4]) {
  const __half2_raw lo = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(w & 0xFFFFu), __NV_E4M3);
  const __half2_raw hi = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(w >> 16), __NV_E4M3);
  const float2 a = __half22float2(__half2(lo));
  const float2 b = __half22float2(__half2(hi));
  f[0] = a.x;
  f[1] = a.y;
  f[2] = b.x;
  f[3] = b.y;
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

// The token's pairs, one a lane: sorted row (-1 dropped) and gate.
__device__ __forceinline__ void load_pair(const int32_t* __restrict__ dst_of,
                                          const float* __restrict__ gate, int64_t t, int K, int lane,
                                          int64_t rows, int& row, float& g, int32_t* dev_err) {
  row = -1;
  g = 0.f;
  if (lane < K) {
    row = __ldg(dst_of + t * K + lane);
    g = __ldg(gate + t * K + lane);
    if (row >= rows) {
      set_dev_err(dev_err, MOE_DEVERR_BAD_INDEX);
      row = -1;
    }
  }
}

template <bool POW2>
__global__ void __launch_bounds__(32 * kCkMaxWarps) combine_checkpoint_kernel(
    const float* __restrict__ Y, int64_t rows, const int32_t* __restrict__ dst_of,
    const float* __restrict__ gate, const float* __restrict__ Ysh, const uint16_t* __restrict__ u,
    int K, int d, float* __restrict__ out, uint8_t* __restrict__ yq, float* __restrict__ ys,
    int32_t* dev_err) {
  const int64_t t = blockIdx.x;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  int row;
  float g;
  load_pair(dst_of, gate, t, K, lane, rows, row, g, dev_err);
  const uint32_t kept = __ballot_sync(0xffffffffu, row >= 0);
  const int tiles = d / 128;
  for (int item = warp; item * kCkTiles < tiles; item += warps) {
    const int j = item * kCkTiles + (lane >> 3);
    const bool in = j < tiles;               // the last step may hold fewer tiles
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
}

// dout is read once a tile and gives all K + 1 gradient tiles.  Its largest
// magnitude is found once: rounding is monotone, so the largest |fl(g x)| is
// fl(|g| max |x|).  Power-of-two scales divide exactly, so one product with
// the inverse gives the quotient.
__global__ void __launch_bounds__(32 * kCkMaxWarps) combine_checkpoint_backward_kernel(
    const float* __restrict__ dout, const int32_t* __restrict__ dst_of,
    const float* __restrict__ gate, const uint8_t* __restrict__ yq, const float* __restrict__ ys,
    int64_t rows, int64_t P, int K, int d, uint8_t* __restrict__ dyq, float* __restrict__ dys,
    float* __restrict__ dy, float* __restrict__ dgate, int32_t* dev_err) {
  __shared__ float dot[kCkMaxWarps][kCkMaxK];
  const int64_t t = blockIdx.x;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  int row;
  float g;
  load_pair(dst_of, gate, t, K, lane, rows < P ? rows : P, row, g, dev_err);
  const uint32_t kept = __ballot_sync(0xffffffffu, row >= 0);
  const int tiles = d / 128;
  dot[warp][lane] = 0.f;
  __syncwarp();
  for (int item = warp; item * kCkTiles < tiles; item += warps) {
    const int j = item * kCkTiles + (lane >> 3);
    const bool in = j < tiles;
    const int64_t col = static_cast<int64_t>(j) * 128 + 4 * (lane & 7);
    float4 a[4];
#pragma unroll
    for (int s = 0; s < 4; ++s)
      a[s] = in ? __ldg(reinterpret_cast<const float4*>(dout + t * d + col + 32 * s)) : make_float4(0.f, 0.f, 0.f, 0.f);
    uint32_t next[4];
    float next_scale = 0.f;
    auto fetch = [&](uint32_t left) {
      const int64_t r = __shfl_sync(0xffffffffu, row, __ffs(left) - 1);
#pragma unroll
      for (int s = 0; s < 4; ++s)
        next[s] = in ? __ldg(reinterpret_cast<const uint32_t*>(yq + r * d + col + 32 * s)) : 0u;
      next_scale = in ? __ldg(ys + r * tiles + j) : 0.f;
    };
    if (kept) fetch(kept);
    const float amax = tile_amax(a);
    auto write_row = [&](int64_t r, float w) {
      const float scale = pow2_ceil(quant_scale(__fmul_rn(fabsf(w), amax)));
      // an infinite maximum leaves no finite scale: every code is NaN
      const float inv = scale < INFINITY ? __frcp_rn(scale) : NAN;
#pragma unroll
      for (int s = 0; s < 4; ++s) {
        const float4 v = make_float4(__fmul_rn(w, a[s].x), __fmul_rn(w, a[s].y), __fmul_rn(w, a[s].z),
                                     __fmul_rn(w, a[s].w));
        *reinterpret_cast<uint32_t*>(dyq + r * d + col + 32 * s) =
            e4m3x4(__fmul_rn(v.x, inv), __fmul_rn(v.y, inv), __fmul_rn(v.z, inv), __fmul_rn(v.w, inv));
        if (dy) *reinterpret_cast<float4*>(dy + r * d + col + 32 * s) = v;
      }
      if ((lane & 7) == 0) dys[r * tiles + j] = scale;
    };
    if (in) write_row(P + t, 1.0f);
    for (uint32_t left = kept; left;) {
      const int k = __ffs(left) - 1;
      left &= left - 1;
      uint32_t code[4];
      const float scale = next_scale;
#pragma unroll
      for (int s = 0; s < 4; ++s) code[s] = next[s];
      if (left) fetch(left);
      const int64_t r = __shfl_sync(0xffffffffu, row, k);
      const float w = __shfl_sync(0xffffffffu, g, k);
      if (in) write_row(r, w);
      float p = 0.f;
#pragma unroll
      for (int s = 0; s < 4; ++s) {
        float f[4];
        codes_to_float(code[s], f);
        p = fmaf(a[s].w, f[3], fmaf(a[s].z, f[2], fmaf(a[s].y, f[1], fmaf(a[s].x, f[0], p))));
      }
      p = __fmul_rn(p, scale);
#pragma unroll
      for (int off = 16; off > 0; off >>= 1) p += __shfl_xor_sync(0xffffffffu, p, off);
      if (lane == 0) dot[warp][k] += p;
    }
  }
  __syncthreads();
  if (threadIdx.x < K) {
    float sum = 0.f;
    for (int w = 0; w < warps; ++w) sum += dot[w][threadIdx.x];
    dgate[t * K + threadIdx.x] = sum;
  }
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
  kern<<<T, 32 * ck_warps(d / 128), 0, static_cast<cudaStream_t>(stream)>>>(
      Y, rows, dst_of, topk_gate, Y_shared, u, K, d, out, yq, ys, dev_err);
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
  if (!dout || !dyq || !dys ||
      (K > 0 && (!dst_of || !topk_gate || !dgate || (rows > 0 && (!yq || !ys)))))
    return MOE_ERR_INVALID_ARG;
  if (!aligned16(dout) || !aligned16(yq) || !aligned16(dyq) || !aligned16(dy) || !aligned4(ys) ||
      !aligned4(dys) || !aligned4(dgate) || !aligned4(dst_of) || !aligned4(topk_gate))
    return MOE_ERR_ALIGN;
  combine_checkpoint_backward_kernel<<<T, 32 * ck_warps(d / 128), 0, static_cast<cudaStream_t>(stream)>>>(
      dout, dst_of, topk_gate, yq, ys, rows, P, K, d, dyq, dys, dy, dgate, dev_err);
  MOE_CUDA_CHECK_LAUNCH();
  return MOE_OK;
}
