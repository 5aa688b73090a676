// The combine with an 8-bit checkpoint of the expert outputs, and its
// backward from the checkpoint.
// "DeepSeek_V3_Report：Annotation", eq. (12), "Fine-Grained Quantization",
// "Low-Precision Activation" (activations kept for the backward in FP8) and
// "Low-Precision Communication" (gradients quantised with power-of-two scales).
//
//   moe_combine_checkpoint           out = u + Ys + sum_k gate_k Y[r_k];  yq, ys = Q(Y[r_k])
//   moe_combine_checkpoint_backward  dy[r_k] = Q2(gate_k dout);  dgate_k = dout . (yq ys)[r_k]
//
// Both are HBM-bound streaming kernels, one CTA per token.
#include <cuda_fp8.h>

#include "epi_math.cuh"
#include "moe_common.cuh"

namespace moe {
namespace {

constexpr int kCkThreads = 256;
constexpr int kCkWarps = kCkThreads / 32;
constexpr int kCkMaxK = 32;

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

__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, off));
  return v;
}

__device__ __forceinline__ uint32_t quant4(const float4& v, float s) {
  const float rs = __frcp_rn(s);
  return e4m3x4(div_by_scale(v.x, s, rs), div_by_scale(v.y, s, rs), div_by_scale(v.z, s, rs),
                div_by_scale(v.w, s, rs));
}

__device__ __forceinline__ float amax4(const float4& v) {
  return fmaxf(fmaxf(fabsf(v.x), fabsf(v.y)), fmaxf(fabsf(v.z), fabsf(v.w)));
}

// One warp per 128-column tile: its K rows are read once, quantised and added.
template <bool POW2>
__global__ void __launch_bounds__(kCkThreads) combine_checkpoint_kernel(
    const float* __restrict__ Y, int64_t rows, const int32_t* __restrict__ dst_of,
    const float* __restrict__ gate, const float* __restrict__ Ysh, const uint16_t* __restrict__ u,
    int K, int d, float* __restrict__ out, uint8_t* __restrict__ yq, float* __restrict__ ys,
    int32_t* dev_err) {
  __shared__ int64_t row[kCkMaxK];
  __shared__ float gs[kCkMaxK];
  const int64_t t = blockIdx.x;
  if (threadIdx.x < K) {
    const int64_t r = dst_of[t * K + threadIdx.x];
    if (r >= rows) set_dev_err(dev_err, MOE_DEVERR_BAD_INDEX);
    row[threadIdx.x] = (r < 0 || r >= rows) ? -1 : r;
    gs[threadIdx.x] = gate[t * K + threadIdx.x];
  }
  __syncthreads();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int tiles = d / 128;
  for (int j = warp; j < tiles; j += kCkWarps) {
    const uint2 ub = __ldg(reinterpret_cast<const uint2*>(u + t * d + j * 128) + lane);
    float4 acc = make_float4(bf16_bits_to_float(ub.x & 0xFFFFu), bf16_bits_to_float(ub.x >> 16),
                             bf16_bits_to_float(ub.y & 0xFFFFu), bf16_bits_to_float(ub.y >> 16));
    if (Ysh) {
      const float4 s = __ldg(reinterpret_cast<const float4*>(Ysh + t * d + j * 128) + lane);
      acc.x += s.x;
      acc.y += s.y;
      acc.z += s.z;
      acc.w += s.w;
    }
    for (int k = 0; k < K; ++k) {
      const int64_t r = row[k];
      if (r < 0) continue;
      const float4 v = __ldg(reinterpret_cast<const float4*>(Y + r * d + j * 128) + lane);
      const float g = gs[k];
      acc.x = fmaf(g, v.x, acc.x);
      acc.y = fmaf(g, v.y, acc.y);
      acc.z = fmaf(g, v.z, acc.z);
      acc.w = fmaf(g, v.w, acc.w);
      const float s0 = quant_scale(warp_max(amax4(v)));
      const float s = POW2 ? pow2_ceil(s0) : s0;
      reinterpret_cast<uint32_t*>(yq + r * d + j * 128)[lane] = quant4(v, s);
      if (lane == 0) ys[r * tiles + j] = s;
    }
    reinterpret_cast<float4*>(out + t * d + j * 128)[lane] = acc;
  }
}

// One warp per 128-column tile: dout's tile is read once and gives the K + 1
// gradient tiles; the checkpoint's tile of each row adds to that gate's dot.
__global__ void __launch_bounds__(kCkThreads) combine_checkpoint_backward_kernel(
    const float* __restrict__ dout, const int32_t* __restrict__ dst_of,
    const float* __restrict__ gate, const uint8_t* __restrict__ yq, const float* __restrict__ ys,
    int64_t rows, int64_t P, int K, int d, uint8_t* __restrict__ dyq, float* __restrict__ dys,
    float* __restrict__ dy, float* __restrict__ dgate, int32_t* dev_err) {
  __shared__ int64_t row[kCkMaxK + 1];
  __shared__ float gs[kCkMaxK + 1];
  __shared__ float dot[kCkWarps][kCkMaxK];
  const int64_t t = blockIdx.x;
  if (threadIdx.x < K) {
    const int64_t r = dst_of[t * K + threadIdx.x];
    const bool bad = r >= rows || r >= P;
    if (bad) set_dev_err(dev_err, MOE_DEVERR_BAD_INDEX);
    row[threadIdx.x] = (r < 0 || bad) ? -1 : r;
    gs[threadIdx.x] = gate[t * K + threadIdx.x];
  }
  if (threadIdx.x == K) {
    row[K] = P + t;
    gs[K] = 1.0f;
  }
  __syncthreads();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int tiles = d / 128;
  if (lane < K) dot[warp][lane] = 0.f;
  __syncwarp();
  for (int j = warp; j < tiles; j += kCkWarps) {
    const float4 a = __ldg(reinterpret_cast<const float4*>(dout + t * d + j * 128) + lane);
    for (int k = 0; k <= K; ++k) {
      const int64_t r = row[k];
      if (r < 0) continue;
      const float g = gs[k];
      const float4 v = make_float4(__fmul_rn(g, a.x), __fmul_rn(g, a.y), __fmul_rn(g, a.z),
                                   __fmul_rn(g, a.w));
      const float s = pow2_ceil(quant_scale(warp_max(amax4(v))));
      reinterpret_cast<uint32_t*>(dyq + r * d + j * 128)[lane] = quant4(v, s);
      if (lane == 0) dys[r * tiles + j] = s;
      if (dy) reinterpret_cast<float4*>(dy + r * d + j * 128)[lane] = v;
      if (k < K) {
        float f[4];
        codes_to_float(__ldg(reinterpret_cast<const uint32_t*>(yq + r * d + j * 128) + lane), f);
        float p = fmaf(a.w, f[3], fmaf(a.z, f[2], fmaf(a.y, f[1], __fmul_rn(a.x, f[0]))));
        p = __fmul_rn(p, __ldg(ys + r * tiles + j));
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) p += __shfl_xor_sync(0xffffffffu, p, off);
        if (lane == 0) dot[warp][k] += p;
      }
    }
  }
  __syncthreads();
  if (threadIdx.x < K) {
    float sum = 0.f;
#pragma unroll
    for (int w = 0; w < kCkWarps; ++w) sum += dot[w][threadIdx.x];
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
  kern<<<T, kCkThreads, 0, static_cast<cudaStream_t>(stream)>>>(Y, rows, dst_of, topk_gate, Y_shared,
                                                               u, K, d, out, yq, ys, dev_err);
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
  combine_checkpoint_backward_kernel<<<T, kCkThreads, 0, static_cast<cudaStream_t>(stream)>>>(
      dout, dst_of, topk_gate, yq, ys, rows, P, K, d, dyq, dys, dy, dgate, dev_err);
  MOE_CUDA_CHECK_LAUNCH();
  return MOE_OK;
}
