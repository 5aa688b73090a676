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
//  2. du = du_base + dz C and dC = dz^T u, in fp32.
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
    float* __restrict__ dz, int32_t* dev_err) {
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
#pragma unroll
  for (int i = 0; i < P; ++i)
    if (32 * i + lane < E) dz[t * E + 32 * i + lane] = out[i];
}

// D [M][N] = base + A B over depth L, with 64 x 64 tiles and 4 x 4 values a
// thread; A and B rows are read through (outer, depth) strides.
template <bool TRANS_A>
__global__ void __launch_bounds__(256) product_kernel(const float* __restrict__ A,
                                                      const uint16_t* __restrict__ B, int64_t ldb,
                                                      int M, int N, int L, int E,
                                                      const float* base, float* D) {
  __shared__ float sa[16][64 + 4];
  __shared__ float sb[16][64 + 4];
  const int m0 = blockIdx.y * 64, n0 = blockIdx.x * 64;
  const int tm = threadIdx.x / 16, tn = threadIdx.x % 16;
  float acc[4][4] = {};
  for (int l0 = 0; l0 < L; l0 += 16) {
    for (int i = threadIdx.x; i < 16 * 64; i += 256) {
      const int n = i % 64, lb = i / 64;
      sb[lb][n] = (l0 + lb < L && n0 + n < N)
                      ? bf16_bits_to_float(B[static_cast<int64_t>(l0 + lb) * ldb + n0 + n]) : 0.f;
      const int m = TRANS_A ? i % 64 : i / 16, la = TRANS_A ? i / 64 : i % 16;
      float v = 0.f;
      if (l0 + la < L && m0 + m < M)
        v = TRANS_A ? A[static_cast<int64_t>(l0 + la) * E + m0 + m]
                    : A[static_cast<int64_t>(m0 + m) * E + l0 + la];
      sa[la][m] = v;
    }
    __syncthreads();
#pragma unroll
    for (int l = 0; l < 16; ++l) {
      float a[4], b[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        a[i] = sa[l][4 * tm + i];
        b[i] = sb[l][4 * tn + i];
      }
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = fmaf(a[i], b[j], acc[i][j]);
    }
    __syncthreads();
  }
  for (int i = 0; i < 4; ++i)
    for (int j = 0; j < 4; ++j) {
      const int m = m0 + 4 * tm + i, n = n0 + 4 * tn + j;
      if (m < M && n < N) {
        const int64_t at = static_cast<int64_t>(m) * N + n;
        D[at] = base ? __fadd_rn(base[at], acc[i][j]) : acc[i][j];
      }
    }
}

template <int P>
void launch_dlogits(cudaStream_t st, const float* dgate, const float* logits, const int32_t* idx,
                    const float* gate, int T, int E, int K, const float* f, const float* dloss,
                    int seq_len, float alpha, float* dz, int32_t* dev_err) {
  const int blocks = (T + kRgThreads / 32 - 1) / (kRgThreads / 32);
  dlogits_kernel<P><<<blocks, kRgThreads, 0, st>>>(dgate, logits, idx, gate, T, E, K, f, dloss,
                                                   seq_len, alpha, dz, dev_err);
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
  *bytes = (static_cast<size_t>(T) * E * sizeof(float) + 255) / 256 * 256;
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
  float* dz = dlogits ? dlogits : static_cast<float*>(ws);
  const int P = (E + 31) / 32;
  auto go = P <= 1 ? launch_dlogits<1> : P <= 2 ? launch_dlogits<2> : P <= 4 ? launch_dlogits<4>
          : P <= 8 ? launch_dlogits<8> : P <= 12 ? launch_dlogits<12> : P <= 16 ? launch_dlogits<16>
          : launch_dlogits<32>;
  go(st, dgate, logits, topk_idx, topk_gate, T, E, K, f, dloss, seq_len, alpha, dz, dev_err);
  MOE_CUDA_CHECK_LAUNCH();
  if (du) {
    dim3 grid((d + 63) / 64, (T + 63) / 64);
    product_kernel<false><<<grid, 256, 0, st>>>(dz, centroids, d, T, d, E, E, du_base, du);
    MOE_CUDA_CHECK_LAUNCH();
  }
  if (dcentroids) {
    dim3 grid((d + 63) / 64, (E + 63) / 64);
    product_kernel<true><<<grid, 256, 0, st>>>(dz, u, ldu, E, d, T, E, nullptr, dcentroids);
    MOE_CUDA_CHECK_LAUNCH();
  }
  return MOE_OK;
}
