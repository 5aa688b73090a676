// Tokens sorted by expert and back in 16 or 32 bits, with both gradients.
// "DeepSeek_V3_Report：Annotation", eq. (12) (the routed experts' outputs
// weighted by the gates).
//
//   moe_sort_rows             xs[dst[t][k]] = x[t]
//   moe_sort_rows_backward    dx[t] = sum_k dxs[dst[t][k]]
//   moe_unsort_rows           out[t] = sum_k w[t][k] y[dst[t][k]]
//   moe_unsort_rows_backward  dy[dst[t][k]] = w[t][k] dout[t], dw[t][k] = dout[t] . y[dst[t][k]]
//
// Two shapes of kernel: a scatter (one token row to K sorted rows) and a
// gather (K sorted rows to one token row).  Both are bound by HBM: every row
// is read once and written once, with a few fp32 operations an element.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "moe_common.cuh"

namespace moe {
namespace {

constexpr int kSrThreads = 256;
constexpr int kSrMaxK = 32;

// N elements of T as one access: 16 bytes, or a single element where the
// rows' alignment allows no more.
template <typename T, int N>
struct alignas(sizeof(T) * N) Pack {
  T e[N];
};

__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(__half v) { return __half2float(v); }
__device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
template <typename T>
__device__ __forceinline__ T from_f32(float v);
template <>
__device__ __forceinline__ float from_f32<float>(float v) { return v; }
template <>
__device__ __forceinline__ __half from_f32<__half>(float v) { return __float2half_rn(v); }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v) {
  return __float2bfloat16_rn(v);
}

// The token's sorted rows and weights into shared memory; -1 for a dropped pair.
__device__ __forceinline__ void load_pairs(const int32_t* __restrict__ dst_of,
                                           const float* __restrict__ weight, int64_t t, int K,
                                           int64_t rows, int64_t* row_sm, float* w_sm,
                                           int32_t* dev_err) {
  if (threadIdx.x < K) {
    const int64_t r = dst_of[t * K + threadIdx.x];
    if (r >= rows) set_dev_err(dev_err, MOE_DEVERR_BAD_INDEX);
    row_sm[threadIdx.x] = (r < 0 || r >= rows) ? -1 : r;
    w_sm[threadIdx.x] = weight ? weight[t * K + threadIdx.x] : 1.0f;
  }
  __syncthreads();
}

// One CTA per token.  WEIGHTED: dst row = round(w * src); DOT: also the dot
// product of the token row with each sorted row of y.
template <typename T, int N, bool WEIGHTED, bool DOT>
__global__ void __launch_bounds__(kSrThreads) scatter_rows_kernel(
    const T* __restrict__ src, int64_t lds, const int32_t* __restrict__ dst_of,
    const float* __restrict__ weight, int K, int d, const T* __restrict__ y, int64_t ldy,
    T* __restrict__ dst, int64_t ldd, int64_t rows, float* __restrict__ dweight,
    int32_t* dev_err) {
  __shared__ int64_t row[kSrMaxK];
  __shared__ float w[kSrMaxK];
  __shared__ float part[kSrThreads / 32];
  const int64_t t = blockIdx.x;
  load_pairs(dst_of, weight, t, K, rows, row, w, dev_err);
  const Pack<T, N>* s = reinterpret_cast<const Pack<T, N>*>(src + t * lds);
  const int nv = d / N;
  for (int k = 0; k < K; ++k) {
    const int64_t r = row[k];
    float acc = 0.f;
    if (r >= 0) {
      for (int v = threadIdx.x; v < nv; v += kSrThreads) {
        const Pack<T, N> a = s[v];
        if (dst) {
          Pack<T, N> o = a;
          if (WEIGHTED) {
#pragma unroll
            for (int i = 0; i < N; ++i) o.e[i] = from_f32<T>(__fmul_rn(w[k], to_f32(a.e[i])));
          }
          reinterpret_cast<Pack<T, N>*>(dst + r * ldd)[v] = o;
        }
        if (DOT) {
          const Pack<T, N> b = reinterpret_cast<const Pack<T, N>*>(y + r * ldy)[v];
#pragma unroll
          for (int i = 0; i < N; ++i) acc = fmaf(to_f32(a.e[i]), to_f32(b.e[i]), acc);
        }
      }
    }
    if (DOT) {
#pragma unroll
      for (int off = 16; off > 0; off >>= 1) acc += __shfl_xor_sync(0xffffffffu, acc, off);
      if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = acc;
      __syncthreads();
      if (threadIdx.x == 0) {
        float sum = 0.f;
#pragma unroll
        for (int i = 0; i < kSrThreads / 32; ++i) sum += part[i];
        dweight[t * K + k] = sum;
      }
      __syncthreads();
    }
  }
}

// One CTA per token: the K rows added in k order in fp32, rounded once.
template <typename T, int N, bool WEIGHTED>
__global__ void __launch_bounds__(kSrThreads) gather_rows_kernel(
    const T* __restrict__ src, int64_t lds, int64_t rows, const int32_t* __restrict__ dst_of,
    const float* __restrict__ weight, int K, int d, T* __restrict__ out, int64_t ldo,
    int32_t* dev_err) {
  __shared__ int64_t row[kSrMaxK];
  __shared__ float w[kSrMaxK];
  const int64_t t = blockIdx.x;
  load_pairs(dst_of, weight, t, K, rows, row, w, dev_err);
  const int nv = d / N;
  for (int v = threadIdx.x; v < nv; v += kSrThreads) {
    float acc[N];
#pragma unroll
    for (int i = 0; i < N; ++i) acc[i] = 0.f;
    for (int k = 0; k < K; ++k) {
      if (row[k] < 0) continue;
      const Pack<T, N> a = reinterpret_cast<const Pack<T, N>*>(src + row[k] * lds)[v];
#pragma unroll
      for (int i = 0; i < N; ++i)
        acc[i] = WEIGHTED ? fmaf(w[k], to_f32(a.e[i]), acc[i]) : __fadd_rn(acc[i], to_f32(a.e[i]));
    }
    Pack<T, N> o;
#pragma unroll
    for (int i = 0; i < N; ++i) o.e[i] = from_f32<T>(acc[i]);
    reinterpret_cast<Pack<T, N>*>(out + t * ldo)[v] = o;
  }
}

int elem_bytes(moe_dtype dt) { return dt == MOE_F32 ? 4 : 2; }

bool elem_aligned(const void* p, int e) {
  return (reinterpret_cast<uintptr_t>(p) & static_cast<uintptr_t>(e - 1)) == 0;
}

// Whether every row starting at p with stride ld can be accessed 16 bytes at a time.
bool rows_aligned16(const void* p, int64_t ld, int e) {
  return (reinterpret_cast<uintptr_t>(p) & 15u) == 0 && (ld * e) % 16 == 0;
}

moe_status check_shape(moe_dtype dt, int T, int K, int d, int64_t rows) {
  if (dt != MOE_BF16 && dt != MOE_F16 && dt != MOE_F32) return MOE_ERR_INVALID_ARG;
  if (T < 0 || K < 0 || d <= 0 || rows < 0) return MOE_ERR_INVALID_ARG;
  if (K > kSrMaxK || rows > 0x7FFFFFFFll) return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

template <typename T, int N>
struct Access {
  using type = T;
  static constexpr int n = N;
};

// fn(Access<T, N>) for the call's element type; N is 16 bytes' worth where
// every row involved is 16-byte aligned, else one element.
template <typename F>
void with_access(moe_dtype dt, bool wide, F&& fn) {
  if (dt == MOE_BF16) wide ? fn(Access<__nv_bfloat16, 8>{}) : fn(Access<__nv_bfloat16, 1>{});
  else if (dt == MOE_F16) wide ? fn(Access<__half, 8>{}) : fn(Access<__half, 1>{});
  else wide ? fn(Access<float, 4>{}) : fn(Access<float, 1>{});
}

moe_status gather(const void* src, moe_dtype dt, int64_t lds, int64_t rows, const int32_t* dst_of,
                  const float* weight, bool weighted, int T, int K, int d, void* out, int64_t ldo,
                  int32_t* dev_err, cudaStream_t st) {
  const moe_status s = check_shape(dt, T, K, d, rows);
  if (s != MOE_OK) return s;
  if (lds < d || ldo < d) return MOE_ERR_SHAPE;
  if (T == 0) return MOE_OK;
  if (!out || (K > 0 && (!dst_of || (weighted && !weight) || (rows > 0 && !src))))
    return MOE_ERR_INVALID_ARG;
  const int e = elem_bytes(dt);
  if (!elem_aligned(src, e) || !elem_aligned(out, e) || !elem_aligned(dst_of, 4) ||
      !elem_aligned(weight, 4))
    return MOE_ERR_ALIGN;
  const bool wide = rows_aligned16(src, lds, e) && rows_aligned16(out, ldo, e) &&
                    (static_cast<int64_t>(d) * e) % 16 == 0;
  with_access(dt, wide, [&](auto access) {
    using E = typename decltype(access)::type;
    constexpr int N = decltype(access)::n;
    auto kern = weighted ? gather_rows_kernel<E, N, true> : gather_rows_kernel<E, N, false>;
    kern<<<T, kSrThreads, 0, st>>>(static_cast<const E*>(src), lds, rows, dst_of, weight, K, d,
                                   static_cast<E*>(out), ldo, dev_err);
  });
  MOE_CUDA_CHECK_LAUNCH();
  return MOE_OK;
}

}  // namespace
}  // namespace moe

extern "C" moe_status moe_sort_rows(const void* x, moe_dtype dtype, int64_t ldx,
                                    const int32_t* dst_of, int T, int K, int d, void* xs,
                                    int64_t ldxs, int64_t rows, int32_t* dev_err,
                                    moe_stream_t stream) {
  using namespace moe;
  const moe_status s = check_shape(dtype, T, K, d, rows);
  if (s != MOE_OK) return s;
  if (ldx < d || ldxs < d) return MOE_ERR_SHAPE;
  if (T == 0 || K == 0) return MOE_OK;
  if (!x || !dst_of || (rows > 0 && !xs)) return MOE_ERR_INVALID_ARG;
  const int e = elem_bytes(dtype);
  if (!elem_aligned(x, e) || !elem_aligned(xs, e) || !elem_aligned(dst_of, 4)) return MOE_ERR_ALIGN;
  const bool wide = rows_aligned16(x, ldx, e) && rows_aligned16(xs, ldxs, e) &&
                    (static_cast<int64_t>(d) * e) % 16 == 0;
  with_access(dtype, wide, [&](auto access) {
    using E = typename decltype(access)::type;
    constexpr int N = decltype(access)::n;
    scatter_rows_kernel<E, N, false, false><<<T, kSrThreads, 0, static_cast<cudaStream_t>(stream)>>>(
        static_cast<const E*>(x), ldx, dst_of, nullptr, K, d, nullptr, 0, static_cast<E*>(xs), ldxs,
        rows, nullptr, dev_err);
  });
  MOE_CUDA_CHECK_LAUNCH();
  return MOE_OK;
}

extern "C" moe_status moe_sort_rows_backward(const void* dxs, moe_dtype dtype, int64_t ldxs,
                                             int64_t rows, const int32_t* dst_of, int T, int K,
                                             int d, void* dx, int64_t ldx, int32_t* dev_err,
                                             moe_stream_t stream) {
  return moe::gather(dxs, dtype, ldxs, rows, dst_of, nullptr, false, T, K, d, dx, ldx, dev_err,
                     static_cast<cudaStream_t>(stream));
}

extern "C" moe_status moe_unsort_rows(const void* y, moe_dtype dtype, int64_t ldy, int64_t rows,
                                      const int32_t* dst_of, const float* weight, int T, int K,
                                      int d, void* out, int64_t ldo, int32_t* dev_err,
                                      moe_stream_t stream) {
  return moe::gather(y, dtype, ldy, rows, dst_of, weight, true, T, K, d, out, ldo, dev_err,
                     static_cast<cudaStream_t>(stream));
}

extern "C" moe_status moe_unsort_rows_backward(const void* dout, moe_dtype dtype, int64_t ldo,
                                               const void* y, int64_t ldy, const int32_t* dst_of,
                                               const float* weight, int T, int K, int d, void* dy,
                                               int64_t lddy, int64_t rows, float* dweight,
                                               int32_t* dev_err, moe_stream_t stream) {
  using namespace moe;
  const moe_status s = check_shape(dtype, T, K, d, rows);
  if (s != MOE_OK) return s;
  if (ldo < d || (dy && lddy < d) || (dweight && ldy < d)) return MOE_ERR_SHAPE;
  if (T == 0 || K == 0) return MOE_OK;
  if (!dout || !dst_of || (dy && !weight) || (dweight && rows > 0 && !y) || (!dy && !dweight && rows > 0))
    return MOE_ERR_INVALID_ARG;
  const int e = elem_bytes(dtype);
  if (!elem_aligned(dout, e) || !elem_aligned(y, e) || !elem_aligned(dy, e) ||
      !elem_aligned(dst_of, 4) || !elem_aligned(weight, 4) || !elem_aligned(dweight, 4))
    return MOE_ERR_ALIGN;
  const bool wide = rows_aligned16(dout, ldo, e) && (!dy || rows_aligned16(dy, lddy, e)) &&
                    (!dweight || rows_aligned16(y, ldy, e)) && (static_cast<int64_t>(d) * e) % 16 == 0;
  with_access(dtype, wide, [&](auto access) {
    using E = typename decltype(access)::type;
    constexpr int N = decltype(access)::n;
    auto kern = dweight ? scatter_rows_kernel<E, N, true, true> : scatter_rows_kernel<E, N, true, false>;
    kern<<<T, kSrThreads, 0, static_cast<cudaStream_t>(stream)>>>(
        static_cast<const E*>(dout), ldo, dst_of, weight, K, d, static_cast<const E*>(y), ldy,
        static_cast<E*>(dy), lddy, rows, dweight, dev_err);
  });
  MOE_CUDA_CHECK_LAUNCH();
  return MOE_OK;
}
