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
// is read once and written once, with a few fp32 operations an element.  A
// warp takes one stretch of a token's columns through all of its K rows: where
// sorted rows are read, the loads of several are in flight together (accesses a
// lane: the gather 8, or 16 of 4 bytes; the dot products 4, or 8 narrow ones; the
// scatter reads one token row, 1 to 8 accesses, for its K rows of stores), and the
// token's values stay in registers as the words they were read as (as separate
// 16-bit elements they cost twice the registers, and with them half the warps that
// hide the latency).
// One B200, rows of 7168 in bf16, one of several launches in a graph, of the
// measured copy rate of 6.44 TB/s (a call in a loop takes about 2 us more):
//   sort            4096 tokens x 8: 87 us, 95%     its backward:    83 us, 99%
//   unsort backward 16384 x 6:      474 us, 100%    one token's sort: 1.8 us
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "moe_common.cuh"

namespace moe {
namespace {

constexpr int kSrMaxK = 32;
constexpr int kSrWarps = 4;      // warps of a CTA, each with a piece of its own
constexpr int kSrDotWarps = 16;  // most warps of a CTA whose warps share a token
constexpr int kSrFlight = 8;     // 16-byte accesses a lane of the gather has in flight: U columns x kSrFlight / U rows

// Columns and rows a lane of the dot kernel has in flight: fewer than elsewhere,
// so that 32 warps an SM fit (16384 x 6: 474 us; four columns 597).
template <int N>
constexpr int kSrDotU = N <= 2 ? 4 : 2;
constexpr int kSrDotB = 2;

// N elements of T as one access of plain words (16 bytes, or where the rows'
// alignment allows no more 4 bytes or a single element), and as floats.
template <typename T, int N>
struct Row;

template <>
struct Row<float, 4> {
  using Raw = uint4;
  static __device__ __forceinline__ void get(const uint4& v, float (&f)[4]) {
    f[0] = __uint_as_float(v.x);
    f[1] = __uint_as_float(v.y);
    f[2] = __uint_as_float(v.z);
    f[3] = __uint_as_float(v.w);
  }
  static __device__ __forceinline__ uint4 put(const float (&f)[4]) {
    return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]),
                      __float_as_uint(f[3]));
  }
};

template <>
struct Row<float, 1> {
  using Raw = uint32_t;
  static __device__ __forceinline__ void get(uint32_t v, float (&f)[1]) { f[0] = __uint_as_float(v); }
  static __device__ __forceinline__ uint32_t put(const float (&f)[1]) { return __float_as_uint(f[0]); }
};

__device__ __forceinline__ float2 two(uint32_t w, __nv_bfloat16) {
  return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
}
__device__ __forceinline__ float2 two(uint32_t w, __half) {
  return __half22float2(*reinterpret_cast<const __half2*>(&w));
}
__device__ __forceinline__ uint32_t two(float lo, float hi, __nv_bfloat16) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ uint32_t two(float lo, float hi, __half) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

template <typename T>
struct Row<T, 8> {
  using Raw = uint4;
  static __device__ __forceinline__ void get(const uint4& v, float (&f)[8]) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 p = two(w[i], T{});
      f[2 * i] = p.x;
      f[2 * i + 1] = p.y;
    }
  }
  static __device__ __forceinline__ uint4 put(const float (&f)[8]) {
    return make_uint4(two(f[0], f[1], T{}), two(f[2], f[3], T{}), two(f[4], f[5], T{}), two(f[6], f[7], T{}));
  }
};

template <typename T>
struct Row<T, 2> {
  using Raw = uint32_t;
  static __device__ __forceinline__ void get(uint32_t v, float (&f)[2]) {
    const float2 p = two(v, T{});
    f[0] = p.x;
    f[1] = p.y;
  }
  static __device__ __forceinline__ uint32_t put(const float (&f)[2]) { return two(f[0], f[1], T{}); }
};

template <typename T>
struct Row<T, 1> {
  using Raw = uint16_t;
  static __device__ __forceinline__ void get(uint16_t v, float (&f)[1]) { f[0] = two(v, T{}).x; }
  static __device__ __forceinline__ uint16_t put(const float (&f)[1]) {
    return static_cast<uint16_t>(two(f[0], 0.f, T{}));
  }
};

// The token's pairs, one a lane: sorted row (-1 dropped) and weight (0
// where dropped: it may hold anything).
__device__ __forceinline__ void load_pair(const int32_t* __restrict__ dst_of,
                                          const float* __restrict__ weight, int64_t t, int K,
                                          int lane, int64_t rows, bool live, int& row, float& w,
                                          int32_t* dev_err) {
  row = -1;
  w = 0.f;
  if (live && lane < K) {
    row = __ldg(dst_of + t * K + lane);
    if (row >= rows) {
      set_dev_err(dev_err, MOE_DEVERR_BAD_INDEX);
      row = -1;
    }
    if (row >= 0) w = weight ? __ldg(weight + t * K + lane) : 1.f;
  }
}

// Pieces of B sorted rows, U accesses each, all read before the first is used; a dropped or missing pair reads nothing and counts as zeros
// with weight zero.
template <typename Raw, int B, int U>
__device__ __forceinline__ void read_rows(Raw (&v)[B][U], const void* base, int64_t ld_bytes, int row,
                                          int k0, int K, int e, int step, int d, int elem) {
#pragma unroll
  for (int m = 0; m < B; ++m) {
    const int64_t r = __shfl_sync(0xffffffffu, row, (k0 + m) & 31);
    const bool have = k0 + m < K && r >= 0;
    const uint8_t* p = static_cast<const uint8_t*>(base) + r * ld_bytes;
#pragma unroll
    for (int i = 0; i < U; ++i)
      v[m][i] = have && e + i * step < d ? *reinterpret_cast<const Raw*>(p + static_cast<int64_t>(e + i * step) * elem) : Raw{};
  }
}

// dst row = round(w * src) (the row itself, bit for bit, without weights).  A
// CTA's warps have a piece of some token's columns each, whatever the token.
template <typename T, int N, int U, bool WEIGHTED>
__global__ void __launch_bounds__(32 * kSrWarps) scatter_rows_kernel(
    const T* __restrict__ src, int64_t lds, const int32_t* __restrict__ dst_of,
    const float* __restrict__ weight, int T_, int K, int d, int items, T* __restrict__ dst,
    int64_t ldd, int64_t rows, int32_t* dev_err) {
  using R = Row<T, N>;
  using Raw = typename R::Raw;
  const int lane = threadIdx.x & 31;
  const int64_t unit = static_cast<int64_t>(blockIdx.x) * kSrWarps + (threadIdx.x >> 5);
  const int64_t t = unit / items;
  if (t >= T_) return;
  int row;
  float w;
  load_pair(dst_of, weight, t, K, lane, rows, true, row, w, dev_err);
  const int e = static_cast<int>(unit - t * items) * 32 * N * U + lane * N;
  Raw a[U];
#pragma unroll
  for (int i = 0; i < U; ++i)
    a[i] = e + 32 * N * i < d ? *reinterpret_cast<const Raw*>(src + t * lds + e + 32 * N * i) : Raw{};
  for (int k = 0; k < K; ++k) {
    const int64_t r = __shfl_sync(0xffffffffu, row, k);
    const float wk = __shfl_sync(0xffffffffu, w, k);
    if (r < 0) continue;
#pragma unroll
    for (int i = 0; i < U; ++i) {
      Raw o = a[i];
      if (WEIGHTED) {
        float f[N];
        R::get(a[i], f);
#pragma unroll
        for (int j = 0; j < N; ++j) f[j] = __fmul_rn(wk, f[j]);
        o = R::put(f);
      }
      if (e + 32 * N * i < d) *reinterpret_cast<Raw*>(dst + r * ldd + e + 32 * N * i) = o;
    }
  }
}

// The same with the dot products of the token row with each sorted row of y
// (dst may be NULL), reduced over the token's warps in a fixed order: one
// token's warps are one CTA's, blockDim = (32 * warps of a token, tokens).
template <typename T, int N>
__global__ void __launch_bounds__(32 * kSrDotWarps, 2) scatter_dot_kernel(
    const T* __restrict__ src, int64_t lds, const int32_t* __restrict__ dst_of,
    const float* __restrict__ weight, int T_, int K, int d, const T* __restrict__ y, int64_t ldy,
    T* __restrict__ dst, int64_t ldd, int64_t rows, float* __restrict__ dweight,
    int32_t* dev_err) {
  using R = Row<T, N>;
  using Raw = typename R::Raw;
  constexpr int U = kSrDotU<N>, B = kSrDotB;
  extern __shared__ float dot[];  // [tokens][warps][K][8]
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  const int64_t t = static_cast<int64_t>(blockIdx.x) * blockDim.y + threadIdx.y;
  const bool live = t < T_;
  int row;
  float w;
  load_pair(dst_of, weight, t, K, lane, rows, live, row, w, dev_err);
  const uint32_t kept = __ballot_sync(0xffffffffu, row >= 0);
  float* my_dot = dot + (threadIdx.y * warps + warp) * K * 8;
  bool first = true;
  for (int e0 = warp * 32 * N * U; e0 < d && live; e0 += warps * 32 * N * U) {
    const int e = e0 + lane * N;
    Raw a[U];
#pragma unroll
    for (int i = 0; i < U; ++i)
      a[i] = e + 32 * N * i < d ? *reinterpret_cast<const Raw*>(src + t * lds + e + 32 * N * i) : Raw{};
    for (int k0 = 0; k0 < K; k0 += B) {
      Raw b[B][U];
      read_rows<Raw, B, U>(b, y, ldy * sizeof(T), row, k0, K, e, 32 * N, d, sizeof(T));
#pragma unroll
      for (int m = 0; m < B; ++m) {
        const int64_t r = __shfl_sync(0xffffffffu, row, (k0 + m) & 31);
        const float wk = __shfl_sync(0xffffffffu, w, (k0 + m) & 31);
        if (k0 + m >= K || r < 0) continue;
        float p = 0.f;
#pragma unroll
        for (int i = 0; i < U; ++i) {
          float fa[N], fb[N];
          R::get(a[i], fa);
          R::get(b[m][i], fb);
#pragma unroll
          for (int j = 0; j < N; ++j) p = fmaf(fa[j], fb[j], p);
          if (dst && e + 32 * N * i < d) {
#pragma unroll
            for (int j = 0; j < N; ++j) fa[j] = __fmul_rn(wk, fa[j]);
            *reinterpret_cast<Raw*>(dst + r * ldd + e + 32 * N * i) = R::put(fa);
          }
        }
        // the rest of the sum over the lanes is left to the end
        p += __shfl_xor_sync(0xffffffffu, p, 16);
        p += __shfl_xor_sync(0xffffffffu, p, 8);
        if (lane < 8) {
          float* at = my_dot + (k0 + m) * 8 + lane;
          *at = first ? p : *at + p;
        }
      }
    }
    first = false;
  }
  __syncthreads();
  if (live && threadIdx.x < K) {
    float sum = 0.f;
    if ((kept >> threadIdx.x) & 1u) {
      for (int i = 0; i < warps; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) sum += dot[((threadIdx.y * warps + i) * K + threadIdx.x) * 8 + j];
    }
    dweight[t * K + threadIdx.x] = sum;
  }
}

// The K rows added in k order in fp32, rounded once.
template <typename T, int N, int U, bool WEIGHTED>
__global__ void __launch_bounds__(32 * kSrWarps) gather_rows_kernel(
    const T* __restrict__ src, int64_t lds, int64_t rows, const int32_t* __restrict__ dst_of,
    const float* __restrict__ weight, int T_, int K, int d, int items, T* __restrict__ out,
    int64_t ldo, int32_t* dev_err) {
  using R = Row<T, N>;
  using Raw = typename R::Raw;
  constexpr int B = N <= 2 ? 2 : kSrFlight / U;
  const int lane = threadIdx.x & 31;
  const int64_t unit = static_cast<int64_t>(blockIdx.x) * kSrWarps + (threadIdx.x >> 5);
  const int64_t t = unit / items;
  if (t >= T_) return;
  int row;
  float w;
  load_pair(dst_of, weight, t, K, lane, rows, true, row, w, dev_err);
  const int e = static_cast<int>(unit - t * items) * 32 * N * U + lane * N;
  float acc[U][N];
#pragma unroll
  for (int i = 0; i < U; ++i)
#pragma unroll
    for (int j = 0; j < N; ++j) acc[i][j] = 0.f;
  for (int k0 = 0; k0 < K; k0 += B) {
    Raw a[B][U];
    read_rows<Raw, B, U>(a, src, lds * sizeof(T), row, k0, K, e, 32 * N, d, sizeof(T));
#pragma unroll
    for (int m = 0; m < B; ++m) {
      const float wk = __shfl_sync(0xffffffffu, w, (k0 + m) & 31);
#pragma unroll
      for (int i = 0; i < U; ++i) {
        float f[N];
        R::get(a[m][i], f);
#pragma unroll
        for (int j = 0; j < N; ++j)
          acc[i][j] = WEIGHTED ? fmaf(wk, f[j], acc[i][j]) : __fadd_rn(acc[i][j], f[j]);
      }
    }
  }
#pragma unroll
  for (int i = 0; i < U; ++i)
    if (e + 32 * N * i < d) *reinterpret_cast<Raw*>(out + t * ldo + e + 32 * N * i) = R::put(acc[i]);
}

// Warps' pieces of a token's row, and CTAs for T tokens of them.
int sr_items(int d, int step) { return (d + step - 1) / step; }
int64_t sr_blocks(int T, int items) {
  return (static_cast<int64_t>(T) * items + kSrWarps - 1) / kSrWarps;
}

struct Shape {
  dim3 block;
  int64_t grid;
  size_t smem;
};

// Four warps a token where the tokens alone give an SM 64, more where they are
// few, up to 16; several tokens a CTA where a token has fewer pieces.  16384 x
// 6 rows of 7168 bf16: 474 us with 4 warps, 597 with 8; 1600 x 8: 73 us with
// 4, 66 with 5; 256 x 8: 14 us with 4, 9.5 with 14.
Shape dot_shape(int T, int K, int items) {
  const int64_t want = (static_cast<int64_t>(moe_num_sms()) * 64 + T - 1) / T;
  const int most = static_cast<int>(want < 4 ? 4 : (want > kSrDotWarps ? kSrDotWarps : want));
  const int steps = (items + most - 1) / most;
  const int warps = (items + steps - 1) / steps;
  const int tokens = warps >= 4 ? 1 : 4 / warps;
  return {dim3(32 * warps, tokens), (static_cast<int64_t>(T) + tokens - 1) / tokens,
          static_cast<size_t>(tokens) * warps * K * 8 * sizeof(float)};
}

int elem_bytes(moe_dtype dt) { return dt == MOE_F32 ? 4 : 2; }

bool elem_aligned(const void* p, int e) {
  return (reinterpret_cast<uintptr_t>(p) & static_cast<uintptr_t>(e - 1)) == 0;
}

// Low bits that a row of d elements at p with stride ld sets: none below 16
// where 16-byte accesses fit.
uintptr_t row_bits(const void* p, int64_t ld, int d, int e) {
  return reinterpret_cast<uintptr_t>(p) | static_cast<uintptr_t>(ld * e) | static_cast<uintptr_t>(static_cast<int64_t>(d) * e);
}
int access_bytes(uintptr_t bits, int e) { return bits % 16 == 0 ? 16 : (bits % 4 == 0 ? 4 : e); }

moe_status check_shape(moe_dtype dt, int T, int K, int d, int64_t rows) {
  if (dt != MOE_BF16 && dt != MOE_F16 && dt != MOE_F32) return MOE_ERR_INVALID_ARG;
  if (T < 0 || K < 0 || d <= 0 || rows < 0) return MOE_ERR_INVALID_ARG;
  if (K > kSrMaxK || rows > 0x7FFFFFFFll || d > 1 << 30) return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

template <typename T, int N, int U>
struct Access {
  using type = T;
  static constexpr int n = N, u = U, step = 32 * N * U;
};

template <typename T, int N, typename F>
void with_unroll(int K, F&& fn) {
  if (K > 4) fn(Access<T, N, 1>{});
  else if (K > 2) fn(Access<T, N, 2>{});
  else fn(Access<T, N, 4>{});
}

// fn(Access<T, N, U>) for the call's element type and the bytes (16, 4 or one
// element) that every row involved is aligned to and made of.  The gather has U
// columns of few rows or one column of many in flight, of narrow accesses U columns
// of two rows.  With fewer bytes in each access there are fewer in flight and more
// instructions: 4096 x 8 rows in bf16 at widths of 7168, 7002 and 7001 take the sort's
// backward 83, 83 and 146 us, the unsort's 164, 266 and 362.
template <typename F>
void with_access(moe_dtype dt, int bytes, int K, F&& fn) {
  if (dt == MOE_BF16) {
    if (bytes == 16) with_unroll<__nv_bfloat16, 8>(K, fn);
    else if (bytes == 4) fn(Access<__nv_bfloat16, 2, 8>{});
    else fn(Access<__nv_bfloat16, 1, 4>{});
  } else if (dt == MOE_F16) {
    if (bytes == 16) with_unroll<__half, 8>(K, fn);
    else if (bytes == 4) fn(Access<__half, 2, 8>{});
    else fn(Access<__half, 1, 4>{});
  } else {
    if (bytes == 16) with_unroll<float, 4>(K, fn);
    else fn(Access<float, 1, 4>{});
  }
}

// One launch of the scatter without dot products.
template <bool WEIGHTED, typename A>
bool launch_scatter(A, const void* src, int64_t lds, const int32_t* dst_of, const float* weight, int T,
                    int K, int d, void* dst, int64_t ldd, int64_t rows, int32_t* dev_err,
                    cudaStream_t st) {
  using E = typename A::type;
  const int items = sr_items(d, A::step);
  const int64_t blocks = sr_blocks(T, items);
  if (blocks > 0x7FFFFFFFll) return false;
  scatter_rows_kernel<E, A::n, A::u, WEIGHTED><<<static_cast<unsigned>(blocks), 32 * kSrWarps, 0, st>>>(
      static_cast<const E*>(src), lds, dst_of, weight, T, K, d, items, static_cast<E*>(dst), ldd, rows,
      dev_err);
  return true;
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
  const int bytes = access_bytes(row_bits(src, lds, d, e) | row_bits(out, ldo, d, e), e);
  bool fits = true;
  with_access(dt, bytes, K, [&](auto access) {
    using E = typename decltype(access)::type;
    constexpr int N = decltype(access)::n, U = decltype(access)::u;
    auto kern = weighted ? gather_rows_kernel<E, N, U, true> : gather_rows_kernel<E, N, U, false>;
    const int items = sr_items(d, decltype(access)::step);
    const int64_t blocks = sr_blocks(T, items);
    if ((fits = blocks <= 0x7FFFFFFFll))
      kern<<<static_cast<unsigned>(blocks), 32 * kSrWarps, 0, st>>>(
          static_cast<const E*>(src), lds, rows, dst_of, weight, T, K, d, items, static_cast<E*>(out),
          ldo, dev_err);
  });
  if (!fits) return MOE_ERR_UNSUPPORTED;
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
  const int bytes = access_bytes(row_bits(x, ldx, d, e) | row_bits(xs, ldxs, d, e), e);
  bool fits = true;
  with_access(dtype, bytes, K, [&](auto access) {
    fits = launch_scatter<false>(access, x, ldx, dst_of, nullptr, T, K, d, xs, ldxs, rows, dev_err,
                                 static_cast<cudaStream_t>(stream));
  });
  if (!fits) return MOE_ERR_UNSUPPORTED;
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
  const int bytes = access_bytes(row_bits(dout, ldo, d, e) | (dy ? row_bits(dy, lddy, d, e) : 0) |
                                     (dweight ? row_bits(y, ldy, d, e) : 0), e);
  bool fits = true;
  with_access(dtype, bytes, K, [&](auto access) {
    using A = decltype(access);
    using E = typename A::type;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (!dweight) {
      fits = launch_scatter<true>(access, dout, ldo, dst_of, weight, T, K, d, dy, lddy, rows, dev_err, st);
      return;
    }
    const Shape sh = dot_shape(T, K, sr_items(d, 32 * A::n * kSrDotU<A::n>));
    scatter_dot_kernel<E, A::n><<<static_cast<unsigned>(sh.grid), sh.block, sh.smem, st>>>(
        static_cast<const E*>(dout), ldo, dst_of, weight, T, K, d, static_cast<const E*>(y), ldy,
        static_cast<E*>(dy), lddy, rows, dweight, dev_err);
  });
  if (!fits) return MOE_ERR_UNSUPPORTED;
  MOE_CUDA_CHECK_LAUNCH();
  return MOE_OK;
}
