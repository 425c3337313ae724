// Root-mean-square norm with the residual's addition and an 8-bit output.
//
// Per row: h = x + r (rounded to the inputs' type and stored: the residual stream of the next
// layer), u = h gamma, rstd = (mean(h^2) + eps)^(-1/2); y = u rstd, and in 8 bits
// q = rint(127 u / max|u|) with the scale max|u| rstd / 127.  rstd cancels in q, so q is decided
// by u alone.
//
// Statistics, u and the decision of q are in fp64: the square of any fp32 value is in range, and
// 127 u is exact for bf16 inputs (16 bits of product, 7 of the factor), so the correctly rounded
// quotient lies on the side of every border where the exact one lies.
#include "gq_internal.cuh"

namespace gq {

namespace {
constexpr int kNThreads = 256;

template <class T>
__device__ __forceinline__ double to_f64(T v);
template <>
__device__ __forceinline__ double to_f64(__nv_bfloat16 v) {
  return (double)__bfloat162float(v);
}
template <>
__device__ __forceinline__ double to_f64(float v) {
  return (double)v;
}
template <class T>
__device__ __forceinline__ T from_f64(double v);
template <>
__device__ __forceinline__ __nv_bfloat16 from_f64(double v) {
  return __float2bfloat16((float)v);
}
template <>
__device__ __forceinline__ float from_f64(double v) {
  return (float)v;
}
}  // namespace

template <class X, class Gm>
__global__ void __launch_bounds__(kNThreads) rmsnorm_kernel(NormArgs a) {
  __shared__ double red_s[kNThreads / 32], red_m[kNThreads / 32];
  const int64_t row = blockIdx.x;
  const X* x = static_cast<const X*>(a.x) + row * a.n;
  const X* r = a.residual ? static_cast<const X*>(a.residual) + row * a.n : nullptr;
  X* sum = a.sum ? static_cast<X*>(a.sum) + row * a.n : nullptr;
  X* y = a.y ? static_cast<X*>(a.y) + row * a.n : nullptr;
  const Gm* gamma = static_cast<const Gm*>(a.gamma);
  double ss = 0.0, top = 0.0;
  for (int64_t i = threadIdx.x; i < a.n; i += kNThreads) {
    X h = x[i];
    if (r) h = from_f64<X>(to_f64<X>(h) + to_f64<X>(r[i]));
    if (sum) sum[i] = h;
    const double d = to_f64<X>(h), u = fabs(d * to_f64<Gm>(gamma[i]));
    ss += d * d;
    top = (u > top || u != u) ? u : top;  // a NaN stays
  }
  for (int o = 16; o > 0; o >>= 1) {
    ss += __shfl_xor_sync(~0u, ss, o);
    const double v = __shfl_xor_sync(~0u, top, o);
    top = (v > top || v != v) ? v : top;
  }
  if ((threadIdx.x & 31) == 0) {
    red_s[threadIdx.x >> 5] = ss;
    red_m[threadIdx.x >> 5] = top;
  }
  __syncthreads();
  ss = 0.0;
  top = 0.0;
  for (int w = 0; w < kNThreads / 32; ++w) {
    ss += red_s[w];
    const double v = red_m[w];
    top = (v > top || v != v) ? v : top;
  }
  const double rstd = 1.0 / sqrt(ss / (double)a.n + a.eps);
  if (a.q && threadIdx.x == 0) a.qscale[row] = (float)(top * rstd / 127.0);
  const bool codes = top > 0.0 && top <= 1.7e308;  // else the row's codes are 0
  for (int64_t i = threadIdx.x; i < a.n; i += kNThreads) {
    X h;
    if (sum) {
      h = sum[i];
    } else {
      h = x[i];
      if (r) h = from_f64<X>(to_f64<X>(h) + to_f64<X>(r[i]));
    }
    const double u = to_f64<X>(h) * to_f64<Gm>(gamma[i]);
    if (y) y[i] = from_f64<X>(u * rstd);
    if (a.q) a.q[row * a.n + i] = codes ? (int8_t)__double2int_rn(127.0 * u / top) : (int8_t)0;
  }
}

cudaError_t launch_rmsnorm(const NormArgs& a, gq_dtype x_dtype, gq_dtype gamma_dtype,
                           cudaStream_t s) {
  if (a.T == 0) return cudaSuccess;
  const unsigned grid = (unsigned)a.T;
  if (x_dtype == GQ_BF16 && gamma_dtype == GQ_BF16)
    rmsnorm_kernel<__nv_bfloat16, __nv_bfloat16><<<grid, kNThreads, 0, s>>>(a);
  else if (x_dtype == GQ_BF16)
    rmsnorm_kernel<__nv_bfloat16, float><<<grid, kNThreads, 0, s>>>(a);
  else if (gamma_dtype == GQ_BF16)
    rmsnorm_kernel<float, __nv_bfloat16><<<grid, kNThreads, 0, s>>>(a);
  else
    rmsnorm_kernel<float, float><<<grid, kNThreads, 0, s>>>(a);
  count_launches(1);
  return cudaGetLastError();
}

}  // namespace gq
