// Root-mean-square norm with the residual's addition and an 8-bit output.
//
// Per row: h = x + r (rounded to the inputs' type and stored: the residual stream of the next
// layer), u = h gamma, rstd = (mean(h^2) + eps)^(-1/2); y = u rstd, and in 8 bits
// q = rint(127 u / max|u|) with the scale max|u| rstd / 127.  rstd cancels in q, so q is decided
// by u alone.
//
// The bound is the traffic: a row is read once, kept in registers and written once; what is done
// per value has to stay below about 40 issue cycles of a warp for that (bf16, 7 bytes a value).
// (8192 x 4096 bf16 with a residual: 59 us against 36 of the traffic; a block's next loads wait for
// its row's stores.)
// h^2 is summed in fp64: the square of any value is in range, and one conversion and one addition
// per value run on pipes of their own.  u = h gamma is exact in fp32 for bf16 inputs and weights,
// in fp64 otherwise.  A code is first taken from the fp32 quotient, which is within 3e-5 of the
// exact one, rounded by adding 1.5 * 2^23; within 1e-4 of a border between two codes it is decided
// by the correctly rounded fp64 quotient 127 u / max|u|.  For bf16 inputs 127 u is exact and
// borders are representable, so that quotient is on the side of the border where the exact one
// is.
#include "gq_internal.cuh"

namespace gq {

namespace {
constexpr int kNMaxThreads = 512;
constexpr int kNSMs = 148;

__device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float to_f32(float v) { return v; }
template <class X>
__device__ __forceinline__ X from_f32(float v);
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32(float v) {
  return __float2bfloat16(v);
}
template <>
__device__ __forceinline__ float from_f32(float v) {
  return v;
}

template <class T>
struct alignas(16) Vec8 {
  T v[8];
};

// x + r rounded to X once (bf16: two at a time, the packed addition rounds the exact sum).
__device__ __forceinline__ void add8(Vec8<float>& x, const Vec8<float>& r) {
#pragma unroll
  for (int e = 0; e < 8; ++e) x.v[e] += r.v[e];
}
__device__ __forceinline__ void add8(Vec8<__nv_bfloat16>& x, const Vec8<__nv_bfloat16>& r) {
  __nv_bfloat162* p = reinterpret_cast<__nv_bfloat162*>(x.v);
  const __nv_bfloat162* q = reinterpret_cast<const __nv_bfloat162*>(r.v);
#pragma unroll
  for (int e = 0; e < 4; ++e) p[e] = __hadd2(p[e], q[e]);
}
// Maximum of magnitudes in which a NaN stays.
__device__ __forceinline__ float max_abs(float top, float u) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(top), "f"(fabsf(u)));
  return r;
}

// Eight values of a row: side by side (kVec: 16-byte accesses), or `threads` apart.
template <bool kVec, class T>
__device__ __forceinline__ void load8(const T* row, int64_t i0, int64_t step, int64_t n, Vec8<T>& o) {
  if constexpr (kVec) {
    if (i0 < n) o = *reinterpret_cast<const Vec8<T>*>(row + i0);
    else
#pragma unroll
      for (int e = 0; e < 8; ++e) o.v[e] = from_f32<T>(0.f);
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) o.v[e] = i0 + e * step < n ? row[i0 + e * step] : from_f32<T>(0.f);
  }
}
template <bool kVec, class T>
__device__ __forceinline__ void store8(T* row, int64_t i0, int64_t step, int64_t n, const Vec8<T>& o) {
  if constexpr (kVec) {
    if (i0 < n) *reinterpret_cast<Vec8<T>*>(row + i0) = o;
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (i0 + e * step < n) row[i0 + e * step] = o.v[e];
  }
}

// Sum and maximum over the block (blockDim.x a multiple of 32), the same in every thread.  Two
// scratch halves taken in turn: one barrier a call.
struct NormScratch {
  double s[2][kNMaxThreads / 32];
  unsigned long long t[2][kNMaxThreads / 32];
};
__device__ __forceinline__ unsigned long long warp_max(unsigned long long v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = max(v, __shfl_xor_sync(~0u, v, o));
  return v;
}
__device__ __forceinline__ uint32_t warp_max(uint32_t v) { return __reduce_max_sync(~0u, v); }
template <class U>
__device__ __forceinline__ void block_reduce(double& ss, U& top, NormScratch& m, int& half) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) ss += __shfl_xor_sync(~0u, ss, o);
  top = warp_max(top);
  const int warps = blockDim.x >> 5, lane = threadIdx.x & 31;
  if (warps == 1) return;
  if (lane == 0) {
    m.s[half][threadIdx.x >> 5] = ss;
    m.t[half][threadIdx.x >> 5] = top;
  }
  __syncthreads();
  ss = lane < warps ? m.s[half][lane] : 0.0;
  top = lane < warps ? (U)m.t[half][lane] : 0;
  static_assert(kNMaxThreads / 32 <= 16, "the sums of the warps lie in sixteen lanes");
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) ss += __shfl_xor_sync(~0u, ss, o);
  ss = __shfl_sync(~0u, ss, 0);
  top = warp_max(top);
  half ^= 1;
}
__device__ __forceinline__ unsigned long long abs_bits(double v) {
  return (unsigned long long)__double_as_longlong(v) & 0x7FFFFFFFFFFFFFFFull;
}
}  // namespace

// Eight codes as bytes.
__device__ __forceinline__ uint2 pack8(const uint32_t (&q)[8]) {
  uint2 p;
  p.x = __byte_perm(__byte_perm(q[0], q[1], 0x0040), __byte_perm(q[2], q[3], 0x0040), 0x5410);
  p.y = __byte_perm(__byte_perm(q[4], q[5], 0x0040), __byte_perm(q[6], q[7], 0x0040), 0x5410);
  return p;
}

// Rows blockIdx.x, blockIdx.x + gridDim.x, ..; V vectors of eight values a thread.  fp64
// magnitudes are compared as bit patterns, where infinities and NaN are above every number.
template <class X, class Gm, int V, bool kVec>
__global__ void __launch_bounds__(V == 8 ? 512 : 256, V <= 2 ? 3 : V == 4 ? 2 : 1)
    rmsnorm_kernel(NormArgs a, double inv_n) {
  constexpr bool kExact32 = sizeof(X) == 2 && sizeof(Gm) == 2;  // u is exact in fp32
  constexpr bool kKeep = kExact32 && V <= 2;  // gamma and u stay in registers
  constexpr float kMagic = 12582912.f;        // 1.5 * 2^23
  __shared__ NormScratch scratch;
  int half = 0;
  const int64_t n = a.n;
  const int nt = blockDim.x, tid = threadIdx.x;
  const int64_t step = kVec ? 1 : nt;
  auto first = [&](int k) { return (int64_t)(kVec ? (k * nt + tid) * 8 : k * 8 * nt + tid); };
  const Gm* gamma = static_cast<const Gm*>(a.gamma);
  float gk[kKeep ? V : 1][8], uk[kKeep ? V : 1][8];
  if constexpr (kKeep) {
#pragma unroll
    for (int k = 0; k < V; ++k) {
      Vec8<Gm> g;
      load8<kVec>(gamma, first(k), step, n, g);
#pragma unroll
      for (int e = 0; e < 8; ++e) gk[k][e] = to_f32(g.v[e]);
    }
  }
  for (int64_t row = blockIdx.x; row < a.T; row += gridDim.x) {
    const X* x = static_cast<const X*>(a.x) + row * n;
    Vec8<X> h[V];
#pragma unroll
    for (int k = 0; k < V; ++k) load8<kVec>(x, first(k), step, n, h[k]);
    if (a.residual) {
      const X* r = static_cast<const X*>(a.residual) + row * n;
      if constexpr (V <= 2) {
        Vec8<X> rv[V];
#pragma unroll
        for (int k = 0; k < V; ++k) load8<kVec>(r, first(k), step, n, rv[k]);
#pragma unroll
        for (int k = 0; k < V; ++k) add8(h[k], rv[k]);
      } else {
#pragma unroll
        for (int k = 0; k < V; ++k) {
          Vec8<X> rv;
          load8<kVec>(r, first(k), step, n, rv);
          add8(h[k], rv);
        }
      }
    }
    if (a.sum)
#pragma unroll
      for (int k = 0; k < V; ++k)
        store8<kVec>(static_cast<X*>(a.sum) + row * n, first(k), step, n, h[k]);

    double ss = 0.0;
    unsigned long long top = 0;
    float top32 = 0.f;
#pragma unroll
    for (int k = 0; k < V; ++k) {
      Vec8<Gm> g;
      if constexpr (!kKeep) load8<kVec>(gamma, first(k), step, n, g);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float v = to_f32(h[k].v[e]);
        const double d = (double)v;
        ss += d * d;
        if constexpr (kKeep) {
          uk[k][e] = v * gk[k][e];
          top32 = max_abs(top32, uk[k][e]);
        } else if constexpr (kExact32) {
          top32 = max_abs(top32, v * to_f32(g.v[e]));
        } else {
          top = max(top, abs_bits(d * (double)to_f32(g.v[e])));
        }
      }
    }
    if constexpr (kExact32) {
      uint32_t bits = __float_as_uint(top32);
      block_reduce(ss, bits, scratch, half);
      top = abs_bits((double)__uint_as_float(bits));
    } else {
      block_reduce(ss, top, scratch, half);
    }
    double topd = __longlong_as_double((long long)top);
    if constexpr (kExact32) {
      // fp32 products that left the normal range: the row's maximum again, in fp64
      if (!(topd >= 0x1p-100 && topd < 0x1p127)) {
        double none = 0.0;
        top = 0;
#pragma unroll 1
        for (int k = 0; k < V; ++k) {
          Vec8<Gm> g;
          Vec8<X> hk = h[0];
#pragma unroll
          for (int j = 1; j < V; ++j)
            if (j == k) hk = h[j];
          load8<kVec>(gamma, first(k), step, n, g);
#pragma unroll
          for (int e = 0; e < 8; ++e)
            top = max(top, abs_bits((double)to_f32(hk.v[e]) * (double)to_f32(g.v[e])));
        }
        block_reduce(none, top, scratch, half);
        topd = __longlong_as_double((long long)top);
      }
    }
    // (fp64 divisions and roots are subroutines of a hundred instructions: one per row where only
    // the scale needs it, and none in the quotient below)
    double rstd = 0.0;
    if (a.y || tid == 0) rstd = rsqrt(ss * inv_n + a.eps);
    if (a.q && tid == 0) a.qscale[row] = (float)(topd * (rstd * (1.0 / 127.0)));
    const bool codes = topd > 0.0 && topd < __longlong_as_double(0x7FF0000000000000ll);
    // 127 / max|u| in fp32 where fp32 holds both; elsewhere every code is decided in fp64
    const bool quick = topd >= 0x1p-100 && topd < 0x1p120;
    const float inv = quick ? __fdividef(127.f, (float)topd) : 0.f, rstd32 = (float)rstd;
    // y = u rstd in fp32 where rstd is a normal fp32 number and what u may have lost below fp32's
    // normal range, 2^-150, stays below a quarter of y's smallest step; else in fp64
    const bool quick_y = quick && rstd >= 0x1p-100 && rstd <= 0x1p15;
#pragma unroll
    for (int k = 0; k < V; ++k) {
      Vec8<Gm> g;
      if constexpr (!kKeep) load8<kVec>(gamma, first(k), step, n, g);
      auto gam = [&](int e) {
        if constexpr (kKeep) return gk[k][e];
        else return to_f32(g.v[e]);
      };
      auto u_of = [&](int e) {
        if constexpr (kKeep) return uk[k][e];
        else return to_f32(h[k].v[e]) * gam(e);
      };
      if (a.y) {
        Vec8<X> yv;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          if (kExact32 && quick_y) yv.v[e] = from_f32<X>(u_of(e) * rstd32);
          else yv.v[e] = from_f32<X>((float)((double)to_f32(h[k].v[e]) * (double)gam(e) * rstd));
        }
        store8<kVec>(static_cast<X*>(a.y) + row * n, first(k), step, n, yv);
      }
      if (a.q) {
        uint32_t q[8];
        float off = 0.f;  // largest distance of a quotient from its code
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float c = u_of(e) * inv, t = c + kMagic;
          q[e] = __float_as_uint(t);
          off = fmaxf(off, fabsf(c - (t - kMagic)));
        }
        if (!quick || off > 0.4999f) {
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const float c = u_of(e) * inv, t = c + kMagic;
            if (!quick || fabsf(c - (t - kMagic)) > 0.4999f)
              q[e] = codes ? (uint32_t)__double2int_rn(
                                 127.0 * ((double)to_f32(h[k].v[e]) * (double)gam(e)) / topd)
                           : 0u;
          }
        }
        int8_t* qr = a.q + row * n;
        if constexpr (kVec) {
          if (first(k) < n) *reinterpret_cast<uint2*>(qr + first(k)) = pack8(q);
        } else {
#pragma unroll
          for (int e = 0; e < 8; ++e)
            if (first(k) + e * step < n) qr[first(k) + e * step] = (int8_t)q[e];
        }
      }
    }
  }
}

namespace {
template <class X, class Gm, int V, bool kVec>
void launch_v(const NormArgs& a, int nt, cudaStream_t s) {
  // the blocks that fit the SMs take row after row (gamma is read once a block)
  const int per_sm = V == 8 ? (nt <= 256 ? 2 : 1) : (V == 4 ? 512 : 768) / nt;
  const int64_t most = (int64_t)kNSMs * (per_sm < 16 ? per_sm : 16);
  rmsnorm_kernel<X, Gm, V, kVec><<<(unsigned)(a.T < most ? a.T : most), nt, 0, s>>>(a, 1.0 / (double)a.n);
}
template <class X, class Gm, bool kVec>
void launch_row(const NormArgs& a, cudaStream_t s) {
  // A thread for each vector of eight up to 256 threads, then more vectors a thread; with rows
  // enough two vectors a thread from the start (8192 x 1024 bf16: 13 us against 17).
  const int64_t nv = (a.n + 7) / 8;
  const int per = a.T >= 8 * kNSMs ? 2 : 1;
  int nt = 32;
  while (nt < 256 && nt * per < nv) nt *= 2;
  if (nv > 8 * nt) nt = kNMaxThreads;
  if (nv <= nt) launch_v<X, Gm, 1, kVec>(a, nt, s);
  else if (nv <= 2 * nt) launch_v<X, Gm, 2, kVec>(a, nt, s);
  else if (nv <= 4 * nt) launch_v<X, Gm, 4, kVec>(a, nt, s);
  else launch_v<X, Gm, 8, kVec>(a, nt, s);
}
template <class X, class Gm>
void launch_types(const NormArgs& a, cudaStream_t s) {
  // 16-byte accesses: rows of whole vectors, every matrix aligned (8-bit rows on 8 bytes)
  auto at16 = [](const void* p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; };
  const bool vec = a.n % 8 == 0 && at16(a.x) && at16(a.residual) && at16(a.gamma) && at16(a.sum) &&
                   at16(a.y) && reinterpret_cast<uintptr_t>(a.q) % 8 == 0;
  if (vec) launch_row<X, Gm, true>(a, s);
  else launch_row<X, Gm, false>(a, s);
}
}  // namespace

cudaError_t launch_rmsnorm(const NormArgs& a, gq_dtype x_dtype, gq_dtype gamma_dtype,
                           cudaStream_t s) {
  if (a.T == 0) return cudaSuccess;
  if (x_dtype == GQ_BF16 && gamma_dtype == GQ_BF16) launch_types<__nv_bfloat16, __nv_bfloat16>(a, s);
  else if (x_dtype == GQ_BF16) launch_types<__nv_bfloat16, float>(a, s);
  else if (gamma_dtype == GQ_BF16) launch_types<float, __nv_bfloat16>(a, s);
  else launch_types<float, float>(a, s);
  count_launches(1);
  return cudaGetLastError();
}

}  // namespace gq
