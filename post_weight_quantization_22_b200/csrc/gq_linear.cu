// Packed products: which kernel a call takes, the tokens' staging for TMA, and the repacking of
// ordered layers.  The kernels are in gq_linear_rows.cuh (few tokens) and gq_linear_tc.cuh.
#include "gq_internal.cuh"
#include "gq_linear.cuh"
#include "gq_unpack.cuh"

#include <type_traits>

namespace gq {

// ---- tokens as bf16 parts: P x T rows of ld elements, columns behind n zero ----
template <LinearInput K>
__global__ void linear_stage_kernel(const void* __restrict__ x, int64_t T, int64_t n, int64_t ld,
                                    const int32_t* __restrict__ perm, uint16_t* __restrict__ out) {
  const int64_t t = blockIdx.x;
  for (int64_t k = threadIdx.x; k < ld; k += blockDim.x) {
    const int64_t src = t * n + (k < n ? (perm ? perm_at(perm, k, n) : k) : 0);
    uint16_t* o = out + t * ld + k;
    if constexpr (K == kXFp32) {
      const float v = k < n ? static_cast<const float*>(x)[src] : 0.f;
      uint32_t h, m, l;
      split3(v, h, m, l);
      o[0] = (uint16_t)(h >> 16);
      o[T * ld] = (uint16_t)(m >> 16);
      o[2 * T * ld] = (uint16_t)(l >> 16);
    } else if constexpr (K == kXInt8) {
      const float v = k < n ? (float)static_cast<const int8_t*>(x)[src] : 0.f;
      o[0] = __bfloat16_as_ushort(__float2bfloat16(v));
    } else {
      o[0] = k < n ? static_cast<const uint16_t*>(x)[src] : (uint16_t)0;
    }
  }
}

namespace {
// What a call does: whether the tokens are staged, the tile and the split of the columns.
struct LinPlan {
  bool tc, staged;
  int P;
  int64_t ld;      // staged row length, elements
};
LinPlan plan_of(int64_t T, int64_t n, LinearInput kind, bool ordered) {
  LinPlan p{};
  p.tc = T > 32;
  p.P = kind == kXFp32 ? 3 : 1;
  // TMA takes rows whose length is a multiple of 16 bytes
  p.staged = kind != kXBf16 || ordered || n % 8 != 0;
  p.ld = (n + 63) / 64 * 64;
  return p;
}

// f(integral_constant<int, bits>)
template <class F>
cudaError_t at_bits(int bits, F f) {
  switch (bits) {
    case 2: return f(std::integral_constant<int, 2>{});
    case 3: return f(std::integral_constant<int, 3>{});
    case 4: return f(std::integral_constant<int, 4>{});
    case 5: return f(std::integral_constant<int, 5>{});
    case 6: return f(std::integral_constant<int, 6>{});
    case 7: return f(std::integral_constant<int, 7>{});
    default: return f(std::integral_constant<int, 8>{});
  }
}
}  // namespace

// ---- codes in processing order ----
// out row = the row's codes at columns perm[0], perm[1], ..; one thread a word of the output.
__global__ void order_codes_kernel(const uint32_t* __restrict__ codes, int64_t n, int bits,
                                   const int32_t* __restrict__ perm, uint32_t* __restrict__ out) {
  const int64_t words = row_words(n, bits);
  const uint32_t* row = codes + blockIdx.x * words;
  const uint32_t mask = (1u << bits) - 1;
  for (int64_t w = threadIdx.x; w < words; w += blockDim.x) {
    const int64_t b0 = w * 32, b1 = min(b0 + 32, n * bits);
    uint32_t v = 0;
    for (int64_t k = b0 / bits; k * bits < b1; ++k) {  // codes with a bit in this word
      const int64_t at = perm_at(perm, k, n) * bits, q = at / 32;
      const int sh = (int)(at % 32);
      uint32_t c = row[q] >> sh;
      if (sh + bits > 32) c |= row[q + 1] << (32 - sh);
      c &= mask;
      const int64_t d = k * bits - b0;
      v |= d >= 0 ? c << d : c >> -d;
    }
    out[blockIdx.x * words + w] = v;
  }
}

cudaError_t launch_order_codes(const uint32_t* codes, int64_t m, int64_t n, int bits,
                               const int32_t* perm, uint32_t* out, cudaStream_t s) {
  const int64_t words = row_words(n, bits);
  order_codes_kernel<<<(unsigned)m, words < 256 ? 64 : 256, 0, s>>>(codes, n, bits, perm, out);
  count_launches(1);
  return cudaGetLastError();
}

size_t linear_ws_bytes(int64_t T, int64_t n, LinearInput kind, bool ordered) {
  const LinPlan p = plan_of(T, n, kind, ordered);
  if (!p.tc) return 0;
  return kAlign + (p.staged ? align_up((size_t)p.P * T * p.ld * 2) : 0);
}

cudaError_t linear_init_attributes() {
  for (int b = 2; b <= 8; ++b) {
    const cudaError_t e = at_bits(b, [](auto w) { return linear_tc_init<decltype(w)::value>(); });
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

cudaError_t launch_linear_rows(const LinearArgs& a, LinearInput kind, cudaStream_t s) {
  if (a.T == 0) return cudaSuccess;
  const uintptr_t p = reinterpret_cast<uintptr_t>(a.x);
  // eight inputs of a token in one or two vector loads: rows have to start aligned
  const int xvec = !a.perm && a.n % 8 == 0 && p % (kind == kXInt8 ? 8 : 16) == 0;
  at_bits(a.bits, [&](auto b) {
    linear_rows_bits<decltype(b)::value>(a, kind, xvec, s);
    return cudaSuccess;
  });
  count_launches(1);
  return cudaGetLastError();
}

cudaError_t launch_linear(const LinearArgs& a, LinearInput kind, void* ws, cudaStream_t s) {
  if (a.T == 0) return cudaSuccess;
  const LinPlan p = plan_of(a.T, a.n, kind, a.perm != nullptr);
  // a misaligned matrix cannot be a tensor map: the warp-level kernel reads it in place
  const bool aligned = p.staged || reinterpret_cast<uintptr_t>(a.x) % 16 == 0;
  const int64_t rows_total = (int64_t)p.P * a.T;
  // (tile coordinates are 32-bit)
  if (!p.tc || !aligned || rows_total > INT32_MAX - 1024) return launch_linear_rows(a, kind, s);
  const void* xt = a.x;
  int64_t ld = a.n, cols = a.n;
  if (p.staged) {
    uint16_t* out = reinterpret_cast<uint16_t*>(static_cast<char*>(ws) + kAlign);
    const unsigned grid = (unsigned)a.T;
    if (kind == kXFp32)
      linear_stage_kernel<kXFp32><<<grid, 256, 0, s>>>(a.x, a.T, a.n, p.ld, a.perm, out);
    else if (kind == kXInt8)
      linear_stage_kernel<kXInt8><<<grid, 256, 0, s>>>(a.x, a.T, a.n, p.ld, a.perm, out);
    else
      linear_stage_kernel<kXBf16><<<grid, 256, 0, s>>>(a.x, a.T, a.n, p.ld, a.perm, out);
    count_launches(1);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    xt = out;
    ld = cols = p.ld;
  }
  LinTcArgs t{};
  t.l = a;
  t.l.perm = nullptr;
  t.planes_t = p.P > 1 ? (int)a.T : 0;
  // widest loads of the packed words: rows start on 16-byte boundaries
  const int64_t words = row_words(a.n, a.bits);
  const int vec = words % 4 == 0 && reinterpret_cast<uintptr_t>(a.codes) % 16 == 0;
  // pairs of CTAs where their 256 x 256 tiles occupy the SMs, and the packed rows can be a
  // tensor map
  const int64_t pairs = ((a.m + 255) / 256) * ((a.T + 255) / 256);
  const bool pair = vec && pairs >= kSMs / 4;
  t.N = pair ? 256 : a.T >= 128 ? 128 : (int)(a.T + 63) / 64 * 64;
  t.mtiles = (int)((a.m + (pair ? 255 : 127)) / (pair ? 256 : 128));
  const int64_t tiles = t.mtiles * ((a.T + t.N - 1) / t.N);
  // (a pair's in whole packed chunks: what lies behind the last column reads as zero)
  t.stages = pair ? (int)((a.n + 127) / 128 * 2) : (int)((a.n + kCols - 1) / kCols);
  t.hdr = static_cast<WsHeader*>(ws);
  t.gshift = a.group ? __builtin_ctz((unsigned)a.group) : 31;
  t.dmask = a.group ? a.group / 16 - 1 : 15;
  t.groups = a.group ? (int)((a.n + a.group - 1) / a.group) : 1;
  if (tiles > INT32_MAX - kSMs) return cudaErrorInvalidValue;
  t.tiles = (int)tiles;
  // columns shared by a cluster while tiles leave SMs idle and every CTA keeps eight stages
  int S = 1;
  while (!pair && S < 8 && tiles * S * 2 <= kSMs && t.stages >= S * 16) S *= 2;
  CUtensorMap map;
  cudaError_t e = encode_tmap_2d(&map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, xt, rows_total, cols,
                                 ld, kCols, (uint32_t)(pair ? 128 : t.N), CU_TENSOR_MAP_SWIZZLE_128B);
  if (e != cudaSuccess) return e;
  const int wide = a.m * (a.y_bf16 ? 2 : 4) % 16 == 0 && reinterpret_cast<uintptr_t>(a.y) % 16 == 0;
  e = at_bits(a.bits, [&](auto b) {
    return linear_tc_bits<decltype(b)::value>(map, t, p.P, pair, vec, wide, S, s);
  });
  count_launches(1);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace gq
