// Packed products: which kernel a call takes, the tokens' staging for TMA, and the repacking of
// ordered layers.  The kernels are in gq_linear_rows.cuh (few tokens) and gq_linear_tc.cuh.
#include "gq_internal.cuh"
#include "gq_linear.cuh"
#include "gq_unpack.cuh"

#include <type_traits>

namespace gq {

// ---- tokens as bf16 parts: P x T rows of ld elements, columns behind n zero ----
// One block a row, eight columns a thread (16-byte stores; 16-byte loads where vec says that rows
// are aligned and taken in order).
template <LinearInput K>
__global__ void linear_stage_kernel(const void* __restrict__ x, int64_t T, int n, int ld,
                                    const int32_t* __restrict__ perm, int vec,
                                    uint16_t* __restrict__ out) {
  constexpr int kSize = K == kXBf16 ? 2 : K == kXFp32 ? 4 : 1;
  constexpr int P = K == kXFp32 ? 3 : 1;
  const int64_t t = blockIdx.x;
  const char* row = static_cast<const char*>(x) + t * n * kSize;
  for (int k = threadIdx.x * 8; k < ld; k += blockDim.x * 8) {
    alignas(16) char in[8 * kSize];
    if (vec && k + 8 <= n) {
      if constexpr (K == kXInt8) {
        *reinterpret_cast<uint2*>(in) = __ldg(reinterpret_cast<const uint2*>(row + k));
      } else {
#pragma unroll
        for (int i = 0; i < kSize / 2; ++i)
          reinterpret_cast<uint4*>(in)[i] =
              __ldg(reinterpret_cast<const uint4*>(row + (int64_t)k * kSize) + i);
      }
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int64_t src = k + i < n ? (perm ? perm_at(perm, k + i, n) : k + i) : -1;
        if constexpr (K == kXInt8)
          in[i] = src < 0 ? 0 : __ldg(reinterpret_cast<const signed char*>(row) + src);
        else if constexpr (K == kXBf16)
          reinterpret_cast<uint16_t*>(in)[i] =
              src < 0 ? (uint16_t)0 : __ldg(reinterpret_cast<const uint16_t*>(row) + src);
        else
          reinterpret_cast<float*>(in)[i] =
              src < 0 ? 0.f : __ldg(reinterpret_cast<const float*>(row) + src);
      }
    }
    uint32_t part[P][4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (K == kXFp32) {
        const float* f = reinterpret_cast<const float*>(in) + 2 * i;
        uint32_t h0, m0, l0, h1, m1, l1;
        split3(f[0], h0, m0, l0);
        split3(f[1], h1, m1, l1);
        part[0][i] = __byte_perm(h0, h1, 0x7632);
        part[1][i] = __byte_perm(m0, m1, 0x7632);
        part[2][i] = __byte_perm(l0, l1, 0x7632);
      } else if constexpr (K == kXInt8) {
        const signed char* c = reinterpret_cast<const signed char*>(in) + 2 * i;
        const __nv_bfloat162 v = __floats2bfloat162_rn((float)c[0], (float)c[1]);  // exact
        part[0][i] = reinterpret_cast<const uint32_t&>(v);
      } else {
        part[0][i] = reinterpret_cast<const uint32_t*>(in)[i];
      }
    }
#pragma unroll
    for (int p = 0; p < P; ++p)
      *reinterpret_cast<uint4*>(out + (p * T + t) * ld + k) =
          make_uint4(part[p][0], part[p][1], part[p][2], part[p][3]);
  }
}

namespace {
// What a call does: whether the tokens are staged, the tile and the split of the columns.
struct LinPlan {
  bool tc, staged;
  int P;
  int64_t ld;      // staged row length, elements
};
LinPlan plan_of(int64_t T, int64_t m, int64_t n, LinearInput kind, bool ordered) {
  LinPlan p{};
  // The warp-level kernel up to 32 tokens, and further while its CTAs (16 rows x 32 tokens) fit
  // the SMs once, where the tcgen05 kernel's fixed steps weigh more (48 tokens, 1024 x 4096, 2
  // bits: 9.0 us against 12.6; 64 tokens, 4096 x 4096: 32 against 18); not for fp32, whose parts
  // cost it three products (23 us against 16).
  // Rows of odd widths, and columns in an order, it reads one value at a time; from nine tokens on
  // staging them for the tcgen05 kernel is faster (4096 x 4095: 16 tokens 29 us against 18, 32
  // tokens 58 against 19).
  const bool whole = n % 8 == 0 && !ordered;
  p.tc = whole ? T > 32 && (kind == kXFp32 || (m + 15) / 16 * ((T + 31) / 32) > kSMs) : T > 8;
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

size_t linear_ws_bytes(int64_t T, int64_t m, int64_t n, LinearInput kind, bool ordered) {
  const LinPlan p = plan_of(T, m, n, kind, ordered);
  if (!p.tc) return 0;
  return kAlign + (p.staged ? align_up((size_t)p.P * T * p.ld * 2) : 0);
}

namespace {
// clusters of 2^i CTAs that a device runs at once (written once per device, before its first call)
int g_clusters[128][4];
// every device's status of all products, and where it lies
__device__ WsHeader g_device_status;
WsHeader* g_device_status_at[128];
}  // namespace

WsHeader* linear_device_status(int dev) { return g_device_status_at[dev & 127]; }

cudaError_t linear_init_attributes() {
  for (int b = 2; b <= 8; ++b) {
    const cudaError_t e = at_bits(b, [](auto w) { return linear_tc_init<decltype(w)::value>(); });
    if (e != cudaSuccess) return e;
  }
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  for (int i = 1; i <= 3 && e == cudaSuccess; ++i)
    e = linear_tc_clusters<4>(1 << i, &g_clusters[dev & 127][i]);
  void* at = nullptr;
  if (e == cudaSuccess) e = cudaGetSymbolAddress(&at, g_device_status);
  if (e == cudaSuccess) g_device_status_at[dev & 127] = static_cast<WsHeader*>(at);
  return e;
}

cudaError_t launch_linear_rows(const LinearArgs& a, LinearInput kind, cudaStream_t s) {
  if (a.T == 0) return cudaSuccess;
  const uintptr_t p = reinterpret_cast<uintptr_t>(a.x);
  // eight inputs of a token in one or two vector loads: rows have to start aligned
  // (one token's row starts where the matrix does, whatever its width)
  const int xvec = !a.perm && (a.n % 8 == 0 || a.T == 1) && p % (kind == kXInt8 ? 8 : 16) == 0;
  at_bits(a.bits, [&](auto b) {
    linear_rows_bits<decltype(b)::value>(a, kind, xvec, s);
    return cudaSuccess;
  });
  count_launches(1);
  return cudaGetLastError();
}

cudaError_t launch_linear(const LinearArgs& a, LinearInput kind, void* ws, cudaStream_t s) {
  if (a.T == 0) return cudaSuccess;
  const LinPlan p = plan_of(a.T, a.m, a.n, kind, a.perm != nullptr);
  // a misaligned matrix cannot be a tensor map: the warp-level kernel reads it in place
  const bool aligned = p.staged || reinterpret_cast<uintptr_t>(a.x) % 16 == 0;
  const int64_t rows_total = (int64_t)p.P * a.T;
  // (tile coordinates are 32-bit)
  if (!p.tc) return launch_linear_rows(a, kind, s);
  if (!aligned || rows_total > INT32_MAX - 1024) {
    // (this call has a workspace, and the warp-level kernel has no status to write)
    const cudaError_t e = cudaMemsetAsync(&static_cast<WsHeader*>(ws)->status, 0, sizeof(int), s);
    return e != cudaSuccess ? e : launch_linear_rows(a, kind, s);
  }
  const void* xt = a.x;
  int64_t ld = a.n, cols = a.n;
  if (p.staged) {
    uint16_t* out = reinterpret_cast<uint16_t*>(static_cast<char*>(ws) + kAlign);
    const unsigned grid = (unsigned)a.T;
    const int row_bytes = (int)a.n * (kind == kXFp32 ? 4 : kind == kXInt8 ? 1 : 2);
    const int align = kind == kXInt8 ? 8 : 16;
    const int xvec = !a.perm && row_bytes % align == 0 &&
                     reinterpret_cast<uintptr_t>(a.x) % align == 0;
    const int nt = p.ld >= 2048 ? 256 : 64;
    if (kind == kXFp32)
      linear_stage_kernel<kXFp32><<<grid, nt, 0, s>>>(a.x, a.T, (int)a.n, (int)p.ld, a.perm, xvec, out);
    else if (kind == kXInt8)
      linear_stage_kernel<kXInt8><<<grid, nt, 0, s>>>(a.x, a.T, (int)a.n, (int)p.ld, a.perm, xvec, out);
    else
      linear_stage_kernel<kXBf16><<<grid, nt, 0, s>>>(a.x, a.T, (int)a.n, (int)p.ld, a.perm, xvec, out);
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
  t.wait = wait_test();
  // (no budget so short that a role gives up before copies that were just issued can have landed)
  t.wait.polls = t.wait.polls < 4096 ? 4096 : t.wait.polls;
  t.gshift = a.group ? __builtin_ctz((unsigned)a.group) : 31;
  t.dmask = a.group ? a.group / 16 - 1 : 15;
  t.groups = a.group ? (int)((a.n + a.group - 1) / a.group) : 1;
  if (tiles > INT32_MAX - kSMs) return cudaErrorInvalidValue;
  t.tiles = (int)tiles;
  // Columns shared by a cluster while the device runs all clusters at once and every CTA keeps
  // eight stages.  (Clusters of eight do not fill every group of SMs: sixteen of them took two
  // waves, 24 us where clusters of four take 17.)
  int dev = 0, S = 1;
  if (cudaGetDevice(&dev) != cudaSuccess) return cudaErrorInvalidDevice;
  t.device_hdr = linear_device_status(dev);
  for (int i = 1; !pair && i <= 3; ++i)
    if (tiles <= g_clusters[dev & 127][i] && t.stages >= 8 << i) S = 1 << i;
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
