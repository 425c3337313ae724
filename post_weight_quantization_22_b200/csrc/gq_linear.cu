// Products with a packed layer for few tokens: y[t][r] = sum_g s[r][g] sum_{k in g} x[t][k]
// (c[r][k] - z[r][g]), the codes read as gq_quantize_layer wrote them.
//
// The bound for one token is the packed stream (m n b / 8 bytes); what has to be kept down beside
// it is the work per weight of unpacking.  A warp multiplies 16 rows with 8 tokens on
// mma.sync m16n8k16 (the tokens' dimension costs nothing up to 8), operands straight from global
// memory in fragment order: in every unit of 32 columns, lane t of a quad takes columns 8t..8t+7
// of its rows' streams (b bytes) and of its token.  Any assignment of columns to the
// instruction's k slots is right as long as both operands agree.  c - z is an exact integer in 16
// bits, the products are exact, and the fp32 sums of one group are multiplied by the group's
// scale in fp32: no weight is rounded.  The eight warps of a CTA share the columns in chunks of
// 128 and add their sums in a fixed order.
//
// fp32 tokens are taken as three bf16 parts (8 + 8 + 8 bits, exact), three products a weight;
// 8-bit tokens as fp16 integers.
#include "gq_internal.cuh"
#include "gq_unpack.cuh"

namespace gq {

namespace {
constexpr int kRThreads = 256;
constexpr int kRWarps = kRThreads / 32;
constexpr int kRRows = 16;

template <bool kHalf>
__device__ __forceinline__ void mma_16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                          uint32_t a3, uint32_t b0, uint32_t b1) {
  if constexpr (kHalf)
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  else
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// The lane's eight codes of one unit: bits [8 t B, 8 (t + 1) B) of the unit's B words.
template <int B>
__device__ __forceinline__ void load_codes(const uint32_t* __restrict__ row, int64_t unit, int t,
                                           int64_t words, uint32_t& lo, uint32_t& hi) {
  const int64_t w = unit * B + (t * B) / 4;
  const uint32_t shift = 8 * ((t * B) % 4);
  const uint32_t w0 = w < words ? __ldg(row + w) : 0u;
  if constexpr (B == 4) {
    lo = w0;
    hi = 0;
  } else if constexpr (B == 2) {
    lo = w0 >> shift;
    hi = 0;
  } else {
    const uint32_t w1 = w + 1 < words ? __ldg(row + w + 1) : 0u;
    lo = __funnelshift_r(w0, w1, shift);
    hi = w1 >> shift;
    if constexpr (B == 7) {
      const uint32_t w2 = w + 2 < words ? __ldg(row + w + 2) : 0u;
      hi = __funnelshift_r(w1, w2, shift);
    }
  }
}

// The lane's eight inputs x[k .. k+7] of one token as pairs (i, i + 4), P parts each.
template <LinearInput K, int P>
__device__ __forceinline__ void load_x(const void* xrow, int64_t k, int64_t n,
                                       const int32_t* __restrict__ perm, bool vec,
                                       uint32_t (&b)[P][4]) {
  if constexpr (K == kXBf16) {
    const uint16_t* x = static_cast<const uint16_t*>(xrow);
    uint32_t r[4] = {0, 0, 0, 0};  // (x0, x1), (x2, x3), ...
    if (vec) {
      if (k < n) {
        const uint4 v = __ldg(reinterpret_cast<const uint4*>(x + k));
        r[0] = v.x; r[1] = v.y; r[2] = v.z; r[3] = v.w;
      }
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (k + i < n)
          r[i >> 1] |= (uint32_t)__ldg(x + (perm ? perm_at(perm, k + i, n) : k + i)) << (16 * (i & 1));
    }
    b[0][0] = __byte_perm(r[0], r[2], 0x5410);
    b[0][1] = __byte_perm(r[0], r[2], 0x7632);
    b[0][2] = __byte_perm(r[1], r[3], 0x5410);
    b[0][3] = __byte_perm(r[1], r[3], 0x7632);
  } else if constexpr (K == kXFp32) {
    const float* x = static_cast<const float*>(xrow);
    float f[8] = {0, 0, 0, 0, 0, 0, 0, 0};
    if (vec) {
      if (k < n) {
        const float4 u = __ldg(reinterpret_cast<const float4*>(x + k));
        const float4 v = __ldg(reinterpret_cast<const float4*>(x + k + 4));
        f[0] = u.x; f[1] = u.y; f[2] = u.z; f[3] = u.w;
        f[4] = v.x; f[5] = v.y; f[6] = v.z; f[7] = v.w;
      }
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (k + i < n) f[i] = __ldg(x + (perm ? perm_at(perm, k + i, n) : k + i));
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      uint32_t h0, m0, l0, h1, m1, l1;
      split3(f[i], h0, m0, l0);
      split3(f[i + 4], h1, m1, l1);
      b[0][i] = __byte_perm(h0, h1, 0x7632);
      b[1][i] = __byte_perm(m0, m1, 0x7632);
      b[2][i] = __byte_perm(l0, l1, 0x7632);
    }
  } else {
    const uint8_t* x = static_cast<const uint8_t*>(xrow);
    uint32_t lo = 0, hi = 0;
    if (vec) {
      if (k < n) {
        const uint2 v = __ldg(reinterpret_cast<const uint2*>(x + k));
        lo = v.x;
        hi = v.y;
      }
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (k + i < n) {
          const uint32_t v = __ldg(x + (perm ? perm_at(perm, k + i, n) : k + i));
          (i < 4 ? lo : hi) |= v << (8 * (i & 3));
        }
    }
    // int8 -> fp16: 1024 + (v + 128), minus 1152
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t p = __byte_perm(lo, hi, 0x0400 + 0x0101 * i);
      b[0][i] = f16x2_sub((p & 0x00FF00FFu) ^ 0x64806480u, 0x64806480u);
    }
  }
}

template <LinearInput K>
__device__ __forceinline__ const void* token_row(const void* x, int64_t t, int64_t n) {
  constexpr int size = K == kXBf16 ? 2 : K == kXFp32 ? 4 : 1;
  return static_cast<const char*>(x) + t * n * size;
}
}  // namespace

// One CTA: 16 rows x (8 NT) tokens.
template <int B, LinearInput K, int NT>
__global__ void __launch_bounds__(kRThreads) linear_rows_kernel(LinearArgs a, int vec) {
  constexpr bool kHalf = K == kXInt8;
  constexpr int P = K == kXFp32 ? 3 : 1;
  __shared__ float red[kRWarps][NT * 8][kRRows + 1];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int64_t row0 = (int64_t)blockIdx.x * kRRows;
  const int64_t rA = min(row0 + g, a.m - 1), rB = min(row0 + g + 8, a.m - 1);
  const int64_t words = row_words(a.n, B);
  const uint32_t* cA = a.codes + rA * words;
  const uint32_t* cB = a.codes + rB * words;
  const int gs = a.group ? a.group : (int)(a.n + 31) / 32 * 32;  // one grid per row: one group
  const int64_t G = (a.n + gs - 1) / gs;
  const float* sA = a.scales + rA * G;
  const float* sB = a.scales + rB * G;
  const uint8_t* zA = a.zeros + rA * G;
  const uint8_t* zB = a.zeros + rB * G;
  const int64_t units = (a.n + 31) / 32;
  const bool g16 = gs == 16;

  for (int64_t t0 = (int64_t)blockIdx.y * NT * 8; t0 < a.T; t0 += (int64_t)gridDim.y * NT * 8) {
    float acc[NT][4];
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[j][i] = 0.f;

    for (int64_t u0 = warp * 4; u0 < units; u0 += kRWarps * 4) {
      uint32_t wa[4][2], wb[4][2];
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        load_codes<B>(cA, u0 + u, t, words, wa[u][0], wa[u][1]);
        load_codes<B>(cB, u0 + u, t, words, wb[u][0], wb[u][1]);
      }
      float part[NT][4];
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int64_t unit = u0 + u, k = unit * 32 + 8 * t;
        // the group of the lane's columns (clamped in the padding behind the last column)
        const int gi = (int)min((unit * 32 + 8 * t) / gs, G - 1);
        uint32_t pa[4], pb[4];
        code_pairs<B>(wa[u][0], wa[u][1], pa);
        code_pairs<B>(wb[u][0], wb[u][1], pb);
        const uint32_t za = zero_pair<B, kHalf>(zA[gi]), zb = zero_pair<B, kHalf>(zB[gi]);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          pa[i] = pair_value<B, kHalf>(pa[i], za);
          pb[i] = pair_value<B, kHalf>(pb[i], zb);
        }
        const bool first = u == 0 || (unit * 32) % gs == 0;
        const bool last = u == 3 || ((unit + 1) * 32) % gs == 0;
        const int g0 = (int)min(unit * 32 / gs, G - 1);
        const float fa = sA[g0], fb = sB[g0];
#pragma unroll
        for (int j = 0; j < NT; ++j) {
          uint32_t b[P][4];
          const int64_t tok = t0 + j * 8 + g;
          if (tok < a.T) {
            load_x<K, P>(token_row<K>(a.x, tok, a.n), k, a.n, a.perm, vec, b);
          } else {
#pragma unroll
            for (int p = 0; p < P; ++p)
#pragma unroll
              for (int i = 0; i < 4; ++i) b[p][i] = 0;
          }
          if (first || g16) {
#pragma unroll
            for (int i = 0; i < 4; ++i) part[j][i] = 0.f;
          }
          if (!g16) {
#pragma unroll
            for (int p = 0; p < P; ++p) {
              mma_16816<kHalf>(part[j], pa[0], pb[0], pa[1], pb[1], b[p][0], b[p][1]);
              mma_16816<kHalf>(part[j], pa[2], pb[2], pa[3], pb[3], b[p][2], b[p][3]);
            }
            if (last) {
              acc[j][0] += fa * part[j][0];
              acc[j][1] += fa * part[j][1];
              acc[j][2] += fb * part[j][2];
              acc[j][3] += fb * part[j][3];
            }
          } else {
            // groups of 16: lanes 0, 1 of a quad hold the unit's first group, lanes 2, 3 its
            // second; each half is multiplied with the other half's inputs at zero
            const int g1 = (int)min(unit * 2 + 1, G - 1);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const bool mine = (t >> 1) == h;
              float c[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
              for (int p = 0; p < P; ++p) {
                mma_16816<kHalf>(c, pa[0], pb[0], pa[1], pb[1], mine ? b[p][0] : 0u,
                                 mine ? b[p][1] : 0u);
                mma_16816<kHalf>(c, pa[2], pb[2], pa[3], pb[3], mine ? b[p][2] : 0u,
                                 mine ? b[p][3] : 0u);
              }
              const float ha = h ? sA[g1] : fa, hb = h ? sB[g1] : fb;
              acc[j][0] += ha * c[0];
              acc[j][1] += ha * c[1];
              acc[j][2] += hb * c[2];
              acc[j][3] += hb * c[3];
            }
          }
        }
      }
    }
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      red[warp][j * 8 + 2 * t][g] = acc[j][0];
      red[warp][j * 8 + 2 * t + 1][g] = acc[j][1];
      red[warp][j * 8 + 2 * t][g + 8] = acc[j][2];
      red[warp][j * 8 + 2 * t + 1][g + 8] = acc[j][3];
    }
    __syncthreads();
    for (int i = threadIdx.x; i < NT * 8 * kRRows; i += kRThreads) {
      const int tt = i / kRRows, rr = i % kRRows;
      const int64_t tok = t0 + tt, row = row0 + rr;
      if (tok < a.T && row < a.m) {
        float v = 0.f;
#pragma unroll
        for (int w = 0; w < kRWarps; ++w) v += red[w][tt][rr];
        if constexpr (K == kXInt8) v *= a.xscale[tok];
        if (a.y_bf16)
          static_cast<__nv_bfloat16*>(a.y)[tok * a.m + row] = __float2bfloat16(v);
        else
          static_cast<float*>(a.y)[tok * a.m + row] = v;
      }
    }
    __syncthreads();
  }
}

namespace {
template <int B, LinearInput K>
void launch_rows(const LinearArgs& a, int vec, cudaStream_t s) {
  const unsigned gx = (unsigned)((a.m + kRRows - 1) / kRRows);
  auto gy = [&](int nt) {
    const int64_t tiles = (a.T + nt * 8 - 1) / (nt * 8);
    return (unsigned)(tiles < 32768 ? tiles : 32768);
  };
  if (a.T <= 8)
    linear_rows_kernel<B, K, 1><<<dim3(gx, gy(1)), kRThreads, 0, s>>>(a, vec);
  else if (a.T <= 16)
    linear_rows_kernel<B, K, 2><<<dim3(gx, gy(2)), kRThreads, 0, s>>>(a, vec);
  else
    linear_rows_kernel<B, K, 4><<<dim3(gx, gy(4)), kRThreads, 0, s>>>(a, vec);
}
template <LinearInput K>
void launch_bits(const LinearArgs& a, int vec, cudaStream_t s) {
  switch (a.bits) {
    case 2: return launch_rows<2, K>(a, vec, s);
    case 3: return launch_rows<3, K>(a, vec, s);
    case 4: return launch_rows<4, K>(a, vec, s);
    case 5: return launch_rows<5, K>(a, vec, s);
    case 6: return launch_rows<6, K>(a, vec, s);
    case 7: return launch_rows<7, K>(a, vec, s);
    default: return launch_rows<8, K>(a, vec, s);
  }
}
}  // namespace

cudaError_t launch_linear_rows(const LinearArgs& a, LinearInput kind, cudaStream_t s) {
  if (a.T == 0) return cudaSuccess;
  const uintptr_t p = reinterpret_cast<uintptr_t>(a.x);
  // eight inputs of a token in one or two vector loads: rows have to start aligned
  const int vec = !a.perm && a.n % 8 == 0 && p % (kind == kXInt8 ? 8 : 16) == 0;
  if (kind == kXBf16) launch_bits<kXBf16>(a, vec, s);
  else if (kind == kXFp32) launch_bits<kXFp32>(a, vec, s);
  else launch_bits<kXInt8>(a, vec, s);
  count_launches(1);
  return cudaGetLastError();
}

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

}  // namespace gq
