// Products with a packed layer for few tokens: y[t][r] = sum_g s[r][g] sum_{k in g} x[t][k]
// (c[r][k] - z[r][g]), the codes read as gq_quantize_layer wrote them.
//
// The bound for one token is the packed stream (m n b / 8 bytes); what has to be kept down beside
// it is the work per weight of unpacking, and enough loads have to be in flight.  A warp
// multiplies 16 rows with 8 tokens on mma.sync m16n8k16 (the tokens' dimension costs nothing up
// to 8), operands straight from global memory in fragment order.  Any assignment of columns to
// the instruction's k slots is right as long as both operands agree, so in a chunk of 128 columns
// lane t of a quad takes columns 32 t .. 32 t + 31 of its two rows: b whole words of the stream, in
// 16-byte loads where rows are aligned.  With groups of 64 two lanes of a quad hold one group and
// two the other; the chunk is then multiplied twice, with the other half's inputs at zero.
// Groups of 32 and 16 take units of 32 columns instead, 8 columns a lane.
// c - z is an exact integer in 16 bits, the products are exact, and the fp32 sums of one group
// are multiplied by the group's scale in fp32: no weight is rounded.  The warps of a CTA share
// the columns in chunks of 128 and add their sums in a fixed order; every warp loads a chunk
// ahead.
//
// fp32 tokens are taken as three bf16 parts (8 + 8 + 8 bits, exact), three products a weight;
// 8-bit tokens as fp16 integers.
#include "gq_internal.cuh"
#include "gq_unpack.cuh"

namespace gq {

namespace {
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
__device__ __forceinline__ void load_codes(const uint32_t* __restrict__ row, int unit, int t,
                                           int words, uint32_t& lo, uint32_t& hi) {
  const int w = unit * B + (t * B) / 4;
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

// Eight inputs x[k .. k+7] of one token as they lie in memory.
template <LinearInput K>
struct Raw {
  uint32_t r[K == kXBf16 ? 4 : K == kXFp32 ? 8 : 2];
};
// fast: whole vectors, all eight columns inside the row.
template <LinearInput K>
__device__ __forceinline__ void load_raw(const void* xrow, int k, int n,
                                         const int32_t* __restrict__ perm, bool fast, Raw<K>& o) {
  constexpr int R = sizeof(o.r) / 4;
  if (fast) {
    const uint32_t* p = reinterpret_cast<const uint32_t*>(
        static_cast<const char*>(xrow) + (int64_t)k * (R / 2));
    if constexpr (R == 2) {
      const uint2 v = __ldg(reinterpret_cast<const uint2*>(p));
      o.r[0] = v.x; o.r[1] = v.y;
    } else {
#pragma unroll
      for (int i = 0; i < R / 4; ++i) {
        const uint4 v = __ldg(reinterpret_cast<const uint4*>(p) + i);
        o.r[4 * i] = v.x; o.r[4 * i + 1] = v.y; o.r[4 * i + 2] = v.z; o.r[4 * i + 3] = v.w;
      }
    }
    return;
  }
#pragma unroll
  for (int i = 0; i < R; ++i) o.r[i] = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    if (k + i >= n) continue;
    const int64_t at = perm ? perm_at(perm, k + i, n) : k + i;
    if constexpr (K == kXBf16)
      o.r[i >> 1] |= (uint32_t)__ldg(static_cast<const uint16_t*>(xrow) + at) << (16 * (i & 1));
    else if constexpr (K == kXFp32)
      o.r[i] = __ldg(static_cast<const uint32_t*>(xrow) + at);
    else
      o.r[i >> 2] |= (uint32_t)__ldg(static_cast<const uint8_t*>(xrow) + at) << (8 * (i & 3));
  }
}
// The same as pairs (i, i + 4) of 16-bit floats, P parts each.
template <LinearInput K, int P>
__device__ __forceinline__ void input_pairs(const Raw<K>& x, uint32_t (&b)[P][4]) {
  if constexpr (K == kXBf16) {
    b[0][0] = __byte_perm(x.r[0], x.r[2], 0x5410);
    b[0][1] = __byte_perm(x.r[0], x.r[2], 0x7632);
    b[0][2] = __byte_perm(x.r[1], x.r[3], 0x5410);
    b[0][3] = __byte_perm(x.r[1], x.r[3], 0x7632);
  } else if constexpr (K == kXFp32) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      uint32_t h0, m0, l0, h1, m1, l1;
      split3(__uint_as_float(x.r[i]), h0, m0, l0);
      split3(__uint_as_float(x.r[i + 4]), h1, m1, l1);
      b[0][i] = __byte_perm(h0, h1, 0x7632);
      b[1][i] = __byte_perm(m0, m1, 0x7632);
      b[2][i] = __byte_perm(l0, l1, 0x7632);
    }
  } else {
    // int8 -> fp16: 1024 + (v + 128), minus 1152
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t p = __byte_perm(x.r[0], x.r[1], 0x0400 + 0x0101 * i);
      b[0][i] = f16x2_sub((p & 0x00FF00FFu) ^ 0x64806480u, 0x64806480u);
    }
  }
}

template <LinearInput K>
__device__ __forceinline__ const void* token_row(const void* x, int64_t t, int64_t n) {
  constexpr int size = K == kXBf16 ? 2 : K == kXFp32 ? 4 : 1;
  return static_cast<const char*>(x) + t * n * size;
}

// B consecutive words of a row from word w0 on (0 behind the row's end).
template <int B>
__device__ __forceinline__ void load_run(const uint32_t* __restrict__ row, int w0, int words,
                                         bool vec, uint32_t (&w)[B]) {
  if (vec && w0 + B <= words) {
    if constexpr (B % 4 == 0) {
#pragma unroll
      for (int i = 0; i < B / 4; ++i) {
        const uint4 v = __ldg(reinterpret_cast<const uint4*>(row + w0) + i);
        w[4 * i] = v.x; w[4 * i + 1] = v.y; w[4 * i + 2] = v.z; w[4 * i + 3] = v.w;
      }
      return;
    } else if constexpr (B % 2 == 0) {
#pragma unroll
      for (int i = 0; i < B / 2; ++i) {
        const uint2 v = __ldg(reinterpret_cast<const uint2*>(row + w0) + i);
        w[2 * i] = v.x; w[2 * i + 1] = v.y;
      }
      return;
    }
  }
#pragma unroll
  for (int i = 0; i < B; ++i) w[i] = w0 + i < words ? __ldg(row + w0 + i) : 0u;
}

// One warp's share of a chunk of 128 columns for its two rows A and B, and of one token's inputs.
template <int B, LinearInput K>
struct Chunk {
  uint32_t wa[B], wb[B];  // lane t's 32 columns
  uint32_t za, zb;        // their zero points
  float fa[2], fb[2];     // scales of the chunk's group, or of its halves'
  Raw<K> x[4];
};
}  // namespace

// One CTA: 16 rows x (8 NT) tokens.  kFine: groups of 16 or 32 columns.  gshift: log2 of the group
// width (31: one grid per row).  xvec, cvec: inputs and packed rows allow wide loads.
template <int B, LinearInput K, int NT, bool kFine, int kWarps>
__global__ void __launch_bounds__(kWarps * 32)
    linear_rows_kernel(LinearArgs a, int gshift, int G, int xvec, int cvec) {
  constexpr bool kHalf = K == kXInt8;
  constexpr int P = K == kXFp32 ? 3 : 1;
  __shared__ float red[kWarps][NT * 8][kRRows + 1];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int64_t row0 = (int64_t)blockIdx.x * kRRows;
  const int64_t rA = min(row0 + g, a.m - 1), rB = min(row0 + g + 8, a.m - 1);
  const int n = (int)a.n, words = (int)row_words(a.n, B), chunks = (n + 127) / 128;
  const uint32_t* cA = a.codes + rA * words;
  const uint32_t* cB = a.codes + rB * words;
  const float* sA = a.scales + rA * G;
  const float* sB = a.scales + rB * G;
  const uint8_t* zA = a.zeros + rA * G;
  const uint8_t* zB = a.zeros + rB * G;

  for (int64_t t0 = (int64_t)blockIdx.y * NT * 8; t0 < a.T; t0 += (int64_t)gridDim.y * NT * 8) {
    float acc[NT][4];
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[j][i] = 0.f;
    // (behind the last token its row again: a column of the product is one token's alone, and
    // these columns are not stored)
    const void* xrow[NT];
#pragma unroll
    for (int j = 0; j < NT; ++j) xrow[j] = token_row<K>(a.x, min(t0 + j * 8 + g, a.T - 1), a.n);
    if constexpr (!kFine) {
      const bool halves = gshift == 6;
      auto fetch = [&](int c, Chunk<B, K>& q) {
        if constexpr (NT == 1) {
          const bool fast = xvec && c * 128 + 128 <= n;
#pragma unroll
          for (int i = 0; i < 4; ++i)
            load_raw<K>(xrow[0], c * 128 + 32 * t + 8 * i, n, a.perm, fast, q.x[i]);
        }
        load_run<B>(cA, (c * 4 + t) * B, words, cvec, q.wa);
        load_run<B>(cB, (c * 4 + t) * B, words, cvec, q.wb);
        const int gl = min((c * 128 + 32 * t) >> gshift, G - 1);
        q.za = __ldg(zA + gl);
        q.zb = __ldg(zB + gl);
        const int g0 = min((c * 128) >> gshift, G - 1);
        q.fa[0] = __ldg(sA + g0);
        q.fb[0] = __ldg(sB + g0);
        if (halves) {
          const int g1 = min(g0 + 1, G - 1);
          q.fa[1] = __ldg(sA + g1);
          q.fb[1] = __ldg(sB + g1);
        }
      };
      auto multiply = [&](int c, const Chunk<B, K>& q) {
        const uint32_t za = zero_pair<B, kHalf>(q.za), zb = zero_pair<B, kHalf>(q.zb);
        const bool fast = xvec && c * 128 + 128 <= n;
        float part[NT][4], part2[NT][4];
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
          for (int i = 0; i < 4; ++i) part[j][i] = part2[j][i] = 0.f;
#pragma unroll
        for (int i = 0; i < 4; ++i) {  // eight columns of the lane
          constexpr int kTop = B - 1;
          const int w = (i * B) / 4, sh = 8 * ((i * B) % 4);
          const int w1 = w + 1 < B ? w + 1 : kTop, w2 = w + 2 < B ? w + 2 : kTop;
          uint32_t pa[4], pb[4];
          code_pairs<B>(__funnelshift_r(q.wa[w], q.wa[w1], sh),
                        __funnelshift_r(q.wa[w1], q.wa[w2], sh), pa);
          code_pairs<B>(__funnelshift_r(q.wb[w], q.wb[w1], sh),
                        __funnelshift_r(q.wb[w1], q.wb[w2], sh), pb);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            pa[e] = pair_value<B, kHalf>(pa[e], za);
            pb[e] = pair_value<B, kHalf>(pb[e], zb);
          }
#pragma unroll
          for (int j = 0; j < NT; ++j) {
            uint32_t b[P][4];
            if constexpr (NT == 1) {
              input_pairs<K, P>(q.x[i], b);
            } else {
              Raw<K> x;
              load_raw<K>(xrow[j], c * 128 + 32 * t + 8 * i, n, a.perm, fast, x);
              input_pairs<K, P>(x, b);
            }
            if (!halves) {
#pragma unroll
              for (int p = 0; p < P; ++p) {
                mma_16816<kHalf>(part[j], pa[0], pb[0], pa[1], pb[1], b[p][0], b[p][1]);
                mma_16816<kHalf>(part[j], pa[2], pb[2], pa[3], pb[3], b[p][2], b[p][3]);
              }
            } else {
              const bool low = t < 2;
#pragma unroll
              for (int p = 0; p < P; ++p) {
#pragma unroll
                for (int e = 0; e < 4; e += 2) {
                  mma_16816<kHalf>(part[j], pa[e], pb[e], pa[e + 1], pb[e + 1],
                                   low ? b[p][e] : 0u, low ? b[p][e + 1] : 0u);
                  mma_16816<kHalf>(part2[j], pa[e], pb[e], pa[e + 1], pb[e + 1],
                                   low ? 0u : b[p][e], low ? 0u : b[p][e + 1]);
                }
              }
            }
          }
        }
#pragma unroll
        for (int j = 0; j < NT; ++j) {
          acc[j][0] += q.fa[0] * part[j][0];
          acc[j][1] += q.fa[0] * part[j][1];
          acc[j][2] += q.fb[0] * part[j][2];
          acc[j][3] += q.fb[0] * part[j][3];
          if (halves) {
            acc[j][0] += q.fa[1] * part2[j][0];
            acc[j][1] += q.fa[1] * part2[j][1];
            acc[j][2] += q.fb[1] * part2[j][2];
            acc[j][3] += q.fb[1] * part2[j][3];
          }
        }
      };
      Chunk<B, K> q0, q1;
      int c = warp;
      if (c < chunks) fetch(c, q0);
      while (c < chunks) {
        if (c + kWarps < chunks) fetch(c + kWarps, q1);
        multiply(c, q0);
        c += kWarps;
        if (c >= chunks) break;
        if (c + kWarps < chunks) fetch(c + kWarps, q0);
        multiply(c, q1);
        c += kWarps;
      }
    } else {
      const bool g16 = gshift == 4;
      for (int u0 = warp * 4; u0 < chunks * 4; u0 += kWarps * 4) {
        uint32_t wa[4][2], wb[4][2];
        uint32_t za[4], zb[4];
        float fa[4], fb[4];
        Raw<K> x1[4];
        const bool fast = xvec && u0 * 32 + 128 <= n;
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const int unit = u0 + u;
          if constexpr (NT == 1) load_raw<K>(xrow[0], unit * 32 + 8 * t, n, a.perm, fast, x1[u]);
          load_codes<B>(cA, unit, t, words, wa[u][0], wa[u][1]);
          load_codes<B>(cB, unit, t, words, wb[u][0], wb[u][1]);
          const int gl = min((unit * 32 + 8 * t) >> gshift, G - 1);
          const int g0 = min((unit * 32) >> gshift, G - 1);
          za[u] = __ldg(zA + gl);
          zb[u] = __ldg(zB + gl);
          fa[u] = __ldg(sA + g0);
          fb[u] = __ldg(sB + g0);
        }
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const int unit = u0 + u;
          uint32_t pa[4], pb[4];
          code_pairs<B>(wa[u][0], wa[u][1], pa);
          code_pairs<B>(wb[u][0], wb[u][1], pb);
          const uint32_t zpa = zero_pair<B, kHalf>(za[u]), zpb = zero_pair<B, kHalf>(zb[u]);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            pa[i] = pair_value<B, kHalf>(pa[i], zpa);
            pb[i] = pair_value<B, kHalf>(pb[i], zpb);
          }
          float ga = 0.f, gb = 0.f;
          if (g16) {
            const int g1 = min(unit * 2 + 1, G - 1);
            ga = __ldg(sA + g1);
            gb = __ldg(sB + g1);
          }
#pragma unroll
          for (int j = 0; j < NT; ++j) {
            uint32_t b[P][4];
            if constexpr (NT == 1) {
              input_pairs<K, P>(x1[u], b);
            } else {
              Raw<K> x;
              load_raw<K>(xrow[j], unit * 32 + 8 * t, n, a.perm, fast, x);
              input_pairs<K, P>(x, b);
            }
            // groups of 16: lanes 0, 1 of a quad hold the unit's first group, lanes 2, 3 its
            // second; each half is multiplied with the other half's inputs at zero
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              if (h == 1 && !g16) break;
              const bool mine = !g16 || (t >> 1) == h;
              float c[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
              for (int p = 0; p < P; ++p) {
                mma_16816<kHalf>(c, pa[0], pb[0], pa[1], pb[1], mine ? b[p][0] : 0u,
                                 mine ? b[p][1] : 0u);
                mma_16816<kHalf>(c, pa[2], pb[2], pa[3], pb[3], mine ? b[p][2] : 0u,
                                 mine ? b[p][3] : 0u);
              }
              const float ha = h ? ga : fa[u], hb = h ? gb : fb[u];
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
    for (int i = threadIdx.x; i < NT * 8 * kRRows; i += kWarps * 32) {
      const int tt = i / kRRows, rr = i % kRRows;
      const int64_t tok = t0 + tt, row = row0 + rr;
      if (tok < a.T && row < a.m) {
        float v = 0.f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) v += red[w][tt][rr];
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
template <int B, LinearInput K, bool kFine>
void launch_rows(const LinearArgs& a, int xvec, cudaStream_t s) {
  const unsigned gx = (unsigned)((a.m + kRRows - 1) / kRRows);
  auto gy = [&](int nt) {
    const int64_t tiles = (a.T + nt * 8 - 1) / (nt * 8);
    return (unsigned)(tiles < 32768 ? tiles : 32768);
  };
  const int gshift = a.group ? __builtin_ctz((unsigned)a.group) : 31;
  const int G = a.group ? (int)((a.n + a.group - 1) / a.group) : 1;
  const int cvec = row_words(a.n, B) % 4 == 0 && reinterpret_cast<uintptr_t>(a.codes) % 16 == 0;
  if (a.T <= 8)
    linear_rows_kernel<B, K, 1, kFine, 8><<<dim3(gx, gy(1)), 256, 0, s>>>(a, gshift, G, xvec, cvec);
  else if (a.T <= 16)
    linear_rows_kernel<B, K, 2, kFine, 8><<<dim3(gx, gy(2)), 256, 0, s>>>(a, gshift, G, xvec, cvec);
  else
    linear_rows_kernel<B, K, 4, kFine, 8><<<dim3(gx, gy(4)), 256, 0, s>>>(a, gshift, G, xvec, cvec);
}
template <LinearInput K>
void launch_bits(const LinearArgs& a, int xvec, cudaStream_t s) {
  const bool fine = a.group == 16 || a.group == 32;
  switch (a.bits) {
    case 2: return fine ? launch_rows<2, K, true>(a, xvec, s) : launch_rows<2, K, false>(a, xvec, s);
    case 3: return fine ? launch_rows<3, K, true>(a, xvec, s) : launch_rows<3, K, false>(a, xvec, s);
    case 4: return fine ? launch_rows<4, K, true>(a, xvec, s) : launch_rows<4, K, false>(a, xvec, s);
    case 5: return fine ? launch_rows<5, K, true>(a, xvec, s) : launch_rows<5, K, false>(a, xvec, s);
    case 6: return fine ? launch_rows<6, K, true>(a, xvec, s) : launch_rows<6, K, false>(a, xvec, s);
    case 7: return fine ? launch_rows<7, K, true>(a, xvec, s) : launch_rows<7, K, false>(a, xvec, s);
    default: return fine ? launch_rows<8, K, true>(a, xvec, s) : launch_rows<8, K, false>(a, xvec, s);
  }
}
}  // namespace

cudaError_t launch_linear_rows(const LinearArgs& a, LinearInput kind, cudaStream_t s) {
  if (a.T == 0) return cudaSuccess;
  const uintptr_t p = reinterpret_cast<uintptr_t>(a.x);
  // eight inputs of a token in one or two vector loads: rows have to start aligned
  const int xvec = !a.perm && a.n % 8 == 0 && p % (kind == kXInt8 ? 8 : 16) == 0;
  if (kind == kXBf16) launch_bits<kXBf16>(a, xvec, s);
  else if (kind == kXFp32) launch_bits<kXFp32>(a, xvec, s);
  else launch_bits<kXInt8>(a, xvec, s);
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
