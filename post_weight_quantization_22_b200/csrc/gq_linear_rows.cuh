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
// Groups of 32 and 16 are multiplied one by one in the same way.
// c - z is an exact integer in 16 bits, the products are exact, and the fp32 sums of one group
// are multiplied by the group's scale in fp32: no weight is rounded.  The warps of a CTA share
// the columns in chunks of 128 and add their sums in a fixed order; every warp loads a chunk
// ahead.  What holds it is latency at its occupancy, with no pipe full (one token, 32768 x 8192, 4
// bits: ALU 47 %, issue 49 %, DRAM 34 %, 24 % of the warps active): the chunk ahead is registers.
//
// fp32 tokens are taken as three bf16 parts (8 + 8 + 8 bits, exact), three products a weight;
// 8-bit tokens as fp16 integers.
#pragma once
#include "gq_internal.cuh"
#include "gq_unpack.cuh"

namespace gq {

namespace {
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

// B words in the widest loads that their size allows (vec: rows are 16-byte aligned).
template <int B>
__device__ __forceinline__ void load_words(const char* p, bool vec, uint32_t (&w)[B]) {
  if (B % 2 == 0 && !vec) {
#pragma unroll
    for (int i = 0; i < B; ++i) w[i] = __ldg(reinterpret_cast<const uint32_t*>(p) + i);
    return;
  }
  if constexpr (B % 4 == 0) {
#pragma unroll
    for (int i = 0; i < B / 4; ++i) {
      const uint4 v = __ldg(reinterpret_cast<const uint4*>(p) + i);
      w[4 * i] = v.x; w[4 * i + 1] = v.y; w[4 * i + 2] = v.z; w[4 * i + 3] = v.w;
    }
  } else if constexpr (B % 2 == 0) {
#pragma unroll
    for (int i = 0; i < B / 2; ++i) {
      const uint2 v = __ldg(reinterpret_cast<const uint2*>(p) + i);
      w[2 * i] = v.x; w[2 * i + 1] = v.y;
    }
  } else {
#pragma unroll
    for (int i = 0; i < B; ++i) w[i] = __ldg(reinterpret_cast<const uint32_t*>(p) + i);
  }
}

// B consecutive words of a row from word w0 on (0 behind the row's end).
template <int B>
__device__ __forceinline__ void load_run(const uint32_t* __restrict__ row, int w0, int words,
                                         bool vec, uint32_t (&w)[B]) {
  if (vec && w0 + B <= words) return load_words<B>(reinterpret_cast<const char*>(row + w0), true, w);
#pragma unroll
  for (int i = 0; i < B; ++i) w[i] = w0 + i < words ? __ldg(row + w0 + i) : 0u;
}

// One warp's share of a chunk of 128 columns for a lane's 2 RT rows, and of one token's inputs.
template <int B, LinearInput K, int RT>
struct Chunk {
  uint32_t w[2 * RT][B];  // lane t's 32 columns
  uint32_t z[2 * RT];     // their zero points
  float f[2 * RT][2];     // scales of the chunk's group, or of its halves'
  Raw<K> x[4];
};
// The groups in a chunk of 128 columns (a row's one grid counts as one).
enum GroupMode { kWhole = 1, kHalves = 2, kQuarters = 4, kEighths = 8 };
}  // namespace

// One CTA: 16 RT rows x (8 NT) tokens.  gshift: log2 of the group width (31: one grid per row).
// xvec, cvec: inputs and packed rows allow wide loads.
template <int B, LinearInput K, int NT, int RT, GroupMode M, int kWarps>
__global__ void __launch_bounds__(kWarps * 32)
    linear_rows_kernel(LinearArgs a, int gshift, int G, int xvec, int cvec) {
  constexpr bool kHalf = K == kXInt8;
  constexpr int P = K == kXFp32 ? 3 : 1;
  constexpr int kRows = 16 * RT;
  __shared__ float red[kWarps][NT * 8][kRows + 1];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int64_t row0 = (int64_t)blockIdx.x * kRows;
  const int n = (int)a.n, words = (int)row_words(a.n, B), chunks = (n + 127) / 128;
  const uint32_t* cp[2 * RT];  // the lane's rows: g, g + 8 of every tile of 16
  const float* sp[2 * RT];
  const uint8_t* zp[2 * RT];
#pragma unroll
  for (int r = 0; r < 2 * RT; ++r) {
    const int64_t row = min(row0 + 8 * r + g, a.m - 1);
    cp[r] = a.codes + row * words;
    sp[r] = a.scales + row * G;
    zp[r] = a.zeros + row * G;
  }

  for (int64_t t0 = (int64_t)blockIdx.y * NT * 8; t0 < a.T; t0 += (int64_t)gridDim.y * NT * 8) {
    float acc[RT][NT][4];
#pragma unroll
    for (int r = 0; r < RT; ++r)
#pragma unroll
      for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[r][j][i] = 0.f;
    // (behind the last token its row again: a column of the product is one token's alone, and
    // these columns are not stored)
    const void* xrow[NT];
#pragma unroll
    for (int j = 0; j < NT; ++j) xrow[j] = token_row<K>(a.x, min(t0 + j * 8 + g, a.T - 1), a.n);

    if constexpr (M <= 2) {
      auto fetch = [&](int c, Chunk<B, K, RT>& q) {
        const bool fast = xvec && c * 128 + 128 <= n;
        if constexpr (NT == 1) {
#pragma unroll
          for (int i = 0; i < 4; ++i)
            load_raw<K>(xrow[0], c * 128 + 32 * t + 8 * i, n, a.perm, fast, q.x[i]);
        }
        const int gl = min((c * 128 + 32 * t) >> gshift, G - 1);
        const int g0 = min((c * 128) >> gshift, G - 1);
#pragma unroll
        for (int r = 0; r < 2 * RT; ++r) {
          load_run<B>(cp[r], (c * 4 + t) * B, words, cvec, q.w[r]);
          q.z[r] = __ldg(zp[r] + gl);
          q.f[r][0] = __ldg(sp[r] + g0);
          if constexpr (M == kHalves) q.f[r][1] = __ldg(sp[r] + min(g0 + 1, G - 1));
        }
      };
      auto multiply = [&](int c, const Chunk<B, K, RT>& q, bool fast) {
        constexpr int kSets = M == kHalves ? 2 : 1;
        uint32_t zz[2 * RT];
#pragma unroll
        for (int r = 0; r < 2 * RT; ++r) zz[r] = zero_pair<B, kHalf>(q.z[r]);
        float part[kSets][RT][NT][4];
#pragma unroll
        for (int h = 0; h < kSets; ++h)
#pragma unroll
          for (int r = 0; r < RT; ++r)
#pragma unroll
            for (int j = 0; j < NT; ++j)
#pragma unroll
              for (int i = 0; i < 4; ++i) part[h][r][j][i] = 0.f;
#pragma unroll
        for (int i = 0; i < 4; ++i) {  // eight columns of the lane
          constexpr int kTop = B - 1;
          const int w = (i * B) / 4, sh = 8 * ((i * B) % 4);
          const int w1 = w + 1 < B ? w + 1 : kTop, w2 = w + 2 < B ? w + 2 : kTop;
          uint32_t pr[2 * RT][4];
#pragma unroll
          for (int r = 0; r < 2 * RT; ++r) {
            code_pairs<B>(__funnelshift_r(q.w[r][w], q.w[r][w1], sh),
                          __funnelshift_r(q.w[r][w1], q.w[r][w2], sh),
                          pair_other<B, kHalf>(), pr[r]);
#pragma unroll
            for (int e = 0; e < 4; ++e) pr[r][e] = pair_value<B, kHalf>(pr[r][e], zz[r]);
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
#pragma unroll
            for (int h = 0; h < kSets; ++h) {
              const bool mine = M == kWhole || (t >> 1) == h;
#pragma unroll
              for (int p = 0; p < P; ++p)
#pragma unroll
                for (int e = 0; e < 4; e += 2) {
                  const uint32_t b0 = mine ? b[p][e] : 0u, b1 = mine ? b[p][e + 1] : 0u;
#pragma unroll
                  for (int r = 0; r < RT; ++r)
                    mma_16816<kHalf>(part[h][r][j], pr[2 * r][e], pr[2 * r + 1][e],
                                     pr[2 * r][e + 1], pr[2 * r + 1][e + 1], b0, b1);
                }
            }
          }
        }
#pragma unroll
        for (int h = 0; h < kSets; ++h)
#pragma unroll
          for (int r = 0; r < RT; ++r)
#pragma unroll
            for (int j = 0; j < NT; ++j)
#pragma unroll
              for (int i = 0; i < 4; ++i)
                acc[r][j][i] += q.f[2 * r + (i >> 1)][h] * part[h][r][j][i];
      };
      // Whole chunks of aligned inputs have no bounds to check, and every address is a base of the
      // block plus a 32-bit offset.  They go to the warps in runs of four: lane t of a quad loads
      // the scales and zero points of the run's chunk t and hands them round (loaded by every
      // lane for every chunk they were half of the kernel's L1 wavefronts).
      const int whole = xvec ? n / 128 : 0, runs = (whole + 3) / 4;
      {
        const char* cb = reinterpret_cast<const char*>(a.codes + row0 * words);
        const char* sb = reinterpret_cast<const char*>(a.scales + row0 * G);
        const char* zb = reinterpret_cast<const char*>(a.zeros + row0 * G);
        constexpr int kPer = M == kHalves ? 2 : 1;  // groups of a chunk
        uint32_t oc[2 * RT], og[2 * RT];
#pragma unroll
        for (int r = 0; r < 2 * RT; ++r) {
          const int row = (int)min((int64_t)(8 * r + g), a.m - 1 - row0);
          oc[r] = (uint32_t)(row * words + t * B) * 4;
          og[r] = (uint32_t)(row * G);
        }
        constexpr int kXBytes = K == kXBf16 ? 2 : K == kXFp32 ? 4 : 1;
        const bool mine = t0 + g < a.T;  // (NT == 1: the other lanes' columns are not stored)
        const char* xb = static_cast<const char*>(a.x) + t0 * n * kXBytes;
        const uint32_t ox = (uint32_t)((mine ? g : 0) * n + 32 * t) * kXBytes;
        struct Run {
          float f[2 * RT][kPer];
          uint32_t z[2 * RT][kPer];
        };
        auto fetch_run = [&](int b, Run& q) {
          const uint32_t gi = gshift == 31 ? 0 : (uint32_t)(min(4 * b + t, whole - 1) * kPer);
#pragma unroll
          for (int r = 0; r < 2 * RT; ++r)
#pragma unroll
            for (int h = 0; h < kPer; ++h) {
              q.f[r][h] = __ldg(reinterpret_cast<const float*>(sb + (og[r] + gi + h) * 4));
              q.z[r][h] = __ldg(reinterpret_cast<const uint8_t*>(zb + (og[r] + gi + h)));
            }
        };
        auto fetch_chunk = [&](int c, Chunk<B, K, RT>& q) {
          if constexpr (NT == 1) {
            if (mine) {
#pragma unroll
              for (int i = 0; i < 4; ++i)
                load_raw<K>(xb + (ox + (uint32_t)c * 128 * kXBytes), 8 * i, n, nullptr, true, q.x[i]);
            }
          }
#pragma unroll
          for (int r = 0; r < 2 * RT; ++r) load_words<B>(cb + (oc[r] + (uint32_t)c * 16 * B), cvec, q.w[r]);
        };
        Chunk<B, K, RT> q[2];
        if constexpr (NT == 1)
#pragma unroll
          for (int k = 0; k < 2; ++k)
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
              for (int e = 0; e < (int)(sizeof(q[k].x[i].r) / 4); ++e) q[k].x[i].r[e] = 0;
        Run run, next;
        if (warp < runs) {
          fetch_run(warp, next);
          fetch_chunk(4 * warp, q[0]);
        }
        for (int b = warp; b < runs; b += kWarps) {
          run = next;
          if (b + kWarps < runs) fetch_run(b + kWarps, next);
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const int c = 4 * b + k;
            // the next chunk: of this run, or the first of the warp's next run
            const int cn = k < 3 && c + 1 < whole ? c + 1 : 4 * (b + kWarps);
            if (c < whole) {
              if (cn < whole) fetch_chunk(cn, q[(k + 1) & 1]);
              const int src = (lane & ~3) | k;
#pragma unroll
              for (int r = 0; r < 2 * RT; ++r) {
#pragma unroll
                for (int h = 0; h < kPer; ++h) q[k & 1].f[r][h] = __shfl_sync(~0u, run.f[r][h], src);
                q[k & 1].z[r] = __shfl_sync(~0u, run.z[r][0], src);
                if constexpr (M == kHalves) {
                  const uint32_t z1 = __shfl_sync(~0u, run.z[r][1], src);
                  if (t >= 2) q[k & 1].z[r] = z1;
                }
              }
              multiply(c, q[k & 1], true);
            }
          }
        }
      }
      for (int c = whole + warp; c < chunks; c += kWarps) {
        Chunk<B, K, RT> q;
        fetch(c, q);
        multiply(c, q, xvec && c * 128 + 128 <= n);
      }
    } else {
      // Groups of 32: lane t's 32 columns are the chunk's group t; of 16: its groups 2 t and
      // 2 t + 1.  Every group's product is an instruction sequence of its own, with the other
      // lanes' inputs at zero: four times the MMAs (the tensor pipe has room for them), with the
      // loads and the unpacking of the wider groups.
      constexpr int kOwn = M / 4;  // groups of a lane
      struct Ahead {
        uint32_t w[2 * RT][B];
        uint32_t z[2 * RT][kOwn];
        float f[2 * RT][kOwn];
        Raw<K> x[4];
      };
      const char* cb = reinterpret_cast<const char*>(a.codes + row0 * words);
      const char* sb = reinterpret_cast<const char*>(a.scales + row0 * G);
      const char* zb = reinterpret_cast<const char*>(a.zeros + row0 * G);
      uint32_t oc[2 * RT], og[2 * RT];
#pragma unroll
      for (int r = 0; r < 2 * RT; ++r) {
        const int row = (int)min((int64_t)(8 * r + g), a.m - 1 - row0);
        oc[r] = (uint32_t)(row * words + t * B) * 4;
        og[r] = (uint32_t)(row * G);
      }
      auto fetch = [&](int c, bool clean, Ahead& q) {
        if constexpr (NT == 1) {
          const bool fast = clean || (xvec && c * 128 + 128 <= n);
#pragma unroll
          for (int i = 0; i < 4; ++i)
            load_raw<K>(xrow[0], c * 128 + 32 * t + 8 * i, n, clean ? nullptr : a.perm, fast, q.x[i]);
        }
#pragma unroll
        for (int r = 0; r < 2 * RT; ++r) {
          if (clean) load_words<B>(cb + (oc[r] + (uint32_t)c * 16 * B), cvec, q.w[r]);
          else load_run<B>(cp[r], (c * 4 + t) * B, words, cvec, q.w[r]);
#pragma unroll
          for (int e = 0; e < kOwn; ++e) {
            int gi = c * M + t * kOwn + e;
            if (!clean) gi = min(gi, G - 1);
            q.z[r][e] = __ldg(reinterpret_cast<const uint8_t*>(zb + (og[r] + gi)));
            q.f[r][e] = __ldg(reinterpret_cast<const float*>(sb + (og[r] + gi) * 4));
          }
        }
      };
      auto multiply = [&](int c, const Ahead& q, bool fast) {
        uint32_t pr[4][2 * RT][4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          constexpr int kTop = B - 1;
          const int w = (i * B) / 4, sh = 8 * ((i * B) % 4);
          const int w1 = w + 1 < B ? w + 1 : kTop, w2 = w + 2 < B ? w + 2 : kTop;
#pragma unroll
          for (int r = 0; r < 2 * RT; ++r) {
            code_pairs<B>(__funnelshift_r(q.w[r][w], q.w[r][w1], sh),
                          __funnelshift_r(q.w[r][w1], q.w[r][w2], sh), pair_other<B, kHalf>(),
                          pr[i][r]);
            const uint32_t zz = zero_pair<B, kHalf>(q.z[r][kOwn == 2 ? i >> 1 : 0]);
#pragma unroll
            for (int e = 0; e < 4; ++e) pr[i][r][e] = pair_value<B, kHalf>(pr[i][r][e], zz);
          }
        }
#pragma unroll
        for (int j = 0; j < NT; ++j) {
          uint32_t b[4][P][4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            if constexpr (NT == 1) {
              input_pairs<K, P>(q.x[i], b[i]);
            } else {
              Raw<K> x;
              load_raw<K>(xrow[j], c * 128 + 32 * t + 8 * i, n, a.perm, fast, x);
              input_pairs<K, P>(x, b[i]);
            }
          }
#pragma unroll
          for (int h = 0; h < 4; ++h) {
#pragma unroll
            for (int e = 0; e < kOwn; ++e) {
              float d[RT][4];
#pragma unroll
              for (int r = 0; r < RT; ++r)
#pragma unroll
                for (int i = 0; i < 4; ++i) d[r][i] = 0.f;
#pragma unroll
              for (int i = e * (4 / kOwn); i < (e + 1) * (4 / kOwn); ++i)
#pragma unroll
                for (int p = 0; p < P; ++p)
#pragma unroll
                  for (int v = 0; v < 4; v += 2) {
                    const uint32_t b0 = t == h ? b[i][p][v] : 0u, b1 = t == h ? b[i][p][v + 1] : 0u;
#pragma unroll
                    for (int r = 0; r < RT; ++r)
                      mma_16816<kHalf>(d[r], pr[i][2 * r][v], pr[i][2 * r + 1][v],
                                       pr[i][2 * r][v + 1], pr[i][2 * r + 1][v + 1], b0, b1);
                  }
              const int src = (lane & ~3) | h;
#pragma unroll
              for (int r = 0; r < RT; ++r) {
                const float fa = __shfl_sync(~0u, q.f[2 * r][e], src);
                const float fb = __shfl_sync(~0u, q.f[2 * r + 1][e], src);
                acc[r][j][0] += fa * d[r][0];
                acc[r][j][1] += fa * d[r][1];
                acc[r][j][2] += fb * d[r][2];
                acc[r][j][3] += fb * d[r][3];
              }
            }
          }
        }
      };
      const int whole = xvec ? n / 128 : 0;
      Ahead q[2];
      if (warp < whole) fetch(warp, true, q[0]);
      for (int c = warp; c < whole; c += 2 * kWarps) {
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const int at = c + k * kWarps;
          if (at < whole) {
            if (at + kWarps < whole) fetch(at + kWarps, true, q[k ^ 1]);
            multiply(at, q[k], true);
          }
        }
      }
      for (int c = whole + warp; c < chunks; c += kWarps) {
        fetch(c, false, q[0]);
        multiply(c, q[0], xvec && c * 128 + 128 <= n);
      }
    }
#pragma unroll
    for (int r = 0; r < RT; ++r)
#pragma unroll
      for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i)
          red[warp][j * 8 + 2 * t + (i & 1)][16 * r + g + 8 * (i >> 1)] = acc[r][j][i];
    __syncthreads();
    for (int i = threadIdx.x; i < NT * 8 * kRows; i += kWarps * 32) {
      const int tt = i / kRows, rr = i % kRows;
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
template <int B, LinearInput K, GroupMode M>
void launch_mode(const LinearArgs& a, int xvec, cudaStream_t s) {
  const int gshift = a.group ? __builtin_ctz((unsigned)a.group) : 31;
  const int G = a.group ? (int)((a.n + a.group - 1) / a.group) : 1;
  const int cvec = row_words(a.n, B) % 4 == 0 && reinterpret_cast<uintptr_t>(a.codes) % 16 == 0;
  auto grid = [&](int rows, int tokens) {
    const int64_t tiles = (a.T + tokens - 1) / tokens;
    return dim3((unsigned)((a.m + rows - 1) / rows), (unsigned)(tiles < 32768 ? tiles : 32768));
  };
  // Two tiles of rows a warp share the inputs' part of the work, which is large for fp32 (three
  // parts) and from a few tokens on; one token of 16 or 8 bits is faster with one tile and more
  // CTAs (4096 x 4096, 4 bits: one bf16 token 4.5 us against 5.0, eight 6.1 against 5.6, one fp32
  // token 10.3 against 7.7), as are few rows.
  const bool two = a.m >= 2048 && (K == kXFp32 || a.T >= 4);
  if (a.T <= 8 && !two)
    linear_rows_kernel<B, K, 1, 1, M, 8><<<grid(16, 8), 256, 0, s>>>(a, gshift, G, xvec, cvec);
  else if (a.T <= 8)
    linear_rows_kernel<B, K, 1, 2, M, 8><<<grid(32, 8), 256, 0, s>>>(a, gshift, G, xvec, cvec);
  else if (a.T <= 16)
    linear_rows_kernel<B, K, 2, 1, M, 8><<<grid(16, 16), 256, 0, s>>>(a, gshift, G, xvec, cvec);
  else
    linear_rows_kernel<B, K, 4, 1, M, 8><<<grid(16, 32), 256, 0, s>>>(a, gshift, G, xvec, cvec);
}
template <int B, LinearInput K>
void launch_input(const LinearArgs& a, int xvec, cudaStream_t s) {
  if (a.group == 16) launch_mode<B, K, kEighths>(a, xvec, s);
  else if (a.group == 32) launch_mode<B, K, kQuarters>(a, xvec, s);
  else if (a.group == 64) launch_mode<B, K, kHalves>(a, xvec, s);
  else launch_mode<B, K, kWhole>(a, xvec, s);
}
}  // namespace

template <int B>
void linear_rows_bits(const LinearArgs& a, LinearInput kind, int xvec, cudaStream_t s) {
  if (kind == kXBf16) launch_input<B, kXBf16>(a, xvec, s);
  else if (kind == kXFp32) launch_input<B, kXFp32>(a, xvec, s);
  else launch_input<B, kXInt8>(a, xvec, s);
}

}  // namespace gq
