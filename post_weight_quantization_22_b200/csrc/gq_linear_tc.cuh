// Products with a packed layer for many tokens, on the 5th-generation tensor cores.
//
// y[t][r] = sum_g s[r][g] sum_{k in g} x[t][k] (c[r][k] - z[r][g]).  A CTA computes 128 rows: the
// rows' codes are unpacked into bf16 tiles (c - z is an integer of at most 8 bits and a sign:
// exact) that are the instruction's A operand, the tokens come by TMA as its B operand, and every
// group's sum is formed in a tensor-memory accumulator of its own, two in turn.  Eight warps take
// a finished accumulator out, multiply it with the group's scale in fp32 (a thread holds one row,
// so the scale is one register) and add it to sums in registers while the next group is
// multiplied.  No weight is rounded, and no chain of tensor-core additions is longer than 256
// columns.
//
// Two forms.  With tiles enough for every SM, two CTAs form a pair (cta_group::2): 256 rows x 256
// tokens, each CTA loading and holding half of the tokens' tile (2048 tokens, 4096 x 4096, per-row
// grid: 76 us against 85 of single CTAs on 256 tokens); the pair takes tile after tile, and the next tile is
// unpacked and multiplied while the last one's sums are stored.  With fewer, a CTA takes 128
// tokens, and up to eight CTAs of a cluster share one tile's columns and add their sums over
// distributed shared memory in a fixed order.
//
// Roles: warp 0 the tokens' TMA loads, warp 1 the MMAs, warps 4-11 unpack (four for the even
// stages of the ring, four for the odd ones), warps 12-19 scale and add.
#pragma once
#include "gq_internal.cuh"
#include "gq_linear.cuh"
#include "gq_tc.cuh"
#include "gq_unpack.cuh"

namespace gq {

namespace {
constexpr int kLinThreads = 640;
constexpr int kUnpackWarp = 4, kScaleWarp = 12;   // first warps of these roles, 8 each
// Registers a thread of the three roles holds, in warpgroups of 128 threads: together what the
// launch has (96 x 640).  A pair's scaling thread holds 128 sums, a single CTA's 64.
constexpr int kRegsLaunch = 96;
template <bool kPair>
struct LinRegs {
  static constexpr int control = kPair ? 32 : 64, unpack = kPair ? 48 : 88,
                       scale = kPair ? 176 : 120;
  static_assert(control + 2 * unpack + 2 * scale == 5 * kRegsLaunch, "register shares");
};
constexpr uint32_t kTile = 128 * kCols * 2;       // 128 rows or tokens of them, 128 bytes each
constexpr uint32_t kOutStage = 1024;              // a scaling warp's output staging
// Shared memory: the ring of stages (each the unpacked rows and P parts of the tokens), the
// pairs' ring of packed chunks of 128 columns (2 KB a bit) in what is left, output staging.
constexpr uint32_t kLinSmem = 226 * 1024;
constexpr uint32_t kLinRings = kLinSmem - 8 * kOutStage - 1024 - 1024;
constexpr int lin_stages(int P, bool pair) { return P == 3 ? 3 : pair ? 5 : 6; }
constexpr int lin_chunks(int B, int P) {
  const int fit = (int)((kLinRings - lin_stages(P, true) * (1 + P) * kTile) / (2048 * B));
  return fit < 8 ? fit : 8;
}

// What a loading thread waits at its end for each of its last copies: they take microseconds, and
// 2^18 looks at a barrier 20 ms, also where the phase stays open because another role has given up.
constexpr uint32_t kDrainPolls = 1u << 18;
constexpr long long kDrainCycles = 4000000;  // the same for a thread that cannot look: 2 ms

// Waits for at most `polls` looks, and gives up when another role of the CTA has.
__device__ __forceinline__ bool wait_or_fail(uint64_t* bar, uint32_t parity, volatile int* fail,
                                             uint32_t polls) {
  for (uint32_t i = 0; i < polls; ++i) {
    if (tc::mbar_try_wait(bar, parity)) return true;
    if ((i & 1023) == 1023 && *fail) return false;
  }
  *fail = 1;
  return false;
}
// The same for a whole warp, with one answer.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, volatile int* fail,
                                          uint32_t polls) {
  return __all_sync(~0u, wait_or_fail(bar, parity, fail, polls));
}

__device__ __forceinline__ void fma2(uint64_t& acc, float a, float b, uint64_t s) {
  uint64_t v;
  asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "f"(a), "f"(b));
  asm("fma.rn.f32x2 %0, %1, %2, %0;" : "+l"(acc) : "l"(v), "l"(s));
}
__device__ __forceinline__ void put(float* p, float v) { *p = v; }
__device__ __forceinline__ void put(__nv_bfloat16* p, float v) { *p = __float2bfloat16(v); }
// A warp's 32 rows x 2 E tokens of sums into y (T x m; y at the warp's first row and token): rows
// < rows and tokens < cnt are written, times the tokens' scales xs (null: 1).  With rows of y on
// 16-byte boundaries the values go through shared memory, so that a lane stores 16 bytes (one
// 2-byte store per value took 11 cycles a warp instruction, 12,000 cycles a tile).
template <int E, class Y>
__device__ __forceinline__ void store_tile(Y* y, int64_t ld, const uint64_t (&acc)[E], int cnt,
                                           int rows, const float* __restrict__ xs, bool wide,
                                           uint8_t* stage, int lane) {
  constexpr int kTok = (int)(kOutStage / (32 * sizeof(Y)));  // tokens per staging pass
  constexpr int kVec = 16 / (int)sizeof(Y);                  // values in 16 bytes
  constexpr int kPer = 32 / kVec;                            // lanes per token
  Y* st = reinterpret_cast<Y*>(stage);
#pragma unroll
  for (int b = 0; b < 2 * E / kTok; ++b) {
    if (b * kTok >= cnt) break;
    if (wide) {
#pragma unroll
      for (int j = 0; j < kTok; ++j) {
        const float2 v2 = *reinterpret_cast<const float2*>(&acc[(b * kTok + j) / 2]);
        float v = (j & 1) ? v2.y : v2.x;
        if (xs && b * kTok + j < cnt) v *= __ldg(xs + b * kTok + j);
        put(st + j * 32 + lane, v);
      }
      __syncwarp();
      const int r = (lane % kPer) * kVec;
#pragma unroll
      for (int i = 0; i < kTok * kPer / 32; ++i) {
        const int j = i * (32 / kPer) + lane / kPer;
        const uint4 v = *reinterpret_cast<const uint4*>(st + j * 32 + r);
        if (b * kTok + j < cnt && r < rows)
          *reinterpret_cast<uint4*>(y + (b * kTok + j) * ld + r) = v;
      }
      __syncwarp();
    } else if (lane < rows) {
#pragma unroll
      for (int j = 0; j < kTok; ++j) {
        const float2 v2 = *reinterpret_cast<const float2*>(&acc[(b * kTok + j) / 2]);
        const float v = (j & 1) ? v2.y : v2.x;
        if (b * kTok + j < cnt)
          put(y + (b * kTok + j) * ld + lane, xs ? v * __ldg(xs + b * kTok + j) : v);
      }
    }
  }
}
__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ uint32_t cluster_size() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ float ld_cluster_f32(uint32_t local, uint32_t rank) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(tc::mapa(local, rank)) : "memory");
  return v;
}

// The B words of one unit of 32 columns (words behind the row's end are 0).  vec: rows and base
// allow the widest loads that a unit's size allows.
template <int B>
__device__ __forceinline__ void load_unit(const uint32_t* __restrict__ row, int unit, int words,
                                          bool vec, uint32_t (&w)[B]) {
  const int w0 = unit * B;
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

// The B words of a unit (unit 0..3 of a chunk's row r) from a packed chunk in shared memory, as
// its TMA load laid it out: 64- and 128-byte rows swizzled, so that eight rows' 16-byte reads
// fall on different banks.
template <int B>
__device__ __forceinline__ void load_unit_smem(const uint8_t* chunk, int r, int unit,
                                               uint32_t (&w)[B]) {
  const uint8_t* row = chunk + r * (16 * B);
  if constexpr (B == 4 || B == 8) {
    const int x = B == 4 ? (r >> 1) & 3 : r & 7;
#pragma unroll
    for (int i = 0; i < B / 4; ++i) {
      const uint4 v = *reinterpret_cast<const uint4*>(row + (((unit * (B / 4) + i) ^ x) << 4));
      w[4 * i] = v.x; w[4 * i + 1] = v.y; w[4 * i + 2] = v.z; w[4 * i + 3] = v.w;
    }
  } else if constexpr (B % 2 == 0) {
#pragma unroll
    for (int i = 0; i < B / 2; ++i) {
      const uint2 v = *reinterpret_cast<const uint2*>(row + unit * 4 * B + 8 * i);
      w[2 * i] = v.x; w[2 * i + 1] = v.y;
    }
  } else {
#pragma unroll
    for (int i = 0; i < B; ++i) w[i] = *reinterpret_cast<const uint32_t*>(row + unit * 4 * B + 4 * i);
  }
}
}  // namespace

// P: parts of the tokens (3 for fp32).  kPair: two CTAs on 256 rows x 256 tokens, else one on 128
// rows x N <= 128 tokens.  vec: the packed rows allow wide loads; wide: rows of y are on 16-byte
// boundaries.
template <int B, int P, bool kPair>
__global__ void __launch_bounds__(kLinThreads, 1)
    linear_tc_kernel(const __grid_constant__ CUtensorMap m_x,
                     const __grid_constant__ CUtensorMap m_c, LinTcArgs a, int vec, int wide) {
  constexpr int kN = kPair ? 256 : 128;                 // accumulator columns
  constexpr uint32_t kStage = (1 + P) * kTile;          // unpacked rows, then the tokens' parts
  constexpr int kStages = lin_stages(P, kPair);
  constexpr int kChunks = lin_chunks(B, P);             // of the packed ring (pairs)
  constexpr uint32_t kChunkBytes = 2048 * B;
  static_assert(kChunks >= 1 && kStages * kStage <= kLinRings, "shared memory");
  extern __shared__ uint8_t lin_smem[];
  uint8_t* base = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(lin_smem) + 1023) & ~uintptr_t(1023));
  uint8_t* cring = base + kStages * kStage;
  uint8_t* ostage = base + kLinRings;
  uint64_t* full = reinterpret_cast<uint64_t*>(ostage + 8 * kOutStage);
  uint64_t* empty = full + kStages;
  uint64_t* c_full = empty + kStages + 5;
  uint64_t* c_empty = c_full + kChunks;
  uint64_t* t_full = empty + kStages;
  uint64_t* t_empty = t_full + 2;
  uint64_t* done = t_empty + 2;
  uint32_t* tslot = reinterpret_cast<uint32_t*>(c_empty + kChunks);
  volatile int* fail = reinterpret_cast<volatile int*>(tslot + 1);
  static_assert((2 * kStages + 5 + 2 * kChunks) * 8 + 8 <= 1024, "barriers");

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t S = cluster_size(), rank = cluster_rank();
  const int tile0 = (int)(blockIdx.x / S), tstep = (int)(gridDim.x / S);
  const int N = a.N;
  const uint32_t polls = a.wait.polls;
  // this CTA's stages: all, or its share of a tile that a cluster splits (in runs of 256 columns,
  // the longest period)
  const int runs = (a.stages + 3) / 4;
  const int st0 = kPair ? 0 : 4 * (int)((int64_t)runs * rank / S);
  const int ns = kPair ? a.stages : min(a.stages, 4 * (int)((int64_t)runs * (rank + 1) / S)) - st0;
  const int steps = ns * 4;                                        // of 16 columns, a tile
  const int periods = (steps + a.dmask) / (a.dmask + 1);           // a tile
  // first row and token of a tile for this CTA's scaling warps; its rows' and tokens' operands
  auto row_of = [&](int tile) {
    return (int64_t)(tile % a.mtiles) * (kPair ? 256 : 128) + (kPair ? 128 * rank : 0);
  };
  auto tok_of = [&](int tile) { return (int64_t)(tile / a.mtiles) * N; };

  if (blockIdx.x == 0 && tid == 0) a.hdr->status = 0;  // no wait can run out for a second yet
  if (tid == 0) {
    constexpr int kCtas = kPair ? 2 : 1;
    for (int i = 0; i < kStages; ++i) {
      tc::mbar_init(&full[i], 4 * kCtas + 1);  // unpacking warps, and the loads' expectation
      tc::mbar_init(&empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      tc::mbar_init(&t_full[i], 1);
      tc::mbar_init(&t_empty[i], 8 * kCtas);
    }
    if constexpr (kPair)
      for (int i = 0; i < kChunks; ++i) {
        tc::mbar_init(&c_full[i], 1);
        tc::mbar_init(&c_empty[i], 8);
      }
    tc::mbar_init(done, 1);
    *fail = 0;
    tc::fence_barrier_init();
    tc::prefetch_tmap(&m_x);
    if constexpr (kPair) tc::prefetch_tmap(&m_c);
  }
  if (warp == 2) {
    if constexpr (kPair) tc::tmem_alloc_pair(tslot, 2 * kN);
    else tc::tmem_alloc(tslot, 2 * kN);
  }
  tc::fence_before_sync();
  __syncthreads();
  if (S > 1) cluster_sync();  // the other CTAs' barriers are there
  tc::fence_after_sync();
  const uint32_t tmem = *tslot;
  // the barriers that the MMA thread waits for are in the pair's first CTA
  const uint32_t full_at = kPair ? tc::mapa(tc::smem_u32(full), 0) : tc::smem_u32(full);
  const uint32_t t_empty_at = kPair ? tc::mapa(tc::smem_u32(t_empty), 0) : tc::smem_u32(t_empty);
  auto arrive = [&](uint32_t bar) {  // for a whole warp
    __syncwarp();
    if (lane == 0) tc::mbar_arrive_cluster(bar);
  };

  if (warp < kUnpackWarp) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(LinRegs<kPair>::control));
    if (warp == 0) {
      if (tc::elect_one()) {
        // tokens: 64 columns of every part per stage
        const int rows = kPair ? 128 : N;
        int i = 0, s = 0;
        uint32_t ph = 1;
        bool ok = true;
        // (test setting: the first CTA withholds its second arrival, so that this stage never fills
        // and every role runs out of looks, behind one stage's MMAs and with the ring loaded)
        const bool held = a.wait.withhold && blockIdx.x == 0;
        for (int tile = tile0; tile < a.tiles && ok; tile += tstep) {
          const int t0 = (int)(tok_of(tile) + (kPair ? 128 * rank : 0));
          for (int st = 0; st < ns; ++st, ++i) {
            if (i >= kStages && !wait_or_fail(&empty[s], ph, fail, polls)) {
              ok = false;
              break;
            }
            if (!kPair || rank == 0) {
              const uint32_t bytes = (uint32_t)((kPair ? 2 : 1) * P * rows * 128);
              if (held && i == 1) tc::mbar_expect_tx(&full[s], bytes);
              else tc::mbar_arrive_expect_tx(&full[s], bytes);
            }
            uint8_t* dst = base + s * kStage + kTile;
#pragma unroll
            for (int p = 0; p < P; ++p) {
              const int x = (st0 + st) * kCols, y = t0 + p * a.planes_t;
              if constexpr (kPair)
                tc::tma_load_2d_pair(dst + p * kTile, &m_x, full_at + 8 * s, x, y);
              else
                tc::tma_load_2d(dst + p * kTile, &m_x, &full[s], x, y);
            }
            if (++s == kStages) {
              s = 0;
              ph ^= 1;
            }
          }
        }
        // No copy may be in flight when the CTAs end, whichever role has given up (where none has,
        // the other roles wait for the same phases): the first CTA's barriers count both CTAs'
        // bytes, and the pair ends together.  The second CTA cannot look at them; where it gives
        // up, it leaves its last copies their time.
        if (!kPair || rank == 0) {
          for (int j = max(0, i - kStages); j < i; ++j)
            tc::mbar_wait_polls(&full[j % kStages], (j / kStages) & 1, kDrainPolls);
        } else if (!ok) {
          const long long t = clock64();
          while (clock64() - t < kDrainCycles) {}
        }
      }
    } else if (kPair && warp == 3) {
      if (tc::elect_one()) {
        // packed chunks of this CTA's rows
        int i = 0, s = 0;
        uint32_t ph = 1;
        bool ok = true;
        for (int tile = tile0; tile < a.tiles && ok; tile += tstep) {
          const int row = (int)row_of(tile);
          for (int c = 0; 2 * c < ns; ++c, ++i) {
            if (i >= kChunks && !wait_or_fail(&c_empty[s], ph, fail, polls)) {
              ok = false;
              break;
            }
            tc::mbar_arrive_expect_tx(&c_full[s], kChunkBytes);
            tc::tma_load_2d(cring + s * kChunkBytes, &m_c, &c_full[s], c * 4 * B, row);
            if (++s == kChunks) {
              s = 0;
              ph ^= 1;
            }
          }
        }
        for (int j = max(0, i - kChunks); j < i; ++j)
          tc::mbar_wait_polls(&c_full[j % kChunks], (j / kChunks) & 1, kDrainPolls);
      }
    } else if (warp == 1 && (!kPair || rank == 0)) {
      if (tc::elect_one()) {
        // One thread issues every MMA; a step of 16 columns takes the tensor cores 128 cycles, so
        // what surrounds it has to be short: descriptors differ in their address field alone,
        // the counters are masks, and the next stage's barrier is looked at (a round trip of 100
        // to 400 cycles to shared memory) before this stage's MMAs are issued.
        const uint32_t idesc = tc::idesc_f32acc(1, 1, 0, 0, kPair ? 256 : 128, (uint32_t)N);
        const uint64_t dbase = tc::sdesc(tc::smem_u32(base), 16, 1024, tc::kLayoutSW128);
        const int dmask = a.dmask;
        auto mma = [&](uint32_t d, uint64_t da, uint64_t db, bool acc) {
          if constexpr (kPair) tc::mma_f16_pair(d, da, db, idesc, acc);
          else tc::mma_f16(d, da, db, idesc, acc);
        };
        auto commit = [&](uint64_t* bar) {
          if constexpr (kPair) tc::mma_commit_pair(bar);
          else tc::mma_commit(bar);
        };
        int s = 0, period = 0;
        uint32_t ph = 0;
        bool ok = true, seen = false, free_seen = false;
        for (int tile = tile0; tile < a.tiles && ok; tile += tstep) {
          int step = 0;
          for (int st = 0; st < ns; ++st) {
            if (!seen && !wait_or_fail(&full[s], ph, fail, polls)) {
              ok = false;
              break;
            }
            const int s_next = s + 1 == kStages ? 0 : s + 1;
            const uint32_t ph_next = s_next ? ph : ph ^ 1;
            const uint64_t da = dbase + s * (kStage >> 4);
            if (dmask >= 3) {  // a period is one or more stages
              const bool first = (step & dmask) == 0;
              if (first && period >= 2 && !free_seen)
                ok = wait_or_fail(&t_empty[period & 1], ((period >> 1) - 1) & 1, fail, polls);
              if (!ok) break;
              seen = tc::mbar_test_wait(&full[s_next], ph_next);
              tc::fence_after_sync();
              const uint32_t d = tmem + (period & 1) * kN;
#pragma unroll
              for (int k = 0; k < 4; ++k)
#pragma unroll
                for (int p = 0; p < P; ++p)
                  mma(d, da + 2 * k, da + (1 + p) * (kTile >> 4) + 2 * k, k > 0 || p > 0 || !first);
              step += 4;
              if ((step & dmask) == 0 || step == steps) {
                commit(&t_full[period & 1]);
                ++period;
                free_seen = period >= 2 &&
                            tc::mbar_test_wait(&t_empty[period & 1], ((period >> 1) - 1) & 1);
              }
            } else {  // groups of 16 or 32 columns: several periods in a stage
              seen = tc::mbar_test_wait(&full[s_next], ph_next);
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                const bool first = (step & dmask) == 0;
                if (first && period >= 2)
                  ok = ok && wait_or_fail(&t_empty[period & 1], ((period >> 1) - 1) & 1, fail, polls);
                if (!ok) break;
                tc::fence_after_sync();
                const uint32_t d = tmem + (period & 1) * kN;
#pragma unroll
                for (int p = 0; p < P; ++p)
                  mma(d, da + 2 * k, da + (1 + p) * (kTile >> 4) + 2 * k, p > 0 || !first);
                ++step;
                if ((step & dmask) == 0) {
                  commit(&t_full[period & 1]);
                  ++period;
                }
              }
              if (!ok) break;
            }
            commit(&empty[s]);
            s = s_next;
            ph = ph_next;
          }
        }
        commit(done);
      }
    }
    __syncwarp();
  } else if (warp < kScaleWarp) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(LinRegs<kPair>::unpack));
    // Unpack.  Warps 4-7 fill the even stages, 8-11 the odd ones; a thread takes one unit of 32
    // columns in each of two rows (a warp reads 16 rows x 8 b bytes at a time; its 16-byte stores
    // of one column block fall on 8 different rows in every quarter, so the swizzled tile takes
    // them without conflicts).
    const int odd = (warp - kUnpackWarp) >> 2;
    const int words = (int)row_words(a.l.n, B);
    const int G = a.groups, gsh = a.gshift;
    const int u2 = (lane >> 3) & 1;
    const int r_in = (warp & 3) * 32 + (lane >> 4) * 8 + (lane & 7);  // and 16 rows on
    const uint32_t* rp[2];
    const uint8_t* zp[2];
    uint32_t w[2][B], z[2][2];
    auto rows_of = [&](int tile) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int64_t r = min(row_of(tile) + r_in + 16 * i, a.l.m - 1);
        if constexpr (!kPair) rp[i] = a.l.codes + r * words;
        zp[i] = a.l.zeros + r * G;
      }
    };
    auto load_zeros = [&](int st, int i) {
      const int g0 = min((((st0 + st) * 2 + u2) * 32) >> gsh, G - 1);
      z[i][0] = __ldg(zp[i] + g0);
      z[i][1] = gsh == 4 ? __ldg(zp[i] + min(g0 + 1, G - 1)) : z[i][0];
    };
    auto load_words = [&](int st, int i) {
      if constexpr (!kPair) load_unit<B>(rp[i], (st0 + st) * 2 + u2, words, vec, w[i]);
    };
    auto store_unit = [&](uint8_t* tilep, int i) {
      const int r = r_in + 16 * i;
#pragma unroll
      for (int j = 0; j < 4; ++j) {  // eight columns
        constexpr int kTop = B - 1;
        const int q = (j * B) / 4, sh = 8 * ((j * B) % 4);
        const uint32_t w0 = w[i][q], w1 = w[i][q + 1 < B ? q + 1 : kTop];
        const uint32_t w2 = w[i][q + 2 < B ? q + 2 : kTop];
        uint32_t pr[4];
        code_pairs<B>(__funnelshift_r(w0, w1, sh), __funnelshift_r(w1, w2, sh),
                      pair_other<B, false>(), pr);
        const uint32_t zz = zero_pair<B, false>(z[i][j >> 1]);
#pragma unroll
        for (int e = 0; e < 4; ++e) pr[e] = pair_value<B, false>(pr[e], zz);
        uint4 v;  // from pairs (e, e + 4) to columns in order
        v.x = __byte_perm(pr[0], pr[1], 0x5410);
        v.y = __byte_perm(pr[2], pr[3], 0x5410);
        v.z = __byte_perm(pr[0], pr[1], 0x7632);
        v.w = __byte_perm(pr[2], pr[3], 0x7632);
        const int blk = u2 * 4 + j;
        *reinterpret_cast<uint4*>(tilep + r * 128 + ((blk ^ (r & 7)) << 4)) = v;
      }
    };
    // The stages of all tiles in one count: this role's are odd, odd + 2, ..  (A pair's tile has an
    // even number of them, so that both roles read every packed chunk: a role that left one out
    // could take the phase before a chunk's barrier for the phase it waits for.)
    int tile = tile0, st = odd, chunk0 = 0;  // chunk0: packed chunks of the tiles before
    const int per_tile = ns / 2;
    while (st >= ns && tile < a.tiles) {
      st -= ns;
      tile += tstep;
      chunk0 += per_tile;
    }
    if (tile < a.tiles) {
      rows_of(tile);
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        load_zeros(st, i);
        load_words(st, i);
      }
    }
    int s = odd, use = 0;
    while (tile < a.tiles) {
      const int cc = chunk0 + (st >> 1), cs = cc % kChunks;
      if constexpr (kPair) {
        if (!warp_wait(&c_full[cs], (cc / kChunks) & 1, fail, polls)) break;
#pragma unroll
        for (int i = 0; i < 2; ++i)
          load_unit_smem<B>(cring + cs * kChunkBytes, r_in + 16 * i, (st & 1) * 2 + u2, w[i]);
      }
      if (use > 0 && !warp_wait(&empty[s], (use - 1) & 1, fail, polls)) break;
      uint8_t* tilep = base + s * kStage;
      int next = tile;
      st += 2;
      while (st >= ns && next < a.tiles) {
        st -= ns;
        next += tstep;
        chunk0 += per_tile;
      }
      const bool more = next < a.tiles;
      if (more && next != tile) rows_of(next);
      tile = next;
#pragma unroll
      for (int i = 0; i < 2; ++i) store_unit(tilep, i);
      tc::fence_proxy_async_smem();
      arrive(full_at + 8 * s);
      // the next stage's loads only now: the fence waits for every access in flight
      if (more) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          load_zeros(st, i);
          load_words(st, i);
        }
      }
      if constexpr (kPair) {
        if (lane == 0) tc::mbar_arrive(&c_empty[cs]);
      }
      s += 2;
      if (s >= kStages) {
        s -= kStages;
        ++use;
      }
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(LinRegs<kPair>::scale));
    // scale and add: thread = row, this warp's half of the tokens
    const int half = (warp - kScaleWarp) >> 2, quarter = warp & 3;
    const int G = a.groups;
    const bool grid1 = a.gshift == 31;  // one scale per row
    const int gfirst = (st0 * kCols) >> a.gshift;
    const uint32_t tcol = tmem + ((uint32_t)(quarter * 32) << 16) + half * (N / 2);
    int pt = 0;  // periods of all tiles
    bool ok = true;
    for (int tile = tile0; tile < a.tiles && ok; tile += tstep) {
      const int64_t row0 = row_of(tile) + quarter * 32;  // this warp's
      const int64_t tk = tok_of(tile) + half * (N / 2);
      const float* sp = a.l.scales + min(row0 + lane, a.l.m - 1) * G;
      uint64_t acc[kN / 4];
#pragma unroll
      for (int j = 0; j < kN / 4; ++j) acc[j] = 0;
      float s_next = __ldg(sp + min(gfirst, G - 1));
      for (int p = 0; p < periods; ++p, ++pt) {
        const float s = s_next;
        if (!grid1 && p + 1 < periods) s_next = __ldg(sp + min(gfirst + p + 1, G - 1));
        if (!warp_wait(&t_full[pt & 1], (pt >> 1) & 1, fail, polls)) {
          ok = false;
          break;
        }
        tc::fence_after_sync();
        uint64_t s2;
        asm("mov.b64 %0, {%1, %1};" : "=l"(s2) : "f"(s));
        const uint32_t at = tcol + (pt & 1) * kN;
#pragma unroll
        for (int cb = 0; cb < kN / 64; ++cb) {
          if (cb * 32 < N / 2) {
            float v[32];
            tc::tmem_ld32(at + cb * 32, v);
#pragma unroll
            for (int e = 0; e < 16; ++e) fma2(acc[cb * 16 + e], v[2 * e], v[2 * e + 1], s2);
          }
        }
        tc::fence_before_sync();
        arrive(t_empty_at + 8 * (pt & 1));
      }
      if (!ok) {
        if (lane == 0) {
          record_status(a.hdr, GQ_ERR_TIMEOUT);
          record_status(a.device_hdr, GQ_ERR_TIMEOUT);
        }
      } else if (kPair || S == 1) {
        const int cnt = (int)min((int64_t)(N / 2), a.l.T - tk);
        const int rows = (int)min((int64_t)32, a.l.m - row0);
        const float* xs = a.l.xscale ? a.l.xscale + tk : nullptr;
        uint8_t* st = ostage + (warp - kScaleWarp) * kOutStage;
        if (a.l.y_bf16)
          store_tile(static_cast<__nv_bfloat16*>(a.l.y) + tk * a.l.m + row0, a.l.m, acc, cnt,
                     rows, xs, wide, st, lane);
        else
          store_tile(static_cast<float*>(a.l.y) + tk * a.l.m + row0, a.l.m, acc, cnt, rows, xs,
                     wide, st, lane);
      } else {
        // partial sums as [token][row] over the ring (a shared tile is the CTA's only one, and
        // every MMA of it is complete: its last accumulator has been read)
        float* part = reinterpret_cast<float*>(base);
#pragma unroll
        for (int e = 0; e < kN / 4; ++e) {
          if (2 * e < N / 2) {
            const float2 v = *reinterpret_cast<const float2*>(&acc[e]);
            float* q = part + (half * (N / 2) + 2 * e) * 128 + quarter * 32 + lane;
            q[0] = v.x;
            q[128] = v.y;
          }
        }
      }
    }
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  // Back to the launch's register share for the common end.  Only behind the barrier: the two
  // smaller shares may not grow before the larger one has been taken and given back, or it could
  // never be taken.
  if (warp >= kScaleWarp)
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsLaunch));
  else
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsLaunch));
  if (warp == 1 && lane == 0) tc::mbar_wait(done, 0);  // also after a failure: no MMA in flight
  __syncwarp();
  if constexpr (kPair) {
    cluster_sync();  // no arrival or operand read of the other CTA is outstanding
  } else if (S > 1) {
    cluster_sync();
    // this CTA adds the parts of its share of the tokens, in the order of the ranks
    const int64_t row0 = row_of(tile0), t0 = tok_of(tile0);
    const uint32_t part = tc::smem_u32(base);
    const int n0 = (int)((int64_t)N * rank / S), n1 = (int)((int64_t)N * (rank + 1) / S);
    for (int i = n0 * 128 + tid; i < n1 * 128; i += kLinThreads) {
      float v = 0.f;
      for (uint32_t q = 0; q < S; ++q) v += ld_cluster_f32(part + i * 4, q);
      const int64_t tok = t0 + i / 128, rr = row0 + i % 128;
      if (tok < a.l.T && rr < a.l.m) {
        if (a.l.xscale) v *= __ldg(a.l.xscale + tok);
        if (a.l.y_bf16)
          static_cast<__nv_bfloat16*>(a.l.y)[tok * a.l.m + rr] = __float2bfloat16(v);
        else
          static_cast<float*>(a.l.y)[tok * a.l.m + rr] = v;
      }
    }
    cluster_sync();  // the parts stay until every CTA of the cluster has read them
  }
  __syncthreads();
  if (warp == 2) {
    if constexpr (kPair) tc::tmem_dealloc_pair(tmem, 2 * kN);
    else tc::tmem_dealloc(tmem, 2 * kN);
  }
}

namespace {
template <int B, int P, bool kPair>
cudaError_t launch_tc(const CUtensorMap& map, const CUtensorMap& cmap, const LinTcArgs& a, int vec,
                      int wide, int S, cudaStream_t s) {
  cudaLaunchConfig_t cfg{};
  // one CTA an SM (or a pair on two) takes tile after tile, or a cluster shares one
  const int ctas = kPair ? 2 * (a.tiles < kSMs / 2 ? a.tiles : kSMs / 2)
                         : S > 1 ? a.tiles * S : a.tiles < kSMs ? a.tiles : kSMs;
  cfg.gridDim = dim3((unsigned)ctas);
  cfg.blockDim = dim3(kLinThreads);
  cfg.dynamicSmemBytes = kLinSmem;
  cfg.stream = s;
  cudaLaunchAttribute at{};
  at.id = cudaLaunchAttributeClusterDimension;
  at.val.clusterDim.x = kPair ? 2 : (unsigned)S;
  at.val.clusterDim.y = at.val.clusterDim.z = 1;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, linear_tc_kernel<B, P, kPair>, map, cmap, a, vec, wide);
}
}  // namespace

template <int B>
cudaError_t linear_tc_bits(const CUtensorMap& map, const LinTcArgs& a, int P, bool pair, int vec,
                           int wide, int S, cudaStream_t s) {
  CUtensorMap cmap = map;  // the packed rows (pairs)
  if (pair) {
    const cudaError_t e = encode_tmap_2d(
        &cmap, CU_TENSOR_MAP_DATA_TYPE_UINT32, 4, a.l.codes, a.l.m, row_words(a.l.n, B),
        row_words(a.l.n, B), 4 * B, 128,
        B == 4 ? CU_TENSOR_MAP_SWIZZLE_64B
               : B == 8 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_NONE);
    if (e != cudaSuccess) return e;
  }
  if (P == 3)
    return pair ? launch_tc<B, 3, true>(map, cmap, a, vec, wide, S, s)
                : launch_tc<B, 3, false>(map, cmap, a, vec, wide, S, s);
  return pair ? launch_tc<B, 1, true>(map, cmap, a, vec, wide, S, s)
              : launch_tc<B, 1, false>(map, cmap, a, vec, wide, S, s);
}
namespace {
template <int B, int P, bool kPair>
cudaError_t init_one() {
  cudaError_t e = cudaFuncSetAttribute(linear_tc_kernel<B, P, kPair>,
                                       cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kLinSmem);
  if (e != cudaSuccess) return e;
  cudaFuncAttributes at;
  if ((e = cudaFuncGetAttributes(&at, linear_tc_kernel<B, P, kPair>))) return e;
  // the roles' register shares are what a launch of 96 registers a thread holds
  return at.numRegs > 88 && at.numRegs <= 96 ? cudaSuccess : cudaErrorInvalidConfiguration;
}
}  // namespace

template <int B>
cudaError_t linear_tc_clusters(int S, int* count) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)S);
  cfg.blockDim = dim3(kLinThreads);
  cfg.dynamicSmemBytes = kLinSmem;
  cudaLaunchAttribute at{};
  at.id = cudaLaunchAttributeClusterDimension;
  at.val.clusterDim.x = (unsigned)S;
  at.val.clusterDim.y = at.val.clusterDim.z = 1;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  return cudaOccupancyMaxActiveClusters(count, linear_tc_kernel<B, 1, false>, &cfg);
}

template <int B>
cudaError_t linear_tc_init() {
  cudaError_t e;
  if ((e = init_one<B, 3, false>())) return e;
  if ((e = init_one<B, 3, true>())) return e;
  if ((e = init_one<B, 1, false>())) return e;
  return init_one<B, 1, true>();
}


}  // namespace gq
