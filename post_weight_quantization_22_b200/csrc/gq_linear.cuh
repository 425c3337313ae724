// What the parts of the packed products share: the dispatcher (gq_linear.cu) and, once per code
// width, the kernels (gq_linear_bits.cu).
#pragma once
#include "gq_internal.cuh"

namespace gq {

constexpr int kSMs = 148;
constexpr int kCols = 64;  // columns per stage of the tcgen05 kernel's ring

struct LinTcArgs {
  LinearArgs l;
  int planes_t;      // rows between two parts of the tokens (0 with one part)
  int N;             // tokens per tile
  int mtiles;        // tiles of 128 rows (pairs: 256)
  int tiles;         // tiles of rows and tokens
  int stages;        // stages of kCols columns
  int gshift;        // log2 of the group width (31: one grid per row, every index is 0)
  int dmask;         // 16-column steps per accumulator period (a power of two) - 1
  int groups;        // groups of a row
  WsHeader* hdr;
  WsHeader* device_hdr;  // the device's own status: kept until it is looked at
  WaitTest wait;     // budget of the kernel's waits (test setting)
};

// The kernels for codes of B bits.  rows: the warp-level product (xvec: inputs allow vector
// loads).  tc: the tcgen05 product; S CTAs share a tile's columns; vec: the packed rows allow
// 16-byte loads; wide: rows of y are on 16-byte boundaries.
template <int B>
void linear_rows_bits(const LinearArgs& a, LinearInput kind, int xvec, cudaStream_t s);
template <int B>
cudaError_t linear_tc_bits(const CUtensorMap& map, const LinTcArgs& a, int P, bool pair, int vec,
                           int wide, int S, cudaStream_t s);
template <int B>
cudaError_t linear_tc_init();
// How many clusters of S CTAs of the single form the current device runs at once.
template <int B>
cudaError_t linear_tc_clusters(int S, int* count);

}  // namespace gq
