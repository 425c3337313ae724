// The packed products' kernels for one code width; compiled once for every width from 2 to 8
// (GQ_LINEAR_BITS), so that the widths compile side by side.
#include "gq_linear_rows.cuh"
#include "gq_linear_tc.cuh"

#ifndef GQ_LINEAR_BITS
#define GQ_LINEAR_BITS 4
#endif

namespace gq {
template void linear_rows_bits<GQ_LINEAR_BITS>(const LinearArgs&, LinearInput, int, cudaStream_t);
template cudaError_t linear_tc_bits<GQ_LINEAR_BITS>(const CUtensorMap&, const LinTcArgs&, int, bool,
                                                    int, int, int, cudaStream_t);
template cudaError_t linear_tc_init<GQ_LINEAR_BITS>();
template cudaError_t linear_tc_clusters<GQ_LINEAR_BITS>(int, int*);
}  // namespace gq
