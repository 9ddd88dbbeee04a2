// Kernels whose lanes hand values to one another without a workgroup's barrier: one
// instantiation of each, to be compiled to assembly.
#ifdef ROWS
#include "qsdp_rows.h"
template __global__ void onebit::k_qsdp_rows<onebit::kGradBF16, 4, 4, 1, 1, 2, 4>(onebit::LinearArgs);
template __global__ void onebit::k_qsdp_rows<onebit::kGradF16, 8, 1, 2, 2, 4, 2>(onebit::LinearArgs);
#else
#include "kvq_append.hip"
template __global__ void onebit::k_kvq_append<onebit::kGradBF16, 128, 8>(onebit::KvqAppendArgs);
#endif
