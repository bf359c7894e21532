// The kernel for few query rows whose queries come in two addends (pa_quant_rows.cuh).
#include "pa_quant_rows.cuh"

namespace pa {
namespace quant {
namespace rows {

template cudaError_t launch_rows_kernel<true>(const Geometry&, const QuantArgs&, const DecP&, int,
                                              int, int);

}  // namespace rows
}  // namespace quant
}  // namespace pa
