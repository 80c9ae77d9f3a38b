// The gradient of the product's rows: the kernels of product_dense.h, built apart from the others so
// that they compile side by side.
#include "product_dense.h"

namespace epdc {

hipError_t launch_dense_rows_grad(const DenseParams &P, DenseForm form, bool out32, hipStream_t stream) {
    return form == kDenseTiles256 ? launch_tiles<kDenseRowsGrad, false, 256, 256>(P, out32, stream)
                                  : launch_tiles<kDenseRowsGrad, false, 128, 128>(P, out32, stream);
}

}  // namespace epdc
