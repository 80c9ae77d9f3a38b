// The product of int8 rows: the kernels of product_dense.h and dense_stream.h, built apart from the others so
// that they compile side by side.
#include "dense_stream.h"
#include "product_dense.h"

namespace epdc {

hipError_t launch_dense_linear_int(const DenseParams &P, DenseForm form, bool out32, hipStream_t stream) {
    switch (form) {
    case kDenseStream16: return launch_stream<true, 1, 2, 3>(P, out32, stream);
    case kDenseStream64: return launch_stream<true, 4, 2, 2>(P, out32, stream);
    case kDenseTiles128: return launch_tiles<kDenseProduct, true, 128, 128>(P, out32, stream);
    case kDenseTiles256: return launch_tiles<kDenseProduct, true, 256, 256>(P, out32, stream);
    }
    return hipErrorInvalidValue;
}

}  // namespace epdc
