// gq_g4_vectors_f16.hip -- gq_g4_matvec of fp16 vectors on the matrix cores (gfx950).
#include "gq_g4_vectors.h"

hipError_t gqk_g4_vectors_f16(const G4Weights& w, const void* x, int batch, void* y, int y_dtype, hipStream_t s) {
    return gqg4::vectors<gqg4::XF16>(w, x, batch, y, y_dtype, s);
}
