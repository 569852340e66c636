// gq_g4_vectors_bf16.hip -- gq_g4_matvec of bf16 vectors on the matrix cores (gfx950).
#include "gq_g4_vectors.h"

hipError_t gqk_g4_vectors_bf16(const G4Weights& w, const void* x, int batch, void* y, int y_dtype, hipStream_t s) {
    return gqg4::vectors<gqg4::XBf16>(w, x, batch, y, y_dtype, s);
}
