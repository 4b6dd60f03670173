// Scalar offsets of buffer loads, apart from the device code so that the host can check them.
//
// The range check compares a lane's offset with the buffer's size minus the scalar offset.
// That is defined while the scalar offset is at most the size (at the size no lane passes),
// so no load has a larger one, whichever rows and steps it is for.
#pragma once

#include <stdint.h>

#ifdef __HIP__
#define FP8W_OFFSET __host__ __device__ __forceinline__
#else
#define FP8W_OFFSET inline
#endif

namespace fp8w {

// `off` bytes into a buffer of `bytes`; its end for a load that is not on, or starts behind it.
FP8W_OFFSET int buffer_offset(bool on, int off, int bytes)
{
    return on && off < bytes ? off : bytes;
}

// Row `row` of a buffer of rows, `off` bytes into it.
FP8W_OFFSET int buffer_offset(bool on, int off, int row, int row_bytes, int bytes)
{
    return buffer_offset(on, off + row * row_bytes, bytes);
}

}  // namespace fp8w
