// Four more bits of a float32 that is stored as bf16, host and device.
//
// With x the float's bits and hi those of its rounding to bf16, to the nearest and on a tie
// to the even number (lower half 0), x - hi lies in -2^15 .. 2^15: the code is its
// multiple of 2^12, -8 .. 7, and stands for the middle of that interval, so a float is
// off by at most 2^11 of its last bits, 2^-12 of itself.  Those are x's bits 12 .. 15, but
// for a tie that went down, whose 2^15 counts to the interval below it (off by 2^11 as
// well): bits 0 .. 16 tell it from one that went up.  x - hi is negative only where the
// rounding went up, so that hi is not 0 and nothing wraps around.  NaN stays NaN with any
// code; infinity becomes one, as it does in the products of split operands.
#pragma once

#include <hip/hip_runtime.h>

namespace gdr {

// the code, in four bits
__host__ __device__ inline unsigned kept_code(unsigned x) {
    return (x - ((x & 0x1ffffu) == 0x8000u ? 1u : 0u)) >> 12 & 15u;
}
// the bits of the float: hi, and the i-th code of a word
__host__ __device__ inline unsigned kept_bits(unsigned hi, unsigned word, int i) {
    const int code = (int)(word << (28 - 4 * i)) >> 28;
    return (hi | 0x800u) + ((unsigned)code << 12);
}

}  // namespace gdr
