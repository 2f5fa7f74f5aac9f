// mhc_mxfp4_plan.h -- layout and launch interface of the microscaled 4-bit floats.
//
// Host-side and plain C++ (no HIP headers), like mhc_plan.h.
#pragma once

#include <cstddef>
#include <cstdint>

namespace mhc {
namespace mx {

constexpr int kBlock = 32;           // values per scale
constexpr int kMaxD = 65536;

// Bytes of a row's codes (whole blocks) and scales (whole words: the products read the scales of
// 128 values at a time).
inline int64_t code_bytes(int64_t D) { return (D + kBlock - 1) / kBlock * 16; }
inline int64_t scale_bytes(int64_t D) { return (D + 127) / 128 * 4; }

// Workgroups of 256 threads of eight values each, rows padded to whole words of scales, or -1 where that
// passes a grid's 2^32 - 1 threads.
inline int64_t octet_blocks(int64_t rows, int64_t D)
{
    const int64_t P = scale_bytes(D) * 4;
    if (rows > (int64_t)0xffffff * 256 / P) return -1;
    return (rows * P + 255) / 256;
}

// Implemented in mhc_mxfp4.hip. Each returns 0 or the HIP error code.
int launch_quantise(int64_t rows, int D, const uint16_t* x, uint8_t* codes, uint8_t* scales, int x_f16, void* stream);
int launch_restore(int64_t rows, int D, const uint8_t* codes, const uint8_t* scales, uint16_t* x, int x_f16, void* stream);

}  // namespace mx
}  // namespace mhc
