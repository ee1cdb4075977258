// kv4.cuh -- layout of the 4-bit paged cache, shared by its kernels.
//
// A row (one token, one head, K or V; 64 values) is held as 64 unsigned 4-bit
// codes c and two bf16 numbers s, z; code c stands for s * c + z.  z is the
// row's minimum (a bf16 input, so exact) and s = (max - min) / 15 rounded up
// to bf16, so all 64 values lie within s / 2 (and 2^-19 s for the differences,
// which are taken in fp32) of what their code stands for.
//
// Rows are grouped into records of 16 tokens of one KV head, the unit every
// kernel moves and computes on:
//   bytes    0.. 511  K codes, 32 bytes a token (dimension d: byte d / 2, the
//                     even dimension in the low half)
//   bytes  512..1023  V codes
//   bytes 1024..1087  K (s, z), 4 bytes a token
//   bytes 1088..1151  V (s, z)
// A block of bs tokens is bs / 16 groups of Hkv records, group after group:
// any run of 16-token groups is one contiguous run of bytes for all heads (one
// bulk copy), whatever the block size.  72 bytes a token and head, 4.5 bits a
// value, against 256 bytes in bf16.
#pragma once

#include <cstdint>

namespace tvl {

constexpr int kRecTokens = 16;
constexpr int kRecBytes = 1152;
constexpr int kRecV = 512;        // V codes
constexpr int kRecKMeta = 1024;   // K (s, z)
constexpr int kRecVMeta = 1088;   // V (s, z)
constexpr int kRowCodes = 32;     // bytes of codes in a row

}  // namespace tvl
