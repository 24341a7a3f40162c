// q4.cuh — the page format of a cache held in 4 bits, shared by the calls that write and read it.
//
// A page of one kv head is one record of bs * (D + 8 * D / group) bytes:
//   key codes [bs][D / 2], value codes [bs][D / 2],
//   key params [bs][D / group], value params [bs][D / group]
// Code d of a row is nibble d % 2 of byte d / 2; a param is a word, f16 scale below f16 zero; a value is
// scale * code + zero.  The 16-byte pieces (32 codes) of row t lie permuted, piece c at place
// c ^ piece_xor<D>(t): eight neighbouring rows then have any one piece in eight different
// 16-byte columns of shared memory's 128, and a record is copied there as it lies and read without
// bank conflicts.
#pragma once

#include <stdint.h>

namespace da {

constexpr int kQ4MinGroup = 32;

inline bool q4_group_ok(int group, int D) {
  return (group == 32 || group == 64 || group == 128) && group <= D;
}

__host__ __device__ constexpr long long q4_page_bytes(int bs, int D, int group) {
  return (long long)bs * (D + 8 * (D / group));
}

template <int D>
__device__ __forceinline__ int piece_xor(int t) {
  return (t / (256 / D)) & (D / 32 - 1);
}

}  // namespace da
