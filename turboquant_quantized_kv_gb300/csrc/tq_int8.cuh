// int8 layers of the cache: the page, and codes as fp16 operands (libtq, sm_103a).
//
// A page is one block of one KV head: 16 records of 128 bytes, byte = code + 128, then the tail
// {fp32 step, uint32 bits of the tokens that hold a coordinate that is not finite, 8 bytes that an
// append uses while it runs}.  A value is code * step, |code| <= 127.
#pragma once

#include "tq_device.cuh"
#include "tq_internal.h"

namespace tq {

constexpr int kI8Codes = kBlock * kD;          // bytes of a page's records
constexpr int kI8Page = kI8Codes + 16;         // and of a page
constexpr float kI8Least = 1.1754943508222875e-38f;  // 2^-126, the least step

// Sequences with more rows (tokens x query heads of a KV head) than this go through the tiles of
// tq_int8_attend.cu, the others through the decode kernel, which reads the pages once for each eight rows, so the rule
// ends with a unit of eight.  By the decode kernel / by the tiles, us a call, 8 KV heads in groups of four:
//                          16 rows      24 rows      32 rows
//   1 sequence  of 30,000   48 /  93     56 / 102     64 / 109
//   4           of 30,000  126 / 153    146 / 154    203 / 158
//   8           of  1,000   32 /  60     35 /  60     39 /  62
//   16          of  8,000  118 / 162    169 / 164    208 / 166
//   24          of  3,000   83 / 124    105 / 124    133 / 124
//   64          of    200   43 /  87     49 /  88     56 /  89
//   64          of  8,000  378 / 461    550 / 462    707 / 468
// (Many long contexts would want the tiles from 17 rows on, few or short ones not at 32: the host knows the tables'
// widths, not the lengths.)
constexpr int kAttRows = 24;
constexpr int kAttMostGroup = 256;  // query heads of a KV head, with more of them every sequence does the latter

// Counters of a call in its workspace: the decode kernel's from 0 on, the tiles' from here on, one a CTA.
constexpr int kAttCounters = 8192;
static_assert(2 * kAttCounters * sizeof(int) <= kCounterRegionBytes, "the counter region");

struct I8Tail {
  float step;
  uint32_t bad;       // bit r: record r is not a number
  uint32_t marks;     // (append) bit r: record r is written by this call
  uint32_t first;     // (append) the least key of this call's tokens in the block
};

// Bytes lo and hi of w as two fp16 codes: the byte under the exponent of 1024 is 1024 + byte, exactly, and
// 1024 + 128 comes off again.  `sel`: 0x4140 for bytes 0 and 1, 0x4342 for bytes 2 and 3.
__device__ __forceinline__ uint32_t i8_pair(uint32_t w, uint32_t sel) {
  const uint32_t u = prmt(w, 0x64646464u, sel);
  const __half2 h = __hsub2(*reinterpret_cast<const __half2*>(&u), __half2half2(__ushort_as_half((unsigned short)0x6480u)));
  return *reinterpret_cast<const uint32_t*>(&h);
}

// The sequences of a call that take tiles (the rest of the call is launch_int8_attend's).
cudaError_t launch_int8_tiles(const AttendCall& c, uint8_t* partials, int num_sms, cudaStream_t st);

}  // namespace tq
