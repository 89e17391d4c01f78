// decode_index.cuh -- the index and angle arithmetic of the decode-side kernels (append.cu, prefix_attn.cu), compiled for
// the host too: the wenc_selftest_* entries of api.cu replay it without a GPU.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include <cmath>

namespace wenc_dev {

// ------------------------------------------------------------------ angles (append.cu)
// 2^64 * frac(f / 2 pi): the turns a position advances the angle by, as a 64-bit fraction.
// 1 / 2 pi = c1 + c2 with c1 of 29 bits, so f * c1 is exact in double. The fraction is taken of |f|:
// of a negative number, x - floor(x) = 1 - |x| would drop the bits of |x| below 2^-54, and a position
// of 31 bits carries those up to 2^-23 of a turn.
__host__ __device__ __forceinline__ unsigned long long turns64(float f) {
  const double c1 = 0x1.45f306dp-3, c2 = 0x1.9391054a7f09dp-32;
  double hi = fabs(static_cast<double>(f)) * c1, lo = fabs(static_cast<double>(f)) * c2;
  hi -= floor(hi);
  // hi in [0, 1): in two 32-bit parts (a conversion of hi * 2^64 could reach 2^64)
  const double h32 = hi * 4294967296.0;
  const unsigned long long top = static_cast<unsigned long long>(h32);
  const unsigned long long low = static_cast<unsigned long long>((h32 - static_cast<double>(top)) * 4294967296.0);
  lo -= floor(lo);
  const double l32 = lo * 4294967296.0;
  const unsigned long long ltop = static_cast<unsigned long long>(l32);
  const unsigned long long llow = static_cast<unsigned long long>((l32 - static_cast<double>(ltop)) * 4294967296.0);
  const unsigned long long turn = (top << 32) + low + (ltop << 32) + llow;
  return f < 0.0f ? 0ull - turn : turn;
}

// The angle of position `at` at `step` turns a position, as pi h + l: h holds its leading 24 bits, exactly, in
// [-1, 1), and l < 2^-21 the next 32.
__host__ __device__ __forceinline__ void angle_parts(int at, unsigned long long step, float& h, float& l) {
  const long long turn = static_cast<long long>(static_cast<unsigned long long>(static_cast<long long>(at)) * step);
  h = static_cast<float>(static_cast<int>(turn >> 32) & ~0xff) * 0x1p-31f;
  l = static_cast<float>(static_cast<uint32_t>(turn >> 8)) * (3.14159265f * 0x1p-55f);
}

// ------------------------------------------------------------------ a token's sequence (append.cu)
// The last index i with start[i] <= t among 0 .. n - 1 (-1: none), 32 probes a step. hits(lo, step, len) counts
// the probes i = 0 .. 31 with i * step < len and start[lo + i * step] <= t. Offsets that do not ascend give some index,
// and no probe outside the array.
template <class Hits>
__host__ __device__ __forceinline__ int last_start(int n, const Hits& hits) {
  int lo = 0, len = n;  // the answer + 1 lies in [lo, lo + len]
  while (len > 0) {
    const int step = (len - 1) / 32 + 1;
    const int h = hits(lo, step, len);
    if (h == 0) return lo - 1;
    const int base = (h - 1) * step;  // start[lo + base] <= t, and the next probe is not
    const int rest = (step < len - base ? step : len - base) - 1;
    lo += base + 1;
    len = rest;
  }
  return lo - 1;
}

// The sequence of row t of n_rows, at or behind sequence s (as last_start gives it for a row at or before t): 0 .. n_seqs -
// 1, and how many rows `left` it has from t on; n_seqs for a row behind the last sequence; -1 where the offsets are out of
// range.
__host__ __device__ __forceinline__ int sequence_of(const int32_t* start, int n_seqs, int n_rows, int t, int s, int& left) {
  left = 0;
  if (s < 0) return -1;  // (offsets that do not start at 0)
  while (s < n_seqs && start[s + 1] <= t) ++s;
  if (start[s] > t) return -1;  // (offsets that do not ascend)
  if (s < n_seqs) {
    if (start[s + 1] > n_rows) return -1;  // (a sequence that ends behind the rows: where they go would be wrong)
    left = start[s + 1] - t;
  }
  return s;
}

// ------------------------------------------------------------------ runs of key steps (prefix_attn.cu)
// Share `part` of `parts` equal runs of n steps.
__host__ __device__ __forceinline__ void run_of(int n, int part, int parts, int& first, int& count) {
  const int per = (n + parts - 1) / parts;
  first = part * per;
  const int left = n - first;
  count = left < 0 ? 0 : left < per ? left : per;
}

// The segment of step t, at or behind segment sg: step0 holds each segment's first step, and the end.
__host__ __device__ __forceinline__ int segment_of(const int* step0, int t, int sg) {
  while (t >= step0[sg + 1]) ++sg;
  return sg;
}

}  // namespace wenc_dev
