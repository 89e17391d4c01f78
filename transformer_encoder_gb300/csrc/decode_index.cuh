// decode_index.cuh -- the index and angle arithmetic of the decode-side kernels (append.cu, prefix_attn.cu,
// chunk_attn.cu, chunk_tc.cu, pages.cu), compiled for the host too: the wenc_selftest_* entries of api.cu replay it without a GPU.
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

// ------------------------------------------------------------------ keys of a run of tokens (chunk_attn.cu, chunk_tc.cu)
// The keys that tokens at positions first .. last of a sequence see between them, in steps of `step` keys: the leading n_first
// steps [0, step), .. for the first `sinks` keys, then the others from lo_step on (a multiple of `align`) up to the last
// token's own. Where the two meet they are one run (n_first 0, lo_step 0). Keys from `lo` on, and below `first`, are seen by
// some token.
struct KeySteps {
  int lo, hi, first;      // keys [lo, hi) and [0, first)
  int n_first, lo_step, n;

  KeySteps() = default;
  __host__ __device__ __forceinline__ KeySteps(int pos0, int pos1, int window, int sinks, int step, int align) {
    hi = pos1 + 1 > 0 ? pos1 + 1 : 0;
    const long long l = static_cast<long long>(pos0) + 1 - window;
    lo = l > 0 ? (l < hi ? static_cast<int>(l) : hi) : 0;
    first = sinks < lo ? sinks : lo;
    n_first = (first + step - 1) / step;
    lo_step = lo / align * align;
    if (lo_step <= static_cast<long long>(n_first) * step) n_first = lo_step = 0;
    n = n_first + (hi - lo_step + step - 1) / step;
  }
  __host__ __device__ __forceinline__ int key0(int t, int step) const { return t < n_first ? t * step : lo_step + (t - n_first) * step; }
  __host__ __device__ __forceinline__ bool seen(int key) const { return key < hi && (key >= lo || key < first); }
};

// ------------------------------------------------------------------ pages (pages.cu)
// The pages that n tokens take.
__host__ __device__ __forceinline__ int pages_of(int n, int page_size) {
  return static_cast<int>((static_cast<uint32_t>(n) + static_cast<uint32_t>(page_size) - 1u) / static_cast<uint32_t>(page_size));
}

// The table entries that a sequence of `len` tokens gives back, as ranges [x, y) and [z, w). `gone`: entries below it went
// back in earlier calls, but for the first `first` ones, which stay while the sequence does. A window (0: none) is past an
// entry when no later token sees any of its keys: the next one, at position len, sees those behind len - window. mark: the
// `gone` of the next call.
__host__ __device__ __forceinline__ int4 gives(int len, bool finished, int gone, int window, int first, int page_size, int& mark) {
  const int total = pages_of(len, page_size);
  const int low = first > gone ? first : gone;
  if (finished) {
    mark = 0;
    return make_int4(0, first < total ? first : total, low, total > low ? total : low);
  }
  const int end = window > 0 && len >= window ? (len - window + 1) / page_size : 0;
  mark = gone > end ? gone : end;
  return make_int4(0, 0, low, end > low ? end : low);
}

}  // namespace wenc_dev
