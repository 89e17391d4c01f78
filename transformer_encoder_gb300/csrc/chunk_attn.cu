// chunk_attn.cu -- attention of chunks of new tokens over a paged cache, with an optional sliding window and first tokens that
// stay visible.
//
// Each sequence of the call brings as many tokens as it likes: one in a decode step, a few as a draft, hundreds of a prompt. Token
// i of the m that a sequence of len keys brings stands at p = len - m + i, and query head h reads key head h / (H / Hkv):
//   out = softmax(scale * q . K_seen) V_seen,   seen: keys j <= p with j > p - window or j < sinks
// (inferencelayer 0.2.4 src/whisper_gpu.rs, DEC_QATTN; oxinfer 0.0.5 src/whisper/model.rs, attention_masked).
//
// A cluster of 1 to 8 CTAs attends one item: a tile of 8 NR rows (token, query head) of one sequence and key head. The keys
// that some row of the tile sees (KeySteps) are cut into steps of 16, of which every warp of the cluster takes an equal run; a
// warp has a ring of cp.async stages of its own, with its keys' pages looked up a step ahead, and no barrier with other warps
// until their results are joined: through shared memory, and between CTAs through distributed shared memory. Only steps at the
// borders of what the rows see are masked (attend.cuh has the steps' arithmetic).
// What bounds it: the bytes of K and V (each read once for a tile's rows), and at small calls the latency of getting at them.
// Measured on the device: 80 single tokens of 20 heads, each behind 1500 keys of a window and 4 first ones (606 MB), 100 us,
// 6.0 TB/s (6.8: a plain copy); one token of 6 heads behind 452 keys 5.7 us; fp32, up to 33 tokens of 24 sequences, 8 heads,
// windows of 500, 21 us: there latency, at 8 warps an SM (255 registers; they issue in 34% of the cycles, the tensor pipe is
// busy in 30%).
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <math_constants.h>

#include <atomic>
#include <cstdio>
#include <string>

#include "attend.cuh"
#include "chunk.cuh"
#include "decode_index.cuh"
#include "launch.h"
#include "ptx.cuh"
#include "wenc.h"

wenc_status wenc_internal_fail(wenc_status s, const char* msg);
void wenc_internal_clear_error();
int wenc_internal_sm_count();
wenc_status wenc_internal_device(int* sms, uint32_t** err);

namespace {

using namespace wenc_dev;
using wenc_host::Range;
using wenc_host::share;
using wenc_host::table_bytes;

constexpr int HD = 64;

struct RowsPlan {
  int tiles;    // row tiles per sequence; 0: the sequences' tiles one after another (found by a search)
  int most;     // sequences with more rows per key head belong to another launch
  int cluster;  // CTAs per item
};

// The sequence and tile that are number t of all sequences' tiles of `rows` rows; by all lanes of a warp.
__device__ __forceinline__ bool find_tile(const ChunkParams& p, const RowsPlan& pl, int rows, int t, int& seq, int& tile, uint32_t* err) {
  const int lane = threadIdx.x & 31;
  for (int s0 = 0; s0 < p.n_seqs; s0 += 32) {
    const int s = s0 + lane;
    int m = 0;
    if (s < p.n_seqs) m = p.per_seq;
    if (s < p.n_seqs && p.seq_start) m = chunk_tokens(p, p.seq_start[s], p.seq_start[s + 1], err);
    const int n = m * p.r <= pl.most ? (m * p.r + rows - 1) / rows : 0;
    int sum = n;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int up = __shfl_up_sync(0xffffffffu, sum, d);
      if (lane >= d) sum += up;
    }
    const uint32_t past = __ballot_sync(0xffffffffu, t < sum);
    if (past) {
      const int at = __ffs(past) - 1;
      seq = s0 + at;
      tile = t - __shfl_sync(0xffffffffu, sum - n, at);
      return true;
    }
    t -= __shfl_sync(0xffffffffu, sum, 31);
  }
  return false;
}

template <typename T, int NR>
__global__ void __launch_bounds__(Cfg<T, NR>::THREADS, NR == 4 ? 1 : Cfg<T, NR>::CTAS)
    chunk_rows_kernel(const __grid_constant__ ChunkParams p, const RowsPlan pl, uint32_t* err) {
  using C = Cfg<T, NR>;
  constexpr bool F32 = C::F32;
  constexpr int KW = C::KW, ST = C::STAGES;
  constexpr int CH = C::ROWB / 16;  // granules per row
  constexpr int RPI = 32 / CH;      // rows a warp's copy instruction covers
  constexpr int NL = KW / RPI;
  constexpr int KS = F32 ? 8 : 4;
  extern __shared__ __align__(128) uint8_t smem[];
  pdl_trigger();
  pdl_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, tq = lane & 3;
  const int rank = blockIdx.x % pl.cluster;
  int b = blockIdx.x / pl.cluster;
  const int hk = b % p.Hkv;
  b /= p.Hkv;
  int seq, tile;
  if (pl.tiles > 0) {
    tile = b % pl.tiles;
    seq = b / pl.tiles;
  } else if (!find_tile(p, pl, C::ROWS, b, seq, tile, err)) {
    return;  // the whole cluster
  }
  const ChunkSeq sq = chunk_seq(p, seq, err);
  const int row0 = tile * C::ROWS, n_rows = sq.m * p.r <= pl.most ? min(sq.m * p.r - row0, C::ROWS) : 0;
  if (n_rows <= 0) return;  // the whole cluster
  const int pos0 = sq.len - sq.m;  // of the sequence's first token
  const int first = pos0 + row0 / p.r, last = pos0 + (row0 + n_rows - 1) / p.r;
  const KeySteps ks(first, last, p.window, p.sinks, KW, KW);
  int step0, n_mine;
  run_of(ks.n, rank * C::NW + warp, pl.cluster * C::NW, step0, n_mine);

  // ---- loads of a step: 16 keys and values. Addresses in units of 16 bytes (32-bit factors, 64-bit sums). Rows RPI i + lr
  // of a stage: two swizzled positions alternate with i.
  const uint32_t s0 = smem_u32(smem) + warp * (ST * 2 * C::HALF);
  const int lc = lane % CH, lr = lane / CH;
  const uint32_t at0 = granule<F32>(lr, lc), at1 = granule<F32>(lr + RPI, lc) - 512u;
  static_assert(RPI * C::ROWB == 512, "a copy instruction covers 512 bytes of a stage");
  const int32_t* table = p.table + seq * p.table_stride;
  int next_page = 0;  // page of the key in the next step's row lane % 16, read one step ahead
  auto page_of = [&](int j) {
    const int key = ks.key0(step0 + j, KW) + (lane & 15);
    const int pi = p.page_shift >= 0 ? key >> p.page_shift : key / p.page_size;
    next_page = ks.seen(key) && in_bounds(pi >= 0 && pi < p.max_pages, err, 118) ? table[pi] : -1;
  };
  auto load = [&](int j, int stage) {
    const uint32_t sk = s0 + stage * (2 * C::HALF), sv = sk + C::HALF;
    const int key = ks.key0(step0 + j, KW) + (lane & 15);
    const int pi = p.page_shift >= 0 ? key >> p.page_shift : key / p.page_size;
    const bool in = static_cast<uint32_t>(next_page) < static_cast<uint32_t>(p.n_pages);
    if (!in && ks.seen(key)) *reinterpret_cast<volatile uint32_t*>(err) = kErrData | (80u << 8);
    const int page = in ? next_page : -1;
    const uint32_t slot = (key - pi * p.page_size) * p.row16, head = hk * CH + lc;
#pragma unroll
    for (int i = 0; i < NL; ++i) {
      const int pg = __shfl_sync(0xffffffffu, page, lr + i * RPI);
      const uint32_t x = __shfl_sync(0xffffffffu, slot, lr + i * RPI) + head;
      const bool ok = pg >= 0;
      const uint32_t upg = ok ? pg : 0, at = ((i & 1) ? at1 : at0) + i * 512;
      cp_async16(sk + at, p.k_pages + ((static_cast<uint64_t>(upg) * p.k_page16 + (ok ? x : 0)) << 4), ok);
      cp_async16(sv + at, p.v_pages + ((static_cast<uint64_t>(upg) * p.v_page16 + (ok ? x : 0)) << 4), ok);
    }
  };
  if (n_mine > 0) page_of(0);
#pragma unroll
  for (int j = 0; j < ST - 1; ++j) {
    if (j < n_mine) {
      load(j, j);
      if (j + 1 < n_mine) page_of(j + 1);
    }
    cp_async_commit();
  }

  // ---- the query rows as B fragments (column g of group r: row 8 r + g)
  uint32_t qh[NR][KS][2], ql[F32 ? NR : 1][KS][2];
#pragma unroll
  for (int r = 0; r < NR; ++r) {
    const int x = row0 + 8 * r + g, tok = x / p.r, head = hk * p.r + x - tok * p.r;
    const long long token = static_cast<long long>(sq.row0) + tok;
    const bool in = 8 * r + g < n_rows && in_bounds(token >= 0 && token < p.n_tokens && head < p.H, err, 119);
    load_query<T>(in ? p.q + token * p.q_stride + head * C::ROWB : nullptr, tq, p.q_keep, p.q_flip, qh[r], ql[F32 ? r : 0]);
  }
  // the positions of this thread's columns of S^T and O^T: rows 8 r + 2 tq + e
  int pos_of[NR][2];
#pragma unroll
  for (int r = 0; r < NR; ++r)
#pragma unroll
    for (int e = 0; e < 2; ++e) pos_of[r][e] = pos0 + (row0 + 8 * r + 2 * tq + e) / p.r;

  RowState<NR> st;
  float u[NR][2];
  clear_rows(st, u);
  for (int j = 0; j < n_mine; ++j) {
    cp_async_wait<ST - 2>();
    __syncwarp();
    if (j + ST - 1 < n_mine) {
      load(j + ST - 1, (j + ST - 1) % ST);
      if (j + ST < n_mine) page_of(j + ST);
    }
    cp_async_commit();
    const int key0 = ks.key0(step0 + j, KW);
    const uint32_t sk = s0 + (j % ST) * (2 * C::HALF), sv = sk + C::HALF;
    float s[NR][4];
    step_scores<T, NR>(sk, qh, ql, s);
    if (key0 + KW - 1 > first || (key0 <= last - p.window && key0 + KW > p.sinks)) {
#pragma unroll
      for (int r = 0; r < NR; ++r)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int key = key0 + g + 8 * (e >> 1), pos = pos_of[r][e & 1];
          if (key > pos || (key <= pos - p.window && key >= p.sinks)) s[r][e] = -CUDART_INF_F;
        }
    }
    step_values<T, NR>(s, p.scale_log2, sv, smem_u32(smem) + C::RING + warp * (NR * 512), st, u);
  }
  cp_async_wait<0>();
  sum_rows(st);
  share_results<T, NR>(smem, st);

  const int x = threadIdx.x >> 3, c8 = (threadIdx.x & 7) * 8;  // 8 threads a row, 8 elements each
  static_assert(C::THREADS / 8 >= C::ROWS, "a row's threads");
  // row y of the tile (all lanes of a warp call; rows from n_rows on are not written)
  auto put = [&](int y, float (&v)[8], float l) {
    const int z = row0 + y, tok = z / p.r, head = hk * p.r + z - tok * p.r;
    const bool in = y < n_rows && in_bounds(head < p.H && sq.row0 + tok < p.n_tokens, err, 120);
    if (__any_sync(0xffffffffu, in && !chunk_numbers(v, l, pos0 + tok))) {
      float vc[8], lc = l;
#pragma unroll
      for (int e = 0; e < 8; ++e) vc[e] = v[e];
      chunk_redo<T>(p, seq, hk, p.q + static_cast<long long>(sq.row0 + tok) * p.q_stride + head * C::ROWB, pos0 + tok, in,
                    ks.lo, ks.hi, ks.first, c8, vc, &lc, err);
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = vc[e];
      l = lc;
    }
    if (in) chunk_write8<T>(p, sq.row0 + tok, head, c8, v, l, err);
  };
  float v[8], m, l;
  if (x < C::ROWS) join_warps<T, NR>(smem, x, c8, v, m, l);  // (whole warps)
  if (pl.cluster == 1) {
    if (x < C::ROWS) put(x, v, l);
    return;
  }
  // the CTAs' results over the first warp's; then the ranks share the rows out
  __syncthreads();
  const uint32_t so = smem_u32(smem), sml = so + C::ML;
  if (x < C::ROWS) {
    float4* d = reinterpret_cast<float4*>(smem + (x * C::OS + c8) * 4);
    d[0] = make_float4(v[0], v[1], v[2], v[3]);
    d[1] = make_float4(v[4], v[5], v[6], v[7]);
    if (c8 == 0) *reinterpret_cast<float2*>(smem + C::ML + x * 8) = make_float2(m, l);
  }
  cluster_arrive_wait();
  const int y = rank + pl.cluster * x;
  if (__any_sync(0xffffffffu, y < n_rows)) {
    const int at = min(y, C::ROWS - 1);
    float2 ml[8];
    m = -CUDART_INF_F;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if (i < pl.cluster) {
        ml[i] = ld_cluster_f2(rank_addr(sml + at * 8, i));
        m = fmaxf(m, ml[i].x);
      }
    }
    const float ref = m == -CUDART_INF_F ? 0.0f : m;
    l = 0.0f;
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if (i < pl.cluster) {
        const float f = ex2_approx(ml[i].x - ref);
        const uint32_t a = rank_addr(so + (at * C::OS + c8) * 4, i);
        const float4 o0 = ld_cluster_f4(a), o1 = ld_cluster_f4(a + 16);
        l += f * ml[i].y;
        v[0] += f * o0.x; v[1] += f * o0.y; v[2] += f * o0.z; v[3] += f * o0.w;
        v[4] += f * o1.x; v[5] += f * o1.y; v[6] += f * o1.z; v[7] += f * o1.w;
      }
    }
    put(y, v, l);
  }
  cluster_arrive_wait();  // no CTA leaves while another reads its results
}

wenc_status bad(wenc_status s, const char* fmt, long long a = 0, long long b = 0) {
  char buf[256];
  snprintf(buf, sizeof(buf), fmt, a, b);
  return wenc_internal_fail(s, buf);
}

// How a call is divided.
struct Plan {
  int nr = 0;              // groups of 8 rows per tile
  RowsPlan rows = {};
  long long blocks = 0;
  bool tc = false;         // sequences with more than rows.most rows per key head go to chunk_tc.cu
  size_t bytes = 0;
};

// bf16: up to kLeastTc rows per key head, and calls of up to kLittle pairs of a query row and a key that they may have, are
// attended here, in tiles of up to 32 rows. Other calls leave sequences of more than kFew rows to chunk_tc.cu, and take tiles
// of 16 for the rest. Measured (us, here / there with its three launches): 40 rows of each of 32 sequences, 4 key heads, 3000
// keys 28 / 52; 8 heads, 1 x 256 tokens behind 256 (0.8 M pairs) 17 / 26, 2 x 256 behind 1000 (4.6 M) 23 / 27, 8 x 256 behind
// 256 (6.3 M) 31 / 29, 16 x 100 behind 500 (7 M) 38 / 30; 20 heads over 4, 128 tokens behind 2000 (5.3 M) 29 / 28, behind 8000
// 71 / 35. The host knows the block table's width, not the lengths: with a table for 32 thousand keys the first of these calls,
// and any other whose caches are much shorter than its table, goes there.
constexpr int kFew = 16, kLeastTc = 64;
constexpr long long kLittle = 1ll << 22;
// Sequences up to which a call may take chunk_tc.cu's kernel: a warp of it looks for the next sequence with work, 32 of them in
// about a microsecond, while others wait under their limit of a second (2^20: some 30 ms).
constexpr int kMostWalked = 1 << 20;

Plan make_plan(const wenc_chunk_attention_args* a, int sms) {
  Plan pl;
  const bool f32 = a->dtype == WENC_DTYPE_F32;
  const long long r = a->n_heads / a->n_kv_heads;
  // (without offsets every sequence's tokens are known, whatever bound was given)
  const int max_new = a->seq_start ? a->max_new : a->n_tokens / a->n_seqs;
  long long most = static_cast<long long>(max_new) * r;
  const long long cap = static_cast<long long>(a->max_pages) * a->page_size;
  const long long in_window = a->window > 0 ? static_cast<long long>(a->window) + a->sinks + max_new : cap, seen = in_window < cap ? in_window : cap;
  if (!f32 && r <= 128 && a->scale > 0.0f && most > kLeastTc && a->n_seqs <= kMostWalked &&
      static_cast<long long>(a->n_tokens) * a->n_heads > kLittle / seen) {
    pl.tc = true;
    pl.bytes = wenc_host::chunk_tc_workspace(sms);
    most = kFew;
  }
  pl.nr = most <= 8 ? 1 : most <= 16 || f32 ? 2 : 4;
  const long long rows = 8 * pl.nr;
  pl.rows.most = static_cast<int>(most);
  // tiles: every sequence's largest number, or, where that leaves many empty, one after another
  const long long each = (most + rows - 1) / rows, dense = a->n_seqs + static_cast<long long>(a->n_tokens) * r / rows;
  const bool search = a->n_seqs * each > 2 * dense;
  pl.rows.tiles = search ? 0 : static_cast<int>(each);
  const long long items = (search ? dense : a->n_seqs * each) * a->n_kv_heads;
  // CTAs within two rounds of the machine (lengths differ, and a round that is full waits for its longest), none without steps
  // for its warps
  const long long kt = f32 ? 64 : 128, key_tiles = (seen + kt - 1) / kt;
  const long long round = (f32 || pl.nr == 1 ? 3ll : pl.nr == 2 ? 2ll : 1ll) * sms;
  pl.rows.cluster = 1;
  while (pl.rows.cluster < 8 && pl.rows.cluster < key_tiles && items * pl.rows.cluster <= round) pl.rows.cluster *= 2;
  pl.blocks = items * pl.rows.cluster;
  return pl;
}

// Whether n rows of `row` bytes at x and at y share none: apart as wholes, or, at one stride, side by side within it.
bool apart(const void* x, long long x_stride, const void* y, long long y_stride, long long row, long long n) {
  const long long a = static_cast<long long>(reinterpret_cast<uintptr_t>(x)), b = static_cast<long long>(reinterpret_cast<uintptr_t>(y));
  if (a + (n - 1) * x_stride + row <= b || b + (n - 1) * y_stride + row <= a) return true;
  if (x_stride != y_stride) return false;
  const long long d = ((b - a) % x_stride + x_stride) % x_stride;
  return d >= row && x_stride - d >= row;
}

constexpr float kLog2e = 1.4426950408889634f;

bool check_sizes(const wenc_chunk_attention_args* a, wenc_status* st) {
  auto no = [&](wenc_status s) {
    *st = s;
    return false;
  };
  if (!a) return no(bad(WENC_ERR_INVALID_ARG, "chunk_attention: args is NULL"));
  if (a->dtype != WENC_DTYPE_F32 && a->dtype != WENC_DTYPE_BF16)
    return no(bad(WENC_ERR_INVALID_ARG, "chunk_attention: dtype %lld unknown", a->dtype));
  if (a->head_dim != HD) return no(bad(WENC_ERR_UNSUPPORTED, "head_dim %lld: only 64 is implemented", a->head_dim));
  if (a->n_seqs < 1 || a->n_tokens < 0 || a->n_heads < 1 || a->n_kv_heads < 1 || a->n_pages < 1 || a->page_size < 1 || a->max_pages < 1)
    return no(bad(WENC_ERR_INVALID_ARG, "chunk_attention: sizes must be positive (n_tokens may be 0)"));
  if (a->n_tokens > 0 && (a->max_new < 1 || a->max_new > a->n_tokens))
    return no(bad(WENC_ERR_INVALID_ARG, "chunk_attention: max_new %lld must be 1..n_tokens (%lld)", a->max_new, a->n_tokens));
  if (!a->seq_start && a->n_tokens % a->n_seqs != 0)
    return no(bad(WENC_ERR_INVALID_ARG, "chunk_attention: %lld tokens are no multiple of %lld sequences (pass seq_start)", a->n_tokens,
                  a->n_seqs));
  if (!a->seq_start && a->n_tokens > 0 && a->max_new < a->n_tokens / a->n_seqs)
    return no(bad(WENC_ERR_INVALID_ARG, "chunk_attention: max_new %lld is less than the %lld tokens of each sequence", a->max_new,
                  a->n_tokens / a->n_seqs));
  if (a->n_heads % a->n_kv_heads != 0)
    return no(bad(WENC_ERR_INVALID_ARG, "n_heads %lld must be a multiple of n_kv_heads %lld", a->n_heads, a->n_kv_heads));
  if (a->n_heads > 4096) return no(bad(WENC_ERR_UNSUPPORTED, "chunk_attention: more than 4096 heads"));
  if (a->window < 0 || a->sinks < 0) return no(bad(WENC_ERR_INVALID_ARG, "chunk_attention: window or sinks is negative"));
  if (a->sinks > 0 && a->window == 0) return no(bad(WENC_ERR_INVALID_ARG, "chunk_attention: sinks go with a window"));
  if (static_cast<long long>(a->max_pages) * a->page_size > 1ll << 30)
    return no(bad(WENC_ERR_UNSUPPORTED, "chunk_attention: max_pages %lld x page_size %lld passes 2^30", a->max_pages, a->page_size));
  if ((static_cast<long long>(a->n_tokens) + a->n_seqs) * a->n_heads > 0x3fffffffll)
    return no(bad(WENC_ERR_UNSUPPORTED, "chunk_attention: %lld tokens of %lld heads are too many rows", a->n_tokens, a->n_heads));
  const float log2_scale = a->scale * kLog2e;
  if (!(log2_scale - log2_scale == 0.0f)) return no(bad(WENC_ERR_INVALID_ARG, "chunk_attention: scale must be below 2^127 (and finite)"));
  return true;
}

template <typename T, int NR>
cudaError_t launch_rows(const ChunkParams& p, const Plan& pl, uint32_t* err, cudaStream_t stream) {
  using C = Cfg<T, NR>;
  auto kern = chunk_rows_kernel<T, NR>;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  static std::atomic<int> configured{-1};
  e = wenc_host::opt_in_smem(kern, C::SMEM, dev, configured);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(pl.blocks));
  cfg.blockDim = dim3(C::THREADS);
  cfg.dynamicSmemBytes = C::SMEM;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = static_cast<unsigned>(pl.rows.cluster);
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = pl.rows.cluster > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kern, p, pl.rows, err);
}

template <typename T>
cudaError_t launch_all(const ChunkParams& p, const Plan& pl, uint32_t* err, cudaStream_t stream) {
  if (pl.nr == 1) return launch_rows<T, 1>(p, pl, err, stream);
  if constexpr (sizeof(T) == 2)
    if (pl.nr == 4) return launch_rows<T, 4>(p, pl, err, stream);
  return launch_rows<T, 2>(p, pl, err, stream);
}

}  // namespace

extern "C" size_t wenc_chunk_attention_workspace(const wenc_chunk_attention_args* a) {
  wenc_internal_clear_error();
  wenc_status st;
  if (!check_sizes(a, &st) || a->n_tokens == 0) return 0;
  return make_plan(a, wenc_internal_sm_count()).bytes;
}

extern "C" wenc_status wenc_chunk_attention(const wenc_chunk_attention_args* a, wenc_stream_t stream) {
  wenc_internal_clear_error();
  wenc_status st;
  if (!check_sizes(a, &st)) return st;
  if (!a->k_pages || !a->v_pages || !a->block_table || !a->lens || !a->q || !a->out)
    return bad(WENC_ERR_INVALID_ARG, "chunk_attention: q, out, the pages, the block table or lens is NULL");
  const long long es = a->dtype == WENC_DTYPE_F32 ? 4 : 2, per16 = 16 / es;
  const long long q_row = static_cast<long long>(a->n_heads) * HD, kv_row = static_cast<long long>(a->n_kv_heads) * HD;
  if (a->q_stride < q_row || a->out_stride < q_row)
    return bad(WENC_ERR_INVALID_ARG, "chunk_attention: a token stride of q or out is smaller than its heads");
  if (a->k_page_stride < kv_row * a->page_size || a->v_page_stride < kv_row * a->page_size)
    return bad(WENC_ERR_INVALID_ARG, "chunk_attention: a page stride is smaller than a page");
  if (a->n_seqs > 1 && a->block_table_stride < a->max_pages)
    return bad(WENC_ERR_INVALID_ARG, "chunk_attention: block_table_stride %lld < max_pages %lld", a->block_table_stride, a->max_pages);
  if (a->k_page_stride / per16 > 0xffffffffll || a->v_page_stride / per16 > 0xffffffffll)
    return bad(WENC_ERR_UNSUPPORTED, "chunk_attention: a page stride passes 2^36 bytes");
  const void* ptrs[] = {a->q, a->out, a->k_pages, a->v_pages};
  for (const void* x : ptrs)
    if (reinterpret_cast<uintptr_t>(x) & 15u) return bad(WENC_ERR_INVALID_ARG, "buffers must be 16-byte aligned");
  const long long strides[] = {a->q_stride, a->out_stride, a->k_page_stride, a->v_page_stride};
  for (long long x : strides)
    if (x % per16 != 0) return bad(WENC_ERR_INVALID_ARG, "strides must be multiples of 16 bytes");
  if (a->n_tokens == 0) return WENC_OK;
  if (!apart(a->q, a->q_stride * es, a->out, a->out_stride * es, q_row * es, a->n_tokens))
    return bad(WENC_ERR_INVALID_ARG, "chunk_attention: out must lie apart from q");
  // (rows are written while others read the cache, the lengths and their queries)
  const long long pages_before = a->n_pages - 1, page = kv_row * a->page_size;
  const Range out_at[] = {{a->out, ((a->n_tokens - 1ll) * a->out_stride + q_row) * es}};
  const Range in[] = {{a->k_pages, (pages_before * a->k_page_stride + page) * es},
                      {a->v_pages, (pages_before * a->v_page_stride + page) * es},
                      {a->block_table, table_bytes(a->n_seqs, a->block_table_stride, a->max_pages)}, {a->lens, 4ll * a->n_seqs},
                      {a->seq_start, 4ll * a->n_seqs + 4}};
  if (share(in, out_at))
    return bad(WENC_ERR_INVALID_ARG, "chunk_attention: out shares memory with the pages, their table, lens or seq_start");
  int sms = 0;
  uint32_t* err = nullptr;
  const wenc_status dst = wenc_internal_device(&sms, &err);
  if (dst != WENC_OK) return dst;
  const Plan pl = make_plan(a, sms);
  if (pl.blocks > 0x7fffffffll) return bad(WENC_ERR_UNSUPPORTED, "chunk_attention: %lld work items pass 2^31 - 1", pl.blocks);
  if (pl.bytes > 0 && (!a->workspace || a->workspace_bytes < pl.bytes))
    return bad(WENC_ERR_INVALID_ARG, "chunk_attention: workspace of %lld bytes needed, %lld given", static_cast<long long>(pl.bytes),
               a->workspace ? static_cast<long long>(a->workspace_bytes) : 0ll);
  if (pl.bytes > 0 && (reinterpret_cast<uintptr_t>(a->workspace) & 255u))
    return bad(WENC_ERR_INVALID_ARG, "chunk_attention: the workspace must be 256-byte aligned");
  const Range room_at[] = {{a->workspace, static_cast<long long>(pl.bytes)}};
  const Range q_at[] = {{a->q, ((a->n_tokens - 1ll) * a->q_stride + q_row) * es}};
  if (share(in, room_at) || share(q_at, room_at) || share(out_at, room_at))
    return bad(WENC_ERR_INVALID_ARG, "chunk_attention: the workspace must lie apart from the other arguments");

  ChunkParams p = {};
  p.q = static_cast<const uint8_t*>(a->q);
  p.out = static_cast<uint8_t*>(a->out);
  p.q_stride = a->q_stride * es;
  p.out_stride = a->out_stride * es;
  p.k_pages = static_cast<const uint8_t*>(a->k_pages);
  p.v_pages = static_cast<const uint8_t*>(a->v_pages);
  p.k_page16 = static_cast<uint32_t>(a->k_page_stride / per16);
  p.v_page16 = static_cast<uint32_t>(a->v_page_stride / per16);
  p.row16 = static_cast<uint32_t>(kv_row / per16);
  p.table = a->block_table;
  p.table_stride = a->block_table_stride;
  p.lens = a->lens;
  p.seq_start = a->seq_start;
  p.n_tokens = a->n_tokens;
  p.n_seqs = a->n_seqs;
  p.per_seq = a->seq_start ? 0 : a->n_tokens / a->n_seqs;
  p.max_new = a->max_new;
  p.H = a->n_heads;
  p.Hkv = a->n_kv_heads;
  p.r = a->n_heads / a->n_kv_heads;
  p.n_pages = a->n_pages;
  p.page_size = a->page_size;
  p.max_pages = a->max_pages;
  p.page_shift = -1;
  for (int s = 0; s < 31; ++s)
    if (a->page_size == 1 << s) p.page_shift = s;
  // (positions are below 2^30: a window of that many hides nothing)
  p.window = a->window > 0 && a->window < 1 << 30 ? a->window : 1 << 30;
  p.sinks = a->window > 0 ? a->sinks : 0;
  // |scale| and the queries' signs; a scale of 0 is 1 on queries of 0
  const bool bf = a->dtype == WENC_DTYPE_BF16;
  p.q_flip = a->scale < 0.0f ? (bf ? 0x80008000u : 0x80000000u) : 0u;
  p.q_keep = a->scale == 0.0f ? 0u : 0xffffffffu;
  p.scale_log2 = (a->scale == 0.0f ? 1.0f : a->scale < 0.0f ? -a->scale : a->scale) * kLog2e;
  const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  cudaError_t e = cudaSuccess;
  if (pl.tc) e = wenc_host::launch_chunk_tc(p, pl.rows.most, a->workspace, err, sms, s);
  // (without offsets every sequence has the rows that the plan counted, more than the few: nothing is left for them)
  if (e == cudaSuccess && !(pl.tc && !a->seq_start)) e = bf ? launch_all<__nv_bfloat16>(p, pl, err, s) : launch_all<float>(p, pl, err, s);
  if (e != cudaSuccess) {
    char buf[200];
    snprintf(buf, sizeof(buf), "chunk_attention launch: %s", cudaGetErrorString(e));
    return wenc_internal_fail(WENC_ERR_CUDA, buf);
  }
  return WENC_OK;
}
