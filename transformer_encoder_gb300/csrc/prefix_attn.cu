// prefix_attn.cu -- attention of a decode step whose sequences share long prefixes.
//
// The beams of a window attend to the same cross-attention keys, and requests behind one prompt to
// the same prompt keys; each sequence adds keys of its own, kept in pages (append.cu). For query
// row (token i of sequence s, head h), with g the group of s and key head h / (H / Hkv):
//   out = softmax(scale * q . [K_prefix(g); K_own(s)]) [V_prefix(g); V_own(s)],
// every prefix key visible, own key j visible when j <= lens[s] - q_len + i, zeros where nothing is
// (inferencelayer 0.2.4 src/whisper_gpu.rs, DEC_QATTN; oxinfer 0.0.5 src/whisper/model.rs,
// CrossLayer::attend and attention_masked).
//
// Rows of one key head: (sequence of the group, token, query head of the key head), so the prefix is read
// once for all of a group's rows. What bounds it: bytes of K and V, and at these sizes the latency of
// getting at them.
//
// Up to 64 rows per key head (beams), and more where there is little to do: one launch. A cluster of 1 to 8 CTAs
// attends one (group, key head, tile of rows): its key list is the prefix followed by the own keys of each sequence of
// the tile, cut into steps of 16 keys that belong to one of these segments each, and every warp of the cluster takes an
// equal run of them. Own keys are scored against all of the tile's rows and masked to their sequence's. The CTAs'
// results (m, l, O) are joined through distributed shared memory: no workspace and no second kernel.
// Else: a work item is a share of a group's prefix, or of one sequence's own keys; items write partial results to
// the workspace and a third kernel joins them. The prefix then runs on the fifth-generation tensor cores
// (prefix_tc.cu, and prefix_tc32.cu for fp32; prefix_part_kernel below takes what those two do not).
//
// Every warp has a ring of cp.async stages of its own and no barrier with other warps until their results
// are joined at the end; an own-key item of the second form is one warp's. The products are transposed:
// S^T = K Q^T and O^T = V^T P^T, with 16 keys (or 16 elements of V) as the MMA's M and 8 query rows as its
// N, so that five beams cost eight columns instead of sixteen rows, and the fragments of K and V
// are loaded once for any number of rows. The running maximum is followed lazily: P keeps its reference
// until a score exceeds it by 2^8, so most tiles need no reduction over lanes and no rescaling.
// mma.sync (m16n8k16 bf16, m16n8k8 TF32): a tcgen05 tile would be 64 or 128 rows and mostly empty.
// bf16: P is split into two bf16 parts before the product with V, so its rounding (2^-16 after the
// split) does not add to the output's own. fp32: every product is three TF32 products of two-part
// operands.
//
// Measured (us on the device, calls of a captured graph over inputs that do not fit L2 together; bytes of K
// and V at the measured copy rate in brackets):
//   16 windows x 5 beams, 20 heads, 1500 cross keys, bf16     22.8 [18.2]   5.4 TB/s
//   the same beams' self-attention, ragged, pages of 16       16.0 [7.0]
//   4 windows x 5 beams x 3 tokens, 8 heads, fp32, pages of 24 12.5 [3.8]
//   1 window, 1 beam, 6 heads, 1500 keys, bf16                 5.3 [0.3]: launch and latency
// What the choices gave, on the first of these unless said: rows as the MMA's M, tiles of 128 keys by four warps 29.5;
// four CTAs a cluster for more CTAs 40.2, one CTA an item and three an SM 23.7 (the CTAs of one round hide each
// other's latency; more of them only repeat the start of a CTA, some 4 us); S^T with eight warps 22.3. On the
// second: 40.7, 26.4 and 22.2, then 18.8 with 32-bit address factors and 15.9 with runs of 16-key steps (tiles of
// 128 left warps idle at every segment's end). Three stages a warp instead of two cost the third CTA of an SM:
// 28.8. What bounds them now: the latency of a warp's steps at 24 warps an SM (the stall counters show waits for
// loads); in fp32, the instructions of the two-part splits at 8 warps an SM (253 registers).
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <math_constants.h>

#include <atomic>
#include <cstdio>
#include <string>

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

constexpr int HD = 64;

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool there) {
  const int n = there ? 16 : 0;  // 0 source bytes: the 16 are filled with zeros
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void ldsm_x4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr));
}
__device__ __forceinline__ void ldsm_x4_t(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr));
}
__device__ __forceinline__ float4 lds_f4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(addr));
  return v;
}
__device__ __forceinline__ void mma_bf16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_tf32(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// x = hi + lo for two TF32 operands: hi is x rounded to 11 significant bits, lo the (exact) rest, of which the
// MMA reads the first 11 bits (it ignores the 13 low bits of a TF32 operand): together they miss x by less
// than 2^-22 |x|, with the sign of lo, which is that of a rounding. A NaN passes: where the addition carries
// it out of hi's exponent, lo is the NaN.
__device__ __forceinline__ void split_tf32(float x, uint32_t& hi, uint32_t& lo) {
  hi = (__float_as_uint(x) + 0x1000u) & 0xffffe000u;
  lo = __float_as_uint(x - __uint_as_float(hi));
}
// Transpose of an 8 x 8 matrix of 16-bit elements (lane: row lane / 4, columns 2 (lane % 4) and the next).
__device__ __forceinline__ uint32_t movm_t(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

struct PrefixParams {
  const uint8_t* q;
  uint8_t* out;
  long long q_stride, out_stride;  // bytes between tokens
  const uint8_t *kp, *vp;
  long long k_group, k_token, v_group, v_token;  // bytes
  const uint8_t *k_pages, *v_pages;
  uint32_t k_page16, v_page16, row16;  // between pages, and between a page's slots, in units of 16 bytes
  const int32_t *group_start, *prefix_lens, *table, *lens;
  long long table_stride;
  int n_seqs, q_len, H, Hkv, r, n_groups, max_group, prefix_max, n_pages, page_size, page_shift, max_pages;
  int np, ns;                    // prefix and own-key splits of the two-launch form (0: no such keys)
  int row_tiles;                 // row tiles per item of this launch
  int cluster;                   // CTAs per item (one-launch form)
  float scale_log2;              // >= 0
  uint32_t q_flip, q_keep;       // a negative scale turns the queries' signs (per 32 bits), a zero one clears them
  float* part_o;                 // [(token * H + head) * (np + ns) + slot][64]
  float2* part_ml;               // the same without [64]: (maximum in log2 units, sum)
};

// NR groups of 8 query rows per CTA.
template <typename T, int NR>
struct Cfg {
  static constexpr bool F32 = sizeof(T) == 4;
  static constexpr int NW = F32 ? 4 : 8;       // warps
  static constexpr int THREADS = 32 * NW;
  static constexpr int KW = 16;                // keys per step of a warp
  static constexpr int ROWS = 8 * NR;
  static constexpr int ROWB = HD * sizeof(T);
  static constexpr int STAGES = 2;
  static constexpr int CTAS = NR == 1 ? 3 : 2;  // per SM, for the registers
  static constexpr uint32_t HALF = KW * ROWB;  // bytes of K (or V) per warp and stage
  static constexpr uint32_t RING = NW * STAGES * 2 * HALF;
  static constexpr uint32_t P_BYTES = F32 ? NW * NR * 16 * 8 * 4 : 0;  // fp32: P on its way to B fragments
  // results over the ring: O [NW][ROWS][OS] floats, (m, l) [NW][ROWS]
  static constexpr int OS = HD + 4;
  static constexpr uint32_t ML = NW * ROWS * OS * 4;
  static constexpr uint32_t RESULTS = ML + NW * ROWS * 8;
  static constexpr uint32_t SMEM = (RING + P_BYTES > RESULTS ? RING + P_BYTES : RESULTS);
};

// What one CTA (or warp) attends: n_rows rows of one key head of a group, against a run of the steps of a list
// of segments: segment 0 is the prefix, segment i the own keys of sequence seq0 + i - 1, which only
// that sequence's rows see.
struct Item {
  const uint8_t *kp, *vp;   // first prefix key of the key head
  int prefix_len;
  int seq0, n_own;          // first sequence of the rows, and how many bring own keys (0: none do)
  int row_off;              // row x of the tile is row row_off + x of sequence seq0's first row on
  int n_rows;
  int hk;
};

constexpr int kMaxOwn = 16;  // own-key segments of an item: at most one per row of a tile
struct SegTable {
  int step0[kMaxOwn + 2];    // first step of each segment, and the end
  int len[kMaxOwn + 1];      // its keys
};

// What the index-checked build asks of every access (ptx.cuh): a token and head of the call, a sequence's table entry, a
// slot of the pool, a key of the prefix, a slot of the partial results.
__device__ __forceinline__ bool row_in(const PrefixParams& p, long long token, int head, uint32_t* err, uint32_t site) {
  return in_bounds(token >= 0 && token < static_cast<long long>(p.n_seqs) * p.q_len && head >= 0 && head < p.H, err, site);
}
__device__ __forceinline__ bool entry_in(const PrefixParams& p, int seq, int page_i, uint32_t* err, uint32_t site) {
  return in_bounds(seq >= 0 && seq < p.n_seqs && page_i >= 0 && page_i < p.max_pages, err, site);
}
__device__ __forceinline__ bool slot_in(const PrefixParams& p, int page, int slot, int hk, uint32_t* err, uint32_t site) {
  return in_bounds(page >= 0 && page < p.n_pages && slot >= 0 && slot < p.page_size && hk >= 0 && hk < p.Hkv, err, site);
}
__device__ __forceinline__ bool key_in(const PrefixParams& p, int key, int hk, uint32_t* err, uint32_t site) {
  return in_bounds(key >= 0 && key < p.prefix_max && hk >= 0 && hk < p.Hkv, err, site);
}

__device__ __forceinline__ int own_len_of(const PrefixParams& p, int seq, uint32_t* err) {
  if (!in_bounds(seq >= 0 && seq < p.n_seqs, err, 83)) return 0;
  int n = p.lens[seq];
  if (n < 0 || n > static_cast<long long>(p.max_pages) * p.page_size) {
    *reinterpret_cast<volatile uint32_t*>(err) = kErrData | (81u << 8);
    n = 0;
  }
  return n;
}

// The segments' steps: a running sum over up to 17 lengths, by warp 0. Ends with a barrier.
__device__ __forceinline__ void fill_segments(const PrefixParams& p, const Item& it, SegTable& seg, uint32_t* err) {
  const int lane = threadIdx.x & 31;
  if (threadIdx.x < 32) {
    const int base = (it.prefix_len + 15) / 16;
    const int n = lane < it.n_own ? own_len_of(p, it.seq0 + lane, err) : 0;
    int sum = (n + 15) / 16;
    if (it.n_own > 1) {
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int up = __shfl_up_sync(0xffffffffu, sum, d);
        if (lane >= d) sum += up;
      }
    }
    if (lane == 0) {
      seg.step0[0] = 0;
      seg.len[0] = it.prefix_len;
      seg.step0[1] = base;
    }
    if (lane < it.n_own) {
      seg.len[1 + lane] = n;
      seg.step0[2 + lane] = base + sum;
    }
  }
  __syncthreads();
}

// 16-byte granule `c` of key row `row` within a warp's stage. bf16 rows have 8 granules (all 32 banks),
// fp32 rows 16; the XOR spreads the rows that an ldmatrix (or a quarter of a fragment load) touches at
// once over all banks.
template <bool F32>
__device__ __forceinline__ uint32_t granule(int row, int c) {
  if constexpr (F32)
    return row * 256u + ((c ^ (((row & 1) << 2) | (row & 2))) << 4);
  else
    return row * 128u + ((c ^ (row & 7)) << 4);
}

// The state of a warp's rows: this thread's columns of O^T and S^T are rows 8 r + 2 (lane % 4) + e.
template <int NR>
struct RowState {
  float o[NR][4][4], m[NR][2], l[NR][2];  // m in log2 units; l of this thread's keys alone until reduced
};

// One warp's run of steps [step0, step0 + n_mine). SOLO: the item is one own-key segment of solo_len keys
// (no table); else the segments are in `seg`.
template <typename T, int NR, bool SOLO>
__device__ __forceinline__ void attend(const PrefixParams& p, const Item& it, uint8_t* smem, const SegTable* seg, int solo_len,
                                       int step0, int n_mine, RowState<NR>& st, uint32_t* err) {
  using C = Cfg<T, NR>;
  constexpr bool F32 = C::F32;
  constexpr int KW = C::KW, ST = C::STAGES;
  constexpr int CH = C::ROWB / 16;  // granules per row
  constexpr int RPI = 32 / CH;      // rows a warp's copy instruction covers
  constexpr int NL = KW / RPI;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, tq = lane & 3;
  const uint32_t s0 = smem_u32(smem) + warp * (ST * 2 * C::HALF);

  // ---- loads of a step: 16 keys and values. Addresses in units of 16 bytes (32-bit
  // factors, 64-bit sums). Rows RPI i + lr of a stage: two swizzled positions alternate with i.
  const int lc = lane % CH, lr = lane / CH;
  const uint32_t at0 = granule<F32>(lr, lc), at1 = granule<F32>(lr + RPI, lc) - 512u;
  static_assert(RPI * C::ROWB == 512, "a copy instruction covers 512 bytes of a stage");
  int lseg = 0, lbegin = 0, lend = 0, lkeys = 0;  // segment of the next step to load, its steps and keys
  int next_page = 0;  // page of the key in the next step's row lane % 16 (own keys), read one step ahead
  auto advance = [&](int t, int& sg, int& begin, int& end, int& keys) {
    if constexpr (SOLO) {
      sg = 1;
      begin = 0;
      end = 0x7fffffff;
      keys = solo_len;
    } else {
      sg = segment_of(seg->step0, t, sg);
      begin = seg->step0[sg];
      end = seg->step0[sg + 1];
      keys = seg->len[sg];
    }
  };
  auto page_of = [&](int j) {
    if (step0 + j >= lend) advance(step0 + j, lseg, lbegin, lend, lkeys);
    if (!SOLO && lseg == 0) return;
    const int key = (step0 + j - lbegin) * KW + (lane & 15);
    const int pi = p.page_shift >= 0 ? key >> p.page_shift : key / p.page_size;
    const int seq = it.seq0 + lseg - 1;
    next_page = key < lkeys && entry_in(p, seq, pi, err, 84) ? p.table[seq * p.table_stride + pi] : -1;
  };
  auto load = [&](int j, int stage) {
    const uint32_t sk = s0 + stage * (2 * C::HALF), sv = sk + C::HALF;
    const int key0 = (step0 + j - lbegin) * KW;
    if (!SOLO && lseg == 0) {
      const uint8_t* ks = it.kp + (key0 + lr) * p.k_token + lc * 16;
      const uint8_t* vs = it.vp + (key0 + lr) * p.v_token + lc * 16;
#pragma unroll
      for (int i = 0; i < NL; ++i) {
        const bool ok = key0 + lr + i * RPI < lkeys && key_in(p, key0 + lr + i * RPI, it.hk, err, 85);
        const uint32_t at = ((i & 1) ? at1 : at0) + i * 512;
        cp_async16(sk + at, ok ? ks : it.kp, ok);
        cp_async16(sv + at, ok ? vs : it.vp, ok);
        ks += RPI * p.k_token;
        vs += RPI * p.v_token;
      }
    } else {
      const int key = key0 + (lane & 15);
      const int pi = p.page_shift >= 0 ? key >> p.page_shift : key / p.page_size;
      const bool in = static_cast<uint32_t>(next_page) < static_cast<uint32_t>(p.n_pages);
      if (!in && key < lkeys) *reinterpret_cast<volatile uint32_t*>(err) = kErrData | (80u << 8);
      const int page = in && slot_in(p, next_page, key - pi * p.page_size, it.hk, err, 86) ? next_page : -1;
      const uint32_t slot = (key - pi * p.page_size) * p.row16, head = it.hk * CH + lc;
#pragma unroll
      for (int i = 0; i < NL; ++i) {
        const int pg = __shfl_sync(0xffffffffu, page, lr + i * RPI);
        const uint32_t x = __shfl_sync(0xffffffffu, slot, lr + i * RPI) + head;
        const bool ok = pg >= 0;
        const uint32_t upg = ok ? pg : 0, at = ((i & 1) ? at1 : at0) + i * 512;
        cp_async16(sk + at, p.k_pages + ((static_cast<uint64_t>(upg) * p.k_page16 + x) << 4), ok);
        cp_async16(sv + at, p.v_pages + ((static_cast<uint64_t>(upg) * p.v_page16 + x) << 4), ok);
      }
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

  // ---- the query rows as B fragments (column g of group r: row 8 r + g); rows past the end are zeros
  constexpr int KS = F32 ? 8 : 4;  // k steps of one score product
  uint32_t qh[NR][KS][2], ql[F32 ? NR : 1][KS][2];
#pragma unroll
  for (int r = 0; r < NR; ++r) {
    const int x = it.row_off + 8 * r + g;
    const int tok = x / p.r;
    const long long token = static_cast<long long>(it.seq0) * p.q_len + tok;
    const int head = it.hk * p.r + x - tok * p.r;
    const bool in = 8 * r + g < it.n_rows && row_in(p, token, head, err, 87);
    const uint8_t* q = p.q + token * p.q_stride + head * C::ROWB;
    if constexpr (F32) {
      // k index tq (and tq + 4) of step 2j (and 2j + 1) stands for element 4 (tq + 4j) + 0, 1 (2, 3)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint4 a = in ? *reinterpret_cast<const uint4*>(q + (tq + 4 * j) * 16) : make_uint4(0u, 0u, 0u, 0u);
        auto part = [&](uint32_t v, uint32_t& hi, uint32_t& lo) {
          split_tf32(__uint_as_float((v & p.q_keep) ^ p.q_flip), hi, lo);
        };
        part(a.x, qh[r][2 * j][0], ql[r][2 * j][0]);
        part(a.y, qh[r][2 * j][1], ql[r][2 * j][1]);
        part(a.z, qh[r][2 * j + 1][0], ql[r][2 * j + 1][0]);
        part(a.w, qh[r][2 * j + 1][1], ql[r][2 * j + 1][1]);
      }
    } else {
#pragma unroll
      for (int k = 0; k < KS; ++k)
#pragma unroll
        for (int h = 0; h < 2; ++h)
          qh[r][k][h] = in ? (*reinterpret_cast<const uint32_t*>(q + (16 * k + 8 * h + 2 * tq) * 2) & p.q_keep) ^ p.q_flip : 0u;
    }
  }
  // this thread's columns of S^T and O^T: rows 8 r + 2 tq + e; their sequence and token
  const int per_seq = p.q_len * p.r;
  int seq_of[NR][2], tok_of[NR][2];
#pragma unroll
  for (int r = 0; r < NR; ++r)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int x = it.row_off + 8 * r + 2 * tq + e;
      seq_of[r][e] = x / per_seq;
      tok_of[r][e] = (x - seq_of[r][e] * per_seq) / p.r;
    }

  auto &o = st.o;
  auto &m = st.m, &l = st.l;
  float u[NR][2];  // the reference in use: m, or 0 while that is -inf
#pragma unroll
  for (int r = 0; r < NR; ++r) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[r][i][e] = 0.0f;
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      m[r][e] = -CUDART_INF_F;
      u[r][e] = l[r][e] = 0.0f;
    }
  }
  const float sc = p.scale_log2;

  int cseg = 0, cbegin = 0, cend = 0, n_keys = 0;  // the segment being scored
  int lim[NR][2] = {};                             // its keys that each of this thread's rows sees
  for (int j = 0; j < n_mine; ++j) {
    cp_async_wait<ST - 2>();
    __syncwarp();
    if (j + ST - 1 < n_mine) {
      load(j + ST - 1, (j + ST - 1) % ST);
      if (j + ST < n_mine) page_of(j + ST);
    }
    cp_async_commit();
    if (step0 + j >= cend) {
      advance(step0 + j, cseg, cbegin, cend, n_keys);
#pragma unroll
      for (int r = 0; r < NR; ++r)
#pragma unroll
        for (int e = 0; e < 2; ++e)
          lim[r][e] = cseg == 0 ? n_keys : seq_of[r][e] == cseg - 1 ? n_keys - p.q_len + 1 + tok_of[r][e] : 0;
    }
    const int key0 = (step0 + j - cbegin) * KW;
    const uint32_t sk = s0 + (j % ST) * (2 * C::HALF), sv = sk + C::HALF;

    // ---- S^T: 16 keys x 8 NR rows
    float s[NR][4];
#pragma unroll
    for (int r = 0; r < NR; ++r)
#pragma unroll
      for (int e = 0; e < 4; ++e) s[r][e] = 0.0f;
    if constexpr (F32) {
      // the products with a small part are summed apart: the tensor core's sums truncate, and these are 2^-11 as large
      float small[NR][4];
#pragma unroll
      for (int r = 0; r < NR; ++r)
#pragma unroll
        for (int e = 0; e < 4; ++e) small[r][e] = 0.0f;
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const float4 ka = lds_f4(sk + granule<true>(g, tq + 4 * c)), kb = lds_f4(sk + granule<true>(g + 8, tq + 4 * c));
        uint32_t h[2][4], w[2][4];
        split_tf32(ka.x, h[0][0], w[0][0]);
        split_tf32(kb.x, h[0][1], w[0][1]);
        split_tf32(ka.y, h[0][2], w[0][2]);
        split_tf32(kb.y, h[0][3], w[0][3]);
        split_tf32(ka.z, h[1][0], w[1][0]);
        split_tf32(kb.z, h[1][1], w[1][1]);
        split_tf32(ka.w, h[1][2], w[1][2]);
        split_tf32(kb.w, h[1][3], w[1][3]);
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int r = 0; r < NR; ++r) {
            mma_tf32(small[r], h[i], ql[r][2 * c + i][0], ql[r][2 * c + i][1]);
            mma_tf32(small[r], w[i], qh[r][2 * c + i][0], qh[r][2 * c + i][1]);
            mma_tf32(s[r], h[i], qh[r][2 * c + i][0], qh[r][2 * c + i][1]);
          }
      }
#pragma unroll
      for (int r = 0; r < NR; ++r)
#pragma unroll
        for (int e = 0; e < 4; ++e) s[r][e] += small[r][e];
    } else {
#pragma unroll
      for (int k = 0; k < KS; ++k) {
        uint32_t a[4];
        ldsm_x4(a, sk + granule<false>(lane & 15, 2 * k + (lane >> 4)));
#pragma unroll
        for (int r = 0; r < NR; ++r) mma_bf16(s[r], a, qh[r][k][0], qh[r][k][1]);
      }
    }
    // ---- mask (element e: key g + 8 (e / 2), row column e % 2), then P
    // (one sequence's own keys: only the newest q_len are hidden from some of its rows)
    if (SOLO ? key0 + KW > n_keys - p.q_len + 1 : cseg > 0 || key0 + KW > n_keys) {
#pragma unroll
      for (int r = 0; r < NR; ++r)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (key0 + g + 8 * (e >> 1) >= lim[r][e & 1]) s[r][e] = -CUDART_INF_F;
    }
    bool move = false;  // some score exceeds its row's reference by more than 2^8
#pragma unroll
    for (int r = 0; r < NR; ++r)
#pragma unroll
      for (int e = 0; e < 2; ++e) move |= fmaxf(s[r][e], s[r][e + 2]) * sc > m[r][e] + 8.0f;
    if (__any_sync(0xffffffffu, move)) {
#pragma unroll
      for (int r = 0; r < NR; ++r)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float x = fmaxf(s[r][e], s[r][e + 2]);
          x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 4));
          x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 8));
          x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 16));
          x = fmaxf(x * sc, m[r][e]);
          const float ref = x == -CUDART_INF_F ? 0.0f : x;
          const float f = ex2_approx(m[r][e] - ref);
          m[r][e] = x;
          u[r][e] = ref;
          l[r][e] *= f;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            o[r][i][e] *= f;
            o[r][i][e + 2] *= f;
          }
        }
    }
#pragma unroll
    for (int r = 0; r < NR; ++r)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        s[r][e] = ex2_approx(fmaf(s[r][e], sc, -u[r][e & 1]));
        l[r][e & 1] += s[r][e];
      }
    // ---- O^T += V^T P^T
    if constexpr (F32) {
      // P through shared memory: written as [key][row], read as B fragments (key tq, row g). The tile's
      // product is formed on its own and added in one rounding, so that the tensor core's accumulation
      // (which truncates) runs over one tile only.
      const uint32_t sp = smem_u32(smem) + C::RING + warp * (NR * 512);
#pragma unroll
      for (int r = 0; r < NR; ++r) {
        asm volatile("st.shared.v2.f32 [%0], {%1, %2};" ::"r"(sp + r * 512 + (g * 8 + 2 * tq) * 4), "f"(s[r][0]), "f"(s[r][1]) : "memory");
        asm volatile("st.shared.v2.f32 [%0], {%1, %2};" ::"r"(sp + r * 512 + ((g + 8) * 8 + 2 * tq) * 4), "f"(s[r][2]), "f"(s[r][3]) : "memory");
      }
      __syncwarp();
      uint32_t ph[NR][2][2], pl[NR][2][2];
#pragma unroll
      for (int r = 0; r < NR; ++r)
#pragma unroll
        for (int k = 0; k < 2; ++k)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            float x;
            asm volatile("ld.shared.f32 %0, [%1];" : "=f"(x) : "r"(sp + r * 512 + ((8 * k + 4 * h + tq) * 8 + g) * 4) : "memory");
            split_tf32(x, ph[r][k][h], pl[r][k][h]);
          }
      __syncwarp();
      // row g (g + 8) of product i stands for element 4 g + i (32 + 4 g + i)
      float t[NR][4][4];
#pragma unroll
      for (int r = 0; r < NR; ++r)
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int e = 0; e < 4; ++e) t[r][i][e] = 0.0f;
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const float4 v0 = lds_f4(sv + granule<true>(8 * k + tq, g)), v1 = lds_f4(sv + granule<true>(8 * k + tq, g + 8));
        const float4 v2 = lds_f4(sv + granule<true>(8 * k + tq + 4, g)), v3 = lds_f4(sv + granule<true>(8 * k + tq + 4, g + 8));
        const float w[4][4] = {{v0.x, v1.x, v2.x, v3.x}, {v0.y, v1.y, v2.y, v3.y}, {v0.z, v1.z, v2.z, v3.z}, {v0.w, v1.w, v2.w, v3.w}};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          uint32_t vh[4], vl[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) split_tf32(w[i][e], vh[e], vl[e]);
#pragma unroll
          for (int r = 0; r < NR; ++r) {
            mma_tf32(t[r][i], vh, pl[r][k][0], pl[r][k][1]);
            mma_tf32(t[r][i], vl, ph[r][k][0], ph[r][k][1]);
            mma_tf32(t[r][i], vh, ph[r][k][0], ph[r][k][1]);
          }
        }
      }
#pragma unroll
      for (int r = 0; r < NR; ++r)
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int e = 0; e < 4; ++e) o[r][i][e] += t[r][i][e];
    } else {
      uint32_t ph[NR][2], pl[NR][2];
#pragma unroll
      for (int r = 0; r < NR; ++r)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const float x = s[r][2 * h], y = s[r][2 * h + 1];
          const uint32_t hi = pack_bf16x2(x, y);
          const uint32_t lo = pack_bf16x2(x - __uint_as_float(hi << 16), y - __uint_as_float(hi & 0xffff0000u));
          ph[r][h] = movm_t(hi);
          pl[r][h] = movm_t(lo);
        }
#pragma unroll
      for (int i = 0; i < 4; ++i) {  // 16 elements of V at a time
        uint32_t a[4];
        ldsm_x4_t(a, sv + granule<false>((lane & 7) + ((lane >> 4) << 3), 2 * i + ((lane >> 3) & 1)));
#pragma unroll
        for (int r = 0; r < NR; ++r) {
          mma_bf16(o[r][i], a, ph[r][0], ph[r][1]);
          mma_bf16(o[r][i], a, pl[r][0], pl[r][1]);
        }
      }
    }
  }

  cp_async_wait<0>();
#pragma unroll
  for (int r = 0; r < NR; ++r)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      l[r][e] += __shfl_xor_sync(0xffffffffu, l[r][e], 4);
      l[r][e] += __shfl_xor_sync(0xffffffffu, l[r][e], 8);
      l[r][e] += __shfl_xor_sync(0xffffffffu, l[r][e], 16);
    }
}

// All warps' results into shared memory, over the rings; begins and ends with a barrier.
template <typename T, int NR>
__device__ __forceinline__ void share_results(uint8_t* smem, const RowState<NR>& st) {
  using C = Cfg<T, NR>;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, tq = lane & 3;
  __syncthreads();
  float* so = reinterpret_cast<float*>(smem) + warp * C::ROWS * C::OS;
  float2* sml = reinterpret_cast<float2*>(smem + C::ML) + warp * C::ROWS;
#pragma unroll
  for (int r = 0; r < NR; ++r)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int x = 8 * r + 2 * tq + e;
      if (g == 0) sml[x] = make_float2(st.m[r][e], st.l[r][e]);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        so[x * C::OS + (C::F32 ? 4 * g + i : 16 * i + g)] = st.o[r][i][e];
        so[x * C::OS + (C::F32 ? 32 + 4 * g + i : 16 * i + g + 8)] = st.o[r][i][e + 2];
      }
    }
  __syncthreads();
}

// Join of the warps' results for row x of the tile, elements c8 .. c8 + 7.
template <typename T, int NR>
__device__ __forceinline__ void join_warps(const uint8_t* smem, int x, int c8, float (&v)[8], float& m, float& l) {
  using C = Cfg<T, NR>;
  const float* so = reinterpret_cast<const float*>(smem);
  const float2* sml = reinterpret_cast<const float2*>(smem + C::ML);
  m = -CUDART_INF_F;
  l = 0.0f;
#pragma unroll
  for (int e = 0; e < 8; ++e) v[e] = 0.0f;
#pragma unroll
  for (int w = 0; w < C::NW; ++w) m = fmaxf(m, sml[w * C::ROWS + x].x);
  const float u = m == -CUDART_INF_F ? 0.0f : m;
#pragma unroll
  for (int w = 0; w < C::NW; ++w) {
    const float2 ml = sml[w * C::ROWS + x];
    const float f = ex2_approx(ml.x - u);
    l += f * ml.y;
    const float4* o = reinterpret_cast<const float4*>(so + (w * C::ROWS + x) * C::OS + c8);
    const float4 a = o[0], b = o[1];
    v[0] += f * a.x; v[1] += f * a.y; v[2] += f * a.z; v[3] += f * a.w;
    v[4] += f * b.x; v[5] += f * b.y; v[6] += f * b.z; v[7] += f * b.w;
  }
}

// Eight elements of a key or query row as fp32.
__device__ __forceinline__ void load8(const float* x, float (&f)[8]) {
  const float4 a = reinterpret_cast<const float4*>(x)[0], b = reinterpret_cast<const float4*>(x)[1];
  f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
  f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
}
__device__ __forceinline__ void load8(const __nv_bfloat16* x, float (&f)[8]) {
  const uint4 u = *reinterpret_cast<const uint4*>(x);
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = __uint_as_float(w[i] << 16);
    f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}

// The products with V are formed for all of a tile's rows, with weights of 0 where a row does not see a key, and in
// two parts; but 0 x inf and 0 x NaN are NaN, so a value that is no number would reach rows that do not see it. And
// the TF32 part of a float32 next to the largest one is infinite. Such elements of a row's O, and all of a row whose
// sum is no number (rare: they are found by that), are formed again here in plain fp32, from the keys alone that the
// row sees among steps [step0, step0 + n_steps). Eight lanes hold a row: x, its elements c8 .. c8 + 7 in v, maximum m
// and sum l. (Looking for them on the joined results of a CTA costs a call 0.1 to 0.2 us, the joined form 0.7; on
// each warp's own state, before the join, it cost 0.4 to 1.3.)
template <typename T, bool SOLO>
__device__ __noinline__ void redo_rows(const PrefixParams& p, const Item& it, const SegTable* seg, int solo_len, int step0, int n_steps,
                                       int x, int c8, float (&v)[8], float& m, float& l, uint32_t* err) {
  const bool in = x < it.n_rows, again = in && !(fabsf(l) < CUDART_INF_F);
  bool bad[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    bad[e] = in && (again || !(fabsf(v[e]) < CUDART_INF_F));
    if (bad[e]) v[e] = 0.0f;
  }
  if (again) {
    m = -CUDART_INF_F;
    l = 0.0f;
  }
  const int y = it.row_off + x, tok = y / p.r, per_seq = p.q_len * p.r, row_seq = y / per_seq, row_tok = (y - row_seq * per_seq) / p.r;
  const long long token = static_cast<long long>(it.seq0) * p.q_len + tok;
  const int head = it.hk * p.r + y - tok * p.r;
  float q[8] = {};
  if (in && row_in(p, token, head, err, 88)) load8(reinterpret_cast<const T*>(p.q + token * p.q_stride) + head * HD + c8, q);
#pragma unroll
  for (int e = 0; e < 8; ++e)
    if (p.q_keep == 0u) q[e] = 0.0f;
    else if (p.q_flip != 0u) q[e] = -q[e];
  // every key of the steps: f(its value row, whether this lane's row sees it, that row's score in log2 units)
  auto each_key = [&](auto&& f) {
    int sg = SOLO ? 1 : 0;
#pragma unroll 1
    for (int t = step0; t < step0 + n_steps; ++t) {
      int begin = 0, n_keys = solo_len;
      if constexpr (!SOLO) {
        sg = segment_of(seg->step0, t, sg);
        begin = seg->step0[sg];
        n_keys = seg->len[sg];
      }
      const int last = min(n_keys, (t - begin + 1) * 16);
#pragma unroll 1
      for (int key = (t - begin) * 16; key < last; ++key) {
        const uint8_t *k, *vr;
        if (sg == 0) {
          if (!key_in(p, key, it.hk, err, 88)) continue;
          k = it.kp + key * p.k_token;
          vr = it.vp + key * p.v_token;
        } else {
          const int pi = key / p.page_size;
          if (!entry_in(p, it.seq0 + sg - 1, pi, err, 88)) continue;
          const int page = p.table[(it.seq0 + sg - 1) * p.table_stride + pi];
          if (page < 0 || page >= p.n_pages) continue;  // (reported when its step was loaded)
          const uint64_t at = static_cast<uint64_t>(key - pi * p.page_size) * p.row16 + it.hk * (HD * sizeof(T) / 16);
          k = p.k_pages + ((static_cast<uint64_t>(page) * p.k_page16 + at) << 4);
          vr = p.v_pages + ((static_cast<uint64_t>(page) * p.v_page16 + at) << 4);
        }
        const bool sees = in && (sg == 0 || (row_seq == sg - 1 && key < n_keys - p.q_len + 1 + row_tok));
        float kf[8], dot = 0.0f;
        load8(reinterpret_cast<const T*>(k) + c8, kf);
#pragma unroll
        for (int e = 0; e < 8; ++e) dot = fmaf(q[e], kf[e], dot);
#pragma unroll
        for (int d = 1; d < 8; d <<= 1) dot += __shfl_xor_sync(0xffffffffu, dot, d);
        f(reinterpret_cast<const T*>(vr) + c8, sees, dot * p.scale_log2);
      }
    }
  };
  if (__any_sync(0xffffffffu, again))
    each_key([&](const T*, bool sees, float s) {
      if (sees && again) m = fmaxf(m, s);
    });
  const float u = m == -CUDART_INF_F ? 0.0f : m;
  each_key([&](const T* row, bool sees, float s) {
    if (!sees) return;
    const float w = ex2_approx(s - u);
    if (again) l += w;
    float vf[8];
    load8(row, vf);
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (bad[e]) v[e] = fmaf(w, vf[e], v[e]);
  });
}

// The check, and rarely the call, with copies so that the values stay in registers otherwise. steps(): the steps.
template <typename T, bool SOLO, class Steps>
__device__ __forceinline__ void redo_if_needed(const PrefixParams& p, const Item& it, const SegTable* seg, int solo_len, const Steps& steps,
                                               int x, int c8, float (&v)[8], float& m, float& l, uint32_t* err) {
  float zero = l * 0.0f;
#pragma unroll
  for (int e = 0; e < 8; ++e) zero = fmaf(v[e], 0.0f, zero);
  if (!__any_sync(0xffffffffu, !(zero == 0.0f))) return;
  const Item item = it;
  int step0, n_steps;
  float vc[8], mc = m, lc = l;
#pragma unroll
  for (int e = 0; e < 8; ++e) vc[e] = v[e];
  steps(step0, n_steps);
  redo_rows<T, SOLO>(p, item, seg, solo_len, step0, n_steps, x, c8, vc, mc, lc, err);
#pragma unroll
  for (int e = 0; e < 8; ++e) v[e] = vc[e];
  m = mc;
  l = lc;
}

// The steps that the NW warps of a CTA take, parts first_part .. first_part + NW - 1 of `parts`.
template <int NW>
__device__ __forceinline__ void cta_run(int n, int first_part, int parts, int& first, int& count) {
  int last, n_last;
  run_of(n, first_part, parts, first, count);
  run_of(n, first_part + NW - 1, parts, last, n_last);
  count = min(n, last + n_last) - first;
}

// Eight elements of an output row, normalised (a row without a visible key: zeros).
template <typename T>
__device__ __forceinline__ void write_out8(const PrefixParams& p, int token, int head, int c8, const float (&v)[8], float l, uint32_t* err) {
  if (!row_in(p, token, head, err, 89)) return;
  const float inv = l != 0.0f ? 1.0f / l : 0.0f;
  uint8_t* dst = p.out + static_cast<long long>(token) * p.out_stride + (head * HD + c8) * static_cast<int>(sizeof(T));
  if constexpr (sizeof(T) == 4) {
    reinterpret_cast<float4*>(dst)[0] = make_float4(v[0] * inv, v[1] * inv, v[2] * inv, v[3] * inv);
    reinterpret_cast<float4*>(dst)[1] = make_float4(v[4] * inv, v[5] * inv, v[6] * inv, v[7] * inv);
  } else {
    *reinterpret_cast<uint4*>(dst) = make_uint4(pack_bf16x2(v[0] * inv, v[1] * inv), pack_bf16x2(v[2] * inv, v[3] * inv),
                                                pack_bf16x2(v[4] * inv, v[5] * inv), pack_bf16x2(v[6] * inv, v[7] * inv));
  }
}

// The sequences of a group (a range that leads outside the batch, or a group larger than max_group,
// is cut and reported).
__device__ __forceinline__ void group_range(const PrefixParams& p, int g, int& begin, int& count, uint32_t* err) {
  if (!p.group_start) {
    begin = g * p.max_group;
    count = p.max_group;
    return;
  }
  begin = p.group_start[g];
  const int end = p.group_start[g + 1];
  count = end - begin;
  if (begin < 0 || count < 0 || end > p.n_seqs || count > p.max_group) {
    *reinterpret_cast<volatile uint32_t*>(err) = kErrData | (82u << 8);
    count = 0;
  }
}

__device__ __forceinline__ int prefix_len_of(const PrefixParams& p, int grp, uint32_t* err) {
  int n = p.prefix_lens ? p.prefix_lens[grp] : p.prefix_max;
  if (n < 0 || n > p.prefix_max) {
    *reinterpret_cast<volatile uint32_t*>(err) = kErrData | (81u << 8);
    n = 0;
  }
  return n;
}

__device__ __forceinline__ float2 ld_cluster_f2(uint32_t a) {
  float2 v;
  asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(a) : "memory");
  return v;
}

// One-launch form: a cluster of p.cluster CTAs attends one (group, key head, tile of rows).
template <typename T, int NR>
__global__ void __launch_bounds__(Cfg<T, NR>::THREADS, Cfg<T, NR>::CTAS) prefix_cluster_kernel(const __grid_constant__ PrefixParams p, uint32_t* err) {
  using C = Cfg<T, NR>;
  extern __shared__ __align__(128) uint8_t smem_dyn[];
  __shared__ SegTable seg;
  pdl_trigger();
  pdl_wait();
  const int rank = blockIdx.x % p.cluster;
  int b = blockIdx.x / p.cluster;
  const int tile = b % p.row_tiles;
  b /= p.row_tiles;
  Item it;
  const int grp = b / p.Hkv;
  it.hk = b % p.Hkv;
  int begin, count;
  group_range(p, grp, begin, count, err);
  const int per_seq = p.q_len * p.r, row0 = tile * C::ROWS;
  it.n_rows = min(count * per_seq - row0, C::ROWS);
  if (it.n_rows <= 0) return;  // the whole cluster
  it.kp = p.kp + grp * p.k_group + it.hk * C::ROWB;
  it.vp = p.vp + grp * p.v_group + it.hk * C::ROWB;
  it.prefix_len = p.kp ? prefix_len_of(p, grp, err) : 0;
  const int first = row0 / per_seq;  // sequences of the tile's rows
  it.seq0 = begin + first;
  it.row_off = row0 - first * per_seq;
  it.n_own = p.k_pages ? (row0 + it.n_rows - 1) / per_seq - first + 1 : 0;
  fill_segments(p, it, seg, err);
  int step0, n_steps;
  run_of(seg.step0[1 + it.n_own], rank * C::NW + (threadIdx.x >> 5), p.cluster * C::NW, step0, n_steps);
  RowState<NR> st;
  attend<T, NR, false>(p, it, smem_dyn, &seg, 0, step0, n_steps, st, err);
  share_results<T, NR>(smem_dyn, st);
  const int x = threadIdx.x >> 3, c8 = (threadIdx.x & 7) * 8;  // 8 threads a row, 8 elements each
  auto put = [&](int row, const float (&v)[8], float l) {
    const int y = it.row_off + row, tok = y / p.r;
    write_out8<T>(p, it.seq0 * p.q_len + tok, it.hk * p.r + y - tok * p.r, c8, v, l, err);
  };
  float v[8], m, l;
  if (x < C::ROWS) {  // (whole warps)
    join_warps<T, NR>(smem_dyn, x, c8, v, m, l);
    redo_if_needed<T, false>(p, it, &seg, 0, [&](int& first, int& n) {
      cta_run<C::NW>(seg.step0[1 + it.n_own], rank * C::NW, p.cluster * C::NW, first, n);
    }, x, c8, v, m, l, err);
  }
  if (p.cluster == 1) {
    if (x < it.n_rows) put(x, v, l);
    return;
  }
  // the CTAs' results over the first warp's; then the ranks share the rows out
  __syncthreads();
  const uint32_t so = smem_u32(smem_dyn), sml = so + C::ML;
  if (x < C::ROWS) {
    float4* d = reinterpret_cast<float4*>(smem_dyn + (x * C::OS + c8) * 4);
    d[0] = make_float4(v[0], v[1], v[2], v[3]);
    d[1] = make_float4(v[4], v[5], v[6], v[7]);
    if (c8 == 0) *reinterpret_cast<float2*>(smem_dyn + C::ML + x * 8) = make_float2(m, l);
  }
  cluster_arrive_wait();
  for (int y = rank + p.cluster * x; y < it.n_rows; y += p.cluster * (C::THREADS / 8)) {
    float2 ml[8];
    m = -CUDART_INF_F;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if (i < p.cluster) {
        ml[i] = ld_cluster_f2(rank_addr(sml + y * 8, i));
        m = fmaxf(m, ml[i].x);
      }
    }
    const float u = m == -CUDART_INF_F ? 0.0f : m;
    l = 0.0f;
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if (i < p.cluster) {
        const float f = ex2_approx(ml[i].x - u);
        const uint32_t a = rank_addr(so + (y * C::OS + c8) * 4, i);
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

__device__ __forceinline__ void write_partial(const PrefixParams& p, int token, int head, int slot, int c8, const float (&v)[8],
                                             float m, float l, uint32_t* err) {
  if (!row_in(p, token, head, err, 90) || !in_bounds(slot >= 0 && slot < p.np + p.ns, err, 90)) return;
  const size_t at = (static_cast<size_t>(token) * p.H + head) * (p.np + p.ns) + slot;
  if (l != 0.0f) {  // (a NaN too: it has to reach the output)
    float4* dst = reinterpret_cast<float4*>(p.part_o + at * HD + c8);
    dst[0] = make_float4(v[0], v[1], v[2], v[3]);
    dst[1] = make_float4(v[4], v[5], v[6], v[7]);
  }
  if (c8 == 0) p.part_ml[at] = make_float2(m, l);
}

// Second form, the prefix: one CTA per (group, key head, split, row tile); writes its rows' partial results.
template <typename T, int NR>
__global__ void __launch_bounds__(Cfg<T, NR>::THREADS, Cfg<T, NR>::CTAS) prefix_part_kernel(const __grid_constant__ PrefixParams p, uint32_t* err) {
  using C = Cfg<T, NR>;
  extern __shared__ __align__(128) uint8_t smem_dyn[];
  __shared__ SegTable seg;
  pdl_trigger();
  pdl_wait();
  int b = blockIdx.x;
  Item it;
  const int row0 = (b % p.row_tiles) * C::ROWS;
  b /= p.row_tiles;
  const int split = b % p.np;
  b /= p.np;
  it.hk = b % p.Hkv;
  const int grp = b / p.Hkv;
  int begin, count;
  group_range(p, grp, begin, count, err);
  it.kp = p.kp + grp * p.k_group + it.hk * C::ROWB;
  it.vp = p.vp + grp * p.v_group + it.hk * C::ROWB;
  it.prefix_len = prefix_len_of(p, grp, err);
  it.n_own = 0;
  it.n_rows = min(count * p.q_len * p.r - row0, C::ROWS);
  if (it.n_rows <= 0) return;
  it.seq0 = begin;
  it.row_off = row0;
  fill_segments(p, it, seg, err);
  int step0, n_steps;
  run_of(seg.step0[1], split * C::NW + (threadIdx.x >> 5), p.np * C::NW, step0, n_steps);
  RowState<NR> st;
  attend<T, NR, false>(p, it, smem_dyn, &seg, 0, step0, n_steps, st, err);
  share_results<T, NR>(smem_dyn, st);
  const int x = threadIdx.x >> 3, c8 = (threadIdx.x & 7) * 8;
  if (x >= C::ROWS) return;  // (whole warps)
  float v[8], m, l;
  join_warps<T, NR>(smem_dyn, x, c8, v, m, l);
  redo_if_needed<T, false>(p, it, &seg, 0, [&](int& first, int& n) { cta_run<C::NW>(seg.step0[1], split * C::NW, p.np * C::NW, first, n); },
                           x, c8, v, m, l, err);
  if (x >= it.n_rows) return;
  const int y = row0 + x, tok = y / p.r;
  write_partial(p, begin * p.q_len + tok, it.hk * p.r + y - tok * p.r, split, c8, v, m, l, err);
}

// (256 sequences x 4 key heads, up to 600 own keys in pages of 64: 20 us for 78 MB; a CTA per item with its warps
// joined was as fast alone but left twice the idle warps behind short sequences, 43.5 against 44.9 us for the call as
// it then was.)
// Second form, own keys: one warp per (sequence, key head, row tile, split); its rows go through the
// warp's stretch of shared memory to full lines of the partial results.
template <typename T, int NR>
__global__ void __launch_bounds__(Cfg<T, NR>::THREADS, Cfg<T, NR>::CTAS) prefix_own_kernel(const __grid_constant__ PrefixParams p, long long n_items,
                                                                                       uint32_t* err) {
  using C = Cfg<T, NR>;
  static_assert(C::STAGES * 2 * C::HALF >= 8 * C::OS * 4, "a warp's ring holds eight rows of results");
  extern __shared__ __align__(128) uint8_t smem_dyn[];
  pdl_trigger();
  // Before the first read, although nothing of the prefix's kernel is read here: only a wait of this grid's own makes
  // the writes of the calls before (new keys, lengths, tables) visible to it.
  pdl_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, tq = lane & 3;
  long long b = static_cast<long long>(blockIdx.x) * C::NW + warp;
  if (b >= n_items) return;
  Item it;
  const int split = static_cast<int>(b % p.ns);
  b /= p.ns;
  const int row0 = static_cast<int>(b % p.row_tiles) * C::ROWS;
  b /= p.row_tiles;
  it.hk = static_cast<int>(b % p.Hkv);
  it.seq0 = static_cast<int>(b / p.Hkv);
  it.n_own = 1;
  it.row_off = row0;
  it.n_rows = min(p.q_len * p.r - row0, C::ROWS);
  // a sequence behind the last group (padding): its length and pages may hold anything, its rows stay as they were
  if (p.np && p.group_start && it.seq0 >= p.group_start[p.n_groups]) return;
  const int len = own_len_of(p, it.seq0, err);
  int step0, n_steps;
  run_of((len + 15) / 16, split, p.ns, step0, n_steps);
  RowState<NR> st;
  attend<T, NR, true>(p, it, smem_dyn, nullptr, len, step0, n_steps, st, err);
  float* so = reinterpret_cast<float*>(smem_dyn + warp * (C::STAGES * 2 * C::HALF));
#pragma unroll
  for (int r = 0; r < NR; ++r) {
    __syncwarp();
#pragma unroll
    for (int e = 0; e < 2; ++e)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        so[(2 * tq + e) * C::OS + (C::F32 ? 4 * g + i : 16 * i + g)] = st.o[r][i][e];
        so[(2 * tq + e) * C::OS + (C::F32 ? 32 + 4 * g + i : 16 * i + g + 8)] = st.o[r][i][e + 2];
      }
    __syncwarp();
    const int c8 = (lane & 7) * 8;
#pragma unroll
    for (int h = 0; h < 2; ++h) {  // four rows at a time, eight lanes each
      const int x = 4 * h + (lane >> 3), y = row0 + 8 * r + x, tok = y / p.r;
      // row x's maximum and sum sit in the lanes of column pair x / 2, element x % 2
      const float m0 = __shfl_sync(0xffffffffu, st.m[r][0], x >> 1), m1 = __shfl_sync(0xffffffffu, st.m[r][1], x >> 1);
      const float l0 = __shfl_sync(0xffffffffu, st.l[r][0], x >> 1), l1 = __shfl_sync(0xffffffffu, st.l[r][1], x >> 1);
      float v[8], m = x & 1 ? m1 : m0, l = x & 1 ? l1 : l0;
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = so[x * C::OS + c8 + e];
      redo_if_needed<T, true>(p, it, nullptr, len, [&](int& first, int& n) { run_of((len + 15) / 16, split, p.ns, first, n); },
                              8 * r + x, c8, v, m, l, err);
      if (8 * r + x < it.n_rows) write_partial(p, it.seq0 * p.q_len + tok, it.hk * p.r + y - tok * p.r, p.np + split, c8, v, m, l, err);
    }
  }
}

// Join of the partial results of one (token, head): sixteen lanes, four elements each.
template <typename T>
__global__ void __launch_bounds__(256) prefix_join_kernel(const PrefixParams p, uint32_t* err) {
  pdl_trigger();
  pdl_wait();
  const long long pair = (static_cast<long long>(blockIdx.x) * blockDim.x + threadIdx.x) >> 4;
  const int c4 = threadIdx.x & 15;
  const long long n_pairs = static_cast<long long>(p.n_seqs) * p.q_len * p.H;
  if (pair >= n_pairs) return;
  const int token = static_cast<int>(pair / p.H), head = static_cast<int>(pair % p.H);
  // rows of no group have no partial results: left as they were
  if (p.np && p.group_start) {
    const int seq = token / p.q_len;
    int lo = 0, hi = p.n_groups;  // the last group that starts at or before seq
    while (hi - lo > 1) {
      const int mid = (lo + hi) / 2;
      if (p.group_start[mid] <= seq) lo = mid;
      else hi = mid;
    }
    const int begin = p.group_start[lo], end = p.group_start[lo + 1];
    if (seq < begin || seq >= end || begin < 0 || end > p.n_seqs || end - begin > p.max_group) return;
  }
  // lane c4 weighs slots c4, c4 + 16, ...; then every lane adds its four elements of all slots, eight
  // loads in flight, the first eight before the weights are known (slots without keys wrote no O: what
  // their memory holds is read but not used)
  const int n = p.np + p.ns;
  const float2* ml = p.part_ml + pair * n;
  const float* po = p.part_o + pair * n * HD + c4 * 4;
  const uint32_t lanes = 0xffffu << (threadIdx.x & 16);  // this row's half of the warp
  float4 o[8];
  auto fetch = [&](int j0) {
#pragma unroll
    for (int j = 0; j < 8; ++j) o[j] = *reinterpret_cast<const float4*>(po + static_cast<size_t>(min(j0 + j, n - 1)) * HD);
  };
  fetch(0);
  float m = -CUDART_INF_F;
  for (int i = c4; i < n; i += 16) m = fmaxf(m, ml[i].x);
#pragma unroll
  for (int d = 1; d < 16; d <<= 1) m = fmaxf(m, __shfl_xor_sync(lanes, m, d));
  const float u = m == -CUDART_INF_F ? 0.0f : m;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  float l = 0.0f;
  for (int i0 = 0; i0 < n; i0 += 16) {
    const float2 x = i0 + c4 < n ? ml[i0 + c4] : make_float2(0.0f, 0.0f);
    const float f = x.y != 0.0f ? ex2_approx(x.x - u) : 0.0f;
    const uint32_t wrote = __ballot_sync(lanes, x.y != 0.0f) >> (threadIdx.x & 16);
    float part = x.y != 0.0f ? f * x.y : 0.0f;
#pragma unroll
    for (int d = 1; d < 16; d <<= 1) part += __shfl_xor_sync(lanes, part, d);
    l += part;
#pragma unroll
    for (int j0 = 0; j0 < 16; j0 += 8) {
      if (i0 + j0 >= n) break;
      if (i0 + j0 > 0) fetch(i0 + j0);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float w = __shfl_sync(lanes, f, j0 + j, 16);
        if ((wrote >> (j0 + j)) & 1u) {
          acc.x += w * o[j].x;
          acc.y += w * o[j].y;
          acc.z += w * o[j].z;
          acc.w += w * o[j].w;
        }
      }
    }
  }
  const float inv = l != 0.0f ? 1.0f / l : 0.0f;
  if (!row_in(p, token, head, err, 91)) return;
  uint8_t* dst = p.out + token * p.out_stride + (head * HD + c4 * 4) * sizeof(T);
  if constexpr (sizeof(T) == 4)
    *reinterpret_cast<float4*>(dst) = make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv);
  else
    *reinterpret_cast<uint2*>(dst) =
        make_uint2(pack_bf16x2(acc.x * inv, acc.y * inv), pack_bf16x2(acc.z * inv, acc.w * inv));
}

wenc_status bad(wenc_status s, const char* fmt, long long a = 0, long long b = 0) {
  char buf[256];
  snprintf(buf, sizeof(buf), fmt, a, b);
  return wenc_internal_fail(s, buf);
}

// How one call is divided, from its sizes alone.
struct Plan {
  int cluster = 0;              // > 0: the one-launch form, CTAs per item
  int nr_p = 0, nr_s = 0;       // groups of 8 rows per tile: prefix (or one-launch) and own-key items
  int rows_p = 0, rows_s = 0;   // row tiles
  int np = 0, ns = 0;           // key splits
  long long items_p = 0, items_s = 0;  // CTAs (one-launch form: items_p; tcgen05 form: work items)
  bool tc = false;              // the prefix runs in prefix_tc.cu (bf16) or prefix_tc32.cu (fp32)
  int tokens = 0;               // its tokens per row tile
  size_t part_o = 0, bytes = 0;  // offset of the (m, l) pairs; workspace bytes
};

// Groups of 8 rows per tile: one or two. More rows take more tiles, which read K and V again from L2: four groups
// a tile leave registers for one CTA an SM (8 windows' 64 rows over 1500 keys 20.1 us, with tiles of 16 rows 13.3;
// 20 rows 23.9 against 10.2).
int row_groups(long long rows) { return rows <= 8 ? 1 : 2; }

// Into how many shares a prefix of `tiles` key tiles is split for `items` row tiles: as the rounds of one CTA an SM
// take the least time, with `start` key tiles of time for what an item costs beside its own.
int split_rounds(long long items, long long tiles, long long start, int sms) {
  int np = 1;
  long long best = 0;
  for (int n = 1; n <= 32 && (n == 1 || n <= tiles); ++n) {
    const long long cost = (items * n + sms - 1) / sms * ((tiles + n - 1) / n + start);
    if (n == 1 || cost < best) {
      best = cost;
      np = n;
    }
  }
  return np;
}
// In key tiles of 128 (prefix_tc.cu: 1 to 4 are alike for 4 groups x 400 rows of 4 key heads over 2000 keys, 17.2 us,
// and for 16 groups x 20 heads x 128 rows over 1500, 82; with 96 rows 1 and 2 take 77, 3 and 4 78.5) and of 64
// (prefix_tc32.cu: 3 to 10 are alike).
constexpr int kTcStart = 2, kTc32Start = 6;

Plan make_plan(const wenc_prefix_attention_args* a, int sms) {
  Plan pl;
  const bool f32 = a->dtype == WENC_DTYPE_F32;
  const int kt = f32 ? 16 * Cfg<float, 1>::NW : 16 * Cfg<__nv_bfloat16, 1>::NW;  // keys of one step of a CTA
  const long long r = a->n_heads / a->n_kv_heads;
  const long long rows_s = a->q_len * r;  // rows of one sequence per key head
  const long long group = a->k_prefix ? a->max_group : 1, n_groups = a->k_prefix ? a->n_groups : a->n_seqs;
  const long long rows = group * rows_s;
  const long long own_cap = a->k_pages ? static_cast<long long>(a->max_pages) * a->page_size : 0;
  const long long prefix = a->k_prefix ? a->prefix_max : 0;
  pl.nr_p = row_groups(rows);
  pl.rows_p = static_cast<int>((rows + 8 * pl.nr_p - 1) / (8 * pl.nr_p));
  // The one-launch form up to 64 rows; with more, while its CTAs fit one round of the machine and the prefix is
  // little work (2^22 pairs of a row and a key; fp32, whose products run as three here, 3 * 2^18). Measured around it
  // (us, one launch / joined; bf16 without own keys): 8 key heads x 256 rows over 2000 keys (4.1 M pairs) 13.7 /
  // 14.9, 384 rows (6.1 M) 20.1 / 14.6, 128 rows over 500 7.1 / 8.6; 4 x 128 over 8000 (4.1 M) 14.1 / 13.4, 4 x 160
  // (5.1 M) 21.5 / 13.8; 20 x 150 over 1500 (4.5 M) 16.3 / 13.8; 2 windows x 20 heads x 128 rows over 1500 (320 CTAs)
  // 25.4 / 16.2; 16 windows x 20 heads x 96 rows 99.3 / 77.0. fp32: 2 key heads x 200 rows over 1500 (0.6 M) 9.5 /
  // 13.9, 8 x 100 over 1000 (0.8 M) 14.9 / 12.9, 2 x 6 heads x 224 over 671 with own keys (1.8 M) 39.1 / 28.4, 8 x
  // 100 over 3000 (2.4 M) 25.8 / 14.8.
  const long long items = n_groups * a->n_kv_heads * pl.rows_p;
  // (fp32 waits on its own instructions: more CTAs than are resident at once still gain, 21.0 against 24.4 us for 4
  // windows x 40 rows)
  const long long round = (f32 || pl.nr_p == 1 ? 3ll : 2ll) * sms;
  const long long little = f32 ? 3ll << 18 : 1ll << 22;
  if (rows <= 64 || (items <= round && n_groups * a->n_kv_heads * rows * prefix <= little)) {
    const long long tiles = (prefix + kt - 1) / kt + group * ((own_cap + kt - 1) / kt);
    // CTAs within one round of the machine, none without a tile of its own
    pl.cluster = 1;
    while (pl.cluster < 8 && pl.cluster < tiles && 2 * items * pl.cluster <= round) pl.cluster *= 2;
    pl.items_p = items * pl.cluster;
    return pl;
  }
  auto splits = [&](long long items, long long keys) {
    const long long tiles = (keys + kt - 1) / kt;
    long long n = (6ll * sms + items - 1) / items;
    if (n > tiles) n = tiles;
    if (n > 32) n = 32;
    return static_cast<int>(n < 1 ? 1 : n);
  };
  // (more than 128 query heads per key head, and in bf16 a negative or zero scale and a group stride of 0, stay
  // with the general form)
  pl.tc = a->k_prefix && r <= 128 &&
          (f32 || (a->scale > 0.0f && (n_groups == 1 || (a->k_group_stride > 0 && a->v_group_stride > 0))));
  if (pl.tc && f32) {
    pl.tokens = static_cast<int>(128 / r);
    pl.rows_p = static_cast<int>((group * a->q_len + pl.tokens - 1) / pl.tokens);
    const long long items = n_groups * a->n_kv_heads * pl.rows_p, tiles = (prefix + 63) / 64;
    pl.np = split_rounds(items, tiles, kTc32Start, sms);
    pl.items_p = items * pl.np;
  } else if (pl.tc) {
    pl.tokens = static_cast<int>(128 / r);
    pl.rows_p = static_cast<int>((group * a->q_len + 2 * pl.tokens - 1) / (2 * pl.tokens));  // pairs of row tiles
    const long long items = n_groups * a->n_kv_heads * pl.rows_p, tiles = (prefix + 127) / 128;
    pl.np = split_rounds(items, tiles, kTcStart, sms);
    pl.items_p = items * pl.np;
  } else if (a->k_prefix) {
    const long long items = n_groups * a->n_kv_heads * pl.rows_p;
    pl.np = splits(items, prefix);
    pl.items_p = items * pl.np;
  }
  if (a->k_pages) {
    pl.nr_s = row_groups(rows_s);
    pl.rows_s = static_cast<int>((rows_s + 8 * pl.nr_s - 1) / (8 * pl.nr_s));
    // warps: within one round of the machine (24 an SM), no split of fewer than 64 keys
    const long long items = static_cast<long long>(a->n_seqs) * a->n_kv_heads * pl.rows_s;
    long long n = 24ll * sms / items;
    if (n > (own_cap + 63) / 64) n = (own_cap + 63) / 64;
    if (n > 32) n = 32;
    pl.ns = static_cast<int>(n < 1 ? 1 : n);
    pl.items_s = items * pl.ns;
  }
  const size_t n = static_cast<size_t>(a->n_seqs) * a->q_len * a->n_heads * (pl.np + pl.ns);
  pl.part_o = n * HD * sizeof(float);
  pl.bytes = pl.part_o + n * sizeof(float2);
  return pl;
}

// Sizes alone (what the plan needs). Returns false with the status set.
bool check_sizes(const wenc_prefix_attention_args* a, wenc_status* st) {
  auto no = [&](wenc_status s, const char* fmt, long long x = 0, long long y = 0) {
    *st = bad(s, fmt, x, y);
    return false;
  };
  if (!a) return no(WENC_ERR_INVALID_ARG, "prefix_attention: args is NULL");
  if (a->dtype != WENC_DTYPE_F32 && a->dtype != WENC_DTYPE_BF16)
    return no(WENC_ERR_INVALID_ARG, "prefix_attention: dtype %lld unknown", a->dtype);
  if (a->head_dim != HD) return no(WENC_ERR_UNSUPPORTED, "head_dim %lld: only 64 is implemented", a->head_dim);
  if (a->n_seqs < 1 || a->q_len < 1 || a->n_heads < 1 || a->n_kv_heads < 1)
    return no(WENC_ERR_INVALID_ARG, "prefix_attention: n_seqs, q_len and the heads must be >= 1");
  if (a->n_heads % a->n_kv_heads != 0)
    return no(WENC_ERR_INVALID_ARG, "prefix_attention: %lld query heads are no multiple of %lld key heads", a->n_heads,
              a->n_kv_heads);
  if (static_cast<long long>(a->n_seqs) * a->q_len > (1ll << 28) || a->n_heads > 4096 ||
      static_cast<long long>(a->n_seqs) * a->q_len * a->n_heads > (1ll << 30))
    return no(WENC_ERR_UNSUPPORTED, "prefix_attention: more than 2^28 tokens, 4096 heads or 2^30 rows of them");
  if (!a->k_prefix && !a->k_pages) return no(WENC_ERR_INVALID_ARG, "prefix_attention: neither prefix nor pages");
  if ((a->k_prefix == nullptr) != (a->v_prefix == nullptr) || (a->k_pages == nullptr) != (a->v_pages == nullptr))
    return no(WENC_ERR_INVALID_ARG, "prefix_attention: keys and values come together");
  if (a->k_prefix) {
    if (a->n_groups < 1 || a->max_group < 1 || a->prefix_max < 1)
      return no(WENC_ERR_INVALID_ARG, "prefix_attention: n_groups, max_group and prefix_max must be >= 1");
    if (a->max_group > a->n_seqs)
      return no(WENC_ERR_INVALID_ARG, "prefix_attention: max_group %lld > n_seqs %lld", a->max_group, a->n_seqs);
    if (!a->group_start && static_cast<long long>(a->n_groups) * a->max_group != a->n_seqs)
      return no(WENC_ERR_INVALID_ARG, "prefix_attention: n_groups * max_group = %lld, but n_seqs = %lld (pass group_start)",
                static_cast<long long>(a->n_groups) * a->max_group, a->n_seqs);
    if (a->prefix_max > (1 << 30)) return no(WENC_ERR_UNSUPPORTED, "prefix_attention: prefix_max %lld > 2^30", a->prefix_max);
  }
  if (a->k_pages) {
    if (a->n_pages < 1 || a->page_size < 1 || a->max_pages < 1)
      return no(WENC_ERR_INVALID_ARG, "prefix_attention: n_pages, page_size and max_pages must be >= 1");
    if (static_cast<long long>(a->max_pages) * a->page_size > (1ll << 30))
      return no(WENC_ERR_UNSUPPORTED, "prefix_attention: max_pages %lld x page_size %lld passes 2^30", a->max_pages,
                a->page_size);
  }
  return true;
}

template <typename K>
cudaError_t opt_in(K kern, uint32_t smem, std::atomic<int>& configured) {
  int dev = 0;
  const cudaError_t e = cudaGetDevice(&dev);
  return e != cudaSuccess ? e : wenc_host::opt_in_smem(kern, smem, dev, configured);
}

template <typename T, int NR>
cudaError_t launch_cluster(const PrefixParams& p, long long blocks, uint32_t* err, cudaStream_t stream) {
  using C = Cfg<T, NR>;
  auto kern = prefix_cluster_kernel<T, NR>;
  static std::atomic<int> configured{-1};
  const cudaError_t e = opt_in(kern, C::SMEM, configured);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(blocks));
  cfg.blockDim = dim3(C::THREADS);
  cfg.dynamicSmemBytes = C::SMEM;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = static_cast<unsigned>(p.cluster);
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = p.cluster > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kern, p, err);
}

template <typename T, int NR>
cudaError_t launch_part(PrefixParams p, int row_tiles, long long blocks, uint32_t* err, cudaStream_t stream) {
  using C = Cfg<T, NR>;
  auto kern = prefix_part_kernel<T, NR>;
  static std::atomic<int> configured{-1};
  const cudaError_t e = opt_in(kern, C::SMEM, configured);
  if (e != cudaSuccess) return e;
  p.row_tiles = row_tiles;
  return wenc_host::launch_pdl(kern, dim3(static_cast<unsigned>(blocks)), dim3(C::THREADS), C::SMEM, stream, p, err);
}

template <typename T, int NR>
cudaError_t launch_own(PrefixParams p, int row_tiles, long long items, uint32_t* err, cudaStream_t stream) {
  using C = Cfg<T, NR>;
  auto kern = prefix_own_kernel<T, NR>;
  static std::atomic<int> configured{-1};
  const cudaError_t e = opt_in(kern, C::RING + C::P_BYTES, configured);
  if (e != cudaSuccess) return e;
  p.row_tiles = row_tiles;
  return wenc_host::launch_pdl(kern, dim3(static_cast<unsigned>((items + C::NW - 1) / C::NW)), dim3(C::THREADS),
                               C::RING + C::P_BYTES, stream, p, items, err);
}

// The prefix part on tcgen05.
wenc_status launch_tc(const wenc_prefix_attention_args* a, const PrefixParams& p, const Plan& pl, uint32_t* err, int sms,
                      cudaStream_t stream) {
  CUtensorMap tq, tk, tv;
  std::string why;
  const uint64_t tokens = static_cast<uint64_t>(a->n_seqs) * a->q_len, cols = static_cast<uint64_t>(a->n_kv_heads) * HD;
  // (with one group its stride may be anything)
  const uint64_t kg = a->n_groups > 1 ? p.k_group : p.k_token * a->prefix_max, vg = a->n_groups > 1 ? p.v_group : p.v_token * a->prefix_max;
  const bool ok =
      wenc_host::make_tmap_3d_bf16_box(&tq, a->q, HD, a->n_heads, tokens, HD * 2, p.q_stride, HD, p.r, pl.tokens, &why) &&
      wenc_host::make_tmap_3d_bf16(&tk, a->k_prefix, cols, a->prefix_max, a->n_groups, p.k_token, kg, HD, 128, &why) &&
      wenc_host::make_tmap_3d_bf16(&tv, a->v_prefix, cols, a->prefix_max, a->n_groups, p.v_token, vg, HD, 128, &why);
  if (!ok) return wenc_internal_fail(WENC_ERR_INVALID_ARG, why.c_str());
  wenc_host::PrefixTcArgs t;
  t.group_start = p.group_start;
  t.prefix_lens = p.prefix_lens;
  t.n_seqs = p.n_seqs;
  t.q_len = p.q_len;
  t.H = p.H;
  t.Hkv = p.Hkv;
  t.r = p.r;
  t.max_group = p.max_group;
  t.prefix_max = p.prefix_max;
  t.tokens = pl.tokens;
  t.n_x = pl.rows_p;
  t.np = pl.np;
  t.n_items = static_cast<int>(pl.items_p);
  t.n_slots = pl.np + pl.ns;
  t.scale_log2 = p.scale_log2;
  t.part_o = p.part_o;
  t.part_ml = p.part_ml;
  const cudaError_t e = wenc_host::launch_prefix_tc(tq, tk, tv, t, err, sms, stream);
  if (e != cudaSuccess) {
    char buf[200];
    snprintf(buf, sizeof(buf), "prefix_attention launch: %s", cudaGetErrorString(e));
    return wenc_internal_fail(WENC_ERR_CUDA, buf);
  }
  return WENC_OK;
}

// The fp32 prefix part on tcgen05.
wenc_status launch_tc32(const PrefixParams& p, const Plan& pl, uint32_t* err, cudaStream_t stream) {
  wenc_host::PrefixTc32Args t;
  t.q = p.q;
  t.kp = p.kp;
  t.vp = p.vp;
  t.q_stride = p.q_stride;
  t.k_group = p.k_group;
  t.k_token = p.k_token;
  t.v_group = p.v_group;
  t.v_token = p.v_token;
  t.group_start = p.group_start;
  t.prefix_lens = p.prefix_lens;
  t.n_seqs = p.n_seqs;
  t.q_len = p.q_len;
  t.H = p.H;
  t.Hkv = p.Hkv;
  t.r = p.r;
  t.max_group = p.max_group;
  t.prefix_max = p.prefix_max;
  t.tokens = pl.tokens;
  t.n_x = pl.rows_p;
  t.np = pl.np;
  t.n_items = static_cast<int>(pl.items_p);
  t.n_slots = pl.np + pl.ns;
  t.scale_log2 = p.scale_log2;
  t.q_flip = p.q_flip;
  t.q_keep = p.q_keep;
  t.part_o = p.part_o;
  t.part_ml = p.part_ml;
  const cudaError_t e = wenc_host::launch_prefix_tc32(t, err, stream);
  if (e != cudaSuccess) {
    char buf[200];
    snprintf(buf, sizeof(buf), "prefix_attention launch: %s", cudaGetErrorString(e));
    return wenc_internal_fail(WENC_ERR_CUDA, buf);
  }
  return WENC_OK;
}

template <typename T>
cudaError_t launch_all(PrefixParams p, const Plan& pl, uint32_t* err, cudaStream_t stream) {
  if (pl.cluster > 0) {
    p.row_tiles = pl.rows_p;
    return pl.nr_p == 1 ? launch_cluster<T, 1>(p, pl.items_p, err, stream) : launch_cluster<T, 2>(p, pl.items_p, err, stream);
  }
  cudaError_t e = cudaSuccess;
  if (pl.items_p > 0 && !pl.tc) e = launch_part<T, 2>(p, pl.rows_p, pl.items_p, err, stream);
  if (e == cudaSuccess && pl.items_s > 0) {
    e = pl.nr_s == 1 ? launch_own<T, 1>(p, pl.rows_s, pl.items_s, err, stream) : launch_own<T, 2>(p, pl.rows_s, pl.items_s, err, stream);
  }
  if (e != cudaSuccess) return e;
  const long long threads = static_cast<long long>(p.n_seqs) * p.q_len * p.H * 16;
  return wenc_host::launch_pdl(prefix_join_kernel<T>, dim3(static_cast<unsigned>((threads + 255) / 256)), dim3(256), 0,
                               stream, p, err);
}

}  // namespace

extern "C" size_t wenc_prefix_attention_workspace(const wenc_prefix_attention_args* a) {
  wenc_internal_clear_error();
  wenc_status st;
  if (!check_sizes(a, &st)) return 0;
  return make_plan(a, wenc_internal_sm_count()).bytes;
}

extern "C" wenc_status wenc_prefix_attention(const wenc_prefix_attention_args* a, wenc_stream_t stream) {
  wenc_internal_clear_error();
  wenc_status st;
  if (!check_sizes(a, &st)) return st;
  if (!a->q || !a->out) return bad(WENC_ERR_INVALID_ARG, "prefix_attention: q or out is NULL");
  if (a->k_pages && (!a->block_table || !a->lens))
    return bad(WENC_ERR_INVALID_ARG, "prefix_attention: pages need block_table and lens");
  const long long es = a->dtype == WENC_DTYPE_F32 ? 4 : 2, per16 = 16 / es;
  const long long q_row = static_cast<long long>(a->n_heads) * HD, kv_row = static_cast<long long>(a->n_kv_heads) * HD;
  if (a->q_stride < q_row || a->out_stride < q_row)
    return bad(WENC_ERR_INVALID_ARG, "prefix_attention: a token stride of q or out is smaller than its heads");
  if (a->k_prefix && (a->k_token_stride < kv_row || a->v_token_stride < kv_row || a->k_group_stride < 0 || a->v_group_stride < 0))
    return bad(WENC_ERR_INVALID_ARG, "prefix_attention: a prefix stride is smaller than its heads");
  if (a->k_pages && (a->k_page_stride < kv_row * a->page_size || a->v_page_stride < kv_row * a->page_size))
    return bad(WENC_ERR_INVALID_ARG, "prefix_attention: a page stride is smaller than a page");
  if (a->k_pages && a->n_seqs > 1 && a->block_table_stride < a->max_pages)
    return bad(WENC_ERR_INVALID_ARG, "prefix_attention: block_table_stride %lld < max_pages %lld", a->block_table_stride,
               a->max_pages);
  if (a->k_pages && (a->k_page_stride / per16 > 0xffffffffll || a->v_page_stride / per16 > 0xffffffffll))
    return bad(WENC_ERR_UNSUPPORTED, "prefix_attention: a page stride passes 2^36 bytes");
  const void* ptrs[] = {a->q, a->out, a->k_prefix, a->v_prefix, a->k_pages, a->v_pages};
  for (const void* x : ptrs)
    if (reinterpret_cast<uintptr_t>(x) & 15u) return bad(WENC_ERR_INVALID_ARG, "buffers must be 16-byte aligned");
  const long long zero = 0;
  const long long strides[] = {a->q_stride, a->out_stride,
                               a->k_prefix ? a->k_group_stride : zero, a->k_prefix ? a->k_token_stride : zero,
                               a->k_prefix ? a->v_group_stride : zero, a->k_prefix ? a->v_token_stride : zero,
                               a->k_pages ? a->k_page_stride : zero, a->k_pages ? a->v_page_stride : zero};
  for (long long x : strides)
    if (x % per16 != 0) return bad(WENC_ERR_INVALID_ARG, "strides must be multiples of 16 bytes");
  int sms = 0;
  uint32_t* err = nullptr;
  const wenc_status dst = wenc_internal_device(&sms, &err);
  if (dst != WENC_OK) return dst;
  const Plan pl = make_plan(a, sms);
  if (pl.items_p > 0x7fffffffll || pl.items_s > 0x7fffffffll)
    return bad(WENC_ERR_UNSUPPORTED, "prefix_attention: %lld work items pass 2^31 - 1", pl.items_p > pl.items_s ? pl.items_p : pl.items_s);
  if (pl.bytes > 0 && (!a->workspace || a->workspace_bytes < pl.bytes))
    return bad(WENC_ERR_INVALID_ARG, "prefix_attention: workspace of %lld bytes needed, %lld given", static_cast<long long>(pl.bytes),
               a->workspace ? static_cast<long long>(a->workspace_bytes) : 0ll);
  if (pl.bytes > 0 && (reinterpret_cast<uintptr_t>(a->workspace) & 255u))
    return bad(WENC_ERR_INVALID_ARG, "prefix_attention: the workspace must be 256-byte aligned");

  PrefixParams p = {};
  p.q = static_cast<const uint8_t*>(a->q);
  p.out = static_cast<uint8_t*>(a->out);
  p.q_stride = a->q_stride * es;
  p.out_stride = a->out_stride * es;
  p.n_seqs = a->n_seqs;
  p.q_len = a->q_len;
  p.H = a->n_heads;
  p.Hkv = a->n_kv_heads;
  p.r = a->n_heads / a->n_kv_heads;
  if (a->k_prefix) {
    p.kp = static_cast<const uint8_t*>(a->k_prefix);
    p.vp = static_cast<const uint8_t*>(a->v_prefix);
    p.k_group = a->k_group_stride * es;
    p.k_token = a->k_token_stride * es;
    p.v_group = a->v_group_stride * es;
    p.v_token = a->v_token_stride * es;
    p.group_start = a->group_start;
    p.prefix_lens = a->prefix_lens;
    p.n_groups = a->n_groups;
    p.max_group = a->max_group;
    p.prefix_max = a->prefix_max;
  }
  if (a->k_pages) {
    p.k_pages = static_cast<const uint8_t*>(a->k_pages);
    p.v_pages = static_cast<const uint8_t*>(a->v_pages);
    p.k_page16 = static_cast<uint32_t>(a->k_page_stride / per16);
    p.v_page16 = static_cast<uint32_t>(a->v_page_stride / per16);
    p.row16 = static_cast<uint32_t>(kv_row / per16);
    p.table = a->block_table;
    p.table_stride = a->block_table_stride;
    p.lens = a->lens;
    p.n_pages = a->n_pages;
    p.page_size = a->page_size;
    p.max_pages = a->max_pages;
    p.page_shift = -1;
    for (int s = 0; s < 31; ++s)
      if (a->page_size == 1 << s) p.page_shift = s;
  }
  if (!a->k_prefix) {  // every sequence a group of its own
    p.n_groups = a->n_seqs;
    p.max_group = 1;
  }
  p.np = pl.np;
  p.ns = pl.ns;
  p.cluster = pl.cluster;
  // |scale| and the queries' signs; a scale of 0 is 1 on queries of 0
  const bool bf = a->dtype == WENC_DTYPE_BF16;
  p.q_flip = a->scale < 0.0f ? (bf ? 0x80008000u : 0x80000000u) : 0u;
  p.q_keep = a->scale == 0.0f ? 0u : 0xffffffffu;
  p.scale_log2 = (a->scale == 0.0f ? 1.0f : a->scale < 0.0f ? -a->scale : a->scale) * 1.4426950408889634f;
  p.part_o = static_cast<float*>(a->workspace);
  p.part_ml = reinterpret_cast<float2*>(static_cast<uint8_t*>(a->workspace) + pl.part_o);
  if (pl.tc) {
    st = bf ? launch_tc(a, p, pl, err, sms, reinterpret_cast<cudaStream_t>(stream))
            : launch_tc32(p, pl, err, reinterpret_cast<cudaStream_t>(stream));
    if (st != WENC_OK) return st;
  }
  const cudaError_t e = a->dtype == WENC_DTYPE_F32
                            ? launch_all<float>(p, pl, err, reinterpret_cast<cudaStream_t>(stream))
                            : launch_all<__nv_bfloat16>(p, pl, err, reinterpret_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) {
    char buf[200];
    snprintf(buf, sizeof(buf), "prefix_attention launch: %s", cudaGetErrorString(e));
    return wenc_internal_fail(WENC_ERR_CUDA, buf);
  }
  return WENC_OK;
}
