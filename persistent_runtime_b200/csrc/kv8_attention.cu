// mk_kv8_attention: attention of a few new rows per sequence over an 8-bit
// paged cache.
//
// Mathematics.  For the query rows r of one kv head (rep heads x n new tokens)
// and the positions p of a sequence:  x_pr = f_r sk_p (k_p . q'_r) with the
// codes k_p as they are, q' = q 2^-e in fp16 (e from the row's largest
// element), f_r = scale log2(e) 2^e and sk_p the scale of p's block; an online
// softmax in base 2 over chunks of kChunk positions; o_r = sum over blocks of
// sv (sum over the block's p of P_pr v_p), so that codes and probabilities
// meet in the tensor cores and the block's scale multiplies an fp32 partial
// sum.  P carries a factor 2^14, which keeps fp16 normal down to 2^-28 of the
// largest probability and cancels against the sum.
//
// What bounds it: the cache is read once, one byte per element, and every
// element takes part in 2 x rows multiply-adds, far below the tensor rate for
// the rows of a decode step: the bound is HBM.  CUDA cores would need rows + 1
// instructions per byte (at 4 heads per kv head that alone is the SM's issue
// rate at the HBM rate), so both products run on mma.sync m16n8k16 (fp16 in,
// fp32 accumulate) with the positions (QK) and the head's dims (PV) as the 16
// rows and 8 query rows as columns: the rows of a decode step fill one column
// tile, where the 128-row tile of tcgen05 would be 15/16 empty and would need
// the codes expanded into shared memory first.
//
// Layout.  The sum over dims may take the dims in any order, so a lane feeds
// its QK fragments from the 16 bytes it loaded itself; for PV a lane holds 16
// (D / 8) dims of four positions.  A lane therefore consumes exactly the bytes
// that it copied: every warp runs its own ring of kStages chunks filled by
// cp.async with no barrier, and shared memory reads are conflict-free whatever
// the page layout.  Positions past the end are filled with zeros by the copy.
//
// Work split.  The (sequence, kv head, row group) pairs, each with
// ceil(length / kChunk) chunks, lie end to end on one line that the grid cuts
// into equal pieces, from the device's own lengths; a pair that crosses a cut
// leaves partial results (o, max, sum) in the workspace and a second, small
// launch adds them up in a fixed order.  Where the page table is so short that
// a pair is at most kPairChunks chunks, a CTA takes one whole pair instead and
// the second launch is left out.
#include <cuda_fp16.h>
#include <cuda_bf16.h>
#include <cuda_fp8.h>

#include <algorithm>
#include <atomic>

#include "kv8.cuh"

namespace mk {
namespace {

constexpr int kWarps = 8;
constexpr int kThreads = kWarps * 32;
constexpr int kChunk = 32;            // positions of a warp's step
constexpr int kTiles = kChunk / 16;   // 16-position MMA tiles of a chunk
constexpr int kStages = 3;            // chunks in a warp's ring
constexpr int kPairChunks = 16;       // longest pair (in chunks) that one CTA takes whole
constexpr int kMinUnits = 4;          // shortest piece (in chunks) of the cut line
constexpr float kPShift = 14.0f;      // log2 of the factor that P carries
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

// How the query rows fill the MMA columns: 8 rows of a 16-bit type, 16 rows of
// a 16-bit type (two column tiles), 8 rows of fp32 (a tile of high terms and
// one of low terms).
enum Mode { kRows8 = 0, kRows16 = 1, kRows8F32 = 2 };

struct AttnArgs {
  mk_kv8_cache c;
  mk_batch b;
  mk_rows q;
  void *out;
  float *lse;
  int layer, n_q_heads, rep;
  float scale;
  int block_log2;
  int pair_mode;  // a CTA takes the pair blockIdx.x, nothing is cut
  int groups;     // pair mode: row groups of max_rows rows
  int4 *head;     // [CTAs][2] the cut pair that begins in each CTA
  float *ml;      // [2 CTAs][rows][2] max, sum of the partial results
  float *part;    // [2 CTAs][rows][D] their unnormalised outputs
  const int32_t *gate;
};

constexpr int group_rows(int mode) { return mode == kRows16 ? 16 : 8; }

// Shared memory of a warp's ring stage: K codes, V codes, K and V scales.
__host__ __device__ constexpr int stage_bytes(int D) { return 2 * kChunk * D + 32; }
__host__ __device__ constexpr int ring_bytes(int D) { return kWarps * kStages * stage_bytes(D); }
__host__ __device__ constexpr int merge_bytes(int D, int rows) { return kWarps * rows * (D + 4) * 4; }
__host__ __device__ constexpr int smem_bytes(int D, int mode) {
  return (ring_bytes(D) > merge_bytes(D, group_rows(mode)) ? ring_bytes(D)
                                                           : merge_bytes(D, group_rows(mode)));
}

template <int BYTES>
__device__ __forceinline__ void cp_async(uint32_t dst, const void *src, bool on) {
  const int n = on ? BYTES : 0;  // 0 bytes: the destination is filled with zeros
  if constexpr (BYTES == 16)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n));
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(dst), "l"(src), "n"(BYTES), "r"(n));
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                        uint32_t a3, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// 8 x 8 b16 matrix across the warp, transposed.
__device__ __forceinline__ uint32_t transpose8x8(uint32_t v) {
  uint32_t r;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
  return r;
}

__device__ __forceinline__ float exp2_fast(float x) {  // 2 ulp; results below 2^-126 become 0
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ uint32_t half2_bits(float a, float b) {
  const __half2 h = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t *>(&h);
}

__device__ __forceinline__ uint32_t hsub2_bits(uint32_t a, uint32_t b) {
  const __half2 r = __hsub2(*reinterpret_cast<const __half2 *>(&a), *reinterpret_cast<const __half2 *>(&b));
  return *reinterpret_cast<const uint32_t *>(&r);
}

// Codes to fp16 pairs, exactly.  int8: 0x6400 | (code ^ 0x80) is the fp16
// number 1024 + 128 + code, from which 1152 is taken away again.
// Word w (4 codes) -> (code 0, code 1), (code 2, code 3).
template <int FMT>
__device__ __forceinline__ void expand(uint32_t w, uint32_t &lo, uint32_t &hi) {
  if constexpr (FMT == MK_KV8_INT8) {
    w ^= 0x80808080u;
    lo = hsub2_bits(__byte_perm(w, 0x64646464u, 0x4140), 0x64806480u);
    hi = hsub2_bits(__byte_perm(w, 0x64646464u, 0x4342), 0x64806480u);
  } else {
    asm("{.reg .b16 a, b; mov.b32 {a, b}, %2; cvt.rn.f16x2.e4m3x2 %0, a; cvt.rn.f16x2.e4m3x2 %1, b;}"
        : "=r"(lo), "=r"(hi)
        : "r"(w));
  }
}

// Words a, b (4 codes of two positions) -> (a_i, b_i) for i = 0 .. 3.
template <int FMT>
__device__ __forceinline__ void expand_pairs(uint32_t a, uint32_t b, uint32_t (&h)[4]) {
  const uint32_t p = __byte_perm(a, b, 0x5140), q = __byte_perm(a, b, 0x7362);
  expand<FMT>(p, h[0], h[1]);
  expand<FMT>(q, h[2], h[3]);
}

__device__ __forceinline__ void load_q16(const mk_rows &q, int64_t at, float (&x)[16]) {
  if (q.dtype == MK_F32) {
    const float4 *p = reinterpret_cast<const float4 *>(static_cast<const float *>(q.data) + at);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float4 v = p[i];
      x[4 * i] = v.x; x[4 * i + 1] = v.y; x[4 * i + 2] = v.z; x[4 * i + 3] = v.w;
    }
  } else {
    const uint4 *p = reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(q.data) + at);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint4 v = p[i];
      const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        float2 f;
        if (q.dtype == MK_BF16)
          f = make_float2(__uint_as_float(u[j] << 16), __uint_as_float(u[j] & 0xffff0000u));
        else
          f = __half22float2(*reinterpret_cast<const __half2 *>(&u[j]));
        x[8 * i + 2 * j] = f.x;
        x[8 * i + 2 * j + 1] = f.y;
      }
    }
  }
}

__device__ __forceinline__ void store_out(void *out, int dtype, int64_t at, float v) {
  if (dtype == MK_F32) static_cast<float *>(out)[at] = v;
  else if (dtype == MK_BF16) static_cast<__nv_bfloat16 *>(out)[at] = __float2bfloat16_rn(v);
  else static_cast<__half *>(out)[at] = __float2half_rn(v);
}

// Chunks [k0, k1) of pair (sequence q.s, kv head hk, row group g) by one CTA;
// `whole`: they are all of it and the result is final, else it goes to
// partial slot `slot`.
template <int D, int FMT, int MODE>
__device__ __forceinline__ void run_segment(const AttnArgs &a, uint8_t *smem, const SeqRows &q,
                                            int hk, int g, int k0, int k1, bool whole, int slot) {
  constexpr int RG = group_rows(MODE);
  constexpr int NS = MODE == kRows8 ? 1 : 2;   // column tiles of the scores' MMAs
  constexpr int NO = MODE == kRows16 ? 2 : 1;  // column tiles of the outputs
  constexpr int NC = D / 64;                   // 64-dim halves of a row
  constexpr int VB = D / 8;                    // bytes of a V row that a lane holds
  constexpr int NM = D / 16;                   // 16-dim m-tiles of the output
  __shared__ float sh_m[kWarps][RG], sh_l[kWarps][RG];
  __shared__ int sh_bad;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int gq = lane >> 2, t = lane & 3;
  const int P = a.c.page_size, rep = a.rep, n_rows = rep * q.n;
  const int end = q.c + q.n;  // positions of the sequence, its new rows included
  if (threadIdx.x == 0) sh_bad = 0;

  // --- copies: the warp's i-th chunk is chunk k0 + warp + i kWarps ---------
  uint8_t *ring = smem + warp * kStages * stage_bytes(D);
  const uint32_t ring_u32 = (uint32_t)__cvta_generic_to_shared(ring);
  const int n_mine = k1 - k0 > warp ? (k1 - k0 - warp + kWarps - 1) / kWarps : 0;
  constexpr int kLook = 32 / kTiles;  // chunks whose pages one lookup (one tile per lane) covers
  const int32_t *table = a.b.d_page_table + (int64_t)q.s * a.b.max_pages;
  bool bad_page = false;
  auto tile_pos = [&](int i0) {  // position of this lane's tile of the lookup at chunk i0
    return (k0 + warp + (i0 + lane / kTiles) * kWarps) * kChunk + (lane % kTiles) * 16;
  };
  auto look = [&](int i0) {
    const int pos = tile_pos(i0);
    return i0 + lane / kTiles < n_mine && pos < end ? table[pos / P] : 0;
  };
  auto tile_row = [&](int i0, int page) -> int64_t {  // row of the pool where the tile begins
    const int pos = tile_pos(i0);
    if (i0 + lane / kTiles >= n_mine || pos >= end) return 0;
    if (page < 0 || page >= a.c.n_pages) {
      bad_page = true;
      record_status(a.c.d_status, MK_ERR_DEVICE, q.s, page, MK_CHECK_PAGE);
      return 0;
    }
    return kv8_slab(a.c, a.layer, page, hk) * P + pos % P;
  };
  int page_next = look(0);
  int64_t rows = 0;
  auto issue = [&](int i) {
    if (i < n_mine) {
      if (i % kLook == 0) {
        rows = tile_row(i, page_next);
        page_next = look(i + kLook);
      }
      const uint32_t st = ring_u32 + (i % kStages) * stage_bytes(D);
      const int pos0 = (k0 + warp + i * kWarps) * kChunk;
      const int from = (i % kLook) * kTiles;
      int64_t at[kTiles];
#pragma unroll
      for (int tl = 0; tl < kTiles; ++tl) at[tl] = __shfl_sync(0xffffffffu, rows, from + tl);
      const uint8_t *kp = static_cast<const uint8_t *>(a.c.d_k);
      const uint8_t *vp = static_cast<const uint8_t *>(a.c.d_v);
#pragma unroll
      for (int tl = 0; tl < kTiles; ++tl) {
        const int left = end - pos0 - 16 * tl;  // rows of the tile that exist
#pragma unroll
        for (int c = 0; c < NC; ++c)
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            const int row = gq + 8 * r;
            cp_async<16>(st + ((tl * NC + c) * 2 + r) * 512 + lane * 16,
                         kp + (at[tl] + row) * D + c * 64 + t * 16, row < left);
          }
      }
      if (lane < 2 * kTiles) {
        // lanes 0 .. kTiles-1: K scales, kTiles .. 2 kTiles-1: V scales
        const int tl = lane % kTiles;
        const float *sp = lane < kTiles ? a.c.d_k_scale : a.c.d_v_scale;
        int64_t r = at[0];  // also for a tile past the end: it may share the first one's block
#pragma unroll
        for (int j = 1; j < kTiles; ++j) r = tl == j && pos0 + 16 * j < end ? at[j] : r;
        cp_async<4>(st + 2 * kChunk * D + lane * 4, sp + (r >> a.block_log2), true);
      }
      cp_commit();
#pragma unroll
      for (int tl = 0; tl < kTiles; ++tl) {
        const int left = end - pos0 - 16 * tl;
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const int row = 2 * t + (r & 1) + (r >> 1) * 8;
          cp_async<VB>(st + kChunk * D + (tl * 4 + r) * (32 * VB) + lane * VB,
                       vp + (at[tl] + row) * D + gq * VB, row < left);
        }
      }
      cp_commit();
    } else {
      cp_commit();
      cp_commit();
    }
  };
#pragma unroll
  for (int i = 0; i < kStages - 1; ++i) issue(i);

  // --- query rows: column gq of column tile j is row g RG + 8 j + gq --------
  uint32_t qf[NS][NC * 4][2];
  float fq[NO];  // f of this lane's row, then of its two columns
  int lim[NO];
#pragma unroll
  for (int j = 0; j < NO; ++j) {
    const int r = g * RG + 8 * j + gq;
    const bool on = r < n_rows;
    const int i = on ? r / rep : 0;
    float x[NC][16];
    float top = 0.0f;
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      if (on) {
        load_q16(a.q, (int64_t)(q.r0 + i) * a.q.row_stride + (int64_t)(hk * rep + r % rep) * a.q.head_stride + c * 64 + t * 16, x[c]);
      } else {
#pragma unroll
        for (int d = 0; d < 16; ++d) x[c][d] = 0.0f;
      }
#pragma unroll
      for (int d = 0; d < 16; ++d) top = fmaxf(top, fabsf(x[c][d]));
    }
    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
    const int e = (int)(__float_as_uint(top) >> 23) - 126;  // |q| < 2^e
    const float shrink = ldexpf(1.0f, -e);
    fq[j] = ldexpf(a.scale * kLog2e, e);
    lim[j] = on ? q.c + i + 1 : 0;
#pragma unroll
    for (int c = 0; c < NC; ++c)
#pragma unroll
      for (int w = 0; w < 4; ++w)
#pragma unroll
        for (int p = 0; p < 2; ++p) {
          const float y0 = x[c][4 * w + 2 * p] * shrink, y1 = x[c][4 * w + 2 * p + 1] * shrink;
          const uint32_t hi = half2_bits(y0, y1);
          qf[j][c * 4 + w][p] = hi;
          if constexpr (MODE == kRows8F32) {
            // the low term carries a factor 2^11, so that it keeps its bits
            const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&hi));
            qf[1][c * 4 + w][p] = half2_bits((y0 - f.x) * 2048.0f, (y1 - f.y) * 2048.0f);
          }
        }
  }
  // columns 2 t, 2 t + 1 of a column tile: what the lanes of rows 2 t, 2 t + 1 hold
  float f[NO][2];
  int limit[NO][2];
  int least = end;  // positions below it are seen by every row
#pragma unroll
  for (int j = 0; j < NO; ++j)
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      f[j][c] = __shfl_sync(0xffffffffu, fq[j], (2 * t + c) * 4);
      limit[j][c] = __shfl_sync(0xffffffffu, lim[j], (2 * t + c) * 4);
    }
  least = q.c + (g * RG) / rep + 1;  // the group's first row sees the fewest

  // --- the warp's chunks ------------------------------------------------------
  float o[NO][NM][4];
  float m[NO][2], l[NO][2];
#pragma unroll
  for (int j = 0; j < NO; ++j) {
#pragma unroll
    for (int i = 0; i < NM; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[j][i][e] = 0.0f;
    m[j][0] = m[j][1] = -INFINITY;
    l[j][0] = l[j][1] = 0.0f;
  }
  for (int i = 0; i < n_mine; ++i) {
    __syncwarp();  // the previous chunk's scales have been read
    issue(i + kStages - 1);
    const uint8_t *st = ring + (i % kStages) * stage_bytes(D);
    const int pos0 = (k0 + warp + i * kWarps) * kChunk;
    cp_wait<2 * kStages - 1>();
    __syncwarp();
    float x[kTiles][NO][4];
    const float *scales = reinterpret_cast<const float *>(st + 2 * kChunk * D);
#pragma unroll
    for (int tl = 0; tl < kTiles; ++tl) {
      float s[NS][4];
#pragma unroll
      for (int j = 0; j < NS; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) s[j][e] = 0.0f;
#pragma unroll
      for (int c = 0; c < NC; ++c) {
        const uint4 r0 = *reinterpret_cast<const uint4 *>(st + ((tl * NC + c) * 2) * 512 + lane * 16);
        const uint4 r1 = *reinterpret_cast<const uint4 *>(st + ((tl * NC + c) * 2 + 1) * 512 + lane * 16);
        const uint32_t w0[4] = {r0.x, r0.y, r0.z, r0.w}, w1[4] = {r1.x, r1.y, r1.z, r1.w};
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          uint32_t a0, a1, a2, a3;
          expand<FMT>(w0[w], a0, a2);
          expand<FMT>(w1[w], a1, a3);
#pragma unroll
          for (int j = 0; j < NS; ++j)
            mma_f16(s[j], a0, a1, a2, a3, qf[j][c * 4 + w][0], qf[j][c * 4 + w][1]);
        }
      }
      const float ks = scales[tl];
#pragma unroll
      for (int j = 0; j < NO; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          float v = s[j][e];
          if constexpr (MODE == kRows8F32) v = fmaf(s[1][e], 1.0f / 2048.0f, v);
          x[tl][j][e] = v * (ks * f[j][e & 1]);
        }
    }
    if (pos0 + kChunk > least) {  // some row does not see all of the chunk
#pragma unroll
      for (int tl = 0; tl < kTiles; ++tl)
#pragma unroll
        for (int j = 0; j < NO; ++j)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (pos0 + 16 * tl + gq + (e >> 1) * 8 >= limit[j][e & 1]) x[tl][j][e] = -INFINITY;
    }
    // a new maximum is rare once a few chunks have passed: all lanes are
    // asked before any shuffles
    float mx[NO][2];
    bool grew = false;
#pragma unroll
    for (int j = 0; j < NO; ++j)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        float v = fmaxf(x[0][j][c], x[0][j][c + 2]);
#pragma unroll
        for (int tl = 1; tl < kTiles; ++tl) v = fmaxf(v, fmaxf(x[tl][j][c], x[tl][j][c + 2]));
        mx[j][c] = v;
        grew |= v > m[j][c];
      }
    if (__any_sync(0xffffffffu, grew)) {
#pragma unroll
      for (int j = 0; j < NO; ++j) {
        float by[2];
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          float v = mx[j][c];
#pragma unroll
          for (int d = 4; d < 32; d <<= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, d));
          v = fmaxf(v, m[j][c]);
          by[c] = v == -INFINITY ? 1.0f : exp2_fast(m[j][c] - v);
          m[j][c] = v;
          l[j][c] *= by[c];
        }
#pragma unroll
        for (int i2 = 0; i2 < NM; ++i2)
#pragma unroll
          for (int e = 0; e < 4; ++e) o[j][i2][e] *= by[e & 1];
      }
    }
    // probabilities, as the B fragments of the second product
    uint32_t pf[kTiles][NS][2];
#pragma unroll
    for (int j = 0; j < NO; ++j) {
      float ref[2];
#pragma unroll
      for (int c = 0; c < 2; ++c) ref[c] = m[j][c] == -INFINITY ? 0.0f : m[j][c] - kPShift;
#pragma unroll
      for (int tl = 0; tl < kTiles; ++tl)
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          const float p0 = exp2_fast(x[tl][j][2 * r] - ref[0]), p1 = exp2_fast(x[tl][j][2 * r + 1] - ref[1]);
          l[j][0] += p0;
          l[j][1] += p1;
          const uint32_t hi = half2_bits(p0, p1);
          pf[tl][j][r] = transpose8x8(hi);
          if constexpr (MODE == kRows8F32) {
            const float2 h = __half22float2(*reinterpret_cast<const __half2 *>(&hi));
            pf[tl][1][r] = transpose8x8(half2_bits(p0 - h.x, p1 - h.y));
          }
        }
    }
    cp_wait<2 * kStages - 2>();
    __syncwarp();
    float part[NO][NM][4];
#pragma unroll
    for (int j = 0; j < NO; ++j)
#pragma unroll
      for (int i2 = 0; i2 < NM; ++i2)
#pragma unroll
        for (int e = 0; e < 4; ++e) part[j][i2][e] = 0.0f;
#pragma unroll
    for (int tl = 0; tl < kTiles; ++tl) {
      uint32_t vw[4][VB / 4];
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const uint8_t *vp = st + kChunk * D + (tl * 4 + r) * (32 * VB) + lane * VB;
        if constexpr (VB == 16) {
          const uint4 u = *reinterpret_cast<const uint4 *>(vp);
          vw[r][0] = u.x; vw[r][1] = u.y; vw[r][2] = u.z; vw[r][3] = u.w;
        } else {
          const uint2 u = *reinterpret_cast<const uint2 *>(vp);
          vw[r][0] = u.x; vw[r][1] = u.y;
        }
      }
#pragma unroll
      for (int w = 0; w < VB / 4; ++w) {
        uint32_t h0[4], h1[4];  // (positions 2 t, 2 t + 1) and (2 t + 8, 2 t + 9) of four dims
        expand_pairs<FMT>(vw[0][w], vw[1][w], h0);
        expand_pairs<FMT>(vw[2][w], vw[3][w], h1);
#pragma unroll
        for (int p = 0; p < 2; ++p)
#pragma unroll
          for (int j = 0; j < NO; ++j) {
            mma_f16(part[j][2 * w + p], h0[2 * p], h0[2 * p + 1], h1[2 * p], h1[2 * p + 1],
                    pf[tl][j][0], pf[tl][j][1]);
            if constexpr (MODE == kRows8F32)
              mma_f16(part[j][2 * w + p], h0[2 * p], h0[2 * p + 1], h1[2 * p], h1[2 * p + 1],
                      pf[tl][1][0], pf[tl][1][1]);
          }
      }
      const int pos = pos0 + 16 * tl;
      if (tl == kTiles - 1 || ((pos + 16) & (a.c.block - 1)) == 0) {
        // the end of the chunk's part of a scale block.  Its scale may be NaN
        // (not finite rows): it must not reach rows that see nothing of it.
        const float vs = scales[kTiles + tl];
        const int begin = pos & ~(a.c.block - 1);
#pragma unroll
        for (int j = 0; j < NO; ++j) {
          const float v[2] = {begin < limit[j][0] ? vs : 0.0f, begin < limit[j][1] ? vs : 0.0f};
#pragma unroll
          for (int i2 = 0; i2 < NM; ++i2)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              o[j][i2][e] = fmaf(part[j][i2][e], v[e & 1], o[j][i2][e]);
              part[j][i2][e] = 0.0f;
            }
        }
      }
    }
  }
  cp_wait<0>();

  // --- the warps' results into one ----------------------------------------------
#pragma unroll
  for (int j = 0; j < NO; ++j)
#pragma unroll
    for (int c = 0; c < 2; ++c)
#pragma unroll
      for (int d = 4; d < 32; d <<= 1) l[j][c] += __shfl_xor_sync(0xffffffffu, l[j][c], d);
  __syncthreads();  // every warp is done with its ring: the results go over it
  if (bad_page) sh_bad = 1;
  const int n_act = min(kWarps, k1 - k0);
  float *om = reinterpret_cast<float *>(smem);
  constexpr int OS = D + 4;  // floats per row: rows begin in different banks
  if (warp < n_act) {
#pragma unroll
    for (int j = 0; j < NO; ++j)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const int col = 8 * j + 2 * t + c;
        if (gq == 0) {
          sh_m[warp][col] = m[j][c];
          sh_l[warp][col] = l[j][c];
        }
        float *dst = om + (warp * RG + col) * OS + gq * VB;
#pragma unroll
        for (int i2 = 0; i2 < NM; ++i2)
          *reinterpret_cast<float2 *>(dst + 2 * i2) = make_float2(o[j][i2][c], o[j][i2][c + 2]);
      }
  }
  __syncthreads();
  const bool bad = sh_bad != 0;
  for (int idx = threadIdx.x; idx < RG * D; idx += kThreads) {
    const int col = idx / D, d = idx - col * D;
    const int r = g * RG + col;
    if (r >= n_rows) continue;
    float top = -INFINITY;
    for (int w = 0; w < n_act; ++w) top = fmaxf(top, sh_m[w][col]);
    const float ref = top == -INFINITY ? 0.0f : top;
    float sum = 0.0f, acc = 0.0f;
    for (int w = 0; w < n_act; ++w) {
      const float by = exp2_fast(sh_m[w][col] - ref);
      sum = fmaf(sh_l[w][col], by, sum);
      acc = fmaf(om[(w * RG + col) * OS + d], by, acc);
    }
    if (bad) sum = __int_as_float(0x7fc00000);
    if (whole) {
      const int i = r / rep, h = hk * rep + r % rep;
      const int64_t row = (int64_t)(q.r0 + i) * a.n_q_heads + h;
      store_out(a.out, a.q.dtype, row * D + d, acc / sum);
      if (a.lse && d == 0) a.lse[row] = (top - kPShift + log2f(sum)) * kLn2;
    } else {
      a.part[((int64_t)slot * RG + col) * D + d] = acc;
      if (d == 0) {
        a.ml[((int64_t)slot * RG + col) * 2] = top;
        a.ml[((int64_t)slot * RG + col) * 2 + 1] = sum;
      }
    }
  }
  __syncthreads();  // before the next segment's copies and flags
}

// NaN for the rows of a sequence that failed a check, by one thread.
__device__ __noinline__ void reject(const AttnArgs &a, const SeqRows &q) {
  record_status(a.c.d_status, MK_ERR_DEVICE, q.s, q.value(a.b), q.bad);
  const int64_t r0 = (int64_t)q.r0 * a.n_q_heads, n = (int64_t)q.n * a.n_q_heads;
  const float nan = __int_as_float(0x7fc00000);
  for (int64_t i = 0; i < n * a.c.head_dim; ++i) store_out(a.out, a.q.dtype, r0 * a.c.head_dim + i, nan);
  if (a.lse)
    for (int64_t i = 0; i < n; ++i) a.lse[r0 + i] = nan;
}

// Chunks on the line of sequence s: pairs x chunks of one pair.
struct SeqLine {
  int chunks, groups;
  int64_t units;
};
template <int MODE>
__device__ __forceinline__ SeqLine seq_line(const AttnArgs &a, const SeqRows &q) {
  if (q.bad || q.n == 0) return {0, 0, 0};
  const int chunks = (int)(((int64_t)q.c + q.n + kChunk - 1) / kChunk);
  const int groups = (a.rep * q.n + group_rows(MODE) - 1) / group_rows(MODE);
  return {chunks, groups, (int64_t)chunks * groups * a.c.n_kv_heads};
}

template <int D, int FMT, int MODE>
__global__ void __launch_bounds__(kThreads, 1) kv8_attention_kernel(const __grid_constant__ AttnArgs a) {
  extern __shared__ __align__(16) uint8_t smem[];
  pdl_trigger();  // the merge launch may get ready; it waits for this grid's end
  if (gated(a.gate)) return;
  if (a.pair_mode) {
    const int g = blockIdx.x % a.groups, rest = blockIdx.x / a.groups;
    const int hk = rest % a.c.n_kv_heads, s = rest / a.c.n_kv_heads;
    const SeqRows q = seq_rows(a.b, a.c.page_size, s);
    const SeqLine y = seq_line<MODE>(a, q);
    if (q.bad && hk == 0 && g == 0 && threadIdx.x == 0) reject(a, q);
    if (g < y.groups) run_segment<D, FMT, MODE>(a, smem, q, hk, g, 0, y.chunks, true, 0);
    return;
  }
  // The line: every CTA adds up all sequences (thread i takes a run of them)
  // and finds the one in which its piece begins.
  __shared__ int64_t warp_sum[kWarps];
  __shared__ int64_t begin_base;
  __shared__ int begin_seq;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int run = (a.b.n_seqs + kThreads - 1) / kThreads;
  const int s0 = min(a.b.n_seqs, (int)threadIdx.x * run), s1 = min(a.b.n_seqs, s0 + run);
  int64_t mine = 0;
  for (int s = s0; s < s1; ++s) {
    const SeqRows q = seq_rows(a.b, a.c.page_size, s);
    if (q.bad && s % (int)gridDim.x == (int)blockIdx.x) reject(a, q);
    mine += seq_line<MODE>(a, q).units;
  }
  int64_t upto = mine;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int64_t v = __shfl_up_sync(0xffffffffu, upto, d);
    if (lane >= d) upto += v;
  }
  if (lane == 31) warp_sum[warp] = upto;
  __syncthreads();
  int64_t total = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    if (w < warp) upto += warp_sum[w];
    total += warp_sum[w];
  }
  const int64_t per = max((int64_t)kMinUnits, (total + gridDim.x - 1) / gridDim.x);
  const int64_t u0 = min(total, per * blockIdx.x), u1 = min(total, u0 + per);
  if (u0 >= upto - mine && u0 < upto) {  // one thread, if the piece is not empty
    int64_t base = upto - mine;
    for (int s = s0; s < s1; ++s) {
      const int64_t n = seq_line<MODE>(a, seq_rows(a.b, a.c.page_size, s)).units;
      if (u0 < base + n) {
        begin_seq = s;
        begin_base = base;
        break;
      }
      base += n;
    }
  }
  __syncthreads();
  int4 cut = make_int4(-1, 0, 0, 0), cut2 = make_int4(0, 0, 0, 0);
  if (u0 < u1) {
    int s = begin_seq;
    int64_t base = begin_base, u = u0;
    while (u < u1) {
      const SeqRows q = seq_rows(a.b, a.c.page_size, s);
      const SeqLine y = seq_line<MODE>(a, q);
      if (u >= base + y.units) {
        base += y.units;
        ++s;
        continue;
      }
      const int64_t loc = u - base;
      const int pair = (int)(loc / y.chunks), k0 = (int)(loc - (int64_t)pair * y.chunks);
      const int k1 = (int)min((int64_t)y.chunks, k0 + (u1 - u));
      const int hk = pair / y.groups, g = pair - hk * y.groups;
      const bool whole = k0 == 0 && k1 == y.chunks;
      run_segment<D, FMT, MODE>(a, smem, q, hk, g, k0, k1, whole,
                                2 * (int)blockIdx.x + (k0 == 0 ? 1 : 0));
      if (k0 == 0 && !whole) {
        // the pair goes on in the CTAs behind this one
        const int64_t last = base + (int64_t)(pair + 1) * y.chunks - 1;
        cut = make_int4(s, hk, g, (int)(last / per));
        cut2 = make_int4(q.r0, q.n, 0, 0);
      }
      u += k1 - k0;
    }
  }
  if (threadIdx.x == 0) {
    a.head[2 * blockIdx.x] = cut;
    a.head[2 * blockIdx.x + 1] = cut2;
  }
}

// Row blockIdx.y of the cut pair that begins in CTA blockIdx.x of the first
// launch: its partial results lie in that CTA's slot 2 c + 1 and in the slots
// 2 c' of the CTAs c' behind it, and are added in that order.
template <int D, int RG>
__global__ void __launch_bounds__(D) kv8_merge_kernel(const __grid_constant__ AttnArgs a) {
  pdl_wait();
  if (gated(a.gate)) return;
  const int c0 = blockIdx.x;
  const int4 cut = a.head[2 * c0];
  if (cut.x < 0) return;
  const int4 rows = a.head[2 * c0 + 1];
  const int col = blockIdx.y, r = cut.z * RG + col;
  if (r >= a.rep * rows.y) return;
  const int n = cut.w - c0 + 1;
  auto slot = [&](int i) { return ((int64_t)(i == 0 ? 2 * c0 + 1 : 2 * (c0 + i)) * RG + col); };
  float top = -INFINITY;
  for (int i = 0; i < n; ++i) top = fmaxf(top, a.ml[slot(i) * 2]);
  const float ref = top == -INFINITY ? 0.0f : top;
  float sum = 0.0f, acc = 0.0f;
#pragma unroll 4
  for (int i = 0; i < n; ++i) {
    const float by = exp2_fast(a.ml[slot(i) * 2] - ref);
    sum = fmaf(a.ml[slot(i) * 2 + 1], by, sum);
    acc = fmaf(a.part[slot(i) * D + threadIdx.x], by, acc);
  }
  const int i = r / a.rep, h = cut.y * a.rep + r % a.rep;
  const int64_t row = (int64_t)(rows.x + i) * a.n_q_heads + h;
  store_out(a.out, a.q.dtype, row * D + threadIdx.x, acc / sum);
  if (a.lse && threadIdx.x == 0) a.lse[row] = (top - kPShift + log2f(sum)) * kLn2;
}

int mode_of(int dtype, int rep, int max_rows) {
  if (dtype == MK_F32) return kRows8F32;
  return rep * max_rows <= 8 ? kRows8 : kRows16;
}

// Grid and workspace of a call, from what the host knows.
struct AttnPlan {
  int mode, groups, ctas;
  bool pair_mode;
  int64_t bytes;
};

AttnPlan plan_of(const mk_kv8_cache &c, const mk_batch &b, int n_q_heads, int dtype) {
  AttnPlan p{};
  const int rep = n_q_heads / c.n_kv_heads;
  p.mode = mode_of(dtype, rep, b.max_rows);
  const int rg = group_rows(p.mode);
  p.groups = (rep * b.max_rows + rg - 1) / rg;
  const int64_t pairs = (int64_t)b.n_seqs * c.n_kv_heads * p.groups;
  const int64_t chunks = ((int64_t)b.max_pages * c.page_size + kChunk - 1) / kChunk;
  p.pair_mode = chunks <= kPairChunks && pairs < (1ll << 30);
  if (p.pair_mode) {
    p.ctas = (int)pairs;
    return p;
  }
  const int sms = sm_count(c.device);
  p.ctas = (int)std::min<int64_t>(sms, (pairs * chunks + kMinUnits - 1) / kMinUnits);
  p.bytes = (int64_t)p.ctas * (32 + 2 * rg * 8 + 2ll * rg * c.head_dim * 4);
  return p;
}

template <int D, int FMT, int MODE>
cudaError_t launch(const AttnArgs &a, const AttnPlan &p, cudaStream_t st) {
  constexpr int smem = smem_bytes(D, MODE);
  static std::atomic<uint64_t> ready{0};  // devices whose limit has been raised
  const uint64_t bit = a.c.device < 64 ? 1ull << a.c.device : 0;
  cudaError_t e = cudaSuccess;
  if (!(ready.load(std::memory_order_relaxed) & bit)) {
    e = cudaFuncSetAttribute(kv8_attention_kernel<D, FMT, MODE>,
                             cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    ready.fetch_or(bit, std::memory_order_relaxed);
  }
  kv8_attention_kernel<D, FMT, MODE><<<p.ctas, kThreads, smem, st>>>(a);
  e = cudaGetLastError();
  if (e != cudaSuccess || p.pair_mode) return e;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(p.ctas, group_rows(MODE));
  cfg.blockDim = dim3(D);
  cfg.stream = st;
  cudaLaunchAttribute at{};
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kv8_merge_kernel<D, group_rows(MODE)>, a);
}

template <int D, int FMT>
cudaError_t launch(const AttnArgs &a, const AttnPlan &p, cudaStream_t st) {
  switch (p.mode) {
    case kRows8: return launch<D, FMT, kRows8>(a, p, st);
    case kRows16: return launch<D, FMT, kRows16>(a, p, st);
    default: return launch<D, FMT, kRows8F32>(a, p, st);
  }
}

const char *check_heads(const mk_kv8_cache *c, int n_q_heads, int dtype, const mk_batch *b) {
  if (n_q_heads < 1 || n_q_heads % c->n_kv_heads) return "n_q_heads must be a multiple of n_kv_heads";
  if (n_q_heads / c->n_kv_heads > 1024) return "more than 1024 query heads per kv head";
  if (dtype < MK_F32 || dtype > MK_F16) return "element type must be MK_F32, MK_BF16 or MK_F16";
  if (b->max_rows > MK_KV8_MAX_ROWS) return "max_rows is above MK_KV8_MAX_ROWS";
  return nullptr;
}

}  // namespace

cudaError_t kv8_attention_launch(const mk_kv8_cache &cache, int layer, const mk_rows &q, int n_q_heads,
                                 float scale, void *out, float *lse, const mk_batch &batch,
                                 void *workspace, const int32_t *gate, cudaStream_t stream) {
  const AttnPlan p = plan_of(cache, batch, n_q_heads, q.dtype);
  AttnArgs a{};
  a.c = cache;
  a.b = batch;
  a.q = q;
  a.out = out;
  a.lse = lse;
  a.layer = layer;
  a.n_q_heads = n_q_heads;
  a.rep = n_q_heads / cache.n_kv_heads;
  a.scale = scale;
  a.block_log2 = __builtin_ctz((unsigned)cache.block);
  a.pair_mode = p.pair_mode;
  a.groups = p.groups;
  a.gate = gate;
  if (p.bytes > 0) {
    const int rg = group_rows(p.mode);
    char *w = static_cast<char *>(workspace);
    a.head = reinterpret_cast<int4 *>(w);
    a.ml = reinterpret_cast<float *>(w + 32ll * p.ctas);
    a.part = a.ml + 4ll * rg * p.ctas;
  }
  if (cache.head_dim == 128)
    return cache.format == MK_KV8_INT8 ? launch<128, MK_KV8_INT8>(a, p, stream)
                                       : launch<128, MK_KV8_E4M3>(a, p, stream);
  return cache.format == MK_KV8_INT8 ? launch<64, MK_KV8_INT8>(a, p, stream)
                                     : launch<64, MK_KV8_E4M3>(a, p, stream);
}

}  // namespace mk

extern "C" mk_status mk_kv8_attention_workspace(const mk_kv8_cache *cache, int n_q_heads, int dtype,
                                                const mk_batch *batch, int64_t *bytes) {
  using namespace mk;
  const char *why = check_kv8_cache(cache, 0);
  if (!why) why = check_batch(batch, cache->page_size);
  if (!why) why = check_heads(cache, n_q_heads, dtype, batch);
  if (!why && !bytes) why = "null result";
  if (why) return ops_fail(MK_ERR_ARG, "mk_kv8_attention_workspace", why);
  *bytes = plan_of(*cache, *batch, n_q_heads, dtype).bytes;
  return MK_OK;
}

extern "C" mk_status mk_kv8_attention(const mk_kv8_cache *cache, int layer, const mk_rows *q,
                                      int n_q_heads, float scale, void *d_out, float *d_lse,
                                      const mk_batch *batch, void *d_workspace,
                                      int64_t workspace_bytes, void *stream) {
  using namespace mk;
  const char *call = "mk_kv8_attention";
  const char *why = check_kv8_cache(cache, layer);
  if (!why) why = check_batch(batch, cache->page_size);
  if (!why && !q) why = "null rows";
  if (!why) why = check_heads(cache, n_q_heads, q->dtype, batch);
  if (!why && batch->n_rows == 0) return MK_OK;
  if (!why) why = check_rows(q);
  if (!why && (!d_out || (reinterpret_cast<uintptr_t>(d_out) & 15)))
    why = "the output is null or not 16-byte aligned";
  if (why) return ops_fail(MK_ERR_ARG, call, why);
  const AttnPlan p = plan_of(*cache, *batch, n_q_heads, q->dtype);
  const mk_status ws = ops_workspace(call, d_workspace, workspace_bytes, p.bytes);
  if (ws != MK_OK) return ws;
  DeviceGuard guard(cache->device);
  if (guard.error() != cudaSuccess) return ops_cuda_fail(guard.error(), call);
  const cudaError_t e = kv8_attention_launch(*cache, layer, *q, n_q_heads, scale, d_out, d_lse, *batch,
                                             d_workspace, nullptr, static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return ops_cuda_fail(e, call);
  return MK_OK;
}
