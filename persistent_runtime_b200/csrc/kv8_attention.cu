// mk_kv8_attention: attention of a few new rows per sequence over an 8-bit
// paged cache.
//
// Mathematics.  For the query rows r of one kv head (rep heads x n new tokens)
// and the positions p of a sequence:  x_pr = f_r sk_p (k_p . q'_r) with the
// codes k_p as they are, q' the row over a power of two, f_r = scale log2(e) /
// that factor and sk_p the scale of p's block; softmax in base 2 over chunks of
// kChunk positions, each relative to its own maximum; o_r = sum over blocks of
// sv w (sum over the block's p of P_pr v_p), where w brings the chunk to the
// running maximum.  Codes and probabilities meet in the tensor cores; scales
// multiply fp32 sums only, so their range does not matter as long as the values'
// own weighted sum stays in that of fp32.
//   int8: codes are MMA operands as they lie in memory.  q' is an integer of
//   at most 127 2^14, three signed 7-bit digits; P an integer of at most 65535,
//   two unsigned 8-bit digits (fp32 rows: 2^23, three); the sums are exact.
//   e4m3: codes become fp16 (exactly), q' is one fp16 number (fp32 rows: two,
//   11 bits apart), P likewise, times 2^14, which keeps fp16 normal down to
//   2^-28 of the chunk's maximum.
//
// What bounds it: the cache is read once, one byte per element, and every
// element takes part in 2 x rows multiply-adds, far below the tensor rate for
// the rows of a decode step: the bound is HBM.  CUDA cores would need rows + 1
// instructions per byte (at 4 heads per kv head that alone is the SM's issue
// rate at the HBM rate), so both products run on mma.sync (m16n8k32 int8,
// m16n8k16 fp16) with the positions (QK) and the head's dims (PV) as the 16
// rows and 8 query rows as columns: the rows of a decode step fill one column
// tile, where the 128-row tile of tcgen05 would be 15/16 empty.
//
// Layout.  Every warp copies its own chunks with cp.async, K and V into a slot
// each, and refills a slot as soon as it has consumed it: no barriers between
// warps.  A warp instruction copies 512 consecutive bytes; copies in the order
// in which the fragments need the bytes (64-byte halves of rows, 16-byte
// columns) reach 4.8 TB/s on a B200 where consecutive ones reach 6.5.  The
// pieces are exchanged on the way in so that fragment reads are free of bank
// conflicts.  The sum over dims may take them in any order, so a lane's QK
// fragments are the words of the 16 bytes it reads; for PV a lane reads D / 8
// dims of four positions and transposes bytes.  Positions past the end are
// filled with zeros by the copy.
//
// Work split.  The (sequence, kv head, row group) pairs, each with
// ceil(length / kChunk) chunks, lie end to end on one line that the grid cuts
// into equal pieces, from the device's own lengths, unless whole pairs come out
// nearly as even; a pair that crosses a cut
// leaves partial results (o, max, sum) in the workspace and a second, small
// launch adds them up in a fixed order.  Where the page table is so short that
// a pair is at most kPairChunks chunks, a CTA takes one whole pair and the second
// launch is left out.
#include <cuda_fp16.h>
#include <cuda_bf16.h>
#include <cuda_fp8.h>

#include <algorithm>
#include <atomic>
#include <type_traits>

#include "kv8.cuh"

namespace mk {
namespace {

constexpr int kChunk = 32;            // positions of a warp's step
constexpr int kTiles = kChunk / 16;   // 16-position MMA tiles of a chunk
constexpr int kPairChunks = 32;       // longest pair (in chunks) for which nothing is ever cut
constexpr int kCutUnits = 8;          // what cutting costs a CTA, in chunks
constexpr int kMinUnits = 4;          // shortest piece of the cut line, in units (chunks)
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

// How the query rows fill the MMA columns: 8 rows of a 16-bit type, 16 rows of
// a 16-bit type (two column tiles), 8 rows of fp32 (a tile of high terms and
// one of low terms).
enum Mode { kRows8 = 0, kRows16 = 1, kRows8F32 = 2 };

// Division of numbers below 2^31 by a divisor that the host knows: with 2^s the
// first power of two >= d and mul = ceil(2^(31 + s) / d), n mul / 2^(31 + s)
// exceeds n / d by less than n / 2^(31 + s) < 1 / d.
struct Divisor {
  uint32_t mul;
  int shift, d;
  Divisor() = default;
  explicit Divisor(int by) : shift(0), d(by) {
    while ((1ll << shift) < by) ++shift;
    mul = (uint32_t)(((1ull << (31 + shift)) + by - 1) / by);
  }
  __device__ __forceinline__ int quotient(int n) const {
    return (int)(((uint64_t)(uint32_t)n * mul) >> (31 + shift));
  }
};
// n / d for a quotient below 2^21: the estimate is off by one at most.
__device__ __forceinline__ int small_quotient(int n, int d) {
  int q = (int)__fdividef((float)n, (float)d);
  const int r = n - q * d;
  q += r >= d ? 1 : r < 0 ? -1 : 0;
  return q;
}

struct AttnArgs {
  mk_kv8_cache c;
  mk_batch b;
  mk_rows q;
  void *out;
  float *lse;
  int layer, n_q_heads;
  Divisor by_page, by_rep, by_grid;
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

// A CTA has 8 warps and an SM to itself, 4 warps and half of one, or 2 and a
// quarter: the registers of 8 warps are an SM's.  Few pairs: 8 (one long sequence
// of e4m3 52.0 us against 54.9 with 4), with fp32 rows and cut lines 4 (batch 8 13.8
// against 14.8; 16 sequences of 8192 50.6 against 56.3, of 1023 14.3 against 13.2).
// More pairs than SMs: 4, more than twice as many: 2, because what a pair costs
// besides its chunks then overlaps with other pairs' (64 sequences of 250: 17.7, 12.7
// and 10.5 us with 8, 4 and 2).
__host__ __device__ constexpr int ctas_per_sm(int warps) { return 8 / warps; }

// More pairs than four CTAs per SM: six CTAs of 2 warps, in 168 registers a thread,
// where the code fits with few spills or none.  head_dim 64 (16 bf16 heads on 8,
// int8): 96 sequences of 1000 37.7 -> 25.5 us, 112 and 512 of 250 13.1 -> 12.4 and 46.0
// -> 36.8, 128 of up to 4000 68.9 -> 58.9.  head_dim 128 with 16-bit rows (32 heads on
// 8): only for short page tables, 96 sequences of 250 18.8 -> 13.1 us, 512 65.0 -> 58.0
// (128, which fill six CTAs just over once, lose: 19.7 -> 21.9); long pairs run at the
// HBM rate and would lose by the spills (96 of up to 4000 72.3 -> 75.5 when it was tried).
constexpr int kCrowd = 6;
__host__ __device__ constexpr bool crowd_fits(int D, int mode) {
  return mode == kRows8 || (D == 64 && mode == kRows8F32);
}

// What a pair costs a CTA besides its chunks (query rows, the warps' results),
// in units of a chunk.
__host__ __device__ constexpr int pair_units(int mode) { return mode == kRows16 ? 16 : 8; }

// Terms of a query element in the MMAs (int8: three signed 7-bit digits, fp16:
// one or, for fp32 rows, two numbers) and of a probability (8-bit digits; fp16
// numbers).  16-bit rows make do with a term less of a probability: with one more,
// outputs differ from those of fp32 probabilities by at most 5e-5 instead of 2.4e-4 to
// 8e-4 (norm of the difference over that of the output), which their rounding to 16
// bits covers (error against 64 bits of bf16 outputs 1.6e-3 both ways; of fp16 rows on
// e4m3 2.1e-4 instead of 2.4e-4), and take longer: 16 x 8192 int8 49.9 -> 56.0 us, e4m3
// 47.8 -> 50.2, 7 x 6001 of five fp16 rows 14.6 -> 16.1, 1024 x 100 68.7 -> 75.9.
__host__ __device__ constexpr int q_terms(int fmt, int mode) {
  return fmt == MK_KV8_INT8 ? 3 : mode == kRows8F32 ? 2 : 1;
}
__host__ __device__ constexpr int p_terms(int fmt, int mode) {
  return (fmt == MK_KV8_INT8 ? 2 : 1) + (mode == kRows8F32 ? 1 : 0);
}

// The factor that P carries in the products, relative to its chunk's maximum:
// int8, 16 bits (the maximum is 65535) or 24 (2^23); fp16: normal down to 2^-28.
// The exponentials are multiplied by it: added to their arguments, its logarithm
// would leave these 19 to 21 bits behind the point.
__host__ __device__ constexpr float p_factor(int fmt, int mode) {
  return fmt != MK_KV8_INT8 ? 16384.0f : mode == kRows8F32 ? 8388608.0f : 65535.0f;
}
// The products are brought back by the power of two that is nearest to it, before a
// scale multiplies them: what is summed up stays as near to the fp32 range's ends as
// the values are.  What is left of the factor goes with the division by the sum.
__host__ __device__ constexpr float p_back(int fmt, int mode) {
  return 1.0f / (fmt != MK_KV8_INT8 ? 16384.0f : mode == kRows8F32 ? 8388608.0f : 65536.0f);
}
__host__ __device__ constexpr float p_rest(int fmt, int mode) { return 1.0f / (p_factor(fmt, mode) * p_back(fmt, mode)); }

// Shared memory: for each warp a slot for a chunk's K codes and scales and one
// for V (later the warps' results), then the query rows' terms.
__host__ __device__ constexpr int slot_bytes(int D) { return kChunk * D + 16; }
__host__ __device__ constexpr int q_offset(int D, int mode, int warps) {
  const int ring = warps * 2 * slot_bytes(D);
  const int merge = warps * group_rows(mode) * (D + 4) * 4;
  return ring > merge ? ring : merge;
}
__host__ __device__ constexpr int smem_bytes(int D, int fmt, int mode, int warps) {
  return q_offset(D, mode, warps) + q_terms(fmt, mode) * group_rows(mode) * D * (fmt == MK_KV8_INT8 ? 1 : 2);
}

// Codes of a chunk in a slot: as in the cache, but with the eight 16-byte
// pieces of every 128-byte line exchanged by swizzle(line), which differs in
// bit 2 for the two lines (D = 128) that eight lanes read for QK and in bits
// 1-2 for the four that they read for PV: both are free of bank conflicts.
template <int D>
__device__ __forceinline__ int swizzle(int line) {
  return D == 128 ? (line & 6) ^ ((line & 1) << 2) : (line & 3) * 2;
}
// Byte of a slot that holds byte `at` (a multiple of 8) of row `row`.
template <int D>
__device__ __forceinline__ int slot_at(int row, int at) {
  const int byte = row * D + at, line = byte >> 7;
  return line * 128 + ((((byte >> 4) & 7) ^ swizzle<D>(line)) << 4) + (byte & 15);
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

__device__ __forceinline__ void mma_s8(int (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                       uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k32.row.col.s32.s8.s8.s32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+r"(d[0]), "+r"(d[1]), "+r"(d[2]), "+r"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_s8u8(int (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k32.row.col.s32.s8.u8.s32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+r"(d[0]), "+r"(d[1]), "+r"(d[2]), "+r"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_s8u8(int (&d)[4], uint32_t a0, uint32_t a1, uint32_t b0) {
  asm("mma.sync.aligned.m16n8k16.row.col.s32.s8.u8.s32 {%0,%1,%2,%3}, {%4,%5}, {%6}, {%0,%1,%2,%3};"
      : "+r"(d[0]), "+r"(d[1]), "+r"(d[2]), "+r"(d[3])
      : "r"(a0), "r"(a1), "r"(b0));
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

// o += (v back) by for two elements, with `back` a power of two: a packed product and a
// packed sum of products.  Without packing the product cost up to 4 % (drafts 14.5 -> 15.1
// us, 16 x 8192 49.1 -> 50.1; packed 14.7 and 50.0, 1024 x 100 even 69.8 -> 68.6).
__device__ __forceinline__ void add2(float &o0, float &o1, float v0, float v1, float back, float by0, float by1) {
  asm("{.reg .b64 o, v, k, b; mov.b64 o, {%0, %1}; mov.b64 v, {%2, %3}; mov.b64 k, {%4, %4}; mov.b64 b, {%5, %6};\n"
      "mul.rn.f32x2 v, v, k; fma.rn.f32x2 o, v, b, o; mov.b64 {%0, %1}, o;}"
      : "+f"(o0), "+f"(o1)
      : "f"(v0), "f"(v1), "f"(back), "f"(by0), "f"(by1));
}

__device__ __forceinline__ uint32_t half2_bits(float a, float b) {
  const __half2 h = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t *>(&h);
}

// x 2^e, for |e| up to 250: in two factors that are normal numbers.
__device__ __forceinline__ float times_pow2(float x, int e) {
  const int h = e >> 1;
  return x * __uint_as_float((uint32_t)(127 + h) << 23) * __uint_as_float((uint32_t)(127 + e - h) << 23);
}

// Codes to fp16 pairs, exactly: word w (4 e4m3 codes) -> (code 0, code 1), (code 2, code 3).
__device__ __forceinline__ void expand_e4m3(uint32_t w, uint32_t &lo, uint32_t &hi) {
  asm("{.reg .b16 a, b; mov.b32 {a, b}, %2; cvt.rn.f16x2.e4m3x2 %0, a; cvt.rn.f16x2.e4m3x2 %1, b;}"
      : "=r"(lo), "=r"(hi)
      : "r"(w));
}

// N (2 or 4) consecutive elements.
template <int N>
__device__ __forceinline__ void load_row(const mk_rows &q, int64_t at, float (&x)[N]) {
  if (q.dtype == MK_F32) {
#pragma unroll
    for (int i = 0; i < N; i += 2) {
      const float2 v = *reinterpret_cast<const float2 *>(static_cast<const float *>(q.data) + at + i);
      x[i] = v.x;
      x[i + 1] = v.y;
    }
  } else {
#pragma unroll
    for (int i = 0; i < N; i += 2) {
      const uint32_t u = *reinterpret_cast<const uint32_t *>(static_cast<const uint16_t *>(q.data) + at + i);
      const float2 f = q.dtype == MK_BF16 ? make_float2(__uint_as_float(u << 16), __uint_as_float(u & 0xffff0000u))
                                          : __half22float2(*reinterpret_cast<const __half2 *>(&u));
      x[i] = f.x;
      x[i + 1] = f.y;
    }
  }
}

__device__ __forceinline__ void store_out(void *out, int dtype, int64_t at, float v) {
  if (dtype == MK_F32) static_cast<float *>(out)[at] = v;
  else if (dtype == MK_BF16) static_cast<__nv_bfloat16 *>(out)[at] = __float2bfloat16_rn(v);
  else static_cast<__half *>(out)[at] = __float2half_rn(v);
}

// The dim in place 16 i + 2 g (+ 1) of a row of results is D / 8 g + 2 i (+ 1).
template <int D>
__device__ __forceinline__ int dim_of(int place) {
  return ((place & 15) >> 1) * (D / 8) + (place >> 4) * 2 + (place & 1);
}
// Two output elements at an even place.
__device__ __forceinline__ void store2(void *out, int dtype, int64_t at, float x, float y) {
  if (dtype == MK_F32) {
    *reinterpret_cast<float2 *>(static_cast<float *>(out) + at) = make_float2(x, y);
  } else if (dtype == MK_BF16) {
    const __nv_bfloat162 p = __floats2bfloat162_rn(x, y);
    *reinterpret_cast<uint32_t *>(static_cast<uint16_t *>(out) + at) = *reinterpret_cast<const uint32_t *>(&p);
  } else {
    *reinterpret_cast<uint32_t *>(static_cast<uint16_t *>(out) + at) = half2_bits(x, y);
  }
}
// Places p .. p + 3 (p a multiple of 4) of the row of results at element `row`.
template <int D>
__device__ __forceinline__ void store_places(void *out, int dtype, int64_t row, int p, float x, float y, float z, float w) {
  store2(out, dtype, row + dim_of<D>(p), x, y);
  store2(out, dtype, row + dim_of<D>(p + 2), z, w);
}

// o += (scale of a block, brought to the running maximum) x sum over the
// block's positions of P v, for one chunk.  GT: tiles that share a scale.
// int8: the digits of P are summed apart, exactly, in 32-bit integers.
template <int D, int FMT, int MODE, int GT, typename PF, typename WC, typename LIM, typename O>
__device__ __forceinline__ void add_values(const uint8_t *vs_, const int (&v_at)[2], int pos0, int block,
                                           const PF &pf, const WC &wc, const LIM &limit, O &o) {
  constexpr bool INT = FMT == MK_KV8_INT8;
  constexpr int NO = MODE == kRows16 ? 2 : 1;
  constexpr int NP = p_terms(FMT, MODE);
  constexpr int VB = D / 8;
  constexpr float kBack = p_back(FMT, MODE);
  // The scale may be NaN (rows that were not finite): it must not reach rows
  // that see nothing of the block.
  float by[kTiles / GT][NO][2];
#pragma unroll
  for (int b = 0; b < kTiles / GT; ++b) {
    const float vs = *reinterpret_cast<const float *>(vs_ + kChunk * D + 4 * b * GT);
    const int begin = (pos0 + 16 * b * GT) & ~(block - 1);
#pragma unroll
    for (int j = 0; j < NO; ++j)
#pragma unroll
      for (int c = 0; c < 2; ++c) by[b][j][c] = begin < limit[j][c] ? vs * wc[j][c] : 0.0f;
  }
  // words at a time: two where two column tiles take up the registers
  constexpr int VW = MODE == kRows16 ? 2 : VB / 4;
#pragma unroll
  for (int w0 = 0; w0 < VB / 4; w0 += VW) {
  uint32_t vw[kTiles][4][VW];
#pragma unroll
  for (int tl = 0; tl < kTiles; ++tl)
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const uint8_t *vp = vs_ + v_at[r & 1] + (tl * 16 + (r >> 1) * 8) * D + 4 * w0;
      if constexpr (VW == 4) {
        const uint4 u = *reinterpret_cast<const uint4 *>(vp);
        vw[tl][r][0] = u.x; vw[tl][r][1] = u.y; vw[tl][r][2] = u.z; vw[tl][r][3] = u.w;
      } else {
        const uint2 u = *reinterpret_cast<const uint2 *>(vp);
        vw[tl][r][0] = u.x; vw[tl][r][1] = u.y;
      }
    }
#pragma unroll
  for (int wi = 0; wi < VW; ++wi) {
    const int w = w0 + wi;  // dims 4 w .. 4 w + 3 of the lane: m-tiles 2 w, 2 w + 1
    // the four positions 2 t, 2 t + 1, 2 t + 8, 2 t + 9 of a tile: int8, one
    // word per dim; e4m3, a pair of fp16 for each two
    uint32_t d[kTiles][INT ? 4 : 8];
#pragma unroll
    for (int tl = 0; tl < kTiles; ++tl) {
      const uint32_t p = __byte_perm(vw[tl][0][wi], vw[tl][1][wi], 0x5140), q = __byte_perm(vw[tl][0][wi], vw[tl][1][wi], 0x7362);
      const uint32_t r = __byte_perm(vw[tl][2][wi], vw[tl][3][wi], 0x5140), s = __byte_perm(vw[tl][2][wi], vw[tl][3][wi], 0x7362);
      if constexpr (INT) {
        d[tl][0] = __byte_perm(p, r, 0x5410);
        d[tl][1] = __byte_perm(p, r, 0x7632);
        d[tl][2] = __byte_perm(q, s, 0x5410);
        d[tl][3] = __byte_perm(q, s, 0x7632);
      } else {
        expand_e4m3(p, d[tl][0], d[tl][1]);
        expand_e4m3(q, d[tl][2], d[tl][3]);
        expand_e4m3(r, d[tl][4], d[tl][5]);
        expand_e4m3(s, d[tl][6], d[tl][7]);
      }
    }
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int j = 0; j < NO; ++j)
#pragma unroll
        for (int b = 0; b < kTiles / GT; ++b) {
          float v[4];
          if constexpr (INT) {
            int acc[NP][4] = {};
#pragma unroll
            for (int u = 0; u < NP; ++u) {
              if constexpr (GT == 2)
                mma_s8u8(acc[u], d[0][2 * h], d[0][2 * h + 1], d[1][2 * h], d[1][2 * h + 1], pf[j][0][u], pf[j][1][u]);
              else
                mma_s8u8(acc[u], d[b][2 * h], d[b][2 * h + 1], pf[j][b][u]);
            }
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              if constexpr (NP == 2) v[e] = (float)(acc[0][e] * 256 + acc[1][e]);
              else v[e] = fmaf((float)(acc[0][e] * 256 + acc[1][e]), 256.0f, (float)acc[NP - 1][e]);
            }
          } else {
            v[0] = v[1] = v[2] = v[3] = 0.0f;
#pragma unroll
            for (int tl = b * GT; tl < (b + 1) * GT; ++tl)
#pragma unroll
              for (int u = 0; u < NP; ++u)
                mma_f16(v, d[tl][2 * h], d[tl][2 * h + 1], d[tl][4 + 2 * h], d[tl][5 + 2 * h], pf[j][tl][2 * u], pf[j][tl][2 * u + 1]);
          }
#pragma unroll
          for (int e = 0; e < 4; e += 2)
            add2(o[j][2 * w + h][e], o[j][2 * w + h][e + 1], v[e], v[e + 1], kBack, by[b][j][0], by[b][j][1]);
        }
  }
  }
}

// Chunks [k0, k1) of pair (sequence q.s, kv head hk, row group g) by one CTA;
// `whole`: they are all of it and the result is final, else it goes to
// partial slot `slot`.
template <int D, int FMT, int MODE, int W>
__device__ __forceinline__ void run_segment(const AttnArgs &a, uint8_t *smem, const SeqRows &q,
                                            int hk, int g, int k0, int k1, bool whole, int slot) {
  constexpr bool INT = FMT == MK_KV8_INT8;
  constexpr int RG = group_rows(MODE);
  constexpr int NO = MODE == kRows16 ? 2 : 1;            // column tiles of 8 rows
  constexpr int NQ = q_terms(FMT, MODE), NP = p_terms(FMT, MODE);
  constexpr int NC = D / 64;                             // 64-dim halves of a row
  constexpr int NK = INT ? D / 32 : D / 16;              // MMA steps over the dims
  constexpr int VB = D / 8;                              // bytes of a V row that a lane holds
  constexpr int NM = D / 16;                             // 16-dim m-tiles of the output
  __shared__ float sh_m[W][RG], sh_l[W][RG], sh_f[RG];
  __shared__ int sh_bad, sh_limit[RG];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int gq = lane >> 2, t = lane & 3;
  const int P = a.c.page_size, rep = a.by_rep.d, n_rows = rep * q.n;
  const int end = q.c + q.n;  // positions of the sequence, its new rows included
  if (threadIdx.x == 0) sh_bad = 0;

  // --- copies: the warp's i-th chunk is chunk k0 + warp + i W ----------------
  uint8_t *ks_ = smem + warp * 2 * slot_bytes(D), *vs_ = ks_ + slot_bytes(D);
  const uint32_t ks_u32 = (uint32_t)__cvta_generic_to_shared(ks_);
  const uint32_t vs_u32 = ks_u32 + slot_bytes(D);
  const int n_mine = k1 - k0 > warp ? (k1 - k0 - warp + W - 1) / W : 0;
  constexpr int kLook = 32 / kTiles;  // chunks whose pages one lookup (one tile per lane) covers
  const int32_t *table = a.b.d_page_table + (int64_t)q.s * a.b.max_pages;
  bool bad_page = false;
  auto tile_pos = [&](int i0) {  // position of this lane's tile of the lookup at chunk i0
    return (k0 + warp + (i0 + lane / kTiles) * W) * kChunk + (lane % kTiles) * 16;
  };
  auto look = [&](int i0) {
    const int pos = tile_pos(i0);
    return i0 + lane / kTiles < n_mine && pos < end ? table[a.by_page.quotient(pos)] : 0;
  };
  auto tile_row = [&](int i0, int page) -> int64_t {  // row of the pool where the tile begins
    const int pos = tile_pos(i0);
    if (i0 + lane / kTiles >= n_mine || pos >= end) return 0;
    if (page < 0 || page >= a.c.n_pages) {
      bad_page = true;
      record_status(a.c.d_status, MK_ERR_DEVICE, q.s, page, MK_CHECK_PAGE);
      return 0;
    }
    return kv8_slab(a.c, a.layer, page, hk) * P + (pos - a.by_page.quotient(pos) * P);
  };
  int page_next = look(0);
  int64_t rows = 0;
  // K (or V) codes and scales of chunk i; V follows K, so the lookup is K's.
  // A warp instruction copies 512 consecutive bytes: four (D = 64: eight) rows.
  constexpr int kRows = 512 / D;
  const int my_row = lane / (D / 16);
  uint32_t to[2];  // where this lane's piece goes, for even and odd groups of rows
#pragma unroll
  for (int b = 0; b < 2; ++b) to[b] = slot_at<D>(b * kRows + my_row, (lane % (D / 16)) * 16) - b * 512;
  auto issue = [&](int i, bool is_v) {
    if (i < n_mine) {
      if (!is_v && i % kLook == 0) {
        rows = tile_row(i, page_next);
        page_next = look(i + kLook);
      }
      const int pos0 = (k0 + warp + i * W) * kChunk;
      const int from = (i % kLook) * kTiles;
      const uint8_t *src = static_cast<const uint8_t *>(is_v ? a.c.d_v : a.c.d_k) + lane * 16;
      const uint32_t st = is_v ? vs_u32 : ks_u32;
#pragma unroll
      for (int tl = 0; tl < kTiles; ++tl) {
        const uint8_t *p = src + __shfl_sync(0xffffffffu, rows, from + tl) * D;
        const int left = end - pos0 - 16 * tl - my_row;  // rows of the tile that exist, from mine on
#pragma unroll
        for (int r = 0; r < 16 / kRows; ++r)
          cp_async<16>(st + tl * 16 * D + r * 512 + to[r & 1], p + r * 512, r * kRows < left);
      }
      // a tile past the end takes the first tile's scale: it may share its block
      const int tl = lane % kTiles;
      const int64_t at = __shfl_sync(0xffffffffu, rows, from + (pos0 + 16 * tl < end ? tl : 0));
      if (lane < kTiles)
        cp_async<4>(st + kChunk * D + lane * 4,
                    (is_v ? a.c.d_v_scale : a.c.d_k_scale) + (at >> a.block_log2), true);
    }
    cp_commit();
  };
  // --- query rows, once for all warps: a warp quantises a row at a time ------
  constexpr int QB = INT ? 1 : 2;  // bytes of a term
  constexpr int NR = (RG + W - 1) / W;
  uint8_t *qs = smem + q_offset(D, MODE, W);  // [term][row][D]
  float x_row[NR][D / 32];
  int lim_row[NR];
#pragma unroll
  for (int n = 0; n < NR; ++n) {
    const int col = warp + n * W, r = g * RG + col;
    const int i = a.by_rep.quotient(r);
    lim_row[n] = col < RG && r < n_rows ? q.c + i + 1 : 0;
    if (lim_row[n]) {
      load_row<D / 32>(a.q, (int64_t)(q.r0 + i) * a.q.row_stride + (int64_t)(hk * rep + r - i * rep) * a.q.head_stride + lane * (D / 32), x_row[n]);
    } else {
#pragma unroll
      for (int d = 0; d < D / 32; ++d) x_row[n][d] = 0.0f;
    }
  }
  issue(0, false);
  issue(0, true);
#pragma unroll
  for (int n = 0; n < NR; ++n) {
    const int col = warp + n * W;
    if (RG % W != 0 && col >= RG) break;
    const float(&x)[D / 32] = x_row[n];
    if (lim_row[n] == 0) {  // no such row: its column adds nothing and is not read
#pragma unroll
      for (int u = 0; u < NQ; ++u) {
        if constexpr (INT && D == 64) *reinterpret_cast<uint16_t *>(qs + u * RG * D + col * D + lane * 2) = 0;
        else if constexpr (INT || D == 64) *reinterpret_cast<uint32_t *>(qs + (u * RG * D + col * D) * QB + lane * 4) = 0;
        else *reinterpret_cast<uint2 *>(qs + (u * RG * D + col * D) * QB + lane * 8) = make_uint2(0, 0);
      }
      if (lane == 0) {
        sh_f[col] = 0.0f;
        sh_limit[col] = 0;
      }
      continue;
    }
    uint32_t top = 0;  // bits of the largest magnitude: above those of infinity for a NaN
#pragma unroll
    for (int d = 0; d < D / 32; ++d) top = max(top, __float_as_uint(x[d]) & 0x7fffffffu);
    top = __reduce_max_sync(0xffffffffu, top);
    const int e = (int)(top >> 23) - 126;  // |q| < 2^e
    const float shrink = times_pow2(1.0f, -e);
    uint8_t *dst = qs + (col * D + lane * (D / 32)) * QB;
    constexpr float kOne = INT ? 127.0f * 16384.0f : 1.0f;
    if constexpr (INT) {
      // q 2^-e in (-1, 1) times 127 2^14, as a sum of three signed 7-bit digits
      uint32_t word[NQ] = {};
#pragma unroll
      for (int d = 0; d < D / 32; ++d) {
        int n = __float2int_rn(x[d] * shrink * kOne);
#pragma unroll
        for (int u = 0; u < NQ; ++u) {
          const int s = 7 * (NQ - 1 - u);
          const int digit = s ? (n + (1 << s >> 1)) >> s : n;
          n -= digit << s;
          word[u] |= (uint32_t)(digit & 0xff) << (8 * d);
        }
      }
#pragma unroll
      for (int u = 0; u < NQ; ++u) {
        if constexpr (D == 128) *reinterpret_cast<uint32_t *>(dst + u * RG * D) = word[u];
        else *reinterpret_cast<uint16_t *>(dst + u * RG * D) = (uint16_t)word[u];
      }
    } else {
#pragma unroll
      for (int d = 0; d < D / 32; d += 2) {
        const float y0 = x[d] * shrink, y1 = x[d + 1] * shrink;
        const uint32_t hi = half2_bits(y0, y1);
        *reinterpret_cast<uint32_t *>(dst + 2 * d) = hi;
        if constexpr (NQ == 2) {
          // the low term carries a factor 2^11, so that it keeps its bits
          const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&hi));
          *reinterpret_cast<uint32_t *>(dst + RG * D * QB + 2 * d) = half2_bits((y0 - f.x) * 2048.0f, (y1 - f.y) * 2048.0f);
        }
      }
    }
    if (lane == 0) {
      // integers have no NaN: the row's factor carries it
      sh_f[col] = INT && top >= 0x7f800000u ? __int_as_float(0x7fc00000) : times_pow2(a.scale * (kLog2e / kOne), e);
      sh_limit[col] = lim_row[n];
    }
  }
  __syncthreads();
  uint32_t qf[NO][NQ][NK][2];
  float f[NO][2];  // of the lane's columns 2 t, 2 t + 1 of a column tile
  int limit[NO][2];
#pragma unroll
  for (int j = 0; j < NO; ++j) {
#pragma unroll
    for (int u = 0; u < NQ; ++u)
#pragma unroll
      for (int c = 0; c < NC * QB; ++c) {
        // 16 dims (8 for fp16) of row 8 j + gq: INT, half c; else half c / 2
        const uint4 w = *reinterpret_cast<const uint4 *>(
            qs + ((u * RG + 8 * j + gq) * D + (c / QB) * 64 + t * 16) * QB + (c % QB) * 16);
        const uint32_t ww[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int k = 0; k < 4; ++k) qf[j][u][c * 2 + k / 2][k & 1] = ww[k];
      }
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      f[j][c] = sh_f[8 * j + 2 * t + c];
      limit[j][c] = sh_limit[8 * j + 2 * t + c];
    }
  }
  const int least = q.c + a.by_rep.quotient(g * RG) + 1;  // the group's first row sees the fewest positions

  // --- the warp's chunks ------------------------------------------------------
  // a lane's pieces: K, 16 bytes of each 64 of the rows gq and gq + 8 of a
  // tile; V, D / 8 bytes of the rows 2 t, 2 t + 1, 2 t + 8 and 2 t + 9
  int k_at[NC], v_at[2];
#pragma unroll
  for (int c = 0; c < NC; ++c) k_at[c] = slot_at<D>(gq, c * 64 + t * 16);
#pragma unroll
  for (int r = 0; r < 2; ++r) v_at[r] = slot_at<D>(2 * t + r, gq * VB);
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
    const int pos0 = (k0 + warp + i * W) * kChunk;
    cp_wait<1>();  // this chunk's K; its V may still be under way
    __syncwarp();
    // scores, in base 2
    float x[NO][kTiles][4];
#pragma unroll
    for (int tl = 0; tl < kTiles; ++tl) {
          uint32_t w0[NC][4], w1[NC][4];  // rows gq and gq + 8 of the tile
#pragma unroll
      for (int c = 0; c < NC; ++c) {
        const uint4 r0 = *reinterpret_cast<const uint4 *>(ks_ + k_at[c] + tl * 16 * D);
        const uint4 r1 = *reinterpret_cast<const uint4 *>(ks_ + k_at[c] + tl * 16 * D + 8 * D);
        w0[c][0] = r0.x; w0[c][1] = r0.y; w0[c][2] = r0.z; w0[c][3] = r0.w;
        w1[c][0] = r1.x; w1[c][1] = r1.y; w1[c][2] = r1.z; w1[c][3] = r1.w;
      }
      const float ks = *reinterpret_cast<const float *>(ks_ + kChunk * D + 4 * tl);
      if constexpr (INT) {
        int s[NO][NQ][4] = {};
#pragma unroll
        for (int k = 0; k < NK; ++k)
#pragma unroll
          for (int j = 0; j < NO; ++j)
#pragma unroll
            for (int u = 0; u < NQ; ++u)
              mma_s8(s[j][u], w0[k / 2][2 * (k & 1)], w1[k / 2][2 * (k & 1)], w0[k / 2][2 * (k & 1) + 1],
                     w1[k / 2][2 * (k & 1) + 1], qf[j][u][k][0], qf[j][u][k][1]);
#pragma unroll
        for (int j = 0; j < NO; ++j)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float v = fmaf((float)s[j][0][e], 16384.0f, (float)(s[j][1][e] * 128 + s[j][NQ - 1][e]));
            x[j][tl][e] = v * (ks * f[j][e & 1]);
          }
      } else {
        float s[NO][NQ][4] = {};
#pragma unroll
        for (int k = 0; k < NK; ++k) {
          uint32_t a0, a1, a2, a3;
          expand_e4m3(w0[k / 4][k & 3], a0, a2);
          expand_e4m3(w1[k / 4][k & 3], a1, a3);
#pragma unroll
          for (int j = 0; j < NO; ++j)
#pragma unroll
            for (int u = 0; u < NQ; ++u)
              mma_f16(s[j][u], a0, a1, a2, a3, qf[j][u][k][0], qf[j][u][k][1]);
        }
#pragma unroll
        for (int j = 0; j < NO; ++j)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            float v = s[j][0][e];
            if constexpr (NQ == 2) v = fmaf(s[j][1][e], 1.0f / 2048.0f, v);
            x[j][tl][e] = v * (ks * f[j][e & 1]);
          }
      }
    }
    __syncwarp();  // every lane has read the scales
    issue(i + 1, false);
    if (pos0 + kChunk > least) {  // some row does not see all of the chunk
#pragma unroll
      for (int tl = 0; tl < kTiles; ++tl)
#pragma unroll
        for (int j = 0; j < NO; ++j)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (pos0 + 16 * tl + gq + (e >> 1) * 8 >= limit[j][e & 1]) x[j][tl][e] = -INFINITY;
    }
    // probabilities relative to the chunk's maximum, as B fragments; wc brings
    // them to the running maximum
    uint32_t pf[NO][kTiles][INT ? NP : 2 * NP];
    float wc[NO][2];
#pragma unroll
    for (int j = 0; j < NO; ++j) {
      float ref[2], by[2];
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        float v = fmaxf(x[j][0][c], x[j][0][c + 2]);
#pragma unroll
        for (int tl = 1; tl < kTiles; ++tl) v = fmaxf(v, fmaxf(x[j][tl][c], x[j][tl][c + 2]));
#pragma unroll
        for (int d = 4; d < 32; d <<= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, d));
        const float now = fmaxf(m[j][c], v);
        const float base = now == -INFINITY ? 0.0f : now;
        by[c] = exp2_fast(m[j][c] - base);
        wc[j][c] = exp2_fast(v - base);
        ref[c] = v == -INFINITY ? 0.0f : v;
        m[j][c] = now;
      }
      float sum[2] = {0.0f, 0.0f};
#pragma unroll
      for (int tl = 0; tl < kTiles; ++tl) {
        uint32_t r0[2], r1[2];
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          constexpr float kUp = p_factor(FMT, MODE);
          const float e0 = exp2_fast(x[j][tl][2 * r] - ref[0]);
          const float e1 = exp2_fast(x[j][tl][2 * r + 1] - ref[1]);
          sum[0] += e0;
          sum[1] += e1;
          const float p0 = e0 * kUp, p1 = e1 * kUp;
          if constexpr (INT && NP == 2) {
            // adding 2^23 rounds to an integer in the low bits
            r0[r] = transpose8x8(__byte_perm(__float_as_uint(fmaf(e0, kUp, 8388608.0f)),
                                             __float_as_uint(fmaf(e1, kUp, 8388608.0f)), 0x5410));
          } else if constexpr (INT) {
            const uint32_t n0 = __float2uint_rn(p0), n1 = __float2uint_rn(p1);
            r0[r] = transpose8x8(__byte_perm(n0, n1, 0x6521));
            r1[r] = transpose8x8(__byte_perm(n0, n1, 0x5410));
          } else {
            const uint32_t hi = half2_bits(p0, p1);
            pf[j][tl][r] = transpose8x8(hi);
            if constexpr (NP == 2) {
              const float2 h = __half22float2(*reinterpret_cast<const __half2 *>(&hi));
              pf[j][tl][2 + r] = transpose8x8(half2_bits(p0 - h.x, p1 - h.y));
            }
          }
        }
        if constexpr (INT) {
          // bytes of positions 2 t, 2 t + 1, 2 t + 8, 2 t + 9: high, middle, low digit
          pf[j][tl][0] = __byte_perm(r0[0], r0[1], 0x7531);
          pf[j][tl][1] = __byte_perm(r0[0], r0[1], 0x6420);
          if constexpr (NP == 3) pf[j][tl][NP - 1] = __byte_perm(r1[0], r1[1], 0x6420);
        }
      }
#pragma unroll
      for (int c = 0; c < 2; ++c) l[j][c] = fmaf(l[j][c], by[c], sum[c] * wc[j][c]);
      // a new maximum is rare once a few chunks have passed
      if (__any_sync(0xffffffffu, by[0] != 1.0f || by[1] != 1.0f)) {
#pragma unroll
        for (int i2 = 0; i2 < NM; ++i2)
#pragma unroll
          for (int e = 0; e < 4; ++e) o[j][i2][e] *= by[e & 1];
      }
    }
    cp_wait<1>();  // this chunk's V; the next K may still be under way
    __syncwarp();
    if (a.c.block == 16)
      add_values<D, FMT, MODE, 1>(vs_, v_at, pos0, a.c.block, pf, wc, limit, o);
    else
      add_values<D, FMT, MODE, 2>(vs_, v_at, pos0, a.c.block, pf, wc, limit, o);
    __syncwarp();
    issue(i + 1, true);
  }
  cp_wait<0>();

  // --- the warps' results into one ----------------------------------------------
#pragma unroll
  for (int j = 0; j < NO; ++j)
#pragma unroll
    for (int c = 0; c < 2; ++c)
#pragma unroll
      for (int d = 4; d < 32; d <<= 1) l[j][c] += __shfl_xor_sync(0xffffffffu, l[j][c], d);
  __syncthreads();  // every warp is done with its slots: the results go over them
  if (bad_page) sh_bad = 1;
  float *om = reinterpret_cast<float *>(smem);
  constexpr int OS = D + 4;  // floats per row: rows begin in different banks
#pragma unroll
  for (int j = 0; j < NO; ++j)
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      const int col = 8 * j + 2 * t + c;
      if (gq == 0) {
        sh_m[warp][col] = m[j][c];
        sh_l[warp][col] = l[j][c];
      }
      // dims gq VB + 2 i2, + 1 go to place 16 i2 + 2 gq: neighbouring lanes write
      // neighbouring places
      float *dst = om + (warp * RG + col) * OS + 2 * gq;
#pragma unroll
      for (int i2 = 0; i2 < NM; ++i2)
        *reinterpret_cast<float2 *>(dst + 16 * i2) = make_float2(o[j][i2][c], o[j][i2][c + 2]);
    }
  __syncthreads();
  if ((int)threadIdx.x < RG) {  // the warps' weights, and the row's maximum and sum
    const int col = threadIdx.x;
    float top = -INFINITY, sum = 0.0f;
#pragma unroll
    for (int w = 0; w < W; ++w) top = fmaxf(top, sh_m[w][col]);
    const float ref = top == -INFINITY ? 0.0f : top;
#pragma unroll
    for (int w = 0; w < W; ++w) {
      const float by = exp2_fast(sh_m[w][col] - ref);
      sum = fmaf(sh_l[w][col], by, sum);
      sh_m[w][col] = by;
    }
    if (sh_bad) sum = __int_as_float(0x7fc00000);
    sh_l[0][col] = sum;
    sh_l[1][col] = top;
  }
  __syncthreads();
  for (int idx = threadIdx.x; idx < RG * (D / 4); idx += W * 32) {
    const int col = idx / (D / 4), d = (idx - col * (D / 4)) * 4;
    const int r = g * RG + col;
    if (r >= n_rows) continue;
    float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
    for (int w = 0; w < W; ++w) {
      const float by = sh_m[w][col];
      const float4 v = *reinterpret_cast<const float4 *>(om + (w * RG + col) * OS + d);
      acc.x = fmaf(v.x, by, acc.x);
      acc.y = fmaf(v.y, by, acc.y);
      acc.z = fmaf(v.z, by, acc.z);
      acc.w = fmaf(v.w, by, acc.w);
    }
    const float sum = sh_l[0][col], top = sh_l[1][col];
    if (whole) {
      const int i = a.by_rep.quotient(r);
      const int64_t row = (int64_t)(q.r0 + i) * a.n_q_heads + hk * rep + r - i * rep;
      const float by = p_rest(FMT, MODE) / sum;
      store_places<D>(a.out, a.q.dtype, row * D, d, acc.x * by, acc.y * by, acc.z * by, acc.w * by);
      if (a.lse && d == 0) a.lse[row] = (top + log2f(sum)) * kLn2;
    } else {
      *reinterpret_cast<float4 *>(a.part + ((int64_t)slot * RG + col) * D + d) = acc;
      if (d == 0) *reinterpret_cast<float2 *>(a.ml + ((int64_t)slot * RG + col) * 2) = make_float2(top, sum);
    }
  }
  __syncthreads();  // before the next segment's copies and flags
}

// NaN for the rows of a sequence that failed a check, by a warp (there may be
// many: max_rows need not bound them).
__device__ __noinline__ void reject(const AttnArgs &a, const SeqRows &q) {
  const int lane = threadIdx.x & 31;
  if (lane == 0) record_status(a.c.d_status, MK_ERR_DEVICE, q.s, q.value(a.b), q.bad);
  const int64_t r0 = (int64_t)q.r0 * a.n_q_heads, n = (int64_t)q.n * a.n_q_heads;
  const float nan = __int_as_float(0x7fc00000);
  for (int64_t i = lane; i < n * a.c.head_dim; i += 32) store_out(a.out, a.q.dtype, r0 * a.c.head_dim + i, nan);
  if (a.lse)
    for (int64_t i = lane; i < n; i += 32) a.lse[r0 + i] = nan;
}
// The same for every such sequence that falls to this CTA, by its warps.
template <int W>
__device__ __noinline__ void reject_all(const AttnArgs &a) {
  for (int first = (threadIdx.x >> 5) * 32; first < a.b.n_seqs; first += W * 32) {
    const int s = first + (threadIdx.x & 31);
    const bool mine = s < a.b.n_seqs && s % (int)gridDim.x == (int)blockIdx.x && seq_rows(a.b, a.c.page_size, s).bad;
    for (uint32_t left = __ballot_sync(0xffffffffu, mine); left; left &= left - 1)
      reject(a, seq_rows(a.b, a.c.page_size, first + __ffs(left) - 1));
  }
}

// Units on the line of sequence s: for every pair its chunks, then
// pair_units that stand for what it costs besides.
struct SeqLine {
  int chunks, groups, units;
};
template <int MODE>
__device__ __forceinline__ SeqLine seq_line(const AttnArgs &a, const SeqRows &q) {
  if (q.bad || q.n == 0) return {0, 0, 0};
  const int chunks = (q.c + q.n + kChunk - 1) / kChunk;
  const int groups = (a.by_rep.d * q.n + group_rows(MODE) - 1) / group_rows(MODE);
  return {chunks, groups, (chunks + pair_units(MODE)) * groups * a.c.n_kv_heads};
}

template <int D, int FMT, int MODE, int W, int CTAS>
__global__ void __launch_bounds__(W * 32, CTAS) kv8_attention_kernel(const __grid_constant__ AttnArgs a) {
  extern __shared__ __align__(16) uint8_t smem[];
  pdl_trigger();  // the launch behind this one may get ready; it waits for this grid's end
  pdl_wait();
  if (gated(a.gate)) return;
  if (a.pair_mode) {
    const int g = blockIdx.x % a.groups, rest = blockIdx.x / a.groups;
    const int hk = rest % a.c.n_kv_heads, s = rest / a.c.n_kv_heads;
    const SeqRows q = seq_rows(a.b, a.c.page_size, s);
    const SeqLine y = seq_line<MODE>(a, q);
    if (q.bad && hk == 0 && g == 0 && threadIdx.x < 32) reject(a, q);
    if (g < y.groups) run_segment<D, FMT, MODE, W>(a, smem, q, hk, g, 0, y.chunks, true, 0);
    return;
  }
  // The line: the units of all sequences, and, 32 at a time by every warp, the
  // sequence in which the CTA's piece begins.
  const int lane = threadIdx.x & 31;
  SeqRows mine;   // sequence s0 + lane
  SeqLine line;
  int upto;       // units of the sequences s0 .. s0 + lane
  int s0;
  bool whole = false;  // nothing is cut: a pair is one unit, and the pieces are dealt out
  auto group = [&](int first) {
    s0 = first;
    line = SeqLine{0, 0, 0};
    mine = SeqRows{first + lane, 0, 0, 0, 0};
    if (first + lane < a.b.n_seqs) {
      mine = seq_rows(a.b, a.c.page_size, first + lane);
      line = seq_line<MODE>(a, mine);
      if (whole) line.units = line.groups * a.c.n_kv_heads;
    }
    upto = line.units;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, upto, d);
      if (lane >= d) upto += v;
    }
  };
  int total = 0, pairs = 0, longest = 0, bad = 0;
  auto count = [&](const SeqRows &q, const SeqLine &y) {
    bad |= q.bad;
    total += y.units;
    pairs += y.groups * a.c.n_kv_heads;
    longest = max(longest, y.chunks);
  };
  if (a.b.n_seqs <= 32) {
    group(0);
    count(mine, line);
  } else {  // the warps share the sequences
#pragma unroll 4
    for (int s = threadIdx.x; s < a.b.n_seqs; s += W * 32) {
      const SeqRows q = seq_rows(a.b, a.c.page_size, s);
      count(q, seq_line<MODE>(a, q));
    }
  }
  if (__any_sync(0xffffffffu, bad)) reject_all<W>(a);
  total = __reduce_add_sync(0xffffffffu, total);
  pairs = __reduce_add_sync(0xffffffffu, pairs);
  longest = __reduce_max_sync(0xffffffffu, longest);
  if (a.b.n_seqs > 32) {
    __shared__ int sums[3][W];
    if (lane == 0) {
      sums[0][threadIdx.x >> 5] = total;
      sums[1][threadIdx.x >> 5] = pairs;
      sums[2][threadIdx.x >> 5] = longest;
    }
    __syncthreads();
    total = pairs = longest = 0;
#pragma unroll
    for (int w = 0; w < W; ++w) {
      total += sums[0][w];
      pairs += sums[1][w];
      longest = max(longest, sums[2][w]);
    }
  }
  // the host allows fewer than 2^30 units
  const int per = max(kMinUnits, a.by_grid.quotient(total + (int)gridDim.x - 1));
  // Whole pairs where the busiest CTA's share is at most 4/3 of an equal one and
  // a bit: an SM alone draws 4/3 of its share of the HBM rate, and cutting
  // costs partial results and their sums (16 sequences of 1023: 12.1 us whole,
  // 15.8 cut; 8 of 256 to 4096: 25.5 whole, 14.0 cut).
  const int64_t busiest = (int64_t)a.by_grid.quotient(pairs + (int)gridDim.x - 1) * (longest + pair_units(MODE));
  whole = 3 * busiest <= 4 * ((int64_t)per + kCutUnits);
  const int u0 = whole ? (int)blockIdx.x : (int)min((int64_t)total, (int64_t)per * blockIdx.x);
  const int u1 = whole ? pairs : min(total, u0 + per);
  int base0 = 0;  // units before sequence s0
  if ((whole || a.b.n_seqs > 32) && u0 < u1) group(0);
  int4 cut = make_int4(-1, 0, 0, 0), cut2 = make_int4(0, 0, 0, 0);
  int u = u0;
  while (u < u1) {
    // the sequence of unit u: the first lane whose sequences reach beyond it
    const uint32_t beyond = __ballot_sync(0xffffffffu, base0 + upto > u);
    if (beyond == 0) {
      base0 += __shfl_sync(0xffffffffu, upto, 31);
      group(s0 + 32);
      continue;
    }
    const int at = __ffs(beyond) - 1;
    const SeqRows q{s0 + at, __shfl_sync(0xffffffffu, mine.r0, at), __shfl_sync(0xffffffffu, mine.n, at),
                    __shfl_sync(0xffffffffu, mine.c, at), 0};
    const int chunks = __shfl_sync(0xffffffffu, line.chunks, at);
    const int groups = __shfl_sync(0xffffffffu, line.groups, at);
    const int base = base0 + __shfl_sync(0xffffffffu, upto - line.units, at);
    const int len = whole ? 1 : chunks + pair_units(MODE);
    const int pair = small_quotient(u - base, len), k0 = u - base - pair * len;
    const int k1 = whole ? chunks : min(chunks, k0 + u1 - u);
    if (k0 < chunks) {
      const int hk = groups == 1 ? pair : small_quotient(pair, groups), g = pair - hk * groups;
      const bool all = k0 == 0 && k1 == chunks;
      run_segment<D, FMT, MODE, W>(a, smem, q, hk, g, k0, k1, all, 2 * (int)blockIdx.x + (k0 == 0 ? 1 : 0));
      if (k0 == 0 && !all) {
        // the pair goes on in the CTAs behind this one, to that of its last chunk
        cut = make_int4(q.s, hk, g, small_quotient(base + pair * len + chunks - 1, per));
        cut2 = make_int4(q.r0, q.n, 0, 0);
      }
    }
    u = whole ? u + (int)gridDim.x : base + (pair + 1) * len;  // the next pair, if the piece goes that far
  }
  if (threadIdx.x == 0) {
    a.head[2 * blockIdx.x] = cut;
    a.head[2 * blockIdx.x + 1] = cut2;
  }
}

// The cut pair that begins in CTA blockIdx.x of the first launch, a warp per
// row: its partial results lie in that CTA's slot 2 c + 1 and in the slots 2 c'
// of the CTAs c' behind it, and are added in that order.
template <int D, int RG>
__global__ void __launch_bounds__(RG * 32) kv8_merge_kernel(const __grid_constant__ AttnArgs a, float p_rest) {
  pdl_trigger();
  pdl_wait();
  if (gated(a.gate)) return;
  const int c0 = blockIdx.x, lane = threadIdx.x & 31, col = threadIdx.x >> 5;
  // what most pairs need is loaded before it is known how many CTAs took part
  constexpr int N = D / 32;
  const float2 *ml = reinterpret_cast<const float2 *>(a.ml);
  auto slot = [&](int i) { return ((int64_t)(i == 0 ? 2 * c0 + 1 : 2 * (c0 + i)) * RG + col); };
  auto load = [&](int i, float (&v)[N]) {
    const float *src = a.part + slot(i) * D + lane * N;
    if constexpr (N == 4) {
      const float4 u = *reinterpret_cast<const float4 *>(src);
      v[0] = u.x; v[1] = u.y; v[2] = u.z; v[3] = u.w;
    } else {
      const float2 u = *reinterpret_cast<const float2 *>(src);
      v[0] = u.x; v[1] = u.y;
    }
  };
  const int last = (int)gridDim.x - 1 - c0;  // slots that exist behind the first
  const int4 cut = a.head[2 * c0], rows = a.head[2 * c0 + 1];
  const float2 early = lane <= last ? ml[slot(lane)] : make_float2(-INFINITY, 0.0f);
  constexpr int kEarly = 4;
  float part[kEarly][N];
#pragma unroll
  for (int i = 0; i < kEarly; ++i) load(min(i, last), part[i]);
  if (cut.x < 0) return;
  const int r = cut.z * RG + col;
  if (r >= a.by_rep.d * rows.y) return;
  const int n = cut.w - c0 + 1;
  float top = lane < n ? early.x : -INFINITY;
  for (int i = lane + 32; i < n; i += 32) top = fmaxf(top, ml[slot(i)].x);
#pragma unroll
  for (int d = 16; d; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
  const float ref = top == -INFINITY ? 0.0f : top;
  float sum = 0.0f, acc[N] = {};
  for (int i0 = 0; i0 < n; i0 += 32) {
    const float2 mine = i0 + lane >= n ? make_float2(-INFINITY, 0.0f) : i0 == 0 ? early : ml[slot(i0 + lane)];
    const float by_mine = exp2_fast(mine.x - ref);
    const int here = min(32, n - i0);
    auto add = [&](int i, const float (&v)[N]) {
      const float by = __shfl_sync(0xffffffffu, by_mine, i);
      sum = fmaf(__shfl_sync(0xffffffffu, mine.y, i), by, sum);
#pragma unroll
      for (int d = 0; d < N; ++d) acc[d] = fmaf(v[d], by, acc[d]);
    };
    int i = 0;
    if (i0 == 0) {
#pragma unroll
      for (int k = 0; k < kEarly; ++k)
        if (k < here) add(k, part[k]);
      i = kEarly;
    }
#pragma unroll 4
    for (; i < here; ++i) {
      float v[N];
      load(i0 + i, v);
      add(i, v);
    }
  }
  const int i = a.by_rep.quotient(r), h = cut.y * a.by_rep.d + r - i * a.by_rep.d;
  const int64_t row = (int64_t)(rows.x + i) * a.n_q_heads + h;
  const float by = p_rest / sum;
#pragma unroll
  for (int d = 0; d < N; d += 2) store2(a.out, a.q.dtype, row * D + dim_of<D>(lane * N + d), acc[d] * by, acc[d + 1] * by);
  if (a.lse && lane == 0) a.lse[row] = (top + log2f(sum)) * kLn2;
}

int mode_of(int dtype, int rep, int max_rows) {
  if (dtype == MK_F32) return kRows8F32;
  return rep * max_rows <= 8 ? kRows8 : kRows16;
}

// Grid and workspace of a call, from what the host knows.
struct AttnPlan {
  int mode, groups, ctas, warps, per_sm;
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
  const int sms = sm_count(c.device);
  const bool crowd = pairs > 4ll * sms && crowd_fits(c.head_dim, p.mode) && (p.pair_mode || c.head_dim == 64);
  if (p.pair_mode) {
    p.ctas = (int)pairs;
    p.warps = pairs <= sms ? 8 : pairs <= 2 * sms ? 4 : 2;
    p.per_sm = crowd ? kCrowd : ctas_per_sm(p.warps);
    return p;
  }
  p.warps = pairs > 2 * sms ? 2 : p.mode == kRows8F32 || pairs > sms ? 4 : 8;
  p.per_sm = crowd ? kCrowd : ctas_per_sm(p.warps);
  p.ctas = (int)std::min<int64_t>((int64_t)sms * p.per_sm, (pairs * chunks + kMinUnits - 1) / kMinUnits);
  p.bytes = (int64_t)p.ctas * (32 + 2 * rg * 8 + 2ll * rg * c.head_dim * 4);
  return p;
}

template <int D, int FMT, int MODE, int W, int CTAS>
cudaError_t launch(const AttnArgs &a, const AttnPlan &p, cudaStream_t st) {
  constexpr int smem = smem_bytes(D, FMT, MODE, W);
  static std::atomic<uint64_t> ready{0};  // devices whose limit has been raised
  const uint64_t bit = a.c.device < 64 ? 1ull << a.c.device : 0;
  cudaError_t e = cudaSuccess;
  if (!(ready.load(std::memory_order_relaxed) & bit)) {
    e = cudaFuncSetAttribute(kv8_attention_kernel<D, FMT, MODE, W, CTAS>,
                             cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    ready.fetch_or(bit, std::memory_order_relaxed);
  }
  e = pdl_launch(kv8_attention_kernel<D, FMT, MODE, W, CTAS>, dim3(p.ctas), W * 32, smem, st, a);
  if (e != cudaSuccess || p.pair_mode) return e;
  return pdl_launch(kv8_merge_kernel<D, group_rows(MODE)>, dim3(p.ctas), group_rows(MODE) * 32, 0, st, a,
                    p_rest(FMT, MODE));
}

template <int D, int FMT, int MODE>
cudaError_t launch(const AttnArgs &a, const AttnPlan &p, cudaStream_t st) {
  if constexpr (crowd_fits(D, MODE))
    if (p.per_sm == kCrowd) return launch<D, FMT, MODE, 2, kCrowd>(a, p, st);
  return p.warps == 2   ? launch<D, FMT, MODE, 2, 4>(a, p, st)
         : p.warps == 4 ? launch<D, FMT, MODE, 4, 2>(a, p, st)
                        : launch<D, FMT, MODE, 8, 1>(a, p, st);
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
  const int64_t chunks = ((int64_t)b->max_pages * c->page_size + kChunk - 1) / kChunk + pair_units(kRows16);
  const int64_t groups = ((int64_t)n_q_heads / c->n_kv_heads * b->max_rows + 7) / 8;
  if ((int64_t)c->n_kv_heads * groups >= (1 << 21)) return "so many heads and rows are not supported";
  // chunks < 2^27, heads x groups < 2^21, sequences <= 2^24: no product of all three
  if (chunks * (c->n_kv_heads * groups) > ((1ll << 30) - 1) / b->n_seqs)
    return "so many positions (page table entries x heads) are not supported";
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
  a.by_rep = Divisor(n_q_heads / cache.n_kv_heads);
  a.by_page = Divisor(cache.page_size);
  a.by_grid = Divisor(p.ctas);
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
