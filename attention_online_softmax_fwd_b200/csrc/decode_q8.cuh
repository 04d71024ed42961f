// Paged decode over an 8-bit cache with one scale per (block of tokens, KV head).
//
// K = ks * kc and V = vs * vc, where kc and vc are E4M3 or int8 codes and ks, vs
// the scales of the token's block. For a query head q and tokens t:
//   x_t = log2(e) * scale * ks_t * sum_d q_d kc_td       (the score in log2 units)
//   O   = sum_t 2^(x_t - X) vs_t vc_t / sum_t 2^(x_t - X),   LSE = ln2 * (X + log2 sum)
// The codes are never widened: they go from shared memory straight into
// tcgen05.mma as the A operand, 128 tokens at a time, and the narrow side is
// split into 8-bit digits:
//   S^T = Kc (128 tokens x D) * [q_hi; q_lo]^T,  q * 2^a = q_hi + q_lo / 16 (E4M3)
//                                          = 256 q_hi + q_lo + q_frac / 128  (int8)
//   O^T = Vc^T (128 dims x 128 tokens) * [p_hi; p_lo]^T,  p likewise
// E4M3: a bf16 value has 8 significant bits, a code 4, so two codes hold q exactly
// down to 2^-14 of the row's largest value; the products accumulate in fp32.
// int8: two digits alone, a 16-bit integer, lose bits below 2^-7 of the row's largest
// value (4e-6 of the LSE at contexts of a few tokens, 100 times an fp32 product's), so q
// takes a third; it too is then exact down to 2^-14, and every product and sum is an
// exact int32. With up to five query rows the third digit needs no wider product.
// The probability that multiplies V is p_t = 2^(y_t - y), y_t = x_t + log2(vs_t) and y
// the largest y_t of the tile: the value scale is part of the exponent, so p <= 1
// whatever the scales are. Two E4M3 digits of 256 p are off by at most 2^-9 of p, or
// 2^-22 where p is below 2^-13; three int8 digits of 32512 p by at most 2^-22. Both are
// steps of a fixed size for small p, so the reference is the tile's own maximum and not
// the running one: a heavy key takes nothing from the tokens of other tiles, and at most
// 127 * 2^-22 of its own weight from its tile's, however long the sequence. (Against the
// running maximum, with two digits for int8, all tokens below 2^-16 of the heaviest were
// lost to O and kept in the sum: half of the tail of 8192 tokens behind a key of weight
// 0.9.)
//
// A tile is 128 tokens x 128 bytes of K and of V: one KV head of D = 128, or two
// neighbouring heads of D = 64 (NH = 2), whose scores come from the two halves of
// the row into columns of their own and whose O^T are the two halves of the lanes.
// So a copy always moves 128-byte rows, and one shape of every product serves both.
// (D = 64 with more than 8 query heads a group takes one head of the row at a time
// and reads the row twice: the digits of both would not fit the tensor memory.)
//
// Work. The batch's tiles in the order (head group, sequence, tile) are cut into as
// many equal runs as there are teams; a team is one CTA for each of up to 8
// neighbouring rows of 128 bytes ("lanes"), which walk the same run. Neighbouring
// 128-byte rows are thus read at about the same time: with each CTA on its own work
// the same copies reach 5.0 to 5.5 TB/s instead of 6.5. A sequence that lies inside a
// run is written at once; the parts of one that is cut are merged by
// decode_q8_merge_kernel, and each CTA has two at most, whatever the lengths. Where
// the block tables hold at most 512 tokens a sequence the runs are of whole sequences:
// nothing is cut, and the merge (2.3 us or more on the GPU, 2.5 on the host) is not
// launched.
//
// A CTA has two softmax warpgroups (one token of a tile per thread), two producer warps
// (one walks the lengths and block tables, copies K by TMA and the scales by
// cp.async, and hands each tile's pages to the other, which copies V: one warp
// takes about 100 cycles to issue a copy, and 16-token pages need 16 of them a
// tile, so with one producer the issue took longer than the tile's share of the
// HBM time, 2570 cycles with two CTAs per SM), a warp that turns the query rows
// into digits and issues the score products, and one that issues the P V products.
// The warpgroups take alternate tiles, each with its own buffers of S^T, P and O^T:
// a tile's way through scores, softmax, P V and accumulation is some 1500 to 3000
// cycles of latency, by the number of query rows, so four tiles a SM are under way
// at a time. The four warps of a warpgroup exchange the tile's maxima of y once, so
// that its 128 tokens share one reference and P V is one accumulation. (Without the
// exchange, each warp keeping a reference and accumulators of its own, O took four
// times the registers and tensor-memory reads: 92 us instead of 73, when it was tried, for
// 16 sequences of 8192 tokens with 8 query heads a group.) O stays in fp32 registers (thread =
// head dimension), the tile's products are brought onto its running reference there
// (by 2^(y - Y), Y the largest y so far), which is why TMEM holds only the tile's own. When the CTA's part of the sequence ends, the warpgroup
// of its last tile adds the other's O, handed over through TMEM.
//
// Bound by HBM up to 8 query rows: 64 sequences of 512 to 8192 tokens (581 MB of E4M3
// codes and scales, 8 KV heads of 128, 4 query heads each) in 99 us with the merge,
// replayed, 5.9 TB/s, and 101 to 106 us a call with other inputs each time; the plain copy
// rate would take 90. One sequence of 32768 tokens (67 MB): 19.2 us, of which some 8 are
// start-up and merge. 32 sequences of 16384 tokens with 8 query heads a group: 195 us E4M3
// and 200 int8, 5.5 and 5.4 TB/s. With 16 rows a thread, one CTA an SM, the softmax sets the
// pace: 8 sequences of 8192 tokens with 16 query heads a group in 58 us (E4M3) and 67 (int8),
// 2.3 and 2.0 TB/s. int8's third digit of P costs 2 % up to 8 rows and 10 % at 16.
#pragma once

#include "decode.cuh"

namespace attn {

constexpr int kQ8Tok = 128;          // tokens per tile
constexpr int kQ8Row = 128;          // bytes of a tile's row
constexpr int kQ8Chunk = 16;         // tokens whose page and scales are looked up together
constexpr int kQ8MaxBox = 64;        // tokens per TMA copy: min(page_size, 64)
constexpr int kQ8SoftmaxWarps = 4;   // of a warpgroup; warpgroups 0 and 1 are softmax, 2 the helpers
constexpr int kQ8KWarp = 2 * kQ8SoftmaxWarps, kQ8VWarp = kQ8KWarp + 1, kQ8ScoreWarp = kQ8KWarp + 2,
              kQ8PvWarp = kQ8KWarp + 3;
constexpr int kQ8Threads = (2 * kQ8SoftmaxWarps + 4) * 32;
constexpr int kQ8Scan = 64;          // sums of tile counts, each over four threads' sequences
constexpr int kQ8MaxTeam = 8;        // lanes of a team
constexpr int kQ8MaxCtas = 320;      // CTAs of a call at most (two on each of 148 SMs); fixes the workspace size

struct DecodeQ8Params {
  const __nv_bfloat16* q;      // [N][Hq][D]
  const int32_t* block_table;  // [N][max_pages]
  const int32_t* seq_lens;     // [N]
  const float* k_scales;       // [num_pages][page_size / block][Hkv]
  const float* v_scales;
  __nv_bfloat16* o;            // [N][Hq][D]
  float* lse;                  // [N][Hq] (natural log) or null
  float* ws_o;                 // [CTA][2][rows][D] fp32 parts of cut sequences (normalised)
  float* ws_lse;               // [CTA][2][rows] their log2-sum-exp
  int4* ws_cut;                // [CTA] the cut sequence whose first part this CTA holds: {seq, group, last team, slot}
  int* status;                 // caller's device status word or null
  int num_seqs, Hq, Hkv, G, max_pages, num_pages, page_size;
  int page_shift;              // log2(page_size)
  int block_shift;             // log2(tokens per scale)
  int box;                     // tokens per TMA copy
  int rows128;                 // 128-byte rows of a token that items are made of (solo: one per KV head)
  int solo;                    // D = 64, one head of a row at a time
  int whole;                   // runs of whole sequences: none is cut
  int team, groups, teams;     // lanes of a team, ceil(rows128 / team), teams
  int part_rows;               // query rows of a part: G, or 2 G for two heads
  float scale_log2;            // softmax scale * log2(e), without the K scale
};

template <int D, int NH, int GP, bool I8>
struct DecodeQ8Smem {
  static constexpr int kR = NH * GP;                       // digit rows: head half * GP + query head
  static constexpr int kN = ((I8 ? 3 : 2) * kR + 15) / 16 * 16;   // columns of a product: hi, lo (and int8's third) digits
  static constexpr int kTileBytes = kQ8Tok * kQ8Row;       // K (or V) codes of one tile
  static constexpr int kStageBytes = 2 * kTileBytes;
  static constexpr int kQBytes = kR * D * 2;               // the query rows of an item
  static constexpr int kBlocks = kR <= 8 ? 2 : 1;          // resident CTAs per SM
  // query rows held: of the part at hand and the next one, or, where those would cost a stage, of one part (the
  // next part's first tile is then copied once this part's rows are digits)
  static constexpr int kQBufs = I8 && kR == 8 ? 1 : 2;
  // digit rows of q and of P, in eights (a product of int8 with R = 8 reads the eight rows behind them as well,
  // into columns that nothing uses)
  static constexpr int kQTile = (!I8 || kR < 8 ? kN : 3 * kR) * kQ8Row, kPTile = kQTile;
  static constexpr int kPerStage = kStageBytes + 64 * NH + 32 + 48 + 24;
  static constexpr int kFixed = 1024 + kQBufs * kQBytes + 2 * kQTile + 2 * kPTile + 4 * (4 * 4 * kR + 2 * 2 * 4 * kR + 2 * kR + 3 * kR) +
                                8 * 18 + 64;
  static constexpr int kFit = (233472 / kBlocks - 1024 - kFixed) / kPerStage;
  static constexpr int kStages = kFit < 8 ? kFit : 8;
  static constexpr int kQT = kStages * kStageBytes;                    // q digits [item parity], 1024-byte aligned
  static constexpr int kPT = kQT + 2 * kQTile;                         // P digits [tile parity]
  static constexpr int kQRows = kPT + 2 * kPTile;                      // query rows [part parity, if two]
  static constexpr int kScales = kQRows + kQBufs * kQBytes;                 // [stage][head half][K 8 | V 8] floats
  static constexpr int kInfo = kScales + 64 * NH * kStages;               // TileInfo per stage
  static constexpr int kJob = kInfo + 32 * kStages;                    // V copies of a stage: 8 pages, t0, byte, mask
  static constexpr int kYmax = (kJob + 48 * kStages + 15) / 16 * 16;   // [warpgroup][use parity][kR][warp] floats
  static constexpr int kMl = kYmax + 4 * 4 * 4 * kR;                   // [warpgroup][warp][kR] x {X, l} floats
  static constexpr int kQf = kMl + 4 * 2 * 2 * 4 * kR;                 // [part parity][kR] floats
  static constexpr int kSwap = kQf + 4 * 2 * kR;                       // [kR] x {X, Y, l} of the other warpgroup
  static constexpr int kBars = (kSwap + 4 * 3 * kR + 7) / 8 * 8;       // mbarriers
  static constexpr int kScan = kScales;                    // sums of tile counts, read before the first scales are copied
  // full[kStages], empty[kStages], v_go[kStages], s_full[2], s_free[2], p_ready[2], o_full[2], q_ready[2],
  // ml_ready[2], done[2], y_ready[2], swap_full, swap_free
  static constexpr int kTotal = kBars + 8 * (3 * kStages + 18);
  static constexpr int kDynamic = kTotal + 1024;
  static constexpr int kSBuf = NH * kN;                    // columns of one score buffer: kN for each head half
  static constexpr int kTmemSwap = 2 * kSBuf + 2 * kN;     // O of the warpgroup that does not finish a part
  static constexpr int kTmemUse = kTmemSwap + GP;
  // registers of a helper and of a softmax thread; together they are the block's launch allocation
  static constexpr int kHelperRegs = kBlocks == 1 ? 80 : 64, kSoftmaxRegs = kBlocks == 1 ? 208 : 88;
  static constexpr int kRegPool = 128 * kHelperRegs + 256 * kSoftmaxRegs;
  static constexpr int kTmemCols = kTmemUse <= 128 ? 128 : kTmemUse <= 256 ? 256 : 512;
  static_assert(kDynamic <= 233472 / kBlocks - 1024, "shared memory per block");
  static_assert(kStages >= 3, "ring depth");
  static_assert(kStages * (64 * NH + 32) >= 4 * kQ8Scan, "the sums lie in the scales and tile infos");
  static_assert(kQ8Scan * 4 <= kQ8Threads, "four threads a sum");
  static_assert(kTmemUse <= kTmemCols && kTmemCols * kBlocks <= 512, "tensor memory");
  static_assert(kR <= 16, "digit rows");
  static_assert(kPT + 2 * kPTile + (kN * kQ8Row - kPTile) <= kTotal, "rows read behind the last digits");
};

// mbar_wait with its limit counted in clock cycles (4e9, at least two seconds): reading %globaltimer takes
// long enough to show in every wait of a tile that does not succeed at once.
__device__ __forceinline__ bool q8_wait(uint64_t* bar, uint32_t parity, volatile int* abort_flag, int* user_status) {
  if (mbar_try_wait(bar, parity)) return true;
  const long long t0 = clock64();
  for (uint32_t i = 1;; ++i) {
    if (mbar_try_wait(bar, parity)) return true;
    if ((i & 31u) == 0) {
      if (*abort_flag) return false;
      if (clock64() - t0 > 4000000000ll) {
        *abort_flag = 1;
        raise_status(user_status, ATTN_ERR_TIMEOUT);
        return false;
      }
    }
  }
}

__device__ __forceinline__ void tma_load_3d(void* dst, const CUtensorMap* map, uint64_t* bar, int c0, int c1, int c2) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(c0), "r"(c1), "r"(c2)
      : "memory");
}
// 4-byte asynchronous copies, and their arrival on an mbarrier once they have landed.
__device__ __forceinline__ void cp_async4(void* dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_arrive_noinc(uint64_t* bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}
__device__ __forceinline__ void cp_async_wait_all() { asm volatile("cp.async.wait_all;" ::: "memory"); }

// D[tmem] (+)= A[smem] * B[smem]^T on 8-bit operands (K = 32): E4M3 -> fp32, or int8 -> int32.
template <bool I8>
__device__ __forceinline__ void umma_q8(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                        uint32_t accumulate) {
  if constexpr (I8)
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::i8 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}
// Instruction descriptor: E4M3 x E4M3 -> f32 (formats 0, 0, 1) or s8 x s8 -> s32 (1, 1, 2).
template <bool I8>
__host__ __device__ constexpr uint32_t make_idesc_q8(int M, int N, int a_mn_major) {
  return (uint32_t(I8 ? 2 : 1) << 4) | (uint32_t(I8 ? 1 : 0) << 7) | (uint32_t(I8 ? 1 : 0) << 10) |
         (uint32_t(a_mn_major) << 15) | (uint32_t(N >> 3) << 17) | (uint32_t(M >> 4) << 24);
}
// Shared-memory descriptor of a tile of 128-byte rows under the 128-byte swizzle, its eight-row
// atoms 1024 bytes apart (both for K-major and for MN-major operands of 128 bytes).
__device__ __forceinline__ uint64_t make_sdesc_rows(uint32_t smem_addr) { return make_sdesc_sw128(smem_addr, 16, 1024); }
// Byte offset of 16-byte unit c of row r in such a tile.
__device__ __forceinline__ uint32_t row_unit(int r, int c) { return uint32_t(r * 128 + ((c ^ (r & 7)) << 4)); }

// NC columns of 32-bit TMEM of this warp's 32 lanes -> registers; no wait (tmem_ld_wait, then reg_fence).
template <int NC>
__device__ __forceinline__ void tmem_ld_cols(uint32_t taddr, uint32_t* r) {
  static_assert(NC == 1 || NC == 2 || NC == 4 || NC == 8 || NC == 16 || NC == 32, "columns");
  if constexpr (NC == 1) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x1.b32 {%0}, [%1];" : "=r"(r[0]) : "r"(taddr) : "memory");
  } else if constexpr (NC == 2) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x2.b32 {%0,%1}, [%2];" : "=r"(r[0]), "=r"(r[1]) : "r"(taddr) : "memory");
  } else if constexpr (NC == 4) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x4.b32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(taddr)
                 : "memory");
  } else if constexpr (NC == 8) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                 : "r"(taddr)
                 : "memory");
  } else {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr)
        : "memory");
    if constexpr (NC == 32) tmem_ld_cols<16>(taddr + 16, r + 16);
  }
}
template <int NC>
__device__ __forceinline__ void tmem_st_cols(uint32_t taddr, const uint32_t* r) {
  if constexpr (NC == 1) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x1.b32 [%0], {%1};" ::"r"(taddr), "r"(r[0]) : "memory");
  } else if constexpr (NC == 2) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x2.b32 [%0], {%1,%2};" ::"r"(taddr), "r"(r[0]), "r"(r[1]) : "memory");
  } else {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x4.b32 [%0], {%1,%2,%3,%4};" ::"r"(taddr), "r"(r[0]), "r"(r[1]),
                 "r"(r[2]), "r"(r[3])
                 : "memory");
    if constexpr (NC > 4) tmem_st_cols<NC - 4>(taddr + 4, r + 4);
  }
}
template <int NC>
__device__ __forceinline__ void reg_fence(uint32_t* r) {
#pragma unroll
  for (int i = 0; i < NC; ++i) asm volatile("" : "+r"(r[i]));
}

// Warp maximum that keeps a NaN, and the maximum of two values that keeps a NaN.
__device__ __forceinline__ float warp_max_nan(float x) {
  float y;
  asm("redux.sync.max.NaN.f32 %0, %1, 0xffffffff;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float max_nan(float a, float b) {
  float y;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(b));
  return y;
}
// Two floats -> two E4M3 codes (lo in the low byte), to nearest even, saturating; and back.
__device__ __forceinline__ uint32_t e4m3x2_of(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ void e4m3x2_back(uint32_t codes, float& lo, float& hi) {
  uint32_t h2;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h2) : "h"(static_cast<uint16_t>(codes)));
  lo = f16_lo(h2);
  hi = f16_hi(h2);
}
// Two values as two digits each: E4M3 v = hi + lo / 16, int8 v = 256 hi + lo, to the nearest integer.
// Bytes: first value's digit in the low byte, the second's in the next.
template <bool I8>
__device__ __forceinline__ void two_digits(float v0, float v1, uint32_t& hi, uint32_t& lo) {
  if constexpr (I8) {
    const int i0 = __float2int_rn(v0), i1 = __float2int_rn(v1);
    hi = (uint32_t((i0 + 128) >> 8) & 0xFFu) | ((uint32_t((i1 + 128) >> 8) & 0xFFu) << 8);
    lo = (uint32_t(i0) & 0xFFu) | ((uint32_t(i1) & 0xFFu) << 8);
  } else {
    hi = e4m3x2_of(v0, v1);
    float b0, b1;
    e4m3x2_back(hi, b0, b1);
    lo = e4m3x2_of((v0 - b0) * 16.f, (v1 - b1) * 16.f);
  }
}
// int8: what rounding two values to integers left over (half at most), in units of 1 / kQ8Frac.
constexpr float kQ8Frac = 128.f;
__device__ __forceinline__ uint32_t third_digits(float v0, float v1) {
  const int i0 = __float2int_rn((v0 - rintf(v0)) * kQ8Frac), i1 = __float2int_rn((v1 - rintf(v1)) * kQ8Frac);
  return (uint32_t(i0) & 0xFFu) | ((uint32_t(i1) & 0xFFu) << 8);
}
// The value of the accumulated digit columns (E4M3 has no third one).
template <bool I8>
__device__ __forceinline__ float join_digits(uint32_t hi, uint32_t lo, uint32_t frac) {
  if constexpr (I8)   // |256 hi + lo| < 2^30: 128 products of at most 2^15 * 2^7
    return fmaf(float(int(frac)), 1.f / kQ8Frac, float(int(hi) * 256 + int(lo)));
  else
    return fmaf(__uint_as_float(lo), 0.0625f, __uint_as_float(hi));
}

// Units of work of a sequence of (clamped) length `len`: its tiles, or one for all of it.
__device__ __forceinline__ int q8_units(int len, int whole) { return whole ? min(len, 1) : (len + kQ8Tok - 1) / kQ8Tok; }
__device__ __forceinline__ int q8_clamp_len(int len, int capacity) { return len < 0 ? 0 : min(len, capacity); }

template <int D, int NH, int GP, bool I8>
__global__ void __launch_bounds__(kQ8Threads, DecodeQ8Smem<D, NH, GP, I8>::kBlocks)
    decode_q8_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                     const DecodeQ8Params p) {
  static_assert(D == 64 || (D == 128 && NH == 1), "heads of a 128-byte row");
  using L = DecodeQ8Smem<D, NH, GP, I8>;
  launch_dependents();   // the merge is scheduled early; it waits for this grid to finish
  constexpr int NS = L::kStages;
  constexpr int KN = L::kN;
  constexpr int R = L::kR;

  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  float* scales = reinterpret_cast<float*>(smem + L::kScales);
  TileInfo* info = reinterpret_cast<TileInfo*>(smem + L::kInfo);
  int* scan = reinterpret_cast<int*>(smem + L::kScan);
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + L::kBars);
  uint64_t* empty = full + NS;
  uint64_t* v_go = empty + NS;       // a stage's V copies may be issued
  uint64_t* s_full = v_go + NS;      // [2]
  uint64_t* s_free = s_full + 2;     // [2]
  uint64_t* p_ready = s_free + 2;    // [2]
  uint64_t* o_full = p_ready + 2;    // [2]
  uint64_t* q_ready = o_full + 2;    // [2]
  uint64_t* ml_ready = q_ready + 2;  // [2]
  uint64_t* done = ml_ready + 2;     // [2]
  uint64_t* y_ready = done + 2;      // [2]
  uint64_t* swap_full = y_ready + 2;
  uint64_t* swap_free = swap_full + 1;
  __shared__ int abort_word;
  __shared__ uint32_t tmem_slot;
  volatile int* abort_flag = &abort_word;

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int capacity = p.max_pages * p.page_size;

  // tiles of each scan entry's share of the sequences, summed by four threads, the loads first. (A sum fits
  // an int: sequences of 2^30 tokens would need block tables of terabytes first.)
  const int per_entry = (p.num_seqs + kQ8Scan - 1) / kQ8Scan;
  const int scan_at = (threadIdx.x >> 2) * per_entry + (threadIdx.x & 3);
  const int scan_end = threadIdx.x < 4 * kQ8Scan ? min((int(threadIdx.x >> 2) + 1) * per_entry, p.num_seqs) : 0;
  int first_len = scan_at < scan_end ? __ldg(&p.seq_lens[scan_at]) : 0;
  // the first 32 lengths, which the K warp walks if its work starts there
  const int window0 = warp == kQ8KWarp && lane < p.num_seqs ? __ldg(&p.seq_lens[lane]) : 0;

  if (warp == kQ8PvWarp) {
    if (lane == 0) abort_word = 0;
    if (lane < NS) {
      mbar_init(&full[lane], 33);    // the producer's expect_tx arrival and its 32 lanes' scale copies
      mbar_init(&empty[lane], 2);    // the stage's P V products, and the V warp (which a stage without copies needs)
      mbar_init(&v_go[lane], 1);
    } else if (lane < NS + 2) {
      const int i = lane - NS;
      mbar_init(&s_full[i], 1);
      mbar_init(&s_free[i], kQ8SoftmaxWarps);
      mbar_init(&p_ready[i], kQ8SoftmaxWarps);
      mbar_init(&o_full[i], 1);
      mbar_init(&q_ready[i], 1);
      mbar_init(&done[i], 1);
      mbar_init(&ml_ready[i], kQ8SoftmaxWarps);
      mbar_init(&y_ready[i], kQ8SoftmaxWarps);
      mbar_init(i == 0 ? swap_full : swap_free, kQ8SoftmaxWarps);
    }
    fence_mbar_init();
  } else if (warp < 2 * kQ8SoftmaxWarps) {
    // digit rows that no query head uses stay zero (q and P digits follow one another)
    for (int i = threadIdx.x * 16; i < 2 * (L::kQTile + L::kPTile); i += 2 * kQ8SoftmaxWarps * 32 * 16)
      *reinterpret_cast<uint4*>(smem + L::kQT + i) = make_uint4(0, 0, 0, 0);
    fence_proxy_async_smem();
  } else if (lane == 0) {
    if (warp == kQ8KWarp) tma_prefetch_desc(&tm_k);
    if (warp == kQ8VWarp) tma_prefetch_desc(&tm_v);
  }
  {
    int sum = 0;
    for (int i = scan_at; i < scan_end; i += 4) {
      const int len = i == scan_at ? first_len : __ldg(&p.seq_lens[i]);
      if (blockIdx.x == 0 && (len < 0 || len > capacity)) raise_status(p.status, ATTN_ERR_DEVICE_BOUNDS);
      sum += q8_units(q8_clamp_len(len, capacity), p.whole);
    }
    sum += __shfl_xor_sync(0xffffffffu, sum, 1);
    sum += __shfl_xor_sync(0xffffffffu, sum, 2);
    if ((threadIdx.x & 3) == 0 && threadIdx.x < 4 * kQ8Scan) scan[threadIdx.x >> 2] = sum;
  }
  if (warp == kQ8ScoreWarp) {
    tmem_alloc(&tmem_slot, L::kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_slot;
  const uint32_t tmem_s = tmem;                    // two buffers of kSBuf columns
  const uint32_t tmem_o = tmem + 2 * L::kSBuf;     // two buffers of KN columns

  if (warp == kQ8KWarp) {
    // ------------------------------------------------------------ producer warp: work, K, scales
    setmaxnreg_dec<L::kHelperRegs>();
    const int c = lane & 7;            // lane: chunk c of the tile; bit 3: V scales; bit 4: second head of the row
    const bool box_lane = lane < 8 && (c & (p.box / kQ8Chunk - 1)) == 0;   // lane of a copy's first chunk
    const float* sc_src = (lane & 8) ? p.v_scales : p.k_scales;
    const int blocks_per_page = p.page_size >> p.block_shift;
    const int team = int(blockIdx.x) / p.team;
    const int team_lane = int(blockIdx.x) % p.team;

    // ---- this team's run of the batch's tiles, and the sequence where it starts. (A CTA runs this code once,
    // at the speed of its instruction fetches: it is kept short, and in 32 bits; the host bounds the tiles.)
    const int mine = scan[2 * lane] + scan[2 * lane + 1];
    int incl = mine;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int up = __shfl_up_sync(0xffffffffu, incl, d);
      if (lane >= d) incl += up;
    }
    const int per_group = __shfl_sync(0xffffffffu, incl, 31);
    const int total = per_group * p.groups;
    // where tiles are few, about two a team, since a cut costs as much as a tile; every team that works has one at
    // least, so none lies without work between two parts of a sequence
    const int teams = min(p.whole ? total : (total + 1) / 2, p.teams);
    const int quot = teams > 0 ? total / teams : 0, extra = total - quot * teams;   // the first `extra` have one more
    const bool work = team < teams;
    const int begin = work ? team * quot + min(team, extra) : 0;
    const int end = work ? begin + quot + (team < extra ? 1 : 0) : 0;
    int pos = begin;
    int grp = 0, seq = 0, a = 0;       // next tile: tile a of (group, sequence)
    int win = 0, win_len = q8_clamp_len(window0, capacity);   // lengths of sequences 32 win .., one per lane
    auto len_at = [&](int s) -> int {
      if ((s >> 5) != win) {
        win = s >> 5;
        const int i = win * 32 + lane;
        win_len = i < p.num_seqs ? q8_clamp_len(__ldg(&p.seq_lens[i]), capacity) : 0;
      }
      return __shfl_sync(0xffffffffu, win_len, s & 31);
    };
    if (work) {
      int x = begin;
      if (p.groups > 1) {
        grp = x / per_group;
        x -= grp * per_group;
      }
      const int l0 = __ffs(int(__ballot_sync(0xffffffffu, incl > x))) - 1;   // some lane: x < per_group
      x -= __shfl_sync(0xffffffffu, incl - mine, l0);
      int t = 2 * l0;
      if (x >= scan[t]) x -= scan[t++];
      __syncwarp();                    // the sums have been read: scales may be copied over them
      seq = t * per_entry;
      for (int units; x >= (units = q8_units(len_at(seq), p.whole)); ++seq) x -= units;
      a = x;
    }
    auto page_of = [&](int s, int t0) -> int {   // physical page of chunk c of the tile at t0
      const int e = (t0 + c * kQ8Chunk) >> p.page_shift;
      return e < p.max_pages ? __ldg(&p.block_table[size_t(s) * p.max_pages + e]) : -1;
    };
    // the part at hand (a run of tiles of one sequence) and the next one, taken while the first tile of this
    // one is on its way, its first pages requested
    struct Part { int seq, grp, t_begin, t_end, n, tiles, pos; };
    Part nx{}, w{};
    int nx_page = -1, page = -1;
    int row = 0, part = 0, head0 = 0, head = 0, byte = 0, q_rows = 0;
    bool head_ok = false;
    int t0 = 0;
    int4 cut = make_int4(-1, 0, 0, 0);
    int slot = 0;
    uint32_t phase = 0;
    uint32_t pending = 0, pending_phase = 0;
    bool ok = true, fetch = true;
    int part_no = -1;
    for (;;) {
      if (fetch) {
        fetch = false;
        nx.n = 0;
        if (pos < end) {
          int len, tiles;
          for (;;) {
            if (seq == p.num_seqs) { seq = 0; ++grp; }
            len = len_at(seq);
            tiles = q8_units(len, p.whole);
            if (tiles > a) break;
            ++seq;
            a = 0;
          }
          nx.seq = seq; nx.grp = grp; nx.tiles = tiles; nx.pos = pos;
          nx.n = min(tiles - a, end - pos);
          nx.t_begin = a * kQ8Tok;
          nx.t_end = p.whole ? len : min((a + nx.n) * kQ8Tok, len);
          nx_page = page_of(seq, nx.t_begin);
          pos += nx.n;
          a += nx.n;
          if (a == tiles) { a = 0; ++seq; }
        }
      }
      if (t0 >= w.t_end) {   // the next part
        if (nx.n == 0) break;
        w = nx;
        ++part_no;
        t0 = w.t_begin;
        page = nx_page;
        row = w.grp * p.team + team_lane;                // 128-byte row of the tokens
        if (row >= p.rows128) break;                     // a lane past the last row: in the last group only
        const bool whole = w.n == w.tiles;
        part = whole ? -1 : int(blockIdx.x) * 2 + (w.pos == begin ? 0 : 1);
        if (!whole && w.t_begin == 0) {   // the first part of a cut sequence, this CTA's last work
          const int last = w.pos + w.tiles - 1, wide = extra * (quot + 1);   // its last tile, and that one's team
          cut = make_int4(w.seq, w.grp, last < wide ? last / (quot + 1) : extra + (last - wide) / quot, part & 1);
        }
        head0 = NH == 2 ? row * 2 : row;                 // first KV head of the row's query rows
        head = head0 + (NH == 2 ? lane >> 4 : 0);
        head_ok = head < p.Hkv && (NH == 2 || lane < 16);
        byte = (p.solo ? row >> 1 : row) * kQ8Row;
        q_rows = min(NH * p.G, p.Hq - head0 * p.G);
      }
      const int page_next = t0 + kQ8Tok < w.t_end ? page_of(w.seq, t0 + kQ8Tok) : -1;
      const int ntok = min(kQ8Tok, w.t_end - t0);
      const bool in_range = page >= 0 && page < p.num_pages;
      const bool held = c * kQ8Chunk < ntok;
      const bool good = held && in_range;
      const uint32_t good_mask = __ballot_sync(0xffffffffu, good) & 0xFFu;
      const uint32_t box_mask = __ballot_sync(0xffffffffu, good && box_lane);   // copies to issue
      if (__any_sync(0xffffffffu, held && !in_range) && lane == 0) raise_status(p.status, ATTN_ERR_DEVICE_BOUNDS);
      const int in_page = (t0 + c * kQ8Chunk) & (p.page_size - 1);
      const bool copy_scale = good && head_ok;
      const float* sc = sc_src + (copy_scale ? (size_t(page) * blocks_per_page + (in_page >> p.block_shift)) * p.Hkv + head
                                             : size_t(0));
      const bool first = t0 == w.t_begin;
      int* job = reinterpret_cast<int*>(smem + L::kJob) + slot * 12;
      ok = __all_sync(0xffffffffu, q8_wait(&empty[slot], phase ^ 1u, abort_flag, p.status));
      // the query rows that the part's own are copied over have been turned into digits
      const int q_before = part_no - L::kQBufs;
      if (first && q_before >= 0)
        ok = __all_sync(0xffffffffu, ok && q8_wait(&q_ready[q_before & 1], uint32_t(q_before >> 1) & 1u, abort_flag, p.status));
      if (!ok) break;
      if (lane < 8) job[lane] = page;
      if (lane == 0) {
        job[8] = t0;
        job[9] = byte;
        job[10] = int(box_mask);
        TileInfo ti;
        ti.seq = w.seq; ti.split = part; ti.kvh = row; ti.t0 = t0;
        ti.ntok = ntok;
        ti.bad = int(~good_mask & 0xFFu);
        // 1: first tile of the part; 2: last; 8: its warpgroup's last of the part; 16: the part has several
        ti.flags = (first ? 1 : 0) | (t0 + kQ8Tok >= w.t_end ? 2 : 0) | (t0 + 2 * kQ8Tok >= w.t_end ? 8 : 0) |
                   (w.t_end - w.t_begin > kQ8Tok ? 16 : 0);
        ti.len = part_no;
        info[slot] = ti;
        const uint32_t qbytes = first ? uint32_t(q_rows * D * 2) : 0u;
        mbar_arrive_expect_tx(&full[slot], uint32_t(__popc(box_mask)) * uint32_t(2 * kQ8Row * p.box) + qbytes);
        if (first)
          bulk_load(smem + L::kQRows + (part_no & (L::kQBufs - 1)) * L::kQBytes, p.q + (size_t(w.seq) * p.Hq + size_t(head0) * p.G) * D, qbytes,
                    &full[slot]);
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&v_go[slot]);
      if ((box_mask >> lane) & 1)
        tma_load_3d(smem + slot * L::kStageBytes + c * (kQ8Chunk * kQ8Row), &tm_k, &full[slot], byte, in_page, page);
      if (copy_scale) cp_async4(scales + slot * 16 * NH + lane, sc);
      cp_async_arrive_noinc(&full[slot]);
      __syncwarp();
      pending |= 1u << slot;
      pending_phase = (pending_phase & ~(1u << slot)) | (phase << slot);
      if (++slot == NS) { slot = 0; phase ^= 1u; }
      page = page_next;
      t0 += kQ8Tok;
      fetch = first;
    }
    if (lane == 0 && !p.whole) p.ws_cut[blockIdx.x] = cut;
    for (int i = 0; i < 2 && ok; ++i) {   // end-of-work markers, one for each warpgroup: stages with no copies
      ok = __all_sync(0xffffffffu, q8_wait(&empty[slot], phase ^ 1u, abort_flag, p.status));
      if (!ok) break;
      if (lane == 0) {
        TileInfo ti{};
        ti.flags = 4;
        info[slot] = ti;
        reinterpret_cast<int*>(smem + L::kJob)[slot * 12 + 10] = -1;
        mbar_arrive_expect_tx(&full[slot], 0u);
        mbar_arrive(&v_go[slot]);
      }
      __syncwarp();
      cp_async_arrive_noinc(&full[slot]);
      if (++slot == NS) { slot = 0; phase ^= 1u; }
    }
    cp_async_wait_all();
    if (!ok && lane == 0) {
      for (int s = 0; s < NS; ++s)
        if (pending & (1u << s)) mbar_drain(&full[s], (pending_phase >> s) & 1u);
    }
  } else if (warp == kQ8VWarp) {
    // ------------------------------------------------------------ producer warp: V, as the first one says
    setmaxnreg_dec<L::kHelperRegs>();
    for (int s = blockIdx.x; s < p.num_seqs; s += gridDim.x) {   // sequences without tokens
      if (__ldg(&p.seq_lens[s]) > 0) continue;
      uint4* rows = reinterpret_cast<uint4*>(p.o + size_t(s) * p.Hq * D);
      for (int i = lane; i < p.Hq * (D / 8); i += 32) rows[i] = make_uint4(0, 0, 0, 0);
      if (p.lse)
        for (int h = lane; h < p.Hq; h += 32) p.lse[size_t(s) * p.Hq + h] = -__int_as_float(0x7f800000);
    }
    int slot = 0;
    uint32_t phase = 0;
    while (__all_sync(0xffffffffu, q8_wait(&v_go[slot], phase, abort_flag, p.status))) {
      const int* job = reinterpret_cast<const int*>(smem + L::kJob) + slot * 12;
      const int mask = job[10];
      if (mask < 0) break;   // end of work
      if (lane < 8 && ((mask >> lane) & 1)) {
        const int in_page = (job[8] + lane * kQ8Chunk) & (p.page_size - 1);
        tma_load_3d(smem + slot * L::kStageBytes + L::kTileBytes + lane * (kQ8Chunk * kQ8Row), &tm_v, &full[slot], job[9],
                    in_page, job[lane]);
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&empty[slot]);
      if (++slot == NS) { slot = 0; phase ^= 1u; }
    }
  } else if (warp == kQ8ScoreWarp) {
    // ------------------------------------------------------------ query digits and score products
    setmaxnreg_dec<L::kHelperRegs>();
    constexpr uint32_t idesc_s = make_idesc_q8<I8>(kQ8Tok, KN, 0);   // K tile: rows = tokens, K-major
    const uint64_t q_desc0 = make_sdesc_rows(smem_u32(smem + L::kQT));
    const uint64_t k_desc0 = make_sdesc_rows(smem_u32(smem));
    int slot = 0, sb = 0, qb = 1;
    uint32_t phase = 0, f_ph = 1;   // a fresh s_free lets the first two tiles pass
    while (__all_sync(0xffffffffu, q8_wait(&full[slot], phase, abort_flag, p.status))) {
      const int flags = info[slot].flags, row = info[slot].kvh;
      if (flags & 4) break;
      if (!__all_sync(0xffffffffu, q8_wait(&s_free[sb], f_ph, abort_flag, p.status))) break;
      const int half = D == 64 && NH == 1 ? row & 1 : 0;   // solo: the head's half of the row
      if (flags & 1) {
        // the item's query rows as digits, scaled by a power of two (exact). The buffer's last reader, the
        // item before the previous one, is done: the scores of the tile two before this one have been read
        qb ^= 1;
        uint8_t* q_tile = smem + L::kQT + qb * L::kQTile;
        float* qf = reinterpret_cast<float*>(smem + L::kQf) + qb * R;
        const int head0 = NH == 2 ? row * 2 : row;
        const int n_rows = NH == 2 && head0 + 1 >= p.Hkv ? p.G : NH * p.G;
        // eight lanes a row, D / 8 values each, four rows at a time
        constexpr int E = D / 8;
        const int part8 = lane & 7;
        for (int i0 = 0; i0 < n_rows; i0 += 4) {
          const int i = min(i0 + (lane >> 3), n_rows - 1);   // a repeated last row writes the same again
          const int nh = NH == 2 && i >= p.G ? 1 : 0;
          const int r = nh * GP + (i - nh * p.G);            // digit row
          const uint4* src = reinterpret_cast<const uint4*>(smem + L::kQRows + (qb & (L::kQBufs - 1)) * L::kQBytes + (i * D + part8 * E) * 2);
          uint32_t w[E / 2];
          uint32_t top = 0;
#pragma unroll
          for (int k = 0; k < E / 8; ++k) {
            const uint4 v = src[k];
            w[4 * k] = v.x; w[4 * k + 1] = v.y; w[4 * k + 2] = v.z; w[4 * k + 3] = v.w;
          }
#pragma unroll
          for (int k = 0; k < E / 2; ++k) top = __vmaxu2(top, w[k] & 0x7FFF7FFFu);
          top = max(top & 0xFFFF0000u, top << 16);
#pragma unroll
          for (int d = 1; d < 8; d <<= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, d));
          const int e = int(top >> 23) - 127, mant = int(top >> 16) & 0x7F;
          const bool finite = top < 0x7F800000u;
          // the largest value lands in (224, 448] or [16320, 32639]
          int sh = I8 ? 14 - e - (mant == 0x7F ? 1 : 0) : 8 - e - (mant > 0x60 ? 1 : 0);
          sh = min(sh, 118);
          const float up = finite ? __uint_as_float(uint32_t(sh + 127) << 23) : 0.f;
          if (part8 == 0)
            qf[r] = finite ? p.scale_log2 * __uint_as_float(uint32_t(127 - sh) << 23) : __int_as_float(0x7fc00000);
          uint32_t hi[E / 4], lo[E / 4], frac[E / 4];
#pragma unroll
          for (int k = 0; k < E / 4; ++k) {
            uint32_t h0 = 0, l0 = 0, h1 = 0, l1 = 0, f0 = 0, f1 = 0;
            if (finite) {
              two_digits<I8>(bf16_lo(w[2 * k]) * up, bf16_hi(w[2 * k]) * up, h0, l0);
              two_digits<I8>(bf16_lo(w[2 * k + 1]) * up, bf16_hi(w[2 * k + 1]) * up, h1, l1);
              if constexpr (I8) {
                f0 = third_digits(bf16_lo(w[2 * k]) * up, bf16_hi(w[2 * k]) * up);
                f1 = third_digits(bf16_lo(w[2 * k + 1]) * up, bf16_hi(w[2 * k + 1]) * up);
              }
            }
            hi[k] = h0 | (h1 << 16);
            lo[k] = l0 | (l1 << 16);
            frac[k] = f0 | (f1 << 16);
          }
          const int at = (half + nh) * 64 + part8 * E;       // byte of the row
          uint8_t* hi_at = q_tile + row_unit(r, at >> 4) + (at & 15);
          uint8_t* lo_at = q_tile + row_unit(R + r, at >> 4) + (at & 15);
          if constexpr (I8) {
            uint8_t* frac_at = q_tile + row_unit(2 * R + r, at >> 4) + (at & 15);
            if constexpr (E == 16) *reinterpret_cast<uint4*>(frac_at) = make_uint4(frac[0], frac[1], frac[2], frac[3]);
            else *reinterpret_cast<uint2*>(frac_at) = make_uint2(frac[0], frac[1]);
          }
          if constexpr (E == 16) {
            *reinterpret_cast<uint4*>(hi_at) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
            *reinterpret_cast<uint4*>(lo_at) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
          } else {
            *reinterpret_cast<uint2*>(hi_at) = make_uint2(hi[0], hi[1]);
            *reinterpret_cast<uint2*>(lo_at) = make_uint2(lo[0], lo[1]);
          }
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&q_ready[qb]);
      }
      if (lane == 0) {
        tc_fence_after();
        const uint64_t k_desc = k_desc0 + uint64_t(slot * (L::kStageBytes >> 4)) + (D == 64 && NH == 1 ? 4 * half : 0);
        const uint64_t q_desc = q_desc0 + uint64_t(qb * (L::kQTile >> 4)) + (D == 64 && NH == 1 ? 4 * half : 0);
        // each head's products run over its own bytes of the row alone, so that a NaN code of one head does
        // not reach the other's scores
#pragma unroll
        for (int h = 0; h < NH; ++h)
#pragma unroll
          for (int k = 0; k < D / 32; ++k)
            umma_q8<I8>(tmem_s + sb * L::kSBuf + h * KN, k_desc + 2 * (h * (D / 32) + k), q_desc + 2 * (h * (D / 32) + k),
                        idesc_s, k > 0);
        umma_commit(&s_full[sb]);
      }
      __syncwarp();
      if (++slot == NS) { slot = 0; phase ^= 1u; }
      if (sb) f_ph ^= 1u;
      sb ^= 1;
    }
    if (lane == 0) {
      umma_commit(&done[0]);   // nothing of this thread is in flight when TMEM is given back
      mbar_drain(&done[0], 0);
    }
    __syncwarp();
  } else if (warp == kQ8PvWarp) {
    // ------------------------------------------------------------ P V products (one thread)
    setmaxnreg_dec<L::kHelperRegs>();
    if (lane == 0) {
      constexpr uint32_t idesc_o = make_idesc_q8<I8>(kQ8Row, KN, 1);   // V tile: rows = head dims, MN-major
      const uint64_t p_desc0 = make_sdesc_rows(smem_u32(smem + L::kPT));
      const uint64_t v_desc0 = make_sdesc_rows(smem_u32(smem + L::kTileBytes));
      int slot = 0, pb = 0;
      uint32_t phase = 0, p_ph = 0;
      while (q8_wait(&full[slot], phase, abort_flag, p.status)) {
        if (info[slot].flags & 4) break;
        if (!q8_wait(&p_ready[pb], p_ph, abort_flag, p.status)) break;
        tc_fence_after();
        const uint64_t v_desc = v_desc0 + uint64_t(slot * (L::kStageBytes >> 4));
        const uint64_t p_desc = p_desc0 + uint64_t(pb * (L::kPTile >> 4));
#pragma unroll
        for (int w = 0; w < 4; ++w)   // tokens 32w .. 32w + 31
          umma_q8<I8>(tmem_o + pb * KN, v_desc + uint64_t(w * (32 * kQ8Row >> 4)), p_desc + 2 * w, idesc_o, w > 0);
        umma_commit(&o_full[pb]);
        umma_commit(&empty[slot]);    // the tile's products are done with its K and V
        if (++slot == NS) { slot = 0; phase ^= 1u; }
        if (pb) p_ph ^= 1u;
        pb ^= 1;
      }
      umma_commit(&done[1]);
      mbar_drain(&done[1], 0);
    }
    __syncwarp();
  } else {
    // ------------------------------------------------------------ softmax warps: thread = token, then head dim
    setmaxnreg_inc<L::kSoftmaxRegs>();
    const float neg_inf = -__int_as_float(0x7f800000);
    // running maxima start below every score that is not -inf, and are finite, so that differences are numbers
    constexpr float kFloor = -3.402823466e38f;
    const int wg = warp >> 2, ww = warp & 3;
    const uint32_t lane_base = uint32_t(ww * 32) << 16;
    const int tok = ww * 32 + lane;           // also the byte of the row whose O this thread holds
    const int my_half = NH == 2 ? ww >> 1 : 0;
    float* ml = reinterpret_cast<float*>(smem + L::kMl) + wg * (4 * R * 2);
    constexpr float kPScale = I8 ? 32512.f : 256.f;   // 127 * 256: both digits stay inside int8
    const uint32_t my_s = tmem_s + wg * L::kSBuf + lane_base;
    const uint32_t my_o = tmem_o + wg * KN + lane_base + my_half * GP;
    const uint32_t my_swap = tmem + L::kTmemSwap + lane_base;
    uint8_t* p_tile = smem + L::kPT + wg * L::kPTile;
    int slot = wg;                            // tiles wg, wg + 2, ... of the CTA
    uint32_t phase = 0, t_ph = 0, m_ph = 0, x_ph = 0;
    bool ok = true;
    int part_no = -1;
    float X[R], l[R];         // X of this warp's tokens, l of this thread's
    float Y[GP], o[GP];       // O of this thread's dimension against the warpgroup's Y
#pragma unroll
    for (int h = 0; h < R; ++h) { X[h] = kFloor; l[h] = 0.f; }
#pragma unroll
    for (int h = 0; h < GP; ++h) { Y[h] = kFloor; o[h] = 0.f; }
    auto wait = [&](uint64_t* bar, uint32_t ph) -> bool {   // the same answer in the whole warp
      return __all_sync(0xffffffffu, q8_wait(bar, ph, abort_flag, p.status));
    };
    while (ok) {
      if (!wait(&full[slot], phase)) { ok = false; break; }
      const int flags = info[slot].flags;
      if (flags & 4) break;
      const TileInfo ti = info[slot];
      uint8_t* stage = smem + slot * L::kStageBytes;
      const int q_par = ti.len & 1;
      if (ti.len != part_no) {   // this warpgroup's first tile of the part
        part_no = ti.len;
        if (!wait(&q_ready[q_par], uint32_t(part_no >> 1) & 1u)) { ok = false; break; }
#pragma unroll
        for (int h = 0; h < R; ++h) { X[h] = kFloor; l[h] = 0.f; }
#pragma unroll
        for (int h = 0; h < GP; ++h) { Y[h] = kFloor; o[h] = 0.f; }
      }
      const bool valid = tok < ti.ntok && !((ti.bad >> (tok >> 4)) & 1);
      if (!valid) {   // a V row that was not copied: 0 * (stale bytes) must not reach O
        uint4* v_row = reinterpret_cast<uint4*>(stage + L::kTileBytes + tok * kQ8Row);
#pragma unroll
        for (int i = 0; i < kQ8Row / 16; ++i) v_row[i] = make_uint4(0, 0, 0, 0);
      }
      float ks[NH], lvs[NH];
#pragma unroll
      for (int n = 0; n < NH; ++n) {
        ks[n] = scales[slot * 16 * NH + n * 16 + (tok >> 4)];
        const float vs = scales[slot * 16 * NH + n * 16 + 8 + (tok >> 4)];
        lvs[n] = valid ? __log2f(vs) : 0.f;   // an absent token's scale was not copied
      }
      float xs[R];
      {
        const float* qs = reinterpret_cast<const float*>(smem + L::kQf) + q_par * R;
#pragma unroll
        for (int h = 0; h < R; ++h) xs[h] = (h % GP < p.G ? qs[h] : 0.f) * ks[h / GP];
      }

      // ---- scores of this token for all heads
      if (!wait(&s_full[wg], t_ph)) { ok = false; break; }
      tc_fence_after();
      {
        uint32_t s_hi[R], s_lo[R], s_frac[R];
#pragma unroll
        for (int n = 0; n < NH; ++n) {
          tmem_ld_cols<GP>(my_s + n * KN + n * GP, s_hi + n * GP);
          tmem_ld_cols<GP>(my_s + n * KN + n * GP + R, s_lo + n * GP);
          if constexpr (I8) tmem_ld_cols<GP>(my_s + n * KN + n * GP + 2 * R, s_frac + n * GP);
        }
        tmem_ld_wait();
        reg_fence<R>(s_hi);
        reg_fence<R>(s_lo);
        if constexpr (I8) reg_fence<R>(s_frac);
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&s_free[wg]);
#pragma unroll
        for (int h = 0; h < R; ++h) {
          xs[h] = valid ? join_digits<I8>(s_hi[h], s_lo[h], s_frac[h]) * xs[h] : neg_inf;
        }
      }
      // ---- maxima: of y over the warpgroup's 128 tokens, of x over this warp's
      float* ymax = reinterpret_cast<float*>(smem + L::kYmax) + (wg * 2 + t_ph) * 4 * R;   // [row][warp]
#pragma unroll
      for (int h = 0; h < R; ++h) {
        const float ty = warp_max_nan(xs[h] + lvs[h / GP]);
        if (lane == 0) ymax[4 * h + ww] = ty;
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&y_ready[wg]);
#pragma unroll
      for (int h = 0; h < R; ++h) {
        const float tx = max_nan(X[h], warp_max_nan(xs[h]));
        if (!(tx == X[h])) {   // it grew (or is a NaN); the same in the whole warp
          l[h] *= fast_exp2(X[h] - tx);
          X[h] = tx;
        }
        l[h] += fast_exp2(xs[h] - X[h]);
      }
      if (!wait(&y_ready[wg], t_ph)) { ok = false; break; }
      float y[R];   // the tile's reference
#pragma unroll
      for (int h = 0; h < R; ++h) {
        const float4 t = *reinterpret_cast<const float4*>(ymax + 4 * h);
        y[h] = max_nan(kFloor, max_nan(max_nan(t.x, t.y), max_nan(t.z, t.w)));
      }
      // ---- P digits: rows h (hi), R + h (lo) and, int8, 2 R + h (third), this token's byte
      {
        const int unit = 2 * ww + (lane >> 4), b = lane & 15;
#pragma unroll
        for (int h = 0; h < R; h += 2) {
          float pv[2] = {0.f, 0.f};
#pragma unroll
          for (int k = 0; k < 2 && h + k < R; ++k)
            pv[k] = fast_exp2(xs[h + k] + lvs[(h + k) / GP] - y[h + k]) * kPScale;
          uint32_t hi, lo, frac = 0;
          two_digits<I8>(pv[0], pv[1], hi, lo);
          if constexpr (I8) frac = third_digits(pv[0], pv[1]);
#pragma unroll
          for (int k = 0; k < 2 && h + k < R; ++k) {
            p_tile[row_unit(h + k, unit) + b] = uint8_t(hi >> (8 * k));
            p_tile[row_unit(R + h + k, unit) + b] = uint8_t(lo >> (8 * k));
            if constexpr (I8) p_tile[row_unit(2 * R + h + k, unit) + b] = uint8_t(frac >> (8 * k));
          }
        }
      }
      fence_proxy_async_smem();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&p_ready[wg]);

      // ---- O^T of the tile: thread = head dimension
      if (!wait(&o_full[wg], t_ph)) { ok = false; break; }
      tc_fence_after();
      {
        uint32_t hi[GP], lo[GP], frac[GP];
        tmem_ld_cols<GP>(my_o, hi);
        tmem_ld_cols<GP>(my_o + R, lo);
        if constexpr (I8) tmem_ld_cols<GP>(my_o + 2 * R, frac);
        tmem_ld_wait();
        reg_fence<GP>(hi);
        reg_fence<GP>(lo);
        if constexpr (I8) reg_fence<GP>(frac);
#pragma unroll
        for (int h = 0; h < GP; ++h) {
          const float v = join_digits<I8>(hi[h], lo[h], frac[h]);
          const float yt = NH == 2 && my_half ? y[(NH - 1) * GP + h] : y[h];
          const float d = yt - Y[h], a = fast_exp2(-fabsf(d));   // the lower reference's onto the higher one
          o[h] = d > 0.f ? fmaf(o[h], a, v) : fmaf(v, a, o[h]);
          Y[h] = max_nan(Y[h], yt);
        }
        tc_fence_before();
      }
      slot += 2;
      if (slot >= NS) { slot -= NS; phase ^= 1u; }
      t_ph ^= 1u;
      if (!(flags & 8)) continue;

      // ---- the part ends for this warpgroup: the sums of its four warps
#pragma unroll
      for (int h = 0; h < R; ++h) {
#pragma unroll
        for (int s = 16; s > 0; s >>= 1) l[h] += __shfl_xor_sync(0xffffffffu, l[h], s);
        if (lane == 0) *reinterpret_cast<float2*>(ml + (ww * R + h) * 2) = make_float2(X[h], l[h]);
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&ml_ready[wg]);
      if (!wait(&ml_ready[wg], m_ph)) { ok = false; break; }
      m_ph ^= 1u;
      const bool finish = (flags & 2) != 0, swap = (flags & 16) != 0;
      float* other = reinterpret_cast<float*>(smem + L::kSwap);
      if (swap && !wait(finish ? swap_full : swap_free, finish ? x_ph : x_ph ^ 1u)) { ok = false; break; }
      x_ph ^= swap ? 1u : 0u;
      uint32_t theirs[GP];
      if (!finish) {
        tc_fence_after();   // the other warpgroup's loads of the part before are done
#pragma unroll
        for (int h = 0; h < GP; ++h) theirs[h] = __float_as_uint(o[h]);
        tmem_st_cols<GP>(my_swap, theirs);
      } else if (swap) {
        tc_fence_after();
        tmem_ld_cols<GP>(my_swap, theirs);
        tmem_ld_wait();
        reg_fence<GP>(theirs);
        tc_fence_before();
      }
      const int row = ti.kvh, part = ti.split;
      const int head = (NH == 2 ? row * 2 : row) + my_half;   // KV head whose dims this thread may hold
      const int dim = D == 64 ? tok & 63 : tok;
      const bool mine = head < p.Hkv && (D == 128 || NH == 2 || (tok >> 6) == (row & 1));
      const size_t at0 = part < 0 ? size_t(ti.seq) * p.Hq + size_t(head) * p.G : size_t(part) * p.part_rows + my_half * p.G;
      const bool writer = (ww & (NH == 2 ? 1 : 3)) == 0 && lane == 0;   // one thread of each head half
#pragma unroll
      for (int h = 0; h < GP; ++h) {
        const int r = NH == 2 && my_half ? GP + h : h;   // the row's number
        const float yh = Y[h];
        float mx = kFloor, lsum = 0.f;
#pragma unroll
        for (int w = 0; w < 4; ++w) mx = max_nan(mx, ml[(w * R + r) * 2]);
        float* sw = other + r * 3;
        float ox = kFloor, oy = kFloor, ol = 0.f;
        if (swap && finish) {
          ox = sw[0]; oy = sw[1]; ol = sw[2];
          mx = max_nan(mx, ox);
        }
#pragma unroll
        for (int w = 0; w < 4; ++w) lsum = fmaf(ml[(w * R + r) * 2 + 1], fast_exp2(ml[(w * R + r) * 2] - mx), lsum);
        if (!finish) {
          if (writer) { sw[0] = mx; sw[1] = yh; sw[2] = lsum; }
          continue;
        }
        lsum = fmaf(ol, fast_exp2(ox - mx), lsum);
        const float my = max_nan(yh, oy);
        float v = o[h] * fast_exp2(yh - my);
        if (swap) v = fmaf(__uint_as_float(theirs[h]), fast_exp2(oy - my), v);
        // lsum is 0 only if every page was invalid; a NaN stays a NaN. The digits' factor and the sum go first and
        // the V scale's exponent in two halves, so that nothing on the way is beyond the result's own range
        const float up = fast_exp2(0.5f * (my - mx));
        v = lsum == 0.f ? 0.f : __fdividef(v * (1.f / kPScale), lsum) * up * up;
        const float lse2 = lsum == 0.f ? neg_inf : mx + __log2f(lsum);
        if (h >= p.G || !mine) continue;
        if (part < 0) {
          p.o[(at0 + h) * D + dim] = __float2bfloat16_rn(v);
          if (p.lse && dim == 0) p.lse[at0 + h] = lse2 * 0.69314718055994531f;
        } else {
          p.ws_o[(at0 + h) * D + dim] = v;
          if (dim == 0) p.ws_lse[at0 + h] = lse2;
        }
      }
      if (swap) {
        if (!finish) {
          tmem_st_wait();
          tc_fence_before();
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(finish ? swap_free : swap_full);
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == kQ8ScoreWarp) tmem_dealloc(tmem, L::kTmemCols);
}

// The cut sequences: CTA (i, r) merges query row r of the one whose first part decode CTA i holds, if
// it holds one; its other parts are the first ones of the same lane in the following teams. Bound by
// latency (its loads are a few KB a CTA, out of L2), so a CTA's four warps take sixteen parts each at a
// time, all sixteen in flight, a lane D / 32 neighbouring dimensions, and a sequence of at most sixteen
// parts ends in warp 0 without an exchange. When they were tried, one thread a dimension over all parts, eight in
// flight, made a call of one sequence of 32768 tokens 19.5 us long with 8 KV heads (37 parts; 18.5 so) and 17.1
// with one (148 parts; 13.8 so); a warp a row over all parts 21.9 with 8 KV heads. Merged instead by the
// decode CTA that finishes the last part, found with a counter in the workspace, a call saves this
// launch but took longer (39 us against 21 when it was tried, and 117 against 102 for 64 sequences): a
// fence and two dependent loads take microseconds while the other CTAs stream.
template <int D>
__global__ void __launch_bounds__(128) decode_q8_merge_kernel(const DecodeQ8Params p) {
  constexpr int E = D / 32;
  __shared__ float sh_m[4], sh_sum[4];
  __shared__ __align__(16) float sh_acc[4][D];
  const float neg_inf = -__int_as_float(0x7f800000);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  grid_dependency_wait();
  const int4 cut = p.ws_cut[blockIdx.x];
  if (cut.x < 0) return;
  const int first = int(blockIdx.x) / p.team, team_lane = int(blockIdx.x) % p.team;
  const int row = cut.y * p.team + team_lane, r = int(blockIdx.y);
  const int nh = p.part_rows > p.G && r >= p.G ? 1 : 0;
  const int head = (p.part_rows > p.G ? row * 2 : row) + nh;
  if (r >= p.part_rows || head >= p.Hkv) return;
  const int n = cut.z - first + 1;                         // parts: at most one per team
  auto part_row = [&](int i) {
    return size_t(((first + i) * p.team + team_lane) * 2 + (i == 0 ? cut.w : 0)) * p.part_rows + r;
  };
  // weights are at most 1 / kQ8MaxCtas: a sum of parts is no larger than the largest of them
  constexpr float kLog2Parts = 9.f, kWeight = 1.f / 512.f;
  static_assert(kQ8MaxCtas <= 512, "parts of a sequence");
  float m = neg_inf, sum = 0.f, acc[E];
#pragma unroll
  for (int e = 0; e < E; ++e) acc[e] = 0.f;
  for (int i0 = warp * 16; i0 < n; i0 += 64) {   // lanes 0..15: the weights of parts i0 + lane
    const int k1 = min(16, n - i0);
    const float lse = lane < k1 ? p.ws_lse[part_row(i0 + lane)] : neg_inf;
    const float mx = max_nan(m, warp_max_nan(lse)), off = mx == neg_inf ? 0.f : mx;
    const float old = fast_exp2(m - off), w = fast_exp2(lse - off) * kWeight;
    m = mx;
    sum = fmaf(sum, old, w);                     // this lane's part of the sum
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] *= old;
    float v[16][E];
#pragma unroll
    for (int k = 0; k < 16; ++k) {
      const float* src = p.ws_o + part_row(min(i0 + k, n - 1)) * D + lane * E;
      if constexpr (E == 4) {
        const float4 t = *reinterpret_cast<const float4*>(src);
        v[k][0] = t.x; v[k][1] = t.y; v[k][2] = t.z; v[k][3] = t.w;
      } else {
        const float2 t = *reinterpret_cast<const float2*>(src);
        v[k][0] = t.x; v[k][1] = t.y;
      }
    }
#pragma unroll
    for (int k = 0; k < 16; ++k) {
      const float wk = __shfl_sync(0xffffffffu, w, k);
#pragma unroll
      for (int e = 0; e < E; ++e) acc[e] = fmaf(k < k1 ? wk : 0.f, v[k][e], acc[e]);
    }
  }
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
  if (n > 16) {                                  // else warp 0 holds it all
    if (lane == 0) { sh_m[warp] = m; sh_sum[warp] = sum; }
#pragma unroll
    for (int e = 0; e < E; ++e) sh_acc[warp][lane * E + e] = acc[e];
    __syncthreads();
    if (warp != 0) return;
#pragma unroll
    for (int w = 0; w < 4; ++w) m = w == 0 ? sh_m[0] : max_nan(m, sh_m[w]);
    const float off = m == neg_inf ? 0.f : m;
    sum = 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] = 0.f;
#pragma unroll
    for (int w = 0; w < 4; ++w) {                  // the four warps' shares onto one maximum
      const float f = fast_exp2(sh_m[w] - off);
      sum = fmaf(f, sh_sum[w], sum);
#pragma unroll
      for (int e = 0; e < E; ++e) acc[e] = fmaf(f, sh_acc[w][lane * E + e], acc[e]);
    }
  } else if (warp != 0) {
    return;
  }
  const size_t at = size_t(cut.x) * p.Hq + size_t(head) * p.G + (r - nh * p.G);
  const float inv = sum == 0.f ? 0.f : 1.f / sum;
  uint32_t out[E / 2];
#pragma unroll
  for (int e = 0; e < E / 2; ++e) out[e] = pack_bf16x2(acc[2 * e] * inv, acc[2 * e + 1] * inv);
  if constexpr (E == 4) *reinterpret_cast<uint2*>(p.o + at * D + lane * E) = make_uint2(out[0], out[1]);
  else *reinterpret_cast<uint32_t*>(p.o + at * D + lane * E) = out[0];
  if (p.lse && lane == 0) p.lse[at] = sum == 0.f ? neg_inf : (m + (__log2f(sum) + kLog2Parts)) * 0.69314718055994531f;
}

}  // namespace attn
