// Paged decode over an 8-bit cache with one scale per (block of tokens, KV head).
//
// K = ks * kc and V = vs * vc, where kc and vc are E4M3 or int8 codes and ks, vs
// the scales of the token's block. For a query head q and tokens t:
//   x_t = log2(e) * scale * ks_t * sum_d q_d kc_td       (the score in log2 units)
//   O   = sum_t 2^(x_t - X) vs_t vc_t / sum_t 2^(x_t - X),   LSE = ln2 * (X + log2 sum)
// The codes are never widened: they go from shared memory straight into
// tcgen05.mma as the A operand, 128 tokens at a time, and the narrow side is
// split into two 8-bit digits so that nothing of it is lost:
//   S^T = Kc (128 tokens x D) * [q_hi; q_lo]^T,  q * 2^a = q_hi + q_lo / 16 (E4M3)
//                                                        = 256 q_hi + q_lo  (int8)
//   O^T_w = Vc^T (D x 32 tokens) * [p_hi; p_lo]^T        for each warp w's 32 tokens
// E4M3: a bf16 value has 8 significant bits, a code 4, so two codes hold q exactly
// down to 2^-14 of the row's largest value; the products accumulate in fp32.
// int8: q becomes a 16-bit integer (exact down to 2^-8 of the row's largest value)
// and every product and sum is an exact int32.
// The probability that multiplies V is p_t = 2^(y_t - Y), y_t = x_t + log2(vs_t):
// the value scale is part of the exponent, so p <= 1 whatever the scales are. Two
// E4M3 digits keep 8 significant bits of 256 p, two int8 digits keep p to 2^-16.
//
// A CTA has four softmax warps (one token per thread of a 128-token tile), a
// producer warp (TMA copies of 16 slots, scales by cp.async) and an MMA warp.
// Each softmax warp keeps its own running maxima X, Y for its 32 tokens of every
// tile, and its own accumulator columns, so the warps exchange no maximum: the
// P V product of a tile is four MMAs of K = 32, one per warp. O stays in fp32
// registers (thread = head dimension) and is rescaled there by each warp's
// factor, which is why TMEM holds only the tile's own products. The four
// accumulators are merged when the item (sequence, split, KV head) ends.
#pragma once

#include "decode.cuh"

namespace attn {

constexpr int kQ8Tok = 128;          // tokens per tile
constexpr int kQ8Chunk = 16;         // tokens per TMA copy (a block-table page is a multiple of it)
constexpr int kQ8SoftmaxWarps = 4;
constexpr int kQ8Threads = (kQ8SoftmaxWarps + 2) * 32;

struct DecodeQ8Params {
  DecodeParams d;         // shared with the merge; scale_log2 does not contain the K scale
  const float* k_scales;  // [num_pages][page_size / block][Hkv]
  const float* v_scales;
  int G;                  // query heads per KV head (<= GP)
  int page_shift;         // log2(page_size)
  int block_shift;        // log2(tokens per scale)
};

template <int D, int GP, bool I8>
struct DecodeQ8Smem {
  static constexpr int kN = GP <= 8 ? 16 : 32;             // columns of S^T and of each O^T_w: hi digits, lo digits
  static constexpr int kTileBytes = kQ8Tok * D;            // K (or V) codes of one tile
  static constexpr int kQBytes = GP * D * 2;               // the item's query rows
  static constexpr int kStageBytes = (2 * kTileBytes + kQBytes + 1023) / 1024 * 1024;
  static constexpr int kBlocks = GP <= 8 ? 2 : 1;          // resident CTAs per SM
  static constexpr int kQTile = kN * D;                    // digit rows of q
  static constexpr int kPTile = kN * kQ8Tok;               // digit rows of P
  static constexpr int kSmall = 64 + 32 + 4 * (2 * 4 * GP + 3 * 4 * GP + GP) + 16 * 8;   // per stage extras below
  static constexpr int kFit =
      (233472 / kBlocks - 1024 - 1024 - kQTile - kPTile - kSmall - 256) / (kStageBytes + 64 + 32 + 16);
  static constexpr int kStages = kFit < 8 ? kFit : 8;
  static constexpr int kQT = kStages * kStageBytes;                    // q digits (1024-byte aligned)
  static constexpr int kPT = kQT + (kQTile + 1023) / 1024 * 1024;      // P digits
  static constexpr int kScales = kPT + kPTile;                         // [stage][K 8 | V 8] floats
  static constexpr int kInfo = kScales + 64 * kStages;                 // TileInfo per stage
  static constexpr int kAlpha = kInfo + 32 * kStages;                  // [2][warp][GP] floats
  static constexpr int kMl = kAlpha + 4 * 2 * 4 * GP;                  // [warp][GP] x {X, Y, l} floats
  static constexpr int kQf = kMl + 4 * 3 * 4 * GP;                     // [GP] floats
  static constexpr int kBars = (kQf + 4 * GP + 7) / 8 * 8;             // mbarriers
  // full[kStages], empty[kStages], s_full[2], p_ready, o_full, q_ready, ml_ready, done
  static constexpr int kTotal = kBars + 8 * (2 * kStages + 7);
  static constexpr int kDynamic = kTotal + 1024;
  static constexpr int kTmemUse = 2 * kN + 4 * kN;
  static constexpr int kTmemCols = kTmemUse <= 128 ? 128 : 256;
  static_assert(kDynamic <= 233472 / kBlocks - 1024, "shared memory per block");
  static_assert(kStages >= 2, "ring depth");
  static_assert(kTmemUse <= kTmemCols && kTmemCols * kBlocks <= 512, "tensor memory");
};

__device__ __forceinline__ bool mbar_test_wait(uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.test_wait.parity.acquire.cta.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(smem_u32(bar)), "r"(parity)
      : "memory");
  return ok != 0;
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
// Shared-memory descriptor of a tile of 128-byte or 64-byte rows under the swizzle of that width;
// eight-row atoms follow one another, so the stride between them is eight rows.
template <int ROW>
__device__ __forceinline__ uint64_t make_sdesc_rows(uint32_t smem_addr) {
  static_assert(ROW == 128 || ROW == 64, "swizzled rows");
  uint64_t d = 0;
  d |= uint64_t((smem_addr >> 4) & 0x3FFFu);
  d |= uint64_t(1) << 16;                          // leading offset: not used, one atom covers it
  d |= uint64_t((8 * ROW) >> 4) << 32;
  d |= uint64_t(1) << 46;                          // descriptor version for sm_100
  d |= uint64_t(ROW == 128 ? 2 : 4) << 61;         // 128-byte or 64-byte swizzle
  return d;
}
// Byte offset of 16-byte unit c of row r in such a tile.
template <int ROW>
__device__ __forceinline__ uint32_t row_unit(int r, int c) {
  return ROW == 128 ? uint32_t(r * 128 + ((c ^ (r & 7)) << 4)) : uint32_t(r * 64 + ((c ^ ((r >> 1) & 3)) << 4));
}

// NC columns of 32-bit TMEM of this warp's 32 lanes -> registers; no wait (tmem_ld_wait, then reg_fence).
template <int NC>
__device__ __forceinline__ void tmem_ld_cols(uint32_t taddr, uint32_t* r) {
  static_assert(NC == 2 || NC == 4 || NC == 8 || NC == 16 || NC == 32, "columns");
  if constexpr (NC == 2) {
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
__device__ __forceinline__ void reg_fence(uint32_t* r) {
#pragma unroll
  for (int i = 0; i < NC; ++i) asm volatile("" : "+r"(r[i]));
}

// Warp maximum that keeps a NaN, and the maximum of two values that keeps a NaN.
__device__ __forceinline__ float warp_max_nan(float x) {
  float y;
  asm volatile("redux.sync.max.NaN.f32 %0, %1, 0xffffffff;" : "=f"(y) : "f"(x));
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
// Two values as two digits each: E4M3 v = hi + lo / 16, int8 (v an integer) v = 256 hi + lo.
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
// The value of two accumulated digit columns.
template <bool I8>
__device__ __forceinline__ float join_digits(uint32_t hi, uint32_t lo) {
  if constexpr (I8) return float(int(hi) * 256 + int(lo));   // |.| < 2^30: 128 products of at most 2^15 * 2^7
  else return fmaf(__uint_as_float(lo), 0.0625f, __uint_as_float(hi));
}

template <int D, int GP, bool I8>
__global__ void __launch_bounds__(kQ8Threads, DecodeQ8Smem<D, GP, I8>::kBlocks)
    decode_q8_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                     const DecodeQ8Params qp, int* ticket_counter) {
  using L = DecodeQ8Smem<D, GP, I8>;
  launch_dependents();   // the merge is scheduled early; it waits for this grid to finish
  constexpr int NS = L::kStages;
  constexpr int KN = L::kN;
  const DecodeParams& p = qp.d;

  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  float* scales = reinterpret_cast<float*>(smem + L::kScales);
  TileInfo* info = reinterpret_cast<TileInfo*>(smem + L::kInfo);
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + L::kBars);
  uint64_t* empty = full + NS;
  uint64_t* s_full = empty + NS;     // [2]
  uint64_t* p_ready = s_full + 2;
  uint64_t* o_full = p_ready + 1;
  uint64_t* q_ready = o_full + 1;
  uint64_t* ml_ready = q_ready + 1;
  uint64_t* done = ml_ready + 1;
  __shared__ int abort_word;
  __shared__ uint32_t tmem_slot;
  volatile int* abort_flag = &abort_word;

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int capacity = p.max_pages * p.page_size;
  const long long num_items = (long long)p.max_splits * p.num_seqs * p.Hkv;

  if (threadIdx.x == 0) {
    abort_word = 0;
    for (int s = 0; s < NS; ++s) {
      mbar_init(&full[s], 33);    // the producer's expect_tx arrival and its 32 lanes' scale copies
      mbar_init(&empty[s], 1);
    }
    mbar_init(&s_full[0], 1);
    mbar_init(&s_full[1], 1);
    mbar_init(p_ready, kQ8SoftmaxWarps);
    mbar_init(o_full, 1);
    mbar_init(q_ready, kQ8SoftmaxWarps);
    mbar_init(ml_ready, kQ8SoftmaxWarps);
    mbar_init(done, 1);
    fence_mbar_init();
  }
  // digit rows that no query head uses stay zero
  for (int i = threadIdx.x * 16; i < L::kQTile; i += kQ8Threads * 16)
    *reinterpret_cast<uint4*>(smem + L::kQT + i) = make_uint4(0, 0, 0, 0);
  for (int i = threadIdx.x * 16; i < L::kPTile; i += kQ8Threads * 16)
    *reinterpret_cast<uint4*>(smem + L::kPT + i) = make_uint4(0, 0, 0, 0);
  fence_proxy_async_smem();
  if (warp == kQ8SoftmaxWarps + 1) {
    tmem_alloc(&tmem_slot, L::kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_slot;
  const uint32_t tmem_s = tmem;                 // two buffers of KN columns
  const uint32_t tmem_o = tmem + 2 * KN;        // four groups of KN columns, one per softmax warp

  if (warp == kQ8SoftmaxWarps) {
    // ------------------------------------------------------------ producer warp
    if (lane == 0) {
      tma_prefetch_desc(&tm_k);
      tma_prefetch_desc(&tm_v);
    }
    const int c = lane & 7;            // lanes 0 .. 7 copy K chunk c, lanes 8 .. 15 V chunk c
    const bool is_v = lane >= 8;
    const CUtensorMap* map = is_v ? &tm_v : &tm_k;
    const float* sc_src = is_v ? qp.v_scales : qp.k_scales;
    const int blocks_per_page = p.page_size >> qp.block_shift;
    int slot = 0;
    uint32_t phase = 0;
    uint32_t pending = 0, pending_phase = 0;
    bool ok = true;
    long long nx_item = 0;
    int nx_len = 0, nx_page = -1;
    bool first_fetch = true;
    auto page_of = [&](int seq, int t0) -> int {   // physical page of chunk c of the tile at t0
      const int e = (t0 + c * kQ8Chunk) >> qp.page_shift;
      return e < p.max_pages ? __ldg(&p.block_table[size_t(seq) * p.max_pages + e]) : -1;
    };
    auto fetch_next = [&]() {   // next item, its length and its first tile's pages, one item ahead
      long long t = 0;
      if (p.static_items) {
        t = first_fetch ? (long long)blockIdx.x : num_items;
      } else {
        if (lane == 0) t = atomicAdd(ticket_counter, 1);
        t = __shfl_sync(0xffffffffu, t, 0);
      }
      first_fetch = false;
      nx_item = t;
      if (t < num_items) {
        const long long per = (long long)p.num_seqs * p.Hkv;
        const int sp = int(t / per), sq = int(t % per) / p.Hkv;
        nx_len = __ldg(&p.seq_lens[sq]);
        nx_page = page_of(sq, sp * p.split_tokens);
      }
    };
    fetch_next();
    while (ok) {
      const long long item = nx_item;
      if (item >= num_items) break;
      int len = nx_len;
      int page = nx_page;
      fetch_next();
      const long long per = (long long)p.num_seqs * p.Hkv;   // splits outermost: full-length splits go first
      const int split = int(item / per), rem = int(item % per);
      const int seq = rem / p.Hkv, kvh = rem % p.Hkv;
      if (len > capacity || len < 0) {
        if (lane == 0 && split == 0 && kvh == 0) raise_status(p.status, ATTN_ERR_DEVICE_BOUNDS);
        len = len < 0 ? 0 : capacity;
      }
      const int t_begin = split * p.split_tokens;
      if (t_begin >= len) continue;
      const int t_end = min(t_begin + p.split_tokens, len);
      for (int t0 = t_begin; t0 < t_end && ok; t0 += kQ8Tok) {
        const int page_next = t0 + kQ8Tok < t_end ? page_of(seq, t0 + kQ8Tok) : -1;
        if (!__all_sync(0xffffffffu, mbar_wait(&empty[slot], phase ^ 1u, abort_flag, p.status))) { ok = false; break; }
        const int ntok = min(kQ8Tok, t_end - t0);
        const bool in_range = page >= 0 && page < p.num_pages;
        const bool good = lane < 16 && c * kQ8Chunk < ntok && in_range;
        const uint32_t good_mask = __ballot_sync(0xffffffffu, good) & 0xFFu;
        const bool outside = __any_sync(0xffffffffu, lane < 8 && c * kQ8Chunk < ntok && !in_range);
        uint8_t* stage = smem + slot * L::kStageBytes;
        if (lane == 0) {
          if (outside) raise_status(p.status, ATTN_ERR_DEVICE_BOUNDS);
          const bool first = t0 == t_begin;
          TileInfo ti;
          ti.seq = seq; ti.split = split; ti.kvh = kvh; ti.t0 = t0;
          ti.ntok = ntok;
          ti.bad = int(~good_mask & 0xFFu);
          ti.flags = (first ? 1 : 0) | (t0 + kQ8Tok >= t_end ? 2 : 0);
          ti.len = len;
          info[slot] = ti;
          const uint32_t qbytes = first ? uint32_t(qp.G * D * 2) : 0u;
          mbar_arrive_expect_tx(&full[slot], uint32_t(__popc(good_mask)) * uint32_t(2 * kQ8Chunk * D) + qbytes);
          if (first)
            bulk_load(stage + 2 * L::kTileBytes, p.q + (size_t(seq) * p.Hq + size_t(kvh) * qp.G) * D, qbytes,
                      &full[slot]);
        }
        __syncwarp();
        if (good) {
          const int in_page = (t0 + c * kQ8Chunk) & (p.page_size - 1);
          tma_load_4d(stage + (is_v ? L::kTileBytes : 0) + c * (kQ8Chunk * D), map, &full[slot], 0, in_page, kvh, page);
          cp_async4(scales + slot * 16 + lane,
                    sc_src + (size_t(page) * blocks_per_page + (in_page >> qp.block_shift)) * p.Hkv + kvh);
        }
        cp_async_arrive_noinc(&full[slot]);
        __syncwarp();
        pending |= 1u << slot;
        pending_phase = (pending_phase & ~(1u << slot)) | (phase << slot);
        if (++slot == NS) { slot = 0; phase ^= 1u; }
        page = page_next;
      }
    }
    if (ok && __all_sync(0xffffffffu, mbar_wait(&empty[slot], phase ^ 1u, abort_flag, p.status))) {
      if (lane == 0) {   // end-of-work marker: a stage with no copies
        TileInfo ti{};
        ti.flags = 4;
        info[slot] = ti;
        mbar_arrive_expect_tx(&full[slot], 0u);
      }
      __syncwarp();
      cp_async_arrive_noinc(&full[slot]);
    } else {
      ok = false;
    }
    cp_async_wait_all();
    if (!ok && lane == 0) {
      for (int s = 0; s < NS; ++s)
        if (pending & (1u << s)) mbar_drain(&full[s], (pending_phase >> s) & 1u);
    }
  } else if (warp == kQ8SoftmaxWarps + 1) {
    // ------------------------------------------------------------ MMA warp (one thread)
    if (lane == 0) {
      constexpr uint32_t idesc_s = make_idesc_q8<I8>(kQ8Tok, KN, 0);   // K tile: rows = tokens, K-major
      constexpr uint32_t idesc_o = make_idesc_q8<I8>(D, KN, 1);        // V tile: rows = head dims, MN-major
      const uint64_t q_desc = make_sdesc_rows<D>(smem_u32(smem + L::kQT));
      const uint64_t p_desc = make_sdesc_rows<128>(smem_u32(smem + L::kPT));
      int slot = 0, sb = 0;
      uint32_t phase = 0, p_ph = 0, q_ph = 0;
      auto issue_s = [&](int s, int b) {   // S^T of stage s into buffer b
        const uint64_t k_desc = make_sdesc_rows<D>(smem_u32(smem + s * L::kStageBytes));
#pragma unroll
        for (int k = 0; k < D / 32; ++k)
          umma_q8<I8>(tmem_s + b * KN, k_desc + 2 * k, q_desc + 2 * k, idesc_s, k > 0);
        umma_commit(&s_full[b]);
      };
      bool ok = mbar_wait(&full[0], 0, abort_flag, p.status);
      bool live = ok && !(info[0].flags & 4);
      if (live) {
        ok = mbar_wait(q_ready, q_ph, abort_flag, p.status);
        q_ph ^= 1u;
        tc_fence_after();
        if (ok) issue_s(0, 0);
      }
      while (ok && live) {
        const int ns = slot + 1 == NS ? 0 : slot + 1;
        const uint32_t nph = ns == 0 ? phase ^ 1u : phase;
        bool issued = false, seen = false;
        int nflags = 0;
        // the next tile's scores while this tile's softmax runs, unless it needs a new query
        const unsigned long long t_start = global_timer_ns();
        for (uint32_t i = 1; !mbar_test_wait(p_ready, p_ph); ++i) {
          if (!seen && mbar_test_wait(&full[ns], nph)) {
            seen = true;
            nflags = info[ns].flags;
            if (!(nflags & 5)) {
              tc_fence_after();
              issue_s(ns, sb ^ 1);
              issued = true;
            }
          }
          if ((i & 63u) == 0) {
            if (*abort_flag) { ok = false; break; }
            if (global_timer_ns() - t_start > kWaitLimitNs) {
              *abort_flag = 1;
              raise_status(p.status, ATTN_ERR_TIMEOUT);
              ok = false;
              break;
            }
          }
        }
        if (!ok) break;
        p_ph ^= 1u;
        tc_fence_after();
        // O^T_w of this tile: tokens 32w .. 32w + 31
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          const uint64_t v_desc =
              make_sdesc_rows<D>(smem_u32(smem + slot * L::kStageBytes + L::kTileBytes + w * 32 * D));
          umma_q8<I8>(tmem_o + w * KN, v_desc, p_desc + 2 * w, idesc_o, 0);
        }
        umma_commit(o_full);
        umma_commit(&empty[slot]);
        if (!seen) {
          if (!mbar_wait(&full[ns], nph, abort_flag, p.status)) { ok = false; break; }
          nflags = info[ns].flags;
        }
        if (nflags & 4) break;
        if (!issued) {
          if (nflags & 1) {
            if (!mbar_wait(q_ready, q_ph, abort_flag, p.status)) { ok = false; break; }
            q_ph ^= 1u;
          }
          tc_fence_after();
          issue_s(ns, sb ^ 1);
        }
        slot = ns;
        phase = nph;
        sb ^= 1;
      }
      umma_commit(done);       // nothing of this thread is in flight when TMEM is given back
      mbar_drain(done, 0);
    }
    __syncwarp();
  } else {
    // ------------------------------------------------------------ softmax warps: thread = token, then head dim
    const float neg_inf = -__int_as_float(0x7f800000);
    const uint32_t lane_base = uint32_t(warp * 32) << 16;
    const int tok = warp * 32 + lane;
    const int dim = D == 128 ? tok : warp * 16 + lane;   // M = 64: rows 16w .. 16w + 15 sit in lanes 32w ..
    const bool dim_valid = D == 128 || lane < 16;
    float* alpha = reinterpret_cast<float*>(smem + L::kAlpha);
    float* ml = reinterpret_cast<float*>(smem + L::kMl);
    float* qf_s = reinterpret_cast<float*>(smem + L::kQf);
    uint8_t* p_tile = smem + L::kPT;
    constexpr float kPScale = I8 ? 32512.f : 256.f;   // 127 * 256: both digits stay inside int8
    int slot = 0, sb = 0;
    uint32_t phase = 0, s_ph = 0, p_ph = 0, o_ph = 0, q_ph = 0, m_ph = 0;
    bool ok = true;
    int seq = 0, split = 0, kvh = 0, n_splits = 0;
    float qf[GP], X[GP], Y[GP], l[GP];
    float o[4][GP];
#pragma unroll
    for (int h = 0; h < GP; ++h) {
      qf[h] = 0.f; X[h] = Y[h] = neg_inf; l[h] = 0.f;
      o[0][h] = o[1][h] = o[2][h] = o[3][h] = 0.f;
    }
    auto wait = [&](uint64_t* bar, uint32_t ph) -> bool {   // the same answer in the whole warp
      return __all_sync(0xffffffffu, mbar_wait(bar, ph, abort_flag, p.status));
    };

    while (ok) {
      if (!wait(&full[slot], phase)) { ok = false; break; }
      const TileInfo ti = info[slot];
      if (ti.flags & 4) break;
      uint8_t* stage = smem + slot * L::kStageBytes;
      if (ti.flags & 1) {
        // ---- the item's query rows as digits, scaled by a power of two (exact)
        seq = ti.seq; split = ti.split; kvh = ti.kvh;
        n_splits = (ti.len + p.split_tokens - 1) / p.split_tokens;
        for (int r = warp; r < qp.G; r += kQ8SoftmaxWarps) {
          constexpr int E = D / 32;   // values per lane
          const uint32_t* src = reinterpret_cast<const uint32_t*>(stage + 2 * L::kTileBytes + r * D * 2) + lane * (E / 2);
          uint32_t w[E / 2];
          uint32_t top = 0;
#pragma unroll
          for (int i = 0; i < E / 2; ++i) {
            w[i] = src[i];
            top = max(top, max((w[i] << 16) & 0x7FFF0000u, w[i] & 0x7FFF0000u));
          }
          top = __reduce_max_sync(0xffffffffu, top);
          const int e = int(top >> 23) - 127, mant = int(top >> 16) & 0x7F;
          const bool finite = top < 0x7F800000u;
          // the largest value lands in (224, 448] or [16320, 32639]
          int a = I8 ? 14 - e - (mant == 0x7F ? 1 : 0) : 8 - e - (mant > 0x60 ? 1 : 0);
          a = min(a, 118);
          const float up = finite ? __uint_as_float(uint32_t(a + 127) << 23) : 0.f;
          if (lane == 0)
            qf_s[r] = finite ? p.scale_log2 * __uint_as_float(uint32_t(127 - a) << 23) : __int_as_float(0x7fc00000);
#pragma unroll
          for (int i = 0; i < E / 2; ++i) {
            uint32_t hi = 0, lo = 0;
            if (finite) two_digits<I8>(bf16_lo(w[i]) * up, bf16_hi(w[i]) * up, hi, lo);
            const int byte = lane * E + 2 * i;
            uint8_t* q_tile = smem + L::kQT;
            *reinterpret_cast<uint16_t*>(q_tile + row_unit<D>(r, byte >> 4) + (byte & 15)) = uint16_t(hi);
            *reinterpret_cast<uint16_t*>(q_tile + row_unit<D>(GP + r, byte >> 4) + (byte & 15)) = uint16_t(lo);
          }
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(q_ready);
        if (!wait(q_ready, q_ph)) { ok = false; break; }
        q_ph ^= 1u;
#pragma unroll
        for (int h = 0; h < GP; ++h) {
          qf[h] = h < qp.G ? qf_s[h] : 0.f;
          X[h] = Y[h] = neg_inf;
          l[h] = 0.f;
          o[0][h] = o[1][h] = o[2][h] = o[3][h] = 0.f;
        }
      }
      const bool last = (ti.flags & 2) != 0;
      const bool valid = tok < ti.ntok && !((ti.bad >> (tok >> 4)) & 1);
      if (!valid) {   // a V row that was not copied: 0 * (stale bytes) must not reach O
        uint4* row = reinterpret_cast<uint4*>(stage + L::kTileBytes + tok * D);
#pragma unroll
        for (int i = 0; i < D / 16; ++i) row[i] = make_uint4(0, 0, 0, 0);
      }
      const float ks = scales[slot * 16 + (tok >> 4)];
      const float lvs = __log2f(scales[slot * 16 + 8 + (tok >> 4)]);

      // ---- scores of this token for all heads
      if (!wait(&s_full[sb], s_ph)) { ok = false; break; }
      tc_fence_after();
      uint32_t sr[2 * GP];
      tmem_ld_cols<2 * GP>(tmem_s + sb * KN + lane_base, sr);
      tmem_ld_wait();
      reg_fence<2 * GP>(sr);
      float pv[GP];
#pragma unroll
      for (int h = 0; h < GP; ++h) {
        const float x = valid ? join_digits<I8>(sr[h], sr[GP + h]) * (qf[h] * ks) : neg_inf;
        const float y = valid ? x + lvs : neg_inf;
        const float nx = max_nan(X[h], warp_max_nan(x)), ny = max_nan(Y[h], warp_max_nan(y));
        const float offx = nx == neg_inf ? 0.f : nx, offy = ny == neg_inf ? 0.f : ny;
        l[h] = fmaf(l[h], fast_exp2(X[h] - offx), fast_exp2(x - offx));
        pv[h] = fast_exp2(y - offy) * kPScale;
        if (lane == 0) alpha[(sb * 4 + warp) * GP + h] = fast_exp2(Y[h] - offy);
        X[h] = nx;
        Y[h] = ny;
      }
      // ---- P digits: row h (hi) and GP + h (lo), this token's byte
      {
        const int unit = 2 * warp + (lane >> 4), b = lane & 15;
#pragma unroll
        for (int h = 0; h < GP; h += 2) {
          uint32_t hi, lo;
          two_digits<I8>(pv[h], h + 1 < GP ? pv[h + 1 < GP ? h + 1 : h] : 0.f, hi, lo);
          p_tile[row_unit<128>(h, unit) + b] = uint8_t(hi);
          p_tile[row_unit<128>(GP + h, unit) + b] = uint8_t(lo);
          if (h + 1 < GP) {
            p_tile[row_unit<128>(h + 1, unit) + b] = uint8_t(hi >> 8);
            p_tile[row_unit<128>(GP + h + 1, unit) + b] = uint8_t(lo >> 8);
          }
        }
      }
      fence_proxy_async_smem();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(p_ready);

      // ---- O of this tile: thread = head dimension, one accumulator per warp's tokens
      if (!wait(p_ready, p_ph)) { ok = false; break; }   // every warp's factors are in
      p_ph ^= 1u;
      if (!wait(o_full, o_ph)) { ok = false; break; }
      o_ph ^= 1u;
      tc_fence_after();
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        uint32_t r[2 * GP];
        tmem_ld_cols<2 * GP>(tmem_o + w * KN + lane_base, r);
        tmem_ld_wait();
        reg_fence<2 * GP>(r);
#pragma unroll
        for (int h = 0; h < GP; ++h)
          o[w][h] = fmaf(o[w][h], alpha[(sb * 4 + w) * GP + h], join_digits<I8>(r[h], r[GP + h]));
      }
      tc_fence_before();
      if (++slot == NS) { slot = 0; phase ^= 1u; }
      if (sb) s_ph ^= 1u;
      sb ^= 1;
      if (!last) continue;

      // ---- the item's result: the four warps' accumulators onto common maxima
#pragma unroll
      for (int h = 0; h < GP; ++h) {
#pragma unroll
        for (int s = 16; s > 0; s >>= 1) l[h] += __shfl_xor_sync(0xffffffffu, l[h], s);
        if (lane == 0) {
          float* m = ml + (warp * GP + h) * 3;
          m[0] = X[h]; m[1] = Y[h]; m[2] = l[h];
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(ml_ready);
      if (!wait(ml_ready, m_ph)) { ok = false; break; }
      m_ph ^= 1u;
#pragma unroll
      for (int h = 0; h < GP; ++h) {
        if (h >= qp.G) continue;
        float mx = neg_inf, my = neg_inf;
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          mx = max_nan(mx, ml[(w * GP + h) * 3]);
          my = max_nan(my, ml[(w * GP + h) * 3 + 1]);
        }
        const float offx = mx == neg_inf ? 0.f : mx, offy = my == neg_inf ? 0.f : my;
        float lsum = 0.f, acc = 0.f;
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          lsum = fmaf(ml[(w * GP + h) * 3 + 2], fast_exp2(ml[(w * GP + h) * 3] - offx), lsum);
          acc = fmaf(o[w][h], fast_exp2(ml[(w * GP + h) * 3 + 1] - offy), acc);
        }
        // lsum is 0 only if every page was invalid; a NaN stays a NaN
        const float out = lsum == 0.f ? 0.f : acc * fast_exp2(offy - offx) * (1.f / kPScale) / lsum;
        const float lse2 = lsum == 0.f ? neg_inf : mx + __log2f(lsum);
        const int hq = kvh * qp.G + h;
        if (n_splits == 1) {
          if (dim_valid) p.o[(size_t(seq) * p.Hq + hq) * D + dim] = __float2bfloat16_rn(out);
          if (p.lse && threadIdx.x == 0) p.lse[size_t(seq) * p.Hq + hq] = lse2 * 0.69314718055994531f;
        } else {
          const uint64_t keep = l2_keep_policy();   // the merge reads these back after the KV stream
          const size_t row = (size_t(seq) * p.max_splits + split) * p.Hq + hq;
          if (dim_valid) st_keep(p.ws_o + row * D + dim, out, keep);
          if (threadIdx.x == 0) st_keep(p.ws_lse + row, lse2, keep);
        }
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == kQ8SoftmaxWarps + 1) tmem_dealloc(tmem, L::kTmemCols);
}

}  // namespace attn
