// The 8-bit paged cache: writing new tokens as codes, and reading tokens back.
//
// A cached value is s * code: code an E4M3 number or an int8 integer, s one fp32
// scale for each block of tokens (16 .. page_size slots of a page) and KV head.
// The scales written here are powers of two, the smallest s >= 2^-100 with
// max|x| <= Q s (Q = 448 or 127). So x / s is exact, each code is rounded once
// (to nearest, ties to even), and s * code is a bf16 number: reading back rounds
// nothing, and the attention kernels that widen the cache and the one that does
// not see the same values. An E4M3 code keeps the same four significant bits at
// any scale; an int8 code gives up at most one bit against s = max|x| / 127.
#pragma once

#include "common.cuh"

namespace attn {

struct KvAppendQ8Params {
  const __nv_bfloat16* k_new;   // [N][T][Hkv][D]
  const __nv_bfloat16* v_new;
  uint8_t* k_codes;             // [num_pages][page_size][Hkv][D]
  uint8_t* v_codes;
  float* k_scales;              // [num_pages][page_size / block][Hkv]
  float* v_scales;
  const int32_t* block_table;   // [N][max_pages]
  const int32_t* start_pos;     // [N]
  int* status;                  // caller's device status or null
  int N, T, Hkv, max_pages, num_pages;
  int page_shift, block_shift;  // log2(page_size), log2(tokens per scale)
  int blocks;                   // blocks that T tokens of a sequence touch at most
  int warps_per_unit;           // min(block / 16, 8)
};

// The block's scale from the bits of its largest |x| (a bf16 value widened to fp32).
// NaN or infinity: a NaN scale, so that the block reads as NaN.
template <bool I8>
__device__ __forceinline__ float q8_scale(uint32_t amax_bits) {
  if (amax_bits >= 0x7F800000u) return __int_as_float(0x7fc00000);
  const int e = int(amax_bits >> 23) - 127, mant = int(amax_bits >> 16) & 0x7F;
  // 448 = 1.75 * 2^8 (mantissa 0x60 of 7 bits), 127 = (1 + 126/128) * 2^6
  int s = I8 ? e - 6 + (mant > 0x7E ? 1 : 0) : e - 8 + (mant > 0x60 ? 1 : 0);
  s = min(max(s, -100), I8 ? 121 : 119);
  return __uint_as_float(uint32_t(s + 127) << 23);
}

// Two values (already divided by the scale) -> two codes, the first in the low byte.
template <bool I8>
__device__ __forceinline__ uint32_t q8_codes2(float a, float b) {
  if constexpr (I8) {
    const int i = max(-127, min(127, __float2int_rn(a))), j = max(-127, min(127, __float2int_rn(b)));
    return (uint32_t(i) & 0xFFu) | ((uint32_t(j) & 0xFFu) << 8);
  } else {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(b), "f"(a));
    return r;
  }
}
// Four codes -> four values (not yet multiplied by the scale).
template <bool I8>
__device__ __forceinline__ void q8_values4(uint32_t four, float (&v)[4]) {
  if constexpr (I8) {
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = float(int8_t(four >> (8 * i)));
  } else {
    uint32_t lo, hi;
    e4m3x4_to_f16x2x2(four, lo, hi);
    v[0] = f16_lo(lo); v[1] = f16_hi(lo); v[2] = f16_lo(hi); v[3] = f16_hi(hi);
  }
}

// Unit = (sequence, touched block, K or V, head): its scale needs the largest |x|
// of the block's new tokens, so one group of warps_per_unit warps owns it whole.
// Each warp holds 16 slots of the block in registers (SEGS = 2: blocks of 256
// slots on 8 warps), so the new tokens are read once. If tokens of an earlier
// call sit before the first new one, the scale may only grow, and if it grows
// their codes are read and rounded again to the new scale. Heads are innermost
// over the warps of the grid, so neighbouring warps read neighbouring 2 D bytes.
template <int D, bool I8, int SEGS>
__global__ void __launch_bounds__(256) kv_append_q8_kernel(const KvAppendQ8Params p) {
  constexpr int LPR = D / 8;              // lanes per row: 8 values each
  constexpr int RPP = 32 / LPR;           // rows per pass
  constexpr int PASSES = 16 / RPP;        // passes over a 16-slot segment
  __shared__ uint32_t sh_amax[8];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int wpu = p.warps_per_unit;
  const int units_per_cta = 8 / wpu;
  const int wi = warp % wpu;              // warp of the unit
  const int row_in_pass = lane / LPR, col = (lane % LPR) * 8;
  const int block = 1 << p.block_shift;
  const long long units = (long long)p.N * p.blocks * 2 * p.Hkv;
  for (long long base = (long long)blockIdx.x * units_per_cta; base < units;
       base += (long long)gridDim.x * units_per_cta) {
    const long long u = base + warp / wpu;
    bool live = u < units;
    const int h = live ? int(u % p.Hkv) : 0;
    const long long r1 = live ? u / p.Hkv : 0;
    const bool is_v = (r1 & 1) != 0;
    const long long r2 = r1 >> 1;
    const int j = int(r2 % p.blocks), b = int(r2 / p.blocks);
    const long long pos0 = __ldg(&p.start_pos[b]);
    const long long blk = (pos0 >> p.block_shift) + j;       // floor, also for a negative start
    const long long s0 = blk << p.block_shift;               // position of the block's first slot
    const long long n_begin = max(pos0, s0), n_end = min(pos0 + p.T, s0 + block);
    live = live && n_begin < n_end;
    int page = -1;
    if (live) {
      const long long lp = s0 >> p.page_shift;
      if (s0 >= 0 && lp < p.max_pages) page = __ldg(&p.block_table[size_t(b) * p.max_pages + lp]);
      if (page < 0 || page >= p.num_pages) {
        if (lane == 0 && wi == 0) raise_status(p.status, ATTN_ERR_DEVICE_BOUNDS);
        live = false;
      }
    }
    const int in_page = int(s0 & ((1ll << p.page_shift) - 1));
    const int kept = live ? int(n_begin - s0) : 0;           // slots of earlier tokens (first block only)
    const int stop = live ? int(n_end - s0) : 0;
    const __nv_bfloat16* src = is_v ? p.v_new : p.k_new;
    uint8_t* codes = (is_v ? p.v_codes : p.k_codes) +
                     ((size_t(live ? page : 0) << p.page_shift) + in_page) * p.Hkv * D + size_t(h) * D;
    float* scale_at = (is_v ? p.v_scales : p.k_scales) +
                      ((size_t(live ? page : 0) << (p.page_shift - p.block_shift)) + (in_page >> p.block_shift)) * p.Hkv + h;

    // ---- the new tokens, and their largest |x|
    uint4 x[SEGS][PASSES];
    uint32_t amax = 0;
#pragma unroll
    for (int g = 0; g < SEGS; ++g)
#pragma unroll
      for (int i = 0; i < PASSES; ++i) {
        const int slot = (g * wpu + wi) * 16 + i * RPP + row_in_pass;
        x[g][i] = make_uint4(0, 0, 0, 0);
        if (slot >= kept && slot < stop) {
          const long long t = s0 + slot - pos0;
          x[g][i] = __ldg(reinterpret_cast<const uint4*>(src + ((size_t(b) * p.T + t) * p.Hkv + h) * D + col));
        }
      }
#pragma unroll
    for (int g = 0; g < SEGS; ++g)
#pragma unroll
      for (int i = 0; i < PASSES; ++i) {
        const uint32_t w[4] = {x[g][i].x, x[g][i].y, x[g][i].z, x[g][i].w};
#pragma unroll
        for (int e = 0; e < 4; ++e) amax = max(amax, max((w[e] << 16) & 0x7FFF0000u, w[e] & 0x7FFF0000u));
      }
    amax = __reduce_max_sync(0xffffffffu, amax);
    const float before = kept > 0 ? *scale_at : 0.f;
    if (wpu > 1) {
      if (lane == 0) sh_amax[warp] = amax;
      __syncthreads();                       // also: every warp has read the scale before one writes it
      for (int w = 0; w < wpu; ++w) amax = max(amax, sh_amax[warp - wi + w]);
      __syncthreads();
    }
    if (!live) continue;                     // whole units; the barriers above are already behind
    const float cand = q8_scale<I8>(amax);
    const float scale = kept > 0 && !(cand > before) && cand == cand ? before : cand;
    const float inv = 1.f / scale;           // exact for a power of two

    // ---- earlier tokens of the block, if the scale grew
    if (kept > 0 && scale != before && scale == scale) {
      const float ratio = before * inv;
#pragma unroll
      for (int g = 0; g < SEGS; ++g)
#pragma unroll
        for (int i = 0; i < PASSES; ++i) {
          const int slot = (g * wpu + wi) * 16 + i * RPP + row_in_pass;
          if (slot >= kept) continue;
          uint2* at = reinterpret_cast<uint2*>(codes + size_t(slot) * p.Hkv * D + col);
          const uint2 old = *at;
          float a[4], c[4];
          q8_values4<I8>(old.x, a);
          q8_values4<I8>(old.y, c);
          uint2 out;
          out.x = q8_codes2<I8>(a[0] * ratio, a[1] * ratio) | (q8_codes2<I8>(a[2] * ratio, a[3] * ratio) << 16);
          out.y = q8_codes2<I8>(c[0] * ratio, c[1] * ratio) | (q8_codes2<I8>(c[2] * ratio, c[3] * ratio) << 16);
          *at = out;
        }
    }
    // ---- the new tokens' codes
#pragma unroll
    for (int g = 0; g < SEGS; ++g)
#pragma unroll
      for (int i = 0; i < PASSES; ++i) {
        const int slot = (g * wpu + wi) * 16 + i * RPP + row_in_pass;
        if (slot < kept || slot >= stop) continue;
        const uint32_t w[4] = {x[g][i].x, x[g][i].y, x[g][i].z, x[g][i].w};
        uint32_t q[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) q[e] = q8_codes2<I8>(bf16_lo(w[e]) * inv, bf16_hi(w[e]) * inv);
        *reinterpret_cast<uint2*>(codes + size_t(slot) * p.Hkv * D + col) =
            make_uint2(q[0] | (q[1] << 16), q[2] | (q[3] << 16));
      }
    if (lane == 0 && wi == 0) *scale_at = scale;
  }
}

struct KvReadQ8Params {
  const uint8_t* k_codes;       // [num_pages][page_size][Hkv][D]
  const uint8_t* v_codes;
  const float* k_scales;        // [num_pages][page_size / block][Hkv]
  const float* v_scales;
  const int32_t* block_table;   // [N][max_pages]
  const int32_t* seq_lens;      // [N]
  __nv_bfloat16* k_out;         // [N][T][Hkv][D]
  __nv_bfloat16* v_out;
  int32_t* identity;            // [N][max_pages] or null: entry (b, i) = b * max_pages + i for the pages in use
  int* status;
  int N, T, Hkv, max_pages, num_pages;
  int min_len;                  // rows read even of a shorter sequence (the chunk of a prefill; 0 otherwise)
  int page_shift, block_shift;
  int ctas_per_seq;
};

// Sixteen codes times a scale -> sixteen bf16, rounded once (exact for scales that are powers of two).
template <bool I8>
__device__ __forceinline__ void q8_widen16(const uint4& c, float s, uint4& a, uint4& b) {
  const uint32_t w[4] = {c.x, c.y, c.z, c.w};
  uint32_t o[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float v[4];
    q8_values4<I8>(w[i], v);
    o[2 * i] = pack_bf16x2(v[0] * s, v[1] * s);
    o[2 * i + 1] = pack_bf16x2(v[2] * s, v[3] * s);
  }
  a = make_uint4(o[0], o[1], o[2], o[3]);
  b = make_uint4(o[4], o[5], o[6], o[7]);
}

// One warp per token row (all heads of K and of V), 16 codes per lane and step.
// Rows at or past a sequence's length are left as they were.
template <int D, bool I8>
__global__ void __launch_bounds__(256) kv_read_q8_kernel(const KvReadQ8Params p) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int b = int(blockIdx.x / unsigned(p.ctas_per_seq)), part = int(blockIdx.x % unsigned(p.ctas_per_seq));
  const int len = __ldg(&p.seq_lens[b]);
  const int held = min(max(len, p.min_len), p.T);
  if (threadIdx.x == 0 && part == 0 && (len < 0 || (len - 1) >> p.page_shift >= p.max_pages))
    raise_status(p.status, ATTN_ERR_DEVICE_BOUNDS);
  const int32_t* table = p.block_table + size_t(b) * p.max_pages;
  if (p.identity) {
    const int pages = (held + (1 << p.page_shift) - 1) >> p.page_shift;
    for (int i = part * 256 + threadIdx.x; i < pages; i += p.ctas_per_seq * 256)
      p.identity[size_t(b) * p.max_pages + i] = b * p.max_pages + i;
  }
  const int vecs = p.Hkv * (D / 16);       // 16-code vectors of a row
  for (int t = part * 8 + warp; t < held; t += p.ctas_per_seq * 8) {
    const int page = __ldg(&table[t >> p.page_shift]);
    const bool good = page >= 0 && page < p.num_pages;
    if (!good && lane == 0) raise_status(p.status, ATTN_ERR_DEVICE_BOUNDS);
    const int slot = t & ((1 << p.page_shift) - 1);
    const size_t row = good ? ((size_t(page) << p.page_shift) + slot) * p.Hkv * D : 0;
    const size_t srow = good ? ((size_t(page) << (p.page_shift - p.block_shift)) + (slot >> p.block_shift)) * p.Hkv : 0;
    const size_t out = (size_t(b) * p.T + t) * p.Hkv * D;
    for (int i = lane; i < vecs; i += 32) {
      uint4 ka = make_uint4(0, 0, 0, 0), kb = ka, va = ka, vb = ka;
      if (good) {
        const uint4 kc = __ldg(reinterpret_cast<const uint4*>(p.k_codes + row) + i);
        const uint4 vc = __ldg(reinterpret_cast<const uint4*>(p.v_codes + row) + i);
        const int h = i / (D / 16);
        q8_widen16<I8>(kc, __ldg(&p.k_scales[srow + h]), ka, kb);
        q8_widen16<I8>(vc, __ldg(&p.v_scales[srow + h]), va, vb);
      }
      uint4* ko = reinterpret_cast<uint4*>(p.k_out + out) + 2 * i;
      uint4* vo = reinterpret_cast<uint4*>(p.v_out + out) + 2 * i;
      ko[0] = ka; ko[1] = kb;
      vo[0] = va; vo[1] = vb;
    }
  }
}

}  // namespace attn
