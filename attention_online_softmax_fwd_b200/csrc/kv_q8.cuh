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
  unsigned units;               // N * blocks * 2 * Hkv
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

// Two bf16 values, each at most 127 * 2^121 in size afterwards.
__device__ __forceinline__ uint32_t q8_saturate(uint32_t w) {
  return __vminu2(w & 0x7FFF7FFFu, 0x7F7E7F7Eu) | (w & 0x80008000u);
}

// Two values (already divided by the scale) -> two codes, the first in the low byte.
template <bool I8>
__device__ __forceinline__ uint32_t q8_codes2(float a, float b) {
  if constexpr (I8) {
    // 1.5 * 2^23 + v holds rint(v) in its low bits, to nearest even: one addition instead of a conversion.
    // |v| <= 127 by the choice of the scale (q8_saturate where the scale is the largest one)
    constexpr float kMagic = 12582912.f;
    return __byte_perm(__float_as_uint(a + kMagic), __float_as_uint(b + kMagic), 0x0040) & 0xFFFFu;
  } else {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(b), "f"(a));
    return r;
  }
}
// x / s and a * b rounded to odd (truncated, the last bit set where something was cut off): rounding that
// again, to a code's few bits, is as good as rounding the exact number. For scales that are no powers of two.
__device__ __forceinline__ float q8_odd(float truncated, float rest) {
  return rest != 0.f ? __uint_as_float(__float_as_uint(truncated) | 1u) : truncated;
}
__device__ __forceinline__ float q8_div_odd(float x, float s) {
  const float q = __fdiv_rz(x, s);
  return q8_odd(q, fmaf(-q, s, x));
}
__device__ __forceinline__ float q8_mul_odd(float a, float b) {
  const float m = __fmul_rz(a, b);
  return q8_odd(m, fmaf(a, b, -m));
}
// int8: a value beyond the codes that are written (-127 .. 127) becomes the last of them.
template <bool I8>
__device__ __forceinline__ float q8_clamp(float v) { return I8 ? fminf(fmaxf(v, -127.f), 127.f) : v; }

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
// Bound by HBM, and by its instructions nearly as much: 201 MB (8 prompts of 4096
// tokens, 8 heads of 128, int8) in 34.2 us, 5.9 TB/s, replayed on the same tokens, and
// 38 to 39 us a call with others each time. Maxima of packed bf16 bits and
// conversions without clamps took it there from 55 us, some of it by 64 registers
// (32 warps an SM); a unit a warp, or its two copies in one thread, would read no less.
template <int D, bool I8, int SEGS>
__global__ void __launch_bounds__(256, SEGS == 1 ? 4 : 2) kv_append_q8_kernel(const KvAppendQ8Params p) {
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
  const unsigned units = p.units;         // below 2^31, so that base cannot wrap
  for (unsigned base = blockIdx.x * units_per_cta; base < units; base += gridDim.x * units_per_cta) {
    const unsigned u = base + warp / wpu;
    bool live = u < units;
    const unsigned r1 = live ? u / unsigned(p.Hkv) : 0u;
    const int h = live ? int(u - r1 * p.Hkv) : 0;
    const bool is_v = (r1 & 1) != 0;
    const int b = int((r1 >> 1) / unsigned(p.blocks)), j = int((r1 >> 1) - unsigned(b) * p.blocks);
    const int pos0 = __ldg(&p.start_pos[b]);
    const int first = (pos0 >> p.block_shift) << p.block_shift;   // first touched block's first position (floor)
    const long long s0 = (long long)first + (long long)j * block;   // this block's first position
    const int before_new = pos0 - first;                          // its slots before the first new token, if j = 0
    const int kept_slots = j == 0 ? before_new : 0;
    // the new token in slot i is number i - token0
    const long long token0 = (long long)before_new - (long long)j * block;
    const long long left = token0 + p.T;
    const int stop_slot = left < block ? int(left) : block;
    live = live && kept_slots < stop_slot;
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
    // slots of earlier tokens (first block only; positions below 0 hold none)
    const int kept = live && first >= 0 ? kept_slots : 0;
    const int begin = live ? kept_slots : 0;                      // first new slot
    const int stop = live ? stop_slot : 0;
    const int row_elems = p.Hkv * D;
    const __nv_bfloat16* new_rows =     // row of the block's slot 0 (read from its first new slot on)
        (is_v ? p.v_new : p.k_new) + ((long long)b * p.T - token0) * row_elems + h * D + col;
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
        if (slot >= begin && slot < stop)
          x[g][i] = __ldg(reinterpret_cast<const uint4*>(new_rows + (long long)slot * row_elems));
      }
#pragma unroll
    for (int g = 0; g < SEGS; ++g)
#pragma unroll
      for (int i = 0; i < PASSES; ++i) {
        // |bf16| orders as its bits do, NaN above infinity above the rest: two 16-bit maxima an instruction
        const uint32_t a = __vmaxu2(x[g][i].x & 0x7FFF7FFFu, x[g][i].y & 0x7FFF7FFFu);
        const uint32_t c = __vmaxu2(x[g][i].z & 0x7FFF7FFFu, x[g][i].w & 0x7FFF7FFFu);
        amax = __vmaxu2(amax, __vmaxu2(a, c));
      }
    amax = __reduce_max_sync(0xffffffffu, max(amax & 0xFFFF0000u, amax << 16));
    const float before = kept > 0 ? *scale_at : 0.f;
    if (wpu > 1) {
      if (lane == 0) sh_amax[warp] = amax;
      __syncthreads();                       // also: every warp has read the scale before one writes it
      for (int w = 0; w < wpu; ++w) amax = max(amax, sh_amax[warp - wi + w]);
      __syncthreads();
    } else {
      __syncwarp();                          // every lane has read the scale before lane 0 writes it
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
#pragma unroll
          for (int e = 0; e < 4; ++e) {   // another writer's codes may hold -128, and its scale any bits
            a[e] = q8_clamp<I8>(q8_mul_odd(a[e], ratio));
            c[e] = q8_clamp<I8>(q8_mul_odd(c[e], ratio));
          }
          *at = make_uint2(q8_codes2<I8>(a[0], a[1]) | (q8_codes2<I8>(a[2], a[3]) << 16),
                           q8_codes2<I8>(c[0], c[1]) | (q8_codes2<I8>(c[2], c[3]) << 16));
        }
    }
    // ---- the new tokens' codes
    if (scale == scale && (__float_as_uint(scale) & 0x7FFFFFu) != 0) {
      // a block begun by another writer, whose scale is no power of two: x * inv would round twice. Rare, so the
      // tokens are read again, and the common path keeps its registers
#pragma unroll 1
      for (int n = 0; n < SEGS * PASSES; ++n) {
        const int slot = (n / PASSES * wpu + wi) * 16 + n % PASSES * RPP + row_in_pass;
        if (slot < begin || slot >= stop) continue;
        const uint4 t = __ldg(reinterpret_cast<const uint4*>(new_rows + (long long)slot * row_elems));
        const uint32_t w[4] = {t.x, t.y, t.z, t.w};
        uint32_t q[4];
#pragma unroll
        for (int e = 0; e < 4; ++e)
          q[e] = q8_codes2<I8>(q8_clamp<I8>(q8_div_odd(bf16_lo(w[e]), scale)), q8_clamp<I8>(q8_div_odd(bf16_hi(w[e]), scale)));
        *reinterpret_cast<uint2*>(codes + size_t(slot) * p.Hkv * D + col) =
            make_uint2(q[0] | (q[1] << 16), q[2] | (q[3] << 16));
      }
    } else {
      if (I8 && amax > 0x7F7E0000u) {   // above 127 * 2^121: the scale could not grow, the values saturate there
#pragma unroll
        for (int g = 0; g < SEGS; ++g)
#pragma unroll
          for (int i = 0; i < PASSES; ++i) {
            x[g][i].x = q8_saturate(x[g][i].x); x[g][i].y = q8_saturate(x[g][i].y);
            x[g][i].z = q8_saturate(x[g][i].z); x[g][i].w = q8_saturate(x[g][i].w);
          }
      }
#pragma unroll
      for (int g = 0; g < SEGS; ++g)
#pragma unroll
        for (int i = 0; i < PASSES; ++i) {
          const int slot = (g * wpu + wi) * 16 + i * RPP + row_in_pass;
          if (slot < begin || slot >= stop) continue;
          const uint32_t w[4] = {x[g][i].x, x[g][i].y, x[g][i].z, x[g][i].w};
          uint32_t q[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) q[e] = q8_codes2<I8>(bf16_lo(w[e]) * inv, bf16_hi(w[e]) * inv);
          *reinterpret_cast<uint2*>(codes + size_t(slot) * p.Hkv * D + col) =
              make_uint2(q[0] | (q[1] << 16), q[2] | (q[3] << 16));
        }
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
  int* status;
  int N, T, Hkv, max_pages, num_pages;
  int min_len;                  // rows read even of a shorter sequence (the chunk of a prefill; 0 otherwise)
  int pad;                      // rows up to the next multiple of this are set to zero (0: left as they were)
  int page_shift, block_shift;
  int group_shift;              // log2(lanes of a row): the power of two >= its 8-code vectors, at most 32
  int ctas_per_seq;
};

// Eight codes times a scale -> eight bf16, rounded once (exact for scales that are powers of two).
template <bool I8>
__device__ __forceinline__ uint4 q8_widen8(const uint2& c, float s) {
  float v[4], w[4];
  q8_values4<I8>(c.x, v);
  q8_values4<I8>(c.y, w);
  return make_uint4(pack_bf16x2(v[0] * s, v[1] * s), pack_bf16x2(v[2] * s, v[3] * s), pack_bf16x2(w[0] * s, w[1] * s),
                    pack_bf16x2(w[2] * s, w[3] * s));
}

// Whether one of eight bf16 is a NaN or an infinity.
__device__ __forceinline__ bool q8_not_finite(const uint4& w) {
  const uint32_t m = __vmaxu2(__vmaxu2(w.x & 0x7FFF7FFFu, w.y & 0x7FFF7FFFu), __vmaxu2(w.z & 0x7FFF7FFFu, w.w & 0x7FFF7FFFu));
  return max(m & 0xFFFF0000u, m << 16) >= 0x7F800000u;
}

// A group of lanes (a warp, or fewer for narrow rows) per token row of K and of V.
// Bound by HBM: 393 MB (16 sequences, 70,000 tokens, 8 heads of 128) in 66 us, 6.0 TB/s.
// Eight codes a lane, so that a warp's stores are whole lines, four such vectors of
// K and of V in flight, and some 32 CTAs per SM in turn; 16 codes a lane took 70 us,
// one vector in flight and 8 CTAs per SM 75 us. Rows at or past a sequence's length
// are left as they were.
// For the prefill (pad > 0) a value that is not finite becomes zero and its key NaN:
// a hidden key's score is replaced, whatever it is, but a hidden value is multiplied
// by a zero in the tensor cores, and would reach the chunk's earlier queries. The
// queries that see the token are NaN either way. A key that is infinite (scale times
// code past the largest number) becomes NaN as well: a score of -inf would only hide it.
template <int D, bool I8>
__global__ void __launch_bounds__(256) kv_read_q8_kernel(const KvReadQ8Params p) {
  const int b = int(blockIdx.x / unsigned(p.ctas_per_seq)), part = int(blockIdx.x % unsigned(p.ctas_per_seq));
  const int len = __ldg(&p.seq_lens[b]);
  const int held = min(max(len, p.min_len), p.T);
  if (threadIdx.x == 0 && part == 0 && (len < 0 || (len - 1) >> p.page_shift >= p.max_pages))
    raise_status(p.status, ATTN_ERR_DEVICE_BOUNDS);
  const int32_t* table = p.block_table + size_t(b) * p.max_pages;
  const int stop = p.pad ? min((held + p.pad - 1) / p.pad * p.pad, p.T) : held;
  const int vecs = p.Hkv * (D / 8);                     // 8-code vectors of a row
  const int group = 1 << p.group_shift;                 // lanes of a row
  const int v0 = threadIdx.x & (group - 1);
  const int rows = 256 >> p.group_shift;                // rows of a CTA at a time
  for (long long t = (long long)part * rows + (threadIdx.x >> p.group_shift); t < stop; t += (long long)p.ctas_per_seq * rows) {
    const int page = t < held ? __ldg(&table[t >> p.page_shift]) : -1;
    const bool good = page >= 0 && page < p.num_pages;
    if (!good && v0 == 0 && t < held) raise_status(p.status, ATTN_ERR_DEVICE_BOUNDS);
    const int slot = int(t) & ((1 << p.page_shift) - 1);
    const size_t row = ((size_t(good ? page : 0) << p.page_shift) + slot) * vecs;
    const size_t srow = ((size_t(good ? page : 0) << (p.page_shift - p.block_shift)) + (slot >> p.block_shift)) * p.Hkv;
    const uint2* kc = reinterpret_cast<const uint2*>(p.k_codes) + row;
    const uint2* vc = reinterpret_cast<const uint2*>(p.v_codes) + row;
    const size_t out = (size_t(b) * p.T + t) * vecs;
    uint4* ko = reinterpret_cast<uint4*>(p.k_out) + out;
    uint4* vo = reinterpret_cast<uint4*>(p.v_out) + out;
    constexpr int U = 4;
    for (int i0 = v0; i0 < vecs; i0 += group * U) {
      uint2 k[U], v[U];
      float ks[U], vs[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int i = i0 + u * group;
        k[u] = v[u] = make_uint2(0, 0);
        ks[u] = vs[u] = 0.f;
        if (i < vecs && good) {
          k[u] = __ldg(kc + i);
          v[u] = __ldg(vc + i);
          ks[u] = __ldg(&p.k_scales[srow + i / (D / 8)]);
          vs[u] = __ldg(&p.v_scales[srow + i / (D / 8)]);
        }
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int i = i0 + u * group;
        if (i >= vecs) continue;
        uint4 kw = q8_widen8<I8>(k[u], ks[u]), vw = q8_widen8<I8>(v[u], vs[u]);
        if (p.pad) {
          const bool bad_v = q8_not_finite(vw);
          if (bad_v || q8_not_finite(kw)) kw = make_uint4(0x7FC07FC0u, 0x7FC07FC0u, 0x7FC07FC0u, 0x7FC07FC0u);
          if (bad_v) vw = make_uint4(0, 0, 0, 0);
        }
        ko[i] = kw;
        vo[i] = vw;
      }
    }
  }
}

}  // namespace attn
