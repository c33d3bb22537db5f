// Device code shared by the few-row kernels (the layer for a few tokens and the
// 4-bit Linear): a wave streams 16 rows of a weight matrix from HBM straight
// into the operand registers of the matrix cores.
//
// C[row, n] = sum_k A[row, k] W[n, k] for up to 16 rows of activations is
// bound by reading W once: a 16x16 MFMA has the rows of A on one side (empty
// rows cost nothing that is not already paid) and 16 rows of W on the other.
// Lane l of a wave holds row l % 16 of either operand and, per MFMA, the k of
// its quarter q = l / 16.  The result has W row n = l % 16 and activation rows
// 4 q .. 4 q + 3 in the lane's four registers.
//
// One step is one 16-byte load per lane and W row tile: 16 k of float32, 32 of
// bf16, 128 of 4-bit codes.  Loads are buffer loads whose range check returns
// zero, without memory traffic, for lanes past the end of k, W rows past the
// matrix and empty activation rows.
#pragma once

#include "moe_internal.h"

namespace moe {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));

constexpr uint32_t kOut = 0x7ffffff0u;   // an offset past every range used here: the load returns zero

__device__ __forceinline__ int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }

__device__ __forceinline__ u32x4 load16(__amdgpu_buffer_rsrc_t r, uint32_t voff, uint32_t soff) {
  return __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(r, static_cast<int>(voff),
                                                                         static_cast<int>(soff), 0));
}

// Weight formats.
//   kK     k of one step (all four quarters)
//   kLane  k of one lane's 16-byte load
//   kActs  16-byte activation loads per lane and step
enum class Fmt { kF32, kBf16, kW4 };
template <Fmt F> struct FmtOf;
template <> struct FmtOf<Fmt::kF32> { static constexpr int kK = 16, kLane = 4, kActs = 1; };
template <> struct FmtOf<Fmt::kBf16> { static constexpr int kK = 32, kLane = 8, kActs = 1; };
template <> struct FmtOf<Fmt::kW4> { static constexpr int kK = 128, kLane = 32, kActs = 4; };

// Where a wave finds 16 rows of W.  Step s's load is at voff[s & 1] + (s >> 1) *
// pair: row-major matrices advance 128 bytes per two steps (voff[1] = voff[0] +
// 64); in the tile-packed layout two steps are one 64-column block, 32 KB apart,
// with the lane's chunk at a position of its own in either half.
// 4-bit: scales [n, K/G] bf16 and zero points [n, K/G] uint8 (or none: 8).
struct WRows {
  __amdgpu_buffer_rsrc_t w;
  uint32_t voff[2];
  uint32_t pair;
  __amdgpu_buffer_rsrc_t s, z;   // 4-bit: this tile's scale and zero-point rows
  uint32_t srow;                 // 4-bit: first scale of the lane's row (elements)
  bool has_z;
};

template <Fmt F>
__device__ __forceinline__ WRows rows_of(const WMat& m, long long mat, int n0, int lane) {
  const int r = lane & 15, q = lane >> 4;
  WRows o;
  const int left = min(16, m.N - n0);
  if constexpr (F == Fmt::kW4) {
    const uint32_t pitch = static_cast<uint32_t>(m.K) / 2;
    const uint32_t ng = static_cast<uint32_t>(m.K) >> m.gshift;
    const long long row0 = mat * m.N + n0;
    o.w = make_rsrc(m.w + row0 * pitch, static_cast<uint32_t>(left) * pitch);
    o.voff[0] = static_cast<uint32_t>(r) * pitch + 16u * q;
    o.voff[1] = o.voff[0] + 64u;
    o.pair = 128u;
    o.s = make_rsrc(m.s + row0 * ng, static_cast<uint32_t>(left) * ng * 2u);
    o.has_z = m.z != nullptr;
    o.z = o.s;
    if (o.has_z) o.z = make_rsrc(m.z + row0 * ng, static_cast<uint32_t>(left) * ng);
    o.srow = static_cast<uint32_t>(r) * ng;
  } else {
    constexpr uint32_t eb = F == Fmt::kF32 ? 4 : 2;
    const uint32_t pitch = static_cast<uint32_t>(m.K) * eb;
    if (F == Fmt::kBf16 && m.packed) {
      const uint32_t nkb = static_cast<uint32_t>(m.K) / 64;
      const uint32_t r256 = static_cast<uint32_t>(n0 % 256 + r);
      const long long blk = (mat * (m.N / 256) + n0 / 256) * nkb;
      const uint32_t sw = (r256 & 7u) ^ ((r256 >> 3) & 1u);
      o.w = make_rsrc(m.w + blk * 32768, nkb * 32768u);
      o.voff[0] = r256 * 128u + ((static_cast<uint32_t>(q) ^ sw) * 16u);
      o.voff[1] = r256 * 128u + ((static_cast<uint32_t>(4 + q) ^ sw) * 16u);
      o.pair = 32768u;
    } else {
      o.w = make_rsrc(m.w + (mat * m.N + n0) * pitch, static_cast<uint32_t>(left) * pitch);
      o.voff[0] = static_cast<uint32_t>(r) * pitch + 16u * q;
      o.voff[1] = o.voff[0] + 64u;
      o.pair = 128u;
    }
    o.s = o.z = o.w;
    o.srow = 0;
    o.has_z = false;
  }
  return o;
}

// ------------------------------------------------------------ 4-bit codes --
// A lane's 16 bytes are 32 codes of one row; the four lane quarters hold 128
// consecutive k.  A scale covers 32 k or a multiple, and an MFMA sums over the
// quarters, so each MFMA must take its 32 k from one block of 32: the dwords
// are exchanged between the quarters as a 4 x 4 transpose (dword g of quarter
// q becomes dword q of quarter g), two register swaps per stage.
__device__ __forceinline__ void transpose_quarters(u32x4& v) {
  // halves: (q0 q1 | q2 q3) dwords 0,1 of the upper half against 2,3 of the lower
  auto a = __builtin_amdgcn_permlane32_swap(v.x, v.z, false, false);
  auto b = __builtin_amdgcn_permlane32_swap(v.y, v.w, false, false);
  auto c = __builtin_amdgcn_permlane16_swap(a[0], b[0], false, false);
  auto d = __builtin_amdgcn_permlane16_swap(a[1], b[1], false, false);
  v.x = c[0];
  v.y = c[1];
  v.z = d[0];
  v.w = d[1];
}

// Eight codes of a dword as bf16 numbers 128 + q: 0x4300 is 128 with a last
// place of 1, so a code is its low bits.  Register i holds codes i and i + 4.
__device__ __forceinline__ bf16x8 codes_to_bf16(uint32_t w) {
  u32x4 o;
  o.x = (w & 0x000f000fu) | 0x43004300u;
  o.y = ((w >> 4) & 0x000f000fu) | 0x43004300u;
  o.z = ((w >> 8) & 0x000f000fu) | 0x43004300u;
  o.w = ((w >> 12) & 0x000f000fu) | 0x43004300u;
  return __builtin_bit_cast(bf16x8, o);
}

// Eight consecutive bf16 activations in the order of codes_to_bf16:
// (0,4) (1,5) (2,6) (3,7).
__device__ __forceinline__ bf16x8 acts_in_code_order(u32x4 v) {
  u32x4 o;
  o.x = __builtin_amdgcn_perm(v.z, v.x, 0x05040100u);
  o.y = __builtin_amdgcn_perm(v.z, v.x, 0x07060302u);
  o.z = __builtin_amdgcn_perm(v.w, v.y, 0x05040100u);
  o.w = __builtin_amdgcn_perm(v.w, v.y, 0x07060302u);
  return __builtin_bit_cast(bf16x8, o);
}

// value v of quarter g in all four quarters
__device__ __forceinline__ void spread_quarters(uint32_t v, uint32_t (&o)[4]) {
  auto h = __builtin_amdgcn_permlane32_swap(v, v, false, false);   // h[0]: q0 q1 q0 q1, h[1]: q2 q3 q2 q3
  auto a = __builtin_amdgcn_permlane16_swap(h[0], h[0], false, false);
  auto b = __builtin_amdgcn_permlane16_swap(h[1], h[1], false, false);
  o[0] = a[0];
  o[1] = a[1];
  o[2] = b[0];
  o[3] = b[1];
}

// ------------------------------------------------------------- streaming --
// acc[j] += A rows of tile j times the 16 rows of W over steps [s0, s1) (of a
// matrix with K columns), for the tiles of `tiles` (bit j).  a: activations;
// aoff[j] the lane's byte offset of row (lane % 16) of tile j plus 16 q, or
// kOut for an empty row.  U steps are loaded together.
template <Fmt F, int NT, int U>
__device__ __forceinline__ void stream_rows(floatx4 (&acc)[NT], const WRows& wr, __amdgpu_buffer_rsrc_t a,
                                            const uint32_t (&aoff)[NT], uint32_t tiles, int s0, int s1, int K,
                                            int gshift, int lane) {
  using Ff = FmtOf<F>;
  static_assert(U % 2 == 0, "a batch starts at the parity of s0");
  const int q = lane >> 4;
  const int kend = min(K, s1 * Ff::kK);
  const uint32_t v0 = s0 & 1 ? wr.voff[1] : wr.voff[0], v1 = s0 & 1 ? wr.voff[0] : wr.voff[1];
  for (int sb = s0; sb < s1; sb += U) {
    u32x4 w[U];
    uint32_t sc[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int s = sb + u;
      const bool in = s * Ff::kK + q * Ff::kLane < kend;
      w[u] = load16(wr.w, in ? (u & 1 ? v1 : v0) : kOut, static_cast<uint32_t>(s >> 1) * wr.pair);
      if constexpr (F == Fmt::kW4) {
        // the lane's scale (high half) and its zero point as the bf16 number
        // -(128 + z) (low half)
        const uint32_t gi = wr.srow + (static_cast<uint32_t>(s * Ff::kK + q * Ff::kLane) >> gshift);
        const uint32_t sv = static_cast<uint16_t>(__builtin_amdgcn_raw_buffer_load_b16(
            wr.s, static_cast<int>(in ? gi * 2u : kOut), 0, 0));
        uint32_t zv = 8;
        if (wr.has_z)
          zv = static_cast<uint8_t>(__builtin_amdgcn_raw_buffer_load_b8(wr.z, static_cast<int>(in ? gi : kOut), 0, 0));
        sc[u] = (sv << 16) | 0xc300u | (zv & 15u);
      }
    }
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      if (NT > 1 && !((tiles >> j) & 1u)) continue;
      u32x4 x[U][Ff::kActs];
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int g = 0; g < Ff::kActs; ++g) {
          const int s = sb + u;
          const bool in = F == Fmt::kW4 ? s * Ff::kK + g * 32 < kend : s * Ff::kK + q * Ff::kLane < kend;
          x[u][g] = load16(a, in ? aoff[j] : kOut,
                           static_cast<uint32_t>(s) * (64u * Ff::kActs) + 64u * static_cast<uint32_t>(g));
        }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if constexpr (F == Fmt::kF32) {
          const floatx4 xv = __builtin_bit_cast(floatx4, x[u][0]);
          const floatx4 wv = __builtin_bit_cast(floatx4, w[u]);
          acc[j] = __builtin_amdgcn_mfma_f32_16x16x4f32(xv.x, wv.x, acc[j], 0, 0, 0);
          acc[j] = __builtin_amdgcn_mfma_f32_16x16x4f32(xv.y, wv.y, acc[j], 0, 0, 0);
          acc[j] = __builtin_amdgcn_mfma_f32_16x16x4f32(xv.z, wv.z, acc[j], 0, 0, 0);
          acc[j] = __builtin_amdgcn_mfma_f32_16x16x4f32(xv.w, wv.w, acc[j], 0, 0, 0);
        } else if constexpr (F == Fmt::kBf16) {
          acc[j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, x[u][0]),
                                                           __builtin_bit_cast(bf16x8, w[u]), acc[j], 0, 0, 0);
        } else {
          // per block of 32 k: sum (128 + q) x - sum (128 + z) x, both products
          // exact in float32 and the difference formed by the accumulator, then
          // times the scale
          u32x4 c = w[u];
          transpose_quarters(c);
          uint32_t sg[4];
          spread_quarters(sc[u], sg);
#pragma unroll
          for (int g = 0; g < 4; ++g) {
            const bf16x8 xv = acts_in_code_order(x[u][g]);
            const uint32_t zz = (sg[g] & 0xffffu) | (sg[g] << 16);
            const u32x4 z4 = {zz, zz, zz, zz};
            floatx4 t = {0.f, 0.f, 0.f, 0.f};
            t = __builtin_amdgcn_mfma_f32_16x16x32_bf16(xv, __builtin_bit_cast(bf16x8, z4), t, 0, 0, 0);
            t = __builtin_amdgcn_mfma_f32_16x16x32_bf16(xv, codes_to_bf16(c[g]), t, 0, 0, 0);
            const float s = __uint_as_float(sg[g] & 0xffff0000u);
#pragma unroll
            for (int i = 0; i < 4; ++i) acc[j][i] = fmaf(s, t[i], acc[j][i]);
          }
        }
      }
    }
  }
}

}  // namespace moe
