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

// Weight formats; 4-bit codes by their group.
enum class Fmt { kF32, kBf16, kW4g32, kW4g64, kW4g128 };
constexpr bool is_w4(Fmt f) { return f != Fmt::kF32 && f != Fmt::kBf16; }
// k of one step (all four quarters), of one lane's 16-byte load, and of one MFMA
constexpr int step_k(Fmt f) { return f == Fmt::kF32 ? 16 : f == Fmt::kBf16 ? 32 : 128; }
constexpr int lane_k(Fmt f) { return step_k(f) / 4; }
constexpr int group_shift(Fmt f) { return f == Fmt::kW4g32 ? 5 : f == Fmt::kW4g64 ? 6 : 7; }
constexpr int acts(Fmt f) { return is_w4(f) ? 4 : 1; }   // 16-byte activation loads per lane and step

// Where a wave finds 16 RT rows of W.  Step s's load of row tile r is at
// voff[s & 1] + r * tile + (s >> 1) * pair: row-major matrices advance 128 bytes
// per two steps (voff[1] = voff[0] + 64); in the tile-packed layout two steps
// are one 64-column block, 32 KB apart, with the lane's chunk at a position of
// its own in either half.
// 4-bit: scales [n, K/group] bf16 and zero points [n, K/group] uint8 (or none: 8).
struct WRows {
  __amdgpu_buffer_rsrc_t w;
  uint32_t voff[2];
  uint32_t pair, tile;
  __amdgpu_buffer_rsrc_t s, z;   // 4-bit: the rows' scales and zero points
  uint32_t srow, stile;          // 4-bit: first scale of the lane's row, scales of 16 rows
};

template <Fmt F, int RT>
__device__ __forceinline__ WRows rows_of(const WMat& m, long long mat, int n0, int lane) {
  const int r = lane & 15, q = lane >> 4;
  WRows o;
  const int left = min(16 * RT, m.N - n0);
  if constexpr (is_w4(F)) {
    const uint32_t pitch = static_cast<uint32_t>(m.K) / 2;
    const uint32_t ng = static_cast<uint32_t>(m.K) >> group_shift(F);
    const long long row0 = mat * m.N + n0;
    o.w = make_rsrc(m.w + row0 * pitch, static_cast<uint32_t>(left) * pitch);
    o.voff[0] = static_cast<uint32_t>(r) * pitch + 16u * q;
    o.voff[1] = o.voff[0] + 64u;
    o.pair = 128u;
    o.tile = 16u * pitch;
    o.s = make_rsrc(m.s + row0 * ng, static_cast<uint32_t>(left) * ng * 2u);
    o.z = o.s;
    if (m.z != nullptr) o.z = make_rsrc(m.z + row0 * ng, static_cast<uint32_t>(left) * ng);
    o.srow = static_cast<uint32_t>(r) * ng;
    o.stile = 16u * ng;
  } else {
    constexpr uint32_t eb = F == Fmt::kF32 ? 4 : 2;
    const uint32_t pitch = static_cast<uint32_t>(m.K) * eb;
    if (F == Fmt::kBf16 && m.packed) {   // 16 RT rows stay in one 256-row block
      const uint32_t nkb = static_cast<uint32_t>(m.K) / 64;
      const uint32_t r256 = static_cast<uint32_t>(n0 % 256 + r);
      const long long blk = (mat * (m.N / 256) + n0 / 256) * nkb;
      const uint32_t sw = (r256 & 7u) ^ ((r256 >> 3) & 1u);
      o.w = make_rsrc(m.w + blk * 32768, nkb * 32768u);
      o.voff[0] = r256 * 128u + ((static_cast<uint32_t>(q) ^ sw) * 16u);
      o.voff[1] = r256 * 128u + ((static_cast<uint32_t>(4 + q) ^ sw) * 16u);
      o.pair = 32768u;
      o.tile = 2048u;
    } else {
      o.w = make_rsrc(m.w + (mat * m.N + n0) * pitch, static_cast<uint32_t>(left) * pitch);
      o.voff[0] = static_cast<uint32_t>(r) * pitch + 16u * q;
      o.voff[1] = o.voff[0] + 64u;
      o.pair = 128u;
      o.tile = 16u * pitch;
    }
    o.s = o.z = o.w;
    o.srow = o.stile = 0;
  }
  return o;
}

// ------------------------------------------------------------ 4-bit codes --
// Eight codes of a dword as bf16 numbers 128 + q: 0x4300 is 128 with a last
// place of 1, so a code is its low bits.  Register i holds codes i and i + 4.
// (The constant comes in a register: an instruction reads one scalar at most,
// and and-or takes the mask from it.)
__device__ __forceinline__ uint32_t code_base() {
  uint32_t v;
  __asm__("v_mov_b32 %0, 0x43004300" : "=v"(v));
  return v;
}
__device__ __forceinline__ bf16x8 codes_to_bf16(uint32_t w, uint32_t base) {
  u32x4 o;
  o.x = (w & 0x000f000fu) | base;
  o.y = ((w >> 4) & 0x000f000fu) | base;
  o.z = ((w >> 8) & 0x000f000fu) | base;
  o.w = ((w >> 12) & 0x000f000fu) | base;
  return __builtin_bit_cast(bf16x8, o);
}

// Position of element k of a row in that order, within its block of eight:
// 0 4 1 5 2 6 3 7.  Activations meant for 4-bit weights are stored so.
__host__ __device__ constexpr int code_order(int k) {
  return (k & ~7) | ((k & 7) < 4 ? 2 * (k & 7) : 2 * (k & 7) - 7);
}
// eight consecutive bf16 activations put into it
__device__ __forceinline__ u32x4 to_code_order(u32x4 v) {
  u32x4 o;
  o.x = __builtin_amdgcn_perm(v.z, v.x, 0x05040100u);
  o.y = __builtin_amdgcn_perm(v.z, v.x, 0x07060302u);
  o.z = __builtin_amdgcn_perm(v.w, v.y, 0x05040100u);
  o.w = __builtin_amdgcn_perm(v.w, v.y, 0x07060302u);
  return o;
}

// An MFMA sums over the lane quarters, so its k must lie in one group.  A
// lane's four dwords are k q 32 + 8 i; within groups of 128 they may stay,
// within groups of 64 the halves exchange dwords (0, 1 of the upper lanes
// against 2, 3 of the lower), within groups of 32 the quarters too (a 4 x 4
// transpose).  MFMA i then takes, in quarter q, the k from quarter_k(q) +
// mfma_k(i) of the step on.
template <Fmt F>
__device__ __forceinline__ void arrange_codes(u32x4& v) {
  if constexpr (F == Fmt::kW4g128) return;
  auto a = __builtin_amdgcn_permlane32_swap(v.x, v.z, false, false);
  auto b = __builtin_amdgcn_permlane32_swap(v.y, v.w, false, false);
  if constexpr (F == Fmt::kW4g64) {
    v.x = a[0];
    v.y = b[0];
    v.z = a[1];
    v.w = b[1];
  } else {
    auto c = __builtin_amdgcn_permlane16_swap(a[0], b[0], false, false);
    auto d = __builtin_amdgcn_permlane16_swap(a[1], b[1], false, false);
    v.x = c[0];
    v.y = c[1];
    v.z = d[0];
    v.w = d[1];
  }
}
template <Fmt F> __device__ __forceinline__ int quarter_k(int q) {
  if constexpr (F == Fmt::kW4g128) return 32 * q;
  else if constexpr (F == Fmt::kW4g64) return 32 * (q & 1) + 16 * (q >> 1);
  else return lane_k(F) < 8 ? 4 * q : 8 * q;   // 4-bit groups of 32, bf16; float32
}
template <Fmt F> constexpr int mfma_k(int i) {
  return F == Fmt::kW4g128 ? 8 * i : F == Fmt::kW4g64 ? 8 * (i & 1) + 64 * (i >> 1) : 32 * i;
}

// Scales of a step: a lane loads the one of its own 32 k; o[g]: that of the
// step's group g in every lane of the row.
template <Fmt F>
__device__ __forceinline__ void spread_scales(uint32_t v, uint32_t (&o)[4]) {
  o[0] = v;
  if constexpr (F == Fmt::kW4g128) return;
  auto h = __builtin_amdgcn_permlane32_swap(v, v, false, false);
  if constexpr (F == Fmt::kW4g64) {
    o[0] = h[0];
    o[1] = h[1];
  } else {
    auto a = __builtin_amdgcn_permlane16_swap(h[0], h[0], false, false);
    auto b = __builtin_amdgcn_permlane16_swap(h[1], h[1], false, false);
    o[0] = a[0];
    o[1] = a[1];
    o[2] = b[0];
    o[3] = b[1];
  }
}

// ------------------------------------------------------------- streaming --
// acc[j][r] += A rows of tile j times the 16 rows of W tile r over steps
// [s0, s1) (of a matrix with K columns), for the first ntile tiles.
// a: activations; aoff[j] the byte offset of the lane's row (lane % 16) of tile
// j, or kOut for an empty row.  U steps are loaded together.
// 4-bit: sum (q - z) x over a group is sum (128 + q) x - sum 136 x + (8 - z)
// sum x.  The products are exact in float32; the middle sum depends on the
// activations alone, is formed once for all RT tiles and starts the first; the
// last takes it times -(8 - z) / 136.  kOrdered: the activations are stored in
// code_order.
template <Fmt F, int NT, int RT, int U, bool kOrdered, bool kZ>
__device__ __forceinline__ void stream_rows(floatx4 (&acc)[NT][RT], const WRows& wr,
                                            __amdgpu_buffer_rsrc_t a, const uint32_t (&arow)[NT], int ntile, int s0,
                                            int s1, int K, int lane) {
  constexpr int kK = step_k(F), kA = acts(F);
  constexpr uint32_t kXe = F == Fmt::kF32 ? 4 : 2;   // bytes of an activation
  const int q = lane >> 4;
  const int kend = min(K, s1 * kK);
  const uint32_t xq = static_cast<uint32_t>(quarter_k<F>(q)) * kXe;
  uint32_t base = 0;
  u32x4 neg = {0xc308c308u, 0xc308c308u, 0xc308c308u, 0xc308c308u};   // -136
  if constexpr (is_w4(F)) base = code_base();
  for (int sb = s0; sb < s1; sb += U) {
    u32x4 w[U][RT];
    uint32_t sc[U][RT], zc[U][RT];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int s = sb + u;
      const bool in = s * kK + q * lane_k(F) < kend;
#pragma unroll
      for (int r = 0; r < RT; ++r) {
        w[u][r] = load16(wr.w, in ? (s & 1 ? wr.voff[1] : wr.voff[0]) + r * wr.tile : kOut,
                         static_cast<uint32_t>(s >> 1) * wr.pair);
        if constexpr (is_w4(F)) {
          const uint32_t gi = wr.srow + r * wr.stile + (static_cast<uint32_t>(s * kK + q * 32) >> group_shift(F));
          sc[u][r] = static_cast<uint16_t>(
              __builtin_amdgcn_raw_buffer_load_b16(wr.s, static_cast<int>(in ? gi * 2u : kOut), 0, 0));
          if constexpr (kZ)
            zc[u][r] = static_cast<uint8_t>(
                __builtin_amdgcn_raw_buffer_load_b8(wr.z, static_cast<int>(in ? gi : kOut), 0, 0));
        }
      }
    }
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      if (NT > 1 && j >= ntile) break;
      if constexpr (NT > 1) __builtin_amdgcn_sched_barrier(0);   // one tile's activations at a time: registers
      u32x4 x[U][kA];
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int g = 0; g < kA; ++g) {
          const int k0 = (sb + u) * kK + (is_w4(F) ? mfma_k<F>(g) : 0);
          const bool in = is_w4(F) ? k0 < kend : k0 + q * lane_k(F) < kend;
          x[u][g] = load16(a, in ? arow[j] + xq : kOut, static_cast<uint32_t>(k0) * kXe);
        }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if constexpr (F == Fmt::kF32) {
          const floatx4 xv = __builtin_bit_cast(floatx4, x[u][0]);
#pragma unroll
          for (int r = 0; r < RT; ++r) {
            const floatx4 wv = __builtin_bit_cast(floatx4, w[u][r]);
#pragma unroll
            for (int i = 0; i < 4; ++i) acc[j][r] = __builtin_amdgcn_mfma_f32_16x16x4f32(xv[i], wv[i], acc[j][r], 0, 0, 0);
          }
        } else if constexpr (F == Fmt::kBf16) {
#pragma unroll
          for (int r = 0; r < RT; ++r)
            acc[j][r] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, x[u][0]),
                                                                __builtin_bit_cast(bf16x8, w[u][r]), acc[j][r], 0, 0, 0);
        } else {
          __builtin_amdgcn_sched_barrier(0);
          constexpr int kG = 128 >> group_shift(F), kPer = 4 / kG;   // groups of a step, MFMAs of a group
          floatx4 n136[kG];
#pragma unroll
          for (int g = 0; g < kG; ++g) {
            n136[g] = floatx4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int i = 0; i < kPer; ++i) {
              u32x4& xv = x[u][g * kPer + i];
              if constexpr (!kOrdered) xv = to_code_order(xv);
              n136[g] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, xv),
                                                                __builtin_bit_cast(bf16x8, neg), n136[g], 0, 0, 0);
            }
          }
#pragma unroll
          for (int r = 0; r < RT; ++r) {
            if constexpr (RT > 1) __builtin_amdgcn_sched_barrier(0);
            u32x4 c = w[u][r];
            // with several tiles the codes are unpacked anew for each: kept
            // unpacked they would take four times the registers
            uint32_t sv = sc[u][r];
            if constexpr (NT > 1) __asm__ volatile("" : "+v"(c.x), "+v"(c.y), "+v"(c.z), "+v"(c.w), "+v"(sv));
            arrange_codes<F>(c);
            uint32_t sg[4], zg[4];
            spread_scales<F>(sv, sg);
            if constexpr (kZ) spread_scales<F>(zc[u][r], zg);
#pragma unroll
            for (int g = 0; g < kG; ++g) {
              floatx4 t = n136[g];
#pragma unroll
              for (int i = 0; i < kPer; ++i)
                t = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, x[u][g * kPer + i]),
                                                            codes_to_bf16(c[g * kPer + i], base), t, 0, 0, 0);
              const float s = __uint_as_float(sg[g] << 16);
              if constexpr (kZ) {
                const float zf = static_cast<float>(zg[g] & 15u) * (1.f / 136.f) - 8.f / 136.f;
#pragma unroll
                for (int i = 0; i < 4; ++i) t[i] = fmaf(zf, n136[g][i], t[i]);
              }
#pragma unroll
              for (int i = 0; i < 4; ++i) acc[j][r][i] = fmaf(s, t[i], acc[j][r][i]);
            }
          }
        }
      }
    }
  }
}

}  // namespace moe
