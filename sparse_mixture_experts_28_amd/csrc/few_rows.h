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

constexpr uint32_t kOut = 0x7ffffff0u;   // an offset past every range used here: the load returns zero

__device__ __forceinline__ int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }

__device__ __forceinline__ u32x4 load16(__amdgpu_buffer_rsrc_t r, uint32_t voff, uint32_t soff) {
  return __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(r, static_cast<int>(voff),
                                                                         static_cast<int>(soff), 0));
}

// Weight formats; 4-bit codes by their group, without and with zero points.
enum class Fmt { kF32, kBf16, kW4g32, kW4g64, kW4g128, kW4g32z, kW4g64z, kW4g128z };
constexpr bool is_w4(Fmt f) { return f != Fmt::kF32 && f != Fmt::kBf16; }
constexpr bool has_zeros(Fmt f) { return f == Fmt::kW4g32z || f == Fmt::kW4g64z || f == Fmt::kW4g128z; }
constexpr int group_shift(Fmt f) {
  return f == Fmt::kW4g32 || f == Fmt::kW4g32z ? 5 : f == Fmt::kW4g64 || f == Fmt::kW4g64z ? 6 : 7;
}
// k of one step (all four quarters) and of one lane's 16-byte load
constexpr int step_k(Fmt f) { return f == Fmt::kF32 ? 16 : f == Fmt::kBf16 ? 32 : 128; }
constexpr int lane_k(Fmt f) { return step_k(f) / 4; }
constexpr int acts(Fmt f) { return is_w4(f) ? 4 : 1; }        // 16-byte activation loads per lane and step
constexpr int act_bytes(Fmt f) { return f == Fmt::kF32 ? 4 : 2; }

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
  int slack;                     // 4-bit: scales from the last row's first to the array's end
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
    // the rest of the array, as far as 32 bits go: a batch's load may reach past
    // the rows' scales, and a word cut by the end of the range would read as zero
    const long long rest = (m.scales - row0 * ng) < (1ll << 28) ? m.scales - row0 * ng : 1ll << 28;
    o.s = make_rsrc(m.s + row0 * ng, static_cast<uint32_t>(rest) * 2u);
    o.z = o.s;
    if (has_zeros(F)) o.z = make_rsrc(m.z + row0 * ng, static_cast<uint32_t>(rest));
    o.slack = m.whole ? 0x7fffffff : static_cast<int>(rest - static_cast<long long>(left - 1) * ng);
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
    o.slack = 0;
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
  if constexpr (group_shift(F) == 7) return;
  auto a = __builtin_amdgcn_permlane32_swap(v.x, v.z, false, false);
  auto b = __builtin_amdgcn_permlane32_swap(v.y, v.w, false, false);
  if constexpr (group_shift(F) == 6) {
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
  if constexpr (!is_w4(F)) return lane_k(F) * q;
  else if constexpr (group_shift(F) == 7) return 32 * q;
  else if constexpr (group_shift(F) == 6) return 32 * (q & 1) + 16 * (q >> 1);
  else return 8 * q;
}
template <Fmt F> constexpr int mfma_k(int i) {
  return !is_w4(F) ? 0 : group_shift(F) == 7 ? 8 * i : group_shift(F) == 6 ? 8 * (i & 1) + 64 * (i >> 1) : 32 * i;
}

// ---------------------------------------------------------------- a batch --
// The weights of U steps from step s0 (a multiple of U) on, k < kend.  4-bit:
// with the batch's scales, two to a word, and zero points, four to a word, in
// every lane of their row, by loads as wide as they come, at any 2-byte (zero
// points: 1-byte) address (one 2-byte load per step cost 3 to 5 us of a 23 us
// phase).  One by one only where the array's end could cut a word of a row that
// is there: in the last batch of the last rows, where K / group is no multiple of
// four.
template <Fmt F, int RT, int U> struct WBatch {
  static constexpr int kS = is_w4(F) ? U << (7 - group_shift(F)) : 2;   // scales of a row and batch
  static_assert(kS >= 2 && kS <= 16, "whole words of scales");
  u32x4 w[U][RT];
  uint32_t sc[RT][kS / 2], zc[RT][(kS + 3) / 4];

  template <int N>
  static __device__ __forceinline__ void words(uint32_t (&o)[N], __amdgpu_buffer_rsrc_t r, uint32_t off) {
    typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
    if constexpr (N == 1) {
      o[0] = __builtin_amdgcn_raw_buffer_load_b32(r, static_cast<int>(off), 0, 0);
    } else if constexpr (N == 2) {
      const u32x2 v = __builtin_bit_cast(u32x2, __builtin_amdgcn_raw_buffer_load_b64(r, static_cast<int>(off), 0, 0));
      o[0] = v.x;
      o[1] = v.y;
    } else {
#pragma unroll
      for (int i = 0; i < N; i += 4) {
        const u32x4 v = load16(r, off + 4u * i, 0);
        o[i] = v.x;
        o[i + 1] = v.y;
        o[i + 2] = v.z;
        o[i + 3] = v.w;
      }
    }
  }

  __device__ __forceinline__ void load(const WRows& wr, int s0, int kend, int q) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int s = s0 + u;
      const bool in = s * step_k(F) + q * lane_k(F) < kend;
      const uint32_t vo = s & 1 ? wr.voff[1] : wr.voff[0];
#pragma unroll
      for (int r = 0; r < RT; ++r)
        w[u][r] = load16(wr.w, in ? vo + r * wr.tile : kOut, static_cast<uint32_t>(s >> 1) * wr.pair);
    }
    if constexpr (is_w4(F)) {
      const uint32_t g0 = static_cast<uint32_t>(s0) << (7 - group_shift(F));
#pragma unroll
      for (int r = 0; r < RT; ++r) {
        const uint32_t gi = wr.srow + r * wr.stile + g0;
        if (static_cast<int>(g0) + kS <= wr.slack) {
          words(sc[r], wr.s, gi * 2u);
          if constexpr (has_zeros(F)) {
            if constexpr (kS == 2) zc[r][0] = static_cast<uint16_t>(__builtin_amdgcn_raw_buffer_load_b16(wr.z, static_cast<int>(gi), 0, 0));
            else words(zc[r], wr.z, gi);
          }
        } else {
#pragma unroll
          for (int i = 0; i < kS; ++i) {
            const uint32_t v = static_cast<uint16_t>(
                __builtin_amdgcn_raw_buffer_load_b16(wr.s, static_cast<int>((gi + i) * 2u), 0, 0));
            sc[r][i / 2] = i % 2 ? sc[r][i / 2] | (v << 16) : v;
          }
          if constexpr (has_zeros(F)) {
#pragma unroll
            for (int i = 0; i < kS; ++i) {
              const uint32_t v = static_cast<uint8_t>(
                  __builtin_amdgcn_raw_buffer_load_b8(wr.z, static_cast<int>(gi + i), 0, 0));
              zc[r][i / 4] = i % 4 ? zc[r][i / 4] | (v << (8 * (i % 4))) : v;
            }
          }
        }
      }
    }
  }
};

// ----------------------------------------------------------------- a step --
// Products of step u of a batch.  x[j]: the lane's activations of the step for
// tile j.  live(g): all ones where group g of the step lies below the end of
// k, else zero (the batch may hold a neighbouring row's scales there).
// 4-bit: sum (q - z) x over a group is sum (128 + q) x - sum 136 x + (8 - z)
// sum x.  The products are exact in float32; the middle sum depends on the
// activations alone, is formed once for all RT tiles and starts the first; the
// last takes it times -(8 - z) / 136.
template <Fmt F, int NT, int RT, int U, typename Live>
__device__ __forceinline__ void multiply_step(floatx4 (&acc)[NT][RT], const WBatch<F, RT, U>& b, int u,
                                              const u32x4 (&x)[NT][acts(F)], Live live) {
  if constexpr (F == Fmt::kF32) {
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      const floatx4 xv = __builtin_bit_cast(floatx4, x[j][0]);
#pragma unroll
      for (int r = 0; r < RT; ++r) {
        const floatx4 wv = __builtin_bit_cast(floatx4, b.w[u][r]);
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[j][r] = __builtin_amdgcn_mfma_f32_16x16x4f32(xv[i], wv[i], acc[j][r], 0, 0, 0);
      }
    }
  } else if constexpr (F == Fmt::kBf16) {
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
      for (int r = 0; r < RT; ++r)
        acc[j][r] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, x[j][0]),
                                                            __builtin_bit_cast(bf16x8, b.w[u][r]), acc[j][r], 0, 0, 0);
  } else {
    constexpr int kG = 128 >> group_shift(F), kPer = 4 / kG;   // groups of a step, MFMAs of a group
    const uint32_t base = code_base();
    const u32x4 neg = {0xc308c308u, 0xc308c308u, 0xc308c308u, 0xc308c308u};   // -136
    floatx4 n136[NT][kG];
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
      for (int g = 0; g < kG; ++g) {
        n136[j][g] = floatx4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int i = 0; i < kPer; ++i)
          n136[j][g] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, x[j][g * kPer + i]),
                                                               __builtin_bit_cast(bf16x8, neg), n136[j][g], 0, 0, 0);
      }
#pragma unroll
    for (int r = 0; r < RT; ++r) {
      u32x4 c = b.w[u][r];
      arrange_codes<F>(c);
      floatx4 t[NT][kG];   // the groups' products are independent: all are under way before the first is used
#pragma unroll
      for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int g = 0; g < kG; ++g) t[j][g] = n136[j][g];
#pragma unroll
      for (int i = 0; i < kPer; ++i)
#pragma unroll
        for (int g = 0; g < kG; ++g) {
          const bf16x8 cv = codes_to_bf16(c[g * kPer + i], base);
#pragma unroll
          for (int j = 0; j < NT; ++j)
            t[j][g] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, x[j][g * kPer + i]), cv, t[j][g], 0, 0, 0);
        }
#pragma unroll
      for (int g = 0; g < kG; ++g) {
        const int si = u * kG + g;
        const uint32_t sw = si % 2 ? b.sc[r][si / 2] & 0xffff0000u : b.sc[r][si / 2] << 16;
        const float s = __uint_as_float(sw & live(g));
        float zf = 0.f;
        if constexpr (has_zeros(F))
          zf = static_cast<float>((b.zc[r][si / 4] >> (8 * (si % 4))) & 15u) * (1.f / 136.f) - 8.f / 136.f;
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            if constexpr (has_zeros(F)) t[j][g][i] = fmaf(zf, n136[j][g][i], t[j][g][i]);
            acc[j][r][i] = fmaf(s, t[j][g][i], acc[j][r][i]);
          }
      }
      // the sums stay here: moved behind the loop's branches, they would keep
      // every group's products in registers until then
#pragma unroll
      for (int j = 0; j < NT; ++j) __asm__ volatile("" : "+v"(acc[j][r]));
    }
  }
}

// -------------------------------------------------------------- a segment --
// A wave's share of a product: W rows (WRows), steps [s0, s1) of them (s0 a
// multiple of U), and `slots` rows of activations.
//
// The activations go through LDS of the wave's own (no barriers).  Most rows of
// an operand are empty when an expert has one or two tokens: read for every step
// by the lanes that need them, the few rows would take as many load instructions
// as the weights; staged, a row's bytes are read once, densely.  Slot i of the
// region holds a chunk of steps of row i, padded by 16 bytes so that neighbouring
// rows start in different banks; the region's last stage_zero bytes are zero: what
// the lanes read for steps past the last.
//
// begin() issues the first loads, run() does the rest: called before the work
// that ends the segment before (sums across waves, activation, stores), begin()
// keeps the memory busy meanwhile.  kAhead: run() loads a batch ahead of its
// products too (registers for one more batch).
constexpr int stage_zero(Fmt f) { return is_w4(f) ? 2 * mfma_k<Fmt::kW4g32>(3) + 16 : 16; }   // a lane's reads of a step

template <Fmt F, int RT, int U, bool kAhead, bool kOrdered, int SLOTS, int STAGE> struct Stream {
  static constexpr int kStageZero = stage_zero(F);
  static constexpr int kStep = step_k(F) * act_bytes(F);     // activation bytes of a step and row
  static constexpr int kLoads = (STAGE - kStageZero + 1023) / 1024;
  static constexpr bool kDense = SLOTS * (U * kStep + 16) + kStageZero > STAGE;   // a chunk may be shorter than a batch
  static_assert(STAGE % 16 == 0 && STAGE >= SLOTS * (kStep + 16) + kStageZero, "one step of all rows fits");

  WRows wr;
  WBatch<F, RT, U> w;
  u32x4 xv[kLoads];
  uint32_t xo[kLoads];
  int s0, s1, kend, slots, cs;

  static __device__ __forceinline__ void clear(char* stage, int lane) {
    if (lane < kStageZero / 4) reinterpret_cast<int*>(stage + STAGE - kStageZero)[lane] = 0;
  }

  // the chunk of activations from step c0 on: slot i at xo[..] = soff(i) + .. bytes of a
  __device__ __forceinline__ void load_x(__amdgpu_buffer_rsrc_t a, int c0, int lane) {
    constexpr int kUnits = kStep == 64 ? 2 : 4;              // log2 of a step's 16-byte units
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      const int at = c0 * kStep + (((i * 64 + lane) & ((1 << (cs + kUnits)) - 1)) << 4);
      xv[i] = load16(a, at < kend * act_bytes(F) ? xo[i] : kOut, static_cast<uint32_t>(c0) * kStep);
    }
  }
  __device__ __forceinline__ void store_x(char* stage, int lane) {
    constexpr int kUnits = kStep == 64 ? 2 : 4;
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      const int unit = i * 64 + lane, slot = unit >> (cs + kUnits);
      if (slot < slots)
        *reinterpret_cast<u32x4*>(stage + slot * ((kStep << cs) + 16) + ((unit & ((1 << (cs + kUnits)) - 1)) << 4)) = xv[i];
    }
  }

  template <typename SlotOff>
  __device__ __forceinline__ void begin(const WRows& rows, __amdgpu_buffer_rsrc_t a, SlotOff soff, int nslots, int first,
                                        int last, int K, int lane) {
    wr = rows;
    slots = nslots;
    s0 = first;
    s1 = last;
    kend = min(K, s1 * step_k(F));
    cs = 0;   // log2 of a chunk's steps: as many as fit
    while (slots * ((kStep << (cs + 1)) + 16) <= STAGE - kStageZero && cs < 10) ++cs;
    if (s0 >= s1) return;
    constexpr int kUnits = kStep == 64 ? 2 : 4;
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      const int unit = i * 64 + lane, slot = unit >> (cs + kUnits);
      xo[i] = slot < slots ? soff(slot) + ((unit & ((1 << (cs + kUnits)) - 1)) << 4) : kOut;
    }
    load_x(a, s0, lane);
    w.load(wr, s0, kend, lane >> 4);
  }

  // acc[j][r] += rows of tile j times the 16 rows of W tile r; rslot[j]: slot of
  // the lane's row (lane % 16) of tile j (any, if the row is empty: its sums are
  // not read)
  template <int NT>
  __device__ __forceinline__ void run(floatx4 (&acc)[NT][RT], __amdgpu_buffer_rsrc_t a, const int (&rslot)[NT],
                                      char* stage, int lane) {
    if (s0 < s1) {
      const int q = lane >> 4, steps = 1 << cs;
      const char* zero = stage + STAGE - kStageZero;
      const char* xrow[NT];
#pragma unroll
      for (int j = 0; j < NT; ++j)
        xrow[j] = stage + rslot[j] * ((kStep << cs) + 16) + quarter_k<F>(q) * act_bytes(F);
      store_x(stage, lane);
      int cb = s0;
      for (int s = s0;;) {
        WBatch<F, RT, U> ready;
        if constexpr (kAhead) {
          ready = w;
          if (s + U < s1) w.load(wr, s + U, kend, q);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
          if ((u == 0 || kDense) && s + u >= cb + steps && s + u < s1) {
            cb = s + u;
            load_x(a, cb, lane);
            store_x(stage, lane);
          }
          u32x4 x[NT][acts(F)];
#pragma unroll
          for (int j = 0; j < NT; ++j) {
            const char* at = s + u < s1 ? xrow[j] + (s + u - cb) * kStep : zero;
#pragma unroll
            for (int g = 0; g < acts(F); ++g) {
              x[j][g] = *reinterpret_cast<const u32x4*>(at + mfma_k<F>(g) * act_bytes(F));
              if constexpr (is_w4(F) && !kOrdered) x[j][g] = to_code_order(x[j][g]);
            }
          }
          multiply_step<F, NT, RT, U>(acc, kAhead ? ready : w, u, x, [&](int g) {
            return (s + u) * step_k(F) + (g << group_shift(F)) < kend ? 0xffffffffu : 0u;
          });
        }
        s += U;
        if (s >= s1) break;
        if constexpr (!kAhead) w.load(wr, s, kend, q);
      }
    }
    // Wait states between the last products and whatever reads them, placed by
    // hand: where a uniform branch separated an MFMA from its reader, hipcc has
    // been seen to leave them out on the taken side.  For the same reason no
    // branch depends on the number of tiles between products.
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
      for (int r = 0; r < RT; ++r) __asm__ volatile("s_nop 15" : "+v"(acc[j][r]));
  }
};

}  // namespace moe
