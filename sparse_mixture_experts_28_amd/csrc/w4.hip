// 4-bit weights with group scales: the quantizer, its inverse and the Linear of a
// few rows.
//
//   w[n, k] = s[n, g] (q[n, k] - z[n, g]),  g = k / group,  q in 0..15
//
// q two to a byte along k (even k in the low nibble), s bf16, z uint8 or 8.
#include "few_rows.h"

namespace moe {
namespace {

// ---------------------------------------------------------------- quantize --
// A lane takes 8 consecutive elements, a group is group / 8 neighbouring lanes.
// Magnitudes are compared as integers (the same order, and an infinity or NaN
// comes out on top).  Maxima over 4, 8 or 16 lanes by row moves: lane ^ 1, lane ^
// 2, then the mirrors, which after the first two pair the same partial results as
// lane ^ 4 and lane ^ 8.
template <int CTRL>
__device__ __forceinline__ int dpp_max(int v) {
  return max(v, __builtin_amdgcn_mov_dpp(v, CTRL, 0xF, 0xF, false));
}
template <int LANES>
__device__ __forceinline__ int group_max(int v) {
  v = dpp_max<0xB1>(v);
  v = dpp_max<0x4E>(v);
  if constexpr (LANES >= 8) v = dpp_max<0x141>(v);
  if constexpr (LANES >= 16) v = dpp_max<0x140>(v);
  return v;
}

// round(v / s) for a bf16 s > 0 and a bf16 v of at most a few times s, ties to
// even, as exact arithmetic rounds it.  s = m 2^e with m in [1/2, 1), r ~ 1 / m:
// the corrected quotient is within a few units in its last place, and exact where
// the quotient is a float32 number; two 8-bit significands have no quotient within
// 2^-9 of a tie k + 1/2 that is not the tie.  (The division of the library takes
// three times the instructions.)
__device__ __forceinline__ float round_quotient(float v, float m, float r, int e) {
  const float n = ldexpf(v, -e);
  float q = n * r;
  q = fmaf(fmaf(-q, m, n), r, q);
  return rintf(q);
}

template <int GSHIFT, bool ZERO>
__device__ __forceinline__ void quantize8(u32x4 raw, long long i, uint32_t* codes, uint16_t* scales, uint8_t* zeros) {
  constexpr int kLanes = 1 << (GSHIFT - 3);
  constexpr int kInf = 0x7f800000;
  int v[8];   // the elements' float32 bits
#pragma unroll
  for (int m = 0; m < 4; ++m) {
    v[2 * m] = static_cast<int>(raw[m] << 16);
    v[2 * m + 1] = static_cast<int>(raw[m] & 0xffff0000u);
  }
  int hi = 0, lo = 0;   // the largest v and the largest -v, at least 0; symmetric: hi of both
#pragma unroll
  for (int m = 0; m < 8; ++m) {
    if constexpr (ZERO) {
      hi = max(hi, v[m]);
      lo = max(lo, v[m] ^ static_cast<int>(0x80000000u));
    } else {
      hi = max(hi, v[m] & 0x7fffffff);
    }
  }
  hi = group_max<kLanes>(hi);
  if constexpr (ZERO) lo = group_max<kLanes>(lo);
  uint16_t sb;
  if constexpr (ZERO) {
    // the quotient by 15 in float64, corrected as above
    const double d = static_cast<double>(__int_as_float(hi)) + static_cast<double>(__int_as_float(lo));
    double q = d * (1.0 / 15.0);
    q = fma(fma(-q, 15.0, d), 1.0 / 15.0, q);
    sb = f32_to_bf16(static_cast<float>(q));
  } else {
    sb = f32_to_bf16(__int_as_float(hi) / 7.f);
  }
  if (hi >= kInf || lo >= kInf) sb = 0x7fc0;   // a group with an infinity or NaN has no scale
  const float s = bf16_to_f32(sb);
  const bool fine = s > 0.f;      // false: all zero (or too small for a scale), or NaN
  int e;
  const float m2 = frexpf(fine ? s : 1.f, &e);
  const float r = __builtin_amdgcn_rcpf(m2);
  float z = 8.f;
  if constexpr (ZERO) z = fine ? fminf(round_quotient(__int_as_float(lo), m2, r, e), 15.f) : 0.f;
  uint32_t c = 0;
#pragma unroll
  for (int m = 0; m < 8; ++m) {
    const float q = fminf(fmaxf(round_quotient(__int_as_float(v[m]), m2, r, e) + z, 0.f), 15.f);
    c |= static_cast<uint32_t>(fine ? q : z) << (4 * m);
  }
  codes[i] = c;
  if ((threadIdx.x & (kLanes - 1)) == 0) {
    const long long g = i >> (GSHIFT - 3);
    scales[g] = sb;
    if constexpr (ZERO) zeros[g] = static_cast<uint8_t>(z);
  }
}

// Two runs of 8 elements a thread, both loaded first.  n8 is a multiple of the
// lanes of a group, so a group is in or out as a whole.  Bound by memory and, with
// zero points, its operations: 2048 x 7168 in groups of 128 10 us (37 MB, 3.8 TB/s);
// 8 x 1001 x 4096 in groups of 32 with zero points 19 us (85 MB, 4.4 TB/s).
template <int GSHIFT, bool ZERO>
__global__ __launch_bounds__(256) void w4_quantize_kernel(const uint16_t* src, long long n8, uint32_t* codes,
                                                          uint16_t* scales, uint8_t* zeros) {
  const long long stride = static_cast<long long>(gridDim.x) * 512;
  for (long long i = static_cast<long long>(blockIdx.x) * 512 + threadIdx.x; i < n8; i += stride) {
    const u32x4 a = reinterpret_cast<const u32x4*>(src)[i];
    const bool two = i + 256 < n8;
    u32x4 b = {0u, 0u, 0u, 0u};
    if (two) b = reinterpret_cast<const u32x4*>(src)[i + 256];
    quantize8<GSHIFT, ZERO>(a, i, codes, scales, zeros);
    if (two) quantize8<GSHIFT, ZERO>(b, i + 256, codes, scales, zeros);
  }
}

// -------------------------------------------------------------- dequantize --
// s (q - z): 8 bits times at most 5, exact in float32, one rounding to bf16.  Bound
// by its writes: 148 MB read and written in 25 us (5.9 TB/s).
__global__ __launch_bounds__(256) void w4_dequantize_kernel(const uint32_t* codes, const uint16_t* scales,
                                                            const uint8_t* zeros, long long n8, int gshift,
                                                            uint16_t* dst) {
  const long long stride = static_cast<long long>(gridDim.x) * blockDim.x;
  for (long long i = static_cast<long long>(blockIdx.x) * blockDim.x + threadIdx.x; i < n8; i += stride) {
    const uint32_t c = codes[i];
    const long long g = i >> (gshift - 3);
    const float s = bf16_to_f32(scales[g]);
    const int z = zeros != nullptr ? zeros[g] & 15 : 8;
    u32x4 o;
#pragma unroll
    for (int m = 0; m < 4; ++m) {
      const float a = s * static_cast<float>(static_cast<int>((c >> (8 * m)) & 15u) - z);
      const float b = s * static_cast<float>(static_cast<int>((c >> (8 * m + 4)) & 15u) - z);
      o[m] = static_cast<uint32_t>(f32_to_bf16(a)) | (static_cast<uint32_t>(f32_to_bf16(b)) << 16);
    }
    reinterpret_cast<u32x4*>(dst)[i] = o;
  }
}

// ------------------------------------------------------------------ Linear --
// y[m, n] = sum_k x[m, k] w[n, k] + b[n] for up to 16 rows.  One workgroup per 16
// columns; its waves split k and add their sums in LDS in wave order.  One row, N
// 4096, K 14336, groups of 128: 11 us a call (30 MB, 4.8 us at the memory's rate: a
// launch, and a wave's 3 to 4 batches one load latency each).
template <Fmt F, int U, int NW, int STAGE>
__global__ __launch_bounds__(NW * 64) void w4_linear_kernel(const uint16_t* x, WMat w, const uint16_t* bias,
                                                            uint16_t* y, int M) {
  // the waves' activation regions, then their sums
  static_assert(STAGE >= 1024, "a wave's sums fit its region");
  __shared__ __attribute__((aligned(16))) char lds[NW * STAGE];
  float* red = reinterpret_cast<float*>(lds);
  const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
  const int n0 = blockIdx.x * 16;
  const uint32_t pitch = static_cast<uint32_t>(w.K) * 2u;
  const __amdgpu_buffer_rsrc_t xr = make_rsrc(x, static_cast<uint32_t>(M) * pitch);
  char* mine = lds + wave * STAGE;
  using St = Stream<F, 1, U, true, false, 16, STAGE>;
  St::clear(mine, lane);
  const int nst = (w.K + 127) / 128, nb = (nst + U - 1) / U;
  const int s0 = wave * nb / NW * U, s1 = min(nst, (wave + 1) * nb / NW * U);
  auto soff = [&](int slot) { return static_cast<uint32_t>(slot) * pitch; };
  St st;
  st.begin(rows_of<F, 1>(w, 0, n0, lane), xr, soff, M, s0, s1, w.K, lane);
  floatx4 acc[1][1] = {{floatx4{0.f, 0.f, 0.f, 0.f}}};
  const int rslot[1] = {min(lane & 15, M - 1)};
  st.run(acc, xr, rslot, mine, lane);
  __syncthreads();
  *reinterpret_cast<floatx4*>(red + (wave * 64 + lane) * 4) = acc[0][0];
  __syncthreads();
  // result (row p, column n): lane (n, p / 4), register p % 4
  const int n = threadIdx.x & 15, p = threadIdx.x >> 4;
  if (p < M && p < 16 && n0 + n < w.N) {
    const float* s = red + ((p >> 2) * 16 + n) * 4 + (p & 3);
    float v = 0.f;
#pragma unroll
    for (int q = 0; q < NW; ++q) v += s[q * 256];
    if (bias != nullptr) v += bf16_to_f32(bias[n0 + n]);
    y[static_cast<size_t>(p) * w.N + n0 + n] = f32_to_bf16(v);
  }
}

// The same for 17 to 64 rows: every step's activations are dense, so they come
// straight from memory (L2) into operand registers, a tile of 16 rows at a time and
// the next tile's ahead of the products; a step's codes are unpacked once for all
// tiles.  A workgroup takes 16 RT columns of up to 64 rows and splits k over its
// waves: each activation is read once per workgroup.  37 rows, 14335 columns, K =
// 4096, groups of 32 with zero points: 27 us; the activations staged in LDS as for
// fewer rows 47 to 74.  Bound by the vector operations on the group sums (half of
// its time) and their waits.
template <Fmt F, int NT, int RT, int NW>
__global__ __launch_bounds__(NW * 64) void w4_linear_rows_kernel(const uint16_t* x, WMat w, const uint16_t* bias,
                                                                 uint16_t* y, int M) {
  constexpr int U = group_shift(F) == 7 ? 2 : 1;   // steps of a batch of weights: whole words of scales
  constexpr int kG = 128 >> group_shift(F), kPer = 4 / kG;
  __shared__ float red[NW][RT * 256];
  const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6), q = lane >> 4;
  const int n0 = blockIdx.x * 16 * RT, m0 = blockIdx.y * 64;
  const int rows = min(M - m0, 16 * NT);
  const uint32_t pitch = static_cast<uint32_t>(w.K) * 2u;
  const __amdgpu_buffer_rsrc_t xr =
      make_rsrc(x + static_cast<size_t>(m0) * w.K, static_cast<uint32_t>(rows) * pitch);
  const uint32_t xq = static_cast<uint32_t>(quarter_k<F>(q)) * 2u;
  uint32_t xo[NT];
  floatx4 acc[NT][RT];
#pragma unroll
  for (int j = 0; j < NT; ++j) {
    const int p = j * 16 + (lane & 15);
    xo[j] = p < rows ? static_cast<uint32_t>(p) * pitch + xq : kOut;
#pragma unroll
    for (int r = 0; r < RT; ++r) acc[j][r] = floatx4{0.f, 0.f, 0.f, 0.f};
  }
  const int nst = (w.K + 127) / 128, nb = (nst + U - 1) / U;
  const int s0 = wave * nb / NW * U, s1 = min(nst, (wave + 1) * nb / NW * U);
  const int kend = min(w.K, s1 * 128);
  const WRows wr = rows_of<F, RT>(w, 0, n0, lane);
  auto load_x = [&](u32x4 (&v)[4], int s, int j) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int k0 = s * 128 + mfma_k<F>(i);
      v[i] = load16(xr, k0 < kend ? xo[j] : kOut, static_cast<uint32_t>(k0) * 2u);
    }
  };
  const uint32_t base = code_base();
  const u32x4 neg = {0xc308c308u, 0xc308c308u, 0xc308c308u, 0xc308c308u};   // -136
  WBatch<F, RT, U> b;
  u32x4 xv[2][4];
  if (s0 < s1) {
    b.load(wr, s0, kend, q);
    load_x(xv[0], s0, 0);
  }
  for (int sb = s0; sb < s1; sb += U) {
    WBatch<F, RT, U> cur = b;
    if (sb + U < s1) b.load(wr, sb + U, kend, q);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int s = sb + u;
      bf16x8 cv[RT][4];
      float sc[RT][kG], zf[RT][kG];
#pragma unroll
      for (int r = 0; r < RT; ++r) {
        u32x4 c = cur.w[u][r];
        arrange_codes<F>(c);
#pragma unroll
        for (int i = 0; i < 4; ++i) cv[r][i] = codes_to_bf16(c[i], base);
#pragma unroll
        for (int g = 0; g < kG; ++g) {
          const int si = u * kG + g;
          const uint32_t sw = si % 2 ? cur.sc[r][si / 2] & 0xffff0000u : cur.sc[r][si / 2] << 16;
          sc[r][g] = s * 128 + (g << group_shift(F)) < kend ? __uint_as_float(sw) : 0.f;
          zf[r][g] = 0.f;
          if constexpr (has_zeros(F))
            zf[r][g] = static_cast<float>((cur.zc[r][si / 4] >> (8 * (si % 4))) & 15u) * (1.f / 136.f) - 8.f / 136.f;
        }
      }
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        const int at = j & 1;
        load_x(xv[at ^ 1], j + 1 < NT ? s : s + 1, j + 1 < NT ? j + 1 : 0);
        u32x4 xt[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) xt[i] = to_code_order(xv[at][i]);
#pragma unroll
        for (int g = 0; g < kG; ++g) {
          floatx4 n136 = {0.f, 0.f, 0.f, 0.f}, t[RT];
#pragma unroll
          for (int i = 0; i < kPer; ++i)
            n136 = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, xt[g * kPer + i]),
                                                           __builtin_bit_cast(bf16x8, neg), n136, 0, 0, 0);
#pragma unroll
          for (int r = 0; r < RT; ++r) t[r] = n136;
#pragma unroll
          for (int i = 0; i < kPer; ++i)
#pragma unroll
            for (int r = 0; r < RT; ++r)
              t[r] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, xt[g * kPer + i]),
                                                             cv[r][g * kPer + i], t[r], 0, 0, 0);
#pragma unroll
          for (int r = 0; r < RT; ++r) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              if constexpr (has_zeros(F)) t[r][i] = fmaf(zf[r][g], n136[i], t[r][i]);
              acc[j][r][i] = fmaf(sc[r][g], t[r][i], acc[j][r][i]);
            }
            __asm__ volatile("" : "+v"(acc[j][r]));   // no product waits behind the loop's branch (few_rows.h)
          }
        }
      }
      if constexpr (NT % 2 != 0) {   // the next step starts at xv[0] again
#pragma unroll
        for (int i = 0; i < 4; ++i) xv[0][i] = xv[1][i];
      }
    }
  }
#pragma unroll
  for (int j = 0; j < NT; ++j) {
    if (j * 16 >= rows) break;
#pragma unroll
    for (int r = 0; r < RT; ++r) *reinterpret_cast<floatx4*>(&red[wave][(r * 64 + lane) * 4]) = acc[j][r];
    __syncthreads();
    for (int i = threadIdx.x; i < RT * 256; i += NW * 64) {
      const int n = (i >> 8) * 16 + (i & 15), pr = (i >> 4) & 15;
      const int p = j * 16 + pr;
      if (p < rows && n0 + n < w.N) {
        float v = 0.f;
#pragma unroll
        for (int k = 0; k < NW; ++k) v += red[k][(i >> 8) * 256 + ((pr >> 2) * 16 + (i & 15)) * 4 + (pr & 3)];
        if (bias != nullptr) v += bf16_to_f32(bias[n0 + n]);
        y[static_cast<size_t>(m0 + p) * w.N + n0 + n] = f32_to_bf16(v);
      }
    }
    __syncthreads();
  }
}

// As few columns to a workgroup as still fit one round of 256 CUs.  Microseconds
// with RT = 1, 2, 4 (37 rows, groups of 128): N 4096 x K 14336 38, 43, 54; 14336 x
// 4096 43, 29, 20; 7168 x 2048 (groups of 64, zero points) 15, 11, 15.
template <Fmt F, int NT>
void launch_rows(const uint16_t* x, int M, const WMat& w, const uint16_t* bias, uint16_t* y, hipStream_t st) {
  const unsigned bm = (M + 63) / 64;
  const auto columns = [&](int rt) { return static_cast<unsigned>((w.N + 16 * rt - 1) / (16 * rt)); };
  if (columns(1) * bm <= 256) w4_linear_rows_kernel<F, NT, 1, 8><<<dim3(columns(1), bm), 512, 0, st>>>(x, w, bias, y, M);
  else if (columns(2) * bm <= 256) w4_linear_rows_kernel<F, NT, 2, 8><<<dim3(columns(2), bm), 512, 0, st>>>(x, w, bias, y, M);
  else w4_linear_rows_kernel<F, NT, 4, 8><<<dim3(columns(4), bm), 512, 0, st>>>(x, w, bias, y, M);
}
template <Fmt F>
hipError_t launch_linear(const uint16_t* x, int M, const WMat& w, const uint16_t* bias, uint16_t* y, hipStream_t st) {
  if (M <= 16)
    w4_linear_kernel<F, 4, 8, 4864><<<dim3((w.N + 15) / 16), 512, 0, st>>>(x, w, bias, y, M);
  else if (M <= 32) launch_rows<F, 2>(x, M, w, bias, y, st);
  else if (M <= 48) launch_rows<F, 3>(x, M, w, bias, y, st);
  else launch_rows<F, 4>(x, M, w, bias, y, st);
  return hipGetLastError();
}

int grid_of(long long n8) {
  const long long g = (n8 + 255) / 256;
  return static_cast<int>(g < 16384 ? g : 16384);
}

}  // namespace

hipError_t launch_w4_quantize(const uint16_t* src, long long n, int gshift, uint8_t* codes, uint16_t* scales,
                              uint8_t* zeros, hipStream_t st) {
  uint32_t* c = reinterpret_cast<uint32_t*>(codes);
  const long long n8 = n / 8;
  const int grid = grid_of((n8 + 1) / 2);
  if (gshift == 5 && zeros) w4_quantize_kernel<5, true><<<grid, 256, 0, st>>>(src, n8, c, scales, zeros);
  else if (gshift == 5) w4_quantize_kernel<5, false><<<grid, 256, 0, st>>>(src, n8, c, scales, zeros);
  else if (gshift == 6 && zeros) w4_quantize_kernel<6, true><<<grid, 256, 0, st>>>(src, n8, c, scales, zeros);
  else if (gshift == 6) w4_quantize_kernel<6, false><<<grid, 256, 0, st>>>(src, n8, c, scales, zeros);
  else if (zeros) w4_quantize_kernel<7, true><<<grid, 256, 0, st>>>(src, n8, c, scales, zeros);
  else w4_quantize_kernel<7, false><<<grid, 256, 0, st>>>(src, n8, c, scales, zeros);
  return hipGetLastError();
}

hipError_t launch_w4_dequantize(const uint8_t* codes, const uint16_t* scales, const uint8_t* zeros, long long n,
                                int gshift, uint16_t* dst, hipStream_t st) {
  w4_dequantize_kernel<<<grid_of(n / 8), 256, 0, st>>>(reinterpret_cast<const uint32_t*>(codes), scales, zeros, n / 8,
                                                      gshift, dst);
  return hipGetLastError();
}

hipError_t launch_w4_linear(const uint16_t* x, int M, const WMat& w, const uint16_t* bias, uint16_t* y,
                            hipStream_t st) {
  if (w.gshift == 5)
    return w.z ? launch_linear<Fmt::kW4g32z>(x, M, w, bias, y, st) : launch_linear<Fmt::kW4g32>(x, M, w, bias, y, st);
  if (w.gshift == 6)
    return w.z ? launch_linear<Fmt::kW4g64z>(x, M, w, bias, y, st) : launch_linear<Fmt::kW4g64>(x, M, w, bias, y, st);
  return w.z ? launch_linear<Fmt::kW4g128z>(x, M, w, bias, y, st) : launch_linear<Fmt::kW4g128>(x, M, w, bias, y, st);
}

}  // namespace moe
