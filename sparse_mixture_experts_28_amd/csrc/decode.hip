// The MoE layer for a few tokens (1..MOE_MAX_DECODE_TOKENS): one generation step
// of a served model.
//
//   out[t] = sum_j w[t,j] FFN_{e(t,j)}(x[t]) + sum_s FFN_{E+s}(x[t])
//   FFN_e(v) = W2_e act(W1_e v + b1_e) + b2_e
//
// Few rows per expert: the products are bound by reading each taken expert's
// weights once from HBM, so the grouped GEMM's 128..256-row tiles would be
// mostly empty.  Here waves stream 16-row weight tiles straight into MFMA
// operands (few_rows.h).
//
//   logits kernel   one workgroup per expert and 16 tokens, float64 logits
//   phase 1         per taken expert and 16 hidden units: act(W1 x + b1) times
//                   the routing weight
//   phase 2         per 16 output columns: the sum over all taken experts
//
// The routed weight is folded into the hidden rows in float32, and the hidden
// rows are kept to 16 bits of mantissa (bf16 layers: a bf16 number and its bf16
// remainder, which ride in the same 16-row MFMA operand as 8 + 8 rows), so the
// output carries one rounding, its own.
#include "few_rows.h"

namespace moe {
namespace {

constexpr int kWaves = 8;                 // waves of a phase workgroup; they split k
constexpr int kThreads = kWaves * kWave;
constexpr int kMaxT = MOE_MAX_DECODE_TOKENS;
constexpr int kMaxE = MOE_MAX_EXPERTS + MOE_MAX_SHARED;

// ------------------------------------------------------------------ logits --
// logits[t, e] in float64.  bf16: products are exact in float32, eight are
// summed in float32 and the sums of eight in float64; float32: float64
// products and sums.
template <bool BF16>
__device__ __forceinline__ void load8(const void* p, size_t off, float (&o)[8]) {
  if constexpr (BF16) {
    const u32x4 v = *reinterpret_cast<const u32x4*>(static_cast<const uint16_t*>(p) + off);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      o[2 * i] = __uint_as_float(v[i] << 16);
      o[2 * i + 1] = __uint_as_float(v[i] & 0xffff0000u);
    }
  } else {
    const floatx4* f = reinterpret_cast<const floatx4*>(static_cast<const float*>(p) + off);
    const floatx4 a = f[0], b = f[1];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      o[i] = a[i];
      o[4 + i] = b[i];
    }
  }
}

template <bool BF16, int NTOK>
__global__ __launch_bounds__(256) void decode_logits_kernel(DecodeArgs a) {
  __shared__ double red[4][NTOK];
  const int e = blockIdx.x, t0 = blockIdx.y * NTOK;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  double acc[NTOK];
#pragma unroll
  for (int i = 0; i < NTOK; ++i) acc[i] = 0.0;
  for (int c = threadIdx.x * 8; c < a.d; c += 256 * 8) {
    float w[8];
    load8<BF16>(a.W_g, static_cast<size_t>(e) * a.d + c, w);
#pragma unroll
    for (int i = 0; i < NTOK; ++i) {
      float x[8];
      const int t = min(t0 + i, a.T - 1);
      load8<BF16>(a.x, static_cast<size_t>(t) * a.d + c, x);
      if constexpr (BF16) {
        float s = x[0] * w[0];
#pragma unroll
        for (int m = 1; m < 8; ++m) s = fmaf(x[m], w[m], s);
        acc[i] += static_cast<double>(s);
      } else {
#pragma unroll
        for (int m = 0; m < 8; ++m) acc[i] = fma(static_cast<double>(x[m]), static_cast<double>(w[m]), acc[i]);
      }
    }
  }
#pragma unroll
  for (int i = 0; i < NTOK; ++i) {
#pragma unroll
    for (int o = 32; o >= 1; o >>= 1) acc[i] += __shfl_xor(acc[i], o);
    if (lane == 0) red[wave][i] = acc[i];
  }
  __syncthreads();
  if (threadIdx.x < NTOK && t0 + static_cast<int>(threadIdx.x) < a.T) {
    const int i = threadIdx.x;
    double l = ((red[0][i] + red[1][i]) + red[2][i]) + red[3][i];
    if (a.b_g != nullptr) l += static_cast<double>(a.b_g[e]);
    a.logits[static_cast<size_t>(t0 + i) * a.E + e] = l;
  }
  // counters of the phase kernels: all workgroups of this launch share the work
  const int nth = gridDim.x * gridDim.y * 256;
  for (int i = (blockIdx.y * gridDim.x + blockIdx.x) * 256 + threadIdx.x; i < a.ncounter; i += nth) a.counters[i] = 0;
}

// --------------------------------------------------------------- selection --
// The routing of the call, rebuilt by every workgroup from the logits (a few
// hundred numbers per token) rather than passed through another launch.
struct Routing {
  int idx[kMaxT][MOE_MAX_TOPK];     // expert of slot j, routed slots only
  float w[kMaxT][MOE_MAX_TOPK];
  unsigned long long mask[kMaxE];   // tokens of each expert
  int list[kMaxE];                  // taken experts, ascending, shared ones last
  int n;                            // their number
  int wsum[kWaves];
};

// One wave, one token: the k largest logits (+ selection bias), ties to the
// lower expert; a NaN ranks below every number.  Lane l holds experts l,
// l + 64, l + 128, l + 192.
__device__ __forceinline__ void select_token(const DecodeArgs& a, Routing& r, int t, int lane, bool write) {
  double key[4], val[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int e = lane + 64 * i;
    val[i] = e < a.E ? a.logits[static_cast<size_t>(t) * a.E + e] : 0.0;
    double kv = val[i];
    if (a.b_sel != nullptr && e < a.E) kv += static_cast<double>(a.b_sel[e]);
    key[i] = kv == kv ? kv : -INFINITY;
  }
  uint32_t taken = 0;
  constexpr int kNone = 0x7fffffff;
  int my_idx = 0;
  double my_l = -INFINITY, m = -INFINITY;
  for (int j = 0; j < a.k; ++j) {
    double bv = -INFINITY, bl = -INFINITY;
    int bi = kNone;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int e = lane + 64 * i;
      const bool take = (e < a.E) & !((taken >> i) & 1u) & ((bi == kNone) | (key[i] > bv));
      bv = take ? key[i] : bv;
      bi = take ? e : bi;
      bl = take ? val[i] : bl;
    }
#pragma unroll
    for (int o = 32; o >= 1; o >>= 1) {
      const double ov = __shfl_xor(bv, o), ol = __shfl_xor(bl, o);
      const int oi = __shfl_xor(bi, o);
      const bool take = (ov > bv) | ((ov == bv) & (oi < bi));
      bv = take ? ov : bv;
      bl = take ? ol : bl;
      bi = take ? oi : bi;
    }
    if ((bi & 63) == lane) taken |= 1u << (bi >> 6);
    if (lane == j) {
      my_idx = bi;
      my_l = bl;
    }
    m = bl > m ? bl : m;
  }
  const float ej = lane < a.k ? expf(static_cast<float>(my_l - m)) : 0.f;
  float sum = 0.f;
  for (int j = 0; j < a.k; ++j) sum += __shfl(ej, j);
  if (lane < a.k) {
    const float w = ej / sum;
    r.idx[t][lane] = my_idx;
    r.w[t][lane] = w;
    if (write) {
      a.topk_idx[t * a.k + lane] = my_idx;
      a.topk_w[t * a.k + lane] = w;
    }
  }
}

__device__ __forceinline__ void build_routing(const DecodeArgs& a, Routing& r, bool write) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int ne = a.E + a.S;
  const unsigned long long all = a.T == 64 ? ~0ull : (1ull << a.T) - 1ull;
  for (int e = threadIdx.x; e < ne; e += kThreads) r.mask[e] = e < a.E ? 0ull : all;
  for (int t = wave; t < a.T; t += kWaves) select_token(a, r, t, lane, write);
  __syncthreads();
  for (int i = threadIdx.x; i < a.T * a.k; i += kThreads) {
    const int t = i / a.k, j = i - t * a.k;
    atomicOr(&r.mask[r.idx[t][j]], 1ull << t);   // a set: the order does not matter
  }
  __syncthreads();
  // ascending list of the taken experts (ne <= 264 < kThreads)
  const bool on = static_cast<int>(threadIdx.x) < ne && r.mask[threadIdx.x] != 0ull;
  const unsigned long long b = __ballot(on);
  if (lane == 0) r.wsum[wave] = __popcll(b);
  __syncthreads();
  int base = 0;
  for (int w = 0; w < wave; ++w) base += r.wsum[w];
  if (on) r.list[base + __popcll(b & ((1ull << lane) - 1ull))] = threadIdx.x;
  if (threadIdx.x == kThreads - 1) r.n = base + r.wsum[wave];
  __syncthreads();
}

// slot of expert e in token t's list: j, or k + s for shared expert s
__device__ __forceinline__ int slot_of(const DecodeArgs& a, const Routing& r, int t, int e) {
  if (e >= a.E) return a.k + e - a.E;
  int j = 0;
  for (int i = 1; i < a.k; ++i) j = r.idx[t][i] == e ? i : j;
  return j;
}

// the p-th set bit of m (p < popcount)
__device__ __forceinline__ int nth_bit(unsigned long long m, int p) {
  for (int i = 0; i < p; ++i) m &= m - 1ull;
  return __ffsll(static_cast<long long>(m)) - 1;
}

template <bool BF16>
__device__ __forceinline__ float load1(const void* p, size_t i) {
  if constexpr (BF16) return bf16_to_f32(static_cast<const uint16_t*>(p)[i]);
  else return static_cast<const float*>(p)[i];
}

// ------------------------------------------------------------------ phase 1 --
// One item: taken expert e and hidden units n0 .. n0 + 15.  The expert's tokens
// are the activation rows, NT tiles of 16; the waves split k and add their
// sums in LDS in wave order.
template <Fmt F, int NT>
__device__ void phase1_item(const DecodeArgs& a, Routing& r, float* red, int item, int ntile) {
  constexpr bool kBf = F != Fmt::kF32;
  constexpr int U = F == Fmt::kW4 ? 4 : 8;
  const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
  const int e = uniform(r.list[item / ntile]);
  const int n0 = (item % ntile) * 16;
  const unsigned long long mask = r.mask[e];
  const int rows = __popcll(mask);
  const uint32_t pitch = static_cast<uint32_t>(a.d) * (kBf ? 2u : 4u);
  const __amdgpu_buffer_rsrc_t xr = make_rsrc(a.x, static_cast<uint32_t>(a.T) * pitch);
  uint32_t aoff[NT];
#pragma unroll
  for (int j = 0; j < NT; ++j) {
    const int p = j * 16 + (lane & 15);
    aoff[j] = p < rows ? static_cast<uint32_t>(nth_bit(mask, p)) * pitch + 16u * (lane >> 4) : kOut;
  }
  floatx4 acc[NT];
#pragma unroll
  for (int j = 0; j < NT; ++j) acc[j] = floatx4{0.f, 0.f, 0.f, 0.f};
  const int nst = (a.d + FmtOf<F>::kK - 1) / FmtOf<F>::kK;
  const int s0 = wave * nst / kWaves, s1 = (wave + 1) * nst / kWaves;
  const uint32_t tiles = (1u << ((rows + 15) / 16)) - 1u;
  const WRows wr = rows_of<F>(a.W1, e, n0, lane);
  stream_rows<F, NT, U>(acc, wr, xr, aoff, tiles, s0, s1, a.d, a.W1.gshift, lane);
#pragma unroll
  for (int j = 0; j < NT; ++j)
    if (NT == 1 || ((tiles >> j) & 1u))
      *reinterpret_cast<floatx4*>(red + ((j * kWaves + wave) * 64 + lane) * 4) = acc[j];
  __syncthreads();
  const int tl = (rows + 15) / 16;
  for (int i = threadIdx.x; i < tl * 256; i += kThreads) {
    // result (row p of the expert's tokens, hidden unit n): lane (n, p / 4 % 4), register p % 4
    const int j = i >> 8, n = i & 15, pr = (i >> 4) & 15;
    const int p = j * 16 + pr;
    if (p >= rows || n0 + n >= a.h) continue;
    const float* s = red + (j * kWaves * 64 + (pr >> 2) * 16 + n) * 4 + (pr & 3);
    float v = 0.f;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) v += s[w * 256];
    if (a.b1 != nullptr) v += load1<kBf>(a.b1, static_cast<size_t>(e) * a.h + n0 + n);
    v = a.act == MOE_ACT_SILU ? v / (1.f + expf(-v)) : 0.5f * v * (1.f + erff(v * 0.70710678118654752440f));
    const int t = nth_bit(mask, p);
    const int slot = slot_of(a, r, t, e);
    if (slot < a.k) v *= r.w[t][slot];
    const size_t row = static_cast<size_t>(t) * (a.k + a.S) + slot;
    if constexpr (kBf) {
      // value and remainder: 16 bits of mantissa; an infinity has no remainder
      const uint16_t hi = f32_to_bf16(v);
      const float hf = bf16_to_f32(hi);
      const uint16_t lo = fabsf(hf) < INFINITY ? f32_to_bf16(v - hf) : 0;
      uint16_t* hb = static_cast<uint16_t*>(a.hid) + row * 2 * a.h + n0 + n;
      hb[0] = hi;
      hb[a.h] = lo;
    } else {
      static_cast<float*>(a.hid)[row * a.h + n0 + n] = v;
    }
  }
  __syncthreads();   // red is written again by the next item
}

// ------------------------------------------------------------------ phase 2 --
// One item: output columns n0 .. n0 + 15 over share sp of the summed range, all
// taken experts' k one after the other.  Activation tiles hold 8 tokens (bf16:
// rows 0..7 the hidden values, 8..15 their remainders) or 16 (float32) by token
// index; an expert's tiles without a token of its own are passed over, and its
// sums are added only to its tokens' rows, so an expert's infinities or NaN
// reach no token that did not take it.
template <Fmt F, int NT>
__device__ void phase2_item(const DecodeArgs& a, Routing& r, float* red, int* flag, int item) {
  constexpr bool kBf = F != Fmt::kF32;
  constexpr int U = F == Fmt::kW4 ? 4 : 8;
  constexpr int kTok = kBf ? 8 : 16;
  const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
  const int sp = item % a.split;
  const int tile = item / a.split;
  const int n0 = tile * 16;
  const int nst = (a.h + FmtOf<F>::kK - 1) / FmtOf<F>::kK;
  const int na = uniform(r.n);
  const long long total = static_cast<long long>(na) * nst;
  const int share = sp * kWaves + wave, shares = a.split * kWaves;
  long long f = total * share / shares;
  const long long fend = total * (share + 1) / shares;
  floatx4 sum[NT];
#pragma unroll
  for (int j = 0; j < NT; ++j) sum[j] = floatx4{0.f, 0.f, 0.f, 0.f};
  const uint32_t pitch = static_cast<uint32_t>(a.h) * (kBf ? 2u : 4u);
  const uint32_t rowb = kBf ? 2u * pitch : pitch;
  const __amdgpu_buffer_rsrc_t hr =
      make_rsrc(a.hid, static_cast<uint32_t>(a.T) * static_cast<uint32_t>(a.k + a.S) * rowb);
  while (f < fend) {
    const int ai = static_cast<int>(f / nst);
    const int s0 = static_cast<int>(f - static_cast<long long>(ai) * nst);
    const int s1 = static_cast<int>(fend - f < nst - s0 ? s0 + (fend - f) : nst);
    const int e = uniform(r.list[ai]);
    const unsigned long long mask = r.mask[e];
    uint32_t tiles = 0;
    uint32_t aoff[NT];
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      constexpr unsigned long long kOnes = (1ull << kTok) - 1ull;
      if ((mask >> (j * kTok)) & kOnes) tiles |= 1u << j;
      const int t = j * kTok + (lane & (kTok - 1));
      aoff[j] = kOut;
      if ((mask >> t) & 1ull) {
        aoff[j] = (static_cast<uint32_t>(t) * (a.k + a.S) + slot_of(a, r, t, e)) * rowb + 16u * (lane >> 4);
        if (kBf && (lane & 8)) aoff[j] += pitch;
      }
    }
    tiles = uniform(tiles);
    floatx4 acc[NT];
#pragma unroll
    for (int j = 0; j < NT; ++j) acc[j] = floatx4{0.f, 0.f, 0.f, 0.f};
    const WRows wr = rows_of<F>(a.W2, e, n0, lane);
    stream_rows<F, NT, U>(acc, wr, hr, aoff, tiles, s0, s1, a.h, a.W2.gshift, lane);
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int t = j * kTok + (((lane >> 4) * 4 + i) & (kTok - 1));
        if ((mask >> t) & 1ull) sum[j][i] += acc[j][i];
      }
    f += s1 - s0;
  }
  // waves, then (bf16) values and remainders, in fixed order
#pragma unroll
  for (int j = 0; j < NT; ++j) {
    *reinterpret_cast<floatx4*>(red + (wave * 64 + lane) * 4) = sum[j];
    __syncthreads();
    for (int i = threadIdx.x; i < kTok * 16; i += kThreads) {
      const int n = i & 15, pr = i >> 4, t = j * kTok + pr;
      if (t < a.T && n0 + n < a.d) {
        float v = 0.f;
#pragma unroll
        for (int w = 0; w < kWaves; ++w) {
          const float* s = red + w * 256 + n * 4 + (pr & 3);
          v += s[(pr >> 2) * 64];
          if (kBf) v += s[((pr >> 2) + 2) * 64];
        }
        if (a.split > 1) {
          a.part[(static_cast<size_t>(sp) * a.T + t) * a.d + n0 + n] = v;
        } else {
          float b = 0.f;
          if (a.b2 != nullptr) {
            for (int q = 0; q < a.k; ++q)
              b = fmaf(r.w[t][q], load1<kBf>(a.b2, static_cast<size_t>(r.idx[t][q]) * a.d + n0 + n), b);
            for (int q = 0; q < a.S; ++q) b += load1<kBf>(a.b2, static_cast<size_t>(a.E + q) * a.d + n0 + n);
          }
          v += b;
          const size_t o = static_cast<size_t>(t) * a.d + n0 + n;
          if (kBf) static_cast<uint16_t*>(a.out)[o] = f32_to_bf16(v);
          else static_cast<float*>(a.out)[o] = v;
        }
      }
    }
    __syncthreads();
  }
  if (a.split == 1) return;
  // the last share of the tile to arrive adds all of them, in share order
  __threadfence();
  __syncthreads();
  if (threadIdx.x == 0) *flag = atomicAdd(&a.counters[tile], 1) == a.split - 1;
  __syncthreads();
  if (*flag) {
    __threadfence();
    for (int i = threadIdx.x; i < a.T * 16; i += kThreads) {
      const int n = i & 15, t = i >> 4;
      if (n0 + n >= a.d) continue;
      float v = 0.f;
      for (int q = 0; q < a.split; ++q) v += a.part[(static_cast<size_t>(q) * a.T + t) * a.d + n0 + n];
      if (a.b2 != nullptr) {
        float b = 0.f;
        for (int q = 0; q < a.k; ++q)
          b = fmaf(r.w[t][q], load1<kBf>(a.b2, static_cast<size_t>(r.idx[t][q]) * a.d + n0 + n), b);
        for (int q = 0; q < a.S; ++q) b += load1<kBf>(a.b2, static_cast<size_t>(a.E + q) * a.d + n0 + n);
        v += b;
      }
      const size_t o = static_cast<size_t>(t) * a.d + n0 + n;
      if (kBf) static_cast<uint16_t*>(a.out)[o] = f32_to_bf16(v);
      else static_cast<float*>(a.out)[o] = v;
    }
  }
  __syncthreads();
}

template <Fmt F, int NT1, int NT2>
__global__ __launch_bounds__(kThreads) void decode_phase_kernel(DecodeArgs a, int phase) {
  __shared__ Routing r;
  __shared__ float red[NT1 * kWaves * 256];
  __shared__ int flag;
  build_routing(a, r, phase == 1 && blockIdx.x == 0);
  const int na = uniform(r.n);
  if (phase == 1) {
    const int ntile = (a.h + 15) / 16;
    for (int i = blockIdx.x; i < na * ntile; i += gridDim.x) phase1_item<F, NT1>(a, r, red, i, ntile);
  } else {
    const int items = (a.d + 15) / 16 * a.split;
    for (int i = blockIdx.x; i < items; i += gridDim.x) phase2_item<F, NT2>(a, r, red, &flag, i);
  }
}

template <Fmt F>
hipError_t launch_phase(const DecodeArgs& a, int grid, int phase, hipStream_t st) {
  constexpr bool kBf = F != Fmt::kF32;
  if (a.T <= 8) decode_phase_kernel<F, 1, 1><<<grid, kThreads, 0, st>>>(a, phase);
  else if (a.T <= 16) decode_phase_kernel<F, 1, kBf ? 2 : 1><<<grid, kThreads, 0, st>>>(a, phase);
  else decode_phase_kernel<F, 4, kBf ? 8 : 4><<<grid, kThreads, 0, st>>>(a, phase);
  return hipGetLastError();
}

template <bool BF16>
void launch_logits(const DecodeArgs& a, hipStream_t st) {
  if (a.T == 1) decode_logits_kernel<BF16, 1><<<dim3(a.E, 1), 256, 0, st>>>(a);
  else if (a.T <= 4) decode_logits_kernel<BF16, 4><<<dim3(a.E, 1), 256, 0, st>>>(a);
  else decode_logits_kernel<BF16, 16><<<dim3(a.E, (a.T + 15) / 16), 256, 0, st>>>(a);
}

}  // namespace

// Shares of the summed range per 16 output columns: enough items for about
// four per workgroup slot, at least 32 KB of weights in each.
int decode_split(int T, int d, int h, int E, int k, int S, long long row_bytes) {
  const long long tiles = (d + 15) / 16;
  long long used = static_cast<long long>(T) * k;
  if (used > E) used = E;
  used += S;
  const long long bytes = used * 16 * row_bytes;   // of one tile
  long long sp = (2048 + tiles - 1) / tiles;
  if (sp > bytes / 32768) sp = bytes / 32768;
  if (sp > 64) sp = 64;
  return sp < 1 ? 1 : static_cast<int>(sp);
}

hipError_t launch_decode(const DecodeArgs& a, hipStream_t st) {
  if (a.fmt == kDecodeF32) launch_logits<false>(a, st);
  else launch_logits<true>(a, st);
  hipError_t e = hipGetLastError();
  const int grid = 2 * device_cu_count();
  for (int phase = 1; phase <= 2 && e == hipSuccess; ++phase) {
    if (a.fmt == kDecodeF32) e = launch_phase<Fmt::kF32>(a, grid, phase, st);
    else if (a.fmt == kDecodeBf16) e = launch_phase<Fmt::kBf16>(a, grid, phase, st);
    else e = launch_phase<Fmt::kW4>(a, grid, phase, st);
  }
  return e;
}

}  // namespace moe
