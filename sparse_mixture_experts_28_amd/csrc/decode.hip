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
// What the logits kernels leave besides the logits: zeroed counters for phase 2
// and, for 4-bit weights, x in the order of the codes.
__device__ __forceinline__ void prepare_phases(const DecodeArgs& a) {
  const int nth = gridDim.x * gridDim.y * blockDim.x;
  const int id = (blockIdx.y * gridDim.x + blockIdx.x) * blockDim.x + threadIdx.x;
  for (int i = id; i < a.ncounter; i += nth) a.counters[i] = 0;
  if (a.fmt == kDecodeW4)
    for (int i = id; i < a.T * (a.d / 8); i += nth)
      static_cast<u32x4*>(a.xord)[i] = to_code_order(static_cast<const u32x4*>(a.x)[i]);
}

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

// One workgroup per expert and NTOK tokens, a thread per 8 elements of d (up to
// 8192 in one pass).  bf16: products are exact in float32, eight are summed in
// float32 and the sums of eight in float64; float32: float64 products and sums.
template <bool BF16, int NTOK>
__global__ __launch_bounds__(1024) void decode_logits_kernel(DecodeArgs a) {
  __shared__ double red[16][NTOK];
  const int e = blockIdx.x, t0 = blockIdx.y * NTOK;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  double acc[NTOK];
#pragma unroll
  for (int i = 0; i < NTOK; ++i) acc[i] = 0.0;
  for (int c = threadIdx.x * 8; c < a.d; c += blockDim.x * 8) {
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
    double l = 0.0;
    for (int w = 0; w < static_cast<int>(blockDim.x >> 6); ++w) l += red[w][i];
    if (a.b_g != nullptr) l += static_cast<double>(a.b_g[e]);
    a.logits[static_cast<size_t>(t0 + i) * a.E + e] = l;
  }
  prepare_phases(a);
}

// bf16, more tokens: 16 experts x 16 tokens per workgroup on the matrix cores,
// 16 waves splitting d.  The float32 sums run over at most 256 elements and are
// added in float64.
__global__ __launch_bounds__(1024) void decode_logits_mfma_kernel(DecodeArgs a) {
  __shared__ double red[16][64][4];
  const int e0 = blockIdx.x * 16, t0 = blockIdx.y * 16;
  const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
  const int r = lane & 15, q = lane >> 4;
  const uint32_t pitch = static_cast<uint32_t>(a.d) * 2u;
  const __amdgpu_buffer_rsrc_t xr = make_rsrc(a.x, static_cast<uint32_t>(a.T) * pitch);
  const __amdgpu_buffer_rsrc_t gr = make_rsrc(a.W_g, static_cast<uint32_t>(a.E) * pitch);
  const uint32_t xo = t0 + r < a.T ? static_cast<uint32_t>(t0 + r) * pitch + 16u * q : kOut;
  const uint32_t go = e0 + r < a.E ? static_cast<uint32_t>(e0 + r) * pitch + 16u * q : kOut;
  const int nst = (a.d + 31) / 32;
  const int s0 = wave * nst / 16, s1 = (wave + 1) * nst / 16;
  double acc[4] = {0.0, 0.0, 0.0, 0.0};
  for (int sb = s0; sb < s1; sb += 8) {
    u32x4 x[8], g[8];
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      const bool in = sb + u < s1 && (sb + u) * 32 + q * 8 < a.d;
      g[u] = load16(gr, in ? go : kOut, static_cast<uint32_t>(sb + u) * 64u);
      x[u] = load16(xr, in ? xo : kOut, static_cast<uint32_t>(sb + u) * 64u);
    }
    floatx4 t = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int u = 0; u < 8; ++u)
      t = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, x[u]), __builtin_bit_cast(bf16x8, g[u]), t,
                                                  0, 0, 0);
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[i] += static_cast<double>(t[i]);
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) red[wave][lane][i] = acc[i];
  __syncthreads();
  if (threadIdx.x < 256) {
    const int ln = threadIdx.x & 63, i = threadIdx.x >> 6;
    const int t = t0 + (ln >> 4) * 4 + i, e = e0 + (ln & 15);
    if (t < a.T && e < a.E) {
      double l = 0.0;
#pragma unroll
      for (int w = 0; w < 16; ++w) l += red[w][ln][i];
      if (a.b_g != nullptr) l += static_cast<double>(a.b_g[e]);
      a.logits[static_cast<size_t>(t) * a.E + e] = l;
    }
  }
  prepare_phases(a);
}

// --------------------------------------------------------------- selection --
// The routing of the call, rebuilt by every workgroup from the logits (a few
// hundred numbers per token) rather than passed through another launch.
struct Routing {
  int idx[kMaxT][MOE_MAX_TOPK];     // expert of slot j, routed slots only
  float w[kMaxT][MOE_MAX_TOPK];
  unsigned long long mask[kMaxE];   // tokens of each expert
  int list[kMaxE];                  // taken experts, ascending, shared ones last
  int off[kMaxE + 1];               // first of each one's rows
  uint16_t row[kMaxT * (MOE_MAX_TOPK + MOE_MAX_SHARED)];   // token + 256 slot, ascending tokens; slot k + s: shared s
  int n;                            // taken experts
  uint32_t wsum[kWaves];
};

template <int CTRL>
__device__ __forceinline__ double dpp_max(double v) {
  const unsigned long long b = __builtin_bit_cast(unsigned long long, v);
  const uint32_t lo = __builtin_amdgcn_mov_dpp(static_cast<int>(static_cast<uint32_t>(b)), CTRL, 0xF, 0xF, false);
  const uint32_t hi = __builtin_amdgcn_mov_dpp(static_cast<int>(static_cast<uint32_t>(b >> 32)), CTRL, 0xF, 0xF, false);
  return fmax(v, __builtin_bit_cast(double, (static_cast<unsigned long long>(hi) << 32) | lo));
}
__device__ __forceinline__ double pair_max(uint32_t l0, uint32_t h0, uint32_t l1, uint32_t h1) {
  return fmax(__builtin_bit_cast(double, (static_cast<unsigned long long>(h0) << 32) | l0),
              __builtin_bit_cast(double, (static_cast<unsigned long long>(h1) << 32) | l1));
}
// maximum over the wave, in every lane: within rows of 16 lanes by row moves
// (lane ^ 1, lane ^ 2, the mirrors), across them by register swaps
__device__ __forceinline__ double wave_max(double v) {
  v = dpp_max<0xB1>(v);
  v = dpp_max<0x4E>(v);
  v = dpp_max<0x141>(v);
  v = dpp_max<0x140>(v);
  unsigned long long b = __builtin_bit_cast(unsigned long long, v);
  uint32_t lo = static_cast<uint32_t>(b), hi = static_cast<uint32_t>(b >> 32);
  auto l = __builtin_amdgcn_permlane16_swap(lo, lo, false, false);
  auto h = __builtin_amdgcn_permlane16_swap(hi, hi, false, false);
  v = pair_max(l[0], h[0], l[1], h[1]);
  b = __builtin_bit_cast(unsigned long long, v);
  lo = static_cast<uint32_t>(b);
  hi = static_cast<uint32_t>(b >> 32);
  l = __builtin_amdgcn_permlane32_swap(lo, lo, false, false);
  h = __builtin_amdgcn_permlane32_swap(hi, hi, false, false);
  return pair_max(l[0], h[0], l[1], h[1]);
}

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
  uint32_t left = 0;   // bit i: expert lane + 64 i is there and not taken
#pragma unroll
  for (int i = 0; i < 4; ++i) left |= lane + 64 * i < a.E ? 1u << i : 0u;
  int my_idx = 0;
  double my_l = -INFINITY, m = -INFINITY;
  for (int j = 0; j < a.k; ++j) {
    double best = -INFINITY;
    int bi = 4;        // the lane's lowest expert of its largest key
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const bool take = ((left >> i) & 1u) && (bi == 4 || key[i] > best);
      best = take ? key[i] : best;
      bi = take ? i : bi;
    }
    const double top = wave_max(best);
    int win = 0;
#pragma unroll
    for (int i = 3; i >= 0; --i) {   // the lowest expert wins: the lowest i, then the lowest lane
      const unsigned long long b = __ballot(bi == i && best == top);
      if (b != 0ull) win = 64 * i + __ffsll(static_cast<long long>(b)) - 1;
    }
    const int wl = win & 63, wi = win >> 6;
    if (lane == wl) left &= ~(1u << wi);
    const double v = wi == 0 ? val[0] : wi == 1 ? val[1] : wi == 2 ? val[2] : val[3];
    const unsigned long long vb = __builtin_bit_cast(unsigned long long, v);
    const uint32_t lo = __builtin_amdgcn_readlane(static_cast<int>(static_cast<uint32_t>(vb)), wl);
    const uint32_t hi = __builtin_amdgcn_readlane(static_cast<int>(static_cast<uint32_t>(vb >> 32)), wl);
    const double l = __builtin_bit_cast(double, (static_cast<unsigned long long>(hi) << 32) | lo);
    if (lane == j) {
      my_idx = win;
      my_l = l;
    }
    m = l > m ? l : m;
  }
  const float ej = lane < a.k ? expf(static_cast<float>(my_l - m)) : 0.f;
  float sum = 0.f;
  for (int j = 0; j < a.k; ++j)
    sum += __uint_as_float(__builtin_amdgcn_readlane(static_cast<int>(__float_as_uint(ej)), j));
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

// Each expert's tokens, the list of the taken experts and their rows, from idx.
// Thread e handles expert e (at most 264 of 512 threads).
__device__ __forceinline__ void list_routing(const DecodeArgs& a, Routing& r) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, e = threadIdx.x;
  const int ne = a.E + a.S, na = a.T * a.k;
  const unsigned long long all = a.T == 64 ? ~0ull : (1ull << a.T) - 1ull;
  unsigned long long mask = e >= a.E && e < ne ? all : 0ull;
  if (na <= 16) {
    __syncthreads();
    for (int t = 0; t < a.T; ++t)
      for (int j = 0; j < a.k; ++j) mask |= r.idx[t][j] == e ? 1ull << t : 0ull;
  } else {
    if (e < a.E) r.mask[e] = 0ull;
    __syncthreads();
    for (int i = threadIdx.x; i < na; i += kThreads) {
      const int t = i / a.k, j = i - t * a.k;
      atomicOr(&r.mask[r.idx[t][j]], 1ull << t);   // a set: the order does not matter
    }
    __syncthreads();
    if (e < a.E) mask = r.mask[e];
  }
  // prefix sums of (taken, rows), in two halves of a word
  const uint32_t own = mask != 0ull ? 0x10000u + __popcll(mask) : 0u;
  uint32_t sc = own;
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const uint32_t up = __shfl_up(sc, o);
    if (lane >= o) sc += up;
  }
  if (lane == 63) r.wsum[wave] = sc;
  __syncthreads();
  uint32_t before = sc - own, total = 0;
  for (int w = 0; w < kWaves; ++w) {
    if (w < wave) before += r.wsum[w];
    total += r.wsum[w];
  }
  if (mask != 0ull) {
    const int pos = before >> 16;
    int o = before & 0xffffu;
    r.list[pos] = e;
    r.off[pos] = o;
    while (mask != 0ull) {
      const int t = __ffsll(static_cast<long long>(mask)) - 1;
      mask &= mask - 1ull;
      int slot = a.k + e - a.E;
      if (e < a.E) {
        slot = 0;
        for (int i = 1; i < a.k; ++i) slot = r.idx[t][i] == e ? i : slot;
      }
      r.row[o++] = static_cast<uint16_t>(t | (slot << 8));
    }
  }
  if (threadIdx.x == 0) {
    r.n = total >> 16;
    r.off[total >> 16] = total & 0xffffu;
  }
  __syncthreads();
}

// from the logits
__device__ __forceinline__ void build_routing(const DecodeArgs& a, Routing& r, bool write) {
  for (int t = threadIdx.x >> 6; t < a.T; t += kWaves) select_token(a, r, t, threadIdx.x & 63, write);
  list_routing(a, r);
}

// from the experts and weights that phase 1 left in the outputs
__device__ __forceinline__ void load_routing(const DecodeArgs& a, Routing& r) {
  for (int i = threadIdx.x; i < a.T * a.k; i += kThreads) {
    const int t = i / a.k, j = i - t * a.k;
    r.idx[t][j] = a.topk_idx[i];
    r.w[t][j] = a.topk_w[i];
  }
  list_routing(a, r);
}

template <bool BF16>
__device__ __forceinline__ float load1(const void* p, size_t i) {
  if constexpr (BF16) return bf16_to_f32(static_cast<const uint16_t*>(p)[i]);
  else return static_cast<const float*>(p)[i];
}

// Numbers that one workgroup of a launch leaves for another, which may run on
// another XCD with an L2 of its own: stored and loaded at agent scope (each such
// access goes past the L2 to memory all XCDs see), and the stores waited for
// before the counter says so.  Agent fences around plain accesses would do the
// same by writing back and dropping whole caches under the weight stream: with
// them in every wave the second phase of the Mixtral-shaped layer took 760 us for
// one token, with these 50.
__device__ __forceinline__ void store_agent(float* p, float v) {
  __hip_atomic_store(p, v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ float load_agent(const float* p) {
  return __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ void stores_done() {
  __asm__ volatile("" ::: "memory");
  __builtin_amdgcn_s_waitcnt(vm_wait_imm(0));
  __asm__ volatile("" ::: "memory");
}

// ------------------------------------------------------------------ phase 1 --
// One item: taken expert number ai and 16 RT hidden units from n0.  The expert's
// tokens are the activation rows, NT tiles of 16; the waves split k and add
// their sums in LDS in wave order.
template <Fmt F, int NT, int RT, int U>
__device__ void phase1_item(const DecodeArgs& a, Routing& r, float* red, int ai, int n0) {
  constexpr bool kBf = F != Fmt::kF32;
  const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
  const int e = uniform(r.list[ai]), o = uniform(r.off[ai]);
  const int rows = uniform(r.off[ai + 1]) - o;
  const uint32_t pitch = static_cast<uint32_t>(a.d) * (kBf ? 2u : 4u);
  const __amdgpu_buffer_rsrc_t xr = make_rsrc(is_w4(F) ? a.xord : a.x, static_cast<uint32_t>(a.T) * pitch);
  const int nst = (a.d + step_k(F) - 1) / step_k(F);
  const int s0 = wave * nst / kWaves, s1 = (wave + 1) * nst / kWaves;
  const WRows wr = rows_of<F, RT>(a.W1, e, n0, lane);
  for (int p0 = 0; p0 < rows; p0 += 16 * NT) {
    uint32_t arow[NT];
    floatx4 acc[NT][RT];
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      const int p = p0 + j * 16 + (lane & 15);
      arow[j] = p < rows ? static_cast<uint32_t>(r.row[o + p] & 255) * pitch : kOut;
#pragma unroll
      for (int i = 0; i < RT; ++i) acc[j][i] = floatx4{0.f, 0.f, 0.f, 0.f};
    }
    const int tl = min(NT, (rows - p0 + 15) / 16);
    if (is_w4(F) && a.W1.z != nullptr) stream_rows<F, NT, RT, U, true, true>(acc, wr, xr, arow, tl, s0, s1, a.d, lane);
    else stream_rows<F, NT, RT, U, true, false>(acc, wr, xr, arow, tl, s0, s1, a.d, lane);
#pragma unroll
    for (int j = 0; j < NT; ++j)
      if (NT == 1 || j < tl) {
#pragma unroll
        for (int i = 0; i < RT; ++i)
          *reinterpret_cast<floatx4*>(red + (((j * RT + i) * kWaves + wave) * 64 + lane) * 4) = acc[j][i];
      }
    __syncthreads();
    for (int i = threadIdx.x; i < tl * RT * 256; i += kThreads) {
      // result (row p of the expert's tokens, hidden unit n): lane (n, p / 4 % 4), register p % 4
      const int jr = i >> 8, n = n0 + (jr % RT) * 16 + (i & 15), pr = (i >> 4) & 15;
      const int p = p0 + jr / RT * 16 + pr;
      if (p >= rows || n >= a.h) continue;
      const float* s = red + (jr * kWaves * 64 + (pr >> 2) * 16 + (i & 15)) * 4 + (pr & 3);
      float v = 0.f;
#pragma unroll
      for (int w = 0; w < kWaves; ++w) v += s[w * 256];
      if (a.b1 != nullptr) v += load1<kBf>(a.b1, static_cast<size_t>(e) * a.h + n);
      v = a.act == MOE_ACT_SILU ? v / (1.f + expf(-v)) : 0.5f * v * (1.f + erff(v * 0.70710678118654752440f));
      const int t = r.row[o + p] & 255, slot = r.row[o + p] >> 8;
      if (slot < a.k) v *= r.w[t][slot];
      const size_t row = static_cast<size_t>(t) * (a.k + a.S) + slot;
      if constexpr (kBf) {
        // value and remainder: 16 bits of mantissa; an infinity has no remainder
        const uint16_t hi = f32_to_bf16(v);
        const float hf = bf16_to_f32(hi);
        const uint16_t lo = fabsf(hf) < INFINITY ? f32_to_bf16(v - hf) : 0;
        uint16_t* hb = static_cast<uint16_t*>(a.hid) + row * 2 * a.h + (is_w4(F) ? code_order(n) : n);
        hb[0] = hi;
        hb[a.h] = lo;
      } else {
        static_cast<float*>(a.hid)[row * a.h + n] = v;
      }
    }
    __syncthreads();   // red is written again
  }
}

// ------------------------------------------------------------------ phase 2 --
// the output element's bias terms and its one rounding
template <bool BF16>
__device__ __forceinline__ void write_out(const DecodeArgs& a, const Routing& r, int t, int n, float v) {
  if (a.b2 != nullptr) {
    float b = 0.f;
    for (int q = 0; q < a.k; ++q)
      b = fmaf(r.w[t][q], load1<BF16>(a.b2, static_cast<size_t>(r.idx[t][q]) * a.d + n), b);
    for (int q = 0; q < a.S; ++q) b += load1<BF16>(a.b2, static_cast<size_t>(a.E + q) * a.d + n);
    v += b;
  }
  const size_t o = static_cast<size_t>(t) * a.d + n;
  if (BF16) static_cast<uint16_t*>(a.out)[o] = f32_to_bf16(v);
  else static_cast<float*>(a.out)[o] = v;
}

// One item: 16 RT output columns from n0 over share sp of the summed range, all
// taken experts' k one after the other.  An expert's tokens are the activation
// rows (bf16: tiles of 8 tokens, rows 0..7 their hidden values, 8..15 the
// remainders; float32: tiles of 16), so an expert with one token costs one
// MFMA, and its sums go to its tokens only.  Each wave adds them to a table of
// its own in LDS, [T][16 RT]; the tables are added in wave order at the end.
template <Fmt F, int NT, int RT, int U, int TMAX>
__device__ void phase2_item(const DecodeArgs& a, Routing& r, float* tab, int* flag, int tile, int sp) {
  constexpr bool kBf = F != Fmt::kF32;
  constexpr int kTok = kBf ? 8 : 16;
  constexpr int kN = 16 * RT;
  const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
  const int n0 = tile * kN;
  const int nst = (a.h + step_k(F) - 1) / step_k(F);
  const int na = uniform(r.n);
  const int total = na * nst;   // at most 264 * 2^16
  const int share = sp * kWaves + wave, shares = a.split * kWaves;
  int f = static_cast<int>(static_cast<long long>(total) * share / shares);
  const int fend = static_cast<int>(static_cast<long long>(total) * (share + 1) / shares);
  float* mine = tab + wave * TMAX * kN;
  for (int i = lane; i < a.T * kN; i += 64) mine[i] = 0.f;
  const uint32_t pitch = static_cast<uint32_t>(a.h) * (kBf ? 2u : 4u);
  const uint32_t rowb = kBf ? 2u * pitch : pitch;
  const __amdgpu_buffer_rsrc_t hr =
      make_rsrc(a.hid, static_cast<uint32_t>(a.T) * static_cast<uint32_t>(a.k + a.S) * rowb);
  int ai = f / nst, s0 = f - ai * nst;
  while (f < fend) {
    const int s1 = min(nst, s0 + fend - f);
    const int e = uniform(r.list[ai]), o = uniform(r.off[ai]);
    const int rows = uniform(r.off[ai + 1]) - o;
    const WRows wr = rows_of<F, RT>(a.W2, e, n0, lane);
    for (int p0 = 0; p0 < rows; p0 += kTok * NT) {
      const int tl = min(NT, (rows - p0 + kTok - 1) / kTok);
      uint32_t arow[NT];
      floatx4 acc[NT][RT];
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        const int p = p0 + j * kTok + (lane & (kTok - 1));
        arow[j] = kOut;
        if (p < rows) {
          const int ts = r.row[o + p];
          arow[j] = (static_cast<uint32_t>(ts & 255) * (a.k + a.S) + (ts >> 8)) * rowb;
          if (kBf && (lane & 8)) arow[j] += pitch;
        }
#pragma unroll
        for (int i = 0; i < RT; ++i) acc[j][i] = floatx4{0.f, 0.f, 0.f, 0.f};
      }
      if (is_w4(F) && a.W2.z != nullptr) stream_rows<F, NT, RT, U, true, true>(acc, wr, hr, arow, tl, s0, s1, a.h, lane);
      else stream_rows<F, NT, RT, U, true, false>(acc, wr, hr, arow, tl, s0, s1, a.h, lane);
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        if (NT > 1 && j >= tl) break;
#pragma unroll
        for (int i = 0; i < RT; ++i)
#pragma unroll
          for (int m = 0; m < 4; ++m) {
            float v = acc[j][i][m];
            if (kBf) {   // values (lane quarters 0, 1) and remainders (2, 3)
              auto hl = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
              v = __uint_as_float(hl[0]) + __uint_as_float(hl[1]);
            }
            const int p = p0 + j * kTok + (lane >> 4) * 4 + m;
            if (p < rows && (!kBf || lane < 32)) mine[(r.row[o + p] & 255) * kN + i * 16 + (lane & 15)] += v;
          }
      }
    }
    f += s1 - s0;
    s0 = 0;
    ++ai;
  }
  __syncthreads();
  for (int i = threadIdx.x; i < a.T * kN; i += kThreads) {
    const int t = i / kN, n = n0 + i % kN;
    if (n >= a.d) continue;
    float v = 0.f;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) v += tab[w * TMAX * kN + i];
    if (a.split > 1) store_agent(a.part + (static_cast<size_t>(sp) * a.T + t) * a.d + n, v);
    else write_out<kBf>(a, r, t, n, v);
  }
  if (a.split > 1) {
    // the last share of the tile to arrive adds all of them, in share order
    stores_done();
    __syncthreads();
    if (threadIdx.x == 0) *flag = atomicAdd(&a.counters[tile], 1) == a.split - 1;
    __syncthreads();
    if (*flag) {
      for (int i = threadIdx.x; i < a.T * kN; i += kThreads) {
        const int t = i / kN, n = n0 + i % kN;
        if (n >= a.d) continue;
        float v = 0.f;
        for (int q = 0; q < a.split; ++q) v += load_agent(a.part + (static_cast<size_t>(q) * a.T + t) * a.d + n);
        write_out<kBf>(a, r, t, n, v);
      }
    }
  }
  __syncthreads();   // tab and flag are written again by the next item
}

#ifndef RTB
#define RTB 1
#endif
#ifndef RTW
#define RTW 4
#endif
#ifndef UB
#define UB 8
#endif
#ifndef UW
#define UW 4
#endif
#ifndef RTB2
#define RTB2 RTB
#endif
#ifndef RTW2
#define RTW2 RTW
#endif
#ifndef W4NT
#define W4NT 2
#endif
#ifndef RT64
#define RT64 1
#endif
#ifndef UW64
#define UW64 2
#endif
#ifndef WG1
#define WG1 2
#endif
#ifndef WG2
#define WG2 2
#endif
// Row tiles of a wave and the steps it loads together: 4 to 16 KB in flight.
template <Fmt F, int TMAX> struct Shape {
  static constexpr int kRT1 = TMAX > 16 ? (is_w4(F) ? RT64 : 1) : is_w4(F) ? RTW : RTB;
  static constexpr int kRT2 = TMAX > 16 ? (is_w4(F) ? RT64 : 1) : is_w4(F) ? RTW2 : RTB2;
  static constexpr int kB = TMAX > 16 ? (is_w4(F) ? UW64 : 4) : is_w4(F) ? UW : UB;
  static constexpr int kU1 = kB / kRT1 > 0 ? kB / kRT1 : 1;
  static constexpr int kU2 = kB / kRT2 > 0 ? kB / kRT2 : 1;
  // tiles of tokens at once; 4-bit: experts with more tokens are streamed again
  static constexpr int kNT1 = is_w4(F) ? (TMAX > 16 ? W4NT : 1) : (TMAX + 15) / 16;
  static constexpr int kNT2 = is_w4(F) ? kNT1 : F == Fmt::kF32 ? kNT1 : (TMAX + 7) / 8;
};

template <Fmt F, int TMAX>
__global__ __launch_bounds__(kThreads) void decode_phase1_kernel(DecodeArgs a) {
  using Sh = Shape<F, TMAX>;
  __shared__ Routing r;
  __shared__ float red[Sh::kNT1 * Sh::kRT1 * kWaves * 256];
  build_routing(a, r, blockIdx.x == 0);
  constexpr int kN = 16 * Sh::kRT1;
  const int ntile = (a.h + kN - 1) / kN;
  const int items = uniform(r.n) * ntile;
  for (int i = blockIdx.x; i < items; i += gridDim.x)
    phase1_item<F, Sh::kNT1, Sh::kRT1, Sh::kU1>(a, r, red, i / ntile, i % ntile * kN);
}

template <Fmt F, int TMAX>
__global__ __launch_bounds__(kThreads) void decode_phase2_kernel(DecodeArgs a) {
  using Sh = Shape<F, TMAX>;
  __shared__ Routing r;
  __shared__ float tab[kWaves * TMAX * 16 * Sh::kRT2];
  __shared__ int flag;
  load_routing(a, r);
  const int items = (a.d + 16 * Sh::kRT2 - 1) / (16 * Sh::kRT2) * a.split;
  for (int i = blockIdx.x; i < items; i += gridDim.x)
    phase2_item<F, Sh::kNT2, Sh::kRT2, Sh::kU2, TMAX>(a, r, tab, &flag, i / a.split, i % a.split);
}

template <Fmt F, int TMAX>
hipError_t launch_phases(const DecodeArgs& a, hipStream_t st) {
  const int cus = device_cu_count();
  decode_phase1_kernel<F, TMAX><<<cus * WG1, kThreads, 0, st>>>(a);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  decode_phase2_kernel<F, TMAX><<<cus * WG2, kThreads, 0, st>>>(a);
  return hipGetLastError();
}
template <Fmt F>
hipError_t launch_phases(const DecodeArgs& a, hipStream_t st) {
  if (a.T <= 8) return launch_phases<F, 8>(a, st);
  if (a.T <= 16) return launch_phases<F, 16>(a, st);
  return launch_phases<F, kMaxT>(a, st);
}

template <bool BF16>
void launch_logits(const DecodeArgs& a, hipStream_t st) {
  const int threads = a.d >= 8192 ? 1024 : (a.d / 8 + 63) / 64 * 64;
  if (a.T == 1) decode_logits_kernel<BF16, 1><<<dim3(a.E, 1), threads, 0, st>>>(a);
  else if (a.T <= 4) decode_logits_kernel<BF16, 4><<<dim3(a.E, 1), threads, 0, st>>>(a);
  else if (BF16) decode_logits_mfma_kernel<<<dim3((a.E + 15) / 16, (a.T + 15) / 16), 1024, 0, st>>>(a);
  else decode_logits_kernel<BF16, 16><<<dim3(a.E, (a.T + 15) / 16), threads, 0, st>>>(a);
}

template <Fmt F>
int row_tiles2(int T) {
  return T <= 8 ? Shape<F, 8>::kRT2 : T <= 16 ? Shape<F, 16>::kRT2 : Shape<F, kMaxT>::kRT2;
}

}  // namespace

// Shares of phase 2's sum per tile of output columns: as few as fill whole
// rounds of the grid, at least 32 KB of weights in each.
int decode_split(int T, int d, int h, int E, int k, int S, int fmt) {
  const int rt = fmt == kDecodeF32 ? row_tiles2<Fmt::kF32>(T) : fmt == kDecodeBf16 ? row_tiles2<Fmt::kBf16>(T)
                                                                                  : row_tiles2<Fmt::kW4g128>(T);
  const long long tiles = (d + 16 * rt - 1) / (16 * rt);
  long long used = static_cast<long long>(T) * k;
  if (used > E) used = E;
  used += S;
  const long long row_bytes = fmt == kDecodeF32 ? 4LL * h : fmt == kDecodeBf16 ? 2LL * h : h / 2;
  const long long bytes = used * 16 * rt * row_bytes;   // of one tile
  long long best = 1;
  double eff = 0;
  for (long long sp = 1; sp <= 64; ++sp) {
    if (sp > 1 && bytes / sp < 32768) break;
    const double rounds = static_cast<double>(tiles * sp) / (256 * WG2);
    const double full = rounds / static_cast<double>(static_cast<long long>(rounds + 0.999999));
    if (full > eff + 0.02) {
      eff = full;
      best = sp;
    }
  }
  return static_cast<int>(best);
}

hipError_t launch_decode(const DecodeArgs& a, hipStream_t st) {
  if (a.fmt == kDecodeF32) launch_logits<false>(a, st);
  else launch_logits<true>(a, st);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  if (a.fmt == kDecodeF32) return launch_phases<Fmt::kF32>(a, st);
  if (a.fmt == kDecodeBf16) return launch_phases<Fmt::kBf16>(a, st);
  if (a.W1.gshift == 5) return launch_phases<Fmt::kW4g32>(a, st);
  if (a.W1.gshift == 6) return launch_phases<Fmt::kW4g64>(a, st);
  return launch_phases<Fmt::kW4g128>(a, st);
}

}  // namespace moe
