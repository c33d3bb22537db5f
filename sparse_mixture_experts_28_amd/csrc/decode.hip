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
//   logits          float64 logits, the counters cleared
//   selection       over eight tokens, else in phase 1's workgroups
//   phase 1         per taken expert and 16 hidden units of a wave: act(W1 x + b1)
//                   times the routing weight
//   phase 2         per 16 or 32 output columns: the sum over all taken experts
//
// The routed weight is folded into the hidden rows in float32, and the hidden
// rows are kept to 16 bits of mantissa (bf16 layers: a bf16 number and its bf16
// remainder, which ride in the same 16-row MFMA operand as 8 + 8 rows), so the
// output carries one rounding, its own.
#include "few_rows.h"

#include <cmath>

namespace moe {
namespace {

constexpr int kWaves = 8;                 // waves of a phase workgroup; they split k
constexpr int kThreads = kWaves * kWave;
constexpr int kParts = 4;                 // parts of the logits' sums, where there are several
constexpr int kMaxT = MOE_MAX_DECODE_TOKENS;
constexpr int kMaxE = MOE_MAX_EXPERTS + MOE_MAX_SHARED;

// ------------------------------------------------------------------ logits --
// What the logits kernels leave besides the logits: zeroed counters for phase 2
// and, for 4-bit weights, x in the order of the codes.
__device__ __forceinline__ void prepare_phases(const DecodeArgs& a) {
  const int nth = gridDim.x * gridDim.y * gridDim.z * blockDim.x;
  const int id = ((blockIdx.z * gridDim.y + blockIdx.y) * gridDim.x + blockIdx.x) * blockDim.x + threadIdx.x;
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
// 16 waves and DecodeArgs::parts workgroups splitting d.  The float32 sums run over
// at most 256 elements and are added in float64.  One part would leave most CUs
// idle: 256 experts, d = 7168, 64 tokens 17 us, in four parts 8.
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
  const int slice = blockIdx.z * 16 + wave, slices = a.parts * 16;
  const int s0 = slice * nst / slices, s1 = (slice + 1) * nst / slices;
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
      if (a.b_g != nullptr && blockIdx.z == 0) l += static_cast<double>(a.b_g[e]);
      a.logits[(static_cast<size_t>(blockIdx.z) * a.T + t) * a.E + e] = l;
    }
  }
  prepare_phases(a);
}

// --------------------------------------------------------------- selection --
// The routing of the call, rebuilt by every workgroup from the logits (a few
// hundred numbers per token) rather than passed through another launch.  A job
// is an expert with up to so many of its tokens as the kernel takes at once; the
// work is shared out by jobs, so an expert with many tokens (a shared one) does
// not hold up the wave that meets it.
constexpr int kMaxRows = kMaxT * (MOE_MAX_TOPK + MOE_MAX_SHARED);
constexpr int kMaxJobs = kMaxE + kMaxRows / 8;
struct Routing {
  int idx[kMaxT][MOE_MAX_TOPK];     // expert of slot j, routed slots only
  float w[kMaxT][MOE_MAX_TOPK];
  unsigned long long mask[kMaxE];   // tokens of each expert
  uint16_t list[kMaxJobs];          // expert of each job, ascending, shared ones last
  uint16_t off[kMaxJobs + 1];       // first of its rows
  uint16_t start[kMaxE];            // first row of each expert
  uint16_t row[kMaxRows];           // token + 256 slot, ascending tokens; slot k + s: shared s
  int n;                            // jobs
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
__device__ __forceinline__ void select_token(const DecodeArgs& a, int t, int lane, int& my_idx, float& my_w) {
  double key[4], val[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int e = lane + 64 * i;
    val[i] = e < a.E ? a.logits[static_cast<size_t>(t) * a.E + e] : 0.0;
    if (a.parts > 1 && e < a.E)
#pragma unroll
      for (int p = 1; p < kParts; ++p) val[i] += a.logits[(static_cast<size_t>(p) * a.T + t) * a.E + e];
    double kv = val[i];
    if (a.b_sel != nullptr && e < a.E) kv += static_cast<double>(a.b_sel[e]);
    key[i] = kv == kv ? kv : -INFINITY;
  }
  uint32_t left = 0;   // bit i: expert lane + 64 i is there and not taken
#pragma unroll
  for (int i = 0; i < 4; ++i) left |= lane + 64 * i < a.E ? 1u << i : 0u;
  my_idx = 0;
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
  my_w = ej / sum;   // lane j: slot j
}

__device__ __forceinline__ void write_choice(const DecodeArgs& a, int t, int lane, int idx, float w) {
  if (lane < a.k) {
    a.topk_idx[t * a.k + lane] = idx;
    a.topk_w[t * a.k + lane] = w;
  }
}

// One wave per token, for batches whose selection would keep every workgroup of
// phase 1 busy for long.
__global__ __launch_bounds__(64) void decode_select_kernel(DecodeArgs a) {
  int idx;
  float w;
  select_token(a, blockIdx.x, threadIdx.x, idx, w);
  write_choice(a, blockIdx.x, threadIdx.x, idx, w);
}

// The jobs and their rows from idx, PER tokens at most to a job.
template <int PER>
__device__ __forceinline__ void list_routing(const DecodeArgs& a, Routing& r) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, e = threadIdx.x;
  const int ne = a.E + a.S, na = a.T * a.k;   // at most 264 experts (a thread each), 512 choices
  if (a.T == 1) {   // the order of the experts is free: slot order
    const int n = a.k + a.S;
    __syncthreads();
    if (e <= n) {
      r.list[e] = static_cast<uint16_t>(e < a.k ? r.idx[0][e] : a.E + e - a.k);
      r.off[e] = static_cast<uint16_t>(e);
      r.row[e] = static_cast<uint16_t>(e << 8);
    }
    if (e == 0) r.n = n;
    __syncthreads();
    return;
  }
  if (e < ne) r.mask[e] = e < a.E ? 0ull : a.T == 64 ? ~0ull : (1ull << a.T) - 1ull;
  __syncthreads();
  const int t = e / a.k, j = e - t * a.k;     // the thread's choice
  const int mine = e < na ? r.idx[t][j] : 0;
  if (e < na) atomicOr(&r.mask[mine], 1ull << t);   // a set: the order does not matter
  __syncthreads();
  const int cnt = e < ne ? __popcll(r.mask[e]) : 0;
  // prefix sums of (jobs, rows), in two halves of a word
  const uint32_t own = (static_cast<uint32_t>((cnt + PER - 1) / PER) << 16) + cnt;
  uint32_t sc = own;
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const uint32_t up = __shfl_up(sc, o);
    if (lane >= o) sc += up;
  }
  if (lane == 63) r.wsum[wave] = sc;
  __syncthreads();
  uint32_t before = sc - own, total = 0;
#pragma unroll
  for (int w = 0; w < kWaves; ++w) {
    const uint32_t v = r.wsum[w];
    if (w < wave) before += v;
    total += v;
  }
  const int o = before & 0xffffu;
  for (int i = 0, pos = before >> 16; i < cnt; i += PER, ++pos) {
    r.list[pos] = static_cast<uint16_t>(e);
    r.off[pos] = static_cast<uint16_t>(o + i);
  }
  if (e < ne) r.start[e] = static_cast<uint16_t>(o);
  if (e == 0) {
    r.n = total >> 16;
    r.off[total >> 16] = static_cast<uint16_t>(total & 0xffffu);
  }
  __syncthreads();
  // a choice's row: behind the expert's earlier tokens
  if (e < na) {
    const int at = r.start[mine] + __popcll(r.mask[mine] & ((1ull << t) - 1ull));
    r.row[at] = static_cast<uint16_t>(t | (j << 8));
  }
  for (int i = e; i < a.S * a.T; i += kThreads) {
    const int s = i / a.T, ts = i - s * a.T;
    r.row[r.start[a.E + s] + ts] = static_cast<uint16_t>(ts | ((a.k + s) << 8));
  }
  __syncthreads();
}

// from the logits, a wave per token (T <= kWaves)
template <int PER>
__device__ __forceinline__ void build_routing(const DecodeArgs& a, Routing& r, bool write) {
  const int lane = threadIdx.x & 63, t = threadIdx.x >> 6;
  if (t < a.T) {
    int idx;
    float w;
    select_token(a, t, lane, idx, w);
    if (lane < a.k) {
      r.idx[t][lane] = idx;
      r.w[t][lane] = w;
    }
    if (write) write_choice(a, t, lane, idx, w);
  }
  list_routing<PER>(a, r);
}

// from the experts and weights in the outputs
template <int PER>
__device__ __forceinline__ void load_routing(const DecodeArgs& a, Routing& r) {
  const int i = threadIdx.x, t = i / a.k, j = i - t * a.k;
  if (i < a.T * a.k) {
    r.idx[t][j] = a.topk_idx[i];
    r.w[t][j] = a.topk_w[i];
  }
  list_routing<PER>(a, r);
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

// Items of a phase go to its workgroups in turn or, where a workgroup has
// megabytes to read (DecodeArgs::dynamic), as they come free: the first by number,
// the others by a counter, asked for while the item before is under way.  Waves
// see memory at uneven rates, and jobs with many tokens cost more: in turn, the
// second phase of the DeepSeek-shaped layer (32 tokens) took 1030 us, its
// workgroups ending between 605 and 1106; by the counter 825.  Short items lose:
// the counter's answer arrives among the weight loads (Mixtral shape, one token,
// 128 KB items: 42.9 us in turn, 46.7 by the counter).
struct Tickets {
  int32_t* counter;
  int* slot;       // two words of LDS, used in turn
  bool dynamic;
  int turn, next;
  __device__ __forceinline__ void ask(int i) {
    next = i + gridDim.x;
    if (dynamic && threadIdx.x == 0) next = gridDim.x + atomicAdd(counter, 1);
  }
  // between ask() and take(), before a barrier
  __device__ __forceinline__ void publish() {
    if (threadIdx.x == 0) slot[turn] = next;
  }
  __device__ __forceinline__ int take() {
    const int i = slot[turn];
    turn ^= 1;
    return uniform(i);
  }
};

// Shapes of the phase kernels by format, token class (1, up to 16 and up to 64
// tokens) and, bf16, whether the experts have many tokens each (DENSE: eight and
// more on average, over 16 tokens): steps loaded together, tiles of tokens at once
// (an expert with more makes several jobs), tiles of 16 weight rows of a wave,
// workgroups of eight waves per CU (two: 128 registers a wave, one: 256), bytes of
// a wave's activation region.  Measured, phase 1 + phase 2 in us:
//   steps    bf16, one token of the Mixtral shape: 2 + 2 steps 47 + 45, 4 + 4 43 +
//            46, 4 + 2 a batch ahead 43 + 44, 8 + 8 44 + 50; 4-bit: 2 + 2 steps 22 +
//            21, 4 + 4 21 + 20
//   WGs      three per CU: 43 + 44 becomes 49 + 53 (one token, Mixtral shape)
//   one WG and two row tiles, where a wave multiplies for longer than it loads:
//     4-bit phase 2 of several tokens: 49 -> 36 (5 tokens, 46 experts, groups of
//     32), 77 -> 45 (18 tokens, 6 experts, groups of 32), the DeepSeek shape's 64
//     tokens 1249 -> 1160 for the layer; phase 1 loses (8 tokens, Mixtral shape: 71
//     -> 81)
//     DENSE, layer, Mixtral shape: 64 tokens 643 -> 512, 32 tokens 460 -> 437; 45
//     tokens of 2 + 1 experts 402 -> 242 (tiles for 48 tokens: no weight is read
//     twice); with few tokens per expert it loses (32 tokens of the DeepSeek
//     shape 1638 -> 1757), as does float32 (728 -> 818)
template <Fmt F, int TMAX, bool DENSE> struct Shape {
  static constexpr bool kW = is_w4(F), kMany = TMAX > 16;
  static constexpr bool kWide2 = DENSE || (kW && TMAX > 1);
  static constexpr int kRT1 = DENSE ? 2 : 1, kWgs1 = DENSE ? 1 : 2;
  static constexpr int kRT2 = kWide2 ? 2 : 1, kWgs2 = kWide2 ? 1 : 2;
  static constexpr int kU1 = 4, kU2 = kW && !(kWide2 && group_shift(F) == 5) ? 4 : 2;
  static constexpr bool kAhead2 = !kW && !kMany;
  static constexpr int kNT1 = DENSE ? 3 : !kMany || kW ? 1 : 2;
  static constexpr int kNT2 = DENSE ? 6 : kW ? 1 : F == Fmt::kF32 ? kNT1 : TMAX == 1 ? 1 : TMAX == 16 ? 2 : 3;
  static constexpr int kRows1 = TMAX == 1 ? 1 : 16 * kNT1, kRows2 = TMAX == 1 ? (F == Fmt::kF32 ? 1 : 2) : 16 * kNT2;
  static constexpr int kStep = kW ? 256 : 64;
  static constexpr int stage(int rows) {
    return (TMAX == 1 ? (kW ? 2048 : 1024) : rows * (kStep + 16)) + 32 + stage_zero(F);
  }
  static constexpr int kStage1 = stage(kRows1) + (DENSE ? 2048 : 0);
  static constexpr int kStage2 = stage(kRows2) + (kWide2 && !DENSE ? 4352 : 0);
};

// a segment's products for one tile of tokens or for all NT (the others then
// hold rows whose sums nobody reads)
template <int NT, int RT, typename St>
__device__ __forceinline__ void run_tiles(St& st, floatx4 (&acc)[NT][RT], __amdgpu_buffer_rsrc_t a,
                                          const int (&rslot)[NT], int tl, char* stage, int lane) {
#pragma unroll
  for (int j = 0; j < NT; ++j)
#pragma unroll
    for (int i = 0; i < RT; ++i) acc[j][i] = floatx4{0.f, 0.f, 0.f, 0.f};
  if (NT > 1 && tl == 1) {
    floatx4 one[1][RT];
    const int rs[1] = {rslot[0]};
#pragma unroll
    for (int i = 0; i < RT; ++i) one[0][i] = acc[0][i];
    st.run(one, a, rs, stage, lane);
#pragma unroll
    for (int i = 0; i < RT; ++i) acc[0][i] = one[0][i];
  } else {
    st.run(acc, a, rslot, stage, lane);
  }
}

// ------------------------------------------------------------------ phase 1 --
// One item: a job and hidden units, 16 for each group of KS waves.  The job's
// tokens are the activation rows, NT tiles of 16; a group's waves split k and add
// their sums in LDS in wave order.  The next item's first loads are issued before
// this one's sums, biases, activations and stores.  Bound by memory: the Mixtral
// shape with one token 43 us (235 MB, 5.5 TB/s), the DeepSeek shape with 32 745 us
// (4.5 GB, 6.0 TB/s); 4-bit with several tokens by vector operations (64 tokens
// of the DeepSeek shape: 520 us, 3.5 TB/s).
template <Fmt F, int TMAX, bool DENSE>
__global__ __launch_bounds__(kThreads, (2 * Shape<F, TMAX, DENSE>::kWgs1)) void decode_phase1_kernel(DecodeArgs a) {
  using Sh = Shape<F, TMAX, DENSE>;
  constexpr bool kBf = F != Fmt::kF32;
  constexpr int NT = Sh::kNT1, RT = Sh::kRT1, U = Sh::kU1;
  const int KS = a.ksplit, kN = 16 * RT * (kWaves / KS);   // waves that split k; hidden units of an item
  using St = Stream<F, RT, U, false, true, Sh::kRows1, Sh::kStage1>;
  __shared__ Routing r;
  __shared__ float red[NT * RT * kWaves * 256];
  __shared__ __attribute__((aligned(16))) char stages[kWaves][Sh::kStage1];
  __shared__ int next[2];
  const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
  char* stage = stages[wave];
  St::clear(stage, lane);
  if (TMAX <= 16 && a.T <= kWaves) build_routing<16 * NT>(a, r, blockIdx.x == 0);
  else load_routing<16 * NT>(a, r);

  const int ntile = (a.h + kN - 1) / kN;
  const int items = uniform(r.n) * ntile;
  const int nst = (a.d + step_k(F) - 1) / step_k(F), nb = (nst + U - 1) / U;
  const int ks = wave % KS, s0 = ks * nb / KS * U, s1 = min(nst, (ks + 1) * nb / KS * U);
  const uint32_t pitch = static_cast<uint32_t>(a.d) * act_bytes(F);
  const __amdgpu_buffer_rsrc_t xr = make_rsrc(is_w4(F) ? a.xord : a.x, static_cast<uint32_t>(a.T) * pitch);
  Tickets tk{a.counters, next, a.dynamic != 0, 0, 0};
  St st;
  int e = 0, n0 = 0, o = 0, rows = 0;   // the item's expert, first hidden unit, first row and rows
  auto soff = [&](int slot) { return static_cast<uint32_t>(r.row[o + slot] & 255) * pitch; };
  auto begin = [&](int item) {
    const int job = item / ntile;
    e = uniform(r.list[job]);
    n0 = (item - job * ntile) * kN;
    o = uniform(r.off[job]);
    rows = uniform(r.off[job + 1]) - o;
    const int nw = n0 + wave / KS * 16 * RT;   // the wave's own rows; none past the last
    st.begin(rows_of<F, RT>(a.W1, e, min(nw, a.h), lane), xr, soff, rows, s0, nw < a.h ? s1 : s0, a.d, lane);
  };
  int item = blockIdx.x;
  if (item < items) begin(item);
  while (item < items) {
    tk.ask(item);
    const int tl = (rows + 15) / 16;
    int rslot[NT];
#pragma unroll
    for (int j = 0; j < NT; ++j) rslot[j] = min(j * 16 + (lane & 15), rows - 1);
    floatx4 acc[NT][RT];
    run_tiles(st, acc, xr, rslot, tl, stage, lane);
#pragma unroll
    for (int j = 0; j < NT; ++j)
      if (j < tl) {
#pragma unroll
        for (int i = 0; i < RT; ++i)
          *reinterpret_cast<floatx4*>(red + (((j * RT + i) * kWaves + wave) * 64 + lane) * 4) = acc[j][i];
      }
    tk.publish();
    __syncthreads();
    const int ce = e, cn0 = n0, co = o, crows = rows;
    item = tk.take();
    if (item < items) begin(item);
    for (int i = threadIdx.x; i < tl * 16 * kN; i += kThreads) {
      // result (row p of the job's tokens, hidden unit n): waves wg KS .., lane (n, p /
      // 4 % 4), register p % 4
      const int rt16 = i >> 8, j = rt16 / (kN / 16), wr = rt16 - j * (kN / 16), wg = wr / RT, rt = wr % RT;
      const int n = cn0 + wr * 16 + (i & 15), pr = (i >> 4) & 15, p = j * 16 + pr;
      if (p >= crows || n >= a.h) continue;
      const float* sum = red + (((j * RT + rt) * kWaves + wg * KS) * 64 + (pr >> 2) * 16 + (i & 15)) * 4 + (pr & 3);
      float v = 0.f;
      // unrolled, so that the loads are under way together (in a loop the 4-bit
      // Mixtral-shaped layer takes 47 us for one token instead of 44)
      if (KS == kWaves) {
#pragma unroll
        for (int w = 0; w < kWaves; ++w) v += sum[w * 256];
      } else {
#pragma unroll
        for (int w = 0; w < kWaves / 2; ++w) {
          const float p = sum[min(w, KS - 1) * 256];
          v += w < KS ? p : 0.f;
        }
      }
      if (a.b1 != nullptr) v += load1<kBf>(a.b1, static_cast<size_t>(ce) * a.h + n);
      v = a.act == MOE_ACT_SILU ? v / (1.f + expf(-v)) : 0.5f * v * (1.f + erff(v * 0.70710678118654752440f));
      const int t = r.row[co + p] & 255, slot = r.row[co + p] >> 8;
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
    __syncthreads();   // red is written again by the next item
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

// One item: 16 RT output columns over a share of the summed range, all jobs' k
// one after the other.  A job's tokens are the activation rows (bf16: tiles of 8
// tokens, rows 0..7 their hidden values, 8..15 the remainders; float32: tiles of
// 16), so an expert with one token costs one MFMA, and its sums go to its tokens
// only.  Each wave adds them to a table of its own in LDS, [T][16 RT]; the tables
// are added in wave order at the end.  Loads run ahead as in phase 1: the next
// job's before a job's sums, the next item's before an item's.  Bound as phase 1:
// 43 us, 783 us, and 4-bit 653 us.
template <Fmt F, int TMAX, bool DENSE>
__global__ __launch_bounds__(kThreads, (2 * Shape<F, TMAX, DENSE>::kWgs2)) void decode_phase2_kernel(DecodeArgs a) {
  using Sh = Shape<F, TMAX, DENSE>;
  constexpr bool kBf = F != Fmt::kF32;
  constexpr int kTok = kBf ? 8 : 16;
  constexpr int NT = Sh::kNT2, RT = Sh::kRT2, U = Sh::kU2, kN = 16 * RT;
  using St = Stream<F, RT, U, Sh::kAhead2, true, Sh::kRows2, Sh::kStage2>;
  __shared__ Routing r;
  __shared__ float tab[kWaves][TMAX * kN];
  __shared__ __attribute__((aligned(16))) char stages[kWaves][Sh::kStage2];
  __shared__ int next[2];
  __shared__ int flag;
  const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
  char* stage = stages[wave];
  float* mine = tab[wave];
  St::clear(stage, lane);
  load_routing<kTok * NT>(a, r);

  const int tiles = (a.d + kN - 1) / kN;
  const int items = tiles * a.split;
  const int nst = (a.h + step_k(F) - 1) / step_k(F), nb = (nst + U - 1) / U;   // steps and batches of a job
  const int total = uniform(r.n) * nb;   // at most 392 * 2^16
  const int shares = a.split * kWaves;
  const uint32_t pitch = static_cast<uint32_t>(a.h) * act_bytes(F);
  const uint32_t rowb = kBf ? 2u * pitch : pitch;
  const __amdgpu_buffer_rsrc_t hr =
      make_rsrc(a.hid, static_cast<uint32_t>(a.T) * static_cast<uint32_t>(a.k + a.S) * rowb);
  Tickets tk{a.counters + 1, next, a.dynamic != 0, 0, 0};
  St st;
  int n0 = 0, f = 0, fend = 0;            // the item's first column; the wave's batches left of it
  int job = 0, b0 = 0, o = 0, rows = 0;   // the segment's job, first batch, first row and rows
  auto soff = [&](int slot) {
    const int p = kBf && slot >= rows ? slot - rows : slot;
    const int ts = r.row[o + p];
    return (static_cast<uint32_t>(ts & 255) * (a.k + a.S) + (ts >> 8)) * rowb + (p != slot ? pitch : 0u);
  };
  auto begin = [&]() {   // the segment of job `job` from batch b0 on
    const int n = min(nb - b0, fend - f);
    f += n;
    o = uniform(r.off[job]);
    rows = uniform(r.off[job + 1]) - o;
    st.begin(rows_of<F, RT>(a.W2, uniform(r.list[job]), n0, lane), hr, soff, kBf ? 2 * rows : rows, b0 * U,
             min(nst, (b0 + n) * U), a.h, lane);
  };
  auto begin_item = [&](int item) {
    const int sp = item / tiles;
    n0 = (item - sp * tiles) * kN;
    const int share = sp * kWaves + wave;
    f = static_cast<int>(static_cast<long long>(total) * share / shares);
    fend = static_cast<int>(static_cast<long long>(total) * (share + 1) / shares);
    job = f / nb;
    b0 = f - job * nb;
    if (f < fend) begin();
    else rows = 0;
  };
  int item = blockIdx.x;
  if (item < items) begin_item(item);
  while (item < items) {
    tk.ask(item);
    for (int i = lane; i < a.T * kN; i += 64) mine[i] = 0.f;
    while (rows > 0) {
      const int tl = (rows + kTok - 1) / kTok;
      int rslot[NT];
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        rslot[j] = min(j * kTok + (lane & (kTok - 1)), rows - 1);
        if (kBf && (lane & 8)) rslot[j] += rows;
      }
      floatx4 acc[NT][RT];
      run_tiles(st, acc, hr, rslot, tl, stage, lane);
      const int co = o, crows = rows;
      rows = 0;
      if (f < fend) {
        ++job;
        b0 = 0;
        begin();
      }
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
            const int p = j * kTok + (lane >> 4) * 4 + m;
            if (p < crows && (!kBf || lane < 32)) mine[(r.row[co + p] & 255) * kN + i * 16 + (lane & 15)] += v;
          }
      }
    }
    tk.publish();
    __syncthreads();
    const int cn0 = n0, sp = item / tiles, tile = item - sp * tiles;
    item = tk.take();
    if (item < items) begin_item(item);
    for (int i = threadIdx.x; i < a.T * kN; i += kThreads) {
      const int t = i / kN, n = cn0 + i % kN;
      if (n >= a.d) continue;
      float v = 0.f;
#pragma unroll
      for (int w = 0; w < kWaves; ++w) v += tab[w][i];
      if (a.split > 1) store_agent(a.part + (static_cast<size_t>(sp) * a.T + t) * a.d + n, v);
      else write_out<kBf>(a, r, t, n, v);
    }
    if (a.split > 1) {
      // the last share of the tile to arrive adds all of them, in share order
      stores_done();
      __syncthreads();
      if (threadIdx.x == 0) flag = atomicAdd(&a.counters[2 + tile], 1) == a.split - 1;
      __syncthreads();
      if (flag) {
        for (int i = threadIdx.x; i < a.T * kN; i += kThreads) {
          const int t = i / kN, n = cn0 + i % kN;
          if (n >= a.d) continue;
          float v = 0.f;
          for (int q0 = 0; q0 < a.split; q0 += 8) {   // eight loads in flight
            float p[8];
#pragma unroll
            for (int q = 0; q < 8; ++q)
              p[q] = load_agent(a.part + (static_cast<size_t>(min(q0 + q, a.split - 1)) * a.T + t) * a.d + n);
#pragma unroll
            for (int q = 0; q < 8; ++q) v += q0 + q < a.split ? p[q] : 0.f;
          }
          write_out<kBf>(a, r, t, n, v);
        }
      }
    }
    __syncthreads();   // tab and flag are written again by the next item
  }
}

// F: the format without zero points, Z: with them (the same where there are none)
template <Fmt F, Fmt Z, int TMAX, bool DENSE>
hipError_t launch_phases(const DecodeArgs& a, hipStream_t st) {
  const int grid = device_cu_count() * Shape<F, TMAX, DENSE>::kWgs1, grid2 = device_cu_count() * Shape<F, TMAX, DENSE>::kWgs2;
  if (a.T > kWaves) decode_select_kernel<<<a.T, 64, 0, st>>>(a);
  if (a.W1.z != nullptr) decode_phase1_kernel<Z, TMAX, DENSE><<<grid, kThreads, 0, st>>>(a);
  else decode_phase1_kernel<F, TMAX, DENSE><<<grid, kThreads, 0, st>>>(a);
  const hipError_t e = hipGetLastError();   // of either launch: a failed one is remembered
  if (e != hipSuccess) return e;
  if (a.W2.z != nullptr) decode_phase2_kernel<Z, TMAX, DENSE><<<grid2, kThreads, 0, st>>>(a);
  else decode_phase2_kernel<F, TMAX, DENSE><<<grid2, kThreads, 0, st>>>(a);
  return hipGetLastError();
}
template <Fmt F, Fmt Z>
hipError_t launch_phases(const DecodeArgs& a, hipStream_t st) {
  if (a.T == 1) return launch_phases<F, Z, 1, false>(a, st);
  if (a.T <= 16) return launch_phases<F, Z, 16, false>(a, st);
  return launch_phases<F, Z, kMaxT, false>(a, st);
}

template <bool BF16>
void launch_logits(const DecodeArgs& a, hipStream_t st) {
  const int threads = a.d >= 8192 ? 1024 : (a.d / 8 + 63) / 64 * 64;
  if (a.T == 1) decode_logits_kernel<BF16, 1><<<dim3(a.E, 1), threads, 0, st>>>(a);
  else if (a.T <= 4) decode_logits_kernel<BF16, 4><<<dim3(a.E, 1), threads, 0, st>>>(a);
  else if (BF16) decode_logits_mfma_kernel<<<dim3((a.E + 15) / 16, (a.T + 15) / 16, a.parts), 1024, 0, st>>>(a);
  else decode_logits_kernel<BF16, 16><<<dim3(a.E, (a.T + 15) / 16), threads, 0, st>>>(a);
}

}  // namespace

// How a call's work is shared out; from the sizes alone, with the experts that
// are taken when T tokens take k of E evenly.
//   split    phase 2: shares of the sum per tile of output columns: as many as fill
//            one round of the grid, or of 1 MB where that makes three rounds and
//            more (a second round that is mostly empty is the worst of both); of
//            32 KB at least, 64 at most
//   dynamic  2 MB or more to read per workgroup and phase
//   ksplit   phase 1: waves that split k, the others take rows of their own: all
//            eight, but no more than there are batches, and fewer while a wave has
//            less than four batches and the items still make two rounds (4-bit, 64
//            tokens of the DeepSeek shape, 14 batches: 8 waves 597 us, 4 536, 2 502;
//            4-bit, d = 1024, two batches: 8 waves leave six without work)
//   dense    bf16: over 16 tokens, eight and more to an expert
//   parts    parts of each logit's sum, added by the selection
DecodePlan decode_plan(int T, int d, int h, int E, int k, int S, int fmt) {
  const double used = E * (1.0 - std::pow(1.0 - static_cast<double>(k) / E, T)) + S;
  const double elem = fmt == kDecodeF32 ? 4.0 : fmt == kDecodeBf16 ? 2.0 : 0.5;
  const bool dense = fmt == kDecodeBf16 && T > 16 && T * k >= 8 * E;
  const int rt1 = dense ? 2 : 1, rt = dense || (fmt == kDecodeW4 && T > 1) ? 2 : 1;   // row tiles of a wave
  const int tiles = (d + 16 * rt - 1) / (16 * rt);
  const double tile_bytes = used * 16 * rt * h * elem;
  const int slots1 = 512 / rt1, slots = 512 / rt;   // workgroups of phase 1 and 2
  int sp = tiles < slots ? slots / tiles : 1;
  const double by_size = tile_bytes / (1 << 20);
  if (by_size >= 3.0 * sp) sp = by_size < 64.0 ? static_cast<int>(by_size) : 64;
  const double most = tile_bytes / 32768;
  if (sp > most) sp = most < 1.0 ? 1 : static_cast<int>(most);
  if (sp > 64) sp = 64;
  const int step = fmt == kDecodeF32 ? 16 : fmt == kDecodeBf16 ? 32 : 128;
  const int nb = ((d + step - 1) / step + 3) / 4;   // batches of four steps
  int ks = kWaves;
  while (ks > 1 && ks > nb) ks >>= 1;
  while (ks > 1 && nb / ks < 4 && used * h / (16. * rt1 * (2 * kWaves / ks)) >= 2.0 * slots1) ks >>= 1;
  const int parts = fmt != kDecodeF32 && T > 4 && d >= 1024 ? kParts : 1;
  return DecodePlan{sp, used * d * h * elem >= (2 << 20) * static_cast<double>(slots1) ? 1 : 0, ks, dense ? 1 : 0, parts};
}

hipError_t launch_decode(const DecodeArgs& a, hipStream_t st) {
  if (a.fmt == kDecodeF32) launch_logits<false>(a, st);
  else launch_logits<true>(a, st);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  if (a.fmt == kDecodeF32) return launch_phases<Fmt::kF32, Fmt::kF32>(a, st);
  if (a.fmt == kDecodeBf16 && a.dense) return launch_phases<Fmt::kBf16, Fmt::kBf16, kMaxT, true>(a, st);
  if (a.fmt == kDecodeBf16) return launch_phases<Fmt::kBf16, Fmt::kBf16>(a, st);
  if (a.W1.gshift == 5) return launch_phases<Fmt::kW4g32, Fmt::kW4g32z>(a, st);
  if (a.W1.gshift == 6) return launch_phases<Fmt::kW4g64, Fmt::kW4g64z>(a, st);
  return launch_phases<Fmt::kW4g128, Fmt::kW4g128z>(a, st);
}

}  // namespace moe
