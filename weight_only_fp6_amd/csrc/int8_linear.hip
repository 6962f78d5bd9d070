// 8-bit integer linear layer for gfx950: the token quantiser, the int8 MFMA
// product with a scale for each token and channel, and their entry points
// (fp6_int8.h).

#include <hip/hip_runtime.h>

#include <cstdint>
#include <type_traits>

#include "fp6_int8.h"
#include "fp6_limits.h"
#include "fpx_cus.h"

namespace {

typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef float float4v __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

int launch(const void* kern, dim3 grid, dim3 block, void** args, hipStream_t stream) {
  return hipLaunchKernel(kern, grid, block, args, 0, stream) == hipSuccess ? FP6_OK : FP6_E_HIP;
}

// ---------------------------------------------------------------------------
// Element types.
// ---------------------------------------------------------------------------
template <int DT>
struct Elem;
template <>
struct Elem<FP6_FP16> {
  using T = _Float16;
  __device__ static float to_float(uint32_t bits) {
    return static_cast<float>(__builtin_bit_cast(_Float16, static_cast<uint16_t>(bits)));
  }
};
template <>
struct Elem<FP6_BF16> {
  using T = __bf16;
  __device__ static float to_float(uint32_t bits) { return __builtin_bit_cast(float, bits << 16); }
};

// ---------------------------------------------------------------------------
// Token quantiser.
//
// q = RNE(127 x / a), a the row's largest magnitude.  With y = x * (127 / a)
// in fp32, |y - 127x/a| < 1.5 * 2^-23 |y|.  x and a have at most 11 significant
// bits, so 127x/a is either exactly halfway between two integers or at least
// 2^-19 of itself away from it (|254 X - (2n+1) A 2^s| >= 1 with X < 2^11).
// Rounding y to 21 bits (half a step there: 2^-21) therefore puts ties exactly
// on the tie and never moves another value onto or across one; RNE of that is
// the exact quotient's rounding, at two integer operations instead of an IEEE
// division per element.
// ---------------------------------------------------------------------------
__device__ __forceinline__ int quant1(float x, float r) {
  const uint32_t b = __builtin_bit_cast(uint32_t, x * r);
  return static_cast<int>(__builtin_rintf(__builtin_bit_cast(float, (b + 4u) & ~7u)));
}

struct RowScale {
  float up, r, s;  // q = quant1(x * up, r); s = the row's scale
};

// top: the row's largest |x| as fp32 bits (an integer maximum of the bits, in
// which infinities and NaN are larger than every finite value).
__device__ __forceinline__ RowScale row_scale_of(uint32_t top) {
  RowScale o;
  const float a = __builtin_bit_cast(float, top);
  o.up = 1.0f;
  if (top >= 0x7F800000u) {
    o.r = 0.0f;
    o.s = __builtin_nanf("");
    o.up = 0.0f;
  } else if (top == 0u) {
    o.r = 0.0f;
    o.s = 0.0f;
  } else {
    // Rows of bf16 values so small that 127 / a would overflow are scaled up first.
    if (a < 0x1p-100f) o.up = 0x1p64f;
    o.r = 127.0f / (a * o.up);
    o.s = a / 127.0f;
  }
  return o;
}

__device__ __forceinline__ uint32_t pack4(int a, int b, int c, int d) {
  return (a & 0xFF) | ((b & 0xFF) << 8) | ((c & 0xFF) << 16) | (static_cast<uint32_t>(d) << 24);
}

// A row per wave (WAVES == 1, four rows per workgroup) or per workgroup of four
// waves.  A thread's units of 8 elements (16 bytes, at any 2-byte alignment)
// stay in registers between the maximum and the codes for rows of up to 8 *
// UNITS * 64 * WAVES elements; longer rows (UNITS == 0) are read twice, the
// second time from the caches.  Bound by the bytes of X and of the codes:
// 4096x8192 bf16 18.6 us, 5.4 TB/s (25.1 us with a second read; rows that start
// at odd elements 18.8 us, 64 us read element by element).
typedef u32x4 u32x4_any __attribute__((aligned(2)));

template <int DT, int UNITS, int WAVES>
__global__ __launch_bounds__(256) void i8_quantize(const uint16_t* __restrict__ X, int64_t ldx, int64_t M, int K, int kp,
                                                   int8_t* __restrict__ Q, float* __restrict__ scales) {
  __shared__ uint32_t wtop[4];
  constexpr int kThreads = 64 * WAVES;
  const int tid = WAVES == 1 ? threadIdx.x & 63 : threadIdx.x;
  const int64_t m = WAVES == 1 ? static_cast<int64_t>(blockIdx.x) * 4 + (threadIdx.x >> 6) : blockIdx.x;
  if (m >= M) return;  // WAVES == 1: no barrier below
  const uint16_t* x = X + m * ldx;
  const int units = kp >> 3;
  auto load = [&](int u) -> u32x4 {
    u32x4 v = {0, 0, 0, 0};
    if (8 * u + 8 <= K) {
      v = *reinterpret_cast<const u32x4_any*>(x + 8 * u);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int k = 8 * u + 2 * i;
        v[i] = (k < K ? x[k] : 0u) | (k + 1 < K ? static_cast<uint32_t>(x[k + 1]) << 16 : 0u);
      }
    }
    return v;
  };
  uint32_t top = 0;
  auto look = [&](const u32x4& v) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t lo = v[i] & 0x7FFFu, hi = (v[i] >> 16) & 0x7FFFu;
      top = lo > top ? lo : top;
      top = hi > top ? hi : top;
    }
  };
  u32x4 held[UNITS > 0 ? UNITS : 1];
  if constexpr (UNITS > 0) {
#pragma unroll
    for (int i = 0; i < UNITS; ++i) {
      const int u = tid + i * kThreads;
      held[i] = u < units ? load(u) : u32x4{0, 0, 0, 0};
    }
#pragma unroll
    for (int i = 0; i < UNITS; ++i) look(held[i]);
  } else {
    for (int u = tid; u < units; u += kThreads) look(load(u));
  }
#pragma unroll
  for (int d = 32; d > 0; d >>= 1) {
    const uint32_t o = __shfl_xor(top, d);
    top = o > top ? o : top;
  }
  if constexpr (WAVES > 1) {
    if ((tid & 63) == 0) wtop[tid >> 6] = top;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < WAVES; ++w) top = wtop[w] > top ? wtop[w] : top;
  }
  const RowScale rs = row_scale_of(__builtin_bit_cast(uint32_t, Elem<DT>::to_float(top)));
  if (tid == 0) scales[m] = rs.s;
  auto store = [&](int u, const u32x4& v) {
    int q[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float f = Elem<DT>::to_float((v[i >> 1] >> (16 * (i & 1))) & 0xFFFFu);
      q[i] = rs.r == 0.0f ? 0 : quant1(f * rs.up, rs.r);
    }
    u32x2 o;
    o[0] = pack4(q[0], q[1], q[2], q[3]);
    o[1] = pack4(q[4], q[5], q[6], q[7]);
    *reinterpret_cast<u32x2*>(Q + m * kp + 8 * u) = o;
  };
  if constexpr (UNITS > 0) {
#pragma unroll
    for (int i = 0; i < UNITS; ++i) {
      const int u = tid + i * kThreads;
      if (u < units) store(u, held[i]);
    }
  } else {
    for (int u = tid; u < units; u += kThreads) store(u, load(u));
  }
}

// ---------------------------------------------------------------------------
// Epilogue: y = (acc * sw) * sx (+ bias) in fp32, one rounding.
// ---------------------------------------------------------------------------
// acc[i][j], lane (r, g): channels n + 16 i + 0..3 of token m + 16 j, with
// n already at the lane's channels and m at its token.  WHOLE: no edge, N % 4 == 0.
template <int DT, int TA, int TB, bool WHOLE>
__device__ __forceinline__ void store_tile(void* __restrict__ Y, const i32x4 (&acc)[TA][TB], const float* __restrict__ sx,
                                           const float* __restrict__ sw, const void* __restrict__ bias, int64_t m,
                                           int64_t n, int64_t M, int64_t N) {
  using T = typename Elem<DT>::T;
  typedef T T4 __attribute__((ext_vector_type(4)));
  const T* b = static_cast<const T*>(bias);
  float xs[TB];
#pragma unroll
  for (int j = 0; j < TB; ++j) xs[j] = sx[WHOLE || m + 16 * j < M ? m + 16 * j : M - 1];
#pragma unroll
  for (int i = 0; i < TA; ++i) {
    float ws[4], bs[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int64_t ni = n + 16 * i + e;
      ws[e] = sw[WHOLE || ni < N ? ni : N - 1];
      if (b) bs[e] = static_cast<float>(b[WHOLE || ni < N ? ni : N - 1]);
    }
#pragma unroll
    for (int j = 0; j < TB; ++j) {
      T4 o;
#pragma unroll
      for (int e = 0; e < 4; ++e) o[e] = static_cast<T>((static_cast<float>(acc[i][j][e]) * ws[e]) * xs[j] + bs[e]);
      T* y = static_cast<T*>(Y) + (m + 16 * j) * N + n + 16 * i;
      if constexpr (WHOLE) {
        *reinterpret_cast<T4*>(y) = o;
      } else if (m + 16 * j < M) {
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (n + 16 * i + e < N) y[e] = o[e];
      }
    }
  }
}

// ---------------------------------------------------------------------------
// Product.  A workgroup of WA x WB waves owns a tile of 16*WA*TA channels x
// 16*WB*TB tokens, a wave 16*TA x 16*TB of it; with WK > 1 (few tokens), WK
// waves own the whole tile, each with a ring of its own and a part of K, and
// add their exact sums through LDS.  K runs in
// steps of 128 bytes (a cache line of every row: with steps of 64, the first
// form, each line came twice from the L2) through a ring of D LDS stages filled
// by direct LDS loads.  A step is two halves of 64 bytes; the fragments of a
// half are read from LDS between the MFMAs of the half before it.  One barrier
// per step, before its second half: every wave waits there until its reads of the
// stage's last fragments are done, so step t+D may be requested into it, and
// until its loads of step t+1 have landed; a load has D-1 steps to arrive.  Each stage is its own LDS array
// and the barrier carries no fence, so that nothing waits for more loads than
// the next step needs.
//
// Unit c (16 bytes) of LDS row r lies at place c ^ (r % 8), so that the eight
// rows of a quarter wave's fragment read cover the eight places of a line.  The
// direct loads are linear on the LDS side, so the turn is made on the global
// side.  Kp need not be a multiple of 128: the last units of the ring are filled
// with zeros.  Rows behind the last repeat it and are not stored.
//
// Few tokens are bound by the weights' bytes: 16x28672x8192 41 us, 5.7 TB/s.
// From some hundred tokens on it is the way from the L2 to LDS that bounds, so
// the tile is as large as registers allow (256x256 over 8 waves):
// 4096x11008x4096 171 us, 2.16 POP/s (128x256 213 us, 128x128 222), 8192^3 421
// us, 2.61 POP/s (556 and 588).  In between the CUs are not full and a step is
// latency: 128x21504x7168 42 us, 168 tiles of 128x128, 3.7 TB/s (64x128 57 us).
// ---------------------------------------------------------------------------
__device__ __forceinline__ void barrier_no_fence() { asm volatile("s_barrier" ::: "memory"); }

// Until at most N of the wave's loads are in flight and its LDS reads are done.
template <int N>
__device__ __forceinline__ void wait_loads() {
  __builtin_amdgcn_s_waitcnt((N & 15) | ((N >> 4) << 14) | (7 << 4));
}

// Workgroup index -> tile, XCD-aware: workgroups go to the 8 XCDs in turn, and
// each XCD gets a contiguous range of the order below, in which kBand token
// tiles by all channel tiles follow one another (they share channels' bytes in
// the XCD's L2).
__device__ __forceinline__ void tile_of(uint32_t b, uint32_t mt, uint32_t nt, uint32_t& tm, uint32_t& tn) {
  constexpr uint32_t kXcds = 8, kBand = 8;
  const uint32_t G = mt * nt, x = b % kXcds, j = b / kXcds, q = G / kXcds, r = G % kXcds;
  const uint32_t l = x * q + (x < r ? x : r) + j;
  const uint32_t band = l / (kBand * nt), in = l - band * kBand * nt;
  const uint32_t rows = mt - band * kBand < kBand ? mt - band * kBand : kBand;
  tn = in / rows;
  tm = band * kBand + (in - tn * rows);
}

//
// The second launch bound keeps the accumulators of the 4-wave forms in vector
// registers; with more room the compiler moves them to and from the
// accumulation registers in every step.
template <int DT, int WA, int WB, int TA, int TB, int D, int WK, bool NT>
__global__ __launch_bounds__(64 * WA * WB * WK, 2) void i8_tiled(const int8_t* __restrict__ Xq, const float* __restrict__ sx,
                                                         const int8_t* __restrict__ Wq, const float* __restrict__ sw,
                                                         const void* __restrict__ bias, void* __restrict__ Y,
                                                         int64_t M, int64_t N, int64_t kp) {
  constexpr int kThreads = 64 * WA * WB, kRowsA = 16 * WA * TA, kRowsB = 16 * WB * TB;
  constexpr int kUnits = (kRowsA + kRowsB) * 8, kLoads = kUnits / kThreads;
  static_assert(kUnits % kThreads == 0 && kRowsA * 8 % kThreads == 0, "a load of the workgroup reads one operand");
  static_assert(D == 2 || D == 4, "ring depths");
  static_assert(WK == 1 || WA * WB == 1, "waves share a ring or split K, not both");
  constexpr bool kShared = WA * WB > 1;  // a ring of several waves: barriers
  __shared__ i32x4 st0[WK * kUnits], st1[WK * kUnits], st2[D > 2 ? WK * kUnits : 1], st3[D > 2 ? WK * kUnits : 1];
  const int wk = kShared ? 0 : __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  i32x4* const ring[4] = {st0 + wk * kUnits, st1 + wk * kUnits, st2 + (D > 2 ? wk * kUnits : 0),
                          st3 + (D > 2 ? wk * kUnits : 0)};
  const int tid = kShared ? threadIdx.x : threadIdx.x & 63, lane = tid & 63, wave = tid >> 6;
  const int r = lane & 15, g = lane >> 4;
  const int wa = wave / WB, wb = wave - wa * WB;
  uint32_t tm, tn;
  tile_of(blockIdx.x, static_cast<uint32_t>((M + kRowsB - 1) / kRowsB), static_cast<uint32_t>((N + kRowsA - 1) / kRowsA),
          tm, tn);
  const int64_t n0 = static_cast<int64_t>(tn) * kRowsA, m0 = static_cast<int64_t>(tm) * kRowsB;

  // The scales and biases of the tile, for the epilogue.
  __shared__ float s_sx[kRowsB], s_sw[kRowsA], s_bias[kRowsA];
  if constexpr (WK == 1) {
    for (int i = threadIdx.x; i < kRowsA; i += kThreads) {
      const int64_t n = n0 + i < N ? n0 + i : N - 1;
      s_sw[i] = sw[n];
      s_bias[i] = bias ? static_cast<float>(static_cast<const typename Elem<DT>::T*>(bias)[n]) : 0.0f;
    }
    for (int i = threadIdx.x; i < kRowsB; i += kThreads) s_sx[i] = sx[m0 + i < M ? m0 + i : M - 1];
  }

  // This thread's units of a stage: place p of LDS row `row` holds unit p ^ (row % 8).
  // Addresses are a wave-uniform base and a 32-bit offset inside the tile's
  // rows (at most 256 * 131056).
  const int8_t* base_a = Wq + n0 * kp;
  const int8_t* base_b = Xq + m0 * kp;
  uint32_t off[kLoads];
#pragma unroll
  for (int i = 0; i < kLoads; ++i) {
    const int p = i * kThreads + tid, row = p >> 3, unit = (p ^ row) & 7;
    const bool in_a = row < kRowsA;
    const int64_t left = in_a ? N - n0 : M - m0;  // rows of the tile that exist
    const int rr = in_a ? row : row - kRowsA;
    off[i] = static_cast<uint32_t>(rr < left ? rr : left - 1) * static_cast<uint32_t>(kp) + 16 * unit;
  }
  // Steps t0 .. t1-1 are this wave's (WK > 1: its part of K), those below
  // `full` are whole lines; behind t1 the ring is filled with zeros.
  const int total = static_cast<int>((kp + 127) >> 7);
  const int t0 = WK == 1 ? 0 : wk * total / WK, t1 = WK == 1 ? total : (wk + 1) * total / WK;
  const int full = t1 < static_cast<int>(kp >> 7) ? t1 : static_cast<int>(kp >> 7);
  const int t_end = t0 + (t1 - t0 + D - 1) / D * D;  // the last round's end
  const int uwave = __builtin_amdgcn_readfirstlane(wave);
  auto load_unit = [&](i32x4* stage, const int8_t* a, const int8_t* b, int i) {
    auto* dst = reinterpret_cast<__attribute__((address_space(3))) void*>(
        reinterpret_cast<uintptr_t>(stage + i * kThreads + uwave * 64));
    constexpr int kNonTemporal = 2;
    if (i * kThreads < kRowsA * 8)
      __builtin_amdgcn_global_load_lds(static_cast<const void*>(a + off[i]), dst, 16, 0, NT ? kNonTemporal : 0);
    else
      __builtin_amdgcn_global_load_lds(static_cast<const void*>(b + off[i]), dst, 16, 0, 0);
  };
  // The same for any step: the row's last, partial step and the zeros behind it
  // go through registers.  Nothing is in flight afterwards, so the next waits
  // find less than they allow for and nothing early.
  auto request_any = [&](i32x4* stage, int t) {
    const int64_t k = static_cast<int64_t>(t) * 128;
    if (t < full) {
#pragma unroll
      for (int i = 0; i < kLoads; ++i) load_unit(stage, base_a + k, base_b + k, i);
      return;
    }
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      const int p = i * kThreads + tid, unit = (p ^ (p >> 3)) & 7;
      i32x4 v = {0, 0, 0, 0};
      if (t < t1 && k + 16 * unit < kp)
        v = *reinterpret_cast<const i32x4*>((i * kThreads < kRowsA * 8 ? base_a : base_b) + k + off[i]);
      stage[p] = v;
      asm volatile("" ::: "memory");  // one at a time: these are few, and registers are short
    }
    __builtin_amdgcn_s_waitcnt(0);
  };
  const int row_a = (wa * TA * 16 + r) * 8, row_b = (kRowsA + wb * TB * 16 + r) * 8;  // rows 16 i + r: i * 128 units on
  const int place[2] = {g ^ (r & 7), (4 + g) ^ (r & 7)};
  i32x4 fa[TA], fb[2][TB], acc[TA][TB] = {};
  auto mul = [&](int i, const i32x4 (&b)[TB], int j) {
    acc[i][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(fa[i], b[j], acc[i][j], 0, 0, 0);
  };
  // The MFMAs of half H with the reads of the half that follows (half `to` of
  // `next`) and, with LOAD, the loads of a later step into `dst`, all spread
  // among them: a wave issues in order, and loads issued in one go would hold
  // its MFMAs back until the address unit has taken them (16 cycles each at
  // 64 bytes per cycle).  Channel fragment i is read as soon as this half is
  // done with it, into the same registers; the token fragments are
  // double-buffered.
  auto half = [&](auto H, const i32x4* next, auto LOAD, i32x4* dst, const int8_t* a, const int8_t* b) {
    constexpr int p = decltype(H)::value, to = 1 - p;
    constexpr int kLd = decltype(LOAD)::value ? (kLoads + TA - 1) / TA : 0;  // loads per channel block
#pragma unroll
    for (int i = 0; i < TA; ++i) {
#pragma unroll
      for (int j = 0; j < TB / 2; ++j) mul(i, fb[p], j);
#pragma unroll
      for (int l = i * kLd; l < (i + 1) * kLd; ++l)
        if (l < kLoads) load_unit(dst, a, b, l);
#pragma unroll
      for (int j = i; j < TB; j += TA) fb[to][j] = next[row_b + 128 * j + place[to]];
#pragma unroll
      for (int j = TB / 2; j < TB; ++j) mul(i, fb[p], j);
      fa[i] = next[row_a + 128 * i + place[to]];
    }
#pragma unroll
    for (int i = 0; i < TA; ++i) {
      if (TB > 1) __builtin_amdgcn_sched_group_barrier(0x008, TB / 2, 0);
      if (kLd > 0 && i * kLd < kLoads) __builtin_amdgcn_sched_group_barrier(0x010, kLd, 0);
      if (i < TB) __builtin_amdgcn_sched_group_barrier(0x100, (TB + TA - 1) / TA, 0);
      __builtin_amdgcn_sched_group_barrier(0x008, TB - TB / 2, 0);
      __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
    }
    __builtin_amdgcn_sched_barrier(0);
  };
  constexpr std::integral_constant<int, 0> first{};
  constexpr std::integral_constant<int, 1> second{};
  auto step = [&](int t, auto S, auto ANY) {  // step t, (t - t0) % D == S
    constexpr int st = decltype(S)::value;
    half(first, ring[st], std::false_type{}, nullptr, nullptr, nullptr);
    // Behind the last whole line fewer loads are in flight than the count allows for.
    if (decltype(ANY)::value && t + D - 1 >= full) wait_loads<0>();
    else wait_loads<(D - 2) * kLoads>();
    if constexpr (kShared) barrier_no_fence();
    if constexpr (decltype(ANY)::value) {
      if (t + D < t_end) request_any(ring[st], t + D);
      half(second, ring[(st + 1) % D], std::false_type{}, nullptr, nullptr, nullptr);
    } else {
      // Opaque scalar bases: added to the offsets by the load itself.  Left to
      // itself the compiler keeps base + offset of every load in registers and
      // adds k to each.
      const int8_t* a = base_a + static_cast<int64_t>(t + D) * 128;
      const int8_t* b = base_b + static_cast<int64_t>(t + D) * 128;
      asm("" : "+s"(a), "+s"(b));
      half(second, ring[(st + 1) % D], std::true_type{}, ring[st], a, b);
    }
  };
#pragma unroll
  for (int i = 0; i < D; ++i) request_any(ring[i], t0 + i);
  wait_loads<(D - 1) * kLoads>();
  if constexpr (kShared) barrier_no_fence();
#pragma unroll
  for (int j = 0; j < TB; ++j) fb[0][j] = ring[0][row_b + 128 * j + place[0]];
#pragma unroll
  for (int i = 0; i < TA; ++i) fa[i] = ring[0][row_a + 128 * i + place[0]];
  auto round = [&](int t, auto ANY) {
    step(t, std::integral_constant<int, 0>{}, ANY);
    step(t + 1, std::integral_constant<int, 1>{}, ANY);
    if constexpr (D > 2) {
      step(t + 2, std::integral_constant<int, 2>{}, ANY);
      step(t + 3, std::integral_constant<int, 3>{}, ANY);
    }
  };
  int t = t0;
  for (; t + 2 * D - 1 < full; t += D) round(t, std::false_type{});
  for (; t < t1; t += D) round(t, std::true_type{});
  __builtin_amdgcn_s_waitcnt(0);  // no load may land after the workgroup has left

  if constexpr (WK > 1) {
    // The waves' sums meet in LDS (exact, so in any order); wave i takes block i, i + WK, ...
    __shared__ i32x4 red[WK][TA * TB][64];
#pragma unroll
    for (int i = 0; i < TA * TB; ++i) red[wk][i][lane] = acc[i / TB][i % TB];
    __syncthreads();
    for (int i = wk; i < TA * TB; i += WK) {
      i32x4 sum[1][1] = {{red[0][i][lane]}};
#pragma unroll
      for (int w = 1; w < WK; ++w) sum[0][0] += red[w][i][lane];
      const int64_t n = n0 + 16 * (i / TB) + 4 * g, m = m0 + 16 * (i % TB) + r;
      if ((N & 3) == 0 && m < M && n < N) store_tile<DT, 1, 1, true>(Y, sum, sx, sw, bias, m, n, M, N);
      else store_tile<DT, 1, 1, false>(Y, sum, sx, sw, bias, m, n, M, N);
    }
    return;
  }
  // Epilogue.  A wave scales its block into its own part of the ring (free
  // after the barrier), a token's channels side by side, and stores whole rows
  // of it, 16 bytes per lane: stored straight from the accumulators, a
  // request would touch 16 rows with 32 bytes each.
  using T = typename Elem<DT>::T;
  typedef T T4 __attribute__((ext_vector_type(4)));
  constexpr int kCols = 16 * TA, kPitch = kCols + 8;  // 16 bytes more: rows start at different banks
  constexpr int kRowsOut = 16 * TB;
  static_assert(kPitch * 2 * 16 <= kUnits * 16 / (WA * WB), "16 tokens of every wave fit one stage");
  const int64_t nw = n0 + wa * kCols, mw = m0 + wb * kRowsOut;
  if constexpr (kShared) __syncthreads();
  T* buf = reinterpret_cast<T*>(st0 + wave * (kUnits / (WA * WB)));
  const T* bv = static_cast<const T*>(bias);
  const bool vec = (N & 7) == 0;
#pragma unroll
  for (int j = 0; j < TB; ++j) {
    const float xs = s_sx[wb * kRowsOut + 16 * j + r];
#pragma unroll
    for (int i = 0; i < TA; ++i) {
      const float4v ws = *reinterpret_cast<const float4v*>(&s_sw[wa * kCols + 16 * i + 4 * g]);
      const float4v bs = *reinterpret_cast<const float4v*>(&s_bias[wa * kCols + 16 * i + 4 * g]);
      T4 o;
#pragma unroll
      for (int e = 0; e < 4; ++e) o[e] = static_cast<T>((static_cast<float>(acc[i][j][e]) * ws[e]) * xs + bs[e]);
      *reinterpret_cast<T4*>(&buf[r * kPitch + 16 * i + 4 * g]) = o;
    }
    __builtin_amdgcn_wave_barrier();
    constexpr int kUnitsRow = kCols / 8;
#pragma unroll
    for (int u0 = 0; u0 < 16 * kUnitsRow; u0 += 64) {
      const int u = u0 + lane, row = u / kUnitsRow, col = (u % kUnitsRow) * 8;
      const int64_t m = mw + 16 * j + row, n = nw + col;
      if (u < 16 * kUnitsRow && m < M && n < N) {
        T* y = static_cast<T*>(Y) + m * N + n;
        const u32x4 v = *reinterpret_cast<const u32x4*>(&buf[row * kPitch + col]);
        if (vec && n + 8 <= N) {
          *reinterpret_cast<u32x4*>(y) = v;
        } else {
#pragma unroll
          for (int e = 0; e < 8; ++e)
            if (n + e < N) y[e] = buf[row * kPitch + col + e];
        }
      }
    }
    __builtin_amdgcn_wave_barrier();
  }
}

// ---------------------------------------------------------------------------
// Quantiser and product in one kernel, for one token: a workgroup of 4 waves
// owns 16 channels and makes the token's codes for itself, in LDS, while its
// first weights are on their way; then the waves split K in contiguous parts
// (weights straight into fragments; every MFMA column repeats the token) and
// add their exact sums.  It saves the quantiser's launch and the codes' way
// through memory: 1x4096x4096 7.6 us against 8.5 (in a graph; a launch less from
// the host, too), 1x8192x8192 17.9 against 18.4.  With more tokens every
// workgroup's own quantising costs more than it saves: 2x8192x2048 9.6 against
// 9.0, 4x4096x4096 13.2 against 8.7.
// ---------------------------------------------------------------------------
constexpr int kOneTokenK = 8192;

template <int DX, int DT>
__global__ __launch_bounds__(256, 2) void i8_one_token(const uint16_t* __restrict__ x, int K,
                                                       const int8_t* __restrict__ Wq, const float* __restrict__ sw,
                                                       const void* __restrict__ bias, void* __restrict__ Y, int64_t N,
                                                       int kp) {
  constexpr int kWaves = 4, kBatch = 8;  // steps of 128 bytes in flight per wave
  __shared__ i32x4 codes[kOneTokenK / 16];
  __shared__ uint32_t wtop[kWaves];
  __shared__ i32x4 red[kWaves][64];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int r = lane & 15, g = lane >> 4;
  const int64_t n0 = static_cast<int64_t>(blockIdx.x) * 16;
  const int total = (kp + 127) >> 7;
  const int t0 = wave * total / kWaves, t1 = (wave + 1) * total / kWaves;
  const int8_t* w = Wq + (n0 + r < N ? n0 + r : N - 1) * kp;
  i32x4 wf[2 * kBatch];
  auto load_w = [&](int t) {  // half h of step t: bytes 128 t + 64 h + 16 g
#pragma unroll
    for (int i = 0; i < 2 * kBatch; ++i) {
      const int k = (t + (i >> 1)) * 128 + (i & 1) * 64 + 16 * g;
      wf[i] = *reinterpret_cast<const i32x4*>(w + (k < kp ? k : 0));  // behind the row: a stand-in, times zero
    }
  };
  load_w(t0);

  const int units = kp >> 3;  // of 8 elements
  auto load_x = [&](int u) -> u32x4 {
    u32x4 v = {0, 0, 0, 0};
    if (8 * u + 8 <= K) {
      v = *reinterpret_cast<const u32x4_any*>(x + 8 * u);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int k = 8 * u + 2 * i;
        v[i] = (k < K ? x[k] : 0u) | (k + 1 < K ? static_cast<uint32_t>(x[k + 1]) << 16 : 0u);
      }
    }
    return v;
  };
  uint32_t top = 0;
  for (int u = tid; u < units; u += 256) {
    const u32x4 v = load_x(u);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t lo = v[i] & 0x7FFFu, hi = (v[i] >> 16) & 0x7FFFu;
      top = lo > top ? lo : top;
      top = hi > top ? hi : top;
    }
  }
#pragma unroll
  for (int d = 32; d > 0; d >>= 1) {
    const uint32_t o = __shfl_xor(top, d);
    top = o > top ? o : top;
  }
  if (lane == 0) wtop[wave] = top;
  __syncthreads();
#pragma unroll
  for (int v = 0; v < kWaves; ++v) top = wtop[v] > top ? wtop[v] : top;
  const RowScale rs = row_scale_of(__builtin_bit_cast(uint32_t, Elem<DX>::to_float(top)));
  // The codes, with zeros up to whole steps.
  for (int u = tid; u < 16 * total; u += 256) {
    u32x2 o = {0, 0};
    if (u < units) {
      const u32x4 v = load_x(u);
      int q[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float f = Elem<DX>::to_float((v[i >> 1] >> (16 * (i & 1))) & 0xFFFFu);
        q[i] = rs.r == 0.0f ? 0 : quant1(f * rs.up, rs.r);
      }
      o[0] = pack4(q[0], q[1], q[2], q[3]);
      o[1] = pack4(q[4], q[5], q[6], q[7]);
    }
    reinterpret_cast<u32x2*>(codes)[u] = o;
  }
  __syncthreads();

  i32x4 acc = {0, 0, 0, 0};
  for (int t = t0; t < t1; t += kBatch) {
#pragma unroll
    for (int i = 0; i < 2 * kBatch; ++i) {
      if (t + (i >> 1) < t1)
        acc = __builtin_amdgcn_mfma_i32_16x16x64_i8(wf[i], codes[(t + (i >> 1)) * 8 + (i & 1) * 4 + g], acc, 0, 0, 0);
    }
    if (t + kBatch < t1) load_w(t + kBatch);
  }
  red[wave][lane] = acc;
  __syncthreads();
  if (wave == 0) {
    i32x4 sum[1][1] = {{red[0][lane]}};
#pragma unroll
    for (int v = 1; v < kWaves; ++v) sum[0][0] += red[v][lane];
    const int64_t n = n0 + 4 * g;
    if (r == 0 && (N & 3) == 0 && n < N) store_tile<DT, 1, 1, true>(Y, sum, &rs.s, sw, bias, 0, n, 1, N);
    else if (r == 0) store_tile<DT, 1, 1, false>(Y, sum, &rs.s, sw, bias, 0, n, 1, N);
  }
}

// ---------------------------------------------------------------------------
// Host side.
// ---------------------------------------------------------------------------
bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }
bool dtype_ok(int d) { return d == FP6_FP16 || d == FP6_BF16; }

template <int DT>
int launch_quantize_t(const void* X, int64_t ldx, int64_t M, int64_t K, void* Xq, void* scales, hipStream_t s) {
  int k = static_cast<int>(K), kp = static_cast<int>(fp6_int8_padded_k(K));
  const void* kern;
  int rows = 1;  // per workgroup
  if (kp <= 2048) {
    rows = 4;
    kern = kp <= 512    ? reinterpret_cast<const void*>(&i8_quantize<DT, 1, 1>)
           : kp <= 1024 ? reinterpret_cast<const void*>(&i8_quantize<DT, 2, 1>)
                        : reinterpret_cast<const void*>(&i8_quantize<DT, 4, 1>);
  } else {
    kern = kp <= 4096    ? reinterpret_cast<const void*>(&i8_quantize<DT, 2, 4>)
           : kp <= 8192  ? reinterpret_cast<const void*>(&i8_quantize<DT, 4, 4>)
           : kp <= 16384 ? reinterpret_cast<const void*>(&i8_quantize<DT, 8, 4>)
                         : reinterpret_cast<const void*>(&i8_quantize<DT, 0, 4>);
  }
  // A grid holds fewer than 2^32 threads: at most 2^22 rows per launch.
  constexpr int64_t kRows = int64_t(1) << 22;
  for (int64_t m0 = 0; m0 < M; m0 += kRows) {
    const uint16_t* x = static_cast<const uint16_t*>(X) + m0 * ldx;
    int8_t* q = static_cast<int8_t*>(Xq) + m0 * kp;
    float* sc = static_cast<float*>(scales) + m0;
    int64_t n = M - m0 < kRows ? M - m0 : kRows;
    void* args[] = {&x, &ldx, &n, &k, &kp, &q, &sc};
    const int st = launch(kern, dim3(static_cast<unsigned>(ceil_div(n, rows))), dim3(256), args, s);
    if (st != FP6_OK) return st;
  }
  return FP6_OK;
}

int launch_quantize(int dtype, const void* X, int64_t ldx, int64_t M, int64_t K, void* Xq, void* scales,
                    hipStream_t s) {
  return dtype == FP6_FP16 ? launch_quantize_t<FP6_FP16>(X, ldx, M, K, Xq, scales, s)
                           : launch_quantize_t<FP6_BF16>(X, ldx, M, K, Xq, scales, s);
}

struct Product {
  const void *xq, *sx, *wq, *sw, *bias;
  void* y;
  int64_t M, N, kp;
};

// Weights of at least this size, read once per call, are loaded with the
// non-temporal hint: 16x28672x8192 46 -> 42 us, 1x28672x8192 42 -> 37 us.
// Smaller ones may still be in the 256 MB cache from the call before
// (16x4096x4096 7.3 us from there, 9.7 us with the hint).
constexpr int64_t kStreamBytes = int64_t(64) << 20;

template <int DT, int WA, int WB, int TA, int TB, int D, int WK = 1>
int launch_tiled(const Product& p, hipStream_t s) {
  const int8_t *x = static_cast<const int8_t*>(p.xq), *w = static_cast<const int8_t*>(p.wq);
  const float *sx = static_cast<const float*>(p.sx), *sw = static_cast<const float*>(p.sw);
  const void* bias = p.bias;
  // The grid (tiles times threads below 2^32) takes this many token tiles at once.
  constexpr int64_t kTileM = 16 * WB * TB, kTileN = 16 * WA * TA, kThreads = 64 * WA * WB * WK;
  const int64_t per = ((int64_t(1) << 31) / kThreads) / ceil_div(p.N, kTileN) * kTileM;
  for (int64_t m0 = 0; m0 < p.M; m0 += per) {
    int64_t M = p.M - m0 < per ? p.M - m0 : per, N = p.N, kp = p.kp;
    const int8_t* xm = x + m0 * kp;
    const float* sxm = sx + m0;
    void* y = static_cast<uint16_t*>(p.y) + m0 * N;
    void* args[] = {&xm, &sxm, &w, &sw, &bias, &y, &M, &N, &kp};
    const dim3 grid(static_cast<unsigned>(ceil_div(M, kTileM) * ceil_div(N, kTileN)));
    const bool nt = M <= kTileM && N * kp >= kStreamBytes;
    const void* kern = nt ? reinterpret_cast<const void*>(&i8_tiled<DT, WA, WB, TA, TB, D, WK, true>)
                          : reinterpret_cast<const void*>(&i8_tiled<DT, WA, WB, TA, TB, D, WK, false>);
    const int st = launch(kern, grid, dim3(kThreads), args, s);
    if (st != FP6_OK) return st;
  }
  return FP6_OK;
}

// Kernel configurations of fp6_int8_linear_plan: channels x tokens per workgroup.
enum Variant : int {
  kAuto, kSplit16x16, kOne16x16, kSplit16x32, kSplit32x32, kSplit32x64,
  kTile64x64, kTile64x128, kTile128x128, kTile128x256, kTile256x256, kNumVariants
};

// The tiled forms' cost on a shape: rounds of workgroups over the CUs, each
// round as long as a full one was measured, the last, partial one between a
// nearly empty and a full one by its fill (us at K = 4096; the form's tile,
// workgroups per CU).  Every cost grows with K alike.
struct TileCost {
  int variant, n, m, per_cu;
  float empty, full;
};
constexpr TileCost kTiles[] = {
    {kTile64x64, 64, 64, 2, 8.9f, 14.5f},     {kTile64x128, 64, 128, 1, 11.1f, 13.4f},
    {kTile128x128, 128, 128, 1, 15.3f, 20.3f}, {kTile128x256, 128, 256, 1, 26.5f, 35.7f},
    {kTile256x256, 256, 256, 1, 41.0f, 60.0f},
};

int choose_variant(const Product& p, int cus) {
  const int64_t nb = ceil_div(p.N, 16);
  // Up to 16 tokens: four waves that split K while that is at most two
  // workgroups per CU (16x4096x4096 6.0 us against 7.2 with one wave,
  // 16x4096x11008 13.0 against 20.8), else one wave per workgroup
  // (16x11008x4096 13.1 against 14.3).
  if (p.M <= 16) return nb <= 2 * cus ? kSplit16x16 : kOne16x16;
  // The forms whose waves split K run one workgroup per CU; the smallest one
  // that needs no second round (32x4096x4096 5.8 us against 8.8 with 64x64
  // tiles, 64x8192x8192 17.0 against 24.3, 128x4096x11008 23.4 against 30.1;
  // where it needs one: 64x11008x4096 20.9 against 15.2).
  if (ceil_div(p.M, 32) * nb <= cus) return kSplit16x32;
  if (ceil_div(p.M, 32) * ceil_div(nb, 2) <= cus) return kSplit32x32;
  if (ceil_div(p.M, 64) * ceil_div(nb, 2) <= cus) return kSplit32x64;
  int best = kTile64x64;
  float best_cost = 0.0f;
  for (const TileCost& t : kTiles) {
    const float rounds = static_cast<float>(ceil_div(p.M, t.m) * ceil_div(p.N, t.n)) / static_cast<float>(cus * t.per_cu);
    const float whole = static_cast<float>(static_cast<int64_t>(rounds)), part = rounds - whole;
    const float cost = whole * t.full + (part > 0.0f ? t.empty + (t.full - t.empty) * part : 0.0f);
    if (best_cost == 0.0f || cost < best_cost) {
      best = t.variant;
      best_cost = cost;
    }
  }
  return best;
}

template <int DT>
int launch_product_t(const Product& p, int variant, hipStream_t s) {
  switch (variant) {  // WA, WB, TA, TB, D, WK
    case kSplit16x16: return launch_tiled<DT, 1, 1, 1, 1, 4, 4>(p, s);
    case kOne16x16: return launch_tiled<DT, 1, 1, 1, 1, 4>(p, s);
    case kSplit16x32: return launch_tiled<DT, 1, 1, 1, 2, 4, 4>(p, s);
    case kSplit32x32: return launch_tiled<DT, 1, 1, 2, 2, 4, 4>(p, s);
    case kSplit32x64: return launch_tiled<DT, 1, 1, 2, 4, 2, 4>(p, s);
    case kTile64x64: return launch_tiled<DT, 2, 2, 2, 2, 4>(p, s);
    case kTile64x128: return launch_tiled<DT, 2, 4, 2, 2, 4>(p, s);
    case kTile128x128: return launch_tiled<DT, 2, 4, 4, 2, 4>(p, s);
    case kTile128x256: return launch_tiled<DT, 2, 4, 4, 4, 2>(p, s);
    case kTile256x256: return launch_tiled<DT, 2, 4, 8, 4, 2>(p, s);
    default: return FP6_E_VALUE;
  }
}

int launch_product(int dtype, const Product& p, int variant, hipStream_t s) {
  if (variant == kAuto) variant = choose_variant(p, fpx::current_cus());
  return dtype == FP6_FP16 ? launch_product_t<FP6_FP16>(p, variant, s) : launch_product_t<FP6_BF16>(p, variant, s);
}

template <int DX>
int launch_one_token(const void* X, int64_t K, const Product& p, int dtype, hipStream_t s) {
  const uint16_t* x = static_cast<const uint16_t*>(X);
  const int8_t* w = static_cast<const int8_t*>(p.wq);
  const float* sw = static_cast<const float*>(p.sw);
  const void* bias = p.bias;
  void* y = p.y;
  int k = static_cast<int>(K), kp = static_cast<int>(p.kp);
  int64_t N = p.N;
  void* args[] = {&x, &k, &w, &sw, &bias, &y, &N, &kp};
  const void* kern = dtype == FP6_FP16 ? reinterpret_cast<const void*>(&i8_one_token<DX, FP6_FP16>)
                                       : reinterpret_cast<const void*>(&i8_one_token<DX, FP6_BF16>);
  return launch(kern, dim3(static_cast<unsigned>(ceil_div(N, 16))), dim3(256), args, s);
}

bool sizes_ok(int64_t M, int64_t N, int64_t kp) {
  return M >= 0 && M <= fp6::kMaxDim && N >= 1 && N <= fp6::kMaxDim && N * kp <= fp6::kMaxNK &&
         M * kp <= fp6::kMaxNK && M * N <= fp6::kMaxNK;
}

}  // namespace

extern "C" {

int fp6_int8_quantize_tokens(int dtype, const void* X, int64_t ldx, int64_t M, int64_t K, void* Xq,
                             void* scales, void* stream) {
  if (!dtype_ok(dtype)) return FP6_E_VALUE;
  const int64_t kp = fp6_int8_padded_k(K);
  if (!kp || M < 0 || M > fp6::kMaxDim || M * kp > fp6::kMaxNK || ldx < K || ldx > fp6::kMaxNK) return FP6_E_SHAPE;
  if (M == 0) return FP6_OK;
  if (!X || !Xq || !scales) return FP6_E_NULL;
  if (!aligned(X, 2) || !aligned(Xq, 16) || !aligned(scales, 4)) return FP6_E_ALIGN;
  return launch_quantize(dtype, X, ldx, M, K, Xq, scales, static_cast<hipStream_t>(stream));
}

int fp6_int8_linear_plan(const void* Xq, const void* sx, const void* Wq, const void* sw, const void* bias, int dtype,
                         void* Y, int64_t M, int64_t N, int64_t Kp, int variant, void* stream) {
  if (!dtype_ok(dtype) || variant < 0 || variant >= kNumVariants) return FP6_E_VALUE;
  if (Kp < 1 || Kp % 16 || Kp > fp6::kInt8MaxK || !sizes_ok(M, N, Kp)) return FP6_E_SHAPE;
  if (M == 0) return FP6_OK;
  if (!Xq || !sx || !Wq || !sw || !Y) return FP6_E_NULL;
  if (!aligned(Xq, 16) || !aligned(Wq, 16) || !aligned(Y, 16) || !aligned(sx, 4) || !aligned(sw, 4) ||
      !aligned(bias, 2))
    return FP6_E_ALIGN;
  return launch_product(dtype, Product{Xq, sx, Wq, sw, bias, Y, M, N, Kp}, variant, static_cast<hipStream_t>(stream));
}

int fp6_int8_linear(const void* Xq, const void* sx, const void* Wq, const void* sw, const void* bias, int dtype,
                    void* Y, int64_t M, int64_t N, int64_t Kp, void* stream) {
  return fp6_int8_linear_plan(Xq, sx, Wq, sw, bias, dtype, Y, M, N, Kp, kAuto, stream);
}

int fp6_int8_linear_tokens(int x_dtype, const void* X, int64_t ldx, const void* Wq, const void* sw,
                           const void* bias, int dtype, void* Y, int64_t M, int64_t N, int64_t K,
                           void* workspace, size_t workspace_bytes, void* stream) {
  if (!dtype_ok(x_dtype) || !dtype_ok(dtype)) return FP6_E_VALUE;
  const int64_t kp = fp6_int8_padded_k(K);
  if (!kp || !sizes_ok(M, N, kp) || ldx < K || ldx > fp6::kMaxNK) return FP6_E_SHAPE;
  if (M == 0) return FP6_OK;
  if (!X || !Wq || !sw || !Y || !workspace) return FP6_E_NULL;
  if (!aligned(X, 2) || !aligned(Wq, 16) || !aligned(Y, 16) || !aligned(workspace, 16) || !aligned(sw, 4) ||
      !aligned(bias, 2))
    return FP6_E_ALIGN;
  if (workspace_bytes < fp6_int8_workspace_bytes(M, K)) return FP6_E_SIZE;
  int8_t* xq = static_cast<int8_t*>(workspace);
  float* sx = reinterpret_cast<float*>(xq + M * kp);  // M*kp is a multiple of 16
  const hipStream_t s = static_cast<hipStream_t>(stream);
  // Every workgroup reads X: for up to two of them per CU.
  if (M == 1 && kp <= kOneTokenK && ceil_div(N, 16) <= 2 * fpx::current_cus()) {
    const Product p{nullptr, nullptr, Wq, sw, bias, Y, M, N, kp};
    return x_dtype == FP6_FP16 ? launch_one_token<FP6_FP16>(X, K, p, dtype, s)
                               : launch_one_token<FP6_BF16>(X, K, p, dtype, s);
  }
  const int st = launch_quantize(x_dtype, X, ldx, M, K, xq, sx, s);
  if (st != FP6_OK) return st;
  return launch_product(dtype, Product{xq, sx, Wq, sw, bias, Y, M, N, kp}, kAuto, s);
}

}  // extern "C"
