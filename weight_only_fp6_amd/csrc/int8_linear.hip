// 8-bit integer linear layer for gfx950: the token quantiser, the int8 MFMA
// product with a scale for each token and channel, and their entry points
// (fp6_int8.h).

#include <hip/hip_runtime.h>

#include <cstdint>
#include <type_traits>

#include "fp6_int8.h"
#include "fp6_limits.h"

namespace {

typedef int i32x4 __attribute__((ext_vector_type(4)));
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

// One row per workgroup.  VEC: rows start at multiples of 16 bytes, 8 elements
// per load; the last, partial unit of a row is read element by element.
template <int DT, bool VEC>
__global__ __launch_bounds__(256) void i8_quantize(const uint16_t* __restrict__ X, int64_t ldx, int K,
                                                   int kp, int8_t* __restrict__ Q,
                                                   float* __restrict__ scales) {
  __shared__ uint32_t wtop[4];
  const int tid = threadIdx.x, nthr = blockDim.x;
  const int64_t m = blockIdx.x;
  const uint16_t* x = X + m * ldx;
  const int units = kp >> 3;  // of 8 elements
  auto load = [&](int u) -> u32x4 {
    u32x4 v;
    if (VEC && 8 * u + 8 <= K) {
      v = *reinterpret_cast<const u32x4*>(x + 8 * u);
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
  for (int u = tid; u < units; u += nthr) {
    const u32x4 v = load(u);
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
  if ((tid & 63) == 0) wtop[tid >> 6] = top;
  __syncthreads();
  for (int w = 0; w < (nthr >> 6); ++w) top = wtop[w] > top ? wtop[w] : top;
  const RowScale rs = row_scale_of(__builtin_bit_cast(uint32_t, Elem<DT>::to_float(top)));
  if (tid == 0) scales[m] = rs.s;
  for (int u = tid; u < units; u += nthr) {
    const u32x4 v = load(u);
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
// Skinny product (few tokens): a workgroup of 8 waves owns 16*RB channels and
// 16*MB tokens; its waves split K in interleaved chunks of 64*S bytes, read
// both operands straight into MFMA fragments (lane (r, g): 16*S contiguous
// bytes of row r at offset 16*S*g of the chunk; both operands take k in the
// same order, so any order is right) and add their exact integer partial sums
// through LDS.
// ---------------------------------------------------------------------------
template <int DT, int RB, int MB, int S>
__global__ __launch_bounds__(512) void i8_skinny(const int8_t* __restrict__ Xq, const float* __restrict__ sx,
                                                 const int8_t* __restrict__ Wq, const float* __restrict__ sw,
                                                 const void* __restrict__ bias, void* __restrict__ Y,
                                                 int64_t M, int64_t N, int64_t kp) {
  constexpr int kWaves = 8, kAcc = RB * MB;
  __shared__ i32x4 red[kWaves][kAcc][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int r = lane & 15, g = lane >> 4;
  const int64_t n0 = static_cast<int64_t>(blockIdx.x) * 16 * RB;
  const int64_t m0 = static_cast<int64_t>(blockIdx.y) * 16 * MB;
  const int chunks = static_cast<int>((kp + 64 * S - 1) / (64 * S));
  const int8_t* w[RB];
  const int8_t* x[MB];
#pragma unroll
  for (int a = 0; a < RB; ++a) {
    const int64_t n = n0 + 16 * a + r;
    w[a] = Wq + (n < N ? n : N - 1) * kp;
  }
#pragma unroll
  for (int b = 0; b < MB; ++b) {
    const int64_t m = m0 + 16 * b + r;
    x[b] = Xq + (m < M ? m : M - 1) * kp;
  }
  i32x4 acc[RB][MB] = {};
  i32x4 wf[2][RB][S], xf[2][MB][S];
  auto load = [&](int slot, int c) {
    const int64_t k0 = static_cast<int64_t>(c) * 64 * S + 16 * S * g;
#pragma unroll
    for (int s = 0; s < S; ++s) {
      const int64_t k = k0 + 16 * s;
      const bool in = k < kp;
      const int64_t kk = in ? k : 0;  // a unit behind the row: a stand-in, times zero
#pragma unroll
      for (int a = 0; a < RB; ++a) wf[slot][a][s] = *reinterpret_cast<const i32x4*>(w[a] + kk);
#pragma unroll
      for (int b = 0; b < MB; ++b) {
        const i32x4 v = *reinterpret_cast<const i32x4*>(x[b] + kk);
        xf[slot][b][s] = in ? v : i32x4{0, 0, 0, 0};
      }
    }
  };
  auto mul = [&](int slot) {
#pragma unroll
    for (int s = 0; s < S; ++s)
#pragma unroll
      for (int a = 0; a < RB; ++a)
#pragma unroll
        for (int b = 0; b < MB; ++b)
          acc[a][b] = __builtin_amdgcn_mfma_i32_16x16x64_i8(wf[slot][a][s], xf[slot][b][s], acc[a][b], 0, 0, 0);
  };
  int c = wave;
  if (c < chunks) {
    load(0, c);
    for (;;) {
      const int c1 = c + kWaves;
      if (c1 >= chunks) {
        mul(0);
        break;
      }
      load(1, c1);
      mul(0);
      const int c2 = c1 + kWaves;
      if (c2 >= chunks) {
        mul(1);
        break;
      }
      load(0, c2);
      mul(1);
      c = c2;
    }
  }
#pragma unroll
  for (int a = 0; a < RB; ++a)
#pragma unroll
    for (int b = 0; b < MB; ++b) red[wave][a * MB + b][lane] = acc[a][b];
  __syncthreads();
  for (int i = wave; i < kAcc; i += kWaves) {
    i32x4 sum = red[0][i][lane];
#pragma unroll
    for (int v = 1; v < kWaves; ++v) sum += red[v][i][lane];
    const int a = i / MB, b = i % MB;
    const int64_t m = m0 + 16 * b + r, n = n0 + 16 * a + 4 * g;
    const i32x4 one[1][1] = {{sum}};
    if ((N & 3) == 0 && m < M && n < N) {
      store_tile<DT, 1, 1, true>(Y, one, sx, sw, bias, m, n, M, N);
    } else {
      store_tile<DT, 1, 1, false>(Y, one, sx, sw, bias, m, n, M, N);
    }
  }
}

// ---------------------------------------------------------------------------
// Tiled product (many tokens).  A workgroup of WA x WB waves owns a tile of
// 16*WA*TA channels x 16*WB*TB tokens, a wave 16*TA x 16*TB of it.  K runs in
// steps of 64 bytes through a ring of four LDS stages, filled by direct LDS
// loads.  Step t multiplies fragments that are in registers, reads those of
// step t+1 from LDS between the MFMAs, and requests step t+3 into the stage
// that step t-1 left; one barrier per step, and a load has two steps to arrive.
// Each stage is its own LDS array and the barrier carries no fence, so that
// nothing waits for more loads than the next step needs.
//
// An LDS row is 64 bytes in four 16-byte units; unit c of row r lies at place
// (c + r/2) % 4, so that 8 rows' fragment reads of one c cover 8 different
// places of a 128-byte line.  The direct loads are linear on the LDS side, so
// the turn is made on the global side.  Units behind a row's end (Kp need not
// be a multiple of 64) are loaded from 16 bytes of zeros; rows behind the last
// repeat it and are not stored.
// ---------------------------------------------------------------------------
__device__ const u32x4 kZeroUnit[1] = {};

__device__ __forceinline__ void barrier_no_fence() { asm volatile("s_barrier" ::: "memory"); }

template <int N>
__device__ __forceinline__ void wait_loads() {  // until at most N of the wave's loads are in flight
  __builtin_amdgcn_s_waitcnt((N & 15) | ((N >> 4) << 14) | (7 << 4) | (15 << 8));
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

template <int DT, int WA, int WB, int TA, int TB>
__global__ __launch_bounds__(64 * WA * WB) void i8_tiled(const int8_t* __restrict__ Xq, const float* __restrict__ sx,
                                                         const int8_t* __restrict__ Wq, const float* __restrict__ sw,
                                                         const void* __restrict__ bias, void* __restrict__ Y,
                                                         int64_t M, int64_t N, int64_t kp) {
  constexpr int kThreads = 64 * WA * WB, kRowsA = 16 * WA * TA, kRowsB = 16 * WB * TB;
  constexpr int kUnits = (kRowsA + kRowsB) * 4, kLoads = kUnits / kThreads;
  static_assert(kUnits % kThreads == 0, "every thread makes the same number of loads");
  __shared__ i32x4 st0[kUnits], st1[kUnits], st2[kUnits], st3[kUnits];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int r = lane & 15, g = lane >> 4;
  const int wa = wave / WB, wb = wave - wa * WB;
  uint32_t tm, tn;
  tile_of(blockIdx.x, static_cast<uint32_t>((M + kRowsB - 1) / kRowsB), static_cast<uint32_t>((N + kRowsA - 1) / kRowsA),
          tm, tn);
  const int64_t n0 = static_cast<int64_t>(tn) * kRowsA, m0 = static_cast<int64_t>(tm) * kRowsB;

  // This thread's units of a stage: place p of row p/4 holds unit (p - row/2) % 4.
  const int8_t* src[kLoads];
  int unit[kLoads];
#pragma unroll
  for (int i = 0; i < kLoads; ++i) {
    const int p = i * kThreads + tid, row = p >> 2;
    unit[i] = ((p & 3) - (row >> 1)) & 3;
    if (row < kRowsA) {
      const int64_t n = n0 + row < N ? n0 + row : N - 1;
      src[i] = Wq + n * kp + 16 * unit[i];
    } else {
      const int64_t m = m0 + row - kRowsA < M ? m0 + row - kRowsA : M - 1;
      src[i] = Xq + m * kp + 16 * unit[i];
    }
  }
  const int steps = static_cast<int>((kp + 63) >> 6);
  const int tail_units = static_cast<int>(kp - (static_cast<int64_t>(steps - 1) << 6)) >> 4;  // 1..4
  auto request = [&](i32x4* stage, int t) {
    const int tt = t < steps ? t : steps - 1;  // behind the end: the last step again, never read
    const bool tail = tt == steps - 1;
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      const int8_t* from = src[i] + static_cast<int64_t>(tt) * 64;
      if (tail && unit[i] >= tail_units) from = reinterpret_cast<const int8_t*>(&kZeroUnit[0]);
      __builtin_amdgcn_global_load_lds(
          static_cast<const void*>(from),
          reinterpret_cast<__attribute__((address_space(3))) void*>(
              reinterpret_cast<uintptr_t>(stage + i * kThreads + wave * 64)),
          16, 0, 0);
    }
  };
  const int place = (g + (r >> 1)) & 3;  // 16-row blocks start at multiples of 4 half-rows
  const int at_a = (wa * TA * 16 + r) * 4 + place, at_b = (kRowsA + wb * TB * 16 + r) * 4 + place;
  i32x4 fa[2][TA], fb[2][TB], acc[TA][TB] = {};
  auto read = [&](const i32x4* stage, i32x4 (&a)[TA], i32x4 (&b)[TB]) {
#pragma unroll
    for (int j = 0; j < TB; ++j) b[j] = stage[at_b + 64 * j];
#pragma unroll
    for (int i = 0; i < TA; ++i) a[i] = stage[at_a + 64 * i];
  };
  auto step = [&](int t, i32x4* next, i32x4* free_stage, auto P) {
    constexpr int p = decltype(P)::value;
    wait_loads<kLoads>();
    barrier_no_fence();
    request(free_stage, t + 3);
    __builtin_amdgcn_sched_barrier(0);
    read(next, fa[1 - p], fb[1 - p]);
#pragma unroll
    for (int i = 0; i < TA; ++i)
#pragma unroll
      for (int j = 0; j < TB; ++j)
        acc[i][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(fa[p][i], fb[p][j], acc[i][j], 0, 0, 0);
    // MFMAs, then the one fragment read that falls to them: the wait before
    // the first MFMA finds only the previous step's reads, long done.
    constexpr int kReads = TA + TB, kPer = TA * TB / kReads > 0 ? TA * TB / kReads : 1;
#pragma unroll
    for (int i = 0; i < kReads; ++i) {
      __builtin_amdgcn_sched_group_barrier(0x008, kPer, 0);
      __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
    }
    __builtin_amdgcn_sched_group_barrier(0x008, TA * TB, 0);
    __builtin_amdgcn_sched_barrier(0);
  };
  request(st0, 0);
  request(st1, 1);
  request(st2, 2);
  wait_loads<2 * kLoads>();
  barrier_no_fence();
  read(st0, fa[0], fb[0]);
  constexpr std::integral_constant<int, 0> even{};
  constexpr std::integral_constant<int, 1> odd{};
  int t = 0;
  for (; t + 4 <= steps; t += 4) {
    step(t, st1, st3, even);
    step(t + 1, st2, st0, odd);
    step(t + 2, st3, st1, even);
    step(t + 3, st0, st2, odd);
  }
  if (t < steps) step(t, st1, st3, even);
  if (t + 1 < steps) step(t + 1, st2, st0, odd);
  if (t + 2 < steps) step(t + 2, st3, st1, even);
  __builtin_amdgcn_s_waitcnt(0);  // no load may land after the workgroup has left

  const bool whole = (N & 3) == 0 && n0 + kRowsA <= N && m0 + kRowsB <= M;
  const int64_t nw = n0 + wa * TA * 16 + 4 * g, mw = m0 + wb * TB * 16 + r;
  if (whole) {
    store_tile<DT, TA, TB, true>(Y, acc, sx, sw, bias, mw, nw, M, N);
  } else {
    store_tile<DT, TA, TB, false>(Y, acc, sx, sw, bias, mw, nw, M, N);
  }
}

// ---------------------------------------------------------------------------
// Host side.
// ---------------------------------------------------------------------------
bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }
bool dtype_ok(int d) { return d == FP6_FP16 || d == FP6_BF16; }

template <int DT, bool VEC>
int launch_quantize_t(const void* X, int64_t ldx, int64_t M, int64_t K, void* Xq, void* scales, hipStream_t s) {
  int k = static_cast<int>(K), kp = static_cast<int>(fp6_int8_padded_k(K));
  const int thr = kp <= 1024 ? 64 : 256;
  // A grid holds fewer than 2^32 threads: at most 2^22 rows per launch.
  constexpr int64_t kRows = int64_t(1) << 22;
  for (int64_t m0 = 0; m0 < M; m0 += kRows) {
    const uint16_t* x = static_cast<const uint16_t*>(X) + m0 * ldx;
    int8_t* q = static_cast<int8_t*>(Xq) + m0 * kp;
    float* sc = static_cast<float*>(scales) + m0;
    void* args[] = {&x, &ldx, &k, &kp, &q, &sc};
    const dim3 grid(static_cast<unsigned>(M - m0 < kRows ? M - m0 : kRows));
    const int st = launch(reinterpret_cast<const void*>(&i8_quantize<DT, VEC>), grid, dim3(thr), args, s);
    if (st != FP6_OK) return st;
  }
  return FP6_OK;
}

int launch_quantize(int dtype, const void* X, int64_t ldx, int64_t M, int64_t K, void* Xq, void* scales,
                    hipStream_t s) {
  const bool vec = aligned(X, 16) && ldx % 8 == 0;
  if (dtype == FP6_FP16)
    return vec ? launch_quantize_t<FP6_FP16, true>(X, ldx, M, K, Xq, scales, s)
               : launch_quantize_t<FP6_FP16, false>(X, ldx, M, K, Xq, scales, s);
  return vec ? launch_quantize_t<FP6_BF16, true>(X, ldx, M, K, Xq, scales, s)
             : launch_quantize_t<FP6_BF16, false>(X, ldx, M, K, Xq, scales, s);
}

struct Product {
  const void *xq, *sx, *wq, *sw, *bias;
  void* y;
  int64_t M, N, kp;
};

template <int DT, int RB, int MB, int S>
int launch_skinny(const Product& p, hipStream_t s) {
  const int8_t *x = static_cast<const int8_t*>(p.xq), *w = static_cast<const int8_t*>(p.wq);
  const float *sx = static_cast<const float*>(p.sx), *sw = static_cast<const float*>(p.sw);
  const void* bias = p.bias;
  // The grid's second dimension holds at most 65535 groups of tokens.
  const int64_t per = int64_t(65535) * 16 * MB;
  for (int64_t m0 = 0; m0 < p.M; m0 += per) {
    int64_t M = p.M - m0 < per ? p.M - m0 : per, N = p.N, kp = p.kp;
    const int8_t* xm = x + m0 * kp;
    const float* sxm = sx + m0;
    void* y = static_cast<uint16_t*>(p.y) + m0 * N;
    void* args[] = {&xm, &sxm, &w, &sw, &bias, &y, &M, &N, &kp};
    const dim3 grid(static_cast<unsigned>(ceil_div(N, 16 * RB)), static_cast<unsigned>(ceil_div(M, 16 * MB)));
    const int st = launch(reinterpret_cast<const void*>(&i8_skinny<DT, RB, MB, S>), grid, dim3(512), args, s);
    if (st != FP6_OK) return st;
  }
  return FP6_OK;
}

template <int DT, int WA, int WB, int TA, int TB>
int launch_tiled(const Product& p, hipStream_t s) {
  const int8_t *x = static_cast<const int8_t*>(p.xq), *w = static_cast<const int8_t*>(p.wq);
  const float *sx = static_cast<const float*>(p.sx), *sw = static_cast<const float*>(p.sw);
  const void* bias = p.bias;
  void* y = p.y;
  int64_t M = p.M, N = p.N, kp = p.kp;
  void* args[] = {&x, &sx, &w, &sw, &bias, &y, &M, &N, &kp};
  // At most 2^36 / 2^12 tiles of 64 * 64 or more, under 2^32 threads in all... 
  const int64_t tiles = ceil_div(M, 16 * WB * TB) * ceil_div(N, 16 * WA * TA);
  return launch(reinterpret_cast<const void*>(&i8_tiled<DT, WA, WB, TA, TB>), dim3(static_cast<unsigned>(tiles)),
                dim3(64 * WA * WB), args, s);
}

template <int DT>
int launch_product_t(const Product& p, hipStream_t s) {
  const int64_t big = ceil_div(p.M, 256) * ceil_div(p.N, 256);
  if (p.M > 64 && big >= 192) return launch_tiled<DT, 2, 4, 8, 4>(p, s);
  if (p.M > 64) return launch_tiled<DT, 2, 2, 4, 4>(p, s);
  if (p.M <= 16) return launch_skinny<DT, 1, 1, 4>(p, s);
  if (p.M <= 32) return launch_skinny<DT, 1, 2, 4>(p, s);
  return launch_skinny<DT, 2, 4, 2>(p, s);
}

int launch_product(int dtype, const Product& p, hipStream_t s) {
  return dtype == FP6_FP16 ? launch_product_t<FP6_FP16>(p, s) : launch_product_t<FP6_BF16>(p, s);
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

int fp6_int8_linear(const void* Xq, const void* sx, const void* Wq, const void* sw, const void* bias, int dtype,
                    void* Y, int64_t M, int64_t N, int64_t Kp, void* stream) {
  if (!dtype_ok(dtype)) return FP6_E_VALUE;
  if (Kp < 1 || Kp % 16 || Kp > fp6::kInt8MaxK || !sizes_ok(M, N, Kp)) return FP6_E_SHAPE;
  if (M == 0) return FP6_OK;
  if (!Xq || !sx || !Wq || !sw || !Y) return FP6_E_NULL;
  if (!aligned(Xq, 16) || !aligned(Wq, 16) || !aligned(Y, 16) || !aligned(sx, 4) || !aligned(sw, 4) ||
      !aligned(bias, 2))
    return FP6_E_ALIGN;
  return launch_product(dtype, Product{Xq, sx, Wq, sw, bias, Y, M, N, Kp}, static_cast<hipStream_t>(stream));
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
  const int st = launch_quantize(x_dtype, X, ldx, M, K, xq, sx, s);
  if (st != FP6_OK) return st;
  return launch_product(dtype, Product{xq, sx, Wq, sw, bias, Y, M, N, kp}, s);
}

}  // extern "C"
