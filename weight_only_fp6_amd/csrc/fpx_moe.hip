// Mixture-of-experts layer for few tokens with FPx weights (fpx_moe.h):
// router, top-k choice, gated experts.  The weights are rebuilt in registers
// with the same splice as the dense kernels (fpx_device.h).
//
// Tokens are handled in groups of 64 (one lane of a wave per token); a group
// is a grid index of its own, and every kernel below is described for one.

#include <hip/hip_runtime.h>

#include <cstdint>

#include "fp6_limits.h"
#include "fpx_device.h"
#include "fpx_moe.h"

namespace {

constexpr int kGroup = 64;  // tokens per group
constexpr int kMaxK = static_cast<int>(fp6::kMoeMaxTopK);
constexpr int kMaxE = static_cast<int>(fp6::kMoeMaxExperts);

// The gated values h go from the first to the second product as two fp16
// numbers, hi = fp16(h * 2^-8) and lo = fp16((h * 2^-8 - hi) * 2^11): 22 bits,
// where one fp16 would cost as much precision as the final rounding does (and
// overflow from 65504 on, which gated values of large models reach).  The
// second product runs both through the matrix units; it is bound by the
// weights' bytes, so the second pass is free.
constexpr float kHScale = 0x1p-8f, kLoScale = 0x1p11f;

struct MoeShape {
  int T, E, k, H, I;
};

// ---------------------------------------------------------------------------
// Router logits in 64 bits.  A product of two fp16 numbers is exact in fp32,
// and a sum of them in fp64 loses nothing that a choice between experts could
// hang on: rows of equal weights tie exactly.  One workgroup per expert and TB
// tokens, its waves and lanes split H; fixed-order sums.
// ---------------------------------------------------------------------------
template <int TB>
__global__ __launch_bounds__(256) void moe_logits(const _Float16* __restrict__ X, const _Float16* __restrict__ R,
                                                  double* __restrict__ logits, int T, int E, int H) {
  __shared__ double part[4][TB];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int e = blockIdx.x, t0 = blockIdx.y * TB;
  const half8v* w = reinterpret_cast<const half8v*>(R + static_cast<int64_t>(e) * H);
  const half8v* x[TB];
#pragma unroll
  for (int b = 0; b < TB; ++b)
    x[b] = reinterpret_cast<const half8v*>(X + static_cast<int64_t>(t0 + b < T ? t0 + b : T - 1) * H);
  double acc[TB] = {};
  for (int u = threadIdx.x; u < H / 8; u += 256) {
    const half8v wv = w[u];
#pragma unroll
    for (int b = 0; b < TB; ++b) {
      const half8v xv = x[b][u];
#pragma unroll
      for (int i = 0; i < 8; ++i) acc[b] += static_cast<double>(static_cast<float>(wv[i]) * static_cast<float>(xv[i]));
    }
  }
#pragma unroll
  for (int b = 0; b < TB; ++b) {
#pragma unroll
    for (int d = 32; d > 0; d >>= 1) acc[b] += __shfl_xor(acc[b], d);
    if (lane == 0) part[wave][b] = acc[b];
  }
  __syncthreads();
  if (threadIdx.x < TB && t0 + static_cast<int>(threadIdx.x) < T)
    logits[static_cast<int64_t>(t0 + threadIdx.x) * E + e] =
        ((part[0][threadIdx.x] + part[1][threadIdx.x]) + part[2][threadIdx.x]) + part[3][threadIdx.x];
}

// A logit as an unsigned key in the same order; -0 ties with +0, NaN is above
// everything.
__device__ __forceinline__ uint64_t logit_key(double l) {
  if (l != l) return ~uint64_t(0);
  const uint64_t b = __builtin_bit_cast(uint64_t, l + 0.0);
  return (b >> 63) ? ~b : b | (uint64_t(1) << 63);
}

// Top-k of one token by one wave: an expert's place is the number of experts
// before it in the order (larger logit first, then lower index), counted
// against every key in LDS.  Softmax in fp32 from differences formed in fp64.
__global__ __launch_bounds__(64) void moe_topk(const double* __restrict__ logits, int E, int k, int renorm,
                                               int* __restrict__ ids, float* __restrict__ weights) {
  __shared__ uint64_t keys[kMaxE];
  __shared__ int best[kMaxK];
  __shared__ double best_l[kMaxK];
  const int lane = threadIdx.x;
  const int64_t t = blockIdx.x;
  const double* l = logits + t * E;
  for (int e = lane; e < E; e += 64) keys[e] = logit_key(l[e]);
  __syncthreads();
  for (int e = lane; e < E; e += 64) {
    const uint64_t key = keys[e];
    int place = 0;
    for (int o = 0; o < E; ++o) {
      const uint64_t other = keys[o];
      place += other > key || (other == key && o < e);
    }
    if (place < k) {
      best[place] = e;
      best_l[place] = l[e];
    }
  }
  __syncthreads();
  const double top = best_l[0];
  float sum = 0.0f;
  if (renorm) {
    for (int j = 0; j < k; ++j) sum += expf(static_cast<float>(best_l[j] - top));
  } else {
    for (int e = lane; e < E; e += 64) sum += expf(static_cast<float>(l[e] - top));
#pragma unroll
    for (int d = 32; d > 0; d >>= 1) sum += __shfl_xor(sum, d);
  }
  if (lane < k) {
    ids[t * k + lane] = best[lane];
    weights[t * k + lane] = expf(static_cast<float>(best_l[lane] - top)) / sum;
  }
}

// ---------------------------------------------------------------------------
// Which tokens of a group chose an expert.  A wave's lane is a token; `first`
// is its first choice of this expert (pair index inside the group) and `w` the
// sum of the weights of all its choices of it.
// ---------------------------------------------------------------------------
__device__ __forceinline__ uint64_t tokens_of(const short* ids, int tokens, int k, int e, int lane, int& first) {
  first = -1;
  if (lane < tokens)
    for (int j = k - 1; j >= 0; --j)
      if (ids[lane * k + j] == e) first = lane * k + j;
  return __ballot(first >= 0);
}

// The group's ids as 16-bit numbers in LDS, -1 for a choice that is not served.
__device__ __forceinline__ void load_ids(short* dst, const int* ids, int pairs, int E) {
  for (int i = threadIdx.x; i < pairs; i += blockDim.x) {
    const int e = ids[i];
    dst[i] = static_cast<short>(e >= 0 && e < E ? e : -1);
  }
}

// ---------------------------------------------------------------------------
// Gate and up products with the gated activation.  A workgroup takes one
// expert and 8/ks row blocks (16 rows of the gate and the same 16 of the up
// projection each); ks waves split K = H of a row block and add through LDS.
// The columns of the MFMAs are the expert's tokens, gathered; columns behind
// the last repeat the first and are not stored.
// ---------------------------------------------------------------------------
template <int F, int MT>
__global__ __launch_bounds__(512) void moe_gate_up(const _Float16* __restrict__ X, const int* __restrict__ ids_g,
                                                   const float* __restrict__ weights_g,
                                                   const u32x4* __restrict__ wp, const _Float16* __restrict__ scales,
                                                   _Float16* __restrict__ hi, _Float16* __restrict__ lo, MoeShape s,
                                                   int ks, int by_pair) {
  __shared__ short ids[kGroup * kMaxK];
  __shared__ short col_token[kGroup], col_pair[kGroup];
  __shared__ float col_w[kGroup];
  __shared__ float4v red[8][2 * MT][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int r = lane & 15, g = lane >> 4;
  const int t0 = blockIdx.z * kGroup;
  const int tokens = s.T - t0 < kGroup ? s.T - t0 : kGroup;
  const int pairs = tokens * s.k;
  load_ids(ids, ids_g + static_cast<int64_t>(t0) * s.k, pairs, s.E);
  __syncthreads();
  // Fewer pairs than experts: the grid has one slot per pair, and the first
  // pair of an expert takes it; else one slot per expert.
  int e = blockIdx.y;
  if (by_pair) {
    if (e >= pairs) return;
    const int p = e;
    e = ids[p];
    if (e < 0) return;
    for (int q = 0; q < p; ++q)
      if (ids[q] == e) return;
  }
  int first;
  const uint64_t mask = tokens_of(ids, tokens, s.k, e, lane, first);
  const int n = __popcll(mask);
  if (n == 0) return;
  if (wave == 0 && first >= 0) {
    const int c = __popcll(mask & ((uint64_t(1) << lane) - 1));
    float w = 0.0f;
    for (int j = 0; j < s.k; ++j)
      if (ids[lane * s.k + j] == e) w += weights_g[static_cast<int64_t>(t0 + lane) * s.k + j];
    col_token[c] = static_cast<short>(lane);
    col_pair[c] = static_cast<short>(first);
    col_w[c] = w;
  }
  __syncthreads();

  const int rb = wave / ks, kslice = wave - rb * ks;
  const int iblocks = s.I >> 4, ktiles = s.H >> 8;
  int nb = blockIdx.x * (8 / ks) + rb;
  const bool live = nb < iblocks;
  if (!live) nb = iblocks - 1;
  const int64_t nblocks = 2 * static_cast<int64_t>(iblocks);
  const int64_t kstr = nblocks * Fmt<F>::kTileQuads;
  const u32x4* wg = wp + static_cast<int64_t>(e) * ktiles * kstr + nb * static_cast<int64_t>(Fmt<F>::kTileQuads) + lane;
  const u32x4* wu = wg + static_cast<int64_t>(iblocks) * Fmt<F>::kTileQuads;
  const _Float16* sc = scales + static_cast<int64_t>(e) * 2 * s.I + nb * 16 + r;
  const half2v sg = scale2_of<F>(sc[0]), su = scale2_of<F>(sc[s.I]);
  const int kt0 = kslice * ktiles / ks, kt1 = (kslice + 1) * ktiles / ks;

  for (int c0 = 0; c0 < n; c0 += 16 * MT) {
    const _Float16* xr[MT];
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      const int c = c0 + 16 * m + r;
      xr[m] = X + static_cast<int64_t>(t0 + col_token[c < n ? c : 0]) * s.H + 8 * g;
    }
    float4v ag[MT], au[MT];
#pragma unroll
    for (int m = 0; m < MT; ++m) ag[m] = au[m] = float4v{0.f, 0.f, 0.f, 0.f};
    for (int kt = kt0; kt < kt1; ++kt) {
      typename Fmt<F>::Tile tg, tu;
      Fmt<F>::template load<true>(tg, wg + kt * kstr, lane);
      Fmt<F>::template load<true>(tu, wu + kt * kstr, lane);
      half8v xf[MT][8];
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int j = 0; j < 8; ++j) xf[m][j] = *reinterpret_cast<const half8v*>(xr[m] + kt * 256 + 32 * j);
      auto step = [&](auto J) {
        constexpr int j = decltype(J)::value;
        const half8v a = Fmt<F>::template step<j>(tg, sg), b = Fmt<F>::template step<j>(tu, su);
#pragma unroll
        for (int m = 0; m < MT; ++m) {
          ag[m] = __builtin_amdgcn_mfma_f32_16x16x32_f16(a, xf[m][j], ag[m], 0, 0, 0);
          au[m] = __builtin_amdgcn_mfma_f32_16x16x32_f16(b, xf[m][j], au[m], 0, 0, 0);
        }
      };
      step(std::integral_constant<int, 0>{}); step(std::integral_constant<int, 1>{});
      step(std::integral_constant<int, 2>{}); step(std::integral_constant<int, 3>{});
      step(std::integral_constant<int, 4>{}); step(std::integral_constant<int, 5>{});
      step(std::integral_constant<int, 6>{}); step(std::integral_constant<int, 7>{});
    }
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      red[wave][2 * m][lane] = ag[m];
      red[wave][2 * m + 1][lane] = au[m];
    }
    __syncthreads();
    // Wave (rb, kslice) sums and stores the column blocks kslice, kslice + ks, ...
    for (int m = kslice; m < MT; m += ks) {
      const int c = c0 + 16 * m + r;
      if (live && c < n) {
        float4v vg = red[rb * ks][2 * m][lane], vu = red[rb * ks][2 * m + 1][lane];
        for (int w = 1; w < ks; ++w) {
          vg += red[rb * ks + w][2 * m][lane];
          vu += red[rb * ks + w][2 * m + 1][lane];
        }
        half4v oh, ol;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float h = (vg[i] / (1.0f + expf(-vg[i]))) * vu[i] * col_w[c] * kHScale;
          oh[i] = static_cast<_Float16>(h);
          const float hf = static_cast<float>(oh[i]);
          ol[i] = __builtin_isinf(hf) ? static_cast<_Float16>(0.0f) : static_cast<_Float16>((h - hf) * kLoScale);
        }
        const int64_t at = (static_cast<int64_t>(t0) * s.k + col_pair[c]) * s.I + nb * 16 + 4 * g;
        *reinterpret_cast<half4v*>(hi + at) = oh;
        *reinterpret_cast<half4v*>(lo + at) = ol;
      }
    }
    __syncthreads();
  }
}

// ---------------------------------------------------------------------------
// Down product and the sum over experts.  A workgroup owns 16 rows of the
// output for all tokens of the group; its waves share the list of (expert,
// k-tile) of the experts that any token chose, in equal contiguous parts.  The
// weights of the choice are already in h, so a wave simply adds: the MFMA
// columns are an expert's tokens, gathered, and after its last tile of an
// expert the wave adds them to its own [token][row] sums in LDS.  The waves'
// sums are added in wave order and rounded once.
// ---------------------------------------------------------------------------
template <int F, int NW, int TT>
__global__ __launch_bounds__(64 * NW) void moe_down(const _Float16* __restrict__ hi, const _Float16* __restrict__ lo,
                                                    const int* __restrict__ ids_g, const u32x4* __restrict__ wp,
                                                    const _Float16* __restrict__ scales, _Float16* __restrict__ Y,
                                                    MoeShape s) {
  __shared__ short ids[kGroup * kMaxK];
  __shared__ short active[kMaxE];
  __shared__ uint64_t chosen[kMaxE / 64];
  __shared__ short cols[NW][kGroup], pair_of[NW][kGroup];
  __shared__ float ysum[NW][TT][16];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int r = lane & 15, g = lane >> 4;
  const int t0 = blockIdx.z * kGroup;
  const int tokens = s.T - t0 < kGroup ? s.T - t0 : kGroup;
  const int pairs = tokens * s.k;
  load_ids(ids, ids_g + static_cast<int64_t>(t0) * s.k, pairs, s.E);
  if (threadIdx.x < kMaxE / 64) chosen[threadIdx.x] = 0;
  for (int i = threadIdx.x; i < NW * TT * 16; i += 64 * NW) (&ysum[0][0][0])[i] = 0.0f;
  __syncthreads();
  for (int i = threadIdx.x; i < pairs; i += 64 * NW) {
    const int e = ids[i];
    if (e >= 0) atomicOr(reinterpret_cast<unsigned long long*>(&chosen[e >> 6]), 1ull << (e & 63));
  }
  __syncthreads();
  int na = 0;
  for (int b = 0; 64 * b < s.E; ++b) {
    const uint64_t m = chosen[b];
    if (wave == 0 && ((m >> lane) & 1)) active[na + __popcll(m & ((uint64_t(1) << lane) - 1))] = static_cast<short>(64 * b + lane);
    na += __popcll(m);
  }
  __syncthreads();

  const int nb = blockIdx.x, ktiles = s.I >> 8;
  const int64_t nblocks = s.H >> 4, kstr = nblocks * Fmt<F>::kTileQuads;
  const int total = na * ktiles;
  const int f0 = static_cast<int>(static_cast<int64_t>(wave) * total / NW);
  const int f1 = static_cast<int>(static_cast<int64_t>(wave + 1) * total / NW);
  for (int f = f0; f < f1;) {
    const int a = f / ktiles, kt0 = f - a * ktiles, e = active[a];
    const int kt1 = f1 - f < ktiles - kt0 ? kt0 + (f1 - f) : ktiles;
    f += kt1 - kt0;
    int first;
    const uint64_t mask = tokens_of(ids, tokens, s.k, e, lane, first);
    const int n = __popcll(mask);
    if (first >= 0) {
      const int c = __popcll(mask & ((uint64_t(1) << lane) - 1));
      cols[wave][c] = static_cast<short>(lane);
      pair_of[wave][c] = static_cast<short>(first);
    }
    __builtin_amdgcn_wave_barrier();
    const half2v s2 = scale2_of<F>(scales[static_cast<int64_t>(e) * s.H + nb * 16 + r]);
    const u32x4* w = wp + static_cast<int64_t>(e) * ktiles * kstr + nb * static_cast<int64_t>(Fmt<F>::kTileQuads) + lane;
    for (int c0 = 0; c0 < n; c0 += 16) {
      const int c = c0 + r;
      const int64_t at = (static_cast<int64_t>(t0) * s.k + pair_of[wave][c < n ? c : 0]) * s.I + 8 * g;
      float4v ah = {0.f, 0.f, 0.f, 0.f}, al = {0.f, 0.f, 0.f, 0.f};
      for (int kt = kt0; kt < kt1; ++kt) {
        typename Fmt<F>::Tile t;
        Fmt<F>::template load<true>(t, w + kt * kstr, lane);
        half8v fh[8], fl[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          fh[j] = *reinterpret_cast<const half8v*>(hi + at + kt * 256 + 32 * j);
          fl[j] = *reinterpret_cast<const half8v*>(lo + at + kt * 256 + 32 * j);
        }
        auto step = [&](auto J) {
          constexpr int j = decltype(J)::value;
          const half8v av = Fmt<F>::template step<j>(t, s2);
          ah = __builtin_amdgcn_mfma_f32_16x16x32_f16(av, fh[j], ah, 0, 0, 0);
          al = __builtin_amdgcn_mfma_f32_16x16x32_f16(av, fl[j], al, 0, 0, 0);
        };
        step(std::integral_constant<int, 0>{}); step(std::integral_constant<int, 1>{});
        step(std::integral_constant<int, 2>{}); step(std::integral_constant<int, 3>{});
        step(std::integral_constant<int, 4>{}); step(std::integral_constant<int, 5>{});
        step(std::integral_constant<int, 6>{}); step(std::integral_constant<int, 7>{});
      }
      if (c < n) {
        float4v* y = reinterpret_cast<float4v*>(&ysum[wave][cols[wave][c]][4 * g]);
        *y = *y + (ah + al * (1.0f / kLoScale));
      }
    }
    __builtin_amdgcn_wave_barrier();
  }
  __syncthreads();
  for (int i = threadIdx.x; i < tokens * 16; i += 64 * NW) {
    const int t = i >> 4, row = i & 15;
    float y = ysum[0][t][row];
    for (int w = 1; w < NW; ++w) y += ysum[w][t][row];
    Y[static_cast<int64_t>(t0 + t) * s.H + nb * 16 + row] = static_cast<_Float16>(y * (1.0f / kHScale));
  }
}

// ---------------------------------------------------------------------------
// Host side.
// ---------------------------------------------------------------------------
bool moe_aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

bool moe_sizes_ok(int64_t T, int64_t E, int64_t k, int64_t H, int64_t I) {
  constexpr int64_t kMaxSide = int64_t(1) << 20;
  return T >= 0 && T <= fp6::kMoeMaxTokens && E >= 1 && E <= fp6::kMoeMaxExperts && k >= 1 && k <= fp6::kMoeMaxTopK &&
         H >= 256 && H <= kMaxSide && H % 256 == 0 && I >= 256 && I <= kMaxSide && I % 256 == 0 &&
         2 * I * H <= fp6::kMaxNK;
}

size_t round256(size_t n) { return (n + 255) / 256 * 256; }

struct Workspace {
  size_t logits, hi, lo, bytes;
};
Workspace workspace_of(int64_t T, int64_t E, int64_t k, int64_t I) {
  Workspace w;
  w.logits = 0;
  w.hi = round256(static_cast<size_t>(T) * E * sizeof(double));
  w.lo = w.hi + round256(static_cast<size_t>(T) * k * I * 2);
  w.bytes = w.lo + round256(static_cast<size_t>(T) * k * I * 2);
  return w;
}

struct MoeCall {
  const _Float16* X;
  const int* ids;
  const float* weights;
  const u32x4 *gate_up, *down;
  const _Float16 *gate_up_scales, *down_scales;
  _Float16 *Y, *hi, *lo;
  MoeShape s;
  hipStream_t stream;
};

int moe_launch(const void* kern, dim3 grid, dim3 block, void** args, hipStream_t stream) {
  return hipLaunchKernel(kern, grid, block, args, 0, stream) == hipSuccess ? FP6_OK : FP6_E_HIP;
}

template <int F>
int launch_experts(const MoeCall& c) {
  MoeShape s = c.s;
  const int group_tokens = s.T < kGroup ? s.T : kGroup;
  const unsigned groups = static_cast<unsigned>(fpx_ceil_div(s.T, kGroup));
  int ks = 8;
  while (ks > 1 && ks > s.H / 256) ks >>= 1;
  int by_pair = group_tokens * s.k < s.E;
  const unsigned slots = by_pair ? group_tokens * s.k : s.E;
  const _Float16* X = c.X;
  const int* ids = c.ids;
  const float* weights = c.weights;
  const u32x4* w = c.gate_up;
  const _Float16* sc = c.gate_up_scales;
  _Float16 *hi = c.hi, *lo = c.lo, *Y = c.Y;
  {
    void* args[] = {&X, &ids, &weights, &w, &sc, &hi, &lo, &s, &ks, &by_pair};
    const dim3 grid(static_cast<unsigned>(fpx_ceil_div(s.I / 16, 8 / ks)), slots, groups);
    const void* kern = group_tokens <= 16 ? reinterpret_cast<const void*>(&moe_gate_up<F, 1>)
                                          : reinterpret_cast<const void*>(&moe_gate_up<F, 2>);
    const int st = moe_launch(kern, grid, dim3(512), args, c.stream);
    if (st != FP6_OK) return st;
  }
  w = c.down;
  sc = c.down_scales;
  void* args[] = {&hi, &lo, &ids, &w, &sc, &Y, &s};
  const dim3 grid(static_cast<unsigned>(s.H / 16), 1, groups);
  const void* kern = group_tokens <= 16 ? reinterpret_cast<const void*>(&moe_down<F, 16, 16>)
                                        : reinterpret_cast<const void*>(&moe_down<F, 8, 64>);
  return moe_launch(kern, grid, dim3(group_tokens <= 16 ? 1024 : 512), args, c.stream);
}

int launch_experts_format(int format, const MoeCall& c) {
  switch (format) {
    case FPX_E3M2: return launch_experts<kE3M2>(c);
    case FPX_E2M3: return launch_experts<kE2M3>(c);
    case FPX_E2M2: return launch_experts<kE2M2>(c);
    case FPX_E2M1: return launch_experts<kE2M1>(c);
    default: return FP6_E_VALUE;
  }
}

template <int TB>
int launch_logits(const _Float16* X, const _Float16* R, double* logits, MoeShape s, hipStream_t stream) {
  void* args[] = {&X, &R, &logits, &s.T, &s.E, &s.H};
  const dim3 grid(s.E, static_cast<unsigned>(fpx_ceil_div(s.T, TB)));
  return moe_launch(reinterpret_cast<const void*>(&moe_logits<TB>), grid, dim3(256), args, stream);
}

int check_experts(int format, const void* X, const void* ids, const void* weights, const void* gate_up,
                  const void* gate_up_scales, const void* down, const void* down_scales, const void* Y, int64_t T,
                  int64_t E, int64_t k, int64_t H, int64_t I, const void* workspace, size_t workspace_bytes) {
  if (format < 0 || format >= fpx::kNumFormats) return FP6_E_VALUE;
  if (!moe_sizes_ok(T, E, k, H, I)) return FP6_E_SHAPE;
  if (T == 0) return FP6_OK;
  if (!X || !ids || !weights || !gate_up || !gate_up_scales || !down || !down_scales || !Y || !workspace)
    return FP6_E_NULL;
  if (!moe_aligned(X, 16) || !moe_aligned(gate_up, 16) || !moe_aligned(down, 16) || !moe_aligned(Y, 16) ||
      !moe_aligned(ids, 4) || !moe_aligned(weights, 4) || !moe_aligned(gate_up_scales, 2) ||
      !moe_aligned(down_scales, 2) || !moe_aligned(workspace, 256))
    return FP6_E_ALIGN;
  if (workspace_bytes < fpx_moe_workspace_bytes(T, E, k, H, I)) return FP6_E_SIZE;
  return FP6_OK;
}

MoeCall make_call(const void* X, const void* ids, const void* weights, const void* gate_up,
                  const void* gate_up_scales, const void* down, const void* down_scales, void* Y, int64_t T, int64_t E,
                  int64_t k, int64_t H, int64_t I, void* workspace, void* stream) {
  const Workspace w = workspace_of(T, E, k, I);
  char* ws = static_cast<char*>(workspace);
  MoeCall c;
  c.X = static_cast<const _Float16*>(X);
  c.ids = static_cast<const int*>(ids);
  c.weights = static_cast<const float*>(weights);
  c.gate_up = static_cast<const u32x4*>(gate_up);
  c.gate_up_scales = static_cast<const _Float16*>(gate_up_scales);
  c.down = static_cast<const u32x4*>(down);
  c.down_scales = static_cast<const _Float16*>(down_scales);
  c.Y = static_cast<_Float16*>(Y);
  c.hi = reinterpret_cast<_Float16*>(ws + w.hi);
  c.lo = reinterpret_cast<_Float16*>(ws + w.lo);
  c.s = MoeShape{static_cast<int>(T), static_cast<int>(E), static_cast<int>(k), static_cast<int>(H), static_cast<int>(I)};
  c.stream = static_cast<hipStream_t>(stream);
  return c;
}

}  // namespace

extern "C" {

size_t fpx_moe_workspace_bytes(int64_t T, int64_t E, int64_t top_k, int64_t H, int64_t I) {
  if (!moe_sizes_ok(T, E, top_k, H, I) || T == 0) return 0;
  return workspace_of(T, E, top_k, I).bytes;
}

int fpx_moe_experts(int format, const void* X, const void* ids, const void* weights, const void* gate_up,
                    const void* gate_up_scales, const void* down, const void* down_scales, void* Y, int64_t T,
                    int64_t E, int64_t top_k, int64_t H, int64_t I, void* workspace, size_t workspace_bytes,
                    void* stream) {
  const int st = check_experts(format, X, ids, weights, gate_up, gate_up_scales, down, down_scales, Y, T, E, top_k, H,
                               I, workspace, workspace_bytes);
  if (st != FP6_OK || T == 0) return st;
  return launch_experts_format(format, make_call(X, ids, weights, gate_up, gate_up_scales, down, down_scales, Y, T, E,
                                                 top_k, H, I, workspace, stream));
}

int fpx_moe_layer(int format, const void* X, const void* router, const void* gate_up, const void* gate_up_scales,
                  const void* down, const void* down_scales, int renormalize, void* Y, void* ids, void* weights,
                  int64_t T, int64_t E, int64_t top_k, int64_t H, int64_t I, void* workspace, size_t workspace_bytes,
                  void* stream) {
  if (renormalize != 0 && renormalize != 1) return FP6_E_VALUE;
  if (top_k > E) return FP6_E_SHAPE;
  int st = check_experts(format, X, ids, weights, gate_up, gate_up_scales, down, down_scales, Y, T, E, top_k, H, I,
                         workspace, workspace_bytes);
  if (st != FP6_OK || T == 0) return st;
  if (!router) return FP6_E_NULL;
  if (!moe_aligned(router, 16)) return FP6_E_ALIGN;
  const MoeCall c = make_call(X, ids, weights, gate_up, gate_up_scales, down, down_scales, Y, T, E, top_k, H, I,
                              workspace, stream);
  double* logits = static_cast<double*>(workspace);
  const _Float16* R = static_cast<const _Float16*>(router);
  st = T <= 4 ? launch_logits<1>(c.X, R, logits, c.s, c.stream) : launch_logits<4>(c.X, R, logits, c.s, c.stream);
  if (st != FP6_OK) return st;
  int* oi = static_cast<int*>(ids);
  float* ow = static_cast<float*>(weights);
  int E32 = c.s.E, k32 = c.s.k;
  void* args[] = {&logits, &E32, &k32, &renormalize, &oi, &ow};
  st = moe_launch(reinterpret_cast<const void*>(&moe_topk), dim3(static_cast<unsigned>(T)), dim3(64), args, c.stream);
  if (st != FP6_OK) return st;
  return launch_experts_format(format, c);
}

}  // extern "C"
