// Mixture-of-experts layer for few tokens with FPx weights (fpx_moe.h):
// router, top-k choice, gated experts.  The weights are rebuilt in registers
// with the same splice as the dense kernels (fpx_device.h).
//
// Tokens are handled in groups of 64 (one lane of a wave per token); a group
// is a grid index of its own, and every kernel below is described for one.

#include <hip/hip_runtime.h>

#include <cstdint>

#include "fp6_limits.h"
#include "fpx_cus.h"
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

// Sizes up to which the choice is made inside the first product, and up to
// which (tokens x experts x H) its logits are, too.  That is one launch less:
// called one by one 21.0 -> 18.7 us.  In a graph 8192 products take 10.8 us
// instead of 11.4, 16384 13.8 instead of 13.2, 32768 16.5 .. 18.7 instead of
// 12.3 .. 15.1: every workgroup pays for all of them.
constexpr int kFusedE = 128, kFusedT = 4, kFusedProducts = 16384;
// More tokens: up to which router (experts x H) one workgroup per token makes
// logits and choice in one launch instead of two.  8 experts x 1024: 16 tokens
// 17.6 -> 15.3 us for the layer, 256 29.3 -> 26.7, 1024 73.8 -> 71.1; 16 x 4096:
// 24.0 -> 23.6, 60.4 -> 58.6, 185 -> 181; 32 x 4096, 16 tokens 30.0 -> 32.5.
constexpr int kRouteE = 128, kRouteProducts = 65536;
enum Route : int { kGiven, kFromLogits, kFromRouter };
constexpr int kFewPairs = 64, kFewTiles = 32;  // moe_down_few: a lane per pair, two tiles per wave

struct MoeShape {
  int T, E, k, H, I;
};

// ---------------------------------------------------------------------------
// Router logits in 64 bits.  A product of two fp16 numbers is exact in fp32,
// and a sum of them in fp64 loses nothing that a choice between experts could
// hang on: rows of equal weights tie exactly.  One workgroup per expert and TB
// tokens, its waves and lanes split H; fixed-order sums.  Launch and latency:
// 64 experts x 2048, one token 2.5 us.
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
// keys[E], best[k], best_l[k]: the wave's own LDS; every lane < k returns its
// place's expert and weight.
__device__ __forceinline__ void wave_topk(const double* __restrict__ l, int E, int k, int renorm, uint64_t* keys,
                                          int* best, double* best_l, int lane, int& id, float& weight) {
  for (int e = lane; e < E; e += 64) keys[e] = logit_key(l[e]);
  __builtin_amdgcn_wave_barrier();
  for (int e = lane; e < E; e += 64) {
    const uint64_t key = keys[e];
    int place = 0;
#pragma unroll 8
    for (int o = 0; o < E; ++o) {
      const uint64_t other = keys[o];
      place += other > key || (other == key && o < e);
    }
    if (place < k) {
      best[place] = e;
      best_l[place] = l[e];
    }
  }
  __builtin_amdgcn_wave_barrier();
  const double top = best_l[0];
  float sum = 0.0f;
  if (renorm) {
    for (int j = 0; j < k; ++j) sum += expf(static_cast<float>(best_l[j] - top));
  } else {
    for (int e = lane; e < E; e += 64) sum += expf(static_cast<float>(l[e] - top));
#pragma unroll
    for (int d = 32; d > 0; d >>= 1) sum += __shfl_xor(sum, d);
  }
  id = -1;
  weight = 0.0f;
  if (lane < k) {
    id = best[lane];
    weight = expf(static_cast<float>(best_l[lane] - top)) / sum;
  }
}

__global__ __launch_bounds__(64) void moe_topk(const double* __restrict__ logits, int E, int k, int renorm,
                                               int* __restrict__ ids, float* __restrict__ weights) {
  __shared__ uint64_t keys[kMaxE];
  __shared__ int best[kMaxK];
  __shared__ double best_l[kMaxK];
  const int lane = threadIdx.x;
  const int64_t t = blockIdx.x;
  int id;
  float w;
  wave_topk(logits + t * E, E, k, renorm, keys, best, best_l, lane, id, w);
  if (lane < k) {
    ids[t * k + lane] = id;
    weights[t * k + lane] = w;
  }
}

// Logits and choice of one token in one workgroup of 16 waves, for small
// routers (16 experts x 4096, 16 tokens 6.9 us against 4.5 and 3.5).
__global__ __launch_bounds__(1024) void moe_route(const _Float16* __restrict__ X, const _Float16* __restrict__ R, int E,
                                                  int k, int H, int renorm, int* __restrict__ ids,
                                                  float* __restrict__ weights) {
  __shared__ double logits[kRouteE];
  __shared__ uint64_t keys[kRouteE];
  __shared__ int best[kMaxK];
  __shared__ double best_l[kMaxK];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t t = blockIdx.x;
  const half8v* x = reinterpret_cast<const half8v*>(X + t * H);
  for (int e = wave; e < E; e += 16) {
    const half8v* w = reinterpret_cast<const half8v*>(R + static_cast<int64_t>(e) * H);
    double acc = 0.0;
#pragma unroll 4
    for (int u = lane; u < H / 8; u += 64) {
      const half8v wv = w[u], xv = x[u];
#pragma unroll
      for (int i = 0; i < 8; ++i) acc += static_cast<double>(static_cast<float>(wv[i]) * static_cast<float>(xv[i]));
    }
#pragma unroll
    for (int d = 32; d > 0; d >>= 1) acc += __shfl_xor(acc, d);
    if (lane == 0) logits[e] = acc;
  }
  __syncthreads();
  if (wave == 0) {
    int id;
    float w;
    wave_topk(logits, E, k, renorm, keys, best, best_l, lane, id, w);
    if (lane < k) {
      ids[t * k + lane] = id;
      weights[t * k + lane] = w;
    }
  }
}

// ---------------------------------------------------------------------------
// Both products give a workgroup of 4 waves one expert, its tokens, 16 at a time
// (the columns of the MFMAs), and (4/ks)*P row blocks of 16 rows: ks waves split
// K, each takes P consecutive row blocks and holds a k-tile's token fragments
// for all of them.  The weights run through a register ring of D k-tiles: as
// soon as tile (row block p, k-tile t) is multiplied, tile (p, t+D) is
// requested, so D*P tiles are in flight per wave; the token fragments of k-tile
// t+1 are requested when k-tile t begins.  Bound by latency at these sizes: one
// token, 64 experts 2048x1024 with the choice 13.1 us (12.6 MB of weights, 1
// TB/s); 7 tokens, 40 experts 1280x768 e2m3, gate/up 10.6 us.
//
// Which expert: with fewer (token, choice) pairs than experts the grid has one
// slot per pair, and the first pair of an expert takes it; else one slot per
// expert.  Workgroups without work leave at once.  (Further workgroups for an
// expert's tokens behind the 16th, most of them without work, cost 15 of 50 us
// at 64 tokens and 64 experts; the workgroup goes over its weights again
// instead, from the L2 or the 256 MB cache.)
//
// A wave's lane is a token of the group here: `first` is its first choice of
// the expert (pair index inside the group, -1: none), `weight` the sum of the
// weights of all its choices of it.
// ---------------------------------------------------------------------------
struct Choice {
  int first;
  float weight;
};
template <bool WEIGHT>
__device__ __forceinline__ Choice choice_of(const int* __restrict__ ids, const float* __restrict__ weights, int tokens,
                                            int k, int e, int lane) {
  Choice c{-1, 0.0f};
  if (lane < tokens) {
    int id[kMaxK];
    float w[kMaxK];
#pragma unroll
    for (int j = 0; j < kMaxK; ++j) {  // all requested before the first is looked at
      id[j] = -1;
      w[j] = 0.0f;
      if (j < k) {
        id[j] = ids[lane * k + j];
        if constexpr (WEIGHT) w[j] = weights[lane * k + j];
      }
    }
#pragma unroll
    for (int j = kMaxK - 1; j >= 0; --j)
      if (j < k && id[j] == e) c.first = lane * k + j;
#pragma unroll
    for (int j = 0; j < kMaxK; ++j)
      if (j < k && id[j] == e) c.weight += w[j];
  }
  return c;
}

// The same where there is one token only: lane = choice, wave-uniform result.
__device__ __forceinline__ Choice choice_of_one(const int* __restrict__ ids, const float* __restrict__ weights, int k,
                                                int e, int lane) {
  const int id = lane < k ? ids[lane] : -1;
  const float w = lane < k ? weights[lane] : 0.0f;
  uint64_t hits = __ballot(lane < k && id == e);
  Choice c{hits ? __ffsll(static_cast<unsigned long long>(hits)) - 1 : -1, 0.0f};
  for (; hits; hits &= hits - 1)
    c.weight += __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, w),
                                                                    __ffsll(static_cast<unsigned long long>(hits)) - 1));
  return c;
}

// Whether this workgroup has work: any token chose its expert, and (slots by
// pair) the slot's pair is the expert's first.
__device__ __forceinline__ bool has_work(uint64_t mask, int first, int by_pair, int slot) {
  if (mask == 0) return false;
  if (!by_pair) return true;
  return __builtin_amdgcn_readlane(first, __ffsll(static_cast<unsigned long long>(mask)) - 1) == slot;
}

// h = w * silu(gate) * up of 4 rows, as its two halves.
__device__ __forceinline__ void store_gated(_Float16* hi, _Float16* lo, const float4v& gate, const float4v& up, float w) {
  half4v oh, ol;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float h = (gate[i] / (1.0f + expf(-gate[i]))) * up[i] * w * kHScale;
    oh[i] = static_cast<_Float16>(h);
    const float hf = static_cast<float>(oh[i]);
    ol[i] = __builtin_isinf(hf) ? static_cast<_Float16>(0.0f) : static_cast<_Float16>((h - hf) * kLoScale);
  }
  *reinterpret_cast<half4v*>(hi) = oh;
  *reinterpret_cast<half4v*>(lo) = ol;
}

// Gate and up products with the gated activation; row block p of the gate and
// of the up projection go together.  ROUTE: the choice is given, or (few tokens,
// few experts) it is made here, wave t for token t, by every workgroup for
// itself, and written out by the first one: from the logits, or, with a small
// router, from the router itself.
template <int F, int P, int D, int ROUTE>
__global__ __launch_bounds__(256, 2) void moe_gate_up(const _Float16* __restrict__ X, const _Float16* __restrict__ R,
                                                   const double* __restrict__ logits,
                                                   int* __restrict__ ids_g, float* __restrict__ weights_g,
                                                   const u32x4* __restrict__ wp, const _Float16* __restrict__ scales,
                                                   _Float16* __restrict__ hi, _Float16* __restrict__ lo,
                                                   MoeShape s, int ks, int by_pair, int renorm) {
  __shared__ short col_token[4][kGroup], col_pair[4][kGroup];
  __shared__ float col_w[4][kGroup];
  __shared__ float4v red[4][2 * P][64];
  constexpr bool kFused = ROUTE != kGiven;
  __shared__ uint64_t keys[kFused ? kFusedT : 1][kFused ? kFusedE : 1];
  __shared__ int best[kFused ? kFusedT : 1][kMaxK];
  __shared__ double best_l[kFused ? kFusedT : 1][kMaxK];
  __shared__ int f_ids[kFused ? kFusedT * kMaxK : 1];
  __shared__ float f_w[kFused ? kFusedT * kMaxK : 1];
  __shared__ double f_logits[ROUTE == kFromRouter ? kFusedT : 1][ROUTE == kFromRouter ? kFusedE : 1];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r = lane & 15, g = lane >> 4;
  const int t0 = blockIdx.z * kGroup;
  const int tokens = s.T - t0 < kGroup ? s.T - t0 : kGroup;
  const bool first_wg = blockIdx.x == 0 && blockIdx.y == 0;
  const int* ids = ids_g + static_cast<int64_t>(t0) * s.k;
  const float* weights = weights_g + static_cast<int64_t>(t0) * s.k;
  const int kslice = wave % ks, ktiles = s.H >> 8;
  const int kt0 = kslice * ktiles / ks, kt1 = (kslice + 1) * ktiles / ks;  // never empty: ks <= ktiles
  // One token: every column repeats it, and it is known before its experts are.
  const bool one = s.T == 1;
  half8v xf[2][8];
  if (one) {
#pragma unroll
    for (int j = 0; j < 8; ++j) xf[0][j] = *reinterpret_cast<const half8v*>(X + 8 * g + kt0 * 256 + 32 * j);
  }
  if constexpr (kFused) {
    if constexpr (ROUTE == kFromRouter) {
      // Wave w takes experts w, w + 4, ...; sums in fp64 as in moe_logits.
      for (int e = wave; e < s.E; e += 4) {
        double acc[kFusedT] = {};
        for (int u = lane; u < s.H / 8; u += 64) {
          const half8v rv = reinterpret_cast<const half8v*>(R + static_cast<int64_t>(e) * s.H)[u];
#pragma unroll
          for (int t = 0; t < kFusedT; ++t) {
            if (t < tokens) {
              const half8v xv = reinterpret_cast<const half8v*>(X + static_cast<int64_t>(t) * s.H)[u];
#pragma unroll
              for (int i = 0; i < 8; ++i) acc[t] += static_cast<double>(static_cast<float>(rv[i]) * static_cast<float>(xv[i]));
            }
          }
        }
#pragma unroll
        for (int t = 0; t < kFusedT; ++t) {
          if (t < tokens) {
#pragma unroll
            for (int d = 32; d > 0; d >>= 1) acc[t] += __shfl_xor(acc[t], d);
            if (lane == 0) f_logits[t][e] = acc[t];
          }
        }
      }
      __syncthreads();
    }
    if (wave < tokens) {
      const double* l = ROUTE == kFromRouter ? f_logits[wave] : logits + wave * s.E;
      int id;
      float w;
      wave_topk(l, s.E, s.k, renorm, keys[wave], best[wave], best_l[wave], lane, id, w);
      if (lane < s.k) {
        f_ids[wave * s.k + lane] = id;
        f_w[wave * s.k + lane] = w;
        if (first_wg) {
          ids_g[wave * s.k + lane] = id;
          weights_g[wave * s.k + lane] = w;
        }
      }
    }
    __syncthreads();
    ids = f_ids;
    weights = f_w;
  }
  const int slot = blockIdx.y;
  int e = slot;
  if (by_pair) {
    if (slot >= tokens * s.k) return;
    e = __builtin_amdgcn_readfirstlane(ids[slot]);
    if (e < 0 || e >= s.E) return;
  }
  const Choice ch = one ? choice_of_one(ids, weights, s.k, e, lane) : choice_of<true>(ids, weights, tokens, s.k, e, lane);

  const int rb = wave / ks;
  const int iblocks = s.I >> 4;
  const int nb = (blockIdx.x * (4 / ks) + rb) * P;
  const int64_t kstr = 2 * static_cast<int64_t>(iblocks) * Fmt<F>::kTileQuads;
  const u32x4* wg = wp + static_cast<int64_t>(e) * ktiles * kstr + nb * static_cast<int64_t>(Fmt<F>::kTileQuads) + lane;
  const u32x4* wu = wg + static_cast<int64_t>(iblocks) * Fmt<F>::kTileQuads;
  typename Fmt<F>::Tile tg[D][P], tu[D][P];
  _Float16 sg[P], su[P];
  const _Float16* sc = scales + static_cast<int64_t>(e) * 2 * s.I + nb * 16 + r;
  auto load_first = [&]() {
#pragma unroll
    for (int d = 0; d < D; ++d) {
      const int64_t at = (kt0 + d < kt1 ? kt0 + d : kt0) * kstr;
#pragma unroll
      for (int p = 0; p < P; ++p) {
        Fmt<F>::template load<true>(tg[d][p], wg + at + p * Fmt<F>::kTileQuads, lane);
        Fmt<F>::template load<true>(tu[d][p], wu + at + p * Fmt<F>::kTileQuads, lane);
      }
    }
  };
  load_first();
#pragma unroll
  for (int p = 0; p < P; ++p) {
    sg[p] = sc[16 * p];
    su[p] = sc[s.I + 16 * p];
  }
  const uint64_t mask = one ? uint64_t(ch.first >= 0) : __ballot(ch.first >= 0);
  if (!has_work(mask, ch.first, by_pair, slot)) return;
  const int n = __popcll(mask);
  if (ch.first >= 0 && !one) {
    const int c = __popcll(mask & ((uint64_t(1) << lane) - 1));
    col_token[wave][c] = static_cast<short>(lane);
    col_pair[wave][c] = static_cast<short>(ch.first);
    col_w[wave][c] = ch.weight;
  }
  __builtin_amdgcn_wave_barrier();
  for (int c0 = 0; c0 < n; c0 += 16) {
    if (c0 > 0) {
      __syncthreads();
      load_first();
    }
    // Column r; columns behind the expert's last token repeat the first of the 16 and are not stored.
    const int c = c0 + r < n ? c0 + r : c0;
    const _Float16* xr = X + static_cast<int64_t>(t0 + (one ? 0 : col_token[wave][c])) * s.H + 8 * g;
    if (!one) {
#pragma unroll
      for (int j = 0; j < 8; ++j) xf[0][j] = *reinterpret_cast<const half8v*>(xr + kt0 * 256 + 32 * j);
    }
    float4v ag[P], au[P];
#pragma unroll
    for (int p = 0; p < P; ++p) ag[p] = au[p] = float4v{0.f, 0.f, 0.f, 0.f};

    auto tile = [&](int kt, auto CUR) {
      constexpr int cur = decltype(CUR)::value;
      const int next = kt + 1 < kt1 ? kt + 1 : kt;  // behind the end: a stand-in
#pragma unroll
      for (int j = 0; j < 8; ++j) xf[1 - cur][j] = *reinterpret_cast<const half8v*>(xr + next * 256 + 32 * j);
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int p = 0; p < P; ++p) {
        const half2v s2g = scale2_of<F>(sg[p]), s2u = scale2_of<F>(su[p]);
        auto step = [&](auto J) {
          constexpr int j = decltype(J)::value;
          ag[p] = __builtin_amdgcn_mfma_f32_16x16x32_f16(Fmt<F>::template step<j>(tg[cur % D][p], s2g), xf[cur][j], ag[p], 0, 0, 0);
          au[p] = __builtin_amdgcn_mfma_f32_16x16x32_f16(Fmt<F>::template step<j>(tu[cur % D][p], s2u), xf[cur][j], au[p], 0, 0, 0);
        };
        step(std::integral_constant<int, 0>{}); step(std::integral_constant<int, 1>{});
        step(std::integral_constant<int, 2>{}); step(std::integral_constant<int, 3>{});
        step(std::integral_constant<int, 4>{}); step(std::integral_constant<int, 5>{});
        step(std::integral_constant<int, 6>{}); step(std::integral_constant<int, 7>{});
        __builtin_amdgcn_sched_barrier(0);
        if (kt + D < kt1) {
          Fmt<F>::template load<true>(tg[cur % D][p], wg + (kt + D) * kstr + p * Fmt<F>::kTileQuads, lane);
          Fmt<F>::template load<true>(tu[cur % D][p], wu + (kt + D) * kstr + p * Fmt<F>::kTileQuads, lane);
        }
        __builtin_amdgcn_sched_barrier(0);
      }
    };
    int kt = kt0;
    for (; kt + 2 <= kt1; kt += 2) {
      tile(kt, std::integral_constant<int, 0>{});
      tile(kt + 1, std::integral_constant<int, 1>{});
    }
    if (kt < kt1) tile(kt, std::integral_constant<int, 0>{});

#pragma unroll
    for (int p = 0; p < P; ++p) {
      red[wave][2 * p][lane] = ag[p];
      red[wave][2 * p + 1][lane] = au[p];
    }
    __syncthreads();
    // Wave (rb, kslice) sums and stores the row blocks kslice, kslice + ks, ...
    if (c0 + r < n) {
      const int64_t at = (static_cast<int64_t>(t0) * s.k + (one ? ch.first : col_pair[wave][c])) * s.I + nb * 16 + 4 * g;
      const float w = one ? ch.weight : col_w[wave][c];
      for (int p = kslice; p < P; p += ks) {
        float4v vg = red[rb * ks][2 * p][lane], vu = red[rb * ks][2 * p + 1][lane];
        for (int q = 1; q < ks; ++q) {
          vg += red[rb * ks + q][2 * p][lane];
          vu += red[rb * ks + q][2 * p + 1][lane];
        }
        store_gated(hi + at + 16 * p, lo + at + 16 * p, vg, vu, w);
      }
    }
  }
}

// ---------------------------------------------------------------------------
// Down product and the sum over experts, more than a few tokens: a workgroup
// stores its expert's part of the outputs, one fp32 row per pair (the weight of
// the choice is already in h), and moe_sum adds each token's parts in the order
// of its choices and rounds once.  (Letting the last workgroup of a row group
// add instead of a kernel of its own: 64 tokens, 64 experts 2048x1024 181 us
// against 37.)
// ---------------------------------------------------------------------------
template <int F>
__global__ __launch_bounds__(256, 2) void moe_down(const _Float16* __restrict__ hi, const _Float16* __restrict__ lo,
                                                const int* __restrict__ ids_g, const u32x4* __restrict__ wp,
                                                const _Float16* __restrict__ scales, float* __restrict__ part, MoeShape s,
                                                int ks, int by_pair) {
  __shared__ short col_pair[4][kGroup];
  constexpr int D = 2;  // k-tiles of weights in flight per wave
  __shared__ float4v red[4][64];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r = lane & 15, g = lane >> 4;
  const int t0 = blockIdx.z * kGroup;
  const int tokens = s.T - t0 < kGroup ? s.T - t0 : kGroup;
  const int* ids = ids_g + static_cast<int64_t>(t0) * s.k;
  const int slot = blockIdx.y;
  const int rows0 = blockIdx.x * (4 / ks) * 16;  // this workgroup's rows of the output
  float* parts = part + static_cast<int64_t>(t0) * s.k * s.H;

  int e = slot;
  if (by_pair) {
    if (slot >= tokens * s.k) return;
    e = __builtin_amdgcn_readfirstlane(ids[slot]);
    if (e < 0 || e >= s.E) return;
  }
  const Choice ch = choice_of<false>(ids, nullptr, tokens, s.k, e, lane);
  const int rb = wave / ks, kslice = wave - rb * ks;
  const int ktiles = s.I >> 8;
  const int nb = blockIdx.x * (4 / ks) + rb;
  const int64_t kstr = static_cast<int64_t>(s.H >> 4) * Fmt<F>::kTileQuads;
  const u32x4* w = wp + static_cast<int64_t>(e) * ktiles * kstr + nb * static_cast<int64_t>(Fmt<F>::kTileQuads) + lane;
  const int kt0 = kslice * ktiles / ks, kt1 = (kslice + 1) * ktiles / ks;
  typename Fmt<F>::Tile tw[D];
  auto load_first = [&]() {
#pragma unroll
    for (int d = 0; d < D; ++d) Fmt<F>::template load<true>(tw[d], w + (kt0 + d < kt1 ? kt0 + d : kt0) * kstr, lane);
  };
  load_first();
  const _Float16 sw = scales[static_cast<int64_t>(e) * s.H + nb * 16 + r];
  const uint64_t mask = __ballot(ch.first >= 0);
  if (!has_work(mask, ch.first, by_pair, slot)) return;
  const int n = __popcll(mask);
  if (ch.first >= 0) col_pair[wave][__popcll(mask & ((uint64_t(1) << lane) - 1))] = static_cast<short>(ch.first);
  __builtin_amdgcn_wave_barrier();
  for (int c0 = 0; c0 < n; c0 += 16) {
    if (c0 > 0) {
      __syncthreads();
      load_first();
    }
    const int c = c0 + r < n ? c0 + r : c0;
    const int pair = col_pair[wave][c];
    const int64_t at = (static_cast<int64_t>(t0) * s.k + pair) * s.I + 8 * g;
    const _Float16 *hr = hi + at, *lr = lo + at;
    half8v fh[2][8], fl[2][8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      fh[0][j] = *reinterpret_cast<const half8v*>(hr + kt0 * 256 + 32 * j);
      fl[0][j] = *reinterpret_cast<const half8v*>(lr + kt0 * 256 + 32 * j);
    }
    float4v ah = {0.f, 0.f, 0.f, 0.f}, al = {0.f, 0.f, 0.f, 0.f};
    auto tile = [&](int kt, auto CUR) {
      constexpr int cur = decltype(CUR)::value;
      const int next = kt + 1 < kt1 ? kt + 1 : kt;  // behind the end: a stand-in
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        fh[1 - cur][j] = *reinterpret_cast<const half8v*>(hr + next * 256 + 32 * j);
        fl[1 - cur][j] = *reinterpret_cast<const half8v*>(lr + next * 256 + 32 * j);
      }
      __builtin_amdgcn_sched_barrier(0);
      const half2v s2 = scale2_of<F>(sw);
      auto step = [&](auto J) {
        constexpr int j = decltype(J)::value;
        const half8v a = Fmt<F>::template step<j>(tw[cur], s2);
        ah = __builtin_amdgcn_mfma_f32_16x16x32_f16(a, fh[cur][j], ah, 0, 0, 0);
        al = __builtin_amdgcn_mfma_f32_16x16x32_f16(a, fl[cur][j], al, 0, 0, 0);
      };
      step(std::integral_constant<int, 0>{}); step(std::integral_constant<int, 1>{});
      step(std::integral_constant<int, 2>{}); step(std::integral_constant<int, 3>{});
      step(std::integral_constant<int, 4>{}); step(std::integral_constant<int, 5>{});
      step(std::integral_constant<int, 6>{}); step(std::integral_constant<int, 7>{});
      __builtin_amdgcn_sched_barrier(0);
      if (kt + D < kt1) Fmt<F>::template load<true>(tw[cur], w + (kt + D) * kstr, lane);
      __builtin_amdgcn_sched_barrier(0);
    };
    int kt = kt0;
    for (; kt + 2 <= kt1; kt += 2) {
      tile(kt, std::integral_constant<int, 0>{});
      tile(kt + 1, std::integral_constant<int, 1>{});
    }
    if (kt < kt1) tile(kt, std::integral_constant<int, 0>{});
    red[wave][lane] = ah + al * (1.0f / kLoScale);
    __syncthreads();
    if (kslice == 0 && c0 + r < n) {
      float4v v = red[rb * ks][lane];
      for (int q = 1; q < ks; ++q) v += red[rb * ks + q][lane];
      *reinterpret_cast<float4v*>(parts + static_cast<int64_t>(pair) * s.H + rows0 + rb * 16 + 4 * g) = v;
    }
  }
}

// ---------------------------------------------------------------------------
// The same products for many row blocks: the 4 waves of a workgroup take P
// consecutive row blocks each over the whole K and share the token fragments
// through LDS, which leaves the registers to a deeper ring of weights (D
// k-tiles): one wave's fragments of a k-tile are 8 KB (h: 16 KB), more than its
// weights, and come once per workgroup instead of once per wave.
//
// LDS buffer of a k-tile (one of D, filled by direct LDS loads): 16 columns x 32
// units of 16 bytes, unit u of column c at place u ^ c, so that 16 columns'
// reads of one unit cover all banks.
//
// Per k-tile t: wait for its columns, barrier (everybody's are there, and k-tile
// t-1's buffer is free), request the columns of k-tile t+D-1, multiply, request
// the weights of k-tile t+D.  Every k-tile issues the same loads, those behind
// the last one from one address: the waits, the compiler's own among them, are
// then fixed counts with D-1 k-tiles of weights and D-2 of columns in flight
// behind.  (With the requests under conditions the compiler waited for all of
// them in one k-tile of D: 64 tokens, 64 experts 2048x1024 gate/up 42.5 us and
// down 32.4 instead of 40.3 and 26.6, 5.0 and 3.8 TB/s of weights.)
// ---------------------------------------------------------------------------
template <int N>
__device__ __forceinline__ void wait_vm() {
  __builtin_amdgcn_s_waitcnt((N & 15) | ((N >> 4) << 14) | (7 << 4));
}

// A loaded value, waited for here: behind the first direct load the compiler
// waits for every load before it uses one.
__device__ __forceinline__ half2v landed(half2v v) {
  asm volatile("" : "+v"(v));
  return v;
}

// Direct loads of one k-tile of 16 columns by 4 waves: wave w fills units
// [128 w, 128 w + 128); at[i]: where this lane's part of the column of unit
// 128 w + 64 i + lane begins, in bytes behind x (below 2^31: 1024 rows of 2^20).
__device__ __forceinline__ void load_columns(half8v* buf, const _Float16* x, const uint32_t (&at)[2], int wave) {
#pragma unroll
  for (int i = 0; i < 2; ++i) lds_load<16>(reinterpret_cast<const char*>(x) + at[i], buf + 128 * wave + 64 * i);
}

template <int F, int P, int D, int NC>
__global__ __launch_bounds__(256, 2) void moe_gate_up_wide(const _Float16* __restrict__ X, const int* __restrict__ ids_g,
                                                        const float* __restrict__ weights_g,
                                                        const u32x4* __restrict__ wp,
                                                        const _Float16* __restrict__ scales, _Float16* __restrict__ hi,
                                                        _Float16* __restrict__ lo, MoeShape s, int by_pair) {
  static_assert(D == 2 || D == 4, "column buffers");
  __shared__ short col_token[4][kGroup], col_pair[4][kGroup];
  __shared__ float col_w[4][kGroup];
  // One array each: the compiler orders direct loads and reads of one array.
  __shared__ half8v buf0[512 * NC], buf1[512 * NC], buf2[D > 2 ? 512 * NC : 1], buf3[D > 2 ? 512 * NC : 1];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r = lane & 15, g = lane >> 4;
  const int t0 = blockIdx.z * kGroup;
  const int tokens = s.T - t0 < kGroup ? s.T - t0 : kGroup;
  const int* ids = ids_g + static_cast<int64_t>(t0) * s.k;
  const int slot = blockIdx.y;
  int e = slot;
  if (by_pair) {
    if (slot >= tokens * s.k) return;
    e = __builtin_amdgcn_readfirstlane(ids[slot]);
    if (e < 0 || e >= s.E) return;
  }
  const Choice ch = choice_of<true>(ids, weights_g + static_cast<int64_t>(t0) * s.k, tokens, s.k, e, lane);
  const int iblocks = s.I >> 4, ktiles = s.H >> 8;
  const int nb = (blockIdx.x * 4 + wave) * P;
  const int64_t kstr = 2 * static_cast<int64_t>(iblocks) * Fmt<F>::kTileQuads;
  int64_t wg = static_cast<int64_t>(e) * ktiles * kstr + nb * static_cast<int64_t>(Fmt<F>::kTileQuads);
  int64_t wu = wg + static_cast<int64_t>(iblocks) * Fmt<F>::kTileQuads;
  _Float16 sg[P], su[P];
  const _Float16* sc = scales + static_cast<int64_t>(e) * 2 * s.I + nb * 16 + r;
#pragma unroll
  for (int p = 0; p < P; ++p) {
    sg[p] = sc[16 * p];
    su[p] = sc[s.I + 16 * p];
  }
  typename Fmt<F>::Tile tg[D][P], tu[D][P];
  constexpr int kW = 2 * P * Fmt<F>::kTileLoads;  // weight loads per k-tile
  auto load_w = [&](int slot_, int kt) {
    const bool in = kt < ktiles;
    const u32x4* pg = wp + (in ? wg + kt * kstr : 0);
    const u32x4* pu = wp + (in ? wu + kt * kstr : 0);
    const unsigned l = in ? lane : 0;
#pragma unroll
    for (int p = 0; p < P; ++p) {
      Fmt<F>::template load<true>(tg[slot_][p], pg + p * Fmt<F>::kTileQuads + l, l);
      Fmt<F>::template load<true>(tu[slot_][p], pu + p * Fmt<F>::kTileQuads + l, l);
    }
  };
  load_w(0, 0);
  const uint64_t mask = __ballot(ch.first >= 0);
  if (!has_work(mask, ch.first, by_pair, slot)) return;
  const int n = __popcll(mask);
  if (ch.first >= 0) {
    const int c = __popcll(mask & ((uint64_t(1) << lane) - 1));
    col_token[wave][c] = static_cast<short>(lane);
    col_pair[wave][c] = static_cast<short>(ch.first);
    col_w[wave][c] = ch.weight;
  }
  __builtin_amdgcn_wave_barrier();
  half2v s2g[P], s2u[P];
#pragma unroll
  for (int p = 0; p < P; ++p) {
    s2g[p] = landed(scale2_of<F>(sg[p]));
    s2u[p] = landed(scale2_of<F>(su[p]));
  }
  // One pass: C groups of 16 columns, from column c0 on.
  auto pass = [&](int c0, auto C) {
    constexpr int nc = decltype(C)::value;
    // Every pass loads its weights itself, at its places in the order.
    asm volatile("" : "+s"(wg), "+s"(wu));
    uint32_t at[nc][2];
    const _Float16* const Xg = X + static_cast<int64_t>(t0) * s.H;
#pragma unroll
    for (int q = 0; q < nc; ++q)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int col = 4 * wave + 2 * i + (lane >> 5), c = c0 + 16 * q + col;
        at[q][i] = 2 * (col_token[wave][c < n ? c : c0] * static_cast<uint32_t>(s.H) + 8 * ((lane & 31) ^ col));
      }
    auto columns = [&](half8v* buf, int kt) {
      const _Float16* x = Xg + (kt < ktiles ? kt * 256 : 0);
#pragma unroll
      for (int q = 0; q < nc; ++q) load_columns(buf + 512 * q, x, at[q], wave);
    };
    // In the order of the loop, which its counts rely on.
    columns(buf0, 0);
    __builtin_amdgcn_sched_barrier(0);
    load_w(1, 1);
    if constexpr (D > 2) {
      __builtin_amdgcn_sched_barrier(0);
      columns(buf1, 1);
      __builtin_amdgcn_sched_barrier(0);
      load_w(2, 2);
      __builtin_amdgcn_sched_barrier(0);
      columns(buf2, 2);
      __builtin_amdgcn_sched_barrier(0);
      load_w(3, 3);
    }
    __builtin_amdgcn_sched_barrier(0);
    float4v ag[nc][P], au[nc][P];
#pragma unroll
    for (int q = 0; q < nc; ++q)
#pragma unroll
      for (int p = 0; p < P; ++p) ag[q][p] = au[q][p] = float4v{0.f, 0.f, 0.f, 0.f};
    auto tile = [&](int kt, auto U, auto W) {
      constexpr int u = decltype(U)::value;
      const half8v* cur = u == 0 ? buf0 : u == 1 ? buf1 : u == 2 ? buf2 : buf3;
      half8v* next = (u + D - 1) % D == 0 ? buf0 : (u + D - 1) % D == 1 ? buf1 : (u + D - 1) % D == 2 ? buf2 : buf3;
      __builtin_amdgcn_sched_barrier(0);
      wait_vm<decltype(W)::value * kW + (D - 2) * 2 * nc>();
      barrier_no_fence();
      columns(next, kt + D - 1);
      __builtin_amdgcn_sched_barrier(0);
      auto step = [&](auto J) {
        constexpr int j = decltype(J)::value;
        half8v x[nc];
#pragma unroll
        for (int q = 0; q < nc; ++q) x[q] = cur[512 * q + r * 32 + ((4 * j + g) ^ r)];
#pragma unroll
        for (int p = 0; p < P; ++p) {
          const half8v a = Fmt<F>::template step<j>(tg[u][p], s2g[p]), b = Fmt<F>::template step<j>(tu[u][p], s2u[p]);
#pragma unroll
          for (int q = 0; q < nc; ++q) {
            ag[q][p] = __builtin_amdgcn_mfma_f32_16x16x32_f16(a, x[q], ag[q][p], 0, 0, 0);
            au[q][p] = __builtin_amdgcn_mfma_f32_16x16x32_f16(b, x[q], au[q][p], 0, 0, 0);
          }
        }
      };
      step(std::integral_constant<int, 0>{}); step(std::integral_constant<int, 1>{});
      step(std::integral_constant<int, 2>{}); step(std::integral_constant<int, 3>{});
      step(std::integral_constant<int, 4>{}); step(std::integral_constant<int, 5>{});
      step(std::integral_constant<int, 6>{}); step(std::integral_constant<int, 7>{});
      __builtin_amdgcn_sched_barrier(0);
    };
    auto turn = [&](int kt, auto U) {
      tile(kt, U, std::integral_constant<int, D - 1>{});
      load_w(decltype(U)::value, kt + D);
    };
    int kt = 0;
    for (; kt + D <= ktiles; kt += D) {
      turn(kt, std::integral_constant<int, 0>{});
      turn(kt + 1, std::integral_constant<int, 1>{});
      if constexpr (D > 2) {
        turn(kt + 2, std::integral_constant<int, 2>{});
        turn(kt + 3, std::integral_constant<int, 3>{});
      }
    }
    // The rest: no weights are requested any more, or, with fewer than D k-tiles
    // in all, not all of the ring's were.
    constexpr std::integral_constant<int, 0> kNone{};
    if (kt < ktiles) tile(kt, std::integral_constant<int, 0>{}, kNone);
    if constexpr (D > 2) {
      if (kt + 1 < ktiles) tile(kt + 1, std::integral_constant<int, 1>{}, kNone);
      if (kt + 2 < ktiles) tile(kt + 2, std::integral_constant<int, 2>{}, kNone);
    }
    wait_vm<0>();  // no load into the buffers outlives its pass
#pragma unroll
    for (int q = 0; q < nc; ++q) {
      const int c = c0 + 16 * q + r;
      if (c < n) {
        const int64_t at = (static_cast<int64_t>(t0) * s.k + col_pair[wave][c]) * s.I + nb * 16 + 4 * g;
#pragma unroll
        for (int p = 0; p < P; ++p) store_gated(hi + at + 16 * p, lo + at + 16 * p, ag[q][p], au[q][p], col_w[wave][c]);
      }
    }
  };
  if constexpr (NC == 2) {
    int c0 = 0;
    for (; n - c0 > 16; c0 += 32) {
      pass(c0, std::integral_constant<int, 2>{});
      __syncthreads();  // the buffers are free again
      if (n - c0 > 32) load_w(0, 0);
    }
    if (c0 < n) pass(c0, std::integral_constant<int, 1>{});
  } else {
    pass(0, std::integral_constant<int, 1>{});  // at most 16 tokens in the group
  }
}

template <int F, int P, int D, int NC>
__global__ __launch_bounds__(256, 2) void moe_down_wide(const _Float16* __restrict__ hi, const _Float16* __restrict__ lo,
                                                     const int* __restrict__ ids_g, const u32x4* __restrict__ wp,
                                                     const _Float16* __restrict__ scales, float* __restrict__ part,
                                                     MoeShape s, int by_pair) {
  static_assert(D == 2 || D == 4, "column buffers");
  __shared__ short col_pair[4][kGroup];
  // The columns' upper halves, and the lower ones behind them.
  __shared__ half8v buf0[1024 * NC], buf1[1024 * NC], buf2[D > 2 ? 1024 * NC : 1], buf3[D > 2 ? 1024 * NC : 1];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r = lane & 15, g = lane >> 4;
  const int t0 = blockIdx.z * kGroup;
  const int tokens = s.T - t0 < kGroup ? s.T - t0 : kGroup;
  const int* ids = ids_g + static_cast<int64_t>(t0) * s.k;
  const int slot = blockIdx.y;
  int e = slot;
  if (by_pair) {
    if (slot >= tokens * s.k) return;
    e = __builtin_amdgcn_readfirstlane(ids[slot]);
    if (e < 0 || e >= s.E) return;
  }
  const Choice ch = choice_of<false>(ids, nullptr, tokens, s.k, e, lane);
  const int ktiles = s.I >> 8;
  const int nb = (blockIdx.x * 4 + wave) * P;
  const int64_t kstr = static_cast<int64_t>(s.H >> 4) * Fmt<F>::kTileQuads;
  int64_t w = static_cast<int64_t>(e) * ktiles * kstr + nb * static_cast<int64_t>(Fmt<F>::kTileQuads);
  _Float16 sw[P];
  const _Float16* sc = scales + static_cast<int64_t>(e) * s.H + nb * 16 + r;
#pragma unroll
  for (int p = 0; p < P; ++p) sw[p] = sc[16 * p];
  typename Fmt<F>::Tile tw[D][P];
  constexpr int kW = P * Fmt<F>::kTileLoads;
  auto load_w = [&](int slot_, int kt) {
    const bool in = kt < ktiles;
    const u32x4* pw = wp + (in ? w + kt * kstr : 0);
    const unsigned l = in ? lane : 0;
#pragma unroll
    for (int p = 0; p < P; ++p) Fmt<F>::template load<true>(tw[slot_][p], pw + p * Fmt<F>::kTileQuads + l, l);
  };
  load_w(0, 0);
  const uint64_t mask = __ballot(ch.first >= 0);
  if (!has_work(mask, ch.first, by_pair, slot)) return;
  const int n = __popcll(mask);
  if (ch.first >= 0) col_pair[wave][__popcll(mask & ((uint64_t(1) << lane) - 1))] = static_cast<short>(ch.first);
  __builtin_amdgcn_wave_barrier();
  half2v s2[P];
#pragma unroll
  for (int p = 0; p < P; ++p) s2[p] = landed(scale2_of<F>(sw[p]));
  auto pass = [&](int c0, auto C) {
    constexpr int nc = decltype(C)::value;
    asm volatile("" : "+s"(w));
    uint32_t at[nc][2];
    const int64_t group = static_cast<int64_t>(t0) * s.k * s.I;
#pragma unroll
    for (int q = 0; q < nc; ++q)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int col = 4 * wave + 2 * i + (lane >> 5), c = c0 + 16 * q + col;
        at[q][i] = 2 * (col_pair[wave][c < n ? c : c0] * static_cast<uint32_t>(s.I) + 8 * ((lane & 31) ^ col));
      }
    auto columns = [&](half8v* buf, int kt) {
      const int64_t from = group + (kt < ktiles ? kt * 256 : 0);
#pragma unroll
      for (int q = 0; q < nc; ++q) {
        load_columns(buf + 512 * q, hi + from, at[q], wave);
        load_columns(buf + 512 * (NC + q), lo + from, at[q], wave);
      }
    };
    // In the order of the loop, which its counts rely on.
    columns(buf0, 0);
    __builtin_amdgcn_sched_barrier(0);
    load_w(1, 1);
    if constexpr (D > 2) {
      __builtin_amdgcn_sched_barrier(0);
      columns(buf1, 1);
      __builtin_amdgcn_sched_barrier(0);
      load_w(2, 2);
      __builtin_amdgcn_sched_barrier(0);
      columns(buf2, 2);
      __builtin_amdgcn_sched_barrier(0);
      load_w(3, 3);
    }
    __builtin_amdgcn_sched_barrier(0);
    float4v ah[nc][P], al[nc][P];
#pragma unroll
    for (int q = 0; q < nc; ++q)
#pragma unroll
      for (int p = 0; p < P; ++p) ah[q][p] = al[q][p] = float4v{0.f, 0.f, 0.f, 0.f};
    auto tile = [&](int kt, auto U, auto W) {
      constexpr int u = decltype(U)::value;
      const half8v* cur = u == 0 ? buf0 : u == 1 ? buf1 : u == 2 ? buf2 : buf3;
      half8v* next = (u + D - 1) % D == 0 ? buf0 : (u + D - 1) % D == 1 ? buf1 : (u + D - 1) % D == 2 ? buf2 : buf3;
      __builtin_amdgcn_sched_barrier(0);
      wait_vm<decltype(W)::value * kW + (D - 2) * 4 * nc>();
      barrier_no_fence();
      columns(next, kt + D - 1);
      __builtin_amdgcn_sched_barrier(0);
      auto step = [&](auto J) {
        constexpr int j = decltype(J)::value;
        const int at = r * 32 + ((4 * j + g) ^ r);
        half8v xh[nc], xl[nc];
#pragma unroll
        for (int q = 0; q < nc; ++q) {
          xh[q] = cur[512 * q + at];
          xl[q] = cur[512 * (NC + q) + at];
        }
#pragma unroll
        for (int p = 0; p < P; ++p) {
          const half8v a = Fmt<F>::template step<j>(tw[u][p], s2[p]);
#pragma unroll
          for (int q = 0; q < nc; ++q) {
            ah[q][p] = __builtin_amdgcn_mfma_f32_16x16x32_f16(a, xh[q], ah[q][p], 0, 0, 0);
            al[q][p] = __builtin_amdgcn_mfma_f32_16x16x32_f16(a, xl[q], al[q][p], 0, 0, 0);
          }
        }
      };
      step(std::integral_constant<int, 0>{}); step(std::integral_constant<int, 1>{});
      step(std::integral_constant<int, 2>{}); step(std::integral_constant<int, 3>{});
      step(std::integral_constant<int, 4>{}); step(std::integral_constant<int, 5>{});
      step(std::integral_constant<int, 6>{}); step(std::integral_constant<int, 7>{});
      __builtin_amdgcn_sched_barrier(0);
    };
    auto turn = [&](int kt, auto U) {
      tile(kt, U, std::integral_constant<int, D - 1>{});
      load_w(decltype(U)::value, kt + D);
    };
    int kt = 0;
    for (; kt + D <= ktiles; kt += D) {
      turn(kt, std::integral_constant<int, 0>{});
      turn(kt + 1, std::integral_constant<int, 1>{});
      if constexpr (D > 2) {
        turn(kt + 2, std::integral_constant<int, 2>{});
        turn(kt + 3, std::integral_constant<int, 3>{});
      }
    }
    // The rest: no weights are requested any more, or, with fewer than D k-tiles
    // in all, not all of the ring's were.
    constexpr std::integral_constant<int, 0> kNone{};
    if (kt < ktiles) tile(kt, std::integral_constant<int, 0>{}, kNone);
    if constexpr (D > 2) {
      if (kt + 1 < ktiles) tile(kt + 1, std::integral_constant<int, 1>{}, kNone);
      if (kt + 2 < ktiles) tile(kt + 2, std::integral_constant<int, 2>{}, kNone);
    }
    wait_vm<0>();  // no load into the buffers outlives its pass
#pragma unroll
    for (int q = 0; q < nc; ++q) {
      const int c = c0 + 16 * q + r;
      if (c < n) {
        float* dst = part + (static_cast<int64_t>(t0) * s.k + col_pair[wave][c]) * s.H + nb * 16 + 4 * g;
#pragma unroll
        for (int p = 0; p < P; ++p) *reinterpret_cast<float4v*>(dst + 16 * p) = ah[q][p] + al[q][p] * (1.0f / kLoScale);
      }
    }
  };
  if constexpr (NC == 2) {
    int c0 = 0;
    for (; n - c0 > 16; c0 += 32) {
      pass(c0, std::integral_constant<int, 2>{});
      __syncthreads();
      if (n - c0 > 32) load_w(0, 0);
    }
    if (c0 < n) pass(c0, std::integral_constant<int, 1>{});
  } else {
    pass(0, std::integral_constant<int, 1>{});  // at most 16 tokens in the group
  }
}

// 4 rows of a token per thread (64 tokens x 2048, 8 parts 4.5 us: launch, one load).
__global__ __launch_bounds__(256) void moe_sum(const float* __restrict__ part, const int* __restrict__ ids,
                                               _Float16* __restrict__ Y, MoeShape s) {
  const int64_t t = blockIdx.y;
  const int row = 4 * (blockIdx.x * 256 + threadIdx.x);
  if (row >= s.H) return;
  ids += t * s.k;
  const float* p = part + t * s.k * s.H + row;
  float4v v[kMaxK];
  int id[kMaxK];
#pragma unroll
  for (int j = 0; j < kMaxK; ++j) {  // requested with the ids, unwritten parts too: those are not used
    id[j] = j < s.k ? ids[j] : -1;
    v[j] = float4v{0.f, 0.f, 0.f, 0.f};
    if (j < s.k) v[j] = *reinterpret_cast<const float4v*>(p + static_cast<int64_t>(j) * s.H);
  }
#pragma unroll
  for (int j = 0; j < kMaxK; ++j) {
    bool use = id[j] >= 0 && id[j] < s.E;
#pragma unroll
    for (int o = 0; o < j; ++o) use = use && id[o] != id[j];  // the same expert again: counted with the first
    if (!use) v[j] = float4v{0.f, 0.f, 0.f, 0.f};
  }
  float4v sum = v[0];
#pragma unroll
  for (int j = 1; j < kMaxK; ++j)
    if (j < s.k) sum += v[j];
  half4v o;
#pragma unroll
  for (int i = 0; i < 4; ++i) o[i] = static_cast<_Float16>(sum[i] * (1.0f / kHScale));
  *reinterpret_cast<half4v*>(Y + t * s.H + row) = o;
}

// ---------------------------------------------------------------------------
// Down product and the sum over experts, few tokens (at most kFewPairs pairs and
// kFewTiles tiles of each row block):
// a workgroup of 16 waves owns 16 rows of the output.  The columns of the MFMAs
// are the tokens themselves, with zeros where a token did not choose the tile's
// expert, so an output is one long product over (expert, k) and nothing but the
// waves' sums has to be added: no parts in memory, no second kernel (one token,
// 64 experts 2048x1024 9.0 us, 0.7 TB/s: a chain of ids, addresses, loads).  The waves
// share the list of (expert, k-tile) of the experts that any token chose, in
// the order of first choice, in equal contiguous parts, and add in wave order.
// ---------------------------------------------------------------------------
template <int F>
__global__ __launch_bounds__(1024) void moe_down_few(const _Float16* __restrict__ hi, const _Float16* __restrict__ lo,
                                                     const int* __restrict__ ids, const u32x4* __restrict__ wp,
                                                     const _Float16* __restrict__ scales, _Float16* __restrict__ Y,
                                                     MoeShape s) {
  constexpr int kWaves = 16;
  __shared__ short s_ids[kFewPairs];
  __shared__ short s_active[kFewPairs];
  __shared__ float4v red[kWaves][64];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r = lane & 15, g = lane >> 4;
  const int pairs = s.T * s.k, ktiles = s.I >> 8, nb = blockIdx.x;
  const int64_t kstr = static_cast<int64_t>(s.H >> 4) * Fmt<F>::kTileQuads;
  const u32x4* w0 = wp + nb * static_cast<int64_t>(Fmt<F>::kTileQuads) + lane;
  float4v ah = {0.f, 0.f, 0.f, 0.f}, al = {0.f, 0.f, 0.f, 0.f};
  struct Weights {
    typename Fmt<F>::Tile t;
    _Float16 scale;
  };
  struct Values {
    half8v h[8], l[8];
  };
  // A tile's product is added to the tokens that chose its expert only: an
  // infinite or NaN weight times another token's zeros would be NaN.
  auto mul = [&](const Weights& w, const Values& v, bool mine) {
    const half2v s2 = scale2_of<F>(w.scale);
    float4v th = {0.f, 0.f, 0.f, 0.f}, tl = {0.f, 0.f, 0.f, 0.f};
    auto step = [&](auto J) {
      constexpr int j = decltype(J)::value;
      const half8v a = Fmt<F>::template step<j>(w.t, s2);
      th = __builtin_amdgcn_mfma_f32_16x16x32_f16(a, v.h[j], th, 0, 0, 0);
      tl = __builtin_amdgcn_mfma_f32_16x16x32_f16(a, v.l[j], tl, 0, 0, 0);
    };
    step(std::integral_constant<int, 0>{}); step(std::integral_constant<int, 1>{});
    step(std::integral_constant<int, 2>{}); step(std::integral_constant<int, 3>{});
    step(std::integral_constant<int, 4>{}); step(std::integral_constant<int, 5>{});
    step(std::integral_constant<int, 6>{}); step(std::integral_constant<int, 7>{});
    if (mine) {
      ah += th;
      al += tl;
    }
  };
  int total = s.k * ktiles;
  int f0 = wave * total / kWaves, f1 = (wave + 1) * total / kWaves;
  // One token whose choices are all served and all different, as moe_layer's
  // are: the list is the choices themselves, and a wave needs nothing but the
  // ids of its own tiles to request everything.
  int id = lane < pairs ? ids[lane] : -1;
  if (id >= s.E) id = -1;
  bool first = id >= 0;  // a pair whose expert no earlier pair chose
  for (int o = 0; o + 1 < pairs; ++o) {
    const int other = __builtin_amdgcn_readlane(id, o);
    first = first && (o >= lane || other != id);
  }
  const uint64_t mask = __ballot(first);
  if (s.T == 1 && __popcll(mask) == s.k) {
    auto load_w = [&](Weights& w, int f) {
      const int j = f / ktiles, e = __builtin_amdgcn_readlane(id, j);
      Fmt<F>::template load<true>(w.t, w0 + (static_cast<int64_t>(e) * ktiles + (f - j * ktiles)) * kstr, lane);
      w.scale = scales[static_cast<int64_t>(e) * s.H + nb * 16 + r];
    };
    auto load_h = [&](Values& v, int f) {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        v.h[j] = *reinterpret_cast<const half8v*>(hi + static_cast<int64_t>(f) * 256 + 8 * g + 32 * j);
        v.l[j] = *reinterpret_cast<const half8v*>(lo + static_cast<int64_t>(f) * 256 + 8 * g + 32 * j);
      }
    };
    if (f0 < f1) {
      Weights wa, wb;
      Values v;
      load_h(v, f0);
      load_w(wa, f0);
      load_w(wb, f1 - 1);
      __builtin_amdgcn_sched_barrier(0);
      mul(wa, v, true);
      if (f0 + 1 < f1) {
        load_h(v, f0 + 1);
        mul(wb, v, true);
      }
    }
  } else {
    // The first pairs stand for their experts.
    if (wave == 0) s_ids[lane] = static_cast<short>(id);
    const int na = __popcll(mask);
    if (wave == 0 && first) s_active[__popcll(mask & ((uint64_t(1) << lane) - 1))] = static_cast<short>(id);
    __syncthreads();
    total = na * ktiles;
    f0 = wave * total / kWaves, f1 = (wave + 1) * total / kWaves;
    auto expert_of = [&](int f) { return __builtin_amdgcn_readfirstlane(s_active[f / ktiles]); };
    auto load_w = [&](Weights& w, int f) {
      const int e = expert_of(f), kt = f % ktiles;
      Fmt<F>::template load<true>(w.t, w0 + (static_cast<int64_t>(e) * ktiles + kt) * kstr, lane);
      w.scale = scales[static_cast<int64_t>(e) * s.H + nb * 16 + r];
    };
    auto load_h = [&](Values& v, int f) {
      const int e = expert_of(f), kt = f % ktiles;
      // Column r is token r (behind the last: the last, not stored); its pair of this expert, if any.
      const int t = r < s.T ? r : s.T - 1;
      int pair = -1;
      for (int j = s.k - 1; j >= 0; --j)
        if (s_ids[t * s.k + j] == e) pair = t * s.k + j;
      const bool mine = pair >= 0;
      const int64_t at = static_cast<int64_t>(mine ? pair : 0) * s.I + kt * 256 + 8 * g;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        v.h[j] = v.l[j] = half8v{};
        if (mine) {
          v.h[j] = *reinterpret_cast<const half8v*>(hi + at + 32 * j);
          v.l[j] = *reinterpret_cast<const half8v*>(lo + at + 32 * j);
        }
      }
      return mine;
    };
    // At most two tiles per wave: the second's weights are requested before the first is multiplied.
    if (f0 < f1) {
      Weights wa, wb;
      Values v;
      load_w(wa, f0);
      bool mine = load_h(v, f0);
      load_w(wb, f1 - 1);
      __builtin_amdgcn_sched_barrier(0);
      mul(wa, v, mine);
      if (f0 + 1 < f1) {
        mine = load_h(v, f0 + 1);
        mul(wb, v, mine);
      }
    }
  }
  red[wave][lane] = ah + al * (1.0f / kLoScale);
  __syncthreads();
  if (wave == 0 && r < s.T) {
    const float4v sum = reduce_waves<kWaves>(red, lane);
    half4v o;
#pragma unroll
    for (int i = 0; i < 4; ++i) o[i] = static_cast<_Float16>(sum[i] * (1.0f / kHScale));
    *reinterpret_cast<half4v*>(Y + static_cast<int64_t>(r) * s.H + nb * 16 + 4 * g) = o;
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
  size_t logits, hi, lo, part, bytes;
};
Workspace workspace_of(int64_t T, int64_t E, int64_t k, int64_t H, int64_t I) {
  Workspace w;
  const size_t pairs = static_cast<size_t>(T) * k;
  w.logits = 0;
  w.hi = round256(static_cast<size_t>(T) * E * sizeof(double));
  w.lo = w.hi + round256(pairs * I * 2);
  w.part = w.lo + round256(pairs * I * 2);
  w.bytes = w.part + round256(pairs * H * sizeof(float));
  return w;
}

struct MoeCall {
  const _Float16* X;
  int* ids;        // written only where the layer makes the choice
  float* weights;
  const u32x4 *gate_up, *down;
  const _Float16 *gate_up_scales, *down_scales;
  _Float16 *Y, *hi, *lo;
  float* part;
  MoeShape s;
  hipStream_t stream;
};

int moe_launch(const void* kern, dim3 grid, dim3 block, void** args, hipStream_t stream) {
  return hipLaunchKernel(kern, grid, block, args, 0, stream) == hipSuccess ? FP6_OK : FP6_E_HIP;
}

// Row blocks per CU, over all slots, from which on the forms with shared
// fragments are used (4 row blocks per workgroup at least: one workgroup).  The
// products with 4 per CU and the other forms: 64 tokens, 8 experts 4096x2048
// 49 against 58 us; 16 tokens 43 and 42; 64 experts 2048x1024 (16 per CU) 75 and
// 86.  With 2 per CU: 8 tokens, 4 experts 4096x2048 31 and 28, 64 tokens 60 and 62.
constexpr int64_t kWideRows = 4;
// Below this the choice is made in the first product, though its form with
// shared fragments, which expects it made, would be faster by itself (2 tokens,
// 64 experts 2048x1024, 4 per CU: 31.5 against 32.7 us).
constexpr int64_t kFusedRows = 8;

// Waves that split K in the forms with fewer row blocks.
int k_slices(int64_t ktiles) { return ktiles >= 4 ? 4 : ktiles >= 2 ? 2 : 1; }

// route: where the choice comes from; all but kGiven make it in the first product.
template <int F>
int launch_experts(const MoeCall& c, Route route, const _Float16* router, const double* logits, int renorm) {
  MoeShape s = c.s;
  const int group_tokens = s.T < kGroup ? s.T : kGroup;
  const unsigned groups = static_cast<unsigned>(fpx_ceil_div(s.T, kGroup));
  int by_pair = group_tokens * s.k < s.E;
  int slots = by_pair ? group_tokens * s.k : s.E;
  const unsigned grid_y = static_cast<unsigned>(slots);
  const bool two = group_tokens > 16;  // two groups of 16 columns at once
  const int cus = fpx::current_cus();
  const _Float16* X = c.X;
  int* ids = c.ids;
  float* weights = c.weights;
  const u32x4* w = c.gate_up;
  const _Float16* sc = c.gate_up_scales;
  _Float16 *hi = c.hi, *lo = c.lo, *Y = c.Y;
  float* part = c.part;
  const int64_t wide_gu = static_cast<int64_t>(slots) * (s.I / 16), wide_dn = static_cast<int64_t>(slots) * (s.H / 16);
  if (route == kGiven && wide_gu >= kWideRows * cus) {
    const int p = wide_gu >= 16 * cus ? 2 : 1;
    void* args[] = {&X, &ids, &weights, &w, &sc, &hi, &lo, &s, &by_pair};
    const dim3 grid(static_cast<unsigned>(s.I / 16 / (4 * p)), grid_y, groups);
    const void* kern = p == 2 ? (two ? reinterpret_cast<const void*>(&moe_gate_up_wide<F, 2, 2, 2>)
                                     : reinterpret_cast<const void*>(&moe_gate_up_wide<F, 2, 2, 1>))
                              : (two ? reinterpret_cast<const void*>(&moe_gate_up_wide<F, 1, 4, 2>)
                                     : reinterpret_cast<const void*>(&moe_gate_up_wide<F, 1, 4, 1>));
    const int st = moe_launch(kern, grid, dim3(256), args, c.stream);
    if (st != FP6_OK) return st;
  } else {
    // Two row blocks per wave where that still gives every CU two workgroups,
    // counting every slot as used.
    int ks = k_slices(s.H / 256);
    const int p = route != kGiven && wide_gu >= 4 * cus ? 2 : 1;
    void* args[] = {&X, &router, &logits, &ids, &weights, &w, &sc, &hi, &lo, &s, &ks, &by_pair, &renorm};
    const dim3 grid(static_cast<unsigned>(s.I / 16 / (4 / ks * p)), grid_y, groups);
    const void* kern = nullptr;
    if (route == kFromRouter)
      kern = p == 2 ? reinterpret_cast<const void*>(&moe_gate_up<F, 2, 1, kFromRouter>)
                    : reinterpret_cast<const void*>(&moe_gate_up<F, 1, 2, kFromRouter>);
    else if (route == kFromLogits)
      kern = p == 2 ? reinterpret_cast<const void*>(&moe_gate_up<F, 2, 1, kFromLogits>)
                    : reinterpret_cast<const void*>(&moe_gate_up<F, 1, 2, kFromLogits>);
    else
      kern = reinterpret_cast<const void*>(&moe_gate_up<F, 1, 2, kGiven>);
    const int st = moe_launch(kern, grid, dim3(256), args, c.stream);
    if (st != FP6_OK) return st;
  }
  w = c.down;
  sc = c.down_scales;
  // The waves of moe_down_few go through their tiles one after another: up to
  // two each (16 waves), and one lane per pair.
  if (s.T <= 16 && s.T * s.k <= kFewPairs && s.T * s.k * (s.I / 256) <= kFewTiles) {
    void* args[] = {&hi, &lo, &ids, &w, &sc, &Y, &s};
    return moe_launch(reinterpret_cast<const void*>(&moe_down_few<F>), dim3(static_cast<unsigned>(s.H / 16)), dim3(1024),
                      args, c.stream);
  }
  int st = FP6_OK;
  if (wide_dn >= kWideRows * cus) {
    // Four row blocks per wave with two column groups: no faster (75.8 us against
    // 75.0 .. 76.5 for 64 tokens, 64 experts 2048x1024).
    const int p = wide_dn < 16 * cus ? 1 : (!two && wide_dn >= 32 * cus ? 4 : 2);
    void* args[] = {&hi, &lo, &ids, &w, &sc, &part, &s, &by_pair};
    const dim3 grid(static_cast<unsigned>(s.H / 16 / (4 * p)), grid_y, groups);
    const void* kern = p == 4   ? reinterpret_cast<const void*>(&moe_down_wide<F, 4, 2, 1>)
                       : p == 1 ? (two ? reinterpret_cast<const void*>(&moe_down_wide<F, 1, 2, 2>)
                                       : reinterpret_cast<const void*>(&moe_down_wide<F, 1, 4, 1>))
                                : (two ? reinterpret_cast<const void*>(&moe_down_wide<F, 2, 2, 2>)
                                     : reinterpret_cast<const void*>(&moe_down_wide<F, 2, 4, 1>));
    st = moe_launch(kern, grid, dim3(256), args, c.stream);
  } else {
    int ks = k_slices(s.I / 256);
    void* args[] = {&hi, &lo, &ids, &w, &sc, &part, &s, &ks, &by_pair};
    const dim3 grid(static_cast<unsigned>(s.H / 16 / (4 / ks)), grid_y, groups);
    st = moe_launch(reinterpret_cast<const void*>(&moe_down<F>), grid, dim3(256), args, c.stream);
  }
  if (st != FP6_OK) return st;
  void* sum_args[] = {&part, &ids, &Y, &s};
  // The grid's second dimension takes T <= 65536 tokens in two parts.
  for (int t = 0; t < s.T; t += 32768) {
    const float* pt = part + static_cast<int64_t>(t) * s.k * s.H;
    const int* it = ids + static_cast<int64_t>(t) * s.k;
    _Float16* yt = Y + static_cast<int64_t>(t) * s.H;
    sum_args[0] = &pt;
    sum_args[1] = &it;
    sum_args[2] = &yt;
    const int rest = s.T - t < 32768 ? s.T - t : 32768;
    const int r = moe_launch(reinterpret_cast<const void*>(&moe_sum),
                             dim3(static_cast<unsigned>(fpx_ceil_div(s.H, 1024)), static_cast<unsigned>(rest)), dim3(256),
                             sum_args, c.stream);
    if (r != FP6_OK) return r;
  }
  return FP6_OK;
}

int launch_experts_format(int format, const MoeCall& c, Route route, const _Float16* router, const double* logits,
                          int renorm) {
  switch (format) {
    case FPX_E3M2: return launch_experts<kE3M2>(c, route, router, logits, renorm);
    case FPX_E2M3: return launch_experts<kE2M3>(c, route, router, logits, renorm);
    case FPX_E2M2: return launch_experts<kE2M2>(c, route, router, logits, renorm);
    case FPX_E2M1: return launch_experts<kE2M1>(c, route, router, logits, renorm);
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
  const Workspace w = workspace_of(T, E, k, H, I);
  char* ws = static_cast<char*>(workspace);
  MoeCall c;
  c.X = static_cast<const _Float16*>(X);
  c.ids = const_cast<int*>(static_cast<const int*>(ids));
  c.weights = const_cast<float*>(static_cast<const float*>(weights));
  c.gate_up = static_cast<const u32x4*>(gate_up);
  c.gate_up_scales = static_cast<const _Float16*>(gate_up_scales);
  c.down = static_cast<const u32x4*>(down);
  c.down_scales = static_cast<const _Float16*>(down_scales);
  c.Y = static_cast<_Float16*>(Y);
  c.hi = reinterpret_cast<_Float16*>(ws + w.hi);
  c.lo = reinterpret_cast<_Float16*>(ws + w.lo);
  c.part = reinterpret_cast<float*>(ws + w.part);
  c.s = MoeShape{static_cast<int>(T), static_cast<int>(E), static_cast<int>(k), static_cast<int>(H), static_cast<int>(I)};
  c.stream = static_cast<hipStream_t>(stream);
  return c;
}

}  // namespace

extern "C" {

size_t fpx_moe_workspace_bytes(int64_t T, int64_t E, int64_t top_k, int64_t H, int64_t I) {
  if (!moe_sizes_ok(T, E, top_k, H, I) || T == 0) return 0;
  return workspace_of(T, E, top_k, H, I).bytes;
}

int fpx_moe_experts(int format, const void* X, const void* ids, const void* weights, const void* gate_up,
                    const void* gate_up_scales, const void* down, const void* down_scales, void* Y, int64_t T,
                    int64_t E, int64_t top_k, int64_t H, int64_t I, void* workspace, size_t workspace_bytes,
                    void* stream) {
  const int st = check_experts(format, X, ids, weights, gate_up, gate_up_scales, down, down_scales, Y, T, E, top_k, H,
                               I, workspace, workspace_bytes);
  if (st != FP6_OK || T == 0) return st;
  return launch_experts_format(format, make_call(X, ids, weights, gate_up, gate_up_scales, down, down_scales, Y, T, E,
                                                 top_k, H, I, workspace, stream), kGiven, nullptr, nullptr, 0);
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
  // The choice inside the first product, where that has few row blocks.
  const int64_t slots = T * top_k < E ? T * top_k : E;
  const bool fused = T <= kFusedT && E <= kFusedE && slots * (I / 16) < kFusedRows * fpx::current_cus();
  if (fused && T * E * H <= kFusedProducts) return launch_experts_format(format, c, kFromRouter, R, nullptr, renormalize);
  if (!fused && E <= kRouteE && E * H <= kRouteProducts && T <= 4 * fpx::current_cus()) {
    int* oi = static_cast<int*>(ids);
    float* ow = static_cast<float*>(weights);
    int e = c.s.E, k = c.s.k, h = c.s.H;
    const _Float16* x = c.X;
    void* args[] = {&x, &R, &e, &k, &h, &renormalize, &oi, &ow};
    st = moe_launch(reinterpret_cast<const void*>(&moe_route), dim3(static_cast<unsigned>(T)), dim3(1024), args, c.stream);
    if (st != FP6_OK) return st;
    return launch_experts_format(format, c, kGiven, nullptr, nullptr, 0);
  }
  st = T <= 4 ? launch_logits<1>(c.X, R, logits, c.s, c.stream) : launch_logits<4>(c.X, R, logits, c.s, c.stream);
  if (st != FP6_OK) return st;
  if (fused) return launch_experts_format(format, c, kFromLogits, nullptr, logits, renormalize);
  int* oi = static_cast<int*>(ids);
  float* ow = static_cast<float*>(weights);
  int E32 = c.s.E, k32 = c.s.k;
  void* args[] = {&logits, &E32, &k32, &renormalize, &oi, &ow};
  st = moe_launch(reinterpret_cast<const void*>(&moe_topk), dim3(static_cast<unsigned>(T)), dim3(64), args, c.stream);
  if (st != FP6_OK) return st;
  return launch_experts_format(format, c, kGiven, nullptr, nullptr, 0);
}

}  // extern "C"
