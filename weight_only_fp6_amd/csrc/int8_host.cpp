// Host side of the 8-bit integer linear layer: size rules and the row quantiser
// of the weights.  Plain C++17, no HIP calls.

#include "fp6_int8.h"
#include "fp6_limits.h"

#include <cmath>
#include <cstring>

extern "C" {

int64_t fp6_int8_padded_k(int64_t K) {
  if (K < 1 || K > fp6::kInt8MaxK) return 0;
  return (K + 15) / 16 * 16;
}

size_t fp6_int8_workspace_bytes(int64_t M, int64_t K) {
  const int64_t kp = fp6_int8_padded_k(K);
  if (!kp || M < 1 || M > fp6::kMaxDim || M * kp > fp6::kMaxNK) return 0;
  return static_cast<size_t>(M) * static_cast<size_t>(kp) + static_cast<size_t>(M) * sizeof(float);
}

int fp6_int8_quantize_rows(const float* W, int64_t N, int64_t K, int8_t* codes, float* scales) {
  if (!W || !codes || !scales) return FP6_E_NULL;
  const int64_t kp = fp6_int8_padded_k(K);
  if (!kp || N < 1 || N > fp6::kMaxDim || N * kp > fp6::kMaxNK) return FP6_E_SHAPE;
  for (int64_t n = 0; n < N; ++n) {
    const float* row = W + n * K;
    int8_t* out = codes + n * kp;
    float top = 0.0f;
    for (int64_t k = 0; k < K; ++k) {
      if (!std::isfinite(row[k])) return FP6_E_VALUE;
      top = std::fmax(top, std::fabs(row[k]));
    }
    scales[n] = static_cast<float>(static_cast<double>(top) / 127.0);
    std::memset(out, 0, static_cast<size_t>(kp));
    if (top == 0.0f) continue;
    // The product with 127 is exact in double and the quotient of two floats
    // of 24 + 7 and 24 bits cannot round onto a tie that it is not.
    for (int64_t k = 0; k < K; ++k)
      out[k] = static_cast<int8_t>(std::nearbyint(127.0 * static_cast<double>(row[k]) / static_cast<double>(top)));
  }
  return FP6_OK;
}

}  // extern "C"
