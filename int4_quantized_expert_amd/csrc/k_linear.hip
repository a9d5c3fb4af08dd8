// k_linear.hip — y = act(W x + b) + r over the library's row-tiled int4 / int8 codes, activations in fp32, bf16 or
// fp16 and not quantized.
#define MOE_ADAPTED 0
#define MOE_TRANSPOSED 0
#include "linear_kernels.h"

namespace moe {

namespace {
int slim_frags(int64_t T) { return T <= 16 ? 1 : 2; }
size_t slim_bytes(int N, int K, int64_t T) {
  const SlimPlan s = slim_plan(N, K / 32, slim_frags(T), T);
  return s.parts > 1 ? (size_t)s.parts * T * N * 4 : 0;
}
}  // namespace

// for any number of tokens up to T
size_t linear_ws_bytes(const moe_linear_config& c, int64_t T) {
  size_t b = is_slim(T, c.rows) ? 256 : linear_plan(c.cols, T).total;
  const int64_t most = std::min(T, std::max<int64_t>(kSlimTokens, kSlimWork / c.rows));
  b = std::max(b, slim_bytes(c.rows, c.cols, std::min<int64_t>(T, 16)));
  for (int64_t t = 32; t < most + 32; t += 32) b = std::max(b, slim_bytes(c.rows, c.cols, std::min(t, most)));
  return b;
}

hipError_t launch_linear(const moe_linear_config& c, const uint8_t* codes, const float* scales, const float* bias,
                         const void* x, int64_t ldx, int T, int dtype, const void* res, int64_t ldr, void* y,
                         int64_t ldy, void* ws, hipStream_t st) {
  const LinearArgs a = linear_args(c, codes, scales, bias, x, ldx, T, dtype, res, ldr, y, ldy, ws);
  const int bits = c.weight_bits == 8 ? 8 : 4;
  if (dtype == MOE_DTYPE_F32) linear_launch<float>(a, bits, ws, st);
  else if (dtype == MOE_DTYPE_BF16) linear_launch<bf16_t>(a, bits, ws, st);
  else linear_launch<_Float16>(a, bits, ws, st);
  return hipGetLastError();
}

}  // namespace moe
