// fp8_rows.cu -- the product of e4m3 codes for a few tokens (fp8_rows.cuh).
#include "fp8_rows.cuh"

namespace bakron {

// This kernel starts and ends sooner and takes longer for a code, the more so
// the more tokens there are.  Microseconds here / on the tensor cores (weights from
// memory, bf16): 1000 -> 512, 1 to 4 tokens 3.6 to 4.6 / 8.6; 4096 -> 4096, 1, 2, 3, 4
// tokens 7.1, 9.6, 11.7, 13.7 / 11.9; 4096 -> 14336, 1, 2 tokens 16.2, 20.4 / 16.3;
// 14336 -> 4096, 1 token 20.4 / 18.2.
bool fp8_few_tokens(int64_t T, int64_t K, int64_t N) {
  return T <= kRowTokens && row_smem(T, K) <= kRowSmem && K * N * (3 * T - 1) <= 100000000;
}

cudaError_t fp8_rows(const Fp8Matmul& p, int32_t* status, cudaStream_t stream) {
  switch (p.y_dtype) {
    case kF32: return fp8_rows_launch<float>(p, status, stream);
    case kF16: return fp8_rows_launch<__half>(p, status, stream);
    default: return fp8_rows_launch<__nv_bfloat16>(p, status, stream);
  }
}

}  // namespace bakron
