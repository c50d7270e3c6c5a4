// C-ABI entry points of the 8-bit block-scaled operators and the token log probabilities:
// argument checks and launches.
#include <cstring>

#include "fi_nvfp4.h"
#include "internal.h"

namespace fi {

static bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

static bool known_dtype(int dtype) {
  return dtype == FI_DTYPE_BF16 || dtype == FI_DTYPE_F16 || dtype == FI_DTYPE_F32;
}

static int dtype_bytes(int dtype) { return dtype == FI_DTYPE_F32 ? 4 : 2; }

// a * b <= 2^62 (sizes whose element offsets stay inside int64, whatever the element size)
static bool product_fits(int64_t a, int64_t b) { return b == 0 || a <= ((int64_t)1 << 60) / b; }

static int quantize(const void* x, int dtype, int64_t rows, int64_t k, bool square, uint8_t* q, float* scale,
                    fi_stream_t stream) {
  clear_error();
  if (!known_dtype(dtype)) return set_error(FI_ERR_INVALID_ARG, "dtype %d is not an fi_dtype", dtype);
  if (rows < 0 || k < 0) return set_error(FI_ERR_INVALID_ARG, "negative size");
  if (k % 16 != 0) return set_error(FI_ERR_UNSUPPORTED_SHAPE, "k=%lld is not a multiple of 16", (long long)k);
  if (!product_fits(rows, k) || fp8_blocks(k) > 0x7fffffffLL)
    return set_error(FI_ERR_UNSUPPORTED_SHAPE, "%lld x %lld is too large", (long long)rows, (long long)k);
  if (rows == 0 || k == 0) return FI_OK;
  if (!x || !q || !scale) return set_error(FI_ERR_INVALID_ARG, "null pointer argument");
  if (!aligned(x, 16) || !aligned(q, 16) || !aligned(scale, 4))
    return set_error(FI_ERR_INVALID_ARG, "the input and the codes must be 16-byte, the scales 4-byte aligned");
  const int rc = check_arch();
  if (rc != FI_OK) return rc;
  return launch_fp8_quantize(x, dtype, rows, k, square, q, scale, reinterpret_cast<cudaStream_t>(stream));
}

static int product(const uint8_t* A, const float* As, const uint8_t* W0, const float* Ws0, const uint8_t* W1,
                   const float* Ws1, bool gated, void* out, int out_dtype, int64_t m, int64_t n, int64_t k, int splits,
                   fi_stream_t stream) {
  clear_error();
  if (!known_dtype(out_dtype)) return set_error(FI_ERR_INVALID_ARG, "out_dtype %d is not an fi_dtype", out_dtype);
  if (m < 0 || n < 0 || k < 0) return set_error(FI_ERR_INVALID_ARG, "negative size");
  if (splits < 0 || splits > kFp8MaxSplits)
    return set_error(FI_ERR_INVALID_ARG, "splits=%d is not in [0, %d]", splits, kFp8MaxSplits);
  if (k % 16 != 0) return set_error(FI_ERR_UNSUPPORTED_SHAPE, "k=%lld is not a multiple of 16", (long long)k);
  if (!product_fits(m, n) || !product_fits(m, k) || !product_fits(n, k))
    return set_error(FI_ERR_UNSUPPORTED_SHAPE, "m=%lld n=%lld k=%lld is too large", (long long)m, (long long)n,
                     (long long)k);
  if (m == 0 || n == 0) return FI_OK;
  if (!out || !aligned(out, dtype_bytes(out_dtype)))
    return set_error(FI_ERR_INVALID_ARG, "out must be a device pointer aligned to its elements");
  if (k > 0) {
    if (!A || !As || !W0 || !Ws0 || (gated && (!W1 || !Ws1)))
      return set_error(FI_ERR_INVALID_ARG, "null pointer argument");
    if (!aligned(A, 16) || !aligned(W0, 16) || (gated && !aligned(W1, 16)))
      return set_error(FI_ERR_INVALID_ARG, "the codes must be 16-byte aligned");
    if (!aligned(As, 4) || !aligned(Ws0, 4) || (gated && !aligned(Ws1, 4)))
      return set_error(FI_ERR_INVALID_ARG, "the scales must be 4-byte aligned");
  }
  const int rc = check_arch();
  if (rc != FI_OK) return rc;
  if (k == 0) {  // empty sums: 0, and silu(0) * 0 = 0
    if (cudaMemsetAsync(out, 0, (size_t)(m * n) * dtype_bytes(out_dtype), reinterpret_cast<cudaStream_t>(stream)) !=
        cudaSuccess)
      return set_cuda_error("cudaMemsetAsync(out)");
    return FI_OK;
  }
  Fp8MmArgs a;
  memset(&a, 0, sizeof(a));
  a.A = A;
  a.As = As;
  a.W[0] = W0;
  a.W[1] = gated ? W1 : W0;
  a.Ws[0] = Ws0;
  a.Ws[1] = gated ? Ws1 : Ws0;
  a.out = out;
  a.out_dtype = out_dtype;
  a.m = m;
  a.n = n;
  a.k = k;
  a.kblocks = (int)fp8_blocks(k);
  return launch_fp8_mm(a, gated, splits, reinterpret_cast<cudaStream_t>(stream));
}

}  // namespace fi

using namespace fi;

extern "C" {

int fi_fp8_quantize(const void* A, int dtype, int64_t m, int64_t k, uint8_t* Aq, float* Ascale, fi_stream_t stream) {
  return quantize(A, dtype, m, k, false, Aq, Ascale, stream);
}

int fi_fp8_pack_weights(const void* W, int dtype, int64_t n, int64_t k, uint8_t* Wq, float* Wscale,
                        fi_stream_t stream) {
  return quantize(W, dtype, n, k, true, Wq, Wscale, stream);
}

int fi_mm_fp8(const uint8_t* Aq, const float* Ascale, const uint8_t* Wq, const float* Wscale, void* out, int out_dtype,
              int64_t m, int64_t n, int64_t k, fi_stream_t stream) {
  return product(Aq, Ascale, Wq, Wscale, nullptr, nullptr, false, out, out_dtype, m, n, k, 0, stream);
}

int fi_mm_fp8_ex(const uint8_t* Aq, const float* Ascale, const uint8_t* Wq, const float* Wscale, void* out,
                 int out_dtype, int64_t m, int64_t n, int64_t k, int splits, fi_stream_t stream) {
  return product(Aq, Ascale, Wq, Wscale, nullptr, nullptr, false, out, out_dtype, m, n, k, splits, stream);
}

int fi_mm_fp8_gated(const uint8_t* Aq, const float* Ascale, const uint8_t* Gq, const float* Gscale, const uint8_t* Uq,
                    const float* Uscale, void* out, int out_dtype, int64_t m, int64_t n, int64_t k,
                    fi_stream_t stream) {
  return product(Aq, Ascale, Gq, Gscale, Uq, Uscale, true, out, out_dtype, m, n, k, 0, stream);
}

int fi_mm_fp8_gated_ex(const uint8_t* Aq, const float* Ascale, const uint8_t* Gq, const float* Gscale,
                       const uint8_t* Uq, const float* Uscale, void* out, int out_dtype, int64_t m, int64_t n,
                       int64_t k, int splits, fi_stream_t stream) {
  return product(Aq, Ascale, Gq, Gscale, Uq, Uscale, true, out, out_dtype, m, n, k, splits, stream);
}

int fi_token_logprobs(const void* logits, int dtype, int64_t rows, int64_t vocab, int64_t ld, const int64_t* tokens,
                      int topk, float* logprob, float* entropy, int64_t* rank, float* top_logprobs, int64_t* top_ids,
                      fi_stream_t stream) {
  clear_error();
  if (!known_dtype(dtype)) return set_error(FI_ERR_INVALID_ARG, "dtype %d is not an fi_dtype", dtype);
  if (rows < 0 || vocab < 0) return set_error(FI_ERR_INVALID_ARG, "negative size");
  if (topk < 0 || topk > kLogprobMaxTopk)
    return set_error(FI_ERR_INVALID_ARG, "topk=%d is not in [0, %d]", topk, kLogprobMaxTopk);
  if (rows == 0) return FI_OK;
  if (vocab == 0) return set_error(FI_ERR_UNSUPPORTED_SHAPE, "an empty vocabulary has no probabilities");
  if (ld < vocab) return set_error(FI_ERR_INVALID_ARG, "ld=%lld is less than vocab=%lld", (long long)ld, (long long)vocab);
  if (vocab > 0x7fff0000LL || !product_fits(rows, ld) || rows > 0x0fffffffLL)
    return set_error(FI_ERR_UNSUPPORTED_SHAPE, "rows=%lld vocab=%lld is too large", (long long)rows, (long long)vocab);
  if (!logits || !tokens || !logprob || !entropy || !rank || (topk > 0 && (!top_logprobs || !top_ids)))
    return set_error(FI_ERR_INVALID_ARG, "null pointer argument");
  if (!aligned(logits, dtype_bytes(dtype)) || !aligned(tokens, 8) || !aligned(logprob, 4) || !aligned(entropy, 4) ||
      !aligned(rank, 8) || !aligned(top_logprobs, 4) || !aligned(top_ids, 8))
    return set_error(FI_ERR_INVALID_ARG, "a pointer is not aligned to its elements");
  const int rc = check_arch();
  if (rc != FI_OK) return rc;
  LogprobArgs a;
  a.logits = logits;
  a.rows = rows;
  a.vocab = vocab;
  a.ld = ld;
  a.tokens = tokens;
  a.topk = topk < vocab ? topk : (int)vocab;
  a.logprob = logprob;
  a.entropy = entropy;
  a.rank = rank;
  a.top_logprobs = top_logprobs;
  a.top_ids = top_ids;
  return launch_token_logprobs(a, dtype, reinterpret_cast<cudaStream_t>(stream));
}

}  // extern "C"
