// Causal attention over a sliding window and a few first tokens.
#include "api_check.h"
#include "common.cuh"
#include "launch.h"

using namespace csa;

extern "C" csa_status csa_window_attn(const void* q, int64_t q_stride, const void* k,
                                      int64_t k_stride, const void* v, int64_t v_stride,
                                      int64_t window, int64_t first, const float* sink,
                                      float scale, int64_t batch, int64_t n_q, int64_t n_k, int nh,
                                      int nkv, int c, csa_dtype dt, void* out, void* stream) {
  API_REQUIRE(api_valid_dt(dt), "dt must be CSA_F32 or CSA_BF16");
  API_REQUIRE(batch >= 0 && n_q >= 0 && n_k >= n_q, "batch and n_q must be >= 0, and n_k >= n_q");
  API_REQUIRE(nkv >= 1 && nh >= 1 && nh % nkv == 0, "nh must be a positive multiple of nkv");
  API_REQUIRE(c >= 8 && c % 8 == 0, "c must be a positive multiple of 8");
  API_REQUIRE(window >= 1, "window must be >= 1");
  API_REQUIRE(first >= 0, "first must be >= 0");
  API_REQUIRE(scale == scale && scale > -3.4e38f && scale < 3.4e38f, "scale must be finite");
  const int64_t unit = dt == CSA_F32 ? 4 : 8;
  API_REQUIRE(q_stride >= (int64_t)nh * c && q_stride % unit == 0 &&
                  k_stride >= (int64_t)nkv * c && k_stride % unit == 0 &&
                  (v == nullptr || (v_stride >= (int64_t)nkv * c && v_stride % unit == 0)),
              "strides must cover a token's heads and be whole 16-byte units");
  if (v == nullptr) {
    API_SUPPORTED(nkv == 1 && n_q == n_k && q_stride == (int64_t)nh * c && k_stride == c,
                  "the shared form needs nkv = 1, n_q = n_k and dense rows");
    API_SUPPORTED(c % 32 == 0 && c <= 512, "attention needs c %% 32 == 0 and c <= 512");
  } else {
    API_SUPPORTED(dt == CSA_BF16 && (c == 64 || c == 128),
                  "window attention with separate values needs bf16 and c = 64 or 128");
    API_SUPPORTED(nh / nkv <= 128, "window attention needs nh / nkv <= 128");
  }
  API_SUPPORTED(n_k < ((int64_t)1 << 30) && batch < ((int64_t)1 << 31),
                "csa_window_attn needs n_k < 2^30");
  if (batch == 0 || n_q == 0) return api_ok();
  API_REQUIRE_PTR(q);
  API_REQUIRE_PTR(k);
  API_REQUIRE_PTR(out);
  API_REQUIRE_OPT_PTR(v);
  API_REQUIRE_OPT_LIST(sink);
  const cudaStream_t s = (cudaStream_t)stream;
  if (v == nullptr) {
    API_SUPPORTED(batch * n_q < ((int64_t)1 << 31) && batch <= 65535, "csa_window_attn: too many rows");
    return api_cuda(launch_attn(q, k, nullptr, 0, k, (int)std::min(window, n_k), sink, scale, batch,
                                n_q, nh, c, 1, dt, nullptr, out, s, first),
                    "csa_window_attn");
  }
  API_SUPPORTED(batch <= (((int64_t)1 << 31) - 1) / nkv / n_q, "csa_window_attn: too many rows");
  unsigned int* flag = device_timeout_flag();
  if (flag == nullptr) return set_last_error(CSA_ERR_CUDA, "csa_window_attn: no device flag");
  return api_cuda(launch_window_attn_tc(q, q_stride, k, k_stride, v, v_stride, window, first, sink,
                                        scale, batch, n_q, n_k, nh, nkv, c, out, flag, s),
                  "csa_window_attn");
}
