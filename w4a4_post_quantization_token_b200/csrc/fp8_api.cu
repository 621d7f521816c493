// C-ABI entry points of the 8-bit operators (declared in include/kq.h): argument checks on the
// host, tensor maps and launches on the caller's stream.
#include <cmath>
#include <cstring>

#include "../../include/kq.h"
#include "fp8.cuh"
#include "host.cuh"

using namespace kq;

namespace {

kq_status check_width(int32_t K) {
  if (K <= 0) return KQ_ERR_INVALID_ARG;
  return K % 32 == 0 && K <= fp8::kMaxWidth ? KQ_OK : KQ_ERR_UNSUPPORTED_SHAPE;
}

kq_status check_fp8(const kq_fp8_desc* d) {
  if (!d || d->K <= 0 || d->N <= 0) return KQ_ERR_INVALID_ARG;
  if (d->gated != 0 && d->gated != 1) return KQ_ERR_INVALID_ARG;
  if (d->activation != KQ_ACT_SILU && d->activation != KQ_ACT_GELU) return KQ_ERR_INVALID_ARG;
  if (d->K % 32 != 0 || d->N % 16 != 0 || d->K > fp8::kMaxWidth || d->N > fp8::kMaxWidth)
    return KQ_ERR_UNSUPPORTED_SHAPE;
  return KQ_OK;
}

fp8::WLayout wlayout(const kq_fp8_desc* d) { return fp8::WLayout::make(d->K, d->N, d->gated != 0); }

// Rows of a caller's matrix: pitch in elements, at least `width`, rows 16-byte aligned.
kq_status check_rows(const void* p, int64_t ld, int32_t width, int elem) {
  if (!p || ld < width) return KQ_ERR_INVALID_ARG;
  return aligned(p) && (ld * elem) % 16 == 0 ? KQ_OK : KQ_ERR_ALIGNMENT;
}

kq_status check_act(const void* act, size_t bytes, int32_t K, int32_t M) {
  if (!act || M <= 0) return KQ_ERR_INVALID_ARG;
  if (!aligned(act)) return KQ_ERR_ALIGNMENT;
  return bytes < fp8::ALayout::make(M, K).total ? KQ_ERR_WORKSPACE_TOO_SMALL : KQ_OK;
}

// Whether two matrices' address ranges meet (rows of `w` bytes, `pitch` bytes apart).
bool meet(const void* a, int64_t pa, int64_t wa, const void* b, int64_t pb, int64_t wb, int32_t rows) {
  const uintptr_t a0 = reinterpret_cast<uintptr_t>(a), b0 = reinterpret_cast<uintptr_t>(b);
  const uintptr_t a1 = a0 + static_cast<uintptr_t>((rows - 1) * pa + wa), b1 = b0 + static_cast<uintptr_t>((rows - 1) * pb + wb);
  return a0 < b1 && b0 < a1;
}

struct Norm {
  void* residual = nullptr;
  int64_t ldr = 0;
  int32_t dtype = KQ_OUT_F32;
  const float* gamma = nullptr;
  float eps = 0.f;
};

kq_status check_norm(const Norm& n, int32_t K) {
  if (!n.gamma || !(n.eps > 0.f) || !std::isfinite(n.eps)) return KQ_ERR_INVALID_ARG;
  if (K > fp8::kNormMaxK) return KQ_ERR_UNSUPPORTED_SHAPE;
  if (!aligned(n.gamma)) return KQ_ERR_ALIGNMENT;
  if (!n.residual) return KQ_OK;
  if (n.dtype != KQ_OUT_F32 && n.dtype != KQ_OUT_BF16) return KQ_ERR_INVALID_ARG;
  return check_rows(n.residual, n.ldr, K, n.dtype == KQ_OUT_BF16 ? 2 : 4);
}

kq_status check_y(const void* Y, int64_t ldy, int32_t N, int32_t out_dtype) {
  if (out_dtype != KQ_OUT_F32 && out_dtype != KQ_OUT_BF16) return KQ_ERR_INVALID_ARG;
  return check_rows(Y, ldy, N, out_dtype == KQ_OUT_BF16 ? 2 : 4);
}

kq_status run_rows(int32_t K, const void* X, int64_t ldx, const Norm* n, int32_t M, uint8_t* act, cudaStream_t st) {
  const fp8::ALayout L = fp8::ALayout::make(M, K);
  fp8::NormParams p;
  std::memset(&p, 0, sizeof(p));
  p.x = X; p.ldx = ldx; p.M = M; p.K = K;
  p.katoms = fp8::katoms(K);
  p.codes = act + L.codes;
  p.sf = act + L.sf;
  p.err = reinterpret_cast<uint32_t*>(act + L.err);
  int res = 0;
  if (n) {
    p.residual = n->residual; p.ldr = n->ldr; p.gamma = n->gamma; p.eps = n->eps;
    res = !n->residual ? 0 : n->dtype == KQ_OUT_BF16 ? 1 : 2;
  }
  return fp8::launch_rows(p, n != nullptr, res, st) == cudaSuccess ? KQ_OK : KQ_ERR_CUDA;
}

// A run whose waits are to end early (kq_fp8_debug_wait_timeout).
struct Withhold { int k_tile = -1; uint64_t wait_ns = kWaitLimitNs; };

// Y (out 0 / 1) or the 8-bit workspace `oact` (out 2) from the activations in `act`.
kq_status run_mm(const kq_fp8_desc* d, const void* weights, uint8_t* act, int32_t M, int out, void* Y,
                 int64_t ldy, uint8_t* oact, uint32_t* err, bool dependent, const DeviceInfo& di, cudaStream_t st,
                 const void* xb = nullptr, int64_t ldx = 0, const Withhold& wh = Withhold()) {
  const fp8::WLayout W = wlayout(d);
  const fp8::ALayout A = fp8::ALayout::make(M, d->K);
  const uint8_t* w = static_cast<const uint8_t*>(weights);
  fp8::MmParams p;
  std::memset(&p, 0, sizeof(p));
  const uint64_t K = static_cast<uint64_t>(d->K);
  const fp8::Device dev = {di.sms, di.device};
  const fp8::PairShape shape = fp8::pair_shape(M, d->N, d->K, d->gated != 0, dev);
  p.pairs = shape.cols;
  p.splits = shape.splits;
  const uint32_t wrows = p.pairs ? static_cast<uint32_t>(p.pairs / 2) : 128;
  for (int i = 0; i < 1 + d->gated; ++i) {
    if (!make_tmap(&p.tmap_w[i], CU_TENSOR_MAP_DATA_TYPE_UINT8, w + W.codes[i], K, static_cast<uint64_t>(d->N), K,
                   128, wrows, CU_TENSOR_MAP_SWIZZLE_128B))
      return KQ_ERR_CUDA;
    p.sfw[i] = w + W.sf[i];
  }
  p.M = M; p.N = d->N; p.K = d->K;
  p.katoms = fp8::katoms(d->K);
  p.act = d->activation;
  p.out = out;
  p.y = Y;
  p.ldy = ldy;
  p.err = err;
  p.wait_ns = wh.wait_ns;
  p.withhold = wh.k_tile;
  if (out == 2) {
    const fp8::ALayout O = fp8::ALayout::make(M, d->N);
    p.ocodes = oact + O.codes;
    p.osf = oact + O.sf;
    p.okatoms = fp8::katoms(d->N);
    p.oerr = reinterpret_cast<uint32_t*>(oact + O.err);
  }
  if (xb) {
    // bf16 activations: few tokens are encoded by the product's own kernel, unless its output may
    // lie on them (other CTAs would still read)
    p.xb = xb;
    p.ldx = ldx;
    const int64_t ye = out == 1 ? 2 : 4;
    const bool apart = !meet(xb, ldx * 2, int64_t{2} * d->K, Y, ldy * ye, ye * d->N, M);
    cudaError_t e = cudaSuccess;
    if (!p.pairs && apart && fp8::try_rows_fused(p, d->gated != 0, dev, st, &e)) return e == cudaSuccess ? KQ_OK : KQ_ERR_CUDA;
    const kq_status s = run_rows(d->K, xb, ldx, nullptr, M, act, st);
    if (s != KQ_OK) return s;
    dependent = true;
  }
  p.dependent = dependent ? 1 : 0;
  if (!make_tmap(&p.tmap_x, CU_TENSOR_MAP_DATA_TYPE_UINT8, act + A.codes, K, static_cast<uint64_t>(M), K, 128,
                 static_cast<uint32_t>(p.pairs ? 128 : fp8::rows_token_tile(M)), CU_TENSOR_MAP_SWIZZLE_128B))
    return KQ_ERR_CUDA;
  p.sfx = act + A.sf;
  if (!p.pairs) return fp8::launch_rows_mm(p, d->gated != 0, dev, st) == cudaSuccess ? KQ_OK : KQ_ERR_CUDA;
  auto atoms = [&](CUtensorMap* m, const uint8_t* sf, int64_t rows) {
    return make_tmap(m, CU_TENSOR_MAP_DATA_TYPE_UINT32, sf, 128, static_cast<uint64_t>(cdiv(rows, 128) * p.katoms), 512,
                     128, 1, CU_TENSOR_MAP_SWIZZLE_NONE);
  };
  if (!atoms(&p.tmap_sfx, p.sfx, M)) return KQ_ERR_CUDA;
  for (int i = 0; i < 1 + d->gated; ++i)
    if (!atoms(&p.tmap_sfw[i], p.sfw[i], d->N)) return KQ_ERR_CUDA;
  return fp8::launch_pair(p, d->gated != 0, di.sms, st) == cudaSuccess ? KQ_OK : KQ_ERR_CUDA;
}

uint32_t* err_word(void* act) { return reinterpret_cast<uint32_t*>(act); }

}  // namespace

extern "C" {

size_t kq_fp8_weights_bytes(const kq_fp8_desc* desc) {
  return check_fp8(desc) == KQ_OK ? wlayout(desc).total : 0;
}

size_t kq_fp8_act_bytes(int32_t K, int32_t M) {
  return check_width(K) == KQ_OK && M > 0 ? fp8::ALayout::make(M, K).total : 0;
}

size_t kq_fp8_ffn_bytes(const kq_fp8_desc* gated, const kq_fp8_desc* down, int32_t M) {
  if (check_fp8(gated) != KQ_OK || check_fp8(down) != KQ_OK || M <= 0) return 0;
  if (gated->gated != 1 || down->gated != 0 || down->K != gated->N) return 0;
  return fp8::ALayout::make(M, gated->K).total + fp8::ALayout::make(M, gated->N).total;
}

kq_status kq_fp8_prepare_weights(const kq_fp8_desc* desc, const void* W_bf16, const void* Wup_bf16, void* weights,
                                 kq_stream_t stream) {
  kq_status s = check_fp8(desc);
  if (s != KQ_OK) return s;
  if (!W_bf16 || !weights || (desc->gated != 0) != (Wup_bf16 != nullptr)) return KQ_ERR_INVALID_ARG;
  if (!aligned(W_bf16) || !aligned(weights) || !aligned(Wup_bf16)) return KQ_ERR_ALIGNMENT;
  DeviceInfo di;
  if ((s = current_device(&di)) != KQ_OK) return s;
  const fp8::WLayout L = wlayout(desc);
  uint8_t* w = static_cast<uint8_t*>(weights);
  const void* src[2] = {W_bf16, Wup_bf16};
  for (int i = 0; i < 1 + desc->gated; ++i)
    if (fp8::launch_weight_quant(src[i], desc->K, desc->N, w + L.codes[i], w + L.sf[i],
                                 reinterpret_cast<cudaStream_t>(stream)) != cudaSuccess)
      return KQ_ERR_CUDA;
  return KQ_OK;
}

static kq_status move_weights(const kq_fp8_desc* desc, void* codes, void* scales, void* up_codes, void* up_scales,
                              void* weights, bool pack, kq_stream_t stream) {
  kq_status s = check_fp8(desc);
  if (s != KQ_OK) return s;
  if (!weights) return KQ_ERR_INVALID_ARG;
  if (!aligned(weights)) return KQ_ERR_ALIGNMENT;
  if (!desc->gated && (up_codes || up_scales)) return KQ_ERR_INVALID_ARG;
  if (pack && (!codes || !scales || (desc->gated && (!up_codes || !up_scales)))) return KQ_ERR_INVALID_ARG;
  DeviceInfo di;
  if ((s = current_device(&di)) != KQ_OK) return s;
  const fp8::WLayout L = wlayout(desc);
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  void* c[2] = {codes, up_codes};
  void* sc[2] = {scales, up_scales};
  const size_t n = static_cast<size_t>(desc->N) * desc->K;
  for (int i = 0; i < 1 + desc->gated; ++i) {
    uint8_t* w = static_cast<uint8_t*>(weights) + L.codes[i];
    if (c[i] && cudaMemcpyAsync(pack ? w : c[i], pack ? c[i] : w, n, cudaMemcpyDeviceToDevice, st) != cudaSuccess)
      return KQ_ERR_CUDA;
    if (sc[i] && fp8::launch_weight_scales(static_cast<uint8_t*>(sc[i]), desc->K, desc->N,
                                           static_cast<uint8_t*>(weights) + L.sf[i], pack, st) != cudaSuccess)
      return KQ_ERR_CUDA;
  }
  return KQ_OK;
}

kq_status kq_fp8_weights_pack(const kq_fp8_desc* desc, const void* codes, const void* scales, const void* up_codes,
                              const void* up_scales, void* weights, kq_stream_t stream) {
  return move_weights(desc, const_cast<void*>(codes), const_cast<void*>(scales), const_cast<void*>(up_codes),
                      const_cast<void*>(up_scales), weights, true, stream);
}

kq_status kq_fp8_weights_unpack(const kq_fp8_desc* desc, const void* weights, void* codes, void* scales,
                                void* up_codes, void* up_scales, kq_stream_t stream) {
  return move_weights(desc, codes, scales, up_codes, up_scales, const_cast<void*>(weights), false, stream);
}

kq_status kq_fp8_quantize_act(int32_t K, const void* X_bf16, int64_t ldx, int32_t M, void* act, size_t act_bytes,
                              kq_stream_t stream) {
  kq_status s = check_width(K);
  if (s != KQ_OK) return s;
  if ((s = check_act(act, act_bytes, K, M)) != KQ_OK) return s;
  if ((s = check_rows(X_bf16, ldx, K, 2)) != KQ_OK) return s;
  DeviceInfo di;
  if ((s = current_device(&di)) != KQ_OK) return s;
  return run_rows(K, X_bf16, ldx, nullptr, M, static_cast<uint8_t*>(act), reinterpret_cast<cudaStream_t>(stream));
}

kq_status kq_fp8_rmsnorm_act(int32_t K, const void* X_bf16, int64_t ldx, void* residual, int64_t ldr,
                             int32_t residual_dtype, const float* gamma, float eps, int32_t M, void* act,
                             size_t act_bytes, kq_stream_t stream) {
  kq_status s = check_width(K);
  if (s != KQ_OK) return s;
  Norm n;
  n.residual = residual; n.ldr = ldr; n.dtype = residual_dtype; n.gamma = gamma; n.eps = eps;
  if ((s = check_act(act, act_bytes, K, M)) != KQ_OK) return s;
  if ((s = check_rows(X_bf16, ldx, K, 2)) != KQ_OK) return s;
  if ((s = check_norm(n, K)) != KQ_OK) return s;
  DeviceInfo di;
  if ((s = current_device(&di)) != KQ_OK) return s;
  return run_rows(K, X_bf16, ldx, &n, M, static_cast<uint8_t*>(act), reinterpret_cast<cudaStream_t>(stream));
}

kq_status kq_fp8_act_pack(int32_t K, const void* codes, const void* scales, int32_t M, void* act, size_t act_bytes,
                          kq_stream_t stream) {
  kq_status s = check_width(K);
  if (s != KQ_OK) return s;
  if ((s = check_act(act, act_bytes, K, M)) != KQ_OK) return s;
  if (!codes || !scales) return KQ_ERR_INVALID_ARG;
  DeviceInfo di;
  if ((s = current_device(&di)) != KQ_OK) return s;
  const fp8::ALayout L = fp8::ALayout::make(M, K);
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  uint8_t* a = static_cast<uint8_t*>(act);
  if (cudaMemsetAsync(a + L.err, 0, 4, st) != cudaSuccess ||
      cudaMemcpyAsync(a + L.codes, codes, static_cast<size_t>(M) * K, cudaMemcpyDeviceToDevice, st) != cudaSuccess ||
      fp8::launch_act_scales(static_cast<uint8_t*>(const_cast<void*>(scales)), K, M, a + L.sf, true, st) !=
          cudaSuccess)
    return KQ_ERR_CUDA;
  return KQ_OK;
}

kq_status kq_fp8_act_unpack(int32_t K, const void* act, int32_t M, void* codes, void* scales, void* values,
                            int32_t values_dtype, kq_stream_t stream) {
  kq_status s = check_width(K);
  if (s != KQ_OK) return s;
  if (!act || M <= 0) return KQ_ERR_INVALID_ARG;
  if (values && values_dtype != KQ_OUT_F32 && values_dtype != KQ_OUT_BF16) return KQ_ERR_INVALID_ARG;
  if (!aligned(act) || !aligned(values)) return KQ_ERR_ALIGNMENT;
  DeviceInfo di;
  if ((s = current_device(&di)) != KQ_OK) return s;
  const fp8::ALayout L = fp8::ALayout::make(M, K);
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  uint8_t* a = static_cast<uint8_t*>(const_cast<void*>(act));
  if (codes && cudaMemcpyAsync(codes, a + L.codes, static_cast<size_t>(M) * K, cudaMemcpyDeviceToDevice, st) !=
                   cudaSuccess)
    return KQ_ERR_CUDA;
  if (scales && fp8::launch_act_scales(static_cast<uint8_t*>(scales), K, M, a + L.sf, false, st) != cudaSuccess)
    return KQ_ERR_CUDA;
  if (values &&
      fp8::launch_act_values(a + L.codes, a + L.sf, K, M, values, values_dtype == KQ_OUT_BF16, st) != cudaSuccess)
    return KQ_ERR_CUDA;
  return KQ_OK;
}

kq_status kq_fp8_gemm(const kq_fp8_desc* desc, const void* weights, void* act, int32_t M, void* Y, int64_t ldy,
                      int32_t out_dtype, kq_stream_t stream) {
  kq_status s = check_fp8(desc);
  if (s != KQ_OK) return s;
  if (M <= 0 || !weights || !act) return KQ_ERR_INVALID_ARG;
  if (!aligned(weights) || !aligned(act)) return KQ_ERR_ALIGNMENT;
  if ((s = check_y(Y, ldy, desc->N, out_dtype)) != KQ_OK) return s;
  DeviceInfo di;
  if ((s = current_device(&di)) != KQ_OK) return s;
  return run_mm(desc, weights, static_cast<uint8_t*>(act), M, out_dtype == KQ_OUT_BF16 ? 1 : 0, Y, ldy, nullptr,
                err_word(act), false, di, reinterpret_cast<cudaStream_t>(stream));
}

kq_status kq_fp8_gated_act(const kq_fp8_desc* desc, const void* weights, void* act, int32_t M, void* out_act,
                           size_t out_act_bytes, kq_stream_t stream) {
  kq_status s = check_fp8(desc);
  if (s != KQ_OK) return s;
  if (!desc->gated || M <= 0 || !weights || !act || act == out_act) return KQ_ERR_INVALID_ARG;
  if ((s = check_width(desc->N)) != KQ_OK) return s;
  if (!aligned(weights) || !aligned(act)) return KQ_ERR_ALIGNMENT;
  if ((s = check_act(out_act, out_act_bytes, desc->N, M)) != KQ_OK) return s;
  DeviceInfo di;
  if ((s = current_device(&di)) != KQ_OK) return s;
  return run_mm(desc, weights, static_cast<uint8_t*>(act), M, 2, nullptr, 0, static_cast<uint8_t*>(out_act),
                err_word(act), false, di, reinterpret_cast<cudaStream_t>(stream));
}

kq_status kq_fp8_linear(const kq_fp8_desc* desc, const void* weights, const void* X_bf16, int64_t ldx, int32_t M,
                        void* Y, int64_t ldy, int32_t out_dtype, void* act, size_t act_bytes, kq_stream_t stream) {
  kq_status s = check_fp8(desc);
  if (s != KQ_OK) return s;
  if (!weights) return KQ_ERR_INVALID_ARG;
  if (!aligned(weights)) return KQ_ERR_ALIGNMENT;
  if ((s = check_act(act, act_bytes, desc->K, M)) != KQ_OK) return s;
  if ((s = check_rows(X_bf16, ldx, desc->K, 2)) != KQ_OK) return s;
  if ((s = check_y(Y, ldy, desc->N, out_dtype)) != KQ_OK) return s;
  DeviceInfo di;
  if ((s = current_device(&di)) != KQ_OK) return s;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  uint8_t* a = static_cast<uint8_t*>(act);
  return run_mm(desc, weights, a, M, out_dtype == KQ_OUT_BF16 ? 1 : 0, Y, ldy, nullptr, err_word(a), false, di, st,
                X_bf16, ldx);
}

kq_status kq_fp8_ffn(const kq_fp8_desc* gated, const void* gated_weights, const kq_fp8_desc* down,
                     const void* down_weights, const void* X_bf16, int64_t ldx, void* residual, int64_t ldr,
                     int32_t residual_dtype, const float* gamma, float eps, int32_t M, void* Y, int64_t ldy,
                     int32_t out_dtype, void* ws, size_t ws_bytes, kq_stream_t stream) {
  kq_status s;
  if ((s = check_fp8(gated)) != KQ_OK || (s = check_fp8(down)) != KQ_OK) return s;
  if (gated->gated != 1 || down->gated != 0 || down->K != gated->N) return KQ_ERR_INVALID_ARG;
  if (M <= 0 || !gated_weights || !down_weights || !ws) return KQ_ERR_INVALID_ARG;
  if (!aligned(gated_weights) || !aligned(down_weights) || !aligned(ws)) return KQ_ERR_ALIGNMENT;
  if (ws_bytes < kq_fp8_ffn_bytes(gated, down, M)) return KQ_ERR_WORKSPACE_TOO_SMALL;
  if ((s = check_rows(X_bf16, ldx, gated->K, 2)) != KQ_OK) return s;
  Norm n;
  n.residual = residual; n.ldr = ldr; n.dtype = residual_dtype; n.gamma = gamma; n.eps = eps;
  if (gamma ? (s = check_norm(n, gated->K)) != KQ_OK : residual != nullptr) return gamma ? s : KQ_ERR_INVALID_ARG;
  if ((s = check_y(Y, ldy, down->N, out_dtype)) != KQ_OK) return s;
  DeviceInfo di;
  if ((s = current_device(&di)) != KQ_OK) return s;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  uint8_t* a = static_cast<uint8_t*>(ws);
  uint8_t* h = a + fp8::ALayout::make(M, gated->K).total;
  if ((s = run_rows(gated->K, X_bf16, ldx, gamma ? &n : nullptr, M, a, st)) != KQ_OK) return s;
  if ((s = run_mm(gated, gated_weights, a, M, 2, nullptr, 0, h, err_word(a), true, di, st)) != KQ_OK) return s;
  return run_mm(down, down_weights, h, M, out_dtype == KQ_OUT_BF16 ? 1 : 0, Y, ldy, nullptr, err_word(a), true, di, st);
}

kq_status kq_fp8_debug_wait_timeout(const kq_fp8_desc* desc, const void* weights, const void* X_bf16, int64_t ldx,
                                    int32_t M, void* Y, int64_t ldy, int32_t out_dtype, void* act, size_t act_bytes,
                                    void* out_act, size_t out_act_bytes, int64_t k_tile, uint32_t limit_us,
                                    kq_stream_t stream) {
  kq_status s = check_fp8(desc);
  if (s != KQ_OK) return s;
  if (!weights || k_tile < 0 || limit_us == 0 || limit_us > 1000000u) return KQ_ERR_INVALID_ARG;
  if (!aligned(weights)) return KQ_ERR_ALIGNMENT;
  if ((s = check_act(act, act_bytes, desc->K, M)) != KQ_OK) return s;
  if (X_bf16 && (s = check_rows(X_bf16, ldx, desc->K, 2)) != KQ_OK) return s;
  if (out_act) {
    if (!desc->gated || act == out_act || X_bf16 || Y) return KQ_ERR_INVALID_ARG;
    if ((s = check_width(desc->N)) != KQ_OK || (s = check_act(out_act, out_act_bytes, desc->N, M)) != KQ_OK) return s;
  } else if ((s = check_y(Y, ldy, desc->N, out_dtype)) != KQ_OK) {
    return s;
  }
  DeviceInfo di;
  if ((s = current_device(&di)) != KQ_OK) return s;
  Withhold wh;
  wh.k_tile = k_tile > INT32_MAX ? -1 : static_cast<int>(k_tile);
  wh.wait_ns = uint64_t{1000} * limit_us;
  return run_mm(desc, weights, static_cast<uint8_t*>(act), M, out_act ? 2 : out_dtype == KQ_OUT_BF16 ? 1 : 0, Y, ldy,
                static_cast<uint8_t*>(out_act), err_word(act), false, di, reinterpret_cast<cudaStream_t>(stream), X_bf16,
                ldx, wh);
}

kq_status kq_fp8_last_device_error(void* act, kq_stream_t stream) {
  if (!act) return KQ_ERR_INVALID_ARG;
  if (!aligned(act)) return KQ_ERR_ALIGNMENT;
  if (cudaStreamSynchronize(reinterpret_cast<cudaStream_t>(stream)) != cudaSuccess) return KQ_ERR_CUDA;
  uint32_t word = 0;
  if (cudaMemcpy(&word, act, 4, cudaMemcpyDeviceToHost) != cudaSuccess) return KQ_ERR_CUDA;
  if (word != 0 && cudaMemset(act, 0, 4) != cudaSuccess) return KQ_ERR_CUDA;
  return word ? KQ_ERR_DEVICE_TIMEOUT : KQ_OK;
}

}  // extern "C"
