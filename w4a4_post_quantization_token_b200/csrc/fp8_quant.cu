// Row kernels of the 8-bit operators: the root-mean-square norm (with the residual's addition)
// and the plain quantizer write E4M3 codes with a power-of-two scale for each token and 128
// features; the weight quantizer does the same for 128 x 128 pieces; the rest convert layouts.
#include <cuda_fp16.h>

#include "fp8.cuh"

namespace kq {
namespace fp8 {

namespace {

__device__ __forceinline__ void unpack8(const uint4& u, float (&v)[8]) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(w[i] << 16);
    v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
}

// Encodes the 8 values that each thread holds of a block shared by 16 neighbouring lanes
// (lanes past a short last block hold zeros); `kb` is the block's index along K.
__device__ __forceinline__ void encode8(const float (&v)[8], bool valid, int row, int chunk, const NormParams& p) {
  uint32_t a = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) a = max(a, abs_bits(v[i]));
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) a = max(a, __shfl_xor_sync(0xffffffffu, a, o));
  const uint32_t byte = scale_byte(a);
  const float is = inv_scale(byte);
  if (!valid) return;
  uint2 c;
  c.x = e4m3x4(v[0] * is, v[1] * is, v[2] * is, v[3] * is);
  c.y = e4m3x4(v[4] * is, v[5] * is, v[6] * is, v[7] * is);
  *reinterpret_cast<uint2*>(p.codes + static_cast<size_t>(row) * p.K + chunk * 8) = c;
  if ((chunk & 15) == 0) p.sf[sf_offset(row, chunk >> 4, p.katoms)] = static_cast<uint8_t>(byte);
}

// One CTA per token. A thread holds C chunks of 8 features (16 bytes of x); 16 neighbouring
// threads share a scale.
//   h = x + residual in fp32, rounded to the residual's type and kept there;
//   r = 1 / sqrt(mean(h^2) + eps), the sum and the root in float64, rounded once to fp32;
//   y = (h r) gamma, two fp32 products; then the block's scale and codes from y.
// The float64 sum makes r, and so every code, independent of the summation order.
template <int C, int RES, bool NORM>
__global__ void __launch_bounds__(512) k_rows(const __grid_constant__ NormParams p) {
  __shared__ double part[16];
  const int row = blockIdx.x;
  const int T = blockDim.x;
  const int nch = p.K / 8;
  const int first = blockIdx.y * (T * C) + threadIdx.x;
  if (p.err != nullptr && blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0) *p.err = 0u;
  grid_dep_launch();
  const uint4* x = reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(p.x) +
                                                  static_cast<int64_t>(row) * p.ldx);
  float h[C][8];
  double sum = 0.0;
#pragma unroll
  for (int c = 0; c < C; ++c) {
    const int ch = first + c * T;
    const bool valid = ch < nch;
    uint4 u = make_uint4(0, 0, 0, 0);
    if (valid) u = x[ch];
    unpack8(u, h[c]);
    if (RES == 1 && valid) {
      uint4* rp = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p.residual) +
                                           static_cast<int64_t>(row) * p.ldr) + ch;
      float r[8];
      unpack8(*rp, r);
      uint32_t o[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const __nv_bfloat162 b = __floats2bfloat162_rn(h[c][2 * i] + r[2 * i], h[c][2 * i + 1] + r[2 * i + 1]);
        o[i] = *reinterpret_cast<const uint32_t*>(&b);
      }
      const uint4 ov = make_uint4(o[0], o[1], o[2], o[3]);
      *rp = ov;
      unpack8(ov, h[c]);
    }
    if (RES == 2 && valid) {
      float4* rp = reinterpret_cast<float4*>(static_cast<float*>(p.residual) +
                                             static_cast<int64_t>(row) * p.ldr) + 2 * ch;
      const float4 r0 = rp[0], r1 = rp[1];
      h[c][0] += r0.x; h[c][1] += r0.y; h[c][2] += r0.z; h[c][3] += r0.w;
      h[c][4] += r1.x; h[c][5] += r1.y; h[c][6] += r1.z; h[c][7] += r1.w;
      rp[0] = make_float4(h[c][0], h[c][1], h[c][2], h[c][3]);
      rp[1] = make_float4(h[c][4], h[c][5], h[c][6], h[c][7]);
    }
    if (NORM) {
#pragma unroll
      for (int i = 0; i < 8; ++i) sum = fma(static_cast<double>(h[c][i]), static_cast<double>(h[c][i]), sum);
    }
  }
  float r = 1.f;
  if (NORM) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = sum;
    __syncthreads();
    double s = 0.0;
    for (int w = 0; w < (T >> 5); ++w) s += part[w];
    r = static_cast<float>(1.0 / sqrt(s / static_cast<double>(p.K) + p.eps));
  }
#pragma unroll
  for (int c = 0; c < C; ++c) {
    const int ch = first + c * T;
    const bool valid = ch < nch;
    if (NORM && valid) {
      const float4* g = reinterpret_cast<const float4*>(p.gamma) + 2 * ch;
      const float4 g0 = __ldg(g), g1 = __ldg(g + 1);
      h[c][0] = h[c][0] * r * g0.x; h[c][1] = h[c][1] * r * g0.y;
      h[c][2] = h[c][2] * r * g0.z; h[c][3] = h[c][3] * r * g0.w;
      h[c][4] = h[c][4] * r * g1.x; h[c][5] = h[c][5] * r * g1.y;
      h[c][6] = h[c][6] * r * g1.z; h[c][7] = h[c][7] * r * g1.w;
    }
    encode8(h[c], valid, row, ch, p);
  }
}

template <int C, bool NORM>
cudaError_t launch_rows_c(const NormParams& p, int res_kind, dim3 grid, int T, cudaStream_t st) {
  if (!NORM || res_kind == 0) k_rows<C, 0, NORM><<<grid, T, 0, st>>>(p);
  else if (res_kind == 1) k_rows<C, 1, NORM><<<grid, T, 0, st>>>(p);
  else k_rows<C, 2, NORM><<<grid, T, 0, st>>>(p);
  return cudaGetLastError();
}

// One CTA per 128 (outputs) x 128 (inputs) piece of W [K, N]: transposed to K-major codes.
__global__ void __launch_bounds__(256) k_weight_quant(const uint16_t* __restrict__ W, int K, int N,
                                                      uint8_t* __restrict__ codes, uint8_t* __restrict__ sf,
                                                      int64_t ka) {
  __shared__ uint16_t tile[128][130];                     // [k][n]
  __shared__ uint32_t top[8];
  const int k0 = blockIdx.x * 128, n0 = blockIdx.y * 128;
  uint32_t a = 0;
  for (int i = threadIdx.x; i < 128 * 128; i += 256) {
    const int k = i >> 7, n = i & 127;
    const uint16_t v = (k0 + k < K && n0 + n < N) ? W[static_cast<size_t>(k0 + k) * N + n0 + n] : uint16_t{0};
    tile[k][n] = v;
    a = max(a, abs_bits(__uint_as_float(static_cast<uint32_t>(v) << 16)));
  }
  a = __reduce_max_sync(0xffffffffu, a);
  if ((threadIdx.x & 31) == 0) top[threadIdx.x >> 5] = a;
  __syncthreads();
  a = 0;
#pragma unroll
  for (int w = 0; w < 8; ++w) a = max(a, top[w]);
  const uint32_t byte = scale_byte(a);
  const float is = inv_scale(byte);
  for (int i = threadIdx.x; i < 128 * 32; i += 256) {
    const int n = i >> 5, k = (i & 31) * 4;
    if (n0 + n >= N || k0 + k >= K) continue;             // K is a multiple of 32
    float v[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] = __uint_as_float(static_cast<uint32_t>(tile[k + j][n]) << 16) * is;
    *reinterpret_cast<uint32_t*>(codes + static_cast<size_t>(n0 + n) * K + k0 + k) = e4m3x4(v[0], v[1], v[2], v[3]);
  }
  if (threadIdx.x < 128) sf[sf_offset(n0 + threadIdx.x, blockIdx.x, ka)] = static_cast<uint8_t>(byte);
}

// Canonical weight scales [cdiv(N, 128), cdiv(K, 128)] <-> atoms (every row of a block alike).
__global__ void k_weight_scales(uint8_t* canon, int kb, int nb, uint8_t* sf, int64_t ka, bool pack) {
  const int64_t i = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x;
  const int64_t rows = static_cast<int64_t>(nb) * 128;
  if (i >= rows * kb) return;
  const int64_t n = i / kb, k = i % kb;
  uint8_t* c = canon + (n / 128) * kb + k;
  if (pack) sf[sf_offset(n, k, ka)] = *c;
  else if (n % 128 == 0) *c = sf[sf_offset(n, k, ka)];
}

// Canonical activation scales [M, cdiv(K, 128)] <-> atoms.
__global__ void k_act_scales(uint8_t* canon, int kb, int64_t count, uint8_t* sf, int64_t ka, bool pack) {
  const int64_t i = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x;
  if (i >= count) return;
  uint8_t* s = sf + sf_offset(i / kb, i % kb, ka);
  if (pack) *s = canon[i];
  else canon[i] = *s;
}

// The values that codes stand for: 8 per thread.
template <bool BF16>
__global__ void __launch_bounds__(256) k_act_values(const uint8_t* __restrict__ codes, const uint8_t* __restrict__ sf,
                                                    int K, int64_t chunks, int64_t ka, void* __restrict__ out) {
  grid_dep_wait();
  const int64_t i = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x;
  if (i >= chunks) return;
  const int per = K / 8;
  const int64_t row = i / per;
  const int ch = static_cast<int>(i - row * per);
  const uint2 c = *reinterpret_cast<const uint2*>(codes + i * 8);
  const float s = scale_value(sf[sf_offset(row, ch >> 4, ka)]);
  const uint32_t w[2] = {c.x, c.y};
  float v[8];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    uint32_t h2;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h2) : "h"(static_cast<uint16_t>(w[j >> 1] >> (16 * (j & 1)))));
    const __half2 hh = *reinterpret_cast<const __half2*>(&h2);
    v[2 * j] = __low2float(hh) * s;
    v[2 * j + 1] = __high2float(hh) * s;
  }
  if (BF16) {
    uint32_t o[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const __nv_bfloat162 b = __floats2bfloat162_rn(v[2 * j], v[2 * j + 1]);
      o[j] = *reinterpret_cast<const uint32_t*>(&b);
    }
    reinterpret_cast<uint4*>(out)[i] = make_uint4(o[0], o[1], o[2], o[3]);
  } else {
    reinterpret_cast<float4*>(out)[2 * i] = make_float4(v[0], v[1], v[2], v[3]);
    reinterpret_cast<float4*>(out)[2 * i + 1] = make_float4(v[4], v[5], v[6], v[7]);
  }
}

}  // namespace

cudaError_t launch_rows(const NormParams& p, bool norm, int res_kind, cudaStream_t st) {
  const int nch = p.K / 8;
  if (!norm) {
    const int T = nch >= 256 ? 256 : static_cast<int>(align_up(nch, 32));
    return launch_rows_c<1, false>(p, 0, dim3(p.M, static_cast<unsigned>(cdiv(nch, T))), T, st);
  }
  int C = 1;
  while (C < 8 && nch > 512 * C) C *= 2;
  const int T = static_cast<int>(align_up(cdiv(nch, C), 32));
  const dim3 grid(p.M);
  switch (C) {
    case 1: return launch_rows_c<1, true>(p, res_kind, grid, T, st);
    case 2: return launch_rows_c<2, true>(p, res_kind, grid, T, st);
    case 4: return launch_rows_c<4, true>(p, res_kind, grid, T, st);
    default: return launch_rows_c<8, true>(p, res_kind, grid, T, st);
  }
}

cudaError_t launch_weight_quant(const void* W, int K, int N, uint8_t* codes, uint8_t* sf, cudaStream_t st) {
  const dim3 grid(static_cast<unsigned>(cdiv(K, 128)), static_cast<unsigned>(cdiv(N, 128)));
  k_weight_quant<<<grid, 256, 0, st>>>(static_cast<const uint16_t*>(W), K, N, codes, sf, katoms(K));
  return cudaGetLastError();
}

cudaError_t launch_weight_scales(uint8_t* canonical, int K, int N, uint8_t* sf, bool pack, cudaStream_t st) {
  const int kb = static_cast<int>(cdiv(K, 128)), nb = static_cast<int>(cdiv(N, 128));
  const int64_t n = static_cast<int64_t>(nb) * 128 * kb;
  k_weight_scales<<<static_cast<unsigned>(cdiv(n, 256)), 256, 0, st>>>(canonical, kb, nb, sf, katoms(K), pack);
  return cudaGetLastError();
}

cudaError_t launch_act_scales(uint8_t* canonical, int K, int M, uint8_t* sf, bool pack, cudaStream_t st) {
  const int kb = static_cast<int>(cdiv(K, 128));
  const int64_t n = static_cast<int64_t>(M) * kb;
  k_act_scales<<<static_cast<unsigned>(cdiv(n, 256)), 256, 0, st>>>(canonical, kb, n, sf, katoms(K), pack);
  return cudaGetLastError();
}

cudaError_t launch_act_values(const uint8_t* codes, const uint8_t* sf, int K, int M, void* values, bool bf16,
                              cudaStream_t st) {
  const int64_t chunks = static_cast<int64_t>(M) * (K / 8);
  const unsigned grid = static_cast<unsigned>(cdiv(chunks, 256));
  if (bf16) k_act_values<true><<<grid, 256, 0, st>>>(codes, sf, K, chunks, katoms(K), values);
  else k_act_values<false><<<grid, 256, 0, st>>>(codes, sf, K, chunks, katoms(K), values);
  return cudaGetLastError();
}

}  // namespace fp8
}  // namespace kq
