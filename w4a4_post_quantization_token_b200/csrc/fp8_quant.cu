// Row kernels of the 8-bit operators: the root-mean-square norm (with the residual's addition)
// and the plain quantizer write E4M3 codes with a power-of-two scale for each token and 128
// features; the weight quantizer does the same for 128 x 128 pieces; the rest convert layouts.
#include <cuda_fp16.h>

#include "fp8.cuh"

namespace kq {
namespace fp8 {

namespace {

// Encodes the 8 values that each thread holds of a block shared by 16 neighbouring lanes (lanes
// without a chunk of the row hold zeros).
__device__ __forceinline__ void encode8(const float (&v)[8], bool valid, int row, int chunk, const NormParams& p) {
  const uint32_t byte = block_byte(v);
  const float is = inv_scale(byte);
  if (!valid) return;
  uint2 c;
  c.x = e4m3x4(v[0] * is, v[1] * is, v[2] * is, v[3] * is);
  c.y = e4m3x4(v[4] * is, v[5] * is, v[6] * is, v[7] * is);
  *reinterpret_cast<uint2*>(p.codes + static_cast<size_t>(row) * p.K + chunk * 8) = c;
  if ((chunk & 15) == 0) p.sf[sf_offset(row, chunk >> 4, p.katoms)] = static_cast<uint8_t>(byte);
}

// Every row kernel starts behind the kernel before it, and lets the next one start only then: a
// kernel that was started early thus knows that all but its direct predecessor have ended.
__device__ __forceinline__ void enter(const NormParams& p) {
  grid_dep_wait();
  grid_dep_launch();
  if (blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0 && threadIdx.y == 0) *p.err = 0u;
}

// 32 bytes as one access where the caller's rows allow it (a warp's 16-byte accesses 32 bytes apart
// would fetch each sector twice), else as two.
__device__ __forceinline__ void load32(const void* p, bool wide, uint32_t (&u)[8]) {
  if (wide) {
    asm volatile("ld.global.v8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=r"(u[0]), "=r"(u[1]), "=r"(u[2]), "=r"(u[3]), "=r"(u[4]), "=r"(u[5]), "=r"(u[6]), "=r"(u[7])
                 : "l"(p) : "memory");
  } else {
    const uint4 a = static_cast<const uint4*>(p)[0], b = static_cast<const uint4*>(p)[1];
    u[0] = a.x; u[1] = a.y; u[2] = a.z; u[3] = a.w;
    u[4] = b.x; u[5] = b.y; u[6] = b.z; u[7] = b.w;
  }
}
__device__ __forceinline__ void store32(void* p, bool wide, const uint32_t* u) {
  if (wide) {
    asm volatile("st.global.v8.b32 [%8], {%0,%1,%2,%3,%4,%5,%6,%7};"
                 ::"r"(u[0]), "r"(u[1]), "r"(u[2]), "r"(u[3]), "r"(u[4]), "r"(u[5]), "r"(u[6]), "r"(u[7]), "l"(p)
                 : "memory");
  } else {
    static_cast<uint4*>(p)[0] = make_uint4(u[0], u[1], u[2], u[3]);
    static_cast<uint4*>(p)[1] = make_uint4(u[4], u[5], u[6], u[7]);
  }
}

// The plain quantizer: kRowsC chunks of 16 features (32 bytes) per thread, loaded together; 8
// neighbouring threads share a scale; blockDim.x threads along a row, blockDim.y rows. Bound by HBM:
// 3 bytes a feature, 8192 x 8192 in 31.6 us (6.4 TB/s, the copy rate; with 16-byte accesses
// 40 us). Few tokens cost one load latency and a launch, 1.8 us for 1 x 4096.
constexpr int kRowsC = 4;
__global__ void __launch_bounds__(256) k_quant(const __grid_constant__ NormParams p, bool wide) {
  enter(p);
  const int64_t row = static_cast<int64_t>(blockIdx.x) * blockDim.y + threadIdx.y;
  const int nch = row < p.M ? p.K / 16 : 0;
  const int first = blockIdx.y * (kRowsC * blockDim.x) + threadIdx.x;
  const __nv_bfloat16* x = static_cast<const __nv_bfloat16*>(p.x) + row * p.ldx;
  uint32_t u[kRowsC][8];
#pragma unroll
  for (int c = 0; c < kRowsC; ++c) {
    const int ch = first + c * static_cast<int>(blockDim.x);
#pragma unroll
    for (int i = 0; i < 8; ++i) u[c][i] = 0;
    if (ch < nch) load32(x + 16 * ch, wide, u[c]);
  }
#pragma unroll
  for (int c = 0; c < kRowsC; ++c) {
    const int ch = first + c * static_cast<int>(blockDim.x);
    float v[16];
    uint32_t a = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      v[2 * i] = __uint_as_float(u[c][i] << 16);
      v[2 * i + 1] = __uint_as_float(u[c][i] & 0xFFFF0000u);
      a = max(a, max(abs_bits(v[2 * i]), abs_bits(v[2 * i + 1])));
    }
#pragma unroll
    for (int o = 4; o > 0; o >>= 1) a = max(a, __shfl_xor_sync(0xffffffffu, a, o));
    const uint32_t byte = scale_byte(a);
    const float is = inv_scale(byte);
    if (ch >= nch) continue;
    uint4 o;
    o.x = e4m3x4(v[0] * is, v[1] * is, v[2] * is, v[3] * is);
    o.y = e4m3x4(v[4] * is, v[5] * is, v[6] * is, v[7] * is);
    o.z = e4m3x4(v[8] * is, v[9] * is, v[10] * is, v[11] * is);
    o.w = e4m3x4(v[12] * is, v[13] * is, v[14] * is, v[15] * is);
    *reinterpret_cast<uint4*>(p.codes + row * p.K + 16 * ch) = o;
    if ((ch & 7) == 0) p.sf[sf_offset(row, ch >> 3, p.katoms)] = static_cast<uint8_t>(byte);
  }
}

// The norm: one CTA per token, C chunks of 8 features per thread, all loads before the first
// store; 16 neighbouring threads share a scale.
//   h = x + residual in fp32, rounded to the residual's type and kept there;
//   r = 1 / sqrt(mean(h^2) + eps), the sum and the root in float64, rounded once to fp32;
//   y = (h r) gamma, two fp32 products; then the block's scale and codes from y.
// The float64 sum is within some K 2^-53 of the exact one in any order, so that another order gives
// another r only where the root lies that close to a border between two fp32 values (a chance of K 2^-28
// a row at most). Bound by HBM: the row stays in registers between the sum and the codes, so that x and the residual are read once:
// 8192 x 8192 with a bf16 residual in 72.7 us (7 bytes a feature, 6.46 TB/s, the copy rate; 106 us
// when a chunk's residual was stored before the next chunk's load), 1 x 4096 in 2.4 us.
template <int C, int RES>
__global__ void __launch_bounds__(512) k_norm(const __grid_constant__ NormParams p) {
  __shared__ double part[16];
  enter(p);
  const int64_t row = blockIdx.x;
  const int T = blockDim.x, nch = p.K / 8;
  const uint4* x = reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(p.x) + row * p.ldx);
  uint4* rb = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p.residual) + row * p.ldr);
  float4* rf = reinterpret_cast<float4*>(static_cast<float*>(p.residual) + row * p.ldr);
  uint4 u[C], r1[RES == 1 ? C : 1];
  float h[C][8];
#pragma unroll
  for (int c = 0; c < C; ++c) {
    const int ch = threadIdx.x + c * T;
    const bool valid = ch < nch;
    u[c] = valid ? x[ch] : make_uint4(0, 0, 0, 0);
    if (RES == 1) r1[c] = valid ? rb[ch] : make_uint4(0, 0, 0, 0);
    if (RES == 2) {
      const float4 z = make_float4(0.f, 0.f, 0.f, 0.f);
      const float4 r0 = valid ? rf[2 * ch] : z, r2 = valid ? rf[2 * ch + 1] : z;
      h[c][0] = r0.x; h[c][1] = r0.y; h[c][2] = r0.z; h[c][3] = r0.w;
      h[c][4] = r2.x; h[c][5] = r2.y; h[c][6] = r2.z; h[c][7] = r2.w;
    }
  }
  double sum = 0.0;
#pragma unroll
  for (int c = 0; c < C; ++c) {
    const int ch = threadIdx.x + c * T;
    const bool valid = ch < nch;
    float v[8];
    unpack8(u[c], v);
    if (RES == 0) {
#pragma unroll
      for (int i = 0; i < 8; ++i) h[c][i] = v[i];
    }
    if (RES == 1) {
      float r[8];
      unpack8(r1[c], r);
      uint32_t o[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const __nv_bfloat162 b = __floats2bfloat162_rn(v[2 * i] + r[2 * i], v[2 * i + 1] + r[2 * i + 1]);
        o[i] = *reinterpret_cast<const uint32_t*>(&b);
      }
      const uint4 ov = make_uint4(o[0], o[1], o[2], o[3]);
      if (valid) rb[ch] = ov;
      unpack8(ov, h[c]);
    }
    if (RES == 2) {
#pragma unroll
      for (int i = 0; i < 8; ++i) h[c][i] = v[i] + h[c][i];
      if (valid) {
        rf[2 * ch] = make_float4(h[c][0], h[c][1], h[c][2], h[c][3]);
        rf[2 * ch + 1] = make_float4(h[c][4], h[c][5], h[c][6], h[c][7]);
      }
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) sum = fma(static_cast<double>(h[c][i]), static_cast<double>(h[c][i]), sum);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = sum;
  __syncthreads();
  double total = 0.0;
  for (int w = 0; w < (T >> 5); ++w) total += part[w];
  const float r = static_cast<float>(1.0 / sqrt(total / static_cast<double>(p.K) + p.eps));
#pragma unroll
  for (int c = 0; c < C; ++c) {
    const int ch = threadIdx.x + c * T;
    const bool valid = ch < nch;
    if (valid) {
      const float4* g = reinterpret_cast<const float4*>(p.gamma) + 2 * ch;
      const float4 g0 = g[0], g1 = g[1];
      h[c][0] = h[c][0] * r * g0.x; h[c][1] = h[c][1] * r * g0.y;
      h[c][2] = h[c][2] * r * g0.z; h[c][3] = h[c][3] * r * g0.w;
      h[c][4] = h[c][4] * r * g1.x; h[c][5] = h[c][5] * r * g1.y;
      h[c][6] = h[c][6] * r * g1.z; h[c][7] = h[c][7] * r * g1.w;
    }
    encode8(h[c], valid, static_cast<int>(row), ch, p);
  }
}

// All of these kernels wait for the kernel before them (griddepcontrol.wait) ahead of their
// first access, so that their start may overlap its end.
template <typename... A>
cudaError_t launch_behind(void (*fn)(A...), dim3 grid, dim3 block, cudaStream_t st, A... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, fn, args...);
}

template <int C>
cudaError_t launch_norm_c(const NormParams& p, int res_kind, dim3 grid, int T, cudaStream_t st) {
  return launch_behind(res_kind == 0 ? k_norm<C, 0> : res_kind == 1 ? k_norm<C, 1> : k_norm<C, 2>, grid, dim3(T), st, p);
}

// One CTA per 128 (outputs) x 128 (inputs) piece of W [K, N]: transposed to K-major codes. (The pieces
// are one grid dimension: a second one ends at 65535.)
__global__ void __launch_bounds__(256) k_weight_quant(const uint16_t* __restrict__ W, int K, int N,
                                                      uint8_t* __restrict__ codes, uint8_t* __restrict__ sf,
                                                      int64_t ka) {
  __shared__ uint16_t tile[128][130];                     // [k][n]
  __shared__ uint32_t top[8];
  const uint32_t kb = static_cast<uint32_t>(cdiv(K, 128)), bk = blockIdx.x % kb;
  const int k0 = static_cast<int>(bk) * 128, n0 = static_cast<int>(blockIdx.x / kb) * 128;
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
  if (threadIdx.x < 128) sf[sf_offset(n0 + threadIdx.x, bk, ka)] = static_cast<uint8_t>(byte);
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

// The values that codes stand for: two chunks of 32 codes per thread (K is a multiple of 32, so a
// chunk lies in one block), both loaded first. `wide`: 32-byte accesses to the codes (1), the
// values (2). Bound by HBM: 8192 x 8192 to bf16 in 31.2 us (6.45 TB/s).
template <bool BF16>
__global__ void __launch_bounds__(256) k_act_values(const uint8_t* codes, const uint8_t* sf, int K, int64_t chunks,
                                                    int64_t ka, uint8_t* out, int wide) {
  grid_dep_wait();
  grid_dep_launch();
  const uint32_t per = static_cast<uint32_t>(K) / 32;
  int64_t at[2];
  uint32_t c[2][8];
  float s[2];
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const int64_t i = at[k] = (static_cast<int64_t>(blockIdx.x) * 2 + k) * 256 + threadIdx.x;
    if (i >= chunks) continue;
    const int64_t row = chunks <= 0xFFFFFFFFll ? static_cast<int64_t>(static_cast<uint32_t>(i) / per) : i / per;
    load32(codes + i * 32, wide & 1, c[k]);
    s[k] = scale_value(sf[sf_offset(row, (i - row * per) >> 2, ka)]);
  }
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    if (at[k] >= chunks) continue;
    uint32_t o[BF16 ? 16 : 32];
#pragma unroll
    for (int j = 0; j < 16; ++j) {
      uint32_t h2;
      asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h2) : "h"(static_cast<uint16_t>(c[k][j >> 1] >> (16 * (j & 1)))));
      const __half2 hh = *reinterpret_cast<const __half2*>(&h2);
      const float lo = __low2float(hh) * s[k], hi = __high2float(hh) * s[k];
      if (BF16) {
        const __nv_bfloat162 b = __floats2bfloat162_rn(lo, hi);
        o[j] = *reinterpret_cast<const uint32_t*>(&b);
      } else {
        o[2 * j] = __float_as_uint(lo);
        o[2 * j + 1] = __float_as_uint(hi);
      }
    }
#pragma unroll
    for (int j = 0; j < (BF16 ? 2 : 4); ++j) store32(out + (at[k] * (BF16 ? 2 : 4) + j) * 32, wide & 2, o + 8 * j);
  }
}

}  // namespace

cudaError_t launch_rows(const NormParams& p, bool norm, int res_kind, cudaStream_t st) {
  const int nch = p.K / 8;
  if (!norm) {
    const int per = static_cast<int>(align_up(p.K / 16, 8));             // whole blocks
    const int want = static_cast<int>(align_up(cdiv(per, kRowsC), 16));
    const int tx = want < 128 ? want : 128;
    const int ty = 256 / tx - (256 / tx * tx % 32 ? 1 : 0);              // whole warps
    const dim3 grid(static_cast<unsigned>(cdiv(p.M, ty)), static_cast<unsigned>(cdiv(per, kRowsC * tx)));
    const bool wide = (reinterpret_cast<uintptr_t>(p.x) | static_cast<uintptr_t>(p.ldx * 2)) % 32 == 0;
    return launch_behind(k_quant, grid, dim3(tx, ty), st, p, wide);
  }
  int C = 1;
  while (C < 8 && nch > 256 * C) C *= 2;
  const int T = static_cast<int>(align_up(cdiv(nch, C), 32));
  const dim3 grid(p.M);
  switch (C) {
    case 1: return launch_norm_c<1>(p, res_kind, grid, T, st);
    case 2: return launch_norm_c<2>(p, res_kind, grid, T, st);
    case 4: return launch_norm_c<4>(p, res_kind, grid, T, st);
    default: return launch_norm_c<8>(p, res_kind, grid, T, st);
  }
}

cudaError_t launch_weight_quant(const void* W, int K, int N, uint8_t* codes, uint8_t* sf, cudaStream_t st) {
  k_weight_quant<<<static_cast<unsigned>(cdiv(K, 128) * cdiv(N, 128)), 256, 0, st>>>(static_cast<const uint16_t*>(W), K, N, codes, sf, katoms(K));
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
  const int64_t chunks = static_cast<int64_t>(M) * (K / 32);
  const int wide = (reinterpret_cast<uintptr_t>(codes) % 32 == 0 ? 1 : 0) | (reinterpret_cast<uintptr_t>(values) % 32 == 0 ? 2 : 0);
  return launch_behind(bf16 ? k_act_values<true> : k_act_values<false>, dim3(static_cast<unsigned>(cdiv(chunks, 512))),
                       dim3(256), st, codes, sf, K, chunks, katoms(K), static_cast<uint8_t*>(values), wide);
}

}  // namespace fp8
}  // namespace kq
