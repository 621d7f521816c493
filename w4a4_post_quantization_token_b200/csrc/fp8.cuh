// The 8-bit operators: layouts of their buffers, encoding, kernel parameter blocks and
// launcher prototypes.
//
// An 8-bit block is up to 128 consecutive features of one token (activations) or a
// 128 x 128 piece of a weight: E4M3 codes and one scale 2^e (E8M0 byte e + 127). e is the
// smallest exponent >= -127 for which no value exceeds 448 * 2^e, so nothing saturates;
// byte 0 for a block of zeros. A block that holds an infinity or NaN gets byte 0xFF and NaN
// codes: whatever is computed from it is NaN.
//
// Codes are row-major with the contraction dimension contiguous (what TMA loads as a K-major
// MMA operand). Scale bytes are stored in the same 512-byte atoms as the MXFP4 scales
// (layout.cuh: 128 rows x 4 blocks), but a block is 128 elements here: one atom serves four
// 128-element k-tiles, k-tile t by byte t % 4.
#pragma once
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "layout.cuh"
#include "sm100.cuh"

namespace kq {
namespace fp8 {

constexpr int kBlk = 128;                    // elements per scale along K; bytes per k-tile row
constexpr int kNormMaxK = 32768;             // the norm keeps a row in registers
// Features of a layer, in or out: grids and 32-bit indices hold them, and a product over so many
// inputs (2^21 k-tiles, 0.3 us each) ends well within the 2 s that its epilogue waits.
constexpr int kMaxWidth = 1 << 28;

__host__ __device__ constexpr int64_t katoms(int64_t K) { return cdiv(K, 4 * kBlk); }

struct WLayout {
  size_t codes[2] = {0, 0};                  // uint8 [N, K], gate (or the only one) and up
  size_t sf[2] = {0, 0};                     // scale atoms, rows padded to 128
  size_t total = 0;
  __host__ __device__ static WLayout make(int64_t K, int64_t N, bool gated) {
    WLayout L;
    size_t o = 0;
    for (int i = 0; i < (gated ? 2 : 1); ++i) {
      L.codes[i] = o; o = align_up(o + static_cast<size_t>(N) * K, kAlign);
      L.sf[i] = o;    o = align_up(o + static_cast<size_t>(cdiv(N, 128)) * katoms(K) * 512u, kAlign);
    }
    L.total = o;
    return L;
  }
};

struct ALayout {
  size_t err = 0;                            // uint32 device error word
  size_t codes = 0;                          // uint8 [M, K]
  size_t sf = 0;                             // scale atoms, rows padded to 128
  size_t total = 0;
  __host__ __device__ static ALayout make(int64_t M, int64_t K) {
    ALayout L;
    size_t o = kHdrBytes;
    L.codes = o = align_up(o, kAlign);
    o = align_up(o + static_cast<size_t>(M) * K, kAlign);
    L.sf = o;
    L.total = align_up(o + static_cast<size_t>(cdiv(M, 128)) * katoms(K) * 512u, kAlign);
    return L;
  }
};

// ------------------------------------------------------------------------- encoding -----
// Scale byte of a block whose largest magnitude has the bits `amax` (sign cleared). 448 is
// 1.75 * 2^8: with amax = m 2^p, 1 <= m < 2, the exponent is p - 8, or p - 7 when m > 1.75,
// read off the bits: adding 2^21 - 1 carries into the exponent exactly when the mantissa field
// exceeds that of 1.75.
__device__ __forceinline__ uint32_t scale_byte(uint32_t amax) {
  if (amax >= 0x7F800000u) return 0xFFu;
  const int32_t p = static_cast<int32_t>((amax + 0x1FFFFFu) >> 23) - 8;   // biased: e + 127
  return static_cast<uint32_t>(p < 0 ? 0 : p);
}
// 2^-e of a scale byte e + 127 <= 247 as fp32 (exact: 2^-120 .. 2^127); the quotient of a
// value by its scale is then exact or, below E4M3's smallest step, rounded far under it.
__device__ __forceinline__ float inv_scale(uint32_t byte) {
  return byte == 0xFFu ? __uint_as_float(0x7FC00000u) : __uint_as_float((254u - byte) << 23);
}
__device__ __forceinline__ float scale_value(uint32_t byte) {
  return byte == 0xFFu ? __uint_as_float(0x7FC00000u)
                       : (byte == 0u ? __uint_as_float(0x00400000u) : __uint_as_float(byte << 23));
}
// Two values -> two E4M3 codes (round to nearest even; NaN -> 0x7F), lo in the low byte.
__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d) {
  return e4m3x2(a, b) | (e4m3x2(c, d) << 16);
}
__device__ __forceinline__ uint32_t abs_bits(float v) { return __float_as_uint(v) & 0x7FFFFFFFu; }

// 8 bf16 values of 16 bytes.
__device__ __forceinline__ void unpack8(const uint4& u, float (&v)[8]) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(w[i] << 16);
    v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
}
// The scale byte of a block that 16 neighbouring lanes hold, 8 values each.
__device__ __forceinline__ uint32_t block_byte(const float (&v)[8]) {
  uint32_t a = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) a = max(a, abs_bits(v[i]));
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) a = max(a, __shfl_xor_sync(0xffffffffu, a, o));
  return scale_byte(a);
}

// SiLU g / (1 + e^-g), from e^-|g|, which cannot overflow; GELU in its erf form,
// g erfc(-g / sqrt 2) / 2. F32: for fp32 outputs the exponential is the full-precision one. The
// approximate one rounds g log2 e first, so it is 2^-18 off at a gate of -60, which is nothing beside
// the rounding to bf16 or E4M3; everywhere it cost 4096 x 256 -> 4096 in bf16 a sixth (32 -> 38 us).
// The quotient, with a divisor of 1 to 2, is within 2 ulps and has no branch (the exact one has,
// which keeps a thread's values from overlapping: 300 x 1152 -> 4608 in fp32 11 -> 24 us).
template <int ACT, bool F32>
__device__ __forceinline__ float gate_act(float g) {
  if (ACT == 0) {
    const float e = F32 ? expf(-fabsf(g)) : __expf(-fabsf(g));
    return __fdividef(g < 0.f ? g * e : g, 1.f + e);
  }
  return 0.5f * g * erfcf(-0.70710678118654752f * g);
}
// v[i] = act(g[i]) u[i] of N outputs of type `out` (MmParams).
template <int ACT, int N>
__device__ __forceinline__ void gate(int out, const float* g, const float* u, float* v) {
  if (ACT == 0 && out == 0) {
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = gate_act<ACT, true>(g[i]) * u[i];
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = gate_act<ACT, false>(g[i]) * u[i];
  }
}

// --------------------------------------------------------------------- parameter blocks --
struct NormParams {
  const void* x;              // bf16 [M, ldx]
  int64_t ldx;
  void* residual;             // bf16 or fp32 [M, ldr], read and rewritten; null: none
  int64_t ldr;
  const float* gamma;         // [K]
  double eps;
  int M, K;
  int64_t katoms;
  uint8_t* codes;
  uint8_t* sf;
  uint32_t* err;              // cleared
};

struct MmParams {
  CUtensorMap tmap_w[2];      // weight codes [N, K] (gate / only, up), box 128 bytes x (64, 96 or 128) rows
  CUtensorMap tmap_x;         // activation codes [M, K], box 128 bytes x token tile (128 for k_mm_pair)
  CUtensorMap tmap_sfw[2];    // pairs: weight and activation scale atoms as [atoms, 512 bytes]
  CUtensorMap tmap_sfx;
  const uint8_t* sfw[2];      // weight scale atoms
  const uint8_t* sfx;         // activation scale atoms
  const void* xb;             // encoded on the way in: bf16 [M, ldx] instead of tmap_x and sfx
  int64_t ldx;
  int M, N, K;
  int64_t katoms;             // of K
  int act;                    // gated: 0 SiLU, 1 GELU
  int out;                    // 0 fp32, 1 bf16, 2 8-bit blocks
  void* y;                    // [M, ldy] fp32 / bf16
  int64_t ldy;
  uint8_t* ocodes;            // 8-bit output: codes [M, N], scale atoms, its katoms and error
  uint8_t* osf;               //   word (cleared)
  int64_t okatoms;
  uint32_t* oerr;
  int pairs;                  // weight rows of k_mm_pair's tile, 0: k_rows_mm
  int splits;                 // k_mm_pair: pairs that share K
  int dependent;              // launched as a programmatic dependent of the kernel that writes
                              //   the activations, whose predecessors had ended
  uint32_t* err;
  uint64_t wait_ns;           // limit of each wait on a barrier
  int withhold;               // >= 0: this k-tile of a CTA's weights is not loaded (a wait runs out)
};

cudaError_t launch_rows(const NormParams& p, bool norm, int res_kind, cudaStream_t st);
cudaError_t launch_weight_quant(const void* W, int K, int N, uint8_t* codes, uint8_t* sf, cudaStream_t st);
cudaError_t launch_weight_scales(uint8_t* canonical, int K, int N, uint8_t* sf, bool pack, cudaStream_t st);
cudaError_t launch_act_scales(uint8_t* canonical, int K, int M, uint8_t* sf, bool pack, cudaStream_t st);
// values: fp32 or bf16 [M, K]
cudaError_t launch_act_values(const uint8_t* codes, const uint8_t* sf, int K, int M, void* values, bool bf16,
                              cudaStream_t st);
struct Device { int sms, device; };

// As the tensor core accumulates in fp32, the error of a sum grows in proportion to its length, as
// one-sided roundings do: 2.7e-7 of the result (relative norm) for 4096 inputs, 1.1e-6 for 12288, of a
// gated output 5.2e-7 and 2.2e-6, where additions that round to nearest are 2e-7 and 3e-7 off at 12288.
// For fp32 outputs (bf16 and E4M3 round off 1e3 times as much) the products therefore accumulate this
// many k-tiles at a time, 8192 inputs or 4096 gated, and the epilogue adds the pieces in registers: 7e-7
// at most for any K. 4096 x 12288 -> 4096 takes 174 us instead of 172, gated 321 instead of 308.
__host__ __device__ constexpr int sum_tiles(bool gated) { return gated ? 32 : 64; }

constexpr int kRowsMaxM = 64;                // tokens that k_rows_mm takes; more go to k_mm_pair
constexpr int kMaxDevices = 64;              // whose cluster limits are kept
// Weight rows of k_mm_pair's tile, 0 where k_rows_mm is taken, and the pairs that share K. The box
// height of MmParams::tmap_w is half of the rows (128 for k_rows_mm).
struct PairShape { int cols, splits; };
PairShape pair_shape(int M, int N, int K, bool gated, const Device& d);
cudaError_t launch_pair(const MmParams& p, bool gated, int sms, cudaStream_t st);
// token tile of k_rows_mm (the box height of MmParams::tmap_x; 128 for k_mm_pair)
int rows_token_tile(int M);
cudaError_t launch_rows_mm(const MmParams& p, bool gated, const Device& d, cudaStream_t st);
// k_rows_mm on bf16 activations (p.xb), which it encodes itself; false where it does not take them
bool try_rows_fused(const MmParams& p, bool gated, const Device& d, cudaStream_t st, cudaError_t* e);

}  // namespace fp8
}  // namespace kq
