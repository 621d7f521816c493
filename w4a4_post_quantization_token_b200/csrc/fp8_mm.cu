// Block-scaled 8-bit matrix product on the 5th-generation tensor cores:
//
//   Y[m, n] = sum_kb 2^(ex[m, kb] + ew[n / 128, kb]) sum_{k in kb} cx[m, k] cw[n, k]
//
// (tcgen05 kind::mxf8f6f4 with E8M0 scales: the tensor core applies both powers of two as it
// accumulates in fp32), and its gated form  H = act(X Wg) * (X Wu)  with both products, the
// activation and the product in one kernel.
//
// k_mm_rows: one CTA per 128 outputs x BT tokens. The weights are the MMA's 128-row operand and
// the tokens its BT columns, so a few tokens cost a few columns. Warp roles:
//   warp 0    TMA producer (one thread): weight and activation k-tiles of 128 bytes per row
//             (128-byte swizzle) into a ring; with the first k-tile of each 512-byte scale atom
//             (4 k-tiles) the atoms themselves.
//   warp 1    TMEM allocator and MMA issuer (one thread): scale atoms to TMEM, 4 MMAs (K = 32)
//             per k-tile and product, a commit that frees the stage.
//   warps 2-5 epilogue: thread = output feature; a warp writes 32 neighbouring features of one
//             token at a time.
#include <cuda_bf16.h>

#include "fp8.cuh"
#include "sm100_fp8.cuh"

namespace kq {
namespace fp8 {

namespace {

constexpr int kThreads = 192;

template <int BT, bool GATED>
struct Rows {
  static constexpr int kProducts = GATED ? 2 : 1;
  static constexpr uint32_t kABytes = 128 * 128;
  static constexpr uint32_t kBBytes = BT * 128;
  static constexpr uint32_t kSfOff = kProducts * kABytes + kBBytes;       // 3 x 512 bytes reserved
  static constexpr uint32_t kStageBytes = kSfOff + 2048;
  // two CTAs share an SM, so that one's epilogue and start-up overlap the other's loads
  static constexpr int kStages = (110 * 1024 - 2048) / kStageBytes;
  static constexpr uint32_t kSmem = 1024 + 1024 + kStages * kStageBytes;  // alignment, barriers
  // accumulators 64 columns apart at least, then 2 scale sets of 16 columns
  static constexpr uint32_t kAccCols = BT < 64 ? 64 : BT;
  static constexpr uint32_t kSfCol = kProducts * kAccCols;
  static constexpr uint32_t kTmemCols = kSfCol + 32 <= 128 ? 128 : (kSfCol + 32 <= 256 ? 256 : 512);
  static_assert(kStages >= 2 && kStageBytes % 1024 == 0, "ring");
};

__device__ __forceinline__ float gate_act(float g, int act) {
  // SiLU g / (1 + e^-g); GELU in its erf form, g erfc(-g / sqrt 2) / 2
  if (act == 0) return __fdividef(g, 1.f + __expf(-g));
  return 0.5f * g * erfcf(-0.70710678118654752f * g);
}

template <int BT, bool GATED>
__global__ void __launch_bounds__(kThreads) k_mm_rows(const __grid_constant__ MmParams p) {
  using C = Rows<BT, GATED>;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(align_up(reinterpret_cast<uintptr_t>(smem_raw), 1024));
  uint64_t* full = reinterpret_cast<uint64_t*>(smem);
  uint64_t* empty = full + C::kStages;
  uint64_t* acc_full = empty + C::kStages;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(acc_full + 1);
  uint32_t* top = reinterpret_cast<uint32_t*>(smem + 512);               // [4 warps][16 tokens]
  uint8_t* ring = smem + 1024;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int n0 = blockIdx.x * 128, t0 = blockIdx.y * BT;
  const int KT = static_cast<int>(cdiv(p.K, kBlk));

  if (threadIdx.x == 0) {
    for (int s = 0; s < C::kStages; ++s) { mbar_init(&full[s], 1); mbar_init(&empty[s], 1); }
    mbar_init(acc_full, 1);
    fence_mbar_init();
    prefetch_tmap(&p.tmap_w[0]);
    if (GATED) prefetch_tmap(&p.tmap_w[1]);
    prefetch_tmap(&p.tmap_x);
  }
  if (warp == 1) { tmem_alloc(tmem_slot, C::kTmemCols); tmem_relinquish(); }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  if (warp == 0) {
    if (lane == 0) {
      grid_dep_wait();
      grid_dep_launch();
      const size_t wrow = static_cast<size_t>(blockIdx.x) * p.katoms * 512u;
      const size_t xrow = static_cast<size_t>(t0 / 128) * p.katoms * 512u;
      int kt = 0;
      bool ok = true;
      for (; kt < KT; ++kt) {
        const int s = kt % C::kStages;
        if (kt >= C::kStages && !mbar_wait(&empty[s], ((kt / C::kStages) - 1) & 1, p.err, KQ_DEV_ERR_TIMEOUT_EMPTY)) {
          ok = false;
          break;
        }
        uint8_t* st = ring + s * C::kStageBytes;
        uint8_t* sf = st + C::kSfOff;
        const bool atom = (kt & 3) == 0;
        mbar_arrive_expect_tx(&full[s], C::kSfOff + (atom ? (C::kProducts + 1) * 512u : 0u));
        for (int i = 0; i < C::kProducts; ++i)
          tma_load_2d(st + i * C::kABytes, &p.tmap_w[i], kt * kBlk, n0, &full[s]);
        tma_load_2d(st + C::kProducts * C::kABytes, &p.tmap_x, kt * kBlk, t0, &full[s]);
        if (atom) {
          const size_t ko = static_cast<size_t>(kt >> 2) * 512u;
          for (int i = 0; i < C::kProducts; ++i) bulk_load(sf + i * 512, p.sfw[i] + wrow + ko, 512, &full[s]);
          bulk_load(sf + C::kProducts * 512, p.sfx + xrow + ko, 512, &full[s]);
        }
      }
      if (!ok) drain_ring(full, C::kStages, kt);
    }
  } else if (warp == 1) {
    if (lane == 0) {
      const uint32_t ring_addr = smem_u32(ring);
      for (int kt = 0; kt < KT; ++kt) {
        const int s = kt % C::kStages;
        if (!mbar_wait(&full[s], (kt / C::kStages) & 1, p.err, KQ_DEV_ERR_TIMEOUT_FULL)) break;
        tc_fence_after();
        const uint32_t st = ring_addr + s * C::kStageBytes;
        // scale sets alternate per atom; copies and MMAs of one thread run in issue order
        const uint32_t set = tmem + C::kSfCol + static_cast<uint32_t>((kt >> 2) & 1) * 16u;
        if ((kt & 3) == 0) {
          for (int i = 0; i <= C::kProducts; ++i)
            tmem_cp_32x128b_warpx4(set + 4 * i, sdesc_plain_rows16(st + C::kSfOff + i * 512));
        }
        const uint32_t id = static_cast<uint32_t>(kt) & 3u;
        const uint32_t idesc = idesc_mxf8(128, BT, 0) | (id << 4) | (id << 29);
        const uint64_t bd = sdesc_sw128_kmajor(st + C::kProducts * C::kABytes);
        const uint32_t fb = (set + 4 * C::kProducts) | (id << 30);
        const int nkk = min(4, static_cast<int>(cdiv(p.K - kt * kBlk, 32)));
        for (int i = 0; i < C::kProducts; ++i) {
          const uint64_t ad = sdesc_sw128_kmajor(st + i * C::kABytes);
          const uint32_t fa = (set + 4 * i) | (id << 30);
          const uint32_t d = tmem + i * C::kAccCols;
          for (int kk = 0; kk < nkk; ++kk)
            mma_mxf8(d, ad + 2 * kk, bd + 2 * kk, idesc, fa, fb, (kt > 0 || kk > 0) ? 1u : 0u);
        }
        tc_commit(&empty[s]);
      }
      tc_commit(acc_full);
    }
  } else {
    grid_dep_wait();
    const int q = warp & 3;                                // TMEM lane quadrant
    const int n = n0 + 32 * q + lane;
    const bool ok = __all_sync(0xffffffffu, mbar_wait(acc_full, 0, p.err, KQ_DEV_ERR_TIMEOUT_ACC));
    tc_fence_after();
    const uint32_t tb = tmem + (static_cast<uint32_t>(32 * q) << 16);
    if (p.out == 2 && blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 64) *p.oerr = 0u;
    const int tokens = min(BT, p.M - t0);
    for (int c = 0; c < tokens; c += 16) {
      uint32_t g[16], u[16];
      tmem_ld_32x32b_x16(tb + c, g);
      if (GATED) tmem_ld_32x32b_x16(tb + C::kAccCols + c, u);
      tmem_ld_wait();
      float v[16];
#pragma unroll
      for (int j = 0; j < 16; ++j) {
        v[j] = __uint_as_float(g[j]);
        if (GATED) v[j] = gate_act(v[j], p.act) * __uint_as_float(u[j]);
      }
      const int lim = ok ? min(16, tokens - c) : 0;
      if (GATED && p.out == 2) {
        // a block of the 8-bit output is this CTA's 128 features of one token
        asm volatile("bar.sync 1, 128;" ::: "memory");      // the last chunk's maxima are read
#pragma unroll
        for (int j = 0; j < 16; ++j) {
          const uint32_t m = __reduce_max_sync(0xffffffffu, n < p.N ? abs_bits(v[j]) : 0u);
          if (lane == 0) top[q * 16 + j] = m;
        }
        asm volatile("bar.sync 1, 128;" ::: "memory");
#pragma unroll
        for (int j = 0; j < 16; ++j) {
          const uint32_t m = max(max(top[j], top[16 + j]), max(top[32 + j], top[48 + j]));
          const uint32_t byte = scale_byte(m);
          const int64_t t = t0 + c + j;
          if (j < lim) {
            if (n < p.N)
              p.ocodes[t * p.N + n] = static_cast<uint8_t>(e4m3x2(v[j] * inv_scale(byte), 0.f));
            if (q == 0 && lane == 0) p.osf[sf_offset(t, n0 / 128, p.okatoms)] = static_cast<uint8_t>(byte);
          }
        }
      } else if (n < p.N) {
#pragma unroll
        for (int j = 0; j < 16; ++j) {
          if (j >= lim) break;
          const int64_t at = (static_cast<int64_t>(t0) + c + j) * p.ldy + n;
          if (p.out == 1) static_cast<__nv_bfloat16*>(p.y)[at] = __float2bfloat16_rn(v[j]);
          else static_cast<float*>(p.y)[at] = v[j];
        }
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, C::kTmemCols);
  }
}

template <int BT, bool GATED>
cudaError_t launch_rows_kernel(const MmParams& p, cudaStream_t st) {
  auto fn = k_mm_rows<BT, GATED>;
  cudaError_t e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       static_cast<int>(Rows<BT, GATED>::kSmem));
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(cdiv(p.N, 128)), static_cast<unsigned>(cdiv(p.M, BT)));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = Rows<BT, GATED>::kSmem;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, fn, p);
}

}  // namespace

int mm_token_tile(int M) { return M <= 16 ? 16 : M <= 32 ? 32 : M <= 64 ? 64 : 128; }

cudaError_t launch_mm(const MmParams& p, bool gated, cudaStream_t st) {
  switch (mm_token_tile(p.M)) {
    case 16: return gated ? launch_rows_kernel<16, true>(p, st) : launch_rows_kernel<16, false>(p, st);
    case 32: return gated ? launch_rows_kernel<32, true>(p, st) : launch_rows_kernel<32, false>(p, st);
    case 64: return gated ? launch_rows_kernel<64, true>(p, st) : launch_rows_kernel<64, false>(p, st);
    default: return gated ? launch_rows_kernel<128, true>(p, st) : launch_rows_kernel<128, false>(p, st);
  }
}

}  // namespace fp8
}  // namespace kq
