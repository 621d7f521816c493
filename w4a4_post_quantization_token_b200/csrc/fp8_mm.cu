// Block-scaled 8-bit matrix product on the 5th-generation tensor cores:
//
//   Y[m, n] = sum_kb 2^(ex[m, kb] + ew[n / 128, kb]) sum_{k in kb} cx[m, k] cw[n, k]
//
// (tcgen05 kind::mxf8f6f4 with E8M0 scales: the tensor core applies both powers of two as it
// accumulates in fp32), and its gated form  H = act(X Wg) * (X Wu)  with both products, the
// activation and the product in one kernel.
//
// k_mm_rows: one CTA per 128 outputs x BT tokens x a share of K. The weights are the MMA's
// 128-row operand and the tokens its BT columns, so a few tokens cost a few columns. Warp roles:
//   warp 0    TMA producer (one thread): weight and activation k-tiles of 128 bytes per row
//             (128-byte swizzle) into a ring; with the first k-tile of each 512-byte scale atom
//             (4 k-tiles) the atoms themselves.
//   warp 1    TMEM allocator and MMA issuer (one thread): scale atoms to TMEM, 4 MMAs (K = 32)
//             per k-tile and product, a commit that frees the stage.
//   warps 2-5 epilogue: thread = output feature; a warp writes 32 neighbouring features of one
//             token at a time.
// Few tokens leave N / 128 tiles for 148 SMs: K is then split over a cluster. Each CTA puts its
// fp32 partial sums into its shared memory and finishes its share of the tokens, adding the
// partials in the order of the splits, so results do not vary from run to run.
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
  // partials, and the 7 rows that a group of 8 tokens reads past its share
  static constexpr bool kCanSplit = (kProducts * BT + 8) * 512u <= kStages * kStageBytes;
  static constexpr uint32_t kTmemCols = kSfCol + 32 <= 128 ? 128 : (kSfCol + 32 <= 256 ? 256 : 512);
  static_assert(kStages >= 2 && kStageBytes % 1024 == 0, "ring");
  // A scale set is rewritten two atoms later, 5 k-tiles at least: its last MMAs have freed the
  // stage that the new atom landed in.
  static_assert(kStages <= 5, "scale sets");
  // The CTAs of a cluster wait for one another, so that none may wait for TMEM columns which a
  // CTA of another cluster on its SM holds.
  static_assert(!kCanSplit || kTmemCols <= 256, "two CTAs per SM");
};

__device__ __forceinline__ float gate_act(float g, int act) {
  // SiLU g / (1 + e^-g); GELU in its erf form, g erfc(-g / sqrt 2) / 2
  if (act == 0) return __fdividef(g, 1.f + __expf(-g));
  return 0.5f * g * erfcf(-0.70710678118654752f * g);
}

// One thread's feature n0 + 32 q + lane of T tokens from `token`, `lim` of which exist. The four
// epilogue warps call it together: a block of the 8-bit output is the CTA's 128 features of one
// token, and its largest value is found across them (`top` [4][16]).
template <int T, bool GATED>
__device__ __forceinline__ void store(const MmParams& p, const float* v, int token, int lim, int n0, int q, int lane,
                                      uint32_t* top) {
  const int n = n0 + 32 * q + lane;
  if (GATED && p.out == 2) {
    asm volatile("bar.sync 1, 128;" ::: "memory");          // the maxima of the last call were read
#pragma unroll
    for (int j = 0; j < T; ++j) {
      const uint32_t m = __reduce_max_sync(0xffffffffu, n < p.N ? abs_bits(v[j]) : 0u);
      if (lane == 0) top[q * 16 + j] = m;
    }
    asm volatile("bar.sync 1, 128;" ::: "memory");
#pragma unroll
    for (int j = 0; j < T; ++j) {
      if (j >= lim) break;
      const uint32_t byte = scale_byte(max(max(top[j], top[16 + j]), max(top[32 + j], top[48 + j])));
      const int64_t t = static_cast<int64_t>(token) + j;
      if (n < p.N) p.ocodes[t * p.N + n] = static_cast<uint8_t>(e4m3x2(v[j] * inv_scale(byte), 0.f));
      if (q == 0 && lane == 0) p.osf[sf_offset(t, n0 / 128, p.okatoms)] = static_cast<uint8_t>(byte);
    }
  } else if (n < p.N) {
#pragma unroll
    for (int j = 0; j < T; ++j) {
      if (j >= lim) break;
      const int64_t at = (static_cast<int64_t>(token) + j) * p.ldy + n;
      if (p.out == 1) static_cast<__nv_bfloat16*>(p.y)[at] = __float2bfloat16_rn(v[j]);
      else static_cast<float*>(p.y)[at] = v[j];
    }
  }
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
  const int splits = static_cast<int>(gridDim.z), rank = static_cast<int>(blockIdx.z);   // a cluster along z
  const int kt0 = KT * rank / splits, kt1 = KT * (rank + 1) / splits;

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
      const size_t wrow = static_cast<size_t>(blockIdx.x) * p.katoms * 512u;
      const size_t xrow = static_cast<size_t>(t0 / 128) * p.katoms * 512u;
      // the weights' part of a stage and the activations' part, with the scale atoms that the
      // first k-tile of an atom (or of this CTA's share) brings
      auto load_w = [&](int i) {
        const int kt = kt0 + i, s = i % C::kStages;
        const bool atom = (kt & 3) == 0 || i == 0;
        uint8_t* st = ring + s * C::kStageBytes;
        mbar_arrive_expect_tx(&full[s], C::kSfOff + (atom ? (C::kProducts + 1) * 512u : 0u));
        for (int j = 0; j < C::kProducts; ++j) {
          tma_load_2d(st + j * C::kABytes, &p.tmap_w[j], kt * kBlk, n0, &full[s]);
          if (atom) bulk_load(st + C::kSfOff + j * 512, p.sfw[j] + wrow + static_cast<size_t>(kt >> 2) * 512u, 512, &full[s]);
        }
      };
      auto load_x = [&](int i) {
        const int kt = kt0 + i, s = i % C::kStages;
        uint8_t* st = ring + s * C::kStageBytes;
        tma_load_2d(st + C::kProducts * C::kABytes, &p.tmap_x, kt * kBlk, t0, &full[s]);
        if ((kt & 3) == 0 || i == 0)
          bulk_load(st + C::kSfOff + C::kProducts * 512, p.sfx + xrow + static_cast<size_t>(kt >> 2) * 512u, 512, &full[s]);
      };
      // The kernel that writes the activations is the one before this in the stream, and what
      // ran before that one has ended (`dependent`): the weights may be read without a wait.
      const int n = kt1 - kt0, early = p.dependent ? min(n, C::kStages) : 0;
      for (int i = 0; i < early; ++i) load_w(i);
      grid_dep_wait();
      grid_dep_launch();
      int i = 0;
      bool ok = true;
      for (; i < n; ++i) {
        if (i >= C::kStages && !mbar_wait(&empty[i % C::kStages], ((i / C::kStages) - 1) & 1, p.err, KQ_DEV_ERR_TIMEOUT_EMPTY)) {
          ok = false;
          break;
        }
        if (i >= early) load_w(i);
        load_x(i);
      }
      if (!ok) drain_ring(full, C::kStages, i);
    }
  } else if (warp == 1) {
    if (lane == 0) {
      const uint32_t ring_addr = smem_u32(ring);
      for (int i = 0; i < kt1 - kt0; ++i) {
        const int kt = kt0 + i, s = i % C::kStages;
        if (!mbar_wait(&full[s], (i / C::kStages) & 1, p.err, KQ_DEV_ERR_TIMEOUT_FULL)) break;
        tc_fence_after();
        const uint32_t st = ring_addr + s * C::kStageBytes;
        const uint32_t set = tmem + C::kSfCol + static_cast<uint32_t>((kt >> 2) & 1) * 16u;
        if ((kt & 3) == 0 || i == 0) {
          for (int j = 0; j <= C::kProducts; ++j)
            tmem_cp_32x128b_warpx4(set + 4 * j, sdesc_plain_rows16(st + C::kSfOff + j * 512));
        }
        const uint32_t id = static_cast<uint32_t>(kt) & 3u;
        const uint32_t idesc = idesc_mxf8(128, BT, 0) | (id << 4) | (id << 29);
        const uint64_t bd = sdesc_sw128_kmajor(st + C::kProducts * C::kABytes);
        const uint32_t fb = (set + 4 * C::kProducts) | (id << 30);
        const int nkk = min(4, static_cast<int>(cdiv(p.K - kt * kBlk, 32)));
        for (int j = 0; j < C::kProducts; ++j) {
          const uint64_t ad = sdesc_sw128_kmajor(st + j * C::kABytes);
          const uint32_t fa = (set + 4 * j) | (id << 30);
          const uint32_t d = tmem + j * C::kAccCols;
          for (int kk = 0; kk < nkk; ++kk)
            mma_mxf8(d, ad + 2 * kk, bd + 2 * kk, idesc, fa, fb, (i > 0 || kk > 0) ? 1u : 0u);
        }
        tc_commit(&empty[s]);
      }
      tc_commit(acc_full);
    }
  }
  const int q = warp & 3;                                  // TMEM lane quadrant
  const int n = n0 + 32 * q + lane;
  const int tokens = min(BT, p.M - t0);
  const uint32_t tb = tmem + (static_cast<uint32_t>(32 * q) << 16);
  bool ok = true;
  if (warp >= 2) {
    ok = __all_sync(0xffffffffu, mbar_wait(acc_full, 0, p.err, KQ_DEV_ERR_TIMEOUT_ACC));
    tc_fence_after();
    grid_dep_wait();                                       // outputs are written after the grid before
    if (p.out == 2 && blockIdx.x == 0 && blockIdx.y == 0 && rank == 0 && threadIdx.x == 64) *p.oerr = 0u;
  }
  if (splits > 1) {
    // partials [product][token][128 features], over the ring (every load in it was consumed)
    float* part = reinterpret_cast<float*>(ring);
    if (warp >= 2) {
      for (int c = 0; c < tokens; c += 16) {
        uint32_t r[C::kProducts][16];
#pragma unroll
        for (int j = 0; j < C::kProducts; ++j) tmem_ld_32x32b_x16(tb + j * C::kAccCols + c, r[j]);
        tmem_ld_wait();
#pragma unroll
        for (int j = 0; j < C::kProducts; ++j)
#pragma unroll
          for (int t = 0; t < 16; ++t)
            part[(j * BT + c + t) * 128 + 32 * q + lane] = __uint_as_float(r[j][t]);
      }
    }
    __syncwarp();
    cluster_sync();
    if (warp >= 2) {
      // eight tokens at a time, so that the remote loads of a group are in flight together
      const uint32_t mine = smem_u32(part) + 4u * static_cast<uint32_t>(32 * q + lane);
      const int t1 = tokens * (rank + 1) / splits;
      for (int t = tokens * rank / splits; t < t1; t += 8) {
        float v[C::kProducts][8] = {};
        for (int s = 0; s < splits; ++s) {
          const uint32_t at = mapa_shared(mine + 512u * static_cast<uint32_t>(t), static_cast<uint32_t>(s));
          float w[C::kProducts][8];
#pragma unroll
          for (int j = 0; j < C::kProducts; ++j)
#pragma unroll
            for (int i = 0; i < 8; ++i) w[j][i] = ld_shared_cluster_f32(at + 512u * static_cast<uint32_t>(j * BT + i));
#pragma unroll
          for (int j = 0; j < C::kProducts; ++j)
#pragma unroll
            for (int i = 0; i < 8; ++i) v[j][i] += w[j][i];
        }
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (GATED) v[0][i] = gate_act(v[0][i], p.act) * v[C::kProducts - 1][i];
        store<8, GATED>(p, v[0], t0 + t, ok ? min(8, t1 - t) : 0, n0, q, lane, top);
      }
    }
    __syncwarp();
    cluster_sync();                                        // no CTA leaves while its partials are read
  } else if (warp >= 2) {
    for (int c = 0; c < tokens; c += 16) {
      uint32_t r[C::kProducts][16];
#pragma unroll
      for (int j = 0; j < C::kProducts; ++j) tmem_ld_32x32b_x16(tb + j * C::kAccCols + c, r[j]);
      tmem_ld_wait();
      float v[16];
#pragma unroll
      for (int t = 0; t < 16; ++t) {
        v[t] = __uint_as_float(r[0][t]);
        if (GATED) v[t] = gate_act(v[t], p.act) * __uint_as_float(r[C::kProducts - 1][t]);
      }
      store<16, GATED>(p, v, t0 + c, ok ? min(16, tokens - c) : 0, n0, q, lane, top);
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
cudaError_t launch_rows_kernel(const MmParams& p, int sms, cudaStream_t st) {
  auto fn = k_mm_rows<BT, GATED>;
  cudaError_t e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       static_cast<int>(Rows<BT, GATED>::kSmem));
  if (e != cudaSuccess) return e;
  // Splits of K: as long as the CTAs still fit on the GPU at once (two per SM) and each keeps a
  // scale atom (4 k-tiles) of work.
  const int64_t tiles = cdiv(p.N, 128) * cdiv(p.M, BT);
  const int64_t kt = cdiv(p.K, kBlk);
  unsigned splits = 1;
  while (Rows<BT, GATED>::kCanSplit && splits < 8 && tiles * 2 * splits <= 2 * sms && kt >= 4 * 2 * splits) splits *= 2;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(cdiv(p.N, 128)), static_cast<unsigned>(cdiv(p.M, BT)), splits);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = Rows<BT, GATED>::kSmem;
  cfg.stream = st;
  // Only the product behind its own activation kernel (`dependent`) may start before that one
  // has ended.
  cudaLaunchAttribute attr[2];
  int na = 0;
  if (splits > 1) {
    attr[na].id = cudaLaunchAttributeClusterDimension;
    attr[na].val.clusterDim.x = 1;
    attr[na].val.clusterDim.y = 1;
    attr[na++].val.clusterDim.z = splits;
  }
  if (p.dependent) {
    attr[na].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[na++].val.programmaticStreamSerializationAllowed = 1;
  }
  cfg.attrs = attr;
  cfg.numAttrs = static_cast<unsigned>(na);
  return cudaLaunchKernelEx(&cfg, fn, p);
}

// k_mm_pair: 256 tokens x 256 weight rows per pair of CTAs (gated: 128 of the gate and the same
// 128 of up, so that both halves of an output meet in one thread). The two CTAs of a cluster run
// one MMA of M = 256 (cta_group::2): each stages its own 128 tokens and half of the weight rows,
// 32 KB per 128-element k-tile instead of the 48 KB a 128 x 256 tile of one CTA would need. Per
// k-tile the MMAs take 512 cycles, so a CTA pulls 64 bytes a cycle from L2, where 96 would
// exceed what an SM gets. Persistent, one pair per two SMs. Warp roles:
//   warp 0     TMA producer in each CTA; all loads of a stage, the peer's too, complete on the
//              first CTA's barrier.
//   warp 1     TMEM allocator; in the first CTA the MMA issuer for both.
//   warps 2-9  epilogue: thread = token, two warps share a TMEM lane quadrant and take half of
//              the columns each; 64-byte rows go through swizzled staging buffers to TMA stores.
// TMEM holds two accumulators of 256 columns that overlap in 64 (0 .. 255 and 192 .. 447) and the
// scales behind them: the epilogue reads the shared 64 columns first, and the next tile's MMAs
// start as soon as those are out.
struct Pair {
  static constexpr int kStages = 5;
  static constexpr uint32_t kTile = 128 * 128;
  static constexpr uint32_t kStageBytes = 2 * kTile;                 // tokens, weight rows
  static constexpr uint32_t kSfBytes = 3 * 512;                      // tokens, both weight halves
  static constexpr uint32_t kStgBytes = 2048;                        // 32 rows x 64 bytes
  static constexpr uint32_t kRingOff = 1024;
  static constexpr uint32_t kStgOff = kRingOff + kStages * kStageBytes;
  static constexpr uint32_t kSfOff = kStgOff + 8 * 2 * kStgBytes;
  static constexpr uint32_t kTopOff = kSfOff + kStages * kSfBytes;   // uint32 [2 halves][128 rows]
  static constexpr uint32_t kSmem = 1024 + kTopOff + 1024;
  static constexpr uint32_t kAccStride = 192;
  // Scale sets of 12 columns (tokens 4, weight rows 8), used in turn by the atoms. A set comes
  // round after kStages atoms, so after kStages k-tiles at least: its last MMAs have freed the
  // stage that the new atom landed in.
  static constexpr uint32_t kSfCol = 448, kSfSet = 12;
  static constexpr int kThreads = 320;
  static_assert(kSmem <= 232448 && kSfCol + kStages * kSfSet <= 512, "shared memory, TMEM");
};

// Tile order: groups of 8 row tiles, row tile fastest, so that the pairs at work share a few
// row tiles and a few column tiles in L2.
__device__ __forceinline__ void pair_tile(int tile, int MT, int NT, int& mt, int& nt) {
  const int per = 8 * NT, g = tile / per, r = tile - g * per;
  const int gm = min(8, MT - g * 8);
  mt = g * 8 + r % gm;
  nt = r / gm;
}

// 64 bytes of one row (16 words) into a warp's staging buffer (64-byte swizzle), then the warp's
// 32 x 64-byte box to global memory. `n` counts the warp's boxes: two buffers alternate.
__device__ __forceinline__ void put_box(const uint32_t (&w)[16], uint8_t* stg, uint32_t& n, const CUtensorMap* map, int x,
                                        int y, bool on, int lane) {
  uint8_t* b = stg + (n & 1u) * Pair::kStgBytes;
  if (lane == 0) bulk_wait_read<1>();
  __syncwarp();
  uint8_t* row = b + lane * 64;
#pragma unroll
  for (int c = 0; c < 4; ++c)
    *reinterpret_cast<uint4*>(row + 16 * (c ^ ((lane >> 1) & 3))) = make_uint4(w[4 * c], w[4 * c + 1], w[4 * c + 2], w[4 * c + 3]);
  fence_async_smem();
  __syncwarp();
  if (lane == 0) {
    if (on) tma_store_2d(map, b, x, y);
    bulk_commit();
  }
  ++n;
}

// CN values of one row from column x as fp32 or bf16 boxes.
template <int CN>
__device__ __forceinline__ void put_values(const MmParams& p, const float (&v)[CN], uint8_t* stg, uint32_t& n, int x, int y,
                                           bool ok, int lane) {
  uint32_t w[16];
  if (p.out == 1) {
#pragma unroll
    for (int c = 0; c < CN; c += 32) {
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const __nv_bfloat162 b = __floats2bfloat162_rn(v[c + 2 * i], v[c + 2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t*>(&b);
      }
      put_box(w, stg, n, &p.tmap_y, x + c, y, ok && x + c < p.N && y < p.M, lane);
    }
  } else {
#pragma unroll
    for (int c = 0; c < CN; c += 16) {
#pragma unroll
      for (int i = 0; i < 16; ++i) w[i] = __float_as_uint(v[c + i]);
      put_box(w, stg, n, &p.tmap_y, x + c, y, ok && x + c < p.N && y < p.M, lane);
    }
  }
}

template <bool GATED>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(Pair::kThreads, 1)
k_mm_pair(const __grid_constant__ MmParams p) {
  using C = Pair;
  constexpr int kBN = GATED ? 128 : 256;                             // output columns of a tile
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(align_up(reinterpret_cast<uintptr_t>(smem_raw), 1024));
  uint64_t* full = reinterpret_cast<uint64_t*>(smem);                // used in the first CTA
  uint64_t* empty = full + C::kStages;
  uint64_t* acc_full = empty + C::kStages;
  uint64_t* acc_free = acc_full + 2;                                 // used in the first CTA
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(acc_free + 2);
  uint8_t* ring = smem + C::kRingOff;
  uint8_t* sfring = smem + C::kSfOff;
  uint32_t* top = reinterpret_cast<uint32_t*>(smem + C::kTopOff);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();
  const int MT = static_cast<int>(cdiv(p.M, 256)), NT = static_cast<int>(cdiv(p.N, kBN)), T = MT * NT;
  const int KT = static_cast<int>(cdiv(p.K, kBlk));
  const int first = static_cast<int>(blockIdx.x >> 1), step = static_cast<int>(gridDim.x >> 1);

  if (threadIdx.x == 0) {
    for (int s = 0; s < C::kStages; ++s) { mbar_init(&full[s], 1); mbar_init(&empty[s], 1); }
    for (int b = 0; b < 2; ++b) { mbar_init(&acc_full[b], 1); mbar_init(&acc_free[b], 16); }
    fence_mbar_init();
    prefetch_tmap(&p.tmap_w[0]);
    if (GATED) prefetch_tmap(&p.tmap_w[1]);
    prefetch_tmap(&p.tmap_x);
  }
  if (warp == 1) { tmem_alloc_pair(tmem_slot, 512); tmem_relinquish_pair(); }
  tc_fence_before();
  __syncthreads();
  cluster_sync();                                                    // both CTAs' barriers exist
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  if (warp == 0) {
    if (lane == 0) {
      const int w = GATED ? static_cast<int>(rank) : 0;              // gated: gate rows here, up rows there
      grid_dep_wait();
      grid_dep_launch();
      int it = 0;
      bool ok = true;
      for (int tile = first; tile < T && ok; tile += step) {
        int mt, nt;
        pair_tile(tile, MT, NT, mt, nt);
        const int m0 = mt * 256 + 128 * static_cast<int>(rank);
        const int n0 = GATED ? nt * 128 : nt * 256 + 128 * static_cast<int>(rank);
        // scale atoms by row group; a group past the last (its rows are not stored) reads the last
        const int ka = static_cast<int>(p.katoms);
        const int xa = min(m0 / 128, static_cast<int>(cdiv(p.M, 128)) - 1) * ka;
        const int nb = static_cast<int>(cdiv(p.N, 128)) - 1;
        const int wa0 = (GATED ? nt : nt * 2) * ka, wa1 = (GATED ? nt : min(nt * 2 + 1, nb)) * ka;
        for (int kt = 0; kt < KT; ++kt, ++it) {
          const int s = it % C::kStages;
          if (it >= C::kStages && !mbar_wait(&empty[s], ((it / C::kStages) - 1) & 1, p.err, KQ_DEV_ERR_TIMEOUT_EMPTY)) {
            ok = false;
            break;
          }
          const bool atom = (kt & 3) == 0;
          const uint32_t bar = mapa_shared(smem_u32(&full[s]), 0);
          if (rank == 0) mbar_arrive_expect_tx(&full[s], 2 * (C::kStageBytes + (atom ? C::kSfBytes : 0u)));
          uint8_t* st = ring + s * C::kStageBytes;
          tma_load_2d_pair(st, &p.tmap_x, kt * kBlk, m0, bar);
          tma_load_2d_pair(st + C::kTile, &p.tmap_w[w], kt * kBlk, n0, bar);
          if (atom) {
            uint8_t* sf = sfring + s * C::kSfBytes;
            tma_load_2d_pair(sf, &p.tmap_sfx, 0, xa + (kt >> 2), bar);
            tma_load_2d_pair(sf + 512, &p.tmap_sfw[0], 0, wa0 + (kt >> 2), bar);
            tma_load_2d_pair(sf + 1024, &p.tmap_sfw[GATED ? 1 : 0], 0, wa1 + (kt >> 2), bar);
          }
        }
      }
      // the first CTA's barriers count the loads of both; the peer leaves after the cluster
      // barrier below, so after this wait
      if (!ok && rank == 0) drain_ring(full, C::kStages, it);
    }
  } else if (warp == 1) {
    if (lane == 0 && rank == 0) {
      const uint64_t ad0 = sdesc_sw128_kmajor(smem_u32(ring)), bd0 = sdesc_sw128_kmajor(smem_u32(ring) + C::kTile);
      const uint64_t sd0 = sdesc_plain_rows16(smem_u32(sfring));
      int s = 0, local = 0;
      uint32_t ph = 0, set = 0;
      bool ok = true;
      for (int tile = first; tile < T && ok; tile += step, ++local) {
        const int buf = local & 1;
        if (local >= 1 && !mbar_wait_cluster(&acc_free[buf], ((local - (buf ? 1 : 2)) >> 1) & 1, p.err, KQ_DEV_ERR_TIMEOUT_ACC)) {
          ok = false;
          break;
        }
        tc_fence_after();
        const uint32_t d = tmem + static_cast<uint32_t>(buf) * C::kAccStride;
        for (int kt = 0; kt < KT; ++kt) {
          if (!mbar_wait(&full[s], ph, p.err, KQ_DEV_ERR_TIMEOUT_FULL)) {
            ok = false;
            break;
          }
          tc_fence_after();
          if ((kt & 3) == 0) {
            set = set + 1 == C::kStages ? 0 : set + 1;
            const uint32_t f = tmem + C::kSfCol + C::kSfSet * set;
            const uint64_t sd = sd0 + static_cast<uint64_t>(s) * (C::kSfBytes >> 4);
            tmem_cp_32x128b_warpx4_pair(f, sd);
            tmem_cp_32x128b_warpx4_pair(f + 4, sd + 32);
            tmem_cp_32x128b_warpx4_pair(f + 8, sd + 64);
          }
          const uint32_t id = static_cast<uint32_t>(kt) & 3u;
          const uint32_t idesc = idesc_mxf8(256, 256, 0) | (id << 4) | (id << 29);
          const uint32_t fa = (tmem + C::kSfCol + C::kSfSet * set) | (id << 30);
          const uint64_t so = static_cast<uint64_t>(s) * (C::kStageBytes >> 4);
          const int nkk = min(4, static_cast<int>(cdiv(p.K - kt * kBlk, 32)));
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
            if (kk < nkk) mma_mxf8_pair(d, ad0 + so + 2 * kk, bd0 + so + 2 * kk, idesc, fa, fa + 4, (kt > 0 || kk > 0) ? 1u : 0u);
          tc_commit_pair(&empty[s]);
          if (++s == C::kStages) { s = 0; ph ^= 1u; }
        }
        tc_commit_pair(&acc_full[buf]);
      }
    }
  } else {
    grid_dep_wait();
    const int q = warp & 3, half = (warp - 2) >> 2;
    uint8_t* stg = smem + C::kStgOff + static_cast<uint32_t>(warp - 2) * 2 * C::kStgBytes;
    uint32_t boxes = 0;
    const uint32_t free0 = mapa_shared(smem_u32(&acc_free[0]), 0);
    if (GATED && p.out == 2 && blockIdx.x == 0 && threadIdx.x == 64) *p.oerr = 0u;
    // The shared columns are the second half's of accumulator 0 and the first half's of 1. Their
    // owner frees the other accumulator after reading them, and its own after reading the rest;
    // the first half's share of accumulator 1's first turn is free from the start.
    if (half == 0 && lane == 0) mbar_arrive_cluster(free0 + 8);
    int local = 0;
    for (int tile = first; tile < T; tile += step, ++local) {
      int mt, nt;
      pair_tile(tile, MT, NT, mt, nt);
      const int m0 = mt * 256 + 128 * static_cast<int>(rank) + 32 * q;
      const int buf = local & 1;
      const bool owner = half != buf;
      const bool ok = __all_sync(0xffffffffu, mbar_wait(&acc_full[buf], (local >> 1) & 1, p.err, KQ_DEV_ERR_TIMEOUT_ACC));
      tc_fence_after();
      const uint32_t tb = tmem + static_cast<uint32_t>(buf) * C::kAccStride + (static_cast<uint32_t>(32 * q) << 16);
      auto release = [&](int b) {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_cluster(free0 + 8u * static_cast<uint32_t>(b));
      };
      if (!GATED) {
        // four chunks of 32 columns, from the shared end: 224, 192, 160, 128 in the second half of
        // accumulator 0; 0, 32, 64, 96 in the first of accumulator 1
        const int n0 = nt * 256 + 128 * half;
#pragma unroll 1
        for (int c = 0; c < 4; ++c) {
          const int col = 32 * (buf == 0 && half == 1 ? 3 - c : c);
          uint32_t r[32];
          tmem_ld_32x32b_x32(tb + 128 * half + col, r);
          tmem_ld_wait();
          if (owner && c == 1) release(buf ^ 1);
          if (owner && c == 3) release(buf);
          float v[32];
#pragma unroll
          for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(r[i]);
          put_values(p, v, stg, boxes, n0 + col, m0, ok, lane);
        }
      } else {
        // outputs 64 half .. 64 half + 63: the operand with the shared columns first (up in
        // accumulator 0, the gate in 1), then the other
        const uint32_t g0 = tb + 64 * half, u0 = g0 + 128;
        float v[64];
        {
          uint32_t r[2][32];
          tmem_ld_32x32b_x32(buf == 0 ? u0 : g0, r[0]);
          tmem_ld_32x32b_x32((buf == 0 ? u0 : g0) + 32, r[1]);
          tmem_ld_wait();
#pragma unroll
          for (int i = 0; i < 64; ++i) v[i] = __uint_as_float(r[i >> 5][i & 31]);
        }
        if (owner) release(buf ^ 1);
        uint32_t a = 0;
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          uint32_t r[32];
          tmem_ld_32x32b_x32((buf == 0 ? g0 : u0) + 32 * c, r);
          tmem_ld_wait();
          if (owner && c == 1) release(buf);
#pragma unroll
          for (int i = 0; i < 32; ++i) {
            const float o = __uint_as_float(r[i]), f = v[32 * c + i];
            v[32 * c + i] = gate_act(buf == 0 ? o : f, p.act) * (buf == 0 ? f : o);
          }
        }
        const int n0 = nt * 128 + 64 * half;
        if (p.out != 2) {
          put_values(p, v, stg, boxes, n0, m0, ok, lane);
        } else {
          // a block is the 128 outputs of a token in this tile: its largest value from both halves
#pragma unroll
          for (int i = 0; i < 64; ++i)
            if (n0 + i < p.N) a = max(a, abs_bits(v[i]));
          top[128 * half + 32 * q + lane] = a;
          asm volatile("bar.sync %0, 64;" ::"r"(1 + q) : "memory");
          a = max(a, top[128 * (half ^ 1) + 32 * q + lane]);
          asm volatile("bar.sync %0, 64;" ::"r"(1 + q) : "memory");
          const uint32_t byte = scale_byte(a);
          const float is = inv_scale(byte);
          uint32_t w[16];
#pragma unroll
          for (int i = 0; i < 16; ++i)
            w[i] = e4m3x4(v[4 * i] * is, v[4 * i + 1] * is, v[4 * i + 2] * is, v[4 * i + 3] * is);
          put_box(w, stg, boxes, &p.tmap_y, n0, m0, ok && n0 < p.N && m0 < p.M, lane);
          if (ok && half == 0 && m0 + lane < p.M) p.osf[sf_offset(m0 + lane, nt, p.okatoms)] = static_cast<uint8_t>(byte);
        }
      }
    }
    if (lane == 0) bulk_wait_all();
    __syncwarp();
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();              // the peer's MMAs, loads and arrivals that reach into this CTA are over
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_pair(tmem, 512);
  }
}

template <bool GATED>
cudaError_t launch_pair_kernel(const MmParams& p, int sms, cudaStream_t st) {
  auto fn = k_mm_pair<GATED>;
  cudaError_t e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(Pair::kSmem));
  if (e != cudaSuccess) return e;
  const int64_t tiles = cdiv(p.M, 256) * cdiv(p.N, GATED ? 128 : 256);
  const int64_t pairs = tiles < sms / 2 ? tiles : sms / 2;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(2 * pairs));
  cfg.blockDim = dim3(Pair::kThreads);
  cfg.dynamicSmemBytes = Pair::kSmem;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = p.dependent ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, fn, p);
}

}  // namespace

bool mm_by_pairs(int M, int N, int K, bool gated, int sms) {
  (void)K; (void)N; (void)gated; (void)sms;
  return M > 256;
}

int mm_token_tile(int M) { return M <= 16 ? 16 : M <= 32 ? 32 : M <= 64 ? 64 : 128; }

cudaError_t launch_mm(const MmParams& p, bool gated, int sms, cudaStream_t st) {
  if (p.pairs) return gated ? launch_pair_kernel<true>(p, sms, st) : launch_pair_kernel<false>(p, sms, st);
  switch (mm_token_tile(p.M)) {
    case 16: return gated ? launch_rows_kernel<16, true>(p, sms, st) : launch_rows_kernel<16, false>(p, sms, st);
    case 32: return gated ? launch_rows_kernel<32, true>(p, sms, st) : launch_rows_kernel<32, false>(p, sms, st);
    case 64: return gated ? launch_rows_kernel<64, true>(p, sms, st) : launch_rows_kernel<64, false>(p, sms, st);
    default: return gated ? launch_rows_kernel<128, true>(p, sms, st) : launch_rows_kernel<128, false>(p, sms, st);
  }
}

}  // namespace fp8
}  // namespace kq
