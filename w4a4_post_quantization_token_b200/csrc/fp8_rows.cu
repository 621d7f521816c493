// Block-scaled 8-bit matrix product on the 5th-generation tensor cores:
//
//   Y[m, n] = sum_kb 2^(ex[m, kb] + ew[n / 128, kb]) sum_{k in kb} cx[m, k] cw[n, k]
//
// (tcgen05 kind::mxf8f6f4 with E8M0 scales: the tensor core applies both powers of two as it
// accumulates in fp32), and its gated form  H = act(X Wg) * (X Wu)  with both products, the
// activation and the product in one kernel. This file: up to 64 tokens, where reading the weights
// once is all that counts; fp8_pair.cu takes more.
//
// k_rows_mm: one CTA per 128 outputs x BT tokens x a share of K. The weights are the MMA's
// 128-row operand and the tokens its BT columns, so a few tokens cost a few columns. Warp roles:
//   warps 0, 6  TMA producers of the weights and of the activations: k-tiles of 128 bytes per row
//             (128-byte swizzle) into a ring; with the first k-tile of each 512-byte scale atom
//             (4 k-tiles) the atoms themselves. One warp alone needs 360 cycles or more for a
//             stage's wait and copies, which holds an SM to 45 bytes a cycle of the 64 it can take.
//   warp 1    TMEM allocator and MMA issuer: scale atoms to TMEM, 4 MMAs (K = 32) per k-tile and
//             product, a commit that frees the stage.
//   warps 2-5 epilogue: thread = output feature; a warp writes 32 neighbouring features of one
//             token at a time.
// LONG: fp32 outputs of more k-tiles than sum_tiles. After each piece the issuer waits until the epilogue
// has added the accumulators to its sums in registers; the ring goes on filling meanwhile.
//
// A wait that runs out ends the kernel without an output: the MMA issuer does not commit the
// accumulators, waits for its MMAs and for the loads under way, and the epilogue's own wait for the
// accumulators runs out too. It stores nothing then, and neither does a CTA that lacks its sums.
// The clocks of all waits start once the kernel before this one has ended.
// FUSED: the activations are bf16 and the kernel encodes its share of K of them itself, while the
// first weights arrive: warps 2-5 and 7-14 write codes (in the swizzled layout of a TMA load) and
// scale bytes to shared memory. Every CTA of the same share does the same work over again, which
// for so few tokens costs less than a kernel of its own ahead of this one.
//
// Few tokens leave N / 128 tiles for 148 SMs: K is then split over a cluster. Each CTA finishes a
// share of the tokens: the others store their fp32 partial sums of it into its shared memory
// (stores to a neighbour need no answer, loads would cost a round trip each), four tokens to a
// store, and it adds them in the order of the splits, so results do not vary from run to run.
//
// Bound by HBM, or L2 where the weights are there, between fixed costs of some 4 us (launch, set-up,
// the first load's latency, exchange and epilogue): one token 12288 -> 12288 25.3 us (151 MB, 6.0
// TB/s; 64 tokens 27.3), gated 8 tokens 4096 -> 12288 18.2 us (101 MB, 5.5 TB/s), one token 4096 ->
// 4096 with the weights in L2 4.7 us, 512 -> 512 2.2 us.
#include <cuda_bf16.h>

#include <atomic>

#include "fp8.cuh"
#include "sm100_fp8.cuh"

namespace kq {
namespace fp8 {

namespace {

constexpr int kMaxSplits = 8;
// FUSED: the warps that encode, and the blocks of 128 values that they load together (two to a warp, kDeep
// times), which is also the most that a CTA encodes.
constexpr int kEncWarps = 12, kDeep = 4;
constexpr int kEncRound = 2 * kEncWarps * kDeep;

template <int BT, bool GATED, bool FUSED>
struct Rows {
  static constexpr int kThreads = FUSED ? 480 : 224;
  static constexpr int kProducts = GATED ? 2 : 1;
  static constexpr uint32_t kABytes = 128 * 128;
  static constexpr uint32_t kBBytes = BT * 128;
  static constexpr uint32_t kSfOff = kProducts * kABytes + (FUSED ? 0 : kBBytes);   // scale atoms: weights, tokens
  static constexpr uint32_t kSfAtoms = kProducts + (FUSED ? 0 : 1);
  static constexpr uint32_t kStageBytes = kSfOff + (kSfAtoms > 2 ? 2048 : 1024);
  // k-tiles that a CTA can encode: kEncRound blocks of the fewest tokens of this tile, 64 KB at most.
  // (128 BT bytes each, and their scale atoms: 4 k-tiles, or fewer at both ends of the share.)
  static constexpr int kEncShare = kEncRound / (BT == 16 ? 1 : 17);
  static constexpr int kMaxShare = FUSED ? (kEncShare < 512 / BT ? kEncShare : 512 / BT) : 1 << 30;
  static constexpr uint32_t kXBytes = FUSED ? kMaxShare * kBBytes : 0;
  // Partials received in the exchange: [split][product][four tokens of the share][128 features] x
  // 16 bytes. Up to 16 tokens they have room of their own; beyond, they go over the ring once the
  // cluster's MMAs are done, which takes a cluster barrier more.
  static constexpr bool kOwnPart = BT <= 16;
  static constexpr uint32_t kPartBytes = kProducts * (kOwnPart ? kMaxSplits : BT / 4 + kMaxSplits) * 2048;
  // As many stages as an SM holds, 9 at most (scale sets, below): every k-tile of a small share is
  // under way at once.
  static constexpr uint32_t kRoom = 226 * 1024 - 2048 - kXBytes - (FUSED ? 5120 : 0) - (kOwnPart ? kPartBytes : 0);
  static constexpr int kStages = kRoom / kStageBytes < 9 ? kRoom / kStageBytes : 9;
  static constexpr uint32_t kRingBytes = kStages * kStageBytes;
  // accumulators 64 columns apart, then 3 scale sets of 16 columns
  static constexpr uint32_t kSfCol = kProducts * 64;
  static constexpr uint32_t kTmemCols = kSfCol + 48 <= 128 ? 128 : 256;
  static constexpr uint32_t smem(int share) {
    return 2048 + kRingBytes + (kOwnPart ? kPartBytes : 0) + (FUSED ? share * kBBytes + (share / 4 + 2) * 512 : 0);
  }
  static_assert(kStages >= 3 && kStageBytes % 1024 == 0 && BT <= 64, "ring");
  static_assert(smem(FUSED ? kMaxShare : 0) + 1024 <= 232448, "shared memory");
  // A scale set is rewritten three atoms later, 9 k-tiles at least after its last use: those
  // MMAs have freed the stage that the new atom landed in.
  static_assert(kStages <= 9, "scale sets");
  static_assert(kPartBytes + 2048 <= kRingBytes, "exchange and codes over the ring");
  // The CTAs of a cluster wait for one another, so that none may wait for TMEM columns which a
  // CTA of another cluster on its SM holds: columns for two.
  static_assert(kTmemCols <= 256, "two CTAs per SM");
};

// One thread's feature n0 + 32 q + lane of T tokens from `token`, `lim` of which exist. The four
// epilogue warps call it together. A block of the 8-bit output is the CTA's 128 features of one
// token: its largest value is found across the warps (`top` [4][16]), the codes are put together
// in `tile` [T][128] and written 16 to a store; nothing is written if `bad` was set in any of them.
// BLOCKS: an 8-bit output is possible.
template <int T, bool BLOCKS>
__device__ __forceinline__ void store(const MmParams& p, const float* v, int token, int lim, int n0, int q, int lane,
                                      uint32_t* top, uint8_t* tile, const volatile uint32_t* bad) {
  const int n = n0 + 32 * q + lane;
  if (BLOCKS && p.out == 2) {
    asm volatile("bar.sync 1, 128;" ::: "memory");          // the last call's maxima and codes were read
    if (*bad) lim = 0;
    uint32_t m = 0;
#pragma unroll
    for (int j = 0; j < T; ++j) {
      const uint32_t mj = __reduce_max_sync(0xffffffffu, n < p.N ? abs_bits(v[j]) : 0u);
      if (lane == j) m = mj;
    }
    if (lane < T) top[q * 16 + lane] = m;
    asm volatile("bar.sync 1, 128;" ::: "memory");
    if (lane < T) m = scale_byte(max(max(top[lane], top[16 + lane]), max(top[32 + lane], top[48 + lane])));
    if (q == 0 && lane < T && lane < lim)
      p.osf[sf_offset(static_cast<int64_t>(token) + lane, n0 / 128, p.okatoms)] = static_cast<uint8_t>(m);
#pragma unroll
    for (int j = 0; j < T; ++j) {
      const float is = inv_scale(__shfl_sync(0xffffffffu, m, j));
      tile[128 * j + 32 * q + lane] = static_cast<uint8_t>(e4m3x2(v[j] * is, 0.f));
    }
    asm volatile("bar.sync 1, 128;" ::: "memory");
    const int i = 32 * q + lane, j = i >> 3, c = 16 * (i & 7);       // 8 threads to a token
    if (j < lim && j < T && n0 + c < p.N)
      *reinterpret_cast<uint4*>(p.ocodes + (static_cast<int64_t>(token) + j) * p.N + n0 + c) =
          *reinterpret_cast<const uint4*>(tile + 128 * j + c);
  } else if (n < p.N) {
    const int64_t at = static_cast<int64_t>(token) * p.ldy + n;
    if (p.out == 1) {
      __nv_bfloat16* y = static_cast<__nv_bfloat16*>(p.y) + at;
#pragma unroll
      for (int j = 0; j < T; ++j, y += p.ldy)
        if (j < lim) *y = __float2bfloat16_rn(v[j]);
    } else {
      float* y = static_cast<float*>(p.y) + at;
#pragma unroll
      for (int j = 0; j < T; ++j, y += p.ldy)
        if (j < lim) *y = v[j];
    }
  }
}

// Encodes k-tiles kt0 .. kt0 + n - 1 of all tokens into shared memory: codes as [k-tile][BT rows
// of 128 bytes] with the 128-byte swizzle, scale bytes as atoms. 16 lanes hold a block of 128
// values, 8 each, and all loads come first. `warp` of kEncWarps; n tokens <= kEncRound.
template <int BT>
__device__ __forceinline__ void encode_share(const MmParams& p, int tokens, int kt0, int n, uint8_t* codes, uint8_t* sf,
                                             int warp, int lane) {
  const int items = n * tokens, l = lane & 15;
  uint4 u[kDeep];
#pragma unroll
  for (int j = 0; j < kDeep; ++j) {
    const int item = 2 * (warp + kEncWarps * j) + (lane >> 4), i = item / tokens, t = item - i * tokens;
    const int k = (kt0 + i) * kBlk + 8 * l;
    u[j] = make_uint4(0, 0, 0, 0);
    if (item < items && k < p.K)
      u[j] = __ldcg(reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(p.xb) + t * p.ldx + k));
  }
#pragma unroll
  for (int j = 0; j < kDeep; ++j) {
    const int item = 2 * (warp + kEncWarps * j) + (lane >> 4), i = item / tokens, t = item - i * tokens;
    if (2 * (warp + kEncWarps * j) >= items) break;                      // the same in both half-warps
    float v[8];
    unpack8(u[j], v);
    const uint32_t byte = block_byte(v);
    const float is = inv_scale(byte);
    if (item < items) {
      *reinterpret_cast<uint2*>(codes + i * (BT * 128) + t * 128 + 16 * ((l >> 1) ^ (t & 7)) + 8 * (l & 1)) =
          make_uint2(e4m3x4(v[0] * is, v[1] * is, v[2] * is, v[3] * is),
                     e4m3x4(v[4] * is, v[5] * is, v[6] * is, v[7] * is));
      // (tokens of a 32-row quarter are 16 bytes apart; no more than 32 tokens are encoded here)
      if (l == 0) sf[512 * (((kt0 + i) >> 2) - (kt0 >> 2)) + 16 * t + ((kt0 + i) & 3)] = static_cast<uint8_t>(byte);
    }
  }
}

// ACT: -1 plain, 0 SiLU-gated, 1 GELU-gated
template <int BT, int ACT, bool FUSED, bool LONG>
__global__ void __launch_bounds__(Rows<BT, ACT >= 0, FUSED>::kThreads) k_rows_mm(const __grid_constant__ MmParams p) {
  constexpr bool GATED = ACT >= 0;
  constexpr int kSum = sum_tiles(GATED);
  using C = Rows<BT, GATED, FUSED>;
  static_assert(!LONG || !FUSED, "a CTA encodes fewer k-tiles");
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(align_up(reinterpret_cast<uintptr_t>(smem_raw), 1024));
  uint64_t* full = reinterpret_cast<uint64_t*>(smem);
  uint64_t* empty = full + C::kStages;
  uint64_t* acc_full = empty + C::kStages;
  uint64_t* x_ready = acc_full + 1;
  uint64_t* acc_free = x_ready + 1;                                      // LONG
  uint64_t* mma_done = acc_free + 1;                                     // after a wait ran out
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(mma_done + 1);
  volatile uint32_t* bad = tmem_slot + 1;                                // sums of this CTA's outputs are missing
  uint32_t* top = reinterpret_cast<uint32_t*>(smem + 512);               // [4 warps][16 tokens]
  uint8_t* ring = smem + 1024;

  const int warp = warp_index(), lane = threadIdx.x & 31;
  const int n0 = blockIdx.x * 128, tokens = p.M;
  const int KT = static_cast<int>(cdiv(p.K, kBlk));
  const int splits = static_cast<int>(gridDim.z), rank = static_cast<int>(blockIdx.z);   // a cluster along z
  const int kt0 = KT * rank / splits, n_kt = KT * (rank + 1) / splits - kt0;
  float4* part = reinterpret_cast<float4*>(C::kOwnPart ? ring + C::kRingBytes : ring);
  uint8_t* xcodes = ring + C::kRingBytes + (C::kOwnPart ? C::kPartBytes : 0);   // FUSED: encoded share, its scales
  uint8_t* xsf = xcodes + n_kt * C::kBBytes;

  if (threadIdx.x == 0) {
    for (int s = 0; s < C::kStages; ++s) { mbar_init(&full[s], 1); mbar_init(&empty[s], 1); }
    mbar_init(acc_full, 1);
    mbar_init(x_ready, 32 * kEncWarps);
    mbar_init(acc_free, 4);
    mbar_init(mma_done, 1);
    *bad = 0;
    fence_mbar_init();
    prefetch_tmap(&p.tmap_w[0]);
    if (GATED) prefetch_tmap(&p.tmap_w[1]);
    if (!FUSED) prefetch_tmap(&p.tmap_x);
  }
  if (warp == 1) { tmem_alloc(tmem_slot, C::kTmemCols); tmem_relinquish(); }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  // kOwnPart: the others may store into this CTA's room once it has started, which they learn here
  if (C::kOwnPart && splits > 1) cluster_arrive();
  if (warp == 0) {
    // The kernel that writes the activations is the one before this in the stream, and what ran
    // before that one has ended (`dependent`): the weights may be read without a wait.
    if (!p.dependent) grid_dep_wait();
    if (FUSED) grid_dep_launch();
    const uint32_t one = elect_one();
    const uint8_t* sfw[2] = {p.sfw[0] + static_cast<size_t>(blockIdx.x) * p.katoms * 512u,
                             GATED ? p.sfw[1] + static_cast<size_t>(blockIdx.x) * p.katoms * 512u : nullptr};
    uint32_t st = smem_u32(ring), bar = smem_u32(full);
    const int skip = p.withhold;
    int s = 0;
    uint32_t ph = 1;
    for (int i = 0; i < n_kt; ++i) {
      if (i == C::kStages) grid_dep_wait();
      if (i >= C::kStages && !mbar_wait(&empty[s], ph, p.err, KQ_DEV_ERR_TIMEOUT_EMPTY, p.wait_ns)) break;
      const int kt = kt0 + i;
      const bool atom = (kt & 3) == 0 || i == 0;
      const uint32_t load = i == skip ? 0u : one;
      expect_tx_if(one, bar, C::kSfOff + (atom ? C::kSfAtoms * 512u : 0u));
#pragma unroll
      for (int j = 0; j < C::kProducts; ++j) {
        tma_load_if(load, st + j * C::kABytes, &p.tmap_w[j], kt * kBlk, n0, bar);
        if (atom) bulk_load_if(one, st + C::kSfOff + j * 512, sfw[j] + static_cast<size_t>(kt >> 2) * 512u, 512, bar);
      }
      st += C::kStageBytes;
      bar += 8;
      if (++s == C::kStages) { s = 0; ph ^= 1u; st = smem_u32(ring); bar = smem_u32(full); }
    }
  } else if (warp == 6) {
    if (!FUSED) {
      grid_dep_wait();
      grid_dep_launch();
      const uint32_t one = elect_one();
      const uint32_t st0 = smem_u32(ring) + C::kProducts * C::kABytes;
      uint32_t st = st0, bar = smem_u32(full);
      int s = 0;
      uint32_t ph = 1;
      for (int i = 0; i < n_kt; ++i) {
        if (i >= C::kStages && !mbar_wait(&empty[s], ph, p.err, KQ_DEV_ERR_TIMEOUT_EMPTY, p.wait_ns)) break;
        const int kt = kt0 + i;
        tma_load_if(one, st, &p.tmap_x, kt * kBlk, 0, bar);
        if ((kt & 3) == 0 || i == 0)
          bulk_load_if(one, st + C::kBBytes + C::kProducts * 512, p.sfx + static_cast<size_t>(kt >> 2) * 512u, 512, bar);
        st += C::kStageBytes;
        bar += 8;
        if (++s == C::kStages) { s = 0; ph ^= 1u; st = st0; bar = smem_u32(full); }
      }
    }
  } else if (warp == 1) {
    const uint32_t one = elect_one();
    const uint32_t ring_addr = smem_u32(ring);
    const uint64_t ad0 = sdesc_sw128_kmajor(ring_addr);
    const uint64_t bd0 = sdesc_sw128_kmajor(FUSED ? smem_u32(xcodes) : ring_addr + C::kProducts * C::kABytes);
    const uint64_t sd0 = sdesc_plain_rows16(ring_addr + C::kSfOff);
    uint64_t so = 0;                                       // the stage's offset in descriptor units
    uint64_t bo = 0, xs = sdesc_plain_rows16(smem_u32(xsf));
    uint32_t bar = smem_u32(empty);
    int s = 0, set = 2, i = 0;
    uint32_t ph = 0, acc = 0;
    grid_dep_wait();
    bool ok = !FUSED || mbar_wait(x_ready, 0, p.err, KQ_DEV_ERR_TIMEOUT_FULL, p.wait_ns);
    for (; i < n_kt && ok; ++i) {
      if (LONG && i > 0 && i % kSum == 0) {
        commit_if<false>(one, smem_u32(acc_full));
        ok = mbar_wait(acc_free, static_cast<uint32_t>(i / kSum - 1) & 1u, p.err, KQ_DEV_ERR_TIMEOUT_ACC, p.wait_ns);
        if (!ok) break;
        acc = 0;
      }
      ok = mbar_wait(&full[s], ph, p.err, KQ_DEV_ERR_TIMEOUT_FULL, p.wait_ns);
      if (!ok) break;
      tc_fence_after();
      const int kt = kt0 + i;
      if ((kt & 3) == 0 || i == 0) {
        set = set == 2 ? 0 : set + 1;
        const uint32_t f = tmem + C::kSfCol + 16u * set;
#pragma unroll
        for (int j = 0; j < C::kProducts; ++j) scale_cp_if<false>(one, f + 4 * j, sd0 + so + 32 * j);
        scale_cp_if<false>(one, f + 4 * C::kProducts, FUSED ? xs : sd0 + so + 32 * C::kProducts);
        xs += 32;
      }
      const uint32_t id = static_cast<uint32_t>(kt) & 3u;
      const uint32_t idesc = idesc_mxf8(128, BT, 0) | (id << 4) | (id << 29);
      const uint32_t f = (tmem + C::kSfCol + 16u * set) | (id << 30);
      const uint64_t b = bd0 + (FUSED ? bo : so);
      // all four K steps of 32, the last k-tile's too: what lies past K was filled with zeros
#pragma unroll
      for (int j = 0; j < C::kProducts; ++j)
#pragma unroll
        for (int kk = 0; kk < 4; ++kk)
          mma_mxf8_if<false>(one, tmem + 64 * j, ad0 + so + (j * C::kABytes >> 4) + 2 * kk, b + 2 * kk, idesc, f + 4 * j,
                             f + 4 * C::kProducts, kk == 0 ? acc : 1u);
      commit_if<false>(one, bar);
      acc = 1;
      bo += C::kBBytes >> 4;
      so += C::kStageBytes >> 4;
      bar += 8;
      if (++s == C::kStages) { s = 0; ph ^= 1u; so = 0; bar = smem_u32(empty); }
    }
    commit_if<false>(one, smem_u32(ok ? acc_full : mma_done));
    if (!ok) {
      drain_after(full, C::kStages, i, n_kt, p.wait_ns);
      mbar_wait(mma_done, 0, nullptr, 0u, p.wait_ns);
    }
  }
  const int q = warp & 3;                                  // TMEM lane quadrant
  const uint32_t tb = tmem + (static_cast<uint32_t>(32 * q) << 16);
  uint8_t* tile = ring + (C::kOwnPart ? 0 : C::kPartBytes);             // the ring is read by then
  const bool epi = warp >= 2 && warp < 6;
  bool ok = true;
  [[maybe_unused]] float sum[C::kProducts][BT];            // LONG
  if (epi || (FUSED && warp > 6)) {
    grid_dep_wait();                                       // bf16 tokens; outputs are written after the grid before
    if (FUSED) {
      if (blockIdx.x == 0 && rank == 0 && threadIdx.x == 64) *p.err = 0u;
      encode_share<BT>(p, tokens, kt0, n_kt, xcodes, xsf, epi ? warp - 2 : warp - 3, lane);
      fence_async_smem();
      mbar_arrive(x_ready);
    }
  }
  if (epi) {
    if (GATED && !FUSED && !LONG && p.out == 2 && blockIdx.x == 0 && rank == 0 && threadIdx.x == 64) *p.oerr = 0u;
    auto come = [&](int piece) {
      ok = __all_sync(0xffffffffu, mbar_wait(acc_full, static_cast<uint32_t>(piece) & 1u, p.err, KQ_DEV_ERR_TIMEOUT_ACC, p.wait_ns));
      tc_fence_after();
      return ok;
    };
    if constexpr (LONG) {
      for (int k = 0; k * kSum < n_kt && come(k); ++k) {
#pragma unroll
        for (int j = 0; j < C::kProducts; ++j) add_columns<BT>(tb + 64 * j, k > 0, sum[j]);
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(acc_free);
      }
    } else {
      come(0);
    }
    if (!ok) *bad = 1u;
  }
  // 16 tokens of this thread's feature, from token c on
  auto take = [&](int c, uint32_t (&r)[C::kProducts][16]) {
#pragma unroll
    for (int j = 0; j < C::kProducts; ++j) {
      if constexpr (LONG) {
#pragma unroll
        for (int t = 0; t < 16; ++t) r[j][t] = __float_as_uint(sum[j][c + t]);
      } else {
        tmem_ld_32x32b_x16(tb + 64 * j + c, r[j]);
      }
    }
    if constexpr (!LONG) tmem_ld_wait();
  };
  constexpr int kUnroll = LONG ? BT / 16 : 1;              // registers are not indexed
  if (splits > 1) {
    // tokens go by fours; the share of split d: fours [Q d / splits, Q (d + 1) / splits)
    const int Q = (tokens + 3) / 4, cap = (Q + splits - 1) / splits;
    __syncwarp();
    if (C::kOwnPart) cluster_wait();
    else cluster_sync();                                   // every CTA's ring has been consumed
    if (epi) {
      const uint32_t mine = smem_u32(part) + 16u * static_cast<uint32_t>(rank * C::kProducts * cap * 128 + 32 * q + lane);
      int d = 0, q0 = 0, q1 = Q / splits;
      uint32_t at = mapa_shared(mine, 0);
#pragma unroll kUnroll
      for (int c = 0; c < (LONG ? BT : tokens); c += 16) {
        if (LONG && c >= tokens) break;
        uint32_t r[C::kProducts][16];
        take(c, r);
#pragma unroll
        for (int t = 0; t < 4; ++t) {
          const int four = c / 4 + t;
          if (four >= Q) break;
          while (four >= q1) {
            ++d;
            q0 = q1;
            q1 = Q * (d + 1) / splits;
            at = mapa_shared(mine, static_cast<uint32_t>(d));
          }
#pragma unroll
          for (int j = 0; j < C::kProducts; ++j)
            st_shared_cluster_v4(at + 2048u * static_cast<uint32_t>(j * cap + four - q0), r[j][4 * t], r[j][4 * t + 1],
                                 r[j][4 * t + 2], r[j][4 * t + 3]);
        }
      }
    }
    if (!ok && lane < splits) st_shared_cluster_u32(mapa_shared(smem_u32(const_cast<uint32_t*>(bad)), lane), 1u);
    __syncwarp();
    cluster_sync();
    if (epi) {
      ok = *bad == 0;
      const int qs = Q * rank / splits, qe = Q * (rank + 1) / splits;
      // up to four fours to a call of store, which the 8-bit output makes a meeting of the warps
      constexpr int F = BT <= 16 ? 1 : 4;
      for (int four = qs; four < qe; four += F) {
        float v[C::kProducts][4 * F] = {};
        for (int s = 0; s < splits; ++s)
#pragma unroll
          for (int j = 0; j < C::kProducts; ++j)
#pragma unroll
            for (int f = 0; f < F; ++f) {
              if (f > 0 && four + f >= qe) break;
              const float4 w = part[((s * C::kProducts + j) * cap + four + f - qs) * 128 + 32 * q + lane];
              v[j][4 * f] += w.x; v[j][4 * f + 1] += w.y; v[j][4 * f + 2] += w.z; v[j][4 * f + 3] += w.w;
            }
        if (GATED) gate<ACT, 4 * F>(p.out, v[0], v[C::kProducts - 1], v[0]);
        store<4 * F, GATED && !FUSED && !LONG>(p, v[0], 4 * four, ok ? min(min(4 * F, 4 * (qe - four)), tokens - 4 * four) : 0, n0, q, lane, top, tile, bad);
      }
    }
  } else if (epi) {
#pragma unroll kUnroll
    for (int c = 0; c < (LONG ? BT : tokens); c += 16) {
      if (LONG && c >= tokens) break;
      uint32_t r[C::kProducts][16];
      take(c, r);
      float v[C::kProducts][16];
#pragma unroll
      for (int j = 0; j < C::kProducts; ++j)
#pragma unroll
        for (int t = 0; t < 16; ++t) v[j][t] = __uint_as_float(r[j][t]);
      if (GATED) gate<ACT, 16>(p.out, v[0], v[C::kProducts - 1], v[0]);
      store<16, GATED && !FUSED && !LONG>(p, v[0], c, ok ? min(16, tokens - c) : 0, n0, q, lane, top, tile, bad);
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, C::kTmemCols);
  }
}

template <int BT, bool GATED, bool FUSED>
cudaLaunchConfig_t rows_config(const MmParams& p, int splits, cudaLaunchAttribute (&attr)[2], cudaStream_t st) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(cdiv(p.N, 128)), 1, static_cast<unsigned>(splits));
  cfg.blockDim = dim3(Rows<BT, GATED, FUSED>::kThreads);
  cfg.dynamicSmemBytes = Rows<BT, GATED, FUSED>::smem(static_cast<int>(cdiv(cdiv(p.K, kBlk), splits)));
  cfg.stream = st;
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = 1;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = static_cast<unsigned>(splits);
  cfg.attrs = attr;
  cfg.numAttrs = splits > 1 ? 2 : 1;
  return cfg;
}

// Clusters of s CTAs of this kernel that the device holds at once (fewer than SMs / s, since a
// cluster stays within a GPC: 15 of 8 CTAs on 148 SMs). Asked once per device, with the most
// shared memory that the kernel takes.
template <int BT, int ACT, bool FUSED>
int max_clusters(int s, int device) {
  static std::atomic<int> known[kMaxDevices][kMaxSplits + 1];
  if (device >= kMaxDevices) return 0;
  int n = known[device][s].load(std::memory_order_relaxed);
  if (n > 0) return n - 1;
  MmParams p = {};
  p.N = 128;
  p.K = kBlk * s * (FUSED ? Rows<BT, ACT >= 0, FUSED>::kMaxShare : 1);
  cudaLaunchAttribute attr[2];
  cudaLaunchConfig_t cfg = rows_config<BT, ACT >= 0, FUSED>(p, s, attr, nullptr);
  cfg.attrs = attr + 1;
  cfg.numAttrs = 1;
  auto fn = k_rows_mm<BT, ACT, FUSED, false>;
  if (cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(cfg.dynamicSmemBytes)) !=
          cudaSuccess ||
      cudaOccupancyMaxActiveClusters(&n, fn, &cfg) != cudaSuccess) {
    cudaGetLastError();
    n = 0;
  }
  known[device][s].store(n + 1, std::memory_order_relaxed);
  return n;
}

// Splits of K for `tiles` tiles of `kt` k-tiles: the number that leaves a CTA the fewest k-tiles
// while all CTAs run at once, one per SM. A split has to take off more than the exchange costs.
template <int BT, int ACT, bool FUSED>
int rows_splits(int64_t tiles, int64_t kt, int sms, int device) {
  int best = 1;
  int64_t cost = cdiv(tiles, sms) * kt;
  for (int s = 2; s <= kMaxSplits && tiles * s <= sms && kt >= 2 * s; ++s) {
    const int64_t c = cdiv(kt, s) + 4;
    if (c < cost && tiles <= max_clusters<BT, ACT, FUSED>(s, device)) { best = s; cost = c; }
  }
  return best;
}

template <int BT, int ACT, bool FUSED>
bool try_rows(const MmParams& p, const Device& d, cudaStream_t st, cudaError_t* e) {
  using C = Rows<BT, ACT >= 0, FUSED>;
  const int64_t kt = cdiv(p.K, kBlk);
  const int splits = rows_splits<BT, ACT, FUSED>(cdiv(p.N, 128), kt, d.sms, d.device);
  auto fn = k_rows_mm<BT, ACT, FUSED, false>;
  if (!FUSED && p.out == 0 && cdiv(kt, splits) > sum_tiles(ACT >= 0)) fn = k_rows_mm<BT, ACT, FUSED, !FUSED>;
  *e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize,
                            static_cast<int>(C::smem(FUSED ? C::kMaxShare : 0)));
  if (*e != cudaSuccess) return true;
  // Encoding on the way in adds 0.8 us to the product for 4 blocks of a CTA, 1.3 for 32, 1.7 for 64
  // and 2.5 for 128 (512 -> 512, 1 to 32 tokens), a kernel of its own 1.6 and a launch, which costs
  // the host more than 2 us: one round of blocks at most.
  if (FUSED && (cdiv(kt, splits) > C::kMaxShare || cdiv(kt, splits) * p.M > kEncRound)) return false;
  cudaLaunchAttribute attr[2];
  const cudaLaunchConfig_t cfg = rows_config<BT, ACT >= 0, FUSED>(p, splits, attr, st);
  *e = cudaLaunchKernelEx(&cfg, fn, p);
  return true;
}

template <int BT, bool FUSED>
bool try_rows_g(const MmParams& p, bool gated, const Device& d, cudaStream_t st, cudaError_t* e) {
  if (!gated) return try_rows<BT, -1, FUSED>(p, d, st, e);
  return p.act == 0 ? try_rows<BT, 0, FUSED>(p, d, st, e) : try_rows<BT, 1, FUSED>(p, d, st, e);
}

}  // namespace

int rows_token_tile(int M) { return M <= 16 ? 16 : M <= 32 ? 32 : 64; }

cudaError_t launch_rows_mm(const MmParams& p, bool gated, const Device& d, cudaStream_t st) {
  cudaError_t e = cudaSuccess;
  switch (rows_token_tile(p.M)) {
    case 16: try_rows_g<16, false>(p, gated, d, st, &e); break;
    case 32: try_rows_g<32, false>(p, gated, d, st, &e); break;
    default: try_rows_g<64, false>(p, gated, d, st, &e); break;
  }
  return e;
}

bool try_rows_fused(const MmParams& p, bool gated, const Device& d, cudaStream_t st, cudaError_t* e) {
  if (p.M > 32) return false;
  return p.M <= 16 ? try_rows_g<16, true>(p, gated, d, st, e) : try_rows_g<32, true>(p, gated, d, st, e);
}

}  // namespace fp8
}  // namespace kq
