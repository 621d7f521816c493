// Block-scaled 8-bit matrix product on the 5th-generation tensor cores, for many tokens
// (fp8_rows.cu has the product for few, and the formulas).
//
// k_mm_pair: 256 tokens x BN weight rows per pair of CTAs (gated: BN = 256, 128 of the gate and the
// same 128 of up, so that both halves of an output meet in one thread). The two CTAs of a cluster
// run one MMA of M = 256 (cta_group::2): each stages its own 128 tokens and half of the weight
// rows, 32 KB per 128-element k-tile of 256 x 256 instead of the 48 KB that a 128 x 256 tile of
// one CTA would need. The MMAs of such a k-tile take 512 cycles, so a CTA pulls 64 bytes a cycle,
// the most that an SM gets from L2. Persistent, one pair per two SMs. Warp roles:
//   warps 0, 10  TMA producers in each CTA, of the tokens and of the weights; all loads of a
//              stage, the peer's too, complete on the first CTA's barrier.
//   warp 1     TMEM allocator; in the first CTA the MMA issuer for both.
//   warps 2-9  epilogue: thread = token, two warps share a TMEM lane quadrant and take half of
//              the columns each and write them through staging buffers in whole pieces of rows.
// TMEM holds two accumulators and the scales behind them. Up to BN = 192 they are apart, and one
// tile's epilogue runs beside the next tile's MMAs. Two of 256 columns overlap in 64 (0 .. 255
// and 192 .. 447): the epilogue reads the shared 64 columns first, and the next tile's MMAs start
// when those are out, some 1800 cycles after the last MMA.
//
// LONG: fp32 outputs of more k-tiles than sum_tiles. A tile's pieces take the two accumulators in turn, as
// tiles do, and the epilogue adds them in registers.
//
// A wait that runs out ends the kernel as in k_rows_mm: the MMA issuer waits for its MMAs and for the
// loads of both CTAs that are under way, an epilogue warp stores nothing from the tile whose
// accumulators did not come, frees none and leaves.
//
// Where tiles are fewer than pairs of SMs, two or four pairs share K and exchange partial sums as in
// k_rows_mm (SPLIT).
//
// Bound by the tensor pipe and, repeated, by the power cap: 8192^3 361 us (3.0 PFLOP/s, nine tenths of
// twice the measured bf16 rate) in bursts, 431 us repeated at 1.2 GHz; 4096 x 1152 -> 4608 20.0 us
// (2.2 PFLOP/s), where set-up, the pause between tiles and the last epilogue are half the time;
// gated 4096 x 4096 -> 12288 273 us (3.0 PFLOP/s), with GELU 287. With few k-tiles GELU's epilogue,
// erfc for 64 values a thread, takes longer than the MMAs: 4096 x 1152 -> 4608 35 us, with GELU 72.
#include <cuda_bf16.h>

#include <atomic>

#include "fp8.cuh"
#include "sm100_fp8.cuh"

namespace kq {
namespace fp8 {

namespace {

template <int BN>
struct Pair {
  static constexpr bool kShared = BN == 256;
  static constexpr int kStages = BN == 256 ? 5 : 6;
  static constexpr uint32_t kATile = 128 * 128;
  static constexpr uint32_t kBTile = BN / 2 * 128;
  static constexpr uint32_t kStageBytes = kATile + kBTile;           // tokens, weight rows
  static constexpr int kWAtoms = BN == 128 ? 1 : 2;                  // scale atoms of the weight rows
  static constexpr uint32_t kSfBytes = (1 + kWAtoms) * 512;
  static constexpr uint32_t kStgBytes = 4096;                        // a warp's 32 rows x 128 bytes
  static constexpr uint32_t kRingOff = 1024;
  static constexpr uint32_t kStgOff = kRingOff + kStages * kStageBytes;
  static constexpr uint32_t kSfOff = kStgOff + 8 * kStgBytes;
  static constexpr uint32_t kTopOff = kSfOff + kStages * kSfBytes;   // uint32 [2 halves][128 rows]
  static constexpr uint32_t kSmem = 1024 + kTopOff + 1024;
  static constexpr uint32_t kAccStride = kShared ? 192 : BN;
  // Scale sets of 12 columns (tokens 4, weight rows 8), used in turn by the atoms. A set comes
  // round after kSets >= kStages atoms, so after kStages k-tiles at least: its last MMAs have
  // freed the stage that the new atom landed in.
  static constexpr uint32_t kSfCol = kAccStride + BN, kSfSet = 12;
  static constexpr int kSets = kStages;
  static constexpr int kThreads = 352;
  static_assert(kSmem <= 232448 && kSfCol + kSets * kSfSet <= 512, "shared memory, TMEM");
  static_assert(kStageBytes % 1024 == 0, "swizzle atoms");
};

// Tile order: groups of 8 row tiles, row tile fastest, so that the pairs at work share a few
// row tiles and a few column tiles in L2.
__device__ __forceinline__ void pair_tile(int tile, int MT, int NT, int& mt, int& nt) {
  const int per = 8 * NT, g = tile / per, r = tile - g * per;
  const int gm = min(8, MT - g * 8);
  mt = g * 8 + r % gm;
  nt = r / gm;
}

// Writes W words (64 or 128 bytes) of each of a warp's 32 rows: through
// a swizzled staging buffer, so that a store instruction covers whole 64- or 128-byte pieces of
// rows. (TMA stores of the same boxes compete with the operand loads for the TMA unit: the fc1
// product of 4096 x 1152 -> 4608 took 33 us with them.) `col` and `pitch` in bytes; `cols` bytes
// of the row exist from col on, `rows` rows from this warp's first.
template <int W>
__device__ __forceinline__ void put_rows(const uint32_t (&w)[W], uint8_t* stg, uint8_t* out, int64_t pitch, int cols,
                                         int rows, int lane) {
  constexpr int kChunks = W / 4;                                     // 16-byte chunks per row: 4 or 8
  constexpr int kStep = 32 / kChunks;                                // rows per store instruction
  __syncwarp();                                                      // the last call's reads are done
#pragma unroll
  for (int c = 0; c < kChunks; ++c) {
    const int sw = kChunks == 8 ? c ^ (lane & 7) : c ^ ((lane >> 1) & 3);
    *reinterpret_cast<uint4*>(stg + lane * (16 * kChunks) + 16 * sw) =
        make_uint4(w[4 * c], w[4 * c + 1], w[4 * c + 2], w[4 * c + 3]);
  }
  __syncwarp();
  const int c = lane % kChunks;
  if (16 * c >= cols) return;
  uint4 v[kChunks];
#pragma unroll
  for (int i = 0; i < kChunks; ++i) {
    const int r = i * kStep + lane / kChunks;
    const int sw = kChunks == 8 ? c ^ (r & 7) : c ^ ((r >> 1) & 3);
    v[i] = *reinterpret_cast<const uint4*>(stg + r * (16 * kChunks) + 16 * sw);
  }
#pragma unroll
  for (int i = 0; i < kChunks; ++i) {
    const int r = i * kStep + lane / kChunks;
    if (r < rows) *reinterpret_cast<uint4*>(out + r * pitch + 16 * c) = v[i];
  }
}

// CH values (32 or 64) of each row from column x on, as fp32 or bf16; y: the warp's first row.
template <int CH>
__device__ __forceinline__ void put_values(const MmParams& p, const float (&v)[CH], uint8_t* stg, int x, int y, bool ok,
                                           int lane) {
  const int rows = ok ? min(32, p.M - y) : 0;
  const int64_t at = static_cast<int64_t>(y) * p.ldy + x;
  if (p.out == 1) {
    uint32_t w[CH / 2];
#pragma unroll
    for (int i = 0; i < CH / 2; ++i) {
      const __nv_bfloat162 b = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t*>(&b);
    }
    put_rows(w, stg, static_cast<uint8_t*>(p.y) + 2 * at, 2 * p.ldy, 2 * (p.N - x), rows, lane);
  } else {
#pragma unroll
    for (int h = 0; h < CH; h += 32) {
      uint32_t w[32];
#pragma unroll
      for (int i = 0; i < 32; ++i) w[i] = __float_as_uint(v[h + i]);
      put_rows(w, stg, static_cast<uint8_t*>(p.y) + 4 * (at + h), 4 * p.ldy, 4 * (p.N - x - h), rows, lane);
    }
  }
}

// Outputs 64 half .. 64 half + 63 of gated tile nt, one token per thread (token m0 + lane). `ok`, the
// same in all lanes: the sums are there; returns whether this is so in the warps that it met.
__device__ __forceinline__ bool put_gated(const MmParams& p, const float (&v)[64], uint8_t* stg, uint32_t* top, int nt,
                                          int half, int q, int m0, bool ok, int lane) {
  const int n0 = nt * 128 + 64 * half;
  if (p.out != 2) {
    put_values(p, v, stg, n0, m0, ok, lane);
    return ok;
  }
  // a block is the 128 outputs of a token in this tile: its largest value from both halves
  uint32_t a = 0;
#pragma unroll
  for (int i = 0; i < 64; ++i)
    if (n0 + i < p.N) a = max(a, abs_bits(v[i]));
  if (!ok) a = ~0u;                                                  // no magnitude
  top[128 * half + 32 * q + lane] = a;
  asm volatile("bar.sync %0, 64;" ::"r"(1 + q) : "memory");
  a = max(a, top[128 * (half ^ 1) + 32 * q + lane]);
  asm volatile("bar.sync %0, 64;" ::"r"(1 + q) : "memory");
  if (a == ~0u) return false;
  const uint32_t byte = scale_byte(a);
  const float is = inv_scale(byte);
  uint32_t w[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) w[i] = e4m3x4(v[4 * i] * is, v[4 * i + 1] * is, v[4 * i + 2] * is, v[4 * i + 3] * is);
  put_rows(w, stg, p.ocodes + static_cast<int64_t>(m0) * p.N + n0, p.N, p.N - n0, min(32, p.M - m0), lane);
  if (half == 0 && m0 + lane < p.M) p.osf[sf_offset(m0 + lane, nt, p.okatoms)] = static_cast<uint8_t>(byte);
  return true;
}

// ACT: -1 plain, 0 SiLU-gated, 1 GELU-gated. SPLIT: K is shared by the 2 or 4 pairs of a cluster.
template <int BN, int ACT, bool SPLIT, bool LONG>
__global__ void __launch_bounds__(Pair<BN>::kThreads, 1) k_mm_pair(const __grid_constant__ MmParams p) {
  using C = Pair<BN>;
  constexpr bool GATED = ACT >= 0;
  constexpr int kBN = GATED ? BN / 2 : BN;                           // output columns of a tile
  constexpr int kSum = sum_tiles(GATED);
  static_assert(!GATED || (BN == 256 && !SPLIT), "an 8-bit block is the 128 outputs of a gated tile");
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(align_up(reinterpret_cast<uintptr_t>(smem_raw), 1024));
  uint64_t* full = reinterpret_cast<uint64_t*>(smem);                // used in the first CTA
  uint64_t* empty = full + C::kStages;
  uint64_t* acc_full = empty + C::kStages;
  uint64_t* acc_free = acc_full + 2;                                 // used in the first CTA
  uint64_t* mma_done = acc_free + 2;                                 // in the first CTA, after a wait ran out
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(mma_done + 1);
  volatile uint32_t* bad = tmem_slot + 1;                            // SPLIT: sums of this CTA's outputs are missing
  uint8_t* ring = smem + C::kRingOff;
  uint8_t* sfring = smem + C::kSfOff;
  uint32_t* top = reinterpret_cast<uint32_t*>(smem + C::kTopOff);

  const int warp = warp_index(), lane = threadIdx.x & 31;
  const uint32_t crank = cluster_ctarank(), rank = crank & 1u, lead = crank & ~1u;
  const int splits = SPLIT ? p.splits : 1, split = static_cast<int>(crank >> 1);
  const uint16_t both = static_cast<uint16_t>(3u << lead);           // the pair's CTAs in the cluster
  const int MT = static_cast<int>(cdiv(p.M, 256)), NT = static_cast<int>(cdiv(p.N, kBN)), T = MT * NT;
  const int KT = static_cast<int>(cdiv(p.K, kBlk));
  const int kt0 = SPLIT ? KT * split / splits : 0, kt1 = SPLIT ? KT * (split + 1) / splits : KT;
  const int first = static_cast<int>(blockIdx.x) / (2 * splits), step = static_cast<int>(gridDim.x) / (2 * splits);

  if (threadIdx.x == 0) {
    for (int s = 0; s < C::kStages; ++s) { mbar_init(&full[s], 1); mbar_init(&empty[s], 1); }
    for (int b = 0; b < 2; ++b) { mbar_init(&acc_full[b], 1); mbar_init(&acc_free[b], 16); }
    mbar_init(mma_done, 1);
    *bad = 0;
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

  // Each warp of both CTAs frees an accumulator when it has read its columns (16 arrivals). Shared
  // columns are the second half's of accumulator 0 and the first half's of 1: their owner frees
  // the other accumulator after reading them, and its own after reading the rest; the first
  // half's share of accumulator 1's first turn is free from the start.
  const uint32_t free0 = mapa_shared(smem_u32(&acc_free[0]), lead);
  auto release = [&](int b) {
    tc_fence_before();
    __syncwarp();
    if (lane == 0) mbar_arrive_cluster(free0 + 8u * static_cast<uint32_t>(b));
  };
  // LONG: the sums of a tile, in the order of its pieces. v: the half's columns (gated: 64 of the gate,
  // then the same of up), the shared ones read first. False if a piece did not come.
  auto sum_tile = [&](int& local, float (&v)[BN / 2]) {
    const int q = warp & 3, half = (warp - 2) >> 2;
    for (int k0 = kt0; k0 < kt1; k0 += kSum, ++local) {
      const int buf = local & 1;
      const bool owner = half != buf, more = k0 > kt0;
      if (!__all_sync(0xffffffffu, mbar_wait(&acc_full[buf], (local >> 1) & 1, p.err, KQ_DEV_ERR_TIMEOUT_ACC, p.wait_ns)))
        return false;
      tc_fence_after();
      const uint32_t tb = tmem + static_cast<uint32_t>(buf) * C::kAccStride + (static_cast<uint32_t>(32 * q) << 16);
      if (!C::kShared) {
        add_columns<BN / 2>(tb + BN / 2 * half, more, v);
        release(buf);
      } else {
        // two runs of 64 columns: gate and up, or the halves of this half
        const uint32_t c0 = tb + (GATED ? 64 : 128) * half, c1 = c0 + (GATED ? 128 : 64);
        const bool swap = buf == 0 && (GATED || half == 1);
        if (swap) add_columns<64>(c1, more, v + 64);
        else add_columns<64>(c0, more, v);
        if (owner) release(buf ^ 1);
        if (swap) add_columns<64>(c0, more, v);
        else add_columns<64>(c1, more, v + 64);
        if (owner) release(buf);
      }
    }
    return true;
  };

  if (warp == 0 || warp == 10) {
    const bool tokens = warp == 0;
    const int w = GATED ? static_cast<int>(rank) : 0;                // gated: gate rows here, up rows there
    if (tokens || !p.dependent) grid_dep_wait();                     // (see k_rows_mm)
    if (tokens) grid_dep_launch();
    const uint32_t one = elect_one();
    const int ka = static_cast<int>(p.katoms), nb = static_cast<int>(cdiv(p.N, 128)) - 1;
    const int xb = static_cast<int>(cdiv(p.M, 128)) - 1;
    const CUtensorMap* map = tokens ? &p.tmap_x : &p.tmap_w[w];
    const uint32_t ring0 = smem_u32(ring) + (tokens ? 0 : C::kATile);
    const uint32_t sf0 = smem_u32(sfring) + (tokens ? 0 : 512);
    const uint32_t bar0 = mapa_shared(smem_u32(&full[0]), lead), mine0 = smem_u32(&full[0]);
    const uint32_t expect = tokens && rank == 0 ? one : 0u;
    const int64_t skip = tokens ? -1 : p.withhold;
    uint32_t off = 0, st = ring0, sf = sf0;
    int s = 0;
    uint32_t ph = 1;
    int64_t it = 0;
    bool ok = true;
    for (int tile = first; tile < T && ok; tile += step) {
      int mt, nt;
      pair_tile(tile, MT, NT, mt, nt);
      const int m0 = mt * 256 + 128 * static_cast<int>(rank);
      const int n0 = GATED ? nt * 128 : nt * BN + BN / 2 * static_cast<int>(rank);
      const int y = tokens ? m0 : n0;
      // scale atoms by row group; a group past the last (its results are not stored) takes the last
      const int xa = min(m0 / 128, xb) * ka, wa0 = (GATED ? nt : nt * BN / 128) * ka,
                wa1 = (GATED ? nt : min(nt * BN / 128 + 1, nb)) * ka;
      for (int kt = kt0; kt < kt1; ++kt, ++it) {
        if (it == C::kStages) grid_dep_wait();
        if (it >= C::kStages && !mbar_wait(&empty[s], ph, p.err, KQ_DEV_ERR_TIMEOUT_EMPTY, p.wait_ns)) {
          ok = false;
          break;
        }
        const bool atom = (kt & 3) == 0 || (SPLIT && kt == kt0);
        expect_tx_if(expect, mine0 + off, 2 * (C::kStageBytes + (atom ? C::kSfBytes : 0u)));
        tma_load_pair_if(it == skip ? 0u : one, st, map, kt * kBlk, y, bar0 + off);
        if (atom) {
          if (tokens) {
            tma_load_pair_if(one, sf, &p.tmap_sfx, 0, xa + (kt >> 2), bar0 + off);
          } else {
            tma_load_pair_if(one, sf, &p.tmap_sfw[0], 0, wa0 + (kt >> 2), bar0 + off);
            if (C::kWAtoms > 1) tma_load_pair_if(one, sf + 512, &p.tmap_sfw[GATED ? 1 : 0], 0, wa1 + (kt >> 2), bar0 + off);
          }
        }
        st += C::kStageBytes;
        sf += C::kSfBytes;
        off += 8;
        if (++s == C::kStages) { s = 0; ph ^= 1u; off = 0; st = ring0; sf = sf0; }
      }
    }
  } else if (warp == 1) {
    if (rank == 0) {
      const uint32_t one = elect_one();
      const uint64_t ad0 = sdesc_sw128_kmajor(smem_u32(ring)), bd0 = sdesc_sw128_kmajor(smem_u32(ring) + C::kATile);
      const uint64_t sd0 = sdesc_plain_rows16(smem_u32(sfring));
      uint64_t so = 0, sd = sd0;
      uint32_t bar = smem_u32(empty), f = tmem + C::kSfCol + C::kSfSet * (C::kSets - 1);
      int s = 0, local = 0, set = C::kSets - 1;
      uint32_t ph = 0;
      const int64_t per = kt1 - kt0;
      int64_t before = 0, stop = -1;                                 // k-tiles of earlier tiles; taken when a wait ran out
      grid_dep_wait();
      for (int tile = first; tile < T && stop < 0; tile += step, before += per) {
        uint32_t shift = 0;                                          // a tile may start in mid-atom
        if (BN % 128 != 0) {
          int mt, nt;
          pair_tile(tile, MT, NT, mt, nt);
          shift = static_cast<uint32_t>(nt * BN % 128) / 32u;
        }
        for (int k0 = kt0, k1; k0 < kt1 && stop < 0; k0 = k1, ++local) {
          k1 = LONG ? min(k0 + kSum, kt1) : kt1;                       // a piece; not LONG: the tile
          const int buf = local & 1;
          const int since = C::kShared && buf ? local - 1 : local - 2;  // pieces since acc_free[buf]'s first phase
          if (since >= 0 && !mbar_wait_cluster(&acc_free[buf], (since >> 1) & 1, p.err, KQ_DEV_ERR_TIMEOUT_ACC, p.wait_ns)) {
            stop = before + k0 - kt0;
            break;
          }
          tc_fence_after();
          const uint32_t d = tmem + static_cast<uint32_t>(buf) * C::kAccStride;
          uint32_t acc = 0;
          for (int kt = k0; kt < k1; ++kt) {
            if (!mbar_wait(&full[s], ph, p.err, KQ_DEV_ERR_TIMEOUT_FULL, p.wait_ns)) {
              stop = before + kt - kt0;
              break;
            }
            tc_fence_after();
            const uint32_t id = static_cast<uint32_t>(kt) & 3u;
            if (id == 0 || (SPLIT && kt == kt0)) {
              set = set + 1 == C::kSets ? 0 : set + 1;
              f = tmem + C::kSfCol + C::kSfSet * set;
              scale_cp_if<true>(one, f, sd);
              scale_cp_if<true>(one, f + 4, sd + 32);
              if (C::kWAtoms > 1) scale_cp_if<true>(one, f + 8, sd + 64);
            }
            const uint32_t idesc = idesc_mxf8(256, BN, 0) | (id << 4) | (id << 29);
            const uint32_t fa = f | (id << 30);
            // all four K steps of 32, the last k-tile's too: what lies past K was filled with zeros
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)
              mma_mxf8_if<true>(one, d, ad0 + so + 2 * kk, bd0 + so + 2 * kk, idesc, fa, fa + 4 + shift, kk == 0 ? acc : 1u);
            commit_if<true>(one, bar, both);
            acc = 1;
            so += C::kStageBytes >> 4;
            sd += C::kSfBytes >> 4;
            bar += 8;
            if (++s == C::kStages) { s = 0; ph ^= 1u; so = 0; sd = sd0; bar = smem_u32(empty); }
          }
          if (stop < 0) commit_if<true>(one, smem_u32(&acc_full[buf]), both);
        }
      }
      if (stop >= 0) {
        // the barriers count the loads of both CTAs; the peer leaves after the cluster barrier below
        commit_if<true>(one, smem_u32(mma_done), static_cast<uint16_t>(1u << lead));
        drain_after(full, C::kStages, stop, cdiv(T - first, step) * per, p.wait_ns);
        mbar_wait(mma_done, 0, nullptr, 0u, p.wait_ns);
      }
    }
  } else {
    grid_dep_wait();
    const int q = warp & 3, half = (warp - 2) >> 2;
    uint8_t* stg = smem + C::kStgOff + static_cast<uint32_t>(warp - 2) * C::kStgBytes;
    if (GATED && p.out == 2 && blockIdx.x == 0 && threadIdx.x == 64) *p.oerr = 0u;
    if ((!SPLIT || LONG) && C::kShared && half == 0 && lane == 0) mbar_arrive_cluster(free0 + 8);
    int local = 0;
    for (int tile = SPLIT ? T : first; tile < T; tile += step, ++local) {
      int mt, nt;
      pair_tile(tile, MT, NT, mt, nt);
      const int m0 = mt * 256 + 128 * static_cast<int>(rank) + 32 * q;
      if constexpr (LONG) {
        float v[BN / 2];
        if (!sum_tile(local, v)) break;
        --local;                                                     // it counted the tile's last piece
#pragma unroll
        for (int c = 0; c < kBN / 2; c += 32) {
          float w[32];
          if constexpr (GATED) {
            gate<ACT, 32>(0, v + c, v + 64 + c, w);
          } else {
#pragma unroll
            for (int i = 0; i < 32; ++i) w[i] = v[c + i];
          }
          const int n0 = nt * kBN + kBN / 2 * half + c;
          if (n0 < p.N) put_values(p, w, stg, n0, m0, true, lane);
        }
        continue;
      }
      const int buf = local & 1;
      const bool owner = half != buf;
      bool ok = __all_sync(0xffffffffu, mbar_wait(&acc_full[buf], (local >> 1) & 1, p.err, KQ_DEV_ERR_TIMEOUT_ACC, p.wait_ns));
      if (!GATED && !ok) break;
      tc_fence_after();
      const uint32_t tb = tmem + static_cast<uint32_t>(buf) * C::kAccStride + (static_cast<uint32_t>(32 * q) << 16);
      if (!GATED) {
        // chunks of 64 (or 32) columns; the shared ones first: 192 .. 255 in the second half of
        // accumulator 0, 0 .. 63 in the first of accumulator 1
        constexpr int kCols = BN / 2, CH = kCols % 64 ? 32 : 64, kChunks = kCols / CH;
        const int n0 = nt * BN + kCols * half;
#pragma unroll 1
        for (int c = 0; c < kChunks; ++c) {
          const int col = CH * (C::kShared && buf == 0 && half == 1 ? kChunks - 1 - c : c);
          uint32_t r[CH / 32][32];
#pragma unroll
          for (int h = 0; h < CH / 32; ++h) tmem_ld_32x32b_x32(tb + kCols * half + col + 32 * h, r[h]);
          tmem_ld_wait();
          if (C::kShared && owner) release(c == 0 ? buf ^ 1 : buf);
          if (!C::kShared && c == kChunks - 1) release(buf);
          float v[CH];
#pragma unroll
          for (int i = 0; i < CH; ++i) v[i] = __uint_as_float(r[i >> 5][i & 31]);
          if (n0 + col < p.N) put_values(p, v, stg, n0 + col, m0, ok, lane);
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
        if (owner && ok) release(buf ^ 1);
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          uint32_t r[32];
          tmem_ld_32x32b_x32((buf == 0 ? g0 : u0) + 32 * c, r);
          tmem_ld_wait();
          if (owner && ok && c == 1) release(buf);
          float g[32], u[32];
#pragma unroll
          for (int i = 0; i < 32; ++i) {
            const float o = __uint_as_float(r[i]), f = v[32 * c + i];
            g[i] = buf == 0 ? o : f;
            u[i] = buf == 0 ? f : o;
          }
          gate<ACT, 32>(p.out, g, u, v + 32 * c);
        }
        ok = put_gated(p, v, stg, top, nt, half, q, m0, ok, lane);
        if (!ok) break;
      }
    }
  }
  if (SPLIT) {
    // The rows of lane quadrant q are finished by split q splits / 4 (2 or 4 splits): every split
    // stores its partial sums of them over that CTA's ring, as [split][quadrant][4 columns][row],
    // and its eight warps add them, 32 columns at a time, in the order of the splits.
    const bool epi = warp >= 2 && warp < 10;
    const int q = warp & 3, nq = 4 / splits;
    bool ok = true;
    [[maybe_unused]] float sum[BN / 2];                              // LONG
    if (epi) {
      if constexpr (LONG) {
        int local = 0;
        ok = sum_tile(local, sum);
      } else {
        ok = __all_sync(0xffffffffu, mbar_wait(&acc_full[0], 0, p.err, KQ_DEV_ERR_TIMEOUT_ACC, p.wait_ns));
        tc_fence_after();
      }
    }
    __syncwarp();
    cluster_sync();                                                  // every CTA's ring has been consumed
    if (epi) {
      const int dest = q / nq, half = (warp - 2) >> 2;
      const uint32_t at = mapa_shared(smem_u32(ring), 2u * static_cast<uint32_t>(dest) + rank) +
                          512u * static_cast<uint32_t>((split * nq + q - dest * nq) * (BN / 4)) +
                          16u * static_cast<uint32_t>(lane);
#pragma unroll(LONG ? BN / 64 : 1)
      for (int c = 0; c < BN / 2; c += 32) {
        uint32_t r[32];
        if constexpr (LONG) {
#pragma unroll
          for (int i = 0; i < 32; ++i) r[i] = __float_as_uint(sum[c + i]);
        } else {
          tmem_ld_32x32b_x32(tmem + (static_cast<uint32_t>(32 * q) << 16) + BN / 2 * half + c, r);
          tmem_ld_wait();
        }
#pragma unroll
        for (int j = 0; j < 8; ++j)
          st_shared_cluster_v4(at + 512u * static_cast<uint32_t>((BN / 2 * half + c) / 4 + j), r[4 * j], r[4 * j + 1],
                               r[4 * j + 2], r[4 * j + 3]);
      }
    }
    if (!ok && lane < 2 * splits) st_shared_cluster_u32(mapa_shared(smem_u32(const_cast<uint32_t*>(bad)), lane), 1u);
    __syncwarp();
    cluster_sync();
    if (epi) {
      ok = *bad == 0;
      const float4* part = reinterpret_cast<const float4*>(ring) + lane;
      int mt, nt;
      pair_tile(first, MT, NT, mt, nt);
      uint8_t* stg = smem + C::kStgOff + static_cast<uint32_t>(warp - 2) * C::kStgBytes;
#pragma unroll 1
      for (int u = warp - 2; u < nq * (BN / 32); u += 8) {
        const int qi = u % nq, c = u / nq * 32;
        float v[32];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          float4 t = part[(qi * (BN / 4) + c / 4 + j) * 32];
          for (int s = 1; s < splits; ++s) {
            const float4 w = part[((s * nq + qi) * (BN / 4) + c / 4 + j) * 32];
            t.x += w.x; t.y += w.y; t.z += w.z; t.w += w.w;
          }
          v[4 * j] = t.x; v[4 * j + 1] = t.y; v[4 * j + 2] = t.z; v[4 * j + 3] = t.w;
        }
        const int m0 = mt * 256 + 128 * static_cast<int>(rank) + 32 * (split * nq + qi);
        if (nt * BN + c < p.N) put_values(p, v, stg, nt * BN + c, m0, ok, lane);
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();              // the peer's MMAs, loads and arrivals that reach into this CTA are over
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_pair(tmem, 512);
  }
}

template <int BN, int ACT, bool SPLIT>
cudaLaunchConfig_t pair_config(int64_t clusters, int splits, cudaLaunchAttribute (&attr)[2], cudaStream_t st) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(2 * splits * clusters));
  cfg.blockDim = dim3(Pair<BN>::kThreads);
  cfg.dynamicSmemBytes = Pair<BN>::kSmem;
  cfg.stream = st;
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = static_cast<unsigned>(2 * splits);
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cfg;
}

template <int BN, int ACT, bool SPLIT>
cudaError_t launch_pair_kernel(const MmParams& p, int sms, cudaStream_t st) {
  auto fn = k_mm_pair<BN, ACT, SPLIT, false>;
  if (p.out == 0 && cdiv(cdiv(p.K, kBlk), SPLIT ? p.splits : 1) > sum_tiles(ACT >= 0)) fn = k_mm_pair<BN, ACT, SPLIT, true>;
  cudaError_t e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(Pair<BN>::kSmem));
  if (e != cudaSuccess) return e;
  const int64_t tiles = cdiv(p.M, 256) * cdiv(p.N, ACT >= 0 ? BN / 2 : BN);
  const int64_t clusters = SPLIT || tiles < sms / 2 ? tiles : sms / 2;
  cudaLaunchAttribute attr[2];
  const cudaLaunchConfig_t cfg = pair_config<BN, ACT, SPLIT>(clusters, SPLIT ? p.splits : 1, attr, st);
  return cudaLaunchKernelEx(&cfg, fn, p);
}

// Clusters of `splits` pairs that the device holds at once, one CTA per SM (a cluster stays within
// a GPC: 33 of 4 CTAs and 15 of 8 on 148 SMs). Asked once per device.
template <int BN>
int64_t max_pair_clusters(int splits, int device) {
  static std::atomic<int> known[kMaxDevices][2];
  if (device >= kMaxDevices) return 0;
  std::atomic<int>& k = known[device][splits / 4];
  int n = k.load(std::memory_order_relaxed);
  if (n > 0) return n - 1;
  auto fn = k_mm_pair<BN, -1, true, false>;
  cudaLaunchAttribute attr[2];
  cudaLaunchConfig_t cfg = pair_config<BN, -1, true>(1, splits, attr, nullptr);
  cfg.numAttrs = 1;
  if (cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(Pair<BN>::kSmem)) !=
          cudaSuccess ||
      cudaOccupancyMaxActiveClusters(&n, fn, &cfg) != cudaSuccess) {
    cudaGetLastError();
    n = 0;
  }
  k.store(n + 1, std::memory_order_relaxed);
  return n;
}

// Keeps in `best` the shape that takes the least time: ns per k-tile and per tile of a pair as
// measured with all SMs busy. Alone on its SMs a k-tile takes three quarters of that, which is what a
// split saves of each, and the exchange 4.4 us (200 x 12288 -> 512: 17.0 us in one piece, 10.5 in
// four; 128 x 4096 -> 4096: 8.6 and, in two, 10.5).
template <int BN>
void consider(int64_t tiles, int64_t kt, bool split, int64_t per_kt, int64_t per_tile, const Device& d, PairShape* best,
              int64_t* cost) {
  const int64_t plain = cdiv(tiles, d.sms / 2) * (per_kt * kt + per_tile);
  if (plain < *cost) { *cost = plain; *best = {BN, 1}; }
  for (int s = 2; split && s <= 4; s += 2) {
    if (kt < 2 * s || tiles * s > d.sms / 2) continue;
    const int64_t c = plain - (kt - cdiv(kt, s)) * per_kt * 3 / 4 + 4400;
    if (c < *cost && tiles <= max_pair_clusters<BN>(s, d.device)) { *cost = c; *best = {BN, s}; }
  }
}

}  // namespace

PairShape pair_shape(int M, int N, int K, bool gated, const Device& d) {
  PairShape best = {0, 1};
  if (M <= kRowsMaxM) return best;
  const int64_t kt = cdiv(K, kBlk), mt = cdiv(M, 256);
  int64_t cost = INT64_MAX;
  consider<256>(mt * cdiv(N, gated ? 128 : 256), kt, !gated, 340, 900, d, &best, &cost);
  if (gated) return best;
  consider<192>(mt * cdiv(N, 192), kt, true, 265, 550, d, &best, &cost);
  consider<128>(mt * cdiv(N, 128), kt, true, 200, 450, d, &best, &cost);
  return best;
}

template <int BN>
static cudaError_t launch_plain(const MmParams& p, int sms, cudaStream_t st) {
  return p.splits > 1 ? launch_pair_kernel<BN, -1, true>(p, sms, st) : launch_pair_kernel<BN, -1, false>(p, sms, st);
}

cudaError_t launch_pair(const MmParams& p, bool gated, int sms, cudaStream_t st) {
  if (gated) return p.act == 0 ? launch_pair_kernel<256, 0, false>(p, sms, st) : launch_pair_kernel<256, 1, false>(p, sms, st);
  switch (p.pairs) {
    case 256: return launch_plain<256>(p, sms, st);
    case 192: return launch_plain<192>(p, sms, st);
    default: return launch_plain<128>(p, sms, st);
  }
}

}  // namespace fp8
}  // namespace kq
