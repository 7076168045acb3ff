// tcgen05 product of two MXFP4 operands, dense and by experts:
//
//   out[token, n] = sum_k x[token, k] * w[n, k]  (+ bias[n]) (ReLU)
//
// The weight is the MMA's A operand (128 rows of n on the 128 TMEM lanes) and
// the tokens its N side: tokens are what a call has few or many of, and the
// MMA's N goes from 32 to 256 while its M stays 128, so one kernel serves a
// single token and long prompts.  It also makes the epilogue simple: a warp
// holds 32 consecutive n of one token in a register, so a plain store writes
// 32 consecutive outputs, and the bias is one value per thread.
//
//   warp 0      TMA producer: per 256 values of K the weight tile (128 rows x
//               128 bytes of codes), the token tile, both 128-byte swizzled, and
//               their scales into a ring of stages
//   warp 1      TMEM owner + MMA issuer: copies the stage's scales to TMEM
//               (tcgen05.cp), then one MMA per 64 values of K into an fp32
//               accumulator
//   warps 2 on  epilogue, two or four warps per TMEM lane quadrant that take turns
//               by 32 tokens: tcgen05.ld, bias, ReLU, rounding, and per token one
//               store of 32 consecutive outputs straight from the registers; in
//               the experts' form, whose rows are scattered, 32 x 32 outputs
//               through the warp's own shared memory and 16-byte stores (65
//               against 78 us for 64 experts, 32768 rows, 2048 x 1024).  One bulk
//               copy per token row took 1.7 times the time: a warp issues the
//               copies of its lanes one by one, ~130 cycles each
//
// More than 128 tokens run as CTA pairs (cta_group::2): 256 rows of the weight x
// 256 tokens per pair, each CTA loading its 128 rows and half of the tokens, so
// that a CTA reads 32 KB per 256 values of K instead of 48 KB -- one CTA's
// shared memory cannot feed 128 x 256 tiles of 4-bit MMAs (both operands
// written once and read once: 192 bytes a cycle against 128).  The pair's two
// accumulators of 256 columns overlap in 64 of them, which leaves room for the
// scales: the epilogue drains the shared columns first and hands them back.
// Tokens that are quantised within the call, and the experts' sorted rows, can be
// tiled by 224 instead: two accumulators of 224 columns leave room for the scales
// without overlapping (the rule: product_atom_shift).
//
// Measured: these MMAs (K = 64) alone run at 9.2 PFLOP/s (7.5 us per 1024 of K at 8192 x
// 4096, the epilogue taken out; the instruction's form with K = 96 is not used and was
// not measured); with the epilogue 8192 x 4096 x 4096 to bf16 takes 43 us (6.4
// PFLOP/s, L2 read at 14 TB/s), 8192^3 142 us (7.7, power-capped), K = 1024 to fp32
// 27.4 us (the output's 134 MB are 20).
//
// Few tokens and a long K: the sum over K is split over a cluster of S <= 8 CTAs.
// Each takes a run of K, writes its partial tile to the others' shared memory
// (CTA r sums rows r * 128 / S .. of n) and the sums are taken in the order of
// the CTAs, so a result does not depend on timing (the rule: pick_splits).
//
// A handful of tokens (FUSED): warps that are idle until an accumulator is done
// (in the experts' form all but four of the epilogue's, which then run ahead of
// the tile being drained) quantise the token rows of a stage themselves into the
// stage's shared memory, so that a decoding step's product is one launch without
// scratch; every CTA repeats that small work (the rules: product_fused,
// experts_fused).
//
// The gradient of the experts' weights (GROUPS) has both operands along the rows
// in expert order; every expert sums over its own run of them.
//
// Persistent CTAs walk the tiles.  In the experts' form a tile is (expert, rows
// of that expert, n); the row counts are only known on the GPU, so every CTA
// sums them up at its start.
#include <atomic>
#include <mutex>

#include "mx_internal.cuh"
#include "mx_quant.cuh"
#include "tc_common.cuh"

namespace imc {
namespace mx {
namespace {

using tc::BM;
using tc::wait_bar;

constexpr int KB = 256;                 // values of K per stage: 128 bytes of codes
constexpr int KSTEP = 64;               // values of K per MMA
constexpr int A_BYTES = BM * KB / 2;    // 16 KB
constexpr int MAX_EXPERTS = 1024;

__device__ int g_watchdog_mx;

// Epilogue warps: four per TMEM lane quadrant in the experts' form, whose tiles
// are short and whose rows are scattered, two otherwise (measured us with 8 / 16:
// 64 experts, 32768 rows, 2048 x 1024, sort apart, 73.0 / 64.9; dense 8192 x 4096 x
// 4096 43.3 / 44.2, K = 2048 26.9 / 28.6).
constexpr int epi_warps(bool experts) { return experts ? 16 : 8; }
constexpr int threads_of(bool experts) { return 64 + 32 * epi_warps(experts); }
constexpr int ROWS_BYTES = 2048;  // a warp's staged rows (experts' form)

template <int BN, bool PAIR, bool EXPERTS>
struct Form {
  static constexpr int BNW = PAIR ? 2 * BM : BM;               // weight rows of a tile
  static constexpr int B_ROWS = PAIR ? BN / 2 : BN;            // token rows a CTA loads
  static constexpr int B_BYTES = B_ROWS * KB / 2;
  static constexpr int B_ATOMS = (BN + 127) / 128;             // row atoms of a token tile
  static constexpr int ATOM_TOKENS = BN / B_ATOMS;             // m0 / this: a tile's first atom
  static constexpr int SA_BYTES = 2 * ATOM_BYTES, SB_BYTES = 2 * ATOM_BYTES * B_ATOMS;
  static constexpr int STAGE = A_BYTES + B_BYTES + SA_BYTES + SB_BYTES;
  static constexpr int STAGES = BN >= 128 ? (EXPERTS ? 5 : 6) : (BN > 32 ? 6 : (EXPERTS ? 7 : 8));
  // TMEM columns: two accumulators (ACC1 apart), then the scales of SETS stages
  static constexpr int SF_COLS = 8 + 8 * B_ATOMS;
  static constexpr bool OVERLAP = 2 * BN + 2 * SF_COLS > 512;
  static constexpr int SETS = BN > 128 ? 2 : STAGES;
  static constexpr int SF_COL0 = 512 - SETS * SF_COLS;
  static constexpr int ACC1 = OVERLAP ? 192 : BN;
  static_assert(ACC1 + BN <= SF_COL0, "TMEM");
  // chunks of 32 columns that hold what the two accumulators share
  static constexpr int SHARED = OVERLAP ? (BN - ACC1 + 31) / 32 : 0;
  static constexpr uint32_t TX = (PAIR ? 2 : 1) * STAGE;       // bytes a stage's barrier waits for
};

struct Ctl {
  uint64_t full[8], empty[8], accf[2], acce[2], drain, part;
  uint32_t tmem_base;
  int abort;
  // experts' form: tiles of the experts before e, first slot and first row of e
  int tiles_before[MAX_EXPERTS + 2], offset[MAX_EXPERTS + 2], start[MAX_EXPERTS + 1];
};

// After the stages: the epilogue warps' rows or (SPLIT) the cluster's partial sums.
template <int BN, bool EXPERTS, bool SPLIT>
constexpr int extra_bytes() {
  return SPLIT ? BN * BM * 4 : (EXPERTS ? epi_warps(true) * ROWS_BYTES : 0);
}
template <int BN, bool PAIR, bool EXPERTS, bool SPLIT>
constexpr int smem_bytes() {
  using F = Form<BN, PAIR, EXPERTS>;
  constexpr int bytes =
      1024 + F::STAGES * F::STAGE + extra_bytes<BN, EXPERTS, SPLIT>() + (int)sizeof(Ctl);
  static_assert(bytes <= 232448, "shared memory");
  return bytes;
}

// One tile: n rows n0.. of expert e's weight (this CTA's 128), token rows m0..
// of x (`rows` of them count).
struct Tile {
  int e, n0, m0, rows;
  int first;  // experts' form: place of row m0 in `order`
};

// wait_bar at cluster scope for the barriers that both CTAs of a pair signal.
template <bool PAIR>
__device__ __forceinline__ bool wait_any(uint64_t* bar, uint32_t parity, volatile int* abort,
                                         int site, int* watchdog) {
  if (!PAIR) return wait_bar(bar, parity, abort, site, watchdog);
  if (ptx::mbar_try_wait_cluster(bar, parity)) return true;
  const uint64_t t0 = ptx::globaltimer_ns();
  for (uint32_t it = 1;; ++it) {
    if (ptx::mbar_try_wait_cluster(bar, parity)) return true;
    if ((it & 127u) == 0) {
      if (*abort) return false;
      if (ptx::globaltimer_ns() - t0 > tc::kWaitLimitNs) {
        *abort = 1;
        atomicCAS(watchdog, 0, site);
        return false;
      }
    }
  }
}

__device__ __forceinline__ uint16_t half_bits(float v) { return __half_as_ushort(__float2half_rn(v)); }
__device__ __forceinline__ uint16_t bf16_bits(float v) {
  return __bfloat16_as_ushort(__float2bfloat16_rn(v));
}

// Stores one output of each of 32 tokens (`live` of them) per lane: token j's is
// at out[j * N], or in the experts' form at out[slot of lane j * N].  `in`: this
// lane's column exists.  For rows that 16-byte stores cannot reach.
template <bool EXPERTS, typename O, typename Bits>
__device__ __forceinline__ void store_tokens(O* out, int64_t N, int slot, int live, bool in,
                                             const uint32_t (&v)[32], Bits bits) {
  if (live == 32) {  // no branch per token
    O* o = out;
#pragma unroll
    for (int j = 0; j < 32; ++j) {
      if (EXPERTS) o = out + (int64_t)__shfl_sync(0xffffffffu, slot, j) * N;
      if (in) *o = bits(v[j]);
      o += N;
    }
  } else {
#pragma unroll
    for (int j = 0; j < 32; ++j) {
      if (j < live) {
        O* o = out + (EXPERTS ? (int64_t)__shfl_sync(0xffffffffu, slot, j) : (int64_t)j) * N;
        if (in) *o = bits(v[j]);
      }
    }
  }
}

// The same by rows: lane l's outputs (column l of the warp's 32) of the tokens go
// to `rows` (ROWS_BYTES: 32 tokens of 16-bit outputs or half of them in fp32),
// and 16 bytes of a row at a time to out, whose column 0 is the warp's; cols of
// the 32 exist.  N * sizeof(O) and out are multiples of 16.
template <typename O, typename Bits>
__device__ __forceinline__ void store_rows(O* out, int64_t N, int slot, int live, int cols,
                                           const uint32_t (&v)[32], uint8_t* rows, Bits bits) {
  constexpr int PER_ROW = 32 * (int)sizeof(O) / 16, AT_ONCE = 32 / PER_ROW;  // lanes, rows
  constexpr int HELD = ROWS_BYTES / (32 * (int)sizeof(O));                   // tokens in `rows`
  const int lane = threadIdx.x & 31, r0 = lane / PER_ROW, unit = lane % PER_ROW;
  const bool in = unit * (16 / (int)sizeof(O)) < cols;
  O* own = reinterpret_cast<O*>(rows) + lane;
#pragma unroll
  for (int h = 0; h < 32; h += HELD) {
#pragma unroll
    for (int j = 0; j < HELD; ++j) own[j * 32] = bits(v[h + j]);
    __syncwarp();
#pragma unroll
    for (int k = 0; k < HELD / AT_ONCE; ++k) {
      const int row = k * AT_ONCE + r0;
      const int64_t to = (int64_t)__shfl_sync(0xffffffffu, slot, h + row);
      if (in && h + row < live)
        *reinterpret_cast<uint4*>(reinterpret_cast<uint8_t*>(out + to * N) + unit * 16) =
            *reinterpret_cast<const uint4*>(rows + row * 32 * (int)sizeof(O) + unit * 16);
    }
    __syncwarp();
  }
}

// One 256-wide block of a token's row, 16 values a lane, quantised into row r of
// the swizzled token tile (128 bytes a row) and its scale atoms.
template <typename T>
__device__ __forceinline__ void quantize_row(const ProductArgs& p, int64_t row, int kb, int r,
                                             uint8_t* tile, uint8_t* scales) {
  const int l = threadIdx.x & 15;  // two rows per warp
  const int64_t col = (int64_t)kb * KB + l * 16;
  const int n = (int)(p.K - col > 16 ? 16 : (p.K > col ? p.K - col : 0));
  const T* x = static_cast<const T*>(p.raw) + row * p.raw_stride + col;
  Raw16<T> raw;
  raw.load(x, row >= 0 ? n : 0, (reinterpret_cast<uintptr_t>(x) & 15u) == 0);
  float v[16];
  raw.widen(v);
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 16; ++i) m = max(m, __float_as_uint(v[i]) & 0x7FFFFFFFu);
  m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
  const uint32_t sb = scale_byte(m);
  const uint2 code = codes16(v, scale_up(sb));
  if (row < 0) return;
  const int b = l >> 1;  // block of 32, one 16-byte unit of the row
  *reinterpret_cast<uint2*>(tile + r * 128 + ((b ^ (r & 7)) << 4) + (l & 1) * 8) = code;
  if ((l & 1) == 0) scales[(b >> 2) * ATOM_BYTES + r * 16 + (b & 3)] = (uint8_t)sb;
}

template <int BN, bool PAIR, bool EXPERTS, bool SPLIT, bool FUSED, bool GROUPS>
__global__ void __launch_bounds__(threads_of(EXPERTS), 1)
    k_mx_gemm(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmX,
              const __grid_constant__ CUtensorMap tmWs, const __grid_constant__ CUtensorMap tmXs,
              const ProductArgs p, const int num_m, const int num_n, const int group,
              const int log_splits, const int wide_rows) {
  using F = Form<BN, PAIR, EXPERTS>;
  constexpr int STAGES = F::STAGES, EPI_WARPS = epi_warps(EXPERTS), TURNS = EPI_WARPS / 4;
  // the experts' fused form: a tile has one chunk, so all but four epilogue warps
  // are free to quantise, ahead of the tiles being drained
  constexpr bool QUANTISERS = FUSED && EXPERTS;
  const int splits = SPLIT ? 1 << log_splits : 1;
  static_assert(!SPLIT || (!PAIR && !EXPERTS), "split form");
  static_assert(!FUSED || BN == 32, "fused form");
  static_assert(!GROUPS || (!EXPERTS && !SPLIT && !FUSED), "groups form");
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = tc::smem_align1024(smem_raw);
  float* part = reinterpret_cast<float*>(smem + STAGES * F::STAGE);  // SPLIT: [src][token][128 / S]
  Ctl* ctl = reinterpret_cast<Ctl*>(smem + STAGES * F::STAGE + extra_bytes<BN, EXPERTS, SPLIT>());
  // Known to be the same for a warp's lanes: what follows from it stays in
  // uniform registers, where the tcgen05 and TMA instructions want their operands.
  const int warp = __shfl_sync(0xffffffffu, (int)threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const int rank = PAIR ? (int)ptx::cluster_rank() : 0;
  const int slice = SPLIT ? (int)ptx::cluster_rank() : 0;
  const int unit = PAIR ? (int)blockIdx.x >> 1 : (SPLIT ? (int)blockIdx.x >> log_splits : (int)blockIdx.x);
  const int units = PAIR ? (int)gridDim.x >> 1 : (SPLIT ? (int)gridDim.x >> log_splits : (int)gridDim.x);
  // this CTA's blocks of K
  const int all_kb = (int)((p.K + KB - 1) / KB);
  const int kb0 = SPLIT ? (int)(((int64_t)all_kb * slice) >> log_splits) : 0;
  const int own_kb = SPLIT ? (int)(((int64_t)all_kb * (slice + 1)) >> log_splits) : all_kb;
  int* wd = &g_watchdog_mx;

  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      ptx::mbar_init(&ctl->full[s], FUSED ? 2 : 1);
      ptx::mbar_init(&ctl->empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      ptx::mbar_init(&ctl->accf[b], 1);
      ptx::mbar_init(&ctl->acce[b], QUANTISERS ? 4 : (PAIR ? 2 * EPI_WARPS : EPI_WARPS));
    }
    ptx::mbar_init(&ctl->drain, 1);
    if (SPLIT) ptx::mbar_init(&ctl->part, (uint32_t)(splits * EPI_WARPS));
    ctl->abort = 0;
    ptx::fence_mbar_init();
  }
  if (warp == 0 && lane == 0) {
    ptx::tma_prefetch_desc(&tmW);
    ptx::tma_prefetch_desc(&tmX);
    ptx::tma_prefetch_desc(&tmWs);
    ptx::tma_prefetch_desc(&tmXs);
  }
  if (warp == 1) ptx::tmem_alloc_g<PAIR>(&ctl->tmem_base, 512);
  if (EXPERTS) {
    ptx::griddep_wait();
    // tiles of each expert (the slots of no expert count as expert E)
    if (warp == 2) {
      int before = 0;
      for (int e0 = 0; e0 <= p.E; e0 += 32) {
        const int e = e0 + lane;
        int n = 0;
        if (e <= p.E) {
          const int off = p.offsets[e];
          ctl->offset[e] = off;
          ctl->start[e] = p.starts[e];
          n = (p.offsets[e + 1] - off + BN - 1) / BN * num_n;
        }
        int sum = n;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
          const int o = __shfl_up_sync(0xffffffffu, sum, d);
          if (lane >= d) sum += o;
        }
        if (e <= p.E) ctl->tiles_before[e] = before + sum - n;
        before += __shfl_sync(0xffffffffu, sum, 31);
      }
      if (lane == 0) {
        ctl->tiles_before[p.E + 1] = before;
        ctl->offset[p.E + 1] = p.slots;
      }
    }
  }
  if (GROUPS) {
    ptx::griddep_wait();
    for (int e = threadIdx.x; e <= p.E; e += blockDim.x) ctl->start[e] = p.starts[e];
  }
  ptx::tc_fence_before();
  __syncthreads();
  if (PAIR || SPLIT) ptx::cluster_sync();  // the other CTAs' barriers are ready
  ptx::tc_fence_after();
  const uint32_t tmem = __shfl_sync(0xffffffffu, ctl->tmem_base, 0);
  volatile int* abort = &ctl->abort;
  const int num_tiles =
      EXPERTS ? __shfl_sync(0xffffffffu, ctl->tiles_before[p.E + 1], 0) : num_m * num_n * (GROUPS ? p.E : 1);
  // first value and number of values of K that a tile sums over
  auto first_k = [&](int t) { return GROUPS ? ctl->start[t / (num_m * num_n)] : 0; };
  auto depth = [&](int t) {
    if (!GROUPS) return p.K;
    const int e = t / (num_m * num_n);
    return (int64_t)(ctl->start[e + 1] - ctl->start[e]);
  };
  auto blocks_of = [&](int t) { return GROUPS ? (int)((depth(t) + KB - 1) / KB) : own_kb; };

  auto tile_of = [&](int t) {
    Tile r;
    if (!EXPERTS) {
      int mt, nt;
      tc::tile_coords(GROUPS ? t % (num_m * num_n) : t, num_m, num_n, group, mt, nt);
      r.e = 0;
      r.n0 = nt * F::BNW + rank * BM;
      r.m0 = mt * BN;
      r.rows = (int)(p.M - r.m0 < BN ? p.M - r.m0 : BN);
      r.first = 0;
    } else {
      int lo = 0, hi = p.E;  // the last expert whose tiles begin at or before t
      while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (ctl->tiles_before[mid] <= t) lo = mid;
        else hi = mid - 1;
      }
      const int count = ctl->offset[lo + 1] - ctl->offset[lo];
      const int mts = (count + BN - 1) / BN, in = t - ctl->tiles_before[lo];
      const int mt = in % mts;  // the expert's token tiles share a weight tile
      r.e = lo;
      r.n0 = in / mts * F::BNW + rank * BM;
      r.m0 = lo < p.E ? (int)sorted_at(ctl->start[lo], BN == 224 ? TILES_224 : 7) + mt * BN : 0;
      r.rows = count - mt * BN < BN ? count - mt * BN : BN;
      r.first = ctl->offset[lo] + mt * BN;
    }
    return r;
  };

  if (warp == 0) {
    // ------------------------------------------------------ TMA producer
    // The whole warp walks the loop and one elected lane issues: a loop inside
    // `if (lane == 0)` has its descriptors and coordinates moved to uniform
    // registers one by one before every instruction (measured in the MMA warp:
    // 690 against the 512 cycles that the MMAs of a stage take).
    // After a pre-pass of this call the weight is known to be there.
    if (!EXPERTS && !GROUPS && !p.inputs_ready) ptx::griddep_wait();
    bool tokens_ready = EXPERTS || GROUPS || !p.inputs_ready;
    int s = 0, issued = 0;
    uint32_t ph = 0;
    for (int t = unit; t < num_tiles && !*abort; t += units) {
      const Tile r = tile_of(t);
      if (EXPERTS && r.e == p.E) break;  // only tiles of no expert follow
      const int xa = r.m0 / F::ATOM_TOKENS, k0 = first_k(t), num_kb = blocks_of(t);
      for (int kb = kb0; kb < num_kb; ++kb) {
        const int kc = k0 / 2 + kb * (KB / 2), ks = k0 + kb * KB;  // bytes of codes, words of scales
        if (!wait_any<PAIR>(&ctl->empty[s], ph ^ 1u, abort, tc::kSiteProducerEmpty, wd)) break;
        __syncwarp();
        uint8_t* st = smem + s * F::STAGE;
        uint8_t* sf = st + A_BYTES + F::B_BYTES;
        if (ptx::elect_one()) {
          if (rank == 0)
            ptx::mbar_arrive_expect_tx(&ctl->full[s], FUSED ? A_BYTES + F::SA_BYTES : F::TX);
          if (PAIR) {
            const uint32_t bar = ptx::cluster_addr(&ctl->full[s], 0);
            ptx::tma_load_3d_pair(st, &tmW, bar, kc, r.n0, r.e);
            ptx::tma_load_3d_pair(sf, &tmWs, bar, ks, r.n0 / BM, r.e);
          } else {
            ptx::tma_load_3d(st, &tmW, &ctl->full[s], kc, r.n0, r.e);
            ptx::tma_load_3d(sf, &tmWs, &ctl->full[s], ks, r.n0 / BM, r.e);
          }
        }
        if (!tokens_ready) ptx::griddep_wait();
        tokens_ready = true;
        if (!FUSED && ptx::elect_one()) {
          if (PAIR) {
            const uint32_t bar = ptx::cluster_addr(&ctl->full[s], 0);
            ptx::tma_load_2d_pair(st + A_BYTES, &tmX, bar, kc, r.m0 + rank * F::B_ROWS);
            ptx::tma_load_2d_pair(sf + F::SA_BYTES, &tmXs, bar, ks, xa);
          } else {
            ptx::tma_load_2d(st + A_BYTES, &tmX, &ctl->full[s], kc, r.m0);
            ptx::tma_load_2d(sf + F::SA_BYTES, &tmXs, &ctl->full[s], ks, xa);
          }
        }
        __syncwarp();
        ++issued;
        if (++s == STAGES) {
          s = 0;
          ph ^= 1u;
        }
      }
    }
    // Every copy issued must have landed before the CTA's shared memory is
    // released (a pair's copies count on CTA 0's barriers, and both CTAs meet
    // at the end), and so must every signal the MMAs send to a pair's barriers.
    for (int j = (issued > STAGES ? issued - STAGES : 0); j < issued; ++j) {
      const uint32_t parity = (uint32_t)((j / STAGES) & 1);
      if (rank == 0) tc::drain_wait(&ctl->full[j % STAGES], parity);
      if (PAIR) tc::drain_wait(&ctl->empty[j % STAGES], parity);
    }
    __syncwarp();
  } else if (warp == 1) {
    // --------------------------------------------------------- MMA issuer
    if (rank == 0) {
      constexpr uint32_t id0 = ptx::idesc_mxf4(F::BNW, BN, 0), id1 = ptx::idesc_mxf4(F::BNW, BN, 2);
      // Descriptors of stage 0 (their low bits hold the shared address >> 4, so
      // a stage, a k-step and a scale atom are plain sums).
      const uint32_t base = ptx::smem_addr(smem);
      const uint64_t da0 = ptx::smem_desc(base, 16, 1024, ptx::kSwizzle128B);
      const uint64_t db0 = ptx::smem_desc(base + A_BYTES, 16, 1024, ptx::kSwizzle128B);
      const uint64_t ds0 = ptx::smem_desc(base + A_BYTES + F::B_BYTES, 16, 128, 0);
      int s = 0, tl = 0, set = 0;
      int old = 0;             // the stage whose block had this block's scale columns
      uint32_t ph = 0, old_ph = 0;
      int block = 0;
      for (int t = unit; t < num_tiles; t += units) {
        if (EXPERTS && t >= ctl->tiles_before[p.E]) break;
        const int num_kb = __shfl_sync(0xffffffffu, blocks_of(t), 0);
        const int num_ks = __shfl_sync(0xffffffffu, (int)((depth(t) + KSTEP - 1) / KSTEP), 0);
        if (GROUPS && num_kb == 0) continue;  // an expert without rows: zeros
        const int buf = tl & 1;
        // the accumulator is free: the tile two before (overlapping ones: the
        // part shared with the tile before) has been read
        const bool free_ =
            F::OVERLAP ? tl == 0 || wait_any<true>(&ctl->acce[0], (uint32_t)(tl - 1) & 1u, abort,
                                                   tc::kSiteMmaAccEmpty, wd)
                       : wait_any<PAIR>(&ctl->acce[buf], ((uint32_t)(tl >> 1) & 1u) ^ 1u, abort,
                                   tc::kSiteMmaAccEmpty, wd);
        if (!free_) break;
        ptx::tc_fence_after();
        const uint32_t d = tmem + (uint32_t)(buf * F::ACC1);
        bool ok = true;
        for (int kb = kb0; kb < num_kb; ++kb, ++block) {
          ok = wait_any<PAIR>(&ctl->full[s], ph, abort, tc::kSiteMmaOperands, wd);
          // the scale columns are free: the MMAs of the block that had them are done
          if (F::SETS < STAGES && ok && block >= F::SETS) {
            ok = wait_any<PAIR>(&ctl->empty[old], old_ph, abort, tc::kSiteMmaOperands, wd);
            if (++old == STAGES) {
              old = 0;
              old_ph ^= 1u;
            }
          }
          if (!ok) break;
          ptx::tc_fence_after();
          __syncwarp();
          const uint64_t off = (uint64_t)(uint32_t)(s * (F::STAGE >> 4));
          const uint64_t da = da0 + off, db = db0 + off, ds = ds0 + off;
          const uint32_t sfa = tmem + (uint32_t)(F::SF_COL0 + set * F::SF_COLS), sfb = sfa + 8;
          const int steps = min(4, num_ks - 4 * kb);
          if (ptx::elect_one()) {
#pragma unroll
            for (int a = 0; a < 2; ++a) {  // block atoms of the stage
              ptx::tmem_cp_scales<PAIR>(sfa + a * 4, ds + (uint64_t)(a * ATOM_BYTES >> 4));
#pragma unroll
              for (int b = 0; b < F::B_ATOMS; ++b)
                ptx::tmem_cp_scales<PAIR>(
                    sfb + a * 4 * F::B_ATOMS + b * 4,
                    ds + (uint64_t)((F::SA_BYTES + (2 * b + a) * ATOM_BYTES) >> 4));
            }
            if (steps == 4) {
#pragma unroll
              for (int j = 0; j < 4; ++j)
                ptx::mma_mxf4<PAIR>(d, da + 2 * j, db + 2 * j, (j & 1) ? id1 : id0,
                                    sfa + (j >> 1) * 4, sfb + (j >> 1) * 4 * F::B_ATOMS,
                                    kb + j > kb0 ? 1u : 0u);
            } else {  // the last block of a K that is no multiple of 256
#pragma unroll
              for (int j = 0; j < 3; ++j)
                if (j < steps)
                  ptx::mma_mxf4<PAIR>(d, da + 2 * j, db + 2 * j, (j & 1) ? id1 : id0,
                                      sfa + (j >> 1) * 4, sfb + (j >> 1) * 4 * F::B_ATOMS,
                                      kb + j > kb0 ? 1u : 0u);
            }
            ptx::mma_commit_g<PAIR>(&ctl->empty[s]);
            if (kb == num_kb - 1) ptx::mma_commit_g<PAIR>(&ctl->accf[buf]);
          }
          __syncwarp();
          if (++set == F::SETS) set = 0;
          if (++s == STAGES) {
            s = 0;
            ph ^= 1u;
          }
        }
        if (!ok) break;
        ++tl;
      }
      // Every MMA issued must be done before TMEM is released.
      __syncwarp();
      if (ptx::elect_one()) ptx::mma_commit_g<PAIR>(&ctl->drain);
    }
    tc::drain_wait(&ctl->drain, 0);
    __syncwarp();
  } else {
    // ----------------------------------------------------------- epilogue
    ptx::griddep_wait();  // bias, and the order of output writes
    const int q = warp & 3;               // TMEM lane quadrant this warp may read
    const int turn = (warp - 2) >> 2;     // it takes every TURNS-th chunk of 32 tokens
    int tl = 0;
    // FUSED: the blocks of K of a tile that are warp `w`'s, every one whose stage is
    // w (a warp that skipped a use of its stage would take an old phase of the
    // stage's barrier for the one it waits for): wait for the stage, write the
    // tokens' rows.  `before`: blocks of earlier tiles.
    auto quantize_tile = [&](const Tile& r, int before, int w) {
      int kb = kb0 + (w - before % STAGES + STAGES) % STAGES;
      for (; kb < own_kb; kb += STAGES) {
        const int block = before + kb - kb0;
        if (!wait_any<false>(&ctl->empty[w], ((uint32_t)(block / STAGES) & 1u) ^ 1u, abort,
                             tc::kSiteProducerEmpty, wd))
          return false;
        __syncwarp();
        uint8_t* tile = smem + w * F::STAGE + A_BYTES;
        uint8_t* scales = tile + F::B_BYTES + F::SA_BYTES;
        for (int j = 0; j < r.rows; j += 2) {
          const int m = j + (lane >> 4);  // half-warps take neighbouring rows
          int64_t row = -1;
          if (m < r.rows) row = EXPERTS ? __ldg(p.order + r.first + m) / p.share : r.m0 + m;
          if (p.raw_dtype == IMC_F32) quantize_row<float>(p, row, kb, m, tile, scales);
          else if (p.raw_dtype == IMC_BF16) quantize_row<__nv_bfloat16>(p, row, kb, m, tile, scales);
          else quantize_row<__half>(p, row, kb, m, tile, scales);
        }
        ptx::fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(&ctl->full[w]);
      }
      return true;
    };
    if (QUANTISERS && turn > 0) {
      const int w = warp - 2 - 4;
      int before = 0;
      for (int t = unit; w < STAGES && t < num_tiles; t += units) {
        const Tile r = tile_of(t);
        if (r.e == p.E || !quantize_tile(r, before, w)) break;
        before += own_kb - kb0;
      }
    }
    for (int t = unit; (!QUANTISERS || turn == 0) && t < num_tiles; t += units) {
      const Tile r = tile_of(t);
      // zeros: slots of no expert, the gradient of an expert without rows
      const bool none = (EXPERTS && r.e == p.E) || (GROUPS && depth(t) == 0);
      const int buf = tl & 1;
      const int64_t n = r.n0 + q * 32 + lane;
      const bool in = n < p.N;
      const float bias = p.bias && in && !none ? __ldg(p.bias + (int64_t)r.e * p.N + n) : 0.0f;
      // accumulator 0 shares its last columns with 1, which shares its first
      auto chunk = [&](int i) {
        return 32 * (F::OVERLAP && buf == 0 ? (i + BN / 32 - F::SHARED) % (BN / 32) : i);
      };
      // the slots of a chunk's tokens, those of both chunks that a warp may have
      // before it waits for the accumulator
      auto slots = [&](int i) {
        const int c = chunk(i) + lane;
        return EXPERTS && i < BN / 32 && c < r.rows ? __ldg(p.order + r.first + c) : 0;
      };
      static_assert(!EXPERTS || BN / 32 <= 2 * TURNS, "two chunks a warp");
      const int slot0 = slots(turn), slot1 = slots(turn + TURNS);
      if (FUSED && !QUANTISERS && !none) {
        static_assert(!FUSED || EXPERTS || EPI_WARPS == STAGES, "a stage belongs to one warp");
        if (!quantize_tile(r, tl * (own_kb - kb0), warp - 2)) break;
      }
      if (!none) {
        int ok = 1;
        if (lane == 0)
          ok = wait_any<PAIR>(&ctl->accf[buf], (uint32_t)(tl >> 1) & 1u, abort,
                              tc::kSiteEpilogueAccFull, wd)
                   ? 1
                   : 0;
        if (!__shfl_sync(0xffffffffu, ok, 0)) break;
        ptx::tc_fence_after();
        ++tl;
      }
      const uint32_t tbase = tmem + ((uint32_t)(q * 32) << 16) + (uint32_t)(buf * F::ACC1);
#pragma unroll 1
      for (int i = turn; i < BN / 32 || i == turn; i += TURNS) {
        const int c = chunk(i);
        const int live = min(32, r.rows - c);  // the same for all lanes
        uint32_t v[32];
        const int this_slot = i == turn ? slot0 : slot1;
        if (live > 0 && !none) {
          ptx::tmem_ld32(tbase + (uint32_t)c, v);
          ptx::tmem_ld_wait();
        } else {
#pragma unroll
          for (int j = 0; j < 32; ++j) v[j] = 0u;
        }
        // after this warp's last chunk (overlapping: its last shared one) the MMA
        // may have the accumulator back
        if (!none && (F::OVERLAP ? i == turn : i + TURNS >= BN / 32)) {
          ptx::tc_fence_before();
          __syncwarp();
          if (lane == 0) {
            if (PAIR)
              ptx::mbar_arrive_cluster_tmem(
                  ptx::cluster_addr(&ctl->acce[F::OVERLAP ? 0 : buf], 0));
            else ptx::mbar_arrive(&ctl->acce[buf]);
          }
        }
        if (live <= 0 || c >= BN) continue;
        if (SPLIT) {  // to the CTA that sums this row of n
          const int nl = (q * 32 + lane) & ((BM >> log_splits) - 1);
          uint32_t to = ptx::cluster_addr(part + (((slice * BN + c) << 7) >> log_splits) + nl,
                                          (uint32_t)((q * 32 + lane) >> (7 - log_splits)));
#pragma unroll
          for (int j = 0; j < 32; ++j) {
            if (j < live) ptx::st_cluster(to, v[j]);
            to += (uint32_t)(BM * 4) >> log_splits;
          }
          continue;
        }
        if (!none) {
#pragma unroll
          for (int j = 0; j < 32; ++j) {
            float y = __uint_as_float(v[j]) + bias;
            if (p.relu) y = fmaxf(y, 0.0f);
            v[j] = __float_as_uint(y);
          }
        }
        const int64_t at =
            (EXPERTS ? 0 : ((GROUPS ? t / (num_m * num_n) * p.M : 0) + r.m0 + c) * p.N) + r.n0 + q * 32;
        auto f32 = [](uint32_t b) { return b; };
        auto bf16 = [](uint32_t b) { return bf16_bits(__uint_as_float(b)); };
        auto f16 = [](uint32_t b) { return half_bits(__uint_as_float(b)); };
        if (EXPERTS && wide_rows) {
          uint8_t* rows = smem + STAGES * F::STAGE + (warp - 2) * ROWS_BYTES;
          const int cols = (int)(p.N - r.n0 - q * 32 < 32 ? p.N - r.n0 - q * 32 : 32);
          if (p.out_dtype == IMC_F32)
            store_rows(static_cast<uint32_t*>(p.out) + at, p.N, this_slot, live, cols, v,
                                rows, f32);
          else if (p.out_dtype == IMC_BF16)
            store_rows(static_cast<uint16_t*>(p.out) + at, p.N, this_slot, live, cols, v,
                                rows, bf16);
          else
            store_rows(static_cast<uint16_t*>(p.out) + at, p.N, this_slot, live, cols, v,
                                rows, f16);
        } else if (p.out_dtype == IMC_F32) {
          store_tokens<EXPERTS>(static_cast<uint32_t*>(p.out) + at + lane, p.N, this_slot, live, in,
                                v, f32);
        } else if (p.out_dtype == IMC_BF16) {
          store_tokens<EXPERTS>(static_cast<uint16_t*>(p.out) + at + lane, p.N, this_slot, live, in,
                                v, bf16);
        } else {
          store_tokens<EXPERTS>(static_cast<uint16_t*>(p.out) + at + lane, p.N, this_slot, live, in,
                                v, f16);
        }
      }
      if (SPLIT) {
        __syncwarp();
        if (lane == 0)
          for (int r2 = 0; r2 < splits; ++r2)
            ptx::mbar_arrive_cluster(ptx::cluster_addr(&ctl->part, (uint32_t)r2));
        if (!wait_any<true>(&ctl->part, 0, abort, tc::kSiteEpilogueAccFull, wd)) break;
        // row x >> lp, column x & (per - 1) of this CTA's share
        const int lp = 7 - log_splits, live = r.rows << lp;
#pragma unroll 4
        for (int x = (int)threadIdx.x - 64; x < live; x += 32 * EPI_WARPS) {
          const int64_t nn = r.n0 + (slice << lp) + (x & ((1 << lp) - 1));
          float y = 0.0f;
          for (int src = 0; src < splits; ++src) y += part[((src * BN) << lp) + x];
          if (nn >= p.N) continue;
          if (p.bias) y += __ldg(p.bias + nn);
          if (p.relu) y = fmaxf(y, 0.0f);
          const int64_t at = (int64_t)(r.m0 + (x >> lp)) * p.N + nn;
          if (p.out_dtype == IMC_F32) static_cast<float*>(p.out)[at] = y;
          else if (p.out_dtype == IMC_BF16) static_cast<__nv_bfloat16*>(p.out)[at] = __float2bfloat16_rn(y);
          else static_cast<__half*>(p.out)[at] = __float2half_rn(y);
        }
        break;  // one tile
      }
    }
  }

  ptx::tc_fence_before();
  __syncthreads();
  if (PAIR || SPLIT) ptx::cluster_sync();  // no CTA leaves while another may signal it
  if (warp == 1) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc_g<PAIR>(tmem, 512);
  }
}

// ------------------------------------------------------------------- host
typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                                  const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                                  const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                  CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn encode_fn() {
  static EncodeTiledFn fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault,
                                         &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<EncodeTiledFn>(p);
    else
      cudaGetLastError();
  });
  return fn;
}

// Codes [batch][rows][pitch] bytes -> tensor map with a {128, box_rows, 1} box,
// 128-byte swizzle, zero fill past each matrix.
bool encode_codes(CUtensorMap* m, const uint8_t* base, const Store& st, uint32_t box_rows, int rank) {
  EncodeTiledFn fn = encode_fn();
  if (!fn) return false;
  const cuuint64_t dims[3] = {(cuuint64_t)st.pitch, (cuuint64_t)st.rows, (cuuint64_t)st.batch};
  const cuuint64_t strides[2] = {(cuuint64_t)st.pitch, (cuuint64_t)(st.rows * st.pitch)};
  const cuuint32_t box[3] = {128, box_rows, 1};
  const cuuint32_t es[3] = {1, 1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, (cuuint32_t)rank, const_cast<uint8_t*>(base), dims,
            strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Scale atoms [batch][row_atoms][block_atoms][512 bytes] -> tensor map with a box
// of two block atoms x `box_atoms` row atoms, as 32-bit words.
bool encode_scales(CUtensorMap* m, const uint8_t* q, const Store& st, uint32_t box_atoms, int rank) {
  EncodeTiledFn fn = encode_fn();
  if (!fn) return false;
  const cuuint64_t row = (cuuint64_t)(st.block_atoms * ATOM_BYTES);
  const cuuint64_t dims[3] = {row / 4, (cuuint64_t)st.row_atoms, (cuuint64_t)st.batch};
  const cuuint64_t strides[2] = {row, row * (cuuint64_t)st.row_atoms};
  const cuuint32_t box[3] = {2 * ATOM_BYTES / 4, box_atoms, 1};
  const cuuint32_t es[3] = {1, 1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT32, (cuuint32_t)rank,
            const_cast<uint8_t*>(q + st.scales_off), dims, strides, box, es,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

constexpr int kMaxDev = 64;

template <int BN, bool PAIR, bool EXPERTS, bool SPLIT = false, bool FUSED = false,
          bool GROUPS = false>
cudaError_t run(const ProductArgs& p, cudaStream_t s, int splits = 1) {
  using F = Form<BN, PAIR, EXPERTS>;
  constexpr int smem = smem_bytes<BN, PAIR, EXPERTS, SPLIT>();
  static std::atomic<bool> ready[kMaxDev];  // per device: the attribute is set (calls may race)
  auto k = k_mx_gemm<BN, PAIR, EXPERTS, SPLIT, FUSED, GROUPS>;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= kMaxDev || !ready[dev].load(std::memory_order_acquire)) {
    e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    if (dev < kMaxDev) ready[dev].store(true, std::memory_order_release);
  }
  const int ctas = PAIR ? 2 : splits, units = device_sm_count() / ctas;
  // a dense product of fewer than 128 rows a tile has one tile of tokens
  const Store sw = store_of(EXPERTS ? p.E : 1, p.N, p.K),
              sx = store_of(1, p.x_rows, p.K,
                            EXPERTS ? experts_atom_shift(p.slots, p.E) : p.x_shift);
  CUtensorMap tw, tx, tws, txs;
  if (!encode_codes(&tw, p.w, sw, BM, 3) || !encode_scales(&tws, p.w, sw, 1, 3))
    return cudaErrorInvalidValue;
  if (FUSED) {  // not read
    tx = tw;
    txs = tws;
  } else if (!encode_codes(&tx, p.x, sx, F::B_ROWS, 2) ||
             !encode_scales(&txs, p.x, sx, F::B_ATOMS, 2)) {
    return cudaErrorInvalidValue;
  }
  const int num_n = (int)ceil_div(p.N, F::BNW), num_m = EXPERTS ? 0 : (int)ceil_div(p.M, BN);
  // experts: at most one partly filled tile per expert beyond the full ones
  const int64_t tiles = EXPERTS ? (p.slots / BN + (p.slots < p.E + 1 ? p.slots : p.E + 1)) *
                                      (int64_t)num_n
                                : (int64_t)num_m * num_n * (GROUPS ? p.E : 1);
  if (tiles > 0x7fffffffLL || (SPLIT && tiles > units)) return cudaErrorInvalidValue;
  const int grid = (int)(tiles < units ? tiles : units) * ctas;
  // rows that 16-byte stores can write
  const int wide_rows = (reinterpret_cast<uintptr_t>(p.out) & 15u) == 0 &&
                        (p.N * dtype_bytes(p.out_dtype)) % 16 == 0 ? 1 : 0;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(threads_of(EXPERTS));
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = ctas;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = PAIR || SPLIT ? 2 : 1;
  e = cudaLaunchKernelEx(&cfg, k, tw, tx, tws, txs, p, num_m, num_n, 8, splits == 8 ? 3 : splits / 2,
                         wide_rows);
  note_launch();
  return e;
}

}  // namespace

bool product_supported() { return encode_fn() != nullptr; }

namespace {
// Token rows of a tile, as log2: the smallest form that holds what a call (or
// one expert, on average) has, 256 for more.
int tile_shift(int64_t rows) { return rows <= 32 ? 5 : (rows <= 64 ? 6 : (rows <= 128 ? 7 : 8)); }
}  // namespace

// Measured fused / with a quantising launch before, us on the GPU in a graph (bf16,
// K x N = 4096 x 4096): 1 token 5.9 / 6.3, 4 tokens 6.4 / 6.3, 8 tokens 7.3 / 6.5, 16
// tokens 9.1 / 7.1.  Issued from Python a call takes 9.6 us fused and 15 with the
// other launch and its scratch, so the form with one launch reaches to 8 tokens; a graph,
// which pays no Python, gives up 0.1 us at 4 tokens and 0.8 at 8 for that.
bool product_fused(int64_t tokens) { return tokens <= 8; }
// 64 experts, 2048 x 1024, 4 slots a token: 2 tokens 4.8 / 6.7, 8 tokens 7.3 / 9.3,
// 32 tokens 11.1 / 13.2; 32 tokens of 8 slots, 1024 x 1024 11.0 / 11.1; 8 experts,
// 4096 x 2048, 32 slots 9.1 / 8.6 (the one launch still saves the call its scratch).
bool experts_fused(int64_t slots, int64_t E) { return slots <= 4 * E && slots <= 256; }

int experts_atom_shift(int64_t slots, int64_t E) {
  const int t = tile_shift(ceil_div(slots, E));
  return t <= 7 ? t : TILES_224;
}

namespace {
// CTAs that share the K of a tile of at most 32 tokens: as many as find an SM
// each and at least eight blocks of 256 values.  Measured in a row, weights
// larger than L2 (us for 1 / 2 / 4 CTAs): 1 x 1024 x 8192 8.1 / 6.9 / 6.0,
// 1 x 4096 x 16384 15.0 / 11.6 / 10.6, 1 x 4096 x 4096 5.5 / 5.7 / 5.7 (where the rule
// begins to split: nothing won yet, 0.2 us lost).  More
// tokens make the sum of the partial tiles cost more than the split saves (64 x
// 4096 x 4096 5.6 / 9.5 / 7.5, 128 x 1024 x 8192 9.4 / 15.3 / 10.5).
int pick_splits(const ProductArgs& p) {
  const int64_t tiles = ceil_div(p.N, BM), blocks = ceil_div(p.K, KB);
  const int sms = device_sm_count();
  int s = 1;
  while (s < 8 && tiles * s * 2 <= sms && blocks >= s * 16) s *= 2;
  return s;
}
}  // namespace

// Pair tiles of 224 tokens have two accumulators without a shared part, so the
// MMAs of a tile do not wait for the epilogue of the one before; tiles of 256 do,
// ~700 cycles (fitted: 530 to 780 from the calls below), but may need fewer rounds.
// Taken: the form whose rounds take fewer cycles, at 2 (1.75) per value of K and 300
// to hand over.  Whole calls, us with 224 / 256: 8192 x 4096 x 4096 60.4 / 61.9,
// K = 2048 36.3 / 37.0, K = 512 24.6 / 24.4, 3000 x 4096 x 4096 25.5 / 27.9, 4096 x
// 1024 x 8192 43.4 / 44.4.
int product_atom_shift(int64_t M, int64_t N, int64_t K) {
  const int64_t n = ceil_div(N, 256), pairs = device_sm_count() / 2;
  if (tile_shift(M) < 8 || ceil_div(M, 256) * n * 4 <= 2 * pairs) return 7;
  const double wide = (double)ceil_div(ceil_div(M, 256) * n, pairs) * (2.0 * (double)K + 700.0);
  const double narrow = (double)ceil_div(ceil_div(M, 224) * n, pairs) * (1.75 * (double)K + 300.0);
  return narrow < wide ? TILES_224 : 7;
}

cudaError_t launch_product(const ProductArgs& p, cudaStream_t s) {
  note_kernel_name(p.raw ? (p.E ? "k_mx_gemm<experts,fused>" : "k_mx_gemm<fused>")
                         : (p.E ? "k_mx_gemm<experts>" : "k_mx_gemm"));
  if (p.groups) return run<256, true, false, false, false, true>(p, s);
  if (p.E) {
    switch (tile_shift(ceil_div(p.slots, p.E))) {
      case 5:
        return p.raw ? run<32, false, true, false, true>(p, s) : run<32, false, true>(p, s);
      case 6: return run<64, false, true>(p, s);
      case 7: return run<128, false, true>(p, s);
      default: return run<224, true, true>(p, s);
    }
  }
  if (p.x_shift == TILES_224) return run<224, true, false>(p, s);
  // Pairs that would leave more than half of the SMs without a tile give way to
  // single CTAs of 128 x 128.
  const int64_t pair_tiles = ceil_div(p.M, 256) * ceil_div(p.N, 256);
  const int shift = tile_shift(p.M);
  if (shift == 5) {
    const int splits = pick_splits(p);
    if (p.raw)
      return splits > 1 ? run<32, false, false, true, true>(p, s, splits)
                        : run<32, false, false, false, true>(p, s);
    return splits > 1 ? run<32, false, false, true>(p, s, splits) : run<32, false, false>(p, s);
  }
  if (shift == 6) return run<64, false, false>(p, s);
  if (shift == 7 || pair_tiles * 4 <= device_sm_count()) return run<128, false, false>(p, s);
  return run<256, true, false>(p, s);
}

cudaError_t product_take_watchdog(int* value) {
  cudaError_t e = cudaMemcpyFromSymbol(value, g_watchdog_mx, sizeof(int));
  if (e != cudaSuccess) return e;
  const int zero = 0;
  return cudaMemcpyToSymbol(g_watchdog_mx, &zero, sizeof(int));
}

}  // namespace mx
}  // namespace imc
