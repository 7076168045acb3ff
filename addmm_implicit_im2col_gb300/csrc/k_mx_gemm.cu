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
//               128 bytes of codes), the token tile (BN rows x 128 bytes), both
//               128-byte swizzled, and their scales (one contiguous copy per
//               128 rows) into a ring of stages
//   warp 1      TMEM owner + MMA issuer: copies the stage's scales to the
//               stage's own TMEM columns (tcgen05.cp), then one MMA per 64
//               values of K into an fp32 accumulator
//   warps 2-5   epilogue: tcgen05.ld, bias, ReLU, rounding, store
//
// One persistent CTA per SM walks the tiles.  In the experts' form a tile is
// (expert, rows of that expert, 128 n); the row counts are only known on the
// GPU, so every CTA sums them up at its start.
#include <atomic>
#include <mutex>

#include "mx_internal.cuh"
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

template <int BN>
struct Form {
  static constexpr int B_BYTES = BN * KB / 2;
  static constexpr int B_ATOMS = BN > 128 ? BN / 128 : 1;      // row atoms of a token tile
  static constexpr int ATOM_TOKENS = BN < 128 ? BN : 128;      // token rows of a scale atom
  static constexpr int SA_BYTES = 2 * ATOM_BYTES, SB_BYTES = 2 * ATOM_BYTES * B_ATOMS;
  static constexpr int STAGE = A_BYTES + B_BYTES + SA_BYTES + SB_BYTES;
  static constexpr int STAGES = BN > 128 ? 4 : (BN > 64 ? 6 : 8);
  static constexpr int NACC = 2 * BN + STAGES * (8 + 8 * B_ATOMS) <= 512 ? 2 : 1;
  static constexpr int SF_COL0 = NACC * BN;                    // scales after the accumulators
  static constexpr int SF_COLS = 8 + 8 * B_ATOMS;              // TMEM columns of a stage's scales
  static_assert(SF_COL0 + STAGES * SF_COLS <= 512, "TMEM");
};

struct Ctl {
  uint64_t full[8], empty[8], accf[2], acce[2], drain;
  uint32_t tmem_base;
  int abort;
  int tiles_before[MAX_EXPERTS + 2];  // experts' form: tiles of the experts before e
};

template <int BN>
constexpr int smem_bytes() {
  return 1024 + Form<BN>::STAGES * Form<BN>::STAGE + (int)sizeof(Ctl);
}
static_assert(smem_bytes<256>() <= 232448 && smem_bytes<128>() <= 232448 &&
                  smem_bytes<64>() <= 232448 && smem_bytes<32>() <= 232448,
              "shared memory");

// One tile: n rows n0.. of expert e's weight, token rows m0.. of x (`rows` of
// them count).
struct Tile {
  int e, n0, m0, rows;
  int first;  // experts' form: place of row m0 in `order`
};

template <typename T>
__device__ __forceinline__ void put(void* out, int64_t at, float v) {
  static_cast<T*>(out)[at] = from_f32<T>(v);
}

template <int BN, bool EXPERTS>
__global__ void __launch_bounds__(192, 1)
    k_mx_gemm(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmX,
              const ProductArgs p, const int num_m, const int num_n, const int group,
              const int64_t x_scales_off, const int64_t w_scales_off) {
  using F = Form<BN>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = tc::smem_align1024(smem_raw);
  Ctl* ctl = reinterpret_cast<Ctl*>(smem + F::STAGES * F::STAGE);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int num_kb = (int)((p.K + KB - 1) / KB);
  const int block_atoms = (int)((p.K + 127) / 128), w_row_atoms = (int)((p.N + 127) / 128);
  int* wd = &g_watchdog_mx;

  if (threadIdx.x == 0) {
    for (int s = 0; s < F::STAGES; ++s) {
      ptx::mbar_init(&ctl->full[s], 1);
      ptx::mbar_init(&ctl->empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      ptx::mbar_init(&ctl->accf[b], 1);
      ptx::mbar_init(&ctl->acce[b], 128);
    }
    ptx::mbar_init(&ctl->drain, 1);
    ctl->abort = 0;
    ptx::fence_mbar_init();
  }
  if (warp == 0 && lane == 0) {
    ptx::tma_prefetch_desc(&tmW);
    ptx::tma_prefetch_desc(&tmX);
  }
  if (warp == 1) {
    ptx::tmem_alloc(&ctl->tmem_base, 512);
    ptx::tmem_relinquish();
  }
  if (EXPERTS) {
    ptx::griddep_wait();
    // tiles of each expert (the slots of no expert count as expert E)
    if (warp == 2) {
      int before = 0;
      for (int e0 = 0; e0 <= p.E; e0 += 32) {
        const int e = e0 + lane;
        int n = 0;
        if (e <= p.E) n = (p.offsets[e + 1] - p.offsets[e] + BN - 1) / BN * num_n;
        int sum = n;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
          const int o = __shfl_up_sync(0xffffffffu, sum, d);
          if (lane >= d) sum += o;
        }
        if (e <= p.E) ctl->tiles_before[e] = before + sum - n;
        before += __shfl_sync(0xffffffffu, sum, 31);
      }
      if (lane == 0) ctl->tiles_before[p.E + 1] = before;
    }
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem = ctl->tmem_base;
  volatile int* abort = &ctl->abort;
  const int num_tiles = EXPERTS ? ctl->tiles_before[p.E + 1] : num_m * num_n;

  auto tile_of = [&](int t) {
    Tile r;
    if (!EXPERTS) {
      int mt, nt;
      tc::tile_coords(t, num_m, num_n, group, mt, nt);
      r.e = 0;
      r.n0 = nt * BM;
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
      const int count = p.offsets[lo + 1] - p.offsets[lo];
      const int mts = (count + BN - 1) / BN, in = t - ctl->tiles_before[lo];
      const int mt = in % mts;  // the expert's token tiles share a weight tile
      r.e = lo;
      r.n0 = in / mts * BM;
      r.m0 = lo < p.E ? p.starts[lo] + mt * BN : 0;
      r.rows = count - mt * BN < BN ? count - mt * BN : BN;
      r.first = p.offsets[lo] + mt * BN;
    }
    return r;
  };

  if (warp == 0) {
    // ------------------------------------------------------ TMA producer
    if (lane == 0) {
      // after a pre-pass of this call the weight is known to be there
      if (!EXPERTS && !p.inputs_ready) ptx::griddep_wait();
      bool tokens_ready = EXPERTS || !p.inputs_ready;
      int s = 0, issued = 0;
      uint32_t ph = 0;
      for (int t = blockIdx.x; t < num_tiles && !*abort; t += gridDim.x) {
        const Tile r = tile_of(t);
        if (EXPERTS && r.e == p.E) break;  // only tiles of no expert follow
        const uint8_t* wsf = p.w + w_scales_off +
                             ((int64_t)r.e * w_row_atoms + r.n0 / 128) * block_atoms * ATOM_BYTES;
        const uint8_t* xsf =
            p.x + x_scales_off + (int64_t)(r.m0 / F::ATOM_TOKENS) * block_atoms * ATOM_BYTES;
        const int b_atoms = F::B_ATOMS > 1 && r.rows > 128 ? F::B_ATOMS : 1;
        for (int kb = 0; kb < num_kb; ++kb) {
          if (!wait_bar(&ctl->empty[s], ph ^ 1u, abort, tc::kSiteProducerEmpty, wd)) break;
          uint8_t* st = smem + s * F::STAGE;
          const uint32_t sf = (uint32_t)min(2, block_atoms - 2 * kb) * ATOM_BYTES;
          ptx::mbar_arrive_expect_tx(&ctl->full[s],
                                     (uint32_t)(A_BYTES + F::B_BYTES) + sf * (1 + b_atoms));
          ptx::tma_load_3d(st, &tmW, &ctl->full[s], kb * (KB / 2), r.n0, r.e);
          ptx::bulk_load(st + A_BYTES + F::B_BYTES, wsf + (int64_t)kb * 2 * ATOM_BYTES, sf,
                         &ctl->full[s]);
          if (!tokens_ready) {
            ptx::griddep_wait();
            tokens_ready = true;
          }
          ptx::tma_load_2d(st + A_BYTES, &tmX, &ctl->full[s], kb * (KB / 2), r.m0);
          for (int a = 0; a < b_atoms; ++a)
            ptx::bulk_load(st + A_BYTES + F::B_BYTES + F::SA_BYTES + a * 2 * ATOM_BYTES,
                           xsf + ((int64_t)a * block_atoms + kb * 2) * ATOM_BYTES, sf,
                           &ctl->full[s]);
          ++issued;
          if (++s == F::STAGES) {
            s = 0;
            ph ^= 1u;
          }
        }
      }
      // Every copy issued must have landed before the CTA's shared memory is released.
      for (int j = (issued > F::STAGES ? issued - F::STAGES : 0); j < issued; ++j)
        tc::drain_wait(&ctl->full[j % F::STAGES], (uint32_t)((j / F::STAGES) & 1));
    }
  } else if (warp == 1) {
    // --------------------------------------------------------- MMA issuer
    if (lane == 0) {
      constexpr uint32_t id0 = ptx::idesc_mxf4(BM, BN, 0), id1 = ptx::idesc_mxf4(BM, BN, 2);
      const int num_ks = (int)((p.K + KSTEP - 1) / KSTEP);
      int s = 0, tl = 0;
      uint32_t ph = 0;
      for (int t = blockIdx.x; t < num_tiles; t += gridDim.x, ++tl) {
        if (EXPERTS && tile_of(t).e == p.E) break;
        const int buf = tl % F::NACC;
        const uint32_t use = (uint32_t)(tl / F::NACC);
        if (!wait_bar(&ctl->acce[buf], (use & 1u) ^ 1u, abort, tc::kSiteMmaAccEmpty, wd)) break;
        ptx::tc_fence_after();
        const uint32_t d = tmem + (uint32_t)(buf * BN);
        bool ok = true;
        for (int kb = 0; kb < num_kb; ++kb) {
          if (!wait_bar(&ctl->full[s], ph, abort, tc::kSiteMmaOperands, wd)) {
            ok = false;
            break;
          }
          ptx::tc_fence_after();
          const uint32_t base = ptx::smem_addr(smem + s * F::STAGE);
          const uint64_t da = ptx::smem_desc(base, 16, 1024, ptx::kSwizzle128B);
          const uint64_t db = ptx::smem_desc(base + A_BYTES, 16, 1024, ptx::kSwizzle128B);
          const uint64_t ds = ptx::smem_desc(base + A_BYTES + F::B_BYTES, 16, 128, 0);
          const uint32_t sfa = tmem + (uint32_t)(F::SF_COL0 + s * F::SF_COLS), sfb = sfa + 8;
#pragma unroll
          for (int a = 0; a < 2; ++a) {  // block atoms of the stage
            ptx::tmem_cp_scales(sfa + a * 4, ds + (uint64_t)(a * ATOM_BYTES >> 4));
#pragma unroll
            for (int b = 0; b < F::B_ATOMS; ++b)
              ptx::tmem_cp_scales(sfb + a * 4 * F::B_ATOMS + b * 4,
                                  ds + (uint64_t)((F::SA_BYTES + (2 * b + a) * ATOM_BYTES) >> 4));
          }
          const int steps = min(4, num_ks - 4 * kb);
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            if (j < steps)
              ptx::mma_mxf4(d, da + 2 * j, db + 2 * j, (j & 1) ? id1 : id0, sfa + (j >> 1) * 4,
                            sfb + (j >> 1) * 4 * F::B_ATOMS, kb + j > 0 ? 1u : 0u);
          }
          ptx::mma_commit(&ctl->empty[s]);
          if (++s == F::STAGES) {
            s = 0;
            ph ^= 1u;
          }
        }
        if (!ok) break;
        ptx::mma_commit(&ctl->accf[buf]);
      }
      // Every MMA issued must be done before TMEM is released.
      ptx::mma_commit(&ctl->drain);
      tc::drain_wait(&ctl->drain, 0);
    }
    __syncwarp();
  } else {
    // ----------------------------------------------------------- epilogue
    ptx::griddep_wait();  // bias, and the order of output writes
    const int q = warp & 3;  // TMEM lane quadrant this warp may read
    int tl = 0;
    for (int t = blockIdx.x; t < num_tiles; t += gridDim.x) {
      const Tile r = tile_of(t);
      const bool none = EXPERTS && r.e == p.E;  // slots of no expert: zeros
      const int buf = tl % F::NACC;
      const int64_t n = r.n0 + q * 32 + lane;
      const bool in = n < p.N;
      const float bias = p.bias && in && !none ? p.bias[(int64_t)r.e * p.N + n] : 0.0f;
      if (!none) {
        const bool ok = tc::warp_wait_bar(&ctl->accf[buf], (uint32_t)(tl / F::NACC) & 1u, abort,
                                          tc::kSiteEpilogueAccFull, wd);
        if (tc::epi_any(!ok)) break;
        ptx::tc_fence_after();
        ++tl;
      }
      const uint32_t tbase = tmem + ((uint32_t)(q * 32) << 16) + (uint32_t)(buf * BN);
#pragma unroll 1
      for (int c = 0; c < BN; c += 32) {
        uint32_t v[32];
        if (!none) {
          ptx::tmem_ld32(tbase + (uint32_t)c, v);
          ptx::tmem_ld_wait();
          if (c + 32 == BN) {  // the accumulator is read: the MMA may have it back
            ptx::tc_fence_before();
            ptx::mbar_arrive(&ctl->acce[buf]);
          }
        } else {
#pragma unroll
          for (int j = 0; j < 32; ++j) v[j] = 0u;
        }
        const int live = min(32, r.rows - c);  // warp-uniform
        if (live <= 0) continue;
        int slot = 0;
        if (EXPERTS) slot = lane < live ? p.order[r.first + c + lane] : 0;
#pragma unroll
        for (int j = 0; j < 32; ++j) {
          if (j < live) {
            const int64_t row = EXPERTS ? (int64_t)__shfl_sync(0xffffffffu, slot, j)
                                        : (int64_t)r.m0 + c + j;
            float y = none ? 0.0f : __uint_as_float(v[j]) + bias;
            if (p.relu) y = fmaxf(y, 0.0f);
            if (in) {
              const int64_t at = row * p.N + n;
              if (p.out_dtype == IMC_F32) put<float>(p.out, at, y);
              else if (p.out_dtype == IMC_F16) put<__half>(p.out, at, y);
              else put<__nv_bfloat16>(p.out, at, y);
            }
          }
        }
      }
    }
  }

  ptx::tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc(tmem, 512);
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

constexpr int kMaxDev = 64;

template <int BN, bool EXPERTS>
cudaError_t run(const ProductArgs& p, cudaStream_t s) {
  constexpr int smem = smem_bytes<BN>();
  static std::atomic<bool> ready[kMaxDev];  // per device: the attribute is set (calls may race)
  auto k = k_mx_gemm<BN, EXPERTS>;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= kMaxDev || !ready[dev].load(std::memory_order_acquire)) {
    e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    if (dev < kMaxDev) ready[dev].store(true, std::memory_order_release);
  }
  const int sms = device_sm_count();
  // a dense product of fewer than 128 rows a tile has one tile of tokens
  const Store sw = store_of(EXPERTS ? p.E : 1, p.N, p.K),
              sx = store_of(1, p.x_rows, p.K,
                            EXPERTS ? experts_atom_shift(p.slots, p.E) : 7);
  CUtensorMap tw, tx;
  if (!encode_codes(&tw, p.w, sw, BM, 3) || !encode_codes(&tx, p.x, sx, BN, 2))
    return cudaErrorInvalidValue;
  const int num_n = (int)ceil_div(p.N, BM), num_m = EXPERTS ? 0 : (int)ceil_div(p.M, BN);
  // experts: at most one partly filled tile per expert beyond the full ones
  const int64_t tiles = EXPERTS ? (p.slots / BN + (p.slots < p.E + 1 ? p.slots : p.E + 1)) *
                                      (int64_t)num_n
                                : (int64_t)num_m * num_n;
  const int grid = (int)(tiles < sms ? tiles : sms);
  e = launch_after_previous(k, dim3(grid), dim3(192), (size_t)smem, s, tw, tx, p, num_m, num_n,
                            -8, sx.scales_off, sw.scales_off);
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

int experts_atom_shift(int64_t slots, int64_t E) {
  const int t = tile_shift(ceil_div(slots, E));
  return t < 7 ? t : 7;
}

cudaError_t launch_product(const ProductArgs& p, cudaStream_t s) {
  note_kernel_name(p.E ? "k_mx_gemm<experts>" : "k_mx_gemm");
  switch (tile_shift(p.E ? ceil_div(p.slots, p.E) : p.M)) {
    case 5: return p.E ? run<32, true>(p, s) : run<32, false>(p, s);
    case 6: return p.E ? run<64, true>(p, s) : run<64, false>(p, s);
    case 7: return p.E ? run<128, true>(p, s) : run<128, false>(p, s);
    default: return p.E ? run<256, true>(p, s) : run<256, false>(p, s);
  }
}

cudaError_t product_take_watchdog(int* value) {
  cudaError_t e = cudaMemcpyFromSymbol(value, g_watchdog_mx, sizeof(int));
  if (e != cudaSuccess) return e;
  const int zero = 0;
  return cudaMemcpyToSymbol(g_watchdog_mx, &zero, sizeof(int));
}

}  // namespace mx
}  // namespace imc
