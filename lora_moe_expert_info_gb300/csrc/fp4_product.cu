// fp4_product.cu -- sorted 4-bit rows times their expert's 4-bit matrix.
//
//   y[r, n] = g_a g_w[e] sum_c A[r, c] W[e, n, c],   e the expert of row r
//
// with A and W given as E2M1 codes and block scales (mlr_fp4.cuh), on the
// block-scaled FP4 tensor cores: the scales are applied inside the MMA, sums
// are held in fp32 and y is rounded once to bf16.  Rows before the first expert's
// and past the last one's are zeros.
//
// An item is 128 outputs (rows of W, the MMA's M) by one tile of up to NT rows
// of one expert (the MMA's N), so that few rows waste little of the tensor
// core and every weight is read once per tile.  One persistent CTA per SM
// walks a static share of the items; roles are warps:
//   warp 0, 3   codes: per K step of 256 columns one TMA box of W (warp 0) and
//               one of A (warp 3), rows of 128 bytes in 128-byte swizzle, into
//               a ring of stages
//   warp 2      the steps' scale atoms into a ring of their own
//   warps 12-15 scales from there to TMEM, ahead of the codes
//   warp 1      one MMA per 64 columns
//   warps 4-11  accumulators from TMEM, scaled and rounded, to y
//
// Few rows are bound by HBM (each expert's weights once), many by the pace of
// the K steps: four MMAs of 128 cycles, and the time from a stage's release to
// its next load, which four stages of 48 KB hide in part.  Measured, device
// time: 32768 rows x 128 experts x 1536 x 2048 NVFP4 69 us (5.3 TB/s of what it
// has to move, 79% of the copy rate; 3.0 PFLOP/s), 8192 rows x 32 experts x 4096 x
// 7168 MXFP4 120 us (74%; 4.0 PFLOP/s), 4096 rows x one 4096 x 7168 matrix 47 us (5.1
// PFLOP/s), 2048 rows x 128 experts x 2048 x 768 MXFP4 24 us (73%), one token's 8
// rows 6.9 us, 2 us of it bytes.
#include <cudaTypedefs.h>

#include "mlr_fp4.cuh"
#include "mlr_profile.cuh"

namespace mlr {
namespace {

constexpr int kProductThreads = 512;
constexpr int kEpilogueThreads = 256;  // warps 4-11: two per TMEM lane quarter
constexpr int kMaxProductExperts = 2048;
constexpr int kKStep = 256;      // columns per ring stage: 128 bytes of codes per row

template <int NT> struct ProductCfg;
// few rows per expert: short row tiles leave room for a deeper ring
template <> struct ProductCfg<64> { static constexpr int kStages = 8, kScaleStages = 6, kAcc1 = 64; };
// two accumulators of 256 columns and the scales do not fit TMEM: the second
// accumulator begins 128 columns in, and the epilogue drains the shared half
// first, so that the next tile's MMAs wait for half a drain only
template <> struct ProductCfg<256> { static constexpr int kStages = 4, kScaleStages = 4, kAcc1 = 128; };

template <int NT, int FMT> struct Shape {
  static constexpr int kAtoms = kKStep / (4 * fp4_block(FMT));  // scale atoms per step and 128 rows
  static constexpr int kRowBlocks = (NT + 127) / 128;
  static constexpr int S = ProductCfg<NT>::kStages, Q = ProductCfg<NT>::kScaleStages;
  static constexpr int kWBytes = 128 * 128, kABytes = NT * 128;  // a stage of codes
  static constexpr int kStride = kWBytes + kABytes;
  static constexpr int kSfBytes = kAtoms * kAtomBytes;  // scales of 128 rows; a stage: W, then A's row blocks
  static constexpr int kSfStride = (1 + kRowBlocks) * kSfBytes;
  static constexpr int kAcc1 = ProductCfg<NT>::kAcc1;  // TMEM column of the second accumulator
  static constexpr int kShared = NT - kAcc1;           // columns that both accumulators use
  // TMEM columns after the accumulators: slots for a step's scales of W and A.
  // With no more slots than stages, a warp that finds its slot free (the MMAs
  // of that many steps ago are done) also finds its stage's barrier past the
  // step before.
  static constexpr int kSfCols = kAtoms * 4 * (1 + kRowBlocks);
  static constexpr int kSfCol0 = kAcc1 + NT;
  static constexpr int kSlots = (512 - kSfCol0) / kSfCols < S ? (512 - kSfCol0) / kSfCols : S;
  static_assert(kSlots >= 2 && S <= 8 && Q <= 8 && kSfCols % 8 == 0, "slots");
  static_assert(kShared == 0 || (kShared == kAcc1 && kShared % 128 == 0), "halves of 128 columns");
};

struct __align__(16) Ctl {
  uint64_t full[8], empty[8];        // a step's codes and scales are there / its MMAs are done
  uint64_t sf_full[8], sf_empty[8];  // a stage of scales has landed / has been read
  uint64_t acc_full[2], acc_empty[2];
  uint64_t edge[2];  // the columns shared with the other accumulator have been read
  uint64_t drain;    // every MMA issued is done
  int steps[7];      // steps that warps 0, 3, 12 to 15 (arrivals on full) and 2 (on sf_full) have arrived for
  uint32_t tmem;
  int abort;
  int tiles[kMaxProductExperts + 1];  // row tiles of all earlier experts
};

template <int NT, int FMT>
constexpr int smem_bytes() {
  return Shape<NT, FMT>::S * Shape<NT, FMT>::kStride + Shape<NT, FMT>::Q * Shape<NT, FMT>::kSfStride +
         (int)sizeof(Ctl) + 1024;
}

struct Maps {
  CUtensorMap w;      // [E * N, pitch] in boxes of 128 rows
  CUtensorMap a[5];   // [P, pitch] in boxes of 16 << i rows
  CUtensorMap sw;     // W's scales, a row per 128-row block, one step per box
  CUtensorMap sa[2];  // A's scales, the same in boxes of one and two row blocks
};

struct Params {
  const float *ga, *gw;
  const int32_t* offsets;
  int P, E, N, nblk, ksteps, cols, atoms;
  uint16_t* y;
  bool pairs;  // two outputs of a row are one aligned word of y
  int32_t* status;
  uint64_t wait_ns;
};

struct Item {
  int e, row0, rows;  // expert, first sorted row, rows of the tile
  int sblk;           // 128-row scale block of row0
  int sf0;            // where row0 begins in that block: TMEM columns of 32 rows
  int n0;             // first output
};

template <int NT>
__device__ __forceinline__ Item item_of(const Params& p, const Ctl& c, int item) {
  const int t = item / p.nblk;
  int lo = 0, hi = p.E;  // tiles[lo] <= t < tiles[hi]
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (c.tiles[mid] <= t) lo = mid;
    else hi = mid;
  }
  Item it;
  it.e = lo;
  const int o0 = __ldg(p.offsets + lo), o1 = __ldg(p.offsets + lo + 1);
  const int j0 = (t - c.tiles[lo]) * NT;
  it.row0 = o0 + j0;
  it.rows = min(NT, o1 - it.row0);
  it.sblk = o0 / 128 + lo + j0 / 128;
  it.sf0 = j0 % 128 / 32;
  it.n0 = (item - t * p.nblk) * 128;
  return it;
}
// The items of a CTA, 32 at a time: lane l looks up the l-th next one, so that
// a role pays the search once for 32 items.  Whole warps call it, for i = 0, 1, ...
template <int NT>
struct ItemWalk {
  Item mine;
  __device__ __forceinline__ Item at(const Params& p, const Ctl& c, int i, int n_items, int lane) {
    if ((i & 31) == 0) {
      const int64_t item = blockIdx.x + (int64_t)(i + lane) * gridDim.x;
      if (item < n_items) mine = item_of<NT>(p, c, (int)item);
    }
    Item it;
    it.e = __shfl_sync(0xffffffffu, mine.e, i & 31);
    it.row0 = __shfl_sync(0xffffffffu, mine.row0, i & 31);
    it.rows = __shfl_sync(0xffffffffu, mine.rows, i & 31);
    it.sblk = __shfl_sync(0xffffffffu, mine.sblk, i & 31);
    it.sf0 = __shfl_sync(0xffffffffu, mine.sf0, i & 31);
    it.n0 = __shfl_sync(0xffffffffu, mine.n0, i & 31);
    return it;
  }
};
__device__ __forceinline__ int mma_rows(int rows) { return (rows + 15) & ~15; }

// Row tiles per expert, scanned over the experts; false (and the status bit)
// if the offsets are not 0 <= o[e] <= o[e + 1] <= P.
template <int NT>
__device__ bool scan_tiles(const Params& p, Ctl& c) {
  __shared__ int warp_tot[kProductThreads / 32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int per = (p.E + kProductThreads - 1) / kProductThreads;
  const int e0 = min(p.E, tid * per), e1 = min(p.E, e0 + per);
  bool bad = tid == 0 && __ldg(p.offsets + p.E) > p.P;
  int local = 0;
  for (int e = e0; e < e1; ++e) {
    const int o0 = __ldg(p.offsets + e), o1 = __ldg(p.offsets + e + 1);
    if (o0 < 0 || o1 < o0) bad = true;
    else local += (int)(((int64_t)o1 - o0 + NT - 1) / NT);
  }
  int inc = local;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += v;
  }
  if (lane == 31) warp_tot[warp] = inc;
  if (__syncthreads_or(bad)) {
    if (tid == 0) set_status(p.status, MLR_STATUS_INDEX);
    return false;
  }
  int run = inc - local;
  for (int w = 0; w < warp; ++w) run += warp_tot[w];
  for (int e = e0; e < e1; ++e) {
    c.tiles[e] = run;
    run += (__ldg(p.offsets + e + 1) - __ldg(p.offsets + e) + NT - 1) / NT;
  }
  if (tid == kProductThreads - 1) c.tiles[p.E] = run;
  __syncthreads();
  return true;
}

// TMEM -> registers without waiting: this warp's 32 lanes, 32 columns.
__device__ __forceinline__ void tmem_ld32_async(uint32_t taddr, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
        "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
        "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr)
      : "memory");
}
// Waits for every load of the warp; the registers pass through it, so that
// they are not read before.
__device__ __forceinline__ void tmem_ld_wait(uint32_t (&r)[32]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
  for (int i = 0; i < 32; ++i) asm volatile("" : "+r"(r[i]));
}

// 32 rows of y from c0 of the tile, this lane's output n.  Neighbouring lanes
// trade values so that each stores two outputs of one row at once, where those
// are a word of y; an odd number of outputs, or a y that begins between two
// words, takes single ones.
__device__ __forceinline__ void store_chunk(const Params& p, uint16_t* yp, const uint32_t (&v)[32], float s, int n,
                                            int c0, int rows, int lane) {
  if (p.pairs) {
    const int odd = lane & 1;
    uint16_t* q = yp + (int64_t)(c0 + odd) * p.N - odd;
#pragma unroll
    for (int j = 0; j < 32; j += 2) {
      const float a = s * __uint_as_float(v[j]), b = s * __uint_as_float(v[j + 1]);
      const float o = __shfl_xor_sync(0xffffffffu, odd ? a : b, 1);
      uint32_t w;
      asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w) : "f"(odd ? b : o), "f"(odd ? o : a));
      if (c0 + j + odd < rows && n < p.N) *reinterpret_cast<uint32_t*>(q) = w;
      q += 2 * (int64_t)p.N;
    }
  } else if (n < p.N) {
#pragma unroll
    for (int j = 0; j < 32; ++j)
      if (c0 + j < rows) yp[(int64_t)(c0 + j) * p.N] = f32_to_bf16_bits(s * __uint_as_float(v[j]));
  }
}

// One arrival for the warp, after all its lanes are done.
__device__ __forceinline__ void warp_arrive(uint64_t* bar, int lane) {
  __syncwarp();
  if (lane == 0) mbar_arrive(bar);
}
// Registers -> TMEM: this warp's 32 lanes, 8 columns; tmem_st_wait waits for all.
__device__ __forceinline__ void tmem_st8(uint32_t taddr, const uint32_t* v) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(taddr), "r"(v[0]),
               "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
               : "memory");
}
__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

template <int NT, int FMT>
__global__ void __launch_bounds__(kProductThreads, 1)
product_kernel(const __grid_constant__ Maps maps, const Params p) {
  using Sh = Shape<NT, FMT>;
  constexpr int S = Sh::S, Q = Sh::Q;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* smem_sf = smem + S * Sh::kStride;
  Ctl& c = *reinterpret_cast<Ctl*>(smem_sf + Q * Sh::kSfStride);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  volatile int* abort = &c.abort;

  if (tid == 0) {
    for (int s = 0; s < S; ++s) {
      mbar_init(&c.full[s], 6);  // W's load, A's load, four warps of scales
      mbar_init(&c.empty[s], 1);
    }
    for (int q = 0; q < Q; ++q) {
      mbar_init(&c.sf_full[q], 1);
      mbar_init(&c.sf_empty[q], 4);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&c.acc_full[b], 1);
      mbar_init(&c.acc_empty[b], kEpilogueThreads / 32);
      mbar_init(&c.edge[b], kEpilogueThreads / 32);
    }
    mbar_init(&c.drain, 1);
    c.abort = 0;
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(&c.tmem, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  pdl_wait();
  pdl_trigger();
  const uint32_t tmem = c.tmem;
  const bool ok_offsets = scan_tiles<NT>(p, c);
  const int n_items = ok_offsets ? c.tiles[p.E] * p.nblk : 0;

  ItemWalk<NT> walk;
  walk.mine = Item{};
  if (warp == 0 || warp == 3) {
    // ================================ codes ================================
    // W by one warp, A by the other: a stage's loads are issued side by side.
    int g = 0, il = 0;
    bool ok = true;
    for (int item = blockIdx.x; item < n_items && ok; item += gridDim.x, ++il) {
      const Item it = walk.at(p, c, il, n_items, lane);
      int bi = 0;  // the shortest box that holds the tile
      while ((16 << bi) < it.rows) ++bi;
      const CUtensorMap* map = warp == 0 ? &maps.w : &maps.a[bi];
      const int row = warp == 0 ? it.e * p.N + it.n0 : it.row0;
      const uint32_t bytes = warp == 0 ? Sh::kWBytes : (16 << bi) * 128;
      for (int k = 0; k < p.ksteps; ++k, ++g) {
        const int st = g % S;
        ok = __all_sync(0xffffffffu, mbar_wait(&c.empty[st], ((g / S) & 1) ^ 1, abort, p.wait_ns));
        if (!ok) break;
        if (elect_one()) {
          mbar_arrive_expect_tx(&c.full[st], bytes);
          tma_load_2d(smem + st * Sh::kStride + (warp == 0 ? 0 : Sh::kWBytes), map, &c.full[st], k * 128, row);
        }
        __syncwarp();
      }
    }
    if (lane == 0) c.steps[warp == 0 ? 0 : 1] = g;
  } else if (warp == 2) {
    // ============================= scale loads =============================
    int g = 0, il = 0;
    bool ok = true;
    for (int item = blockIdx.x; item < n_items && ok; item += gridDim.x, ++il) {
      const Item it = walk.at(p, c, il, n_items, lane);
      const int two = Sh::kRowBlocks > 1 && it.rows > 128;
      const int wb = it.e * p.nblk + it.n0 / 128;
      for (int k = 0; k < p.ksteps; ++k, ++g) {
        const int q = g % Q;
        ok = __all_sync(0xffffffffu, mbar_wait(&c.sf_empty[q], ((g / Q) & 1) ^ 1, abort, p.wait_ns));
        if (!ok) break;
        uint8_t* sf = smem_sf + q * Sh::kSfStride;
        if (elect_one()) {
          mbar_arrive_expect_tx(&c.sf_full[q], (2 + two) * Sh::kSfBytes);
          tma_load_2d(sf, &maps.sw, &c.sf_full[q], k * Sh::kAtoms * (kAtomBytes / 8), wb);
          tma_load_2d(sf + Sh::kSfBytes, &maps.sa[two], &c.sf_full[q], k * Sh::kAtoms * (kAtomBytes / 8), it.sblk);
        }
        __syncwarp();
      }
    }
    if (lane == 0) c.steps[6] = g;
  } else if (warp == 1) {
    // ================================= MMA =================================
    // The whole warp walks the steps, so that every operand is uniform over it
    // and stays in uniform registers; one elected lane issues.  (With a single
    // lane in the loop each MMA took 240 cycles to issue whatever its N.)
    const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
    const uint32_t sb0 = smem_u32(smem);
    int g = 0, il = 0;
    bool ok = true;
    for (int item = blockIdx.x; item < n_items && ok; item += gridDim.x, ++il) {
      const Item it = walk.at(p, c, il, n_items, lane);
      const int b = il & 1;
      ok = mbar_wait(&c.acc_empty[b], ((il >> 1) & 1) ^ 1, abort, p.wait_ns);
      if (Sh::kShared > 0 && il > 0)
        ok = mbar_wait(&c.edge[b ^ 1], ((il - 1) >> 1) & 1, abort, p.wait_ns) && ok;
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      tc_fence_after();
      const uint32_t acc = tm + b * Sh::kAcc1;
      const uint32_t id0 = idesc_fp4<FMT>(128, mma_rows(it.rows), 0), id2 = idesc_fp4<FMT>(128, mma_rows(it.rows), 2);
      for (int k = 0; k < p.ksteps; ++k, ++g) {
        const int st = g % S;
        // the codes have landed, and their scales are in TMEM
        ok = __all_sync(0xffffffffu, mbar_wait(&c.full[st], (g / S) & 1, abort, p.wait_ns));
        if (!ok) break;
        tc_fence_after();
        const uint32_t sb = sb0 + st * Sh::kStride;
        const uint32_t tw = tm + Sh::kSfCol0 + (g % Sh::kSlots) * Sh::kSfCols;
        const uint32_t ta = tw + 4 * Sh::kAtoms + it.sf0;
        const int nm = (p.cols - k * kKStep + 63) / 64;
        if (elect_one()) {
#pragma unroll
          for (int m = 0; m < 4; ++m) {
            const int i = FMT == MLR_FP4_MX ? m >> 1 : m;
            if (m < nm)
              mma_fp4<FMT>(acc, sdesc_sw128(sb + m * 32), sdesc_sw128(sb + Sh::kWBytes + m * 32),
                                 FMT == MLR_FP4_MX && (m & 1) ? id2 : id0, tw + 4 * i, ta + 4 * Sh::kRowBlocks * i,
                                 (k > 0 || m > 0) ? 1u : 0u);
          }
          mma_commit(&c.empty[st]);
        }
        __syncwarp();
      }
      if (ok && elect_one()) mma_commit(&c.acc_full[b]);
      __syncwarp();
    }
    // the MMAs read shared memory and write TMEM: whatever has given up, all that
    // were issued are done before either is freed
    if (elect_one()) mma_commit(&c.drain);
    __syncwarp();
    if (!mbar_wait_for(&c.drain, 0, kWaitLimitNs)) *abort = 1;
  } else if (warp >= 12) {
    // ============================ scales to TMEM ===========================
    // Each of the four warps writes its own lane quarter, a repetition of the
    // same 32 lanes: lane l holds bytes 16 l to 16 l + 15 of every atom, four
    // columns of it.  (Copies by tcgen05.cp take about 28 cycles each in the
    // tensor pipe, between the MMAs: 12 a step for NVFP4; 4096 rows x 4096 x 7168
    // took 57 us with them, 47 us so.)
    const uint32_t t0 = tmem + Sh::kSfCol0 + ((uint32_t)(warp & 3) << 21);
    const uint32_t sf0 = smem_u32(smem_sf) + lane * 16;
    int g = 0, il = 0;
    bool ok = true;
    for (int item = blockIdx.x; item < n_items && ok; item += gridDim.x, ++il) {
      const bool two = Sh::kRowBlocks > 1 && walk.at(p, c, il, n_items, lane).rows > 128;
      for (int k = 0; k < p.ksteps; ++k, ++g) {
        const int q = g % Q;
        ok = mbar_wait(&c.sf_full[q], (g / Q) & 1, abort, p.wait_ns);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        const uint32_t sf = sf0 + q * Sh::kSfStride;
        uint32_t v[Sh::kSfCols];  // per atom W's four columns; then per atom those of A's row blocks
#pragma unroll
        for (int i = 0; i < Sh::kAtoms; ++i) {
          const uint4 w = lds128(sf + i * kAtomBytes);
          v[4 * i] = w.x;
          v[4 * i + 1] = w.y;
          v[4 * i + 2] = w.z;
          v[4 * i + 3] = w.w;
#pragma unroll
          for (int r = 0; r < Sh::kRowBlocks; ++r) {
            uint4 a = make_uint4(0, 0, 0, 0);
            if (r == 0 || two) a = lds128(sf + (1 + r) * Sh::kSfBytes + i * kAtomBytes);
            const int o = 4 * Sh::kAtoms + 4 * (Sh::kRowBlocks * i + r);
            v[o] = a.x;
            v[o + 1] = a.y;
            v[o + 2] = a.z;
            v[o + 3] = a.w;
          }
        }
        // the MMAs of the step that used this TMEM slot last are done
        if (g >= Sh::kSlots)
          ok = mbar_wait(&c.empty[(g - Sh::kSlots) % S], ((g - Sh::kSlots) / S) & 1, abort, p.wait_ns);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        tc_fence_after();
        const uint32_t t = t0 + (g % Sh::kSlots) * Sh::kSfCols;
#pragma unroll
        for (int i = 0; i < Sh::kSfCols; i += 8) tmem_st8(t + i, v + i);
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(&c.sf_empty[q]);
          mbar_arrive(&c.full[g % S]);
        }
      }
    }
    if (lane == 0) c.steps[warp - 10] = g;
  } else if (warp >= 4) {  // 4 to 11
    // =============================== epilogue ==============================
    // Two warps per lane quarter take alternate chunks of 32 accumulator
    // columns (rows of y), first those that the next tile's accumulator shares.
    const int m = (warp & 3) * 32 + lane;  // output of the item; TMEM lane
    const int half = (warp - 4) >> 2;
    if (ok_offsets) {
      const int64_t first = (int64_t)blockIdx.x * kEpilogueThreads + tid - 128;
      const int64_t step = (int64_t)gridDim.x * kEpilogueThreads;
      for (int64_t i = first; i < (int64_t)__ldg(p.offsets) * p.N; i += step) p.y[i] = 0;
      for (int64_t i = (int64_t)__ldg(p.offsets + p.E) * p.N + first; i < (int64_t)p.P * p.N; i += step) p.y[i] = 0;
    }
    int il = 0;
    for (int item = blockIdx.x; item < n_items; item += gridDim.x, ++il) {
      const Item it = walk.at(p, c, il, n_items, lane);
      const float s = (p.ga ? __ldg(p.ga) : 1.f) * (p.gw ? __ldg(p.gw + it.e) : 1.f);
      const int b = il & 1;
      // the warp leaves together: the TMEM loads take all its lanes
      const bool w_ok = mbar_wait(&c.acc_full[b], (il >> 1) & 1, abort, p.wait_ns);
      if (!__all_sync(0xffffffffu, w_ok)) break;
      tc_fence_after();
      const uint32_t t = tmem + b * Sh::kAcc1 + ((uint32_t)(warp & 3) << 21);
      const int n = it.n0 + m;
      uint16_t* yp = p.y + (int64_t)it.row0 * p.N + n;
      constexpr int kParts = NT > 128 ? 2 : 1;  // parts of up to 128 columns, two chunks per warp
#pragma unroll
      for (int part = 0; part < kParts; ++part) {
        // the second part of the first accumulator is the first of the second
        const int c0 = (kParts == 2 && part == b ? 128 : 0) + half * 32, c1 = c0 + 64;
        uint32_t v[2][32];
        if (c0 < it.rows) tmem_ld32_async(t + c0, v[0]);
        if (NT > 64 && c1 < it.rows) tmem_ld32_async(t + c1, v[1]);
        tmem_ld_wait(v[0]);
        tmem_ld_wait(v[1]);
        tc_fence_before();
        if (Sh::kShared > 0 && part == 0) warp_arrive(&c.edge[b], lane);
        if (part == kParts - 1) warp_arrive(&c.acc_empty[b], lane);
        if (c0 < it.rows) store_chunk(p, yp, v[0], s, n, c0, it.rows, lane);
        if (NT > 64 && c1 < it.rows) store_chunk(p, yp, v[1], s, n, c1, it.rows, lane);
      }
    }
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();  // every role has left: the abort flag is final
  if (*abort) {
    if (tid == 0) set_status(p.status, MLR_STATUS_TIMEOUT);
    // Copies already issued land before their shared memory is given up.  A stage
    // has at most one step whose copies may be under way, the last that a loader
    // arrived for (it found the MMAs of the step before done): roles that did not
    // come to that step are stood in for, so that its barrier completes with its
    // bytes.  Scales have their loader's arrival only.
    if (tid < S) {
      const int last = c.steps[0] > c.steps[1] ? c.steps[0] : c.steps[1];
      if (last > tid) {
        const int g = tid + (last - 1 - tid) / S * S;
        for (int r = 0; r < 6; ++r)
          if (c.steps[r] <= g) mbar_arrive(&c.full[tid]);
        mbar_wait_for(&c.full[tid], (g / S) & 1, kWaitLimitNs);
      }
    } else if (tid >= 32 && tid - 32 < Q && c.steps[6] > tid - 32) {
      const int q = tid - 32, g = q + (c.steps[6] - 1 - q) / Q * Q;
      mbar_wait_for(&c.sf_full[q], (g / Q) & 1, kWaitLimitNs);
    }
  }
  __syncthreads();
  if (warp == 1) tmem_dealloc(tmem, 512);
}

// ------------------------------------------------------------------ host side --
PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = [] {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      f = nullptr;
    return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(f);
  }();
  return fn;
}

// Code rows of `pitch` bytes in boxes of 128 bytes x box_rows, 128-byte swizzle.
// Bytes past the pitch and rows past the last read as zero codes.
bool code_map(CUtensorMap* m, const void* base, uint64_t pitch, uint64_t rows, uint32_t box_rows) {
  auto fn = encode_fn();
  if (fn == nullptr) return false;
  cuuint64_t dims[2] = {pitch, rows};
  cuuint64_t strides[1] = {pitch};
  cuuint32_t box[2] = {128, box_rows};
  cuuint32_t es[2] = {1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(base), dims, strides, box, es,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Scales as rows of 128-row blocks, in boxes of one step of `boxes` row blocks;
// atoms past the last one read as zeros.
bool scale_map(CUtensorMap* m, const void* base, uint64_t atoms, uint64_t blocks, uint32_t box_atoms, uint32_t boxes) {
  auto fn = encode_fn();
  if (fn == nullptr) return false;
  cuuint64_t dims[2] = {atoms * (kAtomBytes / 8), blocks};  // in 8-byte elements: a box has at most 256 a side
  cuuint64_t strides[1] = {atoms * kAtomBytes};
  cuuint32_t box[2] = {box_atoms * (kAtomBytes / 8), boxes};
  cuuint32_t es[2] = {1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_INT64, 2, const_cast<void*>(base), dims, strides, box, es,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// SMs of the current device, after opting the kernel in to its shared memory;
// kept per device.  0: an error.
template <int NT, int FMT>
int product_sms() {
  constexpr int smem = smem_bytes<NT, FMT>();
  static_assert(smem <= 227 * 1024, "shared memory per CTA");
  static int sms[64] = {};
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 0;
  if (sms[dev] != 0) return sms[dev];
  if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n <= 0 ||
      cudaFuncSetAttribute(product_kernel<NT, FMT>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess)
    return 0;
  sms[dev] = n;
  return n;
}

template <int NT, int FMT>
int launch_product(Maps& maps, Params& p, const uint8_t* a, const uint8_t* sa, const uint8_t* sw, uint64_t pitch,
                   cudaStream_t stream) {
  using Sh = Shape<NT, FMT>;
  // at most one partial tile per expert beyond the full ones
  const int64_t tiles = (p.P < p.E ? p.P : p.E) + (int64_t)p.P / NT;
  const int64_t items = tiles * p.nblk;
  if (items > INT32_MAX) return MLR_ERR_UNSUPPORTED;
  const int sms = product_sms<NT, FMT>();
  if (sms == 0) {
    (void)cudaGetLastError();
    return MLR_ERR_CUDA;
  }
  bool ok = scale_map(&maps.sw, sw, p.atoms, (uint64_t)p.E * p.nblk, Sh::kAtoms, 1);
  for (int i = 0; i < Sh::kRowBlocks; ++i)
    ok = ok && scale_map(&maps.sa[i], sa, p.atoms, (uint64_t)p.P / 128 + p.E, Sh::kAtoms, i + 1);
  for (uint32_t i = 0, rows = 16; rows <= NT; ++i, rows *= 2)
    ok = ok && code_map(&maps.a[i], a, pitch, (uint64_t)p.P, rows);
  if (!ok) return MLR_ERR_CUDA;
  if (launch_pdl(product_kernel<NT, FMT>, dim3((unsigned)(items < sms ? items : sms)), dim3(kProductThreads),
                 smem_bytes<NT, FMT>(), stream, maps, p) != cudaSuccess) {
    (void)cudaGetLastError();
    return MLR_ERR_CUDA;
  }
  note_launch();
  return MLR_OK;
}

}  // namespace
}  // namespace mlr

extern "C" int moe_fp4_expert_product(const uint8_t* a_codes, const uint8_t* a_scales, const float* a_tensor_scale,
                                      const uint8_t* w_codes, const uint8_t* w_scales, const float* w_tensor_scale,
                                      const int32_t* expert_offsets, int32_t num_rows, int32_t num_experts,
                                      int32_t outputs, int32_t cols, int32_t fmt, mlr_bf16* y, int32_t* d_status,
                                      void* stream_) {
  using namespace mlr;
  cudaStream_t stream = static_cast<cudaStream_t>(stream_);
  if (num_rows < 0 || num_experts < 1 || outputs < 1 || cols < 1 || (fmt != MLR_FP4_MX && fmt != MLR_FP4_NV))
    return MLR_ERR_INVALID;
  if (fmt == MLR_FP4_MX && (a_tensor_scale != nullptr || w_tensor_scale != nullptr)) return MLR_ERR_INVALID;
  if (num_experts > kMaxProductExperts || cols > (1 << 19) || (int64_t)num_experts * outputs > INT32_MAX)
    return MLR_ERR_UNSUPPORTED;
  if (num_rows == 0) return MLR_OK;
  for (const void* q : {static_cast<const void*>(a_codes), static_cast<const void*>(a_scales),
                        static_cast<const void*>(w_codes), static_cast<const void*>(w_scales)})
    if (q == nullptr || (reinterpret_cast<uintptr_t>(q) & 15) != 0) return MLR_ERR_INVALID;
  const uintptr_t ya = reinterpret_cast<uintptr_t>(y);
  if (expert_offsets == nullptr || y == nullptr || (ya & 1) != 0) return MLR_ERR_INVALID;
  const uint64_t pitch = (uint64_t)fp4_pitch(cols);
  Maps maps = {};
  if (!code_map(&maps.w, w_codes, pitch, (uint64_t)num_experts * outputs, 128)) return MLR_ERR_CUDA;
  Params p{a_tensor_scale, w_tensor_scale, expert_offsets, num_rows, num_experts, outputs,
           (int)ceil_div(outputs, 128), (int)ceil_div(cols, kKStep), cols, fp4_atoms(cols, fmt), y,
           outputs % 2 == 0 && ya % 4 == 0, d_status, wait_limit_ns()};
  // an average expert of at most 32 rows rarely needs a second 64-row tile
  const bool small = num_rows <= 32 * (int64_t)num_experts || num_rows <= 64;
  auto run = [&](auto launch) { return launch(maps, p, a_codes, a_scales, w_scales, pitch, stream); };
  if (fmt == MLR_FP4_MX) return small ? run(launch_product<64, MLR_FP4_MX>) : run(launch_product<256, MLR_FP4_MX>);
  return small ? run(launch_product<64, MLR_FP4_NV>) : run(launch_product<256, MLR_FP4_NV>);
}
