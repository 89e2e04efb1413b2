// permute.cu -- tokens sorted by expert and back, with their gradients.
//
// A pair p = t*K + k is token t's k-th choice, e(p) = topk_ids[p] its expert.
// The sorted order is stable: by expert, then by p; pairs whose id is not in
// [0, E) ("masked") come after all others, in increasing p.  With pos(p) the
// place of pair p:
//   permute            rows[pos(p)] = x[p / K], 0 for a masked pair
//   its gradient       dx[t] = sum_k d_rows[pos(t, k)]
//   unpermute          y[t] = sum_k w[t, k] rows[pos(t, k)]
//   its gradients      d_rows[pos(t, k)] = w[t, k] dy[t];  dw[t, k] = <dy[t], rows[pos(t, k)]>
// where the sums over k skip masked pairs, run in increasing k and are held in
// fp32, so results are bit-identical between runs.  pair_pos stores pos(p),
// or ~pos(p) (negative) for a masked pair.
//
// All four move rows once and are bound by HBM (bytes = rows read + rows
// written; copy rate 6.67 TB/s), small ones by launch latency.  8192 tokens x 8
// experts x 7168 bf16: permute 182 us (87% of the copy rate, 11 us of it the
// sort), its gradient and unpermute 154 us (103%), unpermute's gradients 300 us
// (100%).  1 to 256 tokens: 6 to 9 us.
#include "mlr_profile.cuh"

namespace mlr {
namespace {

constexpr int kSortThreads = 256;
constexpr int kChunkPairs = 256;     // pairs of one block, ranked by comparison in shared memory
constexpr int kCountChunks = 8;      // chunks counted by one block, a warp each
constexpr int kMaxSortTopk = 256;    // one token's pairs fit a chunk
constexpr int kMaxSortExperts = 16384;
constexpr int kMaxHidden = 1 << 24;
// Up to this many pairs every block counts all of them itself, which saves the
// two launches that count and scan them for larger batches; twice as many where
// no rows are copied (9186 pairs: 7.3 us, in three launches 11.6, 16000: 9.7 and
// 11.6, 24000: 10.3 to 11.7; with rows of 4 KB copied, 9600 pairs 16 and 14).
constexpr int64_t kOneLaunchPairs = 8192;
constexpr int64_t kOneLaunchSorted = 16384;

struct SortPlan {
  bool ok;
  int code;
  int64_t P;
  int tpb;        // tokens per block
  int64_t G, Gp;  // blocks (chunks), and their number rounded up to whole 32-byte sectors of counts
  bool one;       // a single launch
  int64_t o_tot;  // workspace: counts [E+1][G], then totals [E+1]
  int64_t bytes;
};

SortPlan sort_plan(int32_t T, int32_t K, int32_t E, int64_t one_launch) {
  SortPlan s{};
  s.code = MLR_ERR_INVALID;
  if (T < 0 || K < 1 || E < 1) return s;
  s.P = (int64_t)T * K;
  if (K > kMaxSortTopk || E > kMaxSortExperts || s.P >= INT32_MAX) {
    s.code = MLR_ERR_UNSUPPORTED;
    return s;
  }
  // enough blocks to spread the copies over the SMs, few enough to keep the
  // count matrix small; a block's pairs never exceed a chunk
  s.one = s.P <= one_launch;
  const int64_t want = ceil_div(T, s.one ? 512 : 1024);
  const int most = kChunkPairs / K;
  s.tpb = (int)(want < 1 ? 1 : want > most ? most : want);
  s.G = ceil_div(T, s.tpb);
  s.Gp = round_up(s.G, kCountChunks);
  s.o_tot = round_up((int64_t)(E + 1) * s.Gp * 4, 256);
  s.bytes = s.one ? 1 : s.o_tot + round_up((int64_t)(E + 1) * 4, 256);  // one launch: nothing is kept
  s.ok = true;
  s.code = MLR_OK;
  return s;
}

__device__ __forceinline__ int sort_key(int id, int E) { return (id < 0 || id >= E) ? E : id; }

// Exclusive scan of s[0..n) in place over the whole block; s[n] gets the total.
__device__ void block_scan(int* s, int n) {
  __shared__ int warp_tot[kSortThreads / 32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int per = (n + kSortThreads - 1) / kSortThreads;
  const int b0 = min(n, (int)threadIdx.x * per), b1 = min(n, b0 + per);
  int local = 0;
  for (int b = b0; b < b1; ++b) local += s[b];
  int inc = local;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += v;
  }
  if (lane == 31) warp_tot[warp] = inc;
  __syncthreads();
  int run = inc - local;
  for (int w = 0; w < warp; ++w) run += warp_tot[w];
  for (int b = b0; b < b1; ++b) {
    const int c = s[b];
    s[b] = run;
    run += c;
  }
  if (threadIdx.x == kSortThreads - 1) s[n] = run;
  __syncthreads();
}

// Counts of eight chunks' pairs per expert (masked pairs as expert E), a warp
// per chunk: cnt[e][g], whole sectors at a time.  WIDE: the histograms of eight
// warps fit shared memory; else the chunks are counted one after another.
template <bool WIDE>
__global__ void __launch_bounds__(kSortThreads)
sort_count_kernel(const int32_t* __restrict__ ids, int64_t P, int E, int chunk, int64_t Gp, int32_t* __restrict__ cnt) {
  extern __shared__ int hist[];  // [WIDE ? 8 : 1][E + 1]
  constexpr int kHist = WIDE ? kCountChunks : 1;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  pdl_wait();
  pdl_trigger();
  for (int c0 = 0; c0 < kCountChunks; c0 += kHist) {
    __syncthreads();
    for (int i = threadIdx.x; i < kHist * (E + 1); i += kSortThreads) hist[i] = 0;
    __syncthreads();
    const int64_t g = (int64_t)blockIdx.x * kCountChunks + c0 + (WIDE ? warp : 0);
    int* h = hist + (WIDE ? warp * (E + 1) : 0);
    for (int i = WIDE ? lane : threadIdx.x; i < chunk; i += WIDE ? 32 : kSortThreads) {
      const int64_t p = g * chunk + i;
      if (p < P) atomicAdd(&h[sort_key(__ldg(ids + p), E)], 1);
    }
    __syncthreads();
    for (int i = threadIdx.x; i < kHist * (E + 1); i += kSortThreads) {
      const int e = i / kHist, c = i - e * kHist;
      cnt[(int64_t)e * Gp + (int64_t)blockIdx.x * kCountChunks + c0 + c] = hist[c * (E + 1) + e];
    }
  }
}

// One block per expert: the exclusive scan of its chunk counts, in place, four
// to a thread, and its total.
__global__ void __launch_bounds__(kSortThreads)
sort_scan_kernel(int32_t* __restrict__ cnt, int64_t Gp, int32_t* __restrict__ tot) {
  __shared__ int warp_tot[kSortThreads / 32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int4* c = reinterpret_cast<int4*>(cnt + (int64_t)blockIdx.x * Gp);
  pdl_wait();
  pdl_trigger();
  int carry = 0;
  for (int64_t g0 = 0; g0 < Gp / 4; g0 += kSortThreads) {
    const int64_t g = g0 + threadIdx.x;
    const int4 v = g < Gp / 4 ? c[g] : make_int4(0, 0, 0, 0);
    const int mine = v.x + v.y + v.z + v.w;
    int inc = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int u = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += u;
    }
    if (lane == 31) warp_tot[warp] = inc;
    __syncthreads();
    int run = carry + inc - mine;
    for (int w = 0; w < kSortThreads / 32; ++w) {
      if (w < warp) run += warp_tot[w];
      carry += warp_tot[w];
    }
    if (g < Gp / 4) c[g] = make_int4(run, run + v.x, run + v.x + v.y, run + v.x + v.y + v.z);
    __syncthreads();
  }
  if (threadIdx.x == 0) tot[blockIdx.x] = carry;
}

// The aligned 16 bytes at a of the array [base, end); where they reach past one
// of its ends, the elements inside, zeros elsewhere.
template <typename E_>
__device__ __forceinline__ uint4 load_piece(const char* a, const E_* base, const E_* end) {
  if (a >= reinterpret_cast<const char*>(base) && a + 16 <= reinterpret_cast<const char*>(end))
    return __ldg(reinterpret_cast<const uint4*>(a));
  uint4 q = make_uint4(0, 0, 0, 0);
  E_* e = reinterpret_cast<E_*>(&q);
#pragma unroll
  for (int i = 0; i < 16 / (int)sizeof(E_); ++i) {
    const E_* p = reinterpret_cast<const E_*>(a) + i;
    if (p >= base && p < end) e[i] = __ldg(p);
  }
  return q;
}
// Bytes s to s + 16 of a and b one after the other (s a multiple of the element).
template <typename E_>
__device__ __forceinline__ uint4 shifted(const uint4& a, const uint4& b, int s) {
  uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
  for (int i = 0; i < 6; ++i) w[i] = s & 8 ? w[i + 2] : w[i];
#pragma unroll
  for (int i = 0; i < 5; ++i) w[i] = s & 4 ? w[i + 1] : w[i];
  if (sizeof(E_) == 2)
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = __funnelshift_r(w[i], w[i + 1], 8 * (s & 2));
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// The part of a row that a warp copies at a time.
constexpr int kItemBytes = 2048;
// Rows of at most as many vectors are copied a vector to a thread, whatever token
// it is of (300000 x 8 rows of 128 bytes: 126 us, by warps 247, 86 of it the sort;
// 15011 x 6 of 512 bytes 18.9 and 19.7, of 1 KB 27.5 and 26.3).
constexpr int kShortVecs = 32;

// One such part (its aligned pieces from byte b on) of a row off the 16-byte
// grid, copied to the K rows by a warp: a lane holds four pieces and what follows
// each, of which every destination takes 16-byte pieces in its own alignment;
// the row's ends, which share 16 bytes with another row, go element by element.
// [x, end): the array; bytes: of the row, at most 2^26.  8192 x 6 rows of 1111
// bf16, sort included: 34 us (through shared memory 41, element by element 61);
// 3000 x 2 of 7001 float32: 53 us (77).
template <typename E_>
__device__ void copy_unaligned(const char* __restrict__ src, int bytes, char* __restrict__ rows,
                               const int* __restrict__ place, int K, const E_* x, const E_* end, int b,
                               int lane) {
  constexpr int kVec = kItemBytes / 512, es = (int)sizeof(E_);
  const int ps = (int)(reinterpret_cast<uintptr_t>(src) & 15);
  uint4 v[kVec], next[kVec];
#pragma unroll
  for (int u = 0; u < kVec; ++u) {
    const int at = b + 16 * (32 * u + lane);
    v[u] = at < ps + bytes ? load_piece<E_>(src - ps + at, x, end) : make_uint4(0, 0, 0, 0);
  }
  uint4 past = make_uint4(0, 0, 0, 0);
  if (lane == 31 && b + kVec * 512 < ps + bytes) past = load_piece<E_>(src - ps + b + kVec * 512, x, end);
#pragma unroll
  for (int u = 0; u < kVec; ++u) {
    const uint4 t = v[u], f = u + 1 < kVec ? v[u + 1 < kVec ? u + 1 : 0] : past;
    // lane 31's neighbour is lane 0 of the next 32 pieces
    const uint4 give = lane == 0 && u + 1 < kVec ? f : t;
    next[u].x = __shfl_sync(0xffffffffu, give.x, (lane + 1) & 31);
    next[u].y = __shfl_sync(0xffffffffu, give.y, (lane + 1) & 31);
    next[u].z = __shfl_sync(0xffffffffu, give.z, (lane + 1) & 31);
    next[u].w = __shfl_sync(0xffffffffu, give.w, (lane + 1) & 31);
    if (u + 1 == kVec && lane == 31) next[u] = past;
  }
  for (int k = 0; k < K; ++k) {
    const int at = place[k];
    char* dst = rows + (int64_t)(at < 0 ? ~at : at) * bytes;
    const int off = (int)(-reinterpret_cast<uintptr_t>(dst) & 15);  // to the first 16-byte piece
    const int r = (ps + off) & 15;
#pragma unroll
    for (int u = 0; u < kVec; ++u) {
      if (b + 512 * u >= ps + bytes) break;
      const int d = b + 16 * (32 * u + lane) + r - ps;
      if (d >= 0 && d + 16 <= bytes)
        *reinterpret_cast<uint4*>(dst + d) = at < 0 ? make_uint4(0, 0, 0, 0) : shifted<E_>(v[u], next[u], r);
    }
    if (b == 0) {  // the row's first bytes (lanes 0 to 7), and its last ones (16 to 23)
      const int tail = bytes <= off ? bytes : off + (bytes - off) / 16 * 16;  // end of the 16-byte pieces
      const int t = lane < 16 ? lane * es : tail + (lane - 16) * es;
      if (t < (lane < 16 ? min(off, bytes) : bytes))
        *reinterpret_cast<E_*>(dst + t) = at < 0 ? E_{} : __ldg(reinterpret_cast<const E_*>(src + t));
    }
  }
}

// Places the pairs of one chunk of tokens and copies this block's column slice
// of their rows.  The rank of a pair inside the chunk is the number of earlier
// chunk pairs with the same key, counted by comparison.  VB: 16 where rows and
// bases are multiples of 16 bytes, 32 for long ones of them, else the element's
// size.
template <int VB> struct CopyElement;
template <> struct CopyElement<4> { using type = uint32_t; };
template <> struct CopyElement<2> { using type = uint16_t; };

// Rows off the grid: four blocks per SM (9836 x 5 rows of 1513 bf16: 46 us, three 52).
template <int VB, bool ONE>
__global__ void __launch_bounds__(kSortThreads, VB < 16 ? 4 : 1)
permute_kernel(const void* __restrict__ x, const int32_t* __restrict__ ids, int T, int K, int E, int tpb, int64_t Gp,
               int64_t row_bytes /* 0: sort only */, void* __restrict__ rows,
               int32_t* __restrict__ pair_pos, int32_t* __restrict__ offsets, const int32_t* __restrict__ cnt,
               const int32_t* __restrict__ tot, int32_t* d_status) {
  extern __shared__ int start[];  // [E + 2] first rows; ONE: and [E + 1] counts of earlier pairs
  __shared__ int key[kChunkPairs];
  __shared__ int place[kChunkPairs];
  const int tid = threadIdx.x;
  const int64_t P = (int64_t)T * K;
  const int64_t t0 = (int64_t)blockIdx.x * tpb;
  const int nt = (int)min((int64_t)tpb, T - t0);
  const int np = nt * K;
  const int64_t p0 = t0 * K;
  int* before = start + E + 2;
  if (ONE) {
    for (int e = tid; e <= E; e += kSortThreads) start[e] = before[e] = 0;
    __syncthreads();
  }
  pdl_wait();
  pdl_trigger();
  if (ONE) {
    for (int p = tid; p < (int)P; p += kSortThreads) {
      const int k = sort_key(__ldg(ids + p), E);
      atomicAdd(&start[k], 1);
      if (p < p0) atomicAdd(&before[k], 1);
    }
  } else {
    for (int e = tid; e <= E; e += kSortThreads) start[e] = __ldg(tot + e);
  }
  int mine = -1;
  if (tid < np) {
    const int id = __ldg(ids + p0 + tid);
    mine = sort_key(id, E);
    key[tid] = mine;
    if (mine == E && id != -1) set_status(d_status, MLR_STATUS_INDEX);
  }
  __syncthreads();
  block_scan(start, E + 1);
  if (tid < np) {
    int r = 0;
    for (int j = 0; j < tid; ++j) r += key[j] == mine;
    r += start[mine] + (ONE ? before[mine] : __ldg(cnt + (int64_t)mine * Gp + blockIdx.x));
    const int at = mine == E ? ~r : r;
    place[tid] = at;
    if (blockIdx.y == 0) pair_pos[p0 + tid] = at;
  }
  if (blockIdx.x == 0 && blockIdx.y == 0)
    for (int e = tid; e <= E; e += kSortThreads) offsets[e] = start[e];
  if (row_bytes == 0) return;
  __syncthreads();
  // each piece of a token's row is read once and written to its K rows; a warp
  // takes a part of 2 KB at a time, as a block may have fewer tokens than warps
  // (4096 x 8 rows of 4 KB: 31.5 us, a token to a warp 36)
  auto row_items = [&](int64_t bytes) {
    return (int)ceil_div(ceil_div(bytes, kItemBytes) - (int64_t)blockIdx.y, (int64_t)gridDim.y);
  };
  const int lane = tid & 31, warp = tid >> 5;
  if constexpr (VB < 16) {
    using V = typename CopyElement<VB>::type;
    const V* end = static_cast<const V*>(x) + T * (row_bytes / (int)sizeof(V));
    const int items = row_items(row_bytes + 15);
    for (int it = warp; it < nt * items; it += kSortThreads / 32) {
      const int i = it / items;
      const int b = ((it - i * items) * (int)gridDim.y + (int)blockIdx.y) * kItemBytes;
      copy_unaligned<V>(static_cast<const char*>(x) + (t0 + i) * row_bytes, (int)row_bytes, static_cast<char*>(rows),
                        place + i * K, K, static_cast<const V*>(x), end, b, lane);
    }
  } else {
    // a warp per part, or for long rows the block, so that their copies are
    // written in long runs (8192 x 8 rows of 14 KB: 183 us, by warps 197;
    // 16384 x 4 rows of 2 KB: 50 us, by warps 38)
    const int64_t nvec = row_bytes / 16;
    const uint4* xv = static_cast<const uint4*>(x);
    uint4* rv = static_cast<uint4*>(rows);
    // vectors c, c + step, c + 2 step and c + 3 step of the block's token i
    auto copy = [&](int i, int64_t c, int64_t step) {
      const uint4* src = xv + (t0 + i) * nvec;
      uint4 v[4];
#pragma unroll
      for (int u = 0; u < 4; ++u)
        if (c + u * step < nvec) v[u] = __ldg(src + c + u * step);
      for (int k = 0; k < K; ++k) {
        const int at = place[i * K + k];
        uint4* dst = rv + (int64_t)(at < 0 ? ~at : at) * nvec;
#pragma unroll
        for (int u = 0; u < 4; ++u)
          if (c + u * step < nvec) dst[c + u * step] = at < 0 ? make_uint4(0, 0, 0, 0) : v[u];
      }
    };
    if (VB == 32) {
      const int64_t step = (int64_t)gridDim.y * kSortThreads;
      for (int i = 0; i < nt; ++i)
        for (int64_t c = (int64_t)blockIdx.y * kSortThreads + tid; c < nvec; c += 4 * step) copy(i, c, step);
    } else if (nvec <= kShortVecs) {
      // the block's tokens are one run of vectors; such rows are never sliced
      const int n = (int)nvec, all = nt * n;
      for (int f = tid; f < all; f += kSortThreads) {
        const int i = f / n, c = f - i * n;
        const uint4 v = __ldg(xv + t0 * nvec + f);
        for (int k = 0; k < K; ++k) {
          const int at = place[i * K + k];
          rv[(int64_t)(at < 0 ? ~at : at) * nvec + c] = at < 0 ? make_uint4(0, 0, 0, 0) : v;
        }
      }
    } else {
      const int items = row_items(row_bytes);
      for (int it = warp; it < nt * items; it += kSortThreads / 32) {
        const int i = it / items;
        copy(i, ((int64_t)(it - i * items) * gridDim.y + blockIdx.y) * (kItemBytes / 16) + lane, 32);
      }
    }
  }
}

// ------------------------------------------------------------ row vectors --
// 16 bytes of a row as fp32 values (4 float32 or 8 bf16), and back.
__device__ __forceinline__ void widen(const uint4& q, float (&v)[4]) {
  v[0] = __uint_as_float(q.x);
  v[1] = __uint_as_float(q.y);
  v[2] = __uint_as_float(q.z);
  v[3] = __uint_as_float(q.w);
}
__device__ __forceinline__ void widen2(uint32_t w, float& a, float& b) {
  a = __uint_as_float(w << 16);
  b = __uint_as_float(w & 0xffff0000u);
}
__device__ __forceinline__ void widen(const uint4& q, float (&v)[8]) {
  widen2(q.x, v[0], v[1]);
  widen2(q.y, v[2], v[3]);
  widen2(q.z, v[4], v[5]);
  widen2(q.w, v[6], v[7]);
}
__device__ __forceinline__ uint32_t narrow2(float a, float b) {
  uint32_t o;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(o) : "f"(b), "f"(a));
  return o;
}
__device__ __forceinline__ void narrow(const float (&v)[4], uint4& q) {
  q = make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3]));
}
__device__ __forceinline__ void narrow(const float (&v)[8], uint4& q) {
  q = make_uint4(narrow2(v[0], v[1]), narrow2(v[2], v[3]), narrow2(v[4], v[5]), narrow2(v[6], v[7]));
}
__device__ __forceinline__ float widen1(uint16_t v) { return __uint_as_float((uint32_t)v << 16); }

// How a thread takes 16 bytes of a row.  kWhole: rows and bases are multiples of
// 16 bytes.  kPieces (bf16 rows off that grid): in the two aligned pieces that
// they lie in, the second one mostly from L1, and shifted.  kStrided (float32
// rows off it): four elements a row of threads apart, each access of a warp
// being 128 bytes in a row.
enum RowAccess { kWhole, kPieces, kStrided };
template <typename E_> constexpr RowAccess kOffGrid = sizeof(E_) == 2 ? kPieces : kStrided;

// Elements c, c + step, ... of a row of H float32, zeros past its end; and back.
__device__ __forceinline__ uint4 load_strided(const float* r, int c, int step, int H) {
  float v[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = c + i * step < H ? __ldg(r + c + i * step) : 0.f;
  return make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3]));
}
__device__ __forceinline__ void store_strided(float* r, int c, int step, int H, const uint4& q) {
  const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (c + i * step < H) r[c + i * step] = __uint_as_float(w[i]);
}

// The threads of a token: a power of two, so that short rows share a block.
int row_threads(int nv, int most) {
  int l = 8;
  while (l < nv && l < most) l *= 2;
  return l;
}

// y[t] = sum_k w[t, k] rows[pos]; w == nullptr: w = 1 (the gradient of permute).
// One thread per 16 bytes of a token, or a few of them a row of threads apart;
// KU rows are loaded before any is added,
// without branches, so that their loads are in flight together.
constexpr int kSumThreads = 128;
// As many that fewest of the last ones have nothing to do (8192 x 6 rows of 1111
// bf16, 139 vectors: 34 us with 16, 41 with 128; 14599 x 4 of 640, 80: 18 and 21).
int sum_threads(int nv) {
  int best = row_threads(nv, kSumThreads);
  for (int l = best / 2; l >= 8; l /= 2)
    if (10 * round_up(nv, l) <= 9 * round_up(nv, best)) best = l;
  return best;
}
// Vectors per thread, so that few rows per token leave as many loads in flight
// (13273 rows of 5656 float32, top-1: 87 us, with one vector 160).
template <int KU, RowAccess A> constexpr int kVecs = A != kWhole || KU >= 6 ? 1 : KU == 4 ? 2 : 4;
template <typename E_, int KU, RowAccess A>
__global__ void __launch_bounds__(kSumThreads)
unpermute_kernel(const E_* __restrict__ rows, const int32_t* __restrict__ pair_pos, const float* __restrict__ w, int T,
                 int K, int H, int lpt_log2, unsigned col_blocks, E_* __restrict__ y, int32_t* d_status) {
  constexpr int N = 16 / (int)sizeof(E_), U = kVecs<KU, A>;
  pdl_wait();
  pdl_trigger();
  const unsigned tb = blockIdx.x / col_blocks, cb = blockIdx.x - tb * col_blocks;
  const int64_t t = ((int64_t)tb << (7 - lpt_log2)) + (threadIdx.x >> lpt_log2);
  const int lpt = 1 << lpt_log2, lt = threadIdx.x & (lpt - 1);
  const int c0 = A == kStrided ? (int)cb * N * lpt + lt : ((int)cb * U * lpt + lt) * N;  // first column
  if (t >= T || c0 >= H) return;
  const int64_t P = (int64_t)T * K;
  float acc[U][N];
#pragma unroll
  for (int j = 0; j < U * N; ++j) acc[j / N][j % N] = 0.f;
  for (int k0 = 0; k0 < K; k0 += KU) {
    uint4 v[KU][U], v2[A == kPieces ? KU : 1];
    int shift[A == kPieces ? KU : 1];
    float wk[KU];
#pragma unroll
    for (int j = 0; j < KU; ++j) {
      const int64_t p = t * K + k0 + j;
      const int q = k0 + j < K ? __ldg(pair_pos + p) : -1;
      const bool use = q >= 0 && q < P;
      if (q >= P) set_status(d_status, MLR_STATUS_INDEX);
      wk[j] = !use ? 0.f : w != nullptr ? __ldg(w + p) : 1.f;
      const E_* r = rows + (int64_t)q * H + c0;
      if constexpr (A == kWhole) {
#pragma unroll
        for (int i = 0; i < U; ++i)
          v[j][i] = use && c0 + i * lpt * N < H ? __ldg(reinterpret_cast<const uint4*>(r) + i * lpt)
                                                : make_uint4(0, 0, 0, 0);
      } else if constexpr (A == kStrided) {
        v[j][0] = load_strided(rows + (int64_t)q * H, c0, lpt, use ? H : 0);
      } else {
        const int s = (int)(reinterpret_cast<uintptr_t>(r) & 15);
        const char* a = reinterpret_cast<const char*>(r) - s;
        const int n = min(N, H - c0) * (int)sizeof(E_);  // bytes of the row from r on
        shift[j] = s;
        v[j][0] = use ? load_piece<E_>(a, rows, rows + P * H) : make_uint4(0, 0, 0, 0);
        v2[j] = use && s + n > 16 ? load_piece<E_>(a + 16, rows, rows + P * H) : make_uint4(0, 0, 0, 0);
      }
    }
#pragma unroll
    for (int j = 0; j < KU; ++j)
#pragma unroll
      for (int i = 0; i < U; ++i) {
        float f[N];
        if constexpr (A == kPieces) widen(shifted<E_>(v[j][i], v2[j], shift[j]), f);
        else widen(v[j][i], f);
#pragma unroll
        for (int u = 0; u < N; ++u) acc[i][u] = fmaf(wk[j], f[u], acc[i][u]);
      }
  }
  E_* out = y + t * H + c0;
#pragma unroll
  for (int i = 0; i < U; ++i) {
    uint4 o;
    narrow(acc[i], o);
    if constexpr (A == kWhole) {
      if (c0 + i * lpt * N < H) reinterpret_cast<uint4*>(out)[i * lpt] = o;
    } else if constexpr (A == kStrided) {
      store_strided(y + t * H, c0, lpt, H, o);
    } else {
      const E_* e = reinterpret_cast<const E_*>(&o);
#pragma unroll
      for (int u = 0; u < N; ++u)
        if (c0 + u < H) out[u] = e[u];
    }
  }
}

// The row gradients of a token's pairs and the dot products that are its
// weights' gradients, by 2^lpt_log2 threads per token (per thread over its
// columns in increasing order, then over lanes and warps in a fixed order).
// Bound by the bytes in flight: eight rows of a token are loaded at once, at
// most 85 registers a thread for three blocks per SM.  8192 x 8 rows of 7168
// bf16: 300 us so, 530 at 110 registers, 324 at 64 (spills); with 128 threads
// per token instead of 256, 4096 x 8 rows of 2048 take 48 us instead of 53.  With
// one or two rows per token a thread takes four or two vectors at once (13273
// rows of 5656 float32, top-1: 126 us instead of 148).
constexpr int kBackThreads = 256, kBackLanes = 128;

// Sums dot[j] over the 2^lpt_log2 threads of a token (whole groups of the block)
// and writes the token's weight gradients of pairs k0 on.
template <int KU>
__device__ __forceinline__ void store_dots(float (&dot)[KU], float (*part)[KU], int lpt, int lt, bool in, int64_t t,
                                           int K, int k0, float* __restrict__ dw) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int j = 0; j < KU; ++j)
    for (int o = min(lpt, 32) >> 1; o > 0; o >>= 1) dot[j] += __shfl_xor_sync(0xffffffffu, dot[j], o);
  if (lpt <= 32) {
    if (lt == 0 && in)
#pragma unroll
      for (int j = 0; j < KU; ++j)
        if (k0 + j < K) dw[t * K + k0 + j] = dot[j];
    return;
  }
  if (lane == 0)
#pragma unroll
    for (int j = 0; j < KU; ++j) part[warp][j] = dot[j];
  __syncthreads();
  if (lt < KU && in && k0 + lt < K) {
    float s = 0.f;
    for (int q = 0; q < lpt / 32; ++q) s += part[warp + q][lt];
    dw[t * K + k0 + lt] = s;
  }
  __syncthreads();
}

// Row (-1: nothing to write), whether the pair counts, and its weight.
struct Pair {
  int row;
  bool use;
  float w;
};
__device__ __forceinline__ Pair load_pair(const int32_t* __restrict__ pair_pos, const float* __restrict__ w, int64_t p,
                                          bool have, int64_t P, bool report, int32_t* d_status) {
  const int q = have ? __ldg(pair_pos + p) : 0;
  const int r = q < 0 ? ~q : q;
  const bool ok = have && r < P;
  if (have && !ok && report) set_status(d_status, MLR_STATUS_INDEX);
  Pair o;
  o.row = ok ? r : -1;
  o.use = ok && q >= 0;
  o.w = o.use ? __ldg(w + p) : 0.f;
  return o;
}

template <typename E_, int KU, RowAccess A>
__global__ void __launch_bounds__(kBackThreads, 3)
unpermute_backward_kernel(const E_* __restrict__ dy, const E_* __restrict__ rows, const int32_t* __restrict__ pair_pos,
                          const float* __restrict__ w, int T, int K, int H, int lpt_log2, E_* __restrict__ d_rows,
                          float* __restrict__ dw, int32_t* d_status) {
  constexpr int N = 16 / (int)sizeof(E_), U = KU == 1 ? 4 : KU == 2 ? 2 : 1;
  __shared__ float part[kBackThreads / 32][KU];
  pdl_wait();
  pdl_trigger();
  const int lpt = 1 << lpt_log2, lt = threadIdx.x & (lpt - 1);
  const int64_t t = ((int64_t)blockIdx.x << (8 - lpt_log2)) + (threadIdx.x >> lpt_log2);
  const bool in = t < T;  // every thread stays for the exchanges
  for (int k0 = 0; k0 < K; k0 += KU) {
    Pair pr[KU];
    float dot[KU];
#pragma unroll
    for (int j = 0; j < KU; ++j) {
      pr[j] = load_pair(pair_pos, w, t * K + k0 + j, in && k0 + j < K, (int64_t)T * K, lt == 0, d_status);
      dot[j] = 0.f;
    }
    if (in)
      for (int c = A == kStrided ? lt : lt * N; c < H; c += U * lpt * N) {
        uint4 gv[U], v[KU][U];
#pragma unroll
        for (int i = 0; i < U; ++i) {
          const int ci = c + i * lpt * N;
          if constexpr (A == kStrided) gv[i] = load_strided(dy + t * H, ci, lpt, H);
          else gv[i] = ci < H ? __ldg(reinterpret_cast<const uint4*>(dy + t * H + ci)) : make_uint4(0, 0, 0, 0);
        }
#pragma unroll
        for (int j = 0; j < KU; ++j)
#pragma unroll
          for (int i = 0; i < U; ++i) {
            const int ci = c + i * lpt * N;
            if constexpr (A == kStrided)
              v[j][i] = load_strided(rows + (int64_t)pr[j].row * H, ci, lpt, pr[j].use ? H : 0);
            else
              v[j][i] = pr[j].use && ci < H ? __ldg(reinterpret_cast<const uint4*>(rows + (int64_t)pr[j].row * H + ci))
                                            : make_uint4(0, 0, 0, 0);
          }
#pragma unroll
        for (int i = 0; i < U; ++i) {
          const int ci = c + i * lpt * N;
          float g[N];
          widen(gv[i], g);
#pragma unroll
          for (int j = 0; j < KU; ++j) {
            float f[N], o[N];
            widen(v[j][i], f);
#pragma unroll
            for (int u = 0; u < N; ++u) {
              o[u] = pr[j].use ? pr[j].w * g[u] : 0.f;
              dot[j] = pr[j].use ? fmaf(g[u], f[u], dot[j]) : 0.f;
            }
            uint4 ov;
            narrow(o, ov);
            if constexpr (A == kStrided) {
              store_strided(d_rows + (int64_t)pr[j].row * H, ci, lpt, pr[j].row >= 0 ? H : 0, ov);
            } else {
              if (pr[j].row >= 0 && ci < H) *reinterpret_cast<uint4*>(d_rows + (int64_t)pr[j].row * H + ci) = ov;
            }
          }
        }
      }
    store_dots<KU>(dot, part, lpt, lt, in, t, K, k0, dw);
  }
}

// The same for bf16 rows off the 16-byte grid: each row of d_rows is written in its
// own aligned 16-byte pieces, with the row of rows (in the same pieces, unless
// the two bases differ) and the token's dy from shared memory at the piece's
// columns; the ends that share 16 bytes with another row go element by element.
// One block per token, 64 threads or for rows of up to 1 KB a warp (8192 x 6 rows
// of 1111 bf16: 62 us, with 128 threads 68, element by element 144; 10000 x 6 of
// 461: 40, with 64 threads 42).
constexpr int kBackSegBytes = 4096;
template <int KU, int LANES>
__global__ void __launch_bounds__(LANES)
unpermute_backward_unaligned_kernel(const uint16_t* __restrict__ dy, const uint16_t* __restrict__ rows,
                                    const int32_t* __restrict__ pair_pos, const float* __restrict__ w, int T, int K,
                                    int H, uint16_t* __restrict__ d_rows, float* __restrict__ dw, int32_t* d_status) {
  using E_ = uint16_t;
  constexpr int es = (int)sizeof(E_), N = 16 / es;
  __shared__ float part[LANES / 32][KU];
  __shared__ __align__(16) E_ seg[(kBackSegBytes + 32) / es];  // dy columns [b0, b0 + span)
  pdl_wait();
  pdl_trigger();
  const int lt = threadIdx.x;
  const int64_t t = blockIdx.x;
  constexpr int kSegCols = kBackSegBytes / es;
  const int rs = (int)((reinterpret_cast<uintptr_t>(rows) - reinterpret_cast<uintptr_t>(d_rows)) & 15);
  for (int k0 = 0; k0 < K; k0 += KU) {
    Pair pr[KU];
    float dot[KU];
    int off[KU];  // columns before the row's first aligned piece
#pragma unroll
    for (int j = 0; j < KU; ++j) {
      pr[j] = load_pair(pair_pos, w, t * K + k0 + j, k0 + j < K, (int64_t)T * K, lt == 0, d_status);
      off[j] = (int)(-reinterpret_cast<uintptr_t>(d_rows + (int64_t)max(pr[j].row, 0) * H) & 15) / es;
      dot[j] = 0.f;
    }
    for (int b0 = 0; b0 < H; b0 += kSegCols) {
      const int span = min(H - b0, kSegCols + N);
      __syncthreads();
      for (int i = lt; i < span; i += LANES) seg[i] = __ldg(dy + t * H + b0 + i);
      __syncthreads();
      for (int i = lt * N; i < min(H - b0, kSegCols); i += LANES * N) {
        uint4 v[KU];
        bool piece[KU];
#pragma unroll
        for (int j = 0; j < KU; ++j) {
          piece[j] = pr[j].row >= 0 && b0 + off[j] + i + N <= H;
          const char* r = reinterpret_cast<const char*>(rows + (int64_t)pr[j].row * H + b0 + off[j] + i);
          if (!(pr[j].use && piece[j])) v[j] = make_uint4(0, 0, 0, 0);
          else if (rs == 0) v[j] = __ldg(reinterpret_cast<const uint4*>(r));
          else v[j] = shifted<E_>(load_piece<E_>(r - rs, rows, rows + (int64_t)T * K * H),
                                  load_piece<E_>(r - rs + 16, rows, rows + (int64_t)T * K * H), rs);
        }
#pragma unroll
        for (int j = 0; j < KU; ++j) {
          if (!piece[j]) continue;
          float f[N], g[N], o[N];
          widen(v[j], f);
          const uint32_t* sw = reinterpret_cast<const uint32_t*>(seg) + (off[j] + i) * es / 4;
          uint4 q = make_uint4(sw[0], sw[1], sw[2], sw[3]);
          const uint32_t last = sw[4];  // dy's columns may begin inside a word
          const int m = 16 * (off[j] & 1);
          q.x = __funnelshift_r(q.x, q.y, m);
          q.y = __funnelshift_r(q.y, q.z, m);
          q.z = __funnelshift_r(q.z, q.w, m);
          q.w = __funnelshift_r(q.w, last, m);
          widen(q, g);
#pragma unroll
          for (int u = 0; u < N; ++u) {
            o[u] = pr[j].use ? pr[j].w * g[u] : 0.f;
            dot[j] = pr[j].use ? fmaf(g[u], f[u], dot[j]) : 0.f;
          }
          uint4 ov;
          narrow(o, ov);
          *reinterpret_cast<uint4*>(d_rows + (int64_t)pr[j].row * H + b0 + off[j] + i) = ov;
        }
      }
      // a row's columns before its first piece (threads 0 to N - 1) and after
      // its last one (threads N to 2N - 1), loaded together
      if (lt < 2 * N) {
        int c[KU];
        E_ e[KU];
#pragma unroll
        for (int j = 0; j < KU; ++j) {
          const int tail = H <= off[j] ? H : off[j] + (H - off[j]) / N * N;
          const bool have = lt < N ? b0 == 0 && lt < min(off[j], H)
                                   : tail >= b0 && tail < b0 + kSegCols && tail + lt - N < H;
          c[j] = have && pr[j].row >= 0 ? (lt < N ? lt : tail + lt - N) : -1;
          e[j] = c[j] >= 0 && pr[j].use ? __ldg(rows + (int64_t)pr[j].row * H + c[j]) : E_{};
        }
#pragma unroll
        for (int j = 0; j < KU; ++j) {
          if (c[j] < 0) continue;
          const float g = widen1(seg[c[j] - b0]);
          d_rows[(int64_t)pr[j].row * H + c[j]] = f32_to_bf16_bits(pr[j].use ? pr[j].w * g : 0.f);
          if (pr[j].use) dot[j] = fmaf(g, widen1(e[j]), dot[j]);
        }
      }
    }
    store_dots<KU>(dot, part, LANES, lt, true, t, K, k0, dw);
  }
}

// Opts a kernel in to the most dynamic shared memory that any call of it needs,
// not to what this one does: a call of fewer experts in another thread would
// lower the limit again before this one's launch.
template <typename Kernel>
cudaError_t allow_smem(Kernel kernel, size_t need, int most) {
  if (need <= 40 * 1024) return cudaSuccess;  // with the static part within the 48 KB that need no opt-in
  return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, most);
}
bool aligned_to(const void* p, int n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

template <int VB>
int launch_permute(const SortPlan& s, const void* x, const int32_t* ids, int T, int K, int E, int64_t row_bytes,
                   void* rows, int32_t* pair_pos, int32_t* offsets, char* ws, int32_t* d_status,
                   cudaStream_t stream) {
  // column slices: with few tokens each block copies a part of its rows (and
  // places its pairs again, which costs less than the copies would)
  int64_t slices = 1;
  if (row_bytes > 0) {
    const int64_t most = ceil_div(row_bytes, 2048);
    slices = s.G >= 304 ? 1 : ceil_div(304, s.G);
    if (slices > most) slices = most;
  }
  int32_t* cnt = reinterpret_cast<int32_t*>(ws);
  int32_t* tot = reinterpret_cast<int32_t*>(ws + s.o_tot);
  const dim3 grid((unsigned)s.G, (unsigned)slices);
  const size_t smem = (size_t)(E + 2) * 4 + (s.one ? (size_t)(E + 1) * 4 : 0);
  auto run = [&](auto kernel) {
    cudaError_t err = allow_smem(kernel, smem, (2 * kMaxSortExperts + 3) * 4);
    if (err == cudaSuccess)
      err = launch_pdl(kernel, grid, dim3(kSortThreads), smem, stream, x, ids, T, K, E, s.tpb, s.Gp, row_bytes, rows,
                       pair_pos, offsets, cnt, tot, d_status);
    return launched(err, 1);
  };
  return s.one ? run(permute_kernel<VB, true>) : run(permute_kernel<VB, false>);
}

int log2_of(int n) {
  int l = 0;
  while ((1 << l) < n) ++l;
  return l;
}

template <typename E_, int KU, RowAccess A>
int launch_unpermute_k(const void* rows, const int32_t* pos, const float* w, int T, int K, int H, void* y,
                       int32_t* d_status, cudaStream_t stream) {
  const int nv = (int)ceil_div((int64_t)H * sizeof(E_), 16 * kVecs<KU, A>), lpt = sum_threads(nv);
  const int64_t col_blocks = ceil_div(nv, lpt), blocks = ceil_div(T, kSumThreads / lpt) * col_blocks;
  if (blocks > INT32_MAX) return MLR_ERR_UNSUPPORTED;
  return launched(launch_pdl(unpermute_kernel<E_, KU, A>, dim3((unsigned)blocks), dim3(kSumThreads), 0, stream,
                             static_cast<const E_*>(rows), pos, w, T, K, H, log2_of(lpt), (unsigned)col_blocks,
                             static_cast<E_*>(y), d_status), 1);
}

// Rows in flight per thread: K in as few equal turns as there are of at most eight
// rows (four of rows off the grid, which take more registers or loads), as an
// empty place costs its instructions all the same (8479 x 5 rows of 2144 bf16:
// 42 us in eight places, 39 in six; 9836 x 5 rows of 1513: 54 and 46 in four and
// three; but on the grid three rows take 22.5 us in four places and 23.4 in three).
template <typename E_, typename... Args>
int launch_unpermute(bool whole, int K, Args... a) {
  constexpr RowAccess O = kOffGrid<E_>;
  const int most = whole ? 8 : 4;
  const int64_t ku = ceil_div(K, ceil_div(K, most));
  if (!whole)
    return ku == 1 ? launch_unpermute_k<E_, 1, O>(a...) : ku == 2 ? launch_unpermute_k<E_, 2, O>(a...)
           : ku == 3 ? launch_unpermute_k<E_, 3, O>(a...) : launch_unpermute_k<E_, 4, O>(a...);
  return ku == 1 ? launch_unpermute_k<E_, 1, kWhole>(a...) : ku == 2 ? launch_unpermute_k<E_, 2, kWhole>(a...)
         : ku <= 4 ? launch_unpermute_k<E_, 4, kWhole>(a...) : ku <= 6 ? launch_unpermute_k<E_, 6, kWhole>(a...)
                                                                       : launch_unpermute_k<E_, 8, kWhole>(a...);
}

template <typename E_, int KU, RowAccess A>
int launch_unpermute_backward_k(const void* dy, const void* rows, const int32_t* pos, const float* w, int T, int K,
                                int H, void* d_rows, float* dw, int32_t* d_status, cudaStream_t stream) {
  const E_ *dyp = static_cast<const E_*>(dy), *rp = static_cast<const E_*>(rows);
  E_* dp = static_cast<E_*>(d_rows);
  cudaError_t err;
  if constexpr (A != kPieces) {
    // strided rows take four times the loads: fewer threads per token leave more
    // tokens in flight (1531 x 6 rows of 1111 float32: 24 us, with 128 28 us)
    const int lpt = row_threads((int)ceil_div((int64_t)H * sizeof(E_), 16), A == kStrided ? kBackLanes / 2 : kBackLanes);
    err = launch_pdl(unpermute_backward_kernel<E_, KU, A>, dim3((unsigned)ceil_div(T, kBackThreads / lpt)),
                     dim3(kBackThreads), 0, stream, dyp, rp, pos, w, T, K, H, log2_of(lpt), dp, dw, d_status);
  } else {
    auto run = [&](auto kernel, int threads) {
      return launch_pdl(kernel, dim3((unsigned)T), dim3(threads), 0, stream, dyp, rp, pos, w, T, K, H, dp, dw, d_status);
    };
    err = H * (int)sizeof(E_) <= 1024 ? run(unpermute_backward_unaligned_kernel<KU, 32>, 32)
                                     : run(unpermute_backward_unaligned_kernel<KU, 64>, 64);
  }
  return launched(err, 1);
}
// Rows in flight as above, but on the grid always four places or eight (8479 x 5
// rows of 2144 bf16: 89 us in eight, 102 in six).
template <typename E_, typename... Args>
int launch_unpermute_backward(bool whole, int K, Args... a) {
  constexpr RowAccess O = kOffGrid<E_>;
  const int64_t ku = ceil_div(K, ceil_div(K, 4));
  if (!whole)
    return ku == 1 ? launch_unpermute_backward_k<E_, 1, O>(a...) : ku == 2 ? launch_unpermute_backward_k<E_, 2, O>(a...)
           : ku == 3 ? launch_unpermute_backward_k<E_, 3, O>(a...) : launch_unpermute_backward_k<E_, 4, O>(a...);
  return K == 1 ? launch_unpermute_backward_k<E_, 1, kWhole>(a...) : K == 2 ? launch_unpermute_backward_k<E_, 2, kWhole>(a...)
         : K <= 4 ? launch_unpermute_backward_k<E_, 4, kWhole>(a...) : launch_unpermute_backward_k<E_, 8, kWhole>(a...);
}

// Common checks of the row operators; the row size in *es.
int check_rows(int32_t T, int32_t K, int32_t H, int32_t dtype, int* es) {
  if (T < 0 || K < 1 || H < 1 || (dtype != MLR_DTYPE_BF16 && dtype != MLR_DTYPE_F32)) return MLR_ERR_INVALID;
  if ((int64_t)T * K >= INT32_MAX || H > kMaxHidden) return MLR_ERR_UNSUPPORTED;
  *es = dtype == MLR_DTYPE_BF16 ? 2 : 4;
  return MLR_OK;
}

}  // namespace
}  // namespace mlr

extern "C" size_t moe_permute_workspace_bytes(int32_t num_tokens, int32_t topk, int32_t num_experts) {
  const mlr::SortPlan s = mlr::sort_plan(num_tokens, topk, num_experts, mlr::kOneLaunchPairs);
  return s.ok ? (size_t)s.bytes : 0;
}

extern "C" size_t moe_sort_pairs_workspace_bytes(int32_t num_tokens, int32_t topk, int32_t num_experts) {
  const mlr::SortPlan s = mlr::sort_plan(num_tokens, topk, num_experts, mlr::kOneLaunchSorted);
  return s.ok ? (size_t)s.bytes : 0;
}

extern "C" int moe_permute(const void* x, const int32_t* topk_ids, int32_t num_tokens, int32_t topk, int32_t hidden,
                           int32_t num_experts, int32_t dtype, void* rows, int32_t* pair_pos, int32_t* expert_offsets,
                           void* workspace, size_t ws_bytes, int32_t* d_status, void* stream_) {
  using namespace mlr;
  cudaStream_t stream = static_cast<cudaStream_t>(stream_);
  const SortPlan s = sort_plan(num_tokens, topk, num_experts, x == nullptr ? kOneLaunchSorted : kOneLaunchPairs);
  if (!s.ok) return s.code;
  if ((x == nullptr) != (rows == nullptr) || expert_offsets == nullptr) return MLR_ERR_INVALID;
  int es = 0;
  if (x != nullptr) {
    const int code = check_rows(num_tokens, topk, hidden, dtype, &es);
    if (code != MLR_OK) return code;
    if (!aligned_to(x, es) || !aligned_to(rows, es)) return MLR_ERR_INVALID;
  }
  if (s.P == 0)
    return launched(cudaMemsetAsync(expert_offsets, 0, (size_t)(num_experts + 1) * 4, stream), 0);
  if (topk_ids == nullptr || pair_pos == nullptr) return MLR_ERR_INVALID;
  if (!(s.one && workspace == nullptr) && (workspace == nullptr || ws_bytes < (size_t)s.bytes)) return MLR_ERR_CAPACITY;
  if (!aligned_to(workspace, 256)) return MLR_ERR_INVALID;
  char* ws = static_cast<char*>(workspace);
  if (!s.one) {
    int32_t* cnt = reinterpret_cast<int32_t*>(ws);
    int32_t* tot = reinterpret_cast<int32_t*>(ws + s.o_tot);
    const size_t one = (size_t)(num_experts + 1) * 4;
    const bool wide = one * kCountChunks <= 48 * 1024;
    const unsigned blocks = (unsigned)(s.Gp / kCountChunks);
    cudaError_t err = wide ? cudaSuccess : allow_smem(sort_count_kernel<false>, one, (kMaxSortExperts + 1) * 4);
    if (err == cudaSuccess)
      err = wide ? launch_pdl(sort_count_kernel<true>, dim3(blocks), dim3(kSortThreads), one * kCountChunks, stream,
                              topk_ids, s.P, num_experts, s.tpb * topk, s.Gp, cnt)
                 : launch_pdl(sort_count_kernel<false>, dim3(blocks), dim3(kSortThreads), one, stream, topk_ids, s.P,
                              num_experts, s.tpb * topk, s.Gp, cnt);
    int code = launched(err, 1);
    if (code != MLR_OK) return code;
    code = launched(launch_pdl(sort_scan_kernel, dim3((unsigned)(num_experts + 1)), dim3(kSortThreads), 0, stream, cnt,
                               s.Gp, tot), 1);
    if (code != MLR_OK) return code;
  }
  const int64_t rb = x == nullptr ? 0 : (int64_t)hidden * es;
  const bool whole = rb % 16 == 0 && aligned_to(x, 16) && aligned_to(rows, 16);
  if (whole && rb >= 8192)
    return launch_permute<32>(s, x, topk_ids, num_tokens, topk, num_experts, rb, rows, pair_pos, expert_offsets, ws,
                              d_status, stream);
  if (whole)
    return launch_permute<16>(s, x, topk_ids, num_tokens, topk, num_experts, rb, rows, pair_pos, expert_offsets, ws,
                              d_status, stream);
  if (es == 4)
    return launch_permute<4>(s, x, topk_ids, num_tokens, topk, num_experts, rb, rows, pair_pos, expert_offsets, ws,
                             d_status, stream);
  return launch_permute<2>(s, x, topk_ids, num_tokens, topk, num_experts, rb, rows, pair_pos, expert_offsets, ws,
                           d_status, stream);
}

extern "C" int moe_unpermute(const void* rows, const int32_t* pair_pos, const float* topk_weights, int32_t num_tokens,
                             int32_t topk, int32_t hidden, int32_t dtype, void* y, int32_t* d_status, void* stream_) {
  using namespace mlr;
  cudaStream_t stream = static_cast<cudaStream_t>(stream_);
  int es = 0;
  const int code = check_rows(num_tokens, topk, hidden, dtype, &es);
  if (code != MLR_OK) return code;
  if (num_tokens == 0) return MLR_OK;
  if (rows == nullptr || pair_pos == nullptr || y == nullptr || !aligned_to(rows, es) || !aligned_to(y, es))
    return MLR_ERR_INVALID;
  const bool al = (int64_t)hidden * es % 16 == 0 && aligned_to(rows, 16) && aligned_to(y, 16);
  const int T = num_tokens, K = topk, H = hidden;
  return dtype == MLR_DTYPE_F32 ? launch_unpermute<float>(al, K, rows, pair_pos, topk_weights, T, K, H, y, d_status, stream)
                                : launch_unpermute<uint16_t>(al, K, rows, pair_pos, topk_weights, T, K, H, y, d_status, stream);
}

extern "C" int moe_unpermute_backward(const void* dy, const void* rows, const int32_t* pair_pos,
                                      const float* topk_weights, int32_t num_tokens, int32_t topk, int32_t hidden,
                                      int32_t dtype, void* d_rows, float* d_weights, int32_t* d_status,
                                      void* stream_) {
  using namespace mlr;
  cudaStream_t stream = static_cast<cudaStream_t>(stream_);
  int es = 0;
  const int code = check_rows(num_tokens, topk, hidden, dtype, &es);
  if (code != MLR_OK) return code;
  if (num_tokens == 0) return MLR_OK;
  for (const void* p : {dy, rows, static_cast<const void*>(d_rows)})
    if (p == nullptr || !aligned_to(p, es)) return MLR_ERR_INVALID;
  if (pair_pos == nullptr || topk_weights == nullptr || d_weights == nullptr) return MLR_ERR_INVALID;
  const bool al = (int64_t)hidden * es % 16 == 0 && aligned_to(dy, 16) && aligned_to(rows, 16) && aligned_to(d_rows, 16);
  const int T = num_tokens, K = topk, H = hidden;
  return dtype == MLR_DTYPE_F32
             ? launch_unpermute_backward<float>(al, K, dy, rows, pair_pos, topk_weights, T, K, H, d_rows, d_weights, d_status, stream)
             : launch_unpermute_backward<uint16_t>(al, K, dy, rows, pair_pos, topk_weights, T, K, H, d_rows, d_weights, d_status, stream);
}
