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
// All four move rows once: they are bound by HBM (bytes = rows read + rows
// written), the sort by launch latency.
#include "mlr_profile.cuh"

namespace mlr {
namespace {

constexpr int kSortThreads = 256;
constexpr int kChunkPairs = 256;     // pairs of one block, ranked by comparison in shared memory
constexpr int kMaxSortTopk = 256;    // one token's pairs fit a chunk
constexpr int kMaxSortExperts = 16384;
// Up to this many pairs every block counts all of them itself, which saves the
// two launches that count and scan them for larger batches.
constexpr int64_t kOneLaunchPairs = 8192;

struct SortPlan {
  bool ok;
  int code;
  int64_t P;
  int tpb;        // tokens per block
  int64_t G;      // blocks (chunks)
  bool one;       // a single launch
  int64_t o_tot;  // workspace: counts [E+1][G], then totals [E+1]
  int64_t bytes;
};

SortPlan sort_plan(int32_t T, int32_t K, int32_t E) {
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
  s.one = s.P <= kOneLaunchPairs;
  const int64_t want = ceil_div(T, s.one ? 512 : 1024);
  const int most = kChunkPairs / K;
  s.tpb = (int)(want < 1 ? 1 : want > most ? most : want);
  s.G = ceil_div(T, s.tpb);
  s.o_tot = round_up((int64_t)(E + 1) * s.G * 4, 256);
  s.bytes = s.one ? 256 : s.o_tot + round_up((int64_t)(E + 1) * 4, 256);
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

// Counts of one chunk's pairs per expert (masked pairs as expert E):
// cnt[e][g].
__global__ void __launch_bounds__(kSortThreads)
sort_count_kernel(const int32_t* __restrict__ ids, int64_t P, int E, int chunk, int64_t G, int32_t* __restrict__ cnt) {
  extern __shared__ int hist[];  // [E + 1]
  for (int e = threadIdx.x; e <= E; e += kSortThreads) hist[e] = 0;
  pdl_wait();
  pdl_trigger();
  __syncthreads();
  const int64_t p = (int64_t)blockIdx.x * chunk + threadIdx.x;
  if ((int)threadIdx.x < chunk && p < P) atomicAdd(&hist[sort_key(__ldg(ids + p), E)], 1);
  __syncthreads();
  for (int e = threadIdx.x; e <= E; e += kSortThreads) cnt[(int64_t)e * G + blockIdx.x] = hist[e];
}

// One block per expert: the exclusive scan of its chunk counts, in place, and
// its total.
__global__ void __launch_bounds__(kSortThreads)
sort_scan_kernel(int32_t* __restrict__ cnt, int64_t G, int32_t* __restrict__ tot) {
  __shared__ int warp_tot[kSortThreads / 32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int32_t* c = cnt + (int64_t)blockIdx.x * G;
  pdl_wait();
  pdl_trigger();
  int carry = 0;
  for (int64_t g0 = 0; g0 < G; g0 += kSortThreads) {
    const int64_t g = g0 + threadIdx.x;
    const int v = g < G ? c[g] : 0;
    int inc = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int u = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += u;
    }
    if (lane == 31) warp_tot[warp] = inc;
    __syncthreads();
    int before = carry, all = 0;
    for (int w = 0; w < kSortThreads / 32; ++w) {
      if (w < warp) before += warp_tot[w];
      all += warp_tot[w];
    }
    if (g < G) c[g] = before + inc - v;
    carry += all;
    __syncthreads();
  }
  if (threadIdx.x == 0) tot[blockIdx.x] = carry;
}

// Places the pairs of one chunk of tokens and copies this block's column slice
// of their rows.  The rank of a pair inside the chunk is the number of earlier
// chunk pairs with the same key, counted by comparison.  VB: bytes per copied
// vector (the largest of 16, 4, 2 that divides a row and both bases).
template <int VB> struct CopyVec;
template <> struct CopyVec<16> { using type = uint4; };
template <> struct CopyVec<4> { using type = uint32_t; };
template <> struct CopyVec<2> { using type = uint16_t; };

template <int VB, bool ONE>
__global__ void __launch_bounds__(kSortThreads)
permute_kernel(const void* __restrict__ x, const int32_t* __restrict__ ids, int T, int K, int E, int tpb, int64_t G,
               int64_t nvec /* vectors per row, 0: sort only */, void* __restrict__ rows,
               int32_t* __restrict__ pair_pos, int32_t* __restrict__ offsets, const int32_t* __restrict__ cnt,
               const int32_t* __restrict__ tot, int32_t* d_status) {
  using V = typename CopyVec<VB>::type;
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
    r += start[mine] + (ONE ? before[mine] : __ldg(cnt + (int64_t)mine * G + blockIdx.x));
    const int at = mine == E ? ~r : r;
    place[tid] = at;
    if (blockIdx.y == 0) pair_pos[p0 + tid] = at;
  }
  if (blockIdx.x == 0 && blockIdx.y == 0)
    for (int e = tid; e <= E; e += kSortThreads) offsets[e] = start[e];
  if (nvec == 0) return;
  __syncthreads();
  // one warp per token and pass: each vector of its row is read once and
  // written to its K rows
  const V* xv = static_cast<const V*>(x);
  V* rv = static_cast<V*>(rows);
  const int lane = tid & 31, warp = tid >> 5;
  const int64_t step = (int64_t)gridDim.y * 32;
  for (int i = warp; i < nt; i += kSortThreads / 32) {
    const V* src = xv + (t0 + i) * nvec;
    const int* pl = place + i * K;
    for (int64_t c = (int64_t)blockIdx.y * 32 + lane; c < nvec; c += 4 * step) {
      V v[4];
#pragma unroll
      for (int u = 0; u < 4; ++u)
        if (c + u * step < nvec) v[u] = __ldg(src + c + u * step);
      for (int k = 0; k < K; ++k) {
        const int at = pl[k];
        V* dst = rv + (int64_t)(at < 0 ? ~at : at) * nvec;
#pragma unroll
        for (int u = 0; u < 4; ++u)
          if (c + u * step < nvec) dst[c + u * step] = at < 0 ? V{} : v[u];
      }
    }
  }
}

// ------------------------------------------------------------ row vectors --
// N consecutive elements of a row: the raw load and its fp32 values.
template <typename E_, int N> struct Vec;
template <> struct Vec<float, 4> { using type = float4; };
template <> struct Vec<float, 1> { using type = float; };
template <> struct Vec<uint16_t, 8> { using type = uint4; };
template <> struct Vec<uint16_t, 2> { using type = uint32_t; };
template <> struct Vec<uint16_t, 1> { using type = uint16_t; };

__device__ __forceinline__ void widen(const float4& q, float (&v)[4]) {
  v[0] = q.x;
  v[1] = q.y;
  v[2] = q.z;
  v[3] = q.w;
}
__device__ __forceinline__ void widen(const float& q, float (&v)[1]) { v[0] = q; }
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
__device__ __forceinline__ void widen(const uint32_t& q, float (&v)[2]) { widen2(q, v[0], v[1]); }
__device__ __forceinline__ void widen(const uint16_t& q, float (&v)[1]) { v[0] = __uint_as_float((uint32_t)q << 16); }

__device__ __forceinline__ uint32_t narrow2(float a, float b) {
  uint32_t o;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(o) : "f"(b), "f"(a));
  return o;
}
__device__ __forceinline__ void narrow(const float (&v)[4], float4& q) { q = make_float4(v[0], v[1], v[2], v[3]); }
__device__ __forceinline__ void narrow(const float (&v)[1], float& q) { q = v[0]; }
__device__ __forceinline__ void narrow(const float (&v)[8], uint4& q) {
  q = make_uint4(narrow2(v[0], v[1]), narrow2(v[2], v[3]), narrow2(v[4], v[5]), narrow2(v[6], v[7]));
}
__device__ __forceinline__ void narrow(const float (&v)[2], uint32_t& q) { q = narrow2(v[0], v[1]); }
__device__ __forceinline__ void narrow(const float (&v)[1], uint16_t& q) { q = f32_to_bf16_bits(v[0]); }

// The threads of a token: a power of two, so that short rows share a block.
int row_threads(int nv, int most) {
  int l = 8;
  while (l < nv && l < most) l *= 2;
  return l;
}

// y[t] = sum_k w[t, k] rows[pos]; w == nullptr: w = 1 (the gradient of permute).
// One thread per vector of a token; KU rows are loaded before any is added,
// without branches, so that their loads are in flight together.
constexpr int kSumThreads = 128;
template <typename E_, int N, int KU>
__global__ void __launch_bounds__(kSumThreads)
unpermute_kernel(const E_* __restrict__ rows, const int32_t* __restrict__ pair_pos, const float* __restrict__ w, int T,
                 int K, int H, int nv, int lpt_log2, unsigned col_blocks, E_* __restrict__ y, int32_t* d_status) {
  using V = typename Vec<E_, N>::type;
  pdl_wait();
  pdl_trigger();
  const unsigned tb = blockIdx.x / col_blocks, cb = blockIdx.x - tb * col_blocks;
  const int64_t t = ((int64_t)tb << (7 - lpt_log2)) + (threadIdx.x >> lpt_log2);
  const int c = (int)(cb << lpt_log2) + (threadIdx.x & ((1 << lpt_log2) - 1));
  if (t >= T || c >= nv) return;
  const int64_t P = (int64_t)T * K;
  float acc[N];
#pragma unroll
  for (int j = 0; j < N; ++j) acc[j] = 0.f;
  for (int k0 = 0; k0 < K; k0 += KU) {
    V v[KU];
    float wk[KU];
#pragma unroll
    for (int j = 0; j < KU; ++j) {
      const int64_t p = t * K + k0 + j;
      const int q = k0 + j < K ? __ldg(pair_pos + p) : -1;
      const bool use = q >= 0 && q < P;
      if (q >= P) set_status(d_status, MLR_STATUS_INDEX);
      wk[j] = !use ? 0.f : w != nullptr ? __ldg(w + p) : 1.f;
      v[j] = use ? __ldg(reinterpret_cast<const V*>(rows + (int64_t)q * H) + c) : V{};
    }
#pragma unroll
    for (int j = 0; j < KU; ++j) {
      float f[N];
      widen(v[j], f);
#pragma unroll
      for (int u = 0; u < N; ++u) acc[u] = fmaf(wk[j], f[u], acc[u]);
    }
  }
  V o;
  narrow(acc, o);
  reinterpret_cast<V*>(y + t * H)[c] = o;
}

// The row gradients of a token's pairs and the dot products that are its
// weights' gradients, by 2^lpt_log2 threads per token (per thread over its
// columns in increasing order, then over lanes and warps in a fixed order).
// Bound by the bytes in flight: eight rows of a token are loaded at once, at
// most 85 registers a thread for three blocks per SM.  8192 x 8 rows of 7168
// bf16: 293 us at 85 registers, 530 at 110, 324 at 64 (spills); with 128
// threads per token instead of 256, 4096 x 8 rows of 2048 take 48 instead of 53.
constexpr int kBackThreads = 256, kBackLanes = 128;
template <typename E_, int N, int KU>
__global__ void __launch_bounds__(kBackThreads, 3)
unpermute_backward_kernel(const E_* __restrict__ dy, const E_* __restrict__ rows, const int32_t* __restrict__ pair_pos,
                          const float* __restrict__ w, int T, int K, int H, int nv, int lpt_log2,
                          E_* __restrict__ d_rows, float* __restrict__ dw, int32_t* d_status) {
  using V = typename Vec<E_, N>::type;
  __shared__ float part[kBackThreads / 32][KU];
  pdl_wait();
  pdl_trigger();
  const int lpt = 1 << lpt_log2, lt = threadIdx.x & (lpt - 1);
  const int64_t t = ((int64_t)blockIdx.x << (8 - lpt_log2)) + (threadIdx.x >> lpt_log2);
  const int64_t P = (int64_t)T * K;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const bool in = t < T;  // every thread stays for the exchanges
  for (int k0 = 0; k0 < K; k0 += KU) {
    int row[KU];  // -1: nothing to write
    bool use[KU];
    float wk[KU], dot[KU];
#pragma unroll
    for (int j = 0; j < KU; ++j) {
      const bool have = in && k0 + j < K;
      const int q = have ? __ldg(pair_pos + t * K + k0 + j) : 0;
      const int r = q < 0 ? ~q : q;
      const bool ok = have && r < P;
      if (have && !ok && lt == 0) set_status(d_status, MLR_STATUS_INDEX);
      row[j] = ok ? r : -1;
      use[j] = ok && q >= 0;
      wk[j] = use[j] ? __ldg(w + t * K + k0 + j) : 0.f;
      dot[j] = 0.f;
    }
    if (in)
      for (int c = lt; c < nv; c += lpt) {
        float g[N];
        V v[KU];
        const V gv = __ldg(reinterpret_cast<const V*>(dy + t * H) + c);
#pragma unroll
        for (int j = 0; j < KU; ++j)
          v[j] = use[j] ? __ldg(reinterpret_cast<const V*>(rows + (int64_t)row[j] * H) + c) : V{};
        widen(gv, g);
#pragma unroll
        for (int j = 0; j < KU; ++j) {
          float f[N], o[N];
          widen(v[j], f);
#pragma unroll
          for (int u = 0; u < N; ++u) {
            o[u] = use[j] ? wk[j] * g[u] : 0.f;
            dot[j] = use[j] ? fmaf(g[u], f[u], dot[j]) : 0.f;
          }
          V ov;
          narrow(o, ov);
          if (row[j] >= 0) reinterpret_cast<V*>(d_rows + (int64_t)row[j] * H)[c] = ov;
        }
      }
#pragma unroll
    for (int j = 0; j < KU; ++j)
      for (int o = min(lpt, 32) >> 1; o > 0; o >>= 1) dot[j] += __shfl_xor_sync(0xffffffffu, dot[j], o);
    if (lpt <= 32) {
      if (lt == 0 && in)
#pragma unroll
        for (int j = 0; j < KU; ++j)
          if (k0 + j < K) dw[t * K + k0 + j] = dot[j];
    } else {
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
  }
}

bool aligned_to(const void* p, int n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

template <int VB>
int launch_permute(const SortPlan& s, const void* x, const int32_t* ids, int T, int K, int E, int64_t row_bytes,
                   void* rows, int32_t* pair_pos, int32_t* offsets, char* ws, int32_t* d_status,
                   cudaStream_t stream) {
  const int64_t nvec = row_bytes / VB;
  // column slices: with few tokens each block copies a part of its rows (and
  // places its pairs again, which costs less than the copies would)
  int64_t slices = 1;
  if (nvec > 0) {
    const int64_t most = ceil_div(nvec, 128);
    slices = s.G >= 304 ? 1 : ceil_div(304, s.G);
    if (slices > most) slices = most;
  }
  int32_t* cnt = reinterpret_cast<int32_t*>(ws);
  int32_t* tot = reinterpret_cast<int32_t*>(ws + s.o_tot);
  const dim3 grid((unsigned)s.G, (unsigned)slices);
  const size_t smem = (size_t)(E + 2) * 4 + (s.one ? (size_t)(E + 1) * 4 : 0);
  auto run = [&](auto kernel) {
    if (smem > 40 * 1024 &&
        cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem) != cudaSuccess)
      return MLR_ERR_CUDA;
    if (launch_pdl(kernel, grid, dim3(kSortThreads), smem, stream, x, ids, T, K, E, s.tpb, s.G, nvec, rows, pair_pos,
                   offsets, cnt, tot, d_status) != cudaSuccess)
      return MLR_ERR_CUDA;
    note_launch();
    return MLR_OK;
  };
  return s.one ? run(permute_kernel<VB, true>) : run(permute_kernel<VB, false>);
}

int log2_of(int n) {
  int l = 0;
  while ((1 << l) < n) ++l;
  return l;
}

template <typename E_, int N, int KU>
int launch_unpermute_k(const void* rows, const int32_t* pos, const float* w, int T, int K, int H, void* y,
                       int32_t* d_status, cudaStream_t stream) {
  const int nv = H / N, lpt = row_threads(nv, kSumThreads);
  const int64_t col_blocks = ceil_div(nv, lpt), blocks = ceil_div(T, kSumThreads / lpt) * col_blocks;
  if (blocks > INT32_MAX) return MLR_ERR_UNSUPPORTED;
  if (launch_pdl(unpermute_kernel<E_, N, KU>, dim3((unsigned)blocks), dim3(kSumThreads), 0, stream,
                 static_cast<const E_*>(rows), pos, w, T, K, H, nv, log2_of(lpt), (unsigned)col_blocks,
                 static_cast<E_*>(y), d_status) != cudaSuccess)
    return MLR_ERR_CUDA;
  note_launch();
  return MLR_OK;
}

// Rows in flight per thread: the smallest of 1, 2, 4, 8 that holds K, so that
// few experts per token cost no empty turns.
template <typename E_, int N, typename... A>
int launch_unpermute(int K, A... a) {
  return K == 1 ? launch_unpermute_k<E_, N, 1>(a...) : K == 2 ? launch_unpermute_k<E_, N, 2>(a...)
         : K <= 4 ? launch_unpermute_k<E_, N, 4>(a...) : launch_unpermute_k<E_, N, 8>(a...);
}

template <typename E_, int N, int KU>
int launch_unpermute_backward_k(const void* dy, const void* rows, const int32_t* pos, const float* w, int T, int K,
                                int H, void* d_rows, float* dw, int32_t* d_status, cudaStream_t stream) {
  const int nv = H / N, lpt = row_threads(nv, kBackLanes);
  if (launch_pdl(unpermute_backward_kernel<E_, N, KU>, dim3((unsigned)ceil_div(T, kBackThreads / lpt)),
                 dim3(kBackThreads), 0, stream, static_cast<const E_*>(dy), static_cast<const E_*>(rows), pos, w, T, K,
                 H, nv, log2_of(lpt), static_cast<E_*>(d_rows), dw, d_status) != cudaSuccess)
    return MLR_ERR_CUDA;
  note_launch();
  return MLR_OK;
}
template <typename E_, int N, typename... A>
int launch_unpermute_backward(int K, A... a) {
  return K == 1 ? launch_unpermute_backward_k<E_, N, 1>(a...) : K == 2 ? launch_unpermute_backward_k<E_, N, 2>(a...)
         : K <= 4 ? launch_unpermute_backward_k<E_, N, 4>(a...) : launch_unpermute_backward_k<E_, N, 8>(a...);
}

// Common checks of the row operators; the row size in *es.
int check_rows(int32_t T, int32_t K, int32_t H, int32_t dtype, int* es) {
  if (T < 0 || K < 1 || H < 1 || (dtype != MLR_DTYPE_BF16 && dtype != MLR_DTYPE_F32)) return MLR_ERR_INVALID;
  if ((int64_t)T * K >= INT32_MAX) return MLR_ERR_UNSUPPORTED;
  *es = dtype == MLR_DTYPE_BF16 ? 2 : 4;
  return MLR_OK;
}

}  // namespace
}  // namespace mlr

extern "C" size_t moe_permute_workspace_bytes(int32_t num_tokens, int32_t topk, int32_t num_experts) {
  const mlr::SortPlan s = mlr::sort_plan(num_tokens, topk, num_experts);
  return s.ok ? (size_t)s.bytes : 0;
}

extern "C" int moe_permute(const void* x, const int32_t* topk_ids, int32_t num_tokens, int32_t topk, int32_t hidden,
                           int32_t num_experts, int32_t dtype, void* rows, int32_t* pair_pos, int32_t* expert_offsets,
                           void* workspace, size_t ws_bytes, int32_t* d_status, void* stream_) {
  using namespace mlr;
  cudaStream_t stream = static_cast<cudaStream_t>(stream_);
  const SortPlan s = sort_plan(num_tokens, topk, num_experts);
  if (!s.ok) return s.code;
  if ((x == nullptr) != (rows == nullptr) || expert_offsets == nullptr) return MLR_ERR_INVALID;
  int es = 0;
  if (x != nullptr) {
    const int code = check_rows(num_tokens, topk, hidden, dtype, &es);
    if (code != MLR_OK) return code;
    if (!aligned_to(x, es) || !aligned_to(rows, es)) return MLR_ERR_INVALID;
  }
  if (s.P == 0)
    return cudaMemsetAsync(expert_offsets, 0, (size_t)(num_experts + 1) * 4, stream) == cudaSuccess ? MLR_OK
                                                                                                     : MLR_ERR_CUDA;
  if (topk_ids == nullptr || pair_pos == nullptr) return MLR_ERR_INVALID;
  if (workspace == nullptr || ws_bytes < (size_t)s.bytes) return MLR_ERR_CAPACITY;
  if (!aligned_to(workspace, 256)) return MLR_ERR_INVALID;
  char* ws = static_cast<char*>(workspace);
  if (!s.one) {
    int32_t* cnt = reinterpret_cast<int32_t*>(ws);
    int32_t* tot = reinterpret_cast<int32_t*>(ws + s.o_tot);
    const size_t smem = (size_t)(num_experts + 1) * 4;
    if (smem > 40 * 1024 && cudaFuncSetAttribute(sort_count_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                 (int)smem) != cudaSuccess)
      return MLR_ERR_CUDA;
    if (launch_pdl(sort_count_kernel, dim3((unsigned)s.G), dim3(kSortThreads), smem, stream, topk_ids, s.P,
                   num_experts, s.tpb * topk, s.G, cnt) != cudaSuccess)
      return MLR_ERR_CUDA;
    if (launch_pdl(sort_scan_kernel, dim3((unsigned)(num_experts + 1)), dim3(kSortThreads), 0, stream, cnt, s.G,
                   tot) != cudaSuccess)
      return MLR_ERR_CUDA;
    note_launch(2);
  }
  const int64_t rb = x == nullptr ? 0 : (int64_t)hidden * es;
  auto fits = [&](int n) { return rb % n == 0 && aligned_to(x, n) && aligned_to(rows, n); };
  if (fits(16))
    return launch_permute<16>(s, x, topk_ids, num_tokens, topk, num_experts, rb, rows, pair_pos, expert_offsets, ws,
                              d_status, stream);
  if (fits(4))
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
  auto fits = [&](int n) { return (int64_t)hidden * es % n == 0 && aligned_to(rows, n) && aligned_to(y, n); };
  const int T = num_tokens, K = topk, H = hidden;
  if (dtype == MLR_DTYPE_F32)
    return fits(16) ? launch_unpermute<float, 4>(K, rows, pair_pos, topk_weights, T, K, H, y, d_status, stream)
                    : launch_unpermute<float, 1>(K, rows, pair_pos, topk_weights, T, K, H, y, d_status, stream);
  return fits(16)  ? launch_unpermute<uint16_t, 8>(K, rows, pair_pos, topk_weights, T, K, H, y, d_status, stream)
         : fits(4) ? launch_unpermute<uint16_t, 2>(K, rows, pair_pos, topk_weights, T, K, H, y, d_status, stream)
                   : launch_unpermute<uint16_t, 1>(K, rows, pair_pos, topk_weights, T, K, H, y, d_status, stream);
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
  auto fits = [&](int n) {
    return (int64_t)hidden * es % n == 0 && aligned_to(dy, n) && aligned_to(rows, n) && aligned_to(d_rows, n);
  };
  const int T = num_tokens, K = topk, H = hidden;
  if (dtype == MLR_DTYPE_F32)
    return fits(16) ? launch_unpermute_backward<float, 4>(K, dy, rows, pair_pos, topk_weights, T, K, H, d_rows, d_weights, d_status, stream)
                    : launch_unpermute_backward<float, 1>(K, dy, rows, pair_pos, topk_weights, T, K, H, d_rows, d_weights, d_status, stream);
  return fits(16)  ? launch_unpermute_backward<uint16_t, 8>(K, dy, rows, pair_pos, topk_weights, T, K, H, d_rows, d_weights, d_status, stream)
         : fits(4) ? launch_unpermute_backward<uint16_t, 2>(K, dy, rows, pair_pos, topk_weights, T, K, H, d_rows, d_weights, d_status, stream)
                   : launch_unpermute_backward<uint16_t, 1>(K, dy, rows, pair_pos, topk_weights, T, K, H, d_rows, d_weights, d_status, stream);
}
