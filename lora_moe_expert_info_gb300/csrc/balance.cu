// balance.cu -- the balance loss over a batch with the tokens per expert, and the
// gradient of the router's logits.
//
// With s = softmax(logits) or sigmoid(logits) (a logit that is not finite counts as
// -inf), p = s [/ its sum over e (sigmoid)], N unmasked tokens and c_e pairs of
// expert e:
//   loss = E / (K N^2) sum_e c_e sum_t p_te
// Gradients, with a_e = dloss E / (K N^2) c_e and g_k what reaches weight k:
//   softmax  dl_e = p_e (a_e - sum_j p_j a_j)           + g's part
//   sigmoid  dl_e = p_e (1 - s_e) (a_e - sum_j p_j a_j) + g's part
// where g's part is, for a chosen expert with weight w = scale s / total,
//   w (g - sum g w / scale) [(1 - s) for sigmoid]       renormalised
//   scale g s (1 - s)                                   sigmoid
//   p (scale g - sum scale g p), of all experts         softmax
//
// Both are bound by HBM: logits are read once a pass, a turn ahead of their use, and a
// token's stay in the registers of its lanes.  262144 x 256 float32, padded, sigmoid: loss
// 49 us (83% of the copy rate), gradient 84 (94%).  4096 x 128: 11 and 3 us.  Rows off the
// 16-byte grid are not fetched ahead and few experts leave lanes idle: turns then follow one
// another at HBM's latency (262144 x 61: 29 and 33 us, 36 and 56%; 262144 x 8: 23 and 22, 7 and 11%).
#include <cooperative_groups.h>
#include <float.h>

#include <type_traits>

#include "mlr_router.cuh"

namespace mlr {
namespace {

constexpr int kBalanceThreads = 256;

// A sum over the block, the same in every thread (E > 1024: a token per block).
__device__ __forceinline__ float block_sum(float v, float* red) {
  v = warp_sum(v);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  v = 0.f;
#pragma unroll
  for (int i = 0; i < kBalanceThreads / 32; ++i) v += red[i];
  return v;
}
__device__ __forceinline__ float block_max(float v, float* red) {
  v = warp_max(v);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  v = red[0];
#pragma unroll
  for (int i = 1; i < kBalanceThreads / 32; ++i) v = fmaxf(v, red[i]);
  return v;
}

// How the threads hold a token's logits.  LPT lanes of a warp with V each (E up to
// 1024), or the block (LPT = 256).
template <int LPT> constexpr bool kBlockTokens = LPT == kBalanceThreads;
template <int LPT> constexpr int kTeams = kBalanceThreads / LPT;
template <int LPT>
__device__ __forceinline__ float team_sum(float v, float* red) {
  if constexpr (kBlockTokens<LPT>) return block_sum(v, red);
  else return part_sum<LPT>(v);
}
template <int LPT>
__device__ __forceinline__ float team_max(float v, float* red) {
  if constexpr (kBlockTokens<LPT>) return block_max(v, red);
  else return part_max<LPT>(v);
}
template <int LPT>
__device__ __forceinline__ void team_sync() {
  if constexpr (kBlockTokens<LPT>) __syncthreads();
  else __syncwarp();
}

// Logits on the 16-byte grid are fetched a turn ahead (two or three turns: 2 to 4% slower).
template <int VEC, int LPT> constexpr bool kRing = VEC > 1 && !kBlockTokens<LPT>;
template <int VEC, int LPT, int V, int THREADS = kBalanceThreads>
constexpr int kRingBytes = kRing<VEC, LPT> ? V / VEC * THREADS * 16 : 0;

// A token's logits in v, those that are not finite and those past E to -inf.  Every thread of
// the warp calls it.
template <int VEC, int LPT, int V>
__device__ __forceinline__ void close_logits(int E, int ll, float (&v)[V]) {
  if (__any_sync(0xffffffffu, !(check_finite(v) == 0.f)))
#pragma unroll
    for (int i = 0; i < V; ++i) v[i] = finite_logit(v[i]);
  close_past<VEC, LPT>(E, ll, v);
}
// 1 / sum, 0 where that is next to 0 (sigmoids have lost bits there, and the quotient might
// overflow) and for a token that is not active.
__device__ __forceinline__ float inverse_of(float sum, bool active) { return active && sum >= FLT_MIN ? 1.f / sum : 0.f; }
// v: a token's logits to s, zeros past E and for logits that are not finite.  Returns the
// inverse of their sum.  Every thread of the warp (the block) calls it.
template <int VEC, int LPT, int V>
__device__ __forceinline__ float scores(int E, bool sigmoid, int ll, bool active, float* red, float (&v)[V]) {
  close_logits<VEC, LPT>(E, ll, v);
  float sum = 0.f;
  if (sigmoid) {
#pragma unroll
    for (int i = 0; i < V; ++i) sum += v[i] = share_sigmoid(v[i]);
  } else {
    float most = team_max<LPT>(max_of<0, 1>(v), red);
    most = most > -CUDART_INF_F ? most : 0.f;
#pragma unroll
    for (int i = 0; i < V; ++i) sum += v[i] = share_exp(v[i] - most);
  }
  return inverse_of(team_sum<LPT>(sum, red), active);
}
// v: a token's logits to s (1 - s) of sigmoids s; `mean` the sum of s coef over that of s.
template <int VEC, int LPT, int V>
__device__ __forceinline__ float slopes(int E, int ll, bool active, float* red, const float (&coef)[V], float (&v)[V],
                                        float& mean) {
  close_logits<VEC, LPT>(E, ll, v);
  float sum = 0.f, dot = 0.f;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const float s = share_sigmoid(v[i], v[i]);
    sum += s;
    dot = fmaf(s, coef[i], dot);
  }
  const float inv = inverse_of(team_sum<LPT>(sum, red), active);
  mean = team_sum<LPT>(dot, red) * inv;
  return inv;
}

// The loss of v = sum over experts of shares times pairs.
__device__ __forceinline__ float loss_of(double v, int tokens, int E, int K) {
  const double n = tokens > 0 ? tokens : 1;
  return (float)(v * E / (K * n * n));
}

constexpr int kLossCluster = 8;
// One cluster of eight blocks can take a batch of up to this many logits, without a workspace
// and a second launch.  It does so up to kOneClusterTokens, which saves a caller 4 us and costs
// the device 0.3 to 6, more with every turn of its few blocks (us of a caller and of the device,
// the cluster and two launches: 1024 x 8 14.6 and 5.1, 19.1 and 4.5; 4096 x 128 15.6 and 11.5,
// 19.6 and 5.8; 8192 x 8 14.6 and 12.1, 19.6 and 6.1; 16384 x 8 20.7 and 20.3, 19.3 and 8.6;
// 65536 x 8 68 and 68, 19.9 and 11.9), and beyond where no workspace is given.
constexpr int64_t kOneClusterLogits = 1 << 19;
constexpr int kOneClusterTokens = 8192;
constexpr uint32_t kTurns = 64;  // of a thread's sum of shares
template <int V> constexpr int kOneThreads = V == 32 ? 512 : 1024;  // of its blocks, by their registers

// Sums of shares and pairs per expert over the block's tokens.  ONE: the grid is one
// cluster, which adds them over distributed shared memory and writes counts and loss;
// else part [blocks][E] and count [blocks][E + 1] (the last one: tokens).
template <int VEC, int LPT, int V, bool ONE, typename E_>
__global__ void __launch_bounds__(ONE ? kOneThreads<V> : kBalanceThreads, ONE ? 1 : V <= 16 && !kBlockTokens<LPT> ? 4 : 2)
balance_kernel(const E_* __restrict__ logits, const int32_t* __restrict__ ids, const uint8_t* __restrict__ mask, int T, int E,
               int K, bool sigmoid, float* __restrict__ part, int32_t* __restrict__ count, float* __restrict__ loss, int32_t* status) {
  extern __shared__ uint4 ring[];  // the ring; then [E + 1] pairs; then float [warps (1 for a block's token)][E] shares
  __shared__ float red[kBalanceThreads / 32];
  constexpr int THREADS = ONE ? kOneThreads<V> : kBalanceThreads;
  constexpr int TEAMS = THREADS / LPT, ROWS = kBlockTokens<LPT> ? 1 : THREADS / 32;
  int* hist = reinterpret_cast<int*>(reinterpret_cast<char*>(ring) + kRingBytes<VEC, LPT, V, THREADS>);
  float* sums = reinterpret_cast<float*>(hist + E + 1);
  const int team = threadIdx.x / LPT, ll = threadIdx.x % LPT;
  for (int e = threadIdx.x; e <= E; e += THREADS) hist[e] = 0;
  __syncthreads();
  pdl_wait();
  pdl_trigger();
  // tokens as unsigned numbers: the one a turn after the last is below 2^32
  const uint32_t step = gridDim.x * TEAMS;
  uint32_t t = blockIdx.x * TEAMS + team;
  auto fetch = [&](uint32_t t) {
    if constexpr (kRing<VEC, LPT>)
      fetch_logits<VEC, LPT, V, THREADS>(ring, logits + (int64_t)t * E, E, ll, t < (uint32_t)T);
  };
  fetch(t);
  int tokens = 0;
  // whether the next turn's token counts, and its place of this lane (the first of more
  // than LPT), asked for a turn before they are used
  auto counts_in = [&](uint32_t t) { return t >= (uint32_t)T ? 0 : mask == nullptr ? 1 : (int)__ldg(mask + t); };
  auto place = [&](uint32_t t) { return t < (uint32_t)T && ll < K ? __ldg(ids + (int64_t)t * K + ll) : -1; };
  int next_active = counts_in(t);  // compared when it is used
  int next_first = place(t);
  // Sums go to the warp's row (the block's) kTurns at a time: in a longer one, rows of one
  // kind would be rounded the same way at every addition.
  uint32_t left = blockIdx.x * TEAMS < (uint32_t)T ? (T - blockIdx.x * TEAMS - 1) / step + 1 : 0;  // turns
  bool added = false;
  do {
    float acc[V] = {};
    uint32_t turns = min(left, kTurns);
    left -= turns;
    for (; turns > 0; --turns, t += step) {
      const bool active = next_active != 0;
      const int first = next_first;
      next_active = counts_in(t + step);
      next_first = place(t + step);
      float v[V];
      if constexpr (kRing<VEC, LPT>) {
        take_logits<VEC, LPT, V, THREADS>(ring, E, ll, active, v);
        fetch(t + step);
      } else {
        load_logits<VEC, LPT>(logits + (active ? (int64_t)t : 0) * E, E, ll, active, v);
      }
      const float inv = scores<VEC, LPT>(E, sigmoid, ll, active, red, v);
#pragma unroll
      for (int i = 0; i < V; i += 2) {
        const float2 q = __ffma2_rn(make_float2(v[i], v[i + 1]), make_float2(inv, inv), make_float2(acc[i], acc[i + 1]));
        acc[i] = q.x;
        acc[i + 1] = q.y;
      }
      if (active) {
        ++tokens;
        for (int k = ll; k < K; k += LPT) {
          const int id = k == ll ? first : __ldg(ids + (int64_t)t * K + k);
          if (id >= 0 && id < E) atomicAdd(&hist[id], 1);
          else if (id != -1) set_status(status, MLR_STATUS_INDEX);
        }
      }
    }
    if constexpr (!kBlockTokens<LPT>)
#pragma unroll
      for (int o = LPT; o < 32; o <<= 1)
#pragma unroll
        for (int i = 0; i < V; ++i) acc[i] += __shfl_xor_sync(0xffffffffu, acc[i], o);
    if (kBlockTokens<LPT> || (threadIdx.x & 31) < LPT)
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const int e = (ll + LPT * (i / VEC)) * VEC + i % VEC;
        float* sum = sums + (kBlockTokens<LPT> ? 0 : threadIdx.x >> 5) * E + e;
        if (e < E) *sum = added ? *sum + acc[i] : acc[i];
      }
    added = true;
  } while (left > 0);
  if (ll == 0) atomicAdd(&hist[E], tokens);
  __syncthreads();
  for (int e = threadIdx.x; e <= E; e += THREADS) {
    if (!ONE) count[(int64_t)blockIdx.x * (E + 1) + e] = hist[e];
    if (e == E) continue;
    float v = 0.f;
#pragma unroll
    for (int i = 0; i < ROWS; ++i) v += sums[i * E + e];
    if (ONE) sums[e] = v;  // read above by this thread alone
    else part[(int64_t)blockIdx.x * E + e] = v;
  }
  if constexpr (ONE) {
    namespace cg = cooperative_groups;
    __shared__ double total;
    const cg::cluster_group cluster = cg::this_cluster();
    cluster.sync();
    double mine = 0.0;
    for (int e = blockIdx.x * 32 + threadIdx.x; threadIdx.x < 32 && e <= E; e += kLossCluster * 32) {
      int c = 0;
      float v = 0.f;
#pragma unroll
      for (int b = 0; b < kLossCluster; ++b) {
        c += cluster.map_shared_rank(hist, b)[e];
        if (e < E) v += cluster.map_shared_rank(sums, b)[e];
      }
      count[e] = c;
      if (e < E) mine += (double)v * c;
    }
    if (threadIdx.x < 32) {
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) mine += __shfl_xor_sync(0xffffffffu, mine, o);
      if (threadIdx.x == 0) total = mine;
    }
    cluster.sync();
    if (blockIdx.x == 0 && threadIdx.x == 0) {
      int n = 0;
      for (int b = 0; b < kLossCluster; ++b) n += cluster.map_shared_rank(hist, b)[E];
      for (int b = 1; b < kLossCluster; ++b) mine += *cluster.map_shared_rank(&total, b);
      *loss = loss_of(mine, n, E, K);
    }
    cluster.sync();  // the blocks' shared memory is read until here
  }
}

// The blocks' sums added in order, by one cluster: a block takes every eighth run of
// 32 experts, a warp every 32nd row; then the loss, over distributed shared memory.
constexpr int kTotalThreads = 1024, kTotalCluster = 8;
__global__ void __cluster_dims__(kTotalCluster, 1, 1) __launch_bounds__(kTotalThreads)
balance_total_kernel(const float* __restrict__ part, const int32_t* __restrict__ count, int blocks, int E, int K,
                     float* __restrict__ loss, int32_t* __restrict__ counts) {
  namespace cg = cooperative_groups;
  __shared__ float sums[32][33];
  __shared__ int pairs[32][33];
  __shared__ double total;   // of this block's experts
  __shared__ int tokens;     // in the block that has column E
  const cg::cluster_group cluster = cg::this_cluster();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  double mine = 0.0;  // warp 0
  pdl_wait();
  pdl_trigger();
  for (int e0 = blockIdx.x * 32; e0 <= E; e0 += kTotalCluster * 32) {
    const int e = e0 + lane;
    float s = 0.f;  // of a few hundred positive terms; fp64 takes 16 cycles an instruction
    int c = 0;
    if (e <= E)
#pragma unroll 4
      for (int b = warp; b < blocks; b += 32) {
        c += count[(int64_t)b * (E + 1) + e];
        if (e < E) s += part[(int64_t)b * E + e];
      }
    __syncthreads();
    sums[warp][lane] = s;
    pairs[warp][lane] = c;
    __syncthreads();
    if (warp == 0 && e <= E) {
      s = 0.f;
      c = 0;
#pragma unroll
      for (int i = 0; i < 32; ++i) {
        s += sums[i][lane];
        c += pairs[i][lane];
      }
      counts[e] = c;
      if (e == E) tokens = c;
      else mine += (double)s * c;
    }
  }
  if (warp == 0) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) mine += __shfl_xor_sync(0xffffffffu, mine, o);
    if (lane == 0) total = mine;
  }
  cluster.sync();
  if (blockIdx.x == 0 && threadIdx.x == 0) {
    double v = 0.0;
    for (int i = 0; i < kTotalCluster; ++i) v += *cluster.map_shared_rank(&total, i);
    const int n = *cluster.map_shared_rank(&tokens, E / 32 % kTotalCluster);
    *loss = loss_of(v, n, E, K);
  }
  cluster.sync();  // the blocks' shared memory is read until here
}

// a b with what its rounding leaves, as the sum of two floats.
__device__ __forceinline__ float2 product2(float a, float b) {
  const float p = a * b;
  return make_float2(p, fmaf(a, b, -p));
}
// d E / (K n^2) so.
__device__ __forceinline__ float2 coefficient2(float d, float E, float K, float n) {
  const float2 nn = product2(n, n), a = product2(d, E);
  float2 b = product2(nn.x, K);
  b.y = fmaf(nn.y, K, b.y);
  const float q = a.x / b.x;
  return make_float2(q, __fdividef(fmaf(-q, b.x, a.x) + fmaf(-q, b.y, a.y), b.x));
}

struct GradArgs {
  const int32_t* ids;
  const float* d_weights;  // nullable: no gradient of the weights
  const int32_t* counts;   // nullable: none of the loss
  const float* d_loss;
  const uint8_t* mask;
  int T, E, K;
  bool sigmoid, renormalize;
  float scale;
};

// Gradient of the logits.  What comes by the weights is put together by lanes that
// take a place each (place ll + LPT c; in a block's token: its first warp) and laid
// in a row of shared memory, zero elsewhere, from where the experts' lanes take it.
template <int VEC, int LPT, int V, typename E_>
__global__ void __launch_bounds__(kBalanceThreads, V <= 16 && !kBlockTokens<LPT> ? 4 : 2)
route_backward_kernel(const E_* __restrict__ logits, const __grid_constant__ GradArgs a, E_* __restrict__ d_logits,
                      int32_t* status) {
  extern __shared__ uint4 ring[];  // the ring (with shares); then float [teams][E], zero but for the chosen experts
  __shared__ float red[kBalanceThreads / 32];
  constexpr int TEAMS = kTeams<LPT>;
  constexpr int PL = kBlockTokens<LPT> ? 32 : LPT;  // lanes that take places
  constexpr int CP = kMaxRouteTopk / PL;
  const int team = threadIdx.x / LPT, ll = threadIdx.x % LPT;
  const int E = a.E, K = a.K;
  const bool by_weights = a.d_weights != nullptr, all_chosen = by_weights && !a.sigmoid && !a.renormalize;
  const bool shares = a.counts != nullptr || all_chosen;
  float* row_s = reinterpret_cast<float*>(reinterpret_cast<char*>(ring) + (shares ? kRingBytes<VEC, LPT, V> : 0)) + team * E;
  if (by_weights) {
    for (int e = ll; e < E; e += LPT) row_s[e] = 0.f;
    team_sync<LPT>();
  }
  pdl_wait();
  pdl_trigger();
  float coef[V] = {};
  if (a.counts != nullptr) {
    // as the sum of two floats, so that a coefficient is rounded once (64-bit operations for
    // every expert of every thread took 14% of the time); counts are, beyond 2^24
    const float2 f = coefficient2(__ldg(a.d_loss), (float)E, (float)K, (float)max(1, __ldg(a.counts + E)));
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int e = (ll + LPT * (i / VEC)) * VEC + i % VEC;
      if (e < E) {
        const float c = (float)__ldg(a.counts + e);
        coef[i] = fmaf(f.x, c, f.y * c);
      }
    }
  }
  const int64_t step = (int64_t)gridDim.x * TEAMS;
  auto fetch = [&](int64_t t) {
    if constexpr (kRing<VEC, LPT>)
      fetch_logits<VEC, LPT, V, kBalanceThreads>(ring, logits + t * E, E, ll, t < a.T);
  };
  if (shares) fetch((int64_t)blockIdx.x * TEAMS + team);
  for (int64_t t0 = (int64_t)blockIdx.x * TEAMS; t0 < a.T; t0 += step) {
    const int64_t t = t0 + team;
    const bool active = t < a.T && (a.mask == nullptr || a.mask[t]);
    const E_* row = logits + (active ? t : 0) * E;
    float v[V] = {};
    float inv = 0.f, dot = 0.f;
    if (shares) {
      if constexpr (kRing<VEC, LPT>) {
        take_logits<VEC, LPT, V, kBalanceThreads>(ring, E, ll, active, v);
        if (a.mask != nullptr) fetch(t + step);
      } else {
        load_logits<VEC, LPT>(row, E, ll, active, v);
      }
      inv = a.sigmoid ? slopes<VEC, LPT>(E, ll, active, red, coef, v, dot) : scores<VEC, LPT>(E, false, ll, active, red, v);
    }
    int id[CP];
    if (by_weights) {
      if (!kBlockTokens<LPT> || threadIdx.x < 32) {
        float dl[CP], s[CP], g[CP];
        float total = 0.f, mean = 0.f, most = -CUDART_INF_F;
#pragma unroll
        for (int c = 0; c < CP; ++c) {
          const int k = ll + c * PL;
          id[c] = active && k < K ? __ldg(a.ids + t * K + k) : -1;
          if (id[c] < -1 || id[c] >= E) {
            set_status(status, MLR_STATUS_INDEX);
            id[c] = -1;
          }
          s[c] = id[c] >= 0 ? finite_logit(row + id[c]) : -CUDART_INF_F;
          if (!(s[c] > -CUDART_INF_F)) id[c] = -1;
          g[c] = id[c] >= 0 ? a.scale * __ldg(a.d_weights + t * K + k) : 0.f;
          most = fmaxf(most, s[c]);
        }
        if (all_chosen) {
#pragma unroll
          for (int c = 0; c < CP; ++c) dl[c] = g[c];  // times p below
        } else {
          if (!a.sigmoid) most = part_max<PL>(most);
#pragma unroll
          for (int c = 0; c < CP; ++c) {
            dl[c] = a.sigmoid ? sigmoid_f(-s[c]) : 1.f;  // not 1 - s, which cancels
            s[c] = id[c] < 0 ? 0.f : a.sigmoid ? sigmoid_f(s[c]) : expf(s[c] - most);
            total += s[c];
          }
          if (a.renormalize) {  // s to the shares of the weights
            total = part_sum<PL>(total);
            const float lift = lift_of(total), inverse = total > 0.f ? 1.f / (total * lift) : 0.f;
#pragma unroll
            for (int c = 0; c < CP; ++c) {
              s[c] = s[c] * lift * inverse;
              mean = fmaf(g[c], s[c], mean);
            }
            mean = part_sum<PL>(mean);
          }
#pragma unroll
          for (int c = 0; c < CP; ++c) dl[c] *= s[c] * (g[c] - mean);
        }
        // an expert that a token holds twice gets both, in order
        bool twice = K > PL;
        if (!twice) {
          const uint32_t same = __match_any_sync(0xffffffffu, id[0] < 0 ? ~(int)threadIdx.x : id[0] + (team % (32 / PL)) * E);
          twice = __any_sync(0xffffffffu, (same & (same - 1)) != 0);
        }
        if (!twice) {
          if (id[0] >= 0) row_s[id[0]] = dl[0];
        } else {
#pragma unroll
          for (int c = 0; c < CP; ++c)
            for (int l = 0; l < PL; ++l) {
              if (ll == l && id[c] >= 0) row_s[id[c]] += dl[c];
              __syncwarp();
            }
        }
      }
      team_sync<LPT>();
    }
    // d: what the place's lane has left of an expert
    if (shares && !a.sigmoid) {
#pragma unroll
      for (int j = 0; j < V / VEC; ++j) {
        const int e = (ll + LPT * j) * VEC;
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
          const int n = j * VEC + i;
          float q = coef[n];
          if (all_chosen && e < E) q += row_s[e + i];
          dot = fmaf(v[n], q, dot);
        }
      }
      dot = team_sum<LPT>(dot, red) * inv;
    }
#pragma unroll
    for (int j = 0; j < V / VEC; ++j) {
      const int e = (ll + LPT * j) * VEC;
      if (e >= E) continue;
      float o[VEC];
#pragma unroll
      for (int i = 0; i < VEC; ++i) {
        const int n = j * VEC + i;
        const float d = by_weights ? row_s[e + i] : 0.f;
        const float p = v[n] * inv;
        o[i] = all_chosen ? p * (coef[n] + d - dot) : fmaf(p, coef[n] - dot, d);
      }
      if (t < a.T) {
        if constexpr (VEC == 1) {
          row_narrow(o[0], d_logits[t * E + e]);
        } else {
          uint4 q;
          row_narrow(o, q);
          *reinterpret_cast<uint4*>(d_logits + t * E + e) = q;
        }
      }
    }
    // A mask's loads space the turns out, and the next logits are best asked for at once;
    // without one after this turn's stores (262144 x 256: 84 and 88 us, 96 and 88).
    if (shares && a.mask == nullptr) fetch(t + step);
    if (by_weights) {
      team_sync<LPT>();
      if (!kBlockTokens<LPT> || threadIdx.x < 32)
#pragma unroll
        for (int c = 0; c < CP; ++c)
          if (id[c] >= 0) row_s[id[c]] = 0.f;
      team_sync<LPT>();
    }
  }
  // Coefficients beyond the range (a loss scale that ran over) made NaN of the masked tokens'
  // zeros: each thread writes its own again.  A coefficient is at most d_loss E, E of them E times that.
  if (a.counts != nullptr && a.mask != nullptr && !(fabsf(__ldg(a.d_loss)) < FLT_MAX / kMaxRouteExperts / kMaxRouteExperts)) {
#pragma unroll 1
    for (int64_t t = (int64_t)blockIdx.x * TEAMS + team; t < a.T; t += step) {
      if (a.mask[t]) continue;
#pragma unroll 1
      for (int e = ll * VEC; e < E; e += LPT * VEC)
        for (int i = 0; i < VEC; ++i) row_narrow(0.f, d_logits[t * E + e + i]);
    }
  }
}

// f<LPT, V>() for E experts.
template <typename F>
int by_experts(int E, F f) {
  using std::integral_constant;
  if (E <= 64) return f(integral_constant<int, 8>{}, integral_constant<int, 8>{});
  if (E <= 128) return f(integral_constant<int, 8>{}, integral_constant<int, 16>{});
  if (E <= 256) return f(integral_constant<int, 8>{}, integral_constant<int, 32>{});
  if (E <= 512) return f(integral_constant<int, 16>{}, integral_constant<int, 32>{});
  if (E <= kPartExperts) return f(integral_constant<int, 32>{}, integral_constant<int, 32>{});
  return f(integral_constant<int, kBalanceThreads>{}, integral_constant<int, 16>{});
}
int lanes_of(int E) { return E <= 256 ? 8 : E <= 512 ? 16 : E <= kPartExperts ? 32 : kBalanceThreads; }

// Blocks of an SM, by the registers of the two kernels.
int blocks_per_sm(int E) { return E <= 128 ? 4 : 2; }
int64_t balance_blocks(int32_t T, int32_t E) {
  const int64_t want = ceil_div(T, kBalanceThreads / lanes_of(E)), most = (int64_t)blocks_per_sm(E) * current_sms();
  return want < 1 ? 1 : want < most ? want : most;
}

bool one_cluster(int32_t T, int32_t E) { return E <= 256 && (int64_t)T * E <= kOneClusterLogits; }

template <int VEC, typename E_>
int run_balance(const void* logits, const int32_t* ids, const uint8_t* mask, int T, int E, int K, bool sigmoid, float* part,
                int32_t* count, float* loss, int32_t* counts, int32_t* status, cudaStream_t stream) {
  const E_* l = static_cast<const E_*>(logits);
  return by_experts(E, [&](auto lpt, auto v) {
    constexpr int ring = kRingBytes<VEC, lpt.value, v.value>;
    constexpr int rows = kBlockTokens<lpt.value> ? 1 : kBalanceThreads / 32, cover = lpt.value * v.value;
    auto bytes = [&](int experts) { return (size_t)ring + (experts + 1) * 4 + (size_t)rows * experts * 4; };
    if constexpr (lpt.value == 8) {
      if (part == nullptr) {
        auto kernel = balance_kernel<VEC, lpt.value, v.value, true, E_>;
        constexpr int threads = kOneThreads<v.value>;
        auto of_one = [&](int experts) {
          return (size_t)kRingBytes<VEC, lpt.value, v.value, threads> + (experts + 1) * 4 + (size_t)threads / 32 * experts * 4;
        };
        const size_t smem = of_one(E);
        cudaError_t err = cudaSuccess;
        if (smem > 46 * 1024)
          err = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)of_one(cover));
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(kLossCluster);
        cfg.blockDim = dim3(threads);
        cfg.dynamicSmemBytes = smem;
        cfg.stream = stream;
        cudaLaunchAttribute attr[2];
        attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[0].val.programmaticStreamSerializationAllowed = 1;
        attr[1].id = cudaLaunchAttributeClusterDimension;
        attr[1].val.clusterDim.x = kLossCluster;
        attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 2;
        if (err == cudaSuccess)
          err = cudaLaunchKernelEx(&cfg, kernel, l, ids, mask, T, E, K, sigmoid, (float*)nullptr, counts, loss, status);
        return launched(err);
      }
    }
    const int blocks = (int)balance_blocks(T, E);
    const int c = launch_with_smem(balance_kernel<VEC, lpt.value, v.value, false, E_>, dim3(blocks), dim3(kBalanceThreads),
                                   bytes(E), (int)bytes(cover), stream, l, ids, mask, T, E, K, sigmoid, part, count,
                                   (float*)nullptr, status);
    if (c != MLR_OK) return c;
    return launched(launch_pdl(balance_total_kernel, dim3(kTotalCluster), dim3(kTotalThreads), 0, stream, (const float*)part,
                               (const int32_t*)count, blocks, E, K, loss, counts));
  });
}

template <int VEC, typename E_>
int run_backward(const void* logits, const GradArgs& a, void* d_logits, int32_t* status, cudaStream_t stream) {
  return by_experts(a.E, [&](auto lpt, auto v) {
    constexpr int teams = kTeams<lpt.value>, ring = kRingBytes<VEC, lpt.value, v.value>, cover = lpt.value * v.value;
    const int64_t want = ceil_div(a.T, teams), most = (int64_t)blocks_per_sm(a.E) * current_sms();
    const bool shares = a.counts != nullptr || (!a.sigmoid && !a.renormalize);
    const size_t smem = (shares ? ring : 0) + (a.d_weights != nullptr ? (size_t)teams * a.E * 4 : 0);
    return launch_with_smem(route_backward_kernel<VEC, lpt.value, v.value, E_>, dim3((unsigned)(want < most ? want : most)),
                            dim3(kBalanceThreads), smem, ring + teams * cover * 4, stream, static_cast<const E_*>(logits), a,
                            static_cast<E_*>(d_logits), status);
  });
}

// f<VEC, E_>() for logits (and their gradient) of a type, in vectors where they lie on the 16-byte grid.
template <typename F>
int by_type(int dtype, int E, const void* logits, const void* d_logits, F f) {
  const bool bf16 = dtype == MLR_DTYPE_BF16;
  const bool whole = E % (bf16 ? 8 : 4) == 0 && aligned_to(logits, 16) && aligned_to(d_logits, 16);
  using std::integral_constant;
  if (bf16) return whole ? f(integral_constant<int, 8>{}, uint16_t{}) : f(integral_constant<int, 1>{}, uint16_t{});
  return whole ? f(integral_constant<int, 4>{}, float{}) : f(integral_constant<int, 1>{}, float{});
}

}  // namespace
}  // namespace mlr

extern "C" size_t moe_balance_loss_workspace_bytes(int32_t num_tokens, int32_t num_experts) {
  using namespace mlr;
  if (num_tokens < 0 || num_experts < 1 || num_experts > kMaxRouteExperts) return 0;
  if (one_cluster(num_tokens, num_experts) && num_tokens <= kOneClusterTokens) return 1;  // nothing is kept
  return (size_t)balance_blocks(num_tokens, num_experts) * (2 * num_experts + 1) * 4;
}

extern "C" int moe_balance_loss(const void* logits, const int32_t* topk_ids, const uint8_t* token_mask, int32_t num_tokens,
                                int32_t num_experts, int32_t topk, int32_t dtype, int32_t scoring, float* loss, int32_t* counts,
                                void* workspace, size_t ws_bytes, int32_t* d_status, void* stream_) {
  using namespace mlr;
  cudaStream_t stream = static_cast<cudaStream_t>(stream_);
  const int code = check_logits(logits, num_tokens, num_experts, topk, dtype, scoring);
  if (code != MLR_OK) return code;
  if (loss == nullptr || counts == nullptr || (num_tokens > 0 && topk_ids == nullptr)) return MLR_ERR_INVALID;
  if (!on_word_grid({topk_ids, loss, counts, d_status})) return MLR_ERR_INVALID;
  const bool one = one_cluster(num_tokens, num_experts);
  const bool fits = workspace != nullptr && ws_bytes >= moe_balance_loss_workspace_bytes(num_tokens, num_experts);
  if (!one && !fits) return MLR_ERR_CAPACITY;
  const bool two = fits && !(one && num_tokens <= kOneClusterTokens);
  if (!aligned_to(workspace, 256)) return MLR_ERR_INVALID;
  float* part = two ? static_cast<float*>(workspace) : nullptr;
  int32_t* count = two ? reinterpret_cast<int32_t*>(part + balance_blocks(num_tokens, num_experts) * num_experts) : nullptr;
  return by_type(dtype, num_experts, logits, nullptr, [&](auto vec, auto e) {
    return run_balance<vec.value, decltype(e)>(logits, topk_ids, token_mask, num_tokens, num_experts, topk, scoring == kSigmoid,
                                               part, count, loss, counts, d_status, stream);
  });
}

extern "C" int moe_route_backward(const void* logits, const int32_t* topk_ids, const float* d_weights, const int32_t* counts,
                                  const float* d_loss, const uint8_t* token_mask, int32_t num_tokens, int32_t num_experts,
                                  int32_t topk, int32_t dtype, int32_t scoring, int32_t renormalize, float scale, void* d_logits,
                                  int32_t* d_status, void* stream_) {
  using namespace mlr;
  cudaStream_t stream = static_cast<cudaStream_t>(stream_);
  const int code = check_logits(logits, num_tokens, num_experts, topk, dtype, scoring);
  if (code != MLR_OK) return code;
  if (num_tokens == 0) return MLR_OK;  // empty tensors may have no address
  if ((counts == nullptr) != (d_loss == nullptr) || (d_weights == nullptr && counts == nullptr)) return MLR_ERR_INVALID;
  if (d_logits == nullptr || !aligned_to(d_logits, dtype == MLR_DTYPE_BF16 ? 2 : 4) || (d_weights != nullptr && topk_ids == nullptr) ||
      !on_word_grid({topk_ids, d_weights, counts, d_loss, d_status}))
    return MLR_ERR_INVALID;
  const GradArgs a{topk_ids, d_weights, counts, d_loss, token_mask, num_tokens, num_experts, topk, scoring == kSigmoid,
                   renormalize != 0, scale};
  return by_type(dtype, num_experts, logits, d_logits, [&](auto vec, auto e) {
    return run_backward<vec.value, decltype(e)>(logits, a, d_logits, d_status, stream);
  });
}
