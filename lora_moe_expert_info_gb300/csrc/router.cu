// router.cu -- the router's choice of experts from its logits.
//
// Logits [T, E]; one that is not finite counts as -inf, and its expert is never
// chosen.  An expert's choice score is its logit, or with a bias or (sigmoid)
// groups sigmoid(logit) + bias.  With groups only the experts of the topk_groups
// best groups stand to choice; a group's score is its best choice score (softmax)
// or the sum of its two best (sigmoid).  Ties go to the lowest index.  With s =
// softmax(logits) or sigmoid(logits): w_k = scale s_k [/ sum of the chosen s].
//
// The choice is decided by the numbers that the scores stand for: where 32 bits do not
// tell two of them apart, they are computed in 64, to a few units of the last place.
//
// A token's logits are read once and stay in registers.  A million tokens, 8 of 256
// experts: 241 us, 70% of the copy rate; what bounds it is the ALU pipe (56% busy) and
// the latency of the merges and ranks, at 45% of the warps.  One token 2.8 us; 256
// tokens of 256 experts in groups with biases 7.5, 10 where some scores are near.
// Few experts cost as much as 64 (a million tokens, 2 of 8: 171 us).  More than 1024
// experts, 16 places, or groups than a token has lanes (8 up to 256 experts, 16 up to 512,
// else 32) go through the exact choice alone: 262144 tokens, 20 of 256 experts 1155 us (16 of
// them 120); 65536 tokens, 8 of 2048 experts 2775 (8 of 1024 64); in 16 groups 1140 (in 8 54).
#include <float.h>

#include "mlr_router.cuh"

namespace mlr {
namespace {

constexpr int kMaxGroups = 256;

// Whether a logit is one that the caller hears of: NaN or +inf.
__device__ __forceinline__ bool bad_logit(float v) { return !(v < CUDART_INF_F); }

struct RouteArgs {
  const float* bias;
  const uint8_t* mask;
  int T, E, K, groups, best;
  bool sigmoid, renormalize;
  float scale;
  int32_t* ids;
  float* weights;
  int32_t* status;
};

// How near two sigmoid + bias may be in fp32 and still be in either order: each is
// off by at most 2.25 2^-23 (ex2 2^-22 and its argument |l| 2^-23, both times s (1 -
// s); 1 + e 2^-24; rcp 2^-23) and the sum's 2^-24 |c|; twice that, rounded up.
__device__ __forceinline__ float near_score(float c) { return fmaf(fabsf(c), 0x1p-22f, 0x1p-20f); }
// Doubles as integers of the same order (there is no -0 among them), which are
// compared in a few cycles: GB300 takes 16 to issue a comparison of doubles.
constexpr long long kLowest = (long long)0x800fffffffffffff;  // -inf
__device__ __forceinline__ long long ordered(double v) {
  const long long b = __double_as_longlong(v);
  return b ^ ((b >> 63) & 0x7fffffffffffffffll);
}
__device__ __forceinline__ double from_ordered(long long k) {
  return __longlong_as_double(k ^ ((k >> 63) & 0x7fffffffffffffffll));
}
// sigmoid(logit) + bias in 64 bits, to a few units of the last place.  With t = e^-|l|
// it is 1 / (1 + t) or t / (1 + t); t = 2^n e^r with n = -|l| / ln 2 rounded, e^r a
// Taylor polynomial (|r| < 0.35: the 14th power's term is below 2^-57) summed
// pairwise, as the latency of one operation after another is what this costs; the
// quotient from a 32-bit one by two Newton steps.
__device__ __noinline__ double exact_score(float l, const float* bias, int e) {
  const double x = -fabs((double)l);
  const double n = rint(fmax(x, -750.0) * 1.4426950408889634);
  const double r = fma(n, -0x1.473de6af278edp-34, fma(n, -0x1.62e42fef00000p-1, x));  // ln 2 in two parts: n times the first is exact
  const double r2 = r * r, r4 = r2 * r2;
  const double p01 = 1.0 + r, p23 = fma(r, 1.0 / 6, 0.5), p45 = fma(r, 1.0 / 120, 1.0 / 24), p67 = fma(r, 1.0 / 5040, 1.0 / 720),
               p89 = fma(r, 1.0 / 362880, 1.0 / 40320), pab = fma(r, 1.0 / 39916800, 1.0 / 3628800),
               pcd = fma(r, 1.0 / 6227020800.0, 1.0 / 479001600);
  const double q0 = fma(r2, p23, p01), q4 = fma(r2, p67, p45), q8 = fma(r2, pab, p89);
  const double p = fma(r4, fma(r4, fma(r4, pcd, q8), q4), q0);
  const double t = x < -708.0 ? 0.0 : p * __longlong_as_double((long long)(1023 + (int)n) << 52);
  const double d = 1.0 + t;
  double y = (double)(1.f / (float)d);
  y = fma(y, fma(-d, y, 1.0), y);
  y = fma(y, fma(-d, y, 1.0), y);
  return (l < 0.f ? t * y : y) + (bias != nullptr ? (double)__ldg(bias + e) : 0.0);
}

// A group's score, the sum of its two best scores, in 64 bits; `third` is set where a
// third one is so near the second that 32 bits do not tell which of them it is, unless
// all that are so near have one logit and one bias.
template <typename E_>
__device__ __noinline__ long long exact_group(const RouteArgs& a, const E_* row, int g, bool& third) {
  const int size = a.E / a.groups;
  float b0 = -CUDART_INF_F, b1 = -CUDART_INF_F, b2 = -CUDART_INF_F;
  int i0 = -1, i1 = -1;
#pragma unroll 1
  for (int e = g * size; e < (g + 1) * size; ++e) {
    const float l = finite_logit(row + e);
    const float c = quick_sigmoid(l) + (a.bias != nullptr ? __ldg(a.bias + e) : 0.f);
    if (!(l > -CUDART_INF_F && c < CUDART_INF_F)) continue;
    if (c > b1) {
      b2 = b1;
      b1 = c;
      i1 = e;
      if (c > b0) {
        b1 = b0;
        i1 = i0;
        b0 = c;
        i0 = e;
      }
    } else {
      b2 = fmaxf(b2, c);
    }
  }
  third = false;
  if (b1 > -CUDART_INF_F && b1 - b2 <= near_score(b1)) {
    const float l1 = finite_logit(row + i1), c1 = a.bias != nullptr ? __ldg(a.bias + i1) : 0.f;
#pragma unroll 1
    for (int e = g * size; e < (g + 1) * size; ++e) {
      const float l = finite_logit(row + e), c = a.bias != nullptr ? __ldg(a.bias + e) : 0.f;
      third |= l > -CUDART_INF_F && fabsf(quick_sigmoid(l) + c - b1) <= near_score(b1) && (l != l1 || c != c1);
    }
  }
  double sum = 0.0;
#pragma unroll 1
  for (int k = 0; k < 2; ++k) {
    const int e = k == 0 ? i0 : i1;
    if (e >= 0) sum += exact_score(finite_logit(row + e), a.bias, e);
  }
  return i0 < 0 ? kLowest : ordered(sum + 0.0);
}

// The larger of two (score, index) pairs over the warp: the larger score, the
// lower index of equal ones.
__device__ __forceinline__ void warp_best(long long& v, int& i) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const long long u = __shfl_xor_sync(0xffffffffu, v, o);
    const int k = __shfl_xor_sync(0xffffffffu, i, o);
    if (u > v || (u == v && k < i)) {
      v = u;
      i = k;
    }
  }
}

// The weights of the chosen experts, lane k place k (id -1: none, and after the others).
template <typename E_>
__device__ __forceinline__ void write_choice(const RouteArgs& a, const E_* row, int64_t t, int id, int lane) {
  float s = 0.f;
  if (a.sigmoid) {
    if (id >= 0) s = sigmoid_f(finite_logit(row + id));
  } else {
    const float l = id >= 0 ? finite_logit(row + id) : -CUDART_INF_F;
    const float most = __shfl_sync(0xffffffffu, l, 0);  // the best one comes first
    s = id >= 0 ? expf(l - most) : 0.f;
    if (!a.renormalize) {
      float all = 0.f;
      if (most > -CUDART_INF_F)
        for (int e = lane; e < a.E; e += 32) all += expf(finite_logit(row + e) - most);
      all = warp_sum(all);
      s = id >= 0 ? s / all : 0.f;
    }
  }
  if (a.renormalize) {
    const float total = warp_sum(s);
    s = total > 0.f ? s / total : 0.f;
  }
  if (lane < a.K) {
    a.ids[t * a.K + lane] = id;
    a.weights[t * a.K + lane] = s * a.scale;
  }
}

// One token by one warp, every score in 64 bits: keys [E] and group scores [groups]
// in shared memory.
template <typename E_>
__device__ __noinline__ void choose_exactly(const RouteArgs& a, const E_* row, int64_t t, long long* key, long long* group,
                                            int lane) {
  const bool logit_key = !a.sigmoid || (a.bias == nullptr && a.groups == 1);
  // loops as they stand: this code is rarely run, and fetching it costs more than running it
#pragma unroll 1
  for (int e = lane; e < a.E; e += 32) {
    const float l = finite_logit(row + e);
    double k = (double)(l + 0.f);  // +0 for -0
    if (!logit_key && l > -CUDART_INF_F) {
      k = exact_score(l, a.bias, e);
      if (!(k < CUDART_INF)) k = -CUDART_INF;  // a bias that is NaN or +inf
    }
    key[e] = ordered(k);
  }
  __syncwarp();
  if (a.groups > 1) {
    const int size = a.E / a.groups;
    for (int g = lane; g < a.groups; g += 32) {
      long long b0 = kLowest, b1 = kLowest;
#pragma unroll 1
      for (int i = 0; i < size; ++i) {
        const long long k = key[g * size + i];
        b1 = max(b1, min(b0, k));
        b0 = max(b0, k);
      }
      group[g] = a.sigmoid && b1 > kLowest ? ordered(from_ordered(b0) + from_ordered(b1) + 0.0) : b0;
    }
    __syncwarp();
    for (int g = lane; g < a.groups; g += 32) {
      const long long mine = group[g];
      int before = 0;
#pragma unroll 1
      for (int o = 0; o < a.groups; ++o) before += group[o] > mine || (group[o] == mine && o < g);
      if (before >= a.best)
#pragma unroll 1
        for (int i = 0; i < size; ++i) key[g * size + i] = kLowest;
    }
    __syncwarp();
  }
  int mine = -1;
#pragma unroll 1
  for (int k = 0; k < a.K; ++k) {
    long long v = kLowest;
    int i = INT32_MAX;
#pragma unroll 1
    for (int e = lane; e < a.E; e += 32)
      if (key[e] > v) {
        v = key[e];
        i = e;
      }
    warp_best(v, i);
    if (v == kLowest) break;
    if (lane == k) mine = i;
    if (lane == (i & 31)) key[i] = kLowest;
    __syncwarp();
  }
  __syncwarp();
  write_choice(a, row, t, mine, lane);
}

constexpr int kRouteThreads = 128;
template <typename E_>
__global__ void __launch_bounds__(kRouteThreads)
route_kernel(const E_* __restrict__ logits, const __grid_constant__ RouteArgs a) {
  extern __shared__ long long smem[];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  long long* key = smem + (size_t)warp * (a.E + a.groups);
  pdl_wait();
  pdl_trigger();
  for (int64_t t = (int64_t)blockIdx.x * warps + warp; t < a.T; t += (int64_t)gridDim.x * warps) {
    const E_* row = logits + t * a.E;
    if (a.mask != nullptr && !a.mask[t]) {
      if (lane < a.K) {
        a.ids[t * a.K + lane] = -1;
        a.weights[t * a.K + lane] = 0.f;
      }
      continue;
    }
    if (a.status != nullptr) {
      bool bad = false;
      for (int e = lane; e < a.E; e += 32) bad |= bad_logit(row_widen(row[e]));
      if (bad) set_status(a.status, MLR_STATUS_VALUE);
    }
    choose_exactly(a, row, t, key, key + a.E, lane);
    __syncwarp();
  }
}

// ------------------------------------------------------- the choice, fast --
// LPT lanes take a token, V logits each (in units of VEC: unit number lane + LPT j),
// so a warp has 32 / LPT tokens at once.  The L-th largest of 4 L block maxima (L >= K
// the length of the sorted lists) is a lower bound of the K-th largest score; the
// few scores above it -- 1.15 L of them where scores are in no order -- are the
// candidates, which are ranked against one another.  Where two candidates are nearer
// than their 32 bits tell, the candidates alone are computed in 64; of equal logits at
// the bound only the first K stay; where there are more than 4 L of them even so, or
// a third expert might be one of a group's two, the token goes through choose_exactly.
//
// A warp's time goes to the ALU pipe (maxima, comparisons), which takes an
// instruction every two cycles.  A block has one turn: blocks that stay and fetch the
// next tokens' logits ahead take 339 us for a million tokens instead of 255 (fewer of
// them for the memory, and candidates that L1 has lost).

__device__ __forceinline__ void order_desc(float& a, float& b) {
  const float hi = fmaxf(a, b), lo = fminf(a, b);
  a = hi;
  b = lo;
}
// A bitonic sequence of N in descending order.
template <int N, int M>
__device__ __forceinline__ void bitonic_desc(float (&x)[M]) {
#pragma unroll
  for (int s = N / 2; s > 0; s >>= 1)
#pragma unroll
    for (int i = 0; i < N; ++i)
      if ((i & s) == 0) order_desc(x[i], x[i + s]);
}
// x[0..N) in descending order (odd-even merge sort).
template <int N, int M>
__device__ __forceinline__ void sort_desc(float (&x)[M]) {
#pragma unroll
  for (int p = 1; p < N; p <<= 1)
#pragma unroll
    for (int k = p; k > 0; k >>= 1)
#pragma unroll
      for (int j = k & (p - 1); j + k < N; j += 2 * k)
#pragma unroll
        for (int i = 0; i < k; ++i)
          if (i + j + k < N && (i + j) / (2 * p) == (i + j + k) / (2 * p)) order_desc(x[i + j], x[i + j + k]);
}
// The lists x[0..N) of LPT lanes merged to their L largest, in descending order, up to
// the last step: x and y are then the lists of a token's two halves.
template <int N, int L, int LPT, int O>
__device__ __forceinline__ void merge_lists(float (&x)[L], float (&y)[L]) {
#pragma unroll
  for (int i = 0; i < N; ++i) y[i] = __shfl_xor_sync(0xffffffffu, x[i], O);
  if constexpr (2 * O < LPT) {
    if constexpr (N < L) {
#pragma unroll
      for (int i = 0; i < N; ++i) x[2 * N - 1 - i] = y[i];
      bitonic_desc<2 * N>(x);
      merge_lists<2 * N, L, LPT, 2 * O>(x, y);
    } else {
#pragma unroll
      for (int i = 0; i < N; ++i) x[i] = fmaxf(x[i], y[N - 1 - i]);
      bitonic_desc<N>(x);
      merge_lists<N, L, LPT, 2 * O>(x, y);
    }
  }
}

// Of the logits in `hit` (bit 31 - i: the lane's i-th) all but those equal to the one at
// the bound, and of these the K of lowest index: no other of them can be chosen.  With
// choice scores, equal are those of one logit and one bias.
template <int VEC, int LPT, int V, typename E_>
__device__ __noinline__ uint32_t first_equals(const E_* row, const float* bias, bool biased, float bound, uint32_t hit, int K, int ll) {
  auto expert = [&](int i) { return (ll + LPT * (i / VEC)) * VEC + i % VEC; };
  auto bias_of = [&](int e) { return biased && bias != nullptr ? __ldg(bias + e) : 0.f; };
  float logit = bound, its_bias = 0.f;
  if (biased) {
    int at = INT32_MAX;
    for (uint32_t left = hit; left != 0; left &= left - 1) {
      const int e = expert(31 - (__ffs(left) - 1));
      if (quick_sigmoid(finite_logit(row + e)) + bias_of(e) == bound) at = min(at, e);
    }
    __syncwarp();
#pragma unroll
    for (int o = LPT / 2; o > 0; o >>= 1) at = min(at, __shfl_xor_sync(0xffffffffu, at, o));
    if (at == INT32_MAX) at = 0;  // none of the hits: then none is equal, or equals of any one go
    logit = finite_logit(row + at);
    its_bias = bias_of(at);
  }
  uint32_t keep = 0;
  for (uint32_t left = hit; left != 0; left &= left - 1) {
    const int i = 31 - (__ffs(left) - 1), e = expert(i);
    if (!(finite_logit(row + e) == logit && bias_of(e) == its_bias)) keep |= 0x80000000u >> i;
  }
  __syncwarp();
  const uint32_t equal = hit & ~keep;
#pragma unroll 1
  for (int j = 0, before = 0; j < V / VEC; ++j) {  // in the order of the experts: by unit, then by lane
    uint32_t own = equal & ((0xffffffffu << (32 - VEC)) >> (j * VEC));
    int upto = __popc(own);
#pragma unroll
    for (int o = 1; o < LPT; o <<= 1) {
      const int u = __shfl_up_sync(0xffffffffu, upto, o, LPT);
      if (ll >= o) upto += u;
    }
    for (int room = K - before - (upto - __popc(own)); own != 0 && room > 0; --room) {
      const uint32_t first = 0x80000000u >> __clz(own);
      keep |= first;
      own &= ~first;
    }
    __syncwarp();
    before += __shfl_sync(0xffffffffu, upto, LPT - 1, LPT);
  }
  return keep;
}

constexpr int kFastThreads = 128;
constexpr int kFastTopk = 16;

// Shared memory of a warp: the candidates' keys and ids, and room that is used for one
// thing at a time: the 64-bit keys of choose_exactly, the groups' two best of each unit,
// the 64-bit keys and the ranks of near candidates.
template <int L> constexpr int kCap = 4 * L;  // candidates of a token
template <int L>
struct alignas(16) Candidates {
  float key[kCap<L>];
  int id[kCap<L>];
};
template <int L>
struct alignas(16) Near {
  long long key[kCap<L>];
  int rank[kCap<L>];
};
template <int L>
int64_t fast_scratch(int E, int groups, int vec, int tokens) {
  const int64_t slow = (int64_t)(E + groups) * 8, best = groups > 1 ? (int64_t)tokens * (E / vec) * 8 : 0,
                near = (int64_t)tokens * sizeof(Near<L>);
  const int64_t most = slow > best ? slow : best;
  return round_up(most > near ? most : near, 16);
}

__device__ __forceinline__ int round_up4(int n) { return (n + 3) & ~3; }

template <typename E_, int VEC, int LPT, int V, int L>
__global__ void __launch_bounds__(kFastThreads, VEC == 1 ? 5 : 8)
route_fast_kernel(const E_* __restrict__ logits, const __grid_constant__ RouteArgs a, int scratch_bytes) {
  constexpr int NU = V / VEC;               // units of a lane
  constexpr int TPW = 32 / LPT;             // tokens of a warp
  constexpr int NB = 4 * L / LPT;           // block maxima of a lane
  constexpr int CAP = kCap<L>, CPL = CAP / LPT < 1 ? 1 : CAP / LPT;  // candidates of a token, of a lane
  static_assert(NB >= 1 && NB <= V && NB <= L && LPT * NB >= L, "lists grow to L");
  extern __shared__ uint4 warp_smem[];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, sub = lane / LPT, ll = lane % LPT;
  const uint32_t team = (LPT == 32 ? 0xffffffffu : ((1u << LPT) - 1) << (sub * LPT));
  char* mine = reinterpret_cast<char*>(warp_smem) + (size_t)warp * (scratch_bytes + TPW * sizeof(Candidates<L>));
  long long* slow_key = reinterpret_cast<long long*>(mine);
  Near<L>& exact = reinterpret_cast<Near<L>*>(mine)[sub];
  Candidates<L>& cand = reinterpret_cast<Candidates<L>*>(mine + scratch_bytes)[sub];
  const int E = a.E, K = a.K;
  const bool biased = a.sigmoid && (a.bias != nullptr || a.groups > 1);
  pdl_wait();
  pdl_trigger();
  const int64_t t0 = ((int64_t)blockIdx.x * (kFastThreads / 32) + warp) * TPW;
  if (t0 >= a.T) return;
  const int64_t t = t0 + sub;
  const bool token = t < a.T, active = token && (a.mask == nullptr || a.mask[t]);
  const E_* row = logits + (active ? t : 0) * E;
  float v[V];
  load_logits<VEC, LPT>(row, E, ll, active, v);
  if (__any_sync(0xffffffffu, !(check_finite(v) == 0.f) || !active)) {
    bool bad = false;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      bad |= bad_logit(v[i]);
      v[i] = active ? finite_logit(v[i]) : -CUDART_INF_F;
    }
    if (bad) set_status(a.status, MLR_STATUS_VALUE);
  }
  close_past<VEC, LPT>(E, ll, v);

  // softmax over all experts: its divisor
  float all = 0.f;
  if (!a.sigmoid && !a.renormalize) {
    const float most = part_max<LPT>(max_of<0, 1>(v));
#pragma unroll
    for (int i = 0; i < V; ++i) all += v[i] > -CUDART_INF_F ? share_exp(v[i] - most) : 0.f;
    all = part_sum<LPT>(all);
  }
  if (biased) {
#pragma unroll
    for (int j = 0; j < NU; ++j) {
      const int e = (ll + LPT * j) * VEC;
      float b[VEC] = {};
      if (a.bias != nullptr && e < E) {
        if constexpr (VEC == 1) {
          b[0] = __ldg(a.bias + e);
        } else {
#pragma unroll
          for (int i = 0; i < VEC; i += 4) {
            const float4 q = __ldg(reinterpret_cast<const float4*>(a.bias + e + i));
            b[i] = q.x; b[i + 1] = q.y; b[i + 2] = q.z; b[i + 3] = q.w;
          }
        }
      }
#pragma unroll
      for (int i = 0; i < VEC; ++i) {
        const float c = quick_sigmoid(v[j * VEC + i]) + b[i];
        v[j * VEC + i] = v[j * VEC + i] > -CUDART_INF_F && c < CUDART_INF_F ? c : -CUDART_INF_F;
      }
    }
  }
  bool slow = false;  // the same for a token's lanes
  if (a.groups > 1) {
    const int units = E / VEC, per = units / a.groups;  // units of a group
    float2* best2 = reinterpret_cast<float2*>(mine) + sub * units;
#pragma unroll
    for (int j = 0; j < NU; ++j) {
      float b0 = v[j * VEC], b1 = -CUDART_INF_F;
#pragma unroll
      for (int i = 1; i < VEC; ++i) {
        b1 = fmaxf(b1, fminf(b0, v[j * VEC + i]));
        b0 = fmaxf(b0, v[j * VEC + i]);
      }
      if (ll + LPT * j < units) best2[ll + LPT * j] = make_float2(b0, b1);
    }
    __syncwarp();
    float score = -CUDART_INF_F, size = 0.f;  // lane g of the token: group g
    if (ll < a.groups) {
      float b0 = -CUDART_INF_F, b1 = -CUDART_INF_F;
      for (int i = 0; i < per; ++i) {
        const float2 u = best2[ll * per + i];
        b1 = fmaxf(fmaxf(b1, u.y), fminf(b0, u.x));
        b0 = fmaxf(b0, u.x);
      }
      score = a.sigmoid && b1 > -CUDART_INF_F ? b0 + b1 : b0;
      size = b1 > -CUDART_INF_F ? fabsf(b0) + fabsf(b1) : b0 > -CUDART_INF_F ? fabsf(b0) : 0.f;
    }
    __syncwarp();
    int before = 0;
    for (int g = 0; g < a.groups; ++g) {
      const float o = __shfl_sync(0xffffffffu, score, g, LPT);
      before += o > score || (o == score && g < ll);
    }
    bool in = ll < a.groups && before < a.best;
    if (a.sigmoid) {  // two sums of two scores: twice as much as two scores may differ, and the sums' roundings
      const float least = -part_max<LPT>(in && score > -CUDART_INF_F ? -score : -CUDART_INF_F);
      const float out = part_max<LPT>(!in ? score : -CUDART_INF_F);
      // a sum that passes fp32's range may look like an empty group's or like another such sum
      const float widest = part_max<LPT>(size), apart = 2.f * near_score(widest);
      const bool close = !(widest < CUDART_INF_F) || (out > -CUDART_INF_F && !(least - out > apart));
      if (__any_sync(0xffffffffu, close)) {
        bool third = false;
        const long long sum = close && ll < a.groups ? exact_group(a, row, ll, third) : kLowest;
        before = 0;
#pragma unroll 1
        for (int g = 0; g < a.groups; ++g) {
          const long long o = __shfl_sync(0xffffffffu, sum, g, LPT);
          before += o > sum || (o == sum && g < ll);
        }
        if (close) in = ll < a.groups && before < a.best;
        slow = (__ballot_sync(0xffffffffu, third) & team) != 0;
      }
    }
    const uint32_t chosen = (__ballot_sync(0xffffffffu, in) & team) >> (sub * LPT);
#pragma unroll
    for (int j = 0; j < NU; ++j)
      if (ll + LPT * j < units && ((chosen >> ((ll + LPT * j) / per)) & 1) == 0)
#pragma unroll
        for (int i = 0; i < VEC; ++i) v[j * VEC + i] = -CUDART_INF_F;
  }

  // the lower bound: the L-th largest block maximum
  float list[L], other[L];
#pragma unroll
  for (int b = 0; b < NB; ++b) {
    list[b] = v[b];  // of every NB-th logit, so that a block has its share of every group
#pragma unroll
    for (int i = b + NB; i < V; i += 2 * NB)
      list[b] = i + NB < V ? max3(list[b], v[i], v[i + NB < V ? i + NB : i]) : fmaxf(list[b], v[i]);
  }
  sort_desc<NB>(list);
  merge_lists<NB, L, LPT, 1>(list, other);
  const float most = fmaxf(list[0], other[0]);
  float bound = fmaxf(list[0], other[L - 1]);
#pragma unroll
  for (int i = 1; i < L; ++i) bound = fminf(bound, fmaxf(list[i], other[L - 1 - i]));
  const float kth = bound;
  if (biased) bound -= near_score(bound);
  bound = fmaxf(bound, -FLT_MAX);
  if (bound == 0.f) bound = -0.f;  // so that either zero less this is +0

  // the candidates: bit 31 - i of `hit` is logit i's, from the sign of a difference
  uint32_t hit = 0xffffffffu;
#pragma unroll
  for (int i = 0; i < V; i += 2) {
    const float2 d = __fadd2_rn(make_float2(v[i], v[i + 1]), make_float2(-bound, -bound));
    hit = __funnelshift_l(__float_as_uint(d.x), hit, 1);
    hit = __funnelshift_l(__float_as_uint(d.y), hit, 1);
  }
  hit = ~hit << (32 - V);
  int at, n;  // where the lane's candidates go, and how many the token has
  auto count = [&] {
    const int own = __popc(hit);
    at = own;
#pragma unroll
    for (int o = 1; o < LPT; o <<= 1) {
      const int u = __shfl_up_sync(0xffffffffu, at, o, LPT);
      if (ll >= o) at += u;
    }
    n = __shfl_sync(0xffffffffu, at, LPT - 1, LPT);
    at -= own;
  };
  count();
  if (__any_sync(0xffffffffu, n > CAP)) {  // rows of equal logits (of zeros, say, that pad a batch)
    const uint32_t fewer = first_equals<VEC, LPT, V>(row, a.bias, biased, kth, hit, K, ll);
    if (n > CAP) hit = fewer;
    count();
  }
  slow |= n > CAP;
  while (hit != 0 && at < CAP) {
    const int i = __clz(hit);
    hit &= ~(0x80000000u >> i);
    cand.id[at++] = (ll + LPT * (i / VEC)) * VEC + i % VEC;
  }
  int longest = n;  // of the warp's tokens
#pragma unroll
  for (int o = LPT; o < 32; o <<= 1) longest = max(longest, __shfl_xor_sync(0xffffffffu, longest, o));
  longest = min(longest, CAP);
  __syncwarp();
  int id[CPL], rank[CPL];
  float key[CPL], logit[CPL];
#pragma unroll
  for (int c = 0; c < CPL; ++c) {
    id[c] = -1;
    rank[c] = K;
    key[c] = logit[c] = -CUDART_INF_F;
    const int i = ll + c * LPT;
    if (c * LPT >= round_up4(longest)) continue;
    if (i < n) {
      id[c] = cand.id[i];
      key[c] = logit[c] = finite_logit(row + id[c]);
      if (biased) key[c] = quick_sigmoid(logit[c]) + (a.bias != nullptr ? __ldg(a.bias + id[c]) : 0.f);
    }
    if (i < CAP) cand.key[i] = key[c];
  }
  __syncwarp();
  // ranks: those surely above, and whether any other is as near as not to tell
  bool near = false;
#pragma unroll
  for (int c = 0; c < CPL; ++c) {
    if (c * LPT >= longest) continue;
    float above = 0.f, about = 0.f;
    if (biased) {
      const float d = near_score(key[c]), hi = key[c] + d, lo = key[c] - d;
      for (int i = 0; i < longest; i += 4) {
        const float4 q = *reinterpret_cast<const float4*>(&cand.key[i]);
        above += (q.x > hi ? 1.f : 0.f) + (q.y > hi ? 1.f : 0.f) + (q.z > hi ? 1.f : 0.f) + (q.w > hi ? 1.f : 0.f);
        about += (q.x >= lo ? 1.f : 0.f) + (q.y >= lo ? 1.f : 0.f) + (q.z >= lo ? 1.f : 0.f) + (q.w >= lo ? 1.f : 0.f);
      }
    } else {
      for (int i = 0; i < longest; i += 4) {
        const float4 q = *reinterpret_cast<const float4*>(&cand.key[i]);
        above += (q.x > key[c] ? 1.f : 0.f) + (q.y > key[c] ? 1.f : 0.f) + (q.z > key[c] ? 1.f : 0.f) + (q.w > key[c] ? 1.f : 0.f);
      }
    }
    if (id[c] >= 0) rank[c] = (int)above;
    near |= biased && rank[c] < K && about - above != 1.f;
  }
  if (!biased) {
    // equal logits have one rank, the lowest, so that there are more of them in the
    // first K or their sum is less
    const int m = min(n, K);
    int ranks = 0;  // sum, and 2^16 for each
#pragma unroll
    for (int c = 0; c < CPL; ++c) ranks += rank[c] < K ? 65536 + rank[c] : 0;
#pragma unroll
    for (int o = LPT / 2; o > 0; o >>= 1) ranks += __shfl_xor_sync(0xffffffffu, ranks, o);
    near = ranks != 65536 * m + m * (m - 1) / 2;
  }
  const uint32_t unsure = __ballot_sync(0xffffffffu, near);
  if (unsure != 0) {
    const bool again = (unsure & team) != 0;
    const int m = again ? min(n, CAP) : 0;
    if (biased) {
#pragma unroll 1
      for (int i = ll; i < m; i += LPT)
        exact.key[i] = ordered(exact_score(finite_logit(row + cand.id[i]), a.bias, cand.id[i]));
      __syncwarp();
    }
#pragma unroll 1
    for (int i = ll; i < m; i += LPT) {
      const long long k64 = biased ? exact.key[i] : 0;
      const float k32 = cand.key[i];
      const int e = cand.id[i];
      int r = 0;
#pragma unroll 1
      for (int o = 0; o < m; ++o) {
        const bool above = biased ? exact.key[o] > k64 : cand.key[o] > k32;
        const bool same = biased ? exact.key[o] == k64 : cand.key[o] == k32;
        r += above || (same && cand.id[o] < e);
      }
      exact.rank[i] = r;
    }
#pragma unroll
    for (int c = 0; c < CPL; ++c)
      if (again && id[c] >= 0) rank[c] = exact.rank[ll + c * LPT];  // written by this lane
  }

  // weights
  float s[CPL], total = 0.f;
#pragma unroll
  for (int c = 0; c < CPL; ++c) {
    s[c] = 0.f;
    if (id[c] >= 0 && rank[c] < K) {
      s[c] = a.sigmoid ? sigmoid_f(logit[c]) : expf(logit[c] - most);
      total += s[c];
    }
  }
  if (a.renormalize) total = part_sum<LPT>(total);
  else total = a.sigmoid ? 1.f : all;
  const float lift = lift_of(total), inverse = total > 0.f ? 1.f / (total * lift) : 0.f;
  if (token && !slow) {
#pragma unroll
    for (int c = 0; c < CPL; ++c)
      if (id[c] >= 0 && rank[c] < K) {
        a.ids[t * K + rank[c]] = id[c];
        a.weights[t * K + rank[c]] = s[c] * lift * inverse * a.scale;  // the quotient, at most 1, before the scale
      }
    for (int k = n + ll; k < K; k += LPT) {
      a.ids[t * K + k] = -1;
      a.weights[t * K + k] = 0.f;
    }
  }
  uint32_t late = __ballot_sync(0xffffffffu, slow && token);
  while (late != 0) {
    const int o = (__ffs(late) - 1) / LPT;
    __syncwarp();  // what the near candidates' keys and ranks are read from is the keys' place here
    late &= LPT == 32 ? 0u : ~(((1u << (LPT & 31)) - 1) << (o * LPT));
    choose_exactly(a, logits + (t0 + o) * E, t0 + o, slow_key, slow_key + E, lane);
    __syncwarp();
  }
}

template <typename E_, int VEC, int LPT, int V, int L>
int launch_fast(const E_* logits, const RouteArgs& a, cudaStream_t stream) {
  constexpr int TPW = 32 / LPT, WARPS = kFastThreads / 32;
  auto kernel = route_fast_kernel<E_, VEC, LPT, V, L>;
  const int64_t scratch = fast_scratch<L>(a.E, a.groups, VEC, TPW);
  const size_t smem = WARPS * (size_t)(scratch + TPW * sizeof(Candidates<L>));  // below 40 KB
  return launched(launch_pdl(kernel, dim3((unsigned)ceil_div(a.T, WARPS * TPW)), dim3(kFastThreads), smem, stream, logits, a,
                             (int)scratch));
}
template <typename E_, int VEC, int L>
int launch_fast_for(const E_* logits, const RouteArgs& a, cudaStream_t stream) {
  if (a.E <= 64) return launch_fast<E_, VEC, 8, 8, L>(logits, a, stream);
  if (a.E <= 128) return launch_fast<E_, VEC, 8, 16, L>(logits, a, stream);
  if (a.E <= 256) return launch_fast<E_, VEC, 8, 32, L>(logits, a, stream);
  if (a.E <= 512) return launch_fast<E_, VEC, 16, 32, L>(logits, a, stream);
  return launch_fast<E_, VEC, 32, 32, L>(logits, a, stream);
}

template <typename E_>
int run_route(const void* logits, const RouteArgs& a, cudaStream_t stream) {
  const E_* l = static_cast<const E_*>(logits);
  const int lpt = a.E <= 256 ? 8 : a.E <= 512 ? 16 : 32;
  if (a.E <= kPartExperts && a.K <= kFastTopk && a.groups <= lpt) {
    constexpr int VEC = 16 / sizeof(E_);
    const bool whole = a.E % VEC == 0 && a.E / a.groups % VEC == 0 && aligned_to(logits, 16) && aligned_to(a.bias, 16);
    if (whole) return a.K <= 8 ? launch_fast_for<E_, VEC, 8>(l, a, stream) : launch_fast_for<E_, VEC, 16>(l, a, stream);
    return a.K <= 8 ? launch_fast_for<E_, 1, 8>(l, a, stream) : launch_fast_for<E_, 1, 16>(l, a, stream);
  }
  const size_t per = (size_t)(a.E + a.groups) * sizeof(long long);
  const int warps = per <= 8 * 1024 ? kRouteThreads / 32 : 1;
  const int64_t blocks = ceil_div(a.T, warps), most = (int64_t)current_sms() * 16;
  return launched(launch_pdl(route_kernel<E_>, dim3((unsigned)(blocks < most ? blocks : most)), dim3(warps * 32), per * warps,
                             stream, l, a));
}

}  // namespace
}  // namespace mlr

extern "C" int moe_route(const void* logits, const float* bias, const uint8_t* token_mask, int32_t num_tokens,
                         int32_t num_experts, int32_t topk, int32_t num_groups, int32_t topk_groups, int32_t dtype,
                         int32_t scoring, int32_t renormalize, float scale, int32_t* topk_ids, float* topk_weights,
                         int32_t* d_status, void* stream_) {
  using namespace mlr;
  const int code = check_logits(logits, num_tokens, num_experts, topk, dtype, scoring);
  if (code != MLR_OK) return code;
  if (num_groups < 1 || topk_groups < 1 || topk_groups > num_groups || num_experts % num_groups != 0 ||
      (int64_t)topk > (int64_t)topk_groups * (num_experts / num_groups) || (bias != nullptr && scoring != kSigmoid) ||
      !on_word_grid({bias, topk_ids, topk_weights, d_status}))
    return MLR_ERR_INVALID;
  if (num_groups > kMaxGroups) return MLR_ERR_UNSUPPORTED;
  if (num_tokens == 0) return MLR_OK;
  if (topk_ids == nullptr || topk_weights == nullptr) return MLR_ERR_INVALID;
  RouteArgs a{bias, token_mask, num_tokens, num_experts, topk, num_groups, topk_groups, scoring == kSigmoid, renormalize != 0,
              scale, topk_ids, topk_weights, d_status};
  cudaStream_t stream = static_cast<cudaStream_t>(stream_);
  return dtype == MLR_DTYPE_BF16 ? run_route<uint16_t>(logits, a, stream) : run_route<float>(logits, a, stream);
}
