// router.cu -- the router's choice of experts from its logits, the balance loss
// over a batch, and their gradients.
//
// Logits [T, E]; one that is not finite counts as -inf, and its expert is never
// chosen.  An expert's choice score is its logit, or with a bias or (sigmoid)
// groups sigmoid(logit) + bias.  With groups only the experts of the topk_groups
// best groups stand to choice; a group's score is its best choice score (softmax)
// or the sum of its two best (sigmoid).  Ties go to the lowest index.  With s =
// softmax(logits) or sigmoid(logits):
//   w_k = scale s_k [/ sum of the chosen s]
//   loss = E / (K N^2) sum_e c_e sum_t p_te,  p = s [/ its sum over e (sigmoid)]
// for N unmasked tokens and c_e pairs of expert e.  Gradients, with a_e = dloss
// E / (K N^2) c_e and g_k what reaches w_k:
//   softmax  dl_e = p_e (q_e - sum_j p_j q_j), q = a plus g's part
//   sigmoid  dl_e = p_e (1 - s_e) (a_e - sum_j p_j a_j) + g's part
//
// The choice is decided by the real numbers that the scores stand for: where
// 32 bits do not tell two of them apart, they are computed in 64.
#include <math_constants.h>

#include <type_traits>

#include "mlr_profile.cuh"
#include "mlr_rows.cuh"

namespace mlr {
namespace {

constexpr int kMaxRouteExperts = 4096;
constexpr int kMaxRouteTopk = 32;  // a lane per place
constexpr int kMaxGroups = 256;

enum Scoring { kSoftmax = 0, kSigmoid = 1 };

// A logit as fp32, -inf where it is not finite.
template <typename E_>
__device__ __forceinline__ float finite_logit(const E_* p) {
  const float v = row_widen(*p);
  return fabsf(v) < CUDART_INF_F ? v : -CUDART_INF_F;
}
// Whether a logit is one that the caller hears of: NaN or +inf.
__device__ __forceinline__ bool bad_logit(float v) { return !(v < CUDART_INF_F); }
__device__ __forceinline__ float sigmoid_f(float v) { return 1.f / (1.f + expf(-v)); }

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

// The larger of two (score, index) pairs over the warp: the larger score, the
// lower index of equal ones.
__device__ __forceinline__ void warp_best(double& v, int& i) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const double u = __shfl_xor_sync(0xffffffffu, v, o);
    const int k = __shfl_xor_sync(0xffffffffu, i, o);
    if (u > v || (u == v && k < i)) {
      v = u;
      i = k;
    }
  }
}

// The weights of the chosen experts, lane k place k (id -1: none); `most` is the
// largest finite logit of the token (softmax).
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
__device__ void choose_exactly(const RouteArgs& a, const E_* row, int64_t t, double* key, double* group, int lane) {
  const bool logit_key = !a.sigmoid || (a.bias == nullptr && a.groups == 1);
  for (int e = lane; e < a.E; e += 32) {
    const float l = finite_logit(row + e);
    double k = (double)l;
    if (!logit_key && l > -CUDART_INF_F) {
      k = 1.0 / (1.0 + exp(-k)) + (a.bias != nullptr ? (double)__ldg(a.bias + e) : 0.0);
      if (!(k < CUDART_INF)) k = -CUDART_INF;  // a bias that is NaN or +inf
    }
    key[e] = k;
  }
  __syncwarp();
  if (a.groups > 1) {
    const int size = a.E / a.groups;
    for (int g = lane; g < a.groups; g += 32) {
      double b0 = -CUDART_INF, b1 = -CUDART_INF;
      for (int i = 0; i < size; ++i) {
        const double k = key[g * size + i];
        if (k > b0) {
          b1 = b0;
          b0 = k;
        } else if (k > b1) {
          b1 = k;
        }
      }
      group[g] = a.sigmoid && b1 > -CUDART_INF ? b0 + b1 : b0;
    }
    __syncwarp();
    for (int g = lane; g < a.groups; g += 32) {
      int before = 0;
      for (int o = 0; o < a.groups; ++o) before += group[o] > group[g] || (group[o] == group[g] && o < g);
      if (before >= a.best)
        for (int i = 0; i < size; ++i) key[g * size + i] = -CUDART_INF;
    }
    __syncwarp();
  }
  int mine = -1;
  for (int k = 0; k < a.K; ++k) {
    double v = -CUDART_INF;
    int i = INT32_MAX;
    for (int e = lane; e < a.E; e += 32)
      if (key[e] > v) {
        v = key[e];
        i = e;
      }
    warp_best(v, i);
    if (!(v > -CUDART_INF)) break;
    if (lane == k) mine = i;
    if (lane == (i & 31)) key[i] = -CUDART_INF;
    __syncwarp();
  }
  __syncwarp();
  write_choice(a, row, t, mine, lane);
}

constexpr int kRouteThreads = 128;
template <typename E_>
__global__ void __launch_bounds__(kRouteThreads)
route_kernel(const E_* __restrict__ logits, RouteArgs a) {
  extern __shared__ double smem[];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  double* key = smem + (size_t)warp * (a.E + a.groups);
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

// ------------------------------------------------- balance loss, gradients --
// A token is taken by TPT threads (a warp, or for more than 512 experts a block
// of 256), thread i holding experts i, i + TPT, ...
template <int TPT>
__device__ __forceinline__ float team_sum(float v, float* red) {
  v = warp_sum(v);
  if (TPT == 32) return v;
  __syncthreads();
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  v = 0.f;
#pragma unroll
  for (int i = 0; i < TPT / 32; ++i) v += red[i];
  return v;
}
template <int TPT>
__device__ __forceinline__ float team_max(float v, float* red) {
  v = warp_max(v);
  if (TPT == 32) return v;
  __syncthreads();
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  v = red[0];
#pragma unroll
  for (int i = 1; i < TPT / 32; ++i) v = fmaxf(v, red[i]);
  return v;
}

// The shares p of a token's experts and (sigmoid) s, zeros without finite logits.
template <int TPT, int VPL, typename E_>
__device__ __forceinline__ void shares(const E_* row, int E, bool sigmoid, int lt, float* red, float (&p)[VPL], float (&s)[VPL]) {
  float l[VPL];
  float most = -CUDART_INF_F;
#pragma unroll
  for (int j = 0; j < VPL; ++j) {
    const int e = lt + j * TPT;
    l[j] = e < E ? finite_logit(row + e) : -CUDART_INF_F;
    most = fmaxf(most, l[j]);
  }
  float sum = 0.f;
  if (sigmoid) {
#pragma unroll
    for (int j = 0; j < VPL; ++j) sum += s[j] = l[j] > -CUDART_INF_F ? sigmoid_f(l[j]) : 0.f;
  } else {
    most = team_max<TPT>(most, red);
#pragma unroll
    for (int j = 0; j < VPL; ++j) sum += s[j] = l[j] > -CUDART_INF_F ? expf(l[j] - most) : 0.f;
  }
  sum = team_sum<TPT>(sum, red);
  const float inv = sum > 0.f ? 1.f / sum : 0.f;
#pragma unroll
  for (int j = 0; j < VPL; ++j) p[j] = s[j] * inv;
}

constexpr int kBalanceThreads = 256;

// Sums of shares and pairs per expert over the block's tokens: part [blocks][E]
// and count [blocks][E + 1] (the last one: tokens).
template <int TPT, int VPL, typename E_>
__global__ void __launch_bounds__(kBalanceThreads)
balance_kernel(const E_* __restrict__ logits, const int32_t* __restrict__ ids, const uint8_t* __restrict__ mask, int T, int E,
               int K, bool sigmoid, float* __restrict__ part, int32_t* __restrict__ count, int32_t* status) {
  extern __shared__ int hist[];  // [E + 1] pairs, then float [teams][E] shares
  __shared__ float red[kBalanceThreads / 32];
  constexpr int TEAMS = kBalanceThreads / TPT;
  float* sums = reinterpret_cast<float*>(hist + E + 1);
  const int team = threadIdx.x / TPT, lt = threadIdx.x - team * TPT;
  for (int e = threadIdx.x; e <= E; e += kBalanceThreads) hist[e] = 0;
  __syncthreads();
  pdl_wait();
  pdl_trigger();
  float acc[VPL] = {};
  int tokens = 0;
  for (int64_t t = (int64_t)blockIdx.x * TEAMS + team; t < T; t += (int64_t)gridDim.x * TEAMS) {
    if (mask != nullptr && !mask[t]) continue;  // the same for the whole team
    ++tokens;
    float p[VPL], s[VPL];
    shares<TPT, VPL>(logits + t * E, E, sigmoid, lt, red, p, s);
#pragma unroll
    for (int j = 0; j < VPL; ++j) acc[j] += p[j];
    for (int k = lt; k < K; k += TPT) {
      const int id = __ldg(ids + t * K + k);
      if (id >= 0 && id < E) atomicAdd(&hist[id], 1);
      else if (id != -1) set_status(status, MLR_STATUS_INDEX);
    }
  }
  if (lt == 0) atomicAdd(&hist[E], tokens);
#pragma unroll
  for (int j = 0; j < VPL; ++j)
    if (lt + j * TPT < E) sums[team * E + lt + j * TPT] = acc[j];
  __syncthreads();
  for (int e = threadIdx.x; e <= E; e += kBalanceThreads) {
    count[(int64_t)blockIdx.x * (E + 1) + e] = hist[e];
    if (e == E) continue;
    float v = 0.f;
#pragma unroll
    for (int i = 0; i < TEAMS; ++i) v += sums[i * E + e];
    part[(int64_t)blockIdx.x * E + e] = v;
  }
}

constexpr int kTotalThreads = 1024;
// The blocks' sums added in order, in one block: counts, and the loss.
__global__ void __launch_bounds__(kTotalThreads)
balance_total_kernel(const float* __restrict__ part, const int32_t* __restrict__ count, int blocks, int E, int K,
                     float* __restrict__ loss, int32_t* __restrict__ counts) {
  __shared__ double red[kTotalThreads / 32];
  __shared__ int tokens;
  pdl_wait();
  pdl_trigger();
  double v = 0.0;
  for (int e = threadIdx.x; e <= E; e += kTotalThreads) {
    int c = 0;
    double s = 0.0;
    for (int b = 0; b < blocks; ++b) {
      c += count[(int64_t)b * (E + 1) + e];
      if (e < E) s += part[(int64_t)b * E + e];
    }
    counts[e] = c;
    if (e == E) tokens = c;
    else v += s * c;
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  if (threadIdx.x == 0) {
    v = 0.0;
    for (int i = 0; i < kTotalThreads / 32; ++i) v += red[i];
    const double n = tokens > 0 ? tokens : 1;
    *loss = (float)(v * E / (K * n * n));
  }
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

// Gradient of the logits.  The part that comes by the weights is put together by
// the token's first warp (lane k place k) in a row of shared memory, from where
// the experts' threads take it.
template <int TPT, int VPL, typename E_>
__global__ void __launch_bounds__(kBalanceThreads)
route_backward_kernel(const E_* __restrict__ logits, GradArgs a, E_* __restrict__ d_logits, int32_t* status) {
  extern __shared__ float rows[];  // [teams][E]
  __shared__ float red[kBalanceThreads / 32];
  constexpr int TEAMS = kBalanceThreads / TPT;
  const int team = threadIdx.x / TPT, lt = threadIdx.x - team * TPT;
  const int E = a.E, K = a.K;
  float* row_s = rows + team * E;
  pdl_wait();
  pdl_trigger();
  float coef[VPL] = {};
  if (a.counts != nullptr) {
    const double n = max(1, __ldg(a.counts + E));
    const double f = (double)__ldg(a.d_loss) * E / (K * n * n);
#pragma unroll
    for (int j = 0; j < VPL; ++j) {
      const int e = lt + j * TPT;
      if (e < E) coef[j] = (float)(f * __ldg(a.counts + e));
    }
  }
  const bool by_weights = a.d_weights != nullptr;
  for (int64_t t = (int64_t)blockIdx.x * TEAMS + team; t < a.T; t += (int64_t)gridDim.x * TEAMS) {
    const E_* row = logits + t * E;
    const bool masked = a.mask != nullptr && !a.mask[t];  // the same for the whole team
    float dot = 0.f;  // sum of g w, which softmax over all experts takes from every one of them
    float d[VPL] = {};
    float p[VPL], s[VPL];
    if (!masked && (a.counts != nullptr || (by_weights && !a.sigmoid && !a.renormalize)))
      shares<TPT, VPL>(row, E, a.sigmoid, lt, red, p, s);
    else
#pragma unroll
      for (int j = 0; j < VPL; ++j) p[j] = s[j] = 0.f;
    if (by_weights && !masked) {
#pragma unroll
      for (int j = 0; j < VPL; ++j)
        if (lt + j * TPT < E) row_s[lt + j * TPT] = 0.f;
      if (TPT > 32) __syncthreads();
      else __syncwarp();
      if (lt < 32) {
        int id = lt < K ? __ldg(a.ids + t * K + lt) : -1;
        if (id < -1 || id >= E) {
          set_status(status, MLR_STATUS_INDEX);
          id = -1;
        }
        const float l = id >= 0 ? finite_logit(row + id) : -CUDART_INF_F;
        const bool in = l > -CUDART_INF_F;
        const float g = in ? a.scale * __ldg(a.d_weights + t * K + lt) : 0.f;
        float dl;
        if (a.sigmoid) {
          const float si = in ? sigmoid_f(l) : 0.f;
          if (a.renormalize) {
            const float total = warp_sum(si);
            const float mean = warp_sum(g * si);
            dl = total > 0.f ? (g - mean / total) / total * si * (1.f - si) : 0.f;
          } else {
            dl = g * si * (1.f - si);
          }
        } else if (a.renormalize) {
          const float most = warp_max(l);
          const float si = in ? expf(l - most) : 0.f;
          const float total = warp_sum(si);
          const float mean = warp_sum(g * si);
          dl = total > 0.f ? si / total * (g - mean / total) : 0.f;
        } else {
          dl = g;  // times p below
        }
        // an id that a token holds twice: the first place adds the others' in order
        const uint32_t same = __match_any_sync(0xffffffffu, id);
        float all = dl;
        if (__any_sync(0xffffffffu, id >= 0 && (same & (same - 1)) != 0))
          for (int k = 1; k < K; ++k) {
            const float o = __shfl_sync(0xffffffffu, dl, k);
            if (k > lt && ((same >> k) & 1)) all += o;
          }
        if (id >= 0 && lt == __ffs(same) - 1) row_s[id] = all;
      }
      if (TPT > 32) __syncthreads();
      else __syncwarp();
#pragma unroll
      for (int j = 0; j < VPL; ++j)
        if (lt + j * TPT < E) d[j] = row_s[lt + j * TPT];
    }
    // q: what multiplies the share; d: added as it is
#pragma unroll
    for (int j = 0; j < VPL; ++j) {
      float q = coef[j];
      if (!a.sigmoid && !a.renormalize) q += d[j];
      dot = fmaf(p[j], q, dot);
    }
    dot = team_sum<TPT>(dot, red);
#pragma unroll
    for (int j = 0; j < VPL; ++j) {
      const int e = lt + j * TPT;
      if (e >= E) continue;
      float v;
      if (a.sigmoid) v = p[j] * (1.f - s[j]) * (coef[j] - dot) + d[j];
      else if (a.renormalize) v = p[j] * (coef[j] - dot) + d[j];
      else v = p[j] * (coef[j] + d[j] - dot);
      row_narrow(v, d_logits[t * E + e]);
    }
    if (TPT == 32) __syncwarp();
  }
}

int launched(cudaError_t err) {
  if (err != cudaSuccess) {
    (void)cudaGetLastError();  // not left for the next call to find
    return MLR_ERR_CUDA;
  }
  note_launch();
  return MLR_OK;
}
int check_logits(const void* logits, int32_t T, int32_t E, int32_t K, int32_t dtype, int32_t scoring) {
  if (T < 0 || E < 1 || K < 1 || (dtype != MLR_DTYPE_BF16 && dtype != MLR_DTYPE_F32) ||
      (scoring != kSoftmax && scoring != kSigmoid))
    return MLR_ERR_INVALID;
  if (E > kMaxRouteExperts || K > kMaxRouteTopk || (int64_t)T * K >= INT32_MAX) return MLR_ERR_UNSUPPORTED;
  if (T > 0 && (logits == nullptr || !aligned_to(logits, dtype == MLR_DTYPE_BF16 ? 2 : 4))) return MLR_ERR_INVALID;
  return MLR_OK;
}

int64_t balance_blocks(int32_t T, int32_t E) {
  const int64_t want = ceil_div(T, E <= 512 ? kBalanceThreads / 32 : 1), most = 2 * (int64_t)current_sms();
  return want < 1 ? 1 : want < most ? want : most;
}

// f<TPT, VPL>() for E experts.
template <typename F>
int by_experts(int E, F f) {
  using std::integral_constant;
  constexpr integral_constant<int, 32> w{};
  constexpr integral_constant<int, 256> b{};
  if (E <= 32) return f(w, integral_constant<int, 1>{});
  if (E <= 64) return f(w, integral_constant<int, 2>{});
  if (E <= 128) return f(w, integral_constant<int, 4>{});
  if (E <= 256) return f(w, integral_constant<int, 8>{});
  if (E <= 512) return f(w, integral_constant<int, 16>{});
  if (E <= 1024) return f(b, integral_constant<int, 4>{});
  if (E <= 2048) return f(b, integral_constant<int, 8>{});
  return f(b, integral_constant<int, 16>{});
}

template <typename E_>
int run_route(const void* logits, const RouteArgs& a, cudaStream_t stream) {
  const size_t per = (size_t)(a.E + a.groups) * sizeof(double);
  const int warps = per <= 8 * 1024 ? kRouteThreads / 32 : 1;
  const int64_t blocks = ceil_div(a.T, warps), most = (int64_t)current_sms() * 16;
  return launched(launch_pdl(route_kernel<E_>, dim3((unsigned)(blocks < most ? blocks : most)), dim3(warps * 32), per * warps,
                             stream, static_cast<const E_*>(logits), a));
}

template <typename E_>
int run_balance(const void* logits, const int32_t* ids, const uint8_t* mask, int T, int E, int K, bool sigmoid, float* part,
                int32_t* count, int32_t* status, cudaStream_t stream) {
  const unsigned blocks = (unsigned)balance_blocks(T, E);
  return by_experts(E, [&](auto tpt, auto vpl) {
    auto kernel = balance_kernel<tpt.value, vpl.value, E_>;
    const size_t smem = (size_t)(E + 1) * 4 + (size_t)(kBalanceThreads / tpt.value) * E * 4;
    return launched(launch_pdl(kernel, dim3(blocks), dim3(kBalanceThreads), smem, stream, static_cast<const E_*>(logits), ids,
                               mask, T, E, K, sigmoid, part, count, status));
  });
}

template <typename E_>
int run_backward(const void* logits, const GradArgs& a, void* d_logits, int32_t* status, cudaStream_t stream) {
  return by_experts(a.E, [&](auto tpt, auto vpl) {
    auto kernel = route_backward_kernel<tpt.value, vpl.value, E_>;
    const int teams = kBalanceThreads / tpt.value;
    const int64_t want = ceil_div(a.T, teams), most = 8 * (int64_t)current_sms();
    return launched(launch_pdl(kernel, dim3((unsigned)(want < most ? want : most)), dim3(kBalanceThreads), (size_t)teams * a.E * 4,
                               stream, static_cast<const E_*>(logits), a, static_cast<E_*>(d_logits), status));
  });
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
      !aligned_to(bias, 4))
    return MLR_ERR_INVALID;
  if (num_groups > kMaxGroups) return MLR_ERR_UNSUPPORTED;
  if (num_tokens == 0) return MLR_OK;
  if (topk_ids == nullptr || topk_weights == nullptr) return MLR_ERR_INVALID;
  RouteArgs a{bias, token_mask, num_tokens, num_experts, topk, num_groups, topk_groups, scoring == kSigmoid, renormalize != 0,
              scale, topk_ids, topk_weights, d_status};
  cudaStream_t stream = static_cast<cudaStream_t>(stream_);
  return dtype == MLR_DTYPE_BF16 ? run_route<uint16_t>(logits, a, stream) : run_route<float>(logits, a, stream);
}

extern "C" size_t moe_balance_loss_workspace_bytes(int32_t num_tokens, int32_t num_experts) {
  using namespace mlr;
  if (num_tokens < 0 || num_experts < 1 || num_experts > kMaxRouteExperts) return 0;
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
  if (workspace == nullptr || ws_bytes < moe_balance_loss_workspace_bytes(num_tokens, num_experts)) return MLR_ERR_CAPACITY;
  if (!aligned_to(workspace, 256)) return MLR_ERR_INVALID;
  const int blocks = (int)balance_blocks(num_tokens, num_experts);
  float* part = static_cast<float*>(workspace);
  int32_t* count = reinterpret_cast<int32_t*>(part + (int64_t)blocks * num_experts);
  auto run = dtype == MLR_DTYPE_BF16 ? run_balance<uint16_t> : run_balance<float>;
  const int c = run(logits, topk_ids, token_mask, num_tokens, num_experts, topk, scoring == kSigmoid, part, count, d_status, stream);
  if (c != MLR_OK) return c;
  return launched(launch_pdl(balance_total_kernel, dim3(1), dim3(kTotalThreads), 0, stream, (const float*)part,
                             (const int32_t*)count, blocks, (int)num_experts, (int)topk, loss, counts));
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
  if (d_logits == nullptr || !aligned_to(d_logits, dtype == MLR_DTYPE_BF16 ? 2 : 4) || (d_weights != nullptr && topk_ids == nullptr))
    return MLR_ERR_INVALID;
  const GradArgs a{topk_ids, d_weights, counts, d_loss, token_mask, num_tokens, num_experts, topk, scoring == kSigmoid,
                   renormalize != 0, scale};
  return dtype == MLR_DTYPE_BF16 ? run_backward<uint16_t>(logits, a, d_logits, d_status, stream)
                                 : run_backward<float>(logits, a, d_logits, d_status, stream);
}
