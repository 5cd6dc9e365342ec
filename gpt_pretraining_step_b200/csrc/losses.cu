// Losses of fine-tuning on logits rows: the clipped policy loss with a KL
// term, and the preference loss over paired log ratios, each with its
// gradient with respect to the logits.
//
// Both need, per row of V logits x, the log-probability of the target y,
// log p_y = (x_y - m) - log sum_j exp(x_j - m), m = max_j x_j, and write
// dx_j = g (1[j = y] - p_j) with a row factor g that the loss defines.  All
// of it is bound by memory: one read and one write of the logits.
#include <math.h>

#include <algorithm>
#include <type_traits>

#include "common.cuh"
#include "losses.cuh"

namespace gpt {

namespace {

using bf16 = __nv_bfloat16;

// A row is worked on by G threads (a whole block), kVecs 16-byte vectors of a
// thread at a time: all loads of a batch are issued before the first value
// is used, so that a block keeps up to 64 KB in flight.  A row of one batch
// stays in the registers between its two passes; a longer one is read again,
// from L2.
constexpr int kVecs = 8;

// log2(e) in two parts: with one, exp(d) is off by 1.3e-8 |d| in the same
// direction for every value, which sums over a sequence's positions.
constexpr float kLog2e = 1.44269502f, kLog2eLow = 1.92596303e-8f;

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float exp_sum(float d) { return ex2(fmaf(d, kLog2e, d * kLog2eLow)); }

// 16 bytes of a row: 8 bf16 or 4 fp32 values
template <typename T>
struct Vec {
  static constexpr int n = 16 / sizeof(T);
};
template <typename T>
__device__ __forceinline__ void unpack(const uint4& w, float (&v)[Vec<T>::n]) {
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (sizeof(T) == 2) {
      v[2 * i] = bf16_lo(u[i]);
      v[2 * i + 1] = bf16_hi(u[i]);
    } else {
      v[i] = __uint_as_float(u[i]);
    }
  }
}
template <typename T>
__device__ __forceinline__ uint4 pack(const float (&v)[Vec<T>::n]) {
  uint32_t u[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (sizeof(T) == 2) u[i] = pack_bf16x2(v[2 * i], v[2 * i + 1]);
    else u[i] = __float_as_uint(v[i]);
  }
  return make_uint4(u[0], u[1], u[2], u[3]);
}
__device__ __forceinline__ float to_f(bf16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float to_f(float x) { return x; }
__device__ __forceinline__ void from_f(bf16* p, float x) { *p = __float2bfloat16_rn(x); }
__device__ __forceinline__ void from_f(float* p, float x) { *p = x; }

// A row in three parts: `head` values before the first 16-byte boundary,
// `vecs` 16-byte vectors, and a tail.
template <typename T>
struct RowParts {
  int head, vecs;
  __device__ RowParts(const T* x, int V) {
    const int off = static_cast<int>(reinterpret_cast<uintptr_t>(x) & 15) / static_cast<int>(sizeof(T));
    head = min(V, off ? Vec<T>::n - off : 0);
    vecs = (V - head) / Vec<T>::n;
  }
};

// Running maximum m and sum s of exp(x - m).  A maximum of -inf (only masked
// values so far) subtracts 0, so that they add exp(-inf) = 0.
struct Softmax {
  float m = -INFINITY, s = 0.f;
  __device__ __forceinline__ static float base(float m) { return m == -INFINITY ? 0.f : m; }
  __device__ __forceinline__ void raise(float to) {
    if (to > m) {
      s *= exp_sum(m - to);
      m = to;
    }
  }
  __device__ __forceinline__ void add(float x) {
    raise(x);
    s += exp_sum(x - base(m));
  }
  __device__ __forceinline__ void merge(float m2, float s2) {
    const float t = fmaxf(m, m2), b = base(t);
    s = s * exp_sum(m - b) + s2 * exp_sum(m2 - b);
    m = t;
  }
};

// The thread's share of a batch: vectors first + threadIdx.x + G k.
template <int G>
__device__ __forceinline__ void load_batch(const uint4* __restrict__ xv, int first, int vecs, uint4 (&w)[kVecs]) {
#pragma unroll
  for (int k = 0; k < kVecs; ++k) {
    const int i = first + k * G + static_cast<int>(threadIdx.x);
    if (i < vecs) w[k] = __ldg(xv + i);
  }
}

// m and s over a whole row, for every thread of the block.  With one batch
// (vecs <= G kVecs) w keeps the row.
template <typename T, int G>
__device__ __forceinline__ Softmax row_softmax(const T* __restrict__ x, int V, const RowParts<T>& part,
                                               uint4 (&w)[kVecs], float2* red) {
  Softmax a;
  const int tid = threadIdx.x;
  const uint4* xv = reinterpret_cast<const uint4*>(x + part.head);
  const int tail = part.head + part.vecs * Vec<T>::n + tid;
  for (int first = 0; first < part.vecs; first += G * kVecs) {
    load_batch<G>(xv, first, part.vecs, w);
    float t = -INFINITY;
#pragma unroll
    for (int k = 0; k < kVecs; ++k) {
      if (first + k * G + tid < part.vecs) {
        float v[Vec<T>::n];
        unpack<T>(w[k], v);
#pragma unroll
        for (int e = 0; e < Vec<T>::n; ++e) t = fmaxf(t, v[e]);
      }
    }
    a.raise(t);
    const float b = Softmax::base(a.m);
#pragma unroll
    for (int k = 0; k < kVecs; ++k) {
      if (first + k * G + tid < part.vecs) {
        float v[Vec<T>::n];
        unpack<T>(w[k], v);
#pragma unroll
        for (int e = 0; e < Vec<T>::n; ++e) a.s += exp_sum(v[e] - b);
      }
    }
  }
  if (tid < part.head) a.add(to_f(x[tid]));
  if (tail < V) a.add(to_f(x[tail]));
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
    a.merge(__shfl_xor_sync(0xffffffffu, a.m, o), __shfl_xor_sync(0xffffffffu, a.s, o));
  if constexpr (G > 32) {
    if (lane_id() == 0) red[warp_id()] = make_float2(a.m, a.s);
    __syncthreads();
    const float2 q = red[lane_id() & (G / 32 - 1)];
    a.m = q.x;
    a.s = q.y;
#pragma unroll
    for (int o = G / 64; o > 0; o >>= 1)
      a.merge(__shfl_xor_sync(0xffffffffu, a.m, o), __shfl_xor_sync(0xffffffffu, a.s, o));
  }
  return a;
}

// dx = g (1[j = y] - p), p = exp(x - m) / s; d may be x.  kHeld: w holds the
// row (one batch), otherwise it is read again.
template <typename T, int G>
__device__ __forceinline__ void row_gradient(const T* x, T* d, int V, const RowParts<T>& part, bool held,
                                             uint4 (&w)[kVecs], int y, float g, float m, float s) {
  const float b = Softmax::base(m), f = -g / s;
  const int tid = threadIdx.x;
  // the target's own value, after which no thread may have written it in place
  auto value = [&](float v) { return f * ex2((v - b) * kLog2e); };
  const uint4* xv = reinterpret_cast<const uint4*>(x + part.head);
  const bool same = ((reinterpret_cast<uintptr_t>(x) ^ reinterpret_cast<uintptr_t>(d)) & 15) == 0;
  for (int first = 0; first < part.vecs; first += G * kVecs) {
    if (!held) load_batch<G>(xv, first, part.vecs, w);
#pragma unroll
    for (int k = 0; k < kVecs; ++k) {
      const int i = first + k * G + tid;
      if (i < part.vecs) {
        float v[Vec<T>::n];
        unpack<T>(w[k], v);
        const int j0 = part.head + i * Vec<T>::n;
#pragma unroll
        for (int e = 0; e < Vec<T>::n; ++e) v[e] = value(v[e]);
        if (static_cast<unsigned>(y - j0) < static_cast<unsigned>(Vec<T>::n)) {
#pragma unroll
          for (int e = 0; e < Vec<T>::n; ++e) v[e] += j0 + e == y ? g : 0.f;
        }
        if (same) {
          *reinterpret_cast<uint4*>(d + j0) = pack<T>(v);
        } else {
#pragma unroll
          for (int e = 0; e < Vec<T>::n; ++e) from_f(d + j0 + e, v[e]);
        }
      }
    }
  }
  auto one = [&](int j) { from_f(d + j, value(to_f(x[j])) + (j == y ? g : 0.f)); };
  if (tid < part.head) one(tid);
  const int tail = part.head + part.vecs * Vec<T>::n + tid;
  if (tail < V) one(tail);
}

template <typename T, int G>
__device__ __forceinline__ void row_zero(T* d, int V) {
  const RowParts<T> part(d, V);
  if (static_cast<int>(threadIdx.x) < part.head) from_f(d + threadIdx.x, 0.f);
  for (int i = threadIdx.x; i < part.vecs; i += G) reinterpret_cast<uint4*>(d + part.head)[i] = make_uint4(0, 0, 0, 0);
  const int tail = part.head + part.vecs * Vec<T>::n + threadIdx.x;
  if (tail < V) from_f(d + tail, 0.f);
}

// The target of row r if it is counted, else -1; ids that are neither are latched.
__device__ __forceinline__ int row_target(const LossRows& R, int r, int* err) {
  const int y = R.targets[r];
  if (y < -1 || y >= R.V) {
    if (threadIdx.x == 0 && err) atomicOr(err, ERRF_TOKEN_RANGE);
    return -1;
  }
  return y;
}

// log p_y from the row's statistics, in 64 bits (one thread's work): its sum
// over a sequence is compared with sums of nearly the same size.
__device__ __forceinline__ double target_logp(float x, const Softmax& a) {
  return static_cast<double>(x) - Softmax::base(a.m) - log(static_cast<double>(a.s));
}

// Calls f with the threads a row of this many bytes is given: one batch where
// it fits (512 threads at most; more would leave one block on an SM).
template <typename F>
void with_row_threads(long long row_bytes, F f) {
  if (row_bytes <= 32 * kVecs * 16) f(std::integral_constant<int, 32>());
  else if (row_bytes <= 128 * kVecs * 16) f(std::integral_constant<int, 128>());
  else f(std::integral_constant<int, 512>());
}

// ------------------------------------------------------------ policy loss
//
// Per counted token: r = exp(lp - old), the surrogate -min(r A, clip(r, 1 -
// low, 1 + high) A), and c k with k = exp(d) - d - 1, d = ref - lp.  With
// dlp the derivative by lp, -A r where the unclipped product is the smaller
// one (at a border both are) and 0 elsewhere, plus c (1 - exp(d)), the row
// factor is g = w dlp.  The scalars of a row are computed in 64 bits: k loses
// half its digits for small d in 32, and it is one thread's work.
struct PolicyRow {
  float g;
  float4 term;   // w times: loss, surrogate, k, clipped
};
__device__ __forceinline__ PolicyRow policy_row(const PolicyArgs& a, int r, double lp, float w32) {
  const double w = w32, adv = a.advantage[r];
  const double ratio = a.old_logp ? exp(lp - a.old_logp[r]) : 1.0;
  const double lo = 1.0 - a.clip_low, hi = 1.0 + a.clip_high;
  const bool cut = adv >= 0.0 ? ratio > hi : ratio < lo;
  const double used = cut ? (adv >= 0.0 ? hi : lo) : ratio;
  double dlp = cut ? 0.0 : -adv * ratio, k = 0.0;
  if (a.ref_logp) {
    const double d = a.ref_logp[r] - lp, e = expm1(d);
    k = e - d;
    dlp -= a.kl_coef * e;
  }
  PolicyRow p;
  p.g = static_cast<float>(w * dlp);
  p.term = make_float4(static_cast<float>(w * (a.kl_coef * k - adv * used)), static_cast<float>(w * (-adv * used)),
                       static_cast<float>(w * k), cut ? w32 : 0.f);
  return p;
}

template <typename T, int G>
__global__ void __launch_bounds__(G, 1024 / G)
    policy_row_kernel(const LossRows R, const PolicyArgs a, float4* __restrict__ terms, int* err) {
  __shared__ float2 red[G / 32];
  __shared__ float gs;
  const int r = blockIdx.x;
  const T* x = static_cast<const T*>(R.logits) + r * R.ld;
  T* d = R.dlogits ? static_cast<T*>(R.dlogits) + r * R.ld_d : nullptr;
  const float wt = a.weight[r];
  const int y = row_target(R, r, err);
  if (y < 0 || wt == 0.f) {
    if (threadIdx.x == 0) {
      a.logp[r] = 0.f;
      terms[r] = make_float4(0.f, 0.f, 0.f, 0.f);
    }
    if (d) row_zero<T, G>(d, R.V);
    return;
  }
  uint4 w[kVecs];
  const RowParts<T> part(x, R.V);
  const float xy = threadIdx.x == 0 ? to_f(x[y]) : 0.f;
  const Softmax sm = row_softmax<T, G>(x, R.V, part, w, red);
  if (threadIdx.x == 0) {
    const double lp = target_logp(xy, sm);
    const PolicyRow p = policy_row(a, r, lp, wt);
    a.logp[r] = static_cast<float>(lp);
    terms[r] = p.term;
    gs = p.g;
  }
  __syncthreads();
  if (d) row_gradient<T, G>(x, d, R.V, part, part.vecs <= G * kVecs, w, y, gs, sm.m, sm.s);
}

// stats = sums of the rows' terms, in 64 bits and a fixed order
__global__ void __launch_bounds__(1024) policy_sum_kernel(const float4* __restrict__ terms, int M, float* stats) {
  __shared__ double red[4][32];
  double s[4] = {0.0, 0.0, 0.0, 0.0};
  for (int i = threadIdx.x; i < M; i += 1024) {
    const float4 t = terms[i];
    s[0] += t.x;
    s[1] += t.y;
    s[2] += t.z;
    s[3] += t.w;
  }
#pragma unroll
  for (int k = 0; k < 4; ++k) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s[k] += __shfl_xor_sync(0xffffffffu, s[k], o);
    if (lane_id() == 0) red[k][warp_id()] = s[k];
  }
  __syncthreads();
  if (threadIdx.x < 4) {
    double t = 0.0;
    for (int w = 0; w < 32; ++w) t += red[threadIdx.x][w];
    stats[threadIdx.x] = static_cast<float>(t);
  }
}

// -------------------------------------------------------- preference loss
//
// Sequences 2 i and 2 i + 1 are the chosen and the rejected answer of pair i;
// L_s = sum of lp over the counted positions of s, z_i = beta ((L_2i - R_2i)
// - (L_2i+1 - R_2i+1)) and the loss is the mean over the pairs of
// -(1 - e) log sigmoid(z) - e log sigmoid(-z).  Its derivative by L_2i is
// beta / pairs (e sigmoid(z) - (1 - e) sigmoid(-z)), by L_2i+1 the negative:
// the row factor g of every counted position of the sequence.
// L, R and z are sums and differences of large numbers: 64 bits.

// Whether the offsets start at 0, do not decrease and end within M rows; the
// rows they cover.
__device__ __forceinline__ int covered_rows(const PreferenceArgs& a, int M, int* err) {
  const int n = 2 * a.n_pairs;
  int bad = a.cu[0] != 0 || a.cu[n] > M;
  for (int i = threadIdx.x; i < n; i += blockDim.x) bad |= a.cu[i + 1] < a.cu[i];
  bad = __syncthreads_or(bad);
  if (bad && blockIdx.x == 0 && threadIdx.x == 0 && err) atomicOr(err, ERRF_SEQUENCE);
  return bad ? -1 : a.cu[n];
}

template <typename T, int G>
__global__ void __launch_bounds__(G, 1024 / G)
    preference_logp_kernel(const LossRows R, const PreferenceArgs a, float2* __restrict__ ms, double* __restrict__ lps,
                           int* err) {
  __shared__ float2 red[G / 32];
  const int rows = covered_rows(a, R.M, err);
  const int r = blockIdx.x;
  if (r >= rows) return;
  const T* x = static_cast<const T*>(R.logits) + r * R.ld;
  const int y = row_target(R, r, err);
  if (y < 0) {
    if (threadIdx.x == 0) {
      a.logp[r] = 0.f;
      lps[r] = 0.0;
    }
    return;
  }
  uint4 w[kVecs];
  const RowParts<T> part(x, R.V);
  const float xy = threadIdx.x == 0 ? to_f(x[y]) : 0.f;
  const Softmax sm = row_softmax<T, G>(x, R.V, part, w, red);
  if (threadIdx.x == 0) {
    const double lp = target_logp(xy, sm);
    ms[r] = make_float2(sm.m, sm.s);
    a.logp[r] = static_cast<float>(lp);
    lps[r] = lp;
  }
}

// The sums, margins, loss and row factors (one per sequence); one block.
__global__ void __launch_bounds__(1024)
    preference_pair_kernel(const LossRows R, const PreferenceArgs a, const double* __restrict__ lps,
                           double* __restrict__ sums, float* __restrict__ g) {
  __shared__ double red[32];
  if (covered_rows(a, R.M, nullptr) < 0) return;
  const int n = 2 * a.n_pairs;
  for (int q = warp_id(); q < n; q += 32) {
    double s = 0.0;
    for (int r = a.cu[q] + lane_id(); r < a.cu[q + 1]; r += 32) s += lps[r];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    if (lane_id() == 0) {
      sums[q] = s;
      a.seq_logp[q] = static_cast<float>(s);
    }
  }
  __syncthreads();
  double loss = 0.0;
  for (int i = threadIdx.x; i < a.n_pairs; i += 1024) {
    const double ref = a.ref_logp ? static_cast<double>(a.ref_logp[2 * i]) - a.ref_logp[2 * i + 1] : 0.0;
    const double z = a.beta * (sums[2 * i] - sums[2 * i + 1] - ref);
    // sigmoid(-|z|), and log sigmoid(+-z) = min(+-z, 0) - log(1 + exp(-|z|))
    const double t = exp(-fabs(z)), soft = log1p(t), less = t / (1.0 + t);
    const double sig_pos = z >= 0.0 ? 1.0 - less : less, sig_neg = z >= 0.0 ? less : 1.0 - less;
    loss += (1.0 - a.smoothing) * (soft + fmax(-z, 0.0)) + a.smoothing * (soft + fmax(z, 0.0));
    const double dz = a.beta / a.n_pairs * (a.smoothing * sig_pos - (1.0 - a.smoothing) * sig_neg);
    a.margin[i] = static_cast<float>(z);
    g[2 * i] = static_cast<float>(dz);
    g[2 * i + 1] = static_cast<float>(-dz);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) loss += __shfl_xor_sync(0xffffffffu, loss, o);
  if (lane_id() == 0) red[warp_id()] = loss;
  __syncthreads();
  if (threadIdx.x == 0) {
    double t = 0.0;
    for (int w = 0; w < 32; ++w) t += red[w];
    *a.loss = static_cast<float>(t / a.n_pairs);
  }
}

// The sequence that holds row r: the last one that starts at or before it.
__device__ __forceinline__ int row_sequence(const int* __restrict__ cu, int n, int r) {
  int l = 0, h = n - 1;
  while (l < h) {
    const int m = (l + h + 1) >> 1;
    if (__ldg(cu + m) <= r) l = m;
    else h = m - 1;
  }
  return l;
}

template <typename T, int G>
__global__ void __launch_bounds__(G, 1024 / G)
    preference_grad_kernel(const LossRows R, const PreferenceArgs a, const float2* __restrict__ ms,
                           const float* __restrict__ g) {
  const int r = blockIdx.x;
  if (r >= covered_rows(a, R.M, nullptr)) return;
  T* d = static_cast<T*>(R.dlogits) + r * R.ld_d;
  const int y = row_target(R, r, nullptr);
  if (y < 0) {
    row_zero<T, G>(d, R.V);
    return;
  }
  uint4 w[kVecs];
  const T* x = static_cast<const T*>(R.logits) + r * R.ld;
  const float2 q = ms[r];
  row_gradient<T, G>(x, d, R.V, RowParts<T>(x, R.V), false, w, y, g[row_sequence(a.cu, 2 * a.n_pairs, r)], q.x, q.y);
}

constexpr size_t al256(size_t x) { return (x + 255) / 256 * 256; }

}  // namespace

size_t policy_loss_scratch(int M) { return al256(static_cast<size_t>(M) * sizeof(float4)) + 256; }

size_t preference_loss_scratch(int M, int n_pairs) {
  return al256(static_cast<size_t>(M) * sizeof(float2)) + al256(static_cast<size_t>(M) * sizeof(double)) +
         al256(2 * static_cast<size_t>(n_pairs) * sizeof(double)) +
         al256(2 * static_cast<size_t>(n_pairs) * sizeof(float));
}

template <typename T>
static void policy_rows(const LossRows& r, const PolicyArgs& a, float4* terms, int* err, cudaStream_t s) {
  with_row_threads(1ll * r.V * sizeof(T), [&](auto g) {
    constexpr int G = decltype(g)::value;
    policy_row_kernel<T, G><<<r.M, G, 0, s>>>(r, a, terms, err);
  });
}

cudaError_t launch_policy_loss(const LossRows& r, const PolicyArgs& a, void* scratch, int* err, cudaStream_t s) {
  float4* terms = static_cast<float4*>(scratch);
  if (r.M > 0) {
    if (r.fp32) policy_rows<float>(r, a, terms, err, s);
    else policy_rows<bf16>(r, a, terms, err, s);
  }
  policy_sum_kernel<<<1, 1024, 0, s>>>(terms, r.M, a.stats);
  return cudaGetLastError();
}

template <typename T>
static void preference_rows(const LossRows& r, const PreferenceArgs& a, void* scratch, int* err, cudaStream_t s) {
  uint8_t* base = static_cast<uint8_t*>(scratch);
  auto take = [&](size_t bytes) {
    uint8_t* p = base;
    base += al256(bytes);
    return p;
  };
  float2* ms = reinterpret_cast<float2*>(take(static_cast<size_t>(r.M) * sizeof(float2)));
  double* lps = reinterpret_cast<double*>(take(static_cast<size_t>(r.M) * sizeof(double)));
  double* sums = reinterpret_cast<double*>(take(2 * static_cast<size_t>(a.n_pairs) * sizeof(double)));
  float* g = reinterpret_cast<float*>(take(2 * static_cast<size_t>(a.n_pairs) * sizeof(float)));
  with_row_threads(1ll * r.V * sizeof(T), [&](auto gs) {
    constexpr int G = decltype(gs)::value;
    // with no rows one block still checks the offsets
    preference_logp_kernel<T, G><<<std::max(r.M, 1), G, 0, s>>>(r, a, ms, lps, err);
    preference_pair_kernel<<<1, 1024, 0, s>>>(r, a, lps, sums, g);
    if (r.dlogits && r.M > 0) preference_grad_kernel<T, G><<<r.M, G, 0, s>>>(r, a, ms, g);
  });
}

cudaError_t launch_preference_loss(const LossRows& r, const PreferenceArgs& a, void* scratch, int* err,
                                   cudaStream_t s) {
  if (r.fp32) preference_rows<float>(r, a, scratch, err, s);
  else preference_rows<bf16>(r, a, scratch, err, s);
  return cudaGetLastError();
}

}  // namespace gpt
