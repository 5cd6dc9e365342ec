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
#include "gemm.h"
#include "losses.cuh"

namespace gpt {

namespace {

using bf16 = __nv_bfloat16;

// A block of G threads works on a row, in pieces of two 16-byte vectors a
// thread that asynchronous copies bring to a ring of S pieces in shared
// memory.  Each thread reads only what it copied itself, so that the ring
// needs no barrier.  A row of at most S pieces stays there for a second pass;
// of a longer one the last S do, and the others come again, mostly from L2.
// At 512 threads a piece is 16 KB: rings of 4 (a policy row of up to 64 KB and
// the preference gradient: three blocks an SM, of which one loads while another
// computes and the third writes), of 6 for longer policy rows (fewer rows then
// compete for L2: 111 us instead of 122 for 1500 rows of 50,257 fp32 values),
// of 2 for the sums (69 us instead of 72 for 5,100 rows of 64 KB).
// Measured: 8192 x 32768 bf16 policy loss, 6,550 rows counted, kernel 179 us, 5.4 TB/s;
// it issues 17 instructions for an element (both passes, two exponentials) and
// the exponentials' unit is half busy, which the copies do not quite hide.
constexpr int kVecs = 2;   // vectors of a thread in a piece

// exp(d) for sums, whose errors must not all go one way: a bias of a row's sum
// adds up over a sequence's positions.  log2(e) comes in two parts (with one,
// exp(d) is off by 1.3e-8 |d|), and kEx2Mean makes up for ex2.approx, whose
// results lie 5e-8 too low on average (2.2e-8 for arguments above -1; measured
// over 2^24 arguments).  The fused step rounds once, so neither is lost, and
// exp(0) stays 1.  Mean error of a log-probability of 131,072 values: 5e-9
// instead of 1.2e-7, with 2e-7 root mean square.
constexpr float kLog2e = 1.44269502f, kLog2eLow = 1.92596303e-8f, kEx2Mean = 6.5e-8f;

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float exp_sum(float d) { return ex2(fmaf(d, kLog2e, fmaf(d, kLog2eLow, kEx2Mean))); }

__device__ __forceinline__ void copy_async16(uint4* dst, const uint4* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() {   // all but the last N groups have landed
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// 16 bytes of a row: 8 bf16 or 4 fp32 values
template <typename T>
struct Vec {
  static constexpr int n = 16 / sizeof(T);
  // every value -inf
  __device__ __forceinline__ static uint4 lowest() {
    const uint32_t u = sizeof(T) == 2 ? 0xff80ff80u : 0xff800000u;
    return make_uint4(u, u, u, u);
  }
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

// V values from x on in three stretches: `head` values before the first
// 16-byte boundary, `vecs` 16-byte vectors, and a tail.
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
  // N vectors of 16 bytes
  template <typename T, int N>
  __device__ __forceinline__ void add(const uint4 (&w)[N]) {
    constexpr int n = Vec<T>::n;
    float v[N][n], t = -INFINITY;
#pragma unroll
    for (int k = 0; k < N; ++k) {
      unpack<T>(w[k], v[k]);
#pragma unroll
      for (int e = 0; e < n; e += 2) t = fmax3(t, v[k][e], v[k][e + 1]);
    }
    raise(t);
    const float b = base(m);
    const uint64_t nb = f2_pack(-b, -b), hi = f2_pack(kLog2e, kLog2e), lo = f2_pack(kLog2eLow, kLog2eLow),
                   mean = f2_pack(kEx2Mean, kEx2Mean);
    uint64_t sum[2] = {f2_pack(0.f, 0.f), f2_pack(0.f, 0.f)};
#pragma unroll
    for (int k = 0; k < N; ++k) {
#pragma unroll
      for (int e = 0; e < n; e += 2) {
        const uint64_t d = f2_add(f2_pack(v[k][e], v[k][e + 1]), nb);
        float x0, x1;
        f2_unpack(f2_fma(d, hi, f2_fma(d, lo, mean)), x0, x1);
        sum[(e >> 1) & 1] = f2_add(sum[(e >> 1) & 1], f2_pack(ex2(x0), ex2(x1)));
      }
    }
    float s0, s1;
    f2_unpack(f2_add(sum[0], sum[1]), s0, s1);
    s += s0 + s1;
  }
};

__device__ __forceinline__ float warp_max_redux(float x) {
  float y;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(y) : "f"(x));
  return y;
}

template <typename T, int G, int S>
struct RowRing {
  static constexpr int kPiece = G * kVecs;   // vectors
  const T* x;
  int V, head, vecs, pieces;
  uint4* ring;
  __device__ RowRing(const T* x_, int V_, uint4* ring_) : x(x_), V(V_), ring(ring_) {
    const RowParts<T> row(x, V);
    head = row.head;
    vecs = row.vecs;
    pieces = (vecs + kPiece - 1) / kPiece;
  }
  __device__ __forceinline__ void fetch(int u) const {
    const uint4* xv = reinterpret_cast<const uint4*>(x + head);
    const int i = (u < pieces ? u : u - pieces) * kPiece + static_cast<int>(threadIdx.x);
    uint4* to = ring + u % S * kPiece + threadIdx.x;
#pragma unroll
    for (int k = 0; k < kVecs; ++k)
      if (i + k * G < vecs) copy_async16(to + k * G, xv + i + k * G);
  }
  // Calls one(j) for the values outside the vectors and piece(i, slot, full)
  // for steps u0 .. u0 + pieces - 1, step u being piece u mod pieces: i is the
  // thread's first vector of the piece, at slot, the others follow at steps of
  // G; full: all are within the row.  held: the first S steps are in the
  // ring already.
  template <typename One, typename Piece>
  __device__ __forceinline__ void pass(int u0, bool held, One one, Piece piece) const {
    const int end = u0 + pieces, tid = threadIdx.x;
    if (!held) {
#pragma unroll
      for (int k = 0; k < S; ++k) {
        if (u0 + k < end) fetch(u0 + k);
        copy_commit();
      }
    }
    if (tid < head) one(tid);
    const int tail = head + vecs * Vec<T>::n + tid;
    if (tail < V) one(tail);
    for (int u = u0; u < end; ++u) {
      copy_wait<S - 1>();
      const int first = (u < pieces ? u : u - pieces) * kPiece;
      const uint4* slot = ring + u % S * kPiece + tid;
      if (first + kPiece <= vecs) piece(first + tid, slot, std::true_type());
      else piece(first + tid, slot, std::false_type());
      if (u + S < end) fetch(u + S);
      copy_commit();
    }
  }
  // first step of a second pass: that of the oldest piece in the ring
  __device__ __forceinline__ int again() const { return max(0, pieces - S); }
};

// m and s over the row, for every thread of the block.
template <typename T, int G, int S>
__device__ __forceinline__ Softmax row_softmax(const RowRing<T, G, S>& row, float2* red) {
  Softmax a;
  row.pass(
      0, false, [&](int j) { a.add(to_f(row.x[j])); },
      [&](int i, const uint4* slot, auto full) {
        uint4 w[kVecs];
#pragma unroll
        for (int k = 0; k < kVecs; ++k)
          w[k] = decltype(full)::value || i + k * G < row.vecs ? slot[k * G] : Vec<T>::lowest();
        a.add<T>(w);
      });
  // over the warp, then over the warps
  a.raise(warp_max_redux(a.m));
  a.s = warp_sum(a.s);
  if constexpr (G > 32) {
    if (lane_id() == 0) red[warp_id()] = make_float2(a.m, a.s);
    __syncthreads();
    const float2 q = red[lane_id() & (G / 32 - 1)];
    a.m = q.x;
    a.s = q.y;
    a.raise(warp_max_redux(a.m));
#pragma unroll
    for (int o = G / 64; o > 0; o >>= 1) a.s += __shfl_xor_sync(0xffffffffu, a.s, o);
  }
  return a;
}

// The gradient g (1[j = y] - p), p = exp(x - m) / s, of one row.
template <typename T>
struct Gradient {
  int y;
  float xy, g, f, b;   // xy: the target's logit
  __device__ Gradient(int y_, float xy_, float g_, float m, float s)
      : y(y_), xy(xy_), g(g_), f(-g_ / s), b(Softmax::base(m)) {}
  __device__ __forceinline__ float value(float x) const { return f * ex2((x - b) * kLog2e); }
  __device__ __forceinline__ void one(const T* x, T* d, int j) const {
    from_f(d + j, value(to_f(x[j])) + (j == y ? g : 0.f));
  }
  // a vector's values but for the target's g, to d
  template <bool kWide>
  __device__ __forceinline__ void vec(const uint4& w, T* d) const {
    constexpr int n = Vec<T>::n;
    float v[n];
    unpack<T>(w, v);
    const uint64_t nb = f2_pack(-b, -b), c = f2_pack(kLog2e, kLog2e), ff = f2_pack(f, f);
#pragma unroll
    for (int e = 0; e < n; e += 2) {
      float x0, x1;
      f2_unpack(f2_mul(f2_add(f2_pack(v[e], v[e + 1]), nb), c), x0, x1);
      f2_unpack(f2_mul(f2_pack(ex2(x0), ex2(x1)), ff), v[e], v[e + 1]);
    }
    if constexpr (kWide) {
      *reinterpret_cast<uint4*>(d) = pack<T>(v);
    } else {
#pragma unroll
      for (int e = 0; e < n; ++e) from_f(d + e, v[e]);
    }
  }
};

// The row's gradient; d may be x.  held: after row_softmax.
template <typename T, int G, int S>
__device__ __forceinline__ void row_gradient(const RowRing<T, G, S>& row, T* d, bool held, const Gradient<T>& grad) {
  constexpr int n = Vec<T>::n;
  auto all = [&](auto wide) {
    row.pass(
        held ? row.again() : 0, held, [&](int j) { grad.one(row.x, d, j); },
        [&](int i, const uint4* slot, auto full) {
          T* to = d + row.head + i * n;
#pragma unroll
          for (int k = 0; k < kVecs; ++k)
            if (decltype(full)::value || i + k * G < row.vecs)
              grad.template vec<decltype(wide)::value>(slot[k * G], to + k * G * n);
        });
  };
  if (((reinterpret_cast<uintptr_t>(row.x) ^ reinterpret_cast<uintptr_t>(d)) & 15) == 0) all(std::true_type());
  else all(std::false_type());
  // the target's value again, by the thread that wrote its vector
  const int at = grad.y - row.head;
  if (at >= 0 && at < row.vecs * n && at / n % G == static_cast<int>(threadIdx.x))
    from_f(d + grad.y, grad.value(grad.xy) + grad.g);
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
    if (err) atomicOr(err, ERRF_TOKEN_RANGE);
    return -1;
  }
  return y;
}

// log p_y from the row's statistics, in 64 bits (one thread's work): its sum
// over a sequence is compared with sums of nearly the same size.
__device__ __forceinline__ double target_logp(float x, const Softmax& a) {
  return static_cast<double>(x) - Softmax::base(a.m) - log(static_cast<double>(a.s));
}

// Launches pick(G, S) over the rows.  G follows the row's bytes: 8 vectors of
// a thread at 64 KB, fewer threads where a row would leave most of them idle.
template <typename T, int S, bool kChained, typename Pick, typename... Args>
cudaError_t launch_rows(const LossRows& r, cudaStream_t s, Pick pick, Args... args) {
  const long long bytes = 1ll * r.V * sizeof(T);
  auto launch = [&](auto kG) -> cudaError_t {
    constexpr int G = decltype(kG)::value, kPieceBytes = G * kVecs * 16;
    auto kern = pick(kG, std::integral_constant<int, S>());
    const int slots = static_cast<int>(std::min<long long>((bytes + kPieceBytes - 1) / kPieceBytes, S));
    if constexpr (S * kPieceBytes > 47 * 1024) {   // with the static words, over the default limit
      static std::atomic<unsigned long long> configured{0};
      const cudaError_t e = set_smem_limit_once(kern, S * kPieceBytes, configured);
      if (e != cudaSuccess) return e;
    }
    if constexpr (kChained) return launch_chained(kern, std::max(r.M, 1), G, slots * kPieceBytes, s, args...);
    kern<<<std::max(r.M, 1), G, slots * kPieceBytes, s>>>(args...);
    return cudaGetLastError();
  };
  if (bytes <= 4096) return launch(std::integral_constant<int, 32>());
  if (bytes <= 16384) return launch(std::integral_constant<int, 128>());
  return launch(std::integral_constant<int, 512>());
}

// ------------------------------------------------------------ policy loss
//
// Per counted token: r = exp(lp - old), the surrogate -min(r A, clip(r, 1 -
// low, 1 + high) A), and c k with k = exp(d) - d - 1, d = ref - lp.  With
// dlp the derivative by lp, -A r where the unclipped product is the smaller
// one (at a border both are) and 0 elsewhere, plus c (1 - exp(d)), the row
// factor is g = w dlp.  The scalars of a row are computed in 64 bits: k loses
// half its digits for small d in 32, and it is one thread's work.
// A term of weight 0 is left out, infinite (the target masked to -inf) or not.
__device__ __forceinline__ double times(double weight, double x) { return weight == 0.0 ? 0.0 : weight * x; }

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
    k = isinf(e) ? e : e - d;
    dlp -= times(a.kl_coef, e);
  }
  PolicyRow p;
  const double surrogate = -adv * used;
  p.g = static_cast<float>(w * dlp);
  p.term = make_float4(static_cast<float>(w * (times(a.kl_coef, k) + surrogate)), static_cast<float>(w * surrogate),
                       static_cast<float>(w * k), cut ? w32 : 0.f);
  return p;
}

template <typename T, int G, int S>
__global__ void __launch_bounds__(G)
    policy_row_kernel(const LossRows R, const PolicyArgs a, float4* __restrict__ terms, int* err) {
  extern __shared__ uint4 ring[];
  chain_go();
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
  const RowRing<T, G, S> row(x, R.V, ring);
  const float xy = to_f(x[y]);
  const Softmax sm = row_softmax(row, red);
  if (threadIdx.x == 0) {
    const double lp = target_logp(xy, sm);
    const PolicyRow p = policy_row(a, r, lp, wt);
    a.logp[r] = static_cast<float>(lp);
    terms[r] = p.term;
    gs = p.g;
  }
  if (!d) return;
  __syncthreads();
  row_gradient(row, d, true, Gradient<T>(y, xy, gs, sm.m, sm.s));
}

// stats = sums of the rows' terms, in 64 bits and a fixed order
__global__ void __launch_bounds__(1024) policy_sum_kernel(const float4* __restrict__ terms, int M, float* stats) {
  __shared__ double red[4][32];
  chain_wait();
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

// Rows that the sequences cover, if their offsets are in order.
__device__ __forceinline__ int last_row(const PreferenceArgs& a, int M) { return min(a.cu[2 * a.n_pairs], M); }

// Words that the kernels of a call share: blocks of the sums' kernel that are
// done, and the rows that the sequences cover (-1 if their offsets are bad).
struct PairWords {
  int done, rows;
};

// Statistics and log-probability of every row, into scratch alone: whether
// the offsets are in order is for the next kernel to say.
template <typename T, int G, int S>
__global__ void __launch_bounds__(G)
    preference_logp_kernel(const LossRows R, const PreferenceArgs a, float2* __restrict__ ms, double* __restrict__ lps,
                           PairWords* words) {
  extern __shared__ uint4 ring[];
  chain_go();
  __shared__ float2 red[G / 32];
  const int r = blockIdx.x;
  if (r == 0 && threadIdx.x == 0) words->done = 0;
  if (r >= R.M) return;
  const int y = R.targets[r];
  if (r >= last_row(a, R.M) || y < 0 || y >= R.V) return;
  const T* x = static_cast<const T*>(R.logits) + r * R.ld;
  const float xy = threadIdx.x == 0 ? to_f(x[y]) : 0.f;
  const Softmax sm = row_softmax(RowRing<T, G, S>(x, R.V, ring), red);
  if (threadIdx.x == 0) {
    ms[r] = make_float2(sm.m, sm.s);
    lps[r] = target_logp(xy, sm);
  }
}

// Checks the offsets: from 0, not decreasing, ending within the rows.  Then
// each block adds up some sequences (a block for a sequence where there are
// few: with a warp for each, long ones took 15 us), and the last one to finish
// computes the margins, the loss and the row factors (one per sequence).  The
// order of every sum is fixed.
constexpr int kSumThreads = 256;
__device__ __forceinline__ double block_sum(double s, double* red) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  __syncthreads();
  if (lane_id() == 0) red[warp_id()] = s;
  __syncthreads();
  double t = 0.0;
#pragma unroll
  for (int w = 0; w < kSumThreads / 32; ++w) t += red[w];
  return t;
}
__global__ void __launch_bounds__(kSumThreads)
    preference_sum_kernel(const LossRows R, const PreferenceArgs a, const double* __restrict__ lps, double* sums,
                          float* __restrict__ g, PairWords* words, int* err) {
  __shared__ double red[kSumThreads / 32];
  __shared__ bool last;
  chain_go();
  chain_wait();
  const int n = 2 * a.n_pairs, tid = threadIdx.x;
  int bad = a.cu[0] != 0 || a.cu[n] > R.M;
  for (int i = tid; i < n; i += kSumThreads) bad |= a.cu[i + 1] < a.cu[i];
  bad = __syncthreads_or(bad);
  if (blockIdx.x == 0 && tid == 0) {
    words->rows = bad ? -1 : a.cu[n];
    if (bad && err) atomicOr(err, ERRF_SEQUENCE);
  }
  if (bad) return;
  // positions past the last sequence are not counted
  for (int r = a.cu[n] + blockIdx.x * kSumThreads + tid; r < R.M; r += gridDim.x * kSumThreads) a.logp[r] = 0.f;
  for (int q = blockIdx.x; q < n; q += gridDim.x) {
    const int r1 = a.cu[q + 1];
    double s = 0.0;
    for (int r = a.cu[q] + tid; r < r1; r += kSumThreads) {
      const double lp = row_target(R, r, err) < 0 ? 0.0 : lps[r];
      a.logp[r] = static_cast<float>(lp);
      s += lp;
    }
    s = block_sum(s, red);
    if (tid == 0) {
      sums[q] = s;
      a.seq_logp[q] = static_cast<float>(s);
    }
  }
  if (tid == 0) {
    __threadfence();
    last = atomicAdd(&words->done, 1) == static_cast<int>(gridDim.x) - 1;
  }
  __syncthreads();
  if (!last) return;
  __threadfence();
  double loss = 0.0;
  for (int i = tid; i < a.n_pairs; i += kSumThreads) {
    const double ref = a.ref_logp ? static_cast<double>(a.ref_logp[2 * i]) - a.ref_logp[2 * i + 1] : 0.0;
    const double z = a.beta * (__ldcg(sums + 2 * i) - __ldcg(sums + 2 * i + 1) - ref);
    // sigmoid(-|z|), and log sigmoid(+-z) = min(+-z, 0) - log(1 + exp(-|z|))
    const double t = exp(-fabs(z)), soft = log1p(t), less = t / (1.0 + t);
    const double sig_pos = z >= 0.0 ? 1.0 - less : less, sig_neg = z >= 0.0 ? less : 1.0 - less;
    loss += soft + times(1.0 - a.smoothing, fmax(-z, 0.0)) + times(a.smoothing, fmax(z, 0.0));
    const double dz = a.beta / a.n_pairs * (a.smoothing * sig_pos - (1.0 - a.smoothing) * sig_neg);
    a.margin[i] = static_cast<float>(z);
    g[2 * i] = static_cast<float>(dz);
    g[2 * i + 1] = static_cast<float>(-dz);
  }
  loss = block_sum(loss, red);
  if (tid == 0) *a.loss = static_cast<float>(loss / a.n_pairs);
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

template <typename T, int G, int S>
__global__ void __launch_bounds__(G)
    preference_grad_kernel(const LossRows R, const PreferenceArgs a, const float2* __restrict__ ms,
                           const float* __restrict__ g, const PairWords* __restrict__ words) {
  extern __shared__ uint4 ring[];
  chain_wait();
  const int r = blockIdx.x, rows = words->rows;
  if (rows < 0 || (r >= rows && !a.clear_past)) return;
  T* d = static_cast<T*>(R.dlogits) + r * R.ld_d;
  const int y = r < rows ? row_target(R, r, nullptr) : -1;
  if (y < 0) {
    row_zero<T, G>(d, R.V);
    return;
  }
  const T* x = static_cast<const T*>(R.logits) + r * R.ld;
  const float2 q = ms[r];
  const float gr = g[row_sequence(a.cu, 2 * a.n_pairs, r)];
  const float xy = to_f(x[y]);
  row_gradient(RowRing<T, G, S>(x, R.V, ring), d, false, Gradient<T>(y, xy, gr, q.x, q.y));
}

constexpr size_t al256(size_t x) { return (x + 255) / 256 * 256; }

}  // namespace

size_t policy_loss_scratch(int M) { return al256(static_cast<size_t>(M) * sizeof(float4)) + 256; }

size_t preference_loss_scratch(int M, int n_pairs) {
  return 256 + al256(static_cast<size_t>(M) * sizeof(float2)) + al256(static_cast<size_t>(M) * sizeof(double)) +
         al256(2 * static_cast<size_t>(n_pairs) * sizeof(double)) +
         al256(2 * static_cast<size_t>(n_pairs) * sizeof(float));
}

template <typename T>
static cudaError_t policy_rows(const LossRows& r, const PolicyArgs& a, float4* terms, int* err, cudaStream_t s) {
  auto pick = [](auto g, auto slots) { return policy_row_kernel<T, decltype(g)::value, decltype(slots)::value>; };
  if (1ll * r.V * sizeof(T) <= 65536) return launch_rows<T, 4, false>(r, s, pick, r, a, terms, err);
  return launch_rows<T, 6, false>(r, s, pick, r, a, terms, err);
}

cudaError_t launch_policy_loss(const LossRows& r, const PolicyArgs& a, void* scratch, int* err, cudaStream_t s) {
  float4* terms = static_cast<float4*>(scratch);
  if (r.M > 0) {
    const cudaError_t e = r.fp32 ? policy_rows<float>(r, a, terms, err, s) : policy_rows<bf16>(r, a, terms, err, s);
    if (e != cudaSuccess) return e;
  }
  return launch_chained(policy_sum_kernel, 1, 1024, 0, s, terms, r.M, a.stats);
}

template <typename T>
static cudaError_t preference_rows(const LossRows& r, const PreferenceArgs& a, void* scratch, int* err,
                                   cudaStream_t s) {
  uint8_t* base = static_cast<uint8_t*>(scratch);
  auto take = [&](size_t bytes) {
    uint8_t* p = base;
    base += al256(bytes);
    return p;
  };
  PairWords* words = reinterpret_cast<PairWords*>(take(sizeof(PairWords)));
  float2* ms = reinterpret_cast<float2*>(take(static_cast<size_t>(r.M) * sizeof(float2)));
  double* lps = reinterpret_cast<double*>(take(static_cast<size_t>(r.M) * sizeof(double)));
  double* sums = reinterpret_cast<double*>(take(2 * static_cast<size_t>(a.n_pairs) * sizeof(double)));
  float* g = reinterpret_cast<float*>(take(2 * static_cast<size_t>(a.n_pairs) * sizeof(float)));
  cudaError_t e = launch_rows<T, 2, false>(
      r, s, [](auto g, auto slots) { return preference_logp_kernel<T, decltype(g)::value, decltype(slots)::value>; },
      r, a, ms, lps, words);
  if (e != cudaSuccess) return e;
  const int blocks = std::min(2 * a.n_pairs, 2 * device_sm_count());
  e = launch_chained(preference_sum_kernel, blocks, kSumThreads, 0, s, r, a, lps, sums, g, words, err);
  if (e != cudaSuccess) return e;
  if (r.dlogits && r.M > 0)
    e = launch_rows<T, 4, true>(
        r, s,
        [](auto g, auto slots) { return preference_grad_kernel<T, decltype(g)::value, decltype(slots)::value>; }, r, a,
        ms, g, words);
  return e;
}

cudaError_t launch_preference_loss(const LossRows& r, const PreferenceArgs& a, void* scratch, int* err,
                                   cudaStream_t s) {
  const cudaError_t e =
      r.fp32 ? preference_rows<float>(r, a, scratch, err, s) : preference_rows<bf16>(r, a, scratch, err, s);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace gpt
