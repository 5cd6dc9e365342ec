// Causal flash attention, forward and backward, head_dim 128, bf16 operands
// with fp32 softmax and accumulation (online softmax; the forward saves the
// row log-sum-exp, the backward recomputes P from it).  Optional sliding
// window (query t sees keys t - window .. t) and grouped kv heads (query head
// h reads kv head h / (H / Hkv)), the two attention variants of "¿Cómo
// Entrenar Tu Propio ChatGPT por $50?", section "1. Modelo GPT".
//
// Layouts: q is [B, H, T, 128], k, v, dk, dv are [B, Hkv, T, 128]; the forward output O and the
// incoming gradient dO are token-major [B, T, H, 128] (the rows of the
// projection GEMMs); dq is accumulated in fp32 [B, H, T, 128]; lse and
// D = rowsum(dO * O) are [B, H, T].
//
// Both directions run on the 5th-generation tensor cores (tcgen05.mma with
// TMEM accumulators), fed by TMA; softmax work runs in dedicated warps that
// exchange tiles with the MMA issuer through mbarriers.
#include <algorithm>
#include <type_traits>

#include "attention.cuh"
#include "common.cuh"
#include "gemm.h"

namespace gpt {

namespace {

constexpr int HD = 128;

// ------------------------------------------------------- packed sequences
//
// For the packed forward and the packed build of the backward (kPacked), T
// positions hold sequences of different lengths end to end, and query t sees
// the keys lo[t] .. t, lo[t] = max(start of t's sequence, t - window).  lo does not
// decrease with t, so a tile of 128 queries sees the key blocks from that of
// lo[first query] to its own: tiles and key blocks stay on the 128-position
// grid whatever the sequence boundaries (a tile may hold many short
// sequences, or parts of two long ones), blocks outside are never visited,
// and the softmax masks by lo per row.  The other way round the queries that
// see key t are t .. hi[t], hi[t] = min(end of the sequence - 1, t + window).
// The plan (attention_plan_kernel, once per batch) holds lo, hi and the work
// items sorted by their number of blocks, longest first.  (Tiles that start
// with their sequence would need 6% fewer blocks on documents of 128 to 2048
// tokens, 14% on chats of 24 to 1024, but more tiles.)
// Positions past the last sequence are not read, and written only as zeros and
// on request (kClear*).  Their memory may hold NaN, which a zero probability
// would not remove: the forward clears those rows of a V tile in shared memory
// (K and Q there reach only scores that are masked and rows that are not
// stored), the backward copies the tensor maps to device memory with their
// token extent cut to the sequences' end, so that TMA fills the rows of all four
// operands with zeros.
// Inside the sequences, too, a tile's products run over keys (or queries) that a
// row does not see, with probability 0.  A NaN or an infinity there makes every
// output that it reaches non-finite, so the kernels look at their outputs, and
// rows that are not finite although all that they see is, are computed again
// from that alone, by a warp each (repair_*).  Looking costs the forward nothing
// measurable, the backward 3 to 5 us.
// Scores, maxima, row sums, lse, D and every sum over keys or queries are fp32.
// Rounded to bf16 are only P, as the operand of P V and P^T dO, and dS, formed
// from P in fp32, as that of dS K and dS^T Q: the tensor cores take both operands
// of a product in one type, and q, k, v and dO are bf16.  Measured in the 2-norm
// against 64 bits on sequences of 2 to 300 tokens, scores of the usual size and
// eight times as large: dq and dk 0.0023 to 0.0025, dv 0.0015 to 0.0023, o 0.0018
// to 0.0021, of which 0.0017 is the rounding of the result.

// A [tokens, heads, 128] bf16 tensor, strides in elements.
struct HeadRows {
  const bf16* ptr;
  long long tok, head;
};
struct PackedArgs {
  const int* meta;          // forward: the plan's kMeta* words
  const int* lo;            // [T]
  const int* hi;            // [T]; -1 past the last sequence
  const int2* fwd;          // forward entries: query tile, first key block that it sees
  const int2* bwd;          // backward entries: key block, number of query blocks that see it
  const int* ctl;           // backward: kCtl* words
  const CUtensorMap* maps;  // backward: q, k, v, dO with the extent patched in
  long long o_tok, o_head;    // forward: strides of o in elements; backward: of dk
  long long dv_tok, dv_head;  // backward: strides of dv
  int clear;                  // forward: kClear* bits
  HeadRows q, k, v;           // forward: for rows to repair
  int* bad;                   // backward: ctl[kCtlBad]
};
// Outputs whose rows past the last sequence become zeros instead of staying as they are.
enum { kClearO = 1, kClearLse = 2, kClearDq = 1, kClearDk = 2, kClearDv = 4 };
// kCtlBad: some row of a gradient is not finite
enum { kCtlSched = 0, kCtlEntries = 1, kCtlValid = 2, kCtlBad = 3 };
// Words of a plan: positions that the sequences hold, forward and backward
// entries, T.
enum { kMetaTotal = 0, kMetaFwd = 1, kMetaBwd = 2, kMetaT = 3, kMetaMagic = 4, kPlanMeta = 64 };
constexpr int kPlanMagic = 0x5e91a7e;

// What the kernels take from a plan is bounded, and entries out of bounds are
// left out and latched as ERRF_SHAPE: a buffer that something else has
// overwritten must not send them out of the tensors or through 2^31 key blocks.
struct PlanSizes {
  bool fits;            // a plan of T positions
  int valid, fwd, bwd;  // positions that hold sequences, entries
};
__device__ __forceinline__ PlanSizes plan_sizes(const int* meta, int T) {
  PlanSizes s = {meta[kMetaMagic] == kPlanMagic && meta[kMetaT] == T, 0, 0, 0};
  if (s.fits) {
    s.valid = max(0, min(meta[kMetaTotal], T));
    const int tiles = (s.valid + 127) / 128;
    s.fwd = max(0, min(meta[kMetaFwd], tiles));
    s.bwd = max(0, min(meta[kMetaBwd], tiles));
  }
  return s;
}
// query tile and first key block
__device__ __forceinline__ bool fwd_entry_ok(int2 e, int valid, int* err) {
  if (e.x >= 0 && e.x < (valid + 127) / 128 && e.y >= 0 && e.y <= e.x) return true;
  if (err) atomicOr(err, ERRF_SHAPE);
  return false;
}
// key block and number of query blocks
__device__ __forceinline__ bool bwd_entry_ok(int2 e, int valid, int* err) {
  const int tiles = (valid + 127) / 128;
  if (e.x >= 0 && e.x < tiles && e.y >= 1 && e.y <= tiles - e.x) return true;
  if (err) atomicOr(err, ERRF_SHAPE);
  return false;
}

// The packed forward takes its items from the grid: it is launched with a
// block for each, and a running block asks for the index of one that has not
// started, which is then never started (cluster launch control).  So items go
// out in order, without a counter in memory that something would have to
// zero first.
__device__ __forceinline__ void next_block_ask(uint4* answer, uint64_t* bar) {
  mbar_arrive_expect_tx(bar, 16);
  asm volatile(
      "clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128 [%0], [%1];" ::"r"(
          smem_u32(answer)),
      "r"(smem_u32(bar))
      : "memory");
}
// Its answer, once the barrier has completed: a block index, -1 if all have started.
__device__ __forceinline__ int next_block_answer(const uint4* answer) {
  int x;
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b128 r;\n\t"
      "ld.shared.b128 r, [%1];\n\t"
      "clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, r;\n\t"
      "mov.s32 %0, -1;\n\t"
      "@p clusterlaunchcontrol.query_cancel.get_first_ctaid::x.b32.b128 %0, r;\n\t}"
      : "=r"(x)
      : "r"(smem_u32(answer))
      : "memory");
  fence_proxy_async_smem();   // read before the next answer is written there
  return x;
}

// makes a tensor map that a kernel wrote to device memory usable by this
// thread's TMA instructions
__device__ __forceinline__ void tensormap_acquire(const CUtensorMap* m) {
  asm volatile("fence.proxy.tensormap::generic.acquire.gpu [%0], 128;" ::"l"(m) : "memory");
}

// ------------------------------------------------- forward on tcgen05 / TMEM
//
// Persistent: one CTA per SM takes work items, a pair of 128-query tiles
// (A = 2p, B = 2p + 1) of one batch*head, until none are left; the pair
// shares every K and V block it loads.  Items are numbered head-major, the
// longest pair of a head first, so the CTAs running at one time share the
// K/V of a few heads in L2; a scheduler word in device memory hands them out
// in that order (an atomic counter, zeroed before the launch), and with no
// word each CTA takes every gridDim.x-th item.  The next item's Q loads and
// first S = Q K^T run while the softmax warps finish the previous item, so
// the per-item load and pipeline-fill latency is hidden.
// 384 threads in three warp groups; the first (TMA, MMA and two idle warps)
// gives registers to the two softmax groups (setmaxnreg 56 / 224 / 224, which
// adds up to the 168 per thread the block is launched with), so each softmax
// thread keeps its whole S row in registers.
//   warp 0      TMA: takes the items and publishes their numbers in a shared
//               ring, loads Q_A and Q_B of each (once every warp has read the
//               item number and the previous Q is no longer read), K_j and
//               V_j through two-slot rings that run on across items
//   warp 1      TMEM owner and MMA issuer.  TMEM columns: S_A [0,128),
//               S_B [128,256), O_A [256,384), O_B [384,512).  Per key block
//               j: O_A += P_A V_j and O_B += P_B V_j, with P read from TMEM
//               (the softmax warps write it as packed bf16 over the first 64
//               columns of S), then S_A = Q_A K_{j+1}^T once O_A's product
//               has read P_A, and then the same for B; the tensor cores thus
//               work on one tile while the other tile's softmax runs.
//   warps 4..7  softmax of tile A, warps 8..11 of tile B, one query row (TMEM
//               lane) per thread: the block max from a first pass over the S
//               row, exp2 into bf16 P, the row sum; after the last
//               block, O / l and the log-sum-exp.
// The reference max of a row only moves when the block max exceeds it by
// more than 8 (log2 units), so P stays below 2^8; when it moves, the warp
// rescales its rows of O in TMEM (the previous P V has completed by then:
// S of this block was issued after it).

// Exponentials per group of 8 scores evaluated on the MUFU unit (the rest by
// the polynomial on the FMA pipe; all on MUFU is fastest) in the kernels over
// whole rows: forward, alternating between two values over consecutive groups;
// backward, one value.  Even numbers (pairs).
#ifndef GPT_FWD_MUFU_EVEN
#define GPT_FWD_MUFU_EVEN 8
#endif
#ifndef GPT_FWD_MUFU_ODD
#define GPT_FWD_MUFU_ODD 8
#endif
#ifndef GPT_BWD_MUFU
#define GPT_BWD_MUFU 8
#endif

constexpr int TF_TILE = 16384;                // one [128 rows][128 B] swizzled tile
constexpr int TF_BUF = 2 * TF_TILE;           // 128 x 128 bf16 as two 64-column tiles
constexpr int TF_STAGE = 16384;               // output rows, 2 KB for each softmax warp
constexpr int TF_SMEM = 6 * TF_BUF + TF_STAGE + 256;
constexpr float TF_RESCALE = 8.f;

__device__ __forceinline__ float ex2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ void tmem_store32(uint32_t taddr, const uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
      "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,"
      "%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]),
      "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]),
      "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]),
      "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
      : "memory");
}

// Waits for the loads so far; no use of x moves above the wait.
__device__ __forceinline__ void tmem_landed(uint32_t (&x)[32]) {
  tmem_wait_ld();
#pragma unroll
  for (int i = 0; i < 32; ++i) asm volatile("" : "+r"(x[i]));
}

__device__ __forceinline__ void tmem_store16(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
      "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]),
      "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}

// Item n: batch*head bh and the pair's first query tile, key blocks j0 ..
// (causal end), per tile counts nkvA, nkvB (0: tile B past the sequence).
struct FwdItem {
  int bh, bkv, qtA, j0, nkvA, nkvB, nkv;
  bool hasB;
};

__device__ __forceinline__ FwdItem fwd_item(int n, int nq, int H, int Hkv, int kvs, int wl) {
  FwdItem it;
  const int npairs = (nq + 1) / 2;
  it.bh = n / npairs;
  const int pair = npairs - 1 - (n - it.bh * npairs);
  // k/v row of this query head's kv head: batch rows of kvs heads each
  it.bkv = (it.bh / H) * kvs + (it.bh - (it.bh / H) * H) / (H / Hkv);
  it.qtA = 2 * pair;
  it.hasB = it.qtA + 1 < nq;
  // both tiles start at the first key block any row of tile A sees; rows for
  // which a block lies wholly outside their window see only masked scores
  it.j0 = max(0, it.qtA * 128 - wl) / 128;
  it.nkvA = it.qtA + 1 - it.j0;
  it.nkvB = it.hasB ? it.qtA + 2 - it.j0 : 0;
  it.nkv = it.hasB ? it.nkvB : it.nkvA;
  return it;
}

// S row of query row 32 Q + lane of a causal diagonal block: keys 32 Q + lane
// + 1 .. 127 become -inf (the keys of chunk Q above the lane, then every
// later chunk); Q is the warp's TMEM lane quarter, so no branch diverges.
template <int Q>
__device__ __forceinline__ void causal_mask_row(uint32_t (&sr)[128], int lane) {
#pragma unroll
  for (int k = 0; k < 32; ++k)
    if (k > lane) sr[32 * Q + k] = __float_as_uint(-INFINITY);
#pragma unroll
  for (int k = 32 * (Q + 1); k < 128; ++k) sr[k] = __float_as_uint(-INFINITY);
}

// kCols fp32 columns from TMEM times f, in bf16, of each lane's row to rows
// dst + row * pitch (elements), row = 0 .. n_rows - 1 of the warp's 32, through
// 64 kCols bytes of shared memory: kCols / 8 lanes write one row's values
// together.  (With a lane for each row a store touched 32 cache lines.)
// kCheck: returns 0 if this lane's values are finite, else NaN.
template <int kCols, bool kCheck = false>
__device__ __forceinline__ float store_rows(uint32_t taddr, float f, uint8_t* stage, bf16* dst, long long pitch,
                                            int n_rows) {
  constexpr int kUnits = kCols / 8, kBytes = kCols * 2;   // of 16 bytes in a row; of a row
  const int lane = lane_id();
  // unit u of row r lies at u ^ swap(r): eight lanes, or rows, meet 32 different banks
  auto swap = [](int r) { return kUnits == 8 ? r & 7 : (r >> 1) & 3; };
  uint32_t w[kCols / 2];
  uint64_t z = f2_pack(0.f, 0.f);
#pragma unroll
  for (int c = 0; c < kCols; c += 32) {
    uint32_t x[32];
    tmem_load32_async(taddr + c, x);
    tmem_landed(x);
    if constexpr (kCheck) {
#pragma unroll
      for (int k = 0; k < 32; k += 2)
        z = f2_fma(f2_pack(__uint_as_float(x[k]), __uint_as_float(x[k + 1])), f2_pack(0.f, 0.f), z);
    }
#pragma unroll
    for (int k = 0; k < 16; ++k)
      w[c / 2 + k] = pack_bf16x2(__uint_as_float(x[2 * k]) * f, __uint_as_float(x[2 * k + 1]) * f);
  }
  __syncwarp();   // the previous contents have been read
#pragma unroll
  for (int u = 0; u < kUnits; ++u)
    *reinterpret_cast<uint4*>(stage + lane * kBytes + ((u ^ swap(lane)) << 4)) =
        make_uint4(w[4 * u], w[4 * u + 1], w[4 * u + 2], w[4 * u + 3]);
  __syncwarp();
  const int u = lane % kUnits;
#pragma unroll
  for (int i = 0; i < kUnits; ++i) {
    const int row = 32 / kUnits * i + lane / kUnits;
    const uint4 v = *reinterpret_cast<const uint4*>(stage + row * kBytes + ((u ^ swap(row)) << 4));
    if (row < n_rows) *reinterpret_cast<uint4*>(dst + row * pitch + u * 8) = v;
  }
  float z0, z1;
  f2_unpack(z, z0, z1);
  return z0 + z1;
}

// ---- rows computed again (a warp for a row, 4 of the 128 dims a lane)

__device__ __forceinline__ float4 row4(const HeadRows& r, int t, int h) {
  const uint2 u = *reinterpret_cast<const uint2*>(r.ptr + t * r.tok + h * r.head + lane_id() * 4);
  return make_float4(bf16_lo(u.x), bf16_hi(u.x), bf16_lo(u.y), bf16_hi(u.y));
}
__device__ __forceinline__ bool finite4(float4 x) { return x.x * 0.f + x.y * 0.f + x.z * 0.f + x.w * 0.f == 0.f; }
__device__ __forceinline__ bool finite_row(float4 x) { return __all_sync(0xffffffffu, finite4(x)); }
__device__ __forceinline__ float dot_row(float4 a, float4 b) {
  return warp_sum(a.x * b.x + a.y * b.y + a.z * b.z + a.w * b.w);
}
__device__ __forceinline__ void add_row(float4& a, float f, float4 x) {
  a.x = fmaf(f, x.x, a.x);
  a.y = fmaf(f, x.y, a.y);
  a.z = fmaf(f, x.z, a.z);
  a.w = fmaf(f, x.w, a.w);
}
__device__ __forceinline__ void put_row(bf16* row, float f, float4 x) {
  *reinterpret_cast<uint2*>(row + lane_id() * 4) = make_uint2(pack_bf16x2(x.x * f, x.y * f), pack_bf16x2(x.z * f, x.w * f));
}

// o of query t of head h, which sees the keys lo .. t of those that its tile
// visits, first .. last: left as it is if they explain it.  The nearest keys
// first, so that a sequence that has diverged is left after a few.
__device__ __noinline__ void repair_o_row(const PackedArgs& a, bf16* o, int h, int hk, int t, int lo, int first,
                                          int last, float lse2, float scale_log2) {
  const float4 q = row4(a.q, t, h);
  if (!finite_row(q)) return;
  lo = min(max(lo, first), t);   // whatever the plan holds
  bool clean = true;
  for (int j = first; j <= last && clean; ++j)
    if (j < lo || j > t) clean = finite_row(row4(a.v, j, hk));
  if (clean) return;
  // eight keys at a time, for their latencies
  constexpr int kKeys = 8;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int j = t; j >= lo; j -= kKeys) {
    float4 k[kKeys], v[kKeys];
#pragma unroll
    for (int i = 0; i < kKeys; ++i) {
      k[i] = row4(a.k, max(j - i, lo), hk);
      v[i] = row4(a.v, max(j - i, lo), hk);
    }
    bool finite = true;
    float s[kKeys];
#pragma unroll
    for (int i = 0; i < kKeys; ++i) {
      finite &= finite4(k[i]) && finite4(v[i]);
      s[i] = dot_row(q, k[i]);
    }
    if (!__all_sync(0xffffffffu, finite)) return;
#pragma unroll
    for (int i = 0; i < kKeys; ++i)
      if (j - i >= lo) add_row(acc, ex2_approx(fmaf(s[i], scale_log2, -lse2)), v[i]);
  }
  put_row(o + t * a.o_tok + h * a.o_head, 1.f, acc);
}

template <bool kFine>
__global__ void __launch_bounds__(384, 1)
    attn_fwd_tc_kernel(const __grid_constant__ CUtensorMap tq, const __grid_constant__ CUtensorMap tk,
                       const __grid_constant__ CUtensorMap tv, bf16* __restrict__ o, float* __restrict__ lse,
                       int H, int Hkv, int kvs, int T, int wl, float scale_log2, int n_items, int* sched,
                       int* err, long long wait_cycles) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  // the 128-byte-swizzled tiles need a 1024-byte-aligned base, which the
  // dynamic shared memory window provides; refuse to run otherwise
  if (smem_u32(smem_raw) & 1023u) {
    if (threadIdx.x == 0 && err) atomicOr(err, ERRF_SHAPE);
    return;
  }
  uint8_t* sm = smem_raw;
  uint8_t* sQ = sm;                  // two tiles: A, B
  uint8_t* sK = sm + 2 * TF_BUF;     // two slots
  uint8_t* sV = sm + 4 * TF_BUF;     // two slots
  uint8_t* sOut = sm + 6 * TF_BUF;
  uint64_t* bars = reinterpret_cast<uint64_t*>(sm + 6 * TF_BUF + TF_STAGE);
  uint64_t* q_full = bars + 0;    // Q of item n landed (or the end marker)
  uint64_t* q_empty = bars + 1;   // item n's S products done and every warp has its number
  uint64_t* k_full = bars + 2;    // [2]
  uint64_t* k_empty = bars + 4;   // [2]
  uint64_t* v_full = bars + 6;    // [2]
  uint64_t* v_empty = bars + 8;   // [2]
  uint64_t* s_full = bars + 10;   // [2] per tile: S of a block in TMEM
  uint64_t* p_full = bars + 12;   // [2] per tile: P of a block in TMEM
  uint64_t* pv_done = bars + 14;  // [2] per tile: P V of a block complete
  uint64_t* drain = bars + 16;
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(bars + 17);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_holder + 1);
  volatile int* item_ring = reinterpret_cast<volatile int*>(tmem_holder + 2);   // [4]

  const int warp = warp_id(), lane = lane_id();
  const int nq = (T + 127) / 128;
  const long long wlim = wait_limit_or_default(wait_cycles);

  if (threadIdx.x == 0) {
    mbar_init(q_full, 1);
    mbar_init(q_empty, 1 + 8);   // the MMA commit and one arrival per softmax warp
    for (int i = 0; i < 2; ++i) {
      mbar_init(&k_full[i], 1); mbar_init(&k_empty[i], 1);
      mbar_init(&v_full[i], 1); mbar_init(&v_empty[i], 1);
      mbar_init(&s_full[i], 1); mbar_init(&p_full[i], 128); mbar_init(&pv_done[i], 1);
    }
    mbar_init(drain, 1);
    *abort_flag = 0;
    fence_barrier_init();
    tma_prefetch_desc(&tq);
    tma_prefetch_desc(&tk);
    tma_prefetch_desc(&tv);
  }
  if (warp == 1) {
    tmem_alloc(tmem_holder, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_holder;

  if (warp < 4) asm volatile("setmaxnreg.dec.sync.aligned.u32 56;\n" ::: "memory");
  if (warp == 0) {
    if (lane == 0) {
      // -------------------------------------------------------------- TMA
      bool ok = true;
      int g = 0, last_q = -1;   // ring position of the next K/V block; last item whose Q was loaded
      for (int n = 0;; ++n) {
        // the previous item's Q is no longer read and every warp has its number
        if (n > 0 && !mbar_wait_t<kFine>(q_empty, (n - 1) & 1, abort_flag, err, wlim)) { ok = false; break; }
        int idx = sched ? atomicAdd(sched, 1) : n * static_cast<int>(gridDim.x) + static_cast<int>(blockIdx.x);
        if (idx >= n_items) idx = -1;
        item_ring[n & 3] = idx;
        if (idx < 0) {
          mbar_arrive(q_full);   // end marker: releases the ring entry
          break;
        }
        const FwdItem it = fwd_item(idx, nq, H, Hkv, kvs, wl);
        mbar_arrive_expect_tx(q_full, it.hasB ? 2 * TF_BUF : TF_BUF);
        tma_load_3d(sQ, &tq, q_full, 0, it.qtA * 128, it.bh);
        tma_load_3d(sQ + TF_TILE, &tq, q_full, 64, it.qtA * 128, it.bh);
        if (it.hasB) {
          tma_load_3d(sQ + TF_BUF, &tq, q_full, 0, it.qtA * 128 + 128, it.bh);
          tma_load_3d(sQ + TF_BUF + TF_TILE, &tq, q_full, 64, it.qtA * 128 + 128, it.bh);
        }
        last_q = n;
        for (int j = 0; j < it.nkv; ++j) {
          const int s = g & 1;
          const uint32_t par = (g >> 1) & 1;
          const int kc = (it.j0 + j) * 128;
          if (!mbar_wait_t<kFine>(&k_empty[s], par ^ 1u, abort_flag, err, wlim)) { ok = false; break; }
          mbar_arrive_expect_tx(&k_full[s], TF_BUF);
          tma_load_3d(sK + s * TF_BUF, &tk, &k_full[s], 0, kc, it.bkv);
          tma_load_3d(sK + s * TF_BUF + TF_TILE, &tk, &k_full[s], 64, kc, it.bkv);
          if (!mbar_wait_t<kFine>(&v_empty[s], par ^ 1u, abort_flag, err, wlim)) {
            // K of this block is in flight: count it, V is not
            for (uint32_t i = 0; i < (1u << 20) && !mbar_try_wait(&k_full[s], par); ++i) {}
            ok = false;
            break;
          }
          mbar_arrive_expect_tx(&v_full[s], TF_BUF);
          tma_load_3d(sV + s * TF_BUF, &tv, &v_full[s], 0, kc, it.bkv);
          tma_load_3d(sV + s * TF_BUF + TF_TILE, &tv, &v_full[s], 64, kc, it.bkv);
          ++g;
        }
        if (!ok) break;
      }
      if (!ok) {
        // let the copies already started land before the CTA exits
        if (last_q >= 0)
          for (uint32_t i = 0; i < (1u << 20) && !mbar_try_wait(q_full, last_q & 1); ++i) {}
        for (int x = (g > 2 ? g - 2 : 0); x < g; ++x) {
          for (uint32_t i = 0; i < (1u << 20) && !mbar_try_wait(&k_full[x & 1], (x >> 1) & 1); ++i) {}
          for (uint32_t i = 0; i < (1u << 20) && !mbar_try_wait(&v_full[x & 1], (x >> 1) & 1); ++i) {}
        }
      }
    }
  } else if (warp == 1) {
    // -------------------------------------------------------------- MMA
    // the whole warp, converged; one lane issues
    const bool leader = elect_lane();
    const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
    auto wait1 = [&](uint64_t* bar, uint32_t par) -> bool {
      return __all_sync(0xffffffffu, mbar_wait_t<kFine>(bar, par, abort_flag, err, wlim));
    };
    constexpr uint32_t IDESC_S = make_idesc(1, 128, false, false);
    constexpr uint32_t IDESC_O = make_idesc(1, 128, false, true);
    // The descriptors of a product are its first one plus the byte offset / 16
    // (the start address field).
    // S_t = Q_t K^T (K in ring slot ks) into TMEM columns 128 t
    auto issue_s = [&](int t, int ks) {
      uint64_t dq = smem_desc_sw128(smem_u32(sQ + t * TF_BUF), 16, 1024);
      uint64_t dk = smem_desc_sw128(smem_u32(sK + ks * TF_BUF), 16, 1024);
#pragma unroll
      for (int kk = 0; kk < 8; ++kk) {
        const uint32_t off16 = ((kk >> 2) * TF_TILE + (kk & 3) * 32) >> 4;
        umma_f16_by(leader, tm + t * 128, dq + off16, dk + off16, IDESC_S, kk > 0 ? 1u : 0u);
      }
      umma_commit_by(leader, &s_full[t]);
    };
    // O_t (+)= P_t V (V in ring slot vs), P_t from TMEM (16 keys = 8 packed columns per step)
    auto issue_pv = [&](int t, int vs, bool acc) {
      uint64_t dv = smem_desc_sw128(smem_u32(sV + vs * TF_BUF), TF_TILE, 1024);
#pragma unroll
      for (int kk = 0; kk < 8; ++kk)
        umma_f16_tmem_a_by(leader, tm + 256 + t * 128, tm + t * 128 + kk * 8, dv + ((kk * 2048) >> 4), IDESC_O,
                        (acc || kk > 0) ? 1u : 0u);
      umma_commit_by(leader, &pv_done[t]);
    };
    bool ok = true;
    int g0 = 0;                  // ring position of the item's first key block
    uint32_t npv[2] = {0u, 0u};  // P V products issued per tile so far
    for (int n = 0; ok; ++n) {
      if (!wait1(q_full, n & 1)) { ok = false; break; }
      const int idx = __shfl_sync(0xffffffffu, item_ring[n & 3], 0);
      if (idx < 0) break;
      const FwdItem it = fwd_item(idx, nq, H, Hkv, kvs, wl);
      // S of the first block on both tiles, each once its previous P V (which
      // reads P from the same columns) has completed
      if (!wait1(&k_full[g0 & 1], (g0 >> 1) & 1)) { ok = false; break; }
      for (int t = 0; t < 2 && ok; ++t) {
        if (t == 1 && !it.hasB) break;
        if (npv[t] > 0 && !wait1(&pv_done[t], (npv[t] - 1) & 1)) { ok = false; break; }
        tc_fence_after();
        issue_s(t, g0 & 1);
      }
      if (!ok) break;
      if (it.nkv == 1) umma_commit_by(leader, q_empty);   // the item's last S
      umma_commit_by(leader, &k_empty[g0 & 1]);
      for (int j = 0; j < it.nkv && ok; ++j) {
        const int gj = g0 + j;
        const int s = gj & 1;
        const int s1 = (gj + 1) & 1;
        if (!wait1(&v_full[s], (gj >> 1) & 1)) { ok = false; break; }
        if (j + 1 < it.nkv && !wait1(&k_full[s1], ((gj + 1) >> 1) & 1)) { ok = false; break; }
        // per tile: O += P V_j, then S of the next block over P once that product
        // has read it (tile B's softmax trails tile A's, so A goes first)
        for (int t = 0; t < 2; ++t) {
          const int nkv_t = t ? it.nkvB : it.nkvA;
          if (j >= nkv_t) continue;
          if (!wait1(&p_full[t], npv[t] & 1)) { ok = false; break; }
          tc_fence_after();
          issue_pv(t, s, j > 0);
          ++npv[t];
          if (j + 1 < nkv_t) {
            if (!wait1(&pv_done[t], (npv[t] - 1) & 1)) { ok = false; break; }
            tc_fence_after();
            issue_s(t, s1);
            if (j + 1 == it.nkv - 1) umma_commit_by(leader, q_empty);   // the item's last S
          }
        }
        if (!ok) break;
        umma_commit_by(leader, &v_empty[s]);
        if (j + 1 < it.nkv) umma_commit_by(leader, &k_empty[s1]);
      }
      g0 += it.nkv;
    }
    umma_commit_by(leader, drain);
    for (uint32_t i = 0; i < (1u << 22) && !mbar_try_wait(drain, 0); ++i) {}
  } else if (warp >= 4) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 224;\n" ::: "memory");
    // ---------------------------------------------------------- softmax
    const int tile = (warp - 4) >> 2;           // 0: A, 1: B
    const int quarter = warp & 3;
    const int r = quarter * 32 + lane;
    const uint32_t lane_base = static_cast<uint32_t>(quarter * 32) << 16;
    const uint32_t t_s = tmem + lane_base + tile * 128;
    const uint32_t t_o = tmem + lane_base + 256 + tile * 128;
    const uint64_t sl2 = f2_pack(scale_log2, scale_log2);
    bool ok = true;
    uint32_t nblk = 0;   // S blocks consumed on this tile so far
    auto wait_all = [&](uint64_t* bar, uint32_t par) -> bool {
      const bool got = mbar_wait_t<kFine>(bar, par, abort_flag, err, wlim);
      __syncwarp();
      return __all_sync(0xffffffffu, got);
    };
    for (int n = 0; ok; ++n) {
      if (!wait_all(q_full, n & 1)) { ok = false; break; }
      const int idx = item_ring[n & 3];
      __syncwarp();
      if (lane == 0) mbar_arrive(q_empty);   // this warp has the item number
      if (idx < 0) break;
      const FwdItem it = fwd_item(idx, nq, H, Hkv, kvs, wl);
      if (tile == 1 && !it.hasB) continue;
      const int qt = it.qtA + tile;
      const int q0 = qt * 128;
      const int q = q0 + r;
      const int nkv_t = tile ? it.nkvB : it.nkvA;
      float m_ref = -INFINITY, l = 0.f;   // reference max (log2 units) and row sum relative to it
      for (int j = 0; j < nkv_t && ok; ++j) {
        if (!wait_all(&s_full[tile], nblk & 1)) { ok = false; break; }
        ++nblk;
        tc_fence_after();
        // the whole S row at once
        uint32_t sr[128];
        {
          uint32_t (&r0)[32] = *reinterpret_cast<uint32_t(*)[32]>(&sr[0]);
          uint32_t (&r1)[32] = *reinterpret_cast<uint32_t(*)[32]>(&sr[32]);
          uint32_t (&r2)[32] = *reinterpret_cast<uint32_t(*)[32]>(&sr[64]);
          uint32_t (&r3)[32] = *reinterpret_cast<uint32_t(*)[32]>(&sr[96]);
          tmem_load32_async(t_s, r0);
          tmem_load32_async(t_s + 32, r1);
          tmem_load32_async(t_s + 64, r2);
          tmem_load32_async(t_s + 96, r3);
          tmem_wait_ld();
        }
        const int kbase = (it.j0 + j) * 128;
        const bool diag = it.j0 + j == qt, edge = (kbase + 128 > T) || (kbase < q0 + 127 - wl);
        if (diag && !edge) {
          // causal diagonal block: only the keys above the row are masked, so
          // per element in one 32-key chunk, whole chunks beyond it
          switch (quarter) {
            case 0: causal_mask_row<0>(sr, lane); break;
            case 1: causal_mask_row<1>(sr, lane); break;
            case 2: causal_mask_row<2>(sr, lane); break;
            default: causal_mask_row<3>(sr, lane); break;
          }
        } else if (diag || edge) {
          // ragged tail or window edge: masked scores become -inf
#pragma unroll
          for (int k = 0; k < 128; ++k) {
            const int key = kbase + k;
            if (key > q || key >= T || key < q - wl) sr[k] = __float_as_uint(-INFINITY);
          }
        }
        // block max of the raw scores (the scale is positive), eight independent
        // chains of three-input maxima (two new scores per instruction)
        float mx8[8];
#pragma unroll
        for (int t = 0; t < 8; ++t) mx8[t] = fmaxf(__uint_as_float(sr[2 * t]), __uint_as_float(sr[2 * t + 1]));
#pragma unroll
        for (int k = 16; k < 128; k += 16) {
#pragma unroll
          for (int t = 0; t < 8; ++t)
            mx8[t] = fmax3(mx8[t], __uint_as_float(sr[k + 2 * t]), __uint_as_float(sr[k + 2 * t + 1]));
        }
        const float mraw = fmax3(fmax3(mx8[0], mx8[1], mx8[2]), fmax3(mx8[3], mx8[4], mx8[5]), fmaxf(mx8[6], mx8[7]));
        const float mblk = mraw * scale_log2;
        const bool move = mblk > m_ref + TF_RESCALE;   // true on the first block with a visible key
        const float m_new = move ? mblk : m_ref;
        // 1 when the reference stays, 0 when it leaves -inf; a row that has seen
        // only masked scores (window edge) keeps -inf and offsets by 0 below
        const bool none = m_new == -INFINITY;
        const float factor = none ? 1.f : ex2_approx(m_ref - m_new);
        // O holds the products of blocks < j (S of this block was issued after
        // the last of them completed), so it may be rescaled now
        if (j >= 1 && __any_sync(0xffffffffu, move)) {
#pragma unroll 1
          for (int c = 0; c < 4; ++c) {
            uint32_t ra[32];
            tmem_load32_async(t_o + c * 32, ra);
            tmem_wait_ld();
#pragma unroll
            for (int k = 0; k < 32; ++k) ra[k] = __float_as_uint(__uint_as_float(ra[k]) * factor);
            tmem_store32(t_o + c * 32, ra);
          }
        }
        // probabilities relative to the reference (masked scores give 0), row sum,
        // bf16 P over the first 64 columns of S
        const float m_off = none ? 0.f : m_new;
        const uint64_t nb2 = f2_pack(-m_off, -m_off);
        uint64_t rs2 = f2_pack(0.f, 0.f);
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          uint32_t pk[32];
#pragma unroll
          for (int k = 0; k < 64; k += 8) {
            float p[8];
#pragma unroll
            for (int e = 0; e < 8; e += 2) {
              float x0, x1;
              f2_unpack(f2_fma(f2_pack(__uint_as_float(sr[c * 64 + k + e]), __uint_as_float(sr[c * 64 + k + e + 1])),
                               sl2, nb2),
                        x0, x1);
              if (e < ((k & 8) ? GPT_FWD_MUFU_ODD : GPT_FWD_MUFU_EVEN)) {
                p[e] = ex2_approx(x0);
                p[e + 1] = ex2_approx(x1);
              } else {
                f2_unpack(f2_exp2_poly(f2_pack(fmaxf(x0, -126.f), fmaxf(x1, -126.f))), p[e], p[e + 1]);
              }
            }
#pragma unroll
            for (int e = 0; e < 8; e += 2) {
              rs2 = f2_add(rs2, f2_pack(p[e], p[e + 1]));
              pk[(k + e) >> 1] = pack_bf16x2(p[e], p[e + 1]);
            }
          }
          tmem_store32(t_s + c * 32, pk);
        }
        asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
        tc_fence_before();
        mbar_arrive(&p_full[tile]);
        float rs0, rs1;
        f2_unpack(rs2, rs0, rs1);
        l = l * factor + (rs0 + rs1);
        m_ref = m_new;
      }
      // epilogue: O / l once the last P V has landed
      if (ok) ok = wait_all(&pv_done[tile], (nblk - 1) & 1);
      if (ok) {
        tc_fence_after();
        const int b = it.bh / H, h = it.bh - (it.bh / H) * H;
        const float inv = 1.f / l;
        const int w0 = q0 + quarter * 32;   // the warp's first row
        const long long pitch = static_cast<long long>(H) * 128;
        bf16* orow = o + (static_cast<long long>(b) * T + w0) * pitch + h * 128;
#pragma unroll 1
        for (int c = 0; c < 128; c += 32)
          store_rows<32>(t_o + c, inv, sOut + (warp - 4) * 2048, orow + c, pitch, T - w0);
        if (q < T) lse[static_cast<long long>(it.bh) * T + q] = (m_ref + log2f(l)) * 0.69314718055994531f;
        // O of this tile has been read: the next item's first P V may overwrite it
        tc_fence_before();
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// bits 0 .. n - 1
__device__ __forceinline__ uint32_t low_bits(int n) { return n <= 0 ? 0u : n >= 32 ? ~0u : (1u << n) - 1u; }

// Scores whose bit is clear become -inf.
__device__ __forceinline__ void mask_scores(uint32_t (&x)[32], uint32_t seen) {
#pragma unroll
  for (int k = 0; k < 32; ++k)
    if (!(seen & (1u << k))) x[k] = __float_as_uint(-INFINITY);
}

// Maximum of 32 scores, four chains of three-input maxima.
__device__ __forceinline__ float max32(const uint32_t (&x)[32], float m) {
  float c[4];
#pragma unroll
  for (int t = 0; t < 4; ++t) c[t] = fmaxf(__uint_as_float(x[2 * t]), __uint_as_float(x[2 * t + 1]));
#pragma unroll
  for (int k = 8; k < 32; k += 8) {
#pragma unroll
    for (int t = 0; t < 4; ++t) c[t] = fmax3(c[t], __uint_as_float(x[k + 2 * t]), __uint_as_float(x[k + 2 * t + 1]));
  }
  return fmax3(fmax3(c[0], c[1], c[2]), c[3], m);
}

// -------------------------------------- packed forward on tcgen05 / TMEM
//
// Persistent, two blocks an SM, each with its own 128-query tiles of one head,
// taken in turn; the two hide each other's softmax and products, start and
// end of a tile.  (Pairs of tiles that share their key blocks in one block, as
// above, leave a fifth of the softmax time idle here: neighbours seldom see
// equally many blocks.  Kernel times, 16,384 tokens of chats of 24 to 1024, 10
// heads over 2: 79 us against 90; 32,768 of documents of 128 to 2048, 10 heads:
// 186 against 205, 500 TFLOP/s of visible pairs, 670 of the blocks it runs.)  A
// tile takes about 4.4 us and 2.35 us a key block, of which S = Q K^T alone fills half
// the shared-memory bandwidth (both operands of a 128 x 128 product): bound by
// the chain S, softmax, P V of the two tiles, with the tensor pipe 36% busy
// and 31% of the issue slots used.  Two threads a row measured the same.
// 192 threads:
//   warps 0..3  softmax, one query row (TMEM lane) per thread, as above; then
//               O / l and the log-sum-exp
//   warp 4      TMA: takes the items and publishes them in a shared ring, loads
//               Q, and K_j and V_j through one buffer each: K_j+1 comes while
//               the softmax of block j runs, V_j+1 while that of j + 1 does
//   warp 5      TMEM owner and MMA issuer: S = Q K_j^T into columns [0,128),
//               O += P V_j into [128,256), P over the first 64 columns of S
constexpr int PF_STAGE = 8192;   // output rows: 2 KB for each softmax warp
constexpr int PF_SMEM = 3 * TF_BUF + PF_STAGE + 256;

template <bool kFine>
__global__ void __launch_bounds__(192, 2)
    attn_packed_fwd_kernel(const __grid_constant__ CUtensorMap tq, const __grid_constant__ CUtensorMap tk,
                           const __grid_constant__ CUtensorMap tv, bf16* __restrict__ o, float* __restrict__ lse,
                           int H, int Hkv, int T, float scale_log2, int* err, long long wait_cycles,
                           const __grid_constant__ PackedArgs pk) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  // the 128-byte-swizzled tiles need a 1024-byte-aligned base, which the
  // dynamic shared memory window provides; refuse to run otherwise
  if (smem_u32(smem_raw) & 1023u) {
    if (threadIdx.x == 0 && err) atomicOr(err, ERRF_SHAPE);
    return;
  }
  uint8_t* sQ = smem_raw;
  uint8_t* sK = smem_raw + TF_BUF;
  uint8_t* sV = smem_raw + 2 * TF_BUF;
  uint8_t* sOut = smem_raw + 3 * TF_BUF;
  uint4* answer = reinterpret_cast<uint4*>(smem_raw + 3 * TF_BUF + PF_STAGE);   // next_block_ask's
  uint64_t* bars = reinterpret_cast<uint64_t*>(answer + 1);
  uint64_t* q_full = bars + 0;    // Q of item n landed (or the end marker)
  uint64_t* q_empty = bars + 1;   // item n's S products done and every softmax warp has its fields
  uint64_t* k_full = bars + 2;
  uint64_t* k_empty = bars + 3;
  uint64_t* v_full = bars + 4;
  uint64_t* v_empty = bars + 5;
  uint64_t* s_full = bars + 6;    // S of a block in TMEM
  uint64_t* p_full = bars + 7;    // P of a block in TMEM
  uint64_t* pv_done = bars + 8;   // P V of a block complete
  uint64_t* drain = bars + 9;
  uint64_t* answered = bars + 10;
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(bars + 11);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_holder + 1);
  // [4][4]: head (-1: end), tile, first key block
  volatile int* item_ring = reinterpret_cast<volatile int*>(tmem_holder + 2);

  const int warp = warp_id(), lane = lane_id();
  const long long wlim = wait_limit_or_default(wait_cycles);

  if (threadIdx.x == 0) {
    mbar_init(q_full, 1);
    mbar_init(q_empty, 1 + 4);   // the MMA commit and one arrival per softmax warp
    mbar_init(k_full, 1); mbar_init(k_empty, 1);
    mbar_init(v_full, 1); mbar_init(v_empty, 1);
    mbar_init(s_full, 1); mbar_init(p_full, 128); mbar_init(pv_done, 1);
    mbar_init(drain, 1);
    mbar_init(answered, 1);
    *abort_flag = 0;
    fence_barrier_init();
    tma_prefetch_desc(&tq);
    tma_prefetch_desc(&tk);
    tma_prefetch_desc(&tv);
  }
  if (warp == 5) {
    tmem_alloc(tmem_holder, 256);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_holder;
  chain_wait();
  // positions that hold sequences; a plan of another T is refused
  const PlanSizes plan = plan_sizes(pk.meta, T);
  const int Tv = plan.valid;
  if (!plan.fits && blockIdx.x == 0 && threadIdx.x == 0 && err) atomicOr(err, ERRF_SHAPE);

  if (warp == 4) {
    if (lane == 0) {
      // -------------------------------------------------------------- TMA
      // item number and fields are fetched one item ahead, so that the answer's
      // and the plan's latency hides behind the current item's loads
      const int entries = plan.fwd, n_items = entries * H;
      int nx_h = -1;
      int2 nx = make_int2(0, 0);
      bool asked = false;
      uint32_t answers = 0;
      // a block for every tile: those past the sequences, after the others, to clear
      const int tiles = (Tv + 127) / 128, past = plan.fits && pk.clear ? (T + 127) / 128 - tiles : 0;
      auto fetch = [&](int idx) {   // false: a block without work
        if (idx < n_items) {
          const int h = idx / entries;
          nx = __ldg(pk.fwd + (idx - h * entries));
          if (!fwd_entry_ok(nx, Tv, err)) return false;
          nx_h = h;
          return true;
        }
        idx -= n_items;
        if (idx >= past * H) return false;
        nx_h = idx / past;
        nx.x = tiles + idx - nx_h * past;
        nx.y = nx.x + 1;   // no key block
        return true;
      };
      auto take = [&] {   // false: the wait expired
        nx_h = -1;
        while (asked) {
          if (!mbar_wait_t<kFine>(answered, answers & 1, abort_flag, err, wlim)) return false;
          ++answers;
          asked = false;
          const int idx = next_block_answer(answer);
          if (idx < 0 || fetch(idx)) break;
          next_block_ask(answer, answered);
          asked = true;
        }
        return true;
      };
      fetch(blockIdx.x);
      bool ok = true;
      uint32_t g = 0;     // key blocks loaded so far
      int last_q = -1;    // last item whose Q was loaded
      for (int n = 0;; ++n) {
        // the previous item's Q is no longer read and every warp has its fields
        if (n > 0 && !mbar_wait_t<kFine>(q_empty, (n - 1) & 1, abort_flag, err, wlim)) { ok = false; break; }
        volatile int* f = item_ring + 4 * (n & 3);
        const int h = nx_h, qt = nx.x, j0 = nx.y;
        f[0] = h; f[1] = qt; f[2] = j0;
        if (h < 0) {
          mbar_arrive(q_full);   // end marker: releases the ring entry
          break;
        }
        next_block_ask(answer, answered);
        asked = true;
        const int hk = h / (H / Hkv);
        if (j0 > qt) {   // rows to clear: no loads
          mbar_arrive(q_full);
          if (!take()) { ok = false; break; }
          continue;
        }
        mbar_arrive_expect_tx(q_full, TF_BUF);
        tma_load_3d(sQ, &tq, q_full, 0, qt * 128, h);
        tma_load_3d(sQ + TF_TILE, &tq, q_full, 64, qt * 128, h);
        last_q = n;
        for (int j = j0; j <= qt; ++j) {
          if (!mbar_wait_t<kFine>(k_empty, (g & 1) ^ 1u, abort_flag, err, wlim)) { ok = false; break; }
          mbar_arrive_expect_tx(k_full, TF_BUF);
          tma_load_3d(sK, &tk, k_full, 0, j * 128, hk);
          tma_load_3d(sK + TF_TILE, &tk, k_full, 64, j * 128, hk);
          if (!mbar_wait_t<kFine>(v_empty, (g & 1) ^ 1u, abort_flag, err, wlim)) {
            // K of this block is in flight, V is not
            for (uint32_t i = 0; i < (1u << 20) && !mbar_try_wait(k_full, g & 1); ++i) {}
            ok = false;
            break;
          }
          mbar_arrive_expect_tx(v_full, TF_BUF);
          tma_load_3d(sV, &tv, v_full, 0, j * 128, hk);
          tma_load_3d(sV + TF_TILE, &tv, v_full, 64, j * 128, hk);
          ++g;
          if (j == j0 && !take()) { ok = false; break; }
        }
        if (!ok) break;
      }
      if (!ok) {
        // let the copies already started land before the CTA exits
        if (asked)
          for (uint32_t i = 0; i < (1u << 20) && !mbar_try_wait(answered, answers & 1); ++i) {}
        if (last_q >= 0)
          for (uint32_t i = 0; i < (1u << 20) && !mbar_try_wait(q_full, last_q & 1); ++i) {}
        if (g > 0) {
          for (uint32_t i = 0; i < (1u << 20) && !mbar_try_wait(k_full, (g - 1) & 1); ++i) {}
          for (uint32_t i = 0; i < (1u << 20) && !mbar_try_wait(v_full, (g - 1) & 1); ++i) {}
        }
      }
    }
  } else if (warp == 5) {
    // -------------------------------------------------------------- MMA
    // the whole warp, converged; one lane issues
    const bool leader = elect_lane();
    const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
    auto wait1 = [&](uint64_t* bar, uint32_t par) -> bool {
      return __all_sync(0xffffffffu, mbar_wait_t<kFine>(bar, par, abort_flag, err, wlim));
    };
    constexpr uint32_t IDESC_S = make_idesc(1, 128, false, false);
    constexpr uint32_t IDESC_O = make_idesc(1, 128, false, true);
    const uint64_t dq = smem_desc_sw128(smem_u32(sQ), 16, 1024), dk = smem_desc_sw128(smem_u32(sK), 16, 1024);
    const uint64_t dv = smem_desc_sw128(smem_u32(sV), TF_TILE, 1024);
    bool ok = true;
    uint32_t g = 0;   // key blocks done so far
    for (int n = 0; ok; ++n) {
      if (!wait1(q_full, n & 1)) break;
      const volatile int* f = item_ring + 4 * (n & 3);
      const int h = __shfl_sync(0xffffffffu, f[0], 0), qt = __shfl_sync(0xffffffffu, f[1], 0);
      const int j0 = __shfl_sync(0xffffffffu, f[2], 0);
      if (h < 0) break;
      if (j0 > qt) umma_commit_by(leader, q_empty);
      for (int j = j0; j <= qt; ++j, ++g) {
        // S over P of the block before, once its product has read it
        if (!wait1(k_full, g & 1) || (g > 0 && !wait1(pv_done, (g - 1) & 1))) { ok = false; break; }
        tc_fence_after();
#pragma unroll
        for (int kk = 0; kk < 8; ++kk) {
          const uint32_t off16 = ((kk >> 2) * TF_TILE + (kk & 3) * 32) >> 4;
          umma_f16_by(leader, tm, dq + off16, dk + off16, IDESC_S, kk > 0 ? 1u : 0u);
        }
        umma_commit_by(leader, s_full);
        umma_commit_by(leader, k_empty);
        if (j == qt) umma_commit_by(leader, q_empty);   // the item's last S
        if (!wait1(v_full, g & 1)) { ok = false; break; }
        const int past = Tv - j * 128;   // rows of V from here on belong to no sequence
        if (Tv < T && past < 128) {
          for (int x = past * 16 + lane; x < 128 * 16; x += 32)
            *reinterpret_cast<uint4*>(sV + ((x >> 3) & 1) * TF_TILE + (x >> 4) * 128 + (x & 7) * 16) =
                make_uint4(0u, 0u, 0u, 0u);
          fence_proxy_async_smem();
          __syncwarp();
        }
        if (!wait1(p_full, g & 1)) { ok = false; break; }
        tc_fence_after();
        // P from TMEM, 16 keys = 8 packed columns per step
#pragma unroll
        for (int kk = 0; kk < 8; ++kk)
          umma_f16_tmem_a_by(leader, tm + 128, tm + kk * 8, dv + ((kk * 2048) >> 4), IDESC_O,
                             (j > j0 || kk > 0) ? 1u : 0u);
        umma_commit_by(leader, pv_done);
        umma_commit_by(leader, v_empty);
      }
    }
    umma_commit_by(leader, drain);
    for (uint32_t i = 0; i < (1u << 22) && !mbar_try_wait(drain, 0); ++i) {}
  } else {
    // ---------------------------------------------------------- softmax
    const uint32_t lane_base = static_cast<uint32_t>(warp * 32) << 16;
    const uint32_t t_s = tmem + lane_base, t_o = tmem + lane_base + 128;
    const uint64_t sl2 = f2_pack(scale_log2, scale_log2);
    bool ok = true;
    uint32_t g = 0;   // S blocks consumed so far
    auto wait_all = [&](uint64_t* bar, uint32_t par) -> bool {
      return __all_sync(0xffffffffu, mbar_wait_t<kFine>(bar, par, abort_flag, err, wlim));
    };
    for (int n = 0; ok; ++n) {
      if (!wait_all(q_full, n & 1)) break;
      const volatile int* f = item_ring + 4 * (n & 3);
      const int h = f[0], qt = f[1], j0 = f[2];
      __syncwarp();
      if (lane == 0) mbar_arrive(q_empty);   // this warp has the fields
      if (h < 0) break;
      const int w0 = qt * 128 + warp * 32, q = w0 + lane;   // the warp's first row, this thread's
      if (pk.clear && w0 + 32 > Tv) {   // rows past the sequences, those of a tile before it is computed
        if (pk.clear & kClearO)
          for (int row = max(w0, Tv) + (lane >> 4); row < min(w0 + 32, T); row += 2)
            *reinterpret_cast<uint4*>(o + row * pk.o_tok + h * pk.o_head + (lane & 15) * 8) = make_uint4(0, 0, 0, 0);
        if ((pk.clear & kClearLse) && q >= Tv && q < T) lse[static_cast<long long>(h) * T + q] = 0.f;
      }
      if (j0 > qt) continue;
      const int lo = q < Tv ? __ldg(pk.lo + q) : 0;         // first key of the row
      const int lo_max = __reduce_max_sync(0xffffffffu, lo);
      float m_ref = -INFINITY, l = 0.f;   // reference max (log2 units) and row sum relative to it
      for (int j = j0; j <= qt; ++j, ++g) {
        if (!wait_all(s_full, g & 1)) { ok = false; break; }
        tc_fence_after();
        const int kbase = j * 128;
        const bool diag = j == qt;
        float mraw = -INFINITY;           // block max of the raw scores (the scale is positive)
        // Masked blocks come at every sequence boundary.  Straight-line code for a
        // row and for each kind of mask, as in the kernel above, left the softmax
        // warps a fifth of their time without instructions, so the row is read
        // from TMEM 32 scores at a time, now and again for P, by loops that stay
        // in the instruction cache, mask by bits and skip the chunks that no row
        // of the warp sees (chats: 90 us instead of 103 when this came in).
        // Keys past the last sequence lie above every row of the diagonal block.
        const bool masked = diag || kbase < lo_max;
        // keys that this row sees, from kbase on: first .. end - 1
        const int first = lo - kbase, end = q + 1 - kbase;
        auto seen_of = [&](int c) { return low_bits(end - 32 * c) & ~low_bits(first - 32 * c); };
        if (!masked) {
          uint32_t xa[32], xb[32];
#pragma unroll 1
          for (int c = 0; c < 4; c += 2) {
            tmem_load32_async(t_s + 32 * c, xa);
            tmem_load32_async(t_s + 32 * c + 32, xb);
            tmem_wait_ld();
            mraw = max32(xb, max32(xa, mraw));
          }
        } else {
#pragma unroll 1
          for (int c = 0; c < 4; ++c) {
            const uint32_t seen = seen_of(c);
            if (__any_sync(0xffffffffu, seen != 0)) {
              uint32_t x[32];
              tmem_load32_async(t_s + 32 * c, x);
              tmem_wait_ld();
              mask_scores(x, seen);
              mraw = max32(x, mraw);
            }
          }
        }
        const float mblk = mraw * scale_log2;
        const bool move = mblk > m_ref + TF_RESCALE;   // true on the first block with a visible key
        const float m_new = move ? mblk : m_ref;
        // 1 when the reference stays, 0 when it leaves -inf; a row that has seen
        // only masked scores (window edge) keeps -inf and offsets by 0 below
        const bool none = m_new == -INFINITY;
        const float factor = none ? 1.f : ex2_approx(m_ref - m_new);
        // O holds the products of blocks < j (S of this block was issued after
        // the last of them completed), so it may be rescaled now
        if (j > j0 && __any_sync(0xffffffffu, move)) {
#pragma unroll 1
          for (int c = 0; c < 4; ++c) {
            uint32_t ra[32];
            tmem_load32_async(t_o + c * 32, ra);
            tmem_wait_ld();
#pragma unroll
            for (int k = 0; k < 32; ++k) ra[k] = __float_as_uint(__uint_as_float(ra[k]) * factor);
            tmem_store32(t_o + c * 32, ra);
          }
        }
        // probabilities relative to the reference (masked scores give 0), row sum,
        // bf16 P over the first 64 columns of S
        const float m_off = none ? 0.f : m_new;
        const uint64_t nb2 = f2_pack(-m_off, -m_off);
        uint64_t rs2 = f2_pack(0.f, 0.f);
        auto probabilities = [&](const uint32_t (&x)[32], int c) {
          uint32_t pk[16];
#pragma unroll
          for (int k = 0; k < 32; k += 2) {
            float x0, x1;
            f2_unpack(f2_fma(f2_pack(__uint_as_float(x[k]), __uint_as_float(x[k + 1])), sl2, nb2), x0, x1);
            const float p0 = ex2_approx(x0), p1 = ex2_approx(x1);
            rs2 = f2_add(rs2, f2_pack(p0, p1));
            pk[k >> 1] = pack_bf16x2(p0, p1);
          }
          tmem_store16(t_s + 16 * c, pk);
        };
        if (!masked) {
          uint32_t xa[32], xb[32];
          tmem_load32_async(t_s, xa);
          tmem_landed(xa);
#pragma unroll 1
          for (int c = 0; c < 4; c += 2) {
            tmem_load32_async(t_s + 32 * c + 32, xb);
            probabilities(xa, c);
            tmem_landed(xb);
            if (c == 0) tmem_load32_async(t_s + 64, xa);
            probabilities(xb, c + 1);
            tmem_landed(xa);
          }
        } else {
#pragma unroll 1
          for (int c = 0; c < 4; ++c) {
            const uint32_t seen = seen_of(c);
            if (__any_sync(0xffffffffu, seen != 0)) {
              uint32_t x[32];
              tmem_load32_async(t_s + 32 * c, x);
              tmem_wait_ld();
              mask_scores(x, seen);
              probabilities(x, c);
            } else {
              uint32_t pk[16];
#pragma unroll
              for (int k = 0; k < 16; ++k) pk[k] = 0u;
              tmem_store16(t_s + 16 * c, pk);
            }
          }
        }
        asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
        tc_fence_before();
        mbar_arrive(p_full);
        float rs0, rs1;
        f2_unpack(rs2, rs0, rs1);
        l = l * factor + (rs0 + rs1);
        m_ref = m_new;
      }
      // epilogue: O / l once the last P V has landed
      if (ok) ok = wait_all(pv_done, (g - 1) & 1);
      if (ok) {
        tc_fence_after();
        const float inv = 1.f / l;
        bf16* orow = o + w0 * pk.o_tok + h * pk.o_head;
        float z = 0.f;
#pragma unroll 1
        for (int c = 0; c < 128; c += 32)
          z += store_rows<32, true>(t_o + c, inv, sOut + warp * 2048, orow + c, pk.o_tok, Tv - w0);
        uint32_t bad = __ballot_sync(0xffffffffu, q < Tv && !(z == 0.f));
        if (bad) {
          const float lse2 = m_ref + log2f(l);
          __syncwarp();   // the rows are stored
          for (; bad; bad &= bad - 1) {
            const int r = __ffs(bad) - 1;
            repair_o_row(pk, o, h, h / (H / Hkv), w0 + r, __shfl_sync(0xffffffffu, lo, r), j0 * 128,
                         min(qt * 128 + 127, Tv - 1), __shfl_sync(0xffffffffu, lse2, r), scale_log2);
          }
        }
        if (q < Tv) lse[static_cast<long long>(h) * T + q] = (m_ref + log2f(l)) * 0.69314718055994531f;
        // O has been read: the next item's first P V may overwrite it
        tc_fence_before();
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 5) {
    tc_fence_after();
    tmem_dealloc(tmem, 256);
  }
}

// ------------------------------------------------ backward on tcgen05 / TMEM
//
// Persistent: one CTA per SM takes work units, key blocks j and nkb - 1 - j
// of one batch*kv head (equal work under the causal mask), until none are
// left.  Units are numbered head-major, the longest of a head first, so the
// CTAs running at one time read the Q and dO of a few heads from L2; a
// scheduler word hands them out in that order (an atomic counter, zeroed
// before the launch), else each CTA takes every gridDim.x-th unit.  Each
// key block of a unit is one item.  The TMA warp publishes each item number in a shared
// ring with the K/V barrier; every other warp acknowledges it on the barrier
// that frees K/V, so no barrier phase can run two ahead of a waiter.  For each key block
// the CTA loops over the query heads of the kv group and, for each, the query
// blocks i >= j that see those keys (up to the last one inside the window);
// dK and dV add up over the whole loop.  The barrier phases run on across
// key blocks, so the next block's Q and dO loads start while the previous
// block's last products run, and its K and V load as soon as those are done.
// 512 threads in four warp groups (the first and the last give registers to
// the softmax groups: 72 / 168 / 168 / 96 per thread):
//   warp 0      TMA: Q_i through a two-slot ring; dO_i; K_j and V_j once per
//               key block (after the previous block's last product).
//   warp 1      TMEM owner and MMA issuer.  TMEM columns: [0,128) S^T_i and
//               dQ_i in turn; [128,256) dP^T_i, then P^T_i as packed bf16
//               (queries 0..63 at 128.., 64..127 at 192..); [256,384) dV;
//               [384,512) dK.  Per query block i:
//                 dV += P^T dO   once P_i is in TMEM (A from TMEM; then
//                                dO_{i+1} may load)
//                 dK += dS^T Q   once dS_i is in shared memory (then Q_{i+2}
//                                may load)
//                 dQ = dS K into [0,128) once S^T_{i+1} has been read (A is
//                                dS^T in shared memory read MN-major, so
//                                the queries land in the TMEM lanes)
//                 dP^T_{i+1} = V dO_{i+1}^T into [128,256)
//                 S^T_{i+2} = K Q_{i+2}^T into [0,128) once dQ_i has been read
//   warps 2, 3  idle
//   warps 4..11 softmax, two warps per TMEM lane quarter, each on 64 of the
//               128 query columns of its key rows: when dP^T_i lands, P_i
//               (computed during the previous block) over the dP^T columns the
//               warp has read, then dS'_i = P_i (dP_i - D) to shared memory
//               while dV runs; then S^T_{i+1}
//               and P_{i+1} while the tensor cores run block i's products.
//               1/sqrt(d) of dS = dS' / sqrt(d) is applied to dK and dQ.
//               After a key block's last products they write its dK and dV.
//   warps 12..15 dQ: one warp per TMEM lane quarter (lane = query), each
//               thread staging its query's row of dQ_i, 64 dims at a time, as
//               fp32 [32 queries][32 dims] boxes (eight 16-byte stores per
//               row) in a 32 KB buffer, and adding them into the fp32 dq
//               buffer by TMA reduce-add, so the reduction runs beside the
//               other warps' work.  (Adding each row with 16-byte vector
//               reductions from registers measured 0.925 ms against 0.68 ms
//               at B 16, H 10, T 2048.)

// The packed build takes single key blocks in the plan's order.  The rows' -lse
// and -D come with Q and dO by bulk copies (from attention_packed_dot_kernel's
// arrays of whole tiles), so that its softmax warps meet at no barrier; the
// masks of a 32-query chunk are bits; dK and dV rows go out through the dS
// tile; P stays in fp32 until dS is formed.  32,768 tokens of documents, 10 heads:
// kernel 360 us (650 TFLOP/s of visible pairs) where the power cap leaves the
// clock alone, 390 to 410 in passes back to back; bound by the softmax
// warps, about 1,800 cycles for P and as many for dS of the 4,400 a block takes.
// (In one build of it all: 466 us with staged lse and D, a form for each kind of
// mask and a lane for each stored row, against 350; P in fp32 cost 1 to 2%.)

// Row r, query columns 64*half .. 64*half+63 of a [128][128] bf16 tile kept as
// two 64-column halves of [128 rows][128 B] with the 128-byte swizzle (16-byte
// unit u of row r at u ^ (r & 7)); w holds the 64 values as packed pairs.
__device__ __forceinline__ void store_row_units(uint8_t* tile, const uint32_t (&w)[32], int half, int r) {
  uint8_t* row = tile + half * TF_TILE + r * 128;
#pragma unroll
  for (int u = 0; u < 8; ++u)
    *reinterpret_cast<uint4*>(row + ((u ^ (r & 7)) << 4)) = make_uint4(w[4 * u], w[4 * u + 1], w[4 * u + 2], w[4 * u + 3]);
}

constexpr int TB_STAGE = 32768;   // dQ staging: 4 warps x two [32 queries][32 dims] fp32 boxes
constexpr int TB_SMEM = 6 * TF_BUF + TB_STAGE + 2048 + 256;

// Copies `bytes` (a multiple of 16; both addresses too) to shared memory, counted on bar.
__device__ __forceinline__ void bulk_load(void* dst, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                   smem_u32(dst)),
               "l"(src), "r"(bytes), "r"(smem_u32(bar))
               : "memory");
}

// Query-block loop of key block j: nb query blocks j .. (window end) for each
// of the G query heads of the group.
struct BwdBlock {
  int bkv, kvrow, j, k0, nb, n_it, b, hk, G;   // kvrow: the k/v row (batch rows of kvs heads)
  __device__ __forceinline__ int q_block(int it) const { return j + it % nb; }
  __device__ __forceinline__ int q_head(int it) const { return hk * G + it / nb; }   // within the batch row
};

// Item idx: kv head idx / nq, key block idx mod nq.
__device__ __forceinline__ BwdBlock bwd_block(int idx, int H, int Hkv, int kvs, int nq, int wl) {
  BwdBlock k;
  k.bkv = idx / nq;
  const int j = idx - k.bkv * nq;
  const int bkv = k.bkv;
  k.j = j;
  k.k0 = j * 128;
  k.b = bkv / Hkv;
  k.hk = bkv - k.b * Hkv;
  k.kvrow = k.b * kvs + k.hk;
  k.G = H / Hkv;
  k.nb = min(nq - 1, (k.k0 + 127 + wl) / 128) - j + 1;
  k.n_it = k.G * k.nb;
  return k;
}

// A packed item as the TMA thread published it: kv head, key block, number of
// query blocks that see it.
__device__ __forceinline__ BwdBlock bwd_block_packed(const volatile int* f, int H, int Hkv) {
  BwdBlock k;
  k.b = 0;
  k.hk = f[0];
  k.j = f[1];
  k.nb = f[2];
  k.k0 = k.j * 128;
  k.bkv = k.kvrow = k.hk;
  k.G = H / Hkv;
  k.n_it = k.G * k.nb;
  return k;
}

template <bool kFine, bool kPacked>
__global__ void __launch_bounds__(512, 1)
    attn_bwd_tc_kernel(const __grid_constant__ CUtensorMap tq, const __grid_constant__ CUtensorMap tk,
                       const __grid_constant__ CUtensorMap tv, const __grid_constant__ CUtensorMap tdo,
                       const __grid_constant__ CUtensorMap tdq, const float* __restrict__ lse,
                       const float* __restrict__ Dv, bf16* __restrict__ dk, bf16* __restrict__ dv, int H, int Hkv,
                       int kvs, int T, int wl, float scale, int n_units, int* sched, int* err,
                       long long wait_cycles, const float* __restrict__ rk, const float2* __restrict__ rope,
                       bf16* __restrict__ dqkv_arg, const PackedArgs pa) {
  bf16* const dqkv = kPacked ? nullptr : dqkv_arg;   // packed: not built
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  // the 128-byte-swizzled tiles need a 1024-byte-aligned base, which the
  // dynamic shared memory window provides; refuse to run otherwise
  if (smem_u32(smem_raw) & 1023u) {
    if (threadIdx.x == 0 && err) atomicOr(err, ERRF_SHAPE);
    return;
  }
  uint8_t* sm = smem_raw;
  uint8_t* sK = sm;
  uint8_t* sV = sm + TF_BUF;
  uint8_t* sQ = sm + 2 * TF_BUF;     // two slots
  uint8_t* sdO = sm + 4 * TF_BUF;
  uint8_t* sdSt = sm + 5 * TF_BUF;
  uint8_t* sStage = sm + 6 * TF_BUF;
  float* lse_s = reinterpret_cast<float*>(sm + 6 * TF_BUF + TB_STAGE);   // [2][128]: -lse * log2(e)
  float* dd_s = lse_s + 256;                                              // [2][128]: -D
  uint64_t* bars = reinterpret_cast<uint64_t*>(sm + 6 * TF_BUF + TB_STAGE + 2048);
  uint64_t* kv_full = bars + 0;
  uint64_t* q_full = bars + 1;    // [2]
  uint64_t* q_empty = bars + 3;   // [2]
  uint64_t* do_full = bars + 5;
  uint64_t* do_empty = bars + 6;  // dV_i complete: dO_i and P_i are no longer read
  uint64_t* s_full = bars + 7;    // S^T_i in TMEM
  uint64_t* s_free = bars + 8;    // S^T_i read by the softmax warps
  uint64_t* dp_full = bars + 9;   // dP^T_i in TMEM
  uint64_t* p_ready = bars + 10;  // P_i in TMEM
  uint64_t* mm_done = bars + 11;  // dV, dK, dQ of block i complete
  uint64_t* dq_free = bars + 12;  // dQ_i read by the dQ warps
  uint64_t* drain = bars + 13;
  uint64_t* ds_ready = bars + 14; // dS_i in shared memory
  uint64_t* kv_empty = bars + 15; // an item's last products complete (K and V free) and every warp has its number
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(bars + 16);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_holder + 1);
  volatile int* item_ring = reinterpret_cast<volatile int*>(tmem_holder + 2);   // [4]
  volatile int* item_info = item_ring + 4;   // [4][4], packed items: bwd_block_packed's fields

  const int warp = warp_id(), lane = lane_id();
  const int nq = (T + 127) / 128;
  const long long wlim = wait_limit_or_default(wait_cycles);
  auto block_of = [&](int n, int idx) -> BwdBlock {
    if constexpr (kPacked) return bwd_block_packed(item_info + 4 * (n & 3), H, Hkv);
    else return bwd_block(idx, H, Hkv, kvs, nq, wl);
  };

  if (threadIdx.x == 0) {
    mbar_init(kv_full, 1);
    mbar_init(kv_empty, 1 + 12);   // the MMA commit and one arrival per softmax and dQ warp
    for (int i = 0; i < 2; ++i) { mbar_init(&q_full[i], 1); mbar_init(&q_empty[i], 1); }
    mbar_init(do_full, 1);
    mbar_init(do_empty, 1);
    mbar_init(s_full, 1);
    mbar_init(s_free, 256);
    mbar_init(dp_full, 1);
    mbar_init(p_ready, 256);
    mbar_init(ds_ready, 256);
    mbar_init(mm_done, 1);
    mbar_init(dq_free, 128);
    mbar_init(drain, 1);
    *abort_flag = 0;
    fence_barrier_init();
    if constexpr (!kPacked) {
      tma_prefetch_desc(&tq);
      tma_prefetch_desc(&tk);
      tma_prefetch_desc(&tv);
      tma_prefetch_desc(&tdo);
    }
    tma_prefetch_desc(&tdq);
  }
  if (warp == 1) {
    tmem_alloc(tmem_holder, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_holder;
  if constexpr (kPacked) chain_wait();
  const int Tv = kPacked ? pa.ctl[kCtlValid] : T;   // positions of a row that hold sequences

  // registers: 72 for the TMA / MMA warp group, 96 for the dQ group, 168 for
  // the two softmax groups (4*72 + 4*96 + 8*168 = 2016 per lane of a warp,
  // within the 16 warps x 128 the block is launched with); packed, whose softmax
  // holds P in fp32: 72, 88 and 176 (4*72 + 4*88 + 8*176 = 2048)
  if (warp < 4) asm volatile("setmaxnreg.dec.sync.aligned.u32 72;\n" ::: "memory");
  if (warp == 0) {
    if (lane == 0) {
      // -------------------------------------------------------------- TMA
      const CUtensorMap* mq = kPacked ? pa.maps : &tq;
      const CUtensorMap* mk = kPacked ? pa.maps + 1 : &tk;
      const CUtensorMap* mv = kPacked ? pa.maps + 2 : &tv;
      const CUtensorMap* mdo = kPacked ? pa.maps + 3 : &tdo;
      int entries = 0;
      if constexpr (kPacked) {
        tensormap_acquire(mq);
        tensormap_acquire(mk);
        tensormap_acquire(mv);
        tensormap_acquire(mdo);
        entries = pa.ctl[kCtlEntries];
        n_units = entries * Hkv;
      }
      // packed: fetched one item ahead, as in the forward
      int nx_idx = -1, nx_hk = 0;
      int2 nx = make_int2(0, 0);
      auto take = [&] {
        do {
          nx_idx = atomicAdd(sched, 1);
          if (nx_idx >= n_units) { nx_idx = -1; return; }
          nx_hk = nx_idx / entries;
          nx = __ldg(pa.bwd + (nx_idx - nx_hk * entries));
        } while (!bwd_entry_ok(nx, Tv, err));
      };
      if constexpr (kPacked) take();
      bool ok = true;
      int g = 0, nblk = 0;          // query blocks and items loaded so far
      int issued_q = 0, issued_do = 0;
      auto load_q_do = [&](const BwdBlock& kb, int it) -> bool {
        const int i = kb.q_block(it), h = kb.q_head(it), bh = kb.b * H + h;
        const int s = g & 1;
        if (!mbar_wait_t<kFine>(&q_empty[s], ((g >> 1) & 1) ^ 1u, abort_flag, err, wlim)) return false;
        // packed: the rows' -lse and -D come with Q and dO, from [H][128 nq] arrays
        constexpr uint32_t kRows = kPacked ? 512 : 0;
        const long long rows = kPacked ? static_cast<long long>(h) * nq * 128 + i * 128 : 0;
        mbar_arrive_expect_tx(&q_full[s], TF_BUF + kRows);
        if constexpr (kPacked) bulk_load(lse_s + s * 128, lse + rows, kRows, &q_full[s]);
        tma_load_3d(sQ + s * TF_BUF, mq, &q_full[s], 0, i * 128, bh);
        tma_load_3d(sQ + s * TF_BUF + TF_TILE, mq, &q_full[s], 64, i * 128, bh);
        ++issued_q;
        if (!mbar_wait_t<kFine>(do_empty, (g & 1) ^ 1u, abort_flag, err, wlim)) return false;
        mbar_arrive_expect_tx(do_full, TF_BUF + kRows);
        if constexpr (kPacked) bulk_load(dd_s + s * 128, Dv + rows, kRows, do_full);
        tma_load_4d(sdO, mdo, do_full, 0, h, i * 128, kb.b);
        tma_load_4d(sdO + TF_TILE, mdo, do_full, 64, h, i * 128, kb.b);
        ++issued_do;
        ++g;
        return true;
      };
      // work is handed out in units of two key blocks, u and nkb - 1 - u of one
      // kv head (the same work under the causal mask), longest unit of a head
      // first; the unit's blocks become consecutive items
      const int nu = (nq + 1) / 2;
      int pending = -1, taken = 0;
      for (int n = 0; ok; ++n) {
        int idx = pending;
        pending = -1;
        if constexpr (kPacked) {
          idx = nx_idx;
          volatile int* f = item_info + 4 * (n & 3);
          f[0] = nx_hk; f[1] = nx.x; f[2] = nx.y;
        } else if (idx < 0) {
          const int unit = sched ? atomicAdd(sched, 1) : taken * static_cast<int>(gridDim.x) + static_cast<int>(blockIdx.x);
          ++taken;
          if (unit < n_units) {
            const int bkv = unit / nu, uu = nu - 1 - (unit - bkv * nu);
            idx = bkv * nq + uu;
            if (nq - 1 - uu != uu) pending = bkv * nq + nq - 1 - uu;
          }
        }
        item_ring[n & 3] = idx;
        if (idx < 0) {
          // end marker, once every warp has the previous item's number
          if (n > 0 && !mbar_wait_t<kFine>(kv_empty, (n - 1) & 1, abort_flag, err, wlim)) { ok = false; break; }
          mbar_arrive(kv_full);
          break;
        }
        const BwdBlock kb = block_of(n, idx);
        // the first query block's Q and dO may load while the previous item
        // finishes; K and V (which publish the item number) once its last
        // products are done
        if (!load_q_do(kb, 0)) { ok = false; break; }
        if (n > 0 && !mbar_wait_t<kFine>(kv_empty, (n - 1) & 1, abort_flag, err, wlim)) { ok = false; break; }
        mbar_arrive_expect_tx(kv_full, 2 * TF_BUF);
        tma_load_3d(sK, mk, kv_full, 0, kb.k0, kb.kvrow);
        tma_load_3d(sK + TF_TILE, mk, kv_full, 64, kb.k0, kb.kvrow);
        tma_load_3d(sV, mv, kv_full, 0, kb.k0, kb.kvrow);
        tma_load_3d(sV + TF_TILE, mv, kv_full, 64, kb.k0, kb.kvrow);
        ++nblk;
        if constexpr (kPacked) take();
        for (int it = 1; it < kb.n_it; ++it)
          if (!load_q_do(kb, it)) { ok = false; break; }
      }
      if (!ok) {
        // let the copies already started land before the CTA exits
        if (nblk > 0)
          for (uint32_t x = 0; x < (1u << 20) && !mbar_try_wait(kv_full, (nblk - 1) & 1); ++x) {}
        for (int it = (issued_q > 2 ? issued_q - 2 : 0); it < issued_q; ++it)
          for (uint32_t x = 0; x < (1u << 20) && !mbar_try_wait(&q_full[it & 1], (it >> 1) & 1); ++x) {}
        if (issued_do > 0)
          for (uint32_t x = 0; x < (1u << 20) && !mbar_try_wait(do_full, (issued_do - 1) & 1); ++x) {}
      }
    }
  } else if (warp == 1) {
    // -------------------------------------------------------------- MMA
    // the whole warp, converged; one lane issues
    const bool leader = elect_lane();
    const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
    auto wait1 = [&](uint64_t* bar, uint32_t par) -> bool {
      return __all_sync(0xffffffffu, mbar_wait_t<kFine>(bar, par, abort_flag, err, wlim));
    };
    auto uniform = [](int x) { return __shfl_sync(0xffffffffu, x, 0); };
    constexpr uint32_t IDESC_KK = make_idesc(1, 128, false, false);   // S^T, dP^T
    constexpr uint32_t IDESC_KM = make_idesc(1, 128, false, true);    // dV (A in TMEM), dK
    constexpr uint32_t IDESC_MM = make_idesc(1, 128, true, true);     // dQ
    const uint32_t k_addr = smem_u32(sK), v_addr = smem_u32(sV), do_addr = smem_u32(sdO);
    const uint32_t dst_addr = smem_u32(sdSt);
    // X^T = A B^T over the 128 head dims, both operands K-major
    auto qk_product = [&](uint32_t d_tmem, uint32_t a_addr, uint32_t b_addr) {
      uint64_t da = smem_desc_sw128(a_addr, 16, 1024), db = smem_desc_sw128(b_addr, 16, 1024);
#pragma unroll
      for (int kk = 0; kk < 8; ++kk) {
        const uint32_t off16 = ((kk >> 2) * TF_TILE + (kk & 3) * 32) >> 4;
        umma_f16_by(leader, d_tmem, da + off16, db + off16, IDESC_KK, kk > 0 ? 1u : 0u);
      }
    };
    bool ok = true;
    int g0 = 0;   // query blocks done so far
    for (int n = 0; ok; ++n) {
      if (!wait1(kv_full, n & 1)) { ok = false; break; }
      const int idx = uniform(item_ring[n & 3]);
      if (idx < 0) break;
      {
        const BwdBlock kb = block_of(n, idx);
        const int n_it = uniform(kb.n_it);
        // S^T of the first query block goes where the previous key block's
        // last dQ was (wait until the dQ warps have read it), dP^T where
        // its last P was (wait until that dV is done)
        ok = wait1(&q_full[g0 & 1], (g0 >> 1) & 1) &&
             (g0 == 0 || wait1(dq_free, (g0 - 1) & 1));
        if (!ok) break;
        tc_fence_after();
        qk_product(tm, k_addr, smem_u32(sQ + (g0 & 1) * TF_BUF));   // S^T of the first block
        umma_commit_by(leader, s_full);
        ok = wait1(do_full, g0 & 1) &&
             (g0 == 0 || wait1(do_empty, (g0 - 1) & 1));
        if (!ok) break;
        tc_fence_after();
        qk_product(tm + 128, v_addr, do_addr);   // dP^T of the first block
        umma_commit_by(leader, dp_full);
        if (n_it > 1) {
          ok = wait1(s_free, g0 & 1) &&
               wait1(&q_full[(g0 + 1) & 1], ((g0 + 1) >> 1) & 1);
          if (!ok) break;
          tc_fence_after();
          qk_product(tm, k_addr, smem_u32(sQ + ((g0 + 1) & 1) * TF_BUF));   // S^T of the second block
          umma_commit_by(leader, s_full);
        }
        for (int it = 0; it < n_it && ok; ++it) {
          const int gi = g0 + it;
          const int s = gi & 1;
          if (!wait1(p_ready, gi & 1)) { ok = false; break; }
          tc_fence_after();
          const uint32_t q_addr = smem_u32(sQ + s * TF_BUF);
          // dV += P^T dO: A = P^T from TMEM, 16 queries = 8 packed columns per
          // step; queries 0..63 at columns 128.., 64..127 at columns 192..
          {
            uint64_t ddo = smem_desc_sw128(do_addr, TF_TILE, 1024);
#pragma unroll
            for (int kk = 0; kk < 8; ++kk)
              umma_f16_tmem_a_by(leader, tm + 256, tm + 128 + (kk >> 2) * 64 + (kk & 3) * 8, ddo + ((kk * 2048) >> 4),
                              IDESC_KM, (it > 0 || kk > 0) ? 1u : 0u);
          }
          umma_commit_by(leader, do_empty);
          // dK and dQ once dS_i is in shared memory (the softmax warps compute it
          // while dV runs)
          if (!wait1(ds_ready, gi & 1)) { ok = false; break; }
          tc_fence_after();
          {
            uint64_t dsa = smem_desc_sw128(dst_addr, 16, 1024), dqb = smem_desc_sw128(q_addr, TF_TILE, 1024);
#pragma unroll
            for (int kk = 0; kk < 8; ++kk) {
              const uint32_t aoff16 = ((kk >> 2) * TF_TILE + (kk & 3) * 32) >> 4;   // K-major A: 16 queries per step
              const uint32_t boff16 = (kk * 2048) >> 4;                            // MN-major B: 16 query rows per step
              umma_f16_by(leader, tm + 384, dsa + aoff16, dqb + boff16, IDESC_KM, (it > 0 || kk > 0) ? 1u : 0u);
            }
          }
          umma_commit_by(leader, &q_empty[s]);
          // dQ_i goes to [0,128), which holds S^T_{i+1} (wait until the softmax
          // warps have read it) or, for the last block, dQ_{i-1} (wait until
          // the dQ warps have read it)
          if (it + 1 < n_it) {
            if (!wait1(s_free, (gi + 1) & 1)) { ok = false; break; }
          } else if (it > 0) {
            if (!wait1(dq_free, (gi - 1) & 1)) { ok = false; break; }
          }
          tc_fence_after();
          {
            uint64_t dka = smem_desc_sw128(k_addr, TF_TILE, 1024), dsb = smem_desc_sw128(dst_addr, TF_TILE, 1024);
#pragma unroll
            for (int kk = 0; kk < 8; ++kk) {
              const uint32_t off16 = (kk * 2048) >> 4;   // 16 keys per step, both operands MN-major
              umma_f16_by(leader, tm, dsb + off16, dka + off16, IDESC_MM, kk > 0 ? 1u : 0u);   // dQ = dS K
            }
          }
          umma_commit_by(leader, mm_done);
          if (it + 1 == n_it) umma_commit_by(leader, kv_empty);   // K and V of this key block are free
          if (it + 1 < n_it) {
            // dP^T_{i+1} overwrites P^T_i: dV_i must have completed
            if (!wait1(do_empty, gi & 1) ||
                !wait1(do_full, (gi + 1) & 1)) { ok = false; break; }
            tc_fence_after();
            qk_product(tm + 128, v_addr, do_addr);
            umma_commit_by(leader, dp_full);
          }
          if (it + 2 < n_it) {
            if (!wait1(dq_free, gi & 1) ||
                !wait1(&q_full[s], ((gi + 2) >> 1) & 1)) { ok = false; break; }
            tc_fence_after();
            qk_product(tm, k_addr, q_addr);   // S^T_{i+2} (same Q slot as block i)
            umma_commit_by(leader, s_full);
          }
        }
        g0 += n_it;
      }
    }
    umma_commit_by(leader, drain);
    for (uint32_t x = 0; x < (1u << 22) && !mbar_try_wait(drain, 0); ++x) {}
  } else if (warp >= 12) {
    if constexpr (kPacked) asm volatile("setmaxnreg.dec.sync.aligned.u32 88;\n" ::: "memory");
    else asm volatile("setmaxnreg.dec.sync.aligned.u32 96;\n" ::: "memory");
    // ------------------------------------------------------------------ dQ
    const int quarter = warp & 3;
    const uint32_t lane_base = static_cast<uint32_t>(quarter * 32) << 16;
    const uint64_t sc2 = f2_pack(scale, scale);
    bool ok = true;
    // dQ of one query block: this thread's query row (TMEM lane) of 128 dims,
    // staged 64 dims at a time as two [32 queries][32 dims] fp32 boxes (a row
    // is 128 bytes: eight 16-byte stores) and added into dq by TMA reduce-add
    uint8_t* box = sStage + quarter * 8192;
    int g = 0;
    for (int n = 0; ok; ++n) {
      {
        const bool got = mbar_wait_t<kFine>(kv_full, n & 1, abort_flag, err, wlim);
        __syncwarp();
        if (!__all_sync(0xffffffffu, got)) { ok = false; break; }
      }
      const int idx = item_ring[n & 3];
      __syncwarp();
      if (lane == 0) mbar_arrive(kv_empty);   // this warp has the item number
      if (idx < 0) break;
      {
        const BwdBlock kb = block_of(n, idx);
        for (int it = 0; it < kb.n_it && ok; ++it, ++g) {
          const int q0 = kb.q_block(it) * 128 + quarter * 32, bh = kb.b * H + kb.q_head(it);
          const bool got = mbar_wait_t<kFine>(mm_done, g & 1, abort_flag, err, wlim);
          __syncwarp();
          if (!__all_sync(0xffffffffu, got)) { ok = false; break; }
          tc_fence_after();
#pragma unroll 1
          for (int hh = 0; hh < 2; ++hh) {
            uint32_t va[32], vb[32];
            tmem_load32_async(tmem + lane_base + hh * 64, va);
            tmem_load32_async(tmem + lane_base + hh * 64 + 32, vb);
            tmem_wait_ld();
            if (hh == 1) {
              tc_fence_before();
              mbar_arrive(dq_free);
            }
            if (lane == 0) bulk_wait_read_all();   // the boxes' previous contents have been read
            __syncwarp();
#pragma unroll
            for (int j = 0; j < 64; j += 4) {
              const uint32_t (&v)[32] = j < 32 ? va : vb;
              const int e = j & 31;
              float a0, a1, a2, a3;
              f2_unpack(f2_mul(f2_pack(__uint_as_float(v[e]), __uint_as_float(v[e + 1])), sc2), a0, a1);
              f2_unpack(f2_mul(f2_pack(__uint_as_float(v[e + 2]), __uint_as_float(v[e + 3])), sc2), a2, a3);
              *reinterpret_cast<float4*>(box + (j >> 5) * 4096 + lane * 128 + ((((e >> 2) ^ lane) & 7) << 4)) =
                  make_float4(a0, a1, a2, a3);
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
              tma_reduce_add_3d(&tdq, box, hh * 64, q0, bh);
              tma_reduce_add_3d(&tdq, box + 4096, hh * 64 + 32, q0, bh);
              bulk_commit();
            }
          }
        }
      }
    }
    if (lane == 0) bulk_wait_all();
  } else if (warp >= 4) {
    if constexpr (kPacked) asm volatile("setmaxnreg.inc.sync.aligned.u32 176;\n" ::: "memory");
    else asm volatile("setmaxnreg.inc.sync.aligned.u32 168;\n" ::: "memory");
    // ------------------------------------------------------- P, dS, dK, dV
    const int quarter = warp & 3;
    const int half = (warp - 4) >> 2;        // which 64 query columns of the row
    const int r = quarter * 32 + lane;       // key row (TMEM lane)
    const int t256 = threadIdx.x - 128;      // 0..255
    const uint32_t lane_base = static_cast<uint32_t>(quarter * 32) << 16;
    const float scale_log2 = scale * 1.4426950408889634f;
    const uint64_t sl2 = f2_pack(scale_log2, scale_log2);
    bool ok = true;
    // Named barrier 1 over the 256 softmax threads, which also tells every
    // thread whether any of them failed its wait (so all leave the loop together)
    auto any_fail = [&](bool got) -> bool {
      __syncwarp();
      uint32_t f;
      asm volatile(
          "{\n\t.reg .pred pi, po;\n\tsetp.eq.u32 pi, %1, 0;\n\t"
          "bar.red.or.pred po, 1, 256, pi;\n\tselp.u32 %0, 1, 0, po;\n\t}"
          : "=r"(f)
          : "r"(got ? 1u : 0u)
          : "memory");
      return f != 0;
    };
    // Every decision to leave a loop is taken by this vote, so the eight
    // warps always meet at the same named barriers: a warp that left on its
    // own would leave the others waiting at the next vote.  The packed build has
    // no such barrier (its lse and D come by TMA), so there a warp decides alone.
    auto passed = [&](bool got) -> bool {
      if constexpr (kPacked) return __all_sync(0xffffffffu, got);
      else return !any_fail(got);
    };
    int g0 = 0;
    for (int n = 0; ok; ++n) {
      {
        const bool got = mbar_wait_t<kFine>(kv_full, n & 1, abort_flag, err, wlim);
        if (!passed(got)) { ok = false; break; }
      }
      const int idx = item_ring[n & 3];
      __syncwarp();
      // this warp has the item number; when dK goes through the QK-norm
      // backward, K stays until the item's epilogue has read its rows
      if (lane == 0 && (idx < 0 || !dqkv)) mbar_arrive(kv_empty);
      if (idx < 0) break;
      {
        const BwdBlock kb = block_of(n, idx);
        const int n_it = kb.n_it, k0 = kb.k0, bkv = kb.kvrow;
        const int key = k0 + r;
        const bool key_ok = key < Tv;
        int hi = 0, hi_min = 0, hi_max = 0;   // packed: last query that sees this key, and over the warp's keys
        if constexpr (kPacked) {
          hi = key_ok ? __ldg(pa.hi + key) : -1;
          hi_min = __reduce_min_sync(0xffffffffu, hi);
          hi_max = __reduce_max_sync(0xffffffffu, hi);
        }
        if (dqkv && key_ok) {
          // the epilogue's rotation table row and inverse RMS, on their way to L2
          asm volatile("prefetch.global.L2 [%0];" ::"l"(rope + static_cast<long long>(key) * 64 + 32 * half));
          asm volatile("prefetch.global.L2 [%0];" ::"l"(rope + static_cast<long long>(key) * 64 + 32 * half + 16));
          asm volatile("prefetch.global.L2 [%0];" ::"l"(rk + (static_cast<long long>(kb.b) * T + key) * H + kb.hk));
        }
        // this thread's share of a query block's -lse (log2 units; -inf past T so
        // P = 0) or -D, fetched a block ahead so the load latency hides
        auto fetch = [&](int it2) -> float {
          const int q0f = kb.q_block(it2) * 128;
          const long long bh = static_cast<long long>(kb.b) * H + kb.q_head(it2);
          if (t256 < 128) {
            const int qq = q0f + t256;
            return qq < Tv ? __ldg(lse + bh * T + qq) * -1.4426950408889634f : -INFINITY;
          }
          const int qq = q0f + t256 - 128;
          return qq < Tv ? -__ldg(Dv + bh * T + qq) : 0.f;
        };
        // block it2's values go to buffer (g0 + it2) & 1; a barrier publishes them
        auto publish = [&](int it2, float v) {
          float* base = (t256 < 128 ? lse_s : dd_s) + ((g0 + it2) & 1) * 128;
          base[t256 & 127] = v;
        };
        // P of block it2 for this thread's key row and 64 query columns: packed bf16,
        // from which dS is formed too; packed build: fp32 for dS, rounded for dV alone
        uint32_t pk[kPacked ? 64 : 32];
        auto compute_p = [&](int it2) {
          const bool diag = it2 % kb.nb == 0;
          const int q0 = kb.q_block(it2) * 128;
          // causal diagonal block, ragged key block, or a query block whose last
          // rows' windows start past this block's first key
          const bool edge = k0 + 128 > T || q0 + 127 - wl > k0;
          const bool masked = diag || edge;
          const float* nls = lse_s + ((g0 + it2) & 1) * 128;
          uint32_t sa[32], sb[32];
          tmem_load32_async(tmem + lane_base + (2 * half) * 32, sa);
          tmem_load32_async(tmem + lane_base + (2 * half + 1) * 32, sb);
          tmem_wait_ld();
          tc_fence_before();
          mbar_arrive(s_free);   // S^T of this block has been read
          // One 32-query chunk of the row in one of four forms, chosen per
          // chunk by a warp-uniform test: no mask, the causal diagonal's lane
          // mask (queries below the key row; packed: a mask of bits), all masked
          // (P = 0), or the general mask (ragged keys, window edge; not packed).  A per-element mask inside one loop
          // was if-converted into every block's path and cost more than the
          // exponentials.
          auto run_chunk = [&](auto kCC, auto kMode, uint32_t seen = 0u) {
            constexpr int cc = decltype(kCC)::value, mode = decltype(kMode)::value;
            const int c = 2 * half + cc;
            const uint32_t (&sr)[32] = cc == 0 ? sa : sb;
            if constexpr (mode == 3) {
#pragma unroll
              for (int x = 0; x < (kPacked ? 32 : 16); ++x) pk[(kPacked ? 32 : 16) * cc + x] = 0u;
            } else {
#pragma unroll
              for (int kq = 0; kq < 32; kq += 8) {
                const float4 la = *reinterpret_cast<const float4*>(nls + c * 32 + kq);
                const float4 lb = *reinterpret_cast<const float4*>(nls + c * 32 + kq + 4);
                const float nl[8] = {la.x, la.y, la.z, la.w, lb.x, lb.y, lb.z, lb.w};   // -lse * log2(e)
                // P = 2^(S * scale * log2(e) - lse * log2(e)): GPT_BWD_MUFU of every
                // eight (packed: all) on the MUFU unit, the rest by the polynomial on the FMA pipe
                float p[8];
#pragma unroll
                for (int e = 0; e < 8; e += 2) {
                  float x0, x1;
                  f2_unpack(f2_fma(f2_pack(__uint_as_float(sr[kq + e]), __uint_as_float(sr[kq + e + 1])), sl2,
                                   f2_pack(nl[e], nl[e + 1])),
                            x0, x1);
                  if (kPacked || e < GPT_BWD_MUFU) {
                    p[e] = ex2_approx(x0);
                    p[e + 1] = ex2_approx(x1);
                  } else {
                    f2_unpack(f2_exp2_poly(f2_pack(fmaxf(x0, -126.f), fmaxf(x1, -126.f))), p[e], p[e + 1]);
                  }
                }
                if constexpr (mode == 1 && kPacked) {
#pragma unroll
                  for (int e = 0; e < 8; ++e)
                    if (!(seen & (1u << (kq + e)))) p[e] = 0.f;
                } else if constexpr (mode == 1) {
#pragma unroll
                  for (int e = 0; e < 8; ++e)
                    if (kq + e < lane) p[e] = 0.f;
                } else if constexpr (mode == 2) {
#pragma unroll
                  for (int e = 0; e < 8; ++e)
                    if (!key_ok || (diag && key > q0 + c * 32 + kq + e) || key < q0 + c * 32 + kq + e - wl) p[e] = 0.f;
                }
                if constexpr (kPacked) {
#pragma unroll
                  for (int e = 0; e < 8; ++e) pk[32 * cc + kq + e] = __float_as_uint(p[e]);
                } else {
#pragma unroll
                  for (int e = 0; e < 8; e += 2) pk[16 * cc + ((kq + e) >> 1)] = pack_bf16x2(p[e], p[e + 1]);
                }
              }
            }
          };
          using M0 = std::integral_constant<int, 0>;
          using M1 = std::integral_constant<int, 1>;
          using M2 = std::integral_constant<int, 2>;
          using M3 = std::integral_constant<int, 3>;
          auto do_chunk = [&](auto kCC) {
            const int c = 2 * half + decltype(kCC)::value;
            if constexpr (kPacked) {
              // the queries qc .. qc + 31 that see this key, key .. hi, as bits
              const int qc = q0 + c * 32;
              if (qc > hi_max || (diag && c < quarter))
                run_chunk(kCC, M3{});
              else if (qc + 31 > hi_min || (diag && c == quarter))
                run_chunk(kCC, M1{}, low_bits(hi + 1 - qc) & ~low_bits(key - qc));
              else
                run_chunk(kCC, M0{});
            } else if (diag && !edge) {
              if (c < quarter)
                run_chunk(kCC, M3{});
              else if (c == quarter)
                run_chunk(kCC, M1{});
              else
                run_chunk(kCC, M0{});
            } else if (masked) {
              run_chunk(kCC, M2{});
            } else {
              run_chunk(kCC, M0{});
            }
          };
          do_chunk(std::integral_constant<int, 0>{});
          do_chunk(std::integral_constant<int, 1>{});
        };

        float staged = 0.f;
        if constexpr (!kPacked) {
          publish(0, fetch(0));
          if (n_it > 1) staged = fetch(1);
        }
        // it = -1 only computes P of the first block
        for (int it = -1; it < n_it && ok; ++it) {
          const int gi = g0 + it;
          if (it >= 0) {
            // dS'_i = P_i (dP_i - D) once dP^T_i is in TMEM
            const bool got = mbar_wait_t<kFine>(dp_full, gi & 1, abort_flag, err, wlim) &&
                             (!kPacked || mbar_wait_t<kFine>(do_full, gi & 1, abort_flag, err, wlim));   // D is here
            if (!passed(got)) { ok = false; break; }
            if constexpr (!kPacked) {
              // every thread is past block i-1's use of buffer (i+1) & 1
              if (it + 1 < n_it) publish(it + 1, staged);
              if (it + 2 < n_it) staged = fetch(it + 2);
            }
            tc_fence_after();
            uint32_t da[32], db[32];
            tmem_load32_async(tmem + lane_base + 128 + (2 * half) * 32, da);
            // P^T_i over the first 32 of this warp's 64 dP^T columns, once they are read
            if constexpr (kPacked) {
              uint32_t pb[32];
#pragma unroll
              for (int x = 0; x < 32; ++x)
                pb[x] = pack_bf16x2(__uint_as_float(pk[2 * x]), __uint_as_float(pk[2 * x + 1]));
              tmem_landed(da);
              tmem_store32(tmem + lane_base + 128 + 64 * half, pb);
            } else {
              tmem_load32_async(tmem + lane_base + 128 + (2 * half + 1) * 32, db);
              tmem_wait_ld();
              tmem_store32(tmem + lane_base + 128 + 64 * half, pk);
            }
            asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
            tc_fence_before();
            mbar_arrive(p_ready);
            // the other 32, which dV leaves alone, while the first become dS (with P in
            // fp32 there are no registers for all 64 before)
            if constexpr (kPacked) tmem_load32_async(tmem + lane_base + 128 + (2 * half + 1) * 32, db);
            const float* nds = dd_s + (gi & 1) * 128;
            uint32_t dk2[32];
#pragma unroll
            for (int cc = 0; cc < 2; ++cc) {
              const int c = 2 * half + cc;
              const uint32_t (&dr)[32] = cc == 0 ? da : db;
              if (kPacked && cc == 1) tmem_landed(db);
#pragma unroll
              for (int kq = 0; kq < 32; kq += 4) {
                const float4 d4 = *reinterpret_cast<const float4*>(nds + c * 32 + kq);
                float pr[4];
                if constexpr (kPacked) {
#pragma unroll
                  for (int e = 0; e < 4; ++e) pr[e] = __uint_as_float(pk[32 * cc + kq + e]);
                } else {
                  const uint32_t w0 = pk[16 * cc + (kq >> 1)], w1 = pk[16 * cc + (kq >> 1) + 1];
                  pr[0] = bf16_lo(w0); pr[1] = bf16_hi(w0); pr[2] = bf16_lo(w1); pr[3] = bf16_hi(w1);
                }
                float a0, a1, a2, a3;
                f2_unpack(f2_mul(f2_pack(pr[0], pr[1]),
                                 f2_add(f2_pack(__uint_as_float(dr[kq]), __uint_as_float(dr[kq + 1])),
                                        f2_pack(d4.x, d4.y))),
                          a0, a1);
                f2_unpack(f2_mul(f2_pack(pr[2], pr[3]),
                                 f2_add(f2_pack(__uint_as_float(dr[kq + 2]), __uint_as_float(dr[kq + 3])),
                                        f2_pack(d4.z, d4.w))),
                          a2, a3);
                dk2[16 * cc + (kq >> 1)] = pack_bf16x2(a0, a1);
                dk2[16 * cc + (kq >> 1) + 1] = pack_bf16x2(a2, a3);
              }
            }
            store_row_units(sdSt, dk2, half, r);
            fence_proxy_async_smem();
            if constexpr (kPacked) tc_fence_before();   // the next dP^T goes where db was read
            mbar_arrive(ds_ready);
          }
          // P_{i+1} while the tensor cores run this block's dV, dK, dQ
          if (it + 1 < n_it) {
            const bool got1 = mbar_wait_t<kFine>(s_full, (gi + 1) & 1, abort_flag, err, wlim) &&
                              (!kPacked || mbar_wait_t<kFine>(&q_full[(gi + 1) & 1], ((gi + 1) >> 1) & 1, abort_flag,
                                                              err, wlim));   // lse is here
            if (!passed(got1)) { ok = false; break; }   // not packed: also publishes lse/D of block i+1
            tc_fence_after();
            compute_p(it + 1);
          }
        }
        // dK and dV of this key block, complete with the last block's products
        if (ok) {
          const bool got = mbar_wait_t<kFine>(mm_done, (g0 + n_it - 1) & 1, abort_flag, err, wlim);
          ok = passed(got);
        }
        if (ok && dqkv) {
          // straight into the token-major q|k|v gradient rows: dV as it is, dK
          // through the backward of the QK RMS norm and of the rotation
          // (head dims i and 64 + i form a rotated pair; this thread takes the
          // pairs 32 * half .. 32 * half + 31, the other half's thread the rest
          // of the row, and the two add up the row's <dK, k> in shared memory)
          tc_fence_after();
          const long long m = static_cast<long long>(kb.b) * T + key;
          const int dqk = H * 128, kvd = Hkv * 128;
          bf16* orow = dqkv + m * (dqk + 2 * kvd) + dqk + kb.hk * 128;
          // the normalised rotated k of this row at the same dims, from the K
          // tile in shared memory (two 64-column halves of [128 rows][128 B],
          // 16-byte unit u of row r at u ^ (r & 7)); then K may be replaced
          uint4 yl[4], yh[4];
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            const int u = (4 * half + x) ^ (r & 7);
            yl[x] = *reinterpret_cast<const uint4*>(sK + r * 128 + u * 16);
            yh[x] = *reinterpret_cast<const uint4*>(sK + TF_TILE + r * 128 + u * 16);
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(kv_empty);
#pragma unroll 1
          for (int c = 0; c < 2; ++c) {
            uint32_t vr[32];
            tmem_load32_async(tmem + lane_base + 256 + 64 * half + 32 * c, vr);
            tmem_wait_ld();
            if (key_ok) {
#pragma unroll
              for (int gg = 0; gg < 32; gg += 8) {
                uint4 wv;
                wv.x = pack_bf16x2(__uint_as_float(vr[gg]), __uint_as_float(vr[gg + 1]));
                wv.y = pack_bf16x2(__uint_as_float(vr[gg + 2]), __uint_as_float(vr[gg + 3]));
                wv.z = pack_bf16x2(__uint_as_float(vr[gg + 4]), __uint_as_float(vr[gg + 5]));
                wv.w = pack_bf16x2(__uint_as_float(vr[gg + 6]), __uint_as_float(vr[gg + 7]));
                *reinterpret_cast<uint4*>(orow + kvd + 64 * half + 32 * c + gg) = wv;
              }
            }
          }
          // <dK, k> over this thread's pairs, 16 at a time (dK read from TMEM
          // twice, here and for the result, to keep the registers down)
          float part = 0.f;
#pragma unroll
          for (int hq = 0; hq < 2; ++hq) {
            uint32_t gl[16], gh[16];
            tmem_load16_async(tmem + lane_base + 384 + 32 * half + 16 * hq, gl);
            tmem_load16_async(tmem + lane_base + 448 + 32 * half + 16 * hq, gh);
            tmem_wait_ld();
#pragma unroll
            for (int x = 0; x < 2; ++x) {
              const uint4 a = yl[2 * hq + x], bq = yh[2 * hq + x];
              const uint32_t wl4[4] = {a.x, a.y, a.z, a.w};
              const uint32_t wh4[4] = {bq.x, bq.y, bq.z, bq.w};
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const int i = 8 * x + 2 * e;
                part += __uint_as_float(gl[i]) * bf16_lo(wl4[e]) + __uint_as_float(gl[i + 1]) * bf16_hi(wl4[e]) +
                        __uint_as_float(gh[i]) * bf16_lo(wh4[e]) + __uint_as_float(gh[i + 1]) * bf16_hi(wh4[e]);
              }
            }
          }
          // the two halves of the row meet in the softmax warps' lse buffer,
          // which no thread reads again before the next item's first vote
          lse_s[half * 128 + r] = part;
          asm volatile("bar.sync 1, 256;" ::: "memory");
          // dK = scale * (the TMEM sums); <dK, k> / 128 over the whole row
          const float dot = (part + lse_s[(half ^ 1) * 128 + r]) * scale * (1.f / 128.f);
          const float rr = key_ok ? rk[m * H + kb.hk] : 0.f;
          const float4* e4 = reinterpret_cast<const float4*>(rope + static_cast<long long>(key_ok ? key : 0) * 64 +
                                                             32 * half);
#pragma unroll
          for (int hq = 0; hq < 2; ++hq) {
            uint32_t gl[16], gh[16];
            tmem_load16_async(tmem + lane_base + 384 + 32 * half + 16 * hq, gl);
            tmem_load16_async(tmem + lane_base + 448 + 32 * half + 16 * hq, gh);
            tmem_wait_ld();
            if (key_ok) {
#pragma unroll
              for (int x = 0; x < 2; ++x) {
                const uint4 a = yl[2 * hq + x], bq = yh[2 * hq + x];
                const uint32_t wl4[4] = {a.x, a.y, a.z, a.w};
                const uint32_t wh4[4] = {bq.x, bq.y, bq.z, bq.w};
                uint32_t ol[4], oh[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                  const int i = 8 * x + 2 * e;
                  const float4 cs = __ldg(e4 + ((16 * hq + i) >> 1));   // (cos, sin) of pairs i and i + 1
                  // gradient w.r.t. the rotated vector, then the transposed rotation
                  const float rl0 = rr * (__uint_as_float(gl[i]) * scale - bf16_lo(wl4[e]) * dot);
                  const float rl1 = rr * (__uint_as_float(gl[i + 1]) * scale - bf16_hi(wl4[e]) * dot);
                  const float rh0 = rr * (__uint_as_float(gh[i]) * scale - bf16_lo(wh4[e]) * dot);
                  const float rh1 = rr * (__uint_as_float(gh[i + 1]) * scale - bf16_hi(wh4[e]) * dot);
                  ol[e] = pack_bf16x2(rl0 * cs.x + rh0 * cs.y, rl1 * cs.z + rh1 * cs.w);
                  oh[e] = pack_bf16x2(-rl0 * cs.y + rh0 * cs.x, -rl1 * cs.w + rh1 * cs.z);
                }
                const int col = 32 * half + 16 * hq + 8 * x;
                *reinterpret_cast<uint4*>(orow + col) = make_uint4(ol[0], ol[1], ol[2], ol[3]);
                *reinterpret_cast<uint4*>(orow + 64 + col) = make_uint4(oh[0], oh[1], oh[2], oh[3]);
              }
            }
          }
          // dK and dV have been read: the next key block's first products may
          // overwrite them (they follow this thread's next p_ready / ds_ready)
          tc_fence_before();
        } else if (ok) {
          tc_fence_after();
          const int w0 = k0 + quarter * 32, rows = min(32, Tv - w0);   // the warp's first key row, its rows
          // dS of the last block has been read: its tile stages the rows, each
          // warp in the part that it writes itself; dV, then dK
#pragma unroll 1
          for (int c = 0; c < 2; ++c) {
            const long long pitch = kPacked ? (c ? pa.o_tok : pa.dv_tok) : 128;
            bf16* row = (c ? dk : dv) + (kPacked ? w0 * pitch + kb.hk * (c ? pa.o_head : pa.dv_head)
                                                 : (static_cast<long long>(bkv) * T + w0) * 128);
            const float z = store_rows<64, kPacked>(tmem + lane_base + 256 + 128 * c + 64 * half, c ? scale : 1.f,
                                                    sdSt + half * TF_TILE + quarter * 4096, row + 64 * half, pitch,
                                                    rows);
            if constexpr (kPacked)
              if (lane < rows && !(z == 0.f) && *static_cast<volatile int*>(pa.bad) == 0) *pa.bad = 1;
          }
          __syncwarp();   // read before the next item's dS goes there
          // dK and dV have been read: the next key block's first products may
          // overwrite them (they follow this thread's next p_ready / ds_ready)
          tc_fence_before();
        }
        g0 += n_it;
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// ---------------------------------------------------------- backward prepass

// D[b, h, t] = sum_i dO[b, t, h, i] * O[b, t, h, i]
__global__ void attn_bwd_dot_kernel(const bf16* __restrict__ o, const bf16* __restrict__ dout,
                                    float* __restrict__ Dv, int B, int H, int T) {
  const long long w = static_cast<long long>(blockIdx.x) * (blockDim.x / 32) + warp_id();
  if (w >= static_cast<long long>(B) * H * T) return;
  const int t = static_cast<int>(w % T);
  const int h = static_cast<int>((w / T) % H);
  const int b = static_cast<int>(w / (static_cast<long long>(T) * H));
  const long long off = ((static_cast<long long>(b) * T + t) * H + h) * HD + lane_id() * 4;
  const uint2 x = *reinterpret_cast<const uint2*>(o + off);
  const uint2 y = *reinterpret_cast<const uint2*>(dout + off);
  float s = bf16_lo(x.x) * bf16_lo(y.x) + bf16_hi(x.x) * bf16_hi(y.x) + bf16_lo(x.y) * bf16_lo(y.y) +
            bf16_hi(x.y) * bf16_hi(y.y);
  s = warp_sum(s);
  if (lane_id() == 0) Dv[w] = s;
}

// --------------------------------------------------- packed: plan and setup

// A plan: kPlanMeta words, lo and hi [T], forward entries [tiles], backward
// entries [key blocks].
struct PlanView {
  int* meta;
  int* lo;
  int* hi;
  int2* fwd;
  int2* bwd;
  size_t bytes;
};
__host__ __device__ inline PlanView plan_view(void* base, int T) {
  const size_t n = (static_cast<size_t>(T) + 1) / 2 * 2, nq = (static_cast<size_t>(T) + 127) / 128;
  int* p = static_cast<int*>(base);
  PlanView v;
  v.meta = p;
  v.lo = p + kPlanMeta;
  v.hi = v.lo + n;
  v.fwd = reinterpret_cast<int2*>(v.hi + n);
  v.bwd = v.fwd + nq;
  v.bytes = (kPlanMeta + 2 * n) * sizeof(int) + 2 * nq * sizeof(int2);
  return v;
}

// Sequence [start, end) of position p < total.  Offsets that are not in order
// give some range that still holds p.
struct SeqRange { int start, end; };
__device__ __forceinline__ SeqRange seq_range(const int* cu, int n_seq, int T, int p) {
  int l = 0, r = n_seq - 1;   // the last s with cu[s] <= p
  while (l < r) {
    const int m = (l + r + 1) >> 1;
    if (cu[m] <= p) l = m;
    else r = m - 1;
  }
  return SeqRange{max(0, min(cu[l], p)), min(T, max(cu[l + 1], p + 1))};
}

// Blocks from the third on fill lo and hi; the first two check the offsets (in
// order, from 0, at most T; otherwise nothing is covered and the error is
// latched) and sort the work entries, the first the forward's, the second the
// backward's, by their number of 128 x 128 steps with a counting sort (longest
// first; entries of one length in no fixed order, which no output of the
// forward depends on).  Bound by latency: the offsets are searched in shared
// memory (up to kPlanSeqs; 4.4 us instead of 7.5 for 46 sequences).
constexpr int kPlanSeqs = 4095;
__global__ void __launch_bounds__(1024)
    attention_plan_kernel(const int* __restrict__ cu_arg, int n_seq, int T, int window, void* plan, int* err) {
  chain_go();
  constexpr int kBuckets = 1024;
  __shared__ int cu_s[kPlanSeqs + 1];
  __shared__ int hist[kBuckets];
  __shared__ int warp_total[32];
  const PlanView P = plan_view(plan, T);
  const int wl = window < 0 ? T : window, tid = threadIdx.x;
  const int* cu = cu_arg;
  if (n_seq <= kPlanSeqs) {
    for (int i = tid; i <= n_seq; i += 1024) cu_s[i] = cu_arg[i];
    hist[tid] = 0;
    __syncthreads();
    cu = cu_s;
  } else {
    hist[tid] = 0;
  }
  const int last = n_seq > 0 ? cu[n_seq] : 0, total = max(0, min(last, T));
  auto lo_of = [&](int t) { return max(seq_range(cu, n_seq, T, t).start, t - min(wl, t)); };
  auto hi_of = [&](int t) { return min(seq_range(cu, n_seq, T, t).end - 1, t + min(wl, T - 1 - t)); };
  if (blockIdx.x > 1) {
    const int t = (blockIdx.x - 2) * 1024 + tid;
    if (t >= T) return;
    P.lo[t] = t < total ? lo_of(t) : 0;
    P.hi[t] = t < total ? hi_of(t) : -1;
    return;
  }
  const int dir = blockIdx.x;
  int bad = (n_seq > 0 && cu[0] != 0) || last > T;
  for (int i = tid; i < n_seq; i += 1024) bad |= cu[i + 1] < cu[i];
  bad = __syncthreads_or(bad);
  const int valid = bad ? 0 : total;
  if (dir == 0 && tid == 0) {
    if (bad && err) atomicOr(err, ERRF_SEQUENCE);
    P.meta[kMetaTotal] = valid;
    P.meta[kMetaT] = T;
    P.meta[kMetaMagic] = kPlanMagic;
  }
  const int count = (valid + 127) / 128;
  // entry e, and its steps
  auto entry = [&](int e, int* steps) -> int2 {
    if (dir) {   // hi grows with the key
      *steps = (hi_of(min(e * 128 + 127, valid - 1)) >> 7) - e + 1;
      return make_int2(e, *steps);
    }
    const int a = lo_of(e * 128) >> 7;
    *steps = e + 1 - a;
    return make_int2(e, a);
  };
  auto bucket = [](int steps) { return kBuckets - min(steps, kBuckets); };
  int steps = 0;
  int2 mine = make_int2(0, 0);   // each thread's first entry is searched once
  if (tid < count) {
    mine = entry(tid, &steps);
    atomicAdd(&hist[bucket(steps)], 1);
  }
  for (int e = tid + 1024; e < count; e += 1024) {
    int n;
    entry(e, &n);
    atomicAdd(&hist[bucket(n)], 1);
  }
  __syncthreads();
  // exclusive sums of the 1024 buckets, one per thread
  const int in_bucket = hist[tid];
  int x = in_bucket;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane_id() >= o) x += y;
  }
  if (lane_id() == 31) warp_total[warp_id()] = x;
  __syncthreads();
  int before = x - in_bucket;
  for (int w = 0; w < warp_id(); ++w) before += warp_total[w];
  if (tid == 0) P.meta[dir ? kMetaBwd : kMetaFwd] = count;
  hist[tid] = before;
  __syncthreads();
  int2* order = dir ? P.bwd : P.fwd;
  if (tid < count) order[atomicAdd(&hist[bucket(steps)], 1)] = mine;
  for (int e = tid + 1024; e < count; e += 1024) {
    int n;
    const int2 v = entry(e, &n);
    order[atomicAdd(&hist[bucket(n)], 1)] = v;
  }
}

// Control words and tensor maps of one packed backward, by one warp.  A plan
// made for another T is refused: no entries, the error latched.
struct SetupMaps {
  CUtensorMap m[4];
};
__device__ __forceinline__ void packed_setup(const SetupMaps& in, CUtensorMap* out, int* ctl, const int* meta, int T,
                                             int* err, CUtensorMap* stage) {
  const int lane = lane_id();
  const PlanSizes plan = plan_sizes(meta, T);
  const int valid = plan.valid;
  if (lane == 0) {
    if (!plan.fits && err) atomicOr(err, ERRF_SHAPE);
    ctl[kCtlSched] = 0;
    ctl[kCtlBad] = 0;
    ctl[kCtlEntries] = plan.bwd;
    ctl[kCtlValid] = plan.fits ? valid : -1;   // -1: no output is touched
  }
  for (int i = 0; i < 4; ++i)
    reinterpret_cast<uint32_t*>(&stage[i])[lane] = reinterpret_cast<const uint32_t*>(&in.m[i])[lane];
  __syncwarp();
  if (lane == 0 && valid > 0 && valid < T) {
    // the token extent (dimension 1 of q, k, v; 2 of dO) ends with the sequences
    for (int i = 0; i < 3; ++i)
      asm volatile("tensormap.replace.tile.global_dim.shared::cta.b1024.b32 [%0], 1, %1;" ::"r"(smem_u32(&stage[i])),
                   "r"(valid)
                   : "memory");
    asm volatile("tensormap.replace.tile.global_dim.shared::cta.b1024.b32 [%0], 2, %1;" ::"r"(smem_u32(&stage[3])),
                 "r"(valid)
                 : "memory");
  }
  __syncwarp();
  for (int i = 0; i < 4; ++i)
    asm volatile(
        "tensormap.cp_fenceproxy.global.shared::cta.tensormap::generic.release.gpu.sync.aligned [%0], [%1], 128;" ::"l"(
            out + i),
        "r"(smem_u32(&stage[i]))
        : "memory");
}

// Before the backward, for the rows that hold sequences: nd = -D, D[h, t] = sum_j
// P_tj dP_tj over the keys that t sees, dP_tj = dO_t . v_j; nl = -lse in log2
// units; both [H][T rounded up to 128] and filled up to the end of the last
// row's tile (nl -inf: P = 0); zeros in the fp32 dq accumulator; and the
// backward's setup.
//
// D could be had as dO_t . o_t from the forward's o, in 50 us instead of 150 to 165
// (32,768 tokens of documents, 10 heads), but o is rounded to bf16, and dS = P (dP
// - D) would carry the whole error of D in rows whose probability sits on one
// key, where dP - D of that key is small: dq and dk were then off by 0.004 to
// 0.008 of their norm on sequences of 2 to 40 tokens, against 0.0024 now.  So the
// kernel takes P and dP as the backward will, S = Q K^T and dP = dO V^T into TMEM
// and P = exp(S - lse), and divides by sum_j P_tj, which makes the row sums of dS
// vanish to fp32.
//
// Persistent, a block an SM, items by cluster launch control as in the
// forward.  608 threads:
//   warps 0..15 two groups of eight, group b for every other key block, in TMEM
//               columns 256 b (S) and 256 b + 128 (dP); two threads for a query
//               row (TMEM lane), each 64 of the block's keys; the four sums of a
//               row meet in shared memory.  (One thread a row and group took
//               a fifth longer.)
//   warp 16     TMA: takes the items and publishes them in a shared ring; loads
//               Q and dO, and K_j and V_j through two-slot rings
//   warp 17     TMEM owner and MMA issuer
//   warp 18     the backward's setup (every block writes the same words)
// DRAM alone takes 75 us (q, k, v, dO read, the zeros written), the products by
// themselves 55, waiting for each tile's Q and dO 51 (3 us a tile); what overlaps
// of these leaves the tensor pipe 41% busy and the issue slots 33%.  Second buffers
// for Q and dO gained 3% alone and nothing in whole passes, where the clock falls
// with the power drawn; two tiles that share their key blocks load half as
// much, but leave no second buffer of S and dP: 193 us against 161.
constexpr int PD_SUMS = 2 * 3 * 128 * 8;
constexpr int PD_SMEM = 6 * TF_BUF + PD_SUMS + 4 * static_cast<int>(sizeof(CUtensorMap)) + 256;

template <bool kFine>
__global__ void __launch_bounds__(608, 1)
    attention_packed_dot_kernel(const __grid_constant__ SetupMaps in, CUtensorMap* maps, int* ctl,
                                const float* __restrict__ lse, float* __restrict__ nl, float* __restrict__ nd,
                                float* __restrict__ dq, int H, int Hkv, int T, float scale_log2, int* err,
                                long long wait_cycles, const PackedArgs pk) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  // the 128-byte-swizzled tiles need a 1024-byte-aligned base, which the
  // dynamic shared memory window provides; refuse to run otherwise
  if (smem_u32(smem_raw) & 1023u) {
    chain_wait();
    if (threadIdx.x == 0) {
      if (err) atomicOr(err, ERRF_SHAPE);
      ctl[kCtlSched] = ctl[kCtlEntries] = ctl[kCtlBad] = 0;   // no backward either
      ctl[kCtlValid] = -1;
    }
    return;
  }
  uint8_t* sQ = smem_raw;
  uint8_t* sdO = smem_raw + TF_BUF;
  uint8_t* sK = smem_raw + 2 * TF_BUF;   // two slots
  uint8_t* sV = smem_raw + 4 * TF_BUF;   // two slots
  float2* sums = reinterpret_cast<float2*>(smem_raw + 6 * TF_BUF);   // [2][3][128]: sums of P and P dP, item n & 1
  CUtensorMap* stage = reinterpret_cast<CUtensorMap*>(smem_raw + 6 * TF_BUF + PD_SUMS);
  uint4* answer = reinterpret_cast<uint4*>(stage + 4);   // next_block_ask's
  uint64_t* bars = reinterpret_cast<uint64_t*>(answer + 1);
  uint64_t* q_full = bars + 0;     // Q and dO of item n landed (or the end marker)
  uint64_t* q_empty = bars + 1;    // item n's products done and every row warp has its fields
  uint64_t* kv_full = bars + 2;    // [2]
  uint64_t* kv_empty = bars + 4;   // [2]
  uint64_t* sd_full = bars + 6;    // [2] per group: S and dP of a block in TMEM
  uint64_t* sd_empty = bars + 8;   // [2] per group: they have been read
  uint64_t* part = bars + 10;      // [2]: the sums of item n, n & 1, are in shared memory
  uint64_t* drain = bars + 12;
  uint64_t* answered = bars + 13;
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(bars + 14);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_holder + 1);
  // [4][4]: head (-1: end), tile, first key block
  volatile int* item_ring = reinterpret_cast<volatile int*>(tmem_holder + 2);

  const int warp = warp_id(), lane = lane_id();
  const long long wlim = wait_limit_or_default(wait_cycles);

  if (threadIdx.x == 0) {
    mbar_init(q_full, 1);
    mbar_init(q_empty, 1 + 16);   // the MMA commit and one arrival per row warp
    for (int i = 0; i < 2; ++i) {
      mbar_init(&kv_full[i], 1); mbar_init(&kv_empty[i], 1);
      mbar_init(&sd_full[i], 1); mbar_init(&sd_empty[i], 256); mbar_init(&part[i], 384);
    }
    mbar_init(drain, 1);
    mbar_init(answered, 1);
    *abort_flag = 0;
    fence_barrier_init();
    for (int i = 0; i < 4; ++i) tma_prefetch_desc(&in.m[i]);
  }
  if (warp == 17) {
    tmem_alloc(tmem_holder, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_holder;
  chain_wait();
  // positions that hold sequences; a plan of another T is refused (by the setup)
  const PlanSizes plan = plan_sizes(pk.meta, T);
  const int Tv = plan.valid;

  if (warp == 18) {
    packed_setup(in, maps, ctl, pk.meta, T, err, stage);
  } else if (warp == 16) {
    if (lane == 0) {
      // -------------------------------------------------------------- TMA
      // item number and fields are fetched one item ahead, as in the forward
      const int entries = plan.fwd, n_items = entries * H;
      int nx_h = -1;
      int2 nx = make_int2(0, 0);
      bool asked = false;
      uint32_t answers = 0;
      auto fetch = [&](int idx) {   // false: a block without work (tiles past the sequences)
        if (idx >= n_items) return false;
        const int h = idx / entries;
        nx = __ldg(pk.fwd + (idx - h * entries));
        if (!fwd_entry_ok(nx, Tv, err)) return false;
        nx_h = h;
        return true;
      };
      auto take = [&] {   // false: the wait expired
        nx_h = -1;
        while (asked) {
          if (!mbar_wait_t<kFine>(answered, answers & 1, abort_flag, err, wlim)) return false;
          ++answers;
          asked = false;
          const int idx = next_block_answer(answer);
          if (idx < 0 || fetch(idx)) break;
          next_block_ask(answer, answered);
          asked = true;
        }
        return true;
      };
      fetch(blockIdx.x);
      bool ok = true;
      uint32_t g = 0;     // key blocks loaded so far
      int last_q = -1;    // last item whose Q was loaded
      for (int n = 0;; ++n) {
        // the previous item's Q and dO are no longer read and every warp has its fields
        if (n > 0 && !mbar_wait_t<kFine>(q_empty, (n - 1) & 1, abort_flag, err, wlim)) { ok = false; break; }
        volatile int* f = item_ring + 4 * (n & 3);
        const int h = nx_h, qt = nx.x, j0 = nx.y;
        f[0] = h; f[1] = qt; f[2] = j0;
        if (h < 0) {
          mbar_arrive(q_full);   // end marker: releases the ring entry
          break;
        }
        next_block_ask(answer, answered);
        asked = true;
        const int hk = h / (H / Hkv);
        mbar_arrive_expect_tx(q_full, 2 * TF_BUF);
        for (int c = 0; c < 2; ++c) {
          tma_load_3d(sQ + c * TF_TILE, &in.m[0], q_full, 64 * c, qt * 128, h);
          tma_load_4d(sdO + c * TF_TILE, &in.m[3], q_full, 64 * c, h, qt * 128, 0);
        }
        last_q = n;
        for (int j = j0; j <= qt; ++j, ++g) {
          const uint32_t s = g & 1;
          if (!mbar_wait_t<kFine>(&kv_empty[s], ((g >> 1) & 1) ^ 1u, abort_flag, err, wlim)) { ok = false; break; }
          mbar_arrive_expect_tx(&kv_full[s], 2 * TF_BUF);
          for (int c = 0; c < 2; ++c) {
            tma_load_3d(sK + s * TF_BUF + c * TF_TILE, &in.m[1], &kv_full[s], 64 * c, j * 128, hk);
            tma_load_3d(sV + s * TF_BUF + c * TF_TILE, &in.m[2], &kv_full[s], 64 * c, j * 128, hk);
          }
          if (j == j0 && !take()) { ++g; ok = false; break; }
        }
        if (!ok) break;
      }
      if (!ok) {
        // let the copies already started land before the CTA exits
        if (asked)
          for (uint32_t i = 0; i < (1u << 20) && !mbar_try_wait(answered, answers & 1); ++i) {}
        if (last_q >= 0)
          for (uint32_t i = 0; i < (1u << 20) && !mbar_try_wait(q_full, last_q & 1); ++i) {}
        for (uint32_t x = g > 2 ? g - 2 : 0; x < g; ++x)
          for (uint32_t i = 0; i < (1u << 20) && !mbar_try_wait(&kv_full[x & 1], (x >> 1) & 1); ++i) {}
      }
    }
  } else if (warp == 17) {
    // -------------------------------------------------------------- MMA
    // the whole warp, converged; one lane issues
    const bool leader = elect_lane();
    const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
    auto wait1 = [&](uint64_t* bar, uint32_t par) -> bool {
      return __all_sync(0xffffffffu, mbar_wait_t<kFine>(bar, par, abort_flag, err, wlim));
    };
    constexpr uint32_t IDESC = make_idesc(1, 128, false, false);
    // X = A B^T over the 128 head dims, both operands K-major
    auto product = [&](uint32_t d_tmem, const uint8_t* a, const uint8_t* b) {
      const uint64_t da = smem_desc_sw128(smem_u32(a), 16, 1024), db = smem_desc_sw128(smem_u32(b), 16, 1024);
#pragma unroll
      for (int kk = 0; kk < 8; ++kk) {
        const uint32_t off16 = ((kk >> 2) * TF_TILE + (kk & 3) * 32) >> 4;
        umma_f16_by(leader, d_tmem, da + off16, db + off16, IDESC, kk > 0 ? 1u : 0u);
      }
    };
    bool ok = true;
    uint32_t g = 0;   // key blocks done so far
    for (int n = 0; ok; ++n) {
      if (!wait1(q_full, n & 1)) break;
      const volatile int* f = item_ring + 4 * (n & 3);
      const int h = __shfl_sync(0xffffffffu, f[0], 0), qt = __shfl_sync(0xffffffffu, f[1], 0);
      const int j0 = __shfl_sync(0xffffffffu, f[2], 0);
      if (h < 0) break;
      for (int j = j0; j <= qt; ++j, ++g) {
        const uint32_t s = g & 1, use = (g >> 1) & 1;
        if (!wait1(&kv_full[s], use) || !wait1(&sd_empty[s], use ^ 1u)) { ok = false; break; }
        tc_fence_after();
        product(tm + 256 * s, sQ, sK + s * TF_BUF);
        product(tm + 256 * s + 128, sdO, sV + s * TF_BUF);
        umma_commit_by(leader, &sd_full[s]);
        umma_commit_by(leader, &kv_empty[s]);
        if (j == qt) umma_commit_by(leader, q_empty);   // the item's last products
      }
    }
    umma_commit_by(leader, drain);
    for (uint32_t i = 0; i < (1u << 22) && !mbar_try_wait(drain, 0); ++i) {}
  } else {
    // ------------------------------------------------------------- rows
    const int grp = warp >> 3, half = (warp >> 2) & 1, quarter = warp & 3;
    const uint32_t t_s = tmem + (static_cast<uint32_t>(quarter * 32) << 16) + 256 * grp, t_d = t_s + 128;
    const uint64_t sl2 = f2_pack(scale_log2, scale_log2);
    const int pitch = (T + 127) / 128 * 128;
    bool ok = true;
    uint32_t g = 0;   // key blocks so far, both groups'
    auto wait_all = [&](uint64_t* bar, uint32_t par) -> bool {
      return __all_sync(0xffffffffu, mbar_wait_t<kFine>(bar, par, abort_flag, err, wlim));
    };
    for (int n = 0; ok; ++n) {
      if (!wait_all(q_full, n & 1)) break;
      const volatile int* f = item_ring + 4 * (n & 3);
      const int h = f[0], qt = f[1], j0 = f[2];
      __syncwarp();
      if (lane == 0) mbar_arrive(q_empty);   // this warp has the fields
      if (h < 0) break;
      const int r = quarter * 32 + lane, q = qt * 128 + r;
      const bool row = q < Tv;
      const int lo = row ? __ldg(pk.lo + q) : 0;   // first key of the row
      const int lo_max = __reduce_max_sync(0xffffffffu, lo);
      const float m = row ? lse[static_cast<long long>(h) * T + q] * -1.4426950408889634f : -INFINITY;
      const uint64_t m2 = f2_pack(m, m);
      // zeros for the sums of dq, each warp every sixteenth row
      for (int x = qt * 128 + warp; x < min(qt * 128 + 128, Tv); x += 16)
        reinterpret_cast<float4*>(dq + (static_cast<long long>(h) * T + x) * HD)[lane] =
            make_float4(0.f, 0.f, 0.f, 0.f);
      uint64_t l2 = f2_pack(0.f, 0.f), d2 = l2;   // sums of P and of P dP
      for (int j = j0; j <= qt; ++j, ++g) {
        if (static_cast<int>(g & 1) != grp) continue;
        if (!wait_all(&sd_full[grp], (g >> 1) & 1)) { ok = false; break; }
        tc_fence_after();
        const int kbase = j * 128;
        const bool masked = j == qt || kbase < lo_max;
        const int first = lo - kbase, end = q + 1 - kbase;   // keys that this row sees: first .. end - 1
        auto add = [&](const uint32_t (&x)[32], const uint32_t (&y)[32]) {
#pragma unroll
          for (int k = 0; k < 32; k += 2) {
            float x0, x1;
            f2_unpack(f2_fma(f2_pack(__uint_as_float(x[k]), __uint_as_float(x[k + 1])), sl2, m2), x0, x1);
            const uint64_t p = f2_pack(ex2_approx(x0), ex2_approx(x1));
            l2 = f2_add(l2, p);
            d2 = f2_fma(p, f2_pack(__uint_as_float(y[k]), __uint_as_float(y[k + 1])), d2);
          }
        };
#pragma unroll 1
        for (int c = 2 * half; c < 2 * half + 2; ++c) {
          const uint32_t seen = masked ? low_bits(end - 32 * c) & ~low_bits(first - 32 * c) : ~0u;
          if (!__any_sync(0xffffffffu, seen != 0)) continue;
          uint32_t x[32], y[32];
          tmem_load32_async(t_s + 32 * c, x);
          tmem_load32_async(t_d + 32 * c, y);
          tmem_landed(x);
          tmem_landed(y);
          if (masked) {
            mask_scores(x, seen);
#pragma unroll
            for (int k = 0; k < 32; ++k)
              if (!(seen & (1u << k))) y[k] = 0u;   // P = 0 would not remove a NaN
          }
          add(x, y);
        }
        tc_fence_before();
        mbar_arrive(&sd_empty[grp]);
      }
      if (!ok) break;
      float l0, l1, d0, d1;
      f2_unpack(l2, l0, l1);
      f2_unpack(d2, d0, d1);
      float2 mine = make_float2(l0 + l1, d0 + d1);
      const int who = warp >> 2;   // group and half
      float2* row_sums = sums + (n & 1) * 3 * 128 + r;
      if (who > 0) {
        // item n - 2's sums have been read: this item was published after every warp had taken the one before
        row_sums[(who - 1) * 128] = mine;
        mbar_arrive(&part[n & 1]);
      } else {
        if (!wait_all(&part[n & 1], (n >> 1) & 1)) break;
#pragma unroll
        for (int x = 0; x < 3; ++x) {
          mine.x += row_sums[x * 128].x;
          mine.y += row_sums[x * 128].y;
        }
        const long long at = static_cast<long long>(h) * pitch + q;
        nl[at] = m;
        nd[at] = row ? -mine.y / mine.x : 0.f;
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 17) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// What the last kernels of a backward need beside dq's sums.
struct FinishArgs {
  HeadRows q, k, v, dout, dq, dk, dv;   // the last three are written
  const int* ctl;
  const int* lo;
  const int* hi;
  const float* nl;   // [H][T rounded up to 128]
  const float* nd;
  int H, Hkv, T, clear;
  float scale;
};
__device__ __forceinline__ bf16* row_of(const HeadRows& r, int t, int h) {
  return const_cast<bf16*>(r.ptr) + t * r.tok + h * r.head;
}

// dq of query t of head h, which sees the keys lo[t] .. t of those that its tile
// visits.
__device__ __noinline__ void repair_dq_row(const FinishArgs& a, int valid, int t, int h) {
  if (finite_row(row4(a.dq, t, h))) return;
  const float4 q = row4(a.q, t, h), d = row4(a.dout, t, h);
  const long long at = static_cast<long long>(h) * ((a.T + 127) / 128 * 128) + t;
  const float nl = a.nl[at], nd = a.nd[at];
  if (!finite_row(q) || !finite_row(d) || !isfinite(nl) || !isfinite(nd)) return;
  const int hk = h / (a.H / a.Hkv), last = min(t | 127, valid - 1);
  const int first = min(max(a.lo[t & ~127], 0), t) & ~127, lo = min(max(a.lo[t], first), t);
  bool clean = true;
  for (int j = first; j <= last && clean; ++j)
    if (j < lo || j > t) clean = finite_row(row4(a.k, j, hk)) && finite_row(row4(a.v, j, hk));
  if (clean) return;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int j = t; j >= lo; --j) {
    const float4 k = row4(a.k, j, hk), v = row4(a.v, j, hk);
    if (!finite_row(k) || !finite_row(v)) return;
    const float p = ex2_approx(fmaf(dot_row(q, k), a.scale * 1.4426950408889634f, nl));
    add_row(acc, p * (dot_row(d, v) + nd), k);
  }
  put_row(row_of(a.dq, t, h), a.scale, acc);
}

// dk and dv of key j of kv head hk, which the queries j .. hi[j] see of those
// that its block visits.
__device__ __noinline__ void repair_dkv_row(const FinishArgs& a, int valid, int j, int hk) {
  if (finite_row(row4(a.dk, j, hk)) && finite_row(row4(a.dv, j, hk))) return;
  const float4 k = row4(a.k, j, hk), v = row4(a.v, j, hk);
  if (!finite_row(k) || !finite_row(v)) return;
  const int G = a.H / a.Hkv, hi = min(max(a.hi[j], j), valid - 1);
  const int last = min(a.hi[min(j | 127, valid - 1)] | 127, valid - 1);
  const long long pitch = (a.T + 127) / 128 * 128;
  bool clean = true;
  for (int t = j & ~127; t <= last && clean; ++t)
    for (int h = hk * G; h < (hk + 1) * G && clean && (t < j || t > hi); ++h)
      clean = finite_row(row4(a.q, t, h)) && finite_row(row4(a.dout, t, h)) && isfinite(a.nl[h * pitch + t]) &&
              isfinite(a.nd[h * pitch + t]);
  if (clean) return;
  float4 sk = make_float4(0.f, 0.f, 0.f, 0.f), sv = sk;
  for (int t = j; t <= hi; ++t)
    for (int h = hk * G; h < (hk + 1) * G; ++h) {
      const float4 q = row4(a.q, t, h), d = row4(a.dout, t, h);
      const float nl = a.nl[h * pitch + t], nd = a.nd[h * pitch + t];
      if (!finite_row(q) || !finite_row(d) || !isfinite(nl) || !isfinite(nd)) return;
      const float p = ex2_approx(fmaf(dot_row(q, k), a.scale * 1.4426950408889634f, nl));
      add_row(sk, p * (dot_row(d, v) + nd), q);
      add_row(sv, p, d);
    }
  put_row(row_of(a.dk, j, hk), a.scale, sk);
  put_row(row_of(a.dv, j, hk), 1.f, sv);
}

// dq in bf16 from the fp32 sums, rows that hold sequences; zeros in the rows past
// them of the gradients that `clear` names (kClear*).  A warp takes
// kRowsPerWarp rows, whose loads are issued together.
constexpr int kRowsPerWarp = 4;
__global__ void __launch_bounds__(256)
    attention_packed_dq_kernel(const float* __restrict__ acc, bf16* __restrict__ dq, long long dq_tok,
                               long long dq_head, int* ctl, const __grid_constant__ FinishArgs a) {
  chain_go();
  chain_wait();
  const int H = a.H, T = a.T, rows = ctl[kCtlValid] * H, w = (blockIdx.x * 8 + warp_id()) * kRowsPerWarp;
  if (rows < 0) return;
  if (a.clear && w + kRowsPerWarp > rows) {
    for (int x = max(w, rows); x < min(w + kRowsPerWarp, T * H); ++x) {
      const int t = x / H, h = x - t * H;
      const float4 zero = make_float4(0.f, 0.f, 0.f, 0.f);
      if (a.clear & kClearDq) put_row(dq + t * dq_tok + h * dq_head, 1.f, zero);
      if (h >= a.Hkv) continue;
      if (a.clear & kClearDk) put_row(row_of(a.dk, t, h), 1.f, zero);
      if (a.clear & kClearDv) put_row(row_of(a.dv, t, h), 1.f, zero);
    }
  }
  float4 v[kRowsPerWarp];
#pragma unroll
  for (int i = 0; i < kRowsPerWarp; ++i) {
    if (w >= rows - i) break;
    const int t = (w + i) / H, h = w + i - t * H;
    v[i] = reinterpret_cast<const float4*>(acc + static_cast<long long>(h * T + t) * HD)[lane_id()];
  }
  bool finite = true;
#pragma unroll
  for (int i = 0; i < kRowsPerWarp; ++i) {
    if (w >= rows - i) break;
    const int t = (w + i) / H, h = w + i - t * H;
    put_row(dq + t * dq_tok + h * dq_head, 1.f, v[i]);
    finite &= finite4(v[i]);
  }
  // the word is set once or a few times: in a batch of NaN a store from every warp took 450 us
  if (!finite && *static_cast<volatile int*>(ctl + kCtlBad) == 0) ctl[kCtlBad] = 1;
}

// The end of a backward whose gradients are not all finite: the rows that need
// not be so.  Returns at once otherwise (in the kernel before, the same work
// doubled its time by its registers).
__global__ void __launch_bounds__(256) attention_packed_repair_kernel(const __grid_constant__ FinishArgs a) {
  chain_wait();
  if (!a.ctl[kCtlBad]) return;
  const int valid = a.ctl[kCtlValid], rows = valid * a.H, step = gridDim.x * 8;
  for (long long x = blockIdx.x * 8 + warp_id(); x < rows; x += step) {
    const int t = static_cast<int>(x) / a.H, h = static_cast<int>(x) - t * a.H;
    repair_dq_row(a, valid, t, h);
    if (h < a.Hkv) repair_dkv_row(a, valid, t, h);
  }
}

}  // namespace

// Window in tokens as the kernels take it: keys t - wl .. t; "no window" is a
// bound no row reaches (kept small enough that k0 + 127 + wl fits in an int).
static int window_bound(int window, int T) { return window < 0 || window >= T ? (1 << 30) : window; }


// Scheduler words for callers that bring none: a ring of 64 library-owned
// counters, one per launch in turn, each zeroed on the launch's stream
// before use (so up to 64 such launches may be in flight at once).
__device__ int g_sched_ring[64];

static int* sched_word(int* sched, cudaStream_t s) {
  if (!sched) {
    static std::atomic<unsigned> next{0};
    int* base = nullptr;
    if (cudaGetSymbolAddress(reinterpret_cast<void**>(&base), g_sched_ring) != cudaSuccess) return nullptr;
    sched = base + (next++ & 63u);
  }
  cudaMemsetAsync(sched, 0, sizeof(int), s);
  return sched;
}

void launch_attn_fwd(const bf16* q, const bf16* k, const bf16* v, bf16* o, float* lse, int B, int H, int T,
                     cudaStream_t s, int* err, int Hkv, int window, int* sched, int kv_stride,
                     long long wait_cycles) {
  // a limit shorter than one blocking probe needs the finely polling build
  const bool fine = wait_limit_or_default(wait_cycles) < kShortWaitCycles;
  auto kern = fine ? attn_fwd_tc_kernel<true> : attn_fwd_tc_kernel<false>;
  static std::atomic<unsigned long long> configured[2] = {};
  if (set_smem_limit_once(kern, TF_SMEM, configured[fine ? 1 : 0]) != cudaSuccess) {
    if (err) cudaMemsetAsync(err, 0xff, sizeof(int), s);   // latched as a device error
    return;
  }
  if (Hkv <= 0) Hkv = H;
  if (kv_stride <= 0) kv_stride = Hkv;
  CUtensorMap mq, mk, mv;
  const long long bh = 1ll * B * H, bhkv = 1ll * B * kv_stride;
  if (H % Hkv || kv_stride < Hkv || !make_map(&mq, q, 2, HD, T, bh, HD, 1ll * T * HD, 64, 128) ||
      !make_map(&mk, k, 2, HD, T, bhkv, HD, 1ll * T * HD, 64, 128) ||
      !make_map(&mv, v, 2, HD, T, bhkv, HD, 1ll * T * HD, 64, 128)) {
    if (err) cudaMemsetAsync(err, 0xff, sizeof(int), s);   // latched as a device error
    return;
  }
  // persistent: one CTA per SM over the pairs of query tiles of every head
  const long long n_items = ((T + 127) / 128 + 1) / 2 * bh;
  const int grid = static_cast<int>(std::min<long long>(n_items, device_sm_count()));
  const float scale_log2 = 1.4426950408889634f / sqrtf(static_cast<float>(HD));
  kern<<<grid, 384, TF_SMEM, s>>>(mq, mk, mv, o, lse, H, Hkv, kv_stride, T, window_bound(window, T),
                                                scale_log2,
                                                static_cast<int>(n_items), sched_word(sched, s), err, wait_cycles);
}

void launch_attn_bwd(const bf16* q, const bf16* k, const bf16* v, const bf16* o, const bf16* dout,
                     const float* lse, float* Dv, float* dq, bf16* dk, bf16* dv, int B, int H, int T,
                     cudaStream_t s, int* err, int Hkv, int window, int* sched, int kv_stride,
                     long long wait_cycles, const float* rk, const float2* rope, bf16* dqkv, bool d_ready) {
  const bool fine = wait_limit_or_default(wait_cycles) < kShortWaitCycles;
  auto kern = fine ? attn_bwd_tc_kernel<true, false> : attn_bwd_tc_kernel<false, false>;
  static std::atomic<unsigned long long> configured[2] = {};
  if (set_smem_limit_once(kern, TB_SMEM, configured[fine ? 1 : 0]) != cudaSuccess) {
    if (err) cudaMemsetAsync(err, 0xff, sizeof(int), s);   // latched as a device error
    return;
  }
  if (Hkv <= 0) Hkv = H;
  const long long rows = 1ll * B * H * T;
  if (!d_ready) attn_bwd_dot_kernel<<<static_cast<int>((rows + 7) / 8), 256, 0, s>>>(o, dout, Dv, B, H, T);
  cudaMemsetAsync(dq, 0, static_cast<size_t>(rows) * HD * sizeof(float), s);
  CUtensorMap mq, mk, mv, mdo, mdq;
  if (kv_stride <= 0) kv_stride = Hkv;
  const long long bh = 1ll * B * H, bhkv = 1ll * B * kv_stride;
  const long long dims[4] = {HD, H, T, B};
  const long long strides[3] = {HD * 2ll, 1ll * H * HD * 2, 1ll * T * H * HD * 2};
  const int box[4] = {64, 1, 128, 1};
  if (H % Hkv || kv_stride < Hkv || !make_map(&mq, q, 2, HD, T, bh, HD, 1ll * T * HD, 64, 128) ||
      !make_map(&mk, k, 2, HD, T, bhkv, HD, 1ll * T * HD, 64, 128) ||
      !make_map(&mv, v, 2, HD, T, bhkv, HD, 1ll * T * HD, 64, 128) || !make_map_4d(&mdo, dout, dims, strides, box) ||
      !make_map(&mdq, dq, 4, HD, T, bh, HD, 1ll * T * HD, 32, 32)) {
    if (err) cudaMemsetAsync(err, 0xff, sizeof(int), s);
    return;
  }
  // persistent: one CTA per SM over units of two key blocks of every kv head.
  // Without a window every unit costs the same and a fixed stride spreads
  // them evenly (measured ~3% faster than the counter, which claims each
  // CTA's next unit ahead of time); with one, unit costs differ and the
  // counter balances them.
  const long long n_units = 1ll * B * Hkv * (((T + 127) / 128 + 1) / 2);
  const int grid = static_cast<int>(std::min<long long>(n_units, device_sm_count()));
  const int wl = window_bound(window, T);
  int* word = wl >= T ? nullptr : sched_word(sched, s);
  kern<<<grid, 512, TB_SMEM, s>>>(mq, mk, mv, mdo, mdq, lse, Dv, dk, dv, H, Hkv, kv_stride, T, wl,
                                                1.f / sqrtf(static_cast<float>(HD)), static_cast<int>(n_units),
                                                word, err, wait_cycles, rk, rope, dqkv, PackedArgs{});
}

// ---------------------------------------------------------- packed launchers

namespace {

constexpr size_t al256(size_t x) { return (x + 255) / 256 * 256; }

// scratch of a backward: control words, then the four tensor maps
constexpr size_t kPackedHead = 256 + 4 * sizeof(CUtensorMap);

// Strides of an extent-1 dimension are never used: any legal value stands in.
long long stride_or(long long extent, long long stride) { return extent > 1 ? stride : HD; }

HeadRows head_rows(const PackedTensor& t) { return HeadRows{static_cast<const bf16*>(t.ptr), t.tok, t.head}; }

bool map_heads(CUtensorMap* m, const PackedTensor& t, long long tokens, long long heads) {
  return make_map(m, t.ptr, 2, HD, tokens, heads, stride_or(tokens, t.tok), stride_or(heads, t.head), 64, 128);
}

}  // namespace

size_t attention_plan_bytes(int T) { return al256(plan_view(nullptr, T).bytes); }

// then -lse and -D, [H][T rounded up to 128] each, and the fp32 dq [H][T][128]
size_t attention_packed_bwd_scratch(int T, int H) {
  const size_t padded = (static_cast<size_t>(T) + 127) / 128 * 128 * H, rows = static_cast<size_t>(T) * H;
  return al256(kPackedHead) + 2 * al256(padded * sizeof(float)) + al256(rows * HD * sizeof(float));
}

void launch_attention_plan(const int* cu, int n_seq, int T, int window, void* plan, int* err, cudaStream_t s) {
  attention_plan_kernel<<<2 + (T + 1023) / 1024, 1024, 0, s>>>(cu, n_seq, T, window, plan, err);
}

cudaError_t launch_attn_packed_fwd(const PackedTensor& q, const PackedTensor& k, const PackedTensor& v,
                                   const PackedTensor& o, float* lse, int H, int Hkv, int T, float scale,
                                   const void* plan, int clear, cudaStream_t s, int* err, long long wait_cycles) {
  const bool fine = wait_limit_or_default(wait_cycles) < kShortWaitCycles;
  auto kern = fine ? attn_packed_fwd_kernel<true> : attn_packed_fwd_kernel<false>;
  static std::atomic<unsigned long long> configured[2] = {};
  cudaError_t e = set_smem_limit_once(kern, PF_SMEM, configured[fine ? 1 : 0]);
  if (e != cudaSuccess) return e;
  CUtensorMap mq, mk, mv;
  if (!map_heads(&mq, q, T, H) || !map_heads(&mk, k, T, Hkv) || !map_heads(&mv, v, T, Hkv))
    return cudaErrorInvalidValue;
  const PlanView P = plan_view(const_cast<void*>(plan), T);
  PackedArgs pa = {};
  pa.meta = P.meta;
  pa.lo = P.lo;
  pa.fwd = P.fwd;
  pa.o_tok = o.tok;
  pa.o_head = o.head;
  pa.clear = clear;
  pa.q = head_rows(q);
  pa.k = head_rows(k);
  pa.v = head_rows(v);
  const int items = (T + 127) / 128 * H;   // a block each; most are taken over before they start
  return launch_chained(kern, items, 192, PF_SMEM, s, mq, mk, mv, static_cast<bf16*>(const_cast<void*>(o.ptr)), lse, H,
                        Hkv, T, scale * 1.4426950408889634f, err, wait_cycles, pa);
}

cudaError_t launch_attn_packed_bwd(const PackedTensor& q, const PackedTensor& k, const PackedTensor& v,
                                   const PackedTensor& dout, const float* lse, const PackedTensor& dq,
                                   const PackedTensor& dk, const PackedTensor& dv, int H, int Hkv, int T, float scale,
                                   const void* plan, void* scratch, int clear, cudaStream_t s, int* err,
                                   long long wait_cycles) {
  const bool fine = wait_limit_or_default(wait_cycles) < kShortWaitCycles;
  auto kern = fine ? attn_bwd_tc_kernel<true, true> : attn_bwd_tc_kernel<false, true>;
  auto dot = fine ? attention_packed_dot_kernel<true> : attention_packed_dot_kernel<false>;
  static std::atomic<unsigned long long> configured[4] = {};
  cudaError_t e = set_smem_limit_once(kern, TB_SMEM, configured[fine ? 1 : 0]);
  if (e == cudaSuccess) e = set_smem_limit_once(dot, PD_SMEM, configured[fine ? 3 : 2]);
  if (e != cudaSuccess) return e;
  const size_t rows = static_cast<size_t>(T) * H;
  uint8_t* base = static_cast<uint8_t*>(scratch);
  int* ctl = reinterpret_cast<int*>(base);
  CUtensorMap* dmaps = reinterpret_cast<CUtensorMap*>(base + 256);
  const size_t padded = al256((static_cast<size_t>(T) + 127) / 128 * 128 * H * sizeof(float));
  float* nl = reinterpret_cast<float*>(base + al256(kPackedHead));
  float* nd = reinterpret_cast<float*>(base + al256(kPackedHead) + padded);
  float* acc = reinterpret_cast<float*>(base + al256(kPackedHead) + 2 * padded);
  SetupMaps maps = {};
  CUtensorMap mdq;
  const long long dims[4] = {HD, H, T, 1};
  const long long strides[3] = {stride_or(H, dout.head) * 2, stride_or(T, dout.tok) * 2, 16};
  const int box[4] = {64, 1, 128, 1};
  if (!map_heads(&maps.m[0], q, T, H) || !map_heads(&maps.m[1], k, T, Hkv) || !map_heads(&maps.m[2], v, T, Hkv) ||
      !make_map_4d(&maps.m[3], dout.ptr, dims, strides, box) ||
      !make_map(&mdq, acc, 4, HD, T, H, HD, 1ll * T * HD, 32, 32))
    return cudaErrorInvalidValue;
  const PlanView P = plan_view(const_cast<void*>(plan), T);
  const int row_blocks = static_cast<int>((rows + 8 * kRowsPerWarp - 1) / (8 * kRowsPerWarp));
  PackedArgs pa = {};
  pa.meta = P.meta;
  pa.lo = P.lo;
  pa.fwd = P.fwd;
  const int items = (T + 127) / 128 * H;   // a block each, as in the forward
  e = launch_chained(dot, items, 608, PD_SMEM, s, maps, dmaps, ctl, lse, nl, nd, acc, H, Hkv, T,
                     scale * 1.4426950408889634f, err, wait_cycles, pa);
  if (e != cudaSuccess) return e;
  pa.hi = P.hi;
  pa.bwd = P.bwd;
  pa.ctl = ctl;
  pa.bad = ctl + kCtlBad;
  pa.maps = dmaps;
  pa.o_tok = dk.tok;
  pa.o_head = dk.head;
  pa.dv_tok = dv.tok;
  pa.dv_head = dv.head;
  const long long units = 1ll * ((T + 127) / 128) * Hkv;
  const int grid = static_cast<int>(std::min<long long>(units, device_sm_count()));
  e = launch_chained(kern, grid, 512, TB_SMEM, s, maps.m[0], maps.m[1], maps.m[2], maps.m[3], mdq, nl, nd,
                     static_cast<bf16*>(const_cast<void*>(dk.ptr)), static_cast<bf16*>(const_cast<void*>(dv.ptr)), H,
                     Hkv, Hkv, T, 1 << 30, scale, 0, ctl + kCtlSched, err, wait_cycles, nullptr, nullptr, nullptr, pa);
  if (e != cudaSuccess) return e;
  FinishArgs fin = {};
  fin.q = head_rows(q);
  fin.k = head_rows(k);
  fin.v = head_rows(v);
  fin.dout = head_rows(dout);
  fin.dq = head_rows(dq);
  fin.dk = head_rows(dk);
  fin.dv = head_rows(dv);
  fin.ctl = ctl;
  fin.lo = P.lo;
  fin.hi = P.hi;
  fin.nl = nl;
  fin.nd = nd;
  fin.H = H;
  fin.Hkv = Hkv;
  fin.T = T;
  fin.clear = clear;
  fin.scale = scale;
  e = launch_chained(attention_packed_dq_kernel, row_blocks, 256, 0, s, acc,
                     static_cast<bf16*>(const_cast<void*>(dq.ptr)), dq.tok, dq.head, ctl, fin);
  if (e != cudaSuccess) return e;
  return launch_chained(attention_packed_repair_kernel, std::min(row_blocks, 2 * device_sm_count()), 256, 0, s, fin);
}

}  // namespace gpt
