// k_route.hip -- softmax gate with per-expert statistics, and the gradient of
// its balance loss and combine weights (gfx950).
//
// Forward, row x: m = max x, Z = sum exp(x - m), p = exp(x - m) / Z; the topk
// largest logits by value, ties to the lowest index, taken from the logits
// themselves, so that the choice does not depend on any rounding.  Counts are
// integers; probability sums are taken per lane over its rows, then over the
// lanes and waves of a workgroup, then over the workgroups, in that order, so
// they do not depend on timing.
//
// Gradient: with g_e = coef f_e / N,
//   dx_e = p_e (g_e + u_e - sum_j p_j (g_j + u_j)),  u = dweights at chosen e,
// for raw weights; for normalised ones w = p / (their sum over the chosen),
//   dx_e = p_e (g_e - sum_j p_j g_j) + [e chosen] w_e (dw_e - sum_i w_i dw_i).
//
// Layout: L lanes take a row and a wave 64 / L rows; a lane holds N logits as
// 16-byte vectors, vector j of lane l being the row's vector j L + l, so that
// a group's loads cover whole lines.  With many rows per wave the cross-lane
// steps of one row (log2 L of them) serve 64 / L rows at once, and they run
// over DPP while L is at most 16.
#include "device_sync.h"
#include "launch.h"
#include "loss.h"
#include "loss_device.h"

namespace simar {
namespace {

constexpr int kWaves = kBlock / 64;

template <int DT, int L, int N>
struct Gate {
  static constexpr int V = epv<DT>(), NV = N / V, kRows = 64 / L, kAll = L * N;
  u32x4 v[NV];

  static __device__ __forceinline__ int col(int j, int l) { return (j * L + l) * V; }

  __device__ __forceinline__ void load(const void* row, int experts, int l) {
    if (experts == kAll) {
#pragma unroll
      for (int j = 0; j < NV; j++) v[j] = ld_row<DT>(row, col(j, l));
    } else if (experts >= V) {
      // the row's last vector where a lane's own would reach past the end, its
      // elements moved to their places and the rest set to -inf: no branch, so
      // all loads are in flight together
#pragma unroll
      for (int j = 0; j < NV; j++) v[j] = Tail<DT>(col(j, l), experts).load(row);
#pragma unroll
      for (int j = 0; j < NV; j++) move_down(v[j], Tail<DT>(col(j, l), experts).skip);
    } else {
#pragma unroll
      for (int j = 0; j < NV; j++) v[j] = ld_guarded<DT>(row, col(j, l), experts);
    }
  }
  // element i becomes element i + skip, -inf past the last
  static __device__ __forceinline__ void move_down(u32x4& w, int skip) {
    constexpr uint32_t n = neg_inf_bits<DT>();
    const int words = skip * Ty<DT>::E / 4;
    u32x4 r = w;
#pragma unroll
    for (int i = 0; i < 4; i++) {
      uint32_t x = n;
#pragma unroll
      for (int k = i; k < 4; k++) x = words == k - i ? w[k] : x;
      r[i] = x;
    }
    if constexpr (Ty<DT>::E == 2) {
      // an odd number of halves: one more half down
      const u32x4 q = r;
#pragma unroll
      for (int i = 0; i < 4; i++) {
        const uint32_t above = i < 3 ? q[i + 1] : n;
        r[i] = skip & 1 ? q[i] >> 16 | above << 16 : q[i];
      }
    }
    w = r;
  }
  __device__ __forceinline__ void blank() {
    constexpr uint32_t n = neg_inf_bits<DT>();
#pragma unroll
    for (int j = 0; j < NV; j++) v[j] = u32x4{n, n, n, n};
  }
  // What is made of the vectors after this is made after it: values kept from
  // one use to the next would take more registers than making them again.
  __device__ __forceinline__ void renew() {
#pragma unroll
    for (int j = 0; j < NV; j++) asm volatile("" : "+v"(v[j]));
  }
  __device__ __forceinline__ void logits(float (&x)[N]) const {
#pragma unroll
    for (int j = 0; j < NV; j++) {
      float f[V];
      unpack<DT>(v[j], f);
#pragma unroll
      for (int t = 0; t < V; t++) x[j * V + t] = f[t];
    }
  }
};

// A float's bits as an unsigned integer that grows with its value (a 16-bit
// type's in the upper half); both zeros get the same one.  NaN with the sign
// clear lies above +inf, with the sign set below -inf.
template <int DT>
__device__ __forceinline__ uint32_t ordered(uint32_t bits) {
  if constexpr (DT == SIM_FP32) {
    // -0 + 0 is +0, and every other value stays
    const uint32_t b = __builtin_bit_cast(uint32_t, __builtin_bit_cast(float, bits) + 0.0f);
    return b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u);
  }
  return ((bits ^ ((bits >> 15) * 0x7fffu | 0x8000u)) + (bits >> 15)) << 16;
}
template <int DT> constexpr uint32_t ordered_inf() {
  return DT == SIM_FP32 ? 0xff800000u : DT == SIM_FP16 ? 0xfc000000u : 0xff800000u;
}
template <int DT> constexpr uint32_t ordered_neg_inf() {
  return DT == SIM_FP32 ? 0x007fffffu : DT == SIM_FP16 ? 0x04000000u : 0x00800000u;
}
__device__ __forceinline__ float from_ordered32(uint32_t key) {
  return __builtin_bit_cast(float, key & 0x80000000u ? key ^ 0x80000000u : ~key);
}
template <int DT>
__device__ __forceinline__ float from_ordered16(uint32_t key) {
  const uint32_t h = key >> 16;
  return widen_bits<DT>(h & 0x8000u ? h ^ 0x8000u : 0x10000u - h);
}

// ---- the eight largest of a group -----------------------------------------------
__device__ __forceinline__ void order2(uint32_t& a, uint32_t& b) {
  const uint32_t hi = max(a, b);
  b = min(a, b);
  a = hi;
}
// any eight keys, largest first (19 exchanges)
__device__ __forceinline__ void sort8(uint32_t (&k)[8]) {
  order2(k[0], k[1]); order2(k[2], k[3]); order2(k[4], k[5]); order2(k[6], k[7]);
  order2(k[0], k[2]); order2(k[1], k[3]); order2(k[4], k[6]); order2(k[5], k[7]);
  order2(k[1], k[2]); order2(k[5], k[6]);
  order2(k[0], k[4]); order2(k[1], k[5]); order2(k[2], k[6]); order2(k[3], k[7]);
  order2(k[2], k[4]); order2(k[3], k[5]);
  order2(k[1], k[2]); order2(k[3], k[4]); order2(k[5], k[6]);
}
// a bitonic sequence of eight, largest first
__device__ __forceinline__ void sort8_bitonic(uint32_t (&k)[8]) {
  order2(k[0], k[4]); order2(k[1], k[5]); order2(k[2], k[6]); order2(k[3], k[7]);
  order2(k[0], k[2]); order2(k[1], k[3]); order2(k[4], k[6]); order2(k[5], k[7]);
  order2(k[0], k[1]); order2(k[2], k[3]); order2(k[4], k[5]); order2(k[6], k[7]);
}
// the value of the lane that differs in one bit, 16 or 32 (a captured flag in
// place of the call goes through LDS: 1,715 rows x 512 fp32 21.7 us, 10.3 so)
template <int BIT>
__device__ __forceinline__ uint32_t from_other(uint32_t k) {
  const auto pick = [](uint32_t a, uint32_t b) { return __lane_id() & BIT ? a : b; };
  if constexpr (BIT == 16) return across_rows(k, pick);
  else return across_halves(k, pick);
}
// the eight largest of two sorted eights: the larger of each element and its
// counterpart from the other end
template <class F>
__device__ __forceinline__ void merge8(uint32_t (&k)[8], F other) {
  uint32_t o[8];
#pragma unroll
  for (int i = 0; i < 8; i++) o[i] = other(k[7 - i], 7 - i);
#pragma unroll
  for (int i = 0; i < 8; i++) k[i] = max(k[i], o[i]);
  sort8_bitonic(k);
}

// Keys that put the value above the distance of the index from the last one,
// so that a larger key is a larger logit or, among equal ones, a lower index.
// 16-bit values fit whole; fp32 values lose their log2(L N) lowest bits, and
// the caller checks that what is left tells the chosen ones apart.  Only keys
// below `limit` take part (0: all do).
template <int DT, int L, int N>
__device__ __forceinline__ void top8(const Gate<DT, L, N>& g, int l, uint32_t limit, uint32_t (&top)[8]) {
  typedef Gate<DT, L, N> G;
  constexpr int V = G::V;
  const uint32_t mine = (uint32_t)((L - 1 - l) * V);
#pragma unroll
  for (int b = 0; b < N / 8; b++) {
    uint32_t k[8];
#pragma unroll
    for (int i = 0; i < 8; i++) {
      const int at = b * 8 + i, j = at / V, t = at % V;
      const uint32_t low = (uint32_t)((G::NV - 1 - j) * L * V + (V - 1 - t));
      if constexpr (Ty<DT>::E == 4) {
        k[i] = (ordered<DT>(g.v[j][t]) & ~(uint32_t)(G::kAll - 1)) | low;
      } else {
        // both halves of a word are ordered at once
        const uint32_t w = g.v[j][t / 2], s = w & 0x80008000u;
        const uint32_t o = (w ^ ((s - (s >> 15)) | 0x80008000u)) + (s >> 15);
        k[i] = (t & 1 ? o & 0xffff0000u : o << 16) | low;
      }
    }
    if (limit != 0) {
#pragma unroll
      for (int i = 0; i < 8; i++) k[i] = (k[i] | mine) < limit ? k[i] : 0;
    }
    sort8(k);
    if (b == 0) {
#pragma unroll
      for (int i = 0; i < 8; i++) top[i] = k[i];
    } else {
      merge8(top, [&](uint32_t, int i) { return k[i]; });
    }
    // one eight after the other: interleaved, their keys would take the
    // registers of two more waves
    __builtin_amdgcn_sched_barrier(0);
  }
#pragma unroll
  for (int i = 0; i < 8; i++) top[i] |= mine;
  merge8(top, [](uint32_t k, int) { return dpp<kDppPair>(k); });
  merge8(top, [](uint32_t k, int) { return dpp<kDppQuad>(k); });
  if constexpr (L >= 8) merge8(top, [](uint32_t k, int) { return dpp<kDppHalfRow>(k); });
  if constexpr (L >= 16) merge8(top, [](uint32_t k, int) { return dpp<kDppRow>(k); });
  // every lane keeps its own row's (half's) eight and takes the other's
  if constexpr (L >= 32) merge8(top, [](uint32_t k, int) { return from_other<16>(k); });
  if constexpr (L >= 64) merge8(top, [](uint32_t k, int) { return from_other<32>(k); });
}

// The topk largest one after the other, exactly, for any topk: lane l gets
// slots l, l + L, ...  NaN and -inf are never taken.
template <int DT, int L, int N, int S>
__device__ __forceinline__ void top_in_turn(const Gate<DT, L, N>& g, int l, int topk, int (&mine)[S]) {
  typedef Gate<DT, L, N> G;
  constexpr int V = G::V;
  uint32_t k[N];
#pragma unroll
  for (int i = 0; i < N; i++) {
    const int j = i / V, t = i % V;
    if constexpr (Ty<DT>::E == 4) k[i] = ordered<DT>(g.v[j][t]);
    else k[i] = ordered<DT>((t & 1) ? g.v[j][t / 2] >> 16 : g.v[j][t / 2] & 0xffffu);
    if (k[i] <= ordered_neg_inf<DT>() || k[i] > ordered_inf<DT>()) k[i] = 0;
  }
#pragma unroll
  for (int s = 0; s < S; s++) mine[s] = -1;
  for (int r = 0; r < topk; r++) {
    uint32_t best = 0;
#pragma unroll
    for (int i = 0; i < N; i++) best = max(best, k[i]);
    best = group_reduce<L>(best, [](uint32_t a, uint32_t b) { return max(a, b); });
    // columns relative to the lane's first, which are constants
    uint32_t at = 0x40000000u;
#pragma unroll
    for (int i = N - 1; i >= 0; i--)
      if (k[i] == best) at = G::col(i / V, 0) + i % V;
    at = group_reduce<L>(at + l * V, [](uint32_t a, uint32_t b) { return min(a, b); });
    const uint32_t own = at - l * V;
#pragma unroll
    for (int i = 0; i < N; i++)
      if (own == (uint32_t)(G::col(i / V, 0) + i % V)) k[i] = 0;
#pragma unroll
    for (int s = 0; s < S; s++)
      if (r == l + L * s && best != 0) mine[s] = (int)at;
    if (!__any(best != 0)) break;
  }
}

// ---- the workgroups' counts and sums ------------------------------------------------
// A word that another workgroup of this launch reads goes to device scope.
__device__ __forceinline__ void put(uint32_t* p, uint32_t v) {
  __hip_atomic_store(p, v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

// The workgroup that arrives last adds up what all of them have written, in
// the workgroups' order.  No workgroup waits for another one.  From its arrival
// on nobody touches the counter, so it reports that first.  This takes a launch
// less than k_route_sum (1,003 rows x 60 fp32, top 4: 7.2 us against
// 9.7).
__device__ __forceinline__ void sum_in_last(const RouteArgs& a, uint32_t* word_s) {
  constexpr int kFlight = 32;  // loads of a thread under way (16: 9.3 us where 32 take 8.5)
  wait_stores();
  __syncthreads();
  if (threadIdx.x == 0) *word_s = __hip_atomic_fetch_add(a.turn.word, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  __syncthreads();
  if (*word_s != a.turn.base + (uint32_t)a.workgroups - 1) return;
  if (threadIdx.x == 0) __hip_atomic_store(a.turn.done, a.turn.call, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_SYSTEM);
  const int all = 2 * a.experts + 1;
  for (int e = threadIdx.x; e < all; e += kBlock) {
    uint32_t n = 0;
    float s = 0.0f;
    for (int w0 = 0; w0 < a.workgroups; w0 += kFlight) {
      uint32_t v[kFlight];
      const uint32_t* from = a.partial + (int64_t)w0 * all + e;
#pragma unroll
      for (int i = 0; i < kFlight; i++) {
        v[i] = 0;
        if (w0 + i < a.workgroups)
          v[i] = __hip_atomic_load(from + (int64_t)i * all, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      }
#pragma unroll
      for (int i = 0; i < kFlight; i++) {
        n += v[i];
        s += __builtin_bit_cast(float, v[i]);
      }
    }
    if (e <= a.experts) a.counts[e] = (int32_t)n;
    else a.sums[e - a.experts - 1] = s;
  }
}

// ---- forward ------------------------------------------------------------------------
// Up to eight chosen experts come from one pass of the exchange networks; each
// further eight from another one below the last key.  MANY: topk > 8.
//
// The vector units bound it: 98 instructions per row of 256 (43 of them the
// networks, 20 the softmax, 18 the keys), 10.5 us of the kernel's 15 at 65,536
// rows, against 6 us for the bytes; with the sums of the workgroups 19 us a call
// (bf16, top 8; one wave per row with eight rounds of a wave-wide maximum: 370).
// 16-bit rows keep 32 logits per lane, so that 8 rows share a wave's cross-lane
// steps (16 per lane: 22 us); fp32 rows 16, as their keys and values take twice
// the registers (32 per lane: 36 us against 32; 28.6 since).
template <int DT, int L, int N, bool MANY>
__global__ void __launch_bounds__(kBlock, N == 32 ? 3 : 4) k_route(RouteArgs a) {
  typedef Gate<DT, L, N> G;
  constexpr int TAKE = L < 8 ? 8 / L : 1;  // slots of a round that a lane may get
  constexpr int S = MANY ? (SIM_ROUTE_MAX_TOPK + L - 1) / L : TAKE;
  __shared__ uint32_t count_s[G::kAll + 1];
  __shared__ float sum_s[kWaves * G::kRows][G::kAll];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, l = lane & (L - 1);
  for (int e = tid; e <= G::kAll; e += kBlock) count_s[e] = 0;
  __syncthreads();
  float sums[N];
#pragma unroll
  for (int i = 0; i < N; i++) sums[i] = 0.0f;
  uint32_t rows = 0;
  const int64_t step = (int64_t)a.workgroups * kWaves * G::kRows;
  for (int64_t first = ((int64_t)blockIdx.x * kWaves + wave) * G::kRows; first < a.tokens; first += step) {
    const bool here = first + lane / L < a.tokens;
    const int64_t row = here ? first + lane / L : first;
    const char* x = (const char*)a.x + row * a.stride * Ty<DT>::E;
    G g;
    g.load(x, a.experts, l);
    const bool kept = here && (!a.keep || a.keep[row]);
    if (!kept) g.blank();

    // the chosen experts
    constexpr uint32_t m = Ty<DT>::E == 4 ? ~(uint32_t)(G::kAll - 1) : 0xffff0000u;  // a key's value bits
    int mine[S];
    float at[S];
#pragma unroll
    for (int s = 0; s < S; s++) {
      mine[s] = -1;
      at[s] = 0.0f;
    }
    float top_logit = kNegInf;
    uint32_t last = 0;
    bool odd_key = false;
    for (int done = 0; done < a.topk; done += 8) {
      uint32_t top[8];
      if (MANY) g.renew();
      top8(g, l, last, top);
      if constexpr (Ty<DT>::E == 4) {
        // exact if the topk keys differ above the index, no other key shares
        // the last one's value bits, and all of them are of finite logits
        if (done == 0) odd_key = (top[0] & m) >= (ordered_inf<DT>() & m);
        else odd_key = odd_key || (top[0] & m) == (last & m);
        last = top[0];
#pragma unroll
        for (int i = 1; i < 8; i++) {
          if (done + i < a.topk) {
            odd_key = odd_key || (top[i] & m) == (top[i - 1] & m);
            last = top[i];
          }
        }
      } else {
        if (done == 0) {
          odd_key = (top[0] & m) > ordered_inf<DT>();  // a NaN
          top_logit = from_ordered16<DT>(top[0]);
        }
        last = top[7];
      }
      // slot done + i goes to lane (done + i) mod L
      const int i0 = MANY ? (l - done) & (L - 1) : l;
#pragma unroll
      for (int u = 0; u < TAKE; u++) {
        const int at_i = i0 + u * L;
        uint32_t k = top[0];
#pragma unroll
        for (int i = 1; i < 8; i++) k = at_i == i ? top[i] : k;
        const bool ok = at_i < 8 && done + at_i < a.topk && (k & m) > (ordered_neg_inf<DT>() & m);
#pragma unroll
        for (int s = 0; s < S; s++) {
          if (MANY ? ok && (done + at_i) / L == s : s == u) {
            mine[s] = ok ? G::kAll - 1 - (int)(k & (uint32_t)(G::kAll - 1)) : -1;
            if constexpr (Ty<DT>::E == 2) at[s] = from_ordered16<DT>(k);
          }
        }
      }
      if (!MANY) break;
    }
    g.renew();
    if constexpr (Ty<DT>::E == 4) {
      odd_key = odd_key || (last & m) <= (ordered_neg_inf<DT>() & m);
      // (values compare like their keys, and as values they need not be made
      // into keys again; a NaN counts as none here and as odd above)
      const float least = from_ordered32(last & m);
      float n = 0.0f;
#pragma unroll
      for (int i = 0; i < N; i++) {
        const uint32_t bits = g.v[i / G::V][i % G::V];
        n += __builtin_bit_cast(float, bits) >= least ? 1.0f : 0.0f;
      }
      odd_key = odd_key || group_sum<L>(n) != (float)a.topk;
    }
    const bool in_turn = __any(odd_key && kept);
    if (in_turn) {
      g.renew();
      top_in_turn<DT, L, N, S>(g, l, a.topk, mine);
    }
    g.renew();

    // the softmax
    float f[N];
    g.logits(f);
    if (Ty<DT>::E == 4 || in_turn) {
      top_logit = kNegInf;
#pragma unroll
      for (int i = 0; i < N; i++) top_logit = fmaxf(top_logit, f[i]);
      top_logit = group_max<L>(top_logit);
    }
    const Against base = against(top_logit, kLog2e);
    float z = 0.0f;
#pragma unroll
    for (int i = 0; i < N; i++) {
      f[i] = exp_against(f[i], base);
      z += f[i];
    }
    z = group_sum<L>(z);
    // Only a row of -inf alone sums to 0: the largest logit's own term is 2^-56
    // or more, and a NaN makes the sum one.  (The keys do not tell an empty row:
    // NaN with the sign set lies below -inf.)
    const bool live = z != 0.0f;
    const float inv = live ? 1.0f / z : 0.0f;
#pragma unroll
    for (int i = 0; i < N; i++) sums[i] = __builtin_fmaf(f[i], inv, sums[i]);
    if (live && l == 0) rows++;

    // the weights of the chosen
    float w[S], total = 0.0f;
#pragma unroll
    for (int s = 0; s < S; s++) {
      if (Ty<DT>::E == 4 || in_turn) at[s] = mine[s] >= 0 ? load_elem<DT>(x, mine[s]) : 0.0f;
      w[s] = mine[s] >= 0 ? exp_against(at[s], base) * inv : 0.0f;
      total += w[s];
    }
    if (a.normalize) {
      const float sum = group_sum<L>(total);
#pragma unroll
      for (int s = 0; s < S; s++)
        if (mine[s] >= 0) w[s] = inv != inv ? inv : w[s] / sum;
    }
#pragma unroll
    for (int s = 0; s < S; s++) {
      const int slot = l + L * s;
      if (here && slot < a.topk) {
        a.chosen[row * a.topk + slot] = mine[s];
        a.weights[row * a.topk + slot] = w[s];
      }
      if (mine[s] >= 0) atomicAdd(&count_s[mine[s]], 1u);
    }
  }
  if (rows) atomicAdd(&count_s[G::kAll], rows);
#pragma unroll
  for (int i = 0; i < N; i++) sum_s[wave * G::kRows + lane / L][G::col(i / G::V, l) + i % G::V] = sums[i];
  __syncthreads();
  uint32_t* part = a.partial + (int64_t)blockIdx.x * (2 * a.experts + 1);
  for (int e = tid; e <= a.experts; e += kBlock) {
    float s = 0.0f;
    if (e < a.experts) {
#pragma unroll
      for (int w = 0; w < kWaves * G::kRows; w++) s += sum_s[w][e];
    }
    const uint32_t n = count_s[e < a.experts ? e : G::kAll];
    if (a.workgroups == 1) {
      a.counts[e] = (int32_t)n;
      if (e < a.experts) a.sums[e] = s;
    } else {
      put(part + e, n);
      if (e < a.experts) put(part + a.experts + 1 + e, __builtin_bit_cast(uint32_t, s));
    }
  }
  if (a.turn.word) sum_in_last(a, &count_s[0]);
}

// The workgroups' counts and sums, kSumCols of them per workgroup: 1024
// threads as kSumRows runs of rows by kSumCols columns, then the runs in order.
// All of a thread's loads are in flight together: 3 to 4 us, a launch's own
// time, at any size (one thread per column: 40 us for 251 workgroups).
constexpr int kSumCols = 16, kSumRows = 64;
__global__ void __launch_bounds__(kSumCols* kSumRows) k_route_sum(RouteArgs a) {
  __shared__ uint32_t n_s[kSumRows][kSumCols];
  __shared__ float s_s[kSumRows][kSumCols];
  const int all = 2 * a.experts + 1, c = threadIdx.x % kSumCols, r = threadIdx.x / kSumCols;
  const int e = blockIdx.x * kSumCols + c;
  const int span = (a.workgroups + kSumRows - 1) / kSumRows;  // at most 16
  const int end = min(a.workgroups, (r + 1) * span);
  uint32_t n = 0;
  float s = 0.0f;
  if (e < all) {
#pragma unroll 8
    for (int w = r * span; w < end; w++) {
      const uint32_t v = a.partial[(int64_t)w * all + e];
      n += v;
      s += __builtin_bit_cast(float, v);
    }
  }
  n_s[r][c] = n;
  s_s[r][c] = s;
  __syncthreads();
  if (r != 0 || e >= all) return;
  for (int i = 1; i < kSumRows; i++) {
    n += n_s[i][c];
    s += s_s[i][c];
  }
  if (e <= a.experts) a.counts[e] = (int32_t)n;
  else a.sums[e - a.experts - 1] = s;
}

// ---- gradient -------------------------------------------------------------------------
// A row's slots are added to its columns through LDS: the lanes that hold
// slots put their terms at the chosen columns of the group's row of zeros,
// all lanes read their own columns, and the slots' lanes put the zeros back.
// A wave only ever touches its own rows there, in program order.
//
// At 65,536 rows x 256 bf16 the vector units take 8.3 us (78 instructions per
// row), the bytes 11: 15.4 us a call.  16 logits per lane here, as six waves per
// SIMD then hide the row's loads (32 per lane, three waves: 18.5).
template <int DT, int L, int N>
__global__ void __launch_bounds__(kBlock) k_route_grad(RouteGradArgs a) {
  typedef Gate<DT, L, N> G;
  constexpr int V = G::V, S = (SIM_ROUTE_MAX_TOPK + L - 1) / L;
  __shared__ float g_s[G::kAll];
  __shared__ float add_s[kWaves * G::kRows][G::kAll];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, l = lane & (L - 1);
  float* add = add_s[wave * G::kRows + lane / L];
  const float n = a.counts ? (float)a.counts[a.experts] : 0.0f;
  const float unit = n > 0.0f ? a.coef * ((float)a.experts / (float)a.topk) / n / n : 0.0f;
  for (int e = tid; e < G::kAll; e += kBlock)
    g_s[e] = n > 0.0f && e < a.experts ? unit * (float)a.counts[e] : 0.0f;
#pragma unroll
  for (int i = 0; i < N; i++) add[l + L * i] = 0.0f;
  __syncthreads();
  if (blockIdx.x == 0 && wave == 0 && a.loss) {
    float loss = 0.0f;
    if (n > 0.0f)
      for (int e = lane; e < a.experts; e += 64) loss += g_s[e] * a.sums[e];
    loss = wave_sum(loss);
    if (lane == 0) *a.loss = loss;
  }
  const int64_t step = (int64_t)gridDim.x * kWaves * G::kRows;
  for (int64_t first = ((int64_t)blockIdx.x * kWaves + wave) * G::kRows; first < a.tokens; first += step) {
    const bool here = first + lane / L < a.tokens;
    const int64_t row = here ? first + lane / L : first;
    const char* x = (const char*)a.x + row * a.stride * Ty<DT>::E;
    char* dx = (char*)a.dx + row * a.dstride * Ty<DT>::E;
    G g;
    g.load(x, a.experts, l);
    int mine[S];
    float dw[S], at[S];
#pragma unroll
    for (int s = 0; s < S; s++) {
      const int slot = l + L * s;
      mine[s] = -1;
      dw[s] = at[s] = 0.0f;
      if (a.dweights && here && slot < a.topk) {
        mine[s] = a.chosen[row * a.topk + slot];
        if (mine[s] < 0 || mine[s] >= a.experts) mine[s] = -1;
        if (mine[s] >= 0) {
          dw[s] = a.dweights[row * a.topk + slot];
          at[s] = load_elem<DT>(x, mine[s]);
        }
      }
    }
    const bool kept = here && (!a.keep || a.keep[row]);
    if (!kept) g.blank();
    float f[N];
    g.logits(f);
    float top = kNegInf;
#pragma unroll
    for (int i = 0; i < N; i++) top = fmaxf(top, f[i]);
    top = group_max<L>(top);
    // a row of NaN and -inf alone is not empty: its sum is NaN
    const Against base = against(top, kLog2e);
    float z = 0.0f;
#pragma unroll
    for (int i = 0; i < N; i++) {
      f[i] = exp_against(f[i], base);
      z += f[i];
    }
    z = group_sum<L>(z);
    const bool live = z != 0.0f;
    const float inv = live ? 1.0f / z : 0.0f;
    float dot = 0.0f;
#pragma unroll
    for (int i = 0; i < N; i++) {
      f[i] *= inv;
      dot = __builtin_fmaf(f[i], g_s[G::col(i / V, l) + i % V], dot);
    }
    float p[S], sum = 0.0f, mean = 0.0f;
#pragma unroll
    for (int s = 0; s < S; s++) {
      p[s] = mine[s] >= 0 && live ? exp_against(at[s], base) * inv : 0.0f;
      sum += p[s];
      mean = __builtin_fmaf(p[s], dw[s], mean);
    }
    if (a.normalize) {
      sum = group_sum<L>(sum);
      mean = group_sum<L>(mean) / sum;
#pragma unroll
      for (int s = 0; s < S; s++)
        if (mine[s] >= 0 && live) add[mine[s]] = p[s] / sum * (dw[s] - mean);
    } else {
      dot += mean;
#pragma unroll
      for (int s = 0; s < S; s++)
        if (mine[s] >= 0 && live) add[mine[s]] = p[s] * dw[s];
    }
    dot = group_sum<L>(dot);
    // (an empty row's p are 0, but its slots' dweights and coef may be anything)
    const bool some_empty = __any(!live);
    wave_fence();
#pragma unroll
    for (int j = 0; j < G::NV; j++) {
      float d[V];
#pragma unroll
      for (int t = 0; t < V; t++) {
        const int e = G::col(j, l) + t;
        d[t] = __builtin_fmaf(f[j * V + t], g_s[e] - dot, add[e]);
      }
      if (some_empty) {
#pragma unroll
        for (int t = 0; t < V; t++) d[t] = live ? d[t] : 0.0f;
      }
      if (here) {
        if (a.experts == G::kAll) st_row<DT>(dx, G::col(j, l), pack_rounded<DT>(d));
        else st_guarded<DT>(dx, G::col(j, l), a.experts, d);
      }
    }
    wave_fence();
#pragma unroll
    for (int s = 0; s < S; s++)
      if (mine[s] >= 0) add[mine[s]] = 0.0f;
  }
}

// ---- launches -----------------------------------------------------------------------
// Workgroups that share the rows evenly, at most `most` of them.
int64_t even_workgroups(int64_t tokens, int per, int64_t most) {
  const int64_t n = (tokens + per - 1) / per, turns = (n + most - 1) / most;
  return n < 1 ? 1 : (n + turns - 1) / turns;
}

template <int DT, bool MANY>
hipError_t route_layout(const RouteArgs& a, hipStream_t s) {
  constexpr int N = Ty<DT>::E == 2 ? 32 : 16;
  const dim3 grid(a.workgroups), block(kBlock);
  if (a.experts <= 32) return launch<k_route<DT, 4, 8, MANY>>(grid, block, s, a);
  if (a.experts <= 64) return launch<k_route<DT, 8, 8, MANY>>(grid, block, s, a);
  if (a.experts <= 128) return launch<k_route<DT, 8, 16, MANY>>(grid, block, s, a);
  if (a.experts <= 256) return launch<k_route<DT, 256 / N, N, MANY>>(grid, block, s, a);
  if (a.experts <= 512) return launch<k_route<DT, 512 / N, N, MANY>>(grid, block, s, a);
  return launch<k_route<DT, 1024 / N, N, MANY>>(grid, block, s, a);
}
template <int DT>
hipError_t route_dtype(const RouteArgs& a, hipStream_t s) {
  return a.topk <= 8 ? route_layout<DT, false>(a, s) : route_layout<DT, true>(a, s);
}
template <int DT>
hipError_t grad_dtype(const RouteGradArgs& a, hipStream_t s) {
  const int rows = a.experts <= 32 ? 16 : a.experts <= 128 ? 8 : a.experts <= 256 ? 4 : a.experts <= 512 ? 2 : 1;
  const dim3 grid((unsigned)even_workgroups(a.tokens, kWaves * rows, 4 * (int64_t)library_cus())), block(kBlock);
  if (a.experts <= 32) return launch<k_route_grad<DT, 4, 8>>(grid, block, s, a);
  if (a.experts <= 64) return launch<k_route_grad<DT, 8, 8>>(grid, block, s, a);
  if (a.experts <= 128) return launch<k_route_grad<DT, 8, 16>>(grid, block, s, a);
  if (a.experts <= 256) return launch<k_route_grad<DT, 16, 16>>(grid, block, s, a);
  if (a.experts <= 512) return launch<k_route_grad<DT, 32, 16>>(grid, block, s, a);
  return launch<k_route_grad<DT, 64, 16>>(grid, block, s, a);
}

}  // namespace

// At most two workgroups per compute unit where a lane holds 32 logits, whose
// registers let no more of them be under way (65,536 rows x 256 bf16: 19.2 us, with
// four 20.4); four otherwise (65,536 x 256 fp32 28.6, with two 32.3; x 128 bf16
// 14.7 and 15.1).
int route_workgroups(int64_t tokens, int experts, int dtype) {
  const int n = dtype == SIM_FP32 ? 16 : 32;
  const int rows = experts <= 32 ? 16 : experts <= 128 ? 8 : 64 * n / (experts <= 256 ? 256 : experts <= 512 ? 512 : 1024);
  const int64_t wg = even_workgroups(tokens, kWaves * rows, (n == 32 && experts > 128 ? 2 : 4) * (int64_t)library_cus());
  return (int)(wg < 3 ? 1 : wg);
}

// One compute unit reads few words at a time: the workgroups add up their own
// sums up to this many words (bf16, top 8: 1,024 rows x 256, 16,416 words, 8.5
// us against 9.7 with the second launch; 2,048 rows, 32,832 words, 11.0 against
// 9.8), and up to as many workgroups as k_route_sum takes in plain order, so
// that both give the same bits.
bool route_sums_itself(int workgroups, int experts) {
  return workgroups > 1 && workgroups <= kSumRows && workgroups * (2 * experts + 1) <= 24 << 10;
}

hipError_t launch_route(const RouteArgs& a, int dtype, hipStream_t s) {
  const hipError_t e = dtype == SIM_FP32   ? route_dtype<SIM_FP32>(a, s)
                       : dtype == SIM_FP16 ? route_dtype<SIM_FP16>(a, s)
                                           : route_dtype<SIM_BF16>(a, s);
  if (e != hipSuccess || a.workgroups == 1 || a.turn.word) return e;
  return launch<k_route_sum>(dim3((2 * a.experts + kSumCols) / kSumCols), dim3(kSumCols * kSumRows), s, a);
}
hipError_t launch_route_grad(const RouteGradArgs& a, int dtype, hipStream_t s) {
  if (dtype == SIM_FP32) return grad_dtype<SIM_FP32>(a, s);
  return dtype == SIM_FP16 ? grad_dtype<SIM_FP16>(a, s) : grad_dtype<SIM_BF16>(a, s);
}

}  // namespace simar
