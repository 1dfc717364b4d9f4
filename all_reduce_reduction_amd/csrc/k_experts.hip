// k_experts.hip -- tokens to their experts' rows and back (gfx950).
//
// A slot is a (token, j) pair with an expert in chosen[token][j]; the expert of
// slot i = token * topk + j is e_i, none where it is outside [0, experts).
//   place_i = the number of slots i' with (e_i', i') < (e_i, i), none counted
// dispatch copies row `token` to rows[place_i]; combine adds rows[place_i] up
// per token with the slots' weights; combine's gradient writes
// weight_i * dy[token] to drows[place_i] and the product of both rows to
// dweight_i.  All three go by token, so that a token's own row is read or
// written once.
//
// A wave takes a token (or a part of its row): lane j holds what slot j has, and
// the slots that are not empty are taken one after the other from their ballot,
// so that a row's address and weight lie in scalar registers and no empty slot
// costs a load.
//
// Bound by memory, and by how it takes rows in no order: 16,384 tokens and 8 slots,
// combine of 8 KiB rows 197 us (1,209 MB at 6.1 TB/s; a copy of as many bytes 182),
// its gradient 406 (weights 185, rows 221; 2,283 MB, 343), dispatch of 4 KiB rows 127
// (places 10.5, rows and scales 115; 624 MB, 94; without the scales 120 in all).  What
// bounds dispatch is how memory takes writes: 537 MB written from its start to its end
// take 80 us when every wave writes 1 KiB once, 97 when it writes eight times in a row,
// 101 when it writes to the rows of a token's eight experts, and 119 with the token's
// row read before (a kernel that does nothing else).  Taking the slots in their rows'
// order instead, each row's token read again from the caches, was slower (146 us).
// Rows of an odd number of 16-bit elements lie across lines that two waves write: 16,384
// tokens, 8 slots of 2,049 and 2,048 bf16 columns dispatch 154 us, 120; combine 130, 97;
// its gradient 278, 210.
#include <algorithm>

#include "launch.h"
#include "layer.h"
#include "row_device.h"

namespace simar {
namespace {

// 16 bytes at any address
typedef uint32_t u32x4_at1 __attribute__((ext_vector_type(4), aligned(1)));
__device__ __forceinline__ u32x4 ld_any(const void* p, int64_t byte) {
  return __builtin_nontemporal_load((__attribute__((address_space(1))) const u32x4_at1*)((const char*)p + byte));
}
template <bool STREAM>
__device__ __forceinline__ void st_any(void* p, int64_t byte, u32x4 v) {
  __attribute__((address_space(1))) u32x4_at1* q = (__attribute__((address_space(1))) u32x4_at1*)((char*)p + byte);
  if constexpr (STREAM) __builtin_nontemporal_store((u32x4_at1)v, q);
  else *q = (u32x4_at1)v;
}

__device__ __forceinline__ int32_t lane_value(int32_t v, int lane) { return __builtin_amdgcn_readlane(v, lane); }
__device__ __forceinline__ float lane_value(float v, int lane) {
  return __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int32_t, v), lane));
}
__device__ __forceinline__ int32_t wave_uniform(int32_t v) { return __builtin_amdgcn_readfirstlane(v); }
// the lowest set bit, taken out
__device__ __forceinline__ int take(uint64_t& mask) {
  const int j = __builtin_ctzll(mask);
  mask &= mask - 1;
  return j;
}

// ---- places ---------------------------------------------------------------------
// a slot's expert, `experts` where it has none
__device__ __forceinline__ uint32_t expert_at(const DispatchArgs& a, int32_t chosen) {
  return (uint32_t)chosen < (uint32_t)a.experts ? (uint32_t)chosen : (uint32_t)a.experts;
}
__device__ __forceinline__ uint32_t expert_of(const DispatchArgs& a, int64_t slot) {
  return expert_at(a, a.chosen[slot]);
}
// the sum of v over the lanes below, and this one
__device__ __forceinline__ uint32_t scan_lanes(uint32_t v, int lane) {
  for (int d = 1; d < 64; d *= 2) {
    const uint32_t o = __shfl_up(v, d);
    if (lane >= d) v += o;
  }
  return v;
}

// Part `part` of a row of `bytes` bytes, 64 vectors of 16 bytes, to the rows of a
// token's slots (lane j: slot j's, < 0 for none).  Of short rows, which have but
// one part, the wave's four quarters take a slot each.
constexpr int kPartBytes = 1024, kShort = 256;
template <bool STREAM>
__device__ __forceinline__ void copy_row(const char* from, int64_t bytes, char* to, int64_t pitch, int32_t place, int part) {
  const int lane = threadIdx.x & 63;
  uint64_t mask = __ballot(place >= 0);
  if (bytes <= kShort) {
    const int l = lane & 15;
    const bool whole = bytes >= 16;
    const int64_t b = whole ? (l * 16 + 16 <= bytes ? l * 16 : bytes - 16) : l;
    u32x4 v = {0, 0, 0, 0};
    if (whole) {
      if (l * 16 < bytes) v = ld_any(from, b);
    } else if (l < bytes) {
      v[0] = (uint8_t)from[b];
    }
    for (int j0 = 0; mask >> j0; j0 += 4) {
      const int32_t row = __shfl(place, j0 + (lane >> 4));
      if (row >= 0 && whole && l * 16 < bytes) st_any<STREAM>(to, row * pitch + b, v);
      if (row >= 0 && !whole && l < bytes) to[row * pitch + b] = (char)v[0];
    }
    return;
  }
  const int64_t b = (int64_t)part * kPartBytes + lane * 16;
  // (the last 16 bytes end with the row; lanes past it keep running, as the others
  // read their places)
  const int64_t at = b + 16 <= bytes ? b : bytes - 16;
  const u32x4 v = ld_any(from, at);
  while (mask) {
    char* row = to + (int64_t)lane_value(place, take(mask)) * pitch;
    asm volatile("" : "+s"(row));
    if (b < bytes) st_any<STREAM>(row, at, v);
  }
}
// a part of a token's row, and of its scales
template <bool STREAM>
__device__ __forceinline__ void move_token(const DispatchArgs& a, int64_t token, int32_t place, int part) {
  if ((int64_t)part * kPartBytes < a.row_bytes)
    copy_row<STREAM>((const char*)a.x + token * a.x_pitch, a.row_bytes, (char*)a.rows, a.rows_pitch, place, part);
  if (a.scales && (int64_t)part * kPartBytes < a.scale_bytes)
    copy_row<STREAM>((const char*)a.scales + token * a.scale_bytes, a.scale_bytes, (char*)a.row_scales, a.scale_bytes, place, part);
}

// Adds a wave's slots to the counts of their experts (e < experts).  Those of the
// first lane's expert go together: a choice that many slots share would otherwise
// add to one word one by one (8,192 slots of one expert 8.7 us, 20.8).
__device__ __forceinline__ void count_slots(uint32_t* counts, uint32_t e, int experts) {
  const uint32_t common = (uint32_t)wave_uniform((int32_t)e);
  const uint64_t same = __ballot(e == common);
  const int lane = threadIdx.x & 63;
  if (e < (uint32_t)experts && (e != common || lane == __builtin_ctzll(same)))
    atomicAdd(&counts[e], e == common ? (uint32_t)__popcll(same) : 1u);
}

// ---- few slots: one launch --------------------------------------------------------
// A token's workgroup counts its slots' predecessors among all slots, each wave
// a quarter of them: a slot before another one has a smaller key e * slots + i.
// Then each wave moves a part of the row.  The last workgroup does the offsets.
__global__ void __launch_bounds__(256) k_dispatch_few(DispatchArgs a, int groups) {
  constexpr int N = 8;
  __shared__ uint32_t wave_s[4], share_s[4][SIM_ROUTE_MAX_TOPK];
  __shared__ uint32_t count_s[SIM_ROUTE_MAX_EXPERTS];
  const int tid = threadIdx.x, lane = tid & 63, wave = wave_uniform(tid >> 6);
  const uint32_t slots = (uint32_t)(a.tokens * a.topk), none = (uint32_t)a.experts;
  if (blockIdx.x == gridDim.x - 1) {
    for (int e = tid; e < a.experts; e += 256) count_s[e] = 0;
    __syncthreads();
    for (uint32_t b0 = 0; b0 < slots; b0 += 256 * N) {
      int32_t c[N];
#pragma unroll
      for (int i = 0; i < N; i++) c[i] = b0 + i * 256 + tid < slots ? a.chosen[b0 + i * 256 + tid] : -1;
#pragma unroll
      for (int i = 0; i < N; i++) count_slots(count_s, (uint32_t)c[i], a.experts);
    }
    __syncthreads();
    // four experts per thread
    uint32_t mine[4], all = 0;
#pragma unroll
    for (int k = 0; k < 4; k++) {
      mine[k] = all;
      all += tid * 4 + k < a.experts ? count_s[tid * 4 + k] : 0;
    }
    uint32_t before = scan_lanes(all, lane);
    if (lane == 63) wave_s[wave] = before;
    __syncthreads();
    before -= all;
    for (int w = 0; w < wave; w++) before += wave_s[w];
#pragma unroll
    for (int k = 0; k < 4; k++)
      if (tid * 4 + k < a.experts) a.offsets[tid * 4 + k] = (int32_t)(before + mine[k]);
    if (tid == 255) a.offsets[a.experts] = (int32_t)(before + all);
    return;
  }
  const int64_t token = blockIdx.x / groups;
  const int part = (int)(blockIdx.x - token * groups) * 4 + wave;
  const uint32_t own = lane < a.topk ? expert_of(a, token * a.topk + lane) : none;
  const uint32_t own_key = own * slots + (uint32_t)(token * a.topk) + lane;
  for (int j0 = 0; j0 < a.topk; j0 += N) {
    uint32_t key[N], n[N];
#pragma unroll
    for (int j = 0; j < N; j++) {
      key[j] = (uint32_t)lane_value((int32_t)own_key, j0 + j < a.topk ? j0 + j : j0);
      n[j] = 0;
    }
    for (uint32_t i0 = wave * 64; i0 < slots; i0 += 256 * N) {
      int32_t c[N];
#pragma unroll
      for (int i = 0; i < N; i++) {
        c[i] = -1;
        if (i0 + i * 256 + lane < slots) c[i] = a.chosen[i0 + i * 256 + lane];
      }
#pragma unroll
      for (int i = 0; i < N; i++) {
        if (i0 + i * 256 >= slots) break;
        const uint32_t k = (uint32_t)c[i] < none ? (uint32_t)c[i] * slots + i0 + i * 256 + lane : 0xffffffffu;
#pragma unroll
        for (int j = 0; j < N; j++) n[j] += (uint32_t)__popcll(__ballot(k < key[j]));
      }
    }
    uint32_t mine = 0;
#pragma unroll
    for (int j = 0; j < N; j++) mine = lane == j0 + j ? n[j] : mine;
    if (lane >= j0 && lane < j0 + N) share_s[wave][lane] = mine;
  }
  __syncthreads();
  int32_t place = -1;
  if (own < none) place = (int32_t)((share_s[0][lane] + share_s[1][lane]) + (share_s[2][lane] + share_s[3][lane]));
  if (part == 0 && lane < a.topk) a.place[token * a.topk + lane] = place;
  move_token<true>(a, token, place, part);
}

// ---- more slots: counts, places, rows -----------------------------------------------
__global__ void __launch_bounds__(256) k_dispatch_count(DispatchArgs a) {
  constexpr int N = 4;
  __shared__ uint32_t count_s[SIM_ROUTE_MAX_EXPERTS];
  const int64_t slots = a.tokens * a.topk, lo = blockIdx.x * a.chunk;
  const int64_t hi = lo + a.chunk < slots ? lo + a.chunk : slots;
  for (int e = threadIdx.x; e < a.experts; e += 256) count_s[e] = 0;
  __syncthreads();
  for (int64_t b0 = lo; b0 < hi; b0 += 256 * N) {
    const int64_t i0 = b0 + threadIdx.x;
    int32_t c[N];
#pragma unroll
    for (int i = 0; i < N; i++) {
      c[i] = -1;
      if (i0 + i * 256 < hi) c[i] = a.chosen[i0 + i * 256];
    }
#pragma unroll
    for (int i = 0; i < N; i++) count_slots(count_s, (uint32_t)c[i], a.experts);
  }
  __syncthreads();
  for (int e = threadIdx.x; e < a.experts; e += 256) a.counts[(int64_t)blockIdx.x * a.experts + e] = count_s[e];
}

// A chunk's places.  The experts' starts and the slots before the chunk come from
// all chunks' counts, or with SELF from all slots themselves; within the chunk each
// wave takes a run of slots, 64 at a time, and a slot's place is its wave's next one
// of its expert plus the number of lanes below it with the same expert.
constexpr int kPlaceThreads = 1024, kPlaceWaves = kPlaceThreads / 64;
template <bool SELF>
__global__ void __launch_bounds__(kPlaceThreads) k_dispatch_place(DispatchArgs a) {
  constexpr int N = 16;  // loads of a thread under way
  __shared__ uint32_t next_s[kPlaceWaves * SIM_ROUTE_MAX_EXPERTS];
  __shared__ uint32_t total_s[SIM_ROUTE_MAX_EXPERTS], before_s[SIM_ROUTE_MAX_EXPERTS];
  __shared__ uint32_t wave_s[kPlaceWaves];
  const int tid = threadIdx.x, lane = tid & 63, wave = wave_uniform(tid >> 6);
  const int experts = a.experts, mine = (int)blockIdx.x;
  const int64_t slots = a.tokens * a.topk, run = a.chunk / kPlaceWaves;
  const int64_t lo = mine * a.chunk + wave * run;
  const int64_t hi = lo + run < slots ? lo + run : slots;
  // the wave's first 64 slots, asked for first
  const uint32_t first_e = lo + lane < hi ? expert_of(a, lo + lane) : (uint32_t)experts;
  uint32_t* next = next_s + wave * experts;
  for (int e = tid; e < experts; e += kPlaceThreads) total_s[e] = before_s[e] = 0;
  for (int e = lane; e < experts; e += 64) next[e] = 0;
  __syncthreads();
  if constexpr (SELF) {
    const int start = (int)(mine * a.chunk);
    for (int w0 = wave * 64; w0 < slots; w0 += kPlaceThreads * N) {
      const int i0 = w0 + lane;
      int32_t c[N];
#pragma unroll
      for (int i = 0; i < N; i++) {
        c[i] = -1;
        if (i0 + i * kPlaceThreads < slots) c[i] = a.chosen[i0 + i * kPlaceThreads];
      }
      // (a wave's 64 slots lie on one side of the chunk's start)
#pragma unroll
      for (int i = 0; i < N; i++)
        count_slots(w0 + i * kPlaceThreads < start ? before_s : total_s, (uint32_t)c[i], experts);
    }
    // (what the counts of all chunks hold in total_s is made of both)
    __syncthreads();
    if (tid < experts) total_s[tid] += before_s[tid];
  } else {
    // as many chunks at once as there are threads for their experts
    const int at_once = kPlaceThreads / experts;
    const int from = tid / experts;
    if (from < at_once) {
      const int e = tid - from * experts;
      uint32_t total = 0, before = 0;
      for (int c0 = from; c0 < a.chunks; c0 += at_once * N) {
        uint32_t n[N];
#pragma unroll
        for (int i = 0; i < N; i++) {
          n[i] = 0;
          if (c0 + i * at_once < a.chunks) n[i] = a.counts[(int64_t)(c0 + i * at_once) * experts + e];
        }
#pragma unroll
        for (int i = 0; i < N; i++) {
          total += n[i];
          before += c0 + i * at_once < mine ? n[i] : 0;
        }
      }
      atomicAdd(&total_s[e], total);
      atomicAdd(&before_s[e], before);
    }
  }
  // this chunk's slots, counted per wave
  count_slots(next, first_e, experts);
  for (int64_t i0 = lo + 64; i0 < hi; i0 += 64)
    count_slots(next, i0 + lane < hi ? expert_of(a, i0 + lane) : (uint32_t)experts, experts);
  __syncthreads();
  // the experts' starts: a scan of the totals, one expert per thread
  const uint32_t total = tid < experts ? total_s[tid] : 0;
  uint32_t start = scan_lanes(total, lane);
  if (lane == 63) wave_s[wave] = start;
  __syncthreads();
  start -= total;
  for (int w = 0; w < wave; w++) start += wave_s[w];
  if (mine == 0) {
    if (tid < experts) a.offsets[tid] = (int32_t)start;
    if (tid == experts - 1) a.offsets[experts] = (int32_t)(start + total);
  }
  if (tid < experts) {
    uint32_t at = start + before_s[tid];
    for (int w = 0; w < kPlaceWaves; w++) {
      const uint32_t n = next_s[w * experts + tid];
      next_s[w * experts + tid] = at;
      at += n;
    }
  }
  __syncthreads();
  for (int64_t i0 = lo; i0 < hi; i0 += 64) {
    const int64_t i = i0 + lane;
    const uint32_t e = i0 == lo ? first_e : i < hi ? expert_of(a, i) : (uint32_t)experts;
    // the lanes with the same expert
    uint64_t same = ~0ull;
    for (int b = 0; (experts >> b) != 0; b++) {
      const uint64_t set = __ballot((e >> b) & 1);
      same &= (e >> b) & 1 ? set : ~set;
    }
    const bool has = e < (uint32_t)experts;
    const uint32_t first = has ? next[e] : 0;
    const uint32_t below = __popcll(same & ((1ull << lane) - 1));
    wave_fence();
    if (has && below == 0) next[e] = first + __popcll(same);
    wave_fence();
    if (i < hi) a.place[i] = has ? (int32_t)(first + below) : -1;
  }
}

// Six waves per SIMD: with eight the writes of more rows interleave in memory
// (8,192 tokens of 16 KiB to 8 places 232 us, 247).
template <bool STREAM>
__global__ void __launch_bounds__(256) __attribute__((amdgpu_waves_per_eu(6, 6))) k_dispatch_rows(DispatchArgs a, int parts) {
  const int lane = threadIdx.x & 63;
  const int64_t step = (int64_t)gridDim.x * 4;
  for (int64_t unit = (int64_t)blockIdx.x * 4 + wave_uniform(threadIdx.x >> 6); unit < a.tokens * parts; unit += step) {
    const int64_t token = unit / parts;
    const int32_t place = lane < a.topk ? a.place[token * a.topk + lane] : -1;
    move_token<STREAM>(a, token, place, (int)(unit - token * parts));
  }
}

// ---- back to the tokens -------------------------------------------------------------
// a token's slots: lane j holds slot j's row and weight
struct TokenSlots {
  int32_t place;
  float weight;
  uint64_t mask;  // the slots that are not empty
  __device__ __forceinline__ TokenSlots(const int32_t* places, const float* weights, int64_t token, int topk, int64_t nrows) {
    const int lane = threadIdx.x & 63;
    place = -1;
    weight = 1.0f;
    if (lane < topk) {
      place = places[token * topk + lane];
      if (weights) weight = weights[token * topk + lane];
    }
    mask = __ballot(place >= 0 && place < nrows);
  }
};

// the next N slots' vectors
template <int DT, int N, class P>
__device__ __forceinline__ void add_rows(const CombineArgs& a, const TokenSlots& s, uint64_t& m, const P& p,
                                         float (&acc)[epv<DT>()]) {
  constexpr int V = epv<DT>();
  u32x4 v[N];
  float w[N];
#pragma unroll
  for (int i = 0; i < N; i++) {
    const int j = take(m);
    w[i] = lane_value(s.weight, j);
    v[i] = p.load((const char*)a.rows + (int64_t)lane_value(s.place, j) * a.rows_stride * Ty<DT>::E);
  }
#pragma unroll
  for (int i = 0; i < N; i++) {
    float f[V];
    unpack<DT>(v[i], f);
#pragma unroll
    for (int t = 0; t < V; t++) acc[t] = __builtin_fmaf(w[i], f[t], acc[t]);
  }
}
// A wave takes part of a token's columns, 64 vectors.  Where the rows are more than the
// caches hold and a wave has many loads under way, fewer WAVES per SIMD than eight are
// enough, and more only interleave more rows in memory (launch below).
template <int DT, int WAVES>
__global__ void __launch_bounds__(256) __attribute__((amdgpu_waves_per_eu(WAVES < 8 ? WAVES : 4, WAVES))) k_combine(CombineArgs a, int parts) {
  constexpr int V = epv<DT>();
  const int lane = threadIdx.x & 63;
  const int64_t step = (int64_t)gridDim.x * 4;
  for (int64_t unit = (int64_t)blockIdx.x * 4 + wave_uniform(threadIdx.x >> 6); unit < a.tokens * parts; unit += step) {
    const int64_t token = unit / parts;
    const TokenSlots s(a.place, a.weights, token, a.topk, a.nrows);
    const int n = __popcll(s.mask);
    const RowPart<DT, kEnd> p(((uint32_t)(unit - token * parts) * 64 + lane) * V, (uint32_t)a.cols);
    float acc[V];
#pragma unroll
    for (int t = 0; t < V; t++) acc[t] = 0.0f;
    uint64_t m = s.mask;
    for (int i = 8; i <= n; i += 8) add_rows<DT, 8>(a, s, m, p, acc);
    if (n & 4) add_rows<DT, 4>(a, s, m, p, acc);
    if (n & 2) add_rows<DT, 2>(a, s, m, p, acc);
    if (n & 1) add_rows<DT, 1>(a, s, m, p, acc);
    if (p.any()) p.store((char*)a.out + token * a.out_stride * Ty<DT>::E, acc);
  }
}

// Rows of up to 32 vectors: L lanes take a token.
template <int DT, int L, bool TINY>
__global__ void __launch_bounds__(256) k_combine_short(CombineArgs a) {
  constexpr int V = epv<DT>(), N = 8;
  const int l = threadIdx.x % L;
  const RowPart<DT, TINY ? kTiny : kEnd> p(l * V, (uint32_t)a.cols);
  for (int64_t token = (int64_t)blockIdx.x * (256 / L) + threadIdx.x / L; token < a.tokens;
       token += (int64_t)gridDim.x * (256 / L)) {
    float acc[V];
#pragma unroll
    for (int t = 0; t < V; t++) acc[t] = 0.0f;
    for (int j0 = 0; j0 < a.topk; j0 += N) {
      int32_t at[N];
      float w[N];
#pragma unroll
      for (int j = 0; j < N; j++) {
        const int64_t i = token * a.topk + (j0 + j < a.topk ? j0 + j : j0);
        at[j] = a.place[i];
        w[j] = a.weights ? a.weights[i] : 1.0f;
      }
      u32x4 v[N];
#pragma unroll
      for (int j = 0; j < N; j++) {
        const bool has = j0 + j < a.topk && at[j] >= 0 && at[j] < a.nrows && p.any();
        w[j] = has ? w[j] : 0.0f;  // (an empty slot's weight may be anything)
        v[j] = u32x4{0, 0, 0, 0};
        if (has) v[j] = p.load((const char*)a.rows + (int64_t)at[j] * a.rows_stride * Ty<DT>::E);
      }
#pragma unroll
      for (int j = 0; j < N; j++) {
        float f[V];
        unpack<DT>(v[j], f);
#pragma unroll
        for (int t = 0; t < V; t++) acc[t] = __builtin_fmaf(w[j], f[t], acc[t]);
      }
    }
    if (p.any()) p.store((char*)a.out + token * a.out_stride * Ty<DT>::E, acc);
  }
}

// ---- the gradient ---------------------------------------------------------------------
// The next N slots: a token's dy against their rows, 64 vectors of columns at a
// time, by W waves in turn.
template <int DT, int N, int W, Where K, bool STREAM>
__device__ __forceinline__ void grad_rows(const CombineGradArgs& a, const TokenSlots& s, uint64_t& m, int64_t token,
                                          float (*dot_s)[8]) {
  constexpr int V = epv<DT>();
  const int lane = threadIdx.x & 63, wave = W > 1 ? wave_uniform(threadIdx.x >> 6) : 0;
  const uint32_t cols = (uint32_t)a.cols;
  const char* dy = (const char*)a.dy + token * a.dy_stride * Ty<DT>::E;
  const char* from[N];
  char* to[N];
  float w[N], dot[N];
  int slot[N];
#pragma unroll
  for (int i = 0; i < N; i++) {
    slot[i] = take(m);
    const int64_t at = lane_value(s.place, slot[i]);
    w[i] = lane_value(s.weight, slot[i]);
    from[i] = (const char*)a.rows + at * a.rows_stride * Ty<DT>::E;
    to[i] = (char*)a.drows + at * a.drows_stride * Ty<DT>::E;
    dot[i] = 0.0f;
  }
  for (uint32_t c = wave * 64 * V; c < cols; c += W * 64 * V) {
    const RowPart<DT, K> p(c + lane * V, cols);
    const u32x4 dv = p.template load<STREAM>(dy);
    u32x4 v[N];
    if (a.dweights) {
#pragma unroll
      for (int i = 0; i < N; i++) v[i] = p.template load<STREAM>(from[i]);
    }
    float d[V];
    unpack<DT>(dv, d);
    p.mask(d);
    if (a.dweights) {
#pragma unroll
      for (int i = 0; i < N; i++) {
        float f[V];
        unpack<DT>(v[i], f);
        // (a masked column's row may hold anything)
#pragma unroll
        for (int t = 0; t < V; t++) dot[i] = p.own(t) ? __builtin_fmaf(d[t], f[t], dot[i]) : dot[i];
      }
    }
    if (a.drows && p.any()) {
#pragma unroll
      for (int i = 0; i < N; i++) {
        float f[V];
#pragma unroll
        for (int t = 0; t < V; t++) f[t] = w[i] * d[t];
        p.store(to[i], f);
      }
    }
  }
  if (!a.dweights) return;
#pragma unroll
  for (int i = 0; i < N; i++) dot[i] = wave_sum(dot[i]);
  if constexpr (W > 1) {
    __syncthreads();
    if (lane == 0) {
#pragma unroll
      for (int i = 0; i < N; i++) dot_s[wave][i] = dot[i];
    }
    __syncthreads();
    if (wave != 0) return;
#pragma unroll
    for (int i = 0; i < N; i++) {
      dot[i] = 0.0f;
#pragma unroll
      for (int q = 0; q < W; q++) dot[i] += dot_s[q][i];
    }
  }
  if (lane == 0) {
#pragma unroll
    for (int i = 0; i < N; i++) a.dweights[token * a.topk + slot[i]] = dot[i];
  }
}
// (Rows of up to 64 vectors have a whole wave too, most of whose lanes idle in short ones:
// 16,384 tokens, 16 slots of 64 bf16 columns 36 us, bound by instructions; 10 for the
// bytes.)
// Where there are too few tokens to fill the GPU with a wave each, up to eight waves
// share one (333 tokens x 2,263 fp32, 6 slots: 9.2 us, four 9.9, sixteen 11.3), but
// no more than its row has 64 vectors for: the others would only wait (bf16, 1,116
// tokens x 737, 14 slots, two waves 12.7 us, eight 22.6; 1,500 x 2,048, 4 slots,
// four waves 11.2, eight 12.8).
template <int DT, int W, Where K, bool STREAM>
__global__ void __launch_bounds__(W > 1 ? 64 * W : 256) k_combine_grad(CombineGradArgs a) {
  __shared__ float dot_s[W][8];
  const int lane = threadIdx.x & 63, wave = wave_uniform(threadIdx.x >> 6);
  for (int64_t token = W > 1 ? (int64_t)blockIdx.x : (int64_t)blockIdx.x * 4 + wave; token < a.tokens;
       token += W > 1 ? (int64_t)gridDim.x : (int64_t)gridDim.x * 4) {
    const TokenSlots s(a.place, a.weights, token, a.topk, a.nrows);
    const int n = __popcll(s.mask);
    if (a.dweights && (W == 1 || wave == 0) && lane < a.topk && !(s.mask >> lane & 1)) a.dweights[token * a.topk + lane] = 0.0f;
    uint64_t m = s.mask;
    for (int i = 8; i <= n; i += 8) grad_rows<DT, 8, W, K, STREAM>(a, s, m, token, dot_s);
    if (n & 4) grad_rows<DT, 4, W, K, STREAM>(a, s, m, token, dot_s);
    if (n & 2) grad_rows<DT, 2, W, K, STREAM>(a, s, m, token, dot_s);
    if (n & 1) grad_rows<DT, 1, W, K, STREAM>(a, s, m, token, dot_s);
  }
}

// The rows' gradient by itself: a wave takes part of a token's columns, as where
// rows are only moved.
template <int DT>
__global__ void __launch_bounds__(256) __attribute__((amdgpu_waves_per_eu(6, 6))) k_combine_grad_rows(CombineGradArgs a, int parts) {
  constexpr int V = epv<DT>();
  const int lane = threadIdx.x & 63;
  const int64_t step = (int64_t)gridDim.x * 4;
  for (int64_t unit = (int64_t)blockIdx.x * 4 + wave_uniform(threadIdx.x >> 6); unit < a.tokens * parts; unit += step) {
    const int64_t token = unit / parts;
    const TokenSlots s(a.place, a.weights, token, a.topk, a.nrows);
    const RowPart<DT, kEnd> p(((uint32_t)(unit - token * parts) * 64 + lane) * V, (uint32_t)a.cols);
    float d[V];
    unpack<DT>(p.load((const char*)a.dy + token * a.dy_stride * Ty<DT>::E), d);
    for (uint64_t m = s.mask; m;) {
      const int j = take(m);
      const float w = lane_value(s.weight, j);
      char* row = (char*)a.drows + (int64_t)lane_value(s.place, j) * a.drows_stride * Ty<DT>::E;
      asm volatile("" : "+s"(row));
      float f[V];
#pragma unroll
      for (int t = 0; t < V; t++) f[t] = w * d[t];
      if (p.any()) p.template store<false>(row, f);
    }
  }
}

// ---- launches ---------------------------------------------------------------------------
unsigned grid_of(int64_t units, int per) {
  return (unsigned)std::min<int64_t>((units + per - 1) / per, (int64_t)1 << 22);
}
template <int DT>
hipError_t combine(const CombineArgs& a, hipStream_t s) {
  constexpr int V = epv<DT>();
  const int64_t nv = (a.cols + V - 1) / V;
  if (a.cols < V) return launch<k_combine_short<DT, 8, true>>(dim3(grid_of(a.tokens, 32)), dim3(256), s, a);
  if (nv <= 8) return launch<k_combine_short<DT, 8, false>>(dim3(grid_of(a.tokens, 32)), dim3(256), s, a);
  if (nv <= 16) return launch<k_combine_short<DT, 16, false>>(dim3(grid_of(a.tokens, 16)), dim3(256), s, a);
  if (nv <= 32) return launch<k_combine_short<DT, 32, false>>(dim3(grid_of(a.tokens, 8)), dim3(256), s, a);
  const int parts = (int)((nv + 63) / 64);
  const dim3 grid(grid_of(a.tokens * parts, 4));
  // By slots (three, four, eight waves, us; bf16): 16,384 tokens of 8 KiB, 2 slots 85, 74,
  // 65; 4 slots 116, 110, 110; 6 slots 160, 151, 160; 8 slots 196, 200, 213; 16 slots 380,
  // 397, 399.  By bytes, in what all slots would read: 4,096 of 16 KiB, 6 slots, 384 MiB
  // 80.7, 76.0, 77.5; 6,000 of 8 KiB, 6 slots, 281 MiB 60.0, 57.8, 56.7; 8 slots, 375 MiB
  // 72.9, 72.7, 74.1; 8,192 of 4 KiB, 8 slots, 256 MiB 49.8, 48.1, 49.5; 4,096 of 4 KiB, 8
  // slots, 128 MiB 25.9, 24.5, 23.6; 1,000 of 8 KiB, 8 slots 12.6, 11.6, 10.7.  How many
  // slots are empty is not known here: with every other one of 8 x 16,384 of 8 KiB three
  // waves lose (125, 112, 112).
  const bool many = (double)a.tokens * a.topk * (double)a.cols * Ty<DT>::E > (double)(320 << 20);
  if (many && a.topk >= 8) return launch<k_combine<DT, 3>>(grid, dim3(256), s, a, parts);
  if (many && a.topk > 4) return launch<k_combine<DT, 4>>(grid, dim3(256), s, a, parts);
  return launch<k_combine<DT, 8>>(grid, dim3(256), s, a, parts);
}
// W waves share a token
template <int DT, int W>
hipError_t combine_grad_shared(const CombineGradArgs& a, bool stream, hipStream_t s) {
  const dim3 grid(grid_of(a.tokens, 1));
  return stream ? launch<k_combine_grad<DT, W, kEnd, true>>(grid, dim3(64 * W), s, a)
                : launch<k_combine_grad<DT, W, kEnd, false>>(grid, dim3(64 * W), s, a);
}
template <int DT>
hipError_t combine_grad(const CombineGradArgs& a, hipStream_t s) {
  constexpr int V = epv<DT>();
  const int64_t nv = (a.cols + V - 1) / V;
  if (a.cols < V) return launch<k_combine_grad<DT, 1, kTiny, false>>(dim3(grid_of(a.tokens, 4)), dim3(256), s, a);
  // Where the rows are more than the caches hold, memory that reads and then writes
  // is faster than memory that does both at once, by more than dy's second reading
  // costs (16,384 tokens of 8 KiB, 8 slots: 406 us, 452 in one launch; 4,096
  // tokens 110, 123; 2,048 tokens 59.5, 55.8; 16,384 tokens, 2 slots 139, 135).
  if (a.drows && a.dweights && a.topk >= 4 && nv > 64 &&
      (double)a.tokens * a.topk * (double)a.cols * Ty<DT>::E > (double)(192 << 20)) {
    CombineGradArgs b = a;
    b.drows = nullptr;
    const hipError_t e = combine_grad<DT>(b, s);
    if (e != hipSuccess) return e;
    const int parts = (int)((nv + 63) / 64);
    return launch<k_combine_grad_rows<DT>>(dim3(grid_of(a.tokens * parts, 4)), dim3(256), s, a, parts);
  }
  // Rows that start inside a line share it: streaming loads would fetch it twice
  // (333 tokens x 2,263 fp32, 6 slots 9.9 us, 13.0 streaming; 4,096 x 5,120 bf16,
  // 4 slots 78, 74 streaming).
  const uintptr_t starts = (uintptr_t)a.dy | (uintptr_t)a.rows | (uintptr_t)(a.dy_stride * Ty<DT>::E) |
                           (uintptr_t)(a.rows_stride * Ty<DT>::E);
  const bool stream = starts % 64 == 0;
  if (nv <= 64 || a.tokens >= 16 * library_cus()) {
    const dim3 grid(grid_of(a.tokens, 4));
    return stream ? launch<k_combine_grad<DT, 1, kEnd, true>>(grid, dim3(256), s, a)
                  : launch<k_combine_grad<DT, 1, kEnd, false>>(grid, dim3(256), s, a);
  }
  if (nv <= 128) return combine_grad_shared<DT, 2>(a, stream, s);
  if (nv <= 256) return combine_grad_shared<DT, 4>(a, stream, s);
  return combine_grad_shared<DT, 8>(a, stream, s);
}

}  // namespace

// Few slots go in one launch while a workgroup reads few of them, once for every 8
// of its token's slots, and all workgroups together not too many; else in two.
// A workgroup's own: 512 tokens of 4 KiB, 8 slots, 4,096 read: 9.2 us, 11.2 in two
// launches; 128, 16 slots, 4,096: 8.7, 9.9; 400, 10 slots, 8,000: 13.1, 10.7; 128, 32
// slots, 16,384: 23.1, 12.0.  All of them: 1,024 of 8 KiB, 2 slots, 4.2 M: 10.8, 11.7;
// 1,600 of 4 KiB, 2 slots, 5.1 M: 11.6, 11.6; 4,096, one slot, 16.8 M: 23.9, 14.7.
constexpr int64_t kFewChunk = 1024, kFewOwn = 6 << 10, kFewReads = 9 << 19;
hipError_t launch_dispatch(const DispatchArgs& args, hipStream_t s) {
  DispatchArgs a = args;
  // a wave for each part of a token's row
  const int64_t longest = std::max(std::max(a.row_bytes, a.scales ? a.scale_bytes : 0), (int64_t)1);
  const int parts = (int)((longest + kPartBytes - 1) / kPartBytes);
  if (a.chunks == 0) {
    const int64_t slots = a.tokens * a.topk, groups = (parts + 3) / 4, own = slots * ((a.topk + 7) / 8);
    if (own <= kFewOwn && a.tokens * groups * own <= kFewReads)
      return launch<k_dispatch_few>(dim3((unsigned)(a.tokens * groups + 1)), dim3(256), s, a, (int)groups);
    a.chunk = kFewChunk;
    a.chunks = (int)((slots + kFewChunk - 1) / kFewChunk);
  }
  hipError_t e;
  if (a.counts) {
    e = launch<k_dispatch_count>(dim3(a.chunks), dim3(256), s, a);
    if (e != hipSuccess) return e;
    e = launch<k_dispatch_place<false>>(dim3(a.chunks), dim3(kPlaceThreads), s, a);
  } else {
    e = launch<k_dispatch_place<true>>(dim3(a.chunks), dim3(kPlaceThreads), s, a);
  }
  if (e != hipSuccess || (a.row_bytes == 0 && !a.scales)) return e;
  // Streaming stores, but not where what is written is far more than the caches
  // hold: 16,384 tokens of 4 KiB to 8 places 130 us, 134 streaming; 1,000 of 4 KiB
  // to 6 places 14.5, 13.1 streaming.
  const int64_t written = a.tokens * a.topk * (a.row_bytes + a.scale_bytes);
  const dim3 grid(grid_of(a.tokens * parts, 4));
  return written > (int64_t)128 << 20 ? launch<k_dispatch_rows<false>>(grid, dim3(256), s, a, parts)
                                      : launch<k_dispatch_rows<true>>(grid, dim3(256), s, a, parts);
}

hipError_t launch_combine(const CombineArgs& a, int dtype, hipStream_t s) {
  return dtype == SIM_FP32   ? combine<SIM_FP32>(a, s)
         : dtype == SIM_FP16 ? combine<SIM_FP16>(a, s)
                             : combine<SIM_BF16>(a, s);
}
hipError_t launch_combine_grad(const CombineGradArgs& a, int dtype, hipStream_t s) {
  return dtype == SIM_FP32   ? combine_grad<SIM_FP32>(a, s)
         : dtype == SIM_FP16 ? combine_grad<SIM_FP16>(a, s)
                             : combine_grad<SIM_BF16>(a, s);
}

}  // namespace simar
