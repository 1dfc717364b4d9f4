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
#include <algorithm>

#include "launch.h"
#include "layer.h"
#include "row_device.h"

namespace simar {
namespace {

// 16 bytes at any address
typedef uint32_t u32x4_at1 __attribute__((ext_vector_type(4), aligned(1)));
__device__ __forceinline__ u32x4 ld_any(const void* p, int64_t byte) {
  return *(__attribute__((address_space(1))) const u32x4_at1*)((const char*)p + byte);
}
__device__ __forceinline__ void st_any(void* p, int64_t byte, u32x4 v) {
  *(__attribute__((address_space(1))) u32x4_at1*)((char*)p + byte) = v;
}

// a slot's expert, `experts` where it has none
__device__ __forceinline__ uint32_t expert_of(const DispatchArgs& a, int64_t slot) {
  const uint32_t e = (uint32_t)a.chosen[slot];
  return e < (uint32_t)a.experts ? e : (uint32_t)a.experts;
}

// ---- rows -----------------------------------------------------------------------
// `bytes` bytes of one row to up to N others, by the threads l, l + lanes, ...
// of `lanes`; to[j] < 0: none.
template <int N>
__device__ __forceinline__ void copy_row(const char* from, int64_t bytes, char* to, int64_t pitch, const int64_t (&at)[N],
                                         int l, int lanes) {
  if (bytes >= 16) {
    for (int64_t b = (int64_t)l * 16; b < bytes; b += (int64_t)lanes * 16) {
      // (the last 16 bytes end with the row)
      const int64_t c = b + 16 <= bytes ? b : bytes - 16;
      const u32x4 v = ld_any(from, c);
#pragma unroll
      for (int j = 0; j < N; j++)
        if (at[j] >= 0) st_any(to, at[j] * pitch + c, v);
    }
  } else {
    for (int64_t b = l; b < bytes; b += lanes) {
      const char v = from[b];
#pragma unroll
      for (int j = 0; j < N; j++)
        if (at[j] >= 0) to[at[j] * pitch + b] = v;
    }
  }
}
// a token's row and scales to its slots' places
constexpr int kCopies = 8;
template <class PLACE>
__device__ __forceinline__ void move_token(const DispatchArgs& a, int64_t token, PLACE place, int l, int lanes) {
  for (int j0 = 0; j0 < a.topk; j0 += kCopies) {
    int64_t at[kCopies];
#pragma unroll
    for (int j = 0; j < kCopies; j++) at[j] = j0 + j < a.topk ? (int64_t)place(j0 + j) : -1;
    if (a.row_bytes) copy_row(a.x ? (const char*)a.x + token * a.x_pitch : nullptr, a.row_bytes, (char*)a.rows, a.rows_pitch, at, l, lanes);
    if (a.scales)
      copy_row((const char*)a.scales + token * a.scale_bytes, a.scale_bytes, (char*)a.row_scales, a.scale_bytes, at, l, lanes);
  }
}

// ---- few slots: one launch --------------------------------------------------------
// A workgroup per token counts its slots' predecessors among all slots: a slot
// before another one has a smaller key e * slots + i.  One workgroup more does
// the offsets.
__global__ void __launch_bounds__(256) k_dispatch_few(DispatchArgs a) {
  __shared__ uint32_t share_s[4][SIM_ROUTE_MAX_TOPK];
  __shared__ uint32_t count_s[SIM_ROUTE_MAX_EXPERTS];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const uint32_t slots = (uint32_t)(a.tokens * a.topk);
  if (blockIdx.x == a.tokens) {
    for (int e = tid; e < a.experts; e += 256) count_s[e] = 0;
    __syncthreads();
    for (uint32_t i = tid; i < slots; i += 256) {
      const uint32_t e = expert_of(a, i);
      if (e < (uint32_t)a.experts) atomicAdd(&count_s[e], 1u);
    }
    __syncthreads();
    // four experts per thread
    uint32_t mine[4], all = 0;
#pragma unroll
    for (int k = 0; k < 4; k++) {
      mine[k] = all;
      all += tid * 4 + k < a.experts ? count_s[tid * 4 + k] : 0;
    }
    uint32_t before = all;
    for (int d = 1; d < 64; d *= 2) {
      const uint32_t o = __shfl_up(before, d);
      if (lane >= d) before += o;
    }
    if (lane == 63) share_s[wave][0] = before;
    __syncthreads();
    before -= all;
    for (int w = 0; w < wave; w++) before += share_s[w][0];
#pragma unroll
    for (int k = 0; k < 4; k++)
      if (tid * 4 + k < a.experts) a.offsets[tid * 4 + k] = (int32_t)(before + mine[k]);
    if (tid == 255) a.offsets[a.experts] = (int32_t)(before + all);
    return;
  }
  const int64_t token = blockIdx.x;
  const uint32_t none = (uint32_t)a.experts;
  for (int j0 = 0; j0 < a.topk; j0 += kCopies) {
    uint32_t key[kCopies], n[kCopies];
#pragma unroll
    for (int j = 0; j < kCopies; j++) {
      const uint32_t i = (uint32_t)(token * a.topk) + j0 + j;
      key[j] = j0 + j < a.topk ? expert_of(a, i) * slots + i : 0;
      n[j] = 0;
    }
    for (uint32_t i0 = wave * 64; i0 < slots; i0 += 256) {
      const uint32_t i = i0 + lane;
      const uint32_t e = i < slots ? expert_of(a, i) : none;
      const uint32_t k = e < none ? e * slots + i : 0xffffffffu;
#pragma unroll
      for (int j = 0; j < kCopies; j++) n[j] += __popcll(__ballot(k < key[j]));
    }
    if (lane == 0) {
#pragma unroll
      for (int j = 0; j < kCopies; j++)
        if (j0 + j < a.topk) share_s[wave][j0 + j] = n[j];
    }
  }
  __syncthreads();
  const auto place = [&](int j) {
    const int32_t p = (int32_t)(share_s[0][j] + share_s[1][j] + share_s[2][j] + share_s[3][j]);
    return expert_of(a, token * a.topk + j) < none ? p : -1;
  };
  if (tid < a.topk) a.place[token * a.topk + tid] = place(tid);
  move_token(a, token, place, tid, 256);
}

// ---- many slots: counts, places, rows -----------------------------------------------
__global__ void __launch_bounds__(256) k_dispatch_count(DispatchArgs a) {
  __shared__ uint32_t count_s[SIM_ROUTE_MAX_EXPERTS];
  for (int e = threadIdx.x; e < a.experts; e += 256) count_s[e] = 0;
  __syncthreads();
  const int64_t slots = a.tokens * a.topk, lo = blockIdx.x * a.chunk;
  const int64_t hi = lo + a.chunk < slots ? lo + a.chunk : slots;
  for (int64_t i = lo + threadIdx.x; i < hi; i += 256) {
    const uint32_t e = expert_of(a, i);
    if (e < (uint32_t)a.experts) atomicAdd(&count_s[e], 1u);
  }
  __syncthreads();
  for (int e = threadIdx.x; e < a.experts; e += 256) a.counts[(int64_t)blockIdx.x * a.experts + e] = count_s[e];
}

// A chunk's places.  The experts' starts and the counts of the chunks before
// come from all chunks' counts; within the chunk each wave takes a run of slots,
// 64 at a time, and a slot's place is its wave's next one of its expert plus the
// number of lanes below it with the same expert.
constexpr int kPlaceThreads = 1024, kPlaceWaves = kPlaceThreads / 64;
__global__ void __launch_bounds__(kPlaceThreads) k_dispatch_place(DispatchArgs a) {
  __shared__ uint32_t next_s[kPlaceWaves][SIM_ROUTE_MAX_EXPERTS];
  __shared__ uint32_t total_s[SIM_ROUTE_MAX_EXPERTS], before_s[SIM_ROUTE_MAX_EXPERTS];
  __shared__ uint32_t wave_s[kPlaceWaves];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int experts = a.experts, mine = (int)blockIdx.x;
  for (int e = tid; e < experts; e += kPlaceThreads) total_s[e] = before_s[e] = 0;
  for (int i = tid; i < kPlaceWaves * SIM_ROUTE_MAX_EXPERTS; i += kPlaceThreads) (&next_s[0][0])[i] = 0;
  __syncthreads();
  // as many chunks at once as there are threads for their experts
  const int at_once = kPlaceThreads / experts;
  const int from = tid / experts;
  if (from < at_once) {
    const int e = tid - from * experts;
    uint32_t total = 0, before = 0;
    for (int c = from; c < a.chunks; c += at_once) {
      const uint32_t n = a.counts[(int64_t)c * experts + e];
      total += n;
      before += c < mine ? n : 0;
    }
    atomicAdd(&total_s[e], total);
    atomicAdd(&before_s[e], before);
  }
  // this chunk's slots, counted per wave
  const int64_t slots = a.tokens * a.topk, run = a.chunk / kPlaceWaves;
  const int64_t lo = mine * a.chunk + wave * run;
  const int64_t hi = lo + run < slots ? lo + run : slots;
  for (int64_t i = lo + lane; i < hi; i += 64) {
    const uint32_t e = expert_of(a, i);
    if (e < (uint32_t)experts) atomicAdd(&next_s[wave][e], 1u);
  }
  __syncthreads();
  // the experts' starts: a scan of the totals, one expert per thread
  const uint32_t total = tid < experts ? total_s[tid] : 0;
  uint32_t start = total;
  for (int d = 1; d < 64; d *= 2) {
    const uint32_t o = __shfl_up(start, d);
    if (lane >= d) start += o;
  }
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
      const uint32_t n = next_s[w][tid];
      next_s[w][tid] = at;
      at += n;
    }
  }
  __syncthreads();
  for (int64_t i0 = lo; i0 < hi; i0 += 64) {
    const int64_t i = i0 + lane;
    const uint32_t e = i < hi ? expert_of(a, i) : (uint32_t)experts;
    // the lanes with the same expert
    uint64_t same = ~0ull;
    for (int b = 0; (experts >> b) != 0; b++) {
      const uint64_t set = __ballot((e >> b) & 1);
      same &= (e >> b) & 1 ? set : ~set;
    }
    const bool has = e < (uint32_t)experts;
    const uint32_t first = has ? next_s[wave][e] : 0;
    const uint32_t below = __popcll(same & ((1ull << lane) - 1));
    wave_fence();
    if (has && below == 0) next_s[wave][e] = first + __popcll(same);
    wave_fence();
    if (i < hi) a.place[i] = has ? (int32_t)(first + below) : -1;
  }
}

// LANES threads move a token's row.
template <int LANES>
__global__ void __launch_bounds__(256) k_dispatch_rows(DispatchArgs a) {
  constexpr int TOKENS = 256 / LANES;
  const int l = threadIdx.x % LANES;
  for (int64_t token = (int64_t)blockIdx.x * TOKENS + threadIdx.x / LANES; token < a.tokens;
       token += (int64_t)gridDim.x * TOKENS)
    move_token(a, token, [&](int j) { return a.place[token * a.topk + j]; }, l, LANES);
}

// ---- back to the tokens -------------------------------------------------------------
// LANES threads take a token; N slots' vectors are under way at once.
template <int DT, int LANES, bool TINY>
__global__ void __launch_bounds__(256) k_combine(CombineArgs a) {
  constexpr int V = epv<DT>(), TOKENS = 256 / LANES, N = 8;
  const int l = threadIdx.x % LANES;
  const uint32_t cols = (uint32_t)a.cols;
  for (int64_t token = (int64_t)blockIdx.x * TOKENS + threadIdx.x / LANES; token < a.tokens;
       token += (int64_t)gridDim.x * TOKENS) {
    const int32_t* place = a.place + token * a.topk;
    const float* weights = a.weights ? a.weights + token * a.topk : nullptr;
    char* out = (char*)a.out + token * a.out_stride * Ty<DT>::E;
    for (uint32_t col = l * V; col < cols; col += LANES * V) {
      const RowPart<DT, TINY> p(col, cols);
      float acc[V];
#pragma unroll
      for (int t = 0; t < V; t++) acc[t] = 0.0f;
      for (int j0 = 0; j0 < a.topk; j0 += N) {
        u32x4 v[N];
        float w[N];
        bool has[N];
#pragma unroll
        for (int j = 0; j < N; j++) {
          const int k = j0 + j < a.topk ? j0 + j : j0;
          const int64_t at = place[k];
          has[j] = j0 + j < a.topk && at >= 0 && at < a.nrows;
          w[j] = weights ? weights[k] : 1.0f;
          v[j] = u32x4{0, 0, 0, 0};
          if (has[j]) v[j] = p.load((const char*)a.rows + at * a.rows_stride * Ty<DT>::E);
        }
#pragma unroll
        for (int j = 0; j < N; j++) {
          float f[V];
          unpack<DT>(v[j], f);
          // (an empty slot's weight may be anything)
          const float x = has[j] ? w[j] : 0.0f;
#pragma unroll
          for (int t = 0; t < V; t++) acc[t] = __builtin_fmaf(x, f[t], acc[t]);
        }
      }
      p.store(out, acc);
    }
  }
}

// The same for the gradient: a token's dy against its slots' rows.
template <int DT, int LANES, bool TINY>
__global__ void __launch_bounds__(256) k_combine_grad(CombineGradArgs a) {
  constexpr int V = epv<DT>(), TOKENS = 256 / LANES, W = LANES / 64, N = 8;
  __shared__ float dot_s[4][N];
  const int l = threadIdx.x % LANES;
  const uint32_t cols = (uint32_t)a.cols;
  // (a workgroup's tokens of a step stay together: its waves meet)
  for (int64_t first = (int64_t)blockIdx.x * TOKENS; first < a.tokens; first += (int64_t)gridDim.x * TOKENS) {
    const bool here = first + threadIdx.x / LANES < a.tokens;
    const int64_t token = here ? first + threadIdx.x / LANES : first;
    const int32_t* place = a.place + token * a.topk;
    const char* dy = (const char*)a.dy + token * a.dy_stride * Ty<DT>::E;
    for (int j0 = 0; j0 < a.topk; j0 += N) {
      int64_t at[N];
      float w[N], dot[N];
#pragma unroll
      for (int j = 0; j < N; j++) {
        const int k = j0 + j < a.topk ? j0 + j : j0;
        at[j] = here && j0 + j < a.topk ? place[k] : -1;
        at[j] = at[j] < a.nrows ? at[j] : -1;
        w[j] = a.weights ? a.weights[token * a.topk + k] : 1.0f;
        dot[j] = 0.0f;
      }
      for (uint32_t col = l * V; col < cols; col += LANES * V) {
        const RowPart<DT, TINY> p(col, cols);
        float d[V];
        unpack<DT>(p.load(dy), d);
        u32x4 v[N];
        if (a.dweights) {
#pragma unroll
          for (int j = 0; j < N; j++)
            if (at[j] >= 0) v[j] = p.load((const char*)a.rows + at[j] * a.rows_stride * Ty<DT>::E);
#pragma unroll
          for (int j = 0; j < N; j++) {
            if (at[j] < 0) continue;
            float f[V];
            unpack<DT>(v[j], f);
#pragma unroll
            for (int t = 0; t < V; t++) dot[j] = p.own(t) ? __builtin_fmaf(d[t], f[t], dot[j]) : dot[j];
          }
        }
        if (a.drows) {
#pragma unroll
          for (int j = 0; j < N; j++) {
            if (at[j] < 0) continue;
            float f[V];
#pragma unroll
            for (int t = 0; t < V; t++) f[t] = w[j] * d[t];
            p.store((char*)a.drows + at[j] * a.drows_stride * Ty<DT>::E, f);
          }
        }
      }
      if (!a.dweights) continue;
#pragma unroll
      for (int j = 0; j < N; j++) dot[j] = group_sum<(LANES < 64 ? LANES : 64)>(dot[j]);
      if constexpr (W > 1) {
        __syncthreads();
        if ((threadIdx.x & 63) == 0) {
#pragma unroll
          for (int j = 0; j < N; j++) dot_s[threadIdx.x >> 6][j] = dot[j];
        }
        __syncthreads();
        if (threadIdx.x < N && j0 + (int)threadIdx.x < a.topk) {
          const int j = threadIdx.x;
          a.dweights[token * a.topk + j0 + j] = (dot_s[0][j] + dot_s[1][j]) + (dot_s[2][j] + dot_s[3][j]);
        }
      } else if (here && l == 0) {
#pragma unroll
        for (int j = 0; j < N; j++)
          if (j0 + j < a.topk) a.dweights[token * a.topk + j0 + j] = dot[j];
      }
    }
  }
}

unsigned grid_of(int64_t tokens, int lanes) {
  const int64_t per = 256 / lanes, wg = (tokens + per - 1) / per;
  return (unsigned)std::min<int64_t>(wg, (int64_t)1 << 22);
}

template <int DT>
hipError_t combine(const CombineArgs& a, hipStream_t s) {
  constexpr int V = epv<DT>();
  const int64_t nv = (a.cols + V - 1) / V;
  if (a.cols < V) return launch<k_combine<DT, 8, true>>(dim3(grid_of(a.tokens, 8)), dim3(256), s, a);
  if (nv <= 8) return launch<k_combine<DT, 8, false>>(dim3(grid_of(a.tokens, 8)), dim3(256), s, a);
  if (nv <= 128) return launch<k_combine<DT, 64, false>>(dim3(grid_of(a.tokens, 64)), dim3(256), s, a);
  return launch<k_combine<DT, 256, false>>(dim3(grid_of(a.tokens, 256)), dim3(256), s, a);
}
template <int DT>
hipError_t combine_grad(const CombineGradArgs& a, hipStream_t s) {
  constexpr int V = epv<DT>();
  const int64_t nv = (a.cols + V - 1) / V;
  if (a.cols < V) return launch<k_combine_grad<DT, 8, true>>(dim3(grid_of(a.tokens, 8)), dim3(256), s, a);
  if (nv <= 8) return launch<k_combine_grad<DT, 8, false>>(dim3(grid_of(a.tokens, 8)), dim3(256), s, a);
  if (nv <= 128) return launch<k_combine_grad<DT, 64, false>>(dim3(grid_of(a.tokens, 64)), dim3(256), s, a);
  return launch<k_combine_grad<DT, 256, false>>(dim3(grid_of(a.tokens, 256)), dim3(256), s, a);
}

}  // namespace

hipError_t launch_dispatch(const DispatchArgs& a, hipStream_t s) {
  if (a.chunks == 0) return launch<k_dispatch_few>(dim3((unsigned)a.tokens + 1), dim3(256), s, a);
  hipError_t e = launch<k_dispatch_count>(dim3(a.chunks), dim3(256), s, a);
  if (e != hipSuccess) return e;
  e = launch<k_dispatch_place>(dim3(a.chunks), dim3(kPlaceThreads), s, a);
  if (e != hipSuccess || (a.row_bytes == 0 && !a.scales)) return e;
  const int64_t bytes = std::max(a.row_bytes, a.scale_bytes);
  if (bytes <= 256) return launch<k_dispatch_rows<16>>(dim3(grid_of(a.tokens, 16)), dim3(256), s, a);
  if (bytes <= 2048) return launch<k_dispatch_rows<64>>(dim3(grid_of(a.tokens, 64)), dim3(256), s, a);
  return launch<k_dispatch_rows<256>>(dim3(grid_of(a.tokens, 256)), dim3(256), s, a);
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
