// Eviction from the paged FP8 latent cache by accumulated weight: a sequence longer than `budget` keeps its last
// `recent` tokens and, of the earlier ones, the budget - recent with the largest mass (of equal ones the earlier), in
// their order, as its tokens 0 .. budget - 1.
//
// Two launches. The first selects: a workgroup a sequence finds the least mass that stays, two bits at a time, by
// counting how many reach each of three candidates (the masses, as integers that rise with them, stay in registers;
// nothing is sorted and no counter is contended), and then places the tokens that stay by sums over the lanes, waves and
// chunks before them. The second moves rows and scale codes. Onto other pages every token goes by itself; in place,
// where a kept token never moves up (its place is the number of kept ones before it), a workgroup moves one column of a
// sequence's rows, a chunk of tokens at a time: what a chunk writes lies before everything that later chunks read, and
// a barrier stands between the reads and the writes of a chunk. Selection is bound by its chain of barriers, the moves
// by HBM.
#include <algorithm>

#include "device_latent.h"
#include "latent.h"
#include "launch.h"

namespace bfp8 {

namespace {

constexpr int kThreads = 1024, kSelectWaves = kThreads / 64;
constexpr int kHeld = 8;                        // masses a thread holds
constexpr int kChunk = kThreads * kHeld;        // tokens of a chunk

// An integer that rises with the mass: NaN above all, -0 as 0. Never 0.
__device__ __forceinline__ uint32_t rising(float m) {
  const uint32_t u = __float_as_uint(m + 0.f);
  if (m != m) return 0xffffffffu;
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}

struct Length {
  int n, kept;
};
__device__ __forceinline__ Length length_of(const LatentEvictArgs& a, int b) {
  const int reach = a.cache.table_width * a.cache.page_size;  // (below 2^31)
  const int n = min(max(a.lens[b], 0), reach);
  return {n, min(n, a.budget)};
}

// Sum over 16 lanes, in the last of them.
__device__ __forceinline__ int sum16(int v) {
  v += __builtin_amdgcn_update_dpp(0, v, 0x111, 0xf, 0xf, false);  // 1, 2, 4, 8 lanes up
  v += __builtin_amdgcn_update_dpp(0, v, 0x112, 0xf, 0xf, false);
  v += __builtin_amdgcn_update_dpp(0, v, 0x114, 0xf, 0xf, false);
  return v + __builtin_amdgcn_update_dpp(0, v, 0x118, 0xf, 0xf, false);
}

// The masses are read a chunk at a time, thread t's i-th of a chunk being token 1024 i + t of it.
__global__ __launch_bounds__(kThreads) void latent_select_kernel(LatentEvictArgs a) {
  __shared__ int wave_sums[2][kHeld][kSelectWaves];
  __shared__ int counts[2][3][kSelectWaves];
  const int b = blockIdx.x, tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const Length len = length_of(a, b);
  const int n = len.n;
  const float* mass = a.mass + (int64_t)b * a.mass_stride;
  float* mass_out = a.mass_out + (int64_t)b * a.mass_out_stride;
  int32_t* kept = a.kept + (int64_t)b * a.budget;
  const bool cut = n > a.budget;
  const int old = cut ? n - a.recent : n;  // tokens that may go
  const int want = len.kept - (n - old);   // of these stay

  float first[kHeld];  // masses of the first chunk
  const int held_chunks = min((n + kThreads - 1) / kThreads, kHeld);
#pragma unroll
  for (int i = 0; i < kHeld; ++i) {
    const int j = i * kThreads + tid;
    first[i] = j < n ? mass[j] : 0.f;
  }
  uint32_t least = 0;  // the least mass that stays, as an integer (0: all stay), and how many of those that equal it
  int equals = 0;
  if (cut && want == 0) least = 0xffffffffu;
  if (cut && want > 0) {
    uint32_t held[kHeld];
#pragma unroll
    for (int i = 0; i < kHeld; ++i) {
      held[i] = i * kThreads + tid < old ? rising(first[i]) : 0u;
    }
    int above = 0;  // masses above every value that starts with the bits found so far
    for (int shift = 30; shift >= 0; shift -= 2) {
      int c[3] = {0, 0, 0};
      auto count = [&](uint32_t u) {
#pragma unroll
        for (uint32_t k = 0; k < 3; ++k) c[k] += __popcll(__ballot(u >= (least | (k + 1) << shift)));
      };
#pragma unroll
      for (int i = 0; i < kHeld; ++i)
        if (i < held_chunks) count(held[i]);  // (uniform)
      for (int j0 = kChunk; j0 < old; j0 += kThreads) count(j0 + tid < old ? rising(mass[j0 + tid]) : 0u);
      const int turn = (shift >> 1) & 1;
      if (lane == 0)
#pragma unroll
        for (int k = 0; k < 3; ++k) counts[turn][k][wave] = c[k];
      __syncthreads();
      int total[3];
#pragma unroll
      for (int k = 0; k < 3; ++k) total[k] = counts[turn][k][lane & (kSelectWaves - 1)];
#pragma unroll
      for (int k = 0; k < 3; ++k) total[k] = __builtin_amdgcn_readlane(sum16(total[k]), 15);
      // the largest candidate that `want` masses reach
      const int k = total[2] >= want ? 3 : total[1] >= want ? 2 : total[0] >= want ? 1 : 0;
      if (k < 3) above = total[k];
      least |= (uint32_t)k << shift;
    }
    equals = want - above;
  }

  // ---- places
  int placed = 0, equal_before = 0;
  for (int j0 = 0; j0 < n; j0 += kChunk) {
    float m[kHeld];
    bool same[kHeld], keep[kHeld];
    int before[kHeld];
#pragma unroll
    for (int i = 0; i < kHeld; ++i) {
      const int j = j0 + i * kThreads + tid;
      m[i] = j0 == 0 ? first[i] : j < n ? mass[j] : 0.f;
      const uint32_t u = rising(m[i]);
      const bool may_go = j < old && cut;
      same[i] = may_go && u == least && want > 0;
      keep[i] = j < n && (!may_go || (want > 0 && u > least));
    }
    wait_copies();  // (every mass has been read before the barriers below, behind which they may be overwritten)
    // of those that equal the least the first stay
    auto count_before = [&](const bool* flag, int turn, int& carry, int* at) {
      uint64_t votes[kHeld];
#pragma unroll
      for (int i = 0; i < kHeld; ++i) {
        votes[i] = __ballot(flag[i]);
        if (lane == 0) wave_sums[turn][i][wave] = __popcll(votes[i]);
      }
      __syncthreads();
      // the kHeld * kSelectWaves = 128 sums in order: lane l scans sums 2 l and 2 l + 1
      const int* flat = &wave_sums[turn][0][0];
      const int x = flat[2 * lane], y = flat[2 * lane + 1], up = wave_scan(x + y);
#pragma unroll
      for (int i = 0; i < kHeld; ++i) {
        const int e = i * kSelectWaves + wave;  // (the same in the whole wave)
        const int through = __shfl(up, e >> 1), last = __shfl(y, e >> 1), first = __shfl(x, e >> 1);
        at[i] = carry + through - last - (e & 1 ? 0 : first) + __popcll(votes[i] & ((1ull << lane) - 1));
      }
      carry += __builtin_amdgcn_readlane(up, 63);
    };
    count_before(same, 0, equal_before, before);
#pragma unroll
    for (int i = 0; i < kHeld; ++i) keep[i] = keep[i] || (same[i] && before[i] < equals);
    count_before(keep, 1, placed, before);
    // (places are no later than their tokens; no more than fit, should the masses change under way)
#pragma unroll
    for (int i = 0; i < kHeld; ++i)
      if (keep[i] && before[i] < len.kept) {
        kept[before[i]] = j0 + i * kThreads + tid;
        mass_out[before[i]] = m[i];
      }
    __syncthreads();
  }
  for (int j = len.kept + tid; j < a.width; j += kThreads) mass_out[j] = 0.f;
  for (int j = len.kept + tid; j < a.budget; j += kThreads) kept[j] = -1;
  if (tid == 0) a.lens_out[b] = len.kept;
}

// Where token `pos` of a sequence lies (-1: nowhere), in rows of the cache.
__device__ __forceinline__ int page_of(const int32_t* table, int width, int pages, int page_size, int pos, int& off) {
  const int col = pos / page_size;
  off = pos - col * page_size;
  const int page = col < width ? table[col] : -1;
  return page >= pages ? -1 : page;
}

constexpr int kPieces = kLatentRow / 16;
// What a token without a page reads as.
__device__ __forceinline__ uint4 missing(int piece) {
  return piece < kLatentDim / 16 ? make_uint4(0, 0, 0, 0) : make_uint4(0x7fff7fffu, 0x7fff7fffu, 0x7fff7fffu, 0x7fff7fffu);
}

// Onto other pages: a wave moves 8 tokens in pieces of 16 bytes.
constexpr int kTokens = 8;
__global__ __launch_bounds__(256) void latent_move_kernel(LatentEvictArgs a, int each) {
  const int b = (int)(blockIdx.x / (unsigned)each), first = (int)(blockIdx.x - (unsigned)b * each);
  const int n = length_of(a, b).kept;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int32_t* kept = a.kept + (int64_t)b * a.budget;
  const int32_t* from = a.cache.table + (int64_t)b * a.cache.table_stride;
  const int32_t* to = a.to + (int64_t)b * a.to_stride;
  for (int t0 = (first * 4 + wave) * kTokens; t0 < n; t0 += each * 4 * kTokens) {
    const int mine = t0 + (lane & (kTokens - 1));
    int src_off = 0, dst_off = 0;
    const bool there = mine < n;
    const int src = there ? page_of(from, a.cache.table_width, a.cache.pages, a.cache.page_size, kept[mine], src_off) : -1;
    const int dst = there ? page_of(to, a.to_width, a.cache.pages, a.cache.page_size, mine, dst_off) : -1;
    const int64_t src_at = src < 0 ? -1 : src * a.cache.page_stride + (int64_t)src_off * kLatentRow;
    const int64_t dst_at = dst < 0 ? -1 : dst * a.cache.page_stride + (int64_t)dst_off * kLatentRow;
    const int code = src < 0 ? 255 : (int)a.cache.scales[src * a.cache.scale_stride + src_off];
    if (dst >= 0 && lane < kTokens) a.scales[dst * a.cache.scale_stride + dst_off] = (uint8_t)code;
    constexpr int kEach = kTokens * kPieces / 64;
    uint4 data[kEach];
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
      const int c = lane + 64 * i, token = c / kPieces, piece = c - token * kPieces;
      const int64_t at = __shfl(src_at, token);
      data[i] = missing(piece);
      if (at >= 0) data[i] = *reinterpret_cast<const uint4*>(a.cache.rows + at + piece * 16);
    }
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
      const int c = lane + 64 * i, token = c / kPieces, piece = c - token * kPieces;
      const int64_t at = __shfl(dst_at, token);
      if (at >= 0) *reinterpret_cast<uint4*>(a.rows + at + piece * 16) = data[i];
    }
  }
}

// In place: workgroup (b, column of 128 bytes); 8 lanes a row, kRounds rows a thread and chunk. The column 0 workgroup
// moves the scale codes too.
constexpr int kColumns = kLatentRow / 128, kMoveThreads = 1024, kRounds = 4;
constexpr int kMoveChunk = kMoveThreads / 8 * kRounds;
__global__ __launch_bounds__(kMoveThreads) void latent_compact_kernel(LatentEvictArgs a) {
  const int b = (int)(blockIdx.x / kColumns), column = (int)(blockIdx.x - (unsigned)b * kColumns);
  const int n = length_of(a, b).kept;
  const int32_t* kept = a.kept + (int64_t)b * a.budget;
  const int32_t* table = a.cache.table + (int64_t)b * a.cache.table_stride;
  const int in_row = column * 128 + (threadIdx.x & 7) * 16;
  const bool codes = column == 0 && (threadIdx.x & 7) == 0;
  for (int t0 = 0; t0 < n; t0 += kMoveChunk) {
    uint4 data[kRounds];
    int code[kRounds];
    bool moves[kRounds];
#pragma unroll
    for (int i = 0; i < kRounds; ++i) {
      const int t = t0 + i * (kMoveThreads / 8) + (threadIdx.x >> 3);
      const int from = t < n ? kept[t] : t;
      moves[i] = from != t;
      int off = 0;
      const int page = moves[i] ? page_of(table, a.cache.table_width, a.cache.pages, a.cache.page_size, from, off) : -1;
      data[i] = missing(in_row / 16);
      code[i] = 255;
      if (page >= 0) {
        data[i] = *reinterpret_cast<const uint4*>(a.rows + page * a.cache.page_stride + (int64_t)off * kLatentRow + in_row);
        if (codes) code[i] = a.scales[page * a.cache.scale_stride + off];
      }
    }
    wait_copies();  // every row of this chunk has been read
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kRounds; ++i) {
      if (!moves[i]) continue;
      const int t = t0 + i * (kMoveThreads / 8) + (threadIdx.x >> 3);
      int off;
      const int page = page_of(table, a.cache.table_width, a.cache.pages, a.cache.page_size, t, off);
      if (page < 0) continue;
      *reinterpret_cast<uint4*>(a.rows + page * a.cache.page_stride + (int64_t)off * kLatentRow + in_row) = data[i];
      if (codes) a.scales[page * a.cache.scale_stride + off] = (uint8_t)code[i];
    }
  }
}

}  // namespace

hipError_t launch_latent_evict(const LatentEvictArgs& a, hipStream_t stream) {
  hipLaunchKernelGGL(latent_select_kernel, dim3((unsigned)a.B), dim3(kThreads), 0, stream, a);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  if (a.to != nullptr) {
    // a workgroup for every 32 tokens that may stay, but no more than 16384 in all beside one a sequence
    const int64_t reach = std::min<int64_t>((int64_t)a.cache.table_width * a.cache.page_size, a.budget);
    const int64_t each = std::max<int64_t>(std::min<int64_t>((reach + 4 * kTokens - 1) / (4 * kTokens), 16384 / a.B + 1), 1);
    hipLaunchKernelGGL(latent_move_kernel, dim3((unsigned)(each * a.B)), dim3(256), 0, stream, a, (int)each);
  } else {
    hipLaunchKernelGGL(latent_compact_kernel, dim3((unsigned)(a.B * kColumns)), dim3(kMoveThreads), 0, stream, a);
  }
  return hipGetLastError();
}

}  // namespace bfp8
