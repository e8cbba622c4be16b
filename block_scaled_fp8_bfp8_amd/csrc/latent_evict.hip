// Eviction from the paged FP8 latent cache by accumulated weight: a sequence longer than `budget` keeps its last
// `recent` tokens and, of the earlier ones, the budget - recent with the largest mass (of equal ones the earlier), in
// their order, as its tokens 0 .. budget - 1.
//
// Two launches. The first selects: a workgroup a sequence finds the least mass that stays, a byte at a time from the top of
// integers that rise with the masses, by counting the values of each byte among those that start like it (8192 masses stay
// in registers; lanes that share a value count together), and then places the tokens that stay by sums over the lanes,
// waves and chunks before them. The second moves rows and scale codes. Onto other pages every token goes by itself; in place,
// where a kept token never moves up (its place is the number of kept ones before it), a workgroup moves one column of a
// sequence's rows, a chunk of tokens at a time, and another its codes: what a chunk writes lies before everything that later
// chunks read, and a barrier stands between the reads and the writes of a chunk. Selection is bound by its chain of barriers, the
// moves by HBM, in place by the latency of a chunk where sequences are few.
//
// Measured: 64 sequences of 500 to 8000 tokens to 4096, onto other pages: selection 15 us, moves 60 us (267 MB, 4.5 TB/s); one of 1111 to
// 1024: 8.1 and 3.8 us. In place, both together: 64 of 8000 83 us, 64 of 4097 48 us, one of 4097 20 to 22 us, one of 32769 to 32768 139 us.
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

// Adds one to the bins of the lanes whose value counts. Most often many lanes share the first one's bin: they add together.
__device__ __forceinline__ void count_bins(int* bins, uint32_t bin, bool counts, int lane) {
  const uint64_t on = __ballot(counts);
  if (on == 0) return;
  const int leader = __builtin_ctzll(on);
  const uint32_t common = (uint32_t)__builtin_amdgcn_readlane((int)bin, leader);
  const bool together = counts && bin == common;
  const int n = __popcll(__ballot(together));
  if (lane == leader) atomicAdd(bins + common, n);
  if (counts && !together) atomicAdd(bins + bin, 1);
}

// The masses are read a chunk at a time, thread t's i-th of a chunk being token 1024 i + t of it.
__global__ __launch_bounds__(kThreads) void latent_select_kernel(LatentEvictArgs a) {
  __shared__ __attribute__((aligned(16))) int bins[4][256];  // of each byte, from the top
  __shared__ int2 wave_sums[2][kHeld * kSelectWaves];
  const int b = blockIdx.x, tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  reinterpret_cast<int*>(bins)[tid] = 0;
  const Length len = length_of(a, b);
  const int n = len.n;
  const float* mass = a.mass + (int64_t)b * a.mass_stride;
  float* mass_out = a.mass_out + (int64_t)b * a.mass_out_stride;
  int32_t* kept = a.kept + (int64_t)b * a.budget;
  const bool cut = n > a.budget;
  const int old = cut ? n - a.recent : n;  // tokens that may go
  const int want = len.kept - (n - old);   // of these stay

  float first[kHeld];  // masses of the first chunk
#pragma unroll
  for (int i = 0; i < kHeld; ++i) {
    const int j = i * kThreads + tid;
    first[i] = j < n ? mass[j] : 0.f;
  }
  uint32_t least = 0;  // the least mass that stays, as an integer, and how many of those that equal it
  int equals = 0;
  if (cut && want > 0) {
    equals = want;
    const int held_chunks = min((old + kThreads - 1) / kThreads, kHeld);
    __syncthreads();
#pragma unroll 1
    for (int byte = 0; byte < 4; ++byte) {
      const int shift = 24 - 8 * byte;
      auto count = [&](uint32_t u, bool there) {  // of the values that start with the bytes found so far
        count_bins(bins[byte], (u >> shift) & 255u, there && (byte == 0 || (u ^ least) >> (shift + 8) == 0), lane);
      };
#pragma unroll
      for (int i = 0; i < kHeld; ++i)
        if (i < held_chunks) count(rising(first[i]), i * kThreads + tid < old);
      for (int j0 = kChunk; j0 < old; j0 += kThreads) count(j0 + tid < old ? rising(mass[j0 + tid]) : 0u, j0 + tid < old);
      __syncthreads();
      // bins from the top, four a lane: the first at which the sum reaches what is still wanted (every wave finds it)
      const v4i c = *reinterpret_cast<const v4i*>(&bins[byte][252 - 4 * lane]);
      const int all = c[0] + c[1] + c[2] + c[3], through = wave_scan(all);
      const uint64_t reached = __ballot(through >= equals);
      const int at = reached ? __builtin_ctzll(reached) : 63;  // (always reached, unless the masses change under way)
      int above = __builtin_amdgcn_readlane(through - all, at), bin = 255 - 4 * at;
#pragma unroll
      for (int k = 3; k > 0; --k) {
        const int here = __builtin_amdgcn_readlane(c[k], at);
        if (bin == 252 - 4 * at + k && above + here < equals) above += here, --bin;
      }
      least |= (uint32_t)bin << shift;
      equals -= above;
    }
  }

  // ---- places: of those that stay for certain, and of those that equal the least, of which the first `equals` stay
  int certain_before = 0, same_before = 0, turn = 0;
  for (int j0 = 0; j0 < n; j0 += kChunk, turn ^= 1) {
    float m[kHeld];
    uint64_t certain[kHeld], same[kHeld];
    const int chunks = min((n - j0 + kThreads - 1) / kThreads, kHeld);
#pragma unroll
    for (int i = 0; i < kHeld; ++i) {
      const int j = j0 + i * kThreads + tid;
      m[i] = j0 == 0 ? first[i] : j < n ? mass[j] : 0.f;
      const uint32_t u = rising(m[i]);
      const bool may_go = j < old && cut;
      certain[i] = __ballot(j < n && (!may_go || (want > 0 && u > least)));
      same[i] = __ballot(may_go && want > 0 && u == least);
      if (lane == 0) wave_sums[turn][i * kSelectWaves + wave] = make_int2(__popcll(certain[i]), __popcll(same[i]));
    }
    wait_copies();  // (every mass of the chunk has been read before the barrier, behind which they may be overwritten)
    __syncthreads();
    // the 128 sums in order: lane l scans sums 2 l and 2 l + 1
    const int2 x = wave_sums[turn][2 * lane], y = wave_sums[turn][2 * lane + 1];
    const int certain_up = wave_scan(x.x + y.x), same_up = wave_scan(x.y + y.y);
#pragma unroll
    for (int i = 0; i < kHeld; ++i) {
      if (i >= chunks) break;
      const int e = i * kSelectWaves + wave, at = e >> 1;  // (the same in the whole wave)
      auto before = [&](int up, int x1, int y1, uint64_t votes) {
        const int sums = __builtin_amdgcn_readlane(up, at) - __builtin_amdgcn_readlane(y1, at) - (e & 1 ? 0 : __builtin_amdgcn_readlane(x1, at));
        return sums + __popcll(votes & ((1ull << lane) - 1));
      };
      const int c = certain_before + before(certain_up, x.x, y.x, certain[i]), s = same_before + before(same_up, x.y, y.y, same[i]);
      const bool keep = (certain[i] >> lane & 1) || ((same[i] >> lane & 1) && s < equals);
      const int place = c + min(s, equals);
      // (places are no later than their tokens; no more than fit, should the masses change under way)
      if (keep && place < len.kept) {
        kept[place] = j0 + i * kThreads + tid;
        mass_out[place] = m[i];
      }
    }
    certain_before += __builtin_amdgcn_readlane(certain_up, 63);
    same_before += __builtin_amdgcn_readlane(same_up, 63);
  }
  __syncthreads();  // (the last chunk's masses have been read)
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

// A row of a token without a page, to read from.
struct MissingRow {
  uint16_t v[kLatentRow / 2];
  constexpr MissingRow() : v{} {
    for (int i = kLatentDim / 2; i < kLatentRow / 2; ++i) v[i] = 0x7fff;
  }
};
__device__ const __attribute__((aligned(16))) MissingRow kMissingRow{};

constexpr int kColumns = kLatentRow / 128, kMoveThreads = 1024, kRounds = 4;
constexpr uint32_t kNowhere = 0xffffffffu;

// In place, a column of 128 bytes of a sequence's rows: 8 lanes move a row's, kRounds rows a thread and chunk. As a token never moves up, a
// chunk is read from its own places on: its reads may pass the writes of the chunk before, and are under way meanwhile, as are the look-ups
// of the two after. Only between a chunk's own reads and writes stands a barrier. A wave's 32 tokens are looked up by a lane each, for the
// place they come from and for the one they go to, and nothing is read under a condition that the compiler would wait for: what
// stays, or lies nowhere, is read from the row of none. (1 sequence, 4096 of
// 4097 tokens, selection included: 22 us, 42 with each chunk's chain of loads by itself; 64 sequences of 8000: 82 and 102.)
__device__ __forceinline__ void compact_rows(const LatentEvictArgs& a, int b, int column) {
  const int n = length_of(a, b).kept;
  if (n == 0) return;
  constexpr int kEach = kMoveThreads / 8, kChunk = kEach * kRounds;
  static_assert(8 * kRounds == 32, "a wave's tokens of a chunk are half its lanes");
  const int32_t* kept = a.kept + (int64_t)b * a.budget;
  const int32_t* table = a.cache.table + (int64_t)b * a.cache.table_stride;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int page_size = a.cache.page_size, last = a.cache.table_width - 1;
  const uint32_t page_units = (uint32_t)(a.cache.page_stride / 128);  // (rows are whole units of 128 bytes)
  // the token of a chunk that the lane looks up, and whether for where it goes
  const int mine = ((lane & 31) >> 3) * kEach + wave * 8 + (lane & 7);
  const bool goes = lane >= 32;
  struct Place {
    int page, off;  // (off < 0: the token stays)
  };
  auto token = [&](int t0) { return kept[min(t0 + mine, n - 1)]; };
  auto look_up = [&](int t0, int from) {
    const int t = t0 + mine, at = goes ? t : from, col = min(at / page_size, last);
    return Place{table[col], t < n && from != t ? at - col * page_size : -1};
  };
  auto unit_of = [&](const Place& p) {
    const bool there = p.off >= 0 && (unsigned)p.page < (unsigned)a.cache.pages;
    return there ? (uint32_t)p.page * page_units + (uint32_t)p.off * (kLatentRow / 128) : kNowhere;
  };
  const int in_row = column * 128 + (lane & 7) * 16, row = lane >> 3;
  const v4i* none = reinterpret_cast<const v4i*>(reinterpret_cast<const uint8_t*>(&kMissingRow) + in_row);
  uint8_t* base = a.rows + in_row;
  auto unit_at = [&](uint32_t units, int from) { return (uint32_t)__builtin_amdgcn_ds_bpermute((from + row) << 2, (int)units); };
  auto read = [&](uint32_t units, v4i* data) {
#pragma unroll
    for (int i = 0; i < kRounds; ++i) {
      const uint32_t u = unit_at(units, 8 * i);
      data[i] = *(u == kNowhere ? none : reinterpret_cast<const v4i*>(base + (uint64_t)u * 128));
    }
  };
  v4i data[kRounds], ahead[kRounds];
  uint32_t here = unit_of(look_up(0, token(0)));
  read(here, data);
  Place next = look_up(kChunk, token(kChunk));
  int from = token(2 * kChunk);
  for (int t0 = 0; t0 < n; t0 += kChunk) {
    const uint32_t then = unit_of(next);
    read(then, ahead);
    next = look_up(t0 + 2 * kChunk, from);
    from = token(t0 + 3 * kChunk);
    // this chunk has been read, by every wave
#pragma unroll
    for (int i = 0; i < kRounds; ++i) asm volatile("" : "+v"(data[i])::"memory");
    lds_barrier();
    asm volatile("" ::: "memory");
#pragma unroll
    for (int i = 0; i < kRounds; ++i) {
      const uint32_t u = unit_at(here, 32 + 8 * i);
      if (u != kNowhere) *reinterpret_cast<v4i*>(base + (uint64_t)u * 128) = data[i];
    }
    here = then;
#pragma unroll
    for (int i = 0; i < kRounds; ++i) data[i] = ahead[i];
  }
}

// In place, a sequence's scale codes, a chunk of kRounds a thread at a time.
__device__ __forceinline__ void compact_codes(const LatentEvictArgs& a, int b) {
  const int n = length_of(a, b).kept;
  const int32_t* kept = a.kept + (int64_t)b * a.budget;
  const int32_t* table = a.cache.table + (int64_t)b * a.cache.table_stride;
  for (int t0 = 0; t0 < n; t0 += kMoveThreads * kRounds) {
    int code[kRounds];
    bool moves[kRounds];
#pragma unroll
    for (int i = 0; i < kRounds; ++i) {
      const int t = t0 + i * kMoveThreads + (int)threadIdx.x;
      const int from = t < n ? kept[t] : t;
      moves[i] = from != t;
      int off = 0;
      const int page = moves[i] ? page_of(table, a.cache.table_width, a.cache.pages, a.cache.page_size, from, off) : -1;
      code[i] = page >= 0 ? a.scales[page * a.cache.scale_stride + off] : 255;
    }
    wait_copies();  // every code of this chunk has been read
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kRounds; ++i) {
      if (!moves[i]) continue;
      int off;
      const int page = page_of(table, a.cache.table_width, a.cache.pages, a.cache.page_size, t0 + i * kMoveThreads + (int)threadIdx.x, off);
      if (page >= 0) a.scales[page * a.cache.scale_stride + off] = (uint8_t)code[i];
    }
  }
}

__global__ __launch_bounds__(kMoveThreads) void latent_compact_kernel(LatentEvictArgs a) {
  const int b = (int)(blockIdx.x / (kColumns + 1)), column = (int)(blockIdx.x - (unsigned)b * (kColumns + 1));
  if (column < kColumns) compact_rows(a, b, column);
  else compact_codes(a, b);
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
    hipLaunchKernelGGL(latent_compact_kernel, dim3((unsigned)(a.B * (kColumns + 1))), dim3(kMoveThreads), 0, stream, a);
  }
  return hipGetLastError();
}

}  // namespace bfp8
