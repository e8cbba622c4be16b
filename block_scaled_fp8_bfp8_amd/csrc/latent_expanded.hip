// Latent attention in the expanded form: ragged causal attention whose keys and values were expanded
// from the latents by a GEMM (kv [Tk][H][256]: 128 key dimensions, then 128 value dimensions of a head)
// and whose keys end in a rotary part that all heads share (rope [Tk][64]).
//
//   o[t, h] = sum_j softmax_j(scale * (q[t, h, :128] . kv[j, h, :128] + q[t, h, 128:] . rope[j])) kv[j, h, 128:]
//
// over the keys j of t's sequence up to t (the last query token sees the last key).
//
// One pass with the running maximum and sum of the softmax. A workgroup takes 128 query rows of one
// head, 32 for each wave, and walks the keys in tiles of 64, copied straight to LDS (a kv row is 512
// bytes, the rotary key 128). Both products are 32x32x16 matrix-core products, formed transposed
// (S^T = K Q^T, O^T = V^T P^T): a lane then holds scores of one query row, r = lane % 32, which are
// its operand of the second product without any exchange, and the running maximum and sum are plain
// per-lane numbers. V is read from the tile with transposing LDS reads.
#include "device_common.h"
#include "latent.h"
#include "launch.h"

namespace bfp8 {

namespace {

constexpr int kTile = 64;    // keys of a tile
constexpr int kBM = 128;     // query rows of a workgroup
constexpr int kNope = 128;   // key dimensions of a head before the rotary part
constexpr int kV = 128;      // value dimensions
constexpr int kKvRow = 2 * (kNope + kV);
constexpr float kNegInf = -__builtin_inff();
// The running maximum may lag by a factor of 2^kSlack: weights stay within 2^8, far inside fp16 and
// bf16, and the accumulator is rescaled only when a tile exceeds that.
constexpr float kSlack = 8.f;

// XOR of the 16-byte columns of a key's 512-byte row in LDS: conflict-free for the score reads (one
// column of 16 consecutive keys) and for the transposing value reads (32 lanes: 64 bytes of 4 consecutive
// keys, so the low two key bits move whole 64-byte pieces).
__device__ __forceinline__ int swz(int key) { return ((key & 3) << 2) | ((key >> 2) & 3); }

template <bool kF16>
__device__ __forceinline__ v16f mfma(const v4i& a, const v4i& b, const v16f& c) {
  if constexpr (kF16)
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(v8h, a), __builtin_bit_cast(v8h, b), c, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(v8bf, a), __builtin_bit_cast(v8bf, b), c, 0, 0, 0);
}

template <bool kF16>
__device__ __forceinline__ uint32_t pack16(float lo, float hi) {
  if constexpr (kF16) return f32_to_f16_rne(lo) | (f32_to_f16_rne(hi) << 16);
  else return pack_bf16(lo, hi);
}

template <bool kF16>
__global__ __launch_bounds__(256, 2) void latent_expanded_kernel(LatentExpandedArgs a) {
  __shared__ __align__(1024) uint8_t tile[kTile * (kKvRow + 2 * kRopeDim)];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int r = lane & 31, g = lane >> 5;
  const int head = blockIdx.x % a.H, index = blockIdx.x / a.H;

  // ---- the index-th block of 128 query rows over all sequences
  int* sh = reinterpret_cast<int*>(tile);
  const int per = (a.B + 255) / 256;
  const int b0 = min(tid * per, a.B), b1 = min(b0 + per, a.B);
  auto clip = [](int v, int top) { return min(max(v, 0), top); };
  int mine = 0;
  for (int b = b0; b < b1; ++b) mine += (max(clip(a.cu_q[b + 1], a.Tq) - clip(a.cu_q[b], a.Tq), 0) + kBM - 1) / kBM;
  int first = mine;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int x = __shfl_up(first, d);
    if (lane >= d) first += x;
  }
  if (lane == 63) sh[wave] = first;
  __syncthreads();
  int total = 0;
  for (int w = 0; w < 4; ++w) {
    if (w < wave) first += sh[w];
    total += sh[w];
  }
  first -= mine;
  if (index >= total) return;
  __syncthreads();
  if (index >= first && index < first + mine) {
    for (int b = b0; b < b1; ++b) {
      const int n = (max(clip(a.cu_q[b + 1], a.Tq) - clip(a.cu_q[b], a.Tq), 0) + kBM - 1) / kBM;
      if (index < first + n) {
        sh[0] = b;
        sh[1] = n - 1 - (index - first);  // a sequence's last block, the longest, first
        break;
      }
      first += n;
    }
  }
  __syncthreads();
  const int b = sh[0], blk = sh[1];
  __syncthreads();
  const int q0 = clip(a.cu_q[b], a.Tq), nq = clip(a.cu_q[b + 1], a.Tq) - q0;
  const int k0 = clip(a.cu_k[b], a.Tk), nk = max(clip(a.cu_k[b + 1], a.Tk) - k0, 0);

  // ---- this lane's query row
  const int row = blk * kBM + wave * 32 + r;
  const bool row_ok = row < nq;
  const int limit = row_ok ? clip(nk - nq + row + 1, nk) : 0;  // keys it sees
  const int keys = clip(nk - nq + min(blk * kBM + kBM, nq), nk);  // keys the block sees
  const uint16_t* qs = a.q + (int64_t)(q0 + (row_ok ? row : 0)) * a.q_tok + (int64_t)head * a.q_head;
  v4i q[12];
#pragma unroll
  for (int ks = 0; ks < 12; ++ks) {
    q[ks] = v4i{0, 0, 0, 0};
    if (row_ok) q[ks] = *reinterpret_cast<const v4i*>(qs + 16 * ks + 8 * g);
  }
  v16f acc[4];
#pragma unroll
  for (int d = 0; d < 4; ++d)
#pragma unroll
    for (int i = 0; i < 16; ++i) acc[d][i] = 0.f;
  float m = kNegInf, l = 0.f;
  const float c = a.scale * 1.44269504088896341f;
  const uint32_t lds = lds_addr(tile);
  const uint8_t* kv = reinterpret_cast<const uint8_t*>(a.kv + (int64_t)k0 * a.kv_tok + (int64_t)head * a.kv_head);
  const uint8_t* rope = reinterpret_cast<const uint8_t*>(a.rope + (int64_t)k0 * a.ld_rope);

  for (int t0 = 0; t0 < keys; t0 += kTile) {
    // the tile into LDS; keys past the block's repeat its last (finite, and masked)
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int kk = (wave * 8 + j) * 2 + (lane >> 5);
      const int64_t key = min(t0 + kk, keys - 1);
      copy16_from(kv + key * a.kv_tok * 2 + (((lane & 31) ^ swz(kk)) << 4), lds + (wave * 8 + j) * 1024);
    }
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int kk = (wave * 2 + j) * 8 + (lane >> 3);
      const int64_t key = min(t0 + kk, keys - 1);
      copy16_from(rope + key * a.ld_rope * 2 + (((lane & 7) ^ lds_swizzle(kk)) << 4),
                  lds + kTile * kKvRow + (wave * 2 + j) * 1024);
    }
    wait_copies();
    __syncthreads();

    // ---- scores of 2 x 32 keys: lane (r, g), register i: key 8 (i / 4) + 4 g + i % 4
    v16f s[2];
#pragma unroll
    for (int kt = 0; kt < 2; ++kt) {
      const int kk = kt * 32 + r;
#pragma unroll
      for (int i = 0; i < 16; ++i) s[kt][i] = 0.f;
#pragma unroll
      for (int ks = 0; ks < 8; ++ks) {
        const v4i k = *reinterpret_cast<const v4i*>(tile + kk * kKvRow + (((2 * ks + g) ^ swz(kk)) << 4));
        s[kt] = mfma<kF16>(k, q[ks], s[kt]);
      }
#pragma unroll
      for (int ks = 0; ks < 4; ++ks) {
        const v4i k = *reinterpret_cast<const v4i*>(tile + kTile * kKvRow + kk * 128 + (((2 * ks + g) ^ lds_swizzle(kk)) << 4));
        s[kt] = mfma<kF16>(k, q[8 + ks], s[kt]);
      }
    }
    float top = kNegInf;
    const bool masked = __any(t0 + kTile > limit);
#pragma unroll
    for (int kt = 0; kt < 2; ++kt)
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        s[kt][i] *= c;
        if (masked && t0 + kt * 32 + 8 * (i >> 2) + 4 * g + (i & 3) >= limit) s[kt][i] = kNegInf;
        top = fmaxf(top, s[kt][i]);
      }
    top = fmaxf(top, __shfl_xor(top, 32));
    if (__any(top > m + kSlack)) {
      const float next = fmaxf(m, top);
      const float f = m == next ? 1.f : __builtin_amdgcn_exp2f(m - next);
      m = next;
      l *= f;
#pragma unroll
      for (int d = 0; d < 4; ++d) acc[d] *= f;
    }
    const float ref = m == kNegInf ? 0.f : m;
#pragma unroll
    for (int kt = 0; kt < 2; ++kt)
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        s[kt][i] = __builtin_amdgcn_exp2f(s[kt][i] - ref);
        l += s[kt][i];
      }
    // ---- O^T += V^T P^T: 16 keys a step, of which lane g holds 4 g + {0..3} and 8 + 4 g + {0..3}
#pragma unroll
    for (int kt = 0; kt < 2; ++kt)
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        v4i p;
#pragma unroll
        for (int i = 0; i < 4; ++i) p[i] = (int)pack16<kF16>(s[kt][8 * u + 2 * i], s[kt][8 * u + 2 * i + 1]);
        typedef short v4s __attribute__((ext_vector_type(4)));
        typedef __attribute__((address_space(3))) v4s lds_v4s;
        // the key row this lane addresses (and the one 8 further on), and its 8 bytes of 32 columns
        const int vk = kt * 32 + 16 * u + 4 * g + ((lane >> 2) & 3);
#pragma unroll
        for (int d = 0; d < 4; ++d) {
          const int col = 16 + 4 * d + 2 * ((lane >> 4) & 1) + ((lane >> 1) & 1);
          const uint8_t* x = tile + vk * kKvRow + ((col ^ swz(vk)) << 4) + 8 * (lane & 1);
          const uint8_t* y = tile + (vk + 8) * kKvRow + ((col ^ swz(vk + 8)) << 4) + 8 * (lane & 1);
          const v2i lo = __builtin_bit_cast(v2i, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4s*)x));
          const v2i hi = __builtin_bit_cast(v2i, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4s*)y));
          acc[d] = mfma<kF16>(v4i{lo[0], lo[1], hi[0], hi[1]}, p, acc[d]);
        }
      }
    __syncthreads();
  }

  l += __shfl_xor(l, 32);
  if (!row_ok) return;
  const float inv = l == 0.f ? 0.f : 1.0f / l;  // a row that sees no key is zero
  uint16_t* dst = a.out + (int64_t)(q0 + row) * a.o_tok + (int64_t)head * a.o_head + 4 * g;
#pragma unroll
  for (int d = 0; d < 4; ++d)
#pragma unroll
    for (int i = 0; i < 4; ++i)
      *reinterpret_cast<uint2*>(dst + 32 * d + 8 * i) =
          make_uint2(pack16<kF16>(acc[d][4 * i] * inv, acc[d][4 * i + 1] * inv),
                     pack16<kF16>(acc[d][4 * i + 2] * inv, acc[d][4 * i + 3] * inv));
}

}  // namespace

int64_t latent_expanded_blocks(int64_t Tq, int64_t B) { return Tq / kBM + (Tq < B ? Tq : B); }

hipError_t launch_latent_expanded(const LatentExpandedArgs& args, bool f16, hipStream_t stream) {
  const dim3 grid((unsigned)(latent_expanded_blocks(args.Tq, args.B) * args.H));
  if (f16) hipLaunchKernelGGL((latent_expanded_kernel<true>), grid, dim3(256), 0, stream, args);
  else hipLaunchKernelGGL((latent_expanded_kernel<false>), grid, dim3(256), 0, stream, args);
  return hipGetLastError();
}

}  // namespace bfp8
