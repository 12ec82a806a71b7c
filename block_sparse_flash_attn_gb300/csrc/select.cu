// Block masks chosen by a cheap score: for every 128-query block, the key
// blocks whose mean key agrees best with its mean query.
//
// The mean over a block's tokens is taken per channel and rounded to 7 bits
// beside the block's largest entry (one power of two a block: with E =
// floor(log2 max |mean|), t = rint(mean 2^(6 - E)), half to even; entries that
// are not finite count as zero).  The score of (query block, key block) is
//   sum_d tq_d * tk_d * 2^(Ek - 6),
// a whole number below 2^22 times a power of two: 32-bit sums of it are exact
// in any order, on any unit.  The query block's own power of two is left out,
// it does not change the order within a row.  So the mask is a function of the
// inputs alone: equal scores go to the lowest index, and a mask never depends
// on the order of a sum.  For the same reason the means themselves are exact
// sums (hi + lo, two-sum), rounded once.
//
// Cost: Q and K are read once (2 bytes an element; the bound: memory), each
// element costs one exact addition (6 operations).  The scores are one small
// matrix product per head on bf16 tensor instructions (whole numbers up to 128
// are exact in bf16); a row's k-th best is searched among the scores'
// order-preserving bit patterns, held in a warp's registers.
//
// Measured at 65536 tokens, 32 + 8 heads of 128, causal: means 104 us (6.4 TB/s,
// 97% of a plain copy's rate), choice 36 us (16384 rows of up to 512 scores,
// bound by instructions: 63% of issue slots), 140 us together.
#include <cstdint>

#include "internal.h"
#include "ops.cuh"

namespace bsattn {
namespace {

constexpr int kPoolThreads = 128;
constexpr int kSelThreads = 256;
constexpr int kSelWarps = kSelThreads / 32;
constexpr uint32_t kForced = 0xFFFFFFFFu;  // key of a block that is always kept
constexpr uint32_t kRuledOut = 0u;         // key of a block that never is

// One CTA per block: its rows' mean, rounded.  The blocks of Q come first
// (whole numbers t), then the blocks of K (t 2^(E - 6)).  A block is 8 to 32 KB
// in a row: it is copied to shared memory at once, each thread the pieces that
// it adds up itself, in two groups so that the first half is summed while the
// second arrives.
template <int D>
__global__ void __launch_bounds__(kPoolThreads)
    block_mean_kernel(const uint16_t* __restrict__ q, const uint16_t* __restrict__ k, int q_blocks,
                      int key_block, uint16_t* __restrict__ mq, uint16_t* __restrict__ mk) {
  extern __shared__ __align__(16) uint8_t block[];
  wait_for_previous_launch();
  const bool is_q = (int)blockIdx.x < q_blocks;
  const int64_t blk = is_q ? blockIdx.x : blockIdx.x - q_blocks;
  const int rows = is_q ? kBlock : key_block;
  const uint4* src = reinterpret_cast<const uint4*>((is_q ? q : k) + blk * rows * D) + threadIdx.x;
  const uint32_t dst = shared_address(block) + threadIdx.x * 16;
  const int pieces = rows * (D / 8) / kPoolThreads;  // a thread's: 4, 8 or 16
  Sum2x2 s[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) s[i].hi = s[i].lo = f2(0.0f);
  const int half = pieces / 2;
#pragma unroll 4
  for (int i = 0; i < half; ++i) copy16(dst + i * (kPoolThreads * 16), src + i * kPoolThreads);
  copy_commit();
#pragma unroll 4
  for (int i = half; i < pieces; ++i) copy16(dst + i * (kPoolThreads * 16), src + i * kPoolThreads);
  copy_commit();
  auto add = [&](int i) {
    const uint4 raw = lds128(dst + i * (kPoolThreads * 16));
    add_exact(s[0], bf16_pair(raw.x));
    add_exact(s[1], bf16_pair(raw.y));
    add_exact(s[2], bf16_pair(raw.z));
    add_exact(s[3], bf16_pair(raw.w));
  };
  copy_wait<1>();
#pragma unroll 2
  for (int i = 0; i < half; ++i) add(i);
  copy_wait<0>();
#pragma unroll 2
  for (int i = half; i < pieces; ++i) add(i);
  allow_next_launch();
  write_rounded_mean<D>(s, rows, is_q, (is_q ? mq : mk) + blk * D);
}

struct SelectParams {
  const uint16_t* mq;  // [B*H*nb][D]
  const uint16_t* mk;  // [B*Hkv*nk][D]
  const uint8_t* allow;  // [B][H or 1][nb][nk], null: all
  int64_t allow_b, allow_h;
  uint8_t* mask;  // [B][H][nb][nk]
  int H, Hkv, nb, nk, kdiv, kshift;  // kdiv = 1 << kshift key blocks a query block
  int keep, sink, local, causal;
  int rows;  // query blocks a CTA: 16, 8 or 4 (select_rows)
};

// A row of n keys held by one warp, four consecutive ones a lane and piece of
// 128.  KP > 0: in registers, KP a lane; KP = 0: in shared memory.  (Keys behind
// n are ruled out.)
template <int KP>
struct RowKeys {
  uint32_t k[KP > 0 ? KP : 1];
  const uint4* sh;
  int pieces, lane;

  __device__ __forceinline__ void load(const uint32_t* row, int n, int ln) {
    sh = reinterpret_cast<const uint4*>(row);
    pieces = (n + 127) / 128;
    lane = ln;
    if (KP > 0) {
#pragma unroll
      for (int i = 0; i < KP / 4; ++i) {
        const uint4 v = piece(i, n);
        k[4 * i] = v.x, k[4 * i + 1] = v.y, k[4 * i + 2] = v.z, k[4 * i + 3] = v.w;
      }
    }
  }
  __device__ __forceinline__ uint4 piece(int i, int n) const {
    return i * 128 + lane * 4 < n ? sh[i * 32 + lane] : make_uint4(0, 0, 0, 0);
  }

  template <typename F>
  __device__ __forceinline__ void each(int n, F f) const {
    if (KP > 0) {
#pragma unroll
      for (int i = 0; i < KP; ++i) f(k[i]);
    } else {
      for (int i = 0; i < pieces; ++i) {
        const uint4 v = piece(i, n);
        f(v.x), f(v.y), f(v.z), f(v.w);
      }
    }
  }
};

// Marks the best keys of a row: `keep` of them, or all that are forced if those
// are more.
template <int KP>
__device__ __forceinline__ void choose_row(const uint32_t* row, int n, int nk, int keep,
                                           uint8_t* out, int lane) {
  RowKeys<KP> keys;
  keys.load(row, n, lane);
  // counts in one word: forced << 16 | allowed (n <= 8192); largest and least
  // of the keys in between
  uint32_t counts = 0, top = 0, least = kForced;
  keys.each(n, [&](uint32_t x) {
    counts += (x != kRuledOut ? 1u : 0u) + (x == kForced ? 65536u : 0u);
    top = max(top, x == kForced ? 0u : x);
    least = min(least, x - 1u);  // 0 wraps: never the least
  });
  counts = __reduce_add_sync(0xFFFFFFFFu, counts);
  top = __reduce_max_sync(0xFFFFFFFFu, top);
  least = __reduce_min_sync(0xFFFFFFFFu, least) + 1u;
  const int allowed = counts & 0xFFFF, forced = counts >> 16;
  const int want = min(max(keep, forced), allowed);
  // `have` >= want keys are >= t
  uint32_t t = 1u;
  int have = allowed;
  if (want == forced) {
    t = kForced;
    have = forced;
  } else if (want < allowed) {
    KeySearch search(least, top, allowed, forced, want);
    while (search.open()) {
      const uint32_t c = search.probe();
      int cnt = 0;
      keys.each(n, [&](uint32_t x) { cnt += x >= c ? 1 : 0; });
      search.count(c, __reduce_add_sync(0xFFFFFFFFu, cnt));
    }
    t = search.t;
    have = search.have;
  }
  // more keys >= t than wanted: those equal to t go in from the left
  int drop_from = 0x7FFFFFFF;  // column from which keys equal to t stay out
  if (have != want) {
    int above = 0;
    keys.each(n, [&](uint32_t x) { above += x > t ? 1 : 0; });
    int ties = want - __reduce_add_sync(0xFFFFFFFFu, above);  // >= 1
    for (int i0 = 0; i0 < n; i0 += 32) {
      const unsigned eq = __ballot_sync(0xFFFFFFFFu, i0 + lane < n && row[i0 + lane] == t);
      if (__popc(eq) >= ties) {
        drop_from = i0 + __fns(eq, 0, ties) + 1;
        break;
      }
      ties -= __popc(eq);
    }
  }
  if (((nk | (int)reinterpret_cast<uintptr_t>(out)) & 3) == 0) {
    // (keys behind n read as ruled out, below any threshold)
    const uint32_t least_in = drop_from == 0x7FFFFFFF ? t : t + 1u;
    for (int i = 0; i * 128 + lane * 4 < nk; ++i) {
      const int col = i * 128 + lane * 4;
      const uint4 v = keys.piece(i, n);
      uint32_t in = (v.x >= least_in ? 1u : 0u) | (v.y >= least_in ? 0x100u : 0u) |
                    (v.z >= least_in ? 0x10000u : 0u) | (v.w >= least_in ? 0x1000000u : 0u);
      if (col < drop_from && least_in != t)
        in |= (v.x == t ? 1u : 0u) | (v.y == t && col + 1 < drop_from ? 0x100u : 0u) |
              (v.z == t && col + 2 < drop_from ? 0x10000u : 0u) |
              (v.w == t && col + 3 < drop_from ? 0x1000000u : 0u);
      *reinterpret_cast<uint32_t*>(out + col) = in;
    }
  } else {
    for (int i = lane; i < nk; i += 32) {
      const uint32_t x = i < n ? row[i] : kRuledOut;
      out[i] = x > t || (x == t && i < drop_from) ? 1 : 0;
    }
  }
}

// One CTA: `rows` query blocks of one head.  Each warp scores 8 key blocks at
// a time against all of them, then takes rows for the choice.
template <int D>
__global__ void __launch_bounds__(kSelThreads, 4) choose_blocks_kernel(const SelectParams p) {
  extern __shared__ __align__(16) uint32_t keys[];  // [rows][stride]
  constexpr int C = D / 32;           // 16-byte pieces a lane holds of a row
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int h = blockIdx.y, b = blockIdx.z;
  // the rows with the most key blocks in reach first
  const int q0 = (gridDim.x - 1 - blockIdx.x) * p.rows;
  const int rows = min(p.rows, p.nb - q0);
  const int stride = (p.nk + 3) & ~3;
  const int g = lane >> 2, j = lane & 3;
  // key blocks that the tile's last row can reach
  const int reach = p.causal ? min(p.nk, (q0 + rows) * p.kdiv) : p.nk;
  wait_for_previous_launch();

  // The channels are taken in the order that 16-byte loads bring them: lane
  // (g, j) holds 16-byte pieces 4c + j of row g, for A and B alike.
  uint4 a[2][C];
  const uint16_t* mq = p.mq + ((int64_t)(b * p.H + h) * p.nb + q0) * D;
#pragma unroll
  for (int r = 0; r < 2; ++r)
#pragma unroll
    for (int c = 0; c < C; ++c)
      a[r][c] = g + 8 * r < rows
                    ? __ldcg(reinterpret_cast<const uint4*>(mq + (g + 8 * r) * D) + 4 * c + j)
                    : make_uint4(0, 0, 0, 0);
  const uint16_t* mk = p.mk + (int64_t)(b * p.Hkv + h / (p.H / p.Hkv)) * p.nk * D;
  const uint8_t* allow =
      p.allow ? p.allow + b * p.allow_b + h * p.allow_h + (int64_t)q0 * p.nk : nullptr;
  for (int n0 = warp * 8; n0 < reach; n0 += kSelWarps * 8) {
    float acc[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    const int kb = min(n0 + g, p.nk - 1);
    uint4 w[C];
#pragma unroll
    for (int c = 0; c < C; ++c)
      w[c] = __ldcg(reinterpret_cast<const uint4*>(mk + (int64_t)kb * D) + 4 * c + j);
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const uint32_t a0[4] = {a[0][c].x, a[1][c].x, a[0][c].y, a[1][c].y};
      const uint32_t a1[4] = {a[0][c].z, a[1][c].z, a[0][c].w, a[1][c].w};
      mma_bf16(acc, a0, w[c].x, w[c].y);
      mma_bf16(acc, a1, w[c].z, w[c].w);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = g + 8 * (i >> 1), col = n0 + 2 * j + (i & 1);
      if (r < rows && col < reach) {
        const int q128 = q0 + r, k128 = col >> p.kshift;
        bool ok = !p.causal || k128 <= q128;
        if (allow) ok = ok && allow[(int64_t)r * p.nk + col] != 0;
        const bool must = col < p.sink || abs(k128 - q128) < p.local;
        keys[r * stride + col] = !ok ? kRuledOut : must ? kForced : ordered_bits(acc[i]);
      }
    }
  }
  __syncthreads();
  for (int r = warp; r < rows; r += kSelWarps) {
    const int n = p.causal ? min(p.nk, (q0 + r + 1) * p.kdiv) : p.nk;
    uint8_t* out = p.mask + (((int64_t)b * p.H + h) * p.nb + q0 + r) * p.nk;
    uint32_t* row = keys + r * stride;
    if (lane < ((4 - (n & 3)) & 3)) row[n + lane] = kRuledOut;  // to a whole piece of four
    __syncwarp();
    if (n <= 128)
      choose_row<4>(row, n, p.nk, p.keep, out, lane);
    else if (n <= 256)
      choose_row<8>(row, n, p.nk, p.keep, out, lane);
    else if (n <= 512)
      choose_row<16>(row, n, p.nk, p.keep, out, lane);
    else
      choose_row<0>(row, n, p.nk, p.keep, out, lane);
  }
}

// 16 query blocks a CTA (the tensor instruction's rows) while their keys fit
// 128 KB of shared memory, 4 above (4 rows of at most 8192 keys); 8, a row a warp,
// where tiles of 16 would leave SMs idle (8 heads of 4096 tokens: 11 us, with 16
// rows 13; 32 heads: 17 and 19; 4 x 32 heads: 39 and 40).
constexpr int kSelKeyBytes = 128 << 10;
int select_rows(int nk, int nb, int64_t heads, int sms) {
  if (16 * ((nk + 3) & ~3) * 4 > kSelKeyBytes) return 4;
  return (nb + 15) / 16 * heads <= sms ? kSelWarps : 16;
}

template <int D>
cudaError_t launch_select(const void* q, const void* k, int q_blocks, int k_blocks, int key_block,
                          uint16_t* mq, uint16_t* mk, const SelectParams& p, int B,
                          cudaStream_t st) {
  const size_t smem = (size_t)p.rows * ((p.nk + 3) & ~3) * sizeof(uint32_t);
  cudaError_t e = allow_shared_memory<choose_blocks_kernel<D>>(kSelKeyBytes);
  if (e != cudaSuccess) return e;
  e = launch_dependent(block_mean_kernel<D>, dim3(q_blocks + k_blocks), dim3(kPoolThreads),
                       (size_t)kBlock * D * 2, st, static_cast<const uint16_t*>(q),
                       static_cast<const uint16_t*>(k), q_blocks, key_block, mq, mk);
  if (e != cudaSuccess) return e;
  return launch_dependent(choose_blocks_kernel<D>, dim3((p.nb + p.rows - 1) / p.rows, p.H, B),
                          dim3(kSelThreads), smem, st, p);
}

bool select_sizes(int B, int H, int Hkv, int S, int D) {
  return B > 0 && H > 0 && Hkv > 0 && H % Hkv == 0 && S > 0 && S % kBlock == 0 &&
         (D == 64 || D == 128);
}

}  // namespace
}  // namespace bsattn

using namespace bsattn;

extern "C" {

size_t bsattn_select_blocks_workspace(int B, int H, int Hkv, int S, int D, unsigned flags) {
  if (!select_sizes(B, H, Hkv, S, D)) return 0;
  const int kdiv = (flags & BSATTN_KEY_BLOCK_64) ? 2 : 1;
  return ((size_t)B * H + (size_t)B * Hkv * kdiv) * (S / kBlock) * D * 2;
}

bsattn_status bsattn_select_blocks(const void* q, const void* k, int B, int H, int Hkv, int S,
                                   int D, int keep, int sink, int local, unsigned flags,
                                   const uint8_t* allow, int allow_heads, uint8_t* mask,
                                   void* workspace, size_t workspace_bytes, void* stream) {
  if (!q || !k || !mask || !workspace) return BSATTN_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(k) || !aligned16(workspace)) return BSATTN_ERR_INVALID_ARG;
  if (B <= 0 || H <= 0 || Hkv <= 0 || H % Hkv != 0 || S <= 0 || S % kBlock != 0)
    return BSATTN_ERR_INVALID_ARG;
  if (D != 64 && D != 128) return BSATTN_ERR_UNSUPPORTED;
  if (flags & ~(unsigned)(BSATTN_CAUSAL | BSATTN_KEY_BLOCK_64)) return BSATTN_ERR_INVALID_ARG;
  if (keep <= 0 || sink < 0 || local < 0) return BSATTN_ERR_INVALID_ARG;
  if (allow && allow_heads != 1 && allow_heads != H) return BSATTN_ERR_INVALID_ARG;
  const int nb = S / kBlock;
  if (nb > kMaxBlocksPerRow || (long long)B * H * S >= (1ll << 31) || H > 65535 || B > 65535)
    return BSATTN_ERR_UNSUPPORTED;
  if (workspace_bytes < bsattn_select_blocks_workspace(B, H, Hkv, S, D, flags))
    return BSATTN_ERR_INVALID_ARG;
  const int kdiv = (flags & BSATTN_KEY_BLOCK_64) ? 2 : 1;
  const int q_blocks = B * H * nb, k_blocks = B * Hkv * nb * kdiv;
  SelectParams p{};
  uint16_t* mq = static_cast<uint16_t*>(workspace);
  uint16_t* mk = mq + (size_t)q_blocks * D;
  p.mq = mq;
  p.mk = mk;
  p.allow = allow;
  p.nb = nb;
  p.nk = nb * kdiv;
  p.allow_h = allow_heads == H ? (int64_t)nb * p.nk : 0;
  p.allow_b = (int64_t)allow_heads * nb * p.nk;
  p.mask = mask;
  p.H = H;
  p.Hkv = Hkv;
  p.kdiv = kdiv;
  p.kshift = kdiv - 1;
  p.keep = keep;
  p.sink = sink;
  p.local = local;
  p.causal = (flags & BSATTN_CAUSAL) ? 1 : 0;
  int dev = -1;
  if (cudaGetDevice(&dev) != cudaSuccess) return BSATTN_ERR_CUDA;
  p.rows = select_rows(p.nk, nb, (int64_t)B * H, device_sm_count(dev));
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const int kb = kBlock / kdiv;
  return from_cuda(D == 64
                       ? launch_select<64>(q, k, q_blocks, k_blocks, kb, mq, mk, p, B, st)
                       : launch_select<128>(q, k, q_blocks, k_blocks, kb, mq, mk, p, B, st));
}

}  // extern "C"
