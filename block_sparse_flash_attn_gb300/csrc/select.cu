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
// are exact in bf16), the rows' k-th best is found by bisection over the
// scores' order-preserving bit patterns, held in registers.
#include <cstdint>

#include "internal.h"
#include "ops.cuh"

namespace bsattn {
namespace {

constexpr int kPoolThreads = 128;
constexpr int kPoolWarps = kPoolThreads / 32;
constexpr int kSelThreads = 256;
constexpr int kSelWarps = kSelThreads / 32;
constexpr uint32_t kForced = 0xFFFFFFFFu;  // key of a block that is always kept
constexpr uint32_t kRuledOut = 0u;         // key of a block that never is

// One CTA per block: its rows' mean, rounded.  The blocks of Q come first
// (whole numbers t), then the blocks of K (t 2^(E - 6)).
template <int D>
__global__ void __launch_bounds__(kPoolThreads)
    block_mean_kernel(const uint16_t* __restrict__ q, const uint16_t* __restrict__ k, int q_blocks,
                      int key_block, uint16_t* __restrict__ mq, uint16_t* __restrict__ mk) {
  constexpr int L = D / 8;
  constexpr int R = 32 / L;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const bool is_q = (int)blockIdx.x < q_blocks;
  const int64_t blk = is_q ? blockIdx.x : blockIdx.x - q_blocks;
  const int rows = is_q ? kBlock : key_block;
  const uint16_t* src = (is_q ? q : k) + blk * rows * D + (lane % L) * 8;

  Sum2x2 s[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) s[i].hi = s[i].lo = f2(0.0f);
  constexpr int U = 4;
  for (int r0 = warp * R + lane / L; r0 < rows; r0 += U * kPoolWarps * R) {
    uint4 raw[U];
#pragma unroll
    for (int u = 0; u < U; ++u)
      raw[u] = __ldg(reinterpret_cast<const uint4*>(src + (r0 + u * kPoolWarps * R) * D));
#pragma unroll
    for (int u = 0; u < U; ++u) {
      add_exact(s[0], bf16_pair(raw[u].x));
      add_exact(s[1], bf16_pair(raw[u].y));
      add_exact(s[2], bf16_pair(raw[u].z));
      add_exact(s[3], bf16_pair(raw[u].w));
    }
  }
  allow_next_launch();
  write_rounded_mean<D>(s, rows, is_q, (is_q ? mq : mk) + blk * D);
}

struct SelectParams {
  const uint16_t* mq;  // [B*H*nb][D]
  const uint16_t* mk;  // [B*Hkv*nk][D]
  const uint8_t* allow;  // [B][H or 1][nb][nk], null: all
  int64_t allow_b, allow_h;
  uint8_t* mask;  // [B][H][nb][nk]
  int H, Hkv, nb, nk, kdiv;
  int keep, sink, local, causal;
  int rows;  // query blocks a CTA: 16, or 4 when 16 rows of keys do not fit
};

// The k-th largest of a row of n keys held by one warp (key i*32 + lane), as
// (threshold, how many keys equal to it are taken, lowest index first).  KP >
// 0: in registers, KP a lane; KP = 0: in shared memory.
template <int KP>
struct RowKeys {
  uint32_t k[KP > 0 ? KP : 1];
  const uint32_t* sh;
  int n, lane;

  __device__ __forceinline__ void load(const uint32_t* row, int count, int ln) {
    sh = row;
    n = count;
    lane = ln;
    if (KP > 0) {
#pragma unroll
      for (int i = 0; i < KP; ++i) k[i] = i * 32 + lane < n ? row[i * 32 + lane] : kRuledOut;
    }
  }
  __device__ __forceinline__ int count_at_least(uint32_t t) const {
    int c = 0;
    if (KP > 0) {
#pragma unroll
      for (int i = 0; i < KP; ++i) c += k[i] >= t ? 1 : 0;
    } else {
      for (int i = lane; i < n; i += 32) c += sh[i] >= t ? 1 : 0;
    }
    return __reduce_add_sync(0xFFFFFFFFu, c);
  }
};

template <int KP>
__device__ __forceinline__ void choose_row(const uint32_t* row, int n, int nk, int keep,
                                           uint8_t* out, int lane) {
  RowKeys<KP> keys;
  keys.load(row, n, lane);
  const int allowed = keys.count_at_least(1u);
  const int forced = keys.count_at_least(kForced);
  const int want = min(max(keep, forced), allowed);
  // largest t with at least `want` keys >= t, bit by bit from the top
  uint32_t t = 1u;
  int above = allowed;
  if (want < allowed) {
    t = 0u;
    for (int bit = 31; bit >= 0; --bit) {
      const uint32_t c = t | (1u << bit);
      const int cnt = keys.count_at_least(c);
      if (cnt >= want) {
        t = c;
        above = cnt;
        if (cnt == want) break;
      }
    }
  }
  // keys > t all go in, and of those equal to t the first ones
  int ties = want - (above == want ? 0 : keys.count_at_least(t + 1u));
  if (above == want) ties = want;  // every key >= t: no border to settle
  const bool all = above == want;
  for (int i0 = 0; i0 < nk; i0 += 32) {
    const int i = i0 + lane;
    const uint32_t key = i < n ? row[i] : kRuledOut;
    const bool eq = key == t && !all;
    const unsigned eqs = __ballot_sync(0xFFFFFFFFu, eq);
    const bool take = (all ? key >= t : key > t) || (eq && __popc(eqs & ((1u << lane) - 1u)) < ties);
    ties -= __popc(eqs);
    if (i < nk) out[i] = take && key != kRuledOut ? 1 : 0;
  }
}

// One CTA: `rows` query blocks of one head.  Each warp scores 8 key blocks at
// a time against all of them, then takes rows for the choice.
template <int D>
__global__ void __launch_bounds__(kSelThreads) choose_blocks_kernel(const SelectParams p) {
  extern __shared__ uint32_t keys[];  // [rows][nk]
  constexpr int C = D / 32;           // 16-byte pieces a lane holds of a row
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int h = blockIdx.y, b = blockIdx.z;
  const int q0 = blockIdx.x * p.rows;
  const int rows = min(p.rows, p.nb - q0);
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
        const int q128 = q0 + r, k128 = col / p.kdiv;
        bool ok = !p.causal || k128 <= q128;
        if (allow) ok = ok && allow[(int64_t)r * p.nk + col] != 0;
        const bool must = col < p.sink || abs(k128 - q128) < p.local;
        keys[r * p.nk + col] = !ok ? kRuledOut : must ? kForced : ordered_bits(acc[i]);
      }
    }
  }
  __syncthreads();
  for (int r = warp; r < rows; r += kSelWarps) {
    const int n = p.causal ? min(p.nk, (q0 + r + 1) * p.kdiv) : p.nk;
    uint8_t* out = p.mask + (((int64_t)b * p.H + h) * p.nb + q0 + r) * p.nk;
    const uint32_t* row = keys + r * p.nk;
    if (n <= 128)
      choose_row<4>(row, n, p.nk, p.keep, out, lane);
    else if (n <= 512)
      choose_row<16>(row, n, p.nk, p.keep, out, lane);
    else
      choose_row<0>(row, n, p.nk, p.keep, out, lane);
  }
}

// 16 query blocks a CTA (the tensor instruction's rows) while their keys fit
// 128 KB of shared memory, 4 above (4 rows of at most 8192 keys).
constexpr int kSelKeyBytes = 128 << 10;
int select_rows(int nk) { return 16 * nk * 4 <= kSelKeyBytes ? 16 : 4; }

template <int D>
cudaError_t launch_select(const void* q, const void* k, int q_blocks, int k_blocks, int key_block,
                          uint16_t* mq, uint16_t* mk, const SelectParams& p, int B,
                          cudaStream_t st) {
  const size_t smem = (size_t)p.rows * p.nk * sizeof(uint32_t);
  cudaError_t e = cudaSuccess;
  if (smem > (48 << 10)) {
    e = cudaFuncSetAttribute(choose_blocks_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             kSelKeyBytes);
    if (e != cudaSuccess) return e;
  }
  block_mean_kernel<D><<<q_blocks + k_blocks, kPoolThreads, 0, st>>>(
      static_cast<const uint16_t*>(q), static_cast<const uint16_t*>(k), q_blocks, key_block, mq,
      mk);
  e = cudaGetLastError();
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
  p.keep = keep;
  p.sink = sink;
  p.local = local;
  p.causal = (flags & BSATTN_CAUSAL) ? 1 : 0;
  p.rows = select_rows(p.nk);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const int kb = kBlock / kdiv;
  return from_cuda(D == 64
                       ? launch_select<64>(q, k, q_blocks, k_blocks, kb, mq, mk, p, B, st)
                       : launch_select<128>(q, k, q_blocks, k_blocks, kb, mq, mk, p, B, st));
}

}  // extern "C"
