// Small device helpers shared by the operators around the attention kernels
// (rope.cu, select.cu, kv4.cu, kv4_attn.cu): bf16 packing, launches, pairs of
// floats, exact sums, block floating point, threshold search, matrix products.
#pragma once

#include <atomic>
#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

namespace bsattn {

constexpr float kLn2 = 0.6931471805599453f;

// two bf16 of a 32-bit word, the lower half first
__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

__device__ __forceinline__ void unpack8(const uint4& v, float (&f)[8]) {
  f[0] = bf16_lo(v.x), f[1] = bf16_hi(v.x), f[2] = bf16_lo(v.y), f[3] = bf16_hi(v.y);
  f[4] = bf16_lo(v.z), f[5] = bf16_hi(v.z), f[6] = bf16_lo(v.w), f[7] = bf16_hi(v.w);
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<uint32_t*>(&h);
}

// Lets a kernel have `bytes` of dynamic shared memory; asks once a device.
template <auto Kernel>
inline cudaError_t allow_shared_memory(int bytes) {
  static std::atomic<int> allowed[64];
  int dev = -1;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess || (dev < 64 && allowed[dev].load(std::memory_order_relaxed) >= bytes))
    return e;
  e = cudaFuncSetAttribute(Kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess && dev < 64) allowed[dev].store(bytes, std::memory_order_relaxed);
  return e;
}

// ---------------------------------------------------------------------------
// Asynchronous copies of 16 bytes into shared memory: bytes in flight that
// hold no registers.
// ---------------------------------------------------------------------------
__device__ __forceinline__ void copy16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ uint4 lds128(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(a));
  return v;
}
__device__ __forceinline__ uint32_t shared_address(const void* p) {
  return static_cast<uint32_t>(__cvta_generic_to_shared(p));
}

// ---------------------------------------------------------------------------
// Two 32-bit floats a register pair: sm_103a adds, multiplies and fuses both
// with one instruction, each rounded as the single instruction rounds.
// ---------------------------------------------------------------------------
struct F2 {
  float2 v;
};
__device__ __forceinline__ F2 f2(float lo, float hi) { return F2{make_float2(lo, hi)}; }
__device__ __forceinline__ F2 f2(float both) { return f2(both, both); }
__device__ __forceinline__ float2 split(F2 a) { return a.v; }
__device__ __forceinline__ F2 operator+(F2 a, F2 b) { return F2{__fadd2_rn(a.v, b.v)}; }
__device__ __forceinline__ F2 operator*(F2 a, F2 b) { return F2{__fmul2_rn(a.v, b.v)}; }
__device__ __forceinline__ F2 fma2(F2 a, F2 b, F2 c) { return F2{__ffma2_rn(a.v, b.v, c.v)}; }
__device__ __forceinline__ F2 bf16_pair(uint32_t w) { return f2(bf16_lo(w), bf16_hi(w)); }
__device__ __forceinline__ uint32_t pack_bf16(F2 a) {
  const float2 s = split(a);
  return pack_bf16(s.x, s.y);
}

// A programmatic dependent waits here for the launch before it (griddepcontrol
// is a no-op in a kernel launched without the attribute).
__device__ __forceinline__ void wait_for_previous_launch() {
  asm volatile("griddepcontrol.wait;" ::: "memory");
}
__device__ __forceinline__ void allow_next_launch() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

// An ordinary load, and no read-only one (ld.global.nc): a kernel launched early
// lives while the launch before it still writes, and the gradient of
// qk_norm_rope may be written over its input; the read-only path is for data
// that nothing writes during the kernel's life.
template <typename T>
__device__ __forceinline__ T load(const T* p) {
  return *p;
}

// Launch with programmatic stream serialisation: the kernel may start while
// the one before it in the stream drains, and waits for it itself.
template <typename... KArgs, typename... Args>
inline cudaError_t launch_dependent(void (*kernel)(KArgs...), dim3 grid, dim3 block, size_t smem,
                                    cudaStream_t stream, Args... args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, KArgs(args)...);
}

// The same in clusters of `cluster` CTAs (along x).
template <typename... KArgs, typename... Args>
inline cudaError_t launch_dependent_clusters(void (*kernel)(KArgs...), dim3 grid, dim3 block,
                                             int cluster, size_t smem, cudaStream_t stream,
                                             Args... args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = cluster;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kernel, KArgs(args)...);
}

// ---------------------------------------------------------------------------
// Exact sums of bf16 (or 32-bit) values: hi + lo with lo the exact error of
// hi (Knuth's two-sum), about 48 bits in all.
// ---------------------------------------------------------------------------
struct Sum2 {
  float hi, lo;
};

__device__ __forceinline__ void add_exact(Sum2& s, float x) {
  const float t = __fadd_rn(s.hi, x);
  const float z = __fadd_rn(t, -s.hi);
  const float e = __fadd_rn(__fadd_rn(s.hi, -__fadd_rn(t, -z)), __fadd_rn(x, -z));
  s.hi = t;
  s.lo = __fadd_rn(s.lo, e);
}

// The same for two sums at once; a - b is taken as fma(b, -1, a), exact alike.
struct Sum2x2 {
  F2 hi, lo;
};

__device__ __forceinline__ void add_exact(Sum2x2& s, F2 x) {
  const F2 neg = f2(-1.0f);
  const F2 t = s.hi + x;
  const F2 z = fma2(s.hi, neg, t);
  const F2 e = fma2(fma2(z, neg, t), neg, s.hi) + fma2(z, neg, x);
  s.hi = t;
  s.lo = s.lo + e;
}

__device__ __forceinline__ void add_exact(Sum2& s, const Sum2& o) {
  add_exact(s, o.hi);
  s.lo = __fadd_rn(s.lo, o.lo);
}

__device__ __forceinline__ void add_exact(Sum2x2& s, const Sum2x2& o) {
  add_exact(s, o.hi);
  s.lo = s.lo + o.lo;
}

// the sums of the lane `o` places away
__device__ __forceinline__ Sum2x2 exchanged(const Sum2x2& s, int o) {
  const float2 hi = split(s.hi), lo = split(s.lo);
  constexpr unsigned all = 0xFFFFFFFFu;
  return Sum2x2{f2(__shfl_xor_sync(all, hi.x, o), __shfl_xor_sync(all, hi.y, o)),
                f2(__shfl_xor_sync(all, lo.x, o), __shfl_xor_sync(all, lo.y, o))};
}

// hi takes everything it can hold: |lo| <= half a step of hi
__device__ __forceinline__ Sum2 renormalised(const Sum2& s) {
  Sum2 r{s.hi, 0.0f};
  add_exact(r, s.lo);
  return r;
}

// floor(log2 |hi + lo|) of a renormalised sum; a very low number for zero and
// for a sum that is not finite (both count as zero).
constexpr int kNoExponent = -100000;
__device__ __forceinline__ int exponent_of(const Sum2& s) {
  const float a = fabsf(s.hi);
  if (!(a > 0.0f) || !(a <= 3.0e38f)) return kNoExponent;
  int e = ilogbf(a);
  // a power of two with a negative rest lies just below it
  const bool pow2 = a == ldexpf(1.0f, e);
  if (pow2 && (s.hi > 0.0f ? s.lo < 0.0f : s.lo > 0.0f)) e -= 1;
  return e;
}

// rint((hi + lo) * 2^shift), half to even, exactly: a whole number of at most
// 8 bits (the caller's shift puts the largest below 2^7).
__device__ __forceinline__ float rint_scaled(const Sum2& s, int shift) {
  const float h = ldexpf(s.hi, shift);
  if (!(fabsf(h) <= 256.0f)) return 0.0f;  // not finite: counts as zero
  float n = rintf(h);
  const float r = h - n;  // exact
  // hi lies on a border: the sign of lo says which side the sum is on
  if (r == 0.5f && s.lo > 0.0f) n += 1.0f;
  if (r == -0.5f && s.lo < 0.0f) n -= 1.0f;
  return n;
}

// Sums of a warp's rows, which lie O lanes apart: of two lanes each passes half
// of its HELD sums on and adds up the other half.
template <int O, int HELD, int N>
__device__ __forceinline__ void add_over_rows(Sum2x2 (&s)[N], int& first) {
  if constexpr (O < 32) {
    constexpr int kHalf = HELD / 2;
    const bool upper = (threadIdx.x & O) != 0;
    first += upper ? kHalf : 0;
#pragma unroll
    for (int i = 0; i < kHalf; ++i) {
      const Sum2x2 low = s[i], high = s[i + kHalf];
      s[i] = upper ? high : low;
      add_exact(s[i], exchanged(upper ? low : high, O));
    }
    add_over_rows<2 * O, kHalf>(s, first);
  }
}

// The mean of `rows` rows of a block (rows a power of two), rounded to 7 bits
// beside its largest entry, by a CTA of 128 threads: a row is held by D / (2 N)
// lanes, pairs[i] are this thread's sums of channels (lane % L) * 2N + 2i and
// 2i + 1 over the rows that it saw.  Writes, as bf16, the whole numbers t =
// rint(mean 2^(6 - E)) or the values t 2^(E - 6).
template <int D, int N>
__device__ __forceinline__ void write_rounded_mean(const Sum2x2 (&pairs)[N], int rows, bool whole,
                                                   uint16_t* out) {
  constexpr int L = D / (2 * N), W = 4;
  __shared__ __align__(16) Sum2 part[W][D];
  __shared__ int top[W];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  Sum2x2 s[N];
#pragma unroll
  for (int i = 0; i < N; ++i) s[i] = pairs[i];
  int first = lane % L * N;  // the first pair that this lane still holds
  add_over_rows<L, N>(s, first);
#pragma unroll
  for (int i = 0; i < N * L / 32; ++i) {
    const float2 hi = split(s[i].hi), lo = split(s[i].lo);
    *reinterpret_cast<float4*>(&part[warp][2 * (first + i)]) = make_float4(hi.x, lo.x, hi.y, lo.y);
  }
  __syncthreads();
  const int c = threadIdx.x;
  Sum2 t{0.0f, 0.0f};
  int e = kNoExponent;
  if (c < D) {
#pragma unroll
    for (int w = 0; w < W; ++w) add_exact(t, part[w][c]);
    t = renormalised(t);
    e = exponent_of(t);
  }
  e = __reduce_max_sync(0xFFFFFFFFu, e);
  if (lane == 0) top[warp] = e;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < W; ++w) e = max(e, top[w]);
  if (c < D) {
    // the mean's exponent is e - log2(rows): t = rint(sum 2^(6 - e))
    const bool none = e == kNoExponent;
    const float n = none ? 0.0f : rint_scaled(t, 6 - e);
    const int shift = none || whole ? 0 : e - 6 - (31 - __clz(rows));
    out[c] = (uint16_t)(__float_as_uint(ldexpf(n, shift)) >> 16);
  }
}

// Order-preserving map of a finite float to uint32 (larger float, larger
// number; 0 and 0xFFFFFFFF are not images of a finite float).
__device__ __forceinline__ uint32_t ordered_bits(float x) {
  const uint32_t u = __float_as_uint(x + 0.0f);  // -0 becomes +0
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

// 32 bytes to global memory, in one store where they are aligned to 32
__device__ __forceinline__ void store32(void* dst, const uint32_t (&v)[8], bool wide) {
  if (wide) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(dst), "r"(v[0]),
                 "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
                 : "memory");
  } else {
    static_cast<uint4*>(dst)[0] = make_uint4(v[0], v[1], v[2], v[3]);
    static_cast<uint4*>(dst)[1] = make_uint4(v[4], v[5], v[6], v[7]);
  }
}

__device__ __forceinline__ float from_ordered_bits(uint32_t u) {
  return __uint_as_float((u & 0x80000000u) ? u ^ 0x80000000u : ~u);
}

__device__ __forceinline__ float log2_fast(float x) {
  float y;
  asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Search for a threshold t among ordered keys with exactly `want` keys >= t,
// or, where equal keys leave none, for the want-th largest key.  Each step
// probes between a key with too many at or above it (t, `have`) and one with too
// few (hi, `over`), by interpolating the logarithm of the count between the two
// scores: a linear tail of that is what scores have (5 to 8 steps for 768 or
// 512 of them, against 9 by halving and up to 35 by interpolating the count).
// An end that stays put twice counts half (the Illinois rule), and from the
// thirteenth step on every other one halves the interval of bit patterns, so
// that 76 steps always end it.
struct KeySearch {
  uint32_t t, hi;
  int have, over, want, step, last;
  float goal, at_t, at_hi;

  // keys between least and top; `all` keys >= least, `more` of them above top
  __device__ __forceinline__ KeySearch(uint32_t least, uint32_t top, int all, int more, int n)
      : t(least), hi(top + 1u), have(all), over(more), want(n), step(0), last(0),
        goal(log2_fast((float)n)), at_t(1.0f), at_hi(1.0f) {}
  __device__ __forceinline__ bool open() const { return have != want && hi - t > 1u; }
  __device__ __forceinline__ uint32_t probe() {
    uint32_t c = t + (hi - t) / 2u;
    if (step < 12 || (step & 1)) {
      const float low = from_ordered_bits(t), high = from_ordered_bits(hi - 1u);
      const float a = (log2_fast((float)have + 0.5f) - goal) * at_t;
      const float b = (goal - log2_fast((float)over + 0.5f)) * at_hi;
      c = ordered_bits(fmaf(high - low, __fdividef(a, a + b), low));
    }
    ++step;
    return min(max(c, t + 1u), hi - 1u);
  }
  __device__ __forceinline__ void count(uint32_t c, int n) {
    if (n >= want) {
      t = c, have = n, at_t = 1.0f;
      if (last > 0) at_hi *= 0.5f;
      last = 1;
    } else {
      hi = c, over = n, at_hi = 1.0f;
      if (last < 0) at_t *= 0.5f;
      last = -1;
    }
  }
};

// D += A B, 16 x 8 x 16: bf16 in, 32-bit sums (A row-major, B column-major)
__device__ __forceinline__ void mma_bf16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0,
                                         uint32_t b1) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ void mma_f16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0,
                                        uint32_t b1) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

}  // namespace bsattn
