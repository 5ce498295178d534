// Kernels of the operators between a gradient sync and the next forward
// ("PyTorch DDP Deep Dive", Part 2: after finalize_backward every rank's
// optimizer applies the same update to the same averaged gradients): the
// global norm of a gradient set, the clipped gradients, the AdamW update.
// All three stream their operands and are bound by HBM from a few tens of MB
// on, and by the latency of a launch and its dependent reads below.
#include <math.h>

#include "launch.h"
#include "optim.cuh"

namespace ddp {
namespace {

// ------------------------------------------------------------- 32 bytes
// The widest access of a thread: eight 32-bit words, one whole 32-byte sector.
// Writing a sector as two 16-byte stores leaves it half written in between:
// scaling the ResNet-50-shaped fp32 set into 8 replicas took 201-209 us that
// way and 137 us with one store (920 MB, 6.7 TB/s).
// L1 is not filled: nothing is read twice by a block, and the tile tables stay there.
struct Words {
  uint32_t w[8];
};
__device__ __forceinline__ Words load32(const void* at) {
  Words x;
  asm volatile("ld.global.L1::no_allocate.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=r"(x.w[0]), "=r"(x.w[1]), "=r"(x.w[2]), "=r"(x.w[3]), "=r"(x.w[4]), "=r"(x.w[5]), "=r"(x.w[6]),
                 "=r"(x.w[7])
               : "l"(at));
  return x;
}
__device__ __forceinline__ void store32(void* at, const Words& x) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(at), "r"(x.w[0]), "r"(x.w[1]),
               "r"(x.w[2]), "r"(x.w[3]), "r"(x.w[4]), "r"(x.w[5]), "r"(x.w[6]), "r"(x.w[7]));
}
__device__ __forceinline__ uint4 load16(const void* at) {
  uint4 v;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(at));
  return v;
}

template <typename T> constexpr int kVec32 = 32 / sizeof(T);
// Words as fp32 elements.
__device__ __forceinline__ void unpack(const Words& x, float* f, float) {
#pragma unroll
  for (int l = 0; l < 8; ++l) f[l] = __uint_as_float(x.w[l]);
}
__device__ __forceinline__ void unpack(const Words& x, float* f, __nv_bfloat16) {
#pragma unroll
  for (int l = 0; l < 8; ++l) Vec<__nv_bfloat16>::unpack2(x.w[l], f + 2 * l);
}
__device__ __forceinline__ Words pack(const float* f, float) {
  Words x;
#pragma unroll
  for (int l = 0; l < 8; ++l) x.w[l] = __float_as_uint(f[l]);
  return x;
}
__device__ __forceinline__ Words pack(const float* f, __nv_bfloat16) {
  Words x;
#pragma unroll
  for (int l = 0; l < 8; ++l) x.w[l] = Vec<__nv_bfloat16>::pack2(f[2 * l], f[2 * l + 1]);
  return x;
}

// ------------------------------------------------------------- 8-vectors
// Eight consecutive elements as fp32, at an 8-element aligned address.
__device__ __forceinline__ void load8(const float* at, float* f) {
  const Words x = load32(at);
#pragma unroll
  for (int l = 0; l < 8; ++l) f[l] = __uint_as_float(x.w[l]);
}
__device__ __forceinline__ void load8(const __nv_bfloat16* at, float* f) {
  Vec<__nv_bfloat16>::unpack(load16(at), f);
}
__device__ __forceinline__ void store8(float* at, const float* f) {
  Words x;
#pragma unroll
  for (int l = 0; l < 8; ++l) x.w[l] = __float_as_uint(f[l]);
  store32(at, x);
}
__device__ __forceinline__ void store8(__nv_bfloat16* at, const float* f) {
  *reinterpret_cast<uint4*>(at) = Vec<__nv_bfloat16>::pack(f);
}

// V consecutive elements at any address: a gradient that is a view at an odd
// offset of a flat bucket, while the other streams keep their vectors. Lanes
// overlap in the lines they read, so these loads do fill L1. ResNet-50-shaped
// set, 8 replicas, aligned gradients and misaligned ones: update 210.6 and 211.1
// us in fp32, 143.0 and 143.5 in bf16 (297.8 in fp32 with every stream element by
// element), clip 161.0 and 161.6, in bf16 85.3 and 87.8.
template <int V, typename T>
__device__ __forceinline__ void load_each(const T* at, float* f) {
#pragma unroll
  for (int l = 0; l < V; ++l) f[l] = widen(at[l]);
}

// --------------------------------------------------------- ragged tiles
// The part of a tile of E elements from x0 that lies in a tensor of n: [lo, hi),
// counted from x0. All of it in a tensor's inner tiles.
struct Part {
  int lo, hi;
};
__device__ __forceinline__ Part part_of(int64_t x0, int64_t n, int E) {
  return {x0 < 0 ? static_cast<int>(-x0) : 0, n - x0 < E ? static_cast<int>(n - x0) : E};
}
// Elements of the part that no whole V-vector of the tile covers: fewer than V
// at either end, one for each lane of a warp (the start's on lanes 0-15, the
// end's on 16-31); -1 for a lane without one.
template <int V>
__device__ __forceinline__ int edge_element(const Part& t, int lane) {
  static_assert(V <= 16, "two edges share the lanes of a warp");
  const int a = (t.lo + V - 1) / V * V, b = t.hi / V * V;  // whole vectors: [a, b)
  const int e = lane < 16 ? t.lo + lane : max(a, b) + lane - 16;
  return e < (lane < 16 ? min(a, t.hi) : t.hi) ? e : -1;
}

// The tensor that tile b belongs to: the last j with tile0[j] <= b (tile0 does
// not decrease, tile0[0] = 0, tile0[k] > b). Each warp searches on its own, 32
// probes a round: the lanes whose probe is <= b form a prefix, and a table of
// up to 1,024 tensors takes two dependent reads, of lines that stay in L1.
// Against a table of every tile's tensor, one read from L2: update of the Llama-1B-shaped
// set 5,806-5,828 -> 5,790 us, of 3,000 small tensors 13.7 -> 12.1 us, the rest even.
__device__ __forceinline__ int32_t tensor_of_tile(const int32_t* tile0, int32_t k, int32_t b) {
  const int lane = threadIdx.x & 31;
  int lo = 0, hi = k;  // tile0[lo] <= b < tile0[hi]
  while (hi - lo > 1) {
    const int step = (hi - lo + 31) >> 5;  // probes at lo + step, lo + 2 step, ..., below hi
    const int q = lo + step * (lane + 1);
    const int c = __popc(__ballot_sync(0xffffffffu, q < hi && tile0[q] <= b));
    hi = min(hi, lo + step * (c + 1));
    lo += step * c;
  }
  return lo;
}

// ------------------------------------------------------------------ norm
template <typename T> constexpr int kNormTile = kNormTileBytes / sizeof(T);
constexpr int kNormBlocksPerSm = 4;
constexpr int kNormLoads = kNormTileBytes / (32 * kNormThreads);

// Sum of squares of N values as fp64. The fp32 sum is exact to a few ulp while
// it lies in [2^-96, 2^96]; outside (squares may have underflowed, or
// overflowed) the values are squared again scaled by a power of two, so that
// every finite input gives the true norm. Infinities and NaN come out of the
// scaled form as they are.
template <int N>
__device__ __forceinline__ double sum_squares(const float* f) {
  float s = 0.0f;
#pragma unroll
  for (int l = 0; l < N; ++l) s = fmaf(f[l], f[l], s);
  if (s >= 0x1p-96f && s <= 0x1p96f) return static_cast<double>(s);
  const float up = s < 1.0f ? 0x1p96f : 0x1p-96f;  // NaN and infinity take the second
  s = 0.0f;
#pragma unroll
  for (int l = 0; l < N; ++l) {
    const float y = f[l] * up;
    s = fmaf(y, y, s);
  }
  return s == 0.0f ? 0.0 : static_cast<double>(s) * (up > 1.0f ? 0x1p-192 : 0x1p192);
}

// Sum of a warp's 32 non-negative doubles, the same for every lane. GB300's
// fp64 rate is a small fraction of its fp32 rate, so the lanes are added as
// integers: their 53-bit significands aligned to the largest exponent, in two
// halves (26 and 27 bits) whose sums over 32 lanes fit 32 bits. What the
// alignment cuts off is below 32 * 2^-52 of the largest. Sums of squares are
// zero, normal (2^-298 and up), infinite or NaN, never subnormal. Against five
// rounds of shuffled fp64 additions: norm of 1.1 MB in ten tensors 4.9 -> 4.0
// us, norms of each of 572 small tensors 19.1 -> 9.4 us.
__device__ __forceinline__ double warp_sum(double a) {
  const uint64_t bits = static_cast<uint64_t>(__double_as_longlong(a));
  const unsigned e = static_cast<unsigned>(bits >> 52) & 0x7FFu, top = __reduce_max_sync(0xffffffffu, e);
  if (top == 0x7FFu) {  // infinity or NaN somewhere
    const bool nan = __any_sync(0xffffffffu, e == top && (bits << 12) != 0);
    return __longlong_as_double(nan ? 0x7FF8000000000000LL : 0x7FF0000000000000LL);
  }
  if (top == 0) return 0.0;
  const unsigned shift = top - e;
  const uint64_t m = e != 0 && shift < 64 ? ((bits & 0xFFFFFFFFFFFFFull) | 0x10000000000000ull) >> shift : 0;
  const uint64_t lo = __reduce_add_sync(0xffffffffu, static_cast<unsigned>(m & 0x3FFFFFFu));
  const uint64_t hi = __reduce_add_sync(0xffffffffu, static_cast<unsigned>(m >> 26));
  // m counts units of 2^(top - 1075)
  const long long sum = __double_as_longlong(static_cast<double>(lo + (hi << 26)));
  return __longlong_as_double(sum + (static_cast<long long>(static_cast<int>(top) - 1075) << 52));
}

// Square root of a non-negative double, to fp32: s = m * 4^q with m in [1, 4), root(s) = root(m) * 2^q.
__device__ __forceinline__ float root(double s) {
  const long long bits = __double_as_longlong(s);
  const int e = static_cast<int>(bits >> 52);
  if (e == 0 || e == 0x7FF) return static_cast<float>(s);
  const int q = (e - 1023) >> 1;
  const float m = static_cast<float>(__longlong_as_double(bits - (static_cast<long long>(2 * q) << 52)));
  return ldexpf(__fsqrt_rn(m), q);
}

// |x| as bits: ordered as the magnitudes are, with NaN above infinity.
__device__ __forceinline__ uint32_t magnitude(float x) { return __float_as_uint(x) & 0x7FFFFFFFu; }

// The two norms' folds: a sum in fp64, or the largest magnitude (its bits,
// held in the low half of a double's place).
template <bool INF> struct Fold;
template <> struct Fold<false> {
  using A = double;
  __device__ __forceinline__ static A zero() { return 0.0; }
  __device__ __forceinline__ static A join(A a, A b) { return a + b; }
  __device__ __forceinline__ static A warp(A a) { return warp_sum(a); }
  template <int N> __device__ __forceinline__ static A of(const float* f) { return sum_squares<N>(f); }
  __device__ __forceinline__ static float finish(A a) { return root(a); }
  __device__ __forceinline__ static double pack(A a) { return a; }
  __device__ __forceinline__ static A unpack(double d) { return d; }
};
template <> struct Fold<true> {
  using A = uint32_t;
  __device__ __forceinline__ static A zero() { return 0u; }
  __device__ __forceinline__ static A join(A a, A b) { return max(a, b); }
  __device__ __forceinline__ static A warp(A a) { return __reduce_max_sync(0xffffffffu, a); }
  template <int N> __device__ __forceinline__ static A of(const float* f) {
    uint32_t m = 0;
#pragma unroll
    for (int l = 0; l < N; ++l) m = max(m, magnitude(f[l]));
    return m;
  }
  __device__ __forceinline__ static float finish(A a) { return __uint_as_float(a); }
  __device__ __forceinline__ static double pack(A a) { return __longlong_as_double(static_cast<long long>(a)); }
  __device__ __forceinline__ static A unpack(double d) { return static_cast<uint32_t>(__double_as_longlong(d)); }
};

// Fold over the block in a fixed order; the result is warp 0's.
template <bool INF>
__device__ __forceinline__ typename Fold<INF>::A block_fold(typename Fold<INF>::A a) {
  using F = Fold<INF>;
  __shared__ typename F::A part[kNormThreads / 32];
  a = F::warp(a);
  __syncthreads();  // an earlier fold's parts have been read
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = a;
  __syncthreads();
  if (threadIdx.x < 32) a = F::warp(threadIdx.x < kNormThreads / 32 ? part[threadIdx.x] : F::zero());
  return a;
}

// Block b takes the tiles [first_tile(b), first_tile(b + 1)) of ntiles.
__device__ __forceinline__ int32_t first_tile(int32_t ntiles, int32_t blocks, int32_t b) {
  return static_cast<int32_t>(static_cast<int64_t>(ntiles) * b / blocks);
}
// The block that takes tile i: the last b with ntiles * b / blocks < i + 1.
__device__ __forceinline__ int32_t block_of_tile(int32_t ntiles, int32_t blocks, int32_t i) {
  return static_cast<int32_t>((static_cast<int64_t>(i + 1) * blocks - 1) / ntiles);
}

// One pass over the gradients, 2 flops an element, bound by HBM. Each block
// walks consecutive tiles, so that a tensor's end is the only place where its
// own sum has to be folded, with the next tile's loads in flight while the
// present one is summed. Measured on the ResNet-50-shaped fp32 (102 MB) and the
// Llama-1B-shaped bf16 set (2.4 GB): 20.3 and 333-337 us (7.2 TB/s, 1.06 of the
// measured copy rate); blocks striding over the tiles 24.8 and 358 us, and with
// no loads ahead 27.4 and 386; 8 KB tiles at 6 or 8 blocks per SM 24-25 and
// 350-383 us; 3 blocks per SM 22.4 and 348. At 4 the bf16 sum of squares fills
// its 64 registers and spills 4 bytes (20 with EACH), at 5 up to 114; the other
// forms spill nothing at 4. Tiles handed out from a counter for the last 10-50 %
// of the set change nothing (22.4-23.5 and 333-336 against 22.9 and 338); that
// was not tried on sets of many ragged tiles, where blocks of equal tile counts
// differ by up to a quarter in bytes from their mean.
template <typename T, bool INF, bool EACH>
__global__ void __launch_bounds__(kNormThreads, kNormBlocksPerSm)
    k_optim_norm(const OptimTable t, const OptimWork w, float* norm) {
  using F = Fold<INF>;
  constexpr int V = kVec32<T>;
  struct Span {
    const T* g;  // of the tile's first element, which may lie before the tensor
    Part part;
    int32_t tensor;
  };
  struct Data {
    Words x[kNormLoads];
    float edge;
    bool some;  // of x comes from the tensor
  };
  int32_t tensor = 0, first = 0, end = 0;  // the tensor of the tile last located, and its tiles
  auto locate = [&](int32_t i) -> Span {
    while (i >= end) {
      ++tensor;
      first = end;
      end = t.tile0[tensor + 1];
    }
    const OptimTensor& r = t.tensors[tensor];
    const int64_t x0 = static_cast<int64_t>(i - first) * kNormTile<T> - r.f;
    return {static_cast<const T*>(r.grad) + x0, part_of(x0, r.n, kNormTile<T>), tensor};
  };
  auto load = [&](const Span& s, Data& d) {
    d.edge = 0.0f;
    d.some = true;
    if (s.part.lo == 0 && s.part.hi == kNormTile<T>) {
#pragma unroll
      for (int j = 0; j < kNormLoads; ++j) d.x[j] = load32(s.g + (threadIdx.x + j * kNormThreads) * V);
    } else {
      d.some = false;
#pragma unroll
      for (int j = 0; j < kNormLoads; ++j) {
        const int at = (threadIdx.x + j * kNormThreads) * V;
        const bool whole = at >= s.part.lo && at + V <= s.part.hi;
        d.x[j] = whole ? load32(s.g + at) : Words{};
        d.some |= whole;
      }
      if (threadIdx.x < 32) {
        const int e = edge_element<V>(s.part, threadIdx.x);
        if (e >= 0) d.edge = widen(s.g[e]);
      }
    }
  };
  pdl_trigger();
  typename F::A acc = F::zero(), part = F::zero();
  int32_t i = first_tile(t.ntiles, gridDim.x, blockIdx.x);
  const int32_t hi = first_tile(t.ntiles, gridDim.x, blockIdx.x + 1);
  Span at{};
  if (i < hi) {  // the tables are static: read while an earlier kernel drains
    tensor = tensor_of_tile(t.tile0, t.k, i);
    first = t.tile0[tensor];
    end = t.tile0[tensor + 1];
    at = locate(i);
  }
  pdl_wait();
  Data x;
  if (i < hi) load(at, x);
  for (; i < hi; ++i) {
    Data next;
    Span after{};
    after.tensor = -1;
    if (i + 1 < hi) {
      after = locate(i + 1);
      load(after, next);
    }
    typename F::A a = F::zero();
    if (x.some) {
      float f[kNormLoads * V];
#pragma unroll
      for (int j = 0; j < kNormLoads; ++j) unpack(x.x[j], f + j * V, T());
      a = F::template of<kNormLoads * V>(f);
    }
    if (x.edge != 0.0f) a = F::join(a, F::template of<1>(&x.edge));
    acc = F::join(acc, a);
    if (EACH) {
      part = F::join(part, a);
      if (after.tensor != at.tensor) {
        part = block_fold<INF>(part);
        if (threadIdx.x == 0) w.part_sum[blockIdx.x + at.tensor] = F::pack(part);
        part = F::zero();
      }
    }
    at = after;
    x = next;
  }
  acc = block_fold<INF>(acc);

  // The block that finishes last joins the blocks' sums, in their order.
  __shared__ bool last;
  if (threadIdx.x == 0) {
    w.block_sum[blockIdx.x] = F::pack(acc);
    __threadfence();
    last = atomicAdd(&w.ticket[0], 1u) == gridDim.x - 1;
  }
  __syncthreads();
  if (!last) return;
  __threadfence();
  acc = F::zero();
  for (unsigned b = threadIdx.x; b < gridDim.x; b += kNormThreads)
    acc = F::join(acc, F::unpack(__ldcg(&w.block_sum[b])));
  acc = block_fold<INF>(acc);
  if (threadIdx.x == 0) {
    *norm = F::finish(acc);
    w.ticket[0] = 0;
  }
}

// One warp per tensor joins its blocks' parts: 4 us more than the norm alone on
// the GPT-2-shaped set's 148 tensors (45.9 against 42 us in bf16).
template <bool INF>
__global__ void __launch_bounds__(kNormThreads) k_optim_norm_each(const OptimTable t, const OptimWork w, float* each) {
  using F = Fold<INF>;
  pdl_trigger();
  const int32_t j = blockIdx.x * (kNormThreads / 32) + (threadIdx.x >> 5);
  int32_t b0 = 0, b1 = -1;
  if (j < t.k && t.tile0[j] < t.tile0[j + 1]) {
    b0 = block_of_tile(t.ntiles, w.norm_blocks, t.tile0[j]);
    b1 = block_of_tile(t.ntiles, w.norm_blocks, t.tile0[j + 1] - 1);
  }
  pdl_wait();
  if (j >= t.k) return;
  typename F::A acc = F::zero();
#pragma unroll 8
  for (int32_t b = b0 + (threadIdx.x & 31); b <= b1; b += 32) acc = F::join(acc, F::unpack(__ldcg(&w.part_sum[b + j])));
  acc = F::warp(acc);
  if ((threadIdx.x & 31) == 0) each[j] = F::finish(acc);
}

// ------------------------------------------------------------------ clip
// min(1, max_norm / (norm + 1e-6)); a NaN norm gives NaN, as the formula does.
// An infinite max_norm clips nothing: under an infinite norm too, where the
// quotient has no value, c is 1. The test is of a kernel argument, the same for
// the whole grid, and costs nothing that shows; a test of each quotient for NaN
// spills in k_optim_scale<float, 2> (ResNet-50-shaped set, p = 1: 51.9 -> 52.6 us).
__device__ __forceinline__ float clip_coefficient(float norm, float max_norm) {
  if (max_norm > 3.402823466e38f) return norm != norm ? norm : 1.0f;
  const float c = __fdiv_rn(max_norm, __fadd_rn(norm, 1e-6f));
  return c > 1.0f ? 1.0f : c;
}

// Scaled copies: one read and p writes an element, bound by HBM; one block per
// tile, LOADS vectors per thread. Of the clip of the ResNet-50-shaped set into
// 8 replicas this part takes 138 us (920 MB, 6.65 TB/s), of the GPT-2-shaped
// bf16 set into 2 116 us (747 MB, 6.4 TB/s). Writing the tile with bulk stores
// from shared memory took the same time within 2 %. With two vectors in bf16 a
// thread spills 8 bytes; the other forms none.
// The gradients come from HBM a second time: the coefficient depends on all
// of them. Visiting the tiles in reverse, or those read last first, and marking
// the replicas' writes evict-first gained at most 3 us of 159, and marking the
// norm's reads evict-last 4, at the price of what else the L2 holds.
template <typename T, int LOADS>
__global__ void __launch_bounds__(kScaleThreads) k_optim_scale(const OptimTable t, const float* norm, float max_norm) {
  constexpr int V = kVec32<T>, E = kScaleThreads * LOADS * V;
  pdl_trigger();
  // The tables are static: all lookups go ahead while the norm drains.
  const int32_t tensor = tensor_of_tile(t.tile0, t.k, blockIdx.x);
  void* const* outs = t.outs + static_cast<int64_t>(tensor) * t.p;
  const OptimTensor& r = t.tensors[tensor];
  const int64_t x0 = static_cast<int64_t>(static_cast<int32_t>(blockIdx.x) - t.tile0[tensor]) * E - r.f;
  const T* g = static_cast<const T*>(r.grad) + x0;
  const Part part = part_of(x0, r.n, E);
  const bool aligned = r.aligned, grad_aligned = r.grad_aligned;
  auto at = [&](int j) { return static_cast<int>(threadIdx.x + j * kScaleThreads) * V; };
  auto whole = [&](int j) { return aligned && at(j) >= part.lo && at(j) + V <= part.hi; };
  int e = -1;
  if (aligned && threadIdx.x < 32 && (part.lo != 0 || part.hi != E)) e = edge_element<V>(part, threadIdx.x);
  pdl_wait();
  Words y[LOADS];
  T y1{};
#pragma unroll
  for (int j = 0; j < LOADS; ++j) {
    if (!whole(j)) continue;
    if (grad_aligned) {
      y[j] = load32(g + at(j));
    } else {
      float f[V];
      load_each<V>(g + at(j), f);
      y[j] = pack(f, T());
    }
  }
  if (e >= 0) y1 = g[e];
  const float c = clip_coefficient(__ldcg(norm), max_norm);
  if (!aligned) {
    for (int i = part.lo + threadIdx.x; i < part.hi; i += kScaleThreads) {
      const T v = narrow<T>(__fmul_rn(widen(g[i]), c));
      for (int q = 0; q < t.p; ++q) static_cast<T*>(outs[q])[x0 + i] = v;
    }
    return;
  }
#pragma unroll
  for (int j = 0; j < LOADS; ++j) {
    float f[V];
    unpack(y[j], f, T());
#pragma unroll
    for (int l = 0; l < V; ++l) f[l] = __fmul_rn(f[l], c);
    y[j] = pack(f, T());
  }
  y1 = narrow<T>(__fmul_rn(widen(y1), c));
#pragma unroll 8
  for (int q = 0; q < t.p; ++q) {
    T* const o = static_cast<T*>(outs[q]) + x0;
#pragma unroll
    for (int j = 0; j < LOADS; ++j)
      if (whole(j)) store32(o + at(j), y[j]);
    if (e >= 0) o[e] = y1;
  }
}

// ----------------------------------------------------------------- adamw
// 1 - beta^t as -expm1(t log beta): the product in fp64, the rest to fp32 accuracy.
__device__ __forceinline__ StepScalars step_scalars(const AdamwArgs& a, int64_t taken) {
  StepScalars s{1.0f, 0.0f, 0.0f, 0};
  if (a.norm) {
    const float norm = __ldcg(a.norm);
    s.skip = !(norm <= 3.402823466e38f);  // infinite or NaN
    s.c = clip_coefficient(norm, a.max_norm);
  }
  const double t = static_cast<double>(taken + 1);
  s.rate = __fdiv_rn(a.lr, -expm1f(static_cast<float>(t * a.log_beta1)));
  s.bias2 = __fdiv_rn(1.0f, -expm1f(static_cast<float>(t * a.log_beta2)));
  return s;
}

// The step's scalars for the update launched next, and the step count. With
// every block of the update deriving them and taking a ticket, the GPT-2-shaped
// mixed-precision update took 611 us, this way 526; with every thread reading
// them as four words of one place, 605.
__global__ void k_optim_begin(const OptimWork w, const AdamwArgs a) {
  pdl_trigger();
  pdl_wait();
  const int64_t taken = __ldcg(a.step);
  const StepScalars s = step_scalars(a, taken);
  w.scalars[threadIdx.x] = s;
  __syncthreads();
  if (threadIdx.x == 0 && !s.skip) *a.step = taken + 1;
}

// The update of N elements (arrays of fp32): m, v and w become the new ones.
template <int N>
__device__ __forceinline__ void update(const AdamwArgs& a, const StepScalars& s, const float* g, float* m, float* v,
                                       float* w) {
#pragma unroll
  for (int l = 0; l < N; ++l) {
    const float gc = __fmul_rn(g[l], s.c);
    m[l] = fmaf(a.one_minus_beta1, gc - m[l], m[l]);
    v[l] = fmaf(a.beta2, v[l], a.one_minus_beta2 * (gc * gc));
    const float den = __fsqrt_rn(v[l] * s.bias2) + a.eps;
    w[l] = fmaf(-a.decay, w[l], w[l]);
    w[l] = fmaf(-s.rate, __fdiv_rn(m[l], den), w[l]);
  }
}

// One block per tile of 1,024 elements, one vector per thread and stream; about
// 15 flops, a root and a division an element, bound by HBM. Measured: ResNet-50-shaped
// fp32 set with 8 replicas 208.5 us (1.43 GB, 6.9 TB/s), GPT-2-shaped with
// bf16 parameters and fp32 master 525 us (3.73 GB, 7.1 TB/s), Llama-1B-shaped bf16
// with master and 4 replicas 5,790 us (41 GB, 7.08 TB/s): 1.01-1.05 of
// the measured copy rate. On flat buffers, blocks of 256 threads took 529 us
// against 506 (GPT-2-shaped fp32), two vectors per thread 559, a grid of
// resident blocks striding over the tiles 542 and more. Nine blocks per SM
// spill: 236.6 us on the first set; 8 and 7 are even.
constexpr int kUpdateBlocksPerSm = 7;

// From this many tiles the scalars get a launch of their own: one wave of
// blocks (7 on each of 152 SMs). Either side of it, without and with that
// launch: 270 tiles 4.8 and 5.1 us, 976 6.2 and 5.7, 3,906 23.2 and 21.1,
// 15,625 77.4 and 69.5; but a launch costs the host 2 us as well.
constexpr int32_t kBeginTiles = 1024;

// BEGUN: k_optim_begin ran before; otherwise every block derives the scalars
// itself and the block that finishes last advances the step.
template <typename TG, typename TP, bool MASTER, bool BEGUN>
__global__ void __launch_bounds__(kOptimThreads, kUpdateBlocksPerSm)
    k_optim_adamw(const OptimTable t, const OptimWork w, const AdamwArgs a) {
  constexpr int V = kOptimVec, E = kOptimTile;
  __shared__ StepScalars scalars;
  pdl_trigger();
  const bool any = static_cast<int32_t>(blockIdx.x) < t.ntiles;  // an empty set's only block has no tile
  const int32_t tensor = any ? tensor_of_tile(t.tile0, t.k, blockIdx.x) : 0;
  void* const* params = t.outs + static_cast<int64_t>(tensor) * t.p;
  const OptimTensor& r = t.tensors[tensor];
  const int64_t x0 = static_cast<int64_t>(static_cast<int32_t>(blockIdx.x) - t.tile0[tensor]) * E - r.f;
  const Part part = any ? part_of(x0, r.n, E) : Part{0, 0};
  const TG* g = static_cast<const TG*>(r.grad) + x0;
  float *const pm = r.m + x0, *const pv = r.v + x0, *const pw = MASTER ? r.master + x0 : nullptr;
  const int at = threadIdx.x * V;
  const bool aligned = r.aligned, grad_aligned = r.grad_aligned, whole = aligned && at >= part.lo && at + V <= part.hi;
  int e = -1;  // this lane's element of a ragged end
  if (aligned && threadIdx.x < 32 && (part.lo != 0 || part.hi != E)) e = edge_element<V>(part, threadIdx.x);
  const TP* const p0 = static_cast<const TP*>(params[0]) + x0;
  pdl_wait();
  float fg[V], fm[V], fv[V], fw[V];
  if (whole) {
    if (grad_aligned) load8(g + at, fg);
    else load_each<V>(g + at, fg);
    load8(pm + at, fm);
    load8(pv + at, fv);
    if constexpr (MASTER) load8(pw + at, fw);
    else load8(p0 + at, fw);
  }
  StepScalars s;
  if constexpr (BEGUN) {
    const float4 q = __ldcg(reinterpret_cast<const float4*>(w.scalars + blockIdx.x % kScalarCopies));
    s = {q.x, q.y, q.z, __float_as_int(q.w)};
  } else {  // while the loads are in flight thread 0 derives the scalars
    if (threadIdx.x == 0) scalars = step_scalars(a, __ldcg(a.step));
    __syncthreads();
    s = scalars;
  }
  if (s.skip) return;
  if (whole) {
    update<V>(a, s, fg, fm, fv, fw);
    store8(pm + at, fm);
    store8(pv + at, fv);
    if constexpr (MASTER) store8(pw + at, fw);
  }
  auto one = [&](int i) -> float {
    float g1 = widen(g[i]), m1 = pm[i], v1 = pv[i], w1;
    if constexpr (MASTER) w1 = pw[i];
    else w1 = widen(p0[i]);
    update<1>(a, s, &g1, &m1, &v1, &w1);
    pm[i] = m1;
    pv[i] = v1;
    if constexpr (MASTER) pw[i] = w1;
    return w1;
  };
  if (aligned) {
    TP w1{};
    if (e >= 0) w1 = narrow<TP>(one(e));
#pragma unroll 8
    for (int q = 0; q < t.p; ++q) {
      TP* const o = static_cast<TP*>(params[q]) + x0;
      if (whole) store8(o + at, fw);
      if (e >= 0) o[e] = w1;
    }
  } else {
    for (int i = part.lo + threadIdx.x; i < part.hi; i += kOptimThreads) {
      const TP v = narrow<TP>(one(i));
      for (int q = 0; q < t.p; ++q) static_cast<TP*>(params[q])[x0 + i] = v;
    }
  }
  if constexpr (!BEGUN) {  // every block has read the step before it takes a ticket
    if (threadIdx.x == 0) {
      __threadfence();
      if (atomicAdd(&w.ticket[1], 1u) == gridDim.x - 1) {
        *a.step += 1;
        w.ticket[1] = 0;
      }
    }
  }
}

cudaError_t launched(cudaError_t e) {
  count_launch();
  return e != cudaSuccess ? e : cudaGetLastError();
}

template <typename T, bool INF>
cudaError_t norm_of(const OptimTable& t, const OptimWork& w, float* norm, float* each, cudaStream_t s) {
  const dim3 grid(w.norm_blocks), block(kNormThreads);
  if (!each) return launched(launch_pdl(k_optim_norm<T, INF, false>, grid, block, 0, s, t, w, norm));
  const cudaError_t e = launched(launch_pdl(k_optim_norm<T, INF, true>, grid, block, 0, s, t, w, norm));
  if (e != cudaSuccess) return e;
  constexpr int kWarps = kNormThreads / 32;
  return launched(launch_pdl(k_optim_norm_each<INF>, dim3((t.k + kWarps - 1) / kWarps), block, 0, s, t, w, each));
}

template <typename T>
cudaError_t scale_of(const OptimTable& t, const float* norm, float max_norm, cudaStream_t s) {
  const dim3 grid(t.ntiles), block(kScaleThreads);
  static_assert(scale_loads(2) == 2 && scale_loads(3) == 1, "one kernel for each tile size");
  return launched(scale_loads(t.p) == 2 ? launch_pdl(k_optim_scale<T, 2>, grid, block, 0, s, t, norm, max_norm)
                                        : launch_pdl(k_optim_scale<T, 1>, grid, block, 0, s, t, norm, max_norm));
}

template <typename TG, bool BEGUN>
cudaError_t adamw_of(const OptimTable& t, const OptimWork& w, ddp_dtype param_dt, bool master, const AdamwArgs& a,
                     cudaStream_t s) {
  const dim3 grid(t.ntiles > 0 ? t.ntiles : 1), block(kOptimThreads);
  if (param_dt == DDP_FLOAT32)
    return launched(launch_pdl(k_optim_adamw<TG, float, false, BEGUN>, grid, block, 0, s, t, w, a));
  return launched(master ? launch_pdl(k_optim_adamw<TG, __nv_bfloat16, true, BEGUN>, grid, block, 0, s, t, w, a)
                         : launch_pdl(k_optim_adamw<TG, __nv_bfloat16, false, BEGUN>, grid, block, 0, s, t, w, a));
}

}  // namespace

int optim_norm_blocks(int32_t ntiles) {
  const int most = sm_count() * kNormBlocksPerSm;
  return ntiles < 1 ? 1 : ntiles < most ? ntiles : most;
}

cudaError_t launch_optim_norm(const OptimTable& t, const OptimWork& w, ddp_dtype dt, ddp_norm kind, float* norm,
                              float* each, cudaStream_t s) {
  if (dt == DDP_FLOAT32)
    return kind == DDP_NORM_INF ? norm_of<float, true>(t, w, norm, each, s) : norm_of<float, false>(t, w, norm, each, s);
  return kind == DDP_NORM_INF ? norm_of<__nv_bfloat16, true>(t, w, norm, each, s)
                              : norm_of<__nv_bfloat16, false>(t, w, norm, each, s);
}

cudaError_t launch_optim_scale(const OptimTable& t, ddp_dtype dt, const float* norm, float max_norm, cudaStream_t s) {
  if (t.ntiles <= 0) return cudaSuccess;
  return dt == DDP_FLOAT32 ? scale_of<float>(t, norm, max_norm, s) : scale_of<__nv_bfloat16>(t, norm, max_norm, s);
}

cudaError_t launch_optim_adamw(const OptimTable& t, const OptimWork& w, ddp_dtype grad_dt, ddp_dtype param_dt,
                               bool master, const AdamwArgs& a, cudaStream_t s) {
  if (t.ntiles <= kBeginTiles)
    return grad_dt == DDP_FLOAT32 ? adamw_of<float, false>(t, w, param_dt, master, a, s)
                                  : adamw_of<__nv_bfloat16, false>(t, w, param_dt, master, a, s);
  const cudaError_t e = launched(launch_pdl(k_optim_begin, dim3(1), dim3(kScalarCopies), 0, s, w, a));
  if (e != cudaSuccess) return e;
  return grad_dt == DDP_FLOAT32 ? adamw_of<float, true>(t, w, param_dt, master, a, s)
                                : adamw_of<__nv_bfloat16, true>(t, w, param_dt, master, a, s);
}

}  // namespace ddp
