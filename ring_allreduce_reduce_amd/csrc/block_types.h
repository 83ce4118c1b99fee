// Element types, activations and kernel arguments of the block operators
// (layer norm, linear, gated feed-forward), shared by their kernels and the
// host side.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

namespace ringar {

// Blocks of a launch's dimension: the runtime counts their threads in 32 bits.
constexpr int64_t most_blocks(int threads) { return 0xffffffffll / threads; }

// Launches `kernel` and returns that launch's own error.  (hipGetLastError()
// would return any error that an earlier call, not the library's perhaps, has
// left behind; a failed launch leaves none, as the result tells of it.)
template <typename... P>
inline hipError_t launch_kernel(void (*kernel)(P...), dim3 grid, unsigned threads, hipStream_t st, std::common_type_t<P>... args) {
  void* params[] = {(void*)&args...};
  const hipError_t e = hipLaunchKernel((const void*)kernel, grid, dim3(threads), params, 0, st);
  if (e != hipSuccess) (void)hipGetLastError();
  return e;
}

// activation codes of the public header
enum : int { kActNone = 0, kActRelu = 1, kActGelu = 2, kActGeluTanh = 3, kActSilu = 4, kActSigmoid = 5 };

// dtype codes of the public header that the block operators take
enum : int { kF16 = 2, kBF16 = 3, kF32 = 4 };

template <int DT> struct ElemOf;
template <> struct ElemOf<kF16> { using type = _Float16; };
template <> struct ElemOf<kBF16> { using type = __bf16; };
template <> struct ElemOf<kF32> { using type = float; };

typedef float f32x4 __attribute__((ext_vector_type(4)));

// N elements moved as one access; rows may start at any element, so the
// alignment promised is the element's own (the hardware takes unaligned
// global accesses as single ones).
template <typename T, int N> struct alignas(sizeof(T)) Pack {
  T v[N];
};
template <typename T, int N> __device__ inline Pack<T, N> load_pack(const T* p) {
  Pack<T, N> r;
  __builtin_memcpy(&r, p, sizeof(r));
  return r;
}
template <typename T, int N> __device__ inline void store_pack(T* p, const Pack<T, N>& v) {
  __builtin_memcpy(p, &v, sizeof(v));
}

// 16 bytes that are not wanted back soon: past the caches' keeping.
typedef float f32x4_any __attribute__((ext_vector_type(4), aligned(2)));
template <typename T, int N> __device__ inline void stream_pack(T* p, const Pack<T, N>& v) {
  static_assert(sizeof(v) % 16 == 0, "whole 16-byte stores");
#pragma unroll
  for (unsigned i = 0; i < sizeof(v) / 16; i++) {
    f32x4 q;
    __builtin_memcpy(&q, (const char*)&v + 16 * i, 16);
    __builtin_nontemporal_store((f32x4_any)q, (f32x4_any*)p + i);
  }
}

// exp and 1/x of the activations: the 16-bit types take the hardware's
// exponential and reciprocal (relative error about 1e-6 against the 2e-3 of
// their own rounding), fp32 the full-precision ones.
template <bool FAST> __device__ inline float act_exp(float x) {
  if constexpr (FAST) return __builtin_amdgcn_exp2f(x * 1.4426950408889634f);
  return expf(x);
}
template <bool FAST> __device__ inline float act_rcp(float x) {
  if constexpr (FAST) return __builtin_amdgcn_rcpf(x);
  return 1.0f / x;
}

template <bool FAST> __device__ inline float sigmoid_of(float z) { return act_rcp<FAST>(1.0f + act_exp<FAST>(-z)); }

// 2u of the tanh form: gelu_tanh(z) = z sigmoid(2u), u = sqrt(2/pi)(z + 0.044715 z^3)
constexpr float kGeluA = 1.5957691216057308f;            // 2 sqrt(2/pi)
constexpr float kGeluB = 0.044715f;
constexpr float kSqrtHalf = 0.70710678118654752f;
constexpr float kInvSqrt2Pi = 0.39894228040143268f;

// The normal distribution function and its density: gelu(z) = z cdf(z).  The
// lower tail comes from erfc, without the cancellation of 1 + erf (4% at z =
// -5 in fp32): what is left is the rounding of erfc's and the exponential's
// argument, z^2 2^-24 of the value.
// FAST: the tail at -a is exp(-a^2 / 2) (c1 t + .. + c6 t^6), t = 1 / (1 + p a),
// p and c fitted to erfcx over 0 .. 13.5 by linear programming on the largest
// weighted relative error: 4e-7 up to a = 0.5, 2.3e-6 at 2, 2.3e-5 from 4 on, where
// a rounding of fp16 is 4.9e-4.  Its exponential is the density's.  (333 x 1024 x
// 2048 fp16: 7.6 us, with silu 7.3.)
template <bool FAST> __device__ inline void normal(float z, float* cdf, float* density) {
  const float e = act_exp<FAST>(-0.5f * z * z);
  *density = e * kInvSqrt2Pi;
  if constexpr (FAST) {
    const float t = act_rcp<FAST>(fmaf(0.29549676f, fabsf(z), 1.0f));
    float poly = fmaf(t, -0.083796522f, 0.24971875f);
    poly = fmaf(t, fmaf(t, fmaf(t, fmaf(t, poly, -0.052759133f), 0.16020395f), 0.10802665f), 0.11860617f);
    const float tail = e * (t * poly);
    *cdf = z < 0.0f ? tail : 1.0f - tail;
  } else {
    *cdf = 0.5f * erfcf(-z * kSqrtHalf);
  }
}

template <bool FAST> __device__ inline float activate(int act, float z) {
  switch (act) {
    case kActRelu: return z < 0.0f ? 0.0f : z;            // NaN stays NaN
    case kActGelu: {
      float cdf, density;
      normal<FAST>(z, &cdf, &density);
      return z * cdf;
    }
    case kActGeluTanh: return z * sigmoid_of<FAST>(kGeluA * z * (1.0f + kGeluB * z * z));
    case kActSilu: return z * sigmoid_of<FAST>(z);
    case kActSigmoid: return sigmoid_of<FAST>(z);
    default: return z;
  }
}

// act(z) and act'(z) together: they share the exponential.
template <bool FAST> __device__ inline void activate_grad(int act, float z, float* a, float* d) {
  switch (act) {
    case kActRelu:
      *a = z < 0.0f ? 0.0f : z;
      *d = z > 0.0f ? 1.0f : 0.0f;
      return;
    case kActGelu: {
      float cdf, density;
      normal<FAST>(z, &cdf, &density);
      *a = z * cdf;
      *d = cdf + z * density;
      return;
    }
    case kActGeluTanh: {
      const float zz = fminf(z * z, 1e30f);      // infinite, it would meet the zero of s (1 - s)
      const float s = sigmoid_of<FAST>(kGeluA * z * (1.0f + kGeluB * zz));
      *a = z * s;
      *d = s + z * (s * (1.0f - s)) * (kGeluA * (1.0f + 3.0f * kGeluB * zz));
      return;
    }
    case kActSilu: {
      const float s = sigmoid_of<FAST>(z);
      *a = z * s;
      *d = s * (1.0f + z * (1.0f - s));
      return;
    }
    case kActSigmoid: {
      const float s = sigmoid_of<FAST>(z);
      *a = s;
      *d = s * (1.0f - s);
      return;
    }
    default:
      *a = z;
      *d = 1.0f;
  }
}

// The same for N values, the choice of activation outside the loop.
template <bool FAST, int N> __device__ inline void activate_grad_n(int act, const float* z, float* a, float* d) {
  switch (act) {
#define RINGAR_EACH(code)                                                                              \
  case code:                                                                                           \
    _Pragma("unroll") for (int i = 0; i < N; i++) activate_grad<FAST>(code, z[i], a + i, d + i);       \
    break;
    RINGAR_EACH(kActRelu)
    RINGAR_EACH(kActGelu)
    RINGAR_EACH(kActGeluTanh)
    RINGAR_EACH(kActSilu)
    RINGAR_EACH(kActSigmoid)
    RINGAR_EACH(kActNone)
#undef RINGAR_EACH
  }
}

// Parts that blocks on different XCDs pass to each other: agent-scope
// accesses, which go past the XCDs' own caches, so that no cache has to be
// written back or discarded (fences that do this for every block cost 40 us
// where the product takes 10).
__device__ inline void put_part(float* p, float v) { __hip_atomic_store(p, v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT); }
__device__ inline float get_part(const float* p) { return __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT); }

// The sum of parts first, first + step, .. below `count`, in that order.  N
// loads are in flight at a time, the last ones too (an unrolled loop takes
// its rest one by one: backward of 4 x 117 x 13184 fp16 11.4 us, not 10.2).
template <int N, typename F> __device__ inline float sum_parts(int first, int step, int count, F load) {
  float s = 0.0f;
  for (int i = first; i < count; i += N * step) {
    float v[N];
#pragma unroll
    for (int j = 0; j < N; j++) v[j] = load(i + j * step < count ? i + j * step : i);
#pragma unroll
    for (int j = 0; j < N; j++) s += i + j * step < count ? v[j] : 0.0f;
  }
  return s;
}

// Called by every thread of `blocks` blocks after their put_part()s: true in
// the block that arrives last, which may then get_part() every part.  The
// counter is zero before and after (it belongs to the workspace).
__device__ inline bool last_to_arrive(uint32_t* counter, int blocks) {
  __shared__ bool last;
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");   // this thread's parts have reached memory
  __syncthreads();
  if (threadIdx.x == 0) {
    last = __hip_atomic_fetch_add(counter, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) == (uint32_t)blocks - 1;
    if (last) __hip_atomic_store(counter, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  }
  __syncthreads();
  return last;
}

// ------------------------------------------------------------- layer norm
struct NormArgs {
  const void* x;
  const void* dy;        // backward
  const void* weight;    // null: ones
  const void* bias;      // null: zeros (forward)
  void* y;               // forward: y; backward: dx (may be null)
  float* mean;           // forward: may be null; backward: inputs
  float* rstd;
  float* part;           // backward: partial sums [groups][dweight, dbias], or null
  void* dweight;         // backward, without part: the sums of the one block, or null
  void* dbias;
  int64_t ldx, lddy, ldy;
  int64_t rows;
  int cols;
  int groups;            // blocks of the backward grid
  float eps;
  float inv_cols;
  bool stream;           // y goes past the caches
};

// ------------------------------------------------- products and their epilogue
// C[m][n] = sum_k A[m][k] B[n][k]; one of each operand's two strides is 1.
// Gated: n counts the outputs; B has 2 n rows, the gate's and then the up
// projection's.
enum : int { kEpiStore = 0, kEpiLinear = 1, kEpiGated = 2 };

// kernels of a product: tiles of 256 x 256, 128 x 128 and 64 x 64 (gated:
// 64 x 128) with direct loads, 64 x 64 with loads through registers (any
// alignment), and the forward product of up to 16 rows
enum : int { kTile256 = 0, kTile128 = 1, kTile64 = 2, kStaged64 = 3, kRows = 4 };

// kRows: blocks of columns
inline int64_t rows_tiles(int epi, int64_t n) { return epi == kEpiGated ? (n + 7) / 8 : (n + 15) / 16; }

struct GemmArgs {
  const void* a;
  const void* b;
  int64_t sam, sak;      // strides of A in elements
  int64_t sbn, sbk;      // strides of B
  int m, n, k;           // n: output columns (gated: F)
  int variant;           // kernel, set with the split by plan_gemm
  int splits;            // parts of k, each a multiple of the tile's k
  int k_per_split;
  int tile_first;        // tiles of this launch (of twice the kernel's tile
  int tile_count;        // either way where `quarters`: four blocks each; kRows: of columns)
  bool quarters;
  int tail_count;        // kTile256: tiles left to 128 x 128 blocks
  float* part;           // splits > 1: [splits][m][n, gated 2n]
  uint32_t* arrived;     // kRows with splits > 1: a zero for every tile
  // epilogue
  const void* bias;      // n (gated: 2F), or null
  const void* residual;  // or null
  void* c;
  void* pre;             // or null
  int64_t ldc, ldr, ldp;
  int act;
};

// A product as planned: its arguments, and the copies of operands whose rows
// do not start at 16-byte boundaries that are made first, where the direct
// loads win back what a copy costs.
struct GemmPlan {
  GemmArgs args;
  int epi;
  bool pack_a, pack_b;
  int64_t packed_a, packed_b;   // the copies' row strides
  size_t bytes;                 // workspace
  bool too_many;                // more blocks than a launch takes
};
struct PackArgs {
  struct One {
    const void* from;
    void* to;
    int64_t ld_from, ld_to;
    int64_t rows;
    int cols;
    unsigned blocks;
  } one[2];               // the second may have no blocks
};

// activation's backward pass and column sums
struct DzArgs {
  const void* dy;        // [rows][n]
  const void* pre;       // [rows][n], gated [rows][2n]
  void* dz;              // [rows][n], gated [rows][2n]; null: not wanted
  float* part;           // [groups][n or 2n] partial column sums, or null
  void* sums;            // the column sums themselves (one group), or null
  int64_t lddy, ldp, lddz;
  int64_t rows;
  int n;
  int groups;
  int act;
  int gated;
};

// sums over p of part[p][0 .. width): the first n0 columns to out0, the rest
// to out1; a null output is not wanted
struct ColSumArgs {
  const float* part;
  int parts;
  int64_t width;
  int64_t n0;
  void* out0;
  void* out1;
};

// backward pass of a few rows (few_rows)
struct FewArgs {
  const void* dy;
  const void* pre;       // or null
  const void* x;
  const void* w;
  void* dx;              // or null
  void* dw;              // or null
  void* db;              // or null
  float* part;           // parts > 1: [parts][rows][k] of dx
  int64_t lddy, ldp, ldx, ldw, lddx, lddw, k;
  int rows, n, wide;     // wide: n, gated 2n
  int act;
  int gated;
  // plan_few
  int n_each, parts, across_log;
};

// One block's 64 columns of column sums: its waves take the partial rows in
// turn, eight loads in flight each; then the waves' sums in order.  smem: 64
// floats a wave.
template <typename O> __device__ inline void col_sum_block(const ColSumArgs& a, unsigned block, int waves, float* smem) {
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  const int64_t c = (int64_t)block * 64 + lane;
  float s = 0.0f;
  if (c < a.width) {
    const float* p = a.part + c;
    s = sum_parts<8>(w, waves, a.parts, [&](int i) { return p[i * a.width]; });
  }
  smem[w * 64 + lane] = s;
  __syncthreads();
  if (w == 0 && c < a.width) {
    s = 0.0f;
    for (int i = 0; i < waves; i++) s += smem[i * 64 + lane];
    O* out = c < a.n0 ? (O*)a.out0 : (O*)a.out1;
    if (out) out[c < a.n0 ? c : c - a.n0] = (O)s;
  }
}

// the kernels' launchers (dtype codes of the public header)
hipError_t launch_norm_forward(int dtype, int wdtype, const NormArgs& a, hipStream_t st);
hipError_t launch_norm_backward(int dtype, int wdtype, const NormArgs& a, hipStream_t st);
constexpr int kNormLongest = 16384;            // columns of the rows that registers hold
int norm_backward_groups(int64_t rows, int cols);
hipError_t launch_col_sum(int out_dtype, const ColSumArgs& a, hipStream_t st);
hipError_t launch_dz(int dtype, const DzArgs& a, hipStream_t st);
int dz_groups(int dtype, int64_t rows, int64_t n);
// Chooses the kernel, the split of k and the copies from sizes, strides and
// alignment alone.
GemmPlan plan_gemm(int dtype, int epi, const GemmArgs& a);
// `ws`: p.bytes of workspace; `counters`: its kCounters zeros.
hipError_t launch_gemm(int dtype, const GemmPlan& p, char* ws, uint32_t* counters, hipStream_t st);
// dx and dweight in one launch (their workspaces apart), where both run the
// same tile: a launch less, and the one fills what the other leaves idle.
// plan_gradients() chooses so, and plans both.
bool plan_gradients(int dtype, const GemmArgs& x, const GemmArgs& w, GemmPlan* px, GemmPlan* pw);
// `sums`: column sums that the launch adds up beside them (no columns: none).
hipError_t launch_gradients(int dtype, const GemmPlan& x, const GemmPlan& w, const ColSumArgs& sums, char* ws_x, char* ws_w, hipStream_t st);
bool few_rows(int dtype, int64_t rows, int64_t wide, int64_t k);
size_t plan_few(int dtype, FewArgs& a);       // returns the bytes of parts
hipError_t launch_few(int dtype, const FewArgs& a, hipStream_t st);
hipError_t launch_pack(int dtype, PackArgs a, hipStream_t st);
hipError_t launch_clear(uint32_t* words, unsigned count, hipStream_t st);

}  // namespace ringar
