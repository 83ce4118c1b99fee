// The forward product of a few rows (single tokens, small decoding batches):
// the weight is read once, straight into registers, and what bounds it is
// how much of it is in flight.
//
// A block takes 16 rows of the weight (gated: 8 of the gate and the same 8 of
// the up projection), its waves the steps of k in turn; a wave's lane loads 16
// bytes of weight row l % 16 at a time, which is the matrix instruction's own
// operand layout, so nothing passes through LDS until the waves' sums are
// added, in wave order.
// The step after the next is on its way while one is multiplied.  Where the
// blocks are too few to fill the GPU, k is split over several; the last of
// them to arrive adds the parts, in their order.  1 x 4096 x 4096 bf16: 8.1 us,
// 4.2 TB/s, 16 rows 9.8; fp32 17.8 and 20.8 (one matrix instruction holds them all).
#pragma once

#include "gemm_kernel.h"

namespace ringar {

constexpr int kRowsMost = 16;      // rows of one matrix instruction

// 16 bytes at an address that is a multiple of 2 alone: from the five words
// around them (each holds at least one of the bytes).  One load there costs
// as much as several (1 x 4095 x 16384 fp16: 31 us, 56 with it).
__device__ inline f32x4 load_from_words(const void* p) {
  typedef uint32_t words __attribute__((ext_vector_type(4), aligned(4)));
  const uintptr_t at = (uintptr_t)p & ~(uintptr_t)3;
  const bool half = (uintptr_t)p & 2;
  const words w = *(const words*)at;
  const uint32_t last = *(const uint32_t*)(at + (half ? 16 : 12));
  const uint32_t shift = half ? 16 : 0;
  typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
  return __builtin_bit_cast(f32x4, u32x4{__builtin_amdgcn_alignbit(w[1], w[0], shift), __builtin_amdgcn_alignbit(w[2], w[1], shift),
                                         __builtin_amdgcn_alignbit(w[3], w[2], shift), __builtin_amdgcn_alignbit(last, w[3], shift)});
}

// HALVES: rows may start between two words.
template <typename T, int EPI, int WAVES, bool HALVES>
__global__ __launch_bounds__(64 * WAVES) void gemm_rows(GemmArgs a) {
  using Frag = typename Mma<T>::Frag;
  constexpr int kVec = 16 / sizeof(T);
  constexpr int U = 4;                       // matrix instructions of a step
  constexpr int kK = 4 * kVec, kStep = U * kK;
  constexpr int kCols = EPI == kEpiGated ? 8 : 16;    // outputs of a block
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, t = lane & 15, g = lane >> 4;
  const int tile = a.tile_first + blockIdx.x / a.splits, split = blockIdx.x % a.splits;
  const int64_t n0 = (int64_t)tile * kCols;
  const int k_end = a.k - split * a.k_per_split < a.k_per_split ? a.k : (split + 1) * a.k_per_split;
  const int64_t col = n0 + t % kCols < a.n ? n0 + t % kCols : a.n - 1;   // past the edge: the last column again, not stored
  const T* w = (const T*)a.b + (col + (kCols == 8 && t >= 8 ? a.n : 0)) * a.sbn;
  const T* x = (const T*)a.a + (t < a.m ? t : 0) * a.sam;

  struct Step {
    Frag w[U], x[U];
  };
  auto load16 = [](const T* p) {
    Frag f;
    if constexpr (HALVES) f = __builtin_bit_cast(Frag, load_from_words(p));
    else __builtin_memcpy(&f, p, 16);
    return f;
  };
  auto load = [&](Step& s, int k0) {
    // What would pass the end starts kVec before it instead, with zeros in
    // place of the values that another lane holds.
    const int at = k0 + g * kVec, last = k_end - kVec;
#pragma unroll
    for (int u = 0; u < U; u++) s.w[u] = load16(w + (at + u * kK < last ? at + u * kK : last));
#pragma unroll
    for (int u = 0; u < U; u++) s.x[u] = load16(x + (at + u * kK < last ? at + u * kK : last));
    if (k0 + kStep > k_end) {
#pragma unroll
      for (int u = 0; u < U; u++)
#pragma unroll
        for (int i = 0; i < kVec; i++)
          if (i < at + u * kK - last) s.w[u][i] = s.x[u][i] = (T)0.0f;
    }
  };
  f32x4 acc = {0.0f, 0.0f, 0.0f, 0.0f};
  auto mma = [&](const Step& s) {
#pragma unroll
    for (int u = 0; u < U; u++) acc = Mma<T>::run(s.w[u], s.x[u], acc);
  };

  // Every block starts at another step: the rows of a weight lie a power of
  // two apart more often than not, and blocks that walk them in step meet in
  // the same memory channels (8192 x 8192 bf16, one row: 32 us, not 25).
  const int k_begin = split * a.k_per_split;
  const int steps = (k_end - k_begin + kStep - 1) / kStep;
  const int first = steps ? (int)((uint32_t)tile * 5u % (uint32_t)steps) : 0;
  auto start = [&](int i) { return k_begin + (i + first < steps ? i + first : i + first - steps) * kStep; };
  Step even, odd;
  int i = wave;
  if (i < steps) load(even, start(i));
  for (; i < steps; i += 2 * WAVES) {
    const bool second = i + WAVES < steps;
    if (second) load(odd, start(i + WAVES));
    mma(even);
    if (i + 2 * WAVES < steps) load(even, start(i + 2 * WAVES));
    if (second) mma(odd);
  }

  // lane: row t of C, columns g * 4 .. + 3
  __shared__ __attribute__((aligned(16))) float sums[WAVES][16][20];
  *(f32x4*)&sums[wave][t][g * 4] = acc;
  __syncthreads();
  const int m = threadIdx.x >> 4, c = threadIdx.x & 15;
  const bool mine = threadIdx.x < 256 && m < a.m;
  float v = 0.0f;
  if (mine) {
#pragma unroll
    for (int i = 0; i < WAVES; i++) v += sums[i][m][c];
  }
  if (a.splits > 1) {
    // [tile][split][m][16]
    float* part = a.part + ((int64_t)tile * a.splits * a.m + m) * 16 + c;
    const int64_t next = (int64_t)a.m * 16;
    if (mine) put_part(part + split * next, v);
    if (!last_to_arrive(a.arrived + tile, a.splits)) return;
    if (mine) v = sum_parts<8>(0, 1, a.splits, [&](int i) { return get_part(part + i * next); });
  }
  if constexpr (EPI == kEpiGated) {
    const float up = __shfl_down(v, 8);      // the up projection's sums sit eight lanes on
    if (mine && c < 8 && n0 + c < a.n) finish_gated<T>(a, m, (int)(n0 + c), v, up);
  } else if (mine && n0 + c < a.n) {
    finish_linear<T>(a, m, (int)(n0 + c), v);
  }
}

}  // namespace ringar
