// Dropout, with the residual's addition, from a generator that counts: the
// mask is computed where it is needed, in the forward pass and again in the
// backward pass, and never stored.
//
//   y = keep ? x / (1 - p) : 0, + residual
//
// Numbers are Philox4x32-10's (J. K. Salmon, M. A. Moraes, R. O. Dror, D. E.
// Shaw, "Parallel random numbers: as easy as 1, 2, 3", 2011): a bijection of
// 128 bits, ten rounds of two 32 x 32 bit products, keyed by the seed and
// counted by (column / 8, row, offset).  A block's 128 bits are the eight
// 16-bit numbers of eight columns; a value is kept where its number is not
// below p 2^16.  16 bits, not 32, a value: p is a multiple of 2^-16, off by 2^-17 at
// most (and the scale is that p's, so the mean is exact), and the ten rounds then
// cost less than the memory's time.  Rows count on their own, so a value's number
// depends on its row and column alone, not on the width, strides or launch.
// Memory bound: with the residual 16384 x 8192 bf16 157 us (5.1 TB/s).
#include "layer_types.h"
#include "norm_rows.h"

namespace ringar {
namespace {

struct Words {
  uint32_t w[4];
};

__device__ inline Words philox(uint32_t c0, uint32_t c1, uint32_t c2, uint32_t c3, uint32_t k0, uint32_t k1) {
#pragma unroll
  for (int i = 0; i < 10; i++) {
    const uint64_t a = (uint64_t)c0 * 0xD2511F53u, b = (uint64_t)c2 * 0xCD9E8D57u;
    c0 = (uint32_t)(b >> 32) ^ c1 ^ k0;
    c2 = (uint32_t)(a >> 32) ^ c3 ^ k1;
    c1 = (uint32_t)b;
    c3 = (uint32_t)a;
    k0 += 0x9E3779B9u;
    k1 += 0xBB67AE85u;
  }
  return Words{{c0, c1, c2, c3}};
}

// A thread takes blocks of eight columns, `step` apart.
template <typename T, bool RESIDUAL, bool STREAM> __global__ __launch_bounds__(256) void dropout(DropArgs a) {
  const int64_t first = (int64_t)blockIdx.x * 256 + threadIdx.x;
  int64_t row = first / a.blocks;
  int block = (int)(first % a.blocks);
  uint64_t offset = a.offset;
  if (a.more) offset += (uint64_t)*a.more;
  while (row < a.rows) {
    const int c = block * 8;
    const T* x = (const T*)a.x + row * a.ldx + c;
    const T* residual = (const T*)a.residual + row * a.ldr + c;
    T* y = (T*)a.y + row * a.ldy + c;
    const Words n = philox((uint32_t)(a.first_block + block), (uint32_t)(a.first_row + row), (uint32_t)offset, (uint32_t)(offset >> 32),
                           a.seed[0], a.seed[1]);
    auto value = [&](int j, T v, T res) {
      const uint32_t number = n.w[j / 2] >> (j % 2 * 16) & 0xffffu;
      float z = number >= a.threshold ? (float)v * a.scale : 0.0f;
      if constexpr (RESIDUAL) z += (float)res;
      return (T)z;
    };
    if (c + 8 <= a.cols) {
      const Pack<T, 8> v = load_pack<T, 8>(x);
      Pack<T, 8> res = {}, out;
      if constexpr (RESIDUAL) res = load_pack<T, 8>(residual);
#pragma unroll
      for (int j = 0; j < 8; j++) out.v[j] = value(j, v.v[j], res.v[j]);
      if constexpr (STREAM) stream_pack<T, 8>(y, out);
      else store_pack<T, 8>(y, out);
    } else {
#pragma unroll
      for (int j = 0; j < 8; j++)
        if (c + j < a.cols) y[j] = value(j, x[j], RESIDUAL ? residual[j] : (T)0.0f);
    }
    row += a.step_rows;
    block += a.step_blocks;
    if (block >= a.blocks) {
      block -= a.blocks;
      row++;
    }
  }
}

template <typename T> hipError_t launch(DropArgs a, bool stream, hipStream_t st) {
  a.blocks = (a.cols + 7) / 8;
  const int64_t wanted = (a.rows * a.blocks + 255) / 256, most = 256 * 8;      // 8 blocks a CU
  const int64_t grid = wanted < most ? wanted : most;
  a.step_rows = grid * 256 / a.blocks;
  a.step_blocks = (int)(grid * 256 % a.blocks);
  auto go = [&](auto kernel) { return launch_kernel(kernel, dim3((unsigned)grid), 256, st, a); };
  if (a.residual) return stream ? go(dropout<T, true, true>) : go(dropout<T, true, false>);
  return stream ? go(dropout<T, false, true>) : go(dropout<T, false, false>);
}

}  // namespace

hipError_t launch_dropout(int dtype, const DropArgs& a, hipStream_t st) {
  const bool stream = beyond_l2(dtype, a.rows, a.cols);
  if (dtype == kF32) return launch<float>(a, stream, st);
  if (dtype == kF16) return launch<_Float16>(a, stream, st);
  return launch<__bf16>(a, stream, st);
}

}  // namespace ringar
