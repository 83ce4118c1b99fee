// What the attention kernels share: 32 x 32 matrix instructions, tiles of key
// or query rows in LDS, and their fragments.
//
// Every product here puts the index that belongs to a lane (a row of softmax
// statistics, or a key) into the columns of the matrix instruction's result:
//   S^T = K Q^T   (columns: query rows)       S = Q K^T    (columns: keys)
// A result's lane l holds column l % 32 and of the 32 rows those that
// result_row() names, four neighbours at a time.  The product that follows
// contracts over just these rows, and a contraction may take its terms in any
// order, the same on both sides: a lane's result values, rounded to the
// operands' type, are the second operand of the next product as they stand, no
// exchange between lanes.  The first operand follows that order: 16-bit ones
// through the transposing LDS read, which returns four rows at a time, fp32
// ones value by value.
#pragma once

#include <utility>

#include "attn_types.h"

namespace ringar {

// f(0), f(1), .. f(N - 1), the number a constant of each call.
template <typename F, int... I> __device__ inline void each_of(F& f, std::integer_sequence<int, I...>) {
  (f(std::integral_constant<int, I>()), ...);
}
template <int N, typename F> __device__ inline void each(F f) { each_of(f, std::make_integer_sequence<int, N>()); }

#define RINGAR_LDS __attribute__((address_space(3)))

typedef float f32x16 __attribute__((ext_vector_type(16)));

// kK: terms of the contraction a step takes; a lane's fragment is the 16-byte
// chunk of its half (lane / 32), so a step takes two chunks of a row.
template <typename T> struct Mma32;
template <> struct Mma32<_Float16> {
  typedef _Float16 Frag __attribute__((ext_vector_type(8)));
  static constexpr int kK = 16;
  static __device__ inline f32x16 run(Frag a, Frag b, f32x16 c) { return __builtin_amdgcn_mfma_f32_32x32x16_f16(a, b, c, 0, 0, 0); }
};
template <> struct Mma32<__bf16> {
  typedef __bf16 Frag __attribute__((ext_vector_type(8)));
  static constexpr int kK = 16;
  static __device__ inline f32x16 run(Frag a, Frag b, f32x16 c) { return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0); }
};
template <> struct Mma32<float> {
  typedef float Frag __attribute__((ext_vector_type(4)));
  static constexpr int kK = 8;
  static __device__ inline f32x16 run(Frag a, Frag b, f32x16 c) {
#pragma unroll
    for (int i = 0; i < 4; i++) c = __builtin_amdgcn_mfma_f32_32x32x2f32(a[i], b[i], c, 0, 0, 0);
    return c;
  }
};

__device__ inline int result_row(int reg, int lane) { return (reg & 3) + 8 * (reg >> 2) + 4 * (lane >> 5); }

// Values first .. of a result as a fragment of the contraction over its rows.
template <typename T> __device__ inline typename Mma32<T>::Frag result_frag(const float* v) {
  typename Mma32<T>::Frag f;
#pragma unroll
  for (int i = 0; i < 16 / (int)sizeof(T); i++) f[i] = (T)v[i];
  return f;
}

__device__ inline f32x16 zero16() { return f32x16{0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0}; }

__device__ inline float fast_exp2(float x) { return __builtin_amdgcn_exp2f(x); }

// Waits until all but the wave's last N loads into LDS have landed and its reads
// are done; the empty asm keeps memory accesses from moving over it.
template <int N = 0> __device__ inline void wait_lds() {
  static_assert(N < 64, "the counter has six bits");
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_waitcnt((N & 15) | 0x70 | (N >> 4 << 14));
  asm volatile("" ::: "memory");
}
__device__ inline void block_barrier() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

// Tiles of rows in memory, one after the other: the buffer of each reaches from
// its first row to the last row's end, and what lies beyond reads as zero.
struct RowStream {
  const char* base;
  int64_t left, step;      // bytes to the last row's end, and from tile to tile

  // from row `row` of `rows`, every `apart` rows
  __device__ inline void start(const void* p, int64_t pitch, int64_t row, int64_t rows, int64_t apart, int row_bytes) {
    base = (const char*)p + row * pitch;
    left = (rows - 1 - row) * pitch + row_bytes;
    step = apart * pitch;
  }
  __device__ inline u32x4 next() {
    const uint32_t size = left >> 31 ? 0x7fffffffu : (uint32_t)left;
    const u32x4 buffer = {(uint32_t)(uintptr_t)base, (uint32_t)((uintptr_t)base >> 32), size, 0x00027000u};
    base += step;
    left -= step;
    return buffer;
  }
  __device__ inline void back(int tiles) {
    base -= tiles * step;
    left += tiles * step;
  }
};

// Loads into LDS, 16 bytes a lane, to `to` and (load_lds2) APART bytes on.  The
// LDS address is taken from m0, one instruction at least after it is set, and
// what a vector instruction has put into a scalar register (the compiler keeps
// scalars in lanes where it has too many) five later: asm gets neither wait
// from the compiler.
__device__ inline void load_lds(uint32_t off, u32x4 buffer, uint32_t to) {
  asm volatile("s_nop 4\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds" :: "{m0}"(to), "v"(off), "s"(buffer) : "memory");
}
template <int APART> __device__ inline void load_lds2(uint32_t off, uint32_t off2, u32x4 buffer, uint32_t to) {
  asm volatile(
      "s_nop 4\n\tbuffer_load_dwordx4 %1, %3, 0 offen lds\n\t"
      "s_add_u32 m0, m0, %4\n\ts_nop 0\n\tbuffer_load_dwordx4 %2, %3, 0 offen lds"
      : "+{m0}"(to) : "v"(off), "v"(off2), "s"(buffer), "n"(APART) : "memory", "scc");
}
// 4 bytes a lane.
__device__ inline void load_lds_word(uint32_t off, u32x4 buffer, uint32_t to) {
  asm volatile("s_nop 4\n\tbuffer_load_dword %1, %2, 0 offen lds" :: "{m0}"(to), "v"(off), "s"(buffer) : "memory");
}

// R rows of D values in LDS, brought by NW waves straight from memory: lines of
// 128 bytes, R of them for each 128 bytes of a row, the eight 16-byte chunks of
// a line in the order c ^ turn(row).  turn() lets both kinds of reads spread
// over all 64 banks in every cycle's 256 bytes: sixteen rows of one chunk (rows
// of like parity lie in one half of the banks, eight turns keep them apart
// there), and four rows of 64 bytes (rows k and k + 2 in different halves of
// their lines).
__device__ inline int turn(int row) { return (row & 2) << 1 | (row & 4) >> 1 | (row & 8) >> 3; }

template <typename T, int D, int R, int NW> struct RowTile {
  static constexpr int kChunk = 16 / sizeof(T);
  static constexpr int kLines = D * (int)sizeof(T) / 128;
  static constexpr int kBytes = R * D * (int)sizeof(T);
  static constexpr int kPlace = kBytes & (kBytes - 1) ? (kBytes / 3) * 4 : kBytes;      // a buffer: a power of two
  static constexpr int kLoads = kBytes / 1024 / NW;
  static_assert(kLoads * NW * 1024 == kBytes && R % 32 == 0, "every wave loads the same share");
  static_assert((kPlace & (kPlace - 1)) == 0, "rows of one, or of three, powers of two");
  static constexpr uint32_t kOutside = 0x80000000u;   // past the end of any buffer

  uint32_t off[kLoads];

  // `pitch`: bytes from row to row; chunks from `dim` on read as zero
  __device__ inline void start(int64_t pitch, int dim, int wave, int lane) {
#pragma unroll
    for (int i = 0; i < kLoads; i++) {
      const int idx = i * NW + wave;
      const int row = idx % (R / 8) * 8 + (lane >> 3), chunk = idx / (R / 8) * 8 + ((lane & 7) ^ turn(row));
      off[i] = chunk * kChunk < dim ? (uint32_t)(row * pitch) + chunk * 16 : kOutside;
    }
  }
  // Starts the loads.  They are asm because the compiler would wait for them
  // before every LDS read that follows; wait_lds() and a barrier come before
  // anything reads what they bring.
  __device__ inline void load(u32x4 buffer, char* lds, int wave) const {
    const uint32_t to = (uint32_t)(uintptr_t)(RINGAR_LDS void*)lds + wave * 1024;
#pragma unroll
    for (int i = 0; i + 1 < kLoads; i += 2) load_lds2<NW * 1024>(off[i], off[i + 1], buffer, to + i * NW * 1024);
    if constexpr (kLoads % 2) load_lds(off[kLoads - 1], buffer, to + (kLoads - 1) * NW * 1024);
  }
  // Zeros from row `from` on, once everything has landed.  Rows that lie over each other
  // (a stride below the row's length, 0 say) do not end where the buffer does: past
  // the last row there are values again, and an infinity there, times a weight
  // of 0, would be NaN.
  static __device__ inline void clear(char* lds, int from, int wave, int lane) {
    for (int row = from + wave; row < R; row += NW)
#pragma unroll
      for (int i = 0; i < kLines; i++)
        if (lane < 32) ((uint32_t*)(lds + (i * R + row) * 128))[lane] = 0;
  }
};

// The lanes' part of the addresses in LDS at which fragments of a RowTile are
// read; what is left, the tile's place and the rows and columns in it, are
// constants of the instruction (a chunk's turn folds into four addresses each).
template <typename T, int R> struct FragReader {
  using Frag = typename Mma32<T>::Frag;
  uint32_t row[4], col[4];

  __device__ inline FragReader(const char* smem, int lane) {
    const uint32_t base = (uint32_t)(uintptr_t)(RINGAR_LDS const void*)smem;
    const int half = lane >> 5, t = lane & 31;
    const uint32_t by_row = base + t * 128 + ((half ^ turn(t)) << 4);
    uint32_t by_col;
    if constexpr (sizeof(T) == 2) {
      // source lane t of 16 gives row t / 4 and four columns; after the
      // transposing read lane t holds column t of the four rows
      const int u = lane & 15, r = 4 * half + (u >> 2);
      by_col = base + r * 128 + ((((lane >> 4 & 1) * 2 + (u >> 1 & 1)) ^ turn(r)) << 4) + (u & 1) * 8;
    } else {
      by_col = base + 4 * half * 128 + (((t >> 2) ^ turn(4 * half)) << 4) + (t & 3) * 4;
    }
#pragma unroll
    for (int i = 0; i < 4; i++) {
      row[i] = by_row ^ (i << 5);
      col[i] = by_col ^ ((i & 1) << 4 | (i & 2) << 5);
    }
  }

  __device__ inline void move_cols(int by) {
#pragma unroll
    for (int i = 0; i < 4; i++) col[i] ^= by;
  }
  // On to another buffer: its place differs in the bits of `apart`.
  __device__ inline void other(int apart) {
#pragma unroll
    for (int i = 0; i < 4; i++) {
      row[i] ^= apart;
      col[i] ^= apart;
    }
  }

  // Rows r0 .. r0 + 31 as the lanes' index, step s of the contraction over D.
  __device__ inline Frag rows(int tile, int r0, int s) const {
    return *(const RINGAR_LDS Frag*)(uintptr_t)(row[s & 3] + tile + s / 4 * (R * 128) + r0 * 128);
  }
  // Columns c0 .. c0 + 31 as the lanes' index, contraction over rows r0 .. in the
  // order of a result's values (r0: a multiple of kK).
  __device__ inline Frag cols(int tile, int r0, int c0) const {
    if constexpr (sizeof(T) == 2) {
      typedef short s16x4 __attribute__((ext_vector_type(4)));
      typedef short s16x8 __attribute__((ext_vector_type(8)));
      s16x4 v[2];
#pragma unroll
      for (int q = 0; q < 2; q++)
        v[q] = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
            (RINGAR_LDS s16x4*)(uintptr_t)(col[(c0 / 32 & 1) * 2 + q] + tile + c0 / 64 * (R * 128) + (r0 + 8 * q) * 128));
      const s16x8 w = {v[0][0], v[0][1], v[0][2], v[0][3], v[1][0], v[1][1], v[1][2], v[1][3]};
      return __builtin_bit_cast(Frag, w);
    } else {
      Frag f;
#pragma unroll
      for (int i = 0; i < 4; i++)
        f[i] = *(const RINGAR_LDS float*)(uintptr_t)(col[(i & 2) + (r0 >> 3 & 1)] + tile + c0 / 32 * (R * 128) + (r0 + i) * 128);
      return f;
    }
  }
};

// 32 rows straight into fragments (their lane index), zeros past `dim` and
// where the lane's row does not exist.
template <typename T, int D> struct RowFrags {
  using Frag = typename Mma32<T>::Frag;
  static constexpr int kSteps = D / Mma32<T>::kK;
  Frag f[kSteps];

  __device__ inline void load(const T* row, bool exists, int dim, int lane) {
    constexpr int kChunk = 16 / sizeof(T);
#pragma unroll
    for (int s = 0; s < kSteps; s++) {
      const int at = (2 * s + (lane >> 5)) * kChunk;
      Frag v = {};
      if (exists && at < dim) v = *(const Frag*)(row + at);
      f[s] = v;
    }
  }
};

// Where a block works.  Blocks go round the 8 XCDs in turn; those that share a
// key head should share an L2, yet sequences of unlike lengths should not lie on
// XCDs of their own.  So a key head's blocks (tiles x splits) are cut into pieces,
// and pieces, not blocks, go round the XCDs.
struct AttnPlace {
  int tile, split, kv_head, batch, length;
  bool valid;                    // (the last round of pieces may be short, and a key head's last piece)
  __device__ inline AttnPlace(const AttnArgs& a) {
    const unsigned each = a.tiles * a.splits, of_xcd = blockIdx.x >> 3;
    const unsigned piece = of_xcd / a.piece * 8 + (blockIdx.x & 7), group = piece / a.pieces;
    const unsigned id = piece % a.pieces * a.piece + of_xcd % a.piece;
    valid = id < each && group < (unsigned)a.kv_heads * a.batch;
    tile = id % a.tiles;
    split = id / a.tiles;
    kv_head = group % a.kv_heads;
    batch = group / a.kv_heads;
    length = a.keys;
    if (a.lengths && valid) {
      const int n = __builtin_amdgcn_readfirstlane(a.lengths[batch]);
      length = n < 0 ? 0 : n < a.keys ? n : a.keys;
    }
  }
  // row r of the group's: its query head and query
  __device__ inline int head(const AttnArgs& a, int r) const { return kv_head * a.group + r / a.queries; }
};

template <typename T> __device__ inline const T* row_at(const HeadRows& v, int64_t batch, int64_t head, int64_t row) {
  return (const T*)v.p + batch * v.batch + head * v.head + row * v.row;
}

// Four neighbouring values of a result.
template <typename T> __device__ inline void put4(T* p, const float* v) {
  Pack<T, 4> o;
#pragma unroll
  for (int i = 0; i < 4; i++) o.v[i] = (T)v[i];
  store_pack<T, 4>(p, o);
}

}  // namespace ringar
