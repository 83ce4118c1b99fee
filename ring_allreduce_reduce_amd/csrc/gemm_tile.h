// The tiled product kernel.
//
// A block of WM x WN waves computes a BM x BN tile of C in steps of 128 bytes
// of k.  Operand tiles go from memory straight into LDS (16 bytes a lane, no
// registers), two buffers in turn: the loads of step t + 2 start as soon as
// the last wave has read step t, and have a whole step of matrix instructions
// to arrive.  Within a step the fragments of one half are read while the
// other half's matrix instructions run, and the next step's first half is
// read across the barrier, so the matrix units wait for LDS only where a
// wave waits for the slowest one.  8192 x 4096 x 16384 bf16: 763 us (1441
// TFLOP/s; a library's plain product 672) forward without an epilogue, 832 with
// bias, gelu and the kept pre-activation (884 over three sets of operands); the matrix units are busy 67 .. 70% of the time at the 1.9 GHz
// that the power leaves.
//
// LDS holds an operand as it lies in memory:
//   ROW (k contiguous): one 128-byte line per row, its eight 16-byte chunks
//     in the order c ^ (row & 7), so that eight rows read the same chunk from
//     different banks.
//   COL (rows contiguous): one line of the tile's rows per k, chunks in the
//     order c ^ col_swizzle(k); 16-bit fragments come through the transposing
//     LDS read, fp32 ones value by value.
// The first matrix operand is B (columns of C), the second A: a lane then
// holds four consecutive columns of one row of C.  The epilogue passes 32 rows
// at a time through the wave's own part of LDS, after which eight lanes hold
// 64 consecutive columns of a row and everything the epilogue reads or writes
// moves in whole 128-byte lines.
#pragma once

#include <type_traits>

#include "gemm_kernel.h"

namespace ringar {

#define RINGAR_LDS __attribute__((address_space(3)))

// One operand's tile: R rows by 128 bytes of k, loaded by NW waves.
template <typename T, bool ROW, int R, int NW> struct Operand {
  static constexpr int kVec = 16 / sizeof(T);
  static constexpr int kBK = 128 / sizeof(T);
  static constexpr int kBytes = R * 128;
  static constexpr int kLoads = kBytes / 1024 / NW;       // load instructions of a wave and step
  static constexpr int kChunks = R * sizeof(T) / 16;      // COL: chunks of a line
  static_assert(kLoads * 1024 * NW == kBytes, "every wave loads the same share");
  static_assert(ROW || kChunks >= (sizeof(T) == 4 ? 16 : 8), "COL lines hold the swizzle's chunks");

  // COL: the k lines that the lanes of one LDS cycle read (32 lanes of the
  // transposing read: lines k .. k + 3 and k + 8 .. k + 11; all four lane
  // groups of fp32) lie in different 32 (64) bytes of the 256 that the banks
  // span.  A line of 8 chunks spans half of them, odd lines the other half.
  static __device__ inline int col_swizzle(int k) {
    if constexpr (sizeof(T) == 4) return ((k >> 2) & 3) << 2;
    if constexpr (kChunks == 8) return ((k >> 1) & 1) << 2 | ((k >> 3) & 1) << 1;
    return (k & 3) << 2 | ((k >> 3) & 1) << 1;
  }

  const char* base;        // of the current step, uniform
  int64_t left;            // bytes from there to the operand's end
  int64_t step;            // bytes of a step
  uint32_t off[kLoads];

  // `bytes`: the operand's size, up to the end of its last 16-byte chunk (a
  // chunk that straddled the descriptor's end would read as zero entirely;
  // what is past the operand in that chunk is cleared or not used).
  __device__ inline void start(const void* p, int64_t at, int64_t bytes, int64_t step_bytes) {
    base = (const char*)p + at;
    left = ((bytes + 15) & ~15ll) - at;
    step = step_bytes;
  }

  // lane's byte offset of load i, given where tile row r lies (ROW)
  template <typename F> __device__ inline void offsets(int64_t pitch, int wave, int lane, F row_offset) {
#pragma unroll
    for (int i = 0; i < kLoads; i++) {
      const int idx = i * NW + wave;
      if constexpr (ROW) {
        const int r = idx * 8 + (lane >> 3);
        off[i] = (uint32_t)row_offset(r) + (((lane & 7) ^ (r & 7)) << 4);
      } else {
        const int k = idx * (64 / kChunks) + lane / kChunks;
        off[i] = (uint32_t)(k * pitch) + (((lane % kChunks) ^ col_swizzle(k)) << 4);
      }
    }
  }

  // next_step() moves on to a step, load(i) starts its i-th load into `lds`.
  // Reads past the operand's end are stopped by the descriptor's size.  The
  // loads are asm
  // because the compiler would wait for them before every transposing LDS
  // read that follows, which is what the second buffer is there to avoid;
  // they have no register result, and wait_loads() waits for all of them
  // before a barrier lets any wave read what they bring.  The LDS address is
  // taken from m0, one instruction at least after it is set: the compiler puts
  // a wait state there for its own loads, not before asm.
  typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
  u32x4 desc;
  __device__ inline void next_step() {
    const uint32_t size = left <= 0 ? 0u : left > 0xffffffffll ? 0xffffffffu : (uint32_t)left;
    desc = u32x4{(uint32_t)(uintptr_t)base, (uint32_t)((uintptr_t)base >> 32), size, 0x00027000u};
    base += step;
    left -= step;
  }
  __device__ inline void load(int i, char* lds, int wave) {
    const uint32_t to = (uint32_t)(uintptr_t)(RINGAR_LDS void*)lds + (i * NW + wave) * 1024;
    asm volatile("s_nop 0\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds" :: "{m0}"(to), "v"(off[i]), "s"(desc) : "memory");
  }

  // Zeros every value of a step from k = `valid` on.
  static __device__ inline void clear_tail(char* lds, int valid) {
    const f32x4 zero = {0.0f, 0.0f, 0.0f, 0.0f};
    for (int i = threadIdx.x; i < R * 8; i += NW * 64) {
      if constexpr (ROW) {
        const int c = (i & 7) ^ ((i >> 3) & 7);
        if (c * kVec >= valid) *(f32x4*)(lds + i * 16) = zero;
        else if (c * kVec + kVec > valid)
          for (int e = valid - c * kVec; e < kVec; e++) ((T*)(lds + i * 16))[e] = (T)0.0f;
      } else {
        if (i / kChunks >= valid) *(f32x4*)(lds + i * 16) = zero;
      }
    }
  }

  // Fragment of rows r0 .. r0 + 15 of half h of the step.
  using Frag = typename Mma<T>::Frag;
  static __device__ inline Frag read(const char* lds, int r0, int h, int lane) {
    const int t = lane & 15, g = lane >> 4;
    if constexpr (ROW) {
      return *(const Frag*)(lds + (r0 + t) * 128 + (((h * 4 + g) ^ (t & 7)) << 4));
    } else if constexpr (sizeof(T) == 2) {
      // source lane t gives k line t / 4 and four columns; after the
      // transposing read lane t holds column t of the four lines
      const int col = r0 + (t & 3) * 4;
      typedef short s16x4 __attribute__((ext_vector_type(4)));
      typedef short s16x8 __attribute__((ext_vector_type(8)));
      s16x4 v[2];
#pragma unroll
      for (int q = 0; q < 2; q++) {
        const int k = h * 32 + g * 8 + q * 4 + (t >> 2);
        const char* p = lds + k * (R * 2) + (((col >> 3) ^ col_swizzle(k)) << 4) + (col & 7) * 2;
        v[q] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((RINGAR_LDS s16x4*)(RINGAR_LDS void*)p);
      }
      const s16x8 w = {v[0][0], v[0][1], v[0][2], v[0][3], v[1][0], v[1][1], v[1][2], v[1][3]};
      return __builtin_bit_cast(Frag, w);
    } else {
      const int col = r0 + t;
      Frag f;
#pragma unroll
      for (int i = 0; i < 4; i++) {
        const int k = h * 16 + g * 4 + i;
        f[i] = *(const float*)(lds + k * (R * 4) + (((col >> 2) ^ col_swizzle(k)) << 4) + (col & 3) * 4);
      }
      return f;
    }
  }
};

// An operand at any alignment: the same tile in LDS, its chunks loaded to
// registers a step ahead and written from there.  Chunks that pass the end
// of a row (ROW: k, COL: columns) are put together value by value, zeros
// past the end, so nothing beyond the operand is read.
template <typename T, bool ROW, int R, int NW> struct StagedOperand : Operand<T, ROW, R, NW> {
  using Base = Operand<T, ROW, R, NW>;
  static constexpr int kVec = Base::kVec, kLoads = Base::kLoads, kChunks = Base::kChunks;
  using typename Base::u32x4;
  const T* from[kLoads];
  int at[kLoads];          // within the step: ROW: first k of the chunk; COL: k line
  int columns[kLoads];     // COL: columns left from the chunk's first
  u32x4 data[kLoads];
  int64_t step_elems;
  int k_end;

  template <typename F>
  __device__ inline void offsets(const T* p, int64_t pitch, int k_begin, int k_stop, int64_t cols_left, int wave, int lane, F row_offset) {
    k_end = k_stop;
    k_now = k_begin;
    all_columns = cols_left >= R;
    step_elems = ROW ? Base::kBK : Base::kBK * pitch;
#pragma unroll
    for (int i = 0; i < kLoads; i++) {
      const int idx = i * NW + wave;
      if constexpr (ROW) {
        const int r = idx * 8 + (lane >> 3), c = (lane & 7) ^ (r & 7);
        at[i] = c * kVec;
        from[i] = p + row_offset(r) + c * kVec;
      } else {
        const int k = idx * (64 / kChunks) + lane / kChunks, q = (lane % kChunks) ^ Base::col_swizzle(k);
        at[i] = k;
        from[i] = p + k * pitch + q * kVec;
        const int64_t left = cols_left - q * kVec;
        columns[i] = (int)(left < 0 ? 0 : left > kVec ? kVec : left);
      }
    }
  }

  // The loads of the next step; `inside`: no chunk of the tile passes an edge
  // (then none branches, and all are in flight together).
  int k_now;               // first k of the step
  bool all_columns;        // COL: the tile's columns all exist
  __device__ inline void load_step() {
    if (k_now + Base::kBK <= k_end && (ROW || all_columns)) {
#pragma unroll
      for (int i = 0; i < kLoads; i++) __builtin_memcpy(&data[i], from[i], 16);
    } else {
#pragma unroll
      for (int i = 0; i < kLoads; i++) {
        const int n = ROW ? k_end - at[i] - k_now : at[i] + k_now < k_end ? columns[i] : 0;
        u32x4 v = {0, 0, 0, 0};
        const T* p = from[i];
#pragma unroll
        for (int e = 0; e < kVec; e++)
          if (e < n) {
            if constexpr (sizeof(T) == 2) v[e / 2] |= (uint32_t)__builtin_bit_cast(uint16_t, p[e]) << (e % 2 * 16);
            else v[e] = __builtin_bit_cast(uint32_t, p[e]);
          }
        data[i] = v;
      }
    }
#pragma unroll
    for (int i = 0; i < kLoads; i++) from[i] += step_elems;
    k_now += Base::kBK;
  }

  __device__ inline void commit(char* lds, int wave, int lane) {
#pragma unroll
    for (int i = 0; i < kLoads; i++) *(u32x4*)(lds + (i * NW + wave) * 1024 + lane * 16) = data[i];
  }
};

// Eight consecutive output columns of one row.
template <typename T> __device__ inline void add8(const void* p, int64_t at, float* z) {
  const Pack<T, 8> b = load_pack<T, 8>((const T*)p + at);
#pragma unroll
  for (int i = 0; i < 8; i++) z[i] += (float)b.v[i];
}

template <typename T, bool STREAM = false> __device__ inline void put8(void* p, int64_t at, const float* z) {
  Pack<T, 8> o;
#pragma unroll
  for (int i = 0; i < 8; i++) o.v[i] = (T)z[i];
  if constexpr (STREAM) stream_pack<T, 8>((T*)p + at, o);
  else store_pack<T, 8>((T*)p + at, o);
}

template <bool FAST> __device__ inline void activate8(int act, float* z) {
  switch (act) {
#define RINGAR_EACH(code)                                                       \
  case code:                                                                    \
    _Pragma("unroll") for (int i = 0; i < 8; i++) z[i] = activate<FAST>(code, z[i]); \
    break;
    RINGAR_EACH(kActRelu)
    RINGAR_EACH(kActGelu)
    RINGAR_EACH(kActGeluTanh)
    RINGAR_EACH(kActSilu)
    RINGAR_EACH(kActSigmoid)
#undef RINGAR_EACH
    default: break;
  }
}

template <typename T, bool STREAM> __device__ inline void finish8_linear(const GemmArgs& a, int64_t m, int64_t n, float* z) {
  if (a.bias) add8<T>(a.bias, n, z);
  if (a.pre) put8<T, STREAM>(a.pre, m * a.ldp + n, z);
  activate8<sizeof(T) == 2>(a.act, z);
  if (a.residual) add8<T>(a.residual, m * a.ldr + n, z);
  put8<T, STREAM>(a.c, m * a.ldc + n, z);
}

template <typename T, bool STREAM> __device__ inline void finish8_gated(const GemmArgs& a, int64_t m, int64_t n, float* g, float* u) {
  if (a.bias) {
    add8<T>(a.bias, n, g);
    add8<T>(a.bias, a.n + n, u);
  }
  if (a.pre) {
    put8<T, STREAM>(a.pre, m * a.ldp + n, g);
    put8<T, STREAM>(a.pre, m * a.ldp + a.n + n, u);
  }
  activate8<sizeof(T) == 2>(a.act, g);
#pragma unroll
  for (int i = 0; i < 8; i++) g[i] *= u[i];
  put8<T, STREAM>(a.c, m * a.ldc + n, g);
}

// Waits until all but the wave's last N loads into LDS have landed, and all
// its fragment reads are done.  The empty asm keeps the compiler from moving
// memory accesses over the wait.
template <int N = 0> __device__ inline void wait_loads() {
  static_assert(N < 64, "the counter has six bits");
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_waitcnt((N & 15) | 0x70 | (N >> 4 << 14));
}
__device__ inline void barrier() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

// One tile's kernel: run() computes block `block` of the product's grid.
template <typename T, bool AROW, bool BROW, int EPI, int BM, int BN, int WM, int WN, bool DIRECT, int STAGES = 2>
struct GemmTile {
  static constexpr int NW = WM * WN, kThreads = 64 * NW;
  using OA = std::conditional_t<DIRECT, Operand<T, AROW, BM, NW>, StagedOperand<T, AROW, BM, NW>>;
  using OB = std::conditional_t<DIRECT, Operand<T, BROW, BN, NW>, StagedOperand<T, BROW, BN, NW>>;
  static constexpr int TM = BM / WM, TN = BN / WN, FM = TM / 16, FN = TN / 16;
  static constexpr int kBK = OA::kBK;
  static_assert(TN == 64 || (TN == 32 && EPI != kEpiGated), "four or eight lanes finish a wave's row");
  static constexpr int kHalf = TN / 2;         // gated: a wave's columns are half gate, half up
  static_assert(BROW || EPI == kEpiStore, "epilogues with columns of their own read weights by rows");
  static constexpr int kStage = OA::kBytes + OB::kBytes;
  // epilogue: a wave's rows in fp32, shifted 16 bytes over the banks
  static constexpr int kPass = TM < 32 ? TM : 32, kRowF = TN + 4;
  static constexpr int kShared = STAGES * kStage > NW * kPass * kRowF * 4 ? STAGES * kStage : NW * kPass * kRowF * 4;

  static __device__ inline void run(const GemmArgs& a, unsigned block, char* smem);
};

template <typename T, bool AROW, bool BROW, int EPI, int BM, int BN, int WM, int WN, bool DIRECT, int STAGES>
__device__ inline void GemmTile<T, AROW, BROW, EPI, BM, BN, WM, WN, DIRECT, STAGES>::run(const GemmArgs& a, unsigned block, char* smem) {
  using Frag = typename Mma<T>::Frag;

  // Blocks go round the 8 XCDs in turn: give each XCD a run of neighbouring
  // tiles, 8 tiles of rows deep, so that its blocks share operands in its L2.
  constexpr int kOut = EPI == kEpiGated ? BN / 2 : BN;    // output columns of a tile
  const int sub = a.quarters ? 2 : 1;
  const int tiles_m = (a.m + BM * sub - 1) / (BM * sub), tiles_n = (a.n + kOut * sub - 1) / (kOut * sub);
  const int tiles = a.tile_count * sub * sub;
  const int total = tiles * a.splits;
  const int q = total >> 3, rest = total & 7, xcd = block & 7;
  const int id = xcd * q + (xcd < rest ? xcd : rest) + (block >> 3);
  const int split = id / tiles, unit = id % tiles, quarter = unit % (sub * sub);
  const int tile = a.tile_first + unit / (sub * sub);
  const int band = tile / (8 * tiles_n), in_band = tile % (8 * tiles_n);
  const int deep = tiles_m - band * 8 < 8 ? tiles_m - band * 8 : 8;
  const int64_t m0 = ((int64_t)(band * 8 + in_band % deep) * sub + (quarter & 1)) * BM;
  const int64_t n0 = ((int64_t)(in_band / deep) * sub + (quarter >> 1)) * kOut;
  if (m0 >= a.m || n0 >= a.n) return;          // a quarter past the edge
  const int k_begin = split * a.k_per_split;
  const int k_len = (a.k - k_begin < a.k_per_split ? a.k - k_begin : a.k_per_split);
  const int steps = (k_len + kBK - 1) / kBK;

  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = (wave % WM) * TM, wn = (wave / WM) * TN;

  OA oa;
  OB ob;
  {
    const int64_t pitch_a = AROW ? a.sam : a.sak, pitch_b = BROW ? a.sbn : a.sbk;
    // rows past the edge read the last one; their results are not stored
    auto row_a = [&](int r) { return m0 + r < a.m ? (int64_t)r : a.m - 1 - m0; };
    auto row_b = [&](int r) -> int64_t {
      if constexpr (EPI == kEpiGated) {
        // a wave's rows: first of the gate, then the same ones of the up projection
        const int64_t c = r / TN * kHalf + r % kHalf;
        return (n0 + c < a.n ? c : a.n - 1 - n0) + (r % TN >= kHalf ? a.n : 0);
      } else {
        return n0 + r < a.n ? r : a.n - 1 - n0;
      }
    };
    const int64_t first_a = AROW ? m0 * pitch_a + k_begin : k_begin * pitch_a + m0;
    const int64_t first_b = BROW ? n0 * pitch_b + k_begin : k_begin * pitch_b + n0;
    if constexpr (DIRECT) {
      constexpr int64_t es = sizeof(T);
      const int64_t rows_b = EPI == kEpiGated ? 2 * (int64_t)a.n : a.n;
      const int64_t size_a = AROW ? (a.m - 1) * pitch_a + a.k : (a.k - 1) * pitch_a + a.m;
      const int64_t size_b = BROW ? (rows_b - 1) * pitch_b + a.k : (a.k - 1) * pitch_b + rows_b;
      oa.start(a.a, first_a * es, size_a * es, AROW ? 128 : kBK * pitch_a * es);
      ob.start(a.b, first_b * es, size_b * es, BROW ? 128 : kBK * pitch_b * es);
      oa.offsets(pitch_a * es, wave, lane, [&](int r) { return row_a(r) * pitch_a * es; });
      ob.offsets(pitch_b * es, wave, lane, [&](int r) { return row_b(r) * pitch_b * es; });
    } else {
      const int k_stop = k_begin + k_len;
      oa.offsets((const T*)a.a + first_a, pitch_a, k_begin, k_stop, a.m - m0, wave, lane, [&](int r) { return row_a(r) * pitch_a; });
      ob.offsets((const T*)a.b + first_b, pitch_b, k_begin, k_stop, a.n - n0, wave, lane, [&](int r) { return row_b(r) * pitch_b; });
    }
  }

  f32x4 acc[FN][FM];
#pragma unroll
  for (int i = 0; i < FN; i++)
#pragma unroll
    for (int j = 0; j < FM; j++) acc[i][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};

  // Load l of the next step into buffer `buf`.  (Not DIRECT: issue() loads to
  // registers, from which commit() writes to the buffer.)
  constexpr int kStepLoads = DIRECT ? OA::kLoads + OB::kLoads : 0;
  auto load = [&](int l, int buf) {
    if constexpr (DIRECT) {
      char* lds = smem + buf * kStage;
      if (l < OA::kLoads) oa.load(l, lds, wave);
      else ob.load(l - OA::kLoads, lds + OA::kBytes, wave);
    }
  };
  auto issue = [&](int buf) {
    if constexpr (DIRECT) {
      oa.next_step();
      ob.next_step();
#pragma unroll
      for (int l = 0; l < kStepLoads; l++) load(l, buf);
    } else {
      oa.load_step();
      ob.load_step();
    }
  };
  auto commit = [&](int buf) {
    if constexpr (!DIRECT) {
      oa.commit(smem + buf * kStage, wave, lane);
      ob.commit(smem + buf * kStage + OA::kBytes, wave, lane);
    }
  };
  auto fix_tail = [&](int s) {        // the last step, where k ends inside it
    if (DIRECT && s == steps - 1 && k_len % kBK != 0) {
      OA::clear_tail(smem + s % STAGES * kStage, k_len % kBK);
      OB::clear_tail(smem + s % STAGES * kStage + OA::kBytes, k_len % kBK);
      wait_loads<>();
      barrier();
    }
  };
  // Fragment r of half h: B's first.
  auto read = [&](int r, int buf, int h, Frag* fa, Frag* fb) {
    const char* pa = smem + buf * kStage;
    if (r < FN) fb[r] = OB::read(pa + OA::kBytes, wn + r * 16, h, lane);
    else fa[r - FN] = OA::read(pa, wm + (r - FN) * 16, h, lane);
  };
  // The matrix instructions of one half, and between them, evenly, the reads
  // of the next half's fragments (buffer `from`) and, LOADS, the loads of a
  // step to come (buffer `to`).  A wave issues in order: a burst of loads
  // would hold its matrix instructions back until the last is accepted.
  auto half = [&](auto loads, const Frag* fa, const Frag* fb, int from, int h, Frag* na, Frag* nb, int to) {
    constexpr int kMma = FN * FM, kReads = FN + FM;
    if constexpr (loads.value) {
      oa.next_step();
      ob.next_step();
    }
#pragma unroll
    for (int t = 0; t < kMma; t++) {
      // reads in the first three quarters, so that they are back at the end
#pragma unroll
      for (int r = 0; r < kReads; r++)
        if (r * kMma * 3 / (kReads * 4) == t) read(r, from, h, na, nb);
      if constexpr (loads.value) {
#pragma unroll
        for (int l = 0; l < kStepLoads; l++)
          if (l * kMma / kStepLoads == t) load(l, to);
      }
      acc[t / FM][t % FM] = Mma<T>::run(fb[t / FM], fa[t % FM], acc[t / FM][t % FM]);
      __builtin_amdgcn_sched_barrier(0);
    }
  };
  auto mma = [&](const Frag* fa, const Frag* fb) {
#pragma unroll
    for (int t = 0; t < FN * FM; t++) acc[t / FM][t % FM] = Mma<T>::run(fb[t / FM], fa[t % FM], acc[t / FM][t % FM]);
  };

  if (steps > 0) {
    static_assert(STAGES == 2 || (STAGES == 3 && DIRECT), "registers hold one step");
    constexpr std::false_type kNoLoads;
    constexpr std::true_type kLoads;
    Frag fa0[FM], fb0[FN], fa1[FM], fb1[FN];
    // STAGES - 1 steps are on their way before the first is used (four, and
    // one block a CU less, were slower: 1866 x 320 x 3200 fp16 gradients 21.0
    // us, not 20.2).  Waits until only the last `ahead` steps' loads are outstanding
    auto wait_all_but = [&](int ahead) {
      if (STAGES == 3 && ahead == 1) wait_loads<STAGES == 3 ? kStepLoads : 0>();
      else wait_loads<>();
    };
#pragma unroll
    for (int i = 0; i < STAGES - 1; i++) {
      if (i >= steps) break;
      issue(i);
      commit(i);
    }
    wait_all_but(steps - 1 < STAGES - 2 ? steps - 1 : STAGES - 2);
    barrier();
    fix_tail(0);
    if (STAGES - 1 < steps) issue(STAGES - 1);
#pragma unroll
    for (int r = 0; r < FN + FM; r++) read(r, 0, 0, fa0, fb0);
    int now = 0, next = 1;            // buffers of steps s and s + 1
    auto first_half = [&](int s) {
      half(kNoLoads, fa0, fb0, now, 1, fa1, fb1, 0);
      commit(next);                   // its readers of step s - 1 passed the last barrier
      // step s + 1 has landed; with more buffers the steps after it may still be on their way
      wait_all_but(steps - 2 - s < STAGES - 2 ? steps - 2 - s : STAGES - 2);
      barrier();
    };
    int s = 0;
    for (; s < steps - STAGES; s++) {
      first_half(s);
      if constexpr (DIRECT) {
        half(kLoads, fa1, fb1, next, 0, fa0, fb0, now);
      } else {
        issue(now);
        half(kNoLoads, fa1, fb1, next, 0, fa0, fb0, 0);
      }
      now = next;
      next = next + 1 == STAGES ? 0 : next + 1;
    }
    for (; s < steps - 1; s++) {
      first_half(s);
      fix_tail(s + 1);
      half(kNoLoads, fa1, fb1, next, 0, fa0, fb0, 0);
      now = next;
      next = next + 1 == STAGES ? 0 : next + 1;
    }
    half(kNoLoads, fa0, fb0, now, 1, fa1, fb1, 0);
    mma(fa1, fb1);
  }

  wait_loads<>();
  barrier();                                   // every wave is done with the operands
  float* rows = (float*)smem + wave * kPass * kRowF;
  // The largest tiles belong to outputs that would push the operands out of
  // the L2s (8192 x 4096 x 16384 bf16: 776 us, not 833).
  constexpr bool kStream = BM == 256;
  constexpr int kLanes = (EPI == kEpiGated ? TN / 2 : TN) / 8;   // lanes of a row, eight columns each
  const int64_t part_cols = EPI == kEpiGated ? 2 * (int64_t)a.n : a.n;
#pragma unroll
  for (int p = 0; p < TM / kPass; p++) {
#pragma unroll
    for (int j = 0; j < kPass / 16; j++)
#pragma unroll
      for (int i = 0; i < FN; i++)
        *(f32x4*)(rows + (j * 16 + (lane & 15)) * kRowF + i * 16 + (lane >> 4) * 4) = acc[i][p * (kPass / 16) + j];
    asm volatile("" ::: "memory");
#pragma unroll 1
    for (int r = lane / kLanes; r < kPass; r += 64 / kLanes) {
      const int64_t m = m0 + wm + p * kPass + r;
      const int64_t c = n0 + (EPI == kEpiGated ? wn >> 1 : wn) + (lane % kLanes) * 8;
      if (m >= a.m || c >= a.n) continue;
      const float* from = rows + r * kRowF + (lane % kLanes) * 8;
      float* part = a.part + ((int64_t)split * a.m + m) * part_cols;
      if (c + 8 <= a.n) {
        float v[8];
        *(f32x4*)v = *(const f32x4*)from;
        *(f32x4*)(v + 4) = *(const f32x4*)(from + 4);
        if constexpr (EPI == kEpiGated) {
          float u[8];
          *(f32x4*)u = *(const f32x4*)(from + kHalf);
          *(f32x4*)(u + 4) = *(const f32x4*)(from + kHalf + 4);
          if (a.splits > 1) {
            put8<float>(part, c, v);
            put8<float>(part, a.n + c, u);
          } else {
            finish8_gated<T, kStream>(a, m, c, v, u);
          }
        } else {
          if (a.splits > 1) put8<float>(part, c, v);
          else if constexpr (EPI == kEpiLinear) finish8_linear<T, kStream>(a, m, c, v);
          else put8<T, kStream>(a.c, m * a.ldc + c, v);
        }
      } else {
#pragma unroll 1
        for (int i = 0; c + i < a.n; i++) {
          if constexpr (EPI == kEpiGated) {
            if (a.splits > 1) {
              part[c + i] = from[i];
              part[a.n + c + i] = from[kHalf + i];
            } else {
              finish_gated<T>(a, m, (int)(c + i), from[i], from[kHalf + i]);
            }
          } else {
            if (a.splits > 1) part[c + i] = from[i];
            else if constexpr (EPI == kEpiLinear) finish_linear<T>(a, m, (int)(c + i), from[i]);
            else ((T*)a.c)[m * a.ldc + c + i] = (T)from[i];
          }
        }
      }
    }
    asm volatile("" ::: "memory");
  }
}

template <typename K, int OCC> __global__ __launch_bounds__(K::kThreads, OCC) void gemm_tile(GemmArgs a) {
  __shared__ __attribute__((aligned(1024))) char smem[K::kShared];
  K::run(a, blockIdx.x, smem);
}

// Two products that do not wait for each other in one launch: the first
// `blocks` blocks are the first's.
template <typename K, typename L, int OCC> __global__ __launch_bounds__(K::kThreads, OCC) void gemm_pair(GemmArgs a, GemmArgs b, unsigned blocks) {
  static_assert(K::kThreads == L::kThreads, "one block size");
  __shared__ __attribute__((aligned(1024))) char smem[K::kShared > L::kShared ? K::kShared : L::kShared];
  if (blockIdx.x < blocks) K::run(a, blockIdx.x, smem);
  else L::run(b, blockIdx.x - blocks, smem);
}

// Both gradient products, and the bias's column sums beside them.
template <typename T, typename K, typename L, int OCC>
__global__ __launch_bounds__(K::kThreads, OCC) void gemm_gradients(GemmArgs a, GemmArgs b, ColSumArgs sums, unsigned blocks_a, unsigned blocks_b) {
  static_assert(K::kThreads == L::kThreads, "one block size");
  __shared__ __attribute__((aligned(1024))) char smem[K::kShared > L::kShared ? K::kShared : L::kShared];
  if (blockIdx.x < blocks_a) K::run(a, blockIdx.x, smem);
  else if (blockIdx.x < blocks_a + blocks_b) L::run(b, blockIdx.x - blocks_a, smem);
  else col_sum_block<T>(sums, blockIdx.x - blocks_a - blocks_b, K::kThreads / 64, (float*)smem);
}

}  // namespace ringar
