// Matrix products over ragged groups of rows (one group for a dense product):
//
//   out[p, n] = sum_k A[src(p), k] W_e[n, k]        for p in group e
//
// with bf16 operands, or FP8 E4M3 operands whose blocks of 128 carry scales:
//
//   out[p, n] = sum_b sa[src(p), b] sw_e[n / 128, b] sum_{k in block b} A[src(p), k] W_e[n, k].
//
// A tile is BM rows of one group by BN weight rows; a step is 128 bytes of the
// contraction axis, i.e. 64 bf16 elements or one FP8 scale block.  Both
// operands of a step are copied into LDS by direct loads (lane i of a load
// writes 16 bytes at base + 16 i), STAGES steps in a ring, while earlier ones
// are multiplied.  A row of a step is
// 128 bytes; its 16-byte chunk j sits in slot j ^ ((row / 2) % 8), so that the
// 16 rows an MFMA operand reads fall into distinct banks.
//
// The weights are the MFMA's A operand and the rows its B operand, so a lane
// (r, q) of a 16 x 16 accumulator holds row r's outputs of weight rows
// 4q .. 4q+3 (16 bytes of fp32; bf16: see col_of), and a row's scale is one
// value per lane.
//
// Rows of the tile past the group's end, weight rows past N and chunks past K
// are loaded with an out-of-range offset: zeros, no memory traffic.
//
// FP8 sums: GT_FP8 feeds the codes to v_mfma_f32_16x16x128_f8f6f4, one
// instruction per scale block, from zero, and adds the scaled result to the
// fp32 sum.  That instruction aligns its 128 products before it adds them and
// keeps about 16 bits below the largest (measured: relative error 1.5e-5 of a
// block's sum for bell-shaped codes, 5e-5 for uniform bytes; the 32-long FP8
// instruction is no better): 1/100 of a bf16 output's half step, but far from
// fp32's.  GT_FP8X converts the codes to bf16 (exact) and uses the bf16
// instruction, whose sums are as good as fp32's (7e-8), at half the rate; it
// serves fp32 outputs and sums whose errors would show in what is made of them
// (fp8_ffn).
//
// What bounds it.  Few rows per group: the weights' read (64 tokens' top 8 of
// 128 bf16 experts of 2048 x 1536, 32-row tiles: 136 us, 5.9 TB/s; a plain read
// reaches 6.2 to 6.5).  Many rows: the 256 x 256 tile takes 136 us for 8192 x
// 4096 x 4096 in FP8, 2.0 PFLOP/s (a library product of that size class 3.1);
// its matrix instructions with the scaled additions between them take 86 us
// alone, with the LDS reads 95 to 105, and its loads, from the L2, 72: what is
// left is how far the two overlap.  Ragged groups of 192 rows on average in
// between: 1.35 ms for 4.7 GB of operands, 3.5 TB/s and 1.2 PFLOP/s.
#pragma once

#include <type_traits>
#include <utility>

#include "ft_internal.hpp"
#include "fp8_util.hpp"

namespace ft {

enum { GT_BF16 = 0, GT_FP8 = 1, GT_FP8X = 2 };  // operand type / instruction
// outputs: the products in fp32 or bf16; silu(gate) * up in fp32, or quantized by 1 x 128 blocks
enum { GE_F32 = 0, GE_BF16 = 1, GE_GLU = 2, GE_GLUQ = 3 };
constexpr bool is_glu(int ep) { return ep == GE_GLU || ep == GE_GLUQ; }

// lambdas that hold register arrays: a call would put those into memory
#define FT_INLINE __attribute__((always_inline))

constexpr int kStepBytes = 128;  // bytes of the contraction axis per step

struct GroupArgs {
  const uint8_t *A;               // operand rows
  int64_t lda;                    // bytes from row to row
  const float *As;                // FP8: scales [rows of A, KB]
  const uint8_t *pool;            // weights of group e: pool + slot * expert_bytes + off_w*
  uint64_t expert_bytes;
  const int32_t *slots;           // NULL: slot e
  int n_slots;
  const uint8_t *shared_blob;     // one more group of T rows (NULL: none)
  uint64_t off_w0, off_w1, off_s0, off_s1;  // GLU: 0 = gate, 1 = up
  int64_t ldw;                    // bytes from weight row to weight row
  int Kb;                         // bytes of a row that are contracted (a multiple of 16)
  int KB;                         // scale blocks per row
  int N;                          // outputs per row (GLU: of one matrix)
  const int32_t *offsets;         // [E+1]; NULL: one group of all rows
  int E, rows;                    // groups, rows behind them
  int T, k;
  const int32_t *sorted_rows;     // A row of row p is sorted_rows[p] / k (NULL: p)
  int64_t a_rows;                 // rows of A that sorted_rows may name
  int a_shared0;                  // first A row of the shared group
  void *out;
  int64_t ldo;                    // elements
  float *out_scales;              // GE_GLUQ: scales of the rows in out, [rows, ceil(N / 128)]
  float *out_shared;              // rows of the shared group (NULL: behind the others in out)
  int n_ntiles;
};

// Rows of group e: first row and count, held inside [0, rows] whatever the offsets say.
__device__ __forceinline__ int group_rows(const GroupArgs &a, int e, int *lo) {
  if (e >= a.E) {
    *lo = 0;
    return 0;
  }
  if (a.offsets == nullptr) {
    *lo = 0;
    return a.rows;
  }
  const int b = max(0, min(a.offsets[e], a.rows)), c = max(0, min(a.offsets[e + 1], a.rows));
  *lo = b;
  return max(0, c - b);
}

struct GroupItem {
  int nt;    // weight tile
  int e;     // group (E: the shared one)
  int lo;    // first row of the group
  int row0;  // first row of the tile inside the group
  int m;     // rows of the tile
};

// This workgroup's tile.  Tiles are group-major; a group's tiles come in columns
// of kColumn weight tiles, row tile by row tile.  Each XCD takes a contiguous
// range of those present (block ids go round robin over the 8 XCDs), so what
// runs on one XCD at a time is a block of a few row tiles by kColumn weight
// tiles, and its L2 serves every operand byte several times.
constexpr int kColumn = 8;

__device__ __forceinline__ void tile_of(int local, int tiles, int NT, int *nt, int *mt) {
  const int c = local / (tiles * kColumn), rest = local - c * tiles * kColumn, w = min(kColumn, NT - c * kColumn);
  *mt = rest / w;
  *nt = c * kColumn + rest % w;
}

template <int THREADS, int BM>
__device__ __forceinline__ bool group_item(const GroupArgs &a, GroupItem *it) {
  constexpr int NW = THREADS / 64;
  __shared__ int s_cnt[NW];
  __shared__ int s_hit[4];
  const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63;
  const int NT = a.n_ntiles;
  // thread t counts the tiles of groups t * per_thread .. and an exclusive scan
  // over the threads finds the one whose range holds the item
  const int per_thread = (a.E + THREADS - 1) / THREADS, e0 = tid * per_thread;
  int mine = 0;
  for (int i = 0; i < per_thread; ++i) {
    int lo;
    mine += (group_rows(a, e0 + i, &lo) + BM - 1) / BM;
  }
  const int incl = wave_incl_scan_i32(mine);
  if (lane == 63) s_cnt[wave] = incl;
  if (tid == 0) s_hit[0] = -1;  // offsets that are no offsets may leave an item without a group
  __syncthreads();
  int total = 0, first = incl - mine;
#pragma unroll
  for (int w = 0; w < NW; ++w) {
    if (w < wave) first += s_cnt[w];
    total += s_cnt[w];
  }
  const int shared_tiles = a.shared_blob != nullptr ? (a.T + BM - 1) / BM : 0;
  const int n_items = (total + shared_tiles) * NT;
  const int per = (n_items + 7) / 8;
  const int b = int(blockIdx.x);
  const int item = (b % 8) * per + b / 8;
  if (b / 8 >= per || item >= n_items) return false;
  if (item >= total * NT) {
    const int local = item - total * NT;
    int mt;
    tile_of(local, shared_tiles, NT, &it->nt, &mt);
    it->e = a.E;
    it->lo = 0;
    it->row0 = mt * BM;
    it->m = min(BM, a.T - it->row0);
    return true;
  }
  if (item >= first * NT && item < (first + mine) * NT) {
    int local = item - first * NT;
    for (int i = 0; i < per_thread; ++i) {
      int lo;
      const int m = group_rows(a, e0 + i, &lo), n = (m + BM - 1) / BM * NT;
      if (local < n) {
        s_hit[0] = e0 + i;
        s_hit[1] = lo;
        s_hit[2] = m;
        s_hit[3] = local;
        break;
      }
      local -= n;
    }
  }
  __syncthreads();
  it->e = __builtin_amdgcn_readfirstlane(s_hit[0]);
  if (it->e < 0) return false;
  it->lo = __builtin_amdgcn_readfirstlane(s_hit[1]);
  const int m = __builtin_amdgcn_readfirstlane(s_hit[2]), local = __builtin_amdgcn_readfirstlane(s_hit[3]);
  const int tiles = (m + BM - 1) / BM;
  int mt;
  tile_of(local, tiles, NT, &it->nt, &mt);
  it->row0 = mt * BM;
  it->m = min(BM, m - it->row0);
  return true;
}

// Lane `lane`'s value, to every lane.
__device__ __forceinline__ float lane_value(float v, int lane) {
  return __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, v), lane));
}

// Direct loads: lane i's 16 (4) bytes at base + off + step go to LDS address
// dst + 16 i (4 i).  Written as assembly, without outputs, because the compiler
// cannot tell one step's buffer from another's when the ring's position is a
// run-time value: it would wait for all loads in flight before every LDS read.
// The kernel counts them itself (wait_vmcnt before the barrier that publishes
// a step); the compiler's own waits only see fewer loads than there are, so
// they wait for more.
__device__ __forceinline__ void lds_load16(u32x4 r, uint32_t dst, uint32_t off, uint32_t step) {
  asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tbuffer_load_dwordx4 %0, %1, %3 offen lds" ::"v"(off), "s"(r), "s"(dst), "s"(step)
               : "memory");
}
__device__ __forceinline__ void lds_load4(u32x4 r, uint32_t dst, uint32_t off, uint32_t step) {
  asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tbuffer_load_dword %0, %1, %3 offen lds" ::"v"(off), "s"(r), "s"(dst), "s"(step)
               : "memory");
}
// The descriptor of make_rsrc as four scalar words.
__device__ __forceinline__ u32x4 rsrc_words(const void *base, uint32_t bytes) {
  const uint64_t p = reinterpret_cast<uint64_t>(base);
  return u32x4{uint32_t(p), uint32_t(p >> 32) & 0xffffu, bytes, 0x00020000u};
}
__device__ __forceinline__ uint32_t lds_address(const void *p) {
  return uint32_t(reinterpret_cast<uintptr_t>((__attribute__((address_space(3))) const void *)p));
}

__device__ __forceinline__ f32x4 fp8_mfma(u32x4 wl, u32x4 wh, u32x4 al, u32x4 ah) {
  const i32x8 w = __builtin_bit_cast(i32x8, __builtin_shufflevector(wl, wh, 0, 1, 2, 3, 4, 5, 6, 7));
  const i32x8 x = __builtin_bit_cast(i32x8, __builtin_shufflevector(al, ah, 0, 1, 2, 3, 4, 5, 6, 7));
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(w, x, f32x4{0.f, 0.f, 0.f, 0.f}, 0, 0, 0, 0, 0, 0);
}

// 16 codes of either operand per lane: 64 products, as bf16
__device__ __forceinline__ f32x4 fp8x_mfma(u32x4 w, u32x4 x, f32x4 p) {
  p = mfma16(fp8x8_to_bf16x8(w[0], w[1]), fp8x8_to_bf16x8(x[0], x[1]), p);
  return mfma16(fp8x8_to_bf16x8(w[2], w[3]), fp8x8_to_bf16x8(x[2], x[3]), p);
}

template <int TY, int EP, int WM, int WN, int MT, int NT, int STAGES>
struct GroupTile {
  static constexpr int WAVES = WM * WN, THREADS = WAVES * 64;
  static constexpr int BM = WM * MT * 16, BN = WN * NT * 16;
  static constexpr int AL = BM / 8 / WAVES, WL = BN / 8 / WAVES;  // direct loads per wave and step
  static constexpr bool FP8 = TY != GT_BF16;
  static constexpr bool GLU = is_glu(EP);
  static constexpr int LOADS = AL + WL + (FP8 ? 1 : 0);
  static constexpr int NCOL = GLU ? BN / 2 : BN;  // outputs per row of a tile
  static constexpr int STAGE_BYTES = (BM + BN) * kStepBytes + (FP8 ? WAVES * 256 : 0);
  static_assert(AL >= 1 && WL >= 1 && AL * WAVES * 8 == BM && WL * WAVES * 8 == BN, "whole direct loads");
  static_assert(NT % 2 == 0 && (!GLU || NT == 4), "tile pairs");
  static_assert(BM / WAVES <= 64, "one row scale per lane");


  // First of the loads that go with row tile i of mtr: evenly over the tiles, or
  // over the first half of them where the ring holds only one step ahead
  static constexpr int load_at(int i, int mtr) {
    const int n = i * LOADS * (STAGES == 2 ? 2 : 1) / mtr;
    return n < LOADS ? n : LOADS;
  }

  // Output of weight row p of the tile's LDS order, relative to the tile's first.
  // fp32: as they come, 4 outputs (16 bytes) per lane and 64 bytes per row and
  // store.  bf16 and codes: pairs of 16-row tiles interleaved by 4, so that a
  // lane's two accumulators are 8 consecutive outputs.
  static __device__ __forceinline__ int col_of(int p) {
    const int pl = p % (NT * 16);
    const int f = EP == GE_F32 || EP == GE_GLU ? pl & 31 : 8 * ((pl & 15) >> 2) + 4 * ((pl >> 4) & 1) + (pl & 3);
    if (GLU) return p / (NT * 16) * 32 + f;
    return p / (NT * 16) * (NT * 16) + (pl & ~31) + f;
  }

  template <int MTR>
  static __device__ __forceinline__ void body(const GroupArgs &a, uint8_t *L, const GroupItem &it, const uint8_t *blob) {
    const int tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid >> 6), lane = tid & 63;
    const int r = lane & 15, q = lane >> 4, wm = wave % WM, wn = wave / WM;
    const bool shared = it.e == a.E;
    const int n0 = it.nt * NCOL;
    const int nk = cdiv(a.Kb, kStepBytes);

    // ---- sources of the direct loads: a lane's offset inside its operand is
    // fixed, the step is the instruction's scalar offset
    const bool gather = a.sorted_rows != nullptr && !shared;
    const int64_t a_first = gather ? 0 : int64_t(shared ? a.a_shared0 : it.lo) + it.row0;
    const int64_t a_count = gather ? a.a_rows : it.m;
    // A row of the tile's row rr, relative to a_first; -1: none
    auto a_row = [&](int rr) -> int {
      if (rr >= it.m) return -1;
      if (!gather) return rr;
      const uint32_t s = uint32_t(a.sorted_rows[it.lo + it.row0 + rr]) / uint32_t(a.k);
      return s < uint32_t(a.a_rows) ? int(s) : -1;  // a negative entry: above every token
    };
    const uint8_t *abase = a.A + a_first * a.lda;
    const uint32_t abytes = uint32_t((a_count - 1) * a.lda + a.Kb);
    const uint8_t *wbase = blob + a.off_w0 + uint64_t(n0) * uint64_t(a.ldw);
    const uint64_t to_up = GLU ? a.off_w1 - a.off_w0 : 0;  // GLU: from gate's rows to up's
    const uint32_t wbytes = uint32_t((min(NCOL, a.N - n0) - 1) * a.ldw + a.Kb);
    uint32_t aoff[AL], woff[WL];
#pragma unroll
    for (int t = 0; t < AL; ++t) {
      const int rr = (wave * AL + t) * 8 + (lane >> 3), src = a_row(rr);
      aoff[t] = src >= 0 ? uint32_t(src) * uint32_t(a.lda) + uint32_t(((lane & 7) ^ ((rr >> 1) & 7)) * 16) : kOOB;
    }
#pragma unroll
    for (int t = 0; t < WL; ++t) {
      const int p = (wave * WL + t) * 8 + (lane >> 3), n = col_of(p);
      woff[t] = n0 + n < a.N ? uint32_t(n) * uint32_t(a.ldw) + uint32_t(((lane & 7) ^ ((p >> 1) & 7)) * 16) : kOOB;
    }
    // the last step of a K that is no multiple of 128 bytes: chunks past it load zeros
    const int tail = a.Kb % kStepBytes;
    auto cut = [&]() {
#pragma unroll
      for (int t = 0; t < AL; ++t)
        if (((lane & 7) ^ ((((wave * AL + t) * 8 + (lane >> 3)) >> 1) & 7)) * 16 >= tail) aoff[t] = kOOB;
#pragma unroll
      for (int t = 0; t < WL; ++t)
        if (((lane & 7) ^ ((((wave * WL + t) * 8 + (lane >> 3)) >> 1) & 7)) * 16 >= tail) woff[t] = kOOB;
    };
    // row scales: the lanes of a wave take the rows that it loads, one value per
    // step.  Weight scales are one value per step for the whole wave (GLU: per
    // matrix): lane l holds those of 64 steps, and a step reads its lane.
    uint32_t soff = kOOB;
    const float *swp0 = nullptr, *swp1 = nullptr;
    if constexpr (FP8) {
      const int src = lane < BM / WAVES ? a_row(wave * (BM / WAVES) + lane) : -1;
      if (src >= 0) soff = uint32_t(src) * uint32_t(a.KB) * 4u;
      const int nb = min((n0 + wn * (GLU ? 32 : NT * 16)) / 128, cdiv(a.N, 128) - 1);
      swp0 = reinterpret_cast<const float *>(blob + a.off_s0) + int64_t(nb) * a.KB;
      if (GLU) swp1 = reinterpret_cast<const float *>(blob + a.off_s1) + int64_t(nb) * a.KB;
    }
    const float *sbase = FP8 ? a.As + a_first * a.KB : nullptr;
    const uint32_t ldsb = __builtin_amdgcn_readfirstlane(lds_address(L));
    // Step c's loads, into the ring at byte `at`.  A step past the end loads
    // nothing (empty buffers, so that every step has the same instructions in
    // flight).
    struct Loads {
      u32x4 ares, wres[GLU ? 2 : 1], sres;
      uint32_t at, st, ss;
    };
    auto plan = [&](int c, uint32_t at) FT_INLINE {
      const bool live = c < nk;
      if (tail != 0 && c == nk - 1) cut();
      Loads l;
      l.at = ldsb + at;
      l.st = live ? uint32_t(c) * kStepBytes : 0u;
      l.ss = live ? uint32_t(c) * 4u : 0u;
      l.ares = rsrc_words(abase, live ? abytes : 0u);
      l.wres[0] = rsrc_words(wbase, live ? wbytes : 0u);
      if constexpr (GLU) l.wres[1] = rsrc_words(wbase + to_up, live ? wbytes : 0u);
      if constexpr (FP8) l.sres = rsrc_words(sbase, live ? uint32_t(a_count * a.KB * 4) : 0u);
      return l;
    };
    auto load = [&](const Loads &l, int t) FT_INLINE {  // the t-th of them, 0 .. LOADS - 1
      const bool up = GLU && ((wave * WL + t) * 8) % (NT * 16) >= 32;
      if (t < WL)
        lds_load16(up ? l.wres[GLU] : l.wres[0], l.at + BM * kStepBytes + (wave * WL + t) * 1024, woff[t], l.st);
      else if (t < WL + AL)
        lds_load16(l.ares, l.at + (wave * AL + t - WL) * 1024, aoff[t - WL], l.st);
      else
        lds_load4(l.sres, l.at + (BM + BN) * kStepBytes + wave * 256, soff, l.ss);
    };

    f32x4 acc[MTR][NT];
#pragma unroll
    for (int i = 0; i < MTR; ++i)
#pragma unroll
      for (int j = 0; j < NT; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};

    const int sw = (r >> 1) & 7;
    const int lo16 = r * kStepBytes + ((q ^ sw) << 4), hi16 = r * kStepBytes + (((4 + q) ^ sw) << 4);

    constexpr int kScaleSteps = 64;
    float swv0 = 0.f, swv1 = 0.f;
    int sw_first = 0;
    auto load_weight_scales = [&](int c) {
      sw_first = c;
      const int b = min(c + lane, a.KB - 1);
      swv0 = swp0[b];
      if (GLU) swv1 = swp1[b];
    };

    // ---- operands of one step: the weights' in registers for the whole step, the
    // rows' one tile ahead of its products
    struct Frag {
      u32x4 wl[NT], wh[NT], al[2], ah[2];
      float sa[2];
    };
    Frag f;
    auto read_w = [&](const uint8_t *buf) FT_INLINE {
      const uint8_t *wb = buf + (BM + wn * NT * 16) * kStepBytes;
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        f.wl[j] = *reinterpret_cast<const u32x4 *>(wb + j * 16 * kStepBytes + lo16);
        f.wh[j] = *reinterpret_cast<const u32x4 *>(wb + j * 16 * kStepBytes + hi16);
      }
    };
    auto read_a = [&](int i, const uint8_t *buf) FT_INLINE {
      const uint8_t *ab = buf + (i * WM + wm) * 16 * kStepBytes;
      f.al[i & 1] = *reinterpret_cast<const u32x4 *>(ab + lo16);
      f.ah[i & 1] = *reinterpret_cast<const u32x4 *>(ab + hi16);
      if constexpr (FP8) {
        const float *sc = reinterpret_cast<const float *>(buf + (BM + BN) * kStepBytes);
        const int row = (i * WM + wm) * 16 + r;
        f.sa[i & 1] = sc[row / (BM / WAVES) * 64 + row % (BM / WAVES)];
      }
    };
    // The products of step c, and the loads of a later step among them: issued
    // in one go, they would hold up the wave (a CU takes 64 bytes of load a
    // clock, so a step's loads take about as long as its products).  FP8
    // additions follow the products they add; the SIMD's other wave multiplies
    // meanwhile.
    auto compute = [&](int c, const uint8_t *buf, const Loads &next) FT_INLINE {
      float sw0 = 0.f, sw1 = 0.f;
      if constexpr (FP8) {
        sw0 = lane_value(swv0, c - sw_first);
        if (GLU) sw1 = lane_value(swv1, c - sw_first);
      }
      read_a(0, buf);
      read_w(buf);
#pragma unroll
      for (int i = 0; i < MTR; ++i) {
        if (i + 1 < MTR) read_a(i + 1, buf);
#pragma unroll
        for (int t = load_at(i, MTR); t < load_at(i + 1, MTR); ++t) load(next, t);
        const u32x4 xl = f.al[i & 1], xh = f.ah[i & 1];
        f32x4 p[NT];
#pragma unroll
        for (int j = 0; j < NT; ++j) {
          if constexpr (!FP8) {
            acc[i][j] = mfma16(as_bf16x8(f.wl[j]), as_bf16x8(xl), acc[i][j]);
            acc[i][j] = mfma16(as_bf16x8(f.wh[j]), as_bf16x8(xh), acc[i][j]);
          } else if constexpr (TY == GT_FP8) {
            p[j] = fp8_mfma(f.wl[j], f.wh[j], xl, xh);
          } else {
            p[j] = fp8x_mfma(f.wh[j], xh, fp8x_mfma(f.wl[j], xl, f32x4{0.f, 0.f, 0.f, 0.f}));
          }
        }
        if constexpr (FP8) {
          const float s0 = f.sa[i & 1] * sw0, s1 = GLU ? f.sa[i & 1] * sw1 : s0;
#pragma unroll
          for (int j = 0; j < NT; ++j) {
            const float s = GLU && j >= NT / 2 ? s1 : s0;
#pragma unroll
            for (int v = 0; v < 4; ++v) acc[i][j][v] = fmaf(p[j][v], s, acc[i][j][v]);
          }
        }
        // here, and not behind the products of all row tiles, which would all stay live
#pragma unroll
        for (int j = 0; j < NT; ++j) asm volatile("" : "+v"(acc[i][j]));
        __builtin_amdgcn_sched_barrier(0);
      }
    };

    // ---- a ring of STAGES steps: at turn c the loads of step c have landed and
    // every wave is done with step c - 1, whose buffer takes step c + STAGES - 1
    if constexpr (FP8) {
      load_weight_scales(0);
      wait_vmcnt<0>();
    }
#pragma unroll
    for (int p = 0; p < STAGES - 1; ++p) {
      const Loads l = plan(p, p * STAGE_BYTES);
#pragma unroll
      for (int t = 0; t < LOADS; ++t) load(l, t);
    }
    uint32_t at = 0, put = (STAGES - 1) * STAGE_BYTES;  // of step c, of step c + STAGES - 1
    for (int c = 0; c < nk; ++c) {
      if (FP8 && c - sw_first == kScaleSteps) {
        load_weight_scales(c);
        wait_vmcnt<0>();
      }
      wait_vmcnt<(STAGES - 2) * LOADS>();
      lds_barrier();
      compute(c, L + at, plan(c + STAGES - 1, put));
      at = at == (STAGES - 1) * STAGE_BYTES ? 0 : at + STAGE_BYTES;
      put = put == (STAGES - 1) * STAGE_BYTES ? 0 : put + STAGE_BYTES;
    }
    wait_vmcnt<0>();

    // ---- epilogue
    const int64_t orow0 = int64_t(shared ? a.rows : it.lo) + it.row0;
    if constexpr (EP == GE_GLUQ) {
      // A tile holds whole 128-blocks of its hidden rows, 32 columns in each of 4
      // waves: their largest magnitudes meet in LDS.  silu(gate) * up goes back
      // into gate's registers meanwhile.
      static_assert(NCOL == 128 && WN == 4, "one block per row and tile");
      __shared__ uint32_t s_max[4][BM];
#pragma unroll
      for (int i = 0; i < MTR; ++i) {
        uint32_t m = 0;
#pragma unroll
        for (int u = 0; u < 8; ++u) {
          float &g = reinterpret_cast<float *>(&acc[i][u / 4])[u % 4];
          g = silu(g) * acc[i][2 + u / 4][u % 4];
          m = max(m, __float_as_uint(g) & 0x7fffffffu);
        }
        m = max(m, uint32_t(__shfl_xor(int(m), 16)));
        m = max(m, uint32_t(__shfl_xor(int(m), 32)));
        if (q == 0) s_max[wn][(i * WM + wm) * 16 + r] = m;
      }
      __syncthreads();
#pragma unroll
      for (int i = 0; i < MTR; ++i) {
        const int rr = (i * WM + wm) * 16 + r, n = n0 + wn * 32 + 8 * q;
        if (rr >= it.m) continue;
        const Fp8Scale sc = fp8_scale(max(max(s_max[0][rr], s_max[1][rr]), max(s_max[2][rr], s_max[3][rr])));
        float v[8];
#pragma unroll
        for (int u = 0; u < 8; ++u) v[u] = acc[i][u / 4][u % 4];
        if (n < a.N) *reinterpret_cast<u32x2 *>(static_cast<uint8_t *>(a.out) + (orow0 + rr) * a.ldo + n) = fp8_codes8(v, sc.inv);
        if (wn == 0 && q == 0) a.out_scales[(orow0 + rr) * cdiv(a.N, 128) + it.nt] = sc.scale;
      }
    } else {
#pragma unroll
      for (int i = 0; i < MTR; ++i) {
        const int rr = (i * WM + wm) * 16 + r;
        if (rr >= it.m) continue;
        if constexpr (EP == GE_BF16) {
          uint16_t *o = static_cast<uint16_t *>(a.out) + (orow0 + rr) * a.ldo;
#pragma unroll
          for (int jj = 0; jj < NT / 2; ++jj) {
            float v[8];
#pragma unroll
            for (int u = 0; u < 8; ++u) v[u] = acc[i][2 * jj + u / 4][u % 4];
            store8(o, n0 + wn * NT * 16 + 32 * jj + 8 * q, a.N, v, a.ldo % 8 == 0);
          }
        } else {
          const bool own = !GLU && shared && a.out_shared != nullptr;
          float *o = own ? a.out_shared + int64_t(it.row0 + rr) * a.ldo : static_cast<float *>(a.out) + (orow0 + rr) * a.ldo;
#pragma unroll
          for (int j = 0; j < (GLU ? NT / 2 : NT); ++j) {
            f32x4 v = acc[i][j];
            if constexpr (GLU) {
#pragma unroll
              for (int u = 0; u < 4; ++u) v[u] = silu(v[u]) * acc[i][2 + j][u];
            }
            store4(o, n0 + wn * (GLU ? 32 : NT * 16) + 16 * j + 4 * q, a.N, v, a.ldo % 4 == 0);
          }
        }
      }
    }
  }

  // Four (eight) consecutive outputs from n on, those below N.
  static __device__ __forceinline__ void store4(float *o, int n, int N, f32x4 v, bool vec) {
    if (vec && n + 4 <= N) {
      *reinterpret_cast<f32x4 *>(o + n) = v;
      return;
    }
#pragma unroll
    for (int u = 0; u < 4; ++u)
      if (n + u < N) o[n + u] = v[u];
  }
  static __device__ __forceinline__ void store8(uint16_t *o, int n, int N, const float (&v)[8], bool vec) {
    uint32_t d[4];
#pragma unroll
    for (int u = 0; u < 4; ++u)
      d[u] = uint32_t(f32_to_bf16_rne(v[2 * u])) | (uint32_t(f32_to_bf16_rne(v[2 * u + 1])) << 16);
    if (vec && n + 8 <= N) {
      st16(o + n, u32x4{d[0], d[1], d[2], d[3]});
      return;
    }
#pragma unroll
    for (int u = 0; u < 8; ++u)
      if (n + u < N) o[n + u] = uint16_t(d[u / 2] >> (16 * (u & 1)));
  }

  // The rows of a group whose weights are not resident.
  static __device__ __forceinline__ void fill_nan(const GroupArgs &a, const GroupItem &it) {
    const int n0 = it.nt * NCOL, w = min(NCOL, a.N - n0);
    if constexpr (EP == GE_GLUQ) return;  // the next stage writes their NaN without reading these
    for (int u = threadIdx.x; u < it.m * w; u += THREADS) {
      const int64_t at = (int64_t(it.lo) + it.row0 + u / w) * a.ldo + n0 + u % w;
      if (EP == GE_BF16)
        static_cast<uint16_t *>(a.out)[at] = 0x7fc0;
      else
        static_cast<float *>(a.out)[at] = __builtin_nanf("");
    }
  }

  static __device__ __forceinline__ void run(const GroupArgs &a, uint8_t *L) {
    GroupItem it;
    if (!group_item<THREADS, BM>(a, &it)) return;
    const uint8_t *blob = a.shared_blob;
    if (it.e < a.E) {
      const int slot = table_slot(a.slots, it.e, a.n_slots);
      if (slot == FT_SLOT_SKIP) return;
      if (slot < 0) {
        fill_nan(a, it);
        return;
      }
      blob = a.pool + uint64_t(slot) * a.expert_bytes;
    }
    // only the row tiles that hold rows
    const int mt = (it.m + WM * 16 - 1) / (WM * 16);
    if constexpr (MT >= 8) {
      if (mt > 6) return body<8>(a, L, it, blob);
      if (mt > 4) return body<6>(a, L, it, blob);
    }
    if constexpr (MT >= 4) {
      if (mt > 3) return body<4>(a, L, it, blob);
      if (mt > 2) return body<3>(a, L, it, blob);
    }
    if constexpr (MT >= 2)
      if (mt > 1) return body<2>(a, L, it, blob);
    body<1>(a, L, it, blob);
  }
};

}  // namespace ft
