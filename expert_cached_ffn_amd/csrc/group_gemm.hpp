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
// writes 16 bytes at base + 16 i), STAGES steps in a ring.  A row of a step is
// 128 bytes; its 16-byte chunk j sits in slot j ^ ((row / 2) % 8), so that the
// 16 rows an MFMA operand reads fall into distinct banks.
//
// The weights are the MFMA's A operand and the rows its B operand, so a lane
// (r, q) of a 16 x 16 accumulator holds row r's outputs of weight rows
// 4q .. 4q+3.  The weight rows of a pair of tiles are laid out in LDS such
// that a lane's two accumulators are 8 consecutive outputs (one 16-byte bf16
// store), and a row's scale is one value per lane.
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
// serves fp32 outputs.
#pragma once

#include <type_traits>
#include <utility>

#include "ft_internal.hpp"
#include "fp8_util.hpp"

namespace ft {

enum { GT_BF16 = 0, GT_FP8 = 1, GT_FP8X = 2 };  // operand type / instruction
enum { GE_OUT = 0, GE_GLU = 1 };                // epilogue: the products; silu(gate) * up (fp32)

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
  int out_bf16;
  int64_t ldo;                    // elements
  float *out_shared;              // rows of the shared group (NULL: behind the others in out)
  int n_ntiles, n_mtiles;
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

// This workgroup's tile.  Tiles are group-major and weight-tile major within a
// group (the row tiles of one weight tile are neighbours), and each XCD takes a
// contiguous range of those present: a group's rows and weights then sit in
// one XCD's L2.  Block ids go round robin over the 8 XCDs.
template <int THREADS, int BM>
__device__ bool group_item(const GroupArgs &a, GroupItem *it) {
  constexpr int NW = THREADS / 64;
  __shared__ int s_cnt[NW];
  __shared__ int s_hit[4];
  const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63;
  const int NT = a.n_ntiles;
  int total = 0, lo0 = 0, m0 = 0;
  for (int c0 = 0; c0 < a.E; c0 += THREADS) {
    int lo = 0;
    const int m = group_rows(a, c0 + tid, &lo);
    if (c0 == 0) {
      lo0 = lo;
      m0 = m;
    }
    const int v = wave_sum_i32((m + BM - 1) / BM);
    if (lane == 0) s_cnt[wave] = v;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < NW; ++w) total += s_cnt[w];
    __syncthreads();
  }
  const int shared_tiles = a.shared_blob != nullptr ? (a.T + BM - 1) / BM : 0;
  const int n_items = (total + shared_tiles) * NT;
  const int per = (n_items + 7) / 8;
  const int b = int(blockIdx.x);
  const int item = (b % 8) * per + b / 8;
  if (b / 8 >= per || item >= n_items) return false;
  if (item >= total * NT) {
    const int local = item - total * NT;
    it->nt = local / shared_tiles;
    it->e = a.E;
    it->lo = 0;
    it->row0 = (local % shared_tiles) * BM;
    it->m = min(BM, a.T - it->row0);
    return true;
  }
  int base = 0;
  for (int c0 = 0; c0 < a.E; c0 += THREADS) {
    int lo = lo0;
    const int m = c0 == 0 ? m0 : group_rows(a, c0 + tid, &lo);
    const int tiles = (m + BM - 1) / BM;
    const int incl = wave_incl_scan_i32(tiles * NT);
    if (lane == 63) s_cnt[wave] = incl;
    __syncthreads();
    int before = base;
#pragma unroll
    for (int w = 0; w < NW; ++w) {
      if (w < wave) before += s_cnt[w];
      base += s_cnt[w];
    }
    const int first = before + incl - tiles * NT;
    if (item >= first && item < before + incl) {
      s_hit[0] = c0 + tid;
      s_hit[1] = lo;
      s_hit[2] = m;
      s_hit[3] = item - first;
    }
    __syncthreads();
    if (item < base) break;
  }
  it->e = __builtin_amdgcn_readfirstlane(s_hit[0]);
  it->lo = __builtin_amdgcn_readfirstlane(s_hit[1]);
  const int m = __builtin_amdgcn_readfirstlane(s_hit[2]), local = __builtin_amdgcn_readfirstlane(s_hit[3]);
  const int tiles = (m + BM - 1) / BM;
  it->nt = local / tiles;
  it->row0 = (local % tiles) * BM;
  it->m = min(BM, m - it->row0);
  return true;
}

__device__ __forceinline__ void lds_load16(rsrc_t r, uint8_t *dst, uint32_t off) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (__attribute__((address_space(3))) void *)dst, 16, off, 0, 0, 0);
}

template <int TY, int EP, int WM, int WN, int MT, int NT, int STAGES>
struct GroupTile {
  static constexpr int WAVES = WM * WN, THREADS = WAVES * 64;
  static constexpr int BM = WM * MT * 16, BN = WN * NT * 16;
  static constexpr int AL = BM / 8 / WAVES, WL = BN / 8 / WAVES;  // direct loads per wave and step
  static constexpr bool FP8 = TY != GT_BF16;
  static constexpr int LOADS = AL + WL + (FP8 ? 1 : 0);
  static constexpr int NCOL = EP == GE_GLU ? BN / 2 : BN;  // outputs per row of a tile
  static constexpr int STAGE_BYTES = (BM + BN) * kStepBytes + (FP8 ? WAVES * 256 : 0);
  static_assert(AL >= 1 && WL >= 1 && AL * WAVES * 8 == BM && WL * WAVES * 8 == BN, "whole direct loads");
  static_assert(NT % 2 == 0 && (EP != GE_GLU || (NT == 4 && WL * 8 <= 32 && 32 % (WL * 8) == 0)), "tile pairs");
  static_assert(BM / WAVES <= 32 && NCOL <= 4096, "scale slots");

  struct Ring {
    uint8_t *b[STAGES];
  };

  // Output of weight row p of the tile's LDS order, relative to the tile's first:
  // pairs of 16-row tiles are interleaved by 4 so that a lane's two
  // accumulators are consecutive.
  static __device__ __forceinline__ int col_of(int p) {
    const int pl = p % (NT * 16), f = 8 * ((pl & 15) >> 2) + 4 * ((pl >> 4) & 1) + (pl & 3);
    if (EP == GE_GLU) return p / (NT * 16) * 32 + f;
    return p / (NT * 16) * (NT * 16) + (pl & ~31) + f;
  }

  template <int MTR>
  static __device__ __forceinline__ void body(const GroupArgs &a, const Ring &L, const GroupItem &it, const uint8_t *blob) {
    const int tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid >> 6), lane = tid & 63;
    const int r = lane & 15, q = lane >> 4, wm = wave % WM, wn = wave / WM;
    const bool shared = it.e == a.E;
    const int n0 = it.nt * NCOL;
    const int nk = cdiv(a.Kb, kStepBytes);

    // ---- sources of the direct loads
    const bool gather = a.sorted_rows != nullptr && !shared;
    const int64_t a_first = gather ? 0 : int64_t(shared ? a.a_shared0 : it.lo) + it.row0;
    const rsrc_t ares = make_rsrc(a.A + a_first * a.lda, uint32_t(((gather ? a.a_rows : it.m) - 1) * a.lda + a.Kb));
    // A row of the tile's row rr, relative to a_first; -1: none
    auto a_row = [&](int rr) -> int {
      if (rr >= it.m) return -1;
      if (!gather) return rr;
      const uint32_t s = uint32_t(a.sorted_rows[it.lo + it.row0 + rr]) / uint32_t(a.k);
      return s < uint32_t(a.a_rows) ? int(s) : -1;  // a negative entry: above every token
    };
    uint32_t aoff[AL], woff[WL];
    int abyte[AL], wbyte[WL];
#pragma unroll
    for (int t = 0; t < AL; ++t) {
      const int rr = (wave * AL + t) * 8 + (lane >> 3), src = a_row(rr);
      abyte[t] = ((lane & 7) ^ ((rr >> 1) & 7)) * 16;
      aoff[t] = src >= 0 ? uint32_t(src) * uint32_t(a.lda) + uint32_t(abyte[t]) : kOOB;
    }
    const bool up = EP == GE_GLU && ((wave * WL * 8) % (NT * 16)) >= 32;
    const rsrc_t wres = make_rsrc(blob + (up ? a.off_w1 : a.off_w0) + uint64_t(n0) * uint64_t(a.ldw),
                                  uint32_t((min(NCOL, a.N - n0) - 1) * a.ldw + a.Kb));
#pragma unroll
    for (int t = 0; t < WL; ++t) {
      const int p = (wave * WL + t) * 8 + (lane >> 3), n = col_of(p);
      wbyte[t] = ((lane & 7) ^ ((p >> 1) & 7)) * 16;
      woff[t] = n0 + n < a.N ? uint32_t(n) * uint32_t(a.ldw) + uint32_t(wbyte[t]) : kOOB;
    }
    // scales: lanes 0..31 of a wave take the rows it loads, lanes 32.. the
    // weights' blocks of the tile (GLU: gate's, then up's); the others reread
    // a value that is there
    constexpr int NSB = (NCOL + 127) / 128;
    const float *sp = nullptr;
    if constexpr (FP8) {
      const float *sw = reinterpret_cast<const float *>(blob + a.off_s0);
      sp = sw;
      if (lane < 32) {
        const int rr = wave * (BM / WAVES) + lane, src = lane < BM / WAVES ? a_row(rr) : -1;
        if (src >= 0) sp = a.As + (a_first + src) * a.KB;
      } else {
        const int u = lane - 32, mat = u / NSB, nb = n0 / 128 + u % NSB;
        if (mat == 1 && EP == GE_GLU) sw = reinterpret_cast<const float *>(blob + a.off_s1);
        if (mat < (EP == GE_GLU ? 2 : 1) && nb < cdiv(a.N, 128)) sp = sw + int64_t(nb) * a.KB;
      }
    }
    auto load = [&](int c, uint8_t *buf) {
      const uint32_t at = uint32_t(c) * kStepBytes;
#pragma unroll
      for (int t = 0; t < AL; ++t)
        lds_load16(ares, buf + (wave * AL + t) * 1024, int(at) + abyte[t] < a.Kb ? aoff[t] + (aoff[t] == kOOB ? 0u : at) : kOOB);
#pragma unroll
      for (int t = 0; t < WL; ++t)
        lds_load16(wres, buf + BM * kStepBytes + (wave * WL + t) * 1024,
                   int(at) + wbyte[t] < a.Kb ? woff[t] + (woff[t] == kOOB ? 0u : at) : kOOB);
      if constexpr (FP8)
        __builtin_amdgcn_global_load_lds(
            (const __attribute__((address_space(1))) void *)(sp + min(c, a.KB - 1)),
            (__attribute__((address_space(3))) void *)(buf + (BM + BN) * kStepBytes + wave * 256), 4, 0, 0);
    };

    f32x4 acc[MTR][NT];
#pragma unroll
    for (int i = 0; i < MTR; ++i)
#pragma unroll
      for (int j = 0; j < NT; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};

    const int sw = (r >> 1) & 7;
    const int lo16 = r * kStepBytes + ((q ^ sw) << 4), hi16 = r * kStepBytes + (((4 + q) ^ sw) << 4);

    auto compute = [&](const uint8_t *buf) {
      const uint8_t *wb = buf + (BM + wn * NT * 16) * kStepBytes;
      u32x4 wl[NT], wh[NT];
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        wl[j] = *reinterpret_cast<const u32x4 *>(wb + j * 16 * kStepBytes + lo16);
        wh[j] = *reinterpret_cast<const u32x4 *>(wb + j * 16 * kStepBytes + hi16);
      }
      const float *sc = reinterpret_cast<const float *>(buf + (BM + BN) * kStepBytes);
      // this wave's weight scales: one for all its columns (GLU: one per matrix)
      float sw0 = 0.f, sw1 = 0.f;
      if constexpr (FP8) {
        const int nb = EP == GE_GLU ? (n0 + wn * 32) / 128 - n0 / 128 : (n0 + wn * NT * 16) / 128 - n0 / 128;
        sw0 = sc[wave * 64 + 32 + nb];
        if (EP == GE_GLU) sw1 = sc[wave * 64 + 32 + NSB + nb];
      }
#pragma unroll
      for (int i = 0; i < MTR; ++i) {
        const uint8_t *ab = buf + (i * WM + wm) * 16 * kStepBytes;
        const u32x4 al = *reinterpret_cast<const u32x4 *>(ab + lo16), ah = *reinterpret_cast<const u32x4 *>(ab + hi16);
        if constexpr (!FP8) {
#pragma unroll
          for (int j = 0; j < NT; ++j) {
            acc[i][j] = mfma16(as_bf16x8(wl[j]), as_bf16x8(al), acc[i][j]);
            acc[i][j] = mfma16(as_bf16x8(wh[j]), as_bf16x8(ah), acc[i][j]);
          }
        } else {
          const int row = (i * WM + wm) * 16 + r;
          const float sa = sc[row / (BM / WAVES) * 64 + row % (BM / WAVES)];
          const float s0 = sa * sw0, s1 = EP == GE_GLU ? sa * sw1 : s0;
#pragma unroll
          for (int j = 0; j < NT; ++j) {
            f32x4 p = {0.f, 0.f, 0.f, 0.f};
            if constexpr (TY == GT_FP8) {
              p = fp8_mfma(wl[j], wh[j], al, ah);
            } else {
              p = fp8x_mfma(wl[j], al, p);
              p = fp8x_mfma(wh[j], ah, p);
            }
            const float s = EP == GE_GLU && j >= NT / 2 ? s1 : s0;
#pragma unroll
            for (int v = 0; v < 4; ++v) acc[i][j][v] = fmaf(p[v], s, acc[i][j][v]);
          }
        }
      }
    };

    // ---- a ring of STAGES steps: at step c the loads of step c have landed
    // and every wave is done with step c - 1, whose buffer takes step
    // c + STAGES - 1
#pragma unroll
    for (int p = 0; p < STAGES - 1; ++p) {
      load(p, L.b[p]);
      __builtin_amdgcn_sched_barrier(0);
    }
    auto step = [&](auto jc, int c) {
      constexpr int J = decltype(jc)::value;
      if (c >= nk) return;
      wait_vmcnt<(STAGES - 2) * LOADS>();
      lds_barrier();
      load(c + STAGES - 1, L.b[(J + STAGES - 1) % STAGES]);
      __builtin_amdgcn_sched_barrier(0);
      compute(L.b[J]);
    };
    for (int c = 0; c < nk; c += STAGES)
      unroll_steps([&](auto jc) { step(jc, c + decltype(jc)::value); }, std::make_integer_sequence<int, STAGES>{});
    wait_vmcnt<0>();

    // ---- epilogue
#pragma unroll
    for (int i = 0; i < MTR; ++i) {
      const int rr = (i * WM + wm) * 16 + r;
      if (rr >= it.m) continue;
      if constexpr (EP == GE_GLU) {
        float *o = static_cast<float *>(a.out) + (int64_t(shared ? a.rows : it.lo) + it.row0 + rr) * a.ldo;
        const int n = n0 + wn * 32 + 8 * q;
        float v[8];
#pragma unroll
        for (int u = 0; u < 8; ++u) {
          const float g = acc[i][u / 4][u % 4];
          v[u] = silu(g) * acc[i][2 + u / 4][u % 4];
        }
        store8(o, n, a.N, v, a.ldo % 4 == 0);
      } else {
        const bool own = shared && a.out_shared != nullptr;
        const int64_t orow = own ? it.row0 + rr : int64_t(shared ? a.rows : it.lo) + it.row0 + rr;
#pragma unroll
        for (int jj = 0; jj < NT / 2; ++jj) {
          const int n = n0 + wn * NT * 16 + 32 * jj + 8 * q;
          float v[8];
#pragma unroll
          for (int u = 0; u < 8; ++u) v[u] = acc[i][2 * jj + u / 4][u % 4];
          if (own)
            store8(a.out_shared + orow * a.ldo, n, a.N, v, a.ldo % 4 == 0);
          else if (a.out_bf16)
            store8(static_cast<uint16_t *>(a.out) + orow * a.ldo, n, a.N, v, a.ldo % 8 == 0);
          else
            store8(static_cast<float *>(a.out) + orow * a.ldo, n, a.N, v, a.ldo % 4 == 0);
        }
      }
    }
  }

  static __device__ __forceinline__ f32x4 fp8_mfma(u32x4 wl, u32x4 wh, u32x4 al, u32x4 ah) {
    const i32x8 w = __builtin_bit_cast(i32x8, __builtin_shufflevector(wl, wh, 0, 1, 2, 3, 4, 5, 6, 7));
    const i32x8 x = __builtin_bit_cast(i32x8, __builtin_shufflevector(al, ah, 0, 1, 2, 3, 4, 5, 6, 7));
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(w, x, f32x4{0.f, 0.f, 0.f, 0.f}, 0, 0, 0, 0, 0, 0);
  }

  // 16 codes of either operand per lane: 64 products, as bf16
  static __device__ __forceinline__ f32x4 fp8x_mfma(u32x4 w, u32x4 x, f32x4 p) {
    p = mfma16(fp8x8_to_bf16x8(w[0], w[1]), fp8x8_to_bf16x8(x[0], x[1]), p);
    return mfma16(fp8x8_to_bf16x8(w[2], w[3]), fp8x8_to_bf16x8(x[2], x[3]), p);
  }

  // Eight consecutive outputs n .. n+7 of a row, those below N.
  static __device__ __forceinline__ void store8(float *o, int n, int N, const float (&v)[8], bool vec) {
    if (vec && n + 8 <= N) {
      *reinterpret_cast<f32x4 *>(o + n) = f32x4{v[0], v[1], v[2], v[3]};
      *reinterpret_cast<f32x4 *>(o + n + 4) = f32x4{v[4], v[5], v[6], v[7]};
      return;
    }
#pragma unroll
    for (int u = 0; u < 8; ++u)
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

  template <typename F, int... J>
  static __device__ __forceinline__ void unroll_steps(F &&f, std::integer_sequence<int, J...>) {
    (f(std::integral_constant<int, J>{}), ...);
  }

  // The rows of a group whose weights are not resident.
  static __device__ __forceinline__ void fill_nan(const GroupArgs &a, const GroupItem &it) {
    const int n0 = it.nt * NCOL, w = min(NCOL, a.N - n0);
    for (int u = threadIdx.x; u < it.m * w; u += THREADS) {
      const int64_t at = (int64_t(it.lo) + it.row0 + u / w) * a.ldo + n0 + u % w;
      if (EP == GE_OUT && a.out_bf16)
        static_cast<uint16_t *>(a.out)[at] = 0x7fc0;
      else
        static_cast<float *>(a.out)[at] = __builtin_nanf("");
    }
  }

  static __device__ __forceinline__ void run(const GroupArgs &a, const Ring &L) {
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
    if constexpr (MT >= 4)
      if (mt > 2) return body<4>(a, L, it, blob);
    if constexpr (MT >= 2)
      if (mt > 1) return body<2>(a, L, it, blob);
    body<1>(a, L, it, blob);
  }
};

}  // namespace ft
