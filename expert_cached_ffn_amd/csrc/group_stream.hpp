// The products of group_gemm.hpp for groups of a few rows (decoding), where
// every weight byte is used a few times at most and the read of the weights is
// all there is: at 16 rows a 128-byte piece of 16 weight rows takes 2 KB of HBM
// and one or two matrix instructions.
//
// A unit is 16 weight rows (GLU: the same 16 of gate and up) by up to 16 rows
// of one group.  The WAVES waves of a workgroup split the contraction axis, BPW
// blocks of 128 bytes each per pass (wave w takes blocks w, w + WAVES, ...), and
// meet in LDS, where the partial sums are added in wave order.  A workgroup
// takes a contiguous run of units, weight tile by weight tile of one row set,
// so the row operands stay in registers, and the next unit's weights are on
// their way while one is multiplied.
//
// Weights are read as whole 128-byte lines, 8 rows a load (half lines streamed
// 5.96 TB/s against 6.85 on a 1 GiB probe); wl_swap then moves a pair of loads into
// the operand layout, after which lane (r, q) holds bytes 32q .. 32q+31 of row
// r's block.  The row operands are loaded in that layout.
//
// The rows may also come as bf16 or fp32 that the kernel quantizes itself, by
// the rule of fp8.hip (a lane's 32 elements and three other lanes' are one
// block): one launch less, and the hidden vector of the FP8 experts keeps its
// fp32 value until then.
//
// Measured: one row by 4096 x 4096 FP8 7.3 us, 77 rows by 1001 x 2000 in fp32
// 7.2 us, one launch being about 5 of both; the FP8 experts' down product of 33
// tokens (H 2048, I 768, about 104 experts' weights, 164 MB) 47 us.
#pragma once

#include "group_gemm.hpp"
#include "stream_gemm.hpp"

namespace ft {

enum { GX_SAME = 0, GX_BF16 = 1, GX_F32 = 2 };  // row operand: as the weights (FP8: codes and scales); to be quantized

constexpr int kStreamMaxE = 1024;     // groups of the LDS table (and one shared)
constexpr int kStreamMaxRows = 4096;
constexpr int kStreamMaxT = 256;      // rows of the shared group
constexpr int kStreamMaxSets = kStreamMaxE + kStreamMaxRows / 16 + kStreamMaxT / 16;  // row sets of all groups, at most

template <int TY, int EP, int GX, int WAVES, int BPW>
struct GroupStream {
  static constexpr int THREADS = WAVES * 64;
  static constexpr int MATS = EP == GE_GLU ? 2 : 1;
  static constexpr bool FP8 = TY != GT_BF16;

  struct Set {  // up to 16 rows of one group
    int slot;   // of its weights; -1: not resident; kSharedSlot: the shared group's
    int row0;   // first output row (shared: rows + first token)
    int m;
  };
  static constexpr int kSharedSlot = -3;

  struct Lds {
    int slot[kStreamMaxSets], row0[kStreamMaxSets], m[kStreamMaxSets];
    int cnt[WAVES];
    float red[2][WAVES][MATS][256];
  };

  // The sets of all groups in order, the shared group's last; groups whose slot
  // is FT_SLOT_SKIP have none.
  static __device__ __forceinline__ int build(const GroupArgs &a, Lds &s) {
    const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63;
    int n = 0;
    for (int c0 = 0; c0 < a.E; c0 += THREADS) {
      const int e = c0 + tid;
      int lo = 0, m = group_rows(a, e, &lo);
      const int slot = m > 0 ? table_slot(a.slots, e, a.n_slots) : 0;
      if (slot == FT_SLOT_SKIP) m = 0;
      const int sets = (m + 15) / 16, incl = wave_incl_scan_i32(sets);
      if (lane == 63) s.cnt[wave] = incl;
      __syncthreads();
      int at = n + incl - sets;
#pragma unroll
      for (int w = 0; w < WAVES; ++w) {
        if (w < wave) at += s.cnt[w];
        n += s.cnt[w];
      }
      for (int g = 0; g < sets && at + g < kStreamMaxSets; ++g) {
        s.slot[at + g] = slot < 0 ? -1 : slot;
        s.row0[at + g] = lo + 16 * g;
        s.m[at + g] = min(16, m - 16 * g);
      }
      __syncthreads();
    }
    if (a.shared_blob != nullptr) {
      const int sets = (a.T + 15) / 16;
      for (int g = tid; g < sets && n + g < kStreamMaxSets; g += THREADS) {
        s.slot[n + g] = kSharedSlot;
        s.row0[n + g] = a.rows + 16 * g;
        s.m[n + g] = min(16, a.T - 16 * g);
      }
      n += sets;
      __syncthreads();
    }
    return min(n, kStreamMaxSets);
  }

  struct Weights {
    u32x4 w[MATS][BPW][2];
    float s[MATS];  // lane c < BPW: scale of block c
  };
  struct Rows {
    u32x4 x[BPW][2];
    float s[BPW];
  };

  static __device__ __forceinline__ int uni(int v) { return __builtin_amdgcn_readfirstlane(v); }

  static __device__ __forceinline__ const uint8_t *blob_of(const GroupArgs &a, int slot) {
    return slot == kSharedSlot ? a.shared_blob : a.pool + uint64_t(max(slot, 0)) * a.expert_bytes;
  }

  // Block c of pass p of this wave.
  static __device__ __forceinline__ int block_of(int p, int c, int wave) { return p * (WAVES * BPW) + c * WAVES + wave; }

  static __device__ __forceinline__ void load_weights(const GroupArgs &a, const Lds &s, int set, int tile, int pass, bool once, bool live,
                                                      Weights &o) {
    const int lane = threadIdx.x & 63, wave = uni(threadIdx.x >> 6);
    const int slot = uni(s.slot[set]), n0 = tile * 16;
    const uint8_t *blob = blob_of(a, slot);
    const int rows = min(16, a.N - n0);
    const bool there = live && slot != -1;
#pragma unroll
    for (int mt = 0; mt < MATS; ++mt) {
      const uint8_t *w = blob + (mt ? a.off_w1 : a.off_w0) + uint64_t(n0) * uint64_t(a.ldw);
      const rsrc_t r = make_rsrc(w, there ? uint32_t((rows - 1) * a.ldw + a.Kb) : 0u);
#pragma unroll
      for (int c = 0; c < BPW; ++c) {
        const int at = block_of(pass, c, wave) * kStepBytes + 16 * (lane >> 3);
#pragma unroll
        for (int d = 0; d < 2; ++d) {
          const int row = 8 * d + (lane & 7);
          const uint32_t off = at < a.Kb && row < rows ? uint32_t(row) * uint32_t(a.ldw) + uint32_t(at) : kOOB;
          o.w[mt][c][d] = once ? bld16nt(r, off) : bld16(r, off);
        }
      }
      if constexpr (FP8) {
        const float *sw = reinterpret_cast<const float *>(blob + (mt ? a.off_s1 : a.off_s0)) + int64_t(n0 / 128) * a.KB;
        const int b = block_of(pass, lane, wave);
        const rsrc_t sr = make_rsrc(sw, there ? uint32_t(a.KB) * 4u : 0u);
        o.s[mt] = __uint_as_float(bld4(sr, lane < BPW && b < a.KB ? uint32_t(b) * 4u : kOOB));
      }
    }
  }

  // Row r's part of this wave's blocks in a pass, in the operand layout.
  static __device__ __forceinline__ void load_rows(const GroupArgs &a, const Lds &s, int set, int pass, Rows &o) {
    const int lane = threadIdx.x & 63, wave = uni(threadIdx.x >> 6), r = lane & 15, q = lane >> 4;
    const int row0 = uni(s.row0[set]), m = uni(s.m[set]);
    const bool shared = uni(s.slot[set]) == kSharedSlot;
    int64_t src = -1;
    if (r < m) {
      if (shared) {
        src = int64_t(a.a_shared0) + (row0 - a.rows) + r;
      } else if (a.sorted_rows != nullptr) {
        const uint32_t t = uint32_t(a.sorted_rows[row0 + r]) / uint32_t(a.k);
        if (t < uint32_t(a.a_rows)) src = t;
      } else {
        src = row0 + r;
      }
    }
    const uint8_t *p = a.A + (src < 0 ? 0 : src) * a.lda;
#pragma unroll
    for (int c = 0; c < BPW; ++c) {
      const int b = block_of(pass, c, wave);
      o.s[c] = 0.f;
      if constexpr (GX == GX_SAME) {
        const int at = b * kStepBytes + 32 * q;
#pragma unroll
        for (int d = 0; d < 2; ++d)
          o.x[c][d] = src >= 0 && at + 16 * d < a.Kb ? ld16(p + at + 16 * d) : u32x4{0, 0, 0, 0};
        if constexpr (FP8)
          if (src >= 0 && b < a.KB) o.s[c] = a.As[src * a.KB + b];
      } else {
        // 32 elements of the block per lane, the block's other 96 in lanes r + 16, r + 32, r + 48
        const int at = b * kFp8Block + 32 * q;
        float v[32];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          float(&t)[8] = *reinterpret_cast<float(*)[8]>(v + 8 * u);
          if (src >= 0 && at + 8 * u < a.Kb) {
            if constexpr (GX == GX_BF16)
              fp8_load8(reinterpret_cast<const uint16_t *>(p) + at + 8 * u, t);
            else
              fp8_load8(reinterpret_cast<const float *>(p) + at + 8 * u, t);
          } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) t[i] = 0.f;
          }
        }
        uint32_t amax = 0;
#pragma unroll
        for (int i = 0; i < 32; ++i) amax = max(amax, __float_as_uint(v[i]) & 0x7fffffffu);
        amax = max(amax, uint32_t(__shfl_xor(int(amax), 16)));
        amax = max(amax, uint32_t(__shfl_xor(int(amax), 32)));
        const Fp8Scale sc = fp8_scale(amax);
        o.s[c] = sc.scale;
#pragma unroll
        for (int d = 0; d < 2; ++d)
#pragma unroll
          for (int u = 0; u < 4; ++u)
            o.x[c][d][u] = fp8_codes4(v[16 * d + 4 * u], v[16 * d + 4 * u + 1], v[16 * d + 4 * u + 2], v[16 * d + 4 * u + 3], sc.inv);
      }
    }
  }

  static __device__ __forceinline__ void multiply(const Weights &w, const Rows &x, f32x4 (&acc)[MATS]) {
#pragma unroll
    for (int c = 0; c < BPW; ++c)
#pragma unroll
      for (int mt = 0; mt < MATS; ++mt) {
        u32x4 lo = w.w[mt][c][0], hi = w.w[mt][c][1];
        wl_swap(lo, hi);
        if constexpr (!FP8) {
          acc[mt] = mfma16(as_bf16x8(lo), as_bf16x8(x.x[c][0]), acc[mt]);
          acc[mt] = mfma16(as_bf16x8(hi), as_bf16x8(x.x[c][1]), acc[mt]);
        } else {
          f32x4 p = {0.f, 0.f, 0.f, 0.f};
          if constexpr (TY == GT_FP8)
            p = fp8_mfma(lo, hi, x.x[c][0], x.x[c][1]);
          else
            p = fp8x_mfma(hi, x.x[c][1], fp8x_mfma(lo, x.x[c][0], p));
          const float sc = lane_value(w.s[mt], c) * x.s[c];
#pragma unroll
          for (int v = 0; v < 4; ++v) acc[mt][v] = fmaf(p[v], sc, acc[mt][v]);
        }
      }
  }

  // The waves' partial sums of a unit, added in wave order, to the outputs.
  static __device__ __forceinline__ void finish(const GroupArgs &a, Lds &s, int set, int tile, int par, const f32x4 (&acc)[MATS]) {
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
#pragma unroll
    for (int mt = 0; mt < MATS; ++mt) *reinterpret_cast<f32x4 *>(&s.red[par][wave][mt][lane * 4]) = acc[mt];
    lds_barrier();
    const int row = tid >> 4, n = tile * 16 + (tid & 15);
    if (tid < 256 && row < s.m[set] && n < a.N) {
      const int at = (row + 16 * ((tid & 15) >> 2)) * 4 + (tid & 3), slot = s.slot[set], orow = s.row0[set] + row;
      float v[MATS];
#pragma unroll
      for (int mt = 0; mt < MATS; ++mt) {
        v[mt] = 0.f;
#pragma unroll
        for (int w = 0; w < WAVES; ++w) v[mt] += s.red[par][w][mt][at];
      }
      float y = EP == GE_GLU ? silu(v[0]) * v[MATS - 1] : v[0];
      if (slot == -1) y = __builtin_nanf("");
      const bool own = EP == GE_F32 && slot == kSharedSlot && a.out_shared != nullptr;
      if constexpr (EP == GE_BF16)
        static_cast<uint16_t *>(a.out)[int64_t(orow) * a.ldo + n] = f32_to_bf16_rne(y);
      else if (own)
        a.out_shared[int64_t(orow - a.rows) * a.ldo + n] = y;
      else
        static_cast<float *>(a.out)[int64_t(orow) * a.ldo + n] = y;
    }
    // the other half of red serves the next unit; the barrier there comes
    // before anyone writes this half again
  }

  static __device__ __forceinline__ void run(const GroupArgs &a, Lds &s) {
    const int sets = build(a, s);
    const int tiles = a.n_ntiles, passes = cdiv(cdiv(a.Kb, kStepBytes), WAVES * BPW);
    const int64_t units = int64_t(sets) * tiles;
    const int u0 = int(units * blockIdx.x / gridDim.x), u1 = int(units * (blockIdx.x + 1) / gridDim.x);
    if (u0 >= u1) return;
    const bool once = a.T <= 16;  // then no weight is read for a second set of rows
    Weights w[2];
    Rows x;
    f32x4 acc[MATS];
    int set = u0 / tiles, tile = u0 - set * tiles, pass = 0, par = 0, held = -1;
    load_weights(a, s, set, tile, 0, once, true, w[0]);
    // one pass of one unit; false at the run's end
    int unit = u0;
    auto turn = [&](Weights &cur, Weights &nxt) FT_INLINE {
      const int key = set * passes + pass;
      if (key != held) {  // (waits for the weights too: in a run over one set it happens once)
        load_rows(a, s, set, pass, x);
        held = key;
      }
      int nset = set, ntile = tile, npass = pass + 1, nunit = unit;
      if (npass == passes) {
        npass = 0;
        ++nunit;
        if (++ntile == tiles) {
          ntile = 0;
          ++nset;
        }
      }
      // (past the run's end too, from empty buffers: behind a branch the compiler
      // would wait for these loads before it multiplies)
      const bool more = nunit < u1;
      load_weights(a, s, more ? nset : set, more ? ntile : tile, npass, once, more, nxt);
      if (pass == 0)
#pragma unroll
        for (int mt = 0; mt < MATS; ++mt) acc[mt] = f32x4{0.f, 0.f, 0.f, 0.f};
      multiply(cur, x, acc);
      if (npass == 0) {
        finish(a, s, set, tile, par, acc);
        par ^= 1;
      }
      set = nset;
      tile = ntile;
      pass = npass;
      unit = nunit;
      return more;
    };
    while (turn(w[0], w[1]) && turn(w[1], w[0])) {
    }
  }
};

}  // namespace ft
