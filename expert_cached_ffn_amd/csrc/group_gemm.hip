// ft_fp8_gemm, ft_grouped_gemm and the FP8 experts of ft_moe_grouped_ffn: the
// entry points and launches of the products in group_gemm.hpp.
#include <algorithm>

#include "ft_internal.hpp"
#include "group_gemm.hpp"
#include "group_ffn.hpp"
#include "group_stream.hpp"

namespace ft {

template <int TY, int EP, int WM, int WN, int MT, int NT, int STAGES>
__global__ __launch_bounds__(WM * WN * 64) void group_gemm_kernel(GroupArgs a) {
  using G = GroupTile<TY, EP, WM, WN, MT, NT, STAGES>;
  __shared__ __attribute__((aligned(16))) uint8_t ring[STAGES * G::STAGE_BYTES];
  G::run(a, ring);
}

// Most row tiles that the groups can have.
static int row_tiles(const GroupArgs &a, int BM) {
  if (a.offsets == nullptr) return cdiv(a.rows, BM);
  return a.rows / BM + std::min(a.E, a.rows) + (a.shared_blob != nullptr ? cdiv(a.T, BM) : 0);
}

template <int TY, int EP, int WM, int WN, int MT, int NT, int STAGES>
static ft_status launch_tiles(GroupArgs a, hipStream_t stream) {
  using G = GroupTile<TY, EP, WM, WN, MT, NT, STAGES>;
  a.n_ntiles = cdiv(a.N, G::NCOL);
  const int64_t items = int64_t(row_tiles(a, G::BM)) * a.n_ntiles;
  const int64_t grid = cdiv<int64_t>(items, 8) * 8;
  FT_SUPPORTED(grid * G::THREADS < (int64_t(1) << 32), "grouped product: more tiles than a launch has workgroups");
  hipLaunchKernelGGL((group_gemm_kernel<TY, EP, WM, WN, MT, NT, STAGES>), dim3(unsigned(grid)), dim3(G::THREADS), 0,
                     stream, a);
  FT_LAUNCHED("group_gemm_kernel");
  return FT_OK;
}

template <int TY, int EP, int GX, int WAVES, int BPW>
__global__ __launch_bounds__(WAVES * 64) void group_stream_kernel(GroupArgs a) {
  using G = GroupStream<TY, EP, GX, WAVES, BPW>;
  __shared__ typename G::Lds s;
  G::run(a, s);
}

// Most sets of up to 16 rows that the groups can have.
static int row_sets(const GroupArgs &a) {
  if (a.offsets == nullptr) return cdiv(a.rows, 16);
  return a.rows / 16 + std::min(a.E, a.rows) + (a.shared_blob != nullptr ? cdiv(a.T, 16) : 0);
}

// Workgroups of a kernel that the chip holds at once.
template <typename K>
static int resident(K kernel, int threads) {
  int dev = 0, cus = 0, per = 0;
  if (hipGetDevice(&dev) != hipSuccess ||
      hipDeviceGetAttribute(&cus, hipDeviceAttributeMultiprocessorCount, dev) != hipSuccess || cus <= 0)
    cus = 256;
  if (hipOccupancyMaxActiveBlocksPerMultiprocessor(&per, reinterpret_cast<const void *>(kernel), threads, 0) != hipSuccess ||
      per <= 0) {
    (void)hipGetLastError();
    per = 1;
  }
  return cus * per;
}

template <int TY, int EP, int GX, int WAVES, int BPW>
static ft_status launch_stream_as(GroupArgs a, hipStream_t stream) {
  static const int fit = resident(&group_stream_kernel<TY, EP, GX, WAVES, BPW>, WAVES * 64);
  a.n_ntiles = cdiv(a.N, 16);
  const int64_t units = int64_t(row_sets(a)) * a.n_ntiles;
  hipLaunchKernelGGL((group_stream_kernel<TY, EP, GX, WAVES, BPW>), dim3(unsigned(std::min<int64_t>(units, fit))),
                     dim3(WAVES * 64), 0, stream, a);
  FT_LAUNCHED("group_stream_kernel");
  return FT_OK;
}

static bool stream_covers(const GroupArgs &a) {
  return a.E <= kStreamMaxE && a.rows <= kStreamMaxRows && (a.shared_blob == nullptr || a.T <= kStreamMaxT) &&
         int64_t(row_sets(a)) * cdiv(a.N, 16) < (int64_t(1) << 30);
}

// The stream kernel where 64-column tiles would leave most of the chip idle: it
// spreads 16-column units over it (one row by 4096 x 4096 FP8: 7.6 against 13.0
// us; 77 rows by 1001 x 2000 in fp32: 7.5 against 10.2).  With enough tiles the
// LDS ring keeps more of the weights on their way (64 tokens, 128 experts,
// bf16: 136 us against 156).
static bool stream_choice(const GroupArgs &a, int64_t cols) {  // cols: weight rows per group
  if (a.rows > (a.offsets != nullptr ? 16 * std::min(a.E, a.rows) : 128)) return false;
  return row_tiles(a, 32) * cdiv<int64_t>(cols, 64) < 200 && stream_covers(a);
}

template <int TY, int EP, int GX>
static ft_status launch_stream(const GroupArgs &a, hipStream_t stream) {
  const int blocks = cdiv(a.Kb, kStepBytes);
  if (blocks <= 8) return launch_stream_as<TY, EP, GX, 8, 1>(a, stream);
  if (blocks <= 16) return launch_stream_as<TY, EP, GX, 8, 2>(a, stream);
  return launch_stream_as<TY, EP, GX, 8, 4>(a, stream);
}

// Tile sizes.  256 x 256 (two steps in the ring, 132 KiB of LDS) moves the
// fewest operand bytes per product; 128 x 256 has room for three steps, which
// counts where the groups are short and the weights come from HBM; 64 x 64
// fills the chip when there are few rows.  Measured, 256 / 128 / 64 rows a
// tile: dense 8192 x 4096 x 4096 FP8 134 / 160 / 257 us; FP8 groups of 192 rows
// on average (256 groups, N = K = 4096) 1.35 / 1.35 / 2.2 ms; the FP8 experts
// with 96 rows on average 2.02 / 1.78 / 2.19 ms; bf16 groups of 256 rows
// (N 2048, K 768) 201 / 210 / 285 us.
enum { TILE_32, TILE_64, TILE_128, TILE_256 };
static int tile_choice(const GroupArgs &a, int cols256) {
  const int groups = a.offsets != nullptr ? std::min(a.E, a.rows) : 1;
  const int mean = a.rows / std::max(1, groups);
  auto tiles = [&](int BM) {
    return (a.offsets != nullptr ? a.rows / BM + groups / 2 : cdiv(a.rows, BM)) * int64_t(cdiv(a.N, cols256));
  };
  if (mean >= 160 && tiles(256) >= 224) return TILE_256;
  if (mean >= 24 && tiles(128) >= 100) return TILE_128;
  return mean > 32 ? TILE_64 : TILE_32;
}

// fp8_ffn asks for GE_GLUQ where the tiles hold whole blocks, for GE_GLU elsewhere.
template <int TY, int EP>
static ft_status launch_products(const GroupArgs &a, hipStream_t stream) {
  constexpr bool GLU = is_glu(EP);
  const int tile = tile_choice(a, GLU ? 128 : 256);
  if constexpr (EP != GE_GLU) {
    if (tile == TILE_256) return launch_tiles<TY, EP, 2, 4, 8, 4, 2>(a, stream);
    if (tile == TILE_128) return launch_tiles<TY, EP, 2, 4, 4, 4, 3>(a, stream);
  }
  if constexpr (EP != GE_GLUQ) {
    if (tile == TILE_64) return launch_tiles<TY, EP, 2, 2, 2, GLU ? 4 : 2, 3>(a, stream);
    if (tile == TILE_32) return launch_tiles<TY, EP, 2, 2, 1, GLU ? 4 : 2, GLU ? 3 : 4>(a, stream);
  }
  return fail(FT_ENOTSUP, "grouped product: no tile of this form");
}

static ft_status group_products(int dtype, int out_dtype, const GroupArgs &a, hipStream_t stream) {
  if (a.rows == 0 || a.N == 0) return FT_OK;
  if (stream_choice(a, a.N)) {
    if (dtype == FT_BF16)
      return out_dtype == FT_BF16 ? launch_stream<GT_BF16, GE_BF16, GX_SAME>(a, stream)
                                  : launch_stream<GT_BF16, GE_F32, GX_SAME>(a, stream);
    return out_dtype == FT_BF16 ? launch_stream<GT_FP8X, GE_BF16, GX_SAME>(a, stream)
                                : launch_stream<GT_FP8X, GE_F32, GX_SAME>(a, stream);
  }
  if (dtype == FT_BF16)
    return out_dtype == FT_BF16 ? launch_products<GT_BF16, GE_BF16>(a, stream) : launch_products<GT_BF16, GE_F32>(a, stream);
  return out_dtype == FT_BF16 ? launch_products<GT_FP8, GE_BF16>(a, stream) : launch_products<GT_FP8X, GE_F32>(a, stream);
}

// ------------------------------------------------------------------ FP8 experts

// Workspace: the tokens' codes and scales, the hidden rows in fp32, their codes and scales.
struct Fp8FfnWorkspace {
  uint64_t xq, xs, h, hq, hs, total;
};
static Fp8FfnWorkspace fp8_ffn_workspace(int64_t T, int64_t k, int64_t H, int64_t I) {
  auto al = [](uint64_t b) { return (b + 255) / 256 * 256; };
  const uint64_t rows = uint64_t(T * k + T);
  Fp8FfnWorkspace w;
  w.h = 0;
  w.hq = w.h + al(rows * I * 4);
  w.hs = w.hq + al(rows * I);
  w.xq = w.hs + al(rows * cdiv<int64_t>(I, kFp8Block) * 4);
  w.xs = w.xq + al(uint64_t(T * H));
  w.total = w.xs + al(uint64_t(T) * cdiv<int64_t>(H, kFp8Block) * 4);
  return w;
}

size_t fp8_ffn_workspace_bytes(int32_t T, int32_t k, int32_t H, int32_t I) {
  return size_t(fp8_ffn_workspace(T, k, H, I).total);
}

ft_status fp8_ffn(const Fp8Ffn &f, hipStream_t stream) {
  const ft_expert_layout &L = *f.L;
  const int H = L.H, I = L.I, routed = f.T * f.k, rows = routed + (f.shared_blob != nullptr ? f.T : 0);
  const Fp8FfnWorkspace W = fp8_ffn_workspace(f.T, f.k, H, I);
  uint8_t *ws = static_cast<uint8_t *>(f.workspace);
  float *xs = reinterpret_cast<float *>(ws + W.xs), *hs = reinterpret_cast<float *>(ws + W.hs);
  GroupArgs a{};
  a.pool = static_cast<const uint8_t *>(f.slot_pool);
  a.expert_bytes = L.expert_bytes;
  a.slots = f.slot_of_expert;
  a.n_slots = f.n_slots;
  a.shared_blob = static_cast<const uint8_t *>(f.shared_blob);
  a.offsets = f.expert_offsets;
  a.E = f.E;
  a.rows = routed;
  a.T = f.T;
  a.k = f.k;
  GroupArgs g = a;  // gate and up
  g.off_w0 = L.off_gate;
  g.off_w1 = L.off_up;
  g.off_s0 = L.off_sgate;
  g.off_s1 = L.off_sup;
  g.ldw = g.Kb = H;
  g.KB = cdiv(H, kFp8Block);
  g.N = I;
  g.sorted_rows = f.sorted_rows;
  g.a_rows = f.T;
  g.out = ws + W.h;
  g.ldo = I;
  GroupArgs d = a;  // down
  d.off_w0 = d.off_w1 = L.off_down;
  d.off_s0 = d.off_s1 = L.off_sdown;
  d.ldw = d.Kb = I;
  d.KB = cdiv(I, kFp8Block);
  d.N = H;
  d.a_rows = rows;
  d.a_shared0 = routed;
  d.out = f.y_rows;
  d.ldo = H;
  d.out_shared = f.y_shared;
  // The same choices whatever stages the call runs (the down stage has to find
  // the hidden rows in the form it takes):
  //  - gate/up of few rows and tiles: the stream kernel, which quantizes x as it
  //    reads it (1 token, 2 of 16 experts, H 2048, I 768: 15 against 22 us for
  //    the whole FFN);
  //  - otherwise x is quantized by a launch of its own.  Tiles of whole 128-blocks
  //    of the hidden rows quantize those as they write them (4096 tokens of 256
  //    experts, H 4096, I 2048: 1.69 against 1.77 ms); smaller tiles leave them in
  //    fp32;
  //  - fp32 hidden rows go to the stream kernel for down if gate/up took it, or if
  //    the tiles have few steps to hide their start behind (33 tokens, 8 of 128
  //    experts, I 768: 113 against 116 us); else they are quantized by a launch
  //    of their own.
  // Gate/up sums decide the hidden rows' codes, where an error of 1.5e-5 moves
  // about one value in 5000 to its neighbour: a token in 30 is then off by up to
  // 8e-3 instead of a bf16 output's 1.7e-3.  Where the weights' read bounds the
  // call the sums are exact (bf16 instruction: 116 against 114 us at 33 tokens);
  // the whole-block tiles of large batches use the FP8 instruction (1.71 against
  // 2.00 ms at 4096 tokens; all tokens together 2.0e-3 off).
  a.N = std::max(H, I);
  const bool stream_gu = stream_choice(a, 2 * int64_t(I));
  const bool whole = !stream_gu && tile_choice(g, 128) >= TILE_128;
  const bool stream_dn =
      stream_gu || (!whole && I <= 1024 && a.rows <= 16 * std::min(a.E, a.rows) && stream_covers(a));
  ft_status st = FT_OK;
  if (f.gate_up && stream_gu) {
    g.A = static_cast<const uint8_t *>(f.x);
    g.lda = 2 * int64_t(H);
    st = launch_stream<GT_FP8X, GE_GLU, GX_BF16>(g, stream);
  } else if (f.gate_up) {
    st = fp8_quantize_launch(f.x, FT_BF16, H, f.T, H, 1, ws + W.xq, H, xs, stream);
    if (st != FT_OK) return st;
    g.A = ws + W.xq;
    g.lda = H;
    g.As = xs;
    if (whole) {
      g.out = ws + W.hq;
      g.out_scales = hs;
      st = launch_products<GT_FP8, GE_GLUQ>(g, stream);
    } else {
      st = launch_products<GT_FP8X, GE_GLU>(g, stream);
    }
  }
  if (st != FT_OK || !f.down) return st;
  if (stream_dn) {
    d.A = ws + W.h;
    d.lda = 4 * int64_t(I);
    return launch_stream<GT_FP8, GE_F32, GX_F32>(d, stream);
  }
  if (!whole) {
    st = fp8_quantize_launch(ws + W.h, FT_F32, I, rows, I, 1, ws + W.hq, I, hs, stream);
    if (st != FT_OK) return st;
  }
  d.A = ws + W.hq;
  d.lda = I;
  d.As = hs;
  return launch_products<GT_FP8, GE_F32>(d, stream);
}

}  // namespace ft

using namespace ft;

constexpr int64_t kMaxPitch = int64_t(1) << 22;  // bytes of a row: a tile's rows stay under 2 GiB

extern "C" ft_status ft_fp8_gemm(const uint8_t *a, int64_t lda, const float *a_scales, const uint8_t *w, int64_t ldw,
                                 const float *w_scales, int64_t M, int32_t N, int32_t K, int32_t out_dtype, void *out,
                                 int64_t ldo, hipStream_t stream) {
  FT_REQUIRE(M >= 0 && N >= 0 && K >= 1, "ft_fp8_gemm: need M >= 0, N >= 0, K >= 1");
  FT_REQUIRE(out_dtype == FT_BF16 || out_dtype == FT_F32, "ft_fp8_gemm: out_dtype must be FT_BF16 or FT_F32");
  FT_SUPPORTED(K % 16 == 0, "ft_fp8_gemm: K must be a multiple of 16");
  FT_REQUIRE(lda >= K && ldw >= K && ldo >= N, "ft_fp8_gemm: row pitch below the row's length");
  FT_SUPPORTED(M < (int64_t(1) << 31) - 512 && lda <= kMaxPitch && ldw <= kMaxPitch,
               "ft_fp8_gemm: M above 2^31 - 512 or a row pitch above 4 MiB");
  if (M == 0 || N == 0) {
    clear_error();
    return FT_OK;
  }
  FT_REQUIRE(a && a_scales && w && w_scales && out, "ft_fp8_gemm: NULL pointer argument");
  FT_REQUIRE(lda % 16 == 0 && ldw % 16 == 0 && aligned(a, 16) && aligned(w, 16) && aligned(out, 16) &&
                 aligned(a_scales, 4) && aligned(w_scales, 4),
             "ft_fp8_gemm: a, w and out must be 16-byte aligned, lda and ldw multiples of 16");
  GroupArgs g{};
  g.A = a;
  g.lda = lda;
  g.As = a_scales;
  g.pool = w;
  g.n_slots = 1;
  g.off_s0 = uint64_t(reinterpret_cast<uintptr_t>(w_scales) - reinterpret_cast<uintptr_t>(w));
  g.ldw = ldw;
  g.Kb = K;
  g.KB = cdiv(K, kFp8Block);
  g.N = N;
  g.E = 1;
  g.rows = int(M);
  g.T = int(M);
  g.k = 1;
  g.a_rows = M;
  g.out = out;
  g.ldo = ldo;
  const ft_status st = group_products(FT_FP8, out_dtype, g, stream);
  if (st != FT_OK) return st;
  clear_error();
  return FT_OK;
}

extern "C" ft_status ft_grouped_gemm(int32_t dtype, const void *a, int64_t lda, const float *a_scales,
                                     const void *slot_pool, uint64_t expert_bytes, uint64_t off_w, uint64_t off_s,
                                     int32_t n_slots, const int32_t *slot_of_expert, int32_t T, int32_t k, int32_t E,
                                     const int32_t *expert_offsets, const int32_t *sorted_rows, int32_t N, int32_t K,
                                     int32_t out_dtype, void *out, int64_t ldo, hipStream_t stream) {
  FT_REQUIRE(dtype == FT_BF16 || dtype == FT_FP8, "ft_grouped_gemm: dtype must be FT_BF16 or FT_FP8");
  FT_REQUIRE(out_dtype == FT_BF16 || out_dtype == FT_F32, "ft_grouped_gemm: out_dtype must be FT_BF16 or FT_F32");
  FT_REQUIRE(T >= 0 && k >= 1 && E >= 1 && N >= 0 && K >= 1,
             "ft_grouped_gemm: need T >= 0, k >= 1, E >= 1, N >= 0, K >= 1");
  FT_SUPPORTED(E <= 4096, "ft_grouped_gemm: E > 4096");
  FT_REQUIRE(int64_t(T) * k < (int64_t(1) << 31) - 512, "ft_grouped_gemm: T*k too large");
  const int es = dtype == FT_BF16 ? 2 : 1;
  FT_SUPPORTED(K % (16 / es) == 0, "ft_grouped_gemm: K must be a multiple of 16 (bf16: of 8)");
  FT_REQUIRE(lda >= K && ldo >= N, "ft_grouped_gemm: row pitch below the row's length");
  FT_SUPPORTED(lda * es <= kMaxPitch && int64_t(K) * es <= kMaxPitch, "ft_grouped_gemm: a row pitch above 4 MiB");
  FT_SUPPORTED(sorted_rows == nullptr || int64_t(T) * lda * es < (int64_t(1) << 31),
               "ft_grouped_gemm: gathered rows of 2 GiB or more");
  if (T == 0 || N == 0) {
    clear_error();
    return FT_OK;
  }
  FT_REQUIRE(a && slot_pool && expert_offsets && out && (dtype == FT_BF16 || a_scales),
             "ft_grouped_gemm: NULL pointer argument");
  FT_REQUIRE(n_slots >= 1 && (slot_of_expert != nullptr || n_slots >= E),
             "ft_grouped_gemm: n_slots must be >= 1, and >= E when slot_of_expert is NULL");
  FT_REQUIRE(aligned(a, 16) && lda * es % 16 == 0 && aligned(out, 16) && aligned(a_scales, 4),
             "ft_grouped_gemm: a and out must be 16-byte aligned, rows of a a multiple of 16 bytes apart");
  FT_REQUIRE(aligned(slot_pool, 16) && expert_bytes % 16 == 0 && off_w % 16 == 0 && off_s % 4 == 0,
             "ft_grouped_gemm: weights must be 16-byte aligned (scales 4-byte)");
  const int KB = cdiv(K, kFp8Block);
  const uint64_t wb = uint64_t(N) * K * es, sb = dtype == FT_FP8 ? uint64_t(cdiv(N, kFp8Block)) * KB * 4 : 0;
  FT_REQUIRE(off_w <= expert_bytes && wb <= expert_bytes - off_w &&
                 (sb == 0 || (off_s <= expert_bytes && sb <= expert_bytes - off_s)),
             "ft_grouped_gemm: weights or scales reach past expert_bytes");
  GroupArgs g{};
  g.A = static_cast<const uint8_t *>(a);
  g.lda = lda * es;
  g.As = a_scales;
  g.pool = static_cast<const uint8_t *>(slot_pool);
  g.expert_bytes = expert_bytes;
  g.slots = slot_of_expert;
  g.n_slots = n_slots;
  g.off_w0 = off_w;
  g.off_s0 = off_s;
  g.ldw = int64_t(K) * es;
  g.Kb = K * es;
  g.KB = KB;
  g.N = N;
  g.offsets = expert_offsets;
  g.E = E;
  g.rows = T * k;
  g.T = T;
  g.k = k;
  g.sorted_rows = sorted_rows;
  g.a_rows = sorted_rows != nullptr ? T : int64_t(T) * k;
  g.out = out;
  g.ldo = ldo;
  const ft_status st = group_products(dtype, out_dtype, g, stream);
  if (st != FT_OK) return st;
  clear_error();
  return FT_OK;
}
