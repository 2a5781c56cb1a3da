// Cross entropy of a linear head, logits = H W^T, without keeping the logits
// (gfx950).
//
//   z[t, v] = sum_k h[t, k] w[v, k]
//   lse[t]  = log sum_v exp z[t, v],   loss[t] = lse[t] - z[t, target[t]]
//   G[t, v] = (exp(z[t, v] - lse[t]) - [v == target[t]]) dloss[t]
//   dH = G W,   dW = G^T H
//
// Forward: one product whose epilogue keeps, per token and tile of 256
// vocabulary columns, the maximum and the sum of exponentials over the tile's
// columns but the target; a second kernel joins the tiles.  The target's share
// of the sum is added last: loss = log(1 + sum_{v != target} exp(z_v -
// z_target)), so that a token whose target has almost all of the probability
// keeps its loss, 1 - p to first order, to fp32's relative precision, where lse
// - z_target would leave the rounding of two large numbers.  The backward takes
// the target's entry of G, p - 1, from that loss as expm1(-loss).  Backward: the vocabulary is taken in
// pieces; per piece the logits are made again, their epilogue turns them into
// G (bf16), and two products add G's share to dH and finish the piece's rows
// of dW.  The workspace holds one piece, whatever the vocabulary.
//
// Every product is the same kernel on bf16 operands (v_mfma_f32_16x16x32_bf16,
// fp32 accumulators).  An operand's rows run along the contraction (H and W in
// the logits, G in dH) or across it (W in dH; G and H in dW): the latter are
// turned by transposing LDS reads, so nothing is ever transposed in memory.
// From a few hundred tokens on the products run at 90 to 95% of a library
// product's rate: 8192 tokens, 131072 x 4096, statistics 6.1 to 6.2 ms (1.43
// PFLOP/s), G 6.6, dH and dW 12.9 to 13.4 ms.  Matrix cores are busy 70%, 60% and
// 64% of the cycles (at 1.9 GHz), and waves wait 35 to 43% of theirs for operands.  With few
// tokens the reading of W bounds them: 33 tokens, 131072 x 5120, forward 223 us
// (6 TB/s).
//
// Rounding: G is held as bf16, the accuracy of the matrix cores' operands.
// It is formed with dloss divided by its largest magnitude, which the
// epilogues multiply back in fp32: with the usual equal weights of a mean
// loss nothing but G's own rounding remains.
//
// A row of G sums to zero, so what all rows of W share cancels in dH.  The
// rounded G's rows do not: their sums (fp32, from the epilogue that rounds
// them) times the target's row of W are taken out of dH in the end, which
// makes dH[t] = sum_v G[t, v] (W[v] - W[target]), where only the rows'
// differences meet G's rounding (and a target's own entry does not matter).
// With sums added up in memory by each wave a step of 8192 tokens, 131072 x
// 4096, takes 1.5% longer.

#include <type_traits>

#include "device_common.h"
#include "launch.h"

namespace fp8bw {

namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef __attribute__((address_space(3))) void lds_void;
typedef __attribute__((address_space(1))) void global_void;
typedef unsigned int u32x4_t __attribute__((ext_vector_type(4)));

constexpr int kMaxStages = 3;   // of 64 contraction elements, in LDS
constexpr int kCus = 256;   // compute units of an MI355X
constexpr float kLog2e = 1.44269504088896340736f;

// What a product's epilogue does with its tile.
enum XentEpilogue {
  kStats = 0,    // maximum and sum of exponentials per row; the targets' logits
  kGrad = 1,     // G in bf16
  kOut = 2,      // bf16, times *scale
  kAcc = 3       // fp32 partial [split][M][N], written or added to
};

// What the tokens of a backward have in common.
struct XentTokens {
  float scale;                     // largest finite |dloss| of those that count
  int masked;                      // one that has no gradient holds an infinity or NaN
  int pad[2];
  float zeros[4];
};

// A token of the backward.
struct alignas(16) XentRow {
  float lse;
  float weight;                    // dloss / scale; 0: it has no gradient
  float entry;                     // p - 1 of its target, or kNoEntry: exp(z - lse) - 1
  int target;                      // column of the whole vocabulary, or -1
};
constexpr float kNoEntry = 2.f;

struct XentGemm {
  // Operands by rows of ld bytes: [M or N][contraction], or, for the kernel's
  // KM operands, [contraction][M or N].  a_rows, b_rows: the rows that exist;
  // kGrad's results past them, up to M and N, are zeros.
  const uint8_t* a; int64_t lda;
  const uint8_t* b; int64_t ldb;
  int a_rows, b_rows;
  int M, N;
  int kblocks;                     // of 64 elements (128 bytes)
  int kb_per_split, splits;
  int rounds;                      // tiles per workgroup (8-wave kernels)
  int tiles_m, tiles_n;
  // kStats
  float2* part;                    // [tiles_n][M] (max, sum of exp(z - max))
  const int64_t* target;
  float* target_logit;             // [M]
  // kGrad
  const XentRow* row;              // [M], kOut [contraction]
  int v0;                          // first vocabulary column of this piece
  float* sums;                     // [tiles_n][a_rows] sums of G's rounded rows over a tile, or nullptr
  // outputs
  void* out; int64_t ldo;          // kGrad, kOut: bf16 elements
  const XentTokens* tokens;        // kOut
  float* acc;                      // kAcc
  int add;                         // acc, sums: add to what is there
};

__device__ __forceinline__ __amdgpu_buffer_rsrc_t rsrc_of(const void* base, int64_t bytes) {
  const uint32_t n = bytes >= 0xFFFFFFFFll ? 0xFFFFFFFFu : (uint32_t)bytes;
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(base), (short)0, (int)n, 0x00020000);
}

// Wait of the slab ring (gfx9 s_waitcnt encoding): at most N of this wave's
// direct loads are still on their way (those of later slabs), its LDS reads
// have returned, then the barrier.
template <int N>
__device__ __forceinline__ void ring_sync() {
  static_assert(N < 64, "vmcnt range");
  __builtin_amdgcn_s_waitcnt((N & 0xF) | (N >> 4) << 14 | 0x7 << 4);
  __builtin_amdgcn_s_barrier();
}

// 16-byte chunk c of LDS row r sits at c ^ swz(r): a fragment read (rows
// l % 16, chunk pair l / 16) and the 1 KB direct writes then meet no bank
// twice in a pass of 16 lanes (rows are 128 bytes).
__device__ __forceinline__ int chunk_swz(int row) { return (row >> 1) & 5; }

__device__ __forceinline__ void tile_order(int tile, int tiles_m, int tiles_n, int* tm, int* tn) {
  constexpr int kGroup = 8;   // row blocks per column sweep: they share W's columns in an XCD's L2
  const int per = kGroup * tiles_n;
  const int g = tile / per, first = g * kGroup;
  const int gm = min(tiles_m - first, kGroup);
  const int in = tile - g * per;
  *tm = first + in % gm;
  *tn = in / gm;
}
// Workgroups are dealt to the 8 XCDs in turn; give each XCD a contiguous range.
__device__ __forceinline__ int xcd_order(int bid, int n) {
  const int x = bid % 8, q = bid / 8, full = n / 8, rem = n % 8;
  return x * full + min(x, rem) + q;
}

__device__ __forceinline__ bf16x8 frag(const uint8_t* tile, uint32_t off) {
  return __builtin_bit_cast(bf16x8, *(const uint4*)(tile + off));
}

// A slab of an operand whose rows run across the contraction: 64 contraction
// rows of C columns, 2 C bytes a row, in units of 32 bytes (16 columns).  Unit
// u of row r sits at u ^ km_swz(r).  A fragment is four consecutive k of one
// column per transposing read (ds_read_b64_tr_b16: element e of lane i of a
// 16-lane group is element i % 4 of the 8 bytes that lane 4 e + i / 4
// addresses), so half a wave reads rows {0-3, 16-19} (+ a constant) of one
// unit column: the swizzle spreads these 8 pieces of 32 bytes over all banks.
// (Rows of 128 bytes, C = 64, alternate between two halves of the banks: two
// bits then do, from the rows of one half.)
template <int C>
__device__ __forceinline__ int km_swz(int row) {
  return C >= 128 ? (row & 3) | ((row >> 4) & 1) << 2 : ((row >> 1) & 1) | ((row >> 4) & 1) << 1;
}
template <int C>
__device__ __forceinline__ bf16x8 frag_km(const uint8_t* tile, uint32_t off) {
  typedef short s16x4 __attribute__((ext_vector_type(4)));
  typedef __attribute__((address_space(3))) s16x4 lds_s16x4;
  typedef __attribute__((address_space(3))) uint8_t lds_u8;
  lds_u8* const t = (lds_u8*)const_cast<uint8_t*>(tile) + off;
  const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)t);
  const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(t + 4 * 2 * C));
  return __builtin_bit_cast(bf16x8, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
}

// One operand's slab by direct loads from LW waves: C rows of 128 bytes,
// or with KM 64 rows of 2 C bytes; 1 KB an instruction either way.  Nothing
// past the operand is read: rows (KM: columns) past its end are replaced by
// ones before it, which reach only results that nobody stores.
// MASK (H in dW, KM): once some token without a gradient holds an infinity or
// NaN, the rows of such tokens are loaded as zeros, as 0 times those is no 0.
template <int C, bool KM, bool MASK, int LW>
struct SlabLoader {
  static constexpr int N = C / (8 * LW);           // loads a wave
  static constexpr int RPL = KM ? 512 / C : 8;     // rows a load covers
  uint32_t off, off_edge;       // a lane's offset in a load's rows; in the load that holds the last row
  uint32_t col0, col1;          // KM: a lane's column bytes, by the swizzle's top bit
  const uint8_t* base;
  int64_t ld;
  int rows, lrow, wave, edge;   // KM: contraction rows; else the load number that holds the last row, -1: all exist
  __amdgpu_buffer_rsrc_t rsrc;
  const XentTokens* tokens;     // MASK
  const XentRow* row;
  bool masked;

  static __device__ __forceinline__ bool upper(int i) { return LW * RPL < 32 && (LW * RPL * i >> 4) & 1; }
  // first: first row (KM: column) of the tile; limit: the operand's; k_rows:
  // its contraction rows (KM).
  __device__ __forceinline__ void init(const uint8_t* p, int64_t ld_, int first, int limit, int k_rows,
                                       int wave_, int lane) {
    ld = ld_;
    wave = wave_;
    rows = k_rows;
    if constexpr (KM) {
      base = p + 2 * (int64_t)first;
      lrow = lane / (64 / RPL);
      const int chunk = lane % (64 / RPL);
      // row = RPL (wave + LW i) + lrow; its bit 4 comes from i or, if LW rows
      // of loads are 32 rows, from the wave
      const int swz = km_swz<C>((RPL * wave + lrow) & 15);
      auto column = [&](int top) {
        const int c = 16 * ((chunk >> 1) ^ (swz | top << (C >= 128 ? 2 : 1))) + 8 * (chunk & 1);
        return (uint32_t)(2 * min(c, limit - first - 8));
      };
      col0 = column(LW * RPL == 32 ? RPL * wave >> 4 : 0);
      col1 = column(1);
      off = (uint32_t)((RPL * wave + lrow) * (int)ld);
    } else {
      base = p + (int64_t)first * ld;
      rsrc = rsrc_of(base, (int64_t)C * ld);
      lrow = lane >> 3;
      const int chunk = (lane & 7) ^ ((4 * (wave & 1) + (lrow >> 1)) & 5);
      const int last = min(limit - first, C) - 1;   // the tile's first row exists
      edge = last + 1 == C ? -1 : last >> 3;
      off = (uint32_t)(lrow * (int)ld + chunk * 16);
      off_edge = (uint32_t)(min(lrow, last & 7) * (int)ld + chunk * 16);
    }
  }
  __device__ __forceinline__ void issue(int kb, uint8_t* lds) const {
#if defined(__HIP_DEVICE_COMPILE__)
    // Load numbers and LDS addresses step from load to load; opaque, or the
    // compiler keeps all N values of each in scalar registers and spills them.
    int to = __builtin_amdgcn_readfirstlane(wave * 1024);
    if constexpr (!KM) {
      const int step = __builtin_amdgcn_readfirstlane(8 * (int)ld);
      if (edge < 0) {   // every row exists
        int so = kb * 128 + __builtin_amdgcn_readfirstlane(wave) * step;
#pragma unroll
        for (int i = 0; i < N; ++i) {
          __builtin_amdgcn_raw_ptr_buffer_load_lds(rsrc, (lds_void*)(lds + to), 16, off, so, 0, 0);
          so += LW * step;
          to += LW * 1024;
          asm volatile("" : "+s"(so), "+s"(to));
        }
      } else {
        int o = __builtin_amdgcn_readfirstlane(wave);
#pragma unroll
        for (int i = 0; i < N; ++i) {
          __builtin_amdgcn_raw_ptr_buffer_load_lds(rsrc, (lds_void*)(lds + to), 16, o < edge ? off : off_edge,
                                                   kb * 128 + min(o, edge) * step, 0, 0);
          o += LW;
          to += LW * 1024;
          asm volatile("" : "+s"(o), "+s"(to));
        }
      }
    } else if (MASK && masked) {
#pragma unroll 1
      for (int i = 0; i < N; ++i) {
        const int t = kb * 64 + RPL * (wave + LW * i) + lrow;
        const bool live = t < rows && row[min(t, rows - 1)].weight != 0.f;
        const uint8_t* const from =
            live ? base + (int64_t)t * ld + (upper(i) ? col1 : col0) : (const uint8_t*)tokens->zeros;
        __builtin_amdgcn_global_load_lds((global_void*)(uintptr_t)from, (lds_void*)(lds + to), 16, 0, 0);
        to = __builtin_amdgcn_readfirstlane(to + LW * 1024);
      }
    } else {
      // A descriptor of its own per slab: offsets stay within 64 rows.
      const __amdgpu_buffer_rsrc_t rs = rsrc_of(base + (int64_t)kb * 64 * ld, 64 * ld);
      const int left = rows - kb * 64;
      if (left >= 64) {
        const int step = __builtin_amdgcn_readfirstlane(LW * RPL * (int)ld);
        int so = 0;
#pragma unroll
        for (int i = 0; i < N; ++i) {
          __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, (lds_void*)(lds + to), 16,
                                                   off + (upper(i) ? col1 : col0), so, 0, 0);
          so += step;
          to += LW * 1024;
          asm volatile("" : "+s"(so), "+s"(to));
        }
      } else {
        // Rows past the last read that one: the other operand is zero there.
#pragma unroll
        for (int i = 0; i < N; ++i)
          __builtin_amdgcn_raw_ptr_buffer_load_lds(
              rs, (lds_void*)(lds + (wave + LW * i) * 1024), 16,
              (uint32_t)(min(RPL * (wave + LW * i) + lrow, left - 1) * (int)ld) +
                  (upper(i) ? col1 : col0),
              0, 0, 0);
      }
    }
#endif
  }
};

// Fragment addresses of one operand's 16-row (16-column) sub-tiles.
template <int C, bool KM>
struct FragReader {
  uint32_t lo, hi;   // !KM: a lane's two 16-byte chunks; KM: lo its row and place in a unit
  int unit, swz;
  // first: the wave's first row (column) in the tile, a multiple of 64
  __device__ __forceinline__ void init(int first, int lane) {
    const int frow = lane & 15, fq = lane >> 4;
    if constexpr (KM) {
      const int row = 16 * fq + (frow >> 2);
      swz = km_swz<C>(row);
      unit = first >> 4;
      lo = row * 2 * C + 8 * (frow & 3);
      hi = 0;
    } else {
      lo = (first + frow) * 128 + (((2 * fq) ^ chunk_swz(first + frow)) << 4);
      hi = (first + frow) * 128 + (((2 * fq + 1) ^ chunk_swz(first + frow)) << 4);
    }
    // Opaque, so that the compiler keeps these and adds constants, instead of
    // one address per fragment and stage.
    asm volatile("" : "+v"(lo));
    if constexpr (!KM) asm volatile("" : "+v"(hi));
  }
  // k = 16 fq + 0 .. 7 (low) and 16 fq + 8 .. 15 (high) of sub-tile i
  __device__ __forceinline__ bf16x8 low(const uint8_t* tile, int i) const {
    if constexpr (KM) return frag_km<C>(tile, lo + (((unit + i) ^ swz) << 5));
    else return frag(tile, lo + 2048 * i);
  }
  __device__ __forceinline__ bf16x8 high(const uint8_t* tile, int i) const {
    if constexpr (KM) return frag_km<C>(tile, lo + (((unit + i) ^ swz) << 5) + 8 * 2 * C);
    else return frag(tile, hi + 2048 * i);
  }
};

// One output tile and its slabs.
struct Tile {
  int m0, n0, tn, split, kb0, kb1;
};

// C[m, n] = sum_k A[m, k] B[n, k] on BM x BN tiles of WGM x WGN waves.  A ring
// of stages of 64 contraction elements in LDS, filled by direct buffer -> LDS
// loads from waves 0 and 1 (a direct load keeps the issuing wave for about 16
// cycles; the others go straight to their MFMAs), or from all four of the 64-row
// kernels, where a tile waits for its slabs (12 tokens, 6853 x 3840: forward 40.2
// us from two, 37.7 from four).  Each stage is an LDS
// variable of its own and the stage loop is unrolled, so that the compiler
// sees that reads of one stage do not depend on loads into another.
//
// 256 x 256 tiles (8 waves, two stages, 128 KB of a CU's 160 KB of LDS and up to
// 17 KB for an epilogue: one workgroup a CU) read the fewest operand bytes per
// product; 128 x 256 tiles (8 waves, three stages, 144 KB) do for 65 to 128
// tokens.  64-row tiles (4 waves, two workgroups a CU) serve few tokens
// or columns: 64 x 256 with two stages where W streams by, 64 x 128 with three
// where a tile takes what the wait for its slabs takes.
//
// A workgroup of the 8-wave kernels runs `rounds` tiles, a chip's worth of
// workgroups apart, and starts the next tile's first slab before it works off
// this one's epilogue, which uses LDS beside that stage; its results are stored
// by the waves that load nothing, so that no load waits for them.
// Any M and N: a tile past an edge loads rows again and stores only its own.
template <int BM, int BN, int WGM, int WGN, int STAGES, int EPI, bool AKM, bool BKM>
__device__ __forceinline__ void xent_tiles(const XentGemm& p, int block, uint8_t* const (&sA)[kMaxStages],
                                           uint8_t* const (&sB)[kMaxStages], uint8_t* sE) {
  constexpr bool SMALL = BM == 64;
  constexpr int LW = SMALL ? 4 : 2;                       // loading waves
  constexpr int LATER = (STAGES - 2) * (BM + BN) / (8 * LW);         // a loading wave's loads of the later slabs
  constexpr int NW = WGM * WGN;
  constexpr int WM = BM / WGM, WN = BN / WGN, TM = WM / 16, TN = WN / 16;
  constexpr bool ROWS = EPI == kStats || EPI == kGrad;       // the epilogue needs its rows' targets
  constexpr int SUM_LD = BM + 16;                            // kGrad's row sums: no bank twice in a write
  constexpr bool STAGED = !SMALL && (EPI == kGrad || EPI == kOut);
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
  const int wm0 = (wave / WGN) * WM, wn0 = (wave % WGN) * WN;
  const int frow = lane & 15, fq = lane >> 4;
  const int tiles = p.tiles_m * p.tiles_n, total = tiles * p.splits;
  // (split, tile), split-major, contiguous per XCD
  auto locate = [&](int n) __attribute__((always_inline)) -> Tile {
    const int id = xcd_order(n, total);
    Tile t;
    t.split = id / tiles;
    int tm;
    tile_order(id - t.split * tiles, p.tiles_m, p.tiles_n, &tm, &t.tn);
    t.m0 = tm * BM;
    t.n0 = t.tn * BN;
    t.kb0 = t.split * p.kb_per_split;
    t.kb1 = min(p.kblocks, t.kb0 + p.kb_per_split);
    return t;
  };
  SlabLoader<BM, AKM, false, LW> la;
  SlabLoader<BN, BKM, EPI == kOut, LW> lb;
  auto issue = [&](int kb, uint8_t* sa, uint8_t* sb) __attribute__((always_inline)) {
    if (LW == WGM * WGN || wave < LW) {
      la.issue(kb, sa);
      lb.issue(kb, sb);
    }
  };
  auto begin = [&](const Tile& t) __attribute__((always_inline)) {
    la.init(p.a, p.lda, t.m0, AKM ? p.tiles_m * BM : p.a_rows, p.a_rows, wave, lane);
    lb.init(p.b, p.ldb, t.n0, BKM ? p.N : p.b_rows, p.b_rows, wave, lane);
    if (t.kb0 < t.kb1) {
#pragma unroll
      for (int st = 0; st < STAGES - 1; ++st) issue(min(t.kb0 + st, t.kb1 - 1), sA[st], sB[st]);
    }
  };
  float scale = 1.f;
  if constexpr (EPI == kOut) {
    scale = p.tokens->scale;
    lb.tokens = p.tokens;
    lb.row = p.row;
    lb.masked = p.tokens->masked != 0;
  }

  // Workgroups 0 .. kCus - 1 start with tiles 0 .. kCus - 1, the next kCus
  // after all of theirs.
  int number = SMALL ? block : block / kCus * (kCus * p.rounds) + block % kCus;
  if (number >= total) return;
  const int last = SMALL ? total : min(total, (block / kCus + 1) * kCus * p.rounds);
  Tile t = locate(number);
  begin(t);
  for (;;) {
    // The epilogue's rows, read before the slabs so that nothing waits for
    // them: target column in this wave's, lse and weight.
    int tgt[ROWS ? TM : 1];
    float2 info[EPI == kGrad ? TM : 1];
    if constexpr (ROWS) {
#pragma unroll
      for (int i = 0; i < TM; ++i) {
        const int r = min(t.m0 + wm0 + 16 * i + frow, p.a_rows - 1);
        int64_t y;
        if constexpr (EPI == kGrad) {
          const XentRow e = p.row[r];
          info[i] = make_float2(e.lse, e.weight);
          y = (int64_t)e.target - p.v0;
        } else {
          y = p.target[r];
        }
        y -= t.n0 + wn0;
        tgt[i] = y >= 0 && y < WN ? (int)y : -1;
        if constexpr (EPI == kGrad) {
          if (t.m0 + wm0 + 16 * i + frow >= p.a_rows) info[i].y = 0.f;
        }
      }
    }
    v4f acc[TM][TN];
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
      for (int j = 0; j < TN; ++j) acc[i][j] = v4f{0.f, 0.f, 0.f, 0.f};

    ring_sync<LATER>();
    for (int it = t.kb0; it < t.kb1; it += STAGES) {
#pragma unroll
      for (int st = 0; st < STAGES; ++st) {
        const int kb = it + st;
        if (kb >= t.kb1) break;
        // past the end the last slab is loaded again, into a stage nobody reads
        issue(min(kb + STAGES - 1, t.kb1 - 1), sA[(st + STAGES - 1) % STAGES], sB[(st + STAGES - 1) % STAGES]);
        const uint8_t* const ta = sA[st];
        const uint8_t* const tb = sB[st];
        FragReader<BM, AKM> ra;
        FragReader<BN, BKM> rb;
        ra.init(wm0, lane);
        rb.init(wn0, lane);
        bf16x8 bl[TN], bh[TN], al[2], ah[2];
        bl[0] = rb.low(tb, 0);
        al[0] = ra.low(ta, 0);
#pragma unroll
        for (int j = 1; j < TN; ++j) bl[j] = rb.low(tb, j);
        ah[0] = ra.high(ta, 0);
#pragma unroll
        for (int j = 0; j < TN; ++j) bh[j] = rb.high(tb, j);
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int i = 0; i < TM; ++i) {
          if (i + 1 < TM) {
            al[(i + 1) & 1] = ra.low(ta, i + 1);
            ah[(i + 1) & 1] = ra.high(ta, i + 1);
            __builtin_amdgcn_sched_barrier(0);   // keep the next row's reads ahead of this row's MFMAs
          }
          // B first: lane l then holds row 16 i + l % 16, columns 16 j + 4 (l / 16) + 0..3
#pragma unroll
          for (int j = 0; j < TN; ++j)
            acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(bl[j], al[i & 1], acc[i][j], 0, 0, 0);
#pragma unroll
          for (int j = 0; j < TN; ++j)
            acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(bh[j], ah[i & 1], acc[i][j], 0, 0, 0);
        }
        ring_sync<LATER>();
      }
    }
    ring_sync<0>();
    __syncthreads();   // every wave's reads and loads are done: the stages are free
    const Tile d = t;
    number += kCus;
    const bool more = !SMALL && number < last;
    if (more) {
      t = locate(number);
      begin(t);
    }

    const int row0 = d.m0 + wm0 + frow;            // + 16 i
    const int col0 = d.n0 + wn0 + 4 * fq;          // + 16 j + v
    const bool whole = d.n0 + wn0 + WN <= p.N;     // every column of this wave's exists
    if constexpr (EPI == kStats) {
      // Maximum and sum of exponentials of each row over this wave's columns
      // (a row's columns lie in lanes frow + 16 q), then over the waves.
      float2* const red = (float2*)sE;          // [WGN][BM]
      auto statistics = [&](auto check) __attribute__((always_inline)) {
        constexpr bool kCheck = decltype(check)::value;
#pragma unroll
        for (int i = 0; i < TM; ++i) {
          const int r = row0 + 16 * i;
          if (__builtin_amdgcn_ballot_w64(tgt[i] >= 0)) {       // a target among these columns: rarely
#pragma unroll
            for (int j = 0; j < TN; ++j)
#pragma unroll
              for (int v = 0; v < 4; ++v)
                if (16 * j + 4 * fq + v == tgt[i]) {
                  if (r < p.M) p.target_logit[r] = acc[i][j][v];
                  acc[i][j][v] = -INFINITY;   // joined to the others last
                }
          }
          float m = -INFINITY;
#pragma unroll
          for (int j = 0; j < TN; ++j)
#pragma unroll
            for (int v = 0; v < 4; ++v) {
              if constexpr (kCheck) {
                if (col0 + 16 * j + v >= p.N) acc[i][j][v] = -INFINITY;
              }
              m = fmaxf(m, acc[i][j][v]);   // drops a NaN; the sum below does not
            }
          m = fmaxf(m, __shfl_xor(m, 16));
          m = fmaxf(m, __shfl_xor(m, 32));
          const float base = m == -INFINITY ? 0.f : m;   // no column, or all at -inf
          float s = 0.f;
#pragma unroll
          for (int j = 0; j < TN; ++j)
#pragma unroll
            for (int v = 0; v < 4; ++v) s += __builtin_amdgcn_exp2f((acc[i][j][v] - base) * kLog2e);
          s += __shfl_xor(s, 16);
          s += __shfl_xor(s, 32);
          if (fq == 0) red[(wave % WGN) * BM + wm0 + 16 * i + frow] = make_float2(m, s);
        }
      };
      if (whole) statistics(std::false_type{});
      else statistics(std::true_type{});
      __syncthreads();
      for (int r = threadIdx.x; r < BM; r += 64 * NW) {
        float m = -INFINITY;
#pragma unroll
        for (int w = 0; w < WGN; ++w) m = fmaxf(m, red[w * BM + r].x);
        float s = 0.f;
#pragma unroll
        for (int w = 0; w < WGN; ++w) {
          const float2 e = red[w * BM + r];
          if (e.x != -INFINITY) s += e.y * __builtin_amdgcn_exp2f((e.x - m) * kLog2e);
          else s += e.y;     // 0, or NaN
        }
        const int row = d.m0 + r;
        if (row < p.M) p.part[(int64_t)d.tn * p.M + row] = make_float2(m, s);
      }
    } else if constexpr (EPI == kAcc) {
      float* const base = p.acc + (int64_t)d.split * p.M * p.N;
#pragma unroll
      for (int i = 0; i < TM; ++i) {
        const int r = row0 + 16 * i;
        if (r >= p.M) continue;
#pragma unroll
        for (int j = 0; j < TN; ++j) {
          const int n = col0 + 16 * j;
          if (n >= p.N) continue;   // N is a multiple of 64: all four columns exist or none
          float4* const at = (float4*)(base + (int64_t)r * p.N + n);
          float4 o = make_float4(acc[i][j][0], acc[i][j][1], acc[i][j][2], acc[i][j][3]);
          if (p.add) {
            const float4 e = *at;
            o.x += e.x; o.y += e.y; o.z += e.z; o.w += e.w;
          }
          *at = o;
        }
      }
    } else {
      uint16_t* const out = (uint16_t*)p.out;
      // Lane row i's columns as bf16: G's, or the product times scale.
      auto results = [&](int i, uint2 (&w)[TN]) __attribute__((always_inline)) {
        if constexpr (EPI == kGrad) {
#pragma unroll
          for (int j = 0; j < TN; ++j)
#pragma unroll
            for (int v = 0; v < 4; ++v)
              acc[i][j][v] = __builtin_amdgcn_exp2f((acc[i][j][v] - info[i].x) * kLog2e);
          if (__builtin_amdgcn_ballot_w64(tgt[i] >= 0)) {
            int r = min(row0 + 16 * i, p.a_rows - 1);
            asm volatile("" : "+v"(r));   // formed here, not for all rows ahead
            const float entry = p.row[r].entry;
#pragma unroll
            for (int j = 0; j < TN; ++j)
#pragma unroll
              for (int v = 0; v < 4; ++v)
                if (16 * j + 4 * fq + v == tgt[i]) acc[i][j][v] = entry == kNoEntry ? acc[i][j][v] - 1.f : entry;
          }
        }
        const float f = EPI == kGrad ? info[i].y : scale;
        // a row of weight zero (an ignored target) has no gradient, whatever its logits
        const uint32_t keep = EPI == kGrad && f == 0.f ? 0u : ~0u;
        if (EPI == kGrad && d.n0 + wn0 + WN > p.b_rows) {
#pragma unroll
          for (int j = 0; j < TN; ++j)
#pragma unroll
            for (int v = 0; v < 4; ++v)
              if (col0 + 16 * j + v >= p.b_rows) acc[i][j][v] = 0.f;
        }
#pragma unroll
        for (int j = 0; j < TN; ++j)
          w[j] = make_uint2(pack_bf16x2_rne(acc[i][j][0] * f, acc[i][j][1] * f) & keep,
                            pack_bf16x2_rne(acc[i][j][2] * f, acc[i][j][3] * f) & keep);
        if constexpr (EPI == kGrad) {   // the lane's share of the rounded row's sum
          float s = 0.f;
#pragma unroll
          for (int j = 0; j < TN; ++j) s += (bf16lo(w[j].x) + bf16hi(w[j].x)) + (bf16lo(w[j].y) + bf16hi(w[j].y));
          ((float*)sE)[(wave % WGN * 4 + fq) * SUM_LD + wm0 + 16 * i + frow] = s;
        }
      };
      // Thread `r` of the last BM joins row r's 4 WGN shares.  What an earlier
      // piece left is read before the epilogue's work.
      auto sum_row = [&]() __attribute__((always_inline)) {
        int r = (int)threadIdx.x - (64 * NW - BM);
        asm volatile("" : "+v"(r));
        return EPI == kGrad && p.sums && r >= 0 && d.m0 + r < p.a_rows ? r : -1;
      };
      float sum = 0.f;
      if (const int r = sum_row(); p.add && r >= 0) sum = p.sums[(int64_t)d.tn * p.a_rows + d.m0 + r];
      auto join = [&]() __attribute__((always_inline)) {
        const int r = sum_row();
        if (r < 0) return;
        float s = 0.f;
#pragma unroll
        for (int k = 0; k < 4 * WGN; ++k) s += ((const float*)sE)[k * SUM_LD + r];
        p.sums[(int64_t)d.tn * p.a_rows + d.m0 + r] = sum + s;
      };
      if constexpr (STAGED) {
        // Through LDS, so that every store writes whole lines (in the MFMA
        // layout a row of a wave's columns would leave in pieces of 32 bytes):
        // half of each wave's rows at a time, rows of 512 bytes in the last
        // stage, which the next tile's first slabs leave alone; 16-byte chunk c
        // of row r at c ^ (r & 15).
#pragma unroll
        for (int h = 0; h < 2; ++h) {
#pragma unroll
          for (int ii = 0; ii < TM / 2; ++ii) {
            uint2 w[TN];
            results(TM / 2 * h + ii, w);
            uint8_t* const rowp = (wm0 ? sB : sA)[STAGES - 1] + (16 * ii + frow) * 512;
#pragma unroll
            for (int j = 0; j < TN; ++j)
              *(uint2*)(rowp + 16 * (((wn0 >> 3) + 2 * j + (fq >> 1)) ^ frow) + 8 * (fq & 1)) = w[j];
          }
          __syncthreads();
          if (h == 1) join();
          const int c = lane & 31, n = d.n0 + 8 * c;
          if (wave >= 2) {
            constexpr int PAIRS = WM / 4;   // of rows, in half of a wave's
            for (int pr = wave - 2; pr < 2 * PAIRS; pr += NW - 2) {
              const int rr = 2 * (pr % PAIRS) + (lane >> 5), r = d.m0 + WM * (pr / PAIRS) + WM / 2 * h + rr;
              const u32x4_t v =
                  *(const u32x4_t*)((pr / PAIRS ? sB : sA)[STAGES - 1] + rr * 512 + 16 * (c ^ (rr & 15)));
              if (r >= p.M || n >= p.N) continue;
              uint16_t* const at = out + (int64_t)r * p.ldo + n;
              if (n + 7 < p.N) {
                if constexpr (EPI == kOut) __builtin_nontemporal_store(v, (u32x4_t*)at);
                else *(u32x4_t*)at = v;   // the next products read G
              } else {
#pragma unroll
                for (int e = 0; e < 8; ++e)
                  if (n + e < p.N) at[e] = (uint16_t)(v[e >> 1] >> (16 * (e & 1)));
              }
            }
          }
          __syncthreads();
        }
      } else {
#pragma unroll
        for (int i = 0; i < TM; ++i) {
          const int r = row0 + 16 * i;
          uint2 w[TN];
          results(i, w);
          if (r >= p.M) continue;
#pragma unroll
          for (int j = 0; j < TN; ++j) {
            const int n = col0 + 16 * j;
            uint16_t* const at = out + (int64_t)r * p.ldo + n;
            if (n + 3 < p.N) {
              *(uint2*)at = w[j];
            } else {
#pragma unroll
              for (int v = 0; v < 4; ++v)
                if (n + v < p.N) at[v] = (uint16_t)((v < 2 ? w[j].x : w[j].y) >> (16 * (v & 1)));
            }
          }
        }
        if constexpr (EPI == kGrad) {
          __syncthreads();
          join();
        }
      }
    }
    if (!more) return;
  }
}

// A kernel's stages, and its waves' row statistics or sums (64-row kernels: in a stage).
#define XENT_LDS(BM, BN, WGN, STAGES, EPI)                                                            \
  __shared__ __attribute__((aligned(1024))) uint8_t sA0[BM * 128], sA1[BM * 128];                     \
  __shared__ __attribute__((aligned(1024))) uint8_t sB0[BN * 128], sB1[BN * 128];                     \
  __shared__ __attribute__((aligned(1024))) uint8_t sA2[STAGES > 2 ? BM * 128 : 16];                  \
  __shared__ __attribute__((aligned(1024))) uint8_t sB2[STAGES > 2 ? BN * 128 : 16];                  \
  __shared__ __attribute__((aligned(16))) uint8_t sums[BM == 64        ? 16                           \
                                                       : EPI == kStats ? WGN * BM * 8                 \
                                                       : EPI == kGrad  ? WGN * (BM + 16) * 16         \
                                                                       : 16];                         \
  uint8_t* const sA[kMaxStages] = {sA0, sA1, sA2};                                                    \
  uint8_t* const sB[kMaxStages] = {sB0, sB1, sB2};                                                    \
  uint8_t* const sE = BM > 64 ? sums : sA0

template <int BM, int BN, int WGM, int WGN, int STAGES, int EPI, bool AKM, bool BKM>
__global__ __launch_bounds__(64 * WGM * WGN) void xent_gemm_kernel(const XentGemm p) {
  XENT_LDS(BM, BN, WGN, STAGES, EPI);
  xent_tiles<BM, BN, WGM, WGN, STAGES, EPI, AKM, BKM>(p, blockIdx.x, sA, sB, sE);
}

// dH's and dW's products in one launch: the first workgroups dH's, which are
// the longer, then dW's, which fill what they leave.
template <int BM, int BN, int WGM, int WGN, int STAGES>
__global__ __launch_bounds__(64 * WGM * WGN) void xent_pair_kernel(const XentGemm h, const XentGemm w, int h_blocks) {
  XENT_LDS(BM, BN, WGN, STAGES, kOut);
  if ((int)blockIdx.x < h_blocks)
    xent_tiles<BM, BN, WGM, WGN, STAGES, kAcc, false, true>(h, blockIdx.x, sA, sB, sE);
  else
    xent_tiles<BM, BN, WGM, WGN, STAGES, kOut, true, true>(w, blockIdx.x - h_blocks, sA, sB, sE);
}

// (m, s) and (m2, s2): sums of exponentials s, s2 beside their maxima.
__device__ __forceinline__ void join_sums(float& m, float& s, float m2, float s2) {
  const float top = fmaxf(m, m2);
  const float base = top == -INFINITY ? 0.f : top;
  s = s * __builtin_amdgcn_exp2f((m - base) * kLog2e) + s2 * __builtin_amdgcn_exp2f((m2 - base) * kLog2e);
  m = top;
}

// lse and loss of a token from the maximum m and the sum of exponentials s of
// the columns beside its target (of all, where the target counts not or is
// outside the vocabulary), and the target's logit z.
__device__ __forceinline__ void token_loss(float m, float s, int64_t y, int64_t V, int64_t ignore_index, float z,
                                           float* lse, float* loss) {
  const bool known = y >= 0 && y < V;
  float l, d;
  if (known && fabsf(z) < INFINITY) {
    // log of the others' sum over the target's exponential
    const float gap = s == 0.f ? -INFINITY : (m - z) + logf(s);
    const float tail = log1pf(expf(-fabsf(gap)));
    d = gap > 0.f ? gap + tail : tail;
    l = gap > 0.f ? (m + logf(s)) + tail : z + tail;
  } else {
    if (known) join_sums(m, s, z, 1.f);
    l = (m == -INFINITY ? 0.f : m) + logf(s);
    d = known ? l - z : __builtin_nanf("");
  }
  *lse = l;
  *loss = y == ignore_index ? 0.f : d;
}

// Joins the tiles' (max, sum) of 16 tokens: 64 threads a token over the
// tiles, then over the threads in a fixed order.
__global__ __launch_bounds__(1024) void xent_join_kernel(const float2* __restrict__ part, int tiles,
                                                         int T, int64_t V,
                                                         const float* __restrict__ target_logit,
                                                         const int64_t* __restrict__ target,
                                                         int64_t ignore_index, float* __restrict__ loss,
                                                         float* __restrict__ lse) {
  __shared__ float2 red[16][17];
  const int c = threadIdx.x & 15, g = threadIdx.x >> 4;
  const int t = blockIdx.x * 16 + c;
  float m = -INFINITY, s = 0.f;
  if (t < T) {
#pragma unroll 4
    for (int i = g; i < tiles; i += 64) {
      const float2 e = part[(int64_t)i * T + t];
      join_sums(m, s, e.x, e.y);
    }
  }
#pragma unroll
  for (int x = 16; x < 64; x *= 2) join_sums(m, s, __shfl_xor(m, x), __shfl_xor(s, x));
  if (threadIdx.x % 64 < 16) red[threadIdx.x >> 6][c] = make_float2(m, s);
  __syncthreads();
  if (g == 0 && t < T) {
#pragma unroll
    for (int i = 1; i < 16; ++i) join_sums(m, s, red[i][c].x, red[i][c].y);
    const int64_t y = target[t];
    const float z = y >= 0 && y < V ? target_logit[t] : 0.f;
    token_loss(m, s, y, V, ignore_index, z, lse + t, loss + t);
  }
}

// scale = max finite |dloss| over the tokens that count, and the tokens' rows;
// ignored and out-of-range targets get weight 0.
// An infinity or NaN in a token's row of H makes every one of its logits
// infinite or NaN, and so its lse.
__global__ __launch_bounds__(1024) void xent_rows_kernel(int T, int64_t V, const int64_t* __restrict__ target,
                                                         int64_t ignore_index, const float* __restrict__ dloss,
                                                         const float* __restrict__ lse, const float* __restrict__ loss,
                                                         XentRow* __restrict__ row, XentTokens* __restrict__ tokens) {
  __shared__ float red[16];
  float m = 0.f;
  for (int t = threadIdx.x; t < T; t += 1024) {
    const int64_t y = target[t];
    const float d = fabsf(dloss[t]);
    if (y != ignore_index && y >= 0 && y < V && d < INFINITY) m = fmaxf(m, d);
  }
  m = wave_max(m);
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = m;
  __syncthreads();
  m = 0.f;
  for (int i = 0; i < 16; ++i) m = fmaxf(m, red[i]);
  bool masked = false;
  for (int t = threadIdx.x; t < T; t += 1024) {
    const int64_t y = target[t];
    const bool counts = y != ignore_index && y >= 0 && y < V;
    XentRow r;
    r.lse = lse[t];
    r.weight = counts && dloss[t] != 0.f ? dloss[t] / m : 0.f;
    r.entry = loss ? expm1f(-loss[t]) : kNoEntry;
    r.target = counts ? (int)y : -1;
    row[t] = r;
    masked |= r.weight == 0.f && !(fabsf(r.lse) < INFINITY);
  }
  const int any = __syncthreads_or(masked);
  if (threadIdx.x == 0) *tokens = XentTokens{m, any, {0, 0}, {0.f, 0.f, 0.f, 0.f}};
}

// Sum over the 256 threads of a workgroup, in a fixed order; `red` is free
// again after the caller's next barrier.
__device__ __forceinline__ float block_sum(float v, float* red) {
#pragma unroll
  for (int x = 1; x < 64; x *= 2) v += __shfl_xor(v, x);
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
  __syncthreads();
  return (red[0] + red[1]) + (red[2] + red[3]);
}

// Columns c .. c + 3 of the sum of `splits` shares of the logits, in order.
__device__ __forceinline__ float4 sum_shares(const float* z, int64_t c, int splits, int64_t share) {
  float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int k = 0; k < splits; ++k) {
    const float4 e = *(const float4*)(z + k * share + c);
    s.x += e.x; s.y += e.y; s.z += e.z; s.w += e.w;
  }
  return s;
}

// One token's lse and loss from shares of its logits, [splits][T][ld].  (16000
// columns: with 256 threads a token 7 us more than with 1024.)
__global__ __launch_bounds__(1024) void xent_few_stats_kernel(const float* __restrict__ z, int splits, int T,
                                                             int64_t V, int64_t ld,
                                                             const int64_t* __restrict__ target,
                                                             int64_t ignore_index, float* __restrict__ loss,
                                                             float* __restrict__ lse) {
  __shared__ float2 red[16];
  const int t = blockIdx.x;
  const float* const row = z + t * ld;
  const int64_t share = T * ld;
  const int64_t y = target[t];
  float m = -INFINITY, s = 0.f;
  for (int64_t c = 4 * threadIdx.x; c < V; c += 4 * blockDim.x) {
    const float4 e = sum_shares(row, c, splits, share);
    if (c != y) join_sums(m, s, e.x, 1.f);
    if (c + 1 < V && c + 1 != y) join_sums(m, s, e.y, 1.f);
    if (c + 2 < V && c + 2 != y) join_sums(m, s, e.z, 1.f);
    if (c + 3 < V && c + 3 != y) join_sums(m, s, e.w, 1.f);
  }
#pragma unroll
  for (int x = 1; x < 64; x *= 2) join_sums(m, s, __shfl_xor(m, x), __shfl_xor(s, x));
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = make_float2(m, s);
  __syncthreads();
  if (threadIdx.x) return;
  for (int i = 1; i < (int)blockDim.x / 64; ++i) join_sums(m, s, red[i].x, red[i].y);
  float own = 0.f;
  if (y >= 0 && y < V)
    for (int k = 0; k < splits; ++k) own += row[k * share + y];
  token_loss(m, s, y, V, ignore_index, own, lse + t, loss + t);
}

// G from shares of the logits, [splits][T][ld]; zeros past T and V.  sums: a
// workgroup's of G's rounded row.
__global__ __launch_bounds__(256) void xent_few_grad_kernel(const float* __restrict__ z, int splits, int T, int V,
                                                            int ld, const XentRow* __restrict__ row, int v0,
                                                            uint16_t* __restrict__ g, int64_t ld_g,
                                                            float* __restrict__ sums) {
  __shared__ float red[4];
  const int t = blockIdx.x, c = 4 * (blockIdx.y * 256 + threadIdx.x);
  uint2 w = make_uint2(0, 0);
  const XentRow info = t < T ? row[t] : XentRow{0.f, 0.f, 0.f, -1};
  if (info.weight != 0.f && c < ld) {
    const float4 e = sum_shares(z + (int64_t)t * ld, c, splits, (int64_t)T * ld);
    float p[4] = {e.x, e.y, e.z, e.w};
    const int y = info.target - v0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      p[i] = __builtin_amdgcn_exp2f((p[i] - info.lse) * kLog2e);
      if (c + i == y) p[i] = info.entry == kNoEntry ? p[i] - 1.f : info.entry;
      p[i] = c + i < V ? p[i] * info.weight : 0.f;
    }
    w = make_uint2(pack_bf16x2_rne(p[0], p[1]), pack_bf16x2_rne(p[2], p[3]));
  }
  if (c < ld) *(uint2*)(g + t * ld_g + c) = w;
  if (!sums || t >= T) return;
  const float s = block_sum((bf16lo(w.x) + bf16hi(w.x)) + (bf16lo(w.y) + bf16hi(w.y)), red);
  if (threadIdx.x == 0) sums[(int64_t)blockIdx.y * T + t] = s;
}

// Zeros in columns [c0, c1) of bf16 rows: one row and 2048 columns a workgroup.
__global__ __launch_bounds__(256) void zero_columns_kernel(uint16_t* out, int64_t ld, int64_t rows, int64_t c0,
                                                           int64_t c1) {
  const int64_t end = min(c1, c0 + ((int64_t)blockIdx.y + 1) * 2048);
  for (int64_t r = blockIdx.x; r < rows; r += gridDim.x)
    for (int64_t c = c0 + (int64_t)blockIdx.y * 2048 + threadIdx.x; c < end; c += 256) out[r * ld + c] = 0;
}

// dH = scale * (sum over the splits of their fp32 shares - the sum of the
// token's rounded G times the target's row of W), to bf16: a token and 1024
// columns a workgroup.
__global__ __launch_bounds__(256) void xent_dh_kernel(const float* __restrict__ acc, int splits, int64_t T,
                                                      int64_t K, const XentTokens* __restrict__ tokens,
                                                      const XentRow* __restrict__ row,
                                                      const float* __restrict__ sums, int parts,
                                                      const uint16_t* __restrict__ w, int64_t ld_w,
                                                      uint16_t* __restrict__ dh, int64_t ld_dh) {
  __shared__ float red[2][4];
  const float f = tokens->scale;
  const int64_t c = ((int64_t)blockIdx.y * 256 + threadIdx.x) * 4;
  int flip = 0;   // one barrier a token
  for (int64_t t = blockIdx.x; t < T; t += gridDim.x, flip ^= 1) {
    float part = 0.f;
    for (int i = threadIdx.x; i < parts; i += 256) part += sums[i * T + t];
    float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
    if (c < K) s = sum_shares(acc + t * K, c, splits, T * K);
    const float off = block_sum(part, red[flip]);
    if (c >= K) continue;
    if (row[t].weight != 0.f) {   // else G is zero, and W's row may be anything
      const uint2 u = *(const uint2*)(w + row[t].target * ld_w + c);
      s.x -= off * bf16lo(u.x); s.y -= off * bf16hi(u.x);
      s.z -= off * bf16lo(u.y); s.w -= off * bf16hi(u.y);
    }
    *(uint2*)(dh + t * ld_dh + c) =
        make_uint2(pack_bf16x2_rne(s.x * f, s.y * f), pack_bf16x2_rne(s.z * f, s.w * f));
  }
}

int64_t pad64(int64_t n) { return (n + 63) & ~(int64_t)63; }

// Large tiles for more than 128 rows, once they (times the splits of the
// contraction) fill half the chip's compute units; else 64-row tiles.
// (131072 x 5120, forward: 100 tokens 337 us on 64-row tiles, 356 us on large
// ones; 131072 x 4096: 255 tokens 402 us and 311 us.)
bool large_tiles(int64_t M, int64_t N, int64_t splits) {
  return M > 128 && ((M + 255) / 256) * ((N + 255) / 256) * splits >= kCus / 2;
}
// Tiles of the logits: rows and columns.  Below the large ones, 128 rows for 65
// to 128 tokens once the columns fill half the chip; else 64, with 256 columns
// once these tiles fill the chip twice.  (100 tokens, 131072 x 5120: 261 us on
// 128 rows, 331 us on 64.  33 tokens: 246 us with 128 columns, 223 to 231 us with
// 256; a step of 128 tokens, 2048 x 512: 43 us with 128, 52 us with 256.  Each
// pair on one build.)
struct TileShape {
  int rows, cols;
};
TileShape logit_tiles(int64_t T, int64_t V) {
  if (large_tiles(T, V, 1)) return {256, 256};
  const int64_t wide = (V + 255) / 256;
  if (T > 64 && T <= 128 && wide >= kCus / 2) return {128, 256};
  return {64, (T + 63) / 64 * wide >= 2 * kCus ? 256 : 128};
}

// Tiles of the gradients' products; `splits` of the contraction (dH).  (dH of
// 100 tokens, 131072 x 4096: 177 us on 128 rows, 354 us on 64.)
TileShape gradient_tiles(int64_t M, int64_t N, int64_t splits) {
  if (large_tiles(M, N, splits)) return {256, 256};
  if (splits > 1 && M > 64 && M <= 128 && (N + 255) / 256 * splits >= kCus / 2) return {128, 256};
  return {64, 128};
}

// Tiles a workgroup: more hide more epilogues, but workgroups drift apart
// within a launch and then share fewer operand slices in the L2.
constexpr int kRounds = 4;

// A product's tiles; the workgroups that run them.
int64_t lay_out(XentGemm* p, TileShape tile, int splits, int rounds) {
  p->tiles_m = (p->M + tile.rows - 1) / tile.rows;
  p->tiles_n = (p->N + tile.cols - 1) / tile.cols;
  p->splits = splits;
  p->kb_per_split = (p->kblocks + splits - 1) / splits;
  p->rounds = rounds;
  const int64_t tiles = (int64_t)p->tiles_m * p->tiles_n * splits;
  return tile.rows == 64 ? tiles : (tiles + kCus * rounds - 1) / (kCus * rounds) * kCus;
}

template <int EPI, bool AKM = false, bool BKM = false>
hipError_t run_gemm(XentGemm p, TileShape tile, int splits, hipStream_t stream) {
  constexpr bool LOGITS = EPI == kStats || EPI == kGrad;
  const dim3 grid((unsigned)lay_out(&p, tile, splits, kRounds));
  if (tile.rows == 256)
    hipLaunchKernelGGL((xent_gemm_kernel<256, 256, 2, 4, 2, EPI, AKM, BKM>), grid, dim3(512), 0, stream, p);
  else if (tile.cols == 128)
    hipLaunchKernelGGL((xent_gemm_kernel<64, 128, 1, 4, 3, EPI, AKM, BKM>), grid, dim3(256), 0, stream, p);
  else if constexpr (EPI != kOut) {   // dW has no shape of few rows and many columns
    if (tile.rows == 128)
      hipLaunchKernelGGL((xent_gemm_kernel<128, 256, 2, 4, 3, EPI, AKM, BKM>), grid, dim3(512), 0, stream, p);
    else if constexpr (LOGITS)
      hipLaunchKernelGGL((xent_gemm_kernel<64, 256, 1, 4, 2, EPI, AKM, BKM>), grid, dim3(256), 0, stream, p);
  }
  return hipGetLastError();
}

// Shares of the logits' contraction, where their tiles leave half the chip idle
// and it is long: a slab takes such a tile about 0.55 us, whether three or six
// stages are on their way.  The fp32 shares, at least 8 slabs each, are then
// summed by kernels of their own.  (12 tokens, 6853 x 3840: forward 38 to 24 us;
// 12 tokens, 3426 x 4224: step 101 to 58 us; 64 tokens, 16000 x 4096: 141 to 127
// us.  With 16 slabs no gain: 12 tokens, 6853 x 1024 16 us either way.)
int logit_splits(int64_t T, int64_t V, int64_t K) {
  const TileShape tile = logit_tiles(T, V);
  const int64_t tiles = ((T + 63) / 64) * ((V + 127) / 128), slabs = K / 64;
  if (tile.rows != 64 || tile.cols != 128 || tiles > kCus / 2 || slabs < 24) return 1;
  return (int)(kCus / tiles < slabs / 8 ? kCus / tiles : slabs / 8);
}

hipError_t run_logit_shares(XentGemm p, int splits, float* z, hipStream_t stream) {
  p.M = p.a_rows;
  p.N = (int)pad64(p.b_rows);
  p.acc = z;
  const dim3 grid((unsigned)lay_out(&p, {64, 128}, splits, 1));
  hipLaunchKernelGGL((xent_gemm_kernel<64, 128, 1, 4, 3, kAcc, false, false>), grid, dim3(256), 0, stream, p);
  return hipGetLastError();
}

// dH's share of a piece and the piece's dW, in one launch where both take the
// same tiles: one launch fewer (128 tokens, 2048 x 512: 42.6 to 38 us a step),
// and dW's tiles fill the compute units that dH's leave (1777 tokens, 50001 x
// 2048: 1287 to 1258 us).  dW's workgroups then run one tile each, as the rest
// of dH's round is of any length; four: 1276 us.
hipError_t run_pair(XentGemm h, int splits, XentGemm w, hipStream_t stream) {
  const TileShape th = gradient_tiles(h.M, h.N, splits), tw = gradient_tiles(w.M, w.N, 1);
  if (th.rows != tw.rows) {
    const hipError_t e = run_gemm<kAcc, false, true>(h, th, splits, stream);
    return e != hipSuccess ? e : run_gemm<kOut, true, true>(w, tw, 1, stream);
  }
  // whole turns of the XCDs, so that dW's workgroups start on the first
  const int64_t nh = (lay_out(&h, th, splits, kRounds) + 7) / 8 * 8;
  const dim3 grid((unsigned)(nh + lay_out(&w, tw, 1, 1)));
  if (th.rows == 256)
    hipLaunchKernelGGL((xent_pair_kernel<256, 256, 2, 4, 2>), grid, dim3(512), 0, stream, h, w, (int)nh);
  else
    hipLaunchKernelGGL((xent_pair_kernel<64, 128, 1, 4, 3>), grid, dim3(256), 0, stream, h, w, (int)nh);
  return hipGetLastError();
}

size_t pad256(size_t n) { return (n + 255) & ~(size_t)255; }

// Vocabulary columns per piece: whole tiles, as many as keep G at 128 MB, so
// that the products after it find it in the memory-side cache (8192 tokens,
// 131072 x 4096: 26.05 ms a step; 256 MB 26.55, 64 MB 26.70, 1 GB 26.28).  But
// for many tokens 8192 columns, as dH's sums are read and written once a piece
// (32768 x 4096: 16640 tokens 14.30 ms with 8192 columns, 14.79 with 4032; 65536
// tokens 53.9 and 79.8 ms with 8192 and 1024).
constexpr int64_t kPieceBytes = (int64_t)128 << 20;
constexpr int64_t kPieceMinCols = 8192;

struct XentLayout {
  int64_t part_tiles;          // vocabulary tiles of the statistics
  int64_t tp, piece, ld_g;     // tokens in whole slabs; columns of a piece; G's row
  int splits;                  // of dH's contraction over the piece
  int z_splits;                // of the logits'; 1: their tiles take all of it
  TileShape grad_tile;         // of G's product, the same in all pieces
  int parts;                   // sums a row of G: one per tile of a piece; every piece adds to the first one's
  size_t z, part, logit, row, tokens, sums, g, acc, total;
};

XentLayout xent_layout(int64_t T, int64_t V, int64_t K, bool backward) {
  XentLayout L = {};
  size_t off = 0;
  auto take = [&](size_t bytes) { const size_t at = off; off += pad256(bytes); return at; };
  L.z_splits = logit_splits(T, V, K);
  if (L.z_splits > 1) L.z = take((size_t)L.z_splits * T * pad64(V) * 4);   // one piece: V columns
  if (!backward) {
    if (L.z_splits > 1) {
      L.total = off;
      return L;
    }
    const int cols = logit_tiles(T, V).cols;
    L.part_tiles = (V + cols - 1) / cols;
    L.part = take((size_t)L.part_tiles * T * sizeof(float2));
    L.logit = take((size_t)T * 4);
    L.total = off;
    return L;
  }
  L.tp = pad64(T);
  int64_t piece = kPieceBytes / 2 / L.tp / 256 * 256;
  if (piece < kPieceMinCols) piece = kPieceMinCols;
  if (piece > V) piece = V;
  const int64_t n = (V + piece - 1) / piece;
  if (n > 1) piece = ((V + n - 1) / n + 255) / 256 * 256;   // even pieces
  L.piece = piece;
  // Whole tiles, and an odd number of 128-byte lines a row, so that rows do not
  // all start on one memory channel.
  L.ld_g = (piece + 255) / 256 * 256 + 64;
  // dH's contraction is split until its tiles fill one round of the chip, at
  // least 8 slabs a split; large tiles if that many splits let them.  (1777 x
  // 2048 outputs over 50001 columns: 56 large tiles x 4 splits.)
  auto splits_of = [&](int64_t bm, int64_t bn) {
    const int64_t tiles = ((T + bm - 1) / bm) * ((K + bn - 1) / bn);
    int64_t s = kCus / tiles;
    if (s > piece / 512) s = piece / 512;
    return s < 1 ? (int64_t)1 : s;
  };
  for (const TileShape t : {TileShape{256, 256}, TileShape{128, 256}, TileShape{64, 128}}) {
    const int64_t n_splits = splits_of(t.rows, t.cols);
    L.splits = (int)n_splits;
    if (gradient_tiles(T, K, n_splits).rows == t.rows) break;   // as the launch will choose
  }
  L.row = take((size_t)T * sizeof(XentRow));
  L.tokens = take(sizeof(XentTokens));
  L.grad_tile = logit_tiles(L.tp, pad64(piece));
  const int sum_cols = L.z_splits > 1 ? 1024 : L.grad_tile.cols;
  L.parts = (int)((pad64(piece) + sum_cols - 1) / sum_cols);
  L.sums = take((size_t)T * L.parts * 4);
  L.g = take((size_t)L.tp * L.ld_g * 2);
  L.acc = take((size_t)L.splits * T * K * 4);
  L.total = off;
  return L;
}

hipError_t zero_columns(uint16_t* out, int64_t ld, int64_t rows, int64_t c0, int64_t c1, hipStream_t stream) {
  hipLaunchKernelGGL(zero_columns_kernel, dim3((unsigned)(rows < 65536 ? rows : 65536), (unsigned)((c1 - c0 + 2047) / 2048)),
                     dim3(256), 0, stream, out, ld, rows, c0, c1);
  return hipGetLastError();
}

}  // namespace

size_t xent_ws_bytes(int64_t T, int64_t V, int64_t K, bool backward) {
  return xent_layout(T, V, K, backward).total;
}

hipError_t launch_xent_fwd(const XentArgs& p, void* ws, hipStream_t stream) {
  const XentLayout L = xent_layout(p.T, p.V, p.K, false);
  uint8_t* const base = (uint8_t*)ws;
  XentGemm g = {};
  g.a = (const uint8_t*)p.h; g.lda = p.ld_h * 2;
  g.b = (const uint8_t*)p.w; g.ldb = p.ld_w * 2;
  g.M = g.a_rows = (int)p.T; g.N = g.b_rows = (int)p.V; g.kblocks = (int)(p.K / 64);
  g.part = (float2*)(base + L.part);
  g.target = p.target;
  g.target_logit = (float*)(base + L.logit);
  hipError_t e;
  if (L.z_splits > 1) {
    float* const z = (float*)(base + L.z);
    if ((e = run_logit_shares(g, L.z_splits, z, stream)) != hipSuccess) return e;
    hipLaunchKernelGGL(xent_few_stats_kernel, dim3((unsigned)p.T), dim3(p.V > 1024 ? 1024 : 256), 0, stream, z, L.z_splits, (int)p.T, p.V,
                       pad64(p.V), p.target, p.ignore_index, p.loss, p.lse);
    return hipGetLastError();
  }
  if ((e = run_gemm<kStats>(g, logit_tiles(g.M, g.N), 1, stream)) != hipSuccess) return e;
  hipLaunchKernelGGL(xent_join_kernel, dim3((unsigned)((p.T + 15) / 16)), dim3(1024), 0, stream, g.part,
                     (int)L.part_tiles, (int)p.T, p.V, g.target_logit, p.target, p.ignore_index,
                     p.loss, p.lse);
  return hipGetLastError();
}

hipError_t launch_xent_bwd(const XentArgs& p, void* ws, hipStream_t stream) {
  const XentLayout L = xent_layout(p.T, p.V, p.K, true);
  uint8_t* const base = (uint8_t*)ws;
  XentRow* const row = (XentRow*)(base + L.row);
  XentTokens* const tokens = (XentTokens*)(base + L.tokens);
  float* const sums = p.dh ? (float*)(base + L.sums) : nullptr;
  uint16_t* const g = (uint16_t*)(base + L.g);
  float* const acc = (float*)(base + L.acc);
  hipLaunchKernelGGL(xent_rows_kernel, dim3(1), dim3(1024), 0, stream, (int)p.T, p.V, p.target,
                     p.ignore_index, p.dloss, p.lse, p.nll, row, tokens);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  for (int64_t v0 = 0; v0 < p.V; v0 += L.piece) {
    const int64_t nv = p.V - v0 < L.piece ? p.V - v0 : L.piece;
    const uint16_t* const w = (const uint16_t*)p.w + v0 * p.ld_w;
    XentGemm z = {};
    z.a = (const uint8_t*)p.h; z.lda = p.ld_h * 2;
    z.b = (const uint8_t*)w; z.ldb = p.ld_w * 2;
    // The tokens and columns that fill the last slabs of the next products have
    // no gradient: zeros.
    z.M = (int)L.tp; z.N = (int)pad64(nv); z.kblocks = (int)(p.K / 64);
    z.a_rows = (int)p.T; z.b_rows = (int)nv;
    z.row = row; z.v0 = (int)v0;
    z.out = g; z.ldo = L.ld_g;
    z.sums = sums; z.add = v0 > 0;
    if (L.z_splits > 1) {
      float* const shares = (float*)(base + L.z);
      if ((e = run_logit_shares(z, L.z_splits, shares, stream)) != hipSuccess) return e;
      hipLaunchKernelGGL(xent_few_grad_kernel, dim3((unsigned)L.tp, (unsigned)((z.N + 1023) / 1024)), dim3(256), 0,
                         stream, shares, L.z_splits, (int)p.T, (int)nv, z.N, row, (int)v0, g, L.ld_g, sums);
      e = hipGetLastError();
    } else {
      e = run_gemm<kGrad>(z, L.grad_tile, 1, stream);
    }
    if (e != hipSuccess) return e;
    XentGemm dw = {};   // dW[v, k] = sum_t G[t, v] H[t, k]
    dw.a = (const uint8_t*)g; dw.lda = L.ld_g * 2; dw.a_rows = (int)L.tp;
    dw.b = (const uint8_t*)p.h; dw.ldb = p.ld_h * 2; dw.b_rows = (int)p.T;
    dw.M = (int)nv; dw.N = (int)p.K; dw.kblocks = (int)(L.tp / 64);
    dw.out = p.dw ? (uint16_t*)p.dw + v0 * p.ld_dw : nullptr; dw.ldo = p.ld_dw; dw.tokens = tokens; dw.row = row;
    XentGemm dh = {};   // dH[t, k] += sum_v G[t, v] W[v, k]
    dh.a = (const uint8_t*)g; dh.lda = L.ld_g * 2; dh.a_rows = (int)p.T;
    dh.b = (const uint8_t*)w; dh.ldb = p.ld_w * 2; dh.b_rows = (int)nv;
    dh.M = (int)p.T; dh.N = (int)p.K; dh.kblocks = (int)(pad64(nv) / 64);
    dh.acc = acc; dh.add = v0 > 0;
    if (p.dh && p.dw) e = run_pair(dh, L.splits, dw, stream);
    else if (p.dw) e = run_gemm<kOut, true, true>(dw, gradient_tiles(dw.M, dw.N, 1), 1, stream);
    else if (p.dh) e = run_gemm<kAcc, false, true>(dh, gradient_tiles(dh.M, dh.N, L.splits), L.splits, stream);
    if (e != hipSuccess) return e;
  }
  if (!p.dh) return hipSuccess;
  const unsigned wide = (unsigned)((p.K + 1023) / 1024);   // at most 2^10
  hipLaunchKernelGGL(xent_dh_kernel, dim3((unsigned)(p.T < (1 << 20) ? p.T : (1 << 20)), wide), dim3(256), 0, stream,
                     acc, L.splits, p.T, p.K, tokens, row, sums, L.parts, (const uint16_t*)p.w, p.ld_w,
                     (uint16_t*)p.dh, p.ld_dh);
  return hipGetLastError();
}

hipError_t launch_zero_rows_bf16(void* out, int64_t rows, int64_t cols, int64_t ld, hipStream_t stream) {
  return zero_columns((uint16_t*)out, ld, rows, 0, cols, stream);
}

}  // namespace fp8bw
