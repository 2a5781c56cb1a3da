// Tokens to experts and back for gfx950: slots sorted by expert, token rows
// gathered into the sorted order (bf16, and E4M3 codes in both layouts), and
// the experts' rows joined again with the router's weights.
//
// A slot i = t * topk + j is token t's j-th choice.  With n_e slots of expert
// e, each expert's rows are padded to a multiple of `align`:
//   end[e]   = sum_{f <= e} ceil(n_f / align) * align
//   row[i]   = end[e - 1] + #{i' < i : expert[i'] == e}     (-1 without an expert)
//   source   = the inverse of row, -1 at padding rows and behind the last end
// and, with w the router's weights,
//   gather   v[r] = w[source[r]] * x[source[r] / topk]      (0 where source < 0)
//   combine  out[t] = sum_j w[t, j] * y[row[t, j]]
//   dweight  dw[t, j] = sum_c x[t, c] * y[row[t, j], c]
// Sums are fp32 in a fixed order without atomics, so results repeat bit for
// bit.

#include "launch.h"
#include "vec8.h"

namespace fp8bw {

// ---------------------------------------------------------------------------
// Sort.  A workgroup takes a run of slots, a wave a run of its run, 64 slots at
// a time: the lanes that hold the same expert are found by one ballot per bit
// of the expert's number, so a slot's rank is its wave's count so far (LDS)
// plus the matching lanes below it, in slot order and without atomics.  Ranks
// stay in registers until the first row of every (wave, expert) is known.  Up to
// kSortOne slots take one workgroup and one launch (the latency of a decoding
// step, 5 us); more take a counting launch and a placing one, whose workgroups
// each add up the counts of those before them.  Bound by latency: 33280 slots of
// 16 experts are 0.4 MB and take 5.6 + 7.7 us, 4662 of 60 experts 9 us (15 in two
// launches), 8 of 128 experts 5.
constexpr int kSortOneWaves = 16;        // 8 for more than 512 experts (LDS)
constexpr int kSortOneRuns = 8;          // times 64 slots a wave
constexpr int kSortWaves = 4, kSortRuns = 4;
constexpr int64_t kSortOne = 64 * kSortOneWaves * kSortOneRuns;

__device__ __forceinline__ int slot_expert(const MoeSortArgs& p, int64_t i, int64_t end) {
  if (i >= end) return p.experts;
  const int64_t e = p.wide ? ((const int64_t*)p.expert)[i] : (int64_t)((const int*)p.expert)[i];
  return e >= 0 && e < p.experts ? (int)e : p.experts;
}

// Lanes with this lane's expert.
__device__ __forceinline__ uint64_t same_expert(int e, int bits) {
  uint32_t lo = ~0u, hi = ~0u;
  for (int b = 0; b < bits; ++b) {
    const uint32_t set = (uint32_t)((int)((uint32_t)e << (31 - b)) >> 31);   // the bit, in every bit
    const uint64_t has = __ballot(set != 0);
    lo &= ~((uint32_t)has ^ set);
    hi &= ~((uint32_t)(has >> 32) ^ set);
  }
  return (uint64_t)hi << 32 | lo;
}

// Counts this lane's slot of expert e among the wave's: its rank there (of no
// meaning without an expert).
__device__ __forceinline__ int count_slot(int e, int experts, int bits, volatile int* count) {
  const int lane = threadIdx.x & 63;
  const uint64_t same = same_expert(e, bits);
  int rank = 0;
  if (e < experts) {
    rank = count[e] + __popcll(same & ((1ull << lane) - 1));
    // the wave runs in step: every lane has read before the last one writes
    __builtin_amdgcn_wave_barrier();
    if ((same >> lane) == 1) count[e] = rank + 1;
  }
  return rank;
}

__device__ __forceinline__ int expert_bits(int experts) { return 32 - __clz(experts); }

// Experts and ranks of `runs` <= RUNS times 64 slots of a wave, all loads first.
template <int RUNS>
struct SlotRanks {
  int expert[RUNS], rank[RUNS];
  __device__ __forceinline__ SlotRanks(const MoeSortArgs& p, int64_t begin, int runs, int bits, int* count) {
    const int lane = threadIdx.x & 63;
#pragma unroll
    for (int k = 0; k < RUNS; ++k)
      if (k < runs) expert[k] = slot_expert(p, begin + 64 * k + lane, p.n);
#pragma unroll
    for (int k = 0; k < RUNS; ++k)
      if (k < runs) rank[k] = count_slot(expert[k], p.experts, bits, count);
  }
};

// The counts of one workgroup's run, a multiple of what its waves take at a time.
template <int WAVES, int RUNS>
__global__ __launch_bounds__(64 * WAVES) void moe_count_kernel(const MoeSortArgs p, int64_t run) {
  extern __shared__ int lds[];
  int* const count = lds;   // [WAVES][experts]
  const int tid = threadIdx.x, wave = tid >> 6;
  for (int k = tid; k < WAVES * p.experts; k += 64 * WAVES) count[k] = 0;
  __syncthreads();
  for (int64_t r = 0; r < run; r += 64 * RUNS * WAVES)
    SlotRanks<RUNS>(p, blockIdx.x * run + r + wave * 64 * RUNS, RUNS, expert_bits(p.experts), count + wave * p.experts);
  __syncthreads();
  for (int e = tid; e < p.experts; e += 64 * WAVES) {
    int n = 0;
#pragma unroll
    for (int w = 0; w < WAVES; ++w) n += count[w * p.experts + e];
    p.counts[(int64_t)blockIdx.x * p.experts + e] = n;
  }
}

// Workgroup b of `groups` places the slots [b run, (b + 1) run), 64 `runs` of each
// wave at a time.
template <int WAVES, int RUNS>
__global__ __launch_bounds__(64 * WAVES) void moe_place_kernel(const MoeSortArgs p, int64_t run, int runs, int groups) {
  constexpr int N = 64 * WAVES;
  extern __shared__ int lds[];
  int* const count = lds;                        // [WAVES][experts], then each wave's first row
  int* const next = lds + WAVES * p.experts;     // [experts] this workgroup's next row of an expert
  int* const total = next + p.experts;           // [experts] an expert's slots
  __shared__ int wave_rows[WAVES];
  const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63, E = p.experts;
  const int bits = expert_bits(E);
  // Slots of this workgroup's first part, while the counts are on their way.
  auto clear = [&]() {
    for (int k = tid; k < WAVES * E; k += N) count[k] = 0;
    __syncthreads();
  };
  clear();
  SlotRanks<RUNS> s(p, blockIdx.x * run + wave * 64 * runs, runs, bits, count + wave * E);
  // Each expert's slots in all, and those of the workgroups before this one.
  // Few experts: several threads share an expert's list of counts.
  if (groups > 1) {
    int* const before = total + E;   // [parts][experts] x 2
    int parts = 1;
    while (parts * 2 * E <= N) parts *= 2;
    for (int e0 = 0; e0 < E; e0 += N) {
      const int part = parts > 1 ? tid / E : 0, e = parts > 1 ? tid % E : e0 + tid;
      int all = 0, mine = 0;
      if (part < parts && e < E) {
#pragma unroll 8
        for (int b = part; b < groups; b += parts) {
          const int c = p.counts[(int64_t)b * E + e];
          all += c;
          mine += b < (int)blockIdx.x ? c : 0;
        }
        before[part * E + e] = mine;
        before[(parts + part) * E + e] = all;
      }
    }
    __syncthreads();
    for (int e = tid; e < E; e += N) {
      int all = 0, mine = 0;
      for (int k = 0; k < parts; ++k) {
        mine += before[k * E + e];
        all += before[(parts + k) * E + e];
      }
      total[e] = all;
      next[e] = mine;   // for now
    }
  } else {
    __syncthreads();
    for (int e = tid; e < E; e += N) {
      int all = 0;
#pragma unroll
      for (int w = 0; w < WAVES; ++w) all += count[w * E + e];
      total[e] = all;
      next[e] = 0;
    }
  }
  __syncthreads();
  // Padded lengths summed over the experts, N experts at a time.
  int base = 0;
  for (int e0 = 0; e0 < E; e0 += N) {
    const int e = e0 + tid;
    const int slots = e < E ? total[e] : 0;
    const int padded = (slots + p.align - 1) / p.align * p.align;
    int sum = padded;
#pragma unroll
    for (int d = 1; d < 64; d *= 2) {
      const int o = __shfl_up(sum, d);
      if (lane >= d) sum += o;
    }
    if (lane == 63) wave_rows[wave] = sum;
    __syncthreads();
    int all = 0;
#pragma unroll
    for (int w = 0; w < WAVES; ++w) {
      if (w < wave) sum += wave_rows[w];
      all += wave_rows[w];
    }
    if (e < E) {
      if (blockIdx.x == 0) p.group_end[e] = base + sum;
      next[e] += base + sum - padded;
      total[e] = base + sum - padded + slots;   // from here on: the expert's last row + 1
    }
    base += all;
    __syncthreads();
  }
  for (int64_t part = 0;;) {
    for (int e = tid; e < E; e += N) {
      int row = next[e];
#pragma unroll
      for (int w = 0; w < WAVES; ++w) {
        const int n = count[w * E + e];
        count[w * E + e] = row;
        row += n;
      }
      next[e] = row;
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < RUNS; ++k) {
      const int64_t i = blockIdx.x * run + part + (wave * runs + k) * 64 + lane;
      if (k >= runs || i >= p.n) continue;
      int r = -1;
      if (s.expert[k] < E) {
        r = count[wave * E + s.expert[k]] + s.rank[k];
        p.source[r] = (int)i;
      }
      p.row[i] = r;
    }
    part += (int64_t)runs * N;
    if (part >= run) break;
    __syncthreads();
    clear();
    s = SlotRanks<RUNS>(p, blockIdx.x * run + part + wave * 64 * runs, runs, bits, count + wave * E);
    __syncthreads();
  }
  // Rows without a slot: from an expert's last row to the next multiple of align
  // (its first row is one), and what lies behind the last end.
  for (int e = (int)blockIdx.x * WAVES + wave; e < E; e += groups * WAVES) {
    const int last = (total[e] + p.align - 1) / p.align * p.align;
    for (int k = total[e] + lane; k < last; k += 64) p.source[k] = -1;
  }
  for (int64_t r = base + (int64_t)blockIdx.x * N + tid; r < p.rows; r += (int64_t)groups * N) p.source[r] = -1;
}

// Workgroups and slots of each; with several, their runs are whole multiples of
// what the waves take at a time, and at most 256 read each other's counts.
static int sort_groups(int64_t n, int experts, int64_t* run) {
  if (n <= (experts > 512 ? kSortOne / 2 : kSortOne)) {
    *run = n;
    return 1;
  }
  const int64_t unit = 64 * kSortWaves * kSortRuns;
  int64_t r = (n + 255) / 256;
  r = (r + unit - 1) / unit * unit;
  *run = r;
  return (int)((n + r - 1) / r);
}

size_t moe_sort_ws_bytes(int64_t n, int experts) {
  int64_t run;
  const int groups = sort_groups(n, experts, &run);
  return groups > 1 ? (size_t)groups * (size_t)experts * sizeof(int) : 0;
}

hipError_t launch_moe_sort(const MoeSortArgs& p, hipStream_t stream) {
  int64_t run;
  const int groups = sort_groups(p.n, p.experts, &run);
  const size_t E = (size_t)p.experts;
  if (groups == 1) {
    constexpr int R = kSortOneRuns;
    const int waves = E > 512 ? kSortOneWaves / 2 : kSortOneWaves;
    const int runs = p.n > 64 * waves ? (int)((p.n + 64 * waves - 1) / (64 * waves)) : 1;
    const size_t lds = (waves + 2) * E * sizeof(int);
    if (E > 512)
      hipLaunchKernelGGL((moe_place_kernel<kSortOneWaves / 2, R>), dim3(1), dim3(64 * waves), lds, stream, p, run, runs, 1);
    else
      hipLaunchKernelGGL((moe_place_kernel<kSortOneWaves, R>), dim3(1), dim3(64 * waves), lds, stream, p, run, runs, 1);
    return hipGetLastError();
  }
  constexpr int W = kSortWaves, R = kSortRuns;
  hipLaunchKernelGGL((moe_count_kernel<W, R>), dim3(groups), dim3(64 * W), W * E * sizeof(int), stream, p, run);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  int parts = 1;
  while (parts * 2 * p.experts <= 64 * W) parts *= 2;
  hipLaunchKernelGGL((moe_place_kernel<W, R>), dim3(groups), dim3(64 * W), (W + 2 + 2 * parts) * E * sizeof(int), stream,
                     p, run, R, groups);
  return hipGetLastError();
}

// ---------------------------------------------------------------------------
// Gather, rows: a wave takes pieces of 512 columns of a token (a 16-lane DPP
// row holds one 1x128 block), reads each once, quantizes it once where the
// copies are alike, and writes it to the token's rows.  The first workgroups
// fill the rows without a slot.  Bound by HBM, and by the launch below some
// thousand pieces: 777 tokens of 2064 columns to 6 experts each, bf16 and codes
// (32 MB), 11 us; one token of 5120 to 8 experts 4 us.
__device__ __forceinline__ float slot_weight(const MoeWeight& w, int64_t i) {
  if (!w.p) return 1.f;
  return w.f32 ? ((const float*)w.p)[i] : bf16lo(((const uint16_t*)w.p)[i]);
}

__device__ __forceinline__ void store_row8(const LayoutsOut& o, int64_t row, int64_t col, const float (&v)[8]) {
  if (o.y) *(uint4*)(o.y + row * o.ld_y + col) = pack8(v);
}

// Codes of a piece; every lane of a DPP row takes part, those past the last
// column with zeros.
__device__ __forceinline__ uint2 block_codes(const float (&v)[8], float* recip) {
  const float s = scale_from_amax(row16_amax(v));
  *recip = recip_of_scale(s);
  return codes8(v, s);
}
__device__ __forceinline__ void store_codes8(const LayoutsOut& o, int64_t row, int64_t col, const uint2& code,
                                             float recip) {
  *(uint2*)(o.q + row * o.ld_q + col) = code;
  if ((threadIdx.x & 15) == 0) o.recip[row * o.rs_row + (col >> 7) * o.rs_kb] = recip;
}

// Zeros in the rows without a slot: 16 rows a workgroup.
__device__ __forceinline__ void fill_empty_rows(const MoeTable& t, const LayoutsOut& o, int64_t cols, int64_t first) {
  const int tid = threadIdx.x;
  const float none = recip_of_scale(scale_from_amax(0.f));
  for (int k = 0; k < 16; ++k) {
    const int64_t r = first + k;
    if (r >= t.rows) return;
    const int slot = t.source[r];
    if (slot >= 0 && slot < t.tokens * t.topk) continue;
    for (int64_t col = tid * 8; col < cols; col += 2048) {
      if (o.y) *(uint4*)(o.y + r * o.ld_y + col) = make_uint4(0, 0, 0, 0);
      if (o.q) store_codes8(o, r, col, make_uint2(0, 0), none);
    }
  }
}

template <int P>
__global__ __launch_bounds__(256) void moe_gather_rows_kernel(const MoeGatherArgs p, uint32_t pieces, int fill) {
  if ((int)blockIdx.x < fill) {
    fill_empty_rows(p.table, p.out, p.cols, (int64_t)blockIdx.x * 16);
    return;
  }
  const int lane = threadIdx.x & 63;
  const MoeTable& t = p.table;
  const Pieces<P> at(blockIdx.x - fill, pieces);
  uint4 u[P];
  int64_t tok[P], col[P];
  bool in[P];
#pragma unroll
  for (int k = 0; k < P; ++k) {
    tok[k] = at.row[k];
    col[k] = at.col[k] + lane * 8;
    in[k] = tok[k] < t.tokens && col[k] < p.cols;
    u[k] = load_stream(p.x + (in[k] ? tok[k] * p.ld_x + col[k] : 0));
    if (!in[k]) u[k] = make_uint4(0, 0, 0, 0);
  }
#pragma unroll
  for (int k = 0; k < P; ++k) {
    if (tok[k] >= t.tokens) return;
    float v[8];
    unpack8(u[k], v);
    uint2 code = {};
    float recip = 0.f;
    if (p.out.q && !p.weight.p) code = block_codes(v, &recip);
    for (int j = 0; j < t.topk; ++j) {
      const int64_t slot = tok[k] * t.topk + j;
      const int r = t.row[slot];
      if (r < 0 || r >= t.rows) continue;
      if (!p.weight.p) {
        if (p.out.y && in[k]) *(uint4*)(p.out.y + r * p.out.ld_y + col[k]) = u[k];
      } else {
        const float w = slot_weight(p.weight, slot);
        unpack8(u[k], v);
#pragma unroll
        for (int c = 0; c < 8; ++c) v[c] *= w;
        if (p.out.y && in[k]) store_row8(p.out, r, col[k], v);
        if (p.out.q) code = block_codes(v, &recip);
      }
      if (p.out.q && in[k]) store_codes8(p.out, r, col[k], code, recip);
    }
  }
}

// Gather with transposed codes: 128 x 128 tiles of the sorted rows, from which
// every layout is written.  A tile's corner is in scalar registers and a thread's
// offsets from it in 32 bits (the host keeps 128 leading dimensions below 2^31
// bytes).
//
// 16640 tokens of 8192 columns to 2 of 16 experts, both code layouts: 205 to 212 us
// for 867 MB, 4.1 TB/s; a token's second reading misses the L2, and the 1147 MB that
// pass it do so at 5.5.  4160 tokens to 8 of 64: 166 us for 767 MB (1168 past the L2).
// Its reads alone take 108 us and its writes 83 to 107: they add up.  What leaves that
// as it is: 30% fewer vector instructions (8 rows a thread, 256 threads, against 4
// and 512), the tiles ordered so that a token's copies are read together (40% fewer
// reads reach HBM: 219 us), several row blocks a workgroup with the next one's
// loads in flight (343 us: too few waves), tiles without bank conflicts.
__global__ __launch_bounds__(256, 4) void moe_gather_tile_kernel(const MoeGatherArgs p, int col_tiles) {
  constexpr int R = 8;
  __shared__ TileLds<1, R> L;
  __shared__ __attribute__((aligned(16))) int token[128];
  __shared__ __attribute__((aligned(16))) float factor[128];
  const int tid = threadIdx.x, lane16 = tid & 15, row0 = (tid >> 4) * R, col = lane16 * 8;
  const int64_t rb = blockIdx.x / col_tiles, cb = blockIdx.x - rb * col_tiles;
  const int rows = (int)min(p.table.rows - rb * 128, (int64_t)128);   // of the tile
  const int cols = (int)min(p.cols - cb * 128, (int64_t)128);
  const LayoutsOut& o = p.out;
  if (tid < 128) {
    const int slot = tid < rows ? p.table.source[rb * 128 + tid] : -1;
    const bool has = slot >= 0 && slot < p.table.tokens * p.table.topk;
    token[tid] = has ? slot / p.table.topk : -1;
    factor[tid] = has ? slot_weight(p.weight, slot) : 0.f;
  }
  __syncthreads();
  const uint16_t* const x = p.x + cb * 128;
  uint4 u[R];
  int tk[R];
  bool whole = col < cols;
#pragma unroll
  for (int k = 0; k < R; ++k) {
    tk[k] = token[row0 + k];
    whole = whole && tk[k] >= 0;
    u[k] = *(const uint4*)(x + (tk[k] >= 0 && col < cols ? tk[k] * p.ld_x + col : 0));
  }
  if (!__all(whole)) {   // padding or a ragged edge
#pragma unroll
    for (int k = 0; k < R; ++k)
      if (tk[k] < 0 || col >= cols) u[k] = make_uint4(0, 0, 0, 0);
  }
  // (Without weights the factor is 1; the product spares the maxima the step
  // that quiets a value of unknown origin.)
  float v[R][8];
#pragma unroll
  for (int k = 0; k < R; ++k) {
    unpack8(u[k], v[k]);
    const float w = factor[row0 + k];
#pragma unroll
    for (int c = 0; c < 8; ++c) v[k][c] *= w;
  }
  tile_column_max(L, 0, v);
  if (o.y) {
    uint16_t* const corner = o.y + rb * 128 * o.ld_y + cb * 128;
    uint32_t at = row0 * (uint32_t)o.ld_y + col;
#pragma unroll
    for (int k = 0; k < R; ++k, at += (uint32_t)o.ld_y)
      if (row0 + k < rows && col < cols) *(uint4*)(corner + at) = pack8(v[k]);
  }
  if (o.q) {
    float amax[R], scale[R];
#pragma unroll
    for (int k = 0; k < R; ++k) amax[k] = row16_amax(v[k]);
    const float recip = row16_scales(amax, scale);
    uint8_t* const corner = o.q + rb * 128 * o.ld_q + cb * 128;
    uint32_t at = row0 * (uint32_t)o.ld_q + col;
#pragma unroll
    for (int k = 0; k < R; ++k, at += (uint32_t)o.ld_q)
      if (row0 + k < rows && col < cols) *(uint2*)(corner + at) = codes8(v[k], scale[k]);
    if (lane16 < R && row0 + lane16 < rows) o.recip[(rb * 128 + row0 + lane16) * o.rs_row + cb * o.rs_kb] = recip;
  }
  __syncthreads();
  if (tid < 128) {
    const float s = tile_column_scale(L, 0, tid);
    if (tid < cols) o.recip_t[(cb * 128 + tid) * o.rst_row + rb * o.rst_kb] = recip_of_scale(s);
  }
  __syncthreads();
  tile_codes(L, 0, v);
  __syncthreads();
  store_transposed(L, 0, o.qt + cb * 128 * o.ld_qt + rb * 128, o.ld_qt, rows, cols);
}

// The router's weights' gradient: one workgroup a token, which reads its row of
// x once and the rows of its slots.  HBM: 16640 tokens of 8192 columns, two slots
// each, 121 to 130 us for 818 MB.  (Together with the copies, 128 x 128 tiles of the
// sorted rows could form the products with the rows of x that they hold, 273 MB of
// 1.7 GB less to read, for partial sums of every tile and a launch that joins them.)
__global__ __launch_bounds__(256) void moe_dweight_kernel(const MoeGatherArgs p) {
  constexpr int CH = 4;
  __shared__ float red[kMoeMaxTopk][4];
  const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63;
  const MoeTable& t = p.table;
  const int64_t tok = blockIdx.x;
  for (int64_t c0 = 0; c0 < p.cols; c0 += 2048 * CH) {
    uint4 x[CH];
#pragma unroll
    for (int k = 0; k < CH; ++k) {
      const int64_t col = c0 + k * 2048 + tid * 8;
      x[k] = make_uint4(0, 0, 0, 0);
      if (col < p.cols) x[k] = load_stream(p.x + tok * p.ld_x + col);
    }
    for (int j = 0; j < t.topk; ++j) {
      const int r = t.row[tok * t.topk + j];
      float dot = 0.f;
      if (r >= 0 && r < t.rows) {
        uint4 y[CH];
#pragma unroll
        for (int k = 0; k < CH; ++k) {
          const int64_t col = c0 + k * 2048 + tid * 8;
          y[k] = make_uint4(0, 0, 0, 0);
          if (col < p.cols) y[k] = load_stream(p.y + r * p.ld_y + col);
        }
#pragma unroll
        for (int k = 0; k < CH; ++k) {
          float a[8], b[8];
          unpack8(x[k], a);
          unpack8(y[k], b);
#pragma unroll
          for (int c = 0; c < 8; ++c) dot = __builtin_fmaf(a[c], b[c], dot);
        }
      }
      dot = wave_sum(dot);
      if (lane == 0) red[j][wave] = c0 == 0 ? dot : red[j][wave] + dot;
    }
  }
  __syncthreads();
  if (tid < t.topk) {
    const float d = (red[tid][0] + red[tid][1]) + (red[tid][2] + red[tid][3]);
    if (p.weight.f32) ((float*)p.dweight)[tok * t.topk + tid] = d;
    else ((uint16_t*)p.dweight)[tok * t.topk + tid] = (uint16_t)f32_to_bf16_rne(d);
  }
}

hipError_t launch_moe_gather(const MoeGatherArgs& p, hipStream_t stream) {
  const MoeTable& t = p.table;
  if (p.dweight && t.tokens > 0) {
    hipLaunchKernelGGL(moe_dweight_kernel, dim3((unsigned)t.tokens), dim3(256), 0, stream, p);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  if (t.rows == 0 || (!p.out.y && !p.out.q && !p.out.qt)) return hipSuccess;
  if (p.out.qt) {
    const int64_t ct = (p.cols + 127) / 128, rt = (t.rows + 127) / 128;
    hipLaunchKernelGGL(moe_gather_tile_kernel, dim3((unsigned)(ct * rt)), dim3(256), 0, stream, p, (int)ct);
    return hipGetLastError();
  }
  const int64_t pieces = (p.cols + 511) / 512, items = t.tokens * pieces, fill = (t.rows + 15) / 16;
  if (items >= 4096)
    hipLaunchKernelGGL(moe_gather_rows_kernel<4>, dim3((unsigned)(fill + (items + 15) / 16)), dim3(256), 0, stream, p,
                       (uint32_t)pieces, (int)fill);
  else
    hipLaunchKernelGGL(moe_gather_rows_kernel<1>, dim3((unsigned)(fill + (items + 3) / 4)), dim3(256), 0, stream, p,
                       (uint32_t)pieces, (int)fill);
  return hipGetLastError();
}

// ---------------------------------------------------------------------------
// Combine: a wave takes P pieces of 512 columns of tokens, and of each the
// token's rows, two slots in flight (eight with one piece, where latency counts);
// fp32 sums in the slots' order.  HBM: 16640 tokens of 8192 columns, two slots each,
// 121 us for 818 MB; one token of 5120 with eight slots 3.3 us.
template <int P>
__global__ __launch_bounds__(256) void moe_combine_kernel(const MoeCombineArgs p, uint32_t pieces) {
  const int lane = threadIdx.x & 63;
  const MoeTable& t = p.table;
  const Pieces<P> at(blockIdx.x, pieces);
  int64_t tok[P], col[P];
  bool in[P];
  float sum[P][8] = {};
#pragma unroll
  for (int k = 0; k < P; ++k) {
    tok[k] = at.row[k];
    col[k] = at.col[k] + lane * 8;
    in[k] = tok[k] < t.tokens && col[k] < p.cols;
  }
  constexpr int J = P == 1 ? 8 : 2;   // slots in flight
  for (int j0 = 0; j0 < t.topk; j0 += J) {
    uint4 u[J][P];
    float w[J][P];
#pragma unroll
    for (int j = 0; j < J; ++j) {
#pragma unroll
      for (int k = 0; k < P; ++k) {
        const int64_t slot = tok[k] * t.topk + j0 + j;
        int r = -1;
        if (j0 + j < t.topk && tok[k] < t.tokens) {
          r = t.row[slot];
          w[j][k] = slot_weight(p.weight, slot);
        }
        const bool has = r >= 0 && r < t.rows;
        u[j][k] = load_stream(p.y + (has && in[k] ? r * p.ld_y + col[k] : 0));
        if (!has) {
          u[j][k] = make_uint4(0, 0, 0, 0);
          w[j][k] = 0.f;
        }
      }
    }
#pragma unroll
    for (int j = 0; j < J; ++j) {
#pragma unroll
      for (int k = 0; k < P; ++k) {
        float v[8];
        unpack8(u[j][k], v);
#pragma unroll
        for (int c = 0; c < 8; ++c) sum[k][c] = __builtin_fmaf(w[j][k], v[c], sum[k][c]);
      }
    }
  }
#pragma unroll
  for (int k = 0; k < P; ++k)
    if (in[k]) *(uint4*)(p.out + tok[k] * p.ld_out + col[k]) = pack8(sum[k]);
}

hipError_t launch_moe_combine(const MoeCombineArgs& p, hipStream_t stream) {
  const int64_t pieces = (p.cols + 511) / 512, items = p.table.tokens * pieces;
  if (items == 0) return hipSuccess;
  if (items >= 4096)
    hipLaunchKernelGGL(moe_combine_kernel<4>, dim3((unsigned)((items + 15) / 16)), dim3(256), 0, stream, p, (uint32_t)pieces);
  else
    hipLaunchKernelGGL(moe_combine_kernel<1>, dim3((unsigned)((items + 3) / 4)), dim3(256), 0, stream, p, (uint32_t)pieces);
  return hipGetLastError();
}

}  // namespace fp8bw
