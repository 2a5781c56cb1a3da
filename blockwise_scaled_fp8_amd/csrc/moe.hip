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
// plus the matching lanes below it, in slot order and without atomics.  Up to
// kSortOne slots take one workgroup and one launch (the latency of a decoding
// step); more take a counting launch and a placing one, whose workgroups each
// add up the counts of those before them.
constexpr int64_t kSortOne = 4096;
constexpr int kSortWaves = 4, kSortOneWaves = 8;

__device__ __forceinline__ int slot_expert(const MoeSortArgs& p, int64_t i, int64_t end) {
  if (i >= end) return p.experts;
  const int64_t e = p.wide ? ((const int64_t*)p.expert)[i] : (int64_t)((const int*)p.expert)[i];
  return e >= 0 && e < p.experts ? (int)e : p.experts;
}

// Lanes with this lane's expert.
__device__ __forceinline__ uint64_t same_expert(int e, int bits) {
  uint64_t m = ~0ull;
  for (int b = 0; b < bits; ++b) {
    const bool set = (e >> b) & 1;
    const uint64_t has = __ballot(set);
    m &= set ? has : ~has;
  }
  return m;
}

// Slots of each expert among [begin, end), which this wave alone counts in
// `count`; visit(i, e, rank) for every slot with an expert.
template <class F>
__device__ __forceinline__ void rank_run(const MoeSortArgs& p, int64_t begin, int64_t end, int bits,
                                         volatile int* count, F visit) {
  const int lane = threadIdx.x & 63;
  const uint64_t below = (1ull << lane) - 1;
  for (int64_t i0 = begin; i0 < end; i0 += 64) {
    const int e = slot_expert(p, i0 + lane, end);
    const uint64_t same = same_expert(e, bits);
    if (e < p.experts) {
      const int rank = count[e] + __popcll(same & below);
      visit(i0 + lane, e, rank);
      // the wave runs in step: every lane has read before the last one writes
      __builtin_amdgcn_wave_barrier();
      if ((same >> lane) == 1) count[e] = rank + 1;
    } else {
      visit(i0 + lane, e, 0);
    }
  }
}

__device__ __forceinline__ int expert_bits(int experts) { return 32 - __clz(experts); }

template <int WAVES>
__global__ __launch_bounds__(64 * WAVES) void moe_count_kernel(const MoeSortArgs p, int64_t run) {
  extern __shared__ int lds[];
  int* const count = lds;   // [WAVES][experts]
  const int tid = threadIdx.x, wave = tid >> 6;
  const int64_t per = run / WAVES;
  for (int k = tid; k < WAVES * p.experts; k += 64 * WAVES) count[k] = 0;
  __syncthreads();
  const int64_t begin = blockIdx.x * run + wave * per;
  rank_run(p, begin, min(begin + per, p.n), expert_bits(p.experts), count + wave * p.experts,
           [](int64_t, int, int) {});
  __syncthreads();
  for (int e = tid; e < p.experts; e += 64 * WAVES) {
    int n = 0;
#pragma unroll
    for (int w = 0; w < WAVES; ++w) n += count[w * p.experts + e];
    p.counts[(int64_t)blockIdx.x * p.experts + e] = n;
  }
}

// Workgroup b of `groups` places the slots [b run, (b + 1) run).
template <int WAVES>
__global__ __launch_bounds__(64 * WAVES) void moe_place_kernel(const MoeSortArgs p, int64_t run, int groups) {
  constexpr int N = 64 * WAVES;
  extern __shared__ int lds[];
  int* const count = lds;                        // [WAVES][experts], then each wave's next row
  int* const first = lds + WAVES * p.experts;    // [experts] first row of an expert
  int* const total = first + p.experts;          // [experts] its slots
  __shared__ int wave_rows[WAVES];
  const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63, E = p.experts;
  const int bits = expert_bits(E);
  const int64_t per = run / WAVES;
  for (int k = tid; k < WAVES * E; k += N) count[k] = 0;
  __syncthreads();
  const int64_t begin = blockIdx.x * run + wave * per, end = min(begin + per, p.n);
  rank_run(p, begin, end, bits, count + wave * E, [](int64_t, int, int) {});
  __syncthreads();
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
#pragma unroll 4
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
      first[e] = mine;   // for now
    }
  } else {
    for (int e = tid; e < E; e += N) {
      int all = 0;
#pragma unroll
      for (int w = 0; w < WAVES; ++w) all += count[w * E + e];
      total[e] = all;
      first[e] = 0;
    }
  }
  __syncthreads();
  // Padded lengths summed over the experts, N experts at a time.
  int base = 0;
  for (int e0 = 0; e0 < E; e0 += N) {
    const int e = e0 + tid;
    const int padded = e < E ? (total[e] + p.align - 1) / p.align * p.align : 0;
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
      int row = base + sum - padded + first[e];   // this workgroup's first row of the expert
      first[e] = base + sum - padded;
#pragma unroll
      for (int w = 0; w < WAVES; ++w) {
        const int n = count[w * E + e];
        count[w * E + e] = row;
        row += n;
      }
    }
    base += all;
    __syncthreads();
  }
  rank_run(p, begin, end, bits, count + wave * E, [&](int64_t i, int e, int r) {
    if (e < E) {
      p.row[i] = r;
      p.source[r] = (int)i;
    } else if (i < end) {
      p.row[i] = -1;
    }
  });
  // Rows without a slot: an expert's padding (one wave an expert), then what
  // lies behind the last end.
  for (int e = (int)blockIdx.x * WAVES + wave; e < E; e += groups * WAVES) {
    const int n = total[e], padded = (n + p.align - 1) / p.align * p.align;
    for (int k = n + lane; k < padded; k += 64) p.source[first[e] + k] = -1;
  }
  for (int64_t r = base + (int64_t)blockIdx.x * N + tid; r < p.rows; r += (int64_t)groups * N) p.source[r] = -1;
}

// Workgroups and slots of each; the runs are whole multiples of what the waves
// take at a time, and at most 256 workgroups read each other's counts.
static int sort_groups(int64_t n, int64_t* run) {
  if (n <= kSortOne) {
    *run = (n + 64 * kSortOneWaves - 1) / (64 * kSortOneWaves) * (64 * kSortOneWaves);
    return 1;
  }
  const int64_t unit = 64 * kSortWaves;
  int64_t r = (n + 255) / 256;
  r = (r + unit - 1) / unit * unit;
  if (r < 4 * unit) r = 4 * unit;
  *run = r;
  return (int)((n + r - 1) / r);
}

size_t moe_sort_ws_bytes(int64_t n, int experts) {
  int64_t run;
  const int groups = sort_groups(n, &run);
  return groups > 1 ? (size_t)groups * (size_t)experts * sizeof(int) : 0;
}

hipError_t launch_moe_sort(const MoeSortArgs& p, hipStream_t stream) {
  int64_t run;
  const int groups = sort_groups(p.n, &run);
  const size_t E = (size_t)p.experts;
  if (groups == 1) {
    hipLaunchKernelGGL(moe_place_kernel<kSortOneWaves>, dim3(1), dim3(64 * kSortOneWaves),
                       (kSortOneWaves + 2) * E * sizeof(int), stream, p, run, 1);
    return hipGetLastError();
  }
  hipLaunchKernelGGL(moe_count_kernel<kSortWaves>, dim3(groups), dim3(64 * kSortWaves),
                     kSortWaves * E * sizeof(int), stream, p, run);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  int parts = 1;
  while (parts * 2 * p.experts <= 64 * kSortWaves) parts *= 2;
  hipLaunchKernelGGL(moe_place_kernel<kSortWaves>, dim3(groups), dim3(64 * kSortWaves),
                     (kSortWaves + 2 + 2 * parts) * E * sizeof(int), stream, p, run, groups);
  return hipGetLastError();
}

// ---------------------------------------------------------------------------
// Gather, rows: a wave takes pieces of 512 columns of a token (a 16-lane DPP
// row holds one 1x128 block), reads each once, quantizes it once where the
// copies are alike, and writes it to the token's rows.  The first workgroups
// fill the rows without a slot.
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
  const float s = scale_from_amax(row16_max(absmax8(v)));
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
__global__ __launch_bounds__(256) void moe_gather_rows_kernel(const MoeGatherArgs p, int64_t pieces, int fill) {
  if ((int)blockIdx.x < fill) {
    fill_empty_rows(p.table, p.out, p.cols, (int64_t)blockIdx.x * 16);
    return;
  }
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
  const MoeTable& t = p.table;
  uint4 u[P];
  int64_t tok[P], col[P];
  bool in[P];
#pragma unroll
  for (int k = 0; k < P; ++k) {
    const int64_t item = ((int64_t)blockIdx.x - fill) * 4 * P + 4 * k + wave;
    tok[k] = item / pieces;
    col[k] = (item - tok[k] * pieces) * 512 + lane * 8;
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
// every layout is written.
__global__ __launch_bounds__(512, 4) void moe_gather_tile_kernel(const MoeGatherArgs p, int col_tiles) {
  __shared__ TileLds<1> L;
  __shared__ int token[128];
  __shared__ float factor[128];
  const int tid = threadIdx.x, g = tid & 15, j = tid >> 4;
  const int64_t rb = blockIdx.x / col_tiles, cb = blockIdx.x - rb * col_tiles;
  const int64_t col = cb * 128 + g * 8;
  const bool col_in = col < p.cols;
  const LayoutsOut& o = p.out;
  if (tid < 128) {
    const int64_t r = rb * 128 + tid;
    const int slot = r < p.table.rows ? p.table.source[r] : -1;
    const int tk = slot < 0 ? -1 : slot / p.table.topk;
    token[tid] = tk < p.table.tokens ? tk : -1;
    factor[tid] = tk < 0 || tk >= p.table.tokens ? 0.f : slot_weight(p.weight, slot);
  }
  __syncthreads();
  uint4 u[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const int tk = token[4 * j + k];
    const bool in = col_in && tk >= 0;
    u[k] = *(const uint4*)(p.x + (in ? tk * p.ld_x + col : 0));
    if (!in) u[k] = make_uint4(0, 0, 0, 0);
  }
  float v[4][8];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    unpack8(u[k], v[k]);
    if (p.weight.p) {
      const float w = factor[4 * j + k];
#pragma unroll
      for (int c = 0; c < 8; ++c) v[k][c] *= w;
    }
  }
  tile_column_max(L, 0, v);
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const int64_t r = rb * 128 + 4 * j + k;
    const bool in = col_in && r < p.table.rows;
    if (o.y && in) store_row8(o, r, col, v[k]);
    if (o.q) {
      float recip;
      const uint2 code = block_codes(v[k], &recip);
      if (in) store_codes8(o, r, col, code, recip);
    }
  }
  __syncthreads();
  if (tid < 128) {
    const float s = tile_column_scale(L, 0, tid);
    if (cb * 128 + tid < p.cols) o.recip_t[(cb * 128 + tid) * o.rst_row + rb * o.rst_kb] = recip_of_scale(s);
  }
  __syncthreads();
  tile_codes(L, 0, v);
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int id = tid + 512 * i, oc = id >> 3, seg = id & 7;
    const uint4 w = tile_piece(L, 0, oc, seg);
    const int64_t orow = cb * 128 + oc, ocol = rb * 128 + 16 * seg;
    if (orow < p.cols && ocol < p.table.rows) {
      const u32x4 t = {w.x, w.y, w.z, w.w};
      __builtin_nontemporal_store(t, (u32x4*)(o.qt + orow * o.ld_qt + ocol));
    }
  }
}

// The router's weights' gradient: one workgroup a token, which reads its row of
// x once and the rows of its slots.
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
    const int64_t ct = (p.cols + 127) / 128;
    hipLaunchKernelGGL(moe_gather_tile_kernel, dim3((unsigned)(ct * ((t.rows + 127) / 128))), dim3(512), 0, stream,
                       p, (int)ct);
    return hipGetLastError();
  }
  const int64_t pieces = (p.cols + 511) / 512, items = t.tokens * pieces, fill = (t.rows + 15) / 16;
  if (items >= 4096)
    hipLaunchKernelGGL(moe_gather_rows_kernel<4>, dim3((unsigned)(fill + (items + 15) / 16)), dim3(256), 0, stream, p,
                       pieces, (int)fill);
  else
    hipLaunchKernelGGL(moe_gather_rows_kernel<1>, dim3((unsigned)(fill + (items + 3) / 4)), dim3(256), 0, stream, p,
                       pieces, (int)fill);
  return hipGetLastError();
}

// ---------------------------------------------------------------------------
// Combine: a wave takes P pieces of 512 columns of tokens, and of each the
// token's rows, two slots in flight; fp32 sums in the slots' order.
template <int P>
__global__ __launch_bounds__(256) void moe_combine_kernel(const MoeCombineArgs p, int64_t pieces) {
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
  const MoeTable& t = p.table;
  int64_t tok[P], col[P];
  bool in[P];
  float sum[P][8] = {};
#pragma unroll
  for (int k = 0; k < P; ++k) {
    const int64_t item = (int64_t)blockIdx.x * 4 * P + 4 * k + wave;
    tok[k] = item / pieces;
    col[k] = (item - tok[k] * pieces) * 512 + lane * 8;
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
    hipLaunchKernelGGL(moe_combine_kernel<4>, dim3((unsigned)((items + 15) / 16)), dim3(256), 0, stream, p, pieces);
  else
    hipLaunchKernelGGL(moe_combine_kernel<1>, dim3((unsigned)((items + 3) / 4)), dim3(256), 0, stream, p, pieces);
  return hipGetLastError();
}

}  // namespace fp8bw
