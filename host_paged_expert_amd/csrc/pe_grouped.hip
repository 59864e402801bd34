// HIP kernels of the products grouped by expert and of the 4-bit products
// (gfx950), and of what stands around them: the order of routed entries by
// expert, the weighted sum of the experts' rows and its gradients.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <type_traits>

#include "../../include/pe.h"
#include "pe_dense.h"
#include "pe_grouped.h"
#include "pe_layout.h"
#include "pe_tiles.h"

namespace pe {

// ------------------------------------------------------------------ order by expert
//
// A stable counting sort of the routed ids without scratch memory: every workgroup counts all ids by expert, those before
// its own 64 NW PER apart, and so knows where its entries go without the others.  Among its own, a wavefront's come in
// the order of its lanes (those of one expert find each other by a ballot for each bit of the id), wavefronts' in
// theirs.  8192 x 8 ids of 128 experts: 10.4 us, where the bytes would take less than one.  It is bound by the counting:
// equal ids among a wavefront's 64 add to one counter of LDS one after another, so that fewer experts take longer (8: 16.5,
// 4: 23, 1: 58), and so does a list of one expert's ids (58).  Beyond a workgroup a unit it grows as n squared: 1048576
// ids 111 us (of one expert 890), and 2^24, the most, 9.9 ms (113 ms).  (A workgroup for each expert that numbers its
// entries took 24: entries of one expert lie far apart, and each was a store of its own to lines that others write.)

// The wavefront's lanes see each other's accesses to LDS in this order: LDS works a wavefront's off one after another,
// the fences keep the compiler from moving one past here (a wave barrier by itself says nothing of memory).
__device__ __forceinline__ void wave_order() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

template <int NW, int PER>
__global__ __launch_bounds__(NW * 64) void group_rows_kernel(GroupRowsArgs a) {
  constexpr int kThreads = NW * 64, kOwn = kThreads * PER, kBatch = 8;
  __shared__ int before[kMaxExperts], rest[kMaxExperts], sums[NW];
  __shared__ uint16_t counts[NW][kMaxExperts];           // of the wavefronts' own entries, 64 PER at most
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, own = blockIdx.x * kOwn;
  for (int e = threadIdx.x; e < a.E; e += kThreads) {
    before[e] = rest[e] = 0;
#pragma unroll
    for (int w = 0; w < NW; ++w) counts[w][e] = 0;
  }
  __syncthreads();
  for (int i0 = threadIdx.x; i0 < a.n; i0 += kThreads * kBatch) {
    uint32_t id[kBatch];
#pragma unroll
    for (int j = 0; j < kBatch; ++j) id[j] = (uint32_t)a.ids[min(i0 + j * kThreads, a.n - 1)];
#pragma unroll
    for (int j = 0; j < kBatch; ++j) {
      const int i = i0 + j * kThreads;
      if (i < a.n && id[j] < (uint32_t)a.E) atomicAdd(i < own ? &before[id[j]] : &rest[id[j]], 1);   // counts: in any order
    }
  }
  // own entries: a wavefront's are 64 PER in a row.  `place` is first the place among the wavefront's of that expert
  int id[PER], place[PER];
  const int bits = 32 - __clz(a.E);
#pragma unroll
  for (int j = 0; j < PER; ++j) {
    const int i = own + wave * 64 * PER + 64 * j + lane;
    id[j] = i < a.n ? a.ids[i] : -1;
    const bool in = (uint32_t)id[j] < (uint32_t)a.E;
    uint64_t same = __ballot(in);
    for (int b = 0; b < bits; ++b) {
      const uint64_t set = __ballot(id[j] >> b & 1);
      same &= id[j] >> b & 1 ? set : ~set;
    }
    place[j] = -1;
    if (in) {
      const int rank = __popcll(same & ((1ull << lane) - 1));
      place[j] = counts[wave][id[j]] + rank;
    }
    wave_order();                                        // all lanes have read before one of an expert's adds theirs
    if (in && (same & ((1ull << lane) - 1)) == 0) counts[wave][id[j]] += (uint16_t)__popcll(same);
    wave_order();
  }
  __syncthreads();
  // offsets: a prefix sum over the experts, E / (64 NW) of them a thread
  constexpr int kEach = (kMaxExperts + kThreads - 1) / kThreads;
  int all[kEach], total = 0;
#pragma unroll
  for (int j = 0; j < kEach; ++j) {
    const int e = threadIdx.x * kEach + j;
    all[j] = e < a.E ? before[e] + rest[e] : 0;
    total += all[j];
  }
  int upto = total;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int v = __shfl_up(upto, d);
    if (lane >= d) upto += v;
  }
  if (lane == 63) sums[wave] = upto;
  __syncthreads();
  int first = upto - total;
#pragma unroll
  for (int w = 0; w < NW; ++w) first += w < wave ? sums[w] : 0;
#pragma unroll
  for (int j = 0; j < kEach; ++j) {
    const int e = threadIdx.x * kEach + j;
    if (e < a.E) {
      before[e] += first;                                // place of the workgroup's first entry of the expert
      if (blockIdx.x == 0) {
        a.offsets[e] = first;
        if (e == a.E - 1) a.offsets[a.E] = first + all[j];
      }
    }
    first += all[j];
  }
  __syncthreads();
#pragma unroll
  for (int j = 0; j < PER; ++j) {
    const int i = own + wave * 64 * PER + 64 * j + lane;
    if (place[j] >= 0) {
      int p = before[id[j]] + place[j];
#pragma unroll
      for (int w = 0; w < NW - 1; ++w) p += w < wave ? counts[w][id[j]] : 0;
      a.rows[p] = i / a.k;
      a.places[i] = p;
    } else if (i < a.n) {
      a.places[i] = -1;
    }
  }
}

template <int NW, int PER>
static void launch_group_rows_n(const GroupRowsArgs& a, hipStream_t s) {
  constexpr int kOwn = NW * 64 * PER;
  group_rows_kernel<NW, PER><<<dim3(std::max(1, (a.n + kOwn - 1) / kOwn)), NW * 64, 0, s>>>(a);
}

void launch_group_rows(const GroupRowsArgs& a, hipStream_t s) {
  // Each workgroup reads all ids, so that the work grows as n squared once they no longer run all at once (here of 128
  // experts): entries of its own one a thread (32 ids 3.5 us against 7.1, 65536 10.3 against 18.4, 262144 29 against 36) up to a
  // workgroup for each unit, eight beyond (1048576 ids 327 against 107).
  if (a.n <= 262144) launch_group_rows_n<16, 1>(a, s);
  else launch_group_rows_n<16, 8>(a, s);
}

// ------------------------------------------------------------------ sum back to tokens
//
// out[t] = sum_j w[t, j] y[places[t, j]] + residual[t], in fp32 and in the order of
// j: LPR lanes share a token's stretch of 8 LPR columns, each with 8 of them and
// four rows of y in flight.  Bound by its bytes, each once: 8192 x 8 rows of 2048,
// 336 MB, 68 us (4.9 TB/s, a large copy's rate; 56 where the caches still hold some).
template <int LPR>
__global__ __launch_bounds__(256) void combine_kernel(CombineArgs a) {
  const int64_t t = (int64_t)blockIdx.x * (256 / LPR) + threadIdx.x / LPR;
  const int c = blockIdx.y * LPR + threadIdx.x % LPR;
  if (t >= a.T || c >= a.H / 8) return;
  float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  for (int j0 = 0; j0 < a.k; j0 += 4) {
    uint4 y[4];
    float w[4];
    bool in[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int at = j0 + j < a.k ? a.places[t * a.k + j0 + j] : -1;
      in[j] = (uint32_t)at < (uint32_t)a.R;
      w[j] = in[j] ? a.w ? a.w[t * a.k + j0 + j] : 1.f : 0.f;
      y[j] = in[j] ? reinterpret_cast<const uint4*>(a.y + at * a.ldy)[c] : make_uint4(0, 0, 0, 0);
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (!in[j]) continue;
      float p[8];
      widen8(y[j], p);
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = __builtin_fmaf(w[j], p[i], v[i]);
    }
  }
  if (a.residual) {
    float r[8];
    widen8(reinterpret_cast<const uint4*>(a.residual + t * a.ldr)[c], r);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] += r[i];
  }
  reinterpret_cast<uint4*>(a.out + t * a.ldo)[c] = narrow8(v);
}

void launch_combine(const CombineArgs& a, hipStream_t s) {
  // us of 64 lanes a row against 256, over four sets of rows in turn: 8192 x 2 rows of 256 5.2 against 7.1, 8192 x 8 of 512
  // 15.5 against 18.5, 8192 x 4 of 1024 19.1 against 19.4, 8192 x 8 of 2048 88 against 68
  const int chunks = a.H / 8;
  if (chunks <= 64) combine_kernel<64><<<dim3((a.T + 3) / 4, 1), 256, 0, s>>>(a);
  else combine_kernel<256><<<dim3(a.T, (chunks + 255) / 256), 256, 0, s>>>(a);
}

// dy[places[t, j]] = w[t, j] dout[t] and dw[t, j] = sum_h dout[t, h] y[places[t, j], h]:
// a wavefront per entry, which shares no sum with another.  Bound by its bytes;
// dout comes from the caches but for a token's first entry (1023 x 4 rows of 2880:
// 53 MB in 10.3 us, 5.1 TB/s).
template <bool DY, bool DW>
__global__ __launch_bounds__(256) void combine_back_kernel(CombineBackArgs a) {
  const int lane = threadIdx.x & 63;
  const int64_t i = (int64_t)blockIdx.x * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  if (i >= (int64_t)a.T * a.k) return;
  const int at = a.places[i];
  if ((uint32_t)at >= (uint32_t)a.R) {
    if (DW && lane == 0) a.dw[i] = 0.f;
    return;
  }
  const float w = a.w ? a.w[i] : 1.f;
  const uint4* dout = reinterpret_cast<const uint4*>(a.dout + (int)(i / a.k) * a.lddo);
  const uint4* y = DW ? reinterpret_cast<const uint4*>(a.y + at * a.ldy) : nullptr;
  uint4* dy = DY ? reinterpret_cast<uint4*>(a.dy + at * a.lddy) : nullptr;
  float sum[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
  for (int c = lane; c < a.H / 8; c += 64) {
    float g[8], v[8];
    widen8(dout[c], g);
    if constexpr (DW) {
      widen8(y[c], v);
#pragma unroll
      for (int e = 0; e < 8; ++e) sum[e] = __builtin_fmaf(g[e], v[e], sum[e]);
    }
    if constexpr (DY) {
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = w * g[e];
      dy[c] = narrow8(v);
    }
  }
  if constexpr (DW) {
    const float total = group_sum<64>(((sum[0] + sum[1]) + (sum[2] + sum[3])) + ((sum[4] + sum[5]) + (sum[6] + sum[7])));
    if (lane == 0) a.dw[i] = total;
  }
}

void launch_combine_back(const CombineBackArgs& a, hipStream_t s) {
  const dim3 grid((unsigned)(((int64_t)a.T * a.k + 3) / 4));
  if (a.dy && a.dw) combine_back_kernel<true, true><<<grid, 256, 0, s>>>(a);
  else if (a.dy) combine_back_kernel<true, false><<<grid, 256, 0, s>>>(a);
  else combine_back_kernel<false, true><<<grid, 256, 0, s>>>(a);
}

// ------------------------------------------------------------------ which rows a workgroup takes
//
// Every expert's rows are cut into tiles of their own, numbered expert after
// expert.  Only the device knows the experts' rows, so the grid holds the most
// tiles there can be (R / BT + min(E, R)) and each workgroup finds its own, or
// that it has none: a lane adds up the tiles of its E / 64 experts, one prefix sum over the
// wavefront gives where they start.  Offsets are held to [0, R], so that whatever they
// are, no row outside the buffers is touched.

namespace {

struct Tile {
  int e;          // expert
  int t0, t1;     // the tile's first row, and one past the expert's last
  int col;        // tile of columns
};

// Sum of the values of all lanes up to and with this one.
__device__ __forceinline__ int prefix_sum(int v) {
  auto add = [&](auto ctrl, auto rows) {
    v += __builtin_amdgcn_update_dpp(0, v, decltype(ctrl)::value, decltype(rows)::value, 0xF, false);
  };
  using std::integral_constant;
  add(integral_constant<int, 0x111>{}, integral_constant<int, 0xF>{});    // from 1, 2, 4 and 8 lanes before, in each 16
  add(integral_constant<int, 0x112>{}, integral_constant<int, 0xF>{});
  add(integral_constant<int, 0x114>{}, integral_constant<int, 0xF>{});
  add(integral_constant<int, 0x118>{}, integral_constant<int, 0xF>{});
  add(integral_constant<int, 0x142>{}, integral_constant<int, 0xA>{});    // lane 15 to the second 16, 47 to the fourth
  add(integral_constant<int, 0x143>{}, integral_constant<int, 0xC>{});    // lane 31 to the upper half
  return v;
}

// find_tile for E / 64 (rounded up) <= PER experts a lane
template <int BT, bool XCD, int PER>
__device__ __forceinline__ bool find_expert_tile(const GroupedArgs& a, int b, int nn, Tile& t) {
  constexpr int kBand = 8;
  const int lane = threadIdx.x & 63, per = (a.E + 63) / 64;
  int o[PER + 1];
#pragma unroll
  for (int i = 0; i <= PER; ++i) o[i] = min(max(a.offsets[min(lane * per + min(i, per), a.E)], 0), a.R);
  int mine = 0;
#pragma unroll
  for (int i = 0; i < PER; ++i) mine += (max(o[i + 1] - o[i], 0) + BT - 1) / BT;
  const int upto = prefix_sum(min(mine, 1 << 24));       // more than there can be: offsets that do not ascend
  const int row_tiles = __builtin_amdgcn_readlane(upto, 63);
  if (row_tiles > a.R / BT + min(a.E, a.R)) return false;        // offsets that do not ascend
  const int total = row_tiles * nn;
  if (b >= total) return false;
  int q = b;
  if constexpr (XCD) {
    constexpr int kXcds = 8;
    const int xcd = b % kXcds;
    q = xcd * (total / kXcds) + min(xcd, total % kXcds) + b / kXcds;
  }
  const int at = XCD ? q / nn : q;                       // row tile, were the columns the faster index
  const int owner = __popcll(__ballot(upto <= at));
  int before = __builtin_amdgcn_readlane(upto - mine, owner), e = owner * per, lo = 0, hi = 0, tiles = 0;
  bool found = false;
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    if (!found) {
      lo = __builtin_amdgcn_readlane(o[i], owner);
      hi = __builtin_amdgcn_readlane(o[i + 1], owner);
      tiles = (max(hi - lo, 0) + BT - 1) / BT;
      found = at < before + tiles;
      if (!found) {
        before += tiles;
        ++e;
      }
    }
  }
  if constexpr (XCD) {
    const int r = q - before * nn;                       // among the expert's own
    const int band = r / (kBand * nn), rows = min(kBand, tiles - band * kBand), in = r - band * kBand * nn;
    t = Tile{e, lo + (band * kBand + in % rows) * BT, hi, in / rows};
  } else {
    t = Tile{e, lo + (at - before) * BT, hi, 0};
  }
  return true;
}

// The tile of block `b` among nn tiles of columns; false if there is none.  XCD: neighbouring tiles go to one XCD, an
// expert's in bands of 8 tiles of rows, column by column (as tile_of does for one matrix).  Otherwise nn is 1.
template <int BT, bool XCD>
__device__ __forceinline__ bool find_tile(const GroupedArgs& a, int b, int nn, Tile& t) {
  if (!a.offsets) {
    const int nt = (a.R + BT - 1) / BT;
    int tt = b, tn = 0;
    if constexpr (XCD) tile_of(b, nt, nn, tt, tn);
    t = Tile{0, tt * BT, a.R, tn};
    return true;
  }
  if (a.E <= 128) return find_expert_tile<BT, XCD, 2>(a, b, nn, t);
  return find_expert_tile<BT, XCD, kMaxExperts / 64>(a, b, nn, t);
}

// The row of x that row p of the output takes.
__device__ __forceinline__ int64_t x_row(const GroupedArgs& a, int p) {
  return a.rows ? (int64_t)min((uint32_t)a.rows[p], (uint32_t)(a.x_rows - 1)) : p;
}

// The K-major operand whose rows lie anywhere: Operand with an address for each lane.
template <int ROWS, int NW>
struct RowOperand {
  static constexpr int kInstr = ROWS / 8, kPer = (kInstr + NW - 1) / NW, kMin = kInstr / NW;
  static_assert(kInstr % NW == 0 || kPer == 1, "copies divide evenly, or go one each to the first");
  const char* at[kPer];
  int kc[kPer];

  // `row(r)`: address of tile row r
  template <class RowOf>
  __device__ __forceinline__ void init(int wave, int lane, RowOf row) {
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int r = 8 * (wave + i * NW) + (lane >> 3);
      kc[i] = ((lane & 7) ^ ((r >> 1) & 7)) * 16;
      at[i] = kMin == kPer || wave < kInstr ? row(r) + kc[i] : nullptr;
    }
  }
  // This wavefront's copies of a step where only the first `rows` rows exist.
  static __device__ __forceinline__ int copies(int wave, int rows) {
    return min(max((rows + 7) / 8 - wave + NW - 1, 0) / NW, kPer);
  }
  // Copy the 128 bytes at byte `from` of each row, of which the first `valid` exist, in this many copies.
  __device__ __forceinline__ void copy(uint32_t lds, int wave, int64_t from, int valid, int n) const {
    if (valid == 128) {
#pragma unroll
      for (int i = 0; i < kPer; ++i)
        if (i < n) copy_to_lds(lds + (wave + i * NW) * 1024, at[i] + from);
    } else {
#pragma unroll
      for (int i = 0; i < kPer; ++i)
        if (i < n)
          copy_to_lds(lds + (wave + i * NW) * 1024, kc[i] < valid ? at[i] + from : reinterpret_cast<const char*>(g_zeros));
    }
  }
};

// wait_stage where each of STEPS steps may be on its way, with A + B copies of this wavefront's each: A of x, at most PER.
template <int STEPS, int PER, int B>
__device__ __forceinline__ void wait_steps(int a) {
  static_assert(PER <= 4, "cases");
  if (PER >= 4 && a == 4) wait_stage<STEPS * (4 + B)>();
  else if (PER >= 3 && a == 3) wait_stage<STEPS * (3 + B)>();
  else if (PER >= 2 && a == 2) wait_stage<STEPS * (2 + B)>();
  else if (a == 1) wait_stage<STEPS * (1 + B)>();
  else wait_stage<STEPS * B>();
}

// The accumulators of a tile go through LDS as fp32 rows (padded by 16 bytes), so that each thread finishes 8 consecutive
// columns with 16-byte loads and stores.
template <DenseOp OP, int WT, int WN, int FT, int FN>
__device__ __forceinline__ void finish_tile(const DenseArgs& a, char* lds, int t0, int n0, const f32x4_t (&acc)[FT][FN]) {
  constexpr int BT = WT * FT * 16, BN = WN * FN * 16, NO = OP == DENSE_GLU ? BN / 2 : BN, LR = BN + 4, kChunks = NO / 8;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, wt = wave / WN, wn = wave % WN;
  float* tile = reinterpret_cast<float*>(lds);
  wait_stage<0>();                                       // the stages have been read
#pragma unroll
  for (int i = 0; i < FT; ++i)
#pragma unroll
    for (int j = 0; j < FN; ++j)
      *reinterpret_cast<f32x4_t*>(tile + ((wt * FT + i) * 16 + (lane & 15)) * LR + (wn * FN + j) * 16 + (lane >> 4) * 4) =
          acc[i][j];
  __syncthreads();
#pragma unroll 1
  for (int idx = threadIdx.x; idx < BT * kChunks; idx += WT * WN * 64) {
    const int r = idx / kChunks, c = (idx % kChunks) * 8;
    finish_chunk<OP>(a, t0 + r, n0 + c, tile + r * LR, c);
  }
}

// The arguments of one expert's product.
__device__ __forceinline__ DenseArgs expert_args(const GroupedArgs& g, int e, int t1, int64_t w_bytes) {
  DenseArgs a = g.d;
  a.b = static_cast<const char*>(a.b) + e * w_bytes;
  if (a.bias) a.bias += (int64_t)e * a.N;
  a.T = t1;
  return a;
}

}  // namespace

// ------------------------------------------------------------------ bf16 products of an expert's rows
//
// The tile of pe_dense.hip over an expert's rows: rows of x are fetched through the row list by the copies into LDS
// themselves, weights K-major (forward) or k-slow (gradients).  An expert's last tile is partly empty: rows that do not
// exist are not copied, by eights, nor multiplied, by sixteens.  128 experts of 128 rows, uneven as a router leaves them, are
// bound by the weights' bytes and by the operands' way from L2 into LDS, which is twice as many: GLU 768 x 2048, 805 MB
// of weights, 222 us (4.0 TB/s with all it reads and writes); dh of the gradients 155, dx 230.  512 rows of 32 experts,
// 2880 x 2880: 686 us, 0.79 PFLOP/s.  (A 256 x 192 tile of two groups of wavefronts in turn, the dense products' best,
// is no faster here: 268 and 699 us.)
template <DenseOp OP, bool BK, int WT, int WN, int FT, int FN, int NST>
__global__ __launch_bounds__(WT * WN * 64) void grouped_tile_kernel(GroupedArgs g) {
  constexpr int NW = WT * WN, BT = WT * FT * 16, BN = WN * FN * 16;
  constexpr int NO = OP == DENSE_GLU ? BN / 2 : BN;
  constexpr int kA = BT * 128, kB = BN * 128, kStage = kA + kB;
  extern __shared__ __align__(16) char lds[];
  Tile tile;
  if (!find_tile<BT, true>(g, blockIdx.x, (g.d.N + NO - 1) / NO, tile)) return;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wt = wave / WN, wn = wave % WN;
  const DenseArgs a = expert_args(g, tile.e, tile.t1, (int64_t)(OP == DENSE_GLU ? 2 : 1) * g.d.N * g.d.K * 2);
  const int t0 = tile.t0, n0 = tile.col * NO;
  const int64_t ldb = a.ldb * 2;
  RowOperand<BT, NW> oa;
  Operand<BN, NW, BK> ob;
  oa.init(wave, lane, [&](int r) { return static_cast<const char*>(a.a) + x_row(g, min(t0 + r, a.T - 1)) * a.lda * 2; });
  ob.init(wave, lane, ldb, [&](int r) {
    if constexpr (OP == DENSE_GLU) return (int64_t)min((r >> 5) * 16 + (r & 15), a.N - 1 - n0);
    return (int64_t)min(r, a.N - 1 - n0);
  }, n0, a.N);
  const char* pb = static_cast<const char*>(a.b) + (BK ? n0 * ldb : 0);
  static_assert(OP != DENSE_GLU || NW % 4 == 0, "a wavefront's copies stay in one half");
  if (OP == DENSE_GLU && (wave & 2)) pb += (int64_t)a.N * ldb;
  pb = uniform(pb);
  Frags<BT, true, FT> fa;
  Frags<BN, BK, FN> fb;
  fa.init(wt * FT * 16, lane);
  fb.init(wn * FN * 16, lane);
  const int nk = (a.K + 63) / 64, tail = a.K - (nk - 1) * 64;
  const int64_t sb = BK ? 128 : 64 * ldb;
  const uint32_t lds0 = lds_addr(lds);
  const int exist = min(BT, a.T - t0), n_a = decltype(oa)::copies(wave, exist);        // rows of the tile that are there
  auto fetch = [&](int k) {
    const uint32_t st = lds0 + k % NST * kStage;
    const bool whole = k < nk - 1 || tail == 64;
    oa.copy(st, wave, (int64_t)k * 128, whole ? 128 : tail * 2, n_a);
    if (whole) ob.copy(st + kA, wave, pb + k * sb);
    else ob.copy_tail(st + kA, wave, pb + k * sb, BK ? tail * 2 : tail);
  };
  f32x4_t acc[FT][FN];
#pragma unroll
  for (int i = 0; i < FT; ++i)
#pragma unroll
    for (int j = 0; j < FN; ++j) acc[i][j] = f32x4_t{0.f, 0.f, 0.f, 0.f};
  const int blocks = __builtin_amdgcn_readfirstlane((exist + 15) / 16 - wt * FT);   // this wavefront's that exist
  auto multiply = [&](const char* st, int upto) {
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      bf16x8_t af[FT], bf[FN];
#pragma unroll
      for (int j = 0; j < FN; ++j) bf[j] = fb.bf16(st + kA, j, s);
#pragma unroll
      for (int i = 0; i < FT; ++i)
        if (i < upto) af[i] = fa.bf16(st, i, s);
#pragma unroll
      for (int i = 0; i < FT; ++i)
        if (i < upto) {
#pragma unroll
          for (int j = 0; j < FN; ++j)
            acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(bf[j], af[i], acc[i][j], 0, 0, 0);
        }
    }
  };
#pragma unroll
  for (int k = 0; k < NST - 1; ++k)
    if (k < nk) fetch(k);
  for (int k = 0; k < nk; ++k) {
    if (NST > 2 && k + NST - 1 <= nk) wait_steps<NST - 2, decltype(oa)::kPer, decltype(ob)::kMin>(n_a);
    else wait_stage<0>();
    const char* st = lds + k % NST * kStage;
    if (k + NST - 1 < nk) fetch(k + NST - 1);
    if (blocks >= FT) multiply(st, FT);
    else if (blocks > 0) multiply(st, blocks);
  }
  finish_tile<OP, WT, WN, FT, FN>(a, lds, t0, n0, acc);
}

// ------------------------------------------------------------------ weight gradients
//
// out[e][m, n] = sum over expert e's rows r of left[r, m] right[r, n]: both operands are k-slow, k being the expert's
// rows, and an expert without rows gets zeros.  Rows of x come through the row list: its part for the next 32 steps lies
// in LDS, where the copies of a step find their rows' addresses.  With some hundred rows to an expert its gradient is
// hardly more than its bytes written: 128 experts of 128 rows, 1536 x 2048, 805 MB in 280 us, one call after another (305
// to 310 behind the products of a backward pass).  Epilogues alone take 133 (6 TB/s), the sums 173: they hardly overlap.
// (Workgroups that went through all tiles of some columns with copies running ahead, with or without wavefronts of their
// own for the stores: 420 to 540.)
template <bool GATHER, int WT, int WN, int FT, int FN, int NST>
__global__ __launch_bounds__(WT * WN * 64) void grouped_weights_kernel(GroupedArgs g) {
  constexpr int NW = WT * WN, BT = WT * FT * 16, BN = WN * FN * 16, kList = 32;
  constexpr int kA = BT * 128, kB = BN * 128, kStage = kA + kB;
  extern __shared__ __align__(16) char lds[];
  int* list = reinterpret_cast<int*>(lds + NST * kStage);
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wt = wave / WN, wn = wave % WN;
  const int nt = (g.d.T + BT - 1) / BT, nn = (g.d.N + BN - 1) / BN;
  // Each XCD takes an eighth of every expert's tiles, column by column: an expert's whole on one XCD would leave
  // the XCDs as uneven as the experts.
  const int share = (nt * nn + 7) / 8, turn = blockIdx.x / 8;
  const int e = turn / share, in = blockIdx.x % 8 * share + turn % share;
  if (in >= nt * nn) return;
  const int t0 = in % nt * BT, n0 = in / nt * BN;
  const int r0 = min(max(g.offsets[e], 0), g.R), r1 = min(max(g.offsets[e + 1], 0), g.R);
  DenseArgs a = g.d;
  a.y = static_cast<uint16_t*>(a.y) + (int64_t)e * a.T * a.N;
  const int64_t lda = a.lda * 2, ldb = a.ldb * 2;
  const int rows = max(r1 - r0, 0), nk = (rows + 63) / 64, tail = rows - (nk - 1) * 64;
  Operand<BT, NW, false> oa;
  Operand<BN, NW, false> ob;
  auto none = [](int) { return (int64_t)0; };
  oa.init(wave, lane, lda, none, t0, a.T);
  ob.init(wave, lane, GATHER ? 0 : ldb, none, n0, a.N);
  const char* pa = uniform(static_cast<const char*>(a.a) + r0 * lda);
  const char* pb = uniform(static_cast<const char*>(a.b) + (GATHER ? 0 : r0 * ldb));
  Frags<BT, false, FT> fa;
  Frags<BN, false, FN> fb;
  fa.init(wt * FT * 16, lane);
  fb.init(wn * FN * 16, lane);
  const uint32_t lds0 = lds_addr(lds);
  // rows of the steps from k on
  auto fill = [&](int k) {
    const int left = min(rows - k * 64, kList * 64);
    for (int i = threadIdx.x; i < left; i += NW * 64) list[i] = (int)x_row(g, r0 + k * 64 + i);
  };
  auto fetch = [&](int k) {
    const uint32_t st = lds0 + k % NST * kStage;
    const int valid = k < nk - 1 ? 64 : tail;
    if (valid == 64) oa.copy(st, wave, pa + k * 64 * lda);
    else oa.copy_tail(st, wave, pa + k * 64 * lda, valid);
    if constexpr (GATHER) {
#pragma unroll
      for (int i = 0; i < decltype(ob)::kPer; ++i) {
        if (decltype(ob)::kMin != decltype(ob)::kPer && wave >= decltype(ob)::kInstr) break;
        const char* p = reinterpret_cast<const char*>(g_zeros);
        if (ob.kc[i] < valid) p = pb + list[k % kList * 64 + ob.kc[i]] * ldb + ob.off[i];
        copy_to_lds(st + kA + (wave + i * NW) * 1024, p);
      }
    } else {
      if (valid == 64) ob.copy(st + kA, wave, pb + k * 64 * ldb);
      else ob.copy_tail(st + kA, wave, pb + k * 64 * ldb, valid);
    }
  };
  constexpr int kCopies = decltype(oa)::kMin + decltype(ob)::kMin;
  f32x4_t acc[FT][FN];
#pragma unroll
  for (int i = 0; i < FT; ++i)
#pragma unroll
    for (int j = 0; j < FN; ++j) acc[i][j] = f32x4_t{0.f, 0.f, 0.f, 0.f};
  if constexpr (GATHER) {
    fill(0);
    __syncthreads();
  }
  static_assert(NST - 1 < kList, "the first steps' rows are in the first list");
#pragma unroll
  for (int k = 0; k < NST - 1; ++k)
    if (k < nk) fetch(k);
  for (int k = 0; k < nk; ++k) {
    if (NST > 2 && k + NST - 1 <= nk) wait_stage<(NST - 2) * kCopies>();
    else wait_stage<0>();
    const char* st = lds + k % NST * kStage;
    const int next = k + NST - 1;
    if (next < nk) {
      if (GATHER && next % kList == 0) {                 // every wavefront has read its rows of the step before
        fill(next);
        __syncthreads();
      }
      fetch(next);
    }
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      bf16x8_t af[FT], bf[FN];
#pragma unroll
      for (int j = 0; j < FN; ++j) bf[j] = fb.bf16(st + kA, j, s);
#pragma unroll
      for (int i = 0; i < FT; ++i) af[i] = fa.bf16(st, i, s);
#pragma unroll
      for (int i = 0; i < FT; ++i)
#pragma unroll
        for (int j = 0; j < FN; ++j)
          acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(bf[j], af[i], acc[i][j], 0, 0, 0);
    }
  }
  // As finish_tile; the gradients are stored past the caches, which the rows of the tiles after them would lose otherwise
  // (dw13 of 128 experts of 128 rows, 1536 x 2048: 340 us through them, 280 past them; dw2 169 and 155).
  constexpr int LR = BN + 4, kChunks = BN / 8;
  float* tile = reinterpret_cast<float*>(lds);
  wait_stage<0>();
#pragma unroll
  for (int i = 0; i < FT; ++i)
#pragma unroll
    for (int j = 0; j < FN; ++j)
      *reinterpret_cast<f32x4_t*>(tile + ((wt * FT + i) * 16 + (lane & 15)) * LR + (wn * FN + j) * 16 + (lane >> 4) * 4) =
          acc[i][j];
  __syncthreads();
#pragma unroll 1
  for (int idx = threadIdx.x; idx < BT * kChunks; idx += NW * 64) {
    const int m = idx / kChunks, c = (idx % kChunks) * 8;
    if (t0 + m >= a.T || n0 + c >= a.N) continue;        // (N is a multiple of 8)
    const float4 lo = *reinterpret_cast<const float4*>(tile + m * LR + c), hi = *reinterpret_cast<const float4*>(tile + m * LR + c + 4);
    const float v[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
    typedef __attribute__((ext_vector_type(4))) uint32_t u32x4_t;
    __builtin_nontemporal_store(__builtin_bit_cast(u32x4_t, narrow8(v)),
                                reinterpret_cast<u32x4_t*>(static_cast<uint16_t*>(a.y) + (int64_t)(t0 + m) * a.N + n0 + c));
  }
}

// ------------------------------------------------------------------ 4-bit weights
//
// The products sum_k x[k] w[k] take the codes' values as bf16, exactly, and a scale as far out as it is constant:
//   MXFP4: an E2M1 value times its block's power of two is exact in bf16 (but for products beyond bf16's range, which
//          are infinite, or below it), so v_cvt_scalef32_pk_bf16_fp4 makes operands that need nothing more.
//   int4:  the fp16 scale of 128 k multiplies the fp32 sum over them.  q ^ 8 as a signed 4-bit number is q - 8, and
//          v_cvt_off_f32_i4 makes (q - 8) / 16 of it, of which the upper half is the bf16 number; the scale is taken
//          times 16.  Every term is so x (q - 8) s and no other: a code of 8 adds nothing to a finite x, an infinity of
//          x gives what its products with the weights give, and sums of 128 k pass fp32's range only where sum
//          |x (q - 8)| / 16 does.

namespace {

template <int WTYPE> constexpr bool kInt4 = WTYPE == PE_W_INT4_G128;
template <int WTYPE> constexpr bool kMx = WTYPE == PE_W_MXFP4_B32;
template <int WTYPE> constexpr int kScaleGroup = kInt4<WTYPE> ? 128 : 32;

// Eight codes (the first in the lowest nibble) as bf16: int4 (q - 8) / 16, MXFP4 the value times `scale`.
template <int WTYPE>
__device__ __forceinline__ bf16x8_t decode8(uint32_t d, float scale) {
  typedef __attribute__((ext_vector_type(2))) __bf16 bf16x2_t;
  if constexpr (kMx<WTYPE>) {
    const bf16x2_t p0 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(d, scale, 0);
    const bf16x2_t p1 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(d, scale, 1);
    const bf16x2_t p2 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(d, scale, 2);
    const bf16x2_t p3 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(d, scale, 3);
    return bf16x8_t{p0[0], p0[1], p1[0], p1[1], p2[0], p2[1], p3[0], p3[1]};
  } else {
    const uint32_t low = d ^ 0x88888888u;
    uint32_t high = low >> 4;
    asm("" : "+v"(high));                                // one shift: the compiler would make one for each code
    uint32_t p[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t a = __float_as_uint(__builtin_amdgcn_cvt_off_f32_i4((int)__builtin_amdgcn_ubfe(low, 8 * i, 8)));
      const uint32_t b = __float_as_uint(__builtin_amdgcn_cvt_off_f32_i4((int)__builtin_amdgcn_ubfe(high, 8 * i, 8)));
      p[i] = __builtin_amdgcn_perm(b, a, 0x07060302u);   // both numbers have zeros in their lower halves
    }
    return __builtin_bit_cast(bf16x8_t, make_uint4(p[0], p[1], p[2], p[3]));
  }
}

// An E8M0 byte as the fp32 number 2^(e - 127); 255 is NaN.
__device__ __forceinline__ float e8m0(uint32_t e) {
  return __uint_as_float(e == 0 ? 0x00400000u : e == 255 ? 0x7FC00000u : e << 23);
}

// What int4 sums are multiplied by: 16 times the fp16 scale.
__device__ __forceinline__ float int4_scale(uint16_t h) { return 16.f * (float)__builtin_bit_cast(_Float16, h); }

}  // namespace

// ------------------------------------------------------------------ products of few rows
//
// A few rows for each matrix (a decode step): the weights' bytes bound the product, so they stream straight from memory
// into MFMA operands.  A wavefront takes F fragments of 16 / P weight rows (of a GLU gate rows and their up rows)
// and 16 / P rows of x, every KW-th step of k with U steps in flight; CW wavefronts take neighbouring columns, KW share
// their sums, which meet in LDS in a fixed order.  A step is 128 bytes of k in bf16 and 64 bytes, 128 k, in 4 bits.  P
// parts of k share the MFMA's 16 x 16 block as in the dense kernel of few rows.  x is the first operand, so that a lane's
// accumulators belong to one weight row and its scale.
// One row of int4 2048 x 6144, 6.4 MB: 5.3 us, of which a launch that does nothing is some 2.5.  Four rows to 30 of 128
// experts, int4 GLU 768 x 2048, 45 MB: 16 us (2.8 TB/s), bf16 177 MB: 37 us (4.8 TB/s).  A workgroup waits for memory once
// for its tile, and then for every KW P U steps: 4 rows of MXFP4 GLU 2880 x 2880 (23 steps, 16 a turn) take 7.4 us for
// 8.9 MB.
template <DenseOp OP, int WTYPE, int F, int CW, int KW, int P, int U>
__global__ __launch_bounds__(CW * KW * 64) void grouped_few_kernel(GroupedArgs g) {
  static_assert(OP != DENSE_GLU || F == 2, "a gate and an up fragment");
  constexpr int NR = 16 / P, FO = OP == DENSE_GLU ? 1 : F, NO = CW * FO * NR;
  constexpr int WM = OP == DENSE_GLU ? 2 : 1;            // matrices of N rows
  constexpr bool Q = WTYPE != PE_W_BF16;
  constexpr int kStep = Q ? 128 : 64, kX = Q ? 4 : 2, kW = Q ? 1 : 2;
  __shared__ f32x4_t red[CW][F][KW][64];
  Tile tile;
  if (!find_tile<NR, false>(g, blockIdx.y, 1, tile)) return;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int cw = wave / KW, kw = wave % KW;
  const int q = lane >> 4, ln = lane & 15, part = ln / NR, lr = ln % NR;
  const int K = g.d.K, N = g.d.N, t0 = tile.t0;
  const int64_t row_bytes = Q ? K / 2 : (int64_t)K * 2;
  const DenseArgs a = expert_args(g, tile.e, tile.t1, WM * N * row_bytes);
  const int64_t row = x_row(g, min(t0 + lr, a.T - 1));
  const int n0 = blockIdx.x * NO, nk = (K + kStep - 1) / kStep;
  // each fragment's first weight row, and this lane's from there: at most 16 rows of 2^23 bytes
  const char* pw[F];
  const char* ps[F];
  uint32_t ow[F], os[F];
#pragma unroll
  for (int f = 0; f < F; ++f) {
    const int first = min(n0 + (OP == DENSE_GLU ? cw : cw * F + f) * NR, N - 1), mine = min(lr, N - 1 - first);
    const int64_t at = first + (OP == DENSE_GLU && f ? (int64_t)N : 0);
    const uint32_t scales = K / kScaleGroup<WTYPE> * (kInt4<WTYPE> ? 2 : 1);     // bytes of a row's
    pw[f] = static_cast<const char*>(a.b) + at * row_bytes;
    ps[f] = static_cast<const char*>(g.ws) + ((int64_t)tile.e * WM * N + at) * scales;
    ow[f] = mine * (uint32_t)row_bytes;
    os[f] = mine * scales;
  }
  f32x4_t acc[F];
#pragma unroll
  for (int f = 0; f < F; ++f) acc[f] = f32x4_t{0.f, 0.f, 0.f, 0.f};
  // U steps from k0 on.  Where not all of them are `whole`, loads beyond the end take the row's last bytes instead and
  // their operands are set to zero: loads under conditions would be issued one after another.
  auto steps = [&](int k0, auto whole_t) {
    constexpr bool whole = decltype(whole_t)::value;
    const uint4 zero = make_uint4(0, 0, 0, 0);
    uint4 w[U][F][kW], x[U][kX];
    uint32_t s[U][F];
    const char* px = static_cast<const char*>(a.a) + row * a.lda * 2;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int k = k0 + u * KW * P + part;
      const int blk = whole ? 4 * k + q : min(4 * k + q, K / 32 - 1);         // 4 bits: this lane's 32 k
#pragma unroll
      for (int f = 0; f < F; ++f) {
        if constexpr (Q) {
          w[u][f][0] = *reinterpret_cast<const uint4*>(pw[f] + (ow[f] + blk * 16u));
          if constexpr (kInt4<WTYPE>) s[u][f] = *reinterpret_cast<const uint16_t*>(ps[f] + (os[f] + (blk / 4) * 2u));
          else s[u][f] = *reinterpret_cast<const uint8_t*>(ps[f] + (os[f] + blk));
        } else {
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            const int at = k * 64 + 32 * c + 8 * q;
            w[u][f][c] = *reinterpret_cast<const uint4*>(pw[f] + (ow[f] + (whole ? at : min(at, K - 8)) * 2u));
          }
        }
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int k = k0 + u * KW * P + part;
#pragma unroll
      for (int c = 0; c < kX; ++c) {
        if constexpr (Q) {
          const int blk = whole ? 4 * k + q : min(4 * k + q, K / 32 - 1);
          x[u][c] = *reinterpret_cast<const uint4*>(px + (int64_t)blk * 64 + 16 * c);
        } else {
          const int at = k * 64 + 32 * c + 8 * q;
          x[u][c] = *reinterpret_cast<const uint4*>(px + (int64_t)(whole ? at : min(at, K - 8)) * 2);
        }
      }
    }
    if constexpr (!whole) {
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int c = 0; c < kX; ++c) {
          const int k = k0 + u * KW * P + part;
          if ((Q ? 128 * k + 32 * q : k * 64 + 32 * c + 8 * q) < K) continue;
          x[u][c] = zero;
#pragma unroll
          for (int f = 0; f < F; ++f) {
            w[u][f][Q ? 0 : c] = zero;
            s[u][f] = kMx<WTYPE> ? 127 : 0;
          }
        }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
#pragma unroll
      for (int f = 0; f < F; ++f) {
        f32x4_t p = kInt4<WTYPE> ? f32x4_t{0.f, 0.f, 0.f, 0.f} : acc[f];
        const float scale = kMx<WTYPE> ? e8m0(s[u][f]) : 0.f;
#pragma unroll
        for (int c = 0; c < kX; ++c) {
          bf16x8_t v;
          if constexpr (Q) {
            const uint32_t d[4] = {w[u][f][0].x, w[u][f][0].y, w[u][f][0].z, w[u][f][0].w};
            v = decode8<WTYPE>(d[c], scale);
          } else {
            v = __builtin_bit_cast(bf16x8_t, w[u][f][c]);
          }
          p = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, x[u][c]), v, p, 0, 0, 0);
        }
        if constexpr (kInt4<WTYPE>) {
          const float by = int4_scale((uint16_t)s[u][f]);
#pragma unroll
          for (int i = 0; i < 4; ++i) acc[f][i] = __builtin_fmaf(p[i], by, acc[f][i]);
        } else {
          acc[f] = p;
        }
      }
    }
  };
  const int full = K / kStep;                            // steps of which everything exists
  int k0 = kw * P;
  for (; k0 + (U - 1) * KW * P + P <= full; k0 += KW * P * U) steps(k0, std::true_type{});
  for (; k0 < nk; k0 += KW * P * U) steps(k0, std::false_type{});
#pragma unroll
  for (int f = 0; f < F; ++f) red[cw][f][kw][lane] = acc[f];
  __syncthreads();

  // Four consecutive columns of one row at a time: their P parts of the KW sums.
  constexpr int kChunks = NO / 4;
  for (int idx = threadIdx.x; idx < NR * kChunks; idx += CW * KW * 64) {
    const int tr = idx / kChunks, c4 = idx % kChunks * 4;
    const int t = t0 + tr, n = n0 + c4;
    if (t >= a.T || n >= N) continue;
    auto sum = [&](int group, int f, int c, float (&v)[4]) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        v[i] = 0.f;
#pragma unroll
        for (int p = 0; p < P; ++p)
#pragma unroll
          for (int w = 0; w < KW; ++w) {
            const int r = p * NR + tr;
            v[i] += reinterpret_cast<const float*>(&red[group][f][w][r / 4 * 16 + p * NR + c + i])[r % 4];
          }
      }
    };
    float v[4];
    if constexpr (OP == DENSE_GLU) {
      float u[4];
      sum(c4 / NR, 0, c4 % NR, v);
      sum(c4 / NR, 1, c4 % NR, u);
      finish_glu(a, t, n, true, v, u);
    } else {
      sum(c4 / (F * NR), c4 / NR % F, c4 % NR, v);
      finish_linear(a, t, n, v);
    }
  }
}

// ------------------------------------------------------------------ 4-bit products of many rows
//
// The tile kernel with codes for weights: steps of 128 k in two halves, x's 128 bytes a row and half and the codes' 32
// copied straight into LDS, the codes decoded by the wavefront that multiplies them.  A row's two 16-byte parts of a half
// are exchanged in every other eight rows, so that the 16 rows of one read fall on all banks.  The scales of 1024 k lie
// in LDS as well (as fp32, int4's by group, MXFP4's by row); those of the next 1024 wait in registers while these are
// used.  2048 x 2048 x 6144: int4 76 us (0.68 PFLOP/s), MXFP4 62 (0.83); 4096 x 6144 x 6144 378 and 296 (0.82, 1.04).
// A wavefront decodes eight codes a lane in 69 clocks for int4 and 26 for MXFP4; the MFMA that takes them adds 10.
template <DenseOp OP, int WTYPE, int WT, int WN, int FT, int FN, int NST>
__global__ __launch_bounds__(WT * WN * 64) void quant_tile_kernel(GroupedArgs g) {
  constexpr int NW = WT * WN, BT = WT * FT * 16, BN = WN * FN * 16, kThreads = NW * 64;
  constexpr int NO = OP == DENSE_GLU ? BN / 2 : BN;
  constexpr int kA = BT * 128, kB = BN * 32, kHalf = kA + kB, kStage = 2 * kHalf;
  constexpr int kChunk = 8;                              // steps that share a stretch of scales
  constexpr int kGroups = kInt4<WTYPE> ? 8 : 32;         // scales of a row in it
  constexpr int kRow = kInt4<WTYPE> ? 4 * BN : 144;      // bytes from group to group, from row to row
  // scales a thread holds: one fp16 each, or four bytes
  constexpr int kHeld = BN * kGroups / (kInt4<WTYPE> ? 1 : 4) / kThreads;
  static_assert(kHeld * kThreads * (kInt4<WTYPE> ? 1 : 4) == BN * kGroups, "threads hold whole shares");
  extern __shared__ __align__(16) char lds[];
  char* scales = lds + NST * kStage;
  Tile tile;
  if (!find_tile<BT, true>(g, blockIdx.x, (g.d.N + NO - 1) / NO, tile)) return;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wt = wave / WN, wn = wave % WN, q = lane >> 4, ln = lane & 15;
  constexpr int F = OP == DENSE_GLU ? 2 : 1;
  const int K = g.d.K, per_row = K / kScaleGroup<WTYPE>;
  const DenseArgs a = expert_args(g, tile.e, tile.t1, (int64_t)F * g.d.N * (K / 2));
  const int t0 = tile.t0, n0 = tile.col * NO;
  // the expert's weight row of tile row r
  auto w_row = [&](int r) {
    if constexpr (OP == DENSE_GLU) return (int64_t)min(n0 + (r >> 5) * 16 + (r & 15), a.N - 1) + (r & 16 ? a.N : 0);
    return (int64_t)min(n0 + r, a.N - 1);
  };
  RowOperand<BT, NW> oa;
  oa.init(wave, lane, [&](int r) { return static_cast<const char*>(a.a) + x_row(g, min(t0 + r, a.T - 1)) * a.lda * 2; });
  constexpr int kCodes = BN / 32, kCodesPer = (kCodes + NW - 1) / NW, kCodesMin = kCodes / NW;   // 1024-byte copies a half
  static_assert(kCodes % NW == 0 || kCodesPer == 1, "copies divide evenly, or go one each to the first");
  const char* codes[kCodesPer];
  int part[kCodesPer];
#pragma unroll
  for (int i = 0; i < kCodesPer; ++i) {
    const int r = 32 * (wave + i * NW) + (lane >> 1);
    part[i] = ((lane & 1) ^ ((r >> 3) & 1)) * 16;
    codes[i] = static_cast<const char*>(a.b) + w_row(min(r, BN - 1)) * (K / 2) + part[i];
  }
  Frags<BT, true, FT> fa;
  fa.init(wt * FT * 16, lane);
  const int nk = (K + 127) / 128;
  const uint32_t lds0 = lds_addr(lds);
  const int exist = min(BT, a.T - t0), n_a = decltype(oa)::copies(wave, exist);        // rows of the tile that are there
  auto fetch = [&](int k) {
    const uint32_t st = lds0 + k % NST * kStage;
    const bool mine = kCodesMin == kCodesPer || wave < kCodes;
    if (128 * k + 128 <= K) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        oa.copy(st + h * kHalf, wave, 256 * (int64_t)k + 128 * h, 128, n_a);
#pragma unroll
        for (int i = 0; i < kCodesPer; ++i)
          if (mine) copy_to_lds(st + h * kHalf + kA + (wave + i * NW) * 1024, codes[i] + 64 * k + 32 * h);
      }
    } else {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int at = 128 * k + 64 * h, valid = min(max(K - at, 0), 64);
        oa.copy(st + h * kHalf, wave, (int64_t)at * 2, valid * 2, n_a);
#pragma unroll
        for (int i = 0; i < kCodesPer; ++i)
          if (mine)
            copy_to_lds(st + h * kHalf + kA + (wave + i * NW) * 1024,
                        part[i] < valid / 2 ? codes[i] + at / 2 : reinterpret_cast<const char*>(g_zeros));
      }
    }
  };
  // this thread's scales of chunk c: thread after thread along the rows
  uint32_t held[kHeld];
  const bool words = K % 128 == 0;                       // MXFP4 rows of whole words
  auto hold = [&](int c) {
#pragma unroll
    for (int i = 0; i < kHeld; ++i) {
      const int idx = threadIdx.x + i * kThreads;
      held[i] = 0;
      if constexpr (kInt4<WTYPE>) {
        const int at = c * 8 + idx % 8;
        if (at < per_row)
          held[i] = static_cast<const uint16_t*>(g.ws)[((int64_t)tile.e * F * a.N + w_row(idx / 8)) * per_row + at];
      } else {
        const int at = c * 32 + idx % 8 * 4;
        const uint8_t* p = static_cast<const uint8_t*>(g.ws) + ((int64_t)tile.e * F * a.N + w_row(idx / 8)) * per_row + at;
        if (words) {
          if (at < per_row) held[i] = *reinterpret_cast<const uint32_t*>(p);
        } else {
#pragma unroll
          for (int b = 0; b < 4; ++b)
            if (at + b < per_row) held[i] |= (uint32_t)p[b] << (8 * b);
        }
      }
    }
  };
  auto place = [&] {
#pragma unroll
    for (int i = 0; i < kHeld; ++i) {
      const int idx = threadIdx.x + i * kThreads;
      if constexpr (kInt4<WTYPE>) {
        *reinterpret_cast<float*>(scales + idx % 8 * kRow + idx / 8 * 4) = int4_scale((uint16_t)held[i]);
      } else {
        f32x4_t v;
#pragma unroll
        for (int j = 0; j < 4; ++j) v[j] = e8m0(held[i] >> (8 * j) & 0xFF);
        *reinterpret_cast<f32x4_t*>(scales + idx / 8 * kRow + idx % 8 * 16) = v;
      }
    }
  };
  f32x4_t acc[FT][FN];
#pragma unroll
  for (int i = 0; i < FT; ++i)
#pragma unroll
    for (int j = 0; j < FN; ++j) acc[i][j] = f32x4_t{0.f, 0.f, 0.f, 0.f};
  const int blocks = __builtin_amdgcn_readfirstlane((exist + 15) / 16 - wt * FT);
  // this lane's codes of the first 32 k of a half, and its scales, of fragment 0
  const int code_at = kA + (wn * FN * 16 + ln) * 32 + ((ln >> 3) << 4) + 4 * q, scale_at = (wn * FN * 16 + ln) * kRow;
  auto multiply = [&](int k, int upto) {
    const char* st = lds + k % NST * kStage;
    const char* const codes_at[2] = {st + code_at, st + (code_at ^ 16)};
    bf16x8_t bf[FN][4];
#pragma unroll
    for (int j = 0; j < FN; ++j) {
      f32x4_t scale = f32x4_t{0.f, 0.f, 0.f, 0.f};       // of the row's four blocks
      if constexpr (kMx<WTYPE>) scale = *reinterpret_cast<const f32x4_t*>(scales + scale_at + j * 16 * kRow + k % kChunk * 16);
#pragma unroll
      for (int s = 0; s < 4; ++s)
        bf[j][s] = decode8<WTYPE>(*reinterpret_cast<const uint32_t*>(codes_at[s & 1] + (s >> 1) * kHalf + j * 512), scale[s]);
    }
    f32x4_t sc[kInt4<WTYPE> ? FN : 1];
    if constexpr (kInt4<WTYPE>) {
#pragma unroll
      for (int j = 0; j < FN; ++j)
        sc[j] = *reinterpret_cast<const f32x4_t*>(scales + k % kChunk * kRow + ((wn * FN + j) * 16 + 4 * q) * 4);
    }
#pragma unroll
    for (int i = 0; i < FT; ++i) {
      if (i >= upto) continue;
      bf16x8_t af[4];
#pragma unroll
      for (int s = 0; s < 4; ++s) af[s] = fa.bf16(st + (s >> 1) * kHalf, i, s & 1);
      if constexpr (kInt4<WTYPE>) {
        f32x4_t p[FN];
#pragma unroll
        for (int j = 0; j < FN; ++j) p[j] = f32x4_t{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int s = 0; s < 4; ++s)
#pragma unroll
          for (int j = 0; j < FN; ++j) p[j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(bf[j][s], af[s], p[j], 0, 0, 0);
#pragma unroll
        for (int j = 0; j < FN; ++j)
#pragma unroll
          for (int e = 0; e < 4; ++e) acc[i][j][e] = __builtin_fmaf(p[j][e], sc[j][e], acc[i][j][e]);
      } else {
#pragma unroll
        for (int s = 0; s < 4; ++s)
#pragma unroll
          for (int j = 0; j < FN; ++j)
            acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(bf[j][s], af[s], acc[i][j], 0, 0, 0);
      }
    }
  };
  hold(0);
#pragma unroll
  for (int k = 0; k < NST - 1; ++k)
    if (k < nk) fetch(k);
  for (int k = 0; k < nk; ++k) {
    if (k % kChunk == 0) {
      __syncthreads();                                   // the scales before these have been used
      place();
    }
    // (scales being fetched only make this wait for more)
    if (NST > 2 && k + NST - 1 <= nk) wait_steps<2 * (NST - 2), decltype(oa)::kPer, kCodesMin>(n_a);
    else wait_stage<0>();
    if (k + NST - 1 < nk) fetch(k + NST - 1);
    if (k % kChunk == 0 && k + kChunk < nk) hold(k / kChunk + 1);
    if (blocks >= FT) multiply(k, FT);
    else if (blocks > 0) multiply(k, blocks);
  }
  finish_tile<OP, WT, WN, FT, FN>(a, lds, t0, n0, acc);
}

// ------------------------------------------------------------------ launches

namespace {

// The most tiles of `bt` rows there can be.
int64_t row_tiles(const GroupedArgs& a, int bt) {
  return a.offsets ? (int64_t)a.R / bt + std::min(a.E, a.R) : ((int64_t)a.R + bt - 1) / bt;
}

template <DenseOp OP, bool BK, int WT, int WN, int FT, int FN, int NST>
void launch_rows(const GroupedArgs& a, hipStream_t s) {
  constexpr int BT = WT * FT * 16, BN = WN * FN * 16, NO = OP == DENSE_GLU ? BN / 2 : BN;
  constexpr int kLds = std::max(NST * (BT + BN) * 128, BT * (BN + 4) * 4);
  static_assert(kLds <= 160 * 1024, "LDS of one workgroup");
  const int64_t tiles = row_tiles(a, BT) * ((a.d.N + NO - 1) / NO);
  grouped_tile_kernel<OP, BK, WT, WN, FT, FN, NST><<<dim3((unsigned)tiles), WT * WN * 64, kLds, s>>>(a);
}

template <DenseOp OP, int WTYPE, int WT, int WN, int FT, int FN, int NST>
void launch_quant(const GroupedArgs& a, hipStream_t s) {
  constexpr int BT = WT * FT * 16, BN = WN * FN * 16, NO = OP == DENSE_GLU ? BN / 2 : BN;
  constexpr int kLds = std::max(NST * 2 * (BT * 128 + BN * 32) + BN * (kInt4<WTYPE> ? 32 : 144), BT * (BN + 4) * 4);
  static_assert(kLds <= 160 * 1024, "LDS of one workgroup");
  const int64_t tiles = row_tiles(a, BT) * ((a.d.N + NO - 1) / NO);
  quant_tile_kernel<OP, WTYPE, WT, WN, FT, FN, NST><<<dim3((unsigned)tiles), WT * WN * 64, kLds, s>>>(a);
}

template <DenseOp OP, int WTYPE, int F, int CW, int KW, int P, int U>
void launch_few(const GroupedArgs& a, hipStream_t s) {
  constexpr int NR = 16 / P, NO = CW * NR * (OP == DENSE_GLU ? 1 : F);
  grouped_few_kernel<OP, WTYPE, F, CW, KW, P, U>
      <<<dim3((a.d.N + NO - 1) / NO, (unsigned)row_tiles(a, NR)), CW * KW * 64, 0, s>>>(a);
}

// us of the two sides of each choice, at rows x columns x k, with `E x rows` where they are grouped.
template <DenseOp OP, int WTYPE>
void launch_sized(const GroupedArgs& a, hipStream_t s) {
  constexpr bool GLU = OP == DENSE_GLU, Q = WTYPE != PE_W_BF16;
  const int rows = a.offsets ? a.R / std::min(a.E, a.R) : a.R;    // of a matrix, on average
  auto blocks = [&](int nr, int cols) { return row_tiles(a, nr) * ((a.d.N + cols - 1) / cols); };
  // Streaming reads a matrix's weights once for every 16 rows and is over when its workgroups are; tiles read them once and
  // keep more on the way, but are mostly empty where rows are few.  Streaming against tiles, by `few` workgroups:
  // - one matrix: to 576 (int4 96 x 2048 x 6144 25 against 34, 48 x 6144 x 2048 14.0 and 14.0, GLU of 32 x 6144 x 2048
  //   14.8 and 14.8, of 128 x 768 x 2048 10.4 against 14.0); of up to 4 rows and a longer k to 1024 (int4 1 x 32768 x
  //   4096 22 against 28, 4 rows 24.5 against 28; 1 x 65536 x 2048 23.1 against 20.6, 1 x 32768 x 1024 10.9 against 10.2);
  // - grouped, up to 16 rows a matrix on average, in 4 bits to 1024 of the workgroups that there can be (int4 GLU
  //   768 x 2048, 4 experts of 4 rows 6.8 against 16, 8 of 16 12.2 against 16.7, 16 of 16 (1536) 16.1 against 16.8;
  //   1536 x 2048, 24 of 4 (1200) 21.6 against 20.0), in bf16, with its bytes, to 288 (GLU 768 x 2048, 4 of 8 10.7
  //   against 17.2, 4 of 24 (480) 18.3 against 16.3; 1536 x 2048, 12 of 4 (720) 19.2 against 16.8);
  // - grouped, under 4 rows, whatever the workgroups: most experts that are reached have one or two (MXFP4 2880 x 2880,
  //   24 of 2 34 against 47).  Where there are very many it is the slower (int4 GLU 768 x 2048, routed to 128 experts:
  //   one row on average 36 against 33, two 50 against 45, three 62 against 49), as where one expert has most of the
  //   rows (all 384 of one of 128: 34 against 17).
  const int64_t few = blocks(16, GLU ? 16 : 32);
  if (a.offsets ? (rows < 4 && blocks(8, 8) < 1 << 24) || (rows <= 16 && few <= (Q ? 1024 : 288))
                : few <= (rows <= 4 && a.d.K > 1024 ? 1024 : 576)) {
    if constexpr (GLU) {
      // 16 rows, or 8 and two parts of k; where those are many, two workgroups' work in one (4 rows for 30 experts, int4
      // 768 x 2048: 17.6 against 19.2; bf16 41.7 against 38.6).  (bf16 comes here grouped alone.)
      if constexpr (Q) {
        if (rows > 8) {
          launch_few<OP, WTYPE, 2, 1, 4, 1, 2>(a, s);
          return;
        }
        if (blocks(8, 8) > 1024) {
          launch_few<OP, WTYPE, 2, 2, 2, 2, 2>(a, s);
          return;
        }
      }
      launch_few<OP, WTYPE, 2, 1, 4, 2, 2>(a, s);
    } else {
      // short sums: wavefronts for columns rather than for parts of k (30 experts, int4 2048 x 768: 12.4 against 14.0)
      if (a.d.K <= 1024) launch_few<OP, WTYPE, 2, 2, 2, 1, 3>(a, s);
      // the smallest workgroups while they are few (1 x 2048 x 6144: 5.5 against 6.7), 32 columns where those
      // make 128 (16 x 6144 x 2048: 7.3 against 8.4), two parts of k otherwise (16 x 2048 x 6144: 9.0 against 15)
      else if (rows <= 8 && blocks(8, 8) <= 512) launch_few<OP, WTYPE, 1, 1, 4, 2, 2>(a, s);
      else if (blocks(16, 32) >= 128) launch_few<OP, WTYPE, 2, 1, 4, 1, 2>(a, s);
      else launch_few<OP, WTYPE, 2, 1, 4, 2, 2>(a, s);
    }
    return;
  }
  if constexpr (Q) {
    // The largest tile that still fills the units where a matrix has the rows for it: 128 x 256 (4096 x 6144 x 6144, int4:
    // 378 against 438 in 128 x 128 and 493 in 64 x 128), 128 x 128 (2048 x 2048 x 6144: 76 against 96 in 32 x 128
    // and 92 in 64 x 128).
    // Below, 16 x 128 where one matrix makes few workgroups (256 x 2048 x 2048: 14.5 against 16.2 in 32 x 128; 1000 x 2880
    // x 2816: 53 against 36), and 32 x 128, of which more fit in a unit, against 64 x 128: int4, 32 experts of 128
    // rows, 2880 x 2816, 133 against 149, 128 of 8, GLU 768 x 2048, 53 against 66; MXFP4, whose tiles cost less to decode
    // and gain from reuse, 167 against 136 and 54 against 62, but of one matrix 1000 x 2880 x 2816 29 against 30.
    const int cols = GLU ? 64 : 128;
    if (rows >= 256 && blocks(128, 2 * cols) >= 256) launch_quant<OP, WTYPE, 2, 4, 4, 4, 2>(a, s);
    else if (rows >= 256 && blocks(128, cols) >= 256) launch_quant<OP, WTYPE, 2, 4, 4, 2, 2>(a, s);
    else if (!a.offsets && blocks(64, cols) < 128) launch_quant<OP, WTYPE, 1, 4, 1, 2, 3>(a, s);
    else if (WTYPE == PE_W_INT4_G128 || !a.offsets || rows <= 16) launch_quant<OP, WTYPE, 1, 4, 2, 2, 2>(a, s);
    else if constexpr (WTYPE != PE_W_INT4_G128) launch_quant<OP, WTYPE, 2, 4, 2, 2, 2>(a, s);
  } else {
    // 64 x 128 in four stages for few rows (8 experts of 64, GLU 768 x 2048: 19.7 against 26.3; 128 of 128: 284 against 227)
    if (rows <= 96) launch_rows<OP, true, 2, 4, 2, 2, 4>(a, s);
    else launch_rows<OP, true, 4, 2, 2, 4, 2>(a, s);
  }
}

}  // namespace

void launch_grouped(DenseOp op, int wtype, const GroupedArgs& a, hipStream_t s) {
  if (wtype == PE_W_BF16) {
    if (op == DENSE_GLU) launch_sized<DENSE_GLU, PE_W_BF16>(a, s);
    else launch_sized<DENSE_LINEAR, PE_W_BF16>(a, s);
  } else if (wtype == PE_W_INT4_G128) {
    if (op == DENSE_GLU) launch_sized<DENSE_GLU, PE_W_INT4_G128>(a, s);
    else launch_sized<DENSE_LINEAR, PE_W_INT4_G128>(a, s);
  } else {
    if (op == DENSE_GLU) launch_sized<DENSE_GLU, PE_W_MXFP4_B32>(a, s);
    else launch_sized<DENSE_LINEAR, PE_W_MXFP4_B32>(a, s);
  }
}

void launch_grouped_back(DenseOp op, const GroupedArgs& a, hipStream_t s) {
  // as in launch_sized (8 experts of 64: dh 21.3 against 31.2, dx 15.5 against 21.3; 128 of 128: dh 178 against 153)
  const bool small = a.R / std::min(a.E, a.R) <= 96;
  if (op == DENSE_DGLU && small) launch_rows<DENSE_DGLU, false, 2, 4, 2, 2, 4>(a, s);
  else if (op == DENSE_DGLU) launch_rows<DENSE_DGLU, false, 4, 2, 2, 4, 2>(a, s);
  else if (small) launch_rows<DENSE_LINEAR, false, 2, 4, 2, 2, 4>(a, s);
  else launch_rows<DENSE_LINEAR, false, 4, 2, 2, 4, 2>(a, s);
}

namespace {

template <bool GATHER, int WT, int WN, int FT, int FN, int NST>
void launch_weights(const GroupedArgs& a, hipStream_t s) {
  constexpr int BT = WT * FT * 16, BN = WN * FN * 16;
  constexpr int kLds = std::max(NST * (BT + BN) * 128 + 32 * 64 * 4, BT * (BN + 4) * 4);
  static_assert(kLds <= 160 * 1024, "LDS of one workgroup");
  const int64_t tiles = (int64_t)((a.d.T + BT - 1) / BT) * ((a.d.N + BN - 1) / BN);
  grouped_weights_kernel<GATHER, WT, WN, FT, FN, NST>
      <<<dim3((unsigned)((tiles + 7) / 8 * 8 * a.E)), WT * WN * 64, kLds, s>>>(a);
}

}  // namespace

void launch_grouped_weights(const GroupedArgs& a, hipStream_t s) {
  if (a.rows) launch_weights<true, 2, 4, 4, 2, 2>(a, s);
  else launch_weights<false, 2, 4, 4, 2, 2>(a, s);
}

}  // namespace pe
