// grad_norm.hip -- the global norm of each rank's gradients over many
// tensors, clipping by it, and the passes that follow the fold of an
// all-reduce with clipping.
//
// All of it waits for memory: a norm is one read of the gradients and two
// 64-bit operations an element, a clip one read and one write. Nothing is
// multiplied but by a scalar, so no matrix instructions.
//
// The tensors are walked through the plan's tiles of 64 vectors (1 KiB), the
// numbering of the in-place bucket all-reduce. In the norm and the clip of
// ranks by themselves a wave takes a group of 16 consecutive tiles of one
// rank: its lanes first fetch the group's metadata, a tile per lane
// (descriptor index, descriptor, gradient address: three dependent loads for
// the whole group instead of three per tensor), then the wave streams the
// tiles, eight loads in flight, with the addresses read back from those
// lanes. Four waves of a workgroup read 64 KiB in a row, and four neighbouring
// workgroups share an XCD and with it the lines of the tile map.
//
// Measured: the norm of the GPT-2 small gradients (498 MB) 74 us, 6.7 TB/s,
// with loads that bypass the caches (86 us without); of one Llama-7B layer in
// bf16 on 8 ranks (3.2 GB) 0.48 ms, 6.7 TB/s; a 2 GiB copy runs at 6.6.
#include <algorithm>
#include <cmath>

#include "bucket_run.hpp"

namespace ddpsim {
namespace {

constexpr int kGroup = kNormGroup;  // tiles of a wave
constexpr int kBatch = 8;           // tiles whose loads are in flight together
constexpr int kWaves = 4;           // waves of a workgroup
constexpr int kFinishWaves = 16;    // waves of a block of the last join
// Sums of a parameter that one wave joins; the block takes longer ones (GPT-2
// small with every parameter's norm: 5.8 us, with 512 here 8.8).
constexpr int64_t kWaveSlots = 1024;
constexpr int kJoinGroup = kNormJoinGroup;
constexpr int kSmallWaves = 16;  // waves of the one-workgroup kernels
// Most tiles of a rank whose norms one workgroup takes: 7 to 8 us a call up
// to 256, where two launches take 10; 512 in bf16 14.
constexpr int kSmallNormTiles = 256;
// The all-reduce with clipping of a small set by one workgroup, a tile per
// wave, against the launches of several workgroups: two, or three where the
// parameters' norms are wanted (us a call, fp32; bf16 takes up to 2 more with
// few ranks and 6 with 64):
//   ranks                      8           16          32          64
//   tiles                    1   16      8   16      8   16      8   16
//   one workgroup           6.5  7.6    8.4  9.7   11.5 16.5   18.2 27.3
//   two launches            9.8 10.1   10.5 10.1   12.1 12.2   16.0 16.1
//   one, parameters' norms  6.9  8.4    9.0 10.2   12.1 17.1   18.8 27.9
//   three launches         13.0 13.4   13.8 13.2   15.0 15.1   18.8 19.3
// A wave folds 8 ranks at a time, so that with many ranks its batches follow
// one another in the one compute unit that the launch fills, and more than 8
// waves then wait for one another. With 32 tiles the waves' second folds cost
// more than the launch they save.
constexpr int kSmallSyncTiles = kSmallWaves;
bool small_sync(int64_t tiles, int32_t p, bool param_norms) {
  if (tiles > (p <= 16 ? kSmallSyncTiles : kSmallSyncTiles / 2)) return false;
  return p <= 32 || param_norms;
}
// Most tile sums that the spreading pass joins by itself: 11 us a call
// against 14 with a launch for the join.
constexpr int kInlineTiles = 1024;
static_assert(kGroup <= 64 && kGroup % kBatch == 0, "a lane per tile");
static_assert(kBucketThreads == 64 && kBucketVpt == 1, "a plan tile is one vector per lane");

// Lane k holds tile (group * kGroup + k) of one rank.
struct LaneTile {
  uint64_t src;   // address of the tile's first whole vector
  int32_t count;  // whole vectors (0..64; 0 beyond the last tile)
  int32_t seg;    // descriptor index, -1 beyond the last tile
  int32_t ends;   // the tile is its parameter's last
  // elements before and after the parameter's whole vectors (first tile only)
  uint64_t head, tail;
  int32_t n_head, n_tail;
};

template <typename Tr>
__device__ __forceinline__ LaneTile lane_tile(const SegDesc *__restrict__ seg,
                                              const int32_t *__restrict__ tile_seg,
                                              int64_t map_stride, int64_t tile, int64_t tiles,
                                              const void *const *__restrict__ grads, bool on) {
  constexpr int V = Tr::kVec;
  constexpr int64_t kElemBytes = sizeof(typename Tr::elem);
  LaneTile x = {};
  x.seg = -1;
  if (!on || tile >= tiles) return x;
  x.seg = tile_seg[tile_map_index(tile, map_stride)];
  const SegDesc d = seg[x.seg];
  const int64_t k = tile - d.tile_begin;
  const uint64_t base = reinterpret_cast<uint64_t>(grads[d.param]);
  const int64_t m = static_cast<int64_t>(base % kVecBytes) / kElemBytes;
  const ChunkSpan c = make_span(m, d.len + m, V);  // indices from the aligned address below base
  const uint64_t aligned = base - static_cast<uint64_t>(m * kElemBytes);
  const int64_t left = (c.ve - c.vs) / V - k * 64;
  x.src = aligned + static_cast<uint64_t>((c.vs / V + k * 64) * kVecBytes);
  x.count = static_cast<int32_t>(left < 0 ? 0 : left > 64 ? 64 : left);
  x.ends = (k + 1) * 64 * V >= d.len;
  if (k == 0) {
    x.head = aligned + static_cast<uint64_t>(c.s * kElemBytes);
    x.n_head = static_cast<int32_t>(c.head_end - c.s);
    x.tail = aligned + static_cast<uint64_t>(c.tail_begin * kElemBytes);
    x.n_tail = static_cast<int32_t>(c.e - c.tail_begin);
  }
  return x;
}

__device__ __forceinline__ uint64_t read_lane(uint64_t v, int lane) {
  const uint32_t lo = __builtin_amdgcn_readlane(static_cast<uint32_t>(v), lane);
  const uint32_t hi = __builtin_amdgcn_readlane(static_cast<uint32_t>(v >> 32), lane);
  return (static_cast<uint64_t>(hi) << 32) | lo;
}

// The partial sums of one wave: group g of `group` tiles (at most kGroup) of
// the rank whose addresses are `grads`, to out[g + descriptor index].
template <typename Tr, int NT>
__device__ __forceinline__ void norm_group(const SegDesc *__restrict__ seg,
                                           const int32_t *__restrict__ tile_seg,
                                           int64_t map_stride, int64_t tiles, int64_t g,
                                           int32_t group, const void *const *__restrict__ grads,
                                           double *out) {
  constexpr int V = Tr::kVec;
  const int lane = static_cast<int>(threadIdx.x) & 63;
  const LaneTile mine = lane_tile<Tr>(seg, tile_seg, map_stride, g * group + lane, tiles, grads,
                                      lane < group);
  out += g;
  // a lane adds the odd elements at its tile's parameter's ends
  NormSum<NT> odd;
  for (int i = 0; i < mine.n_head; ++i) {
    odd.add(Tr::load1(reinterpret_cast<const void *>(mine.head), i));
  }
  for (int i = 0; i < mine.n_tail; ++i) {
    odd.add(Tr::load1(reinterpret_cast<const void *>(mine.tail), i));
  }
  int32_t cur = __builtin_amdgcn_readlane(mine.seg, 0);
  NormSum<NT> sum;
  auto flush = [&]() {
    if (mine.seg == cur) sum.join(odd);
    join_wave(sum);
    if (lane == 0) out[cur] = sum.part();
    sum = NormSum<NT>();
  };
#pragma unroll
  for (int b = 0; b < kGroup; b += kBatch) {
    uint4 x[kBatch];
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      const uint64_t src = read_lane(mine.src, b + u);
      const int32_t count = __builtin_amdgcn_readlane(mine.count, b + u);
      x[u] = lane < count ? load_vec<true>(reinterpret_cast<const void *>(src), lane)
                          : make_uint4(0, 0, 0, 0);
    }
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      const int32_t s = __builtin_amdgcn_readlane(mine.seg, b + u);
      if (s != cur && s >= 0) {
        flush();
        cur = s;
      }
      float w[V];
      Tr::widen(x[u], w);
#pragma unroll
      for (int e = 0; e < V; ++e) sum.add(w[e]);
    }
  }
  flush();
  // the group's last tile, and the slot after it if its parameter ends there
  const int64_t left = tiles - g * group;
  const int32_t last = static_cast<int32_t>(left < group ? left : group) - 1;
  if (lane == last && mine.ends) out[cur + 1] = 0.0;
}

template <typename Tr, int NT>
__global__ __launch_bounds__(64 * kWaves) void grad_norm_kernel(
    const SegDesc *__restrict__ seg, const int32_t *__restrict__ tile_seg, int64_t map_stride,
    int64_t tiles, int64_t groups, int32_t n_params, const void *const *__restrict__ ptrs,
    double *__restrict__ partial, int64_t slots) {
  const int64_t g = xcd_run<kXcdRun>(blockIdx.x, gridDim.x) * kWaves +
                    __builtin_amdgcn_readfirstlane(static_cast<int32_t>(threadIdx.x) >> 6);
  if (g >= groups) return;
  const int32_t rank = static_cast<int32_t>(blockIdx.y);
  norm_group<Tr, NT>(seg, tile_seg, map_stride, tiles, g, kGroup,
                     ptrs + static_cast<int64_t>(rank) * n_params,
                     partial + static_cast<int64_t>(rank) * slots);
}

// The tile sums of a large plan, joined in groups of kJoinGroup tiles before
// the last join: a wave per group, a slot per (group, descriptor) as in
// grad_norm_kernel. One workgroup joining the 486,093 tile sums of the GPT-2
// small gradients by itself took 210 us; this takes 6 and the last join 4.
template <int NT>
__global__ __launch_bounds__(64) void norm_join_kernel(
    const double *__restrict__ tile_sums, int64_t tiles, const SegDesc *__restrict__ seg,
    const int32_t *__restrict__ tile_seg, int64_t map_stride, int64_t tile_elems,
    double *__restrict__ joined) {
  const int lane = static_cast<int>(threadIdx.x);
  const int64_t g = blockIdx.x;
  const int64_t end = std::min((g + 1) * kJoinGroup, tiles);
  int32_t s = tile_seg[tile_map_index(g * kJoinGroup, map_stride)];
  for (int64_t t = g * kJoinGroup; t < end; ++s) {
    const SegDesc d = seg[s];
    const int64_t seg_end = d.tile_begin + (d.len + tile_elems - 1) / tile_elems;
    const int64_t stop = std::min(seg_end, end);
    NormSum<NT> sum;
#pragma unroll
    for (int k = 0; k < kJoinGroup / 64; ++k) {
      if (t + k * 64 + lane < stop) sum.join_part(tile_sums[t + k * 64 + lane]);
    }
    join_wave(sum);
    if (lane == 0) {
      joined[g + s] = sum.part();
      if (stop == end && stop == seg_end) joined[g + s + 1] = 0.0;
    }
    t = stop;
  }
}

// The sum of partial[i0 .. i1) over `width` threads, of which this is `me`;
// the loads of a batch are in flight together.
template <int NT>
__device__ __forceinline__ NormSum<NT> join_range(const double *__restrict__ partial, int64_t i0,
                                                  int64_t i1, int me, int width) {
  constexpr int kLoads = 8;
  NormSum<NT> sum;
  for (int64_t i = i0 + me; i < i1; i += kLoads * width) {
    double x[kLoads];
#pragma unroll
    for (int k = 0; k < kLoads; ++k) {
      const int64_t j = i + static_cast<int64_t>(k) * width;
      x[k] = j < i1 ? partial[j] : 0.0;
    }
#pragma unroll
    for (int k = 0; k < kLoads; ++k) sum.join_part(x[k]);
  }
  return sum;
}

// The partial sums [i0, i1) of descriptor i, with `group` tiles per sum (1: a
// sum per tile, without gaps).
__device__ __forceinline__ void slots_of_param(const SegDesc &d, int32_t i, int32_t group,
                                               int64_t tile_elems, int64_t &i0, int64_t &i1) {
  const int64_t a = d.tile_begin, b = a + (d.len + tile_elems - 1) / tile_elems;
  i0 = group == 1 ? a : a / group + i;
  i1 = group == 1 ? b : (b - 1) / group + i + 1;
}

// Block 0 joins all of a rank's partial sums into its norm; the other blocks
// take kFinishWaves descriptors each and join those of each parameter, a wave
// per parameter, or the whole block for one of more than kWaveSlots sums.
template <int NT>
__global__ __launch_bounds__(64 * kFinishWaves) void norm_finish_kernel(
    const double *__restrict__ partial, int64_t slots, const SegDesc *__restrict__ seg,
    int32_t nseg, int32_t group, int64_t tile_elems, int32_t n_params,
    float *__restrict__ norms, float *__restrict__ param_norms) {
  __shared__ double parts[kFinishWaves];
  const int32_t rank = static_cast<int32_t>(blockIdx.y);
  const int tid = static_cast<int>(threadIdx.x);
  const double *src = partial + static_cast<int64_t>(rank) * slots;
  auto block_norm = [&](int64_t i0, int64_t i1, float *out) {
    NormSum<NT> sum = join_range<NT>(src, i0, i1, tid, 64 * kFinishWaves);
    join_wave(sum);
    if ((tid & 63) == 0) parts[tid >> 6] = sum.part();
    __syncthreads();
    if (tid == 0) {
      NormSum<NT> all;
      for (int w = 0; w < kFinishWaves; ++w) all.join_part(parts[w]);
      *out = all.norm();
    }
    __syncthreads();
  };
  if (blockIdx.x == 0) {
    block_norm(0, slots, norms + rank);
    return;
  }
  const int32_t s0 = (static_cast<int32_t>(blockIdx.x) - 1) * kFinishWaves;
  const auto range_of = [&](int32_t i, int64_t &i0, int64_t &i1) {
    const SegDesc d = seg[i];
    slots_of_param(d, i, group, tile_elems, i0, i1);
    return param_norms + static_cast<int64_t>(rank) * n_params + d.param;
  };
  __shared__ int32_t large[kFinishWaves];
  const int32_t mine = s0 + (tid >> 6);
  int64_t i0 = 0, i1 = 0;
  if (mine < nseg) {
    float *out = range_of(mine, i0, i1);
    if (i1 - i0 <= kWaveSlots) {
      NormSum<NT> sum = join_range<NT>(src, i0, i1, tid & 63, 64);
      join_wave(sum);
      if ((tid & 63) == 0) *out = sum.norm();
    }
  }
  if ((tid & 63) == 0) large[tid >> 6] = i1 - i0 > kWaveSlots;
  __syncthreads();
  for (int k = 0; k < kFinishWaves; ++k) {
    if (!large[k]) continue;  // the same for every thread
    float *out = range_of(s0 + k, i0, i1);
    block_norm(i0, i1, out);
  }
}

// A rank's norms from sums in LDS, by one workgroup of kSmallWaves waves that
// all have passed a barrier since the sums were written: wave 0 the norm
// (returned to every wave), all of them the parameters'.
template <int NT>
__device__ __forceinline__ float finish_in_lds(const double *sums, int64_t slots,
                                               const SegDesc *__restrict__ seg, int32_t nseg,
                                               int32_t group, int64_t tile_elems,
                                               int32_t n_params, float *norm,
                                               float *param_norms) {
  const int lane = static_cast<int>(threadIdx.x) & 63;
  const int wave = static_cast<int>(threadIdx.x) >> 6;
  NormSum<NT> all;
  for (int64_t i = lane; i < slots; i += 64) all.join_part(sums[i]);
  join_wave(all);
  if (threadIdx.x == 0) *norm = all.norm();
  if (param_norms != nullptr) {
    for (int32_t s = wave; s < nseg; s += kSmallWaves) {
      const SegDesc d = seg[s];
      int64_t i0, i1;
      slots_of_param(d, s, group, tile_elems, i0, i1);
      NormSum<NT> sum;
      for (int64_t i = i0 + lane; i < i1; i += 64) sum.join_part(sums[i]);
      join_wave(sum);
      if (lane == 0) param_norms[d.param] = sum.norm();
    }
  }
  return all.norm();
}

// Parameters without elements have no descriptor: their norms, before the
// others' (a barrier lies between).
__device__ __forceinline__ void zero_norms(float *param_norms, int32_t nseg, int32_t n_params) {
  if (param_norms == nullptr || nseg == n_params) return;
  for (int32_t i = static_cast<int32_t>(threadIdx.x); i < n_params; i += 64 * kSmallWaves) {
    param_norms[i] = 0.0f;
  }
}

// The norms of a small set in one launch, a workgroup per rank: no sum leaves
// it, so that nothing waits for a second kernel.
template <typename Tr, int NT>
__global__ __launch_bounds__(64 * kSmallWaves) void small_norm_kernel(
    const SegDesc *__restrict__ seg, const int32_t *__restrict__ tile_seg, int64_t map_stride,
    int32_t tiles, int32_t nseg, int32_t n_params, const void *const *__restrict__ ptrs,
    float *__restrict__ norms, float *__restrict__ param_norms) {
  __shared__ double sums[kSmallNormTiles / 2 + kSmallNormTiles + 1];
  const int32_t rank = static_cast<int32_t>(blockIdx.x);
  const int64_t first = static_cast<int64_t>(rank) * n_params;
  if (param_norms != nullptr) param_norms += first;
  zero_norms(param_norms, nseg, n_params);
  // groups of equal work for the waves, but of two tiles at least: slots of
  // single tiles would be those of tile sums
  const int32_t group =
      std::max(2, std::min(kGroup, (tiles + kSmallWaves - 1) / kSmallWaves));
  const int32_t groups = (tiles + group - 1) / group;
  const int32_t wave = __builtin_amdgcn_readfirstlane(static_cast<int32_t>(threadIdx.x) >> 6);
  for (int32_t g = wave; g < groups; g += kSmallWaves) {
    norm_group<Tr, NT>(seg, tile_seg, map_stride, tiles, g, group, ptrs + first, sums);
  }
  __syncthreads();
  finish_in_lds<NT>(sums, groups + nseg, seg, nseg, group, 64 * Tr::kVec, n_params, norms + rank,
                    param_norms);
}

// All-reduce, norm and clip of a small set (a tile per wave) by one workgroup,
// in one launch: the averages are staged as kStageNorm does, and spread by
// the waves that folded them.
template <typename Tr, int NT>
__global__ __launch_bounds__(64 * kSmallWaves) void small_sync_kernel(
    const SegDesc *__restrict__ seg, const int32_t *__restrict__ tile_seg, int64_t map_stride,
    int32_t tiles, int32_t nseg, int32_t n_params, const void *const *__restrict__ ptrs,
    int32_t p, Divide div, float max_norm, float eps, float *__restrict__ norm,
    float *__restrict__ param_norms) {
  __shared__ double sums[kSmallSyncTiles];
  constexpr int64_t kTile = 64 * Tr::kVec;
  const int32_t wave = __builtin_amdgcn_readfirstlane(static_cast<int32_t>(threadIdx.x) >> 6);
  zero_norms(param_norms, nseg, n_params);
  for (int32_t tile = wave; tile < tiles; tile += kSmallWaves) {
    const SegDesc d = seg[tile_seg[tile_map_index(tile, map_stride)]];
    const int64_t t = tile - d.tile_begin;
    Epilogue<kStageNorm, NT> epi;
    bucket_run<Tr, 1, 8, false>(d, t, t + 1, tile, n_params, ptrs, p, div, epi);
    join_wave(epi.sum);
    if ((threadIdx.x & 63) == 0) sums[tile] = epi.sum.part();
  }
  __syncthreads();
  const float c = clip_coefficient(
      finish_in_lds<NT>(sums, tiles, seg, nseg, 1, kTile, n_params, norm, param_norms), max_norm,
      eps);
  for (int32_t tile = wave; tile < tiles; tile += kSmallWaves) {
    const SegDesc d = seg[tile_seg[tile_map_index(tile, map_stride)]];
    spread_tile<Tr, true, false>(d, tile, n_params, ptrs, p, 0, p, c, false);
  }
}

__global__ void zero_floats_kernel(float *p, int64_t n) {
  const int64_t i = int64_t(blockIdx.x) * blockDim.x + threadIdx.x;
  if (i < n) p[i] = 0.0f;
}

template <typename Tr, bool kNt>
__device__ __forceinline__ void clip_tiles(const LaneTile &mine, int lane, float c) {
  constexpr int V = Tr::kVec;
#pragma unroll
  for (int b = 0; b < kGroup; b += kBatch) {
    uint4 x[kBatch];
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      const uint64_t src = read_lane(mine.src, b + u);
      const int32_t count = __builtin_amdgcn_readlane(mine.count, b + u);
      x[u] = lane < count ? load_vec<kNt>(reinterpret_cast<const void *>(src), lane)
                          : make_uint4(0, 0, 0, 0);
    }
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      const uint64_t dst = read_lane(mine.src, b + u);
      const int32_t count = __builtin_amdgcn_readlane(mine.count, b + u);
      float w[V];
      Tr::widen(x[u], w);
#pragma unroll
      for (int e = 0; e < V; ++e) w[e] = w[e] * c;
      if (lane < count) store_vec<kNt>(reinterpret_cast<void *>(dst), lane, Tr::narrow(w));
    }
  }
}

// One wave per group of tiles of one rank: load, scale, store. A coefficient
// of one changes no value, so such a rank's gradients are not touched. Whole
// lines go past the caches when the gradients outgrow them, as in spread_tile
// (GPT-2 small on 8 ranks, each by itself: 1.43 ms against 1.50 with ordinary
// accesses; tiles inside lines: 0.18 ms ordinary, 0.23 past the caches).
template <typename Tr>
__global__ __launch_bounds__(64 * kWaves) void clip_kernel(
    const SegDesc *__restrict__ seg, const int32_t *__restrict__ tile_seg, int64_t map_stride,
    int64_t tiles, int64_t groups, int32_t n_params, const void *const *__restrict__ ptrs,
    const float *__restrict__ norms, int32_t norm_step, float max_norm, float eps, bool stream) {
  const int32_t rank = static_cast<int32_t>(blockIdx.y);
  const float c = clip_coefficient(norms[rank * norm_step], max_norm, eps);
  if (c == 1.0f) return;
  const int lane = static_cast<int>(threadIdx.x) & 63;
  const int64_t g = xcd_run<kXcdRun>(blockIdx.x, gridDim.x) * kWaves +
                    __builtin_amdgcn_readfirstlane(static_cast<int32_t>(threadIdx.x) >> 6);
  if (g >= groups) return;
  const LaneTile mine = lane_tile<Tr>(seg, tile_seg, map_stride, g * kGroup + lane, tiles,
                                      ptrs + static_cast<int64_t>(rank) * n_params,
                                      lane < kGroup);
  for (int i = 0; i < mine.n_head; ++i) {
    void *at = reinterpret_cast<void *>(mine.head);
    Tr::store1(at, i, Tr::load1(at, i) * c);
  }
  for (int i = 0; i < mine.n_tail; ++i) {
    void *at = reinterpret_cast<void *>(mine.tail);
    Tr::store1(at, i, Tr::load1(at, i) * c);
  }
  if (stream && __all(mine.count == 0 || mine.src % static_cast<uint64_t>(kLineBytes) == 0)) {
    clip_tiles<Tr, true>(mine, lane, c);
  } else {
    clip_tiles<Tr, false>(mine, lane, c);
  }
}

// The norm of at most kInlineTiles tile sums, by every wave for itself.
template <int NT>
__device__ __forceinline__ float wave_norm(const double *__restrict__ partial, int32_t n) {
  NormSum<NT> sum = join_range<NT>(partial, 0, n, static_cast<int>(threadIdx.x) & 63, 64);
  join_wave(sum);
  return sum.norm();
}

// What the spreading pass scales by: a norm in memory, or (kJoin) the pass's
// own join of the tile sums, which one wave writes down. Up to kInlineTiles
// sums that costs less than one more launch.
struct NormSource {
  float *norm;
  const double *partial;
  int32_t sums;  // 0: the norm is there
  int32_t norm_type;
};
template <bool kJoin>
__device__ __forceinline__ float read_norm(const NormSource &src) {
  if constexpr (!kJoin) return *src.norm;
  const float n = src.norm_type == DDP_NORM_L2   ? wave_norm<DDP_NORM_L2>(src.partial, src.sums)
                  : src.norm_type == DDP_NORM_L1 ? wave_norm<DDP_NORM_L1>(src.partial, src.sums)
                                                 : wave_norm<DDP_NORM_INF>(src.partial, src.sums);
  if (blockIdx.x == 0 && threadIdx.x == 0) *src.norm = n;
  return n;
}

// A workgroup takes a tile; its waves split the ranks (fanout_waves).
template <typename Tr, bool kStaged, bool kJoin>
__global__ __launch_bounds__(64 * kMaxFanoutWaves) void clip_fanout_kernel(
    const SegDesc *__restrict__ seg, const int32_t *__restrict__ tile_seg, int64_t map_stride,
    int64_t tiles, int32_t n_params, const void *const *__restrict__ ptrs, int32_t p,
    NormSource source, float max_norm, float eps, bool stream, bool runs) {
  const float c = clip_coefficient(read_norm<kJoin>(source), max_norm, eps);
  if (!kStaged && c == 1.0f) return;
  const int32_t waves = static_cast<int32_t>(blockDim.x) / 64;
  const int32_t wave = __builtin_amdgcn_readfirstlane(static_cast<int32_t>(threadIdx.x) >> 6);
  for (int64_t w = blockIdx.x; w < tiles; w += gridDim.x) {
    const int64_t tile = runs ? xcd_run<kXcdRun>(w, tiles) : w;
    const SegDesc d = seg[tile_seg[tile_map_index(tile, map_stride)]];
    spread_tile<Tr, kStaged, true>(d, tile, n_params, ptrs, p, wave * p / waves,
                                   (wave + 1) * p / waves, c, stream);
  }
}

// Plan, rank count, type and table of a norm or clip call. Whether the plan
// has its descriptor table is asked last (check_uploaded).
ddp_status check_call(const char *what, const ddp_plan *plan, int32_t p, const void *d_grad_ptrs,
                      int32_t dtype, PlanTiles *t) {
  if (!plan_tiles(plan, t)) return fail(DDP_EINVAL, "%s: plan is NULL", what);
  ddp_status s = check_p(p, what);
  if (s != DDP_OK) return s;
  const int eb = elem_bytes_of(dtype);
  if (eb == 0) return fail(DDP_EINVAL, "%s: unknown dtype %d", what, dtype);
  if (eb != t->elem_bytes) {
    return fail(DDP_EINVAL, "%s: dtype has %d-byte elements, the plan %d", what, eb,
                t->elem_bytes);
  }
  if (t->tiles > 0 && d_grad_ptrs == nullptr) {
    return fail(DDP_EINVAL, "%s: gradient pointer table is NULL", what);
  }
  return DDP_OK;
}

ddp_status check_uploaded(const char *what, const PlanTiles &t) {
  if (t.seg_p != 0) return DDP_OK;
  return fail(DDP_ENOTREADY, "%s: call ddp_plan_upload_segments first", what);
}

ddp_status check_norm_type(const char *what, int32_t norm_type) {
  if (norm_type != DDP_NORM_L2 && norm_type != DDP_NORM_L1 && norm_type != DDP_NORM_INF) {
    return fail(DDP_EINVAL, "%s: unknown norm type %d", what, norm_type);
  }
  return DDP_OK;
}

ddp_status check_bound(const char *what, float max_norm, float eps) {
  if (!(max_norm >= 0.0f)) return fail(DDP_EINVAL, "%s: max_norm must be >= 0", what);
  if (!(eps >= 0.0f) || std::isinf(eps)) {
    return fail(DDP_EINVAL, "%s: eps must be finite and >= 0", what);
  }
  return DDP_OK;
}

// n norms and n_each parameters' norms, and the workspace of `need` bytes
// that their sums lie in: the last join writes norms while it reads sums, so
// that none of the three may share memory with another.
ddp_status check_out(const char *what, const float *d_norms, int64_t n, const float *d_param_norms,
                     int64_t n_each, const void *workspace, size_t bytes, size_t need) {
  if (d_norms == nullptr) return fail(DDP_EINVAL, "%s: d_norms is NULL", what);
  if (reinterpret_cast<uintptr_t>(d_norms) % 4 != 0 ||
      reinterpret_cast<uintptr_t>(d_param_norms) % 4 != 0) {
    return fail(DDP_EALIGN, "%s: the norms are not 4-byte aligned", what);
  }
  ddp_status s = check_workspace(what, workspace, bytes, need, nullptr, 0, 0);
  if (s != DDP_OK) return s;
  n_each = d_param_norms != nullptr ? n_each : 0;
  const auto overlap = [](const void *a, int64_t na, const void *b, int64_t nb) {
    return na > 0 && nb > 0 && ranges_overlap(a, na, b, nb);
  };
  const int64_t ws = static_cast<int64_t>(need);
  if (overlap(d_norms, 4 * n, workspace, ws) || overlap(d_param_norms, 4 * n_each, workspace, ws)) {
    return fail(DDP_EALIAS, "%s: the norms overlap the workspace", what);
  }
  if (overlap(d_norms, 4 * n, d_param_norms, 4 * n_each)) {
    return fail(DDP_EALIAS, "%s: d_norms and d_param_norms overlap", what);
  }
  return DDP_OK;
}

template <int NT>
ddp_status launch_finish_nt(const PlanTiles &t, const double *partial, int64_t slots,
                            int32_t group, int32_t ranks, float *d_norms, float *d_param_norms,
                            hipStream_t stream, CallTimer &timer, bool last) {
  if (d_param_norms != nullptr && t.nseg < t.n_params) {
    // parameters without elements have no descriptor
    const int64_t n = static_cast<int64_t>(ranks) * t.n_params;
    ddp_status s = launch(zero_floats_kernel, dim3(static_cast<uint32_t>(ceil_div(n, 256))),
                          dim3(256), stream, timer, false, "zero_floats_kernel launch",
                          d_param_norms, n);
    if (s != DDP_OK) return s;
  }
  const int64_t tile_elems = bucket_tile_elems(kVecBytes / t.elem_bytes);
  const int64_t blocks = 1 + (d_param_norms != nullptr ? ceil_div(t.nseg, kFinishWaves) : 0);
  return launch(norm_finish_kernel<NT>,
                dim3(static_cast<uint32_t>(blocks), static_cast<uint32_t>(ranks)),
                dim3(64 * kFinishWaves), stream, timer, last, "norm_finish_kernel launch",
                partial, slots, t.seg, t.nseg, group, tile_elems, t.n_params, d_norms,
                d_param_norms);
}

// The tile sums of a plan in `partial` into its norms: at once, or through
// norm_join_kernel, whose sums follow the tiles'. Up to kNormJoinTiles sums
// one more launch costs more than it saves.
template <int NT>
ddp_status launch_tile_finish_nt(const PlanTiles &t, double *partial, float *d_norm,
                                 float *d_param_norms, hipStream_t stream, CallTimer &timer,
                                 bool last) {
  if (t.tiles <= kNormJoinTiles) {
    return launch_finish_nt<NT>(t, partial, t.tiles, 1, 1, d_norm, d_param_norms, stream, timer,
                                last);
  }
  const int64_t groups = ceil_div(t.tiles, kJoinGroup);
  double *joined = partial + t.tiles;
  ddp_status s = launch(norm_join_kernel<NT>, dim3(static_cast<uint32_t>(groups)), dim3(64),
                        stream, timer, false, "norm_join_kernel launch", partial, t.tiles, t.seg,
                        t.tile_seg, t.map_stride, bucket_tile_elems(kVecBytes / t.elem_bytes),
                        joined);
  if (s != DDP_OK) return s;
  return launch_finish_nt<NT>(t, joined, groups + t.nseg, kJoinGroup, 1, d_norm, d_param_norms,
                              stream, timer, last);
}

ddp_status launch_tile_finish(const PlanTiles &t, int32_t norm_type, double *partial,
                              float *d_norm, float *d_param_norms, hipStream_t stream,
                              CallTimer &timer, bool last) {
  switch (norm_type) {
    case DDP_NORM_L2:
      return launch_tile_finish_nt<DDP_NORM_L2>(t, partial, d_norm, d_param_norms, stream, timer,
                                                last);
    case DDP_NORM_L1:
      return launch_tile_finish_nt<DDP_NORM_L1>(t, partial, d_norm, d_param_norms, stream, timer,
                                                last);
    default:
      return launch_tile_finish_nt<DDP_NORM_INF>(t, partial, d_norm, d_param_norms, stream, timer,
                                                 last);
  }
}

template <typename Tr, int NT>
ddp_status launch_small_norm(const PlanTiles &t, int32_t p, const void *const *ptrs,
                             float *d_norms, float *d_param_norms, hipStream_t stream,
                             CallTimer &timer, bool last) {
  return launch(small_norm_kernel<Tr, NT>, dim3(static_cast<uint32_t>(p)), dim3(64 * kSmallWaves),
                stream, timer, last, "small_norm_kernel launch", t.seg, t.tile_seg, t.map_stride,
                static_cast<int32_t>(t.tiles), t.nseg, t.n_params, ptrs, d_norms, d_param_norms);
}

template <typename Tr, int NT>
ddp_status launch_small_sync(const PlanTiles &t, int32_t p, const void *const *ptrs,
                             const Divide &div, float max_norm, float eps, float *d_norm,
                             float *d_param_norms, hipStream_t stream, CallTimer &timer) {
  return launch(small_sync_kernel<Tr, NT>, dim3(1), dim3(64 * kSmallWaves), stream, timer, true,
                "small_sync_kernel launch", t.seg, t.tile_seg, t.map_stride,
                static_cast<int32_t>(t.tiles), t.nseg, t.n_params, ptrs, p, div, max_norm, eps,
                d_norm, d_param_norms);
}

template <typename Tr>
ddp_status launch_small_sync_type(int32_t norm_type, const PlanTiles &t, int32_t p,
                                  const void *const *ptrs, const Divide &div, float max_norm,
                                  float eps, float *d_norm, float *d_param_norms,
                                  hipStream_t stream, CallTimer &timer) {
  switch (norm_type) {
    case DDP_NORM_L2:
      return launch_small_sync<Tr, DDP_NORM_L2>(t, p, ptrs, div, max_norm, eps, d_norm,
                                                d_param_norms, stream, timer);
    case DDP_NORM_L1:
      return launch_small_sync<Tr, DDP_NORM_L1>(t, p, ptrs, div, max_norm, eps, d_norm,
                                                d_param_norms, stream, timer);
    default:
      return launch_small_sync<Tr, DDP_NORM_INF>(t, p, ptrs, div, max_norm, eps, d_norm,
                                                 d_param_norms, stream, timer);
  }
}

template <typename Tr, int NT>
ddp_status launch_norm(const PlanTiles &t, int32_t p, const void *const *ptrs, double *partial,
                       float *d_norms, float *d_param_norms, hipStream_t stream,
                       CallTimer &timer, bool last) {
  if (t.tiles > 0 && t.tiles <= kSmallNormTiles) {
    return launch_small_norm<Tr, NT>(t, p, ptrs, d_norms, d_param_norms, stream, timer, last);
  }
  const int64_t slots = norm_slots(t);
  if (t.tiles > 0) {
    const int64_t groups = norm_groups(t);
    ddp_status s = launch(grad_norm_kernel<Tr, NT>,
                          dim3(static_cast<uint32_t>(ceil_div(groups, kWaves)),
                               static_cast<uint32_t>(p)),
                          dim3(64 * kWaves), stream, timer, false, "grad_norm_kernel launch",
                          t.seg, t.tile_seg, t.map_stride, t.tiles, groups, t.n_params, ptrs,
                          partial, slots);
    if (s != DDP_OK) return s;
  }
  return launch_finish_nt<NT>(t, partial, slots, kGroup, p, d_norms, d_param_norms, stream, timer,
                              last);
}

template <typename Tr>
ddp_status launch_norm_of(int32_t norm_type, const PlanTiles &t, int32_t p,
                          const void *const *ptrs, double *partial, float *d_norms,
                          float *d_param_norms, hipStream_t stream, CallTimer &timer, bool last) {
  switch (norm_type) {
    case DDP_NORM_L2:
      return launch_norm<Tr, DDP_NORM_L2>(t, p, ptrs, partial, d_norms, d_param_norms, stream,
                                          timer, last);
    case DDP_NORM_L1:
      return launch_norm<Tr, DDP_NORM_L1>(t, p, ptrs, partial, d_norms, d_param_norms, stream,
                                          timer, last);
    default:
      return launch_norm<Tr, DDP_NORM_INF>(t, p, ptrs, partial, d_norms, d_param_norms, stream,
                                           timer, last);
  }
}

ddp_status launch_norm_type(int32_t dtype, int32_t norm_type, const PlanTiles &t, int32_t p,
                            const void *const *ptrs, double *partial, float *d_norms,
                            float *d_param_norms, hipStream_t stream, CallTimer &timer,
                            bool last) {
  return dtype == DDP_F32 ? launch_norm_of<F32Traits>(norm_type, t, p, ptrs, partial, d_norms,
                                                      d_param_norms, stream, timer, last)
                          : launch_norm_of<BF16Traits>(norm_type, t, p, ptrs, partial, d_norms,
                                                       d_param_norms, stream, timer, last);
}

template <typename Tr, bool kStaged>
ddp_status launch_fanout(const PlanTiles &t, int32_t p, const void *const *ptrs,
                         const NormSource &source, float max_norm, float eps, hipStream_t stream,
                         CallTimer &timer) {
  const int32_t waves = fanout_waves(p);
  // a launch holds at most 2^32 - 1 work-items along x
  const int64_t blocks = std::min(t.tiles, int64_t(UINT32_MAX) / (64 * waves));
  const bool past_cache = int64_t(p) * t.elems * t.elem_bytes > kCacheBytes;
  auto kernel = clip_fanout_kernel<Tr, kStaged, false>;
  if constexpr (kStaged) {
    if (source.sums > 0) kernel = clip_fanout_kernel<Tr, true, true>;
  }
  return launch(kernel, dim3(static_cast<uint32_t>(blocks)),
                dim3(static_cast<uint32_t>(64 * waves)), stream, timer, true,
                "clip_fanout_kernel launch", t.seg, t.tile_seg, t.map_stride, t.tiles, t.n_params,
                ptrs, p, source, max_norm, eps, past_cache, runs_per_xcd(t, p));
}

template <typename Tr>
ddp_status launch_clip_of(const PlanTiles &t, int32_t p, const void *const *ptrs,
                          const float *d_norms, int32_t n_norms, float max_norm, float eps,
                          bool replicated, hipStream_t stream, CallTimer &timer) {
  if (replicated && p > 1) {
    const NormSource source = {const_cast<float *>(d_norms), nullptr, 0, 0};
    return launch_fanout<Tr, false>(t, p, ptrs, source, max_norm, eps, stream, timer);
  }
  const int64_t groups = norm_groups(t);
  const bool past_cache = int64_t(p) * t.elems * t.elem_bytes > kCacheBytes;
  // Past the caches a full CU of waves, each with a stream in and one out,
  // opens more DRAM rows than pay: GPT-2 small on 8 ranks 1.36 ms, with 2
  // workgroups per CU 1.28, with 4 1.33; tensors that are not whole lines
  // prefer 4 (100 odd bf16 tensors on 4 ranks 0.39 ms, unbounded 0.42, with 2
  // 0.48).
  const size_t lds = past_cache ? residency_lds(t.whole_lines ? 2 : 4) : 0;
  return launch_lds(clip_kernel<Tr>,
                    dim3(static_cast<uint32_t>(ceil_div(groups, kWaves)),
                         static_cast<uint32_t>(p)),
                    dim3(64 * kWaves), lds, stream, timer, true,
                    "clip_kernel launch", t.seg, t.tile_seg, t.map_stride, t.tiles, groups,
                    t.n_params, ptrs, d_norms, n_norms == 1 ? 0 : 1, max_norm, eps, past_cache);
}

ddp_status launch_clip(int32_t dtype, const PlanTiles &t, int32_t p, const void *const *ptrs,
                       const float *d_norms, int32_t n_norms, float max_norm, float eps,
                       bool replicated, hipStream_t stream, CallTimer &timer) {
  return dtype == DDP_F32 ? launch_clip_of<F32Traits>(t, p, ptrs, d_norms, n_norms, max_norm, eps,
                                                      replicated, stream, timer)
                          : launch_clip_of<BF16Traits>(t, p, ptrs, d_norms, n_norms, max_norm,
                                                       eps, replicated, stream, timer);
}

}  // namespace
}  // namespace ddpsim

using namespace ddpsim;

extern "C" ddp_status ddp_grad_norm(const ddp_plan *plan, int32_t p,
                                    const void *const *d_grad_ptrs, int32_t dtype,
                                    int32_t norm_type, float *d_norms, float *d_param_norms,
                                    void *workspace, size_t workspace_bytes,
                                    hipStream_t stream) {
  clear_error();
  CallTimer timer = CallTimer::take();
  const char *what = "ddp_grad_norm";
  PlanTiles t;
  ddp_status s = check_call(what, plan, p, d_grad_ptrs, dtype, &t);
  if (s == DDP_OK) s = check_norm_type(what, norm_type);
  if (s == DDP_OK) {
    s = check_out(what, d_norms, p, d_param_norms, int64_t(p) * t.n_params, workspace,
                  workspace_bytes, ddp_grad_norm_workspace(plan, p));
  }
  if (s == DDP_OK) s = check_uploaded(what, t);
  if (s != DDP_OK) return s;
  return launch_norm_type(dtype, norm_type, t, p, d_grad_ptrs, static_cast<double *>(workspace),
                          d_norms, d_param_norms, stream, timer, true);
}

extern "C" ddp_status ddp_clip_grads(const ddp_plan *plan, int32_t p, void *const *d_grad_ptrs,
                                     int32_t dtype, const float *d_norms, int32_t n_norms,
                                     float max_norm, float eps, int32_t replicated,
                                     hipStream_t stream) {
  clear_error();
  CallTimer timer = CallTimer::take();
  const char *what = "ddp_clip_grads";
  PlanTiles t;
  ddp_status s = check_call(what, plan, p, d_grad_ptrs, dtype, &t);
  if (s == DDP_OK) s = check_out(what, d_norms, n_norms, nullptr, 0, nullptr, 0, 0);
  if (s == DDP_OK) s = check_bound(what, max_norm, eps);
  if (s == DDP_OK) s = check_uploaded(what, t);
  if (s != DDP_OK) return s;
  if (replicated != 0 && replicated != 1) {
    return fail(DDP_EINVAL, "%s: replicated must be 0 or 1", what);
  }
  if (n_norms != 1 && (n_norms != p || replicated)) {
    return fail(DDP_EINVAL, "%s: n_norms=%d: one norm%s", what, n_norms,
                replicated ? " for replicated gradients" : ", or one per rank");
  }
  if (t.tiles == 0) return DDP_OK;
  return launch_clip(dtype, t, p, d_grad_ptrs, d_norms, n_norms, max_norm, eps, replicated != 0,
                     stream, timer);
}

extern "C" ddp_status ddp_allreduce_buckets_norm(const ddp_plan *plan, int32_t first_bucket,
                                                 int32_t n_buckets, int32_t p,
                                                 void *const *d_grad_ptrs, int32_t dtype,
                                                 int32_t avg_mode, const int64_t *tokens,
                                                 int32_t norm_type, void *workspace,
                                                 size_t workspace_bytes, hipStream_t stream,
                                                 ddp_comm_stats *stats) {
  clear_error();
  CallTimer timer = CallTimer::take();
  const char *what = "ddp_allreduce_buckets_norm";
  ddp_status s = check_norm_type(what, norm_type);
  if (s == DDP_OK) {
    s = check_workspace(what, workspace, workspace_bytes, ddp_sync_norm_workspace(plan), nullptr,
                        0, 0);
  }
  if (s != DDP_OK) return s;
  const SyncEpilogue epi = {kSyncNorm, norm_type, static_cast<double *>(workspace), nullptr, 0, 0,
                            false, false};
  return allreduce_buckets(plan, first_bucket, n_buckets, p, d_grad_ptrs, dtype, avg_mode, tokens,
                           stream, stats, DDPSIM_BUCKET_MAX_WORKGROUPS, &epi, &timer);
}

extern "C" ddp_status ddp_grad_norm_finish(const ddp_plan *plan, int32_t norm_type,
                                           float *d_norm, float *d_param_norms, void *workspace,
                                           size_t workspace_bytes, hipStream_t stream) {
  clear_error();
  CallTimer timer = CallTimer::take();
  const char *what = "ddp_grad_norm_finish";
  PlanTiles t;
  if (!plan_tiles(plan, &t)) return fail(DDP_EINVAL, "%s: plan is NULL", what);
  ddp_status s = check_norm_type(what, norm_type);
  if (s == DDP_OK) {
    s = check_out(what, d_norm, 1, d_param_norms, t.n_params, workspace, workspace_bytes,
                  ddp_sync_norm_workspace(plan));
  }
  if (s == DDP_OK) s = check_uploaded(what, t);
  if (s != DDP_OK) return s;
  return launch_tile_finish(t, norm_type, static_cast<double *>(workspace), d_norm,
                            d_param_norms, stream, timer, true);
}

extern "C" ddp_status ddp_allreduce_clip(const ddp_plan *plan, int32_t p,
                                         void *const *d_grad_ptrs, int32_t dtype,
                                         int32_t avg_mode, const int64_t *tokens,
                                         int32_t norm_type, float max_norm, float eps,
                                         float *d_norm, float *d_param_norms, void *workspace,
                                         size_t workspace_bytes, hipStream_t stream,
                                         ddp_comm_stats *stats) {
  clear_error();
  CallTimer timer = CallTimer::take();
  const char *what = "ddp_allreduce_clip";
  PlanTiles t;
  ddp_status s = check_call(what, plan, p, d_grad_ptrs, dtype, &t);
  if (s == DDP_OK) s = check_norm_type(what, norm_type);
  if (s == DDP_OK) s = check_bound(what, max_norm, eps);
  if (s == DDP_OK) {
    s = check_out(what, d_norm, 1, d_param_norms, t.n_params, workspace, workspace_bytes,
                  ddp_sync_norm_workspace(plan));
  }
  if (s == DDP_OK) s = check_uploaded(what, t);
  if (s != DDP_OK) return s;
  if (t.seg_p != p) {
    return fail(DDP_ENOTREADY, "%s: call ddp_plan_upload_segments with p=%d first", what, p);
  }
  Divide div;
  s = make_divide(avg_mode, p, tokens, &div);
  if (s != DDP_OK) return s;
  // The norm needs every average before the first result can be written.
  // The first pass keeps the averages in place of one rank's gradients (two
  // ranks' for bf16) and the second spreads them: (2 p + 2) n or (2 p + 4) n
  // elements moved. Folding the gradients twice instead, 3 p n, was slower at
  // every p from 2 on (GPT-2 small fp32: 0.75 against 0.64 ms at p = 2, 1.88
  // against 1.50 at p = 8; bf16 0.48 against 0.41 at p = 2); a single rank
  // has no sum to keep.
  const bool staged = p > 1;
  const int32_t nb = ddp_plan_num_buckets(plan);
  ddp_comm_stats local;
  if (stats == nullptr) stats = &local;
  *stats = ddp_comm_stats{};
  double *sums = static_cast<double *>(workspace);
  if (p == 1 && div.mode == kNone && t.tiles > 0) {
    // one rank's gradients are their own average
    s = launch_norm_type(dtype, norm_type, t, 1, d_grad_ptrs, sums, d_norm, d_param_norms, stream,
                         timer, false);
    if (s != DDP_OK) return s;
    s = launch_clip(dtype, t, 1, d_grad_ptrs, d_norm, 1, max_norm, eps, false, stream, timer);
  } else if (staged && t.tiles > 0 && small_sync(t.tiles, p, d_param_norms != nullptr)) {
    for (int32_t b = 0; b < nb; ++b) add_ring_stats(p, ddp_plan_bucket_numel(plan, b), stats);
    s = dtype == DDP_F32
            ? launch_small_sync_type<F32Traits>(norm_type, t, p, d_grad_ptrs, div, max_norm, eps,
                                                d_norm, d_param_norms, stream, timer)
            : launch_small_sync_type<BF16Traits>(norm_type, t, p, d_grad_ptrs, div, max_norm,
                                                 eps, d_norm, d_param_norms, stream, timer);
  } else {
    SyncEpilogue epi = {staged ? kStageNorm : kFoldNorm, norm_type, sums, d_norm, max_norm, eps,
                        runs_per_xcd(t, p), int64_t(p) * t.elems * t.elem_bytes <= kCacheBytes};
    if (nb > 0) {
      s = allreduce_buckets(plan, 0, nb, p, d_grad_ptrs, dtype, avg_mode, tokens, stream, stats,
                            DDPSIM_BUCKET_MAX_WORKGROUPS, &epi, &timer, false);
      if (s != DDP_OK) return s;
    }
    NormSource source = {d_norm, sums, 0, norm_type};
    if (staged && t.tiles > 0 && t.tiles <= kInlineTiles && d_param_norms == nullptr) {
      source.sums = static_cast<int32_t>(t.tiles);
    } else {
      s = launch_tile_finish(t, norm_type, sums, d_norm, d_param_norms, stream, timer,
                             t.tiles == 0);
      if (s != DDP_OK || t.tiles == 0) return s;
    }
    if (staged) {
      s = dtype == DDP_F32 ? launch_fanout<F32Traits, true>(t, p, d_grad_ptrs, source, max_norm,
                                                            eps, stream, timer)
                           : launch_fanout<BF16Traits, true>(t, p, d_grad_ptrs, source, max_norm,
                                                             eps, stream, timer);
    } else {
      epi.mode = kSyncScale;
      s = allreduce_buckets(plan, 0, nb, p, d_grad_ptrs, dtype, avg_mode, tokens, stream, nullptr,
                            DDPSIM_BUCKET_MAX_WORKGROUPS, &epi, &timer, true);
    }
  }
  const int64_t moved = staged ? 2 * p + (dtype == DDP_F32 ? 2 : 4) : 3 * p;
  stats->hbm_bytes = moved * t.elems * t.elem_bytes;
  return s;
}
