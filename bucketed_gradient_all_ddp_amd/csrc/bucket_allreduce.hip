// bucket_allreduce.hip -- the bucket's all-reduce done in place on the
// per-parameter gradients: the same bits as ddp_flatten, then
// ring_allreduce_sim on the flat buffers, then ddp_unflatten, in one pass
// over HBM.
//
// The reducer copies every gradient into its slot of the bucket's flat
// buffer, all-reduces the buffer and copies the result back ("PyTorch DDP
// Deep Dive", Part 2 "Step 2: backward" item 1 and "Step 3:
// finalize_backward"). The ring's chunk geometry lives in the bucket's flat
// index space ("Collective Ops From Scratch", "Ring allreduce in two
// passes"). Nothing in that arithmetic needs the flat copy to exist: element
// j of parameter i is element offset_i + j of the bucket, and its ring chunk
// is (offset_i + j) / C. So a workgroup takes a tile of one parameter, folds
// every element across the p ranks' gradients of that parameter in ring
// order starting at the element's chunk, and writes the result back to all
// p ranks. HBM traffic 2 p n eb per bucket instead of 6 p n eb.
//
// A tile inside one chunk folds with one rank order for the whole wave. A
// tile that crosses chunk boundaries (small parameters, small chunks) folds
// per lane: each lane loads the ranks in the order of the chunk of its
// vector's first element, and an element whose chunk starts d ranks later
// skips the first d loads and adds them at the end, which is its own ring
// order. Tiles are therefore whole parameters cut into 64-vector runs, with
// no lanes left idle at chunk ends.
//
// The same pass can also take the norm of the averaged gradient, one partial
// sum per tile, from the fp32 values before they are rounded to the
// gradients' type, and it can scale them by the clip coefficient of a norm
// in device memory (SyncMode). In fp32 the norm costs the all-reduce nothing
// that can be measured: GPT-2 small, 8 ranks, 1.27 to 1.31 ms a launch on the
// boxes where the plain launch takes 1.27 to 1.29; in bf16 2%: two Llama-7B
// layers, 8 ranks, 2.14 ms (6.05 TB/s) where the plain launch takes 2.09. As
// the first pass of an all-reduce with clipping (8 ranks read, one written) it
// runs at 6.1 TB/s, 0.73 ms, and at 6.1 to 6.4 TB/s on two Llama-7B layers in
// bf16 (two written).
#include <algorithm>

#include "bucket_run.hpp"

namespace ddpsim {
int32_t plan_num_buckets(const ddp_plan *plan);
const int32_t *plan_tile_map(const ddp_plan *plan, int64_t *stride);
bool plan_segment_info(const ddp_plan *plan, int32_t b, int32_t *first, int32_t *count,
                       int32_t *tiles, int32_t *tile_first, int64_t *elems,
                       const void **table, int32_t *seg_p, int32_t *n_params,
                       int32_t *elem_bytes);

namespace {

// One tile of the plan's numbering; the tile map names the parameter
// descriptor (index into seg) each tile belongs to.
template <typename Tr, int VPT, int RB, bool kNT>
__device__ __forceinline__ void bucket_tile(const SegDesc *__restrict__ seg,
                                            const int32_t *__restrict__ tile_seg,
                                            int64_t map_stride, int32_t tile, int32_t n_params,
                                            const void *const *__restrict__ grads, int32_t p,
                                            const Divide &div) {
  constexpr int V = Tr::kVec;
  constexpr int64_t kElemBytes = sizeof(typename Tr::elem);
  const SegDesc d = seg[tile_seg[tile_map_index(tile, map_stride)]];
  const int32_t t = tile - d.tile_begin;
  const int tid = static_cast<int>(threadIdx.x);
  constexpr int kThr = kBucketThreads;
  constexpr int64_t kTile = int64_t(kThr) * VPT * V;

  // The vector path needs every rank's copy of this parameter to sit at the
  // same offset from a 16-byte boundary.
  // lane r loads rank r's address (p <= 64 = the wave size)
  const int my_lane = tid & 63;
  const uint64_t mine =
      my_lane < p
          ? reinterpret_cast<uint64_t>(grads[static_cast<int64_t>(my_lane) * n_params + d.param])
          : 0;
  const uintptr_t phase =
      __builtin_amdgcn_readlane(static_cast<uint32_t>(mine), 0) % static_cast<uint32_t>(kVecBytes);
  const bool same =
      phase % kElemBytes == 0 && __all(my_lane >= p || mine % kVecBytes == phase);

  if (!same) {
    const GradPtrs at{grads, n_params, d.param, 0};
    const int64_t j0 = static_cast<int64_t>(t) * kTile;
    const int64_t j1 = std::min(j0 + kTile, d.len);
    for (int64_t j = j0 + tid; j < j1; j += kThr) {
      const float y = apply_divide(fold_scalar<Tr>(at, p, chunk_of(d.offset, j, d.chunk), j), div);
      for (int32_t r = 0; r < p; ++r) Tr::store1(at(r), j, y);
    }
    return;
  }

  // Shifted coordinates: index J = j + m addresses element j of the
  // parameter from a base moved back by m elements, which is 16-byte
  // aligned for every rank.
  const int64_t m = static_cast<int64_t>(phase) / kElemBytes;
  const GradPtrs at{grads, n_params, d.param, m * kElemBytes};
  const ChunkSpan k = make_span(m, d.len + m, V);

  if (t == 0 && tid >= kThr - 2 * (V - 1)) {
    const int lane = tid - (kThr - 2 * (V - 1));
    const bool head = lane < V - 1;
    const int64_t J = head ? k.s + lane : k.tail_begin + (lane - (V - 1));
    if (J < (head ? k.head_end : k.e)) {
      const float y =
          apply_divide(fold_scalar<Tr>(at, p, chunk_of(d.offset, J - m, d.chunk), J), div);
      for (int32_t r = 0; r < p; ++r) Tr::store1(at(r), J, y);
    }
  }

  const int64_t nv = (k.ve - k.vs) / V;
  const int64_t base = static_cast<int64_t>(t) * (kThr * VPT);
  if (base >= nv) return;
  int64_t vi[VPT];
  bool ok[VPT];
#pragma unroll
  for (int u = 0; u < VPT; ++u) {
    const int64_t jj = base + u * kThr + tid;
    ok[u] = jj < nv;
    vi[u] = k.vs / V + jj;
  }
  const uint64_t shifted = mine - static_cast<uint64_t>(m * kElemBytes);
  const LanePtrs lat{shifted};
  // chunks of the tile's first and last element (wave-uniform)
  const int64_t last_v = k.vs / V + std::min(base + int64_t(kThr) * VPT, nv) - 1;
  const int32_t c_first = chunk_of(d.offset, k.vs + base * V - m, d.chunk);
  const int32_t c_last = chunk_of(d.offset, last_v * V + V - 1 - m, d.chunk);
  float acc[VPT][V];
  if (c_first == c_last) {
    fold_vectors<Tr, VPT, RB, kNT>(lat, p, c_first, vi, ok, acc);
  } else {
#pragma unroll
    for (int u = 0; u < VPT; ++u) {
      // a lane past the body computes with the last vector (never stored)
      const int64_t v = ok[u] ? vi[u] : last_v;
      const int64_t j0 = v * V - m;
      const int32_t c0 = chunk_of(d.offset, j0, d.chunk);
      int32_t dist[V];
      int64_t next = (static_cast<int64_t>(c0) + 1) * d.chunk - d.offset;  // next chunk's first j
      int32_t dd = 0;
#pragma unroll
      for (int e = 0; e < V; ++e) {
        while (j0 + e >= next) {
          ++dd;
          next += d.chunk;
        }
        dist[e] = dd;
      }
      fold_vector_per_lane<Tr, RB, kNT>(shifted, p, c0, dist, vi[u], ok[u], acc[u]);
    }
  }
  uint4 y[VPT];
#pragma unroll
  for (int u = 0; u < VPT; ++u) {
#pragma unroll
    for (int e = 0; e < V; ++e) acc[u][e] = apply_divide(acc[u][e], div);
    y[u] = Tr::narrow(acc[u]);
  }
  const int32_t rot = store_rotation(p, tile);
  for (int32_t r = 0; r < p; ++r) {
    void *dst = lat(ring_rank(rot, r, p));
#pragma unroll
    for (int u = 0; u < VPT; ++u) {
      if (ok[u]) store_vec<kNT>(dst, vi[u], y[u]);
    }
  }
}

// Workgroup w handles tiles tile_base + w, + gridDim.x, ... of the n_tiles
// of a run of buckets: one tile each when the grid covers them all (the
// default), several when the caller capped the number of workgroups so the
// all-reduce leaves compute units to kernels running beside it.
template <typename Tr, int VPT, int RB, bool kNT>
__global__ __launch_bounds__(kBucketThreads) void bucket_allreduce_kernel(
    const SegDesc *__restrict__ seg, const int32_t *__restrict__ tile_seg, int64_t map_stride,
    int32_t tile_base, int32_t n_tiles, int32_t n_params,
    const void *const *__restrict__ grads, int32_t p, Divide div) {
  for (int32_t w = static_cast<int32_t>(blockIdx.x); w < n_tiles;
       w += static_cast<int32_t>(gridDim.x)) {
    bucket_tile<Tr, VPT, RB, kNT>(seg, tile_seg, map_stride, tile_base + w, n_params, grads, p,
                                  div);
  }
}

// The all-reduce's tiles with an epilogue, G consecutive ones per wave: each
// wave leaves its tiles' part of the norm in partial (the sum of a run of one
// parameter's tiles at its first tile, zeros at the others), or scales by the
// coefficient.
template <typename Tr, int G, int RB, int kMode, int NT, bool kNT>
__global__ __launch_bounds__(64) void bucket_epilogue_kernel(
    const SegDesc *__restrict__ seg, const int32_t *__restrict__ tile_seg, int64_t map_stride,
    int32_t tile_base, int32_t n_tiles, int32_t n_params,
    const void *const *__restrict__ grads, int32_t p, Divide div, double *__restrict__ partial,
    const float *__restrict__ norm, float max_norm, float eps, bool runs) {
  static_assert(kBucketThreads == 64 && kBucketVpt == 1, "a tile is one vector per lane");
  const int32_t groups = (n_tiles + G - 1) / G;
  for (int32_t w = static_cast<int32_t>(blockIdx.x); w < groups;
       w += static_cast<int32_t>(gridDim.x)) {
    const int32_t g = runs ? static_cast<int32_t>(xcd_run<kXcdRun>(w, groups)) : w;
    int32_t tile = tile_base + g * G;
    const int32_t end = std::min(tile + G, tile_base + n_tiles);
    int32_t s = tile_seg[tile_map_index(tile, map_stride)];
    do {
      const SegDesc d = seg[s++];
      constexpr int64_t kTile = 64 * Tr::kVec;
      const int64_t t = tile - d.tile_begin;
      const int64_t t1 = std::min((d.len + kTile - 1) / kTile, t + (end - tile));
      Epilogue<kMode, NT> epi;
      if constexpr (kMode == kSyncScale) epi.scale = clip_coefficient(*norm, max_norm, eps);
      bucket_run<Tr, G, RB, kNT>(d, t, t1, tile, n_params, grads, p, div, epi);
      const int32_t count = static_cast<int32_t>(t1 - t);
      if constexpr (kMode != kSyncScale) {
        join_wave(epi.sum);
        if (static_cast<int32_t>(threadIdx.x) < count) {
          partial[tile + threadIdx.x] = threadIdx.x == 0 ? epi.sum.part() : 0.0;
        }
      }
      tile += count;
    } while (tile < end);
  }
}

// Tiles per wave of an epilogue launch and rank loads in flight of each.
// With few ranks a tile is little work next to fetching its descriptor and
// addresses, so that a wave takes as many as keep about 8 loads in flight,
// if they leave waves enough and its parameters are not smaller. First pass
// on GPT-2 small fp32, 1 / 2 / 4 tiles per wave: 0.34 / 0.19 / 0.12 ms for
// one rank, 0.41 / 0.28 / 0.23 for 2, 0.45 / 0.33 / 0.35 for 3, 0.47 / 0.41 /
// 0.42 for 4, 0.49 / 0.51 / 0.53 for 5.
// With more than 8 ranks and tiles for few waves, one wave's folds follow one
// another with the chip nearly empty: 32 loads in flight instead of 8. All-reduce
// with norm, fp32, us of 32 / 8 loads:
//   tiles         500          1000          2000          4000
//   16 ranks   10.7 / 11.3   11.8 / 11.8   17.0 / 17.1   32.9 / 32.2
//   32 ranks   14.8 / 16.8   19.4 / 20.6   33.0 / 32.3   65.1 / 64.9
//   64 ranks   25.6 / 30.0   36.6 / 38.4   65.9 / 65.5    130 / 131
// and with clipping much the same (both passes, 4000 tiles of 16 ranks: 38.6 /
// 35.1). The registers of 32 loads leave 2 waves per SIMD, those of 8 loads 5
// (bf16 4).
constexpr int64_t kFullTiles = 16384;  // waves that fill the chip twice over
constexpr int64_t kFewTiles = 1536;
struct WaveShape {
  int32_t tiles, loads;
};
WaveShape wave_shape(int32_t p, int64_t tiles, int64_t params) {
  int32_t g = p <= 2 ? 4 : p <= 4 ? 2 : 1;
  while (g > 1 && (tiles < g * kFullTiles || tiles < g * params)) g /= 2;
  if (p > 8 && tiles < kFewTiles) return {1, 32};
  return {g, 8 / g};
}

// The arguments of one bucket launch, and its kernel by type, mode and norm.
struct BucketLaunch {
  const SegDesc *seg;
  const int32_t *tile_seg;
  int64_t map_stride;
  int32_t tile0, tiles, n_params;
  const void *const *grads;
  int32_t p;
  Divide div;
  dim3 grid;
  size_t lds;
  hipStream_t stream;
  WaveShape shape;
};

template <typename Tr, int G, int RB, int kMode, int NT, bool kNT = true>
ddp_status launch_epilogue(const BucketLaunch &b, const SyncEpilogue &e, CallTimer &timer,
                           bool last) {
  return launch_lds(bucket_epilogue_kernel<Tr, G, RB, kMode, NT, kNT>, b.grid, dim3(64), b.lds,
                    b.stream, timer, last, "bucket_epilogue_kernel launch", b.seg, b.tile_seg,
                    b.map_stride, b.tile0, b.tiles, b.n_params, b.grads, b.p, b.div, e.partial,
                    e.norm, e.max_norm, e.eps, e.runs);
}

template <typename Tr, int G, int RB, int kMode, bool kNT = true>
ddp_status launch_norm_type(const BucketLaunch &b, const SyncEpilogue &e, CallTimer &timer,
                            bool last) {
  switch (e.norm_type) {
    case DDP_NORM_L2: return launch_epilogue<Tr, G, RB, kMode, DDP_NORM_L2, kNT>(b, e, timer, last);
    case DDP_NORM_L1: return launch_epilogue<Tr, G, RB, kMode, DDP_NORM_L1, kNT>(b, e, timer, last);
    default: return launch_epilogue<Tr, G, RB, kMode, DDP_NORM_INF, kNT>(b, e, timer, last);
  }
}

// kFoldNorm and kSyncScale are the two passes of a single rank.
template <typename Tr, int G, int RB>
ddp_status launch_mode(const BucketLaunch &b, const SyncEpilogue &e, CallTimer &timer,
                       bool last) {
  // one rank's gradients are their own average: nothing to write
  const bool stays = b.p == 1 && b.div.mode == kNone;
  if (e.mode == kSyncNorm && !stays) {
    return launch_norm_type<Tr, G, RB, kSyncNorm>(b, e, timer, last);
  }
  if (e.mode == kStageNorm) {
    // Ordinary accesses where the gradients fit the cache: 36 us a call
    // against 39 for 64 MB on 8 ranks (bf16 39 against 43), 17.5 against 18.3
    // for 16 MB.
    if (RB == 32 || e.cached) {
      return launch_norm_type<Tr, G, RB, kStageNorm, false>(b, e, timer, last);
    }
    if constexpr (RB != 32) return launch_norm_type<Tr, G, RB, kStageNorm>(b, e, timer, last);
  }
  if constexpr (RB != 32) {  // many loads in flight are for many ranks
    if (e.mode != kSyncScale) return launch_norm_type<Tr, G, RB, kFoldNorm>(b, e, timer, last);
    return launch_epilogue<Tr, G, RB, kSyncScale, DDP_NORM_L2>(b, e, timer, last);
  }
  return fail(DDP_EINVAL, "no such launch for %d ranks", b.p);
}

template <typename Tr>
ddp_status launch_bucket(const BucketLaunch &b, const SyncEpilogue *e, CallTimer &timer,
                         bool last) {
  if (e == nullptr) {
    return launch_lds(bucket_allreduce_kernel<Tr, kBucketVpt, kBucketRb, kBucketNt>, b.grid,
                      dim3(kBucketThreads), b.lds, b.stream, timer, last,
                      "bucket_allreduce_kernel launch", b.seg, b.tile_seg, b.map_stride, b.tile0,
                      b.tiles, b.n_params, b.grads, b.p, b.div);
  }
  if (b.shape.loads == 32) return launch_mode<Tr, 1, 32>(b, *e, timer, last);
  if (b.shape.tiles == 4) return launch_mode<Tr, 4, 2>(b, *e, timer, last);
  if (b.shape.tiles == 2) return launch_mode<Tr, 2, 4>(b, *e, timer, last);
  return launch_mode<Tr, 1, 8>(b, *e, timer, last);
}

}  // namespace
}  // namespace ddpsim

using namespace ddpsim;

namespace ddpsim {

ddp_status allreduce_buckets(const ddp_plan *plan, int32_t first_bucket, int32_t n_buckets,
                             int32_t p, void *const *d_grad_ptrs, int32_t dtype,
                             int32_t avg_mode, const int64_t *tokens, hipStream_t stream,
                             ddp_comm_stats *stats, int32_t max_workgroups,
                             const SyncEpilogue *epi, CallTimer *call_timer, bool last) {
  clear_error();
  CallTimer own_timer = call_timer == nullptr ? CallTimer::take() : CallTimer();
  CallTimer &timer = call_timer == nullptr ? own_timer : *call_timer;
  const char *what = "ddp_allreduce_buckets";
  if (plan == nullptr) return fail(DDP_EINVAL, "%s: plan is NULL", what);
  const int32_t nbk = plan_num_buckets(plan);
  if (n_buckets < 1 || first_bucket < 0 || first_bucket >= nbk ||
      n_buckets > nbk - first_bucket) {
    return fail(DDP_ERANGE, "%s: buckets [%d, %d) outside [0, %d)", what, first_bucket,
                first_bucket + n_buckets, nbk);
  }
  ddp_status s = check_p(p, what);
  if (s != DDP_OK) return s;
  int32_t seg0 = 0, nseg = 0, tiles = 0, tile0 = 0, seg_p = 0, n_params = 0, eb_plan = 0;
  int64_t elems = 0;
  const void *table = nullptr;
  int64_t C_sum = 0;
  for (int32_t b = first_bucket; b < first_bucket + n_buckets; ++b) {
    int32_t f, c, t, tf;
    int64_t e;
    plan_segment_info(plan, b, &f, &c, &t, &tf, &e, &table, &seg_p, &n_params, &eb_plan);
    if (seg_p != p) {
      return fail(DDP_ENOTREADY, "%s: call ddp_plan_upload_segments with p=%d first", what, p);
    }
    if (b == first_bucket) {
      seg0 = f;
      tile0 = tf;
    }
    nseg += c;
    tiles += t;
    elems += e;
    C_sum += e > 0 ? ceil_div(e, p) : 0;
  }
  const int eb = elem_bytes_of(dtype);
  if (eb == 0) return fail(DDP_EINVAL, "%s: unknown dtype %d", what, dtype);
  if (eb != eb_plan) {
    return fail(DDP_EINVAL, "%s: dtype has %d-byte elements, the plan %d", what, eb, eb_plan);
  }
  if (tiles > 0 && d_grad_ptrs == nullptr) {
    return fail(DDP_EINVAL, "%s: gradient pointer table is NULL", what);
  }
  Divide div;
  s = make_divide(avg_mode, p, tokens, &div);
  if (s != DDP_OK) return s;
  if (stats != nullptr) {
    // one ring all-reduce per bucket
    stats->steps = 2 * int64_t(p - 1) * n_buckets;
    stats->messages = 2 * int64_t(p) * (p - 1) * n_buckets;
    stats->bytes_sent_per_rank = 2 * int64_t(p - 1) * C_sum * 4;
    stats->bytes_recv_per_rank = stats->bytes_sent_per_rank;
    stats->total_bytes = 2 * int64_t(p) * (p - 1) * C_sum * 4;
    stats->hbm_bytes = 2 * int64_t(p) * elems * eb;
  }
  if (tiles == 0) return DDP_OK;
  (void)seg0;
  const SegDesc *seg = static_cast<const SegDesc *>(table);
  int64_t map_stride = 0;
  const int32_t *tile_seg = plan_tile_map(plan, &map_stride);
  const void *const *grads = d_grad_ptrs;
  const WaveShape shape = epi == nullptr ? WaveShape{1, kBucketRb} : wave_shape(p, tiles, nseg);
  const int32_t units = (tiles - 1) / shape.tiles + 1;
  // a launch holds at most 2^32 - 1 work-items along x
  int32_t blocks = std::min(units, static_cast<int32_t>(UINT32_MAX / kBucketThreads));
  if (max_workgroups > 0) blocks = std::min(blocks, max_workgroups);
  const dim3 grid(static_cast<uint32_t>(blocks));
  // Each workgroup keeps 2p streams of 1 KiB in flight (p loads, p
  // stores); a CU full of them (32 one-wave workgroups) puts more streams on
  // every HBM channel than it keeps rows open. Bounding residency at 11 per
  // CU raised the GPT-2 p=8 launch from 5.76 to 6.05 TB/s and the Llama bf16
  // buckets by 3-4%; 6 per CU starved the channels (5.2). A pass that stores
  // to one or two ranks or none has half as many: bounded at 11 it read the 8
  // ranks' GPT-2 gradients at 5.3 TB/s, at 14, 18 and 24 per CU at 6.5, 6.9
  // and 6.8 (Llama layers in bf16 4.7, and 5.9, 6.3, 6.3). The kernels'
  // registers bound it too: one tile a wave at 20 per CU in fp32 and 16 in
  // bf16, four tiles a wave at 20 and 12, 32 loads in flight at 8.
  const bool reads = epi != nullptr && (epi->mode == kFoldNorm || epi->mode == kStageNorm);
  const size_t lds = residency_lds(
      fold_residency(reads ? DDPSIM_FOLD_WGS_PER_CU : DDPSIM_BUCKET_WGS_PER_CU, p * shape.tiles));
  const BucketLaunch launch = {seg,   tile_seg, map_stride, tile0, tiles,  n_params, grads,
                               p,     div,      grid,       lds,   stream, shape};
  return dtype == DDP_F32 ? launch_bucket<F32Traits>(launch, epi, timer, last)
                          : launch_bucket<BF16Traits>(launch, epi, timer, last);
}

}  // namespace ddpsim

extern "C" ddp_status ddp_allreduce_buckets(const ddp_plan *plan, int32_t first_bucket,
                                            int32_t n_buckets, int32_t p,
                                            void *const *d_grad_ptrs, int32_t dtype,
                                            int32_t avg_mode, const int64_t *tokens,
                                            hipStream_t stream, ddp_comm_stats *stats) {
  return allreduce_buckets(plan, first_bucket, n_buckets, p, d_grad_ptrs, dtype, avg_mode,
                           tokens, stream, stats, DDPSIM_BUCKET_MAX_WORKGROUPS);
}

extern "C" ddp_status ddp_allreduce_bucket(const ddp_plan *plan, int32_t bucket, int32_t p,
                                           void *const *d_grad_ptrs, int32_t dtype,
                                           int32_t avg_mode, const int64_t *tokens,
                                           hipStream_t stream, ddp_comm_stats *stats) {
  if (plan != nullptr && (bucket < 0 || bucket >= plan_num_buckets(plan))) {
    clear_error();
    CallTimer::take();
    return fail(DDP_ERANGE, "ddp_allreduce_bucket: bucket %d out of range", bucket);
  }
  return ddp_allreduce_buckets(plan, bucket, 1, p, d_grad_ptrs, dtype, avg_mode, tokens,
                               stream, stats);
}
