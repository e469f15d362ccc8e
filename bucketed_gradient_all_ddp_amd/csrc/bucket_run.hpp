// bucket_run.hpp -- a wave's tiles of the in-place bucket all-reduce: the fold
// of elements whose ring chunks differ from lane to lane, and the fold of a
// run of tiles with what happens to the averages (the norm's sums, the clip
// coefficient, staging) on the way to the ranks.
#pragma once

#include <algorithm>

#include "fold.hpp"
#include "norm.hpp"

namespace ddpsim {
namespace {

// Element j of a parameter at bucket offset `off` is in ring chunk
// (off + j) / C; j may run past the parameter by a few elements (a clamped
// lane), which only moves the chunk of results that are never stored.
__device__ __forceinline__ int32_t chunk_of(int64_t off, int64_t j, int64_t C) {
  return static_cast<int32_t>((off + j) / C);
}

// The fold of one lane's vectors when the ranks' order differs between
// lanes: lane-held rank addresses (lane r holds rank r's, moved back by the
// alignment shift) are fetched per lane with a cross-lane read. For vector
// u, c0 is the chunk of its first element and dist[e] how many chunks later
// element e's chunk starts (0..V-1; it is below p because every chunk index
// is). Loads run in the order c0, c0+1, ...; element e adds load t only from
// t = dist[e] on, then loads 0..dist[e]-1 after the last one, so it sums
// ranks c0+dist[e], ..., c0+dist[e]+p-1 (mod p) left to right: its own
// ring order.
template <typename Tr, int RB, bool kNT>
__device__ __forceinline__ void fold_vector_per_lane(uint64_t mine, int32_t p, int32_t c0,
                                                     const int32_t (&dist)[Tr::kVec],
                                                     int64_t vi, bool ok,
                                                     float (&acc)[Tr::kVec]) {
  constexpr int V = Tr::kVec;
  static_assert(RB >= V - 1, "the first batch must hold the loads added last");
#pragma unroll
  for (int e = 0; e < V; ++e) acc[e] = -0.0f;
  uint4 keep[V > 1 ? V - 1 : 1];
  const uint32_t lo = static_cast<uint32_t>(mine);
  const uint32_t hi = static_cast<uint32_t>(mine >> 32);
  for (int32_t s0 = 0; s0 < p; s0 += RB) {
    uint4 x[RB];
#pragma unroll
    for (int j = 0; j < RB; ++j) {
      const bool live = s0 + j < p;  // wave-uniform
      x[j] = make_uint4(0, 0, 0, 0);
      if (live) {
        const int32_t r = ring_rank(c0, s0 + j, p);
        // every lane takes part in the cross-lane reads (no divergence here)
        const uint32_t alo = static_cast<uint32_t>(__shfl(static_cast<int>(lo), r, 64));
        const uint32_t ahi = static_cast<uint32_t>(__shfl(static_cast<int>(hi), r, 64));
        const void *src =
            reinterpret_cast<const void *>((static_cast<uint64_t>(ahi) << 32) | alo);
        if (ok) x[j] = load_vec<kNT>(src, vi);
      }
    }
    if (s0 == 0) {
#pragma unroll
      for (int j = 0; j < V - 1; ++j) keep[j] = x[j];
    }
#pragma unroll
    for (int j = 0; j < RB; ++j) {
      const int32_t t = s0 + j;
      if (t < p) {
        float w[V];
        Tr::widen(x[j], w);
#pragma unroll
        for (int e = 0; e < V; ++e) {
          if (t >= dist[e]) acc[e] = acc[e] + w[e];
        }
      }
    }
  }
#pragma unroll
  for (int j = 0; j < V - 1; ++j) {
    if (j < p) {
      float w[V];
      Tr::widen(keep[j], w);
#pragma unroll
      for (int e = 0; e < V; ++e) {
        if (j < dist[e]) acc[e] = acc[e] + w[e];
      }
    }
  }
}

// The elements before and after a parameter's whole vectors (V - 1 of them at
// most on either side) belong to its first tile: one each for the wave's last
// lanes.
struct OddElement {
  int64_t at;  // index from the aligned address
  bool here;   // this lane has one
};
__device__ __forceinline__ OddElement odd_element(const ChunkSpan &k, int64_t t, int lane, int V) {
  const int i = lane - (64 - 2 * (V - 1));
  if (t != 0 || i < 0) return {0, false};
  const bool head = i < V - 1;
  const int64_t at = head ? k.s + i : k.tail_begin + (i - (V - 1));
  return {at, at < (head ? k.head_end : k.e)};
}

// The ring-order fold of one element per lane, each lane from its own chunk,
// with the ranks' addresses held by the lanes (every lane takes part). The
// loads have no condition and stay as loaded until their additions: a test or
// a conversion beside each load would wait for it before the next.
template <typename Tr>
__device__ __forceinline__ float fold_lane_element(uint64_t mine, int32_t p, int32_t first,
                                                   int64_t i) {
  constexpr int kBatch = 32;
  const int lo = static_cast<int>(static_cast<uint32_t>(mine));
  const int hi = static_cast<int>(static_cast<uint32_t>(mine >> 32));
  float acc = -0.0f;
  for (int32_t s0 = 0; s0 < p; s0 += kBatch) {
    typename Tr::elem x[kBatch];
#pragma unroll
    for (int j = 0; j < kBatch; ++j) {
      const int32_t r = ring_rank(first, std::min(s0 + j, p - 1), p);
      const uint32_t alo = static_cast<uint32_t>(__shfl(lo, r, 64));
      const uint32_t ahi = static_cast<uint32_t>(__shfl(hi, r, 64));
      const void *src = reinterpret_cast<const void *>((static_cast<uint64_t>(ahi) << 32) | alo);
      x[j] = global_ptr<typename Tr::elem>(src)[i];
    }
#pragma unroll
    for (int j = 0; j < kBatch; ++j) {
      if (s0 + j < p) acc = acc + Tr::widen1(x[j]);
    }
  }
  return acc;
}

// What becomes of a finished fp32 value on its way to the ranks: kMode as
// SyncMode, `sum` this lane's part of the norm, `scale` the clip coefficient.
template <int kMode, int NT>
struct Epilogue {
  static constexpr bool kNorm = kMode != kSyncScale;
  static constexpr bool kSpread = kMode == kSyncNorm || kMode == kSyncScale;  // to every rank
  static constexpr bool kStage = kMode == kStageNorm;
  NormSum<NT> sum;
  float scale = 1.0f;
  __device__ __forceinline__ float operator()(float y) {
    if constexpr (kNorm) sum.add(y);
    if constexpr (kMode == kSyncScale) y = y * scale;
    return y;
  }
  // One element to where it goes, by the lanes that have one (`here`).
  template <typename Tr, typename Ptrs>
  __device__ __forceinline__ void store1(const Ptrs &at, int32_t p, int32_t tile, int64_t i,
                                         float y, bool here) const {
    if constexpr (kStage) {
      const int32_t a = stage_rank(p, tile);
      void *hi = at(a), *lo = at(ring_rank(a, 1, p));
      if (here) Tr::stage1(hi, lo, i, y);
    }
    for (int32_t r = 0; kSpread && r < p; ++r) {
      void *dst = at(r);
      if (here) Tr::store1(dst, i, y);
    }
  }
};

// bucket_tile for up to G consecutive tiles of one parameter, [t, t1) of its
// own, the first of them tile `tile` of the plan, with an epilogue. One fetch
// of the addresses serves them all, and G * RB loads are in flight.
// kNT: accesses that bypass the caches.
template <typename Tr, int G, int RB, bool kNT, typename Epi>
__device__ __forceinline__ void bucket_run(const SegDesc &d, int64_t t, int64_t t1, int32_t tile,
                                           int32_t n_params,
                                           const void *const *__restrict__ grads, int32_t p,
                                           const Divide &div, Epi &epi) {
  constexpr int V = Tr::kVec;
  constexpr int64_t kElemBytes = sizeof(typename Tr::elem);
  constexpr int64_t kTile = 64 * V;
  const int lane = static_cast<int>(threadIdx.x) & 63;
  const uint64_t mine =
      lane < p ? reinterpret_cast<uint64_t>(grads[static_cast<int64_t>(lane) * n_params + d.param])
               : 0;
  const uint64_t phase = __builtin_amdgcn_readlane(static_cast<uint32_t>(mine), 0) %
                         static_cast<uint32_t>(kVecBytes);
  if (!__all(lane >= p || mine % kVecBytes == phase)) {
    const GradPtrs at{grads, n_params, d.param, 0};
    const int64_t j1 = std::min(t1 * kTile, d.len);
    for (int64_t j = t * kTile + lane; j < j1; j += 64) {
      const float y =
          epi(apply_divide(fold_scalar<Tr>(at, p, chunk_of(d.offset, j, d.chunk), j), div));
      epi.template store1<Tr>(at, p, tile + static_cast<int32_t>(j / kTile - t), j, y, true);
    }
    return;
  }
  // indices from the aligned address m elements below each rank's base
  const int64_t m = static_cast<int64_t>(phase) / kElemBytes;
  const ChunkSpan k = make_span(m, d.len + m, V);
  const uint64_t shifted = mine - static_cast<uint64_t>(m * kElemBytes);
  const LanePtrs lat{shifted};
  const OddElement odd = odd_element(k, t, lane, V);
  if (__any(odd.here)) {
    // a lane without one folds the parameter's first element
    const int64_t i = odd.here ? odd.at : k.s;
    const float f = fold_lane_element<Tr>(shifted, p, chunk_of(d.offset, i - m, d.chunk), i);
    float y = apply_divide(f, div);
    if (odd.here) y = epi(y);
    epi.template store1<Tr>(lat, p, tile, i, y, odd.here);
  }
  const int64_t v0 = k.vs / V + t * 64;
  const int64_t v1 = std::min(k.ve / V, k.vs / V + t1 * 64);
  if (v0 >= v1) return;
  int64_t vi[G];
  bool ok[G];
#pragma unroll
  for (int u = 0; u < G; ++u) {
    vi[u] = v0 + u * 64 + lane;
    ok[u] = vi[u] < v1;
  }
  const int32_t c_first = chunk_of(d.offset, v0 * V - m, d.chunk);
  const int32_t c_last = chunk_of(d.offset, v1 * V - 1 - m, d.chunk);
  float acc[G][V];
  if (c_first == c_last) {
    fold_vectors<Tr, G, RB, kNT>(lat, p, c_first, vi, ok, acc);
  } else {
#pragma unroll
    for (int u = 0; u < G; ++u) {
      // a lane past the body computes with the last vector (never stored)
      const int64_t j0 = (ok[u] ? vi[u] : v1 - 1) * V - m;
      const int32_t c0 = chunk_of(d.offset, j0, d.chunk);
      int32_t dist[V];
      int64_t next = (static_cast<int64_t>(c0) + 1) * d.chunk - d.offset;
      int32_t dd = 0;
#pragma unroll
      for (int e = 0; e < V; ++e) {
        while (j0 + e >= next) {
          ++dd;
          next += d.chunk;
        }
        dist[e] = dd;
      }
      fold_vector_per_lane<Tr, (RB > 8 ? RB : 8), kNT>(shifted, p, c0, dist, vi[u], ok[u], acc[u]);
    }
  }
#pragma unroll
  for (int u = 0; u < G; ++u) {
#pragma unroll
    for (int e = 0; e < V; ++e) {
      const float v = apply_divide(acc[u][e], div);
      acc[u][e] = ok[u] ? epi(v) : v;
    }
  }
  if constexpr (Epi::kStage) {
#pragma unroll
    for (int u = 0; u < G; ++u) {
      const int32_t a = stage_rank(p, tile + u);
      uint4 hi, lo;
      Tr::split(acc[u], hi, lo);
      // past the caches: 0.73 ms for GPT-2 small on 8 ranks, 0.83 with
      // ordinary stores
      if (ok[u]) {
        store_vec<kNT>(lat(a), vi[u], hi);
        if constexpr (Tr::kStageRanks == 2) store_vec<kNT>(lat(ring_rank(a, 1, p)), vi[u], lo);
      }
    }
  }
  if constexpr (Epi::kSpread) {
    uint4 y[G];
#pragma unroll
    for (int u = 0; u < G; ++u) y[u] = Tr::narrow(acc[u]);
    const int32_t rot = store_rotation(p, tile);
    for (int32_t r = 0; r < p; ++r) {
      void *dst = lat(ring_rank(rot, r, p));
#pragma unroll
      for (int u = 0; u < G; ++u) {
        if (ok[u]) store_vec<kNT>(dst, vi[u], y[u]);
      }
    }
  }
}

// One source, p destinations: a tile's values are read from rank 0 (kStaged
// false: replicated gradients) or from where kStageNorm left them, scaled, and
// written to the ranks at ring positions [k0, k1) of the tile's rotated order.
// Several waves may share a tile (kBarrier): the source is among the
// destinations, so all of them have loaded before any stores. Ranks whose
// copies of a parameter sit at different offsets from a 16-byte boundary take
// elements.
//
// Tiles that start on a cache line are stored past the caches when the
// gradients outgrow them (`stream`): GPT-2 small on 8 ranks 0.72 ms against
// 0.81 with ordinary stores. A tile that starts inside a line leaves lines to
// two workgroups, whose halves an L2 has to put together: ordinary stores,
// and neighbouring tiles on one XCD (runs_per_xcd), take 0.94 ms instead of
// 1.07 for 300 odd tensors of that size, and 0.13 instead of 0.21 for 300 on
// 64 ranks. One stream in and eight out runs at 5.9 to 6.0 TB/s, bf16 (two in)
// at 5.4 to 5.6, where the fan-out copy reaches 6.4 to 6.6; what holds it is
// not shown by a counter. On fp32 bounding residency slowed it (0.96 ms at 8
// workgroups per CU), and so did groups of 2 and 4 tiles a wave (0.76, 0.77)
// and a grid-stride loop that fetches the next tiles ahead (0.98). With 2 or 8
// destinations a wave instead of 4 it took 0.97 and 0.77.
template <typename Tr, bool kStaged, bool kBarrier>
__device__ __forceinline__ void spread_tile(const SegDesc &d, int64_t tile, int32_t n_params,
                                            const void *const *__restrict__ ptrs, int32_t p,
                                            int32_t k0, int32_t k1, float c, bool stream) {
  constexpr int V = Tr::kVec;
  constexpr int64_t kElemBytes = sizeof(typename Tr::elem);
  constexpr int64_t kTile = 64 * V;
  const int lane = static_cast<int>(threadIdx.x) & 63;
  const int64_t t = tile - d.tile_begin;
  const int32_t a = kStaged ? stage_rank(p, static_cast<int32_t>(tile)) : 0;
  const int32_t b = ring_rank(a, 1, p);
  const int32_t rot = store_rotation(p, static_cast<uint32_t>(tile));
  const uint64_t mine =
      lane < p ? reinterpret_cast<uint64_t>(ptrs[static_cast<int64_t>(lane) * n_params + d.param])
               : 0;
  const uint64_t phase = __builtin_amdgcn_readlane(static_cast<uint32_t>(mine), 0) %
                         static_cast<uint32_t>(kVecBytes);
  const bool same = __all(lane >= p || mine % kVecBytes == phase);
  const int64_t m = same ? static_cast<int64_t>(phase) / kElemBytes : 0;
  const GradPtrs at{ptrs, n_params, d.param, m * kElemBytes};
  const LanePtrs lat{mine - static_cast<uint64_t>(m * kElemBytes)};
  if (!same) {  // the same for every wave
    for (int64_t i = t * kTile + lane; i < (t + 1) * kTile; i += 64) {
      const bool in = i < d.len;
      float y = 0.0f;
      if (in) y = (kStaged ? Tr::unstage1(at(a), at(b), i) : Tr::load1(at(0), i)) * c;
      asm volatile("" : "+v"(y));
      if constexpr (kBarrier) __syncthreads();
      for (int32_t r = k0; in && r < k1; ++r) Tr::store1(at(r), i, y);
    }
    return;
  }
  // this lane's vector, and on a parameter's first tile an odd element
  const ChunkSpan k = make_span(m, d.len + m, V);
  const int64_t v0 = k.vs / V + t * 64;
  const int64_t v = v0 + lane;
  const bool ok = v < k.ve / V;
  const void *pa = lat(a), *pb = lat(b);
  uint4 x = make_uint4(0, 0, 0, 0), x2 = x;
  if (ok) {
    x = load_vec(pa, v);
    if constexpr (kStaged && Tr::kStageRanks == 2) x2 = load_vec(pb, v);
  }
  const OddElement odd = odd_element(k, t, lane, V);
  const bool any_odd = __any(odd.here);
  float y1 = 0.0f;
  if (odd.here) y1 = (kStaged ? Tr::unstage1(pa, pb, odd.at) : Tr::load1(pa, odd.at)) * c;
  float f[V];
  if constexpr (kStaged) {
    Tr::unsplit(x, x2, f);
  } else {
    Tr::widen(x, f);
  }
#pragma unroll
  for (int e = 0; e < V; ++e) f[e] = f[e] * c;
  uint4 y = Tr::narrow(f);
  // what is stored has been computed, so every load has returned, before
  // the barrier that lets the other waves overwrite the source
  asm volatile("" : "+v"(y.x), "+v"(y.y), "+v"(y.z), "+v"(y.w), "+v"(y1));
  if constexpr (kBarrier) __syncthreads();
  const bool lines =
      stream && __all(lane >= p || (lat.mine + static_cast<uint64_t>(v0) * kVecBytes) %
                                           static_cast<uint64_t>(kLineBytes) == 0);
  // two loops: one loop with two kinds of store would be given one kind
  if (lines) {
    for (int32_t r = k0; r < k1; ++r) {
      void *dst = lat(ring_rank(rot, r, p));
      if (ok) store_vec<true>(dst, v, y);
    }
  } else {
    for (int32_t r = k0; r < k1; ++r) {
      void *dst = lat(ring_rank(rot, r, p));
      if (ok) store_vec<false>(dst, v, y);
    }
  }
  for (int32_t r = k0; any_odd && r < k1; ++r) {
    void *dst = lat(ring_rank(rot, r, p));
    if (odd.here) Tr::store1(dst, odd.at, y1);
  }
}

}  // namespace
}  // namespace ddpsim
