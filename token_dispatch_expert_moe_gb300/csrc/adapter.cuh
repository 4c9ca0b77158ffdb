// What the kernels of the adapters share: the map of a batch, its tiles and
// chunks, and where the scratch lies in the workspace.
#pragma once
#include "launch.cuh"
#include "philox.cuh"
#include "tc.cuh"

namespace moe {

constexpr int kTileRows = 128;   // tokens of a tile, all of one adapter

// Tokens of a chunk: the weight gradients are summed over a chunk's tokens in
// one CTA, and over an adapter's chunks in a second pass. A sixteenth of the
// batch gives that pass few partial sums and the first enough CTAs (32768 x 8192
// with dropout: an eighth 508 us, a sixteenth 490 us, a thirty-second 505 us);
// under 256 tokens a CTA's start weighs more than what it does (backward of 1000
// x 2048, rank 128: 47 us with 128, 41 us with 256 or 512; 2048 x 4096, rank 16:
// 42, 36 and 39 us).
__host__ __device__ constexpr int64_t chunk_rows(int64_t T) {
  const int64_t e = (T / 16 + kTileRows - 1) / kTileRows * kTileRows;
  return e < 256 ? 256 : e;
}
// An adapter of several chunks has more than one chunk's tokens, so at most
// twice as many chunks as full ones.
constexpr int kMaxSlots = 32;
__host__ __device__ constexpr int slots_of(int64_t T) { return T > chunk_rows(T) ? kMaxSlots : 0; }

// The map, in 32-bit words: a header, order [T] (the tokens by adapter, in
// their order inside one; those without an adapter last), and, 16-byte aligned,
// tiles, chunks and groups.
constexpr int kMapHeader = 16;
enum { kMapT = 0, kMapN = 1, kMapTiles = 2, kMapChunks = 3 };
// tile: {adapter or -1, first position, rows, 0};
// chunk: {adapter, first position, rows, slot of its partial sum, or -1: the only one of its adapter}
// group: {first slot, chunks} of an adapter
struct MapLayout {
  int64_t order, tiles, chunks, groups, words;
  int64_t max_tiles, max_chunks;
};
__host__ __device__ inline MapLayout map_layout(int64_t T, int n) {
  MapLayout m;
  const int64_t few = n + 1 < T ? n + 1 : T, used = n < T ? n : T;
  m.max_tiles = T / kTileRows + few;
  m.max_chunks = T / chunk_rows(T) + used;
  m.order = kMapHeader;
  m.tiles = m.order + (T + 3) / 4 * 4;
  m.chunks = m.tiles + 4 * m.max_tiles;
  m.groups = m.chunks + 4 * m.max_chunks;
  m.words = m.groups + 2 * (int64_t)n;
  return m;
}

// The tokens' grouping as a kernel reads it: a map, or none: adapter 0 for all
// tokens in their order. Whatever the map's words hold, tiles and chunks stay
// inside the batch.
struct Plan {
  const int32_t *map;   // NULL: none
  int64_t T;
  int n;
  uint32_t *status;

  __device__ __forceinline__ bool of_this_batch() const {
    return map == nullptr || this_batch(*reinterpret_cast<const int4 *>(map));
  }
  // Tile i of a grid of at most max_tiles: -1 and no rows beyond the batch's. The
  // header and the tile are read at once.
  __device__ __forceinline__ int4 tile_of(int64_t i) const {
    if (map == nullptr) return i < tiles() ? tile(i) : make_int4(-1, 0, 0, 0);
    const int4 head = *reinterpret_cast<const int4 *>(map);
    const int4 t = reinterpret_cast<const int4 *>(map + map_layout(T, n).tiles)[i];
    return this_batch(head) && i < head.z ? checked(t, kTileRows) : make_int4(-1, 0, 0, 0);
  }
  __device__ __forceinline__ int4 chunk_of(int64_t i) const {
    if (map == nullptr) return i < chunks() ? chunk(i) : make_int4(-1, 0, 0, -1);
    const int4 head = *reinterpret_cast<const int4 *>(map);
    const int4 c = reinterpret_cast<const int4 *>(map + map_layout(T, n).chunks)[i];
    return this_batch(head) && i < head.w ? checked_chunk(c) : make_int4(-1, 0, 0, -1);
  }
  __device__ __forceinline__ bool this_batch(const int4 &head) const {
    if (head.x == (int32_t)T && head.y == n) return true;
    report(status, MOE_ERR_DEVICE, kInfoAdapterMap);
    return false;
  }
  __device__ __forceinline__ int4 checked_chunk(int4 c) const {
    c = checked(c, chunk_rows(T));
    if (c.x >= 0 && c.w >= slots_of(T)) report(status, MOE_ERR_DEVICE, kInfoAdapterMap);
    if (c.x < 0 || c.w >= slots_of(T)) c.z = 0;
    return c;
  }
  __device__ __forceinline__ int64_t tiles() const {
    if (map == nullptr) return (T + kTileRows - 1) / kTileRows;
    if (!of_this_batch()) return 0;
    const int64_t m = map_layout(T, n).max_tiles, k = map[kMapTiles];
    return k < m ? k : m;
  }
  __device__ __forceinline__ int64_t chunks() const {
    if (map == nullptr) return (T + chunk_rows(T) - 1) / chunk_rows(T);
    if (!of_this_batch()) return 0;
    const int64_t m = map_layout(T, n).max_chunks, k = map[kMapChunks];
    return k < m ? k : m;
  }
  __device__ __forceinline__ int4 checked(int4 t, int64_t most) const {
    if (t.x < -1 || t.x >= n || t.y < 0 || t.z < 0 || t.z > most || (int64_t)t.y + t.z > T) {
      report(status, MOE_ERR_DEVICE, kInfoAdapterMap);
      t = make_int4(-1, 0, 0, -1);
    }
    return t;
  }
  __device__ __forceinline__ int4 tile(int64_t i) const {
    if (map == nullptr) {
      const int64_t left = T - i * kTileRows;
      return make_int4(0, (int)(i * kTileRows), (int)(left < kTileRows ? left : kTileRows), 0);
    }
    return checked(reinterpret_cast<const int4 *>(map + map_layout(T, n).tiles)[i], kTileRows);
  }
  __device__ __forceinline__ int4 chunk(int64_t i) const {
    const int64_t C = chunk_rows(T);
    if (map == nullptr) {
      const int64_t left = T - i * C;
      return make_int4(0, (int)(i * C), (int)(left < C ? left : C), T > C ? (int)i : -1);
    }
    return checked_chunk(reinterpret_cast<const int4 *>(map + map_layout(T, n).chunks)[i]);
  }
  __device__ __forceinline__ int2 group(int a) const {
    if (map == nullptr) {
      const int64_t k = (T + chunk_rows(T) - 1) / chunk_rows(T);
      return a == 0 ? make_int2(0, (int)k) : make_int2(0, 0);
    }
    int2 g = reinterpret_cast<const int2 *>(map + map_layout(T, n).groups)[a];
    // compared without a sum, which words that make no sense would overflow
    if (g.y < 0 || (g.y > 1 && (g.y > slots_of(T) || g.x < 0 || g.x > slots_of(T) - g.y))) {
      report(status, MOE_ERR_DEVICE, kInfoAdapterMap);
      g = make_int2(0, 0);
    }
    return g;
  }
  __device__ __forceinline__ int64_t token(int64_t pos) const {
    if (map == nullptr) return pos;
    const int64_t t = map[kMapHeader + pos];
    if ((uint64_t)t < (uint64_t)T) return t;
    report(status, MOE_ERR_DEVICE, kInfoAdapterMap);
    return 0;
  }
};

// The cluster's barrier, thread by thread: the warps come to it out of loops and
// branches that lanes leave at different times, and the .aligned forms (of
// cluster_sync) want whole warps.
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire;" ::: "memory"); }
__device__ __forceinline__ void cluster_meet() {
  cluster_arrive();
  cluster_wait();
}
// a word of another CTA's shared memory
__device__ __forceinline__ int remote_int(const void *p, uint32_t rank) {
  int v;
  asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v) : "r"(map_to_cta(smem_u32(p), rank)) : "memory");
  return v;
}
__device__ __forceinline__ float remote_float(const void *p, uint32_t rank) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(map_to_cta(smem_u32(p), rank)) : "memory");
  return v;
}

inline Plan plan_of(const AdapterArgs &a) { return Plan{a.map, a.T, a.n, a.status}; }
inline int64_t host_tiles(const AdapterArgs &a) {
  return a.map != nullptr ? map_layout(a.T, a.n).max_tiles : (a.T + kTileRows - 1) / kTileRows;
}
inline int64_t host_chunks(const AdapterArgs &a) {
  return a.map != nullptr ? map_layout(a.T, a.n).max_chunks : (a.T + chunk_rows(a.T) - 1) / chunk_rows(a.T);
}

// Columns of one part of u: 16, 32, 64 or 128, so that no part crosses 64 columns
// of an operand's box unless it fills whole ones.
__host__ __device__ constexpr int padded_rank(int rank) { return rank <= 16 ? 16 : rank <= 32 ? 32 : rank <= 64 ? 64 : 128; }

// Scratch: u and du by position, then the chunks' partial sums.
struct Scratch {
  size_t u, du, dA, dB, bytes;
};
__host__ inline Scratch scratch_of(int64_t T, int d_in, int d_out, int rank) {
  auto up = [](size_t v) { return (v + 255) & ~size_t(255); };
  Scratch s;
  // fp32 [T, rank], or bf16 [T, 3 padded_rank]: the three parts of u
  const size_t each = up((size_t)T * padded_rank(rank) * 6);
  const size_t slots = (size_t)slots_of(T);
  s.u = 0;
  s.du = each;
  s.dA = 2 * each;
  s.dB = s.dA + up(slots * rank * (size_t)d_in * 4);
  s.bytes = s.dB + up(slots * rank * (size_t)d_out * 4);
  return s;
}

// bf16 on the tensor cores (adapter_tc.cu)
cudaError_t launch_adapter_tc(const AdapterArgs &a, cudaStream_t s);
cudaError_t launch_adapter_bwd_tc(const AdapterArgs &a, cudaStream_t s);

// The second pass of the weight gradients (adapter.cu).
cudaError_t launch_adapter_join(const AdapterArgs &a, cudaStream_t s);

}  // namespace moe
