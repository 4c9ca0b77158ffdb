// The bf16 adapters' tiles on the tensor cores (tcgen05, accumulators in TMEM).
//
// Three products over a batch grouped by adapter, each bound by the memory
// traffic of its token rows (2 rank flops a byte, 4 with the parts):
//   shrink  v = x W^T       128 tokens of one adapter x rank, K = the width
//   expand  out += v V^T    128 tokens x 128 columns, K = 2 rank
//   wgrad   G = x^T v       128 columns x 2 rank, K = a chunk's tokens
// x, W and V are bf16 as they are. v (u or du) is an fp32 sum; it goes into the
// second products as two bf16 parts, hi = bf16(v) and lo = bf16(v - hi), side by
// side along K (expand) or N (wgrad): 2^-16 of v is left out where one part
// alone would leave 2^-8, and the products stay below the memory time.
//
// Rows are gathered (a tile's tokens lie anywhere in the batch), so the loader
// threads copy 16 bytes at a time with cp.async into the 128-byte-swizzled
// layout that the products read; the same thread takes dropped elements out of
// what it copied itself, before it passes the stage on.
#include "adapter.cuh"

namespace moe {
namespace {

using bf16 = __nv_bfloat16;

constexpr int kLoaders = 128;             // threads that copy, and then read the accumulator
constexpr int kPipeThreads = kLoaders + 32;   // and a warp that issues the products
constexpr int kMaxStages = 5;

// Roles in kInfoAdapterTimeout + role
enum { kRoleEmpty = 1, kRoleFull = 2, kRoleDone = 3, kRoleExpand = 4 };

struct Shared {
  uint64_t full[kMaxStages], empty[kMaxStages], done;
  uint32_t tmem;
  volatile int abort;
};

__device__ __forceinline__ bool wait(volatile int *abort, uint64_t *bar, uint32_t parity, uint32_t *status,
                                     uint32_t role) {
  const uint32_t b = smem_u32(bar);
  if (mbar_try_wait(b, parity)) return true;
  const uint64_t t0 = globaltimer();
  while (true) {
#pragma unroll 1
    for (int i = 0; i < 64; ++i)
      if (mbar_try_wait(b, parity)) return true;
    if (*abort) return false;
    if (globaltimer() - t0 > kTimeoutNs) {
      report(status, MOE_ERR_TIMEOUT, kInfoAdapterTimeout + role);
      *abort = 1;
      return false;
    }
  }
}

// 16 bytes from global memory, or zeros
__device__ __forceinline__ void copy16(uint32_t dst, const void *src, bool in) {
  const int n = in ? 16 : 0;
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N> __device__ __forceinline__ void copies_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// byte of 16-byte chunk c of row r in rows of 128 swizzled bytes
__device__ __forceinline__ uint32_t swz(int r, int c) { return (uint32_t)(r * 128 + ((c ^ (r & 7)) << 4)); }

template <int COLS> __device__ __forceinline__ void tmem_alloc(uint32_t *at) {
  asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(at)), "r"(COLS)
               : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
}
template <int COLS> __device__ __forceinline__ void tmem_free(uint32_t at) {
  asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(at), "r"(COLS) : "memory");
}
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, float (&v)[16]) {
  uint32_t r[16];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr)
      : "memory");
#pragma unroll
  for (int i = 0; i < 16; ++i) v[i] = __uint_as_float(r[i]);
}

// Eight elements (16 bytes of bf16), zeros in the dropped ones' place. Two
// elements a word at once: the low 15 bits of both halves against the
// threshold's by one addition (a carry into bit 15 or 31 says >=), the top bits
// by the majority with the threshold's, the resulting bits spread over their
// halves.
struct Mask {
  Philox g;
  uint32_t add, maj;
  __device__ __forceinline__ Mask(const uint64_t *rng, uint32_t t)
      : g(rng, t), add((0x8000u - (t & 0x7FFFu)) * 0x10001u), maj(t < 0x8000u ? 0xFFFFFFFFu : 0u) {}
  __device__ __forceinline__ uint32_t word(uint32_t w) const {
    const uint32_t u = (w & 0x7FFF7FFFu) + add;
    uint32_t m;   // bytes 1 and 3, each twice, by their sign
    asm("prmt.b32 %0, %1, 0, 0xBB99;" : "=r"(m) : "r"((u & w) | ((u | w) & maj)));
    return m;
  }
  __device__ __forceinline__ void apply(uint64_t block, uint4 &v) const {
    const uint4 w = g.block(block);
    v.x &= word(w.x);
    v.y &= word(w.y);
    v.z &= word(w.z);
    v.w &= word(w.w);
  }
};

// hi and lo parts of eight values
__device__ __forceinline__ void split8(const float (&v)[8], uint4 &hi, uint4 &lo) {
  uint32_t h[4], l[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 a = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
    const float2 f = __bfloat1622float2(a);
    const __nv_bfloat162 b = __floats2bfloat162_rn(v[2 * i] - f.x, v[2 * i + 1] - f.y);
    h[i] = *reinterpret_cast<const uint32_t *>(&a);
    l[i] = *reinterpret_cast<const uint32_t *>(&b);
  }
  hi = make_uint4(h[0], h[1], h[2], h[3]);
  lo = make_uint4(l[0], l[1], l[2], l[3]);
}

__device__ __forceinline__ void setup(Shared &st, int stages) {
  if (threadIdx.x == 0) {
    st.abort = 0;
    for (int s = 0; s < stages; ++s) {
      mbar_init(smem_u32(&st.full[s]), kLoaders);
      mbar_init(smem_u32(&st.empty[s]), 1);
    }
    mbar_init(smem_u32(&st.done), 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    fence_proxy_async();
  }
}

// The loaders' loop over `steps` stages: copy(step, stage) starts a step's
// copies, own(step, stage) takes out what is dropped from this thread's copies
// once they have landed. A step is passed on NST - 2 steps after its copies
// started, so that many stages are in flight.
template <int NST, typename Copy, typename Own>
__device__ __forceinline__ bool load_loop(Shared &st, int steps, uint32_t *status, Copy copy, Own own) {
  constexpr int LAG = NST - 2;
  bool ok = true;
  for (int i = 0; i < steps + LAG; ++i) {
    if (i < steps) {
      if (i >= NST && !wait(&st.abort, &st.empty[i % NST], (uint32_t)((i / NST - 1) & 1), status, kRoleEmpty)) {
        ok = false;
        break;
      }
      copy(i, i % NST);
    }
    copies_commit();
    const int j = i - LAG;
    if (j >= 0) {
      copies_wait<LAG>();
      own(j, j % NST);
      fence_proxy_async();
      mbar_arrive(smem_u32(&st.full[j % NST]));
    }
  }
  copies_wait<0>();
  return ok;
}

// The issuing warp's loop: mma(step, stage) by one lane for every stage passed on.
template <int NST, typename Mma>
__device__ __forceinline__ void mma_loop(Shared &st, int steps, int lane, uint32_t *status, Mma mma) {
  for (int i = 0; i < steps; ++i) {
    if (!__all_sync(0xffffffffu, wait(&st.abort, &st.full[i % NST], (uint32_t)((i / NST) & 1), status, kRoleFull))) break;
    tc_fence_after();
    if (lane == 0) {
      mma(i, i % NST);
      tc_commit(smem_u32(&st.empty[i % NST]));
    }
    __syncwarp();
  }
  if (lane == 0) {   // after every product issued so far
    if (steps > 0) tc_commit(smem_u32(&st.done));
    else mbar_arrive(smem_u32(&st.done));
  }
  __syncwarp();
}

// ---------------------------------------------------------------------------
// Shrink. A cluster of `split` CTAs takes a tile; each runs through a part of
// the width, the fp32 sums meet in shared memory and every CTA finishes a part
// of the rows, adding in the CTAs' order.
struct ShrinkTc {
  Plan plan;
  const bf16 *x, *W;    // W_a [rank, d], or [d, rank] (WT)
  int64_t ld;
  int d, rank, rp;      // rp: rank rounded up to 16
  int split, per;       // CTAs a tile, 64-column steps a CTA
  uint32_t threshold;
  const uint64_t *rng;
  const float *scale;   // per adapter, or NULL
  float factor;
  bf16 *parts;          // [T, 2 rp] by position: hi | lo
  float *by_token;      // [T, rank], or NULL; 0 without an adapter
  const float *u_in;    // [T, rank] by token, or NULL: parts_in gets its parts
  bf16 *parts_in;
};

template <int RPMAX, bool WT> struct ShrinkSize {
  static constexpr int kW = WT ? 8192 * ((RPMAX + 63) / 64) : RPMAX * 128;
  static constexpr int kStage = 16384 + kW;
  static constexpr int kStages = RPMAX <= 32 ? 5 : RPMAX <= 64 ? 4 : 3;
  static constexpr size_t kSmem = (size_t)kStages * kStage + 1024;
};

template <int RPMAX, bool WT>
__global__ void __launch_bounds__(kPipeThreads) shrink_tc_kernel(const ShrinkTc p) {
  using Z = ShrinkSize<RPMAX, WT>;
  constexpr int NST = Z::kStages, COLS = RPMAX;   // 32, 64 or 128 columns of TMEM
  extern __shared__ uint8_t raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
  __shared__ Shared st;
  __shared__ int64_t tok[kTileRows];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  setup(st, NST);
  pdl_wait();
  const int64_t ti = blockIdx.x / p.split;
  const int q = (int)(blockIdx.x % p.split);   // the CTA's rank in its cluster
  const bool on = ti < p.plan.tiles();
  const int4 tile = on ? p.plan.tile(ti) : make_int4(-1, 0, 0, 0);
  if (tile.x < 0) {   // the whole cluster
    if (p.by_token != nullptr && q == 0)
      for (int i = tid; i < tile.z * p.rank; i += kPipeThreads)
        p.by_token[p.plan.token(tile.y + i / p.rank) * p.rank + i % p.rank] = 0.0f;
    return;
  }
  if (tid < kTileRows) tok[tid] = tid < tile.z ? p.plan.token(tile.y + tid) : -1;
  if (warp == 4) tmem_alloc<COLS>(&st.tmem);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = st.tmem;
  const int k0 = q * p.per, all = (p.d + 63) / 64, steps = max(0, min(p.per, all - k0));
  const bf16 *W = p.W + (int64_t)tile.x * p.rank * p.d;

  if (warp < 4) {
    const int c = tid & 7, r0 = tid >> 3;   // this thread's chunk and first row of 16 apart
    int64_t at[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) at[i] = tok[r0 + 16 * i];
    const Mask mask(p.rng, p.threshold);
    const bool drops = p.threshold != 0;
    auto copy = [&](int step, int s) {
      const int k = (k0 + step) * 64 + c * 8;
      const uint32_t xs = smem_u32(smem + s * Z::kStage), ws = xs + 16384;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const bool in = at[i] >= 0 && k < p.d;
        copy16(xs + swz(r0 + 16 * i, c), in ? p.x + at[i] * p.ld + k : p.x, in);
      }
      if constexpr (!WT) {
        for (int j = r0; j < p.rp; j += 16) {
          const bool in = j < p.rank && k < p.d;
          copy16(ws + swz(j, c), in ? W + (int64_t)j * p.d + k : W, in);
        }
      } else {
        // rows of the width, rank in chunks of 64
        const int chunks = p.rp / 8;
        for (int i = tid; i < 64 * chunks; i += kLoaders) {
          const int kr = i / chunks, jc = i % chunks, kk = (k0 + step) * 64 + kr;
          const bool in = jc * 8 < p.rank && kk < p.d;
          copy16(ws + (jc >> 3) * 8192 + swz(kr, jc & 7), in ? W + (int64_t)kk * p.rank + jc * 8 : W, in);
        }
      }
    };
    auto own = [&](int step, int s) {
      if (!drops) return;
      const int k = (k0 + step) * 64 + c * 8;
      if (k >= p.d) return;
      uint8_t *xs = smem + s * Z::kStage;
#pragma unroll 2
      for (int i = 0; i < 8; ++i) {
        if (at[i] < 0) continue;
        uint4 *v = reinterpret_cast<uint4 *>(xs + swz(r0 + 16 * i, c));
        uint4 w = *v;
        mask.apply((uint64_t)(at[i] * p.d + k) >> 3, w);
        *v = w;
      }
    };
    load_loop<NST>(st, steps, p.plan.status, copy, own);
  } else {
    const uint32_t idesc = instr_desc(128, p.rp, 0, WT ? 1 : 0);
    mma_loop<NST>(st, steps, lane, p.plan.status, [&](int step, int s) {
      const uint32_t xs = smem_u32(smem + s * Z::kStage), ws = xs + 16384;
#pragma unroll
      for (int ks = 0; ks < 4; ++ks) {
        const uint64_t ad = smem_desc(xs + ks * 32, 16, 1024);
        const uint64_t bd = WT ? smem_desc(ws + ks * 2048, 8192, 1024) : smem_desc(ws + ks * 32, 16, 1024);
        tc_mma(tmem, ad, bd, idesc, (step > 0 || ks > 0) ? 1u : 0u);
      }
    });
  }
  // every product has ended: the ring is free, the accumulator whole
  wait(&st.abort, &st.done, 0, p.plan.status, kRoleDone);
  tc_fence_after();
  __syncthreads();
  const bool good = st.abort == 0;
  const int ls = p.rp + 4;   // floats from row to row of the sums
  float *sums = reinterpret_cast<float *>(smem);
  if (warp < 4) {
    for (int j = 0; j < p.rp; j += 16) {
      float v[16];
      if (steps > 0 && good) {
        tmem_ld16(tmem + ((uint32_t)(warp * 32) << 16) + j, v);
      } else {
#pragma unroll
        for (int i = 0; i < 16; ++i) v[i] = 0.0f;
      }
#pragma unroll
      for (int i = 0; i < 16; i += 4)
        *reinterpret_cast<float4 *>(sums + tid * ls + j + i) = make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]);
    }
  }
  tc_fence_before();
  if (p.split > 1) cluster_sync();
  else __syncthreads();
  tc_fence_after();
  if (warp == 4) tmem_free<COLS>(tmem);
  // rows of this CTA, eight values a thread at a time
  const int rows = kTileRows / p.split, g8 = p.rp / 8;
  const float f = p.factor * (p.scale != nullptr ? p.scale[tile.x] : 1.0f);
  if (good)
    for (int i = tid; i < rows * g8; i += kPipeThreads) {
      const int row = q * rows + i / g8, j = (i % g8) * 8;
      if (row >= tile.z) break;
      float v[8];
#pragma unroll
      for (int c = 0; c < 8; ++c) v[c] = 0.0f;
      for (int z = 0; z < p.split; ++z) {
        const uint32_t a = map_to_cta(smem_u32(sums + row * ls + j), (uint32_t)z);
        float w[8];
#pragma unroll
        for (int h = 0; h < 2; ++h)
          asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                       : "=f"(w[4 * h]), "=f"(w[4 * h + 1]), "=f"(w[4 * h + 2]), "=f"(w[4 * h + 3])
                       : "r"(a + 16 * h)
                       : "memory");
#pragma unroll
        for (int c = 0; c < 8; ++c) v[c] += w[c];
      }
      const bool in = j < p.rank;   // rank is a multiple of 8
#pragma unroll
      for (int c = 0; c < 8; ++c) v[c] = in ? v[c] * f : 0.0f;
      uint4 hi, lo;
      split8(v, hi, lo);
      bf16 *dst = p.parts + (int64_t)(tile.y + row) * 2 * p.rp + j;
      *reinterpret_cast<uint4 *>(dst) = hi;
      *reinterpret_cast<uint4 *>(dst + p.rp) = lo;
      const int64_t t = tok[row];
      if (p.by_token != nullptr && in) {
        float4 *o = reinterpret_cast<float4 *>(p.by_token + t * p.rank + j);
        o[0] = make_float4(v[0], v[1], v[2], v[3]);
        o[1] = make_float4(v[4], v[5], v[6], v[7]);
      }
      if (p.u_in != nullptr) {
        float w[8] = {};
        if (in) {
          const float4 *o = reinterpret_cast<const float4 *>(p.u_in + t * p.rank + j);
          const float4 a = o[0], b = o[1];
          w[0] = a.x; w[1] = a.y; w[2] = a.z; w[3] = a.w; w[4] = b.x; w[5] = b.y; w[6] = b.z; w[7] = b.w;
        }
        split8(w, hi, lo);
        dst = p.parts_in + (int64_t)(tile.y + row) * 2 * p.rp + j;
        *reinterpret_cast<uint4 *>(dst) = hi;
        *reinterpret_cast<uint4 *>(dst + p.rp) = lo;
      }
    }
  if (p.split > 1) cluster_sync();   // no CTA leaves while another reads its sums
}

// ---------------------------------------------------------------------------
// Expand: a CTA takes 128 columns of a tile.
struct ExpandTc {
  Plan plan;
  const bf16 *parts, *V;   // V_a [d, rank], or [rank, d] (VT)
  const void *base;
  void *out;
  int64_t ld;
  int d, rank, rp;
  uint32_t threshold;
  const uint64_t *rng;
  const float *scale;
  float factor;
};
constexpr int kCols = 128;

template <int RPMAX, typename TO, bool VT> struct ExpandSize {
  static constexpr int kParts = 16384 * ((2 * RPMAX + 63) / 64);
  static constexpr int kV = VT ? RPMAX * 256 : 16384 * ((RPMAX + 63) / 64);
  static constexpr int kPer = 128 / sizeof(TO);      // columns of a slab: rows of 128 bytes
  static constexpr int kSlabs = kCols / kPer;
  static constexpr size_t kSmem = kParts + kV + kSlabs * 16384 + 1024;
};

template <int RPMAX, typename TO, bool VT>
__global__ void __launch_bounds__(kLoaders) expand_tc_kernel(const ExpandTc p) {
  using Z = ExpandSize<RPMAX, TO, VT>;
  constexpr int VN = 16 / sizeof(TO);   // columns of a chunk
  extern __shared__ uint8_t raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
  uint8_t *vs = smem + Z::kParts, *slabs = vs + Z::kV;
  __shared__ Shared st;
  __shared__ int64_t tok[kTileRows];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  setup(st, 0);
  pdl_wait();
  const int blocks = (p.d + kCols - 1) / kCols;   // the columns of a tile one after another
  const int64_t ti = blockIdx.x / blocks;
  if (ti >= p.plan.tiles()) return;
  const int4 tile = p.plan.tile(ti);
  const TO *base = static_cast<const TO *>(p.base);
  TO *out = static_cast<TO *>(p.out);
  if (tile.z <= 0 || (tile.x < 0 && base == out)) return;
  tok[tid] = tid < tile.z ? p.plan.token(tile.y + tid) : -1;
  if (warp == 0 && tile.x >= 0) tmem_alloc<kCols>(&st.tmem);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const int c0 = (int)(blockIdx.x % blocks) * kCols;

  // parts and V, then the base rows: a warp copies what it alone reads and writes
  if (tile.x >= 0) {
    const int pc = p.rp / 4;   // chunks of a row of parts
    const bf16 *parts = p.parts + (int64_t)tile.y * 2 * p.rp;
    for (int i = tid; i < kTileRows * pc; i += kLoaders) {
      const int row = i / pc, c = i % pc;
      const bool in = row < tile.z;
      copy16(smem_u32(smem) + (c >> 3) * 16384 + swz(row, c & 7), in ? parts + (int64_t)row * 2 * p.rp + c * 8 : parts, in);
    }
    const bf16 *V = p.V + (int64_t)tile.x * p.rank * p.d;
    if constexpr (!VT) {
      const int vc = p.rp / 8;
      for (int i = tid; i < kCols * vc; i += kLoaders) {
        const int col = i / vc, c = i % vc;
        const bool in = c * 8 < p.rank && c0 + col < p.d;
        copy16(smem_u32(vs) + (c >> 3) * 16384 + swz(col, c & 7), in ? V + (int64_t)(c0 + col) * p.rank + c * 8 : V, in);
      }
    } else {
      for (int i = tid; i < p.rp * 16; i += kLoaders) {
        const int j = i >> 4, c = i & 15;
        const bool in = j < p.rank && c0 + c * 8 < p.d;
        copy16(smem_u32(vs) + (c >> 3) * (p.rp * 128) + swz(j, c & 7), in ? V + (int64_t)j * p.d + c0 + c * 8 : V, in);
      }
    }
  }
  copies_commit();
  const int rq = lane >> 3, ch = lane & 7;   // four rows at once, eight chunks each
  if (base != nullptr) {
#pragma unroll
    for (int s = 0; s < Z::kSlabs; ++s)
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int row = warp * 32 + i * 4 + rq, col = c0 + s * Z::kPer + ch * VN;
        const int64_t t = tok[row];
        const bool in = t >= 0 && col < p.d;
        copy16(smem_u32(slabs) + s * 16384 + swz(row, ch), in ? base + t * p.ld + col : base, in);
      }
  }
  copies_commit();
  bool good = true;
  if (tile.x >= 0) {
    copies_wait<1>();
    fence_proxy_async();
    __syncthreads();
    if (tid == 0) {
      const uint32_t idesc = instr_desc(128, kCols, 0, VT ? 1 : 0);
      const uint32_t as = smem_u32(smem), bs = smem_u32(vs);
      for (int ks = 0; ks < p.rp / 8; ++ks) {   // 2 rp / 16: hi, then lo, against the same V
        const int kb = ks < p.rp / 16 ? ks : ks - p.rp / 16;
        const uint64_t ad = smem_desc(as + (ks >> 2) * 16384 + (ks & 3) * 32, 16, 1024);
        const uint64_t bd = VT ? smem_desc(bs + kb * 2048, (uint32_t)p.rp * 128, 1024)
                               : smem_desc(bs + (kb >> 2) * 16384 + (kb & 3) * 32, 16, 1024);
        tc_mma(st.tmem, ad, bd, idesc, ks > 0 ? 1u : 0u);
      }
      tc_commit(smem_u32(&st.done));
    }
    copies_wait<0>();
    wait(&st.abort, &st.done, 0, p.plan.status, kRoleExpand);
    tc_fence_after();
    __syncthreads();
    good = st.abort == 0;
  } else {
    copies_wait<0>();
    __syncwarp();
  }
  if (good) {
    const float f = p.factor * (tile.x >= 0 && p.scale != nullptr ? p.scale[tile.x] : 1.0f);
    const Philox g(p.rng, p.threshold);
    const int row = warp * 32 + lane;
    const int64_t t = tok[row];
#pragma unroll 1
    for (int s = 0; s < Z::kSlabs; ++s) {
      uint8_t *slab = slabs + s * 16384;
#pragma unroll 1
      for (int h = 0; h < Z::kPer / 32; ++h) {
        const int col = c0 + s * Z::kPer + h * 32;
        float v[32];
        if (tile.x >= 0) tmem_ld32(st.tmem + ((uint32_t)(warp * 32) << 16) + s * Z::kPer + h * 32, v);
#pragma unroll
        for (int e = 0; e < 32; e += 8) {
          if (tile.x >= 0 && p.threshold != 0 && t >= 0 && col + e < p.d) {
            const uint4 w = g.block((uint64_t)(t * p.d + col + e) >> 3);
            if (!g.kept<0>(w)) v[e] = 0.0f;
            if (!g.kept<1>(w)) v[e + 1] = 0.0f;
            if (!g.kept<2>(w)) v[e + 2] = 0.0f;
            if (!g.kept<3>(w)) v[e + 3] = 0.0f;
            if (!g.kept<4>(w)) v[e + 4] = 0.0f;
            if (!g.kept<5>(w)) v[e + 5] = 0.0f;
            if (!g.kept<6>(w)) v[e + 6] = 0.0f;
            if (!g.kept<7>(w)) v[e + 7] = 0.0f;
          }
#pragma unroll
          for (int k = 0; k < 8; k += VN) {
            TO *at = reinterpret_cast<TO *>(slab + swz(row, (h * 32 + e + k) / VN));
            float b[VN];
            if (base != nullptr) {
              load16<TO>(at, b);
            } else {
#pragma unroll
              for (int i = 0; i < VN; ++i) b[i] = 0.0f;
            }
            if (tile.x >= 0)
#pragma unroll
              for (int i = 0; i < VN; ++i) b[i] = fmaf(f, v[e + k + i], b[i]);
            store16<TO>(at, b);
          }
        }
      }
      __syncwarp();
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int r = warp * 32 + i * 4 + rq, col = c0 + s * Z::kPer + ch * VN;
        const int64_t tr = tok[r];
        if (tr >= 0 && col < p.d)
          *reinterpret_cast<uint4 *>(out + tr * p.ld + col) = *reinterpret_cast<const uint4 *>(slab + swz(r, ch));
      }
    }
  }
  if (tile.x >= 0) {
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 0) tmem_free<kCols>(st.tmem);
  }
}

// ---------------------------------------------------------------------------
// Weight gradients: a CTA takes 128 columns of a chunk and runs through its
// tokens, 64 a step: both operands have the tokens (K) as rows.
struct WgradTc {
  Plan plan;
  const bf16 *z, *parts;   // [.., d] by token, [T, 2 rp] by position
  int64_t ld;
  int d, rank, rp;
  uint32_t threshold;
  const uint64_t *rng;
  const float *scale;
  float factor;
  float *out, *partial;    // [n, rank, d], or [n, d, rank] (GT); [slots, ..]
};

template <int RPMAX> struct WgradSize {
  static constexpr int kStage = 16384 + 8192 * ((2 * RPMAX + 63) / 64);
  static constexpr int kStages = RPMAX <= 32 ? 4 : RPMAX <= 64 ? 3 : 4;
  static constexpr size_t kSmem = (size_t)kStages * kStage + 1024;
};

template <int RPMAX, bool GT>
__global__ void __launch_bounds__(kPipeThreads) wgrad_tc_kernel(const WgradTc p) {
  using Z = WgradSize<RPMAX>;
  constexpr int NST = Z::kStages, COLS = 2 * RPMAX;
  extern __shared__ uint8_t raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
  __shared__ Shared st;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  setup(st, NST);
  pdl_wait();
  if (blockIdx.y >= p.plan.chunks()) return;
  const int4 ch = p.plan.chunk(blockIdx.y);
  if (ch.z <= 0) return;
  if (warp == 4) tmem_alloc<COLS>(&st.tmem);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = st.tmem;
  const int c0 = blockIdx.x * kCols, steps = (ch.z + 63) / 64;

  if (warp < 4) {
    const int c = tid & 15, r0 = tid >> 4;   // chunk of 8 columns, rows 8 apart
    const bool in_width = c0 + c * 8 < p.d;
    const bf16 *z = p.z + c0 + c * 8;
    const Mask mask(p.rng, p.threshold);
    const bool drops = p.threshold != 0;
    const int pc = p.rp / 4;
    int64_t next[8];
    auto tokens = [&](int step) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int row = step * 64 + r0 + 8 * i;
        next[i] = row < ch.z ? p.plan.token(ch.y + row) : -1;
      }
    };
    tokens(0);
    auto copy = [&](int step, int s) {
      const uint32_t zs = smem_u32(smem + s * Z::kStage), ps = zs + 16384;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const bool in = next[i] >= 0 && in_width;
        copy16(zs + (c >> 3) * 8192 + swz(r0 + 8 * i, c & 7), in ? z + next[i] * p.ld : p.z, in);
      }
      const bf16 *parts = p.parts + (int64_t)(ch.y + step * 64) * 2 * p.rp;
      const int rows = min(64, ch.z - step * 64);
      for (int i = tid; i < 64 * pc; i += kLoaders) {
        const int row = i / pc, k = i % pc;
        const bool in = row < rows;
        copy16(ps + (k >> 3) * 8192 + swz(row, k & 7), in ? parts + (int64_t)row * 2 * p.rp + k * 8 : p.parts, in);
      }
      if (step + 1 < steps) tokens(step + 1);
    };
    auto own = [&](int step, int s) {
      if (!drops || !in_width) return;
      uint8_t *zs = smem + s * Z::kStage;
#pragma unroll 2
      for (int i = 0; i < 8; ++i) {
        const int row = step * 64 + r0 + 8 * i;
        if (row >= ch.z) continue;
        uint4 *v = reinterpret_cast<uint4 *>(zs + (c >> 3) * 8192 + swz(r0 + 8 * i, c & 7));
        uint4 w = *v;
        mask.apply((uint64_t)(p.plan.token(ch.y + row) * p.d + c0 + c * 8) >> 3, w);
        *v = w;
      }
    };
    load_loop<NST>(st, steps, p.plan.status, copy, own);
  } else {
    const uint32_t idesc = instr_desc(128, 2 * p.rp, 1, 1);
    mma_loop<NST>(st, steps, lane, p.plan.status, [&](int step, int s) {
      const uint32_t zs = smem_u32(smem + s * Z::kStage), ps = zs + 16384;
#pragma unroll
      for (int ks = 0; ks < 4; ++ks)
        tc_mma(tmem, smem_desc(zs + ks * 2048, 8192, 1024), smem_desc(ps + ks * 2048, 8192, 1024), idesc,
               (step > 0 || ks > 0) ? 1u : 0u);
    });
  }
  wait(&st.abort, &st.done, 0, p.plan.status, kRoleDone);
  tc_fence_after();
  __syncthreads();
  if (warp < 4 && st.abort == 0) {
    const float f = p.factor * (p.scale != nullptr ? p.scale[ch.x] : 1.0f);
    float *out = ch.w < 0 ? p.out + (int64_t)ch.x * p.rank * p.d : p.partial + (int64_t)ch.w * p.rank * p.d;
    const int col = c0 + tid;
    const uint32_t at = tmem + ((uint32_t)(warp * 32) << 16);
    for (int j = 0; j < p.rp; j += 16) {
      float hi[16], lo[16];
      tmem_ld16(at + j, hi);
      tmem_ld16(at + p.rp + j, lo);
#pragma unroll
      for (int i = 0; i < 16; ++i) hi[i] = f * (hi[i] + lo[i]);
      if (col < p.d) {
        if constexpr (GT) {   // a thread's values lie side by side
#pragma unroll
          for (int i = 0; i < 16; i += 4)
            if (j + i < p.rank)
              *reinterpret_cast<float4 *>(out + (int64_t)col * p.rank + j + i) =
                  make_float4(hi[i], hi[i + 1], hi[i + 2], hi[i + 3]);
        } else {
#pragma unroll
          for (int i = 0; i < 16; ++i)
            if (j + i < p.rank) out[(int64_t)(j + i) * p.d + col] = hi[i];
        }
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 4) tmem_free<COLS>(tmem);
}

// ---------------------------------------------------------------------------
template <typename K> cudaError_t allow(K kernel, size_t smem) {
  return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
}

// CTAs a tile: until two a SM have work, as far as four steps are left to each
void set_split(const AdapterArgs &a, ShrinkTc &p) {
  const int64_t tiles = host_tiles(a), all = (p.d + 63) / 64;
  p.split = 1;
  while (p.split < 8 && tiles * p.split < 2 * sm_count() && all / (p.split * 2) >= 4) p.split *= 2;
  p.per = (int)((all + p.split - 1) / p.split);
}

template <int RPMAX, bool WT> cudaError_t shrink(const AdapterArgs &a, const ShrinkTc &p, cudaStream_t s) {
  constexpr size_t smem = ShrinkSize<RPMAX, WT>::kSmem;
  cudaError_t e = allow(shrink_tc_kernel<RPMAX, WT>, smem);
  if (e != cudaSuccess) return e;
  return launch_pdl_clusters(shrink_tc_kernel<RPMAX, WT>, dim3((unsigned)(host_tiles(a) * p.split)), dim3(kPipeThreads),
                             p.split, smem, s, p);
}
template <int RPMAX, typename TO, bool VT>
cudaError_t expand(const AdapterArgs &a, const ExpandTc &p, cudaStream_t s) {
  constexpr size_t smem = ExpandSize<RPMAX, TO, VT>::kSmem;
  cudaError_t e = allow(expand_tc_kernel<RPMAX, TO, VT>, smem);
  if (e != cudaSuccess) return e;
  return launch_pdl(expand_tc_kernel<RPMAX, TO, VT>, dim3((unsigned)((p.d + kCols - 1) / kCols * host_tiles(a))),
                    dim3(kLoaders), smem, s, p);
}
template <int RPMAX, bool GT> cudaError_t wgrad(const AdapterArgs &a, const WgradTc &p, cudaStream_t s) {
  constexpr size_t smem = WgradSize<RPMAX>::kSmem;
  cudaError_t e = allow(wgrad_tc_kernel<RPMAX, GT>, smem);
  if (e != cudaSuccess) return e;
  return launch_pdl(wgrad_tc_kernel<RPMAX, GT>, dim3((unsigned)((p.d + kCols - 1) / kCols), (unsigned)host_chunks(a)),
                    dim3(kPipeThreads), smem, s, p);
}

template <int RPMAX> cudaError_t forward(const AdapterArgs &a, int rp, cudaStream_t s) {
  const Scratch sc = scratch_of(a.T, a.d_in, a.d_out, a.rank);
  bf16 *parts = reinterpret_cast<bf16 *>(a.ws + sc.u);
  ShrinkTc sh{};
  sh.plan = plan_of(a);
  sh.x = static_cast<const bf16 *>(a.x); sh.W = static_cast<const bf16 *>(a.A); sh.ld = a.ld_in; sh.d = a.d_in;
  sh.rank = a.rank; sh.rp = rp; sh.threshold = a.threshold; sh.rng = a.rng; sh.factor = drop_scale(a.threshold);
  sh.parts = parts; sh.by_token = a.u;
  set_split(a, sh);
  cudaError_t e = shrink<RPMAX, false>(a, sh, s);
  if (e != cudaSuccess) return e;
  ExpandTc ex{};
  ex.plan = sh.plan; ex.parts = parts; ex.V = static_cast<const bf16 *>(a.B); ex.base = a.base; ex.out = a.y;
  ex.ld = a.ld_out; ex.d = a.d_out; ex.rank = a.rank; ex.rp = rp; ex.scale = a.scale; ex.factor = 1.0f;
  return expand<RPMAX, bf16, false>(a, ex, s);
}

template <int RPMAX> cudaError_t backward(const AdapterArgs &a, int rp, cudaStream_t s) {
  const Scratch sc = scratch_of(a.T, a.d_in, a.d_out, a.rank);
  bf16 *u = reinterpret_cast<bf16 *>(a.ws + sc.u), *du = reinterpret_cast<bf16 *>(a.ws + sc.du);
  const float keep = drop_scale(a.threshold);
  ShrinkTc sh{};
  sh.plan = plan_of(a);
  sh.x = static_cast<const bf16 *>(a.dy); sh.W = static_cast<const bf16 *>(a.B); sh.ld = a.ld_out; sh.d = a.d_out;
  sh.rank = a.rank; sh.rp = rp; sh.scale = a.scale; sh.factor = 1.0f; sh.parts = du;
  if (a.dA != nullptr) { sh.u_in = a.u_in; sh.parts_in = u; }
  set_split(a, sh);
  cudaError_t e = shrink<RPMAX, true>(a, sh, s);
  if (e == cudaSuccess && a.dA != nullptr) {
    WgradTc w{};
    w.plan = sh.plan; w.rank = a.rank; w.rp = rp;
    w.z = static_cast<const bf16 *>(a.dy); w.parts = u; w.ld = a.ld_out; w.d = a.d_out; w.scale = a.scale; w.factor = 1.0f;
    w.out = a.dB; w.partial = reinterpret_cast<float *>(a.ws + sc.dB);
    e = wgrad<RPMAX, true>(a, w, s);
    w.z = static_cast<const bf16 *>(a.x); w.parts = du; w.ld = a.ld_in; w.d = a.d_in; w.scale = nullptr; w.factor = keep;
    w.threshold = a.threshold; w.rng = a.rng; w.out = a.dA; w.partial = reinterpret_cast<float *>(a.ws + sc.dA);
    if (e == cudaSuccess) e = wgrad<RPMAX, false>(a, w, s);
    if (e == cudaSuccess) e = launch_adapter_join(a, s);
  }
  if (e == cudaSuccess && a.dx != nullptr) {
    ExpandTc ex{};
    ex.plan = sh.plan; ex.parts = du; ex.V = static_cast<const bf16 *>(a.A); ex.base = a.dx_in; ex.out = a.dx;
    ex.ld = a.d_in; ex.d = a.d_in; ex.rank = a.rank; ex.rp = rp; ex.threshold = a.threshold; ex.rng = a.rng;
    ex.factor = keep;
    e = a.dx_dtype == MOE_F32 ? expand<RPMAX, float, true>(a, ex, s) : expand<RPMAX, bf16, true>(a, ex, s);
  }
  return e;
}

}  // namespace

// Shared memory and TMEM are taken for ranks up to 32, 64 or 128.
cudaError_t launch_adapter_tc(const AdapterArgs &a, cudaStream_t s) {
  const int rp = (a.rank + 15) / 16 * 16;
  return rp <= 32 ? forward<32>(a, rp, s) : rp <= 64 ? forward<64>(a, rp, s) : forward<128>(a, rp, s);
}
cudaError_t launch_adapter_bwd_tc(const AdapterArgs &a, cudaStream_t s) {
  const int rp = (a.rank + 15) / 16 * 16;
  return rp <= 32 ? backward<32>(a, rp, s) : rp <= 64 ? backward<64>(a, rp, s) : backward<128>(a, rp, s);
}

}  // namespace moe
