// tree_short.cu -- attention of small trees of drafted tokens over short paged caches, sm_103a.
//
// What tree_attn.cu computes, for up to 64 query rows on a KV head and caches of some hundred
// tokens.  There the time is that of a CTA's chain of dependent reads and products, and the
// pipeline of tree_attn.cu, one CTA an SM, takes long to fill.  Here a CTA of four warps takes a
// (request, KV head) by itself, three of them share an SM, and a warp does everything for its
// rows with warp-level products (m16n8k16): the fragments of Q stay in registers, K and V come
// 64 keys at a time from shared memory, where one TMA box a 16-token block puts them, two tiles
// in flight.  Up to 16 rows all four warps work on the same rows and take a quarter of the
// keys of each tile, up to 32 rows a half; their results are joined in shared memory at the end.
//
// A tile of 64 keys takes some 0.45 us with up to 16 rows, latencies of its loads and products,
// and 1.9 with 64 (D 128: 128 products a warp, whose accumulators and queries leave three CTAs an
// SM 56 bytes a thread too few registers: with two, which spill nothing, one request of 48 rows and
// 66 keys takes 6.2 us instead of 7.6, 64 of up to 100 keys 7.7 instead of 9.4, 100 of 64 rows and up
// to 280 keys 37.1 instead of 37.8), where tree_attn.cu takes 1.6 for 128 keys and up to 128 rows.
// shape_of in tree_attn.cu has the sizes up to which this kernel is taken, both sides measured.
// Eight warps a CTA and four tiles in flight for calls of at most a CTA an SM were no faster up to
// those sizes (12 heads x 8 nodes on 2 KV heads, 5 requests of 100 tokens: 8.5 us, four warps 7.7).
#include <cuda_runtime.h>

#include "gbattn.h"
#include "paged.cuh"
#include "ptx.cuh"
#include "tree.h"

namespace gbattn {

namespace {

constexpr int kKeys = 64;     // of a tile
constexpr int kBS = kPagedBlock;
constexpr int kBlocks = kKeys / kBS;
constexpr int kRows = kTreeShortRows;
constexpr float kRescaleLog2 = 8.f;  // move the running max only if it grows by > 2^8

constexpr int kThreads = 128;

template <int D>
struct Cfg {
  static constexpr int kCtasPerSm = 3;
  static constexpr int NS = 2;                      // tiles in flight
  static constexpr int KB = D / 64;                 // 64-column (128-byte) boxes of a row
  static constexpr int BOX = kKeys * 128;           // 64 rows x 128 bytes
  static constexpr int STAGE = 2 * KB * BOX;        // K then V
  static constexpr int OFF_SEEN = NS * STAGE;       // [64] what a node sees of the tree
  static constexpr int OFF_PARENT = OFF_SEEN + kRows * 8;  // [64] int8_t
  static constexpr int OFF_JOIN = OFF_PARENT + kRows;      // [4 warps][16 rows] float2: maximum, sum
  static constexpr int OFF_BAR = OFF_JOIN + 4 * 16 * 8;
  static constexpr int OFF_ABORT = OFF_BAR + NS * 8;
  static constexpr int SMEM = OFF_ABORT + 16 + 1024;       // slack for 1024-byte alignment
  static_assert(4 * 16 * D * 4 <= NS * STAGE, "the joined outputs take the tiles' place");
};

__device__ __forceinline__ void ldsm_x4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldsm_x4_t(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
// D = A * B + D, m16n8k16, bf16 inputs, fp32 accumulators.
__device__ __forceinline__ void mma_bf16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                         uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Address of 16-byte chunk `chunk` of row `row` of a tile of 64-column boxes with the 128-byte
// swizzle that TMA applies.
__device__ __forceinline__ uint32_t at(uint32_t tile, int row, int chunk) {
  return tile + (chunk >> 3) * (kKeys * 128) + row * 128 + (((chunk & 7) ^ (row & 7)) << 4);
}

// WR warps take 16 rows each, and 4 / WR warps share the keys of a tile.
template <int D, int WR>
__global__ void __launch_bounds__(kThreads, Cfg<D>::kCtasPerSm)
    tree_short_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                      const __grid_constant__ TreeParams p) {
  using C = Cfg<D>;
  constexpr int WK = 4 / WR;
  constexpr int WKEYS = kKeys / WK;  // a warp's keys of a tile
  constexpr int NT = WKEYS / 8;      // and tiles of 8 of them
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t sbase = (raw + 1023u) & ~1023u;
  uint8_t* smem = smem_raw + (sbase - raw);
  const uint32_t bars = sbase + C::OFF_BAR;
  volatile int* abort = reinterpret_cast<volatile int*>(smem + C::OFF_ABORT);
  unsigned long long* seen = reinterpret_cast<unsigned long long*>(smem + C::OFF_SEEN);
  int8_t* parent = reinterpret_cast<int8_t*>(smem + C::OFF_PARENT);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int g = lane >> 2, t4 = lane & 3;
  const int wr = warp % WR, wk = warp / WR;

  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (tid == 0) {
    for (int s = 0; s < C::NS; ++s) mbar_init(bars + 8 * s, 1);
    *abort = 0;
    fence_barrier_init();
    fence_proxy_async_smem();
    tma_prefetch_desc(&tmK);
    tma_prefetch_desc(&tmV);
  }
  const int r = blockIdx.x / p.Hkv, h = blockIdx.x - r * p.Hkv;
  const int rows = p.Hq / p.Hkv * p.Tn;
  // the preceding kernel's writes (an append's) are complete and visible past this point
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int32_t* table = p.block_table + static_cast<size_t>(r) * p.max_blocks;
  // (entry and parent are read before the lengths are known: at places that exist)
  int L = p.seq_lens[r], n = p.tree_lens ? p.tree_lens[r] : p.Tn;
  int first_entry = warp == 0 && lane < kBlocks && lane < p.max_blocks ? table[lane] : 0;
  int up = tid < p.Tn ? p.parents[static_cast<size_t>(r) * p.Tn + tid] : -1;
  // Q: rows g and g + 8 of the warp's 16
  uint32_t q[D / 16][4];
  {
    const int row = wr * 16 + g;
    const uint16_t* base = static_cast<const uint16_t*>(p.q) +
                           (static_cast<size_t>(blockIdx.x) * rows + row) * D + 2 * t4;
#pragma unroll
    for (int kk = 0; kk < D / 16; ++kk) {
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        q[kk][2 * c] = row < rows ? *reinterpret_cast<const uint32_t*>(base + 16 * kk + 8 * c) : 0u;
        q[kk][2 * c + 1] =
            row + 8 < rows ? *reinterpret_cast<const uint32_t*>(base + 8 * D + 16 * kk + 8 * c) : 0u;
      }
    }
  }
  const long long sum_len = static_cast<long long>(L) + n;
  const bool bad_len = L < 0 || n < 0 || n > p.Tn || sum_len > p.max_seq_len ||
                       sum_len > static_cast<long long>(p.max_blocks) * kBS;
  if (bad_len) L = n = 0;
  const int keys = n > 0 ? L + n : 0;
  const int tiles = (keys + kKeys - 1) / kKeys, blocks = (keys + kBS - 1) / kBS;
  const bool bad_node = tid < n && (up < -1 || up >= tid);
  if (bad_node) up = -1;
  if (tid < kRows) parent[tid] = static_cast<int8_t>(up);
  const bool bad_tree = __syncthreads_or(bad_node);  // (the barriers are ready too)
  if (tid == 0 && h == 0 && (bad_len || bad_tree))
    raise_flag(p.flags, bad_len ? DEVFLAG_BAD_SEQLEN : DEVFLAG_BAD_TREE);

  // copies of tile t (warp 0: a lane a block)
  auto issue = [&](int t, int phys) {
    const int s = t % C::NS, nblk = min(kBlocks, blocks - t * kBlocks);
    if (p.withhold_copy && t == 0) return;  // test hook: the first tile never arrives
    if (lane == 0) mbar_arrive_expect_tx(bars + 8 * s, nblk * 2 * kBS * D * 2);
    __syncwarp();
    if (lane < nblk) {
      if (phys < 0 || phys >= p.num_pool_blocks) {
        raise_flag(p.flags, DEVFLAG_BAD_BLOCK);
        phys = 0;
      }
      const uint32_t dst = sbase + s * C::STAGE + lane * (kBS * 128);
      const int row = (phys * p.Hkv + h) * kBS;
#pragma unroll
      for (int kb = 0; kb < C::KB; ++kb) {
        tma_load_2d(dst + kb * C::BOX, &tmK, bars + 8 * s, kb * 64, row);
        tma_load_2d(dst + (C::KB + kb) * C::BOX, &tmV, bars + 8 * s, kb * 64, row);
      }
    }
  };
  auto entry = [&](int t) {
    const int b = t * kBlocks + lane;
    return lane < kBlocks && b < blocks ? table[b] : 0;
  };
  if (warp == 0) {
    if (tiles > 0) issue(0, first_entry);
    for (int t = 1; t < C::NS && t < tiles; ++t) issue(t, entry(t));
  } else if (tid >= 64 && tid < 64 + kRows) {
    // what node tid - 64 sees of the tree
    const int i = tid - 64;
    unsigned long long bits = 0;
    for (int a = i < n ? i : -1; a >= 0; a = parent[a]) bits |= 1ull << a;
    seen[i] = bits;
  }
  __syncthreads();
  // rows without a node see nothing
  const int row0 = wr * 16 + g;
  const int node0 = row0 % p.Tn, node1 = (row0 + 8) % p.Tn;
  const unsigned long long seen0 = seen[node0], seen1 = seen[node1];
  const float sl2 = p.scale_log2;
  float o[D / 8][4], m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
#pragma unroll
  for (int j = 0; j < D / 8; ++j) o[j][0] = o[j][1] = o[j][2] = o[j][3] = 0.f;

  const int mat = lane >> 3, rr = lane & 7;
  int next_entry = warp == 0 && C::NS < tiles ? entry(C::NS) : 0;
  int t = 0;
  for (; t < tiles; ++t) {
    const int s = t % C::NS;
    const bool ok = mbar_wait_warp(bars + 8 * s, (t / C::NS) & 1, abort, p.flags, p.wait_limit_ns);
    const uint32_t kt = sbase + s * C::STAGE, vt = kt + C::KB * C::BOX;
    if (t == tiles - 1) {
      // Rows past the last key hold stale or arbitrary data (even NaN); their probabilities
      // are 0, but 0 * NaN would reach O.
      for (int e = (keys - t * kKeys) * (D / 8) + tid; e < kKeys * (D / 8); e += kThreads)
        st_shared_v4(at(vt, e / (D / 8), e % (D / 8)), 0u, 0u, 0u, 0u);
      __syncthreads();
    }
    if (ok) {
      // ---- S = Q K^T ----
      float sc[NT][4];
#pragma unroll
      for (int j = 0; j < NT; ++j) sc[j][0] = sc[j][1] = sc[j][2] = sc[j][3] = 0.f;
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk) {
#pragma unroll
        for (int j = 0; j < NT; j += 2) {
          uint32_t b[4];  // 16 keys x 16 channels
          ldsm_x4(at(kt, wk * WKEYS + 8 * j + (mat >> 1) * 8 + rr, 2 * kk + (mat & 1)), b);
          mma_bf16(sc[j], q[kk], b[0], b[1]);
          mma_bf16(sc[j + 1], q[kk], b[2], b[3]);
        }
      }
      const int x0 = t * kKeys + wk * WKEYS - L;  // the warp's first key, counted from node 0
      if (x0 + WKEYS > 0) {
#pragma unroll
        for (int j = 0; j < NT; ++j) {
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int x = x0 + 8 * j + 2 * t4 + e;
            if (x >= 0) {
              if (x >= 64 || !(seen0 >> (x & 63) & 1)) sc[j][e] = -INFINITY;
              if (x >= 64 || !(seen1 >> (x & 63) & 1)) sc[j][2 + e] = -INFINITY;
            }
          }
        }
      }
      // ---- softmax update ----
      float ms[2], al[2];
      bool grown = false;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        float mx = fmaxf(sc[0][2 * i], sc[0][2 * i + 1]);
#pragma unroll
        for (int j = 1; j < NT; ++j) mx = fmax3(mx, sc[j][2 * i], sc[j][2 * i + 1]);
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
        const bool grow = (mx - m[i]) * sl2 > kRescaleLog2;
        al[i] = grow ? ex2((m[i] - mx) * sl2) : 1.f;
        m[i] = grow ? mx : m[i];
        grown |= grow;
        ms[i] = m[i] == -INFINITY ? 0.f : m[i] * sl2;
        l[i] *= al[i];
      }
      if (__any_sync(0xffffffffu, grown)) {
#pragma unroll
        for (int j = 0; j < D / 8; ++j) {
          o[j][0] *= al[0];
          o[j][1] *= al[0];
          o[j][2] *= al[1];
          o[j][3] *= al[1];
        }
      }
#pragma unroll
      for (int j = 0; j < NT; ++j) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          sc[j][e] = ex2(fmaf(sc[j][e], sl2, -ms[e >> 1]));
          l[e >> 1] += sc[j][e];
        }
      }
      // ---- O += P V ----
#pragma unroll
      for (int ks = 0; ks < NT / 2; ++ks) {
        const uint32_t a[4] = {pack_bf16x2(sc[2 * ks][0], sc[2 * ks][1]),
                               pack_bf16x2(sc[2 * ks][2], sc[2 * ks][3]),
                               pack_bf16x2(sc[2 * ks + 1][0], sc[2 * ks + 1][1]),
                               pack_bf16x2(sc[2 * ks + 1][2], sc[2 * ks + 1][3])};
#pragma unroll
        for (int j = 0; j < D / 8; j += 2) {
          uint32_t b[4];  // 16 keys x 16 channels, transposed
          ldsm_x4_t(at(vt, wk * WKEYS + 16 * ks + (mat & 1) * 8 + rr, j + (mat >> 1)), b);
          mma_bf16(o[j], a, b[0], b[1]);
          mma_bf16(o[j + 1], a, b[2], b[3]);
        }
      }
    }
    if (!__syncthreads_and(ok)) break;  // (all have read the tile)
    if (warp == 0 && t + C::NS < tiles) {
      issue(t + C::NS, next_entry);
      next_entry = entry(t + C::NS + 1);
    }
  }
  if (t < tiles) {
    // A wait ran out: copies still in flight land before the CTA's shared memory goes away.
    if (tid == 0)
      for (int i = t; i < min(tiles, t + C::NS); ++i)
        if (!(p.withhold_copy && i == 0)) mbar_wait_quiet(bars + 8 * (i % C::NS), (i / C::NS) & 1, 500000000ull);
    return;
  }
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    l[i] += __shfl_xor_sync(0xffffffffu, l[i], 1);
    l[i] += __shfl_xor_sync(0xffffffffu, l[i], 2);
  }

  // ---- results ----
  const float nan = __int_as_float(0x7fc00000);
  uint16_t* out = static_cast<uint16_t*>(p.o) + static_cast<size_t>(blockIdx.x) * rows * D;
  float* out_lse = p.lse ? p.lse + static_cast<size_t>(blockIdx.x) * rows : nullptr;
  // (a row without a node has seen the cached tokens only)
  auto factor = [&](int node, float sum) {
    if (bad_len || (bad_tree && node < n)) return nan;
    return node >= n || sum == 0.f ? 0.f : 1.f / sum;
  };
  auto log_sum = [&](int node, float mx, float sum) {
    if (bad_len || (bad_tree && node < n)) return nan;
    return node >= n || sum == 0.f ? -INFINITY : mx * p.scale + logf(sum);
  };
  if constexpr (WK == 1) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int row = row0 + 8 * i, node = i ? node1 : node0;
      if (row >= rows) continue;
      const float f = factor(node, l[i]);
      const bool keep = f > 0.f;  // (else 0 or NaN, whatever the sums are)
#pragma unroll
      for (int j = 0; j < D / 8; ++j)
        *reinterpret_cast<uint32_t*>(out + static_cast<size_t>(row) * D + 8 * j + 2 * t4) =
            keep ? pack_bf16x2(o[j][2 * i] * f, o[j][2 * i + 1] * f) : pack_bf16x2(f, f);
      if (out_lse && t4 == 0) out_lse[row] = log_sum(node, m[i], l[i]);
    }
  } else {
    float* po = reinterpret_cast<float*>(smem);                  // [4 warps][16][D]
    float2* pm = reinterpret_cast<float2*>(smem + C::OFF_JOIN);  // [4 warps][16]
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int row = warp * 16 + g + 8 * i;
#pragma unroll
      for (int j = 0; j < D / 8; ++j)
        *reinterpret_cast<float2*>(po + row * D + 8 * j + 2 * t4) =
            make_float2(o[j][2 * i], o[j][2 * i + 1]);
      if (t4 == 0) pm[row] = make_float2(m[i], l[i]);
    }
    __syncthreads();
    constexpr int TPR = D / 4;  // threads of a row, four channels each
    for (int row = tid / TPR; row < min(rows, 16 * WR); row += kThreads / TPR) {
      const int c = tid % TPR * 4;
      float mx = -INFINITY;
#pragma unroll
      for (int k = 0; k < WK; ++k) mx = fmaxf(mx, pm[k * (16 * WR) + row].x);
      const float mr = mx == -INFINITY ? 0.f : mx;
      float sum = 0.f, v[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int k = 0; k < WK; ++k) {
        const float2 ml = pm[k * (16 * WR) + row];
        const float f = ex2((ml.x - mr) * sl2);
        const float4 y = *reinterpret_cast<const float4*>(po + (k * (16 * WR) + row) * D + c);
        sum = fmaf(f, ml.y, sum);
        v[0] = fmaf(f, y.x, v[0]);
        v[1] = fmaf(f, y.y, v[1]);
        v[2] = fmaf(f, y.z, v[2]);
        v[3] = fmaf(f, y.w, v[3]);
      }
      const int node = row % p.Tn;
      const float f = factor(node, sum);
      uint2 w = make_uint2(pack_bf16x2(f, f), pack_bf16x2(f, f));
      if (f > 0.f) w = make_uint2(pack_bf16x2(v[0] * f, v[1] * f), pack_bf16x2(v[2] * f, v[3] * f));
      *reinterpret_cast<uint2*>(out + static_cast<size_t>(row) * D + c) = w;
      if (out_lse && c == 0) out_lse[row] = log_sum(node, mx, sum);
    }
  }
}

template <int D, int WR>
cudaError_t launch(const CUtensorMap& tmK, const CUtensorMap& tmV, const TreeParams& p,
                   cudaStream_t stream) {
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(p.S) * p.Hkv);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = Cfg<D>::SMEM;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, tree_short_kernel<D, WR>, tmK, tmV, p);
}

template <int D>
cudaError_t launch_rows(const CUtensorMap& tmK, const CUtensorMap& tmV, const TreeParams& p,
                        cudaStream_t stream) {
  const int rows = p.Hq / p.Hkv * p.Tn;
  if (rows <= 16) return launch<D, 1>(tmK, tmV, p, stream);
  if (rows <= 32) return launch<D, 2>(tmK, tmV, p, stream);
  return launch<D, 4>(tmK, tmV, p, stream);
}

template <int D>
cudaError_t set_smem() {
  cudaError_t e = cudaSuccess;
  auto set = [&](const void* fn) {
    if (e == cudaSuccess)
      e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg<D>::SMEM);
  };
  set(reinterpret_cast<const void*>(tree_short_kernel<D, 1>));
  set(reinterpret_cast<const void*>(tree_short_kernel<D, 2>));
  set(reinterpret_cast<const void*>(tree_short_kernel<D, 4>));
  return e;
}

}  // namespace

cudaError_t prepare_tree_short() {
  const cudaError_t e = set_smem<64>();
  return e != cudaSuccess ? e : set_smem<128>();
}

cudaError_t launch_tree_short(const CUtensorMap& tmK, const CUtensorMap& tmV, const TreeParams& p,
                              cudaStream_t stream) {
  return p.D == 64 ? launch_rows<64>(tmK, tmV, p, stream) : launch_rows<128>(tmK, tmV, p, stream);
}

}  // namespace gbattn
