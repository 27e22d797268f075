// The whole layer for a few tokens on its bf16 weights (sm_103a): router, top-k,
// experts and combine in two kernels.
//
// With one to 64 tokens the layer is the reading of its weights: W_router and the
// three matrices of every expert that a token takes.  The products run on the tensor
// cores with the operands' places exchanged: 128 rows of weights are the M of a
// tcgen05.mma, the expert's tokens (rounded up to 16) its N, so that every byte of
// weights goes once from HBM through TMA into shared memory and into the MMA, without
// an instruction per element.
//
//   up     clusters of CTAs share the router: each CTA multiplies its part of the
//          columns, the parts' sums change hands through distributed shared memory, and
//          each CTA ranks some of the tokens for its cluster (every cluster does this
//          for itself: no wait on the grid).  Then the active experts' gate and up rows
//          are dealt out in groups of eight, equal shares for all CTAs; the epilogue
//          leaves a = silu(h) u of every route in the workspace (bf16, as the layer).
//   down   a cluster owns some of d_model's rows for all experts; its CTAs take equal
//          parts of the (expert, d_ff) axis, add gate * y of their parts in 32 bits and
//          join them through distributed shared memory: sums in a fixed order.
//
// Tiles are built from TMA boxes of eight rows, the unit of the 128-byte swizzle, so
// that a share may begin at any group of eight rows; an MMA row without weights holds
// whatever the memory held, and its results are not read.  A token's rows are fetched
// by index (gather) into the MMA's N.
#include <atomic>

#include "common.cuh"
#include "kernels.h"
#include "few.h"

namespace moe {

namespace {

constexpr int kThreads = 192;          // TMA, MMA, four warps of the epilogue
constexpr int kEpi = 128;
constexpr int kWeightBytes = 128 * 128;   // of a stage: 128 rows of 64 columns
constexpr int kMaxStages = 12;
constexpr int kAccCols = 64;           // of an accumulator: tokens of an expert
constexpr int kTmem = 2 * kAccCols;

// 32 lanes x 16 columns of tensor memory.
MOE_DEV void tmem_ld16(uint32_t taddr, float* r) {
  uint32_t* q = reinterpret_cast<uint32_t*>(r);
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(q[0]), "=r"(q[1]), "=r"(q[2]), "=r"(q[3]), "=r"(q[4]), "=r"(q[5]), "=r"(q[6]), "=r"(q[7]), "=r"(q[8]),
        "=r"(q[9]), "=r"(q[10]), "=r"(q[11]), "=r"(q[12]), "=r"(q[13]), "=r"(q[14]), "=r"(q[15])
      : "r"(taddr)
      : "memory");
}

// Four rows of a matrix, by index, to four neighbouring rows of a swizzled tile.
MOE_DEV void tma_gather4(uint32_t dst, const CUtensorMap* map, uint64_t* bar, int x, int y0, int y1, int y2, int y3) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile::gather4.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5, %6, %7}], [%2];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(x), "r"(y0), "r"(y1), "r"(y2), "r"(y3)
      : "memory");
}
MOE_DEV void tma_box(uint32_t dst, const CUtensorMap* map, uint64_t* bar, int x, int y) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4}], [%2];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(x), "r"(y)
      : "memory");
}
MOE_DEV void st_cluster(uint32_t addr, float v) {
  asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(addr), "f"(v) : "memory");
}
MOE_DEV void st_cluster(uint32_t addr, int v) {
  asm volatile("st.shared::cluster.b32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}
MOE_DEV float ld_cluster(uint32_t addr) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
  return v;
}

struct Ctl {
  uint64_t full[kMaxStages], empty[kMaxStages];
  uint64_t tfull[2], tempty[2];
  uint64_t fin;
  uint32_t tmem;
  int abort;
  int n_act;                            // experts with routes
  uint32_t mask[256][2];                // tokens of an expert
  uint16_t base[257];                   // first route of an active expert, in their order
  uint8_t act[256], slot[256];          // active expert -> expert and back
  uint8_t tok[kFewMaxRoutes];           // token of a route
  int sel[kFewMaxRoutes];               // expert of (token, choice), -1: none
  float gate[kFewMaxRoutes];            // gate of a route
};

// From sel: the active experts in ascending order, their routes in the tokens' order.
// An expert that a token names twice is one route with the sum of its gates.
MOE_DEV void build_lists(Ctl& s, const FewParams& p, const float* gates) {
  const int R = p.T * p.k, tid = threadIdx.x;
  for (int i = tid; i < 2 * p.E; i += kThreads) (&s.mask[0][0])[i] = 0u;
  __syncthreads();
  for (int r = tid; r < R; r += kThreads) {
    const int e = s.sel[r], t = r / p.k;
    if (e >= 0) atomicOr(&s.mask[e][t >> 5], 1u << (t & 31));
  }
  __syncthreads();
  if (tid < 32) {   // eight experts a lane
    int routes[8], n = 0, act = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int e = tid * 8 + i;
      routes[i] = e < p.E ? __popc(s.mask[e][0]) + __popc(s.mask[e][1]) : 0;
      n += routes[i];
      act += routes[i] > 0;
    }
    int n0 = n, act0 = act;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int a = __shfl_up_sync(0xffffffffu, n0, off), b = __shfl_up_sync(0xffffffffu, act0, off);
      if (tid >= off) {
        n0 += a;
        act0 += b;
      }
    }
    if (tid == 31) {
      s.n_act = act0;
      s.base[act0] = (uint16_t)n0;
    }
    n0 -= n;
    act0 -= act;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if (routes[i]) {
        s.act[act0] = (uint8_t)(tid * 8 + i);
        s.slot[tid * 8 + i] = (uint8_t)act0;
        s.base[act0] = (uint16_t)n0;
        n0 += routes[i];
        ++act0;
      }
    }
  }
  __syncthreads();
  for (int r = tid; r < R; r += kThreads) {
    const int e = s.sel[r], t = r / p.k;
    if (e < 0) continue;
    bool first = true;
    for (int i = t * p.k; i < r; ++i) first = first && s.sel[i] != e;
    if (!first) continue;
    int at = s.base[s.slot[e]] + __popc(s.mask[e][t >> 5] & ((1u << (t & 31)) - 1u));
    if (t >= 32) at += __popc(s.mask[e][0]);
    s.tok[at] = (uint8_t)t;
    if (gates != nullptr) {
      float g = 0.0f;
      for (int i = r; i < (t + 1) * p.k; ++i)
        if (s.sel[i] == e) g += gates[i];
      s.gate[at] = g;
    }
  }
  __syncthreads();
}

// sel from indices in global memory; those outside [-1, E) are reported and left out.
MOE_DEV void read_routes(Ctl& s, const FewParams& p) {
  for (int r = threadIdx.x; r < p.T * p.k; r += kThreads) {
    int e = p.topk_idx[r];
    if (e < -1 || e >= p.E) {
      raise_error(p.err, MOE_DEVERR_BOUNDS);
      e = -1;
    }
    s.sel[r] = e;
  }
  __syncthreads();
}

// The k largest of a token's E logits and their gates, as the layer's routing ranks
// them: larger first, lower expert first among equals, a NaN below everything; the
// gates' sum over 32 lanes in the butterfly's order.  `logit` gives expert e's.
template <typename Logit, typename Sel>
MOE_DEV void rank_token(const FewParams& p, int t, bool write, Logit logit, Sel put) {
  const int lane = threadIdx.x & 31;
  float key[8];
  uint32_t taken = 0;
  bool bad = false;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int e = lane + 32 * i;
    float v = 0.0f;
    if (e < p.E) {
      v = logit(e);
      if (write && p.logits) p.logits[(size_t)t * p.E + e] = v;
      bad = bad || !isfinite(v);
    } else {
      taken |= 1u << i;
    }
    key[i] = v != v ? -INFINITY : v;
  }
  bad = __any_sync(0xffffffffu, bad);
  float mine = 0.0f, top = 0.0f;
  int id = 0;
  for (int j = 0; j < p.k; ++j) {
    float bv = 0.0f;
    int be = -1;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if (!(taken >> i & 1u) && (be < 0 || key[i] > bv)) {
        bv = key[i];
        be = lane + 32 * i;
      }
    }
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) {
      const float ov = __shfl_xor_sync(0xffffffffu, bv, off);
      const int oe = __shfl_xor_sync(0xffffffffu, be, off);
      if (oe >= 0 && (be < 0 || ov > bv || (ov == bv && oe < be))) {
        bv = ov;
        be = oe;
      }
    }
    if ((be & 31) == lane) taken |= 1u << (be >> 5);
    if (j == 0) top = bv;
    if (lane == j) {
      mine = bv;
      id = be;
    }
    if (lane == 0) put(j, be);
  }
  const float ex = lane < p.k ? expf(mine - top) : 0.0f;
  float sum = ex;
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
  if (write && lane < p.k) {
    p.topk_idx[t * p.k + lane] = id;
    p.gates[t * p.k + lane] = bad ? 0.0f : ex / sum;
  }
  if (write && bad && lane == 0) raise_error(p.err, MOE_DEVERR_NONFINITE_LOGIT);
}

// Barriers, tensor memory; the previous kernel's outputs are visible from here on.
MOE_DEV void begin(Ctl& s, const FewParams& p) {
  pdl_launch_dependents();
  if (threadIdx.x == 0) {
    for (int i = 0; i < p.stages; ++i) {
      mbar_init(&s.full[i], 1);
      mbar_init(&s.empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&s.tfull[i], 1);
      mbar_init(&s.tempty[i], kEpi);
    }
    mbar_init(&s.fin, 1);
    s.abort = 0;
    fence_barrier_init();
  }
  pdl_wait();
  if (threadIdx.x / 32 == 1) tmem_alloc(&s.tmem, kTmem);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
}

// Where a role stands in the ring and in the accumulators.
struct Place {
  int stage = 0;
  uint32_t phase = 0;
  int it = 0;   // accumulators used so far
  long issued = 0;
  MOE_DEV void next(const FewParams& p) {
    ++issued;
    if (++stage == p.stages) {
      stage = 0;
      phase ^= 1u;
    }
  }
};

// One warp: the next free stage, its copies announced.
MOE_DEV bool claim(Ctl& s, const FewParams& p, const Place& at, uint32_t bytes) {
  const bool ok = __all_sync(0xffffffffu, mbar_wait(&s.empty[at.stage], at.phase ^ 1u, &s.abort, p.err));
  if (ok && (threadIdx.x & 31) == 0) mbar_arrive_expect_tx(&s.full[at.stage], bytes);
  __syncwarp();
  return ok;
}
// The producer gave up: the copies that it announced land first.
MOE_DEV void drain(Ctl& s, const FewParams& p, const Place& at) {
  for (long i = at.issued > p.stages ? at.issued - p.stages : 0; i < at.issued; ++i) {
    const uint32_t bar = smem_u32(&s.full[(int)(i % p.stages)]);
    const uint64_t t0 = globaltimer();
    while (!mbar_try_wait(bar, (uint32_t)((i / p.stages) & 1)))
      if (globaltimer() - t0 > kWaitLimitNs) break;
  }
}

// One thread: `chunks` stages multiplied into the next accumulator.
MOE_DEV bool multiply(Ctl& s, const FewParams& p, uint8_t* ring, Place& at, int chunks, int n) {
  const int acc = at.it & 1;
  if (!mbar_wait(&s.tempty[acc], ((uint32_t)(at.it >> 1) & 1u) ^ 1u, &s.abort, p.err)) return false;
  tc_fence_after();
  const uint32_t d = s.tmem + acc * kAccCols, idesc = idesc_bf16_f32(128, n, 0, 0);
  for (int c = 0; c < chunks; ++c) {
    if (!mbar_wait(&s.full[at.stage], at.phase, &s.abort, p.err)) return false;
    tc_fence_after();
    const uint32_t a = smem_u32(ring + (size_t)at.stage * p.stage_bytes), b = a + kWeightBytes;
#pragma unroll
    for (int k = 0; k < 4; ++k)
      tc_mma_bf16(d, smem_desc_sw128(a + k * 32, 16, 1024), smem_desc_sw128(b + k * 32, 16, 1024), idesc, (c | k) != 0);
    tc_commit(&s.empty[at.stage]);
    at.next(p);
  }
  tc_commit(&s.tfull[acc]);
  ++at.it;
  return true;
}
// Its last word: every MMA that was issued has ended.
MOE_DEV void finish(Ctl& s, const FewParams& p) {
  tc_commit(&s.fin);
  const uint64_t t0 = globaltimer();
  while (!mbar_try_wait(smem_u32(&s.fin), 0)) {
    if (globaltimer() - t0 > kWaitLimitNs) {
      raise_error(p.err, MOE_DEVERR_TIMEOUT);
      break;
    }
  }
}

// The epilogue's threads: the accumulator `it` is complete / may be used again.
MOE_DEV bool results(Ctl& s, const FewParams& p, int it) {
  const bool ok = __all_sync(0xffffffffu, mbar_wait(&s.tfull[it & 1], (uint32_t)(it >> 1) & 1u, &s.abort, p.err));
  tc_fence_after();
  return ok;
}
MOE_DEV void release(Ctl& s, int it) {
  tc_fence_before();
  mbar_arrive(&s.tempty[it & 1]);
}

MOE_DEV void leave(Ctl& s) {
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (threadIdx.x / 32 == 1) {
    __syncwarp();
    tmem_dealloc(s.tmem, kTmem);
  }
}

MOE_DEV int share(int64_t total, int i, int n) { return (int)(total * i / n); }
MOE_DEV int round16(int n) { return (n + 15) & ~15; }

// The next rows of a share of (active expert, group of eight d_ff rows): at most eight
// groups of one expert, a run in equal pieces.
struct UpPiece {
  int a, g, n;   // active expert, first group, groups
  MOE_DEV bool next(int& from, int to, int groups) {
    if (from >= to) return false;
    a = from / groups;
    g = from - a * groups;
    const int run = min(to, (a + 1) * groups) - from, pieces = (run + 7) / 8;
    n = (run + pieces - 1) / pieces;
    from += n;
    return true;
  }
};

__global__ void __launch_bounds__(kThreads, 1)
    few_up_kernel(const __grid_constant__ CUtensorMap t_gate, const __grid_constant__ CUtensorMap t_up,
                  const __grid_constant__ CUtensorMap t_rows, const __grid_constant__ CUtensorMap t_x,
                  const __grid_constant__ CUtensorMap t_router, const FewParams p) {
  extern __shared__ __align__(1024) uint8_t smem[];
  uint8_t* ring = smem;
  Ctl& s = *reinterpret_cast<Ctl*>(smem + (size_t)p.stages * p.stage_bytes);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int quarter = warp & 3, row = quarter * 32 + lane;   // of the epilogue's threads
  begin(s, p);
  const uint32_t tmem = s.tmem + ((uint32_t)(quarter * 32) << 16);
  const int chunks = p.d / 64;
  Place at;
  bool ok = true;
  if (p.router) {
    const int C = p.cluster, rank = (int)cluster_ctarank(), own = (p.T + C - 1) / C;
    const int c0 = share(chunks, rank, C), c1 = share(chunks, rank + 1, C), tiles = (p.E + 127) / 128;
    cluster_sync();   // every CTA of the cluster has begun
    if (warp == 0) {
      for (int m = 0; m < tiles && ok; ++m) {
        for (int c = c0; c < c1; ++c) {
          ok = claim(s, p, at, kWeightBytes + p.t_pad * 128);
          if (!ok) break;
          const uint32_t to = smem_u32(ring + (size_t)at.stage * p.stage_bytes);
          if (lane == 0) {
            tma_box(to, &t_router, &s.full[at.stage], c * 64, m * 128);
            tma_box(to + kWeightBytes, &t_x, &s.full[at.stage], c * 64, 0);
          }
          at.next(p);
        }
      }
      __syncwarp();
    } else if (warp == 1) {
      if (lane == 0)
        for (int m = 0; m < tiles && ok; ++m) ok = multiply(s, p, ring, at, c1 - c0, p.t_pad);
      __syncwarp();
    } else {
      for (int m = 0; m < tiles; ++m) ok = results(s, p, m) && ok;
    }
    __syncwarp();
    cluster_sync();   // no CTA's ring is in use
    // the part of this CTA's columns to the CTA that ranks the token: [source, its
    // token, expert] in the ring
    if (warp >= 2) {
      const uint32_t mine = smem_u32(ring) + (uint32_t)(rank * own * p.E) * 4u;
      for (int m = 0; m < tiles; ++m) {
        const int e = m * 128 + row;
        for (int c = 0; c < p.t_pad; c += 16) {
          float v[16];
          tmem_ld16(tmem + m * kAccCols + c, v);
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            const int t = c + i;
            if (t < p.T && e < p.E)
              st_cluster(mapa_shared(mine + (uint32_t)((t / C) * p.E + e) * 4u, t % C), c1 > c0 ? v[i] : 0.0f);
          }
        }
        release(s, m);
      }
    }
    at.it = tiles;
    __syncwarp();
    cluster_sync();   // the parts are there
    const float* part = reinterpret_cast<const float*>(ring);
    const bool write = blockIdx.x < C;   // one cluster writes the routing
    for (int i = warp; rank + i * C < p.T; i += kThreads / 32) {
      const int t = rank + i * C;
      rank_token(
          p, t, write,
          [&](int e) {
            float v = 0.0f;
            for (int q = 0; q < C; ++q) v += part[(q * own + i) * p.E + e];
            return p.bias ? v + p.bias[(size_t)t * p.E + e] : v;
          },
          [&](int j, int e) {
            const uint32_t to = smem_u32(&s.sel[t * p.k + j]);
            for (int q = 0; q < C; ++q) st_cluster(mapa_shared(to, q), e);
          });
    }
    fence_proxy_async_smem();   // the ring was read and written by threads
    __syncwarp();
    cluster_sync();   // and the routing
  } else {
    read_routes(s, p);
  }
  build_lists(s, p, nullptr);

  const int groups = p.f / 8;
  const int64_t total = (int64_t)s.n_act * groups;
  int g = share(total, blockIdx.x, gridDim.x);
  const int g_end = share(total, blockIdx.x + 1, gridDim.x);
  UpPiece u;
  if (warp == 0) {
    while (ok && u.next(g, g_end, groups)) {
      const int e = s.act[u.a], r0 = s.base[u.a], m = s.base[u.a + 1] - r0, fours = (m + 3) / 4;
      // lanes 0-15: eight rows each, gate and up by turns (a pair of groups fills 32
      // rows, so that one warp of the epilogue sees both products of a row); lanes
      // 16-31: four tokens each
      const int j = lane >> 1, side = lane & 1;
      const uint32_t place = lane < 16 ? ((j >> 1) * 4 + (j & 1) * 2 + side) * 1024u : kWeightBytes + (lane - 16) * 512u;
      const int y = e * p.f + (u.g + j) * 8, i = (lane - 16) * 4;
      int y0 = 0, y1 = 0, y2 = 0, y3 = 0;
      if (lane >= 16 && i < m) {
        y0 = s.tok[r0 + i];
        y1 = s.tok[r0 + min(i + 1, m - 1)];
        y2 = s.tok[r0 + min(i + 2, m - 1)];
        y3 = s.tok[r0 + min(i + 3, m - 1)];
      }
      for (int c = 0; c < chunks; ++c) {
        ok = claim(s, p, at, u.n * 2048 + fours * 512);
        if (!ok) break;
        const uint32_t to = smem_u32(ring + (size_t)at.stage * p.stage_bytes) + place;
        if (lane < 2 * u.n)
          tma_box(to, side ? &t_up : &t_gate, &s.full[at.stage], c * 64, y);
        else if (lane >= 16 && i < m)
          tma_gather4(to, &t_rows, &s.full[at.stage], c * 64, y0, y1, y2, y3);
        at.next(p);
      }
    }
    if (!ok && lane == 0) drain(s, p, at);
  } else if (warp == 1) {
    if (lane == 0) {
      while (ok && u.next(g, g_end, groups))
        ok = multiply(s, p, ring, at, chunks, round16(s.base[u.a + 1] - s.base[u.a]));
      finish(s, p);
    }
  } else {
    // lanes 0-7 and 16-23 hold gate rows, the eight lanes after them the up rows
    const int group = quarter * 2 + (lane >> 4), r = lane & 7;
    const bool upper = lane & 8;
    __nv_bfloat16* act = static_cast<__nv_bfloat16*>(p.act);
    while (ok && u.next(g, g_end, groups)) {
      ok = results(s, p, at.it);
      if (!ok) break;
      const int r0 = s.base[u.a], m = s.base[u.a + 1] - r0;
      const size_t col = (size_t)(u.g + group) * 8 + r;
      for (int c = 0; c < m; c += 16) {
        float v[16];
        tmem_ld16(tmem + (at.it & 1) * kAccCols + c, v);
        // of two neighbouring tokens each lane of the pair takes one
#pragma unroll
        for (int i = 0; i < 16; i += 2) {
          const float got = __shfl_xor_sync(0xffffffffu, upper ? v[i] : v[i + 1], 8);
          const float h = upper ? got : v[i], up = upper ? v[i + 1] : got;
          const int t = c + i + upper;
          if (group < u.n && t < m) {
            const float a = __fdividef(h, 1.0f + __expf(-h)) * up;
            act[(size_t)(r0 + t) * p.f + col] = __float2bfloat16_rn(a);
          }
        }
      }
      release(s, at.it);
      ++at.it;
    }
  }
  leave(s);
}

// The next part of a CTA's share of (active expert, 64 columns of d_ff): one expert's.
struct DownPiece {
  int a, c, n;   // active expert, first chunk, chunks
  MOE_DEV bool next(int& from, int to, int chunks) {
    if (from >= to) return false;
    a = from / chunks;
    c = from - a * chunks;
    n = min(to, (a + 1) * chunks) - from;
    from += n;
    return true;
  }
};

__global__ void __launch_bounds__(kThreads, 1)
    few_down_kernel(const __grid_constant__ CUtensorMap t_down, const __grid_constant__ CUtensorMap t_act,
                    const FewParams p) {
  extern __shared__ __align__(1024) uint8_t smem[];
  uint8_t* ring = smem;
  float* sums = reinterpret_cast<float*>(smem + (size_t)p.stages * p.stage_bytes);   // [T][128]
  Ctl& s = *reinterpret_cast<Ctl*>(sums + p.T * 128);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int quarter = warp & 3, row = quarter * 32 + lane;
  begin(s, p);
  read_routes(s, p);
  build_lists(s, p, p.gates);
  const uint32_t tmem = s.tmem + ((uint32_t)(quarter * 32) << 16);
  const int C = p.cluster, rank = (int)cluster_ctarank(), clusters = gridDim.x / C, cluster = blockIdx.x / C;
  const int chunks = p.f / 64, total = s.n_act * chunks;
  const int from = share(total, rank, C), to = share(total, rank + 1, C);
  const int d0 = share(p.d / 8, cluster, clusters), d1 = share(p.d / 8, cluster + 1, clusters);
  const int tiles = (d1 - d0 + 15) / 16;
  Place at;
  bool ok = true;
  for (int tile = 0; tile < tiles; ++tile) {   // the same number in every CTA of the cluster
    const int g0 = d0 + share(d1 - d0, tile, tiles), n = d0 + share(d1 - d0, tile + 1, tiles) - g0;
    for (int i = threadIdx.x; i < p.T * 128; i += kThreads) sums[i] = 0.0f;
    __syncthreads();
    int c0 = from;
    DownPiece u;
    if (warp == 0) {
      while (ok && u.next(c0, to, chunks)) {
        const int e = s.act[u.a], r0 = s.base[u.a], eights = (s.base[u.a + 1] - r0 + 7) / 8;
        // lanes 0-15: eight rows of weights each, lanes 16-23: eight routes
        const uint32_t place = lane < 16 ? lane * 1024u : kWeightBytes + (lane - 16) * 1024u;
        const int y = lane < 16 ? e * p.d + (g0 + lane) * 8 : r0 + (lane - 16) * 8;
        const bool weights = lane < n, routes = lane >= 16 && lane - 16 < eights;
        for (int c = u.c; c < u.c + u.n; ++c) {
          ok = claim(s, p, at, (n + eights) * 1024);
          if (!ok) break;
          const uint32_t dst = smem_u32(ring + (size_t)at.stage * p.stage_bytes) + place;
          if (weights || routes) tma_box(dst, routes ? &t_act : &t_down, &s.full[at.stage], c * 64, y);
          at.next(p);
        }
      }
      __syncwarp();
    } else if (warp == 1) {
      if (lane == 0)
        while (ok && u.next(c0, to, chunks))
          ok = multiply(s, p, ring, at, u.n, round16(s.base[u.a + 1] - s.base[u.a]));
      __syncwarp();
    } else {
      while (ok && u.next(c0, to, chunks)) {
        ok = results(s, p, at.it);
        if (!ok) break;
        const int r0 = s.base[u.a], m = s.base[u.a + 1] - r0;
        for (int c = 0; c < m; c += 16) {
          float v[16];
          tmem_ld16(tmem + (at.it & 1) * kAccCols + c, v);
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            if (c + i < m) {
              float& sum = sums[s.tok[r0 + c + i] * 128 + row];
              sum = fmaf(s.gate[r0 + c + i], v[i], sum);
            }
          }
        }
        release(s, at.it);
        ++at.it;
      }
    }
    __syncwarp();
    cluster_sync();   // every CTA's sums are there
    const int rows = (128 + C - 1) / C;
    const uint32_t mine = smem_u32(sums);
    __nv_bfloat16* out = static_cast<__nv_bfloat16*>(p.out);
    for (int i = threadIdx.x; i < rows * p.T; i += kThreads) {
      const int t = i / rows, r = i - t * rows + rank * rows;
      if (r >= n * 8) continue;
      float v = 0.0f;
      for (int q = 0; q < C; ++q) v += ld_cluster(mapa_shared(mine + (uint32_t)(t * 128 + r) * 4u, q));
      out[(size_t)t * p.d + g0 * 8 + r] = __float2bfloat16_rn(v);
    }
    __syncwarp();
    cluster_sync();   // and have been read
  }
  if (warp == 0 && !ok && lane == 0) drain(s, p, at);
  if (warp == 1 && lane == 0) finish(s, p);
  leave(s);
}

constexpr int kCluster = 4;
constexpr int kRingBytes = 200 * 1024;

// CTAs of whole clusters that stay on the device at once.
int resident_ctas(const void* kernel, int smem, int device) {
  static std::atomic<int> known[kMaxDevices];
  int n = known[device].load();
  if (n == 0) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(kCluster);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim = {kCluster, 1, 1};
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (cudaOccupancyMaxActiveClusters(&n, kernel, &cfg) != cudaSuccess || n < 1) return 0;
    known[device].store(n *= kCluster);
  }
  return n;
}

template <typename... KArgs, typename... Args>
cudaError_t launch_clusters(void (*kernel)(KArgs...), int ctas, int smem, cudaStream_t s, const Args&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)ctas);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim = {kCluster, 1, 1};
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

}  // namespace

cudaError_t launch_few(const FewParams& args, const FewTensors& w, cudaStream_t s) {
  const DeviceInfo* dev = device_info();
  FewParams p = args;
  p.cluster = kCluster;
  p.router = w.w_router != nullptr;
  p.t_pad = (p.T + 15) & ~15;
  p.stage_bytes = kWeightBytes + p.t_pad * 128;
  const uint64_t d = (uint64_t)p.d, f = (uint64_t)p.f, E = (uint64_t)p.E;
  const uint64_t routes = ((uint64_t)p.T * p.k + 7) / 8 * 8;
  CUtensorMap gate, up, rows, x, router, down, act;
  if (!make_bf16_map(&gate, w.w_gate, d, E * f, 64, 8) || !make_bf16_map(&up, w.w_up, d, E * f, 64, 8) ||
      !make_bf16_map(&rows, w.x, d, (uint64_t)p.T, 64, 1) ||
      !make_bf16_map(&x, w.x, d, (uint64_t)p.T, 64, (uint32_t)p.t_pad) ||
      !make_bf16_map(&router, p.router ? w.w_router : w.w_gate, d, p.router ? E : E * f, 64, 128) ||
      !make_bf16_map(&down, w.w_down, f, E * d, 64, 8) || !make_bf16_map(&act, p.act, f, routes, 64, 8))
    return cudaErrorInvalidValue;
  const int up_stages = kRingBytes / p.stage_bytes, down_stages = (kRingBytes - p.T * 512) / p.stage_bytes;
  static SmemLimit up_limit, down_limit;
  constexpr int most = kRingBytes + (int)sizeof(Ctl);
  cudaError_t e = up_limit.raise(reinterpret_cast<const void*>(&few_up_kernel), most);
  if (e == cudaSuccess) e = down_limit.raise(reinterpret_cast<const void*>(&few_down_kernel), most);
  if (e != cudaSuccess) return e;
  const int ctas = resident_ctas(reinterpret_cast<const void*>(&few_up_kernel), most, dev->index);
  if (ctas == 0) return cudaErrorInvalidConfiguration;
  p.stages = up_stages < kMaxStages ? up_stages : kMaxStages;
  e = launch_clusters(&few_up_kernel, ctas, p.stages * p.stage_bytes + (int)sizeof(Ctl), s, gate, up, rows, x, router, p);
  if (e != cudaSuccess) return e;
  p.stages = down_stages < kMaxStages ? down_stages : kMaxStages;
  return launch_clusters(&few_down_kernel, ctas, p.stages * p.stage_bytes + p.T * 512 + (int)sizeof(Ctl), s, down, act, p);
}

}  // namespace moe
