// The SwiGLU experts on 4-bit weights for a few tokens (sm_103a).
//
//   act[r] = gate_r silu(W_gate x) * (W_up x)      r = (token, choice), its expert's weights
//   out[t] = sum over the token's routes of W_down act[r]
// How the weights are streamed: w4.cuh.  The first kernel goes through the
// experts that have routes and writes act.  For one token the second kernel
// takes W_down of all its experts as one matrix of k f columns and writes out;
// for more it writes each route's product, and a third kernel adds them up.
// Both kernels stage their vectors (fp16, act in two parts) while shared memory
// has room for four at a time (or half the tokens, if those are fewer);
// otherwise (d above 12 K, f above 6 K, or many routes) they read them from
// global memory, x as it is and act as two bf16 parts in fragment order.  Either way act keeps 16 bits or more, so that storing it costs no
// accuracy beside a bf16 or fp16 result.
//
// Measured (us, bf16, weights from HBM, random routes): 64 experts of 2048 x 1408,
// four a token, groups of 64: 14.4 for one token, 41.9 for eight, 78.0 for 32, 88.3 for
// 64 (285 MB, 3.2 TB/s), 123 for 128, 381 for 512.  64 experts of 4096 x 2048, eight a
// token, groups of 128: 32.0 for one token (104 MB, 3.2 TB/s), 131 for eight (4.4
// TB/s).  Read from global memory instead, the first took 155 us with 64 tokens
// and the second 46 us with one; 32 experts of 4096 x 4096, where seven vectors
// are staged at a time, 64 tokens, 504 us rather than 304.
// (Included by one file per type, so that they compile side by side.)
#pragma once

#include "w4.cuh"

namespace moe {

namespace {

struct Plan {        // launch constants beside the call's
  int seg_tiles;     // most tiles of a segment (shared memory of the parts)
  int most;          // vectors of a round
  int smem_lists;    // byte where the lists start
};

// Shared lists of a block: the routes' experts, the experts in use with their
// routes' number, and the routes of the present expert.  before[i]: rounds of the
// used experts before the i-th (a round serves up to Plan::most routes).
struct Lists {
  int32_t* counts;      // [256 + 1 + kW4Warps] routes of an expert; a counter; scratch
  int32_t* before;      // [257]
  uint8_t* used;        // [256]
  int16_t* expert_of;   // [R], -1: none
  uint16_t* routes;     // [R]
  float* gates;         // [R] gates of `routes` (first kernel)
};
constexpr int kListsFixed = (256 + 1 + kW4Warps + 257) * 4 + 256 + 8;
static_assert(kListsFixed % 16 == 0, "the route lists follow");
__host__ __device__ inline int lists_bytes(int R) { return kListsFixed + ((R * 8 + 15) & ~15); }
MOE_DEV Lists lists_at(uint8_t* p, int R) {
  Lists l;
  l.counts = reinterpret_cast<int32_t*>(p);
  l.before = l.counts + 257 + kW4Warps;
  l.used = reinterpret_cast<uint8_t*>(l.before + 257);
  l.gates = reinterpret_cast<float*>(p + kListsFixed);
  l.expert_of = reinterpret_cast<int16_t*>(l.gates + R);
  l.routes = reinterpret_cast<uint16_t*>(l.expert_of + R);
  return l;
}

// Experts with routes, ascending; returns their number.  Every thread calls;
// mine0 is idx[threadIdx.x], loaded earlier (-1 past R).
MOE_DEV int find_used(const Lists& l, const int32_t* idx, int mine0, int R, int E, int most) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  int32_t* scratch = l.counts + 257;
  if (tid < 256) l.counts[tid] = 0;
  __syncthreads();
  for (int r = tid; r < R; r += kW4Threads) {
    const int e = r == tid ? mine0 : __ldcg(idx + r);
    const bool ok = e >= 0 && e < E;
    l.expert_of[r] = (int16_t)(ok ? e : -1);
    if (ok) atomicAdd(l.counts + e, 1);
  }
  __syncthreads();
  const int mine = tid < 256 ? (l.counts[tid] + most - 1) / most : 0;   // rounds
  const uint32_t ballot = __ballot_sync(0xffffffffu, mine > 0);
  int sum = mine;   // inclusive over the warp
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const int o = __shfl_up_sync(0xffffffffu, sum, off);
    if (lane >= off) sum += o;
  }
  if (lane == 31) scratch[warp] = __popc(ballot) << 16 | sum;
  __syncthreads();
  int at = __popc(ballot & ((1u << lane) - 1)), rounds = sum - mine, n = 0, all = 0;
  for (int w = 0; w < 8; ++w) {
    const int s = scratch[w];
    if (w < warp) {
      at += s >> 16;
      rounds += s & 0xFFFF;
    }
    n += s >> 16;
    all += s & 0xFFFF;
  }
  if (mine > 0) {
    l.used[at] = (uint8_t)tid;
    l.before[at] = rounds;
  }
  if (tid == 0) l.before[n] = all;
  __syncthreads();
  return n;
}

// The routes of expert e in l.routes (and their gates).  Every thread calls.
MOE_DEV void find_routes(const Lists& l, int R, int e, const float* gates) {
  int32_t* count = l.counts + 256;
  if (threadIdx.x == 0) *count = 0;
  __syncthreads();
  for (int r = threadIdx.x; r < R; r += kW4Threads)
    if (l.expert_of[r] == e) {
      // the order, and so the round and the column of a route, changes no result:
      // a column's products are the same instructions whatever lies beside it
      const int at = atomicAdd(count, 1);
      l.routes[at] = (uint16_t)r;
      if (gates) l.gates[at] = gates[r];
    }
  __syncthreads();
}

// This block's share of all (used expert, tile) pairs: a range of work units, a
// tile of an expert with w rounds being w of them.  Tiles belong to the block in
// whose range their first unit lies.  Going on to another expert costs a block
// about as much as kTurnUnits tiles (the last warps, the sums, the next
// vectors), so as many empty units lie between two experts.  Measured with 2, 4, 8
// and 12 (us; with the shorter conversion of stage_vectors' comment): 64 experts of 2048 x 1408, eight tokens 40.3, 38.7, 38.2, 39.1; 64
// tokens 85.8, 85.1, 84.7, 85.6; 128 tokens 123.2, 122.6, 119.4, 118.0; 8 experts of
// 1536 x 1024, two a token, 64 tokens 38.3, 36.9, 31.7, 31.9.  Where every expert
// has one round and the blocks divide among the experts with hardly a loss, they
// do not cross from one to another.
constexpr int kTurnUnits = 8;
struct Share {
  int per;             // tiles of an expert
  int i;               // present expert (of the used ones)
  int turn;            // empty units between experts
  int64_t first, last;
  MOE_DEV int64_t start(const Lists& l, int e) const { return (int64_t)l.before[e] * per + (int64_t)e * turn; }
  MOE_DEV Share(const Lists& l, int used, int per_) : per(per_), i(0), turn(kTurnUnits) {
    const int all = used > 0 ? l.before[used] : 0;
    const int c = used > 0 ? gridDim.x / used : 0;
    if (c > 0 && all == used && c * used * 20 >= (int)gridDim.x * 19) {
      turn = 0;
      const int e = blockIdx.x / c, b = blockIdx.x - e * c;
      first = last = 0;
      if (e < used) {
        first = (int64_t)e * per + b * per / c;
        last = (int64_t)e * per + (b + 1) * per / c;
        i = e;
      }
    } else {
      const int64_t units = start(l, used);
      first = (int64_t)blockIdx.x * units / gridDim.x;
      last = (int64_t)(blockIdx.x + 1) * units / gridDim.x;
      while (i < used && start(l, i + 1) <= first) ++i;
    }
  }
  // The tiles [t0, t1) of expert i; false: past the share.
  MOE_DEV bool tiles(const Lists& l, int used, int* t0, int* t1) const {
    if (i >= used) return false;
    const int64_t from = start(l, i);
    if (from >= last) return false;
    const int w = l.before[i + 1] - l.before[i];
    *t0 = first > from ? (int)min((int64_t)per, (first - from + w - 1) / w) : 0;
    *t1 = (int)min((int64_t)per, (last - from + w - 1) / w);
    return true;
  }
};

// The share as passes over weights: up to `seg` tiles of an expert for up to
// `most` of its routes.
struct Pass {
  Share share;
  int used, seg, most;
  int expert, t0, tiles, m0, here;   // the present pass: its tiles, its routes
  int end;                           // of the expert's tiles in the share
  bool enter;                        // it is the first of its expert
  bool other;                        // its routes are not those of the pass before
  bool valid;
  MOE_DEV Pass(const Lists& l, int used_, int per, int seg_, int most_)
      : share(l, used_, per), used(used_), seg(seg_), most(most_) {
    open(l);
  }
  MOE_DEV void open(const Lists& l) {
    int first;
    while ((valid = share.tiles(l, used, &first, &end)) && first >= end) ++share.i;
    if (!valid) return;
    expert = l.used[share.i];
    t0 = first;
    tiles = min(end - first, seg);
    m0 = 0;
    here = min(l.counts[expert], most);
    enter = other = true;
  }
  MOE_DEV void next(const Lists& l) {
    const int n = l.counts[expert];
    enter = false;
    other = n > most;
    m0 += most;
    if (m0 >= n) {
      m0 = 0;
      t0 += seg;
      if (t0 >= end) {
        ++share.i;
        open(l);
        return;
      }
      tiles = min(end - t0, seg);
    }
    here = min(n - m0, most);
  }
};

// Eight gate rows and the same eight up rows a tile.
template <typename S, int W> struct UpRows {
  const ExpertsW4Params& p;
  int64_t row0;   // first row of tile 0, over all experts
  MOE_DEV RowPtr operator()(int tile, int, int stage) const {
    const int lane = threadIdx.x & 31;
    const int64_t base = row0 + tile * 8;
    const int64_t at = (base + (lane >> 3)) * (p.d / 2) + stage * 64 + (lane & 7) * 16, four = 4 * (int64_t)(p.d / 2);
    const S* sc = static_cast<const S*>(lane & 8 ? p.up_s : p.gate_s) + (base + (lane & 7)) * (p.d / (32 * W));
    return {{p.gate_q + at, p.gate_q + at + four, p.up_q + at, p.up_q + at + four},
            reinterpret_cast<const uint8_t*>(sc + stage * (4 / W))};
  }
};
template <typename S, int W> struct DownRows {
  const ExpertsW4Params& p;
  int64_t row0;
  MOE_DEV RowPtr operator()(int tile, int, int stage) const {
    const int lane = threadIdx.x & 31;
    const int64_t base = row0 + tile * 16;
    const uint8_t* at = p.down_q + (base + (lane >> 3)) * (p.f / 2) + stage * 64 + (lane & 7) * 16;
    const int64_t four = 4 * (int64_t)(p.f / 2);
    const S* sc = static_cast<const S*>(p.down_s) + (base + (lane & 15)) * (p.f / (32 * W));
    return {{at, at + four, at + 2 * four, at + 3 * four}, reinterpret_cast<const uint8_t*>(sc + stage * (4 / W))};
  }
};
// W_down of all the experts of one token, side by side: run j is expert j.
template <typename S, int W> struct TokenRows {
  const ExpertsW4Params& p;
  const int16_t* expert_of;
  int64_t d0;
  MOE_DEV RowPtr operator()(int tile, int j, int stage) const {
    const DownRows<S, W> rows = {p, (int64_t)expert_of[j] * p.d + d0};
    return rows(tile, 0, stage);
  }
};

template <typename T, int W, int NT, XSource XS>
__global__ void __launch_bounds__(kW4Threads, 1) experts_w4_up_kernel(ExpertsW4Params p, Plan plan) {
  extern __shared__ __align__(128) uint8_t smem[];
  // the next kernel may start once every block here is past this wait: what
  // lies before this kernel (the weights, the routes) is then complete
  pdl_wait();
  pdl_launch_dependents();
  const int R = p.T * p.k;
  const int idx0 = threadIdx.x < R ? __ldcg(p.topk_idx + threadIdx.x) : -1;
  const uint32_t rings = smem_u32(smem);
  float* parts = reinterpret_cast<float*>(smem + kRingsBytes);
  const Lists l = lists_at(smem + plan.smem_lists, R);
  const int g = (threadIdx.x & 31) >> 2;
  const int stages = p.d / 128, steps = (stages + 1) / 2;
  StagedAt at;
  at.x = rings + kRingsBytes + (plan.seg_tiles + kW4Warps) * NT * 512;
  at.low = 0;
  at.stride = staged_stride(p.d);
  at.table = at.x + plan.most * at.stride;
  const T* x = static_cast<const T*>(p.x);
  float* act = static_cast<float*>(p.act);
  __nv_bfloat16* hi = static_cast<__nv_bfloat16*>(p.act);
  __nv_bfloat16* lo = hi + (int64_t)R * p.f;
  if (XS == kStaged && p.T == 1) stage_vectors<T, W, false, 8 * NT>(at, 1, p.d, [&](int) { return x; });
  const int used = find_used(l, p.topk_idx, idx0, R, p.E, plan.most);
  Pass ps(l, used, p.f / 8, plan.seg_tiles, plan.most);
  using Seg = Segment<T, T, W, NT, false, XS, true, false, 8 * NT, UpRows<T, W>>;
  const void* no_end = reinterpret_cast<const void*>(~uintptr_t(0));
  UpRows<T, W> rows = {p, ps.valid ? (int64_t)ps.expert * p.f + ps.t0 * 8 : 0};
  Seg seg(rings, rows, ps.valid ? ps.tiles : 0, 1, stages, p.d, no_end);
  seg.start();
  while (ps.valid) {
    if (ps.enter) find_routes(l, R, ps.expert, p.gates);
    auto token = [&](int m) { return x + (int64_t)(l.routes[ps.m0 + m] / p.k) * p.ld_x; };
    if constexpr (XS == kStaged) {
      if (p.T > 1 && ps.other) stage_vectors<T, W, false, 8 * NT>(at, ps.here, p.d, token);
    }
    __syncthreads();   // the vectors are staged, and the parts of the pass before are read
    Vectors<T, NT> v;
    if constexpr (XS == kStaged) {
      staged_at(v, at, ps.here);
    } else {
#pragma unroll
      for (int j = 0; j < NT; ++j) v.x[j] = token(min(j * 8 + g, ps.here - 1));   // past the last: unused
    }
    seg.finish(v, (ps.here + 7) / 8, parts);
    const Pass done = ps;
    ps.next(l);
    if (ps.valid) {   // the next pass's weights are on their way during what follows
      seg.rows.row0 = (int64_t)ps.expert * p.f + ps.t0 * 8;
      seg.reset(ps.tiles);
      seg.start();
    }
    __syncthreads();
    for (int i = threadIdx.x; i < done.tiles * done.here * 8; i += kW4Threads) {
      const int r8 = i & 7, tile = (i >> 3) / done.here, col = (i >> 3) - tile * done.here;
      const PartRange w(tile, done.tiles, steps);
      const int from = (col >> 3) * 128 + r8 * 8 + (col & 7);
      const float h = sum_parts(parts, NT * 128, tile, w, from);
      const float up = sum_parts(parts, NT * 128, tile, w, from + 64);
      const int route = l.routes[done.m0 + col];
      const float a = h / (1.0f + expf(-h)) * up * l.gates[done.m0 + col];
      const int piece = done.t0 + tile;   // the tile's eight columns of d_ff
      if constexpr (XS == kStaged) {
        act[(int64_t)route * p.f + piece * 8 + r8] = a;
      } else {
        const __nv_bfloat16 ah = __float2bfloat16_rn(a);
        const int64_t to = (int64_t)route * p.f + (piece >> 4) * 128 + piece_place<W>(piece & 15) * 8 + in_piece(r8);
        hi[to] = ah;
        lo[to] = __float2bfloat16_rn(a - __bfloat162float(ah));
      }
    }
    if (ps.valid && ps.enter) __syncthreads();   // the routes are read
  }
}

// y[route] = W_down act[route].
template <typename T, int W, int NT, XSource XS>
__global__ void __launch_bounds__(kW4Threads, 1) experts_w4_down_kernel(ExpertsW4Params p, Plan plan) {
  extern __shared__ __align__(128) uint8_t smem[];
  const int R = p.T * p.k;
  const int idx0 = threadIdx.x < R ? __ldcg(p.topk_idx + threadIdx.x) : -1;
  const uint32_t rings = smem_u32(smem);
  float* parts = reinterpret_cast<float*>(smem + kRingsBytes);
  const Lists l = lists_at(smem + plan.smem_lists, R);
  const int g = (threadIdx.x & 31) >> 2;
  const int stages = p.f / 128, steps = (stages + 1) / 2;
  StagedAt at;
  at.x = rings + kRingsBytes + (plan.seg_tiles + kW4Warps) * NT * 512;
  at.stride = staged_stride(p.f);
  at.low = at.x + plan.most * at.stride;
  at.table = at.low + plan.most * at.stride;
  // weights and routes were complete before the first kernel let this one start
  const int used = find_used(l, p.topk_idx, idx0, R, p.E, plan.most);
  const float* act = static_cast<const float*>(p.act);
  const __nv_bfloat16* hi = static_cast<const __nv_bfloat16*>(p.act);
  Pass ps(l, used, p.d / 16, plan.seg_tiles, plan.most);
  using Seg = Segment<__nv_bfloat16, T, W, NT, true, XS, true, false, 8 * NT, DownRows<T, W>>;
  const void* no_end = reinterpret_cast<const void*>(~uintptr_t(0));
  DownRows<T, W> rows = {p, ps.valid ? (int64_t)ps.expert * p.d + ps.t0 * 16 : 0};
  Seg seg(rings, rows, ps.valid ? ps.tiles : 0, 1, stages, p.f, no_end);
  seg.start();
  pdl_wait();   // act
  pdl_launch_dependents();
  while (ps.valid) {
    if (ps.enter) find_routes(l, R, ps.expert, nullptr);
    if (XS == kStaged && ps.other)
      stage_vectors<float, W, true, 8 * NT>(at, ps.here, p.f, [&](int m) { return act + (int64_t)l.routes[ps.m0 + m] * p.f; });
    __syncthreads();   // the vectors are staged, and the parts of the pass before are read
    Vectors<__nv_bfloat16, NT> v;
    if constexpr (XS == kStaged) {
      staged_at(v, at, ps.here);
    } else {
#pragma unroll
      for (int j = 0; j < NT; ++j) v.x[j] = hi + (int64_t)l.routes[ps.m0 + min(j * 8 + g, ps.here - 1)] * p.f;
      v.low = (int64_t)R * p.f;
    }
    seg.finish(v, (ps.here + 7) / 8, parts);
    const Pass done = ps;
    ps.next(l);
    if (ps.valid) {
      seg.rows.row0 = (int64_t)ps.expert * p.d + ps.t0 * 16;
      seg.reset(ps.tiles);
      seg.start();
    }
    __syncthreads();
    for (int i = threadIdx.x; i < done.tiles * done.here * 16; i += kW4Threads) {
      const int r16 = i & 15, tile = (i >> 4) / done.here, col = (i >> 4) - tile * done.here;
      const PartRange w(tile, done.tiles, steps);
      p.y[(int64_t)l.routes[done.m0 + col] * p.d + (done.t0 + tile) * 16 + r16] =
          sum_parts(parts, NT * 128, tile, w, (col >> 3) * 128 + r16 * 8 + (col & 7));
    }
    if (ps.valid && ps.enter) __syncthreads();   // the routes are read
  }
}

// One token: out = sum over its routes of W_down act, as one product with k f
// columns.  Routes without an expert are left out.
template <typename T, int W>
__global__ void __launch_bounds__(kW4Threads, 1) experts_w4_token_kernel(ExpertsW4Params p, Plan plan) {
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ int16_t expert_of[32];
  __shared__ int16_t route_of[32];
  __shared__ int32_t n_routes;
  const uint32_t rings = smem_u32(smem);
  float* parts = reinterpret_cast<float*>(smem + kRingsBytes);
  // weights and routes were complete before the first kernel let this one start
  if (threadIdx.x < 32) {
    const int lane = threadIdx.x;
    const int e = lane < p.k ? __ldcg(p.topk_idx + lane) : -1;
    const bool ok = e >= 0 && e < p.E;
    const uint32_t ballot = __ballot_sync(0xffffffffu, ok);
    const int to = __popc(ballot & ((1u << lane) - 1));
    if (ok) {
      expert_of[to] = (int16_t)e;
      route_of[to] = (int16_t)lane;
    }
    if (lane == 0) n_routes = __popc(ballot);
    if (blockIdx.x == 0 && !ok && e != -1) raise_error(p.err, MOE_DEVERR_BOUNDS);
  }
  __syncthreads();
  const int per = p.d / 16, run = p.f / 128;
  const int n = n_routes;
  StagedAt at;
  at.x = rings + kRingsBytes + (plan.seg_tiles + kW4Warps) * 512;
  at.stride = 2 * p.f;   // the routes one after the other
  at.low = at.x + n * at.stride;
  at.table = at.low + n * at.stride;
  const int first = (int)((int64_t)blockIdx.x * per / gridDim.x);
  const int last = (int)((int64_t)(blockIdx.x + 1) * per / gridDim.x);
  const float* act = static_cast<const float*>(p.act);
  T* out = static_cast<T*>(p.out);
  for (int t0 = first; t0 < last; t0 += plan.seg_tiles) {
    const int tiles = min(last - t0, plan.seg_tiles);
    if (n > 0) {
      const TokenRows<T, W> rows = {p, expert_of, (int64_t)t0 * 16};
      Segment<__nv_bfloat16, T, W, 1, true, kStaged, true, true, 1, TokenRows<T, W>> seg(
          rings, rows, tiles, n, run, p.f, reinterpret_cast<const void*>(~uintptr_t(0)));
      seg.start();
      if (t0 == first) {
        pdl_wait();   // act
        pdl_launch_dependents();
        stage_vectors<float, W, true, 1>(at, n, p.f, [&](int j) { return act + (int64_t)route_of[j] * p.f; });
        __syncthreads();
      }
      Vectors<__nv_bfloat16, 1> v;
      v.s = at.x;   // every column of the fragment repeats the one vector
      v.s_low = at.low;
      v.to[0] = 0;
      v.table = at.table;
      seg.finish(v, 1, parts);
      __syncthreads();
    } else if (t0 == first) {
      pdl_wait();
    }
    for (int i = threadIdx.x; i < tiles * 16; i += kW4Threads) {
      const int r16 = i & 15, tile = i >> 4;
      float s = 0.0f;
      if (n > 0) s = sum_parts(parts, 128, tile, PartRange(tile, tiles, n * ((run + 1) / 2)), r16 * 8);
      out[(t0 + tile) * 16 + r16] = Elem<T>::from_f(s);
    }
    __syncthreads();
  }
}

// out[t] = sum of the routes' outputs in j order; a route without an expert
// (-1) adds nothing, an expert id out of range is reported and adds nothing.
template <typename T>
__global__ void __launch_bounds__(256) experts_w4_join_kernel(ExpertsW4Params p) {
  pdl_launch_dependents();
  const int c = (blockIdx.x * 256 + threadIdx.x) * 4;
  const int t = blockIdx.y;
  // the routes were complete before the first kernel let the others start
  const int mine = (threadIdx.x & 31) < p.k ? __ldcg(p.topk_idx + t * p.k + (threadIdx.x & 31)) : -1;
  pdl_wait();
  float a[4] = {0.0f, 0.0f, 0.0f, 0.0f};
  for (int j = 0; j < p.k; ++j) {
    const int r = t * p.k + j;
    const int e = __shfl_sync(0xffffffffu, mine, j);
    if (c >= p.d) continue;
    if (e >= 0 && e < p.E) {
      const float4 v = *reinterpret_cast<const float4*>(p.y + (int64_t)r * p.d + c);
      a[0] += v.x; a[1] += v.y; a[2] += v.z; a[3] += v.w;
    } else if (e != -1 && c == 0) {
      raise_error(p.err, MOE_DEVERR_BOUNDS);
    }
  }
  if (c >= p.d) return;
  T* out = static_cast<T*>(p.out) + t * p.ld_out + c;
#pragma unroll
  for (int i = 0; i < 4; ++i) out[i] = Elem<T>::from_f(a[i]);
}

// Shared memory of a kernel with `lists` bytes of lists and `x` of vectors, and
// the most tiles that the parts of a segment have room for.
size_t plan_smem(int share, int NT, int x, int lists, Plan* plan) {
  const int room = (kSmemMost - kRingsBytes - x - lists - 16) / (NT * 512) - kW4Warps;
  plan->seg_tiles = share < room ? share : room;
  plan->smem_lists = (kRingsBytes + (plan->seg_tiles + kW4Warps) * NT * 512 + x + 15) & ~15;
  return plan->smem_lists + lists;
}

// Staged vectors of K values in `parts` parts with a table for `cols` columns,
// and whether they leave room for the parts of eight tiles.
int64_t staged_bytes(int count, int K, int parts, int cols) {
  return (int64_t)count * parts * staged_stride(K) + (int64_t)K / 128 * cols * 4;
}
bool staged_fits(int64_t bytes, int lists, int NT) {
  return bytes <= kSmemMost - kRingsBytes - lists - 16 - (8 + kW4Warps) * NT * 512;
}
// The most vectors a round can stage, up to 8 NT and the tokens there are.
int most_staged(const ExpertsW4Params& p, int K, int parts, int NT) {
  int n = p.T < 8 * NT ? p.T : 8 * NT;
  while (n > 0 && !staged_fits(staged_bytes(n, K, parts, 8 * NT), lists_bytes(p.T * p.k), NT)) --n;
  return n;
}

int share_of(const ExpertsW4Params& p, int per) {
  const int R = p.T * p.k, used = R < p.E ? R : p.E, sms = device_info()->sm_count;
  return (int)(((int64_t)used * per + sms - 1) / sms) + 1;
}

// The plan of a kernel with `per` tiles of an expert and vectors of K values in
// `parts` parts.
struct Launch {
  Plan plan;
  size_t smem;
  Launch(const ExpertsW4Params& p, int per, int K, int parts, int NT, bool staged) {
    plan.most = staged ? most_staged(p, K, parts, NT) : 8 * NT;
    smem = plan_smem(share_of(p, per), NT, staged ? (int)staged_bytes(plan.most, K, parts, 8 * NT) : 0,
                     lists_bytes(p.T * p.k), &plan);
  }
  // Sixteen vectors a round: they are staged, and a block's tiles are one segment.
  bool serves(const ExpertsW4Params& p, int per) const { return plan.most > 8 && plan.seg_tiles >= share_of(p, per); }
};

template <typename T, int W, int NT, XSource XS>
cudaError_t up_launch(const ExpertsW4Params& p, cudaStream_t s) {
  static SmemLimit limit;
  const Launch l(p, p.f / 8, p.d, 1, NT, XS == kStaged);
  return launch_w4(limit, &experts_w4_up_kernel<T, W, NT, XS>, dim3(device_info()->sm_count), l.smem, 0, s, p, l.plan);
}

template <typename T, int W, int NT, XSource XS>
cudaError_t down_launch(const ExpertsW4Params& p, cudaStream_t s) {
  static SmemLimit limit;
  const Launch l(p, p.d / 16, p.f, 2, NT, XS == kStaged);
  const cudaError_t e = launch_w4(limit, &experts_w4_down_kernel<T, W, NT, XS>, dim3(device_info()->sm_count), l.smem,
                                  0, s, p, l.plan);
  if (e != cudaSuccess) return e;
  return launch_pdl(experts_w4_join_kernel<T>, dim3((p.d + 1023) / 1024, p.T), dim3(256), 0, s, p);
}

int64_t token_bytes(const ExpertsW4Params& p) { return (int64_t)p.k * p.f * 4 + (int64_t)p.k * p.f / 128 * 4; }
constexpr int kTokenStatic = 256;   // its static shared memory, rounded up

template <typename T, int W> cudaError_t token_launch(const ExpertsW4Params& p, cudaStream_t s) {
  static SmemLimit limit;
  const int sms = device_info()->sm_count, per = p.d / 16;
  const int blocks = per < sms ? per : sms;
  Plan plan;
  plan.most = 1;
  const size_t smem = plan_smem((per + blocks - 1) / blocks, 1, (int)token_bytes(p), kTokenStatic, &plan) - kTokenStatic;
  return launch_w4(limit, &experts_w4_token_kernel<T, W>, dim3(blocks), smem, kTokenStatic, s, p, plan);
}

// Staged rounds serve eight routes of an expert, or sixteen where the experts
// have more than six on average and a block still takes its tiles of an expert
// in one segment.  Measured, eight and sixteen (us): 8 experts of 1536 x 1024, 12
// tokens on all of them 30.9 and 26.7, 64 tokens 96 and 80; 64 experts of 2048 x
// 1408, whose tiles would become two and more segments, 128 tokens 123 and 139.
// One token: W_down of all its experts as one product, 14.4 us, or a product for
// each and their sum, 17.2 (2048 x 1408, four experts); 32.2 and 35.0 (4096 x 2048,
// eight).
template <typename T, int W> cudaError_t experts_nt(const ExpertsW4Params& p, cudaStream_t s) {
  const int R = p.T * p.k, few = p.T < 8 ? p.T : 8;
  const bool token = p.T == 1 && staged_fits(token_bytes(p), kTokenStatic, 1);
  // both kernels or none: they agree on the form of act
  const bool staged = most_staged(p, p.d, 1, 1) * 2 >= few && (token || most_staged(p, p.f, 2, 1) * 2 >= few);
  if (!staged) {
    const cudaError_t e = up_launch<T, W, 2, kNatural>(p, s);
    return e == cudaSuccess ? down_launch<T, W, 2, kOrdered>(p, s) : e;
  }
  const bool many = R > 6 * p.E;
  const bool up2 = many && Launch(p, p.f / 8, p.d, 1, 2, true).serves(p, p.f / 8);
  const cudaError_t e = up2 ? up_launch<T, W, 2, kStaged>(p, s) : up_launch<T, W, 1, kStaged>(p, s);
  if (e != cudaSuccess) return e;
  if (token) return token_launch<T, W>(p, s);
  const bool down2 = many && Launch(p, p.d / 16, p.f, 2, 2, true).serves(p, p.d / 16);
  return down2 ? down_launch<T, W, 2, kStaged>(p, s) : down_launch<T, W, 1, kStaged>(p, s);
}

template <typename T> cudaError_t experts_group(int group, const ExpertsW4Params& p, cudaStream_t s) {
  if (group == 32) return experts_nt<T, 1>(p, s);
  if (group == 64) return experts_nt<T, 2>(p, s);
  return experts_nt<T, 4>(p, s);
}

}  // namespace

}  // namespace moe
