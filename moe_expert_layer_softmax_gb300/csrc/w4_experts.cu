// The SwiGLU experts on 4-bit weights for a few tokens (sm_103a).
//
//   act[r] = gate_r silu(W_gate x) * (W_up x)      r = (token, choice), its expert's weights
//   out[t] = sum over the token's routes of W_down act[r]
// How the weights are streamed: w4.cuh.  The first kernel goes through the
// experts that have routes and writes act.  For one token the second kernel
// takes W_down of all its experts as one matrix of k f columns and writes out;
// for more it writes each route's product, and a third kernel adds them up.
// Few routes an expert (up to six on average): both kernels stage their vectors
// (fp16, act in two parts); more: they read them from global memory, x as it is
// and act as two bf16 parts in fragment order.  Either way act keeps 16 bits or
// more, so that storing it costs no accuracy beside a bf16 or fp16 result.
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
};
constexpr int kListsFixed = (256 + 1 + kW4Warps + 257) * 4 + 256 + 8;
static_assert(kListsFixed % 16 == 0, "the route lists follow");
__host__ __device__ inline int lists_bytes(int R) { return kListsFixed + ((R * 4 + 15) & ~15); }
MOE_DEV Lists lists_at(uint8_t* p, int R) {
  Lists l;
  l.counts = reinterpret_cast<int32_t*>(p);
  l.before = l.counts + 257 + kW4Warps;
  l.used = reinterpret_cast<uint8_t*>(l.before + 257);
  l.expert_of = reinterpret_cast<int16_t*>(p + kListsFixed);
  l.routes = reinterpret_cast<uint16_t*>(l.expert_of + R);
  return l;
}

// Experts with routes, ascending; returns their number.  Every thread calls.
MOE_DEV int find_used(const Lists& l, const int32_t* idx, int R, int E, int most) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  int32_t* scratch = l.counts + 257;
  if (tid < 256) l.counts[tid] = 0;
  __syncthreads();
  for (int r = tid; r < R; r += kW4Threads) {
    const int e = __ldcg(idx + r);
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

// The routes of expert e in l.routes; returns their number.  Every thread calls.
MOE_DEV int find_routes(const Lists& l, int R, int e) {
  int32_t* count = l.counts + 256;
  if (threadIdx.x == 0) *count = 0;
  __syncthreads();
  for (int r = threadIdx.x; r < R; r += kW4Threads)
    if (l.expert_of[r] == e) l.routes[atomicAdd(count, 1)] = (uint16_t)r;   // the order changes no result
  __syncthreads();
  return *count;
}

// This block's share of all (used expert, tile) pairs: a range of work units, a
// tile of an expert with w rounds being w of them.  Tiles belong to the block in
// whose range their first unit lies.  Where every expert has one round and the
// blocks divide among the experts with hardly a loss, they do not cross from
// one expert to another, which would cost a drain of the pipeline.
struct Share {
  int per;             // tiles of an expert
  int i;               // present expert (of the used ones)
  int64_t first, last;
  MOE_DEV Share(const Lists& l, int used, int per_) : per(per_), i(0) {
    const int all = used > 0 ? l.before[used] : 0;
    const int c = used > 0 ? gridDim.x / used : 0;
    if (c > 0 && all == used && c * used * 20 >= (int)gridDim.x * 19) {
      const int e = blockIdx.x / c, b = blockIdx.x - e * c;
      first = last = 0;
      if (e < used) {
        first = (int64_t)e * per + b * per / c;
        last = (int64_t)e * per + (b + 1) * per / c;
        i = e;
      }
    } else {
      first = (int64_t)blockIdx.x * all * per / gridDim.x;
      last = (int64_t)(blockIdx.x + 1) * all * per / gridDim.x;
      while (i < used && (int64_t)l.before[i + 1] * per <= first) ++i;
    }
  }
  // The tiles [t0, t1) of expert i; false: past the share.
  MOE_DEV bool tiles(const Lists& l, int used, int* t0, int* t1) const {
    if (i >= used) return false;
    const int64_t start = (int64_t)l.before[i] * per;
    if (start >= last) return false;
    const int w = l.before[i + 1] - l.before[i];
    *t0 = first > start ? (int)((first - start + w - 1) / w) : 0;
    *t1 = (int)min((int64_t)per, (last - start + w - 1) / w);
    return true;
  }
};

// Eight gate rows and the same eight up rows a tile.
template <typename S, int W> struct UpRows {
  const ExpertsW4Params& p;
  int64_t row0;   // first row of tile 0, over all experts
  MOE_DEV RowPtr operator()(int tile, int stage) const {
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const int64_t base = row0 + tile * 8;
    const int64_t at = (base + g) * (p.d / 2) + stage * 64 + t * 16;
    const S* sc = static_cast<const S*>(lane & 8 ? p.up_s : p.gate_s) + (base + (lane & 7)) * (p.d / (32 * W));
    return {p.gate_q + at, p.up_q + at, reinterpret_cast<const uint8_t*>(sc + stage * (4 / W))};
  }
};
template <typename S, int W> struct DownRows {
  const ExpertsW4Params& p;
  int64_t row0;
  MOE_DEV RowPtr operator()(int tile, int stage) const {
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const int64_t base = row0 + tile * 16;
    const int64_t at = (base + g) * (p.f / 2) + stage * 64 + t * 16;
    const S* sc = static_cast<const S*>(p.down_s) + (base + (lane & 15)) * (p.f / (32 * W));
    return {p.down_q + at, p.down_q + at + 8 * (int64_t)(p.f / 2), reinterpret_cast<const uint8_t*>(sc + stage * (4 / W))};
  }
};
// W_down of all the experts of one token, side by side.
template <typename S, int W> struct TokenRows {
  const ExpertsW4Params& p;
  const int16_t* expert_of;
  int64_t d0;
  int run;   // stages of an expert
  MOE_DEV RowPtr operator()(int tile, int stage) const {
    const int j = stage / run;
    const DownRows<S, W> rows = {p, (int64_t)expert_of[j] * p.d + d0};
    return rows(tile, stage - j * run);
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
  const uint32_t rings = smem_u32(smem);
  float* parts = reinterpret_cast<float*>(smem + kRingsBytes);
  const Lists l = lists_at(smem + plan.smem_lists, R);
  const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int stages = p.d / 128;
  StagedAt at;
  at.x = rings + kRingsBytes + (plan.seg_tiles + kW4Warps) * NT * 512;
  at.low = 0;
  at.stride = staged_stride(p.d);
  at.table = at.x + plan.most * at.stride;
  const int used = find_used(l, p.topk_idx, R, p.E, plan.most);
  Share share(l, used, p.f / 8);
  const T* x = static_cast<const T*>(p.x);
  float* act = static_cast<float*>(p.act);
  __nv_bfloat16* hi = static_cast<__nv_bfloat16*>(p.act);
  __nv_bfloat16* lo = hi + (int64_t)R * p.f;
  int first, last;
  for (; share.tiles(l, used, &first, &last); ++share.i) {
    const int e = l.used[share.i];
    const int n = first < last ? find_routes(l, R, e) : 0;
    for (int t0 = first; t0 < last; t0 += plan.seg_tiles) {
      const int tiles = min(last - t0, plan.seg_tiles);
      const UpRows<T, W> rows = {p, (int64_t)e * p.f + t0 * 8};
      for (int m0 = 0; m0 < n; m0 += plan.most) {
        Segment<T, T, W, NT, false, XS, true, false, 8, UpRows<T, W>> seg(
            rings, rows, tiles, stages, stages, p.d, reinterpret_cast<const void*>(~uintptr_t(0)));
        seg.start();
        const int here = min(n - m0, plan.most);   // vectors past it repeat the last one, unused
        auto token = [&](int m) { return x + (int64_t)(l.routes[m0 + m] / p.k) * p.ld_x; };
        if constexpr (XS == kStaged) {
          stage_vectors<T, W, false, 8>(at, here, p.d, token);
          __syncthreads();
        }
        Vectors<T, NT> v;
#pragma unroll
        for (int j = 0; j < NT; ++j) v.x[j] = token(min(j * 8 + g, here - 1));
        v.low = 0;
        v.s = at.x + min(g, here - 1) * at.stride;
        v.s_low = 0;
        v.table = at.table + t * 16;
        seg.finish(v, (here + 7) / 8, parts);
        __syncthreads();
        for (int i = threadIdx.x; i < tiles * here * 8; i += kW4Threads) {
          const int r8 = i & 7, tile = (i >> 3) / here, col = (i >> 3) - tile * here;
          const PartRange w(tile, tiles, stages);
          const int from = (col >> 3) * 128 + r8 * 8 + (col & 7);
          const float h = sum_parts(parts, NT * 128, tile, w, from);
          const float up = sum_parts(parts, NT * 128, tile, w, from + 64);
          const int route = l.routes[m0 + col];
          const float a = h / (1.0f + expf(-h)) * up * p.gates[route];
          const int piece = t0 + tile;   // the tile's eight columns of d_ff
          if constexpr (XS == kStaged) {
            act[(int64_t)route * p.f + piece * 8 + r8] = a;
          } else {
            const __nv_bfloat16 ah = __float2bfloat16_rn(a);
            const int64_t to = (int64_t)route * p.f + (piece >> 4) * 128 + piece_place<W>(piece & 15) * 8 + in_piece(r8);
            hi[to] = ah;
            lo[to] = __float2bfloat16_rn(a - __bfloat162float(ah));
          }
        }
        __syncthreads();
      }
    }
  }
}

// y[route] = W_down act[route].
template <typename T, int W, int NT, XSource XS>
__global__ void __launch_bounds__(kW4Threads, 1) experts_w4_down_kernel(ExpertsW4Params p, Plan plan) {
  extern __shared__ __align__(128) uint8_t smem[];
  const int R = p.T * p.k;
  const uint32_t rings = smem_u32(smem);
  float* parts = reinterpret_cast<float*>(smem + kRingsBytes);
  const Lists l = lists_at(smem + plan.smem_lists, R);
  const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int stages = p.f / 128;
  StagedAt at;
  at.x = rings + kRingsBytes + (plan.seg_tiles + kW4Warps) * NT * 512;
  at.stride = staged_stride(p.f);
  at.low = at.x + plan.most * at.stride;
  at.table = at.low + plan.most * at.stride;
  // weights and routes were complete before the first kernel let this one start
  const int used = find_used(l, p.topk_idx, R, p.E, plan.most);
  Share share(l, used, p.d / 16);
  const float* act = static_cast<const float*>(p.act);
  const __nv_bfloat16* hi = static_cast<const __nv_bfloat16*>(p.act);
  bool waited = false;
  int first, last;
  for (; share.tiles(l, used, &first, &last); ++share.i) {
    const int e = l.used[share.i];
    const int n = first < last ? find_routes(l, R, e) : 0;
    for (int t0 = first; t0 < last; t0 += plan.seg_tiles) {
      const int tiles = min(last - t0, plan.seg_tiles);
      const DownRows<T, W> rows = {p, (int64_t)e * p.d + t0 * 16};
      for (int m0 = 0; m0 < n; m0 += plan.most) {
        Segment<__nv_bfloat16, T, W, NT, true, XS, true, false, 8, DownRows<T, W>> seg(
            rings, rows, tiles, stages, stages, p.f, reinterpret_cast<const void*>(~uintptr_t(0)));
        seg.start();
        if (!waited) {
          pdl_wait();   // act
          pdl_launch_dependents();
          waited = true;
        }
        const int here = min(n - m0, plan.most);
        if constexpr (XS == kStaged) {
          stage_vectors<float, W, true, 8>(at, here, p.f, [&](int m) { return act + (int64_t)l.routes[m0 + m] * p.f; });
          __syncthreads();
        }
        Vectors<__nv_bfloat16, NT> v;
#pragma unroll
        for (int j = 0; j < NT; ++j) v.x[j] = hi + (int64_t)l.routes[m0 + min(j * 8 + g, here - 1)] * p.f;
        v.low = (int64_t)R * p.f;
        v.s = at.x + min(g, here - 1) * at.stride;
        v.s_low = v.s + plan.most * at.stride;
        v.table = at.table + t * 16;
        seg.finish(v, (here + 7) / 8, parts);
        __syncthreads();
        for (int i = threadIdx.x; i < tiles * here * 16; i += kW4Threads) {
          const int r16 = i & 15, tile = (i >> 4) / here, col = (i >> 4) - tile * here;
          const PartRange w(tile, tiles, stages);
          p.y[(int64_t)l.routes[m0 + col] * p.d + (t0 + tile) * 16 + r16] =
              sum_parts(parts, NT * 128, tile, w, (col >> 3) * 128 + r16 * 8 + (col & 7));
        }
        __syncthreads();
      }
    }
  }
  if (!waited) pdl_wait();
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
  const int n = n_routes, stages = n * run;
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
      const TokenRows<T, W> rows = {p, expert_of, (int64_t)t0 * 16, run};
      Segment<__nv_bfloat16, T, W, 1, true, kStaged, true, true, 1, TokenRows<T, W>> seg(
          rings, rows, tiles, stages, run, p.f, reinterpret_cast<const void*>(~uintptr_t(0)));
      seg.start();
      if (t0 == first) {
        pdl_wait();   // act
        pdl_launch_dependents();
        stage_vectors<float, W, true, 1>(at, n, p.f, [&](int j) { return act + (int64_t)route_of[j] * p.f; });
        __syncthreads();
      }
      Vectors<__nv_bfloat16, 1> v;
      v.x[0] = nullptr;
      v.low = 0;
      v.s = at.x;   // every column of the fragment repeats the one vector
      v.s_low = at.low;
      v.table = at.table;
      seg.finish(v, 1, parts);
      __syncthreads();
    } else if (t0 == first) {
      pdl_wait();
    }
    for (int i = threadIdx.x; i < tiles * 16; i += kW4Threads) {
      const int r16 = i & 15, tile = i >> 4;
      float s = 0.0f;
      if (n > 0) s = sum_parts(parts, 128, tile, PartRange(tile, tiles, stages), r16 * 8);
      out[(t0 + tile) * 16 + r16] = Elem<T>::from_f(s);
    }
    __syncthreads();
  }
}

// out[t] = sum of the routes' outputs in j order; a route without an expert
// (-1) adds nothing, an expert id out of range is reported and adds nothing.
template <typename T>
__global__ void __launch_bounds__(256) experts_w4_join_kernel(ExpertsW4Params p) {
  pdl_begin();
  const int c = (blockIdx.x * 256 + threadIdx.x) * 4;
  const int t = blockIdx.y;
  if (c >= p.d) return;
  float a[4] = {0.0f, 0.0f, 0.0f, 0.0f};
  for (int j = 0; j < p.k; ++j) {
    const int r = t * p.k + j;
    const int e = p.topk_idx[r];
    if (e >= 0 && e < p.E) {
      const float4 v = *reinterpret_cast<const float4*>(p.y + (int64_t)r * p.d + c);
      a[0] += v.x; a[1] += v.y; a[2] += v.z; a[3] += v.w;
    } else if (e != -1 && c == 0) {
      raise_error(p.err, MOE_DEVERR_BOUNDS);
    }
  }
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
int64_t staged_bytes(int count, int K, int parts, int cols, int W) {
  return (int64_t)count * parts * staged_stride(K) + (int64_t)K / (32 * W) * cols * 8;
}
bool staged_fits(int64_t bytes, int lists) {
  return bytes <= kSmemMost - kRingsBytes - lists - 16 - (8 + kW4Warps) * 512;
}

int share_of(const ExpertsW4Params& p, int per) {
  const int R = p.T * p.k, used = R < p.E ? R : p.E, sms = device_info()->sm_count;
  return (int)(((int64_t)used * per + sms - 1) / sms) + 1;
}

template <typename T, int W, int NT, XSource XS>
cudaError_t up_launch(const ExpertsW4Params* p, cudaStream_t s) {
  auto* kernel = &experts_w4_up_kernel<T, W, NT, XS>;
  if (p == nullptr) return allow_smem(kernel);
  Plan plan;
  plan.most = XS == kStaged && p->T < 8 ? p->T : 8 * NT;
  const int x = XS == kStaged ? (int)staged_bytes(plan.most, p->d, 1, 8, W) : 0;
  const size_t smem = plan_smem(share_of(*p, p->f / 8), NT, x, lists_bytes(p->T * p->k), &plan);
  return launch_pdl(kernel, dim3(device_info()->sm_count), dim3(kW4Threads), smem, s, *p, plan);
}

template <typename T, int W, int NT, XSource XS>
cudaError_t down_launch(const ExpertsW4Params* p, cudaStream_t s) {
  auto* kernel = &experts_w4_down_kernel<T, W, NT, XS>;
  if (p == nullptr) return allow_smem(kernel);
  Plan plan;
  plan.most = XS == kStaged && p->T < 8 ? p->T : 8 * NT;
  const int x = XS == kStaged ? (int)staged_bytes(plan.most, p->f, 2, 8, W) : 0;
  const size_t smem = plan_smem(share_of(*p, p->d / 16), NT, x, lists_bytes(p->T * p->k), &plan);
  cudaError_t e = launch_pdl(kernel, dim3(device_info()->sm_count), dim3(kW4Threads), smem, s, *p, plan);
  if (e != cudaSuccess) return e;
  return launch_pdl(experts_w4_join_kernel<T>, dim3((p->d + 1023) / 1024, p->T), dim3(256), 0, s, *p);
}

int64_t token_bytes(const ExpertsW4Params& p, int W) {
  return (int64_t)p.k * p.f * 4 + (int64_t)p.k * p.f / (32 * W) * 8;
}
constexpr int kTokenStatic = 256;   // its static shared memory, rounded up

template <typename T, int W> cudaError_t token_launch(const ExpertsW4Params* p, cudaStream_t s) {
  auto* kernel = &experts_w4_token_kernel<T, W>;
  if (p == nullptr) return allow_smem(kernel, kTokenStatic);
  const int sms = device_info()->sm_count, per = p->d / 16;
  const int blocks = per < sms ? per : sms;
  Plan plan;
  plan.most = 1;
  const size_t smem = plan_smem((per + blocks - 1) / blocks, 1, (int)token_bytes(*p, W), kTokenStatic, &plan) - kTokenStatic;
  return launch_pdl(kernel, dim3(blocks), dim3(kW4Threads), smem, s, *p, plan);
}

// p = NULL: raise every variant's shared memory limit.  Staged vectors serve up
// to eight routes a round; where experts have more than six on average a second
// round would read most weights again, and 16 or 32 vectors a pass are read from
// global memory instead.
template <typename T, int W> cudaError_t experts_nt(const ExpertsW4Params* p, cudaStream_t s) {
  cudaError_t e = cudaSuccess;
  if (p == nullptr) {
    e = up_launch<T, W, 1, kStaged>(p, s);
    if (e == cudaSuccess) e = up_launch<T, W, 2, kNatural>(p, s);
    if (e == cudaSuccess) e = up_launch<T, W, 4, kNatural>(p, s);
    if (e == cudaSuccess) e = down_launch<T, W, 1, kStaged>(p, s);
    if (e == cudaSuccess) e = down_launch<T, W, 2, kOrdered>(p, s);
    if (e == cudaSuccess) e = down_launch<T, W, 4, kOrdered>(p, s);
    return e == cudaSuccess ? token_launch<T, W>(p, s) : e;
  }
  const int R = p->T * p->k, lists = lists_bytes(R);
  const int few = p->T < 8 ? p->T : 8;
  const bool token = p->T == 1 && staged_fits(token_bytes(*p, W), kTokenStatic);
  const bool staged = (p->T <= 8 || R <= 6 * p->E) && staged_fits(staged_bytes(few, p->d, 1, 8, W), lists) &&
                      (token || staged_fits(staged_bytes(few, p->f, 2, 8, W), lists));
  if (staged) {
    e = up_launch<T, W, 1, kStaged>(p, s);
    if (e != cudaSuccess) return e;
    return token ? token_launch<T, W>(p, s) : down_launch<T, W, 1, kStaged>(p, s);
  }
  const bool two = R <= 16 * p->E;
  e = two ? up_launch<T, W, 2, kNatural>(p, s) : up_launch<T, W, 4, kNatural>(p, s);
  if (e != cudaSuccess) return e;
  return two ? down_launch<T, W, 2, kOrdered>(p, s) : down_launch<T, W, 4, kOrdered>(p, s);
}

template <typename T> cudaError_t experts_group(int group, const ExpertsW4Params* p, cudaStream_t s) {
  if (group == 32) return experts_nt<T, 1>(p, s);
  if (group == 64) return experts_nt<T, 2>(p, s);
  return experts_nt<T, 4>(p, s);
}

}  // namespace

cudaError_t experts_w4_init() {
  cudaError_t e = cudaSuccess;
  for (int g = 32; g <= 128 && e == cudaSuccess; g *= 2) {
    e = experts_group<__nv_bfloat16>(g, nullptr, nullptr);
    if (e == cudaSuccess) e = experts_group<__half>(g, nullptr, nullptr);
  }
  return e;
}

cudaError_t launch_experts_w4(const ExpertsW4Params& p, int dtype, cudaStream_t s) {
  return dtype == MOE_DT_BF16 ? experts_group<__nv_bfloat16>(p.group, &p, s) : experts_group<__half>(p.group, &p, s);
}

}  // namespace moe
