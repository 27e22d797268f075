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
//          leaves a = silu(h) u of every route in the workspace, as two bf16 numbers (a
//          and what its rounding leaves over): they are two columns of the down MMA's N,
//          whose 16 at least are there anyway, and cost the result no second rounding.
//   down   a cluster owns some of d_model's rows for all experts; its CTAs take equal
//          parts of the (expert, d_ff) axis, add gate * y of their parts in 32 bits and
//          join them through distributed shared memory: sums in a fixed order.
//
// Shares begin at any group of eight rows, the unit of the 128-byte swizzle; a tile is
// built from TMA boxes of 8 to 128 rows; an MMA row without weights holds
// whatever the memory held, and its results are not read.  A token's rows are fetched
// by index (gather) into the MMA's N.
//
// Bound by HBM, behind a fixed cost.  Measured (floor at a copy's 6.78 TB/s), bf16:
//   1 token,   8 of 64 experts, 4096 x 2048   84 us (59.5): up 6.6, down 6.1 TB/s while
//              weights stream, 62 us; routing 9; the kernels' starts and joins 12
//   16 tokens, 4 of 32, 2048 x 1024           78 us (52.5): 7.0 and 5.6 TB/s; routing 7
//   64 tokens, 4 of 64, 2048 x 1408           192 us (161); routing 16, sixteen tokens a CTA
// The fixed cost shows most on small layers: 1 token, 4 of 64 experts of 2048 x 1408 31 us
// (10.2), 8 of 64 of 2048 x 1024 36 us (14.9), 4 tokens, 2 of 8 of 512 x 128 20 us (under 1);
// 64 tokens, 8 of 128 of 1024 x 512 115 us (58.5), pieces of four tokens.  Neither kernel
// starts before the other has ended: each takes all of the shared memory, the second all
// of the tensor memory.
// A TMA copy costs about as much as 2 to 4 KB of data, whatever its size: with boxes of
// eight rows alone the first took 148 us.  Clusters of two instead of four fill all 152
// multiprocessors (four: 144) but read W_router twice as often: 16 to 30 % slower.
#include <cudaTypedefs.h>

#include <atomic>
#include <mutex>

#include "common.cuh"
#include "kernels.h"
#include "few.h"

namespace moe {

namespace {

constexpr int kThreads = 224;          // TMA, MMA, four warps of the epilogue, MMA
constexpr int kEpi = 128;
constexpr int kCluster = 4;
constexpr int kMaxSteps = 8;           // times 64 columns of a stage
constexpr int kStageBytes = 36 * 1024;   // 128 columns of 128 rows of weights and of 16 tokens
constexpr int kMaxStages = 6, kRouterStages = 16;
// Columns of an accumulator: tokens of an expert, in the down kernel two for each.
constexpr int kUpCols = MOE_FEW_MAX_TOKENS, kDownCols = 2 * MOE_FEW_MAX_TOKENS;
constexpr int kIssuers = 2;            // threads that issue MMAs, stage by stage in turn, each with its accumulators
constexpr int kAccs = 2;               // accumulators: one is multiplied into while the other is read
static_assert(kAccs * kIssuers * kDownCols <= 512, "tensor memory");

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
// 64 columns of rows, several times: {column of 64, row, which 64 columns}.
MOE_DEV void tma_box3(uint32_t dst, const CUtensorMap* map, uint64_t* bar, int x, int y, int z) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(x), "r"(y), "r"(z)
      : "memory");
}
MOE_DEV void st_cluster(uint32_t addr, float v) {
  asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(addr), "f"(v) : "memory");
}
MOE_DEV void or_cluster(uint32_t addr, uint32_t v) {
  asm volatile("red.relaxed.cluster.shared::cluster.or.b32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}
MOE_DEV float4 ld_cluster4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(addr) : "memory");
  return v;
}
MOE_DEV void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
MOE_DEV void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }

// Boxes of 8, 16, 32, 64 (and 128) rows: a run of groups of eight rows is as many copies
// as its number has bits.
struct UpMaps {
  CUtensorMap gate[4], up[4], rows, x, router[2];
};
struct DownMaps {
  CUtensorMap down[5], act[5];
  CUtensorMap down4, act2[2], act4[2];   // eight rows (act: or 16), two or four times 64 columns
};
// Row groups in front of the box of 2^b groups of a run of n.
MOE_DEV int box_before(int n, int b) { return n & ~((2 << b) - 1); }

// More tokens than this are all tokens' rows in one copy, not four rows a copy.
constexpr int kGather = 16;

struct Ctl {
  uint64_t full[kMaxStages], empty[kMaxStages];
  uint64_t rfull[kRouterStages], rempty[kRouterStages];
  uint64_t tfull[2], tempty[2];
  uint64_t fin;
  uint32_t tmem;
  int abort;
  int cols;                   // of an accumulator
  int n_act;                  // experts with routes
  uint16_t base[257];         // first route of an active expert, in their order
  uint8_t act[256];           // their experts
};
struct UpCtl : Ctl {
  uint32_t mask[256][2];      // tokens of an expert
  uint8_t slot[256];          // expert -> active expert
  uint8_t four[kGather];      // tokens of the piece that is being loaded
  float up[64][17];           // sixteen tokens' up products
};
struct DownCtl : Ctl {
  uint8_t tok[kFewMaxRoutes];   // token of a route
  float gate[kFewMaxRoutes];    // its gate
};

// Shared memory.  An MMA reads 64 or 128 rows (8 or 16 KB) from where its rows begin,
// however few of them are weights: what lies behind the last stage has to be the CTA's.
constexpr int kOverread = 16 * 1024, kSumBytes = MOE_FEW_MAX_TOKENS * 512;
constexpr int kStages = kMaxStages, kRingBytes = kStages * kStageBytes;
constexpr int kDownStages = 5, kDownRingBytes = kDownStages * kStageBytes;
constexpr int kUpSmem = kRingBytes + (int)sizeof(UpCtl);
constexpr int kDownSmem = kDownRingBytes + kSumBytes + (int)sizeof(DownCtl);
static_assert(kUpSmem <= 227 * 1024 && kDownSmem <= 227 * 1024 && kSumBytes >= kOverread, "shared memory of a CTA");
// up: s rows' parts of `a` bytes end s b bytes before the stage's end and s (a + b) <= the
// stage, so that the last one begins 12 KB before it at least (a = 4 KB, s = 7)
static_assert(sizeof(UpCtl) >= 4096, "what an MMA reads behind the up kernel's ring");
// a wide stage has at most seven groups, 4 KB apart, and its MMAs read eight: from the
// fourth step of the last stage on, (3 + 29) KB
static_assert((kDownStages - 1) * kStageBytes + 32 * 1024 <= kDownSmem, "what an MMA reads behind the down kernel's ring");
// the router's parts (16 KB at least, for its MMAs) leave two stages of (16 + 8) KB
static_assert(kRingBytes - MOE_FEW_MAX_TOKENS * 256 * 4 >= 2 * 24 * 1024, "the router's stages");

// From the masks (complete, behind a barrier): the active experts in ascending order and
// where their routes begin.  Ends in a barrier.
MOE_DEV void build_lists(UpCtl& s, const FewParams& p) {
  const int lane = threadIdx.x;
  if (lane < 32) {   // eight experts a lane
    int routes[8], n = 0, act = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      routes[i] = __popc(s.mask[lane * 8 + i][0]) + __popc(s.mask[lane * 8 + i][1]);
      n += routes[i];
      act += routes[i] > 0;
    }
    int both = n << 16 | act;   // at most 2048 routes, 256 experts
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int before = __shfl_up_sync(0xffffffffu, both, off);
      if (lane >= off) both += before;
    }
    int at = both >> 16, a = both & 0xFFFF;
    if (lane == 31) {
      s.n_act = a;
      s.base[a] = (uint16_t)at;
    }
    at -= n;
    a -= act;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if (routes[i]) {
        s.act[a] = (uint8_t)(lane * 8 + i);
        s.slot[lane * 8 + i] = (uint8_t)a;
        s.base[a] = (uint16_t)at;
        at += routes[i];
        ++a;
      }
    }
  }
  __syncthreads();
}

// One CTA, its epilogue's threads: the lists for the down kernel.  Routes of an expert
// are in the tokens' order; one that a token names twice is one route with the sum of
// its gates.
MOE_DEV void write_lists(const UpCtl& s, const FewParams& p) {
  const int tid = threadIdx.x - 64;
  FewLists& l = *p.lists;
  if (tid == 0) l.n_act = s.n_act;
  for (int a = tid; a <= s.n_act; a += kEpi) {
    l.base[a] = s.base[a];
    if (a < s.n_act) l.act[a] = s.act[a];
  }
  for (int r = tid; r < p.T * p.k; r += kEpi) {
    const int t = r / p.k, e = p.topk_idx[r];
    if (e == -1) continue;
    if (e < 0 || e >= p.E) {
      raise_error(p.err, MOE_DEVERR_BOUNDS);
      continue;
    }
    bool first = true;
    for (int i = t * p.k; i < r; ++i) first = first && p.topk_idx[i] != e;
    if (!first) continue;
    float g = 0.0f;
    for (int i = r; i < (t + 1) * p.k; ++i)
      if (p.topk_idx[i] == e) g += p.gates[i];
    int at = s.base[s.slot[e]] + __popc(s.mask[e][t >> 5] & ((1u << (t & 31)) - 1u));
    if (t >= 32) at += __popc(s.mask[e][0]);
    l.tok[at] = (uint8_t)t;
    l.gate[at] = g;
  }
}

// Floats as unsigned numbers in the same order; 0 is below all of them.
MOE_DEV uint32_t ordered(float v) {
  const uint32_t b = __float_as_uint(v);
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}
MOE_DEV float unordered(uint32_t b) { return __uint_as_float(b & 0x80000000u ? b & 0x7FFFFFFFu : ~b); }

// The k largest of a token's E logits and their gates, as the layer's routing ranks
// them: larger first, lower expert first among equals, a NaN below everything; the
// gates' sum over 32 lanes in the butterfly's order.  `logit` gives expert e's; `put`
// takes lane j's choice j.
template <typename Logit, typename Put>
MOE_DEV void rank_token(const FewParams& p, int t, bool write, Logit logit, Put put) {
  const int lane = threadIdx.x & 31;
  uint32_t key[8];
  bool bad = false;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    key[i] = 0u;
    const int e = lane + 32 * i;
    if (32 * i < p.E && e < p.E) {
      const float v = logit(e);
      if (write && p.logits) p.logits[(size_t)t * p.E + e] = v;
      bad = bad || !isfinite(v);
      // both zeros are one value: the lower expert goes first among them
      key[i] = ordered(v != v ? -INFINITY : v == 0.0f ? 0.0f : v);
    }
  }
  bad = __any_sync(0xffffffffu, bad);
  float mine = 0.0f, top = 0.0f;
  int id = 0;
  for (int j = 0; j < p.k; ++j) {
    uint32_t best = 0u;
    int e = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if (32 * i < p.E && key[i] > best) {
        best = key[i];
        e = lane + 32 * i;
      }
    }
    const uint32_t max = __reduce_max_sync(0xffffffffu, best);
    e = (int)__reduce_min_sync(0xffffffffu, best == max ? (uint32_t)e : 0xFFFFFFFFu);
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (e == lane + 32 * i) key[i] = 0u;
    if (j == 0) top = unordered(max);
    if (lane == j) {
      mine = unordered(max);
      id = e;
    }
  }
  if (lane < p.k) put(lane, id);
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
MOE_DEV void begin(Ctl& s, const FewParams& p, int cols) {
  pdl_launch_dependents();
  if (threadIdx.x == 0) {
    for (int i = 0; i < kMaxStages; ++i) {
      mbar_init(&s.full[i], 1);
      mbar_init(&s.empty[i], 1);
    }
    for (int i = 0; i < kRouterStages; ++i) {
      mbar_init(&s.rfull[i], 1);
      mbar_init(&s.rempty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&s.tfull[i], kIssuers);
      mbar_init(&s.tempty[i], kEpi);
    }
    mbar_init(&s.fin, kIssuers);
    s.abort = 0;
    s.cols = cols;
    fence_barrier_init();
  }
  pdl_wait();
  if (threadIdx.x / 32 == 1) tmem_alloc(&s.tmem, kAccs * kIssuers * cols);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
}

// The stages and where a role stands in them.
struct Ring {
  uint64_t *full, *empty;
  uint32_t base;
  int bytes, stages, stage = 0;
  uint32_t phase = 0;
  long issued = 0;
  MOE_DEV Ring(uint64_t* full_, uint64_t* empty_, const void* smem, int bytes_, int stages_)
      : full(full_), empty(empty_), base(smem_u32(smem)), bytes(bytes_), stages(stages_) {}
  MOE_DEV uint32_t at() const { return base + (uint32_t)(stage * bytes); }
  MOE_DEV void next() {
    ++issued;
    if (++stage == stages) {
      stage = 0;
      phase ^= 1u;
    }
  }
};

// How a piece of rows fills its stages: `s` times 64 columns, the weights' rows of each
// behind one another, then the tokens'.  `wide`: a full stage holds s times 64 columns of
// each group of eight rows behind one another (a copy for each group).
struct Fill {
  int s;
  uint32_t a, b;   // bytes of 64 columns
  bool wide = false;
  MOE_DEV Fill(uint32_t a_, uint32_t b_) : s(max(1, min(kMaxSteps, kStageBytes / (int)(a_ + b_)))), a(a_), b(b_) {}
};

// One warp: the next free stage, its copies announced.
MOE_DEV bool claim(Ctl& s, const FewParams& p, const Ring& r, uint32_t bytes) {
  const bool ok = __all_sync(0xffffffffu, mbar_wait(&r.empty[r.stage], r.phase ^ 1u, &s.abort, p.err));
  if (ok && (threadIdx.x & 31) == 0) mbar_arrive_expect_tx(&r.full[r.stage], bytes);
  __syncwarp();
  return ok;
}
// The producer gave up: the copies that it announced land first.
MOE_DEV void drain(const Ring& r) {
  for (long i = r.issued > r.stages ? r.issued - r.stages : 0; i < r.issued; ++i) {
    const uint32_t bar = smem_u32(&r.full[(int)(i % r.stages)]);
    const uint64_t t0 = globaltimer();
    while (!mbar_try_wait(bar, (uint32_t)((i / r.stages) & 1)))
      if (globaltimer() - t0 > kWaitLimitNs) break;
  }
}

// The words of smem_desc_sw128(address, 16, group).
MOE_DEV uint32_t desc_lo(uint32_t address) { return (address & 0x3FFFFu) >> 4 | 1u << 16; }
MOE_DEV uint32_t desc_hi(uint32_t group) { return group >> 4 | 1u << 14 | 2u << 29; }

// Four MMAs: 64 columns of K.
MOE_DEV void mma_64(uint32_t d, uint32_t a_lo, uint32_t a_hi, uint32_t b_lo, uint32_t b_hi, uint32_t idesc, bool accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, t;\n\t.reg .b64 a0, a1, a2, a3, b0, b1, b2, b3;\n\t.reg .b32 x, y;\n\t"
      "setp.ne.b32 p, %6, 0;\n\tsetp.eq.b32 t, 0, 0;\n\t"
      "mov.b64 a0, {%1, %2};\n\tmov.b64 b0, {%3, %4};\n\t"
      "add.u32 x, %1, 2;\n\tadd.u32 y, %3, 2;\n\tmov.b64 a1, {x, %2};\n\tmov.b64 b1, {y, %4};\n\t"
      "add.u32 x, %1, 4;\n\tadd.u32 y, %3, 4;\n\tmov.b64 a2, {x, %2};\n\tmov.b64 b2, {y, %4};\n\t"
      "add.u32 x, %1, 6;\n\tadd.u32 y, %3, 6;\n\tmov.b64 a3, {x, %2};\n\tmov.b64 b3, {y, %4};\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], a0, b0, %5, p;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], a1, b1, %5, t;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], a2, b2, %5, t;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], a3, b3, %5, t;\n\t}" ::"r"(d),
      "r"(a_lo), "r"(a_hi), "r"(b_lo), "r"(b_hi), "r"(idesc), "r"((uint32_t)accumulate)
      : "memory");
}

// One of the issuers: `chunks` times 64 columns multiplied into its columns of
// accumulator `it`.  A stage of the ring belongs to one issuer for good, the even ones to
// the first: its barriers' phases are waited for by one thread, none of them left out.
// An MMA takes 57 cycles of the thread that issues it, whatever its shape up to 64
// columns; with two threads one takes 28 (64 rows) and 39 (128).
MOE_DEV bool multiply(Ctl& s, const FewParams& p, Ring& r, int issuer, int it, const Fill& fill, int chunks, int rows, int n) {
  const int acc = it & 1;
  if (!mbar_wait(&s.tempty[acc], ((uint32_t)(it >> 1) & 1u) ^ 1u, &s.abort, p.err)) return false;
  tc_fence_after();
  const uint32_t d = s.tmem + (acc * kIssuers + issuer) * s.cols, idesc = idesc_bf16_f32(rows <= 64 ? 64 : 128, n, 0, 0);
  bool started = false;
  for (int c = 0; c < chunks; c += fill.s) {
    if (r.stage % kIssuers != issuer) {
      r.next();
      continue;
    }
    if (!mbar_wait(&r.full[r.stage], r.phase, &s.abort, p.err)) return false;
    tc_fence_after();
    const uint32_t a = r.at(), b = a + fill.s * fill.a;
    const bool wide = fill.wide && c + fill.s <= chunks;
    const uint32_t step = wide ? 1024 : fill.a, group = wide ? fill.s * 1024 : 1024;
    const uint32_t a_hi = desc_hi(group), b_hi = desc_hi(1024);
    uint32_t a_lo = desc_lo(a), b_lo = desc_lo(b);
    for (int q = 0; q < fill.s && c + q < chunks; ++q, a_lo += step >> 4, b_lo += fill.b >> 4) {
      mma_64(d, a_lo, a_hi, b_lo, b_hi, idesc, started);
      started = true;
    }
    tc_commit(&r.empty[r.stage]);
    r.next();
  }
  tc_commit(&s.tfull[acc]);
  return true;
}
// Which of the issuers (bits) had a stage of a piece; the ring's place moves past it.
MOE_DEV int issuers_of(int& stage, int stages, const Fill& fill, int chunks) {
  const int n = (chunks + fill.s - 1) / fill.s;
  int had = 0;
  for (int i = 0, at = stage; i < min(n, 3); ++i, at = at + 1 < stages ? at + 1 : 0) had |= 1 << at % kIssuers;
  stage = (stage + n) % stages;
  return had;
}
static_assert(kIssuers == 2, "of three stages in a row two are different issuers'");

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

// The row that a thread of the epilogue holds of an accumulator with `rows` rows (-1:
// none): a lane each, or of an MMA of 64 rows sixteen lanes of each warp.
MOE_DEV int row_of(int rows) {
  const int warp = (int)(threadIdx.x >> 5) & 3, lane = (int)(threadIdx.x & 31);
  const int row = rows > 64 ? warp * 32 + lane : lane < 16 ? warp * 16 + lane : rows;
  return row < rows ? row : -1;
}
// Sixteen columns of an accumulator of `cols`: the sum of the issuers that had a part.
MOE_DEV void sum16(uint32_t taddr, int cols, int issuers, float* v) {
  tmem_ld16(taddr + (issuers & 1 ? 0 : cols), v);
  if (issuers == 3) {
    float w[16];
    tmem_ld16(taddr + cols, w);
#pragma unroll
    for (int j = 0; j < 16; ++j) v[j] += w[j];
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
    tmem_dealloc(s.tmem, kAccs * kIssuers * s.cols);
  }
}

// Where share i of n begins, floor(total i / n): whole experts where they divide the CTAs
// evenly.  64 bits (a slow division) only where 32 do not hold the product.
MOE_DEV int share(int total, int i, int n) {
  return total < (1 << 23) ? (int)((uint32_t)total * (uint32_t)i / (uint32_t)n) : (int)((int64_t)total * i / n);
}
MOE_DEV int round16(int n) { return (n + 15) & ~15; }

// The next rows of a share of (active expert, group of eight d_ff rows): at most eight
// groups of one expert.
struct UpPiece {
  int a, g, n;   // active expert, first group, groups
  MOE_DEV bool next(int& from, int to, int groups) {
    if (from >= to) return false;
    a = from / groups;
    g = from - a * groups;
    n = min(8, min(to, (a + 1) * groups) - from);
    from += n;
    return true;
  }
};

// Where CTA i's share begins.  Not one or two groups beside an expert's end: they would be
// a piece of their own, of many small copies (1 token, 8 experts of 4096 x 2048: the last
// of 144 CTAs 63 us after the start, the median 53).
MOE_DEV int up_share(int total, int groups, int i) {
  const int at = share(total, i, gridDim.x), r = at % groups, near = min(2, total / ((int)gridDim.x * 4));
  return r <= near ? at - r : groups - r <= near ? at + groups - r : at;
}

// Columns of the MMA for an expert of m tokens; how n groups of gate and of up rows and
// these tokens fill a stage.
MOE_DEV int up_columns(const FewParams& p, int m) { return m > kGather ? p.t_pad : round16(m); }
MOE_DEV Fill up_fill(const FewParams& p, int n, int m) {
  return Fill(n * 2048, m > kGather ? p.t_pad * 128 : (m + 7) / 8 * 1024);
}

__global__ void __launch_bounds__(kThreads, 1)
    few_up_kernel(const __grid_constant__ UpMaps maps, const FewParams p) {
  extern __shared__ __align__(1024) uint8_t smem[];
  UpCtl& s = *reinterpret_cast<UpCtl*>(smem + kRingBytes);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int issuer = warp == 1 ? 0 : warp == 6 ? 1 : -1;
  const int quarter = warp & 3, row = quarter * 32 + lane;   // of the epilogue's threads
  const bool writer = (int)blockIdx.x >= (int)gridDim.x - kCluster;   // the cluster that writes the routing
  for (int i = threadIdx.x; i < 512; i += kThreads) (&s.mask[0][0])[i] = 0u;
  begin(s, p, kUpCols);
  const uint32_t tmem = s.tmem + ((uint32_t)(quarter * 32) << 16);
  const int chunks = p.d / 64;
  Ring ring(s.full, s.empty, smem, kStageBytes, kStages), first(s.rfull, s.rempty, smem, p.router_bytes, p.router_stages);
  int it = 0;   // accumulators used so far
  bool ok = true;
  if (p.router) {
    cluster_arrive();
    const int rank = (int)cluster_ctarank(), own = (p.T + kCluster - 1) / kCluster;
    const int c0 = share(chunks, rank, kCluster), c1 = share(chunks, rank + 1, kCluster), tiles = (p.E + 127) / 128;
    const uint32_t a_bytes = (uint32_t)(min(p.E, 128) + 7) / 8 * 1024, b_bytes = (uint32_t)p.router_bytes - a_bytes;
    Fill fill(a_bytes, b_bytes);
    fill.s = 1;
    if (warp == 0) {
      for (int m = 0; m < tiles && ok; ++m) {
        const int rows = min(p.E - m * 128, 128);
        for (int c = c0; c < c1; ++c) {
          ok = claim(s, p, first, (rows + p.T) * 128);
          if (!ok) break;
          if (lane == 0) tma_box(first.at(), &maps.router[m], &first.full[first.stage], c * 64, m * 128);
          if (lane == 1) tma_box(first.at() + a_bytes, &maps.x, &first.full[first.stage], c * 64, 0);
          first.next();
        }
      }
      if (!ok && lane == 0) drain(first);
    } else if (issuer >= 0) {
      if (lane == 0)
        for (int m = 0; m < tiles && ok; ++m) ok = multiply(s, p, first, issuer, m, fill, c1 - c0, 128, p.t_pad);
    } else {
      for (int m = 0; m < tiles; ++m) ok = results(s, p, m) && ok;
    }
    __syncwarp();
    cluster_wait();   // every CTA of the cluster has begun
    // the part of this CTA's columns to the CTA that ranks the token: [source, its
    // token, expert] behind the stages
    if (warp >= 2 && issuer < 0) {
      const uint32_t mine = smem_u32(smem + p.part_at) + (uint32_t)(rank * own * p.E) * 4u;
      for (int m = 0, at = 0; m < tiles; ++m) {
        const int e = m * 128 + row, issuers = issuers_of(at, p.router_stages, fill, c1 - c0);
        for (int c = 0; c < p.T; c += 16) {
          float v[16];
          if (c1 > c0) sum16(tmem + m * kIssuers * kUpCols + c, kUpCols, issuers, v);
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            const int t = c + i;
            if (t < p.T && e < p.E)
              st_cluster(mapa_shared(mine + (uint32_t)(t / kCluster * p.E + e) * 4u, t % kCluster), c1 > c0 ? v[i] : 0.0f);
          }
        }
        release(s, m);
      }
    }
    it = tiles;
    __syncwarp();
    cluster_sync();   // the parts are there
    const float* part = reinterpret_cast<const float*>(smem + p.part_at);
    for (int i = warp; rank + i * kCluster < p.T; i += kThreads / 32) {
      const int t = rank + i * kCluster;
      rank_token(
          p, t, writer,
          [&](int e) {
            float v = 0.0f;
#pragma unroll
            for (int q = 0; q < kCluster; ++q) v += part[(q * own + i) * p.E + e];
            return p.bias ? v + p.bias[(size_t)t * p.E + e] : v;
          },
          [&](int j, int e) {
            const uint32_t to = smem_u32(&s.mask[e][t >> 5]);
#pragma unroll
            for (int q = 0; q < kCluster; ++q) or_cluster(mapa_shared(to, q), 1u << (t & 31));
          });
    }
    fence_proxy_async_smem();   // the ring was written and read by threads
    __syncwarp();
    cluster_sync();   // and the routing
  } else {
    for (int r = threadIdx.x; r < p.T * p.k; r += kThreads) {
      const int e = p.topk_idx[r], t = r / p.k;   // others than [0, E): write_lists
      if (e >= 0 && e < p.E) atomicOr(&s.mask[e][t >> 5], 1u << (t & 31));
    }
    __syncthreads();
  }
  build_lists(s, p);

  const int groups = p.f / 8;
  const int total = s.n_act * groups;
  int g = up_share(total, groups, blockIdx.x);
  const int g_end = up_share(total, groups, blockIdx.x + 1);
  UpPiece u;
  if (warp == 0) {
    while (ok && u.next(g, g_end, groups)) {
      const int e = s.act[u.a], m = s.base[u.a + 1] - s.base[u.a];
      // lanes 0-3: gate rows, lanes 4-7: the up rows behind them; lanes 8-11: four tokens
      // each, or lane 8: all tokens
      const Fill fill = up_fill(p, u.n, m);
      const bool all = m > kGather;
      if (!all) {   // the expert's tokens in a row
        const uint32_t m0 = s.mask[e][0], m1 = s.mask[e][1], below = (1u << lane) - 1u;
        __syncwarp();
        if (m0 >> lane & 1u) s.four[__popc(m0 & below)] = (uint8_t)lane;
        if (m1 >> lane & 1u) s.four[__popc(m0) + __popc(m1 & below)] = (uint8_t)(lane + 32);
        __syncwarp();
      }
      const int b = lane & 3, before = box_before(u.n, b), i = (lane - 8) * 4;
      const bool weights = lane < 8 && (u.n >> b & 1), four = !all && lane >= 8 && lane < 12 && i < m;
      const CUtensorMap* map = lane < 4 ? &maps.gate[b] : &maps.up[b];
      const uint32_t place = lane < 8 ? (before + (lane < 4 ? 0 : u.n)) * 1024u : fill.s * fill.a + (lane - 8) * 512u;
      const uint32_t step = lane < 8 ? fill.a : fill.b;
      const uint32_t bytes = u.n * 2048 + (all ? p.T * 128 : (m + 3) / 4 * 512);
      const int y = e * p.f + (u.g + before) * 8;
      int y0 = 0, y1 = 0, y2 = 0, y3 = 0;
      if (four) {
        y0 = s.four[i];
        y1 = s.four[min(i + 1, m - 1)];
        y2 = s.four[min(i + 2, m - 1)];
        y3 = s.four[min(i + 3, m - 1)];
      }
      for (int c = 0; c < chunks; c += fill.s) {
        const int n = min(fill.s, chunks - c);
        ok = claim(s, p, ring, n * bytes);
        if (!ok) break;
        uint32_t to = ring.at() + place;
        for (int q = c; q < c + n; ++q, to += step) {
          if (weights) tma_box(to, map, &ring.full[ring.stage], q * 64, y);
          if (four) tma_gather4(to, &maps.rows, &ring.full[ring.stage], q * 64, y0, y1, y2, y3);
          if (all && lane == 8) tma_box(to, &maps.x, &ring.full[ring.stage], q * 64, 0);
        }
        ring.next();
      }
    }
    if (!ok && lane == 0) drain(ring);
  } else if (issuer >= 0) {
    if (lane == 0) {
      while (ok && u.next(g, g_end, groups)) {
        const int m = s.base[u.a + 1] - s.base[u.a];
        ok = multiply(s, p, ring, issuer, it++, up_fill(p, u.n, m), chunks, u.n * 16, up_columns(p, m));
      }
      finish(s, p);
    }
  } else {
    // the first 8 n lanes hold gate rows, the next 8 n the up rows, which change hands
    // sixteen tokens at a time
    __nv_bfloat16* act = static_cast<__nv_bfloat16*>(p.act);
    int at_stage = 0;
    if (blockIdx.x == gridDim.x - 1) write_lists(s, p);
    while (ok && u.next(g, g_end, groups)) {
      ok = bar_and(1, kEpi, results(s, p, it));
      if (!ok) break;
      const int e = s.act[u.a], r0 = s.base[u.a], m = s.base[u.a + 1] - r0, columns = m > kGather ? p.T : m;
      const uint32_t m0 = s.mask[e][0], m1 = s.mask[e][1];
      const int rows = u.n * 8, row = row_of(2 * rows), issuers = issuers_of(at_stage, kStages, up_fill(p, u.n, m), chunks);
      const size_t col = (size_t)u.g * 8 + row;
      for (int c = 0; c < columns; c += 16) {
        float v[16];
        sum16(tmem + (it & 1) * kIssuers * kUpCols + c, kUpCols, issuers, v);
        if (row >= rows) {
#pragma unroll
          for (int i = 0; i < 16; ++i) s.up[row - rows][i] = v[i];
        }
        bar_sync(1, kEpi);
        if (row >= 0 && row < rows) {
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            const int t = c + i;
            int at = t;   // the route of this column
            bool in = t < m;
            if (m > kGather) {
              in = (t < 32 ? m0 >> t : m1 >> (t - 32)) & 1u;
              at = t < 32 ? __popc(m0 & ((1u << t) - 1u)) : __popc(m0) + __popc(m1 & ((1u << (t - 32)) - 1u));
            }
            if (in && t < columns) {
              // the fast exponential and quotient, as the layer's own: off by 2 + 1.2 |h| and
              // two last places, less than what the sum before them was cut off by
              const float a = __fdividef(v[i], 1.0f + __expf(-v[i])) * s.up[row][i];
              const __nv_bfloat16 high = __float2bfloat16_rn(a);
              const float rest = a - __bfloat162float(high);
              __nv_bfloat16* to = act + (size_t)(r0 + at) * 2 * p.f + col;
              to[0] = high;
              to[p.f] = __float2bfloat16_rn(fabsf(rest) < INFINITY ? rest : 0.0f);
            }
          }
        }
        bar_sync(1, kEpi);
      }
      release(s, it++);
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

// The box of 8 << b rows that holds the activations of m routes, two rows each; how n
// groups of rows of weights and these fill a stage.
MOE_DEV int route_box(int m) { return m <= 4 ? 0 : m <= 8 ? 1 : m <= 16 ? 2 : m <= 32 ? 3 : 4; }
MOE_DEV Fill down_fill(int n, int m) {
  Fill f(n * 1024, 1024 << route_box(m));
  if (m <= 8 && n >= 4 && n <= 8 && 4 * (f.a + f.b) <= kStageBytes) {   // fewer and larger copies
    f.s = 4;
    f.wide = n < 8;
  }
  return f;
}

#ifdef MOE_CHECKS
// What the up kernel has listed, before it becomes rows of copies and places of sums; a list
// with a wrong entry is taken as empty.
MOE_DEV void check_lists(DownCtl& s, const FewParams& p) {
  if (threadIdx.x == 0) {
    const int R = p.T * p.k;
    bool ok = MOE_CHECK_OK(s.n_act, min(p.E, R) + 1);
    for (int a = 0; ok && a < s.n_act; ++a)
      ok = MOE_CHECK_OK(s.act[a], p.E) && MOE_CHECK_OK(s.base[a + 1], R + 1) &&
           MOE_CHECK_OK(s.base[a + 1] - s.base[a] - 1, p.T);
    for (int r = 0; ok && r < (s.n_act ? s.base[s.n_act] : 0); ++r) ok = MOE_CHECK_OK(s.tok[r], p.T);
    if (!ok) s.n_act = 0;
  }
  __syncthreads();
}
#endif

__global__ void __launch_bounds__(kThreads, 1)
    few_down_kernel(const __grid_constant__ DownMaps maps, const FewParams p) {
  extern __shared__ __align__(1024) uint8_t smem[];
  float* sums = reinterpret_cast<float*>(smem + kDownRingBytes);   // [T][128]
  DownCtl& s = *reinterpret_cast<DownCtl*>(smem + kDownRingBytes + kSumBytes);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int issuer = warp == 1 ? 0 : warp == 6 ? 1 : -1;
  const int quarter = warp & 3;
  begin(s, p, kDownCols);
  {   // what the up kernel has listed, all of it at once
    const FewLists& l = *p.lists;
    const int R = p.T * p.k, most = min(p.E, R);
    if (threadIdx.x == 0) s.n_act = l.n_act;
    for (int i = threadIdx.x; i <= most; i += kThreads) s.base[i] = l.base[i];
    for (int i = threadIdx.x; i < most; i += kThreads) s.act[i] = l.act[i];
    for (int i = threadIdx.x; i < R; i += kThreads) {
      s.tok[i] = l.tok[i];
      s.gate[i] = l.gate[i];
    }
    for (int i = threadIdx.x; i < p.T * 32; i += kThreads) reinterpret_cast<float4*>(sums)[i] = {};
    __syncthreads();
#ifdef MOE_CHECKS
    check_lists(s, p);
#endif
  }
  const uint32_t tmem = s.tmem + ((uint32_t)(quarter * 32) << 16);
  const int rank = (int)cluster_ctarank(), clusters = gridDim.x / kCluster, cluster = blockIdx.x / kCluster;
  const int chunks = p.f / 64, total = s.n_act * chunks;
  const int from = share(total, rank, kCluster), to = share(total, rank + 1, kCluster);
  const int d0 = share(p.d / 8, cluster, clusters), d1 = share(p.d / 8, cluster + 1, clusters);
  const int tiles = (d1 - d0 + 15) / 16;
  Ring ring(s.full, s.empty, smem, kStageBytes, kDownStages);
  int it = 0, at_stage = 0;
  bool ok = true;
  for (int tile = 0; tile < tiles; ++tile) {   // the same number in every CTA of the cluster
    const int g0 = d0 + share(d1 - d0, tile, tiles), n = d0 + share(d1 - d0, tile + 1, tiles) - g0;
    int c0 = from;
    DownPiece u;
    if (warp == 0) {
      while (ok && u.next(c0, to, chunks)) {
        const int e = s.act[u.a], r0 = s.base[u.a], m = s.base[u.a + 1] - r0;
        // lanes 0-4: rows of weights, lane 8: the routes, the smallest box that holds them
        const Fill fill = down_fill(n, m);
        // (a wide stage: lanes 0-6, a group each)
        const int b = lane < 5 ? lane : 0, before = box_before(n, b), act = route_box(m);
        const bool weights = lane < 5 && (n >> b & 1), routes = lane == 8;
        const bool once = m <= 8 && (fill.s == 2 || fill.s == 4 || fill.s == 8);   // the routes of a full stage in one copy (eight steps: in two)
        const uint32_t place = routes ? fill.s * fill.a : before * 1024u, step = routes ? fill.b : fill.a;
        const CUtensorMap* map = routes ? &maps.act[act] : &maps.down[b];
        const CUtensorMap* many = fill.s == 2 ? &maps.act2[act & 1] : &maps.act4[act & 1];
        const int y = routes ? 2 * r0 : e * p.d + (g0 + before) * 8;
        for (int c = u.c; c < u.c + u.n; c += fill.s) {
          const int steps = min(fill.s, u.c + u.n - c);
          const bool full = steps == fill.s, wide = full && fill.wide, one = full && once;
          ok = claim(s, p, ring, steps * (fill.a + fill.b));
          if (!ok) break;
          const uint32_t at = ring.at();
          uint64_t* bar = &ring.full[ring.stage];
          if (one && routes) {
            tma_box3(at + place, many, bar, 0, y, c);
            if (fill.s == 8) tma_box3(at + place + 4 * step, many, bar, 0, y, c + 4);
          }
          if (wide && lane < n) tma_box3(at + lane * fill.s * 1024u, &maps.down4, bar, 0, e * p.d + (g0 + lane) * 8, c);
          if ((weights && !wide) || (routes && !one)) {
            uint32_t dst = at + place;
            for (int q = c; q < c + steps; ++q, dst += step) tma_box(dst, map, bar, q * 64, y);
          }
          ring.next();
        }
      }
    } else if (issuer >= 0) {
      if (lane == 0)
        while (ok && u.next(c0, to, chunks)) {
          const int m = s.base[u.a + 1] - s.base[u.a];
          ok = multiply(s, p, ring, issuer, it++, down_fill(n, m), u.n, n * 8, round16(2 * m));
        }
    } else {
      while (ok && u.next(c0, to, chunks)) {
        ok = results(s, p, it);
        if (!ok) break;
        const int r0 = s.base[u.a], m = s.base[u.a + 1] - r0, row = row_of(n * 8), issuers = issuers_of(at_stage, kDownStages, down_fill(n, m), u.n);
        for (int c = 0; c < m; c += 8) {   // eight routes: sixteen columns
          float v[16];
          sum16(tmem + (it & 1) * kIssuers * kDownCols + 2 * c, kDownCols, issuers, v);
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            if (c + i < m && row >= 0) {
              float& sum = sums[s.tok[r0 + c + i] * 128 + row];
              sum = fmaf(s.gate[r0 + c + i], v[2 * i] + v[2 * i + 1], sum);
            }
          }
        }
        release(s, it++);
      }
    }
    __syncwarp();
    cluster_sync();   // every CTA's sums are there
    // this CTA's quarter of the rows, four neighbours a thread
    constexpr int fours = 128 / kCluster / 4;
    const uint32_t mine = smem_u32(sums);
    __nv_bfloat16* out = static_cast<__nv_bfloat16*>(p.out);
    for (int i = threadIdx.x; i < fours * p.T; i += kThreads) {
      const int t = i / fours, r = (rank * fours + i % fours) * 4;
      if (r >= n * 8) continue;
      float4 v[kCluster];
#pragma unroll
      for (int q = 0; q < kCluster; ++q) v[q] = ld_cluster4(mapa_shared(mine + (uint32_t)(t * 128 + r) * 4u, q));
      float4 sum = v[0];
#pragma unroll
      for (int q = 1; q < kCluster; ++q) sum = make_float4(sum.x + v[q].x, sum.y + v[q].y, sum.z + v[q].z, sum.w + v[q].w);
      *reinterpret_cast<uint2*>(out + (size_t)t * p.d + g0 * 8 + r) =
          make_uint2(pack_bf16x2(sum.x, sum.y), pack_bf16x2(sum.z, sum.w));
    }
    __syncwarp();
    cluster_sync();   // and have been read
    if (tile + 1 < tiles) {
      for (int i = threadIdx.x; i < p.T * 32; i += kThreads) reinterpret_cast<float4*>(sums)[i] = {};
      __syncthreads();
    }
  }
  if (warp == 0 && !ok && lane == 0) drain(ring);
  if (issuer >= 0 && lane == 0) finish(s, p);
  leave(s);
}

PFN_cuTensorMapEncodeTiled_v12000 g_encode = nullptr;
std::once_flag g_encode_once;

// Tensor map of `outer` rows of `inner` bf16 elements with 128-byte swizzle: boxes of 64
// columns of `box_rows` rows, zeros behind the last row.  `steps` > 0: the rows as
// [inner / 64][outer][64], `steps` times 64 columns in a box, one step behind the other.
bool make_map(CUtensorMap* m, const void* ptr, uint64_t inner, uint64_t outer, uint32_t box_rows, uint32_t steps = 0) {
  std::call_once(g_encode_once, [] {
    void* fn = nullptr;
    cudaDriverEntryPointQueryResult found;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault, &found) == cudaSuccess &&
        found == cudaDriverEntryPointSuccess)
      g_encode = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(fn);
  });
  if (!g_encode) return false;
  const cuuint64_t dims[3] = {steps ? 64 : inner, outer, inner / 64}, strides[2] = {inner * 2, 128};
  const cuuint32_t box[3] = {64, box_rows, steps}, ones[3] = {1, 1, 1};
  return g_encode(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, steps ? 3 : 2, const_cast<void*>(ptr), dims, strides, box, ones,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

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
  p.router = w.w_router != nullptr;
  p.t_pad = p.T <= 16 ? 16 : p.T <= 32 ? 32 : 64;   // rows of the largest box of tokens or routes
  const uint64_t d = (uint64_t)p.d, f = (uint64_t)p.f, E = (uint64_t)p.E;
  const uint64_t routes = ((uint64_t)p.T * p.k * 2 + 7) / 8 * 8;   // rows of activations
  // the router's stages in front of the parts of its products
  p.router_bytes = ((p.E < 128 ? p.E : 128) + 7) / 8 * 1024 + (p.T + 7) / 8 * 1024;
  const int parts = kCluster * ((p.T + kCluster - 1) / kCluster) * p.E * 4;
  p.part_at = (kRingBytes - (parts > kOverread ? parts : kOverread)) / 1024 * 1024;
  p.router_stages = p.part_at / p.router_bytes < kRouterStages ? p.part_at / p.router_bytes : kRouterStages;
  UpMaps up;
  DownMaps down;
  const void* wr = p.router ? w.w_router : w.w_gate;   // a map that is not used is one all the same
  bool made = make_map(&up.rows, w.x, d, (uint64_t)p.T, 1) &&
              make_map(&up.x, w.x, d, (uint64_t)p.T, (uint32_t)p.T) &&
              make_map(&up.router[0], wr, d, p.router ? E : E * f, p.E < 128 ? p.E : 128) &&
              make_map(&up.router[1], wr, d, p.router ? E : E * f, p.E > 128 ? p.E - 128 : 1);
  for (int b = 0; b < 5; ++b) {
    const uint32_t height = 8u << b;
    made = made && make_map(&down.down[b], w.w_down, f, E * d, height) &&
           make_map(&down.act[b], p.act, f, routes, height);
    if (b < 4)
      made = made && make_map(&up.gate[b], w.w_gate, d, E * f, height) &&
             make_map(&up.up[b], w.w_up, d, E * f, height);
    if (b < 2)
      made = made && make_map(&down.act2[b], p.act, f, routes, height, 2) &&
             make_map(&down.act4[b], p.act, f, routes, height, 4);
  }
  made = made && make_map(&down.down4, w.w_down, f, E * d, 8, 4);
  if (!made) return cudaErrorInvalidValue;
  static SmemLimit up_limit, down_limit;
  cudaError_t e = up_limit.raise(reinterpret_cast<const void*>(&few_up_kernel), kUpSmem);
  if (e == cudaSuccess) e = down_limit.raise(reinterpret_cast<const void*>(&few_down_kernel), kDownSmem);
  if (e != cudaSuccess) return e;
  const int ctas = resident_ctas(reinterpret_cast<const void*>(&few_up_kernel), kUpSmem, dev->index);
  if (ctas == 0) return cudaErrorInvalidConfiguration;
  e = launch_clusters(&few_up_kernel, ctas, kUpSmem, s, up, p);
  if (e != cudaSuccess) return e;
  return launch_clusters(&few_down_kernel, ctas, kDownSmem, s, down, p);
}

MOE_CHECK_WORD_ACCESSOR(few)

}  // namespace moe
