// 4-bit weights with group scales (sm_103a): the stream of weights that the
// products with a few vectors are made of.
//
//   W[n, k] = (code[n, k] - 8) * scale[n, k / G],   G = 32, 64 or 128
// Two codes a byte, the even column in the low nibble; row-major, so one row of
// K columns is K/2 contiguous bytes.
//
// Bound by the weights' bytes: every weight is read once and used for a handful
// of vectors.  The products run on mma.sync m16n8k16 with 16 weight rows as A
// and eight vectors as B: the tensor core only has to keep up with HBM here, and
// the fragment form lets each lane turn its 4-bit words into operands itself.
// What comes next to bounding it is that conversion (two logic operations and
// one subtraction for two weights, a third of the issue slots at full HBM rate).
// The sum over k may visit columns in any order as long as A and B agree, so a
// lane's fragment columns are simply those of the words it holds.  Products of
// a group are exact integers times activations, summed in fp32; the group's
// scale multiplies the fp32 sum.
//
// One block of 16 warps runs on each SM and takes an equal share of the tiles;
// its warps split the share's (tile, stage) pairs evenly, whatever the number
// of tiles, and add up a tile's parts in shared memory in a fixed order.
#pragma once

#include "block.cuh"
#include "block.h"
#include "kernels.h"

namespace moe {

constexpr int kW4Warps = 16;
constexpr int kW4Threads = kW4Warps * 32;

// ------------------------------------------------------------------ fragments
// widen(w, a): the eight codes of a word as four register pairs, a[q] = the
// codes of columns (q, q + 4) minus 8, exactly.
MOE_DEV uint32_t and_or(uint32_t a, uint32_t b, uint32_t c) {   // (a & b) | c, one operation
  uint32_t r;
  asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(r) : "r"(a), "r"(b), "r"(c));
  return r;
}

template <typename T> struct MmaT;
template <> struct MmaT<__nv_bfloat16> {
  // a nibble in the low mantissa bits of 128 (0x4300) is 128 + code
  static MOE_DEV void widen(uint32_t w, uint32_t* a) {
    const __nv_bfloat162 off = __floats2bfloat162_rn(136.0f, 136.0f);
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      uint32_t v = and_or(w >> (4 * q), 0x000F000Fu, 0x43004300u);
      __nv_bfloat162 h = __hsub2(*reinterpret_cast<__nv_bfloat162*>(&v), off);
      a[q] = *reinterpret_cast<uint32_t*>(&h);
    }
  }
  static MOE_DEV void mma(float* c, const float* z, uint32_t a0, uint32_t a1, uint32_t a2,
                          uint32_t a3, uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
        "{%8, %9}, {%10, %11, %12, %13};"
        : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(z[0]), "f"(z[1]), "f"(z[2]), "f"(z[3]));
  }
};
template <> struct MmaT<__half> {
  // 1024 (0x6400) holds a nibble in bits 0-3 as 1024 + code, in bits 4-7 as
  // 1024 + 16 code: one shift serves four pairs
  static MOE_DEV void widen(uint32_t w, uint32_t* a) {
    const __half2 off = __floats2half2_rn(1032.0f, 1032.0f);
    const __half2 sc = __floats2half2_rn(0.0625f, 0.0625f), off16 = __floats2half2_rn(-72.0f, -72.0f);
#pragma unroll
    for (int q = 0; q < 4; q += 2) {
      const uint32_t u = w >> (4 * q);
      uint32_t v = and_or(u, 0x000F000Fu, 0x64006400u);
      uint32_t v16 = and_or(u, 0x00F000F0u, 0x64006400u);
      __half2 h = __hsub2(*reinterpret_cast<__half2*>(&v), off);
      __half2 h16 = __hfma2(*reinterpret_cast<__half2*>(&v16), sc, off16);
      a[q] = *reinterpret_cast<uint32_t*>(&h);
      a[q + 1] = *reinterpret_cast<uint32_t*>(&h16);
    }
  }
  static MOE_DEV void mma(float* c, const float* z, uint32_t a0, uint32_t a1, uint32_t a2,
                          uint32_t a3, uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
        "{%8, %9}, {%10, %11, %12, %13};"
        : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(z[0]), "f"(z[1]), "f"(z[2]), "f"(z[3]));
  }
};

// Staged vectors take the codes themselves as fp16 subnormals: a nibble in bits
// 0-3 is code 2^-24, in bits 4-7 code 2^-20 (the vector's columns 1 3 5 7 are
// divided by 16 for that).  No subtraction: the group's sum of the vector, times
// 8, comes off the fp32 result.  One shift and four ands for eight weights,
// against three, four and four for the exact bf16 operands: with one token the
// products of the first expert matrices took 197 instructions a stage that way.
MOE_DEV void codes_fp16(uint32_t w, uint32_t* a) {
  const uint32_t u = w >> 8;
  a[0] = w & 0x000F000Fu;
  a[1] = w & 0x00F000F0u;
  a[2] = u & 0x000F000Fu;
  a[3] = u & 0x00F000F0u;
}

// ------------------------------------------------------------------ weight stream
// A warp works on tiles of 16 weight rows.  A stage is 128 columns of a tile (1
// KB of codes and the scales); the lanes copy it in 16-byte pieces with cp.async
// into the warp's own ring, kRing - 1 stages ahead, past L1.  Only the warp
// itself waits for its ring, so no barrier of the block lies in the loop, and
// five stages a warp stay in flight without registers.
constexpr int kRing = 6;
constexpr int kStageBytes = 1024 + 128;   // codes, scales (16 rows x 8 bytes)
constexpr int kRingBytes = kRing * kStageBytes;
constexpr int kRingsBytes = kW4Warps * kRingBytes;
constexpr int kSmemMost = 227 * 1024;

MOE_DEV void cp_async16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
template <int N> MOE_DEV void cp_async_small(uint32_t dst, const void* src, int bytes) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(dst), "l"(src), "n"(N), "r"(bytes) : "memory");
}
MOE_DEV void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N> MOE_DEV void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// 16-byte pieces of a row's 64 bytes are permuted by the row, so that lanes
// reading one, two or four words of eight rows touch every bank once.
MOE_DEV int piece_swizzle(int g) { return ((g >> 1) & 1) << 1 | ((g >> 2) & 1); }

// Where a lane finds its vectors.
//   kStaged   in shared memory, as fp16 with a power of two per 128 columns
//             (below); the products run in fp16 whatever the vectors' type
//   kOrdered  in global memory, in fragment order (bf16, a high and a low part)
//   kNatural  in global memory, column by column
// Fragment order of a stage's 128 values: sixteen pieces of eight; the piece of
// columns [8 c, 8 c + 8) holds them as 0 4 1 5 2 6 3 7, which is how the codes of
// a word come apart, and lies at piece_place(c), where the four lanes of a
// fragment row read neighbouring pieces.
enum XSource { kStaged, kOrdered, kNatural };
template <int W> MOE_DEV int piece_place(int c) {
  const int j = c / (4 * W), t = c / W % 4, i = c % W;
  return (j * W + i) * 4 + t;
}
MOE_DEV int in_piece(int r) { return (r & 3) * 2 + (r >> 2); }
MOE_DEV uint4 order_piece(const uint4& x) {
  return make_uint4(__byte_perm(x.x, x.z, 0x5410), __byte_perm(x.x, x.z, 0x7632),
                    __byte_perm(x.y, x.w, 0x5410), __byte_perm(x.y, x.w, 0x7632));
}

// This lane's vector of each tile of eight vectors, at stage 0.
template <typename T, int NT> struct Vectors {
  const T* x[NT];        // kOrdered, kNatural
  int64_t low;           // kOrdered: distance of the low parts
  uint32_t s, s_low;     // kStaged: the vector and its low parts
  uint32_t table;        // kStaged: (factor, 8 sum) of this lane's two columns
};

template <int W> struct Words { uint32_t w[W]; };
template <int W> MOE_DEV Words<W> load_words(uint32_t at) {
  Words<W> r;
  if constexpr (W == 4)
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(r.w[0]), "=r"(r.w[1]), "=r"(r.w[2]), "=r"(r.w[3]) : "r"(at));
  else if constexpr (W == 2)
    asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(r.w[0]), "=r"(r.w[1]) : "r"(at));
  else
    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(r.w[0]) : "r"(at));
  return r;
}

// What a tile's rows are, for this lane: codes of rows g and g + 8 (its piece t
// of a stage) and scales of row lane % 16, at some stage.
struct RowPtr {
  const uint8_t* a;
  const uint8_t* b;
  const uint8_t* s;
};

// One warp's share of a segment: `tiles` tiles of `stages` stages each.  The
// rows of a tile are contiguous for `run` stages (RUNS: run < stages, each run of
// the same K); rows(tile, stage) gives the pointers where a run starts or the
// share does.  Parts of tiles go to parts[tile + warp] (NT x 16 rows x 8 vectors
// each): the slot is the warp's own, since a warp starts no earlier than in the
// tile where the one before it ends.
//   FULL   K is a multiple of 128, scales come through the ring; otherwise (K
//          32 or 64 more than that) the last stage is cut and the scales are
//          read directly
//   T      type of the vectors, S of the scales;  LOW: a vector has two parts
//   VC     vectors that the table of kStaged is for: 8, or 1 (all columns the same)
template <typename T, typename S, int W, int NT, bool LOW, XSource XS, bool FULL, bool RUNS, int VC, typename Rows>
struct Segment {
  static constexpr int kScales = 4 / W;   // of a row in a stage
  using Mma = MmaT<T>;
  const Rows& rows;
  uint32_t put, get, swz, scl, ring;
  int stages, run, groups, v0, n;
  int copy_tile, copy_stage, copy_left, copy_run;   // next stage to copy
  int row_bytes;
  RowPtr r;
  const uint8_t* scales_end;

  MOE_DEV Segment(uint32_t rings, const Rows& rows_, int tiles, int stages_, int run_, int K,
                  const void* scales_end_)
      : rows(rows_), stages(stages_), run(run_), groups(K / (32 * W)), row_bytes(K / 2),
        scales_end(static_cast<const uint8_t*>(scales_end_)) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
    ring = rings + warp * kRingBytes;
    swz = piece_swizzle(g) << 4;
    put = ring + g * 64 + ((t << 4) ^ swz);
    get = ring + g * 64;
    scl = ring + 1024 + (lane & 15) * 8;
    const int V = tiles * stages;
    v0 = warp * V / kW4Warps;
    n = (warp + 1) * V / kW4Warps - v0;
    copy_tile = v0 / stages;
    copy_stage = v0 - copy_tile * stages;
    copy_run = RUNS ? run - copy_stage % run : 0;
    copy_left = n;
    if (n > 0) r = rows(copy_tile, copy_stage);
  }

  MOE_DEV void copy(int slot) {
    const int lane = threadIdx.x & 31;
    if (copy_left > 0) {
      const bool there = FULL || (copy_stage * 64 + (lane & 3) * 16) < row_bytes;
      if (there) {
        cp_async16(put + slot * kStageBytes, r.a);
        cp_async16(put + slot * kStageBytes + 512, r.b);
      }
      if (FULL && lane < 16) {
        if constexpr (W == 4) {   // one scale: the aligned word that holds it
          const uint8_t* w = reinterpret_cast<const uint8_t*>(reinterpret_cast<uintptr_t>(r.s) & ~uintptr_t(3));
          cp_async_small<4>(scl + slot * kStageBytes, w, w + 4 > scales_end ? 2 : 4);
        } else {
          cp_async_small<2 * kScales>(scl + slot * kStageBytes, r.s, 2 * kScales);
        }
      }
      r.a += 64;
      r.b += 64;
      r.s += 2 * kScales;
      ++copy_stage;
      --copy_left;
      bool turn = copy_stage == stages;
      if (turn) {
        copy_stage = 0;
        ++copy_tile;
      }
      if (RUNS && --copy_run == 0) {
        turn = true;
        copy_run = run;
      }
      if (turn && copy_left > 0) r = rows(copy_tile, copy_stage);
    }
    cp_async_commit();
  }

  MOE_DEV void start() {
#pragma unroll
    for (int i = 0; i < kRing - 1; ++i) copy(i);
  }

  // The scales of a stage's groups for this lane's rows g and g + 8; `q` is the
  // stage within its run.
  MOE_DEV void load_scales(int slot, int tile, int stage, int q, float* fa, float* fb) const {
    const int lane = threadIdx.x & 31, g = lane >> 2;
    if constexpr (FULL) {
      const uint32_t at = ring + slot * kStageBytes + 1024 + g * 8;
      if constexpr (W == 4) {
        // rows are numbered from an even one: the half-word is known from g
        const uint32_t half = at + (((g * groups + q) & 1) << 1);
        uint16_t a, b;
        asm volatile("ld.shared.u16 %0, [%1];" : "=h"(a) : "r"(half));
        asm volatile("ld.shared.u16 %0, [%1];" : "=h"(b) : "r"(half + 64));
        fa[0] = Elem<S>::to_f(*reinterpret_cast<S*>(&a));
        fb[0] = Elem<S>::to_f(*reinterpret_cast<S*>(&b));
      } else {
        const Words<kScales / 2> a = load_words<kScales / 2>(at), b = load_words<kScales / 2>(at + 64);
        const S* pa = reinterpret_cast<const S*>(&a);
        const S* pb = reinterpret_cast<const S*>(&b);
#pragma unroll
        for (int j = 0; j < kScales; ++j) { fa[j] = Elem<S>::to_f(pa[j]); fb[j] = Elem<S>::to_f(pb[j]); }
      }
    } else {
      const S *pa, *pb;
      rows.scales(tile, &pa, &pb);
#pragma unroll
      for (int j = 0; j < kScales; ++j) {
        const int i = stage * kScales + j;
        fa[j] = i < groups ? Elem<S>::to_f(pa[i]) : 0.0f;
        fb[j] = i < groups ? Elem<S>::to_f(pb[i]) : 0.0f;
      }
    }
  }

  MOE_DEV void product(int slot, int tile, int stage, int q, const Vectors<T, NT>& v, int nt,
                       float (*acc)[4]) const {
    const int t = threadIdx.x & 3;
    float fa[kScales], fb[kScales];
    load_scales(slot, tile, stage, q, fa, fb);
    const float zero[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int j = 0; j < kScales; ++j) {
      if (!FULL && stage * kScales + j >= groups) break;
      const int at = (j * 4 * W + t * W) * 4;   // byte of the row's 64
      const uint32_t p = get + ((at & 48) ^ swz) + (at & 15) + slot * kStageBytes;
      const Words<W> wa = load_words<W>(p), wb = load_words<W>(p + 512);
      if constexpr (XS == kStaged) {
        float c[4], cl[4];
#pragma unroll
        for (int i = 0; i < W; ++i) {
          uint32_t a[4], b[4];
          codes_fp16(wa.w[i], a);
          codes_fp16(wb.w[i], b);
          const uint32_t to = stage * 256 + t * 16 + (j * W + i) * 64;
          const Words<4> x = load_words<4>(v.s + to);
          MmaT<__half>::mma(c, i == 0 ? zero : c, a[0], b[0], a[1], b[1], x.w[0], x.w[1]);
          MmaT<__half>::mma(c, c, a[2], b[2], a[3], b[3], x.w[2], x.w[3]);
          if constexpr (LOW) {
            const Words<4> y = load_words<4>(v.s_low + to);
            MmaT<__half>::mma(cl, i == 0 ? zero : cl, a[0], b[0], a[1], b[1], y.w[0], y.w[1]);
            MmaT<__half>::mma(cl, cl, a[2], b[2], a[3], b[3], y.w[2], y.w[3]);
          }
        }
        float f0, s0, f1, s1;   // factor and 8 times the group's sum, of two columns
        const uint32_t entry = v.table + (stage * kScales + j) * (VC * 8);
        if constexpr (VC == 8) {
          asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(f0), "=f"(s0), "=f"(f1), "=f"(s1) : "r"(entry));
        } else {
          asm volatile("ld.shared.v2.f32 {%0, %1}, [%2];" : "=f"(f0), "=f"(s0) : "r"(entry));
          f1 = f0;
          s1 = s0;
        }
        if constexpr (LOW) {
#pragma unroll
          for (int i = 0; i < 4; ++i) c[i] += cl[i];
        }
        acc[0][0] = fmaf(fa[j], fmaf(c[0], f0, -s0), acc[0][0]);
        acc[0][1] = fmaf(fa[j], fmaf(c[1], f1, -s1), acc[0][1]);
        acc[0][2] = fmaf(fb[j], fmaf(c[2], f0, -s0), acc[0][2]);
        acc[0][3] = fmaf(fb[j], fmaf(c[3], f1, -s1), acc[0][3]);
      } else {
        float c[NT][4];
#pragma unroll
        for (int i = 0; i < W; ++i) {
          uint32_t a[4], b[4];
          Mma::widen(wa.w[i], a);
          Mma::widen(wb.w[i], b);
#pragma unroll
          for (int m = 0; m < NT; ++m) {
            if (m < nt) {
#pragma unroll
              for (int part = 0; part < (LOW ? 2 : 1); ++part) {
                uint4 x;
                if constexpr (XS == kOrdered)
                  x = *reinterpret_cast<const uint4*>(v.x[m] + part * v.low + stage * 128 + ((j * W + i) * 4 + t) * 8);
                else
                  x = order_piece(*reinterpret_cast<const uint4*>(v.x[m] + stage * 128 + j * 32 * W + t * 8 * W + i * 8));
                Mma::mma(c[m], i == 0 && part == 0 ? zero : c[m], a[0], b[0], a[1], b[1], x.x, x.y);
                Mma::mma(c[m], c[m], a[2], b[2], a[3], b[3], x.z, x.w);
              }
            }
          }
        }
#pragma unroll
        for (int m = 0; m < NT; ++m) {
          if (m < nt) {
            acc[m][0] = fmaf(fa[j], c[m][0], acc[m][0]);
            acc[m][1] = fmaf(fa[j], c[m][1], acc[m][1]);
            acc[m][2] = fmaf(fb[j], c[m][2], acc[m][2]);
            acc[m][3] = fmaf(fb[j], c[m][3], acc[m][3]);
          }
        }
      }
    }
  }

  MOE_DEV void store_part(float* parts, int tile, float (*acc)[4]) const {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
    float* at = parts + (tile + warp) * (NT * 128) + g * 8 + 2 * t;
#pragma unroll
    for (int m = 0; m < NT; ++m) {
      *reinterpret_cast<float2*>(at + m * 128) = make_float2(acc[m][0], acc[m][1]);
      *reinterpret_cast<float2*>(at + m * 128 + 64) = make_float2(acc[m][2], acc[m][3]);
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[m][i] = 0.0f;
    }
  }

  MOE_DEV void finish(const Vectors<T, NT>& v, int nt, float* parts) {
    float acc[NT][4];
#pragma unroll
    for (int m = 0; m < NT; ++m)
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[m][i] = 0.0f;
    int tile = v0 / stages, stage = v0 - tile * stages;
    int q = RUNS ? stage % run : stage;
    for (int i0 = 0; i0 < n; i0 += kRing) {
#pragma unroll
      for (int u = 0; u < kRing; ++u) {
        if (i0 + u >= n) break;
        copy((u + kRing - 1) % kRing);
        cp_async_wait<kRing - 1>();
        __syncwarp();
        product(u, tile, stage, RUNS ? q : stage, v, nt, acc);
        __syncwarp();   // the slot is free for every lane's next copy
        if (RUNS && ++q == run) q = 0;
        if (++stage == stages) {
          store_part(parts, tile, acc);
          stage = 0;
          ++tile;
        }
      }
    }
    // a warp without stages leaves zeros: its slot lies among its tile's parts
    if (n == 0 || stage != 0) store_part(parts, tile, acc);
    cp_async_wait<0>();
  }
};

// Sum of a tile's parts at `at` (vector tile * 128 + row * 8 + vector), warp by
// warp: warp_of(v) is the warp whose share has stage v of V.
MOE_DEV int warp_of(int v, int V) { return (int)((uint32_t)(kW4Warps * (v + 1) - 1) / (uint32_t)V); }
struct PartRange {
  int first, last;
  MOE_DEV PartRange(int tile, int tiles, int stages)
      : first(warp_of(tile * stages, tiles * stages)), last(warp_of(tile * stages + stages - 1, tiles * stages)) {}
};
MOE_DEV float sum_parts(const float* parts, int slot_floats, int tile, const PartRange& w, int at) {
  float s = 0.0f;
  for (int i = w.first; i <= w.last; ++i) s += parts[(tile + i) * slot_floats + at];
  return s;
}

// ------------------------------------------------------------------ staged vectors
// Each 128 columns (a stage) of a vector become fp16 after a power of two that
// puts their largest value into [2^13, 2^14): 8 or 11 significant bits stay 31
// binary orders below the largest value, and what is lost further down (2^-35 of
// it) is below the rounding of the fp32 sums.  LOW keeps a second fp16 part, 22
// bits together.  A vector with an infinity or NaN gives results that are not
// finite.  The table has, for each group, the factor back to the vector's units
// (2^24 of the codes included) and 8 times the sum of its values.

// Bytes between staged vectors: 64 more than a multiple of 128, so that two
// rows do not share banks.
__host__ __device__ inline int staged_stride(int K) { return K * 2 + 64; }

struct StagedAt {
  uint32_t x, low;        // vector 0 and its low parts
  int stride;             // bytes between vectors
  uint32_t table;         // entries [group][vectors of the table]
};

MOE_DEV void load_f8(const __nv_bfloat16* p, float* f) { widen8(load8<__nv_bfloat16, true>(p, 0, 8), f); }
MOE_DEV void load_f8(const __half* p, float* f) { widen8(load8<__half, true>(p, 0, 8), f); }
MOE_DEV void load_f8(const float* p, float* f) { widen8(load8<float, true>(p, 0, 8), f); }

// Stage `count` vectors of K values (K a multiple of 128); row(m) is vector m.
// Every thread of the block calls; no barrier.
template <typename T, int W, bool LOW, int VC, typename Row>
MOE_DEV void stage_vectors(const StagedAt& at, int count, int K, Row row) {
  constexpr int U = 4;   // pieces a thread has in flight
  const int pieces = K / 8, all = count * pieces;
  for (int base = 0; base < all; base += U * kW4Threads) {
    float f[U][8];
    int m[U], c[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int i = base + u * kW4Threads + threadIdx.x;
      m[u] = i / pieces;
      c[u] = i - m[u] * pieces;
      if (i < all) {
        load_f8(row(m[u]) + c[u] * 8, f[u]);
      } else {
        m[u] = -1;
#pragma unroll
        for (int j = 0; j < 8; ++j) f[u][j] = 0.0f;
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      float top = 0.0f, sum = 0.0f;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        top = fmaxf(top, fabsf(f[u][j]));
        sum += f[u][j];
      }
#pragma unroll
      for (int off = 1; off < 16; off <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
#pragma unroll
      for (int off = 1; off < 4 * W; off <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
      const int k = top > 0.0f ? max(min(140 - (int)(__float_as_uint(top) >> 23), 126), -103) : 0;
      const float scale = exp2i(k);
      uint32_t hi[4], lo[4];
#pragma unroll
      for (int q = 0; q < 4; ++q) {   // columns q and q + 4
        const float sc = q & 1 ? scale * 0.0625f : scale;
        const float a = f[u][q] * sc, b = f[u][q + 4] * sc;
        const __half2 h = __floats2half2_rn(a, b);
        hi[q] = *reinterpret_cast<const uint32_t*>(&h);
        if (LOW) {
          const __half2 l = __floats2half2_rn(a - __low2float(h), b - __high2float(h));
          lo[q] = *reinterpret_cast<const uint32_t*>(&l);
        }
      }
      if (m[u] < 0) continue;
      const uint32_t to = m[u] * at.stride + (c[u] >> 4) * 256 + piece_place<W>(c[u] & 15) * 16;
      asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(at.x + to), "r"(hi[0]), "r"(hi[1]), "r"(hi[2]), "r"(hi[3]) : "memory");
      if (LOW)
        asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(at.low + to), "r"(lo[0]), "r"(lo[1]), "r"(lo[2]), "r"(lo[3]) : "memory");
      if (c[u] % (4 * W) == 0) {
        const int group = c[u] / (4 * W);
        const uint32_t entry = at.table + (VC == 8 ? (group * 8 + m[u]) * 8 : (m[u] * (K / (32 * W)) + group) * 8);
        asm volatile("st.shared.v2.f32 [%0], {%1, %2};" ::"r"(entry), "f"(exp2i(24 - k)), "f"(8.0f * sum) : "memory");
      }
    }
  }
}

// Raise a kernel's dynamic shared memory limit (once, from moe_init).
template <typename F> cudaError_t allow_smem(F* kernel, int static_bytes = 0) {
  return cudaFuncSetAttribute(reinterpret_cast<const void*>(kernel),
                              cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemMost - static_bytes);
}

}  // namespace moe
