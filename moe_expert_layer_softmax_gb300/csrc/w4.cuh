// 4-bit weights with group scales (sm_103a): the stream of weights that the
// products with a few vectors are made of.
//
//   W[n, k] = (code[n, k] - 8) * scale[n, k / G],   G = 32, 64 or 128
// Two codes a byte, the even column in the low nibble; row-major, so one row of
// K columns is K/2 contiguous bytes.
//
// The least a call costs is the weights' bytes: every weight is read once and
// used for a handful of vectors.  The products run on mma.sync m16n8k16 with 16
// weight rows as A and eight vectors as B: each lane turns its own 4-bit words
// into operands, and eight vectors do not fill a larger matrix instruction.
// What bounds it in fact is issue: about 185 instructions for each 128 columns of
// 16 rows (220 with two-part vectors), 72 of them the conversion of the codes, at
// 47-65% of the issue slots; the rest waits on instructions before it (fixed
// latencies first, then the 16-bit arithmetic of the conversion, then shared memory,
// whose path is at 38-48%).  Weights that already lie in L2 take the same time.  64
// experts (2048 x 1408, 64 tokens) stream 3.3 TB/s, eight tokens on experts of 4096 x
// 2048 4.4 TB/s.  Tried without gain, with a shorter conversion (stage_vectors):
// weights fetched by TMA tiles (one lane, 128-byte boxes: 88.8 against 87.8 us) or
// by one bulk copy a row (104 us), and two chains of matrix instructions for one
// (87.2 against 85.2 us).
// The sum over k may visit columns in any order as long as A and B agree, so a
// lane's fragment columns are simply those of the words it holds.  Products of
// a group are exact integers times activations, summed in fp32; the group's
// scale multiplies the fp32 sum.
//
// One block of 16 warps runs on each SM and takes an equal share of the tiles;
// its warps split the share's (tile, step) pairs evenly, whatever the number
// of tiles, and add up a tile's parts in shared memory in a fixed order.  (64
// experts as above, 64 tokens, and one token on eight of 4096 x 2048, with the
// shorter conversion: 16 warps with rings of three steps 87.8 and 32.9 us, 12 with
// three 90.6 and 32.4, 12 with four 88.0 and 31.9, 24 and more spill.)
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
  // (Y. J. Kim, R. Henry, R. Fahim, H. H. Awadalla, "Who Says Elephants Can't Run:
  // Bringing Large Scale MoE Models into Cloud Scale Production", SustaiNLP 2022.)
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

// The warp's number, known to be the same in all its lanes: what follows from it
// (shares, counters, slots) then stays in uniform registers.
MOE_DEV int warp_id() { return __shfl_sync(0xffffffffu, (int)(threadIdx.x >> 5), 0); }

// ------------------------------------------------------------------ weight stream
// A warp works on tiles of 16 weight rows.  A stage is 128 columns of a tile (1
// KB of codes and the scales), a step two stages; the lanes copy a step in
// 16-byte pieces with cp.async into the warp's own ring, kRing - 1 steps ahead,
// past L1.  Only the warp itself waits for its ring, so no barrier of the block
// lies in the loop, and four stages a warp stay in flight without registers.  The
// two stages of a step are independent chains of matrix instructions.
constexpr int kRing = 3;
constexpr int kStepBytes = 2048 + 256;   // 16 rows of 128 bytes of codes, 16 of 16 bytes for scales
constexpr int kRingBytes = kRing * kStepBytes;
constexpr int kRingsBytes = kW4Warps * kRingBytes;
constexpr int kSmemMost = 227 * 1024;

template <int N> MOE_DEV void cp_async_small(uint32_t dst, const void* src, int bytes) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(dst), "l"(src), "n"(N), "r"(bytes) : "memory");
}

// The eight 16-byte pieces of a row's 128 bytes are permuted by the row, so that
// lanes reading one, two or four words of eight rows touch every bank once.
MOE_DEV int piece_swizzle(int g) { return (g & 1) << 2 | ((g >> 1) & 1) << 1 | ((g >> 2) & 1); }

// Where a lane finds its vectors.
//   kStaged   in shared memory, as fp16 with a power of two per 128 columns
//             (below); the products take fp16 whatever the vectors' type
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
  uint32_t s, s_low;     // kStaged: the first tile's vector and its low parts
  uint32_t to[NT];       // kStaged: bytes from it to each tile's
  uint32_t table;        // kStaged: the factors of this lane's two columns
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

// A tile's rows as this lane copies them, from some stage on: its piece (lane %
// 8) of rows lane / 8 + 0, 4, 8 and 12, and the scales of row lane % 16.
struct RowPtr {
  const uint8_t* row[4];
  const uint8_t* s;
};

// One warp's share of a segment: `tiles` tiles of `runs` runs of `run` stages
// each; a run's rows are contiguous (RUNS: more than one run a tile).  The share
// is counted in steps; a run's last step is half a step where `run` is odd.
// rows(tile, r, stage) gives the pointers to a stage of run r.  Parts of tiles go
// to parts[tile + warp] (NT x 16 rows x 8 vectors each): the slot is the warp's
// own, since a warp starts no earlier than in the tile where the one before it
// ends.
//   FULL   K is a multiple of 128, scales come through the ring; otherwise (K
//          32 or 64 more than that) the last stage is cut and the scales are
//          read directly
//   T      type of the vectors, S of the scales;  LOW: a vector has two parts
//   VC     vectors that the table of kStaged is for: 8 NT, or 1 (the same in all columns)
template <typename T, typename S, int W, int NT, bool LOW, XSource XS, bool FULL, bool RUNS, int VC, typename Rows>
struct Segment {
  static constexpr int kScales = 4 / W;   // of a row in a stage
  using Mma = MmaT<T>;
  Rows rows;
  uint32_t put, put4, get, swz, scl, sget;
  int run, runs, steps, groups, n;   // steps of a run, of the share
  int tile0, run0, step0;            // where the share begins: tile, run, step of the run
  int copy_tile, copy_run, copy_step;   // the next step to copy
  RowPtr r;                          // of the next step to copy
  uint32_t copy_slot;                // bytes
  int copy_left;                     // steps to copy
  const uint8_t* scales_end;

  MOE_DEV Segment(uint32_t rings, const Rows& rows_, int tiles, int runs_, int run_, int K,
                  const void* scales_end_)
      : rows(rows_), run(run_), runs(RUNS ? runs_ : 1), steps((run_ + 1) / 2), groups(K / (32 * W)),
        scales_end(static_cast<const uint8_t*>(scales_end_)) {
    const int lane = threadIdx.x & 31, g = lane >> 2;
    const uint32_t ring = rings + warp_id() * kRingBytes;
    swz = piece_swizzle(g) << 4;
    get = ring + g * 128;
    // rows lane / 8 and 4 more have swizzles that differ in the lowest bit alone
    put = ring + (lane >> 3) * 128 + (((lane & 7) ^ piece_swizzle(lane >> 3)) << 4);
    put4 = ring + ((lane >> 3) + 4) * 128 + (((lane & 7) ^ piece_swizzle((lane >> 3) + 4)) << 4);
    scl = ring + 2048 + (lane & 15) * 16;
    sget = ring + 2048 + g * 16;
    reset(tiles);
  }

  // A segment of as many tiles of the same kind (rows may have changed).
  MOE_DEV void reset(int tiles) {
    const int warp = warp_id();
    tiles = __shfl_sync(0xffffffffu, tiles, 0);
    const int per = steps * runs, V = tiles * per, v0 = warp * V / kW4Warps;
    n = (warp + 1) * V / kW4Warps - v0;
    tile0 = v0 / per;
    const int in = v0 - tile0 * per;
    run0 = RUNS ? in / steps : 0;
    step0 = in - run0 * steps;
    copy_tile = tile0;
    copy_run = run0;
    copy_step = step0;
    copy_left = n;
    if (n > 0) r = rows(copy_tile, copy_run, copy_step * 2);
  }

  MOE_DEV static uint32_t next_slot(uint32_t slot) {
    return slot == (kRing - 1) * kStepBytes ? 0 : slot + kStepBytes;
  }

  MOE_DEV void copy() {
    if (copy_left > 0) {
      const int lane = threadIdx.x & 31;
      // the second half of a run's last step may lie past its end
      const bool two = copy_step * 2 + 1 < run;
      if (FULL ? (lane & 4) == 0 || two : copy_step * 128 + (lane & 7) * 16 < groups * (16 * W)) {
        cp_async16(put + copy_slot, r.row[0]);
        cp_async16(put4 + copy_slot, r.row[1]);
        cp_async16(put + copy_slot + 1024, r.row[2]);
        cp_async16(put4 + copy_slot + 1024, r.row[3]);
      }
      if (FULL && lane < 16) {
        const uint32_t to = scl + copy_slot;
        if constexpr (W == 4) {   // two scales: the aligned words that hold them
          const uint8_t* p = reinterpret_cast<const uint8_t*>(reinterpret_cast<uintptr_t>(r.s) & ~uintptr_t(3));
          cp_async_small<4>(to, p, p + 4 > scales_end ? 2 : 4);
          if (groups & 1) {   // every other row starts in the middle of a word
            const int there = two ? (p + 8 > scales_end ? (p + 4 >= scales_end ? 0 : 2) : 4) : 0;
            cp_async_small<4>(to + 4, there ? p + 4 : p, there);
          }
        } else {
          cp_async_small<2 * kScales>(to, r.s, 2 * kScales);
          if (two) cp_async_small<2 * kScales>(to + 2 * kScales, r.s + 2 * kScales, 2 * kScales);
        }
      }
      copy_slot = next_slot(copy_slot);
      --copy_left;
      if (++copy_step == steps) {
        if (copy_left > 0) {
          copy_step = 0;
          if (!RUNS || ++copy_run == runs) {
            copy_run = 0;
            ++copy_tile;
          }
          r = rows(copy_tile, copy_run, 0);
        }
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) r.row[i] += 128;
        r.s += 4 * kScales;
      }
    }
    cp_async_commit();
  }

  // Fill the ring (empty before).
  MOE_DEV void start() {
    copy_slot = 0;
#pragma unroll 1
    for (int i = 0; i < kRing - 1; ++i) copy();
  }

  // Where the consumer stands.
  struct At {
    int tile, stage;        // stage: within its run
    uint32_t slot;
    uint32_t half;          // W = 4: byte of a step's first scale in its word
    uint32_t x, low, table;
  };

  // The scales of a stage's groups for this lane's rows g and g + 8.
  MOE_DEV void load_scales(int h, const At& at, float* fa, float* fb) const {
    if constexpr (FULL) {
      const uint32_t from = sget + at.slot + h * (2 * kScales);
      if constexpr (W == 4) {
        uint16_t a, b;
        asm volatile("ld.shared.u16 %0, [%1];" : "=h"(a) : "r"(from + at.half));
        asm volatile("ld.shared.u16 %0, [%1];" : "=h"(b) : "r"(from + at.half + 128));
        fa[0] = Elem<S>::to_f(*reinterpret_cast<S*>(&a));
        fb[0] = Elem<S>::to_f(*reinterpret_cast<S*>(&b));
      } else {
        const Words<kScales / 2> a = load_words<kScales / 2>(from), b = load_words<kScales / 2>(from + 128);
        const S* pa = reinterpret_cast<const S*>(&a);
        const S* pb = reinterpret_cast<const S*>(&b);
#pragma unroll
        for (int j = 0; j < kScales; ++j) { fa[j] = Elem<S>::to_f(pa[j]); fb[j] = Elem<S>::to_f(pb[j]); }
      }
    } else {
      const S *pa, *pb;
      rows.scales(at.tile, &pa, &pb);
#pragma unroll
      for (int j = 0; j < kScales; ++j) {
        const int i = (at.stage + h) * kScales + j;
        fa[j] = i < groups ? Elem<S>::to_f(pa[i]) : 0.0f;
        fb[j] = i < groups ? Elem<S>::to_f(pb[i]) : 0.0f;
      }
    }
  }

  // Stage h of the present step, for M tiles of vectors.
  template <int M> MOE_DEV void product(int h, const At& at, const Vectors<T, NT>& v, float (*acc)[4]) const {
    const int t = threadIdx.x & 3;
    float fa[kScales], fb[kScales];
    load_scales(h, at, fa, fb);
    const float zero[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    float sum[M][4];   // kStaged: of the stage, in the units of its vectors
#pragma unroll
    for (int j = 0; j < kScales; ++j) {
      if (!FULL && (at.stage + h) * kScales + j >= groups) break;
      const int byte = h * 64 + (j * 4 * W + t * W) * 4;   // of the row's 128
      const uint32_t p = get + ((byte & 112) ^ swz) + (byte & 15) + at.slot;
      const Words<W> wa = load_words<W>(p), wb = load_words<W>(p + 1024);
      if constexpr (XS == kStaged) {
        // low parts of a single tile sum on their own: two chains of products.
        // Not where a round may serve more than one tile: a vector's sum must not
        // depend on the round that it falls into (M is the round's).
        constexpr bool own = LOW && NT == 1;
        float c[M][4], cl[4];
#pragma unroll
        for (int i = 0; i < W; ++i) {
          uint32_t a[4], b[4];
          MmaT<__half>::widen(wa.w[i], a);
          MmaT<__half>::widen(wb.w[i], b);
          const int to = h * 256 + (j * W + i) * 64;
#pragma unroll
          for (int m = 0; m < M; ++m) {
            const Words<4> x = load_words<4>(at.x + (m ? v.to[m] : 0) + to);
            MmaT<__half>::mma(c[m], i == 0 ? zero : c[m], a[0], b[0], a[1], b[1], x.w[0], x.w[1]);
            MmaT<__half>::mma(c[m], c[m], a[2], b[2], a[3], b[3], x.w[2], x.w[3]);
            if constexpr (LOW) {
              const Words<4> y = load_words<4>(at.low + (m ? v.to[m] : 0) + to);
              float* l = own ? cl : c[m];
              MmaT<__half>::mma(l, own && i == 0 ? zero : l, a[0], b[0], a[1], b[1], y.w[0], y.w[1]);
              MmaT<__half>::mma(l, l, a[2], b[2], a[3], b[3], y.w[2], y.w[3]);
            }
          }
        }
        if constexpr (own) {
#pragma unroll
          for (int i = 0; i < 4; ++i) c[0][i] += cl[i];
        }
#pragma unroll
        for (int m = 0; m < M; ++m) {
          sum[m][0] = j ? fmaf(fa[j], c[m][0], sum[m][0]) : fa[j] * c[m][0];
          sum[m][1] = j ? fmaf(fa[j], c[m][1], sum[m][1]) : fa[j] * c[m][1];
          sum[m][2] = j ? fmaf(fb[j], c[m][2], sum[m][2]) : fb[j] * c[m][2];
          sum[m][3] = j ? fmaf(fb[j], c[m][3], sum[m][3]) : fb[j] * c[m][3];
        }
      } else {
        float c[M][4];
#pragma unroll
        for (int i = 0; i < W; ++i) {
          uint32_t a[4], b[4];
          Mma::widen(wa.w[i], a);
          Mma::widen(wb.w[i], b);
#pragma unroll
          for (int m = 0; m < M; ++m) {
#pragma unroll
            for (int part = 0; part < (LOW ? 2 : 1); ++part) {
              uint4 x;
              if constexpr (XS == kOrdered)
                x = *reinterpret_cast<const uint4*>(v.x[m] + part * v.low + (at.stage + h) * 128 + ((j * W + i) * 4 + t) * 8);
              else
                x = order_piece(*reinterpret_cast<const uint4*>(v.x[m] + (at.stage + h) * 128 + j * 32 * W + t * 8 * W + i * 8));
              Mma::mma(c[m], i == 0 && part == 0 ? zero : c[m], a[0], b[0], a[1], b[1], x.x, x.y);
              Mma::mma(c[m], c[m], a[2], b[2], a[3], b[3], x.z, x.w);
            }
          }
        }
#pragma unroll
        for (int m = 0; m < M; ++m) {
          acc[m][0] = fmaf(fa[j], c[m][0], acc[m][0]);
          acc[m][1] = fmaf(fa[j], c[m][1], acc[m][1]);
          acc[m][2] = fmaf(fb[j], c[m][2], acc[m][2]);
          acc[m][3] = fmaf(fb[j], c[m][3], acc[m][3]);
        }
      }
    }
    if constexpr (XS == kStaged) {
#pragma unroll
      for (int m = 0; m < M; ++m) {
        float f0, f1;   // factors of two columns
        const uint32_t entry = at.table + h * (VC * 4) + m * 32;
        if constexpr (VC > 1) {
          asm volatile("ld.shared.v2.f32 {%0, %1}, [%2];" : "=f"(f0), "=f"(f1) : "r"(entry));
        } else {
          asm volatile("ld.shared.f32 %0, [%1];" : "=f"(f0) : "r"(entry));
          f1 = f0;
        }
        acc[m][0] = fmaf(sum[m][0], f0, acc[m][0]);
        acc[m][1] = fmaf(sum[m][1], f1, acc[m][1]);
        acc[m][2] = fmaf(sum[m][2], f0, acc[m][2]);
        acc[m][3] = fmaf(sum[m][3], f1, acc[m][3]);
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

  // The share's products with `nt` tiles of vectors.
  MOE_DEV void finish(const Vectors<T, NT>& v, int nt, float* parts) {
    if (NT == 1 || nt == 1)
      run_share<1>(v, parts);
    else if (NT == 2 || nt == 2)
      run_share<NT == 1 ? 1 : 2>(v, parts);
    else
      run_share<NT>(v, parts);
  }
  template <int M> MOE_DEV void run_share(const Vectors<T, NT>& v, float* parts) {
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    float acc[NT][4];
#pragma unroll
    for (int m = 0; m < NT; ++m)
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[m][i] = 0.0f;
    At at;
    // rows are numbered from an even one: a scale's half-word is known from g
    // (a step starts at an even stage)
    at.half = W == 4 ? (uint32_t)((g * groups) & 1) << 1 : 0;
    at.tile = tile0;
    at.stage = step0 * 2;
    int in_run = run0, turn = steps - step0, left = n;
    at.slot = 0;
    auto enter = [&](int step) {   // at a step of run in_run
      const int stage = (RUNS ? in_run * run : 0) + step * 2;
      at.x = v.s + t * 16 + stage * 256;
      at.low = v.s_low + t * 16 + stage * 256;
      at.table = v.table + stage * VC * 4;
    };
    enter(step0);
#pragma unroll 1
    for (; left > 0; --left) {
      copy();   // into the slot of the step before
      cp_async_wait<kRing - 1>();
      __syncwarp();
      if (at.stage + 1 < run) {
        product<M>(0, at, v, acc);
        product<M>(1, at, v, acc);
      } else {
        product<M>(0, at, v, acc);
      }
      __syncwarp();   // the slot is free for every lane's next copy
      at.slot = next_slot(at.slot);
      at.stage += 2;
      at.x += 512;
      at.low += 512;
      at.table += 2 * VC * 4;
      if (--turn == 0) {
        turn = steps;
        at.stage = 0;
        if (!RUNS || ++in_run == runs) {
          in_run = 0;
          store_part(parts, at.tile, acc);
          ++at.tile;
        }
        enter(0);
      }
    }
    // a warp without steps leaves zeros: its slot lies among its tile's parts
    if (n == 0 || turn != steps || in_run != 0) store_part(parts, at.tile, acc);
    cp_async_wait<0>();
  }
};

// Sum of a tile's parts at `at` (vector tile * 128 + row * 8 + vector), warp by
// warp: warp_of(v) is the warp whose share has step v of V.
MOE_DEV int warp_of(int v, int V) { return (int)((uint32_t)(kW4Warps * (v + 1) - 1) / (uint32_t)V); }
struct PartRange {
  int first, last;
  // `per`: steps of a tile
  MOE_DEV PartRange(int tile, int tiles, int per)
      : first(warp_of(tile * per, tiles * per)), last(warp_of(tile * per + per - 1, tiles * per)) {}
};
MOE_DEV float sum_parts(const float* parts, int slot_floats, int tile, const PartRange& w, int at) {
  float s = 0.0f;
  for (int i = w.first; i <= w.last; ++i) s += parts[(tile + i) * slot_floats + at];
  return s;
}

// ------------------------------------------------------------------ staged vectors
// Each 128 columns (a stage) of a vector become fp16 after a power of two that
// puts their largest value into [2^13, 2^14): the 8 or 11 significant bits are
// all there down to 2^-27 of the largest value, and what is lost further down
// (2^-38 of it) is below the rounding of the fp32 sums.  LOW keeps a second fp16
// part, 22 bits together.  The table has, for each stage, the factor back to the
// vector's units.
// (The codes themselves as fp16 subnormals, with 8 times a group's sum taken off
// its products, take four instructions fewer for eight weights, but the matrix
// instruction then keeps about 17 bits below the largest value times 8: beside
// a value 1000 times the others whose weight is zero, results were off by 7%.)

// Bytes between staged vectors: 64 more than a multiple of 128, so that two
// rows do not share banks.
__host__ __device__ inline int staged_stride(int K) { return K * 2 + 64; }

struct StagedAt {
  uint32_t x, low;        // vector 0 and its low parts
  int stride;             // bytes between vectors
  uint32_t table;         // entries [stage][vectors of the table]
};

MOE_DEV void load_f8(const __nv_bfloat16* p, float* f) { widen8(load8<__nv_bfloat16, 8>(p, 0, 1, 8), f); }
MOE_DEV void load_f8(const __half* p, float* f) { widen8(load8<__half, 8>(p, 0, 1, 8), f); }
MOE_DEV void load_f8(const float* p, float* f) { widen8(load8<float, 8>(p, 0, 1, 8), f); }

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
      if (base + u * kW4Threads >= all) break;
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
      if (base + u * kW4Threads >= all) break;
      float top = 0.0f;
#pragma unroll
      for (int j = 0; j < 8; ++j) top = fmaxf(top, fabsf(f[u][j]));
#pragma unroll
      for (int off = 1; off < 16; off <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
      const int k = top > 0.0f ? max(min(140 - (int)(__float_as_uint(top) >> 23), 126), -114) : 0;
      const float scale = exp2i(k);
      uint32_t hi[4], lo[4];
#pragma unroll
      for (int q = 0; q < 4; ++q) {   // columns q and q + 4
        const float a = f[u][q] * scale, b = f[u][q + 4] * scale;
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
      if ((c[u] & 15) == 0) {
        const int stage = c[u] >> 4;
        const uint32_t entry = at.table + (VC > 1 ? stage * VC + m[u] : m[u] * (K / 128) + stage) * 4;
        asm volatile("st.shared.f32 [%0], %1;" ::"r"(entry), "f"(exp2i(-k)) : "memory");
      }
    }
  }
}

// Where this lane finds its staged vectors, `here` of them (places past the last
// repeat it, unused).
template <typename T, int NT> MOE_DEV void staged_at(Vectors<T, NT>& v, const StagedAt& at, int here) {
  const int g = (threadIdx.x & 31) >> 2, t = threadIdx.x & 3;
  v.s = at.x + min(g, here - 1) * at.stride;
  v.s_low = v.s + (at.low - at.x);
#pragma unroll
  for (int m = 0; m < NT; ++m) v.to[m] = (min(m * 8 + g, here - 1) - min(g, here - 1)) * at.stride;
  v.table = at.table + t * 8;
}

// Launch a kernel that may have as much dynamic shared memory as there is beside its
// `static_bytes`.
template <typename... KArgs, typename... Args>
cudaError_t launch_w4(SmemLimit& limit, void (*kernel)(KArgs...), dim3 grid, size_t smem, int static_bytes,
                      cudaStream_t s, Args&&... args) {
  const cudaError_t e = limit.raise(reinterpret_cast<const void*>(kernel), kSmemMost - static_bytes);
  if (e != cudaSuccess) return e;
  return launch_pdl(kernel, grid, dim3(kW4Threads), smem, s, std::forward<Args>(args)...);
}

}  // namespace moe
