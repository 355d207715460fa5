// Matrix product of e4m3 operands with an fp32 scale for each block of 128 along k:
//   out[i][j] = sum over blocks c of sa[i][c] sb[j / b_rows][c] (sum over the block's k of a[i][k] b[j][k])
//
// A block's inner sum is matrix instructions' work (two v_mfma_f32_32x32x64_f8f6f4 for 32 x 32 results in large products,
// one v_mfma_f32_16x16x128_f8f6f4 for 16 x 16 where a has few rows); it goes into the fp32 sums times the product of the two
// scales, one fma for each result and block.  (The scales meet first in every kernel: an inner sum, 2^24 at most, times one of
// them may be out of range where their product is an ordinary number.)  b is the first operand, so that a lane's results are of
// one row of a, with one scale of a for them all, and neighbours in it, for wide stores.
//
// Inside, the 8-bit matrix instructions (of every shape) align their products to the largest of a group and drop what lies
// below about 2^-12 of it: measured 1.4e-5 of the result's 2-norm for values of a normal distribution, 5e-5 for codes drawn
// evenly (3.1e-4 to 5.6e-4 between the rounded results and the correctly rounded ones).  A bf16 result, whose own rounding is
// 1.7e-3, is computed with them: the bf16 instructions, which drop nothing, have half their rate.  An fp32 result (a weight
// gradient) is not: its codes become bf16, which holds them exactly, on the way into the bf16 matrix instructions, which sum in
// fp32 (1.5e-7).
//
// Large products are bound by the matrix cores, the fmas that apply the scales (a quarter of the vector unit's cycles: with
// instructions of 16 x 16 x 128, whose results come twice as often for the same work, a loop without memory reached 3562 TF,
// with these 4015) and, above all, by the copies into LDS that run beside them: 8192^3 takes 540 us, without the copies 440.
// Measured, bf16 results and one scale for 128 rows of b: 16384 x 10576 x 2560 437 to 468 us (2030 to 1900 TF; the matrix cores
// are busy 57 % of the time, the clock falls to 1.9 GHz under the power limit; a library product with one scale for each whole
// tensor takes 392 to 470), 4099 x 2560 x 5120 58 to 62 us; rows of b with scales of their own: 10576 x 2560 x 8192 344 to 370
// us (tiles of 128 x 128, whose copies are twice those of 256 x 256 for the same products, and two vector operations for each
// result and block), with fp32 results 470 to 510 (945 to 870 TF), bound by the conversions, those operations and power.
// Products of one turn are bound by a CU's copies (about 45 B/ns): 256 x 10576 x 2560 15 us, 1000 x 2560 x 2560 15.8 (library
// 15.7 for 1024).  Few rows are bound by the reading of b: 1 row at 10576 x 2560 7.6 us (3.6 TB/s with the launch).
//
// Tried and not kept, for the large products: four waves of 128 x 128 results each (their sums move between register files:
// 801 us at 8192^3), lines touched ahead of their copies (5 to 10 % slower), all of a stage's copies at once (3 % slower), raised
// priority around the matrix instructions (15 % slower), 12 or 16 waves over 192 x 256 (4099 x 2560 x 5120 65.7 us for 62.5);
// for few tiles k split over workgroups with a join (512 x 2560 x 2560 24.9 us; 11.8 now).
#include "fp8.hpp"

namespace ssm57 {
namespace {

typedef int v8i __attribute__((ext_vector_type(8)));
typedef int v4i __attribute__((ext_vector_type(4)));
typedef __bf16 v8bf __attribute__((ext_vector_type(8)));
typedef __attribute__((address_space(3))) void lds_mvoid;

struct MatmulArgs {
  const uint8_t* a;
  const uint8_t* b;
  const float* sa;
  const float* sb;
  void* out;
  int64_t as, bs, os, sas, sbs;
  int m, n, k, blocks;    // blocks of 128 along k
  int tiles_m, tiles_n;
  int whole, halved;      // tiles, and tiles in halves behind them
};

typedef float v16f __attribute__((ext_vector_type(16)));

// what lies at an address of LDS
template <typename T>
__device__ __forceinline__ T from_lds(uint32_t at) {
  return *reinterpret_cast<__attribute__((address_space(3))) const T*>(static_cast<uintptr_t>(at));
}

__device__ __forceinline__ v8bf widen(int lo, int hi) {
  const pbf2 a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.0f, false), b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.0f, true);
  const pbf2 c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.0f, false), d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.0f, true);
  return v8bf{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}

// A lane's 32 codes of a row, as they are or as bf16: half a block (64 k) of 32 rows, or a block of 16.
template <bool WIDE>
struct Frag {
  v8i v;
  __device__ __forceinline__ void set(v8i x) { v = x; }
};
template <>
struct Frag<true> {
  v8bf v[4];
  __device__ __forceinline__ void set(v8i x) {
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = widen(x[2 * i], x[2 * i + 1]);
  }
};
__device__ __forceinline__ v16f mfma_half(const Frag<false>& b, const Frag<false>& a, v16f d) {
  return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(b.v, a.v, d, 0, 0, 0, 0, 0, 0);
}
__device__ __forceinline__ v16f mfma_half(const Frag<true>& b, const Frag<true>& a, v16f d) {
#pragma unroll
  for (int i = 0; i < 4; ++i) d = __builtin_amdgcn_mfma_f32_32x32x16_bf16(b.v[i], a.v[i], d, 0, 0, 0);
  return d;
}

// A whole block of 16 rows.
__device__ __forceinline__ pf4 mfma_block(const Frag<false>& b, const Frag<false>& a) {
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(b.v, a.v, pf4{0.0f, 0.0f, 0.0f, 0.0f}, 0, 0, 0, 0, 0, 0);
}
__device__ __forceinline__ pf4 mfma_block(const Frag<true>& b, const Frag<true>& a) {
  pf4 d{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
  for (int i = 0; i < 4; ++i) d = __builtin_amdgcn_mfma_f32_16x16x32_bf16(b.v[i], a.v[i], d, 0, 0, 0);
  return d;
}
__device__ __forceinline__ v8i join(v4i lo, v4i hi) { return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7); }

// Neighbouring results of a row, four (eight) of them, of which cnt are inside the row.
template <typename TO>
__device__ __forceinline__ void store4(TO* p, pf4 v, int cnt) {
  if constexpr (sizeof(TO) == 4) {
    if (cnt >= 4) *reinterpret_cast<pf4u*>(p) = v;
    else
#pragma unroll
      for (int i = 0; i < 3; ++i)
        if (i < cnt) p[i] = v[i];
  } else {
    typedef uint32_t u2e __attribute__((ext_vector_type(2), aligned(2)));
    if (cnt >= 4) *reinterpret_cast<u2e*>(p) = u2e{pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3])};
    else
#pragma unroll
      for (int i = 0; i < 3; ++i)
        if (i < cnt) Elem<uint16_t>::st(p, i, v[i]);
  }
}
template <typename TO>
__device__ __forceinline__ void store8(TO* p, pf4 v, pf4 w, int cnt) {
  if (cnt >= 8 && sizeof(TO) == 2) {
    *reinterpret_cast<pu4e*>(p) = pu4{pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(w[0], w[1]), pack_bf16(w[2], w[3])};
  } else {
    store4<TO>(p, v, cnt);
    store4<TO>(p + 4, w, cnt - 4);
  }
}

__device__ __forceinline__ __amdgpu_buffer_rsrc_t bytes_rsrc(const void* base, uint32_t bytes) {   // at most 2^31
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(base), static_cast<short>(0), static_cast<int>(bytes),
                                           static_cast<int>(kRsrcWord3));
}
// Values that are the same in a whole wave, in scalar registers.
__device__ __forceinline__ uint32_t uniform(uint32_t v) { return __builtin_amdgcn_readfirstlane(v); }
template <typename T>
__device__ __forceinline__ T* uniform(T* p) {
  const uint64_t v = reinterpret_cast<uint64_t>(p);
  return reinterpret_cast<T*>(uint64_t(uniform(static_cast<uint32_t>(v >> 32))) << 32 | uniform(static_cast<uint32_t>(v)));
}
// Waits until at most N of this wave's memory operations, or none of its LDS operations, are under way.  (The empty asm
// keeps the compiler from moving reads and copies over the wait.)
template <int N = 0>
__device__ __forceinline__ void wait_memory() {
  static_assert(N < 64);
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_waitcnt(0x0F70 | (N & 15) | (N >> 4 << 14));
  asm volatile("" ::: "memory");
}
__device__ __forceinline__ void barrier() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}
__device__ __forceinline__ void wait_lds() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_waitcnt(0xC07F);   // lgkmcnt(0)
  asm volatile("" ::: "memory");
}

template <int TM, int WM, int WN, int BROWS>
constexpr int kTileLds = 2 * (32 * TM * WM + 64 * WN) * 128 +
                         4 * 256 * ((32 * TM * WM / 64 + (BROWS == 1 ? WN : 1) + WM * WN - 1) / (WM * WN)) * WM * WN;

// A workgroup's tiles of (32 TM WM) x (64 WN) results, one after the other; a wave has 32 TM x 64 of them.  The tiles are
// numbers first to first + count, or (PARTS > 1) the parts of that many rows of tiles that are PARTS times as high.
// BROWS: rows of b under one scale.  WIDE: bf16 products.
template <int TM, int WM, int WN, int BROWS, bool WIDE, int PARTS, typename TO>
__device__ __forceinline__ void matmul_tiles(const MatmulArgs& g, uint8_t* lds, int first, int count) {
  constexpr int BM = 32 * TM * WM, BN = 64 * WN, NW = WM * WN, TN = 2;
  constexpr int kA = BM / 8 / NW, kB = BN / 8 / NW;         // a wave's copies of 1 KB (8 rows of a block) in a stage
  constexpr int kScales = BM / 64 + (BROWS == 1 ? BN / 64 : 1), kSlots = (kScales + NW - 1) / NW;
  // A wave's copies of a stage are given out between its products: the first of them a block early, as soon as the stage is
  // free, the others over the next block's first products.  (All at once they hold up the products behind them.)
  constexpr int kCopies = kA + kB + kSlots, kPer = (kCopies + TM * TN - 1) / (TM * TN), kEarly = kPer * TN;
  static_assert(kEarly <= kCopies);
  constexpr int kStores = TM * (sizeof(TO) == 2 ? 4 : 8);   // of a wave's results, where its tile is whole
  constexpr int kStageA = BM * 128, kStageB = BN * 128, kStageS = 256 * kSlots * NW;
  static_assert(BM / 8 % NW == 0 && BN / 8 % NW == 0 && NW % 2 == 0 && TM >= 2);
  constexpr int kSlotsA = TM % 2 ? 3 : 2;                   // fragments of a in registers: the one in use and those ahead
  static_assert(TM % kSlotsA == 0);
  // Two stages of a and of b; four of scales, which are read until the end of a block, when the copies for the one behind
  // the next may be under way.
  static_assert(kTileLds<TM, WM, WN, BROWS> == 2 * (kStageA + kStageB) + 4 * kStageS);
  const uint32_t at_b = 2 * kStageA, at_s = 2 * (kStageA + kStageB);
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wave % WM, wn = wave / WM;
  const int r32 = lane & 31, half = lane >> 5;

  // Workgroups go to the 8 XCDs in turn: each XCD takes a run of tiles that walks along n four tiles of m at a time, so
  // that the 32 tiles it has in work share 4 + 8 panels in its L2.
  const int total = count * PARTS;
  const int xcd = blockIdx.x & 7, each = total / 8, more = total % 8;
  const int step = gridDim.x / 8 + (xcd < static_cast<int>(gridDim.x % 8) ? 1 : 0);
  const int end = (xcd + 1) * each + min(xcd + 1, more);
  struct Place {
    int m0, n0;
  };
  auto place_of = [&](int id) {
    const int tile = first + id / PARTS;
    const int band = tile / (4 * g.tiles_n), in_band = tile % (4 * g.tiles_n), high = min(4, g.tiles_m - 4 * band);
    return Place{((band * 4 + in_band % high) * PARTS + id % PARTS) * BM, in_band / high * BN};
  };

  // A copy's lane has row lane / 8 of eight, and the unit of 16 bytes whose place in LDS is lane % 8: units are exchanged by
  // bits 1 to 3 of the row, so that the rows that 16 lanes read at once lie in different banks.
  const int unit = (lane & 7) ^ (lane >> 4) ^ ((wave & 1) << 2);
  const uint32_t as = static_cast<uint32_t>(g.as), bs = static_cast<uint32_t>(g.bs);
  const uint32_t first_a = (wave * 8 + (lane >> 3)) * as + unit * 16u, first_b = (wave * 8 + (lane >> 3)) * bs + unit * 16u;
  // (a wave's scales are those of a or those of b: one place and one stride)
  uint32_t first_s[kSlots];
#pragma unroll
  for (int i = 0; i < kSlots; ++i) {
    const int p = wave + NW * i;
    first_s[i] = p < BM / 64 ? 4u * (p * 64 + lane) * static_cast<uint32_t>(g.sas)
                             : 4u * ((p - BM / 64) * 64 + lane) * static_cast<uint32_t>(g.sbs);
  }
  // The ranges of the tile that is copied next begin at its first block and end with its last row; the block is an offset that
  // the check of the range may or may not count: rows behind the last one are out of range either way.
  __amdgpu_buffer_rsrc_t ra, rb, rs[kSlots];
  int lid = xcd * each + min(xcd, more) + (blockIdx.x >> 3);   // the tile's number
  int block = 0, left = 0;                      // the block in it, and what is left of k
  auto enter = [&]() {
    const Place t = place_of(lid);
    const int m0 = min(t.m0, g.m - 1);          // (a part may lie behind the last row: it reads that one, and writes nothing)
    const int rows_m = min(BM, g.m - m0), rows_n = min(BN, g.n - t.n0);
    const int sb_rows = BROWS == 1 ? rows_n : min(BN / 128 + 1, (g.n - t.n0 / 128 * 128 + 127) / 128);
    block = 0;
    left = g.k;
    ra = bytes_rsrc(uniform(g.a + m0 * g.as), uniform(static_cast<uint32_t>(rows_m - 1) * as + g.k));
    rb = bytes_rsrc(uniform(g.b + t.n0 * g.bs), uniform(static_cast<uint32_t>(rows_n - 1) * bs + g.k));
#pragma unroll
    for (int i = 0; i < kSlots; ++i) {
      const bool of_a = wave + NW * i < BM / 64;
      rs[i] = bytes_rsrc(uniform(of_a ? g.sa + m0 * g.sas : g.sb + t.n0 / BROWS * g.sbs),
                         uniform(4u * ((of_a ? static_cast<uint32_t>(rows_m - 1) * static_cast<uint32_t>(g.sas)
                                             : static_cast<uint32_t>(sb_rows - 1) * static_cast<uint32_t>(g.sbs)) + g.blocks)));
    }
  };
  // copy i of a wave's copies of a stage (past the end of k, behind the last row, and in slots behind the last scale: zeros)
  auto copy = [&](int s, int ss, int i) {
    const bool in = unit * 16 < left;
    if (i < kA)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(ra, (lds_mvoid*)(lds + s * kStageA + (wave + NW * i) * 1024), 16,
                                               static_cast<int>((in ? first_a : kDropOffset) + i * NW * 8 * as), block * 128, 0, 0);
    else if (i < kA + kB)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rb, (lds_mvoid*)(lds + at_b + s * kStageB + (wave + NW * (i - kA)) * 1024), 16,
                                               static_cast<int>((in ? first_b : kDropOffset) + (i - kA) * NW * 8 * bs), block * 128, 0, 0);
    else
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rs[i - kA - kB], (lds_mvoid*)(lds + at_s + ss * kStageS + (wave + NW * (i - kA - kB)) * 256),
                                               4, static_cast<int>(left > 0 ? first_s[i - kA - kB] : kDropOffset), block * 4, 0, 0);
  };
  auto advance = [&]() {   // to the block behind the one that was copied last; behind the last of all there are zeros
    ++block;
    left -= 128;
    if (left <= 0) {
      lid += step;
      if (lid < end) enter();
      else lid = end, left = 0;
    }
  };

  // Where a lane reads in a stage: rows of a in order; rows of b such that a lane's 32 results are runs of 8 neighbours: the
  // matrix instruction's row 8 q + 4 h + r of fragment j, which is register 4 q + r of the lanes with half h, is row
  // 32 j + 16 (q / 2) + 8 h + 4 (q % 2) + r.
  const int key_a = (r32 >> 1) & 7;
  const int row_b = ((r32 >> 4) << 4) | (((r32 >> 2) & 1) << 3) | (((r32 >> 3) & 1) << 2) | (r32 & 3);
  const int key_b = (row_b >> 1) & 7;
  // (half a block kh of a row is units 4 kh + 2 half and the one behind it)
  const uint32_t base = static_cast<uint32_t>(reinterpret_cast<uintptr_t>((lds_mvoid*)lds));
  const uint32_t at_frag_a = base + (wm * TM * 32 + r32) * 128 + ((2 * half) ^ key_a) * 16;
  const uint32_t at_frag_b = base + at_b + (wn * 64 + row_b) * 128 + ((2 * half) ^ key_b) * 16;
  const uint32_t at_scale = base + at_s + (wm * TM * 32 + r32) * 4;
  int cur = 0, cur_s = 0;
  auto read_a = [&](int s, int i, int kh) {
    const uint32_t p = at_frag_a + s * kStageA;
    return __builtin_shufflevector(from_lds<v4i>((p ^ (kh * 64)) + i * 4096), from_lds<v4i>((p ^ (kh * 64 + 16)) + i * 4096), 0, 1, 2, 3, 4, 5, 6, 7);
  };
  auto read_b = [&](int s, int j, int kh) {
    const uint32_t p = at_frag_b + s * kStageB;
    return __builtin_shufflevector(from_lds<v4i>((p ^ (kh * 64)) + j * 4096), from_lds<v4i>((p ^ (kh * 64 + 16)) + j * 4096), 0, 1, 2, 3, 4, 5, 6, 7);
  };

  int id = lid;
  if (id >= end) return;
  enter();
#pragma unroll
  for (int i = 0; i < kCopies; ++i) copy(0, 0, i);
  advance();
#pragma unroll
  for (int i = 0; i < kEarly; ++i) copy(1, 1, i);
  wait_memory<kEarly>();
  barrier();

  Frag<WIDE> bf[TN][2];
  v8i af[kSlotsA][2];
  float sa[kSlotsA];
  Place t = place_of(id);
  bool stored = false, ahead = false;
#pragma unroll
  for (int kh = 0; kh < 2; ++kh) {
    af[0][kh] = read_a(0, 0, kh);
#pragma unroll
    for (int j = 0; j < TN; ++j) bf[j][kh].set(read_b(0, j, kh));
  }
  sa[0] = from_lds<float>(at_scale);
  float sb = BROWS == 1 ? 1.0f : from_lds<float>(base + at_s + BM * 4 + (t.n0 % 128 + wn * 64) / 128 * 4);

  while (true) {
    v16f acc[TM][TN] = {};
    v16f d[2];
    float s[2] = {0.0f, 0.0f};
    d[1] = v16f{};
    // the product k (fragment k / 2 of a, k % 2 of b) of the block with its scales in stage ss goes into the sums
    auto add = [&](int k, int ss) {
      v16f& to = acc[k / TN][k % TN];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        pf4 sbn[2];
        if constexpr (BROWS == 1) {
          const uint32_t p = base + at_s + ss * kStageS + BM * 4 + (wn * 64 + k % TN * 32 + h * 16 + half * 8) * 4;
          sbn[0] = from_lds<pf4>(p);
          sbn[1] = from_lds<pf4>(p + 16);
        }
#pragma unroll
        for (int r = 8 * h; r < 8 * h + 8; ++r)
          to[r] = fmaf(d[k & 1][r], BROWS == 1 ? sbn[(r - 8 * h) / 4][r % 4] * s[(k / TN) & 1] : s[(k / TN) & 1], to[r]);
      }
      asm volatile("" : "+v"(to));   // (here, not at the end of the block)
    };
    for (int c = 0; c < g.blocks; ++c) {
      const int nx = cur ^ 1, nx_s = (cur_s + 1) & 3;
      const int n_next = c + 1 == g.blocks && id + step < end ? place_of(id + step).n0 : t.n0;
#pragma unroll
      for (int i = 0; i < TM; ++i) {
        if (i + 1 < TM) {
          const int to = (i + 1) % kSlotsA;
#pragma unroll
          for (int kh = 0; kh < 2; ++kh) af[to][kh] = read_a(cur, i + 1, kh);
          sa[to] = from_lds<float>(at_scale + cur_s * kStageS + (i + 1) * 128);
        }
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int j = 0; j < TN; ++j) {
          const int k = i * TN + j;
          // A product's two instructions, then the sums of the one before it: as many instructions lie between a result and its
          // use as the matrix cores need, and they work on this product meanwhile.
#pragma unroll
          for (int kh = 0; kh < 2; ++kh) {
            Frag<WIDE> fa;
            fa.set(af[i % kSlotsA][kh]);
            d[k & 1] = mfma_half(bf[j][kh], fa, kh ? d[k & 1] : v16f{});
          }
          __builtin_amdgcn_sched_barrier(0);
          if (i == TM - 1 && j == 0) {
            // All of this wave's reads of the stage (but scales) are done, and its part of the next one has arrived: behind the
            // barrier that holds for every wave, so the next block's fragments can be read and this stage filled again.
            // (Behind the last block what is copied and read is not used.)
            wait_lds();
            if (stored) wait_memory<kStores>();   // (results on their way out were given to memory behind those copies)
            else wait_memory();
            stored = false;
            barrier();
#pragma unroll
            for (int kh = 0; kh < 2; ++kh) af[0][kh] = read_a(nx, 0, kh);
            sa[0] = from_lds<float>(at_scale + nx_s * kStageS);
          }
          if (i == TM - 1) {
#pragma unroll
            for (int e = kPer * j; e < kPer * (j + 1); ++e) copy(cur, (cur_s + 2) & 3, e);
            if (j == TN - 1) {
              ahead = c + 1 == g.blocks;   // (before results are stored all of them: they are waited for without those)
              if (ahead)
#pragma unroll
                for (int e = kEarly; e < kCopies; ++e) copy(cur, (cur_s + 2) & 3, e);
            }
          } else if (kEarly + kPer * k < kCopies) {
            if (!ahead)
#pragma unroll
              for (int e = kEarly + kPer * k; e < min(kEarly + kPer * (k + 1), kCopies); ++e) copy(nx, nx_s, e);
          }
          if (k == TN * (TM - 1) - 1) advance();
          // (the block's last product goes into the sums in the next one)
          if (k > 0) add(k - 1, cur_s);
          else if (BROWS != 1 || c > 0) add(TM * TN - 1, (cur_s + 3) & 3);
          if (j == 0) s[i & 1] = sa[i % kSlotsA] * sb;
          if (i == TM - 1) {
#pragma unroll
            for (int kh = 0; kh < 2; ++kh) bf[j][kh].set(read_b(nx, j, kh));
          }
          __builtin_amdgcn_sched_barrier(0);
        }
      }
      if constexpr (BROWS != 1) sb = from_lds<float>(base + at_s + nx_s * kStageS + BM * 4 + (n_next % 128 + wn * 64) / 128 * 4);
      cur = nx;
      cur_s = nx_s;
    }
    add(TM * TN - 1, (cur_s + 3) & 3);
    TO* out = static_cast<TO*>(g.out);
    const int col = t.n0 + wn * 64 + half * 8;
#pragma unroll
    for (int i = 0; i < TM; ++i) {
      const int row = t.m0 + (wm * TM + i) * 32 + r32;
      if (row < g.m)
#pragma unroll
        for (int j = 0; j < TN; ++j)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const v16f& v = acc[i][j];
            const int e = col + 32 * j + 16 * h;
            store8<TO>(out + row * g.os + e, pf4{v[8 * h], v[8 * h + 1], v[8 * h + 2], v[8 * h + 3]},
                       pf4{v[8 * h + 4], v[8 * h + 5], v[8 * h + 6], v[8 * h + 7]}, g.n - e);
          }
    }
    stored = t.m0 + BM <= g.m && t.n0 + BN <= g.n;
    id += step;
    if (id >= end) break;
    t = place_of(id);
  }
  wait_memory();   // (the zeros that were copied behind the last block: LDS is given up only now)
}

// The tiles of a product.  HALVES: those of the last turn are cut in two, so that as many workgroups again have work in it.
template <int TM, int WM, int WN, int BROWS, bool WIDE, bool HALVES, typename TO>
__global__ void __launch_bounds__(64 * WM * WN, 2) matmul_tile_kernel(MatmulArgs g) {
  __shared__ __align__(1024) uint8_t lds[kTileLds<TM, WM, WN, BROWS>];
  matmul_tiles<TM, WM, WN, BROWS, WIDE, 1, TO>(g, lds, 0, g.whole);
  if constexpr (HALVES) {
    if (g.halved > 0) {
      __syncthreads();
      matmul_tiles<TM / 2, WM, WN, BROWS, WIDE, 2, TO>(g, lds, g.whole, g.halved);
    }
  }
}

// Tiles that all run at a time, one to a CU, with nothing beside them that would cover their waits: three stages of LDS, so that
// a block's copies have two blocks' time, and 8 or 12 waves with one or two fragments of results each, for whose products, LDS
// reads and fmas the other waves on a SIMD make up.  (768 x 2560 x 2560 in 240 tiles of 128 x 64 12.1 us; 21.5 in tiles of
// 128 x 128 as above, of 128 x 64 20.9, and the same with operands in the L2: a block took as long as its copies' way.  Five
// stages 13.3; 1000 x 2560 x 2560 in 216 tiles of 128 x 96 by 12 waves 14.9, by four with three fragments each 19.2.)
// Lanes, swizzle and fragments are those of matmul_tiles.
template <int TM, int WM, int WN, int BROWS>
__global__ void __launch_bounds__(64 * WM * WN) matmul_own_kernel(MatmulArgs g) {
  constexpr int BM = 32 * TM * WM, BN = 32 * WN, NW = WM * WN, S = 3;
  // A stage's copies, given to the waves in turn: 1 KB each of a and of b (8 rows of a block), then the scales of 64 rows each.
  constexpr int kA = BM / 8, kAB = (BM + BN) / 8, kSB = kAB + BM / 64, kAll = kSB + (BROWS == 1 ? (BN + 63) / 64 : 1);
  constexpr int kCopies = (kAll + NW - 1) / NW, kStage = (BM + BN) * 128 + 256 * (kCopies * NW - kAB);
  static_assert(BM % 64 == 0 && BN % 32 == 0 && NW % 2 == 0 && S * kStage <= 163840);
  __shared__ __align__(1024) uint8_t lds[S * kStage];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wave % WM, wn = wave / WM, r32 = lane & 31, half = lane >> 5;
  const int xcd = blockIdx.x & 7, id = xcd * (gridDim.x / 8) + min(xcd, static_cast<int>(gridDim.x % 8)) + (blockIdx.x >> 3);
  const int m0 = id % g.tiles_m * BM, n0 = id / g.tiles_m * BN;
  const int rows_m = min(BM, g.m - m0), rows_n = min(BN, g.n - n0);

  const int unit = (lane & 7) ^ (lane >> 4) ^ ((wave & 1) << 2);
  const uint32_t as = static_cast<uint32_t>(g.as), bs = static_cast<uint32_t>(g.bs);
  const uint32_t sas = static_cast<uint32_t>(g.sas), sbs = static_cast<uint32_t>(g.sbs);
  const uint32_t first_a = (wave * 8 + (lane >> 3)) * as + unit * 16u, first_b = (wave * 8 + (lane >> 3)) * bs + unit * 16u;
  const auto ra = bytes_rsrc(uniform(g.a + m0 * g.as), uniform(static_cast<uint32_t>(rows_m - 1) * as + g.k));
  const auto rb = bytes_rsrc(uniform(g.b + n0 * g.bs), uniform(static_cast<uint32_t>(rows_n - 1) * bs + g.k));
  const uint32_t last_sb = BROWS == 1 ? rows_n - 1 : (n0 % 128 + rows_n - 1) / 128;
  const auto rsa = bytes_rsrc(uniform(g.sa + m0 * g.sas), uniform(4u * (static_cast<uint32_t>(rows_m - 1) * sas + g.blocks)));
  const auto rsb = bytes_rsrc(uniform(g.sb + n0 / BROWS * g.sbs), uniform(4u * (last_sb * sbs + g.blocks)));
  // block c into a stage (past the end of k, behind the last row, and behind the last scale: zeros)
  auto copy = [&](int c, int s) {
    uint8_t* to = lds + s * kStage;
    const bool in = unit * 16 < g.k - c * 128;
#pragma unroll
    for (int i = 0; i < kCopies; ++i) {
      const int p = wave + NW * i;   // (the same branch for a whole wave)
      if (p < kA)
        __builtin_amdgcn_raw_ptr_buffer_load_lds(ra, (lds_mvoid*)(to + p * 1024), 16,
                                                 static_cast<int>((in ? first_a : kDropOffset) + i * NW * 8 * as), c * 128, 0, 0);
      else if (p < kAB)
        __builtin_amdgcn_raw_ptr_buffer_load_lds(rb, (lds_mvoid*)(to + p * 1024), 16,
                                                 static_cast<int>((in ? first_b : kDropOffset) + (i * NW - kA) * 8 * bs), c * 128, 0, 0);
      else
        __builtin_amdgcn_raw_ptr_buffer_load_lds(p < kSB ? rsa : rsb, (lds_mvoid*)(to + kAB * 1024 + (p - kAB) * 256), 4,
                                                 static_cast<int>(c < g.blocks ? 4u * (((p - (p < kSB ? kAB : kSB)) * 64 + lane) *
                                                                                       (p < kSB ? sas : sbs)) : kDropOffset),
                                                 c * 4, 0, 0);
    }
  };
#pragma unroll
  for (int c = 0; c < S - 1; ++c) copy(c, c);

  const int key_a = (r32 >> 1) & 7;
  const int row_b = ((r32 >> 4) << 4) | (((r32 >> 2) & 1) << 3) | (((r32 >> 3) & 1) << 2) | (r32 & 3);
  const int key_b = (row_b >> 1) & 7;
  const uint32_t base = static_cast<uint32_t>(reinterpret_cast<uintptr_t>((lds_mvoid*)lds));
  const uint32_t at_a = base + (wm * TM * 32 + r32) * 128 + ((2 * half) ^ key_a) * 16;
  const uint32_t at_b = base + BM * 128 + (wn * 32 + row_b) * 128 + ((2 * half) ^ key_b) * 16;
  const uint32_t at_sa = base + (BM + BN) * 128 + (wm * TM * 32 + r32) * 4, at_sb = base + (BM + BN) * 128 + BM * 4;
  v16f acc[TM] = {};
  int s = 0;
  for (int c = 0; c < g.blocks; ++c) {
    wait_memory<(S - 2) * kCopies>();
    barrier();   // (block c has arrived, and every wave has read block c - 1)
    copy(c + S - 1, s == 0 ? S - 1 : s - 1);
    const uint32_t o = s * kStage;
    Frag<false> fa[TM][2], fb[2];
    float sa[TM], sb = 1.0f;
    pf4 sbn[4];
#pragma unroll
    for (int kh = 0; kh < 2; ++kh) {
      fb[kh].set(join(from_lds<v4i>((at_b + o) ^ (kh * 64)), from_lds<v4i>((at_b + o) ^ (kh * 64 + 16))));
#pragma unroll
      for (int i = 0; i < TM; ++i)
        fa[i][kh].set(join(from_lds<v4i>(((at_a + o) ^ (kh * 64)) + i * 4096), from_lds<v4i>(((at_a + o) ^ (kh * 64 + 16)) + i * 4096)));
    }
#pragma unroll
    for (int i = 0; i < TM; ++i) sa[i] = from_lds<float>(at_sa + o + i * 128);
    if constexpr (BROWS == 1) {
#pragma unroll
      for (int h = 0; h < 4; ++h) sbn[h] = from_lds<pf4>(at_sb + o + (wn * 32 + h / 2 * 16 + half * 8 + h % 2 * 4) * 4);
    } else {
      sb = from_lds<float>(at_sb + o + (n0 % 128 + wn * 32) / 128 * 4);
    }
#pragma unroll
    for (int i = 0; i < TM; ++i) {
      v16f d{};
#pragma unroll
      for (int kh = 0; kh < 2; ++kh) d = mfma_half(fb[kh], fa[i][kh], d);
      const float t = sa[i] * sb;
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[i][r] = fmaf(d[r], BROWS == 1 ? sbn[r / 4][r % 4] * t : t, acc[i][r]);
    }
    wait_lds();
    s = s + 1 == S ? 0 : s + 1;
  }
  uint16_t* out = static_cast<uint16_t*>(g.out);
#pragma unroll
  for (int i = 0; i < TM; ++i) {
    const int row = m0 + (wm * TM + i) * 32 + r32;
    if (row < g.m)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const v16f& v = acc[i];
        const int e = n0 + wn * 32 + 16 * h + half * 8;
        store8<uint16_t>(out + row * g.os + e, pf4{v[8 * h], v[8 * h + 1], v[8 * h + 2], v[8 * h + 3]},
                         pf4{v[8 * h + 4], v[8 * h + 5], v[8 * h + 6], v[8 * h + 7]}, g.n - e);
      }
  }
  wait_memory();   // (the zeros that were copied behind the last block: LDS is given up only now)
}

// Few rows of a, or few tiles: a workgroup has 16 MT rows of a and 16 NT of b and is bound by the reading of them.  Its W waves
// take the blocks of k in turn, each with a stage of its own in LDS that it alone fills and reads, so that no wave waits for
// another, and the waves' sums are joined in LDS in a fixed order.  (Read straight into registers, 16 rows and half a line of
// each to an instruction, the operands took 1.05 to 1.8 times as long.)
// v_mfma_f32_16x16x128_f8f6f4: a lane has 32 codes of row lane % 16 of a and of b, and the result's four neighbouring j.
template <int MT, int NT, int W, int BROWS, bool WIDE, typename TO>
__global__ void __launch_bounds__(64 * W) matmul_few_kernel(MatmulArgs g) {
  constexpr int kStage = (MT + NT) * 2048, kPart = MT * NT * 1024;
  // sums that need more memory than the stages are joined in two steps
  constexpr int kParts = kPart > kStage ? W / 2 : W;
  static_assert(kParts * kPart <= W * kStage);
  __shared__ __align__(1024) uint8_t lds[W * kStage];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r16 = lane & 15, kg = lane >> 4;
  // (as in the tiles the workgroups that share rows of b are neighbours on one XCD: 512 x 2560 x 2560 11.8 us, and 15.9 without)
  const int xcd = blockIdx.x & 7, id = xcd * (gridDim.x / 8) + min(xcd, static_cast<int>(gridDim.x % 8)) + (blockIdx.x >> 3);
  const int m0 = id % g.tiles_m * 16 * MT, n0 = id / g.tiles_m * 16 * NT;
  const int rows_m = min(16 * MT, g.m - m0), rows_n = min(16 * NT, g.n - n0);
  const uint32_t as = static_cast<uint32_t>(g.as), bs = static_cast<uint32_t>(g.bs);
  const auto ra = bytes_rsrc(g.a + m0 * g.as, static_cast<uint32_t>(rows_m - 1) * as + g.k);
  const auto rb = bytes_rsrc(g.b + n0 * g.bs, static_cast<uint32_t>(rows_n - 1) * bs + g.k);
  const auto rsa = make_rsrc(g.sa + m0 * g.sas, (rows_m - 1) * g.sas + g.blocks);
  const auto rsb = make_rsrc(g.sb + n0 / BROWS * g.sbs, (BROWS == 1 ? rows_n - 1 : (n0 % 128 + rows_n - 1) / 128) * g.sbs + g.blocks);
  uint8_t* stage = lds + wave * kStage;          // rows of b, then of a
  constexpr int kSa = (MT + 3) / 4, kSb = BROWS == 1 ? (NT + 3) / 4 : 1;
  float sa[kSa] = {}, sb[kSb] = {};              // of rows `lane`, `lane` + 64 of a and of b; or of the block of 16 rows `lane` of b
  const uint32_t at_sb = BROWS == 1 ? lane * static_cast<uint32_t>(g.sbs)
                                    : (n0 % 128 + lane % NT * 16) / 128 * static_cast<uint32_t>(g.sbs);
  const int unit = (lane & 7) ^ (lane >> 4);     // as in the tiles; the second of two copies has it ^ 4
  auto load = [&](int c) {
    // (past the end of k, and behind the last row: zeros)
#pragma unroll
    for (int p = 0; p < 2 * (MT + NT); ++p) {
      const int q = p < 2 * NT ? p : p - 2 * NT, at = (unit ^ (p % 2 * 4)) * 16;
      const uint32_t o = (q * 8 + (lane >> 3)) * (p < 2 * NT ? bs : as) + c * 128u + at;
      __builtin_amdgcn_raw_ptr_buffer_load_lds(p < 2 * NT ? rb : ra, (lds_mvoid*)(stage + p * 1024), 16,
                                               static_cast<int>(at < g.k - c * 128 ? o : kDropOffset), 0, 0, 0);
    }
#pragma unroll
    for (int i = 0; i < kSa; ++i)
      sa[i] = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(
          rsa, static_cast<int>(4u * ((lane % (16 * MT) + 64 * i) * static_cast<uint32_t>(g.sas) + c)), 0, 0));
#pragma unroll
    for (int i = 0; i < kSb; ++i)
      sb[i] = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(
          rsb, static_cast<int>(4u * (at_sb + 64 * i * static_cast<uint32_t>(g.sbs) + c)), 0, 0));
  };
  const uint8_t* frag = stage + r16 * 128 + (kg ^ (r16 >> 1)) * 16;
  auto read = [&](int f) {                       // (units kg and kg + 4 of a row)
    const uint8_t* p = frag + f * 2048;
    const uint8_t* q = stage + r16 * 128 + (((kg ^ (r16 >> 1)) * 16) ^ 64) + f * 2048;
    return join(*reinterpret_cast<const v4i*>(p), *reinterpret_cast<const v4i*>(q));
  };
  pf4 acc[MT][NT] = {};
  int c = wave;
  if (c < g.blocks) load(c);
  for (; c < g.blocks; c += W) {
    wait_memory();
    v8i va[MT], vb[NT];
#pragma unroll
    for (int j = 0; j < NT; ++j) vb[j] = read(j);
#pragma unroll
    for (int i = 0; i < MT; ++i) va[i] = read(NT + i);
    float sac[kSa];
#pragma unroll
    for (int i = 0; i < kSa; ++i) sac[i] = sa[i];
    float sbc[kSb];
#pragma unroll
    for (int i = 0; i < kSb; ++i) sbc[i] = sb[i];
    wait_lds();                                  // (the stage has been read)
    if (c + W < g.blocks) load(c + W);
    Frag<WIDE> fb[NT];
#pragma unroll
    for (int j = 0; j < NT; ++j) fb[j].set(vb[j]);
    constexpr bool kOne = BROWS != 1 && 128 % (16 * NT) == 0;   // all rows of b here are under one scale
    float sbn[kOne ? 1 : BROWS == 1 ? 4 * NT : NT] = {sbc[0]};
    if constexpr (!kOne) {
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        if constexpr (BROWS == 1) {
#pragma unroll
          for (int r = 0; r < 4; ++r) sbn[4 * j + r] = __shfl(sbc[j / 4], j % 4 * 16 + kg * 4 + r);
        } else {
          sbn[j] = __shfl(sbc[0], j);
        }
      }
    }
#pragma unroll
    for (int i = 0; i < MT; ++i) {
      Frag<WIDE> fa;
      fa.set(va[i]);
      const float s = MT == 1 ? sac[0] : __shfl(sac[i / 4], i % 4 * 16 + r16);
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        const pf4 d = mfma_block(fb[j], fa);
#pragma unroll
        for (int r = 0; r < 4; ++r) acc[i][j][r] = fmaf(d[r], s * sbn[kOne ? 0 : BROWS == 1 ? 4 * j + r : j], acc[i][j][r]);
      }
    }
  }
  __syncthreads();                               // (every stage has been read)
  pf4* part = reinterpret_cast<pf4*>(lds);       // [kParts][MT NT][64]
#pragma unroll
  for (int step = W / kParts - 1; step >= 0; --step) {
    if (wave / kParts == step) {
#pragma unroll
      for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int j = 0; j < NT; ++j) {
          pf4& to = part[(wave % kParts * MT * NT + i * NT + j) * 64 + lane];
          to = step + 1 < W / kParts ? acc[i][j] + to : acc[i][j];
        }
    }
    __syncthreads();
  }
  for (int t = wave; t < MT * NT; t += W) {
    pf4 sum = part[t * 64 + lane];
#pragma unroll
    for (int w = 1; w < kParts; ++w) sum += part[(w * MT * NT + t) * 64 + lane];
    const int row = m0 + t / NT * 16 + r16, col = n0 + t % NT * 16 + kg * 4;
    if (row < g.m) store4<TO>(static_cast<TO*>(g.out) + row * g.os + col, sum, g.n - col);
  }
}

struct MatmulPlan {
  int few;              // fragments of 16 rows of b to a workgroup that shares k among its waves; 0: tiles
  int bm, bn;
  int slots;            // workgroups that run at a time; 0: of the tiles that have a CU to themselves, which all do
};

int few_rows(int64_t m) { return m <= 16 ? 1 : m <= 32 ? 2 : 4; }   // fragments of 16 rows of a to a workgroup

struct FewWidth {
  int nt;
  int64_t cost;
};
// Fragments of b to a workgroup that has mt of a: with more of them a is read less often, with fewer there are more workgroups.
// What counts is the fragments that the busiest CU reads.  (Width 1, 2, 3, 4 and 6 in us, k = 2560: 16 rows at n = 10576 8.7,
// 9.1, 7.7, 8.1, -, at 5120 5.1, 4.6, 5.1, 5.6, -; 64 rows at 10576 15.7, 15.8, 11.0, 11.7, 14.7, at 16384 19.1, 16.0, 18.5,
// 12.8, 15.2; 128 rows at 10576 25.2, 21.6, 18.3, 20.5, 14.9; 512 rows at 2560 -, 16.5, 14.2, 15.5, 11.8.)  With bf16 products
// four fragments of a and six of b do not fit the registers (512 rows at 2560: 16.0 us with three of b, 17.2 with six).
FewWidth few_width(const ssm_matmul_fp8_params* p) {
  const int mt = few_rows(p->m);
  FewWidth best{};
  for (int nt : {1, 2, 3, 4, 6}) {
    if (nt == 6 && mt == 4 && p->out_dtype == SSM_F32) continue;
    const int64_t groups = ((p->m + 16 * mt - 1) / (16 * mt)) * ((p->n + 16 * nt - 1) / (16 * nt));
    const int64_t cost = (groups + 255) / 256 * (mt + nt);
    if (best.nt == 0 || cost < best.cost) best = {nt, cost};
  }
  return best;
}

MatmulPlan plan_of(const ssm_matmul_fp8_params* p) {
  const bool narrow = p->b_rows == kBlock && p->out_dtype == SSM_BF16;
  auto tiles = [&](int64_t bm, int64_t bn) { return ((p->m + bm - 1) / bm) * ((p->n + bn - 1) / bn); };
  // Small products take as long as their busiest CU reads.  Where one tile to a CU is enough for all of them, the smallest such
  // tile, or workgroups that share a tile's k among their waves, whichever has a CU read less (us, shared k and tiles:
  // 512 x 2560 x 2560 11.8, 11.4; 640 x 2560 15.4, 12.1; 256 x 10576 25.5, 18.0; 512 x 5120 22.4, 16.3; 128 x 10576 14.9, 16.3;
  // 768 x 768 x 8192 17.6, 47; 256 x 96 and two tiles of 128 x 128 to a CU: 1024 x 5120 x 2560 22.7, 26.0, 2048 x 2560 x 5120
  // 43.2, 46.7; 192 x 256, 256 x 128 and others of that kind are no faster than the tiles below).  With fp32 results, whose
  // tiles are only those of 128 x 128 below, shared k as far as 16 fragments (512 x 2560 x 2560 16.0 and 29.1 us,
  // 192 x 10576 x 2560 24.0 and 30.4).
  const FewWidth few = few_width(p);
  MatmulPlan own{};
  if (p->out_dtype == SSM_BF16) {
    static const int sizes[][2] = {{128, 64}, {128, 96}, {128, 128}, {256, 96}};
    for (const auto& c : sizes)
      if (tiles(c[0], c[1]) <= 256) {
        own = {0, c[0], c[1], 0};
        break;
      }
  }
  if (p->m <= 64 || few.cost <= (own.bm ? (own.bm + own.bn) / 16 : 16)) return {few.nt, 0, 0, 0};
  if (own.bm) return own;
  // Tiles of 128 x 128, two workgroups to a CU, which wait for their own copies only.  Where a lane has one scale of b for all
  // of its results and the products are 8-bit, the sums of 256 x 256 or 192 x 256 fit the registers of one, and large products
  // are faster so: what the turns of all workgroups take is counted in hundredths of one of 256 x 256 tiles, with the last of
  // those in halves where they fit.  (A turn at k = 8192: 256 rows 125 to 129 us, 192 rows 98 to 112, 128 rows 90, 512 tiles of
  // 128 x 128 82 to 85.  2800 x 2560 x 2560 takes 39, 35 and 29 us in tiles of 256, 192 and 128 rows, 3600 x 2560 x 2560 39, 36
  // and 42.  With a scale for each row of b 10576 x 2560 x 8192 takes 347 us in tiles of 128 x 128 and 407 in tiles of
  // 128 x 256, as fp32 503 and 571.)
  MatmulPlan t{0, 128, 128, 512};
  if (narrow) {
    const int64_t whole = tiles(256, 256), last = whole % 256, small = tiles(128, 128), rest = small % 512;
    const int64_t cost = whole / 256 * 100 + (last == 0 ? 0 : whole > 256 && last <= 128 ? 70 : 100);
    const int64_t low = (tiles(192, 256) + 255) / 256 * 80;
    const int64_t least = small / 512 * 68 + (rest == 0 ? 0 : rest <= 256 ? 45 : 68);
    if (least > (low < cost ? low : cost)) t = {0, low < cost ? 192 : 256, 256, 256};
  }
  return t;
}

ssm_status check_matmul(const ssm_matmul_fp8_params* p) {
  if (!p) return fail(SSM_ERR_NULL, "params is NULL");
  if (p->reserved[0] != 0 || p->reserved[1] != 0) return fail(SSM_ERR_UNSUPPORTED, "reserved must be 0");
  if (p->m < 1 || p->n < 1 || p->k < 1) return fail(SSM_ERR_SHAPE, "m, n and k must be >= 1");
  if (p->m >= (int64_t(1) << 30) || p->n >= (int64_t(1) << 30)) return fail(SSM_ERR_SHAPE, "m and n must be below 2^30");
  if (p->k % 16) return fail(SSM_ERR_SHAPE, "k (%lld) must be a multiple of 16", (long long)p->k);
  if (p->b_rows != 1 && p->b_rows != kBlock) return fail(SSM_ERR_UNSUPPORTED, "b_rows must be 1 or %d", kBlock);
  if (p->out_dtype != SSM_F32 && p->out_dtype != SSM_BF16) return fail(SSM_ERR_DTYPE, "unknown out_dtype %d", p->out_dtype);
  const int64_t blocks = blocks_of(p->k);
  const struct { int64_t stride, row, most; } rows[] = {{p->a_stride, p->k, 1 << 23}, {p->b_stride, p->k, 1 << 23},
                                                        {p->a_scale_stride, blocks, 1 << 20}, {p->b_scale_stride, blocks, 1 << 20},
                                                        {p->out_stride, p->n, int64_t(1) << 40}};
  if (p->k >= (1 << 23)) return fail(SSM_ERR_SHAPE, "k must be below 2^23");
  for (const auto& r : rows)
    if (r.stride != 0 && (r.stride < r.row || r.stride >= r.most))
      return fail(SSM_ERR_SHAPE, "a row stride of %lld: at least a row of %lld, below %lld", (long long)r.stride,
                  (long long)r.row, (long long)r.most);
  // (the numbers of tiles are 32-bit; the workgroups that share a tile's k have 16 columns at least)
  if (((p->m + 127) / 128) * ((p->n + 127) / 128) >= (int64_t(1) << 30) || !fits_launch((p->n + 15) / 16, 512))
    return fail(SSM_ERR_SHAPE, "a product of %lld x %lld does not fit a launch", (long long)p->m, (long long)p->n);
  return SSM_OK;
}

template <int TM, int WM, int WN, int BROWS, bool WIDE, bool HALVES, typename TO>
void launch_tile(MatmulArgs g, int64_t items, int slots, hipStream_t st) {
  const int last = static_cast<int>(items % slots);
  g.halved = HALVES && items > slots && last * 2 <= slots ? last : 0;
  g.whole = static_cast<int>(items) - g.halved;
  hipLaunchKernelGGL((matmul_tile_kernel<TM, WM, WN, BROWS, WIDE, HALVES, TO>), dim3(static_cast<uint32_t>(items < slots ? items : slots)),
                     dim3(64 * WM * WN), 0, st, g);
}

template <int MT, int NT, int W, bool WIDE, typename TO>
void launch_few(MatmulArgs g, int brows, hipStream_t st) {
  g.tiles_m = (g.m + 16 * MT - 1) / (16 * MT);
  const dim3 grid(g.tiles_m * ((g.n + 16 * NT - 1) / (16 * NT))), block(64 * W);
  if (brows == 1) hipLaunchKernelGGL((matmul_few_kernel<MT, NT, W, 1, WIDE, TO>), grid, block, 0, st, g);
  else hipLaunchKernelGGL((matmul_few_kernel<MT, NT, W, kBlock, WIDE, TO>), grid, block, 0, st, g);
}

template <int MT, bool WIDE, typename TO>
void launch_few_width(const MatmulArgs& g, int nt, int brows, hipStream_t st) {
  if (nt == 1) launch_few<MT, 1, 8, WIDE, TO>(g, brows, st);
  else if (nt == 2) launch_few<MT, 2, 8, WIDE, TO>(g, brows, st);
  else if (nt == 3) launch_few<MT, 3, 8, WIDE, TO>(g, brows, st);
  else if (nt == 4) launch_few<MT, 4, 8, WIDE, TO>(g, brows, st);
  else if constexpr (!WIDE || MT < 4) launch_few<MT, 6, 8, WIDE, TO>(g, brows, st);
}

template <bool WIDE, typename TO>
void launch_few_rows(const MatmulArgs& g, int nt, int brows, hipStream_t st) {
  const int mt = few_rows(g.m);
  if (mt == 1) launch_few_width<1, WIDE, TO>(g, nt, brows, st);
  else if (mt == 2) launch_few_width<2, WIDE, TO>(g, nt, brows, st);
  else launch_few_width<4, WIDE, TO>(g, nt, brows, st);
}

template <int TM, int WM, int WN>
void launch_own(const MatmulArgs& g, int brows, hipStream_t st) {
  const dim3 grid(g.tiles_m * g.tiles_n), block(64 * WM * WN);
  if (brows == 1) hipLaunchKernelGGL((matmul_own_kernel<TM, WM, WN, 1>), grid, block, 0, st, g);
  else hipLaunchKernelGGL((matmul_own_kernel<TM, WM, WN, kBlock>), grid, block, 0, st, g);
}

template <bool WIDE, typename TO>
void launch_tiles(const MatmulArgs& g, const MatmulPlan& t, int brows, int64_t items, hipStream_t st) {
  if (brows == 1) {
    launch_tile<2, 2, 2, 1, WIDE, false, TO>(g, items, t.slots, st);
  } else if (t.bm == 128) {
    launch_tile<2, 2, 2, kBlock, WIDE, false, TO>(g, items, t.slots, st);
  } else if constexpr (!WIDE) {
    if (t.bm == 192) launch_tile<3, 2, 4, kBlock, false, false, TO>(g, items, t.slots, st);
    else launch_tile<4, 2, 4, kBlock, false, true, TO>(g, items, t.slots, st);
  }
}

}  // namespace
}  // namespace ssm57

using namespace ssm57;

extern "C" ssm_status ssm_matmul_fp8(const ssm_matmul_fp8_params* p, const void* a, const float* a_scale, const void* b,
                                     const float* b_scale, void* out, void* stream) {
  g_err[0] = 0;
  if (ssm_status s = check_matmul(p); s != SSM_OK) return s;
  if (!a || !a_scale || !b || !b_scale || !out) return fail(SSM_ERR_NULL, "a, a_scale, b, b_scale and out are required");
  if (!aligned(a_scale, 4) || !aligned(b_scale, 4) || !aligned(out, p->out_dtype == SSM_BF16 ? 2 : 4))
    return fail(SSM_ERR_ALIGN, "a pointer is not aligned to its element size");
  if (!aligned(a, 16) || !aligned(b, 16) || p->a_stride % 16 || p->b_stride % 16)
    return fail(SSM_ERR_ALIGN, "rows of a and b must be 16-byte aligned");
  const MatmulPlan t = plan_of(p);
  MatmulArgs g{};
  g.a = static_cast<const uint8_t*>(a);
  g.b = static_cast<const uint8_t*>(b);
  g.sa = a_scale;
  g.sb = b_scale;
  g.out = out;
  g.m = static_cast<int>(p->m);
  g.n = static_cast<int>(p->n);
  g.k = static_cast<int>(p->k);
  g.blocks = static_cast<int>(blocks_of(p->k));
  g.as = p->a_stride ? p->a_stride : p->k;
  g.bs = p->b_stride ? p->b_stride : p->k;
  g.os = p->out_stride ? p->out_stride : p->n;
  g.sas = p->a_scale_stride ? p->a_scale_stride : g.blocks;
  g.sbs = p->b_scale_stride ? p->b_scale_stride : g.blocks;
  hipStream_t st = static_cast<hipStream_t>(stream);
  if (t.few) {
    if (p->out_dtype == SSM_F32) launch_few_rows<true, float>(g, t.few, p->b_rows, st);
    else launch_few_rows<false, uint16_t>(g, t.few, p->b_rows, st);
  } else {
    g.tiles_m = (g.m + t.bm - 1) / t.bm;
    g.tiles_n = (g.n + t.bn - 1) / t.bn;
    const int64_t tiles = int64_t(g.tiles_m) * g.tiles_n;
    if (t.slots == 0 && t.bm == 256) launch_own<2, 4, 3>(g, p->b_rows, st);
    else if (t.slots == 0 && t.bn == 64) launch_own<1, 4, 2>(g, p->b_rows, st);
    else if (t.slots == 0 && t.bn == 96) launch_own<1, 4, 3>(g, p->b_rows, st);
    else if (t.slots == 0) launch_own<2, 2, 4>(g, p->b_rows, st);
    else if (p->out_dtype == SSM_F32) launch_tiles<true, float>(g, t, p->b_rows, tiles, st);
    else launch_tiles<false, uint16_t>(g, t, p->b_rows, tiles, st);
  }
  const hipError_t e = hipGetLastError();
  return e == hipSuccess ? SSM_OK : fail(SSM_ERR_HIP, "matmul launch: %s", hipGetErrorString(e));
}
