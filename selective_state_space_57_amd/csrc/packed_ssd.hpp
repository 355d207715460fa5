// Device helpers of the SSD kernels over packed sequences (ssm_packed_ssd.hip, ssm_packed_ssd_bwd.hip): matrix-core
// operands, the chunk copies into LDS, per-step scalars, and the segments that sequences are cut into.
//
// v_mfma_f32_16x16x32_bf16: lane l holds A[l%16][8(l/16)+q] and B[8(l/16)+q][l%16], q = 0..7, and the result
// D[4(l/16)+c][l%16] in register c.  Which rows, columns or k a lane's index stands for is free as long as the operands
// agree, so accumulator tiles become operands without moving data between lanes, and two 16-row tiles 2i, 2i + 1 are
// numbered 32 i + 8 (r / 4) + 4 (tile & 1) + r % 4: a lane's four values of each then stand for eight consecutive
// rows, which is one 16-byte access to memory or LDS.
#pragma once

#include "packed.hpp"

namespace ssm57 {

typedef __bf16 pb8 __attribute__((ext_vector_type(8)));
typedef short pv4s __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) pv4s lds_pv4s;
typedef __attribute__((address_space(3))) void lds_pvoid;

constexpr int kChunk = 64;   // steps per chunk
constexpr int kHead = 64;    // head width

__device__ __forceinline__ pf4 mma(pu4 a, pu4 b, pf4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(pb8, a), __builtin_bit_cast(pb8, b), c, 0, 0, 0);
}
__device__ __forceinline__ pu2 bf16x4(float a, float b, float c, float d) { return pu2{pack_bf16(a, b), pack_bf16(c, d)}; }
__device__ __forceinline__ pu4 join(pu2 a, pu2 b) { return pu4{a[0], a[1], b[0], b[1]}; }
// Eight values in three bf16 parts, each the rounded rest behind the ones before it: 24 significant bits, all of an fp32
// value (a third part costs half as much again in products, and keeps states and what hangs on them at fp32 quality: with
// two, dA and the step sizes' gradients were 1.4e-6 to 3e-6 off, ten times an fp32 computation).
struct Parts {
  pu4 p[3];
};
// what four packed values leave of the ones they were rounded from
__device__ __forceinline__ pf4 rest_of(pf4 a, pu2 u) {
  return pf4{a[0] - lo_f32(u[0]), a[1] - hi_f32(u[0]), a[2] - lo_f32(u[1]), a[3] - hi_f32(u[1])};
}
// Four values in two bf16 parts (2^-16 of the value is left out at most).
__device__ __forceinline__ void split2(pf4 a, pu2& hi, pu2& lo) {
  hi = bf16x4(a[0], a[1], a[2], a[3]);
  const pf4 r = rest_of(a, hi);
  lo = bf16x4(r[0], r[1], r[2], r[3]);
}
__device__ __forceinline__ Parts split3(pf4 a, pf4 b) {
  Parts o;
#pragma unroll
  for (int i = 0; i < 3; ++i) {
    const pu2 u = bf16x4(a[0], a[1], a[2], a[3]), v = bf16x4(b[0], b[1], b[2], b[3]);
    o.p[i] = join(u, v);
    if (i < 2) {
      a = rest_of(a, u);
      b = rest_of(b, v);
    }
  }
  return o;
}
__device__ __forceinline__ pf4 unpack4(uint32_t a, uint32_t b) { return pf4{lo_f32(a), hi_f32(a), lo_f32(b), hi_f32(b)}; }

// Packed bf16 pairs: the larger magnitude's bits of each half, and whether either half of the magnitudes is not finite.
typedef unsigned short pus2 __attribute__((ext_vector_type(2)));
__device__ __forceinline__ uint32_t larger_bits(uint32_t most, uint32_t pair) {
  return __builtin_bit_cast(uint32_t, __builtin_elementwise_max(__builtin_bit_cast(pus2, most),
                                                                __builtin_bit_cast(pus2, pair & 0x7fff7fffu)));
}
__device__ __forceinline__ bool not_finite(uint32_t most) { return most >= 0x7f800000u || (most & 0xffffu) >= 0x7f80u; }

// Rows of a chunk in LDS: U 16-byte units each, unit u of row r at u ^ swz(r).  16-byte reads go 8 lanes at a time over
// 128 bytes of banks: 8 consecutive rows of one unit need 8 different places (the low three bits).  Transposing reads
// go 32 lanes over 256 bytes: 8 consecutive rows x 4 consecutive units, one 8-byte half of each, spread over all 16
// places by bit 3.
template <int U>
__device__ __forceinline__ int swz_unit(int r, int u) {
  return u ^ (((r & 7) | ((r & 2) << 2)) & (U - 1));
}
// byte address of unit u of row r
template <int U>
__device__ __forceinline__ int unit_at(int r, int u) {
  return (r * U + swz_unit<U>(r, u)) * 16;
}
__device__ __forceinline__ pu4 lds_u4(const void* base, int byte) {
  return *reinterpret_cast<const pu4*>(static_cast<const char*>(base) + byte);
}
// ds_read_b64_tr_b16: within each 16 lanes, lane i receives element i%4 of the 8-byte pieces that lanes 4q + i/4
// (q = 0..3) point at.  Lane j points at row k0 + j/4, columns 4(j%4).. of tile `tile` (16 columns, numbered as above):
// lane i receives column i of the tile at rows k0 .. k0+3.
template <int U>
__device__ __forceinline__ pu2 lds_tr(const void* base, int k0, int tile, int l16) {
  const int byte = unit_at<U>(k0 + (l16 >> 2), 4 * (tile >> 1) + (l16 & 3)) + 8 * (tile & 1);
  return __builtin_bit_cast(pu2, __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                                     (lds_pv4s*)(static_cast<const char*>(base) + byte)));
}
// operand over 32 rows (the k index) of a tile's 16 columns; the lane's k: rows 32 kk + 4 g4 + c and 16 more
template <int U>
__device__ __forceinline__ pu4 lds_tr_operand(const void* base, int kk, int tile, int l16, int g4) {
  return join(lds_tr<U>(base, 32 * kk + 4 * g4, tile, l16), lds_tr<U>(base, 32 * kk + 16 + 4 * g4, tile, l16));
}
// the same with the lane's k as in lds_row_operand: rows 32 kk + 8 g4 .. + 7
template <int U>
__device__ __forceinline__ pu4 lds_tr_operand8(const void* base, int kk, int tile, int l16, int g4) {
  return join(lds_tr<U>(base, 32 * kk + 8 * g4, tile, l16), lds_tr<U>(base, 32 * kk + 8 * g4 + 4, tile, l16));
}
// a tile whose 16 columns are numbered plainly (16 tile + column)
template <int U>
__device__ __forceinline__ pu2 lds_tr_plain(const void* base, int k0, int tile, int l16) {
  const int byte = unit_at<U>(k0 + (l16 >> 2), 2 * tile + ((l16 & 3) >> 1)) + 8 * (l16 & 1);
  return __builtin_bit_cast(pu2, __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                                     (lds_pv4s*)(static_cast<const char*>(base) + byte)));
}
// operand of a plainly numbered tile; EIGHT: the lane's k as in lds_row_operand, else as in lds_tr_operand
template <int U, bool EIGHT>
__device__ __forceinline__ pu4 lds_tr_plain_operand(const void* base, int kk, int tile, int l16, int g4) {
  return join(lds_tr_plain<U>(base, 32 * kk + (EIGHT ? 8 : 4) * g4, tile, l16),
              lds_tr_plain<U>(base, 32 * kk + (EIGHT ? 8 * g4 + 4 : 4 * g4 + 16), tile, l16));
}
// operand whose row (or column) index is a row of LDS and whose k are 32 consecutive columns from 32 kk
template <int U>
__device__ __forceinline__ pu4 lds_row_operand(const void* base, int row, int kk, int g4) {
  return lds_u4(base, unit_at<U>(row, 4 * kk + g4));
}

// A chunk's rows of one tensor: a buffer range that starts at the chunk's first row and ends with its last valid one,
// so that rows behind it read as zeros and are not written.  The base is 64-bit; only offsets inside a chunk are 32-bit.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t chunk_rsrc(const uint16_t* base, int64_t row, int64_t stride, int rows,
                                                             int width) {
  return make_rsrc(base + row * stride, rows > 0 ? int64_t(rows - 1) * stride + width : 0);
}

// Copy of a chunk's 64 rows x U units into LDS by NW waves.
template <int U, int NW>
__device__ __forceinline__ void copy_rows(void* dst, __amdgpu_buffer_rsrc_t rsrc, int wave, int lane,
                                          uint32_t row_bytes) {
  constexpr int kInstr = (kChunk * U + 64 * NW - 1) / (64 * NW);
  constexpr int kStep = 64 * NW / U;   // rows between a lane's copies
  static_assert(kStep % 8 == 0, "a lane's copies share their place in the row");
  if (kChunk * U < 64 * NW && wave >= kChunk * U / 64) return;   // (more waves than pieces)
  const int place = 64 * wave + lane;
  const int r = place / U;
  const uint32_t base = static_cast<uint32_t>(r) * row_bytes + 16u * static_cast<uint32_t>(swz_unit<U>(r, place % U));
#pragma unroll
  for (int i = 0; i < kInstr; ++i)
    __builtin_amdgcn_raw_ptr_buffer_load_lds(
        rsrc, (lds_pvoid*)(static_cast<char*>(dst) + 1024 * (wave + NW * i)), 16,
        static_cast<int>(base + static_cast<uint32_t>(i * kStep) * row_bytes), 0, 0, 0);
}

__device__ __forceinline__ void wait_memory() { __builtin_amdgcn_s_waitcnt(0x0F70); }   // vmcnt(0)
// Keeps the parts of a chunk apart for the compiler: operands read from LDS for one are not kept in registers for the
// next (they are read again), nor read ahead of it, so that the parts' registers do not add up.
__device__ __forceinline__ void part_ends() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_sched_barrier(0);
}
// The same value, unknown to the compiler: what is computed from it is computed here, and not kept in registers over
// the loop around.
__device__ __forceinline__ int afresh(int v) {
  asm volatile("" : "+v"(v));
  return v;
}
// Waits for this wave's LDS operations: what it read is in registers before anything that follows is issued.
__device__ __forceinline__ void wait_lds() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_waitcnt(0xC07F);   // lgkmcnt(0)
  asm volatile("" ::: "memory");
}
// Barrier for LDS written by ds_write: waits for this wave's LDS operations only.  (The empty asm keeps the compiler
// from moving memory accesses across it.)
__device__ __forceinline__ void barrier_lds() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_waitcnt(0xC07F);   // lgkmcnt(0)
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

template <int K>
__device__ __forceinline__ float lanes_shr(float v) {   // lane i of a 16-lane row reads lane i - K, 0 before the row
  return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), 0x110 + K, 0xf, 0xf,
                                                               false));
}
template <int K>
__device__ __forceinline__ float lanes_shl(float v) {   // lane i + K, 0 behind the row
  return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), 0x100 + K, 0xf, 0xf,
                                                               false));
}
__device__ __forceinline__ float lane_value(float v, int lane) {
  return __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, v), lane));
}
// sums over the wave's four rows of 16 lanes (lanes that differ in their row), and over all 64 lanes, in every lane
__device__ __forceinline__ float sum_rows(float v) {
  const uint32_t u = __float_as_uint(v);
  const auto a = __builtin_amdgcn_permlane16_swap(u, u, false, false);   // rows (0, 0, 2, 2) and (1, 1, 3, 3)
  const uint32_t a0 = a[0], a1 = a[1];
  const float w = __uint_as_float(a0) + __uint_as_float(a1);
  const uint32_t x = __float_as_uint(w);
  const auto b = __builtin_amdgcn_permlane32_swap(x, x, false, false);   // halves (0, 0) and (1, 1)
  const uint32_t b0 = b[0], b1 = b[1];
  return __uint_as_float(b0) + __uint_as_float(b1);
}
__device__ __forceinline__ float sum_row(float v) {   // over the 16 lanes of a row
  v += row_ror<8>(v);
  v += row_ror<4>(v);
  v += row_ror<2>(v);
  return v + row_ror<1>(v);
}
__device__ __forceinline__ float sum_wave(float v) { return sum_rows(sum_row(v)); }

// sums over the lanes of the 16-lane row up to this one, or from it on
__device__ __forceinline__ float row_prefix(float v) {
  v += lanes_shr<1>(v);
  v += lanes_shr<2>(v);
  v += lanes_shr<4>(v);
  return v + lanes_shr<8>(v);
}
__device__ __forceinline__ float row_suffix(float v) {
  v += lanes_shl<1>(v);
  v += lanes_shl<2>(v);
  v += lanes_shl<4>(v);
  return v + lanes_shl<8>(v);
}
// the same for the row, and the sum over the rows before it
__device__ __forceinline__ void row_prefix(float v, int lane, float& in_row, float& before) {
  in_row = row_prefix(v);
  const float r0 = lane_value(in_row, 15), r1 = lane_value(in_row, 31), r2 = lane_value(in_row, 47);
  const int row = lane >> 4;
  before = (row >= 1 ? r0 : 0.0f) + (row >= 2 ? r1 : 0.0f) + (row >= 3 ? r2 : 0.0f);
}
// sum over lanes 0..lane
__device__ __forceinline__ float wave_prefix(float v, int lane) {
  float in_row, before;
  row_prefix(v, lane, in_row, before);
  return in_row + before;
}
// sum over lanes lane..63
__device__ __forceinline__ float wave_suffix(float v, int lane) {
  v = row_suffix(v);
  const float r1 = lane_value(v, 16), r2 = lane_value(v, 32), r3 = lane_value(v, 48);
  const int row = lane >> 4;
  return v + (row <= 2 ? r3 : 0.0f) + (row <= 1 ? r2 : 0.0f) + (row <= 0 ? r1 : 0.0f);
}

// A double moved across lanes by two 32-bit DPP moves (0 where the source or the row mask gives none).
template <int CTRL, int ROWS>
__device__ __forceinline__ double lanes_move(double v) {
  const uint64_t u = __builtin_bit_cast(uint64_t, v);
  const int lo = __builtin_amdgcn_update_dpp(0, static_cast<int>(u), CTRL, ROWS, 0xf, false);
  const int hi = __builtin_amdgcn_update_dpp(0, static_cast<int>(u >> 32), CTRL, ROWS, 0xf, false);
  return __builtin_bit_cast(double, static_cast<uint64_t>(static_cast<uint32_t>(hi)) << 32 | static_cast<uint32_t>(lo));
}
// Running sum over lanes 0..lane of the decays' logarithms, and the sum over all, in 64 bits: what is left between two steps
// is a difference of two of these, which a few steps that decay (nearly) everything make large.  In fp32 one such step
// of 2^12 would cost the decays between all steps behind it 2^-12.
struct DecaySum {
  double upto, all;
  __device__ __forceinline__ float behind() const { return static_cast<float>(all - upto); }   // sum over the lanes behind
};
__device__ __forceinline__ DecaySum sum_decays(float la) {
  double d = la;
  d += lanes_move<0x111, 0xf>(d);   // row_shr: 1, 2, 4, 8
  d += lanes_move<0x112, 0xf>(d);
  d += lanes_move<0x114, 0xf>(d);
  d += lanes_move<0x118, 0xf>(d);
  d += lanes_move<0x142, 0xa>(d);   // row_bcast: lane 15 into the second and fourth row, then lane 31 into the last two
  d += lanes_move<0x143, 0xc>(d);
  const uint64_t u = __builtin_bit_cast(uint64_t, d);
  const uint32_t lo = __builtin_amdgcn_readlane(static_cast<int>(u), 63);
  const uint32_t hi = __builtin_amdgcn_readlane(static_cast<int>(u >> 32), 63);
  return DecaySum{d, __builtin_bit_cast(double, static_cast<uint64_t>(hi) << 32 | lo)};
}

// Pieces: sequence s is cut every `steps` tokens (segments of a walk, or chunk groups of the backward).  Piece i of a
// sequence that begins at token b has the number s + b / steps + i: that is unique, needs no sum over the sequences
// before it, and stays below nseqs + ntokens / steps + 1 (some numbers belong to no piece).
struct Piece {
  int seq, begin, end;   // sequence and its tokens
  int index, count;      // piece within the sequence, and how many it has (an empty sequence has one)
  int first;             // number of the sequence's first piece
  int place;             // of its first piece among those of sequences that have several
};
__host__ __device__ constexpr int64_t piece_numbers(int64_t nseqs, int64_t ntokens, int64_t steps) {
  return nseqs + ntokens / steps + 1;
}
// What only sequences of several pieces need is kept at place 2 (b / steps) + i: a sequence longer than `steps` has at most
// twice as many pieces as it has whole ones, so these stay apart, and below 2 (ntokens / steps) however many sequences.
__host__ __device__ constexpr int64_t piece_places(int64_t ntokens, int64_t steps) { return 2 * (ntokens / steps); }
__device__ __forceinline__ void pieces_of(const int32_t* cu, int s, int ntokens, int steps, Piece& p) {
  seq_range(cu, s, ntokens, p.begin, p.end);
  p.seq = s;
  p.first = s + p.begin / steps;
  p.place = 2 * (p.begin / steps);
  p.count = max((p.end - p.begin + steps - 1) / steps, 1);
}
// The piece of that number; false where there is none.
__device__ __forceinline__ bool find_piece(const int32_t* cu, int nseqs, int ntokens, int steps, int number, Piece& p) {
  int lo = 0, hi = nseqs;   // the last sequence whose first piece has at most this number
  while (hi - lo > 1) {
    const int mid = lo + (hi - lo) / 2;
    if (mid + min(max(cu[mid], 0), ntokens) / steps <= number) lo = mid; else hi = mid;
  }
  pieces_of(cu, lo, ntokens, steps, p);
  p.index = number - p.first;
  return p.index >= 0 && p.index < p.count;
}

// exp(-|u|), good to about 2^-23: the rounding of the exponent's product with log2(e), which the exponential would
// magnify by |u|, is put back (a step's errors are the same for every column of a head, so they do not average out in
// dA and the step sizes' gradients).  It is 0 from 128 on, infinite u among them (whose rest would be no number; NaN stays).
__device__ __forceinline__ float exp_neg_abs(float u) {
  constexpr float kLog2eLo = 1.925963033500e-8f;   // log2(e) - float(log2(e))
  const float x = fabsf(u) > 128.0f ? -128.0f : -fabsf(u);
  const float p = x * kLog2e;
  const float rest = fmaf(x, kLog2e, -p) + x * kLog2eLo;
  const float v = hw_exp2(p);
  return fmaf(v * kLn2, rest, v);
}
// log(1 + v), 0 <= v <= 1: 2 atanh(s), s = v / (2 + v) <= 1/3, by its series (the first term left out is 3e-9 of it)
__device__ __forceinline__ float log1p_series(float v) {
  const float s = v / (2.0f + v), q = s * s;
  float p = 1.0f / 15.0f;
  p = fmaf(p, q, 1.0f / 13.0f);
  p = fmaf(p, q, 1.0f / 11.0f);
  p = fmaf(p, q, 1.0f / 9.0f);
  p = fmaf(p, q, 1.0f / 7.0f);
  p = fmaf(p, q, 0.2f);
  p = fmaf(p, q, 1.0f / 3.0f);
  return 2.0f * fmaf(s * q, p, s);
}
__device__ __forceinline__ float softplus_fine(float u) { return fmaxf(u, 0.0f) + log1p_series(exp_neg_abs(u)); }
// its derivative 1 / (1 + exp(-u))
__device__ __forceinline__ float softplus_slope(float u) {
  const float v = exp_neg_abs(u);
  return (u >= 0.0f ? 1.0f : v) / (1.0f + v);
}

// Logarithm (base 2) of a step's decay.  Held within 2^14, far behind where its exponential is 0 (or infinite): sums of it
// stay finite, and so do their differences.  (A NaN stays one.)
__device__ __forceinline__ float decay_log(float delta, float A) {
  constexpr float kMost = 16384.0f;
  float la = delta * A * kLog2e;
  la = la < -kMost ? -kMost : la;
  return la > kMost ? kMost : la;
}

// Step size, its weight and the decay's logarithm (base 2) of one step; zeros behind the sequence.
__device__ __forceinline__ void step_scalars(float dt, float bias, float A, bool use_softplus, bool zoh, bool live,
                                             float& delta, float& phi, float& la) {
  const float u = dt + bias;
  delta = use_softplus ? softplus_fine(u) : u;
  delta = live ? delta : 0.0f;
  la = decay_log(delta, A);
  phi = delta;
  if (zoh && A != 0.0f) {
    const float e = delta * A;
    phi = expm1_from(e, hw_exp2(e * kLog2e)) / A;
  }
}

// Workgroups are dealt to the 8 XCDs in turn: give each XCD a run of consecutive items (the grid is a multiple of 8).
__device__ __forceinline__ int xcd_item() {
  const int per = static_cast<int>(gridDim.x) / 8;
  return (static_cast<int>(blockIdx.x) % 8) * per + static_cast<int>(blockIdx.x) / 8;
}

// ---------------------------------------------------------------------------------------------------------------
// host side

ssm_status check_packed_ssd(const ssm_ssd_packed_params* p, bool step);

// A workgroup that walks a segment: 8 waves, each with the state of half of a head (32 columns: N / 2 registers a lane).
// For N <= 128 two workgroups share a CU and cover each other's waits.
constexpr int kWalkWaves = 8, kWalkHeads = 4;

struct PackedPlan {
  int hblocks;    // workgroups per group of heads
  int cps;        // chunks per segment
  int64_t nseg;   // numbers of segments
  int64_t places; // for the states that enter segments
  bool split;     // whether a sequence can have more than one
};
PackedPlan packed_plan(const ssm_ssd_packed_params* p);

// Byte of a lane's four values of a saved state: S[p][n] for n = 16 nt + lane % 16, p = 32 (i / 2) + 8 (lane / 16) +
// 4 (i % 2) + 0..3, so that tiles 2j and 2j + 1 are an operand over 32 p, and a wave's access one run of 1 KB (against rows
// of 64 p, 16 bytes of every 32 at a time: walks of 16384 tokens, 2.7B layer, 379 instead of 483 us).
__host__ __device__ constexpr int state_operand(int nt, int i, int lane) { return ((nt * 4 + i) * 64 + lane) * 16; }

// A walk over the states of packed sequences, chunk by chunk and from each sequence's first state (ssm_packed_states.hip):
// forward, S <- exp(c_63) S + sum_s (phi_s exp(c_63 - c_s) v_s) k_s^T with v = x, k = B, or in reverse order,
// G <- exp(c_63) G + sum_t exp(c_t) v_t k_t^T with v = dy, k = C.
struct StatesArgs {
  const uint16_t* v;
  const uint16_t* k;
  const uint16_t* dt;
  const float* dt_bias;
  const float* A;
  const int32_t* cu;
  const float* init;     // [slots][H][64][N], or by sequence where idx and has are null
  const int32_t* idx;
  const uint8_t* has;
  float* last;           // [seqs][H][64][N] or null: the state behind the whole walk of a sequence
  float* ws_state;       // [places][H][64][N]: state entering each segment (where a sequence has more than one)
  float* ws_decay;       // [places][H]
  float* save;           // [chunk numbers][H][64 N] or null (no walk behind the join): state entering each chunk
  int64_t vs, ks, dts, nslots;
  int T, S, H, G, hpg, hblocks, cps, nseg;
  int softplus, zoh;
};
// Brings ws_state up to date where a sequence can have several segments (split), and then, with save, walks all: f in
// order, and beside it r, over the same segments, in reverse order (or null).
ssm_status launch_states(const StatesArgs& f, const StatesArgs* r, int dstate, bool split, hipStream_t st);

inline size_t up256(size_t v) { return (v + 255) / 256 * 256; }

}  // namespace ssm57
