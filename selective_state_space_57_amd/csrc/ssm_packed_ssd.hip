// The Mamba-2 SSD layer over packed sequences on gfx950: prompts (chunked matrix form on the bf16 matrix cores) and
// single tokens, with the recurrent state of each sequence in a slot of a pool.
//
//   Delta_t = softplus(dt + bias);  a_t = exp(Delta_t A);  phi_t = Delta_t or expm1(Delta_t A) / A
//   S_t[p][n] = a_t S_{t-1}[p][n] + phi_t x_t[p] B_t[n];   y_t[p] = sum_n S_t[p][n] C_t[n] + D x_t[p]
// In chunks of 64 steps, with c_t the running sum of Delta A inside a chunk and S the state entering it:
//   y_t = exp(c_t) S C_t + sum_{s<=t} M[t][s] x_s + D x_t,   M[t][s] = (C_t . B_s) exp(c_t - c_s) phi_s
//   S  <- exp(c_63) S + sum_s (phi_s exp(c_63 - c_s) x_s) B_s^T
//
// A workgroup takes 4 heads of one group over one segment of a sequence and walks its chunks.  A wave holds the state of
// half of a head in registers (32 columns, which do not meet the other half's): so four waves share a SIMD, of two
// workgroups, and cover each other's waits.  What heads share is done once: B and C are copied to LDS for all of them,
// and the 10 lower tiles of C B^T are shared out over the waves.  Everything else belongs to one wave.
// Sequences longer than a segment: a walk over the states alone (ssm_packed_states.hip) finds the state entering every
// segment first, and all segments run at once.
//
// Precision: fp32 state and accumulation; x, B and C enter the matrix cores as they are.  The weighted x of the state
// update is split into three bf16 parts, so the state keeps fp32 quality over long sequences (two parts, 2^-17, are 11 %
// faster when tried).  M (but for s = t, which is added in fp32) and the state that meets C only reach y: they are split into two,
// which leave out 2^-16 of them at most, so that y is the 64-bit value rounded once but for 5e-5 of it in the 2-norm
// (rounded to bf16 once each, they added 1.4e-3 to the rounding's own 1.66e-3; on 16384 tokens of the 2.7B layer the
// second part of M takes 24 us, that of the state 36).
//
// Measured on 16384 tokens of 80 heads, N = 128 (0.40 GB in and out, 43 GFLOP): 340 us a call.  Under the profiler, where
// every kernel is somewhat longer, this pass takes 272, the walk 89 and its join 23.  VALU 53 % of the cycles, MFMA 22 %,
// the rest waits.  The kernel of N = 128 is over its 128 registers by 6 (28 bytes a lane in scratch memory).  The step
// kernel: 256 tokens of the same layer 250 us, 5.4 TB/s of states.
#include "packed_ssd.hpp"

namespace ssm57 {
namespace {

struct PSsdArgs {
  const uint16_t* x;
  const uint16_t* dt;
  const uint16_t* B;
  const uint16_t* C;
  const float* dt_bias;
  const float* A;
  const float* Dskip;
  const int32_t* cu;
  const float* state;
  const int32_t* idx;
  const uint8_t* has;
  float* state_out;
  uint16_t* y;
  const float* ws_state;   // [places][H][64][N]: the state entering each, where a sequence has several
  int64_t xs, dts, bs, cs, ys, nslots;
  int T, S, H, G, hpg, hblocks;   // hblocks: workgroups per group
  int cps, nwork;
  int softplus, zoh;
};

// scalars of one chunk, per wave
struct alignas(16) HeadScalars {
  // c_t (base 2), rounded to fp32: differences of these are good to their own rounding, and the rests r_t that the
  // rounding left go into factors, exp(c_t - c_s) = exp2(c[t] - c[s]) exp2(r_t) exp2(-r_s)
  float c[kChunk];
  float rest[kChunk];  // exp2(r_t)
  float phi[kChunk];   // phi_s exp2(-r_s)
  float w[kChunk];     // phi_s exp(c_63 - c_s)
  float own[kChunk];   // M[t][t] exp2(-r_t)
};

template <int N>
__global__ void __launch_bounds__(kWalkWaves * 64) __attribute__((amdgpu_waves_per_eu(N == 256 ? 2 : 4, N == 256 ? 2 : 4)))
packed_ssd_fwd_kernel(PSsdArgs a) {
  constexpr int NW = kWalkWaves;
  constexpr int PT = 2;        // 16-column tiles of a wave
  constexpr int kParts = 2;    // waves of a head
  constexpr int UX = 2 * PT;             // 16-byte units of its columns
  constexpr int U = N / 8;
  constexpr int NT = N / 16;   // 16-row tiles of the state
  constexpr int NK = N / 32;
  // (B and C once: two workgroups of 80 KB fit a CU, and the copy of the one runs beside the products of the other)
  __shared__ alignas(16) uint16_t B[kChunk * N], C[kChunk * N];
  __shared__ alignas(16) uint16_t sX[NW][kChunk * 16 * PT];
  __shared__ pf4 sCB[10][64];   // tiles of C B^T on and below the diagonal
  __shared__ HeadScalars sS[NW / kParts];   // (the waves of a head write the same values)
  __shared__ alignas(8) uint8_t sSpoilt[NW][16 * PT];   // per column, the chunk's first step whose x is not finite

  // (in launch order, heads fastest: the heads of a segment go round the XCDs, so that segments of any length, and numbers
  // without one, spread evenly; runs of items per XCD, which share B and C in its L2, left some with two rounds)
  const int item = blockIdx.x;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int l16 = lane & 15, g4 = lane >> 4;
  const int hb = item % (a.G * a.hblocks);
  Piece seg;
  if (!find_piece(a.cu, a.S, a.T, a.cps * kChunk, item / (a.G * a.hblocks), seg)) return;
  const int g = hb / a.hblocks;
  const int hg = (hb % a.hblocks) * (NW / kParts) + wave / kParts;   // head within the group
  const int p0 = (wave % kParts) * 16 * PT;            // first column of this wave
  const bool on = hg < a.hpg;                          // (a wave without a head computes the last one's, unstored)
  const int h = g * a.hpg + (on ? hg : a.hpg - 1);

  const int t_begin = seg.begin + seg.index * a.cps * kChunk;
  const int t_end = min(seg.end, t_begin + a.cps * kChunk);
  const int nchunks = (t_end - t_begin + kChunk - 1) / kChunk;

  const float Ah = a.A[h];
  const float bias = a.dt_bias ? a.dt_bias[h] : 0.0f;
  const float Dh = a.Dskip ? a.Dskip[h] : 0.0f;
  const uint16_t* xh = a.x + int64_t(h) * kHead + p0;
  const uint16_t* Bg = a.B + int64_t(g) * N;
  const uint16_t* Cg = a.C + int64_t(g) * N;
  const uint32_t xrow = static_cast<uint32_t>(a.xs) * 2u, brow = static_cast<uint32_t>(a.bs) * 2u,
                 crow = static_cast<uint32_t>(a.cs) * 2u, yrow = static_cast<uint32_t>(a.ys) * 2u;

  auto rows_of = [&](int ck) { return min(max(t_end - (t_begin + ck * kChunk), 0), kChunk); };
  auto copy_group = [&](int ck, uint16_t* dst, const uint16_t* src, int64_t stride, uint32_t row_bytes)
                        __attribute__((always_inline)) {
    const int64_t t0 = t_begin + int64_t(ck) * kChunk;
    const int rows = rows_of(ck);
    copy_rows<U, NW>(dst, chunk_rsrc(src, rows ? t0 : 0, stride, rows, N), wave, afresh(lane), row_bytes);
  };
  auto copy_x = [&](int ck) __attribute__((always_inline)) {
    const int64_t t0 = t_begin + int64_t(ck) * kChunk;
    const int rows = rows_of(ck);
    copy_rows<UX, 1>(sX[wave], chunk_rsrc(xh, rows ? t0 : 0, a.xs, rows, 16 * PT), 0, afresh(lane), xrow);
  };
  auto load_dt = [&](int ck) __attribute__((always_inline)) -> uint32_t {
    const int64_t t = t_begin + int64_t(ck) * kChunk + afresh(lane);
    return a.dt[(t < t_end ? t : (t_begin < a.T ? t_begin : 0)) * a.dts + h];
  };

  // state tiles: S[nt][pt][c] = S[p][n], n = 32 (nt/2) + 8 g4 + 4 (nt%2) + c, p = p0 + 32 (pt/2) + 8 (l16/4) + 4 (pt%2) + l16%4
  pf4 S[NT][PT];
  const int64_t head_size = int64_t(kHead) * N;
  const int lane_entry = (p0 + 8 * (l16 >> 2) + (l16 & 3)) * N + 8 * g4;
  auto entry = [&](int nt, int pt) __attribute__((always_inline)) {
    return lane_entry + (32 * (pt >> 1) + 4 * (pt & 1)) * N + 32 * (nt >> 1) + 4 * (nt & 1);
  };
  {
    const float* from = nullptr;
    if (seg.count > 1) {
      from = a.ws_state + (int64_t(seg.place + seg.index) * a.H + h) * head_size;
    } else if (a.state && (!a.has || a.has[seg.seq])) {
      const int64_t slot = slot_of(a.idx, seg.seq, a.nslots);
      if (slot >= 0) from = a.state + (slot * a.H + h) * head_size;
    }
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int pt = 0; pt < PT; ++pt)
        S[nt][pt] = from ? *reinterpret_cast<const pf4*>(from + entry(nt, pt)) : pf4{0.0f, 0.0f, 0.0f, 0.0f};
  }

  HeadScalars& sc = sS[wave / kParts];
  const uint16_t* X = sX[wave];

  uint32_t dtv = load_dt(0);
  copy_x(0);
  for (int ck = 0; ck < nchunks; ++ck) {
    barrier_lds();    // everyone is done with the chunk before
    copy_group(ck, B, Bg, a.bs, brow);
    copy_group(ck, C, Cg, a.cs, crow);
    const int rows = rows_of(ck);
    {
      const int lane = afresh(threadIdx.x) & 63;
      float delta, phi, la;
      step_scalars(lo_f32(dtv), bias, Ah, a.softplus, a.zoh, lane < rows, delta, phi, la);
      const DecaySum sum = sum_decays(la);
      const float c = static_cast<float>(sum.upto), r = static_cast<float>(sum.upto - c);
      sc.c[lane] = c;
      sc.rest[lane] = hw_exp2(r);
      sc.phi[lane] = phi * hw_exp2(-r);
      sc.w[lane] = phi * hw_exp2(sum.behind());
    }
    wait_memory();    // this wave's copies
    barrier_lds();    // and everyone's
    dtv = load_dt(ck + 1);
    // M is 0 for s > t, but 0 times what is not finite is not 0.  Such an x is taken out, and its column of y and of the state
    // is made NaN from its step on: nothing in front of it changes.  (Looking for one takes 10 of 342 us, 16384 tokens of the
    // 2.7B layer.)
    bool spoilt;
    {
      uint32_t most = 0u;
#pragma unroll
      for (int i = 0; i < kChunk * UX / 64; ++i) {
        const pu4 v = lds_u4(X, (64 * i + afresh(lane)) * 16);
#pragma unroll
        for (int j = 0; j < 4; ++j) most = larger_bits(most, v[j]);
      }
      spoilt = __builtin_amdgcn_ballot_w64(not_finite(most)) != 0;
    }
    if (spoilt) {
      const int p = afresh(lane) % (16 * PT);
      int first = kChunk;
      for (int r = kChunk - 1; r >= 0; --r) {
        uint16_t* at = sX[wave] + (unit_at<UX>(r, p >> 3) >> 1) + (p & 7);
        if ((*at & 0x7f80u) == 0x7f80u) {
          first = r;
          *at = 0;
        }
      }
      sSpoilt[wave][p] = static_cast<uint8_t>(first);
      wave_lds_sync();
    }
    {
      // C B^T, tile i = (tb, sb), sb <= tb: rows s, columns t
      for (int i = wave; i < 10; i += NW) {
        const int l = afresh(lane), l16 = l & 15, g4 = l >> 4;
        const int tb = i >= 6 ? 3 : (i >= 3 ? 2 : (i >= 1 ? 1 : 0)), sb = i - tb * (tb + 1) / 2;
        pf4 v = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int kk = 0; kk < NK; ++kk)
          v = mma(lds_row_operand<U>(B, 16 * sb + l16, kk, g4), lds_row_operand<U>(C, 16 * tb + l16, kk, g4), v);
        sCB[i][lane] = v;
      }
      barrier_lds();
      const int64_t t0 = t_begin + int64_t(ck) * kChunk;
      const auto ry = chunk_rsrc(a.y + int64_t(h) * kHead + p0, t0, a.ys, on ? rows : 0, 16 * PT);
      // two tiles of steps (32) at a time: Y^T[p][t = 16 tb + l16], tb = 2 th + i
#pragma unroll
      for (int th = 0; th < 2; ++th) {
        part_ends();
        const int l = afresh(lane), l16 = l & 15, g4 = l >> 4;
        // (the state's bf16 copy is made again for the second half: kept, it would take N / 4 registers)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int pt = 0; pt < PT; ++pt) asm volatile("" : "+v"(S[nt][pt]));
        pf4 acc[2][PT];
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int pt = 0; pt < PT; ++pt) acc[i][pt] = pf4{0.0f, 0.0f, 0.0f, 0.0f};
        // what the entering state gives: S C_t, scaled by exp(c_t)
#pragma unroll
        for (int kn = 0; kn < NK; ++kn) {
          pu4 c[2];
#pragma unroll
          for (int i = 0; i < 2; ++i) c[i] = lds_row_operand<U>(C, 32 * th + 16 * i + l16, kn, g4);
#pragma unroll
          for (int pt = 0; pt < PT; ++pt) {
            pu2 hi[2], lo[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) split2(S[2 * kn + e][pt], hi[e], lo[e]);
#pragma unroll
            for (int i = 0; i < 2; ++i) acc[i][pt] = mma(join(lo[0], lo[1]), c[i], acc[i][pt]);
#pragma unroll
            for (int i = 0; i < 2; ++i) acc[i][pt] = mma(join(hi[0], hi[1]), c[i], acc[i][pt]);
          }
        }
        float ct[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          ct[i] = sc.c[32 * th + 16 * i + l16];
          const float f = hw_exp2(ct[i]);
#pragma unroll
          for (int pt = 0; pt < PT; ++pt) acc[i][pt] *= f;
        }
        // inside the chunk: sum_{s<t} x_s M[t][s], 32 steps s at a time
#pragma unroll
        for (int kk = 0; kk <= th; ++kk) {
          pu4 xt[PT];
#pragma unroll
          for (int pt = 0; pt < PT; ++pt) xt[pt] = lds_tr_operand<UX>(X, kk, pt, l16, g4);
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const int tb = 2 * th + i;
            part_ends();
            pu2 hi[2], lo[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const int sb = 2 * kk + e;
              if (sb > tb) {
                hi[e] = lo[e] = pu2{0u, 0u};
                continue;
              }
              const pf4 cb = sCB[tb * (tb + 1) / 2 + sb][lane];
              const pf4 cs = *reinterpret_cast<const pf4*>(&sc.c[16 * sb + 4 * g4]);
              const pf4 ph = *reinterpret_cast<const pf4*>(&sc.phi[16 * sb + 4 * g4]);
              pf4 m;
#pragma unroll
              for (int c = 0; c < 4; ++c) {
                // (above the diagonal the difference can be large and positive: masked after the fact)
                m[c] = cb[c] * (hw_exp2(ct[i] - cs[c]) * ph[c]);
                if (sb == tb) {
                  // a step's own x goes into its y in fp32, together with D
                  if (4 * g4 + c == l16) sc.own[16 * tb + l16] = m[c];
                  m[c] = 4 * g4 + c < l16 ? m[c] : 0.0f;
                }
              }
              split2(m, hi[e], lo[e]);
            }
#pragma unroll
            for (int pt = 0; pt < PT; ++pt) acc[i][pt] = mma(xt[pt], join(lo[0], lo[1]), acc[i][pt]);
#pragma unroll
            for (int pt = 0; pt < PT; ++pt) acc[i][pt] = mma(xt[pt], join(hi[0], hi[1]), acc[i][pt]);
          }
        }
        wave_lds_sync();
        // a lane's two tiles of columns are eight consecutive ones of its step
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int t = 32 * th + 16 * i + l16;
          const float up = sc.rest[t], own = fmaf(sc.own[t], up, Dh);
          const pu4 xv = lds_u4(X, unit_at<UX>(t, g4));
          const pf4 y0 = acc[i][0] * up, y1 = acc[i][1] * up;
          pu4 o = {pack_bf16(fmaf(own, lo_f32(xv[0]), y0[0]), fmaf(own, hi_f32(xv[0]), y0[1])),
                         pack_bf16(fmaf(own, lo_f32(xv[1]), y0[2]), fmaf(own, hi_f32(xv[1]), y0[3])),
                         pack_bf16(fmaf(own, lo_f32(xv[2]), y1[0]), fmaf(own, hi_f32(xv[2]), y1[1])),
                         pack_bf16(fmaf(own, lo_f32(xv[3]), y1[2]), fmaf(own, hi_f32(xv[3]), y1[3]))};
          if (spoilt) {
            const pu2 first = *reinterpret_cast<const pu2*>(&sSpoilt[wave][8 * g4]);
#pragma unroll
            for (int j = 0; j < 8; ++j)
              if (static_cast<int>((first[j >> 2] >> (8 * (j & 3))) & 0xffu) <= t)
                o[j >> 1] = (j & 1) ? (o[j >> 1] & 0xffffu) | 0x7fc00000u : (o[j >> 1] & 0xffff0000u) | 0x7fc0u;
          }
          __builtin_amdgcn_raw_buffer_store_b128(
              o, ry, static_cast<int>(static_cast<uint32_t>(t) * yrow + 16u * g4), 0, 0);
        }
      }
    }
    part_ends();
    // state update
    const int l = afresh(lane), l16 = l & 15, g4 = l >> 4;
    const float fade = hw_exp2(sc.c[kChunk - 1]) * sc.rest[kChunk - 1];
#pragma unroll
    for (int kk = 0; kk < 2; ++kk) {
      const pf4 w0 = *reinterpret_cast<const pf4*>(&sc.w[32 * kk + 4 * g4]);
      const pf4 w1 = *reinterpret_cast<const pf4*>(&sc.w[32 * kk + 16 + 4 * g4]);
      Parts w[PT];   // the weighted rows
#pragma unroll
      for (int pt = 0; pt < PT; ++pt) {
        const pu4 v = lds_tr_operand<UX>(X, kk, pt, l16, g4);
        w[pt] = split3(unpack4(v[0], v[1]) * w0, unpack4(v[2], v[3]) * w1);
      }
      if (kk == 1) {
        wait_lds();
        copy_x(ck + 1);   // every read of this chunk's rows has its value
      }
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        const pu4 b = lds_tr_operand<U>(B, kk, nt, l16, g4);
#pragma unroll
        for (int pt = 0; pt < PT; ++pt) {
          pf4 v = kk == 0 ? S[nt][pt] * fade : S[nt][pt];
#pragma unroll
          for (int i = 0; i < 3; ++i) v = mma(b, w[pt].p[i], v);
          S[nt][pt] = v;
        }
      }
    }
    if (spoilt) {
#pragma unroll
      for (int pt = 0; pt < PT; ++pt) {
        const int p = 32 * (pt >> 1) + 8 * (l16 >> 2) + 4 * (pt & 1) + (l16 & 3);
        const float add = sSpoilt[wave][p] < kChunk ? __builtin_nanf("") : 0.0f;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) S[nt][pt] += add;
      }
    }
  }
  wait_memory();   // (the copies issued past the last chunk)

  if (a.state_out && seg.index == seg.count - 1 && on) {
    const int64_t slot = slot_of(a.idx, seg.seq, a.nslots);
    if (slot >= 0) {
      float* to = a.state_out + (slot * a.H + h) * head_size;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int pt = 0; pt < PT; ++pt) *reinterpret_cast<pf4*>(to + entry(nt, pt)) = S[nt][pt];
    }
  }
}

// One step for each row: 16 lanes own a state row, so a load instruction of theirs covers 256 contiguous bytes; the state
// is read and written once, and everything else is small beside it.
template <int N>
__global__ void __launch_bounds__(256) packed_ssd_step_kernel(PSsdArgs a) {
  constexpr int kV = N / 64;   // 16-byte pieces a lane holds of a row
  const int64_t row = int64_t(blockIdx.x) * 16 + threadIdx.x / 16;   // (token, head, p); 64 rows a head: all in range
  const int q = threadIdx.x % 16;
  const int64_t th = row / kHead;
  const int p = static_cast<int>(row % kHead);
  const int h = static_cast<int>(th % a.H);
  const int t = static_cast<int>(th / a.H);
  const int g = h / a.hpg;
  const int64_t slot = slot_of(a.idx, t, a.nslots);
  float* st = a.state_out + ((max(slot, int64_t(0)) * a.H + h) * kHead + p) * N;
  const uint16_t* Bt = a.B + t * a.bs + int64_t(g) * N;
  const uint16_t* Ct = a.C + t * a.cs + int64_t(g) * N;
  pf4 s[kV];
  pu2 bw[kV], cw[kV];
#pragma unroll
  for (int i = 0; i < kV; ++i) {
    const int n = 4 * (q + 16 * i);
    s[i] = *reinterpret_cast<const pf4*>(st + n);
    bw[i] = *reinterpret_cast<const pu2*>(Bt + n);
    cw[i] = *reinterpret_cast<const pu2*>(Ct + n);
  }
  const float xv = lo_f32(a.x[t * a.xs + int64_t(h) * kHead + p]);
  const float Dh = a.Dskip ? a.Dskip[h] : 0.0f;
  float delta, phi, la;
  step_scalars(lo_f32(a.dt[t * a.dts + h]), a.dt_bias ? a.dt_bias[h] : 0.0f, a.A[h], a.softplus, a.zoh, true, delta, phi,
               la);
  const float fade = slot >= 0 ? hw_exp2(la) : 0.0f;
  const float in = phi * xv;
  float acc = 0.0f;
#pragma unroll
  for (int i = 0; i < kV; ++i) {
    const float bv[4] = {lo_f32(bw[i][0]), hi_f32(bw[i][0]), lo_f32(bw[i][1]), hi_f32(bw[i][1])};
    const float cv[4] = {lo_f32(cw[i][0]), hi_f32(cw[i][0]), lo_f32(cw[i][1]), hi_f32(cw[i][1])};
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      // (without a state the row starts from zero, whatever the place read in its stead holds)
      s[i][c] = fmaf(fade, slot >= 0 ? s[i][c] : 0.0f, in * bv[c]);
      acc = fmaf(cv[c], s[i][c], acc);
    }
    if (slot >= 0) *reinterpret_cast<pf4*>(st + 4 * (q + 16 * i)) = s[i];
  }
  acc += row_ror<8>(acc);
  acc += row_ror<4>(acc);
  acc += row_ror<2>(acc);
  acc += row_ror<1>(acc);
  if (q == 0) Elem<uint16_t>::st(a.y, t * a.ys + int64_t(h) * kHead + p, fmaf(Dh, xv, acc));
}

template <int N>
ssm_status launch_fwd(const PSsdArgs& a, hipStream_t st) {
  hipLaunchKernelGGL((packed_ssd_fwd_kernel<N>), dim3(a.nwork), dim3(kWalkWaves * 64), 0, st, a);
  const hipError_t e = hipGetLastError();
  return e == hipSuccess ? SSM_OK : fail(SSM_ERR_HIP, "packed SSD launch: %s", hipGetErrorString(e));
}

template <int N>
ssm_status launch_step(const PSsdArgs& a, hipStream_t st) {
  hipLaunchKernelGGL((packed_ssd_step_kernel<N>), dim3(static_cast<uint32_t>(int64_t(a.T) * a.H * (kHead / 16))),
                     dim3(256), 0, st, a);
  const hipError_t e = hipGetLastError();
  return e == hipSuccess ? SSM_OK : fail(SSM_ERR_HIP, "packed SSD step launch: %s", hipGetErrorString(e));
}

size_t fwd_workspace(const ssm_ssd_packed_params* p) {
  const PackedPlan pl = packed_plan(p);
  if (!pl.split) return 0;
  return up256(size_t(pl.places) * p->nheads * kHead * p->dstate * 4) + up256(size_t(pl.places) * p->nheads * 4);
}

PSsdArgs ssd_args(const ssm_ssd_packed_params* p) {
  PSsdArgs a{};
  a.T = static_cast<int>(p->ntokens);
  a.S = static_cast<int>(p->nseqs);
  a.H = static_cast<int>(p->nheads);
  a.G = static_cast<int>(p->ngroups);
  a.hpg = a.H / a.G;
  a.nslots = p->nslots;
  a.xs = p->x_stride ? p->x_stride : p->nheads * kHead;
  a.ys = p->y_stride ? p->y_stride : p->nheads * kHead;
  a.dts = p->dt_stride ? p->dt_stride : p->nheads;
  a.bs = p->b_stride ? p->b_stride : p->ngroups * p->dstate;
  a.cs = p->c_stride ? p->c_stride : p->ngroups * p->dstate;
  a.softplus = p->dt_softplus;
  a.zoh = p->disc == SSM_DISC_ZOH;
  return a;
}

}  // namespace

ssm_status check_packed_ssd(const ssm_ssd_packed_params* p, bool step) {
  if (!p) return fail(SSM_ERR_NULL, "params is NULL");
  if (p->reserved != 0) return fail(SSM_ERR_UNSUPPORTED, "reserved must be 0");
  if (p->ntokens < 1 || p->nheads < 1 || p->ngroups < 1 || (!step && p->nseqs < 1) || p->nslots < 0)
    return fail(SSM_ERR_SHAPE, "ntokens, nseqs, nheads and ngroups must be >= 1, nslots >= 0");
  if (p->nheads % p->ngroups) return fail(SSM_ERR_SHAPE, "nheads (%lld) must be a multiple of ngroups (%lld)",
                                          (long long)p->nheads, (long long)p->ngroups);
  if (p->headdim != kHead) return fail(SSM_ERR_UNSUPPORTED, "headdim must be %d (got %lld)", kHead, (long long)p->headdim);
  if (p->dstate != 64 && p->dstate != 128 && p->dstate != 256)
    return fail(SSM_ERR_UNSUPPORTED, "dstate must be 64, 128 or 256 (got %lld)", (long long)p->dstate);
  if (p->ntokens >= (int64_t(1) << 30) || p->nheads > (int64_t(1) << 20) ||
      (!step && (p->nseqs > (int64_t(1) << 20))))
    return fail(SSM_ERR_SHAPE, "ntokens must be below 2^30, nheads and nseqs at most 2^20");
  if (p->io_dtype != SSM_BF16)
    return fail(SSM_ERR_DTYPE, "the SSD path takes bf16 x, dt, B and C (io_dtype must be SSM_BF16)");
  if (p->disc != SSM_DISC_EULER_B && p->disc != SSM_DISC_ZOH) return fail(SSM_ERR_UNSUPPORTED, "unknown disc %d", p->disc);
  if (p->dt_softplus != 0 && p->dt_softplus != 1)
    return fail(SSM_ERR_UNSUPPORTED, "dt_softplus must be 0 or 1 (got %d)", p->dt_softplus);
  if (p->segment_chunks < 0) return fail(SSM_ERR_UNSUPPORTED, "segment_chunks must be >= 0 (got %d)", p->segment_chunks);
  const int64_t head = p->nheads * kHead, grp = p->ngroups * p->dstate;
  const struct { int64_t s, row; } rows[] = {{p->x_stride, head}, {p->y_stride, head}, {p->dt_stride, p->nheads},
                                             {p->b_stride, grp}, {p->c_stride, grp}, {p->dy_stride, head},
                                             {p->dx_stride, head}, {p->ddt_stride, p->nheads}, {p->db_stride, grp},
                                             {p->dc_stride, grp}};
  // a chunk of 64 rows is addressed with 32-bit byte offsets
  const int64_t most = int64_t(1) << 24;
  for (const auto& r : rows) {
    if (r.s != 0 && r.s < r.row)
      return fail(SSM_ERR_SHAPE, "a row stride of %lld is shorter than a row of %lld", (long long)r.s, (long long)r.row);
    if (r.s >= most || r.row >= most)
      return fail(SSM_ERR_SHAPE, "rows and row strides must stay below 2^24 elements");
  }
  if (step && !fits_launch(p->ntokens * p->nheads * (kHead / 16), 256))
    return fail(SSM_ERR_SHAPE, "ntokens * nheads must be below 2^22 for one launch (got %lld)",
                (long long)(p->ntokens * p->nheads));
  if (!step) {
    const PackedPlan pl = packed_plan(p);
    if (!fits_launch(pl.nseg * p->ngroups * pl.hblocks, kWalkWaves * 64))
      return fail(SSM_ERR_SHAPE, "too many work items (segments times workgroups of 4 heads) for one launch");
    if (p->nheads * kHead * p->dstate / 1024 >= 65535) return fail(SSM_ERR_SHAPE, "nheads is too large");
  }
  return SSM_OK;
}

PackedPlan packed_plan(const ssm_ssd_packed_params* p) {
  PackedPlan pl{};
  const int64_t hpg = p->nheads / p->ngroups;
  pl.hblocks = static_cast<int>((hpg + kWalkHeads - 1) / kWalkHeads);
  const int64_t longest = (p->ntokens + kChunk - 1) / kChunk;      // chunks of one sequence, at most
  int64_t cps = p->segment_chunks;
  if (cps == 0) {
    // Every workgroup resident at once, two to a CU: the chunks over the places that are left after about half a segment
    // for the end of each sequence.  Where the sequences alone take more than half of the places, they follow one another
    // and only long ones are cut.  Segments below four chunks cost more than they spread (their states weigh as much as four chunks).
    const int64_t places = p->dstate == 256 ? 256 : 512, blocks = p->ngroups * pl.hblocks;
    const int64_t work = (p->ntokens / kChunk + p->nseqs / 2 + 1) * blocks, ends = p->nseqs * blocks / 2;
    cps = 2 * ends <= places ? (work + places - ends - 1) / (places - ends) : (2 * work + places - 1) / places;
    if (cps < 4) cps = 4;
  }
  if (cps > longest) cps = longest;
  pl.cps = static_cast<int>(cps);
  pl.split = longest > cps;
  pl.nseg = piece_numbers(p->nseqs, p->ntokens, cps * kChunk);
  pl.places = piece_places(p->ntokens, cps * kChunk);
  return pl;
}

}  // namespace ssm57

using namespace ssm57;

extern "C" size_t ssm_ssd_packed_fwd_workspace_bytes(const ssm_ssd_packed_params* p) {
  return check_packed_ssd(p, false) == SSM_OK ? fwd_workspace(p) : 0;
}

extern "C" ssm_status ssm_ssd_packed_fwd(const ssm_ssd_packed_params* p, const void* x, const void* dt,
                                         const float* dt_bias, const float* A, const void* B, const void* C,
                                         const float* Dskip, const int32_t* cu_seqlens, const float* state,
                                         const int32_t* state_idx, const uint8_t* has_state, float* state_out, void* y,
                                         void* workspace, size_t workspace_bytes, void* stream) {
  g_err[0] = 0;
  if (ssm_status s = check_packed_ssd(p, false); s != SSM_OK) return s;
  if (!x || !dt || !A || !B || !C || !cu_seqlens || !y)
    return fail(SSM_ERR_NULL, "x, dt, A, B, C, cu_seqlens and y are required");
  PSsdArgs a = ssd_args(p);
  if (!aligned(x, 16) || !aligned(B, 16) || !aligned(C, 16) || !aligned(y, 16) || a.xs % 8 || a.bs % 8 || a.cs % 8 ||
      a.ys % 8 || !aligned(state, 16) || !aligned(state_out, 16) || !aligned(dt, 2) || !aligned(A, 4) ||
      !aligned(dt_bias, 4) || !aligned(Dskip, 4) || !aligned(cu_seqlens, 4) || !aligned(state_idx, 4))
    return fail(SSM_ERR_ALIGN, "rows of x, B, C and y, and the states, must be 16-byte aligned");
  const size_t need = fwd_workspace(p);
  if (need > 0 && (!workspace || workspace_bytes < need || !aligned(workspace, 16)))
    return fail(SSM_ERR_WORKSPACE, "workspace of %zu bytes (16-byte aligned) needed, got %zu at %p", need,
                workspace_bytes, workspace);
  const PackedPlan pl = packed_plan(p);
  a.x = static_cast<const uint16_t*>(x);
  a.dt = static_cast<const uint16_t*>(dt);
  a.B = static_cast<const uint16_t*>(B);
  a.C = static_cast<const uint16_t*>(C);
  a.dt_bias = dt_bias;
  a.A = A;
  a.Dskip = Dskip;
  a.cu = cu_seqlens;
  a.state = state;
  a.idx = state_idx;
  a.has = has_state;
  a.state_out = state_out;
  a.y = static_cast<uint16_t*>(y);
  a.hblocks = pl.hblocks;
  a.cps = pl.cps;
  a.ws_state = static_cast<float*>(workspace);
  hipStream_t st = static_cast<hipStream_t>(stream);
  a.nwork = static_cast<int>(pl.nseg) * a.G * a.hblocks;
  if (pl.split) {
    StatesArgs w{};
    w.v = a.x;
    w.k = a.B;
    w.dt = a.dt;
    w.dt_bias = dt_bias;
    w.A = A;
    w.cu = cu_seqlens;
    w.init = state;
    w.idx = state_idx;
    w.has = has_state;
    w.ws_state = static_cast<float*>(workspace);
    w.ws_decay = reinterpret_cast<float*>(static_cast<char*>(workspace) +
                                          up256(size_t(pl.places) * p->nheads * kHead * p->dstate * 4));
    w.vs = a.xs;
    w.ks = a.bs;
    w.dts = a.dts;
    w.nslots = p->nslots;
    w.T = a.T;
    w.S = a.S;
    w.H = a.H;
    w.G = a.G;
    w.hpg = a.hpg;
    w.hblocks = a.hblocks;
    w.cps = a.cps;
    w.nseg = static_cast<int>(pl.nseg);
    w.softplus = a.softplus;
    w.zoh = a.zoh;
    if (ssm_status s = launch_states(w, nullptr, static_cast<int>(p->dstate), true, st); s != SSM_OK) return s;
  }
  switch (p->dstate) {
    case 64: return launch_fwd<64>(a, st);
    case 128: return launch_fwd<128>(a, st);
    default: return launch_fwd<256>(a, st);
  }
}

extern "C" ssm_status ssm_ssd_slot_update(const ssm_ssd_packed_params* p, float* state, const void* x, const void* dt,
                                          const float* dt_bias, const float* A, const void* B, const void* C,
                                          const float* Dskip, const int32_t* state_idx, void* y, void* stream) {
  g_err[0] = 0;
  if (ssm_status s = check_packed_ssd(p, true); s != SSM_OK) return s;
  if (!state || !x || !dt || !A || !B || !C || !y) return fail(SSM_ERR_NULL, "state, x, dt, A, B, C and y are required");
  if (p->nslots < 1) return fail(SSM_ERR_SHAPE, "nslots must be >= 1");
  PSsdArgs a = ssd_args(p);
  if (!aligned(state, 16) || !aligned(B, 8) || !aligned(C, 8) || a.bs % 4 || a.cs % 4 || !aligned(x, 2) ||
      !aligned(dt, 2) || !aligned(y, 2) || !aligned(A, 4) || !aligned(dt_bias, 4) || !aligned(Dskip, 4) ||
      !aligned(state_idx, 4))
    return fail(SSM_ERR_ALIGN, "state must be 16-byte and the rows of B and C 8-byte aligned");
  a.x = static_cast<const uint16_t*>(x);
  a.dt = static_cast<const uint16_t*>(dt);
  a.B = static_cast<const uint16_t*>(B);
  a.C = static_cast<const uint16_t*>(C);
  a.dt_bias = dt_bias;
  a.A = A;
  a.Dskip = Dskip;
  a.idx = state_idx;
  a.state_out = state;
  a.y = static_cast<uint16_t*>(y);
  hipStream_t st = static_cast<hipStream_t>(stream);
  switch (p->dstate) {
    case 64: return launch_step<64>(a, st);
    case 128: return launch_step<128>(a, st);
    default: return launch_step<256>(a, st);
  }
}
