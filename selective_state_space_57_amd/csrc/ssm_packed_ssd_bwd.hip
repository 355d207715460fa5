// Backward of the SSD layer over packed sequences.  With S_t the states and G_t = dL/dS_t:
//   G_t = dy_t C_t^T + a_{t+1} G_{t+1};  dx_t = phi_t G_t B_t + D dy_t;  dB_t = phi_t G_t^T x_t;  dC_t = S_t^T dy_t
//   dphi_t = x_t . G_t B_t;  dl_t = a_t <G_t, S_{t-1}> (l = Delta A, the decay's logarithm)
//   dDelta = A dl + phi'(Delta) dphi,  dA = sum Delta dl (+ sum dphi d phi/dA),  dD = sum dy . x
// (dB and dC summed over the heads of a group).  In chunks of 64 steps, with c the running sum of l in the chunk, S the
// state entering it and G the adjoint behind its last step, and for s <= t
//   L[t][s] = exp(c_t - c_s),  E_t = exp(c_t),  F_s = exp(c_63 - c_s),  X[t][s] = dy_t . x_s,  Z[t][s] = C_t . B_s:
//   dx_s = sum_t L Z phi_s dy_t + phi_s F_s G B_s + D dy_s
//   dC_t = sum_s K B_s + E_t S^T dy_t,  dB_s = sum_t K C_t + phi_s F_s G^T x_s,  K[t][s] = L X phi_s
//   dphi_s = sum_t W0[t][s] + F_s x_s . G B_s,  W0 = L X Z;  with W = W0 phi_s, u_t = E_t C_t . S^T dy_t and
//   v_s = phi_s F_s B_s . G^T x_s:
//   dl_r = sum_{t>=r} (sum_{s<t} W[t][s] - sum_{t'>t} W[t'][t]) + sum_{t>=r} u_t + sum_{s<r} v_s + exp(c_63) <G, S>
// Every sum in dl_r has the decays of what it stands for in it, so nothing large cancels: only the row and column sums
// of W do, and those are sums of the same fp32 numbers.
//
// Two walks (ssm_packed_states.hip) leave S and G of every chunk, laid out as operands over p; then a workgroup takes a
// chunk and runs over heads one after the other.  A wave has 16 of the N columns of the states, for every head: the sums
// of dB and dC over heads add up in its registers.  K is summed over heads in registers as well, and multiplied with B and
// C once at the end.  What a head needs across waves (dx, and the sums over n in u, v and <G, S>) goes through LDS, where
// the parts of G take turns and M's second part takes the place of x.  The next head's states are on their way while this
// head's dx is computed.
// Two workgroups share a CU (N <= 128), so that one's barriers and loads run beside the other's products: with chunks of
// 128 steps to a workgroup, which halve the saved states but recompute them in between, one filled the LDS and took
// 790 us instead of 566 (2.7B layer, 16384 tokens, states in two bf16 parts each).
// Measured on that layer: 703 to 777 us under the profiler, in a call of 1250 us whose walks, joins and sums over heads are
// the rest.  It reads 1.4 GB of states and 0.34 GB of inputs and writes 0.24 GB and what it spills; MFMA 13 % and VALU 45 % of
// the cycles: no single one is full, the stages of a head and the barriers between them are its time.  The kernel of N = 128
// is over its 128 registers by 18 (44 bytes a lane in scratch memory), that of 256 by 15.
//
// Precision: fp32 accumulation; the states are split into three bf16 parts, so that u, v and <G, S>, and with them dDelta
// and dA, are good to fp32 quality.  G in dx, M = L Z phi and the head sum K (both but for s = t, which is added in fp32)
// only reach dx, dB and dC: they are split into two parts, which leave out 2^-16 at most, so that these are the 64-bit
// values rounded once but for 1e-4 of them in the 2-norm (rounded to bf16 once each: 1e-3 to 2.4e-3, beside the outputs'
// own 1.66e-3, in a call of 1141 us).
#include "packed_ssd.hpp"

namespace ssm57 {
namespace {

struct BwdArgs {
  const uint16_t* x;
  const uint16_t* dt;
  const uint16_t* B;
  const uint16_t* C;
  const uint16_t* dy;
  const float* dt_bias;
  const float* A;
  const float* Dskip;
  const int32_t* cu;
  const float* S;      // [numbers][H][64 N] as state_operand lays them out: state entering each chunk
  const float* Gs;     // likewise: adjoint behind it
  uint16_t* dx;
  uint16_t* ddt;
  uint16_t* dB;
  uint16_t* dC;
  float* part_b;       // [splits][T][G N]
  float* part_c;
  float* part_h;       // [numbers][H][4]: sums of Delta dl (+ phi's share), ddt, dy . x
  float* dA;
  float* ddt_bias;
  float* dD;
  int64_t xs, dts, bs, cs, dys, dxs, ddts, dbs, dcs;
  int T, S_, H, G, hpg, splits, hps, numbers, nwork;
  int softplus, zoh;
};

struct alignas(16) ChunkScalars {
  // c_t (base 2) in two parts: differences of the first are good to their own rounding, and the second is what it leaves
  float c[kChunk], rest[kChunk];
  float phi[kChunk];
  float e[kChunk];                // exp(c_t)
  float pf[kChunk];               // phi_t exp(c_63 - c_t)
  float f[kChunk];                // exp(c_63 - c_t)
  float delta[kChunk], slope[kChunk];   // Delta_t, d Delta / d dt
};

__host__ __device__ constexpr int tile_row(int i) { return i >= 6 ? 3 : (i >= 3 ? 2 : (i >= 1 ? 1 : 0)); }
// place of the operand over 32 rows t (kk) of column tile sb: (0,0) (0,1) (1,0) (1,1) (2,1) (3,1)
__host__ __device__ constexpr int m_slot(int sb, int kk) { return sb < 2 ? 2 * sb + kk : sb + 2; }

// d phi / dA of the zero-order hold, phi = (exp(e) - 1) / A with e = Delta A: (e exp(e) - exp(e) + 1) / A^2, by its series
// times Delta^2 where the numerator cancels (the first term left out is below 2^-21 of the value for |e| < 1/2); 1 / A^2
// where the decay a = exp(e) is 0
__device__ __forceinline__ float zoh_slope(float delta, float A, float a) {
  const float e = delta * A;
  float p = 1.0f / 5760.0f;
  p = fmaf(p, e, 1.0f / 840.0f);
  p = fmaf(p, e, 1.0f / 144.0f);
  p = fmaf(p, e, 1.0f / 30.0f);
  p = fmaf(p, e, 0.125f);
  p = fmaf(p, e, 1.0f / 3.0f);
  p = fmaf(p, e, 0.5f);
  return fabsf(e) < 0.5f ? delta * delta * p : ((a == 0.0f ? 0.0f : fmaf(e, a, -a)) + 1.0f) / (A * A);
}

template <int N>
__global__ void __launch_bounds__(N * 4) __attribute__((amdgpu_waves_per_eu(N == 64 ? 3 : 4)))
packed_ssd_bwd_kernel(BwdArgs a) {
  constexpr int NW = N / 16;
  constexpr int U = N / 8, NK = N / 32;
  constexpr int kTiles = (10 + NW - 1) / NW;   // tiles on and below the diagonal that a wave owns
  constexpr int kJobs = NW < 8 ? 8 / NW : 1;   // pieces of dx a wave computes
  __shared__ alignas(16) uint16_t Bk[kChunk * N], Ck[kChunk * N];
  __shared__ alignas(16) uint16_t Xk[kChunk * kHead], Yk[kChunk * kHead];   // x and dy of the head
  __shared__ pu4 sM[6][64];                           // M, operands over t
  __shared__ alignas(16) uint16_t sG[N * kHead];       // G, transposed
  __shared__ ChunkScalars sc;
  __shared__ float sU[NW][kChunk], sV[NW][kChunk], sE[NW];
  // of 8 waves, two have a second tile of K: it waits in LDS and not in four more registers of every wave, which would spill
  // (16384 tokens, 2.7B layer, when tried: 642 us, else 690)
  constexpr int kHeld = NW == 8 ? 1 : kTiles;
  __shared__ pf4 sK2[kHeld < kTiles ? 2 : 1][64];
  __shared__ float sRow[10][16], sCol[10][16], sOwn[4][16], sDirect[4][16], sDiag[4], sTotal[10];

  const int item = xcd_item();
  if (item >= a.nwork) return;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int nt = wave;   // n-tile of the wave
  const int split = item % a.splits;
  const int g = item / a.splits % a.G;
  const int number = item / (a.splits * a.G);
  const int h_begin = g * a.hpg + split * a.hps, h_end = min(h_begin + a.hps, (g + 1) * a.hpg);
  Piece ck;
  if (!find_piece(a.cu, a.S_, a.T, kChunk, number, ck) || ck.end <= ck.begin) {
    // a number without a chunk adds nothing to the sums over all of them
    for (int h = h_begin + tid; h < h_end; h += NW * 64)
      *reinterpret_cast<pf4*>(a.part_h + (int64_t(number) * a.H + h) * 4) = pf4{0.0f, 0.0f, 0.0f, 0.0f};
    return;
  }
  const int64_t t_first = ck.begin + ck.index * kChunk;
  const int rows = min(ck.end - static_cast<int>(t_first), kChunk);
  const pf4 zero = {0.0f, 0.0f, 0.0f, 0.0f};

  // B and C of the group stay for all heads, and so does C B^T: rows t, columns s
  {
    const uint32_t brow = static_cast<uint32_t>(a.bs) * 2u, crow = static_cast<uint32_t>(a.cs) * 2u;
    copy_rows<U, NW>(Bk, chunk_rsrc(a.B + int64_t(g) * N, t_first, a.bs, rows, N), nt, lane, brow);
    copy_rows<U, NW>(Ck, chunk_rsrc(a.C + int64_t(g) * N, t_first, a.cs, rows, N), nt, lane, crow);
    if (nt == 0) {   // the halves of operands that lie above the diagonal stay zero
      reinterpret_cast<pu2*>(&sM[m_slot(1, 0)][lane])[0] = pu2{0u, 0u};
      reinterpret_cast<pu2*>(&sM[m_slot(3, 1)][lane])[0] = pu2{0u, 0u};
    }
    wait_memory();
    barrier_lds();
  }
  pf4 aB[4], aC[4];   // dB^T, dC^T: n = 16 nt + 4 g4 + c, step 16 b + l16
  pf4 aK[kHeld];      // K: rows t, columns s
#pragma unroll
  for (int b = 0; b < 4; ++b) aB[b] = aC[b] = zero;
#pragma unroll
  for (int i = 0; i < kHeld; ++i) aK[i] = zero;
  if (kHeld < kTiles && nt < 10 - NW) sK2[nt][lane] = zero;
  const int64_t head_size = int64_t(kHead) * N;

  const uint32_t xrow = static_cast<uint32_t>(a.xs) * 2u, yrow = static_cast<uint32_t>(a.dys) * 2u;
  auto copy_head = [&](uint16_t* dst, const uint16_t* src, int h, int64_t stride, uint32_t row_bytes)
                       __attribute__((always_inline)) {
    copy_rows<8, NW>(dst, chunk_rsrc(src + int64_t(h) * kHead, t_first, stride, rows, kHead), nt, afresh(lane), row_bytes);
  };
  // S and G of this wave's columns: n = 16 nt + l16, p = 32 (i/2) + 8 g4 + 4 (i%2) + c
  pf4 S[4], G[4];
  auto load_states = [&](int h) __attribute__((always_inline)) {
    const auto rs = make_rsrc(a.S + (int64_t(number) * a.H + h) * head_size, head_size);
    const auto rg = make_rsrc(a.Gs + (int64_t(number) * a.H + h) * head_size, head_size);
    const int l = afresh(lane);
    const int at = state_operand(nt, 0, l);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      S[i] = __builtin_bit_cast(pf4, __builtin_amdgcn_raw_buffer_load_b128(rs, at, state_operand(0, i, 0), 0));
      G[i] = __builtin_bit_cast(pf4, __builtin_amdgcn_raw_buffer_load_b128(rg, at, state_operand(0, i, 0), 0));
    }
  };

  // second parts of this wave's tiles as operands over t, laid out as sM (the halves above the diagonal are zeros)
  auto put_parts = [&](pu4 (*to)[64], const pu2 (&lo)[kTiles]) __attribute__((always_inline)) {
    const int l = afresh(lane);
#pragma unroll
    for (int ti = 0; ti < kTiles; ++ti) {
      const int i = nt + NW * ti;
      if (i >= 10) break;
      const int tb = tile_row(i), sb = i - tb * (tb + 1) / 2;
      pu2* at = reinterpret_cast<pu2*>(&to[m_slot(sb, tb >> 1)][l]);
      at[tb & 1] = lo[ti];
      if (sb == tb && (tb & 1)) at[0] = pu2{0u, 0u};
    }
  };
  load_states(h_begin);
  for (int h = h_begin; h < h_end; ++h) {
    const float Ah = a.A[h];
    const float Dh = a.Dskip ? a.Dskip[h] : 0.0f;
    barrier_lds();   // everyone is done with the head before
    copy_head(Xk, a.x, h, a.xs, xrow);
    copy_head(Yk, a.dy, h, a.dys, yrow);
    constexpr int kScalarTile = NW - 1;   // the wave of a chunk that works on its steps
    if (nt == kScalarTile) {
      const int lane = afresh(threadIdx.x) & 63;
      const float dtv = lo_f32(a.dt[(lane < rows ? t_first + lane : t_first) * a.dts + h]);
      const float bias = a.dt_bias ? a.dt_bias[h] : 0.0f;
      float delta, phi, la;
      step_scalars(dtv, bias, Ah, a.softplus, a.zoh, lane < rows, delta, phi, la);
      const DecaySum sum = sum_decays(la);
      const float c = static_cast<float>(sum.upto), f = hw_exp2(sum.behind());
      sc.c[lane] = c;
      sc.rest[lane] = static_cast<float>(sum.upto - c);
      sc.phi[lane] = phi;
      sc.e[lane] = hw_exp2(c);
      sc.f[lane] = f;
      sc.pf[lane] = phi * f;
      sc.delta[lane] = delta;
      sc.slope[lane] = a.softplus ? softplus_slope(dtv + bias) : 1.0f;
    }
    wait_memory();
    barrier_lds();   // x, dy and the scalars are there
    part_ends();
    pu4 g_lo[2];   // the second part of this wave's G, as its rows of sG
    {
      // ---- products with the states: <G, S>, q^T = S^T dy^T, r^T = G^T x^T
      const int l = afresh(lane), l16 = l & 15, g4 = l >> 4;
      float e = 0.0f;
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int c = 0; c < 4; ++c) e = fmaf(S[i][c], G[i][c], e);
      e = sum_wave(e);
      if (l == 0) sE[wave] = e;
      // sum over p of D rows against V's rows, the sum's share in u or v, and its part of dC or dB
      auto product = [&](pf4 (&D)[4], const uint16_t* V, const uint16_t* K, float* out, const float* weight,
                         pf4 (&acc)[4], bool keep) __attribute__((always_inline)) {
        part_ends();
#pragma unroll
        for (int i = 0; i < 4; ++i) asm volatile("" : "+v"(D[i]));   // (split now, not before)
        const Parts d[2] = {split3(D[0], D[1]), split3(D[2], D[3])};
        if (keep) {   // the row of n = 16 nt + l16 holds G[.][n]
#pragma unroll
          for (int kk = 0; kk < 2; ++kk)
            *reinterpret_cast<pu4*>(reinterpret_cast<char*>(sG) + unit_at<8>(16 * nt + l16, 4 * kk + g4)) = d[kk].p[0];
#pragma unroll
          for (int kk = 0; kk < 2; ++kk) g_lo[kk] = d[kk].p[1];
        }
#pragma unroll
        for (int b = 0; b < 4; ++b) {
          part_ends();
          const int row = 16 * b + l16;
          pf4 q[2] = {zero, zero};
#pragma unroll
          for (int kk = 0; kk < 2; ++kk) {
            const pu4 v = lds_row_operand<8>(V, row, kk, g4);
#pragma unroll
            for (int i = 0; i < 3; ++i) q[kk] = mma(d[kk].p[i], v, q[kk]);
          }
          const pf4 t = q[0] + q[1];
          const pu2 w = *reinterpret_cast<const pu2*>(reinterpret_cast<const char*>(K) +
                                                      unit_at<U>(row, 2 * nt + (g4 >> 1)) + 8 * (g4 & 1));
          const float s = sum_rows((t[0] * lo_f32(w[0]) + t[1] * hi_f32(w[0])) + (t[2] * lo_f32(w[1]) + t[3] * hi_f32(w[1])));
          if (g4 == 0) out[row] = s;
          acc[b] += t * weight[row];
          asm volatile("" : "+v"(acc[b]));   // (here, and not behind the loop with t kept for it)
        }
      };
      product(S, Yk, Ck, sU[wave], sc.e, aC, false);
      product(G, Xk, Bk, sV[wave], sc.pf, aB, true);
    }
    part_ends();
    // ---- tiles of L, X, Z
    pu2 m_lo[kTiles];
#pragma unroll
    for (int ti = 0; ti < kTiles; ++ti) {
      const int i = nt + NW * ti;
      if (i >= 10) break;
      const int l = afresh(lane), l16 = l & 15, g4 = l >> 4;
      const int tb = tile_row(i), sb = i - tb * (tb + 1) / 2;
      pf4 X = zero;
#pragma unroll
      for (int kk = 0; kk < 2; ++kk)
        X = mma(lds_row_operand<8>(Yk, 16 * tb + l16, kk, g4), lds_row_operand<8>(Xk, 16 * sb + l16, kk, g4), X);
      const float ph = sc.phi[16 * sb + l16];
      pf4 Z = zero;
#pragma unroll
      for (int kk = 0; kk < NK; ++kk) {
        if (kk % 2 == 0) part_ends();
        Z = mma(lds_row_operand<U>(Ck, 16 * tb + l16, kk, g4), lds_row_operand<U>(Bk, 16 * sb + l16, kk, g4), Z);
      }
      part_ends();
      // c_t - c_s
      const pf4 gap = (*reinterpret_cast<const pf4*>(&sc.c[16 * tb + 4 * g4]) - sc.c[16 * sb + l16]) +
                      (*reinterpret_cast<const pf4*>(&sc.rest[16 * tb + 4 * g4]) - sc.rest[16 * sb + l16]);
      pf4 k = ti < kHeld ? aK[min(ti, kHeld - 1)] : sK2[nt][l];
      pf4 m;
      float row[4], col = 0.0f;
      if (sb < tb) {
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const float L = hw_exp2(gap[c]), lx = L * X[c];
          k[c] = fmaf(lx, ph, k[c]);
          m[c] = L * Z[c] * ph;
          const float w0 = lx * Z[c];
          row[c] = w0 * ph;
          col += w0;
        }
      } else {
        float own = 0.0f, direct = 0.0f, diag = 0.0f;
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const int above = l16 - (4 * g4 + c);   // column minus row
          const float L = above <= 0 ? hw_exp2(gap[c]) : 0.0f, lx = L * X[c];
          k[c] = fmaf(lx, ph, k[c]);
          const float mm = L * Z[c] * ph, w0 = lx * Z[c];
          // a step's own terms: its dy goes into its dx in fp32, together with D, and W[t][t] is in its row and in its
          // column and would cancel but for rounding
          m[c] = above == 0 ? 0.0f : mm;
          row[c] = above == 0 ? 0.0f : w0 * ph;
          col += above == 0 ? 0.0f : w0;
          own += above == 0 ? w0 : 0.0f;
          direct += above == 0 ? mm : 0.0f;
          diag += above == 0 ? X[c] : 0.0f;
        }
        own = sum_rows(own);
        direct = sum_rows(direct);
        diag = sum_wave(diag);
        if (g4 == 0) {
          sOwn[tb][l16] = own;
          sDirect[tb][l16] = direct + Dh;
        }
        if (l == 0) sDiag[tb] = diag;
      }
      pu2 m_hi;
      split2(m, m_hi, m_lo[ti]);
      reinterpret_cast<pu2*>(&sM[m_slot(sb, tb >> 1)][l])[tb & 1] = m_hi;
      if (ti < kHeld) {
        aK[min(ti, kHeld - 1)] = k;
        asm volatile("" : "+v"(aK[min(ti, kHeld - 1)]));
      } else {
        sK2[nt][l] = k;
      }
      part_ends();
#pragma unroll
      for (int c = 0; c < 4; ++c) row[c] = sum_row(row[c]);
      if (l16 < 4) sRow[i][4 * g4 + l16] = (l16 & 2) ? ((l16 & 1) ? row[3] : row[2]) : ((l16 & 1) ? row[1] : row[0]);
      col = sum_rows(col);
      if (g4 == 0) sCol[i][l16] = col;
      const float tile = sum_rows((row[0] + row[1]) + (row[2] + row[3]));
      if (l == 0) sTotal[i] = tile;
    }
    barrier_lds();   // M, G and the partial sums are there, and x is read
    if (h + 1 < h_end) load_states(h + 1);
    pu4 (*sMl)[64] = reinterpret_cast<pu4(*)[64]>(Xk);   // M's second part takes the place of x
    put_parts(sMl, m_lo);
    part_ends();
    // ---- dx: a pair of column tiles (32 p) of one tile of steps at a time.  G's parts take turns in sG.
    pf4 d[kJobs][2], dm[kJobs][2];
    auto add_g = [&]() __attribute__((always_inline)) {
#pragma unroll
      for (int j = 0; j < kJobs; ++j) {
        const int job = nt + NW * j;
        if (job >= 8) break;
        const int l = afresh(lane), l16 = l & 15, g4 = l >> 4;
        const int sb = job & 3, pp = job >> 2;
#pragma unroll
        for (int kk = 0; kk < NK; ++kk) {
          const pu4 b = lds_row_operand<U>(Bk, 16 * sb + l16, kk, g4);
#pragma unroll
          for (int e = 0; e < 2; ++e) d[j][e] = mma(lds_tr_operand8<8>(sG, kk, 2 * pp + e, l16, g4), b, d[j][e]);
        }
      }
    };
#pragma unroll
    for (int j = 0; j < kJobs; ++j) d[j][0] = d[j][1] = dm[j][0] = dm[j][1] = zero;
    add_g();
    barrier_lds();   // the first part of G is read, the second of M is there
    part_ends();
    {
      const int l = afresh(lane), l16 = l & 15, g4 = l >> 4;
#pragma unroll
      for (int kk = 0; kk < 2; ++kk)
        *reinterpret_cast<pu4*>(reinterpret_cast<char*>(sG) + unit_at<8>(16 * nt + l16, 4 * kk + g4)) = g_lo[kk];
#pragma unroll
      for (int j = 0; j < kJobs; ++j) {
        const int job = nt + NW * j;
        if (job >= 8) break;
        const int sb = job & 3, pp = job >> 2;
#pragma unroll
        for (int kk = 0; kk < 2; ++kk) {
          if (sb >= 2 && kk == 0) continue;   // no step of the first half follows one of the second
          const pu4 m = sM[m_slot(sb, kk)][l], ml = sMl[m_slot(sb, kk)][l];
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const pu4 y = lds_tr_operand<8>(Yk, kk, 2 * pp + e, l16, g4);
            dm[j][e] = mma(y, ml, dm[j][e]);
            dm[j][e] = mma(y, m, dm[j][e]);
          }
        }
      }
    }
    barrier_lds();   // the second part of G is there
    part_ends();
    add_g();
#pragma unroll
    for (int j = 0; j < kJobs; ++j) {
      const int job = nt + NW * j;
      if (job >= 8) break;
      const int l = afresh(lane), l16 = l & 15, g4 = l >> 4;
      const int sb = job & 3, pp = job >> 2;
      const float pf = sc.pf[16 * sb + l16], dr = sDirect[sb][l16];
      const pu4 yv = lds_u4(Yk, unit_at<8>(16 * sb + l16, 4 * pp + g4));
      const pf4 d0 = dm[j][0] + d[j][0] * pf, d1 = dm[j][1] + d[j][1] * pf;
      const pu4 o = {pack_bf16(fmaf(dr, lo_f32(yv[0]), d0[0]), fmaf(dr, hi_f32(yv[0]), d0[1])),
                     pack_bf16(fmaf(dr, lo_f32(yv[1]), d0[2]), fmaf(dr, hi_f32(yv[1]), d0[3])),
                     pack_bf16(fmaf(dr, lo_f32(yv[2]), d1[0]), fmaf(dr, hi_f32(yv[2]), d1[1])),
                     pack_bf16(fmaf(dr, lo_f32(yv[3]), d1[2]), fmaf(dr, hi_f32(yv[3]), d1[3]))};
      __builtin_amdgcn_raw_buffer_store_b128(
          o, chunk_rsrc(a.dx + int64_t(h) * kHead, t_first, a.dxs, rows, kHead),
          static_cast<int>(static_cast<uint32_t>(16 * sb + l16) * (static_cast<uint32_t>(a.dxs) * 2u) +
                           (32u * pp + 8u * g4) * 2u), 0, 0);
    }
    part_ends();
    // ---- the steps' own gradients
    if (nt == kScalarTile) {
      const int lane = afresh(threadIdx.x) & 63, l16 = lane & 15, tl = lane >> 4;
      part_ends();
      // sums of W over the row, and of W0 over the column, of step `lane`: in its own tile, and in those beside and below
      const float row = sRow[tl * (tl + 1) / 2 + tl][l16], col = sCol[tl * (tl + 1) / 2 + tl][l16];
      float row_off = 0.0f, col_off = 0.0f, u = 0.0f, v = 0.0f, e = 0.0f;
#pragma unroll
      for (int o = 0; o < 4; ++o) {
        row_off += o < tl ? sRow[tl * (tl + 1) / 2 + min(o, tl)][l16] : 0.0f;
        const int tt = max(o, tl);
        col_off += o > tl ? sCol[tt * (tt + 1) / 2 + tl][l16] : 0.0f;
      }
#pragma unroll
      for (int w = 0; w < NW; ++w) {
        if (w % 4 == 0) part_ends();
        u += sU[w][lane];
        v += sV[w][lane];
        e += sE[w];
        asm volatile("" : "+v"(u), "+v"(v), "+v"(e));
      }
      const float phi = sc.phi[lane];
      u *= sc.e[lane];
      v *= sc.f[lane];
      const float dphi = col + col_off + sOwn[tl][l16] + v;
      const float before = phi * v, off = phi * col_off;
      // sum_{t>=r, s<r} W: the tiles below and beside the step's own, in full (their numbers are tb (tb + 1) / 2 + sb), the
      // rows from r on of those beside, the columns before r of those below, and the own tile's corner, where alone rows
      // less columns are taken, over 16 steps (over the whole chunk, sums much larger than dl would cancel)
      const float far = tl == 1 ? sTotal[3] + sTotal[6] : tl == 2 ? sTotal[6] + sTotal[7] : 0.0f;
      float dl = row_suffix(row_off + (row - phi * col)) + (row_prefix(off) - off) + far + wave_suffix(u, lane) +
                       (wave_prefix(before, lane) - before) + sc.e[kChunk - 1] * e;
      const float delta = sc.delta[lane], decay = hw_exp2(decay_log(delta, Ah));
      // (dl = a <G, S> is nothing where a is: what the sums leave by rounding would count Delta times in dA)
      dl = decay == 0.0f ? 0.0f : dl;
      const float dd = (Ah * dl + (a.zoh ? decay * dphi : dphi)) * sc.slope[lane];
      float sum_a = 0.0f, sum_t = 0.0f, sum_d = lane < 4 ? sDiag[lane] : 0.0f;
      if (lane < rows) {
        Elem<uint16_t>::st(a.ddt, (t_first + lane) * a.ddts + h, dd);
        sum_a = delta * dl + (a.zoh ? zoh_slope(delta, Ah, decay) * dphi : 0.0f);
        sum_t = dd;
      }
      sum_a = sum_wave(sum_a);
      sum_t = sum_wave(sum_t);
      sum_d = sum_wave(sum_d);
      if (lane == 0)
        *reinterpret_cast<pf4*>(a.part_h + (int64_t(number) * a.H + h) * 4) = pf4{sum_a, sum_t, sum_d, 0.0f};
    }
  }

  // ---- the heads' K with B and C, and the sums over this workgroup's heads
  barrier_lds();
  const int l16 = lane & 15, g4 = lane >> 4;
  // K in two parts: row by row where x and dy were, and as operands over t in sM and where G was
  pu4 (*sMl)[64] = reinterpret_cast<pu4(*)[64]>(sG);
  pu2 k_lo[kTiles];
#pragma unroll
  for (int ti = 0; ti < kTiles; ++ti) {
    const int i = nt + NW * ti;
    if (i >= 10) break;
    const int tb = tile_row(i), sb = i - tb * (tb + 1) / 2;
    pf4 v = ti < kHeld ? aK[min(ti, kHeld - 1)] : sK2[nt][lane];
    if (sb == tb) {   // a step's own term is added in fp32
      float own = 0.0f;
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        own += l16 == 4 * g4 + c ? v[c] : 0.0f;
        v[c] = l16 == 4 * g4 + c ? 0.0f : v[c];
      }
      own = sum_rows(own);
      if (g4 == 0) sOwn[tb][l16] = own;
    }
    pu2 hi;
    split2(v, hi, k_lo[ti]);
    reinterpret_cast<pu2*>(&sM[m_slot(sb, tb >> 1)][lane])[tb & 1] = hi;
#pragma unroll
    for (int part = 0; part < 2; ++part) {
      char* at = reinterpret_cast<char*>(part ? Yk : Xk);
      const pu2 k = part ? k_lo[ti] : hi;
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const int row = 16 * tb + 4 * g4 + c, byte = 2 * (l16 & 7);
        *reinterpret_cast<uint16_t*>(at + unit_at<8>(row, 2 * sb + (l16 >> 3)) + byte) =
            static_cast<uint16_t>(k[c >> 1] >> (16 * (c & 1)));
        // (the tile right of an even diagonal tile belongs to the same operand)
        if (sb == tb && (tb & 1) == 0)
          *reinterpret_cast<uint16_t*>(at + unit_at<8>(row, 2 * (sb + 1) + (l16 >> 3)) + byte) = 0;
      }
    }
  }
  put_parts(sMl, k_lo);
  barrier_lds();
#pragma unroll
  for (int kk = 0; kk < 2; ++kk) {
    const pu4 bt = lds_tr_plain_operand<U, true>(Bk, kk, nt, l16, g4);
    const pu4 ct = lds_tr_plain_operand<U, false>(Ck, kk, nt, l16, g4);
#pragma unroll
    for (int b = 0; b < 4; ++b) {
      if (kk <= b / 2) {
        aC[b] = mma(bt, lds_row_operand<8>(Yk, 16 * b + l16, kk, g4), aC[b]);
        aC[b] = mma(bt, lds_row_operand<8>(Xk, 16 * b + l16, kk, g4), aC[b]);
      }
      if (kk == 1 || b < 2) {
        aB[b] = mma(ct, sMl[m_slot(b, kk)][lane], aB[b]);
        aB[b] = mma(ct, sM[m_slot(b, kk)][lane], aB[b]);
      }
    }
  }
#pragma unroll
  for (int b = 0; b < 4; ++b) {
    const int t = 16 * b + l16;
    const int64_t at = ((int64_t(split) * a.T + t_first + t) * a.G + g) * N + 16 * nt + 4 * g4;
    const float own = sOwn[b][l16];
    const int place = unit_at<U>(t, 2 * nt + (g4 >> 1)) + 8 * (g4 & 1);
    const pu2 cw = *reinterpret_cast<const pu2*>(reinterpret_cast<const char*>(Ck) + place);
    const pu2 bw = *reinterpret_cast<const pu2*>(reinterpret_cast<const char*>(Bk) + place);
    if (t < rows) {
      *reinterpret_cast<pf4*>(a.part_b + at) =
          aB[b] + own * pf4{lo_f32(cw[0]), hi_f32(cw[0]), lo_f32(cw[1]), hi_f32(cw[1])};
      *reinterpret_cast<pf4*>(a.part_c + at) =
          aC[b] + own * pf4{lo_f32(bw[0]), hi_f32(bw[0]), lo_f32(bw[1]), hi_f32(bw[1])};
    }
  }
}

// What the workgroups left in parts.  The first H blocks: dA, ddt_bias and dD of a head, the chunks' sums, 256 interleaved
// runs joined in a fixed order.  The others: dB (y = 0) and dC, the splits' sums in order, rounded once; a thread owns four
// columns of a row, and rows outside every sequence stay as they are.
__global__ void __launch_bounds__(256) packed_ssd_bwd_sums_kernel(BwdArgs a, int cols) {
  if (static_cast<int>(blockIdx.x) < a.H) {
    __shared__ pf4 sum[256];
    if (blockIdx.y) return;
    const int h = blockIdx.x;
    pf4 v = {0.0f, 0.0f, 0.0f, 0.0f};
    for (int i = threadIdx.x; i < a.numbers; i += 256)
      v += *reinterpret_cast<const pf4*>(a.part_h + (int64_t(i) * a.H + h) * 4);
    sum[threadIdx.x] = v;
    __syncthreads();
    for (int m = 128; m >= 1; m >>= 1) {
      if (static_cast<int>(threadIdx.x) < m) sum[threadIdx.x] += sum[threadIdx.x + m];
      __syncthreads();
    }
    if (threadIdx.x == 0) {
      a.dA[h] = sum[0][0];
      if (a.ddt_bias) a.ddt_bias[h] = sum[0][1];
      if (a.dD) a.dD[h] = sum[0][2];
    }
    return;
  }
  const int64_t at = int64_t(blockIdx.x - a.H) * 256 + threadIdx.x;
  const int64_t t = at / (cols / 4);
  const int col = static_cast<int>(at % (cols / 4)) * 4;
  if (t >= a.T || t < a.cu[0] || t >= a.cu[a.S_]) return;
  const float* part = (blockIdx.y ? a.part_c : a.part_b) + t * cols + col;
  pf4 v = *reinterpret_cast<const pf4*>(part);
  for (int s = 1; s < a.splits; ++s) v += *reinterpret_cast<const pf4*>(part + int64_t(s) * a.T * cols);
  uint16_t* out = (blockIdx.y ? a.dC + t * a.dcs : a.dB + t * a.dbs) + col;
  *reinterpret_cast<pu2*>(out) = bf16x4(v[0], v[1], v[2], v[3]);
}

struct BwdPlan {
  PackedPlan walk;
  int splits, hps;
  int64_t numbers;
  size_t states, ws_state, ws_decay, part, part_h, total;   // bytes: one set of saved states, ..., one of part_b and part_c
};
BwdPlan bwd_plan(const ssm_ssd_packed_params* p) {
  BwdPlan b{};
  b.walk = packed_plan(p);
  b.numbers = piece_numbers(p->nseqs, p->ntokens, kChunk);
  const int64_t hpg = p->nheads / p->ngroups;
  // four workgroups for each place on the 256 CUs, to even out their lengths; each split costs a partial dB and dC (16384
  // tokens, 2.7B layer: about 1024, 2048 and 4096 workgroups 1180, 1137 and 1166 us a call on one card)
  int64_t splits = (2048 + b.numbers * p->ngroups - 1) / (b.numbers * p->ngroups);
  if (splits > hpg) splits = hpg;
  b.hps = static_cast<int>((hpg + splits - 1) / splits);
  b.splits = static_cast<int>((hpg + b.hps - 1) / b.hps);
  const size_t state = size_t(p->nheads) * kHead * p->dstate * 4;
  b.states = up256(size_t(b.numbers) * state);
  b.ws_state = b.walk.split ? up256(size_t(b.walk.places) * state) : 0;
  b.ws_decay = b.walk.split ? up256(size_t(b.walk.places) * p->nheads * 4) : 0;
  b.part = up256(size_t(b.splits) * p->ntokens * p->ngroups * p->dstate * 4);
  b.part_h = up256(size_t(b.numbers) * p->nheads * 16);
  b.total = 2 * (b.states + b.ws_state + b.ws_decay + b.part) + b.part_h;
  return b;
}

ssm_status check_bwd(const ssm_ssd_packed_params* p) {
  if (ssm_status s = check_packed_ssd(p, false); s != SSM_OK) return s;
  const BwdPlan b = bwd_plan(p);
  // (the main pass's grid is rounded up to the 8 XCDs; the sums' blocks take four columns of a row a thread)
  if (!fits_launch(b.numbers * b.splits * p->ngroups + 7, static_cast<int>(p->dstate) * 4))
    return fail(SSM_ERR_SHAPE, "too many work items (chunks times groups) for one launch");
  if (!fits_launch(p->nheads + p->ntokens * p->ngroups * p->dstate / 1024 + 1, 256))
    return fail(SSM_ERR_SHAPE, "ntokens * ngroups * dstate is too large for one launch");
  return SSM_OK;
}

template <int N>
void launch_bwd(const BwdArgs& a, hipStream_t st) {
  hipLaunchKernelGGL((packed_ssd_bwd_kernel<N>), dim3((a.nwork + 7) / 8 * 8), dim3(N * 4), 0, st, a);
}

}  // namespace
}  // namespace ssm57

using namespace ssm57;

extern "C" size_t ssm_ssd_packed_bwd_workspace_bytes(const ssm_ssd_packed_params* p) {
  return check_bwd(p) == SSM_OK ? bwd_plan(p).total : 0;
}

extern "C" ssm_status ssm_ssd_packed_bwd(const ssm_ssd_packed_params* p, const void* x, const void* dt,
                                         const float* dt_bias, const float* A, const void* B, const void* C,
                                         const float* Dskip, const int32_t* cu_seqlens, const float* state,
                                         const int32_t* state_idx, const uint8_t* has_state, const void* dy,
                                         const float* dstate_out, void* dx, void* ddt, float* dA, void* dB, void* dC,
                                         float* dDskip, float* ddt_bias, float* dstate, void* workspace,
                                         size_t workspace_bytes, void* stream) {
  g_err[0] = 0;
  if (ssm_status s = check_bwd(p); s != SSM_OK) return s;
  if (!x || !dt || !A || !B || !C || !cu_seqlens || !dy || !dx || !ddt || !dA || !dB || !dC)
    return fail(SSM_ERR_NULL, "x, dt, A, B, C, cu_seqlens, dy, dx, ddt, dA, dB and dC are required");
  auto row = [](int64_t s, int64_t dense) { return s ? s : dense; };
  const int64_t heads = p->nheads * kHead, grp = p->ngroups * p->dstate;
  BwdArgs a{};
  a.xs = row(p->x_stride, heads);
  a.dts = row(p->dt_stride, p->nheads);
  a.bs = row(p->b_stride, grp);
  a.cs = row(p->c_stride, grp);
  a.dys = row(p->dy_stride, heads);
  a.dxs = row(p->dx_stride, heads);
  a.ddts = row(p->ddt_stride, p->nheads);
  a.dbs = row(p->db_stride, grp);
  a.dcs = row(p->dc_stride, grp);
  if (!aligned(x, 16) || !aligned(B, 16) || !aligned(C, 16) || !aligned(dy, 16) || !aligned(dx, 16) || a.xs % 8 ||
      a.bs % 8 || a.cs % 8 || a.dys % 8 || a.dxs % 8 || !aligned(state, 16) || !aligned(dstate_out, 16) ||
      !aligned(dstate, 16) || !aligned(dB, 8) || !aligned(dC, 8) || a.dbs % 4 || a.dcs % 4 || !aligned(dt, 2) ||
      !aligned(ddt, 2) || !aligned(A, 4) || !aligned(dt_bias, 4) || !aligned(Dskip, 4) || !aligned(cu_seqlens, 4) ||
      !aligned(state_idx, 4) || !aligned(dA, 4) || !aligned(dDskip, 4) || !aligned(ddt_bias, 4))
    return fail(SSM_ERR_ALIGN, "rows of x, B, C, dy and dx, and the states, must be 16-byte aligned, of dB and dC 8-byte");
  const BwdPlan b = bwd_plan(p);
  if (!workspace || workspace_bytes < b.total || !aligned(workspace, 16))
    return fail(SSM_ERR_WORKSPACE, "workspace of %zu bytes (16-byte aligned) needed, got %zu at %p", b.total,
                workspace_bytes, workspace);
  char* at = static_cast<char*>(workspace);
  auto take = [&](size_t bytes) {
    float* f = reinterpret_cast<float*>(at);
    at += bytes;
    return f;
  };
  float* save_s = take(b.states);
  float* save_g = take(b.states);
  StatesArgs w{};
  w.ws_state = take(b.ws_state);
  w.ws_decay = take(b.ws_decay);
  float* walk_g = take(b.ws_state);
  float* decay_g = take(b.ws_decay);
  a.part_b = take(b.part);
  a.part_c = take(b.part);
  a.part_h = take(b.part_h);
  a.x = static_cast<const uint16_t*>(x);
  a.dt = static_cast<const uint16_t*>(dt);
  a.B = static_cast<const uint16_t*>(B);
  a.C = static_cast<const uint16_t*>(C);
  a.dy = static_cast<const uint16_t*>(dy);
  a.dt_bias = dt_bias;
  a.A = A;
  a.Dskip = Dskip;
  a.cu = cu_seqlens;
  a.S = save_s;
  a.Gs = save_g;
  a.dx = static_cast<uint16_t*>(dx);
  a.ddt = static_cast<uint16_t*>(ddt);
  a.dB = static_cast<uint16_t*>(dB);
  a.dC = static_cast<uint16_t*>(dC);
  a.dA = dA;
  a.ddt_bias = ddt_bias;
  a.dD = dDskip;
  a.T = static_cast<int>(p->ntokens);
  a.S_ = static_cast<int>(p->nseqs);
  a.H = static_cast<int>(p->nheads);
  a.G = static_cast<int>(p->ngroups);
  a.hpg = a.H / a.G;
  a.splits = b.splits;
  a.hps = b.hps;
  a.numbers = static_cast<int>(b.numbers);
  a.nwork = a.numbers * a.G * a.splits;
  a.softplus = p->dt_softplus;
  a.zoh = p->disc == SSM_DISC_ZOH;
  hipStream_t st = static_cast<hipStream_t>(stream);

  w.dt = a.dt;
  w.dt_bias = dt_bias;
  w.A = A;
  w.cu = cu_seqlens;
  w.dts = a.dts;
  w.T = a.T;
  w.S = a.S_;
  w.H = a.H;
  w.G = a.G;
  w.hpg = a.hpg;
  w.hblocks = b.walk.hblocks;
  w.cps = b.walk.cps;
  w.nseg = static_cast<int>(b.walk.nseg);
  w.softplus = a.softplus;
  w.zoh = a.zoh;
  // the states, forward from the slots, and the adjoints, in reverse order from dstate_out
  w.v = a.x;
  w.vs = a.xs;
  w.k = a.B;
  w.ks = a.bs;
  w.init = state;
  w.idx = state_idx;
  w.has = has_state;
  w.nslots = p->nslots;
  w.save = save_s;
  StatesArgs r = w;
  r.ws_state = walk_g;
  r.ws_decay = decay_g;
  r.v = a.dy;
  r.vs = a.dys;
  r.k = a.C;
  r.ks = a.cs;
  r.init = dstate_out;
  r.idx = nullptr;
  r.has = nullptr;
  r.nslots = p->nseqs;
  r.save = save_g;
  r.last = dstate;
  if (ssm_status s = launch_states(w, &r, static_cast<int>(p->dstate), b.walk.split, st); s != SSM_OK) return s;
  switch (p->dstate) {
    case 64: launch_bwd<64>(a, st); break;
    case 128: launch_bwd<128>(a, st); break;
    default: launch_bwd<256>(a, st); break;
  }
  const int cols = static_cast<int>(grp);
  hipLaunchKernelGGL(packed_ssd_bwd_sums_kernel,
                     dim3(static_cast<uint32_t>(a.H + (int64_t(a.T) * (cols / 4) + 255) / 256), 2), dim3(256), 0, st, a, cols);
  const hipError_t e = hipGetLastError();
  return e == hipSuccess ? SSM_OK : fail(SSM_ERR_HIP, "packed SSD backward launch: %s", hipGetErrorString(e));
}
