// The residual's addition and the root mean square norm in front of a projection, forward and backward, with an output in
// 8 bits for the projection's matrix product:
//   h = x + residual,  r = 1 / sqrt(mean(h^2) + eps),  y = h r w
//   backward, with dn = dy w:  dsum = dh + r (dn - h r^2 mean(dn h)),  dw = sum over rows of dy h r
//
// Bound by memory: every array is read or written once.  A team of lanes (one wave, 4 or 16) holds a row in registers,
// eight consecutive channels to a chunk, so that 16 lanes hold a block of 128 and its largest magnitude is four DPP steps.
// A workgroup walks down the rows with the weight in registers; the backward's weight gradient adds up in registers, and
// the workgroups' partial sums are joined in a fixed order by a second kernel.  h, sums, r and weight gradients are fp32;
// the norm is taken of the fp32 h, also where the residual that is written is rounded to bf16.  A row whose squares leave fp32's
// range is summed again, times a power of two (what every row pays for the check, us with it and without: 16384 rows of 2560
// forward 90.0 and 89.9, 8191 backward 68.8 and 68.1, 2000 rows of 16384 backward 114.3 and 111.6).
//
// Measured (a large copy reaches 5.1 TB/s): 16384 rows of 2560, bf16 with an fp32 residual and 8-bit output, 461 MB, 88 us
// (5.2 TB/s); 4099 rows 25 us; 64 rows 3.6 us, all but a little of it latency: load, two barriers, store.  Backward, 8191 rows
// of 2560, 336 MB, 64 to 66 us (5.2 TB/s) and 4 for the join.
#include "fp8.hpp"

namespace ssm57 {
namespace {

constexpr int kMaxDim = 16384;

struct AddNormArgs {
  const void* x;
  const void* res;     // residual; in the backward dh
  const float* w;
  void* h;             // residual_out; in the backward the sum (read)
  void* y;
  float* scale;
  const void* dy;
  void* dx;
  void* dres;
  float* part;         // [nb][dim]: partial sums of dw
  float* dw;
  int64_t xs, rs, hs, ys, ss, dys, dxs, drs;
  int T, D, D16, nb;
  float eps;
  int f8;
};

// sums of K values over a team, in every lane of it
template <int TEAM, int K>
__device__ __forceinline__ void team_sum(float (&v)[K], float (*lds)[K]) {
#pragma unroll
  for (int m = 32; m >= 1; m >>= 1)
#pragma unroll
    for (int k = 0; k < K; ++k) v[k] += __shfl_xor(v[k], m);
  if constexpr (TEAM > 64) {
    __syncthreads();   // (the sums before this one have been read)
    if ((threadIdx.x & 63) == 0) {
#pragma unroll
      for (int k = 0; k < K; ++k) lds[threadIdx.x >> 6][k] = v[k];
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < K; ++k) v[k] = 0.0f;
#pragma unroll
    for (int i = 0; i < TEAM / 64; ++i)
#pragma unroll
      for (int k = 0; k < K; ++k) v[k] += lds[i][k];
  }
}

// Rows whose squares leave fp32's range: the power of two that brings them back, or 1.  m: mean square and eps, the same in all
// lanes of a team.  (Below the upper bound and above the lower one r^2 and the sums of up to 2^14 squares are ordinary numbers;
// infinities and NaN stay what they are.)
__device__ __forceinline__ float unusual(float m) { return m > 0x1p100f ? 0x1p-80f : m < 0x1p-100f ? 0x1p100f : 1.0f; }

// A lane's chunk of a row: all of it, the row's end, or nothing.  FULL: dim is a multiple of 8, there is no cut chunk.
template <typename T, bool FULL>
__device__ __forceinline__ void load_chunk(Eight<T>& e, const T* p, int at, int cnt) {
  if constexpr (FULL) {
    if (cnt > 0) e.load(p + at);
    else e.zero();
  } else {
    if (cnt >= 8) e.load(p + at);
    else e.load(p + at, cnt);
  }
}
template <typename T, bool FULL>
__device__ __forceinline__ void store_chunk(T* p, const float* v, int at, int cnt) {
  if (FULL ? cnt > 0 : cnt >= 8) Eight<T>::store(p + at, v);
  else if constexpr (!FULL) Eight<T>::store(p + at, v, cnt);
}

template <typename TX, typename TR, int TEAM, int R, bool FULL>
__global__ void __launch_bounds__(TEAM < 256 ? 256 : TEAM) add_norm_fwd_kernel(AddNormArgs a) {
  constexpr int kTeams = TEAM < 256 ? 256 / TEAM : 1;
  __shared__ float red[TEAM < 256 ? 1 : TEAM / 64][1];
  const int lane = threadIdx.x % TEAM, team = threadIdx.x / TEAM;
  const float inv_n = 1.0f / static_cast<float>(a.D);
  int at[R], cnt[R];
  float w[R][8];
#pragma unroll
  for (int j = 0; j < R; ++j) {
    at[j] = (j * TEAM + lane) * 8;
    cnt[j] = a.D - at[j];
    Eight<float> e;
    load_chunk<float, FULL>(e, a.w, at[j], cnt[j]);
    e.get(w[j]);
  }
  const TX* x = static_cast<const TX*>(a.x);
  const TR* res = static_cast<const TR*>(a.res);
  // (the teams of a workgroup run the same number of turns: a row past the end is computed as row 0 and not stored)
  for (int64_t r0 = int64_t(blockIdx.x) * kTeams; r0 < a.T; r0 += int64_t(a.nb) * kTeams) {
    const bool on = r0 + team < a.T;
    const int64_t row = on ? r0 + team : 0;
    Eight<TX> px[R];
    Eight<TR> pr[R];
#pragma unroll
    for (int j = 0; j < R; ++j) {
      load_chunk<TX, FULL>(px[j], x + row * a.xs, at[j], cnt[j]);
      if (res) load_chunk<TR, FULL>(pr[j], res + row * a.rs, at[j], cnt[j]);
    }
    float h[R][8], q[1] = {0.0f};
#pragma unroll
    for (int j = 0; j < R; ++j) {
      px[j].get(h[j]);
      if (res) {
        float t[8];
        pr[j].get(t);
#pragma unroll
        for (int v = 0; v < 8; ++v) h[j][v] += t[v];
      }
#pragma unroll
      for (int v = 0; v < 8; ++v) q[0] = fmaf(h[j][v], h[j][v], q[0]);
    }
    if (a.h && on) {
#pragma unroll
      for (int j = 0; j < R; ++j) store_chunk<TR, FULL>(static_cast<TR*>(a.h) + row * a.hs, h[j], at[j], cnt[j]);
    }
    team_sum<TEAM, 1>(q, red);
    float m = fmaf(q[0], inv_n, a.eps);
    if (const float f = unusual(m); f != 1.0f) {
      q[0] = 0.0f;
#pragma unroll
      for (int j = 0; j < R; ++j)
#pragma unroll
        for (int v = 0; v < 8; ++v) {
          h[j][v] *= f;
          q[0] = fmaf(h[j][v], h[j][v], q[0]);
        }
      team_sum<TEAM, 1>(q, red);
      m = fmaf(q[0], inv_n, a.eps * f * f);
    }
    const float rstd = 1.0f / sqrtf(m);
#pragma unroll
    for (int j = 0; j < R; ++j) {
      float o[8];
#pragma unroll
      for (int v = 0; v < 8; ++v) o[v] = h[j][v] * rstd * w[j][v];
      if (!a.f8) {
        if (on) store_chunk<TX, FULL>(static_cast<TX*>(a.y) + row * a.ys, o, at[j], cnt[j]);
      } else {
        if constexpr (!FULL) {   // (behind the row's end 0 r would be NaN where r is not finite)
#pragma unroll
          for (int v = 0; v < 8; ++v) o[v] = v < cnt[j] ? o[v] : 0.0f;
        }
        const float scale = scale_of(row_largest(FULL && cnt[j] <= 0 ? 0u : largest(o)));
        pu2 c = codes8(o, scale);
        if constexpr (!FULL) {
          if (cnt[j] < 8) {
            uint64_t bits = __builtin_bit_cast(uint64_t, c);
            bits = cnt[j] <= 0 ? 0 : bits & ((uint64_t(1) << (8 * cnt[j])) - 1);
            c = __builtin_bit_cast(pu2, bits);
          }
        } else {
          if (cnt[j] <= 0) c = pu2{0, 0};
        }
        if (on && at[j] < a.D16) *reinterpret_cast<pu2e*>(static_cast<uint8_t*>(a.y) + row * a.ys + at[j]) = c;
        if (on && cnt[j] > 0 && (lane & 15) == 0) a.scale[row * a.ss + at[j] / kBlock] = scale;
      }
    }
  }
}

template <typename TX, typename TR, int TEAM, int R, bool FULL>
__global__ void __launch_bounds__(TEAM < 256 ? 256 : TEAM) add_norm_bwd_kernel(AddNormArgs a) {
  constexpr int kTeams = TEAM < 256 ? 256 / TEAM : 1;
  __shared__ float red[TEAM < 256 ? 1 : TEAM / 64][2];
  const int lane = threadIdx.x % TEAM, team = threadIdx.x / TEAM;
  const float inv_n = 1.0f / static_cast<float>(a.D);
  int at[R], cnt[R];
  float w[R][8], gw[R][8] = {};
#pragma unroll
  for (int j = 0; j < R; ++j) {
    at[j] = (j * TEAM + lane) * 8;
    cnt[j] = a.D - at[j];
    Eight<float> e;
    load_chunk<float, FULL>(e, a.w, at[j], cnt[j]);
    e.get(w[j]);
  }
  const TR* hp = static_cast<const TR*>(a.h);
  const TX* dy = static_cast<const TX*>(a.dy);
  const TR* dh = static_cast<const TR*>(a.res);
  for (int64_t r0 = int64_t(blockIdx.x) * kTeams; r0 < a.T; r0 += int64_t(a.nb) * kTeams) {
    const bool on = r0 + team < a.T;
    const int64_t row = on ? r0 + team : 0;
    Eight<TR> ph[R], pd[R];
    Eight<TX> py[R];
#pragma unroll
    for (int j = 0; j < R; ++j) {
      load_chunk<TR, FULL>(ph[j], hp + row * a.hs, at[j], cnt[j]);
      load_chunk<TX, FULL>(py[j], dy + row * a.dys, at[j], cnt[j]);
      if (dh) load_chunk<TR, FULL>(pd[j], dh + row * a.rs, at[j], cnt[j]);
    }
    float h[R][8], g[R][8], q[2], f = 1.0f, m;
#pragma unroll
    for (int j = 0; j < R; ++j) {
      ph[j].get(h[j]);
      py[j].get(g[j]);
    }
#pragma clang loop unroll(disable)
    while (true) {   // (once, but for an unusual row)
      q[0] = q[1] = 0.0f;
#pragma unroll
      for (int j = 0; j < R; ++j)
#pragma unroll
        for (int v = 0; v < 8; ++v) {
          h[j][v] *= f;
          q[0] = fmaf(h[j][v], h[j][v], q[0]);
          q[1] = fmaf(g[j][v] * h[j][v], w[j][v], q[1]);
        }
      team_sum<TEAM, 2>(q, red);
      m = fmaf(q[0], inv_n, a.eps * f * f);
      if (f != 1.0f || unusual(m) == 1.0f) break;
      f = unusual(m);
    }
    const float rstd = 1.0f / sqrtf(m), slope = rstd * f;   // of f h, and of h
    const float proj = q[1] * rstd * rstd * inv_n;
#pragma unroll
    for (int j = 0; j < R; ++j) {
      float o[8], t[8] = {};
      if (dh) pd[j].get(t);
#pragma unroll
      for (int v = 0; v < 8; ++v) {
        o[v] = fmaf(slope, fmaf(-h[j][v], proj, g[j][v] * w[j][v]), t[v]);
        if (on) gw[j][v] = fmaf(g[j][v], h[j][v] * rstd, gw[j][v]);
      }
      if (on) {
        if (a.dres) store_chunk<TR, FULL>(static_cast<TR*>(a.dres) + row * a.drs, o, at[j], cnt[j]);
        if (a.dx) store_chunk<TX, FULL>(static_cast<TX*>(a.dx) + row * a.dxs, o, at[j], cnt[j]);
      }
    }
  }
  // the workgroup's sum: each team adds what the ones before it hold, the last one's goes out
  if constexpr (kTeams > 1) {
    __shared__ float sum[R * 8][TEAM];
    for (int t = 0; t < kTeams; ++t) {
      if (team == t) {
#pragma unroll
        for (int j = 0; j < R; ++j)
#pragma unroll
          for (int v = 0; v < 8; ++v) {
            if (t > 0) gw[j][v] += sum[j * 8 + v][lane];
            sum[j * 8 + v][lane] = gw[j][v];
          }
      }
      __syncthreads();
    }
  }
  if (team == kTeams - 1) {
#pragma unroll
    for (int j = 0; j < R; ++j) store_chunk<float, FULL>(a.part + int64_t(blockIdx.x) * a.D, gw[j], at[j], cnt[j]);
  }
}

// dw: the partial sums of a channel, 32 interleaved runs of them (eight loads at once), joined in a fixed order
__global__ void __launch_bounds__(1024) add_norm_reduce_kernel(AddNormArgs a) {
  __shared__ float sum[32][33];
  const int cl = threadIdx.x & 31, r = threadIdx.x >> 5;
  const int c = blockIdx.x * 32 + cl;
  float v = 0.0f;
  if (c < a.D) {
    for (int i = r; i < a.nb; i += 256) {
      float t[8];
#pragma unroll
      for (int u = 0; u < 8; ++u) t[u] = i + 32 * u < a.nb ? a.part[int64_t(i + 32 * u) * a.D + c] : 0.0f;
#pragma unroll
      for (int u = 0; u < 8; ++u) v += t[u];
    }
  }
  sum[r][cl] = v;
  __syncthreads();
  if (r == 0 && c < a.D) {
    float t = 0.0f;
#pragma unroll
    for (int i = 0; i < 32; ++i) t += sum[i][cl];
    a.dw[c] = t;
  }
}

ssm_status check_add_norm(const ssm_add_norm_params* p) {
  if (!p) return fail(SSM_ERR_NULL, "params is NULL");
  if (p->reserved != 0) return fail(SSM_ERR_UNSUPPORTED, "reserved must be 0");
  if (p->ntokens < 1 || p->dim < 1) return fail(SSM_ERR_SHAPE, "ntokens and dim must be >= 1");
  if (p->ntokens >= (int64_t(1) << 31)) return fail(SSM_ERR_SHAPE, "ntokens must be below 2^31");
  if (p->dim > kMaxDim) return fail(SSM_ERR_UNSUPPORTED, "rows of %lld channels: at most %d", (long long)p->dim, kMaxDim);
  if (p->io_dtype != SSM_F32 && p->io_dtype != SSM_BF16) return fail(SSM_ERR_DTYPE, "unknown io_dtype %d", p->io_dtype);
  if (p->res_dtype != SSM_F32 && p->res_dtype != SSM_BF16) return fail(SSM_ERR_DTYPE, "unknown res_dtype %d", p->res_dtype);
  if (p->y_dtype != p->io_dtype && p->y_dtype != SSM_E4M3)
    return fail(SSM_ERR_DTYPE, "y_dtype %d: io_dtype or SSM_E4M3", p->y_dtype);
  if (!(p->eps >= 0.0f)) return fail(SSM_ERR_UNSUPPORTED, "eps must be >= 0");
  const int64_t most = int64_t(1) << 40;
  for (int64_t s : {p->x_stride, p->residual_stride, p->h_stride, p->dy_stride, p->dh_stride, p->dx_stride, p->dresidual_stride})
    if (s != 0 && (s < p->dim || s > most)) return fail(SSM_ERR_SHAPE, "a row stride of %lld is shorter than a row of %lld",
                                                        (long long)s, (long long)p->dim);
  const int64_t yl = p->y_dtype == SSM_E4M3 ? up16(p->dim) : p->dim;
  if (p->y_stride != 0 && (p->y_stride < yl || p->y_stride > most))
    return fail(SSM_ERR_SHAPE, "y_stride %lld is shorter than a row of %lld", (long long)p->y_stride, (long long)yl);
  if (p->scale_stride != 0 && (p->scale_stride < blocks_of(p->dim) || p->scale_stride > most))
    return fail(SSM_ERR_SHAPE, "scale_stride %lld is shorter than a row of %lld", (long long)p->scale_stride,
                (long long)blocks_of(p->dim));
  return SSM_OK;
}

struct AddNormShape {
  int team, r, nb;
};

// The smallest team and number of chunks that holds a row.  One wave takes up to 1024 channels, four the rows behind: with
// 2560 channels in one wave 64 rows took 5.0 us forward and 6.3 backward, in four 3.6 and 3.9, and 8191 rows backward 70.8 and
// 63.4 (16384 rows forward 87.0 and 88.4); with 768 channels in four waves 8191 rows took 22.5 us backward, in one 16.0.
AddNormShape shape_of(const ssm_add_norm_params* p, bool bwd) {
  static const int cfgs[][2] = {{64, 1}, {64, 2}, {256, 1}, {256, 2}, {256, 4}, {1024, 2}};
  AddNormShape s{};
  for (const auto& c : cfgs)
    if (int64_t(c[0]) * c[1] * 8 >= up16(p->dim)) {
      s.team = c[0];
      s.r = c[1];
      break;
    }
  const int64_t waves = s.team < 256 ? 4 : s.team / 64;
  // 16 waves for each SIMD in the forward (16384 rows of 2560: 87 us, with two for each SIMD 90); in the backward, whose
  // partial sums grow with the workgroups, two workgroups of four waves to a CU or one of 16 (8001 rows of 1001 23.4 us, twice as
  // many 27.1; 2000 rows of 16384 112 us, half as many 143)
  int64_t nb = bwd ? (s.team == 1024 ? 256 : 512) : 16384 / waves;
  const int64_t teams = s.team < 256 ? 256 / s.team : 1, rows = (p->ntokens + teams - 1) / teams;
  s.nb = static_cast<int>(nb > rows ? rows : nb);
  return s;
}

template <typename TX, typename TR, bool FULL, bool BWD>
void launch_shape(const AddNormArgs& a, const AddNormShape& s, hipStream_t st) {
  const dim3 grid(a.nb), block(s.team < 256 ? 256 : s.team);
#define SSM57_CFG(TEAM, R)                                                                                          \
  if (s.team == TEAM && s.r == R) {                                                                                 \
    if constexpr (BWD) hipLaunchKernelGGL((add_norm_bwd_kernel<TX, TR, TEAM, R, FULL>), grid, block, 0, st, a);     \
    else hipLaunchKernelGGL((add_norm_fwd_kernel<TX, TR, TEAM, R, FULL>), grid, block, 0, st, a);                   \
  }
  SSM57_CFG(64, 1)
  SSM57_CFG(64, 2)
  SSM57_CFG(256, 1)
  SSM57_CFG(256, 2)
  SSM57_CFG(256, 4)
  SSM57_CFG(1024, 2)
#undef SSM57_CFG
}

template <bool BWD>
ssm_status dispatch_add_norm(const ssm_add_norm_params* p, AddNormArgs& a, hipStream_t st) {
  const AddNormShape s = shape_of(p, BWD);
  a.nb = s.nb;
  const bool xb = p->io_dtype == SSM_BF16, rb = p->res_dtype == SSM_BF16, full = a.D % 8 == 0;
  auto go = [&](auto tx, auto tr) {
    using TX = decltype(tx);
    using TR = decltype(tr);
    if (full) launch_shape<TX, TR, true, BWD>(a, s, st);
    else launch_shape<TX, TR, false, BWD>(a, s, st);
  };
  if (xb && rb) go(uint16_t{}, uint16_t{});
  else if (xb) go(uint16_t{}, float{});
  else if (rb) go(float{}, uint16_t{});
  else go(float{}, float{});
  if constexpr (BWD) hipLaunchKernelGGL(add_norm_reduce_kernel, dim3((a.D + 31) / 32), dim3(1024), 0, st, a);
  const hipError_t e = hipGetLastError();
  return e == hipSuccess ? SSM_OK : fail(SSM_ERR_HIP, "add norm launch: %s", hipGetErrorString(e));
}

AddNormArgs add_norm_args(const ssm_add_norm_params* p) {
  AddNormArgs a{};
  a.T = static_cast<int>(p->ntokens);
  a.D = static_cast<int>(p->dim);
  a.D16 = static_cast<int>(up16(p->dim));
  a.eps = p->eps;
  a.f8 = p->y_dtype == SSM_E4M3;
  auto row = [&](int64_t s) { return s ? s : p->dim; };
  a.xs = row(p->x_stride);
  a.hs = row(p->h_stride);
  a.dys = row(p->dy_stride);
  a.dxs = row(p->dx_stride);
  a.drs = row(p->dresidual_stride);
  a.ys = p->y_stride ? p->y_stride : a.f8 ? a.D16 : p->dim;
  a.ss = p->scale_stride ? p->scale_stride : blocks_of(p->dim);
  return a;
}

}  // namespace
}  // namespace ssm57

using namespace ssm57;

extern "C" ssm_status ssm_add_norm_fwd(const ssm_add_norm_params* p, const void* x, const void* residual,
                                       const float* weight, void* residual_out, void* y, float* y_scale, void* stream) {
  g_err[0] = 0;
  if (ssm_status s = check_add_norm(p); s != SSM_OK) return s;
  if (!x || !weight || !y) return fail(SSM_ERR_NULL, "x, weight and y are required");
  const bool f8 = p->y_dtype == SSM_E4M3;
  if (f8 != (y_scale != nullptr)) return fail(SSM_ERR_NULL, "y_scale is required with an 8-bit y and must be NULL without");
  const int es = p->io_dtype == SSM_BF16 ? 2 : 4, rs = p->res_dtype == SSM_BF16 ? 2 : 4;
  if (!aligned(x, es) || !aligned(residual, rs) || !aligned(residual_out, rs) || !aligned(weight, 4) || !aligned(y_scale, 4))
    return fail(SSM_ERR_ALIGN, "a pointer is not aligned to its element size");
  if (!aligned(y, f8 ? 8 : es) || (f8 && p->y_stride % 8))
    return fail(SSM_ERR_ALIGN, "y: rows must be aligned to %d bytes", f8 ? 8 : es);
  AddNormArgs a = add_norm_args(p);
  a.x = x;
  a.res = residual;
  a.rs = p->residual_stride ? p->residual_stride : p->dim;
  a.w = weight;
  a.h = residual_out;
  a.y = y;
  a.scale = y_scale;
  return dispatch_add_norm<false>(p, a, static_cast<hipStream_t>(stream));
}

extern "C" size_t ssm_add_norm_bwd_workspace_bytes(const ssm_add_norm_params* p) {
  if (check_add_norm(p) != SSM_OK) return 0;
  return size_t(shape_of(p, true).nb) * p->dim * 4;
}

extern "C" ssm_status ssm_add_norm_bwd(const ssm_add_norm_params* p, const void* h, const float* weight, const void* dy,
                                       const void* dh, void* dx, void* dresidual, float* dweight, void* workspace,
                                       size_t workspace_bytes, void* stream) {
  g_err[0] = 0;
  if (ssm_status s = check_add_norm(p); s != SSM_OK) return s;
  if (!h || !weight || !dy || !dweight || (!dx && !dresidual))
    return fail(SSM_ERR_NULL, "h, weight, dy, dweight and one of dx and dresidual are required");
  const int es = p->io_dtype == SSM_BF16 ? 2 : 4, rs = p->res_dtype == SSM_BF16 ? 2 : 4;
  if (!aligned(h, rs) || !aligned(dh, rs) || !aligned(dresidual, rs) || !aligned(dy, es) || !aligned(dx, es) ||
      !aligned(weight, 4) || !aligned(dweight, 4))
    return fail(SSM_ERR_ALIGN, "a pointer is not aligned to its element size");
  const size_t need = size_t(shape_of(p, true).nb) * p->dim * 4;
  if (!workspace || workspace_bytes < need || !aligned(workspace, 4))
    return fail(SSM_ERR_WORKSPACE, "workspace of %zu bytes needed, got %zu at %p", need, workspace_bytes, workspace);
  AddNormArgs a = add_norm_args(p);
  a.h = const_cast<void*>(h);
  a.res = dh;
  a.rs = p->dh_stride ? p->dh_stride : p->dim;
  a.w = weight;
  a.dy = dy;
  a.dx = dx;
  a.dres = dresidual;
  a.part = static_cast<float*>(workspace);
  a.dw = dweight;
  return dispatch_add_norm<true>(p, a, static_cast<hipStream_t>(stream));
}
