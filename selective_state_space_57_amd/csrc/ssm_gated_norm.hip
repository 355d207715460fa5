// Group norm of the Mamba-2 block's output, channels last, with its SiLU gate, forward and backward.  Each row (token)
// of dim channels is cut into ngroups groups of n channels with statistics of their own:
//   gate first:  h = x silu(z), y = (h - m) r w + b;   gate behind:  h = x, y = ((h - m) r w + b) silu(z)
//   r = 1 / sqrt(mean((h - m)^2) + eps),  m = mean(h) with `center`, else 0 (root mean square norm)
// Backward, with dn = (dL/d line) w and nh = (h - m) r:  dh = r (dn - nh mean(dn nh) [- mean(dn) with center]).
//
// Bound by memory: x, z (and dy) are read once and y (dx, dz) written once.  A team of lanes (one wave, a workgroup of
// 4 waves, or one of 16) holds a whole group of a row in registers, so nothing is read twice and nothing but the sums
// goes through LDS.  That holds up to groups of 8192 channels (4096 where rows are not 16-byte aligned).  Above, the
// workgroup of 16 waves has 128 registers a lane: enough for the forward (its form for unaligned rows spills up to 12), but
// not for the backward, which spills 62 to 140 with a gate (212 to 372 bytes a lane; up to 175 for unaligned rows) and goes
// through scratch memory for them.  A workgroup keeps its group and walks down the rows, so weight and bias are read once per
// workgroup, and the backward's weight gradient adds up in registers; the workgroups' partial sums are joined in a fixed
// order by a second kernel.  The team is the smallest that holds the group at the given number of chunks per lane.
// Measured with gate, bf16, rows of 5120: 16384 rows in one group 90 us (5.6 TB/s), gradients of 8191 rows in 8 groups
// 89 us (4.7 TB/s; 106 with a partial sum for each team instead of each workgroup).  Gradients of 420 MB of gated rows in
// one group: 5120 channels of fp32 111 us, 10240 and 16384 of bf16 385 and 299 us (1.1 and 1.4 TB/s), 16384 of fp32 202 us.
#include "packed.hpp"

namespace ssm57 {
namespace {

constexpr int kMaxGroup = 16384;

struct NormArgs {
  const void* x;
  const void* z;
  const float* w;
  const float* b;
  void* y;
  const void* dy;
  void* dx;
  void* dz;
  float* part;     // [parts][2][dim]: partial sums of dw and dbias
  float* dw;
  float* dbias;
  int64_t xs, zs, ys, dys, dxs, dzs;
  int T, D, G, n, nb;
  float eps;
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

// GATE: 0 none, 1 before the norm, 2 behind it
template <typename T, int V, int TEAM, int R, int GATE, bool CENTER, bool BWD>
__global__ void __launch_bounds__(TEAM < 256 ? 256 : TEAM) gated_norm_kernel(NormArgs a) {
  constexpr int kTeams = TEAM < 256 ? 256 / TEAM : 1;
  constexpr int kWaves = TEAM < 256 ? 1 : TEAM / 64;
  __shared__ float red1[kWaves][1], red2[kWaves][2];
  const int lane = threadIdx.x % TEAM, team = threadIdx.x / TEAM;
  const int g = blockIdx.x % a.G, blk = blockIdx.x / a.G;
  const int c0 = g * a.n;
  const float inv = 1.0f / static_cast<float>(a.n);
  // a lane's chunk j starts at channel (j TEAM + lane) V of the group; one past its end reads the last, times zero
  int at[R];
  bool live[R];
#pragma unroll
  for (int j = 0; j < R; ++j) {
    const int e = (j * TEAM + lane) * V;
    live[j] = e < a.n;
    at[j] = c0 + (live[j] ? e : a.n - V);
  }
  float w[R][V], b[R][V];
#pragma unroll
  for (int j = 0; j < R; ++j) {
    load_floats<V>(a.w + at[j], w[j]);
#pragma unroll
    for (int v = 0; v < V; ++v) b[j][v] = 0.0f;
    if (a.b) load_floats<V>(a.b + at[j], b[j]);
  }
  float gw[BWD ? R : 1][V] = {}, gb[BWD ? R : 1][V] = {};
  const T* x = static_cast<const T*>(a.x);
  const T* z = static_cast<const T*>(a.z);
  const T* dy = static_cast<const T*>(a.dy);
  // (the teams of a workgroup run the same number of turns: a row past the end is computed as row 0 and not stored)
  for (int64_t r0 = int64_t(blk) * kTeams; r0 < a.T; r0 += int64_t(a.nb) * kTeams) {
    const bool on = r0 + team < a.T;
    const int64_t row = on ? r0 + team : 0;
    Pack<T, V> px[R], pz[GATE ? R : 1], pd[BWD ? R : 1];
#pragma unroll
    for (int j = 0; j < R; ++j) {
      px[j].load(x + row * a.xs + at[j]);
      if constexpr (GATE != 0) pz[j].load(z + row * a.zs + at[j]);
      if constexpr (BWD) pd[j].load(dy + row * a.dys + at[j]);
    }
    float h[R][V];
    float s1[1] = {0.0f};
#pragma unroll
    for (int j = 0; j < R; ++j) {
      px[j].get(h[j]);
      if constexpr (GATE == 1) {
        float zz[V];
        pz[j].get(zz);
#pragma unroll
        for (int v = 0; v < V; ++v) h[j][v] *= zz[v] * sigmoid(zz[v]);
      }
      if constexpr (CENTER) {
        float t = 0.0f;
#pragma unroll
        for (int v = 0; v < V; ++v) t += h[j][v];
        s1[0] += live[j] ? t : 0.0f;
      }
    }
    if constexpr (CENTER) {
      team_sum<TEAM, 1>(s1, red1);
      const float mean = s1[0] * inv;
#pragma unroll
      for (int j = 0; j < R; ++j)
#pragma unroll
        for (int v = 0; v < V; ++v) h[j][v] -= mean;
    }
    if constexpr (!BWD) {
      float q[1] = {0.0f};
#pragma unroll
      for (int j = 0; j < R; ++j) {
        float t = 0.0f;
#pragma unroll
        for (int v = 0; v < V; ++v) t = fmaf(h[j][v], h[j][v], t);
        q[0] += live[j] ? t : 0.0f;
      }
      team_sum<TEAM, 1>(q, red1);
      const float rstd = 1.0f / sqrtf(fmaf(q[0], inv, a.eps));
#pragma unroll
      for (int j = 0; j < R; ++j) {
        float o[V];
#pragma unroll
        for (int v = 0; v < V; ++v) o[v] = fmaf(h[j][v] * rstd, w[j][v], b[j][v]);
        if constexpr (GATE == 2) {
          float zz[V];
          pz[j].get(zz);
#pragma unroll
          for (int v = 0; v < V; ++v) o[v] *= zz[v] * sigmoid(zz[v]);
        }
        if (live[j] && on) Pack<T, V>::store(static_cast<T*>(a.y) + row * a.ys + at[j], o);
      }
    } else {
      // q = (sum h^2, sum dn h); with center also sum dn
      float q[2] = {0.0f, 0.0f}, sd[1] = {0.0f};
      float dl[R][V];   // dL / d line
#pragma unroll
      for (int j = 0; j < R; ++j) {
        pd[j].get(dl[j]);
        if constexpr (GATE == 2) {
          float zz[V];
          pz[j].get(zz);
#pragma unroll
          for (int v = 0; v < V; ++v) dl[j][v] *= zz[v] * sigmoid(zz[v]);
        }
        float t0 = 0.0f, t1 = 0.0f, t2 = 0.0f;
#pragma unroll
        for (int v = 0; v < V; ++v) {
          t0 = fmaf(h[j][v], h[j][v], t0);
          const float dn = dl[j][v] * w[j][v];
          t1 = fmaf(dn, h[j][v], t1);
          t2 += dn;
        }
        q[0] += live[j] ? t0 : 0.0f;
        q[1] += live[j] ? t1 : 0.0f;
        if constexpr (CENTER) sd[0] += live[j] ? t2 : 0.0f;
      }
      team_sum<TEAM, 2>(q, red2);
      if constexpr (CENTER) team_sum<TEAM, 1>(sd, red1);
      const float rstd = 1.0f / sqrtf(fmaf(q[0], inv, a.eps));
      const float proj = q[1] * rstd * rstd * inv;   // mean(dn nh) r
      const float md = CENTER ? sd[0] * inv : 0.0f;
#pragma unroll
      for (int j = 0; j < R; ++j) {
        float xx[V], zz[V], ox[V], oz[V];
        px[j].get(xx);
        if constexpr (GATE != 0) pz[j].get(zz);
#pragma unroll
        for (int v = 0; v < V; ++v) {
          const float nh = h[j][v] * rstd;
          const float dh = rstd * (dl[j][v] * w[j][v] - h[j][v] * proj - md);
          if (on) {
            gw[j][v] = fmaf(dl[j][v], nh, gw[j][v]);
            gb[j][v] += dl[j][v];
          }
          if constexpr (GATE != 0) {
            const float sg = sigmoid(zz[v]);
            const float slope = sg * fmaf(zz[v], 1.0f - sg, 1.0f);
            if constexpr (GATE == 1) {
              ox[v] = dh * zz[v] * sg;
              oz[v] = dh * xx[v] * slope;
            } else {
              ox[v] = dh;
              oz[v] = fmaf(nh, w[j][v], b[j][v]) * slope;
            }
          } else {
            ox[v] = dh;
          }
        }
        if constexpr (GATE == 2) {
          float dd[V];
          pd[j].get(dd);
#pragma unroll
          for (int v = 0; v < V; ++v) oz[v] *= dd[v];
        }
        if (live[j] && on) {
          Pack<T, V>::store(static_cast<T*>(a.dx) + row * a.dxs + at[j], ox);
          if constexpr (GATE != 0) Pack<T, V>::store(static_cast<T*>(a.dz) + row * a.dzs + at[j], oz);
        }
      }
    }
  }
  if constexpr (BWD) {
    // the workgroup's sum: each team adds what the ones before it hold, the last one's goes out
    if constexpr (kTeams > 1) {
      __shared__ float sum[2 * R * V][TEAM];
      for (int t = 0; t < kTeams; ++t) {
        if (team == t) {
#pragma unroll
          for (int j = 0; j < R; ++j)
#pragma unroll
            for (int v = 0; v < V; ++v) {
              if (t > 0) {
                gw[j][v] += sum[2 * (j * V + v)][lane];
                gb[j][v] += sum[2 * (j * V + v) + 1][lane];
              }
              sum[2 * (j * V + v)][lane] = gw[j][v];
              sum[2 * (j * V + v) + 1][lane] = gb[j][v];
            }
        }
        __syncthreads();
      }
    }
    float* part = a.part + int64_t(blk) * 2 * a.D;
    if (team == kTeams - 1) {
#pragma unroll
      for (int j = 0; j < R; ++j)
        if (live[j]) {
#pragma unroll
          for (int v = 0; v < V; ++v) {
            part[at[j] + v] = gw[j][v];
            if (a.dbias) part[a.D + at[j] + v] = gb[j][v];
          }
        }
    }
  }
}

// dw and dbias: the partial sums of a channel, 16 interleaved runs, joined in a fixed order
__global__ void __launch_bounds__(256) gated_norm_reduce_kernel(NormArgs a, int parts) {
  __shared__ float sum[16][17];
  const int cl = threadIdx.x & 15, r = threadIdx.x >> 4;
  const int c = blockIdx.x * 16 + cl;
  float v = 0.0f;
  if (c < a.D)
    for (int i = r; i < parts; i += 16) v += a.part[(int64_t(i) * 2 + blockIdx.y) * a.D + c];
  sum[r][cl] = v;
  __syncthreads();
  if (r == 0 && c < a.D) {
    float t = 0.0f;
    for (int i = 0; i < 16; ++i) t += sum[i][cl];
    float* out = blockIdx.y == 0 ? a.dw : a.dbias;
    if (out) out[c] = t;
  }
}

ssm_status check_norm(const ssm_gated_norm_params* p) {
  if (!p) return fail(SSM_ERR_NULL, "params is NULL");
  if (p->reserved != 0) return fail(SSM_ERR_UNSUPPORTED, "reserved must be 0");
  if (p->ntokens < 1 || p->dim < 1 || p->ngroups < 1)
    return fail(SSM_ERR_SHAPE, "ntokens, dim and ngroups must be >= 1");
  if (p->ntokens >= (int64_t(1) << 31) || p->dim >= (int64_t(1) << 24))
    return fail(SSM_ERR_SHAPE, "ntokens must be below 2^31 and dim below 2^24");
  if (p->dim % p->ngroups) return fail(SSM_ERR_SHAPE, "dim (%lld) must be a multiple of ngroups (%lld)",
                                       (long long)p->dim, (long long)p->ngroups);
  if (p->dim / p->ngroups > kMaxGroup)
    return fail(SSM_ERR_UNSUPPORTED, "a group of %lld channels: at most %d", (long long)(p->dim / p->ngroups), kMaxGroup);
  if (p->io_dtype != SSM_F32 && p->io_dtype != SSM_BF16) return fail(SSM_ERR_DTYPE, "unknown io_dtype %d", p->io_dtype);
  if ((p->gate_first != 0 && p->gate_first != 1) || (p->center != 0 && p->center != 1))
    return fail(SSM_ERR_UNSUPPORTED, "gate_first and center must be 0 or 1");
  if (!(p->eps >= 0.0f)) return fail(SSM_ERR_UNSUPPORTED, "eps must be >= 0");
  const int64_t most = int64_t(1) << 40;
  for (int64_t s : {p->x_stride, p->z_stride, p->y_stride, p->dy_stride, p->dx_stride, p->dz_stride})
    if (s != 0 && (s < p->dim || s > most)) return fail(SSM_ERR_SHAPE, "a row stride of %lld is shorter than a row of %lld",
                                                        (long long)s, (long long)p->dim);
  return SSM_OK;
}

struct NormShape {
  int v, team, r;
  int nb;      // workgroups per group
};

// The smallest team and number of chunks that holds a group of n channels.
NormShape shape_of(const ssm_gated_norm_params* p, bool vec, bool bwd) {
  struct Cfg { int v, team, r; };
  static const Cfg cfgs[] = {{8, 64, 1}, {8, 64, 2}, {8, 64, 4}, {8, 256, 2}, {8, 256, 3}, {8, 256, 4}, {8, 1024, 2},
                             {4, 64, 1}, {4, 64, 2}, {4, 64, 4}, {4, 256, 2}, {4, 256, 4}, {4, 256, 8}, {4, 1024, 4},
                             {1, 64, 1}, {1, 64, 4}, {1, 256, 4}, {1, 256, 16}, {1, 1024, 16}};
  const int v = vec ? (p->io_dtype == SSM_BF16 ? 8 : 4) : 1;
  const int64_t n = p->dim / p->ngroups;
  NormShape s{};
  for (const Cfg& c : cfgs)
    if (c.v == v && int64_t(c.v) * c.team * c.r >= n) {
      s.v = c.v;
      s.team = c.team;
      s.r = c.r;
      break;
    }
  // about 16 waves for each SIMD in the forward (16384 rows of 5120: 91 us; 8: 94), 2 in the backward, whose partial sums
  // grow with the workgroups (8191 rows of 5120 in 8 groups: 90 us; 4: 93, 8: 101)
  const int64_t waves = s.team < 256 ? 4 : s.team / 64;
  const int64_t want = (bwd ? 2048 : 16384) / waves;
  int64_t nb = (want + p->ngroups - 1) / p->ngroups;
  const int64_t teams = s.team < 256 ? 256 / s.team : 1, rows = (p->ntokens + teams - 1) / teams;
  if (nb > rows) nb = rows;
  s.nb = static_cast<int>(nb < 1 ? 1 : nb);
  return s;
}

template <typename T, int V, int TEAM, int R, bool BWD>
void launch_norm(const NormArgs& a, bool gate, bool first, bool center, hipStream_t st) {
  const dim3 grid(static_cast<uint32_t>(a.nb) * a.G), block(TEAM < 256 ? 256 : TEAM);
#define SSM57_NORM(GATE, CENTER) \
  hipLaunchKernelGGL((gated_norm_kernel<T, V, TEAM, R, GATE, CENTER, BWD>), grid, block, 0, st, a)
  if (!gate) { if (center) SSM57_NORM(0, true); else SSM57_NORM(0, false); }
  else if (first) { if (center) SSM57_NORM(1, true); else SSM57_NORM(1, false); }
  else { if (center) SSM57_NORM(2, true); else SSM57_NORM(2, false); }
#undef SSM57_NORM
}

template <bool BWD>
ssm_status dispatch_norm(const ssm_gated_norm_params* p, NormArgs& a, bool vec, hipStream_t st) {
  const NormShape s = shape_of(p, vec, BWD);
  a.nb = s.nb;
  const bool gate = a.z != nullptr, first = p->gate_first, center = p->center;
#define SSM57_CFG(T, V, TEAM, R) \
  if (s.v == V && s.team == TEAM && s.r == R) launch_norm<T, V, TEAM, R, BWD>(a, gate, first, center, st)
  if (p->io_dtype == SSM_BF16) {
    SSM57_CFG(uint16_t, 8, 64, 1);
    SSM57_CFG(uint16_t, 8, 64, 2);
    SSM57_CFG(uint16_t, 8, 64, 4);
    SSM57_CFG(uint16_t, 8, 256, 2);
    SSM57_CFG(uint16_t, 8, 256, 3);
    SSM57_CFG(uint16_t, 8, 256, 4);
    SSM57_CFG(uint16_t, 8, 1024, 2);
    SSM57_CFG(uint16_t, 1, 64, 1);
    SSM57_CFG(uint16_t, 1, 64, 4);
    SSM57_CFG(uint16_t, 1, 256, 4);
    SSM57_CFG(uint16_t, 1, 256, 16);
    SSM57_CFG(uint16_t, 1, 1024, 16);
  } else {
    SSM57_CFG(float, 4, 64, 1);
    SSM57_CFG(float, 4, 64, 2);
    SSM57_CFG(float, 4, 64, 4);
    SSM57_CFG(float, 4, 256, 2);
    SSM57_CFG(float, 4, 256, 4);
    SSM57_CFG(float, 4, 256, 8);
    SSM57_CFG(float, 4, 1024, 4);
    SSM57_CFG(float, 1, 64, 1);
    SSM57_CFG(float, 1, 64, 4);
    SSM57_CFG(float, 1, 256, 4);
    SSM57_CFG(float, 1, 256, 16);
    SSM57_CFG(float, 1, 1024, 16);
  }
#undef SSM57_CFG
  if constexpr (BWD)
    hipLaunchKernelGGL(gated_norm_reduce_kernel, dim3((a.D + 15) / 16, a.dbias ? 2 : 1), dim3(256), 0, st, a, s.nb);
  const hipError_t e = hipGetLastError();
  return e == hipSuccess ? SSM_OK : fail(SSM_ERR_HIP, "gated norm launch: %s", hipGetErrorString(e));
}

NormArgs norm_args(const ssm_gated_norm_params* p) {
  NormArgs a{};
  a.T = static_cast<int>(p->ntokens);
  a.D = static_cast<int>(p->dim);
  a.G = static_cast<int>(p->ngroups);
  a.n = a.D / a.G;
  a.eps = p->eps;
  auto row = [&](int64_t s) { return s ? s : p->dim; };
  a.xs = row(p->x_stride);
  a.zs = row(p->z_stride);
  a.ys = row(p->y_stride);
  a.dys = row(p->dy_stride);
  a.dxs = row(p->dx_stride);
  a.dzs = row(p->dz_stride);
  return a;
}

bool norm_rows(const void* ptr, int64_t stride, int64_t n, int es) {
  const int64_t v = 16 / es;
  return aligned(ptr, 16) && stride % v == 0 && n % v == 0;
}

// (the vector and the scalar form have different numbers of partial sums: the larger)
size_t norm_workspace(const ssm_gated_norm_params* p) {
  size_t most = 0;
  for (bool vec : {false, true}) {
    const int64_t v = vec ? (p->io_dtype == SSM_BF16 ? 8 : 4) : 1;
    if ((p->dim / p->ngroups) % v) continue;
    const NormShape s = shape_of(p, vec, true);
    const size_t need = size_t(s.nb) * 2 * p->dim * 4;
    most = need > most ? need : most;
  }
  return most;
}

}  // namespace
}  // namespace ssm57

using namespace ssm57;

extern "C" ssm_status ssm_gated_norm_fwd(const ssm_gated_norm_params* p, const void* x, const void* z,
                                         const float* weight, const float* bias, void* y, void* stream) {
  g_err[0] = 0;
  if (ssm_status s = check_norm(p); s != SSM_OK) return s;
  if (!x || !weight || !y) return fail(SSM_ERR_NULL, "x, weight and y are required");
  const int es = p->io_dtype == SSM_BF16 ? 2 : 4;
  if (!aligned(x, es) || !aligned(z, es) || !aligned(y, es) || !aligned(weight, 4) || !aligned(bias, 4))
    return fail(SSM_ERR_ALIGN, "a pointer is not aligned to its element size");
  NormArgs a = norm_args(p);
  a.x = x;
  a.z = z;
  a.w = weight;
  a.b = bias;
  a.y = y;
  const bool vec = norm_rows(x, a.xs, a.n, es) && norm_rows(y, a.ys, a.n, es) && (!z || norm_rows(z, a.zs, a.n, es));
  return dispatch_norm<false>(p, a, vec, static_cast<hipStream_t>(stream));
}

extern "C" size_t ssm_gated_norm_bwd_workspace_bytes(const ssm_gated_norm_params* p) {
  return check_norm(p) == SSM_OK ? norm_workspace(p) : 0;
}

extern "C" ssm_status ssm_gated_norm_bwd(const ssm_gated_norm_params* p, const void* x, const void* z,
                                         const float* weight, const float* bias, const void* dy, void* dx, void* dz,
                                         float* dweight, float* dbias, void* workspace, size_t workspace_bytes,
                                         void* stream) {
  g_err[0] = 0;
  if (ssm_status s = check_norm(p); s != SSM_OK) return s;
  if (!x || !weight || !dy || !dx || !dweight) return fail(SSM_ERR_NULL, "x, weight, dy, dx and dweight are required");
  if ((z == nullptr) != (dz == nullptr)) return fail(SSM_ERR_NULL, "dz is required with z and must be NULL without it");
  const int es = p->io_dtype == SSM_BF16 ? 2 : 4;
  if (!aligned(x, es) || !aligned(z, es) || !aligned(dy, es) || !aligned(dx, es) || !aligned(dz, es) ||
      !aligned(weight, 4) || !aligned(bias, 4) || !aligned(dweight, 4) || !aligned(dbias, 4))
    return fail(SSM_ERR_ALIGN, "a pointer is not aligned to its element size");
  const size_t need = norm_workspace(p);
  if (!workspace || workspace_bytes < need || !aligned(workspace, 4))
    return fail(SSM_ERR_WORKSPACE, "workspace of %zu bytes needed, got %zu at %p", need, workspace_bytes, workspace);
  NormArgs a = norm_args(p);
  a.x = x;
  a.z = z;
  a.w = weight;
  a.b = bias;
  a.dy = dy;
  a.dx = dx;
  a.dz = dz;
  a.part = static_cast<float*>(workspace);
  a.dw = dweight;
  a.dbias = dbias;
  const bool vec = norm_rows(x, a.xs, a.n, es) && norm_rows(dy, a.dys, a.n, es) && norm_rows(dx, a.dxs, a.n, es) &&
                   (!z || (norm_rows(z, a.zs, a.n, es) && norm_rows(dz, a.dzs, a.n, es)));
  return dispatch_norm<true>(p, a, vec, static_cast<hipStream_t>(stream));
}
