// The causal depthwise convolution (+ SiLU) of the Mamba-2 block over packed sequences, channels last: rows are tokens
// (any row stride), sequences lie one behind the other (cu_seqlens), and the window of the width - 1 inputs before a
// sequence lives in a slot of a state pool.  Prompts, single tokens, and the backward pass:
//   pre_t = bias + sum_k w[k] x_{t-(K-1)+k} (within the sequence; the window, or zeros, before it),  u_t = silu(pre_t)
//   dpre_t = du_t silu'(pre_t);  dx_t = sum_j w[K-1-j] dpre_{t+j};  dw[k] = sum_t dpre_t x_{t-(K-1)+k};
//   dbias = sum_t dpre_t
// All of it is a stream of x (and du) in and u (dx) out, bound by memory: a thread owns V channels (16 bytes of a row)
// and walks down a tile of tokens with the K - 1 inputs before it in registers, so each value is read once and a halo
// of K - 1 rows per tile (out of the L2) on top.  At 4.3 TB/s forward (16384 tokens of 5376 bf16 channels: 81 us).  The
// backward takes 87 us for 8191 tokens (3.0 TB/s): neither memory nor its arithmetic (280 instructions for a wave's row of
// 512 channels, VALU 56 % of the cycles) is full; at 194 registers a lane two waves share a SIMD, and latency shows.  In
// fp32 (114 registers) it reaches 3.9 TB/s, the forward 4.4.
#include <algorithm>

#include "packed.hpp"

namespace ssm57 {
namespace {

constexpr int kThreads = 256, kBwdThreads = 64;

struct PConvArgs {
  const void* x;
  const float* w;
  const float* bias;
  const int32_t* cu;
  const float* state;
  const int32_t* idx;
  const uint8_t* has;
  float* state_out;
  void* u;
  const void* du;
  const float* dstate_out;
  void* dx;
  float* part;     // [tiles][K + 1][C]: partial sums of dw[0..K-1] and dbias
  float* dw;
  float* dbias;
  float* dstate;
  int64_t xs, us, dus, dxs, nslots;
  int T, S, C, tile, ntiles, silu;
};

// one channel vector's taps and bias
template <int K, int V>
struct Taps {
  float w[K][V], b[V];
  __device__ __forceinline__ void load(const PConvArgs& a, int c) {
    float t[V * K];
    load_floats<V * K>(a.w + int64_t(c) * K, t);
#pragma unroll
    for (int v = 0; v < V; ++v) {
#pragma unroll
      for (int k = 0; k < K; ++k) w[k][v] = t[v * K + k];
      b[v] = 0.0f;
    }
    if (a.bias) load_floats<V>(a.bias + c, b);
  }
};

// a slot's window of V channels from channel c on, oldest input first
template <int K, int V>
__device__ __forceinline__ void get_window(const float* p, float (&win)[K][V]) {
  if constexpr (K > 1) {
    float t[V * (K - 1)];
    load_floats<V * (K - 1)>(p, t);
#pragma unroll
    for (int v = 0; v < V; ++v)
#pragma unroll
      for (int k = 0; k < K - 1; ++k) win[k][v] = t[v * (K - 1) + k];
  }
}
// win[first] .. win[first + K - 2]
template <int K, int V>
__device__ __forceinline__ void put_window(float* p, const float (&win)[K][V], int first) {
  if constexpr (K > 1) {
    float t[V * (K - 1)];
#pragma unroll
    for (int v = 0; v < V; ++v)
#pragma unroll
      for (int k = 0; k < K - 1; ++k) t[v * (K - 1) + k] = first ? win[k + 1][v] : win[k][v];
    store_floats<V * (K - 1)>(p, t);
  }
}
// window of sequence s before its first token: the slot's, or zeros
template <int K, int V>
__device__ __forceinline__ void load_window(const PConvArgs& a, int s, int c, float (&win)[K][V]) {
  const int64_t slot = a.state && (!a.has || a.has[s]) ? slot_of(a.idx, s, a.nslots) : -1;
#pragma unroll
  for (int k = 0; k < K - 1; ++k)
#pragma unroll
    for (int v = 0; v < V; ++v) win[k][v] = 0.0f;
  if (slot >= 0) get_window<K, V>(a.state + (slot * a.C + c) * (K - 1), win);
}

template <int K, int V>
__device__ __forceinline__ void conv_pre(const Taps<K, V>& tp, const float (&win)[K][V], float (&pre)[V]) {
#pragma unroll
  for (int v = 0; v < V; ++v) {
    pre[v] = tp.b[v];
#pragma unroll
    for (int k = 0; k < K; ++k) pre[v] = fmaf(tp.w[k][v], win[k][v], pre[v]);
  }
}
template <int K, int V>
__device__ __forceinline__ void shift(float (&win)[K][V]) {
#pragma unroll
  for (int k = 0; k + 1 < K; ++k)
#pragma unroll
    for (int v = 0; v < V; ++v) win[k][v] = win[k + 1][v];
}
// d act / d pre (SiLU: s (1 + pre (1 - s)), s = sigmoid(pre))
__device__ __forceinline__ float slope(float pre, int silu) {
  if (!silu) return 1.0f;
  const float s = sigmoid(pre);
  return s * fmaf(pre, 1.0f - s, 1.0f);
}

// Blocks below ntiles each take a tile of tokens and leave out the first K - 1 of every sequence; block ntiles + s takes
// those of sequence s, which alone depend on the window, and then writes the sequence's last window.  So a slot is
// read and written by the same thread, and the window can be updated in place without a second launch.
template <typename T, int V, int K>
__global__ void __launch_bounds__(kThreads) packed_conv_fwd_kernel(PConvArgs a) {
  const int c = (blockIdx.y * kThreads + threadIdx.x) * V;
  if (c >= a.C) return;
  const T* x = static_cast<const T*>(a.x) + c;
  T* u = static_cast<T*>(a.u) + c;
  Taps<K, V> tp;
  tp.load(a, c);
  float win[K][V], pre[V];
  auto emit = [&](int t) __attribute__((always_inline)) {
    conv_pre<K, V>(tp, win, pre);
    if (a.silu) {
#pragma unroll
      for (int v = 0; v < V; ++v) pre[v] *= sigmoid(pre[v]);
    }
    Pack<T, V>::store(u + int64_t(t) * a.us, pre);
  };
  if (static_cast<int>(blockIdx.x) >= a.ntiles) {
    const int s = blockIdx.x - a.ntiles;
    int begin, end;
    seq_range(a.cu, s, a.T, begin, end);
    load_window<K, V>(a, s, c, win);
    const int first = min(begin + K - 1, end);
    for (int t = begin; t < first; ++t) {
      Pack<T, V> p;
      p.load(x + int64_t(t) * a.xs);
      p.get(win[K - 1]);
      emit(t);
      shift<K, V>(win);
    }
    if (K > 1 && a.state_out) {
      const int64_t slot = slot_of(a.idx, s, a.nslots);
      if (slot >= 0) {
        if (end - begin > K - 1) {   // (otherwise win holds the last inputs already)
#pragma unroll
          for (int k = 0; k < K - 1; ++k) {
            Pack<T, V> p;
            p.load(x + int64_t(end - (K - 1) + k) * a.xs);
            p.get(win[k]);
          }
        }
        put_window<K, V>(a.state_out + (slot * a.C + c) * (K - 1), win, 0);
      }
    }
    return;
  }
  const int t0 = blockIdx.x * a.tile, t1 = min(t0 + a.tile, a.T);
  int s = find_seq(a.cu, a.S, t0);
  int begin = s >= 0 ? a.cu[s] : 0, next = s < a.S ? a.cu[s + 1] : a.T;
#pragma unroll
  for (int k = 0; k < K - 1; ++k) {
    Pack<T, V> p;
    p.load(x + int64_t(max(t0 - (K - 1) + k, 0)) * a.xs);   // (a row before the sequence is read, and not used)
    p.get(win[k]);
  }
  constexpr int kAhead = 8;   // rows in flight (4: 88 instead of 81 us, 16: 153, too many registers)
  for (int tb = t0; tb < t1; tb += kAhead) {
    Pack<T, V> row[kAhead];
#pragma unroll
    for (int i = 0; i < kAhead; ++i) row[i].load(x + int64_t(min(tb + i, a.T - 1)) * a.xs);
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      const int t = tb + i;
      if (t >= t1) break;
      while (s < a.S && t >= next) {
        ++s;
        begin = next;
        next = s < a.S ? a.cu[s + 1] : a.T;
      }
      row[i].get(win[K - 1]);
      if (s >= 0 && s < a.S && t - begin >= K - 1) emit(t);
      shift<K, V>(win);
    }
  }
}

// One token for each row: the window is shifted in place.  A thread owns V channels of a row.
template <typename T, int V, int K>
__global__ void __launch_bounds__(kThreads) packed_conv_step_kernel(PConvArgs a) {
  const int c = (blockIdx.x * kThreads + threadIdx.x) * V;
  if (c >= a.C) return;
  const int row = blockIdx.y;
  const int64_t slot = slot_of(a.idx, row, a.nslots);
  float* st = a.state_out + (max(slot, int64_t(0)) * a.C + c) * (K - 1);
  float win[K][V], pre[V];
  Pack<T, V> p;
  p.load(static_cast<const T*>(a.x) + int64_t(row) * a.xs + c);
  if constexpr (K > 1) get_window<K, V>(st, win);   // (without a slot, the first one's, and not used)
  Taps<K, V> tp;
  tp.load(a, c);
#pragma unroll
  for (int k = 0; k < K - 1; ++k)
#pragma unroll
    for (int v = 0; v < V; ++v) win[k][v] = slot >= 0 ? win[k][v] : 0.0f;
  p.get(win[K - 1]);
  conv_pre<K, V>(tp, win, pre);
  if (a.silu) {
#pragma unroll
    for (int v = 0; v < V; ++v) pre[v] *= sigmoid(pre[v]);
  }
  Pack<T, V>::store(static_cast<T*>(a.u) + int64_t(row) * a.us + c, pre);
  if (slot >= 0) put_window<K, V>(st, win, 1);
}

// Backward.  A tile's threads walk its tokens and K - 1 more (whose dpre reaches back into the tile); acc[j] is dx of
// the token j steps back.  dw and dbias of the tile go to the workspace, summed over the tiles in order afterwards.
// Block ntiles + s gives the gradient of sequence s's window.
template <typename T, int V, int K>
__global__ void __launch_bounds__(kBwdThreads) packed_conv_bwd_kernel(PConvArgs a) {
  const int c = (blockIdx.y * kBwdThreads + threadIdx.x) * V;
  if (c >= a.C) return;
  const T* x = static_cast<const T*>(a.x) + c;
  const T* du = static_cast<const T*>(a.du) + c;
  T* dx = static_cast<T*>(a.dx) + c;
  Taps<K, V> tp;
  tp.load(a, c);
  float win[K][V], pre[V], dp[V];
  auto grad = [&](const Pack<T, V>& g) __attribute__((always_inline)) {   // dp of the token at the end of win
    conv_pre<K, V>(tp, win, pre);
    g.get(dp);
#pragma unroll
    for (int v = 0; v < V; ++v) dp[v] *= slope(pre[v], a.silu);
  };
  if (static_cast<int>(blockIdx.x) >= a.ntiles) {
    const int s = blockIdx.x - a.ntiles;
    int begin, end;
    seq_range(a.cu, s, a.T, begin, end);
    const int n = end - begin;
    load_window<K, V>(a, s, c, win);
    float g[K][V] = {};   // gradient of window entry i
#pragma unroll
    for (int i = 0; i < K - 1; ++i) {
      if (i < n) {
        Pack<T, V> px, pd;
        px.load(x + int64_t(begin + i) * a.xs);
        pd.load(du + int64_t(begin + i) * a.dus);
        px.get(win[K - 1]);
        grad(pd);
        // entry j of the first window is tap j - i of token i
#pragma unroll
        for (int j = i; j < K - 1; ++j)
#pragma unroll
          for (int v = 0; v < V; ++v) g[j][v] = fmaf(tp.w[j - i][v], dp[v], g[j][v]);
        shift<K, V>(win);
      }
    }
#pragma unroll
    for (int j = 0; j < K - 1; ++j)
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const int64_t at = (int64_t(s) * a.C + c + v) * (K - 1);
        // an entry that the sequence does not push out is entry j - n of the last window
        const float kept = a.dstate_out && j >= n ? a.dstate_out[at + j - n] : 0.0f;
        a.dstate[at + j] = g[j][v] + kept;
      }
    return;
  }
  const int t0 = blockIdx.x * a.tile, t1 = min(t0 + a.tile, a.T);
  int s = find_seq(a.cu, a.S, t0);
  int begin = s >= 0 ? a.cu[s] : 0, next = s < a.S ? a.cu[s + 1] : a.T;
  const int first = a.cu[0], last = a.cu[a.S];   // rows outside every sequence are left as they are
  bool in = s >= 0 && s < a.S;
  if (in && t0 - begin < K - 1) {
    // the window reaches before the sequence: the initial one, moved on by the tokens before the tile
    load_window<K, V>(a, s, c, win);
    for (int t = max(begin, 0); t < t0; ++t) {
      Pack<T, V> p;
      p.load(x + int64_t(t) * a.xs);
      p.get(win[K - 1]);
      shift<K, V>(win);
    }
  } else {
#pragma unroll
    for (int k = 0; k < K - 1; ++k) {
      Pack<T, V> p;
      p.load(x + int64_t(max(t0 - (K - 1) + k, 0)) * a.xs);
      p.get(win[k]);
    }
  }
  float acc[K][V] = {}, gw[K][V] = {}, gb[V] = {};
  constexpr int kAhead = 4;   // rows in flight (2: 112 instead of 100 us, 8: 100)
  const int tend = min(t1 + K - 1, a.T);
  for (int tb = t0; tb < t1 + K - 1; tb += kAhead) {
    Pack<T, V> rx[kAhead], rg[kAhead];
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      rx[i].load(x + int64_t(min(tb + i, a.T - 1)) * a.xs);
      rg[i].load(du + int64_t(min(tb + i, a.T - 1)) * a.dus);
    }
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      const int t = tb + i;
      if (t >= t1 + K - 1) break;
      // acc[j]: dx of token t - j
#pragma unroll
      for (int j = K - 1; j > 0; --j)
#pragma unroll
        for (int v = 0; v < V; ++v) acc[j][v] = acc[j - 1][v];
#pragma unroll
      for (int v = 0; v < V; ++v) acc[0][v] = 0.0f;
      if (t < tend) {
        while (s < a.S && t >= next) {
          ++s;
          begin = next;
          next = s < a.S ? a.cu[s + 1] : a.T;
          in = s < a.S;
          if (in) load_window<K, V>(a, s, c, win);
        }
        if (in) {
          rx[i].get(win[K - 1]);
          grad(rg[i]);
          const int pos = t - begin;
#pragma unroll
          for (int j = 0; j < K; ++j)
            if (pos >= j) {
#pragma unroll
              for (int v = 0; v < V; ++v) acc[j][v] = fmaf(tp.w[K - 1 - j][v], dp[v], acc[j][v]);
            }
          if (t < t1) {
#pragma unroll
            for (int v = 0; v < V; ++v) {
#pragma unroll
              for (int k = 0; k < K; ++k) gw[k][v] = fmaf(dp[v], win[k][v], gw[k][v]);
              gb[v] += dp[v];
            }
            // the last K - 1 inputs are the sequence's last window
            if (K > 1 && a.dstate_out && t >= next - (K - 1)) {
#pragma unroll
              for (int v = 0; v < V; ++v)
                acc[0][v] += a.dstate_out[(int64_t(s) * a.C + c + v) * (K - 1) + t - (next - (K - 1))];
            }
          }
          shift<K, V>(win);
        }
      }
      const int td = t - (K - 1);
      if (td >= t0 && td < t1) {
        if (td >= first && td < last) Pack<T, V>::store(dx + int64_t(td) * a.dxs, acc[K - 1]);
      }
    }
  }
  float* part = a.part + int64_t(blockIdx.x) * (K + 1) * a.C + c;
#pragma unroll
  for (int v = 0; v < V; ++v) {
#pragma unroll
    for (int k = 0; k < K; ++k) part[int64_t(k) * a.C + v] = gw[k][v];
    part[int64_t(K) * a.C + v] = gb[v];
  }
}

// dw[c][k] and dbias[c]: the tiles' partial sums, 16 interleaved runs of tiles per channel, joined in a fixed order.
__global__ void __launch_bounds__(kThreads) packed_conv_reduce_kernel(PConvArgs a, int K) {
  __shared__ float sum[16][17];
  const int j = blockIdx.y;   // row k of the taps, or the bias
  const int cl = threadIdx.x & 15, r = threadIdx.x >> 4;
  const int c = blockIdx.x * 16 + cl;
  float v = 0.0f;
  if (c < a.C)
    for (int i = r; i < a.ntiles; i += 16) v += a.part[(int64_t(i) * (K + 1) + j) * a.C + c];
  sum[r][cl] = v;
  __syncthreads();
  if (r == 0 && c < a.C) {
    float t = 0.0f;
    for (int i = 0; i < 16; ++i) t += sum[i][cl];
    if (j < K) a.dw[int64_t(c) * K + j] = t;
    else if (a.dbias) a.dbias[c] = t;
  }
}

ssm_status check_pconv(const ssm_conv_packed_params* p, bool step) {
  if (!p) return fail(SSM_ERR_NULL, "params is NULL");
  if (p->reserved != 0) return fail(SSM_ERR_UNSUPPORTED, "reserved must be 0");
  if (p->ntokens < 1 || p->dim < 1 || (!step && p->nseqs < 1) || p->nslots < 0)
    return fail(SSM_ERR_SHAPE, "ntokens, nseqs and dim must be >= 1, nslots >= 0");
  if (p->ntokens >= (int64_t(1) << 30) || p->dim >= (int64_t(1) << 24))
    return fail(SSM_ERR_SHAPE, "ntokens must be below 2^30 and dim below 2^24");
  if (!step && p->nseqs > (int64_t(1) << 24)) return fail(SSM_ERR_SHAPE, "nseqs must not exceed 2^24");
  if (step && p->ntokens > 65535) return fail(SSM_ERR_SHAPE, "a step takes at most 65535 tokens (got %lld)",
                                              (long long)p->ntokens);
  if (p->width < 1 || p->width > 4) return fail(SSM_ERR_SHAPE, "width must be 1 to 4 (got %d)", p->width);
  if (p->activation != 0 && p->activation != 1)
    return fail(SSM_ERR_UNSUPPORTED, "activation must be 0 or 1 (got %d)", p->activation);
  if (p->io_dtype != SSM_F32 && p->io_dtype != SSM_BF16) return fail(SSM_ERR_DTYPE, "unknown io_dtype %d", p->io_dtype);
  const int64_t most = int64_t(1) << 40;
  for (int64_t s : {p->x_stride, p->u_stride, p->du_stride, p->dx_stride})
    if (s != 0 && (s < p->dim || s > most)) return fail(SSM_ERR_SHAPE, "a row stride of %lld is shorter than a row of %lld",
                                                        (long long)s, (long long)p->dim);
  return SSM_OK;
}

PConvArgs args_of(const ssm_conv_packed_params* p) {
  PConvArgs a{};
  a.T = static_cast<int>(p->ntokens);
  a.S = static_cast<int>(p->nseqs);
  a.C = static_cast<int>(p->dim);
  a.nslots = p->nslots;
  a.silu = p->activation;
  a.xs = p->x_stride ? p->x_stride : p->dim;
  a.us = p->u_stride ? p->u_stride : p->dim;
  a.dus = p->du_stride ? p->du_stride : p->dim;
  a.dxs = p->dx_stride ? p->dx_stride : p->dim;
  return a;
}

bool rows_aligned(const void* ptr, int64_t stride, int64_t dim, int elem) {
  const int64_t v = 16 / elem;
  return aligned(ptr, 16) && stride % v == 0 && dim % v == 0;
}

// Tokens per tile of the forward: as long as the launch still has about two waves for each of the 1024 SIMDs (a longer
// tile re-reads fewer halo rows), and at most 64.  Measured on bf16 rows of 5376 channels, width 4, 16384 tokens (352 MB
// moved): tiles of 16, 32, 40, 64 and 128 tokens 85, 94, 89, 81 and 91 us.
int fwd_tile(const PConvArgs& a, int v) {
  const int64_t lanes = (a.C + v - 1) / v;
  int64_t tile = int64_t(a.T) * lanes / (2 * 1024 * 64);
  tile = tile < 8 ? 8 : (tile > 64 ? 64 : tile);
  return static_cast<int>(tile / 8 * 8);
}
// Tokens per tile of the backward, where latency and arithmetic of a wave count: its waves on the busiest SIMD, times the rows that
// each of them walks (the halo, and about 8 rows' worth of taps and partial sums, on top), as few as possible.  Measured
// on 8191 tokens of the same rows (264 MB): 32, 48, 64 and 96 tokens (3, 2, 2 and 1 waves) 105, 87, 100 and 104 us.
int bwd_tile(const PConvArgs& a, int v, int K) {
  const int64_t across = (a.C + v * kBwdThreads - 1) / (v * kBwdThreads);
  int best = 8;
  int64_t least = INT64_MAX;
  for (int tile = 8; tile <= 64; tile += 8) {
    const int64_t waves = (a.T + tile - 1) / tile * across;
    const int64_t cost = (waves + 1023) / 1024 * (tile + K - 1 + 8);
    if (cost < least) {
      least = cost;
      best = tile;
    }
  }
  return best;
}

template <typename F>
ssm_status by_width(int width, F&& f) {
  switch (width) {
    case 1: f(std::integral_constant<int, 1>{}); break;
    case 2: f(std::integral_constant<int, 2>{}); break;
    case 3: f(std::integral_constant<int, 3>{}); break;
    default: f(std::integral_constant<int, 4>{}); break;
  }
  const hipError_t e = hipGetLastError();
  return e == hipSuccess ? SSM_OK : fail(SSM_ERR_HIP, "packed convolution launch: %s", hipGetErrorString(e));
}

int elem_size(const ssm_conv_packed_params* p) { return p->io_dtype == SSM_BF16 ? 2 : 4; }

size_t bwd_workspace(const ssm_conv_packed_params* p) {
  const PConvArgs a = args_of(p);
  // for whichever of the vector and the scalar form runs
  const int tile = std::min(bwd_tile(a, 16 / elem_size(p), p->width), bwd_tile(a, 1, p->width));
  return size_t((a.T + tile - 1) / tile) * (p->width + 1) * a.C * 4;
}

}  // namespace
}  // namespace ssm57

using namespace ssm57;

extern "C" ssm_status ssm_conv1d_packed_fwd(const ssm_conv_packed_params* p, const void* x, const float* weight,
                                            const float* bias, const int32_t* cu_seqlens, const float* state,
                                            const int32_t* state_idx, const uint8_t* has_state, float* state_out,
                                            void* u, void* stream) {
  g_err[0] = 0;
  if (ssm_status s = check_pconv(p, false); s != SSM_OK) return s;
  if (!x || !weight || !cu_seqlens || !u) return fail(SSM_ERR_NULL, "x, weight, cu_seqlens and u are required");
  const int es = elem_size(p);
  if (!aligned(x, es) || !aligned(u, es) || !aligned(weight, 4) || !aligned(bias, 4) || !aligned(cu_seqlens, 4) ||
      !aligned(state, 4) || !aligned(state_idx, 4) || !aligned(state_out, 4))
    return fail(SSM_ERR_ALIGN, "a pointer is not aligned to its element size");
  PConvArgs a = args_of(p);
  a.x = x;
  a.w = weight;
  a.bias = bias;
  a.cu = cu_seqlens;
  a.state = state;
  a.idx = state_idx;
  a.has = has_state;
  a.state_out = state_out;
  a.u = u;
  const bool vec = rows_aligned(x, a.xs, a.C, es) && rows_aligned(u, a.us, a.C, es);
  const int V = vec ? 16 / es : 1;
  a.tile = fwd_tile(a, V);
  a.ntiles = (a.T + a.tile - 1) / a.tile;
  if (!fits_launch(int64_t(a.ntiles) + a.S, kThreads)) return fail(SSM_ERR_SHAPE, "too many tokens and sequences for one launch");
  const dim3 grid(a.ntiles + a.S, (a.C + V * kThreads - 1) / (V * kThreads));
  if (grid.y > 65535) return fail(SSM_ERR_SHAPE, "dim is too large");
  hipStream_t st = static_cast<hipStream_t>(stream);
  return by_width(p->width, [&](auto k) {
    constexpr int K = decltype(k)::value;
    if (es == 2 && vec) hipLaunchKernelGGL((packed_conv_fwd_kernel<uint16_t, 8, K>), grid, dim3(kThreads), 0, st, a);
    else if (es == 2) hipLaunchKernelGGL((packed_conv_fwd_kernel<uint16_t, 1, K>), grid, dim3(kThreads), 0, st, a);
    else if (vec) hipLaunchKernelGGL((packed_conv_fwd_kernel<float, 4, K>), grid, dim3(kThreads), 0, st, a);
    else hipLaunchKernelGGL((packed_conv_fwd_kernel<float, 1, K>), grid, dim3(kThreads), 0, st, a);
  });
}

extern "C" ssm_status ssm_conv1d_slot_update(const ssm_conv_packed_params* p, const void* x, const float* weight,
                                             const float* bias, float* state, const int32_t* state_idx, void* u,
                                             void* stream) {
  g_err[0] = 0;
  if (ssm_status s = check_pconv(p, true); s != SSM_OK) return s;
  if (!x || !weight || !u || (p->width > 1 && !state))
    return fail(SSM_ERR_NULL, "x, weight, u and (for width > 1) state are required");
  // (a row without a slot reads the first one's window, and does not use it)
  if (p->width > 1 && p->nslots < 1) return fail(SSM_ERR_SHAPE, "nslots must be >= 1");
  const int es = elem_size(p);
  if (!aligned(x, es) || !aligned(u, es) || !aligned(weight, 4) || !aligned(bias, 4) || !aligned(state, 4) ||
      !aligned(state_idx, 4))
    return fail(SSM_ERR_ALIGN, "a pointer is not aligned to its element size");
  PConvArgs a = args_of(p);
  a.x = x;
  a.w = weight;
  a.bias = bias;
  a.idx = state_idx;
  a.state_out = state;
  a.u = u;
  const bool vec = rows_aligned(x, a.xs, a.C, es) && rows_aligned(u, a.us, a.C, es);
  const int V = vec ? 16 / es : 1;
  const dim3 grid((a.C + V * kThreads - 1) / (V * kThreads), a.T);
  hipStream_t st = static_cast<hipStream_t>(stream);
  return by_width(p->width, [&](auto k) {
    constexpr int K = decltype(k)::value;
    if (es == 2 && vec) hipLaunchKernelGGL((packed_conv_step_kernel<uint16_t, 8, K>), grid, dim3(kThreads), 0, st, a);
    else if (es == 2) hipLaunchKernelGGL((packed_conv_step_kernel<uint16_t, 1, K>), grid, dim3(kThreads), 0, st, a);
    else if (vec) hipLaunchKernelGGL((packed_conv_step_kernel<float, 4, K>), grid, dim3(kThreads), 0, st, a);
    else hipLaunchKernelGGL((packed_conv_step_kernel<float, 1, K>), grid, dim3(kThreads), 0, st, a);
  });
}

extern "C" size_t ssm_conv1d_packed_bwd_workspace_bytes(const ssm_conv_packed_params* p) {
  return check_pconv(p, false) == SSM_OK ? bwd_workspace(p) : 0;
}

extern "C" ssm_status ssm_conv1d_packed_bwd(const ssm_conv_packed_params* p, const void* x, const float* weight,
                                            const float* bias, const int32_t* cu_seqlens, const float* state,
                                            const int32_t* state_idx, const uint8_t* has_state, const void* du,
                                            const float* dstate_out, void* dx, float* dweight, float* dbias,
                                            float* dstate, void* workspace, size_t workspace_bytes, void* stream) {
  g_err[0] = 0;
  if (ssm_status s = check_pconv(p, false); s != SSM_OK) return s;
  if (!x || !weight || !cu_seqlens || !du || !dx || !dweight)
    return fail(SSM_ERR_NULL, "x, weight, cu_seqlens, du, dx and dweight are required");
  const int es = elem_size(p);
  if (!aligned(x, es) || !aligned(du, es) || !aligned(dx, es) || !aligned(weight, 4) || !aligned(bias, 4) ||
      !aligned(cu_seqlens, 4) || !aligned(state, 4) || !aligned(state_idx, 4) || !aligned(dstate_out, 4) ||
      !aligned(dweight, 4) || !aligned(dbias, 4) || !aligned(dstate, 4))
    return fail(SSM_ERR_ALIGN, "a pointer is not aligned to its element size");
  const size_t need = bwd_workspace(p);
  if (!workspace || workspace_bytes < need || !aligned(workspace, 4))
    return fail(SSM_ERR_WORKSPACE, "workspace of %zu bytes needed, got %zu at %p", need, workspace_bytes, workspace);
  PConvArgs a = args_of(p);
  a.x = x;
  a.w = weight;
  a.bias = bias;
  a.cu = cu_seqlens;
  a.state = state;
  a.idx = state_idx;
  a.has = has_state;
  a.du = du;
  a.dstate_out = dstate_out;
  a.dx = dx;
  a.part = static_cast<float*>(workspace);
  a.dw = dweight;
  a.dbias = dbias;
  a.dstate = dstate;
  const bool vec = rows_aligned(x, a.xs, a.C, es) && rows_aligned(du, a.dus, a.C, es) &&
                   rows_aligned(dx, a.dxs, a.C, es);
  const int V = vec ? 16 / es : 1;
  a.tile = bwd_tile(a, V, p->width);
  a.ntiles = (a.T + a.tile - 1) / a.tile;
  const dim3 grid(a.ntiles + (dstate && p->width > 1 ? a.S : 0), (a.C + V * kBwdThreads - 1) / (V * kBwdThreads));
  if (grid.y > 65535) return fail(SSM_ERR_SHAPE, "dim is too large");
  hipStream_t st = static_cast<hipStream_t>(stream);
  return by_width(p->width, [&](auto k) {
    constexpr int K = decltype(k)::value;
    if (es == 2 && vec) hipLaunchKernelGGL((packed_conv_bwd_kernel<uint16_t, 8, K>), grid, dim3(kBwdThreads), 0, st, a);
    else if (es == 2) hipLaunchKernelGGL((packed_conv_bwd_kernel<uint16_t, 1, K>), grid, dim3(kBwdThreads), 0, st, a);
    else if (vec) hipLaunchKernelGGL((packed_conv_bwd_kernel<float, 4, K>), grid, dim3(kBwdThreads), 0, st, a);
    else hipLaunchKernelGGL((packed_conv_bwd_kernel<float, 1, K>), grid, dim3(kBwdThreads), 0, st, a);
    hipLaunchKernelGGL(packed_conv_reduce_kernel, dim3((a.C + 15) / 16, K + 1), dim3(kThreads), 0, st, a, K);
  });
}
