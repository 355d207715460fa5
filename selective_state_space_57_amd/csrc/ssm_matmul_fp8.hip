// Matrix product of e4m3 operands with an fp32 scale for each block of 128 along k:
//   out[i][j] = sum over blocks c of sa[i][c] sb[j / b_rows][c] (sum over the block's k of a[i][k] b[j][k])
//
// v_mfma_f32_16x16x128_f8f6f4 takes a whole block of 128 k at once: its result is the block's inner sum, which goes into
// the fp32 sums times the two scales.  b is the first operand, so that a lane's four results are four neighbouring j of
// one i: one scale of a for them all, and one store.
//
// Inside, the 8-bit matrix instructions (of every shape) align their products to the largest of a group and drop what lies
// below about 2^-12 of it: measured 1.4e-5 of the result's 2-norm for values of a normal distribution, 5e-5 for codes drawn
// evenly.  A bf16 result, whose own rounding is 1.7e-3, is computed with them.  An fp32 result (a weight gradient) is not:
// its codes become bf16, which holds them exactly, on the way into v_mfma_f32_16x16x32_bf16, which sums in fp32.
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
  float* part;            // [splits][m][n]: the sums of each piece of k
  int64_t as, bs, os, sas, sbs;
  int m, n, k, blocks;    // blocks of 128 along k
  int tiles_n;
  int splits, per;        // pieces of k, blocks of a piece
};

__device__ __forceinline__ v8i join(v4i lo, v4i hi) {
  return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
}
__device__ __forceinline__ v8bf widen(int lo, int hi) {
  const pbf2 a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.0f, false), b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.0f, true);
  const pbf2 c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.0f, false), d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.0f, true);
  return v8bf{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}

// A wave's 16 rows of a block: a lane's 32 codes, as they are or as bf16.
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
__device__ __forceinline__ pf4 mfma_block(const Frag<false>& b, const Frag<false>& a) {
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(b.v, a.v, pf4{0.0f, 0.0f, 0.0f, 0.0f}, 0, 0, 0, 0, 0, 0);
}
__device__ __forceinline__ pf4 mfma_block(const Frag<true>& b, const Frag<true>& a) {
  pf4 d{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
  for (int i = 0; i < 4; ++i) d = __builtin_amdgcn_mfma_f32_16x16x32_bf16(b.v[i], a.v[i], d, 0, 0, 0);
  return d;
}

// four neighbouring results, of which cnt are inside the row
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

// A workgroup's tile of BM x BN results; WM x WN waves.  BROWS: rows of b under one scale.  WIDE: bf16 products.
template <int BM, int BN, int WM, int WN, int BROWS, bool WIDE, typename TO>
__global__ void __launch_bounds__(64 * WM * WN) matmul_tile_kernel(MatmulArgs g) {
  constexpr int NW = WM * WN, TM = BM / 16 / WM, TN = BN / 16 / WN;
  constexpr int kLoads = (BM + BN) / 8;          // copies of 1 KB (8 rows of a block) in a stage
  static_assert(kLoads % NW == 0 && BM / 8 % NW == 0);
  struct Stage {
    uint8_t rows[(BM + BN) * 128];
    float scale[BM + (BROWS == 1 ? BN : 0)];
  };
  __shared__ __align__(1024) Stage stage[2];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wave % WM, wn = wave / WM;
  const int tile = blockIdx.x / g.splits, piece = blockIdx.x % g.splits;
  const int m0 = tile / g.tiles_n * BM, n0 = tile % g.tiles_n * BN;
  const int c0 = piece * g.per, c1 = min(c0 + g.per, g.blocks);
  const int rows_m = min(BM, g.m - m0), rows_n = min(BN, g.n - n0);
  const auto ra = make_rsrc(g.a + m0 * g.as, (rows_m - 1) * g.as + g.k);
  const auto rb = make_rsrc(g.b + n0 * g.bs, (rows_n - 1) * g.bs + g.k);
  const auto rsa = make_rsrc(g.sa + m0 * g.sas, (rows_m - 1) * g.sas + g.blocks);
  const auto rsb = make_rsrc(g.sb + (BROWS == 1 ? n0 * g.sbs : 0), BROWS == 1 ? (rows_n - 1) * g.sbs + g.blocks : 0);

  // A copy's lane has row lane / 8 of eight, and the unit of 16 bytes whose place in LDS is lane % 8: units are exchanged by
  // row so that 8 rows' equal units lie in different banks.
  const int unit = (lane & 7) ^ (lane >> 3);
  const uint32_t voff_a = static_cast<uint32_t>(lane >> 3) * static_cast<uint32_t>(g.as) + 16u * unit;
  const uint32_t voff_b = static_cast<uint32_t>(lane >> 3) * static_cast<uint32_t>(g.bs) + 16u * unit;
  auto load = [&](int c, Stage& st) {
    const bool in = c * 128 + unit * 16 < g.k;   // (past the end of k: zeros)
#pragma unroll
    for (int i = 0; i < kLoads / NW; ++i) {
      const int piece8 = wave + NW * i;          // eight rows
      const bool is_a = NW * i < BM / 8;
      const uint32_t row = is_a ? piece8 * 8 : (piece8 - BM / 8) * 8;
      const uint32_t off = (is_a ? voff_a : voff_b) + row * static_cast<uint32_t>(is_a ? g.as : g.bs) + c * 128u;
      __builtin_amdgcn_raw_ptr_buffer_load_lds(is_a ? ra : rb, (lds_mvoid*)(st.rows + piece8 * 1024), 16,
                                               static_cast<int>(in ? off : kDropOffset), 0, 0, 0);
    }
    constexpr int kScales = BM / 64 + (BROWS == 1 ? BN / 64 : 0);
#pragma unroll
    for (int i = 0; i < (kScales + NW - 1) / NW; ++i) {
      const int p = wave + NW * i;
      if (p < kScales) {
        const bool is_a = p < BM / 64;
        const uint32_t row = (is_a ? p : p - BM / 64) * 64u + lane;
        const uint32_t off = 4u * (row * static_cast<uint32_t>(is_a ? g.sas : g.sbs) + c);
        if (is_a) __builtin_amdgcn_raw_ptr_buffer_load_lds(rsa, (lds_mvoid*)(st.scale + p * 64), 4, static_cast<int>(off), 0, 0, 0);
        else __builtin_amdgcn_raw_ptr_buffer_load_lds(rsb, (lds_mvoid*)(st.scale + p * 64), 4, static_cast<int>(off), 0, 0, 0);
      }
    }
  };

  pf4 acc[TM][TN] = {};
  const int r16 = lane & 15, kg = lane >> 4;
  const int u0 = ((2 * kg) ^ (r16 & 7)) * 16, u1 = ((2 * kg + 1) ^ (r16 & 7)) * 16;
  const float* sb_row = g.sb + (n0 + wn * TN * 16) / 128 * g.sbs;
  if (c0 < c1) load(c0, stage[0]);
  for (int c = c0; c < c1; ++c) {
    Stage& st = stage[(c - c0) & 1];
    __syncthreads();
    if (c + 1 < c1) load(c + 1, stage[(c + 1 - c0) & 1]);
    Frag<WIDE> bf[TN];
    pf4 sbn[TN];
#pragma unroll
    for (int j = 0; j < TN; ++j) {
      const uint8_t* p = st.rows + (BM + (wn * TN + j) * 16 + r16) * 128;
      bf[j].set(join(*reinterpret_cast<const v4i*>(p + u0), *reinterpret_cast<const v4i*>(p + u1)));
      if constexpr (BROWS == 1) sbn[j] = *reinterpret_cast<const pf4*>(st.scale + BM + (wn * TN + j) * 16 + kg * 4);
    }
    const float sb = BROWS == 1 ? 1.0f : sb_row[c];
#pragma unroll
    for (int i = 0; i < TM; ++i) {
      const uint8_t* p = st.rows + ((wm * TM + i) * 16 + r16) * 128;
      Frag<WIDE> af;
      af.set(join(*reinterpret_cast<const v4i*>(p + u0), *reinterpret_cast<const v4i*>(p + u1)));
      const float s = st.scale[(wm * TM + i) * 16 + r16] * sb;
#pragma unroll
      for (int j = 0; j < TN; ++j) {
        const pf4 d = mfma_block(bf[j], af);
#pragma unroll
        for (int r = 0; r < 4; ++r) acc[i][j][r] = fmaf(BROWS == 1 ? d[r] * sbn[j][r] : d[r], s, acc[i][j][r]);
      }
    }
  }
  TO* out = g.splits > 1 ? reinterpret_cast<TO*>(g.part + int64_t(piece) * g.m * g.n) : static_cast<TO*>(g.out);
  const int64_t os = g.splits > 1 ? g.n : g.os;
#pragma unroll
  for (int i = 0; i < TM; ++i) {
    const int row = m0 + (wm * TM + i) * 16 + r16;
#pragma unroll
    for (int j = 0; j < TN; ++j) {
      const int col = n0 + (wn * TN + j) * 16 + kg * 4;
      if (row < g.m) store4<TO>(out + row * os + col, acc[i][j], g.n - col);
    }
  }
}

// out: the sums of the pieces of k, in their order
template <typename TO>
__global__ void __launch_bounds__(256) matmul_join_kernel(MatmulArgs g) {
  const int64_t quads = (int64_t(g.n) + 3) / 4, id = int64_t(blockIdx.x) * 256 + threadIdx.x;
  if (id >= quads * g.m) return;
  const int64_t row = id / quads;
  const int col = static_cast<int>(id % quads) * 4, cnt = min(4, g.n - col);
  pf4 sum = {};
  for (int s = 0; s < g.splits; ++s) {
    const float* p = g.part + (int64_t(s) * g.m + row) * g.n + col;
    if (cnt == 4) sum += *reinterpret_cast<const pf4u*>(p);
    else
#pragma unroll
      for (int i = 0; i < 3; ++i)
        if (i < cnt) sum[i] += p[i];
  }
  store4<TO>(static_cast<TO*>(g.out) + row * g.os + col, sum, cnt);
}

struct MatmulPlan {
  int bm, bn, splits, per;
};

MatmulPlan plan_of(const ssm_matmul_fp8_params* p) {
  MatmulPlan t{128, 128, 1, 0};
  const int64_t blocks = blocks_of(p->k);
  const int64_t tiles = ((p->m + t.bm - 1) / t.bm) * ((p->n + t.bn - 1) / t.bn);
  int64_t s = p->splits > 0 ? p->splits : tiles >= 256 ? 1 : 512 / tiles;
  if (p->splits == 0 && s > 16) s = 16;
  if (s > blocks) s = blocks;
  t.per = static_cast<int>((blocks + s - 1) / s);
  t.splits = static_cast<int>((blocks + t.per - 1) / t.per);
  return t;
}

ssm_status check_matmul(const ssm_matmul_fp8_params* p) {
  if (!p) return fail(SSM_ERR_NULL, "params is NULL");
  if (p->reserved != 0) return fail(SSM_ERR_UNSUPPORTED, "reserved must be 0");
  if (p->m < 1 || p->n < 1 || p->k < 1) return fail(SSM_ERR_SHAPE, "m, n and k must be >= 1");
  if (p->m >= (int64_t(1) << 30) || p->n >= (int64_t(1) << 30)) return fail(SSM_ERR_SHAPE, "m and n must be below 2^30");
  if (p->k % 16) return fail(SSM_ERR_SHAPE, "k (%lld) must be a multiple of 16", (long long)p->k);
  if (p->b_rows != 1 && p->b_rows != kBlock) return fail(SSM_ERR_UNSUPPORTED, "b_rows must be 1 or %d", kBlock);
  if (p->out_dtype != SSM_F32 && p->out_dtype != SSM_BF16) return fail(SSM_ERR_DTYPE, "unknown out_dtype %d", p->out_dtype);
  if (p->splits < 0 || p->splits > 64) return fail(SSM_ERR_UNSUPPORTED, "splits must be 0 to 64");
  const int64_t blocks = blocks_of(p->k);
  const struct { int64_t stride, row, most; } rows[] = {{p->a_stride, p->k, 1 << 23}, {p->b_stride, p->k, 1 << 23},
                                                        {p->a_scale_stride, blocks, 1 << 20}, {p->b_scale_stride, blocks, 1 << 20},
                                                        {p->out_stride, p->n, int64_t(1) << 40}};
  if (p->k >= (1 << 23)) return fail(SSM_ERR_SHAPE, "k must be below 2^23");
  for (const auto& r : rows)
    if (r.stride != 0 && (r.stride < r.row || r.stride >= r.most))
      return fail(SSM_ERR_SHAPE, "a row stride of %lld: at least a row of %lld, below %lld", (long long)r.stride,
                  (long long)r.row, (long long)r.most);
  const MatmulPlan t = plan_of(p);
  const int64_t tiles = ((p->m + t.bm - 1) / t.bm) * ((p->n + t.bn - 1) / t.bn);
  if (!fits_launch(tiles * t.splits, 512) || !fits_launch(p->m * ((p->n + 3) / 4) / 256 + 1, 256))
    return fail(SSM_ERR_SHAPE, "a product of %lld x %lld does not fit a launch", (long long)p->m, (long long)p->n);
  return SSM_OK;
}

template <int BM, int BN, int WM, int WN, bool WIDE, typename TO>
void launch_tile(const MatmulArgs& g, int brows, int64_t tiles, hipStream_t st) {
  const dim3 grid(static_cast<uint32_t>(tiles * g.splits)), block(64 * WM * WN);
  if (brows == 1) hipLaunchKernelGGL((matmul_tile_kernel<BM, BN, WM, WN, 1, WIDE, TO>), grid, block, 0, st, g);
  else hipLaunchKernelGGL((matmul_tile_kernel<BM, BN, WM, WN, 128, WIDE, TO>), grid, block, 0, st, g);
}

}  // namespace
}  // namespace ssm57

using namespace ssm57;

extern "C" size_t ssm_matmul_fp8_workspace_bytes(const ssm_matmul_fp8_params* p) {
  if (check_matmul(p) != SSM_OK) return 0;
  const MatmulPlan t = plan_of(p);
  return t.splits > 1 ? size_t(t.splits) * p->m * p->n * 4 : 0;
}

extern "C" ssm_status ssm_matmul_fp8(const ssm_matmul_fp8_params* p, const void* a, const float* a_scale, const void* b,
                                     const float* b_scale, void* out, void* workspace, size_t workspace_bytes,
                                     void* stream) {
  g_err[0] = 0;
  if (ssm_status s = check_matmul(p); s != SSM_OK) return s;
  if (!a || !a_scale || !b || !b_scale || !out) return fail(SSM_ERR_NULL, "a, a_scale, b, b_scale and out are required");
  if (!aligned(a_scale, 4) || !aligned(b_scale, 4) || !aligned(out, p->out_dtype == SSM_BF16 ? 2 : 4))
    return fail(SSM_ERR_ALIGN, "a pointer is not aligned to its element size");
  if (!aligned(a, 16) || !aligned(b, 16) || p->a_stride % 16 || p->b_stride % 16)
    return fail(SSM_ERR_ALIGN, "rows of a and b must be 16-byte aligned");
  const MatmulPlan t = plan_of(p);
  const size_t need = t.splits > 1 ? size_t(t.splits) * p->m * p->n * 4 : 0;
  if (need && (!workspace || workspace_bytes < need || !aligned(workspace, 16)))
    return fail(SSM_ERR_WORKSPACE, "workspace of %zu bytes needed, got %zu at %p", need, workspace_bytes, workspace);
  MatmulArgs g{};
  g.a = static_cast<const uint8_t*>(a);
  g.b = static_cast<const uint8_t*>(b);
  g.sa = a_scale;
  g.sb = b_scale;
  g.out = out;
  g.part = static_cast<float*>(workspace);
  g.m = static_cast<int>(p->m);
  g.n = static_cast<int>(p->n);
  g.k = static_cast<int>(p->k);
  g.blocks = static_cast<int>(blocks_of(p->k));
  g.as = p->a_stride ? p->a_stride : p->k;
  g.bs = p->b_stride ? p->b_stride : p->k;
  g.os = p->out_stride ? p->out_stride : p->n;
  g.sas = p->a_scale_stride ? p->a_scale_stride : g.blocks;
  g.sbs = p->b_scale_stride ? p->b_scale_stride : g.blocks;
  g.splits = t.splits;
  g.per = t.per;
  g.tiles_n = (g.n + t.bn - 1) / t.bn;
  const int64_t tiles = int64_t((g.m + t.bm - 1) / t.bm) * g.tiles_n;
  hipStream_t st = static_cast<hipStream_t>(stream);
  if (p->out_dtype == SSM_F32) launch_tile<128, 128, 2, 2, true, float>(g, p->b_rows, tiles, st);
  else if (g.splits > 1) launch_tile<128, 128, 2, 2, false, float>(g, p->b_rows, tiles, st);
  else launch_tile<128, 128, 2, 2, false, uint16_t>(g, p->b_rows, tiles, st);
  if (g.splits > 1) {
    const dim3 grid(static_cast<uint32_t>((int64_t(g.m) * ((g.n + 3) / 4) + 255) / 256));
    if (p->out_dtype == SSM_F32) hipLaunchKernelGGL((matmul_join_kernel<float>), grid, dim3(256), 0, st, g);
    else hipLaunchKernelGGL((matmul_join_kernel<uint16_t>), grid, dim3(256), 0, st, g);
  }
  const hipError_t e = hipGetLastError();
  return e == hipSuccess ? SSM_OK : fail(SSM_ERR_HIP, "matmul launch: %s", hipGetErrorString(e));
}
