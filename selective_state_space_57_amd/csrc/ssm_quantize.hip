// Quantisation to e4m3 with an fp32 scale for each block of 128: along the rows (the product over channels), along the
// columns and laid out transposed (the weight gradient's product over tokens), or for blocks of 128 rows and columns
// (weights) in either layout.  scale = max(largest magnitude, 2^-100) / 448, code = round(value / scale).
//
// Bound by memory: x is read once, whatever is written.  Eight consecutive elements make a lane's chunk, so 16 lanes hold
// a block of a row and its largest magnitude is four DPP steps.  Rows alone need nothing else.  What goes along columns is
// done by tiles of 128 x 128 in a workgroup of 256 threads with 8 x 8 elements each in registers: the column maxima meet in
// LDS, and the transposed codes go through LDS (16 KB, slots of 8 bytes exchanged by column so that neither side's accesses
// meet in a bank) so that they leave in runs of 128 bytes.  A tile's elements stay in registers from the maxima to the codes.
//
// Measured (a large copy reaches 5.1 TB/s): 8191 x 5120 bf16, rows and columns, 168 MB, 40 us (4.2 TB/s); rows or columns
// alone, 126 MB, 26 and 27; blocks of 10576 x 2560 fp32, both layouts, 162 MB, 33 us (5.0 TB/s); 256 rows of 5120 3.1 us,
// latency.
#include "fp8.hpp"

namespace ssm57 {
namespace {

struct QuantArgs {
  const void* x;
  uint8_t* q;
  float* s;
  uint8_t* qt;
  float* st;
  int64_t xs, qs, ss, qts, sts;
  int rows, cols, cols16, rows16;
  int chunks;      // of 512 columns in a row (rows only), tiles of 128 columns else
};

// codes of eight values, zeros from the cnt-th on
__device__ __forceinline__ pu2 codes8_part(const float* v, float scale, int cnt) {
  pu2 c = codes8(v, scale);
  if (cnt < 8) {
    uint64_t bits = __builtin_bit_cast(uint64_t, c);
    bits = cnt <= 0 ? 0 : bits & ((uint64_t(1) << (8 * cnt)) - 1);
    c = __builtin_bit_cast(pu2, bits);
  }
  return c;
}

template <typename T>
__device__ __forceinline__ void load_part(Eight<T>& e, const T* p, int cnt) {
  if (cnt >= 8) e.load(p);
  else e.load(p, cnt);
}

// Rows only: a wave takes 512 columns of a row.  (Two or four such units to a wave, loaded together, are no faster: bf16
// rows of 2560, 256 of them 2.8, 3.2 and 4.1 us, 4096 7.5, 7.8 and 8.2, 16384 24.2, 22.9 and 23.4; fp32, 16384 36.6 and 40.6
// with four.)
template <typename T>
__global__ void __launch_bounds__(256) quantize_rows_kernel(QuantArgs a) {
  const int lane = threadIdx.x & 63;
  const int64_t units = int64_t(a.rows) * a.chunks;
  for (int64_t u = int64_t(blockIdx.x) * 4 + (threadIdx.x >> 6); u < units; u += int64_t(gridDim.x) * 4) {
    const int64_t row = u / a.chunks;
    const int at = static_cast<int>(u - row * a.chunks) * 512 + lane * 8;
    Eight<T> e;
    load_part(e, static_cast<const T*>(a.x) + row * a.xs + at, a.cols - at);
    float v[8];
    e.get(v);
    const float scale = scale_of(row_largest(largest(v)));
    if (at < a.cols16) *reinterpret_cast<pu2e*>(a.q + row * a.qs + at) = codes8_part(v, scale, a.cols - at);
    if ((lane & 15) == 0 && at < a.cols) a.s[row * a.ss + at / kBlock] = scale;
  }
}

template <typename T, bool SQUARE>
__global__ void __launch_bounds__(256) quantize_tile_kernel(QuantArgs a) {
  __shared__ uint32_t most[16][kBlock];
  __shared__ pu4 turn[kBlock][kBlock / 16];
  const int ct = blockIdx.x % a.chunks, rt = blockIdx.x / a.chunks;
  const int cl = threadIdx.x & 15, rg = threadIdx.x >> 4;
  const int c0 = ct * kBlock, r0 = rt * kBlock;
  const int col = c0 + cl * 8, row = r0 + rg * 8;
  const int ccnt = a.cols - col, rcnt = a.rows - row;   // of this lane's 8 columns and rows: inside
  Eight<T> e[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    if (i < rcnt) load_part(e[i], static_cast<const T*>(a.x) + int64_t(row + i) * a.xs + col, ccnt);
    else e[i].zero();
  }
  uint32_t cm[8] = {}, rm[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    float v[8];
    e[i].get(v);
    rm[i] = largest(v);
#pragma unroll
    for (int j = 0; j < 8; ++j) cm[j] = max(cm[j], magnitude(v[j]));
  }
  float whole = 0.0f;
  if constexpr (SQUARE) {
    uint32_t m = rm[0];
#pragma unroll
    for (int i = 1; i < 8; ++i) m = max(m, rm[i]);
    m = row_largest(m);
    if (cl == 0) most[0][rg] = m;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 16; ++i) m = max(m, most[0][i]);
    whole = scale_of(m);
    if (threadIdx.x == 0) {
      if (a.q) a.s[rt * a.ss + ct] = whole;
      if (a.qt) a.st[ct * a.sts + rt] = whole;
    }
  } else if (a.qt) {
#pragma unroll
    for (int j = 0; j < 8; ++j) most[rg][cl * 8 + j] = cm[j];
    __syncthreads();
    if (threadIdx.x < kBlock) {
      uint32_t m = most[0][threadIdx.x];
#pragma unroll
      for (int i = 1; i < 16; ++i) m = max(m, most[i][threadIdx.x]);
      const float scale = scale_of(m);
      most[0][threadIdx.x] = __float_as_uint(scale);
      if (c0 + static_cast<int>(threadIdx.x) < a.cols) a.st[int64_t(c0 + threadIdx.x) * a.sts + rt] = scale;
    }
  }
  if (a.q) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      float v[8];
      e[i].get(v);
      const float scale = SQUARE ? whole : scale_of(row_largest(rm[i]));
      if (i < rcnt) {
        if (col < a.cols16) *reinterpret_cast<pu2e*>(a.q + int64_t(row + i) * a.qs + col) = codes8_part(v, scale, ccnt);
        if (!SQUARE && cl == 0) a.s[int64_t(row + i) * a.ss + ct] = scale;
      }
    }
  }
  if (!a.qt) return;
  __syncthreads();   // (the columns' scales)
  float t[8][8];
#pragma unroll
  for (int i = 0; i < 8; ++i) e[i].get(t[i]);
  uint2* slot = reinterpret_cast<uint2*>(&turn[0][0]);
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const float scale = SQUARE ? whole : __uint_as_float(most[0][cl * 8 + j]);
    float v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = t[i][j];
    const pu2 c = codes8_part(v, scale, rcnt);
    slot[(cl * 8 + j) * 16 + (rg ^ cl)] = uint2{c[0], c[1]};
  }
  __syncthreads();
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const int c = k * 32 + (threadIdx.x >> 3), u = threadIdx.x & 7;   // a column's 16 rows
    const int key = (c >> 3) & 15;
    pu4 v = turn[c][u ^ (key >> 1)];
    if (key & 1) v = pu4{v[2], v[3], v[0], v[1]};
    if (c0 + c < a.cols && r0 + u * 16 < a.rows16) *reinterpret_cast<pu4*>(a.qt + int64_t(c0 + c) * a.qts + r0 + u * 16) = v;
  }
}

ssm_status check_quantize(const ssm_quantize_fp8_params* p) {
  if (!p) return fail(SSM_ERR_NULL, "params is NULL");
  if (p->reserved[0] != 0 || p->reserved[1] != 0) return fail(SSM_ERR_UNSUPPORTED, "reserved must be 0");
  if (p->rows < 1 || p->cols < 1) return fail(SSM_ERR_SHAPE, "rows and cols must be >= 1");
  if (p->rows >= (int64_t(1) << 30) || p->cols >= (int64_t(1) << 30))
    return fail(SSM_ERR_SHAPE, "rows and cols must be below 2^30");
  if (p->io_dtype != SSM_F32 && p->io_dtype != SSM_BF16) return fail(SSM_ERR_DTYPE, "unknown io_dtype %d", p->io_dtype);
  if (p->square != 0 && p->square != 1) return fail(SSM_ERR_UNSUPPORTED, "square must be 0 or 1");
  const int64_t most = int64_t(1) << 40;
  const int64_t rb = blocks_of(p->rows), cb = blocks_of(p->cols);
  const struct { int64_t stride, row; } rows[] = {{p->x_stride, p->cols}, {p->q_stride, up16(p->cols)}, {p->scale_stride, cb},
                                                  {p->qt_stride, up16(p->rows)}, {p->scale_t_stride, rb}};
  for (const auto& r : rows)
    if (r.stride != 0 && (r.stride < r.row || r.stride > most))
      return fail(SSM_ERR_SHAPE, "a row stride of %lld is shorter than a row of %lld", (long long)r.stride, (long long)r.row);
  if (!fits_launch(rb * cb, 256))
    return fail(SSM_ERR_SHAPE, "%lld rows of %lld do not fit a launch", (long long)p->rows, (long long)p->cols);
  return SSM_OK;
}

template <typename T>
void launch_quantize(QuantArgs& a, bool square, hipStream_t st) {
  if (!a.qt && !square) {
    a.chunks = (a.cols16 + 511) / 512;
    const int64_t groups = (int64_t(a.rows) * a.chunks + 3) / 4, most = 1 << 23;   // (2^31 threads at most)
    hipLaunchKernelGGL((quantize_rows_kernel<T>), dim3(static_cast<uint32_t>(groups < most ? groups : most)), dim3(256), 0, st, a);
    return;
  }
  a.chunks = static_cast<int>(blocks_of(a.cols));
  const dim3 grid(static_cast<uint32_t>(a.chunks * blocks_of(a.rows)));
  if (square) hipLaunchKernelGGL((quantize_tile_kernel<T, true>), grid, dim3(256), 0, st, a);
  else hipLaunchKernelGGL((quantize_tile_kernel<T, false>), grid, dim3(256), 0, st, a);
}

}  // namespace
}  // namespace ssm57

using namespace ssm57;

extern "C" ssm_status ssm_quantize_fp8(const ssm_quantize_fp8_params* p, const void* x, void* q, float* scale, void* qt,
                                       float* scale_t, void* stream) {
  g_err[0] = 0;
  if (ssm_status s = check_quantize(p); s != SSM_OK) return s;
  if (!x || (!q && !qt) || (q != nullptr) != (scale != nullptr) || (qt != nullptr) != (scale_t != nullptr))
    return fail(SSM_ERR_NULL, "x, and q with scale or qt with scale_t or both are required");
  if (!aligned(x, p->io_dtype == SSM_BF16 ? 2 : 4) || !aligned(scale, 4) || !aligned(scale_t, 4))
    return fail(SSM_ERR_ALIGN, "a pointer is not aligned to its element size");
  if (!aligned(q, 16) || !aligned(qt, 16) || p->q_stride % 16 || p->qt_stride % 16)
    return fail(SSM_ERR_ALIGN, "rows of q and qt must be 16-byte aligned");
  QuantArgs a{};
  a.x = x;
  a.q = static_cast<uint8_t*>(q);
  a.s = scale;
  a.qt = static_cast<uint8_t*>(qt);
  a.st = scale_t;
  a.rows = static_cast<int>(p->rows);
  a.cols = static_cast<int>(p->cols);
  a.rows16 = static_cast<int>(up16(p->rows));
  a.cols16 = static_cast<int>(up16(p->cols));
  const int64_t rb = blocks_of(p->rows), cb = blocks_of(p->cols);
  a.xs = p->x_stride ? p->x_stride : p->cols;
  a.qs = p->q_stride ? p->q_stride : a.cols16;
  a.ss = p->scale_stride ? p->scale_stride : cb;
  a.qts = p->qt_stride ? p->qt_stride : a.rows16;
  a.sts = p->scale_t_stride ? p->scale_t_stride : rb;
  if (p->io_dtype == SSM_BF16) launch_quantize<uint16_t>(a, p->square, static_cast<hipStream_t>(stream));
  else launch_quantize<float>(a, p->square, static_cast<hipStream_t>(stream));
  const hipError_t e = hipGetLastError();
  return e == hipSuccess ? SSM_OK : fail(SSM_ERR_HIP, "quantize launch: %s", hipGetErrorString(e));
}
