// The states of packed SSD sequences where other kernels start from them: at the segments of the forward, and at every
// chunk for the backward, together with the adjoint states, which are walked in reverse order.
//
// As in the forward, a workgroup takes 4 heads of one group over one segment, a wave holds the state of half of a head's
// columns in registers, and the shared k rows (B or C) go to LDS once for all waves.  The weighted v rows are split into
// three bf16 parts, so states keep fp32 quality.  A sequence of several segments takes three launches: every segment from
// zero, a join in order, and the walk proper, which saves the state entering every chunk.
//
// Measured under the profiler on 16384 tokens of 80 heads, N = 128: the forward's first pass 89 us and its join 23; for the
// backward both first passes 147 us, the joins 41 and both walks 378, in which they write 1.3 GB (3.6 TB/s): the saving is
// their bound.
#include "packed_ssd.hpp"

namespace ssm57 {
namespace {

constexpr int PT = 2;       // 16-column tiles of a wave
constexpr int kParts = 2;   // waves of a head

// SAVE: the walk proper; otherwise the first pass, each segment from zero
template <int N, bool REV, bool SAVE>
__device__ __forceinline__ void walk(const StatesArgs& a, uint16_t* sK0, uint16_t* sK1, uint16_t* V, float* W) {
  constexpr int U = N / 8;
  constexpr int NT = N / 16;             // 16-row tiles of the state
  constexpr int kWaves = kWalkWaves;
  constexpr int UV = 2 * PT;             // 16-byte units of its columns

  // (in launch order, heads fastest: the heads of a segment go round the XCDs, so that segments of any length, and numbers
  // without one, spread evenly; runs of items per XCD, which share B and C in its L2, left some with two rounds)
  const int item = blockIdx.x;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int l16 = lane & 15, g4 = lane >> 4;
  const int hb = item % (a.G * a.hblocks);
  Piece seg;
  if (!find_piece(a.cu, a.S, a.T, a.cps * kChunk, item / (a.G * a.hblocks), seg)) return;
  // (nothing starts from the end of the walk's last segment)
  if (!SAVE && seg.index == (REV ? 0 : seg.count - 1)) return;
  const int64_t kept = seg.place + seg.index;
  const int g = hb / a.hblocks;
  const int hg = (hb % a.hblocks) * (kWaves / kParts) + wave / kParts;   // head within the group
  const int p0 = (wave % kParts) * 16 * PT;                              // first column of this wave
  const bool on = hg < a.hpg;                                            // (a wave without a head computes the last one's)
  const int h = g * a.hpg + (on ? hg : a.hpg - 1);
  const int t_begin = seg.begin + seg.index * a.cps * kChunk;
  const int t_end = min(seg.end, t_begin + a.cps * kChunk);
  const int nchunks = (t_end - t_begin + kChunk - 1) / kChunk;

  const float Ah = a.A[h];
  const float bias = a.dt_bias ? a.dt_bias[h] : 0.0f;
  const uint16_t* vh = a.v + int64_t(h) * kHead + p0;
  const uint16_t* kg = a.k + int64_t(g) * N;
  const uint32_t vrow = static_cast<uint32_t>(a.vs) * 2u, krow = static_cast<uint32_t>(a.ks) * 2u;
  // chunk of turn i: its first token and rows (a turn past the last has none)
  auto place = [&](int i, int64_t& t0, int& rows) __attribute__((always_inline)) {
    const int ck = REV ? nchunks - 1 - i : i;
    t0 = t_begin + int64_t(ck) * kChunk;
    rows = i < nchunks ? min(t_end - static_cast<int>(t0), kChunk) : 0;
    if (rows <= 0) { t0 = 0; rows = 0; }
  };
  auto copy_k = [&](int i, uint16_t* dst) __attribute__((always_inline)) {
    int64_t t0;
    int rows;
    place(i, t0, rows);
    copy_rows<U, kWaves>(dst, chunk_rsrc(kg, t0, a.ks, rows, N), wave, lane, krow);
  };
  auto copy_v = [&](int i) __attribute__((always_inline)) {
    int64_t t0;
    int rows;
    place(i, t0, rows);
    copy_rows<UV, 1>(V, chunk_rsrc(vh, t0, a.vs, rows, 16 * PT), 0, lane, vrow);
  };
  auto load_dt = [&](int i) __attribute__((always_inline)) -> uint32_t {
    int64_t t0;
    int rows;
    place(i, t0, rows);
    return a.dt[(lane < rows ? t0 + lane : t0) * a.dts + h];
  };

  // state tiles: S[nt][pt][c] = S[p][n], n = 16 nt + l16, p = p0 + 8 g4 + 4 pt + c: a lane's two tiles are eight
  // consecutive p of a row n, an operand over p as the backward wants it
  pf4 S[NT][PT];
  const int64_t head_size = int64_t(kHead) * N;
  const int lane_entry = ((p0 + 8 * g4) * N + l16) * 4;   // bytes
  auto put = [&](float* to) __attribute__((always_inline)) {
    const auto r = make_rsrc(to, head_size);
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int pt = 0; pt < PT; ++pt)
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const float v = S[nt][pt][c];
          __builtin_amdgcn_raw_buffer_store_b32(__float_as_int(v), r, lane_entry, ((4 * pt + c) * N + 16 * nt) * 4, 0);
        }
  };
  // the state as operands over p (state_operand): a tile and lane after the other
  auto save = [&](float* to) __attribute__((always_inline)) {
    const auto r = make_rsrc(to, head_size);
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int pt = 0; pt < PT; ++pt)
        __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(pu4, S[nt][pt]), r, state_operand(0, p0 / 16, lane),
                                               state_operand(nt, pt, 0), 0);
  };
  {
    const float* from = nullptr;
    if constexpr (SAVE) {
      if (seg.count > 1) {
        from = a.ws_state + (kept * a.H + h) * head_size;
      } else if (a.init && (!a.has || a.has[seg.seq])) {
        const int64_t slot = slot_of(a.idx, seg.seq, a.nslots);
        if (slot >= 0) from = a.init + (slot * a.H + h) * head_size;
      }
    }
    const auto r = make_rsrc(from ? from : a.A, from ? head_size : 0);   // (an empty range reads as zeros)
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int pt = 0; pt < PT; ++pt)
#pragma unroll
        for (int c = 0; c < 4; ++c)
          S[nt][pt][c] = __int_as_float(
              __builtin_amdgcn_raw_buffer_load_b32(r, lane_entry, ((4 * pt + c) * N + 16 * nt) * 4, 0));
  }
  float decay = 0.0f;   // sum of log2 decays over the segment (first pass)

  auto chunk = [&](const int i, const uint16_t* K, uint16_t* Kn, const uint32_t dtv) __attribute__((always_inline))
               -> uint32_t {
    wait_memory();    // this wave's copies of the chunk
    barrier_lds();    // everyone's, and the previous chunk's readers are done
    copy_k(i + 1, Kn);
    const uint32_t dt_next = load_dt(i + 1);
    int64_t t0;
    int rows;
    place(i, t0, rows);
    if constexpr (SAVE) {
      if (on)   // the chunk's number: its place in the sequence behind that of the sequence's first
        save(a.save + ((int64_t(seg.seq) + seg.begin / kChunk + (static_cast<int>(t0) - seg.begin) / kChunk) * a.H + h) *
                          head_size);
    }
    float delta, phi, la;
    step_scalars(lo_f32(dtv), bias, Ah, a.softplus, a.zoh, lane < rows, delta, phi, la);
    const DecaySum sum = sum_decays(la);
    const float total = static_cast<float>(sum.all);
    W[lane] = REV ? hw_exp2(static_cast<float>(sum.upto)) : phi * hw_exp2(sum.behind());
    wave_lds_sync();
    const float fade = hw_exp2(total);
#pragma unroll
    for (int kk = 0; kk < 2; ++kk) {
      const pf4 w0 = *reinterpret_cast<const pf4*>(&W[32 * kk + 4 * g4]);
      const pf4 w1 = *reinterpret_cast<const pf4*>(&W[32 * kk + 16 + 4 * g4]);
      Parts w[PT];   // the weighted rows
#pragma unroll
      for (int pt = 0; pt < PT; ++pt) {
        const pu4 v = lds_tr_operand<UV>(V, kk, pt, l16, g4);
        w[pt] = split3(unpack4(v[0], v[1]) * w0, unpack4(v[2], v[3]) * w1);
      }
      if (kk == 1) {
        wait_lds();
        copy_v(i + 1);   // every read of this chunk's rows has its value
      }
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        const pu4 b = lds_tr_plain_operand<U, false>(K, kk, nt, l16, g4);
#pragma unroll
        for (int pt = 0; pt < PT; ++pt) {
          pf4 v = kk == 0 ? S[nt][pt] * fade : S[nt][pt];
#pragma unroll
          for (int i = 0; i < 3; ++i) v = mma(w[pt].p[i], b, v);
          S[nt][pt] = v;
        }
      }
    }
    decay += total;
    return dt_next;
  };

  uint32_t dtv = load_dt(0);
  copy_k(0, sK0);
  copy_v(0);
  for (int i = 0; i < nchunks; i += 2) {
    dtv = chunk(i, sK0, sK1, dtv);
    if (i + 1 < nchunks) dtv = chunk(i + 1, sK1, sK0, dtv);
  }
  wait_memory();   // (the copies issued past the last chunk)

  if (!on) return;
  if constexpr (!SAVE) {
    put(a.ws_state + (kept * a.H + h) * head_size);
    if (p0 == 0 && lane == 0) a.ws_decay[kept * a.H + h] = decay;
  } else if (a.last && seg.index == (REV ? 0 : seg.count - 1)) {
    put(a.last + (int64_t(seg.seq) * a.H + h) * head_size);
  }
}

// The walk over states (f) and, in blocks of y = 1, the one over adjoints in reverse order (r), which do not depend on each
// other: side by side they fill the CUs that either one's last round leaves idle.
template <int N, bool SAVE>
__global__ void __launch_bounds__(kWalkWaves * 64) __attribute__((amdgpu_waves_per_eu(N == 256 ? 2 : 4, N == 256 ? 2 : 4)))
packed_states_kernel(StatesArgs f, StatesArgs r) {
  __shared__ alignas(16) uint16_t sK0[kChunk * N], sK1[kChunk * N];
  __shared__ alignas(16) uint16_t sV[kWalkWaves][kChunk * 16 * PT];
  __shared__ alignas(16) float sW[kWalkWaves][kChunk];
  const int wave = __builtin_amdgcn_readfirstlane(static_cast<int>(threadIdx.x) >> 6);
  if (blockIdx.y == 0) walk<N, false, SAVE>(f, sK0, sK1, sV[wave], sW[wave]);
  else walk<N, true, SAVE>(r, sK0, sK1, sV[wave], sW[wave]);
}

// Joins the segments of a sequence in walk order: the end state that the first pass left for a segment (from zero) gives
// way to the state entering the segment.  A thread owns four entries; nothing to do for one segment.
__global__ void __launch_bounds__(256) packed_join_kernel(StatesArgs f, StatesArgs r, int entries) {
  const bool rev = blockIdx.z != 0;
  const StatesArgs& a = rev ? r : f;
  Piece seg;
  pieces_of(a.cu, blockIdx.x, a.T, a.cps * kChunk, seg);
  const int count = seg.count;
  if (count <= 1) return;
  const int64_t e = (int64_t(blockIdx.y) * 256 + threadIdx.x) * 4;
  const int64_t per = int64_t(a.H) * entries;
  if (e >= per) return;
  const int h = static_cast<int>(e / entries);
  pf4 s = {0.0f, 0.0f, 0.0f, 0.0f};
  if (a.init && (!a.has || a.has[seg.seq])) {
    const int64_t slot = slot_of(a.idx, seg.seq, a.nslots);
    if (slot >= 0) s = *reinterpret_cast<const pf4*>(a.init + slot * per + e);
  }
  constexpr int kAhead = 8;   // segments whose loads are on their way together (65537 tokens of 24 heads: 303 us, else 317)
  for (int i = 0; i < count; i += kAhead) {
    pf4 own[kAhead];
    float d[kAhead];
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {   // (the last one's end is not needed: nothing was left there)
      const int64_t j = seg.place + (rev ? count - 1 - min(i + k, count - 2) : min(i + k, count - 2));
      own[k] = *reinterpret_cast<const pf4*>(a.ws_state + j * per + e);
      d[k] = a.ws_decay[j * a.H + h];
    }
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      if (i + k >= count) break;
      const int64_t j = seg.place + (rev ? count - 1 - i - k : i + k);
      *reinterpret_cast<pf4*>(a.ws_state + j * per + e) = s;
      s = s * hw_exp2(d[k]) + own[k];
    }
  }
}

template <int N>
ssm_status launch_states_of(const StatesArgs& f, const StatesArgs& r, int walks, bool split, hipStream_t st) {
  const dim3 grid(f.nseg * f.G * f.hblocks, walks), block(kWalkWaves * 64);
  if (split) {
    hipLaunchKernelGGL((packed_states_kernel<N, false>), grid, block, 0, st, f, r);
    const int64_t entries = int64_t(kHead) * N;
    hipLaunchKernelGGL(packed_join_kernel, dim3(f.S, static_cast<uint32_t>((f.H * entries / 4 + 255) / 256), walks),
                       dim3(256), 0, st, f, r, static_cast<int>(entries));
  }
  if (f.save) hipLaunchKernelGGL((packed_states_kernel<N, true>), grid, block, 0, st, f, r);
  const hipError_t e = hipGetLastError();
  return e == hipSuccess ? SSM_OK : fail(SSM_ERR_HIP, "packed SSD states launch: %s", hipGetErrorString(e));
}

}  // namespace

ssm_status launch_states(const StatesArgs& f, const StatesArgs* r, int dstate, bool split, hipStream_t st) {
  const int walks = r ? 2 : 1;
  const StatesArgs& back = r ? *r : f;
  switch (dstate) {
    case 64: return launch_states_of<64>(f, back, walks, split, st);
    case 128: return launch_states_of<128>(f, back, walks, split, st);
    default: return launch_states_of<256>(f, back, walks, split, st);
  }
}

}  // namespace ssm57
