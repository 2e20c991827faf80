// Linear attention with a decay for each head over a packed batch: the states in front of the segments, and the
// outputs of a walk over each (see linear.hpp).
#include "launch.hpp"
#include "linear.hpp"

namespace rs {

namespace {

constexpr int kWaves = 4;  // of a workgroup, which share their key head's rows
constexpr int kThreads = kWaves * 64;

// ---- what each segment adds to the state --------------------------------------

template <typename T, int DK>
struct StatesLds {
  using Rows = Tile<kWide<DK>, Parts<T>::in>;
  static constexpr int y = 0, z = y + Rows::kBytes, scalars = z + kWaves * Values<T>::kBytes,
                       total = scalars + kWaves * (int)sizeof(RowScalars);
};

template <typename T, int DK>
__global__ void __launch_bounds__(kThreads) linear_states_kernel(const LinearArgs a, const Side d, int chunks) {
  using L = StatesLds<T, DK>;
  extern __shared__ __align__(16) char lds[];
  const int chunk = blockIdx.x % chunks, hk = blockIdx.x / chunks % a.Hk, b = blockIdx.x / chunks / a.Hk;
  const Segment seg = linear_segment(a, b);
  if (!seg.ok || seg.index == (d.reverse ? 0 : seg.count - 1)) return;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), g = lane >> 4;
  const Place at = place_of<T>(a, hk, chunk * kWaves + wave);
  const typename L::Rows Y(lds + L::y);
  const Values<T> Z(lds + L::z + wave * Values<T>::kBytes);
  RowScalars* rows = reinterpret_cast<RowScalars*>(lds + L::scalars) + wave;
  const T* y = static_cast<const T*>(d.y) + (int64_t)hk * DK;
  const T* z = static_cast<const T*>(d.z) + (int64_t)at.head * a.dv + at.row0;
  KeyMajor<T, DK> state;
  state.zero();
  double all = 0.0;
  for (Blocks blk(seg, d.reverse); blk.more(); blk.next()) {
    __syncthreads();
    stage_rows<T, DK>(Y, y, d.y_stride, blk, kThreads);
    stage_values<T>(Z, z, d.z_stride, blk, at.columns);
    const double end = row_scalars(a, d, blk, seg.end, at.head, rows);
    all += end;
    __syncthreads();
    const float whole = expf((float)end);
#pragma unroll
    for (int m = 0; m < kTiles<T>; ++m)
      if (16 * m < at.columns) {
        Split<kMid> w[2];
#pragma unroll
        for (int ks = 0; ks < 2; ++ks) w[ks] = weighted<T>(Z.template read<false>(m, ks, lane), rows->last, ks, g);
        state.update(m, whole, Y, w);
      }
  }
  if (!at.live) return;
  state.store(d.starts + (((int64_t)b * a.H + at.head) * a.dv + at.row0) * DK, at.columns, 1.f);
  if (lane == 0 && at.row0 == 0) d.decays[(int64_t)b * a.H + at.head] = expf((float)all);
}

// ---- the states in front of the segments ------------------------------------------
// One thread per four entries of a sequence's states: start <- decay start + what the segment adds, in place.

__global__ void __launch_bounds__(256) linear_join_kernel(const LinearArgs a, const Side d) {
  int b0;
  const Segment seq = linear_sequence(a, blockIdx.y, &b0);
  if (!seq.ok || seq.count < 2) return;
  const int64_t size = (int64_t)a.H * a.dv * a.dk;
  const int64_t at = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 4;
  if (at >= size) return;
  const int h = (int)(at / (a.dv * a.dk));
  f32x4 state = d.first ? ld4(d.first + seq.s * size + at) : f32x4{};
  const int step = d.reverse ? -1 : 1;
  int b = d.reverse ? b0 + seq.count - 1 : b0;
  f32x4 add = ld4(d.starts + b * size + at);
  for (int i = 0; i < seq.count; ++i, b += step) {
    f32x4 next{};
    if (i + 2 < seq.count) next = ld4(d.starts + (b + step) * size + at);  // (the last segment's is not there)
    st4(d.starts + b * size + at, state);
    if (i + 1 < seq.count) state = state * d.decays[(int64_t)b * a.H + h] + add;
    add = next;
  }
}

// ---- the outputs ----------------------------------------------------------------------

template <typename T, int DK>
struct OutLds {
  using Rows = Tile<kWide<DK>, Parts<T>::in>;
  static constexpr int x = 0, y = x + Rows::kBytes, z = y + Rows::kBytes, scalars = z + kWaves * Values<T>::kBytes,
                       total = scalars + kWaves * (int)sizeof(RowScalars);
  static_assert(total <= 160 * 1024, "the LDS of a compute unit");
};

// Frag of P^T for rows 16 rt + n and columns 32 ks + 8 g ..: which of the six it is (ks <= rt / 2).
__device__ __forceinline__ constexpr int p_frag(int rt, int ks) { return rt < 2 ? rt : 2 + 2 * (rt - 2) + ks; }

template <typename T>
__device__ __forceinline__ void store4(T* p, const f32x4& x) {
  typedef T vec __attribute__((ext_vector_type(4)));
  *reinterpret_cast<vec*>(p) = __builtin_convertvector(x, vec);
}

// Sequences without tokens, and the flag of those whose tables are bad.
template <typename T>
__device__ __forceinline__ void linear_empty(const LinearArgs& a, const Side& d, int s, int hk, int chunk) {
  int b0;
  const Segment seq = linear_sequence(a, s, &b0);
  if (!seq.ok) {
    if (threadIdx.x == 0 && hk == 0 && chunk == 0) atomicOr(a.err, REPLAYSSM_DEVERR_RANGE);
    return;
  }
  if (seq.count != 0 || d.last == nullptr || d.last == d.first) return;
  const Place at = place_of<T>(a, hk, chunk * kWaves + (threadIdx.x >> 6));
  if (!at.live) return;
  const int64_t base = (((int64_t)s * a.H + at.head) * a.dv + at.row0) * a.dk;
  for (int i = (threadIdx.x & 63) * 4; i < at.columns * a.dk; i += 256)
    st4(d.last + base + i, d.first ? ld4(d.first + base + i) : f32x4{});
}

template <typename T, int DK>
__global__ void __launch_bounds__(kThreads) linear_out_kernel(const LinearArgs a, const Side d, const void* xs, int64_t x_stride, void* outs,
                                                              int chunks) {
  constexpr int in = Parts<T>::in, low = Parts<T>::low;
  constexpr int kK = kWide<DK> / 32;
  using L = OutLds<T, DK>;
  extern __shared__ __align__(16) char lds[];
  const int chunk = blockIdx.x % chunks, hk = blockIdx.x / chunks % a.Hk, b = blockIdx.x / chunks / a.Hk;
  if (b >= a.max_segments) return linear_empty<T>(a, d, b - a.max_segments, hk, chunk);
  const Segment seg = linear_segment(a, b);
  if (!seg.ok) return;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int n = lane & 15, g = lane >> 4;
  const Place at = place_of<T>(a, hk, chunk * kWaves + wave);
  const typename L::Rows X(lds + L::x), Y(lds + L::y);
  const Values<T> Z(lds + L::z + wave * Values<T>::kBytes);
  RowScalars* rows = reinterpret_cast<RowScalars*>(lds + L::scalars) + wave;
  const T* x = static_cast<const T*>(xs) + (int64_t)hk * DK;
  const T* y = static_cast<const T*>(d.y) + (int64_t)hk * DK;
  const int64_t head = (int64_t)at.head * a.dv + at.row0;
  const T* z = static_cast<const T*>(d.z) + head;
  T* out = static_cast<T*>(outs) + head;
  const float skip = a.skip ? a.skip[at.head] : 0.f;
  const bool closes = seg.index == (d.reverse ? 0 : seg.count - 1);
  KeyMajor<T, DK> state;
  {
    const int64_t one = (int64_t)a.H * a.dv * DK, off = head * DK;
    if (seg.count > 1)
      state.load(d.starts + b * one + off, at.columns);
    else if (d.first)
      state.load(d.first + seg.s * one + off, at.columns);
    else
      state.zero();
  }
  const bool keep = closes && d.last != nullptr;
  for (Blocks blk(seg, d.reverse); blk.more(); blk.next()) {
    __syncthreads();
    stage_rows<T, DK>(X, x, x_stride, blk, kThreads);
    stage_rows<T, DK>(Y, y, d.y_stride, blk, kThreads);
    stage_values<T>(Z, z, d.z_stride, blk, at.columns);
    const double end = row_scalars(a, d, blk, seg.end, at.head, rows);
    __syncthreads();
    const float whole = expf((float)end);
    // P[r][c] = row_r col_c e^{G_r - G_c} (x_r . y_c), with the skip weight on the diagonal
    Split<low> P[6];
#pragma unroll
    for (int rt = 0; rt < 4; ++rt) {
      const int r = 16 * rt + n;
      const double Gr = rows->G[r];
      const float row = rows->row[r];
#pragma unroll
      for (int ks = 0; ks <= rt / 2; ++ks) {
        f32x4 t0{}, t1{};
#pragma unroll
        for (int k = 0; k < kK; ++k) {
          const Split<in> xr = X.row8(r, k, g);
          t0 = mma(Y.row8(dealt(2 * ks, n), k, g), xr, t0);
          t1 = mma(Y.row8(dealt(2 * ks + 1, n), k, g), xr, t1);
        }
        f32x8 p = join(t0, t1);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const int c = 32 * ks + 8 * g + e;
          const float w = expf((float)(Gr - rows->G[c])) * rows->col[c] * row;
          p[e] = c <= r ? p[e] * w : 0.f;
          if (c == r) p[e] += skip;
        }
        P[p_frag(rt, ks)] = split8<low>(p);
      }
    }
    const bool update = keep || !blk.final();
#pragma unroll
    for (int m = 0; m < kTiles<T>; ++m) {
      if (16 * m < at.columns) {
        f32x4 acc[4];
#pragma unroll
        for (int rt = 0; rt < 4; ++rt) acc[rt] = f32x4{};
#pragma unroll
        for (int k = 0; k < kK; ++k) {
          const Split<low> s = split8<low>(join(state.S[2 * k][m], state.S[2 * k + 1][m]));
#pragma unroll
          for (int rt = 0; rt < 4; ++rt) acc[rt] = mma(s, X.row8(16 * rt + n, k, g), acc[rt]);
        }
#pragma unroll
        for (int rt = 0; rt < 4; ++rt) acc[rt] *= rows->first[16 * rt + n] * rows->row[16 * rt + n];
        Raw8<T> v[2];
#pragma unroll
        for (int ks = 0; ks < 2; ++ks) v[ks] = Z.template read<false>(m, ks, lane);
#pragma unroll
        for (int ks = 0; ks < 2; ++ks) {
          const Split<in> vs = v[ks].split();
#pragma unroll
          for (int rt = 2 * ks; rt < 4; ++rt) acc[rt] = mma(vs, P[p_frag(rt, ks)], acc[rt]);
        }
        if (at.live) {
#pragma unroll
          for (int rt = 0; rt < 4; ++rt)
            if (16 * rt + n < blk.n) store4(out + blk.token(16 * rt + n) * a.H * a.dv + 16 * m + 4 * g, acc[rt]);
        }
        if (update) {
          Split<kMid> w[2];
#pragma unroll
          for (int ks = 0; ks < 2; ++ks) w[ks] = weighted<T>(v[ks], rows->last, ks, g);
          state.update(m, whole, Y, w);
        }
      }
    }
  }
  if (keep && at.live) {
    // backwards the first token's own decay lies between it and the state in front of it
    const float decay = d.reverse ? expf((float)closed_gate(a.g[(int64_t)seg.begin * a.H + at.head])) : 1.f;
    state.store(d.last + ((int64_t)seg.s * a.H * a.dv + head) * DK, at.columns, decay);
  }
}

int item_chunks(const LinearArgs& a, int slice) { return (a.H / a.Hk * slices_of(a.dv, slice) + kWaves - 1) / kWaves; }

template <typename T, int DK>
hipError_t start_states(const LinearArgs& a, const Side& d, hipStream_t s) {
  const int chunks = item_chunks(a, kSlice<T>);
  constexpr auto kernel = linear_states_kernel<T, DK>;
  const hipError_t e = allow_lds<decltype(kernel), kernel>(StatesLds<T, DK>::total);
  if (e != hipSuccess) return e;
  kernel<<<dim3((unsigned)(a.max_segments * a.Hk * chunks)), dim3(kThreads), StatesLds<T, DK>::total, s>>>(a, d, chunks);
  return hipGetLastError();
}

template <typename T, int DK>
hipError_t start_out(const LinearArgs& a, const Side& d, const void* x, int64_t x_stride, void* out, hipStream_t s) {
  const int chunks = item_chunks(a, kSlice<T>);
  constexpr auto kernel = linear_out_kernel<T, DK>;
  const hipError_t e = allow_lds<decltype(kernel), kernel>(OutLds<T, DK>::total);
  if (e != hipSuccess) return e;
  kernel<<<dim3((unsigned)((a.max_segments + a.n_seqs) * a.Hk * chunks)), dim3(kThreads), OutLds<T, DK>::total, s>>>(
      a, d, x, x_stride, out, chunks);
  return hipGetLastError();
}

// f(type, key size) with both as compile-time values
template <typename F>
hipError_t by_type(const LinearArgs& a, const F& f) {
  const auto keys = [&](auto type) {
    switch (a.dk) {
      case 16: return f(type, std::integral_constant<int, 16>());
      case 32: return f(type, std::integral_constant<int, 32>());
      case 64: return f(type, std::integral_constant<int, 64>());
      default: return f(type, std::integral_constant<int, 128>());
    }
  };
  switch (a.dtype) {
    case REPLAYSSM_BF16: return keys(Bf16());
    case REPLAYSSM_F16: return keys(F16());
    default: return keys(F32());
  }
}

}  // namespace

hipError_t linear_starts(const LinearArgs& a, const Side& d, hipStream_t s) {
  if (a.n_tokens <= a.segment) return hipSuccess;
  hipError_t e = by_type(a, [&](auto type, auto dk) { return start_states<typename decltype(type)::type, decltype(dk)::value>(a, d, s); });
  if (e != hipSuccess) return e;
  const int64_t quads = (int64_t)a.H * a.dv * a.dk / 4;
  linear_join_kernel<<<dim3((unsigned)((quads + 255) / 256), (unsigned)a.n_seqs), dim3(256), 0, s>>>(a, d);
  return hipGetLastError();
}

hipError_t linear_out(const LinearArgs& a, const Side& d, const void* x, int64_t x_stride, void* out, hipStream_t s) {
  return by_type(a, [&](auto type, auto dk) { return start_out<typename decltype(type)::type, decltype(dk)::value>(a, d, x, x_stride, out, s); });
}

// Blocks of 64 tokens are dealt so that about two thousand wavefronts (two a SIMD) each walk one segment: shorter ones cost
// memory for the states between them, longer ones leave compute units idle.
int linear_segment_for(const replayssm_linear_config& c) {
  const int slice = c.dtype == REPLAYSSM_BF16 ? kSlice<__bf16> : kSlice<float>;
  const int64_t work = (c.n_tokens + kRows - 1) / kRows * c.H * slices_of(c.dv, slice);
  int blocks = 4;
  while (blocks < 64 && work >= (int64_t)blocks * 2 * 2048) blocks *= 2;
  while (blocks < 1024 && c.H * (c.n_tokens / (blocks * kRows) + c.n_seqs) * ((c.dv + 31) / 32) > (int64_t)1 << 23) blocks *= 2;
  return blocks * kRows;
}

static int64_t padded(int64_t bytes) { return (bytes + 255) & ~(int64_t)255; }

int64_t linear_side_bytes(const replayssm_linear_config& c, int max_segments) {
  if (c.n_tokens <= c.segment) return 0;
  return padded((int64_t)max_segments * c.H * c.dv * c.dk * 4) + padded((int64_t)max_segments * c.H * 4);
}

int64_t linear_forward_bytes(const replayssm_linear_config& c, int max_segments) { return linear_side_bytes(c, max_segments); }

hipError_t launch_linear_prompt(const LinearArgs& a, hipStream_t s) {
  Side d{};
  d.y = a.k;
  d.y_stride = a.k_stride;
  d.z = a.v;
  d.z_stride = a.v_stride;
  d.beta = a.beta;
  d.weight = 1.f;
  d.row = nullptr;
  d.row_weight = a.scale;
  d.first = a.S0;
  d.last = a.S_out;
  d.starts = static_cast<float*>(a.ws);
  d.decays = d.starts + padded((int64_t)a.max_segments * a.H * a.dv * a.dk * 4) / 4;
  d.reverse = 0;
  const hipError_t e = linear_starts(a, d, s);
  return e != hipSuccess ? e : linear_out(a, d, a.q, a.q_stride, a.out, s);
}

}  // namespace rs
