// Gradients of linear attention with a decay for each head over a packed batch (see linear.hpp):
//   1. the states in front of every segment, and the gradients of the states behind them (linear_starts, both ways)
//   2. linear_keys forwards: dq, and per token and head the parts of dg that come from in front of it
//   3. linear_keys backwards: dk, dg and dbeta
//   4. linear_out backwards: dv and dS0
//   5. sums over workgroups: dq and dk of key heads that several workgroups share, dskip
//
// linear_keys multiplies the state from its other side. With u the rows that meet it (do, or v backwards), w those that made it
// (v, or do backwards) and y, e the key-side rows (k and q, or q and k backwards), per block and value head
//     result_r = row_r (e^{G_r} S^T u_r + sum_{c<=r} e^{G_r - G_c} col_c (u_r . w_c) y_c)
// and the result is summed over the value heads of a key head, in a workgroup over its wavefronts.
//
// dg_t = sum over all pairs j < t <= i of E_ij, E_ij = scale e^{G_i - G_j} beta_j (do_i . v_j)(q_i . k_j). Inside a block this is a
// reversed running sum of (what token i has with the tokens in front, E over j < i) minus (what token j has with those
// behind), plus rho, the pairs that span the block's end. Forwards the walk finds, per token, x (pairs with tokens in front of the
// block) and i (pairs inside it), backwards the same towards the end, and rho goes from block to block by
// rho - sum x' + sum x. It starts at a segment's end as e^{g} <S, dS> of the states there, so that rounding does not pile up over a
// long sequence.
#include "launch.hpp"
#include "linear.hpp"

namespace rs {

namespace {

constexpr int kMaxWaves = 8;  // a head of 256 rows

// What linear_keys leaves per token, head and slice: pairs with tokens in front of its block, and inside it.
struct Pairs {
  float outer, inner;
};

struct KeysArgs {
  Side d;
  const void* u;  // [H][dv] rows per token
  const void* w;
  const void* e;  // [Hk][dk] rows per token
  int64_t u_stride, w_stride, e_stride;
  void* out;       // [n_tokens][Hk][dk], or
  float* partial;  // [parts][n_tokens][Hk][dk] where a key head has several workgroups
  Pairs* pairs;    // [slices][n_tokens][H]: written forwards, read backwards
  float* rho;      // [slices][segments][H]: written forwards, read backwards
  const float* other;  // forwards: the other side's starts
  const float* other_first;
  float* skips;  // [slices][segments][H]: sums of u . w, or NULL
  float* dg;
  float* dbeta;
  Deal deal;
};

template <typename T, int DK>
struct KeysLds {
  using Rows = Tile<kWide<DK>, Parts<T>::in>;
  // tiles of 16 rows whose results are summed over the wavefronts at a time (fp32, whose rows fill LDS, takes one)
  static constexpr int kSumTiles = sizeof(T) == 4 ? 1 : 4;
  // a wavefront's results of 16 channels, and, when those have been read, its three sums per row
  static constexpr int kSum = kSumTiles * 64 * 16;
  static constexpr int kWave = Values<T>::kBytes + (int)sizeof(PairScalars) + kSum;
  static_assert(3 * kRows * 4 <= kSum, "room for both");
  static constexpr int y = 0, waves = Rows::kBytes;
  static int total(int n) { return waves + n * kWave; }
};

__device__ __forceinline__ int pair_frag(int rt, int ks) { return rt < 2 ? rt : 2 + 2 * (rt - 2) + ks; }

// States in registers as [dv][dk]: S[m][i] is the tile of rows dealt(m, .) by dk columns 16 i + n.
template <typename T, int DK>
struct ValueMajor {
  static constexpr int kI = DK / 16, kM = kTiles;
  f32x4 S[kM][kI];
  __device__ __forceinline__ void load(const float* p, int columns) {
    const int lane = threadIdx.x & 63, n = lane & 15, g = lane >> 4;
#pragma unroll
    for (int m = 0; m < kM; ++m)
#pragma unroll
      for (int i = 0; i < kI; ++i)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const int row = dealt(m, 4 * g + r);
          S[m][i][r] = p != nullptr && row < columns ? p[row * DK + 16 * i + n] : 0.f;
        }
  }
  // Sum of products with another state, over the whole wavefront.
  __device__ __forceinline__ float dot(const float* p, int columns) const {
    const int lane = threadIdx.x & 63, n = lane & 15, g = lane >> 4;
    float s = 0.f;
#pragma unroll
    for (int m = 0; m < kM; ++m)
#pragma unroll
      for (int i = 0; i < kI; ++i)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const int row = dealt(m, 4 * g + r);
          if (row < columns) s = __builtin_fmaf(S[m][i][r], p[row * DK + 16 * i + n], s);
        }
    return sum_width<64>(s);
  }
};

template <typename T, int DK, bool BACK>
__global__ void __launch_bounds__(kMaxWaves * 64) linear_keys_kernel(const LinearArgs a, const KeysArgs p) {
  constexpr int in = Parts<T>::in, low = Parts<T>::low;
  constexpr int kK = kWide<DK> / 32, kV = kTiles / 2;
  constexpr int kWhole = 2 * in - 1 > kMid ? kMid : 2 * in - 1;  // products of inputs on the way to dg and dbeta: all (fp32: to 24 bits)
  using L = KeysLds<T, DK>;
  using State = ValueMajor<T, DK>;
  extern __shared__ __align__(16) char lds[];
  const Side& d = p.d;
  const int part = blockIdx.x % p.deal.chunks, hk = blockIdx.x / p.deal.chunks % a.Hk, b = blockIdx.x / p.deal.chunks / a.Hk;
  const Segment seg = linear_segment(a, b);
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int n = lane & 15, g = lane >> 4;
  const Place at = place_of(a, p.deal, hk, part, wave);
  const int slices = p.deal.slices, slice = at.slice;
  if (!seg.ok) {
    if (!BACK && p.skips && at.live && lane == 0) p.skips[((int64_t)slice * a.max_segments + b) * a.H + at.head] = 0.f;
    return;
  }
  char* mine = lds + L::waves + wave * L::kWave;
  const typename L::Rows Y(lds + L::y);
  const Values<T> W(mine);
  PairScalars* rows = reinterpret_cast<PairScalars*>(mine + Values<T>::kBytes);
  const int sum_at = L::waves + Values<T>::kBytes + (int)sizeof(PairScalars);  // of wavefront 0
  const auto sum_of = [&](int w) { return reinterpret_cast<f32x4*>(lds + sum_at + w * L::kWave); };
  const auto red_of = [&](int w) { return reinterpret_cast<float*>(lds + sum_at + w * L::kWave); };
  const T* y = static_cast<const T*>(d.y) + (int64_t)hk * DK;
  const T* e = static_cast<const T*>(p.e) + (int64_t)hk * DK;
  const int64_t head = (int64_t)at.head * a.dv + at.row0;
  const T* u = static_cast<const T*>(p.u) + head;
  const T* w = static_cast<const T*>(p.w) + head;
  const int64_t one = (int64_t)a.H * a.dv * DK, off = head * DK;
  State state;
  state.load(seg.count > 1 ? d.starts + b * one + off : d.first ? d.first + seg.s * one + off : nullptr, at.columns);
  // BACK: pairs that span the end of the block walked now
  double rho = 0.0;
  if (BACK && slice == 0) {
    for (int s = 0; s < slices; ++s) rho += (double)p.rho[((int64_t)s * a.max_segments + b) * a.H + at.head];
  }
  float skips = 0.f;
  RowFeed<T, DK> yf(y, d.y_stride, BACK);
  ValueFeed<T> wf(w, p.w_stride, BACK, at.columns);
  ScalarFeed scalars(a, d, at.head, seg.end);
  for (Blocks blk(seg, BACK); blk.more(); blk.next()) {
    __syncthreads();
    yf.stage(Y, blk, wave, p.deal.waves * 64);
    wf.stage(W, blk);
    scalars.load(blk);
    const double end = scalars.make(scalars.gates, rows);
    copies_landed();
    __syncthreads();
    const float whole = decay_of(end);
    // this wavefront's rows u, as operands
    Split<in> U[4][kV];
    const int64_t u_step = BACK ? -p.u_stride : p.u_stride, e_step = BACK ? -p.e_stride : p.e_stride;
    const T* u0 = u + blk.token(0) * p.u_stride;
    const T* e0 = e + blk.token(0) * p.e_stride;
#pragma unroll
    for (int rt = 0; rt < 4; ++rt)
#pragma unroll
      for (int ks = 0; ks < kV; ++ks) {
        Raw8<T> x;
        if (16 * rt + n < blk.n && 32 * ks + 8 * g < at.columns)
          x.load(u0 + (16 * rt + n) * u_step + 32 * ks + 8 * g);
        else
          x.zero();
        U[rt][ks] = x.split();
      }
    // pairs inside the block: D[r][c] = col_c e^{G_r - G_c} u_r . w_c, and their sums with e_r . y_c
    Split<low> D[6];
    float inner[4], diag[4], outer[4];
#pragma unroll
    for (int rt = 0; rt < 4; ++rt) {
      inner[rt] = diag[rt] = outer[rt] = 0.f;
      const int r = 16 * rt + n;
      const double Gr = rows->G[r];
#pragma unroll
      for (int ks = 0; ks <= rt / 2; ++ks) {
        f32x4 p0{}, p1{}, t0{}, t1{};
#pragma unroll
        for (int k = 0; k < kV; ++k) {
          p0 = mma_to<kWhole>(value_row<T>(W, dealt(2 * ks, n), k, g).split(), U[rt][k], p0);
          p1 = mma_to<kWhole>(value_row<T>(W, dealt(2 * ks + 1, n), k, g).split(), U[rt][k], p1);
        }
#pragma unroll
        for (int k = 0; k < kK; ++k) {
          Raw8<T> x;
          if (r < blk.n && 32 * k + 8 * g < DK)
            x.load(e0 + r * e_step + 32 * k + 8 * g);
          else
            x.zero();
          const Split<in> er = x.split();
          t0 = mma_to<kWhole>(Y.row8(dealt(2 * ks, n), k, g), er, t0);
          t1 = mma_to<kWhole>(Y.row8(dealt(2 * ks + 1, n), k, g), er, t1);
        }
        f32x8 dp = join(p0, p1);
        const f32x8 tt = join(t0, t1), w8 = pair_weights(rows, rt, ks, n, g) * pair_scale(rows, Gr, rt, ks, n, g);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int c = 32 * ks + 8 * g + i;
          const float x = dp[i] * w8[i];
          if (ks == rt / 2) {
            skips += c == r ? dp[i] : 0.f;
            const float both = x * tt[i];
            diag[rt] += c == r ? both : 0.f;
            inner[rt] += c < r ? both : 0.f;
          } else {
            inner[rt] = __builtin_fmaf(x, tt[i], inner[rt]);
          }
          dp[i] = x;
        }
        D[pair_frag(rt, ks)] = split8<low>(dp);
      }
    }
    // sixteen key channels at a time: their results, summed over the wavefronts, and their columns of the state
#pragma unroll
    for (int i = 0; i < DK / 16; ++i) {
      f32x4 acc[4];
#pragma unroll
      for (int rt = 0; rt < 4; ++rt) acc[rt] = f32x4{};
#pragma unroll
      for (int ks = 0; ks < kV; ++ks)
        if (32 * ks < at.columns) {
          const Split<kMid> s = split8<kMid>(join(state.S[2 * ks][i], state.S[2 * ks + 1][i]));
#pragma unroll
          for (int rt = 0; rt < 4; ++rt) acc[rt] = mma(s, U[rt][ks], acc[rt]);
        }
      Split<in> ys[2];
#pragma unroll
      for (int ks = 0; ks < 2; ++ks) ys[ks] = Y.template col8<false>(i, ks, lane);
#pragma unroll
      for (int rt = 0; rt < 4; ++rt) {
        const int r = 16 * rt + n;
        acc[rt] *= rows->first[r];
        if (r < blk.n) {
          const T* er = e0 + r * e_step + 16 * i + 4 * g;
#pragma unroll
          for (int j = 0; j < 4; ++j) outer[rt] = __builtin_fmaf(acc[rt][j], (float)er[j], outer[rt]);
        }
#pragma unroll
        for (int ks = 0; ks <= rt / 2; ++ks) acc[rt] = mma(ys[ks], D[pair_frag(rt, ks)], acc[rt]);
        acc[rt] *= rows->row[r];
      }
#pragma unroll
      for (int r0 = 0; r0 < 4; r0 += L::kSumTiles) {
#pragma unroll
        for (int rt = 0; rt < L::kSumTiles; ++rt) sum_of(wave)[rt * 64 + lane] = at.live ? acc[r0 + rt] : f32x4{};
        __syncthreads();
        for (int v = threadIdx.x; v < L::kSumTiles * 64; v += p.deal.waves * 64) {
          f32x4 s = sum_of(0)[v];
          for (int k = 1; k < p.deal.waves; ++k) s += sum_of(k)[v];
          const int r = 16 * (r0 + (v >> 6)) + (v & 15), c = 16 * i + 4 * ((v >> 4) & 3);
          if (r < blk.n) {
            const int64_t to = (blk.token(r) * a.Hk + hk) * DK + c;
            if (p.partial) {
              st4(p.partial + part * (a.n_tokens * a.Hk * DK) + to, s);
            } else {
              typedef T vec __attribute__((ext_vector_type(4)));
              *reinterpret_cast<vec*>(static_cast<T*>(p.out) + to) = __builtin_convertvector(s, vec);
            }
          }
        }
        __syncthreads();
      }
    }
    // sums per row, over this head's slices
    float* red = red_of(wave);
#pragma unroll
    for (int rt = 0; rt < 4; ++rt) {
      const float o = sum_groups(outer[rt]), s = sum_groups(inner[rt]), q = sum_groups(diag[rt]);
      if (g == 0) {
        red[16 * rt + n] = o;
        red[kRows + 16 * rt + n] = s;
        red[2 * kRows + 16 * rt + n] = q;
      }
    }
    __syncthreads();
    if (!BACK) {
      if (at.live && lane < blk.n)
        p.pairs[((int64_t)slice * a.n_tokens + blk.token(lane)) * a.H + at.head] =
            Pairs{red[lane] * rows->row[lane], red[kRows + lane] * rows->row[lane]};
    } else if (slice == 0) {
      float o = 0.f, s = 0.f, q = 0.f;
      double x = 0.0, within = 0.0;
      const bool here = lane < blk.n;
      const int64_t to = (here ? blk.token(lane) : blk.t0) * a.H + at.head;
      for (int k = 0; k < slices; ++k) {
        const float* r = red_of(wave + k);
        o += r[lane];
        s += r[kRows + lane];
        q += r[2 * kRows + lane];
        if (here) {
          const Pairs f = p.pairs[k * (a.n_tokens * a.H) + to];
          x += (double)f.outer;
          within += (double)f.inner;
        }
      }
      const double row = rows->row[lane], z = row * o;
      double sum = here ? x + within - z - row * s : 0.0, span = here ? x - z : 0.0;
#pragma unroll
      for (int k = 1; k < 64; k <<= 1) {
        const double up = __shfl_up(sum, k), wide = __shfl_up(span, k);
        if (lane >= k) {
          sum += up;
          span += wide;
        }
      }
      if (here && at.live) {
        p.dg[to] = (float)(rho + sum);
        if (p.dbeta) p.dbeta[to] = o + s + q;
      }
      rho += __shfl(span, 63);
    }
    if (BACK && blk.final()) break;
    // the state behind the block
#pragma unroll
    for (int m = 0; m < kTiles; ++m)
      if (16 * (m & ~1) < at.columns) {
        Split<kMid> z[2];
#pragma unroll
        for (int ks = 0; ks < 2; ++ks) z[ks] = split8<kMid>(W.template read<true>(m, ks, lane).f32() * load8(rows->last + 32 * ks + 8 * g));
#pragma unroll
        for (int i = 0; i < DK / 16; ++i) {
          f32x4 s = state.S[m][i] * whole;
#pragma unroll
          for (int ks = 0; ks < 2; ++ks) s = mma(z[ks], Y.template col8<false>(i, ks, lane), s);
          state.S[m][i] = s;
        }
      }
  }
  if (BACK) return;
  // what the pairs over the segment's end begin with, and the skip weight's gradient
  const int64_t to = ((int64_t)slice * a.max_segments + b) * a.H + at.head;
  const float* behind = seg.count > 1 ? p.other + b * one + off : p.other_first ? p.other_first + seg.s * one + off : nullptr;
  float product = 0.f;
  if (behind) {
    product = state.dot(behind, at.columns);
    if (seg.t1 < seg.end) product *= expf(closed_gate(a.g[seg.t1 * a.H + at.head]));
  }
  skips = sum_width<64>(skips);
  if (lane == 0 && at.live) {
    p.rho[to] = product;
    if (p.skips) p.skips[to] = skips;
  }
}

// dst = sum of the parts, in the type of the gradients, for the tokens of a segment. (Rows of no sequence are left as they were.)
template <typename T>
__global__ void __launch_bounds__(256) linear_sum_kernel(const LinearArgs a, const float* partial, int parts, T* dst) {
  const Segment seg = linear_segment(a, blockIdx.y);
  if (!seg.ok) return;
  const int row = a.Hk * a.dk;
  const int64_t size = a.n_tokens * row, end = seg.t1 * row;
  for (int64_t at = seg.t0 * row + ((int64_t)blockIdx.x * 256 + threadIdx.x) * 8; at < end; at += (int64_t)gridDim.x * 2048) {
    f32x8 s = load8(partial + at);
    for (int p = 1; p < parts; ++p) s += load8(partial + p * size + at);
    store8(dst + at, s);
  }
}

__global__ void __launch_bounds__(256) linear_skip_kernel(const LinearArgs a, const float* skips, int rows) {
  __shared__ double sums[4];
  const int h = blockIdx.x;
  double s = 0.0;
  for (int i = threadIdx.x; i < rows; i += 256) s += (double)skips[(int64_t)i * a.H + h];
#pragma unroll
  for (int k = 32; k > 0; k >>= 1) s += __shfl_xor(s, k);
  if ((threadIdx.x & 63) == 0) sums[threadIdx.x >> 6] = s;
  __syncthreads();
  if (threadIdx.x == 0) a.dskip[h] = (float)((sums[0] + sums[1]) + (sums[2] + sums[3]));
}

// How the value heads of a key head are dealt to workgroups, and what lies where in the workspace.
struct KeysPlan {
  Deal deal;
  int64_t forward, reverse, pairs, rho, skips, partial, total;
};

int64_t padded(int64_t bytes) { return (bytes + 255) & ~(int64_t)255; }

KeysPlan keys_plan(const replayssm_linear_config& c, int max_segments) {
  KeysPlan p;
  p.deal = deal(c.dv, c.H / c.Hk, kMaxWaves, kMaxWaves);
  const int64_t side = linear_side_bytes(c, max_segments), per = padded((int64_t)p.deal.slices * max_segments * c.H * 4);
  p.forward = 0;
  p.reverse = side;
  p.pairs = p.reverse + side;
  p.rho = p.pairs + padded((int64_t)p.deal.slices * c.n_tokens * c.H * sizeof(Pairs));
  p.skips = p.rho + per;
  p.partial = p.skips + per;
  p.total = p.partial + (p.deal.chunks > 1 ? padded((int64_t)p.deal.chunks * c.n_tokens * c.Hk * c.dk * 4) : 0);
  return p;
}

replayssm_linear_config config_of(const LinearArgs& a) {
  replayssm_linear_config c{};
  c.n_seqs = a.n_seqs;
  c.H = a.H;
  c.Hk = a.Hk;
  c.dk = a.dk;
  c.dv = a.dv;
  c.dtype = a.dtype;
  c.n_tokens = a.n_tokens;
  c.segment = a.segment;
  return c;
}

template <typename T, int DK, bool BACK>
hipError_t start_keys(const LinearArgs& a, const KeysArgs& p, hipStream_t s) {
  const int bytes = KeysLds<T, DK>::total(p.deal.waves);
  static_assert(KeysLds<T, DK>::waves + kMaxWaves * KeysLds<T, DK>::kWave <= 160 * 1024, "the LDS of a compute unit");
  constexpr auto kernel = linear_keys_kernel<T, DK, BACK>;
  const hipError_t e = allow_lds<decltype(kernel), kernel>(160 * 1024);
  if (e != hipSuccess) return e;
  kernel<<<dim3((unsigned)(a.max_segments * a.Hk * p.deal.chunks)), dim3(p.deal.waves * 64), bytes, s>>>(a, p);
  return hipGetLastError();
}

template <typename T, bool BACK>
hipError_t keys(const LinearArgs& a, const KeysArgs& p, hipStream_t s) {
  hipError_t e;
  switch (a.dk) {
    case 16: e = start_keys<T, 16, BACK>(a, p, s); break;
    case 32: e = start_keys<T, 32, BACK>(a, p, s); break;
    case 64: e = start_keys<T, 64, BACK>(a, p, s); break;
    default: e = start_keys<T, 128, BACK>(a, p, s);
  }
  if (e != hipSuccess || p.partial == nullptr) return e;
  const int64_t units = ((int64_t)a.segment * a.Hk * a.dk + 2047) / 2048;
  linear_sum_kernel<T><<<dim3((unsigned)(units < 1024 ? units : 1024), (unsigned)a.max_segments), dim3(256), 0, s>>>(a, p.partial, p.deal.chunks,
                                                                                                                  static_cast<T*>(p.out));
  return hipGetLastError();
}

template <bool BACK>
hipError_t keys_by_type(const LinearArgs& a, const KeysArgs& p, hipStream_t s) {
  switch (a.dtype) {
    case REPLAYSSM_BF16: return keys<__bf16, BACK>(a, p, s);
    case REPLAYSSM_F16: return keys<_Float16, BACK>(a, p, s);
    default: return keys<float, BACK>(a, p, s);
  }
}

}  // namespace

int64_t linear_backward_bytes(const replayssm_linear_config& c, int max_segments) { return keys_plan(c, max_segments).total; }

hipError_t launch_linear_prompt_backward(const LinearArgs& a, hipStream_t s) {
  const replayssm_linear_config c = config_of(a);
  const KeysPlan plan = keys_plan(c, a.max_segments);
  char* ws = static_cast<char*>(a.ws);
  const int64_t states = padded((int64_t)a.max_segments * a.H * a.dv * a.dk * 4);
  Side f{}, r{};
  f.y = a.k;
  f.y_stride = a.k_stride;
  f.z = a.v;
  f.z_stride = a.v_stride;
  f.beta = a.beta;
  f.weight = 1.f;
  f.row_weight = a.scale;
  f.first = a.S0;
  f.starts = reinterpret_cast<float*>(ws + plan.forward);
  f.decays = reinterpret_cast<float*>(ws + plan.forward + states);
  r.y = a.q;
  r.y_stride = a.q_stride;
  r.z = a.dout;
  r.z_stride = (int64_t)a.H * a.dv;
  r.weight = a.scale;
  r.row = a.beta;
  r.row_weight = 1.f;
  r.first = a.dS_out;
  r.last = a.dS0;
  r.starts = reinterpret_cast<float*>(ws + plan.reverse);
  r.decays = reinterpret_cast<float*>(ws + plan.reverse + states);
  r.reverse = 1;
  hipError_t e = linear_starts(a, f, s);
  if (e == hipSuccess) e = linear_starts(a, r, s);
  if (e != hipSuccess) return e;
  KeysArgs p{};
  p.deal = plan.deal;
  p.partial = plan.deal.chunks > 1 ? reinterpret_cast<float*>(ws + plan.partial) : nullptr;
  p.pairs = reinterpret_cast<Pairs*>(ws + plan.pairs);
  p.rho = reinterpret_cast<float*>(ws + plan.rho);
  p.skips = a.dskip ? reinterpret_cast<float*>(ws + plan.skips) : nullptr;
  p.d = f;
  p.u = a.dout;
  p.u_stride = r.z_stride;
  p.w = a.v;
  p.w_stride = a.v_stride;
  p.e = a.q;
  p.e_stride = a.q_stride;
  p.out = a.dq;
  p.other = r.starts;
  p.other_first = a.dS_out;
  e = keys_by_type<false>(a, p, s);
  if (e != hipSuccess) return e;
  p.d = r;
  p.u = a.v;
  p.u_stride = a.v_stride;
  p.w = a.dout;
  p.w_stride = r.z_stride;
  p.e = a.k;
  p.e_stride = a.k_stride;
  p.out = a.dk_;
  p.dg = a.dg;
  p.dbeta = a.dbeta;
  e = keys_by_type<true>(a, p, s);
  if (e != hipSuccess) return e;
  e = linear_out(a, r, a.k, a.k_stride, a.dv_, s);
  if (e != hipSuccess || a.dskip == nullptr) return e;
  linear_skip_kernel<<<dim3((unsigned)a.H), dim3(256), 0, s>>>(a, p.skips, plan.deal.slices * a.max_segments);
  return hipGetLastError();
}

}  // namespace rs
