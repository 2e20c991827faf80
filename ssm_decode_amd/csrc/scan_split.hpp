// The serial walk over a sequence's blocks where there are few sequences and heads.
//
// A workgroup takes 16 state rows of one value head (rows are independent) and its four wavefronts
// divide every product of a block by rows of the left operand: wavefront w has the block's 16 dealt
// tokens w for K S, T X, Q S and P U, and a quarter of the channels for the update. What a wavefront
// reads from memory - its rows of K and Q, its fragments of T and P - comes into
// registers and is asked for a block ahead; the rows go to LDS when the block in front is done, for the wavefront's own
// left operands and, transposed, for everybody's channels in the update. The right operands (S, X, U) are
// exchanged through LDS in operand layout, 16 bytes per lane, with three barriers per block.
//
// The lambdas that ask and put are inlined by force: one that is not by the time the arrays are taken apart leaves them in
// scratch memory, and every load is waited for where it is asked for (fp16 and fp32, dk = 128: a block took 10.4 and 14.9 us).
//
// The chain of a block is then 12 + 6..12 + 12 matrix instructions (bf16, dk = 128) and four exchanges. Against the
// kernels whose wavefronts take whole rows through all products (scan_rows.hpp) it reads K, Q, T and P four
// times as often for the same rows, so it is used where those would leave most compute units idle. Measured,
// bf16, 128 x 128, split against rows: one sequence of 32768 tokens, 32 heads, 0.97 against 1.92 ms; 24 ragged
// sequences of 32 heads, 0.52 against 0.33 ms; the backward pass's two walks over 8 sequences of 2048 tokens and 16
// heads, 0.58 against 0.40 ms. Whole calls of 4096 tokens a sequence, with 64 sequences times heads: 272 against 329 us, backward
// 1103 against 1163; with 96: 431 against 374, backward 1663 against 1480.
#pragma once

#include "scan.hpp"

namespace rs {

namespace {

// Workgroup index -> item (sequence and head) and slice of its rows. Workgroups go to the eight dies in turn; the
// slices of one item read the same K, Q, T and P, so they are placed on one die, behind one L2.
__device__ __forceinline__ void item_slice(int slices, int* item, int* slice) {
  const int per = 8 * slices, round = blockIdx.x / per, in_round = blockIdx.x - round * per;
  *slice = in_round / 8;
  *item = round * 8 + (in_round & 7);
}
__host__ __device__ constexpr int64_t item_grid(int64_t items, int slices) { return (items + 7) / 8 * 8 * slices; }

// Right operands in LDS: [step][part][lane] of 16 bytes; a result tile of a pair fills its half of each lane's.
template <int N>
__device__ __forceinline__ void put_half(char* base, int step, int half, int lane, const f32x4& x) {
#pragma clang fp contract(off)
  typedef float f32x2 __attribute__((ext_vector_type(2)));
  typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
  typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
  f32x4 rest = x;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    u32x2 packed;
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const bf16x2 pair = __builtin_convertvector((f32x2{rest[2 * e], rest[2 * e + 1]}), bf16x2);
      packed[e] = __builtin_bit_cast(uint32_t, pair);
      rest[2 * e] -= bf16_lo(packed[e]);
      rest[2 * e + 1] -= bf16_hi(packed[e]);
    }
    *reinterpret_cast<u32x2*>(base + ((step * N + i) * 64 + lane) * 16 + half * 8) = packed;
  }
}
template <int N>
constexpr int kStepBytes = N * 1024;  // of one step's right operand

// A wavefront's 16 dealt rows of a block: loads of whole rows (16 segments of 64 bytes per instruction, as the
// operands want them, made the walk a fifth longer), then stores into a tile of the block, where the
// wavefront finds its left operands and all wavefronts find columns.
template <typename T, int DK>
struct OwnRows {
  static constexpr int kPer = kWide<DK> / 32, kChunks = kWide<DK> / 8, kRows = 64 / kChunks;  // rows per instruction
  using Block = Tile<kWide<DK>, Parts<T>::in>;
  Raw8<T> x[kPer];
  int wave, row, chunk;  // row: the lane's place among the instruction's rows
  __device__ __forceinline__ explicit OwnRows(int w)
      : wave(w), row((threadIdx.x & 63) / kChunks), chunk(threadIdx.x % kChunks) {}
  __device__ __forceinline__ int at(int i) const { return dealt(wave, i * kRows + row); }
  // p: the block's first row; n rows of the block exist (others read the last one, and are zeroed on the way)
  __device__ __forceinline__ void load(const T* p, int64_t stride, int n) {
    const T* q = p + (chunk * 8 < DK ? chunk * 8 : 0);
#pragma unroll
    for (int i = 0; i < kPer; ++i) x[i].load(q + (int64_t)(at(i) < n ? at(i) : n - 1) * stride);
  }
  __device__ __forceinline__ void store(const Block& t, int n) {
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      if (at(i) >= n || chunk * 8 >= DK) x[i].zero();
      t.put(at(i), chunk, x[i].split());
    }
  }
};

template <typename T, int DK>
struct SplitLds {
  static constexpr int in = Parts<T>::in, mid = kMid, low = Parts<T>::low, kSteps = kWide<DK> / 32;
  static constexpr int s = 0, x = s + kSteps * kStepBytes<mid>, u = x + 2 * kStepBytes<mid>,
                       ul = u + 2 * kStepBytes<low>, k = ul + 2 * kStepBytes<mid>,
                       q = k + Tile<kWide<DK>, in>::kBytes,
                       total = q + Tile<kWide<DK>, in>::kBytes;
};

// With KEEP (the backward pass) it writes the state before each block and the block's corrections in place of
// outputs. Outputs are computed transposed (state rows by tokens): the operands of a product can change places, and
// a lane then holds four neighbouring state rows of one token, which it stores in one piece.
template <typename T, int DK, typename Ops, bool KEEP>
__global__ void __launch_bounds__(kChunkThreads, Parts<T>::in == 1 ? 2 : 1)
    delta_scan_split_kernel(const DeltaArgs a, const Kept kept) {
  constexpr int in = Parts<T>::in, mid = kMid, low = Parts<T>::low;
  constexpr int kSteps = kWide<DK> / 32, kTiles = 2 * kSteps;
  constexpr int kOwn = kTiles >= 4 ? kTiles / 4 : 1;  // state tiles of a wavefront
  using L = SplitLds<T, DK>;
  extern __shared__ __align__(16) char lds[];
  const int slices = (a.dv + 15) / 16;
  int item, slice;
  item_slice(slices, &item, &slice);
  if (item >= a.n_seqs * a.H) return;
  const int h = item % a.H, s = by_length(a, item / a.H);
  const SeqRange seq = seq_range(a, s);
  if (!seq.ok) {
    if (threadIdx.x == 0 && slice == 0 && h == 0) atomicOr(a.err, REPLAYSSM_DEVERR_RANGE);
    return;
  }
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int n = lane & 15, g = lane >> 4;
  const int hk = h / (a.H / a.Hk);
  const int col = 16 * slice + n;  // of the head's dv
  const bool live = col < a.dv;
  const int64_t state = ((int64_t)s * a.H + h) * a.dv * DK;
  const int tile0 = wave * kOwn;  // the wavefront's state tiles; with dk <= 32 two wavefronts have none
  const bool owner = tile0 < kTiles;

  // S^T: a tile's rows are channels, dealt; its columns state rows
  const auto channel = [&](int tl) { return 32 * (tl >> 1) + 8 * g + 4 * (tl & 1); };
  f32x4 S[kOwn];
#pragma unroll
  for (int i = 0; i < kOwn; ++i) {
    S[i] = f32x4{0.f, 0.f, 0.f, 0.f};
    const int c = channel(tile0 + i);
    if (owner && a.S0 != nullptr && live && c < DK) S[i] = ld4(a.S0 + state + (int64_t)col * DK + c);
    if (owner) put_half<mid>(lds + L::s, (tile0 + i) >> 1, (tile0 + i) & 1, lane, S[i]);
  }

  const T* kp = static_cast<const T*>(a.k) + (int64_t)hk * DK;
  const T* qp = static_cast<const T*>(a.q) + (int64_t)hk * DK;
  const T* vp = static_cast<const T*>(a.v) + (int64_t)h * a.dv;
  const int64_t out_stride = (int64_t)a.H * a.dv;
  const int out_col = 16 * slice + 4 * g;  // the first of the lane's neighbouring output rows
  T* op = static_cast<T*>(a.out) + (int64_t)h * a.dv + out_col;
  const char* ws = static_cast<const char*>(a.ws) + ((int64_t)seq.block0 * a.H + h) * Ops::bytes;
  const int64_t ws_step = (int64_t)a.H * Ops::bytes;

  OwnRows<T, DK> K(wave), Q(wave);
  const typename OwnRows<T, DK>::Block Kt(lds + L::k), Qt(lds + L::q);
  Split<mid> tf[2];
  Split<low> pf[2];
  T v[4];
  // A block's scalars: of the lane's four tokens (rows of a result tile), of token dealt(wave, n), and of the block.
  // Two sets, of even and odd blocks: one is still in use when the next is asked for.
  f32x4 first4[2], last4[2];
  float first1[2], whole[2];
  const int row4 = dealt(wave, 4 * g);
  const auto token = [&](int c) { return (int64_t)seq.begin + (int64_t)c * kBlock; };
  const auto rows_of = [&](int c) {
    const int64_t left = seq.end - token(c);
    return left < kBlock ? (int)left : kBlock;
  };
  const auto ask_rows = [&](int c) __attribute__((always_inline)) {
    K.load(kp + token(c) * a.k_stride, a.k_stride, rows_of(c));
    if constexpr (!KEEP) Q.load(qp + token(c) * a.q_stride, a.q_stride, rows_of(c));
  };
  const auto ask_values = [&](int c, int set) __attribute__((always_inline)) {
    const int rows = rows_of(c);
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const T* p = vp + (token(c) + (row4 + r < rows ? row4 + r : rows - 1)) * a.v_stride;
      v[r] = p[live ? col : 0];
    }
    const BlockScalars* sc = reinterpret_cast<const BlockScalars*>(ws + c * ws_step + Ops::scalars);
    first4[set] = ld4(sc->first + row4);
    last4[set] = ld4(sc->last + row4);
    first1[set] = sc->first[dealt(wave, n)];
    whole[set] = sc->first[kBlock - 1];
  };
  const auto ask_t = [&](int c) __attribute__((always_inline)) {
#pragma unroll
    for (int p = 0; p < 2; ++p)
      tf[p] = get_frag<mid>(ws + c * ws_step + Ops::t, lower_frag(wave, p <= wave / 2 ? p : 0), lane);
  };
  const auto ask_p = [&](int c) __attribute__((always_inline)) {
    if constexpr (!KEEP) {
#pragma unroll
      for (int p = 0; p < 2; ++p)
        pf[p] = get_frag<low>(ws + c * ws_step + Ops::p, lower_frag(wave, p <= wave / 2 ? p : 0), lane);
    }
  };
  const auto put_rows = [&](int c) __attribute__((always_inline)) {
    K.store(Kt, rows_of(c));
    if constexpr (!KEEP) Q.store(Qt, rows_of(c));
  };
  if (seq.blocks > 0) {
    ask_rows(0);
    ask_values(0, 0);
    ask_t(0);
    ask_p(0);
  }
  if (!owns(a, s, seq)) {
    if (slice == 0) skip_sequence<Ops>(a, s, seq, h);
    return;
  }
  if (seq.blocks > 0) put_rows(0);
  const auto block = [&](int c, int set) __attribute__((always_inline)) {
    const int rows = rows_of(c);
    const int64_t t0 = token(c);
    // (The last block asks for itself again. Loads under a condition would join their registers with the old ones
    // by moves, and a move waits for the load right where it was asked for.)
    const int next = c + 1 < seq.blocks ? c + 1 : c;
    const int64_t place = (int64_t)(seq.block0 + c) * a.H + h;
    const int own = dealt(wave, n);
    Split<in> kf[kSteps];
#pragma unroll
    for (int ks = 0; ks < kSteps; ++ks) kf[ks] = Kt.row8(own, ks, g);  // (the wavefront's own)
    __syncthreads();  // S and K are there
    ask_rows(next);  // (asked for after Q S, a block took 0.2 us longer)
    f32x4 y = {0.f, 0.f, 0.f, 0.f}, o = y;
    {
      Split<mid> bs[kSteps];
#pragma unroll
      for (int ks = 0; ks < kSteps; ++ks) bs[ks] = get_frag<mid>(lds + L::s, ks, lane);
#pragma unroll
      for (int ks = 0; ks < kSteps; ++ks) y = mma(kf[ks], bs[ks], y);
      // (the chain goes on from y; Q S fills the time of its exchange)
      f32x4 x;
#pragma unroll
      for (int r = 0; r < 4; ++r) x[r] = fused(-first4[set][r], y[r], row4 + r < rows && live ? (float)v[r] : 0.f);
      put_half<mid>(lds + L::x, wave >> 1, wave & 1, lane, x);  // (beta is in T's columns)
      if constexpr (!KEEP) {
#pragma unroll
        for (int ks = 0; ks < kSteps; ++ks) {
          const Split<in> qf = Qt.row8(own, ks, g);
          products<in, low>([&](int i, int j) { o = mfma(bs[ks].p[j], qf.p[i], o); });
        }
      }
    }
    ask_values(next, set ^ 1);
    __syncthreads();  // X is there
    f32x4 U = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int p = 0; p < 2; ++p)
      if (p <= wave / 2) U = mma(tf[p], get_frag<mid>(lds + L::x, p, lane), U);
    put_half<mid>(lds + L::ul, wave >> 1, wave & 1, lane, last4[set] * U);
    if constexpr (!KEEP) put_half<low>(lds + L::u, wave >> 1, wave & 1, lane, U);
    // the update's left operands, transposed
    Split<in> kc[kOwn][2];
    if (owner) {
#pragma unroll
      for (int i = 0; i < kOwn; ++i)
#pragma unroll
        for (int p = 0; p < 2; ++p) kc[i][p] = Kt.template col8<true>(tile0 + i, p, lane);
    }
    ask_t(next);
    if (KEEP && live) {
      if (owner) {
#pragma unroll
        for (int i = 0; i < kOwn; ++i)
          if (channel(tile0 + i) < DK) st4(kept.S + (place * a.dv + col) * DK + channel(tile0 + i), S[i]);
      }
#pragma unroll
      for (int r = 0; r < 4; ++r) kept.U[(place * kBlock + row4 + r) * a.dv + col] = U[r];
    }
    __syncthreads();  // U is there
    if (owner) {
#pragma unroll
      for (int i = 0; i < kOwn; ++i) S[i] *= whole[set];
#pragma unroll
      for (int p = 0; p < 2; ++p) {
        const Split<mid> ul = get_frag<mid>(lds + L::ul, p, lane);
#pragma unroll
        for (int i = 0; i < kOwn; ++i) S[i] = mma(kc[i][p], ul, S[i]);
      }
#pragma unroll
      for (int i = 0; i < kOwn; ++i)
        put_half<mid>(lds + L::s, (tile0 + i) >> 1, (tile0 + i) & 1, lane, S[i]);
    }
    put_rows(next);  // (the update's operands have been read)
    if constexpr (!KEEP) {  // (scale is in P)
      o *= a.scale * first1[set];
#pragma unroll
      for (int p = 0; p < 2; ++p)
        if (p <= wave / 2) o = mma(get_frag<low>(lds + L::u, p, lane), pf[p], o);
      if (out_col < a.dv && dealt(wave, n) < rows) {
        T* dst = op + (t0 + dealt(wave, n)) * out_stride;
        typedef T vec __attribute__((ext_vector_type(4)));
        *reinterpret_cast<vec*>(dst) = __builtin_convertvector(o, vec);
      }
      ask_p(next);
    }
  };
  for (int c = 0; c < seq.blocks; c += 2) {
    block(c, 0);
    if (c + 1 < seq.blocks) block(c + 1, 1);
  }
  if (a.S_out == nullptr || KEEP || !owner) return;
#pragma unroll
  for (int i = 0; i < kOwn; ++i)
    if (live && channel(tile0 + i) < DK)
      st4(a.S_out + state + (int64_t)col * DK + channel(tile0 + i), S[i]);
}

template <typename T, int DK, typename Ops, bool KEEP>
hipError_t launch_scan_split(const DeltaArgs& a, const Kept& kept, hipStream_t s) {
  using L = SplitLds<T, DK>;
  constexpr auto kernel = delta_scan_split_kernel<T, DK, Ops, KEEP>;
  const hipError_t e = allow_lds<decltype(kernel), kernel>(L::total);
  if (e != hipSuccess) return e;
  const int slices = (a.dv + 15) / 16;
  kernel<<<dim3((unsigned)item_grid((int64_t)a.n_seqs * a.H, slices)), dim3(kChunkThreads), L::total, s>>>(a, kept);
  return hipGetLastError();
}

template <typename T, int DK>
struct ReverseSplitLds {
  static constexpr int in = Parts<T>::in, mid = kMid, kSteps = kWide<DK> / 32;
  // dS; dO; e^G d; dU; -e^G beta dX
  static constexpr int s = 0, d = s + kSteps * kStepBytes<mid>, df = d + 2 * kStepBytes<in>,
                       u = df + 2 * kStepBytes<mid>, x = u + 2 * kStepBytes<mid>,
                       k = x + 2 * kStepBytes<mid>, q = k + Tile<kWide<DK>, in>::kBytes,
                       total = q + Tile<kWide<DK>, in>::kBytes;
};

// The scan's division of labour, from the last block to the first.
template <typename T, int DK, typename Ops>
__global__ void __launch_bounds__(kChunkThreads, Parts<T>::in == 1 ? 2 : 1)
    delta_reverse_split_kernel(const DeltaArgs a, const Kept kept) {
  constexpr int in = Parts<T>::in, mid = kMid;
  constexpr int kSteps = kWide<DK> / 32, kTiles = 2 * kSteps;
  constexpr int kOwn = kTiles >= 4 ? kTiles / 4 : 1;
  using L = ReverseSplitLds<T, DK>;
  extern __shared__ __align__(16) char lds[];
  const int slices = (a.dv + 15) / 16;
  int item, slice;
  item_slice(slices, &item, &slice);
  if (item >= a.n_seqs * a.H) return;
  const int h = item % a.H, s = by_length(a, item / a.H);
  const SeqRange seq = seq_range(a, s);
  if (!seq.ok) return;  // (flagged by the scan)
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int n = lane & 15, g = lane >> 4;
  const int hk = h / (a.H / a.Hk);
  const int col = 16 * slice + n;
  const bool live = col < a.dv;
  const int64_t state = ((int64_t)s * a.H + h) * a.dv * DK;
  const int tile0 = wave * kOwn;
  const bool owner = tile0 < kTiles;
  const auto channel = [&](int tl) { return 32 * (tl >> 1) + 8 * g + 4 * (tl & 1); };
  char* const s_frags = lds + L::s;
  f32x4 dS[kOwn];  // transposed, as S in the scan
#pragma unroll
  for (int i = 0; i < kOwn; ++i) {
    dS[i] = f32x4{0.f, 0.f, 0.f, 0.f};
    const int c = channel(tile0 + i);
    if (owner && a.dS_out != nullptr && live && c < DK) dS[i] = ld4(a.dS_out + state + (int64_t)col * DK + c);
    if (owner) put_half<mid>(s_frags, (tile0 + i) >> 1, (tile0 + i) & 1, lane, dS[i]);
  }

  const T* kp = static_cast<const T*>(a.k) + (int64_t)hk * DK;
  const T* qp = static_cast<const T*>(a.q) + (int64_t)hk * DK;
  const int64_t do_stride = (int64_t)a.H * a.dv;
  const T* dop = static_cast<const T*>(a.dout) + (int64_t)h * a.dv;
  const char* ws = static_cast<const char*>(a.ws) + ((int64_t)seq.block0 * a.H + h) * Ops::bytes;
  const int64_t ws_step = (int64_t)a.H * Ops::bytes;
  OwnRows<T, DK> K(wave), Q(wave);
  const typename OwnRows<T, DK>::Block Kt(lds + L::k), Qt(lds + L::q);
  Split<mid> tf[2], pf[2];
  T d[4];
  f32x4 first4[2], last4[2], beta4[2];  // two sets, as in the scan
  float whole[2];
  const int row4 = dealt(wave, 4 * g);
  const auto token = [&](int c) { return (int64_t)seq.begin + (int64_t)c * kBlock; };
  const auto rows_of = [&](int c) {
    const int64_t left = seq.end - token(c);
    return left < kBlock ? (int)left : kBlock;
  };
  const auto ask_values = [&](int c, int set) __attribute__((always_inline)) {
    const int rows = rows_of(c);
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const T* p = dop + (token(c) + (row4 + r < rows ? row4 + r : rows - 1)) * do_stride;
      d[r] = p[live ? col : 0];
    }
    const BlockScalars* sc = reinterpret_cast<const BlockScalars*>(ws + c * ws_step + Ops::scalars);
    first4[set] = ld4(sc->first + row4);
    last4[set] = ld4(sc->last + row4);
    beta4[set] = ld4(sc->beta + row4);
    whole[set] = sc->first[kBlock - 1];
  };
  const auto ask_rows = [&](int c) __attribute__((always_inline)) {
    K.load(kp + token(c) * a.k_stride, a.k_stride, rows_of(c));
    Q.load(qp + token(c) * a.q_stride, a.q_stride, rows_of(c));
  };
  const auto put_rows = [&](int c) __attribute__((always_inline)) {
    K.store(Kt, rows_of(c));
    Q.store(Qt, rows_of(c));
  };
  const auto ask_p = [&](int c) __attribute__((always_inline)) {
#pragma unroll
    for (int p = 0; p < 2; ++p)
      pf[p] = get_frag<mid>(ws + c * ws_step + Ops::pt, upper_frag(wave, p >= wave / 2 ? p : 1), lane);
  };
  const auto ask_t = [&](int c) __attribute__((always_inline)) {
#pragma unroll
    for (int p = 0; p < 2; ++p)
      tf[p] = get_frag<mid>(ws + c * ws_step + Ops::tt, upper_frag(wave, p >= wave / 2 ? p : 1), lane);
  };
  char* const d_frags = lds + L::d;
  // dO of the block that was asked for, as an operand
  const auto put_values = [&](int c) __attribute__((always_inline)) {
    const int rows = rows_of(c);
    f32x4 x;
#pragma unroll
    for (int r = 0; r < 4; ++r) x[r] = row4 + r < rows && live ? (float)d[r] : 0.f;
    put_half<in>(d_frags, wave >> 1, wave & 1, lane, x);  // exact
  };
  if (seq.blocks > 0) {
    ask_values(seq.blocks - 1, 0);
    ask_rows(seq.blocks - 1);
    ask_p(seq.blocks - 1);
    ask_t(seq.blocks - 1);
  }
  if (!owns(a, s, seq)) return;
  if (seq.blocks > 0) {
    put_values(seq.blocks - 1);
    put_rows(seq.blocks - 1);
  }
  const auto block = [&](int c, int set) __attribute__((always_inline)) {
    const int rows = rows_of(c);
    const int next = c > 0 ? c - 1 : 0;  // (loads under no condition, as in the scan)
    const int64_t place = (int64_t)(seq.block0 + c) * a.H + h;
    Split<in> kf[kSteps];
#pragma unroll
    for (int ks = 0; ks < kSteps; ++ks) kf[ks] = Kt.row8(dealt(wave, n), ks, g);  // (the wavefront's own)
    __syncthreads();  // dS, dO, K and Q are there
    ask_rows(next);
    f32x4 y = {0.f, 0.f, 0.f, 0.f}, w = y;
    {
      Split<mid> bs[kSteps];
#pragma unroll
      for (int ks = 0; ks < kSteps; ++ks) bs[ks] = get_frag<mid>(s_frags, ks, lane);
#pragma unroll
      for (int p = 0; p < 2; ++p)
        if (p >= wave / 2) w = mma(pf[p], get_frag<in>(d_frags, p, lane), w);
#pragma unroll
      for (int ks = 0; ks < kSteps; ++ks) y = mma(kf[ks], bs[ks], y);
    }
    {
      put_half<mid>(lds + L::u, wave >> 1, wave & 1, lane, fused(last4[set], y, a.scale * w));
      f32x4 x;
#pragma unroll
      for (int r = 0; r < 4; ++r)
        x[r] = row4 + r < rows && live ? a.scale * first4[set][r] * (float)d[r] : 0.f;
      put_half<mid>(lds + L::df, wave >> 1, wave & 1, lane, x);
    }
    ask_values(next, set ^ 1);
    ask_p(next);
    // the gradient of the state after the block
    if (owner) {
#pragma unroll
      for (int i = 0; i < kOwn; ++i)
        if (live && channel(tile0 + i) < DK)
          st4(kept.dS + (place * a.dv + col) * DK + channel(tile0 + i), dS[i]);
    }
    __syncthreads();  // dU and e^G d are there
    f32x4 dX = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int p = 0; p < 2; ++p)
      if (p >= wave / 2) dX = mma(tf[p], get_frag<mid>(lds + L::u, p, lane), dX);
    put_half<mid>(lds + L::x, wave >> 1, wave & 1, lane, -first4[set] * beta4[set] * dX);
    ask_t(next);
    // (Q's part of the update fills the time of the exchange)
    Split<in> kc[kOwn][2];
    if (owner) {
#pragma unroll
      for (int i = 0; i < kOwn; ++i) dS[i] *= whole[set];
#pragma unroll
      for (int p = 0; p < 2; ++p) {
#pragma unroll
        for (int i = 0; i < kOwn; ++i) {
          const Split<in> qc = Qt.template col8<true>(tile0 + i, p, lane);
          kc[i][p] = Kt.template col8<true>(tile0 + i, p, lane);
          dS[i] = mma(qc, get_frag<mid>(lds + L::df, p, lane), dS[i]);
        }
      }
    }
    if (live) {
#pragma unroll
      for (int r = 0; r < 4; ++r) kept.dX[(place * kBlock + row4 + r) * a.dv + col] = dX[r];
    }
    __syncthreads();  // dX is there
    if (owner) {
#pragma unroll
      for (int p = 0; p < 2; ++p) {
        const Split<mid> bx = get_frag<mid>(lds + L::x, p, lane);
#pragma unroll
        for (int i = 0; i < kOwn; ++i) dS[i] = mma(kc[i][p], bx, dS[i]);
      }
#pragma unroll
      for (int i = 0; i < kOwn; ++i)
        put_half<mid>(s_frags, (tile0 + i) >> 1, (tile0 + i) & 1, lane, dS[i]);
    }
    put_values(next);
    put_rows(next);  // (the update's operands have been read)
  };
  for (int c = seq.blocks - 1; c >= 0; c -= 2) {
    block(c, 0);
    if (c > 0) block(c - 1, 1);
  }
  if (a.dS0 == nullptr || !owner) return;
#pragma unroll
    for (int i = 0; i < kOwn; ++i)
      if (live && channel(tile0 + i) < DK)
        st4(a.dS0 + state + (int64_t)col * DK + channel(tile0 + i), dS[i]);
}

template <typename T, int DK, typename Ops>
hipError_t launch_reverse_split(const DeltaArgs& a, const Kept& kept, hipStream_t s) {
  using L = ReverseSplitLds<T, DK>;
  constexpr auto kernel = delta_reverse_split_kernel<T, DK, Ops>;
  const hipError_t e = allow_lds<decltype(kernel), kernel>(L::total);
  if (e != hipSuccess) return e;
  const int slices = (a.dv + 15) / 16;
  kernel<<<dim3((unsigned)item_grid((int64_t)a.n_seqs * a.H, slices)), dim3(kChunkThreads), L::total, s>>>(a, kept);
  return hipGetLastError();
}

}  // namespace

}  // namespace rs
