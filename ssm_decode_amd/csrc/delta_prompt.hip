// The gated delta rule over packed sequences, in blocks of 64 tokens.
//
// Inside a block that starts from state S, with G_i the sum of g over its tokens up to i:
//     (I + A) U = X,   A_ij = beta_i e^{G_i - G_j} (k_i . k_j) for j < i,
//     X_i = beta_i (v_i - e^{G_i} S k_i),   U = T X,  T = (I + A)^{-1}
//     O_i = scale (e^{G_i} S q_i + sum_{j <= i} P_ij u_j),   P_ij = e^{G_i - G_j} (q_i . k_j)
//     S' = e^{G_end} S + sum_j e^{G_end - G_j} u_j k_j^T
// so the only serial part is S -> S' from block to block; T and P need no state.
//
//   prepare  (one workgroup per block and value head): T and P as matrix operands, and the
//            block's decays. G is summed in fp64: differences of long sums of g stay exact enough, and
//            a gate that is closed (g = -infinity, kept as -1e4) leaves later differences whole.
//   scan     (workgroups per sequence, value head and slice of state rows): walks the
//            sequence's blocks. State rows are independent; they and every product with them are
//            kept transposed, so that a product's result is the next one's operand as it is.
#include "walk.hpp"

namespace rs {

namespace {

// Where a block's operands lie in the workspace.
template <int LOW>
struct ForwardBlock {
  static constexpr bool backward = false;
  static constexpr int64_t t = 0, scalars = t + frag_bytes(kMid), p = scalars + sizeof(BlockScalars),
                           bytes = p + frag_bytes(LOW), scan_bytes = bytes;
};

template <typename T, int DK>
hipError_t launch_forward(const DeltaArgs& a, hipStream_t s) {
  hipError_t e = launch_prepare<T, DK, ForwardBlock<Parts<T>::low>>(a, s);
  if (e != hipSuccess) return e;
  return launch_scan<T, DK, ForwardBlock<Parts<T>::low>, false>(a, Kept{}, s);
}

template <typename T>
hipError_t launch_dk(const DeltaArgs& a, hipStream_t s) {
  switch (a.dk) {
    case 16: return launch_forward<T, 16>(a, s);
    case 32: return launch_forward<T, 32>(a, s);
    case 64: return launch_forward<T, 64>(a, s);
    default: return launch_forward<T, 128>(a, s);
  }
}

}  // namespace

int64_t delta_forward_bytes(const replayssm_delta_config& c, int max_blocks) {
  const int64_t block = c.dtype == REPLAYSSM_F32 ? ForwardBlock<3>::bytes : ForwardBlock<2>::bytes;
  return (int64_t)max_blocks * c.H * block;
}

hipError_t launch_delta_prompt(const DeltaArgs& a, hipStream_t s) {
  switch (a.dtype) {
    case REPLAYSSM_BF16: return launch_dk<__bf16>(a, s);
    case REPLAYSSM_F16: return launch_dk<_Float16>(a, s);
    default: return launch_dk<float>(a, s);
  }
}

}  // namespace rs
