// Tables of a packed ragged batch, built on the GPU from the requests' lengths.
//
//   cu_tokens[i] = sum_{s<i} len_s          cu_blocks[i] = sum_{s<i} ceil(len_s / block)
//   token_seq[t] = the request of packed token t, token_pos[t] = history + its place in it
//   block_seq[b] = the request of block b (blocks never cross requests)
//
// One launch: the lengths are a few KB, so every workgroup scans all of them into its LDS
// (32 KB at 4096 requests) and then writes its share of the token and block rows, four
// consecutive rows per thread from one binary search. That trades re-reads that stay in L2
// for the second launch that a separate scan would take. Measured: 256 requests of 20011 tokens 5.6 us, 4096 of
// 1000003 tokens 10 us (a launch alone is 4 to 5; the scan of 4096 lengths is most of the rest). Sums saturate at max_tokens + 1
// (saturating addition is associative, so the scan is exact for any lengths).
#include "device.hpp"
#include "prompt.hpp"

namespace rs {

namespace {

constexpr int kRaggedThreads = 1024;
constexpr int kRaggedWaves = kRaggedThreads / 64;

__device__ __forceinline__ uint32_t sat_add(uint32_t a, uint32_t b, uint32_t cap) {
  const uint32_t s = a + b;  // both at most 2^31
  return s < cap ? s : cap;
}

// Exclusive saturating scan over the workgroup; *total is the whole sum.
__device__ uint32_t scan_exclusive(uint32_t x, uint32_t cap, uint32_t* waves, uint32_t* total) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  uint32_t inc = x;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const uint32_t up = __shfl_up(inc, d);
    if (lane >= d) inc = sat_add(inc, up, cap);
  }
  if (lane == 63) waves[wave] = inc;
  __syncthreads();
  uint32_t base = 0, all = 0;
  for (int w = 0; w < kRaggedWaves; ++w) {
    if (w < wave) base = sat_add(base, waves[w], cap);
    all = sat_add(all, waves[w], cap);
  }
  __syncthreads();  // (the scratch is used again)
  *total = all;
  const uint32_t before = __shfl_up(inc, 1);
  return lane == 0 ? base : sat_add(base, before, cap);
}

// The last i in [0, n) with table[i] <= x (table ascending, table[0] = 0).
__device__ __forceinline__ int find(const uint32_t* table, int n, uint32_t x) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (table[mid] <= x)
      lo = mid;
    else
      hi = mid;
  }
  return lo;
}

__global__ void __launch_bounds__(kRaggedThreads) ragged_kernel(const RaggedArgs a) {
  extern __shared__ uint32_t lds[];
  __shared__ uint32_t waves[kRaggedWaves];
  __shared__ int flags;
  const int n = a.n, tid = threadIdx.x;
  uint32_t* cu = lds;            // [n + 1], first the clamped lengths
  uint32_t* cub = lds + n + 1;   // [n + 1]
  if (tid == 0) flags = 0;
  __syncthreads();
  bool negative = false;
  for (int i = tid; i < n; i += kRaggedThreads) {
    const int32_t len = a.lengths[i];
    negative |= len < 0;
    cu[i] = len > 0 ? (uint32_t)len : 0u;
  }
  if (negative) flags = 1;
  __syncthreads();
  // each thread takes `per` consecutive requests
  const int per = (n + kRaggedThreads - 1) / kRaggedThreads;
  const int i0 = tid * per < n ? tid * per : n, i1 = i0 + per < n ? i0 + per : n;
  const uint32_t cap = a.max_tokens + 1;
  uint32_t sum = 0, total;
  for (int i = i0; i < i1; ++i) sum = sat_add(sum, cu[i], cap);
  uint32_t run = scan_exclusive(sum, cap, waves, &total);
  uint32_t blocks = 0;
  for (int i = i0; i < i1; ++i) {
    const uint32_t begin = run < a.max_tokens ? run : a.max_tokens;
    run = sat_add(run, cu[i], cap);
    const uint32_t end = run < a.max_tokens ? run : a.max_tokens;
    cu[i] = begin;
    const uint32_t nb = (end - begin + (uint32_t)a.block - 1) / (uint32_t)a.block;
    cub[i] = nb;
    blocks += nb;
  }
  uint32_t total_blocks;
  uint32_t brun = scan_exclusive(blocks, 0x7fffffffu, waves, &total_blocks);
  for (int i = i0; i < i1; ++i) {
    const uint32_t nb = cub[i];
    cub[i] = brun;
    brun += nb;
  }
  const uint32_t tokens = total < a.max_tokens ? total : a.max_tokens;
  if (tid == 0) {
    cu[n] = tokens;
    cub[n] = total_blocks;
  }
  __syncthreads();
  if (blockIdx.x == 0) {
    for (int i = tid; i <= n; i += kRaggedThreads) {
      a.cu_tokens[i] = (int32_t)cu[i];
      a.cu_blocks[i] = (int32_t)cub[i];
    }
    if (tid == 0) {
      const int bits = (flags || total > a.max_tokens) ? REPLAYSSM_DEVERR_RANGE : 0;
      if (bits) atomicOr(a.err, bits);
    }
  }
  const int64_t stride = (int64_t)gridDim.x * kRaggedThreads;
  for (int64_t quad = (int64_t)blockIdx.x * kRaggedThreads + tid; quad * 4 < (int64_t)a.max_tokens; quad += stride) {
    const uint32_t t0 = (uint32_t)(quad * 4);
    int32_t seq[4], pos[4];
    int i = 0;
    uint32_t next = 0;
    int32_t hist = 0;
    if (t0 < tokens) {
      i = find(cu, n, t0);
      next = cu[i + 1];
      hist = a.history ? a.history[i] : 0;
    }
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const uint32_t t = t0 + r;
      seq[r] = pos[r] = -1;
      if (t < tokens) {
        if (t >= next) {
          while (t >= next) next = cu[++i + 1];  // (empty requests are passed over; t < cu[n] ends it)
          hist = a.history ? a.history[i] : 0;
        }
        seq[r] = i;
        pos[r] = (int32_t)((uint32_t)hist + (t - cu[i]));
      }
    }
    if (t0 + 4 <= a.max_tokens) {
      *reinterpret_cast<int4*>(a.token_seq + t0) = int4{seq[0], seq[1], seq[2], seq[3]};
      *reinterpret_cast<int4*>(a.token_pos + t0) = int4{pos[0], pos[1], pos[2], pos[3]};
    } else {
      for (int r = 0; t0 + r < a.max_tokens; ++r) {
        a.token_seq[t0 + r] = seq[r];
        a.token_pos[t0 + r] = pos[r];
      }
    }
  }
  for (int64_t b = (int64_t)blockIdx.x * kRaggedThreads + tid; b < a.max_blocks; b += stride)
    a.block_seq[b] = b < (int64_t)total_blocks ? find(cub, n, (uint32_t)b) : -1;
}

}  // namespace

hipError_t launch_ragged(const RaggedArgs& a, hipStream_t s) {
  const size_t smem = (size_t)(a.n + 1) * 8;
  if (smem > 48 * 1024) {
    const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(ragged_kernel),
                                             hipFuncAttributeMaxDynamicSharedMemorySize,
                                             (REPLAYSSM_RAGGED_SEQS + 1) * 8);
    if (e != hipSuccess) return e;
  }
  int cus = 0;
  const hipError_t e = device_cus(&cus);
  if (e != hipSuccess) return e;
  const int64_t rows = (int64_t)a.max_tokens / 4 > a.max_blocks ? (int64_t)a.max_tokens / 4 : a.max_blocks;
  int64_t grid = (rows + kRaggedThreads) / kRaggedThreads;
  if (grid > cus) grid = cus;
  ragged_kernel<<<dim3((unsigned)grid), dim3(kRaggedThreads), smem, s>>>(a);
  return hipGetLastError();
}

}  // namespace rs
