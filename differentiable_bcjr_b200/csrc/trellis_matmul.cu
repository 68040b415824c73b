// trellis_matmul.cu -- a few tokens times packed trellis weights (bcjr_trellis_matmul).
//
// A weight is codebook[state], and a step's state is a window of the packed
// stream, so the weights of a chunk of CH steps come out of two or three
// words by funnel shifts.  The codebook sits in shared memory; its random
// gathers bound the call: 32 lanes hit 32 banks at random, about 3.5 clocks a
// warp, where the packed words themselves are k bits a weight.  Small
// codebooks are kept in several copies, lane l reading copy l mod copies, so
// that lanes of different copies never meet in a bank.
//
// A lane keeps the inputs of its chunk of columns in registers and walks down
// the rows; a row's sums are added over the warp with a transposing butterfly
// (eight sums in nine shuffles) and over the warps in a fixed order.
//
// Codebooks up to 2^15 states are held in float32 (other types convert
// exactly), 2^16 states of a 16-bit type as they are (128 KiB), and 2^16
// float32 states in two halves, one after the other: the rows are walked
// twice, every state's gather being skipped in the walk that lacks it.
#include "layer_util.cuh"

namespace {

using namespace bcjr;

constexpr int kWarps = 16;
constexpr int kSums = 512;  // row sums a warp can hold in shared memory

struct Params {
  const void* x;
  const uint32_t* packed;
  const void* codebook;
  const float* scales;
  void* y;
  int x_dtype, c_dtype;
  int tokens, rows, cols, n, words;
  int L, group;
  int seqs;         // sequences of a row
  int per_seq;      // chunks of a sequence
  int chunks;       // of a row
  int wide;         // warps that share a row
  int copies_log2;  // of the codebook
};

enum Held { F32, B16, H16, HALVES };

// Row sums of eight values a lane each: lane l gets in v[0] the warp's sum of
// value l >> 2.
__device__ __forceinline__ void sum8(float (&v)[8], int lane) {
#pragma unroll
  for (int step = 0; step < 3; ++step) {
    const int half = 4 >> step, d = 16 >> step;
    const bool upper = (lane & d) != 0;
#pragma unroll
    for (int i = 0; i < half; ++i) {
      const float give = upper ? v[i] : v[i + half], keep = upper ? v[i + half] : v[i];
      v[i] = keep + __shfl_xor_sync(~0u, give, d);
    }
  }
  v[0] += __shfl_xor_sync(~0u, v[0], 2);
  v[0] += __shfl_xor_sync(~0u, v[0], 1);
}

template <int K, int MT, int CH, Held HELD>
__global__ void __launch_bounds__(kWarps * 32) trellis_matmul_kernel(const __grid_constant__ Params p) {
  constexpr int ROWS = 8 / MT;  // rows whose sums are added over the warp together
  // a chunk starts at a multiple of CH K bits, so at worst at this bit of a word
  constexpr int STEP = (CH * K) % 32 == 0 ? 32 : (CH * K) % 16 == 0 ? 16 : 8;
  constexpr int WORDS = (32 - STEP + (CH - 1) * K + 16 + 31) / 32;
  extern __shared__ __align__(16) unsigned char smem[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int S = 1 << p.L;
  const size_t table_bytes = HELD == F32 ? (static_cast<size_t>(S) * 4 << p.copies_log2)
                                                                                      : static_cast<size_t>(S) * 2;
  float* const sums = reinterpret_cast<float*>(smem + (table_bytes + 15) / 16 * 16);  // [kWarps][kSums]
  const uint32_t copies = 1u << p.copies_log2;
  const unsigned char* const mine = smem + (HELD == F32 ? (lane & (copies - 1)) * 4 : 0);
  const int shift = 32 - p.L;

  const int tiles = (p.chunks + 31) / 32;
  const int teams = kWarps / p.wide;          // rows walked side by side
  const int team = warp / p.wide, place = warp % p.wide;
  const int r_begin = static_cast<int>(static_cast<long long>(p.rows) * blockIdx.x / gridDim.x);
  const int r_end = static_cast<int>(static_cast<long long>(p.rows) * (blockIdx.x + 1) / gridDim.x);
  constexpr int ROOM = kSums / MT;            // rows a team can hold sums of
  const int token0 = blockIdx.y * MT;
  const int tokens = min(MT, p.tokens - token0);

  constexpr int PHASES = HELD == HALVES ? 2 : 1;
  for (int r0 = r_begin; r0 < r_end; r0 += ROOM * teams) {
    const int r1 = min(r0 + ROOM * teams, r_end);
    for (int i = lane; i < kSums; i += 32) sums[warp * kSums + i] = 0.f;
    __syncwarp();
    for (int phase = 0; phase < PHASES; ++phase) {
      if (HELD == HALVES || r0 == r_begin) {
        __syncthreads();  // the last half's readers are done
        if constexpr (HELD == HALVES) {
          const float* const from = static_cast<const float*>(p.codebook) + phase * (S / 2);
          for (int i = threadIdx.x; i < S / 2; i += kWarps * 32) reinterpret_cast<float*>(smem)[i] = from[i];
        } else if constexpr (HELD == F32) {
          for (int i = threadIdx.x; i < (S << p.copies_log2); i += kWarps * 32)
            reinterpret_cast<float*>(smem)[i] = load_as_f32(p.codebook, p.c_dtype, i >> p.copies_log2);
        } else {
          for (int i = threadIdx.x; i < S; i += kWarps * 32)
            reinterpret_cast<uint16_t*>(smem)[i] = static_cast<const uint16_t*>(p.codebook)[i];
        }
        __syncthreads();
      }
      for (int tile = place; tile < tiles; tile += p.wide) {
        const int q = tile * 32 + lane;
        const bool have = q < p.chunks;
        const int seq = (have ? q : 0) / p.per_seq;
        const int t0 = ((have ? q : 0) - seq * p.per_seq) * CH;
        const int count = have ? min(CH, p.n - t0) : 0;
        const int col = seq * p.n + t0;
        float x[CH][MT];
#pragma unroll
        for (int m = 0; m < MT; ++m) {
          const size_t at = static_cast<size_t>(token0 + min(m, tokens - 1)) * p.cols + col;
#pragma unroll
          for (int i = 0; i < CH; ++i) x[i][m] = i < count ? load_as_f32(p.x, p.x_dtype, at + i) : 0.f;
        }
        const int bit = t0 * K, word = bit >> 5, skew = bit & 31;
        const float* const scale = p.scales ? p.scales + static_cast<size_t>(col / p.group) * p.rows : nullptr;
        for (int rb = r0 + team * ROWS; rb < r1; rb += teams * ROWS) {
          float v[8];
#pragma unroll
          for (int rr = 0; rr < ROWS; ++rr) {
            const int row = min(rb + rr, r1 - 1);
            const uint32_t* const stream = p.packed + (static_cast<size_t>(row) * p.seqs + seq) * p.words;
            uint32_t a[WORDS + 1];
#pragma unroll
            for (int i = 0; i < WORDS; ++i) a[i] = stream[min(word + i, p.words - 1)];
            a[WORDS] = 0;
            if constexpr (STEP != 32) {
#pragma unroll
              for (int i = 0; i < WORDS; ++i) a[i] = __funnelshift_l(a[i + 1], a[i], skew);
            }
            float acc[MT] = {};
#pragma unroll
            for (int i = 0; i < CH; ++i) {
              const int at = i * K;  // of the chunk's bits
              const uint32_t s = __funnelshift_l(a[at / 32 + 1], a[at / 32], at % 32) >> shift;
              float c = 0.f;
              bool add = true;
              if constexpr (HELD == F32) {
                c = *reinterpret_cast<const float*>(mine + (s << (p.copies_log2 + 2)));
              } else if constexpr (HELD == B16) {
                c = __uint_as_float(static_cast<uint32_t>(reinterpret_cast<const uint16_t*>(smem)[s]) << 16);
              } else if constexpr (HELD == H16) {
                c = __half2float(reinterpret_cast<const __half*>(smem)[s]);
              } else {
                add = (s >> 15) == phase;
                if (add) c = reinterpret_cast<const float*>(smem)[s & 0x7FFFu];
              }
              if (i >= count) c = 0.f;  // a step behind the end, whatever its window reads
              if (add) {                // (0 would not do for the other half: an input may be infinite)
#pragma unroll
                for (int m = 0; m < MT; ++m) acc[m] = fmaf(c, x[i][m], acc[m]);
              }
            }
            const float sc = scale ? scale[row] : 1.f;
#pragma unroll
            for (int m = 0; m < MT; ++m) v[rr * MT + m] = have ? acc[m] * sc : 0.f;
          }
          sum8(v, lane);
          if ((lane & 3) == 0) {
            const int i = lane >> 2;
            const int rr = i / MT, m = i % MT;
            const int at = ((rb - r0) / (teams * ROWS) * ROWS + rr) * MT + m;
            if (rb + rr < r1) sums[warp * kSums + at] += v[0];
          }
          __syncwarp();
        }
      }
    }
    __syncthreads();
    for (int i = threadIdx.x; i < (r1 - r0) * tokens; i += kWarps * 32) {
      const int row = i % (r1 - r0), m = i / (r1 - r0);
      const int turn = row / (teams * ROWS), of = row % (teams * ROWS);
      const float* const from = sums + (of / ROWS * p.wide) * kSums + (turn * ROWS + of % ROWS) * MT + m;
      float v = 0.f;
      for (int w = 0; w < p.wide; ++w) v += from[w * kSums];
      store_from_f32(p.y, p.x_dtype, static_cast<size_t>(token0 + m) * p.rows + r0 + row, v);
    }
    __syncthreads();
  }
}

template <int K, int MT, int CH, Held HELD>
bcjr_status launch(Params p, int sms, cudaStream_t s) {
  p.per_seq = (p.n + CH - 1) / CH;
  p.chunks = p.seqs * p.per_seq;
  const int tiles = (p.chunks + 31) / 32;
  p.wide = 1;
  while (p.wide < kWarps && p.wide < tiles) p.wide *= 2;
  const size_t S = size_t{1} << p.L;
  p.copies_log2 = 0;
  if (HELD == F32) {
    while (p.copies_log2 < 5 && (S * 4 << (p.copies_log2 + 1)) <= (128u << 10)) ++p.copies_log2;
  }
  const size_t table = HELD == HALVES ? S * 2 : HELD == F32 ? S * 4 << p.copies_log2 : S * 2;
  const size_t smem = (table + 15) / 16 * 16 + sizeof(float) * kWarps * kSums;
  auto* const kernel = trellis_matmul_kernel<K, MT, CH, HELD>;
  if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem)) != cudaSuccess) {
    cudaGetLastError();
    return BCJR_ERR_CUDA;
  }
  const int teams = kWarps / p.wide, rows_a_turn = teams * (8 / MT);
  const int most = (p.rows + rows_a_turn - 1) / rows_a_turn;
  const dim3 grid(static_cast<unsigned>(most < sms ? most : sms), static_cast<unsigned>((p.tokens + MT - 1) / MT));
  kernel<<<grid, kWarps * 32, smem, s>>>(p);
  return launched();
}

template <int K, Held HELD>
bcjr_status launch_tokens(const Params& p, int sms, cudaStream_t s) {
  if (p.tokens == 1) return launch<K, 1, 16, HELD>(p, sms, s);
  if (p.tokens == 2) return launch<K, 2, 16, HELD>(p, sms, s);
  return launch<K, 4, 16, HELD>(p, sms, s);
}

template <int K>
bcjr_status launch_held(const Params& p, int sms, cudaStream_t s) {
  if (p.L < 16) return launch_tokens<K, F32>(p, sms, s);
  if (p.c_dtype == BCJR_F32) return launch_tokens<K, HALVES>(p, sms, s);
  if (p.c_dtype == BCJR_BF16) return launch_tokens<K, B16>(p, sms, s);
  return launch_tokens<K, H16>(p, sms, s);
}

}  // namespace

extern "C" bcjr_status bcjr_trellis_matmul(const void* x, int x_dtype, int tokens, int rows, int cols,
                                           const uint32_t* packed, const void* codebook, int codebook_dtype,
                                           int state_bits, int k, int seq_len, const float* scales, int group_size,
                                           void* y, bcjr_stream_t stream) {
  if (!dtype_ok(x_dtype) || !dtype_ok(codebook_dtype) || tokens < 0 || rows < 0 || cols < 1 || seq_len < 1 ||
      state_bits < 1 || k < 1 || k > state_bits || group_size < 0)
    return BCJR_ERR_INVALID_ARG;
  if (cols % seq_len != 0) return BCJR_ERR_INVALID_ARG;
  // token passes are the second grid dimension; columns and bits are counted in ints
  if (k > 4 || state_bits > 16 || tokens > 65535 || rows > (1 << 30) || cols > (1 << 28)) return BCJR_ERR_UNSUPPORTED;
  int group = cols;
  if (scales && group_size > 0) {
    group = group_size;
    const bool whole = group % seq_len == 0 && cols % group == 0;
    const bool part = group % 16 == 0 && seq_len % group == 0;
    if (!whole && !part) return BCJR_ERR_UNSUPPORTED;
  }
  if (tokens == 0 || rows == 0) return BCJR_OK;
  if (!x || !packed || !codebook || !y || !ptr_aligned(x, dtype_size(x_dtype)) || !ptr_aligned(y, dtype_size(x_dtype)) ||
      !ptr_aligned(packed, 4) || !ptr_aligned(codebook, dtype_size(codebook_dtype)) || !ptr_aligned(scales, 4))
    return BCJR_ERR_INVALID_ARG;
  const int sms = sm_count();
  if (sms <= 0) return BCJR_ERR_CUDA;
  Params p = {};
  p.x = x;
  p.packed = packed;
  p.codebook = codebook;
  p.scales = scales;
  p.y = y;
  p.x_dtype = x_dtype;
  p.c_dtype = codebook_dtype;
  p.tokens = tokens;
  p.rows = rows;
  p.cols = cols;
  p.n = seq_len;
  p.words = static_cast<int>((static_cast<long long>(seq_len) * k + state_bits - k + 31) / 32);
  p.L = state_bits;
  p.group = group;
  p.seqs = cols / seq_len;
  cudaStream_t s = as_stream(stream);
  switch (k) {
    case 1: return launch_held<1>(p, sms, s);
    case 2: return launch_held<2>(p, sms, s);
    case 3: return launch_held<3>(p, sms, s);
    default: return launch_held<4>(p, sms, s);
  }
}
