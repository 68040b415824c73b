// trellis_matmul.cuh -- a few tokens times packed trellis weights (bcjr_trellis_matmul).
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
// the rows, the next rows' words on their way; a row's sums are added over the
// warp with a transposing butterfly (eight sums in nine shuffles) and over the
// warps in a fixed order.
//
// Codebooks up to 2^15 states are held in float32 (other types convert
// exactly), 2^16 states of a 16-bit type as they are (128 KiB), and 2^16
// float32 states in two halves, one after the other: the rows are walked
// twice, every state's gather being skipped in the walk that lacks it (half
// the lanes of a gather meet in fewer banks, so both walks together take less
// than two full ones).
//
// Measured, device time a call with the words in memory (in the L2 cache): 2048 x
// 8192, k = 2, 2^16 states, one token 13.5 us (12.4) with a bf16 codebook (its
// gathers alone, at 3.5 clocks a warp, would take 6.6 us), 20.0 (19.0) with a float32
// one, whose halves every CTA copies and walks its rows for one after the other;
// four bf16 tokens 31.8 (29.5), eight 49.7 (46.0).  Several tokens of the codebook's
// own 16-bit type take the kernel of trellis_mma.cuh.
#pragma once
#include <type_traits>

#include "layer_util.cuh"
#include "trellis_internal.h"
#include "trellis_mma.cuh"

namespace bcjr {
namespace {

using Params = TrellisMatmulParams;

constexpr int kWarps = 16;
constexpr int kSums = 512;  // row sums a warp can hold in shared memory

constexpr uint32_t kHalf = 131072;  // bytes of 2^15 float32 codewords, or 2^16 of 16 bits

enum Held { F32, B16, H16, HALVES };

// The sums over the warp of eight values a lane: lane l gets in v[0] that of value l >> 2.
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

// bits [at, at + 32) of a stream's words
template <int N>
__device__ __forceinline__ uint32_t shifted(const uint32_t (&a)[N], int at) {
  return at % 32 == 0 ? a[at / 32] : __funnelshift_l(a[at / 32 + 1], a[at / 32], at % 32);
}

__device__ __forceinline__ float shared_f32(uint32_t at) {
  float v;
  asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(at));
  return v;
}
__device__ __forceinline__ uint32_t shared_u16(uint32_t at) {
  uint16_t v;
  asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(at));
  return v;
}

// The codeword of the state whose first bit is bit `at` of the chunk; 0 where
// it is in the other half of the codebook.  `table`: its shared-memory address
// (F32: of the lane's copy; HALVES: a zero follows the half).
template <Held HELD, int N>
__device__ __forceinline__ float codeword(uint32_t table, int shift, uint32_t mask, uint32_t phase_bit,
                                          const uint32_t (&a)[N], int at, bool& here) {
  here = true;
  if constexpr (HELD == F32) {
    // shift and mask leave the state times the bytes between its copies
    return shared_f32(table + ((shifted(a, at) >> shift) & mask));
  } else {
    // 16 bits a state: constant shifts put it above the byte offset's low bits
    constexpr int LOW = HELD == HALVES ? 2 : 1;
    const int down = 48 - at % 32 - LOW;
    const uint32_t q = down >= 32 ? a[at / 32] >> (down - 32) : __funnelshift_r(a[at / 32 + 1], a[at / 32], down);
    if constexpr (HELD == HALVES) {
      const uint32_t offset = (q ^ phase_bit) & 0x3FFFCu;  // 2^17 and more: in the other half
      here = offset < kHalf;
      return shared_f32(table + min(offset, kHalf));
    } else if constexpr (HELD == B16) {
      return __uint_as_float(shared_u16(table + (q & 0x1FFFEu)) << 16);
    } else {
      return __half2float(__ushort_as_half(static_cast<uint16_t>(shared_u16(table + (q & 0x1FFFEu)))));
    }
  }
}

__device__ __forceinline__ bool finite_bits(uint32_t bits, uint32_t exponent) { return (bits & exponent) != exponent; }

// 2^17 bytes of codewords into shared memory, 16 at a time where the source
// allows.  False if this thread met one that is not finite; `exponent`: the
// exponent field of one, or of the upper of two in a word.
template <int BYTES>
__device__ __forceinline__ bool copy_in(unsigned char* to, const unsigned char* from, uint32_t exponent) {
  bool fine = true;
  auto check = [&](uint32_t w) {
    fine = fine && finite_bits(w, exponent);
    if (BYTES == 2) fine = fine && finite_bits(w << 16, exponent);
  };
  if ((reinterpret_cast<uintptr_t>(from) & 15) == 0) {
#pragma unroll 8
    for (int i = threadIdx.x; i < static_cast<int>(kHalf / 16); i += kWarps * 32) {
      const uint4 v = __ldg(reinterpret_cast<const uint4*>(from) + i);
      reinterpret_cast<uint4*>(to)[i] = v;
      check(v.x);
      check(v.y);
      check(v.z);
      check(v.w);
    }
  } else {
    for (int i = threadIdx.x; i < static_cast<int>(kHalf / BYTES); i += kWarps * 32) {
      if (BYTES == 2) {
        const uint16_t v = reinterpret_cast<const uint16_t*>(from)[i];
        reinterpret_cast<uint16_t*>(to)[i] = v;
        check(static_cast<uint32_t>(v) << 16);
      } else {
        const uint32_t v = reinterpret_cast<const uint32_t*>(from)[i];
        reinterpret_cast<uint32_t*>(to)[i] = v;
        check(v);
      }
    }
  }
  return fine;
}

// Sums of MT tokens, two to a packed multiply-add where there are several.
template <int MT>
struct Sums {
  float2 v[MT / 2];
  __device__ __forceinline__ void add(float c, const Sums& x) {
#pragma unroll
    for (int m = 0; m < MT / 2; ++m) v[m] = __ffma2_rn(make_float2(c, c), x.v[m], v[m]);
  }
  __device__ __forceinline__ float get(int m) const { return m & 1 ? v[m / 2].y : v[m / 2].x; }
  __device__ __forceinline__ void set(int m, float f) {
    if (m & 1) v[m / 2].y = f;
    else v[m / 2].x = f;
  }
};
template <>
struct Sums<1> {
  float v;
  __device__ __forceinline__ void add(float c, const Sums& x) { v = fmaf(c, x.v, v); }
  __device__ __forceinline__ float get(int) const { return v; }
  __device__ __forceinline__ void set(int, float f) { v = f; }
};

template <int K, int MT, int CH, Held HELD>
__global__ void __launch_bounds__(kWarps * 32, 1) trellis_matmul_kernel(const __grid_constant__ Params p) {
  constexpr int ROWS = 8 / MT;               // rows whose sums are added over the warp together
  constexpr int BATCH = ROWS < 4 ? 4 : ROWS; // rows whose words are fetched together
  // a chunk starts at a multiple of CH K bits, so at worst at this bit of a word
  constexpr int STEP = (CH * K) % 32 == 0 ? 32 : (CH * K) % 16 == 0 ? 16 : 8;
  constexpr int WORDS = (32 - STEP + (CH - 1) * K + 16 + 31) / 32;
  extern __shared__ __align__(16) unsigned char smem[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int S = 1 << p.L;
  const size_t table_bytes = HELD == F32 ? static_cast<size_t>(S) * 4 << p.copies_log2 : HELD == HALVES ? kHalf + 16 : kHalf;
  float* const sums = reinterpret_cast<float*>(smem + (table_bytes + 15) / 16 * 16) + warp * kSums;  // of [kWarps][kSums]
  uint32_t table;  // kept in a register
  asm volatile("mov.u32 %0, %1;" : "=r"(table) : "r"(static_cast<uint32_t>(__cvta_generic_to_shared(smem))));
  if (HELD == F32) table += (lane & ((1u << p.copies_log2) - 1u)) * 4;
  const int shift = 30 - p.L - p.copies_log2;
  const uint32_t mask = (static_cast<uint32_t>(S) - 1u) << (2 + p.copies_log2);

  const int tiles = (p.chunks + 31) / 32;
  const int teams = kWarps / p.wide;  // rows walked side by side
  const int team = warp / p.wide, place = warp % p.wide;
  const int r_begin = static_cast<int>(static_cast<long long>(p.rows) * blockIdx.x / gridDim.x);
  const int r_end = static_cast<int>(static_cast<long long>(p.rows) * (blockIdx.x + 1) / gridDim.x);
  constexpr int ROOM = kSums / MT;  // rows a team can hold sums of
  const int token0 = blockIdx.y * MT;
  const int tokens = min(MT, p.tokens - token0);

  constexpr int PHASES = HELD == HALVES ? 2 : 1;
  bool all_finite = true;  // every codeword at hand is
  for (int r0 = r_begin; r0 < r_end; r0 += ROOM * teams) {
    const int r1 = min(r0 + ROOM * teams, r_end);
    for (int i = lane; i < kSums; i += 32) sums[i] = 0.f;
    __syncwarp();
    for (int phase = 0; phase < PHASES; ++phase) {
      if (HELD == HALVES || r0 == r_begin) {
        if (HELD == HALVES) __syncthreads();  // the last half's readers are done
        bool fine = true;
        if constexpr (HELD == F32) {
#pragma unroll 8
          for (int i = threadIdx.x; i < (S << p.copies_log2); i += kWarps * 32) {
            const float v = load_as_f32(p.codebook, p.c_dtype, i >> p.copies_log2);
            reinterpret_cast<float*>(smem)[i] = v;
            fine = fine && finite_bits(__float_as_uint(v), 0x7F800000u);
          }
        } else {
          const unsigned char* const from = static_cast<const unsigned char*>(p.codebook) + phase * kHalf;
          if (HELD == HALVES && threadIdx.x == 0) *reinterpret_cast<float*>(smem + kHalf) = 0.f;
          // without padding nothing has to be known of the codewords
          if (!p.padded && (reinterpret_cast<uintptr_t>(from) & 15) == 0) {
            const uint32_t at = static_cast<uint32_t>(__cvta_generic_to_shared(smem));
#pragma unroll
            for (int i = threadIdx.x; i < static_cast<int>(kHalf / 16); i += kWarps * 32)
              asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(at + i * 16), "l"(from + i * 16) : "memory");
            asm volatile("cp.async.wait_all;" ::: "memory");
          } else {
            fine = copy_in<HELD == HALVES ? 4 : 2>(smem, from, HELD == H16 ? 0x7C000000u : 0x7F800000u);
          }
        }
        all_finite = __syncthreads_and(fine) != 0;
      }
      const uint32_t phase_bit = phase ? 0x20000u : 0u;
      for (int tile = place; tile < tiles; tile += p.wide) {
        const int q = tile * 32 + lane;
        const bool have = q < p.chunks;
        const int seq = (have ? q : 0) / p.per_seq;
        const int t0 = ((have ? q : 0) - seq * p.per_seq) * CH;
        const int count = have ? min(CH, p.n - t0) : 0;
        const int col = seq * p.n + t0;
        Sums<MT> x[CH];
        bool fine = all_finite;
#pragma unroll
        for (int m = 0; m < MT; ++m) {
          const size_t at = static_cast<size_t>(token0 + min(m, tokens - 1)) * p.cols + col;
#pragma unroll
          for (int i = 0; i < CH; ++i) {
            const float v = i < count ? load_as_f32(p.x, p.x_dtype, at + i) : 0.f;
            x[i].set(m, v);
            fine = fine && finite_bits(__float_as_uint(v), 0x7F800000u);
          }
        }
        const int bit = t0 * K, skew = bit & 31;
        const uint32_t* const stream = p.packed + static_cast<size_t>(seq) * p.words;
        int word[WORDS];  // a chunk at the sequence's end may have fewer words left
#pragma unroll
        for (int i = 0; i < WORDS; ++i) word[i] = min((bit >> 5) + i, p.words - 1);
        const size_t row_words = static_cast<size_t>(p.seqs) * p.words;
        // (a lane without a chunk has sums of 0, which an infinite scale would spoil)
        const float* const scale = p.scales && have ? p.scales + static_cast<size_t>(col / p.group) * p.rows : nullptr;

        // GUARDED: a step behind the chunk's end and a state of the other half
        // are left out.  Otherwise they are a product with 0, which is enough
        // where codewords and inputs are finite.
        auto walk = [&](auto guarded) {
          constexpr bool GUARDED = decltype(guarded)::value;
          uint32_t next[BATCH][WORDS];
          float next_scale[BATCH];
          auto fetch = [&](int rb) {
#pragma unroll
            for (int rr = 0; rr < BATCH; ++rr) {
              if (rb + rr >= r1) break;
              const uint32_t* const from = stream + (rb + rr) * row_words;
#pragma unroll
              for (int i = 0; i < WORDS; ++i) next[rr][i] = __ldg(from + word[i]);
              next_scale[rr] = scale ? __ldg(scale + rb + rr) : 1.f;
            }
          };
          fetch(r0 + team * BATCH);
          int at_sum = 0;  // of the team's sums
          for (int rb = r0 + team * BATCH; rb < r1; rb += teams * BATCH) {
            uint32_t now[BATCH][WORDS];
            float now_scale[BATCH];
#pragma unroll
            for (int rr = 0; rr < BATCH; ++rr) {
#pragma unroll
              for (int i = 0; i < WORDS; ++i) now[rr][i] = next[rr][i];
              now_scale[rr] = next_scale[rr];
            }
            fetch(rb + teams * BATCH);
#pragma unroll
            for (int r8 = 0; r8 < BATCH; r8 += ROWS) {
              if (rb + r8 >= r1) break;
              float v[8];
#pragma unroll
              for (int rr = 0; rr < ROWS; ++rr) {
                Sums<MT> acc;
#pragma unroll
                for (int m = 0; m < MT; ++m) acc.set(m, 0.f);
                if (rb + r8 + rr < r1) {
                  uint32_t a[WORDS + 1];
#pragma unroll
                  for (int i = 0; i < WORDS; ++i) a[i] = now[r8 + rr][i];
                  a[WORDS] = 0;
                  if constexpr (STEP != 32) {
#pragma unroll
                    for (int i = 0; i < WORDS; ++i) a[i] = __funnelshift_l(a[i + 1], a[i], skew);
                  }
#pragma unroll
                  for (int i = 0; i < CH; ++i) {
                    bool here;
                    const float c = codeword<HELD>(table, shift, mask, phase_bit, a, i * K, here);
                    if (!GUARDED || (here && i < count)) acc.add(c, x[i]);
                  }
                }
#pragma unroll
                for (int m = 0; m < MT; ++m) {
                  const float sum = acc.get(m);
                  // (a chunk may have none of its states in this half: nothing times an infinite scale is nothing)
                  v[rr * MT + m] = HELD == HALVES && sum == 0.f ? 0.f : sum * now_scale[r8 + rr];
                }
              }
              sum8(v, lane);
              if ((lane & 3) == 0) {
                const int i = lane >> 2;
                if (rb + r8 + i / MT < r1) sums[at_sum + r8 * MT + i] += v[0];
              }
            }
            at_sum += BATCH * MT;
            __syncwarp();
          }
        };
        if (__all_sync(~0u, fine)) walk(std::false_type{});
        else walk(std::true_type{});
      }
    }
    __syncthreads();
    const float* const all = sums - warp * kSums;
    for (int i = threadIdx.x; i < (r1 - r0) * tokens; i += kWarps * 32) {
      const int row = i % (r1 - r0), m = i / (r1 - r0);
      const int turn = row / (teams * BATCH), of = row % (teams * BATCH);
      const float* const from = all + (of / BATCH * p.wide) * kSums + (turn * BATCH + of % BATCH) * MT + m;
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
  p.padded = p.n % CH != 0 || p.chunks % 32 != 0;
  p.wide = 1;
  while (p.wide < kWarps && p.wide < tiles) p.wide *= 2;
  const size_t S = size_t{1} << p.L;
  p.copies_log2 = 0;
  if (HELD == F32) {
    while (p.copies_log2 < 5 && (S * 4 << (p.copies_log2 + 1)) <= (128u << 10)) ++p.copies_log2;
  }
  const size_t table = HELD == F32 ? S * 4 << p.copies_log2 : HELD == HALVES ? kHalf + 16 : kHalf;
  const size_t smem = (table + 15) / 16 * 16 + sizeof(float) * kWarps * kSums;
  auto* const kernel = trellis_matmul_kernel<K, MT, CH, HELD>;
  static PerDevice done;
  if (!allow_shared(reinterpret_cast<const void*>(kernel), done)) return BCJR_ERR_CUDA;
  const int teams = kWarps / p.wide;
  const int useful = (p.rows + teams - 1) / teams;
  const dim3 grid(static_cast<unsigned>(useful < sms ? useful : sms), static_cast<unsigned>((p.tokens + MT - 1) / MT));
  kernel<<<grid, kWarps * 32, smem, s>>>(p);
  return launched();
}

template <int K, Held HELD>
bcjr_status launch_tokens(const Params& p, int sms, cudaStream_t s) {
  // 16 columns a lane while their inputs leave registers for the rows' words: one
  // token 20.4 us (8 columns: 23.8), four 43.7 us (8 columns: 27.0)
  if (p.tokens == 1) return launch<K, 1, 16, HELD>(p, sms, s);
  if (p.tokens <= 4) return launch<K, 4, 8, HELD>(p, sms, s);
  return launch<K, 8, 8, HELD>(p, sms, s);
}

template <int K>
bcjr_status launch_held(Params p, int sms, cudaStream_t s) {
  if (tokens_mma::plan(p, sms)) return tokens_mma::launch_types<K>(p, sms, s);
  if (p.L < 16) return launch_tokens<K, F32>(p, sms, s);
  if (p.c_dtype == BCJR_F32) return launch_tokens<K, HALVES>(p, sms, s);
  if (p.c_dtype == BCJR_BF16) return launch_tokens<K, B16>(p, sms, s);
  return launch_tokens<K, H16>(p, sms, s);
}

}  // namespace
}  // namespace bcjr
