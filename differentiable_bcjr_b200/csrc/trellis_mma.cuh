// trellis_mma.cuh -- tokens times packed trellis weights where both are of one 16-bit type (bcjr_trellis_matmul).
//
// Codewords and inputs are then fragments of mma.m16n8k16 as they are: 16 rows
// of weights are its rows and eight tokens its columns, so that the matrix
// instruction adds the products up and a weight costs its gather, its window (a
// shift and a mask) and half a packing, for one token or eight.  What k index of
// the instruction a column of the matrix has is free as long as both operands
// agree: a lane takes 16 consecutive steps of two rows, four instructions'
// worth, out of two or three words of each row's stream.
//
// The gathers bound it: 32 random ones meet in about 3.5 of 32 banks.  2^16
// states are held as they are (16 bits each); smaller codebooks as words, in
// 2^(15 - L) copies up to 32, lane l reading copy l mod copies, 2^(17 - L) bytes
// apart so that the same constant shifts lead to any of them.
//
// A warp keeps the tokens of its 64 columns in registers and walks down its
// tiles of 16 rows, two tiles' words on their way; its sums stay in shared
// memory, where the warps of other columns are added in a fixed order.  CTAs
// share the rows out by eights; a tile of only eight skips the gathers of its
// lower half.
//
// Measured, device time a call with the words in memory (in the L2 cache), bf16:
// 8192 x 2048, k = 4, 2^16 states, 8 tokens 16.5 us (15.2; multiply-adds and warp
// sums: 21.8; the gathers alone 6.6; launch and codebook 4.1), 16 tokens 23.6
// (19.8); 8192 x 8192, k = 2, 2^8 states, 2 tokens 31.4 (29.1).  More than 16 tokens
// take as many passes over the words (256 tokens of 8192 x 2048: 301 us).
#pragma once
#include <cooperative_groups.h>

#include <type_traits>

#include "layer_util.cuh"
#include "trellis_internal.h"

namespace bcjr {
namespace {
namespace tokens_mma {

namespace cg = cooperative_groups;

using Params = TrellisMatmulParams;

constexpr int kWarps = 16;
constexpr int kTiles = 4;             // whose sums a warp has room for
constexpr uint32_t kTable = 131072;   // bytes of the codebook
constexpr int kSplit = 4;             // CTAs of a cluster at most

// c += a b, or c = a b for the FIRST
template <bool F16, bool FIRST>
__device__ __forceinline__ void mma(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  if constexpr (FIRST && F16)
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
        : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
  else if constexpr (FIRST)
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
        : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
  else if constexpr (F16)
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// a / b by the number 2^40 / b, rounded up: exact where a b < 2^40.
__device__ __forceinline__ int divided(int a, uint64_t inverse) { return static_cast<int>(static_cast<uint64_t>(a) * inverse >> 40); }

// bits [at, at + 16) of a stream's words, one place up
template <int N>
__device__ __forceinline__ uint32_t window(const uint32_t (&a)[N], int at) {
  const int down = 47 - at % 32;
  return down >= 32 ? a[at / 32] >> (down - 32) : __funnelshift_r(a[at / 32 + 1], a[at / 32], down);
}

__device__ __forceinline__ bool finite16(uint32_t bits, uint32_t exponent) { return (bits & exponent) != exponent; }

// The codebook into shared memory, asynchronously where nothing has to be known of it.  False if this thread met a codeword that is
// not finite; `exponent`: the exponent field of one.
template <bool WORDS>
__device__ __forceinline__ bool copy_in(unsigned char* to, const Params& p, int copies_log2, uint32_t exponent) {
  const uint16_t* const from = static_cast<const uint16_t*>(p.codebook);
  bool fine = true;
  if constexpr (WORDS) {
#pragma unroll 8
    for (int i = threadIdx.x; i < (1 << p.L << copies_log2); i += kWarps * 32) {
      const int state = i >> copies_log2, copy = i & ((1 << copies_log2) - 1);
      const uint32_t v = __ldg(from + state);
      *reinterpret_cast<uint32_t*>(to + (state << (17 - p.L)) + copy * 4) = v;
      fine = fine && finite16(v, exponent);
    }
  } else if (!p.padded && (reinterpret_cast<uintptr_t>(from) & 15) == 0) {
    const uint32_t at = static_cast<uint32_t>(__cvta_generic_to_shared(to));
#pragma unroll
    for (int i = threadIdx.x; i < static_cast<int>(kTable / 16); i += kWarps * 32)
      asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(at + i * 16), "l"(from + i * 8) : "memory");
  } else if ((reinterpret_cast<uintptr_t>(from) & 15) == 0) {
    auto check = [&](uint32_t w) { fine = fine && finite16(w, exponent) && finite16(w >> 16, exponent); };
#pragma unroll 8
    for (int i = threadIdx.x; i < static_cast<int>(kTable / 16); i += kWarps * 32) {
      const uint4 v = __ldg(reinterpret_cast<const uint4*>(from) + i);
      reinterpret_cast<uint4*>(to)[i] = v;
      check(v.x);
      check(v.y);
      check(v.z);
      check(v.w);
    }
  } else {
    for (int i = threadIdx.x; i < static_cast<int>(kTable / 2); i += kWarps * 32) {
      const uint16_t v = from[i];
      reinterpret_cast<uint16_t*>(to)[i] = v;
      fine = fine && finite16(v, exponent);
    }
  }
  return fine;
}

// WORDS: a codeword in a word (L < 16).  SETS: of eight tokens.
template <int K, bool WORDS, bool F16, int SETS>
__global__ void __launch_bounds__(kWarps * 32, 1) trellis_mma_kernel(const __grid_constant__ Params p) {
  constexpr int CH = 16;  // steps of a chunk
  constexpr int STEP = (CH * K) % 32 == 0 ? 32 : 16;  // a chunk's first bit in its word is a multiple of this
  constexpr int N = (32 - STEP + (CH - 1) * K + 16 + 31) / 32;
  constexpr int RING = 2;
  extern __shared__ __align__(16) unsigned char smem[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  float4* const sums = reinterpret_cast<float4*>(smem + kTable) + warp * kTiles * SETS * 32 + lane;  // [tile][set][lane]
  const int copies_log2 = WORDS ? min(15 - p.L, 5) : 0;
  const uint32_t mask = WORDS ? 0x1FFFEu & ~((2u << (16 - p.L)) - 1u) : 0x1FFFEu;
  const uint32_t copy = WORDS ? (lane & ((1 << copies_log2) - 1)) * 4 : 0;

  const int teams = kWarps / p.wide, team = warp / p.wide, place = warp % p.wide;
  cg::cluster_group cluster = cg::this_cluster();
  const int split = static_cast<int>(cluster.num_blocks()), part = static_cast<int>(cluster.block_rank());
  const int first = part * p.wide + place, stride = p.wide * split;  // of the warp's columns
  const int octets = (p.rows + 7) / 8, shares = gridDim.x / split, share = blockIdx.x / split;
  const int r_begin = static_cast<int>(static_cast<long long>(octets) * share / shares) * 8;
  const int r_end = min(static_cast<int>(static_cast<long long>(octets) * (share + 1) / shares) * 8, p.rows);
  const int token0 = blockIdx.y * 8 * SETS;
  const int tokens = min(8 * SETS, p.tokens - token0);
  const uint32_t row_words = static_cast<uint32_t>(p.seqs) * p.words;
  const uint16_t* const x = static_cast<const uint16_t*>(p.x);

  // codewords that are not finite matter where a chunk is padded
  const bool fine = copy_in<WORDS>(smem, p, copies_log2, F16 ? 0x7C00u : 0x7F80u);
  const bool all_finite = p.padded ? __syncthreads_and(fine) != 0 : true;

  for (int r0 = r_begin; r0 < r_end; r0 += kTiles * 16 * teams) {
    const int r1 = min(r0 + kTiles * 16 * teams, r_end);
    const int mine = max(0, ((r1 - r0 + 15) / 16 - team + teams - 1) / teams);  // tiles of this team
    // GUARDED: what lies behind a chunk's end is left out.  Otherwise it is a
    // product with an input of 0, which is enough where codewords are finite.
    auto walk = [&](auto guarded) {
      constexpr bool GUARDED = decltype(guarded)::value;
      const char* const base = reinterpret_cast<const char*>(p.packed + static_cast<size_t>(r0) * row_words);  // offsets from here fit 32 bits

      // what is on its way: words, tokens and scales of a tile and 64 columns
      uint32_t words[RING][2][N], xs[RING][SETS][8];
      float scale[RING][2];
      int count[RING], skew[RING];  // steps of the lane's chunk, its first bit's place
      // the next to be fetched: columns and tile, and for the columns the lane's chunk
      int f_step = first, f_tile = 0, f_count = 0, f_col = 0, f_skew = 0;
      uint32_t f_word[N];
      const float* f_scale = nullptr;

      auto fetch = [&](int slot) {
        if (f_step >= p.steps || mine == 0) return;
        if (f_tile == 0) {
          const int unit = divided(f_step, p.unit_inverse), at = (f_step - unit * p.unit_steps) * 4 + t;
          const bool have = at < p.unit_chunks;
          const int q = have ? unit * p.unit_chunks + at : 0;
          const int seq = divided(q, p.seq_inverse), t0 = (q - seq * p.per_seq) * CH;
          f_count = have ? min(CH, p.n - t0) : 0;
          f_col = seq * p.n + t0;
          // a chunk at the sequence's end may have fewer words left
#pragma unroll
          for (int i = 0; i < N; ++i) f_word[i] = (seq * p.words + min((t0 * K >> 5) + i, p.words - 1)) * 4;
          f_skew = t0 * K & 31;
          if (p.scales) f_scale = p.scales + static_cast<size_t>(unit) * p.rows;
        }
        if (f_tile < RING) {  // this slot has the tokens of other columns
          count[slot] = f_count;
          skew[slot] = f_skew;
#pragma unroll
          for (int set = 0; set < SETS; ++set) {
            // (columns of the instruction behind the last token compute with it; nobody reads their sums)
            const uint16_t* const from = x + static_cast<size_t>(token0 + min(set * 8 + g, tokens - 1)) * p.cols + f_col;
            if (f_count == CH && (reinterpret_cast<uintptr_t>(from) & 15) == 0) {
              const uint4 lo = __ldg(reinterpret_cast<const uint4*>(from)), hi = __ldg(reinterpret_cast<const uint4*>(from) + 1);
              xs[slot][set][0] = lo.x, xs[slot][set][1] = lo.y, xs[slot][set][2] = lo.z, xs[slot][set][3] = lo.w;
              xs[slot][set][4] = hi.x, xs[slot][set][5] = hi.y, xs[slot][set][6] = hi.z, xs[slot][set][7] = hi.w;
            } else {
#pragma unroll
              for (int i = 0; i < 8; ++i) {
                const uint32_t a = 2 * i < f_count ? __ldg(from + 2 * i) : 0u, b = 2 * i + 1 < f_count ? __ldg(from + 2 * i + 1) : 0u;
                xs[slot][set][i] = a | b << 16;
              }
            }
          }
        }
        // rows behind the last compute with it
        const int row = (team + f_tile * teams) * 16 + g, last = r1 - r0 - 1;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int at = min(row + 8 * h, last);
#pragma unroll
          for (int i = 0; i < N; ++i) words[slot][h][i] = __ldg(reinterpret_cast<const uint32_t*>(base + (static_cast<uint32_t>(at) * (row_words * 4) + f_word[i])));
          scale[slot][h] = p.scales ? __ldg(f_scale + r0 + at) : 1.f;
        }
        if (++f_tile == mine) {
          f_tile = 0;
          f_step += stride;
        }
      };
#pragma unroll
      for (int i = 0; i < RING; ++i) fetch(i);
      if (!p.padded && r0 == r_begin) {  // the codebook is there now
        asm volatile("cp.async.wait_all;" ::: "memory");
        __syncthreads();
      }

      // walked in the order in which they were fetched
      int tile = 0, step = first;
      while (step < p.steps && mine != 0) {
#pragma unroll
        for (int slot = 0; slot < RING; ++slot) {
          if (step >= p.steps) break;
          uint32_t w[4][4];  // the fragments of four instructions
          auto gather = [&](int h) {
            uint32_t a[N + 1];
#pragma unroll
            for (int i = 0; i < N; ++i) a[i] = words[slot][h][i];
            a[N] = 0;
            if constexpr (STEP != 32) {
#pragma unroll
              for (int i = 0; i < N; ++i) a[i] = __funnelshift_l(a[i + 1], a[i], skew[slot]);
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const uint32_t lo = (window(a, 2 * i * K) & mask) | copy, hi = (window(a, (2 * i + 1) * K) & mask) | copy;
              uint32_t v;
              if constexpr (WORDS)
                v = __byte_perm(*reinterpret_cast<const uint32_t*>(smem + lo), *reinterpret_cast<const uint32_t*>(smem + hi), 0x5410);
              else
                v = __byte_perm(*reinterpret_cast<const uint16_t*>(smem + lo), *reinterpret_cast<const uint16_t*>(smem + hi), 0x5410);
              if (GUARDED) v = 2 * i + 1 < count[slot] ? v : 2 * i < count[slot] ? v & 0xFFFFu : 0u;
              w[i / 2][i % 2 * 2 + h] = v;
            }
          };
          gather(0);
          if ((team + tile * teams) * 16 + 8 < r1 - r0) gather(1);
          else w[0][1] = w[0][3] = w[1][1] = w[1][3] = w[2][1] = w[2][3] = w[3][1] = w[3][3] = 0;
#pragma unroll
          for (int set = 0; set < SETS; ++set) {
            float c[4];
            mma<F16, true>(c, w[0], xs[slot][set][0], xs[slot][set][1]);
#pragma unroll
            for (int j = 1; j < 4; ++j) mma<F16, false>(c, w[j], xs[slot][set][2 * j], xs[slot][set][2 * j + 1]);
            float4* const to = sums + (tile * SETS + set) * 32;
            float4 v = make_float4(c[0] * scale[slot][0], c[1] * scale[slot][0], c[2] * scale[slot][1], c[3] * scale[slot][1]);
            if (step != first) {
              const float4 before = *to;
              v.x += before.x;
              v.y += before.y;
              v.z += before.z;
              v.w += before.w;
            }
            *to = v;
          }
          fetch(slot);
          if (++tile == mine) {
            tile = 0;
            step += stride;
          }
        }
      }
    };
    if (all_finite) walk(std::false_type{});
    else walk(std::true_type{});
    if (split > 1) cluster.sync();
    else __syncthreads();
    const int rows = r1 - r0, in_use = min(stride, p.steps);
    for (int i = part * kWarps * 32 + threadIdx.x; i < rows * tokens; i += split * kWarps * 32) {
      const int token = i / rows, row = i - token * rows, of = row >> 4;
      // lane 4 (row mod 8) + (token mod 8) / 2 has tokens / 2 and the next of two rows
      const int at = ((of % teams * p.wide * kTiles + of / teams) * SETS + (token >> 3)) * 128 +
                     ((row & 7) * 4 + (token & 7) / 2) * 4 + (row >> 3 & 1) * 2 + (token & 1);
      float v = 0.f;
      for (int q = 0; q * p.wide < in_use; ++q) {
        const float* const all = reinterpret_cast<const float*>(smem + kTable);
        const float* const from = (split == 1 ? all : cluster.map_shared_rank(all, q)) + at;
        const int warps = min(p.wide, in_use - q * p.wide);
#pragma unroll 4
        for (int w = 0; w < warps; ++w) v += from[w * kTiles * SETS * 128];
      }
      store_from_f32(p.y, p.x_dtype, static_cast<size_t>(token0 + token) * p.rows + r0 + row, v);
    }
    if (split > 1) cluster.sync();  // nobody goes on while its sums are read
    else __syncthreads();
  }
}

template <int K, bool WORDS, bool F16, int SETS>
bcjr_status launch(Params p, int sms, cudaStream_t s) {
  p.wide = 1;
  while (p.wide < kWarps && p.wide < p.steps) p.wide *= 2;
  const int smem = static_cast<int>(kTable) + kWarps * kTiles * SETS * 32 * static_cast<int>(sizeof(float4));
  auto* const kernel = trellis_mma_kernel<K, WORDS, F16, SETS>;
  static PerDevice done;
  if (!allow_shared(reinterpret_cast<const void*>(kernel), done)) return BCJR_ERR_CUDA;
  const int teams = kWarps / p.wide, useful = ((p.rows + 7) / 8 + teams - 1) / teams;
  // Few rows: the CTAs of a cluster split the columns (8 tokens of 100 x 8192: 11.2 us
  // with one, 8.8 with two, 8.3 with four, 10.3 with eight).
  int split = 1;
  while (split < kSplit && useful * split * 2 <= sms && p.steps >= 2 * kWarps * split) split *= 2;
  const int shares = useful < sms / split ? useful : sms / split;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(shares * split), static_cast<unsigned>((p.tokens + 8 * SETS - 1) / (8 * SETS)));
  cfg.blockDim = dim3(kWarps * 32);
  cfg.dynamicSmemBytes = static_cast<size_t>(smem);
  cfg.stream = s;
  cudaLaunchAttribute attr = {};
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = static_cast<unsigned>(split);
  attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, kernel, p) != cudaSuccess) {
    cudaGetLastError();
    return BCJR_ERR_CUDA;
  }
  return BCJR_OK;
}

// Whether the call takes this form, and the plan for it: columns in chunks of
// 16 steps, four of which (one scale's) a warp takes at a time.
//
// One token leaves seven of the instruction's eight columns idle; multiply-adds
// of a lane's own gathers are then less work (bf16, 2048 x 8192, 2^16 states, one
// token: 12.3 us against 15.5; 8192 x 8192, 2^8 states: 25.0 against 28.9; two
// tokens: 16.6 against 15.8 and 41.1 against 29.2), unless a row has not a
// chunk for each lane (64 x 256: 6.5 against 4.1).  So are a few tokens where
// there are few rows to share out and many columns (2 tokens of 100 x 8192: 7.1
// against 8.2; 8 tokens: 10.3 against 8.3).
inline bool plan(Params& p, int sms) {
  if (p.x_dtype != p.c_dtype || p.x_dtype == BCJR_F32) return false;
  // the rows of a CTA's walk are addressed with 32 bits
  if (static_cast<long long>(p.seqs) * p.words >= (1LL << 30) / (kTiles * 16 * kWarps)) return false;
  p.per_seq = (p.n + 15) / 16;
  p.chunks = p.seqs * p.per_seq;
  p.unit_chunks = !p.scales ? p.chunks : p.group < p.n ? p.group / 16 : p.group / p.n * p.per_seq;
  p.unit_steps = (p.unit_chunks + 3) / 4;
  p.steps = p.chunks / p.unit_chunks * p.unit_steps;
  p.padded = p.n % 16 != 0 || p.unit_chunks % 4 != 0;
  if (p.steps >= 1 << 18) return false;  // four chunks each: quotients are exact
  if (p.tokens == 1 && p.chunks >= 32) return false;
  if (p.tokens <= 4 && p.rows <= 2 * sms && p.chunks >= 256) return false;
  p.seq_inverse = ((1ull << 40) + p.per_seq - 1) / p.per_seq;
  p.unit_inverse = ((1ull << 40) + p.unit_steps - 1) / p.unit_steps;
  return true;
}

template <int K, bool WORDS, bool F16>
bcjr_status launch_sets(const Params& p, int sms, cudaStream_t s) {
  return p.tokens <= 8 ? launch<K, WORDS, F16, 1>(p, sms, s) : launch<K, WORDS, F16, 2>(p, sms, s);
}

template <int K>
bcjr_status launch_types(const Params& p, int sms, cudaStream_t s) {
  if (p.x_dtype == BCJR_F16) return p.L < 16 ? launch_sets<K, true, true>(p, sms, s) : launch_sets<K, false, true>(p, sms, s);
  return p.L < 16 ? launch_sets<K, true, false>(p, sms, s) : launch_sets<K, false, false>(p, sms, s);
}

}  // namespace tokens_mma
}  // namespace
}  // namespace bcjr
