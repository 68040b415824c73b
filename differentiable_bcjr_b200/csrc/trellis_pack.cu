// trellis_pack.cu -- hard-decoded states to k bits a weight (bcjr_trellis_pack).
//
// The stream of a sequence is the state_bits - k upper bits of its first state
// and then the low k bits of every state.  A warp takes 32 (or 8)
// pieces of 32 states: it loads them piece by piece, coalesced, leaves the low bits as bytes in
// shared memory, and then lane l puts the words of piece l together.  What
// precedes a piece in the stream are the upper bits of its first state, so no
// piece waits for another.  Reading the states (4 B a weight) bounds the call:
// 65536 sequences of 256 states take 16.1 us from memory (4.7 TB/s), 9.3 from the
// L2 cache.
#include "layer_util.cuh"

namespace {

using namespace bcjr;

constexpr int kWarps = 8;
constexpr int kPitch = 36;  // bytes of a piece's codes in shared memory: lanes read theirs from different banks

struct Params {
  const int32_t* states;
  uint32_t* packed;
  int* bad;
  int L, n, words;
  int per_seq;      // pieces of a sequence
  bool dense;       // all pieces are whole, and 16-byte aligned
  long long total;  // pieces of all sequences
};

// PIECES: of a warp; 8 where 32 would leave most of the GPU without a warp.
template <int K, bool CHECK, int PIECES>
__global__ void __launch_bounds__(kWarps * 32) trellis_pack_kernel(const __grid_constant__ Params p) {
  __shared__ __align__(4) uint8_t codes[kWarps][32 * kPitch];
  const int lane = threadIdx.x & 31;
  uint8_t* const mine = codes[threadIdx.x >> 5];
  const long long q0 = (static_cast<long long>(blockIdx.x) * kWarps + (threadIdx.x >> 5)) * PIECES;
  if (q0 >= p.total) return;
  // (a division of 64 bits takes as long as a piece)
  long long seq = p.total <= 0x7FFFFFFFll ? static_cast<uint32_t>(q0) / static_cast<uint32_t>(p.per_seq) : q0 / p.per_seq;
  int piece = static_cast<int>(q0 - seq * p.per_seq);
  // lane l's own piece
  const int ahead = (piece + lane) / p.per_seq;
  const long long my_seq = seq + ahead;
  const int my_piece = piece + lane - ahead * p.per_seq;
  const bool have = lane < PIECES && q0 + lane < p.total;
  const uint32_t my_first = have ? static_cast<uint32_t>(p.states[my_seq * p.n + 32 * my_piece]) : 0u;

  bool bad = false;
  if (!CHECK && p.dense && q0 + PIECES <= p.total) {
    // whole pieces that follow one another: four states a lane at a time
    const int4* const from = reinterpret_cast<const int4*>(p.states + q0 * 32) + lane;
    int4 v[PIECES / 4];
#pragma unroll
    for (int i = 0; i < PIECES / 4; ++i) v[i] = __ldcs(from + i * 32);
#pragma unroll
    for (int i = 0; i < PIECES / 4; ++i) {
      constexpr uint32_t low = (1u << K) - 1u;
      const uint32_t four = (v[i].x & low) | ((v[i].y & low) << 8) | ((v[i].z & low) << 16) | ((v[i].w & low) << 24);
      *reinterpret_cast<uint32_t*>(mine + (i * 4 + (lane >> 3)) * kPitch + (lane & 7) * 4) = four;
    }
  } else
#pragma unroll 8
  for (int i = 0; i < PIECES; ++i) {
    uint32_t state = 0;
    if (q0 + i < p.total) {
      const int t = 32 * piece + lane;
      const int32_t* const at = p.states + seq * p.n + t;
      if (t < p.n) state = static_cast<uint32_t>(*at);
      if constexpr (CHECK) {
        const uint32_t mask = (1u << p.L) - 1u;
        uint32_t before = __shfl_up_sync(~0u, state, 1);
        if (lane == 0 && t > 0) before = static_cast<uint32_t>(at[-1]);
        if (t < p.n) bad |= (state & ~mask) != 0u || (t > 0 && (state >> K) != (before & (mask >> K)));
      }
    }
    mine[i * kPitch + lane] = static_cast<uint8_t>(state & ((1u << K) - 1u));
    if (++piece == p.per_seq) {
      piece = 0;
      ++seq;
    }
  }
  if (CHECK && bad) *p.bad = 1;
  __syncwarp();
  if (!have) return;

  uint32_t body[K + 1];  // 32 K bits, the first state's highest; then none
#pragma unroll
  for (int w = 0; w <= K; ++w) body[w] = 0;
#pragma unroll
  for (int w = 0; w < 8; ++w) {
    const uint32_t four = *reinterpret_cast<const uint32_t*>(mine + lane * kPitch + 4 * w);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t c = (four >> (8 * i)) & ((1u << K) - 1u);
      const int bit = (4 * w + i) * K, up = 32 - K - bit % 32;  // places below the word's last bit
      if (up >= 0) {
        body[bit / 32] |= c << up;
      } else {
        body[bit / 32] |= c >> -up;
        body[bit / 32 + 1] |= c << (32 + up);
      }
    }
  }
  const int o = p.L - K;  // bits before the piece that belong to its first word
  uint32_t* const out = p.packed + my_seq * p.words;
  uint32_t before = my_first >> K;
#pragma unroll
  for (int w = 0; w <= K; ++w) {
    // the word after the last piece's holds the bits that are left over
    const int j = K * my_piece + w;
    if (j < p.words && (w < K || my_piece == p.per_seq - 1)) out[j] = __funnelshift_r(body[w], before, o);
    before = body[w];
  }
}

template <int K, int PIECES>
bcjr_status launch_pieces(const Params& p, cudaStream_t s) {
  const long long grid = (p.total + PIECES * kWarps - 1) / (PIECES * kWarps);
  if (grid > 0x7FFFFFFFll) return BCJR_ERR_UNSUPPORTED;
  if (p.bad) trellis_pack_kernel<K, true, PIECES><<<static_cast<unsigned>(grid), kWarps * 32, 0, s>>>(p);
  else trellis_pack_kernel<K, false, PIECES><<<static_cast<unsigned>(grid), kWarps * 32, 0, s>>>(p);
  return launched();
}

template <int K>
bcjr_status launch(const Params& p, int sms, cudaStream_t s) {
  return p.total < 32ll * kWarps * 2 * sms ? launch_pieces<K, 8>(p, s) : launch_pieces<K, 32>(p, s);
}

}  // namespace

extern "C" bcjr_status bcjr_trellis_pack(const int32_t* states, int state_bits, int k, int seq_len, int n_seq,
                                         uint32_t* packed, int* bad, bcjr_stream_t stream) {
  if (state_bits < 1 || k < 1 || k > state_bits || seq_len < 1 || n_seq < 0) return BCJR_ERR_INVALID_ARG;
  // bit positions are counted in ints
  if (k > 4 || state_bits > 16 || seq_len > (1 << 28)) return BCJR_ERR_UNSUPPORTED;
  if (n_seq == 0) return BCJR_OK;
  if (!states || !packed || !ptr_aligned(states, 4) || !ptr_aligned(packed, 4) || !ptr_aligned(bad, 4))
    return BCJR_ERR_INVALID_ARG;
  Params p = {};
  p.states = states;
  p.packed = packed;
  p.bad = bad;
  p.L = state_bits;
  p.n = seq_len;
  p.words = static_cast<int>((static_cast<long long>(seq_len) * k + state_bits - k + 31) / 32);
  p.per_seq = (seq_len + 31) / 32;
  p.dense = seq_len % 32 == 0 && ptr_aligned(states, 16);
  p.total = static_cast<long long>(p.per_seq) * n_seq;
  const int sms = sm_count();
  if (sms <= 0) return BCJR_ERR_CUDA;
  cudaStream_t s = as_stream(stream);
  switch (k) {
    case 1: return launch<1>(p, sms, s);
    case 2: return launch<2>(p, sms, s);
    case 3: return launch<3>(p, sms, s);
    default: return launch<4>(p, sms, s);
  }
}
