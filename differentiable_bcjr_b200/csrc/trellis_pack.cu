// trellis_pack.cu -- hard-decoded states to k bits a weight (bcjr_trellis_pack).
//
// A thread writes one 32-bit word of a sequence's stream from the low k bits
// of the 8 to 33 states that begin or end in it.  Reading the states (4 B a
// weight) bounds the call.
#include "layer_util.cuh"

namespace {

using namespace bcjr;

struct Params {
  const int32_t* states;
  uint32_t* packed;
  int* bad;
  int L, n, words;
  long long total;  // words of all sequences
};

template <int K>
__global__ void __launch_bounds__(256) trellis_pack_kernel(const __grid_constant__ Params p) {
  const long long id = static_cast<long long>(blockIdx.x) * 256 + threadIdx.x;
  if (id >= p.total) return;
  const long long seq = id / p.words;
  const int j = static_cast<int>(id - seq * p.words);
  const int32_t* const s = p.states + seq * p.n;
  // Step t ends at bit t K + L of the stream; the steps that end behind the
  // word's first bit and do not begin behind its last are those that touch it
  // with their last K bits (or, the first step, with any).
  const int begin = 32 * j;
  uint32_t word = 0;
  bool bad = false;
  int t = (begin - p.L) / K + 1;  // the first step that ends behind `begin`
  if (begin < p.L) t = 0;
  uint32_t before = t > 0 ? static_cast<uint32_t>(s[t - 1]) : 0u;
  for (; t < p.n; ++t) {
    const int end = t * K + p.L;  // relative to the stream
    const int bits = t == 0 ? p.L : K;
    if (end - bits >= begin + 32) break;
    const uint32_t state = static_cast<uint32_t>(s[t]);
    const uint32_t mask = (1u << p.L) - 1u;
    bad |= (state & ~mask) != 0u || (t > 0 && (state >> K) != (before & (mask >> K)));
    before = state;
    const uint32_t v = state & ((1u << bits) - 1u);
    const int up = begin + 32 - end;  // places below the word's last bit
    word |= up >= 0 ? v << up : v >> -up;
  }
  p.packed[id] = word;
  if (bad && p.bad) *p.bad = 1;
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
  p.total = static_cast<long long>(p.words) * n_seq;
  const long long grid = (p.total + 255) / 256;
  if (grid > 0x7FFFFFFFll) return BCJR_ERR_UNSUPPORTED;
  cudaStream_t s = as_stream(stream);
  switch (k) {
    case 1: trellis_pack_kernel<1><<<static_cast<unsigned>(grid), 256, 0, s>>>(p); break;
    case 2: trellis_pack_kernel<2><<<static_cast<unsigned>(grid), 256, 0, s>>>(p); break;
    case 3: trellis_pack_kernel<3><<<static_cast<unsigned>(grid), 256, 0, s>>>(p); break;
    default: trellis_pack_kernel<4><<<static_cast<unsigned>(grid), 256, 0, s>>>(p); break;
  }
  return launched();
}
