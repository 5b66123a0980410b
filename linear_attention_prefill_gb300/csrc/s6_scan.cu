// s6_scan.cu - the S6 scan on bf16 inputs (s6_scan.cuh), and how a call is split over time.
#include "s6_scan.cuh"

namespace gdn {

S6Split s6_split(int N, int T, int dim, int Ns, bool packed) {
  const int tiles = (dim + kCh - 1) / kCh;
  S6Split s{tiles, 0, 0, 0, 0, 0, 0};
  if (N <= 0) return s;
  const long long ctas = (long long)N * tiles;
  const long long per_seq = (packed ? (long long)T : (long long)N * T) / N;  // packed: their mean
  const long long waves = (ctas + kSms - 1) / kSms;
  // Cycles an SM takes for a token of 32 channels (measured at Ns = 16, bf16, 4096 tokens with
  // the launch and the ends): 62 with one CTA, 117 with two, 192 with four (the rule's 48 n + 20
  // gives 116 and 212: at four and more a split is taken a little early); 74 for the two passes of
  // a split channel, with four CTAs an SM; 170 for the two passes along one chunk, and about 10000
  // for the summaries' launch and the chunks' beginnings.  Other state counts and fp32 go by the
  // same numbers, which were not measured for them (with 64 states, for one, a single CTA fits an SM).
  const auto cost = [](long long ctas_an_sm) { return ctas_an_sm == 1 ? 62 : 48 * ctas_an_sm + 20; };
  const auto chunk_of = [&](long long parts) {
    parts = parts < 2 ? 2 : parts > 128 ? 128 : parts;
    const long long c = (per_seq + parts - 1) / parts;
    return (c < 128 ? 128 : (c + 15) / 16 * 16);
  };
  const auto cost_split = [&](long long tiles_split, long long chunk) {
    const long long work = tiles_split * per_seq * 74 / kSms, chain = chunk * 170;
    return (work > chain ? work : chain) + 10000;
  };
  const long long none = per_seq * cost(waves);
  // every channel split, into enough chunks for four rounds of two CTAs an SM; or whole waves of
  // CTAs and the tiles beyond them split, one more CTA an SM beside the whole ones
  const long long chunk_all = chunk_of(8 * kSms / ctas);
  const long long all = cost_split(ctas, chunk_all);
  const long long rounds = ctas / kSms;
  const int full = (int)(rounds * kSms / N);
  const long long rest = ctas - (long long)N * full;
  const bool can = full > 0 && rest > 0;
  const long long chunk_rest = can ? chunk_of(kSms / rest) : 0;
  const long long some = can ? per_seq * cost(rounds) + cost_split(rest, 0) : 0;
  s.lone = waves == 1 ? 1 : 0;
  if (none <= all && (!can || none <= some)) {
    // Packed sequences' lengths are not known here: one long sequence among short ones would
    // leave a few CTAs alone with it.  Where it has few channels its chunks are of twice the
    // mean length; whatever is shorter is one chunk and computed once, as it would be anyway.
    // 512 channels, one of 8000 tokens and 15 of 12: 348 -> 115 us; 40 of 200: 33 -> 37; 16 of
    // 1024: 64 -> 84.  With more channels (2049) even batches lose more (72 -> 95) and uneven
    // ones gain less.  (The mean rounds down, to 0 where there are more sequences than tokens.)
    const long long chunk = per_seq ? (2 * per_seq + 127) / 128 * 128 : 128;
    if (!packed || tiles > kSms / 4 || chunk >= T) return s;
    s.whole = 0;
    s.chunk = (int)chunk;
  } else {
    const bool part = can && some < all;
    s.whole = part ? full : 0;
    s.lone = part && rounds == 1 ? 1 : 0;
    s.chunk = (int)(part ? chunk_rest : chunk_all);
  }
  s.slots = packed ? (long long)T / s.chunk + N + 1
                   : (long long)N * (((long long)T + s.chunk - 1) / s.chunk);
  const size_t up = 63, wdim = dim - s.whole * kCh;
  s.sum_floats = ((size_t)s.slots * wdim + up) & ~up;
  s.h_floats = ((size_t)s.slots * wdim * Ns + up) & ~up;
  s.ws_bytes = (s.sum_floats + s.h_floats + (size_t)N * wdim * Ns) * sizeof(float);
  return s;
}

cudaError_t launch_s6_f32(const S6Params& p, cudaStream_t stream);

cudaError_t launch_s6(const S6Params& p, bool f32, cudaStream_t stream) {
  return f32 ? launch_s6_f32(p, stream) : launch_scan<__nv_bfloat16>(p, stream);
}

}  // namespace gdn
