// How reads over 8-bit caches are spread over the GPU: host arithmetic, plain C++.
//
// The host knows how many tokens a call has and how many sequences, but not the offsets.
// A plan chooses how the work is done, from what the range of sequences is likely to
// hold; whatever the offsets say, all of it is done, and every bound holds.
#pragma once

#include <algorithm>
#include <cstdint>

#ifdef __CUDACC__
#define PA_HOST_DEVICE __host__ __device__
#else
#define PA_HOST_DEVICE
#endif

namespace pa {
namespace quant {

// Tokens that a read of nseq of a call's num_seqs sequences is planned with. The others
// are taken to have one token each: a prefill range stands beside decode sequences. (With
// the call's tokens instead, 200 decode sequences of 500 to 4000 keys and 4 drafts of 5 tokens
// over up to 16000, 4 heads per kv head, took 340 us; now 226, of which 186 and 39 are
// theirs in calls of their own.)
inline int64_t range_tokens(int64_t num_tokens, int64_t num_seqs, int64_t nseq) {
  return std::max<int64_t>(1, num_tokens - (num_seqs - nseq));
}

// The grid of the prefill kernel, a CTA per unit (`per` consecutive tokens of a sequence) and
// kv head. Where the planned ones are few, each is split: `splits` CTAs share its keys.
struct PrefillGrid {
  int64_t ctas;     // units and kv heads, at most (whatever the offsets)
  int64_t planned;  // of them those that are split
  int splits;
  int64_t launched() const { return ctas + planned * (splits - 1); }
};
inline PrefillGrid prefill_grid(int64_t num_tokens, int64_t tokens, int64_t nseq, int64_t kvh,
                                int64_t per, int64_t tiles, int num_sms) {
  // (a sequence with tokens has at most one unit that is not full)
  auto units = [&](int64_t t) { return (t / per + std::min(nseq, t)) * kvh; };
  PrefillGrid g;
  g.ctas = units(num_tokens);
  g.planned = std::min(g.ctas, units(tokens));
  // parts of four tiles at least, as long as there are SMs
  g.splits = (int)std::max<int64_t>(1, std::min<int64_t>(num_sms / g.planned, tiles / 4));
  return g;
}

// What CTA `cta` of such a grid does: part `split` of `splits` of unit and kv head `at`. Only
// CTAs below planned * splits <= num_sms share their unit.
struct PrefillPart {
  int at, split, splits;
};
PA_HOST_DEVICE inline PrefillPart prefill_part(int cta, int planned, int splits) {
  if (cta >= planned * splits) return {cta - planned * (splits - 1), 0, 1};
  return {cta / splits, cta % splits, splits};
}

}  // namespace quant
}  // namespace pa
