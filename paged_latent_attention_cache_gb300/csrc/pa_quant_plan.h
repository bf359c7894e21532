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

// Write: threads of a CTA (a run, the tokens of one sequence in one page, and a kv head),
// and rows that its shared memory holds at once; a run of more goes in pieces.
//
// Threads: warps by the kilobyte of rows, for what a run waits for is other runs' time, and
// the more rows there are the fewer runs an SM holds. 128 threads up to kFewBytes of rows, 256
// up to half of kRowBytes, then 512 with all of it. Measured with 128, 256, 512 threads (us; four
// prompts of 14740 tokens, 8 kv heads of 128 / 128): pages of 16 rows 42.6, 58.5, 114.8; 32: 37.8,
// 43.1, 66.8; 64: 47.7, 39.5, 49.0; 128: 70.3, 53.2, 43.3; one row for each of 32 sequences 4.4, 5.2, 7.1.
//
// Rows: a page, as long as all CTAs run at once so, or else the mean of the runs, 8 at least. Many CTAs of
// single tokens that each hold room for a page run in several waves, and the last one keeps
// room from the read behind it: its three CTAs an SM come to two and one. Both in us, room for
// pages of 64 rows and by the mean, heads as above: 512 single tokens 32.0, 21.3; write and read of
// 200 sequences with a new token each 255, 195, of 400 325, 230, of 200 and a chunk of 200 tokens 300, 244;
// of 64 and a prompt of 1000 147, 149. Where one wave is enough, 8 and a chunk of 300: 67, 71.
constexpr int kRowBytes = 96 * 1024, kFewBytes = 24 * 1024;
constexpr int kSharedOfSm = 228 * 1024, kSharedOfCta = 1024;  // (the latter beside its own)
struct WritePlan {
  int threads, cap;
  int64_t runs;  // numbers of runs, used or not (see quant_write_kernel)
};
// lanes: of a row, a power of two; row_bytes: of shared memory
inline WritePlan write_plan(int64_t num_tokens, int64_t num_seqs, int64_t kvh, int bs, int lanes,
                            int row_bytes, int num_sms) {
  WritePlan w;
  w.runs = 2 * num_seqs + num_tokens / bs;
  const int64_t mean = std::min<int64_t>(bs, (num_tokens + num_seqs - 1) / num_seqs);
  w.threads = mean * row_bytes <= kFewBytes ? 128 : mean * row_bytes <= kRowBytes / 2 ? 256 : 512;
  const int at_once = w.threads / lanes;
  const int room = (w.threads == 512 ? kRowBytes : kRowBytes / 2) / row_bytes / at_once * at_once;
  auto rows = [&](int64_t n) { return (int)std::min<int64_t>(room, (n + at_once - 1) / at_once * at_once); };
  w.cap = rows(bs);
  const int64_t at_a_time = kSharedOfSm / (w.cap * row_bytes + bs + kSharedOfCta) * (int64_t)num_sms;
  if (w.runs * kvh > at_a_time) w.cap = std::min(w.cap, rows(std::max<int64_t>(mean, 8)));
  return w;
}

// Which kernel takes a prefill range: the one for few rows takes sequences of at most `few`
// tokens, the one for many rows the others; either is left out where nothing is left for it.
//
// Batches with at most kFewRows query rows per sequence and kv head, on average, go to the kernel
// for few rows, which reads the keys once per 16 of them; the other takes as long whatever
// their number, up to two tiles of 128. Measured, rows there and here (us; 8 kv heads of 128
// with 4 query heads each): 16 sequences of 2000 to 16000 keys 16 rows 76, 270; 48: 167, 273;
// 64: 214, 274; 96: 309, 274; 32 sequences of 100 to 1000 keys 48: 64, 68; 64: 84, 70.
//
// In such a batch one sequence may still be long, and nothing tells the host. From kBothRows
// rows in all on, both kernels are launched, and sequences of more than kLongRows are the
// other one's. With one kernel and with both (us; heads as above): 300 sequences of one token over 100
// to 1000 keys and one of 8192 rows 852, 252; one of 8192 behind 8000 keys 1813, 517; 64 over 500
// to 4000 and one of 2048 behind 8000 404, 203; one of 512 behind none 93, 105. A launch that finds nothing
// costs 8 to 14: 128 drafts of 5 tokens 477, 490; below kBothRows it would be 32 of 12 tokens 98,
// 111. (The reverse, single tokens beside a prompt that lifts the mean, is left to the one kernel:
// 64 and a prompt of 2000 tokens 267, with both 189, but 32 sequences of 16 tokens 50, with both 83.)
constexpr int64_t kFewRows = 48, kLongRows = 1024, kBothRows = 2048;
constexpr int32_t kAnyTokens = INT32_MAX;
struct ReadChoice {
  int32_t few;
  bool rows, many;
};
inline ReadChoice choose_kernels(int64_t tokens, int64_t nseq, int64_t group) {
  if (tokens * group > kFewRows * nseq) return {0, false, true};
  if (tokens * group <= kBothRows) return {kAnyTokens, true, false};
  return {(int32_t)(kLongRows / group), true, true};
}

// The grid of the prefill kernel, a CTA per unit (`per` consecutive tokens of a sequence of more
// than `few`) and kv head. Where the planned ones are few, each is split: `splits` CTAs share its
// keys.
struct PrefillGrid {
  int64_t ctas;     // units and kv heads, at most (whatever the offsets)
  int64_t planned;  // of them those that are split
  int splits = 1;
  int64_t launched() const { return ctas + planned * (splits - 1); }
};
inline PrefillGrid prefill_grid(int64_t num_tokens, int64_t tokens, int64_t nseq, int64_t few,
                                int64_t kvh, int64_t per, int64_t tiles, int num_sms) {
  // (a sequence with so many tokens has at most one unit that is not full)
  auto units = [&](int64_t t) { return (t / per + std::min(nseq, t / (few + 1))) * kvh; };
  PrefillGrid g;
  g.ctas = units(num_tokens);
  // (beside sequences for the other kernel: one, with the tokens that they leave)
  g.planned = few > 0 ? (std::max<int64_t>(0, tokens - nseq) / per + 1) * kvh : units(tokens);
  g.planned = std::min(g.ctas, g.planned);
  if (g.planned == 0) return g;  // (no such sequence at all)
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
