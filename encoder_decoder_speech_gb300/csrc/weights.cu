// Dispatch of the gathered attention weights, and what is decided by sizes.
#include <algorithm>

#include "paged_work.cuh"
#include "weights.cuh"

namespace cxa {
namespace {

constexpr int kFewRows16 = 16;              // query rows a K/V head of a few-rows product
constexpr double kSplitChunks = 8192;

// A tile of 128 rows holds whole tokens, so G query heads have to fit into it.
bool on_tiles(int G, bool bf16) { return bf16 && G <= 128; }
// (16 single tokens over up to 4000 keys of 8 heads of 64 in fp32: 194 us the way of many rows, 31 this.)
bool few_in_fp32(int G, int max_new, bool bf16) { return !bf16 && static_cast<long long>(G) * max_new <= kFewRows16; }

}  // namespace

// All have few rows, where no sequence can have more than a product's 16; otherwise those of one or two
// tokens (more would take room for scores that hardly any use), if their scores can be kept, there is more than
// one sequence, and the keys are many enough to pay for two more launches. (20 single tokens beside 4 chunks of a
// prompt, up to 8191 keys of 20 heads each: 534 us all with the many, 236 so; 5 tokens in each of 16 sequences of
// up to 1500 keys of 8 heads: 39 us and 45.) Whether the keys can be enough goes by the table's width and the pool:
// where they are not, in wide tables of a large pool, the launches cost 13 us (24 sequences, 300 tokens, up to 500 keys: 35 us and 48). Asked of
// the device, the kernels that then find nothing to do cost more: 52 us, and 248 in place of 241 where they have.
WeightsSplit weights_split(int B, int width, int page_shift, int num_pages, int Hkv, int G, int max_new) {
  WeightsSplit s;
  s.chunks = weights_chunks(B, width, page_shift, Hkv);
  s.many = static_cast<long long>(G) * max_new > kFewRows16;
  const int tokens = kFewRows16 / G < 2 ? kFewRows16 / G : 2;
  const double sound = std::min(s.chunks, weights_pool_chunks(B, num_pages, page_shift, Hkv));
  s.few_rows = !s.many ? G * max_new : B == 1 || sound < kSplitChunks ? 0 : tokens * G;
  const double each = static_cast<double>(score_chunk_bytes(s.few_rows)), all = s.chunks * each;
  const double most = static_cast<double>(kMaxScoreBytes);
  s.most = static_cast<size_t>(all <= most ? all : std::min(sound * each, most));
  return s;
}

ScoreRule score_rule(const WeightsSplit& s, const WeightsPlaces& at) {
  ScoreRule r = {};
  if (s.few_rows == 0) return r;
  // (no more than a workspace of the full size has: what a larger one gave would depend on other calls)
  const size_t room = std::min(at.score_bytes, s.most) / score_chunk_bytes(s.few_rows);
  r.room = static_cast<int>(std::min<size_t>(room, 0x7FFFFFFE));
  r.max_rows = s.few_rows;
  r.others = s.many;
  r.kept = s.chunks <= r.room;
  r.ask = !r.kept && r.room > 0;
  r.word = at.word;
  return r;
}

WeightsWorkspace weights_workspace(int B, int n_tokens, int width, int page_shift, int num_pages, int Hq, int Hkv,
                                   int max_new, bool bf16) {
  const int G = Hq / Hkv;
  const size_t fixed = weights_fixed_bytes(static_cast<long long>(n_tokens) * Hq);
  WeightsSplit s = {};
  if (on_tiles(G, bf16) || few_in_fp32(G, max_new, bf16)) s = weights_split(B, width, page_shift, num_pages, Hkv, G, max_new);
  const bool fit = s.chunks * static_cast<double>(score_chunk_bytes(s.few_rows)) <= static_cast<double>(kMaxScoreBytes);
  return {fixed + (fit ? s.most : 0), fixed + s.most};
}

bool weights_countable(const PagedBatch& bt, int page_shift, int Hkv, int G, bool bf16) {
  return on_tiles(G, bf16) ? work_bound(bt, page_shift, Hkv, G, 2 * (128 / G * G), 7) < kCountLimit
                           : work_bound(bt, page_shift, Hkv, G, 32, 6) < kCountLimit;
}

cudaError_t launch_weights(const WeightsLaunch& a, const DeviceInfo& dev, cudaStream_t stream, std::string* msg) {
  const int G = a.Hq / a.layer.Hkv;
  if (on_tiles(G, a.bf16)) return launch_weights_tile(a, dev, stream, msg);
  if (few_in_fp32(G, a.max_new, a.bf16)) return launch_weights_few_rows(a, dev, stream);
  return launch_weights_rows(a, nullptr, dev, stream);
}

}  // namespace cxa
