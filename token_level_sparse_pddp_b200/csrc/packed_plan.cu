// Packed attention calls: the planner (host) and the entry points.
//
// The planner turns the lengths of a batch into a table of work items, so the
// kernels' grids, the split of long key ranges over CTAs and the merge of
// their partial results are all settled on the host, once per batch.
//   tile items   up to a tile's rows of one sequence against its keys (and the
//                prefix), or the rows of many short sequences against the
//                prefix, which is then read once for all of them;
//   token items  up to 16 rows (the tokens of one sequence, or of several with the
//                prefix) against their keys: memory-bound, split until the GPU is full;
//   merge items  tokens whose keys were split.
#include <algorithm>
#include <cmath>
#include <cstring>
#include <queue>
#include <vector>

#include "overlap.h"
#include "packed.h"

namespace tlsp {
namespace {

constexpr size_t kAlign = 256;
constexpr size_t kStatusBytes = 256;
constexpr int64_t kMaxItems = int64_t(1) << 22;  // tile items of a plan
constexpr int64_t kMaxRows = 0x7ffffeff;  // kernels index tokens with 32 bits (element offsets with 64)
constexpr int kSms = 148;  // planning assumes a B200
constexpr int kTokenSlots = 2 * kSms;  // CTAs of token items resident at once
constexpr int kGpcs = 8;               // a cluster's CTAs lie in one of them
constexpr int kTokenKeys = 107;        // that such a CTA takes in 1.7 us, of either head_dim
constexpr int kTokenBlock = 16;        // keys a warp of a token item takes at a time

int validate_desc(const tlsp_packed_desc* d) {
  if (!d) return TLSP_ERR_INVALID_ARG;
  if (d->num_seqs < 1 || d->heads < 1 || d->kv_heads < 1 || d->heads % d->kv_heads)
    return TLSP_ERR_INVALID_ARG;
  if (d->head_dim != 64 && d->head_dim != 128) return TLSP_ERR_INVALID_ARG;
  if (d->dtype != TLSP_F32 && d->dtype != TLSP_BF16) return TLSP_ERR_INVALID_ARG;
  if ((d->causal != 0 && d->causal != 1) || d->prefix_len < 0) return TLSP_ERR_INVALID_ARG;
  if (d->heads / d->kv_heads > 64 || d->kv_heads > 65535) return TLSP_ERR_UNSUPPORTED;
  return TLSP_OK;
}

size_t align_up(size_t x) { return (x + kAlign - 1) / kAlign * kAlign; }

struct WsLayout {
  size_t lse, o, total;
};
WsLayout ws_layout(const tlsp_packed_plan& p) {
  WsLayout L{};
  L.lse = kStatusBytes;
  L.o = align_up(L.lse + sizeof(float) * (size_t)p.part_rows * p.desc.heads);
  L.total = align_up(L.o + sizeof(float) * (size_t)p.part_rows * p.desc.heads * p.desc.head_dim);
  return L;
}

// An item's steps, and what one of them costs.
struct Load {
  int64_t steps;
  double cost;
  // parts of at most `most` cost, each of one step at least
  int64_t parts(double most) const {
    return std::max<int64_t>(1, std::min<int64_t>(steps, (int64_t)std::ceil((double)steps * cost / most)));
  }
};

// Time of tile items on `slots` CTAs taking them longest first, when item i is cut into
// parts[i] and `fixed` is spent on starting and finishing each part.
double makespan(const std::vector<Load>& loads, const std::vector<int64_t>& parts, int kv_heads,
                double fixed, int slots) {
  std::vector<double> jobs;
  for (size_t x = 0; x < loads.size(); ++x) {
    const Load& l = loads[x];
    for (int64_t i = 0; i < parts[x]; ++i)
      for (int h = 0; h < kv_heads; ++h)
        jobs.push_back((double)(l.steps * (i + 1) / parts[x] - l.steps * i / parts[x]) * l.cost +
                       fixed * (parts[x] > 1 ? 1.5 : 1));
  }
  std::sort(jobs.begin(), jobs.end(), std::greater<double>());
  std::priority_queue<double, std::vector<double>, std::greater<double>> ends;
  double last = 0;
  for (double j : jobs) {
    double at = 0;
    if ((int)ends.size() == slots) {
      at = ends.top();
      ends.pop();
    }
    ends.push(at + j);
    last = std::max(last, at + j);
  }
  return last;
}

class Planner {
 public:
  Planner(const tlsp_packed_desc& d, const int32_t* q_lens, const int32_t* kv_lens,
          const int64_t* kv_starts)
      : d_(d), q_lens_(q_lens), kv_lens_(kv_lens), kv_starts_(kv_starts) {
    group_ = d.heads / d.kv_heads;
    chunk_ = d.dtype == TLSP_BF16 ? 128 : 64;
    tile_tokens_ = tile_tokens(d.dtype == TLSP_BF16, group_);
  }

  int run() {
    TLSP_TRY(place());
    // Tile items first; those left whole, then those split.
    std::vector<PackedItem> whole;
    std::vector<int> own;  // sequences whose prefix part is shared: their items of own keys
    for (int s = 0; s < d_.num_seqs; ++s)
      if (!share_[s])
        for (int t0 = 0; t0 < q_lens_[s]; t0 += tile_tokens_) whole.push_back(own_tile(s, t0));
    const size_t owns = whole.size();  // those items stand from here
    for (int s = 0; s < d_.num_seqs; ++s)
      if (share_[s] && !few_[s]) {
        own.push_back(s);
        whole.push_back(own_tile(s, 0));
        whole.back().pre_n = 0;
      }
    std::vector<PackedItem> shared;  // rows of short sequences against the prefix
    if (d_.prefix_len > 0) {
      for (int s = 0; s < d_.num_seqs;) {
        if (!share_[s]) {
          ++s;
          continue;
        }
        int e = s;  // a run of such sequences: their queries are consecutive
        while (e < d_.num_seqs && share_[e]) ++e;
        const int64_t q0 = q0_[s], n = q0_[e - 1] + q_lens_[e - 1] - q0;
        if (as_token_items(s, e)) {
          for (int x = s; x < e;) {
            const int y = end_of_group(x, e);
            const int64_t nt = q0_[y - 1] + q_lens_[y - 1] - q0_[x];
            if (nt > 0) shared.push_back({(int32_t)q0_[x], (int32_t)nt, 0, 0, 0, d_.prefix_len, 0, 0});
            x = y;
          }
          s = e;
          continue;
        }
        for (int64_t i = 0; i < n; i += tile_tokens_)
          shared.push_back({(int32_t)(q0 + i), (int32_t)std::min<int64_t>(tile_tokens_, n - i), 0, 0, 0,
                            d_.prefix_len, 0, 0});
        s = e;
      }
    }
    // prefix work of at most kTokenRows rows goes to the token kernel
    const auto few_rows = std::stable_partition(
        shared.begin(), shared.end(),
        [&](const PackedItem& t) { return (int64_t)t.nt * group_ > kTokenRows; });
    const std::vector<PackedItem> shared_tokens(few_rows, shared.end());
    shared.erase(few_rows, shared.end());
    const std::vector<int64_t> cut = tile_split(whole, shared, shared_tokens);
    std::vector<Piece> own_parts;
    for (size_t x = 0; x < whole.size(); ++x) {
      const PackedItem& t = whole[x];
      const int64_t parts = x >= owns && t.kv_n == 0 ? 0 : cut[x];
      if (x < owns && parts == 1) {
        tiles.push_back(t);
        continue;
      }
      const int64_t base = take_slots(parts * t.nt);
      if (parts > 0) split(t, parts, base, tiles);
      if (x < owns)
        add_merge(t.q0, t.nt, base, parts, t.nt, 0, 0, 0);
      else
        own_parts.push_back({t.q0, t.nt, base, parts});
    }
    std::vector<Piece> pieces;  // where the prefix results of each token lie
    for (size_t x = 0; x < shared.size(); ++x) {
      const PackedItem& t = shared[x];
      const int64_t parts = cut[whole.size() + x], base = take_slots(parts * t.nt);
      split(t, parts, base, tiles);
      pieces.push_back({t.q0, t.nt, base, parts});
    }
    if (d_.dtype == TLSP_BF16)
      plan_tokens(shared_tokens, pieces);
    else
      plan_tokens_simt(shared_tokens, pieces);
    size_t at = 0;  // (the pieces ascend)
    for (size_t x = 0; x < own.size(); ++x)
      merge_sequence(own[x], own_parts[x].slot, own_parts[x].parts, pieces, at);
    if (part_rows_ > 0x7fffffffLL) return TLSP_ERR_UNSUPPORTED;
    // longest first: the grid is handed out in this order
    auto longer = [&](const PackedItem& a, const PackedItem& b) {
      return steps_of(a) > steps_of(b);
    };
    std::stable_sort(tiles.begin(), tiles.end(), longer);
    std::stable_sort(tokens.begin(), tokens.end(), longer);
    std::stable_sort(token_items.begin(), token_items.end(), [&](const TokenItem& a, const TokenItem& b) {
      return keys_of(a) > keys_of(b);
    });
    const int64_t most_items =
        std::max({tiles.size(), tokens.size(), token_items.size() * (size_t)cluster, merges.size()}) *
        (uint64_t)d_.kv_heads;
    if (most_items > 0x7fffffffLL) return TLSP_ERR_UNSUPPORTED;
    for (const MergeItem& t : merges) merge_parts = std::max(merge_parts, t.a_parts + t.b_parts);
    if (!merges.empty() && merge_blocks(d_.heads, merge_parts) > kMaxGridY) return TLSP_ERR_UNSUPPORTED;
    return TLSP_OK;
  }

  std::vector<PackedItem> tiles, tokens;
  std::vector<TokenItem> token_items;
  std::vector<TokenSegment> segments;
  std::vector<MergeItem> merges;
  int cluster = 1;
  int merge_parts = 0;  // most parts of a merge item
  int64_t q_rows = 0, kv_rows = 0;
  int64_t part_rows() const { return part_rows_; }

 private:
  struct Piece {
    int64_t q0, nt, slot, parts;
  };

  int place() {
    q0_.resize(d_.num_seqs);
    kv0_.resize(d_.num_seqs);
    few_.resize(d_.num_seqs);
    int64_t end = 0;
    if (d_.prefix_len > kMaxRows) return TLSP_ERR_UNSUPPORTED;
    for (int s = 0; s < d_.num_seqs; ++s) {
      const int32_t n = q_lens_[s], m = kv_lens_[s];
      if (n < 0 || m < 0) return TLSP_ERR_INVALID_ARG;
      q0_[s] = q_rows;
      kv0_[s] = kv_starts_ ? kv_starts_[s] : end;
      if (kv0_[s] < 0) return TLSP_ERR_INVALID_ARG;
      if (m > 0 && kv0_[s] > kMaxRows - m) return TLSP_ERR_UNSUPPORTED;
      end += m;
      q_rows += n;
      if (m > 0) kv_rows = std::max(kv_rows, kv0_[s] + m);
      if (m == 0) kv0_[s] = 0;
      few_[s] = (int64_t)n * group_ <= kTokenRows;
    }
    // A few short sequences among longer ones go with their tile items: they end sooner
    // than those, and save a launch (24 prompts, two of them of 2 and 4 tokens: 244 -> 240
    // us). Of 210 batches of 1 to 70 short sequences among 1, 4 or 16 prompts of 100 to 4000
    // tokens, those with up to kSms / 2 such items are 2 to 3% faster this way beside 4 or
    // more prompts and 1 to 4% slower beside one, within 2.5% up to kSms, and above 2 kSms 7
    // to 23% slower.
    if (d_.dtype == TLSP_BF16 && d_.prefix_len == 0) {
      int64_t longest = 0, most = 0, count = 0;  // keys of a tile item, of a few-query sequence
      for (int s = 0; s < d_.num_seqs; ++s) {
        if (!few_[s]) longest = std::max<int64_t>(longest, kv_lens_[s]);
        if (few_[s] && q_lens_[s] > 0) {
          most = std::max<int64_t>(most, kv_lens_[s]);
          ++count;
        }
      }
      if (most <= longest && longest > 0 && count * d_.kv_heads <= kSms / 2)
        std::fill(few_.begin(), few_.end(), 0);
    }
    choose_shared();
    if (q_rows > kMaxRows) return TLSP_ERR_UNSUPPORTED;
    int64_t items = 0;
    for (int s = 0; s < d_.num_seqs; ++s)
      if (!few_[s]) items += ceil_div(q_lens_[s], tile_tokens_);
    return items > kMaxItems ? TLSP_ERR_UNSUPPORTED : TLSP_OK;
  }

  // Short sequences share the work on the prefix: their rows take it together, and their
  // own keys are items of their own, merged with it. Those of a token item always do; longer
  // ones, of up to a tile item, where that is clearly less work (in steps of a tile item): 48
  // sequences of 1 to 3 tokens behind 15329 keys, 16 / 2 heads: 31 us, with the prefix alone
  // for each of 3 tokens (24 rows) 62 us. Of 150 batches of 2 to 48 sequences of up to 60
  // tokens behind 500 to 30000 keys, 93 are different without this rule, 30% slower on
  // average; with any gain taken instead of a tenth, 7 are, 2% slower.
  void choose_shared() {
    share_ = few_;
    if (d_.dtype != TLSP_BF16 || d_.prefix_len == 0) return;
    const double pre = (double)ceil_div(d_.prefix_len, chunk_);
    const int64_t half = tile_tokens_ / 2;
    auto own_steps = [&](int s) { return (double)ceil_div(own_tile(s, 0).kv_n, chunk_); };
    // sequences of up to `most` tokens share, if one beside them does: work of all that might
    auto work = [&](int64_t most, std::vector<char>& share) {
      double sum = 0;
      for (int s = 0; s < d_.num_seqs;) {
        int e = s, n = 0;
        int64_t tokens = 0;
        for (; e < d_.num_seqs && (few_[e] || q_lens_[e] <= most); ++e) {
          n += q_lens_[e] > 0;
          tokens += q_lens_[e];
        }
        const int end = std::max(e, s + 1);
        if (e > s && (n > 1 || few_[s])) {
          const int64_t rest = tokens % tile_tokens_;
          sum += pre * ((double)(tokens / tile_tokens_) +
                        (rest == 0 ? 0 : rest * group_ <= kTokenRows ? 0.5 : rest <= half ? 0.75 : 1.0));
        }
        for (; s < end; ++s) {
          share[(size_t)s] = few_[s] || (e > s && n > 1);
          if (few_[s] || q_lens_[s] > tile_tokens_) continue;  // the same either way
          const double steps = own_steps(s) + (share[(size_t)s] ? 0.0 : pre);
          sum += 3 + steps * (q_lens_[s] <= half ? 0.6 : 1.0);
        }
      }
      return sum;
    };
    double least = work(0, share_);
    for (int64_t most : {half / 2, half, (int64_t)tile_tokens_}) {
      std::vector<char> share = few_;
      const double w = work(most, share);
      if (w < 0.9 * least) {
        least = w;
        share_ = std::move(share);
      }
    }
  }

  // The sequences from x on, before e, whose rows fit into a token item together.
  int end_of_group(int x, int e) const {
    int64_t tokens = 0;
    int y = x;
    for (; y < e && (tokens + q_lens_[y]) * group_ <= kTokenRows; ++y) tokens += q_lens_[y];
    return y;
  }
  // Whether a run of few-query sequences takes the prefix in token items of up to 16 rows,
  // with their own keys and nothing to merge, not in tile items: the prefix is read for
  // every 16 rows then, but tile items and merge take some 4 steps besides their work (21
  // sequences of one token behind 334 keys, 3 / 1 heads: 10 us instead of 13.5). Of 144
  // batches of 2 to 64 single tokens behind 100 to 8000 keys, 62 are different without this
  // rule, 22% slower on average; with 8 steps for 4, 18 are, 10% slower. A key costs a token
  // item as much with 64 channels as with 128: counted at half, 99 of 720 plans change, and
  // take 13% longer.
  bool as_token_items(int s, int e) const {
    if (d_.dtype != TLSP_BF16) return false;
    int64_t keys = 0, longest = 0, tokens = 0, jobs = 0;
    for (int x = s; x < e;) {
      if (!few_[x]) return false;
      const int y = end_of_group(x, e);
      int64_t all = 0;
      for (int i = x; i < y; ++i)
        if (q_lens_[i] > 0) {
          all += kv_lens_[i];
          tokens += q_lens_[i];
        }
      if (q0_[y - 1] + q_lens_[y - 1] > q0_[x]) all += d_.prefix_len;
      keys += all;
      longest = std::max(longest, all);
      jobs += all > 0 ? d_.kv_heads : 0;
      x = y;
    }
    int ctas = 1;  // of an item
    while (ctas < kMaxCluster && jobs * 2 * ctas <= kTokenSlots) ctas *= 2;
    const double each = std::max((double)keys * d_.kv_heads / kTokenSlots, (double)longest / ctas);
    const double tile_work = (double)ceil_div(d_.prefix_len, chunk_) *
                             (double)ceil_div(tokens, tile_tokens_) * d_.kv_heads / kSms;
    return each / kTokenKeys <= 4 + tile_work;
  }

  // Chunks of keys a tile item steps through.
  int64_t steps_of(const PackedItem& t) const { return ceil_div(t.pre_n, chunk_) + ceil_div(t.kv_n, chunk_); }

  static int32_t clamp_diag(int64_t diag, int64_t kv_n) {
    return (int32_t)std::max<int64_t>(-0x40000000LL, std::min<int64_t>(diag, kv_n));
  }

  // Tile of the sequence's tokens from t0, with the keys that any of them sees.
  PackedItem own_tile(int s, int t0) const {
    const int64_t n = q_lens_[s], m = kv_lens_[s];
    const int64_t nt = std::min<int64_t>(tile_tokens_, n - t0);
    const int64_t diag = d_.causal ? m - n + t0 : m;
    const int64_t keys = std::max<int64_t>(0, std::min<int64_t>(m, diag + nt));
    return {(int32_t)(q0_[s] + t0), (int32_t)nt, (int32_t)kv0_[s], (int32_t)keys,
            0, d_.prefix_len, clamp_diag(diag, m), -1};
  }

  // Cuts an item's keys (prefix, then own) at whole chunks into `parts`.
  void split(const PackedItem& t, int64_t parts, int64_t base, std::vector<PackedItem>& to) {
    const int64_t pre_steps = ceil_div(t.pre_n, chunk_), steps = steps_of(t);
    for (int64_t p = 0; p < parts; ++p) {
      const int64_t a = steps * p / parts, b = steps * (p + 1) / parts;
      PackedItem x = t;
      const int64_t pa = std::min(a, pre_steps) * chunk_, pb = std::min(b, pre_steps) * chunk_;
      x.pre0 = (int32_t)(t.pre0 + std::min<int64_t>(pa, t.pre_n));
      x.pre_n = (int32_t)(std::min<int64_t>(pb, t.pre_n) - std::min<int64_t>(pa, t.pre_n));
      const int64_t oa = std::max<int64_t>(0, a - pre_steps) * chunk_;
      const int64_t ob = std::max<int64_t>(0, b - pre_steps) * chunk_;
      x.kv0 = (int32_t)(t.kv0 + std::min<int64_t>(oa, t.kv_n));
      x.kv_n = (int32_t)(std::min<int64_t>(ob, t.kv_n) - std::min<int64_t>(oa, t.kv_n));
      x.diag = clamp_diag((int64_t)t.diag - oa, x.kv_n);
      x.slot = (int32_t)(base + p * t.nt);
      to.push_back(x);
    }
  }

  int64_t take_slots(int64_t n) {
    const int64_t at = part_rows_;
    part_rows_ += n;
    return at;
  }

  void add_merge(int64_t q0, int64_t n, int64_t a, int64_t a_parts, int64_t a_stride, int64_t b,
                 int64_t b_parts, int64_t b_stride) {
    for (int64_t i = 0; i < n; i += kMergeTokens)
      merges.push_back({(int32_t)(q0 + i), (int32_t)std::min<int64_t>(kMergeTokens, n - i),
                        (int32_t)(a + i), (int32_t)a_parts, (int32_t)a_stride, (int32_t)(b + i),
                        (int32_t)b_parts, (int32_t)b_stride});
  }

  // A step of an item with one query tile takes 0.6 of one with two (measured with
  // d = 128: 1.0 us and 1.7 us), and 0.75 where few-query sequences share the prefix,
  // whose keys come from memory for a few items only (1.8 and 2.5 us on all SMs).
  Load load_of(const PackedItem& t, bool shared) const {
    const bool one_tile = d_.dtype == TLSP_BF16 && 2 * t.nt <= tile_tokens_;
    return {steps_of(t), !one_tile ? 1.0 : shared ? 0.75 : 0.6};
  }

  // fp32 tile items that share an SM: as many as its registers and shared memory take (with
  // 3 for 4 and for 2 here, six ragged sequences with d = 64 took 72 us instead of 65.5, and
  // with d = 128 85 us instead of 73).
  int simt_ctas() const { return (d_.head_dim == 64 ? 4 : 2) / (group_ > 32 ? 2 : 1); }
  double keys_of_step() const { return 110e3 / (4 * d_.head_dim); }

  // Work of the token items in steps of a tile item, with which they share the SMs:
  // an SM reads about 110 KB of keys and values in the 1.7 us of a step.
  double token_steps(const std::vector<PackedItem>& shared_tokens) const {
    if (d_.dtype != TLSP_BF16) return 0;
    double keys = 0;
    for (const PackedItem& t : shared_tokens) keys += t.pre_n;
    for (int s = 0; s < d_.num_seqs; ++s)
      if (few_[s] && q_lens_[s] > 0) keys += kv_lens_[s];
    return keys * d_.kv_heads / keys_of_step();
  }

  // Parts of each tile item. With many more items than SMs they stay whole; else the
  // split of least estimated time is taken: all items cut to a size that fills the SMs
  // evenly a few times over, long items cut to a share of the mean, or only the shortest
  // ones, those of the last, incomplete round. Starting and finishing an item takes about
  // three steps of 1.7 us (fp32: one). Token items run
  // on the SMs that tile items leave, so what counts is the sum of both, and fewer and
  // longer tile items that leave SMs free from the start are tried too: what bounds
  // these is the matrix rate, what bounds token items the memory (64 sequences of 16 to
  // 2000 keys behind a prefix of 32760, 40 heads of 128 in 8 groups, on a cool GPU: one
  // kernel after the other 106 us, beside each other 98 us with tile items on 144 SMs, 88 us
  // on 104; back to back, at the power limit, 103 us). Cutting the last round's items alone
  // makes 24 of 80 batches of 1 to 16 prompts 6% faster.
  std::vector<int64_t> tile_split(const std::vector<PackedItem>& whole,
                                  const std::vector<PackedItem>& shared,
                                  const std::vector<PackedItem>& shared_tokens) {
    std::vector<Load> loads;
    double longest = 1, total = 0;
    for (const auto* v : {&whole, &shared})
      for (const PackedItem& t : *v) {
        loads.push_back(load_of(t, v == &shared));
        const double all = (double)loads.back().steps * loads.back().cost;
        total += all;
        longest = std::max(longest, all);
      }
    std::vector<int64_t> best(loads.size(), 1);
    if (loads.empty()) return best;
    const int64_t jobs = (int64_t)loads.size() * d_.kv_heads;
    const int slots = d_.dtype == TLSP_BF16 ? kSms : simt_ctas() * kSms;
    const double mean = total * d_.kv_heads / slots;
    tile_time_ = mean;
    if (jobs > 16 * slots && (longest < mean / 2 || jobs > 100000)) return best;
    const double fixed = d_.dtype == TLSP_BF16 ? 3.0 : 1.0;
    // No part is shorter, which bounds the merging (bf16, few tokens before long caches on
    // an empty GPU: 13 to 17 us, with 4 instead 17 to 21, with 1 no better).
    const double shortest = d_.dtype == TLSP_BF16 ? 2.0 : 1.0;
    const double beside = token_steps(shared_tokens);
    // The least time that a split can take: its longest part's, or all SMs busy to the end.
    auto bound_of = [&](const std::vector<int64_t>& parts) {
      double sum = total * d_.kv_heads + beside, most = 0;
      for (size_t x = 0; x < loads.size(); ++x) {
        const double each = fixed * (parts[x] > 1 ? 1.5 : 1);
        sum += each * (double)parts[x] * d_.kv_heads;
        most = std::max(most, (double)ceil_div(loads[x].steps, parts[x]) * loads[x].cost + each);
      }
      return std::max(most, sum / slots);
    };
    auto time_of = [&](const std::vector<int64_t>& parts, double bound) {
      const double t = makespan(loads, parts, d_.kv_heads, fixed, slots);
      return beside > 0 ? std::max(t, bound) : t;
    };
    double least = time_of(best, bound_of(best));
    auto try_parts = [&](std::vector<int64_t> parts) {
      const double bound = bound_of(parts);
      if (bound >= 0.98 * least) return;
      const double t = time_of(parts, bound);
      if (t < 0.98 * least) {
        least = t;
        best = std::move(parts);
      }
    };
    auto try_split = [&](double most) {
      if (most >= longest) return;
      std::vector<int64_t> parts;
      for (const Load& l : loads) parts.push_back(l.parts(most));
      try_parts(std::move(parts));
    };
    auto try_items = [&](int64_t places) {  // as long as `places` items can be
      if (jobs > places) return;
      double lo = shortest, hi = longest;
      for (int i = 0; i < 12; ++i) {
        const double mid = 0.5 * (lo + hi);
        int64_t n = 0;
        for (const Load& l : loads) n += l.parts(mid);
        (n * d_.kv_heads <= places ? hi : lo) = mid;
      }
      try_split(hi);
    };
    if (beside > 0)
      for (int places = slots / 4; places < slots; places += 8) try_items(places);
    for (int rounds = 1; rounds <= 4; ++rounds) try_items((int64_t)rounds * slots);
    if (2 * jobs > slots)
      for (int k = 1; k <= 4; ++k) try_split(std::max(shortest, mean / k));
    if (jobs > slots && least > 1.03 * (mean + fixed * (double)jobs / slots)) {
      std::vector<size_t> order(loads.size());
      for (size_t i = 0; i < order.size(); ++i) order[i] = i;
      std::stable_sort(order.begin(), order.end(), [&](size_t a, size_t b) {
        return (double)loads[a].steps * loads[a].cost > (double)loads[b].steps * loads[b].cost;
      });
      for (int64_t rounds = jobs / slots; rounds >= std::max<int64_t>(1, jobs / slots - 1); --rounds)
        for (int64_t p : {2, 3, 4, 6}) {
          std::vector<int64_t> parts(loads.size(), 1);
          for (size_t i = (size_t)(rounds * slots / d_.kv_heads); i < order.size(); ++i) {
            const Load& l = loads[order[i]];
            parts[order[i]] = std::max<int64_t>(1, std::min(p, l.steps / 8));
          }
          try_parts(std::move(parts));
        }
    }
    tile_time_ = least;
    return best;
  }

  // Keys of a token item of the fp32 kernel: small enough to give every SM its CTAs in
  // one go where the keys are few, about three rounds of them where they are many.
  int64_t simt_range(const std::vector<PackedItem>& shared_tokens) const {
    std::vector<int64_t> lens;
    for (int s = 0; s < d_.num_seqs; ++s)
      if (few_[s] && q_lens_[s] > 0 && kv_lens_[s] > 0) lens.push_back(kv_lens_[s]);
    for (const PackedItem& t : shared_tokens) lens.push_back(t.pre_n);
    int64_t range = chunk_;
    while (range < 2048 && parts_of(lens, range) * d_.kv_heads > kTokenSlots) range += chunk_;
    return range;
  }

  static int64_t parts_of(const std::vector<int64_t>& lens, int64_t range) {
    int64_t n = 0;
    for (int64_t l : lens) n += std::max<int64_t>(1, ceil_div(l, range));
    return n;
  }

  // Merge entries of a few-query sequence: its prefix results lie in `pieces`, its own
  // in `parts` partial rows from `base`.
  void merge_sequence(int s, int64_t base, int64_t parts, const std::vector<Piece>& pieces,
                      size_t& at) {
    const int32_t n = q_lens_[s];
    if (d_.prefix_len == 0) {
      add_merge(q0_[s], n, base, parts, n, 0, 0, 0);
      return;
    }
    int64_t q = q0_[s];
    while (q < q0_[s] + n) {  // the pieces that hold its prefix results
      while (pieces[at].q0 + pieces[at].nt <= q) ++at;
      const Piece& p = pieces[at];
      const int64_t to = std::min<int64_t>(q0_[s] + n, p.q0 + p.nt);
      add_merge(q, to - q, p.slot + (q - p.q0), p.parts, p.nt, base + (q - q0_[s]), parts, n);
      q = to;
    }
  }

  void plan_tokens_simt(const std::vector<PackedItem>& shared_tokens, std::vector<Piece>& pieces) {
    const int64_t range = simt_range(shared_tokens);
    for (const PackedItem& t : shared_tokens) {
      const int64_t parts = std::max<int64_t>(1, ceil_div(t.pre_n, range));
      const int64_t base = take_slots(parts * t.nt);
      split(t, parts, base, tokens);
      pieces.push_back({t.q0, t.nt, base, parts});
    }
    std::sort(pieces.begin(), pieces.end(),
              [](const Piece& a, const Piece& b) { return a.q0 < b.q0; });
    size_t at = 0;
    for (int s = 0; s < d_.num_seqs; ++s) {
      if (!few_[s] || q_lens_[s] == 0) continue;
      const int32_t n = q_lens_[s], m = kv_lens_[s];
      const int64_t parts = d_.prefix_len > 0 && m == 0 ? 0 : std::max<int64_t>(1, ceil_div(m, range));
      const PackedItem t = {(int32_t)q0_[s], n, (int32_t)kv0_[s], m, 0, 0, own_diag(s), -1};
      if (parts == 1 && d_.prefix_len == 0) {
        tokens.push_back(t);
        continue;
      }
      const int64_t base = take_slots(parts * n);
      if (parts > 0) split(t, parts, base, tokens);
      merge_sequence(s, base, parts, pieces, at);
    }
  }

  int32_t own_diag(int s) const {
    return clamp_diag(d_.causal ? (int64_t)kv_lens_[s] - q_lens_[s] : kv_lens_[s], kv_lens_[s]);
  }

  // bf16: an item's keys are shared by the CTAs of a cluster, which join their results
  // through each other's shared memory: a batch of a few sequences takes one launch.
  // Only what a cluster cannot hold (long caches of very few sequences) is cut into
  // several items and merged, and what shares the prefix by tile items.
  void plan_tokens(const std::vector<PackedItem>& shared_tokens, std::vector<Piece>& pieces) {
    struct Draft {
      TokenItem item;
      std::vector<TokenSegment> segs;
      int64_t keys = 0;
      bool piece = false;  // prefix results alone, of tokens whose own keys come elsewhere
      int seq = -1;        // own keys alone of this sequence
      int64_t parts = 0, base = -1;
    };
    std::vector<Draft> drafts;
    auto add = [](Draft& d, const TokenSegment& s) {
      if (s.n == 0) return;
      d.segs.push_back(s);
      d.keys += s.n;
    };
    std::vector<char> taken((size_t)d_.num_seqs, 0);
    for (const PackedItem& t : shared_tokens) {
      Draft d;
      d.item = {t.q0, t.nt, 0, 0, -1, {}};
      add(d, {t.pre0, t.pre_n, 0, t.nt, t.pre_n, 1, {}});
      // with all its tokens' own keys, if no sequence has tokens elsewhere too
      const int first = sequence_of(t.q0), last = sequence_of((int64_t)t.q0 + t.nt - 1);
      d.piece = q0_[first] < t.q0 || q0_[last] + q_lens_[last] > t.q0 + t.nt;
      for (int s = first; s <= last && !d.piece; ++s) {
        if (q_lens_[s] == 0) continue;
        taken[(size_t)s] = 1;
        add(d, {(int32_t)kv0_[s], kv_lens_[s], (int32_t)(q0_[s] - t.q0), q_lens_[s], own_diag(s), 0, {}});
      }
      drafts.push_back(std::move(d));
    }
    for (int s = 0; s < d_.num_seqs; ++s) {
      if (!few_[s] || q_lens_[s] == 0 || taken[(size_t)s]) continue;
      Draft d;
      d.item = {(int32_t)q0_[s], q_lens_[s], 0, 0, -1, {}};
      add(d, {(int32_t)kv0_[s], kv_lens_[s], 0, q_lens_[s], own_diag(s), 0, {}});
      if (d_.prefix_len > 0) d.seq = s;
      drafts.push_back(std::move(d));
    }
    if (drafts.empty()) return;
    // CTAs of an item: as many as fill the GPU in one go, with 64 keys each at least
    std::vector<int64_t> lens;
    int64_t longest = 0, total = 0;
    for (const Draft& d : drafts) {
      lens.push_back(d.keys);
      longest = std::max(longest, d.keys);
      total += d.keys;
    }
    const int64_t jobs = (int64_t)drafts.size() * d_.kv_heads;
    // Places beside the tile items, if they are enough and done with their share before
    // those are (else most start behind those: all).
    // A wider cluster than they take would wait for the end of tile items: 8 sequences of
    // 1 to 30 tokens 20 us instead of 16.
    int64_t places = kTokenSlots - 2 * (int64_t)tiles.size() * d_.kv_heads;
    if (places < std::max<int64_t>(jobs, kGpcs) ||
        (double)total * d_.kv_heads / (double)places > tile_time_ * keys_of_step() / 2)
      places = kTokenSlots;
    const int64_t widest = std::min<int64_t>(kMaxCluster, places / kGpcs);  // that fits into what is free
    while (2 * cluster <= widest && jobs * 2 * cluster <= places && longest > 64 * cluster)
      cluster *= 2;
    // Items of more keys than a cluster's share are cut: where the GPU would stay empty,
    // to fill it; else at twice the mean keys of a place for a CTA, 512 at least.
    const int64_t mean = ceil_div(total * d_.kv_heads, places);
    int64_t range = std::max<int64_t>(512, 2 * mean) * cluster;
    if (jobs * cluster * 2 <= places) {
      range = 256 * cluster;
      while (parts_of(lens, range) * d_.kv_heads * cluster > places) range += 32 * cluster;
    }
    for (Draft& d : drafts) {
      d.parts = d.seq >= 0 && d.keys == 0 ? 0 : std::max<int64_t>(1, ceil_div(d.keys, range));
      const bool merged = d.parts > 1 || d.seq >= 0 || d.piece;
      if (merged) d.base = take_slots(d.parts * d.item.nt);
      for (int64_t p = 0; p < d.parts; ++p) {  // keys [a, b) of the concatenated segments
        const int64_t a = d.keys * p / d.parts / kTokenBlock * kTokenBlock;
        const int64_t b =
            p + 1 == d.parts ? d.keys : d.keys * (p + 1) / d.parts / kTokenBlock * kTokenBlock;
        TokenItem t = d.item;
        t.seg0 = (int32_t)segments.size();
        t.slot = merged ? (int32_t)(d.base + p * t.nt) : -1;
        int64_t from = 0;
        for (const TokenSegment& s : d.segs) {
          const int64_t lo = std::max<int64_t>(a - from, 0), hi = std::min<int64_t>(b - from, s.n);
          from += s.n;
          if (lo >= hi) continue;
          TokenSegment x = s;
          x.k0 = (int32_t)(s.k0 + lo);
          x.n = (int32_t)(hi - lo);
          x.diag = clamp_diag((int64_t)s.diag - lo, x.n);
          segments.push_back(x);
        }
        t.nseg = (int32_t)segments.size() - t.seg0;
        token_items.push_back(t);
      }
      if (d.piece)
        pieces.push_back({d.item.q0, d.item.nt, d.base, d.parts});
      else if (merged && d.seq < 0)
        add_merge(d.item.q0, d.item.nt, d.base, d.parts, d.item.nt, 0, 0, 0);
    }
    std::sort(pieces.begin(), pieces.end(),
              [](const Piece& a, const Piece& b) { return a.q0 < b.q0; });
    size_t at = 0;
    for (const Draft& d : drafts)
      if (d.seq >= 0) merge_sequence(d.seq, d.base, d.parts, pieces, at);
  }

  int sequence_of(int64_t token) const {  // the one that holds it
    auto it = std::upper_bound(q0_.begin(), q0_.end(), token);
    return (int)(it - q0_.begin()) - 1;
  }

  int64_t keys_of(const TokenItem& t) const {
    int64_t n = 0;
    for (int i = 0; i < t.nseg; ++i) n += segments[(size_t)(t.seg0 + i)].n;
    return n;
  }

  tlsp_packed_desc d_;
  const int32_t *q_lens_, *kv_lens_;
  const int64_t* kv_starts_;
  int group_, tile_tokens_;
  int chunk_;  // keys a tile item takes at a time
  std::vector<int64_t> q0_, kv0_;
  std::vector<char> few_;    // sequences of at most kTokenRows rows
  std::vector<char> share_;  // those, and others that share the work on the prefix
  int64_t part_rows_ = 0;
  double tile_time_ = 0;  // of the tile items, in steps
};

bool aligned16(const void* p) { return ((uintptr_t)p & 15u) == 0; }

// A [rows, heads, d] operand the kernels can read 16 bytes at a time.
int validate_rows(const tlsp_rows* r, int64_t rows, int heads, int d, int size) {
  if (rows == 0) return TLSP_OK;
  if (!r || !r->ptr || !aligned16(r->ptr)) return TLSP_ERR_INVALID_ARG;
  const int64_t unit = 16 / size;
  if (rows > 1 && (r->row_stride < d || r->row_stride % unit)) return TLSP_ERR_INVALID_ARG;
  if (heads > 1 && (r->head_stride < d || r->head_stride % unit)) return TLSP_ERR_INVALID_ARG;
  return TLSP_OK;
}

// An output's rows and heads must not share memory: one axis steps over the whole other.
int validate_output(const tlsp_rows* r, int64_t rows, int heads, int d) {
  if (rows <= 1 || heads <= 1) return TLSP_OK;
  const bool rows_outside = r->row_stride >= (heads - 1) * r->head_stride + d;
  const bool heads_outside = r->head_stride >= (rows - 1) * r->row_stride + d;
  return rows_outside || heads_outside ? TLSP_OK : TLSP_ERR_INVALID_ARG;
}

Span span_of(const tlsp_rows& r, int64_t rows, int heads, int d, int size) {
  return Span(r.ptr, (int64_t)d * size)
      .with(rows, (__int128)r.row_stride * size)
      .with(heads, (__int128)r.head_stride * size);
}

// What a call writes (O, lse, its workspace) shares no memory with what it reads, nor with
// each other: other items still read their queries and keys while one's rows are written.
int validate_overlap(const PackedArgs& a, int size, size_t ws_bytes) {
  const Span O = span_of(a.O, a.q_rows, a.heads, a.d, size);
  const Span lse(a.lse, a.lse ? a.q_rows * a.heads * (int64_t)sizeof(float) : 0);
  const Span ws(a.status, (int64_t)ws_bytes);
  if (!apart(O, lse) || !apart(O, ws) || !apart(lse, ws)) return TLSP_ERR_INVALID_ARG;
  const Span read[] = {span_of(a.Q, a.q_rows, a.heads, a.d, size),
                       span_of(a.K, a.kv_rows, a.kv_heads, a.d, size),
                       span_of(a.V, a.kv_rows, a.kv_heads, a.d, size),
                       span_of(a.Kp, a.prefix_len, a.kv_heads, a.d, size),
                       span_of(a.Vp, a.prefix_len, a.kv_heads, a.d, size)};
  for (const Span& r : read)
    if (!apart(O, r) || !apart(lse, r) || !apart(ws, r)) return TLSP_ERR_INVALID_ARG;
  return TLSP_OK;
}

// Strides of axes of length 1 are never used: set to something valid.
tlsp_rows tidy(const tlsp_rows* r, int64_t rows, int heads, int d) {
  tlsp_rows t{};
  if (rows == 0) return t;
  t = *r;
  if (heads <= 1) t.head_stride = d;
  if (rows <= 1) t.row_stride = (int64_t)heads * d;
  return t;
}

int validate_packed(const tlsp_packed_plan* p) {
  if (!p) return TLSP_ERR_INVALID_ARG;
  TLSP_TRY(validate_desc(&p->desc));
  if (p->tile_items < 0 || p->token_items < 0 || p->token_segments < 0 || p->merge_items < 0 || p->q_rows < 0 ||
      p->kv_rows < 0 || p->part_rows < 0 || p->q_rows > kMaxRows || p->kv_rows > kMaxRows)
    return TLSP_ERR_INVALID_ARG;
  return TLSP_OK;
}

int attention(const tlsp_packed_plan* plan, const void* items, const tlsp_rows* Q,
              const tlsp_rows* Kp, const tlsp_rows* Vp, const tlsp_rows* K, const tlsp_rows* V,
              const tlsp_rows* O, float* lse, float scale, void* ws, size_t ws_bytes,
              void* stream) {
  const tlsp_packed_desc& d = plan->desc;
  const bool bf16 = d.dtype == TLSP_BF16;
  const int size = bf16 ? 2 : 4;
  if (!(std::fabs(scale * 1.4426950408889634f) < INFINITY)) return TLSP_ERR_INVALID_ARG;  // as the kernels take it
  TLSP_TRY(validate_rows(Q, plan->q_rows, d.heads, d.head_dim, size));
  TLSP_TRY(validate_rows(O, plan->q_rows, d.heads, d.head_dim, size));
  TLSP_TRY(validate_output(O, plan->q_rows, d.heads, d.head_dim));
  TLSP_TRY(validate_rows(K, plan->kv_rows, d.kv_heads, d.head_dim, size));
  TLSP_TRY(validate_rows(V, plan->kv_rows, d.kv_heads, d.head_dim, size));
  TLSP_TRY(validate_rows(Kp, d.prefix_len, d.kv_heads, d.head_dim, size));
  TLSP_TRY(validate_rows(Vp, d.prefix_len, d.kv_heads, d.head_dim, size));
  if (!ws || !aligned16(ws) || (lse && (uintptr_t)lse % 4)) return TLSP_ERR_INVALID_ARG;
  const WsLayout L = ws_layout(*plan);
  if (ws_bytes < L.total) return TLSP_ERR_WORKSPACE;
  if (plan->q_rows == 0) return TLSP_OK;
  if (!items || !aligned16(items)) return TLSP_ERR_INVALID_ARG;
  PackedArgs a{};
  a.tiles = static_cast<const PackedItem*>(items);
  a.tokens = a.tiles + plan->tile_items;
  a.token_items = reinterpret_cast<const TokenItem*>(a.tokens);
  a.segments = reinterpret_cast<const TokenSegment*>(a.tokens + plan->token_items);
  a.merges = reinterpret_cast<const MergeItem*>(a.segments + plan->token_segments);
  a.n_segments = plan->token_segments;
  a.cluster = plan->cluster;
  a.n_tiles = plan->tile_items;
  a.n_tokens = plan->token_items;
  a.n_merges = plan->merge_items;
  a.merge_parts = plan->merge_parts;
  a.heads = d.heads;
  a.kv_heads = d.kv_heads;
  a.group = d.heads / d.kv_heads;
  a.d = d.head_dim;
  a.q_rows = plan->q_rows;
  a.kv_rows = plan->kv_rows;
  a.prefix_len = d.prefix_len;
  a.part_rows = plan->part_rows;
  a.Q = tidy(Q, plan->q_rows, d.heads, d.head_dim);
  a.O = tidy(O, plan->q_rows, d.heads, d.head_dim);
  a.K = tidy(K, plan->kv_rows, d.kv_heads, d.head_dim);
  a.V = tidy(V, plan->kv_rows, d.kv_heads, d.head_dim);
  a.Kp = tidy(Kp, d.prefix_len, d.kv_heads, d.head_dim);
  a.Vp = tidy(Vp, d.prefix_len, d.kv_heads, d.head_dim);
  a.lse = lse;
  a.scale = scale != 0.f ? scale : 1.f / sqrtf((float)d.head_dim);
  char* base = static_cast<char*>(ws);
  a.status = reinterpret_cast<int*>(base);
  a.part_lse = reinterpret_cast<float*>(base + L.lse);
  a.part_o = reinterpret_cast<float*>(base + L.o);
  TLSP_TRY(validate_overlap(a, size, L.total));
  cudaStream_t st = (cudaStream_t)stream;
  if (bf16) {
    if (a.n_tiles > 0) TLSP_TRY(packed_tile(a, st));
    if (a.n_tokens > 0) TLSP_TRY(packed_token(a, a.n_tiles > 0, st));
  } else {
    TLSP_TRY(packed_simt(a, st));
  }
  if (a.n_merges > 0) TLSP_TRY(packed_merge(a, bf16, st));
  return TLSP_OK;
}

}  // namespace
}  // namespace tlsp

using namespace tlsp;

extern "C" {

int tlsp_packed_make_plan(const tlsp_packed_desc* desc, const int32_t* q_lens,
                          const int32_t* kv_lens, const int64_t* kv_starts, void* items,
                          size_t items_bytes, tlsp_packed_plan* plan) {
  TLSP_TRY(validate_desc(desc));
  if (!q_lens || !kv_lens || !plan) return TLSP_ERR_INVALID_ARG;
  try {
    Planner p(*desc, q_lens, kv_lens, kv_starts);
    TLSP_TRY(p.run());
    tlsp_packed_plan out{};
    out.desc = *desc;
    out.tile_items = (int32_t)p.tiles.size();
    out.token_items = (int32_t)(p.tokens.size() + p.token_items.size());
    out.token_segments = (int32_t)p.segments.size();
    out.cluster = p.cluster;
    out.merge_parts = p.merge_parts;
    out.merge_items = (int32_t)p.merges.size();
    out.q_rows = p.q_rows;
    out.kv_rows = p.kv_rows;
    out.part_rows = p.part_rows();
    out.items_bytes =
        sizeof(PackedItem) * (p.tiles.size() + p.tokens.size() + p.token_items.size() +
                              p.segments.size() + p.merges.size());
    out.ws_bytes = ws_layout(out).total;
    *plan = out;
    if (items_bytes < out.items_bytes || (out.items_bytes > 0 && !items)) return TLSP_ERR_WORKSPACE;
    char* to = static_cast<char*>(items);
    auto put = [&](const void* from, size_t bytes) {
      if (bytes) std::memcpy(to, from, bytes);
      to += bytes;
    };
    put(p.tiles.data(), sizeof(PackedItem) * p.tiles.size());
    put(p.tokens.data(), sizeof(PackedItem) * p.tokens.size());
    put(p.token_items.data(), sizeof(TokenItem) * p.token_items.size());
    put(p.segments.data(), sizeof(TokenSegment) * p.segments.size());
    put(p.merges.data(), sizeof(MergeItem) * p.merges.size());
  } catch (...) {  // out of host memory
    return TLSP_ERR_UNSUPPORTED;
  }
  return TLSP_OK;
}

int tlsp_packed_attention(const tlsp_packed_plan* plan, const void* items, const tlsp_rows* Q,
                          const tlsp_rows* K, const tlsp_rows* V, const tlsp_rows* O, float* lse,
                          float scale, void* ws, size_t ws_bytes, void* stream) {
  TLSP_TRY(validate_packed(plan));
  if (plan->desc.prefix_len != 0) return TLSP_ERR_INVALID_ARG;
  return attention(plan, items, Q, nullptr, nullptr, K, V, O, lse, scale, ws, ws_bytes, stream);
}

int tlsp_prefix_attention(const tlsp_packed_plan* plan, const void* items, const tlsp_rows* Q,
                          const tlsp_rows* Kp, const tlsp_rows* Vp, const tlsp_rows* K,
                          const tlsp_rows* V, const tlsp_rows* O, float* lse, float scale,
                          void* ws, size_t ws_bytes, void* stream) {
  TLSP_TRY(validate_packed(plan));
  if (plan->desc.prefix_len < 1) return TLSP_ERR_INVALID_ARG;
  return attention(plan, items, Q, Kp, Vp, K, V, O, lse, scale, ws, ws_bytes, stream);
}

}  // extern "C"
