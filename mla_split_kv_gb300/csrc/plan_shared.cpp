// Work of a batch whose contexts start with the same tokens (host only, no GPU access).
//
// The common tokens are cut into pieces for every group of 128 of the batch's rows, each request's own tokens for its
// own groups: into equally long ones, or into ones of a length and what is left. A piece is two units of work (one half
// of the value columns each), the units go longest first to the CTA (one an SM) that is free first, and the way and
// length are those among some tried whose busiest CTA and merge are done first.
#include <algorithm>
#include <cstdint>
#include <functional>
#include <queue>
#include <vector>

#include "kernels.h"
#include "mla_split_kv.h"

namespace {

constexpr int64_t kTile = 64;   // tokens
constexpr int64_t kGroup = 128; // rows
// A unit's time in tiles of about 1.1 us: its tiles, and the start and the end (queries, the first loads, the partial
// output; plans made with 4 or 8 are within 1%). A row's part costs the merge about 2 KB of L2, of which the device
// reads 5 MB in the time of a tile.
constexpr int64_t kUnitTiles = 6;
constexpr int64_t kMergeParts = 2500;

struct Piece {
  int64_t row0, rows;
  int32_t request;
  int64_t t0, t1, tiles, slot;
};

int64_t tiles_of(int64_t tokens) { return (tokens + kTile - 1) / kTile; }
// How runs are cut: no piece longer than `length` tiles, all but the last as long as `of` says.
struct Cut {
  int64_t length;
  bool even;
  int64_t pieces(int64_t tiles) const { return std::max<int64_t>(1, (tiles + length - 1) / length); }
  int64_t of(int64_t tiles) const {
    const int64_t n = pieces(tiles);
    return even ? std::max<int64_t>(1, (tiles + n - 1) / n) : length;
  }
};

}  // namespace

extern "C" mla_status_t mla_plan_shared(const int32_t* context_lens_host, int32_t B, int32_t num_heads, int32_t q_len,
                                        int32_t block_size, const mla_device_info_t* dev, mla_shared_plan_t* plan) try {
  if (context_lens_host == nullptr || dev == nullptr || plan == nullptr) return MLA_ERR_INVALID_ARG;
  if (B < 1 || dev->num_sms < 1 || plan->unit_capacity < 0) return MLA_ERR_INVALID_ARG;
  if (num_heads != 16 && num_heads != 64 && num_heads != 128) return MLA_ERR_UNSUPPORTED;
  if (q_len < 1 || q_len > MLA_MAX_Q_LEN) return MLA_ERR_UNSUPPORTED;
  if (block_size != 16 && block_size != 32 && block_size != 64) return MLA_ERR_UNSUPPORTED;
  const int64_t P = plan->shared_tokens;
  if (P < block_size || P % block_size != 0) return MLA_ERR_INVALID_ARG;
  const int64_t per = static_cast<int64_t>(q_len) * num_heads, rows = per * B;
  if (rows > (1ll << 28)) return MLA_ERR_UNSUPPORTED;
  int64_t longest = 0;
  for (int32_t b = 0; b < B; ++b) {
    if (context_lens_host[b] < 0) return MLA_ERR_INVALID_ARG;
    longest = std::max<int64_t>(longest, context_lens_host[b]);
  }
  const int64_t groups = (rows + kGroup - 1) / kGroup, own_groups = (per + kGroup - 1) / kGroup;
  const int64_t common = tiles_of(P);
  std::vector<int64_t> own(B);
  int64_t all = groups * common, most = common;
  for (int32_t b = 0; b < B; ++b) {
    own[b] = tiles_of(std::max<int64_t>(0, context_lens_host[b] - P));
    all += own_groups * own[b];
    most = std::max(most, own[b]);
  }

  // tile counts a piece may have, around an even share of one SM's two units at a time
  const int64_t share = std::max<int64_t>(1, 2 * all / dev->num_sms);
  Cut best{most, true};
  int64_t best_cost = -1, tried = 0;
  // (many requests even out by themselves: fewer lengths are tried)
  const int64_t step = groups + static_cast<int64_t>(B) * own_groups > 500 ? 8 : 1;
  for (int64_t part = 8; part <= 64; part += step) {  // 32nds of the share
    const int64_t length = std::min(most, std::max<int64_t>(2, (share * part + 31) / 32));
    if (length == tried) continue;
    tried = length;
    for (const bool even : {true, false}) {
      const Cut cut{length, even};
      std::vector<std::pair<int64_t, int64_t>> units;  // tiles, how many
      int64_t parts = 0, sum = 0;
      auto add = [&](int64_t tiles, int64_t times, int64_t rows_of) {
        const int64_t n = cut.pieces(tiles), each = cut.of(tiles);
        if (n > 1) units.emplace_back(each, 2 * times * (n - 1));
        units.emplace_back(tiles - (n - 1) * each, 2 * times);
        parts += n * rows_of;
        sum += 2 * times * (tiles + n * kUnitTiles);
      };
      add(common, groups, rows);
      for (int32_t b = 0; b < B; ++b) add(own[b], own_groups, per);
      // (no better than the average, and none that is already as long as the best is gone on with)
      const int64_t merge = parts / kMergeParts;
      int64_t busiest = (sum + dev->num_sms - 1) / dev->num_sms;
      auto lost = [&] { return best_cost >= 0 && busiest + merge >= best_cost; };
      if (lost()) continue;
      std::sort(units.begin(), units.end(), std::greater<>());
      std::priority_queue<int64_t, std::vector<int64_t>, std::greater<int64_t>> ends;
      for (int32_t i = 0; i < dev->num_sms; ++i) ends.push(0);
      for (const auto& u : units) {
        for (int64_t i = 0; i < u.second && !lost(); ++i) {
          const int64_t end = ends.top() + u.first + kUnitTiles;
          ends.pop();
          ends.push(end);
          busiest = std::max(busiest, end);
        }
      }
      if (lost()) continue;
      best_cost = busiest + merge;
      best = cut;
    }
  }

  std::vector<Piece> pieces;
  int64_t slot = 0;
  auto cut = [&](int64_t row0, int64_t n_rows, int32_t request, int64_t t0, int64_t tokens, bool open) {
    const int64_t tiles = tiles_of(tokens), n = best.pieces(tiles), each = best.of(tiles);
    for (int64_t j = 0; j < n; ++j) {
      const int64_t a = std::min(tokens, j * each * kTile), e = std::min(tokens, (j + 1) * each * kTile);
      const bool last = j + 1 == n;
      pieces.push_back(Piece{row0, n_rows, request, t0 + a, last && open ? 0x7fffffffll : t0 + e, tiles_of(e - a), slot++});
    }
    return n;
  };
  int64_t parts = 0;
  for (int64_t g = 0; g < groups; ++g)
    parts = cut(g * kGroup, std::min(kGroup, rows - g * kGroup), -1, 0, P, false);
  std::vector<int64_t> first;
  for (int32_t b = 0; b < B; ++b) {
    for (int64_t g = 0; g < own_groups; ++g) {
      first.push_back(slot);
      cut(b * per + g * kGroup, std::min(kGroup, per - g * kGroup), b, P, std::max<int64_t>(0, context_lens_host[b] - P), true);
    }
  }
  first.push_back(slot);
  if (slot > (1ll << 27)) return MLA_ERR_UNSUPPORTED;
  plan->num_units = 2 * static_cast<int32_t>(pieces.size());
  plan->num_slots = static_cast<int32_t>(slot);
  plan->shared_parts = static_cast<int32_t>(parts);
  plan->num_ctas = std::min(dev->num_sms, plan->num_units);
  if (plan->num_units > plan->unit_capacity) return MLA_ERR_CAPACITY;
  if (plan->units == nullptr || plan->own_indptr == nullptr || plan->cta_indptr == nullptr) return MLA_ERR_INVALID_ARG;
  std::stable_sort(pieces.begin(), pieces.end(), [](const Piece& a, const Piece& b) { return a.tiles > b.tiles; });
  std::vector<std::vector<int32_t>> lists(plan->num_ctas);
  std::priority_queue<std::pair<int64_t, int32_t>, std::vector<std::pair<int64_t, int32_t>>, std::greater<>> free_at;
  for (int32_t c = 0; c < plan->num_ctas; ++c) free_at.emplace(0, c);
  for (int32_t u = 0; u < plan->num_units; ++u) {
    const auto next = free_at.top();
    free_at.pop();
    lists[next.second].push_back(u);
    free_at.emplace(next.first + pieces[u >> 1].tiles + kUnitTiles, next.second);
  }
  int32_t at = 0;
  for (int32_t c = 0; c < plan->num_ctas; ++c) {
    plan->cta_indptr[c] = at;
    for (const int32_t u : lists[c]) {
      const Piece& x = pieces[u >> 1];
      plan->units[at++] = mla_shared_unit_t{static_cast<int32_t>(x.row0), static_cast<int32_t>(x.rows), x.request,
                                            static_cast<int32_t>(x.t0), static_cast<int32_t>(x.t1), static_cast<int32_t>(x.slot), u & 1, 0};
    }
  }
  plan->cta_indptr[plan->num_ctas] = at;
  for (size_t i = 0; i < first.size(); ++i) plan->own_indptr[i] = static_cast<int32_t>(first[i]);
  return MLA_OK;
} catch (...) {  // out of memory
  return MLA_ERR_CAPACITY;
}
