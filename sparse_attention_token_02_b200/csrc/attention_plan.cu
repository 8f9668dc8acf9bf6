// How a call of attention over the latent cache is cut into work items: host code only.
#include <cuda_runtime.h>

#include <algorithm>

#include "internal.h"

namespace dsa {

namespace {

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// Time until `sms` SMs that take items in order are done with n1 items of cost c1 and then n2 of cost c2.
double finish(int64_t n1, double c1, int64_t n2, double c2, int64_t sms) {
  const int64_t ahead = n1 % sms;                        // SMs with one item more than the others
  const double low = double(n1 / sms) * c1, high = ahead ? low + c1 : low;
  if (n2 == 0) return high;
  double lo = std::max(high, low), hi = high + double(ceil_div(n2, sms)) * c2;
  auto room = [&](double t) { return ahead * int64_t((t - high) / c2 + 1e-9) + (sms - ahead) * int64_t((t - low) / c2 + 1e-9); };
  if (room(lo) >= n2) return lo;
  for (int i = 0; i < 20; ++i) {
    const double t = 0.5 * (lo + hi);
    (room(t) >= n2 ? hi : lo) = t;
  }
  return hi;
}

// Cuts a call into items, in units of a tile's time (1.3 us).  An item costs its tiles and about four tiles' time beside
// them (set-up, queries, result); its products always have 64 rows, but with fewer rows of its own there is less to
// write and to join: few tokens are cut into groups of 16 or 32 heads, as long as there are SMs for them (1 x 128 heads
// over 2048 keys 15.5 -> 12.6 us, 8 x 64 heads over 512 keys 14.3 -> 11.9).  Splitting a row costs its join: in a cluster
// (two to sixteen parts) one to five tiles' time, through memory a second kernel and the parts' traffic.  A pair's tile
// takes 0.85 of the time of one CTA's, an FP8 tile that is expanded on the way 1.4.  A token's rows are whole groups where
// H is a multiple of 64; sharing a prefix then saves no tile, and shared positions are read by the tokens' own items.
// Where the device does not say how many clusters it holds, *answered is false and the plan does without.
AttnPlan make_plan(int64_t T, int32_t H, int64_t shared_keys, int64_t own_keys, bool fp8, int sms, bool* answered) {
  const int64_t R = T * H, shared_groups = ceil_div(R, kAttnRows), own_groups = ceil_div(H, kAttnRows);
  int64_t shared_tiles = ceil_div(shared_keys, kAttnTile);
  // Expanding FP8 rows to bf16 costs the loading warps more time than a tile's products take; a prefix that many
  // groups of rows read is expanded once instead (23 x 128 heads over 16001 keys: 248 -> 173 us
  // then, 151 in pairs).
  const bool expand = fp8 && shared_groups >= 4 && shared_groups * shared_tiles >= 8 * sms;
  if (H % kAttnRows == 0 && !expand) {
    own_keys += shared_keys;
    shared_tiles = 0;
  }
  // a call with no keys at all still writes its empty rows
  const int64_t own_tiles = own_keys > 0 || shared_tiles == 0 ? std::max<int64_t>(1, ceil_div(own_keys, kAttnTile)) : 0;
  const int64_t longest = std::max(shared_tiles, own_tiles);
  AttnPlan best{};
  double best_cost = 0.0;
  auto consider = [&](int64_t chunk, int cluster, bool pair = false, int rows = kAttnRows) {
    AttnPlan p{};
    const int64_t own_groups = ceil_div(H, rows);
    p.own_rows = rows;
    p.pair = pair;
    p.shared_groups = static_cast<int32_t>(shared_groups);
    p.own_groups = static_cast<int32_t>(own_groups);
    p.shared_slots = static_cast<int32_t>(ceil_div(shared_tiles, chunk));
    p.own_slots = cluster > 1 ? cluster : static_cast<int32_t>(ceil_div(own_tiles, chunk));
    p.shared_chunk = p.own_chunk = static_cast<int32_t>(chunk * kAttnTile);
    p.cluster = cluster;
    p.expand = expand;
    const int room = cluster > 1 ? cluster_room(cluster, sms, answered) : sms;
    if (p.slots() > kMaxSlots || room < cluster) return;
    // an item's time beside its tiles: for full groups, and for a token's own with the cluster's join
    const double share = double(rows) / kAttnRows, own_share = std::min(1.0, double(std::min(rows, H)) / kAttnRows);
    const double full = 4.3, fp8_start = fp8 && chunk > 1 ? 0.8 : 0.0;
    const double item = 2.8 + 1.5 * own_share + fp8_start + (cluster > 1 ? 1.9 + (1.0 + 0.24 * cluster) * share : 0.0);
    // bf16 keys of tokens that each read their own: 115 SMs take all that HBM gives
    const double readers = double(std::min<int64_t>(T * own_groups * p.own_slots, sms)) / own_groups;
    const double own_tile = fp8 ? 1.4 : std::max(1.0, readers / 115);
    double cost = cluster == 1 && p.slots() > 1 ? 1.9 + p.slots() * (0.045 + R * 0.0004) : 0.0;
    if (pair) {
      // two SMs an item; an FP8 cache's own items stay with the single kernel, launched behind
      const double tile = 0.85, own_item = 3.0 + std::min(2.0, H / 64.0);
      const int64_t shared_pairs = (shared_groups + 1) / 2 * p.shared_slots, own_pairs = fp8 ? 0 : T * p.own_slots;
      cost += finish(shared_pairs, double(chunk) * tile + 5.0, own_pairs, double(std::min(chunk, own_tiles)) * tile + own_item,
                     cluster_room(2, sms, answered) / 2);
      if (fp8 && p.own_slots)
        cost += 1.0 + finish(T * own_groups * p.own_slots, double(std::min(chunk, own_tiles)) * own_tile + item, 0, 1.0, sms);
    } else {
      cost += finish(shared_groups * p.shared_slots, double(chunk) * (expand ? 1.0 : own_tile) + full, T * own_groups * p.own_slots,
                     double(std::min(chunk, own_tiles)) * own_tile + item, room);
    }
    if (best.slots() == 0 || cost < best_cost) {
      best = p;
      best_cost = cost;
    }
  };
  consider(longest, 1);
  // in pairs: bf16 keys that at least two groups of rows share
  const bool pairs = (fp8 ? expand : shared_tiles > 0 || own_groups == 2) && cluster_room(2, sms, answered) >= 2;
  if (pairs) consider(longest, 1, true);
  // chunks with which the longer part fills one to four rounds of the SMs, alone or with the other part beside it
  const int64_t least = ceil_div(longest, kMaxSlots / 2);
  auto cuts = [&](bool pair, int rows) {
    const int64_t own = pair ? 1 : ceil_div(H, rows), shared = pair ? (shared_groups + 1) / 2 : shared_groups;
    const int64_t units = pair ? std::max(1, cluster_room(2, sms, answered) / 2) : sms;       // that take an item each
    const int64_t groups = shared_tiles ? shared : T * own;
    const int64_t tiles = shared * shared_tiles + (pair && fp8 ? 0 : T * own * own_tiles);
    for (int rounds = 1; rounds <= 4; ++rounds) {
      const int64_t pieces = int64_t(rounds) * units / groups;      // of each group of rows
      if (pieces > 1) consider(std::max(ceil_div(longest, pieces), least), 1, pair, rows);
      // rounding up to whole chunks can need a few items too many: larger chunks need fewer
      int64_t chunk = std::max(ceil_div(tiles, int64_t(rounds) * units), least);
      for (int x = 0; x < 4 && chunk < longest; ++x, chunk += std::max<int64_t>(1, chunk / 16)) consider(chunk, 1, pair, rows);
    }
  };
  cuts(false, kAttnRows);
  if (pairs) cuts(true, kAttnRows);
  if (shared_tiles == 0)
    for (int rows = kAttnRows; rows >= 16; rows /= 2) {
      if (rows < kAttnRows && (rows >= H || T * ceil_div(H, rows) > sms)) continue;
      for (int cluster = 2; cluster <= kMaxCluster && cluster <= own_tiles; cluster *= 2)
        consider(ceil_div(own_tiles, cluster), cluster, false, rows);
      if (rows < kAttnRows) {
        consider(longest, 1, false, rows);
        cuts(false, rows);
      }
    }
  return best;
}

}  // namespace

// The plan depends on the sizes and the device (how its SMs fall into GPCs) alone; a call and the workspace query
// before it ask for the same one.  One that was made without the device's answer serves its call only.
AttnPlan plan_attention(int64_t T, int32_t H, int64_t shared_keys, int64_t own_keys, bool fp8, int sms) {
  struct Last {
    int64_t T = 0, shared_keys = 0, own_keys = 0;
    int32_t H = 0, fp8 = 0, sms = 0, device = 0;
    AttnPlan plan{};
  };
  thread_local Last last;
  int device = 0;
  if (cudaGetDevice(&device) != cudaSuccess) device = -1;
  if (last.T == T && last.H == H && last.shared_keys == shared_keys && last.own_keys == own_keys && last.fp8 == static_cast<int32_t>(fp8) &&
      last.sms == sms && last.device == device)
    return last.plan;
  bool answered = true;
  const AttnPlan plan = make_plan(T, H, shared_keys, own_keys, fp8, sms, &answered);
  if (answered) last = Last{T, shared_keys, own_keys, H, fp8, sms, device, plan};
  return plan;
}

}  // namespace dsa
