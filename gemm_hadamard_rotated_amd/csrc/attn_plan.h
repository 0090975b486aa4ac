// How an attention call is cut into workgroups.  Host code without a GPU in it:
// a function of the call's sizes alone.
#pragma once

#include <stddef.h>
#include <stdint.h>

namespace pq1 {

constexpr int kTileRows = 256;  // rows of a many-rows tile
constexpr int kKeys = 32;       // keys of a tile of the few-rows kernel
constexpr int kWaves = 4;       // waves of its workgroup
constexpr int kMaxKeys = 0x7fff0000;  // of a sequence: key numbers plus a tile stay in 31 bits

struct AttnPlan {
  int64_t tokens = 0;     // new tokens of the longest chunk
  bool many = false;      // tiles of many rows (paged_attention_tiles.hip)
  int tile_rows = 16;     // rows of a row tile
  int64_t row_tiles = 0;  // row tiles of one (sequence, cache head)
  int nsplit = 1;         // parts of the keys
  int chunk = 0;          // keys of a part
  size_t workspace_bytes = 0;
  bool fits = false;      // the grid is launchable
};

// Which kernel: estimated times, in ns, of a call whose work fills the device.
// A CU takes 0.19 D ns a key for a 32-row tile of the few-rows kernel, whose
// start costs as much as 130 keys, and 20 + 0.16 D ns a key for a 256-row tile
// of the other, which needs 7 us more before its first key.  At D = 128, 8
// cache heads, few rows against many: 64 sequences of 1000 keys, 24 rows 46 and
// 82 us, 72 rows 120 and 87; one sequence of 8000 keys, 48 rows 18 and 28, 144
// rows 44 and 31; of 500 keys, 384 rows 14 and 25.
inline bool prefer_many(int64_t units, int64_t rows, int64_t keys, int D) {
  const double per_cu = static_cast<double>(units) / 256;
  const double few = static_cast<double>((rows + 31) / 32) * per_cu * (keys + 130.0) * 0.19 * D;
  const double many = static_cast<double>((rows + kTileRows - 1) / kTileRows) * per_cu * keys *
                          (20 + 0.16 * D) + 7000;
  return rows > 32 && many < few;
}

// Up to this many elements of K a head's keys stay in one part where rows are
// few: one launch.  One token of 4 cache heads at D = 256, calls one after
// another: 300 keys 10.9 us in one part and 14.7 in several, 700 keys 17.4 and
// 14.6; at D = 128 700 keys 10.8 and 14.5, 1500 keys 16.7 and 14.7.
constexpr int64_t kShort = 98304;

inline AttnPlan plan_attention(int64_t B, int64_t T, int Hq, int Hk, int D, int64_t max_q,
                               int64_t max_kv, int window = 0) {
  // A launch holds less than 2^32 threads.  Kernels walk on over rows that
  // their grid has no workgroup for, so a long chunk only costs balance.
  constexpr int64_t most = (int64_t{1} << 32) / (2 * kTileRows) - 1;
  constexpr int64_t cus = 256;
  AttnPlan p;
  if (B * Hk > most) return p;
  p.fits = true;
  p.tokens = max_q < 1 ? 1 : max_q < T ? max_q : T;
  const int64_t rows = p.tokens * (Hq / Hk);
  // No sequence has more than kMaxKeys, so that one part can hold all its keys.
  int64_t kv = max_kv < 1 ? 1 : max_kv > kMaxKeys ? kMaxKeys : max_kv;
  p.many = prefer_many(B * Hk, rows, kv, D);
  p.tile_rows = p.many ? kTileRows : rows <= 16 ? 16 : 32;
  p.row_tiles = (rows + p.tile_rows - 1) / p.tile_rows;
  if (p.row_tiles > most / (B * Hk)) p.row_tiles = most / (B * Hk);
  const int64_t units = B * Hk * p.row_tiles;
  const int64_t step = kKeys * kWaves;
  auto cut = [&](int64_t keys) {  // parts of that many keys
    int64_t parts = 1;
    if (p.many) {
      // One workgroup to a CU: as many parts as the device takes at once.
      // More, to even out a last round, cost more than they give (192
      // workgroups of 7168 keys: 396 us; in 4 parts, three full rounds: 407 us
      // and 48 to join them): idle CUs leave the others a higher clock.
      while (units * (parts + 1) <= cus && (parts + 1) * 256 <= keys) ++parts;
    } else if (units < cus && keys * D > kShort) {
      parts = (cus + units - 1) / units;
    }
    // no part shorter than one key tile for each wave
    const int64_t most_parts = (keys + step - 1) / step;
    return parts < most_parts ? parts : most_parts;
  };
  // The workspace is for all keys, of which a window may leave fewer (a tile's
  // rows see the window's keys, one more for each row after the first, and the
  // start is rounded down): no more parts, shorter ones.
  const int64_t parts = cut(kv);
  p.workspace_bytes = parts > 1 ? static_cast<size_t>(parts) * T * Hq * (D * 4 + 8) : 0;
  const int64_t reach = int64_t{window} + p.tile_rows + 64;
  if (window > 0 && reach < kv) kv = reach;
  // Parts of at least kv / n keys are at most n (kMaxKeys is a multiple of the
  // step, so rounding up stays within 31 bits).
  static_assert(kMaxKeys % (kKeys * kWaves) == 0, "");
  const int64_t n = cut(kv);
  p.chunk = static_cast<int>(((kv + n - 1) / n + step - 1) / step * step);
  p.nsplit = static_cast<int>((kv + p.chunk - 1) / p.chunk);
  return p;
}

}  // namespace pq1
