// How an attention call is cut into workgroups.  Host code without a GPU in it:
// a function of the call's sizes alone (where it says stretches, the kernel cuts
// these by the sequences' lengths).
#pragma once

#include <stddef.h>
#include <stdint.h>

namespace pq1 {

constexpr int kTileRows = 256;  // rows of a many-rows tile
constexpr int kKeys = 32;       // keys of a tile of the few-rows kernel
constexpr int kWaves = 4;       // waves of its workgroup
template <int D>
constexpr int kTileKeys = D == 256 ? 32 : 64;  // keys of a tile of the many-rows kernel
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
  // plan_window, few rows: workgroups among which the batch's work is cut evenly;
  // 0: nsplit parts of every (sequence, cache head, row tile)
  int wgs = 0;
  bool joined = false;    // plan_window: a second launch joins parts
};

// Which kernel: estimated times, in ns, of a call whose work fills the device.
// A CU takes 0.19 D ns a key for a 32-row tile of the few-rows kernel, whose
// start costs as much as 130 keys, and 20 + 0.16 D ns a key for a 256-row tile
// of the other, which needs 7 us more before its first key.  At D = 128, 8
// cache heads, few rows against many: 64 sequences of 1000 keys, 24 rows 46 and
// 82 us, 72 rows 120 and 87; one sequence of 8000 keys, 48 rows 18 and 28, 144
// rows 44 and 31; of 500 keys, 384 rows 14 and 25.
//
// Of a 4-bit cache the few-rows kernel takes 0.1 D ns, the other converts what it
// reads and takes what it did.  64 sequences of 1000 keys, 40 rows at D = 128 and 256:
// 50 and 75, 101 and 121 us, 72 rows 69 and 75, 148 and 127, 144 rows 113 and 86, 249
// and 147; one of 8000 keys, 40 rows 20 and 24, 25 and 33, 288 rows 44 and 42, 78 and 55.
inline bool prefer_many(int64_t units, int64_t rows, int64_t keys, int D, bool four = false) {
  const double per_cu = static_cast<double>(units) / 256;
  const double few = static_cast<double>((rows + 31) / 32) * per_cu * (keys + 130.0) *
                     (four ? 0.1 : 0.19) * D;
  const double many = static_cast<double>((rows + kTileRows - 1) / kTileRows) * per_cu * keys *
                          (20 + 0.16 * D) + 7000;
  return rows > 32 && many < few;
}

// Up to this many elements of K a head's keys stay in one part where rows are
// few: one launch.  One token of 4 cache heads at D = 256, calls one after
// another: 300 keys 10.9 us in one part and 14.7 in several, 700 keys 17.4 and
// 14.6; at D = 128 700 keys 10.8 and 14.5, 1500 keys 16.7 and 14.7.
constexpr int64_t kShort = 98304;
// plan_window: with parts as short as that a batch of different lengths is not
// worth cutting evenly: finding a stretch costs 2 us and more (4-bit, D = 256, in
// parts and in stretches: one sequence of 700 keys 14.1 and 14.9 us, of 131070 42
// and 45; 16 sequences of 4000 22 and 24; 200 of 1000 54 and 63).
constexpr int64_t kPart = 262144;

// Parts of that many keys for so many (sequence, cache head, row tile)s.
inline int64_t parts_of(bool many, int64_t units, int64_t keys, int D) {
  constexpr int64_t cus = 256, step = kKeys * kWaves;
  int64_t parts = 1;
  if (many) {
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
}

inline AttnPlan plan_attention(int64_t B, int64_t T, int Hq, int Hk, int D, int64_t max_q,
                               int64_t max_kv, int window = 0) {
  // A launch holds less than 2^32 threads.  Kernels walk on over rows that
  // their grid has no workgroup for, so a long chunk only costs balance.
  constexpr int64_t most = (int64_t{1} << 32) / (2 * kTileRows) - 1;
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
  auto cut = [&](int64_t keys) { return parts_of(p.many, units, keys, D); };
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

// The same for the calls whose workspace knows the window: the kernel is chosen,
// and the workspace made, by the keys that a tile of rows walks over (with
// `sinks` first keys that stay visible).
inline AttnPlan plan_window(int64_t B, int64_t T, int Hq, int Hk, int D, int64_t max_q,
                            int64_t max_kv, int window, int sinks, bool four) {
  constexpr int64_t most = (int64_t{1} << 32) / (2 * kTileRows) - 1;
  AttnPlan p;
  if (B * Hk > most) return p;
  p.fits = true;
  p.tokens = max_q < 1 ? 1 : max_q < T ? max_q : T;
  const int64_t G = Hq / Hk, rows = p.tokens * G;
  const int64_t kv = max_kv < 1 ? 1 : max_kv > kMaxKeys ? kMaxKeys : max_kv;
  auto walk = [&](int64_t tile_rows) {
    // the window of its first row, a key more for each token after that, the
    // rounding of the start, and the first keys, rounded up
    const int64_t tokens = (tile_rows + G - 1) / G + 1;
    const int64_t tile = tile_rows < kTileRows ? kKeys : D == 256 ? kTileKeys<256> : kTileKeys<64>;
    const int64_t reach = int64_t{window} + (tokens < p.tokens ? tokens : p.tokens) - 1 + tile - 1 +
                          (int64_t{sinks} + tile - 1) / tile * tile;
    return window > 0 && reach < kv ? reach : kv;
  };
  p.many = prefer_many(B * Hk, rows, walk(kTileRows), D, four);
  p.tile_rows = p.many ? kTileRows : rows <= 16 ? 16 : 32;
  p.row_tiles = (rows + p.tile_rows - 1) / p.tile_rows;
  if (p.row_tiles > most / (B * Hk)) p.row_tiles = most / (B * Hk);
  const int64_t units = B * Hk * p.row_tiles;
  const int64_t keys = walk(p.tile_rows), step = kKeys * kWaves;
  if (p.many) {
    const int64_t n = parts_of(true, units, keys, D);
    p.chunk = static_cast<int>(((keys + n - 1) / n + step - 1) / step * step);
    p.nsplit = static_cast<int>((keys + p.chunk - 1) / p.chunk);
    p.joined = p.nsplit > 1;
    if (p.joined) p.workspace_bytes = static_cast<size_t>(p.nsplit) * T * Hq * (D * 4 + 8);
    return p;
  }
  // Few rows: whole tiles where keys are few, where a window keeps the lengths alike
  // and where tiles are many; parts for one sequence or where they are short; else
  // stretches, as many as the device holds at once.  A window does so up to about 0.6
  // of the longest sequence (64 sequences of 200 to 8000 keys, 4 cache heads, D = 256,
  // in stretches and whole: 4-bit, windows of 1024, 4000, 6000 and 8000 24 and 21, 59
  // and 55, 69 and 76, 72 and 93 us; two-byte 63 and 52, 159 and 148, 193 and 194, 205
  // and 234; 48 sequences of 8 heads, D = 128, two-byte 46 and 43, 120 and 122, 138 and
  // 168, 146 and 188).
  const int per_cu = D == 256 && (!four || p.tile_rows == 32) ? 1 : 2;
  const int64_t slots = 256 * per_cu, steps = (keys + step - 1) / step;
  const int64_t n = (slots + units - 1) / units;
  if (keys * D <= kShort || units >= (5 * keys <= 3 * kv ? 256 : 4 * slots)) return p;
  p.joined = true;
  if (B == 1 || keys * D <= n * kPart) {
    p.nsplit = static_cast<int>(n < steps ? n : steps);
    p.joined = p.nsplit > 1;
    if (p.joined) p.workspace_bytes = static_cast<size_t>(p.nsplit) * T * Hq * (D * 4 + 8);
    return p;
  }
  p.wgs = static_cast<int>(units * steps < slots ? units * steps : slots);
  p.workspace_bytes = static_cast<size_t>(2 * p.wgs) * p.tile_rows * (D * 4 + 8) +
                      static_cast<size_t>((T * G / p.tile_rows + B + 1) * Hk) * 8;
  return p;
}

}  // namespace pq1
