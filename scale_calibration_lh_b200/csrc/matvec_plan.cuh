// How a product of lhcal_matvec is laid out over warps and shared memory. Host arithmetic alone, so that its
// bounds can be checked over all sizes without a GPU.
#pragma once

#include <stdint.h>

#include "lhcal.h"

namespace lhcal {

constexpr int kMaxWarps = 20;               // that multiply; one more copies
constexpr int kXBlock = LHCAL_SCALE_BLOCK;  // channels of one activation scale
constexpr int kPieceK = 2 * kXBlock;        // channels of a warp
constexpr int kTile = 16;                   // rows of a stage
constexpr int kTokens = 8;                  // slots of an entry
constexpr int kMaxSmem = 227 * 1024;
constexpr int kStaticSmem = 512;            // what is kept for the barriers
constexpr int kMinRows = 8;                 // rows a CTA takes at least
constexpr int kStages = 8;                  // aimed at; up to kMaxStages for a multiple of wr
constexpr int kMaxStages = 16;
// Below as many tiles a CTA, one warp takes each: more would load the same activations (1 x 10 of 512
// experts 1280 x 2560, 6 tiles: 11.0 against 12.6 us, 8 x 10, 44 tiles: 33.0 against 32.4).
constexpr int kFewTiles = 16;

struct MatvecSizes {
  bool routed;
  bool wide;
  int32_t slots, per_row, groups;
  int64_t rows, cin;
  int32_t sms;
};

struct MatvecPlan {
  int wide;      // 16-byte reads of weights and whole words of scales; 8 bytes and single ones otherwise
  int passes;
  int wk, wr;    // warps over the channels and over the row tiles
  int room;      // floats of a warp's sums
  int stages;    // a multiple of wr
  int w_pitch, c_pitch;  // bytes of a row in a stage: weights, scale codes
  int grid;
  uint32_t per_row;  // 2^20 / slots of a row of x, rounded up: quotients of slots are exact
  uint64_t per_cta;  // floor(2^64 / grid)
  uint32_t stage, codes_at, red, list, smem;  // bytes: of a stage, its codes' place, and where the others begin
};

inline MatvecPlan make_matvec_plan(const MatvecSizes& m) {
  auto ceil = [](int64_t a, int64_t b) { return (a + b - 1) / b; };
  auto least_of = [](int64_t a, int64_t b) { return a < b ? a : b; };
  MatvecPlan p = {};
  p.wide = m.wide;
  const int pieces = static_cast<int>(ceil(m.cin, kPieceK));
  p.passes = static_cast<int>(ceil(pieces, kMaxWarps));
  p.wk = static_cast<int>(ceil(pieces, p.passes));
  p.wr = static_cast<int>(least_of(kMaxWarps / p.wk, kStages));
  const int64_t entries = m.routed ? least_of(m.slots, m.groups) : 1;
  p.grid = static_cast<int>(least_of(m.sms, ceil(m.rows * entries, kMinRows)));
  p.per_row = (1u << 20) / static_cast<uint32_t>(m.per_row) + ((1u << 20) % static_cast<uint32_t>(m.per_row) != 0);
  p.per_cta = p.grid == 1 ? 0 : ~uint64_t{0} / static_cast<uint64_t>(p.grid);
  const int64_t all = ceil(ceil(m.rows * entries, p.grid) + 1, kTile);  // tiles of a CTA at most
  if (all < kFewTiles) p.wr = 1;
  if (p.passes == 1) {  // a tile's rows as they lie
    p.w_pitch = static_cast<int>(m.cin / 2);
    p.c_pitch = static_cast<int>(m.cin / LHCAL_BLOCK);
    p.codes_at = static_cast<uint32_t>(ceil(kTile * p.w_pitch + 16, 128) * 128);
    p.stage = p.codes_at + static_cast<uint32_t>(ceil(kTile * p.c_pitch + 32, 128) * 128);
  } else {
    // Row by row, with the 16-byte units around it; 64 bytes apart modulo 128, so that the 8 lanes
    // that read two rows together read 128 different bytes.
    p.w_pitch = static_cast<int>(ceil(p.wk * kPieceK / 2 + 16, 128)) * 128 + 64;
    p.c_pitch = p.wk * kPieceK / LHCAL_BLOCK + 16;
    p.codes_at = static_cast<uint32_t>(kTile * p.w_pitch);
    p.stage = p.codes_at + static_cast<uint32_t>(kTile * p.c_pitch);
  }
  const uint32_t lists = m.routed ? (5u * (m.slots < 64 ? 64 : (m.slots + 31) & ~31) + 1) * 4 : 0;
  // Sums: a tile of 8 slots of a warp at least, all rows of a CTA at most, twice. What they leave
  // of the memory goes to the stages.
  const int64_t least = kTile * kTokens;
  const int64_t fit = (kMaxSmem - kStaticSmem - static_cast<int64_t>(lists) - 3 * static_cast<int64_t>(p.stage)) / (2 * p.wk * 4) / least;
  const int64_t room = least_of(least_of(fit, 4), all);
  p.room = static_cast<int>((room > 1 ? room : 1) * least);
  const int64_t rest = kMaxSmem - kStaticSmem - static_cast<int64_t>(lists) - 2 * p.wk * p.room * 4;
  // A stage is always the same warps': stages are a multiple of wr. A wait for a stage goes by its parity, so it
  // is only right for a warp that has seen the lap before. With 7 stages and 2 warps, say, the warp of the even
  // tiles could be at tile 8 (stage 1, second lap) before tile 1 has come in: it would take that lap's parity for
  // its own, read what lies there and free the stage in the other warp's place.
  const int64_t most = least_of(ceil(kStages, p.wr) * p.wr, rest / p.stage), used = all * p.passes > 2 ? all * p.passes : 2;
  p.stages = static_cast<int>(least_of(most, used));
  if (p.wr > p.stages) p.wr = p.stages;
  p.stages -= p.stages % p.wr;
  p.red = static_cast<uint32_t>(p.stages) * p.stage;
  p.list = p.red + 2u * p.wk * p.room * 4;
  // The counts of the experts, two a word, lie below the lists until those are made. The lists hold 8-byte pairs.
  const uint32_t counts = (m.groups / 2u + 1) * 4;
  if (m.routed && p.list < counts) p.list = counts;
  p.list = (p.list + 15) & ~15u;
  p.smem = p.list + lists;
  return p;
}

}  // namespace lhcal
