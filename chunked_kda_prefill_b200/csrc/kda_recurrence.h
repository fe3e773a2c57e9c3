// kda_recurrence.h -- plan format of the gated recurrence (internal).
#pragma once

#include "kda_internal.h"

namespace kda {

// A plan is an int32 header followed by one record per tile.  A tile is kRecTileElems / D
// consecutive tokens of one sequence, for all heads (a work item is a tile and a head).  The first
// RH_CHAIN records are the tiles that hold valid tokens, ordered by their index within the
// sequence and then longest sequence first: every tile comes after its predecessor, and the tiles
// in flight at one time belong to as many sequences as possible.  The records after them are the
// tiles of pure padding, whose output rows are only zeroed.
constexpr int32_t kRecMagic = 0x4B524331;  // "KRC1"
constexpr int32_t kRecVersion = 1;
constexpr int kRecHeader = 16;
constexpr int kRecRecord = 8;
constexpr int kRecTileElems = 8192;
constexpr int rec_tile_rows(int D) { return kRecTileElems / D; }

enum RecHeader : int {
  RH_MAGIC = 0, RH_VERSION, RH_HEADER_WORDS, RH_RECORD_WORDS, RH_TILES, RH_CHAIN, RH_LAYOUT, RH_B,
  RH_N, RH_S, RH_D, RH_MAX_TILES, RH_TILE_ROWS, RH_RESERVED, RH_TABLE_HASH, RH_CHECKSUM
};
// RR_SLOT is the sequence, RR_ROW0 the tile's first token row within its slot (or in the packed
// rows), RR_VALID its tokens, RR_STORE its output rows (RR_VALID and the padding after it),
// RR_INDEX its place in the states and workspace arrays (consecutive within a sequence), RR_TILE
// its index within the sequence and RR_COUNT the sequence's tiles.
enum RecRecord : int {
  RR_SLOT = 0, RR_ROW0, RR_VALID, RR_STORE, RR_INDEX, RR_TILE, RR_COUNT, RR_RESERVED
};

kda_status_t validate_recurrence_shape(const kda_recurrence_shape_t* s);
// Checks a host plan's header (its own checksum, which covers a hash of the records) and, when
// s is given, that it was built for that shape.
kda_status_t validate_recurrence_plan(const int32_t* plan, size_t n,
                                      const kda_recurrence_shape_t* s);

}  // namespace kda
