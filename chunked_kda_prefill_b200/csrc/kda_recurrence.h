// kda_recurrence.h -- plan format of the gated recurrence (internal).
#pragma once

#include "kda_internal.h"

namespace kda {

// A plan is an int32 header followed by one record per segment, longest first.  A segment is a
// sequence, or one of the equal parts of a long one; a tile is kRecTileElems / D consecutive tokens
// of a segment in one head.
constexpr int32_t kRecMagic = 0x4B524331;  // "KRC1"
constexpr int32_t kRecVersion = 2;
constexpr int kRecHeader = 24;
constexpr int kRecRecord = 8;
constexpr int kRecTileElems = 1024;
constexpr int rec_tile_rows(int D) { return kRecTileElems / D; }
constexpr int kRecRing = 16;     // warps that walk a segment together, at the most
constexpr int kRecSpread = 148;  // multiprocessors that a plan spreads long sequences over

// RH_TILES is the number of tiles in one head, RH_MAPS the rows of maps that the segments of cut
// sequences need (0: none is cut), RH_PARTS the rows of the parameters' partial gradients,
// RH_LONGEST the tiles of the longest segment, RH_PADDED whether rows lie behind a sequence's tokens,
// RH_SOLO whether a segment is a single warp's.
enum RecHeader : int {
  RH_MAGIC = 0, RH_VERSION, RH_HEADER_WORDS, RH_RECORD_WORDS, RH_LAYOUT, RH_B, RH_N, RH_S, RH_D,
  RH_TILE_ROWS, RH_TILES, RH_RECORDS, RH_MAPS, RH_PARTS, RH_LONGEST, RH_PADDED, RH_TABLE_HASH, RH_SOLO,
  RH_CHECKSUM = kRecHeader - 1
};
// RR_SLOT is the sequence, RR_START the segment's first token within its slot (or in the packed
// rows), RR_LEN its tokens, RR_TILE its first tile, RR_PART its first row of partial gradients (it
// has one for each of its tiles, kRecRing at the most, or a single one for a single warp), RR_SEGMENT its place among the RR_SEGMENTS
// of its sequence and RR_MAP the sequence's first row of maps.
enum RecRecord : int {
  RR_SLOT = 0, RR_START, RR_LEN, RR_TILE, RR_PART, RR_SEGMENT, RR_SEGMENTS, RR_MAP
};

kda_status_t validate_recurrence_shape(const kda_recurrence_shape_t* s);
// Checks a host plan's header (its own checksum, which covers a hash of the records) and, when
// s is given, that it was built for that shape.
kda_status_t validate_recurrence_plan(const int32_t* plan, size_t n,
                                      const kda_recurrence_shape_t* s);

}  // namespace kda
