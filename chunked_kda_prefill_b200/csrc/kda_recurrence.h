// kda_recurrence.h -- plan format of the gated recurrence (internal).
#pragma once

#include "kda_internal.h"

namespace kda {

// A plan is an int32 header followed by one record per sequence, longest first.  A tile is
// kRecTileElems / D consecutive tokens of one (sequence, head); a cluster of blocks walks one
// (sequence, head) at a time, a tile per block and step.
constexpr int32_t kRecMagic = 0x4B524331;  // "KRC1"
constexpr int32_t kRecVersion = 1;
constexpr int kRecHeader = 24;
constexpr int kRecRecord = 4;
constexpr int kRecTileElems = 8192;
constexpr int rec_tile_rows(int D) { return kRecTileElems / D; }
// Cluster sizes that a launch chooses from: 1, 2, 4, 8.
constexpr int kRecClusters = 4;

// RH_CHAIN is the number of tiles with tokens, RH_MAX_TILES that of the sequence with most tiles
// (padding rows included), RH_STEPS + c the steps of one head of every sequence on clusters of 2^c.
enum RecHeader : int {
  RH_MAGIC = 0, RH_VERSION, RH_HEADER_WORDS, RH_RECORD_WORDS, RH_LAYOUT, RH_B, RH_N, RH_S, RH_D,
  RH_TILE_ROWS, RH_CHAIN, RH_MAX_TILES, RH_STEPS, RH_TABLE_HASH = RH_STEPS + kRecClusters,
  RH_CHECKSUM = kRecHeader - 1
};
// RR_SLOT is the sequence, RR_START its first token within its slot (or in the packed rows),
// RR_LEN its tokens and RR_BASE the place of its first tile in the states.
enum RecRecord : int { RR_SLOT = 0, RR_START, RR_LEN, RR_BASE };

kda_status_t validate_recurrence_shape(const kda_recurrence_shape_t* s);
// Checks a host plan's header (its own checksum, which covers a hash of the records) and, when
// s is given, that it was built for that shape.
kda_status_t validate_recurrence_plan(const int32_t* plan, size_t n,
                                      const kda_recurrence_shape_t* s);

}  // namespace kda
