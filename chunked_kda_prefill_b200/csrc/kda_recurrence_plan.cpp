// kda_recurrence_plan.cpp -- host planner of the gated recurrence: the tiles of every sequence in
// an order that any work item's predecessors precede.  Reads lengths only; never touches the GPU.
#include <algorithm>
#include <climits>
#include <cstring>
#include <new>
#include <vector>

#include "kda_recurrence.h"

namespace kda {

kda_status_t validate_recurrence_shape(const kda_recurrence_shape_t* s) {
  if (!s) return KDA_ERR_NULL;
  if (s->layout < KDA_LAYOUT_BNSD || s->layout > KDA_LAYOUT_TND) return KDA_ERR_LAYOUT;
  if (s->D != 128 && s->D != 64) return KDA_ERR_DIM;
  if (s->dtype < KDA_BF16 || s->dtype > KDA_FP32) return KDA_ERR_DTYPE;
  if (s->B < 1 || s->S < 1) return KDA_ERR_SHAPE;
  if (s->N < 1) return KDA_ERR_HEADS;
  const long long rows = s->layout == KDA_LAYOUT_TND ? (long long)s->S : (long long)s->B * s->S;
  if ((long long)s->B * s->N > INT_MAX / 2) return KDA_ERR_SHAPE;
  // rows <= 2^62 and N < 2^31 need a division, not a product, to compare without overflow
  if (rows > (1LL << 46) / s->D / s->N) return KDA_ERR_SHAPE;
  return KDA_OK;
}

namespace {

uint32_t fnv(const int32_t* w, size_t n, uint32_t h = 2166136261u) {
  for (size_t i = 0; i < n; ++i) h = (h ^ (uint32_t)w[i]) * 16777619u;
  return h;
}

// Tile counts of a problem: records in all, and those with valid tokens.  Calls f(b, len) for
// every sequence.
template <class F>
kda_status_t each_length(const kda_recurrence_shape_t& s, const int32_t* cu, F&& f) {
  const bool tnd = s.layout == KDA_LAYOUT_TND;
  if (tnd && !cu) return KDA_ERR_SEQLENS;
  if (cu && (cu[0] != 0 || (tnd && cu[s.B] != s.S))) return KDA_ERR_SEQLENS;
  for (int b = 0; b < s.B; ++b) {
    const long long len = cu ? (long long)cu[b + 1] - cu[b] : s.S;
    if (len < 1 || len > s.S) return KDA_ERR_SEQLENS;
    f(b, (int32_t)len);
  }
  return KDA_OK;
}

struct Counts {
  long long tiles = 0, chain = 0;
};

kda_status_t count_tiles(const kda_recurrence_shape_t& s, const int32_t* cu, Counts* c) {
  const int R = rec_tile_rows(s.D);
  const long long slot_tiles = ((long long)s.S + R - 1) / R;
  const kda_status_t st = each_length(s, cu, [&](int, int32_t len) {
    const long long n = ((long long)len + R - 1) / R;
    c->chain += n;
    c->tiles += s.layout == KDA_LAYOUT_TND ? n : slot_tiles;
  });
  if (st != KDA_OK) return st;
  // a launch has one block per (tile, head)
  if (c->tiles > INT_MAX / kRecRecord - kRecHeader || c->tiles * s.N > INT_MAX) return KDA_ERR_SHAPE;
  return KDA_OK;
}

kda_status_t build(const kda_recurrence_shape_t& s, const int32_t* cu, int32_t* plan, size_t n) {
  Counts c;
  kda_status_t st = count_tiles(s, cu, &c);
  if (st != KDA_OK) return st;
  if (n < (size_t)kRecHeader + (size_t)c.tiles * kRecRecord) return KDA_ERR_PLAN;

  const int R = rec_tile_rows(s.D);
  struct Seq { int32_t b, start, len, tiles, base; };
  std::vector<Seq> seqs;
  seqs.reserve(s.B);
  each_length(s, cu, [&](int b, int32_t len) {
    const int32_t start = s.layout == KDA_LAYOUT_TND ? cu[b] : 0;
    seqs.push_back({b, start, len, (int32_t)(((long long)len + R - 1) / R), 0});
  });
  std::stable_sort(seqs.begin(), seqs.end(),
                   [](const Seq& a, const Seq& d) { return a.tiles > d.tiles; });
  int32_t base = 0;
  for (Seq& q : seqs) {
    q.base = base;
    base += q.tiles;
  }

  int32_t* rec = plan + kRecHeader;
  auto put = [&](const Seq& q, int32_t j, int32_t valid, int32_t store, int32_t index) {
    rec[RR_SLOT] = q.b;
    rec[RR_ROW0] = q.start + j * R;
    rec[RR_VALID] = valid;
    rec[RR_STORE] = store;
    rec[RR_INDEX] = index;
    rec[RR_TILE] = j;
    rec[RR_COUNT] = q.tiles;
    rec[RR_RESERVED] = 0;
    rec += kRecRecord;
  };
  const bool tnd = s.layout == KDA_LAYOUT_TND;
  for (int32_t j = 0; j < seqs.front().tiles; ++j)
    for (const Seq& q : seqs) {
      if (q.tiles <= j) break;  // the rest are shorter
      const int32_t valid = std::min(R, q.len - j * R);
      put(q, j, valid, tnd ? valid : std::min(R, s.S - j * R), q.base + j);
    }
  if (!tnd) {
    const int32_t slot_tiles = (int32_t)(((long long)s.S + R - 1) / R);
    for (const Seq& q : seqs)
      for (int32_t j = q.tiles; j < slot_tiles; ++j) put(q, j, 0, std::min(R, s.S - j * R), 0);
  }

  std::memset(plan, 0, kRecHeader * sizeof(int32_t));
  plan[RH_MAGIC] = kRecMagic;
  plan[RH_VERSION] = kRecVersion;
  plan[RH_HEADER_WORDS] = kRecHeader;
  plan[RH_RECORD_WORDS] = kRecRecord;
  plan[RH_TILES] = (int32_t)c.tiles;
  plan[RH_CHAIN] = (int32_t)c.chain;
  plan[RH_LAYOUT] = s.layout;
  plan[RH_B] = s.B;
  plan[RH_N] = s.N;
  plan[RH_S] = s.S;
  plan[RH_D] = s.D;
  plan[RH_MAX_TILES] = seqs.front().tiles;
  plan[RH_TILE_ROWS] = R;
  plan[RH_TABLE_HASH] = (int32_t)(fnv(plan + kRecHeader, (size_t)c.tiles * kRecRecord) & 0x7fffffff);
  plan[RH_CHECKSUM] = (int32_t)(fnv(plan, RH_CHECKSUM) & 0x7fffffff);
  return KDA_OK;
}

}  // namespace

kda_status_t validate_recurrence_plan(const int32_t* p, size_t n, const kda_recurrence_shape_t* s) {
  if (!p) return KDA_ERR_NULL;
  if (n < (size_t)kRecHeader) return KDA_ERR_PLAN;
  if (p[RH_MAGIC] != kRecMagic || p[RH_VERSION] != kRecVersion ||
      p[RH_HEADER_WORDS] != kRecHeader || p[RH_RECORD_WORDS] != kRecRecord)
    return KDA_ERR_PLAN;
  if ((int32_t)(fnv(p, RH_CHECKSUM) & 0x7fffffff) != p[RH_CHECKSUM]) return KDA_ERR_PLAN;
  if (p[RH_TILES] < 1 || n < (size_t)kRecHeader + (size_t)p[RH_TILES] * kRecRecord)
    return KDA_ERR_PLAN;
  if (s && (p[RH_LAYOUT] != s->layout || p[RH_B] != s->B || p[RH_N] != s->N || p[RH_S] != s->S ||
            p[RH_D] != s->D))
    return KDA_ERR_PLAN;
  return KDA_OK;
}

}  // namespace kda

using namespace kda;

extern "C" kda_status_t kda_recurrence_plan_size(const kda_recurrence_shape_t* shape,
                                                 const int32_t* cu, size_t* n_int32) {
  if (!n_int32) return KDA_ERR_NULL;
  kda_status_t st = validate_recurrence_shape(shape);
  if (st != KDA_OK) return st;
  Counts c;
  st = count_tiles(*shape, cu, &c);
  if (st != KDA_OK) return st;
  *n_int32 = (size_t)kRecHeader + (size_t)c.tiles * kRecRecord;
  return KDA_OK;
}

extern "C" kda_status_t kda_recurrence_plan(const kda_recurrence_shape_t* shape,
                                            const int32_t* cu, int32_t* plan, size_t n_int32) {
  const kda_status_t st = validate_recurrence_shape(shape);
  if (st != KDA_OK) return st;
  if (!plan) return KDA_ERR_NULL;
  try {
    return build(*shape, cu, plan, n_int32);
  } catch (const std::bad_alloc&) {
    return KDA_ERR_SHAPE;
  }
}
