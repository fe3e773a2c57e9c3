// kda_recurrence_plan.cpp -- host planner of the gated recurrence: which sequences are cut, and the
// segments, longest first.  Reads lengths only; never touches the GPU.
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

// Calls f(b, len) for every sequence of a well-formed problem.
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

long long tiles_of(long long rows, int R) { return (rows + R - 1) / R; }

struct Cut {
  long long most = 0;      // tiles of a segment, at the most; 0: no sequence is cut
  long long segments = 0;  // of all sequences
};

long long segments_of(long long tiles, long long most) {
  return most ? (tiles + most - 1) / most : 1;
}

// Whether the lengths are well formed and everything fits the kernels' 32-bit counters, and how the
// sequences are cut.
//
// Counted in tiles of a multiprocessor (about 0.16 us each), a pass takes as long, uncut, as its
// longest sequence, one tile after another, or as all tiles over the multiprocessors.  Cut, a segment
// costs 8 more for filling its ring, the maps 0.6 of all tiles and 25 for their launch, and the joins
// 0.3 for each segment before.  Of the cuts into segments for one to eight rounds over the
// multiprocessors the cheapest is taken.  The costs are those of bf16 sequences of equal length and
// stand for both passes and all types; the maps of sequences that stay whole are counted though none
// are formed, and uncut lengths are taken to fill all multiprocessors alike (a document of 16384
// tokens with fifty of 700 and 32 heads gives the fullest one 2928 tiles, with 1394 on average).
kda_status_t check_lengths(const kda_recurrence_shape_t& s, const int32_t* cu, Cut* cut) {
  const int R = rec_tile_rows(s.D);
  long long tiles = 0, longest = 0;
  const kda_status_t st = each_length(s, cu, [&](int, int32_t len) {
    tiles += tiles_of(len, R);
    longest = std::max(longest, tiles_of(len, R));
  });
  if (st != KDA_OK) return st;
  if (tiles > INT_MAX / 64) return KDA_ERR_SHAPE;
  *cut = Cut{0, s.B};
  const double all = (double)tiles * s.N / kRecSpread;
  double least = std::max(all, (double)longest);
  for (int rounds = 1; rounds <= 8; ++rounds) {
    // the smallest segments of which every multiprocessor has `rounds`
    const long long room = (long long)kRecSpread * rounds / s.N;
    if (room < s.B) continue;
    long long lo = 1, hi = longest, count = 0;
    auto segments = [&](long long most) {
      long long n = 0;
      each_length(s, cu, [&](int, int32_t len) { n += segments_of(tiles_of(len, R), most); });
      return n;
    };
    while (lo < hi) {
      const long long mid = (lo + hi) / 2;
      if (segments(mid) <= room) hi = mid;
      else lo = mid + 1;
    }
    count = segments(lo);
    const double cost = rounds * (lo + 8.0 + 0.3 * segments_of(longest, lo)) + 0.6 * all + 25;
    if (count > s.B && cost < least) {
      least = cost;
      *cut = Cut{lo, count};
    }
  }
  return KDA_OK;
}

size_t plan_words(const Cut& cut) { return (size_t)kRecHeader + (size_t)cut.segments * kRecRecord; }

kda_status_t build(const kda_recurrence_shape_t& s, const int32_t* cu, int32_t* plan, size_t n) {
  Cut cut;
  kda_status_t st = check_lengths(s, cu, &cut);
  if (st != KDA_OK) return st;
  if (n < plan_words(cut)) return KDA_ERR_PLAN;
  const int R = rec_tile_rows(s.D);
  const bool tnd = s.layout == KDA_LAYOUT_TND;
  struct Segment { int32_t b, start, len, index, count, map; };
  std::vector<Segment> segs;
  segs.reserve(cut.segments);
  long long maps = 0;
  bool padded = false;
  each_length(s, cu, [&](int b, int32_t len) {
    const long long tiles = tiles_of(len, R), count = segments_of(tiles, cut.most);
    for (long long k = 0; k < count; ++k) {
      const long long lo = tiles * k / count * R, hi = std::min((long long)len, tiles * (k + 1) / count * R);
      segs.push_back({b, (int32_t)((tnd ? cu[b] : 0) + lo), (int32_t)(hi - lo), (int32_t)k,
                      (int32_t)count, (int32_t)maps});
    }
    if (count > 1) maps += count;
    padded |= !tnd && len < s.S;
  });
  std::stable_sort(segs.begin(), segs.end(),
                   [](const Segment& a, const Segment& d) { return a.len > d.len; });
  // Many short segments: a warp each, if the longest one is no more than a warp's share of all tiles
  // (else warps would stand idle behind it).  Against a ring for each, 16 heads, bf16, 65536 tokens
  // forward, in documents of an eighth of that border 156 us against 190, a quarter 159 (175), half
  // 144 (166), 0.9 of it 196 (158), 1.1 of it 148 (157), twice 197 (149), four times 324 (147):
  // near the border it is the number of units over all warps that decides, which the rule leaves out.
  long long all = 0;
  for (const Segment& q : segs) all += tiles_of(q.len, R);
  const bool solo = tiles_of(segs[0].len, R) * kRecSpread * kRecRing <= all * s.N;
  std::memset(plan, 0, kRecHeader * sizeof(int32_t));
  int32_t* rec = plan + kRecHeader;
  long long tile = 0, part = 0;
  for (const Segment& q : segs) {
    const long long tiles = tiles_of(q.len, R);
    rec[RR_SLOT] = q.b;
    rec[RR_START] = q.start;
    rec[RR_LEN] = q.len;
    rec[RR_TILE] = (int32_t)tile;
    rec[RR_PART] = (int32_t)part;
    rec[RR_SEGMENT] = q.index;
    rec[RR_SEGMENTS] = q.count;
    rec[RR_MAP] = q.map;
    rec += kRecRecord;
    tile += tiles;
    part += std::min<long long>(tiles, solo ? 1 : kRecRing);
  }
  plan[RH_MAGIC] = kRecMagic;
  plan[RH_VERSION] = kRecVersion;
  plan[RH_HEADER_WORDS] = kRecHeader;
  plan[RH_RECORD_WORDS] = kRecRecord;
  plan[RH_LAYOUT] = s.layout;
  plan[RH_B] = s.B;
  plan[RH_N] = s.N;
  plan[RH_S] = s.S;
  plan[RH_D] = s.D;
  plan[RH_TILE_ROWS] = R;
  plan[RH_TILES] = (int32_t)tile;
  plan[RH_RECORDS] = (int32_t)segs.size();
  plan[RH_MAPS] = (int32_t)maps;
  plan[RH_PARTS] = (int32_t)part;
  plan[RH_LONGEST] = (int32_t)tiles_of(segs[0].len, R);
  plan[RH_PADDED] = padded;
  plan[RH_SOLO] = solo;
  plan[RH_TABLE_HASH] = (int32_t)(fnv(plan + kRecHeader, segs.size() * kRecRecord) & 0x7fffffff);
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
  if (p[RH_RECORDS] < 1 || n < (size_t)kRecHeader + (size_t)p[RH_RECORDS] * kRecRecord)
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
  Cut cut;
  st = check_lengths(*shape, cu, &cut);
  if (st != KDA_OK) return st;
  *n_int32 = plan_words(cut);
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
