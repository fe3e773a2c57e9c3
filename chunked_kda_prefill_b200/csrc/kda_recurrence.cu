// kda_recurrence.cu -- the gated recurrence, the vector form of the KDA state:
//     a_t = exp(lb sigmoid(e^A (g_t + bias))),  h_t = a_t h_{t-1} + sigmoid(beta_t) x_t.
//
// A ring of warps, a block's (a single warp where segments are many and short), walks one segment (a sequence, or a part of a long one) of one head, a
// tile of 1024 values a warp at a time: the warp's own copies bring its next tiles to shared memory, it
// forms all decays and writes of its tile and what the tile makes of a state of zero, waits for the
// state that the warp before it leaves, passes on the state after the tile (one multiply-add) and only
// then finishes its results.  So what happens one after another is a hand-over of about 120 ns for
// 1024 values, the rest runs side by side, and no barrier stops a block.  The backward pass is the
// same walk from the end with the state's gradient, the states before the tiles given.
//
// Where a few long sequences would leave multiprocessors idle, the plan cuts them.  A kernel before
// the walk then forms the map h -> A h + H of each segment, and a segment starts from the maps
// before it.  Three heads of 8192 tokens take 128 us whole and 14 us in 49 segments each.
//
// The bound is HBM: 6 bytes a value forward (16-bit; 6.5 with the states of a training step), 10.5
// backward.  Each kernel says how near it comes.
#include <cuda_runtime.h>

#include <algorithm>
#include <climits>
#include <cmath>
#include <cstdint>
#include <type_traits>

#include "kda_args.h"
#include "kda_io.cuh"
#include "kda_once.h"
#include "kda_recurrence.h"

namespace kda {
namespace {

struct RecParams {
  kda_view_t x, g, beta, dout;  // device addresses and strides
  const int32_t* plan;
  int32_t checksum;
  int32_t N, units;   // units: segments times heads
  int32_t slot_rows;  // rows that a slot's outputs have; 0 where none lies behind a sequence's tokens
  bool spread;        // all blocks write the zeros behind every sequence, not just their units'
  const float* begin;  // [B][N][D] the walk's start (forward h0, backward dfinal), or null for zeros
  const float* A_log;
  const float* dt_bias;
  float lower_bound;
  int32_t* status;  // or null
  float* maps;    // [RH_MAPS][N][2][D] of the cut sequences
  float* states;  // [tiles][N][D] the states before the tiles: forward writes, backward reads
  void* out;      // forward: out; backward: dx
  void* dg;
  void* dbeta;
  float* end;        // [B][N][D] the walk's end: final_state, or dh0 (null: not wanted)
  float* part_bias;  // [RH_PARTS][N][D]
  float* part_A;     // [RH_PARTS][N]
  kda_view_t od, bd;  // strides of the dense outputs with and without channels
  // bytes from a copy's rows to the next copy's, and from a warp's tile to its next one, of g, x, dout
  // and (tiles only) beta
  long long copy_step[3], tile_step[4];
};

template <class T>
__device__ __forceinline__ const T* at(const kda_view_t& v, long long b, long long n, long long s) {
  return static_cast<const T*>(v.data) + b * v.stride_b + n * v.stride_n + s * v.stride_s;
}

// A lane's channels and a tile's tokens.
template <int D>
struct Shape {
  static constexpr int V = D / 32;          // channels of a lane
  static constexpr int K = kRecTileElems / D;  // tokens of a tile
  using F = Pairs<V / 2>;
};

// The warps of a block, one block a multiprocessor, are a ring: as many as the registers allow (128 a
// thread forward, 168 backward; fp32's tiles are twice as large).  A warp has the copies of kStages tiles under way or at work, as many as shared memory holds.
template <class T, bool BACKWARD>
struct Block {
  static constexpr int kWarps = sizeof(T) == 4 ? 8 : BACKWARD ? 12 : 16;
  static constexpr int kStages = BACKWARD ? 2 : 3;
  static constexpr int kTensors = BACKWARD ? 3 : 2;
};
template <class T, int D, bool BACKWARD>
constexpr int kStageBytes =
    Block<T, BACKWARD>::kTensors * kRecTileElems * (int)sizeof(T) + (BACKWARD ? D * 4 : 0);
template <class T, int D, bool BACKWARD>
constexpr int kWalkSmem =
    Block<T, BACKWARD>::kWarps * Block<T, BACKWARD>::kStages * kStageBytes<T, D, BACKWARD>;

// What a warp keeps of a tile from the start of its copies on: the lane's write logit, and the number
// of tokens (0: no tile is left) with flags.
struct Ahead {
  float logit;
  int info;
};
enum : int {
  kTokens = 31,
  kFresh = 32,    // the warp's first tile in the unit
  kFirst = 64,    // the segment's first tile of the walk
  kLast = 128,    // the segment's last tile of the walk
  kEnd = 256,     // of the segment that the walk of the sequence ends with
  kCut = 512,     // of a cut sequence
  kStop = 1024    // the ring's last tile
};
// The same of a unit, with its first tile: `row` of its first token, `place` of its state, `order` of
// the segment in the walk of its sequence.
struct __align__(16) Entry {
  int slot, row, n, place;
  int map, part, order;
  int parts;  // rows of partial gradients that the unit has behind the warp's own
};

// Whether the plan on the device is the host's; block 0 leaves the status.
__device__ __forceinline__ bool same_plan(const RecParams& p) {
  const bool same = p.plan[RH_CHECKSUM] == p.checksum;
  if (blockIdx.x == 0 && threadIdx.x == 0 && p.status) *p.status = same ? DS_OK : DS_PLAN;
  return same;
}

__device__ __forceinline__ const int4* record(const RecParams& p, int i) {
  return reinterpret_cast<const int4*>(p.plan + kRecHeader) + 2 * i;
}

// 16 bytes from global to shared memory
__device__ __forceinline__ void copy16(uint32_t to, const void* from) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to), "l"(from) : "memory");
}
// A warp's way through the tiles of its block's (or its own) units, and the copies of the next one.
// The units are dealt to the blocks in rounds, every other one in reverse, so that with the plan's
// order (longest first) no block gets the longer unit of every round.
template <class T, int D, bool BACKWARD, bool SOLO>
struct Walk {
  using B = Block<T, BACKWARD>;
  static constexpr int K = Shape<D>::K, W = B::kWarps, kRow = D * (int)sizeof(T);
  static constexpr int kRing = SOLO ? 1 : W;  // warps that walk a unit
  static constexpr int kLanes = kRow / 16;    // lanes of a row's copy
  static constexpr int kRows = 32 / kLanes;   // rows of a copy
  int slot, start, len, tile0;        // the record
  int part, segment, segments, map;
  int n, t, tiles, round;
  int place, places;                  // the warp's, or its block's, among those that units go to
  bool fresh, done;
  const char *g, *x, *dout, *beta, *state;  // the lane's, of the next tile
  int4 r0, r1;

  // The first record is on its way while the plan is checked.
  __device__ Walk(const RecParams& p) {
    const int warp = threadIdx.x >> 5;
    places = SOLO ? gridDim.x * W : gridDim.x;
    place = SOLO ? blockIdx.x + warp * gridDim.x : blockIdx.x;
    round = 0;
    fetch(p);
  }

  __device__ long long unit_of(int round) const {
    return (long long)round * places + (round & 1 ? places - 1 - place : place);
  }
  // the lane's part of a tile's first copy
  __device__ const char* lane_rows(const kda_view_t& v, int row) const {
    const int lane = threadIdx.x & 31;
    return reinterpret_cast<const char*>(at<T>(v, slot, n, row + lane / kLanes)) +
           lane % kLanes * 16;
  }
  // The record of the round's unit.
  __device__ void fetch(const RecParams& p) {
    const long long unit = unit_of(round);
    done = unit >= p.units;
    if (done) return;
    const int i = (int)unit / p.N;
    n = (int)unit - i * p.N;
    r0 = __ldg(record(p, i));
    r1 = __ldg(record(p, i) + 1);
  }
  // zero(slot, n, row, end, warps, warp): writes the rows behind a sequence's last token, a share of them
  template <bool FIRST = false, class Zero>
  __device__ void enter(const RecParams& p, Zero&& zero) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    for (bool fetched = FIRST;; ++round) {
      if (!fetched) fetch(p);
      fetched = false;
      if (done) return;
      slot = r0.x; start = r0.y; len = r0.z; tile0 = r0.w;
      part = r1.x; segment = r1.y; segments = r1.z; map = r1.w;
      tiles = (len + K - 1) / K;
      if (p.slot_rows && !p.spread && segment + 1 == segments)
        zero(slot, n, start + len, p.slot_rows, kRing, SOLO ? 0 : warp);
      if (t < tiles) break;
      t -= tiles;
    }
    fresh = true;
    const int k = BACKWARD ? tiles - 1 - t : t, row = start + k * K;
    g = lane_rows(p.g, row);
    x = lane_rows(p.x, row);
    beta = reinterpret_cast<const char*>(at<T>(p.beta, slot, n, row + lane));
    if (BACKWARD) {
      if (p.dout.data) dout = lane_rows(p.dout, row);
      state = reinterpret_cast<const char*>(p.states + ((size_t)(tile0 + k) * p.N + n) * D) + lane * 16;
    }
  }
  // The rows behind all sequences, over all warps of the grid (there are fewer units than
  // multiprocessors); the records are read 32 at a time.
  template <class Zero>
  __device__ void zero_all(const RecParams& p, Zero&& zero) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, records = p.units / p.N;
    for (int base = 0; base < records; base += 32) {
      int at = 0, row = p.slot_rows;
      if (base + lane < records) {
        const int4 r0 = __ldg(record(p, base + lane)), r1 = __ldg(record(p, base + lane) + 1);
        at = r0.x;
        if (r1.y + 1 == r1.z) row = r0.y + r0.z;
      }
      for (unsigned left = __ballot_sync(0xffffffffu, row < p.slot_rows); left; left &= left - 1) {
        const int from = __ffs(left) - 1;
        const int s = __shfl_sync(0xffffffffu, at, from), r = __shfl_sync(0xffffffffu, row, from);
        const unsigned rows = p.slot_rows - r, step = W * gridDim.x;
        if (rows >= step) {
          for (int h = 0; h < p.N; ++h)
            zero(s, h, r, p.slot_rows, step, warp * gridDim.x + blockIdx.x);
          continue;
        }
        // fewer rows than warps: all heads' rows one after another
        const unsigned step_heads = step / rows, step_rows = step - step_heads * rows;
        unsigned k = warp * gridDim.x + blockIdx.x, h = k / rows;
        k -= h * rows;
        while (h < (unsigned)p.N) {
          zero(s, (int)h, r + (int)k, r + (int)k + 1, 1, 0);
          h += step_heads;
          k += step_rows;
          if (k >= rows) {
            k -= rows;
            ++h;
          }
        }
      }
    }
  }
  template <class Zero>
  __device__ void begin(const RecParams& p, int warp, Zero&& zero) {
    dout = state = nullptr;
    t = SOLO ? 0 : warp;
    enter<true>(p, zero);
  }
  template <class Zero>
  __device__ void next(const RecParams& p, Zero&& zero) {
    fresh = false;
    t += kRing;
    if (t < tiles) {
      g += p.tile_step[0];
      x += p.tile_step[1];
      beta += p.tile_step[3];
      if (BACKWARD) {
        dout += p.tile_step[2];
        state -= (size_t)kRing * p.N * D * 4;
      }
      return;
    }
    t -= tiles;
    ++round;
    enter(p, zero);
  }
  // (a branch for whole tiles, without the comparisons, was 10 % slower in both passes)
  __device__ static void copy_rows(uint32_t to, const char* from, long long step, int valid) {
    const int lane = threadIdx.x & 31;
    to += lane * 16;
#pragma unroll
    for (int k = 0; k < K; k += kRows) {
      if (valid == K || k + lane / kLanes < valid) copy16(to + k * kRow, from);
      from += step;
    }
  }
  // Starts the copies of the next tile to `stage`.
  template <class Zero>
  __device__ Ahead issue(const RecParams& p, uint32_t stage, Entry* entry, Zero&& zero) {
    const int lane = threadIdx.x & 31;
    __syncwarp();  // all lanes have read what the stage held
    Ahead ahead{0.f, 0};
    if (!done) {
      int valid = K;
      ahead.info = K;
      if (fresh || t == tiles - 1) {
        const int k = BACKWARD ? tiles - 1 - t : t;
        const int order = BACKWARD ? segments - 1 - segment : segment;
        const bool last = t == tiles - 1;
        valid = min(K, len - k * K);
        ahead.info = valid | (fresh ? kFresh : 0) | (t == 0 ? kFirst : 0) | (last ? kLast : 0) |
                     (order == segments - 1 ? kEnd : 0) | (segments > 1 ? kCut : 0) |
                     (last && unit_of(round + 1) >= p.units ? kStop : 0);
        if (fresh && lane == 0) {
          int4* const to = reinterpret_cast<int4*>(entry);
          to[0] = make_int4(slot, start + k * K, n, tile0 + k);
          to[1] = make_int4(map, part + t, order, min(SOLO ? 1 : kRecRing, tiles) - t);
        }
      }
      copy_rows(stage, g, p.copy_step[0], valid);
      copy_rows(stage + K * kRow, x, p.copy_step[1], valid);
      if (BACKWARD) {
        if (p.dout.data) copy_rows(stage + 2 * K * kRow, dout, p.copy_step[2], valid);
        if (lane < D / 4) copy16(stage + 3 * K * kRow + lane * 16, state);
      }
      if (lane < valid) ahead.logit = to_f32(__ldg(reinterpret_cast<const T*>(beta)));
      next(p, zero);
    }
    copies_issued();
    return ahead;
  }
};

// The state that a cut segment starts from: the maps of those before it in the walk's order, the
// first of which is constant.
template <int D>
__device__ __noinline__ Pairs<D / 64> join(const RecParams& p, int map, int order, int n, int chan) {
  constexpr int P = D / 64;
  using F = Pairs<P>;
  F s = splat<P>(0.f);
  wait_dependencies();
  const float* m = p.maps + ((size_t)map * p.N + n) * 2 * D + chan;
  const size_t row = (size_t)p.N * 2 * D;
  constexpr int kAhead = 16;  // loads under way at a time
  for (int k = 0; k <= order; k += kAhead) {
    F a[kAhead], h[kAhead];
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      const float* const from = m + min(k + i, order) * row;
      a[i] = load<P>(from);
      h[i] = load<P>(from + D);
    }
#pragma unroll
    for (int i = 0; i < kAhead; ++i)
      if (k + i <= order) s = fma(a[i], s, h[i]);
  }
  return s;
}

// A warp's place in its block's ring: the state is handed on through shared memory, with a barrier of
// the two warps that only the later one waits at.  (One warp more that runs through maps which the
// others post took 220 ns a tile, a wait at an mbarrier and two accesses to shared memory.)
template <int W, int D, bool SOLO>
struct Ring {
  float *inbox, *outbox;  // the state handed to this warp, and to the next one (its own, of one warp)
  int warp;
  __device__ explicit Ring(int w) : warp(w) {
    __shared__ __align__(16) float box[W][D];
    inbox = box[warp];
    outbox = box[SOLO ? warp : (warp + 1) % W];
  }
  __device__ void wait() const {
    if (SOLO) __syncwarp();  // keeps what is before and after apart; without it registers spill
    else named_bar_sync(warp, 64);
  }
  __device__ void pass() const {
    if (SOLO) __syncwarp();
    else named_bar_arrive((warp + 1) % W, 64);
  }
};

// The rows of a partial tile that hold no token become closed gates (decay one) and zero writes.  Where
// a broken factor or a bias that is no number would open them again, the rows with tokens take it in
// and the tile is computed without: g + inf as a row, and then + 0.  (Decays that are set to one after
// the gates cost 8 % of a training step with many partial tiles of 64 channels, this 2 %; picking the
// end state from the tile's last token instead keeps all its states alive: twice the time.)
template <int P>
struct TileGate {
  Pairs<P> bias;
  float nz;
};
template <class T, int D, int TENSORS>
__device__ __noinline__ TileGate<D / 64> fill_rows(T* stage, int valid, TileGate<D / 64> gate) {
  using S = Shape<D>;
  constexpr int P = S::V / 2;
  stage += (threadIdx.x & 31) * S::V;
  for (int k = valid; k < S::K; ++k)
    for (int i = 0; i < TENSORS; ++i)
      store(stage + i * kRecTileElems + k * D, splat<P>(i == 0 ? -INFINITY : 0.f));
  // zero, or NaN where the factor or the bias is not a number, or the infinite bias
  const float broken = gate.nz == gate.nz ? 0.f : gate.nz;
  const Pairs<P> extra = each(gate.bias, [=](float b) { return (fabsf(b) < INFINITY ? 0.f : b) + broken; });
  bool any = false;
  for (int i = 0; i < P; ++i) any |= extra.v[i].x != 0.f || extra.v[i].y != 0.f;
  if (!any) return gate;
  for (int k = 0; k < valid; ++k) store(stage + k * D, load<P>(stage + k * D) + extra);
  gate.bias = each(gate.bias, [](float b) { return fabsf(b) < INFINITY ? b : 0.f; });
  if (broken != 0.f) gate.nz = -1.f;
  return gate;
}

// Stores a tile's rows; `next` is the distance of two rows.
template <class T, int D, int K, int P>
__device__ __forceinline__ void store_rows(T* to, long long next, int valid, const Pairs<P> (&v)[K]) {
  if (valid == K && next == D) {
#pragma unroll
    for (int k = 0; k < K; ++k) store(to + k * D, v[k]);
  } else {
#pragma unroll
    for (int k = 0; k < K; ++k) {
      if (k < valid) store(to, v[k]);
      to += next;
    }
  }
}

// 4x32x16384 bf16: 295 us, 5.5 TB/s of the 6.47 that a copy reaches (6.2 TB/s where 148 units keep
// every multiprocessor busy).  What else is busy: 65 % of the special-function unit, three results a
// value.  Sharing one reciprocal between two values (289 us against 292) is not worth its second path
// for products that overflow; 12 warps took 305 us, a stage fewer 325 us.
// The gate's powers and its reciprocal are the approximate instructions (off by 2^-22 and by one unit in
// the last place; values below the normal range become zero): 16-bit results do not hold the rest, fp32
// ones come out with 0.4 to 2 times the error of separate fp32 operations.
template <class T, int D, bool SOLO>
__global__ void __launch_bounds__(32 * Block<T, false>::kWarps, 1)
    rec_forward_kernel(const __grid_constant__ RecParams p) {
  using B = Block<T, false>;
  using S = Shape<D>;
  using F = typename S::F;
  constexpr int K = S::K, V = S::V, P = V / 2, kStages = B::kStages, W = B::kWarps;
  constexpr int kRing = SOLO ? 1 : W;
  constexpr int kStage = kStageBytes<T, D, false>;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ Entry entries[W][kStages];
  __shared__ float2 writes[W][K];  // b and b
  Walk<T, D, false, SOLO> walk(p);
  if (!same_plan(p)) return;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, chan = lane * V;
  const Ring<W, D, SOLO> ring(warp);
  uint8_t* const stages = smem + warp * kStages * kStage;
  T* const out = static_cast<T*>(p.out);
  const long long orow = p.od.stride_s;
  auto zero = [&](int slot, int n, int row, int end, int warps, int mine) {
    T* const o = out + slot * p.od.stride_b + n * p.od.stride_n + chan;
    for (long long k = row + mine; k < end; k += warps) store(o + k * orow, splat<P>(0.f));
  };
  walk.begin(p, warp, zero);
  auto issue = [&](int s) {
    return walk.issue(p, smem_u32(stages + s * kStage), &entries[warp][s], zero);
  };
  Ahead ahead[kStages - 1];
#pragma unroll
  for (int s = 0; s < kStages - 1; ++s) ahead[s] = issue(s);
  if (p.spread) walk.zero_all(p, zero);

  GateScale gc{};
  F bias = splat<P>(0.f);
  T* o = nullptr;
  float* state = nullptr;
  int slot = 0, n = 0, s = 0, fill = kStages - 1;
  for (bool begun = SOLO || warp > 0;; begun = true) {  // a ring's first tile has none before it
    const int info = ahead[0].info, valid = info & kTokens;
    if (valid == 0) break;
    const float b = sigmoid(ahead[0].logit);
#pragma unroll
    for (int k = 0; k + 1 < kStages - 1; ++k) ahead[k] = ahead[k + 1];
    ahead[kStages - 2] = issue(fill);
    fill = fill + 1 == kStages ? 0 : fill + 1;
    if (lane < K) writes[warp][lane] = make_float2(b, b);
    if (info & kFresh) {
      const Entry& t = entries[warp][s];
      slot = t.slot;
      n = t.n;
      gc = gate_scale(__ldg(p.A_log + n), p.lower_bound);
      bias = load_const<P>(p.dt_bias + (size_t)n * D + chan);
      o = out + slot * p.od.stride_b + n * p.od.stride_n + t.row * orow + chan;
      state = p.states + ((size_t)t.place * p.N + n) * D + chan;
    }
    F start = splat<P>(0.f);
    if (info & kFirst) {
      if (info & kCut)
        start = join<D>(p, entries[warp][s].map, entries[warp][s].order, n, chan);
      else if (p.begin)
        start = load<P>(p.begin + ((size_t)slot * p.N + n) * D + chan);
    }
    T* const tg = reinterpret_cast<T*>(stages + s * kStage);
    copies_arrived<kStages - 1>();
    if (valid < K) {  // the warp's last tile of the unit
      const TileGate<P> gate = fill_rows<T, D, 2>(tg, valid, TileGate<P>{bias, gc.nz});
      bias = gate.bias;
      gc.nz = gate.nz;
    }

    // decays and writes, and what the tile makes of a state of zero; a becomes the decay since the
    // tile's start
    F a[K], u[K];
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const F e = each((load<P>(tg + k * D + chan) + bias) * gc.nz, ex2);
      a[k] = each(each(e + splat<P>(1.f), rcp) * gc.l2, ex2);
      u[k] = load<P>(tg + kRecTileElems + k * D + chan) * both<P>(writes[warp][k]);
      if (k > 0) {
        u[k] = fma(a[k], u[k - 1], u[k]);
        a[k] = a[k] * a[k - 1];
      }
    }
    // the state before the tile
    F h = start;
    if (begun) {
      ring.wait();
      if (!(info & kFirst)) h = load<P>(ring.inbox + chan);
    }
    const F before = h;
    h = fma(a[K - 1], h, u[K - 1]);
    store(ring.outbox + chan, h);
    if (SOLO || !(info & kStop)) ring.pass();
#pragma unroll
    for (int k = 0; k < K - 1; ++k) u[k] = fma(a[k], before, u[k]);
    u[K - 1] = h;
    if (p.states) {
      store(state, before);
      state += (size_t)kRing * p.N * D;
    }
    store_rows<T, D>(o, orow, valid, u);
    o += kRing * K * orow;
    if ((info & (kLast | kEnd)) == (kLast | kEnd))
      store(p.end + ((size_t)slot * p.N + n) * D + chan, h);
    s = s + 1 == kStages ? 0 : s + 1;
  }
}

// Sums of K values over a warp, by halving the values as the distance halves: 32 / K lanes in a row
// end with the sum of the same value.
template <int K>
__device__ __forceinline__ float warp_sums(float (&v)[K], int lane) {
  int n = K, o = 16;
#pragma unroll
  for (; n > 1; n /= 2, o /= 2) {
    const bool upper = lane & o;
#pragma unroll
    for (int i = 0; i < K / 2; ++i) {
      if (i >= n / 2) break;
      const float keep = upper ? v[i + n / 2] : v[i], give = upper ? v[i] : v[i + n / 2];
      v[i] = keep + __shfl_xor_sync(0xffffffffu, give, o);
    }
  }
#pragma unroll
  for (; o > 0; o /= 2) v[0] += __shfl_xor_sync(0xffffffffu, v[0], o);
  return v[0];
}

// 4x32x16384 bf16: 480 us, 5.9 TB/s (6.45 TB/s where 148 units keep every multiprocessor busy).  35
// instructions a value take 58 % of the issue slots.  13 or 14 warps spill registers (840-910 us); 11
// warps with a stage more took 520 us.
// The parameters' gradients are fp32 sums over a warp's tiles of a segment, fp64 from there on: fp64
// sums over the tiles would take 8 registers more of the 168, which are all in use.
template <class T, int D, bool SOLO>
__global__ void __launch_bounds__(32 * Block<T, true>::kWarps, 1)
    rec_backward_kernel(const __grid_constant__ RecParams p) {
  using B = Block<T, true>;
  using S = Shape<D>;
  using F = typename S::F;
  constexpr int K = S::K, V = S::V, P = V / 2, kStages = B::kStages, W = B::kWarps;
  constexpr int kRing = SOLO ? 1 : W;
  constexpr int kStage = kStageBytes<T, D, true>, kElems = kRecTileElems;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ Entry entries[W][kStages];
  __shared__ float2 writes[W][K];  // b and b
  launch_dependents();
  Walk<T, D, true, SOLO> walk(p);
  if (!same_plan(p)) return;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, chan = lane * V;
  const Ring<W, D, SOLO> ring(warp);
  uint8_t* const stages = smem + warp * kStages * kStage;  // a stage: g, x, dout, state
  const long long orow = p.od.stride_s;
  if (!p.dout.data) {
    for (int s = 0; s < kStages; ++s)
      for (int k = 0; k < K; ++k)
        store(reinterpret_cast<T*>(stages + s * kStage) + 2 * kElems + k * D + chan,
              splat<P>(0.f));
  }
  auto zero = [&](int slot, int n, int row, int end, int warps, int mine) {
    const long long o = slot * p.od.stride_b + n * p.od.stride_n + chan;
    T* const ob = static_cast<T*>(p.dbeta) + slot * p.bd.stride_b + n * p.bd.stride_n;
    for (long long k = row + mine; k < end; k += warps) {
      store(static_cast<T*>(p.out) + o + k * orow, splat<P>(0.f));
      store(static_cast<T*>(p.dg) + o + k * orow, splat<P>(0.f));
      if (lane == 0) ob[k * p.bd.stride_s] = from_f32<T>(0.f);
    }
  };
  walk.begin(p, warp, zero);
  auto issue = [&](int s) {
    return walk.issue(p, smem_u32(stages + s * kStage), &entries[warp][s], zero);
  };
  Ahead ahead[kStages - 1];
#pragma unroll
  for (int s = 0; s < kStages - 1; ++s) ahead[s] = issue(s);
  if (p.spread) walk.zero_all(p, zero);

  // the warp's part of the parameters' gradients in the unit, and where it goes
  F sum_b = splat<P>(0.f), sum_raw = splat<P>(0.f);
  constexpr size_t kNone = ~(size_t)0;
  size_t part = kNone;
  int parts = 0;
  auto flush = [&]() {
    float raw = sum(sum_raw);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) raw += __shfl_xor_sync(0xffffffffu, raw, o);
    // a unit has up to kRecRing rows, more than the ring has warps: zeros in those left over
    for (int i = 0; i < parts; i += kRing) {
      store(p.part_bias + part * D + chan, sum_b);
      if (lane == 0) p.part_A[part] = raw;
      sum_b = sum_raw = splat<P>(0.f);
      raw = 0.f;
      part += (size_t)kRing * p.N;
    }
  };

  GateScale gc{};
  F bias = splat<P>(0.f);
  long long o = 0;        // of the tile's rows in dx and dg
  T* dbeta = nullptr;     // of the lane's token
  constexpr int kEach = 32 / K;  // lanes that end with the same token's sum
  int slot = 0, n = 0, s = 0, fill = kStages - 1;
  for (bool begun = SOLO || warp > 0;; begun = true) {  // a ring's first tile has none before it
    const int info = ahead[0].info, valid = info & kTokens;
    if (valid == 0) break;
    // b, and its slope b (1 - b) without cancellation: 1 - b is e b
    const float e_own = expf(-ahead[0].logit), b_own = 1.f / (1.f + e_own);
    const float slope_own = e_own > 3e38f ? 0.f : b_own * (e_own * b_own);
#pragma unroll
    for (int k = 0; k + 1 < kStages - 1; ++k) ahead[k] = ahead[k + 1];
    ahead[kStages - 2] = issue(fill);
    fill = fill + 1 == kStages ? 0 : fill + 1;
    if (lane < K) writes[warp][lane] = make_float2(b_own, b_own);
    if (info & kFresh) {
      const Entry& t = entries[warp][s];
      if (part != kNone) flush();
      slot = t.slot;
      n = t.n;
      part = (size_t)t.part * p.N + n;
      parts = t.parts;
      gc = gate_scale(__ldg(p.A_log + n), p.lower_bound);
      bias = load_const<P>(p.dt_bias + (size_t)n * D + chan);
      o = slot * p.od.stride_b + n * p.od.stride_n + t.row * orow + chan;
      dbeta = static_cast<T*>(p.dbeta) + slot * p.bd.stride_b + n * p.bd.stride_n +
              (t.row + lane / kEach) * p.bd.stride_s;
    }
    F start = splat<P>(0.f);
    if (info & kFirst) {
      if (info & kCut)
        start = join<D>(p, entries[warp][s].map, entries[warp][s].order, n, chan);
      else if (p.begin)
        start = load<P>(p.begin + ((size_t)slot * p.N + n) * D + chan);
    }
    T* const tg = reinterpret_cast<T*>(stages + s * kStage);
    const T* const tx = tg + kElems + chan;
    const T* const td = tx + kElems;
    copies_arrived<kStages - 1>();
    if (valid < K) {
      const TileGate<P> gate = fill_rows<T, D, 3>(tg, valid, TileGate<P>{bias, gc.nz});
      bias = gate.bias;
      gc.nz = gate.nz;
    }

    // decays, and the factors w of dg = lam w
    F a[K], w[K];
    F h = load<P>(reinterpret_cast<const float*>(tg + 3 * kElems) + chan);
    const float slope = p.lower_bound * gc.ea;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      // e is kept finite: 1 - sigmoid is e sigmoid, without cancellation, and where the sigmoid
      // is zero so is their product
      const F e = each((load<P>(tg + k * D + chan) + bias) * gc.nz,
                       [](float z) { return min_nan(ex2(z), 3e38f); });
      const F sig = each(e + splat<P>(1.f), rcp);
      a[k] = each(sig * gc.l2, ex2);
      w[k] = sig * (e * sig) * (a[k] * slope) * h;
      h = fma(a[k], h, load<P>(tx + k * D) * both<P>(writes[warp][k]));
    }
    // lam of a tile with nothing behind it, and the decays from its end
    F lam[K], c0 = splat<P>(0.f);
#pragma unroll
    for (int k = K - 1; k >= 0; --k) {
      lam[k] = load<P>(td + k * D) + c0;
      c0 = a[k] * lam[k];
      if (k < K - 1) a[k] = a[k] * a[k + 1];
    }
    // a lam of the token behind the tile
    F c = start;
    if (begun) {
      ring.wait();
      if (!(info & kFirst)) c = load<P>(ring.inbox + chan);
    }
    const F behind = c;
    c = fma(a[0], c, c0);
    store(ring.outbox + chan, c);
    if (SOLO || !(info & kStop)) ring.pass();
#pragma unroll
    for (int k = 0; k < K - 1; ++k) lam[k] = fma(a[k + 1], behind, lam[k]);
    lam[K - 1] = lam[K - 1] + behind;
    if ((info & (kLast | kEnd)) == (kLast | kEnd) && p.end)
      store(p.end + ((size_t)slot * p.N + n) * D + chan, c);
    float dot[K];
    F here_b = splat<P>(0.f), here_raw = splat<P>(0.f);
#pragma unroll
    for (int k = 0; k < K; ++k) {
      w[k] = lam[k] * w[k];
      here_b = here_b + w[k];
      if (k < valid) here_raw = fma(w[k], load<P>(tg + k * D + chan) + bias, here_raw);
      dot[k] = sum(lam[k] * load<P>(tx + k * D));
      lam[k] = lam[k] * both<P>(writes[warp][k]);
    }
    store_rows<T, D>(static_cast<T*>(p.out) + o, orow, valid, lam);
    store_rows<T, D>(static_cast<T*>(p.dg) + o, orow, valid, w);
    if (valid < K) {
      // of rows behind the last token w is zero times the state behind it, which may be infinite
      here_b = splat<P>(0.f);
#pragma unroll
      for (int k = 0; k < K - 1; ++k)
        if (k < valid) here_b = here_b + w[k];
      gc = gate_scale(__ldg(p.A_log + n), p.lower_bound);  // the gate of the unit's other tiles
      bias = load_const<P>(p.dt_bias + (size_t)n * D + chan);
    }
    sum_b = sum_b + here_b;
    sum_raw = sum_raw + here_raw;
    const int k = lane / kEach;
    const float total = warp_sums<K>(dot, lane) * __shfl_sync(0xffffffffu, slope_own, k);
    if (lane % kEach == 0 && k < valid) *dbeta = from_f32<T>(total);
    o -= kRing * K * orow;
    dbeta -= kRing * K * p.bd.stride_s;
    s = s + 1 == kStages ? 0 : s + 1;
  }
  if (part != kNone) flush();
}

constexpr int kMapWarps = 16;

// The maps of the segments of cut sequences, one block each: row 0 of a sequence is its start, row
// k + 1 the map of the walk's k-th segment (the last one's is not needed).  A warp takes a
// sixteenth of the tokens, a batch at a time with the next one's loads under way.
// Bound by the special-function unit as the walk is: 2x16x4000 in 9 segments 20 us, of which the
// unit needs 11.
template <class T, int D, bool BACKWARD>
__global__ void __launch_bounds__(32 * kMapWarps, 1) rec_maps_kernel(const __grid_constant__ RecParams p) {
  using S = Shape<D>;
  using F = typename S::F;
  constexpr int V = S::V, P = V / 2, kBatch = 8 / (int)sizeof(T);
  __shared__ __align__(16) float sa[kMapWarps][D], sh[kMapWarps][D];
  launch_dependents();
  const int i = blockIdx.x / p.N, n = blockIdx.x - i * p.N;
  const int4 r0 = __ldg(record(p, i)), r1 = __ldg(record(p, i) + 1);
  if (p.plan[RH_CHECKSUM] != p.checksum) return;
  const int order = BACKWARD ? r1.z - 1 - r1.y : r1.y;
  if (order + 1 == r1.z) return;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, chan = lane * V;
  const kda_view_t& second = BACKWARD ? p.dout : p.x;
  const bool have = second.data != nullptr;
  const int share = (r0.z + kMapWarps - 1) / kMapWarps, lo = min(r0.z, warp * share), count = min(r0.z - lo, share);
  // the walk's first token of the share, and the way to the next one
  const int first = r0.y + (BACKWARD ? lo + count - 1 : lo), step = BACKWARD ? -1 : 1;
  F pa = splat<P>(1.f), ph = splat<P>(0.f);
  if (count > 0) {
    const T* const g = at<T>(p.g, r0.x, n, first) + chan;
    const T* const x = have ? at<T>(second, r0.x, n, first) + chan : nullptr;
    const T* const beta = at<T>(p.beta, r0.x, n, first);
    struct Batch {
      Bits<T, V> g[kBatch], x[kBatch];
      float logit;
    };
    auto fetch = [&](int from) {
      Batch b;
#pragma unroll
      for (int k = 0; k < kBatch; ++k) {
        const long long token = step * min(from + k, count - 1);
        b.g[k] = __ldg(reinterpret_cast<const Bits<T, V>*>(g + token * p.g.stride_s));
        b.x[k] = Bits<T, V>{};
        if (have) b.x[k] = __ldg(reinterpret_cast<const Bits<T, V>*>(x + token * second.stride_s));
      }
      b.logit = 0.f;
      if (!BACKWARD && from + lane < count && lane < kBatch)
        b.logit = to_f32(__ldg(beta + (long long)(from + lane) * p.beta.stride_s));
      return b;
    };
    Batch now = fetch(0);
    const GateScale gc = gate_scale(__ldg(p.A_log + n), p.lower_bound);
    const F bias = load_const<P>(p.dt_bias + (size_t)n * D + chan);
    for (int from = 0; from < count; from += kBatch) {
      const Batch next = fetch(min(from + kBatch, count - 1));
      const float own = BACKWARD ? 0.f : sigmoid(now.logit);
#pragma unroll
      for (int k = 0; k < kBatch; ++k) {
        const float b = BACKWARD ? 0.f : __shfl_sync(0xffffffffu, own, k);
        if (from + k < count) {
          const F raw = widen<T, V>(now.g[k]) + bias, v = widen<T, V>(now.x[k]);
          const F a = each(each(each(raw * gc.nz, ex2) + splat<P>(1.f), rcp) * gc.l2, ex2);
          pa = pa * a;
          ph = BACKWARD ? a * (ph + v) : fma(a, ph, v * b);
        }
      }
      now = next;
    }
  }
  // a product that is too small for fp32 stays above zero, so that an infinite state stays infinite
  auto above_zero = [](float v) { return v == 0.f ? 1.4e-45f : v; };
  store(&sa[warp][chan], each(pa, above_zero));
  store(&sh[warp][chan], ph);
  __syncthreads();
  if (warp > 0) return;
  pa = splat<P>(1.f);
  ph = splat<P>(0.f);
#pragma unroll
  for (int k = 0; k < kMapWarps; ++k) {
    const int w = BACKWARD ? kMapWarps - 1 - k : k;
    const F ka = load<P>(&sa[w][chan]);
    pa = pa * ka;
    ph = fma(ka, ph, load<P>(&sh[w][chan]));
  }
  float* m = p.maps + ((size_t)(r1.w + order + 1) * p.N + n) * 2 * D + chan;
  store(m, each(pa, above_zero));
  store(m + D, ph);
  if (order == 0) {
    m -= (size_t)p.N * 2 * D;
    store(m, splat<P>(0.f));
    store(m + D, p.begin ? load<P>(p.begin + ((size_t)r0.x * p.N + n) * D + chan) : splat<P>(0.f));
  }
}

// ddt_bias and dA_log: the warps' parts in a fixed order, in fp64.  A block has 8 channels of a head
// (the first one of a head its dA_log too); 128 threads a channel take the parts in turn.  About 4 us
// behind the walk, most of it the launch.
constexpr int kParamChannels = 8;
template <int D>
__global__ void __launch_bounds__(1024) rec_params_kernel(const __grid_constant__ RecParams p,
                                                          int parts, float* dA_log,
                                                          float* ddt_bias) {
  constexpr int kBlocks = D / kParamChannels, kRows = 1024 / kParamChannels;
  __shared__ double red[kParamChannels + 1][kRows];
  const int n = blockIdx.x / kBlocks, d0 = blockIdx.x % kBlocks * kParamChannels;
  const int c = threadIdx.x % kParamChannels, row = threadIdx.x / kParamChannels;
  wait_dependencies();
  if (p.plan[RH_CHECKSUM] != p.checksum) return;
  double sum = 0, raw = 0;
#pragma unroll 8
  for (int i = row; i < parts; i += kRows) {
    const size_t part = (size_t)i * p.N + n;
    sum += p.part_bias[part * D + d0 + c];
    if (d0 == 0 && c == 0) raw += p.part_A[part];
  }
  red[c][row] = sum;
  if (c == 0) red[kParamChannels][row] = raw;
  __syncthreads();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (warp > kParamChannels) return;
  sum = 0;
#pragma unroll
  for (int i = lane; i < kRows; i += 32) sum += red[warp][i];
  sum = warp_sum(sum);
  if (lane > 0) return;
  if (warp < kParamChannels) ddt_bias[(size_t)n * D + d0 + warp] = (float)sum;
  else if (d0 == 0) dA_log[n] = (float)sum;
}

// One token of every sequence, 4 channels a thread.  Bound by the launch and by HBM, 14 bytes a value
// (16-bit): one sequence 1.7 us, 256 x 32 x 128 3.9 us (3.8 TB/s; 3.3 us from L2).
template <class T, int D>
__global__ void __launch_bounds__(256) rec_step_kernel(const T* x, const T* g, const T* beta,
                                                       const float* h0, const float* A_log,
                                                       const float* dt_bias, float lower_bound,
                                                       T* out, float* h1, int N, int rows) {
  constexpr int kLanes = D / 4;
  const int row = blockIdx.x * (256 / kLanes) + threadIdx.x / kLanes;
  if (row >= rows) return;
  const int n = row % N, chan = threadIdx.x % kLanes * 4;
  const size_t i = (size_t)row * D + chan;
  const Pairs<2> raw = load_const<2>(g + i), v = load_const<2>(x + i);
  const Pairs<2> h = h0 ? load<2>(h0 + i) : splat<2>(0.f);  // may be h1
  const GateScale c = gate_scale(__ldg(A_log + n), lower_bound);
  const Pairs<2> bias = load_const<2>(dt_bias + (size_t)n * D + chan);
  const float b = sigmoid(to_f32(__ldg(beta + row)));
  const Pairs<2> a =
      each(each(each((raw + bias) * c.nz, ex2) + splat<2>(1.f), rcp) * c.l2, ex2);
  const Pairs<2> next = fma(a, h, v * b);
  store(h1 + i, next);
  store(out + i, next);
}

struct Sizes {
  size_t elem, x, rows, state, params;  // bytes of: an element, x dense, beta dense, a state array
};

Sizes sizes_of(const kda_recurrence_shape_t& s) {
  const size_t rows = (s.layout == KDA_LAYOUT_TND ? (size_t)s.S : (size_t)s.B * s.S) * s.N;
  const size_t e = dtype_bytes(s.dtype);
  return {e, rows * s.D * e, rows * e, (size_t)s.B * s.N * s.D * 4, (size_t)s.N * s.D * 4};
}

int slots(const kda_recurrence_shape_t& s) { return s.layout == KDA_LAYOUT_TND ? 1 : s.B; }

// What both passes check: shape, plan, views, pointers, alignment.  Fills p and the input ranges.
kda_status_t prepare(const kda_recurrence_shape_t* shape, const int32_t* plan_host,
                     const int32_t* plan_dev, size_t n_int32, const kda_view_t* x,
                     const kda_view_t* g, const kda_view_t* beta, const float* h0,
                     const float* A_log, const float* dt_bias, float lower_bound, void* workspace,
                     size_t workspace_bytes, bool backward, RecParams* p, ByteRange (&in)[9]) {
  kda_status_t st = validate_recurrence_shape(shape);
  if (st != KDA_OK) return st;
  if (!plan_host || !plan_dev || !x || !g || !beta || !A_log || !dt_bias)
    return KDA_ERR_NULL;
  st = validate_recurrence_plan(plan_host, n_int32, shape);
  if (st != KDA_OK) return st;
  if (!(lower_bound >= -5.0f && lower_bound <= 0.0f)) return KDA_ERR_LOWER_BOUND;
  size_t need = 0;
  st = kda_recurrence_workspace_size(plan_host, n_int32, backward, &need);
  if (st != KDA_OK) return st;
  // a workspace of the status word alone may be left out
  if (!workspace && need > kWsHeaderBytes) return KDA_ERR_NULL;
  if ((workspace && workspace_bytes < need) || (reinterpret_cast<uintptr_t>(workspace) & 255u))
    return KDA_ERR_WORKSPACE;
  for (const void* ptr : {(const void*)h0, (const void*)A_log, (const void*)dt_bias,
                          (const void*)plan_dev})
    if (!aligned16(ptr)) return KDA_ERR_ALIGN;
  const Sizes z = sizes_of(*shape);
  const int nb = slots(*shape);
  p->x = *x;
  p->g = *g;
  p->beta = *beta;
  if ((st = check_view(&p->x, nb, shape->N, shape->S, shape->D, z.elem, &in[0])) != KDA_OK ||
      (st = check_view(&p->g, nb, shape->N, shape->S, shape->D, z.elem, &in[1])) != KDA_OK ||
      (st = check_view(&p->beta, nb, shape->N, shape->S, 1, z.elem, &in[2])) != KDA_OK)
    return st;
  in[3] = dense_range(h0, z.state);
  in[4] = dense_range(A_log, (size_t)shape->N * 4);
  in[5] = dense_range(dt_bias, z.params);
  in[6] = dense_range(plan_dev, n_int32 * 4);
  in[7] = dense_range(workspace, workspace ? need : 0);
  for (int i = 0; i < 7; ++i)  // it is written to
    if (overlap(in[i], in[7])) return KDA_ERR_ALIAS;
  p->plan = plan_dev;
  p->checksum = plan_host[RH_CHECKSUM];
  p->N = shape->N;
  p->units = plan_host[RH_RECORDS] * shape->N;
  p->slot_rows = plan_host[RH_PADDED] ? shape->S : 0;
  p->A_log = A_log;
  p->dt_bias = dt_bias;
  p->lower_bound = lower_bound;
  p->status = static_cast<int32_t*>(workspace);
  p->maps = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + kWsHeaderBytes);
  p->od = dense_view(nullptr, shape->layout, shape->N, shape->S, shape->D);
  p->bd = dense_view(nullptr, shape->layout, shape->N, shape->S, 1);
  if (nb == 1) p->od.stride_b = p->bd.stride_b = 0;
  return KDA_OK;
}

size_t states_floats(const int32_t* plan) {
  return (size_t)plan[RH_TILES] * plan[RH_N] * plan[RH_D];
}

// The workspace after its header: the maps of cut sequences, and the parameters' partial gradients of
// a backward pass.
struct Scratch {
  size_t bias, A, total;
  Scratch(const int32_t* plan, bool backward) {
    const size_t N = plan[RH_N], row = N * plan[RH_D] * 4;
    bias = kWsHeaderBytes + plan[RH_MAPS] * 2 * row;
    A = bias + (backward ? plan[RH_PARTS] * row : 0);
    total = A + (backward ? plan[RH_PARTS] * N * 4 : 0);
  }
};

// Launches a pass: the maps where sequences are cut, and the walk, a block on every multiprocessor
// that has a unit or rows to write zeros to.
template <class T, int D, bool BACKWARD, bool SOLO, class Kernel>
cudaError_t launch(Kernel kernel, PerDevice& once, RecParams& p, const int32_t* plan,
                   cudaStream_t s) {
  using B = Block<T, BACKWARD>;
  constexpr int kSmem = kWalkSmem<T, D, BACKWARD>;
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  e = once_per_device(once, dev, &sms, [&](int d, int* n) {
    const cudaError_t err =
        cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
    return err == cudaSuccess ? cudaDeviceGetAttribute(n, cudaDevAttrMultiProcessorCount, d) : err;
  });
  if (e != cudaSuccess) return e;
  constexpr int kRing = SOLO ? 1 : B::kWarps;
  p.spread = p.slot_rows && p.units < sms;
  const int blocks = p.spread ? sms : std::min(sms, p.units);
  constexpr int K = Shape<D>::K, kCopy = 512 / (D * (int)sizeof(T));
  const kda_view_t* const views[] = {&p.g, &p.x, &p.dout, &p.beta};
  for (int i = 0; i < 4; ++i) {
    const long long row = views[i]->stride_s * (long long)sizeof(T);
    if (i < 3) p.copy_step[i] = kCopy * row;
    p.tile_step[i] = (BACKWARD ? -kRing : kRing) * K * row;
  }
  if (plan[RH_MAPS]) {
    rec_maps_kernel<T, D, BACKWARD><<<(unsigned)p.units, 32 * kMapWarps, 0, s>>>(p);
    e = cudaGetLastError();
    return e != cudaSuccess ? e : launch_early(kernel, blocks, 32 * B::kWarps, kSmem, s, p);
  }
  kernel<<<(unsigned)blocks, 32 * B::kWarps, kSmem, s>>>(p);
  return cudaGetLastError();
}

template <class T, int D>
cudaError_t launch_forward(RecParams& p, const int32_t* plan, cudaStream_t s) {
  static PerDevice once[2];
  return plan[RH_SOLO] ? launch<T, D, false, true>(rec_forward_kernel<T, D, true>, once[1], p, plan, s)
                       : launch<T, D, false, false>(rec_forward_kernel<T, D, false>, once[0], p, plan, s);
}

template <class T, int D>
cudaError_t launch_backward(RecParams& p, const int32_t* plan, cudaStream_t s) {
  static PerDevice once[2];
  return plan[RH_SOLO] ? launch<T, D, true, true>(rec_backward_kernel<T, D, true>, once[1], p, plan, s)
                       : launch<T, D, true, false>(rec_backward_kernel<T, D, false>, once[0], p, plan, s);
}

template <class F>
cudaError_t dispatch(const kda_recurrence_shape_t& s, F&& f) {
  auto with_type = [&](auto* tag) {
    return s.D == 128 ? f(tag, std::integral_constant<int, 128>())
                      : f(tag, std::integral_constant<int, 64>());
  };
  if (s.dtype == KDA_BF16) return with_type((__nv_bfloat16*)nullptr);
  if (s.dtype == KDA_FP16) return with_type((__half*)nullptr);
  return with_type((float*)nullptr);
}

// every output against every input and every other output
template <int NI, int NO>
bool any_overlap(const ByteRange (&in)[NI], const ByteRange (&out)[NO]) {
  for (int o = 0; o < NO; ++o) {
    for (const ByteRange& r : in)
      if (overlap(r, out[o])) return true;
    for (int q = 0; q < o; ++q)
      if (overlap(out[q], out[o])) return true;
  }
  return false;
}

}  // namespace
}  // namespace kda

using namespace kda;

extern "C" kda_status_t kda_recurrence_states_size(const int32_t* plan, size_t n, size_t* floats) {
  if (!floats) return KDA_ERR_NULL;
  const kda_status_t st = validate_recurrence_plan(plan, n, nullptr);
  if (st != KDA_OK) return st;
  *floats = states_floats(plan);
  return KDA_OK;
}

extern "C" kda_status_t kda_recurrence_workspace_size(const int32_t* plan, size_t n,
                                                      int32_t backward, size_t* bytes) {
  if (!bytes) return KDA_ERR_NULL;
  const kda_status_t st = validate_recurrence_plan(plan, n, nullptr);
  if (st != KDA_OK) return st;
  *bytes = Scratch(plan, backward != 0).total;
  return KDA_OK;
}

extern "C" kda_status_t kda_recurrence_forward(
    const kda_recurrence_shape_t* shape, const int32_t* plan_host, const int32_t* plan_dev,
    size_t n_int32, const kda_view_t* x, const kda_view_t* g, const kda_view_t* beta,
    const float* initial_state, const float* A_log, const float* dt_bias, float lower_bound,
    float* states, void* workspace, size_t workspace_bytes, void* out, float* final_state,
    kda_stream_t stream) {
  RecParams p{};
  ByteRange in[9];
  kda_status_t st = prepare(shape, plan_host, plan_dev, n_int32, x, g, beta, initial_state, A_log,
                            dt_bias, lower_bound, workspace, workspace_bytes, false, &p, in);
  if (st != KDA_OK) return st;
  if (!out || !final_state) return KDA_ERR_NULL;
  if (!aligned16(out) || !aligned16(final_state) || !aligned16(states)) return KDA_ERR_ALIGN;
  const Sizes z = sizes_of(*shape);
  // final_state may be initial_state itself: the end of a sequence that is not cut follows from its
  // start, and of one that is cut the start is among the maps, which are done before the walk
  if (final_state == initial_state) in[3] = ByteRange{};
  const ByteRange outs[] = {dense_range(out, z.x), dense_range(final_state, z.state),
                            dense_range(states, states_floats(plan_host) * 4)};
  if (any_overlap(in, outs)) return KDA_ERR_ALIAS;
  if ((st = check_device()) != KDA_OK) return st;

  const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  p.states = states;
  p.out = out;
  p.begin = initial_state;
  p.end = final_state;
  const cudaError_t e = dispatch(*shape, [&](auto* tag, auto d) {
    return launch_forward<std::remove_pointer_t<decltype(tag)>, decltype(d)::value>(p, plan_host, s);
  });
  return e == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
}

extern "C" kda_status_t kda_recurrence_backward(
    const kda_recurrence_shape_t* shape, const int32_t* plan_host, const int32_t* plan_dev,
    size_t n_int32, const kda_view_t* dout, const float* dfinal_state, const kda_view_t* x,
    const kda_view_t* g, const kda_view_t* beta, const float* A_log, const float* dt_bias,
    float lower_bound, const float* states, void* workspace, size_t workspace_bytes, void* dx,
    void* dg, void* dbeta, float* dinitial_state, float* dA_log, float* ddt_bias,
    kda_stream_t stream) {
  RecParams p{};
  ByteRange in[9], r_dout;
  kda_status_t st = prepare(shape, plan_host, plan_dev, n_int32, x, g, beta, nullptr, A_log,
                            dt_bias, lower_bound, workspace, workspace_bytes, true, &p, in);
  if (st != KDA_OK) return st;
  if (!states || !dx || !dg || !dbeta || !dA_log || !ddt_bias) return KDA_ERR_NULL;
  for (const void* ptr : {(const void*)dfinal_state, (const void*)states, (const void*)dx,
                          (const void*)dg, (const void*)dinitial_state, (const void*)dA_log,
                          (const void*)ddt_bias})
    if (!aligned16(ptr)) return KDA_ERR_ALIGN;
  const Sizes z = sizes_of(*shape);
  if (reinterpret_cast<uintptr_t>(dbeta) % z.elem) return KDA_ERR_ALIGN;
  if (dout && dout->data) {
    p.dout = *dout;
    st = check_view(&p.dout, slots(*shape), shape->N, shape->S, shape->D, z.elem, &r_dout);
    if (st != KDA_OK) return st;
  }
  in[8] = dense_range(states, states_floats(plan_host) * 4);
  const ByteRange outs[] = {dense_range(dx, z.x), dense_range(dg, z.x), dense_range(dbeta, z.rows),
                            dense_range(dinitial_state, z.state),
                            dense_range(dA_log, (size_t)shape->N * 4),
                            dense_range(ddt_bias, z.params)};
  const ByteRange grads[] = {r_dout, dense_range(dfinal_state, z.state)};
  if (any_overlap(in, outs) || any_overlap(grads, outs)) return KDA_ERR_ALIAS;
  for (const ByteRange& r : {grads[0], grads[1], in[8]})
    if (overlap(r, in[7])) return KDA_ERR_ALIAS;  // the workspace
  if ((st = check_device()) != KDA_OK) return st;

  const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const Scratch scratch(plan_host, true);
  uint8_t* const ws = static_cast<uint8_t*>(workspace);
  p.part_bias = reinterpret_cast<float*>(ws + scratch.bias);
  p.part_A = reinterpret_cast<float*>(ws + scratch.A);
  p.states = const_cast<float*>(states);
  p.begin = dfinal_state;
  p.out = dx;
  p.dg = dg;
  p.dbeta = dbeta;
  p.end = dinitial_state;
  const cudaError_t e = dispatch(*shape, [&](auto* tag, auto d) {
    constexpr int D = decltype(d)::value;
    using T = std::remove_pointer_t<decltype(tag)>;
    const cudaError_t err = launch_backward<T, D>(p, plan_host, s);
    if (err != cudaSuccess) return err;
    return launch_early(rec_params_kernel<D>, shape->N * (D / kParamChannels), 1024, 0,
                        s, p, plan_host[RH_PARTS], dA_log, ddt_bias);
  });
  return e == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
}

extern "C" kda_status_t kda_recurrence_step(int32_t B, int32_t N, int32_t D, int32_t dtype,
                                            const void* x, const void* g, const void* beta,
                                            const float* state_in, const float* A_log,
                                            const float* dt_bias, float lower_bound, void* out,
                                            float* state_out, kda_stream_t stream) {
  // a step is the recurrence's shape with one token per sequence
  const kda_recurrence_shape_t shape = {KDA_LAYOUT_BSND, B, N, 1, D, dtype};
  kda_status_t st = validate_recurrence_shape(&shape);
  if (st != KDA_OK) return st;
  if (!x || !g || !beta || !A_log || !dt_bias || !out || !state_out) return KDA_ERR_NULL;
  if (!(lower_bound >= -5.0f && lower_bound <= 0.0f)) return KDA_ERR_LOWER_BOUND;
  for (const void* ptr : {x, g, (const void*)state_in, (const void*)A_log, (const void*)dt_bias,
                          (const void*)out, (const void*)state_out})
    if (!aligned16(ptr)) return KDA_ERR_ALIGN;
  const Sizes z = sizes_of(shape);
  if (reinterpret_cast<uintptr_t>(beta) % z.elem) return KDA_ERR_ALIGN;
  const ByteRange in[] = {dense_range(x, z.x), dense_range(g, z.x), dense_range(beta, z.rows),
                          dense_range(A_log, (size_t)N * 4), dense_range(dt_bias, z.params),
                          state_in == state_out ? ByteRange{} : dense_range(state_in, z.state)};
  const ByteRange outs[] = {dense_range(out, z.x), dense_range(state_out, z.state)};
  if (any_overlap(in, outs)) return KDA_ERR_ALIAS;
  if ((st = check_device()) != KDA_OK) return st;

  const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const int rows = B * N;  // at most INT_MAX / 2
  auto launch = [&](auto* tag) {
    using T = std::remove_pointer_t<decltype(tag)>;
    const int per_block = 1024 / D;
    (D == 128 ? rec_step_kernel<T, 128> : rec_step_kernel<T, 64>)
        <<<(unsigned)((rows + per_block - 1) / per_block), 256, 0, s>>>(
            static_cast<const T*>(x), static_cast<const T*>(g), static_cast<const T*>(beta), state_in,
            A_log, dt_bias, lower_bound, static_cast<T*>(out), state_out, N, rows);
  };
  if (dtype == KDA_BF16) launch((__nv_bfloat16*)nullptr);
  else if (dtype == KDA_FP16) launch((__half*)nullptr);
  else launch((float*)nullptr);
  return cudaGetLastError() == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
}
