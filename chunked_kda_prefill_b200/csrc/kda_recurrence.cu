// kda_recurrence.cu -- the gated recurrence, the vector form of the KDA state:
//     a_t = exp(lb sigmoid(e^A (g_t + bias))),  h_t = a_t h_{t-1} + sigmoid(beta_t) x_t.
//
// A ring of warps walks one segment (a sequence, or a part of a long one) of one head, a tile of
// 1024 values a warp at a time: the warp's own copies bring its next tiles to shared memory, it
// forms all decays and writes of its tile, waits for the state that the warp before it leaves,
// runs through its 8 or 16 tokens, passes the state on and only then writes its results.  So what
// happens one after another is a wait, 8 or 16 fused multiply-adds and a hand-over (about 150 ns
// for 1024 values), the rest runs side by side, and no barrier stops a block.  The backward pass
// is the same walk from the end with the state's gradient, the states before the tiles given.
//
// Where a few long sequences would leave multiprocessors idle, the plan cuts them.  A kernel before
// the walk then forms the map h -> A h + H of each segment, and a segment starts from the maps
// before it.
//
// Both passes are bound by HBM: 6 bytes a value forward (16-bit), 10 backward.
#include <cuda_runtime.h>

#include <algorithm>
#include <climits>
#include <cmath>
#include <cstdint>
#include <cstdlib>
#include <type_traits>

#include "kda_args.h"
#include "kda_io.cuh"
#include "kda_once.h"
#include "kda_recurrence.h"

namespace kda {
namespace {

constexpr uint32_t kWaitLimit = 1u << 26;

struct RecParams {
  kda_view_t x, g, beta, dout;  // device addresses and strides
  const int32_t* plan;
  int32_t checksum;
  int32_t N, units;   // units: segments times heads
  int32_t slot_rows;  // rows that a slot's outputs have, padding included; 0 for packed rows
  int32_t ring;       // warps of a ring
  const float* begin;  // [B][N][D] the walk's start (forward h0, backward dfinal), or null for zeros
  const float* A_log;
  const float* dt_bias;
  float lower_bound;
  int32_t* status;
  float* maps;    // [RH_MAPS][N][2][D] of the cut sequences
  float* states;  // [tiles][N][D] the states before the tiles: forward writes, backward reads
  void* out;      // forward: out; backward: dx
  void* dg;
  void* dbeta;
  float* end;        // [B][N][D] the walk's end: final_state, or dh0 (null: not wanted)
  float* part_bias;  // [RH_PARTS][N][D]
  float* part_A;     // [RH_PARTS][N]
  kda_view_t od, bd;  // strides of the dense outputs with and without channels
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

// Warps of a block, one block a multiprocessor, and the tiles whose copies a warp has under way or at
// work: as many as the registers (forward 128 a thread, backward 168) and shared memory allow.
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

// A tile as its copies' issuer describes it to the same warp later.
struct __align__(16) Tile {
  int slot, row, valid, place;  // row: of its first token; place: of its state
  int n, flags, map, part;
};
enum : int {
  kFresh = 1,   // the warp's first tile in the unit
  kFirst = 2,   // the segment's first tile of the walk
  kLast = 4,    // the segment's last tile of the walk
  kBegin = 8,   // of the segment that the walk of the sequence begins with
  kEnd = 16,    // of the segment that it ends with
  kCut = 32,    // of a cut sequence
  kOrder = 6    // flags >> kOrder: the segment's place in the walk of its sequence
};

// Whether the plan on the device is the host's; block 0 leaves the status.
__device__ __forceinline__ bool same_plan(const RecParams& p) {
  const bool same = p.plan[RH_CHECKSUM] == p.checksum;
  if (blockIdx.x == 0 && threadIdx.x == 0) *p.status = same ? DS_OK : DS_PLAN;
  return same;
}

__device__ __forceinline__ const int4* record(const RecParams& p, int i) {
  return reinterpret_cast<const int4*>(p.plan + kRecHeader) + 2 * i;
}

// A warp's way through the tiles of its ring's units.  The units are dealt to the blocks in rounds,
// every other one in reverse, so that with the plan's order (longest first) no block gets the longer
// unit of every round; a block's rings take its rounds in turn.
template <int K, bool BACKWARD>
struct Walk {
  int4 r0, r1;  // the record: slot, start, len, tile; part, segment, segments, map
  int n, t, tiles, round;
  bool fresh, done;

  // zero(slot, n, row, rows): called for the rows behind a sequence's last token
  template <class Zero>
  __device__ void enter(const RecParams& p, int rings, Zero&& zero) {
    for (;; round += rings) {
      const long long base = (long long)round * gridDim.x;
      const long long unit = base + (round & 1 ? gridDim.x - 1 - blockIdx.x : blockIdx.x);
      done = unit >= p.units;
      if (done) return;
      const int i = (int)unit / p.N;
      n = (int)unit - i * p.N;
      r0 = __ldg(record(p, i));
      r1 = __ldg(record(p, i) + 1);
      tiles = (r0.z + K - 1) / K;
      fresh = true;
      if (p.slot_rows && r1.y + 1 == r1.z) zero(r0.x, n, r0.y + r0.z, p.slot_rows - r0.y - r0.z);
      if (t < tiles) return;
      t -= tiles;
    }
  }
  template <class Zero>
  __device__ void next(const RecParams& p, int rings, Zero&& zero) {
    fresh = false;
    t += p.ring;
    if (t < tiles) return;
    t -= tiles;
    round += rings;
    enter(p, rings, zero);
  }
  __device__ Tile tile(int* valid) const {
    const int k = BACKWARD ? tiles - 1 - t : t;
    const int order = BACKWARD ? r1.z - 1 - r1.y : r1.y;
    *valid = min(K, r0.z - k * K);
    return {r0.x, r0.y + k * K, *valid, r0.w + k, n,
            (fresh ? kFresh : 0) | (t == 0 ? kFirst : 0) | (t == tiles - 1 ? kLast : 0) |
                (order == 0 ? kBegin : 0) | (order == r1.z - 1 ? kEnd : 0) |
                (r1.z > 1 ? kCut : 0) | order << kOrder,
            r1.w, r1.x + t};
  }
};

// Starts the copies of a tile's rows of one tensor, a row a lane or, where the rows lie side by side,
// all rows at once.
template <class T, int D>
__device__ __forceinline__ void copy_rows(uint32_t dst, const kda_view_t& v, const Tile& t,
                                          int first_lane, int lane, uint32_t bar) {
  const int k = lane - first_lane;
  if (k < 0 || k >= t.valid) return;
  const T* from = at<T>(v, t.slot, t.n, t.row);
  if (v.stride_s == D) {
    if (k == 0) bulk_load(dst, from, t.valid * D * (int)sizeof(T), bar);
  } else {
    bulk_load(dst + k * D * (int)sizeof(T), from + k * v.stride_s, D * (int)sizeof(T), bar);
  }
}

// The state that a cut segment starts from: the maps of those before it in the walk's order, the
// first of which is constant.
template <int D>
__device__ typename Shape<D>::F join(const RecParams& p, int map, int order, int n, int chan) {
  constexpr int P = Shape<D>::V / 2;
  auto s = splat<P>(0.f);
  const float* m = p.maps + ((size_t)map * p.N + n) * 2 * D + chan;
#pragma unroll 4
  for (int k = 0; k <= order; ++k) {
    s = fma(load<P>(m), s, load<P>(m + D));
    m += (size_t)p.N * 2 * D;
  }
  return s;
}

// What every warp of a walk sets up, and its waits.
template <int STAGES>
struct Lines {
  uint32_t full, mine, theirs;  // barriers: a stage is loaded; this warp's turn, the next one's
  float* inbox;                 // the state handed to this warp, and to the next one
  float* outbox;
  bool failed;
  __device__ void wait(uint32_t bar, uint32_t phase) {
    if (!failed && !mbar_wait_bounded(bar, phase & 1, kWaitLimit)) failed = true;
  }
};

template <class T, int D, bool BACKWARD>
__device__ __forceinline__ Lines<Block<T, BACKWARD>::kStages> lines(const RecParams& p, int warp,
                                                                    int lane) {
  using B = Block<T, BACKWARD>;
  __shared__ uint64_t full[B::kWarps][B::kStages], turn[B::kWarps];
  __shared__ __align__(16) float box[B::kWarps][D];
  const int place = warp % p.ring, after = warp - place + (place + 1) % p.ring;
  Lines<B::kStages> l;
  l.full = smem_u32(full[warp]);
  l.mine = smem_u32(&turn[warp]);
  l.theirs = smem_u32(&turn[after]);
  l.inbox = box[warp];
  l.outbox = box[after];
  l.failed = false;
  if (lane == 0) {
    for (int s = 0; s < B::kStages; ++s) mbar_init(l.full + 8 * s, 1);
    mbar_init(l.mine, 1);
    fence_barrier_init();
  }
  __syncthreads();
  return l;
}

// A wait has run out: says so, and stays until the copies under way have ended.
template <int STAGES>
__device__ __noinline__ void give_up(const RecParams& p, const Lines<STAGES>& l, const Tile* tiles,
                                     uint32_t i, int lane) {
  if (lane == 0) atomicExch(p.status, DS_TIMEOUT);
  for (uint32_t j = i; j < i + STAGES; ++j)
    if (tiles[j % STAGES].valid)
      mbar_wait_bounded(l.full + 8 * (j % STAGES), (j / STAGES) & 1, kWaitLimit);
}

// Rows of a partial tile that hold no token: closed gates (decay one) and zero writes.
template <class T, int D, int TENSORS>
__device__ __noinline__ void fill_rows(T* stage, int valid) {
  using S = Shape<D>;
  const int chan = (threadIdx.x & 31) * S::V;
  for (int k = valid; k < S::K; ++k)
    for (int i = 0; i < TENSORS; ++i)
      store(stage + i * kRecTileElems + k * D + chan, splat<S::V / 2>(i == 0 ? -INFINITY : 0.f));
  fence_proxy_async_smem();  // a later copy writes these rows too
}

template <class T, int D>
__global__ void __launch_bounds__(32 * Block<T, false>::kWarps, 1)
    rec_forward_kernel(const __grid_constant__ RecParams p) {
  using B = Block<T, false>;
  using S = Shape<D>;
  using F = typename S::F;
  constexpr int K = S::K, V = S::V, P = V / 2, kStages = B::kStages;
  constexpr int kStage = kStageBytes<T, D, false>;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ Tile tiles[B::kWarps][kStages];
  if (!same_plan(p)) return;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, chan = lane * V;
  const int rings = B::kWarps / p.ring;
  auto l = lines<T, D, false>(p, warp, lane);
  uint8_t* const stages = smem + warp * kStages * kStage;
  T* const out = static_cast<T*>(p.out);
  const long long orow = p.od.stride_s;

  Walk<K, false> walk;
  auto zero = [&](int slot, int n, int row, int rows) {
    T* o = out + slot * p.od.stride_b + n * p.od.stride_n + row * orow + chan;
    for (int k = warp % p.ring; k < rows; k += p.ring) store(o + k * orow, splat<P>(0.f));
  };
  walk.round = warp / p.ring;
  walk.t = warp % p.ring;
  walk.enter(p, rings, zero);
  // the copies of the next tile of the way; returns the lane's write logit of that tile
  auto issue = [&](int s) {
    __syncwarp();  // all lanes have read what the stage held
    float logit = 0.f;
    if (walk.done) {
      if (lane == 0) tiles[warp][s].valid = 0;
    } else {
      int valid;
      const Tile t = walk.tile(&valid);
      const uint32_t bar = l.full + 8 * s, dst = smem_u32(stages + s * kStage);
      if (lane == 0) {
        tiles[warp][s] = t;
        mbar_arrive_expect_tx(bar, 2 * valid * D * (int)sizeof(T));
      }
      __syncwarp();
      copy_rows<T, D>(dst, p.g, t, 0, lane, bar);
      copy_rows<T, D>(dst + kRecTileElems * sizeof(T), p.x, t, 16, lane, bar);
      if (lane < valid) logit = to_f32(__ldg(at<T>(p.beta, t.slot, t.n, t.row + lane)));
      walk.next(p, rings, zero);
    }
    return logit;
  };
  float logits[kStages - 1];
#pragma unroll
  for (int s = 0; s < kStages - 1; ++s) logits[s] = issue(s);

  GateScale gc{};
  F bias = splat<P>(0.f), h = splat<P>(0.f);
  int s = 0, fill = kStages - 1;
  uint32_t i = 0;
  for (;; ++i) {
    const float b = sigmoid(logits[0]);
#pragma unroll
    for (int k = 0; k + 1 < kStages - 1; ++k) logits[k] = logits[k + 1];
    logits[kStages - 2] = issue(fill);
    fill = fill + 1 == kStages ? 0 : fill + 1;
    __syncwarp();
    const Tile t = tiles[warp][s];
    if (t.valid == 0) break;
    if (t.flags & kFresh) {
      gc = gate_scale(__ldg(p.A_log + t.n), p.lower_bound);
      bias = load_const<P>(p.dt_bias + (size_t)t.n * D + chan);
    }
    F start = splat<P>(0.f);
    if (t.flags & kFirst) {
      if (t.flags & kCut) start = join<D>(p, t.map, t.flags >> kOrder, t.n, chan);
      else if (p.begin) start = load<P>(p.begin + ((size_t)t.slot * p.N + t.n) * D + chan);
    }
    T* const tg = reinterpret_cast<T*>(stages + s * kStage);
    l.wait(l.full + 8 * s, i / kStages);
    if (t.valid < K) fill_rows<T, D, 2>(tg, t.valid);

    // decays and writes
    F a[K], u[K];
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const F e = each((load<P>(tg + k * D + chan) + bias) * gc.nz, ex2);
      a[k] = each(each(e + splat<P>(1.f), rcp) * gc.l2, ex2);
      u[k] = load<P>(tg + kRecTileElems + k * D + chan) * __shfl_sync(0xffffffffu, b, k);
    }
    // the state before the tile
    if (p.ring > 1 && (i > 0 || warp % p.ring > 0)) {
      l.wait(l.mine, warp % p.ring > 0 ? i : i - 1);
      h = load<P>(l.inbox + chan);
    }
    if (l.failed) break;
    if (t.flags & kFirst) h = start;
    const F before = h;
#pragma unroll
    for (int k = 0; k < K; ++k) h = u[k] = fma(a[k], h, u[k]);
    if (p.ring > 1) {
      store(l.outbox + chan, h);
      __syncwarp();
      if (lane == 0) mbar_arrive(l.theirs);
    }
    if (p.states) store(p.states + ((size_t)t.place * p.N + t.n) * D + chan, before);
    T* o = out + t.slot * p.od.stride_b + t.n * p.od.stride_n + t.row * orow + chan;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      if (k < t.valid) store(o, u[k]);
      o += orow;
    }
    if ((t.flags & (kLast | kEnd)) == (kLast | kEnd))
      store(p.end + ((size_t)t.slot * p.N + t.n) * D + chan, h);
    s = s + 1 == kStages ? 0 : s + 1;
  }
  if (l.failed) give_up(p, l, tiles[warp], i, lane);
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

template <class T, int D>
__global__ void __launch_bounds__(32 * Block<T, true>::kWarps, 1)
    rec_backward_kernel(const __grid_constant__ RecParams p) {
  using B = Block<T, true>;
  using S = Shape<D>;
  using F = typename S::F;
  constexpr int K = S::K, V = S::V, P = V / 2, kStages = B::kStages;
  constexpr int kStage = kStageBytes<T, D, true>, kElems = kRecTileElems;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ Tile tiles[B::kWarps][kStages];
  if (!same_plan(p)) return;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, chan = lane * V;
  const int rings = B::kWarps / p.ring;
  auto l = lines<T, D, true>(p, warp, lane);
  uint8_t* const stages = smem + warp * kStages * kStage;  // a stage: g, x, dout, state
  T* const dx = static_cast<T*>(p.out);
  T* const dg = static_cast<T*>(p.dg);
  T* const dbeta = static_cast<T*>(p.dbeta);
  const long long orow = p.od.stride_s;
  if (!p.dout.data) {
    for (int s = 0; s < kStages; ++s)
      for (int k = 0; k < K; ++k)
        store(reinterpret_cast<T*>(stages + s * kStage) + 2 * kElems + k * D + chan,
              splat<P>(0.f));
  }

  Walk<K, true> walk;
  auto zero = [&](int slot, int n, int row, int rows) {
    const long long o = slot * p.od.stride_b + n * p.od.stride_n + row * orow + chan;
    T* const ob = dbeta + slot * p.bd.stride_b + n * p.bd.stride_n + row * p.bd.stride_s;
    for (int k = warp % p.ring; k < rows; k += p.ring) {
      store(dx + o + k * orow, splat<P>(0.f));
      store(dg + o + k * orow, splat<P>(0.f));
      if (lane == 0) ob[k * p.bd.stride_s] = from_f32<T>(0.f);
    }
  };
  walk.round = warp / p.ring;
  walk.t = warp % p.ring;
  walk.enter(p, rings, zero);
  auto issue = [&](int s) {
    __syncwarp();  // all lanes have read what the stage held
    float logit = 0.f;
    if (walk.done) {
      if (lane == 0) tiles[warp][s].valid = 0;
    } else {
      int valid;
      const Tile t = walk.tile(&valid);
      const uint32_t bar = l.full + 8 * s, dst = smem_u32(stages + s * kStage);
      if (lane == 0) {
        tiles[warp][s] = t;
        mbar_arrive_expect_tx(
            bar, (p.dout.data ? 3 : 2) * valid * D * (int)sizeof(T) + D * (int)sizeof(float));
      }
      __syncwarp();
      copy_rows<T, D>(dst, p.g, t, 0, lane, bar);
      copy_rows<T, D>(dst + kElems * sizeof(T), p.x, t, 16, lane, bar);
      if (p.dout.data) copy_rows<T, D>(dst + 2 * kElems * sizeof(T), p.dout, t, K == 8 ? 8 : 0, lane, bar);
      if (lane == 31)
        bulk_load(dst + 3 * kElems * sizeof(T), p.states + ((size_t)t.place * p.N + t.n) * D, D * 4, bar);
      if (lane < valid) logit = to_f32(__ldg(at<T>(p.beta, t.slot, t.n, t.row + lane)));
      walk.next(p, rings, zero);
    }
    return logit;
  };
  float logits[kStages - 1];
#pragma unroll
  for (int s = 0; s < kStages - 1; ++s) logits[s] = issue(s);

  // the warp's part of the parameters' gradients in the unit, and where it goes
  F sum_b = splat<P>(0.f), sum_raw = splat<P>(0.f);
  int part = -1, part_n = 0;
  auto flush = [&]() {
    if (part < 0) return;
    float raw = sum(sum_raw);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) raw += __shfl_xor_sync(0xffffffffu, raw, o);
    const size_t to = (size_t)part * p.N + part_n;
    store(p.part_bias + to * D + chan, sum_b);
    if (lane == 0) p.part_A[to] = raw;
    sum_b = sum_raw = splat<P>(0.f);
  };

  GateScale gc{};
  F bias = splat<P>(0.f), c = splat<P>(0.f);
  int s = 0, fill = kStages - 1;
  uint32_t i = 0;
  for (;; ++i) {
    const float b_own = sigmoid(logits[0]), slope_own = b_own * sigmoid(-logits[0]);
#pragma unroll
    for (int k = 0; k + 1 < kStages - 1; ++k) logits[k] = logits[k + 1];
    logits[kStages - 2] = issue(fill);
    fill = fill + 1 == kStages ? 0 : fill + 1;
    __syncwarp();
    const Tile t = tiles[warp][s];
    if (t.valid == 0) break;
    if (t.flags & kFresh) {
      gc = gate_scale(__ldg(p.A_log + t.n), p.lower_bound);
      bias = load_const<P>(p.dt_bias + (size_t)t.n * D + chan);
      flush();
      part = t.part;
      part_n = t.n;
    }
    F start = splat<P>(0.f);
    if (t.flags & kFirst) {
      if (t.flags & kCut) start = join<D>(p, t.map, t.flags >> kOrder, t.n, chan);
      else if (p.begin) start = load<P>(p.begin + ((size_t)t.slot * p.N + t.n) * D + chan);
    }
    T* const tg = reinterpret_cast<T*>(stages + s * kStage);
    const T* const tx = tg + kElems + chan;
    const T* const td = tx + kElems;
    l.wait(l.full + 8 * s, i / kStages);
    if (t.valid < K) fill_rows<T, D, 3>(tg, t.valid);

    // decays, and the factors w of dg = lam w
    F a[K], w[K];
    F h = load<P>(reinterpret_cast<const float*>(tg + 3 * kElems) + chan);
    const float slope = p.lower_bound * gc.ea;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      // e is kept finite: 1 - sigmoid is e sigmoid, without cancellation, and where the sigmoid
      // is zero so is their product
      const F e = each((load<P>(tg + k * D + chan) + bias) * gc.nz,
                       [](float z) { return fminf(ex2(z), 3e38f); });
      const F sig = each(e + splat<P>(1.f), rcp);
      a[k] = each(sig * gc.l2, ex2);
      w[k] = sig * (e * sig) * (a[k] * slope) * h;
      h = fma(a[k], h, load<P>(tx + k * D) * __shfl_sync(0xffffffffu, b_own, k));
    }
    // a lam of the token behind the tile
    if (p.ring > 1 && (i > 0 || warp % p.ring > 0)) {
      l.wait(l.mine, warp % p.ring > 0 ? i : i - 1);
      c = load<P>(l.inbox + chan);
    }
    if (l.failed) break;
    if (t.flags & kFirst) c = start;
    // a becomes lam
#pragma unroll
    for (int k = K - 1; k >= 0; --k) {
      const F lam = load<P>(td + k * D) + c;
      c = a[k] * lam;
      a[k] = lam;
    }
    if (p.ring > 1) {
      store(l.outbox + chan, c);
      __syncwarp();
      if (lane == 0) mbar_arrive(l.theirs);
    }
    if ((t.flags & (kLast | kEnd)) == (kLast | kEnd) && p.end)
      store(p.end + ((size_t)t.slot * p.N + t.n) * D + chan, c);
    const long long o = t.slot * p.od.stride_b + t.n * p.od.stride_n + t.row * orow + chan;
    T* ox = dx + o;
    T* og = dg + o;
    float dot[K];
    F here_b = splat<P>(0.f), here_raw = splat<P>(0.f);
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const F d = a[k] * w[k];
      if (k < t.valid) {
        store(ox, a[k] * __shfl_sync(0xffffffffu, b_own, k));
        store(og, d);
        here_b = here_b + d;
        here_raw = fma(d, load<P>(tg + k * D + chan) + bias, here_raw);
      }
      dot[k] = sum(a[k] * load<P>(tx + k * D));
      ox += orow;
      og += orow;
    }
    sum_b = sum_b + here_b;
    sum_raw = sum_raw + here_raw;
    constexpr int kEach = 32 / K;  // lanes that end with the same token
    const int k = lane / kEach;
    const float total = warp_sums<K>(dot, lane) * __shfl_sync(0xffffffffu, slope_own, k);
    if (lane % kEach == 0 && k < t.valid)
      dbeta[t.slot * p.bd.stride_b + t.n * p.bd.stride_n + (t.row + k) * p.bd.stride_s] =
          from_f32<T>(total);
    s = s + 1 == kStages ? 0 : s + 1;
  }
  flush();
  if (l.failed) give_up(p, l, tiles[warp], i, lane);
}

// The maps of the segments of cut sequences, one block each: row 0 of a sequence is its start, row
// k + 1 the map of the walk's k-th segment (the last one's is not needed).  A warp takes an eighth
// of the tokens.
template <class T, int D, bool BACKWARD>
__global__ void __launch_bounds__(256) rec_maps_kernel(const __grid_constant__ RecParams p) {
  using S = Shape<D>;
  using F = typename S::F;
  constexpr int V = S::V, P = V / 2;
  __shared__ __align__(16) float sa[8][D], sh[8][D];
  if (p.plan[RH_CHECKSUM] != p.checksum) return;
  const int i = blockIdx.x / p.N, n = blockIdx.x - i * p.N;
  const int4 r0 = __ldg(record(p, i)), r1 = __ldg(record(p, i) + 1);
  const int order = BACKWARD ? r1.z - 1 - r1.y : r1.y;
  if (order + 1 == r1.z) return;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, chan = lane * V;
  const GateScale gc = gate_scale(__ldg(p.A_log + n), p.lower_bound);
  const F bias = load_const<P>(p.dt_bias + (size_t)n * D + chan);
  const kda_view_t& second = BACKWARD ? p.dout : p.x;
  const int each_warp = (r0.z + 7) / 8, lo = min(r0.z, warp * each_warp), hi = min(r0.z, lo + each_warp);
  F pa = splat<P>(1.f), ph = splat<P>(0.f);
  for (int c0 = 0; c0 < hi - lo; c0 += 32) {
    // up to 32 tokens, in the walk's order
    const int count = min(32, hi - lo - c0), first = BACKWARD ? hi - 1 - c0 : lo + c0;
    const int step = BACKWARD ? -1 : 1;
    float b = 0.f;
    if (!BACKWARD && lane < count)
      b = sigmoid(to_f32(__ldg(at<T>(p.beta, r0.x, n, r0.y + first + lane))));
    const T* g = at<T>(p.g, r0.x, n, r0.y + first) + chan;
    const T* x = second.data ? at<T>(second, r0.x, n, r0.y + first) + chan : nullptr;
#pragma unroll 8
    for (int k = 0; k < count; ++k) {
      const F raw = load_const<P>(g) + bias;
      F v = x ? load_const<P>(x) : splat<P>(0.f);
      const F a = each(each(each(raw * gc.nz, ex2) + splat<P>(1.f), rcp) * gc.l2, ex2);
      pa = pa * a;
      if (BACKWARD) {
        ph = a * (ph + v);
      } else {
        ph = fma(a, ph, v * __shfl_sync(0xffffffffu, b, k));
      }
      g += step * p.g.stride_s;
      if (x) x += step * second.stride_s;
    }
  }
  store(&sa[warp][chan], pa);
  store(&sh[warp][chan], ph);
  __syncthreads();
  if (warp > 0) return;
  pa = splat<P>(1.f);
  ph = splat<P>(0.f);
  for (int k = 0; k < 8; ++k) {
    const int w = BACKWARD ? 7 - k : k;
    const F ka = load<P>(&sa[w][chan]);
    pa = pa * ka;
    ph = fma(ka, ph, load<P>(&sh[w][chan]));
  }
  float* m = p.maps + ((size_t)(r1.w + order + 1) * p.N + n) * 2 * D + chan;
  store(m, pa);
  store(m + D, ph);
  if (order == 0) {
    m -= (size_t)p.N * 2 * D;
    store(m, splat<P>(0.f));
    store(m + D, p.begin ? load<P>(p.begin + ((size_t)r0.x * p.N + n) * D + chan) : splat<P>(0.f));
  }
}

// ddt_bias and dA_log: the warps' parts in a fixed order, in fp64.  A block has 32 channels of a
// head (the first one of a head its dA_log too); 32 threads a channel take the segments in turn.
template <int D>
__global__ void __launch_bounds__(1024) rec_params_kernel(const __grid_constant__ RecParams p,
                                                          float* dA_log, float* ddt_bias) {
  __shared__ double red[32][33];
  constexpr int kBlocks = D / 32, K = Shape<D>::K;
  const int n = blockIdx.x / kBlocks, d = (blockIdx.x % kBlocks) * 32 + (threadIdx.x & 31);
  const int lane = threadIdx.x & 31, row = threadIdx.x >> 5, records = p.units / p.N;
  if (p.plan[RH_CHECKSUM] != p.checksum) return;
  double sum = 0, raw = 0;
  for (int k = row; k < records; k += 32) {
    const int4 r0 = __ldg(record(p, k)), r1 = __ldg(record(p, k) + 1);
    const int parts = min(p.ring, (r0.z + K - 1) / K);
    const float* b = p.part_bias + ((size_t)r1.x * p.N + n) * D + d;
#pragma unroll 4
    for (int i = 0; i < parts; ++i) sum += b[(size_t)i * p.N * D];
    if (lane < parts) raw += p.part_A[(size_t)(r1.x + lane) * p.N + n];
  }
  red[row][lane] = sum;
  __syncthreads();
  if (row == 0) {
    for (int k = 1; k < 32; ++k) sum += red[k][lane];
    ddt_bias[(size_t)n * D + d] = (float)sum;
  }
  if (blockIdx.x % kBlocks != 0) return;
  __syncthreads();
  red[row][lane] = raw;
  __syncthreads();
  if (row == 0) {
    for (int k = 1; k < 32; ++k) raw += red[k][lane];
    for (int o = 16; o > 0; o >>= 1) raw += __shfl_down_sync(0xffffffffu, raw, o);
    if (lane == 0) dA_log[n] = (float)raw;
  }
}

template <class T>
__global__ void rec_step_kernel(const T* x, const T* g, const T* beta, const float* h0,
                                const float* A_log, const float* dt_bias, float lower_bound, T* out,
                                float* h1, int N, int D, long long total) {
  const long long i = (long long)blockIdx.x * blockDim.x + threadIdx.x;
  if (i >= total) return;
  const long long row = i / D;
  const int n = (int)(row % N), d = (int)(i % D);
  const GateScale c = gate_scale(A_log[n], lower_bound);
  float t;
  const float sg = gate_sigmoid(c, to_f32(g[i]) + dt_bias[(size_t)n * D + d], &t);
  const float h = ex2(c.l2 * sg) * (h0 ? h0[i] : 0.f) + sigmoid(to_f32(beta[row])) * to_f32(x[i]);
  h1[i] = h;
  out[i] = from_f32<T>(h);
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
  if (!plan_host || !plan_dev || !x || !g || !beta || !A_log || !dt_bias || !workspace)
    return KDA_ERR_NULL;
  st = validate_recurrence_plan(plan_host, n_int32, shape);
  if (st != KDA_OK) return st;
  if (!(lower_bound >= -5.0f && lower_bound <= 0.0f)) return KDA_ERR_LOWER_BOUND;
  size_t need = 0;
  st = kda_recurrence_workspace_size(plan_host, n_int32, backward, &need);
  if (st != KDA_OK) return st;
  if (workspace_bytes < need || (reinterpret_cast<uintptr_t>(workspace) & 255u))
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
  in[7] = dense_range(workspace, need);
  p->plan = plan_dev;
  p->checksum = plan_host[RH_CHECKSUM];
  p->N = shape->N;
  p->units = plan_host[RH_RECORDS] * shape->N;
  p->slot_rows = shape->layout == KDA_LAYOUT_TND ? 0 : shape->S;
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
// that has a unit.
template <class T, int D, bool BACKWARD, class Kernel>
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
  const int blocks = std::min(sms, p.units), rounds = (p.units - 1) / blocks + 1;
  p.ring = B::kWarps;
  while (p.ring > 1 && (B::kWarps % p.ring || p.ring * std::min(rounds, 2) > B::kWarps)) --p.ring;
  if (const char* r = getenv(BACKWARD ? "RB" : "RF")) p.ring = atoi(r);
  if (plan[RH_MAPS]) {
    rec_maps_kernel<T, D, BACKWARD><<<(unsigned)p.units, 256, 0, s>>>(p);
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;
  }
  kernel<<<(unsigned)blocks, 32 * B::kWarps, kSmem, s>>>(p);
  return cudaGetLastError();
}

template <class T, int D>
cudaError_t launch_forward(RecParams& p, const int32_t* plan, cudaStream_t s) {
  static PerDevice once;
  return launch<T, D, false>(rec_forward_kernel<T, D>, once, p, plan, s);
}

template <class T, int D>
cudaError_t launch_backward(RecParams& p, const int32_t* plan, cudaStream_t s) {
  static PerDevice once;
  return launch<T, D, true>(rec_backward_kernel<T, D>, once, p, plan, s);
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
    rec_params_kernel<D><<<(unsigned)shape->N * (D / 32), 1024, 0, s>>>(p, dA_log, ddt_bias);
    return cudaGetLastError();
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
  const long long total = (long long)B * N * D;
  const long long blocks = (total + 255) / 256;
  if (blocks > INT_MAX) return KDA_ERR_SHAPE;
  auto launch = [&](auto* tag) {
    using T = std::remove_pointer_t<decltype(tag)>;
    rec_step_kernel<T><<<(unsigned)blocks, 256, 0, s>>>(
        static_cast<const T*>(x), static_cast<const T*>(g), static_cast<const T*>(beta), state_in,
        A_log, dt_bias, lower_bound, static_cast<T*>(out), state_out, N, D, total);
  };
  if (dtype == KDA_BF16) launch((__nv_bfloat16*)nullptr);
  else if (dtype == KDA_FP16) launch((__half*)nullptr);
  else launch((float*)nullptr);
  return cudaGetLastError() == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
}
