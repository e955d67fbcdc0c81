// scan.cuh — gated linear recurrence over the tokens of a sequence, forward,
// backward and one token at a time.
//
// Per sequence and feature f = (c, t), with gate logits g per channel (shared
// over the group axis) or per (c, t):
//   a_l = sigma(g_l),  h_l = a_l h_{l-1} + (1 - a_l) u_l,  h_{-1} = h0
// Pointwise in the group index, so it commutes with the group's action; convex,
// so |h| <= max(|h0|, |u|) and fp16 outputs stay in range.  Backward:
//   delta_l = dh_l + c_l,  c_{l-1} = a_l delta_l  (c of the last row: dhN),
//   du = (1 - a) delta,  dg = delta (h_{l-1} - u) a (1 - a),  dh0 = c_{-1}
//
// HBM-bound (some ten operations per value), but serial along the sequence.
// An affine step (a, b): h -> a h + b composes associatively, so a block takes a
// tile of rows x 32 features at once: a thread scans R rows of V neighbouring
// features in registers (local states and prefix products), the row groups of
// a warp join by shuffles and the warps through shared memory, one barrier per
// tile; the block then walks to the next tile with the state in shared memory.
// Rows come a tile ahead by cp.async into slots that only the
// copying thread reads (no barrier), so loads never wait for the joins.  Every
// value is read once and written once.  States, products and sums are fp32.
//
// Where whole sequences are too few or too uneven to fill the GPU, or their last
// round fills less than half of it, rows are cut into segments of seg_rows (of the
// last round's sequences, in the last case), a block to each: a first kernel reads u and
// g and reduces each segment to its affine map, and the main kernel's block of a
// segment starts from the maps before it.  That reads the inputs twice, the
// second time partly from L2, for as many more blocks.  (Sequences of one
// segment have no map and cost nothing more.)
//
// The backward pass needs h_{l-1} - u_l.  With fp32 data it reads the forward's h and
// u.  The h of fp16 data is rounded, which moves dg by half a step of h against h - u,
// without bound where they are close (slowly varying features), so the forward of a
// training step writes the difference of its fp32 states in fp32 (kDiff), and the
// backward reads that in the place of u and h: the same bytes there, 4 a value more in
// the forward.  (16 bits of the difference were not enough: their rounding adds to
// dg's own, where the bound is one.)
//
// Measured, fp16: 128 x 3136 x 24 x 4 with channel gates, forward 44 us (173 MB,
// 3.9 TB/s), of a training step 63 (327 MB, 5.2 TB/s), and backward 74 us (346 MB, 4.7
// TB/s) with 9 for its maps; one sequence of 65536 x 96 x 4, 25 us for the maps and 35
// for the scan (151 MB, 252 with the second reading).  DRAM is 40 to 54 % busy and the
// instructions issue on 50 to 60 % of the cycles: the converts, the joins and the walk
// over the rows bound it as much as the loads.
#pragma once

#include <cuda_fp16.h>
#include <stdint.h>

#include "vec.cuh"

namespace feql {

// Tiles in shared memory: one in use, the others on their way.  (A third was
// measured: no faster, 68 against 62 us on 65536 x 96 x 4, forward.)
constexpr int kStages = 2;

struct ScanShape {
  const int *offsets;  // [B + 1] row offsets of packed sequences, or nullptr (dense)
  int64_t N;           // rows of all sequences
  int64_t L;           // rows per sequence (dense)
  int B, F, C, T;
  int FG;              // gates per row: F, or C when shared over the group axis
  int m;               // shared gates: lanes per channel (T / V)
  int FT;              // features per tile
  int ntiles;
  int64_t seg_rows;    // rows of a segment (a multiple of the tiles), 0: sequences are whole
  int64_t slots;       // segment slots: N / seg_rows + B, dense whole + (B - whole) per
  int whole, per;      // dense: the first sequences stay whole, the others' segments
  float *maps;         // [slots][ntiles][2][TX V] affine maps of the segments
};

// Sequence b's rows [s, e), forced into the buffers whatever the offsets hold.
__device__ __forceinline__ void scan_rows(const ScanShape &p, int b, int64_t &s, int64_t &e) {
  if (p.offsets == nullptr) {
    s = b * p.L;
    e = s + p.L;
    return;
  }
  s = p.offsets[b];
  e = p.offsets[b + 1];
  if (s < 0) s = 0;
  if (s > p.N) s = p.N;
  if (e > p.N) e = p.N;
  if (e < s) e = s;
}

// Segment slots: sequence b's k-th segment is slot s / seg_rows + b + k, so that
// the slots of two sequences cannot meet: ceil(len / n) <= e / n - s / n + 1.
// Which sequence a slot belongs to: the last b whose first slot is not behind it,
// by a search over the offsets, 32 candidates a round (the whole warp calls).
__device__ __forceinline__ int scan_slot_owner(const ScanShape &p, int64_t slot) {
  if (p.seg_rows == 0 || slot < p.whole) return static_cast<int>(slot);
  if (p.offsets == nullptr) return p.whole + static_cast<int>(slot - p.whole) / p.per;
  int lo = 0, hi = p.B;  // the owner is in [lo, hi)
  while (hi - lo > 1) {
    const int step = (hi - lo + 31) / 32;
    const int c = lo + static_cast<int>(threadIdx.x & 31) * step;
    bool ok = false;
    if (c < hi) {
      int64_t s, e;
      scan_rows(p, c, s, e);
      ok = s / p.seg_rows + c <= slot;
    }
    // ascending offsets: a run of lanes from 0; whatever they hold, lane 0 stands for lo
    const unsigned m = __ballot_sync(0xffffffffu, ok) | 1u;
    const int last = 31 - __clz(m);
    const int top = lo + (last + 1) * step;
    lo += last * step;
    hi = top < hi ? top : hi;
  }
  return lo;
}

// fp32 states of V neighbouring features (F and f are multiples of V).
template <int V>
__device__ __forceinline__ void load_state(const float *p, float (&v)[V]) {
  Pack<float, V> k;
  k.load(p);
  k.unpack(v);
}
template <int V>
__device__ __forceinline__ void store_state(float *p, const float (&v)[V]) {
  Pack<float, V> k;
  k.pack(v);
  k.store(p);
}

// Row r of a thread's local scan: the prefix product and the state from zero.
template <int V, int GV>
__device__ __forceinline__ void scan_local(int r, const float (&a)[GV], const float (&na)[GV],
                                           const float (&u)[V], float (&P)[GV],
                                           const float (&Pb)[GV], float (&h)[V],
                                           const float (&hb)[V]) {
  float nav[V], av[V], b[V];
  spread(nav, na);
  vec_mul(b, nav, u);
  if (r == 0) {
#pragma unroll
    for (int j = 0; j < GV; ++j) P[j] = a[j];
#pragma unroll
    for (int j = 0; j < V; ++j) h[j] = b[j];
  } else {
    spread(av, a);
    vec_mul(P, a, Pb);
    vec_fma(h, av, hb, b);
  }
}

// The tile loops below come in two forms: kFull, every row of the tile is there
// and nothing is checked, and the general one for a sequence's last tile.
template <bool kFull>
struct ScanRows {
  int n;  // rows of this thread
  __device__ __forceinline__ bool has(int r) const { return kFull || r < n; }
};

// Rows of one operand on their way to a thread: R rows of V values per tile.
// kAsync (4 bytes or more): by cp.async into kStages slots of shared memory;
// else in registers, one tile ahead.
template <typename Ty, int V, int R, int NT, bool kAsync>
struct ScanFeed {
  static constexpr int kAhead = kStages - 1;
  static constexpr int kBytes = kStages * R * NT * V * static_cast<int>(sizeof(Ty));
  Ty *base;  // this thread's values of slot 0
  int slot = 0;
  __device__ __forceinline__ void init(uint8_t *smem) {
    base = reinterpret_cast<Ty *>(smem) + threadIdx.x * V;
  }
  __device__ __forceinline__ Ty *at(int st, int r) { return base + (st * R + r) * NT * V; }
  template <bool kFull>
  __device__ __forceinline__ void issue(int st, const Ty *p, int stride, ScanRows<kFull> rows,
                                        bool skip0 = false) {
#pragma unroll
    for (int r = 0; r < R; ++r)
      if (rows.has(r) && !(r == 0 && skip0)) {
        const uint32_t d = static_cast<uint32_t>(__cvta_generic_to_shared(at(st, r)));
        constexpr int kN = V * static_cast<int>(sizeof(Ty));
        asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(d), "l"(
                         p + static_cast<int64_t>(r) * stride),
                     "n"(kN)
                     : "memory");
      }
  }
  __device__ __forceinline__ void take(int st) { slot = st; }
  __device__ __forceinline__ void get(int r, float (&f)[V]) {
    Pack<Ty, V> k;
    k.load(at(slot, r));
    k.unpack(f);
  }
};

template <typename Ty, int V, int R, int NT>
struct ScanFeed<Ty, V, R, NT, false> {
  static constexpr int kAhead = 1;
  static constexpr int kBytes = 0;
  Pack<Ty, V> now[R], next[R];
  __device__ __forceinline__ void init(uint8_t *) {}
  template <bool kFull>
  __device__ __forceinline__ void issue(int, const Ty *p, int stride, ScanRows<kFull> rows,
                                        bool skip0 = false) {
#pragma unroll
    for (int r = 0; r < R; ++r)
      if (rows.has(r) && !(r == 0 && skip0)) next[r].load(p + static_cast<int64_t>(r) * stride);
  }
  __device__ __forceinline__ void take(int) {
#pragma unroll
    for (int r = 0; r < R; ++r) now[r] = next[r];
  }
  __device__ __forceinline__ void get(int r, float (&f)[V]) { now[r].unpack(f); }
};

template <typename Ty, int V>
constexpr bool scan_async() { return V * sizeof(Ty) >= 4; }

// Shared memory of the feeds: u (or dh with u and h, or with diff), and g unless it is
// shared over the group axis (a two-byte gate per row and channel comes by registers).
template <typename Ty, int V, int R, int NW, bool kShared>
constexpr int scan_feed_bytes(int streams, bool diff) {
  return (streams + (kShared ? 0 : 1)) * ScanFeed<Ty, V, R, NW * 32, scan_async<Ty, V>()>::kBytes +
         (diff ? ScanFeed<float, V, R, NW * 32, true>::kBytes : 0);
}

__device__ __forceinline__ void async_commit() {
  asm volatile("cp.async.commit_group;" ::: "memory");
}
template <int kStages>
__device__ __forceinline__ void async_wait_tile() {  // the oldest tile is there
  asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 2) : "memory");
}

// Block-wide join of the threads' affine maps in scan order (kRev: from the last
// row to the first).  A thread holds the map (A, B) of its rows; GV values of A,
// 1 when its V features share a gate.
template <int F, int NW>
struct ScanJoinSmem {
  float tot[2][NW][2][F];  // [parity][warp][A | B][feature]
  float carry[2][F];       // state that enters the tile of this parity
};

template <int V, int TX, int NW, int GV, bool kRev>
struct ScanJoin {
  static constexpr int RG = 32 / TX;         // row groups of a warp
  using Smem = ScanJoinSmem<TX * V, NW>;
  float ia[GV], ib[V];                       // inclusive map within the warp
  float ea[GV], eb[V];                       // exclusive map within the warp

  __device__ __forceinline__ static int tx() { return threadIdx.x % TX; }
  __device__ __forceinline__ static int pos() {  // the row group's place within the warp
    const int ty = (threadIdx.x & 31) / TX;
    return kRev ? RG - 1 - ty : ty;
  }
  __device__ __forceinline__ static int wpos() {  // the warp's place within the block
    const int w = threadIdx.x >> 5;
    return kRev ? NW - 1 - w : w;
  }
  // the threads that end up with the state after the tile's last row
  __device__ __forceinline__ static bool last() { return pos() == RG - 1 && wpos() == NW - 1; }

  __device__ __forceinline__ static float prev(float v, int o) {
    return kRev ? __shfl_down_sync(0xffffffffu, v, o * TX) : __shfl_up_sync(0xffffffffu, v, o * TX);
  }

  // Scans the warp's row groups and leaves the warp's total for the others.
  __device__ __forceinline__ void scan(Smem &sm, int parity, const float (&A)[GV],
                                       const float (&B)[V]) {
    const int ps = pos();
#pragma unroll
    for (int j = 0; j < GV; ++j) ia[j] = A[j];
#pragma unroll
    for (int j = 0; j < V; ++j) ib[j] = B[j];
#pragma unroll
    for (int o = 1; o < RG; o <<= 1) {
      float pa[GV], pb[V];
#pragma unroll
      for (int j = 0; j < GV; ++j) pa[j] = prev(ia[j], o);
#pragma unroll
      for (int j = 0; j < V; ++j) pb[j] = prev(ib[j], o);
      if (ps >= o) {
#pragma unroll
        for (int j = 0; j < V; ++j) ib[j] = fmaf(ia[GV == 1 ? 0 : j], pb[j], ib[j]);
#pragma unroll
        for (int j = 0; j < GV; ++j) ia[j] *= pa[j];
      }
    }
#pragma unroll
    for (int j = 0; j < GV; ++j) {
      const float q = RG > 1 ? prev(ia[j], 1) : 1.f;
      ea[j] = ps > 0 ? q : 1.f;
    }
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const float q = RG > 1 ? prev(ib[j], 1) : 0.f;
      eb[j] = ps > 0 ? q : 0.f;
    }
    if (NW > 1 && ps == RG - 1) {
#pragma unroll
      for (int j = 0; j < V; ++j) {
        sm.tot[parity][wpos()][0][tx() * V + j] = ia[GV == 1 ? 0 : j];
        sm.tot[parity][wpos()][1][tx() * V + j] = ib[j];
      }
    }
  }

  // After the block's barrier: `in` = the state that enters this thread's rows.
  // The state that enters the tile is `carry` at first, then in shared memory; the
  // last() threads leave the one after the tile there and in `carry`.
  __device__ __forceinline__ void join(Smem &sm, int parity, bool first, float (&carry)[V],
                                       float (&in)[V]) {
    float c[V];
#pragma unroll
    for (int j = 0; j < V; ++j)
      c[j] = (first || NW == 1) ? carry[j] : sm.carry[parity][tx() * V + j];
    if (NW > 1) {
      const int w1 = wpos();
#pragma unroll
      for (int w = 0; w < NW - 1; ++w)
        if (w < w1) {  // the same for a whole warp
          float wa[V], wb[V];
          load_state<V>(&sm.tot[parity][w][0][tx() * V], wa);
          load_state<V>(&sm.tot[parity][w][1][tx() * V], wb);
          vec_fma(c, wa, c, wb);
        }
    }
#pragma unroll
    for (int j = 0; j < V; ++j) in[j] = fmaf(ea[GV == 1 ? 0 : j], c[j], eb[j]);
#pragma unroll
    for (int j = 0; j < V; ++j) c[j] = fmaf(ia[GV == 1 ? 0 : j], c[j], ib[j]);
    if (NW == 1) {  // from the last row group's lanes to all
      const int src = (kRev ? 0 : RG - 1) * TX + tx();
#pragma unroll
      for (int j = 0; j < V; ++j) carry[j] = __shfl_sync(0xffffffffu, c[j], src);
    } else if (last()) {
#pragma unroll
      for (int j = 0; j < V; ++j) {
        carry[j] = c[j];
        sm.carry[parity ^ 1][tx() * V + j] = c[j];
      }
    }
  }
};

// Rows that belong to no sequence (before the first offset, behind the last)
// are zeroed in the outputs, so that what consumes them sees numbers: by all
// blocks, those without a segment among them, each for its features.  (The blocks
// of the first and last sequence alone took 420 us for 401408 x 24 x 4 of which
// sequences cover 4000 rows.)
template <typename Ty, int V, int TY>
__device__ __forceinline__ void scan_zero_rest(const ScanShape &p, int64_t slot, int ty, Ty *out,
                                               int width, int col, bool live) {
  if (p.offsets == nullptr || !live) return;
  int64_t s, e, last;
  scan_rows(p, 0, s, e);
  scan_rows(p, p.B - 1, e, last);
  Pack<Ty, V> z;
  z.zero();
  const int64_t step = p.slots * TY, first = slot * TY + ty;
  for (int64_t r = first; r < s; r += step) z.store(out + r * width + col);
  for (int64_t r = last + first; r < p.N; r += step) z.store(out + r * width + col);
}

// Blocks of NW warps that an SM holds: by registers (128 a thread, 80 where the
// walks keep little).
constexpr int scan_blocks(int NW, bool lean) { return NW == 8 ? (lean ? 3 : 2) : 16; }

// What a block works on: sequence b, its segment seg of nseg (a sequence without
// rows has one, empty), feature tile; a thread's features f .. f + V, and its row
// group ty.
template <int V, int TX, int NW, bool kShared>
struct ScanPlace {
  int b, seg, nseg, tile, tx, ty, f, gf;
  int64_t slot;
  bool live;                  // this thread's features exist
  bool work;                  // the slot holds a segment
  int64_t s, e, len, r0, r1;  // rows of the sequence; the segment's within it
  __device__ __forceinline__ explicit ScanPlace(const ScanShape &p, int first = 0) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    tx = lane % TX;
    ty = warp * (32 / TX) + lane / TX;
    slot = first + blockIdx.x / p.ntiles;
    tile = blockIdx.x % p.ntiles;
    f = tile * p.FT + tx * V;
    live = tx * V < p.FT && f < p.F;
    if (!live) f = tile * p.FT;  // a lane without features reads another's and writes nothing
    gf = kShared ? f / p.T : f;
    b = scan_slot_owner(p, slot);
    scan_rows(p, b, s, e);
    len = e - s;
    seg = 0;
    nseg = 1;
    r0 = 0;
    r1 = len;
    if (p.seg_rows != 0 && slot >= p.whole) {
      seg = static_cast<int>(p.offsets == nullptr ? (slot - p.whole) % p.per
                                                  : slot - (s / p.seg_rows + b));
      nseg = static_cast<int>((len + p.seg_rows - 1) / p.seg_rows);
      if (nseg < 1) nseg = 1;
      r0 = seg * p.seg_rows;
      r1 = r0 + p.seg_rows < len ? r0 + p.seg_rows : len;
    }
    work = seg >= 0 && seg < nseg;
  }
  // The map of segment q, this thread's features: A at [0][..], B at [1][..].
  __device__ __forceinline__ float *map(const ScanShape &p, int q) const {
    return p.maps + ((slot - seg + q) * p.ntiles + tile) * 2 * TX * V + tx * V;
  }
};

// kRev: the gradient's maps c -> A c + B, B from dh; else the states', B from u.
// Each row group walks its share of the segment's rows by itself, R at a time
// with the next R on their way, and the groups join once at the end.
template <typename Ty, int V, int TX, int NW, bool kShared, bool kRev>
__global__ void __launch_bounds__(NW * 32, 2)
scan_maps_kernel(const Ty *__restrict__ x, const Ty *__restrict__ g, const ScanShape p) {
  constexpr int GV = kShared ? 1 : V;
  constexpr int TY = NW * 32 / TX, R = 4;
  using J = ScanJoin<V, TX, NW, GV, kRev>;
  __shared__ __align__(16) typename J::Smem sm;
  // the main kernel's blocks may start: those of whole sequences run, the others
  // bring their first tile and wait
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const ScanPlace<V, TX, NW, kShared> at(p, p.whole);
  // (the same for a whole block; a sequence's last segment in scan order has no use)
  if (!at.work || at.seg == (kRev ? 0 : at.nseg - 1)) return;
  const int64_t rows = at.r1 - at.r0;
  const int64_t share = (rows + TY - 1) / TY;
  const int64_t l0 = at.r0 + at.ty * share;
  const int64_t l1 = l0 + share < at.r1 ? l0 + share : at.r1;
  float A[GV], B[V];
#pragma unroll
  for (int j = 0; j < GV; ++j) A[j] = 1.f;
#pragma unroll
  for (int j = 0; j < V; ++j) B[j] = 0.f;
  const int64_t n = l1 > l0 ? l1 - l0 : 0;
  const int64_t first = at.s + (kRev ? l1 - 1 : l0);
  const Ty *px = x + first * p.F + at.f, *pg = g + first * p.FG + at.gf;
  const int sx = kRev ? -p.F : p.F, sg = kRev ? -p.FG : p.FG;
  Pack<Ty, V> rx[2][R];
  Pack<Ty, GV> rg[2][R];
  auto fetch = [&](int h, auto rows) {
#pragma unroll
    for (int r = 0; r < R; ++r)
      if (rows.has(r)) {
        rx[h][r].load(px + static_cast<int64_t>(r) * sx);
        rg[h][r].load(pg + static_cast<int64_t>(r) * sg);
      }
    px += static_cast<int64_t>(R) * sx;
    pg += static_cast<int64_t>(R) * sg;
  };
  auto walk = [&](int h, auto rows) {
#pragma unroll
    for (int r = 0; r < R; ++r)
      if (rows.has(r)) {
        float xv[V], gv[GV], a[GV], na[GV], av[V], nav[V];
        rx[h][r].unpack(xv);
        rg[h][r].unpack(gv);
#pragma unroll
        for (int j = 0; j < GV; ++j) sigmoid_pair<sizeof(Ty) == 2>(gv[j], a[j], na[j]);
        spread(av, a);
        if constexpr (kRev) {
          vec_add(B, B, xv);
          vec_mul(B, B, av);
        } else {
          spread(nav, na);
          vec_mul(xv, nav, xv);
          vec_fma(B, av, B, xv);
        }
        vec_mul(A, A, a);
      }
  };
  auto some = [&](int64_t k) {
    return ScanRows<false>{k >= n ? 0 : n - k < R ? static_cast<int>(n - k) : R};
  };
  const ScanRows<true> all{R};
  fetch(0, some(0));
  fetch(1, some(R));
  int64_t k = 0;
  for (; k + 4 * R <= n; k += 2 * R) {  // nothing to check
    walk(0, all);
    fetch(0, all);
    walk(1, all);
    fetch(1, all);
  }
  for (; k < n; k += 2 * R) {
    walk(0, some(k));
    fetch(0, some(k + 2 * R));
    walk(1, some(k + R));
    fetch(1, some(k + 3 * R));
  }
  // joined: the map's constant part is where a zero state goes, its factor the product
  J join;
  join.scan(sm, 0, A, B);
  if (NW > 1) __syncthreads();
  float carry[V] = {}, in[V], prod[V];
#pragma unroll
  for (int j = 0; j < V; ++j) prod[j] = 1.f;
  join.join(sm, 0, true, carry, in);
  if (NW > 1) {
#pragma unroll
    for (int w = 0; w < NW - 1; ++w)
#pragma unroll
      for (int j = 0; j < V; ++j) prod[j] *= sm.tot[0][w][0][at.tx * V + j];
  }
  if (J::last() && at.live) {
    float *to = at.map(p, at.seg);
#pragma unroll
    for (int j = 0; j < V; ++j) {
      to[j] = prod[j] * join.ia[GV == 1 ? 0 : j];
      to[TX * V + j] = carry[j];
    }
  }
}

// The state that enters segment seg: the maps before it (kRev: behind it, from
// the sequence's last one), applied to the state at the sequence's end.
template <bool kRev, int V, int TX, int NW, bool kShared>
__device__ __forceinline__ void scan_enter(const ScanShape &p,
                                           const ScanPlace<V, TX, NW, kShared> &at,
                                           float (&carry)[V]) {
  const int n = kRev ? at.nseg - 1 - at.seg : at.seg;
#pragma unroll 8
  for (int i = 0; i < n; ++i) {
    const float *m = at.map(p, kRev ? at.nseg - 1 - i : i);
    float A[V], B[V];
    load_state<V>(m, A);
    load_state<V>(m + TX * V, B);
    vec_fma(carry, A, carry, B);
  }
}

// Before the first use of the maps: their kernel has finished.  Every block of a
// cut sequence waits, and there are some, so the grid never ends before it.
__device__ __forceinline__ void scan_wait_maps(const ScanShape &p) {
  if (p.seg_rows != 0) asm volatile("griddepcontrol.wait;" ::: "memory");
}

// A row's gates; rows that are not there pass the state on: a = 1, 1 - a = 0.
template <typename Ty, int GV, class Feed>
__device__ __forceinline__ void scan_row_gates(Feed &fg, int r, bool there, float (&a)[GV],
                                               float (&na)[GV]) {
  if (there) {
    float gv[GV];
    fg.get(r, gv);
#pragma unroll
    for (int j = 0; j < GV; ++j) sigmoid_pair<sizeof(Ty) == 2>(gv[j], a[j], na[j]);
  } else {
#pragma unroll
    for (int j = 0; j < GV; ++j) { a[j] = 1.f; na[j] = 0.f; }
  }
}

// kDiff: writes h_{l-1} - u_l too.
template <typename Ty, int V, int TX, int R, int NW, bool kShared, bool kDiff>
__global__ void __launch_bounds__(NW * 32, scan_blocks(NW, kShared && V > 1))
scan_fwd_kernel(const Ty *__restrict__ u, const Ty *__restrict__ g, const float *__restrict__ h0,
                Ty *__restrict__ h, float *__restrict__ hN, float *__restrict__ diff,
                const ScanShape p) {
  constexpr int GV = kShared ? 1 : V;
  constexpr int TY = NW * 32 / TX, RT = TY * R, NT = NW * 32;
  constexpr bool kAsync = scan_async<Ty, V>(), kLean = kShared && V > 1;
  using J = ScanJoin<V, TX, NW, GV, false>;
  extern __shared__ __align__(16) uint8_t feeds[];
  __shared__ __align__(16) typename J::Smem sm;
  ScanFeed<Ty, V, R, NT, kAsync> fu;
  ScanFeed<Ty, GV, R, NT, kAsync && !kShared> fg;
  fu.init(feeds);
  fg.init(feeds + fu.kBytes);
  const ScanPlace<V, TX, NW, kShared> at(p);
  if (!at.work) {
    scan_zero_rest<Ty, V, TY>(p, at.slot, at.ty, h, p.F, at.f, at.live);
    scan_wait_maps(p);
    return;
  }
  const int64_t rows = at.r1 - at.r0;
  const int steps = static_cast<int>((rows + RT - 1) / RT);
  const int whole = static_cast<int>(rows / RT);  // tiles with all their rows
  const int64_t row = at.s + at.r0 + at.ty * R;   // this thread's first row of the next load
  const Ty *pu = u + row * p.F + at.f, *pg = g + row * p.FG + at.gf;
  const int64_t du = static_cast<int64_t>(RT) * p.F, dg = static_cast<int64_t>(RT) * p.FG;
  // rows of tile i that are this thread's
  auto have = [&](int i) {
    const int64_t n = rows - (static_cast<int64_t>(i) * RT + at.ty * R);
    return n < 0 ? 0 : (n < R ? static_cast<int>(n) : R);
  };
  auto issue_u = [&](int i) {
    if (i < whole) fu.issue(i % kStages, pu, p.F, ScanRows<true>{R});
    else if (i < steps) fu.issue(i % kStages, pu, p.F, ScanRows<false>{have(i)});
    pu += du;
  };
  auto issue_g = [&](int i) {
    if (i < whole) fg.issue(i % kStages, pg, p.FG, ScanRows<true>{R});
    else if (i < steps) fg.issue(i % kStages, pg, p.FG, ScanRows<false>{have(i)});
    pg += dg;
  };
#pragma unroll
  for (int i = 0; i < kStages - 1; ++i) {
    if (i < fu.kAhead) issue_u(i);
    if (i < fg.kAhead) issue_g(i);
    async_commit();
  }
  float carry[V] = {};
  if (h0 != nullptr) load_state<V>(h0 + static_cast<int64_t>(at.b) * p.F + at.f, carry);
  if (at.slot >= p.whole) scan_wait_maps(p);
  scan_enter<false>(p, at, carry);
  Ty *ph = h + row * p.F + at.f;
  float *pq = kDiff ? diff + row * p.F + at.f : nullptr;
  auto tile = [&](int i, auto rows_of) {
    // the map of the thread's rows: a gate per channel is kept and u read again
    // for the second walk, a gate per value the local states and products
    constexpr int K = kLean ? 1 : R;
    float a[R][GV], na[R][GV], P[K][GV], hl[K][V];
#pragma unroll
    for (int r = 0; r < R; ++r) {
      float uv[V] = {};
      scan_row_gates<Ty, GV>(fg, r, rows_of.has(r), a[r], na[r]);
      if (rows_of.has(r)) fu.get(r, uv);
      const int k = kLean ? 0 : r, kb = kLean || r == 0 ? 0 : r - 1;
      scan_local<V, GV>(r, a[r], na[r], uv, P[k], P[kb], hl[k], hl[kb]);
    }
    J join;
    float in[V];
    join.scan(sm, i & 1, P[K - 1], hl[K - 1]);
    if (NW > 1) __syncthreads();
    join.join(sm, i & 1, i == 0, carry, in);
    if (!at.live) return;
    float before[V];
#pragma unroll
    for (int j = 0; j < V; ++j) before[j] = in[j];
#pragma unroll
    for (int r = 0; r < R; ++r)
      if (rows_of.has(r)) {
        float o[V];
        if constexpr (kLean) {
          float uv[V], av[V], nav[V];
          fu.get(r, uv);
          if constexpr (kDiff) {
            float q[V];
            vec_sub(q, in, uv);
            store_state<V>(pq + static_cast<int64_t>(r) * p.F, q);
          }
          spread(av, a[r]);
          spread(nav, na[r]);
          vec_mul(uv, nav, uv);
          vec_fma(in, av, in, uv);
#pragma unroll
          for (int j = 0; j < V; ++j) o[j] = in[j];
        } else {
          float pv[V];
          spread(pv, P[kLean ? 0 : r]);
          vec_fma(o, pv, in, hl[kLean ? 0 : r]);
          if constexpr (kDiff) {
            float uv[V];
            fu.get(r, uv);
            vec_sub(uv, before, uv);
            store_state<V>(pq + static_cast<int64_t>(r) * p.F, uv);
#pragma unroll
            for (int j = 0; j < V; ++j) before[j] = o[j];
          }
        }
        Pack<Ty, V> k;
        k.pack(o);
        k.store(ph + static_cast<int64_t>(r) * p.F);
      }
  };
  for (int i = 0; i < steps; ++i, ph += du, pq += kDiff ? du : 0) {
    async_wait_tile<kStages>();
    fu.take(i % kStages);
    fg.take(i % kStages);
    issue_u(i + fu.kAhead);
    issue_g(i + fg.kAhead);
    async_commit();
    if (i < whole) tile(i, ScanRows<true>{R});
    else tile(i, ScanRows<false>{have(i)});
  }
  if (hN != nullptr && at.live && at.seg == at.nseg - 1 && J::last())
    store_state<V>(hN + static_cast<int64_t>(at.b) * p.F + at.f, carry);
  scan_zero_rest<Ty, V, TY>(p, at.slot, at.ty, h, p.F, at.f, at.live);
}

// diff: h_{l-1} - u_l as the forward wrote it (kDiff); else from u and h, the forward's
// output, where the state before the first row of a sequence is h0.
template <typename Ty, int V, int TX, int R, int NW, bool kShared, bool kDiff>
__global__ void __launch_bounds__(NW * 32, scan_blocks(NW, false))
scan_bwd_kernel(const Ty *__restrict__ dh, const Ty *__restrict__ u, const Ty *__restrict__ g,
                const Ty *__restrict__ h, const float *__restrict__ h0,
                const float *__restrict__ diff, const float *__restrict__ dhN,
                Ty *__restrict__ du, Ty *__restrict__ dg, float *__restrict__ dh0,
                const ScanShape p) {
  constexpr int GV = kShared ? 1 : V;
  constexpr int TY = NW * 32 / TX, RT = TY * R, NT = NW * 32;
  constexpr bool kAsync = scan_async<Ty, V>();
  using J = ScanJoin<V, TX, NW, GV, true>;
  extern __shared__ __align__(16) uint8_t feeds[];
  __shared__ __align__(16) typename J::Smem sm;
  ScanFeed<Ty, V, R, NT, kAsync> fu, fd, fh;
  ScanFeed<float, V, R, NT, true> fq;
  ScanFeed<Ty, GV, R, NT, kAsync && !kShared> fg;
  fd.init(feeds);
  if constexpr (kDiff) {
    fq.init(feeds + fd.kBytes);
    fg.init(feeds + fd.kBytes + fq.kBytes);
  } else {
    fu.init(feeds + fd.kBytes);
    fh.init(feeds + 2 * fd.kBytes);
    fg.init(feeds + 3 * fd.kBytes);
  }
  const ScanPlace<V, TX, NW, kShared> at(p);
  auto zero_rest = [&]() {
    scan_zero_rest<Ty, V, TY>(p, at.slot, at.ty, du, p.F, at.f, at.live);
    scan_zero_rest<Ty, GV, TY>(p, at.slot, at.ty, dg, p.FG, at.gf,
                               at.live && (!kShared || at.tx % p.m == 0));
  };
  if (!at.work) {
    zero_rest();
    scan_wait_maps(p);
    return;
  }
  const int64_t rows = at.r1 - at.r0;
  const int steps = static_cast<int>((rows + RT - 1) / RT);
  const int part = steps - static_cast<int>(rows / RT);  // 1: the first step's tile lacks rows
  // step i takes tile steps - 1 - i: the tiles run from the segment's end
  const int64_t row = at.s + at.r0 + static_cast<int64_t>(steps - 1) * RT + at.ty * R;
  const Ty *pd = dh + row * p.F + at.f;
  const float *pq = kDiff ? diff + row * p.F + at.f : nullptr;
  // the rows before; before the sequence's first row stands h0
  const Ty *pu = kDiff ? nullptr : u + row * p.F + at.f;
  const Ty *ph = kDiff ? nullptr : h + (row - 1) * p.F + at.f;
  const bool top = at.seg == 0 && at.ty == 0;
  const Ty *pg = g + row * p.FG + at.gf;
  const int64_t step = static_cast<int64_t>(RT) * p.F, gstep = static_cast<int64_t>(RT) * p.FG;
  auto have = [&]() {  // this thread's rows of the last tile
    const int64_t n = rows - (static_cast<int64_t>(steps - 1) * RT + at.ty * R);
    return n < 0 ? 0 : (n < R ? static_cast<int>(n) : R);
  };
  auto issue_x = [&](int i) {
    if (i < steps) {
      const int st = i % kStages;
      const bool none = top && i == steps - 1;
      auto rows_of = [&](auto n) {
        fd.issue(st, pd, p.F, n);
        if constexpr (kDiff) {
          fq.issue(st, pq, p.F, n);
        } else {
          fu.issue(st, pu, p.F, n);
          fh.issue(st, ph, p.F, n, none);
        }
      };
      if (i < part) rows_of(ScanRows<false>{have()});
      else rows_of(ScanRows<true>{R});
    }
    pd -= step;
    if constexpr (kDiff) {
      pq -= step;
    } else {
      pu -= step;
      ph -= step;
    }
  };
  auto issue_g = [&](int i) {
    if (i < part) fg.issue(i % kStages, pg, p.FG, ScanRows<false>{have()});
    else if (i < steps) fg.issue(i % kStages, pg, p.FG, ScanRows<true>{R});
    pg -= gstep;
  };
#pragma unroll
  for (int i = 0; i < kStages - 1; ++i) {
    if (i < fd.kAhead) issue_x(i);
    if (i < fg.kAhead) issue_g(i);
    async_commit();
  }
  float carry[V] = {}, start[V] = {};
  const int64_t state = static_cast<int64_t>(at.b) * p.F + at.f;
  if (dhN != nullptr) load_state<V>(dhN + state, carry);
  if (!kDiff && top && h0 != nullptr) load_state<V>(h0 + state, start);
  if (at.slot >= p.whole) scan_wait_maps(p);
  scan_enter<true>(p, at, carry);
  Ty *pdu = du + row * p.F + at.f, *pdg = dg + row * p.FG + at.gf;
  auto tile = [&](int i, auto rows_of) {
    float a[R][GV], na[R][GV], A[GV], d[R][V], Bc[V] = {}, cin[V];
#pragma unroll
    for (int j = 0; j < GV; ++j) A[j] = 1.f;
#pragma unroll
    for (int r = R - 1; r >= 0; --r) {
      float av[V];
      scan_row_gates<Ty, GV>(fg, r, rows_of.has(r), a[r], na[r]);
#pragma unroll
      for (int j = 0; j < V; ++j) d[r][j] = 0.f;
      if (rows_of.has(r)) fd.get(r, d[r]);
      spread(av, a[r]);
      vec_add(Bc, Bc, d[r]);
      vec_mul(Bc, Bc, av);
      vec_mul(A, A, a[r]);
    }
    J join;
    join.scan(sm, i & 1, A, Bc);
    if (NW > 1) __syncthreads();
    join.join(sm, i & 1, i == 0, carry, cin);
#pragma unroll
    for (int r = R - 1; r >= 0; --r) {
      float off[V] = {}, o[V], gg[V], av[V], nav[V], og[GV];  // off: h_{l-1} - u_l
      if constexpr (kDiff) {
        if (rows_of.has(r)) fq.get(r, off);
      } else {
        float uv[V] = {};
        if (rows_of.has(r)) {
          fu.get(r, uv);
          fh.get(r, off);
        }
        if (r == 0 && top && i == steps - 1) {
#pragma unroll
          for (int j = 0; j < V; ++j) off[j] = start[j];
        }
        vec_sub(off, off, uv);
      }
      spread(av, a[r]);
      spread(nav, na[r]);
      vec_add(d[r], d[r], cin);  // delta
      vec_mul(o, nav, d[r]);
      vec_mul(cin, av, d[r]);
      if constexpr (kShared) {
        vec_mul(gg, d[r], off);
        float gsum = gg[0];
#pragma unroll
        for (int j = 1; j < V; ++j) gsum += gg[j];
        gsum *= a[r][0] * na[r][0];
        // a channel's T features sit in m neighbouring lanes
        float sum = gsum;
        for (int k = 1; k < p.m; ++k) sum += __shfl_down_sync(0xffffffffu, gsum, k);
        og[0] = sum;
      } else {
        vec_mul(gg, o, off);
        vec_mul(gg, gg, av);
#pragma unroll
        for (int j = 0; j < V; ++j) og[GV == 1 ? 0 : j] = gg[j];
      }
      if (rows_of.has(r) && at.live) {
        Pack<Ty, V> k;
        k.pack(o);
        k.store(pdu + static_cast<int64_t>(r) * p.F);
        Pack<Ty, GV> kg;
        kg.pack(og);
        if (!kShared || at.tx % p.m == 0) kg.store(pdg + static_cast<int64_t>(r) * p.FG);
      }
    }
  };
  for (int i = 0; i < steps; ++i, pdu -= step, pdg -= gstep) {
    async_wait_tile<kStages>();
    fd.take(i % kStages);
    if constexpr (kDiff) {
      fq.take(i % kStages);
    } else {
      fu.take(i % kStages);
      fh.take(i % kStages);
    }
    fg.take(i % kStages);
    issue_x(i + fd.kAhead);
    issue_g(i + fg.kAhead);
    async_commit();
    if (i < part) tile(i, ScanRows<false>{have()});
    else tile(i, ScanRows<true>{R});
  }
  if (dh0 != nullptr && at.live && at.seg == 0 && J::last()) store_state<V>(dh0 + state, carry);
  zero_rest();
}

// One token of each of B sequences: h = a h + (1 - a) u on the fp32 states in
// place, and the new state rounded to the data type.  Latency-bound: one value
// per thread, one launch.
template <typename Ty>
__global__ void __launch_bounds__(256)
scan_step_kernel(const Ty *__restrict__ u, const Ty *__restrict__ g, float *__restrict__ state,
                 Ty *__restrict__ h, int64_t n, int T) {
  const int64_t step = static_cast<int64_t>(gridDim.x) * blockDim.x;
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x; i < n; i += step) {
    float a, na;
    // T = 1 for a gate per (c, t)
    sigmoid_pair<sizeof(Ty) == 2>(widen(g[i / T]), a, na);
    const float v = fmaf(a, state[i], na * widen(u[i]));
    state[i] = v;
    h[i] = narrow<Ty>(v);
  }
}

}  // namespace feql
