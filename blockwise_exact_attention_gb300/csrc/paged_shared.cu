// Attention of one new token per request, where groups of requests have their
// first keys in common: those are read once for the whole group.
//
// The keys of request r are a prefix that its group shares and its own rest. The
// prefix is a product of many queries with the same keys: the queries of all the
// group's requests, and of the g = h / h_kv heads that read a K/V head, are the rows
// of one matrix, so it runs like the forward, on the tensor cores:
//   S = Q K^T, P = exp2(scale S - m) with a running maximum m, O += P V, l += sum P.
// Its bytes are the prefix once, its flops 6 d a (query row, key), P being two terms: from
// 190 rows a K/V head on the products are the bound, not HBM. The rest is paged_decode's kernel, told
// where each request's own keys begin. A last kernel joins the two by their maxima and
// sums, in a fixed order.
//
// Only whole tiles of 128 keys count as prefix, and only up to the shortest request of
// the group and the first page that lies outside the cache: what is left over is the
// requests' own, as are all keys of a request whose table names other pages there. So
// the kernel has no masks, and what the shared path leaves out the other one computes.
//
// The prefix kernel. A UNIT is up to 256 query rows of one (group, K/V head), its keys
// a list of tiles; the units' tiles, one after another, are cut into runs of equal
// cost, one per CTA. Warps as in the forward: 0-3 and 4-7 softmax of 128 rows each
// (thread = row), 8 and 10 load K and V tiles by TMA, boxes of a page, 9 issues the
// products. With more than 128 rows both halves meet every tile; with up to 128 rows
// both have the same rows and take the tiles in turn, which keeps the tensor core and
// the exponentials overlapped, and each half writes its own part.
//
// P enters the second product as two bf16 terms, 16 bits of it (cut off, then the rest
// rounded; P's last bit is set, so that something is left of it and an infinite value
// stays infinite). One rounded term, as in the forward, is off by up to 2^-8 of each
// weight, on average as much as a bf16 output's own rounding (0.0024 of its size against
// fp64, 0.0017 with two), and takes 64 requests behind 32k keys from 75.2 to 61.3 us, 256
// behind 16k from 119 to 97, 96 in three groups from 73.2 to 69.7: paged_decode's weights
// have all their bits, and a call that takes its place gives the same. The sums of weights
// are in fp32, those of P V in the tensor core's accumulator for some tiles and in fp32 above.
//
// Order of the launches: the setup, which finds what each group shares; the rest's
// kernel; the prefix; the join. The prefix kernel waits for nothing when it starts: it
// is launched once every CTA of the rest's kernel has begun and has waited for the
// setup, and its CTAs start as those of the rest's end, SM by SM. It waits for that
// kernel before it ends, so that the join finds both done.
//
// Measured (GPU time, three sets of inputs in turn; h / h_kv 32 / 8, d = 128): 64
// requests behind 32k shared keys, up to 1k own ones each, 75 us, where 188 MB take
// 28 and the products 27 (behind 16k 67 us, 490 without sharing); 256 behind 16k, up
// to 600 own, 120 us (27, 54). Of the latter 5 go to the setup, 29 to the rest (its
// bytes at 5 TB/s), 78 to the prefix and 8 to the join. A step of a unit takes 2.4
// us, 1.5 of them (3072 cycles) the tensor core's: the chain S, maximum, exponentials
// and their terms, P V of two halves in turn. Before a CTA's first scores 4.5 us pass
// (schedule, queries, keys, cold instructions), and its part takes 3 to write, all
// CTAs' 20 MB at once. Tried without gain, with one term: two threads to a row (640
// threads at 96 registers), which meet to exchange maxima; runs that get shorter from
// CTA to CTA, as these start up to 10 us apart (most of them at the end of that); the
// rest's kernel on 64-112 SMs and the prefix beside it (both take longer); tiles called
// into L2 a step ahead.
#include <cuda_bf16.h>

#include "launch_cache.cuh"
#include "paged_shared.cuh"
#include "ptx.cuh"

namespace bea {
namespace {

constexpr int kTile = 128;      // keys of a tile, rows of a half
constexpr int kUnitRows = 256;  // of a unit
constexpr int kMaxCtas = 160;   // one per SM
constexpr int kThreads = 384;
// As in the forward: 256 threads at 200 registers and 128 at 104 are what 384 are launched with.
constexpr int kRegsLaunch = 168, kRegsSoftmax = 200, kRegsOther = 104;
static_assert(256 * kRegsSoftmax + 128 * kRegsOther == kThreads * kRegsLaunch, "register split");
constexpr int kKWarp = 8, kMmaWarp = 9, kVWarp = 10;
// The sum of weights of a part without keys, whose O is not written. (Of keys without a maximum it is 0 or NaN, and NaN belongs
// to the result.)
constexpr float kNoKeys = -1.f;
constexpr float kRescale = 8.f;  // log2: O is rescaled only when a maximum grows by more
constexpr uint32_t kPReadyBar = 1, kPReadyThreads = 128 + 32, kBothBar = 3;
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
// Of a unit besides its steps, in steps: a run in two units fetches queries and writes parts twice. A fifth of a run, within these
// bounds. (2 and 5 everywhere, runs of 27 steps, 256 requests behind 16k keys: 123.0, 119.5 us; of 13, 64 behind 32k: the same;
// of 5, 96 in three groups: 72.2, 75.3 us, 16 behind 4k: 25.4, 27.2 us.)
constexpr int kLeastUnitCost = 2, kMostUnitCost = 5;
// A run's cut is moved by up to so many steps (and a quarter of a run) to a unit's border.
constexpr int kSnap = 2;
// Tiles that are summed in one accumulator before it joins the part in memory, in fp32: the tensor core cuts off what it adds up.
// Values of 1, runs of 216 tiles: one accumulator 1.5e-4 low, 526 us; 64 tiles 4.1e-5, 554 us; 16 7e-6, 640 us. A weight is off by
// up to 3e-5, a bf16 output by 4e-3.
constexpr int kFlushF32 = 16, kFlushBf16 = 64;

template <int D>
struct Cfg {
  static constexpr int kBoxes = D / 64;
  static constexpr int kTileBytes = kTile * D * 2;
  static constexpr int kStages = D == 128 ? 2 : 4;
  static constexpr int kKOff = 2 * kTileBytes;
  static constexpr int kVOff = kKOff + kStages * kTileBytes;
  static constexpr int kBarOff = kVOff + kStages * kTileBytes;
  static constexpr int kNumBars = 1 + 4 * kStages + 2 + 2 + 1;
  static constexpr int kTableOff = kBarOff + kNumBars * 8 + 16;
  static constexpr int kGroupOff = (kTableOff + 2 * (kMaxGroups + 1) * 4 + 15) / 16 * 16;
  static constexpr int kFirstOff = kGroupOff + kMaxGroups * 16;
  static constexpr int kUnitOff = kFirstOff + 128;  // each softmax warp's unit, 64 bytes
  static constexpr int kSmem = kUnitOff + 8 * 64 + 1024 /*alignment*/;
  static constexpr uint32_t kIdescS = idesc_bf16_f32(128, 128, false, false);
  static constexpr uint32_t kIdescPV = idesc_bf16_f32(128, D, false, true);
  static constexpr uint32_t kVLbo = 64 * 128 * 2;
};

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_wait_all() { asm volatile("cp.async.wait_all;" ::: "memory"); }

// 32 bytes, a sector of memory, by one thread.
__device__ __forceinline__ void store_sector(float* to, const uint32_t* x) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(to), "r"(x[0]), "r"(x[1]), "r"(x[2]), "r"(x[3]),
               "r"(x[4]), "r"(x[5]), "r"(x[6]), "r"(x[7])
               : "memory");
}

// ---- schedule ----------------------------------------------------------------------

// A group as the setup finds it: its rows, the first of them that has keys, the tiles that are shared.
struct alignas(16) Group {
  int row0, rows, owner, tiles;
};

// Of a group: units of two halves, rows of a last unit of one half (0: none), and steps, a step being a tile of a unit of
// two halves or two tiles of the other.
struct Shape {
  int rows, twos, one, tiles, one_steps;
  __device__ Shape(int q_rows, int t) : rows(q_rows), tiles(t) {
    twos = q_rows / kUnitRows;
    one = q_rows - twos * kUnitRows;
    if (one > kTile) one = 0, ++twos;
    if (t == 0) twos = one = 0;
    one_steps = one > 0 ? (t + 1) / 2 : 0;
  }
  // what a K/V head's units cost: their steps, and behind them unit_cost each
  __device__ int cost(int unit_cost) const { return twos * (tiles + unit_cost) + (one > 0 ? one_steps + unit_cost : 0); }
  __device__ int part_rows() const { return twos * kUnitRows + 2 * one; }  // rows of its parts
};

// Where the groups' costs and parts' rows begin, [groups + 1] each; and the runs.
struct First;
struct Schedule {
  const int *costs, *rows;
  const Group* groups;
  int n_groups, heads;  // heads: query heads of a K/V head
  int total, ctas, snap, unit;  // unit: a unit's cost besides its steps

  __device__ Schedule(const int* c, const int* r, const Group* g, int n, int query_heads, int most_ctas, int unit_cost)
      : costs(c), rows(r), groups(g), n_groups(n), heads(query_heads), total(c[n]), unit(unit_cost) {
    ctas = min(most_ctas, max(1, total));  // a step each at least
    snap = min(kSnap, total / ctas / 4);
  }
  __device__ Schedule(const int* c, const int* r, const Group* g, int n, int query_heads, const First& f);
  // The group that cost v belongs to: the last that begins at it or before.
  __device__ int group_of(int v) const {
    int lo = 0, hi = n_groups - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (costs[mid] <= v)
        lo = mid;
      else
        hi = mid - 1;
    }
    return lo;
  }
  // Where CTA c's run begins: equal shares of the cost, but a unit's border that is near takes the cut's place.
  __device__ int begin(int c) const {
    const int v = (int)((int64_t)total * c / ctas);
    if (v == 0 || v >= total) return v;
    const int g = group_of(v);
    const Shape sh(groups[g].rows * heads, groups[g].tiles);
    int in = (v - costs[g]) % sh.cost(unit);
    const int each = sh.tiles + unit, u = min(in / each, sh.twos), steps = u < sh.twos ? sh.tiles : sh.one_steps;
    in -= u * each;
    return in <= snap ? v - in : in >= steps - snap ? v + steps + unit - in : v;
  }
  __device__ int cta_of(int v) const {
    int c = (int)((((int64_t)v + 1) * ctas - 1) / total);
    while (begin(c) > v) --c;
    while (begin(c + 1) <= v) ++c;
    return c;
  }
};

// A run's piece in one unit: steps [a, b) of it.
struct Seg {
  Group g;
  int hk, q0, rows, two, a, b, part;  // q0: first query row in the group; part: first row of the unit's parts
  int last, next;                     // costs: of the unit's last step; where the run goes on
  __device__ int count(int t) const {  // half t's tiles
    if (two) return b - a;
    const int end = min(2 * b, g.tiles);
    return max(0, (end - 2 * a - t + 1) / 2);
  }
  __device__ int tile0() const { return two ? a : 2 * a; }
  __device__ int tile1() const { return two ? b : min(2 * b, g.tiles); }
};

// The piece that begins at cost v, which is that of a step, of a run that ends at `end`.
__device__ __forceinline__ Seg seg_at(const Schedule& s, int v, int end) {
  const int lo = s.group_of(v);
  Seg r;
  r.g = s.groups[lo];
  const Shape sh(r.g.rows * s.heads, r.g.tiles);
  const int in_group = v - s.costs[lo], each = sh.tiles + s.unit, head = sh.cost(s.unit);
  r.hk = in_group / head;
  const int in = in_group - r.hk * head, u = min(in / each, sh.twos);
  r.two = u < sh.twos;
  r.q0 = u * kUnitRows;
  r.rows = r.two ? min(kUnitRows, sh.rows - r.q0) : sh.one;
  r.a = in - u * each;
  const int all = r.two ? sh.tiles : sh.one_steps;
  r.b = min(all, r.a + (end - v));
  r.last = v - r.a + all - 1;
  r.next = min(end, r.last + 1 + s.unit);
  r.part = s.rows[lo] + r.hk * sh.part_rows() + r.q0;
  return r;
}

// What a CTA's warps find of the schedule when they begin.
struct First {
  int total, ctas, snap, unit, run0, run1;
  Seg seg;  // of the run's first unit
};
static_assert(sizeof(First) <= 128 && sizeof(Seg) <= 64, "their places");

__device__ __forceinline__ Schedule::Schedule(const int* c, const int* r, const Group* g, int n, int query_heads, const First& f)
    : costs(c), rows(r), groups(g), n_groups(n), heads(query_heads), total(f.total), ctas(f.ctas), snap(f.snap), unit(f.unit) {}

// Workspace.
struct Layout {
  size_t skip, groups, rows, cuts, suffix, suffix_lse, decode, ml, o, total;
};
inline size_t up256(size_t x) { return (x + 255) / 256 * 256; }
inline Layout layout(int64_t n, int64_t h, int64_t d, int64_t groups, size_t decode_bytes) {
  Layout w;
  const size_t rows = 2 * (size_t)(n * h) + (size_t)kUnitRows * kMaxCtas;
  w.skip = 0;
  w.groups = w.skip + up256((size_t)n * 4);
  w.rows = w.groups + up256((size_t)groups * sizeof(Group));
  w.cuts = w.rows + up256((size_t)n * h * sizeof(int4));
  w.suffix = w.cuts + up256((size_t)n * h * 4);
  w.suffix_lse = w.suffix + up256((size_t)n * h * d * 4);
  w.decode = w.suffix_lse + up256((size_t)n * h * 4);
  w.ml = w.decode + up256(decode_bytes);
  w.o = w.ml + up256(rows * 8);
  w.total = w.o + up256(rows * d * 4);
  return w;
}

struct Args {
  int n, h, hkv, d, groups, max_keys, num_pages, page, box, max_ctas;
  const int32_t *group_rows, *shared_lens, *lens, *table;
  int64_t table_stride;
  Seq4 q, out;
  Lse3 lse;
  int out_is_f32;
  int flush;  // tiles that are summed in one accumulator, less 1; a power of two of them
  float sl2;
  int* skip;
  Group* group;
  int4* row;  // of every (request, head) with a shared prefix: where its parts are
  const int* cuts;
  const float *suffix, *suffix_lse;  // of the requests' own keys, where these are not cut; else
  const float2* rest_ml;             // their parts
  const float* rest_o;
  int rest_rows;
  float2* ml;
  float* o;
  uint32_t* status;
};

// ---- setup -------------------------------------------------------------------------

constexpr int kSetupThreads = 512, kSetupWarps = kSetupThreads / 32;
constexpr int kSetupRows = 4;  // compared at a time

// gridDim.y blocks to a group, which take its rows in turn: its shortest request, how much is shared, and where each
// request's own keys begin. A row whose table names another page than the owner's among the shared ones shares nothing: the
// join passes over its prefix' parts. That comparison takes 1-2 us (64 requests behind 32k keys in pages of 16 88.8 -> 91.0, 256
// behind 16k 118.6 -> 120.3; by one block to a group 89 -> 218).
__global__ void __launch_bounds__(kSetupThreads) shared_setup_kernel(const __grid_constant__ Args p) {
  __shared__ int3 words[kSetupWarps];
  __shared__ int first_bad, first_other[kSetupRows];
  grid_launch_dependents();
  grid_dependency_wait();
  const int g = blockIdx.x, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int turn = blockIdx.y, turns = gridDim.y;
  int shared = p.shared_lens[g], r0 = p.group_rows[g], r1 = p.group_rows[g + 1];
  // rows that are not in ascending order make no groups at all
  bool wrong = false;
  for (int i = tid; i <= p.groups; i += kSetupThreads) {
    const int x = p.group_rows[i];
    wrong = wrong || x < 0 || x > p.n || (i > 0 && p.group_rows[i - 1] > x);
  }
  const bool bad = __syncthreads_or(wrong);
  if (bad) r0 = r1 = 0;
  if (g == 0 && turn == 0) {  // rows of no group
    const int a = bad ? p.n : p.group_rows[0], b = bad ? p.n : p.group_rows[p.groups];
    for (int r = tid; r < p.n; r += kSetupThreads)
      if (r < a || r >= b) p.skip[r] = 0;
    if (bad && tid == 0) report_status(p.status, BEA_STATUS_PAGES);
  }
  if (turn > 0 && turn >= r1 - r0) return;
  if (tid == 0) {
    first_bad = INT32_MAX;
    if (shared < 0 && turn == 0) report_status(p.status, BEA_STATUS_PAGES);
  }
  int shortest = INT32_MAX, owner = INT32_MAX, live = 0;
  for (int r = r0 + tid; r < r1; r += kSetupThreads) {
    const int len = p.lens[r];
    if (len <= 0) continue;
    shortest = min(shortest, len);
    owner = min(owner, r);
    ++live;
  }
  shortest = __reduce_min_sync(~0u, shortest);
  owner = __reduce_min_sync(~0u, owner);
  live = __reduce_add_sync(~0u, live);
  if (lane == 0) words[warp] = make_int3(shortest, owner, live);
  __syncthreads();
  const int3 w = words[lane % kSetupWarps];
  shortest = __reduce_min_sync(~0u, w.x);
  owner = __reduce_min_sync(~0u, w.y);
  live = __reduce_add_sync(~0u, lane < kSetupWarps ? w.z : 0);
  // nothing is shared by one request
  const int most = live > 1 ? max(0, min(min(shared, shortest), p.max_keys)) / kTile : 0;
  const int pages = (int)(((int64_t)most * kTile + p.page - 1) / p.page);
  const int32_t* entries = p.table + owner * p.table_stride;  // read where there is one
  // Forks of a prompt have the page that it ends in as copies of their own: where a row goes along up to the last page and
  // names another one there, that page is left out for all.
  bool other_end = false;
  for (int r = r0 + tid; pages > 1 && r < r1; r += kSetupThreads) {
    const int32_t* end = p.table + r * p.table_stride + pages - 2;
    other_end = other_end || (p.lens[r] > 0 && end[0] == entries[pages - 2] && end[1] != entries[pages - 1]);
  }
  for (int64_t row = r0 + turn; row < r1 || row == r0; row += (int64_t)turns * kSetupRows) {
    if (tid < kSetupRows) first_other[tid] = INT32_MAX;
    __syncthreads();
    const int32_t* others[kSetupRows];
#pragma unroll
    for (int z = 0; z < kSetupRows; ++z) {  // of a row without a request, or behind the last: the owner's again
      const int64_t r = row + z * turns;
      others[z] = most > 0 && r < r1 && p.lens[r] > 0 ? p.table + r * p.table_stride : entries;
    }
    int at = INT32_MAX, other[kSetupRows];
#pragma unroll
    for (int z = 0; z < kSetupRows; ++z) other[z] = INT32_MAX;
#pragma unroll 4
    for (int i = tid; i < pages; i += kSetupThreads) {
      const int id = entries[i];
      if (id < 0 || id >= p.num_pages) at = min(at, i);
#pragma unroll
      for (int z = 0; z < kSetupRows; ++z)
        if (others[z][i] != id) other[z] = min(other[z], i);
    }
    if (at != INT32_MAX) atomicMin(&first_bad, at);
#pragma unroll
    for (int z = 0; z < kSetupRows; ++z)
      if (other[z] != INT32_MAX) atomicMin(&first_other[z], other[z]);
    const int last = __syncthreads_or(other_end) ? pages - 1 : INT32_MAX, end = min(first_bad, last);
    const int tiles = end != INT32_MAX ? (int)((int64_t)end * p.page / kTile) : most;
    if (tid < kSetupRows) {
      const int64_t r = row + tid * turns;
      if (r < r1) p.skip[r] = p.lens[r] > 0 && (int64_t)first_other[tid] * p.page >= (int64_t)tiles * kTile ? tiles * kTile : 0;
    }
    if (turn == 0 && row == r0 && tid == 0) p.group[g] = Group{r0, r1 - r0, owner, tiles};
    __syncthreads();
  }
}

// ---- the prefix --------------------------------------------------------------------

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
    shared_prefix_kernel(const __grid_constant__ PageMaps maps, const __grid_constant__ Args p) {
  using C = Cfg<D>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::kBarOff);
  uint64_t *q_full = bars, *k_full = bars + 1, *v_full = k_full + C::kStages, *k_empty = v_full + C::kStages,
           *v_empty = k_empty + C::kStages, *s_full = v_empty + C::kStages, *o_full = s_full + 2, *mma_done = o_full + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + C::kNumBars);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  int* first_cost = reinterpret_cast<int*>(smem + C::kTableOff);
  int* first_row = first_cost + kMaxGroups + 1;
  Group* groups = reinterpret_cast<Group*>(smem + C::kGroupOff);
  First& first = *reinterpret_cast<First*>(smem + C::kFirstOff);
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int heads = p.h / p.hkv;

  if (threadIdx.x == 0) {
    *abort_flag = 0;
    for (int i = 0; i < C::kNumBars; ++i) mbar_init(&bars[i], i == 0 ? 256 : 1);
    fence_mbar_init();
  }
  if (warp == kKWarp && lane == 0) {
    prefetch_tmap(&maps.k[0]);
    prefetch_tmap(&maps.v[0]);
  }
  if (warp == kMmaWarp) {
    tmem_alloc(tmem_slot, 512);
    tmem_relinquish();
  }
  grid_launch_dependents();
  if (warp == kVWarp) {  // sums of costs and part rows over the groups
    int costs = 0, rows = 0, steps = 0;
    for (int i = lane; i < p.groups; i += 32) {
      // past L1, like all that this kernel reads before it has waited for the launch before it
      const int4 raw = __ldcg(reinterpret_cast<const int4*>(p.group + i));
      groups[i] = Group{raw.x, raw.y, raw.z, raw.w};
      steps += Shape(raw.y * heads, raw.w).cost(0) * p.hkv;
    }
    steps = __reduce_add_sync(~0u, steps);
    const int unit_cost = min(max(steps / (5 * (int)gridDim.x), kLeastUnitCost), kMostUnitCost);
    for (int g0 = 0; g0 < p.groups; g0 += 32) {
      int s = 0, r = 0;
      if (g0 + lane < p.groups) {
        const Group g = groups[g0 + lane];
        const Shape sh(g.rows * heads, g.tiles);
        s = sh.cost(unit_cost) * p.hkv;
        r = sh.part_rows() * p.hkv;
      }
      int si = s, ri = r;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int x = __shfl_up_sync(~0u, si, o), y = __shfl_up_sync(~0u, ri, o);
        if (lane >= o) si += x, ri += y;
      }
      if (g0 + lane < p.groups) {
        first_cost[g0 + lane] = costs + si - s;
        first_row[g0 + lane] = rows + ri - r;
      }
      costs += __shfl_sync(~0u, si, 31);
      rows += __shfl_sync(~0u, ri, 31);
    }
    if (lane == 0) first_cost[p.groups] = costs, first_row[p.groups] = rows;
    __syncwarp();
    // The run and its first unit, once for all warps: what each of them does not run when it begins it does not wait for, and
    // cold instructions are most of what passes until a CTA's first load.
    const Schedule sc(first_cost, first_row, groups, p.groups, heads, gridDim.x, unit_cost);
    const int cta = blockIdx.x, at = cta < sc.ctas ? sc.begin(cta + (lane & 1)) : 0;
    const int run0 = __shfl_sync(~0u, at, 0), run1 = __shfl_sync(~0u, at, 1);
    if (lane == 0) {
      first.total = sc.total, first.ctas = sc.ctas, first.snap = sc.snap, first.unit = sc.unit;
      first.run0 = run0, first.run1 = run1;
      if (run0 < run1) first.seg = seg_at(sc, run0, run1);
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  // (read again from shared memory where it is needed: few registers are free in between)
  auto schedule = [&]() { return Schedule(first_cost, first_row, groups, p.groups, heads, first); };
  const int cta = blockIdx.x, run0 = first.run0;
  auto unit_at = [&](int v) { return v == run0 ? first.seg : seg_at(schedule(), v, first.run1); };
  if (warp >= 8) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsOther));
    if (warp == kKWarp || warp == kVWarp) {
      // ========================== loads: boxes of 64 columns, the pages dealt to the lanes ==========================
      const bool is_k = warp == kKWarp;
      const CUtensorMap* map = is_k ? maps.k : maps.v;
      uint64_t *full = is_k ? k_full : v_full, *empty = is_k ? k_empty : v_empty;
      uint8_t* area = smem + (is_k ? C::kKOff : C::kVOff);
      const int smallest = __ffs(p.box) - 1;
      constexpr int kMost = kTile / 32;
      bool ok = true;
      int it = 0;
      for (int v = run0; ok && v < first.run1;) {
        const Seg sg = unit_at(v);
        v = sg.next;
        const int32_t* entries = p.table + sg.g.owner * p.table_stride;
        int id[kMost], first_page = 0;  // of this lane's pages in the next tile
        auto look_up = [&](int j) {
          if (j >= sg.tile1()) return;
          first_page = j * kTile / p.page;
#pragma unroll
          for (int i = 0; i < kMost; ++i) {
            const int pg = first_page + lane + 32 * i;
            if (pg * (int64_t)p.page < (j + 1) * kTile) id[i] = __ldcg(entries + pg);
          }
        };
        look_up(sg.tile0());
        for (int j = sg.tile0(); j < sg.tile1(); ++j, ++it) {
          const int s = it % C::kStages;
          if (it >= C::kStages && !(ok = warp_wait_parity(&empty[s], ((it / C::kStages) & 1) ^ 1, abort_flag, p.status))) break;
          if (lane == 0) mbar_arrive_expect_tx(&full[s], C::kTileBytes);
          __syncwarp();
          uint8_t* dst = area + s * C::kTileBytes;
#pragma unroll
          for (int i = 0; i < kMost; ++i) {
            // A page's rows in this tile, the largest box that fits first. (Boxes of one size, that which divides the page, for 20
            // requests of 16 heads behind 32k keys and P in one term: pages of 50 tokens 169 us, so 83, of 20 115, 86, of 7 284,
            // 158; of 32 78, 80: more boxes than one in 30 ns are what bounds a tile. In two terms 95, 100, 166, 93.)
            const int64_t from = (first_page + lane + 32 * i) * (int64_t)p.page - j * kTile;
            int row = (int)max(from, (int64_t)0);
            const int end = (int)min(from + p.page, (int64_t)kTile);
            while (row < end) {
              const int size = 31 - __clz(end - row);
              for (int x = 0; x < C::kBoxes; ++x)
                tma_load_4d(dst + x * 16384 + row * 128, map + (size - smallest), &full[s], x * 64, sg.hk, (int)(row - from), id[i]);
              row += 1 << size;
            }
          }
          look_up(j + 1);
        }
      }
      // loads in flight must land before the CTA's shared memory goes away
      for (int k = max(0, it - C::kStages); k < it; ++k) {
        volatile int no_abort = 0;
        wait_parity(&full[k % C::kStages], (k / C::kStages) & 1, &no_abort, p.status, 200000000ull);
      }
      __syncwarp();
    } else if (warp == kMmaWarp) {
      // ========================== products ==========================
      const uint64_t q_desc = sdesc_sw128(smem_u32(smem), 16, 1024);
      const uint64_t k_desc = sdesc_sw128(smem_u32(smem + C::kKOff), 16, 1024);
      const uint64_t v_desc = sdesc_sw128(smem_u32(smem + C::kVOff), C::kVLbo, 1024);
      bool ok = true;
      int base = 0, seg = 0;
      for (int v = run0; v < first.run1; ++seg) {
        const Seg sg = unit_at(v);
        v = sg.next;
        const int most = sg.count(0);  // the second half has as many tiles or one less
        // half t's x-th tile is the ring's slot(t, x)-th
        auto slot = [&](int t, int x) { return base + (sg.two ? x : 2 * x + t); };
        auto issue_s = [&](int t, int x) {
          const int i = slot(t, x), s = i % C::kStages;
          if (ok) ok = warp_wait_parity(&k_full[s], (i / C::kStages) & 1, abort_flag, p.status);
          if (!ok) return;
          tc_fence_after();
          const uint64_t qd = sdesc_add(q_desc, sg.two ? t * C::kTileBytes : 0), kd = sdesc_add(k_desc, s * C::kTileBytes);
#pragma unroll
          for (int k = 0; k < D / 16; ++k) {
            const uint32_t at = (k / 4) * 16384 + (k % 4) * 32;
            umma_ss_warp(tmem + t * 128, sdesc_add(qd, at), sdesc_add(kd, at), C::kIdescS, k > 0 ? 1u : 0u);
          }
          umma_commit_warp(&s_full[t]);
          if (!sg.two || t == 1) umma_commit_warp(&k_empty[s]);
        };
        auto issue_pv = [&](int t, int x, int n) {
          const int i = slot(t, x), s = i % C::kStages;
          if (ok) ok = warp_wait_parity(&v_full[s], (i / C::kStages) & 1, abort_flag, p.status);
          named_bar_sync(kPReadyBar + t, kPReadyThreads);  // P of the tile is in TMEM; joined after an abort too
          if (!ok) return;
          tc_fence_after();
          const uint64_t vd = sdesc_add(v_desc, s * C::kTileBytes);
#pragma unroll
          for (int term = 1; term >= 0; --term)  // small terms first
#pragma unroll
            for (int k = 0; k < kTile / 16; ++k)
              umma_ts_warp(tmem + 256 + t * 128, tmem + t * 128 + term * 64 + k * 8, sdesc_add(vd, k * 2048), C::kIdescPV,
                           term == 0 || k > 0 || (x & p.flush) != 0 ? 1u : 0u);
          if (!sg.two || t == 1) umma_commit_warp(&v_empty[s]);
          if (x == n - 1 || (x & p.flush) == p.flush) umma_commit_warp(&o_full[t]);
        };
        if (ok) ok = warp_wait_parity(q_full, seg & 1, abort_flag, p.status);
        const int n1 = sg.count(1);
        issue_s(0, 0);
        if (n1 > 0) issue_s(1, 0);
        for (int x = 0; x < most; ++x) {
          issue_pv(0, x, most);
          if (x + 1 < most) issue_s(0, x + 1);
          if (x < n1) issue_pv(1, x, n1);
          if (x + 1 < n1) issue_s(1, x + 1);
        }
        base += sg.tile1() - sg.tile0();
      }
      umma_commit_warp(mma_done);
      volatile int no_abort = 0;
      wait_parity(mma_done, 0, &no_abort, p.status, 200000000ull);
      __syncwarp();
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsSoftmax));
    // ========================== softmax ==========================
    const int t = warp / 4, r = threadIdx.x % 128;
    const uint32_t lane_base = (uint32_t)((warp % 4) * 32) << 16;
    const uint32_t s_tmem = tmem + lane_base + t * 128, o_tmem = tmem + lane_base + 256 + t * 128;
    bool ok = true;
    int met = 0, done = 0;  // tiles and segments of this half so far
    Seg& unit = *reinterpret_cast<Seg*>(smem + C::kUnitOff + warp * 64);  // the tiles' loop has no registers for it
    // A unit's queries, 16 bytes of a row at a time, copied without passing through registers (where the prefetched ones
    // would be spilled); rows behind the last repeat it and go nowhere.
    constexpr int kPieces = D / 8, kRows = 256 / kPieces, kTimes = kUnitRows / kRows;
    const int q_piece = threadIdx.x % kPieces, q_row = threadIdx.x / kPieces;
    auto each_row = [&](const Seg& sg, auto f) {
      const __nv_bfloat16* base = static_cast<const __nv_bfloat16*>(p.q.ptr) + sg.g.row0 * p.q.sn +
                                  (int64_t)sg.hk * heads * p.q.sh + q_piece * 8;
      const int step_b = kRows / heads, step_h = kRows - step_b * heads, last = sg.q0 + sg.rows - 1;
      const int last_b = last / heads, last_h = last - last_b * heads;
      int b = (sg.q0 + q_row) / heads, hh = sg.q0 + q_row - b * heads;
#pragma unroll
      for (int i = 0; i < kTimes; ++i) {
        const bool in = b < last_b || (b == last_b && hh <= last_h);
        f(q_row + i * kRows, base + (in ? b : last_b) * p.q.sn + (in ? hh : last_h) * p.q.sh);
        b += step_b, hh += step_h;
        if (hh >= heads) hh -= heads, ++b;
      }
    };
    // into shared memory, 128-byte swizzled like the forward's
    auto copy_queries = [&](const Seg& sg) {
      each_row(sg, [&](int row, const __nv_bfloat16* from) {
        const int in = row % kTile;
        if (row < kTile || sg.two) cp_async16(smem_u32(smem + (row / kTile) * C::kTileBytes + (q_piece / 8) * 16384 + in * 128 +
                                                       (((q_piece & 7) ^ (in & 7)) << 4)),
                                              from);
      });
    };
    auto queries_there = [&]() {
      cp_async_wait_all();
      fence_proxy_async_smem();
      mbar_arrive(q_full);
    };
    if (run0 < first.run1) {
      copy_queries(first.seg);
      queries_there();
    }
    for (int v = run0; v < first.run1;) {
      int n;
      {
        const Seg begun = unit_at(v);
        v = begun.next;
        n = begun.count(t);
        if (lane == 0) unit = begun;
        __syncwarp();
      }
      float m_ref = -INFINITY, l_sum = 0.f;
      int x = 0;
      do {
        const int end = min(n, x + p.flush + 1);
        for (; x < end; ++x, ++met) {
          if (ok) ok = warp_wait_parity(&s_full[t], met & 1, abort_flag, p.status);
          if (!ok) {
            named_bar_sync(kPReadyBar + t, kPReadyThreads);  // aborted: the phases stay matched
            continue;
          }
          tc_fence_after();
          uint32_t sr[128];
          tmem_ld32(s_tmem, sr);
          tmem_ld32(s_tmem + 32, sr + 32);
          tmem_ld32(s_tmem + 64, sr + 64);
          tmem_ld32(s_tmem + 96, sr + 96);
          tmem_wait_ld();
          reg_fence<128>(sr);
          float m8[8];
#pragma unroll
          for (int u = 0; u < 8; ++u) {
            float m = fmax3(__uint_as_float(sr[u]), __uint_as_float(sr[u + 8]), __uint_as_float(sr[u + 16]));
#pragma unroll
            for (int k = 3; k < 15; k += 2) m = fmax3(m, __uint_as_float(sr[u + 8 * k]), __uint_as_float(sr[u + 8 * k + 8]));
            m8[u] = fmaxf(m, __uint_as_float(sr[u + 120]));
          }
          const float mx = fmax3(fmax3(m8[0], m8[1], m8[2]), fmax3(m8[3], m8[4], m8[5]), fmaxf(m8[6], m8[7])) * p.sl2;
          const float m_new = fmaxf(m_ref, mx);
          const bool grow = m_new > m_ref + kRescale;
          float f = 1.f;
          bool rescale = false;
          if (x == 0) {
            m_ref = m_new;  // the first product overwrites O
          } else {
            rescale = __any_sync(~0u, grow) && (x & p.flush) != 0;  // else the next product overwrites O too
            if (grow) {
              f = ex2_approx(m_ref - m_new);
              m_ref = m_new;
              l_sum *= f;
            }
          }
          const float neg_m = m_ref == -INFINITY ? 0.f : -m_ref;
          const uint64_t sl2 = f2(p.sl2, p.sl2), nm2 = f2(neg_m, neg_m);
          uint64_t ps[4] = {0ull, 0ull, 0ull, 0ull};
#pragma unroll
          for (int hf = 0; hf < 2; ++hf) {
            uint32_t hi[32], lo[32];
#pragma unroll
            for (int c = 0; c < 32; ++c) {
              const int e = 64 * hf + 2 * c;
              const uint64_t a = f2_fma(f2(__uint_as_float(sr[e]), __uint_as_float(sr[e + 1])), sl2, nm2);
              float p0 = ex2_approx(f2_lo(a)), p1 = ex2_approx(f2_hi(a));
              // the last bit set, so that something is left behind the first term
              p0 = __uint_as_float(__float_as_uint(p0) | 1u), p1 = __uint_as_float(__float_as_uint(p1) | 1u);
              ps[c & 3] = f2_add(ps[c & 3], f2(p0, p1));
              hi[c] = __byte_perm(__float_as_uint(p0), __float_as_uint(p1), 0x7632);
              // less the first term: its 8 bits, with the sign of a subtraction
              const uint64_t rest = f2_add(f2(p0, p1), f2(__uint_as_float((__float_as_uint(p0) & 0xFFFF0000u) | 0x80000000u),
                                                          __uint_as_float((__float_as_uint(p1) & 0xFFFF0000u) | 0x80000000u)));
              lo[c] = pack_bf16x2(f2_lo(rest), f2_hi(rest));
            }
            tmem_st32(s_tmem + 32 * hf, hi);
            tmem_st32(s_tmem + 64 + 32 * hf, lo);
          }
          const uint64_t s2 = f2_add(f2_add(ps[0], ps[1]), f2_add(ps[2], ps[3]));
          l_sum += f2_lo(s2) + f2_hi(s2);
          if (rescale) {
#pragma unroll 1
            for (int c0 = 0; c0 < D; c0 += 32) {
              uint32_t orow[32];
              tmem_ld32(o_tmem + c0, orow);
              tmem_wait_ld();
              reg_fence<32>(orow);
#pragma unroll
              for (int c = 0; c < 32; ++c) orow[c] = __float_as_uint(__uint_as_float(orow[c]) * f);
              tmem_st32(o_tmem + c0, orow);
            }
          }
          tmem_wait_st();
          tc_fence_before();
          named_bar_sync(kPReadyBar + t, kPReadyThreads);
        }
        const Seg sg = unit;
        const int rows = sg.two ? min(kTile, sg.rows - t * kTile) : sg.rows;  // of this half
        const int64_t part = (int64_t)kUnitRows * cta + sg.part + t * (sg.two ? kTile : sg.rows) + r;
        if (x == n) {
          // Both halves have met the unit's last S: the next one's queries may take the place of its queries, and their S
          // products run while this unit's parts are written.
          const bool more = v < first.run1;
          if (more) {
            named_bar_sync(kBothBar, 256);
            copy_queries(unit_at(v));
          }
          if (sg.a == 0) {
            // for the kernel that joins: each row's first part, the parts' number, and the second half's distance
            const int parts = (schedule().cta_of(sg.last) - cta + 1) * (sg.two ? 1 : 2);
            for (int i = threadIdx.x; i < sg.rows; i += 256) {
              const int qr = sg.q0 + i, b = qr / heads, hh = sg.hk * heads + (qr - b * heads);
              p.row[(int64_t)(sg.g.row0 + b) * p.h + hh] = make_int4(kUnitRows * cta + sg.part + i, parts, sg.two ? 0 : sg.rows, 0);
            }
          }
          if (more) queries_there();
          if (n == 0 && r < rows) p.ml[part] = make_float2(-INFINITY, kNoKeys);
        }
        if (n > 0) {
          // ---- what the accumulator holds joins this half's part, each thread its row, whole 32-byte sectors of it at a time ----
          if (ok) ok = warp_wait_parity(&o_full[t], done & 1, abort_flag, p.status);
          ++done;
          tc_fence_after();
          if (ok) {
            const bool some = x > p.flush + 1;  // of it has been written, by the maximum that stands beside it
            float f = 1.f;
            if (r < rows) {
              const float m = some ? p.ml[part].x : m_ref;
              if (m != m_ref) f = ex2_approx(m - m_ref);
              p.ml[part] = make_float2(m_ref, l_sum);
            }
#pragma unroll
            for (int c0 = 0; c0 < D; c0 += 64) {
              uint32_t orow[64];
              tmem_ld32(o_tmem + c0, orow);
              tmem_ld32(o_tmem + c0 + 32, orow + 32);
              tmem_wait_ld();
              reg_fence<64>(orow);
              float* to = p.o + part * D + c0;
              if (r < rows) {
                if (some) {
#pragma unroll
                  for (int k = 0; k < 16; ++k) {
                    const float4 y = *reinterpret_cast<const float4*>(to + 4 * k);
                    uint32_t* z = orow + 4 * k;
                    z[0] = __float_as_uint(fmaf(y.x, f, __uint_as_float(z[0])));
                    z[1] = __float_as_uint(fmaf(y.y, f, __uint_as_float(z[1])));
                    z[2] = __float_as_uint(fmaf(y.z, f, __uint_as_float(z[2])));
                    z[3] = __float_as_uint(fmaf(y.w, f, __uint_as_float(z[3])));
                  }
                }
#pragma unroll
                for (int k = 0; k < 8; ++k) store_sector(to + 8 * k, orow + 8 * k);
              }
              __syncwarp();
            }
          }
          tc_fence_before();
        }
      } while (x < n);
    }
  }

  // the rest's kernel, which ran beside this one, has to be over when this one is
  grid_dependency_wait();
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (warp == kMmaWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// ---- join --------------------------------------------------------------------------

constexpr int kJoinWarps = 4;

// kSplit warps of a block to a (request, query head), a lane D / 32 columns: the parts of its prefix and of its own keys,
// dealt to the warps, or its own keys' result. A chain of two memory latencies (where the parts are, the parts) as long as a
// warp has at most kBatch of them.
template <int D, int kSplit, int kBatch>
__global__ void __launch_bounds__(kJoinWarps * 32, kBatch == 4 ? 8 : 1) shared_join_kernel(const __grid_constant__ Args p) {
  constexpr int N = D / 32;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, turn = warp % kSplit;
  const int64_t item = (int64_t)blockIdx.x * (kJoinWarps / kSplit) + warp / kSplit;
  grid_dependency_wait();
  const bool live = item < (int64_t)p.n * p.h;
  if (kSplit == 1 && !live) return;
  const int b = live ? (int)(item / p.h) : 0, hh = live ? (int)(item - (int64_t)b * p.h) : 0;
  const int64_t row = (int64_t)b * p.h + hh;
  const int skip = p.skip[b];
  const int4 where = p.row[row];  // of no request that shares: anything
  const Cut cut(p.cuts[row]);
  float o[N], top = p.suffix_lse[row] * kLog2e;
#pragma unroll
  for (int j = 0; j < N; ++j) o[j] = p.suffix[row * D + lane * N + j];
  if (cut.parts > 0 || turn > 0) {  // not written, or another warp's
    top = -INFINITY;
#pragma unroll
    for (int j = 0; j < N; ++j) o[j] = 0.f;
  }
  float sum = top == -INFINITY ? 0.f : 1.f;  // without keys o is zeros
  // the prefix' parts, one a CTA or two, then those of the rest; this warp's: turn, turn + kSplit, ...
  const int shared = skip > 0 ? where.y : 0, parts = shared + cut.parts;
  const int rest_row = hh % (p.h / p.hkv) % p.rest_rows;
  auto prefix_row = [&](int i) {
    return where.z == 0 ? where.x + (int64_t)kUnitRows * i : where.x + (int64_t)kUnitRows * (i >> 1) + (i & 1) * where.z;
  };
  auto rest_slot = [&](int i) { return i == 0 ? 2 * cut.cta + 1 : 2 * (cut.cta + i * cut.planes); };
  auto ml_of = [&](int i) {
    return i < shared ? p.ml + prefix_row(i) : p.rest_ml + rest_slot(i - shared) * 16 + rest_row;
  };
  auto o_of = [&](int i) {
    return i < shared ? p.o + prefix_row(i) * D
                      : p.rest_o + ((int64_t)rest_slot(i - shared) * p.rest_rows + rest_row) * D;
  };
  const int mine = (parts - turn + kSplit - 1) / kSplit;
  for (int i0 = 0; i0 < mine; i0 += 32) {
    const int n = min(32, mine - i0);
    const float2 e = lane < n ? *ml_of((i0 + lane) * kSplit + turn) : make_float2(-INFINITY, kNoKeys);
    const bool keys = e.y != kNoKeys;
    float w = 0.f;
    for (int i1 = 0; i1 < n; i1 += kBatch) {
      float y[kBatch][N];
#pragma unroll
      for (int z = 0; z < kBatch; ++z) {
#pragma unroll
        for (int j = 0; j < N; ++j) y[z][j] = 0.f;
        if (i1 + z < n) {
          const float* from = o_of((i0 + i1 + z) * kSplit + turn) + lane * N;
          if constexpr (N == 4) {
            const float4 x = __ldcs(reinterpret_cast<const float4*>(from));
            y[z][0] = x.x, y[z][1] = x.y, y[z][2] = x.z, y[z][3] = x.w;
          } else {
            const float2 x = __ldcs(reinterpret_cast<const float2*>(from));
            y[z][0] = x.x, y[z][1] = x.y;
          }
        }
      }
      if (i1 == 0) {  // the weights, while the first parts are under way
        float m = e.x;
#pragma unroll
        for (int x = 16; x > 0; x >>= 1) m = fmaxf(m, __shfl_xor_sync(~0u, m, x));
        m = fmaxf(m, top);
        const float ref = m == -INFINITY ? 0.f : m, old = top == -INFINITY ? 0.f : ex2_approx(top - ref);
        w = ex2_approx(e.x - ref);  // 0 where there is no maximum
        float l = keys ? w * e.y : 0.f;
#pragma unroll
        for (int x = 16; x > 0; x >>= 1) l += __shfl_xor_sync(~0u, l, x);
        sum = sum * old + l;
        top = m;
#pragma unroll
        for (int j = 0; j < N; ++j) o[j] *= old;
      }
#pragma unroll
      for (int z = 0; z < kBatch; ++z) {
        const float g1 = __shfl_sync(~0u, w, (i1 + z) & 31);
        const bool there = __shfl_sync(~0u, keys, (i1 + z) & 31) && i1 + z < n;
#pragma unroll
        for (int j = 0; j < N; ++j) o[j] = there ? fmaf(g1, y[z][j], o[j]) : o[j];
      }
    }
  }
  if constexpr (kSplit > 1) {  // the warps' results, in order
    __shared__ float part[kJoinWarps][D];
    __shared__ float2 part_ml[kJoinWarps];
#pragma unroll
    for (int j = 0; j < N; ++j) part[warp][lane * N + j] = o[j];
    if (lane == 0) part_ml[warp] = make_float2(top, sum);
    __syncthreads();
    if (turn > 0 || !live) return;
#pragma unroll
    for (int x = 1; x < kSplit; ++x) {
      const float2 e = part_ml[warp + x];
      const float m = fmaxf(top, e.x), ref = m == -INFINITY ? 0.f : m;
      const float f = top == -INFINITY ? 0.f : ex2_approx(top - ref), g = e.x == -INFINITY ? 0.f : ex2_approx(e.x - ref);
      top = m;
      sum = sum * f + e.y * g;
#pragma unroll
      for (int j = 0; j < N; ++j) o[j] = o[j] * f + part[warp + x][lane * N + j] * g;
    }
  }
  if (lane == 0) p.lse.ptr[b * p.lse.sn + hh * p.lse.sh] = sum == 0.f ? -INFINITY : (top + log2f(sum)) * kLn2;
  const float inv = sum == 0.f ? 0.f : 1.f / sum;
  const int64_t to = b * p.out.sn + hh * p.out.sh + lane * N;
#pragma unroll
  for (int j = 0; j < N; ++j) o[j] *= inv;
  if (p.out_is_f32) {
    float* y = static_cast<float*>(p.out.ptr) + to;
    if constexpr (N == 4)
      *reinterpret_cast<float4*>(y) = make_float4(o[0], o[1], o[2], o[3]);
    else
      *reinterpret_cast<float2*>(y) = make_float2(o[0], o[1]);
  } else {
    __nv_bfloat16* y = static_cast<__nv_bfloat16*>(p.out.ptr) + to;
    if constexpr (N == 4)
      *reinterpret_cast<uint2*>(y) = make_uint2(pack_bf16x2(o[0], o[1]), pack_bf16x2(o[2], o[3]));
    else
      *reinterpret_cast<uint32_t*>(y) = pack_bf16x2(o[0], o[1]);
  }
}

template <int D>
cudaError_t launch(const PagedSharedParams& p, const PageMaps& maps, cudaStream_t s, int* nlaunch) {
  using C = Cfg<D>;
  struct Facts {
    int ctas, regs;
  };
  static PerContext<Facts> cache;
  Facts f{};
  cudaError_t e = cache.get(
      [](Facts* v) {
        cudaError_t r = cudaFuncSetAttribute(shared_prefix_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
        if (r != cudaSuccess) return r;
        cudaFuncAttributes fa;
        if ((r = cudaFuncGetAttributes(&fa, shared_prefix_kernel<D>)) != cudaSuccess) return r;
        v->regs = fa.numRegs;
        if ((r = device_sm_count(&v->ctas)) != cudaSuccess) return r;
        if (v->ctas > kMaxCtas) v->ctas = kMaxCtas;
        return r;
      },
      &f);
  if (e != cudaSuccess) return e;
  if (f.regs != kRegsLaunch) return cudaErrorInvalidConfiguration;  // the register split holds for that number only
  const PagedDecodeParams& d = p.d;
  uint8_t* ws = static_cast<uint8_t*>(d.ws);
  const size_t decode_bytes = paged_decode_workspace(d.h, d.hkv, d.d, (int64_t)d.max_pages * d.page);
  const Layout w = layout(d.n, d.h, d.d, p.groups, decode_bytes);
  Args a = {};
  a.n = d.n, a.h = d.h, a.hkv = d.hkv, a.d = d.d, a.groups = p.groups;
  a.max_keys = d.max_pages * d.page;
  a.num_pages = d.num_pages;
  a.page = d.page;
  a.box = paged_shared_box(d.page);
  a.max_ctas = f.ctas;
  a.group_rows = p.group_rows, a.shared_lens = p.shared_lens, a.lens = d.lens, a.table = d.table;
  a.table_stride = d.table_stride;
  a.q = d.q, a.out = d.out, a.lse = d.lse;
  a.out_is_f32 = d.out_is_f32;
  a.flush = (d.out_is_f32 ? kFlushF32 : kFlushBf16) - 1;
  a.sl2 = d.scale * kLog2e;
  a.skip = reinterpret_cast<int*>(ws + w.skip);
  a.group = reinterpret_cast<Group*>(ws + w.groups);
  a.row = reinterpret_cast<int4*>(ws + w.rows);
  a.cuts = reinterpret_cast<int*>(ws + w.cuts);
  a.suffix = reinterpret_cast<float*>(ws + w.suffix);
  const DecodeParts rest = paged_decode_parts(d.h, d.hkv, d.d);
  a.rest_ml = reinterpret_cast<float2*>(ws + w.decode + rest.ml);
  a.rest_o = reinterpret_cast<float*>(ws + w.decode + rest.o);
  a.rest_rows = rest.rows;
  a.suffix_lse = reinterpret_cast<float*>(ws + w.suffix_lse);
  a.ml = reinterpret_cast<float2*>(ws + w.ml);
  a.o = reinterpret_cast<float*>(ws + w.o);
  a.status = d.status;
  const int turns = f.ctas / p.groups < 1 ? 1 : f.ctas / p.groups < d.n ? f.ctas / p.groups : d.n;
  if ((e = launch_dependent(shared_setup_kernel, dim3(p.groups, turns), kSetupThreads, 0, s, a)) != cudaSuccess) return e;
  *nlaunch += 1;
  // the requests' own keys, in fp32, with their log-sum-exp
  PagedDecodeParams own = d;
  own.skip = a.skip;
  own.cuts = reinterpret_cast<int*>(ws + w.cuts);
  own.out = Seq4{ws + w.suffix, (int64_t)d.h * d.d, 0, d.d};
  own.out_is_f32 = 1;
  own.lse = Lse3{reinterpret_cast<float*>(ws + w.suffix_lse), d.h, 1};
  own.ws = ws + w.decode;
  if ((e = launch_paged_decode_rest(own, s, nlaunch)) != cudaSuccess) return e;
  if ((e = launch_dependent(shared_prefix_kernel<D>, dim3(f.ctas), kThreads, C::kSmem, s, maps, a)) != cudaSuccess) return e;
  *nlaunch += 1;
  const int64_t items = (int64_t)d.n * d.h;
  // Rows that do not fill the GPU have many parts each, four warps a row then; where there are warps enough to hide the
  // latency fewer loads at a time leave room for more of them. (256 requests of 32 heads: 118.7 us with 4 at a time, 122.3 with
  // 8; 64 requests 76.5, 74.7 us; 8 requests 23.6 us, with one warp a row 27.0.)
  const bool few = items <= f.ctas * 8, many = items > f.ctas * 32;
  const int64_t warps = items * (few ? kJoinWarps : 1);
  auto join = few ? shared_join_kernel<D, kJoinWarps, 8> : many ? shared_join_kernel<D, 1, 4> : shared_join_kernel<D, 1, 8>;
  e = launch_dependent(join, dim3((unsigned)((warps + kJoinWarps - 1) / kJoinWarps)), kJoinWarps * 32, 0, s, a);
  if (e == cudaSuccess) *nlaunch += 1;
  return e;
}

}  // namespace

// Up to so many bytes of keys and values that sharing saves the other kernels take longer than reading them again. 32 / 8
// heads of 128, GPU time with and without sharing: 4 requests behind 4k keys (50 MB) 22.5, 16.3 us, 8 behind 4k (117 MB)
// 23.6, 23.8 us, 4 behind 16k (201 MB) 34.6, 40.7 us; 16 / 16 heads of 64: 8 behind 4k (117 MB) 24.0, 27.7 us.
constexpr int64_t kLeastSaved = 96000000;

static bool saves_little(int64_t n, int64_t h_kv, int64_t d, int64_t max_keys, int64_t groups) {
  return groups == 0 || max_keys < kTile || (n - 1) * max_keys <= kLeastSaved / (h_kv * d * 4);
}

bool paged_shared_is_plain(const PagedDecodeParams& d, int64_t groups) {
  return d.num_pages == 0 || saves_little(d.n, d.hkv, d.d, (int64_t)d.max_pages * d.page, groups);
}

int paged_shared_box(int64_t page) {
  int b = kTile;
  while (page % b != 0) b /= 2;
  return b;
}

size_t paged_shared_workspace(int64_t n, int64_t h, int64_t h_kv, int64_t d, int64_t max_keys, int64_t groups) {
  const size_t rest = paged_decode_workspace(h, h_kv, d, max_keys);
  return saves_little(n, h_kv, d, max_keys, groups) ? rest : layout(n, h, d, groups, rest).total;
}

bool paged_shared_fits(int64_t n, int64_t h, int64_t h_kv, int64_t max_keys, int64_t groups) {
  const int64_t most = (int64_t(1) << 31) - 1;
  if (2 * n * h + (int64_t)kUnitRows * kMaxCtas > most) return false;
  const int64_t units = h_kv * (n * (h / h_kv) / kUnitRows + (groups < n ? groups : n));
  return units <= most / (max_keys / kTile + 1 + kMostUnitCost);
}

cudaError_t launch_paged_shared(const PagedSharedParams& p, const PageMaps& maps, cudaStream_t s, int* nlaunch) {
  return p.d.d == 64 ? launch<64>(p, maps, s, nlaunch) : launch<128>(p, maps, s, nlaunch);
}

}  // namespace bea
