// RMS norm of every head of q and k, then the rotation, in one pass; and its gradient.
//
// A row x of d elements becomes y = w * x * r, r = 1 / sqrt(mean(x^2) + eps), and y's first 2 * pairs elements are
// turned pair by pair, (a, b) -> (a c - b s, b c + a s), with c and s the angle's cosine and sine times the amplitude.
// Pairs are (x_p, x_{p + pairs}) or, interleaved, (x_{2p}, x_{2p + 1}); what lies behind passes. Without the norm it is
// the rotation alone. All of it in fp32, one rounding at the end. With g the gradient turned back (the rotation's
// adjoint), the gradients are
//   dw = sum over rows of g * x r,   dx = r (w g - x r^2 mean(w g x)).
//
// HBM-bound: forward 2 elements moved for one of x, backward 3; but only just, a bf16 row leaves the SMs some 130
// instructions for a lane's 16 elements. So elements go by pairs (fma.f32x2), the weights are multiplied into the
// cosines and sines, and these are worked out once for a thread's whole token. A row belongs to `lanes` neighbouring lanes
// of a warp, a power of two; each holds two 16-byte pieces of it, both ends of its pairs (half layout: a piece of the first
// half and its partner in the second; interleaved: 32 bytes in a row), so the rotation needs no exchange and the norm a
// shuffle tree of log2(lanes) steps. A thread takes a token's heads kHeads at a time, a CHUNK: it reduces, turns and stores
// one while the next is on its way into shared memory, where the norm leaves bf16 rows little time to send loads and wait
// (forward 113 us with loads into registers, 110 so; of a thread with one chunk there is no next, and f32 rows and those without
// a norm gain nothing or lose 3-8%: loads into registers there). Tokens that do not fill the GPU are shared out between
// several threads.
//
// The weights' gradient is a sum over all rows. A thread keeps its columns' sums in fp32 over all the rows it meets
// (the grid is one wave, each block only q or only k), a block adds up its threads in shared memory, and a second kernel
// the blocks, all in a fixed order: the same call gives the same bits.
//
// Measured (GPU time, inputs larger than L2): [1, 32768, 32 + 8, 128] bf16 forward 110 us (6.1 TB/s), with its gradient
// 286 us (5.9 TB/s; a copy reaches 6.7), interleaved too; interleaved without the norm 103 us (6.5 TB/s). [1, 16384, 16 + 16,
// 128] f32 85 and 216 us (6.3, 6.2 TB/s). 256 tokens of 32 + 8 heads: 5.1 us, the host takes 7.1-8.6
#include <type_traits>

#include <cuda_bf16.h>

#include "launch_cache.cuh"
#include "norm_rope.cuh"
#include "ptx.cuh"
#include "rotary.cuh"

namespace bea {
namespace {

constexpr int kThreads = 128;
// Threads of an SM that a forward's tokens are shared out between, at least: two waves of them. Fewer slices of a token compute
// its angles less often, more of them end together ([8, 4096, 16 + 16, 64] bf16: 640 threads 50.6 us, 1280 46.2; [1, 4096,
// 32 + 8, 128]: 20.8, 17.4 us; 2048 16-20% slower than 1280, with loads into registers).
constexpr int kSmThreads = 1280;
constexpr int kMaxD = 2 * kRopeMaxPairs;
// Heads of a chunk. Forward: 2 heads three stages deep 111.5 us for [1, 32768, 32 + 8, 128] bf16 (now 110), 2 and 8 with loads
// into registers 131 and 127 us; 6 blocks to an SM 123 us. Backward: 1 head three or four stages deep 2-4% slower; 3 or 5
// blocks to an SM 318 and 350 us for the training step (now 286).
constexpr int kFwdHeads = 4, kFwdStages = 2;
constexpr int kBwdHeads = 2, kBwdStages = 2, kBwdBlocks = 4;

__device__ __forceinline__ float weight_at(const void* w, int is_f32, int c) {
  if (w == nullptr) return 1.f;
  return is_f32 ? static_cast<const float*>(w)[c] : __bfloat162float(static_cast<const __nv_bfloat16*>(w)[c]);
}

// Where lane `i` of a row finds its two pieces (of N elements): columns a and b, and its pairs: i * N + j, j < N.
template <bool kInter, int N>
struct Place {
  int a, b, pair;
  bool mine;
  __device__ __forceinline__ Place(int i, int d, int pairs) {
    pair = i * N;
    mine = 2 * i * N < d;
    if (kInter) {
      a = 2 * i * N;
      b = a + N;
    } else if (pair < pairs) {  // pairs is a multiple of N
      a = pair;
      b = pair + pairs;
    } else {
      a = 2 * i * N;
      b = a + N;
    }
  }
  // The column of the first and second element of pair j.
  __device__ __forceinline__ int first(int j) const { return kInter ? a + 2 * j : a + j; }
  __device__ __forceinline__ int second(int j) const { return kInter ? a + 2 * j + 1 : b + j; }
};

// A lane's two pieces as the first (u) and second (v) elements of its pairs, two pairs to a packed value, and back.
template <bool kF32, bool kInter>
__device__ __forceinline__ void unpack(const uint4& a, const uint4& b, uint64_t* u, uint64_t* v) {
  auto f = [](uint32_t x) { return __uint_as_float(x); };
  if constexpr (kF32) {
    if constexpr (kInter) {
      u[0] = f2(f(a.x), f(a.z)), u[1] = f2(f(b.x), f(b.z));
      v[0] = f2(f(a.y), f(a.w)), v[1] = f2(f(b.y), f(b.w));
    } else {
      u[0] = f2(f(a.x), f(a.y)), u[1] = f2(f(a.z), f(a.w));
      v[0] = f2(f(b.x), f(b.y)), v[1] = f2(f(b.z), f(b.w));
    }
  } else {
    const uint32_t x[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (kInter) {
        u[i] = f2(f(x[2 * i] << 16), f(x[2 * i + 1] << 16));
        v[i] = f2(f(x[2 * i] & 0xFFFF0000u), f(x[2 * i + 1] & 0xFFFF0000u));
      } else {
        u[i] = f2(f(x[i] << 16), f(x[i] & 0xFFFF0000u));
        v[i] = f2(f(x[4 + i] << 16), f(x[4 + i] & 0xFFFF0000u));
      }
    }
  }
}
template <bool kF32, bool kInter>
__device__ __forceinline__ void pack(const uint64_t* u, const uint64_t* v, uint4& a, uint4& b) {
  if constexpr (kF32) {
    auto w = [](float x) { return __float_as_uint(x); };
    if constexpr (kInter) {
      a = make_uint4(w(f2_lo(u[0])), w(f2_lo(v[0])), w(f2_hi(u[0])), w(f2_hi(v[0])));
      b = make_uint4(w(f2_lo(u[1])), w(f2_lo(v[1])), w(f2_hi(u[1])), w(f2_hi(v[1])));
    } else {
      a = make_uint4(w(f2_lo(u[0])), w(f2_hi(u[0])), w(f2_lo(u[1])), w(f2_hi(u[1])));
      b = make_uint4(w(f2_lo(v[0])), w(f2_hi(v[0])), w(f2_lo(v[1])), w(f2_hi(v[1])));
    }
  } else {
    uint32_t x[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (kInter) {
        x[2 * i] = pack_bf16x2(f2_lo(u[i]), f2_lo(v[i]));
        x[2 * i + 1] = pack_bf16x2(f2_hi(u[i]), f2_hi(v[i]));
      } else {
        x[i] = pack_bf16x2(f2_lo(u[i]), f2_hi(u[i]));
        x[4 + i] = pack_bf16x2(f2_lo(v[i]), f2_hi(v[i]));
      }
    }
    a = make_uint4(x[0], x[1], x[2], x[3]);
    b = make_uint4(x[4], x[5], x[6], x[7]);
  }
}

__device__ __forceinline__ uint64_t f2_select(bool lo, bool hi, uint64_t a, uint64_t b) {
  return f2(lo ? f2_lo(a) : f2_lo(b), hi ? f2_hi(a) : f2_hi(b));
}
__device__ __forceinline__ uint64_t f2_neg(uint64_t a) { return a ^ 0x8000000080000000ull; }

// 1 / sqrt(x): for bf16 rows the instruction, good to 2 units in the last place.
template <bool kF32>
__device__ __forceinline__ float root_inverse(float x) {
  if constexpr (kF32) return __frsqrt_rn(x);
  return rsqrtf(x);
}

struct Tables {
  uint64_t turn[kRopeMaxPairs];
  uint8_t axis[kRopeMaxPairs];
  float w[2][kMaxD];
};
// Those of the launch before the wait on the kernel before, the weights after it.
template <bool kNorm>
__device__ __forceinline__ void load_tables(const NormRopeParams& p, Tables& t) {
  for (int i = threadIdx.x; i < p.pairs; i += blockDim.x) {
    t.turn[i] = p.turn[i];
    t.axis[i] = p.axis[i];
  }
  grid_dependency_wait();
  if constexpr (kNorm) {
    for (int i = threadIdx.x; i < p.d; i += blockDim.x) {
      t.w[0][i] = weight_at(p.wq, p.wq_f32, i);
      t.w[1][i] = weight_at(p.wk, p.wk_f32, i);
    }
  }
  __syncthreads();
}

// Cosines and sines of a lane's pairs, times the amplitude; of those that pass 1 and 0.
template <int N>
__device__ __forceinline__ void angles(const NormRopeParams& p, const Tables& t, int64_t b, int i, int pair, int inverse,
                                       uint64_t* c, uint64_t* s) {
#pragma unroll
  for (int j = 0; j < N; j += 2) {
    float cs[2] = {1.f, 1.f}, sn[2] = {0.f, 0.f};
#pragma unroll
    for (int z = 0; z < 2; ++z) {
      if (pair + j + z < p.pairs) {
        const int64_t pos = p.pos[t.axis[pair + j + z] * p.pos_sa + b * p.pos_sn + i];
        cos_sin(pos, t.turn[pair + j + z], inverse, &cs[z], &sn[z]);
        cs[z] *= p.amplitude;
        sn[z] *= p.amplitude;
      }
    }
    c[j / 2] = f2(cs[0], cs[1]);
    s[j / 2] = f2(sn[0], sn[1]);
  }
}

__device__ __forceinline__ int lane_shift(int d, int n) {  // lanes of a row: half its pieces, up to a power of two
  const int half = (d / n + 1) / 2;
  return half <= 1 ? 0 : 32 - __clz(half - 1);
}
int host_lane_shift(int d, int n) {
  int s = 0;
  while ((1 << s) * 2 * n < d) ++s;
  return s;
}

// An item: lane, token and a slice of `per` of its chunks of kHeads heads (q's, then k's).
struct Item {
  int64_t b;
  int i, chunk0, lane;
  __device__ Item(const NormRopeParams& p, int64_t it, int shift, int slices, int per) {
    lane = (int)it & ((1 << shift) - 1);
    const int64_t ts = it >> shift;
    int64_t t;
    if (ts < (int64_t(1) << 32)) {  // divisions in 32 bits where they are enough
      t = (uint32_t)ts / (uint32_t)slices;
      b = (uint32_t)t / (uint32_t)p.l;
    } else {
      t = ts / slices;
      b = t / p.l;
    }
    i = (int)(t - b * p.l);
    chunk0 = (int)(ts - t * slices) * per;
  }
};

// Rows on their way through shared memory, by asynchronous copies that need no registers: a slot of 16 bytes for every piece,
// 2 * lanes of them to a row. kOwn: each thread copies and reads back what is its own, so nothing but its own copies is waited
// for. Else a row's lanes copy its pieces in memory's order, whichever they need, so that every copy fills whole sectors
// where a lane's two pieces lie side by side (a 32k training step, interleaved, 371 us with kOwn, 288 without; with half of
// the head turned, 8k, 116 and 104 us); the last bit is turned so that eight lanes that read every other piece meet
// different banks.
template <bool kF32, bool kOwn>
struct Staged {
  static constexpr int kN = Piece<kF32>::kN;
  static constexpr int kBytes = kThreads * 2 * 16;  // of a row for each group of lanes
  int first, second;                                // the pieces this lane copies, -1: none
  uint32_t to0, to1, from0, from1;
  __device__ Staged(int shift, int d, int a, int b, bool mine) {
    if constexpr (kOwn) {
      first = mine ? a / kN : -1;
      second = mine ? b / kN : -1;
      to0 = from0 = threadIdx.x * 16;
      to1 = from1 = (kThreads + threadIdx.x) * 16;
    } else {
      const int lanes = 1 << shift, row = (threadIdx.x >> shift) << (shift + 1), pieces = d / kN;
      const int i = threadIdx.x & (lanes - 1);
      auto slot = [](int x) { return (uint32_t)(x ^ ((x >> 3) & 1)) * 16; };
      first = i < pieces ? i : -1;
      second = i + lanes < pieces ? i + lanes : -1;
      to0 = slot(row + i);
      to1 = slot(row + i + lanes);
      from0 = slot(row + a / kN);
      from1 = slot(row + b / kN);
    }
  }
  // src: the row, or any address where nothing is read and the slots become zeros.
  __device__ __forceinline__ void copy(uint32_t area, const char* src, bool read) const {
    one(area + to0, src, first, read);
    one(area + to1, src, second, read);
  }
  __device__ __forceinline__ void one(uint32_t dst, const char* src, int piece, bool read) const {
    read = read && piece >= 0;
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src + (read ? piece * 16 : 0)), "r"(read ? 16 : 0)
                 : "memory");
  }
  // Ends a chunk's copies; of chunks without any too, so that groups count chunks.
  __device__ __forceinline__ void commit() const { asm volatile("cp.async.commit_group;" ::: "memory"); }
  // Before copies go where something has been read.
  __device__ __forceinline__ void been_read() const {
    if constexpr (!kOwn) __syncwarp();
  }
  // All chunks but the last kLeft are there.
  template <int kLeft>
  __device__ __forceinline__ void there() const {
    asm volatile("cp.async.wait_group %0;" ::"n"(kLeft) : "memory");
    if constexpr (!kOwn) __syncwarp();
  }
  __device__ __forceinline__ void read(const uint8_t* area, uint4& a, uint4& b) const {
    a = *reinterpret_cast<const uint4*>(area + from0);
    b = *reinterpret_cast<const uint4*>(area + from1);
  }
};

// kPartial: only a part of the head is turned. kStages: chunks in shared memory, kStages - 1 of them ahead; 0: loads into
// registers.
template <bool kF32, bool kNorm, bool kInter, bool kPartial, int kHeads, int kStages>
__global__ void __launch_bounds__(kThreads, 5) norm_rope_kernel(const __grid_constant__ NormRopeParams p, int slices, int per) {
  constexpr int N = Piece<kF32>::kN, H = N / 2;
  using S = Staged<kF32, !kInter && !kPartial>;
  extern __shared__ __align__(16) uint8_t rows[];  // [stage][head] of S::kBytes
  __shared__ Tables tables;
  // A thread's cosines and sines, without the weights of q or k: worked out again for k, and with a chunk's missing heads
  // computed along, 6 + 3 heads of [14, 6507] took 97 us, not 80.
  __shared__ uint64_t kept[kNorm ? 2 * H : 1][kThreads];
  load_tables<kNorm>(p, tables);
  constexpr int es = kF32 ? 4 : 2;
  const int shift = lane_shift(p.d, N);
  const Place<kInter, N> at(threadIdx.x & ((1 << shift) - 1), p.d, p.pairs);
  const int cq = (p.hq + kHeads - 1) / kHeads, chunks = cq + (p.hk + kHeads - 1) / kHeads;
  const int64_t total = ((int64_t)p.n * p.l * slices) << shift;
  const float inv_d = 1.f / (float)p.d;
  const S st(shift, p.d, at.a, at.b, at.mine);
  const int64_t first = (int64_t)blockIdx.x * kThreads + threadIdx.x, step = (int64_t)gridDim.x * kThreads;
  // what is copied next: chunk c_ahead, the `ahead`-th of item it_ahead
  int64_t it_ahead = first, b_ahead = 0;
  int i_ahead = 0, c_ahead = 0, ahead = 0, stage_ahead = 0, stage = 0;
  auto copy_next = [&]() {
    if ((it_ahead & ~int64_t(31)) < total) {
      if (ahead == 0) {
        const Item m(p, it_ahead < total ? it_ahead : 0, shift, slices, per);
        b_ahead = m.b, i_ahead = m.i, c_ahead = m.chunk0;
      }
      const bool k_now = c_ahead >= cq;
      const int h0 = (k_now ? c_ahead - cq : c_ahead) * kHeads, heads = c_ahead < chunks ? (k_now ? p.hk : p.hq) : 0;
      const Seq4& from = k_now && p.hk > 0 ? p.k : p.q;
      const char* src = static_cast<const char*>(from.ptr) + (b_ahead * from.sn + i_ahead * from.sl) * es;
#pragma unroll
      for (int x = 0; x < kHeads; ++x) {
        const bool read = it_ahead < total && h0 + x < heads;
        st.copy(smem_u32(rows) + (stage_ahead * kHeads + x) * S::kBytes, read ? src + (h0 + x) * from.sh * es : src, read);
      }
      ++c_ahead;
      if (++ahead == per) ahead = 0, it_ahead += step;
    }
    stage_ahead = stage_ahead + 1 == kStages ? 0 : stage_ahead + 1;
    st.commit();
  };
#pragma unroll
  for (int z = 0; z + 1 < kStages; ++z) copy_next();
  // a warp goes on while any of its items is one, so that all its lanes meet in the shuffles
  for (int64_t it = first; (it & ~int64_t(31)) < total; it += step) {
    const bool live = it < total && at.mine;
    const Item m(p, it < total ? it : 0, shift, slices, per);
    // What a row's elements are multiplied by, r apart: with the first and second element of each pair and its partner.
    uint64_t c[H], s[H], fc[H], fs[H];  // cos, sin of the first element; of the second (with other weights)
    bool is_k = false;
    for (int x0 = 0; x0 < per; ++x0) {
      const int chunk = m.chunk0 + x0;
      const bool k_now = chunk >= cq;
      const int h0 = (k_now ? chunk - cq : chunk) * kHeads, heads = chunk < chunks ? (k_now ? p.hk : p.hq) : 0;
      const Seq4 &from = k_now ? p.k : p.q, &to = k_now ? p.ko : p.qo;
      uint4 ra[kHeads], rb[kHeads];
      const uint8_t* here = rows + stage * kHeads * S::kBytes;
      if constexpr (kStages > 0) {
        st.been_read();
        copy_next();
        st.template there<kStages - 1>();
        stage = stage + 1 == kStages ? 0 : stage + 1;
      } else {
        const char* src = static_cast<const char*>(from.ptr) + (m.b * from.sn + m.i * from.sl + h0 * from.sh) * es;
#pragma unroll
        for (int x = 0; x < kHeads; ++x) {
          ra[x] = rb[x] = make_uint4(0u, 0u, 0u, 0u);
          if (live && h0 + x < heads) {
            ra[x] = __ldcs(reinterpret_cast<const uint4*>(src + (x * from.sh + at.a) * es));
            rb[x] = __ldcs(reinterpret_cast<const uint4*>(src + (x * from.sh + at.b) * es));
          }
        }
      }
      if (x0 == 0 || (kNorm && k_now != is_k)) {
        is_k = k_now;
        if (x0 == 0) {
          angles<N>(p, tables, m.b, m.i, at.mine ? at.pair : p.pairs, p.inverse, c, s);
          if constexpr (kNorm) {
#pragma unroll
            for (int j = 0; j < H; ++j) kept[2 * j][threadIdx.x] = c[j], kept[2 * j + 1][threadIdx.x] = s[j];
          }
        } else if constexpr (kNorm) {
#pragma unroll
          for (int j = 0; j < H; ++j) c[j] = kept[2 * j][threadIdx.x], s[j] = kept[2 * j + 1][threadIdx.x];
        }
        if constexpr (kNorm) {
          const float* w = tables.w[is_k];
#pragma unroll
          for (int j = 0; j < H; ++j) {
            const uint64_t wu = at.mine ? f2(w[at.first(2 * j)], w[at.first(2 * j + 1)]) : 0ull;
            const uint64_t wv = at.mine ? f2(w[at.second(2 * j)], w[at.second(2 * j + 1)]) : 0ull;
            fc[j] = f2_mul(wv, c[j]);
            fs[j] = f2_mul(wu, s[j]);
            c[j] = f2_mul(wu, c[j]);
            s[j] = f2_neg(f2_mul(wv, s[j]));
          }
        } else {
#pragma unroll
          for (int j = 0; j < H; ++j) fs[j] = s[j], s[j] = f2_neg(s[j]), fc[j] = c[j];
        }
      }
      char* dst = static_cast<char*>(to.ptr) + (m.b * to.sn + m.i * to.sl + h0 * to.sh) * es;
      const int most = __reduce_max_sync(~0u, heads - h0);  // heads that some lane of the warp has
#pragma unroll
      for (int x = 0; x < kHeads; ++x) {
        if (x >= most) break;
        uint64_t u[H], v[H];
        if constexpr (kStages > 0) st.read(here + x * S::kBytes, ra[x], rb[x]);
        unpack<kF32, kInter>(ra[x], rb[x], u, v);
        if constexpr (kNorm) {
          uint64_t sq = 0ull;
#pragma unroll
          for (int j = 0; j < H; ++j) sq = f2_fma(u[j], u[j], f2_fma(v[j], v[j], sq));
          float ss = f2_lo(sq) + f2_hi(sq);
          for (int o = 1; o < (1 << shift); o <<= 1) ss += __shfl_xor_sync(~0u, ss, o);
          const float r = root_inverse<kF32>(fmaf(ss, inv_d, p.eps));
          const uint64_t rr = f2(r, r);
#pragma unroll
          for (int j = 0; j < H; ++j) u[j] = f2_mul(u[j], rr), v[j] = f2_mul(v[j], rr);
        }
#pragma unroll
        for (int j = 0; j < H; ++j) {
          const uint64_t pu = f2_mul(u[j], c[j]), pv = f2_mul(v[j], fc[j]);
          const uint64_t tu = f2_fma(v[j], s[j], pu), tv = f2_fma(u[j], fs[j], pv);
          if constexpr (kPartial) {  // an element that passes does so whatever its neighbour holds
            const bool lo = at.pair + 2 * j < p.pairs, hi = at.pair + 2 * j + 1 < p.pairs;
            u[j] = f2_select(lo, hi, tu, pu);
            v[j] = f2_select(lo, hi, tv, pv);
          } else {
            u[j] = tu, v[j] = tv;
          }
        }
        if (live && h0 + x < heads) {
          uint4 oa, ob;
          pack<kF32, kInter>(u, v, oa, ob);
          __stcs(reinterpret_cast<uint4*>(dst + (x * to.sh + at.a) * es), oa);
          __stcs(reinterpret_cast<uint4*>(dst + (x * to.sh + at.b) * es), ob);
        }
      }
    }
  }
}

// The gradient under the norm. Blocks [0, bq) do q, the others k; a block's threads step over its part's items.
//
// A chunk is the rows of kHeads heads, x and the gradient, which go through shared memory by asynchronous copies, kStages -
// 1 chunks ahead (a 32k training step with loads into registers 301 us, with 2 heads a chunk).
struct BwdPart {
  int bq, slices_q, per_q, slices_k, per_k;
};
template <int kHeads, int kStages>
__host__ __device__ constexpr int bwd_smem() {
  return kStages * kHeads * 2 * kThreads * 2 * 16;
}

template <bool kF32, bool kInter, bool kPartial, int kHeads, int kStages>
__global__ void __launch_bounds__(kThreads, kBwdBlocks) norm_rope_bwd_kernel(const __grid_constant__ NormRopeParams p, const __grid_constant__ BwdPart q) {
  constexpr int N = Piece<kF32>::kN, H = N / 2;
  __shared__ Tables tables;
  using S = Staged<kF32, !kInter && !kPartial>;
  extern __shared__ __align__(16) uint8_t staged[];  // [stage][head][x, gradient] of S::kBytes
  static_assert(bwd_smem<kHeads, kStages>() >= kThreads * 2 * N * 4, "the sums take its place");
  load_tables<true>(p, tables);
  constexpr int es = kF32 ? 4 : 2;
  const int shift = lane_shift(p.d, N);
  const Place<kInter, N> at(threadIdx.x & ((1 << shift) - 1), p.d, p.pairs);
  const bool is_k = (int)blockIdx.x >= q.bq;
  const int64_t block = is_k ? blockIdx.x - q.bq : blockIdx.x, blocks = is_k ? gridDim.x - q.bq : q.bq;
  const int heads = is_k ? p.hk : p.hq, slices = is_k ? q.slices_k : q.slices_q, per = is_k ? q.per_k : q.per_q;
  const Seq4 &from = is_k ? p.k : p.q, &grad = is_k ? p.gk : p.gq, &to = is_k ? p.ko : p.qo;
  const int64_t total = ((int64_t)p.n * p.l * slices) << shift, first = block * kThreads + threadIdx.x, step = blocks * kThreads;
  const float inv_d = 1.f / (float)p.d;
  uint64_t wu[H], wv[H], du[H], dv[H];  // weights and their gradients' sums, of this lane's pairs
#pragma unroll
  for (int j = 0; j < H; ++j) {
    const float* w = tables.w[is_k];
    wu[j] = at.mine ? f2(w[at.first(2 * j)], w[at.first(2 * j + 1)]) : 0ull;
    wv[j] = at.mine ? f2(w[at.second(2 * j)], w[at.second(2 * j + 1)]) : 0ull;
    du[j] = dv[j] = 0ull;
  }
  // what is copied next: chunk `ahead` of item `it_ahead`
  const S st(shift, p.d, at.a, at.b, at.mine);
  int64_t it_ahead = first;
  int ahead = 0, stage_ahead = 0, h_ahead = 0;
  const char *src = nullptr, *gsrc = nullptr;
  auto copy_next = [&]() {
    if ((it_ahead & ~int64_t(31)) < total) {
      if (ahead == 0) {
        const Item m(p, it_ahead < total ? it_ahead : 0, shift, slices, per);
        h_ahead = m.chunk0 * kHeads;
        src = static_cast<const char*>(from.ptr) + (m.b * from.sn + m.i * from.sl + h_ahead * from.sh) * es;
        gsrc = static_cast<const char*>(grad.ptr) + (m.b * grad.sn + m.i * grad.sl + h_ahead * grad.sh) * es;
      }
#pragma unroll
      for (int x = 0; x < kHeads; ++x) {
        const bool read = it_ahead < total && h_ahead + x < heads;
        const uint32_t area = smem_u32(staged) + (stage_ahead * kHeads + x) * 2 * S::kBytes;
        st.copy(area, read ? src + x * from.sh * es : src, read);  // src: an address that is one
        st.copy(area + S::kBytes, read ? gsrc + x * grad.sh * es : gsrc, read);
      }
      h_ahead += kHeads;
      src += kHeads * from.sh * es;
      gsrc += kHeads * grad.sh * es;
      if (++ahead == per) ahead = 0, it_ahead += step;
    }
    stage_ahead = stage_ahead + 1 == kStages ? 0 : stage_ahead + 1;
    st.commit();
  };
#pragma unroll
  for (int z = 0; z < kStages - 1; ++z) copy_next();
  int stage = 0;
  for (int64_t it = first; (it & ~int64_t(31)) < total; it += step) {
    const bool live = it < total && at.mine;
    const Item m(p, it < total ? it : 0, shift, slices, per);
    uint64_t c[H], s[H];
    angles<N>(p, tables, m.b, m.i, at.mine ? at.pair : p.pairs, 0, c, s);
    int h0 = m.chunk0 * kHeads;
    char* dst = static_cast<char*>(to.ptr) + (m.b * to.sn + m.i * to.sl + h0 * to.sh) * es;
    for (int x0 = 0; x0 < per; ++x0, h0 += kHeads, dst += kHeads * to.sh * es) {
      st.been_read();
      copy_next();
      st.template there<kStages - 1>();
      const uint8_t* here = staged + stage * kHeads * 2 * S::kBytes;
      stage = stage + 1 == kStages ? 0 : stage + 1;
      const int most = __reduce_max_sync(~0u, heads - h0);
#pragma unroll
      for (int x = 0; x < kHeads; ++x) {
        if (x >= most) break;
        uint64_t u[H], v[H], gu[H], gv[H];
        uint4 ia, ib;
        st.read(here + x * 2 * S::kBytes, ia, ib);
        unpack<kF32, kInter>(ia, ib, u, v);
        st.read(here + (x * 2 + 1) * S::kBytes, ia, ib);
        unpack<kF32, kInter>(ia, ib, gu, gv);
        uint64_t sq = 0ull, dot2 = 0ull, yu[H], yv[H];
#pragma unroll
        for (int j = 0; j < H; ++j) {
          // turned back: (g_u c + g_v s, g_v c - g_u s)
          const uint64_t pu = f2_mul(gu[j], c[j]), pv = f2_mul(gv[j], c[j]);
          const uint64_t tu = f2_fma(gv[j], s[j], pu), tv = f2_fma(gu[j], f2_neg(s[j]), pv);
          if constexpr (kPartial) {
            const bool lo = at.pair + 2 * j < p.pairs, hi = at.pair + 2 * j + 1 < p.pairs;
            gu[j] = f2_select(lo, hi, tu, pu);
            gv[j] = f2_select(lo, hi, tv, pv);
          } else {
            gu[j] = tu, gv[j] = tv;
          }
          yu[j] = f2_mul(gu[j], wu[j]);
          yv[j] = f2_mul(gv[j], wv[j]);
          sq = f2_fma(u[j], u[j], f2_fma(v[j], v[j], sq));
          dot2 = f2_fma(yu[j], u[j], f2_fma(yv[j], v[j], dot2));
        }
        float ss = f2_lo(sq) + f2_hi(sq), dot = f2_lo(dot2) + f2_hi(dot2);
        for (int o = 1; o < (1 << shift); o <<= 1) {
          ss += __shfl_xor_sync(~0u, ss, o);
          dot += __shfl_xor_sync(~0u, dot, o);
        }
        if (!(live && h0 + x < heads)) continue;
        const float r = root_inverse<kF32>(fmaf(ss, inv_d, p.eps)), k = -dot * inv_d * r * r * r;
        const uint64_t rr = f2(r, r), kk = f2(k, k);
#pragma unroll
        for (int j = 0; j < H; ++j) {
          du[j] = f2_fma(gu[j], f2_mul(u[j], rr), du[j]);
          dv[j] = f2_fma(gv[j], f2_mul(v[j], rr), dv[j]);
          u[j] = f2_fma(u[j], kk, f2_mul(yu[j], rr));
          v[j] = f2_fma(v[j], kk, f2_mul(yv[j], rr));
        }
        uint4 oa, ob;
        pack<kF32, kInter>(u, v, oa, ob);
        __stcs(reinterpret_cast<uint4*>(dst + (x * to.sh + at.a) * es), oa);
        __stcs(reinterpret_cast<uint4*>(dst + (x * to.sh + at.b) * es), ob);
      }
    }
  }
  asm volatile("cp.async.wait_all;" ::: "memory");
  if ((is_k ? p.dwk : p.dwq) == nullptr) return;
  __syncthreads();
  // rows of d: one of every group of lanes
  float* sums = reinterpret_cast<float*>(staged);
  if (at.mine) {
    float* row = sums + (threadIdx.x >> shift) * p.d;
#pragma unroll
    for (int j = 0; j < N; ++j) {
      row[at.first(j)] = j & 1 ? f2_hi(du[j / 2]) : f2_lo(du[j / 2]);
      row[at.second(j)] = j & 1 ? f2_hi(dv[j / 2]) : f2_lo(dv[j / 2]);
    }
  }
  __syncthreads();
  for (int c = threadIdx.x; c < p.d; c += kThreads) {
    float s = 0.f;
    for (int r = 0; r < (kThreads >> shift); ++r) s += sums[r * p.d + c];
    p.partial[(int64_t)blockIdx.x * p.d + c] = s;
  }
}

// The blocks' sums, 32 columns a block, a warp every kSumWarps-th of them.
constexpr int kSumWarps = 32;
__global__ void __launch_bounds__(kSumWarps * 32) norm_rope_weight_kernel(const __grid_constant__ NormRopeParams p, int bq, int blocks) {
  __shared__ float part[kSumWarps][33];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, c = blockIdx.x * 32 + lane, is_k = blockIdx.y;
  grid_dependency_wait();
  void* out = is_k ? p.dwk : p.dwq;
  if (out == nullptr) return;
  const int b0 = is_k ? bq : 0, b1 = is_k ? blocks : bq;
  float s = 0.f;
  if (c < p.d) {
#pragma unroll 8
    for (int b = b0 + warp; b < b1; b += kSumWarps) s += p.partial[(int64_t)b * p.d + c];
  }
  part[warp][lane] = s;
  __syncthreads();
  s = part[lane][warp];  // column blockIdx.x * 32 + warp, part `lane`
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(~0u, s, o);
  const int col = blockIdx.x * 32 + warp;
  if (lane == 0 && col < p.d) {
    if (is_k ? p.wk_f32 : p.wq_f32)
      static_cast<float*>(out)[col] = s;
    else
      static_cast<__nv_bfloat16*>(out)[col] = __float2bfloat16(s);
  }
}

// A runtime truth value as a type.
template <typename F>
auto with(bool x, F f) {
  return x ? f(std::true_type{}) : f(std::false_type{});
}

// Into how many slices the chunks of a token go, so that `threads` threads have work, and how many chunks that is each.
struct Slices {
  int slices, per;
  Slices(int64_t lanes_of_tokens, int chunks, int64_t threads) {
    int64_t want = lanes_of_tokens > 0 ? (threads + lanes_of_tokens - 1) / lanes_of_tokens : 1;
    if (want > chunks) want = chunks;
    if (want < 1) want = 1;
    per = (int)((chunks + want - 1) / want);
    slices = per > 0 ? (chunks + per - 1) / per : 0;
  }
};

constexpr int kBwdMaxBlocks = 2048;

template <bool kF32, bool kNorm, bool kInter, bool kPartial>
cudaError_t launch_fwd(const NormRopeParams& p, cudaStream_t s) {
  constexpr int N = kF32 ? 4 : 8;
  const int shift = host_lane_shift(p.d, N);
  int sms = 0;
  cudaError_t e = device_sm_count(&sms);
  if (e != cudaSuccess) return e;
  const int chunks = (p.hq + kFwdHeads - 1) / kFwdHeads + (p.hk + kFwdHeads - 1) / kFwdHeads;
  const Slices c(((int64_t)p.n * p.l) << shift, chunks, (int64_t)sms * kSmThreads);
  int64_t blocks = ((((int64_t)p.n * p.l * c.slices) << shift) + kThreads - 1) / kThreads;
  if (blocks > (int64_t(1) << 30)) blocks = int64_t(1) << 30;  // the kernel strides over the rest
  auto launch = [&](auto kern, int smem) {
    return launch_dependent(kern, dim3((unsigned)blocks), kThreads, smem, s, p, c.slices, c.per);
  };
  if constexpr (kNorm && !kF32) {
    constexpr int smem = kFwdStages * kFwdHeads * Staged<kF32, true>::kBytes;
    if (c.per > 1) return launch(norm_rope_kernel<kF32, kNorm, kInter, kPartial, kFwdHeads, kFwdStages>, smem);
  }
  return launch(norm_rope_kernel<kF32, kNorm, kInter, kPartial, kFwdHeads, 0>, 0);
}

template <bool kF32, bool kInter, bool kPartial>
cudaError_t launch_bwd(const NormRopeParams& p, cudaStream_t s, int* bq, int* blocks) {
  constexpr int N = kF32 ? 4 : 8;
  static PerContext<int> cache;
  int cap = 0;
  auto kern = norm_rope_bwd_kernel<kF32, kInter, kPartial, kBwdHeads, kBwdStages>;
  constexpr int smem = bwd_smem<kBwdHeads, kBwdStages>();
  cudaError_t e = wave_cap(cache, kern, kThreads, smem, &cap);
  if (e != cudaSuccess) return e;
  if (cap > kBwdMaxBlocks) cap = kBwdMaxBlocks;
  const int shift = host_lane_shift(p.d, N);
  const int64_t lanes = ((int64_t)p.n * p.l) << shift;
  const int cq = (p.hq + kBwdHeads - 1) / kBwdHeads, ck = (p.hk + kBwdHeads - 1) / kBwdHeads;
  // a wave shared out by work, at least a block for each that has some
  int64_t nq = cq + ck > 0 ? (int64_t)((double)cap * cq / (cq + ck) + 0.5) : 0;
  if (cq > 0 && nq < 1) nq = 1;
  if (ck > 0 && nq > cap - 1) nq = cap - 1;
  int64_t nk = ck > 0 ? cap - nq : 0;
  const Slices sq(lanes, cq, nq * kThreads), sk(lanes, ck, nk * kThreads);
  auto most = [&](const Slices& c) { return (lanes * c.slices + kThreads - 1) / kThreads; };
  if (nq > most(sq)) nq = most(sq);
  if (nk > most(sk)) nk = most(sk);
  *bq = (int)nq;
  *blocks = (int)(nq + nk);
  if (*blocks == 0) return cudaSuccess;
  const BwdPart part{*bq, sq.slices, sq.per, sk.slices, sk.per};
  return launch_dependent(kern, dim3((unsigned)*blocks), kThreads, smem, s, p, part);
}

}  // namespace

cudaError_t launch_norm_rope(const NormRopeParams& p, cudaStream_t s, int* nlaunch) {
  const cudaError_t e = with(p.is_f32, [&](auto f32) {
    return with(p.norm, [&](auto norm) {
      return with(p.interleaved, [&](auto inter) {
        return with(2 * p.pairs != p.d, [&](auto partial) {
          return launch_fwd<decltype(f32)::value, decltype(norm)::value, decltype(inter)::value, decltype(partial)::value>(p, s);
        });
      });
    });
  });
  if (e == cudaSuccess) *nlaunch += 1;
  return e;
}

size_t norm_rope_bwd_workspace(int64_t d) { return (size_t)kBwdMaxBlocks * (size_t)d * 4; }

cudaError_t launch_norm_rope_bwd(const NormRopeParams& p, cudaStream_t s, int* nlaunch) {
  int bq = 0, blocks = 0;
  cudaError_t e = with(p.is_f32, [&](auto f32) {
    return with(p.interleaved, [&](auto inter) {
      return with(2 * p.pairs != p.d, [&](auto partial) {
        return launch_bwd<decltype(f32)::value, decltype(inter)::value, decltype(partial)::value>(p, s, &bq, &blocks);
      });
    });
  });
  if (e != cudaSuccess) return e;
  if (blocks > 0) *nlaunch += 1;
  if (p.dwq == nullptr && p.dwk == nullptr) return e;
  e = launch_dependent(norm_rope_weight_kernel, dim3((unsigned)((p.d + 31) / 32), 2), kSumWarps * 32, 0, s, p, bq, blocks);
  if (e == cudaSuccess) *nlaunch += 1;
  return e;
}

}  // namespace bea
