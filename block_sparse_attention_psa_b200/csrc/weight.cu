// weight.cu -- accumulated attention weight of each cached key:
//   score_j += sum over the queries i that see j of e^{s_ij - lse_i},
//   s_ij = q_i . k_j / sqrt(d),
// the column sums of the softmax matrix, recomputed from the queries' lse
// (nothing of size queries x keys is stored).
//
// One product S^T = K Q^T per tile of 128 keys x 128 queries (tcgen05, both
// operands K-major in shared memory): a thread owns one TMEM lane, i.e. one
// key, so a key's sum runs inside a thread and needs no exchange.  The lse of
// the queries runs along the columns and is read from shared memory, four
// columns per broadcast load; a warp of its own gathers it tile by tile (-lse
// log2 e, -inf in columns without a query, with a mark for columns of -inf), up
// to four tiles ahead. (Laid out by a kernel of its own beforehand it cost a
// launch: 48 queries of 1000 keys 14.7 -> 13.5 us, 64 of 128K 109 -> 108.)
//
//  * Decode reads K once for few queries: bound by DRAM.  A prefill does 2 d
//    operations and one exponential per (query, key) pair: an SM's tensor
//    core takes 256 cycles for a tile at d = 64 and 512 at d = 128, its 16
//    exponentials a cycle 1024, so it is bound by the exponentials.
//  * Up to 32 queries per key (16 at d = 128; decode): stream_kernel. 16 keys x 8 queries per
//    mma.sync, with K going from DRAM straight to registers: a thread's four
//    16-byte pieces of two key rows are its A operands, in an order of the d
//    features that the queries' registers share. No shared memory and no barriers, so nothing
//    stands between the loads; the legacy tensor path has an order of
//    magnitude to spare at this ratio.
//  * More: weight_kernel. Unit: a pair of key tiles (256 keys) of one KV head,
//    held in shared memory, with the query tiles streamed past it, so that a
//    query tile is loaded once for both key tiles; each key tile has two S
//    buffers (512 TMEM columns in all) and two warpgroups that take half the
//    columns each, four warps per scheduler in all (with two, a tile took 2700
//    cycles instead of ~1900: loads from TMEM, waits and chains of the
//    polynomial were exposed).  One warp
//    works out the units and publishes them; the others only step through
//    them (divisions in every role had cost more than the products).
//  * Query tiles: T >= 128 tokens: 128 tokens of one head, so that causal
//    tiles past the diagonal are skipped; fewer: up to 128 of the G T rows
//    that share the KV head, over several sequences when they share the keys.
//    A head's pairs that lie in one CTA's run make one unit, and where all its
//    query tiles fit the ring (two, at d = 64 four) they stay for all of them
//    (64-token window 111 -> 107 us).
//  * Units of equal cost (T < 128) lie on one line that is cut into equal
//    runs; a prefill's go to the CTAs in turn, forwards and backwards, heaviest
//    (fewest keys hidden) first.  Where that leaves the last SM at work for longer
//    the query tiles of a unit are split over several (make_plan), whose sums a
//    second kernel adds in a fixed order.
//  * One in eight exponentials runs on the FMA pipe (exp2_parts, 2.1e-7), whose
//    other work leaves it half idle (8K prefill 354 -> 349 us, 64-token window
//    121 -> 114; two in eight 348 and 117, three 380 and 127: the chains of
//    the polynomial then cost more than the unit is relieved of).
//  * Sums: 128 columns in four fp32 accumulators, tile sums added with a
//    compensation term (a key of a long prefill sums 10^5 terms). The terms
//    inside a tile (32 in a row) and the parts of a split unit are added
//    without one: the 8K prefill is off by 5.6e-7 relative to 64 bits, a plain
//    fp32 form by 1.3e-7; the window and single tokens by 3e-8, as that is.
// Measured on one B200 (device time): one token of 48 caches of up to 4099,
// 8 KV heads of 3, d = 64: 23 us, 5.5 TB/s (floor 19 us: the reads of K; of 64
// caches of up to 4096 at d = 128 51 us, 6.3 TB/s). Last
// 64 queries of a 128K prefill, 8 KV heads of 4, d = 128: 108 us (60:
// exponentials). A whole 8K causal prefill of 32 heads: 345 us, 797 TFLOP/s
// (floors: 238 exponentials alone, 166 tensor core). A tile of 128 x 128 x 2
// takes 2350 cycles, 1800 of them sums (88% of the exponential unit), the rest
// hand-overs between tiles, and 2100 of 6100 between units of two tiles.
// Every wait is bounded.
#include <climits>
#include <cmath>

#include "internal.h"
#include "sm100.cuh"

namespace psa {
namespace {

constexpr int kThreads = 640;      // WG0: K/Q loads, MMA issue, lse loads, units; WG1..4: half the columns of a key tile each
constexpr int kRegsProducer = 64;  // 128 x 64 + 512 x 104 = 640 x 96
constexpr int kRegsSum = 104;
constexpr int kLse = 4;            // query tiles whose lse is in shared memory
constexpr int kNl = 132;           // words of a tile's lse: 128 columns, then per 32 of them whether one is -inf
constexpr int kRing = 4;           // units in flight
constexpr int kPlanSms = 148;      // SMs the split is planned for (fixed: it sizes the workspace)
constexpr int kPoly = 1;           // of eight pairs of exponentials, those on the FMA pipe
constexpr float kLog2e = 1.4426950408889634f;

template <int D>
struct Cfg {
  static constexpr int kChunks = D / 64;
  static constexpr int kTile = 128 * D * 2;
  static constexpr int kQStages = D == 128 ? 2 : 4;
  static constexpr int kOffK = 0;               // two pairs of key tiles
  static constexpr int kOffQ = 4 * kTile;
  static constexpr int kOffLse = kOffQ + kQStages * kTile;
  static constexpr int kOffMisc = kOffLse + kLse * kNl * 4;
  static constexpr int kSmem = kOffMisc + 1024 + 2048 + 1024;  // barriers, half sums, alignment slack
  static_assert(kSmem <= 232448, "shared memory of one CTA");
};

struct Params {
  const float* lse;
  const int* key_len;
  const float* score_in;  // nullable
  float* score_out;
  float* part;            // [Z][Bk * Hkv][C] when Z > 1
  int B, G, Hkv, T, Bk, n, C, causal;
  int GT, by_head;        // by_head: query tiles of one head
  int nb, rb;             // query tile: sequences x rows (box)
  int tiles;              // by_head: tiles of one head; else row tiles of a KV head (all n sequences)
  int all;                // tiles of a KV head: n G heads' (by_head) or `tiles`
  int N;                  // columns of the products: nb * rb rounded up to 16
  int Z, pairs;
  int resident;           // a unit's query tiles stay on chip for all its pairs
  long long units;
  float scale_log2;
  int* status;
  int stall;              // test hook: CTA 0 withholds its first hand-off of S^T
};

// A unit, as the scheduler publishes it.
struct Unit {
  int bk, hkv, key0, len;
  int nt;          // query tiles; -1 ends the walk
  int i, g, r0;    // first tile: sequence of the group, query head of the KV head (by_head), row
  int r_min;       // by_head: first visible row of every head
  int z;
  int np;          // pairs of key tiles, one after the other, with the same query tiles
  int pad;         // a multiple of 16 bytes: read as vectors
};
constexpr int kUnitInts = sizeof(Unit) / 4;
static_assert(kUnitInts == 12, "");

__device__ __forceinline__ void read_unit(Unit& x, const int* slot) {
  int4* w = reinterpret_cast<int4*>(&x);
#pragma unroll
  for (int i = 0; i < kUnitInts / 4; ++i)
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(w[i].x), "=r"(w[i].y), "=r"(w[i].z), "=r"(w[i].w)
                 : "r"(smem_u32(slot + 4 * i))
                 : "memory");
}

__device__ __forceinline__ void mbar_drain(uint64_t* bar, uint32_t parity) {
  const long long t0 = clock64();
  while (!mbar_try_wait(bar, parity)) {
    if (clock64() - t0 > kWaitCycles) return;
  }
}
template <int N>
__device__ __forceinline__ void reg_dealloc() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;\n" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void reg_alloc() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;\n" ::"n"(N));
}

__device__ __forceinline__ int clamped_len(const Params& p, int bk) {
  const int n = p.key_len ? p.key_len[bk] : p.C;
  return min(max(n, 0), p.C);
}

// Query tile of a unit; next() steps to the following one.
struct Tile {
  int i, g, r0;
  __device__ __forceinline__ void next(const Params& p, const Unit& x) {
    if (p.by_head) {
      r0 += 128;
      if (r0 >= p.T) {
        r0 = x.r_min;
        if (++g == p.G) {
          g = 0;
          ++i;
        }
      }
    } else if (p.GT >= 128) {
      r0 += 128;
      if (r0 >= p.GT) {
        r0 = 0;
        ++i;
      }
    } else {
      i += p.nb;
    }
  }
};

// Unit (row of heads bh, key pair, part z) with its tiles.
__device__ __forceinline__ Unit make_unit(const Params& p, int bh, int pair, int z, int len) {
  Unit x;
  x.bk = bh / p.Hkv;
  x.hkv = bh - x.bk * p.Hkv;
  x.key0 = 256 * pair;
  x.len = len;
  x.z = z;
  x.np = 1;
  x.r_min = 0;
  int per = p.tiles, total = p.tiles;
  if (p.by_head) {
    // token t sees key j iff j <= len - T + t
    const int t_min = p.causal ? max(0, x.key0 - (len - p.T)) / 128 : 0;
    x.r_min = 128 * t_min;
    per = max(p.tiles - t_min, 0);
    total = p.n * p.G * per;
  }
  if (x.key0 >= len) total = 0;
  const int f0 = static_cast<int>(static_cast<long long>(total) * z / p.Z);
  const int f1 = static_cast<int>(static_cast<long long>(total) * (z + 1) / p.Z);
  x.nt = f1 - f0;
  x.i = x.g = x.r0 = 0;
  if (x.nt > 0) {
    if (p.by_head) {
      const int o = f0 / per;
      x.i = o / p.G;
      x.g = o - x.i * p.G;
      x.r0 = x.r_min + 128 * (f0 - o * per);
    } else if (p.GT >= 128) {
      const int of = (p.GT + 127) / 128;
      x.i = f0 / of;
      x.r0 = 128 * (f0 - x.i * of);
    } else {
      x.i = f0 * p.nb;
    }
  }
  return x;
}

// Sum of 2^(v * scale + nl) over 32 columns; nl from shared memory.
__device__ __forceinline__ void sum32(const float (&v)[32], const float* nl, float scale, float (&a)[4]) {
#pragma unroll
  for (int i = 0; i < 32; i += 4) {
    const float4 l4 = *reinterpret_cast<const float4*>(nl + i);
    float x0, x1, x2, x3;
    ffma2(x0, x1, v[i], v[i + 1], scale, scale, l4.x, l4.y);
    ffma2(x2, x3, v[i + 2], v[i + 3], scale, scale, l4.z, l4.w);
    fadd2(a[0], a[1], a[0], a[1], ex2_approx(x0), ex2_approx(x1));
    const int k = (i / 4) % 4;
    if (k < kPoly) {
      float p0, p1, s0, s1;
      exp2_parts(x2, x3, p0, p1, s0, s1);
      ffma2(a[2], a[3], p0, p1, s0, s1, a[2], a[3]);
    } else {
      fadd2(a[2], a[3], a[2], a[3], ex2_approx(x2), ex2_approx(x3));
    }
  }
}

template <int D, bool FP16>
__global__ void __launch_bounds__(kThreads, 1)
    weight_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK, const Params p) {
  using C = Cfg<D>;
  constexpr int kQ = C::kQStages;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sK = smem + C::kOffK;
  uint8_t* sQ = smem + C::kOffQ;
  float* sLse = reinterpret_cast<float*>(smem + C::kOffLse);  // [kLse][kNl] -lse in log2 units
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::kOffMisc);
  uint64_t* k_full = bars + 0;    // [2] a pair of key tiles landed  (TMA)
  uint64_t* k_empty = bars + 2;   // [2] its last product done       (commit)
  uint64_t* q_full = bars + 4;    // [kQ]
  uint64_t* q_empty = bars + 8;   // [kQ]
  uint64_t* s_full = bars + 12;   // [2 streams][2] S^T ready        (commit)
  uint64_t* s_empty = bars + 16;  // [2 streams][2] read             (4 warps)
  uint64_t* l_full = bars + 20;   // [kLse] lse of a query tile      (warp 2)
  uint64_t* l_empty = bars + 24;  // [kLse] read                     (16 warps)
  uint64_t* u_full = bars + 28;   // [kRing] a unit published
  uint64_t* u_empty = bars + 32;  // [kRing] read by loads, lse, MMA issue, 16 warps
  uint64_t* drain = bars + 36;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::kOffMisc + 320);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  int* start_bk = reinterpret_cast<int*>(tmem_slot + 2);
  long long* start_off = reinterpret_cast<long long*>(smem + C::kOffMisc + 336);
  long long* red = start_off + 1;                                                  // [kThreads / 32]
  int* ring = reinterpret_cast<int*>(smem + C::kOffMisc + 768);  // [kRing][kUnitInts]
  float* half_sum = reinterpret_cast<float*>(smem + C::kOffMisc + 1024);           // [parity][key tile][128]

  const int warp = uniform(threadIdx.x / 32), lane = threadIdx.x % 32;
  if (threadIdx.x == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&k_full[i], 1);
      mbar_init(&k_empty[i], 1);
    }
    for (int i = 0; i < kQ; ++i) {
      mbar_init(&q_full[i], 1);
      mbar_init(&q_empty[i], 1);
    }
    for (int i = 0; i < 4; ++i) {
      mbar_init(&s_full[i], 1);
      mbar_init(&s_empty[i], 8);
    }
    for (int i = 0; i < kLse; ++i) {
      mbar_init(&l_full[i], 1);
      mbar_init(&l_empty[i], 16);
    }
    for (int i = 0; i < kRing; ++i) {
      mbar_init(&u_full[i], 1);
      mbar_init(&u_empty[i], 19);
    }
    mbar_init(drain, 1);
    *abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, 512);
    tmem_relinquish();
  }
  if (warp == 2 && lane == 0) {
    tma_prefetch_desc(&tmQ);
    tma_prefetch_desc(&tmK);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tbase = *tmem_slot;
  grid_dep_launch();
  grid_dep_wait();

  if (blockIdx.x == 0) {
    // one writer of the status word: the lengths of all key sets
    bool bad = false;
    if (p.key_len)
      for (int i = threadIdx.x; i < p.Bk; i += kThreads) {
        const int n = p.key_len[i];
        bad |= n < 0 || n > p.C;
      }
    bad = __syncthreads_or(bad);
    if (threadIdx.x == 0) *p.status = bad ? kStatusLength : 0;
  }
  // Units of equal cost: the line of all valid (key set, head, pair, part),
  // and where this CTA's run of it starts.
  long long x0 = 0, x1 = 0;
  if (!p.by_head) {
    const int per = p.Hkv * p.Z;
    long long mine = 0;
    for (int i = threadIdx.x; i < p.Bk; i += kThreads)
      mine += static_cast<long long>((clamped_len(p, i) + 255) / 256) * per;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) mine += __shfl_xor_sync(0xffffffffu, mine, o);
    if (lane == 0) red[warp] = mine;
    __syncthreads();
    long long total = 0;
    for (int w = 0; w < kThreads / 32; ++w) total += red[w];
    x0 = total * blockIdx.x / gridDim.x;
    x1 = total * (blockIdx.x + 1) / gridDim.x;
    long long run = 0;
    for (int b0 = 0; b0 < p.Bk && x0 < x1; b0 += kThreads) {
      const int bk = b0 + threadIdx.x;
      const long long t = bk < p.Bk ? static_cast<long long>((clamped_len(p, bk) + 255) / 256) * per : 0;
      long long inc = t;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const long long u = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += u;
      }
      __syncthreads();
      if (lane == 31) red[warp] = inc;
      __syncthreads();
      long long base = run;
      for (int w = 0; w < kThreads / 32; ++w) {
        base += w < warp ? red[w] : 0;
        run += red[w];
      }
      if (base + inc - t <= x0 && x0 < base + inc) {
        *start_bk = bk;
        *start_off = base + inc - t;
      }
    }
    __syncthreads();
  }

  if (warp < 4) {
    reg_dealloc<kRegsProducer>();
    int nu = 0;
    // the next unit for a single thread or a whole warp; nt < 0 at the end or on a timeout
    auto next_unit = [&](Unit& x, bool reads) {
      const int slot = nu % kRing;
      if (!mbar_sleep(&u_full[slot], (nu / kRing) & 1, abort_flag, p.status)) {
        x.nt = -1;
        return;
      }
      read_unit(x, ring + slot * kUnitInts);
      if (reads) mbar_arrive(&u_empty[slot]);
      ++nu;
    };
    if (warp == 3) {
      // ---------------------------------------------------- units
      if (lane == 0) {
        bool ok = true;
        auto publish = [&](const Unit& x) -> bool {
          const int slot = nu % kRing;
          if (nu >= kRing && !mbar_sleep(&u_empty[slot], ((nu / kRing) - 1) & 1, abort_flag, p.status)) return false;
          *reinterpret_cast<Unit*>(ring + slot * kUnitInts) = x;
          mbar_arrive(&u_full[slot]);
          ++nu;
          return true;
        };
        if (p.by_head) {
          const int BH = p.Bk * p.Hkv, g = static_cast<int>(gridDim.x), c = static_cast<int>(blockIdx.x);
          for (long long w = 0; ok && w * g < p.units; ++w) {
            const long long u = w * g + ((w & 1) ? g - 1 - c : c);
            if (u >= p.units) continue;
            const long long pz = u / BH;
            const int bh = static_cast<int>(u - pz * BH), pair = static_cast<int>(pz / p.Z);
            ok = publish(make_unit(p, bh, pair, static_cast<int>(pz - static_cast<long long>(pair) * p.Z),
                                   clamped_len(p, bh / p.Hkv)));
          }
        } else if (x0 < x1) {
          int bk = *start_bk;
          int len = clamped_len(p, bk), pairs = (len + 255) / 256;
          long long rel = x0 - *start_off;  // place inside the key set: (head, pair, part)
          int hkv = static_cast<int>(rel / (static_cast<long long>(pairs) * p.Z));
          rel -= static_cast<long long>(hkv) * pairs * p.Z;
          int pair = static_cast<int>(rel / p.Z), z = static_cast<int>(rel - static_cast<long long>(pair) * p.Z);
          for (long long x = x0; ok && x < x1; ++x) {
            Unit u = make_unit(p, bk * p.Hkv + hkv, pair, z, len);
            if (p.Z == 1) {
              // the rest of the head's pairs that lie in the run: one unit
              u.np = static_cast<int>(min(static_cast<long long>(pairs - pair), x1 - x));
              x += u.np - 1;
              pair += u.np - 1;
            }
            ok = publish(u);
            if (++z < p.Z) continue;
            z = 0;
            if (++pair < pairs) continue;
            pair = 0;
            if (++hkv < p.Hkv || x + 1 >= x1) continue;
            hkv = 0;
            do {  // the run goes on, so a key set with keys follows
              ++bk;
              len = clamped_len(p, bk);
            } while (len == 0);
            pairs = (len + 255) / 256;
          }
        }
        Unit end = {};
        end.nt = -1;
        if (ok) publish(end);
      }
    } else if (warp == 0 && lane == 0) {
      // ---------------------------------------------------- K and Q loads
      int ku = 0, qt = 0;  // pairs and query tiles loaded
      bool ok = true;
      for (;;) {
        Unit x;
        next_unit(x, true);
        if (x.nt < 0 || !ok) break;
        if (x.nt == 0) continue;
        const uint32_t bytes = static_cast<uint32_t>(p.nb * p.rb) * 128 * C::kChunks;
        for (int pp = 0; ok && pp < x.np; ++pp) {
          const int kb = ku & 1, key0 = x.key0 + 256 * pp;
          if (!(ok = mbar_sleep(&k_empty[kb], ((ku >> 1) & 1) ^ 1, abort_flag, p.status))) break;
          // 64-key boxes; none that starts past the length
          const int boxes = min(4, (x.len - key0 + 63) / 64);
          mbar_arrive_expect_tx(&k_full[kb], boxes * 64 * 128 * C::kChunks);
          for (int i = 0; i < boxes; ++i)
#pragma unroll
            for (int ch = 0; ch < C::kChunks; ++ch)
              tma_load_3d(&tmK, sK + (2 * kb + (i >> 1)) * C::kTile + ch * 16384 + (i & 1) * 8192, &k_full[kb],
                          64 * ch, key0 + 64 * i, x.bk * p.Hkv + x.hkv);
          ++ku;
          if (pp > 0 && p.resident) continue;
          Tile t = {x.i, x.g, x.r0};
          for (int f = 0; f < x.nt; ++f, ++qt) {
            const int st = qt % kQ;
            if (!(ok = mbar_sleep(&q_empty[st], ((qt / kQ) & 1) ^ 1, abort_flag, p.status))) break;
            mbar_arrive_expect_tx(&q_full[st], bytes);
#pragma unroll
            for (int ch = 0; ch < C::kChunks; ++ch)
              tma_load_4d(&tmQ, sQ + st * C::kTile + ch * 16384, &q_full[st], 64 * ch, t.r0,
                          p.by_head ? x.hkv * p.G + t.g : x.hkv, x.bk * p.n + t.i);
            t.next(p, x);
          }
        }
      }
      // no bulk copy may still be writing shared memory when the CTA leaves
      for (int i = max(0, ku - 2); i < ku; ++i) mbar_drain(&k_full[i & 1], (i >> 1) & 1);
      for (int i = max(0, qt - kQ); i < qt; ++i) mbar_drain(&q_full[i % kQ], (i / kQ) & 1);
    } else if (warp == 2) {
      // ---------------------------------------------------- lse of the query tiles
      // -lse log2(e) in the order of the columns, -inf in columns without a
      // query, four columns a lane; the loads of a tile are under way before
      // its place is free.
      int qt = 0, at[4];
      bool in[4], ok = true;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int c = 32 * j + lane;
        if (p.by_head || p.GT >= 128) {
          at[j] = c;
          in[j] = true;
        } else {
          at[j] = c / p.GT;  // sequence of the tile
          in[j] = c < p.nb * p.GT;
        }
      }
      while (ok) {
        Unit x;
        next_unit(x, false);
        __syncwarp();
        // (lanes wait for themselves: one whose wait ran out has no unit)
        if (!__all_sync(0xffffffffu, x.nt >= 0)) break;
        const int nt = uniform(x.nt), np = uniform(x.np);
        if (lane == 0) mbar_arrive(&u_empty[(nu - 1) % kRing]);
        __syncwarp();
        for (int pp = 0; ok && pp < (p.resident ? 1 : np); ++pp) {
          Tile t = {x.i, x.g, x.r0};
          for (int f = 0; ok && f < nt; ++f, ++qt) {
            const int lt = qt % kLse;
            float* dst = sLse + kNl * lt;
            float l[4];
            const long long seq = static_cast<long long>(x.bk) * p.n + t.i;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const int c = 32 * j + lane;
              l[j] = -INFINITY;
              if (p.by_head) {
                if (t.r0 + c < p.T)
                  l[j] = p.lse[((seq * p.Hkv + x.hkv) * p.G + t.g) * p.T + t.r0 + c];
              } else if (p.GT >= 128) {
                if (t.r0 + c < p.GT) l[j] = p.lse[(seq * p.Hkv + x.hkv) * p.GT + t.r0 + c];
              } else if (in[j] && t.i + at[j] < p.n) {
                l[j] = p.lse[((seq + at[j]) * p.Hkv + x.hkv) * p.GT + c - at[j] * p.GT];
              }
            }
            ok = mbar_sleep(&l_empty[lt], ((qt / kLse) & 1) ^ 1, abort_flag, p.status);
            __syncwarp();
            if (!(ok = __all_sync(0xffffffffu, ok))) break;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              // a query that saw nothing (lse -inf) adds nothing
              const bool none = l[j] == -INFINITY;
              dst[32 * j + lane] = none ? -INFINITY : -l[j] * kLog2e;
              const int any = __any_sync(0xffffffffu, none);
              if (lane == 0) dst[128 + j] = __int_as_float(any);
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&l_full[lt]);
            __syncwarp();
            t.next(p, x);
          }
        }
      }
    } else if (warp == 1) {
      // ---------------------------------------------------- MMA issue
      // The whole warp walks the tiles in step; one elected lane issues.  The
      // lanes wait without a vote and agree on stopping once per pair.
      const uint64_t dK0 = sdesc_sw128(smem_u32(sK), 16, 1024);
      const uint64_t dQ0 = sdesc_sw128(smem_u32(sQ), 16, 1024);
      constexpr uint64_t kStep = C::kTile >> 4;
      const uint32_t idesc = idesc_f16_f32(FP16, 128, p.N, 0, 0);
      int ku = 0, qt = 0, it = 0;  // pairs, query tiles done with, products
      bool ok = true;
      while (ok) {
        Unit x;
        next_unit(x, false);
        __syncwarp();
        // (lanes wait for themselves: one whose wait ran out has no unit)
        if (!__all_sync(0xffffffffu, x.nt >= 0)) break;
        const int nt = uniform(x.nt), np = uniform(x.np);
        if (elect_one()) mbar_arrive(&u_empty[(nu - 1) % kRing]);
        __syncwarp();
        if (nt == 0) continue;
        for (int pp = 0; ok && pp < np; ++pp) {
          const bool release = !p.resident || pp == np - 1;  // of the query tiles
          const int kb = ku & 1;
          ok = mbar_sleep(&k_full[kb], (ku >> 1) & 1, abort_flag, p.status);
          for (int f = 0; f < nt; ++f, ++it) {
            const int st = (qt + f) % kQ, buf = it & 1;
            const uint32_t eh = ((it >> 1) & 1) ^ 1, qh = ((qt + f) / kQ) & 1;
            // one look at all three barriers, whose latencies then overlap
            const bool rq = mbar_try_wait(&q_full[st], qh), r0 = mbar_try_wait(&s_empty[buf], eh),
                       r1 = mbar_try_wait(&s_empty[2 + buf], eh);
            const uint64_t a = dK0 + 2 * kb * kStep, b = dQ0 + st * kStep;
            if (!rq) ok &= mbar_sleep(&q_full[st], qh, abort_flag, p.status);
            if (!r0) ok &= mbar_sleep(&s_empty[buf], eh, abort_flag, p.status);
            __syncwarp();
            tc_fence_after();
            if (elect_one()) {
#pragma unroll
              for (int kk = 0; kk < D / 16; ++kk)
                tc_mma_bf16(tbase + 128 * buf, a + (kk >> 2) * 1024 + (kk & 3) * 2,
                            b + (kk >> 2) * 1024 + (kk & 3) * 2, idesc, kk ? 1u : 0u);
              if (!(p.stall && blockIdx.x == 0 && it == 0)) tc_commit(&s_full[buf]);
            }
            if (!r1) ok &= mbar_sleep(&s_empty[2 + buf], eh, abort_flag, p.status);
            __syncwarp();
            tc_fence_after();
            if (elect_one()) {
#pragma unroll
              for (int kk = 0; kk < D / 16; ++kk)
                tc_mma_bf16(tbase + 256 + 128 * buf, a + kStep + (kk >> 2) * 1024 + (kk & 3) * 2,
                            b + (kk >> 2) * 1024 + (kk & 3) * 2, idesc, kk ? 1u : 0u);
              tc_commit(&s_full[2 + buf]);
              if (release) tc_commit(&q_empty[st]);
              if (f == nt - 1) tc_commit(&k_empty[kb]);
            }
            __syncwarp();
          }
          if (release) qt += nt;
          ok = __all_sync(0xffffffffu, ok);
          ++ku;
        }
      }
      if (elect_one()) {
        tc_commit(drain);
        mbar_drain(drain, 0);
      }
    }
    __syncwarp();
  } else {
    reg_alloc<kRegsSum>();
    // -------------------------------------------------------- sums per key
    const int s = (warp - 4) >> 3, half = ((warp - 4) >> 2) & 1;  // key tile, columns [64 half, 64 half + 64)
    const int row = (warp & 3) * 32 + lane;
    const uint32_t s_addr = tbase + (static_cast<uint32_t>((warp & 3) * 32) << 16) + 256 * s + 64 * half;
    const int lim = p.by_head ? p.T : (p.GT >= 128 ? p.GT : p.n * p.GT);
    const int step = p.nb * p.rb;
    int nu = 0, qt = 0, it = 0, joins = 0;
    bool ok = true, met = false;
    const int pair_bar = 1 + 4 * s + (warp & 3);  // named barrier of the two warps of a row
    // The two warps of a row meet once per pair of key tiles, and once more when
    // they leave.  Each says there whether it has given up or seen that another
    // did, and the barrier gives both the same answer: they part at one meeting,
    // and none waits there for a partner that is gone.  (The abort flag itself
    // may change between two looks at it.)
    auto meet = [&](bool gone) -> bool { return named_barrier_or(pair_bar, 64, gone || *abort_flag); };
    for (;;) {
      const int slot = nu % kRing;
      ok = mbar_sleep_warp(&u_full[slot], (nu / kRing) & 1, abort_flag, p.status);
      if (!ok) break;
      Unit x;
      read_unit(x, ring + slot * kUnitInts);
      x.nt = uniform(x.nt);
      x.key0 = uniform(x.key0);
      x.len = uniform(x.len);
      x.r0 = uniform(x.r0);
      x.r_min = uniform(x.r_min);
      x.i = uniform(x.i);
      x.np = uniform(x.np);
      __syncwarp();
      if (lane == 0) mbar_arrive(&u_empty[slot]);
      __syncwarp();
      ++nu;
      if (x.nt < 0) break;
      for (int pp = 0; pp < x.np; ++pp) {
        const bool release = !p.resident || pp == x.np - 1;
        const int tile0 = x.key0 + 256 * pp + 128 * s, key = tile0 + row;
        const long long at = static_cast<long long>(x.bk * p.Hkv + x.hkv) * p.C + key;
        const float before = p.Z == 1 && !half && p.score_in && key < x.len ? p.score_in[at] : 0.f;
        float acc = 0.f, comp = 0.f;
        // rows r, r + step, .. below lim, from r_min again for every head
        int r = p.by_head || p.GT >= 128 ? x.r0 : x.i * p.GT;
        // first row whose token sees every key of this tile
        const int r_open = !p.causal ? INT_MIN : tile0 + 127 - (x.len - p.T);
#pragma unroll 1
        for (int f = 0; f < x.nt; ++f, ++it) {
          const int buf = it & 1, st = (qt + f) % kLse;
          const int cols = min(step, lim - r);
          const bool mask = (p.by_head ? r : 0) < r_open;
          const uint32_t lh = ((qt + f) / kLse) & 1, sh = (it >> 1) & 1;
          const bool lr = mbar_try_wait(&l_full[st], lh), sr = mbar_try_wait(&s_full[2 * s + buf], sh);
          ok = lr || mbar_sleep(&l_full[st], lh, abort_flag, p.status);
          const float* nl = sLse + kNl * st + 64 * half;
          // a query without lse adds nothing, whatever its logits (NaN too)
          const int2 gone = *reinterpret_cast<const int2*>(sLse + kNl * st + 128 + 2 * half);
          ok &= sr || mbar_sleep(&s_full[2 * s + buf], sh, abort_flag, p.status);
          __syncwarp();
          if (!(ok = __all_sync(0xffffffffu, ok))) break;
          tc_fence_after();
          const uint32_t src = s_addr + 128 * buf;
          float a[4] = {0.f, 0.f, 0.f, 0.f};
          // (the first columns are on their way while the marks are read)
          float va[32];
          tmem_ld32(src, va);
          const bool whole = __all_sync(0xffffffffu, !mask && cols == 128 && (gone.x | gone.y) == 0);
          tc_wait_ld();
          if (whole) {
            float vb[32];
            tmem_ld32(src + 32, vb);  // on its way meanwhile
            sum32(va, nl, p.scale_log2, a);
            tc_wait_ld();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&s_empty[2 * s + buf]);
            __syncwarp();
            sum32(vb, nl + 32, p.scale_log2, a);
            __syncwarp();
            if (lane == 0 && release) mbar_arrive(&l_empty[st]);
            __syncwarp();
          } else {
            const int chunks = (min(cols - 64 * half, 64) + 31) >> 5;
#pragma unroll 1
            for (int c = 0; c < chunks; ++c) {
              // last key that the query of column 64 half + 32 c + lane sees;
              // none where there is no query, or none that counts (its column
              // holds anything)
              const int col = 64 * half + 32 * c + lane;
              int last = -1;
              if (col < cols && nl[32 * c + lane] != -INFINITY) last = !mask ? INT_MAX : x.len - p.T + (p.by_head ? r + col : (r + col) % p.T);
              float v[32];
              tmem_ld32(src + 32 * c, v);
              tc_wait_ld();
#pragma unroll
              for (int i = 0; i < 32; ++i) {
                const float e = ex2_approx(fmaf(v[i], p.scale_log2, nl[32 * c + i]));
                if (key <= __shfl_sync(0xffffffffu, last, i)) a[i & 3] += e;
              }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
              mbar_arrive(&s_empty[2 * s + buf]);
              if (release) mbar_arrive(&l_empty[st]);
            }
            __syncwarp();
          }
          // compensated: the tile's sum joins the key's
          const float y = ((a[0] + a[1]) + (a[2] + a[3])) - comp;
          const float z = acc + y;
          comp = (z - acc) - y;
          acc = z;
          r += step;
          if (r >= lim) r = x.r_min;
        }
        if (!ok) break;
        if (release) qt += x.nt;
        // the halves join
        float* hs = half_sum + 256 * (joins & 1) + 128 * s;
        ++joins;
        if (half) hs[row] = acc;
        __syncwarp();
        if ((met = meet(false))) break;
        if (!half) acc += hs[row];
        if (!half && key < p.C) {
          if (p.Z > 1) {
            p.part[static_cast<long long>(x.z) * p.Bk * p.Hkv * p.C + at] = acc;
          } else {
            p.score_out[at] = key < x.len ? before + acc : 0.f;
          }
        }
      }
      if (!ok || met) break;
    }
    __syncwarp();
    if (!met) meet(true);
    // units of a line end at the keys: the slots of the pairs behind them
    if (!p.by_head && p.Z == 1) {
      const int tid = threadIdx.x - 128;
      const long long tail = static_cast<long long>(p.Bk) * p.Hkv * p.pairs;
      for (long long u = 2LL * blockIdx.x + (tid >> 8); u < tail; u += 2LL * gridDim.x) {
        const int bh = static_cast<int>(u / p.pairs), key = static_cast<int>(u - static_cast<long long>(bh) * p.pairs) * 256;
        if (key >= clamped_len(p, bh / p.Hkv) && key + (tid & 255) < p.C)
          p.score_out[static_cast<long long>(bh) * p.C + key + (tid & 255)] = 0.f;
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tbase, 512);
  }
}

// ------------------------------------------------------------------ few queries
// Queries per key set and KV head, at most.  32 caches of 4096, 8 KV heads, us a call,
// this kernel against weight_kernel: d = 64: 12 rows 20 / 37, 28 rows 29 / 37;
// d = 128: 12 rows 30 / 42, 20 rows 50 / 42.
template <int D>
constexpr int kStreamRows = D == 64 ? 32 : 16;
constexpr int kStreamThreads = 256;

template <bool FP16>
__device__ __forceinline__ void mma_16x8x16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                            uint32_t b0, uint32_t b1) {
  if constexpr (FP16) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  } else {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  }
}

// NT: groups of eight queries.  A warp takes 16 keys a step; lane 4 g + t holds
// pieces t, t + 4, .. (16 bytes each) of keys g and g + 8, and the same
// pieces of query g of every group.
template <int D, bool FP16, int NT>
__global__ void __launch_bounds__(kStreamThreads, NT == 4 ? 1 : (D == 64 ? 3 : 2))
    stream_kernel(const uint4* q, const uint4* k, const Params p, int chunk, int chunks) {
  constexpr int kP = D / 32;  // pieces per lane and row
  constexpr int kWarps = kStreamThreads / 32;
  grid_dep_launch();
  grid_dep_wait();
  const int bh = blockIdx.x / chunks, c0 = (blockIdx.x - bh * chunks) * chunk;
  const int bk = bh / p.Hkv, hkv = bh - bk * p.Hkv;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
  if (blockIdx.x == 0) {
    bool bad = false;
    if (p.key_len)
      for (int i = threadIdx.x; i < p.Bk; i += kStreamThreads) {
        const int n = p.key_len[i];
        bad |= n < 0 || n > p.C;
      }
    bad = __syncthreads_or(bad);
    if (threadIdx.x == 0) *p.status = bad ? kStatusLength : 0;
  }
  const int len = clamped_len(p, bk);
  const int end = min(c0 + chunk, p.C);
  const long long base = static_cast<long long>(bh) * p.C;
  const uint4* kb = k + base * (D / 8);
  // K of the first step before anything else.  Each key is read once and evicted
  // first (48 caches of one token 22.7 us, 24.4 with plain loads; 64 of 4096 at
  // d = 128 51 and 55); queries and lse, which all warps read, by plain loads.
  uint4 cur[2][kP];
  float sin = 0.f;
  auto fetch = [&](int key0, uint4 (&f)[2][kP], float& si) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int key = key0 + g + 8 * h;
#pragma unroll
      for (int i = 0; i < kP; ++i)
        f[h][i] = key < len ? __ldcs(kb + static_cast<long long>(key) * (D / 8) + t + 4 * i) : make_uint4(0, 0, 0, 0);
    }
    // lanes t = 0 and 1 finish keys g and g + 8
    const int key = key0 + g + 8 * t;
    si = p.score_in && t < 2 && key < len ? p.score_in[base + key] : 0.f;
  };
  int key0 = c0 + 16 * warp;
  if (key0 < min(end, len)) fetch(key0, cur, sin);
  uint4 qf[NT][kP];
  float nl[NT][2];
  int lim[NT][2];
  const int rows = p.n * p.GT;
  // (rows past the last one read that again: loads under no condition are all
  // under way at once; 28 rows a key 31.6 -> 28.9 us)
  auto row_at = [&](int r) -> long long {
    r = min(r, rows - 1);
    const int i = r / p.GT;
    return (static_cast<long long>(bk * p.n + i) * p.Hkv + hkv) * p.GT + (r - i * p.GT);
  };
  float lq[NT];
#pragma unroll
  for (int j = 0; j < NT; ++j) {
    const long long at = row_at(8 * j + g);
#pragma unroll
    for (int m = 0; m < kP; ++m) qf[j][m] = q[at * (D / 8) + t + 4 * m];
    lq[j] = p.lse[at];
#pragma unroll
    for (int e = 0; e < 2; ++e) nl[j][e] = p.lse[row_at(8 * j + 2 * t + e)];
  }
#pragma unroll
  for (int j = 0; j < NT; ++j) {
    // a query without lse adds nothing, whatever it holds (NaN too)
    if (8 * j + g >= rows || lq[j] == -INFINITY)
#pragma unroll
      for (int m = 0; m < kP; ++m) qf[j][m] = make_uint4(0, 0, 0, 0);
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      // a query that saw nothing (lse -inf) adds nothing, to keys of NaN or
      // infinities neither (0 of the query times such a key is NaN)
      const int r = 8 * j + 2 * t + e;
      const bool none = r >= rows || nl[j][e] == -INFINITY;
      nl[j][e] = none ? -INFINITY : -nl[j][e] * kLog2e;
      lim[j][e] = none ? -1 : (p.causal ? len - p.T + r % p.T : INT_MAX);
    }
  }
  for (; key0 < min(end, len); key0 += 16 * kWarps) {
    uint4 nxt[2][kP];
    float sn = 0.f;
    const int kn = key0 + 16 * kWarps;
    if (kn < min(end, len)) fetch(kn, nxt, sn);
    float w0 = 0.f, w1 = 0.f;  // keys g and g + 8
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      float c[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int m = 0; m < kP; ++m) {
        mma_16x8x16<FP16>(c, cur[0][m].x, cur[1][m].x, cur[0][m].y, cur[1][m].y, qf[j][m].x, qf[j][m].y);
        mma_16x8x16<FP16>(c, cur[0][m].z, cur[1][m].z, cur[0][m].w, cur[1][m].w, qf[j][m].z, qf[j][m].w);
      }
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const float e0 = ex2_approx(fmaf(c[e], p.scale_log2, nl[j][e]));
        const float e1 = ex2_approx(fmaf(c[2 + e], p.scale_log2, nl[j][e]));
        w0 += key0 + g <= lim[j][e] ? e0 : 0.f;
        w1 += key0 + g + 8 <= lim[j][e] ? e1 : 0.f;
      }
    }
#pragma unroll
    for (int o = 1; o < 4; o <<= 1) {
      w0 += __shfl_xor_sync(0xffffffffu, w0, o);
      w1 += __shfl_xor_sync(0xffffffffu, w1, o);
    }
    const int key = key0 + g + 8 * t;
    if (t < 2 && key < end) p.score_out[base + key] = key < len ? sin + (t ? w1 : w0) : 0.f;
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int i = 0; i < kP; ++i) cur[h][i] = nxt[h][i];
    sin = sn;
  }
  // slots of the chunk behind the last step
  const int done = max(c0, len > c0 ? c0 + (min(end, len) - c0 + 15) / 16 * 16 : c0);
  for (int key = done + threadIdx.x; key < end; key += kStreamThreads) p.score_out[base + key] = 0.f;
}

// score_out = score_in + the parts of a split unit, in order.
__global__ void __launch_bounds__(256) weight_sum_kernel(const Params p) {
  grid_dep_launch();
  grid_dep_wait();
  const long long n = static_cast<long long>(p.Bk) * p.Hkv * p.C;
  const long long i = blockIdx.x * 256LL + threadIdx.x;
  if (i >= n) return;
  const int key = static_cast<int>(i % p.C), bk = static_cast<int>(i / p.C / p.Hkv);
  float a = 0.f;
  if (key < clamped_len(p, bk)) {
    float w = 0.f;
    for (int z = 0; z < p.Z; ++z) w += p.part[z * n + i];
    a = (p.score_in ? p.score_in[i] : 0.f) + w;
  }
  p.score_out[i] = a;
}

bool make_plan(Params& p, int B, int G, int Hkv, int T, int Bk, int C) {
  p.B = B;
  p.G = G;
  p.Hkv = Hkv;
  p.T = T;
  p.Bk = Bk;
  p.n = B / Bk;
  p.C = C;
  p.GT = G * T;
  p.by_head = T >= 128;
  long long tiles;
  if (p.by_head) {
    p.nb = 1;
    p.rb = 128;
    p.tiles = (T + 127) / 128;
    tiles = static_cast<long long>(p.n) * G * p.tiles;
  } else if (p.GT >= 128) {
    p.nb = 1;
    p.rb = 128;
    tiles = static_cast<long long>(p.n) * ((p.GT + 127) / 128);
  } else {
    p.nb = 128 / p.GT < p.n ? 128 / p.GT : p.n;
    p.rb = p.GT;
    tiles = (p.n + p.nb - 1) / p.nb;
  }
  if (tiles > INT_MAX) return false;
  if (!p.by_head) p.tiles = static_cast<int>(tiles);
  p.all = static_cast<int>(tiles);
  p.N = (p.nb * p.rb + 15) & ~15;
  p.pairs = (C + 255) / 256;
  const long long units = static_cast<long long>(Bk) * Hkv * p.pairs;
  // Parts, 16 at most: the split whose last SM is done first, counted in query
  // tiles, where a unit's start costs one (a prefill's two) and the sum of the
  // parts two; more parts have to gain 1% of the whole, since they are memory.
  // Units of one size come in rounds; those of a prefill (T > C / 2: from all
  // query tiles down to none) even out but for about the longest one's length.
  // (Us a call, against two units per SM of four query tiles or more: 300
  // queries of 300 keys, 8 heads of 2 KV heads, 15.5 -> 12.1; 64 of 1000, 16 of
  // 2, 16.8 -> 12.4; 150 of 4000, 64 of 8, 33.2 -> 30.5; 4096 of 4096, 16 of 8,
  // 61.0 -> 59.5.)
  const bool even = !(p.by_head && 2LL * T > C);
  double least = 0, gain = 0;
  p.Z = 1;
  for (int z = 1; z <= 16 && z <= tiles; ++z) {
    const double rounds = static_cast<double>(units) * z / kPlanSms, each = static_cast<double>(tiles) / z;
    const double cost =
        (even ? std::ceil(rounds) * (std::ceil(each) + 1) : rounds * (0.5 * each + 2) + each) + (z > 1 ? 2 : 0);
    if (z == 1) gain = 0.01 * cost;
    if (z == 1 || cost < least - gain) least = cost, p.Z = z;
  }
  p.units = units * p.Z;
  return units <= INT_MAX && static_cast<long long>(Bk) * Hkv * tiles <= INT_MAX;
}

template <int D, bool FP16>
cudaError_t run(const Params& p, const CUtensorMap& mq, const CUtensorMap& mk, int grid, cudaStream_t st) {
  cudaError_t e = cudaFuncSetAttribute(weight_kernel<D, FP16>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       Cfg<D>::kSmem);
  if (e != cudaSuccess) return e;
  e = launch_chained(weight_kernel<D, FP16>, dim3(grid), dim3(kThreads), Cfg<D>::kSmem, st, mq, mk, p);
  if (e != cudaSuccess || p.Z == 1) return e;
  const long long n = static_cast<long long>(p.Bk) * p.Hkv * p.C;
  return launch_chained(weight_sum_kernel, dim3(static_cast<unsigned>((n + 255) / 256)), dim3(256), 0, st, p);
}

size_t align256(size_t v) { return (v + 255) & ~static_cast<size_t>(255); }

bool streams(const Params& p, int d) {
  return static_cast<long long>(p.n) * p.GT <= (d == 64 ? kStreamRows<64> : kStreamRows<128>);
}

template <int D, bool FP16>
cudaError_t run_stream(const WeightLaunch& a, const Params& p, cudaStream_t st) {
  // keys per CTA: eight steps a warp, fewer while the grid is under two
  // CTAs per SM twice over
  const long long heads = static_cast<long long>(p.Bk) * p.Hkv;
  int chunk = 1024;
  while (chunk > 128 && heads * ((p.C + chunk - 1) / chunk) < 4 * kPlanSms) chunk /= 2;
  const int chunks = (p.C + chunk - 1) / chunk;
  const dim3 grid(static_cast<unsigned>(heads * chunks));
  const uint4* q = static_cast<const uint4*>(a.q);
  const uint4* k = static_cast<const uint4*>(a.k);
  const int rows = p.n * p.GT;
  if (rows <= 8) return launch_chained(stream_kernel<D, FP16, 1>, grid, dim3(kStreamThreads), 0, st, q, k, p, chunk, chunks);
  if (rows <= 16) return launch_chained(stream_kernel<D, FP16, 2>, grid, dim3(kStreamThreads), 0, st, q, k, p, chunk, chunks);
  if constexpr (kStreamRows<D> > 16)
    return launch_chained(stream_kernel<D, FP16, 4>, grid, dim3(kStreamThreads), 0, st, q, k, p, chunk, chunks);
  return cudaErrorInvalidValue;
}

}  // namespace

size_t weight_workspace_bytes(int B, int G, int Hkv, int T, int d, int Bk, int C) {
  Params p = {};
  if (!make_plan(p, B, G, Hkv, T, Bk, C)) return 0;
  if (streams(p, d)) return 256;
  return 256 + align256(p.Z > 1 ? static_cast<size_t>(p.Z) * Bk * Hkv * C * 4 : 0);
}

cudaError_t launch_weight(const WeightLaunch& a, cudaStream_t st) {
  Params p = {};
  if (!make_plan(p, a.B, a.G, a.Hkv, a.T, a.Bk, a.C)) return cudaErrorInvalidValue;
  p.lse = a.lse;
  p.key_len = a.key_len;
  p.score_in = a.score_in;
  p.score_out = a.score_out;
  p.causal = a.causal;
  p.scale_log2 = kLog2e / (a.d == 128 ? 11.313708498984761f : 8.0f);
  p.status = reinterpret_cast<int*>(a.ws);
  p.part = reinterpret_cast<float*>(a.ws + 256);
  if (streams(p, a.d)) {
    if (a.d == 128) return a.fp16 ? run_stream<128, true>(a, p, st) : run_stream<128, false>(a, p, st);
    return a.fp16 ? run_stream<64, true>(a, p, st) : run_stream<64, false>(a, p, st);
  }
  p.stall = take_serve_stall_request();
  p.resident = !p.by_head && p.Z == 1 && p.all <= (a.d == 128 ? Cfg<128>::kQStages : Cfg<64>::kQStages);
  CUtensorMap mq, mk;
  const uint64_t u = 1;
  const uint64_t by_kv[4] = {u * a.d, u * p.GT, u * a.Hkv, u * a.B};
  const uint64_t by_head[4] = {u * a.d, u * a.T, u * a.Hkv * a.G, u * a.B};
  const uint32_t bq[4] = {64, static_cast<uint32_t>(p.rb), 1, static_cast<uint32_t>(p.nb)};
  const uint64_t dk[3] = {u * a.d, u * a.C, u * a.Bk * a.Hkv};
  const uint32_t bk[3] = {64, 64, 1};
  if (encode_tensor_map_16(&mq, a.q, a.fp16, 4, p.by_head ? by_head : by_kv, bq) != CUDA_SUCCESS ||
      encode_tensor_map_16(&mk, a.k, a.fp16, 3, dk, bk) != CUDA_SUCCESS)
    return cudaErrorInvalidValue;
  int grid = device_sm_count();
  if (p.units < grid) grid = static_cast<int>(p.units);
  if (a.d == 128) return a.fp16 ? run<128, true>(p, mq, mk, grid, st) : run<128, false>(p, mq, mk, grid, st);
  return a.fp16 ? run<64, true>(p, mq, mk, grid, st) : run<64, false>(p, mq, mk, grid, st);
}

}  // namespace psa
