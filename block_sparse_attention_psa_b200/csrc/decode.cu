// decode.cu -- attention of a batch's new tokens over a prefix that groups
// of sequences share and over each sequence's own cache, in one softmax:
//   out_t = sum_j e^{s_tj} v_j / sum_j e^{s_tj},  s = q.k / sqrt(d)
// over the visible prefix keys and cache slots.  The largest exponent, the
// sum and the weighted values of disjoint key sets combine exactly, so the
// keys are cut wherever the machine wants them cut (decode_kernel) and the
// parts joined afterwards (merge_kernel).
//
// Work is bound by reading K and V once at few rows per key (4 d rows
// operations against 4 d bytes), by the exponentials and the tensor cores at
// many.
//  * Rows.  All rows that read the same K and V share one pass over them: the
//    G query heads of a KV head, the T new tokens and, for the prefix, the
//    sequences of the group.  A row tile is up to 128 of them, the M of the
//    products S = Q K^T (Q, K in shared memory) and O += P V (P in TMEM,
//    written over S; V MN-major in shared memory).  An unfilled tile costs
//    tensor time, which few rows leave idle.
//  * Streams.  A CTA runs two softmax streams, each with its own S/P and O in
//    TMEM (512 columns in all).  With two row tiles or more each takes one of
//    a pair, so that K and V are read once for 256 rows; with one row tile
//    they take alternate key tiles and give two parts.  Items go to the
//    streams in turn, one thread issues every product: PV of the item two
//    back, then S of this one, so that one stream's softmax covers the other's
//    products.  A stream is a chain S -> softmax -> PV -> S (P lies over S and
//    TMEM has no room for a second); the PV product of a tile's first 64 keys
//    starts when their half of P is there.
//  * Split.  The key tiles of all units (KV head x row-tile pair) are laid
//    out in two lines, the prefixes' and the caches', a tile for a pair twice
//    as long, and each line is cut into equal runs, one per SM, whatever the
//    lengths, which live on the device.  (One line for both left the SMs that
//    got the caches, short units with a load and a part each, twice as long at
//    work as the others.)  A unit's run in one CTA is a piece; its parts
//    (running maximum, sum and unnormalised O, fp32) go to the workspace.
//  * Stabiliser.  A row's reference exponent only moves when a tile's maximum
//    passes it by 2^8, so O is rarely rescaled, and terms stay below 2^8.
//  * Rounding.  P is rounded to the inputs' type for the tensor core (half a
//    step, 2^-9 of the term in bf16), sums, O and the parts stay in fp32, the
//    output is rounded once.
//  * V rows past a sequence's length are cleared in shared memory before the
//    product (0 x NaN would reach the sum); K rows past it only touch columns
//    that are masked.
// Measured on one B200 (device time, a call in a stream of calls; floors from
// 6.54 TB/s and 1658 TFLOP/s): 64 ragged caches of up to 4096, 8 KV heads of 4
// query heads, d = 128: 93 us, 5.9 TB/s (floor 85). 16 samples of a 32K prompt:
// 42 us (23): 22 us of streaming at the DRAM's rate, the rest is the schedule
// (1.7), the first load (3), the last tile's chain (5), the imbalance of the
// SMs (4) and the join (5). 64 sequences of 64 heads over a 128K prefix: 299 to
// 311 us replayed, 339 to 360 as called in a long run, 770 to 920 TFLOP/s
// (166): a pair of items takes ~3280 cycles, set by
// one stream's chain S -> softmax (2030: 128 exponentials of a thread alone are
// 1024) -> PV -> S, the tensor core working 2048 of them, under the power cap
// (1.4 GHz). Tried and slower there: the softmax of a row over two
// warpgroups, a share of the exponentials on the FMA pipe, terms formed before
// the new maximum is known.
// Every wait is bounded.
#include "internal.h"
#include "sm100.cuh"

namespace psa {
namespace {

constexpr int kThreads = 384;      // WG0: Q/K loads, MMA issue, V loads; WG1, WG2: softmax streams
constexpr int kRegsProducer = 72;  // 128 x 72 + 256 x 216 = 384 x 168
constexpr int kRegsSoftmax = 216;
constexpr int kMaxCtas = 256;      // upper bound of the grid the workspace is sized for
constexpr int kRing = 4;           // pieces in flight between the scheduler and its readers
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kRescale = 8.0f;   // log2 units the reference may lag behind the maximum

template <int D>
struct Cfg {
  static constexpr int kChunks = D / 64;        // 128-byte column chunks
  static constexpr int kTile = 128 * D * 2;     // 128 rows
  static constexpr int kStages = D == 128 ? 2 : 4;
  static constexpr int kOffQ = 0;               // two row tiles
  static constexpr int kOffK = 2 * kTile;
  static constexpr int kOffV = kOffK + kStages * kTile;
  static constexpr int kOffMisc = kOffV + kStages * kTile;
  static constexpr int kSmem = kOffMisc + 1024 + 1024;  // + alignment slack
  static_assert(kSmem <= 232448, "shared memory of one CTA");
};

struct Params {
  const int* prefix_len;
  const int* cache_len;
  int B, G, Hkv, T, Bp, n, P, C;
  int GT;              // rows of one sequence and KV head
  int nseg;            // prefixes (if any), then caches (if any)
  int npre;            // prefixes among them
  int pre_nb, pre_rb;  // prefix row tile: sequences x rows of each
  int pre_rt, pre_up;  // row tiles and units (pairs) per (prefix, KV head)
  int own_rb, own_rt, own_up;
  float scale_log2;
  long long pre_slots; // slots of the prefix region: the caches' parts start behind it
  long long own_unit0; // place of the caches' units in unit_ctas
  int2* unit_ctas;     // per unit: the runs that have its first and its last key tile
  float* part_o;       // parts: rows x d
  float2* part_ml;     // reference (log2 units), sum
  int* status;
  int stall;           // test hook: CTA 0 withholds its first S hand-off
};

// A piece: part of one unit's key tiles, as the scheduler publishes it.
struct Piece {
  int prefix;     // 1: a prefix, 0: a cache
  int outer, hkv; // prefix or sequence, KV head
  int tile0;      // first row tile
  int pair;       // 1: both streams read every key tile, for two row tiles
  int j0, nt;     // key tiles
  int len;        // valid keys of the segment
  int slot;       // unit + run within the region: the place of its parts
  int tiles, items, qpos;  // running counts of this CTA at the piece's start
};
constexpr int kPieceInts = sizeof(Piece) / 4;

__device__ __forceinline__ int seg_len(const Params& p, int s) {
  if (s < p.npre) return min(max(p.prefix_len ? p.prefix_len[s] : p.P, 0), p.P);
  return min(max(p.cache_len ? p.cache_len[s - p.npre] : p.C, 0), p.C);
}
__device__ __forceinline__ bool seg_bad(const Params& p, int s) {
  if (s < p.npre) return p.prefix_len && (p.prefix_len[s] < 0 || p.prefix_len[s] > p.P);
  return p.cache_len && (p.cache_len[s - p.npre] < 0 || p.cache_len[s - p.npre] > p.C);
}
// Length of a segment on the line: its row tiles times its key tiles (the
// last unit of a KV head has one row tile when their number is odd), and
// `pad` for each unit.
__device__ __forceinline__ int seg_work(const Params& p, int s, int len, int pad) {
  const bool pre = s < p.npre;
  return len == 0 ? 0 : p.Hkv * ((len + 127) / 128 * (pre ? p.pre_rt : p.own_rt) + pad * (pre ? p.pre_up : p.own_up));
}
// Key tiles of a unit (whose tiles start at `o` on the line, w = 1 or 2 per
// tile) before x: a cut inside a tile leaves it to the run it starts in.
__device__ __forceinline__ int tiles_before(int x, int o, int w) {
  return x <= o ? 0 : (w == 1 ? x - o : (x - o + 1) >> 1);
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

// Terms of 64 keys of one row, 2^(s * scale + neg), packed to the input type,
// with their sum.
template <bool FP16>
__device__ __forceinline__ void exps(const float* v, float scale, float neg, float (&l)[4], uint32_t (&pk)[32]) {
#pragma unroll
  for (int i = 0; i < 32; ++i) {
    float x0, x1;
    ffma2(x0, x1, v[2 * i], v[2 * i + 1], scale, scale, neg, neg);
    x0 = ex2_approx(x0);
    x1 = ex2_approx(x1);
    fadd2(l[2 * (i & 1)], l[2 * (i & 1) + 1], l[2 * (i & 1)], l[2 * (i & 1) + 1], x0, x1);
    pk[i] = pack_16x2<FP16>(x0, x1);
  }
}

template <int D, bool FP16>
__global__ void __launch_bounds__(kThreads, 1)
    decode_kernel(const __grid_constant__ CUtensorMap tmQp, const __grid_constant__ CUtensorMap tmQc,
                  const __grid_constant__ CUtensorMap tmKp, const __grid_constant__ CUtensorMap tmVp,
                  const __grid_constant__ CUtensorMap tmKc, const __grid_constant__ CUtensorMap tmVc, const Params p) {
  using C = Cfg<D>;
  constexpr int kSt = C::kStages;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sQ = smem + C::kOffQ;
  uint8_t* sK = smem + C::kOffK;
  uint8_t* sV = smem + C::kOffV;
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::kOffMisc);
  uint64_t* q_full = bars + 0;    // [2] a row tile landed              (TMA)
  uint64_t* q_empty = bars + 2;   // [2] its last S product done        (commit)
  uint64_t* k_full = bars + 4;    // [kSt]
  uint64_t* k_empty = bars + 8;   // [kSt] last S product of the tile   (commit)
  uint64_t* v_full = bars + 12;   // [kSt]
  uint64_t* v_empty = bars + 16;  // [kSt] last PV product of the tile  (commit)
  uint64_t* s_full = bars + 20;   // [2] S of the stream ready          (commit)
  uint64_t* p_full = bars + 22;   // [2][2] half of P written over it   (4 warps)
  uint64_t* o_full = bars + 26;   // [2] last PV of the piece done      (commit)
  uint64_t* pc_full = bars + 28;  // [kRing] a piece published
  uint64_t* pc_empty = bars + 32; // [kRing] read by V loads, MMA issue, 8 softmax warps
  uint64_t* drain = bars + 36;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::kOffMisc + 320);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  volatile int* ring = reinterpret_cast<volatile int*>(smem + C::kOffMisc + 512); // [kRing][kPieceInts]

  const int warp = uniform(threadIdx.x / 32), lane = threadIdx.x % 32;
  if (threadIdx.x == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&q_full[i], 1);
      mbar_init(&q_empty[i], 1);
      mbar_init(&s_full[i], 1);
      mbar_init(&p_full[2 * i], 4);
      mbar_init(&p_full[2 * i + 1], 4);
      mbar_init(&o_full[i], 1);
    }
    for (int i = 0; i < kSt; ++i) {
      mbar_init(&k_full[i], 1);
      mbar_init(&k_empty[i], 1);
      mbar_init(&v_full[i], 1);
      mbar_init(&v_empty[i], 1);
    }
    for (int i = 0; i < kRing; ++i) {
      mbar_init(&pc_full[i], 1);
      mbar_init(&pc_empty[i], 10);
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
    tma_prefetch_desc(&tmKp);
    tma_prefetch_desc(&tmVp);
    tma_prefetch_desc(&tmKc);
    tma_prefetch_desc(&tmVc);
    tma_prefetch_desc(&tmQp);
    tma_prefetch_desc(&tmQc);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tbase = *tmem_slot;
  grid_dep_launch();
  grid_dep_wait();

  if (warp < 4) {
    reg_dealloc<kRegsProducer>();
    if (warp == 0) {
      // ---------------------------------------------------- scheduler, Q and K loads
      int tiles = 0, items = 0, qpos = 0, np = 0, kl = 0, ql = 0;
      bool ok = true;
      for (int line = 0; line < 2; ++line) {
        const int sa = line ? p.npre : 0, sb = line ? p.nseg : p.npre;
        // the line's length, and this CTA's run of it: no empty runs between
        // others, since every CTA between a unit's first and its last one
        // writes that unit's parts
        int tile_sum = 0, unit_sum = 0;
        const int front = sa + lane < sb ? seg_len(p, sa + lane) : 0;  // of its first 32 segments
        for (int s = sa + lane; s < sb; s += 32) {
          const int len = s == sa + lane ? front : seg_len(p, s);
          tile_sum += seg_work(p, s, len, 0);
          unit_sum += len > 0 ? p.Hkv * (line ? p.own_up : p.pre_up) : 0;
        }
        tile_sum = static_cast<int>(__reduce_add_sync(0xffffffffu, static_cast<uint32_t>(tile_sum)));
        unit_sum = static_cast<int>(__reduce_add_sync(0xffffffffu, static_cast<uint32_t>(unit_sum)));
        // A unit's start and end cost about as much as a tile, and count as one
        // on the line (a batch of ragged caches without it: the CTAs with two
        // units were done after 93 us, those with eleven after 103); not where
        // a run is only a few tiles, which the pads would make uneven.
        const int pad = tile_sum >= 4 * static_cast<int>(gridDim.x) ? 1 : 0;
        const int total = tile_sum + pad * unit_sum;
        // the second line is dealt from the last CTA backwards, so that not
        // the same ones get the longer runs of both
        const int g = min(total, static_cast<int>(gridDim.x));
        const int cta = line ? static_cast<int>(gridDim.x) - 1 - static_cast<int>(blockIdx.x) : static_cast<int>(blockIdx.x);
        if (cta >= g) continue;
        const int q = total / g, more = total - q * g;
        int x = cta * q + min(cta, more);
        const int xe = x + q + (cta < more ? 1 : 0);
        // the segment in which it starts, and that segment's place
        int lens0 = sa, lens = 0, off = 0, s = sa;  // lane l holds the length of segment lens0 + l
        for (;; lens0 += 32) {
          lens = lens0 == sa ? front : (lens0 + lane < sb ? seg_len(p, lens0 + lane) : 0);
          const int w = lens0 + lane < sb ? seg_work(p, lens0 + lane, lens, pad) : 0;
          int inc = w;
#pragma unroll
          for (int o = 1; o < 32; o <<= 1) {
            const int u = __shfl_up_sync(0xffffffffu, inc, o);
            if (lane >= o) inc += u;
          }
          const uint32_t past = __ballot_sync(0xffffffffu, off + inc > x);
          if (past) {
            const int owner = __ffs(past) - 1;
            s = lens0 + owner;
            off += __shfl_sync(0xffffffffu, inc - w, owner);
            break;
          }
          off += __shfl_sync(0xffffffffu, inc, 31);
        }
        while (ok && x < xe) {
          if (s - lens0 >= 32) {
            lens0 = s;
            lens = s + lane < sb ? seg_len(p, s + lane) : 0;
          }
          const int len = __shfl_sync(0xffffffffu, lens, s - lens0);
          const int nkt = (len + 127) / 128;
          const bool pre = s < p.npre;
          const int up = pre ? p.pre_up : p.own_up, rt = pre ? p.pre_rt : p.own_rt;
          const int per_head = nkt > 0 ? nkt * rt + pad * up : 0, here = per_head * p.Hkv;
          if (x >= off + here) {
            off += here;
            ++s;
            continue;
          }
          Piece c;
          c.prefix = pre;
          c.outer = pre ? s : s - p.npre;
          c.hkv = (x - off) / per_head;
          const int head0 = off + c.hkv * per_head;
          const int u = (x - head0) / (pad + 2 * nkt);  // every unit before the last is a pair
          const int lu = c.hkv * up + u;
          c.tile0 = 2 * u;
          c.pair = c.tile0 + 1 < rt;
          const int o0 = head0 + u * (pad + 2 * nkt) + pad, o1 = o0 + nkt * (1 + c.pair);
          c.j0 = tiles_before(x, o0, 1 + c.pair);
          c.nt = tiles_before(min(o1, xe), o0, 1 + c.pair) - c.j0;
          x = min(o1, xe);
          c.len = len;
          const int unit = c.outer * p.Hkv * up + lu;
          c.slot = unit + cta;
          if (c.nt == 0) {
            // the rest of a tile that the run before took, or a unit's start
            // alone: parts without terms
            const int rows = 2 * (pre ? p.pre_nb * p.pre_rb : p.own_rb);
            float2* ml = p.part_ml + (pre ? 0 : p.pre_slots) + static_cast<long long>(c.slot) * rows;
            for (int i = lane; i < rows; i += 32) ml[i] = make_float2(-INFINITY, 0.f);
            continue;
          }
          if (lane == 0) {
            int2* uc = p.unit_ctas + (pre ? 0 : p.own_unit0) + unit;
            if (c.j0 == 0) uc->x = cta;
            if (c.j0 + c.nt == nkt) uc->y = cta;
          }
          c.tiles = tiles;
          c.items = items;
          c.qpos = qpos;
          if (lane == 0) {
            const int slot = np % kRing;
            if (np >= kRing) ok = mbar_sleep(&pc_empty[slot], ((np / kRing) - 1) & 1, abort_flag, p.status);
            if (ok) {
              const int* w = reinterpret_cast<const int*>(&c);
              for (int i = 0; i < kPieceInts; ++i) ring[slot * kPieceInts + i] = w[i];
              mbar_arrive(&pc_full[slot]);
            }
            // Q
            const CUtensorMap* mq = c.prefix ? &tmQp : &tmQc;
            for (int i = 0; i <= c.pair && ok; ++i) {
              const int qs = (qpos + i) & 1, n = (qpos + i) >> 1;
              ok = mbar_sleep(&q_empty[qs], (n & 1) ^ 1, abort_flag, p.status);
              if (!ok) break;
              const int tile = c.tile0 + i;
              int r = 0, b;
              uint32_t rows;
              if (c.prefix) {
                if (p.GT >= 128) {
                  const int per = (p.GT + 127) / 128;
                  b = c.outer * p.n + tile / per;
                  r = tile % per * 128;
                } else {
                  b = c.outer * p.n + tile * p.pre_nb;
                }
                rows = static_cast<uint32_t>(p.pre_nb * p.pre_rb);
              } else {
                b = c.outer;
                r = tile * 128;
                rows = 128;
              }
              mbar_arrive_expect_tx(&q_full[qs], rows * 128 * C::kChunks);
#pragma unroll
              for (int ch = 0; ch < C::kChunks; ++ch)
                tma_load_4d(mq, sQ + qs * C::kTile + ch * 16384, &q_full[qs], 64 * ch, r, c.hkv, b);
              ql = qpos + i + 1;
            }
            // K
            const CUtensorMap* mk = c.prefix ? &tmKp : &tmKc;
            for (int j = 0; j < c.nt && ok; ++j) {
              const int st = (tiles + j) % kSt, n = (tiles + j) / kSt;
              ok = mbar_sleep(&k_empty[st], (n & 1) ^ 1, abort_flag, p.status);
              if (!ok) break;
              const int y = 128 * (c.j0 + j);
              const int halves = c.len - y > 64 ? 2 : 1;
              mbar_arrive_expect_tx(&k_full[st], halves * 64 * 128 * C::kChunks);
              for (int h = 0; h < halves; ++h)
#pragma unroll
                for (int ch = 0; ch < C::kChunks; ++ch)
                  tma_load_3d(mk, sK + st * C::kTile + ch * 16384 + h * 8192, &k_full[st], 64 * ch, y + 64 * h,
                              c.outer * p.Hkv + c.hkv);
              kl = tiles + j + 1;
            }
          }
          ok = __shfl_sync(0xffffffffu, ok, 0);
          tiles += c.nt;
          items += c.pair ? 2 * c.nt : c.nt;
          qpos += 1 + c.pair;
          ++np;
        }
      }
      if (lane == 0) {
        // the end mark: a piece without tiles
        const int slot = np % kRing;
        if (ok && np >= kRing) ok = mbar_sleep(&pc_empty[slot], ((np / kRing) - 1) & 1, abort_flag, p.status);
        if (ok) {
          for (int i = 0; i < kPieceInts; ++i) ring[slot * kPieceInts + i] = 0;
          mbar_arrive(&pc_full[slot]);
        }
        // no bulk copy may still be writing shared memory when the CTA leaves
        for (int t = max(0, kl - kSt); t < kl; ++t) mbar_drain(&k_full[t % kSt], (t / kSt) & 1);
        for (int t = max(0, ql - 2); t < ql; ++t) mbar_drain(&q_full[t & 1], (t >> 1) & 1);
      }
      __syncwarp();
    } else if (warp == 3) {
      if (blockIdx.x == 0) {
        // one writer of the status word at the start: the lengths
        bool bad = false;
        for (int s = lane; s < p.nseg; s += 32) bad |= seg_bad(p, s);
        bad = __any_sync(0xffffffffu, bad);
        if (lane == 0) *p.status = bad ? kStatusLength : 0;
      }
    } else if (warp == 2 && lane == 0) {
      // ---------------------------------------------------- V loads
      int np = 0, vl = 0;
      bool ok = true;
      while (ok) {
        const int slot = np % kRing;
        if (!(ok = mbar_sleep(&pc_full[slot], (np / kRing) & 1, abort_flag, p.status))) break;
        Piece c;
        int* w = reinterpret_cast<int*>(&c);
        for (int i = 0; i < kPieceInts; ++i) w[i] = ring[slot * kPieceInts + i];
        mbar_arrive(&pc_empty[slot]);
        ++np;
        if (c.nt == 0) break;
        const CUtensorMap* mv = c.prefix ? &tmVp : &tmVc;
        for (int j = 0; j < c.nt; ++j) {
          const int st = (c.tiles + j) % kSt, n = (c.tiles + j) / kSt;
          if (!(ok = mbar_sleep(&v_empty[st], (n & 1) ^ 1, abort_flag, p.status))) break;
          const int y = 128 * (c.j0 + j);
          const int halves = c.len - y > 64 ? 2 : 1;
          mbar_arrive_expect_tx(&v_full[st], halves * 64 * 128 * C::kChunks);
          for (int h = 0; h < halves; ++h)
#pragma unroll
            for (int ch = 0; ch < C::kChunks; ++ch)
              tma_load_3d(mv, sV + st * C::kTile + ch * 16384 + h * 8192, &v_full[st], 64 * ch, y + 64 * h,
                          c.outer * p.Hkv + c.hkv);
          vl = c.tiles + j + 1;
        }
      }
      for (int t = max(0, vl - kSt); t < vl; ++t) mbar_drain(&v_full[t % kSt], (t / kSt) & 1);
    } else if (warp == 1) {
      // ---------------------------------------------------- MMA issue
      // The whole warp walks the items in step; one elected lane issues.
      constexpr uint32_t kIdescS = idesc_f16_f32(FP16, 128, 128, 0, 0);
      constexpr uint32_t kIdescO = idesc_f16_f32(FP16, 128, D, 0, 1);
      const uint64_t dQ0 = sdesc_sw128(smem_u32(sQ), 16, 1024);
      const uint64_t dK0 = sdesc_sw128(smem_u32(sK), 16, 1024);
      // V is read MN-major: 64-feature atoms 16 KB apart (d = 64: one atom)
      const uint64_t dV0 = sdesc_sw128(smem_u32(sV), D == 128 ? 16384 : 0, 1024);
      constexpr uint64_t kStep = C::kTile >> 4;
      auto wait = [&](uint64_t* bar, uint32_t parity) -> bool {
        return mbar_sleep_warp(bar, parity, abort_flag, p.status);
      };
      bool held = p.stall && blockIdx.x == 0;  // the test hook's first hand-off
      int np = 0, cnt = 0;         // pieces read, items issued
      int t = 0;                   // running key tile
      // the PV products due, of the items cnt - 2 and cnt - 1: tile and
      // 1: adds to O, 2: last of its tile, 4: last of its piece on the stream
      int t2 = -1, t1 = -1;
      uint32_t f2 = 0, f1 = 0;
      bool ok = true;
      // Inside an item the lanes wait without a vote (a product issued after a
      // wait that ran out reads stale operands, and its result is dropped);
      // they agree on stopping once per item.
      auto issue_pv = [&](int item, int tile, uint32_t f) -> bool {
        const int s = item & 1, st = tile % kSt;
        const uint32_t ph = (item >> 1) & 1, vh = (tile / kSt) & 1;
        // one look at both barriers, whose latencies then overlap
        const bool pr = mbar_try_wait(&p_full[2 * s], ph), vr = mbar_try_wait(&v_full[st], vh);
        bool good = vr || mbar_sleep(&v_full[st], vh, abort_flag, p.status);
        good &= pr || mbar_sleep(&p_full[2 * s], ph, abort_flag, p.status);
        __syncwarp();
        tc_fence_after();
        const uint32_t a = tbase + 128 * s, o = tbase + 256 + D * s;
        const uint64_t b = dV0 + st * kStep;
        const uint32_t add = f & 1u;
        if (elect_one()) {
          tc_mma_f16_ts(o, a, b, kIdescO, add);
#pragma unroll
          for (int kk = 1; kk < 4; ++kk) tc_mma_f16_ts(o, a + 8 * kk, b + 128 * kk, kIdescO, 1u);
        }
        __syncwarp();
        good &= mbar_sleep(&p_full[2 * s + 1], (item >> 1) & 1, abort_flag, p.status);
        __syncwarp();
        tc_fence_after();
        if (elect_one()) {
#pragma unroll
          for (int kk = 4; kk < 8; ++kk) tc_mma_f16_ts(o, a + 8 * kk, b + 128 * kk, kIdescO, 1u);
          if (f & 2u) tc_commit(&v_empty[st]);
          if (f & 4u) tc_commit(&o_full[s]);
        }
        __syncwarp();
        return good;
      };
      while (ok) {
        const int slot = np % kRing;
        if (!(ok = wait(&pc_full[slot], (np / kRing) & 1))) break;
        const volatile Piece* c = reinterpret_cast<volatile Piece*>(ring + slot * kPieceInts);
        const int nt = __shfl_sync(0xffffffffu, c->nt, 0), pair = __shfl_sync(0xffffffffu, c->pair, 0);
        const int qpos = __shfl_sync(0xffffffffu, c->qpos, 0);
        __syncwarp();
        if (elect_one()) mbar_arrive(&pc_empty[slot]);
        ++np;
        if (nt == 0) break;
        const int ni = pair ? 2 * nt : nt;
        for (int i = 0; i < ni; ++i) {
          const int s = cnt & 1, st = t % kSt;
          const int q = qpos + (i & pair), qs = q & 1;
          const uint32_t kh = (t / kSt) & 1;
          const bool kr = mbar_try_wait(&k_full[st], kh);
          if (t2 >= 0) ok = issue_pv(cnt - 2, t2, f2);
          if (i <= pair) ok &= mbar_sleep(&q_full[qs], (q >> 1) & 1, abort_flag, p.status);
          if (!kr) ok &= mbar_sleep(&k_full[st], kh, abort_flag, p.status);
          __syncwarp();
          tc_fence_after();
          const uint64_t a = dQ0 + qs * kStep, b = dK0 + st * kStep;
          const uint32_t ds = tbase + 128 * s;
          const bool tile_end = !pair || (i & 1);
          if (elect_one()) {
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk)
              tc_mma_bf16(ds, a + (kk >> 2) * 1024 + (kk & 3) * 2, b + (kk >> 2) * 1024 + (kk & 3) * 2, kIdescS,
                          kk ? 1u : 0u);
            if (!held) tc_commit(&s_full[s]);
            if (tile_end) tc_commit(&k_empty[st]);
            if (i >= ni - 1 - pair) tc_commit(&q_empty[qs]);
          }
          __syncwarp();
          if (!(ok = __all_sync(0xffffffffu, ok))) break;
          t2 = t1;
          f2 = f1;
          t1 = t;
          f1 = (i >= 2 ? 1u : 0u) | (tile_end ? 2u : 0u) | (i >= ni - 2 ? 4u : 0u);
          ++cnt;
          held = false;
          t += tile_end;
        }
      }
      if (ok && t2 >= 0) ok = __all_sync(0xffffffffu, issue_pv(cnt - 2, t2, f2));
      if (ok && t1 >= 0) ok = __all_sync(0xffffffffu, issue_pv(cnt - 1, t1, f1));
      // every product must be done before TMEM is freed
      if (elect_one()) {
        tc_commit(drain);
        mbar_drain(drain, 0);
      }
    }
    __syncwarp();
  } else {
    reg_alloc<kRegsSoftmax>();
    // -------------------------------------------------------- softmax streams
    const int s = (warp >> 2) - 1;         // stream
    const int x = (warp & 3) * 32 + lane;  // row of the tile = TMEM lane
    const uint32_t lane_addr = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t s_addr = tbase + lane_addr + 128 * s;
    const uint32_t o_addr = tbase + lane_addr + 256 + D * s;
    int np = 0, ns = 0, no = 0;
    bool ok = true;
    auto wait = [&](uint64_t* bar, uint32_t parity) -> bool {
      return mbar_sleep_warp(bar, parity, abort_flag, p.status);
    };
    while (ok) {
      const int slot = np % kRing;
      if (!(ok = wait(&pc_full[slot], (np / kRing) & 1))) break;
      Piece c;
      {
        int* w = reinterpret_cast<int*>(&c);
#pragma unroll
        for (int i = 0; i < kPieceInts; ++i) w[i] = uniform(ring[slot * kPieceInts + i]);
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&pc_empty[slot]);
      __syncwarp();
      ++np;
      if (c.nt == 0) break;
      const int sub = s ^ (c.items & 1);
      if (!c.pair && sub >= c.nt) {
        // a single tile, the other stream's: a part without terms
        const int stride = c.prefix ? p.pre_nb * p.pre_rb : p.own_rb;
        if (x < stride)
          p.part_ml[(c.prefix ? 0 : p.pre_slots) + (static_cast<long long>(c.slot) * 2 + sub) * stride + x] =
              make_float2(-INFINITY, 0.f);
        continue;
      }
      const int tile = c.tile0 + (c.pair ? sub : 0);
      // this thread's row
      int r;
      bool valid;
      int stride;
      if (c.prefix) {
        stride = p.pre_nb * p.pre_rb;
        if (p.GT >= 128) {
          r = tile % ((p.GT + 127) / 128) * 128 + x;
          valid = r < p.GT;
        } else {
          const int i = x / p.GT;
          r = x - i * p.GT;
          valid = i < p.pre_nb && tile * p.pre_nb + i < p.n;
        }
      } else {
        stride = p.own_rb;
        r = tile * 128 + x;
        valid = x < p.own_rb && r < p.GT;
      }
      const int vis = c.prefix ? c.len : c.len - (p.T - 1 - r % p.T);  // keys this row sees
      const int vis_min = c.prefix ? c.len : c.len - (p.T - 1);
      const bool any_valid = __any_sync(0xffffffffu, valid);
      float m = -INFINITY, l = 0.f;
      const int step = c.pair ? 1 : 2;
      for (int j = c.pair ? 0 : sub; j < c.nt; j += step) {
        const int key0 = 128 * (c.j0 + j);
        if (!(ok = wait(&s_full[s], ns & 1))) break;
        ++ns;
        if (c.len - key0 < 128) {
          // the segment's last tile: clear the V rows past its length
          const int t = c.tiles + j, st = t % kSt;
          if (!(ok = wait(&v_full[st], (t / kSt) & 1))) break;
          const int first = c.len - key0, bytes = (128 - first) * 128;
#pragma unroll
          for (int ch = 0; ch < C::kChunks; ++ch) {
            const uint32_t base = smem_u32(sV + st * C::kTile + ch * 16384) + first * 128;
            for (int o = x * 16; o < bytes; o += 128 * 16) st_shared_v4(base + o, 0u, 0u, 0u, 0u);
          }
          fence_async_shared();
          __syncwarp();
        }
        if (any_valid) {
          tc_fence_after();
          float sv[128];
#pragma unroll
          for (int i = 0; i < 4; ++i) tmem_ld32(s_addr + 32 * i, *reinterpret_cast<float(*)[32]>(&sv[32 * i]));
          tc_wait_ld();
          if (key0 + 128 > vis_min) {
            // the masked keys' logits may be anything, NaN included; their
            // terms come out as 2^-inf = 0
            const int lim = vis - key0;
#pragma unroll
            for (int i = 0; i < 128; ++i) sv[i] = i < lim ? sv[i] : -INFINITY;
          }
          float mx[4] = {sv[0], sv[1], sv[2], sv[3]};
#pragma unroll
          for (int i = 4; i < 124; i += 8)
#pragma unroll
            for (int k = 0; k < 4; ++k) mx[k] = max3(mx[k], sv[i + 2 * k], sv[i + 2 * k + 1]);
          mx[0] = max3(mx[0], sv[124], sv[125]);
          mx[1] = max3(mx[1], sv[126], sv[127]);
          const float top = max3(fmaxf(mx[0], mx[1]), mx[2], mx[3]) * p.scale_log2;
          if (j < step) {
            m = top;  // the piece's first tile on this stream: O starts from zero
          } else if (__any_sync(0xffffffffu, top > m + kRescale)) {
            // move the reference: S of this tile is ready, so the PV product
            // before it (same issuing thread) is done and O is still
            const float mn = fmaxf(m, top);
            const float f = mn == -INFINITY ? 1.f : ex2_approx(m - mn);
            l *= f;
            m = mn;
#pragma unroll 1
            for (int i = 0; i < D / 16; ++i) {
              uint32_t ou[16];
              tmem_ld16(o_addr + 16 * i, ou);
              tc_wait_ld();
#pragma unroll
              for (int k = 0; k < 16; ++k) ou[k] = __float_as_uint(__uint_as_float(ou[k]) * f);
              tmem_st16(o_addr + 16 * i, ou);
            }
          }
          const float neg = m == -INFINITY ? 0.f : -m;
          float ls[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            uint32_t pk[32];
            exps<FP16>(sv + 64 * h, p.scale_log2, neg, ls, pk);
            tmem_st32(s_addr + 32 * h, pk);
            tc_wait_st();
            tc_fence_before();
            if (h == 0) {
              __syncwarp();
              if (lane == 0) mbar_arrive(&p_full[2 * s]);
              __syncwarp();
            }
          }
          l += (ls[0] + ls[1]) + (ls[2] + ls[3]);
        } else if (lane == 0) {
          mbar_arrive(&p_full[2 * s]);
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&p_full[2 * s + 1]);
        __syncwarp();
      }
      if (!ok) break;
      // the piece's part
      if (!(ok = wait(&o_full[s], no & 1))) break;
      ++no;
      if (any_valid) {
        tc_fence_after();
        const long long at =
            (c.prefix ? 0 : p.pre_slots) + (static_cast<long long>(c.slot) * 2 + sub) * stride + x;
        float* po = p.part_o + at * D;
#pragma unroll 1
        for (int i = 0; i < D / 32; ++i) {
          float ov[32];
          tmem_ld32(o_addr + 32 * i, ov);
          tc_wait_ld();
          if (valid) {
#pragma unroll
            for (int k = 0; k < 32; k += 4)
              *reinterpret_cast<float4*>(po + 32 * i + k) = make_float4(ov[k], ov[k + 1], ov[k + 2], ov[k + 3]);
          }
        }
        if (valid) p.part_ml[at] = make_float2(m, l);
        tc_fence_before();
      }
      __syncwarp();
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tbase, 512);
  }
}

// ------------------------------------------------------------------ merge
// With M the largest reference of a row's parts,
//   out = sum_p 2^(m_p - M) O_p / sum_p 2^(m_p - M) l_p.
// A row's parts are its prefix unit's and its cache unit's, one (pair) or two
// per run that has tiles of the unit; the order of the sums is fixed.

// Where the parts of output row `row` = (b, hkv, r) are: part q of segment
// kind h (0: prefix, 1: cache) at place first[h] + q * step[h].
struct RowParts {
  int cnt[2], first[2], step[2];
};
__device__ __forceinline__ RowParts row_parts(const Params& p, int row) {
  RowParts k = {{0, 0}, {0, 0}, {0, 0}};
  const int bh = row / p.GT, r = row - bh * p.GT;
  const int b = bh / p.Hkv, hkv = bh - b * p.Hkv;
#pragma unroll
  for (int half = 0; half < 2; ++half) {
    if (half == 0 ? p.npre == 0 : p.nseg == p.npre) continue;
    const int outer = half == 0 ? b / p.n : b;
    const int len = seg_len(p, half == 0 ? outer : p.npre + b);
    const int up = half == 0 ? p.pre_up : p.own_up, rt = half == 0 ? p.pre_rt : p.own_rt;
    const int stride = half == 0 ? p.pre_nb * p.pre_rb : p.own_rb;
    int tile, x;
    if (half == 0 && p.GT < 128) {
      const int i = b - outer * p.n;
      tile = i / p.pre_nb;
      x = (i - tile * p.pre_nb) * p.GT + r;
    } else {
      tile = r / 128 + (half == 0 ? (b - outer * p.n) * ((p.GT + 127) / 128) : 0);
      x = r % 128;
    }
    const bool pair = (tile | 1) < rt;
    const int unit = (outer * p.Hkv + hkv) * up + (tile >> 1);
    int2 c = p.unit_ctas[(half == 0 ? 0 : p.own_unit0) + unit];
    if (len == 0) continue;  // no pieces, and `c` is not this call's
    // after a wait that ran out it may be unwritten: no place past the parts
    c.x = min(max(c.x, 0), kMaxCtas - 1);
    c.y = min(max(c.y, c.x), kMaxCtas - 1);
    // a pair's row has one part per run (stream tile & 1), another's two
    k.cnt[half] = (c.y - c.x + 1) * (pair ? 1 : 2);
    k.step[half] = pair ? 2 * stride : stride;
    k.first[half] = static_cast<int>((half == 0 ? 0 : p.pre_slots) + 2LL * (unit + c.x) * stride +
                                     (pair ? (tile & 1) * stride : 0)) + x;
  }
  return k;
}
__device__ __forceinline__ int part_at(const RowParts& k, int q) {
  return q < k.cnt[0] ? k.first[0] + q * k.step[0] : k.first[1] + (q - k.cnt[0]) * k.step[1];
}

template <int kV>
__device__ __forceinline__ void load_part(float (&v)[kV], const float* src) {
  if constexpr (kV == 4) {
    const float4 u = *reinterpret_cast<const float4*>(src);
    v[0] = u.x, v[1] = u.y, v[2] = u.z, v[3] = u.w;
  } else {
    const float2 u = *reinterpret_cast<const float2*>(src);
    v[0] = u.x, v[1] = u.y;
  }
}
template <int kV>
__device__ __forceinline__ void add_part(float (&acc)[kV], float f, const float (&v)[kV]) {
#pragma unroll
  for (int i = 0; i < kV; ++i) acc[i] += f * v[i];
}
template <int kV>
__device__ __forceinline__ void add_part(float (&acc)[kV], float f, const float* src) {
  float v[kV];
  load_part<kV>(v, src);
  add_part<kV>(acc, f, v);
}
// O of a warp's first parts is fetched along with the references, before it is
// known which parts count (a part that does not is not added, whatever is
// there).  A round trip less: 16 samples of a 32K prompt 43.6 -> 42.6 us a call
// with four, 41.6 with eight (five of a warp's parts there).
constexpr int kAhead = 8;

// Few parts per row: a warp per row, 32 parts at a time.  (4096 rows of 14
// parts: 22 us with a block of eight warps per row, whose barriers and waves
// cost more than the parts.)
template <int D, bool FP16>
__global__ void __launch_bounds__(128) merge_kernel(const Params p, int rows, uint16_t* out, float* lse) {
  constexpr int kV = D / 32;  // values per lane
  grid_dep_launch();
  grid_dep_wait();
  const int lane = threadIdx.x & 31;
  const int row = static_cast<int>(blockIdx.x) * 4 + uniform(threadIdx.x >> 5);
  if (row >= rows) return;
  const RowParts k = row_parts(p, row);
  const int n = uniform(k.cnt[0] + k.cnt[1]);
  float acc[kV];
#pragma unroll
  for (int i = 0; i < kV; ++i) acc[i] = 0.f;
  float M = -INFINITY, L = 0.f;
  float ahead[kAhead][kV];
#pragma unroll
  for (int j = 0; j < kAhead; ++j)
    if (j < n) load_part<kV>(ahead[j], p.part_o + static_cast<long long>(part_at(k, j)) * D + lane * kV);
  for (int q0 = 0; q0 < n; q0 += 32) {
    const int at = q0 + lane < n ? part_at(k, q0 + lane) : 0;
    const float2 ml = q0 + lane < n ? p.part_ml[at] : make_float2(-INFINITY, 0.f);
    float top = ml.x;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    top = fmaxf(top, M);
    const float old = M == -INFINITY ? (L == 0.f ? 0.f : 1.f) : ex2_approx(M - top);
    // nothing visible in this part: weight 0, and its O is not read
    const float f = ml.x == -INFINITY && ml.y == 0.f ? 0.f : ex2_approx(ml.x - top);
    float l = f == 0.f ? 0.f : f * ml.y;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
    M = top;
    L = L * old + l;
#pragma unroll
    for (int i = 0; i < kV; ++i) acc[i] *= old;
    const int m = min(32, n - q0);
    if (q0 == 0) {
#pragma unroll
      for (int j = 0; j < kAhead; ++j) {
        const float fj = __shfl_sync(0xffffffffu, f, j);  // (0 from n on)
        if (fj != 0.f) add_part<kV>(acc, fj, ahead[j]);
      }
    }
#pragma unroll 8
    for (int j = q0 == 0 ? kAhead : 0; j < m; ++j) {
      const float fj = __shfl_sync(0xffffffffu, f, j);
      const int aj = __shfl_sync(0xffffffffu, at, j);
      if (fj != 0.f) add_part<kV>(acc, fj, p.part_o + static_cast<long long>(aj) * D + lane * kV);
    }
  }
  const bool empty = M == -INFINITY && L == 0.f;
  const float inv = 1.f / L;
  uint16_t* dst = out + static_cast<long long>(row) * D + lane * kV;
  if constexpr (kV == 4) {
    const uint2 u = empty ? make_uint2(0, 0) : make_uint2(pack_16x2<FP16>(acc[0] * inv, acc[1] * inv),
                                                          pack_16x2<FP16>(acc[2] * inv, acc[3] * inv));
    *reinterpret_cast<uint2*>(dst) = u;
  } else {
    *reinterpret_cast<uint32_t*>(dst) = empty ? 0u : pack_16x2<FP16>(acc[0] * inv, acc[1] * inv);
  }
  if (lse && lane == 0) lse[row] = empty ? -INFINITY : (M + log2f(L)) * kLn2;
}

// A prefix cut over the whole machine: eight warps per row, whose reads of O
// would be one warp's chain of round trips (shared 32K prefix, 40 parts: 8 us
// with four warps, 5 with eight).
constexpr int kMaxParts = 4 * kMaxCtas;  // two per run of the prefixes, two of the caches

template <int D, bool FP16>
__global__ void __launch_bounds__(256) merge_wide_kernel(const Params p, uint16_t* out, float* lse) {
  constexpr int kV = D / 32, W = 8;
  __shared__ float w[kMaxParts];
  __shared__ int at[kMaxParts];
  __shared__ float so[W][D];
  __shared__ float red[W];
  grid_dep_launch();
  grid_dep_wait();
  const int row = blockIdx.x;
  const int warp = uniform(threadIdx.x >> 5), lane = threadIdx.x & 31;
  const RowParts k = row_parts(p, row);
  const int n = uniform(k.cnt[0] + k.cnt[1]);
  float ahead[kAhead][kV];
#pragma unroll
  for (int j = 0; j < kAhead; ++j)
    if (warp + W * j < n)
      load_part<kV>(ahead[j], p.part_o + static_cast<long long>(part_at(k, warp + W * j)) * D + lane * kV);
  float M = -INFINITY;
  for (int q = threadIdx.x; q < n; q += 32 * W) {
    const int a = part_at(k, q);
    at[q] = a;
    M = fmaxf(M, p.part_ml[a].x);
  }
  __syncwarp();
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
  if (lane == 0) red[warp] = M;
  __syncthreads();
  M = red[0];
#pragma unroll
  for (int i = 1; i < W; ++i) M = fmaxf(M, red[i]);
  float L = 0.f;
  for (int q = threadIdx.x; q < n; q += 32 * W) {
    const float2 ml = p.part_ml[at[q]];
    const float f = ml.x == -INFINITY && ml.y == 0.f ? 0.f : ex2_approx(ml.x - M);
    w[q] = f;
    if (f != 0.f) L += f * ml.y;
  }
  __syncwarp();
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) L += __shfl_xor_sync(0xffffffffu, L, o);
  __syncthreads();
  if (lane == 0) red[warp] = L;
  __syncthreads();
  L = 0.f;
#pragma unroll
  for (int i = 0; i < W; ++i) L += red[i];
  float acc[kV];
#pragma unroll
  for (int i = 0; i < kV; ++i) acc[i] = 0.f;
#pragma unroll
  for (int j = 0; j < kAhead; ++j) {
    const float f = warp + W * j < n ? w[warp + W * j] : 0.f;
    if (f != 0.f) add_part<kV>(acc, f, ahead[j]);
  }
#pragma unroll 4
  for (int q = warp + W * kAhead; q < n; q += W) {
    const float f = w[q];
    if (f != 0.f) add_part<kV>(acc, f, p.part_o + static_cast<long long>(at[q]) * D + lane * kV);
  }
#pragma unroll
  for (int i = 0; i < kV; ++i) so[warp][lane * kV + i] = acc[i];
  __syncthreads();
  const bool empty = M == -INFINITY && L == 0.f;
  const int i = 2 * threadIdx.x;
  if (i < D) {
    float a0 = 0.f, a1 = 0.f;
#pragma unroll
    for (int j = 0; j < W; ++j) {
      a0 += so[j][i];
      a1 += so[j][i + 1];
    }
    const uint32_t u = empty ? 0u : pack_16x2<FP16>(a0 / L, a1 / L);
    *reinterpret_cast<uint32_t*>(out + static_cast<long long>(row) * D + i) = u;
  }
  if (lse && threadIdx.x == 0) lse[row] = empty ? -INFINITY : (M + log2f(L)) * kLn2;
}

size_t align256(size_t v) { return (v + 255) & ~static_cast<size_t>(255); }

struct Plan {
  Params p = {};
  long long pre_units = 0, own_units = 0, part_rows = 0;
  size_t off_units = 0, off_ml = 0, off_o = 0, total = 0;
};

// Everything that follows from the sizes alone.
bool make_plan(Plan& w, int B, int G, int Hkv, int T, int d, int Bp, int P, int C) {
  Params& p = w.p;
  p.B = B;
  p.G = G;
  p.Hkv = Hkv;
  p.T = T;
  p.Bp = Bp;
  p.n = B / Bp;
  p.P = P;
  p.C = C;
  p.GT = G * T;
  p.npre = P > 0 ? Bp : 0;
  p.nseg = p.npre + (C > 0 ? B : 0);
  if (p.GT >= 128) {
    p.pre_nb = 1;
    p.pre_rb = 128;
    p.pre_rt = p.n * ((p.GT + 127) / 128);
  } else {
    p.pre_nb = 128 / p.GT < p.n ? 128 / p.GT : p.n;
    p.pre_rb = p.GT;
    p.pre_rt = (p.n + p.pre_nb - 1) / p.pre_nb;
  }
  p.pre_up = (p.pre_rt + 1) / 2;
  p.own_rb = p.GT < 128 ? p.GT : 128;
  p.own_rt = (p.GT + 127) / 128;
  p.own_up = (p.own_rt + 1) / 2;
  w.pre_units = P > 0 ? static_cast<long long>(Bp) * Hkv * p.pre_up : 0;
  w.own_units = C > 0 ? static_cast<long long>(B) * Hkv * p.own_up : 0;
  const long long work = static_cast<long long>(p.npre) * Hkv * p.pre_rt * ((P + 127LL) / 128) +
                         (C > 0 ? static_cast<long long>(B) * Hkv * p.own_rt * ((C + 127LL) / 128) : 0);
  if (w.pre_units + w.own_units > (1LL << 30) || work > (1LL << 30)) return false;
  p.own_unit0 = w.pre_units;
  p.pre_slots = P > 0 ? (w.pre_units + kMaxCtas) * 2 * p.pre_nb * p.pre_rb : 0;
  w.part_rows = p.pre_slots + (C > 0 ? (w.own_units + kMaxCtas) * 2 * p.own_rb : 0);
  if (w.part_rows >= (1LL << 31)) return false;
  size_t o = 256;
  w.off_units = o;
  o += align256(static_cast<size_t>(w.pre_units + w.own_units) * 8);
  w.off_ml = o;
  o += align256(static_cast<size_t>(w.part_rows) * 8);
  w.off_o = o;
  o += align256(static_cast<size_t>(w.part_rows) * d * 4);
  w.total = o;
  return true;
}

template <int D, bool FP16>
cudaError_t run(const DecodeLaunch& a, const Plan& w, const CUtensorMap (&m)[6], int grid, cudaStream_t st) {
  const cudaError_t e = cudaFuncSetAttribute(decode_kernel<D, FP16>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             Cfg<D>::kSmem);
  if (e != cudaSuccess) return e;
  const cudaError_t e2 = launch_chained(decode_kernel<D, FP16>, dim3(grid), dim3(kThreads), Cfg<D>::kSmem, st, m[0],
                                        m[1], m[2], m[3], m[4], m[5], w.p);
  if (e2 != cudaSuccess) return e2;
  const int rows = a.B * a.Hkv * w.p.GT;
  // parts per row: the runs that share one unit's keys, two of each where a
  // unit is a single row tile
  const bool pre = w.pre_units > 0;
  const long long units = pre ? w.pre_units : w.own_units;
  const long long parts = (pre ? w.p.pre_rt : w.p.own_rt) > 1 ? grid / units : 2 * grid / units;
  uint16_t* out = static_cast<uint16_t*>(a.out);
  // few rows leave the machine idle: a block each (two rows of 16 parts 9.0 us a
  // call against 11.2); many rows of few parts want a warp each
  if (parts > 16 || (parts > 2 && rows <= 4 * device_sm_count()))
    return launch_chained(merge_wide_kernel<D, FP16>, dim3(static_cast<unsigned>(rows)), dim3(256), 0, st, w.p, out,
                          a.lse);
  return launch_chained(merge_kernel<D, FP16>, dim3(static_cast<unsigned>((rows + 3) / 4)), dim3(128), 0, st, w.p,
                        rows, out, a.lse);
}

}  // namespace

size_t decode_workspace_bytes(int B, int G, int Hkv, int T, int d, int Bp, int P, int C) {
  Plan w;
  return make_plan(w, B, G, Hkv, T, d, Bp, P, C) ? w.total : 0;
}

cudaError_t launch_decode(const DecodeLaunch& a, cudaStream_t st) {
  Plan w;
  if (!make_plan(w, a.B, a.G, a.Hkv, a.T, a.d, a.Bp, a.P, a.C)) return cudaErrorInvalidValue;
  Params& p = w.p;
  p.prefix_len = a.prefix_len;
  p.cache_len = a.cache_len;
  p.scale_log2 = 1.4426950408889634f / (a.d == 128 ? 11.313708498984761f : 8.0f);
  p.status = reinterpret_cast<int*>(a.ws);
  p.unit_ctas = reinterpret_cast<int2*>(a.ws + w.off_units);
  p.part_ml = reinterpret_cast<float2*>(a.ws + w.off_ml);
  p.part_o = reinterpret_cast<float*>(a.ws + w.off_o);
  p.stall = take_serve_stall_request();
  // Q: [B][Hkv][G T][d]; prefix tiles take pre_nb sequences at once
  CUtensorMap m[6];
  const uint64_t u = 1;
  const uint64_t dq[4] = {u * a.d, u * p.GT, u * a.Hkv, u * a.B};
  const uint32_t bp[4] = {64, static_cast<uint32_t>(p.pre_rb), 1, static_cast<uint32_t>(p.pre_nb)};
  // A cache's box is a whole tile, whose rows past G T come in as zeros: products
  // of zeros cost less power than products of whatever was there (64 ragged
  // caches of 4 rows, after 500 calls: 102 -> 98 us).
  const uint32_t bc[4] = {64, 128, 1, 1};
  const uint32_t bk[3] = {64, 64, 1};
  const uint64_t dp[3] = {u * a.d, u * a.P, u * a.Bp * a.Hkv}, dc[3] = {u * a.d, u * a.C, u * a.B * a.Hkv};
  CUresult r = encode_tensor_map_16(&m[0], a.q, a.fp16, 4, dq, bp);
  if (r == CUDA_SUCCESS) r = encode_tensor_map_16(&m[1], a.q, a.fp16, 4, dq, bc);
  if (a.P > 0) {
    if (r == CUDA_SUCCESS) r = encode_tensor_map_16(&m[2], a.k_prefix, a.fp16, 3, dp, bk);
    if (r == CUDA_SUCCESS) r = encode_tensor_map_16(&m[3], a.v_prefix, a.fp16, 3, dp, bk);
  }
  if (a.C > 0) {
    if (r == CUDA_SUCCESS) r = encode_tensor_map_16(&m[4], a.k_cache, a.fp16, 3, dc, bk);
    if (r == CUDA_SUCCESS) r = encode_tensor_map_16(&m[5], a.v_cache, a.fp16, 3, dc, bk);
  }
  if (r != CUDA_SUCCESS) return cudaErrorInvalidValue;
  if (a.P == 0) m[2] = m[4], m[3] = m[5];
  if (a.C == 0) m[4] = m[2], m[5] = m[3];
  // one CTA per SM; no more than there can be tiles (a pair's count once)
  const long long tiles = w.pre_units * ((a.P + 127LL) / 128) + w.own_units * ((a.C + 127LL) / 128);
  int grid = device_sm_count();
  if (grid > kMaxCtas) grid = kMaxCtas;
  if (tiles < grid) grid = static_cast<int>(tiles < 1 ? 1 : tiles);
  if (a.d == 128)
    return a.fp16 ? run<128, true>(a, w, m, grid, st) : run<128, false>(a, w, m, grid, st);
  return a.fp16 ? run<64, true>(a, w, m, grid, st) : run<64, false>(a, w, m, grid, st);
}

}  // namespace psa
