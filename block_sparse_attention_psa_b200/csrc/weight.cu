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
// columns per broadcast load.
//
//  * Decode reads K once for few queries: bound by DRAM.  A prefill does 2 d
//    operations and one exponential per (query, key) pair: an SM's tensor
//    core takes 256 cycles for a tile, its 16 exponentials a cycle 1024, so
//    it is bound by the exponentials.
//  * Unit: a pair of key tiles (256 keys) of one KV head, held in shared
//    memory, with the query tiles streamed past it; each of the two
//    warpgroups owns one key tile, so a query tile is loaded once for both,
//    and each has two S buffers (512 TMEM columns in all).
//  * Query tiles: T >= 128 tokens: 128 tokens of one head, so that causal
//    tiles past the diagonal are skipped; fewer: up to 128 of the G T rows
//    that share the KV head, over several sequences when they share the keys.
//  * Units go to the CTAs in turn, forwards and backwards, heaviest (fewest
//    keys hidden) first.  When there are fewer units than two per SM the query
//    tiles of a unit are split over several, whose sums a second kernel adds
//    in a fixed order.
//  * Sums: 128 columns in four fp32 accumulators, tile sums added with a
//    compensation term (a key of a long prefill sums 10^5 terms).
// Every wait is bounded.
#include <climits>

#include "internal.h"
#include "sm100.cuh"

namespace psa {
namespace {

constexpr int kThreads = 384;      // WG0: K/Q loads, MMA issue, lse loads; WG1, WG2: one key tile each
constexpr int kRegsProducer = 72;  // 128 x 72 + 256 x 216 = 384 x 168
constexpr int kRegsSum = 216;
constexpr int kLse = 4;            // query tiles whose lse is in shared memory
constexpr int kPlanSms = 148;      // SMs the split is planned for (fixed: it sizes the workspace)
constexpr float kLog2e = 1.4426950408889634f;

template <int D>
struct Cfg {
  static constexpr int kChunks = D / 64;
  static constexpr int kTile = 128 * D * 2;
  static constexpr int kQStages = D == 128 ? 2 : 4;
  static constexpr int kOffK = 0;               // two pairs of key tiles
  static constexpr int kOffQ = 4 * kTile;
  static constexpr int kOffLse = kOffQ + kQStages * kTile;
  static constexpr int kOffMisc = kOffLse + kLse * 1024;
  static constexpr int kSmem = kOffMisc + 512 + 1024;  // + alignment slack
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
  int Z, pairs, units;
  float scale_log2;
  int* status;
};

struct Unit {
  int bk, hkv, key0, len;
  int t_min, per;         // by_head: first visible tile, tiles per head
  int f0, f1;             // query tiles of this unit
};

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
  const int n = p.key_len ? __ldg(p.key_len + bk) : p.C;
  return min(max(n, 0), p.C);
}

// The w-th unit of this CTA, or -1: rows of gridDim.x units, every other row
// taken backwards.
__device__ __forceinline__ int unit_id(const Params& p, int w) {
  const int g = static_cast<int>(gridDim.x), c = static_cast<int>(blockIdx.x);
  const long long u = static_cast<long long>(w) * g + ((w & 1) ? g - 1 - c : c);
  return u < p.units ? static_cast<int>(u) : (static_cast<long long>(w) * g < p.units ? -2 : -1);
}

__device__ __forceinline__ int unit_bk(const Params& p, int u) { return u % (p.Bk * p.Hkv) / p.Hkv; }

__device__ __forceinline__ Unit make_unit(const Params& p, int u, int len) {
  Unit x;
  const int bh = u % (p.Bk * p.Hkv), pz = u / (p.Bk * p.Hkv);
  const int pair = pz / p.Z, z = pz - pair * p.Z;
  x.bk = bh / p.Hkv;
  x.hkv = bh - x.bk * p.Hkv;
  x.key0 = 256 * pair;
  x.len = len;
  int total = p.tiles;
  x.t_min = 0;
  x.per = p.tiles;
  if (p.by_head) {
    // token t sees key j iff j <= len - T + t
    if (p.causal) x.t_min = max(0, x.key0 - (len - p.T)) / 128;
    x.per = max(p.tiles - x.t_min, 0);
    total = p.n * p.G * x.per;
  }
  if (x.key0 >= len) total = 0;
  x.f0 = static_cast<int>(static_cast<long long>(total) * z / p.Z);
  x.f1 = static_cast<int>(static_cast<long long>(total) * (z + 1) / p.Z);
  return x;
}

// Query tile f of a unit.
struct Tile {
  int b, head, r0;  // first sequence, query head (by_head) and row
  int cols;         // valid columns
};
__device__ __forceinline__ Tile make_tile(const Params& p, const Unit& x, int f) {
  Tile t;
  t.head = 0;
  if (p.by_head) {
    const int o = f / x.per, i = o / p.G;
    t.b = x.bk * p.n + i;
    t.head = x.hkv * p.G + (o - i * p.G);
    t.r0 = 128 * (x.t_min + f - o * x.per);
    t.cols = min(128, p.T - t.r0);
  } else if (p.GT >= 128) {
    const int per = (p.GT + 127) / 128, i = f / per;
    t.b = x.bk * p.n + i;
    t.r0 = 128 * (f - i * per);
    t.cols = min(128, p.GT - t.r0);
  } else {
    t.b = x.bk * p.n + f * p.nb;
    t.r0 = 0;
    t.cols = min(p.nb, p.n - f * p.nb) * p.GT;
  }
  return t;
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
  float* sLse = reinterpret_cast<float*>(smem + C::kOffLse);           // [kLse][128] log2 units
  int* sLim = reinterpret_cast<int*>(smem + C::kOffLse + kLse * 512);  // [kLse][128] last visible key
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::kOffMisc);
  uint64_t* k_full = bars + 0;    // [2] a pair of key tiles landed  (TMA)
  uint64_t* k_empty = bars + 2;   // [2] its last product done       (commit)
  uint64_t* q_full = bars + 4;    // [kQ]
  uint64_t* q_empty = bars + 8;   // [kQ]
  uint64_t* s_full = bars + 12;   // [2 streams][2] S^T ready        (commit)
  uint64_t* s_empty = bars + 16;  // [2 streams][2] read             (4 warps)
  uint64_t* l_full = bars + 20;   // [kLse] lse of a query tile      (lse warp)
  uint64_t* l_empty = bars + 24;  // [kLse] read                     (8 warps)
  uint64_t* drain = bars + 28;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::kOffMisc + 256);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
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
      mbar_init(&s_empty[i], 4);
    }
    for (int i = 0; i < kLse; ++i) {
      mbar_init(&l_full[i], 1);
      mbar_init(&l_empty[i], 8);
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
        const int n = __ldg(p.key_len + i);
        bad |= n < 0 || n > p.C;
      }
    bad = __syncthreads_or(bad);
    if (threadIdx.x == 0) *p.status = bad ? kStatusLength : 0;
  }

  // Every role walks the CTA's units on its own, with the next unit's length
  // loaded ahead.  unit_id: -1 ends the walk, -2 is an empty place of the last row.
  auto first = [&](int& u, int& len) {
    u = unit_id(p, 0);
    len = u >= 0 ? clamped_len(p, unit_bk(p, u)) : 0;
  };

  if (warp < 4) {
    reg_dealloc<kRegsProducer>();
    if (warp == 0 && lane == 0) {
      // ---------------------------------------------------- K and Q loads
      int ku = 0, qt = 0;  // pairs and query tiles loaded
      bool ok = true;
      int u, len;
      first(u, len);
      for (int w = 0; ok && u != -1; ++w) {
        const int un = unit_id(p, w + 1), ln = un >= 0 ? clamped_len(p, unit_bk(p, un)) : 0;
        if (u >= 0) {
          const Unit x = make_unit(p, u, len);
          if (x.f0 < x.f1) {
            const int kb = ku & 1;
            ok = mbar_wait(&k_empty[kb], ((ku >> 1) & 1) ^ 1, abort_flag, p.status);
            if (!ok) break;
            // 64-key boxes; none that starts past the length
            const int boxes = min(4, (x.len - x.key0 + 63) / 64);
            mbar_arrive_expect_tx(&k_full[kb], boxes * 64 * 128 * C::kChunks);
            for (int i = 0; i < boxes; ++i)
#pragma unroll
              for (int ch = 0; ch < C::kChunks; ++ch)
                tma_load_3d(&tmK, sK + (2 * kb + (i >> 1)) * C::kTile + ch * 16384 + (i & 1) * 8192, &k_full[kb],
                            64 * ch, x.key0 + 64 * i, x.bk * p.Hkv + x.hkv);
            ++ku;
            for (int f = x.f0; f < x.f1; ++f, ++qt) {
              const int st = qt % kQ;
              ok = mbar_wait(&q_empty[st], ((qt / kQ) & 1) ^ 1, abort_flag, p.status);
              if (!ok) break;
              const Tile t = make_tile(p, x, f);
              mbar_arrive_expect_tx(&q_full[st], static_cast<uint32_t>(p.nb * p.rb) * 128 * C::kChunks);
#pragma unroll
              for (int ch = 0; ch < C::kChunks; ++ch)
                tma_load_4d(&tmQ, sQ + st * C::kTile + ch * 16384, &q_full[st], 64 * ch, t.r0,
                            p.by_head ? t.head : x.hkv, t.b);
            }
          }
        }
        u = un;
        len = ln;
      }
      // no bulk copy may still be writing shared memory when the CTA leaves
      for (int i = max(0, ku - 2); i < ku; ++i) mbar_drain(&k_full[i & 1], (i >> 1) & 1);
      for (int i = max(0, qt - kQ); i < qt; ++i) mbar_drain(&q_full[i % kQ], (i / kQ) & 1);
    } else if (warp == 1 && lane == 0) {
      // ---------------------------------------------------- MMA issue
      const uint64_t dK0 = sdesc_sw128(smem_u32(sK), 16, 1024);
      const uint64_t dQ0 = sdesc_sw128(smem_u32(sQ), 16, 1024);
      constexpr uint64_t kStep = C::kTile >> 4;
      int ku = 0, qt = 0;
      bool ok = true;
      int u, len;
      first(u, len);
      for (int w = 0; ok && u != -1; ++w) {
        const int un = unit_id(p, w + 1), ln = un >= 0 ? clamped_len(p, unit_bk(p, un)) : 0;
        if (u >= 0) {
          const Unit x = make_unit(p, u, len);
          if (x.f0 < x.f1) {
            const int kb = ku & 1;
            if (!(ok = mbar_wait(&k_full[kb], (ku >> 1) & 1, abort_flag, p.status))) break;
            for (int f = x.f0; f < x.f1 && ok; ++f, ++qt) {
              const int st = qt % kQ, buf = qt & 1;
              const Tile t = make_tile(p, x, f);
              const uint32_t idesc = idesc_f16_f32(FP16, 128, (t.cols + 15) & ~15, 0, 0);
              if (!(ok = mbar_wait(&q_full[st], (qt / kQ) & 1, abort_flag, p.status))) break;
#pragma unroll
              for (int s = 0; s < 2; ++s) {
                if (!(ok = mbar_wait(&s_empty[2 * s + buf], ((qt >> 1) & 1) ^ 1, abort_flag, p.status))) break;
                tc_fence_after();
                const uint64_t a = dK0 + (2 * kb + s) * kStep, b = dQ0 + st * kStep;
#pragma unroll
                for (int kk = 0; kk < D / 16; ++kk)
                  tc_mma_bf16(tbase + 256 * s + 128 * buf, a + (kk >> 2) * 1024 + (kk & 3) * 2,
                              b + (kk >> 2) * 1024 + (kk & 3) * 2, idesc, kk ? 1u : 0u);
                tc_commit(&s_full[2 * s + buf]);
              }
              if (!ok) break;
              tc_commit(&q_empty[st]);
              if (f == x.f1 - 1) tc_commit(&k_empty[kb]);
            }
            ++ku;
          }
        }
        u = un;
        len = ln;
      }
      tc_commit(drain);
      mbar_drain(drain, 0);
    } else if (warp == 2) {
      // ---------------------------------------------------- lse and limits per column
      int qt = 0;
      bool ok = true;
      int u, len;
      first(u, len);
      for (int w = 0; ok && u != -1; ++w) {
        const int un = unit_id(p, w + 1), ln = un >= 0 ? clamped_len(p, unit_bk(p, un)) : 0;
        if (u >= 0) {
          const Unit x = make_unit(p, u, len);
          for (int f = x.f0; f < x.f1; ++f, ++qt) {
            const Tile t = make_tile(p, x, f);
            float v[4];
            int lim[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const int c = lane + 32 * i;
              v[i] = INFINITY;
              lim[i] = -1;
              if (c < t.cols) {
                long long at;
                int tok;
                if (p.by_head) {
                  tok = t.r0 + c;
                  at = (static_cast<long long>(t.b) * p.Hkv * p.G + t.head) * p.T + tok;
                } else if (p.GT >= 128) {
                  tok = (t.r0 + c) % p.T;
                  at = (static_cast<long long>(t.b) * p.Hkv + x.hkv) * p.GT + t.r0 + c;
                } else {
                  const int i2 = c / p.GT, r = c - i2 * p.GT;
                  tok = r % p.T;
                  at = (static_cast<long long>(t.b + i2) * p.Hkv + x.hkv) * p.GT + r;
                }
                const float l = __ldg(p.lse + at);
                v[i] = l == -INFINITY ? INFINITY : l * kLog2e;  // a query that saw nothing adds nothing
                lim[i] = p.causal ? x.len - p.T + tok : INT_MAX;
              }
            }
            const int st = qt % kLse;
            ok = __all_sync(0xffffffffu, mbar_wait(&l_empty[st], ((qt / kLse) & 1) ^ 1, abort_flag, p.status));
            if (!ok) break;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              sLse[128 * st + lane + 32 * i] = v[i];
              sLim[128 * st + lane + 32 * i] = lim[i];
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&l_full[st]);
          }
        }
        u = un;
        len = ln;
      }
    }
    __syncwarp();
  } else {
    reg_alloc<kRegsSum>();
    // -------------------------------------------------------- sums per key
    const int s = (warp >> 2) - 1;
    const int row = (warp & 3) * 32 + lane;
    const uint32_t s_addr = tbase + (static_cast<uint32_t>((warp & 3) * 32) << 16) + 256 * s;
    int qt = 0;
    bool ok = true;
    auto wait = [&](uint64_t* bar, uint32_t parity) -> bool {
      return __all_sync(0xffffffffu, mbar_wait(bar, parity, abort_flag, p.status));
    };
    int u, len;
    first(u, len);
    for (int w = 0; ok && u != -1; ++w) {
      const int un = unit_id(p, w + 1), ln = un >= 0 ? clamped_len(p, unit_bk(p, un)) : 0;
      if (u >= 0) {
        const Unit x = make_unit(p, u, len);
        const int tile0 = x.key0 + 128 * s, key = tile0 + row;
        const long long at = static_cast<long long>(x.bk * p.Hkv + x.hkv) * p.C + key;
        const float before = p.Z == 1 && p.score_in && key < x.len ? p.score_in[at] : 0.f;
        float acc = 0.f, comp = 0.f;
        for (int f = x.f0; f < x.f1; ++f, ++qt) {
          const int buf = qt & 1, st = qt % kLse;
          const Tile t = make_tile(p, x, f);
          const bool mask =
              p.causal && tile0 + 127 > x.len - p.T + (p.by_head ? t.r0 : 0);
          if (!(ok = wait(&l_full[st], (qt / kLse) & 1))) break;
          if (!(ok = wait(&s_full[2 * s + buf], (qt >> 1) & 1))) break;
          tc_fence_after();
          const float* ls = sLse + 128 * st;
          const int* lm = sLim + 128 * st;
          float a0 = 0.f, a1 = 0.f, a2 = 0.f, a3 = 0.f;
          const int chunks = (t.cols + 31) >> 5;
#pragma unroll 1
          for (int c = 0; c < chunks; ++c) {
            float v[32];
            tmem_ld32(s_addr + 128 * buf + 32 * c, v);
            tc_wait_ld();
            if (mask || t.cols < 32 * (c + 1)) {
#pragma unroll
              for (int i = 0; i < 32; ++i) {
                const int col = 32 * c + i;
                const float e = ex2_approx(fmaf(v[i], p.scale_log2, -ls[col]));
                // a column that is no query of this tile has the limit -1
                if (key <= lm[col]) a0 += e;
              }
            } else {
#pragma unroll
              for (int i = 0; i < 32; i += 4) {
                const float4 l4 = *reinterpret_cast<const float4*>(ls + 32 * c + i);
                float x0, x1, x2, x3;
                ffma2(x0, x1, v[i], v[i + 1], p.scale_log2, p.scale_log2, -l4.x, -l4.y);
                ffma2(x2, x3, v[i + 2], v[i + 3], p.scale_log2, p.scale_log2, -l4.z, -l4.w);
                fadd2(a0, a1, a0, a1, ex2_approx(x0), ex2_approx(x1));
                fadd2(a2, a3, a2, a3, ex2_approx(x2), ex2_approx(x3));
              }
            }
          }
          tc_fence_before();
          __syncwarp();
          if (lane == 0) {
            mbar_arrive(&s_empty[2 * s + buf]);
            mbar_arrive(&l_empty[st]);
          }
          // compensated: the tile's sum joins the key's
          const float y = ((a0 + a1) + (a2 + a3)) - comp;
          const float z = acc + y;
          comp = (z - acc) - y;
          acc = z;
        }
        if (!ok) break;
        if (key < p.C) {
          if (p.Z > 1) {
            const int z = u / (p.Bk * p.Hkv) % p.Z;
            p.part[static_cast<long long>(z) * p.Bk * p.Hkv * p.C + at] = acc;
          } else {
            p.score_out[at] = key < x.len ? before + acc : 0.f;
          }
        }
      }
      u = un;
      len = ln;
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tbase, 512);
  }
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
  p.pairs = (C + 255) / 256;
  const long long units = static_cast<long long>(Bk) * Hkv * p.pairs;
  // two units per SM, of at least four query tiles each, 16 parts at most
  long long z = (2LL * kPlanSms + units - 1) / units;
  if (z > tiles / 4) z = tiles / 4;
  if (z > 16) z = 16;
  p.Z = z < 1 ? 1 : static_cast<int>(z);
  if (units * p.Z > INT_MAX / 2) return false;
  p.units = static_cast<int>(units * p.Z);
  return true;
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

}  // namespace

size_t weight_workspace_bytes(int B, int G, int Hkv, int T, int Bk, int C) {
  Params p = {};
  if (!make_plan(p, B, G, Hkv, T, Bk, C)) return 0;
  const size_t part = p.Z > 1 ? static_cast<size_t>(p.Z) * Bk * Hkv * C * 4 : 0;
  return 256 + ((part + 255) & ~static_cast<size_t>(255));
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
  if (p.units < grid) grid = p.units;
  if (a.d == 128) return a.fp16 ? run<128, true>(p, mq, mk, grid, st) : run<128, false>(p, mq, mk, grid, st);
  return a.fp16 ? run<64, true>(p, mq, mk, grid, st) : run<64, false>(p, mq, mk, grid, st);
}

}  // namespace psa
