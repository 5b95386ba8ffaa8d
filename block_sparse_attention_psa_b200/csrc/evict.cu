// evict.cu -- eviction from a key/value cache by accumulated attention
// weight: which entries stay (select_kernel) and the move of their rows
// (move_kernel).
//
// For one (sequence, KV head) with len entries and nk = min(len, budget):
// every entry gets a 32-bit key that orders as its score does (protected
// entries above all, with one key: which of them is first only matters where
// more of them than nk, at positions that repeat or are negative, leave no room
// for others; the cut then falls on that key, and the entries are keyed anew,
// the protected ones by score), the nk-th largest key K* is found by a radix select of
// 11 + 11 + 10 bits, and an entry stays iff key > K*, or key == K* and it is
// among the first (nk - #{key > K*}) such entries in slot order.  Slots below
// nk whose entry stays keep it; the r-th hole (ascending) takes the r-th
// survivor from slot nk on (ascending).  Sources lie at or past nk and
// destinations below it, so the move is free of hazards in place, and a step
// that evicts one entry moves one row.
//
// select_kernel is bound by its passes over the slots of one head and by the
// block-wide steps between them, so a head is split over a cluster of up to 8
// CTAs (16 no longer run side by side: 8 heads of 131072 slots 54 -> 73 us):
// each keeps its slice's keys in shared memory, and histograms, counts and
// ranks are combined through distributed shared memory, a few words per CTA
// (sums of 64 bins first, then one group's bins).  Scores and positions are
// read from DRAM once.  Every warp owns a contiguous run of slots for the tie
// ranks; holes and survivors are ranked from one bit per slot, a word per thread,
// and a survivor finds its hole's slot in the shared memory of the CTA that has it.
// move_kernel is a gather of 2d-byte rows: 16 bytes per lane, K and V rows of
// several slots in flight per warp; bound by DRAM.
// Measured on one B200 (device time): 32 caches of up to 5001 entries down to
// 4096, 8 heads, d = 128: 152 us, 6.0 TB/s (floor 139); a 128K prefill down to
// 16384: 53 us (22), about half of it the selection (two radix rounds of 4 us,
// the keys 6, ranks and lists 7); one entry of 1025: 5.6 us, all latency.
#include <climits>
#include <cooperative_groups.h>

#include "internal.h"
#include "sm100.cuh"

namespace psa {
namespace {

namespace cg = cooperative_groups;

constexpr int kBins = 2048;
constexpr int kSmemKeys = 32768;  // keys of a slice kept on chip (128 KB); a longer slice is read again per pass
constexpr int kMaxThreads = 1024;
constexpr uint32_t kSafe = 0xffffffffu;  // key of a protected entry (+inf has 0xff800000)
constexpr uint32_t kBehind = 1u;         // of any other, where the protected ones rank by score (-inf has 0x007fffff)

struct SelectParams {
  const float* score;
  const int* pos;        // null: the slot index
  const int* cache_len;  // null: C
  int* kept;             // [B * Hkv][budget]
  int* holes;            // scratch [B * Hkv][budget] where the keys are not on chip: the holes, ascending
  int* nk_out;           // scratch [B]
  int* status;
  int B, Hkv, C, budget, sink, recent;
  int slice;             // slots per CTA, a multiple of 32 * warps
  int keys_on_chip, pos_on_chip;
};

// Order-preserving key of a score: NaN as the lowest (-inf), -0 as +0.
__device__ __forceinline__ uint32_t score_key(float f) {
  if (f != f) f = -INFINITY;
  const uint32_t b = __float_as_uint(f + 0.0f);
  return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}

// Exclusive prefix over the block's warps of two warp-uniform counts, and the
// block's totals.  `buf` holds 33 pairs.
__device__ __forceinline__ int2 warps_exclusive(int2* buf, int2 mine, int2& total) {
  const int warp = uniform(threadIdx.x >> 5), lane = threadIdx.x & 31, warps = blockDim.x >> 5;
  __syncthreads();
  if (lane == 0) buf[warp] = mine;
  __syncthreads();
  __syncwarp();
  // every warp scans for itself: no third barrier
  int2 v = lane < warps ? buf[lane] : make_int2(0, 0), s = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int ux = __shfl_up_sync(0xffffffffu, s.x, o), uy = __shfl_up_sync(0xffffffffu, s.y, o);
    if (lane >= o) {
      s.x += ux;
      s.y += uy;
    }
  }
  total = make_int2(__shfl_sync(0xffffffffu, s.x, 31), __shfl_sync(0xffffffffu, s.y, 31));
  return make_int2(__shfl_sync(0xffffffffu, s.x - v.x, warp), __shfl_sync(0xffffffffu, s.y - v.y, warp));
}

// Shared by the cluster's CTAs (each reads the others').
struct SelectShared {
  uint32_t hist[3][kBins];  // one per round: nothing is cleared while it may still be read
  uint32_t coarse[3][32];   // sums of 64 bins
  int2 count[2];            // totals of a CTA (or its lowest key and slot), one per exchange
  int last;                 // latest position
};

// CL: the head is split over a cluster; else one CTA has it all and the
// cluster's barriers are the block's.
template <bool CL>
__global__ void __launch_bounds__(kMaxThreads, 1) select_kernel(const SelectParams p) {
  extern __shared__ __align__(16) uint32_t smem[];
  __shared__ __align__(16) SelectShared sh;
  __shared__ int2 buf[33];
  __shared__ uint32_t pick[3];  // chosen bin, keys above it, keys in it
  __shared__ int hole_count[8]; // of each CTA
  cg::cluster_group cl = cg::this_cluster();
  const int rank = CL ? static_cast<int>(cl.block_rank()) : 0;
  const int ncta = CL ? static_cast<int>(cl.num_blocks()) : 1;
  auto sync_all = [&]() {
    if constexpr (CL) {
      cl.sync();
    } else {
      __syncthreads();
    }
  };
  auto peer = [&](int r) -> const SelectShared* { return CL ? cl.map_shared_rank(&sh, r) : &sh; };
  const int bh = blockIdx.x / ncta;
  const int b = bh / p.Hkv;
  const int tid = threadIdx.x, lane = tid & 31, warp = uniform(tid >> 5), nthr = blockDim.x;
  const int words = p.slice >> 5;
  uint32_t* stay = smem;                                  // one bit per slot of the slice
  int2* rank_at = reinterpret_cast<int2*>(smem + words);  // holes and late survivors before each word
  uint32_t* keys = smem + 3 * words;                      // the slice's keys (when they fit), 0 past its end
  for (int i = tid; i < 3 * kBins / 4; i += nthr) reinterpret_cast<uint4*>(&sh.hist[0][0])[i] = make_uint4(0, 0, 0, 0);
  grid_dep_launch();
  grid_dep_wait();

  int len = p.cache_len ? p.cache_len[b] : p.C;
  len = uniform(min(max(len, 0), p.C));
  if (blockIdx.x == 0) {
    // one writer of the status word: the lengths of all sequences
    bool bad = false;
    if (p.cache_len)
      for (int i = tid; i < p.B; i += nthr) {
        const int n = p.cache_len[i];
        bad |= n < 0 || n > p.C;
      }
    bad = __syncthreads_or(bad);
    if (tid == 0) *p.status = bad ? kStatusLength : 0;
  }
  const int nk = min(len, p.budget);
  if (rank == 0 && bh % p.Hkv == 0 && tid == 0) p.nk_out[b] = nk;
  int* kept = p.kept + static_cast<long long>(bh) * p.budget;
  const float* score = p.score + static_cast<long long>(bh) * p.C;
  const int* pos = p.pos ? p.pos + static_cast<long long>(bh) * p.C : nullptr;

  for (int i = nk + rank * nthr + tid; i < p.budget; i += ncta * nthr) kept[i] = -1;
  if (len <= p.budget) {  // the same for the whole cluster
    for (int i = rank * nthr + tid; i < nk; i += ncta * nthr) kept[i] = i;
    return;
  }

  // ---- keys, and the latest position of the head
  const int s0 = rank * p.slice, s1 = min(s0 + p.slice, len);
  const bool guarded = pos && p.recent > 0;
  int last = len - 1;
  int* spos = reinterpret_cast<int*>(keys + p.slice);  // positions next to the keys (pos_on_chip)
  if (guarded) {
    last = INT_MIN;
    if (p.pos_on_chip) {
#pragma unroll 8
      for (int i = s0 + tid; i < s1; i += nthr) {
        const int at = pos[i];
        const float f = score[i];
        spos[i - s0] = at;
        keys[i - s0] = score_key(f);
        last = max(last, at);
      }
    } else {
#pragma unroll 8
      for (int i = s0 + tid; i < s1; i += nthr) last = max(last, pos[i]);
    }
    __syncwarp();
    last = __reduce_max_sync(0xffffffffu, last);
    if (lane == 0) buf[warp].x = last;
    __syncthreads();
    __syncwarp();
    last = __reduce_max_sync(0xffffffffu, lane < (nthr >> 5) ? buf[lane].x : INT_MIN);
    if constexpr (CL) {
      if (tid == 0) sh.last = last;
      cl.sync();
      __syncwarp();
      last = __reduce_max_sync(0xffffffffu, lane < ncta ? peer(lane)->last : INT_MIN);
    }
  }
  // positions after `last - recent` are protected; 64 bits, so that no
  // position a caller stores can wrap it
  const long long guard = p.recent > 0 ? static_cast<long long>(last) - p.recent : LLONG_MAX;
  bool scored = false;  // more entries are protected than stay: they rank by score
  auto make_key = [&](int i) -> uint32_t {
    const int at = pos ? pos[i] : i;
    const uint32_t k = score_key(score[i]);
    const bool safe = at < p.sink || at > guard;
    return scored ? (safe ? k : kBehind) : (safe ? kSafe : k);
  };
  if (guarded && p.pos_on_chip) {
    for (int i = tid; i < s1 - s0; i += nthr)
      if (spos[i] < p.sink || spos[i] > guard) keys[i] = kSafe;
  } else if (p.keys_on_chip) {
#pragma unroll 8
    for (int i = s0 + tid; i < s1; i += nthr) keys[i - s0] = make_key(i);
  }
  // (no entry has key 0: the lowest score, -inf, has 0x007fffff)
  if (p.keys_on_chip)
    for (int i = max(s1 - s0, 0) + tid; i < p.slice; i += nthr) keys[i] = 0u;
  auto key = [&](int i) -> uint32_t { return p.keys_on_chip ? keys[i - s0] : (i < s1 ? make_key(i) : 0u); };
  auto score_safe = [&]() {
    scored = true;
    if (p.keys_on_chip)
      for (int i = tid; i < s1 - s0; i += nthr)
        keys[i] = keys[i] == kSafe ? score_key(score[s0 + i]) : kBehind;
  };
  __syncthreads();

  if (len - nk == 1) {
    // ---- one entry goes (a decode step at its budget): the lowest key, of
    // equal ones the last; slot nk takes its place.  One reduction instead of
    // three rounds and the ranks: a call on 1025 entries 11.7 -> 5.6 us.
    uint32_t hi, lo;  // key, ~slot
    auto lowest = [&]() {
      const uint32_t k = __reduce_min_sync(0xffffffffu, hi);
      lo = __reduce_min_sync(0xffffffffu, hi == k ? lo : 0xffffffffu);
      hi = k;
    };
    auto give = [&](int2 v, bool there) {
      hi = there ? static_cast<uint32_t>(v.x) : 0xffffffffu;
      lo = there ? static_cast<uint32_t>(v.y) : 0xffffffffu;
    };
#pragma unroll 1
    for (;;) {
      hi = lo = 0xffffffffu;
#pragma unroll 4
      for (int i = s0 + tid; i < s1; i += nthr) {
        const uint32_t k = key(i);
        if (k <= hi) hi = k, lo = ~static_cast<uint32_t>(i);
      }
      __syncwarp();
      lowest();
      if (lane == 0) buf[warp] = make_int2(static_cast<int>(hi), static_cast<int>(lo));
      __syncthreads();
      __syncwarp();
      give(lane < (nthr >> 5) ? buf[lane] : make_int2(0, 0), lane < (nthr >> 5));
      lowest();
      if constexpr (CL) {
        if (tid == 0) sh.count[scored] = make_int2(static_cast<int>(hi), static_cast<int>(lo));
        cl.sync();
        __syncwarp();
        give(lane < ncta ? peer(lane)->count[scored] : make_int2(0, 0), lane < ncta);
        lowest();
      }
      if (uniform(scored || hi != kSafe)) break;
      score_safe();     // every entry is protected
      __syncthreads();  // `buf` has been read
    }
    const int gone = static_cast<int>(~lo);
    for (int i = s0 + tid; i < min(s1, nk); i += nthr) kept[i] = i == gone ? nk : i;
    if constexpr (CL) cl.sync();  // the others' shared memory has been read
    return;
  }

  // ---- radix select of the nk-th largest key
  // After a round whose bin is needed whole, the bits so far decide.
  uint32_t prefix = 0, need = static_cast<uint32_t>(nk), equal = 0;
  int shift = 0;
#pragma unroll 1
  for (int round = 0; round < 3 && need != equal; ++round) {
    shift = round == 0 ? 21 : (round == 1 ? 10 : 0);
    const int bits = round == 2 ? 10 : 11;
    const uint32_t mask = (1u << bits) - 1u;
    uint32_t* hist = sh.hist[round];
    // four keys per thread and step
#pragma unroll 2
    for (int it = tid; it < p.slice / 4; it += nthr) {
      uint32_t k[4];
      if (p.keys_on_chip) {
        const uint4 q = reinterpret_cast<const uint4*>(keys)[it];
        k[0] = q.x, k[1] = q.y, k[2] = q.z, k[3] = q.w;
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) k[j] = key(s0 + 4 * it + j);
      }
      bool in[4], one = true;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        in[j] = k[j] != 0u && (round == 0 || (k[j] >> (shift + bits)) == prefix);
        k[j] = (k[j] >> shift) & mask;
        one = one && in[j] && k[j] == k[0];
      }
      // a warp whose keys share one bin (equal scores) adds once
      const uint32_t lead = static_cast<uint32_t>(uniform(k[0]));  // (all lanes take part)
      one = one && k[0] == lead;
      if (__all_sync(0xffffffffu, one)) {
        if (lane == 0) atomicAdd(&hist[k[0]], 128u);
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (in[j]) atomicAdd(&hist[k[j]], 1u);
      }
    }
    __syncthreads();
    for (int c = warp; c < 32; c += nthr >> 5) {
      const uint2 h = reinterpret_cast<const uint2*>(hist)[32 * c + lane];
      __syncwarp();
      const uint32_t n = __reduce_add_sync(0xffffffffu, h.x + h.y);
      if (lane == 0) sh.coarse[round][c] = n;
      __syncwarp();
    }
    sync_all();
    __syncwarp();
    if (warp == 0) {
      // the group of 64 bins in which the count from the top passes `need`,
      // then the bin: two reads of every CTA, a few words each
      uint32_t n = 0, above = 0;
      int c = 31 - lane;
#pragma unroll
      for (int r = 0; r < (CL ? 8 : 1); ++r)
        if (r < ncta) n += peer(r)->coarse[round][c];
      uint32_t inc = n;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const uint32_t u = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += u;
      }
      int owner = __ffs(__ballot_sync(0xffffffffu, inc >= need)) - 1;
      above = __shfl_sync(0xffffffffu, inc - n, owner);
      c = __shfl_sync(0xffffffffu, c, owner);
      // lane l: the bins 64 c + 63 - 2 l (first) and the one below it
      uint32_t hi = 0, lo = 0;
#pragma unroll
      for (int r = 0; r < (CL ? 8 : 1); ++r)
        if (r < ncta) {
          const uint2 h = reinterpret_cast<const uint2*>(peer(r)->hist[round])[32 * c + 31 - lane];
          hi += h.y;
          lo += h.x;
        }
      n = hi + lo;
      inc = n;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const uint32_t u = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += u;
      }
      owner = __ffs(__ballot_sync(0xffffffffu, above + inc >= need)) - 1;
      if (lane == owner) {
        above += inc - n;
        const bool first = above + hi >= need;
        pick[0] = static_cast<uint32_t>(64 * c + 63 - 2 * lane - (first ? 0 : 1));
        pick[1] = first ? above : above + hi;
        pick[2] = first ? hi : lo;
      }
    }
    __syncthreads();
    __syncwarp();
    prefix = (prefix << bits) | static_cast<uint32_t>(uniform(pick[0]));
    need -= static_cast<uint32_t>(uniform(pick[1]));
    equal = static_cast<uint32_t>(uniform(pick[2]));
    // (the next round's barriers keep `pick` until all have read)
    if (round == 0 && !scored && prefix == kSafe >> 21 && need < equal) {
      // more protected entries than nk: once more, with the keys of that case
      sync_all();  // all have read the histograms
      score_safe();
      for (int i = tid; i < kBins; i += nthr) sh.hist[0][i] = 0u;
      prefix = 0, need = static_cast<uint32_t>(nk), equal = 0, round = -1;
      __syncthreads();
    }
  }
  // prefix is K* (its bits from `shift` on); of the `equal` entries with them
  // the first `need` stay

  // ---- which entries stay; each warp owns the slots [w0, w1)
  const int per_warp = p.slice / (nthr >> 5);
  const int w0 = min(s0 + warp * per_warp, s1), w1 = min(w0 + per_warp, s1);
  int2 total;
  int eq_at = 0;
  if (need < equal) {  // the same everywhere: ties are cut, so they are ranked
    int eq = 0;
    for (int i = w0 + lane; i - lane < w1; i += 32) {
      const bool tie = i < w1 && key(i) >> shift == prefix;
      __syncwarp();
      eq += __popc(__ballot_sync(0xffffffffu, tie));
    }
    __syncwarp();
    eq_at = warps_exclusive(buf, make_int2(eq, 0), total).x;
    if constexpr (CL) {
      if (tid == 0) sh.count[0] = total;
      cl.sync();
      __syncwarp();
      for (int r = 0; r < rank; ++r) eq_at += peer(r)->count[0].x;
    }
  }
  // slots of a word (32 from i0 on) below x
  auto below = [](int x, int i0) -> uint32_t {
    return x >= i0 + 32 ? 0xffffffffu : (x <= i0 ? 0u : (1u << (x - i0)) - 1u);
  };
  const bool cut = need < equal;
#pragma unroll 2
  for (int i0 = w0; i0 < w1; i0 += 32) {
    const uint32_t k = key(i0 + lane) >> shift;
    bool in = k >= prefix;
    if (cut) {
      const uint32_t tie = __ballot_sync(0xffffffffu, k == prefix);
      in = in && (k > prefix || eq_at + __popc(tie & ((1u << lane) - 1u)) < static_cast<int>(need));
      eq_at += __popc(tie);
    }
    const uint32_t word = __ballot_sync(0xffffffffu, in);
    if (lane == 0) stay[(i0 - s0) >> 5] = word;
  }
  // ranks of the holes and of the late survivors, a word per thread
  int2 base = make_int2(0, 0);
  const int have = (max(s1 - s0, 0) + 31) >> 5;
  for (int w = 0; w < have; w += nthr) {
    int2 n = make_int2(0, 0), total;
    if (w == 0) __syncthreads();  // all of stay[] is there
    if (w + tid < have) {
      const uint32_t word = stay[w + tid], all = below(s1, s0 + 32 * (w + tid)), early = below(nk, s0 + 32 * (w + tid));
      n.x = __popc(all & early & ~word);
      n.y = __popc(word & ~early);
    }
    int2 inc = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int ux = __shfl_up_sync(0xffffffffu, inc.x, o), uy = __shfl_up_sync(0xffffffffu, inc.y, o);
      if (lane >= o) {
        inc.x += ux;
        inc.y += uy;
      }
    }
    const int2 warp_total =
        make_int2(__shfl_sync(0xffffffffu, inc.x, 31), __shfl_sync(0xffffffffu, inc.y, 31));
    const int2 before = warps_exclusive(buf, warp_total, total);
    if (w + tid < have)
      rank_at[w + tid] = make_int2(base.x + before.x + inc.x - n.x, base.y + before.y + inc.y - n.y);
    base.x += total.x;
    base.y += total.y;
  }
  int2 first = make_int2(0, 0);
  if constexpr (CL) {
    if (tid == 0) sh.count[1] = base;
    cl.sync();
    if (tid < ncta) hole_count[tid] = peer(tid)->count[1].x;
    for (int r = 0; r < rank; ++r) {
      const int2 c = peer(r)->count[1];
      first.x += c.x;
      first.y += c.y;
    }
  } else {
    __syncthreads();
  }
  // The holes' slots, ascending, take the keys' place (all of them are read).
  int* holes = p.holes + static_cast<long long>(bh) * p.budget;
  int* mine = p.keys_on_chip ? reinterpret_cast<int*>(keys) : holes + first.x;
#pragma unroll 2
  for (int i0 = w0; i0 < min(w1, nk); i0 += 32) {
    const int w = (i0 - s0) >> 5;
    const uint32_t word = stay[w], early = below(min(nk, w1), i0), bit = 1u << lane;
    const uint32_t open = early & ~word;
    if (open & bit) mine[rank_at[w].x + __popc(open & (bit - 1u))] = i0 + lane;
    if (word & early & bit) kept[i0 + lane] = i0 + lane;
  }
  sync_all();
  // the r-th late survivor goes to the r-th hole
#pragma unroll 2
  for (int i0 = max(w0, nk & ~31); i0 < w1; i0 += 32) {
    const int w = (i0 - s0) >> 5;
    const uint32_t far = stay[w] & ~below(nk, i0), bit = 1u << lane;
    if (far & bit) {
      int at = first.y + rank_at[w].y + __popc(far & (bit - 1u));
      if (!p.keys_on_chip) {
        at = __ldcg(holes + at);
      } else if constexpr (CL) {
        int r = 0;
        for (; r < ncta - 1 && at >= hole_count[r]; ++r) at -= hole_count[r];
        at = cl.map_shared_rank(mine, r)[at];
      } else {
        at = mine[at];
      }
      kept[at] = i0 + lane;
    }
  }
  if constexpr (CL) cl.sync();  // the others' shared memory has been read
}

struct MoveParams {
  const uint4* k;
  const uint4* v;
  const float* score;
  const int* pos;
  const int* kept;
  const int* nk;
  uint4* k_out;
  uint4* v_out;
  float* score_out;
  int* pos_out;
  int* len_out;
  int B, Hkv, C, C_out, budget;
  int in_place, chunks;
};

constexpr int kMoveThreads = 256;
constexpr int kMoveSlots = 64;  // slots per CTA: 8 per warp, K and V rows 16 bytes per lane

template <int D>
__global__ void __launch_bounds__(kMoveThreads) move_kernel(const MoveParams p) {
  constexpr int kLanes = D / 8;           // 16-byte pieces of a row
  constexpr int kRows = 32 / kLanes;      // rows per warp-wide access
  constexpr int kPerWarp = kMoveSlots / (kMoveThreads / 32);
  constexpr int kSteps = kPerWarp / kRows;
  grid_dep_launch();
  grid_dep_wait();
  const int bh = blockIdx.x / p.chunks, chunk = blockIdx.x - bh * p.chunks;
  const int slot0 = chunk * kMoveSlots;
  const int* kept = p.kept + static_cast<long long>(bh) * p.budget;
  const long long in0 = static_cast<long long>(bh) * p.C, out0 = static_cast<long long>(bh) * p.C_out;
  if (chunk == 0 && bh % p.Hkv == 0 && threadIdx.x == 0) p.len_out[bh / p.Hkv] = p.nk[bh / p.Hkv];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int sub = lane / kLanes, piece = lane % kLanes;
  int src[kSteps];
  uint4 kr[kSteps], vr[kSteps];
#pragma unroll
  for (int j = 0; j < kSteps; ++j) {
    const int i = slot0 + warp * kPerWarp + j * kRows + sub;
    src[j] = i < p.budget ? kept[i] : -1;
    if (p.in_place && src[j] == i) src[j] = -1;
  }
#pragma unroll
  for (int j = 0; j < kSteps; ++j)
    if (src[j] >= 0) {
      kr[j] = p.k[(in0 + src[j]) * kLanes + piece];
      vr[j] = p.v[(in0 + src[j]) * kLanes + piece];
    }
#pragma unroll
  for (int j = 0; j < kSteps; ++j)
    if (src[j] >= 0) {
      const long long o = (out0 + slot0 + warp * kPerWarp + j * kRows + sub) * kLanes + piece;
      p.k_out[o] = kr[j];
      p.v_out[o] = vr[j];
    }
  if (threadIdx.x < kMoveSlots) {
    const int i = slot0 + threadIdx.x;
    const int s = i < p.budget ? kept[i] : -1;
    if (s >= 0) {
      // in place a slot that stays still needs its position when none came in
      if (!(p.in_place && s == i)) p.score_out[out0 + i] = p.score[in0 + s];
      if (!(p.in_place && p.pos && s == i)) p.pos_out[out0 + i] = p.pos ? p.pos[in0 + s] : s;
    }
  }
}

}  // namespace

cudaError_t launch_evict(const EvictLaunch& a, cudaStream_t st) {
  SelectParams s = {};
  s.score = a.score;
  s.pos = a.pos;
  s.cache_len = a.cache_len;
  s.kept = a.kept;
  s.holes = a.holes;
  s.nk_out = a.nk;
  s.status = a.status;
  s.B = a.B;
  s.Hkv = a.Hkv;
  s.C = a.C;
  s.budget = a.budget;
  s.sink = a.sink;
  s.recent = a.recent;
  // CTAs per head: slices of about 8192 slots, while the heads alone do not
  // fill the machine (a cluster costs its barriers); 8 is the portable limit
  const long long heads = static_cast<long long>(a.B) * a.Hkv;
  int ncta = 1;
  while (ncta < 8 && a.C > 8192 * ncta && heads * ncta * 2 <= 296) ncta *= 2;
  while (ncta < 8 && (a.C + ncta - 1) / ncta > kSmemKeys) ncta *= 2;
  const int part = (a.C + ncta - 1) / ncta;
  // four slots or more per thread; two CTAs per SM when there are more heads than SMs
  int threads = heads * ncta > 148 ? kMaxThreads / 2 : kMaxThreads;
  while (threads > 128 && threads * 4 > part) threads /= 2;
  s.slice = (part + 4 * threads - 1) / (4 * threads) * 4 * threads;
  s.keys_on_chip = s.slice <= kSmemKeys;
  s.pos_on_chip = 2 * s.slice <= kSmemKeys;
  const size_t smem =
      static_cast<size_t>(3 * (s.slice / 32) + (s.keys_on_chip ? s.slice : 0) + (s.pos_on_chip ? s.slice : 0)) * 4;
  auto kernel = ncta > 1 ? select_kernel<true> : select_kernel<false>;
  cudaError_t e = cudaSuccess;
  if (smem > 20 * 1024) e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, 180 * 1024);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(heads * ncta));
  cfg.blockDim = dim3(static_cast<unsigned>(threads));
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = static_cast<unsigned>(ncta);
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = ncta > 1 ? 2 : 1;
  if ((e = cudaLaunchKernelEx(&cfg, kernel, s)) != cudaSuccess) return e;

  MoveParams m = {};
  m.k = reinterpret_cast<const uint4*>(a.k);
  m.v = reinterpret_cast<const uint4*>(a.v);
  m.score = a.score;
  m.pos = a.pos;
  m.kept = a.kept;
  m.nk = a.nk;
  m.k_out = reinterpret_cast<uint4*>(a.k_out);
  m.v_out = reinterpret_cast<uint4*>(a.v_out);
  m.score_out = a.score_out;
  m.pos_out = a.pos_out;
  m.len_out = a.len_out;
  m.B = a.B;
  m.Hkv = a.Hkv;
  m.C = a.C;
  m.C_out = a.C_out;
  m.budget = a.budget;
  m.in_place = a.k == a.k_out;
  m.chunks = (a.budget + kMoveSlots - 1) / kMoveSlots;
  const dim3 grid(static_cast<unsigned>(heads * m.chunks));
  return a.d == 128 ? launch_chained(move_kernel<128>, grid, dim3(kMoveThreads), 0, st, m)
                    : launch_chained(move_kernel<64>, grid, dim3(kMoveThreads), 0, st, m);
}

}  // namespace psa
