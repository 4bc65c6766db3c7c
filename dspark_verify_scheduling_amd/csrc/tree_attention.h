// Attention of packed verify rows (a chain or tree of drafts per request) over
// the paged cache: the split kernel's templates, one translation unit per head
// dimension, and the schedule it shares with the joining kernel.
#pragma once

#include "kv_dev.h"

namespace dspark {
namespace attn {

// What the split kernel leaves for the joining kernel: the schedule's prefix
// sums, and per partial segment the running maximum (less Types::kAbove) and sum of
// each of its rows and their unnormalised outputs. Workgroup w has segments 2 w (the one its
// range starts with) and 2 w + 1 (a later one that its range ends in).
struct Parts {
  int64_t* base;  // [B + 1] first unit of each request, then the total
  float* m;       // [2 * wgs][rows]
  float* l;
  float* o;       // [2 * wgs][rows][D]
  int wgs;        // workgroups of the split kernel
  int rows;       // rows of a segment, at most
};

// Waves of a workgroup, one to each 16-row tile of a segment: the more rows meet
// in a segment the fewer reads of its keys; with few rows in a request four
// waves do, and feed the tiles with less work around it (32 chains of 9 rows,
// 32 query heads on 8, 1k to 8k keys: 110 us against 125 with eight; 64 trees of
// up to 17 rows, 64 on 8, 8-bit: 245 us against 233).
constexpr int kMostWaves = 8, kFewWaves = 4;  // (shape_of() shifts by them)
// (Its share of a tile has to stay within a page: 16 keys.)
inline int waves_for(int rows, int dim) {
  return rows <= 16 * kFewWaves && dim >= 128 ? kFewWaves : kMostWaves;
}

// Keys of a unit.
template <int D>
struct Size {
  static constexpr int kKeys = D >= 128 ? 32 : 64;
};

// Rows of a (request, key/value head): m = j * group + g for row j and the g-th
// of the head's queries, in tiles of 16, several tiles to a segment.
struct Shape {
  int len, prefix, c0;
  int mrows, mtiles;
  int nseg, per;  // segments side by side, tiles of each
  int keys;
  int nku;        // units along the keys
};

// Whether a request's rows are well formed (its tree and pages apart); their
// place and its prefix.
__device__ inline bool rows_of(const AttnArgs& a, int r, int total_eff, int* c0, int* len,
                               int* prefix) {
  const bool ok = request_rows(a.req, r, total_eff, c0, len);
  *prefix = a.req.prefix[r];
  const int64_t keys = (int64_t)*prefix + *len;
  // (cache indices in 32 bits, a unit beyond included)
  return ok && *prefix >= 0 && keys <= ((int64_t)a.req.width << a.kv.page_shift) &&
         keys <= 0x7FFFFF00LL;
}

template <int D>
__device__ inline Shape shape_of(const AttnArgs& a, int c0, int len, int prefix) {
  constexpr int kK = Size<D>::kKeys;
  Shape s;
  s.c0 = c0;
  s.len = len;
  s.prefix = prefix;
  s.keys = prefix + len;
  s.mrows = a.group * len;
  s.mtiles = (s.mrows + 15) >> 4;
  s.nseg = (s.mtiles + a.waves - 1) >> (a.waves == kFewWaves ? 2 : 3);
  s.per = (s.mtiles + s.nseg - 1) / s.nseg;
  s.nku = (s.keys + kK - 1) / kK;
  return s;
}

template <int D>
__device__ inline int64_t units_of(const AttnArgs& a, int c0, int len, int prefix) {
  const Shape s = shape_of<D>(a, c0, len, prefix);
  return (int64_t)a.kv.hkv * s.nseg * s.nku;
}

// Workgroups that get units: never one without.
__device__ inline int wgs_in_use(int64_t total, int wgs) { return (int)min((int64_t)wgs, total); }

// Workgroups go to the eight XCDs in turn. Shares are numbered so that an XCD's
// are consecutive: the heads of a request and the segments of a head then meet
// in one L2, and an XCD's requests spread over the memory's channels (with share =
// workgroup and eight heads, each XCD read one head of all pages).
constexpr int kXcds = 8;
__device__ inline int share_of(int wg, int wgs) {
  return wgs % kXcds ? wg : wg % kXcds * (wgs / kXcds) + wg / kXcds;
}

// The first unit of share w of n <= total.
__device__ inline int64_t wg_start(int64_t total, int w, int n) { return total * w / n; }

// The weights of a row are 2^(score - m), m its running maximum (in log2) less
// kAbove. m follows the scores only when they pass it by kAbove + kSlack, so most
// steps rescale nothing, and the weights stay below 2^(kAbove + kSlack).
// bfloat16 has float32's exponents and needs no kAbove. float16 holds 2^15 to
// 2^-24: with kAbove a weight counts down to 2^-36 of the largest, 25 below it in
// e; with the largest at 1 it would end at 2^-25, and the tail of a long context
// under one large weight with it.
template <typename T>
struct Types;
template <>
struct Types<__bf16> {
  static constexpr float kSlack = 8.0f, kAbove = 0.0f;
  typedef bf16x8 V8;
  typedef bf16x4 V4;
  static constexpr unsigned kExpMask = 0x7F80u;
  static __device__ f32x4 mfma(V8 a, V8 b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
  }
};
template <>
struct Types<_Float16> {
  static constexpr float kSlack = 4.0f, kAbove = 11.0f;
  typedef f16x8 V8;
  typedef f16x4 V4;
  static constexpr unsigned kExpMask = 0x7C00u;
  static __device__ f32x4 mfma(V8 a, V8 b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
  }
};

typedef __attribute__((address_space(3))) unsigned char lds_u8;

// Four rows of sixteen 16-bit elements, transposed: with the 16 lanes of a
// group pointing at the rows' quarters in order, lane i gets column i.
template <typename V4>
__device__ inline V4 lds_columns(unsigned at) {
  typedef __attribute__((ext_vector_type(4))) short s16x4;
  typedef __attribute__((address_space(3))) s16x4 lds_s16x4;
  return __builtin_bit_cast(V4, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(uintptr_t)at));
}

template <typename X>
__device__ inline X lds_read(unsigned at) {
  return *(__attribute__((address_space(3))) const X*)(uintptr_t)at;
}
template <typename X>
__device__ inline void lds_write(unsigned at, X x) {
  *(__attribute__((address_space(3))) X*)(uintptr_t)at = x;
}

// Memory straight into LDS, 16 (or 4) bytes a lane at lds_at + 16 (4) * lane.
// `from` and `lds_at` are wave-uniform; M0 holds lds_at (nothing else here uses
// it). As inline assembly, the compiler's waits do not see the copies: its own
// waits for loads only become more conservative by them, and wait_copies()
// waits for the copies.
__device__ inline void copy16(const unsigned char* from, unsigned lane_bytes, unsigned lds_at) {
  asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, %1 nt"
               :
               : "v"(lane_bytes), "s"(from), "s"(__builtin_amdgcn_readfirstlane((int)lds_at))
               : "memory");
}
__device__ inline void copy4(const unsigned char* from, unsigned lane_bytes, unsigned lds_at) {
  asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tglobal_load_lds_dword %0, %1"
               :
               : "v"(lane_bytes), "s"(from), "s"(__builtin_amdgcn_readfirstlane((int)lds_at))
               : "memory");
}
// A loaded value has arrived here. Without it, the wait for a load from before
// a loop stands at its first use inside, and there waits for the copies of
// every step.
template <typename X>
__device__ inline void settle(X& x) {
  asm volatile("" : "+v"(x));
}
// All but the last `N` loads of the wave are done (they end in order).
template <int N>
__device__ inline void wait_copies() {
  static_assert(N >= 0 && N < 64, "the counter's width");
  asm volatile("s_waitcnt vmcnt(%0)" : : "n"(N) : "memory");
}
__device__ inline void barrier() {
  asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" : : : "memory");
}

template <typename X>
__device__ inline X* uniform(X* p) {
  const uint64_t u = (uint64_t)p;
  return (X*)(((uint64_t)(unsigned)__builtin_amdgcn_readfirstlane((int)(u >> 32)) << 32) |
              (unsigned)__builtin_amdgcn_readfirstlane((int)(unsigned)u));
}

__device__ inline float group_max(float x) {
  x = fmaxf(x, __shfl_xor(x, 16, kWave));
  return fmaxf(x, __shfl_xor(x, 32, kWave));
}

__device__ inline float group_sum(float x) {
  x += __shfl_xor(x, 16, kWave);
  return x + __shfl_xor(x, 32, kWave);
}

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

// Workgroups to a CU, by their LDS. Small ones over an 8-bit cache have fewer
// pieces under way and are three instead: the widening is latency (64 single
// tokens, 64 query heads on 8, up to 4k keys: 87 us against 113; over 16 bits, 112
// against 110).
constexpr int per_cu(int dim, bool e8, int waves) {
  return dim == 256 ? 1 : (e8 && waves == kFewWaves ? 3 : 2);
}

// LDS of a workgroup. A tile of keys and values in 16 bits is shared by its
// waves; rows are unpadded (copies into LDS write densely), and 16-byte chunk c
// of a row lies at chunk c ^ swizzle(row), so that the 16 rows which a wave reads
// at one column spread over all banks.
//   16-bit caches: a ring of kStages tiles, filled straight from memory.
//   8-bit caches: each wave has a ring of kStages pieces of codes and exponents
//   for itself, and widens its piece of the next tile into one of two tiles.
template <bool E8, int D, int W>
struct Ring {
  static constexpr int CB = E8 ? 1 : 2;
  static constexpr int kKeys = Size<D>::kKeys;
  static constexpr int kGroups = kKeys / 16;
  static constexpr int kRow = 2 * D;                  // bytes of a row of a tile
  static constexpr int kTile = kKeys * kRow;          // keys, or values
  static constexpr int kTiles = 2 * kTile;            // both
  // a wave's share of a tile: kRows keys (the first half of the waves) or values
  // (the second), in copies of kWave 16-byte chunks
  static constexpr int kRows = kKeys / (W / 2);
  static constexpr int kChunks = D * CB / 16;         // of a cache row
  static constexpr int kRowsPerCopy = kWave / kChunks;
  static constexpr int kCopies = kRows / kRowsPerCopy;
  static_assert(kCopies * kRowsPerCopy == kRows, "whole copies");
  static_assert(kRows <= 16, "of one page");
  static constexpr int kPerWave = kCopies + (E8 ? 1 : 0);
  static constexpr int kPiece = kRows * D + 64;       // codes, exponents; 8 bits
  static constexpr int kRaw = 2 * kTiles;             // offset of the waves' rings
  // (what the LDS of a CU, or of half a CU, holds; even in an 8-bit ring)
  static constexpr int kStages =
      D == 256 ? 4 : (E8 ? (W == kFewWaves ? 2 : 4) : (65536 / kTiles < 4 ? 65536 / kTiles : 4));
  // rows with NaN or infinity, a bit each; of two tiles
  static constexpr int kOdd = E8 ? kRaw + kStages * W * kPiece : kStages * kTiles;
  static constexpr int kReqs = kOdd + 16;  // rows of up to kWave requests, 3 words each
  static constexpr int kBytes = kReqs + 12 * kWave;
  static constexpr int kPerCu = per_cu(D, E8, W);
  static_assert(kBytes <= 163840 / kPerCu - 256, "a CU's LDS");
  static_assert(!E8 || kStages % 2 == 0, "pieces go to the two tiles in turn");
  static __device__ int swizzle(int row) {
    return D >= 128 ? row & 15 : (row >> 1) & 7;
  }
};

// One segment: the queries of several 16-row tiles of one (request, key/value
// head) over some units of its keys. What the copies need of it,
struct Span {
  int r, h;
  int first;  // its first key
  int n;      // units; 0: there is no such segment
  int keys;   // of the request
};
// and the rest.
struct Job {
  Shape s;
  int tile0, mt;
  int slot;    // its place among the parts
  bool whole;  // it covers all the request's keys
};

// Where a wave is in its workgroup's share of the units.
struct Cursor {
  int64_t left;  // units of the share still to come
  int64_t off;   // next unit within request r
  int r;
  int share;
  int begun;     // 0 before the share's first segment
};

// The next segment of a share. `reqs`: the requests' rows in LDS where a wave's
// lanes hold the batch (len 0: malformed); otherwise they are read from memory.
template <int D>
__device__ __forceinline__ Span next_span(const AttnArgs& a, unsigned reqs, Cursor& c, Job* job) {
  Span j;
  j.n = 0;
  while (c.left > 0) {
    int c0 = 0, len = 0, prefix = 0;
    if (a.req.B <= kWave) {
      const unsigned at = reqs + 12 * c.r;
      c0 = lds_read<int>(at);
      len = lds_read<int>(at + 4);
      prefix = lds_read<int>(at + 8);
    } else {
      int total;
      const int total_eff = rows_in_use(a.req, &total);
      if (!rows_of(a, c.r, total_eff, &c0, &len, &prefix)) len = 0;
    }
    c0 = __builtin_amdgcn_readfirstlane(c0);
    len = __builtin_amdgcn_readfirstlane(len);
    prefix = __builtin_amdgcn_readfirstlane(prefix);
    const Shape s = shape_of<D>(a, c0, len, prefix);
    if (c.off >= (len ? (int64_t)a.kv.hkv * s.nseg * s.nku : 0)) {
      ++c.r;
      c.off = 0;
      continue;
    }
    const int item = __builtin_amdgcn_readfirstlane((int)(c.off / s.nku));
    const int ku0 = (int)(c.off - (int64_t)item * s.nku);
    j.r = c.r;
    j.n = (int)min((int64_t)(s.nku - ku0), c.left);
    j.h = item / s.nseg;
    j.first = ku0 * Size<D>::kKeys;
    j.keys = s.keys;
    if (job) {
      const int seg = item - j.h * s.nseg;
      job->s = s;
      job->tile0 = seg * s.per;
      job->mt = min(s.per, s.mtiles - job->tile0);
      job->whole = j.n == s.nku;
      job->slot = 2 * c.share + c.begun;
    }
    c.begun = 1;
    c.off += j.n;
    c.left -= j.n;
    break;
  }
  return j;
}

// The producing side of the ring: this wave's copies of the next tile. Few
// registers are kept for it: a reload of a spilled one would wait for every copy
// under way.
template <bool E8, int D, int W>
struct Feeder {
  typedef Ring<E8, D, W> R;
  typedef unsigned long long u64;
  Cursor c;
  Span j, nj;      // the segment copied from, and the one after it
  int t;           // its tile in lane 0 of `ids`
  int idx, end;    // next lane, lanes that hold a tile: 0 when nothing is left
  int ids, nids;   // pages of the wave's rows: of j from tile t on, of nj from its first
  u64 bad, nbad;   // bit l: some page of lane l's tile is none
  int stage;
  unsigned none;   // bit per stage: some page of its tile is none

  // The pages of 64 tiles from tile t on, a tile to a lane.
  static __device__ int fetch(const AttnArgs& a, const Span& x, int t, int wave, u64* bad) {
    const int group = ((wave & (W / 2 - 1)) * R::kRows) >> 4;
    int own = 0;
    const int64_t first = (int64_t)x.first + (int64_t)(t + lane_id()) * R::kKeys;
    int id[R::kGroups];
#pragma unroll
    for (int g = 0; g < R::kGroups; ++g)
      id[g] = a.req.table[(size_t)x.r * a.req.width +
                          ((int)min(first + g * 16, (int64_t)x.keys - 1) >> a.kv.page_shift)];
    u64 b = 0;
#pragma unroll
    for (int g = 0; g < R::kGroups; ++g) {
      const bool none = id[g] < 0 || id[g] >= a.kv.num_blocks;
      b |= __ballot(none);
      // a page that is none: any valid one, its keys are masked
      if (g == group) own = none ? 0 : id[g];
    }
    *bad = b;
    settle(own);
    return own;
  }

  __device__ void start(const AttnArgs& a, unsigned lds, const Cursor& from, int wave) {
    c = from;
    j = next_span<D>(a, lds + R::kReqs, c, nullptr);
    ids = fetch(a, j, 0, wave, &bad);
    nj = next_span<D>(a, lds + R::kReqs, c, nullptr);
    nids = 0;
    nbad = 0;
    if (nj.n > 0) nids = fetch(a, nj, 0, wave, &nbad);
    t = idx = stage = 0;
    end = min(j.n, kWave);
    none = 0;
  }

  // Starts the wave's copies of the next tile.
  __device__ __forceinline__ void next(const AttnArgs& a, unsigned lds, int wave) {
    if (end == 0) return;
    const int lane = lane_id();
    const bool values = wave >= W / 2;
    const int row0 = (wave & (W / 2 - 1)) * R::kRows;
    const int id = __builtin_amdgcn_readlane(ids, idx);
    const int key = j.first + (t + idx) * R::kKeys + row0;
    const int64_t row =
        ((int64_t)j.h << a.kv.page_shift) + (key & ((1 << a.kv.page_shift) - 1));
    const unsigned char* from =
        (values ? a.kv.v : a.kv.k) + id * a.kv.page_bytes + row * (D * R::CB);
    const unsigned to = E8 ? lds + R::kRaw + (stage * W + wave) * R::kPiece
                           : lds + stage * R::kTiles + (values ? R::kTile : 0) + row0 * R::kRow;
#pragma unroll
    for (int n = 0; n < R::kCopies; ++n) {
      // 16 bits: as rows of a tile
      const int r = row0 + n * R::kRowsPerCopy + lane / R::kChunks;
      const int chunk = E8 ? lane % R::kChunks : (lane % R::kChunks) ^ R::swizzle(r);
      copy16(uniform(from) + n * R::kRowsPerCopy * D * R::CB,
             (lane / R::kChunks) * D * R::CB + (unsigned)chunk * 16, to + n * 1024);
    }
    if constexpr (E8) {
      const unsigned char* e = (values ? a.kv.vs : a.kv.ks) + id * a.kv.scale_page_bytes + row;
      if (lane < R::kRows / 4) copy4(uniform(e), lane * 4, to + R::kRows * D);
    }
    if (__builtin_expect((bad | none) != 0, 0))
      none = (none & ~(1u << stage)) | ((unsigned)(bad >> idx) & 1u) << stage;
    stage = stage + 1 == R::kStages ? 0 : stage + 1;
    if (__builtin_expect(++idx == end, 0)) {
      t += end;
      idx = 0;
      if (t < j.n) {
        ids = fetch(a, j, t, wave, &bad);
      } else {
        j = nj;
        ids = nids;
        bad = nbad;
        t = 0;
        if (j.n > 0) {
          nj = next_span<D>(a, lds + R::kReqs, c, nullptr);
          if (nj.n > 0) nids = fetch(a, nj, 0, wave, &nbad);
        }
      }
      end = min(j.n - t, kWave);
    }
  }
};

// A wave's part of a segment: its 16-row tile (ROWS false: none, the wave only
// feeds the ring) over all its keys, which the waves bring into LDS together.
// The products are
//   S^T = K Q^T: keys are its rows and queries its columns, so a lane holds the
//   scores of one query (lane & 15) for four keys of each sixteen, which are in
//   place as the operand of  O^T = V^T P^T.
template <typename T, bool E8, int D, int W, bool ROWS>
__device__ __forceinline__ void segment(const AttnArgs& a, const Parts& ws, const Span& span,
                                        const Job& job, Feeder<E8, D, W>& feed, unsigned lds,
                                        int left, int& stage) {
  typedef Types<T> TT;
  typedef typename TT::V8 V8;
  typedef typename TT::V4 V4;
  typedef Ring<E8, D, W> R;
  constexpr int NF = D / 32;         // operand chunks of a key
  constexpr int ND = D / 16;         // 16-column tiles of the output
  constexpr int NG = R::kGroups;     // 16-key groups of a tile
  const Shape& s = job.s;
  const int lane = lane_id(), qi = lane & 15, g = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int len = s.len, prefix = s.prefix, keys = s.keys;
  const SmallDiv by_group(a.group);
  const int m = (job.tile0 + wave) * 16 + qi;
  const int qrow = by_group.quo(m);  // the request's row that the lane's query belongs to
  const bool live = ROWS && m < s.mrows;

  // rows of the step's own tree that the lane's query sees, bit l for row l + 1;
  // row 0 is everybody's. Bit l of anc, in lane l, is row l + 1 itself, with its
  // ancestors' bits.
  unsigned long long seen = qrow >= 64 ? ~0ull : (1ull << qrow) - 1;
  if (ROWS && a.req.parents) {
    int up = lane + 1 < len ? a.req.parents[(size_t)span.r * a.req.gamma + lane] : 0;
    unsigned long long anc = 1ull << lane;
    for (int i = 0; i < 6; ++i) {
      const int from = max(up - 1, 0);
      const unsigned long long more = __shfl(anc, from, kWave);
      const int next = __shfl(up, from, kWave);
      if (up > 0) {
        anc |= more;
        up = next;
      }
    }
    const unsigned long long path = __shfl(anc, max(qrow - 1, 0) & 63, kWave);
    seen = qrow > 0 ? path : 0;
  }
  // Scores in units of log2 with a positive factor, so that a masked score stays
  // -infinity under it: the scale's sign and its zero go into the queries.
  float sl = fminf(fabsf(a.scale) * kLog2e, 3.4028235e38f);
  const bool flat = sl == 0.0f;
  if (flat) sl = 1.0f;
  const unsigned sign = a.scale < 0.0f ? 0x80008000u : 0u;
  // queries as operands
  V8 qf[NF];
  f32x4 o[ND];
  float mx = -__builtin_inff(), l = 0.0f;
  {
    const unsigned char* src = a.q + (size_t)(s.c0 + qrow) * a.q_ld +
                               ((size_t)(span.h * a.group + (m - qrow * a.group)) * D + g * 8) * 2;
    kv_u32x4 w[NF];
#pragma unroll
    for (int f = 0; f < NF; ++f) {
      w[f] = (kv_u32x4){0, 0, 0, 0};
      if (live && !flat) w[f] = *reinterpret_cast<const kv_u32x4*>(src + f * 64) ^ sign;
    }
#pragma unroll
    for (int f = 0; f < NF; ++f) {
      settle(w[f]);
      qf[f] = __builtin_bit_cast(V8, w[f]);
    }
#pragma unroll
    for (int d = 0; d < ND; ++d) o[d] = (f32x4){0, 0, 0, 0};
  }

  // lane's offsets in a tile: its chunk of a key, its piece of a value row
  const int key_at = qi * R::kRow + ((g ^ R::swizzle(qi)) << 4);
  const int vrow = g * 4 + (qi >> 2);
  const int val_at = R::kTile + vrow * R::kRow + ((((qi >> 1) & 1) ^ R::swizzle(vrow)) << 4) +
                     (qi & 1) * 8;

  for (int i = 0; i < span.n; ++i, --left) {
    const int key0 = span.first + i * R::kKeys;
    // 16-key groups on a page that is none
    unsigned missing = 0;
    if (__builtin_expect((feed.none >> stage) & 1, 0)) {
#pragma unroll
      for (int b = 0; b < NG; ++b) {
        const int p = min(key0 + 16 * b, keys - 1) >> a.kv.page_shift;
        int id = a.req.table[(size_t)span.r * a.req.width + p];
        settle(id);
        if (id < 0 || id >= a.kv.num_blocks) missing |= 1u << b;
      }
      missing = __builtin_amdgcn_readfirstlane(missing);
    }
    // the tile holds keys that some query does not see (the request's own rows
    // after its root, keys past its last), or such a group
    const bool edge = key0 + R::kKeys > prefix + 1 || missing;
    unsigned buf, odd_at = lds + R::kOdd;
    // Values of keys that do not exist are anything: zeros in their place. NaN and
    // infinity in a row that some query does not see must not meet its zero
    // weight: such elements are left out here and added below. 16 bytes at a
    // time; returns whether something was left out.
    auto clean = [&](kv_u32x4& w, bool there) {
      unsigned strange = 0;
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        unsigned out = 0;
#pragma unroll
        for (int y = 0; y < 4 / R::CB; ++y) {
          constexpr unsigned E = E8 ? 0x7Fu : TT::kExpMask, all = E8 ? 0xFFu : 0xFFFFu;
          const int sh = y * 8 * R::CB;
          if (((w[x] >> sh) & E) == E) out |= all << sh;
        }
        strange |= out;
        w[x] = there ? w[x] & ~out : 0;
      }
      return strange != 0 && there;
    };
    // the wave's rows that a ballot over copy n's lanes names
    auto rows_in = [&](unsigned long long found, int n) {
      unsigned rows = 0;
      while (found) {
        rows |= 1u << (n * R::kRowsPerCopy + (int)__builtin_ctzll(found) / R::kChunks);
        found &= found - 1;
      }
      return rows;
    };
    auto put_odd = [&](unsigned rows) {
      if (lane == 0) {
        if constexpr (R::kRows == 8) {
          lds_write<unsigned char>(odd_at + (wave & (W / 2 - 1)), (unsigned char)rows);
        } else {
          lds_write<unsigned short>(odd_at + 2 * (wave & (W / 2 - 1)), (unsigned short)rows);
        }
      }
    };
    const bool values = wave >= W / 2;
    const int row0 = (wave & (W / 2 - 1)) * R::kRows;  // of the wave's keys, or values
    __builtin_amdgcn_s_setprio(0);
    if constexpr (E8) {
      // the wave's piece of this tile: done when the pieces after it may not be
      if (left > R::kStages - 1) {
        wait_copies<(R::kStages - 1) * R::kPerWave>();
      } else {
        wait_copies<0>();
      }
      const int tile = stage & 1;  // (an even number of stages)
      buf = lds + tile * R::kTiles;
      odd_at += tile * 8;
      const unsigned from = lds + R::kRaw + (stage * W + wave) * R::kPiece;
      const unsigned to = buf + (values ? R::kTile : 0);
      unsigned strange_rows = 0;
#pragma unroll
      for (int n = 0; n < R::kCopies; ++n) {
        const int r = n * R::kRowsPerCopy + lane / R::kChunks, row = row0 + r;
        const int c = lane % R::kChunks;
        kv_u32x4 w = lds_read<kv_u32x4>(from + n * 1024 + lane * 16);
        unsigned b = lds_read<unsigned char>(from + R::kRows * D + r);
        if (values && edge) {
          const bool there = key0 + row < keys && !((missing >> (row >> 4)) & 1);
          strange_rows |= rows_in(__ballot(clean(w, there)), n);
          // (no row that append writes has more than 246; a code may pass every finite
          // number under it, and rows that do not see the row must not)
          b = there ? min(b, 246u) : 127u;
        }
        const float e = __builtin_bit_cast(float, b << 23);
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          kv_u32x4 z;
#pragma unroll
          for (int y = 0; y < 2; ++y) {
            z[2 * y] = __builtin_bit_cast(
                unsigned, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w[2 * x + y], e, false));
            z[2 * y + 1] = __builtin_bit_cast(
                unsigned, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w[2 * x + y], e, true));
          }
          lds_write(to + row * R::kRow + (((2 * c + x) ^ R::swizzle(row)) << 4), z);
        }
      }
      if (values && edge) put_odd(strange_rows);
      feed.next(a, lds, wave);
      barrier();
    } else {
      // this tile's copies are done when those of the stages after it may not be
      if (left > R::kStages - 2) {
        wait_copies<(R::kStages - 2) * R::kPerWave>();
      } else {
        wait_copies<0>();
      }
      barrier();
      buf = lds + stage * R::kTiles;
      feed.next(a, lds, wave);
      if (edge) {
        if (values) {
          unsigned strange_rows = 0;
#pragma unroll
          for (int n = 0; n < R::kCopies; ++n) {
            const int row = row0 + n * R::kRowsPerCopy + lane / R::kChunks;
            const bool there = key0 + row < keys && !((missing >> (row >> 4)) & 1);
            const unsigned at = buf + R::kTile + row0 * R::kRow + n * 1024 + lane * 16;
            kv_u32x4 w = lds_read<kv_u32x4>(at);
            strange_rows |= rows_in(__ballot(clean(w, there)), n);
            lds_write(at, w);
          }
          put_odd(strange_rows);
        }
        barrier();
      }
    }
    stage = stage + 1 == R::kStages ? 0 : stage + 1;
    // products before other waves' copies (64 trees, 8-bit: 243 -> 233 us)
    __builtin_amdgcn_s_setprio(2);
    if constexpr (ROWS) {
      // Scores. Reads from LDS go out in batches, ahead of the products that use
      // them and, for the values, of the softmax.
      f32x4 sc[NG];
#pragma unroll
      for (int b = 0; b < NG; ++b) sc[b] = (f32x4){0, 0, 0, 0};
      constexpr int FB = 2;
#pragma unroll
      for (int b = 0; b < NG; b += 2)
#pragma unroll
        for (int f0 = 0; f0 < NF; f0 += FB) {
          V8 kf[FB][2];
#pragma unroll
          for (int f = 0; f < FB; ++f)
#pragma unroll
            for (int x = 0; x < 2; ++x)
              kf[f][x] =
                  lds_read<V8>(buf + ((key_at ^ ((f0 + f) << 6)) + (b + x) * 16 * R::kRow));
          __builtin_amdgcn_sched_barrier(0);
#pragma unroll
          for (int f = 0; f < FB; ++f)
#pragma unroll
            for (int x = 0; x < 2; ++x) sc[b + x] = TT::mfma(kf[f][x], qf[f0 + f], sc[b + x]);
        }
      constexpr int DB = ND / 2;
      V4 vl[DB][NG / 2], vh[DB][NG / 2];
      auto read_values = [&](int d0) {
#pragma unroll
        for (int d = 0; d < DB; ++d)
#pragma unroll
          for (int c = 0; c < NG / 2; ++c) {
            const unsigned at = buf + ((val_at ^ ((d0 + d) << 5)) + c * 32 * R::kRow);
            vl[d][c] = lds_columns<V4>(at);
            vh[d][c] = lds_columns<V4>(at + 16 * R::kRow);
          }
        __builtin_amdgcn_sched_barrier(0);
      };
      read_values(0);
      if (edge) {
#pragma unroll
        for (int b = 0; b < NG; ++b)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int rel = key0 + b * 16 + g * 4 + e - prefix;
            const bool own = rel < len && ((seen >> ((rel - 1) & 63)) & 1);
            if (((missing >> b) & 1) || (rel > 0 && !own)) sc[b][e] = -__builtin_inff();
          }
      }
      // Weights. The product with the scale rounds before the maximum is taken off.
      // One fma for both would leave the largest weight up to half a step of its
      // score away from 1, which at scores from 2^30 on is a power of two that
      // overflows or leaves nothing (64 8-bit trees: 234 us with it, 239 without).
      float top = sc[0][0];
#pragma unroll
      for (int b = 0; b < NG; ++b)
#pragma unroll
        for (int e = 0; e < 4; ++e) top = fmaxf(top, sc[b][e]);
      // (a difference: mx + kSlack would round by such a step too)
      if (__any(top * sl - mx > TT::kAbove + TT::kSlack)) {
        float next = group_max(top * sl);
        if constexpr (TT::kAbove > 0.0f) {
          // (not where kAbove rounds up to more than a weight may be)
          const float less = next - TT::kAbove;
          next = next - less > TT::kAbove + TT::kSlack ? next : less;
        }
        next = fmaxf(mx, next);
        const float fix = next == -__builtin_inff() ? 1.0f : __builtin_amdgcn_exp2f(mx - next);
        mx = next;
        l *= fix;
#pragma unroll
        for (int d = 0; d < ND; ++d) o[d] *= fix;
      }
      const float ref = mx == -__builtin_inff() ? 0.0f : mx;
      // The product takes weights of the query type, each off by up to half its step;
      // their sum takes them as they are. The outputs' error against 64 bits is 0.0023
      // of their size for it in bfloat16 and 0.00028 in float16, where weights in
      // float32 leave 0.0017 and 0.00021. Split in two halves with a product each they
      // nearly would: 329 us the 64 8-bit trees against 243, 112 the chains against 110.
      V8 pf[NG / 2];
#pragma unroll
      for (int b = 0; b < NG; ++b)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float p = __builtin_amdgcn_exp2f(sc[b][e] * sl - ref);
          l += p;
          pf[b >> 1][(b & 1) * 4 + e] = (T)p;
        }
      // O^T += V^T P^T
#pragma unroll
      for (int d0 = 0; d0 < ND; d0 += DB) {
        if (d0) read_values(d0);
#pragma unroll
        for (int c = 0; c < NG / 2; ++c)
#pragma unroll
          for (int d = 0; d < DB; ++d) {
            const V8 vf = __builtin_shufflevector(vl[d][c], vh[d][c], 0, 1, 2, 3, 4, 5, 6, 7);
            o[d0 + d] = TT::mfma(vf, pf[c], o[d0 + d]);
          }
      }
      if (edge) {
        unsigned long long odd = 0;  // rows of the tile that hold NaN or infinity
        if constexpr (NG == 4) {
          odd = read_lane(lds_read<unsigned long long>(odd_at), 0);
        } else {
          odd = (unsigned)read_lane((int)lds_read<unsigned>(odd_at), 0);
        }
        while (odd) {
          // they go to the queries that see the row
          const int row = (int)__builtin_ctzll(odd);
          odd &= odd - 1;
          const int key = key0 + row, rel = key - prefix;
          const int64_t id = a.req.table[(size_t)span.r * a.req.width + (key >> a.kv.page_shift)];
          const int64_t at =
              ((int64_t)span.h << a.kv.page_shift) + (key & ((1 << a.kv.page_shift) - 1));
          const unsigned char* src = a.kv.v + id * a.kv.page_bytes + at * (D * R::CB);
          const bool vis = rel <= 0 || ((seen >> ((rel - 1) & 63)) & 1);
#pragma unroll
          for (int d = 0; d < ND; ++d) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const int col = d * 16 + g * 4 + e;
              float v;
              if (E8) {
                v = (src[col] & 127) == 127 ? __builtin_nanf("") : 0.0f;
              } else {
                v = (float)reinterpret_cast<const T*>(src)[col];
                v = finite_f32(v) ? 0.0f : v;
              }
              settle(v);  // one at a time: no registers for a rare path
              o[d][e] += vis ? v : 0.0f;
            }
          }
        }
      }
    }
  }

  if constexpr (ROWS) {
    const float sum = group_sum(l);
    if (live && job.whole) {
      const int head = span.h * a.group + (m - qrow * a.group);
      const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
      T* dst = reinterpret_cast<T*>(a.out + (size_t)(s.c0 + qrow) * a.out_ld) + head * D + g * 4;
#pragma unroll
      for (int d = 0; d < ND; ++d) {
        V4 z;
#pragma unroll
        for (int e = 0; e < 4; ++e) z[e] = (T)(o[d][e] * inv);
        *reinterpret_cast<V4*>(dst + d * 16) = z;
      }
      if (a.lse && g == 0)
        a.lse[(size_t)(s.c0 + qrow) * a.num_heads + head] =
            sum == 0.0f ? -__builtin_inff() : (mx + __builtin_amdgcn_logf(sum)) * kLn2;
    } else if (live) {
      const size_t at = (size_t)job.slot * ws.rows + wave * 16 + qi;
      float* dst = ws.o + at * D + g * 4;
#pragma unroll
      for (int d = 0; d < ND; ++d) *reinterpret_cast<f32x4*>(dst + d * 16) = o[d];
      if (g == 0) {
        ws.m[at] = mx;
        ws.l[at] = sum;
      }
    }
  }
}

// out = sum_k e^(s_k - m) v_k / sum_k e^(s_k - m) in one pass over the keys: running
// maximum m, sum and outputs in float32 registers, m moved only when a score
// passes it by Types::kSlack. Parts of a row join by (m, sum, outputs) in join_kernel.
//
// Persistent over the units of all (request, key/value head, row segment)s in
// order: workgroup w takes the w-th equal share, so ragged contexts balance by
// themselves and a long one is split over many workgroups. The ring of tiles
// runs on across segments.
//
// Bound. Few rows to a head: the stream of keys and values. 32 chains of up to 9
// rows, 32 query heads on 8 of 128, bf16, 1k to 8k keys: 607 MB, 105 us and 5 for
// the join (5.8 TB/s of the 7.0 that a plain read reaches; without the products
// 104). Many rows over 8 bits: the latency of one tile's widening, products and
// barrier, with four waves to a SIMD to cover it. 64 trees of up to 17 rows, 64 on
// 8: 580 MB and 76 GFLOP, 243 us and 12 (2.4 TB/s, 313 TFLOP/s; the copies alone
// 120). A tree of 65 rows and a single row over 70k and 131k keys, 16 on 2 of 64,
// f16: 103 MB; 88 us and 16.5 with the tree over the 131k (35 GFLOP), 67 and 13.5
// over the 70k (19 GFLOP; the product of 8192 x 8192 matrices of the vendor's
// library reaches 1207 TFLOP/s here). One token over 700 keys: 8 us and 4, all of it
// the chain of dependent reads (lengths, pages, queries, keys).
//
// Tried and not kept: keys and values straight into registers, a wave to 32 keys
// (846 us the 64 trees, and spills); 64 keys to a step of 8-bit tiles (252 to 313);
// five stages (240); exponents copied for four tiles at once (251); two row tiles to
// each of four waves (263).
template <typename T, bool E8, int D, int W>
__global__ __launch_bounds__(W * kWave, (Ring<E8, D, W>::kPerCu * W / 4)) void split_kernel(
    AttnArgs a, Parts ws) {
  constexpr int kThreads = W * kWave;
  typedef Ring<E8, D, W> R;
  __shared__ __align__(1024) unsigned char lds_mem[R::kBytes];
  __shared__ int64_t wsum[W];
  __shared__ int start_r;
  __shared__ int64_t start_off;
  const ReqView& q = a.req;
  const int tid = threadIdx.x;
  const int wave = __builtin_amdgcn_readfirstlane(tid / kWave);
  const unsigned lds = (unsigned)(uintptr_t)(lds_u8*)lds_mem;
  int rows_total;
  const int total_eff = rows_in_use(q, &rows_total);
  // every wave finds its workgroup's share by itself where a wave's lanes hold
  // the batch; the workgroup together where they do not
  Cursor cur;
  cur.begun = 0;
  int64_t u0, u1;
  int64_t total;
  const int wgs_all = gridDim.x;
  if (q.B <= kWave) {
    int c0 = 0, len = 0, prefix = 0;
    if (lane_id() < q.B && !rows_of(a, lane_id(), total_eff, &c0, &len, &prefix)) len = 0;
    if (wave == 0) {
      lds_write(lds + R::kReqs + 12 * lane_id(), c0);
      lds_write(lds + R::kReqs + 12 * lane_id() + 4, len);
      lds_write(lds + R::kReqs + 12 * lane_id() + 8, prefix);
    }
    const int64_t mine = len ? units_of<D>(a, c0, len, prefix) : 0;
    const int64_t incl = wave_incl_scan_op(mine, (int64_t)0, OpAdd{});
    total = read_lane(incl, kWave - 1);
    if (blockIdx.x == 0 && tid < q.B) ws.base[tid] = incl - mine;
    const int wgs = wgs_in_use(total, wgs_all);
    cur.share = share_of(blockIdx.x, wgs);
    u0 = (int)blockIdx.x < wgs ? wg_start(total, cur.share, wgs) : total;
    u1 = (int)blockIdx.x < wgs ? wg_start(total, cur.share + 1, wgs) : total;
    const unsigned long long past = __ballot(u0 < incl);
    cur.r = past ? (int)__builtin_ctzll(past) : 0;
    cur.off = u0 - read_lane(incl - mine, cur.r);
    barrier();
  } else {
    auto units = [&](int r) {
      int c0, len, prefix;
      return rows_of(a, r, total_eff, &c0, &len, &prefix) ? units_of<D>(a, c0, len, prefix)
                                                          : (int64_t)0;
    };
    const int per = (q.B + kThreads - 1) / kThreads;
    const int r0 = min(tid * per, q.B), r1 = min(r0 + per, q.B);
    int64_t mine = 0;
    for (int r = r0; r < r1; ++r) mine += units(r);
    int64_t at = block_excl_scan<int64_t, kThreads>(mine, wsum, &total);
    if (blockIdx.x == 0) {
      int64_t b = at;
      for (int r = r0; r < r1; ++r) {
        ws.base[r] = b;
        b += units(r);
      }
    }
    const int wgs = wgs_in_use(total, wgs_all);
    cur.share = share_of(blockIdx.x, wgs);
    u0 = (int)blockIdx.x < wgs ? wg_start(total, cur.share, wgs) : total;
    u1 = (int)blockIdx.x < wgs ? wg_start(total, cur.share + 1, wgs) : total;
    if (at <= u0 && u0 < at + mine) {
      for (int r = r0; r < r1; ++r) {
        const int64_t n = units(r);
        if (u0 < at + n) {
          start_r = r;
          start_off = u0 - at;
          break;
        }
        at += n;
      }
    }
    __syncthreads();
    cur.r = __builtin_amdgcn_readfirstlane(start_r);
    cur.off = read_lane(start_off, 0);
  }
  if (blockIdx.x == 0 && tid == 0) {
    ws.base[q.B] = total;
    a.meta[0] = rows_total;
    a.meta[1] = rows_total != total_eff ? DSPARK_DATA_BAD_LENS : 0;
  }
  if (u0 >= u1) return;
  cur.left = u1 - u0;
  Feeder<E8, D, W> feed;
  feed.start(a, lds, cur, wave);
#pragma unroll
  for (int i = 0; i < (E8 ? R::kStages : R::kStages - 1); ++i) feed.next(a, lds, wave);
  int64_t left = u1 - u0;
  int stage = 0;
  for (;;) {
    Job job;
    const Span span = next_span<D>(a, lds + R::kReqs, cur, &job);
    if (span.n == 0) break;
    // the wave has a tile of it, or not; nobody has of a request whose tree is none
    bool rows = wave < job.mt;
    if (q.parents) {
      const int lane = lane_id();
      const int up = lane + 1 < job.s.len ? q.parents[(size_t)span.r * q.gamma + lane] : 0;
      if (__ballot(up < 0 || up > lane)) rows = false;
    }
    // tiles still to come, as far as the end of the ring is concerned
    const int near = (int)min(left, (int64_t)1 << 30);
    if (rows) {
      segment<T, E8, D, W, true>(a, ws, span, job, feed, lds, near, stage);
    } else {
      segment<T, E8, D, W, false>(a, ws, span, job, feed, lds, near, stage);
    }
    left -= span.n;
  }
}

template <int D, int W>
void launch_waves(const AttnArgs& a, const Parts& ws, dspark_dtype dt, hipStream_t s) {
  const dim3 grid((unsigned)ws.wgs), block(W * kWave);
  if (a.kv.cb == 1) {
    hipLaunchKernelGGL((split_kernel<__bf16, true, D, W>), grid, block, 0, s, a, ws);
  } else if (dt == DSPARK_BF16) {
    hipLaunchKernelGGL((split_kernel<__bf16, false, D, W>), grid, block, 0, s, a, ws);
  } else {
    hipLaunchKernelGGL((split_kernel<_Float16, false, D, W>), grid, block, 0, s, a, ws);
  }
}

template <int D>
void launch_dim(const AttnArgs& a, const Parts& ws, dspark_dtype dt, hipStream_t s) {
  if constexpr (D >= 128) {
    if (a.waves == kFewWaves) return launch_waves<D, kFewWaves>(a, ws, dt, s);
  }
  launch_waves<D, kMostWaves>(a, ws, dt, s);
}

void launch_dim64(const AttnArgs& a, const Parts& ws, dspark_dtype dt, hipStream_t s);
void launch_dim128(const AttnArgs& a, const Parts& ws, dspark_dtype dt, hipStream_t s);
void launch_dim256(const AttnArgs& a, const Parts& ws, dspark_dtype dt, hipStream_t s);

}  // namespace attn
}  // namespace dspark
