// Attention of packed verify rows (a chain or tree of drafts per request) over
// the paged cache: the split kernel's templates, one translation unit per head
// dimension, and the schedule it shares with the joining kernel.
#pragma once

#include "kv_dev.h"

namespace dspark {
namespace attn {

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / kWave;

// What the split kernel leaves for the joining kernel: the schedule's prefix
// sums, and per partial segment the running maximum and sum of each of its rows
// and their unnormalised outputs. Workgroup w has segments 2 w (the one its
// range starts with) and 2 w + 1 (a later one that its range ends in).
struct Parts {
  int64_t* base;  // [B + 1] first unit of each request, then the total
  float* m;       // [2 * wgs][rows]
  float* l;
  float* o;       // [2 * wgs][rows][D]
  int wgs;        // workgroups of the split kernel
  int rows;       // rows of a segment, at most
};

// Tiles of 16 query rows of a segment, at most, and keys of a unit.
template <int D>
struct Size {
  static constexpr int kTilesPerWave = D == 256 ? 1 : 2;
  static constexpr int kTiles = kWaves * kTilesPerWave;
  static constexpr int kKeys = D == 256 ? 32 : 64;
};

// Rows of a (request, key/value head): m = j * group + g for row j and the g-th
// of the head's queries, in tiles of 16, several tiles to a segment.
struct Shape {
  int len, prefix, c0;
  int mrows, mtiles;
  int nseg, per;  // segments side by side, tiles of each
  int64_t keys;
  int nku;        // units along the keys
};

template <int D>
__device__ inline bool shape_of(const AttnArgs& a, int r, int total_eff, Shape* s) {
  constexpr int kT = Size<D>::kTiles, kK = Size<D>::kKeys;
  if (!request_rows(a.req, r, total_eff, &s->c0, &s->len)) return false;
  s->prefix = a.req.prefix[r];
  s->keys = (int64_t)s->prefix + s->len;
  if (s->prefix < 0 || s->keys > ((int64_t)a.req.width << a.kv.page_shift) ||
      s->keys > 0x7FFFFF00LL)  // cache indices in 32 bits, a unit beyond included
    return false;
  s->mrows = a.group * s->len;
  s->mtiles = (s->mrows + 15) >> 4;
  s->nseg = (s->mtiles + kT - 1) / kT;
  s->per = (s->mtiles + s->nseg - 1) / s->nseg;
  s->nku = (int)((s->keys + kK - 1) / kK);
  return true;
}

template <int D>
__device__ inline int64_t units_of(const AttnArgs& a, int r, int total_eff) {
  Shape s;
  return shape_of<D>(a, r, total_eff, &s) ? (int64_t)a.kv.hkv * s.nseg * s.nku : 0;
}

// Workgroups that get units: never one without.
__device__ inline int wgs_in_use(int64_t total, int wgs) { return (int)min((int64_t)wgs, total); }

// The first unit of workgroup w of n <= total.
__device__ inline int64_t wg_start(int64_t total, int w, int n) { return total * w / n; }

template <typename T>
struct Types;
template <>
struct Types<__bf16> {
  typedef bf16x8 V8;
  typedef bf16x4 V4;
  static constexpr unsigned kExpMask = 0x7F80u;
  static __device__ f32x4 mfma(V8 a, V8 b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
  }
};
template <>
struct Types<_Float16> {
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

// Eight rows of sixteen 8-bit elements, transposed: lanes point at the rows'
// halves, lane i gets column i.
__device__ inline kv_u32x2 lds_columns8(unsigned at) {
  typedef __attribute__((ext_vector_type(2))) int i32x2;
  typedef __attribute__((address_space(3))) i32x2 lds_i32x2;
  return __builtin_bit_cast(kv_u32x2, __builtin_amdgcn_ds_read_tr8_b64_v2i32((lds_i32x2*)(uintptr_t)at));
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
  asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, %1"
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
// A row's maximum follows its scores only when they pass it by this much (in
// log2): weights then stay below 2^kSlack, and most steps rescale nothing.
constexpr float kSlack = 8.0f;

// The tile of keys and values that a workgroup's waves share in LDS, in a ring
// of kStages. Rows are unpadded (the copies into LDS write densely); 16-byte
// chunk c of a row lies at chunk c ^ swizzle(row), so that the 16 rows which a
// wave reads at one column spread over all banks.
template <bool E8, int D>
struct Ring {
  static constexpr int CB = E8 ? 1 : 2;
  static constexpr int kKeys = Size<D>::kKeys;
  static constexpr int kGroups = kKeys / 16;
  static constexpr int kRow = D * CB;                 // bytes of a row
  static constexpr int kChunks = kRow / 16;
  static constexpr int kRowsPerCopy = kWave / kChunks;
  static constexpr int kCopies = 16 / kRowsPerCopy;   // copies of 16 rows
  static constexpr int kTile = kKeys * kRow;          // keys, or values
  static constexpr int kScales = 2 * kTile;           // offset of the exponents
  static constexpr int kStage = 2 * kTile + (E8 ? 2 * kKeys : 0);
  static constexpr int kStages = 65536 / (2 * kTile) < 4 ? 65536 / (2 * kTile) : 4;
  // copies of a wave per stage: with 64 keys wave w has 16 keys and their
  // values, with 32 keys 16 keys or their values
  static constexpr int kPerWave = kGroups == 4 ? 2 * kCopies + (E8 ? 2 : 0) : kCopies + (E8 ? 1 : 0);
  static constexpr int kFlags = kStages * kStage;     // bad pages, a byte per stage and wave
  static constexpr int kOdd = kFlags + 4 * kStages;   // rows with NaN or infinity, 16 bits a group
  static constexpr int kBytes = kOdd + 8 + (16 - (4 * kStages + 8) % 16) % 16;
  static __device__ int swizzle(int row) {
    return kChunks >= 16 ? row & 15 : (kChunks == 8 ? (row >> 1) & 7 : (row >> 2) & 3);
  }
};

// One segment: the queries of several 16-row tiles of one (request, key/value
// head) over units [ku0, ku0 + n) of its keys.
struct Job {
  Shape s;
  int r, h, tile0, mt;
  int n;         // units; 0: there is no such segment
  int slot;      // its place among the parts
  bool whole;    // it covers all the request's keys
  int first;     // its first key
};

// Where a workgroup is in its share of the units.
struct Cursor {
  int64_t u, u1, off;  // next unit, end, next unit within request r
  int64_t u0;
  int64_t n_r;         // units of request r, -1: not known yet
  int r;
  Shape s;
};

template <int D>
__device__ __forceinline__ Job next_job(const AttnArgs& a, int total_eff, Cursor& c) {
  Job j;
  j.n = 0;
  while (c.u < c.u1) {
    if (c.n_r < 0)
      c.n_r = shape_of<D>(a, c.r, total_eff, &c.s) ? (int64_t)a.kv.hkv * c.s.nseg * c.s.nku : 0;
    if (c.off >= c.n_r) {
      ++c.r;
      c.off = 0;
      c.n_r = -1;
      continue;
    }
    const Shape& s = c.s;
    const int item = (int)(c.off / s.nku);
    const int ku0 = (int)(c.off - (int64_t)item * s.nku);
    j.s = s;
    j.r = c.r;
    j.n = (int)min((int64_t)(s.nku - ku0), c.u1 - c.u);
    j.h = item / s.nseg;
    const int seg = item - j.h * s.nseg;
    j.tile0 = seg * s.per;
    j.mt = min(s.per, s.mtiles - j.tile0);
    j.whole = j.n == s.nku;
    j.slot = 2 * blockIdx.x + (c.u == c.u0 ? 0 : 1);
    j.first = ku0 * Size<D>::kKeys;
    c.off += j.n;
    c.u += j.n;
    break;
  }
  return j;
}

// The producing side of the ring: this wave's copies of the next tile.
template <bool E8, int D>
struct Feeder {
  typedef Ring<E8, D> R;
  Cursor c;
  Job j, nj;     // the job copied from, and the one after it
  int i;         // its next tile
  int ids, nids; // page ids of the wave's rows, lane l: tile id_first + l
  int id_first;
  int stage;

  static __device__ int group_of(int wave) { return wave % R::kGroups; }

  // The page ids have arrived here, and not at each of their uses: a wait for
  // them would be one for the copies behind them too.
  __device__ void settle() { asm volatile("" : "+v"(ids)); }

  // lanes 0..63: the pages of 64 tiles from tile i on
  __device__ int fetch(const AttnArgs& a, const Job& x, int t, int wave) const {
    const int64_t key =
        (int64_t)x.first + (int64_t)(t + lane_id()) * R::kKeys + group_of(wave) * 16;
    const int p = (int)min(key, x.s.keys - 1) >> a.kv.page_shift;
    return a.req.table[(size_t)x.r * a.req.width + p];
  }

  __device__ void start(const AttnArgs& a, int total_eff, const Cursor& at, int wave) {
    c = at;
    j = next_job<D>(a, total_eff, c);
    ids = fetch(a, j, 0, wave);
    settle();
    nj = next_job<D>(a, total_eff, c);
    nids = nj.n > 0 ? fetch(a, nj, 0, wave) : 0;
    i = id_first = stage = 0;
  }

  __device__ void copies(const unsigned char* from, unsigned lds_at) const {
    const int lane = lane_id();
#pragma unroll
    for (int n = 0; n < R::kCopies; ++n) {
      const int row = n * R::kRowsPerCopy + lane / R::kChunks;
      const unsigned chunk = (unsigned)((lane % R::kChunks) ^ R::swizzle(row));
      copy16(from + n * R::kRowsPerCopy * R::kRow, (lane / R::kChunks) * R::kRow + chunk * 16,
             lds_at + n * 1024);
    }
  }

  __device__ void next(const AttnArgs& a, int total_eff, unsigned lds, int wave) {
    if (j.n == 0) return;
    const int g = group_of(wave);
    const int key = j.first + i * R::kKeys + g * 16;
    int id = __builtin_amdgcn_readlane(ids, i - id_first);
    const bool bad = id < 0 || id >= a.kv.num_blocks;
    if (bad) id = 0;  // any valid page: its keys are masked
    const int64_t row =
        ((int64_t)j.h << a.kv.page_shift) + (key & ((1 << a.kv.page_shift) - 1));
    const unsigned base = lds + stage * R::kStage;
    const unsigned char* k = uniform(a.kv.k + (int64_t)id * a.kv.page_bytes + row * R::kRow);
    const unsigned char* v = uniform(a.kv.v + (int64_t)id * a.kv.page_bytes + row * R::kRow);
    const unsigned kat = base + g * 16 * R::kRow, vat = kat + R::kTile;
    if (R::kGroups == 4 || wave < 2) copies(k, kat);
    if (R::kGroups == 4 || wave >= 2) copies(v, vat);
    if constexpr (E8) {
      const int64_t at = (int64_t)id * a.kv.scale_page_bytes + row;
      const unsigned sc = base + R::kScales + g * 16;
      if (lane_id() < 4) {
        if (R::kGroups == 4 || wave < 2) copy4(uniform(a.kv.ks + at), lane_id() * 4, sc);
        if (R::kGroups == 4 || wave >= 2)
          copy4(uniform(a.kv.vs + at), lane_id() * 4, sc + R::kKeys);
      }
    }
    if (lane_id() == 0)
      lds_write<unsigned char>(lds + R::kFlags + stage * 4 + wave, bad ? 1 : 0);
    stage = stage + 1 == R::kStages ? 0 : stage + 1;
    if (++i == j.n) {
      j = nj;
      ids = nids;
      settle();
      i = id_first = 0;
      if (j.n > 0) {
        nj = next_job<D>(a, total_eff, c);
        nids = nj.n > 0 ? fetch(a, nj, 0, wave) : 0;
      }
    } else if (i - id_first == kWave) {
      ids = fetch(a, j, i, wave);
      settle();
      id_first = i;
    }
  }
};

// A wave's part of a segment: NT of its 16-row tiles (tile w, w + 4, ..; none for
// a wave past the last) over all its keys, which the four waves bring into LDS
// together. The products are
//   S^T = K Q^T: keys are its rows and queries its columns, so a lane holds the
//   scores of one query (lane & 15) for four keys of each sixteen, which are in
//   place as the operand of  O^T = V^T P^T.
template <typename T, bool E8, int D, int NT>
__device__ __forceinline__ void segment(const AttnArgs& a, const Parts& ws, const Job& job,
                                        Feeder<E8, D>& feed, int total_eff, unsigned lds,
                                        int64_t left, int& stage) {
  typedef Types<T> TT;
  typedef typename TT::V8 V8;
  typedef typename TT::V4 V4;
  typedef Ring<E8, D> R;
  constexpr int NF = D / 32;         // operand chunks of a key
  constexpr int ND = D / 16;         // 16-column tiles of the output
  constexpr int NG = R::kGroups;     // 16-key groups of a tile
  constexpr int NTX = NT ? NT : 1;
  const Shape& s = job.s;
  const int lane = lane_id(), qi = lane & 15, g = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int len = s.len, prefix = s.prefix;
  const int keys = (int)s.keys;
  const SmallDiv by_group(a.group);

  // the step's own tree: bit l of anc, in lane l, is row l + 1 itself, with its
  // ancestors' bits; row 0 is everybody's
  unsigned long long anc = 0;
  if (NT > 0 && a.req.parents) {
    int up = lane + 1 < len ? a.req.parents[(size_t)job.r * a.req.gamma + lane] : 0;
    anc = 1ull << lane;
    for (int i = 0; i < 6; ++i) {
      const int from = max(up - 1, 0);
      const unsigned long long more = __shfl(anc, from, kWave);
      const int next = __shfl(up, from, kWave);
      if (up > 0) {
        anc |= more;
        up = next;
      }
    }
  }
  // Scores in units of log2 with a positive factor, so that a masked score stays
  // -infinity under it: the scale's sign and its zero go into the queries.
  float sl = fminf(fabsf(a.scale) * kLog2e, 3.4028235e38f);
  const bool flat = sl == 0.0f;
  if (flat) sl = 1.0f;
  const unsigned sign = a.scale < 0.0f ? 0x80008000u : 0u;
  // queries as operands. A lane's place in a key: of two 8-bit chunks in one read
  V8 qf[NTX][NF];
  f32x4 o[NTX][ND];
  float mx[NTX], l[NTX];
  int qrow[NTX];  // the request's row that the lane's query belongs to
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    const int m = (job.tile0 + wave + kWaves * t) * 16 + qi;
    const int row = by_group.quo(m);
    qrow[t] = row;
    const unsigned char* src = a.q + (size_t)(s.c0 + row) * a.q_ld +
                               (size_t)(job.h * a.group + (m - row * a.group)) * D * 2;
#pragma unroll
    for (int f = 0; f < NF; ++f) {
      const int d = E8 ? (f >> 1) * 64 + g * 16 + (f & 1) * 8 : f * 32 + g * 8;
      kv_u32x4 w = (kv_u32x4){0, 0, 0, 0};
      if (m < s.mrows && !flat) w = *reinterpret_cast<const kv_u32x4*>(src + d * 2) ^ sign;
      qf[t][f] = __builtin_bit_cast(V8, w);
    }
    mx[t] = -__builtin_inff();
    l[t] = 0.0f;
#pragma unroll
    for (int d = 0; d < ND; ++d) o[t][d] = (f32x4){0, 0, 0, 0};
  }

  // eight 8-bit elements, widened
  auto widen = [](unsigned lo, unsigned hi, float e) {
    kv_u32x4 w;
    w[0] = __builtin_bit_cast(unsigned, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, e, false));
    w[1] = __builtin_bit_cast(unsigned, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, e, true));
    w[2] = __builtin_bit_cast(unsigned, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, e, false));
    w[3] = __builtin_bit_cast(unsigned, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, e, true));
    return __builtin_bit_cast(V8, w);
  };
  // rows of the step's own tree that the lane's query sees, bit l for row l + 1
  auto seen_by = [&](int t) {
    const int j = qrow[t];
    if (!a.req.parents) return j >= 64 ? ~0ull : (1ull << j) - 1;
    const unsigned long long path = __shfl(anc, max(j - 1, 0) & 63, kWave);
    return j > 0 ? path : 0ull;
  };

  // lane's offsets in a tile: its chunk of a key, its piece of a value row
  const int key_at = qi * R::kRow + ((g ^ R::swizzle(qi)) << 4);
  const int vrow = E8 ? g * 4 + ((qi >> 1) & 3) : g * 4 + (qi >> 2);
  const int val_at = R::kTile +
                     (E8 ? ((qi >> 3) * 16 + vrow) * R::kRow + (R::swizzle(vrow) << 4)
                         : vrow * R::kRow + ((((qi >> 1) & 1) ^ R::swizzle(vrow)) << 4)) +
                     (qi & 1) * 8;

  for (int i = 0; i < job.n; ++i, --left) {
    // this tile's copies are done when those of the stages after it may not be
    if (left > R::kStages - 2) {
      wait_copies<(R::kStages - 2) * R::kPerWave>();
    } else {
      wait_copies<0>();
    }
    barrier();
    const unsigned buf = lds + stage * R::kStage;
    const unsigned flags = lds_read<unsigned>(lds + R::kFlags + stage * 4);
    feed.next(a, total_eff, lds, wave);
    stage = stage + 1 == R::kStages ? 0 : stage + 1;
    const int key0 = job.first + i * R::kKeys;
    // the tile holds keys that some query does not see (the request's own rows
    // after its root, keys past its last), or rows of a page that is none
    const bool edge = key0 + R::kKeys > prefix + 1 ||
                      __builtin_amdgcn_readfirstlane((int)flags) != 0;
    auto missing = [&](int group) { return (flags >> (8 * group)) & 255u; };
    unsigned long long odd = 0;  // rows of the tile that hold NaN or infinity
    if (edge) {
      // Values of keys that do not exist are anything: zeros in their place. NaN
      // and infinity in a row that some query does not see must not meet its
      // zero weight: such elements are left out here and added below.
      if (wave < NG) {
        unsigned strange_rows = 0;
#pragma unroll
        for (int n = 0; n < R::kCopies; ++n) {
          const int row16 = n * R::kRowsPerCopy + lane / R::kChunks;
          const bool there = key0 + wave * 16 + row16 < keys && !missing(wave);
          const unsigned at = buf + R::kTile + wave * 16 * R::kRow + n * 1024 + lane * 16;
          kv_u32x4 w = lds_read<kv_u32x4>(at);
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
          lds_write(at, w);
          unsigned long long found = __ballot(strange && there);
          while (found) {
            strange_rows |= 1u << (n * R::kRowsPerCopy + (int)__builtin_ctzll(found) / R::kChunks);
            found &= found - 1;
          }
        }
        if (E8 && lane < 16 && (key0 + wave * 16 + lane >= keys || missing(wave)))
          lds_write<unsigned char>(buf + R::kScales + R::kKeys + wave * 16 + lane, 127);
        if (lane == 0) lds_write<unsigned short>(lds + R::kOdd + wave * 2, (unsigned short)strange_rows);
      }
      barrier();
      if constexpr (NG == 4) {
        odd = lds_read<unsigned long long>(lds + R::kOdd);
      } else {
        odd = lds_read<unsigned>(lds + R::kOdd);
      }
      odd = read_lane(odd, 0);
    }
    if constexpr (NT > 0) {
      // scores
      f32x4 sc[NT][NG];
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int b = 0; b < NG; ++b) sc[t][b] = (f32x4){0, 0, 0, 0};
#pragma unroll
      for (int b = 0; b < NG; b += 2) {
        if constexpr (E8) {
          float e[2];
#pragma unroll
          for (int x = 0; x < 2; ++x)
            e[x] = __builtin_bit_cast(
                float,
                (unsigned)lds_read<unsigned char>(buf + R::kScales + (b + x) * 16 + qi) << 23);
#pragma unroll
          for (int p = 0; p < NF / 2; ++p) {
            kv_u32x4 w[2];
#pragma unroll
            for (int x = 0; x < 2; ++x)
              w[x] = lds_read<kv_u32x4>(buf + ((key_at ^ (p << 6)) + (b + x) * 16 * R::kRow));
#pragma unroll
            for (int y = 0; y < 2; ++y)
#pragma unroll
              for (int x = 0; x < 2; ++x) {
                const V8 kf = widen(w[x][2 * y], w[x][2 * y + 1], e[x]);
#pragma unroll
                for (int t = 0; t < NT; ++t)
                  sc[t][b + x] = TT::mfma(kf, qf[t][2 * p + y], sc[t][b + x]);
              }
          }
        } else {
#pragma unroll
          for (int f = 0; f < NF; ++f)
#pragma unroll
            for (int x = 0; x < 2; ++x) {
              const V8 kf = lds_read<V8>(buf + ((key_at ^ (f << 6)) + (b + x) * 16 * R::kRow));
#pragma unroll
              for (int t = 0; t < NT; ++t)
                sc[t][b + x] = TT::mfma(kf, qf[t][f], sc[t][b + x]);
            }
        }
      }
      if (edge) {
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          const unsigned long long seen = seen_by(t);
#pragma unroll
          for (int b = 0; b < NG; ++b)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const int rel = key0 + b * 16 + g * 4 + e - prefix;
              const bool own = rel < len && ((seen >> ((rel - 1) & 63)) & 1);
              if (missing(b) || (rel > 0 && !own)) sc[t][b][e] = -__builtin_inff();
            }
        }
      }
      // weights
      float vs[E8 ? NG : 1][4];
      if constexpr (E8) {
#pragma unroll
        for (int b = 0; b < NG; ++b) {
          const unsigned w = lds_read<unsigned>(buf + R::kScales + R::kKeys + b * 16 + g * 4);
#pragma unroll
          for (int e = 0; e < 4; ++e)
            vs[b][e] = __builtin_bit_cast(float, ((w >> (8 * e)) & 255u) << 23);
        }
      }
      V8 pf[NT][NG / 2];
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        float top = sc[t][0][0];
#pragma unroll
        for (int b = 0; b < NG; ++b)
#pragma unroll
          for (int e = 0; e < 4; ++e) top = fmaxf(top, sc[t][b][e]);
        if (__any(top * sl > mx[t] + kSlack)) {
          const float next = fmaxf(mx[t], group_max(top * sl));
          const float fix =
              next == -__builtin_inff() ? 1.0f : __builtin_amdgcn_exp2f(mx[t] - next);
          mx[t] = next;
          l[t] *= fix;
#pragma unroll
          for (int d = 0; d < ND; ++d) o[t][d] *= fix;
        }
        const float ref = mx[t] == -__builtin_inff() ? 0.0f : mx[t];
#pragma unroll
        for (int b = 0; b < NG; ++b)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            float p = __builtin_amdgcn_exp2f(__builtin_fmaf(sc[t][b][e], sl, -ref));
            l[t] += p;
            // an 8-bit value's power of two goes to its weight, exactly
            if constexpr (E8) p *= vs[b][e];
            pf[t][b >> 1][(b & 1) * 4 + e] = (T)p;
          }
      }
      // O^T += V^T P^T
#pragma unroll
      for (int d0 = 0; d0 < ND; d0 += 2)
#pragma unroll
        for (int c = 0; c < NG / 2; ++c)
#pragma unroll
          for (int d = d0; d < d0 + 2; ++d) {
            V8 vf;
            if constexpr (E8) {
              const kv_u32x2 w = lds_columns8(buf + ((val_at ^ (d << 4)) + c * 32 * R::kRow));
              vf = widen(w[0], w[1], 1.0f);
            } else {
              const unsigned at = buf + ((val_at ^ (d << 5)) + c * 32 * R::kRow);
              const V4 lo = lds_columns<V4>(at);
              const V4 hi = lds_columns<V4>(at + 16 * R::kRow);
              vf = __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
            }
#pragma unroll
            for (int t = 0; t < NT; ++t) o[t][d] = TT::mfma(vf, pf[t][c], o[t][d]);
          }
      while (odd) {
        // a row with NaN or infinity: they go to the queries that see it
        const int row = (int)__builtin_ctzll(odd);
        odd &= odd - 1;
        const int key = key0 + row, rel = key - prefix;
        const int64_t id = a.req.table[(size_t)job.r * a.req.width + (key >> a.kv.page_shift)];
        const int64_t at =
            ((int64_t)job.h << a.kv.page_shift) + (key & ((1 << a.kv.page_shift) - 1));
        const unsigned char* src = a.kv.v + id * a.kv.page_bytes + at * R::kRow;
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
#pragma unroll
            for (int t = 0; t < NT; ++t) {
              const bool vis = rel <= 0 || ((seen_by(t) >> ((rel - 1) & 63)) & 1);
              if (vis) o[t][d][e] += v;
            }
            asm volatile("" ::: "memory");  // one element at a time: no registers for a rare path
          }
        }
      }
    }
  }

#pragma unroll
  for (int t = 0; t < NT; ++t) {
    const float sum = group_sum(l[t]);
    const int m = (job.tile0 + wave + kWaves * t) * 16 + qi;
    if (m >= s.mrows) continue;
    if (job.whole) {
      const int head = job.h * a.group + (m - qrow[t] * a.group);
      const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
      T* dst = reinterpret_cast<T*>(a.out + (size_t)(s.c0 + qrow[t]) * a.out_ld) + head * D + g * 4;
#pragma unroll
      for (int d = 0; d < ND; ++d) {
        V4 z;
#pragma unroll
        for (int e = 0; e < 4; ++e) z[e] = (T)(o[t][d][e] * inv);
        *reinterpret_cast<V4*>(dst + d * 16) = z;
      }
      if (a.lse && g == 0)
        a.lse[(size_t)(s.c0 + qrow[t]) * a.num_heads + head] =
            sum == 0.0f ? -__builtin_inff() : (mx[t] + __builtin_amdgcn_logf(sum)) * kLn2;
    } else {
      const size_t at = (size_t)job.slot * ws.rows + (wave + kWaves * t) * 16 + qi;
      float* dst = ws.o + at * D + g * 4;
#pragma unroll
      for (int d = 0; d < ND; ++d) *reinterpret_cast<f32x4*>(dst + d * 16) = o[t][d];
      if (g == 0) {
        ws.m[at] = mx[t];
        ws.l[at] = sum;
      }
    }
  }
}

// Persistent over the units of all (request, key/value head, row segment)s in
// order: workgroup w takes the w-th equal share, so ragged contexts balance by
// themselves and a long one is split over many workgroups. The ring of tiles
// runs on across segments.
template <typename T, bool E8, int D>
__global__ __launch_bounds__(kThreads, 2) void split_kernel(AttnArgs a, Parts ws) {
  typedef Ring<E8, D> R;
  __shared__ __align__(1024) unsigned char lds_mem[R::kBytes];
  __shared__ int64_t wsum[kWaves];
  __shared__ int start_r;
  __shared__ int64_t start_off;
  const ReqView& q = a.req;
  const int tid = threadIdx.x;
  const int wave = __builtin_amdgcn_readfirstlane(tid / kWave);
  const unsigned lds = (unsigned)(uintptr_t)(lds_u8*)lds_mem;
  int rows_total;
  const int total_eff = rows_in_use(q, &rows_total);
  // every workgroup sums the requests' units by itself
  const int per = (q.B + kThreads - 1) / kThreads;
  const int r0 = min(tid * per, q.B), r1 = min(r0 + per, q.B);
  int64_t mine = 0;
  for (int r = r0; r < r1; ++r) mine += units_of<D>(a, r, total_eff);
  int64_t total;
  int64_t at = block_excl_scan<int64_t, kThreads>(mine, wsum, &total);
  const int wgs = wgs_in_use(total, gridDim.x);
  if (blockIdx.x == 0) {
    int64_t b = at;
    for (int r = r0; r < r1; ++r) {
      ws.base[r] = b;
      b += units_of<D>(a, r, total_eff);
    }
    if (tid == 0) {
      ws.base[q.B] = total;
      a.meta[0] = rows_total;
      a.meta[1] = rows_total != total_eff ? DSPARK_DATA_BAD_LENS : 0;
    }
  }
  if ((int)blockIdx.x >= wgs) return;
  const int64_t u0 = wg_start(total, blockIdx.x, wgs), u1 = wg_start(total, blockIdx.x + 1, wgs);
  if (at <= u0 && u0 < at + mine) {
    for (int r = r0; r < r1; ++r) {
      const int64_t n = units_of<D>(a, r, total_eff);
      if (u0 < at + n) {
        start_r = r;
        start_off = u0 - at;
        break;
      }
      at += n;
    }
  }
  __syncthreads();
  Cursor cur;
  cur.u0 = cur.u = u0;
  cur.u1 = u1;
  cur.r = __builtin_amdgcn_readfirstlane(start_r);
  cur.off = read_lane(start_off, 0);
  cur.n_r = -1;
  Feeder<E8, D> feed;
  feed.start(a, total_eff, cur, wave);
#pragma unroll
  for (int i = 0; i < R::kStages - 1; ++i) feed.next(a, total_eff, lds, wave);
  int64_t left = u1 - u0;
  int stage = 0;
  for (;;) {
    const Job job = next_job<D>(a, total_eff, cur);
    if (job.n == 0) break;
    // tiles of this wave; none of a request whose tree is none
    int nt = max(0, (job.mt - wave + kWaves - 1) / kWaves);
    if (q.parents) {
      const int lane = lane_id();
      const int up = lane + 1 < job.s.len ? q.parents[(size_t)job.r * q.gamma + lane] : 0;
      if (__ballot(up < 0 || up > lane)) nt = 0;
    }
    if (nt == 0) {
      segment<T, E8, D, 0>(a, ws, job, feed, total_eff, lds, left, stage);
    } else if (nt == 1) {
      segment<T, E8, D, 1>(a, ws, job, feed, total_eff, lds, left, stage);
    } else if constexpr (Size<D>::kTilesPerWave > 1) {
      segment<T, E8, D, 2>(a, ws, job, feed, total_eff, lds, left, stage);
    }
    left -= job.n;
  }
}

template <int D>
void launch_dim(const AttnArgs& a, const Parts& ws, dspark_dtype dt, hipStream_t s) {
  const dim3 grid((unsigned)ws.wgs), block(kThreads);
  if (a.kv.cb == 1) {
    hipLaunchKernelGGL((split_kernel<__bf16, true, D>), grid, block, 0, s, a, ws);
  } else if (dt == DSPARK_BF16) {
    hipLaunchKernelGGL((split_kernel<__bf16, false, D>), grid, block, 0, s, a, ws);
  } else {
    hipLaunchKernelGGL((split_kernel<_Float16, false, D>), grid, block, 0, s, a, ws);
  }
}

void launch_dim64(const AttnArgs& a, const Parts& ws, dspark_dtype dt, hipStream_t s);
void launch_dim128(const AttnArgs& a, const Parts& ws, dspark_dtype dt, hipStream_t s);
void launch_dim256(const AttnArgs& a, const Parts& ws, dspark_dtype dt, hipStream_t s);

}  // namespace attn
}  // namespace dspark
