// Attention of packed verify rows (a chain or tree of drafts per request) over the
// latents of a paged cache: the split kernel's templates, one translation unit per
// latent size, and the schedule it shares with the joining kernel.
#pragma once

#include "latent.h"
#include "lds_dev.h"

namespace dspark {
namespace lattn {

using attn::barrier;
using attn::copy16_shared;
using attn::copy4;
using attn::f32x16;
using attn::kLn2;
using attn::kLog2e;
using attn::lds_columns;
using attn::lds_columns8;
using attn::lds_i32x2;
using attn::lds_read;
using attn::lds_u8;
using attn::lds_write;
using attn::settle;
using attn::Types;
using attn::uniform;
using attn::wait_copies;

// Row tiles of a workgroup, at most: what its registers hold. A wave keeps the
// queries of one tile and the outputs of all of them for its share of the columns.
constexpr int row_tiles(int dim) { return dim == 512 ? 2 : 4; }
constexpr int waves(int dim) { return 2 * row_tiles(dim); }
constexpr int kRowTile = 32;
constexpr int kKeys = 64;  // keys of a unit

// A row's weights are 2^(score - m), m its running maximum (in log2) less kAbove,
// which follows the scores when they pass it by kAbove + kSlack (see attn::Types).
// Moving one row's here stops its workgroup, so that float16 gives two of its bits
// for fewer moves: a weight counts down to 2^-34 of the largest, 23 below it in e.
template <typename T>
struct Soft {
  static constexpr float kSlack = 8.0f, kAbove = 0.0f;
};
template <>
struct Soft<_Float16> {
  static constexpr float kSlack = 6.0f, kAbove = 9.0f;
};

// What the split kernel leaves for the joining kernel: the schedule's prefix
// sums, and per partial segment the running maximum (less Soft::kAbove) and sum
// of each of its rows and their unnormalised outputs. Workgroup w has segments 2 w
// (the one its range starts with) and 2 w + 1 (a later one that its range ends in).
// The outputs lie as the lanes hold them, so that both kernels' accesses are whole
// lines: 32 columns of a row tile are a block of four times 64 lanes' four floats.
struct Parts {
  int64_t* base;  // [B + 1] first unit of each request, then the total
  float* m;       // [2 * wgs][rows]
  float* l;
  float* o;       // [2 * wgs][rows / kRowTile][L / 32][4][kWave][4]
  int wgs;        // workgroups of the split kernel
  int rows;       // rows of a segment, at most
};

// Units that a segment counts for before its first: its start and end (queries in,
// outputs out) take as long as some tiles do. In equal shares of the units alone, the
// workgroups with two segments were last, by 13 us (16 trees of up to 17 rows, 32
// heads, 8 bits, both kernels: 144 us; with 2, 4, 6, 8 units a segment 126, 121, 114,
// 120).
constexpr int kSetup = 6;

// Rows of a request: m = j * heads + h for row j and head h, in tiles of kRowTile,
// up to row_tiles(L) tiles to a segment.
struct Shape {
  int len, prefix, c0;
  int mrows, mtiles;
  int nseg, per;  // segments side by side, tiles of each
  int keys;
  int nku;        // units along the keys
  __device__ int64_t units() const { return (int64_t)nseg * (nku + kSetup); }
};

// Whether a request's rows are well formed (its tree and pages apart); their
// place and its prefix.
__device__ inline bool rows_of(const ReqView& q, int page_shift, int r, int total_eff, int* c0,
                               int* len, int* prefix) {
  const bool ok = request_rows(q, r, total_eff, c0, len);
  *prefix = q.prefix[r];
  const int64_t keys = (int64_t)*prefix + *len;
  // (cache indices in 32 bits, a unit beyond included)
  return ok && *prefix >= 0 && keys <= ((int64_t)q.width << page_shift) && keys <= 0x7FFFFF00LL;
}

template <int L>
__device__ inline Shape shape_of(int heads, int c0, int len, int prefix) {
  Shape s;
  s.c0 = c0;
  s.len = len;
  s.prefix = prefix;
  s.keys = prefix + len;
  s.mrows = heads * len;
  s.mtiles = (s.mrows + kRowTile - 1) / kRowTile;
  s.nseg = (s.mtiles + row_tiles(L) - 1) / row_tiles(L);
  s.per = (s.mtiles + s.nseg - 1) / s.nseg;
  s.nku = (s.keys + kKeys - 1) / kKeys;
  return s;
}

template <int L>
__device__ inline int64_t units_of(int heads, int c0, int len, int prefix) {
  return shape_of<L>(heads, c0, len, prefix).units();
}

// Workgroups that get units. A unit each where there are few: the launch is then one
// tile's latency (a context of 1500 at 32 heads: 18.2 us; two units each, 19.5).
__device__ inline int wgs_in_use(int64_t total, int wgs) { return (int)min((int64_t)wgs, total); }

// Workgroups go to the eight XCDs in turn. Shares are numbered so that an XCD's
// are consecutive: the segments of a request then meet in one L2.
constexpr int kXcds = 8;
__device__ inline int share_of(int wg, int wgs) {
  return wgs % kXcds ? wg : wg % kXcds * (wgs / kXcds) + wg / kXcds;
}

// The first unit of share w of n <= total. (A division in 64 bits is a hundred
// instructions, which a workgroup's start would fetch.)
__device__ inline int64_t wg_start(int64_t total, int w, int n) {
  const int64_t x = total * w;
  return x >> 32 ? x / n : (int64_t)((unsigned)x / (unsigned)n);
}

// LDS of a workgroup. A tile is kKeys latents in 16 bits and their rotated parts,
// unpadded; 16-byte chunk c of latent row r lies at chunk c ^ swizzle(r), so that
// the rows which a wave reads at one column, and the eight rows whose columns it
// reads transposed, spread over all banks.
//   16-bit caches: a ring of kStages tiles, filled straight from memory.
//   8-bit caches: the same ring of codes, with the rows' exponents; a code becomes a
//   16-bit operand between the products that read it (four conversions to a product
//   take no time of their own: 34 cycles instead of 32). Widened into a tile of its
//   own first, 16 trees of up to 17 rows took 160 us instead of 144.
template <bool E8, int L>
struct Ring {
  static constexpr int CB = E8 ? 1 : 2;
  static constexpr int W = waves(L);
  static constexpr int kOwn = kKeys / W;  // keys of a tile that a wave copies
  static constexpr int kMaxRows = row_tiles(L) * kRowTile;
  static constexpr int kRow = CB * L;
  static constexpr int kLat = kKeys * kRow;
  static constexpr int kGroups = L / kLatGroup;  // exponents of a row
  static constexpr int kTurned = kKeys * kRope * 2;
  static constexpr int kChunks = L * CB / 16;  // of a cache row
  static constexpr int kRowsPerCopy = kWave / kChunks;
  static constexpr int kCopies = kOwn / kRowsPerCopy;
  static constexpr int kTurnedCopies = kOwn / 8;
  static_assert(kCopies * kRowsPerCopy == kOwn && kOwn <= 16, "whole copies of one page");
  static constexpr int kPerWave = kCopies + kTurnedCopies + (E8 ? 1 : 0);
  static constexpr int kPowers = kLat;  // in a stage: exponents, 64 bytes a wave; 8 bits
  static constexpr int kTurnedAt = kLat + (E8 ? W * 64 : 0);
  static constexpr int kStage = kTurnedAt + kTurned;
  static constexpr int kStages = L == 512 && !E8 ? 2 : 3;
  static constexpr int kRing = 0;  // offset of the ring
  // weights in 16 bits: [row][kKeys], 16-byte chunks c of row r at c ^ (r >> 1 & 7)
  static constexpr int kWeights = kRing + kStages * kStage;
  // of the waves' rows: largest score, or sum, of each half of the keys
  static constexpr int kHalves = kWeights + kMaxRows * kKeys * 2;
  static constexpr int kFix = kHalves + 2 * kMaxRows * 4;  // and what their outputs shrink by
  static constexpr int kFlag = kFix + kMaxRows * 4;        // some maximum moves; of two tiles
  // rows with NaN or infinity, kOwn bits for each wave
  static constexpr int kOdd = kFlag + 8;
  // up to kWave requests' rows, 3 words each, or, where they are more, bits of those
  // that are left out for rows of others (see split_kernel)
  static constexpr int kReqs = kOdd + 8;
  static constexpr int kReqBytes =
      12 * kWave > DSPARK_MAX_BATCH / 8 ? 12 * kWave : DSPARK_MAX_BATCH / 8;
  // what a key's weights lose in exponent, 16 bits a key for each wave; 8 bits
  static constexpr int kDown = kReqs + kReqBytes;
  static constexpr int kBytes = kDown + (E8 ? W * kKeys * 2 : 0);
  static_assert(kStage % 256 == 0 && kDown % 16 == 0, "a swizzle is an exclusive or of addresses");
  static_assert(kBytes <= 163840 - 256, "a CU's LDS");
  static __device__ int swizzle(int row) {
    return E8 ? (row & 3) << 1 | (row & 8) | ((row >> 2) & 1)
              : (row & 3) << 2 | ((row >> 2) & 3);
  }
  static __device__ int turned_swizzle(int row) { return (row >> 1) & 7; }
};

// One segment: the queries of several row tiles of one request over some units of
// its keys. What the copies need of it,
struct Span {
  int r;
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

// Whether request r's bit of the words at `bits` in LDS is set.
__device__ __forceinline__ bool left_out(unsigned bits, int r) {
  return (lds_read<unsigned>(bits + (r >> 5) * 4) >> (r & 31)) & 1;
}

// The next segment of a share. `reqs`: the requests' rows in LDS where a wave's
// lanes hold the batch (len 0: left out); otherwise they are read from memory, and
// there are the bits of those that are left out though they are well formed.
template <int L>
__device__ __forceinline__ Span next_span(const LatentAttnArgs& a, unsigned reqs, Cursor& c,
                                          Job* job) {
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
      if (!rows_of(a.req, a.kv.page_shift, c.r, total_eff, &c0, &len, &prefix) ||
          left_out(reqs, c.r))
        len = 0;
    }
    c0 = __builtin_amdgcn_readfirstlane(c0);
    len = __builtin_amdgcn_readfirstlane(len);
    prefix = __builtin_amdgcn_readfirstlane(prefix);
    const Shape s = shape_of<L>(a.num_heads, c0, len, prefix);
    if (c.off >= (len ? s.units() : 0)) {
      ++c.r;
      c.off = 0;
      continue;
    }
    // (off < 2^9 segments of less than 2^26: the estimate is one off at most)
    const int stride = s.nku + kSetup;
    int seg = (int)((float)c.off * __builtin_amdgcn_rcpf((float)stride));
    seg += (int64_t)(seg + 1) * stride <= c.off ? 1 : 0;
    seg = __builtin_amdgcn_readfirstlane(seg - ((int64_t)seg * stride > c.off ? 1 : 0));
    const int within = (int)(c.off - (int64_t)seg * stride);
    const int n = __builtin_amdgcn_readfirstlane((int)min((int64_t)(stride - within), c.left));
    c.off += n;
    c.left -= n;
    const int ku0 = max(within - kSetup, 0);
    j.n = n - max(kSetup - within, 0);
    if (j.n <= 0) {
      j.n = 0;
      continue;
    }
    j.r = c.r;
    j.first = ku0 * kKeys;
    j.keys = s.keys;
    if (job) {
      job->s = s;
      job->tile0 = seg * s.per;
      job->mt = min(s.per, s.mtiles - job->tile0);
      job->whole = j.n == s.nku;
      job->slot = 2 * c.share + c.begun;
    }
    c.begun = 1;
    break;
  }
  return j;
}

// The producing side of the ring: this wave's copies of the next tile.
template <bool E8, int L>
struct Feeder {
  typedef Ring<E8, L> R;
  typedef unsigned long long u64;
  Cursor c;
  Span j, nj;      // the segment copied from, and the one after it
  int t;           // its tile in lane 0 of `ids`
  int idx, end;    // next lane, lanes that hold a tile: 0 when nothing is left
  int ids, nids;   // pages of the wave's rows: of j from tile t on, of nj from its first
  u64 bad, nbad;   // bit l: some page of lane l's tile is none
  int stage;
  unsigned none;   // bit per stage: some page of its tile is none

  // The pages of 64 tiles of x from tile t on, a tile to a lane: the loads,
  struct Pages {
    int id[kKeys / 16];
  };
  static __device__ __forceinline__ Pages ask(const LatentAttnArgs& a, const Span& x, int t) {
    Pages p;
    const int64_t first = (int64_t)x.first + (int64_t)(t + lane_id()) * kKeys;
#pragma unroll
    for (int g = 0; g < kKeys / 16; ++g)
      p.id[g] = a.req.table[(size_t)x.r * a.req.width +
                            ((int)min(first + g * 16, (int64_t)x.keys - 1) >> a.kv.page_shift)];
    return p;
  }
  // and what the wave keeps of them.
  static __device__ __forceinline__ int take(const LatentAttnArgs& a, const Pages& p, int wave,
                                             u64* bad) {
    int own = 0;
    u64 b = 0;
#pragma unroll
    for (int g = 0; g < kKeys / 16; ++g) {
      const bool none = p.id[g] < 0 || p.id[g] >= a.kv.num_blocks;
      b |= __ballot(none);
      // a page that is none: any valid one, its keys are masked
      if (g == wave * R::kOwn / 16) own = none ? 0 : p.id[g];
    }
    *bad = b;
    settle(own);
    return own;
  }

  // Of the share's first segment, at whose end `after` is.
  __device__ __forceinline__ void start(const LatentAttnArgs& a, const Span& first,
                                        const Cursor& after, const Pages& p, int wave) {
    c = after;
    j = first;
    ids = take(a, p, wave, &bad);
    t = idx = stage = 0;
    end = __builtin_amdgcn_readfirstlane(min(j.n, kWave));
    none = 0;
    nj.n = 0;
    nids = 0;
    nbad = 0;
  }
  // The segment after it: its pages are asked for, and taken later.
  __device__ __forceinline__ Pages look_ahead(const LatentAttnArgs& a, unsigned lds) {
    nj = next_span<L>(a, lds + R::kReqs, c, nullptr);
    Pages p;
#pragma unroll
    for (int g = 0; g < kKeys / 16; ++g) p.id[g] = 0;
    if (nj.n > 0) p = ask(a, nj, 0);
    return p;
  }

  // The wave's copies of the next tile: begin(), each of the kPerWave copies once, so
  // that they can go out between products, and end(). Where no tile is left, the
  // last one's go out once more, into a stage that nobody reads.
  const unsigned char *from, *turned, *exps;
  unsigned at;
  __device__ __forceinline__ void begin(const LatentAttnArgs& a, unsigned lds, int wave) {
    at = lds + R::kRing + stage * R::kStage;
    if (end == 0) return;
    const int64_t id = __builtin_amdgcn_readlane(ids, idx);
    const int key = j.first + (t + idx) * kKeys + wave * R::kOwn;
    const int off = key & ((1 << a.kv.page_shift) - 1);
    from = uniform(a.kv.latent + id * a.kv.page_bytes + off * (L * R::CB));
    turned = uniform(a.kv.rope + id * a.kv.rope_page_bytes + off * (kRope * 2));
    if constexpr (E8)
      exps = uniform(a.kv.scale + id * a.kv.scale_page_bytes + off * (L / kLatGroup));
  }

  template <int N>
  __device__ __forceinline__ void copy(int wave) {
    const int lane = lane_id(), row0 = wave * R::kOwn;
    if constexpr (N < R::kCopies) {
      const int r = N * R::kRowsPerCopy + lane / R::kChunks;
      const int chunk = (lane % R::kChunks) ^ R::swizzle(row0 + r);
      copy16_shared(from + N * R::kRowsPerCopy * L * R::CB,
                    (lane / R::kChunks) * L * R::CB + (unsigned)chunk * 16,
                    at + row0 * R::kRow + N * 1024);
    } else if constexpr (N < R::kCopies + R::kTurnedCopies) {
      constexpr int n = N - R::kCopies;
      copy16_shared(turned + n * 1024,
                    (lane & ~7) * 16 +
                        (((lane & 7) ^ R::turned_swizzle(row0 + n * 8 + (lane >> 3))) << 4),
                    at + R::kTurnedAt + row0 * (kRope * 2) + n * 1024);
    } else {
      constexpr int kBytes = R::kOwn * (L / kLatGroup);
      if (lane < kBytes / 4) copy4(exps, lane * 4, at + R::kPowers + wave * 64);
    }
  }

  // end_tile() before the segment's last tile, and before any page is known to be none
  __device__ __forceinline__ void end_tile_within() {
    none = (none & ~(1u << stage)) | ((unsigned)(bad >> idx) & 1u) << stage;
    stage = stage + 1 == R::kStages ? 0 : stage + 1;
    ++idx;
  }
  __device__ __forceinline__ void end_tile(const LatentAttnArgs& a, unsigned lds, int wave) {
    if (end == 0) return;
    if (__builtin_expect((bad | none) != 0, 0))
      none = (none & ~(1u << stage)) | ((unsigned)(bad >> idx) & 1u) << stage;
    stage = stage + 1 == R::kStages ? 0 : stage + 1;
    if (__builtin_expect(++idx == end, 0)) {
      t += end;
      idx = 0;
      const bool more = t < j.n;
      if (!more) {
        j = nj;
        ids = nids;
        bad = nbad;
        t = 0;
        if (j.n > 0) nj = next_span<L>(a, lds + R::kReqs, c, nullptr);
      }
      Span x = nj;
      if (more) x = j;
      if (more || (j.n > 0 && nj.n > 0)) {
        u64 b;
        const int got = take(a, ask(a, x, t), wave, &b);
        if (more) {
          ids = got;
          bad = b;
        } else {
          nids = got;
          nbad = b;
        }
      }
      end = __builtin_amdgcn_readfirstlane(min(j.n - t, kWave));
    }
  }

  template <int N = 0>
  __device__ __forceinline__ void copies(int wave) {
    copy<N>(wave);
    if constexpr (N + 1 < R::kPerWave) copies<N + 1>(wave);
  }
};

// o *= fix for outputs that stay in the accumulation registers. As plain code the
// product would come out in other registers, and every step of the loop would move
// all outputs between the two (1 KB a lane, and spills). No product that writes o
// is under way here: the scores' products, which are later ones, have been read.
// The waits are those between a write of a register and its read as an operand.
__device__ inline void shrink(f32x16& o, float fix) {
#pragma unroll
  for (int e = 0; e < 16; ++e) {
    float x = o[e], y;
    asm volatile(
        "v_accvgpr_read_b32 %1, %0\n\ts_nop 1\n\tv_mul_f32 %1, %1, %2\n\ts_nop 1\n\t"
        "v_accvgpr_write_b32 %0, %1\n\ts_nop 1"
        : "+a"(x), "=&v"(y)
        : "v"(fix));
    o[e] = x;
  }
}

// Four times four columns of a row, 8 apart, less those that lane ^ 32 has, to memory:
// the two lanes swap halves, so that each stores eight in a row.
template <typename T>
__device__ inline void store_columns(T* row, const float (&y)[16]) {
  typedef typename Types<T>::V8 V8;
  const int hi = lane_id() >> 5;
#pragma unroll
  for (int x = 0; x < 4; x += 2) {
    V8 z;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float mine = hi ? y[4 * x + 4 + e] : y[4 * x + e];
      const float other = __shfl_xor(hi ? y[4 * x + e] : y[4 * x + 4 + e], 32, kWave);
      z[e] = (T)(hi ? other : mine);
      z[4 + e] = (T)(hi ? mine : other);
    }
    *reinterpret_cast<V8*>(row + (x + hi) * 8) = z;
  }
}

// Eight codes of a row or column and their exponent's power of two as an operand.
template <typename V8>
__device__ __forceinline__ V8 widen(unsigned x, unsigned y, float power) {
  kv_u32x4 z;
  z[0] = __builtin_bit_cast(unsigned, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(x, power, false));
  z[1] = __builtin_bit_cast(unsigned, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(x, power, true));
  z[2] = __builtin_bit_cast(unsigned, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(y, power, false));
  z[3] = __builtin_bit_cast(unsigned, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(y, power, true));
  return __builtin_bit_cast(V8, z);
}

// What lane l meets in step N of six that bring a maximum of all lanes into the last:
// neighbours in a pair and in a quad, mirrors of 8 and 16 lanes, the row and the half
// before.
template <int N>
__device__ __forceinline__ int across(int x) {
  constexpr int kSteps[6] = {0xB1, 0x4E, 0x141, 0x140, 0x142, 0x143};
  return __builtin_amdgcn_update_dpp(x, x, kSteps[N], 0xF, 0xF, false);
}

template <int N>
struct Index {
  static constexpr int value = N;
};

// A segment: some row tiles over some units of the keys, which the waves bring into
// LDS together. (Tiles without rows, and those of a request whose tree is none, are
// computed and not written.) Wave (t, half) = (wave / 2, wave % 2) has row tile t and
// half the keys of a tile for the scores, and a share of the columns for the outputs:
//   S^T = K Q^T: keys are its rows and queries its columns, so a lane holds the
//   scores of one query (lane & 31) for sixteen keys, four in a row each. Its
//   weights go to LDS as the operand of
//   O^T = C^T P^T, whose C^T (the same latents) comes transposed out of LDS in that
//   order of keys. Every wave reads all rows' weights and its columns of the tile.
// The rows' running maximum is kept by both waves of a row tile. It moves when some
// score passes it by Soft::kSlack: a wave that sees one raises a flag, and then the
// halves' maxima meet in LDS, the weights are taken again and the outputs shrink.
template <typename T, bool E8, int L>
__device__ __forceinline__ void segment(const LatentAttnArgs& a, const Parts& ws, const Span& span,
                                        const Job& job, bool first, Cursor after, Feeder<E8, L>& feed,
                                        unsigned lds, int& stage, int& tick) {
  typedef Types<T> TT;
  typedef typename TT::V8 V8;
  typedef typename TT::V4 V4;
  typedef Ring<E8, L> R;
  constexpr int NL = L / 16, NF = NL + kRope / 16;  // operand chunks of a latent, of a key
  constexpr int NT = row_tiles(L);
  constexpr int ND = L / 32 / R::W;                 // 32-column tiles of a wave's outputs
  constexpr int kOwn = R::kOwn;
  const Shape& s = job.s;
  const int lane = lane_id(), qi = lane & 31, hi = lane >> 5;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int tile = wave >> 1, half = wave & 1;
  const int len = s.len, prefix = s.prefix, keys = s.keys;
  const int m = (job.tile0 + tile) * kRowTile + qi;
  const int qrow = m / a.num_heads;  // the request's row that the lane's query belongs to

  // A share's first segment starts the ring. What it reads is asked for in one go:
  // its pages, its rows' parents, its queries; then the first tiles; then the next
  // segment's pages.
  typename Feeder<E8, L>::Pages pages;
  if (first) pages = feed.ask(a, span, 0);
  int up = 0;
  if (a.req.parents && lane + 1 < len)
    up = a.req.parents[(size_t)span.r * a.req.gamma + lane];
  // Scores in units of log2 with a positive factor, so that a masked score stays
  // -infinity under it: the scale's sign and its zero go into the queries.
  float sl = fminf(fabsf(a.scale) * kLog2e, 3.4028235e38f);
  const bool flat = sl == 0.0f;
  if (flat) sl = 1.0f;
  const unsigned sign = a.scale < 0.0f ? 0x80008000u : 0u;
  // queries as operands
  V8 qf[NF];
  f32x16 o[NT][ND];
  float mx = -__builtin_inff(), l = 0.0f;
  {
    // Loaded with four lanes to 64 bytes of a row, so that a line is asked for once
    // (a lane per row and 16 bytes: 6.5 us instead of 2 for a segment), and turned
    // through the wave's part of the weights' place. LDS keeps the order of a wave's
    // accesses.
    kv_u32x4 w[NF];
    const int row4 = lane >> 2, chunk = lane & 3;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int mm = (job.tile0 + tile) * kRowTile + row4 + 16 * i;
      const int r = mm / a.num_heads, head = mm - r * a.num_heads;
      const bool there = tile < job.mt && mm < s.mrows && !flat;
      const size_t row = (size_t)(s.c0 + r);
      const unsigned char* ql = a.ql + row * a.ql_ld + head * a.ql_head_ld + chunk * 16;
      const unsigned char* qr = a.qr + row * a.qr_ld + head * a.qr_head_ld + chunk * 16;
      // (one branch for all: a use of a value in it would wait for each load)
#pragma unroll
      for (int f = i; f < NF; f += 2) w[f] = (kv_u32x4){0, 0, 0, 0};
      if (there) {
#pragma unroll
        for (int f = i; f < NF; f += 2)
          w[f] = *reinterpret_cast<const kv_u32x4*>(f < NL ? ql + (f - i) * 32
                                                           : qr + (f - i - NL) * 32);
      }
    }
    bool second = false;
    if (first) {
      feed.start(a, span, after, pages, wave);
      feed.begin(a, lds, wave);
      feed.copies(wave);
      pages = feed.look_ahead(a, lds);
      second = R::kStages > 2 && span.n > 1;
      if (second) {
        feed.end_tile_within();
        feed.begin(a, lds, wave);
        feed.copies(wave);
      }
    }
    // (a key's codes are read sixteen to a lane, for two products)
    const unsigned own = lds + R::kWeights + wave * 2048;
#pragma unroll
    for (int f = 0; f < NF; f += 2) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        settle(w[f + i]);
        const int r = row4 + 16 * i;
        lds_write(own + r * 64 + ((chunk ^ ((r >> 2) & 3)) << 4), w[f + i] ^ sign);
      }
#pragma unroll
      for (int i = 0; i < 2; ++i)
        qf[f + i] = lds_read<V8>(
            own + qi * 64 +
            (((E8 && f < NL ? 2 * hi + i : 2 * i + hi) ^ ((qi >> 2) & 3)) << 4));
    }
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int d = 0; d < ND; ++d)
#pragma unroll
        for (int e = 0; e < 16; ++e) o[t][d][e] = 0.0f;
    if (first) {
      if (feed.nj.n > 0) feed.nids = feed.take(a, pages, wave, &feed.nbad);
      feed.end_tile(a, lds, wave);
      if (R::kStages > 2 && !second) {
        feed.begin(a, lds, wave);
        feed.copies(wave);
        feed.end_tile(a, lds, wave);
      }
    }
  }
  // rows of the step's own tree that the lane's query sees, bit l for row l + 1;
  // row 0 is everybody's. Bit l of anc, in lane l, is row l + 1 itself, with its
  // ancestors' bits.
  unsigned long long seen = qrow >= 64 ? ~0ull : (1ull << qrow) - 1;
  bool good = true;  // the parents are a tree's
  if (a.req.parents) {
    settle(up);
    good = __ballot(up < 0 || up > lane) == 0;
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

  // lane's offsets in a tile: its chunk of a latent and of a rotated part (of its
  // wave's half of the keys), its piece of a row that is read for its columns
  const int key_row = half * 32 + qi;
  const int lat_at = key_row * R::kRow + ((hi ^ R::swizzle(key_row)) << 4);
  const int turned_at = key_row * (kRope * 2) + ((hi ^ R::turned_swizzle(key_row)) << 4);
  const int t4 = lane & 15;
  // (a swizzle changes bits 4 to 7 of an address: what lies above is a sum)
  int val_at;
  if constexpr (E8) {
    const int vrow = (t4 >> 3) * 8 + hi * 4 + ((t4 >> 1) & 3);
    val_at = vrow * R::kRow +
             ((((lane >> 4) & 1) + (wave * ND * 2 & 15)) ^ R::swizzle(vrow)) * 16 + (t4 & 1) * 8 +
             (wave * ND * 2 >> 4) * 256;
  } else {
    const int vrow = hi * 4 + (t4 >> 2);
    val_at = vrow * R::kRow +
             (((((lane >> 4) & 1) * 2 + ((t4 >> 1) & 1) + (wave * ND & 3) * 4) ^ R::swizzle(vrow))
              << 4) +
             (t4 & 1) * 8 + (wave * ND >> 2) * 256;
  }
  // its chunk of the weights of row lane & 31 of a row tile
  const unsigned weight_at = lds + R::kWeights + qi * (kKeys * 2) + ((hi ^ ((qi >> 1) & 7)) << 4);
  // a word of its row in the row statistics
  const unsigned row_at = (tile * kRowTile + qi) * 4;
  // in 8 bits: the exponents of its row of keys; that of key `lane` for the wave's
  // columns; and where key `lane` stands among the weights
  const int powers_at = R::kPowers + key_row / kOwn * 64 + key_row % kOwn * R::kGroups;
  const int power_at =
      R::kPowers + lane / kOwn * 64 + lane % kOwn * R::kGroups + wave * ND * 32 / kLatGroup;
  const unsigned down = lds + R::kDown + wave * (kKeys * 2);
  const unsigned down_at =
      down + ((lane >> 4) * 16 + ((lane >> 2) & 1) * 8 + ((lane >> 3) & 1) * 4 + (lane & 3)) * 2;

  for (int i = 0; i < span.n; ++i) {
    const int key0 = span.first + i * kKeys;
    // 16-key groups on a page that is none
    unsigned missing = 0;
    if (__builtin_expect((feed.none >> stage) & 1, 0)) {
#pragma unroll
      for (int b = 0; b < kKeys / 16; ++b) {
        const int p = min(key0 + 16 * b, keys - 1) >> a.kv.page_shift;
        int id = a.req.table[(size_t)span.r * a.req.width + p];
        settle(id);
        if (id < 0 || id >= a.kv.num_blocks) missing |= 1u << b;
      }
      missing = __builtin_amdgcn_readfirstlane(missing);
    }
    // the tile holds keys that some query does not see (the request's own rows
    // after its root, keys past its last), or such a group
    const bool edge = key0 + kKeys > prefix + 1 || missing;
    const unsigned raw = lds + R::kRing + stage * R::kStage;
    const unsigned turned = raw + R::kTurnedAt;
    const int row0 = wave * kOwn;  // of the wave's keys
    // The wave's rows that hold nothing for some query, as bits: keys that do not
    // exist (anything may be there), and rows with a NaN or infinite element, which
    // must not meet a zero weight. They become zeros; queries that see one of the
    // latter get a NaN score below instead. `strange`: rows with such elements.
    auto hide = [&](unsigned strange) {
      unsigned there = 0;
#pragma unroll
      for (int x = 0; x < kOwn; ++x)
        if (key0 + row0 + x < keys && !((missing >> ((row0 + x) >> 4)) & 1)) there |= 1u << x;
      if (lane == 0) {
        if constexpr (kOwn == 8) {
          lds_write<unsigned char>(lds + R::kOdd + wave, (unsigned char)(strange & there));
        } else {
          lds_write<unsigned short>(lds + R::kOdd + 2 * wave, (unsigned short)(strange & there));
        }
      }
      return strange | (~there & ((1u << kOwn) - 1));
    };
    // rows that a ballot over lanes names, `chunks` lanes a row
    auto rows_in = [&](unsigned long long found, int chunks, int first) {
      unsigned rows = 0;
      while (found) {
        rows |= 1u << (first + (int)__builtin_ctzll(found) / chunks);
        found &= found - 1;
      }
      return rows;
    };
    auto strange16 = [&](const kv_u32x4& w) {
      bool bad = false;
#pragma unroll
      for (int x = 0; x < 4; ++x)
        bad |= (w[x] & TT::kExpMask) == TT::kExpMask ||
               (w[x] >> 16 & TT::kExpMask) == TT::kExpMask;
      return bad;
    };
    const unsigned own_turned = turned + row0 * (kRope * 2) + lane * 16;
    auto strange_turned = [&]() {
      unsigned rows = 0;
#pragma unroll
      for (int n = 0; n < R::kTurnedCopies; ++n)
        rows |= rows_in(__ballot(strange16(lds_read<kv_u32x4>(own_turned + n * 1024))), 8, n * 8);
      return rows;
    };
    auto hide_turned = [&](unsigned hidden) {
#pragma unroll
      for (int n = 0; n < R::kTurnedCopies; ++n)
        if ((hidden >> (n * 8 + (lane >> 3))) & 1)
          lds_write(own_turned + n * 1024, (kv_u32x4){0, 0, 0, 0});
    };
    // this tile's copies are done when those of the stages after it may not be
    wait_copies<(R::kStages - 2) * R::kPerWave>();
    const unsigned buf = raw;
    if (edge) {
      const unsigned own = buf + row0 * R::kRow + lane * 16;
      unsigned strange = strange_turned();
#pragma unroll
      for (int n = 0; n < R::kCopies; ++n) {
        const kv_u32x4 w = lds_read<kv_u32x4>(own + n * 1024);
        bool bad = false;
        if constexpr (E8) {
#pragma unroll
          for (int x = 0; x < 4; ++x)
#pragma unroll
            for (int y = 0; y < 32; y += 8) bad |= ((w[x] >> y) & 0x7Fu) == 0x7Fu;
        } else {
          bad = strange16(w);
        }
        strange |= rows_in(__ballot(bad), R::kChunks, n * R::kRowsPerCopy);
      }
      if constexpr (E8) {
        // (no row that append writes has an exponent byte above 246; a code may
        // pass every finite number under it)
        const bool bad = lane < kOwn * R::kGroups &&
                         lds_read<unsigned char>(buf + R::kPowers + wave * 64 + lane) > 246;
        strange |= rows_in(__ballot(bad), R::kGroups, 0);
      }
      const unsigned hidden = hide(strange);
      hide_turned(hidden);
#pragma unroll
      for (int n = 0; n < R::kCopies; ++n)
        if ((hidden >> (n * R::kRowsPerCopy + lane / R::kChunks)) & 1)
          lds_write(own + n * 1024, (kv_u32x4){0, 0, 0, 0});
      if constexpr (E8) {
        if (lane < kOwn * R::kGroups && ((hidden >> (lane / R::kGroups)) & 1))
          lds_write<unsigned char>(buf + R::kPowers + wave * 64 + lane, 127);
      }
    }
    barrier();
    feed.begin(a, lds, wave);
    stage = stage + 1 == R::kStages ? 0 : stage + 1;
    const unsigned flag = lds + R::kFlag + tick * 4, other_flag = lds + R::kFlag + (tick ^ 1) * 4;
    tick ^= 1;
    if (wave == 0 && lane == 0) lds_write<unsigned>(other_flag, 0u);

    f32x16 sc;
    float top = -__builtin_inff();
    V8 pf[2];
    // in 8 bits, of the wave's columns: key `lane`'s exponent byte, the tile's largest
    int own_power = 0, top_power = 0;
    // The product takes weights of the query type, each off by up to half its step;
    // their sum takes them as they are.
    auto weigh = [&](float* sum) {
      const float ref = mx == -__builtin_inff() ? 0.0f : mx;
      *sum = 0.0f;
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        const float p = __builtin_amdgcn_exp2f(sc[e] * sl - ref);
        *sum += p;
        pf[e >> 3][e & 7] = (T)p;
      }
#pragma unroll
      for (int c = 0; c < 2; ++c)
        lds_write((weight_at ^ ((half * 2 + c) << 5)) + tile * (kRowTile * kKeys * 2), pf[c]);
    };
    float sum = 0.0f;
    {
      // Scores, in two sums by turns: a product waits for the one before it in its own
      // sum (36 in one sum: 44 cycles each, in two 32). Between the products go the
      // reads of operands kAhead products later and the copies of the next tile.
      f32x16 s2;
#pragma unroll
      for (int e = 0; e < 16; ++e) sc[e] = s2[e] = 0.0f;
      constexpr int kAhead = 6;
      unsigned ka[8], ta = turned + turned_at;
      {
        unsigned at = buf + lat_at;
        settle(at);
#pragma unroll
        for (int f = 0; f < 8; ++f) ka[f] = at ^ (f << 5);
        settle(ta);
      }
      V8 kf[kAhead + 1], now;
      kv_u32x4 kc[kAhead / 2 + 1];  // codes
      float power[R::kGroups];
      auto read_key = [&](int f) {
        if (f >= NL) {
          kf[f % (kAhead + 1)] = lds_read<V8>(ta ^ ((f - NL) << 5));
        } else if constexpr (E8) {
          if (f % 2 == 0)
            kc[f / 2 % (kAhead / 2 + 1)] =
                lds_read<kv_u32x4>(ka[(f >> 1) & 7] + (f >> 4) * 256);
        } else {
          kf[f % (kAhead + 1)] = lds_read<V8>(ka[f & 7] + (f >> 3) * 256);
        }
      };
      auto operand = [&](int f) {
        if (E8 && f < NL) {
          const kv_u32x4 c = kc[f / 2 % (kAhead / 2 + 1)];
          return widen<V8>(c[f % 2 * 2], c[f % 2 * 2 + 1], power[f * 16 / kLatGroup]);
        }
        return kf[f % (kAhead + 1)];
      };
      if constexpr (E8) {
        own_power = lds_read<unsigned char>(raw + power_at);
        const unsigned x = R::kGroups == 4 ? lds_read<unsigned>(raw + powers_at)
                                           : lds_read<unsigned short>(raw + powers_at);
#pragma unroll
        for (int g = 0; g < R::kGroups; ++g)
          power[g] = __builtin_bit_cast(float, ((x >> (8 * g)) & 255u) << 23);
      }
#pragma unroll
      for (int f = 0; f < kAhead; ++f) read_key(f);
      now = operand(0);
      auto step = [&](auto self, auto at) {
        constexpr int f = decltype(at)::value;
        if constexpr (f + kAhead < NF) read_key(f + kAhead);
        __builtin_amdgcn_sched_barrier(0);
        if constexpr (f & 1) {
          s2 = TT::mfma32(now, qf[f], s2);
        } else {
          sc = TT::mfma32(now, qf[f], sc);
        }
        if constexpr (f + 1 < NF) now = operand(f + 1);
        // (a step of the largest exponent's way through the wave behind each product)
        if constexpr (E8 && f < 8) {
          if constexpr (f == 1) top_power = own_power;
          if constexpr (f >= 2) top_power = max(top_power, across<f - 2>(top_power));
        }
        // copy n goes out behind product n * NF / kPerWave
        constexpr int n0 = (f * R::kPerWave + NF - 1) / NF, n1 = ((f + 1) * R::kPerWave + NF - 1) / NF;
        if constexpr (n0 < n1) feed.template copy<n0>(wave);
        static_assert(n1 - n0 <= 1, "a copy to a product");
        __builtin_amdgcn_sched_barrier(0);
        if constexpr (f + 1 < NF) self(self, Index<f + 1>{});
      };
      step(step, Index<0>{});
      feed.end_tile(a, lds, wave);
#pragma unroll
      for (int e = 0; e < 16; ++e) sc[e] += s2[e];
      if (edge) {
        const unsigned odd = lds_read<unsigned>(lds + R::kOdd + half * 4);
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          const int k = 8 * (e >> 2) + 4 * hi + (e & 3);
          const int rel = key0 + half * 32 + k - prefix;
          const bool own = (rel < len) & ((int)(seen >> ((rel - 1) & 63)) & 1);
          const bool gone = ((missing >> (half * 2 + (e >> 3))) & 1) | ((rel > 0) & !own);
          sc[e] = gone ? -__builtin_inff() : ((odd >> k) & 1 ? __builtin_nanf("") : sc[e]);
        }
      }
      // Weights. The product with the scale rounds before the maximum is taken off,
      // so that the largest weight is 1 whatever the size of its score.
      top = sc[0];
#pragma unroll
      for (int e = 1; e < 16; ++e) top = fmaxf(top, sc[e]);
      top *= sl;
      if (__any(top - mx > Soft<T>::kAbove + Soft<T>::kSlack)) {
        if (lane == 0) lds_write<unsigned>(flag, 1u);
      } else {
        weigh(&sum);
      }
    }
    // Columns of the tile, the wave's share: operand k is 16 keys' (k / ND) of 32
    // columns. In 8 bits a column's keys have an exponent each, and the conversion
    // takes one for all: the tile's largest, and what a key's own is less its weights
    // lose, exactly, as an integer subtraction from their bits. (A weight of less than
    // a normal number's size after it is none; so a tile in which exponents are
    // kFar apart or more is taken in passes.)
    constexpr int NV = kKeys / 16 * ND, kVAhead = 3, kFar = 100;
    typedef unsigned short u16x8 __attribute__((ext_vector_type(8)));
    bool rest = false;  // key `lane` is left for another pass
    auto lower = [&]() {
      const int less = top_power - own_power;
      lds_write<unsigned short>(down_at, less < 0 || less > kFar ? 0xFFFF
                                                                 : (unsigned short)(less << 7));
      rest = less > kFar;
    };
    if constexpr (E8) {
      top_power = __builtin_amdgcn_readlane(top_power, kWave - 1);
      lower();
    }
    unsigned va[ND], wa = weight_at;
    {
      unsigned at = buf + val_at;
      settle(at);
#pragma unroll
      for (int d = 0; d < ND; ++d) va[d] = at ^ (d << (E8 ? 5 : 6));
      settle(wa);
    }
    V4 vl[kVAhead + 1], vh[kVAhead + 1];
    lds_i32x2 vc[kVAhead + 1];
    V8 pw[2][NT];
    u16x8 dw[2];
    auto read_value = [&](int k) {
      const int c = k / ND, d = k % ND;
      if constexpr (E8) {
        vc[k % (kVAhead + 1)] = lds_columns8(va[d] + c * 16 * R::kRow);
      } else {
        vl[k % (kVAhead + 1)] = lds_columns<V4>(va[d] + c * 16 * R::kRow);
        vh[k % (kVAhead + 1)] = lds_columns<V4>((va[d] ^ 32) + (c * 16 + 8) * R::kRow);
      }
    };
    auto read_weight = [&](int c, int t) {
      pw[c & 1][t] = lds_read<V8>((wa ^ (c << 5)) + t * (kRowTile * kKeys * 2));
      if (E8 && t == 0) dw[c & 1] = lds_read<u16x8>(down + (c * 2 + hi) * 16);
    };
    auto value = [&](int k) {
      if constexpr (E8) {
        const lds_i32x2 x = vc[k % (kVAhead + 1)];
        return widen<V8>(x[0], x[1], __builtin_bit_cast(float, top_power << 23));
      } else {
        return __builtin_shufflevector(vl[k % (kVAhead + 1)], vh[k % (kVAhead + 1)], 0, 1, 2, 3, 4,
                                       5, 6, 7);
      }
    };
    auto adjust = [&](int c, int t) {
      if constexpr (E8)
        pw[c & 1][t] = __builtin_bit_cast(
            V8, __builtin_elementwise_sub_sat(__builtin_bit_cast(u16x8, pw[c & 1][t]), dw[c & 1]));
    };
#pragma unroll
    for (int k = 0; k < kVAhead; ++k) read_value(k);
    barrier();
    const unsigned moved = lds_read<unsigned>(flag);
#pragma unroll
    for (int t = 0; t < NT; ++t) read_weight(0, t);
    if (__builtin_expect(moved != 0, 0)) {
      top = fmaxf(top, __shfl_xor(top, 32, kWave));
      if (hi == 0)
        lds_write<float>(lds + R::kHalves + half * (R::kMaxRows * 4) + row_at, top);
      barrier();
      {
        float next = fmaxf(top, lds_read<float>(lds + R::kHalves + (half ^ 1) * (R::kMaxRows * 4) +
                                                row_at));
        if (next - mx > Soft<T>::kAbove + Soft<T>::kSlack) {
          if constexpr (Soft<T>::kAbove > 0.0f) {
            // (not where kAbove rounds up to more than a weight may be)
            const float less = next - Soft<T>::kAbove;
            next = next - less > Soft<T>::kAbove + Soft<T>::kSlack ? next : less;
          }
          next = fmaxf(mx, next);
        } else {
          next = mx;
        }
        const float fix = next == -__builtin_inff() ? 1.0f : __builtin_amdgcn_exp2f(mx - next);
        mx = next;
        l *= fix;
        if (hi == 0 && half == 0) lds_write<float>(lds + R::kFix + row_at, fix);
        weigh(&sum);
      }
      barrier();
#pragma unroll
      for (int t = 0; t < NT; ++t) read_weight(0, t);
      if (i > 0) {  // (zeros before)
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          const float fix = lds_read<float>(lds + R::kFix + (t * kRowTile + qi) * 4);
#pragma unroll
          for (int d = 0; d < ND; ++d) {
            if constexpr (L == 512) {
              shrink(o[t][d], fix);
            } else {
              o[t][d] *= fix;
            }
          }
        }
      }
    }
    l += sum;
    // O^T += C^T P^T, the reads of operands kVAhead later between the products; the
    // first operands' reads are under way
    auto products = [&]() {
#pragma unroll
      for (int t = 0; t < NT; ++t) adjust(0, t);
      V8 vf = value(0);
#pragma unroll
      for (int k = 0; k < NV; ++k) {
        const int c = k / ND, d = k % ND;
        if (k + kVAhead < NV) read_value(k + kVAhead);
        if (c + 1 < kKeys / 16) {
          if (ND == 1) {
#pragma unroll
            for (int t = 0; t < NT; ++t) read_weight(c + 1, t);
          } else if (d < NT) {
            read_weight(c + 1, d);
          }
        }
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int t = 0; t < NT; ++t) o[t][d] = TT::mfma32(vf, pw[c & 1][t], o[t][d]);
        if (k + 1 < NV) vf = value(k + 1);
        if (c + 1 < kKeys / 16) {
          if (ND == 1) {
#pragma unroll
            for (int t = 0; t < NT; ++t) adjust(c + 1, t);
          } else if (d >= ND - NT) {
            adjust(c + 1, d - (ND - NT));
          }
        }
        __builtin_amdgcn_sched_barrier(0);
      }
    };
    static_assert(ND == 1 || ND >= 2 * NT, "weights are read before they are adjusted");
    if constexpr (!E8) {
      products();
    } else {
      for (;;) {
        products();
        if (__builtin_expect(!__any(rest), 1)) break;
        top_power = rest ? own_power : 0;
        top_power = max(top_power, across<0>(top_power));
        top_power = max(top_power, across<1>(top_power));
        top_power = max(top_power, across<2>(top_power));
        top_power = max(top_power, across<3>(top_power));
        top_power = max(top_power, across<4>(top_power));
        top_power = max(top_power, across<5>(top_power));
        top_power = __builtin_amdgcn_readlane(top_power, kWave - 1);
        lower();
#pragma unroll
        for (int k = 0; k < kVAhead; ++k) read_value(k);
#pragma unroll
        for (int t = 0; t < NT; ++t) read_weight(0, t);
      }
    }
    // (the next tile's first barrier comes before anything here is overwritten:
    // the weights, the statistics and, in 8 bits, the tile)
  }

  // the halves' sums meet
  l += __shfl_xor(l, 32, kWave);
  barrier();
  if (hi == 0) lds_write<float>(lds + R::kHalves + half * (R::kMaxRows * 4) + row_at, l);
  barrier();
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    if (!good || t >= job.mt) continue;
    const int mm = (job.tile0 + t) * kRowTile + qi;
    const bool there = mm < s.mrows;
    const unsigned at = lds + R::kHalves + (t * kRowTile + qi) * 4;
    const float sum = lds_read<float>(at) + lds_read<float>(at + R::kMaxRows * 4);
    if (job.whole) {
      const int row = mm / a.num_heads, head = mm - row * a.num_heads;
      const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
      T* dst = reinterpret_cast<T*>(a.out + (size_t)(s.c0 + row) * a.out_ld) + head * L +
               wave * (ND * 32);
#pragma unroll
      for (int d = 0; d < ND; ++d) {
        float y[16];
#pragma unroll
        for (int e = 0; e < 16; ++e) y[e] = o[t][d][e] * inv;
        if (there) store_columns(dst + d * 32, y);
      }
      if (a.lse && there && hi == 0 && wave == 2 * t)
        a.lse[(size_t)(s.c0 + row) * a.num_heads + head] =
            sum == 0.0f ? -__builtin_inff() : (mx + __builtin_amdgcn_logf(sum)) * kLn2;
    } else {
      const size_t part = (size_t)job.slot * ws.rows + t * kRowTile;
      float* dst = ws.o + part * L + wave * (ND * 32 * kRowTile) + lane * 4;
#pragma unroll
      for (int d = 0; d < ND; ++d)
#pragma unroll
        for (int x = 0; x < 4; ++x)
          *reinterpret_cast<f32x4*>(dst + (d * 4 + x) * (kWave * 4)) =
              (f32x4){o[t][d][4 * x], o[t][d][4 * x + 1], o[t][d][4 * x + 2], o[t][d][4 * x + 3]};
      if (hi == 0 && wave == 2 * t) {
        ws.m[part + qi] = mx;
        ws.l[part + qi] = sum;
      }
    }
  }
}

// out = sum_k e^(s_k - m) c_k / sum_k e^(s_k - m) in one pass over the cached rows,
// which are keys and values at once: running maximum m, sum and outputs in float32
// registers, m moved only when a score passes it by Soft::kSlack. Parts of a row
// join by (m, sum, outputs) in join_kernel.
//
// Bound by what a workgroup does in turn for a tile of 64 keys: 68 products of 32
// cycles to a SIMD (L = 512, 64 rows; 144 at L = 256, 128 rows, for its two waves), the
// scores' reads of LDS beside them, then the exponentials, around two meetings of its
// waves and four where a maximum moves. 32 chains of up to 4 rows at 128 heads over 1k to
// 8k keys: 110 us, 760 TFLOP/s, 5,140 cycles a tile with the starts and ends of segments,
// 42 % of them products, and 640 MB past the L2; 16 trees of up to 17 rows at 32 heads,
// 8 bits: 119 us, 660, 6,070 cycles, 36 %; contexts of 40k and 131k at 20 heads (L = 256):
// 71 us, 280, nine tiles to a workgroup and more than half of the products for rows that
// are not there; one row at 32 heads over 1500 keys: 14.0 us, a chain of reads. A
// wave with all products of 32 rows needs 512 outputs a lane beside its queries and
// went through scratch memory (the chains: 508 us), hence columns to a wave. (At L = 256
// 45 registers are spilled and read back around the loop, none in it.)
//
// Persistent over the units of all (request, row segment)s in order: workgroup w
// takes the w-th equal share, so ragged contexts balance by themselves and a long
// one is split over many workgroups. The ring of tiles runs on across segments.
//
// Requests can claim the same rows only where some word of cu_seqlens is less than the
// one before it. Then one that has rows of a well-formed request ahead of it is left out:
// it has no units, by which the joining kernel knows it. A row has one writer.
template <typename T, bool E8, int L>
__global__ __launch_bounds__(waves(L) * kWave, waves(L) / 4) void split_kernel(LatentAttnArgs a,
                                                                               Parts ws) {
  constexpr int kThreads = waves(L) * kWave;
  typedef Ring<E8, L> R;
  __shared__ __align__(1024) unsigned char lds_mem[R::kBytes];
  __shared__ int64_t wsum[waves(L)];
  __shared__ int start_r;
  __shared__ int64_t start_off;
  fetch_args<sizeof(a) + sizeof(ws)>();
  const ReqView& q = a.req;
  const int tid = threadIdx.x;
  const int wave = __builtin_amdgcn_readfirstlane(tid / kWave);
  const unsigned lds = (unsigned)(uintptr_t)(lds_u8*)lds_mem;
  int rows_total;
  const int total_eff = rows_in_use(q, &rows_total);
  const int shift = a.kv.page_shift;
  // every wave finds its workgroup's share by itself where a wave's lanes hold
  // the batch; the workgroup together where they do not
  Cursor cur;
  cur.begun = 0;
  int64_t u0, u1;
  int64_t total;
  const int wgs_all = gridDim.x;
  if (q.B <= kWave) {
    int c0 = 0, len = 0, prefix = 0;
    const int lane = lane_id();
    if (lane < q.B && !rows_of(q, shift, lane, total_eff, &c0, &len, &prefix)) len = 0;
    if (__builtin_expect(__any(lane < q.B && q.cu[lane + 1] < q.cu[lane]), 0)) {
      bool taken = false;
      for (int p = 0; p + 1 < q.B; ++p) {
        const int at = read_lane(c0, p), n = read_lane(len, p);
        taken |= p < lane && n && len && at < c0 + len && c0 < at + n;
      }
      if (taken) len = 0;
    }
    if (wave == 0) {
      lds_write(lds + R::kReqs + 12 * lane_id(), c0);
      lds_write(lds + R::kReqs + 12 * lane_id() + 4, len);
      lds_write(lds + R::kReqs + 12 * lane_id() + 8, prefix);
    }
    const int64_t mine = len ? units_of<L>(a.num_heads, c0, len, prefix) : 0;
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
    const unsigned lost = lds + R::kReqs;
    for (int i = tid; i < DSPARK_MAX_BATCH / 32; i += kThreads) lds_write(lost + i * 4, 0u);
    __syncthreads();
    auto units = [&](int r) {
      int c0, len, prefix;
      return rows_of(q, shift, r, total_eff, &c0, &len, &prefix) && !left_out(lost, r)
                 ? units_of<L>(a.num_heads, c0, len, prefix)
                 : (int64_t)0;
    };
    const int per = (q.B + kThreads - 1) / kThreads;
    const int r0 = min(tid * per, q.B), r1 = min(r0 + per, q.B);
    // (all units are less than 2^13 requests of 2^8 segments of 2^26)
    constexpr int64_t kDisorder = (int64_t)1 << 48;
    int64_t mine = 0;
    for (int r = r0; r < r1; ++r) mine += units(r) + (q.cu[r + 1] < q.cu[r] ? kDisorder : 0);
    int64_t at = block_excl_scan<int64_t, kThreads>(mine, wsum, &total);
    if (__builtin_expect(total >= kDisorder, 0)) {
      for (int r = r0; r < r1; ++r) {
        int c0, len, c1, n, prefix;
        bool taken = false;
        if (rows_of(q, shift, r, total_eff, &c0, &len, &prefix))
          for (int p = 0; p < r; ++p)
            taken |= rows_of(q, shift, p, total_eff, &c1, &n, &prefix) && c1 < c0 + len &&
                     c0 < c1 + n;
        if (taken)
          __hip_atomic_fetch_or(
              (__attribute__((address_space(3))) unsigned*)(uintptr_t)(lost + (r >> 5) * 4),
              1u << (r & 31), __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_WORKGROUP);
      }
      __syncthreads();
      mine = 0;
      for (int r = r0; r < r1; ++r) mine += units(r);
      at = block_excl_scan<int64_t, kThreads>(mine, wsum, &total);
    }
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
  // (uniform for the compiler too, which a copy's operands have to be)
  cur.left = read_lane(u1 - u0, 0);
  cur.off = read_lane(cur.off, 0);
  cur.r = __builtin_amdgcn_readfirstlane(cur.r);
  Feeder<E8, L> feed;
  int stage = 0, tick = 0;
  if (tid == 0) lds_write<unsigned>(lds + R::kFlag, 0u);
  for (bool first = true;; first = false) {
    Job job;
    const Span span = next_span<L>(a, lds + R::kReqs, cur, &job);
    if (span.n == 0) break;
    segment<T, E8, L>(a, ws, span, job, first, cur, feed, lds, stage, tick);
  }
  wait_copies<0>();
}

template <int L>
void launch_split(const LatentAttnArgs& a, const Parts& ws, dspark_dtype dt, hipStream_t s) {
  const dim3 grid((unsigned)ws.wgs), block(waves(L) * kWave);
  if (a.kv.cb == 1) {
    hipLaunchKernelGGL((split_kernel<__bf16, true, L>), grid, block, 0, s, a, ws);
  } else if (dt == DSPARK_BF16) {
    hipLaunchKernelGGL((split_kernel<__bf16, false, L>), grid, block, 0, s, a, ws);
  } else {
    hipLaunchKernelGGL((split_kernel<_Float16, false, L>), grid, block, 0, s, a, ws);
  }
}

void launch_dim256(const LatentAttnArgs& a, const Parts& ws, dspark_dtype dt, hipStream_t s);
void launch_dim512(const LatentAttnArgs& a, const Parts& ws, dspark_dtype dt, hipStream_t s);

}  // namespace lattn
}  // namespace dspark
