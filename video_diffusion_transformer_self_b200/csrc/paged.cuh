// paged.cuh -- what the plan of a paged step (paged.cu) and the attention
// over the pages (paged_attn.cuh) agree on: the division of the step's work
// that the plan writes into wan_paged_t.work.
#pragma once

#include "wan_internal.cuh"

namespace wan {
namespace paged {

constexpr int kMaxStreams = 1024;

// Streams whose rows (new tokens x query heads of one key head) fit one
// 16-row tile run on the kernel that streams the cache through mma.sync
// (kFew); longer ones on the 256-row tcgen05 kernel (kTile).
constexpr int kFewRows = 16;
// kModeNone: no plan has been made.
constexpr int kModeNone = 0, kModeFew = 1, kModeTile = 2;

// kFew: the (stream, key head, 64-key stage) items form one line that is cut
// into equal parts, one per CTA.
// kTile: a row tile holds tile_tokens() tokens x tile_pack() query heads of
// one key head.  Units are (tile pair, tile_pack() heads), numbered streams by
// falling length, then heads, then tile pair (the stream's last one first: it
// sees the most keys).  H_WAVES rounds of one whole unit per CTA come first,
// in turn up and down the CTAs; the units behind them form a line of their
// weights that is cut so that all CTAs end together (LINE[c] .. LINE[c + 1]
// for CTA c), inside a unit's keys where it falls there.
constexpr int kStage = 64;
constexpr int kBlock = 128;
constexpr int kTile = 128;           // rows of a tile
constexpr int kTileRows = 2 * kTile;  // rows of a unit
constexpr int kFewCtasPerSm = 2;
constexpr int kMaxCtas = 511;

// Weight of a unit: 8 a 128-key block with two row tiles, 6 with one, and
// kUnitWeight for its start and end.  Measured with one-tile weights of 4, 5
// and 6: 816, 771 and 749 us for 4,680 rows x 12 heads over 32,760 keys, 100,
// 92 and 88 us for 20 to 400 rows of six streams; starts of 24, 48 and 96:
// 91.5, 89.0 and 88.3 us for the latter.
constexpr int kPairWeight = 8;
constexpr int kOneWeight = 6;
constexpr int kUnitWeight = 48;

// work: a header, LINE[0 .. kMaxCtas], kJoinInts ints per unit of the line
// (at most three rounds of them), then kEnt ints per active stream (written
// and read four at a time, in the order of the E_ fields).
constexpr int kLine = 16;
constexpr int kJoin = kLine + kMaxCtas + 1;
constexpr int kJoinInts = 8;
constexpr int kHdr = kJoin + 3 * kMaxCtas * kJoinInts + 8;
constexpr int kEnt = 16;
enum : int {
  J_ROW = 0,    // packed row of the unit's first token
  J_TOKENS = 1,  // its tokens, 0: one CTA has the unit to itself
  J_HEAD = 2,   // its first head
  J_PART = 3,   // slot of its first part; the others are 2 c, c from ...
  J_CTA = 4,    // ... this CTA on
  J_PARTS = 5   // parts, the first one included
};
enum : int {
  H_KIND = 0,     // work_kind() of the plan's descriptor
  H_ACTIVE = 1,   // entries
  H_TOTAL = 2,    // kFew: stages x key heads; kTile: units
  H_CTAS = 3,     // CTAs that take part
  H_WAVES = 4     // kTile: rounds of whole units
};
enum : int {
  E_STREAM = 0,
  E_BASE = 1,     // kFew: stages before it; kTile: units before it
  E_COUNT = 2,    // kFew: its stages; kTile: its tile pairs
  // kFew: what a CTA needs to start fetching, in one 32-byte read
  E_STAGE0 = 3,   // first stage
  E_KV = 4,       // tokens of the stream
  E_ROWS = 5,     // its new tokens
  E_Q0 = 6,       // their first packed row
  // kTile
  E_FULL = 3,     // weight of a unit with two row tiles
  E_LAST = 4,     // weight of a unit of the last tile pair
  E_FIRST = 5,    // the line's place at which those on it start
  E_LINE = 6,     // (64 bits) the line's place at which the stream's units
                  // would start, had all of them been on it
  E_TKV = 8,      // tokens of the stream
  E_TROWS = 9,    // its new tokens
  E_TQ0 = 10,     // their first packed row
  E_CHUNK = 11,
  E_WINDOW = 12
};

// Weight of a stream's units before its unit n (the last tile pair, which
// may be lighter, is the first unit of each head).
__host__ __device__ __forceinline__ int64_t weight_before(int n, int tiles,
                                                          int full, int last) {
  const int rag = (n + tiles - 1) / tiles;
  return static_cast<int64_t>(n - rag) * full +
         static_cast<int64_t>(rag) * last;
}

// kFew: CTA c of `ctas` takes places [first(c), first(c + 1)) of the line of
// `total`; the first total % ctas CTAs take one more.
struct Line {
  int each, more;
  __host__ __device__ __forceinline__ Line(int total, int ctas)
      : each(total / ctas), more(total % ctas) {}
  __host__ __device__ __forceinline__ int first(int c) const {
    return c * each + (c < more ? c : more);
  }
  __host__ __device__ __forceinline__ int cta_of(int x) const {
    const int big = more * (each + 1);
    return x < big ? x / (each + 1) : more + (x - big) / each;
  }
};

// First key that the query at position a sees, and one past its last.
__host__ __device__ __forceinline__ int64_t chunk_end(int a, int chunk) {
  return (static_cast<int64_t>(a / chunk) + 1) * chunk;
}
__host__ __device__ __forceinline__ int key_lo(int a, int chunk, int window) {
  if (window <= 0) return 0;
  const int64_t lo = chunk_end(a, chunk) - window;
  return lo < 0 ? 0 : lo > 0x7FFFFFFF ? 0x7FFFFFFF : static_cast<int>(lo);
}
__host__ __device__ __forceinline__ int key_hi(int a, int chunk, int kv) {
  if (a < 0) return 0;
  const int64_t e = chunk_end(a, chunk);
  return e < kv ? (e > 0 ? static_cast<int>(e) : 0) : kv;
}

// Unit of a stream that holds place y of its units' weights: its head group
// (returned), tile pair (0: the last one), weight and the place in it.  There
// are at most 1,024 groups, so the fp32 quotient is off by at most 1.  A
// group's weights pass 32 bits (16 heads of one key head, 2^20 tokens over as
// many keys: 2^32), so the place in it is divided in 64.
__host__ __device__ __forceinline__ int unit_of(int64_t y, int tiles, int full,
                                                int last, int* tile,
                                                int* weight, int* off) {
  const int64_t period = static_cast<int64_t>(tiles - 1) * full + last;
  int g = static_cast<int>(static_cast<float>(y) /
                           static_cast<float>(period));
  int64_t rest = y - g * period;
  if (rest < 0) {
    --g;
    rest += period;
  } else if (rest >= period) {
    ++g;
    rest -= period;
  }
  if (rest < last) {
    *tile = 0;
    *weight = last;
    *off = static_cast<int>(rest);
  } else {
    const uint64_t r = static_cast<uint64_t>(rest - last);
    const uint64_t d = static_cast<uint64_t>(full);
    const uint64_t n = r / d;
    *tile = 1 + static_cast<int>(n);
    *weight = full;
    *off = static_cast<int>(r - n * d);
  }
  return g;
}

inline bool few_mode(const wan_paged_t* c) {
  return static_cast<int64_t>(c->max_new) * (c->heads / c->kv_heads) <=
         kFewRows;
}

// Query heads of one key head that share a row tile: the most, up to 16, that
// divide them.  Short streams then fill their tiles and read their keys once
// for all of them; where the tile does not come out even (5 heads x 25 tokens
// are 125 rows) long ones would only lose rows.
inline int tile_pack(const wan_paged_t* c) {
  const int group = c->heads / c->kv_heads;
  int p = 1;
  for (int i = 2; i <= 16; ++i)
    if (group % i == 0) p = i;
  return kTile % p != 0 && c->max_new > 1024 ? 1 : p;
}
inline int tile_tokens(const wan_paged_t* c) { return kTile / tile_pack(c); }

// What the work list's layout depends on, in one number that is never
// kModeNone: the kernel, the heads and, of max_new, the rows of a key head
// (kFew) or the heads of a row tile (kTile).  The attention reads a list only
// if its own descriptor gives the number that the plan wrote.
inline int work_kind(const wan_paged_t* c) {
  const int mode = few_mode(c) ? kModeFew : kModeTile;
  const int rows = few_mode(c) ? c->max_new * (c->heads / c->kv_heads)
                               : tile_pack(c);
  return mode | rows << 2 | c->heads << 7 | c->kv_heads << 18;
}

// Checks of the sizes and of the pointers every call needs.
int check_cache(const wan_paged_t* c);

}  // namespace paged
}  // namespace wan
