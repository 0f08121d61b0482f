// paged.cu -- the plan of a step over a paged K / V cache and the write of
// the step's tokens into the pages.
//
// Long-video survey (atlascloud.ai), section "Route 3 · Self Forcing": the
// video grows chunk by chunk against a KV cache that may be capped; Wan2.2
// source reading, ch. 4, section "3D RoPE": q and k pass an RMSNorm, then
// turn by the token's frame, row and column.  The calls and their layouts
// are described in wan.h.
#include <mutex>

#include "paged.cuh"
#include "rope_common.cuh"

namespace wan {
namespace paged {

int check_cache(const wan_paged_t* c) {
  if (!c) return WAN_EINVAL;
  if (c->n_streams < 1 || c->n_streams > kMaxStreams || c->max_pages < 1 ||
      c->n_pages < 1 || c->n_pages > (1 << 30) || c->token_cap < 1 ||
      c->token_cap > (1 << 27) || c->max_new < 1 || c->heads < 1 ||
      c->heads > 1024 || c->kv_heads < 1 || c->heads % c->kv_heads != 0)
    return WAN_EINVAL;
  if (c->page_size != 16 && c->page_size != 32 && c->page_size != 64 &&
      c->page_size != 128)
    return WAN_EINVAL;
  const int64_t lim = 1ll << 31;
  if (static_cast<int64_t>(c->n_streams) * c->max_pages >= lim ||
      static_cast<int64_t>(c->max_pages) * c->page_size > lim / 2 ||
      static_cast<int64_t>(c->n_pages) * c->page_size >= lim ||
      static_cast<int64_t>(c->token_cap) * c->heads >= lim ||
      (static_cast<int64_t>(c->n_pages) * c->page_size / kStage +
       2ll * c->n_streams) * c->kv_heads >= lim)
    return WAN_EINVAL;
  if (wan_rope3d_table_bytes(c->grid, 128) == 0) return WAN_EINVAL;
  const void* all[] = {c->streams,    c->kv_lens, c->first_pages,
                       c->block_table, c->free_ring, c->ring_state,
                       c->q_start,    c->q_lens,  c->status,
                       c->tokens,     c->work};
  for (const void* p : all)
    if (!p) return WAN_EINVAL;
  for (const void* p : all)
    if (!aligned16(p)) return WAN_EALIGN;
  return WAN_OK;
}

namespace {

// ------------------------------------------------------------- the plan --
//
// Bound by a launch and the chain of scans: 76 KB to 2 MB move in 8 to 14 us
// (1 stream x 4,685 records 8.0 us, 48 streams x 114,041 records 12.6, 777 x
// 6,348 13.8; 2 us of each is the caller's copy of the state in those runs).
// One cluster of CTAs.  Every CTA reads all streams (one thread a stream)
// and finds the same prefix sums; the moves of pages and the tokens' records
// are then spread over the threads of all CTAs, each finding its stream by a
// binary search of the sums.  Pages come back to the ring's tail and leave
// from its head, which never meet: what the ring holds and what the streams
// hold add up to n_pages.  One cluster barrier separates the reads of the
// old state and the pages coming back from the writes of the new state and
// the pages going out, so no second launch is needed and no CTA waits for
// another kernel.
// Threads of a CTA, T below: at least one a stream and one an SM.  Every warp
// runs the scans, so up to 64 streams take 256 threads, more streams or
// records 1,024.  Measured against each other when that was chosen: 4,685
// records of one stream 7.1 us with 256 and 9.8 with 1,024; 32 streams,
// 23,243 records 12.1 and 13.4; 100 streams 16.2 and 16.1; 256 streams 11.4
// and 10.5.
constexpr int kPlanThreads = 1024;
constexpr int kPlanThreadsFew = 256;
constexpr int kPlanStreamsFew = 64;

struct PlanArgs {
  wan_paged_t c;
  const int32_t* new_lens;
  int page_shift;
  int sms;
  int few, kind;
  int pack, tile_tokens;  // of the tile kernel
};

// n / d for 0 <= n < 2^31, 1 <= d <= 2^20, inv = 1 / d rounded.  The three
// roundings of the first quotient are below 2^-22 of n / d, so with the
// truncation what it leaves is less than 2^9 + d in size, and the second one
// is off by at most 1.
__device__ __forceinline__ int div_by(int n, int d, float inv) {
  int q = static_cast<int>(static_cast<float>(n) * inv);
  int rest = n - q * d;
  q += static_cast<int>(static_cast<float>(rest) * inv);
  rest = n - q * d;
  return rest < 0 ? q - 1 : rest >= d ? q + 1 : q;
}

// Cluster barrier in two halves.
__device__ __forceinline__ void cluster_arrive() {
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// Inclusive sum over the block's threads.  one_warp: only the first 32
// threads have values (up to 32 streams): one level of the two.
template <int T>
__device__ __forceinline__ uint64_t block_scan(uint64_t v, uint64_t* red,
                                               bool one_warp = false) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint64_t u = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += u;
  }
  __syncthreads();  // red is reused by consecutive calls
  if (lane == 31) red[warp] = v;
  __syncthreads();
  if (one_warp) return warp ? red[0] : v;
  if (warp == 0) {
    uint64_t t = lane < T / 32 ? red[lane] : 0;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint64_t u = __shfl_up_sync(0xffffffffu, t, o);
      if (lane >= o) t += u;
    }
    if (lane < T / 32) red[lane] = t;
  }
  __syncthreads();
  return warp ? v + red[warp - 1] : v;
}

template <int T>
__device__ __forceinline__ uint64_t block_max(uint64_t v, uint64_t* red) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const uint64_t u = __shfl_xor_sync(0xffffffffu, v, o);
    v = u > v ? u : v;
  }
  __syncthreads();  // red is reused by consecutive calls
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  v = red[threadIdx.x & (T / 32 - 1)];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const uint64_t u = __shfl_xor_sync(0xffffffffu, v, o);
    v = u > v ? u : v;
  }
  return v;
}

// First r in [0, n) with incl[r] > x (n - 1 if there is none).
__device__ __forceinline__ int find_stream(const int* incl, int n, int x) {
  int lo = 0, hi = n - 1;
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (incl[mid] > x)
      hi = mid;
    else
      lo = mid + 1;
  }
  return lo;
}

// How far a cut stays from the ends of the unit it falls into (a piece costs
// its start, its partial result and the join of it, about six key blocks).
// Two cuts inside one unit may be closer: a CTA that lacks little gets little.
constexpr int kMinPiece = 64;
// Where there are more CTAs than units, down to a quarter of it for very few
// units: 2 units of 80 blocks 36 us with 64, 23 with 16; 12 of 260 51 and 45;
// 72 of 4 blocks 22 with 64, 33 with 16.
constexpr int kMinPieceIdle = 16;

// Rounds of whole units beyond which the CTAs' loads count as equal.
constexpr int kManyRounds = 16;

// Scratch of build_work, one entry a stream or CTA.
struct WorkMem {
  int *a, *b, *c, *d, *e, *f, *g;
  unsigned long long* load;   // one a CTA
  int64_t* start;             // one a stream
};

// The few-row kernel's line: 64-key stages from the first row's first key to
// the end of the stream; at least one, so that rows that see nothing are
// written too.
template <int T>
__device__ void build_few(const PlanArgs& a, int ql, int kv, int q0, int lo,
                          uint64_t* red) {
  const int r = threadIdx.x;
  int32_t* work = a.c.work;
  const bool on = ql > 0;
  const int stage0 = on ? min(lo, kv - 1) / kStage : 0;
  const int n = on ? (kv + kStage - 1) / kStage - stage0 : 0;
  const uint64_t sc = block_scan<T>(
      (static_cast<uint64_t>(on) << 40) | static_cast<uint64_t>(n), red,
      a.c.n_streams <= 32);
  const int idx = static_cast<int>(sc >> 40) - on;
  const int base = static_cast<int>(sc & 0xFFFFFFFFFFull) - n;
  if (on) {
    int4* e = reinterpret_cast<int4*>(work + kHdr + kEnt * idx);
    e[0] = make_int4(r, base, n, stage0);
    e[1] = make_int4(kv, ql, q0, 0);
  }
  if (r == T - 1) {
    const int64_t total = static_cast<int64_t>(base + n) * a.c.kv_heads;
    // a stage each up to one CTA an SM, then two (12 heads over 2,000 keys,
    // 384 stages: 8.3 us on 192 CTAs, 9.0 on 296)
    const int64_t most = min(max(total / 2, static_cast<int64_t>(a.sms)),
                             static_cast<int64_t>(a.sms) * kFewCtasPerSm);
    work[H_KIND] = a.kind;
    work[H_ACTIVE] = idx + on;
    work[H_TOTAL] = static_cast<int>(total);
    work[H_CTAS] =
        static_cast<int>(total < 1 ? 1 : total > most ? most : total);
    work[H_WAVES] = 0;
  }
}

// Orders the streams with rows by falling length: thread i gets the i-th's
// number (of the n_act there are; any number past them), and stream i's place
// in *place.  By length classes,
// four to the doubling and 32 of them down from the longest, streams in
// their own order within a class: that is close enough for CTAs that take
// units up and down the list (a full sort of 1,024 took 6 us instead of 1).
template <int T>
__device__ __forceinline__ int sorted_stream(bool on, int nb, int* order,
                                             int* hist, uint64_t* red,
                                             int* place) {
  const int r = threadIdx.x, lane = r & 31, warp = r >> 5;
  const int longest =
      static_cast<int>(block_max<T>(static_cast<uint64_t>(on ? nb : 0), red));
  hist[r] = 0;
  __syncthreads();
  int cls = 32;  // no rows
  if (on)
    cls = min(31, static_cast<int>(4.f * __log2f(static_cast<float>(longest) /
                                                 static_cast<float>(nb))));
  const unsigned same = __match_any_sync(0xffffffffu, cls);
  const int before = __popc(same & ((1u << lane) - 1u));
  if (on && before == 0) hist[cls * (T / 32) + warp] = __popc(same);
  __syncthreads();
  const int n = hist[r];
  const int upto =
      static_cast<int>(block_scan<T>(static_cast<uint64_t>(n), red));
  __syncthreads();
  hist[r] = upto - n;
  __syncthreads();
  if (on) {
    *place = hist[cls * (T / 32) + warp] + before;
    order[*place] = r;
  }
  __syncthreads();
  return order[r];
}

// Weights of a stream's units: nb key blocks, ql new tokens, `tokens` a tile.
__device__ __forceinline__ int full_weight(int nb) {
  return kPairWeight * nb + kUnitWeight;
}
__device__ __forceinline__ int last_weight(int nb, int ql, int tokens) {
  const int rest = ql % (2 * tokens);
  return (rest >= 1 && rest <= tokens ? kOneWeight : kPairWeight) * nb +
         kUnitWeight;
}

// The tile kernel's division of the work.  Whole units in rounds over the
// CTAs keep neighbours on the same head and keys in step (their K and V
// blocks are read once into L2); a last round that is not full would leave
// SMs idle (760 units on 148 SMs are 5.14 rounds: 14 % of the time), so the
// last one to two rounds' units are cut by weight instead.
template <int T>
__device__ void build_tiles(const PlanArgs& a, int ql, int kv, int q0,
                            int chunk, int window, int nb, uint64_t* red,
                            const WorkMem& mem) {
  const int r = threadIdx.x;
  const bool on = ql > 0;
  const bool small = a.c.n_streams <= 32;
  const int heads = a.c.heads / a.pack;  // head groups of a tile
  const int pair = 2 * a.tile_tokens;
  __shared__ int s_units, s_act, s_long;
  __shared__ unsigned long long s_sum;
  unsigned long long* s_load = mem.load;
  int src = 0, place = 0;
  if (a.c.n_streams > 1) {
    mem.a[r] = 0;  // places past the last
    src = sorted_stream<T>(on, nb, mem.a, mem.b, red, &place);
  }
  const int n_act = __syncthreads_count(on);
  mem.a[r] = nb;
  mem.b[r] = ql;
  __syncthreads();
  const bool mine = r < n_act;
  const int m_nb = mine ? mem.a[src] : 0;
  const int m_ql = mine ? mem.b[src] : 0;
  const int m_tiles = (m_ql + pair - 1) / pair;
  // (lengths past 65,535 blocks are scaled so that the line fits 32 bits; the
  // first stream is within a fifth of the longest)
  if (r == 0) s_long = m_nb;
  __syncthreads();
  const int down = max(0, 16 - __clz(s_long));
  const int w_nb = m_nb >> down;
  const int m_full = full_weight(w_nb);
  const int m_last = last_weight(w_nb, m_ql, a.tile_tokens);
  const int units = m_tiles * heads;
  const int upto =
      static_cast<int>(block_scan<T>(static_cast<uint64_t>(units), red, small));
  const uint64_t weight =
      mine ? static_cast<uint64_t>(heads) *
                 (static_cast<uint64_t>(m_tiles - 1) * m_full + m_last)
           : 0;
  const uint64_t all = block_scan<T>(weight, red, small);
  __syncthreads();
  mem.a[r] = upto;           // units up to and with the r-th stream
  mem.b[r] = m_tiles;
  mem.c[r] = m_full;
  mem.d[r] = m_last;
  if (r == T - 1) {
    s_units = upto;
    s_act = n_act;
    s_sum = all;
  }
  __syncthreads();
  const int U = s_units;
  // fewer CTAs where there is not enough for all: 4 blocks each
  const int64_t parts = static_cast<int64_t>(s_sum) / (kPairWeight * 4);
  int G = a.sms;
  if (U < G) G = static_cast<int>(min(static_cast<int64_t>(G),
                                      max(static_cast<int64_t>(U), parts)));
  if (G < 1) G = 1;
  // Loads of the CTAs after K rounds, `share` threads a CTA; the most rounds
  // whose heaviest CTA stays within the mean, at most two fewer than there
  // are (the rounds go up and down, which leaves little beyond a unit's
  // length between the CTAs).  After many rounds that little is not worth
  // the sums: the loads count as equal.
  int K = U / G;
  uint64_t lack = 1;
  if (K < kManyRounds) {
    const int share = T / G;
    const int c = r % G, part = r / G;
    auto unit_weight = [&](int u) {
      const int i = find_stream(mem.a, n_act, u);
      const int at = u - (i ? mem.a[i - 1] : 0);
      return at % mem.b[i] == 0 ? mem.d[i] : mem.c[i];
    };
    if (r < G) s_load[r] = 0;
    __syncthreads();
    if (part < share && part < K) {
      unsigned long long sum = 0;
      for (int k = part; k < K; k += share)
        sum += unit_weight(k * G + (k & 1 ? G - 1 - c : c));
      atomicAdd(&s_load[c], sum);
    }
    for (int tries = 0;; ++tries) {
      __syncthreads();
      const uint64_t top = block_max<T>(r < G ? s_load[r] : 0, red);
      if (K == 0 || tries == 2 || top * G <= s_sum) break;
      --K;
      if (r < G) s_load[r] -= unit_weight(K * G + (K & 1 ? G - 1 - r : r));
    }
    const uint64_t mean =
        static_cast<uint64_t>(static_cast<double>(s_sum) / G) + 1;
    lack = r < G && s_load[r] < mean ? mean - s_load[r] : 0;
  }
  // the line: places in proportion to what each CTA lacks
  const uint64_t lack_upto = block_scan<T>(r < G ? lack : 0, red);
  const int first = K * G;  // units before the line
  const int base = upto - units;
  // the stream's units before the line
  const int before = min(max(first - base, 0), units);
  const uint64_t skipped =
      mine ? weight_before(before, m_tiles, m_full, m_last) : 0;
  const uint64_t on_line = weight - skipped;
  const uint64_t line_upto = block_scan<T>(on_line, red, small);
  __shared__ unsigned long long s_lack, s_line;
  if (r == T - 1) {
    s_lack = lack_upto;
    s_line = line_upto;
  }
  __syncthreads();
  int32_t* work = a.c.work;
  int* s_cut = reinterpret_cast<int*>(s_load);
  __syncthreads();
  if (on) {
    // thread r has stream r here, the entries' threads their place
    int4* e = reinterpret_cast<int4*>(work + kHdr + kEnt * place);
    e[E_TKV / 4] = make_int4(kv, ql, q0, chunk);
    e[E_WINDOW / 4] = make_int4(window, 0, 0, 0);
    mem.e[place] = q0;
  }
  if (mine) {
    int4* e = reinterpret_cast<int4*>(work + kHdr + kEnt * r);
    const int64_t start = static_cast<int64_t>(line_upto - on_line) -
                          static_cast<int64_t>(skipped);
    e[0] = make_int4(src, base, m_tiles, m_full);
    e[1] = make_int4(m_last, static_cast<int>(line_upto - on_line),
                     static_cast<int>(start & 0xFFFFFFFFll),
                     static_cast<int>(start >> 32));
    mem.f[r] = m_ql;
    mem.start[r] = start;
    mem.g[r] = static_cast<int>(line_upto);
  }
  __syncthreads();
  if (r < G) {
    // (fp32: a cut may be off by a few places, but cuts do not cross)
    const float scale = static_cast<float>(s_line) /
                        static_cast<float>(s_lack ? s_lack : 1);
    int end = static_cast<int>(s_line);
    const int least =
        K ? kMinPiece
          : kMinPieceIdle +
                (kMinPiece - kMinPieceIdle) * min(2 * U, a.sms) / a.sms;
    if (r < G - 1) {
      end = min(end, static_cast<int>(static_cast<float>(lack_upto) * scale));
      if (end < static_cast<int>(s_line)) {
        // the unit it falls into, and no piece too small to pay for itself
        const int i = find_stream(mem.g, n_act, end);
        int tile, len, off;
        unit_of(end - mem.start[i], mem.b[i], mem.c[i], mem.d[i], &tile, &len,
                &off);
        if (off < least || len - off < least)
          end += 2 * off < len ? -off : len - off;
      }
    }
    s_cut[r + 1] = end;
    work[kLine + r + 1] = end;
    if (r == 0) s_cut[0] = work[kLine] = 0;
  }
  __syncthreads();
  // what the joining pass needs of every unit on the line
  for (int j = r; j < U - first; j += T) {
    const int u = first + j;
    const int i = find_stream(mem.a, n_act, u);
    const int local = u - (i ? mem.a[i - 1] : 0);
    const int tiles = mem.b[i];
    const int head = local / tiles, tile = local - head * tiles;
    const int x0 = static_cast<int>(
        mem.start[i] + weight_before(local, tiles, mem.c[i], mem.d[i]));
    const int x1 = x0 + (tile == 0 ? mem.d[i] : mem.c[i]) - 1;
    // CTAs that hold its first and its last place
    const int c0 = find_stream(s_cut + 1, G, x0);
    const int c1 = find_stream(s_cut + 1, G, x1);
    const int tok0 = (tiles - 1 - tile) * pair;
    int32_t rec[kJoinInts] = {0, 0, 0, 0, 0, 0, 0, 0};
    rec[J_ROW] = mem.e[i] + tok0;
    rec[J_TOKENS] = c0 == c1 ? 0 : min(mem.f[i] - tok0, pair);
    rec[J_HEAD] = head * a.pack;
    rec[J_PART] = 2 * c0 + (x0 > s_cut[c0] ? 1 : 0);
    rec[J_CTA] = c0 + 1;
    rec[J_PARTS] = c1 - c0 + 1;
    int4* dst = reinterpret_cast<int4*>(work + kJoin + kJoinInts * j);
    dst[0] = make_int4(rec[0], rec[1], rec[2], rec[3]);
    dst[1] = make_int4(rec[4], rec[5], rec[6], rec[7]);
  }
  if (r == 0) {
    work[H_KIND] = a.kind;
    work[H_ACTIVE] = s_act;
    work[H_TOTAL] = U;
    work[H_CTAS] = G;
    work[H_WAVES] = K;
  }
}

// The attention's work list, by one CTA.  ql and kv are stream threadIdx.x's
// rows and keys, q0 its first packed row.
template <int T>
__device__ void build_work(const PlanArgs& a, int ql, int kv, int q0,
                           int chunk, int window, uint64_t* red,
                           const WorkMem& mem) {
  const int lo = ql > 0 ? key_lo(kv - ql, chunk, window) : 0;
  if (a.few) {
    build_few<T>(a, ql, kv, q0, lo, red);
    return;
  }
  // 128-key blocks of the longest tile (an upper bound under a window)
  int nb = 0;
  if (ql > 0) {
    nb = max((kv + kBlock - 1) / kBlock - min(lo, kv - 1) / kBlock, 1);
    if (window > 0) {
      const int64_t rows = 2 * a.tile_tokens;
      const int64_t keys = window + (rows + chunk - 1) / chunk * chunk;
      nb = static_cast<int>(min(static_cast<int64_t>(nb), keys / kBlock + 2));
    }
  }
  build_tiles<T>(a, ql, kv, q0, chunk, window, nb, red, mem);
}

template <int T>
__global__ void __launch_bounds__(T)
    paged_plan_kernel(const __grid_constant__ PlanArgs a) {
  // (s_inv_w also serves as scratch: a 64-bit number a CTA)
  constexpr int kScratch = T > 2 * (kMaxCtas + 1) ? T : 2 * (kMaxCtas + 1);
  __shared__ uint64_t red[32];
  __shared__ int s_end[T];    // packed rows up to and with stream r
  __shared__ int s_rows[T];   // admitted rows
  __shared__ int s_back[T];   // pages coming back, inclusive
  __shared__ int s_need[T];   // pages going out, inclusive
  __shared__ int s_old[T];    // tokens before the step
  __shared__ int s_from[T];   // first page coming back
  // tokens of a frame and of a row, and one over them
  __shared__ __align__(8) int s_dims[2 * T];
  int* s_hw = s_dims;
  int* s_w = s_dims + T;
  __shared__ float s_inv_hw[T];
  __shared__ __align__(8) float s_inv_w[kScratch];
  __shared__ int s_extra[T];            // scratch
  const wan_paged_t& c = a.c;
  const int R = c.n_streams;
  const int r = threadIdx.x;
  const int ps = c.page_size;
  const uint32_t np = static_cast<uint32_t>(c.n_pages);
  const uint32_t head = static_cast<uint32_t>(c.ring_state[0]) % np;
  const int count = min(max(c.ring_state[1], 0), c.n_pages);
  int nw = 0, old = 0, first = 0;
  int4 cfg = make_int4(1, 1, 1, 0);
  if (r < R) {
    nw = a.new_lens[r];
    old = max(c.kv_lens[r], 0);
    first = max(c.first_pages[r], 0);
    cfg = reinterpret_cast<const int4*>(c.streams)[r];
  }
  const int rows = max(nw, 0);
  const bool ended = nw < 0;
  const int64_t end = static_cast<int64_t>(
      block_scan<T>(static_cast<uint64_t>(rows), red, R <= 32));
  const int64_t total = static_cast<int64_t>(old) + rows;
  const int64_t cap = c.token_cap;
  const bool fit =
      cfg.x >= 1 && cfg.y >= 1 && cfg.x <= c.grid.H && cfg.y <= c.grid.W &&
      cfg.z >= 1 && cfg.w >= 0 && rows <= c.max_new &&
      total <= static_cast<int64_t>(c.max_pages) * ps &&
      total <= static_cast<int64_t>(c.grid.F) * cfg.x * cfg.y && end <= cap;
  const bool valid = nw > 0 && fit;
  // pages held before the step, and those of them that come back
  const int64_t pages = (static_cast<int64_t>(old) + ps - 1) >> a.page_shift;
  const int held = min(static_cast<int>(pages), c.max_pages);
  first = min(first, held);
  int gone = first;
  if (ended)
    gone = held;
  else if (valid)
    gone = max(first, min(key_lo(old, cfg.z, cfg.w), old) >> a.page_shift);
  const int back = gone - first;
  const int top =
      valid ? static_cast<int>((total + ps - 1) >> a.page_shift) : held;
  const int need = valid ? top - held : 0;
  const uint64_t sums = block_scan<T>(
      (static_cast<uint64_t>(back) << 32) | static_cast<uint64_t>(need), red,
      R <= 32);
  const int back_incl = static_cast<int>(sums >> 32);
  const int need_incl = static_cast<int>(sums & 0xFFFFFFFFull);
  s_back[r] = back_incl;
  s_from[r] = first;
  s_old[r] = old;
  s_end[r] = static_cast<int>(end < cap ? end : cap);
  __syncthreads();
  const int n_back = s_back[T - 1];
  const int free_now = min(count + n_back, c.n_pages);
  const bool admit = valid && need_incl <= free_now;
  s_need[r] = need_incl;
  s_rows[r] = admit ? rows : 0;
  if (admit) {  // H and W lie in the grid, so H W <= 2^20
    s_hw[r] = cfg.x * cfg.y;
    s_w[r] = cfg.y;
    s_inv_hw[r] = 1.0f / static_cast<float>(cfg.x * cfg.y);
    s_inv_w[r] = 1.0f / static_cast<float>(cfg.y);
  }
  // admission stops for good at the first stream that does not fit, so the
  // admitted needs are a prefix of the line of needs
  const int n_out = static_cast<int>(
      block_scan<T>(admit ? static_cast<uint64_t>(need) : 0ull, red, R <= 32));
  __shared__ int s_out;
  if (r == T - 1) s_out = n_out;
  const WorkMem mem = {s_back,
                       s_need,
                       s_from,
                       s_rows,
                       s_old,
                       reinterpret_cast<int*>(s_inv_hw),
                       s_extra,
                       reinterpret_cast<unsigned long long*>(s_inv_w),
                       reinterpret_cast<int64_t*>(s_dims)};
  const int kv = ended ? 0 : old + (admit ? rows : 0);
  const int ctas = gridDim.x;
  const int rank = blockIdx.x;
  // the last CTA divides the attention's work (no global state but its own
  // output), the others do the moves
  const int movers = ctas - 1;
  const int step = movers * T;
  const int me = rank * T + r;
  if (rank < movers) {
    for (int i = me; i < n_back; i += step) {
      const int q = find_stream(s_back, R, i);
      const int at = i - (q ? s_back[q - 1] : 0);
      int32_t* ent = c.block_table +
                     static_cast<int64_t>(q) * c.max_pages + s_from[q] + at;
      c.free_ring[(head + static_cast<uint32_t>(count) + i) % np] = *ent;
      *ent = -1;
    }
  }
  __syncthreads();
  cluster_arrive();
  if (rank == movers) {
    build_work<T>(a, admit ? rows : 0, kv, r ? s_end[r - 1] : 0, cfg.z, cfg.w,
                  red, mem);
    __syncthreads();
    cluster_wait();
    return;
  }
  // once all pages are back and all CTAs have read the old state
  cluster_wait();
  const int out = s_out;
  for (int i = me; i < out; i += step) {
    const int q = find_stream(s_need, R, i);
    const int at = i - (q ? s_need[q - 1] : 0);
    const int p = ((s_old[q] + ps - 1) >> a.page_shift) + at;
    c.block_table[static_cast<int64_t>(q) * c.max_pages + p] =
        c.free_ring[(head + i) % np];
  }
  if (rank == 0) {
    if (r < R) {
      c.kv_lens[r] = kv;
      c.first_pages[r] = ended ? 0 : gone;
      const int64_t start = end - rows;
      c.q_start[r] = static_cast<int>(start < cap ? start : cap);
      c.q_lens[r] = admit ? rows : 0;
      c.status[r] = (nw > 0 && !fit)        ? WAN_EINVAL
                    : (valid && !admit)     ? WAN_ENOSPACE
                                            : WAN_OK;
      if (r == R - 1) c.q_start[R] = s_end[r];
    }
    if (r == 0) {
      c.ring_state[0] = static_cast<int>((head + out) % np);
      c.ring_state[1] = free_now - out;
    }
  }
  // The tokens' records: the page of a new position is either one the stream
  // held (its table entry does not change) or comes from the ring.  A warp
  // takes consecutive records, so that its stream moves on by a step or two
  // between them; divisions by a stream's frame and row are products.
  int4* tok = reinterpret_cast<int4*>(c.tokens);
  const int n_rows = s_end[R - 1];
  const int warps = movers * (T / 32);
  const int share = ((c.token_cap + warps - 1) / warps + 31) & ~31;
  const int i0 = (me >> 5) * share;
  const int i1 = min(i0 + share, c.token_cap);
  int q = i0 < n_rows ? find_stream(s_end, R, min(i0 + (r & 31), n_rows - 1))
                      : 0;
  // the stream's numbers stay in registers while it lasts
  int upto = -1, start = 0, live = 0, old_q = 0, hw = 1, w = 1, held_q = 0;
  float inv_hw = 1.f, inv_w = 1.f;
  uint32_t from = 0;  // ring place of its first new page
  for (int i = i0 + (r & 31); i < i1; i += 32) {
    int4 rec = make_int4(0, 0, 0, -1);
    if (i < n_rows) {
      if (i >= upto) {
        while (s_end[q] <= i) ++q;
        upto = s_end[q];
        // rows of the stream start where those of the one before end
        start = q ? s_end[q - 1] : 0;
        live = s_rows[q];
        old_q = s_old[q];
        hw = s_hw[q];
        w = s_w[q];
        inv_hw = s_inv_hw[q];
        inv_w = s_inv_w[q];
        held_q = (old_q + ps - 1) >> a.page_shift;
        from = head + (q ? s_need[q - 1] : 0);
      }
      const int off = i - start;
      if (off < live) {
        const int pos = old_q + off;
        rec.x = div_by(pos, hw, inv_hw);
        const int rest = pos - rec.x * hw;
        rec.y = div_by(rest, w, inv_w);
        rec.z = rest - rec.y * w;
        const int p = pos >> a.page_shift;
        // (the ring's place is below 2 np: what goes out is at most np)
        const uint32_t at = from + (p - held_q);
        const int page =
            p < held_q
                ? c.block_table[static_cast<int64_t>(q) * c.max_pages + p]
                : c.free_ring[at < np ? at : at - np];
        rec.w = (page << a.page_shift) + (pos & (ps - 1));
      }
    }
    tok[i] = rec;
  }
}

// ------------------------------------------------------------ the write --
//
// HBM-bound: every row of q, k and v is read once and written once.  One
// warp per (row, tensor); lane l holds 16-byte chunk l & 15 of heads l >> 4,
// l >> 4 + 2, ... in registers (kRows of them), so a row is one batch of
// independent loads, one reduction and one batch of stores; a head's 256
// bytes land contiguously in its page.  For more than 2 * 20 heads the row
// is read twice (the second time from L2).  One item a warp and as many CTAs
// as that takes, two warps each: new CTAs load while others store, where a
// warp that walked several items alternated between the two.  43,200 rows x
// 40 heads, 2.65 GB: 400 us, 6.6 TB/s (4-warp CTAs 403, walking 446; 12 warps
// an SM instead of 16: 499 us).  4,680 rows x 12 heads, 86 MB: 13.6 us out of
// L2, 20.6 after other traffic (a plain copy of as much: 9.5 and 15.4), bound
// by the latency of a warp's chain (record, row, weights) over 3.3 rounds of
// CTAs; two or three rows a warp took 15 to 23 us there, the weights fetched
// ahead of the row 18.9.
constexpr int kWrThreads = 64;
constexpr int kWrWarps = kWrThreads / 32;
constexpr int kWrMaxRows = 20;

struct WriteArgs {
  const uint4* in[3];      // q, k, v
  uint4* out[3];           // q_out, k_pages, v_pages
  const float4* w[2];      // weights of q and k
  const float4* table;     // RoPE rows of 11 float4
  const int4* tokens;
  const int32_t* n_rows;   // packed rows of the streams (q_start[R])
  int rows;                // packed rows of the tensors
  int heads, kv_heads;
  int F, H, W;
  int page_shift;
  int slots;               // n_pages * page_size
  float eps;
};

// resident CTAs an SM that each row-register budget allows
template <int kRows>
constexpr int wr_min_blocks() {
  return kRows == 0   ? 16
         : kRows <= 4 ? 18
         : kRows <= 6 ? 16
         : kRows <= 8 ? 14
         : kRows <= 12 ? 12
                       : 8;
}

// kRows 0: any head count, two passes over the row.
template <int kRows>
__global__ void
__launch_bounds__(kWrThreads, wr_min_blocks<kRows>())
    paged_write_kernel(const __grid_constant__ WriteArgs a) {
  const int lane = threadIdx.x & 31;
  const int c = lane & 15;
  const int hsub = lane >> 4;
  const unsigned it = blockIdx.x * kWrWarps + (threadIdx.x >> 5);
  const int row = static_cast<int>(it / 3);
  const int which = static_cast<int>(it - 3u * row);
  if (row < a.rows) {
    const int4 tk = __ldg(a.tokens + row);
    if (row >= __ldg(a.n_rows)) return;  // behind the last stream
    const int nh = which == 0 ? a.heads : a.kv_heads;
    // selects, not indexes: a runtime index into the parameters would copy
    // them to the stack
    const uint4* in = which == 0 ? a.in[0] : which == 1 ? a.in[1] : a.in[2];
    uint4* out = which == 0 ? a.out[0] : which == 1 ? a.out[1] : a.out[2];
    in += static_cast<int64_t>(row) * nh * 16 + c;
    uint4 x[kRows ? kRows : 1];
    if (kRows) {
#pragma unroll
      for (int k = 0; k < kRows; ++k)
        if (hsub + 2 * k < nh) x[k] = in[(hsub + 2 * k) * 16];
    }
    // records that no plan writes, rows of refused streams
    if (tk.w < 0 || tk.w >= a.slots || static_cast<unsigned>(tk.x) >= a.F ||
        static_cast<unsigned>(tk.y) >= a.H ||
        static_cast<unsigned>(tk.z) >= a.W)
      return;
    int64_t hstep = 16;  // uint4 from one head's row to the next
    if (which == 0) {
      out += static_cast<int64_t>(row) * nh * 16 + c;
    } else {
      const int page = tk.w >> a.page_shift;
      const int off = tk.w & ((1 << a.page_shift) - 1);
      hstep = 16ll << a.page_shift;
      out += static_cast<int64_t>(page) * nh * hstep + off * 16 + c;
    }
    float ss = 0.f;
    auto squares = [&](const uint4& v) {
      const uint32_t vv[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float2 f = bf16x2_to_float2(vv[e]);
        ss = fmaf(f.x, f.x, fmaf(f.y, f.y, ss));
      }
    };
    if (which == 2) {
      if (kRows) {
#pragma unroll
        for (int k = 0; k < kRows; ++k)
          if (hsub + 2 * k < nh) out[(hsub + 2 * k) * hstep] = x[k];
      } else {
        for (int h = hsub; h < nh; h += 2) out[h * hstep] = in[h * 16];
      }
      return;
    }
    const float4* tt = a.table + static_cast<int64_t>(tk.x) * 11;
    const float4* th = a.table + static_cast<int64_t>(a.F + tk.y) * 11;
    const float4* tw = a.table + static_cast<int64_t>(a.F + a.H + tk.z) * 11;
    const float4 cs0 = pair_cs(4 * c, tt, th, tw);
    const float4 cs1 = pair_cs(4 * c + 2, tt, th, tw);
    if (kRows) {
#pragma unroll
      for (int k = 0; k < kRows; ++k)
        if (hsub + 2 * k < nh) squares(x[k]);
    } else {
#pragma unroll 4
      for (int h = hsub; h < nh; h += 2) squares(in[h * 16]);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
    const float f = rsqrtf(ss / (128.0f * nh) + a.eps);
    const float4* wt = (which ? a.w[1] : a.w[0]) + 2 * c;
    auto turned = [&](const uint4& v, int h) {
      const float4 w0 = __ldg(wt + h * 32);
      const float4 w1 = __ldg(wt + h * 32 + 1);
      return make_uint4(norm_rot2(v.x, f, w0.x, w0.y, cs0.x, cs0.y),
                        norm_rot2(v.y, f, w0.z, w0.w, cs0.z, cs0.w),
                        norm_rot2(v.z, f, w1.x, w1.y, cs1.x, cs1.y),
                        norm_rot2(v.w, f, w1.z, w1.w, cs1.z, cs1.w));
    };
    if (kRows) {
#pragma unroll
      for (int k = 0; k < kRows; ++k)
        if (hsub + 2 * k < nh)
          out[(hsub + 2 * k) * hstep] = turned(x[k], hsub + 2 * k);
    } else {
#pragma unroll 4
      for (int h = hsub; h < nh; h += 2) out[h * hstep] = turned(in[h * 16], h);
    }
  }
}

int page_shift_of(int page_size) {
  int s = 0;
  while ((1 << s) < page_size) ++s;
  return s;
}

// 16 if a cluster of 16 plan CTAs can be resident on the device, else 8.
unsigned big_cluster(int dev) {
  static std::mutex mu;
  static unsigned size[64];
  if (dev < 0 || dev >= 64) return 8;
  std::lock_guard<std::mutex> lock(mu);
  if (size[dev] == 0) {
    size[dev] = 8;
    if (cudaFuncSetAttribute(paged_plan_kernel<kPlanThreads>,
                             cudaFuncAttributeNonPortableClusterSizeAllowed,
                             1) == cudaSuccess) {
      cudaLaunchConfig_t cfg = {};
      cfg.gridDim = dim3(16);
      cfg.blockDim = dim3(kPlanThreads);
      cudaLaunchAttribute at[1];
      at[0].id = cudaLaunchAttributeClusterDimension;
      at[0].val.clusterDim.x = 16;
      at[0].val.clusterDim.y = 1;
      at[0].val.clusterDim.z = 1;
      cfg.attrs = at;
      cfg.numAttrs = 1;
      int n = 0;
      if (cudaOccupancyMaxActiveClusters(&n, paged_plan_kernel<kPlanThreads>,
                                         &cfg) == cudaSuccess &&
          n > 0)
        size[dev] = 16;
    }
    cudaGetLastError();
  }
  return size[dev];
}

int device_sms(int dev) {
  int n = 0;
  if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) !=
      cudaSuccess)
    return 0;
  return n;
}

}  // namespace
}  // namespace paged
}  // namespace wan

extern "C" {

size_t wan_paged_work_bytes(int n_streams) {
  if (n_streams < 1 || n_streams > wan::paged::kMaxStreams) return 0;
  return sizeof(int32_t) *
         (wan::paged::kHdr + static_cast<size_t>(wan::paged::kEnt) * n_streams);
}

int wan_paged_plan(const wan_paged_t* c, const int32_t* new_lens, void* s) {
  using namespace wan;
  using namespace wan::paged;
  int st = check_cache(c);
  if (st != WAN_OK) return st;
  if (!new_lens) return WAN_EINVAL;
  int dev = 0;
  if ((st = check_device(&dev)) != WAN_OK) return st;
  PlanArgs a;
  a.c = *c;
  a.new_lens = new_lens;
  a.page_shift = page_shift_of(c->page_size);
  a.sms = device_sms(dev);
  if (a.sms < 1 || a.sms * kFewCtasPerSm > kMaxCtas) return WAN_ECUDA;
  a.few = few_mode(c) ? 1 : 0;
  a.kind = work_kind(c);
  a.pack = tile_pack(c);
  a.tile_tokens = tile_tokens(c);
  cudaLaunchConfig_t cfg = {};
  // A cluster of 8 up to 32,768 records, of 16 beyond where the device can run
  // one (114,041 records of 48 streams: 13.4 us with 16, 18.7 with 8).  One
  // CTA is no faster for a few records (7.5 us) and takes 33 us where streams
  // end that held thousands of pages.
  const bool few = c->n_streams <= kPlanStreamsFew &&
                   a.sms <= kPlanThreadsFew && c->token_cap <= 32768;
  const unsigned ctas = c->token_cap <= 32768 ? 8 : big_cluster(dev);
  cfg.gridDim = dim3(ctas);
  cfg.blockDim = dim3(few ? kPlanThreadsFew : kPlanThreads);
  cfg.stream = as_stream(s);
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = ctas;
  at[0].val.clusterDim.y = 1;
  at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg,
                            few ? paged_plan_kernel<kPlanThreadsFew>
                                : paged_plan_kernel<kPlanThreads>,
                            a) == cudaSuccess
             ? WAN_OK
             : WAN_ECUDA;
}

int wan_paged_write(const wan_paged_t* c, const void* q, void* q_out,
                    const void* k, const void* v, const float* wq,
                    const float* wk, void* k_pages, void* v_pages,
                    const void* d_table, float eps, void* s) {
  using namespace wan;
  using namespace wan::paged;
  int st = check_cache(c);
  if (st != WAN_OK) return st;
  const void* all[] = {q, q_out, k, v, wq, wk, k_pages, v_pages, d_table};
  for (const void* p : all)
    if (!p) return WAN_EINVAL;
  if (!(eps > 0.f) || k_pages == v_pages || q == k || q_out == k ||
      q_out == v || q_out == k_pages || q_out == v_pages || k == k_pages ||
      v == v_pages)
    return WAN_EINVAL;
  for (const void* p : all)
    if (!aligned16(p)) return WAN_EALIGN;
  int dev = 0;
  if ((st = check_device(&dev)) != WAN_OK) return st;
  WriteArgs a;
  a.in[0] = static_cast<const uint4*>(q);
  a.in[1] = static_cast<const uint4*>(k);
  a.in[2] = static_cast<const uint4*>(v);
  a.out[0] = static_cast<uint4*>(q_out);
  a.out[1] = static_cast<uint4*>(k_pages);
  a.out[2] = static_cast<uint4*>(v_pages);
  a.w[0] = reinterpret_cast<const float4*>(wq);
  a.w[1] = reinterpret_cast<const float4*>(wk);
  a.table = static_cast<const float4*>(d_table);
  a.tokens = reinterpret_cast<const int4*>(c->tokens);
  a.n_rows = c->q_start + c->n_streams;
  a.rows = c->token_cap;
  a.heads = c->heads;
  a.kv_heads = c->kv_heads;
  a.F = c->grid.F;
  a.H = c->grid.H;
  a.W = c->grid.W;
  a.page_shift = page_shift_of(c->page_size);
  a.slots = c->n_pages * c->page_size;
  a.eps = eps;
  void (*kern)(WriteArgs) =
      c->heads <= 8    ? paged_write_kernel<4>
      : c->heads <= 12 ? paged_write_kernel<6>
      : c->heads <= 16 ? paged_write_kernel<8>
      : c->heads <= 24 ? paged_write_kernel<12>
      : c->heads <= 2 * kWrMaxRows
          ? paged_write_kernel<kWrMaxRows>
          : paged_write_kernel<0>;
  const int64_t blocks = (3ll * a.rows + kWrWarps - 1) / kWrWarps;
  kern<<<static_cast<unsigned>(blocks), kWrThreads, 0, as_stream(s)>>>(a);
  return cudaGetLastError() == cudaSuccess ? WAN_OK : WAN_ECUDA;
}

}  // extern "C"
