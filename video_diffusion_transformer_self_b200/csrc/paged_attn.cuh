// paged_attn.cuh -- attention of the new tokens of several streams over a
// paged K / V cache (part of attention.cu, whose tile and softmax pieces it
// uses).
//
// Long-video survey (atlascloud.ai), section "Route 3 · Self Forcing": chunk
// after chunk against a KV cache.  For the row at position a of a stream,
//   o = sum_j p_j v_j / sum_j p_j,  p_j = 2^(q . k_j scale log2(e) - m),
// over the keys lo(a) <= j < hi(a) of its chunk rule and window (paged.cuh),
// with the running maximum m of the online softmax.  Position j lies in row
// j % page_size of page block_table[stream][j / page_size]; a page's rows of
// one head are contiguous, so one TMA box per page and 64-channel half
// brings it into a tile.  A page that is not in [0, n_pages) is asked for
// past the tensor map's end, which reads zeros.
//
// Two kernels, chosen by the host from max_new * heads / kv_heads, the most
// rows that share a key head (the plan divides the work for one of them):
//   up to 16  paged_few_kernel: bound by the cache's bytes.
//   above     paged_tile_kernel: bound by the tensor cores.
#include "paged.cuh"

namespace wan {
namespace {
namespace pg = paged;

struct PagedArgs {
  wan_paged_t c;
  const __nv_bfloat16* q;
  __nv_bfloat16* o;
  float* part_o;       // [slot][rows][128] unnormalised fp32 O
  float2* part_ml;     // [slot][rows] (row max in log2 units, row sum)
  float scale_log2;
  int group;           // query heads of one key head
  int page_shift;
  int box_shift;       // rows of one TMA box, min(page_size, 64)
  int pack, tile_tokens;  // heads and tokens of a row tile
  uint32_t pack_inv;   // ceil(2^16 / pack)
  int kind;            // the work list's H_KIND
};

// A work list that was made for another descriptor (another max_new, say, by
// a graph replayed since) would be read as other heads and tokens, past o
// even: nothing is written then, and the device status word says so.  Once a
// call, by the main kernel; a list never planned (zeros) is an empty step.
__device__ __forceinline__ void report_kind(int kind) {
  if (blockIdx.x == 0 && threadIdx.x == 0 && kind != pg::kModeNone)
    atomicCAS(&g_wan_status, 0, WAN_EINVAL);
}

// TMA: 3-D tiled bulk tensor load into shared memory.
__device__ __forceinline__ void tma_load_3d(void* dst, const CUtensorMap* map,
                                            uint64_t* bar, int c0, int c1,
                                            int c2) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::"
      "complete_tx::bytes [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(
          smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(c0),
      "r"(c1), "r"(c2)
      : "memory");
}

// Page of position pos of a stream, as a tensor-map coordinate.
__device__ __forceinline__ int page_of(const PagedArgs& a, int stream,
                                       int64_t pos) {
  const int64_t p = pos >> a.page_shift;
  int page = -1;
  if (p < a.c.max_pages)
    page = a.c.block_table[static_cast<int64_t>(stream) * a.c.max_pages + p];
  return page >= 0 && page < a.c.n_pages ? page : a.c.n_pages;
}

// Last entry of the work list whose field f, times mul, is <= x (the first
// one's is 0).  By the whole warp, with the same x: one round of loads for up
// to 32 entries, two for the rest.
__device__ __forceinline__ const int32_t* find_entry(const int32_t* work,
                                                     int n, int f, int mul,
                                                     int x) {
  const int32_t* list = work + pg::kHdr;
  if (n <= 1) return list;
  const int lane = threadIdx.x & 31;
  const int step = (n + 31) >> 5;
  int i = lane * step;
  unsigned at = __ballot_sync(
      0xffffffffu, i < n && __ldg(list + pg::kEnt * i + f) * mul <= x);
  int first = (31 - __clz(at)) * step;
  if (step > 1) {
    i = first + lane;
    at = __ballot_sync(0xffffffffu, lane < step && i < n &&
                                        __ldg(list + pg::kEnt * i + f) * mul <=
                                            x);
    first += 31 - __clz(at);
  }
  return list + pg::kEnt * first;
}

// Waits until the kernel before this one on the stream has finished (the
// joins are launched early, while it still runs).
__device__ __forceinline__ void grid_dependency_wait() {
  asm volatile("griddepcontrol.wait;" ::: "memory");
}

__device__ __forceinline__ void launch_dependents() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

// Weighted sum of a row's partial results: lane l holds channels 4 l .. + 3.
template <int kBatch>
struct JoinAcc {
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  float m = -INFINITY, l = 0.f;
  // Parts 0 .. n - 1 (those that has(k) says were written), part k at
  // row_of(k) of the workspace.  32 parts at a time: their maxima and sums
  // come with one load a lane, their O rows with batches of independent
  // loads, the first of them before the maxima are there (loads under a
  // condition ran one after the other: 25 parts took 13 us instead of 4).
  // A part without keys (a sum of exactly 0; any other holds its maximum's
  // weight of 1) is loaded too, whatever it holds, and dropped.  A NaN sum
  // goes into the row's, and so into the result.
  template <typename RowOf, typename Has>
  __device__ __forceinline__ void add_all(int n, int lane, const PagedArgs& a,
                                          RowOf row_of, Has has) {
    for (int k0 = 0; k0 < n; k0 += 32) {
      const int cnt = min(n - k0, 32);
      float4 v[kBatch];
      auto load = [&](int b) {
#pragma unroll
        for (int k = 0; k < kBatch; ++k)
          v[k] = reinterpret_cast<const float4*>(
              a.part_o + row_of(k0 + min(b + k, cnt - 1)) * HD)[lane];
      };
      float2 ml = make_float2(-INFINITY, 0.f);
      if (lane < cnt && has(k0 + lane)) ml = a.part_ml[row_of(k0 + lane)];
      load(0);
      const bool some = ml.y != 0.f;
      if (!__any_sync(0xffffffffu, some)) continue;
      float top = some ? ml.x : -INFINITY;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1)
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
      const float mn = fmaxf(m, top);
      const float w0 = m == -INFINITY ? 0.f : ex2(m - mn);
      const float w = some ? ex2(ml.x - mn) : 0.f;
      float sum = ml.y * w;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1)
        sum += __shfl_xor_sync(0xffffffffu, sum, o);
      l = fmaf(l, w0, sum);
      m = mn;
      acc = make_float4(acc.x * w0, acc.y * w0, acc.z * w0, acc.w * w0);
      for (int b = 0;;) {
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
          const float wk = __shfl_sync(0xffffffffu, w, (b + k) & 31);
          if (b + k < cnt && wk > 0.f) {
            acc.x = fmaf(v[k].x, wk, acc.x);
            acc.y = fmaf(v[k].y, wk, acc.y);
            acc.z = fmaf(v[k].z, wk, acc.z);
            acc.w = fmaf(v[k].w, wk, acc.w);
          }
        }
        b += kBatch;
        if (b >= cnt) break;
        load(b);
      }
    }
  }
  __device__ __forceinline__ void write(__nv_bfloat16* dst, int lane) const {
    const float inv = l == 0.f ? 0.f : 1.f / l;
    reinterpret_cast<uint2*>(dst)[lane] =
        make_uint2(pack_bf16x2(acc.x * inv, acc.y * inv),
                   pack_bf16x2(acc.z * inv, acc.w * inv));
  }
};

// ============================================================== few rows ==
//
// The cache's bytes bound this: per key and head 512 bytes are read for at
// most 16 rows, 32 operations a byte, so the legacy mma.sync (m16n8k16) is
// fast enough and keeps everything in registers.  The step's (stream, key
// head, 64-key stage) items form one line that is cut into equal parts, one
// per CTA, so every SM reads the same number of bytes whatever the streams'
// lengths.  Each of a CTA's four warps takes 16 keys of every stage (4 KB of
// K and of V, contiguous in their page) through a 3-deep ring of its own,
// filled with cp.async, so no warp waits for another until the CTA leaves an
// item and the four softmax states are joined; the ring runs on across
// items.  Two CTAs per SM keep up to 192 KB in flight.  An item that several
// CTAs share is written as partial results (at most two per CTA) and joined
// by paged_few_join.  Measured, join included: 24 streams x 8 key heads x
// 32,760 keys (3.2 GB) 488 us, 6.6 TB/s; 24 ragged streams (689 MB) 122 us,
// 5.6 TB/s; 1 token x 12 heads x 7,800 keys (48 MB) 13.8 us, 5.3 of them two
// launches and the chain work list -> block table -> keys.
namespace few {
constexpr int kWarps = 4;
constexpr int kThreads = 32 * kWarps;
constexpr int kDepth = 3;
constexpr int kKeys = pg::kStage / kWarps;     // keys of a warp's part: 16
constexpr uint32_t kPart = kKeys * HD * 2;     // its K (or V): 4 KB
constexpr uint32_t kWarpRing = kDepth * 2 * kPart;
constexpr int kRows = pg::kFewRows;
constexpr int kJoinRow = HD + 4;  // floats; the pad spreads rows over banks
constexpr uint32_t kJoinFloats = kRows * kJoinRow + 2 * kRows;
constexpr uint32_t kSmem = kWarps * kWarpRing + 2 * kJoinFloats * 4;
static_assert(kKeys == 16, "one k-step of P V, and never two pages");

struct Segment {
  int stream, head, kv, ql, q0;  // q0: packed row of the stream's first row
  int stage0, n;                 // stages [stage0, stage0 + n) of 64 keys
  bool whole;                    // the item in full
};

// The work list as a warp holds it: lane i has entry i of up to 32, read
// together with the header; longer lists are searched in memory.
struct List {
  int4 e0, e1;
  int active;
};

__device__ __forceinline__ List read_list(const PagedArgs& a) {
  List t;
  const int lane = threadIdx.x & 31;
  const int4* e = reinterpret_cast<const int4*>(a.c.work + pg::kHdr) +
                  pg::kEnt / 4 * min(lane, a.c.n_streams - 1);
  t.e0 = __ldg(e);
  t.e1 = __ldg(e + 1);
  return t;
}

// The part of an item that starts at x, up to x1 on the line.  By the whole
// warp, with the same x.
__device__ __forceinline__ Segment segment_at(const PagedArgs& a,
                                              const List& t, int x, int x1) {
  const unsigned all = 0xffffffffu;
  const int kvh = a.c.kv_heads;
  const int lane = threadIdx.x & 31;
  int4 e0, e1;
  if (t.active <= 32) {
    const int i =
        31 - __clz(__ballot_sync(all, lane < t.active && t.e0.y * kvh <= x));
    e0 = make_int4(__shfl_sync(all, t.e0.x, i), __shfl_sync(all, t.e0.y, i),
                   __shfl_sync(all, t.e0.z, i), __shfl_sync(all, t.e0.w, i));
    e1 = make_int4(__shfl_sync(all, t.e1.x, i), __shfl_sync(all, t.e1.y, i),
                   __shfl_sync(all, t.e1.z, i), 0);
  } else {
    const int4* e = reinterpret_cast<const int4*>(
        find_entry(a.c.work, t.active, pg::E_BASE, kvh, x));
    e0 = __ldg(e);
    e1 = __ldg(e + 1);
  }
  Segment s;
  s.stream = e0.x;
  // (at least one stage, so that the walk ends whatever the list holds)
  const int n = max(e0.z, 1);
  const int local = x - e0.y * kvh;
  s.head = local / n;
  const int at = local - s.head * n;
  s.n = max(min(n - at, x1 - x), 1);
  s.whole = s.n == n;
  s.stage0 = e0.w + at;
  s.kv = e1.x;
  s.ql = e1.y;
  s.q0 = e1.z;
  return s;
}

// 16 bytes global -> shared, zeros instead of the global bytes if !live.
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src,
                                           bool live) {
  const int n = live ? 16 : 0;
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst),
               "l"(src), "r"(n)
               : "memory");
}
__device__ __forceinline__ void cp_async_commit() {
  asm volatile("cp.async.commit_group;" ::: "memory");
}
template <int kPending>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(kPending) : "memory");
}

// Row r, 16-byte chunk c of a warp's 16 rows of 256 bytes: the chunk's low
// bits are turned by the row, so that the 8 rows of an ldmatrix lie in
// different banks.
__device__ __forceinline__ uint32_t swz(int r, int c) {
  return r * 256 + ((c ^ (r & 7)) << 4);
}

__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile(
      "ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
      : "r"(addr)
      : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile(
      "ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
      : "r"(addr)
      : "memory");
}
__device__ __forceinline__ void mma16816(float (&d)[4],
                                         const uint32_t (&a)[4], uint32_t b0,
                                         uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 "
      "{%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__global__ void __launch_bounds__(kThreads, pg::kFewCtasPerSm)
    paged_few_kernel(const __nv_bfloat16* __restrict__ k_pages,
                     const __nv_bfloat16* __restrict__ v_pages,
                     const __grid_constant__ PagedArgs args) {
  extern __shared__ __align__(128) uint8_t smem_raw[];
  const int32_t* work = args.c.work;
  List list = read_list(args);
  // {H_KIND, H_ACTIVE, H_TOTAL, H_CTAS}
  const int4 hdr = __ldg(reinterpret_cast<const int4*>(work));
  const int cta = blockIdx.x;
  if (hdr.x != args.kind) {
    report_kind(hdr.x);
    return;
  }
  if (hdr.y < 1 || cta >= hdr.w) return;
  list.active = hdr.y;
  const pg::Line line(hdr.z, hdr.w);
  const int x0 = line.first(cta), x1 = line.first(cta + 1);
  launch_dependents();
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  float* join = reinterpret_cast<float*>(smem_raw + kWarps * kWarpRing);
  const uint32_t ring = smem_u32(smem_raw) + warp * kWarpRing;
  const float c2 = args.scale_log2;
  const int heads = args.c.heads;
  const int page_mask = (1 << args.page_shift) - 1;
  const int64_t head_bytes = 256ll << args.page_shift;
  const int64_t page_bytes = head_bytes * args.c.kv_heads;

  // The loading side: stage lj of segment ls is the next one to fetch.
  Segment ls = segment_at(args, list, x0, x1);
  int lx = x0;
  int lj = 0, lg = 0;
  // pages of this warp's part of the segment's stages, 32 at a time (one a
  // lane: a read a stage sat between the fetches)
  auto pages_from = [&](int j) {
    return page_of(args, ls.stream,
                   static_cast<int64_t>(ls.stage0 + j + lane) * pg::kStage +
                       warp * kKeys);
  };
  int pages = pages_from(0);
  const int total_stages = x1 - x0;
  const uint32_t dst0 = swz(lane >> 4, lane & 15);
  auto fetch = [&]() {
    if (lg < total_stages) {
      const int64_t pos =
          static_cast<int64_t>(ls.stage0 + lj) * pg::kStage + warp * kKeys;
      const int lpage = __shfl_sync(0xffffffffu, pages, lj & 31);
      const bool live = lpage < args.c.n_pages;
      const int64_t off =
          (live ? lpage * page_bytes + ls.head * head_bytes +
                      (static_cast<int>(pos) & page_mask) * 256
                : 0) +
          lane * 16;
      const uint32_t st = ring + (lg % kDepth) * (2 * kPart);
      const char* kg = reinterpret_cast<const char*>(k_pages) + off;
      const char* vg = reinterpret_cast<const char*>(v_pages) + off;
      // piece i: rows 2 i and 2 i + 1; their swizzle is (2 i + lane / 16) & 7
#pragma unroll
      for (int i = 0; i < 8; ++i)
        cp_async16(st + i * 512 + (dst0 ^ ((2 * i & 7) << 4)), kg + i * 512,
                   live);
#pragma unroll
      for (int i = 0; i < 8; ++i)
        cp_async16(st + kPart + i * 512 + (dst0 ^ ((2 * i & 7) << 4)),
                   vg + i * 512, live);
      ++lg;
      if (++lj == ls.n) {
        lx += ls.n;
        lj = 0;
        if (lx < x1) {
          ls = segment_at(args, list, lx, x1);
          pages = pages_from(0);
        }
      } else if ((lj & 31) == 0) {
        pages = pages_from(lj);
      }
    }
    cp_async_commit();  // an empty group keeps the count
  };
  // Fragments of m16n8k16: thread (gr, t4) = (lane / 4, lane % 4) holds rows
  // gr and gr + 8, columns 2 t4, 2 t4 + 1 (+ 8) of A and of the results.
  const int gr = lane >> 2, t4 = lane & 3;
  // rows gr and gr + 8 of a segment: row r is query head head * group +
  // r % group of new token r / group
  uint32_t qf[8][4];
  int lo[2], hi[2], item_lo;
  int64_t orow[2];
  auto load_rows = [&](const Segment& s) {
    const int4 cfg =
        __ldg(reinterpret_cast<const int4*>(args.c.streams) + s.stream);
    const int rows = min(s.ql * args.group, kRows);
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int r = gr + 8 * e;
      const int i = r / args.group;
      orow[e] = (static_cast<int64_t>(s.q0) + i) * heads +
                s.head * args.group + (r - i * args.group);
      const bool on = r < rows && s.q0 + i < args.c.token_cap;
      if (!on) orow[e] = -1;
      const uint32_t* src = reinterpret_cast<const uint32_t*>(
          args.q + (on ? orow[e] : 0) * HD);
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        qf[k][e] = on ? __ldg(src + k * 8 + t4) : 0u;
        qf[k][2 + e] = on ? __ldg(src + k * 8 + 4 + t4) : 0u;
      }
      // a row of padding takes part unmasked and is never written
      const int a = s.kv - s.ql + i;
      lo[e] = on ? pg::key_lo(max(a, 0), cfg.z, cfg.w) : 0;
      hi[e] = on ? pg::key_hi(a, cfg.z, s.kv) : INT32_MAX;
    }
    item_lo = pg::key_lo(max(s.kv - s.ql, 0), cfg.z, cfg.w);
  };
  // the first rows' reads are under way before the first fetches wait for
  // their pages
  Segment s = ls;
  load_rows(s);
#pragma unroll
  for (int i = 0; i < kDepth - 1; ++i) fetch();
  int g = 0;
  for (int x = x0;;) {
    float o[16][4];
#pragma unroll
    for (int d = 0; d < 16; ++d)
      o[d][0] = o[d][1] = o[d][2] = o[d][3] = 0.f;
    float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
    for (int j = 0; j < s.n; ++j, ++g) {
      __syncwarp();  // the ring slot that is filled next has been read
      fetch();
      cp_async_wait<kDepth - 1>();
      __syncwarp();
      const uint32_t ks = ring + (g % kDepth) * (2 * kPart);
      const uint32_t vs = ks + kPart;
      const int key0 = (s.stage0 + j) * pg::kStage + warp * kKeys;
      // S = Q K^T: two 8-key tiles, even and odd k-steps in chains of four
      float sc[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
      float sd[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
      {
        const int row = (lane & 7) + ((lane >> 4) << 3);
        const int sub = (lane >> 3) & 1;
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          uint32_t b[4];
          ldsm4(ks + swz(row, 2 * k + sub), b);
          mma16816(k & 1 ? sd[0] : sc[0], qf[k], b[0], b[1]);
          mma16816(k & 1 ? sd[1] : sc[1], qf[k], b[2], b[3]);
        }
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        sc[0][e] += sd[0][e];
        sc[1][e] += sd[1][e];
      }
      const bool edge = __any_sync(
          0xffffffffu, lo[0] > key0 || lo[1] > key0 ||
                           hi[0] < key0 + kKeys || hi[1] < key0 + kKeys);
      if (edge) {
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int key = key0 + n * 8 + 2 * t4 + (e & 1);
            if (key < lo[e >> 1] || key >= hi[e >> 1]) sc[n][e] = -INFINITY;
          }
      }
      // running maximum, kept until a row's grows by more than 2^8 (the
      // result is exact after the final division)
      bool need = false;
      float mx[2];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float v = fmaxf(fmaxf(sc[0][2 * e], sc[0][2 * e + 1]),
                        fmaxf(sc[1][2 * e], sc[1][2 * e + 1]));
        v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 1));
        v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 2));
        mx[e] = v * c2;
        need = need || mx[e] > m[e] + RESCALE_LOG2;
      }
      if (__any_sync(0xffffffffu, need)) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const bool up = mx[e] > m[e];
          const float alpha = up ? ex2(m[e] - mx[e]) : 1.f;
          if (up) m[e] = mx[e];
          l[e] *= alpha;
#pragma unroll
          for (int d = 0; d < 16; ++d) {
            o[d][2 * e] *= alpha;
            o[d][2 * e + 1] *= alpha;
          }
        }
      }
      uint32_t p[4];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const float base = m[e] == -INFINITY ? 0.f : m[e];
        const float p0 = ex2(fmaf(sc[0][2 * e], c2, -base));
        const float p1 = ex2(fmaf(sc[0][2 * e + 1], c2, -base));
        const float p2 = ex2(fmaf(sc[1][2 * e], c2, -base));
        const float p3 = ex2(fmaf(sc[1][2 * e + 1], c2, -base));
        l[e] += (p0 + p1) + (p2 + p3);
        p[e] = pack_bf16x2(p0, p1);
        p[2 + e] = pack_bf16x2(p2, p3);
      }
      // values outside [item_lo, kv) may be anything: their weight is 0, but
      // 0 * NaN is not.  vm masks this thread's keys 2 t4, + 1 and + 8, + 9.
      const bool vedge = key0 < item_lo || key0 + kKeys > s.kv;
      uint32_t vm[2] = {0xffffffffu, 0xffffffffu};
      if (vedge) {
#pragma unroll
        for (int n = 0; n < 2; ++n) {
          const int key = key0 + n * 8 + 2 * t4;
          vm[n] = (key >= item_lo && key < s.kv ? 0x0000ffffu : 0u) |
                  (key + 1 >= item_lo && key + 1 < s.kv ? 0xffff0000u : 0u);
        }
      }
      {
        const int row = lane & 15;
        const int sub = lane >> 4;
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          uint32_t b[4];
          ldsm4t(vs + swz(row, 2 * k + sub), b);
          if (vedge) {
            b[0] &= vm[0];
            b[1] &= vm[1];
            b[2] &= vm[0];
            b[3] &= vm[1];
          }
          mma16816(o[2 * k], p, b[0], b[1]);
          mma16816(o[2 * k + 1], p, b[2], b[3]);
        }
      }
    }
    // -------------------------------------------- join the four warps --
    // warps 2, 3 into 0, 1, then 1 into 0
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      l[e] += __shfl_xor_sync(0xffffffffu, l[e], 1);
      l[e] += __shfl_xor_sync(0xffffffffu, l[e], 2);
    }
    auto put = [&](float* dst) {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int r = gr + 8 * e;
        if (t4 == 0) {
          dst[kRows * kJoinRow + r] = m[e];
          dst[kRows * kJoinRow + kRows + r] = l[e];
        }
#pragma unroll
        for (int d = 0; d < 16; ++d)
          *reinterpret_cast<float2*>(dst + r * kJoinRow + d * 8 + 2 * t4) =
              make_float2(o[d][2 * e], o[d][2 * e + 1]);
      }
    };
    auto take = [&](const float* src) {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int r = gr + 8 * e;
        const float m2 = src[kRows * kJoinRow + r];
        const float mn = fmaxf(m[e], m2);
        const float w1 = m[e] == -INFINITY ? 0.f : ex2(m[e] - mn);
        const float w2 = m2 == -INFINITY ? 0.f : ex2(m2 - mn);
        l[e] = l[e] * w1 + src[kRows * kJoinRow + kRows + r] * w2;
        m[e] = mn;
#pragma unroll
        for (int d = 0; d < 16; ++d) {
          const float2 v = *reinterpret_cast<const float2*>(
              src + r * kJoinRow + d * 8 + 2 * t4);
          o[d][2 * e] = fmaf(v.x, w2, o[d][2 * e] * w1);
          o[d][2 * e + 1] = fmaf(v.y, w2, o[d][2 * e + 1] * w1);
        }
      }
    };
    __syncthreads();
    if (warp >= 2) put(join + (warp - 2) * kJoinFloats);
    __syncthreads();
    if (warp < 2) take(join + warp * kJoinFloats);
    __syncthreads();
    if (warp == 1) put(join);
    __syncthreads();
    if (warp == 0) {
      take(join);
      if (s.whole) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const float inv = l[e] > 0.f ? 1.f / l[e] : 0.f;
          if (orow[e] >= 0) {
            uint32_t* dst = reinterpret_cast<uint32_t*>(args.o + orow[e] * HD);
#pragma unroll
            for (int d = 0; d < 16; ++d)
              dst[d * 4 + t4] =
                  pack_bf16x2(o[d][2 * e] * inv, o[d][2 * e + 1] * inv);
          }
        }
      } else {
        const int64_t slot = 2ll * cta + (x != x0 ? 1 : 0);
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int r = gr + 8 * e;
          if (orow[e] < 0) continue;
          const int64_t prow = slot * kRows + r;
          if (t4 == 0) args.part_ml[prow] = make_float2(m[e], l[e]);
#pragma unroll
          for (int d = 0; d < 16; ++d)
            *reinterpret_cast<float2*>(args.part_o + prow * HD + d * 8 +
                                       2 * t4) =
                make_float2(o[d][2 * e], o[d][2 * e + 1]);
        }
      }
    }
    x += s.n;
    if (x >= x1) break;
    s = segment_at(args, list, x, x1);
    load_rows(s);
  }
}

// One warp per (stream, key head, row) whose item several CTAs shared.
__global__ void __launch_bounds__(128)
    paged_few_join(const __grid_constant__ PagedArgs args) {
  const int32_t* work = args.c.work;
  if (__ldg(work + pg::H_KIND) != args.kind) return;
  const int kvh = args.c.kv_heads;
  const int rows = min(args.c.max_new * args.group, kRows);
  const int64_t items =
      static_cast<int64_t>(__ldg(work + pg::H_ACTIVE)) * kvh * rows;
  if (items == 0) return;
  const pg::Line line(__ldg(work + pg::H_TOTAL), __ldg(work + pg::H_CTAS));
  const int lane = threadIdx.x & 31;
  const int64_t warps = static_cast<int64_t>(gridDim.x) * 4;
  grid_dependency_wait();
  for (int64_t it = blockIdx.x * 4ll + (threadIdx.x >> 5); it < items;
       it += warps) {
    const int r = static_cast<int>(it % rows);
    const int64_t ih = it / rows;
    const int head = static_cast<int>(ih % kvh);
    const int32_t* e = work + pg::kHdr + pg::kEnt * (ih / kvh);
    const int n = __ldg(e + pg::E_COUNT);
    const int xs = __ldg(e + pg::E_BASE) * kvh + head * n;
    const int c0 = line.cta_of(xs), c1 = line.cta_of(xs + n - 1);
    if (c0 == c1) continue;
    const int i = r / args.group;
    const int q0 = __ldg(e + pg::E_Q0);
    if (r >= __ldg(e + pg::E_ROWS) * args.group || q0 + i >= args.c.token_cap)
      continue;
    JoinAcc<16> acc;
    // the first CTA's part is its last one unless the item starts it
    const bool mid = xs > line.first(c0);
    acc.add_all(c1 - c0 + 1, lane, args, [&](int k) {
      return (2ll * (c0 + k) + (k == 0 && mid ? 1 : 0)) * kRows + r;
    }, [](int) { return true; });
    acc.write(args.o + ((static_cast<int64_t>(q0) + i) * args.c.heads +
                        head * args.group + (r - i * args.group)) * HD,
              lane);
  }
}
}  // namespace few

// ============================================================= row tiles ==
//
// The two-tile pipeline of attn_fwd_kernel (same warp roles, rings, tensor
// memory and softmax) fed from pages: a 128-key block is 2 to 8 TMA boxes
// per 64-channel half, one lane of the producer warp per box, the block
// table entry of the next block fetched while this one loads.  One
// persistent CTA per SM walks its share of the plan's division: rounds of
// whole units (two row tiles of a stream and head group), then its part of
// the line of the last units, so that all CTAs end together whatever the
// streams' lengths.  The producer warp works the units out ahead and hands
// them to the others through a ring in shared memory.  Query heads of one key
// head share a tile (row r: token r / pack, head r % pack), so their keys
// are read once: 6 streams x 40 heads over 8 x 43 to 86 rows 47 -> 22.4 us.
// A unit whose rows fit one tile gives both tiles the same Q rows and every
// other key block: the two softmax chains still hide each other (one chain
// alone takes about 1 us a block), and the halves are joined at the end.
// Output rows are staged in the tile's own Q buffer (free once the unit's
// last P V is done) and stored 512 contiguous bytes a warp instruction with
// a row check, since a stream's last tile ends inside the next stream's rows
// (a TMA store would overwrite them).  A unit with a part of its keys writes
// fp32 partial results instead, joined by paged_tile_join.
// Bound, like attn_fwd_kernel, by each tile's chain of softmax and matrix
// products (tensor pipe 61 % active), and by the power cap in long calls.
// Measured: 4,680 rows x 12 heads over 32,760 keys 740 to 900 us by clock
// (1,050 to 1,270 TFLOP/s), x 40 heads over 65,520 keys 5.0 to 5.85 ms (1,075
// to 1,250); with units of 256 rows a CTA in turn they took 965 us and 6.0 ms.
// 20 to 400 rows of six streams x 12 heads take 83 us: 26 key blocks a CTA of
// about 1.9 us, the rest starts and ends of units, partial results (128 KB a
// piece) and their join.  The kernel needs 44 bytes of spill stores and 72 of
// loads a thread, which attn_fwd_kernel does without.
// Rows stored from registers instead of through the Q buffer, the next unit's
// scores started meanwhile: small calls 4 % shorter to 6 % longer, long ones
// unchanged, two to three registers spilled.
namespace tile {
enum : int {
  QFULL = 0,
  KFULL = 1,
  KEMPTY = KFULL + NSK,
  VFULL = KEMPTY + NSK,
  VEMPTY = VFULL + NSV,
  SFULL = VEMPTY + NSV,    // per tile
  PREADY = SFULL + QT,     // per tile: 4 warps stored P
  OFINAL = PREADY + QT,    // per tile: a unit's last P V done
  TFREE = OFINAL + QT,     // per tile: O read and Q buffer free (4 warps)
  HALF1 = TFREE + QT,      // tile 1's half of a shared unit is done (4 warps)
  UFULL = HALF1 + 1,       // unit ring
  UEMPTY = UFULL + 4,      //   (9 warps have read the unit)
  DRAIN = UEMPTY + 4,
  NBAR
};

// Where a CTA is in its share of the work: whole unit k while k < waves,
// then place x of the line.
struct Walk {
  int k, x;
  int active, ctas, waves;  // of the work list's header
  int x0, x1;               // the CTA's part of the line
};

constexpr int kUnits = 4;  // unit ring

struct Unit {
  int stream;        // -1: the CTA's share ends here
  int head;          // first query head
  int q0;            // packed row of the first token
  int tokens;        // at most two tiles of them
  int a0;            // the first one's position
  int kv, chunk, window;
  int lo, hi;        // keys that any of the rows sees
  int kb0, nblk;     // key blocks of the part (may be none)
  int slot;          // partial-result slot, -1: the unit's keys in full
  int span;          // places of the line
};

__device__ __forceinline__ Walk walk_begin(const PagedArgs& a) {
  const int32_t* work = a.c.work;
  // {H_KIND, H_ACTIVE, H_TOTAL, H_CTAS}
  const int4 hdr = __ldg(reinterpret_cast<const int4*>(work));
  Walk w;
  w.k = 0;
  w.active = hdr.y;
  w.ctas = hdr.w;
  w.waves = __ldg(work + pg::H_WAVES);
  w.x = w.x0 = __ldg(work + pg::kLine + blockIdx.x);
  w.x1 = __ldg(work + pg::kLine + blockIdx.x + 1);
  return w;
}

__device__ __forceinline__ void walk_next(Walk& w, int span) {
  if (w.k < w.waves)
    ++w.k;
  else
    w.x += span;
}

// Key blocks of a unit's nb before place s of its `weight` places.
// (fp32: 0 and nb at the ends, and neighbours agree on the cut between them)
__device__ __forceinline__ int cut(int nb, int s, int weight) {
  return static_cast<int>(static_cast<float>(nb) *
                          (static_cast<float>(s) / static_cast<float>(weight)));
}

// The part at w; false at the end of the CTA's share.
__device__ __forceinline__ bool unit_at(const PagedArgs& a, const Walk& w,
                                        Unit& t) {
  const int32_t* work = a.c.work;
  const int32_t* e;
  int local, s0 = 0, s1 = 1, weight = 1;
  t.slot = -1;
  t.span = 0;
  if (w.k < w.waves) {
    const int c = blockIdx.x;
    const int u = w.k * w.ctas + (w.k & 1 ? w.ctas - 1 - c : c);
    e = find_entry(work, w.active, pg::E_BASE, 1, u);
    local = u - __ldg(e + pg::E_BASE);
  } else {
    if (w.x >= w.x1) return false;
    // the stream whose units hold place x, and the place among them
    e = find_entry(work, w.active, pg::E_FIRST, 1, w.x);
    const int tiles = max(__ldg(e + pg::E_COUNT), 1);
    const int full = __ldg(e + pg::E_FULL), last = __ldg(e + pg::E_LAST);
    const int64_t y =
        w.x - __ldg(reinterpret_cast<const long long*>(e + pg::E_LINE));
    int tile, off;
    const int head = pg::unit_of(y, tiles, full, last, &tile, &weight, &off);
    local = head * tiles + tile;
    // (at least one place, so that the walk ends whatever the list holds)
    t.span = max(min(weight - off, w.x1 - w.x), 1);
    s0 = off;
    s1 = off + t.span;
    if (t.span < weight) t.slot = 2 * blockIdx.x + (w.x == w.x0 ? 0 : 1);
  }
  t.stream = __ldg(e + pg::E_STREAM);
  const int tiles = __ldg(e + pg::E_COUNT);
  const int hgroup = local / tiles;
  const int tx = tiles - 1 - (local - hgroup * tiles);
  t.head = hgroup * a.pack;
  const int pair = 2 * a.tile_tokens;
  const int ql = __ldg(e + pg::E_TROWS);
  t.kv = __ldg(e + pg::E_TKV);
  t.chunk = __ldg(e + pg::E_CHUNK);
  t.window = __ldg(e + pg::E_WINDOW);
  t.q0 = __ldg(e + pg::E_TQ0) + tx * pair;
  t.tokens = min(ql - tx * pair, pair);
  t.a0 = t.kv - ql + tx * pair;
  t.lo = pg::key_lo(max(t.a0, 0), t.chunk, t.window);
  t.hi = pg::key_hi(t.a0 + t.tokens - 1, t.chunk, t.kv);
  const int b0 = t.lo / BN;
  const int nb = max((t.hi + BN - 1) / BN - b0, 0);
  t.kb0 = b0 + cut(nb, s0, weight);
  t.nblk = t.tokens > 0 ? b0 + cut(nb, s1, weight) - t.kb0 : 0;
  return true;
}

__global__ void __launch_bounds__(wan::kThreads, 1)
    paged_tile_kernel(const __grid_constant__ CUtensorMap tm_q,
                      const __grid_constant__ CUtensorMap tm_k,
                      const __grid_constant__ CUtensorMap tm_v,
                      const __grid_constant__ PagedArgs args) {
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t bar[NBAR];
  __shared__ uint32_t s_tmem;
  __shared__ int s_abort;
  __shared__ float2 s_half[BM];  // tile 1's (row max, row sum), shared units
  __shared__ Unit s_unit[kUnits];
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int kind = __ldg(args.c.work + pg::H_KIND);
  if (kind != args.kind) {
    report_kind(kind);
    return;
  }
  if (static_cast<int>(blockIdx.x) >= __ldg(args.c.work + pg::H_CTAS) ||
      __ldg(args.c.work + pg::H_TOTAL) < 1)
    return;
  launch_dependents();
  volatile int* abort_flag = &s_abort;
  int* status = &g_wan_status;
  const uint32_t raw = smem_u32(smem_raw);
  uint8_t* sm = smem_raw + (((raw + 1023u) & ~1023u) - raw);
  uint8_t* sQ = sm;
  uint8_t* sK = sm + QT * TILE;
  uint8_t* sV = sK + NSK * TILE;
  if (threadIdx.x == 0) {
    s_abort = 0;
    mbar_init(&bar[QFULL], 1);
    for (int i = 0; i < NSK; ++i) {
      mbar_init(&bar[KFULL + i], 1);
      mbar_init(&bar[KEMPTY + i], 1);
    }
    for (int i = 0; i < NSV; ++i) {
      mbar_init(&bar[VFULL + i], 1);
      mbar_init(&bar[VEMPTY + i], 1);
    }
    for (int t = 0; t < QT; ++t) {
      mbar_init(&bar[SFULL + t], 1);
      mbar_init(&bar[PREADY + t], 4);
      mbar_init(&bar[OFINAL + t], 1);
      mbar_init(&bar[TFREE + t], 4);
    }
    mbar_init(&bar[HALF1], 4);
    for (int i = 0; i < kUnits; ++i) {
      mbar_init(&bar[UFULL + i], 1);
      mbar_init(&bar[UEMPTY + i], 9);
    }
    mbar_init(&bar[DRAIN], 1);
    fence_mbar_init();
  }
  if (warp == 9) tmem_alloc(&s_tmem, TMEM_COLS);
  // the first unit is worked out while tensor memory is allocated
  Walk w;
  Unit u0;
  if (warp == 8) {
    w = walk_begin(args);
    if (!unit_at(args, w, u0)) u0.stream = -1;
    if (lane == 0) {
      prefetch_tmap(&tm_q);
      prefetch_tmap(&tm_k);
      prefetch_tmap(&tm_v);
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = s_tmem;

  if (warp >= 8) {
    setmaxnreg_dec();
    if (warp == 8) {
      // ---------------------------------------------------- TMA producer --
      const bool leader = elect_one();
      const int boxes = BN >> args.box_shift;
      const uint32_t box_bytes = 128u << args.box_shift;
      const int in_mask = (1 << args.page_shift) - 1;
      const int row0 = lane << args.box_shift;  // this lane's box
      bool ok = true;
      int nq = 0, nq1 = 0;  // units of tile 0, of tile 1
      int nk = 0, nv = 0;   // K and V tiles issued
      const uint32_t q_bytes = 256u * args.pack * args.tile_tokens;
      Unit c = u0;
      for (int nu = 0; ok; ++nu) {
        if (nu > 0 && !unit_at(args, w, c)) c.stream = -1;
        const int us = nu % kUnits;
        if (nu >= kUnits)
          ok = wait_warp(&bar[UEMPTY + us], (nu / kUnits - 1) & 1, abort_flag,
                         status);
        if (!ok) break;
        if (lane == 0) {
          s_unit[us] = c;
          mbar_arrive(&bar[UFULL + us]);
        }
        __syncwarp();
        if (c.stream < 0) break;
        walk_next(w, c.span);
        if (c.nblk == 0) continue;
        const bool two = c.tokens > args.tile_tokens;
        int64_t pos = static_cast<int64_t>(c.kb0) * BN + row0;
        int page = lane < boxes ? page_of(args, c.stream, pos) : 0;
        if (nq > 0)
          ok = wait_warp(&bar[TFREE + 0], (nq - 1) & 1, abort_flag, status);
        if (ok && two && nq1 > 0)
          ok = wait_warp(&bar[TFREE + 1], (nq1 - 1) & 1, abort_flag, status);
        if (!ok) break;
        if (leader) {
          mbar_expect_tx(&bar[QFULL], two ? QT * q_bytes : q_bytes);
          for (int t = 0; t < (two ? QT : 1); ++t) {
            const int row = c.q0 + t * args.tile_tokens;
            tma_load_3d(sQ + t * TILE, &tm_q, &bar[QFULL], 0, c.head, row);
            tma_load_3d(sQ + t * TILE + HALF, &tm_q, &bar[QFULL], 64, c.head,
                        row);
          }
        }
        ++nq;
        nq1 += two || c.nblk > 1;
        const int kvhead = c.head / args.group;
        for (int j = 0; j < c.nblk && ok; ++j) {
          const int g = nk;
          const int in_page = static_cast<int>(pos) & in_mask;
          const int sk = g % NSK, uk = g / NSK;
          if (uk > 0)
            ok = wait_warp(&bar[KEMPTY + sk], (uk - 1) & 1, abort_flag, status);
          if (!ok) break;
          if (leader) mbar_expect_tx(&bar[KFULL + sk], TILE);
          __syncwarp();
          if (lane < boxes) {
            uint8_t* dst = sK + sk * TILE + lane * box_bytes;
            tma_load_4d(dst, &tm_k, &bar[KFULL + sk], 0, in_page, kvhead, page);
            tma_load_4d(dst + HALF, &tm_k, &bar[KFULL + sk], 64, in_page,
                        kvhead, page);
          }
          ++nk;
          const int sv = g % NSV, uv = g / NSV;
          if (uv > 0)
            ok = wait_warp(&bar[VEMPTY + sv], (uv - 1) & 1, abort_flag, status);
          if (!ok) break;
          if (leader) mbar_expect_tx(&bar[VFULL + sv], TILE);
          __syncwarp();
          if (lane < boxes) {
            uint8_t* dst = sV + sv * TILE + lane * box_bytes;
            tma_load_4d(dst, &tm_v, &bar[VFULL + sv], 0, in_page, kvhead, page);
            tma_load_4d(dst + HALF, &tm_v, &bar[VFULL + sv], 64, in_page,
                        kvhead, page);
            pos += BN;
            if (j + 1 < c.nblk) page = page_of(args, c.stream, pos);
          }
          ++nv;
          __syncwarp();
        }
      }
      if (*abort_flag) {
        // copies already issued land before the CTA leaves
        if (nq > 0) wait_warp_drain(&bar[QFULL], (nq - 1) & 1, status);
        for (int g = (nk > NSK ? nk - NSK : 0); g < nk; ++g)
          wait_warp_drain(&bar[KFULL + g % NSK], (g / NSK) & 1, status);
        for (int g = (nv > NSV ? nv - NSV : 0); g < nv; ++g)
          wait_warp_drain(&bar[VFULL + g % NSV], (g / NSV) & 1, status);
      }
    } else if (warp == 9) {
      // ------------------------------------------------------ MMA issuer --
      const uint64_t dq = sdesc_sw128(smem_u32(sQ), 16, 1024);
      const uint64_t dk = sdesc_sw128(smem_u32(sK), 16, 1024);
      const uint64_t dv = sdesc_sw128(smem_u32(sV), HALF, 1024);
      const bool leader = elect_one();
      // scores of tile t (whose Q rows are in buffer qb) for ring block g
      auto issue_s = [&](int t, int qb, int g) {
        const uint64_t a0 = dq + ((qb * TILE) >> 4);
        const uint64_t b0 = dk + (((g % NSK) * TILE) >> 4);
        const uint32_t d = tmem + t * 128;
        if (leader) {
#pragma unroll
          for (int k = 0; k < HD / 16; ++k) {
            const uint32_t off = ((k >> 2) * HALF + (k & 3) * 32) >> 4;
            umma_ss(d, a0 + off, b0 + off, IDESC_S, k > 0 ? 1u : 0u);
          }
          umma_commit(&bar[SFULL + t]);
        }
        __syncwarp();
      };
      auto commit = [&](uint64_t* b) {
        if (leader) umma_commit(b);
        __syncwarp();
      };
      // Waits for V of block g and clears the rows that no row of the unit
      // sees (before its window, behind its last key): they may hold
      // anything, and 0 * NaN is not 0.
      auto ready_v = [&](int g, int kb, const Unit& c) -> bool {
        if (!wait_warp(&bar[VFULL + g % NSV], (g / NSV) & 1, abort_flag,
                       status))
          return false;
        const int first = c.lo - kb * BN, last = c.hi - kb * BN;
        if (first > 0 || last < BN) {
          uint8_t* vt = sV + (g % NSV) * TILE;
          for (int idx = lane; idx < BN * 16; idx += 32) {
            const int r = idx >> 4, ch = idx & 15;
            if (r < first || r >= last)
              *reinterpret_cast<uint4*>(vt + (ch >> 3) * HALF + r * 128 +
                                        ((ch & 7) << 4)) =
                  make_uint4(0, 0, 0, 0);
          }
          fence_proxy_async_smem();
          __syncwarp();
        }
        return true;
      };
      // O_t += P_t V of ring block g; gt: tile t's own count of blocks, jl:
      // the block's place in the unit, nt: the tile's units before this one.
      auto pv = [&](int t, int g, int gt, int jl, int nt) -> bool {
        if (jl == 0 && nt > 0 &&
            !wait_warp(&bar[TFREE + t], (nt - 1) & 1, abort_flag, status))
          return false;
        if (!wait_warp(&bar[PREADY + t], gt & 1, abort_flag, status))
          return false;
        tc_fence_after();
        const uint64_t b0 = dv + (((g % NSV) * TILE) >> 4);
        if (leader) {
#pragma unroll
          for (int k = 0; k < BN / 16; ++k)
            umma_ts(tmem + TM_O + t * 128, tmem + t * 128 + k * 8,
                    b0 + ((k * 2048) >> 4), IDESC_PV,
                    (jl > 0 || k > 0) ? 1u : 0u);
        }
        __syncwarp();
        return true;
      };
      bool ok = true;
      int g0 = 0;              // ring blocks of earlier units
      int b0 = 0, b1 = 0;      // blocks of each tile in earlier units
      int n0 = 0, n1 = 0;      // units of each tile before this one
      for (int nu = 0; ok; ++nu) {
        const int us = nu % kUnits;
        ok = wait_warp(&bar[UFULL + us], (nu / kUnits) & 1, abort_flag,
                       status);
        if (!ok) break;
        const Unit c = s_unit[us];
        __syncwarp();
        if (lane == 0) mbar_arrive(&bar[UEMPTY + us]);
        if (c.stream < 0) break;
        if (c.nblk == 0) continue;
        const bool two = c.tokens > args.tile_tokens;
        ok = wait_warp(&bar[QFULL], n0 & 1, abort_flag, status);
        if (two) {
          for (int j = 0; j < c.nblk && ok; ++j) {
            const int g = g0 + j;
            if (j > 0) {
              ok = ready_v(g - 1, c.kb0 + j - 1, c) &&
                   pv(0, g - 1, b0 + j - 1, j - 1, n0);
              if (!ok) break;
            }
            ok = wait_warp(&bar[KFULL + g % NSK], (g / NSK) & 1, abort_flag,
                           status);
            if (!ok) break;
            tc_fence_after();
            issue_s(0, 0, g);
            if (j > 0) {
              ok = pv(1, g - 1, b1 + j - 1, j - 1, n1);
              if (!ok) break;
              commit(&bar[VEMPTY + (g - 1) % NSV]);
            }
            issue_s(1, 1, g);
            commit(&bar[KEMPTY + g % NSK]);
          }
          if (ok) {
            const int jl = c.nblk - 1, g = g0 + jl;
            ok = ready_v(g, c.kb0 + jl, c) && pv(0, g, b0 + jl, jl, n0);
            if (ok) {
              commit(&bar[OFINAL + 0]);
              ok = pv(1, g, b1 + jl, jl, n1);
            }
            if (ok) {
              commit(&bar[OFINAL + 1]);
              commit(&bar[VEMPTY + g % NSV]);
            }
          }
          b0 += c.nblk;
          b1 += c.nblk;
          ++n0;
          ++n1;
        } else {
          // one row tile: block j runs on tile j & 1, its P V two blocks on
          const int pairs = c.nblk > 1 ? 2 : 1;
          for (int j = 0; j < c.nblk + pairs && ok; ++j) {
            const int t = pairs == 2 ? j & 1 : 0;
            if (j >= pairs) {
              const int jv = j - pairs, g = g0 + jv, own = jv / pairs;
              ok = ready_v(g, c.kb0 + jv, c) &&
                   pv(t, g, (t ? b1 : b0) + own, own, t ? n1 : n0);
              if (!ok) break;
              commit(&bar[VEMPTY + g % NSV]);
              // the tile's last block
              if (j >= c.nblk) commit(&bar[OFINAL + t]);
            }
            if (j < c.nblk) {
              const int g = g0 + j;
              ok = wait_warp(&bar[KFULL + g % NSK], (g / NSK) & 1, abort_flag,
                             status);
              if (!ok) break;
              tc_fence_after();
              issue_s(t, 0, g);
              commit(&bar[KEMPTY + g % NSK]);
            }
          }
          b0 += (c.nblk + pairs - 1) / pairs;
          ++n0;
          if (pairs == 2) {
            b1 += c.nblk / 2;
            ++n1;
          }
        }
        g0 += c.nblk;
      }
      commit(&bar[DRAIN]);
      wait_warp_drain(&bar[DRAIN], 0, status);
    }
  } else {
    // ---------------------------------------------------------- softmax --
    setmaxnreg_inc();
    const int t = warp >> 2;
    const int r = threadIdx.x & 127;  // row in the tile == TMEM lane
    const uint32_t lane_base =
        tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);
    const uint32_t s_col = lane_base + t * 128;
    const uint32_t o_col = lane_base + TM_O + t * 128;
    const float c2 = args.scale_log2;
    bool ok = true;
    // phases of this tile's scores, its units and its shared units
    uint32_t sph = 0, uph = 0, hph = 0;
    // token and head of this thread's row in a tile
    const int tok_r = static_cast<int>((r * args.pack_inv) >> 16);
    for (int nu = 0; ok; ++nu) {
      const int us = nu % kUnits;
      const Unit& c = s_unit[us];
      ok = wait_warp(&bar[UFULL + us], (nu / kUnits) & 1, abort_flag, status);
      if (!ok || c.stream < 0) break;
      // this warp has read the unit for the last time
      auto done_with_unit = [&]() {
        __syncwarp();
        if (lane == 0) mbar_arrive(&bar[UEMPTY + us]);
      };
      int nblk = c.nblk, lim_lo = 0, lim_hi = INT32_MAX;
      int key_step = BN;  // keys from one of this tile's blocks to the next
      {
        int tok = t * args.tile_tokens + tok_r;
        int kb0 = c.kb0;
        if (c.tokens <= args.tile_tokens) {
          if (nblk > 1) {  // shared: every other block, the same rows
            tok = tok_r;
            nblk = (nblk + 1 - t) >> 1;
            key_step = 2 * BN;
            kb0 += t;
          } else if (t > 0) {
            done_with_unit();
            continue;
          }
        }
        // rows of no token take part unmasked and are never written
        if (tok_r < args.tile_tokens && tok < c.tokens) {
          const int a = c.a0 + tok;
          lim_lo = pg::key_lo(max(a, 0), c.chunk, c.window) - kb0 * BN;
          lim_hi = pg::key_hi(a, c.chunk, c.kv) - kb0 * BN;
        }
      }
      float m_run = -INFINITY;
      float l_run = 0.f;
      for (int j = 0; j < nblk; ++j) {
        ok = wait_warp(&bar[SFULL + t], sph, abort_flag, status);
        if (!ok) break;
        sph ^= 1;
        tc_fence_after();
        float s[BN];
        tmem_ld128(s_col, s);
        tmem_ld_wait128(s);
        const bool masked =
            __any_sync(0xffffffffu, lim_hi < BN || lim_lo > 0);
        if (masked) {
#pragma unroll
          for (int c = 0; c < BN; ++c)
            if (c >= lim_hi || c < lim_lo) s[c] = -INFINITY;
        }
        lim_lo -= key_step;
        lim_hi -= key_step;
        const float mx = (masked ? rowmax_masked<BN>(s) : rowmax<BN>(s)) * c2;
        if (j == 0) {
          m_run = mx;
        } else {
          // S_t(j) complete implies P V_t(j - 1) complete, so O holds
          // exactly the earlier blocks
          const bool need = mx > m_run + RESCALE_LOG2;
          if (__any_sync(0xffffffffu, need)) {
            // (a row without keys so far keeps m = -inf and factor 1)
            const float alpha = need ? ex2(m_run - mx) : 1.f;
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              float o[32];
              tmem_ld32(o_col + c * 32, o);
              tmem_ld_wait32(o);
#pragma unroll
              for (int e = 0; e < 32; e += 2) {
                const float2 v =
                    ffma2(make_float2(o[e], o[e + 1]),
                          make_float2(alpha, alpha), make_float2(0.f, 0.f));
                o[e] = v.x;
                o[e + 1] = v.y;
              }
              tmem_st32(o_col + c * 32, o);
            }
            l_run *= alpha;
            if (need) m_run = mx;
          }
        }
        float2 acc[4] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f),
                         make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
        if (masked)
          exp_store_chunks<false>(s, c2, m_run == -INFINITY ? 0.f : m_run,
                                  s_col, acc, 0, 4);
        else
          exp_store_chunks<true>(s, c2, m_run, s_col, acc, 0, 4);
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bar[PREADY + t]);
        const float2 tsum = fadd2(fadd2(acc[0], acc[1]), fadd2(acc[2], acc[3]));
        l_run += tsum.x + tsum.y;
      }
      if (!ok) break;
      if (nblk > 0) {
        ok = wait_warp(&bar[OFINAL + t], uph, abort_flag, status);
        if (!ok) break;
        uph ^= 1;
        tc_fence_after();
      }
      const bool shared = c.tokens <= args.tile_tokens && c.nblk > 1;
      float f0 = 1.f, f1 = 0.f;  // factors of the halves of a shared unit
      if (shared) {
        if (t == 1) {
          s_half[r] = make_float2(m_run, l_run);
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&bar[HALF1]);
          done_with_unit();
          continue;  // tile 0's warps read O of both and free both
        }
        ok = wait_warp(&bar[HALF1], hph, abort_flag, status);
        if (!ok) break;
        hph ^= 1;
        tc_fence_after();
        const float2 other = s_half[r];
        const float mn = fmaxf(m_run, other.x);
        f0 = m_run == -INFINITY ? 0.f : ex2(m_run - mn);
        f1 = other.x == -INFINITY ? 0.f : ex2(other.x - mn);
        l_run = l_run * f0 + other.y * f1;
        m_run = mn;
      }
      // 32 columns of O, the halves joined
      auto load_o = [&](int col, float (&o)[32]) {
        tmem_ld32(o_col + col, o);
        if (!shared) {
          tmem_ld_wait32(o);
        } else {
          float o1[32];
          tmem_ld32(o_col + 128 + col, o1);
          tmem_ld_wait32(o);
          tmem_ld_wait32(o1);
#pragma unroll
          for (int e = 0; e < 32; ++e) o[e] = o[e] * f0 + o1[e] * f1;
        }
      };
      const int wrow0 = (warp & 3) * 32;  // this warp's rows of the tile
      // rows that are written: packed row of the tile's row, or -1
      const int tok0 = t * args.tile_tokens;
      const int most = min(min(c.tokens - tok0, args.tile_tokens),
                           args.c.token_cap - c.q0 - tok0);
      const int slot = c.slot, head = c.head, row_q = c.q0 + tok0;
      done_with_unit();
      auto row_at = [&](int row) -> int64_t {
        const int tok = static_cast<int>((row * args.pack_inv) >> 16);
        if (tok >= most) return -1;
        return static_cast<int64_t>(row_q + tok) * args.c.heads + head +
               (row - tok * args.pack);
      };
      uint8_t* stg = sQ + t * TILE;
      // A row's 16 pieces of 16 bytes go to its place in the Q buffer
      // (swizzled by row, as TMA leaves Q), then half-warps store whole
      // 256-byte rows.
      auto stage = [&](int piece, uint4 v) {
        *reinterpret_cast<uint4*>(stg + (piece >> 3) * HALF + r * 128 +
                                  (((piece & 7) ^ (r & 7)) << 4)) = v;
      };
      auto flush = [&](auto address) {
        __syncwarp();
        const int piece = lane & 15;
#pragma unroll 4
        for (int i = 0; i < 16; ++i) {
          const int row = wrow0 + 2 * i + (lane >> 4);
          const uint4 v = *reinterpret_cast<const uint4*>(
              stg + (piece >> 3) * HALF + row * 128 +
              (((piece & 7) ^ (row & 7)) << 4));
          const int64_t at = row_at(row);
          if (at >= 0) address(row, at)[piece] = v;
        }
        __syncwarp();
      };
      if (slot >= 0) {
        const int64_t prow =
            static_cast<int64_t>(slot) * pg::kTileRows + t * BM;
        if (row_at(r) >= 0) args.part_ml[prow + r] = make_float2(m_run, l_run);
        if (nblk > 0) {
#pragma unroll 1
          for (int hc = 0; hc < 2; ++hc) {
#pragma unroll
            for (int cc = 0; cc < 2; ++cc) {
              float o[32];
              load_o(hc * 64 + cc * 32, o);
#pragma unroll
              for (int e = 0; e < 8; ++e)
                stage(cc * 8 + e,
                      make_uint4(__float_as_uint(o[4 * e]),
                                 __float_as_uint(o[4 * e + 1]),
                                 __float_as_uint(o[4 * e + 2]),
                                 __float_as_uint(o[4 * e + 3])));
            }
            flush([&](int row, int64_t) {
              return reinterpret_cast<uint4*>(args.part_o + (prow + row) * HD +
                                              hc * 64);
            });
          }
        }
      } else if (nblk == 0) {
        // no row sees a key (the Q buffer is not this unit's: no staging)
        for (int i = lane >> 4; i < 32; i += 2) {
          const int64_t at = row_at(wrow0 + i);
          if (at >= 0)
            reinterpret_cast<uint4*>(args.o + at * HD)[lane & 15] =
                make_uint4(0, 0, 0, 0);
        }
      } else {
        const float inv = l_run > 0.f ? 1.0f / l_run : 0.f;
#pragma unroll
        for (int cc = 0; cc < 4; ++cc) {
          float o[32];
          load_o(cc * 32, o);
#pragma unroll
          for (int e = 0; e < 4; ++e)
            stage(cc * 4 + e,
                  make_uint4(
                      pack_bf16x2(o[8 * e] * inv, o[8 * e + 1] * inv),
                      pack_bf16x2(o[8 * e + 2] * inv, o[8 * e + 3] * inv),
                      pack_bf16x2(o[8 * e + 4] * inv, o[8 * e + 5] * inv),
                      pack_bf16x2(o[8 * e + 6] * inv, o[8 * e + 7] * inv)));
        }
        flush([&](int, int64_t at) {
          return reinterpret_cast<uint4*>(args.o + at * HD);
        });
      }
      if (nblk > 0) {
        // O is read and the staging rows too: the next unit's first P V and
        // Q load may overwrite them
        fence_proxy_async_smem();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(&bar[TFREE + t]);
          if (shared) mbar_arrive(&bar[TFREE + 1]);
        }
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 9) {
    tc_fence_after();
    tmem_dealloc(tmem, TMEM_COLS);
  }
}

// One warp per row of the line's units that several CTAs shared, from the
// plan's record of the unit.
__global__ void __launch_bounds__(128)
    paged_tile_join(const __grid_constant__ PagedArgs args) {
  const int32_t* work = args.c.work;
  if (__ldg(work + pg::H_KIND) != args.kind) return;
  const int n = __ldg(work + pg::H_TOTAL) -
                __ldg(work + pg::H_WAVES) * __ldg(work + pg::H_CTAS);
  const int4* recs = reinterpret_cast<const int4*>(work + pg::kJoin);
  const int lane = threadIdx.x & 31;
  const int warps = gridDim.x * 4;
  grid_dependency_wait();
  for (int it = blockIdx.x * 4 + (threadIdx.x >> 5);
       it < n * pg::kTileRows; it += warps) {
    const int i = it % pg::kTileRows;
    const int4 r0 = __ldg(recs + 2 * (it / pg::kTileRows));
    const int4 r1 = __ldg(recs + 2 * (it / pg::kTileRows) + 1);
    const int r = i & (BM - 1);
    const int in_tile = static_cast<int>((r * args.pack_inv) >> 16);
    const int tok = (i / BM) * args.tile_tokens + in_tile;
    const int row = r0.x + tok;
    if (in_tile >= args.tile_tokens || tok >= r0.y || row >= args.c.token_cap)
      continue;
    const int head = r0.z + r - in_tile * args.pack;
    const int32_t* cut = work + pg::kLine + r1.x - 1;
    JoinAcc<4> acc;
    acc.add_all(
        r1.y, lane, args,
        [&](int k) {
          const int slot = k ? 2 * (r1.x - 1 + k) : r0.w;
          return static_cast<int64_t>(slot) * pg::kTileRows + i;
        },
        // a CTA between the first and the last may have no share of the line
        [&](int k) { return __ldg(cut + k) < __ldg(cut + k + 1); });
    acc.write(args.o + (static_cast<int64_t>(row) * args.c.heads + head) * HD,
              lane);
  }
}
}  // namespace tile

int paged_log2(int v) {
  int s = 0;
  while ((1 << s) < v) ++s;
  return s;
}

int paged_sms() {
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) !=
          cudaSuccess)
    return 0;
  return n;
}

// Partial-result slots of the device and rows of one slot.
int64_t paged_slots(const wan_paged_t* c, int sms) {
  return pg::few_mode(c) ? 2ll * pg::kFewCtasPerSm * sms : 2ll * sms;
}
int paged_slot_rows(const wan_paged_t* c) {
  return pg::few_mode(c) ? pg::kFewRows : pg::kTileRows;
}

// Launches a joining kernel behind the kernel just launched on s: its CTAs
// may start while that one still runs and wait for its end in
// grid_dependency_wait.
int launch_join(void (*kern)(PagedArgs), int64_t blocks, const PagedArgs& a,
                cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(blocks));
  cfg.blockDim = dim3(128);
  cfg.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, a) == cudaSuccess ? WAN_OK
                                                          : WAN_ECUDA;
}

int launch_few(const void* k_pages, const void* v_pages, const PagedArgs& a,
               int sms, cudaStream_t s) {
  static std::mutex mu;
  static bool ready[64];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64)
    return WAN_ECUDA;
  {
    std::lock_guard<std::mutex> lock(mu);
    if (!ready[dev]) {
      if (cudaFuncSetAttribute(few::paged_few_kernel,
                               cudaFuncAttributeMaxDynamicSharedMemorySize,
                               few::kSmem) != cudaSuccess)
        return WAN_ECUDA;
      ready[dev] = true;
    }
  }
  few::paged_few_kernel<<<pg::kFewCtasPerSm * sms, few::kThreads, few::kSmem,
                          s>>>(static_cast<const __nv_bfloat16*>(k_pages),
                               static_cast<const __nv_bfloat16*>(v_pages), a);
  if (cudaGetLastError() != cudaSuccess) return WAN_ECUDA;
  const int64_t rows = static_cast<int64_t>(a.c.n_streams) * a.c.kv_heads *
                       a.c.max_new * a.group;
  int64_t blocks = (rows + 3) / 4;
  if (blocks > 8ll * sms) blocks = 8ll * sms;
  return launch_join(few::paged_few_join, blocks, a, s);
}

int launch_tile(const void* k_pages, const void* v_pages,
                const PagedArgs& a, int sms, cudaStream_t s) {
  static std::mutex mu;
  static int state[64];  // 0 unknown, 1 ready, 2 unusable
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64)
    return WAN_ECUDA;
  {
    std::lock_guard<std::mutex> lock(mu);
    if (state[dev] == 0) {
      // setmaxnreg draws on the registers the CTA was launched with
      cudaFuncAttributes fa;
      if (cudaFuncGetAttributes(&fa, tile::paged_tile_kernel) != cudaSuccess)
        return WAN_ECUDA;
      if (fa.numRegs * kThreads <
          8 * 32 * kSoftmaxRegs + 4 * 32 * kOtherRegs) {
        state[dev] = 2;
      } else if (cudaFuncSetAttribute(
                     tile::paged_tile_kernel,
                     cudaFuncAttributeMaxDynamicSharedMemorySize,
                     SMEM_DYN) != cudaSuccess) {
        return WAN_ECUDA;
      } else {
        state[dev] = 1;
      }
    }
    if (state[dev] != 1) return WAN_EUNSUPPORTED;
  }
  CUtensorMap mq, mk, mv;
  int st = make_map_rows(&mq, a.q, a.c.token_cap, a.c.heads, a.pack,
                         a.tile_tokens);
  if (st != WAN_OK) return st;
  const int box = 1 << a.box_shift;
  if ((st = make_map_pages(&mk, k_pages, a.c.n_pages, a.c.kv_heads,
                           a.c.page_size, box)) != WAN_OK ||
      (st = make_map_pages(&mv, v_pages, a.c.n_pages, a.c.kv_heads,
                           a.c.page_size, box)) != WAN_OK)
    return st;
  tile::paged_tile_kernel<<<sms, kThreads, SMEM_DYN, s>>>(mq, mk, mv, a);
  if (cudaGetLastError() != cudaSuccess) return WAN_ECUDA;
  return launch_join(tile::paged_tile_join, 8ll * sms, a, s);
}

}  // namespace
}  // namespace wan

extern "C" {

size_t wan_paged_workspace_bytes(const wan_paged_t* c) {
  using namespace wan;
  if (!c || c->kv_heads < 1 || c->heads < 1) return 0;
  const int sms = paged_sms();
  return static_cast<size_t>(paged_slots(c, sms)) * paged_slot_rows(c) *
         (HD * sizeof(float) + sizeof(float2));
}

int wan_paged_attn(const wan_paged_t* c, const void* q, const void* k_pages,
                   const void* v_pages, void* o, float softmax_scale,
                   void* workspace, size_t workspace_bytes, void* s) {
  using namespace wan;
  int st = paged::check_cache(c);
  if (st != WAN_OK) return st;
  if (!q || !k_pages || !v_pages || !o || !workspace) return WAN_EINVAL;
  if (!(softmax_scale > 0.f) || !isfinite(softmax_scale)) return WAN_EINVAL;
  if (o == q || o == k_pages || o == v_pages) return WAN_EINVAL;
  if (!aligned16(q) || !aligned16(k_pages) || !aligned16(v_pages) ||
      !aligned16(o) || !aligned16(workspace))
    return WAN_EALIGN;
  if ((st = check_device(nullptr)) != WAN_OK) return st;
  const int sms = paged_sms();
  if (sms < 1) return WAN_ECUDA;
  if (workspace_bytes < wan_paged_workspace_bytes(c)) return WAN_ENOSPACE;
  PagedArgs a;
  a.c = *c;
  a.q = static_cast<const __nv_bfloat16*>(q);
  a.o = static_cast<__nv_bfloat16*>(o);
  a.part_o = static_cast<float*>(workspace);
  a.part_ml = reinterpret_cast<float2*>(
      a.part_o + paged_slots(c, sms) * paged_slot_rows(c) * HD);
  a.scale_log2 = softmax_scale * 1.4426950408889634f;
  a.group = c->heads / c->kv_heads;
  a.page_shift = paged_log2(c->page_size);
  a.box_shift = paged_log2(c->page_size < 64 ? c->page_size : 64);
  a.pack = paged::tile_pack(c);
  a.tile_tokens = paged::tile_tokens(c);
  a.pack_inv = (65536u + a.pack - 1) / a.pack;
  a.kind = paged::work_kind(c);
  return paged::few_mode(c)
             ? launch_few(k_pages, v_pages, a, sms, as_stream(s))
             : launch_tile(k_pages, v_pages, a, sms, as_stream(s));
}

}  // extern "C"
