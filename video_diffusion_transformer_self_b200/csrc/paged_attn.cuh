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
};

// Page of position pos of a stream, as a tensor-map coordinate.
__device__ __forceinline__ int page_of(const PagedArgs& a, int stream,
                                       int64_t pos) {
  const int64_t p = pos >> a.page_shift;
  int page = -1;
  if (p < a.c.max_pages)
    page = a.c.block_table[static_cast<int64_t>(stream) * a.c.max_pages + p];
  return page >= 0 && page < a.c.n_pages ? page : a.c.n_pages;
}

// Last entry of the work list whose field f is <= x.
__device__ __forceinline__ const int32_t* find_entry(const int32_t* work,
                                                     int f, int64_t mul,
                                                     int64_t x) {
  int lo = 0, hi = __ldg(work + pg::H_ACTIVE) - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (__ldg(work + pg::kHdr + pg::kEnt * mid + f) * mul <= x)
      lo = mid;
    else
      hi = mid - 1;
  }
  return work + pg::kHdr + pg::kEnt * lo;
}

// Keys of a stream that its table can hold.
__device__ __forceinline__ int keys_of(const PagedArgs& a, int stream) {
  const int64_t most = static_cast<int64_t>(a.c.max_pages) << a.page_shift;
  const int kv = max(__ldg(a.c.kv_lens + stream), 0);
  return kv < most ? kv : static_cast<int>(most);
}

// ============================================================== few rows ==
//
// The cache's bytes bound this: per key and head 512 bytes are read for at
// most 16 rows, 32 operations a byte, so the legacy mma.sync (m16n8k16) is
// fast enough and keeps everything in registers.  The step's (stream, key
// head, 64-key stage) items form one line that is cut into equal parts, one
// per CTA, so every SM reads the same number of bytes whatever the streams'
// lengths.  Warp 4 fetches stages (K and V, 32 KB) through a 3-stage TMA
// ring, 192 KB in flight per SM with two CTAs; warps 0-3 take 16 keys of a
// stage each, with a softmax state of their own, and are joined when the
// CTA leaves an item.  An item that several CTAs share is written as
// partial results (at most two per CTA) and joined by paged_few_join.
namespace few {
constexpr int kThreads = 160;
constexpr int kStages = 3;
constexpr uint32_t kHalf = pg::kStage * 128;   // [64 keys][64 ch] bf16
constexpr uint32_t kStageBytes = 4 * kHalf;    // K halves, V halves
constexpr int kRows = pg::kFewRows;
constexpr uint32_t kJoinFloats = kRows * HD + 2 * kRows;
constexpr uint32_t kSmem =
    kStages * kStageBytes + 2 * kJoinFloats * 4 + 1024;

struct Segment {
  int stream, head, kv, ql, q0;  // q0: packed row of the stream's first row
  int stage0, n;                 // stages [stage0, stage0 + n) of 64 keys
  bool whole;                    // the item in full
  int chunk, window;
};

// The part of an item that starts at x, up to x1 on the line.
__device__ __forceinline__ Segment segment_at(const PagedArgs& a, int64_t x,
                                              int64_t x1) {
  Segment s;
  const int kvh = a.c.kv_heads;
  const int32_t* e = find_entry(a.c.work, pg::E_BASE, kvh, x);
  s.stream = __ldg(e + pg::E_STREAM);
  const int n = __ldg(e + pg::E_COUNT);
  const int64_t local = x - static_cast<int64_t>(__ldg(e + pg::E_BASE)) * kvh;
  s.head = static_cast<int>(local / n);
  const int at = static_cast<int>(local - static_cast<int64_t>(s.head) * n);
  s.n = static_cast<int>(n - at < x1 - x ? n - at : x1 - x);
  s.whole = s.n == n;
  s.kv = keys_of(a, s.stream);
  s.ql = __ldg(a.c.q_lens + s.stream);
  s.q0 = __ldg(a.c.q_start + s.stream);
  const int4 cfg = __ldg(reinterpret_cast<const int4*>(a.c.streams) + s.stream);
  s.chunk = cfg.z;
  s.window = cfg.w;
  const int lo = pg::key_lo(max(s.kv - s.ql, 0), s.chunk, s.window);
  s.stage0 = max(min(lo, s.kv - 1), 0) / pg::kStage + at;
  return s;
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

__global__ void __launch_bounds__(kThreads)
    paged_few_kernel(const __grid_constant__ CUtensorMap tm_k,
                     const __grid_constant__ CUtensorMap tm_v,
                     const __grid_constant__ PagedArgs args) {
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t full[kStages];
  __shared__ __align__(8) uint64_t empty[kStages];
  __shared__ int s_abort;
  const int32_t* work = args.c.work;
  const int ctas = __ldg(work + pg::H_CTAS);
  const int cta = blockIdx.x;
  if (__ldg(work + pg::H_MODE) != pg::kModeFew || cta >= ctas ||
      __ldg(work + pg::H_ACTIVE) < 1)
    return;
  const int64_t total = __ldg(work + pg::H_TOTAL);
  const int64_t x0 = cta * total / ctas, x1 = (cta + 1) * total / ctas;

  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t sm = (raw + 1023u) & ~1023u;
  float* join = reinterpret_cast<float*>(smem_raw + (sm - raw) +
                                         kStages * kStageBytes);
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  volatile int* abort_flag = &s_abort;
  int* status = &g_wan_status;
  if (threadIdx.x == 0) {
    s_abort = 0;
    for (int i = 0; i < kStages; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 4);
    }
    fence_mbar_init();
  }
  __syncthreads();

  if (warp == 4) {
    // ------------------------------------------------------- producer --
    if (lane == 0) {
      prefetch_tmap(&tm_k);
      prefetch_tmap(&tm_v);
    }
    const int boxes = pg::kStage >> args.box_shift;  // per stage: 1, 2 or 4
    const uint32_t box_bytes = 128u << args.box_shift;
    int g = 0;
    bool ok = true;
    for (int64_t x = x0; x < x1 && ok;) {
      const Segment s = segment_at(args, x, x1);
      x += s.n;
      const int row0 = lane << args.box_shift;  // this lane's box
      int page = 0;
      if (lane < boxes)
        page = page_of(args, s.stream,
                       static_cast<int64_t>(s.stage0) * pg::kStage + row0);
      for (int j = 0; j < s.n; ++j, ++g) {
        const int st = g % kStages, u = g / kStages;
        if (u > 0) ok = wait_warp(&empty[st], (u - 1) & 1, abort_flag, status);
        if (!ok) break;
        if (lane == 0) mbar_expect_tx(&full[st], kStageBytes);
        __syncwarp();
        const int64_t pos =
            static_cast<int64_t>(s.stage0 + j) * pg::kStage + row0;
        if (lane < boxes) {
          const int in_page =
              static_cast<int>(pos) & ((1 << args.page_shift) - 1);
          uint8_t* dst = smem_raw + (sm - raw) + st * kStageBytes +
                         lane * box_bytes;
          tma_load_4d(dst, &tm_k, &full[st], 0, in_page, s.head, page);
          tma_load_4d(dst + kHalf, &tm_k, &full[st], 64, in_page, s.head,
                      page);
          tma_load_4d(dst + 2 * kHalf, &tm_v, &full[st], 0, in_page, s.head,
                      page);
          tma_load_4d(dst + 3 * kHalf, &tm_v, &full[st], 64, in_page, s.head,
                      page);
          // the next stage's page arrives while this one is loaded
          if (j + 1 < s.n) page = page_of(args, s.stream, pos + pg::kStage);
        }
        __syncwarp();
      }
    }
    if (*abort_flag) {
      for (int i = (g > kStages ? g - kStages : 0); i < g; ++i)
        wait_warp_drain(&full[i % kStages], (i / kStages) & 1, status);
    }
    return;
  }

  // --------------------------------------------------------- consumers --
  // Fragments of m16n8k16: thread (gr, t4) = (lane / 4, lane % 4) holds rows
  // gr and gr + 8, columns 2 t4, 2 t4 + 1 (+ 8) of A and of the results.
  const int gr = lane >> 2, t4 = lane & 3;
  const float c2 = args.scale_log2;
  const int heads = args.c.heads;
  int g = 0;
  bool ok = true;
  for (int64_t x = x0; x < x1;) {
    const Segment s = segment_at(args, x, x1);
    const int rows = min(s.ql * args.group, kRows);
    // rows gr and gr + 8: row r is query head head * group + r % group of
    // new token r / group
    uint32_t qf[8][4];
    int lo[2], hi[2];
    int64_t orow[2];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int r = gr + 8 * e;
      const int i = r / args.group;
      orow[e] = (static_cast<int64_t>(s.q0) + i) * heads +
                s.head * args.group + (r - i * args.group);
      const bool on = r < rows && s.q0 + i < args.c.token_cap;
      if (!on) orow[e] = -1;
      const int a = s.kv - s.ql + i;
      // a row of padding takes part unmasked and is never written
      lo[e] = on ? pg::key_lo(max(a, 0), s.chunk, s.window) : 0;
      hi[e] = on ? pg::key_hi(a, s.chunk, s.kv) : INT32_MAX;
      const uint32_t* src = reinterpret_cast<const uint32_t*>(
          args.q + (on ? orow[e] : 0) * HD);
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        qf[k][e] = on ? __ldg(src + k * 8 + t4) : 0u;
        qf[k][2 + e] = on ? __ldg(src + k * 8 + 4 + t4) : 0u;
      }
    }
    const int item_lo = pg::key_lo(max(s.kv - s.ql, 0), s.chunk, s.window);
    float o[16][4];
#pragma unroll
    for (int d = 0; d < 16; ++d)
      o[d][0] = o[d][1] = o[d][2] = o[d][3] = 0.f;
    float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
    for (int j = 0; j < s.n; ++j, ++g) {
      const int st = g % kStages;
      if (ok) ok = wait_warp(&full[st], (g / kStages) & 1, abort_flag, status);
      if (!ok) continue;
      const uint32_t ks = sm + st * kStageBytes;
      const uint32_t vs = ks + 2 * kHalf;
      const int key0 = (s.stage0 + j) * pg::kStage + warp * 16;
      // S = Q K^T for this warp's 16 keys: two 8-key tiles
      float sc[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
      {
        const int row = warp * 16 + (lane & 7) + ((lane >> 4) << 3);
        const int sub = (lane >> 3) & 1;
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const int ch = 2 * k + sub;  // 16-byte chunk of the 256-byte row
          uint32_t b[4];
          ldsm4(ks + (ch >> 3) * kHalf + row * 128 +
                    (((ch & 7) ^ (row & 7)) << 4),
                b);
          mma16816(sc[0], qf[k], b[0], b[1]);
          mma16816(sc[1], qf[k], b[2], b[3]);
        }
      }
      const bool edge = __any_sync(
          0xffffffffu, lo[0] > key0 || lo[1] > key0 || hi[0] < key0 + 16 ||
                           hi[1] < key0 + 16);
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
      const bool vedge = key0 < item_lo || key0 + 16 > s.kv;
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
        const int row = warp * 16 + (lane & 15);
        const int sub = lane >> 4;
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const int ch = 2 * k + sub;
          uint32_t b[4];
          ldsm4t(vs + (ch >> 3) * kHalf + row * 128 +
                     (((ch & 7) ^ (row & 7)) << 4),
                 b);
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
      __syncwarp();
      if (lane == 0) mbar_arrive(&empty[st]);
    }
    // -------------------------------------------- join the four warps --
    // warps 2, 3 into 0, 1, then 1 into 0; every warp takes every barrier,
    // also after a wait gave up
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
          dst[kRows * HD + r] = m[e];
          dst[kRows * HD + kRows + r] = l[e];
        }
#pragma unroll
        for (int d = 0; d < 16; ++d)
          *reinterpret_cast<float2*>(dst + r * HD + d * 8 + 2 * t4) =
              make_float2(o[d][2 * e], o[d][2 * e + 1]);
      }
    };
    auto take = [&](const float* src) {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int r = gr + 8 * e;
        const float m2 = src[kRows * HD + r];
        const float mn = fmaxf(m[e], m2);
        const float w1 = m[e] == -INFINITY ? 0.f : ex2(m[e] - mn);
        const float w2 = m2 == -INFINITY ? 0.f : ex2(m2 - mn);
        l[e] = l[e] * w1 + src[kRows * HD + kRows + r] * w2;
        m[e] = mn;
#pragma unroll
        for (int d = 0; d < 16; ++d) {
          const float2 v = *reinterpret_cast<const float2*>(src + r * HD +
                                                            d * 8 + 2 * t4);
          o[d][2 * e] = fmaf(v.x, w2, o[d][2 * e] * w1);
          o[d][2 * e + 1] = fmaf(v.y, w2, o[d][2 * e + 1] * w1);
        }
      }
    };
    named_bar_sync(1, 128);
    if (warp >= 2) put(join + (warp - 2) * kJoinFloats);
    named_bar_sync(1, 128);
    if (warp < 2) take(join + warp * kJoinFloats);
    named_bar_sync(1, 128);
    if (warp == 1) put(join);
    named_bar_sync(1, 128);
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
  }
}

// Weighted sum of a row's partial results: lane l holds channels 4 l .. + 3.
struct JoinAcc {
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  float m = -INFINITY, l = 0.f;
  __device__ __forceinline__ void add(const float2 ml, const float* row,
                                      int lane) {
    if (!(ml.y > 0.f)) return;  // saw no key: its O is not read
    const float4 v = reinterpret_cast<const float4*>(row)[lane];
    const float mn = fmaxf(m, ml.x);
    const float w1 = m == -INFINITY ? 0.f : ex2(m - mn);
    const float w2 = ex2(ml.x - mn);
    acc.x = fmaf(v.x, w2, acc.x * w1);
    acc.y = fmaf(v.y, w2, acc.y * w1);
    acc.z = fmaf(v.z, w2, acc.z * w1);
    acc.w = fmaf(v.w, w2, acc.w * w1);
    l = fmaf(ml.y, w2, l * w1);
    m = mn;
  }
  __device__ __forceinline__ void write(__nv_bfloat16* dst, int lane) const {
    const float inv = l > 0.f ? 1.f / l : 0.f;
    reinterpret_cast<uint2*>(dst)[lane] =
        make_uint2(pack_bf16x2(acc.x * inv, acc.y * inv),
                   pack_bf16x2(acc.z * inv, acc.w * inv));
  }
};

// One warp per (stream, key head, row) whose item several CTAs shared.
__global__ void __launch_bounds__(128)
    paged_few_join(const __grid_constant__ PagedArgs args) {
  const int32_t* work = args.c.work;
  if (work[pg::H_MODE] != pg::kModeFew) return;
  const int64_t total = work[pg::H_TOTAL];
  const int64_t ctas = work[pg::H_CTAS];
  const int kvh = args.c.kv_heads;
  const int64_t items =
      static_cast<int64_t>(work[pg::H_ACTIVE]) * kvh * kRows;
  const int lane = threadIdx.x & 31;
  const int64_t warps = static_cast<int64_t>(gridDim.x) * 4;
  for (int64_t it = blockIdx.x * 4ll + (threadIdx.x >> 5); it < items;
       it += warps) {
    const int r = static_cast<int>(it % kRows);
    const int64_t ih = it / kRows;
    const int head = static_cast<int>(ih % kvh);
    const int32_t* e = work + pg::kHdr + pg::kEnt * (ih / kvh);
    const int64_t n = e[pg::E_COUNT];
    const int64_t xs = e[pg::E_BASE] * static_cast<int64_t>(kvh) + head * n;
    // CTA c holds [c total / ctas, (c + 1) total / ctas)
    const int64_t c0 = ((xs + 1) * ctas - 1) / total;
    const int64_t c1 = ((xs + n) * ctas - 1) / total;
    if (c0 == c1) continue;
    const int stream = e[pg::E_STREAM];
    const int i = r / args.group;
    const int q0 = args.c.q_start[stream];
    if (r >= args.c.q_lens[stream] * args.group || q0 + i >= args.c.token_cap)
      continue;
    JoinAcc acc;
    for (int64_t c = c0; c <= c1; ++c) {
      const int64_t start = c * total / ctas;
      const int64_t prow = (2 * c + (xs > start ? 1 : 0)) * kRows + r;
      acc.add(args.part_ml[prow], args.part_o + prow * HD, lane);
    }
    acc.write(args.o + ((static_cast<int64_t>(q0) + i) * args.c.heads +
                        head * args.group + (r - i * args.group)) * HD,
              lane);
  }
}
}  // namespace few

int paged_box_rows(const wan_paged_t* c) {
  return c->page_size < 64 ? c->page_size : 64;
}

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
  return pg::few_mode(c) ? 2ll * pg::kFewCtasPerSm * sms
                         : static_cast<int64_t>(pg::kTileSlotsPerSm) * sms;
}
int paged_slot_rows(const wan_paged_t* c) {
  return pg::few_mode(c) ? pg::kFewRows : pg::kTileRows;
}

int launch_few(const CUtensorMap& mk, const CUtensorMap& mv,
               const PagedArgs& a, int sms, cudaStream_t s) {
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
                          s>>>(mk, mv, a);
  if (cudaGetLastError() != cudaSuccess) return WAN_ECUDA;
  const int64_t rows =
      static_cast<int64_t>(a.c.n_streams) * a.c.kv_heads * pg::kFewRows;
  int64_t blocks = (rows + 3) / 4;
  if (blocks > 8ll * sms) blocks = 8ll * sms;
  few::paged_few_join<<<static_cast<unsigned>(blocks), 128, 0, s>>>(a);
  return cudaGetLastError() == cudaSuccess ? WAN_OK : WAN_ECUDA;
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
  const int box = paged_box_rows(c);
  CUtensorMap mk, mv;
  if ((st = make_map_pages(&mk, k_pages, c->n_pages, c->kv_heads,
                           c->page_size, box)) != WAN_OK)
    return st;
  if ((st = make_map_pages(&mv, v_pages, c->n_pages, c->kv_heads,
                           c->page_size, box)) != WAN_OK)
    return st;
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
  a.box_shift = paged_log2(box);
  if (!paged::few_mode(c)) return WAN_EUNSUPPORTED;
  return launch_few(mk, mv, a, sms, as_stream(s));
}

}  // extern "C"
