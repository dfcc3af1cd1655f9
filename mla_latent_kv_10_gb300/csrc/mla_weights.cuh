// mla_weights.cuh — the attention weight that a step's queries pay to each
// cached token, added up over all query rows:
//     weight[b][s] += sum_{(l,h) sees s} exp(x_s - lse[b,l,h]),
//     x_s = (q . c_g(h)[s] + q_R . k_R[s]) * scale
// a second pass over the scores with the log-sum-exp already known, so no
// softmax state is carried: one tensor-core product per tile and a sum.
//
// GB300 design: as in the FP4 decode the cache rows are the 128-row operand
// (S^T[128 tokens, N query rows], N = 32, 64 or 128), so that a token is a tensor
// memory lane: one thread adds a token's N weights in registers and owns its
// place in `weight`.  No exchange, no atomics, the same bits every time.
//   * The tile streams through a ring of boxes (128 tokens x 64 columns,
//     16 KiB, 128-byte swizzled rows); nothing of it is kept, so the query
//     may take 144 KiB of shared memory (N = 128 at 512 latents).
//   * A CTA walks its share of all tiles once per latent group and block of
//     128 query rows (several passes add to the same token from the same
//     thread, in order).
//   * bf16 cache: boxes by TMA.  FP8, FP4: eight warps convert codes * scale
//     to f16 (exact, see the decodes); the RoPE keys come by TMA in bf16.
//   * warps 0-3 sum, 4-11 load (query, conversion), 12 issues MMAs, 13 copies.
// 16 sequences of 4096 tokens, 128 heads, FP4: 20.0 us (1.8 more with all eight
// converting warps on one box at a time).  Of 35,000 cycles 10,500 stage the
// query (147 KB a CTA, 22 MB over all of them, from L2), then each of four tiles
// takes 5,000, bound by the way of a box from its conversion over the products
// to a free place in a ring of three.  Over long bf16 sequences it reads at 0.53
// of the memory's rate (5 of 777 to 30011 tokens, 3 x 64 rows, 4 groups: 29.7 us).
#pragma once
#include <cmath>

#include "mla_internal.h"
#include "mla_plan.cuh"
#include "mla_tile.cuh"

namespace mla {
namespace {

constexpr int kWTok = 128;
constexpr int kSumWarps = 4, kLoadWarps = 8, kWMma = kSumWarps + kLoadWarps, kWCopy = kWMma + 1;
constexpr int kWThreads = 32 * (kWCopy + 1);
constexpr int kWBox = kWTok * 128;  // 128 tokens x 64 16-bit columns

template <int kFormat, int DG, int N>
struct WCfg {
  static constexpr int kNB = DG / 64;              // latent boxes per tile
  // the converting warps work on two boxes at a time: the ring then takes the
  // halves of the latent boxes in turn
  static constexpr bool kSplit = kFormat != MLA_KV_BF16 && kNB > 1;
  __device__ static int box(int k) { return kSplit ? (k & 1) * (kNB / 2) + (k >> 1) : k; }  // the k-th of a tile
  static constexpr int kQBox = N * 128;
  static constexpr int kQBytes = (kNB + 1) * kQBox;
  // shared memory: the query twice where it fits (the next pass's is staged
  // while this one runs), six ring boxes where they fit, else three
  static constexpr int kLimit = 232448 - 4096;
  static constexpr bool kBig = 2 * kQBytes + 4 * kWBox > kLimit;   // one query only
  static constexpr bool kFew = (kBig ? 1 : 2) * kQBytes + 8 * kWBox > kLimit;
  static constexpr int kQBuf = kBig ? 1 : 2;
  static constexpr int kNR = kFew ? 3 : 6;         // ring boxes
  static constexpr int kRope = kFew ? 1 : 2;       // RoPE buffers
  static constexpr int kRopeOff = kNR * kWBox;
  static constexpr int kQOff = kRopeOff + kRope * kWBox;
  static constexpr int kShOff = kQOff + kQBuf * kQBytes;
};

// Barriers (ring box x sits in slot x % kNR; tile t; pass p = one latent
// group and row block over one range of tiles):
//   full, empty[slot]       the box landed or was converted; its product is done
//   rope_full, rope_empty   the same for the tile's RoPE keys (slot t % kRope)
//   s_full, s_free[t & 1]   the scores are complete; they have been read
//   q_full, q_free[p % kQBuf]  the pass's query is in shared memory; its products are done
//   never                   testing: nothing completes it
struct WShared {
  uint64_t full[6], empty[6], rope_full[2], rope_empty[2], s_full[2], s_free[2], q_full[2], q_free[2], drain, never;
  alignas(16) float lse[128];  // log2 units, rounded; +inf where a row adds nothing
  alignas(16) float fix[128];  // 2^-(what the rounding left off)
  int lrow[128];
  int sum[2][16];
  UnitRec rec;
  SegIterT<kWTok> walk[kWCopy + 1];  // each warp's place
  uint32_t tmem;
  int abort;
};
template <int kFormat, int DG, int N>
constexpr int w_smem() { return WCfg<kFormat, DG, N>::kShOff + (int)((sizeof(WShared) + 15) & ~size_t(15)); }

// This CTA's share [start, end) of all tiles, and the sequence it starts in.
// All threads call it; any batch size.
__device__ __forceinline__ void share_of(const DecodeArgs& a, int (*scr)[16], UnitRec* rec) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, nw = kWThreads / 32;
  const int lo = a.Lq, hi = a.max_pages * kPage;
  if (a.B <= 32) {  // one warp, a sequence a lane: no barriers between the steps
    if (warp == 0) {
      const int n0 = lane < a.B ? a.seq_lens[lane] : 0, n = clamp_len(n0, lo, hi);
      const int np = lane < a.B ? (n + kWTok - 1) / kWTok : 0;
      if (blockIdx.x == 0 && lane < a.B && n != n0) set_status(a.ws, MLA_ERR_BAD_SEQLEN);
      int incl = np;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int x = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += x;
      }
      const int total = __shfl_sync(0xffffffffu, incl, 31), chunk = (total + (int)gridDim.x - 1) / (int)gridDim.x;
      const int start = min((int)blockIdx.x * chunk, total), end = min(start + chunk, total);
      if (lane == 0 && start >= end) *rec = UnitRec{a.B, 0, 0, 0, 0};
      if (start < end && incl - np <= start && start < incl) *rec = UnitRec{lane, incl - np, start, end, 0};
    }
    return;  // (the caller synchronises)
  }
  auto tiles = [&](int b) { return (clamp_len(a.seq_lens[b], lo, hi) + kWTok - 1) / kWTok; };
  int total = 0;
  for (int b = tid; b < a.B; b += kWThreads) {
    total += tiles(b);
    if (blockIdx.x == 0 && clamp_len(a.seq_lens[b], lo, hi) != a.seq_lens[b]) set_status(a.ws, MLA_ERR_BAD_SEQLEN);
  }
  total = __reduce_add_sync(0xffffffffu, total);
  if (lane == 0) scr[0][warp] = total;
  __syncthreads();
  total = __reduce_add_sync(0xffffffffu, lane < nw ? scr[0][lane] : 0);
  const int chunk = (total + (int)gridDim.x - 1) / (int)gridDim.x;
  const int start = min((int)blockIdx.x * chunk, total), end = min(start + chunk, total);
  if (tid == 0) *rec = UnitRec{a.B, 0, 0, 0, 0};
  __syncthreads();
  int off = 0;  // tiles before sequence `base`
  for (int base = 0; base < a.B && start < end; base += kWThreads) {
    const int b = base + tid, np = b < a.B ? tiles(b) : 0;
    int incl = np;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int x = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += x;
    }
    if (lane == 31) scr[1][warp] = incl;
    __syncthreads();
    int before = 0, all = 0;
    for (int w = 0; w < nw; ++w) {
      before += w < warp ? scr[1][w] : 0;
      all += scr[1][w];
    }
    const int o0 = off + before + incl - np;
    if (np > 0 && o0 <= start && start < o0 + np) *rec = UnitRec{b, o0, start, end, 0};
    off += all;
    __syncthreads();
  }
}

template <int kFormat, int DG, int N>
__global__ void __launch_bounds__(kWThreads, 1)
    weights_kernel(const __grid_constant__ CUtensorMap tm_lat, const __grid_constant__ CUtensorMap tm_rope,
                   const uint8_t* __restrict__ cache, const float* __restrict__ lse, float* __restrict__ weight,
                   const float scale_lo, const DecodeArgs a) {
  using C = WCfg<kFormat, DG, N>;
  constexpr int NB = C::kNB, NR = C::kNR;
  constexpr bool kConvert = kFormat != MLA_KV_BF16;
  extern __shared__ __align__(1024) uint8_t smem[];
  WShared& sh = *reinterpret_cast<WShared*>(smem + C::kShOff);
  const uint32_t ring = smem_u32(smem), qbase = ring + C::kQOff;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  WsHeader* ws = a.ws;
  if (ring & 1023u) {  // 128-byte swizzled tiles need it
    griddep_wait();
    if (threadIdx.x == 0) set_status(ws, MLA_ERR_UNSUPPORTED);
    return;
  }
  const uint64_t lim = a.wait_ns;
  auto bar = [](uint64_t& x) { return smem_u32(&x); };
  if (threadIdx.x == kWMma * 32) {
    sh.abort = 0;
    for (int s = 0; s < 6; ++s) {
      mbar_init(bar(sh.full[s]), !kConvert ? 1 : (C::kSplit ? kLoadWarps / 2 : kLoadWarps));
      mbar_init(bar(sh.empty[s]), 1);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(bar(sh.rope_full[s]), 1);
      mbar_init(bar(sh.rope_empty[s]), 1);
      mbar_init(bar(sh.s_full[s]), 1);
      mbar_init(bar(sh.s_free[s]), kSumWarps);
      mbar_init(bar(sh.q_full[s]), kLoadWarps);
      mbar_init(bar(sh.q_free[s]), 1);
    }
    mbar_init(bar(sh.drain), 1);
    mbar_init(bar(sh.never), 1);
    fence_mbar_init();
  }
  if (warp == kWMma) {
    tmem_alloc(smem_u32(&sh.tmem), 512);
    tmem_relinquish();
  }
  griddep_wait();
  share_of(a, sh.sum, &sh.rec);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  // Not before this block holds its tensor memory: a block of the next kernel
  // that got there first (while another stream's kernel kept this one waiting)
  // would wait for this kernel's end, and this kernel for its columns.
  griddep_launch_dependents();
  const uint32_t tmem = sh.tmem;
  volatile int* abort = &sh.abort;
  auto fail = [&]() {
    *abort = 1;
    set_status(ws, MLA_ERR_TIMEOUT);
  };
  const int hg = a.H / a.G, rows_g = a.Lq * hg;
  const int blocks = (rows_g + N - 1) / N, passes = a.G * blocks;
  // this warp's walk over the CTA's ranges; each range is walked `passes` times
  SegIterT<kWTok>& walk = sh.walk[warp];
  if (lane == 0) walk.init(sh.rec, a.seq_lens, true);
  __syncwarp();
  int sb = 0, ta = 0, tb = 0;
  auto next_range = [&]() {
    bool any = false;
    if (lane == 0) any = walk.next(a, sb, ta, tb);
    any = __shfl_sync(0xffffffffu, (int)any, 0) != 0;
    sb = __shfl_sync(0xffffffffu, sb, 0);
    ta = __shfl_sync(0xffffffffu, ta, 0);
    tb = __shfl_sync(0xffffffffu, tb, 0);
    return any;
  };
  bool ok = true;
  auto wait = [&](uint64_t& x, uint32_t parity) {
    return __all_sync(0xffffffffu, mbar_wait(bar(x), parity & 1, abort, lim)) != 0;
  };

  if (warp == kWMma) {
    // ------------------------------------------------------------ MMA issuer
    constexpr uint32_t id_l = kConvert ? idesc_f16(128, N, false, false) : idesc_bf16(128, N, false, false);
    constexpr uint32_t id_r = idesc_bf16(128, N, false, false);
    const uint32_t td = desc_lo(ring, 16), qd0 = desc_lo(qbase, 16), e = elect_one();
    const uint32_t stall = a.stall_page >= 0 ? (uint32_t)a.stall_page / (kWTok / kPage) : 0xffffffffu;
    uint32_t x = 0, t = 0, p = 0;
    while (ok && next_range())
      for (int pass = 0; ok && pass < passes; ++pass, ++p) {
        const uint32_t qs = p % C::kQBuf, qd = qd0 + ((qs * C::kQBytes) >> 4);
        if (!(ok = wait(sh.q_full[qs], p / C::kQBuf))) break;
        for (int i = ta; ok && i < tb; ++i, ++t) {
          if (t == stall && !(ok = wait(sh.never, 0))) break;
          if (t >= 2 && !(ok = wait(sh.s_free[t & 1], (t >> 1) - 1))) break;
          tc_fence_after();
          // two accumulators: the first half of the latent boxes, and the rest
          // with the RoPE keys.  The tensor core rounds each step's sum toward
          // zero, so the score's error grows with the length of the chain.
          const uint32_t d0 = tmem + 2 * N * (t & 1);
          constexpr int kHalf = (NB + 1) / 2;
#pragma unroll 1
          for (int k = 0; k < NB; ++k, ++x) {
            const int j = C::box(k);
            const uint32_t slot = x % NR, d = j < kHalf ? d0 : d0 + N;
            const uint32_t fresh = j == 0 || j == kHalf ? 0u : 1u;
            if (!(ok = wait(sh.full[slot], x / NR))) break;
            const uint32_t kd = td + ((slot * kWBox) >> 4), qb = qd + ((j * C::kQBox) >> 4);
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)
              mma_ss_if(e, d, kd + ((kk * 32) >> 4), qb + ((kk * 32) >> 4), id_l, kk > 0 ? 1u : fresh);
            mma_commit_if(e, bar(sh.empty[slot]));
          }
          if (!ok) break;
          const uint32_t rs = t % C::kRope;
          if (!(ok = wait(sh.rope_full[rs], t / C::kRope))) break;
          const uint32_t kd = td + ((C::kRopeOff + rs * kWBox) >> 4), qb = qd + ((NB * C::kQBox) >> 4);
#pragma unroll
          for (int kk = 0; kk < 4; ++kk) 
            mma_ss_if(e, d0 + N, kd + ((kk * 32) >> 4), qb + ((kk * 32) >> 4), id_r, (kk > 0 || NB > kHalf) ? 1u : 0u);
          mma_commit_if(e, bar(sh.rope_empty[rs]));
          mma_commit_if(e, bar(sh.s_full[t & 1]));
        }
        mma_commit_if(e, bar(sh.q_free[qs]));
      }
    if (!ok && lane == 0) fail();
    mma_commit_if(e, bar(sh.drain));
    if (!mbar_wait_quiet(bar(sh.drain), 0) && lane == 0) set_status(ws, MLA_ERR_TIMEOUT);
    __syncwarp();
  } else if (warp == kWCopy) {
    // ------------------------------------------------------------ copies
    // RoPE keys of every tile; over the bf16 cache the latent boxes too.  A
    // missing second page of a tile: the first one's rows, masked later.
    uint32_t x = 0, t = 0;
    auto page_of = [&](int i, int half, int n) {
      if (i * kWTok + half * kPage >= n) return -1;
      int pg = a.block_table[(size_t)sb * a.max_pages + 2 * i + half];
      if (pg < 0 || pg >= a.num_pages) {  // never dereferenced: clamped and reported
        if (lane == 0) set_status(ws, MLA_ERR_BAD_TABLE);
        pg = 0;
      }
      return pg;
    };
    while (ok && next_range()) {
      const int n = walk.len(a, sb);
      for (int pass = 0; ok && pass < passes; ++pass) {
        const int g = pass / blocks;
        for (int i = ta; ok && i < tb; ++i, ++t) {
          const int p0 = page_of(i, 0, n), p1 = page_of(i, 1, n);
          const int y0 = p0 * kPage, y1 = (p1 < 0 ? p0 : p1) * kPage;
          if (kConvert && pass == 0 && lane < 2) {  // the pages of a tile two on into L2 (contiguous)
            const int pf = i + 2 < tb ? page_of(i + 2, lane, n) : -1;
            if (pf >= 0)
              asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(
                               cache + (size_t)pf * kPage * (kFormat == MLA_KV_FP8 ? kRowBytesFp8 : kRowBytesFp4)),
                           "r"(kPage * (kFormat == MLA_KV_FP8 ? kRowBytesFp8 : kRowBytesFp4)) : "memory");
          }
          if (!kConvert) {
            for (int j = 0; j < NB; ++j, ++x) {
              const uint32_t slot = x % NR;
              if (x >= (uint32_t)NR && !(ok = wait(sh.empty[slot], x / NR - 1))) break;
              if (lane == 0) {
                mbar_arrive_expect_tx(bar(sh.full[slot]), kWBox);
                tma_load_2d(ring + slot * kWBox, &tm_lat, bar(sh.full[slot]), g * DG + 64 * j, y0);
                tma_load_2d(ring + slot * kWBox + kWBox / 2, &tm_lat, bar(sh.full[slot]), g * DG + 64 * j, y1);
              }
              __syncwarp();
            }
            if (!ok) break;
          }
          const uint32_t rs = t % C::kRope;
          if (t >= (uint32_t)C::kRope && !(ok = wait(sh.rope_empty[rs], t / C::kRope - 1))) break;
          constexpr int kRopeCol = kFormat == MLA_KV_BF16 ? kDc : (kFormat == MLA_KV_FP8 ? kFp8RopeByte : kFp4RopeByte) / 2;
          if (lane == 0) {
            const uint32_t dst = ring + C::kRopeOff + rs * kWBox;
            mbar_arrive_expect_tx(bar(sh.rope_full[rs]), kWBox);
            tma_load_2d(dst, &tm_rope, bar(sh.rope_full[rs]), kRopeCol, y0);
            tma_load_2d(dst + kWBox / 2, &tm_rope, bar(sh.rope_full[rs]), kRopeCol, y1);
          }
          __syncwarp();
        }
      }
    }
    if (!ok && lane == 0) fail();
    if (lane == 0) {  // what is in flight lands before the memory goes
      auto drain = [&](uint64_t& b, uint32_t parity) {
        if (!mbar_wait_quiet(bar(b), parity & 1)) set_status(ws, MLA_ERR_TIMEOUT);
      };
      for (uint32_t k = t > (uint32_t)C::kRope ? t - C::kRope : 0; k < t; ++k) drain(sh.rope_full[k % C::kRope], k / C::kRope);
      if (!kConvert)
        for (uint32_t k = x > (uint32_t)NR ? x - NR : 0; k < x; ++k) drain(sh.full[k % NR], k / NR);
    }
    __syncwarp();
  } else if (warp >= kSumWarps) {
    // ------------------------------------------------------------ loading warps
    const int w = warp - kSumWarps;
    constexpr int kRowB = kFormat == MLA_KV_FP8 ? kRowBytesFp8 : kRowBytesFp4;
    // Conversion: a lane owns half of one or two tokens' 64 codes in each of
    // its boxes.  Where there are several boxes, four warps take the first
    // half of them and four the second, so that two boxes are on their way.
    constexpr int kMine = C::kSplit ? NB / 2 : NB, kTk = C::kSplit ? 2 : 1;
    constexpr int kCodeW = kFormat == MLA_KV_FP8 ? 8 : 4;           // 32-bit words of 32 codes
    constexpr int kScW = kFormat == MLA_KV_FP8 ? (kMine + 1) / 2 : kMine;  // words of its boxes' scales
    const int grp = C::kSplit ? w >> 2 : 0, wi = C::kSplit ? w & 3 : w;
    const int hf = lane & 1, tk = 16 * kTk * wi + (lane >> 1);  // (the second token: 16 on)
    uint32_t code[kConvert ? kMine : 1][kTk][kCodeW], sc[kTk][kScW];
    bool bad = false;
    int entry = 0;  // the next tile's table entry, requested a tile ahead of use
    auto request = [&](int i) {
      entry = a.block_table[(size_t)sb * a.max_pages + min(2 * i + (kTk * wi >> 2), a.max_pages - 1)];
    };
    auto load_tile = [&](int i, int n, int g) {
      int pg = entry;
      if (pg < 0 || pg >= a.num_pages) pg = 0;  // (the copying warp reports it)
      if (i + 1 < tb) request(i + 1);
#pragma unroll
      for (int y = 0; y < kTk; ++y) {
#pragma unroll
        for (int j = 0; j < kMine; ++j)
#pragma unroll
          for (int q = 0; q < kCodeW; ++q) code[j][y][q] = 0u;
#pragma unroll
        for (int q = 0; q < kScW; ++q) sc[y][q] = 0u;
        if (i * kWTok + tk + 16 * y < n) {
          const uint8_t* p = cache + ((size_t)pg * kPage + ((tk + 16 * y) & (kPage - 1))) * kRowB;
          const int c0 = g * DG + 64 * kMine * grp;  // first column of its boxes
          if constexpr (kFormat == MLA_KV_FP8) {
            ldg<kScW>(p + kFp8ScaleByte + 4 * (c0 / 128), sc[y]);
#pragma unroll
            for (int j = 0; j < kMine; ++j) {
              uint32_t(&d)[kCodeW] = code[j][y];
              ldg<4>(p + c0 + 64 * j + 32 * hf, reinterpret_cast<uint32_t(&)[4]>(d[0]));
              ldg<4>(p + c0 + 64 * j + 32 * hf + 16, reinterpret_cast<uint32_t(&)[4]>(d[4]));
            }
          } else {
            ldg<kScW>(p + kFp4ScaleByte + c0 / 16, sc[y]);
#pragma unroll
            for (int j = 0; j < kMine; ++j) ldg<4>(p + (c0 + 64 * j + 32 * hf) / 2, reinterpret_cast<uint32_t(&)[4]>(code[j][y][0]));
          }
        }
      }
    };
    uint32_t x0 = 0, p = 0;  // boxes before this tile; passes
    auto convert = [&]() {
#pragma unroll
      for (int j = 0; j < kMine; ++j) {
        const uint32_t x = x0 + (C::kSplit ? 2 * j + grp : j), slot = x % NR;
        if (x >= (uint32_t)NR) ok = wait(sh.empty[slot], x / NR - 1);
        if (!ok) return;
#pragma unroll
        for (int y = 0; y < kTk; ++y) {
          const int row = tk + 16 * y;
          const uint32_t drow = ring + slot * kWBox + row * 128;
#pragma unroll
          for (int q = 0; q < 4; ++q) {  // eight codes, one 16-byte chunk
            uint32_t h[4], s;
            if constexpr (kFormat == MLA_KV_FP8) {
              const float f = __uint_as_float(sc[y][j / 2]);
              s = pack_f16x2(f, f);
              e4m3x4_to_f16x2x2(code[j][y][2 * q], h[0], h[1]);
              e4m3x4_to_f16x2x2(code[j][y][2 * q + 1], h[2], h[3]);
            } else {
              // the lane's two scales of the box: bytes 2 * hf, 2 * hf + 1 of word j
              const uint32_t s2 = e4m3x2_to_f16x2(hf ? sc[y][j] >> 16 : sc[y][j]);
              s = __byte_perm(s2, s2, q < 2 ? 0x1010 : 0x3232);
              e2m1x8_to_f16(code[j][y][q], h);
            }
            st_shared_v4(drow + (((4 * hf + q) ^ (row & 7)) << 4), mul_f16x2(h[0], s), mul_f16x2(h[1], s),
                         mul_f16x2(h[2], s), mul_f16x2(h[3], s));
          }
        }
        fence_proxy_async();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(sh.full[slot]));
      }
      x0 += NB;
#pragma unroll
      for (int y = 0; y < kTk; ++y)
#pragma unroll
        for (int q = 0; q < kScW; ++q) {
          if constexpr (kFormat == MLA_KV_FP8) {
            const float f = __uint_as_float(sc[y][q]);
            bad |= !(f == 0.f || (f >= 0x1p-15f && f <= 0x1p7f));
          } else {
            bad |= (((sc[y][q] & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u) != 0;  // a NaN scale
          }
        }
    };
    uint32_t top = 0;
    while (ok && next_range()) {
      const int n = walk.len(a, sb);
      for (int pass = 0; ok && pass < passes; ++pass, ++p) {
        const int g = pass / blocks, r0 = (pass % blocks) * N;
        // the first tile's codes are in flight while the query is staged (the
        // 64 registers of an FP8 row's would spill there)
        constexpr bool kEarly = kFormat == MLA_KV_FP4;
        if constexpr (kConvert) request(ta);
        if constexpr (kEarly) load_tile(ta, n, g);
        const uint32_t qs = p % C::kQBuf;
        if (p >= (uint32_t)C::kQBuf && !(ok = wait(sh.q_free[qs], p / C::kQBuf - 1))) break;
        // the query rows: latents (f16 where the cache is converted), RoPE
        top = __vmaxu2(top, stage_query<DG, 1, N, kLoadWarps, kConvert>(qbase + qs * C::kQBytes, w, [&](int row) {
          const int r = r0 + row, l = r / hg, h = g * hg + r - l * hg;
          return r < rows_g ? a.q_cat + (((size_t)sb * a.Lq + l) * a.H + h) * (DG + kDr) : nullptr;
        }));
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(sh.q_full[qs]));
        if constexpr (kConvert && !kEarly) load_tile(ta, n, g);
        if constexpr (kConvert) {
          for (int i = ta; ok && i < tb; ++i) {
            convert();
            if (ok && i + 1 < tb) load_tile(i + 1, n, g);
          }
        }
      }
    }
    if (!ok && lane == 0) fail();
    if (__any_sync(0xffffffffu, bad || (kConvert && beyond_f16(top))) && lane == 0) set_status(ws, MLA_ERR_RANGE);
  } else {
    // ------------------------------------------------------------ summing warps
    const int r = 32 * warp + lane;  // token in the tile = TMEM lane
    const uint32_t lane_base = tmem + ((uint32_t)(32 * warp) << 16);
    // score of a key that a row does not see: weighs nothing at every scale, as
    // both parts of the scale are above zero
    constexpr float hidden = -INFINITY;
    uint32_t t = 0;
    while (next_range()) {
      const int n = walk.len(a, sb);
      // `weight` outlives the call: nothing is added to a sequence whose length
      // was clamped, nor to tokens behind a table entry that was replaced
      const bool whole = a.seq_lens[sb] == n;
      for (int pass = 0; pass < passes; ++pass) {
        const int g = pass / blocks, r0 = (pass % blocks) * N;
        bar_sync(1, 32 * kSumWarps);  // the pass before has read its rows
        if (threadIdx.x < N) {
          const int q = r0 + threadIdx.x;
          // lse in log2 units as hi + lo (the product's rounding, and what
          // log2 e has beyond 32 bits): each row's rounding would scale all
          // of its weights one way
          constexpr float kLog2e = 1.44269502162933349609f, kLog2eLo = 1.92596299112661e-8f;
          float v = INFINITY, lo = 0.f;
          int l = 0;
          if (q < rows_g) {
            l = q / hg;
            const float x = lse[((size_t)sb * a.Lq + l) * a.H + g * hg + q - l * hg];
            if (x != -INFINITY) {
              v = x * kLog2e;
              lo = fmaf(x, kLog2eLo, fmaf(x, kLog2e, -v));
            }
          }
          sh.lse[threadIdx.x] = v;
          sh.fix[threadIdx.x] = ex2(-lo);
          sh.lrow[threadIdx.x] = a.causal ? l : a.Lq - 1;
        }
        bar_sync(1, 32 * kSumWarps);
        for (int i = ta; i < tb; ++i, ++t) {
          const int at = i * kWTok + r;  // requested ahead of the wait
          const int page = whole && at < n ? a.block_table[(size_t)sb * a.max_pages + at / kPage] : -1;
          if (ok) ok = wait(sh.s_full[t & 1], t >> 1);
          if (!ok) continue;  // (the barriers above still see every warp)
          tc_fence_after();
          const int past0 = i * kWTok - (n - a.Lq), past = past0 + r;  // visible to rows with l >= past
          float sum = 0.f;
#pragma unroll 1
          for (int c = 0; c < N; c += 32) {
            uint32_t v[32], u[32];
            tmem_ld32(lane_base + 2 * N * (t & 1) + c, v);
            tmem_ld32(lane_base + 2 * N * (t & 1) + N + c, u);
            tmem_wait_ld();
#pragma unroll
            for (int j = 0; j < 32; ++j) v[j] = __float_as_uint(__uint_as_float(v[j]) + __uint_as_float(u[j]));
            float s4[4] = {0.f, 0.f, 0.f, 0.f};
            if (past0 + kWTok > 1) {
#pragma unroll
              for (int j = 0; j < 32; ++j)
                if (sh.lrow[c + j] < past) v[j] = __float_as_uint(hidden);
            }
#pragma unroll
            for (int j = 0; j < 32; j += 4) {
              const float4 m = *reinterpret_cast<const float4*>(&sh.lse[c + j]);
              const float4 f = *reinterpret_cast<const float4*>(&sh.fix[c + j]);
              // the small part last: added to the reference it would be
              // rounded away (an exponent of hundreds has a half unit of 2^-16)
              auto weigh = [&](uint32_t x, float ref) {
                const float y = __uint_as_float(x);
                return ex2(fmaf(y, scale_lo, fmaf(y, a.scale_log2, -ref)));
              };
              s4[0] = fmaf(weigh(v[j], m.x), f.x, s4[0]);
              s4[1] = fmaf(weigh(v[j + 1], m.y), f.y, s4[1]);
              s4[2] = fmaf(weigh(v[j + 2], m.z), f.z, s4[2]);
              s4[3] = fmaf(weigh(v[j + 3], m.w), f.w, s4[3]);
            }
            sum += (s4[0] + s4[1]) + (s4[2] + s4[3]);
          }
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(sh.s_free[t & 1]));
          if (page >= 0 && page < a.num_pages) weight[(size_t)sb * a.max_pages * kPage + at] += sum;
        }
      }
    }
    if (!ok && lane == 0) fail();
  }

  tc_fence_before();
  __syncthreads();
  if (warp == kWMma) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

template <int kFormat, int DG, int N>
cudaError_t launch_weights_one(const CUtensorMap& tl, const CUtensorMap& tr, const void* cache, const float* lse,
                               float* weight, const DecodeArgs& a, float scale_lo, cudaStream_t st) {
  static_assert(w_smem<kFormat, DG, N>() <= 232448, "weights kernel exceeds 227 KiB of shared memory");
  const cudaError_t e = raise_smem<weights_kernel<kFormat, DG, N>>(w_smem<kFormat, DG, N>());
  if (e != cudaSuccess) return e;
  return launch_chained(weights_kernel<kFormat, DG, N>, dim3(a.units), dim3(kWThreads), w_smem<kFormat, DG, N>(), st, tl, tr,
                        static_cast<const uint8_t*>(cache), lse, weight, scale_lo, a);
}
template <int kFormat, int DG>
cudaError_t launch_weights_dg(const CUtensorMap& tl, const CUtensorMap& tr, const void* cache, const float* lse,
                              float* weight, const DecodeArgs& a, float scale_lo, cudaStream_t st) {
  // a product costs 45 cycles up to 32 columns, 48 at 64 and 64 at 128, and a
  // smaller query leaves room for a second one and a longer ring
  const int rows = a.Lq * a.H / a.G;
  if (rows <= 32) return launch_weights_one<kFormat, DG, 32>(tl, tr, cache, lse, weight, a, scale_lo, st);
  if (rows <= 64) return launch_weights_one<kFormat, DG, 64>(tl, tr, cache, lse, weight, a, scale_lo, st);
  return launch_weights_one<kFormat, DG, 128>(tl, tr, cache, lse, weight, a, scale_lo, st);
}
template <int kFormat>
cudaError_t launch_weights_fmt(const CUtensorMap& tl, const CUtensorMap& tr, const void* cache, const float* lse,
                               float* weight, const DecodeArgs& a, float scale_lo, cudaStream_t st) {
  switch (a.d_g) {
    case 512: return launch_weights_dg<kFormat, 512>(tl, tr, cache, lse, weight, a, scale_lo, st);
    case 256: return launch_weights_dg<kFormat, 256>(tl, tr, cache, lse, weight, a, scale_lo, st);
    case 128: return launch_weights_dg<kFormat, 128>(tl, tr, cache, lse, weight, a, scale_lo, st);
    default: return launch_weights_dg<kFormat, 64>(tl, tr, cache, lse, weight, a, scale_lo, st);
  }
}

}  // namespace
}  // namespace mla
