// mla_cache.cu — the paged latent cache's upkeep: appending tokens to it
// (bf16, FP8 or FP4 rows) and evicting tokens by the attention weight they
// have gathered.
#include <cmath>

#include "mla_internal.h"
#include "ptx.cuh"

namespace mla {
namespace {

__device__ __forceinline__ void set_status(WsHeader* ws, int code) { atomicCAS(&ws->status, 0, code); }

// ---------------------------------------------------------------- append
// One warp per new token; lane j holds columns 16j .. 16j + 15, which is one
// block of the FP4 row and an eighth of a block of the FP8 row.
//   FP4: s = e4m3(min(amax / 6, 448)), code = e2m1(|x| / s), both to nearest
//        even.  A quotient next to a rounding border of e2m1 (a multiple of
//        1/4) must not cross it: |x| / s is a border exactly, or at least
//        2^-10 away (x has 8 and s 4 significant bits), so the product with
//        the rounded reciprocal, rounded to multiples of 2^-11, is on the
//        same side, and on the border where the quotient is.
//   FP8: s = 2^k with the least k in [-15, 7] such that amax / s <= 448;
//        the division is exact, code = e4m3(clamp(x / s)).
// Bound by memory: 1152 bytes read, 416 (656, 1152) written a token, and
// 1024 more where the stored values are asked for.  A warp's loads do not
// wait for the lengths and the table, so a token costs one round trip
// (reading the lengths first and no padding measured the same).  8 prompts of
// up to 4096 tokens into FP4 rows: 12.5 us, 5.3 TB/s; a step of 16: 2.1 us.
constexpr int kAppendWarps = 4;  // (8: 3 % slower on prompts, 16: 11 %)

__device__ __forceinline__ uint32_t abs_max_bf16x2(uint32_t m, uint32_t w) {  // two running maxima of |bf16| as integers
  const uint32_t a = w & 0x7fff7fffu;
  return __vmaxu2(m, a);
}
__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }
// e4m3 code of a value in [0, 448], to nearest even
__device__ __forceinline__ uint32_t to_e4m3(float x) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(0.f), "f"(x));
  return r & 0xffu;
}
__device__ __forceinline__ uint32_t to_e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ float2 from_e4m3x2(uint32_t c) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)c));
  float lo, hi;
  asm("{ .reg .b16 l, h; mov.b32 {l, h}, %2; cvt.f32.f16 %0, l; cvt.f32.f16 %1, h; }" : "=f"(lo), "=f"(hi) : "r"(h));
  return make_float2(lo, hi);
}
// two e2m1 magnitudes (low nibble first)
__device__ __forceinline__ uint32_t to_e2m1x2(float lo, float hi) {
  uint32_t r;
  asm("{ .reg .b8 b; cvt.rn.satfinite.e2m1x2.f32 b, %1, %2; mov.b32 %0, {b, b, b, b}; }"
      : "=r"(r) : "f"(hi), "f"(lo));
  return r & 0xffu;
}
__device__ __forceinline__ float2 from_e2m1x2(uint32_t c) {
  uint32_t h;
  asm("{ .reg .b8 b0, b1, b2, b3; mov.b32 {b0, b1, b2, b3}, %1; cvt.rn.f16x2.e2m1x2 %0, b0; }" : "=r"(h) : "r"(c));
  float lo, hi;
  asm("{ .reg .b16 l, h; mov.b32 {l, h}, %2; cvt.f32.f16 %0, l; cvt.f32.f16 %1, h; }" : "=f"(lo), "=f"(hi) : "r"(h));
  return make_float2(lo, hi);
}

// pairs of fp32 in one 64-bit register, one instruction for both
__device__ __forceinline__ uint64_t pack_f32x2(float lo, float hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ void unpack_f32x2(uint64_t v, float& lo, float& hi) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}
__device__ __forceinline__ uint64_t mul_f32x2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t add_f32x2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint32_t add_bf16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("add.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

template <int kFormat>
__global__ void __launch_bounds__(32 * kAppendWarps)
    append_kernel(const uint4* __restrict__ c_kv, const uint32_t* __restrict__ k_rope,
                  const int32_t* __restrict__ block_table, const int32_t* __restrict__ seq_lens,
                  const int32_t* __restrict__ n_new, const int32_t* __restrict__ start_position,
                  uint8_t* __restrict__ cache, int32_t* __restrict__ position, uint4* __restrict__ c_cached,
                  WsHeader* ws, int tokens, int Lq, int max_pages, int num_pages) {
  const int lane = threadIdx.x & 31;
  const int tok = (int)blockIdx.x * kAppendWarps + (threadIdx.x >> 5);
  griddep_wait();
  griddep_launch_dependents();
  if (tok >= tokens) return;
  const int b = tok / Lq, l = tok - b * Lq;
  const uint4 v0 = c_kv[(size_t)tok * 64 + 2 * lane], v1 = c_kv[(size_t)tok * 64 + 2 * lane + 1];
  const uint32_t kr = k_rope[(size_t)tok * 32 + lane];
  const int n = seq_lens[b], m = n_new ? n_new[b] : Lq;
  if (m < 0 || m > Lq || n < m || n > max_pages * kPage) {
    if (lane == 0 && l == 0) set_status(ws, MLA_ERR_BAD_SEQLEN);
    return;
  }
  if (l >= m) return;  // padding
  const int at = n - m + l;
  const int page = block_table[(size_t)b * max_pages + at / kPage];
  if (page < 0 || page >= num_pages) {
    if (lane == 0) set_status(ws, MLA_ERR_BAD_TABLE);
    return;
  }
  constexpr int kRowBytes = kFormat == MLA_KV_BF16 ? kRow * 2 : (kFormat == MLA_KV_FP8 ? kRowBytesFp8 : kRowBytesFp4);
  uint8_t* row = cache + ((size_t)page * kPage + at % kPage) * kRowBytes;
  if (position && lane == 0) position[(size_t)b * max_pages * kPage + at] = start_position ? start_position[b] + l : at;
  uint32_t w[8] = {v0.x, v0.y, v0.z, v0.w, v1.x, v1.y, v1.z, v1.w};
  if constexpr (kFormat == MLA_KV_BF16) {
    reinterpret_cast<uint4*>(row)[2 * lane] = v0;
    reinterpret_cast<uint4*>(row)[2 * lane + 1] = v1;
    reinterpret_cast<uint32_t*>(row + 2 * kDc)[lane] = kr;
  } else {
    uint32_t mx = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) mx = abs_max_bf16x2(mx, w[i]);
    mx = max(mx & 0xffffu, mx >> 16);
    if constexpr (kFormat == MLA_KV_FP4) {
      const bool bad = mx >= 0x7f80u;  // an infinity or a NaN: the block reads back as NaN
      const uint32_t s8 = bad ? 0x7fu : to_e4m3(fminf(__fdiv_rn(__uint_as_float(mx << 16), 6.f), 448.f));
      const float s = from_e4m3x2(s8).x;
      const float inv = (bad || s8 == 0) ? 0.f : __frcp_rn(s);
      // signs where there are codes; that of a negative value that rounds to
      // zero is kept, that of a negative zero is not
      const uint32_t signs = inv != 0.f ? 0x88u : 0u;
      const uint64_t inv2 = pack_f32x2(inv, inv), s2 = pack_f32x2(s, s);
      const uint64_t grid = pack_f32x2(6144.f, 6144.f), off = pack_f32x2(-6144.f, -6144.f);
      uint32_t code[2] = {0u, 0u};
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const uint32_t x = add_bf16x2(w[i], 0u);  // -0 becomes +0
        uint64_t y = pack_f32x2(__uint_as_float((x << 16) & 0x7fffffffu), __uint_as_float(x & 0x7fff0000u));
        // |x| / s, rounded to multiples of 2^-11 by adding and taking off
        y = add_f32x2(add_f32x2(mul_f32x2(y, inv2), grid), off);
        float lo, hi;
        unpack_f32x2(y, lo, hi);
        uint32_t c = to_e2m1x2(lo, hi) | (((x >> 12) & 8u | (x >> 24) & 0x80u) & signs);
        if (bad) c = 0u;  // (an infinity times zero above)
        code[i >> 2] |= c << (8 * (i & 3));
        if (c_cached) {
          const float2 v = from_e2m1x2(c);
          float a, b;
          unpack_f32x2(mul_f32x2(pack_f32x2(v.x, v.y), s2), a, b);
          w[i] = pack_bf16x2(a, b);
        }
      }
      if (bad) set_status(ws, MLA_ERR_RANGE);
      reinterpret_cast<uint2*>(row)[lane] = make_uint2(code[0], code[1]);
      row[kFp4ScaleByte + lane] = (uint8_t)s8;
      reinterpret_cast<uint32_t*>(row + kFp4RopeByte)[lane] = kr;
    } else {
#pragma unroll
      for (int o = 1; o < 8; o <<= 1) mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, o));
      const bool bad = mx >= 0x7f80u;
      // amax = f * 2^e, 1 <= f < 2, against 448 = 1.75 * 2^8
      const int e = (int)(mx >> 7) - 127;
      int k = (mx & 0x7fu) <= 0x60u ? e - 8 : e - 7;
      k = bad ? 0 : (k < -15 ? -15 : (k > 7 ? 7 : k));
      const float s = __uint_as_float((uint32_t)(k + 127) << 23), inv = __uint_as_float((uint32_t)(127 - k) << 23);
      uint32_t code[4];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const uint32_t c = bad ? 0x7f7fu : to_e4m3x2(bf16_lo(w[i]) * inv, bf16_hi(w[i]) * inv);
        code[i >> 1] = (i & 1) ? (code[i >> 1] | c << 16) : c;
        if (c_cached) {
          const float2 y = from_e4m3x2(c);
          w[i] = pack_bf16x2(y.x * s, y.y * s);
        }
      }
      if (bad) set_status(ws, MLA_ERR_RANGE);
      reinterpret_cast<uint4*>(row)[lane] = make_uint4(code[0], code[1], code[2], code[3]);
      reinterpret_cast<uint32_t*>(row + kFp8RopeByte)[lane] = kr;
      if ((lane & 7) == 0) reinterpret_cast<float*>(row + kFp8ScaleByte)[lane >> 3] = s;
    }
  }
  if (c_cached) {  // what the row stands for
    c_cached[(size_t)tok * 64 + 2 * lane] = make_uint4(w[0], w[1], w[2], w[3]);
    c_cached[(size_t)tok * 64 + 2 * lane + 1] = make_uint4(w[4], w[5], w[6], w[7]);
  }
}

// ---------------------------------------------------------------- evict
// One cluster per sequence; CTA r owns a contiguous slice of its tokens, warp
// w a contiguous part of the slice, so that every rank below is a running
// count in token order.
//   1. keys (the weight's bits in an order that compares as integers, NaN
//      greatest) and positions to shared memory; newest position; one bit a
//      token: protected (newer than `recent`, or among the `first` positions).
//   2. the k-th greatest key of the candidates by digits of 11, 11 and 10
//      bits: histograms in shared memory, summed over the cluster.  The first
//      digit holds the exponent and two bits of the mantissa, which spreads
//      weights over the bins.  Candidates are the unprotected tokens, k =
//      budget - protected; should more be protected than fit (known with the
//      first histogram), those, k = budget.
//   3. equal keys are kept from the lowest place on.  Places: evicted tokens
//      below the budget; movers: kept tokens behind it; both in token order,
//      the i-th mover goes to the i-th place.  Four counts a warp, exchanged
//      once, give every warp where its ties, places and movers begin.
//   4. rows, weights and positions move (source and destination sets are
//      disjoint); vacated weights become zero; the length becomes the budget.
// Filling the places instead of closing up moves one row in a step that
// evicts one token, and at most min(budget, n - budget) rows ever.
// Bound by latency: seven steps across the cluster, each a barrier and a round
// trip; a warp moves 32 rows at a time, four in flight.  16 sequences
// of 2049 tokens, one leaves each: 8.7 us.  8 prompts of 30001 to 65536 tokens
// cut to 8192: 33 us, of which the moves take 9.5 (46 MB through the 64 SMs of
// eight clusters), the histograms 12, lists and ranks 6.
constexpr int kEvictThreads = 1024, kEvictWarps = kEvictThreads / 32;
constexpr int kBins = 2048, kMaxCtas = 8;
constexpr int kKeyCap = 20 * 1024;  // tokens of a slice held in shared memory at most; later ones are read again
struct EvictShared {
  uint32_t hist[4][kBins];               // one per pass; [3]: the first again, over the protected
  uint4 counts[kEvictWarps];             // per warp: ties and kept below the budget, ties and kept behind it
  uint32_t newest, protect;              // of this CTA's slice
  uint32_t sum[kEvictWarps];
  uint32_t bin, above;                   // chosen digit, candidates above it
  uint32_t ties[kEvictWarps], places[kEvictWarps], movers[kEvictWarps];  // before this CTA's warps
  uint32_t total;                        // movers of the sequence
};
constexpr int evict_smem(int cap) { return (int)sizeof(EvictShared) + cap * 8 + cap / 8; }

__device__ __forceinline__ uint32_t ld_cluster(uint32_t local, uint32_t rank) {
  uint32_t v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(mapa(local, rank)) : "memory");
  return v;
}
__device__ __forceinline__ uint2 ld_cluster_v2(uint32_t local, uint32_t rank) {
  uint2 v;
  asm volatile("ld.shared::cluster.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(mapa(local, rank)) : "memory");
  return v;
}
__device__ __forceinline__ uint4 ld_cluster_v4(uint32_t local, uint32_t rank) {
  uint4 v;
  asm volatile("ld.shared::cluster.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(mapa(local, rank)) : "memory");
  return v;
}
__device__ __forceinline__ uint32_t order_key(float w) {
  const uint32_t u = __float_as_uint(w + 0.f);  // -0 compares as 0
  if ((u & 0x7fffffffu) > 0x7f800000u) return 0xffffffffu;
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}
__device__ __forceinline__ uint32_t warp_incl(uint32_t v) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t x = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += x;
  }
  return v;
}

struct EvictArgs {
  uint8_t* cache;
  const int32_t* block_table;
  int32_t* seq_lens;
  float* weight;
  int32_t* position;
  int32_t* lists;  // [B][2][S / 2]: places, movers
  WsHeader* ws;
  int budget, recent, first, max_pages, num_pages, row_bytes;
  int key_cap;  // tokens of a slice held in shared memory (a multiple of 32)
};

// kOne: the cluster is a single CTA, which synchronises as a block.  A cluster
// barrier takes about 1,000 cycles, even of one CTA (16 sequences of 2049
// tokens, one leaves each: 10.8 -> 8.7 us).
template <bool kOne>
__global__ void __launch_bounds__(kEvictThreads) evict_kernel(const EvictArgs a) {
  constexpr int kMoveRows = 4;  // rows of a warp in flight at the end (6: the same, 8: spills, slower)
  extern __shared__ __align__(16) uint8_t esm[];
  EvictShared& sh = *reinterpret_cast<EvictShared*>(esm);
  uint32_t* keys = reinterpret_cast<uint32_t*>(esm + sizeof(EvictShared));
  int32_t* pos = reinterpret_cast<int32_t*>(keys + a.key_cap);
  uint32_t* bits = reinterpret_cast<uint32_t*>(pos + a.key_cap);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t rank = kOne ? 0u : cluster_ctarank(), ctas = kOne ? 1u : cluster_nctarank();
  const int b = (int)(blockIdx.x / ctas);
  const uint32_t full = 0xffffffffu;
  auto sync = [&]() {
    if constexpr (kOne) __syncthreads();
    else cluster_sync();
  };
  for (int i = tid; i < 4 * kBins; i += kEvictThreads) (&sh.hist[0][0])[i] = 0;
  griddep_wait();
  griddep_launch_dependents();
  const int S = a.max_pages * kPage;
  const int n = a.seq_lens[b];
  if (n < 0 || n > S) {
    if (tid == 0 && rank == 0) set_status(a.ws, MLA_ERR_BAD_SEQLEN);
    return;  // the whole cluster
  }
  if (n <= a.budget) return;
  float* weight = a.weight + (size_t)b * S;
  int32_t* position = a.position + (size_t)b * S;
  // slice of this CTA, part of this warp: multiples of 32 tokens
  const int per_cta = ((n + (int)ctas - 1) / (int)ctas + 31) & ~31;
  const int s0 = min((int)rank * per_cta, n), s1 = min(s0 + per_cta, n);
  const int per_warp = ((s1 - s0 + kEvictWarps - 1) / kEvictWarps + 31) & ~31;
  const int w0 = min(s0 + warp * per_warp, s1), w1 = min(w0 + per_warp, s1);
  const int held = s0 + a.key_cap;  // tokens from here on are read from global memory again

  // ---- 1. newest position (as an unsigned offset, so that any int compares)
  uint32_t newest = 0;
#pragma unroll 4
  for (int i = w0 + lane; i < w1; i += 32) {
    const int p = position[i];
    const float w = weight[i];
    newest = max(newest, (uint32_t)p ^ 0x80000000u);
    if (i < held) {
      keys[i - s0] = order_key(w);
      pos[i - s0] = p;
    }
  }
  newest = __reduce_max_sync(full, newest);
  if (lane == 0) sh.sum[warp] = newest;
  __syncthreads();
  if (warp == 0) {
    newest = __reduce_max_sync(full, sh.sum[lane]);
    if (lane == 0) sh.newest = newest;
  }
  sync();
  // lane r reads CTA r's value
  newest = __reduce_max_sync(full, lane < (int)ctas ? ld_cluster(smem_u32(&sh.newest), lane) : 0u);
  const long long recent_from = (long long)(int32_t)(newest ^ 0x80000000u) - a.recent;  // protected: position above it
  auto protects = [&](int p) { return p > recent_from || p < a.first; };
  uint32_t np = 0;
  for (int i = w0 + lane; i - lane < w1; i += 32) {
    const bool p = i < w1 && protects(i < held ? pos[i - s0] : position[i]);
    const uint32_t m = __ballot_sync(full, p);
    np += __popc(m);
    if (lane == 0 && i < held) bits[(i - s0) >> 5] = m;
  }
  if (lane == 0) sh.sum[warp] = np;
  __syncthreads();
  if (warp == 0) {
    np = __reduce_add_sync(full, sh.sum[lane]);
    if (lane == 0) sh.protect = np;
  }
  auto key_of = [&](int i) -> uint32_t { return i < held ? keys[i - s0] : order_key(weight[i]); };
  auto is_protected = [&](int i) -> bool {
    return i < held ? (bits[(i - s0) >> 5] >> ((i - s0) & 31)) & 1u : protects(position[i]);
  };

  // ---- 2. threshold key: `prefix` holds the digits found so far; among the
  // candidates that match it, the k-th greatest is sought
  bool among_protected = false;
  uint32_t prefix = 0, mask = 0, k = 0;
#pragma unroll 1
  for (int pass = 0; pass < 3; ++pass) {
    const int shift = pass == 0 ? 21 : (pass == 1 ? 10 : 0);
    const uint32_t digits = pass == 2 ? 1024u : 2048u;
    uint32_t* hist = sh.hist[pass];
    auto count = [&]() {
      for (int i = w0 + lane; i < w1; i += 32) {
        const uint32_t key = key_of(i);
        if ((key & mask) == prefix && is_protected(i) == among_protected)
          atomicAdd(&hist[(key >> shift) & (digits - 1)], 1u);
      }
      sync();
    };
    count();
    if (pass == 0) {
      np = __reduce_add_sync(full, lane < (int)ctas ? ld_cluster(smem_u32(&sh.protect), lane) : 0u);
      among_protected = np >= (uint32_t)a.budget;
      k = among_protected ? (uint32_t)a.budget : (uint32_t)a.budget - np;  // 1 <= k <= candidates
      if (among_protected) {
        hist = sh.hist[3];
        count();
      }
    }
    // bins of thread t, counted from the top digit down; all CTAs' in flight at once
    constexpr int kPer = kBins / kEvictThreads;
    static_assert(kPer == 2, "a thread reads a pair of bins");
    const uint32_t at = smem_u32(&hist[kBins - 2 - 2 * tid]);
    uint32_t c[kPer] = {0u, 0u};
    if constexpr (kOne) {
      const uint2 v = *reinterpret_cast<const uint2*>(&hist[kBins - 2 - 2 * tid]);
      c[0] = v.y;
      c[1] = v.x;
    } else {
#pragma unroll
      for (uint32_t r = 0; r < kMaxCtas; ++r) {
        const uint2 v = r < ctas ? ld_cluster_v2(at, r) : make_uint2(0u, 0u);
        c[0] += v.y;
        c[1] += v.x;
      }
    }
    const uint32_t tot = c[0] + c[1];
    const uint32_t incl = warp_incl(tot);
    if (lane == 31) sh.sum[warp] = incl;
    __syncthreads();
    uint32_t before = incl - tot + __reduce_add_sync(full, lane < warp ? sh.sum[lane] : 0u);
#pragma unroll
    for (int q = 0; q < kPer; ++q) {
      if (before < k && before + c[q] >= k) {  // exactly one bin of the block
        sh.bin = (uint32_t)(kBins - 1 - (kPer * tid + q));
        sh.above = before;
      }
      before += c[q];
    }
    __syncthreads();
    prefix |= sh.bin << shift;
    mask |= (digits - 1) << shift;
    k -= sh.above;
  }

  // ---- 3. a token's class: kept for certain, a tie (kept for the first k of
  // them in token order), or evicted
  auto classify = [&](int i, bool& tie) {  // lanes past w1: neither
    tie = false;
    if (i >= w1) return false;
    const uint32_t key = key_of(i);
    if (is_protected(i) != among_protected) return !among_protected;  // protected where the others compete
    tie = key == prefix;
    return key > prefix;
  };
  uint4 mine = make_uint4(0, 0, 0, 0);
  for (int i = w0 + lane; i - lane < w1; i += 32) {
    bool tie;
    const bool kept = classify(i, tie), low = i < a.budget;
    mine.x += __popc(__ballot_sync(full, tie && low));
    mine.y += __popc(__ballot_sync(full, kept && low));
    mine.z += __popc(__ballot_sync(full, tie && !low));
    mine.w += __popc(__ballot_sync(full, kept && !low));
  }
  if (lane == 0) sh.counts[warp] = mine;
  sync();
  {
    // thread t < 32 * ctas stands for warp t % 32 of CTA t / 32
    const uint32_t r = (uint32_t)warp;
    const bool on = r < ctas;
    const uint4 c = on ? ld_cluster_v4(smem_u32(&sh.counts[lane]), r) : make_uint4(0, 0, 0, 0);
    // that warp's tokens below the budget
    const int rs0 = min((int)r * per_cta, n), rs1 = min(rs0 + per_cta, n);
    const int rpw = ((rs1 - rs0 + kEvictWarps - 1) / kEvictWarps + 31) & ~31;
    const int rw0 = min(rs0 + lane * rpw, rs1), rw1 = min(rw0 + rpw, rs1);
    const int low = on ? max(0, min(rw1, a.budget) - min(rw0, a.budget)) : 0;
    const uint32_t t_incl = warp_incl(c.x + c.z);
    if (lane == 31) sh.sum[warp] = t_incl;
    __syncthreads();
    const uint32_t ties = t_incl - (c.x + c.z) + __reduce_add_sync(full, lane < warp ? sh.sum[lane] : 0u);
    const uint32_t left = ties < k ? k - ties : 0u;  // ties this warp may keep
    const uint32_t kl = min(left, c.x), kh = min(left - kl, c.z);
    const uint32_t places = (uint32_t)low - c.y - kl, movers = c.w + kh;
    const uint32_t p_incl = warp_incl(places), m_incl = warp_incl(movers);
    __syncthreads();
    if (lane == 31) sh.sum[warp] = p_incl;
    __syncthreads();
    const uint32_t p0 = p_incl - places + __reduce_add_sync(full, lane < warp ? sh.sum[lane] : 0u);
    __syncthreads();
    if (lane == 31) sh.sum[warp] = m_incl;
    __syncthreads();
    const uint32_t m0 = m_incl - movers + __reduce_add_sync(full, lane < warp ? sh.sum[lane] : 0u);
    if (r == rank) {
      sh.ties[lane] = ties;
      sh.places[lane] = p0;
      sh.movers[lane] = m0;
    }
    if (tid == kEvictThreads - 1) sh.total = m0 + movers;
    __syncthreads();
  }
  int32_t* place_list = a.lists + (size_t)b * S;
  int32_t* mover_list = place_list + S / 2;
  {
    uint32_t seen = sh.ties[warp], place0 = sh.places[warp], mover0 = sh.movers[warp];
    const uint32_t lt = (1u << lane) - 1u;
    for (int i = w0 + lane; i - lane < w1; i += 32) {
      bool tie;
      bool kept = classify(i, tie);
      const uint32_t m = __ballot_sync(full, tie);
      kept |= tie && seen + __popc(m & lt) < k;
      seen += __popc(m);
      const bool in = i < w1, pl = in && !kept && i < a.budget, mv = in && kept && i >= a.budget;
      const uint32_t mp = __ballot_sync(full, pl), mm = __ballot_sync(full, mv);
      if (pl) place_list[place0 + __popc(mp & lt)] = i;
      if (mv) mover_list[mover0 + __popc(mm & lt)] = i;
      place0 += __popc(mp);
      mover0 += __popc(mm);
      if (in && !kept && i >= a.budget) weight[i] = 0.f;  // its key is not read again
    }
  }
  sync();  // the lists, seen by every CTA of the cluster

  // ---- 4. the moves: a warp takes 32 pairs (fewer where there are not
  // enough for all warps), kMoveRows rows in flight
  const uint32_t total = sh.total;
  const int32_t* table = a.block_table + (size_t)b * a.max_pages;
  const int chunks = a.row_bytes / 16;
  const uint32_t nw = ctas * kEvictWarps, me = rank + ctas * (uint32_t)warp;
  const uint32_t batch = min(32u, (total + nw - 1) / nw);
  for (uint32_t j0 = me * batch; j0 < total; j0 += nw * batch) {
    const uint32_t cnt = min(batch, total - j0);
    long long src = 0, dst = -1;  // 16-byte chunks; -1: not moved
    if (lane < (int)cnt) {
      const int to = place_list[j0 + lane], from = mover_list[j0 + lane];
      const int pt = table[to / kPage], pf = table[from / kPage];
      const float w = weight[from];
      const int p = position[from];
      if (pt < 0 || pt >= a.num_pages || pf < 0 || pf >= a.num_pages) {
        // never dereferenced; the place keeps its row, and what is said of it
        set_status(a.ws, MLA_ERR_BAD_TABLE);
      } else {
        src = ((long long)pf * kPage + from % kPage) * chunks;
        dst = ((long long)pt * kPage + to % kPage) * chunks;
        weight[to] = w;
        position[to] = p;
      }
      weight[from] = 0.f;
    }
    uint4* rows = reinterpret_cast<uint4*>(a.cache);
    for (uint32_t q0 = 0; q0 < cnt; q0 += kMoveRows) {
      for (int c = lane; c - lane < chunks; c += 32) {
        uint4 v[kMoveRows];
#pragma unroll
        for (int q = 0; q < kMoveRows; ++q) {
          const long long s = __shfl_sync(full, src, (int)(q0 + q) & 31);
          if (q0 + q < cnt && c < chunks) v[q] = rows[s + c];
        }
#pragma unroll
        for (int q = 0; q < kMoveRows; ++q) {
          const long long d = __shfl_sync(full, dst, (int)(q0 + q) & 31);
          if (q0 + q < cnt && c < chunks && d >= 0) rows[d + c] = v[q];
        }
      }
    }
  }
  if (tid == 0 && rank == 0) a.seq_lens[b] = a.budget;
  sync();  // no CTA leaves while another may read its shared memory
}

}  // namespace

cudaError_t launch_append(int kv_format, const void* c_kv, const void* k_rope, const int32_t* block_table,
                          const int32_t* seq_lens, const int32_t* n_new, const int32_t* start_position, void* cache,
                          int32_t* position, void* c_cached, WsHeader* ws, int B, int Lq, int max_pages, int num_pages,
                          cudaStream_t st) {
  const int tokens = B * Lq;
  const dim3 grid((tokens + kAppendWarps - 1) / kAppendWarps), block(32 * kAppendWarps);
  auto go = [&](auto kernel) {
    return launch_chained(kernel, grid, block, 0, st, static_cast<const uint4*>(c_kv),
                          static_cast<const uint32_t*>(k_rope), block_table, seq_lens, n_new, start_position,
                          static_cast<uint8_t*>(cache), position, static_cast<uint4*>(c_cached), ws, tokens, Lq,
                          max_pages, num_pages);
  };
  if (kv_format == MLA_KV_FP4) return go(append_kernel<MLA_KV_FP4>);
  if (kv_format == MLA_KV_FP8) return go(append_kernel<MLA_KV_FP8>);
  return go(append_kernel<MLA_KV_BF16>);
}

cudaError_t launch_evict(void* cache, int row_bytes, const int32_t* block_table, int32_t* seq_lens, float* weight,
                         int32_t* position, int32_t* lists, WsHeader* ws, int B, int max_pages, int num_pages,
                         int budget, int recent, int first, cudaStream_t st) {
  EvictArgs a;
  a.cache = static_cast<uint8_t*>(cache);
  a.block_table = block_table;
  a.seq_lens = seq_lens;
  a.weight = weight;
  a.position = position;
  a.lists = lists;
  a.ws = ws;
  a.budget = budget;
  a.recent = recent;
  a.first = first;
  a.max_pages = max_pages;
  a.num_pages = num_pages;
  a.row_bytes = row_bytes;
  // one CTA for every 4096 tokens of capacity, up to the portable cluster size
  const int S = max_pages * kPage;
  const int ctas = S <= 4096 ? 1 : (S <= 8192 ? 2 : (S <= 16384 ? 4 : kMaxCtas));
  const int slice = ((S + ctas - 1) / ctas + 31) & ~31;
  a.key_cap = slice < kKeyCap ? slice : kKeyCap;
  const cudaError_t e = ctas == 1 ? raise_smem<evict_kernel<true>>(evict_smem(4096))
                                  : raise_smem<evict_kernel<false>>(evict_smem(kKeyCap));
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)B * ctas);
  cfg.blockDim = dim3(kEvictThreads);
  cfg.dynamicSmemBytes = evict_smem(a.key_cap);
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = ctas;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, ctas == 1 ? evict_kernel<true> : evict_kernel<false>, a);
}

}  // namespace mla
