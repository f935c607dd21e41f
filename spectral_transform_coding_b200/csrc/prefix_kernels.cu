// Attention of a batch over a prefix that all its sequences share, over the packed
// latent cache (spectra_decode_attend_shared).
//
// For the rows r = (sequence, q head) of KV head a, with the latents c of the shared
// pages:  s_rt = q_lat,r . c_K,t (log2 units),  m_r >= max_t s_rt - 7.9,
// l_r = sum_t 2^(s_rt - m_r),  o_r = sum_t 2^(s_rt - m_r) c_V,t.  Each CTA leaves
// (m, l, o) of its part of the prefix in the records that the decode kernel merges
// with those of the sequences' own pages.
//
// Every code is unpacked once for up to 128 rows, so the work is that of two matrix
// products and one exponential per (token, row):
//   S^T [128 tokens x rows] = C_K [tokens x coordinates] Q^T (twice, for Q's two parts),
//   O^T [coordinates x rows] += C_V^T [coordinates x tokens] P.
// Both run on tcgen05 with fp32 accumulators in TMEM.  Tokens are S^T's TMEM lanes, so
// the number of rows (the MMA's N) can be small without idle lanes; a thread holds one
// token's scores against a half or a quarter of the rows.
//
// Tiles of 128 tokens (8 blocks of 16, one or two warps each).  Per tile:
//   1. unpack: a lane's 8 codes of a (block, group) come as fp16 integers by one
//      and/or (code | 0x6400 = 1024 + code, or code << 4 | 0x5400 = 64 + code), one
//      subtraction and one product with the token's scale.  Values: c = rn(code s + z),
//      one fma, rounded once.  Keys exactly, as decode_attend's: c = (code - 1) s + s + z,
//      where (code - 1) s is an fp16 number for widths 1 and 2 (-s .. 2 s) and the sum of two
//      for the others (the second ones are further coordinates of the row), and s and z of
//      each group are two more coordinates, against the sum of the group's q_lat.
//      The packed layout is that of MMA fragments, so four lanes hold 8
//      adjacent coordinates of a token (K) or 8 adjacent tokens of a coordinate (V) and
//      a warp's store fills whole 128-byte core matrices without bank conflicts.  K
//      rows are ordered so that even tokens 2i and odd tokens 2i + 1 of a block's
//      half take rows i and i ^ 4 of its core matrix;
//   2. scores from TMEM; p = 2^(s - m + 8) as fp16, P in shared memory with the
//      rows contiguous (each thread writes its token's line in 16-byte pieces).
// m is not the running maximum but a maximum taken when a score last exceeded it by
// more than 7.9 (p < 2^16 fits fp16); the check costs one max per score and one vote
// that the tile's barrier carries, and the exact maxima and the rescaling of O run
// only then (always in the first tile).  l is summed in fp32 registers per thread (as a
// third product, of P with ones, it doubles the MMAs of the tile's second half: 16
// sequences x 32k at 12x took 49 us instead of 40 when that was tried, 64 x 28k at 4x no less).
// 8 or 16 warps do this; one more issues the MMAs and the page copies, so that neither
// their issue time (about 50 cycles an MMA) nor the page ids' latency stands in the
// others' way.  S of tile t + 1 is computed while tile t's scores turn into P, O of
// tile t while the keys of tile t + 2 are unpacked.
//
// Bound: the issue of the unpacking and softmax instructions and the waits between the
// phases of a tile, not HBM (3 to 9 % busy) and not the tensor cores (7 to 21 %).  This
// kernel alone, cold: 4 sequences of 7 heads x 4 KV heads behind 128k tokens at 8x take
// 52 us (issue slots 50 % busy), 8 x 32k at 4x 48 us, 16 x 32k at 12x 47 us, 64 x 28k at
// 4x 114 us.
//
// Rounding: q_lat as two fp16 parts (2^-22), which multiply the exact keys, so that a score is
// off by 2^-22 of its |q_lat c| and by the fold's two bf16 parts of W_up (2^-16).  (With one
// part of q_lat and c = rn(code s + z) scores were off by 2^-11 of |q_lat| |c|: for keys far from
// zero more than a code step, shared and own tokens' scores apart by it, outputs by up to six
// times 2e-3; that took 3 to 12 us less a call.)  p is rounded to 2^-11 of itself, c_V to 2^-11 of
// |c_V|: both average out over the tokens, and p's is also the decode kernel's.
//
// Every wait on an mbarrier is bounded; on a timeout the compute warps record
// SPECTRA_ERR_TIMEOUT, agree in a vote, tell the MMA warp and leave; it waits for the
// copies and MMAs in flight, and the CTA frees its TMEM and returns.  (Named barriers
// join warps of the CTA that all reach them.)
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdlib>

#include "attend_kernel.cuh"
#include "tcgen05_device.cuh"

namespace spectra {

namespace {

using attend::kMaxG;
using attend::LaneAddr;

constexpr int kPfTok = 128;       // tokens of a tile
constexpr int kPfMaxStages = 32;
// p = 2^(s - m + 8), as the decode kernel's: all 11 bits down to 2^-22 of a split's largest weight,
// nothing lost above 2^-32.  (From 2^-3 instead of 2^8 the first tile's m served longer, and 16
// sequences x 32k at 12x took 3 us less, but weights below 2^-22 of the largest vanished from O and
// stayed in l: behind a first token with 0.99 of the weight and no value the output was several percent off.)
constexpr float kPfOff = attend::kPScaleLog2;
constexpr float kPfLimit = 15.9f;   // exponent of p above which m is taken again (fp16 ends at 2^15.999)

// shared memory (bytes): barriers, tables, then V | K | Q | P | page ring
constexpr int kPfBars = 0;       // uint64 [kPfMaxStages + 4]: pages, S, O, drain, fold
constexpr int kPfMisc = 320;     // int: TMEM address, stop flag, pages of this CTA, K steps and positions with low parts
constexpr int kPfOrd = 384;      // int4 [2][kMaxG] groups in width-class order {block off, record off, group, width}
constexpr int kPfOffs = 640;      // float [4][128] kPfOff - m of each row (added to a score), a copy per token quarter
constexpr int kPfWMax = 2688;     // float [4][128] by token quarter: the first tile's maxima, after the last the sums
constexpr int kPfFac = kPfWMax;   // (between) float [4][128] a warp's own: the factors of a rescaling
constexpr int kPfOver = 4736;     // int [2][128] maxima above the limit, ordered as integers
constexpr int kPfLane = 5760;     // uint4 [2][kMaxG][32] lane tables of the groups (width 8: not read)
constexpr int kPfPos = kPfLane + 2 * kMaxG * 512;  // K groups: int [8] record offsets by position, int [8] bytes to the
                                                   // low parts' chunks in class order, int [8] the steps of 16
                                                   // coordinates with low parts
constexpr int kPfV = kPfPos + 128;  // operands (128-byte aligned)
static_assert(kPfV % 128 == 0, "core matrices are 128-byte blocks");

// named barriers (0 is __syncthreads): the compute warps' vote; keys unpacked; P and
// values written (compute warps arrive, the MMA warp waits); prologues done
constexpr int kBarVote = 1, kBarKeys = 2, kBarValues = 3, kBarReady = 4;

struct PrefixArgs {
  const CodecDev* cd;
  int32_t* err;  // the codec's error word
  const uint8_t* pool;
  const int32_t* pages;
  const uint16_t* q;
  float* rec;
  int64_t n_pool_pages, page_bytes;
  long long wait_cycles;  // limit of a wait
  int pages_lo, pages_rem;  // splits take pages_lo pages each, the first pages_rem one more
  int rec_stride, rec_first, n_merge, rows;
  int fold_dims;  // dims folded at a time: 128, or 64 where shared memory is short
  int pages_per, tiles_per, stages, stage_bytes, off_k, off_q, off_p, off_ring;
  int n_q, n_kv, d_h, P, gq;
  int drop_page;  // test hook: page of CTA (0, 0, 0) whose copy is never issued; -1: none
  float q_scale;
  alignas(16) int32_t hm[kMaxKV][12];  // as AttendArgs::hm, then the chunks of a K row
};

// 16-byte chunks of 8 coordinates of a K row, whole MMA steps of 16:
//   [kept coordinates, at least a step] [z of 8 groups | s of 8 groups] [low parts of wide groups]
// and of a Q row: [q_lat's high parts | its groups' sums twice] [low parts of both].
__host__ __device__ inline int main_chunks(int kept) { return kept > 0 ? (kept + 15) / 16 * 2 : 2; }
__host__ __device__ inline int q_chunks(int kept) { return 2 * (main_chunks(kept) + 2); }
// Widths whose (code - 1) s has more bits than fp16 (width 2: -s .. 2 s).
__host__ __device__ inline bool wide_code(int b) { return b >= 3; }

__device__ __forceinline__ void st_s32(uint32_t a, uint32_t v) {
  asm volatile("st.shared.b32 [%0], %1;" ::"r"(a), "r"(v) : "memory");
}
__device__ __forceinline__ void st_s128(uint32_t a, uint32_t x, uint32_t y, uint32_t z, uint32_t w) {
  asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(a), "r"(x), "r"(y), "r"(z), "r"(w) : "memory");
}

// The lane's 8-bit codes (K side: less 1) of one block (half `odd` of a 32-token block for G = 8) as
// four registers of two fp16 integers each, fragment order (registers 1 and 3: rows + 8).
template <int G>
__device__ __forceinline__ void load_bytes(uint32_t blk, int side, int odd, __half2 (&c)[4]) {
  uint32_t r[4];
  const uint2 w = attend::ld_s64<0>(blk);
  if (G == 16) {
    r[0] = w.x;
    r[1] = w.x >> 8;
    r[2] = w.y;
    r[3] = w.y >> 8;
  } else if (side == 0) {
    r[0] = odd ? w.y : w.x;
    r[1] = r[0] >> 8;
    r[2] = r[3] = 0u;
  } else {
    r[0] = odd ? (w.x >> 8) : w.x;
    r[2] = odd ? (w.y >> 8) : w.y;
    r[1] = r[3] = 0u;
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    r[i] = (r[i] & 0x00FF00FFu) | 0x64006400u;
    c[i] = __hsub2(*reinterpret_cast<__half2*>(&r[i]), __float2half2_rn(side == 0 ? 1025.f : 1024.f));
  }
}

__device__ __forceinline__ __half2 as_half2(uint32_t x) { return *reinterpret_cast<__half2*>(&x); }
__device__ __forceinline__ uint32_t fma_bits(__half2 a, __half2 b, __half2 c) {
  const __half2 r = __hfma2(a, b, c);
  return *reinterpret_cast<const uint32_t*>(&r);
}
__device__ __forceinline__ uint32_t bits_of(__half2 x) { return *reinterpret_cast<const uint32_t*>(&x); }
// What rn(c s) lacks of c s; fp16 holds it exactly.
__device__ __forceinline__ uint32_t low_part(__half2 c, __half2 s) { return fma_bits(c, s, __hneg2(__hmul2(c, s))); }

__device__ __forceinline__ uint32_t ld_s32(uint32_t a) { return attend::ld_s32<0>(a); }
__device__ __forceinline__ uint2 ld_s64(uint32_t a) { return attend::ld_s64<0>(a); }
__device__ __forceinline__ uint4 ld_s128(uint32_t a) { return attend::ld_s128<0>(a); }

// Maximum (or sum) over groups of L lanes of v[0..N): lane l of a group ends with that of column
// l / (L / N) in v[0] (N > L: of N / L columns from l N / L on).  The lanes halve the columns they
// hold at each step.
template <int N, bool MAX, int L = 32>
__device__ __forceinline__ void column_reduce(float (&v)[N], int lane) {
  auto op = [](float x, float y) { return MAX ? fmaxf(x, y) : x + y; };
  int w = N;
#pragma unroll
  for (int o = L / 2; o >= 1; o >>= 1) {
    if (w > 1) {
      w >>= 1;
      const bool up = lane & o;
#pragma unroll
      for (int i = 0; i < N / 2; ++i) {
        if (i < w) {
          const float give = up ? v[i] : v[i + w], keep = up ? v[i + w] : v[i];
          v[i] = op(keep, __shfl_xor_sync(0xffffffffu, give, o));
        }
      }
    } else {
      v[0] = op(v[0], __shfl_xor_sync(0xffffffffu, v[0], o));
    }
  }
}

// x as two fp16 parts, the low one `low` bytes behind the high one.
__device__ __forceinline__ void st_two_parts(uint32_t at, uint32_t low, float x) {
  const __half hi = __float2half_rn(x), lo = __float2half_rn(x - __half2float(hi));
  asm volatile("st.shared.u16 [%0], %1;" ::"r"(at), "h"(__half_as_ushort(hi)) : "memory");
  asm volatile("st.shared.u16 [%0], %1;" ::"r"(at + low), "h"(__half_as_ushort(lo)) : "memory");
}

// (a0, a1) += (b0, b1) in one instruction; the largest of three in one.
__device__ __forceinline__ void add_pair(float& a0, float& a1, float b0, float b1) {
  asm("{\n .reg .b64 a, b;\n mov.b64 a, {%0, %1};\n mov.b64 b, {%2, %3};\n add.rn.f32x2 a, a, b;\n mov.b64 {%0, %1}, a;\n}"
      : "+f"(a0), "+f"(a1)
      : "f"(b0), "f"(b1));
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

template <int THREADS>
__device__ __forceinline__ void bar_arrive(int id) {
  asm volatile("barrier.cta.arrive %0, %1;" ::"r"(id), "n"(THREADS) : "memory");
}
template <int THREADS>
__device__ __forceinline__ void bar_sync(int id) {
  asm volatile("barrier.cta.sync %0, %1;" ::"r"(id), "n"(THREADS) : "memory");
}
// Barrier of the compute warps; true if `p` is for any of their threads.
template <int THREADS>
__device__ __forceinline__ bool bar_vote(bool p) {
  uint32_t r;
  asm volatile(
      "{\n .reg .pred p, q;\n setp.ne.u32 p, %1, 0;\n barrier.cta.red.or.pred q, %2, %3, p;\n selp.u32 %0, 1, 0, q;\n}"
      : "=r"(r)
      : "r"((uint32_t)p), "n"(kBarVote), "n"(THREADS)
      : "memory");
  return r != 0;
}

// A bounded wait on an mbarrier in a few instructions (it stands at every wait of the
// tile loop) that counts SM cycles: reading the global timer costs more than the wait.
// The hint lets the hardware suspend the warp, so that it does not take issue slots.
__device__ __forceinline__ bool try_wait_hint(uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n .reg .pred p;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n selp.u32 %0, 1, 0, p;\n}"
      : "=r"(ok)
      : "r"(smem_u32(bar)), "r"(parity), "r"(20000u)
      : "memory");
  return ok != 0;
}
__device__ __forceinline__ bool wait_bounded(uint64_t* bar, uint32_t parity, long long limit_cycles) {
  if (try_wait_hint(bar, parity)) return true;
  const long long t0 = clock64();
  bool ok;
#pragma unroll 1
  do {
    ok = try_wait_hint(bar, parity);
  } while (!ok && clock64() - t0 <= limit_cycles);
  return ok;
}

// Groups c .. c + U - 1 (past n_end: that one again, the same bytes to the same place) of a
// block, all of width 4, 2 or 1, or all of width 3 (B3), from the lane table
// `tab`: the loads of all of them first, then the arithmetic and the stores.
// K side (SIDE 0): (code - 1) s of coordinates 2 t4 (+ 8) of an even token (dst) and an odd
// one (dst2), of the groups before n_lo in two parts, the low ones at their groups' offsets
// `lo`; V side: c = rn(code s + z) of coordinates gid (+ 8) of token pairs t4 and t4 + 4.
template <int G, int SIDE, int U, bool B3>
__device__ __forceinline__ void unpack_batch(uint32_t tab, int c, int n_end, uint32_t sec, uint32_t blk, uint32_t rec,
                                             int tpp, uint32_t more_shift, uint32_t hi_word, uint32_t rot,
                                             int n_lo, uint32_t lo, uint32_t dst, uint32_t dst2) {
  uint4 d[U];  // {word offset, record offset, mask, shift | 32 width << 8 | operand offset << 16}
  uint32_t w[U], w3[U];
  uint2 ra[U], rb[U];
#pragma unroll
  for (int u = 0; u < U; ++u) d[u] = ld_s128(tab + (uint32_t)min(c + u, n_end) * 512u);
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const uint32_t code = sec + d[u].x + blk * __byte_perm(d[u].w, 0u, 0x4441);
    w[u] = ld_s32(code);
    if (B3) w3[u] = ld_s32(code + hi_word);  // code bit 2
    if (SIDE == 0) ra[u].x = ld_s32(sec + d[u].y + rec);
    if (SIDE == 1) ra[u] = ld_s64(sec + d[u].y + rec);
    if (SIDE == 1) rb[u] = ld_s64(sec + d[u].y + rec + (uint32_t)(32 * tpp));
  }
  const __half2 h1024 = __float2half2_rn(SIDE == 0 ? 1025.f : 1024.f), h64 = __float2half2_rn(SIDE == 0 ? 65.f : 64.f);
#pragma unroll
  for (int u = 0; u < U; ++u) {
    {
      uint32_t x = __funnelshift_r(w[u], 0u, d[u].w);  // (its low five bits)
      if (B3) x = (x & 0x33333333u) | (__funnelshift_r(w3[u], w3[u], rot) & 0xCCCCCCCCu);
      if (G == 8) x >>= more_shift;
      const uint32_t y = x >> 8, m = d[u].z, m4 = m << 4;
      const __half2 c0 = __hsub2(as_half2((x & m) | 0x64006400u), h1024);
      const __half2 c1 = __hsub2(as_half2((x & m4) | 0x54005400u), h64);
      const __half2 c2 = __hsub2(as_half2((y & m) | 0x64006400u), h1024);
      const __half2 c3 = __hsub2(as_half2((y & m4) | 0x54005400u), h64);
      const uint32_t o = d[u].w >> 16;
      if (SIDE == 0) {
        const __half2 s = as_half2(ra[u].x), se = __low2half2(s), so = __high2half2(s);
        st_s32(dst + o, bits_of(__hmul2(c0, se)));
        st_s32(dst2 + o, bits_of(__hmul2(c1, so)));
        if (G == 16) {
          st_s32(dst + o + 128, bits_of(__hmul2(c2, se)));
          st_s32(dst2 + o + 128, bits_of(__hmul2(c3, so)));
        }
        const int k = min(c + u, n_end);
        if (B3 || k < n_lo) {
          const uint32_t l = ld_s32(lo + (uint32_t)k * 4u);
          st_s32(dst + l, low_part(c0, se));
          st_s32(dst2 + l, low_part(c1, so));
          if (G == 16) {
            st_s32(dst + l + 128, low_part(c2, se));
            st_s32(dst2 + l + 128, low_part(c3, so));
          }
        }
      } else {
        st_s32(dst + o, fma_bits(c0, as_half2(ra[u].x), as_half2(ra[u].y)));
        st_s32(dst + o + 128, fma_bits(c2, as_half2(rb[u].x), as_half2(rb[u].y)));
        if (G == 16) {
          st_s32(dst + o + 2048, fma_bits(c1, as_half2(ra[u].x), as_half2(ra[u].y)));
          st_s32(dst + o + 2048 + 128, fma_bits(c3, as_half2(rb[u].x), as_half2(rb[u].y)));
        }
      }
    }
  }
}

// The kept groups of one side of a 16-token block (`blk16` of the page's section), all
// of them or half `part` (pairs of the plain ones in turn, the others in turn).  K side:
// groups of width 4 (the first n_four), 3 and 8 go in two parts.
template <int G, int SIDE, int PARTS>
__device__ __forceinline__ void unpack_block(const int4* ord, uint32_t tab, int n_four, int n_plain, int n_three, int n_all,
                                             uint32_t sec, int blk16, int tpp, int part, const LaneAddr& L, int gid, int t4,
                                             uint32_t lo, uint32_t dst, uint32_t dst2) {
  const uint32_t blk = (uint32_t)(G == 16 ? blk16 : blk16 >> 1), rec = (uint32_t)(blk16 * 8);
  const uint32_t more = G == 16 ? 0u : (uint32_t)((blk16 & 1) * (SIDE == 0 ? 8 : 4));
  constexpr int kAny = 1 << 20;  // no clamp
#pragma unroll 1
  for (int c = PARTS == 2 ? 2 * part : 0; c < n_plain; c += 4) {
    const int n = n_plain - c;
    if (PARTS == 2) {
      unpack_batch<G, SIDE, 2, false>(tab, c, n_plain - 1, sec, blk, rec, tpp, more, 0u, 0u, n_four, lo, dst, dst2);
    } else if (n >= 4) {
      unpack_batch<G, SIDE, 4, false>(tab, c, kAny, sec, blk, rec, tpp, more, 0u, 0u, n_four, lo, dst, dst2);
    } else {
      if (n >= 2) unpack_batch<G, SIDE, 2, false>(tab, c, kAny, sec, blk, rec, tpp, more, 0u, 0u, n_four, lo, dst, dst2);
      if (n & 1) unpack_batch<G, SIDE, 1, false>(tab, c + n - 1, kAny, sec, blk, rec, tpp, more, 0u, 0u, n_four, lo, dst, dst2);
    }
  }
#pragma unroll 1
  for (int c = n_plain + (PARTS == 2 ? 2 * part : 0); c < n_three; c += 2 * PARTS) {
    const uint32_t hi = 64u + L.off1 - L.off2;
    if (PARTS == 2 || n_three - c >= 2)
      unpack_batch<G, SIDE, 2, true>(tab, c, PARTS == 2 ? n_three - 1 : kAny, sec, blk, rec, tpp, more, hi, L.rot1, n_four, lo, dst, dst2);
    else
      unpack_batch<G, SIDE, 1, true>(tab, c, kAny, sec, blk, rec, tpp, more, hi, L.rot1, n_four, lo, dst, dst2);
  }
#pragma unroll 1
  for (int c = n_three + (PARTS == 2 ? part : 0); c < n_all; c += PARTS) {  // width 8
    const int4 g = ord[c];
    __half2 v[4];
    load_bytes<G>(sec + (uint32_t)g.x + blk * 256u + L.off8, SIDE, blk16 & 1, v);
    const uint2 a = ld_s64(sec + (uint32_t)g.y + (uint32_t)((SIDE == 0 ? gid : t4) * tpp * 8) + rec);
    if (SIDE == 0) {
      const __half2 s = as_half2(a.x), se = __low2half2(s), so = __high2half2(s);
      const uint32_t o = (uint32_t)(g.z * (G / 8 * 128)), l = ld_s32(lo + (uint32_t)c * 4u);
#pragma unroll
      for (int i = 0; i < (G == 16 ? 4 : 2); ++i) {
        const uint32_t at = (i & 1 ? dst2 : dst) + (uint32_t)(i / 2 * 128);
        st_s32(at + o, bits_of(__hmul2(v[i], i & 1 ? so : se)));
        st_s32(at + l, low_part(v[i], i & 1 ? so : se));
      }
    } else {
      const uint2 b = ld_s64(sec + (uint32_t)g.y + (uint32_t)((t4 + 4) * tpp * 8) + rec);
      const uint32_t o = (uint32_t)(g.z * (G / 8 * 2048));
      st_s32(dst + o, fma_bits(v[0], as_half2(a.x), as_half2(a.y)));
      st_s32(dst + o + 128, fma_bits(v[2], as_half2(b.x), as_half2(b.y)));
      if (G == 16) {
        st_s32(dst + o + 2048, fma_bits(v[1], as_half2(a.x), as_half2(a.y)));
        st_s32(dst + o + 2048 + 128, fma_bits(v[3], as_half2(b.x), as_half2(b.y)));
      }
    }
  }
}

// z and s of every K group of a 16-token block: lane (pair of groups lane >> 3, pair of
// tokens lane & 7); zeros for the groups that there are not.  dst: the z chunk's row of the even
// token, dst2: of the odd one.
__device__ __forceinline__ void unpack_offsets(uint32_t pos, int n_groups, uint32_t sec, int blk16, int tpp, int lane,
                                               uint32_t dst, uint32_t dst2) {
  const int p = (lane >> 3) * 2;
  const uint32_t at = sec + (uint32_t)(((lane & 7) * tpp + blk16) * 8);
  const uint2 off = ld_s64(pos + (uint32_t)p * 4u);
  uint2 a = make_uint2(0u, 0u), b = a;
  if (p < n_groups) a = ld_s64(at + off.x);
  if (p + 1 < n_groups) b = ld_s64(at + off.y);
  const uint32_t word = (uint32_t)(lane >> 3) * 4u;
  st_s32(dst + word, __byte_perm(a.y, b.y, 0x5410));
  st_s32(dst2 + word, __byte_perm(a.y, b.y, 0x7632));
  st_s32(dst + word + 128u, __byte_perm(a.x, b.x, 0x5410));
  st_s32(dst2 + word + 128u, __byte_perm(a.x, b.x, 0x7632));
}

template <int G, int NB, int W, int CTAS>
__global__ void __launch_bounds__(32 * W + 32, CTAS) prefix_kernel(const __grid_constant__ PrefixArgs A) {
  // W compute warps (8 or 16): 4 token quarters (TMEM lanes) x W / 4 parts of the rows for
  // the softmax; 8 blocks of a tile x W / 8 shares of the groups for the unpacking
  constexpr int kPfWarps = W, kPfCompute = 32 * W, kPfThreads = kPfCompute + 32, PARTS = W / 8;
  constexpr int HC = NB * 4 / W;         // rows (columns of S^T) per thread
  // The next tile's keys are unpacked while this tile's scores wait in TMEM.  With 128 rows, whose
  // operands leave the ring two tiles, they come after the scores have turned into P, when their
  // pages have landed (64 x 28k at 4x: 171 us a call instead of 190; with fewer rows and a deep
  // ring the later S would cost: 70.5 us instead of 69.2, 4 x 128k at 8x).
  constexpr bool kLate = NB == 128;
  constexpr uint32_t kTmemCols = 4 * NB;  // (a power of two)
  constexpr uint32_t kS = 0, kO = 2 * NB;  // TMEM columns: two S buffers, O
  constexpr uint32_t kIdS = tc::idesc(kPfTok, NB, false), kIdO = tc::idesc(128, NB, true);
  constexpr uint32_t kIdF = tc::idesc(128, NB, false, true);
  extern __shared__ __align__(128) uint8_t smem[];
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + kPfBars);
  uint64_t* bar_s = bars + kPfMaxStages;
  uint64_t* bar_o = bar_s + 1;
  uint64_t* bar_d = bar_s + 2;
  uint64_t* bar_f = bar_s + 3;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + kPfMisc);
  volatile int* quit = reinterpret_cast<volatile int*>(smem + kPfMisc + 4);
  int* own_s = reinterpret_cast<int*>(smem + kPfMisc + 8);
  int* low_s = reinterpret_cast<int*>(smem + kPfMisc + 12);  // K steps and positions (bits) with low parts
  int4* ord = reinterpret_cast<int4*>(smem + kPfOrd);
  float* wmax_s = reinterpret_cast<float*>(smem + kPfWMax);
  uint4* lane_t = reinterpret_cast<uint4*>(smem + kPfLane);
  const uint32_t sV = smem_u32(smem + kPfV), sK = smem_u32(smem) + A.off_k, sQ = smem_u32(smem) + A.off_q,
                 sP = smem_u32(smem) + A.off_p, ring = smem_u32(smem) + A.off_ring;

  const CodecDev* __restrict__ cd = A.cd;
  const int split = blockIdx.x, a = blockIdx.y, r0 = blockIdx.z * NB;
  const int tid = threadIdx.x, lane = tid & 31, gid = lane >> 2, t4 = lane & 3;
  const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);  // (uniform for the compiler)
  const int sub = warp & 3, col0 = ((warp >> 2) & (W / 4 - 1)) * HC;  // its TMEM lanes and rows
  const int block = warp & 7, part = PARTS == 2 ? (warp >> 3) & 1 : 0;  // its 16-token block of a tile, its share
  // (read once: the compiler reloads a dynamically indexed parameter after every asm)
  const int4 hm0 = reinterpret_cast<const int4*>(A.hm[a])[0], hm1 = reinterpret_cast<const int4*>(A.hm[a])[1],
             hm2 = reinterpret_cast<const int4*>(A.hm[a])[2];
  const int sec_off = hm0.x, sec_bytes = hm0.y;
  const int P = A.P, tpp = P / 16, S = A.stages, nK = hm0.z, nV = hm0.w, nkK = hm1.x, nkV = hm1.y;
  const int nkd = main_chunks(nkK), ck = hm2.x, cq = q_chunks(nkK);  // chunks: kept coordinates, K row, Q row
  LaneAddr L;
  L.off4 = lane * 4;
  L.off8 = lane * 8;
  L.off2 = (2 * gid + (t4 >> 1)) * 4;
  L.off1 = gid * 4;
  L.sh2 = 2u * (uint32_t)(t4 & 1);
  L.sh1 = (uint32_t)t4;
  L.rot1 = (uint32_t)(t4 - 2) & 31u;

  // ---- tables ---------------------------------------------------------------------
  const DecodeOrder* __restrict__ dec = &cd->head[a].dec;
  // groups of width 4, 2 and 1 come first, then those of width 3
  const int fourK = dec->cls[0][1], plainK = dec->cls[0][3], plainV = dec->cls[1][3], threeK = dec->cls[0][4], threeV = dec->cls[1][4];
  if (warp < kPfWarps) {
#pragma unroll
    for (int s = part; s < 2; s += PARTS) {  // this warp's entries of the sides' lists
      const int e = s * kMaxG + block;
      const int4 g = __ldg(reinterpret_cast<const int4*>(dec->ord[s][block]));
      if (lane == 0) ord[e] = g;
      const uint32_t off = g.w == 4 ? L.off4 : (g.w == 1 ? L.off1 : L.off2);
      const uint32_t sh = g.w == 4 ? 0u : (g.w == 1 ? L.sh1 : L.sh2);
      lane_t[e * 32 + lane] =
          make_uint4((uint32_t)g.x + off, (uint32_t)(g.y + (s ? t4 : gid) * tpp * 8), ((1u << g.w) - 1u) * 0x00010001u,
                     sh | (uint32_t)(g.w << 13) | (uint32_t)(g.z * (s ? G / 8 * 2048 : G / 8 * 128)) << 16);
    }
  }
  int* pos_s = reinterpret_cast<int*>(smem + kPfPos);  // [3][8], see kPfPos
  if (warp == 0) {
    const int4 g = lane < nK ? __ldg(reinterpret_cast<const int4*>(dec->ord[0][lane])) : make_int4(0, 0, 0, 0);
    const int step = g.z * G / 16;
    const bool wide = lane < nK && wide_code(g.w);
    const uint32_t steps = __reduce_or_sync(0xffffffffu, wide ? 1u << step : 0u);
    const uint32_t wides = __reduce_or_sync(0xffffffffu, wide ? 1u << g.z : 0u);
    if (lane < nK) {
      pos_s[g.z] = g.y;
      pos_s[kMaxG + lane] = (nkd + 2 + 2 * __popc(steps & ((1u << step) - 1u)) + (G == 8 ? g.z & 1 : 0)) * 128;
    }
    if ((steps >> lane) & 1u) pos_s[2 * kMaxG + __popc(steps & ((1u << lane) - 1u))] = lane;
    if (lane == 0) {
      low_s[0] = (int)steps;
      low_s[1] = (int)wides;
    }
  }
  // pages of at most 128 tokens: `pages_per` whole pages per tile; longer pages:
  // `tiles_per` tiles per page
  const bool small = P <= kPfTok;
  const int pages_per = A.pages_per, tiles_per = A.tiles_per;
  float l[HC];
#pragma unroll
  for (int c = 0; c < HC; ++c) l[c] = 0.f;
  bool failed = false;  // a wait of this thread ran out
  bool done = true;     // every tile was summed (compute warps)
  uint32_t tmem = 0;

  if (warp == kPfWarps) {
    // ================= the MMA and copy warp =================
    if (lane == 0) {
      for (int s = 0; s < S; ++s) mbar_init(&bars[s], 1);
      mbar_init(bar_s, 1);
      mbar_init(bar_o, 1);
      mbar_init(bar_d, 1);
      mbar_init(bar_f, 1);
      fence_mbar_init();
      *quit = 0;
    }
    tc::alloc(tmem_slot, kTmemCols);
    pdl_wait();  // the pages may come from earlier kernels
    const int p0 = split * A.pages_lo + min(split, A.pages_rem);
    int n_own = A.pages_lo + (split < A.pages_rem ? 1 : 0);
    bool bad = false;
    int first_pid = 0;  // of page `lane`
    for (int i = lane; i < n_own; i += 32) {
      const int pid = A.pages[p0 + i];
      if (i == lane) first_pid = pid;
      bad |= pid < 0 || (int64_t)pid >= A.n_pool_pages;
    }
    if (__any_sync(0xffffffffu, bad)) {
      if (lane == 0) device_error(A.err, SPECTRA_ERR_INVALID);
      n_own = 0;
    }
    auto issue_copy = [&](int i, int pid) {  // page i of this CTA into stage i % S (one thread)
      if (i == A.drop_page && (split | a | r0) == 0) return;
      const uint8_t* src = A.pool + (size_t)pid * (size_t)A.page_bytes + sec_off;
      mbar_arrive_expect_tx(&bars[i % S], (uint32_t)sec_bytes);
      bulk_copy_g2s(smem + A.off_ring + (size_t)(i % S) * A.stage_bytes, src, (uint32_t)sec_bytes, &bars[i % S]);
    };
    int n_issued = sec_bytes > 0 ? min(S, n_own) : 0;
    if (lane < n_issued) issue_copy(lane, first_pid);
    if (lane == 0) *own_s = n_own;
    tc::fence_before();
    bar_sync<kPfThreads>(kBarReady);
    tc::fence_after();
    pdl_launch_dependents();  // (see the compute warps)
    tmem = *tmem_slot;
    const int T = small ? (n_own + pages_per - 1) / pages_per : n_own * tiles_per;
    int sub_tile = 0;  // of the page, for long pages
    // the fold: bf16 parts of W_up^K (from V's bytes on) times q (P's bytes)
    {
      const int fd = A.fold_dims;
      const uint64_t dW = tc::desc(sV, 128, fd * 32), dq = tc::desc(sP, 128, fd * 16);
#pragma unroll 1
      for (int db = 0; db < A.d_h; db += fd) {
        if (db > 0) {
          bar_sync<kPfThreads>(kBarKeys);
          tc::fence_after();
        }
        const int n = min(fd, A.d_h - db) / 16;
        if (tc::elect()) {
#pragma unroll 1
          for (int k = 0; k < n; ++k) {
            tc::mma(tmem + kS, dW + (uint64_t)(k * 16), dq + (uint64_t)(k * 16), kIdF, db > 0 || k > 0);
            tc::mma(tmem + kS, dW + (uint64_t)(fd + k * 16), dq + (uint64_t)(k * 16), kIdF, true);
          }
          tc::commit(bar_f);
        }
        __syncwarp();
      }
    }
    const uint64_t dK = tc::desc(sK, 128, ck * 128), dQ = tc::desc(sQ, 128, cq * 128);
    const int n_main = nkd / 2, n_low = __popc((uint32_t)low_s[0]);
    const uint64_t dV = tc::desc(sV, 128, 2048), dP = tc::desc(sP, 128, 2048);
    int t = -1;
    for (; t < T; ++t) {  // iteration t: S of tile t + 1, then O of tile t
      if (t + 1 < T) {
        bar_sync<kPfThreads>(kBarKeys);
        tc::fence_after();
        if (tc::elect()) {
          const uint32_t d = tmem + kS + (uint32_t)(((t + 1) & 1) * NB);
#pragma unroll 1
          for (int k = 0; k <= n_main; ++k) {  // the last: z and s
            tc::mma(d, dK + (uint64_t)(k * 16), dQ + (uint64_t)(k * 16), kIdS, k > 0);
            tc::mma(d, dK + (uint64_t)(k * 16), dQ + (uint64_t)((n_main + 1 + k) * 16), kIdS, true);
          }
#pragma unroll 1
          for (int i = 0; i < n_low; ++i)
            tc::mma(d, dK + (uint64_t)((n_main + 1 + i) * 16), dQ + (uint64_t)(pos_s[2 * kMaxG + i] * 16), kIdS, true);
          tc::commit(bar_s);
        }
        __syncwarp();
      }
      if (t < 0) continue;
      bar_sync<kPfThreads>(kBarValues);
      if (*quit) break;
      tc::fence_after();
      const int n = nkV == 0 ? 0 : (small ? min(pages_per, n_own - t * pages_per) * tpp
                                          : min(kPfTok, P - sub_tile * kPfTok) / 16);
      if (tc::elect()) {
#pragma unroll 1
        for (int k = 0; k < n; ++k)
          tc::mma(tmem + kO, dV + (uint64_t)(k * 16), dP + (uint64_t)(k * 16), kIdO, t > 0 || k > 0);
        tc::commit(bar_o);
      }
      __syncwarp();
      // the pages that this tile finished leave their stages to the next ones
      int first = t * pages_per, count = pages_per;
      if (!small) {
        first = t / tiles_per;
        count = ++sub_tile == tiles_per ? 1 : 0;
        if (count) sub_tile = 0;
      }
      const int i = first + S + lane;
      if (sec_bytes > 0 && lane < count && i < n_own) issue_copy(i, A.pages[p0 + i]);
      __syncwarp();
      if (sec_bytes > 0) n_issued = max(n_issued, min(n_own, first + count + S));
    }
    if (t < T && lane == 0) {
      // a wait ran out in the compute warps: MMAs and copies in flight end before the
      // TMEM and the shared memory go
      tc::commit(bar_d);
      wait_bounded(bar_d, 0u, A.wait_cycles);
      for (int i = max(0, n_issued - S); i < n_issued; ++i)
        wait_bounded(&bars[i % S], (uint32_t)((i / S) & 1), A.wait_cycles);
    }
    __syncwarp();
  } else {
    // ================= the compute warps =================
    auto wait = [&](uint64_t* bar, int phase) -> bool {
      const bool ok = wait_bounded(bar, (uint32_t)(phase & 1), A.wait_cycles);
      if (!ok) {
        device_error(A.err, SPECTRA_ERR_TIMEOUT);
        failed = true;
      }
      return __all_sync(0xffffffffu, ok);
    };
    // ---- the fold: Q [rows][coordinates] = q W_up^K^T, fp16, K-major core matrices.
    // Per fold_dims (fd) dims: W_up^K as bf16 parts hi and lo (from V's bytes on; for every
    // 8 coordinates hi's fd / 8 chunks of 8 dims, then lo's) and q (in P's); the products
    // come back from TMEM, coordinates in lanes.
    const int fd = A.fold_dims, fc = fd >> 3, fcs = fd == 128 ? 4 : 3;  // chunks of 8 dims, log2
#pragma unroll 1
    for (int db = 0, ph = 0; db < A.d_h; db += fd, ++ph) {
      const int nd = min(fd, A.d_h - db);
      if (db > 0) wait(bar_f, ph - 1);
      const float* wk = cd->w_up + hm1.z + db;
#pragma unroll 2
      for (int e = tid; e < (nkd * 8) << fcs; e += kPfCompute) {
        const int kg = e >> (3 + fcs), k = kg * 8 + (e & 7), c8 = (e >> 3) & (fc - 1);
        float4 x = make_float4(0.f, 0.f, 0.f, 0.f), y = x;
        if (k < nkK && c8 * 8 < nd) {
          const float4* src = reinterpret_cast<const float4*>(wk + (size_t)k * A.d_h + c8 * 8);
          x = __ldg(src);
          y = __ldg(src + 1);
        }
        const float v[8] = {x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w};
        uint32_t hi[4], lo[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
          const __nv_bfloat162 r = __floats2bfloat162_rn(v[2 * i] - __low2float(h), v[2 * i + 1] - __high2float(h));
          hi[i] = *reinterpret_cast<const uint32_t*>(&h);
          lo[i] = *reinterpret_cast<const uint32_t*>(&r);
        }
        const uint32_t dst = sV + (uint32_t)(kg * fd * 32 + c8 * 128 + (e & 7) * 16);
        st_s128(dst, hi[0], hi[1], hi[2], hi[3]);
        st_s128(dst + (uint32_t)(fd * 16), lo[0], lo[1], lo[2], lo[3]);
      }
      if (db == 0) pdl_wait();  // (W_up is the codec's) q may come from an earlier kernel
#pragma unroll 2
      for (int e = tid; e < NB << fcs; e += kPfCompute) {
        const int ng = e >> (3 + fcs), n = ng * 8 + (e & 7), c8 = (e >> 3) & (fc - 1), r = r0 + n, b = r / A.gq;
        uint4 v = make_uint4(0u, 0u, 0u, 0u);
        if (r < A.rows && c8 * 8 < nd)
          v = __ldcg(reinterpret_cast<const uint4*>(
              A.q + ((size_t)b * A.n_q + (size_t)a * A.gq + (r - b * A.gq)) * A.d_h + db + c8 * 8));
        st_s128(sP + (uint32_t)(ng * fd * 16 + c8 * 128 + (e & 7) * 16), v.x, v.y, v.z, v.w);
      }
      fence_proxy_async_smem();
      if (db == 0) {
        bar_sync<kPfThreads>(kBarReady);  // barriers, TMEM and this CTA's pages are known too
        tc::fence_after();
        tmem = *tmem_slot;
        // Only now: with this CTA's TMEM in hand a later kernel's CTAs that hold TMEM and
        // wait for this grid cannot keep it from its own; and every thread has passed its
        // dependency wait, on which the decode kernel behind relies (AttendArgs::late_wait).
        pdl_launch_dependents();
      } else {
        bar_arrive<kPfThreads>(kBarKeys);
      }
    }
    const int n_own = *own_s;
    const int T = small ? (n_own + pages_per - 1) / pages_per : n_own * tiles_per;
    // this thread's token: S^T row `row` of the tile, token `tok` in page order
    const int row = sub * 32 + lane;
    const int pos = row & 7, half8 = (row >> 3) & 1;
    const int tok = (row & ~15) + half8 * 8 + 2 * (pos & 3) + ((pos >> 2) ^ half8);
    const uint32_t lane_base = tmem + ((uint32_t)(sub * 32) << 16) + (uint32_t)col0;
    const uint32_t p_dst = sP + (uint32_t)((col0 / 8) * 2048 + (tok >> 3) * 128 + (tok & 7) * 16 + (col0 & 7) * 2);
    {
      wait(bar_f, (A.d_h - 1) >> (3 + fcs));
      tc::fence_after();
      float v[HC];
      tc::ld<HC>(lane_base + kS, v);
      tc::fence_before();
      // coordinate `row` (zero beyond the kept ones) of rows col0 .., and its group's sum
      const uint32_t low = (uint32_t)((nkd + 2) * 128);
      const uint32_t at = sQ + (uint32_t)((col0 / 8) * cq * 128 + (row >> 3) * 128 + (row & 7) * 2 + (col0 & 7) * 16);
      const int g = row / G;
      const uint32_t at_sum = sQ + (uint32_t)((col0 / 8) * cq * 128 + nkd * 128 + g * 2 + (col0 & 7) * 16);
#pragma unroll
      for (int c = 0; c < HC; ++c) {
        v[c] *= A.q_scale;
        if (row < nkd * 8) st_two_parts(at + (uint32_t)((c >> 3) * cq * 128 + (c & 7) * 16), low, v[c]);
      }
      column_reduce<HC, false, G>(v, lane);
      constexpr int kMine = HC > G ? HC / G : 1, kSame = HC > G ? 1 : G / HC;  // columns of a lane, lanes of a column
      if (g < kMaxG && lane % kSame == 0) {
#pragma unroll
        for (int i = 0; i < kMine; ++i) {
          const int c = lane % G / kSame * kMine + i;
          const uint32_t at_c = at_sum + (uint32_t)((c >> 3) * cq * 128 + (c & 7) * 16);
          const float sum = g < nK ? v[i] : 0.f;
          st_two_parts(at_c, low, sum);         // times z
          st_two_parts(at_c + 128u, low, sum);  // times s
        }
      }
    }
    // the chunks of K that no group writes: padding (an odd number of 8-coordinate groups, or no
    // keys at all) and, beside the low parts of a group of 8, those of its step's other group
    if (tid < kPfTok) {
      const uint32_t at = sK + (uint32_t)((tid >> 3) * ck * 128 + (tid & 7) * 16);
      for (int kd = nkK / 8; kd < nkd; ++kd) st_s128(at + (uint32_t)(kd * 128), 0u, 0u, 0u, 0u);
      if (G == 8) {
        const uint32_t steps = (uint32_t)low_s[0], wides = (uint32_t)low_s[1];
        for (int p = 0; p < 2 * (nkd / 2); ++p)
          if (((steps >> (p >> 1)) & 1u) && !((wides >> p) & 1u))
            st_s128(at + (uint32_t)((nkd + 2 + 2 * __popc(steps & ((1u << (p >> 1)) - 1u)) + (p & 1)) * 128), 0u, 0u, 0u, 0u);
      }
    }

    // ---- tiles --------------------------------------------------------------------
    const uint32_t tabK = smem_u32(lane_t) + (uint32_t)(lane * 16), tabV = tabK + kMaxG * 512;
    const uint32_t k_dst = sK + (uint32_t)((block * 2 + (gid >> 2)) * ck * 128 + t4 * 4);
    const uint32_t z_dst = sK + (uint32_t)(((block * 2 + ((lane & 7) >> 2)) * ck + nkd) * 128);
    const uint32_t pos_a = smem_u32(pos_s);
    const uint32_t v_dst = sV + (uint32_t)(block * 256 + gid * 16 + t4 * 4);
    // this warp's block of the tile whose keys come next: page (of this CTA's list) and
    // its stage and phase, first token in the page; the block whose values come next
    // follows one tile behind
    const int k_page = small ? block * 16 / P : 0;
    int page = k_page, stage = k_page, phase = 0, tau = block * 16 - k_page * P;
    uint32_t v_sec = 0;
    int v_blk = -1;
    auto unpack_keys = [&]() {
      const bool here = small ? k_page < pages_per && page < n_own : tau < P;
      const uint32_t sec = ring + (uint32_t)(stage * A.stage_bytes);
      v_blk = -1;
      if (here && (sec_bytes == 0 || wait(&bars[stage], phase))) {
        v_sec = sec;
        v_blk = tau >> 4;
        unpack_block<G, 0, PARTS>(ord, tabK, fourK, plainK, threeK, nK, sec, v_blk, tpp, part, L, gid, t4, pos_a + 32u,
                                  k_dst + (uint32_t)(gid * 16), k_dst + (uint32_t)((gid ^ 4) * 16));
        if (part == PARTS - 1)
          unpack_offsets(pos_a, nK, sec, v_blk, tpp, lane, z_dst + (uint32_t)((lane & 7) * 16),
                         z_dst + (uint32_t)(((lane & 7) ^ 4) * 16));
      }
      int adv = pages_per;
      if (!small) {
        tau += kPfTok;
        adv = tau >= tiles_per * kPfTok ? 1 : 0;
        if (adv) tau = block * 16;
      }
      page += adv;
      stage += adv;
      if (stage >= S) {
        stage -= S;
        phase ^= 1;
      }
    };

    auto next_keys = [&](int t) {
      if (t + 1 < T) {
        unpack_keys();
        fence_proxy_async_smem();
        tc::fence_before();
        bar_arrive<kPfThreads>(kBarKeys);
      }
    };

    if (T > 0) {
      unpack_keys();
      fence_proxy_async_smem();  // (and the Q tile)
      bar_arrive<kPfThreads>(kBarKeys);
    }
    float m_run = -CUDART_INF_F;  // lane l: m of row col0 + l / (32 / HC)
    float* off_w = reinterpret_cast<float*>(smem + kPfOffs) + sub * 128 + col0;
    float* fac_w = reinterpret_cast<float*>(smem + kPfFac) + sub * 128 + col0;
    if (lane < HC) off_w[lane] = 0.f;
    float off_run = 0.f;
    constexpr int kLc = 32 / HC;  // lanes per row of the state m_run, off_run
    int* over_s = reinterpret_cast<int*>(smem + kPfOver) + col0;  // [event & 1][128]
    int event = 0;
    if (sub == 0 && lane < HC) over_s[lane] = over_s[128 + lane] = INT_MIN;
    __syncwarp();
    int sub_tile = 0;  // of the page, for long pages
    for (int t = 0; t < T; ++t) {
      wait(bar_s, t);  // S of tile t is there, K's bytes are free
      tc::fence_after();
      const uint32_t sec_t = v_sec;
      const int blk_t = v_blk;
      if (!kLate) next_keys(t);
      // tokens of a short tile's missing blocks: none
      const int n_blk = small ? min(pages_per, n_own - t * pages_per) * tpp : min(kPfTok, P - sub_tile * kPfTok) / 16;
      if (!small && ++sub_tile == tiles_per) sub_tile = 0;
      const bool live = (row >> 4) < n_blk;
      auto add_offsets = [&](float (&v)[HC]) {
#pragma unroll
        for (int c = 0; c < HC; c += 4) {
          const float4 o = *reinterpret_cast<const float4*>(off_w + c);
          add_pair(v[c], v[c + 1], o.x, o.y);
          add_pair(v[c + 2], v[c + 3], o.z, o.w);
        }
      };
      auto drop_missing = [&](float (&v)[HC]) {
        if (!live) {
#pragma unroll
          for (int c = 0; c < HC; ++c) v[c] = -CUDART_INF_F;
        }
      };
      const uint32_t s_addr = lane_base + kS + (uint32_t)((t & 1) * NB);
      float y[HC];
      tc::ld<HC>(s_addr, y);
      float mx = -CUDART_INF_F;
      add_offsets(y);
      if (n_blk < kPfTok / 16) drop_missing(y);
#pragma unroll
      for (int c = 0; c < HC; c += 2) mx = max3(mx, y[c], y[c + 1]);
      const bool failed_now = failed;
      if (bar_vote<kPfCompute>(t == 0 || failed_now || mx > kPfLimit)) {
        // The first tile: the exact maxima of its scores by row (column of S^T).  Later:
        // the maxima of the rows that went over the limit.  They become the new m; l
        // and O of these rows go from the old m to it.
        int* over = over_s + (event & 1) * 128;
        if (t == 0) {
          column_reduce<HC, true>(y, lane);  // (fmaxf: a NaN counts only where nothing else stands)
          if (lane % kLc == 0) wmax_s[sub * 128 + col0 + lane / kLc] = y[0];
        } else {
          if (mx > kPfLimit) {
#pragma unroll
            for (int c = 0; c < HC; ++c)
              if (y[c] > kPfLimit) atomicMax(over + c, __float_as_int(y[c]));  // (positive: ordered as integers)
          }
          wait(bar_o, t - 1);
        }
        if (bar_vote<kPfCompute>(failed_now)) {
          done = false;
          *quit = 1;
          if (kLate && t + 1 < T) bar_arrive<kPfThreads>(kBarKeys);  // (which the MMA warp waits for first)
          bar_arrive<kPfThreads>(kBarValues);  // (orders the flag before the MMA warp's look at it)
          break;
        }
        // (each warp for its own rows: the four warps of a row half get the same)
        float m = m_run;
        if (t == 0) {
          const float* w = wmax_s + col0 + lane / kLc;
          m = fmaxf(fmaxf(fmaxf(w[0], w[128]), fmaxf(w[256], w[384])), m_run);
        } else {
          const int v = over[lane / kLc];
          if (v != INT_MIN) m = __int_as_float(v) - off_run;
          if (sub == 0 && lane < HC) over_s[((event & 1) ^ 1) * 128 + lane] = INT_MIN;  // for the next event
          ++event;
        }
        const float off_new = m == -CUDART_INF_F ? 0.f : kPfOff - m;
        const float fac = m == m_run ? 1.f : (m_run == -CUDART_INF_F ? 0.f : attend::ex2_approx(m_run - m));
        if (lane % kLc == 0) {
          off_w[lane / kLc] = off_new;
          if (t > 0) fac_w[lane / kLc] = fac;  // (the first tile's maxima may still be read)
        }
        const uint32_t moved = __ballot_sync(0xffffffffu, m != m_run && lane % kLc == 0);
        m_run = m;
        off_run = off_new;
        __syncwarp();
        if (t == 0) {
          tc::ld<HC>(s_addr, y);
        } else {
          tc::fence_after();
          if (moved) {
            float o[HC];
            tc::ld<HC>(lane_base + kO, o);
#pragma unroll
            for (int c = 0; c < HC; c += 4) {
              const float4 f = *reinterpret_cast<const float4*>(fac_w + c);
              o[c] *= f.x;
              o[c + 1] *= f.y;
              o[c + 2] *= f.z;
              o[c + 3] *= f.w;
              l[c] *= f.x;
              l[c + 1] *= f.y;
              l[c + 2] *= f.z;
              l[c + 3] *= f.w;
            }
            tc::st<HC>(lane_base + kO, o);
          }
          tc::ld<HC>(s_addr, y);  // (not kept over the rescaling: registers)
        }
        add_offsets(y);
        drop_missing(y);
      }
      uint32_t pk[HC / 2];
#pragma unroll
      for (int c = 0; c < HC; c += 2) {
        const float pa = attend::ex2_approx(y[c]), pb = attend::ex2_approx(y[c + 1]);
        add_pair(l[c], l[c + 1], pa, pb);
        pk[c / 2] = pack_half2(pa, pb);
      }
      if (t > 0) wait(bar_o, t - 1);  // P and V are free
      if constexpr (HC == 4) {
        asm volatile("st.shared.v2.b32 [%0], {%1,%2};" ::"r"(p_dst), "r"(pk[0]), "r"(pk[1]) : "memory");
      } else {
#pragma unroll
        for (int c = 0; c < HC / 8; ++c)
          st_s128(p_dst + c * 2048, pk[4 * c], pk[4 * c + 1], pk[4 * c + 2], pk[4 * c + 3]);
      }
      if (kLate) next_keys(t);
      if (blk_t >= 0)
        unpack_block<G, 1, PARTS>(ord + kMaxG, tabV, 0, plainV, threeV, nV, sec_t, blk_t, tpp, part ^ (PARTS - 1), L, gid, t4,
                                  0u, v_dst, 0u);
      fence_proxy_async_smem();
      tc::fence_before();
      bar_arrive<kPfThreads>(kBarValues);
    }

    // ---- records ---------------------------------------------------------------------
    // o: latent sums of coordinate `row` for this thread's rows col0 ..; rows step
    // through (sequence, q head)
    float o[HC];
    const bool any = done && T > 0;
    if (any) {
      wait(bar_o, T - 1);
      tc::fence_after();
      tc::ld<HC>(lane_base + kO, o);
    } else {
#pragma unroll
      for (int c = 0; c < HC; ++c) o[c] = 0.f;
    }
    const size_t head_step = A.rec_stride;
    const size_t seq_step = ((size_t)A.n_kv * A.n_merge * A.gq - (A.gq - 1)) * A.rec_stride;
    auto record = [&](int r) -> float* {
      const int b = r / A.gq, h = r - b * A.gq;
      return A.rec + ((((size_t)b * A.n_kv + a) * A.n_merge + A.rec_first + split) * A.gq + h) * A.rec_stride;
    };
    if (row < nkV) {
      float* dst = record(r0 + col0) + 4 + row;
      int h = (r0 + col0) % A.gq;
#pragma unroll
      for (int c = 0; c < HC; ++c) {
        if (r0 + col0 + c < A.rows) *dst = o[c];
        const bool wrap = ++h == A.gq;
        dst += wrap ? seq_step : head_step;
        h = wrap ? 0 : h;
      }
    }
    column_reduce<HC, false>(l, lane);
    if (lane % kLc == 0) wmax_s[sub * 128 + col0 + lane / kLc] = l[0];
    bar_vote<kPfCompute>(false);
    if (sub == 0 && lane % kLc == 0) {
      const int c = col0 + lane / kLc;
      if (r0 + c < A.rows) {
        const float sum = (wmax_s[c] + wmax_s[128 + c]) + (wmax_s[256 + c] + wmax_s[384 + c]);
        // the records' convention is p = 2^(s - m + 8)
        *reinterpret_cast<float2*>(record(r0 + c)) =
            make_float2(any && m_run != -CUDART_INF_F ? attend::kPScaleLog2 - off_run : -CUDART_INF_F, any ? sum : 0.f);
      }
    }
  }
  tc::fence_before();
  __syncthreads();
  if (warp == kPfWarps) tc::dealloc(tmem, kTmemCols);
}

using PrefixKernel = void (*)(const PrefixArgs);

// Two CTAs of 8 compute warps where shared memory holds two, else one of 16: with one CTA of
// 8 warps 8 sequences x 32k at 4x took 63.7 us a call, with 16 warps 62.2 (keys then in one part).  Two CTAs of 16
// warps have 56 registers a thread, which suits 16 rows only: with 32 or 64 rows they took 78 and
// 59 us where 8 warps took 75 and 50 (4 x 128k at 8x, 16 x 32k at 12x).
template <int G>
PrefixKernel prefix_kernel_of(int n_cols, int ctas, int* warps) {
  *warps = ctas == 1 || n_cols == 16 ? 16 : 8;
  switch (n_cols) {
    case 16: return prefix_kernel<G, 16, 16, 2>;
    case 32: return ctas == 1 ? prefix_kernel<G, 32, 16, 1> : prefix_kernel<G, 32, 8, 2>;
    case 64: return ctas == 1 ? prefix_kernel<G, 64, 16, 1> : prefix_kernel<G, 64, 8, 2>;
    default: return prefix_kernel<G, 128, 16, 1>;
  }
}

// Chunks of a K row of head `hd`: kept coordinates, z and s, a step for each with a wide group.
int k_chunks(const CodecDev& h, const HeadDev& hd) {
  const SideDev& k = hd.side[0];
  uint32_t steps = 0;
  for (int j = 0; j < k.n_groups; ++j)
    if (wide_code(k.grp[j].b)) steps |= 1u << (j * h.group / 16);
  int n = 0;
  for (; steps; steps &= steps - 1) ++n;
  return main_chunks(k.n_kept) + 2 + 2 * n;
}

struct PrefixSmem {
  int off_k, off_q, off_p, off_ring, stage_bytes, stages, total, fold_dims;
};

constexpr int kPfSmemMax = 227 * 1024;  // of a CTA that has an SM for itself

// V, K, Q, P, and as many page stages as leave room for two CTAs per SM, else for one: two tiles'
// pages at least, eight tiles' at most.
PrefixSmem prefix_smem(const CodecDev& h, int n_cols) {
  PrefixSmem s{};
  auto up = [](int x) { return (x + 127) / 128 * 128; };
  const int nkd = main_chunks(h.max_kept_k);
  int ck = 0;
  for (int a = 0; a < h.n_kv; ++a) ck = std::max(ck, k_chunks(h, h.head[a]));
  s.off_k = up(kPfV + h.max_kept_v / 8 * 2048);
  s.off_q = s.off_k + 16 * ck * 128;
  s.off_p = s.off_q + n_cols / 8 * q_chunks(h.max_kept_k) * 128;
  s.off_ring = s.off_p + n_cols / 8 * 2048;
  // the fold's W_up^K takes V's, K's and Q's bytes (its MMA reads 128 coordinates)
  s.fold_dims = h.d_h > 64 && nkd * 4096 <= s.off_p - kPfV ? 128 : 64;
  s.stage_bytes = std::max(16, (h.max_sec_bytes + 15) / 16 * 16);
  const int per = h.P <= kPfTok ? kPfTok / h.P : 1;
  const int lo = 2 * per, hi = std::min(kPfMaxStages, 8 * per);
  const int one = kPfSmemMax, two = 113 * 1024;
  auto fit = [&](int budget) { return std::min(hi, std::max(0, budget - s.off_ring) / s.stage_bytes); };
  s.stages = n_cols == 128 ? 0 : fit(two);
  if (s.stages < lo) s.stages = std::max(lo, fit(one));
  // (the MMAs read 128 rows of V, and of W_up^K in its place, whatever is there)
  s.total = std::max(s.off_ring + s.stages * s.stage_bytes, kPfV + 16 * s.fold_dims * 32);
  return s;
}

}  // namespace

// The fewest columns of 16, 32, 64 and 128 that hold the rows (128: several blocks).
// Fewer columns cost fewer score and exp2 instructions a token; in blocks of 64 rows 64
// sequences x 28k at 4x unpacked every code four times and took 239 us, in blocks of 128 165 us.
// Fewer where two tiles' pages would not fit beside the operands (many wide groups; 32 always fit:
// 8 groups of 16 at 8 bits on both sides, the most there is, take 225,024 bytes).
int prefix_columns(const CodecDev& h, int rows) {
  int n = rows <= 16 ? 16 : (rows <= 32 ? 32 : (rows <= 64 ? 64 : 128));
  while (n > 32 && prefix_smem(h, n).total > kPfSmemMax) n /= 2;
  return n;
}

int prefix_smem_bytes(const CodecDev& h, int n_cols, int* stages) {
  const PrefixSmem s = prefix_smem(h, n_cols);
  *stages = s.stages;
  return s.total;
}

int prefix_ctas_per_sm(int n_cols, int smem) {
  return n_cols < 128 && smem <= 113 * 1024 ? 2 : 1;
}

cudaError_t launch_prefix(const CodecDev& h, const CodecDev* d, const spectra_cache& cache, const uint16_t* q,
                          const int32_t* prefix_pages, int n_prefix, float* rec, int rec_stride, int rec_first,
                          int n_merge, const SharedPlan& plan, cudaStream_t st) {
  const PrefixSmem s = prefix_smem(h, plan.n_cols);
  PrefixArgs A{};
  A.cd = d;
  A.err = h.err;
  A.pool = static_cast<const uint8_t*>(cache.pool);
  A.pages = prefix_pages;
  A.q = q;
  A.rec = rec;
  A.n_pool_pages = cache.n_pages;
  A.page_bytes = h.page_bytes;
  // test hooks for the bounded waits: SPECTRA_PREFIX_TEST_DROP_PAGE makes the first CTA skip
  // the copy of that page of its list, SPECTRA_DECODE_TEST_WAIT_NS shortens every wait's limit
  const char* drop = std::getenv("SPECTRA_PREFIX_TEST_DROP_PAGE");
  A.drop_page = drop ? std::atoi(drop) : -1;
  const char* w = std::getenv("SPECTRA_DECODE_TEST_WAIT_NS");
  const long long wn = w ? std::atoll(w) : 0;
  A.wait_cycles = 2 * (wn > 0 ? wn : (long long)attend::kWaitLimitNs);  // at most 2 GHz
  A.pages_lo = n_prefix / plan.n_prefix_split;
  A.pages_rem = n_prefix % plan.n_prefix_split;
  A.rec_stride = rec_stride;
  A.rec_first = rec_first;
  A.n_merge = n_merge;
  A.rows = cache.batch * h.gq;
  A.pages_per = h.P <= kPfTok ? kPfTok / h.P : 1;
  A.tiles_per = h.P <= kPfTok ? 1 : (h.P + kPfTok - 1) / kPfTok;
  A.fold_dims = s.fold_dims;
  A.stages = s.stages;
  A.stage_bytes = s.stage_bytes;
  A.off_k = s.off_k;
  A.off_q = s.off_q;
  A.off_p = s.off_p;
  A.off_ring = s.off_ring;
  A.n_q = h.n_q;
  A.n_kv = h.n_kv;
  A.d_h = h.d_h;
  A.P = h.P;
  A.gq = h.gq;
  A.q_scale = 1.4426950408889634f / sqrtf((float)h.d_h);
  for (int a = 0; a < h.n_kv; ++a) {
    const HeadDev& hd = h.head[a];
    int32_t* m = A.hm[a];
    m[0] = hd.sec_off;
    m[1] = hd.sec_bytes;
    m[2] = hd.side[0].n_groups;
    m[3] = hd.side[1].n_groups;
    m[4] = hd.side[0].n_kept;
    m[5] = hd.side[1].n_kept;
    m[6] = hd.wupk_rows_off;
    m[7] = hd.side[1].wup_off;
    m[8] = k_chunks(h, hd);
  }
  int warps = 0;
  const int ctas = prefix_ctas_per_sm(plan.n_cols, s.total);
  const PrefixKernel kern =
      h.group == 16 ? prefix_kernel_of<16>(plan.n_cols, ctas, &warps) : prefix_kernel_of<8>(plan.n_cols, ctas, &warps);
  const cudaError_t e = ensure_dynamic_smem(reinterpret_cast<const void*>(kern), s.total);
  if (e != cudaSuccess) return e;
  return launch_dependent(kern, dim3(plan.n_prefix_split, h.n_kv, plan.n_blocks), dim3(32 * warps + 32), s.total, st, A);
}

}  // namespace spectra
