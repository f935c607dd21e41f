// Rotary positions of query and key heads (spectra_rope_apply).
//
// Every pair (x, y) of a head's leading rot_dim dimensions turns by the token's
// position times the pair's frequency:  (x c - y s, x s + y c), c = m cos a,
// s = m sin a (inverse: a -> -a, m -> 1/m).  The pairs are (i, i + r/2) or
// (2i, 2i + 1); the frequencies come from the host (rope_frequencies).
//
// Bound: HBM.  Every element is read once and written once, and one sincos per (token,
// pair) is shared by all of the token's heads.  A CTA takes `tok` tokens and a range of
// the heads.  A thread has one token and one vector of VEC pairs (two vectors of VEC
// elements) and walks every `lanes`-th head of the queries, then of the keys, kRopeBatch
// at a time; its {c, s} come once from a table in shared memory that the CTA forms
// while the first heads' loads are under way.  VEC is the widest (up to 16 bytes)
// that the strides, addresses, rot_dim and d_head allow.
// Measured: 65536 tokens of 28 + 4 heads of 128 in bf16 take 174 us, 6.17 TB/s (94 % of
// a copy's rate); batches of two heads 199 us, items (token, head, vector) dealt
// out evenly with {c, s} read from the table for each 275 us, walks of
// both tensors in registers at once 221-241 us.  4097 tokens of 8 + 8 heads of 128 in fp32,
// 96 dimensions turned, take 19 us.  A decode step (16 tokens of 32 + 8 heads) takes 3.7 us, of which
// the launch and one round trip to memory are most.
// Angles: turns of pi, position x frequency / pi, are formed in fp64 and reduced
// to [-1, 1] there (fp32 has no digits left at position 10^6); the remainder goes
// through sincospif in fp32.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>

#include "device_common.cuh"
#include "kernels.h"

namespace spectra {

namespace {

constexpr int kRopeThreads = 256;
constexpr int kRopeTokMax = 8;  // tokens of one CTA
constexpr int kRopeBatch = 4;   // heads a thread has under way

struct RopeTensor {
  const uint8_t* in;
  uint8_t* out;
  int64_t in_tok, in_head, out_tok, out_head;  // strides in elements
  int heads;
};

struct RopeArgs {
  RopeTensor x[2];  // queries, keys
  const int32_t* positions;
  int64_t n_tokens;
  int d_head, rot, tok, split;  // split: head ranges per token tile (gridDim.y)
  int n_rot, n_all;             // vectors of pairs, and with the copied dimensions, of a head
  int lanes;                    // threads that share a token's vector: kRopeThreads / (tok n_all)
  float mag, sign;
  double half_turns[kRopeMaxPairs];
};

template <int BYTES>
struct Raw;
template <>
struct Raw<2> { using T = uint16_t; };
template <>
struct Raw<4> { using T = uint32_t; };
template <>
struct Raw<8> { using T = uint2; };
template <>
struct Raw<16> { using T = uint4; };

template <typename E, int VEC>
struct Vec {
  union {
    typename Raw<sizeof(E) * VEC>::T raw;
    E e[VEC];
  };
  __device__ __forceinline__ Vec() {}
  __device__ __forceinline__ void load(const E* p) { raw = *reinterpret_cast<const decltype(raw)*>(p); }
  __device__ __forceinline__ void store(E* p) const { *reinterpret_cast<decltype(raw)*>(p) = raw; }
};

__device__ __forceinline__ float to_f(float x) { return x; }
__device__ __forceinline__ float to_f(uint16_t x) { return __uint_as_float((uint32_t)x << 16); }
__device__ __forceinline__ void from_f(float& d, float x) { d = x; }
__device__ __forceinline__ void from_f(uint16_t& d, float x) { d = __bfloat16_as_ushort(__float2bfloat16_rn(x)); }

// Turns VEC pairs held in two vectors.
template <typename E, int VEC, bool INTER>
__device__ __forceinline__ void turn_vectors(Vec<E, VEC>& a, Vec<E, VEC>& b, const float2 (&cs)[VEC]) {
  auto turn = [](E& p, E& q, float2 c) {
    const float x = to_f(p), y = to_f(q);
    from_f(p, x * c.x - y * c.y);
    from_f(q, x * c.y + y * c.x);
  };
  if constexpr (INTER && VEC == 1) {
    turn(a.e[0], b.e[0], cs[0]);
  } else if constexpr (INTER) {  // pairs lie side by side: VEC / 2 in a, VEC / 2 in b
#pragma unroll
    for (int k = 0; k < VEC / 2; ++k) {
      turn(a.e[2 * k], a.e[2 * k + 1], cs[k]);
      turn(b.e[2 * k], b.e[2 * k + 1], cs[VEC / 2 + k]);
    }
  } else {
#pragma unroll
    for (int k = 0; k < VEC; ++k) turn(a.e[k], b.e[k], cs[k]);
  }
}

// {c, s} of the CTA's tokens and pairs.
__device__ __forceinline__ void form_table(const RopeArgs& A, int64_t t0, int nt, int half, float2* cs_s) {
  for (int i = threadIdx.x; i < nt * half; i += kRopeThreads) {
    const int t = i / half, k = i - t * half;
    const double turns = (double)A.positions[t0 + t] * A.half_turns[k];
    const float r = (float)(turns - 2.0 * rint(0.5 * turns));
    float sn, cn;
    sincospif(r, &sn, &cn);
    cs_s[i] = make_float2(cn * A.mag, sn * A.mag * A.sign);
  }
}

// E: float, or uint16_t holding bf16 bits
template <typename E, int VEC, bool INTER>
__global__ void __launch_bounds__(kRopeThreads) rope_kernel(const __grid_constant__ RopeArgs A) {
  constexpr int U = kRopeBatch;
  extern __shared__ float2 cs_s[];  // [tok][rot / 2] {c, s}
  const int tid = threadIdx.x;
  const int64_t t0 = (int64_t)blockIdx.x * A.tok;
  const int nt = (int)min((int64_t)A.tok, A.n_tokens - t0);
  const int half = A.rot >> 1;
  const int per = A.tok * A.n_all, lane_h = tid / per, tv = tid - lane_h * per;
  const int t = tv / A.n_all, v = tv - t * A.n_all;
  const bool pairs = v < A.n_rot;
  // of this thread's vectors in a head: the first, and from it to the second
  const int ia = pairs ? (INTER ? 2 * v * VEC : v * VEC) : A.rot + (v - A.n_rot) * VEC;
  const int ib = INTER ? VEC : half;
  pdl_wait();
  const int pos = t < nt ? A.positions[t0 + t] : -1;
  const bool on = pos >= 0 && lane_h < A.lanes;  // (a negative position: the token is left out)

  Vec<E, VEC> a[U], b[U];
  float2 cs[VEC];
#pragma unroll
  for (int w = 0; w < 2; ++w) {
    const RopeTensor& X = A.x[w];
    const int h1 = (int)((int64_t)X.heads * (blockIdx.y + 1) / A.split);
    int h = (int)((int64_t)X.heads * blockIdx.y / A.split) + lane_h;
    const E* src = reinterpret_cast<const E*>(X.in) + (t0 + t) * X.in_tok + h * X.in_head + ia;
    E* dst = reinterpret_cast<E*>(X.out) + (t0 + t) * X.out_tok + h * X.out_head + ia;
    const int64_t in_step = A.lanes * X.in_head, out_step = A.lanes * X.out_head;
    const bool move = on && (pairs || X.in != X.out);
    auto load = [&]() {
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (move && h + u * A.lanes < h1) {
          a[u].load(src + u * in_step);
          if (pairs) b[u].load(src + u * in_step + ib);
        }
      }
    };
    load();
    if (w == 0) {
      form_table(A, t0, nt, half, cs_s);
      __syncthreads();
      if (on && pairs) {
#pragma unroll
        for (int k = 0; k < VEC; ++k) cs[k] = cs_s[t * half + v * VEC + k];
      }
    }
    if (!move) continue;
    while (true) {
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (h + u * A.lanes < h1) {
          if (pairs) {
            turn_vectors<E, VEC, INTER>(a[u], b[u], cs);
            b[u].store(dst + u * out_step + ib);
          }
          a[u].store(dst + u * out_step);
        }
      }
      h += U * A.lanes;
      if (h >= h1) break;
      src += U * in_step;
      dst += U * out_step;
      load();
    }
  }
}

// Short calls: one thread's head of one tensor.
template <typename E, int VEC, bool INTER>
struct OneHead {
  Vec<E, VEC> a, b;
  const E* src;
  E* dst;
  bool move;

  __device__ __forceinline__ OneHead(const RopeTensor& X, const RopeArgs& A, int64_t token, int lane_h, bool in,
                                     bool pairs, int ia) {
    const int h = (int)((int64_t)X.heads * blockIdx.y / A.split) + lane_h;
    src = reinterpret_cast<const E*>(X.in) + token * X.in_tok + h * X.in_head + ia;
    dst = reinterpret_cast<E*>(X.out) + token * X.out_tok + h * X.out_head + ia;
    move = in && h < (int)((int64_t)X.heads * (blockIdx.y + 1) / A.split) && (pairs || X.in != X.out);
  }
  __device__ __forceinline__ void load(bool pairs, int ib) {
    if (move) {
      a.load(src);
      if (pairs) b.load(src + ib);
    }
  }
  __device__ __forceinline__ void store(bool pairs, int ib, const float2 (&cs)[VEC]) {
    if (move) {
      if (pairs) {
        turn_vectors<E, VEC, INTER>(a, b, cs);
        b.store(dst + ib);
      }
      a.store(dst);
    }
  }
};

// The same for calls whose threads have one head of each tensor at most (a decode step):
// both tensors' loads go out first.
template <typename E, int VEC, bool INTER>
__global__ void __launch_bounds__(kRopeThreads) rope_short_kernel(const __grid_constant__ RopeArgs A) {
  extern __shared__ float2 cs_s[];  // [tok][rot / 2] {c, s}
  const int tid = threadIdx.x;
  const int64_t t0 = (int64_t)blockIdx.x * A.tok;
  const int nt = (int)min((int64_t)A.tok, A.n_tokens - t0);
  const int half = A.rot >> 1;
  const int per = A.tok * A.n_all, lane_h = tid / per, tv = tid - lane_h * per;
  const int t = tv / A.n_all, v = tv - t * A.n_all;
  const bool pairs = v < A.n_rot;
  const int ia = pairs ? (INTER ? 2 * v * VEC : v * VEC) : A.rot + (v - A.n_rot) * VEC;
  const int ib = INTER ? VEC : half;
  pdl_wait();
  const bool in = t < nt && lane_h < A.lanes;
  OneHead<E, VEC, INTER> q(A.x[0], A, t0 + t, lane_h, in, pairs, ia), k(A.x[1], A, t0 + t, lane_h, in, pairs, ia);
  q.load(pairs, ib);
  k.load(pairs, ib);
  form_table(A, t0, nt, half, cs_s);
  __syncthreads();
  if (!in || A.positions[t0 + t] < 0) return;  // (a negative position: the token is left out)
  float2 cs[VEC];
  if (pairs) {
#pragma unroll
    for (int j = 0; j < VEC; ++j) cs[j] = cs_s[t * half + v * VEC + j];
  }
  q.store(pairs, ib, cs);
  k.store(pairs, ib, cs);
}

template <typename E, int VEC>
auto rope_kernel_of(bool inter, bool short_call) -> void (*)(const RopeArgs) {
  if (short_call) return inter ? rope_short_kernel<E, VEC, true> : rope_short_kernel<E, VEC, false>;
  return inter ? rope_kernel<E, VEC, true> : rope_kernel<E, VEC, false>;
}

template <typename E>
auto rope_kernel_for(int vec, bool inter, bool short_call) -> void (*)(const RopeArgs) {
  switch (vec) {
    case 8:
      if constexpr (sizeof(E) == 2) return rope_kernel_of<E, 8>(inter, short_call);
      return nullptr;
    case 4: return rope_kernel_of<E, 4>(inter, short_call);
    case 2: return rope_kernel_of<E, 2>(inter, short_call);
    default: return rope_kernel_of<E, 1>(inter, short_call);
  }
}

}  // namespace

cudaError_t launch_rope(const RopeFreq& f, bool bf16, int d_head, const int32_t* positions, int64_t n_tokens,
                        const spectra_heads* const in[2], const spectra_heads* const out[2], bool inverse,
                        cudaStream_t st) {
  RopeArgs A{};
  const int esz = bf16 ? 2 : 4;
  const int half = f.rot / 2, tail = d_head - f.rot;
  // widest vector: it divides the pairs, the copied dimensions, the strides and
  // the addresses, and holds at most 16 bytes
  int vec = 16 / esz;
  int heads = 0;
  for (int w = 0; w < 2; ++w) {
    RopeTensor& x = A.x[w];
    if (!in[w] || in[w]->n_heads == 0) continue;
    x.in = static_cast<const uint8_t*>(in[w]->data);
    x.out = static_cast<uint8_t*>(out[w]->data);
    x.in_tok = in[w]->token_stride;
    x.in_head = in[w]->head_stride;
    x.out_tok = out[w]->token_stride;
    x.out_head = out[w]->head_stride;
    x.heads = in[w]->n_heads;
    heads += x.heads;
    while (vec > 1 && (half % vec || tail % vec || x.in_tok % vec || x.in_head % vec || x.out_tok % vec ||
                       x.out_head % vec || reinterpret_cast<uintptr_t>(x.in) % (vec * esz) ||
                       reinterpret_cast<uintptr_t>(x.out) % (vec * esz)))
      vec /= 2;
  }
  if (n_tokens == 0 || heads == 0) return cudaSuccess;
  A.positions = positions;
  A.n_tokens = n_tokens;
  A.d_head = d_head;
  A.rot = f.rot;
  A.mag = (float)(inverse ? 1.0 / f.magnitude : f.magnitude);
  A.sign = inverse ? -1.f : 1.f;
  for (int i = 0; i < half; ++i) A.half_turns[i] = f.freq[i] / 3.14159265358979323846;
  A.n_rot = half / vec;
  A.n_all = A.n_rot + tail / vec;
  // Tokens per CTA: up to 8, while a thread still walks several heads and the grid fills
  // the GPU; a short call splits each token's heads over CTAs instead (each forms the
  // sincos again).
  int tok = 1;
  while (tok < kRopeTokMax && 2 * tok * A.n_all <= kRopeThreads && (n_tokens + 2 * tok - 1) / (2 * tok) >= 4 * sm_count())
    tok *= 2;
  const int64_t tiles = (n_tokens + tok - 1) / tok;
  int split = 1;
  while (tiles * split < sm_count() && split * 2 <= heads) split *= 2;
  A.tok = tok;
  A.split = split;
  A.lanes = kRopeThreads / (tok * A.n_all);
  const bool one = (std::max(A.x[0].heads, A.x[1].heads) + split - 1) / split <= A.lanes;
  auto kern = bf16 ? rope_kernel_for<uint16_t>(vec, f.interleaved, one) : rope_kernel_for<float>(vec, f.interleaved, one);
  // No programmatic launch: what follows may read the outputs before its own
  // dependency wait, so it may start only when this kernel has finished.
  kern<<<dim3((unsigned)tiles, (unsigned)split), kRopeThreads, (size_t)tok * half * sizeof(float2), st>>>(A);
  return cudaGetLastError();
}

}  // namespace spectra
