// Rotary positions (dsa_rope_steps, dsa_rope_apply): the rotated columns of up to
// four tensors of a layer in one launch, forwards and transposed.
//
// The angle of a pair is pos * f.  In fp32 that product has no bits of the turn's
// fraction left at far positions, and a table of sines is one more thing to read.
// Here f is a 64-bit fraction of a turn (good to some 2^-51 of itself, from fp64 on the host),
// and the product is taken modulo 2^64, that is modulo a turn: nothing is lost of it at any
// position.  Its upper 32 bits become a float, which keeps 24 of them (an angle is rounded
// by pi 2^-25 = 9e-8 radians at most, near half a turn), and go through sincospif.
//
// A CTA takes consecutive rows (a row: one head of one token), its threads the same pairs
// of several of them; sines and cosines of its tokens are computed once, into shared
// memory, while the first rows are on their way.  (Each thread its own instead: 122
// registers, a quarter of the SM's warps, 520 us where this takes 172.)
//
// Bound: HBM for many tokens.  16,384 tokens of the latent shapes (128 heads of 64 of 576
// columns, 64 index heads of 128; 1.09 GB) 172 us, 6.3 TB/s, 93 % of the copy's measured rate; the gradients of
// 8,192 90 us (90 %); 768 tokens 13 us (51 MB, 4.0 TB/s: launch and latency); one token 3 us.
// With few heads the table takes longer than the rows, and most of that is the steps: they are the
// kernel's parameters, read with another index by each lane, which goes one address after the
// other.  13,897 tokens of 8 + 1 heads of 256 bf16 columns 45 us (128 MB: 19 at the copy's rate), of 4 + 1 heads
// 38; with the steps in shared memory 30 and 23.
#include <math.h>

#include "dsa_common.cuh"

namespace dsa {
namespace rope {

constexpr int kThreads = 256;
constexpr int kTable = 2048;                       // pairs whose sine and cosine a CTA holds at once

struct Part {
  const uint8_t* x;
  uint8_t* out;
  long long x_tok, x_head, out_tok, out_head;      // strides in elements
  int heads, offset;
  int rot_slots, slots;                            // threads of a row: rotating ones, and copying ones behind them
  int kind;                                        // bit 0 fp32, bit 1 half layout, bit 2 sixteen bytes at a time
  unsigned rows, rows_cta, first_cta;              // rows in all and of a CTA
};
struct Args {
  Part part[DSA_ROPE_PARTS];
  int n_parts, half;                               // pairs of a row
  float mscale, sign;
  uint64_t step[DSA_ROPE_MAX_DIM / 2];
};

__device__ __forceinline__ void turn(int pos, uint64_t step, float m, float sign, float& c, float& s) {
  const uint64_t a = (uint64_t)(int64_t)pos * step;
  sincospif((float)(int32_t)(uint32_t)(a >> 32) * 4.6566128730773926e-10f, &s, &c);  // 2^-31: half turns
  c *= m;
  s *= m * sign;
}

// What a thread holds of a row, as it lies in memory: P pairs (or, of the columns that are
// copied, E elements).
template <typename T, bool HALF, bool VEC>
struct Piece;
template <typename T, bool HALF>
struct Piece<T, HALF, false> {
  static constexpr int P = 1, E = 1;
  T u, v;
  __device__ __forceinline__ void load(const T* p, int half) { u = p[0], v = p[HALF ? half : 1]; }
  __device__ __forceinline__ void store(T* p, int half) const { p[0] = u, p[HALF ? half : 1] = v; }
  __device__ __forceinline__ void load_copy(const T* p) { u = *p; }
  __device__ __forceinline__ void store_copy(T* p) const { *p = u; }
  __device__ __forceinline__ void get(float (&a)[1], float (&b)[1]) const { a[0] = to_f32(u), b[0] = to_f32(v); }
  __device__ __forceinline__ void set(const float (&a)[1], const float (&b)[1]) {
    u = from_f32<T>(a[0]), v = from_f32<T>(b[0]);
  }
};
template <bool HALF>
struct Piece<float, HALF, true> {
  static constexpr int P = 4, E = 4;
  float4 u, v;
  __device__ __forceinline__ void load(const float* p, int half) {
    u = *reinterpret_cast<const float4*>(p), v = *reinterpret_cast<const float4*>(p + (HALF ? half : 4));
  }
  __device__ __forceinline__ void store(float* p, int half) const {
    *reinterpret_cast<float4*>(p) = u, *reinterpret_cast<float4*>(p + (HALF ? half : 4)) = v;
  }
  __device__ __forceinline__ void load_copy(const float* p) { u = *reinterpret_cast<const float4*>(p); }
  __device__ __forceinline__ void store_copy(float* p) const { *reinterpret_cast<float4*>(p) = u; }
  __device__ __forceinline__ void get(float (&a)[4], float (&b)[4]) const {
    if constexpr (HALF) {
      a[0] = u.x, a[1] = u.y, a[2] = u.z, a[3] = u.w, b[0] = v.x, b[1] = v.y, b[2] = v.z, b[3] = v.w;
    } else {
      a[0] = u.x, b[0] = u.y, a[1] = u.z, b[1] = u.w, a[2] = v.x, b[2] = v.y, a[3] = v.z, b[3] = v.w;
    }
  }
  __device__ __forceinline__ void set(const float (&a)[4], const float (&b)[4]) {
    if constexpr (HALF) {
      u = make_float4(a[0], a[1], a[2], a[3]), v = make_float4(b[0], b[1], b[2], b[3]);
    } else {
      u = make_float4(a[0], b[0], a[1], b[1]), v = make_float4(a[2], b[2], a[3], b[3]);
    }
  }
};
template <bool HALF>
struct Piece<__nv_bfloat16, HALF, true> {
  static constexpr int P = 4, E = 8;
  uint2 u, v;
  __device__ __forceinline__ void load(const __nv_bfloat16* p, int half) {
    if constexpr (HALF) u = *reinterpret_cast<const uint2*>(p), v = *reinterpret_cast<const uint2*>(p + half);
    else load_copy(p);
  }
  __device__ __forceinline__ void store(__nv_bfloat16* p, int half) const {
    if constexpr (HALF) *reinterpret_cast<uint2*>(p) = u, *reinterpret_cast<uint2*>(p + half) = v;
    else store_copy(p);
  }
  __device__ __forceinline__ void load_copy(const __nv_bfloat16* p) {
    const uint4 w = *reinterpret_cast<const uint4*>(p);
    u = make_uint2(w.x, w.y), v = make_uint2(w.z, w.w);
  }
  __device__ __forceinline__ void store_copy(__nv_bfloat16* p) const {
    *reinterpret_cast<uint4*>(p) = make_uint4(u.x, u.y, v.x, v.y);
  }
  static __device__ __forceinline__ float lo(uint32_t w) { return __uint_as_float(w << 16); }
  static __device__ __forceinline__ float hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }
  __device__ __forceinline__ void get(float (&a)[4], float (&b)[4]) const {
    if constexpr (HALF) {
      a[0] = lo(u.x), a[1] = hi(u.x), a[2] = lo(u.y), a[3] = hi(u.y);
      b[0] = lo(v.x), b[1] = hi(v.x), b[2] = lo(v.y), b[3] = hi(v.y);
    } else {
      a[0] = lo(u.x), b[0] = hi(u.x), a[1] = lo(u.y), b[1] = hi(u.y);
      a[2] = lo(v.x), b[2] = hi(v.x), a[3] = lo(v.y), b[3] = hi(v.y);
    }
  }
  __device__ __forceinline__ void set(const float (&a)[4], const float (&b)[4]) {
    if constexpr (HALF) {
      u = make_uint2(pack_bf16x2(a[0], a[1]), pack_bf16x2(a[2], a[3]));
      v = make_uint2(pack_bf16x2(b[0], b[1]), pack_bf16x2(b[2], b[3]));
    } else {
      u = make_uint2(pack_bf16x2(a[0], b[0]), pack_bf16x2(a[1], b[1]));
      v = make_uint2(pack_bf16x2(a[2], b[2]), pack_bf16x2(a[3], b[3]));
    }
  }
};

template <typename T, bool HALF, bool VEC>
__device__ __forceinline__ void rotate_rows(const Args& g, const Part& p, const int32_t* __restrict__ pos, unsigned cta,
                                            float* __restrict__ cosines, float* __restrict__ sines) {
  using Q = Piece<T, HALF, VEC>;
  constexpr int P = Q::P, kUnroll = VEC && sizeof(T) == 4 ? 2 : 4;  // rows in flight: 64 bytes
  const int width = min(p.slots, kThreads);        // threads of a row
  const int rows_step = kThreads / width;
  const int r0 = threadIdx.x / width, s0 = threadIdx.x - r0 * width;
  const unsigned heads = p.heads, begin = cta * p.rows_cta, end = min(begin + p.rows_cta, p.rows);
  const unsigned token0 = begin / heads, tokens = (end - 1) / heads - token0 + 1;
  const unsigned h_step = rows_step % heads, t_step = rows_step / heads;
  const T* x = (const T*)p.x;
  T* out = (T*)p.out;
  bool tabled = false;
  for (int s = s0; s - s0 < p.slots; s += width) {
    const bool here = r0 < rows_step && s < p.slots, rotates = here && s < p.rot_slots;
    int col = p.offset + s * P * (HALF ? 1 : 2);   // first column of this thread
    if (!rotates) {
      col = (s - p.rot_slots) * Q::E;
      if (col >= p.offset) col += 2 * g.half;
    }
    unsigned row = here ? begin + r0 : end;
    unsigned t = row / heads, h = row - t * heads;
    const auto next = [&](unsigned& t, unsigned& h) {
      t += t_step, h += h_step;
      if (h >= heads) h -= heads, ++t;
    };
    Q q[kUnroll];
    const auto load = [&](unsigned row, unsigned t, unsigned h) {
#pragma unroll
      for (int k = 0; k < kUnroll; ++k, next(t, h))
        if (row + k * rows_step < end) {
          const T* at = x + t * p.x_tok + h * p.x_head + col;
          if (rotates) q[k].load(at, g.half);
          else q[k].load_copy(at);
        }
    };
    load(row, t, h);
    if (!tabled) {                                 // the first rows are on their way: sines and cosines of the tokens
      for (unsigned i = threadIdx.x; i < tokens * g.half; i += kThreads) {
        const unsigned k = i / g.half;
        turn(pos[token0 + k], g.step[i - k * g.half], g.mscale, g.sign, cosines[i], sines[i]);
      }
      __syncthreads();
      tabled = true;
    }
    float c[P], d[P];
    unsigned token = 0xFFFFFFFFu;
    while (row < end) {
#pragma unroll
      for (int k = 0; k < kUnroll; ++k) {
        if (row + k * rows_step < end) {
          T* at = out + t * p.out_tok + h * p.out_head + col;
          if (rotates) {
            if (t != token) {
              token = t;
              const int i = (t - token0) * g.half + s * P;
              if constexpr (P == 4) {
                const float4 e = *reinterpret_cast<const float4*>(cosines + i), f = *reinterpret_cast<const float4*>(sines + i);
                c[0] = e.x, c[1] = e.y, c[2] = e.z, c[3] = e.w, d[0] = f.x, d[1] = f.y, d[2] = f.z, d[3] = f.w;
              } else {
                c[0] = cosines[i], d[0] = sines[i];
              }
            }
            float a[P], b[P];
            q[k].get(a, b);
#pragma unroll
            for (int i = 0; i < P; ++i) {
              const float u = a[i] * c[i] - b[i] * d[i];
              b[i] = a[i] * d[i] + b[i] * c[i];
              a[i] = u;
            }
            q[k].set(a, b);
            q[k].store(at, g.half);
          } else {
            q[k].store_copy(at);
          }
        }
        next(t, h);
      }
      row += kUnroll * rows_step;
      if (row < end) load(row, t, h);
      else let_next_launch();                      // (not earlier: 300 tokens 7.9 us instead of 9.0)
    }
  }
}

__global__ void __launch_bounds__(kThreads, 4) rope_kernel(const __grid_constant__ Args g, const int32_t* __restrict__ pos) {
  __shared__ __align__(16) float cosines[kTable], sines[kTable];
  wait_for_earlier();
  int i = 0;
  while (i + 1 < g.n_parts && blockIdx.x >= g.part[i + 1].first_cta) ++i;
  const Part& p = g.part[i];
  const unsigned cta = blockIdx.x - p.first_cta;
  switch (p.kind) {
    case 0: return rotate_rows<__nv_bfloat16, false, false>(g, p, pos, cta, cosines, sines);
    case 1: return rotate_rows<float, false, false>(g, p, pos, cta, cosines, sines);
    case 2: return rotate_rows<__nv_bfloat16, true, false>(g, p, pos, cta, cosines, sines);
    case 3: return rotate_rows<float, true, false>(g, p, pos, cta, cosines, sines);
    case 4: return rotate_rows<__nv_bfloat16, false, true>(g, p, pos, cta, cosines, sines);
    case 5: return rotate_rows<float, false, true>(g, p, pos, cta, cosines, sines);
    case 6: return rotate_rows<__nv_bfloat16, true, true>(g, p, pos, cta, cosines, sines);
    default: return rotate_rows<float, true, true>(g, p, pos, cta, cosines, sines);
  }
}

// --------------------------------- host side ---------------------------------
// Elements from the first to behind the last one of a tensor's rows; false: they run
// into each other (apart: they must not) or out of 2^62.
static bool span(const dsa_rope_rows& r, long long n_tok, long long heads, long long dim, bool apart, long long* n) {
  const long long limit = 1ll << 40;
  if (r.tok_stride < 0 || r.head_stride < 0 || r.tok_stride > limit || r.head_stride > limit) return false;
  long long s0 = heads > 1 ? r.head_stride : 0, n0 = heads, s1 = n_tok > 1 ? r.tok_stride : 0, n1 = n_tok;
  if (n0 == 1 || (n1 > 1 && s0 > s1)) {
    const long long s = s0, k = n0;
    s0 = s1, n0 = n1, s1 = s, n1 = k;
  }
  if (apart && n0 > 1 && s0 < dim) return false;
  const __int128 inner = (__int128)(n0 - 1) * s0 + dim;
  if (apart && n1 > 1 && s1 < inner) return false;
  const __int128 all = inner + (__int128)(n1 - 1) * s1;
  if (all > ((__int128)1 << 58)) return false;
  *n = (long long)all;
  return true;
}

static int check(const dsa_rope* p) {
  if (!p) return DSA_ERR_INVALID_ARG;
  if (p->rot_dim < 2 || (p->rot_dim & 1) || p->n_parts < 1 || p->n_parts > DSA_ROPE_PARTS || !isfinite(p->mscale))
    return DSA_ERR_INVALID_ARG;
  if (p->rot_dim > DSA_ROPE_MAX_DIM) return DSA_ERR_UNSUPPORTED;
  for (int i = 0; i < p->n_parts; ++i) {
    const dsa_rope_part& q = p->part[i];
    if (q.dtype != DSA_BF16 && q.dtype != DSA_FP32) return DSA_ERR_UNSUPPORTED;
    if (q.layout != DSA_ROPE_INTERLEAVED && q.layout != DSA_ROPE_HALF) return DSA_ERR_INVALID_ARG;
    if (q.heads < 1 || q.dim < p->rot_dim || q.offset < 0 || q.offset > q.dim - p->rot_dim) return DSA_ERR_INVALID_ARG;
    if (q.dim > (1 << 20)) return DSA_ERR_UNSUPPORTED;
  }
  return DSA_OK;
}

}  // namespace rope
}  // namespace dsa

using namespace dsa;
using namespace dsa::rope;

extern "C" {

int dsa_rope_steps(dsa_rope* p, double base, int scaling, double factor, double original, double beta_fast,
                   double beta_slow) {
  if (!p || p->rot_dim < 2 || (p->rot_dim & 1)) return DSA_ERR_INVALID_ARG;
  if (p->rot_dim > DSA_ROPE_MAX_DIM) return DSA_ERR_UNSUPPORTED;
  if (scaling < DSA_ROPE_PLAIN || scaling > DSA_ROPE_YARN) return DSA_ERR_UNSUPPORTED;
  if (!(base > 1.0) || !isfinite(base)) return DSA_ERR_INVALID_ARG;
  if (scaling != DSA_ROPE_PLAIN && (!(factor >= 1.0) || !isfinite(factor))) return DSA_ERR_INVALID_ARG;
  const double r = p->rot_dim, two_pi = 6.283185307179586;
  double low = 0, high = 0;
  if (scaling == DSA_ROPE_YARN) {
    if (!(original > 0) || !isfinite(original) || !(beta_slow > 0) || !(beta_fast >= beta_slow) || !isfinite(beta_fast))
      return DSA_ERR_INVALID_ARG;
    // the pair that turns so many times in `original` positions
    const auto pair = [&](double turns) { return r * log(original / (turns * two_pi)) / (2 * log(base)); };
    low = fmax(floor(pair(beta_fast)), 0.0);
    high = fmin(ceil(pair(beta_slow)), r - 1);
  }
  if (scaling == DSA_ROPE_NTK && p->rot_dim > 2) base *= pow(factor, r / (r - 2));
  if (!isfinite(base)) return DSA_ERR_INVALID_ARG;
  for (int i = 0; i < p->rot_dim / 2; ++i) {
    double f = pow(base, -2.0 * i / r);
    if (scaling == DSA_ROPE_LINEAR) f /= factor;
    if (scaling == DSA_ROPE_YARN) {
      const double g = fmin(fmax((i - low) / fmax(high - low, 0.001), 0.0), 1.0);
      f = f * (1 - g) + f / factor * g;
    }
    p->step[i] = (uint64_t)(f / two_pi * 18446744073709551616.0);  // f <= 1: below 2^62
  }
  return DSA_OK;
}

int dsa_rope_apply(const dsa_rope* p, int64_t n_tok, const int32_t* pos, const dsa_rope_rows* x,
                   const dsa_rope_rows* out, int transposed, dsa_stream_t stream) {
  int rc = check(p);
  if (rc) return rc;
  if (n_tok < 1 || !pos || ((uintptr_t)pos & 3u) || !x || !out) return DSA_ERR_INVALID_ARG;
  Args g = {};
  g.n_parts = p->n_parts;
  g.half = p->rot_dim / 2;
  g.mscale = p->mscale;
  g.sign = transposed ? -1.f : 1.f;
  for (int i = 0; i < g.half; ++i) g.step[i] = p->step[i];
  long long work = 0, ctas = 0;                    // rows of all parts, in passes of a CTA's threads over them
  for (int i = 0; i < p->n_parts; ++i) {
    const dsa_rope_part& q = p->part[i];
    Part& t = g.part[i];
    const uintptr_t esz = q.dtype == DSA_BF16 ? 2 : 4;
    if (!x[i].base || !out[i].base || ((uintptr_t)x[i].base & (esz - 1)) || ((uintptr_t)out[i].base & (esz - 1)))
      return DSA_ERR_INVALID_ARG;
    if (q.heads >= (1ll << 31) || n_tok >= (1ll << 31) || q.heads * n_tok >= (1ll << 31)) return DSA_ERR_UNSUPPORTED;
    long long nx, no;
    if (!span(x[i], n_tok, q.heads, q.dim, false, &nx) || !span(out[i], n_tok, q.heads, q.dim, true, &no))
      return DSA_ERR_INVALID_ARG;
    const bool in_place = x[i].base == out[i].base && (n_tok == 1 || x[i].tok_stride == out[i].tok_stride) &&
                          (q.heads == 1 || x[i].head_stride == out[i].head_stride);
    const uintptr_t bx = (uintptr_t)x[i].base, bo = (uintptr_t)out[i].base;
    if (!in_place && bx < bo + no * esz && bo < bx + nx * esz) return DSA_ERR_INVALID_ARG;
    t.x = (const uint8_t*)x[i].base;
    t.out = (uint8_t*)out[i].base;
    t.x_tok = x[i].tok_stride, t.x_head = x[i].head_stride, t.out_tok = out[i].tok_stride, t.out_head = out[i].head_stride;
    t.heads = (int)q.heads, t.offset = (int)q.offset;
    const int rest = in_place ? 0 : (int)q.dim - p->rot_dim, e = 16 / (int)esz;
    // sixteen bytes at a time where rows, columns and the pairs of a thread allow it
    const uintptr_t at = bx | bo | (uintptr_t)((n_tok > 1 ? x[i].tok_stride | out[i].tok_stride : 0) * esz) |
                         (uintptr_t)((q.heads > 1 ? x[i].head_stride | out[i].head_stride : 0) * esz);
    const bool vec = (at & 15) == 0 && p->rot_dim % 8 == 0 && q.offset % e == 0 && rest % e == 0;
    t.kind = (q.dtype == DSA_FP32) | (q.layout == DSA_ROPE_HALF) << 1 | vec << 2;
    t.rot_slots = vec ? g.half / 4 : g.half;
    t.slots = t.rot_slots + (vec ? rest / e : rest);
    const int width = t.slots < kThreads ? t.slots : kThreads, rows_step = kThreads / width;
    t.rows = (unsigned)(q.heads * n_tok);
    work += t.rows / rows_step + 1;
  }
  // Passes of a CTA: as many as leave 512 CTAs (3.4 per SM), 16 at most.  1 / 2 / 4 / 8 / 16
  // passes: 16,384 tokens of the latent shapes 464 / 278 / 197 / 180 / 172 us, 768 tokens
  // 24.5 / 16.6 / 14.3 / 13.0 / 13.7, 333 tokens x 10 heads of 80 fp32 5.0 / 3.4 / 3.8 / 5.1 / 7.1.
  int passes = 1;
  while (passes < 16 && work / (2 * passes) >= 512) passes *= 2;
  for (int i = 0; i < p->n_parts; ++i) {
    Part& t = g.part[i];
    const int rows_step = kThreads / (t.slots < kThreads ? t.slots : kThreads);
    int n = passes;                                // the sines of the CTA's tokens have to fit the table
    while (n > 1 && (((long long)rows_step * n + t.heads - 2) / t.heads + 1) * g.half > kTable) --n;
    t.rows_cta = (unsigned)(rows_step * n);
    t.first_cta = (unsigned)ctas;
    ctas += (t.rows + t.rows_cta - 1) / t.rows_cta;
  }
  if (ctas >= (1ll << 31)) return DSA_ERR_UNSUPPORTED;
  return launch_programmatic(rope_kernel, dim3((unsigned)ctas), dim3(kThreads), 0, (cudaStream_t)stream, 1, g, pos)
             ? DSA_OK
             : DSA_ERR_CUDA;
}

}  // extern "C"
