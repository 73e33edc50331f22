// Rotary positions fused with the append to the K/V cache (spd_rope_init, spd_rope_append).
//
// Pair i of a head turns by the angle theta_i = pos * f_i:  (a, b) -> m (a cos - b sin, a sin + b cos),
// the pair being elements (i, i + r/2) (half layout) or (2i, 2i + 1) (interleaved) of the first r elements.
//
// The angle is formed in turns, in 64-bit fixed point: the plan holds f_i / 2 pi as a fraction of 2^64, so that the
// integer product pos * f wraps at whole turns by itself.  The range reduction is exact at any position and sign
// (error below |pos| 2^-65 turns) and needs none of the double-precision unit, which is slow here; the top 32 bits
// then go through sincospif.
//
// Bound by memory: every element is read once and written once (bf16, 8192 tokens of 32 + 2 x 8 heads x 128: 201 MB).
// A block takes whole tokens, so that the r/2 cosines and sines of a token are formed once, by its first threads, and
// serve all heads from shared memory; a thread's loads are issued before that.  Blocks are persistent over tokens: a
// thread reads its frequency once.
#include <cmath>
#include <cstdio>
#include <cstring>

#include "spd_internal.cuh"

namespace spd {
namespace rope {

constexpr int kThreads = 256;

struct Params {
  uint64_t turns[SPD_ROPE_MAX_PAIRS];
  float mscale;
  int rot, hd, hq, hkv, T;
  const void *q, *k, *v;
  long long qs, ks, vs, qos;
  void *qo, *kc, *vc;
  const int *pos, *slot, *seq;
  int n_seqs, max_seq;
};

// one rounding order for every path: aligned and unaligned rows give the same bits
__device__ __forceinline__ void turn(float& a, float& b, float2 c) {
  const float x = a, y = b;
  a = fmaf(x, c.x, -__fmul_rn(y, c.y));
  b = fmaf(x, c.y, __fmul_rn(y, c.x));
}

template <typename T, int N> struct alignas(sizeof(T) * N <= 16 ? sizeof(T) * N : 16) Pack { T v[N]; };

template <typename T, int N>
__device__ __forceinline__ void load_f(const T* p, float* f) {
  const Pack<T, N> x = *reinterpret_cast<const Pack<T, N>*>(p);
#pragma unroll
  for (int i = 0; i < N; ++i) f[i] = WTraits<T>::to_f(x.v[i]);
}
template <typename T, int N>
__device__ __forceinline__ void store_f(T* p, const float* f) {
  Pack<T, N> x;
#pragma unroll
  for (int i = 0; i < N; ++i) x.v[i] = WTraits<T>::from_f(f[i]);
  *reinterpret_cast<Pack<T, N>*>(p) = x;
}

// A unit is 2 * VE elements of one head: VE pairs while inside the rotated part.  In the half layout its two vectors of
// VE elements lie r/2 apart; elsewhere they are neighbours.  VE = 16 bytes of X, or 1 where strides, addresses or r/2 do
// not allow whole vectors.
template <typename X, typename C, int VE, bool INTER>
__global__ void __launch_bounds__(kThreads) rope_kernel(const __grid_constant__ Params p) {
  __shared__ float2 cs[2][SPD_ROPE_MAX_PAIRS];
  const int tid = threadIdx.x, half = p.rot >> 1;
  const int per_head = p.hd / (2 * VE), units = (p.hq + 2 * p.hkv) * per_head;
  const uint64_t f = tid < half ? p.turns[tid] : 0;
  constexpr int kB = VE == 1 ? 1 : 4;  // units a thread holds at once
  int buf = 0;
  for (int t = blockIdx.x; t < p.T; t += gridDim.x) {
    const int pos = p.pos[t];
    int slot = -1, sq = 0;
    if (p.slot) {
      slot = p.slot[t];
      sq = p.seq ? p.seq[t] : 0;
    }
    const bool keep = slot >= 0 && slot < p.max_seq && sq >= 0 && sq < p.n_seqs;
    const int n = keep ? units : p.hq * per_head;
    if (n == 0) continue;  // no barrier for this token: the buffers keep their turn
    for (int u0 = tid; u0 - tid < n; u0 += kThreads * kB) {
      float a[kB][VE], b[kB][VE];
      int e0[kB], e1[kB], head[kB];
#pragma unroll
      for (int j = 0; j < kB; ++j) {
        const int u = u0 + j * kThreads;
        if (u >= n) continue;
        head[j] = u / per_head;
        const int w = u - head[j] * per_head;
        if (!INTER && w * VE < half) {
          e0[j] = w * VE;
          e1[j] = e0[j] + half;
        } else {
          e0[j] = w * 2 * VE;
          e1[j] = e0[j] + VE;
        }
        const X* src;
        if (head[j] < p.hq) src = static_cast<const X*>(p.q) + t * p.qs + (long long)head[j] * p.hd;
        else if (head[j] < p.hq + p.hkv) src = static_cast<const X*>(p.k) + t * p.ks + (long long)(head[j] - p.hq) * p.hd;
        else {
          src = static_cast<const X*>(p.v) + t * p.vs + (long long)(head[j] - p.hq - p.hkv) * p.hd;
          e0[j] = w * 2 * VE;
          e1[j] = e0[j] + VE;
        }
        load_f<X, VE>(src + e0[j], a[j]);
        load_f<X, VE>(src + e1[j], b[j]);
      }
      if (u0 == tid) {
        if (tid < half) {
          const uint64_t angle = (uint64_t)(long long)pos * f;
          float s, c;
          sincospif((float)(int32_t)(angle >> 32) * 4.656612873077393e-10f, &s, &c);  // 2 x 2^-32
          cs[buf][tid] = make_float2(c * p.mscale, s * p.mscale);
        }
        __syncthreads();  // the other buffer's readers are past this one before it is written again
      }
#pragma unroll
      for (int j = 0; j < kB; ++j) {
        const int u = u0 + j * kThreads;
        if (u >= n) continue;
        if (head[j] < p.hq + p.hkv) {
          if (INTER && VE > 1) {
#pragma unroll
            for (int i = 0; i + 1 < VE; i += 2) {
              const int p0 = (e0[j] + i) >> 1, p1 = (e1[j] + i) >> 1;
              if (p0 < half) turn(a[j][i], a[j][i + 1], cs[buf][p0]);
              if (p1 < half) turn(b[j][i], b[j][i + 1], cs[buf][p1]);
            }
          } else {
            const int p0 = INTER ? e0[j] >> 1 : e0[j];  // first pair of the unit (a and b are its two sides)
            if (p0 < half) {
#pragma unroll
              for (int i = 0; i < VE; ++i) turn(a[j][i], b[j][i], cs[buf][p0 + i]);
            }
          }
        }
        if (head[j] < p.hq) {
          X* dst = static_cast<X*>(p.qo) + t * p.qos + (long long)head[j] * p.hd;
          store_f<X, VE>(dst + e0[j], a[j]);
          store_f<X, VE>(dst + e1[j], b[j]);
        } else {
          const bool is_v = head[j] >= p.hq + p.hkv;
          const int h = head[j] - p.hq - (is_v ? p.hkv : 0);
          C* dst = static_cast<C*>(is_v ? p.vc : p.kc) + (((long long)sq * p.hkv + h) * p.max_seq + slot) * p.hd;
          store_f<C, VE>(dst + e0[j], a[j]);
          store_f<C, VE>(dst + e1[j], b[j]);
        }
      }
    }
    buf ^= 1;
  }
}

template <typename X, typename C, int VE>
void launch(const Params& p, bool inter, int grid, cudaStream_t s) {
  if (inter) rope_kernel<X, C, VE, true><<<grid, kThreads, 0, s>>>(p);
  else rope_kernel<X, C, VE, false><<<grid, kThreads, 0, s>>>(p);
}

}  // namespace rope
}  // namespace spd

using namespace spd;

extern "C" int spd_rope_init(spd_rope* out, int32_t head_dim, int32_t rot_dim, int32_t layout, double theta,
                             int32_t scaling, double factor, int32_t original_context) {
  if (!out || head_dim < 16 || head_dim % 16 || head_dim > 2 * SPD_ROPE_MAX_PAIRS || rot_dim < 2 || rot_dim % 2 ||
      rot_dim > head_dim || (layout != SPD_ROPE_HALF && layout != SPD_ROPE_INTERLEAVED) || !(theta > 1.0) ||
      !std::isfinite(theta) || scaling < SPD_ROPE_NONE || scaling > SPD_ROPE_YARN)
    return spd_internal_fail(SPD_EINVAL, "spd_rope_init: bad arguments");
  if (scaling != SPD_ROPE_NONE && (!(factor >= 1.0) || !std::isfinite(factor)))
    return spd_internal_fail(SPD_EINVAL, "spd_rope_init: the factor of a scaled context is finite and at least 1");
  if (scaling == SPD_ROPE_YARN && original_context < 1)
    return spd_internal_fail(SPD_EINVAL, "spd_rope_init: YaRN needs the original context's length");
  const double r = rot_dim, pi = 3.14159265358979323846;
  if (scaling == SPD_ROPE_NTK && rot_dim > 2) theta *= std::pow(factor, r / (r - 2.0));
  memset(out, 0, sizeof(*out));
  out->head_dim = head_dim; out->rot_dim = rot_dim; out->layout = layout;
  out->mscale = scaling == SPD_ROPE_YARN ? (float)(0.1 * std::log(factor) + 1.0) : 1.0f;
  // YaRN's ramp over the pairs: those that turn more than 32 times within the original context stay, those that turn
  // less than once are interpolated (beta_fast = 32, beta_slow = 1)
  double lo = 0, hi = 0;
  if (scaling == SPD_ROPE_YARN) {
    const double top = rot_dim / 2 - 1;
    lo = std::floor(r * std::log(original_context / (2 * pi * 32.0)) / (2 * std::log(theta)));
    hi = std::ceil(r * std::log(original_context / (2 * pi)) / (2 * std::log(theta)));
    lo = lo < 0 ? 0 : lo > top ? top : lo;
    hi = hi < 0 ? 0 : hi > top ? top : hi;
  }
  for (int i = 0; i < rot_dim / 2; ++i) {
    double f = std::pow(theta, -2.0 * i / r);
    if (scaling == SPD_ROPE_LINEAR) f /= factor;
    if (scaling == SPD_ROPE_YARN) {
      double g = (i - lo) / (hi - lo > 0.001 ? hi - lo : 0.001);
      g = 1.0 - (g < 0 ? 0 : g > 1 ? 1 : g);
      f = f / factor * (1.0 - g) + f * g;
    }
    // f <= 1 radian, so f / 2 pi < 1/2 turn; 11 bits of the product lie below a double's last place
    out->turns[i] = (uint64_t)std::ldexp(f / (2.0 * pi), 64);
  }
  return SPD_OK;
}

extern "C" int spd_rope_append(const spd_rope* rope, const void* q, int64_t q_stride, void* q_out, int64_t q_out_stride,
                               const void* k, int64_t k_stride, const void* v, int64_t v_stride, int32_t x_dtype,
                               const int32_t* pos, int32_t T, int32_t n_heads, int32_t n_kv_heads, void* k_cache,
                               void* v_cache, int32_t cache_dtype, const int32_t* slot, const int32_t* seq, int32_t n_seqs,
                               int32_t max_seq, void* cuda_stream) {
  auto bad = [](const char* m) { return spd_internal_fail(SPD_EINVAL, m); };
  if (!rope || rope->head_dim < 16 || rope->head_dim % 16 || rope->head_dim > 2 * SPD_ROPE_MAX_PAIRS || rope->rot_dim < 2 ||
      rope->rot_dim % 2 || rope->rot_dim > rope->head_dim ||
      (rope->layout != SPD_ROPE_HALF && rope->layout != SPD_ROPE_INTERLEAVED))
    return bad("spd_rope_append: the plan is not one of spd_rope_init");
  if ((x_dtype != SPD_DTYPE_F32 && x_dtype != SPD_DTYPE_BF16) || (cache_dtype != SPD_DTYPE_F32 && cache_dtype != SPD_DTYPE_BF16))
    return bad("spd_rope_append: bad dtype");
  if (T < 0 || n_heads < 0 || n_kv_heads < 0 || n_heads > 65536 || n_kv_heads > 65536 || n_heads + n_kv_heads < 1)
    return bad("spd_rope_append: bad sizes");
  if (T == 0) return SPD_OK;
  const int hd = rope->head_dim;
  const long long qw = (long long)n_heads * hd, kw = (long long)n_kv_heads * hd;
  if (!pos || (n_heads && (!q || !q_out))) return bad("spd_rope_append: NULL pointer");
  if (n_heads && (q_stride < qw || q_out_stride < qw)) return bad("spd_rope_append: a row stride is below the row's length");
  if (n_heads && q == q_out && q_stride != q_out_stride) return bad("spd_rope_append: in place needs equal strides");
  if (n_kv_heads) {
    if (!k || !v || !k_cache || !v_cache || !slot) return bad("spd_rope_append: NULL pointer");
    if (k_stride < kw || v_stride < kw) return bad("spd_rope_append: a row stride is below the row's length");
    if (n_seqs < 1 || max_seq < 1) return bad("spd_rope_append: bad cache sizes");
  }
  rope::Params p;
  memset(&p, 0, sizeof(p));
  memcpy(p.turns, rope->turns, sizeof(p.turns));
  p.mscale = rope->mscale; p.rot = rope->rot_dim; p.hd = hd; p.hq = n_heads; p.hkv = n_kv_heads; p.T = T;
  p.q = q; p.k = k; p.v = v; p.qs = q_stride; p.ks = k_stride; p.vs = v_stride; p.qos = q_out_stride;
  p.qo = q_out; p.kc = k_cache; p.vc = v_cache; p.pos = pos; p.slot = n_kv_heads ? slot : nullptr;
  p.seq = n_kv_heads ? seq : nullptr; p.n_seqs = n_seqs; p.max_seq = max_seq;
  const bool xf = x_dtype == SPD_DTYPE_F32, cf = cache_dtype == SPD_DTYPE_F32, inter = rope->layout == SPD_ROPE_INTERLEAVED;
  const int ve = xf ? 4 : 8;
  // whole vectors: every row starts on 16 bytes, and in the half layout so does the second side of a pair
  bool vec = inter || (rope->rot_dim / 2) % ve == 0;
  auto ok = [](const void* ptr, long long stride, int n) { return reinterpret_cast<uintptr_t>(ptr) % 16 == 0 && stride % n == 0; };
  if (n_heads) vec = vec && ok(q, q_stride, ve) && ok(q_out, q_out_stride, ve);
  if (n_kv_heads) vec = vec && ok(k, k_stride, ve) && ok(v, v_stride, ve) && ok(k_cache, 0, 1) && ok(v_cache, 0, 1);
  const int grid = T < 8 * num_sms() ? T : 8 * num_sms();
  cudaStream_t s = reinterpret_cast<cudaStream_t>(cuda_stream);
  cudaGetLastError();
#define SPD_ROPE_GO(X, C, VE) rope::launch<X, C, VE>(p, inter, grid, s)
  if (xf && cf) { if (vec) SPD_ROPE_GO(float, float, 4); else SPD_ROPE_GO(float, float, 1); }
  else if (xf) { if (vec) SPD_ROPE_GO(float, __nv_bfloat16, 4); else SPD_ROPE_GO(float, __nv_bfloat16, 1); }
  else if (cf) { if (vec) SPD_ROPE_GO(__nv_bfloat16, float, 8); else SPD_ROPE_GO(__nv_bfloat16, float, 1); }
  else { if (vec) SPD_ROPE_GO(__nv_bfloat16, __nv_bfloat16, 8); else SPD_ROPE_GO(__nv_bfloat16, __nv_bfloat16, 1); }
#undef SPD_ROPE_GO
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) {
    char msg[160];
    snprintf(msg, sizeof(msg), "spd_rope_append: launch: %s", cudaGetErrorString(e));
    return spd_internal_fail(SPD_ECUDA, msg);
  }
  return SPD_OK;
}
