// Decode attention of a batch that shares a prefix (spd_shared_prefix_attention).
//
//   out[b][h] = sum_j p_j v_j / sum_j p_j,  p_j = exp(q[b][h] . k_j / sqrt(hd) - m),  over the shared keys 0..P-1 and
// the sequence's own keys 0..len-1: the softmax is taken in one pass with a running maximum and sum, over parts of the
// keys, and the parts (O, m, l) are joined as  O = sum_i O_i e^(m_i - m),  l = sum_i l_i e^(m_i - m).
//
// rows kernel: one block per (sequence, kv head, up to 8 query heads of its group).  Its warps take 32 keys in turn and
// work on mma.sync m16n8k16: S^T = K Q^T (16 keys x 8 heads), then O^T += V^T P^T (16 head elements x 8 heads).  K and V go
// from global memory straight into operand registers: the order of the head elements in a dot product is free, so a lane
// reads 16 consecutive bytes; V's pairs of keys are put together with byte permutes.  fp32 queries and their
// probabilities enter as three bf16 terms (exact), bf16 queries' probabilities as one (rounded to bf16, 2^-9 relative,
// like the output).  Statistics and sums are fp32.
#include <cmath>
#include <cstdio>
#include <cstring>

#include "spd_internal.cuh"

namespace spd {
namespace spa {

constexpr int kWarps = 8;
constexpr int kThreads = 32 * kWarps;
constexpr int kHeads = 8;  // query heads of a block (the mma's 8 columns)
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

struct Params {
  const void* q;
  const __nv_bfloat16 *pk, *pv, *kc, *vc;
  const int* lens;
  void* out;
  float* lse;
  float* part;
  long long prefix_cap, max_seq;
  int P, B, hq, hkv, gq, hblocks;
  float scale_log2;  // log2(e) / sqrt(hd)
};

__device__ __forceinline__ void mma16816(float* c, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
               : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
               : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t movm(uint32_t x) {  // transpose of an 8 x 8 matrix of 16-bit elements
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// the next bf16 term of a pair; a and b keep the rest
__device__ __forceinline__ uint32_t take_pair(float& a, float& b) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  const float2 f = __bfloat1622float2(h);
  a = fabsf(f.x) == INFINITY ? 0.f : a - f.x;
  b = fabsf(f.y) == INFINITY ? 0.f : b - f.y;
  return *reinterpret_cast<const uint32_t*>(&h);
}

// One 16-key step of the keys at `k0`, `n` of them in range (the others repeat the last one and weigh nothing).
template <int HD> struct KeyRegs { uint4 v[2][HD / 32]; };

template <int HD, int TERMS>
__global__ void __launch_bounds__(kThreads) rows_kernel(const __grid_constant__ Params p) {
  constexpr int KI = HD / 32;  // 16-byte pieces of a key a lane reads
  extern __shared__ __align__(16) unsigned char smem[];
  float* s_o = reinterpret_cast<float*>(smem);  // [warp][head][HD]
  __shared__ float s_m[kWarps][kHeads], s_l[kWarps][kHeads];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
  const int hb = blockIdx.x % p.hblocks, kh = blockIdx.x / p.hblocks % p.hkv, b = blockIdx.x / p.hblocks / p.hkv;
  const int h0 = kh * p.gq + hb * kHeads, nh = min(kHeads, p.gq - hb * kHeads);
  const int len = p.max_seq > 0 ? p.lens[b] : 0;
  const bool bad = len < 0 || len > p.max_seq;

  // Q^T as the second operand: head g, elements 32 i + 8 t + 4 s + {0, 1}, {2, 3}
  uint32_t qb[TERMS][KI][2][2];
#pragma unroll
  for (int i = 0; i < KI; ++i) {
    float x[8];
    const long long at = ((long long)b * p.hq + h0 + g) * HD + 32 * i + 8 * t;
#pragma unroll
    for (int j = 0; j < 8; ++j)
      x[j] = g >= nh ? 0.f
                     : TERMS > 1 ? static_cast<const float*>(p.q)[at + j] : __bfloat162float(static_cast<const __nv_bfloat16*>(p.q)[at + j]);
#pragma unroll
    for (int e = 0; e < TERMS; ++e)
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        qb[e][i][s][0] = take_pair(x[4 * s], x[4 * s + 1]);
        qb[e][i][s][1] = take_pair(x[4 * s + 2], x[4 * s + 3]);
      }
  }
  float o[HD / 16][4];
#pragma unroll
  for (int e = 0; e < HD / 16; ++e) o[e][0] = o[e][1] = o[e][2] = o[e][3] = 0.f;
  float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};  // heads 2 t, 2 t + 1

  const int nkeys = bad ? 0 : p.P + len;
  for (int key0 = warp * 16; key0 < nkeys; key0 += kWarps * 16) {
    // keys of this lane: as rows g, g + 8 of K and as 2 t, 2 t + 1, 2 t + 8, 2 t + 9 of V
    auto row = [&](const __nv_bfloat16* pre, const __nv_bfloat16* own, int key) {
      key = min(key, nkeys - 1);
      return key < p.P ? pre + ((long long)kh * p.prefix_cap + key) * HD
                       : own + (((long long)b * p.hkv + kh) * p.max_seq + (key - p.P)) * HD;
    };
    float s[4] = {0.f, 0.f, 0.f, 0.f};
    const __nv_bfloat16 *ka = row(p.pk, p.kc, key0 + g) + 8 * t, *kb = row(p.pk, p.kc, key0 + g + 8) + 8 * t;
#pragma unroll
    for (int i = 0; i < KI; ++i) {
      const uint4 a = *reinterpret_cast<const uint4*>(ka + 32 * i), c = *reinterpret_cast<const uint4*>(kb + 32 * i);
#pragma unroll
      for (int e = TERMS - 1; e >= 0; --e) {
        mma16816(s, a.x, c.x, a.y, c.y, qb[e][i][0][0], qb[e][i][0][1]);
        mma16816(s, a.z, c.z, a.w, c.w, qb[e][i][1][0], qb[e][i][1][1]);
      }
    }
    // s: (key g, heads 2t, 2t+1), (key g + 8, heads 2t, 2t+1)
    float al[2];
    float pr[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) s[j] = key0 + g + 8 * (j >> 1) < nkeys ? s[j] * p.scale_log2 : -INFINITY;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      float mx = fmaxf(s[j], s[j + 2]);
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 4));
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 8));
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 16));
      const float mn = fmaxf(m[j], mx), mu = mn == -INFINITY ? 0.f : mn;
      al[j] = ex2(m[j] - mu);
      m[j] = mn;
      pr[j] = ex2(s[j] - mu);
      pr[j + 2] = ex2(s[j + 2] - mu);
      l[j] = l[j] * al[j] + pr[j] + pr[j + 2];
    }
#pragma unroll
    for (int e = 0; e < HD / 16; ++e) {
      o[e][0] *= al[0]; o[e][1] *= al[1]; o[e][2] *= al[0]; o[e][3] *= al[1];
    }
    uint32_t pb[TERMS][2];
#pragma unroll
    for (int e = 0; e < TERMS; ++e) {
      pb[e][0] = movm(take_pair(pr[0], pr[1]));
      pb[e][1] = movm(take_pair(pr[2], pr[3]));
    }
    const __nv_bfloat16* vr[4] = {row(p.pv, p.vc, key0 + 2 * t), row(p.pv, p.vc, key0 + 2 * t + 1), row(p.pv, p.vc, key0 + 2 * t + 8),
                                  row(p.pv, p.vc, key0 + 2 * t + 9)};
    // element e of this lane's two pieces of 8: rows g -> g * 8 + e and g + 8 -> 64 + g * 8 + e (hd 128), or
    // g * 8 + 2 e and g * 8 + 2 e + 1 (hd 64)
    uint32_t w[4][HD / 16];
#pragma unroll
    for (int k = 0; k < 4; ++k)
#pragma unroll
      for (int c = 0; c < HD / 64; ++c) {
        const uint4 x = *reinterpret_cast<const uint4*>(vr[k] + 64 * c + 8 * g);
        w[k][4 * c] = x.x; w[k][4 * c + 1] = x.y; w[k][4 * c + 2] = x.z; w[k][4 * c + 3] = x.w;
      }
    auto take = [&](int k, int el) {  // elements el of keys k and k + 1
      return __byte_perm(w[k][el >> 1], w[k + 1][el >> 1], el & 1 ? 0x7632 : 0x5410);
    };
#pragma unroll
    for (int e = 0; e < HD / 16; ++e) {
      const int lo = HD == 128 ? e : 2 * e, hi = HD == 128 ? e + 8 : 2 * e + 1;
      const uint32_t a0 = take(0, lo), a1 = take(0, hi), a2 = take(2, lo), a3 = take(2, hi);
#pragma unroll
      for (int x = TERMS - 1; x >= 0; --x) mma16816(o[e], a0, a1, a2, a3, pb[x][0], pb[x][1]);
    }
  }
  // this warp's part
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    l[j] += __shfl_xor_sync(0xffffffffu, l[j], 4);
    l[j] += __shfl_xor_sync(0xffffffffu, l[j], 8);
    l[j] += __shfl_xor_sync(0xffffffffu, l[j], 16);
    if (g == 0) {
      s_m[warp][2 * t + j] = m[j];
      s_l[warp][2 * t + j] = l[j];
    }
  }
#pragma unroll
  for (int e = 0; e < HD / 16; ++e) {
    const int lo = HD == 128 ? g * 8 + e : g * 8 + 2 * e, hi = HD == 128 ? 64 + g * 8 + e : g * 8 + 2 * e + 1;
    float* d0 = s_o + (warp * kHeads + 2 * t) * HD;
    d0[lo] = o[e][0]; d0[HD + lo] = o[e][1]; d0[hi] = o[e][2]; d0[HD + hi] = o[e][3];
  }
  __syncthreads();
  for (int i = tid; i < nh * HD; i += kThreads) {
    const int h = i / HD, d = i % HD;
    float mx = -INFINITY;
    for (int w = 0; w < kWarps; ++w) mx = fmaxf(mx, s_m[w][h]);
    const float mu = mx == -INFINITY ? 0.f : mx;
    float lt = 0.f, ot = 0.f;
    for (int w = 0; w < kWarps; ++w) {
      const float a = ex2(s_m[w][h] - mu);
      lt += s_l[w][h] * a;
      ot += s_o[(w * kHeads + h) * HD + d] * a;
    }
    float y = bad ? NAN : nkeys == 0 ? 0.f : ot / lt;
    const long long at = ((long long)b * p.hq + h0 + h) * HD + d;
    if (TERMS > 1) static_cast<float*>(p.out)[at] = y;
    else static_cast<__nv_bfloat16*>(p.out)[at] = __float2bfloat16_rn(y);
    if (d == 0 && p.lse) p.lse[(long long)b * p.hq + h0 + h] = bad ? NAN : nkeys == 0 ? -INFINITY : mx * kLn2 + logf(lt);
  }
}

template <int HD, int TERMS>
cudaError_t launch_rows(const Params& p, cudaStream_t s) {
  const size_t smem = (size_t)kWarps * kHeads * HD * 4;
  rows_kernel<HD, TERMS><<<(unsigned)(p.B * p.hkv * p.hblocks), kThreads, smem, s>>>(p);
  return cudaGetLastError();
}

bool sizes_ok(int B, int hq, int hkv, int hd, int P) {
  return B >= 1 && B <= 4096 && hkv >= 1 && hq >= 1 && hq <= 1024 && hq % hkv == 0 && (hd == 64 || hd == 128) && P >= 0;
}

}  // namespace spa
}  // namespace spd

using namespace spd;

extern "C" size_t spd_shared_prefix_attention_workspace_bytes(int32_t B, int32_t n_heads, int32_t n_kv_heads, int32_t head_dim,
                                                              int32_t prefix_len) {
  if (!spa::sizes_ok(B, n_heads, n_kv_heads, head_dim, prefix_len)) return 0;
  return 16;
}

extern "C" int spd_shared_prefix_attention(const void* q, int32_t q_dtype, const void* prefix_k, const void* prefix_v,
                                           int32_t prefix_len, int32_t prefix_cap, const void* k_cache, const void* v_cache,
                                           const int32_t* lens, int32_t max_seq, int32_t B, int32_t n_heads, int32_t n_kv_heads,
                                           int32_t head_dim, void* out, float* lse, void* workspace, size_t workspace_bytes,
                                           void* cuda_stream) {
  auto bad = [](const char* m) { return spd_internal_fail(SPD_EINVAL, m); };
  auto al = [](const void* ptr, size_t n) { return reinterpret_cast<uintptr_t>(ptr) % n == 0; };
  if (B < 0 || !spa::sizes_ok(B > 0 ? B : 1, n_heads, n_kv_heads, head_dim, prefix_len) || prefix_cap < prefix_len || max_seq < 0 ||
      (q_dtype != SPD_DTYPE_F32 && q_dtype != SPD_DTYPE_BF16))
    return bad("spd_shared_prefix_attention: bad sizes or dtype");
  if (B == 0) return SPD_OK;
  if (!q || !out || !workspace || (prefix_len && (!prefix_k || !prefix_v)) || (max_seq && (!k_cache || !v_cache || !lens)))
    return bad("spd_shared_prefix_attention: NULL pointer");
  if (!al(q, 16) || !al(out, 16) || !al(workspace, 16) || !al(prefix_k, 16) || !al(prefix_v, 16) || !al(k_cache, 16) ||
      !al(v_cache, 16) || !al(lens, 4) || !al(lse, 4))
    return bad("spd_shared_prefix_attention: unaligned pointer");
  if (workspace_bytes < spd_shared_prefix_attention_workspace_bytes(B, n_heads, n_kv_heads, head_dim, prefix_len))
    return bad("spd_shared_prefix_attention: workspace too small");
  spa::Params p;
  memset(&p, 0, sizeof(p));
  p.q = q;
  p.pk = static_cast<const __nv_bfloat16*>(prefix_k); p.pv = static_cast<const __nv_bfloat16*>(prefix_v);
  p.kc = static_cast<const __nv_bfloat16*>(k_cache); p.vc = static_cast<const __nv_bfloat16*>(v_cache);
  p.lens = lens; p.out = out; p.lse = lse; p.part = static_cast<float*>(workspace);
  p.prefix_cap = prefix_cap; p.max_seq = max_seq; p.P = prefix_len; p.B = B; p.hq = n_heads; p.hkv = n_kv_heads;
  p.gq = n_heads / n_kv_heads;
  p.hblocks = (p.gq + spa::kHeads - 1) / spa::kHeads;
  p.scale_log2 = spa::kLog2e / std::sqrt((float)head_dim);
  cudaStream_t s = reinterpret_cast<cudaStream_t>(cuda_stream);
  cudaGetLastError();
  cudaError_t e;
  if (head_dim == 128) e = q_dtype == SPD_DTYPE_F32 ? spa::launch_rows<128, 3>(p, s) : spa::launch_rows<128, 1>(p, s);
  else e = q_dtype == SPD_DTYPE_F32 ? spa::launch_rows<64, 3>(p, s) : spa::launch_rows<64, 1>(p, s);
  if (e != cudaSuccess) {
    char msg[160];
    snprintf(msg, sizeof(msg), "spd_shared_prefix_attention: launch: %s", cudaGetErrorString(e));
    return spd_internal_fail(SPD_ECUDA, msg);
  }
  return SPD_OK;
}
