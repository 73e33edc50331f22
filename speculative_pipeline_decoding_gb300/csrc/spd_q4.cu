// Grouped matrix-vector products with 4-bit weights and group scales (spd_q4_quantize, spd_q4_pack, spd_q4_gemv).
//
//   y[m][r] = sum over groups of columns  scale[r][group] * sum_{c in group} (code[r][c] - zero[r][group]) x[m][c]
//
// The inner sums run on mma.sync m16n8k16 (bf16 operands, fp32 sums): a code less its zero point is a small whole
// number, exact in bf16, so the weights lose nothing; the scale is applied to the group's fp32 sum.  fp32 vectors enter
// as three bf16 terms of 8 bits each (x = t0 + t1 + t2 exactly, by truncation), as three columns of the 8-wide operand.
//
// Packed layout: one record for each 16 rows (tile) and 128 columns (block), records of a tile in a row:
//   1024 B codes   [h 0..1][lane 0..31][word 0..3]: word w of lane (g = lane / 4, t = lane % 4) holds the 8 codes of
//                  row g + 8 h, columns 32 w + 8 t .. + 7, lowest column in the lowest bits
//   scales         [128 / group][16 rows], scale_dtype
//   zeros          [128 / group][16 rows] bf16 of 128 + zero (only with zeros)
// so that a warp reads a record in two 16-byte loads a lane, already in the order of the mma's A operand: the four bf16
// pairs of a word are (code i, code i + 4), i = 0..3, taken as (w >> 4 i) & 0x000f000f | 0x43004300 = 128 + code.  Columns
// beyond `cols` and rows beyond `rows` hold code = zero and scale 0.
#include <cmath>
#include <cstdio>
#include <cstring>
#include <mutex>

#include "spd_internal.cuh"

namespace spd {
namespace q4 {

constexpr int kWarps = 8;
constexpr int kThreads = 32 * kWarps;
constexpr int kMaxCols = 32768;
constexpr int kMaxM = 32;

inline size_t record_bytes(int group, int scale_dtype, int has_zeros) {
  const int ng = 128 / group;
  return 1024 + (size_t)ng * 16 * (scale_dtype == SPD_DTYPE_F32 ? 4 : 2) + (has_zeros ? (size_t)ng * 32 : 0);
}

// ---------------------------------------------------------------------------------------------
// quantise and pack
// ---------------------------------------------------------------------------------------------
template <typename T>
__global__ void quantize_kernel(const T* w, long long ngroups, int group, int s_f32, uint8_t* codes, void* scales, uint8_t* zeros) {
  // one warp per group of 32, 64 or 128 columns; lane l holds columns l * n .. + n - 1
  const long long gi = (long long)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5);
  if (gi >= ngroups) return;
  const int lane = threadIdx.x & 31, n = group >> 5;
  float v[4], hi = 0.f, lo = 0.f;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (i < n) {
      v[i] = WTraits<T>::to_f(w[gi * group + lane * n + i]);
      hi = fmaxf(hi, v[i]);
      lo = fminf(lo, v[i]);
    }
#pragma unroll
  for (int o = 16; o; o >>= 1) {
    hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, o));
    lo = fminf(lo, __shfl_xor_sync(0xffffffffu, lo, o));
  }
  float s = zeros ? __fdiv_rn(hi - lo, 15.f) : __fdiv_rn(fmaxf(hi, -lo), 7.f);
  if (!s_f32) s = __bfloat162float(__float2bfloat16_rn(s));
  const float z = zeros ? (s > 0.f ? fminf(fmaxf(rintf(__fdiv_rn(-lo, s)), 0.f), 15.f) : 0.f) : 8.f;
  uint32_t code[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    code[i] = i < n ? (uint32_t)fminf(fmaxf((s > 0.f ? rintf(__fdiv_rn(v[i], s)) : 0.f) + z, 0.f), 15.f) : 0u;
  uint8_t* out = codes + gi * (group >> 1);
  if (n == 1) {
    const uint32_t up = __shfl_down_sync(0xffffffffu, code[0], 1);
    if (!(lane & 1)) out[lane >> 1] = (uint8_t)(code[0] | (up << 4));
  } else {
    out[lane * (n >> 1)] = (uint8_t)(code[0] | (code[1] << 4));
    if (n == 4) out[lane * 2 + 1] = (uint8_t)(code[2] | (code[3] << 4));
  }
  if (lane == 0) {
    if (s_f32) static_cast<float*>(scales)[gi] = s;
    else static_cast<__nv_bfloat16*>(scales)[gi] = __float2bfloat16_rn(s);
    if (zeros) zeros[gi] = (uint8_t)z;
  }
}

// one warp per record
__global__ void pack_kernel(const uint8_t* codes, const void* scales, const uint8_t* zeros, int rows, int cols, int group, int s_f32,
                            int nkb, long long nrec, unsigned char* packed, int rec) {
  const long long ri = (long long)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5);
  if (ri >= nrec) return;
  const int lane = threadIdx.x & 31, tile = (int)(ri / nkb), kb = (int)(ri % nkb), per_row = cols / group, ng = 128 / group;
  unsigned char* out = packed + ri * rec;
  for (int h = 0; h < 2; ++h) {
    const int r = tile * 16 + (lane >> 2) + 8 * h;
    uint32_t w[4];
    for (int i = 0; i < 4; ++i) {
      const int c = kb * 128 + 32 * i + 8 * (lane & 3);
      w[i] = 0x88888888u;
      if (r < rows && c < cols) {  // whole words: cols is a multiple of 32
        const uint8_t* src = codes + (long long)r * (cols >> 1) + (c >> 1);
        w[i] = (uint32_t)src[0] | (uint32_t)src[1] << 8 | (uint32_t)src[2] << 16 | (uint32_t)src[3] << 24;
      }
    }
    *reinterpret_cast<uint4*>(out + h * 512 + lane * 16) = make_uint4(w[0], w[1], w[2], w[3]);
  }
  for (int i = lane; i < ng * 16; i += 32) {
    const int r = tile * 16 + (i & 15), gc = kb * ng + (i >> 4);
    const bool in = r < rows && gc < per_row;
    const long long at = (long long)r * per_row + gc;
    if (s_f32) reinterpret_cast<float*>(out + 1024)[i] = in ? static_cast<const float*>(scales)[at] : 0.f;
    else reinterpret_cast<__nv_bfloat16*>(out + 1024)[i] = in ? static_cast<const __nv_bfloat16*>(scales)[at] : __nv_bfloat16(0.f);
    if (zeros)
      reinterpret_cast<__nv_bfloat16*>(out + 1024 + ng * 16 * (s_f32 ? 4 : 2))[i] = __float2bfloat16_rn(128.f + (in ? zeros[at] : 8));
  }
}

// ---------------------------------------------------------------------------------------------
// products
// ---------------------------------------------------------------------------------------------
struct Group {
  const unsigned char* w;
  const void* x;
  void* y;
  long long xs, ys;
  int rows, tile0;  // first tile of the group
};
struct Params {
  Group g[kMaxExplicit];
  int G, M, cols, nkb, tiles;
  int gw;            // 32-column words of a group: 1, 2 or 4
  int rec, s_f32, has_z, x_f32;
  int terms, mb;     // bf16 terms of a vector, vectors of a block
  const float* nw;
  float eps;
};

__device__ __forceinline__ void mma16816(float* c, const uint32_t* a, uint32_t b0, uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
               : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
               : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// pair i of a word, less its zero point: (code i - z, code i + 4 - z) in bf16, exact
__device__ __forceinline__ uint32_t pair(uint32_t w, int i, __nv_bfloat162 z) {
  uint32_t u = ((w >> (4 * i)) & 0x000f000fu) | 0x43004300u;
  __nv_bfloat162 v = __hsub2(*reinterpret_cast<__nv_bfloat162*>(&u), z);
  return *reinterpret_cast<uint32_t*>(&v);
}
// the next bf16 term of v by truncation (no overflow to infinity); v keeps the rest
__device__ __forceinline__ uint32_t take_term(float& v) {
  const uint32_t u = (__float_as_uint(v) & 0xffff0000u) | (v != v ? 0x400000u : 0u);  // a NaN stays one
  const float h = __uint_as_float(u);
  v = fabsf(h) == INFINITY ? 0.f : v - h;  // an infinity's rest is not NaN
  return u >> 16;
}

// Block: 8 warps share a tile of 16 rows, each taking a run of its 128-column blocks; sums of the warps meet in shared
// memory.  Blocks are persistent over tiles; the vectors are split into terms once per block, into shared memory as
// [column block][word][operand column][t] of 16 bytes (two mma steps of a lane).
template <int NT>
__global__ void __launch_bounds__(kThreads) gemv_kernel(const __grid_constant__ Params p) {
  extern __shared__ __align__(16) unsigned char smem[];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g4 = lane >> 2, t4 = lane & 3;
  const int m0 = blockIdx.y * p.mb, mb = min(p.mb, p.M - m0), ncol = mb * p.terms;
  uint4* xs = reinterpret_cast<uint4*>(smem);
  float* part = reinterpret_cast<float*>(smem + (size_t)p.nkb * 4 * p.mb * p.terms * 64);  // [2][warp][16][NT * 8 + 1]
  __shared__ float s_ss[kMaxM];
  constexpr int PC = NT * 8 + 1;
  const int kb0 = warp * p.nkb / kWarps, kb1 = (warp + 1) * p.nkb / kWarps;
  const void* staged = nullptr;
  int parity = 0;
  for (int tile = blockIdx.x; tile < p.tiles; tile += gridDim.x, parity ^= 1) {
    int gi = 0;
    while (gi + 1 < p.G && tile >= p.g[gi + 1].tile0) ++gi;
    const Group& G = p.g[gi];
    if (G.x != staged) {
      __syncthreads();
      if (tid < kMaxM) s_ss[tid] = 0.f;
      __syncthreads();
      // 8 consecutive columns of one vector a thread
      const int per = p.nkb * 16;
      for (int m = warp; m < mb; m += kWarps) {
        float ss = 0.f;
        for (int i = lane; i < per; i += 32) {
          const int c = i * 8;
          float v[8];
          for (int j = 0; j < 8; ++j) v[j] = 0.f;
          if (c < p.cols) {
            const long long at = (long long)(m0 + m) * G.xs + c;
            for (int j = 0; j < 8; ++j)
              v[j] = p.x_f32 ? static_cast<const float*>(G.x)[at + j] : __bfloat162float(static_cast<const __nv_bfloat16*>(G.x)[at + j]);
            if (p.nw)
              for (int j = 0; j < 8; ++j) {
                ss += v[j] * v[j];
                v[j] *= p.nw[c + j];
              }
          }
          for (int e = 0; e < p.terms; ++e) {
            uint32_t b[8];
            for (int j = 0; j < 8; ++j) b[j] = take_term(v[j]);
            // columns 8 i .. = block i / 16, word (i % 16) / 4, t = i % 4; pairs (j, j + 4)
            xs[((i >> 2) * ncol + m * p.terms + e) * 4 + (i & 3)] =
                make_uint4(b[0] | b[4] << 16, b[1] | b[5] << 16, b[2] | b[6] << 16, b[3] | b[7] << 16);
          }
        }
        if (p.nw) {
          for (int o = 16; o; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
          if (lane == 0) s_ss[m] = rsqrtf(ss / p.cols + p.eps);
        }
      }
      __syncthreads();
      staged = G.x;
    }
    float tot[NT][4], acc[NT][4];
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int i = 0; i < 4; ++i) tot[n][i] = acc[n][i] = 0.f;
    const unsigned char* base = G.w + (size_t)(tile - G.tile0) * p.nkb * p.rec;
    const int ng = 4 / p.gw, soff = 1024, zoff = 1024 + ng * 16 * (p.s_f32 ? 4 : 2);
    for (int kb = kb0; kb < kb1; ++kb) {
      const unsigned char* r = base + (size_t)kb * p.rec;
      const uint4 a0 = __ldcs(reinterpret_cast<const uint4*>(r) + lane), a1 = __ldcs(reinterpret_cast<const uint4*>(r + 512) + lane);
      const uint32_t w0[4] = {a0.x, a0.y, a0.z, a0.w}, w1[4] = {a1.x, a1.y, a1.z, a1.w};
      __nv_bfloat162 z0 = __float2bfloat162_rn(136.f), z1 = z0;
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        const int gr = w / p.gw;
        if (p.has_z && w % p.gw == 0) {
          const __nv_bfloat16* z = reinterpret_cast<const __nv_bfloat16*>(r + zoff) + gr * 16;
          z0 = __bfloat162bfloat162(z[g4]);
          z1 = __bfloat162bfloat162(z[g4 + 8]);
        }
        uint4 b[NT];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          const int col = n * 8 + g4;
          b[n] = col < ncol ? xs[((kb * 4 + w) * ncol + col) * 4 + t4] : make_uint4(0, 0, 0, 0);
        }
        uint32_t a[4];
        a[0] = pair(w0[w], 0, z0); a[1] = pair(w1[w], 0, z1); a[2] = pair(w0[w], 1, z0); a[3] = pair(w1[w], 1, z1);
#pragma unroll
        for (int n = 0; n < NT; ++n) mma16816(acc[n], a, b[n].x, b[n].y);
        a[0] = pair(w0[w], 2, z0); a[1] = pair(w1[w], 2, z1); a[2] = pair(w0[w], 3, z0); a[3] = pair(w1[w], 3, z1);
#pragma unroll
        for (int n = 0; n < NT; ++n) mma16816(acc[n], a, b[n].z, b[n].w);
        if ((w + 1) % p.gw == 0) {
          float s0, s1;
          if (p.s_f32) {
            const float* s = reinterpret_cast<const float*>(r + soff) + gr * 16;
            s0 = s[g4]; s1 = s[g4 + 8];
          } else {
            const __nv_bfloat16* s = reinterpret_cast<const __nv_bfloat16*>(r + soff) + gr * 16;
            s0 = __bfloat162float(s[g4]); s1 = __bfloat162float(s[g4 + 8]);
          }
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            tot[n][0] += s0 * acc[n][0]; tot[n][1] += s0 * acc[n][1];
            tot[n][2] += s1 * acc[n][2]; tot[n][3] += s1 * acc[n][3];
            acc[n][0] = acc[n][1] = acc[n][2] = acc[n][3] = 0.f;
          }
        }
      }
    }
    float* mine = part + (size_t)(parity * kWarps + warp) * 16 * PC;
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      mine[g4 * PC + n * 8 + 2 * t4] = tot[n][0];
      mine[g4 * PC + n * 8 + 2 * t4 + 1] = tot[n][1];
      mine[(g4 + 8) * PC + n * 8 + 2 * t4] = tot[n][2];
      mine[(g4 + 8) * PC + n * 8 + 2 * t4 + 1] = tot[n][3];
    }
    __syncthreads();
    for (int o = tid; o < 16 * mb; o += kThreads) {
      const int row = o & 15, m = o >> 4, r = (tile - G.tile0) * 16 + row;
      if (r >= G.rows) continue;
      float y = 0.f;
      for (int w = 0; w < kWarps; ++w)
        for (int e = p.terms - 1; e >= 0; --e) y += part[((size_t)(parity * kWarps + w) * 16 + row) * PC + m * p.terms + e];
      if (p.nw) y *= s_ss[m];
      const long long at = (long long)(m0 + m) * G.ys + r;
      if (p.x_f32) static_cast<float*>(G.y)[at] = y;
      else static_cast<__nv_bfloat16*>(G.y)[at] = __float2bfloat16_rn(y);
    }
  }
}

size_t gemv_smem(int nkb, int mb, int terms, int nt) {
  return (size_t)nkb * 4 * mb * terms * 64 + (size_t)2 * kWarps * 16 * (nt * 8 + 1) * 4;
}

template <int NT>
cudaError_t launch(const Params& p, dim3 grid, size_t smem, cudaStream_t s) {
  static std::mutex mu;
  static size_t have[64] = {};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  {
    std::lock_guard<std::mutex> lock(mu);
    if (dev >= 64 || have[dev] < smem) {
      e = cudaFuncSetAttribute(gemv_kernel<NT>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
      if (e != cudaSuccess) return e;
      if (dev < 64) have[dev] = smem;
    }
  }
  gemv_kernel<NT><<<grid, kThreads, smem, s>>>(p);
  return cudaGetLastError();
}

bool sizes_ok(int rows, int cols, int group, int scale_dtype) {
  return rows >= 1 && (group == 32 || group == 64 || group == 128) && cols >= group && cols % group == 0 && cols <= kMaxCols &&
         (scale_dtype == SPD_DTYPE_F32 || scale_dtype == SPD_DTYPE_BF16);
}
bool aligned(const void* p, size_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }
int launch_status(const char* who) {
  const cudaError_t e = cudaGetLastError();
  if (e == cudaSuccess) return SPD_OK;
  char msg[160];
  snprintf(msg, sizeof(msg), "%s: launch: %s", who, cudaGetErrorString(e));
  return spd_internal_fail(SPD_ECUDA, msg);
}

}  // namespace q4
}  // namespace spd

using namespace spd;

extern "C" size_t spd_q4_packed_bytes(int32_t rows, int32_t cols, int32_t group, int32_t scale_dtype, int32_t has_zeros) {
  if (!q4::sizes_ok(rows, cols, group, scale_dtype)) return 0;
  return (size_t)((rows + 15LL) / 16) * ((cols + 127) / 128) * q4::record_bytes(group, scale_dtype, has_zeros);
}

extern "C" int spd_q4_quantize(const void* w, int32_t dtype, int32_t rows, int32_t cols, int32_t group, int32_t scale_dtype,
                               uint8_t* codes, void* scales, uint8_t* zeros, void* cuda_stream) {
  if (!q4::sizes_ok(rows, cols, group, scale_dtype) || (dtype != SPD_DTYPE_F32 && dtype != SPD_DTYPE_BF16))
    return spd_internal_fail(SPD_EINVAL, "spd_q4_quantize: bad sizes or dtypes");
  if (!w || !codes || !scales) return spd_internal_fail(SPD_EINVAL, "spd_q4_quantize: NULL pointer");
  if (!q4::aligned(w, dtype == SPD_DTYPE_F32 ? 4 : 2) || !q4::aligned(scales, scale_dtype == SPD_DTYPE_F32 ? 4 : 2))
    return spd_internal_fail(SPD_EINVAL, "spd_q4_quantize: unaligned pointer");
  const long long ng = (long long)rows * (cols / group);
  const long long blocks = (ng + 7) / 8;
  if (blocks > 0x7fffffffLL) return spd_internal_fail(SPD_EINVAL, "spd_q4_quantize: matrix too large");
  cudaGetLastError();
  cudaStream_t s = reinterpret_cast<cudaStream_t>(cuda_stream);
  const int f = scale_dtype == SPD_DTYPE_F32;
  if (dtype == SPD_DTYPE_F32) q4::quantize_kernel<float><<<(unsigned)blocks, 256, 0, s>>>(static_cast<const float*>(w), ng, group, f, codes, scales, zeros);
  else q4::quantize_kernel<__nv_bfloat16><<<(unsigned)blocks, 256, 0, s>>>(static_cast<const __nv_bfloat16*>(w), ng, group, f, codes, scales, zeros);
  return q4::launch_status("spd_q4_quantize");
}

extern "C" int spd_q4_pack(const uint8_t* codes, const void* scales, const uint8_t* zeros, int32_t rows, int32_t cols, int32_t group,
                           int32_t scale_dtype, void* packed, size_t packed_bytes, void* cuda_stream) {
  if (!q4::sizes_ok(rows, cols, group, scale_dtype)) return spd_internal_fail(SPD_EINVAL, "spd_q4_pack: bad sizes");
  if (!codes || !scales || !packed) return spd_internal_fail(SPD_EINVAL, "spd_q4_pack: NULL pointer");
  if (!q4::aligned(packed, 16) || !q4::aligned(scales, scale_dtype == SPD_DTYPE_F32 ? 4 : 2))
    return spd_internal_fail(SPD_EINVAL, "spd_q4_pack: unaligned pointer");
  if (packed_bytes < spd_q4_packed_bytes(rows, cols, group, scale_dtype, zeros != nullptr))
    return spd_internal_fail(SPD_EINVAL, "spd_q4_pack: the packed buffer is too small");
  const int nkb = (cols + 127) / 128;
  const long long nrec = (rows + 15LL) / 16 * nkb;
  cudaGetLastError();
  q4::pack_kernel<<<(unsigned)((nrec + 7) / 8), 256, 0, reinterpret_cast<cudaStream_t>(cuda_stream)>>>(
      codes, scales, zeros, rows, cols, group, scale_dtype == SPD_DTYPE_F32, nkb, nrec, static_cast<unsigned char*>(packed),
      (int)q4::record_bytes(group, scale_dtype, zeros != nullptr));
  return q4::launch_status("spd_q4_pack");
}

extern "C" int spd_q4_gemv(const spd_q4_group* groups, int32_t G, int32_t M, int32_t cols, int32_t group, int32_t scale_dtype,
                           int32_t has_zeros, int32_t x_dtype, const float* nw, float eps, void* cuda_stream) {
  if (!groups || G < 1 || G > kMaxExplicit || M < 1 || M > q4::kMaxM || !q4::sizes_ok(1, cols, group, scale_dtype) ||
      (x_dtype != SPD_DTYPE_F32 && x_dtype != SPD_DTYPE_BF16))
    return spd_internal_fail(SPD_EINVAL, "spd_q4_gemv: bad sizes or dtypes");
  const size_t esz = x_dtype == SPD_DTYPE_F32 ? 4 : 2;
  if (nw && (!q4::aligned(nw, 4) || !(eps >= 0.f) || !std::isfinite(eps)))
    return spd_internal_fail(SPD_EINVAL, "spd_q4_gemv: bad norm weight or eps");
  q4::Params p;
  memset(&p, 0, sizeof(p));
  long long tiles = 0;
  for (int g = 0; g < G; ++g) {
    const spd_q4_group& s = groups[g];
    if (s.rows < 1 || !s.w || !s.x || !s.y || !q4::aligned(s.w, 16) || !q4::aligned(s.x, esz) || !q4::aligned(s.y, esz) ||
        (M > 1 && (s.x_stride < cols || s.y_stride < s.rows))) {
      char msg[128];
      snprintf(msg, sizeof(msg), "spd_q4_gemv: group %d: NULL or unaligned pointer, no rows, or a stride below the row", g);
      return spd_internal_fail(SPD_EINVAL, msg);
    }
    q4::Group& d = p.g[g];
    d.w = static_cast<const unsigned char*>(s.w); d.x = s.x; d.y = s.y; d.xs = s.x_stride; d.ys = s.y_stride;
    d.rows = s.rows; d.tile0 = (int)tiles;
    tiles += (s.rows + 15LL) / 16;
  }
  if (tiles > 0x7fffffffLL) return spd_internal_fail(SPD_EINVAL, "spd_q4_gemv: too many rows");
  p.G = G; p.M = M; p.cols = cols; p.nkb = (cols + 127) / 128; p.tiles = (int)tiles; p.gw = group / 32;
  p.rec = (int)q4::record_bytes(group, scale_dtype, has_zeros);
  p.s_f32 = scale_dtype == SPD_DTYPE_F32; p.has_z = has_zeros != 0; p.x_f32 = x_dtype == SPD_DTYPE_F32;
  p.nw = nw; p.eps = eps;
  p.terms = p.x_f32 ? 3 : nw ? 2 : 1;
  // vectors of a block: as many as shared memory and six operand tiles hold, in even shares
  int mb = M;
  while ((mb * p.terms > 48 || q4::gemv_smem(p.nkb, mb, p.terms, (mb * p.terms + 7) / 8) > 220 * 1024) && mb > 1) mb = (mb + 1) / 2;
  p.mb = mb;
  const int nt = (mb * p.terms + 7) / 8;
  const size_t smem = q4::gemv_smem(p.nkb, mb, p.terms, nt <= 4 ? nt : 6);
  const dim3 grid((unsigned)(tiles < 2 * num_sms() ? tiles : 2 * num_sms()), (unsigned)((M + mb - 1) / mb));
  cudaStream_t s = reinterpret_cast<cudaStream_t>(cuda_stream);
  cudaGetLastError();
  cudaError_t e;
  switch (nt) {
    case 1: e = q4::launch<1>(p, grid, smem, s); break;
    case 2: e = q4::launch<2>(p, grid, smem, s); break;
    case 3: e = q4::launch<3>(p, grid, smem, s); break;
    case 4: e = q4::launch<4>(p, grid, smem, s); break;
    default: e = q4::launch<6>(p, grid, smem, s); break;
  }
  if (e != cudaSuccess) {
    char msg[160];
    snprintf(msg, sizeof(msg), "spd_q4_gemv: launch: %s", cudaGetErrorString(e));
    return spd_internal_fail(SPD_ECUDA, msg);
  }
  return SPD_OK;
}
