// Decode attention of a batch that shares a prefix (spd_shared_prefix_attention).
//
//   out[b][h] = sum_j p_j v_j / sum_j p_j,  p_j = exp(q[b][h] . k_j / sqrt(hd) - m),  over the shared keys 0..P-1 and
// the sequence's own keys 0..len-1: the softmax is taken in one pass with a running maximum and sum, over parts of the
// keys, and the parts (O, m, l) are joined as  O = sum_i O_i e^(m_i - m),  l = sum_i l_i e^(m_i - m).
//
// prefix kernel (tcgen05): the queries of one kv head, all sequences' together, are the 128 rows of an MMA tile:
//   S = Q K_c^T  (M 128 x N 128 keys x K hd, fp32 in TMEM);  P = exp2(S - m) goes back to TMEM as bf16, over S, and is the A
//   operand of  O += P V_c  (M 128 x N hd x K 128 keys).
// One thread per row holds the row's 128 scores in registers, its running maximum and sum.  O is rescaled only when the
// maximum has grown by more than 8 (a factor of 256, which bf16's and fp32's exponents take without loss), so nearly never
// after the first chunk.  K and V chunks of 128 keys come by TMA through a ring of shared-memory stages; the tensor maps end
// at the prefix's length, so that rows beyond it are zeros whatever the buffer holds.  bf16 queries: two tiles a block
// alternate, one in the tensor core while the other's softmax runs.  fp32 queries: one tile, Q and P as three bf16 terms.
// The work, (row tiles) x (chunks), is cut into equal runs, one per SM; a run that crosses from one tile to the next leaves
// a part for each.  A chunk (64 KB at hd 128) feeds 2 x 4.2 MMAC a tile: the memory bounds up to about 256 rows a kv head,
// the tensor cores and exponentials beyond.
//
// rows kernel: joins those parts with the sequence's own keys.  One block per (sequence, kv head, up to 8 query heads of its group).  Its warps take 32 keys in turn and
// work on mma.sync m16n8k16: S^T = K Q^T (16 keys x 8 heads), then O^T += V^T P^T (16 head elements x 8 heads).  K and V go
// from global memory straight into operand registers: the order of the head elements in a dot product is free, so a lane
// reads 16 consecutive bytes; V's pairs of keys are put together with byte permutes.  fp32 queries and their
// probabilities enter as three bf16 terms (exact), bf16 queries' probabilities as one (rounded to bf16, 2^-9 relative,
// like the output).  Statistics and sums are fp32.
#include <cudaTypedefs.h>

#include <cmath>
#include <cstdio>
#include <cstring>
#include <mutex>

#include "spd_internal.cuh"
#include "spd_tc.cuh"

namespace spd {
namespace spa {

constexpr int kWarps = 4;   // most warps of a block of the rows kernel
constexpr int kThreads = 32 * kWarps;
constexpr int kHeads = 8;  // query heads of a block (the mma's 8 columns)
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

struct Params {
  const void* q;
  const __nv_bfloat16 *pk, *pv, *kc, *vc;
  const int* lens;
  void* out;
  float* lse;
  float* part;      // prefix parts: unnormalised O [slot][tile of the unit][hd / 4][row][4]
  float2* part_ml;  // their maximum and sum [slot][row of the unit]
  long long prefix_cap, max_seq;
  int P, B, hq, hkv, gq, hblocks;
  float scale_log2;  // log2(e) / sqrt(hd)
  // prefix kernel: `units` row tiles (pairs) x nch chunks, cut into n_cta runs; the part of run i for unit u is slot i + u
  int units_per_kv, units, nch, n_cta;
  int use_prefix;
  int row_cluster, parts;  // rows kernel: blocks of a sequence and kv head; most parts of a row
};

// first chunk of run i
__host__ __device__ inline long long run_start(long long total, int n, int i) { return total * i / n; }

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


// ---------------------------------------------------------------------------------------------
// prefix kernel
// ---------------------------------------------------------------------------------------------
constexpr int kTile = 128;   // rows of a tile, keys of a chunk
template <int HD, int TERMS> struct Cfg {
  static constexpr int kSlots = TERMS == 1 ? 2 : 1;              // row tiles of a block
  static constexpr int kTB = HD / 64 * kTile * 128;              // bytes of a 128-row operand
  static constexpr int kQ = kSlots * TERMS * kTB;                // Q
  static constexpr int kStages = (227 * 1024 - 2048 - kQ) / kTB > 8 ? 8 : (227 * 1024 - 2048 - kQ) / kTB;
  static constexpr int kSmem = 1024 + kQ + kStages * kTB;
  // softmax warps, a copying and a multiplying warp; two tiles: a whole third warpgroup, which gives up registers
  static constexpr int kThreads = kSlots == 2 ? 384 : 192;
  // TMEM columns: two tiles: S0 S1 O0 O1, P over S; one tile: S, O, and three P
  static constexpr uint32_t s_col(int i) { return 128u * i; }
  static constexpr uint32_t o_col(int i) { return kSlots == 2 ? 256u + 128u * i : 128u; }
  static constexpr uint32_t p_col(int i) { return kSlots == 2 ? 128u * i : 256u; }
};

struct PrefixMaps {
  CUtensorMap k, v;
};

__device__ __forceinline__ void tma3(void* dst, const CUtensorMap* map, int x, int y, int z, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];"
      ::"r"(smem_u32(dst)), "l"(map), "r"(x), "r"(y), "r"(z), "r"(smem_u32(bar))
      : "memory");
}
// The multiplying warp runs as a whole, so that descriptors stay in uniform registers; one elected lane issues.
__device__ __forceinline__ uint32_t elect_one() {
  uint32_t y;
  asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}\n" : "=r"(y));
  return y;
}
__device__ __forceinline__ void mma_ss(uint32_t lead, uint32_t d, uint64_t da, uint64_t db, uint32_t id, uint32_t accumulate) {
  asm volatile("{\n .reg .pred p, q;\n setp.ne.b32 p, %4, 0;\n setp.ne.b32 q, %5, 0;\n"
               " @q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}\n" ::"r"(d), "l"(da), "l"(db), "r"(id),
               "r"(accumulate), "r"(lead)
               : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t lead, uint32_t d, uint32_t a, uint64_t db, uint32_t id, uint32_t accumulate) {
  asm volatile("{\n .reg .pred p, q;\n setp.ne.b32 p, %4, 0;\n setp.ne.b32 q, %5, 0;\n"
               " @q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}\n" ::"r"(d), "r"(a), "l"(db), "r"(id),
               "r"(accumulate), "r"(lead)
               : "memory");
}
__device__ __forceinline__ void commit_if(uint32_t lead, uint64_t* bar) {
  asm volatile("{\n .reg .pred q;\n setp.ne.b32 q, %1, 0;\n"
               " @q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n}\n" ::"r"(smem_u32(bar)), "r"(lead)
               : "memory");
}
// V as the second operand, keys along K: rows of 128 bytes, 8-key groups 1024 B apart, the halves of hd one tile apart
__device__ __forceinline__ uint64_t desc_v(uint32_t a) {
  return (uint64_t)((a & 0x3FFFFu) >> 4) | ((uint64_t)((kTile * 128) >> 4) << 16) | ((uint64_t)(1024 >> 4) << 32) |
         ((uint64_t)1 << 46) | ((uint64_t)2 << 61);
}
__host__ __device__ constexpr uint32_t idesc(int n, int b_mn_major) {
  return (1u << 4) | (1u << 7) | (1u << 10) | ((uint32_t)b_mn_major << 16) | ((uint32_t)(n >> 3) << 17) |
         ((uint32_t)(kTile >> 4) << 24);
}
__device__ __forceinline__ void tm_st32(uint32_t ta, const uint32_t* v) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,"
      "%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};"
      ::"r"(ta), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]),
        "r"(v[8]), "r"(v[9]), "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15]),
        "r"(v[16]), "r"(v[17]), "r"(v[18]), "r"(v[19]), "r"(v[20]), "r"(v[21]), "r"(v[22]), "r"(v[23]),
        "r"(v[24]), "r"(v[25]), "r"(v[26]), "r"(v[27]), "r"(v[28]), "r"(v[29]), "r"(v[30]), "r"(v[31])
      : "memory");
}
__device__ __forceinline__ void tm_st16(uint32_t ta, const uint32_t* v) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};"
               ::"r"(ta), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]),
                 "r"(v[8]), "r"(v[9]), "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
               : "memory");
}
__device__ __forceinline__ void tm_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

__device__ __forceinline__ void opaque(uint64_t& x) { asm volatile("" : "+l"(x)); }

// Byte offset of element (row r, column e) in a [64-element chunk][128 rows][128 B] operand with the 128-byte swizzle.
__device__ __forceinline__ uint32_t swz(int r, int e) {
  return (uint32_t)((e >> 6) * (kTile * 128) + r * 128 + ((((e & 63) >> 3) ^ (r & 7)) << 4) + (e & 7) * 2);
}

// Bounded wait that also ends once another role of the block has given up.
__device__ __forceinline__ bool wait(uint64_t* bar, uint32_t parity, volatile int* fail) {
  if (mbar_try_wait(bar, parity)) return true;
  const uint64_t t0 = globaltimer_ns();
  for (uint32_t it = 0;; ++it) {
    if (mbar_try_wait(bar, parity)) return true;
    if ((it & 63u) == 63u && (*fail || globaltimer_ns() - t0 > kWaitLimitNs)) {
      *fail = 1;
      return false;
    }
  }
}

template <int HD, int TERMS>
__global__ void __launch_bounds__(Cfg<HD, TERMS>::kThreads, 1)
prefix_kernel(const __grid_constant__ Params p, const __grid_constant__ PrefixMaps maps) {
  using C = Cfg<HD, TERMS>;
  constexpr int NS = C::kSlots, ST = C::kStages;
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  unsigned char* sq = reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
  unsigned char* ring = sq + C::kQ;
  __shared__ __align__(8) uint64_t full[ST], empty[ST], q_ready[NS], s_full[NS], p_ready[NS], o_full[NS], s_free[NS], pv_done, drain;
  __shared__ uint32_t s_tmem;
  __shared__ int s_fail_;
  volatile int& s_fail = *const_cast<volatile int*>(&s_fail_);
  const int tid = threadIdx.x, warp = tid >> 5;
  constexpr int kCopyWarp = NS * 4, kMmaWarp = NS * 4 + 1;
  if (tid == 0) {
    for (int i = 0; i < ST; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 1);
    }
    for (int i = 0; i < NS; ++i) {
      mbar_init(&q_ready[i], 128);
      mbar_init(&s_full[i], 1);
      mbar_init(&p_ready[i], 128);
      mbar_init(&o_full[i], 1);
      mbar_init(&s_free[i], 128);
    }
    mbar_init(&pv_done, 1);
    mbar_init(&drain, 1);
    s_fail_ = 0;
    fence_mbar_init();
  }
  if (warp == kMmaWarp) tc::alloc_cols(&s_tmem, 512);
  if (warp == kCopyWarp && (tid & 31) < 2)
    asm volatile("prefetch.tensormap [%0];" ::"l"((tid & 31) ? &maps.v : &maps.k));
  tc::fence_before();
  __syncthreads();
  tc::fence_after();
  pdl_wait();
  pdl_trigger();  // the rows kernel may start its own keys beside this one
  const uint32_t tm = s_tmem;
  const long long total = (long long)p.units * p.nch;
  const long long w0 = run_start(total, p.n_cta, blockIdx.x), w1 = run_start(total, p.n_cta, blockIdx.x + 1);
  const int rows = p.B * p.gq;

  // a piece: the chunks [c0, c1) of one unit; the unit's tiles with rows
  struct Piece { int u, c0, c1, kh, row0, nt; };
  auto piece_at = [&](long long w) {
    Piece x;
    x.u = (int)(w / p.nch);
    x.c0 = (int)(w - (long long)x.u * p.nch);
    x.c1 = (int)min((long long)p.nch, x.c0 + (w1 - w));
    x.kh = x.u / p.units_per_kv;
    x.row0 = (x.u - x.kh * p.units_per_kv) * NS * kTile;
    x.nt = min(NS, (rows - x.row0 + kTile - 1) / kTile);
    return x;
  };

  // Two tiles: 384 threads start with 168 registers each (64,512 in all); 224 for a softmax thread, which holds 128 scores,
  // and 56 for the others are 2 x 128 x 224 + 128 x 56 = 64,512.
  if (warp >= NS * 4) {
    if (NS == 2) asm volatile("setmaxnreg.dec.sync.aligned.u32 56;");
  if (warp == kCopyWarp) {
    if ((tid & 31) == 0) {
      int st = 0;
      uint32_t ph = 0;  // the first pass over the stages waits for nothing
      int issued = 0;
      bool ok = true;
      for (long long w = w0; w < w1 && ok;) {
        const Piece x = piece_at(w);
        for (int c = x.c0; c < x.c1 && ok; ++c)
          for (int kv = 0; kv < 2 && ok; ++kv) {
            ok = wait(&empty[st], ph ^ 1, &s_fail);
            if (!ok) break;
            mbar_arrive_expect_tx(&full[st], C::kTB);
            for (int h = 0; h < HD / 64; ++h)
              tma3(ring + st * C::kTB + h * kTile * 128, kv ? &maps.v : &maps.k, h * 64, c * kTile, x.kh, &full[st]);
            ++issued;
            if (++st == ST) { st = 0; ph ^= 1; }
          }
        w += x.c1 - x.c0;
      }
      if (!ok)  // the copies in flight land before the block leaves
        for (int i = 0; i < ST && i < issued; ++i) {
          const int at = issued - 1 - i;
          mbar_wait_bounded(&full[at % ST], (at / ST) & 1);
        }
    }
    __syncwarp();
  } else if (warp == kMmaWarp) {
    const uint32_t lead = elect_one();
    uint32_t st = 0, ph = 0;         // the next stage to take, K and V in turn
    uint32_t ph_q = 0, ph_p = 0, ph_f = 0;  // one bit a tile
    bool ok = true;
    constexpr uint32_t id_s = idesc(kTile, 0), id_o = idesc(HD, 1);
    const uint64_t dq0 = tc::sdesc(tc::su32(sq)), dk0 = tc::sdesc(tc::su32(ring)), dv0 = desc_v(tc::su32(ring));
    auto take = [&](uint32_t& at, uint32_t& parity) {
      at = st;
      parity = ph;
      if (++st == ST) { st = 0; ph ^= 1; }
    };
    auto await = [&](uint64_t* bar, uint32_t parity) { return __all_sync(0xffffffffu, wait(bar, parity, &s_fail)) != 0; };
    auto scores = [&](int i, uint32_t stage) {
      uint64_t dk = dk0 + (uint64_t)(stage * (C::kTB >> 4)), dq = dq0 + (uint64_t)(i * (TERMS * C::kTB >> 4));
      opaque(dk);  // descriptors are added up in place: hoisted out of the loop they would spill
      opaque(dq);
#pragma unroll
      for (int e = TERMS - 1; e >= 0; --e)  // the small terms first
#pragma unroll
        for (int ks = 0; ks < HD / 16; ++ks) {
          const int off = (ks >> 2) * kTile * 128 + (ks & 3) * 32;
          mma_ss(lead, tm + C::s_col(i), dq + ((e * C::kTB + off) >> 4), dk + (off >> 4), id_s, e < TERMS - 1 || ks > 0);
        }
      commit_if(lead, &s_full[i]);
    };
    for (long long w = w0; w < w1 && ok;) {
      const Piece x = piece_at(w);
      for (int i = 0; i < x.nt && ok; ++i) {
        ok = await(&q_ready[i], ph_q >> i & 1);
        ph_q ^= 1u << i;
      }
      if (!ok) break;
      tc::fence_after();
      uint32_t kst, kph;
      take(kst, kph);
      ok = await(&full[kst], kph);
      if (!ok) break;
      for (int i = 0; i < x.nt; ++i) scores(i, kst);
      commit_if(lead, &empty[kst]);
      for (int c = x.c0; c < x.c1 && ok; ++c) {
        const bool more = c + 1 < x.c1;
        uint32_t vst, vph, k2 = 0, k2ph = 0;
        take(vst, vph);
        if (more) take(k2, k2ph);
#pragma unroll
        for (int i = 0; i < NS; ++i) {
          if (i >= x.nt || !ok) break;
          if (NS == 1 && more) {  // P does not lie over S: the next scores run during this chunk's softmax
            ok = await(&s_free[i], ph_f & 1) && await(&full[k2], k2ph);
            ph_f ^= 1;
            if (!ok) break;
            tc::fence_after();
            scores(i, k2);
            commit_if(lead, &empty[k2]);
          }
          ok = await(&p_ready[i], ph_p >> i & 1);
          ph_p ^= 1u << i;
          if (ok && i == 0) ok = await(&full[vst], vph);
          if (!ok) break;
          tc::fence_after();
          uint64_t dv = dv0 + (uint64_t)(vst * (C::kTB >> 4));
          opaque(dv);
#pragma unroll
          for (int e = TERMS - 1; e >= 0; --e)
#pragma unroll
            for (int ks = 0; ks < kTile / 16; ++ks)
              mma_ts(lead, tm + C::o_col(i), tm + C::p_col(i) + e * 64 + ks * 8, dv + ((ks * 2048) >> 4), id_o,
                     c > x.c0 || e < TERMS - 1 || ks > 0);
          if (i == x.nt - 1) commit_if(lead, &empty[vst]);
          if (!more) commit_if(lead, &o_full[i]);
          if (NS == 2 && more) {
            if (i == 0) ok = await(&full[k2], k2ph);
            if (!ok) break;
            scores(i, k2);  // after this tile's P V, which reads what it overwrites
            if (i == x.nt - 1) commit_if(lead, &empty[k2]);
          }
          if (NS == 1 && more) commit_if(lead, &pv_done);
        }
      }
      w += x.c1 - x.c0;
    }
    if (!ok) {  // the products in flight end before the block leaves
      commit_if(lead, &drain);
      mbar_wait_bounded(&drain, 0);
    }
    __syncwarp();
  }
  } else {
    if (NS == 2) asm volatile("setmaxnreg.inc.sync.aligned.u32 224;");
    const int slot = warp >> 2, r = tid & 127;
    const uint32_t lanes = (uint32_t)(32 * (warp & 3)) << 16;
    const uint32_t to = tm + C::o_col(slot) + lanes, tp = tm + C::p_col(slot) + lanes;
    uint32_t ph_s = 0, ph_o = 0, ph_v = 0;
    bool ok = true;
    for (long long w = w0; w < w1 && ok;) {
      const Piece x = piece_at(w);
      w += x.c1 - x.c0;
      if (slot >= x.nt) continue;
      const int row = x.row0 + slot * kTile + r;
      const bool valid = row < rows;
      {
        const int b = row / p.gq, h = x.kh * p.gq + row % p.gq;
        const long long at = ((long long)b * p.hq + h) * HD;
        unsigned char* dst = sq + slot * TERMS * C::kTB;
#pragma unroll (TERMS == 1 ? HD / 8 : 4)
        for (int e = 0; e < HD; e += 8) {
          if (TERMS == 1) {
            const uint4 v = valid ? *reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(p.q) + at + e) : make_uint4(0, 0, 0, 0);
            *reinterpret_cast<uint4*>(dst + swz(r, e)) = v;
          } else {
            float f[8] = {};
            if (valid) {
              const float4 a = *reinterpret_cast<const float4*>(static_cast<const float*>(p.q) + at + e);
              const float4 c = *reinterpret_cast<const float4*>(static_cast<const float*>(p.q) + at + e + 4);
              f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w; f[4] = c.x; f[5] = c.y; f[6] = c.z; f[7] = c.w;
            }
#pragma unroll
            for (int t = 0; t < TERMS; ++t) {
              uint4 v;
              v.x = take_pair(f[0], f[1]); v.y = take_pair(f[2], f[3]); v.z = take_pair(f[4], f[5]); v.w = take_pair(f[6], f[7]);
              *reinterpret_cast<uint4*>(dst + t * C::kTB + swz(r, e)) = v;
            }
          }
        }
      }
      tc::fence_async_smem();
      mbar_arrive(&q_ready[slot]);
      float m = -INFINITY, l = 0.f;
      for (int c = x.c0; c < x.c1; ++c) {
        ok = wait(&s_full[slot], ph_s, &s_fail);
        ph_s ^= 1;
        if (!ok) break;
        tc::fence_after();
        float sv[kTile];
#pragma unroll
        for (int j = 0; j < kTile; j += 32) tc::load_rows(tm + C::s_col(slot) + j, warp, reinterpret_cast<uint32_t*>(sv + j));
        if (NS == 1 && c + 1 < x.c1) {
          tc::fence_before();
          mbar_arrive(&s_free[slot]);
        }
        const int left = p.P - c * kTile;  // keys of this chunk
        if (left < kTile) {
#pragma unroll
          for (int j = 0; j < kTile; ++j)
            if (j >= left) sv[j] = -INFINITY;
        }
        float mx[4] = {sv[0], sv[1], sv[2], sv[3]};
#pragma unroll
        for (int j = 4; j < kTile; ++j) mx[j & 3] = fmaxf(mx[j & 3], sv[j]);
        const float mc = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * p.scale_log2;
        const bool grow = c == x.c0 || mc > m + 8.f;
        float al = 1.f;
        if (grow) {
          const float mn = fmaxf(m, mc);
          al = mn == -INFINITY ? 1.f : ex2(m - mn);
          m = mn;
          l *= al;
        }
        if (NS == 1 && c > x.c0) {  // P and O are this thread's once the last P V is done
          ok = wait(&pv_done, ph_v, &s_fail);
          ph_v ^= 1;
          if (!ok) break;
          tc::fence_after();
        }
        // with two tiles every P V so far is done: the scores just read were issued after it
        if (c > x.c0 && __any_sync(0xffffffffu, grow)) {
#pragma unroll
          for (int j = 0; j < HD; j += 16) {
            uint32_t ov[16];
            tc::load_rows16(tm + C::o_col(slot) + j, warp, ov);
#pragma unroll
            for (int t = 0; t < 16; ++t) ov[t] = __float_as_uint(__uint_as_float(ov[t]) * al);
            tm_st16(to + j, ov);
          }
          tm_st_wait();
        }
        const float mu = m == -INFINITY ? 0.f : m;
        float ls[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int j = 0; j < kTile; j += 64) {
#pragma unroll
          for (int t = 0; t < 64; ++t) {
            sv[j + t] = ex2(fmaf(sv[j + t], p.scale_log2, -mu));
            ls[t & 3] += sv[j + t];
          }
#pragma unroll
          for (int e = 0; e < TERMS; ++e) {
            uint32_t pk[32];
#pragma unroll
            for (int t = 0; t < 32; ++t) pk[t] = take_pair(sv[j + 2 * t], sv[j + 2 * t + 1]);
            tm_st32(tp + e * 64 + j / 2, pk);
          }
        }
        l += (ls[0] + ls[1]) + (ls[2] + ls[3]);
        tm_st_wait();
        tc::fence_before();
        mbar_arrive(&p_ready[slot]);
      }
      if (!ok) break;
      ok = wait(&o_full[slot], ph_o, &s_fail);
      ph_o ^= 1;
      if (!ok) break;
      tc::fence_after();
      // unnormalised O and (m, l) of the row
      const long long part_tile = (long long)(blockIdx.x + x.u) * NS + slot;
      float* po = p.part + part_tile * (kTile * HD) + r * 4;  // [element / 4][row][4]: neighbours write neighbours
#pragma unroll
      for (int j = 0; j < HD; j += 32) {
        uint32_t ov[32];
        tc::load_rows(tm + C::o_col(slot) + j, warp, ov);
        if (valid)
#pragma unroll
          for (int t = 0; t < 32; t += 4)
            *reinterpret_cast<uint4*>(po + (j + t) * kTile) = make_uint4(ov[t], ov[t + 1], ov[t + 2], ov[t + 3]);
      }
      p.part_ml[part_tile * kTile + r] = make_float2(m, l);
    }
    if (!ok)  // a wait gave up: the rows of this block's pieces come out NaN
      for (long long w = w0; w < w1;) {
        const Piece x = piece_at(w);
        w += x.c1 - x.c0;
        p.part_ml[(long long)(blockIdx.x + x.u) * (NS * kTile) + slot * kTile + r] = make_float2(0.f, NAN);
      }
  }
  tc::fence_before();
  __syncthreads();
  if (warp == kMmaWarp) tc::free_cols(tm, 512);
}


// The sum over the cluster's blocks goes through their shared memory.
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ uint32_t remote_addr(const void* p, int rank) {  // the same place in another block of the cluster
  uint32_t a;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_u32(p)), "r"(rank));
  return a;
}
__device__ __forceinline__ float remote(const float* p, int rank) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(remote_addr(p, rank)) : "memory");
  return v;
}
__device__ __forceinline__ float4 remote4(const float* p, int rank) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0,%1,%2,%3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(remote_addr(p, rank)) : "memory");
  return v;
}

template <int N> struct Int { static constexpr int value = N; };

// Shared memory of the rows kernel: the warps' rings (afterwards O, maxima and sums of the warps), the weights of the parts,
// the barriers.
constexpr int kRing = 3;                                       // steps of 16 keys that a warp has under way
constexpr int stage_bytes(int hd) { return 2 * 16 * hd * 2; }  // K and V
__host__ __device__ constexpr int rows_smem(int warps, int hd, int parts) {
  return warps * kRing * stage_bytes(hd) + (kHeads * parts * 4 + 7) / 8 * 8 + warps * kRing * 8;
}

template <int HD, int TERMS>
__global__ void __launch_bounds__(kThreads, TERMS == 1 ? 3 : 2) rows_kernel(const __grid_constant__ Params p) {
  constexpr int KI = HD / 32;  // 16-byte pieces of a key a lane reads
  constexpr int NS = Cfg<HD, TERMS>::kSlots;
  extern __shared__ __align__(128) unsigned char smem[];
  const int W = blockDim.x >> 5;
  float* s_o = reinterpret_cast<float*>(smem);  // [warp][head][HD], over the rings
  float* s_m = s_o + W * kHeads * HD;           // [warp][head]
  float* s_l = s_m + W * kHeads;                // [warp][head]
  float* s_w = reinterpret_cast<float*>(smem + W * kRing * stage_bytes(HD));  // [head][part]
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + rows_smem(W, HD, p.parts) - W * kRing * 8);
  static_assert(kRing * stage_bytes(HD) >= kHeads * (HD + 2) * 4, "a warp's sums fit over its ring");
  __shared__ float s_sum[kHeads];
  __shared__ int s_fail;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
  const int CS = p.row_cluster, rank = blockIdx.x % CS, pair = blockIdx.x / CS;
  const int hb = pair % p.hblocks, kh = pair / p.hblocks % p.hkv, b = pair / p.hblocks / p.hkv;
  const int h0 = kh * p.gq + hb * kHeads, nh = min(kHeads, p.gq - hb * kHeads);
  unsigned char* ring = smem + warp * kRing * stage_bytes(HD);
  uint64_t* bar = bars + warp * kRing;
  if (lane == 0) {
    for (int i = 0; i < kRing; ++i) mbar_init(&bar[i], 1);
    fence_mbar_init();
  }
  if (tid == 0) s_fail = 0;
  const int len = p.max_seq > 0 ? p.lens[b] : 0;
  const bool bad = len < 0 || len > p.max_seq;
  const int P = p.use_prefix ? 0 : p.P;  // prefix keys that this kernel reads itself
  const int nkeys = bad ? 0 : P + len;
  const int key_step = CS * W * 16;
  int key0 = (rank * W + warp) * 16;
  const __nv_bfloat16* own_k = p.kc + ((long long)b * p.hkv + kh) * p.max_seq * HD;
  const __nv_bfloat16* own_v = p.vc + ((long long)b * p.hkv + kh) * p.max_seq * HD;
  const __nv_bfloat16* pre_k = p.pk + (long long)kh * p.prefix_cap * HD;
  const __nv_bfloat16* pre_v = p.pv + (long long)kh * p.prefix_cap * HD;
  // the rows of 16 keys from k0, those that exist, into a stage: K [16][HD], V [16][HD]
  const uint64_t pol = l2_evict_first_policy();
  auto fetch = [&](int st, int k0) {  // lane 0
    unsigned char* dst = ring + st * stage_bytes(HD);
    const int n = min(16, nkeys - k0), a = max(0, min(n, P - k0));  // a of them in the prefix
    mbar_arrive_expect_tx(&bar[st], (uint32_t)n * HD * 4);
    if (a > 0) {
      bulk_g2s(dst, pre_k + (long long)k0 * HD, a * HD * 2, &bar[st], pol);
      bulk_g2s(dst + 16 * HD * 2, pre_v + (long long)k0 * HD, a * HD * 2, &bar[st], pol);
    }
    if (a < n) {
      const long long at = (long long)(k0 + a - P) * HD;
      bulk_g2s(dst + a * HD * 2, own_k + at, (n - a) * HD * 2, &bar[st], pol);
      bulk_g2s(dst + (16 + a) * HD * 2, own_v + at, (n - a) * HD * 2, &bar[st], pol);
    }
  };
  if (lane == 0)
    for (int i = 0; i < kRing; ++i)
      if (key0 + i * key_step < nkeys) fetch(i, key0 + i * key_step);
  // Q^T as the second operand: head g, elements 32 i + 8 t + 4 s + {0, 1}, {2, 3}
  uint32_t qb[TERMS][KI][2][2];
#pragma unroll
  for (int i = 0; i < KI; ++i) {
    const long long at = ((long long)b * p.hq + h0 + min(g, nh - 1)) * HD + 32 * i + 8 * t;
    float x[8];
    if (TERMS > 1) {
      const float4 a = *reinterpret_cast<const float4*>(static_cast<const float*>(p.q) + at);
      const float4 c = *reinterpret_cast<const float4*>(static_cast<const float*>(p.q) + at + 4);
      x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w; x[4] = c.x; x[5] = c.y; x[6] = c.z; x[7] = c.w;
#pragma unroll
      for (int e = 0; e < TERMS; ++e)
#pragma unroll
        for (int s = 0; s < 2; ++s) {
          qb[e][i][s][0] = take_pair(x[4 * s], x[4 * s + 1]);
          qb[e][i][s][1] = take_pair(x[4 * s + 2], x[4 * s + 3]);
        }
    } else {
      const uint4 a = *reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(p.q) + at);
      qb[0][i][0][0] = a.x; qb[0][i][0][1] = a.y; qb[0][i][1][0] = a.z; qb[0][i][1][1] = a.w;
    }
  }
  float o[HD / 16][4];
#pragma unroll
  for (int e = 0; e < HD / 16; ++e) o[e][0] = o[e][1] = o[e][2] = o[e][3] = 0.f;
  float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};  // heads 2 t, 2 t + 1

  __syncwarp();  // the barriers are set up
  bool ok = true;
  int st = 0;
  uint32_t ph = 0;
  for (; key0 < nkeys; key0 += key_step) {
    if (ok) ok = __all_sync(0xffffffffu, mbar_wait_bounded(&bar[st], ph)) != 0;
    unsigned char* stage = ring + st * stage_bytes(HD);
    if (nkeys - key0 < 16) {  // rows that no key fills weigh nothing, but must not hold NaN
      for (int i = (nkeys - key0) * (HD / 8) + lane; i < 16 * (HD / 8); i += 32)
        reinterpret_cast<uint4*>(stage + 16 * HD * 2)[i] = make_uint4(0, 0, 0, 0);
      __syncwarp();
    }
    uint4 kr[2][KI], vr[4][HD / 64];  // keys g, g + 8; keys 2 t, 2 t + 1, 2 t + 8, 2 t + 9
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int i = 0; i < KI; ++i) kr[j][i] = *reinterpret_cast<const uint4*>(stage + (g + 8 * j) * HD * 2 + 16 * t + 64 * i);
    // the hardware's sums drop bits: the small terms first, in chains of their own
    float s[4] = {0.f, 0.f, 0.f, 0.f}, s2[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int e = TERMS - 1; e >= 0; --e)
#pragma unroll
      for (int i = 0; i < KI; ++i) {
        float* c = e > 0 ? s2 : s;
        mma16816(c, kr[0][i].x, kr[1][i].x, kr[0][i].y, kr[1][i].y, qb[e][i][0][0], qb[e][i][0][1]);
        mma16816(c, kr[0][i].z, kr[1][i].z, kr[0][i].w, kr[1][i].w, qb[e][i][1][0], qb[e][i][1][1]);
      }
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int c = 0; c < HD / 64; ++c)
        vr[j][c] = *reinterpret_cast<const uint4*>(stage + (16 + 2 * t + (j & 1) + 8 * (j >> 1)) * HD * 2 + 16 * g + 128 * c);
    // s: (key g, heads 2t, 2t+1), (key g + 8, heads 2t, 2t+1)
    float al[2], pr[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) s[j] = key0 + g + 8 * (j >> 1) < nkeys ? (s[j] + s2[j]) * p.scale_log2 : -INFINITY;
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
    if (__any_sync(0xffffffffu, al[0] != 1.f || al[1] != 1.f)) {
#pragma unroll
      for (int e = 0; e < HD / 16; ++e) {
        o[e][0] *= al[0]; o[e][1] *= al[1]; o[e][2] *= al[0]; o[e][3] *= al[1];
      }
    }
    uint32_t pb[TERMS][2];
#pragma unroll
    for (int e = 0; e < TERMS; ++e) {
      pb[e][0] = movm(take_pair(pr[0], pr[1]));
      pb[e][1] = movm(take_pair(pr[2], pr[3]));
    }
    // element e of this lane's two pieces of 8: rows g -> g * 8 + e and g + 8 -> 64 + g * 8 + e (hd 128), or
    // g * 8 + 2 e and g * 8 + 2 e + 1 (hd 64)
    auto word = [&](int k, int i) {
      const uint4& x = vr[k][i >> 2];
      return (i & 3) == 0 ? x.x : (i & 3) == 1 ? x.y : (i & 3) == 2 ? x.z : x.w;
    };
    auto take = [&](int k, int el) {  // elements el of keys k and k + 1
      return __byte_perm(word(k, el >> 1), word(k + 1, el >> 1), el & 1 ? 0x7632 : 0x5410);
    };
#pragma unroll
    for (int e = 0; e < HD / 16; ++e) {
      const int lo = HD == 128 ? e : 2 * e, hi = HD == 128 ? e + 8 : 2 * e + 1;
      const uint32_t a0 = take(0, lo), a1 = take(0, hi), a2 = take(2, lo), a3 = take(2, hi);
      if (TERMS == 1) {
        mma16816(o[e], a0, a1, a2, a3, pb[0][0], pb[0][1]);
      } else {  // this step's sum apart from the total, which is added to with rounding
        float c[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int x = TERMS - 1; x >= 0; --x) mma16816(c, a0, a1, a2, a3, pb[x][0], pb[x][1]);
#pragma unroll
        for (int x = 0; x < 4; ++x) o[e][x] += c[x];
      }
    }
    __syncwarp();  // every lane has read the stage
    if (lane == 0 && ok && key0 + kRing * key_step < nkeys) fetch(st, key0 + kRing * key_step);
    if (++st == kRing) { st = 0; ph ^= 1; }
  }
  if (!ok) {  // a wait gave up: the copies in flight land, the row comes out NaN
    for (int i = 0; i < kRing; ++i) mbar_wait_bounded(&bar[(st + i) % kRing], ph ^ (st + i >= kRing), 10000000ull);
    s_fail = 1;
  }
  __syncthreads();  // the rings are read, and the sums may lie over them
  // this warp's part
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    l[j] += __shfl_xor_sync(0xffffffffu, l[j], 4);
    l[j] += __shfl_xor_sync(0xffffffffu, l[j], 8);
    l[j] += __shfl_xor_sync(0xffffffffu, l[j], 16);
    if (g == 0) {
      s_m[warp * kHeads + 2 * t + j] = m[j];
      s_l[warp * kHeads + 2 * t + j] = l[j];
    }
  }
#pragma unroll
  for (int e = 0; e < HD / 16; ++e) {
    const int lo = HD == 128 ? g * 8 + e : g * 8 + 2 * e, hi = HD == 128 ? 64 + g * 8 + e : g * 8 + 2 * e + 1;
    float* d0 = s_o + (warp * kHeads + 2 * t) * HD;
    d0[lo] = o[e][0]; d0[HD + lo] = o[e][1]; d0[hi] = o[e][2]; d0[HD + hi] = o[e][3];
  }
  __syncthreads();
  // The parts of a row: W warps of this block, or the blocks of the cluster (each first adds up its own warps, in the place
  // of its first), then the prefix kernel's.
  auto combine = [&](float& y, float w, float v) { y = fmaf(w, v, y); };
  if (CS > 1) {
    for (int i = tid; i < nh * (HD / 4); i += blockDim.x) {
      const int h = i / (HD / 4), d = i % (HD / 4) * 4;
      float mx = -INFINITY;
      for (int w = 0; w < W; ++w) mx = fmaxf(mx, s_m[w * kHeads + h]);
      const float mu = mx == -INFINITY ? 0.f : mx;
      float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
      for (int w = 0; w < W; ++w) {
        const float a = ex2(s_m[w * kHeads + h] - mu);
        const float4 v = *reinterpret_cast<const float4*>(s_o + (w * kHeads + h) * HD + d);
        combine(y.x, a, v.x); combine(y.y, a, v.y); combine(y.z, a, v.z); combine(y.w, a, v.w);
      }
      *reinterpret_cast<float4*>(s_o + h * HD + d) = y;  // read by this thread only
    }
    __syncthreads();
    if (tid < nh) {
      float mx = -INFINITY, lt = 0.f;
      for (int w = 0; w < W; ++w) mx = fmaxf(mx, s_m[w * kHeads + tid]);
      const float mu = mx == -INFINITY ? 0.f : mx;
      for (int w = 0; w < W; ++w) lt += s_l[w * kHeads + tid] * ex2(s_m[w * kHeads + tid] - mu);
      s_m[tid] = mx;
      s_l[tid] = lt;
    }
    cluster_sync();
  }
  pdl_wait();  // the prefix kernel's parts are there (every block waits, so that this grid ends after that one)
  const int nw = CS > 1 ? CS : W;
  const bool none = p.P == 0 && len == 0;
  if (rank == 0) {
    // the row's parts of the prefix: slots first + u .. last + u of its unit
    __shared__ long long s_at[kHeads];
    __shared__ int s_np[kHeads];
    auto prefix_parts = [&](int h, int* np) {
      const int prow = b * p.gq + hb * kHeads + h, u = kh * p.units_per_kv + prow / (NS * kTile);
      if (!p.use_prefix) {
        *np = 0;
        return 0LL;
      }
      const long long total = (long long)p.units * p.nch;
      int first;
      if (total * p.n_cta < 0x7fffffffLL) {  // 32-bit divisions where they do
        first = ((u * p.nch + 1) * p.n_cta - 1) / (int)total;
        *np = ((u + 1) * p.nch * p.n_cta - 1) / (int)total - first + 1;
      } else {
        first = (int)((((long long)u * p.nch + 1) * p.n_cta - 1) / total);
        *np = (int)(((long long)(u + 1) * p.nch * p.n_cta - 1) / total) - first + 1;
      }
      return (long long)(first + u) * (NS * kTile) + prow % (NS * kTile);
    };
    // Weights of the parts: 4 W neighbouring lanes a head, all heads at once.
    {
      const int L = 4 * W, h = min(tid / L, nh - 1), l0 = tid % L;  // heads that do not exist repeat the last one
      int np;
      const long long at = prefix_parts(h, &np);
      const float2* ml = p.part_ml + at;
      float* wt = s_w + h * p.parts;
      const int n = nw + np;
      auto get = [&](int j) {
        return j < nw ? (CS > 1 ? make_float2(remote(&s_m[h], j), remote(&s_l[h], j)) : make_float2(s_m[j * kHeads + h], s_l[j * kHeads + h]))
                      : __ldcg(ml + (long long)(j - nw) * NS * kTile);
      };
      float mx = -INFINITY, lt = 0.f;
      for (int j = l0; j < n; j += 4 * L) {
        float2 v[4];
#pragma unroll
        for (int x = 0; x < 4; ++x) v[x] = j + x * L < n ? get(j + x * L) : make_float2(-INFINITY, 0.f);
        const float mn = fmaxf(fmaxf(mx, fmaxf(v[0].x, v[1].x)), fmaxf(v[2].x, v[3].x)), mu = mn == -INFINITY ? 0.f : mn;
        lt *= ex2(mx - mu);
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          lt += v[x].y * ex2(v[x].x - mu);
          if (j + x * L < n && tid / L < nh) wt[j + x * L] = v[x].x;
        }
        mx = mn;
      }
      float ma = mx;
      for (int x = L >> 1; x; x >>= 1) ma = fmaxf(ma, __shfl_xor_sync(0xffffffffu, ma, x));
      const float mu = ma == -INFINITY ? 0.f : ma;
      lt *= ex2(mx - mu);
      for (int x = L >> 1; x; x >>= 1) lt += __shfl_xor_sync(0xffffffffu, lt, x);
      if (tid / L < nh) {
        for (int j = l0; j < n; j += L) wt[j] = ex2(wt[j] - mu);
        if (l0 == 0) {
          s_at[h] = at;
          s_np[h] = np;
          s_sum[h] = lt;
          if (p.lse) p.lse[(long long)b * p.hq + h0 + h] = bad || s_fail ? NAN : none ? -INFINITY : ma * kLn2 + logf(lt);
        }
      }
    }
    __syncthreads();
    // Four elements of a head a thread and item; neighbours take the heads, whose rows lie side by side in a part.  A few
    // items' loads, or a few parts', are under way together.
    const int items = nh * (HD / 4);
    auto outputs = [&](auto n_items, auto n_parts) {
      constexpr int NI = decltype(n_items)::value, NP = decltype(n_parts)::value;
      for (int i0 = tid; i0 < items; i0 += NI * blockDim.x) {
        float4 y[NI];
        const float* src[NI];
        const float* wt[NI];
        int most = 0, np[NI];
#pragma unroll
        for (int x = 0; x < NI; ++x) {
          const int i = min(i0 + x * (int)blockDim.x, items - 1), h = i % nh, d = i / nh * 4;
          y[x] = make_float4(0.f, 0.f, 0.f, 0.f);
          np[x] = s_np[h];
          most = max(most, np[x]);
          wt[x] = s_w + h * p.parts;
          src[x] = p.part + s_at[h] / kTile * (kTile * HD) + d * kTile + s_at[h] % kTile * 4;
        }
        auto add = [&](float4& y, float w, const float4& v) {
          combine(y.x, w, v.x); combine(y.y, w, v.y); combine(y.z, w, v.z); combine(y.w, w, v.w);
        };
        for (int j = 0; j < most; j += NP) {
          float4 v[NP][NI];
#pragma unroll
          for (int k = 0; k < NP; ++k)
#pragma unroll
            for (int x = 0; x < NI; ++x)
              if (j + k < np[x]) v[k][x] = __ldcg(reinterpret_cast<const float4*>(src[x] + (long long)(j + k) * NS * kTile * HD));
#pragma unroll
          for (int k = 0; k < NP; ++k)
#pragma unroll
            for (int x = 0; x < NI; ++x)
              if (j + k < np[x]) add(y[x], wt[x][nw + j + k], v[k][x]);
        }
#pragma unroll
        for (int x = 0; x < NI; ++x) {
          const int i = i0 + x * (int)blockDim.x;
          if (i >= items) break;
          const int h = i % nh, d = i / nh * 4;
          for (int j = 0; j < nw; ++j)
            add(y[x], wt[x][j], CS > 1 ? remote4(s_o + h * HD + d, j) : *reinterpret_cast<const float4*>(s_o + (j * kHeads + h) * HD + d));
          const float inv = 1.0f / s_sum[h];
          float4 o4 = make_float4(y[x].x * inv, y[x].y * inv, y[x].z * inv, y[x].w * inv);
          if (bad || s_fail) o4 = make_float4(NAN, NAN, NAN, NAN);
          else if (none) o4 = make_float4(0.f, 0.f, 0.f, 0.f);
          const long long at = ((long long)b * p.hq + h0 + h) * HD + d;
          if (TERMS > 1) {
            *reinterpret_cast<float4*>(static_cast<float*>(p.out) + at) = o4;
          } else {
            const __nv_bfloat162 lo = __floats2bfloat162_rn(o4.x, o4.y), hi = __floats2bfloat162_rn(o4.z, o4.w);
            *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(p.out) + at) =
                make_uint2(*reinterpret_cast<const uint32_t*>(&lo), *reinterpret_cast<const uint32_t*>(&hi));
          }
        }
      }
    };
    if (items > 2 * (int)blockDim.x) outputs(Int<4>(), Int<4>());
    else outputs(Int<1>(), Int<12>());
  }
  if (CS > 1) cluster_sync();  // nobody reads this block's shared memory any more
}

// Prefix keys through the tensor cores, or read by the rows kernel of every sequence: the tensor cores' part costs some 8 us
// before it gains anything.  Bytes that all sequences together would read: at 17 MB (32 x 128 keys, 8 kv heads) 7.8 us
// directly and 11.0 through the tensor cores, at 34 MB (4 x 2048) 11.5 and 12.3, at 67 MB (16 x 1024) 15.7 and 11.8, at 155 MB
// (17 x 1111, 16 kv heads, fp32 queries) 32 and 25.
bool prefix_pays(int B, int hkv, int hd, int P) { return (long long)B * hkv * P * hd * 4 > (48LL << 20); }

// Units, runs and chunks of the prefix kernel; `ns` row tiles a unit.
void prefix_geometry(int rows, int hkv, int P, int ns, int sms, Params* p) {
  p->units_per_kv = (rows + ns * kTile - 1) / (ns * kTile);
  p->units = hkv * p->units_per_kv;
  p->nch = (P + kTile - 1) / kTile;
  const long long total = (long long)p->units * p->nch;
  p->n_cta = (int)(total < sms ? total : sms);
}
size_t part_rows(const Params& p, int ns) { return ((size_t)p.n_cta + p.units) * ns * kTile; }

cudaError_t encode_map(CUtensorMap* out, const void* base, int hd, int P, int cap, int hkv) {
  static PFN_cuTensorMapEncodeTiled_v12000 encode = nullptr;
  static std::mutex mu;
  {
    std::lock_guard<std::mutex> lock(mu);
    if (!encode) {
      void* fn = nullptr;
      cudaDriverEntryPointQueryResult q = cudaDriverEntryPointSymbolNotFound;
      const cudaError_t e = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault, &q);
      if (e != cudaSuccess) return e;
      if (q != cudaDriverEntryPointSuccess || !fn) return cudaErrorNotSupported;
      encode = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(fn);
    }
  }
  // (element, key, kv head); the key dimension ends at P: keys beyond it are zeros in shared memory
  const cuuint64_t dim[3] = {(cuuint64_t)hd, (cuuint64_t)P, (cuuint64_t)hkv};
  const cuuint64_t stride[2] = {(cuuint64_t)hd * 2, (cuuint64_t)cap * hd * 2};
  const cuuint32_t box[3] = {64, (cuuint32_t)kTile, 1};
  const cuuint32_t one[3] = {1, 1, 1};
  const CUresult r = encode(out, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dim, stride, box, one,
                            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

template <int HD, int TERMS>
cudaError_t launch(Params& p, void* workspace, cudaStream_t s) {
  using C = Cfg<HD, TERMS>;
  static std::mutex mu;
  static bool set[64] = {};  // the shared-memory limits belong to a device
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  {
    std::lock_guard<std::mutex> lock(mu);
    if (dev >= 64 || !set[dev]) {
      e = cudaFuncSetAttribute(prefix_kernel<HD, TERMS>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
      if (e == cudaSuccess)
        e = cudaFuncSetAttribute(rows_kernel<HD, TERMS>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 rows_smem(kWarps, HD, 8 + num_sms()));
      if (e != cudaSuccess) return e;
      if (dev < 64) set[dev] = true;
    }
  }
  if (p.use_prefix) {
    prefix_geometry(p.B * p.gq, p.hkv, p.P, C::kSlots, num_sms(), &p);
    p.part = static_cast<float*>(workspace);
    p.part_ml = reinterpret_cast<float2*>(p.part + part_rows(p, C::kSlots) * HD);
    PrefixMaps maps;
    e = encode_map(&maps.k, p.pk, HD, p.P, (int)p.prefix_cap, p.hkv);
    if (e == cudaSuccess) e = encode_map(&maps.v, p.pv, HD, p.P, (int)p.prefix_cap, p.hkv);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t pc;
    memset(&pc, 0, sizeof(pc));
    pc.gridDim = dim3((unsigned)p.n_cta);
    pc.blockDim = dim3(C::kThreads);
    pc.dynamicSmemBytes = C::kSmem;
    pc.stream = s;
    cudaLaunchAttribute pa[1];
    pa[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    pa[0].val.programmaticStreamSerializationAllowed = 1;
    pc.attrs = pa;
    pc.numAttrs = 1;
    if ((e = cudaLaunchKernelEx(&pc, prefix_kernel<HD, TERMS>, p, maps)) != cudaSuccess) return e;
  }
  // Warps of a pair (sequence, kv head): as many as run at once (8 an SM, by their rings), and enough for a warp to take 1024
  // keys at most of a full cache; where 4 are too few, blocks in a cluster.
  const long long pairs = (long long)p.B * p.hkv * p.hblocks, keys = p.max_seq + (p.use_prefix ? 0 : p.P);
  int warps = 1;
  while (warps < kWarps * 8 && warps * 16 < keys && (pairs * warps * 2 <= 8LL * num_sms() || warps * 1024 < keys)) warps *= 2;
  p.row_cluster = warps > kWarps ? warps / kWarps : 1;
  warps /= p.row_cluster;
  p.parts = 8 + (p.use_prefix ? p.n_cta : 0);  // warps or blocks of a cluster: 8 at most
  cudaLaunchConfig_t cfg;
  memset(&cfg, 0, sizeof(cfg));
  cfg.gridDim = dim3((unsigned)(pairs * p.row_cluster));
  cfg.blockDim = dim3((unsigned)(32 * warps));
  cfg.dynamicSmemBytes = (size_t)rows_smem(warps, HD, p.parts);
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  int n = 0;
  if (p.use_prefix) {
    attr[n].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[n++].val.programmaticStreamSerializationAllowed = 1;
  }
  if (p.row_cluster > 1) {
    attr[n].id = cudaLaunchAttributeClusterDimension;
    attr[n].val.clusterDim.x = (unsigned)p.row_cluster;
    attr[n].val.clusterDim.y = attr[n].val.clusterDim.z = 1;
    ++n;
  }
  cfg.attrs = attr;
  cfg.numAttrs = n;
  return cudaLaunchKernelEx(&cfg, rows_kernel<HD, TERMS>, p);
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
  if (!spa::prefix_pays(B, n_kv_heads, head_dim, prefix_len)) return 16;
  size_t rows = 0;
  for (int ns = 1; ns <= 2; ++ns) {  // tiles a unit: fp32 and bf16 queries
    spa::Params p;
    spa::prefix_geometry(B * (n_heads / n_kv_heads), n_kv_heads, prefix_len, ns, num_sms(), &p);
    const size_t n = spa::part_rows(p, ns);
    rows = n > rows ? n : rows;
  }
  return rows * (head_dim * sizeof(float) + sizeof(float2));
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
  p.lens = lens; p.out = out; p.lse = lse;
  p.prefix_cap = prefix_cap; p.max_seq = max_seq; p.P = prefix_len; p.B = B; p.hq = n_heads; p.hkv = n_kv_heads;
  p.gq = n_heads / n_kv_heads;
  p.hblocks = (p.gq + spa::kHeads - 1) / spa::kHeads;
  p.scale_log2 = spa::kLog2e / std::sqrt((float)head_dim);
  p.use_prefix = spa::prefix_pays(B, n_kv_heads, head_dim, prefix_len);
  cudaStream_t s = reinterpret_cast<cudaStream_t>(cuda_stream);
  cudaGetLastError();
  cudaError_t e;
  if (head_dim == 128) e = q_dtype == SPD_DTYPE_F32 ? spa::launch<128, 3>(p, workspace, s) : spa::launch<128, 1>(p, workspace, s);
  else e = q_dtype == SPD_DTYPE_F32 ? spa::launch<64, 3>(p, workspace, s) : spa::launch<64, 1>(p, workspace, s);
  if (e != cudaSuccess) {
    char msg[160];
    snprintf(msg, sizeof(msg), "spd_shared_prefix_attention: launch: %s", cudaGetErrorString(e));
    return spd_internal_fail(SPD_ECUDA, msg);
  }
  return SPD_OK;
}
