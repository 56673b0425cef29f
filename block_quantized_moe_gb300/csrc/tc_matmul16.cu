// Products grouped by expert in 16 bits on the 5th-generation tensor cores (tcgen05 + TMEM + TMA).
//
// The three directions, for the rows [lo, hi) of each expert e:
//   product       out[r, i]    = sum_j a[r, j] w[e, i, j]
//   input grad    out[r, j]    = sum_i a[r, i] w[e, i, j]
//   weight grad   dw[e, i, j] (+)= sum_r dy[r, i] x[r, j]
// are one tile product D[m, c] = sum_l A[m, l] B[c, l] whose result is stored transposed,
// out[c, m]: m runs along the contiguous axis of the output (i, j and j), c along its rows (the
// expert's rows, or i). So the 32 lanes of an epilogue warp, which hold 32 consecutive m of one
// column c, always write consecutive addresses, and the ragged axis is always the MMA's N, which
// an instruction descriptor sets at run time in steps of 32:
//   product       A = w (l contiguous, "K-major")   B = a rows (K-major)      l: j, c: rows
//   input grad    A = w (m contiguous, "MN-major")  B = a rows (K-major)      l: i, c: rows
//   weight grad   A = x (MN-major)                  B = dy (MN-major)         l: rows, c: i
// One kernel therefore serves one row per expert and thousands: an expert's m_e rows make
// ceil(m_e / 256) column tiles of equal width, rounded up to 32.
//
// A unit (256 of m) x (up to 256 of c) runs on a CTA pair (cluster of two, tcgen05
// cta_group::2, M = 256): each CTA loads 128 rows of A and half of B per 64-deep step of l,
// 32 KiB a stage, so an SM reads 64 bytes a clock from L2 at the full MMA rate, half of what a
// 128 x 256 tile on one SM needs. Two accumulators of 256 TMEM columns let the epilogue of one
// unit run under the next unit's MMAs. Persistent pairs take units p, p + P, ...; units of one
// expert are adjacent, column tiles innermost, so that pairs working at the same time share
// weight blocks and rows in L2.
//
// Weight gradient: l is the ragged axis. TMA cannot stop at an expert's last row, so the last
// step of a segment lands on a barrier of its own; a warp then zeroes the rows past the
// segment, in A and in B (what is there may be NaN), up to the next multiple of 16, and hands
// the stage to the MMA issuer, which runs only the 16-row steps that hold rows.
// From saved rows (MXFP8), A arrives as codes; eight warps decode them into the operand tile,
// one 32-wide group with its power-of-two scale per thread, exactly.
//
// Roles: warp 0 TMA, warp 1 MMA issue and TMEM, warp 2 segment tails (weight grad), warps 4-11
// epilogue, warps 12-19 decode (saved rows). Every mbarrier wait is bounded: on timeout the
// kernel raises FTMOE_ERR_WAIT_TIMEOUT, stops its roles, waits for its own loads and MMAs,
// frees its TMEM and returns.
#include <cuda.h>

#include "common.cuh"
#include "elem16.cuh"
#include "internal.h"
#include "ptx.cuh"

namespace ftmoe {

namespace tc16 {

enum Mode { kProduct = 0, kInputGrad = 1, kWeightGrad = 2, kWeightGradSaved = 3 };

constexpr int kBK = 64;                   // elements of l per stage: one 128-byte swizzle atom
constexpr int kM = 256, kN = 256;         // of the pair
constexpr int kTile = 128 * kBK * 2;      // 16 KiB: this CTA's half of A, and of B at most
constexpr int kRaw = 128 * kBK;           // saved rows: 8 KiB of codes
constexpr int kEpiWarps = 8, kDecWarps = 8;
constexpr int kMaxExperts = 4096;

__host__ __device__ constexpr bool is_wgrad(int mode) { return mode >= kWeightGrad; }
__host__ __device__ constexpr int stage_bytes(int mode) { return 2 * kTile + (mode == kWeightGradSaved ? kRaw : 0); }
__host__ __device__ constexpr int stages(int mode) { return mode == kWeightGradSaved ? 5 : 6; }
__host__ __device__ constexpr int threads(int mode) { return 32 * (4 + kEpiWarps + (mode == kWeightGradSaved ? kDecWarps : 0)); }

struct Params {
  const int32_t* offsets;
  const uint8_t* x_scales;   // saved rows: [rows][k / 32]
  void* out;
  int64_t ld_out, out_expert;  // elements; out_expert 0 unless a weight gradient
  int64_t rows;
  int m_dim;                 // extent of m
  int l_dim;                 // extent of l (product, input grad)
  int c_dim;                 // weight grad: extent of c
  int E, out_dtype, bf16, accumulate;
};

// One MMA of the pair, issued by one lane of a converged warp: with the whole warp in the issue
// loop the descriptors stay in uniform registers. (A loop run by lane 0 alone moved each of them
// over for every MMA: measured on GB300, 830 clocks a stage of four MMAs, with no loads at all,
// against the 512 that the tensor cores take.)
__device__ __forceinline__ void mma_f16_pair(uint32_t d_tmem, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n .reg .pred p, q;\n setp.ne.b32 p, %4, 0;\n elect.sync _|q, 0xffffffff;\n"
      " @q tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n}" ::"r"(d_tmem),
      "l"(a), "l"(b), "r"(idesc), "r"(acc)
      : "memory");
}
// the same where `on`: a predicate, no branch
__device__ __forceinline__ void mma_f16_pair_if(uint32_t d_tmem, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc,
                                                bool on) {
  asm volatile(
      "{\n .reg .pred p, q, r;\n setp.ne.b32 p, %4, 0;\n setp.ne.b32 r, %5, 0;\n elect.sync _|q, 0xffffffff;\n"
      " and.pred q, q, r;\n @q tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n}" ::"r"(d_tmem),
      "l"(a), "l"(b), "r"(idesc), "r"(acc), "r"((uint32_t)on)
      : "memory");
}
// mma_commit_pair by the lane that issued the MMAs (elect.sync names the same one each time)
__device__ __forceinline__ void commit_pair_elected(uint32_t bar) {
  asm volatile(
      "{\n .reg .pred q;\n elect.sync _|q, 0xffffffff;\n"
      " @q tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;\n}" ::"r"(
          bar),
      "h"((uint16_t)0x3)
      : "memory");
}

// Operand tile whose m (or c) axis is contiguous: 64-element columns of 128-byte lines, one line
// per l, written by TMA with the 128-byte swizzle; the next 64 elements lie kBK lines further
// (leading offset), the next 8 lines 1024 bytes further (stride offset).
__device__ __forceinline__ uint64_t smem_desc_mn_sw128(uint32_t addr) {
  uint64_t d = 0;
  d |= (uint64_t)((addr & 0x3FFFF) >> 4);
  d |= (uint64_t)((kBK * 128) >> 4) << 16;
  d |= (uint64_t)(1024 >> 4) << 32;
  d |= (uint64_t)1 << 46;
  d |= (uint64_t)2 << 61;
  return d;
}

__device__ __forceinline__ void tma_pair_2d(uint32_t dst, const CUtensorMap* map, uint32_t bar, int x, int y) {
  asm volatile(
      "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4}], [%2];" ::"r"(
          dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(x), "r"(y)
      : "memory");
}
__device__ __forceinline__ void tma_pair_3d(uint32_t dst, const CUtensorMap* map, uint32_t bar, int x, int y, int z) {
  asm volatile(
      "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(
          dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(x), "r"(y), "r"(z)
      : "memory");
}

// arrive on a barrier of the pair's first CTA, releasing this CTA's shared-memory writes (fenced
// into the async proxy before) to the thread that issues the pair's MMAs
__device__ __forceinline__ void arrive_release_cluster(uint32_t cluster_addr) {
  asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr) : "memory");
}
__device__ __forceinline__ bool try_wait_cluster(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n .reg .pred p;\n mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2, 100;\n selp.u32 %0, 1, 0, p;\n}"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0;
}
// mbar_wait with acquire at cluster scope
__device__ __forceinline__ bool wait_cluster(uint32_t bar, uint32_t parity, volatile int* abort_flag) {
  if (try_wait_cluster(bar, parity)) return true;
  const unsigned long long t0 = globaltimer();
  while (!try_wait_cluster(bar, parity)) {
    if (*abort_flag) return false;
    if (globaltimer() - t0 > kTimeoutNs) {
      raise_error(FTMOE_ERR_WAIT_TIMEOUT);
      *abort_flag = 1;
      return false;
    }
  }
  return true;
}
__device__ __forceinline__ void fence_async_shared() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }
__device__ __forceinline__ void st_shared_16(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}
__device__ __forceinline__ uint4 ld_shared_16(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr));
  return v;
}

// One unit of work: 256 of m from m0, cols of c (width of the MMA's N), l in steps of kBK.
struct Unit {
  int e, m0;
  int c0, cols;    // first row of the output (or first i of a weight gradient) and how many
  int n;           // N of the MMA: cols rounded up to 32
  int l0, len;     // weight grad: first row of the segment and its length; else 0 and l_dim
};

// Two 16-bit roundings of the values of one lane pair: see store_columns.
template <typename Elem>
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  return (uint32_t)Elem::put(lo) | ((uint32_t)Elem::put(hi) << 16);
}

// 32 columns d[0..31] of this lane's m into out[(c0 + j) * ld + m], j < cols, m < m_dim. 16-bit
// types: neighbouring lanes trade every second column, so that each stores two adjacent m of
// one column as one word (where `words` says that rows keep 4-byte alignment).
template <typename Elem>
__device__ __forceinline__ void store_columns(typename Elem::T* out, int64_t ld, const float (&d)[32], int cols, int m,
                                              int m_dim, int lane, bool words, bool accumulate) {
  using T = typename Elem::T;
  if (sizeof(T) == 2 && words && !accumulate) {
    const bool odd = lane & 1;
    T* o = out + (m & ~1) + (odd ? ld : 0);
    const bool in = (m | 1) < m_dim;
#pragma unroll
    for (int j = 0; j < 32; j += 2) {
      const float got = __shfl_xor_sync(0xffffffffu, odd ? d[j] : d[j + 1], 1);
      const uint32_t w = odd ? pack2<Elem>(got, d[j + 1]) : pack2<Elem>(d[j], got);
      if (j + (odd ? 1 : 0) < cols) {
        if (in)
          *reinterpret_cast<uint32_t*>(o + j * ld) = w;
        else if ((m & ~1) < m_dim)  // m_dim odd: the last m alone
          o[j * ld] = (T)(w & 0xffffu);
      }
    }
  } else if (m < m_dim) {
    T* o = out + m;
    float old[32];
    if (accumulate) {
#pragma unroll
      for (int j = 0; j < 32; ++j) old[j] = j < cols ? Elem::get(o[j * ld]) : 0.0f;
    }
#pragma unroll
    for (int j = 0; j < 32; ++j)
      if (j < cols) o[j * ld] = Elem::put(accumulate ? old[j] + d[j] : d[j]);
  }
}

template <int MODE>
__global__ void __launch_bounds__(threads(MODE), 1)
    tc_matmul16_kernel(const __grid_constant__ CUtensorMap map_a, const __grid_constant__ CUtensorMap map_b0,
                       const __grid_constant__ CUtensorMap map_b1, const __grid_constant__ CUtensorMap map_b2,
                       const __grid_constant__ CUtensorMap map_b3, Params p) {
  constexpr bool kWG = is_wgrad(MODE), kSaved = MODE == kWeightGradSaved;
  constexpr int S = stages(MODE), kStage = stage_bytes(MODE);
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* tiles = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
  int* cum = reinterpret_cast<int*>(tiles + (size_t)S * kStage);  // [E + 1] units before expert e (not weight grad)
  __shared__ __align__(8) uint64_t full[S], empty[S], lfull[S], tfull[2], tempty[2];
  __shared__ uint32_t s_tmem;
  __shared__ volatile int s_abort;

  const int warp = __shfl_sync(0xffffffffu, (int)(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;
  const uint32_t crank = cluster_rank();
  const int MB = (p.m_dim + kM - 1) / kM;
  const int CB = kWG ? (p.c_dim + kN - 1) / kN : 0;

  auto bounds = [&](int e, int& lo, int& hi) {
    lo = __ldg(p.offsets + e);
    hi = __ldg(p.offsets + e + 1);
    lo = lo < 0 ? 0 : lo;
    hi = hi > p.rows ? (int)p.rows : hi;
    if (hi < lo) hi = lo;
  };

  if (threadIdx.x == 0) {
    s_abort = 0;
    for (int i = 0; i < S; ++i) {
      // saved rows: every decoding warp of both CTAs and the first CTA's producer; weight grad:
      // two arrivals of the first CTA's producer, or one of each CTA's tail warp; else its one
      mbar_init(smem_u32(&full[i]), kSaved ? 2 * kDecWarps + 1 : kWG ? 2 : 1);
      mbar_init(smem_u32(&empty[i]), 1);
      mbar_init(smem_u32(&lfull[i]), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_u32(&tfull[i]), 1);
      mbar_init(smem_u32(&tempty[i]), 2 * kEpiWarps);
    }
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if constexpr (!kWG) {
    if (warp == 0) {
      int run = 0;
      for (int base = 0; base < p.E; base += 32) {
        const int e = base + lane;
        int u = 0;
        if (e < p.E) {
          int lo, hi;
          bounds(e, lo, hi);
          u = (hi - lo + kN - 1) / kN * MB;
        }
        int inc = u;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int t = __shfl_up_sync(0xffffffffu, inc, o);
          if (lane >= o) inc += t;
        }
        if (e < p.E) cum[e] = run + inc - u;
        run += __shfl_sync(0xffffffffu, inc, 31);
      }
      if (lane == 0) cum[p.E] = run;
    }
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&s_tmem)), "r"(512));
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;");
  }
  fence_before();
  cluster_sync();  // both CTAs' barriers are initialised before either reports to the other
  fence_after();
  const uint32_t tmem_base = s_tmem;
  const int u_end = kWG ? p.E * MB * CB : cum[p.E];
  const int u_begin = (int)cluster_id_x(), u_step = (int)cluster_count_x();

  auto decode = [&](int u, Unit& t) {
    if constexpr (kWG) {
      // units of one expert adjacent: they read the same rows
      t.e = u / (MB * CB);
      const int local = u - t.e * MB * CB;
      t.m0 = local / CB * kM;
      t.c0 = local % CB * kN;
      t.cols = min(kN, p.c_dim - t.c0);
      int lo, hi;
      bounds(t.e, lo, hi);
      t.l0 = lo;
      t.len = hi - lo;
    } else {
      int a = 0, b = p.E - 1;
      while (a < b) {  // the last expert whose units begin at or before u
        const int mid = (a + b + 1) >> 1;
        if (cum[mid] <= u) a = mid; else b = mid - 1;
      }
      t.e = a;
      const int units = cum[a + 1] - cum[a], nt = units / MB, local = u - cum[a];
      int lo, hi;
      bounds(a, lo, hi);
      const int per = ((hi - lo + nt - 1) / nt + 31) & ~31;
      t.m0 = local / nt * kM;
      t.c0 = lo + local % nt * per;
      t.cols = min(per, hi - t.c0);
      t.l0 = 0;
      t.len = p.l_dim;
    }
    t.n = (t.cols + 31) & ~31;
  };

  if (warp == 0) {
    // ------------------------------- TMA producer -------------------------------
    if (lane == 0) {
      uint32_t it = 0, tails = 0, tail_ph = 0;  // bit st: slot st's last use was a tail; its phase
      for (int u = u_begin; u < u_end && !s_abort; u += u_step) {
        Unit t;
        decode(u, t);
        const int half = t.n >> 1;  // of c in each CTA
        const int steps = (t.len + kBK - 1) / kBK;
        const int cb = t.c0 + (int)crank * half, ma = t.m0 + (int)crank * 128;
        // K-major B: the smallest box that holds the half tile
        const int hb = half <= 16 ? 16 : half <= 32 ? 32 : half <= 64 ? 64 : 128;
        const CUtensorMap* mb = half <= 16 ? &map_b3 : half <= 32 ? &map_b2 : half <= 64 ? &map_b1 : &map_b0;
        const uint32_t bytes_b = kWG ? (half > 64 ? kTile : kTile / 2) : (uint32_t)hb * 128;
        for (int s = 0; s < steps; ++s, ++it) {
          const int st = it % S;
          if (!mbar_wait(smem_u32(&empty[st]), ((it / S) & 1) ^ 1, &s_abort)) break;
          const uint32_t ta = smem_u32(tiles + (size_t)st * kStage), tb = ta + kTile;
          const uint32_t fb = mapa_shared(smem_u32(&full[st]), 0);
          if constexpr (kWG) {
            const bool tail = t.len - s * kBK < kBK;
            const int l = t.l0 + s * kBK;
            const uint32_t local = smem_u32(&lfull[st]);
            tails = tail ? tails | (1u << st) : tails & ~(1u << st);
            if constexpr (kSaved) {
              mbar_expect_tx(local, kRaw + (tail ? bytes_b : 0));
              tail_ph ^= 1u << st;
              tma_pair_2d(tb + kTile, &map_a, local, ma, l);  // 128 codes of 64 rows
              if (crank == 0) {
                if (tail) mbar_arrive(smem_u32(&full[st]));
                else mbar_expect_tx(smem_u32(&full[st]), 2 * bytes_b);
              }
            } else if (tail) {
              mbar_expect_tx(local, kTile + bytes_b);
              tail_ph ^= 1u << st;
            } else if (crank == 0) {
              mbar_expect_tx(smem_u32(&full[st]), 2 * (kTile + bytes_b));
              mbar_arrive(smem_u32(&full[st]));
            }
            const uint32_t bar = tail ? local : fb;
            if constexpr (!kSaved) {
              tma_pair_2d(ta, &map_a, bar, ma, l);
              tma_pair_2d(ta + kTile / 2, &map_a, bar, ma + 64, l);
            }
            tma_pair_2d(tb, &map_b0, bar, cb, l);
            if (half > 64) tma_pair_2d(tb + kTile / 2, &map_b0, bar, cb + 64, l);
          } else {
            if (crank == 0) mbar_expect_tx(smem_u32(&full[st]), 2 * (kTile + bytes_b));
            if constexpr (MODE == kProduct) {
              tma_pair_3d(ta, &map_a, fb, s * kBK, ma, t.e);
            } else {
              tma_pair_3d(ta, &map_a, fb, ma, s * kBK, t.e);
              tma_pair_3d(ta + kTile / 2, &map_a, fb, ma + 64, s * kBK, t.e);
            }
            tma_pair_2d(tb, mb, fb, s * kBK, cb);
          }
        }
      }
      // Loads still in flight after an abort (bounded): tails and codes land on this CTA's
      // barriers, the rest on the first CTA's, which the second outlives no longer than the
      // closing cluster barrier.
      for (int st = 0; st < S && (uint32_t)st < it; ++st) {
        const uint32_t last = it - 1 - ((it - 1 - st) % S);
        const bool on_local = kSaved || (tails >> st & 1);
        if (!on_local && crank != 0) continue;
        const uint32_t bar = on_local ? smem_u32(&lfull[st]) : smem_u32(&full[st]);
        const uint32_t ph = on_local ? (tail_ph >> st & 1) ^ 1 : (last / S) & 1;
        const unsigned long long t0 = globaltimer();
        while (!mbar_try_wait(bar, ph) && globaltimer() - t0 < kTimeoutNs) {
        }
      }
    }
  } else if (warp == 1) {
    // -------------------------------- MMA issuer --------------------------------
    // (the whole warp runs the loop, one elected lane issues)
    if (crank == 0) {
      uint32_t it = 0, acc = 0;
      for (int u = u_begin; u < u_end; u += u_step) {
        Unit t;
        decode(u, t);
        if (t.len == 0) continue;
        const uint32_t idesc = (1u << 4) | ((uint32_t)p.bf16 << 7) | ((uint32_t)p.bf16 << 10) |
                               (MODE == kProduct ? 0u : 1u << 15) | (kWG ? 1u << 16 : 0u) |
                               ((uint32_t)(t.n >> 3) << 17) | ((uint32_t)(kM >> 4) << 24);
        const int buf = (int)(acc & 1);
        if (!__all_sync(0xffffffffu, mbar_wait(smem_u32(&tempty[buf]), ((acc >> 1) & 1) ^ 1, &s_abort))) break;
        fence_after();
        const uint32_t d = tmem_base + buf * kN;
        const int steps = (t.len + kBK - 1) / kBK;
        bool ok = true;
        for (int s = 0; s < steps; ++s, ++it) {
          const int st = it % S;
          ok = kWG ? wait_cluster(smem_u32(&full[st]), (it / S) & 1, &s_abort)
                   : mbar_wait(smem_u32(&full[st]), (it / S) & 1, &s_abort);
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
          fence_after();
          const uint32_t ta = smem_u32(tiles + (size_t)st * kStage), tb = ta + kTile;
          // No branch between the MMAs of a stage: one in front of each took the stage from 512
          // clocks to 900. Past l_dim TMA has filled in zeros; a segment's last stage turns off
          // the MMAs past its rows by predicate.
          const int left = t.len - s * kBK;
#pragma unroll
          for (int j = 0; j < kBK / 16; ++j) {
            const uint32_t acc_on = s > 0 || j > 0 ? 1u : 0u;
            if constexpr (kWG)
              mma_f16_pair_if(d, smem_desc_mn_sw128(ta + 2048 * j), smem_desc_mn_sw128(tb + 2048 * j), idesc, acc_on,
                              16 * j < left);
            else
              mma_f16_pair(d, MODE == kProduct ? smem_desc_sw128(ta + 32 * j) : smem_desc_mn_sw128(ta + 2048 * j),
                           smem_desc_sw128(tb + 32 * j), idesc, acc_on);
          }
          commit_pair_elected(smem_u32(&empty[st]));
        }
        if (!ok) break;
        commit_pair_elected(smem_u32(&tfull[buf]));
        ++acc;
      }
      // MMAs still running write TMEM: wait (bounded) for the last commit of each accumulator
      for (uint32_t b = 0; b < 2 && b < acc; ++b) {
        const uint32_t last = acc - 1 - ((acc - 1 - b) & 1);
        const unsigned long long t0 = globaltimer();
        while (!mbar_try_wait(smem_u32(&tfull[b]), (last >> 1) & 1) && globaltimer() - t0 < kTimeoutNs) {
        }
      }
    }
  } else if (MODE == kWeightGrad && warp == 2) {
    // ------------------------- tails of segments -------------------------
    uint32_t it = 0, ph = 0;
    bool ok = true;
    for (int u = u_begin; u < u_end && ok; u += u_step) {
      Unit t;
      decode(u, t);
      const int steps = (t.len + kBK - 1) / kBK, v = t.len % kBK;
      if (v != 0) {
        const int st = (it + steps - 1) % S;
        ok = mbar_wait(smem_u32(&lfull[st]), ph >> st & 1, &s_abort);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        ph ^= 1u << st;
        const uint32_t ta = smem_u32(tiles + (size_t)st * kStage);
        const int vr = (v + 15) & ~15;
        // lines v .. vr - 1 of the four 64-column boxes (A and B), 8 chunks of 16 bytes each
        for (int i = lane; i < (vr - v) * 32; i += 32)
          st_shared_16(ta + (i / 8 % 4) * (kTile / 2) + (v + i / 32) * 128 + (i % 8) * 16, 0, 0, 0, 0);
        fence_async_shared();
        __syncwarp();
        if (lane == 0) arrive_release_cluster(mapa_shared(smem_u32(&full[st]), 0));
      }
      it += steps;
    }
  } else if (warp >= 4 && warp < 4 + kEpiWarps) {
    // --------------------------------- epilogue ---------------------------------
    const int ew = warp - 4, quarter = warp & 3, half = ew >> 2;
    uint32_t acc = 0;
    const bool words = p.ld_out % 2 == 0 && p.out_expert % 2 == 0 && reinterpret_cast<uintptr_t>(p.out) % 4 == 0;
    for (int u = u_begin; u < u_end; u += u_step) {
      Unit t;
      decode(u, t);
      const bool none = kWG && t.len == 0;  // an expert without rows: zeros, or nothing to add
      if (none && p.accumulate) continue;
      const int buf = (int)(acc & 1);
      if (!none) {
        const int got = mbar_wait(smem_u32(&tfull[buf]), (acc >> 1) & 1, &s_abort) ? 1 : 0;
        if (__all_sync(0xffffffffu, got) == 0) break;
        fence_after();
        ++acc;
      }
      const uint32_t taddr = tmem_base + ((uint32_t)(32 * quarter) << 16) + buf * kN;
      const int m = t.m0 + (int)crank * 128 + 32 * quarter + lane;
      const int64_t first = (int64_t)t.e * p.out_expert + (int64_t)t.c0 * p.ld_out;
      // chunks of 32 columns, the two groups of four warps in turn
      for (int c = 32 * half; c < t.cols; c += 64) {
        float d[32];
        if (none) {
#pragma unroll
          for (int j = 0; j < 32; ++j) d[j] = 0.0f;
        } else {
          tmem_ld<32>(taddr + c, d);
          tmem_ld_wait();
        }
        const int64_t o = first + (int64_t)c * p.ld_out;
        const int cols = t.cols - c;
        if (p.out_dtype == FTMOE_OUT_FP32)
          store_columns<ElemF32>(static_cast<float*>(p.out) + o, p.ld_out, d, cols, m, p.m_dim, lane, words, p.accumulate);
        else if (p.out_dtype == FTMOE_OUT_BF16)
          store_columns<ElemBf16>(static_cast<uint16_t*>(p.out) + o, p.ld_out, d, cols, m, p.m_dim, lane, words, p.accumulate);
        else
          store_columns<ElemF16>(static_cast<uint16_t*>(p.out) + o, p.ld_out, d, cols, m, p.m_dim, lane, words, p.accumulate);
      }
      if (!none) {
        fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_cluster(mapa_shared(smem_u32(&tempty[buf]), 0));
      }
    }
  } else if (kSaved && warp >= 4 + kEpiWarps) {
    // ------------------------ saved rows: decode ------------------------
    // Thread (warp dw, lane): line r = 8 dw + lane % 8 of the stage's 64, 32-wide group lane / 8
    // of its 128 codes. Eight lanes with consecutive lines touch eight different 16-byte columns
    // of the swizzled lines, reading and writing.
    const int dw = warp - 4 - kEpiWarps, r = 8 * dw + (lane & 7), grp = lane >> 3;
    const int kg = p.m_dim / kMxBlock;
    uint32_t it = 0, ph = 0;
    bool ok = true;
    for (int u = u_begin; u < u_end && ok; u += u_step) {
      Unit t;
      decode(u, t);
      const int steps = (t.len + kBK - 1) / kBK;
      const int g = (t.m0 + (int)crank * 128) / kMxBlock + grp;
      // scale bytes are fetched a step ahead of their codes
      auto scale_at = [&](int s) {
        const int l = s * kBK + r;
        return g < kg && l < t.len ? (int)__ldg(p.x_scales + (int64_t)(t.l0 + l) * kg + g) : 0;
      };
      int next = steps > 0 ? scale_at(0) : 0;
      for (int s = 0; s < steps; ++s, ++it) {
        const int st = it % S;
        const float sc = e8m0_to_f((uint8_t)next);
        if (s + 1 < steps) next = scale_at(s + 1);
        ok = mbar_wait(smem_u32(&lfull[st]), ph >> st & 1, &s_abort);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        ph ^= 1u << st;
        const uint32_t ta = smem_u32(tiles + (size_t)st * kStage), raw = ta + 2 * kTile;
        const int left = t.len - s * kBK;
        const bool live = r < left;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const uint4 c = ld_shared_16(raw + r * 128 + (((2 * grp + h) ^ (r & 7)) << 4));
          const uint32_t cw[4] = {c.x, c.y, c.z, c.w};
          uint32_t o[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const uint32_t two = (cw[i >> 1] >> (16 * (i & 1))) & 0xffffu;
            const __half2_raw hr = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)two, __NV_E4M3);
            const float2 f = __half22float2(__half2(hr));
            const float lo = f.x * sc, hi = f.y * sc;
            o[i] = !live ? 0u : p.bf16 ? pack2<ElemBf16>(lo, hi) : pack2<ElemF16>(lo, hi);
          }
          // columns 32 grp + 16 h .. + 15: two 16-byte columns of the line in box grp / 2
          const uint32_t line = ta + (grp >> 1) * (kTile / 2) + r * 128;
          const int col = (grp & 1) * 4 + 2 * h;
          st_shared_16(line + ((col ^ (r & 7)) << 4), o[0], o[1], o[2], o[3]);
          st_shared_16(line + (((col + 1) ^ (r & 7)) << 4), o[4], o[5], o[6], o[7]);
        }
        if (left < kBK && r >= left) {
          // the segment's last step: dy's lines past its end (both 64-column boxes, this
          // thread's quarter of each)
          const uint32_t line = ta + kTile + r * 128;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int chunk = grp * 4 + i;
            st_shared_16(line + (chunk >> 3) * (kTile / 2) + ((chunk & 7) << 4), 0, 0, 0, 0);
          }
        }
        fence_async_shared();
        __syncwarp();
        if (lane == 0) arrive_release_cluster(mapa_shared(smem_u32(&full[st]), 0));
      }
    }
  }

  fence_before();
  // neither CTA leaves, or frees TMEM, while the other may still read its shared memory, signal
  // its barriers or (the MMAs of the first) write its TMEM
  __syncwarp();
  cluster_sync();
  if (warp == 1) {
    __syncwarp();
    fence_after();
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem_base), "r"(512));
  }
}

static bool encode16(CUtensorMap* map, const void* base, int rank, const uint64_t* dims, const uint64_t* strides,
                     const uint32_t* box) {
  EncodeTiledFn enc = encode_fn();
  if (!enc) return false;
  cuuint64_t d[3], st[2];
  cuuint32_t b[3], es[3] = {1, 1, 1};
  for (int i = 0; i < rank; ++i) d[i] = dims[i], b[i] = box[i];
  for (int i = 0; i + 1 < rank; ++i) st[i] = strides[i];
  return enc(map, CU_TENSOR_MAP_DATA_TYPE_UINT16, (cuuint32_t)rank, const_cast<void*>(base), d, st, b, es,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int MODE>
static cudaError_t launch(const CUtensorMap* maps, const Params& p, cudaStream_t st, int* unsupported) {
  const size_t smem = 1024 + (size_t)stages(MODE) * stage_bytes(MODE) + (is_wgrad(MODE) ? 0 : ((size_t)p.E + 1) * 4);
  int dev = 0;
  cudaGetDevice(&dev);
  // per device: CTA pairs that can be resident at once, with the largest shared memory this
  // kernel asks for (one CTA per SM either way)
  static int pairs[64] = {};
  int np = dev >= 0 && dev < 64 ? pairs[dev] : 0;
  if (np == 0) {
    const size_t most = 1024 + (size_t)stages(MODE) * stage_bytes(MODE) + (is_wgrad(MODE) ? 0 : (kMaxExperts + 1) * 4);
    const cudaError_t e =
        cudaFuncSetAttribute(tc_matmul16_kernel<MODE>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)most);
    if (e != cudaSuccess) return e;
    np = max_active_clusters(tc_matmul16_kernel<MODE>, dim3(threads(MODE)), most, 2, 2 * (sm_count() / 2));
    if (np > sm_count() / 2) np = sm_count() / 2;
    if (dev >= 0 && dev < 64) pairs[dev] = np;
  }
  if (np < 1) {
    *unsupported = 1;
    return cudaSuccess;
  }
  return launch_kernel_cluster(tc_matmul16_kernel<MODE>, dim3(2 * np), dim3(threads(MODE)), smem, st, false, 2, maps[0],
                               maps[1], maps[2], maps[3], maps[4], p);
}

}  // namespace tc16

// whether rows of 2-byte elements can be read by TMA: 16-byte base and stride
static bool tma16(const void* base, int64_t ld) { return (uintptr_t)base % 16 == 0 && ld % 8 == 0; }

cudaError_t launch_tc_matmul16(const Matmul16Args& a, cudaStream_t st, int* unsupported) {
  using namespace tc16;
  *unsupported = 1;
  const ftmoe_matrix_bank& w = a.w;
  const int64_t E = w.num_experts;
  if (E > kMaxExperts || a.rows < 1) return cudaSuccess;
  CUtensorMap maps[5];
  Params p = {};
  p.offsets = a.offsets;
  p.rows = a.rows;
  p.E = (int)E;
  p.bf16 = a.dtype == FTMOE_OUT_BF16;
  const uint64_t R = (uint64_t)a.rows;
  if (!a.wgrad) {
    const int64_t m = a.input_grad ? w.k : w.n, l = a.input_grad ? w.n : w.k;
    const int64_t units = (a.rows / kN + (a.rows < E ? a.rows : E)) * cdiv(m, kM);
    if (!tma16(a.a, a.ld_a) || !tma16(w.w, w.ld) || (E > 1 && w.expert_stride % 8 != 0) || units > 0x7fffffff)
      return cudaSuccess;
    // (a single expert's stride is never used, but has to be encodable)
    const uint64_t es = E > 1 ? (uint64_t)w.expert_stride : (uint64_t)w.n * w.ld;
    const uint64_t wd[3] = {(uint64_t)w.k, (uint64_t)w.n, (uint64_t)E}, ws[2] = {2 * (uint64_t)w.ld, 2 * es};
    const uint32_t wb[3] = {64, a.input_grad ? 64u : 128u, 1};
    if (!encode16(&maps[0], w.w, 3, wd, ws, wb)) return cudaSuccess;
    const uint64_t ad[2] = {(uint64_t)l, R}, as[1] = {2 * (uint64_t)a.ld_a};
    for (int i = 0; i < 4; ++i) {
      const uint32_t ab[2] = {64, 128u >> i};
      if (!encode16(&maps[1 + i], a.a, 2, ad, as, ab)) return cudaSuccess;
    }
    p.out = a.out;
    p.ld_out = a.ld_out;
    p.m_dim = (int)m;
    p.l_dim = (int)l;
    p.out_dtype = a.out_dtype;
    *unsupported = 0;
    return a.input_grad ? launch<kInputGrad>(maps, p, st, unsupported) : launch<kProduct>(maps, p, st, unsupported);
  }
  if (!tma16(a.a, a.ld_a) || E * cdiv(w.k, kM) * cdiv(w.n, kN) > 0x7fffffff) return cudaSuccess;
  const uint64_t dd[2] = {(uint64_t)w.n, R}, ds[1] = {2 * (uint64_t)a.ld_a};
  const uint32_t box[2] = {64, 64};
  if (!encode16(&maps[1], a.a, 2, dd, ds, box)) return cudaSuccess;
  maps[2] = maps[3] = maps[4] = maps[1];
  const uint64_t xd[2] = {(uint64_t)w.k, R};
  if (a.x_scales) {
    if ((uintptr_t)a.x % 16 != 0 || a.ld_x % 16 != 0) return cudaSuccess;
    const uint64_t xs[1] = {(uint64_t)a.ld_x};
    const uint32_t xb[2] = {128, 64};
    if (!encode_u8_tmap(&maps[0], a.x, 2, xd, xs, xb)) return cudaSuccess;
  } else {
    if (!tma16(a.x, a.ld_x)) return cudaSuccess;
    const uint64_t xs[1] = {2 * (uint64_t)a.ld_x};
    if (!encode16(&maps[0], a.x, 2, xd, xs, box)) return cudaSuccess;
  }
  p.x_scales = a.x_scales;
  p.out = w.w;
  p.ld_out = w.ld;
  p.out_expert = w.expert_stride;
  p.m_dim = (int)w.k;
  p.c_dim = (int)w.n;
  p.out_dtype = w.dtype;
  p.accumulate = a.accumulate;
  *unsupported = 0;
  return a.x_scales ? launch<kWeightGradSaved>(maps, p, st, unsupported) : launch<kWeightGrad>(maps, p, st, unsupported);
}

FTMOE_DEFINE_ERR_READER(read_err_tc_matmul16)

}  // namespace ftmoe
