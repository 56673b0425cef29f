// Products grouped by expert in 16 bits on the 5th-generation tensor cores (tcgen05 + TMEM + TMA).
//
// The three directions, for the rows [lo, hi) of each expert e:
//   product       out[r, i]    = sum_j a[r, j] w[e, i, j]
//   input grad    out[r, j]    = sum_i a[r, i] w[e, i, j]
//   weight grad   dw[e, i, j] (+)= sum_r dy[r, i] x[r, j]
// are one tile product D[m, c] = sum_l A[m, l] B[c, l], m along the lanes of an accumulator and c
// along its columns, whose width an instruction descriptor sets at run time in steps of 32:
//   product       A = w (l contiguous, "K-major")   B = a rows (K-major)      l: j, m: i, c: rows
//   input grad    A = w (m contiguous, "MN-major")  B = a rows (K-major)      l: i, m: j, c: rows
//   weight grad   A = dy (MN-major)                 B = x (MN-major)          l: rows, m: i, c: j
// The first two keep the ragged axis in c and store the result transposed, out[c, m]: the 32
// lanes of an epilogue warp, 32 consecutive m of one column, write consecutive addresses. The
// weight gradient's accumulator is a tile of dw as it lies in memory, or (fp32, long segments) its
// transpose, with A and B exchanged.
// One kernel therefore serves one row per expert and thousands: an expert's m_e rows make
// ceil(m_e / 256) column tiles of equal width, rounded up to 32.
//
// A unit (256 of m) x (up to 256 of c) runs on a CTA pair (cluster of two, tcgen05
// cta_group::2, M = 256): each CTA loads 128 rows of A and half of B per 64-deep step of l,
// 32 KiB a stage, so an SM reads 64 bytes a clock from L2 at the full MMA rate, half of what a
// 128 x 256 tile on one SM needs. Two accumulators of 256 TMEM columns let the epilogue of one
// unit run under the next unit's MMAs. Persistent pairs take units p, p + P, ...; units of one
// expert are adjacent (product: column tiles innermost), so that pairs working at the same time
// share weight blocks and rows in L2.
//
// Weight gradient: l is the ragged axis. TMA cannot stop at an expert's last row, so the last
// step of a segment lands on a barrier of its own; a warp then zeroes the rows past the
// segment, in A and in B (what is there may be NaN), up to the next multiple of 16, and hands
// the stage to the MMA issuer, which runs only the 16-row steps that hold rows.
// From saved rows (MXFP8), B arrives as codes; teams of warps decode them into the operand tile,
// a 32-wide group with its power-of-two scale at a time, exactly.
//
// Long sums. The tensor core cuts low bits off as it adds a product to its fp32 accumulator: the
// error is a bias that grows with the number of additions (measured: 4.4e-6 of the result's norm
// over 4,096 terms, where fp32 sums rounded to nearest have 6e-7). So an accumulator takes 8 stages
// (512 terms) for fp32 outputs and 32 (2,048 terms) for 16-bit ones, and the epilogue adds the
// accumulators up in registers, 128 per thread, the control warps giving up theirs. 16-bit products
// cost nothing by it (32 stages, 8 stages and one accumulator throughout: 24,576 rows over 32 experts,
// 4096 x 7168: 911, 925, 910 us). 16-bit weight gradients do, as their output boxes then leave in
// bursts (500 rows for each of 64 experts, 2048 x 4096: 409 us against 391; the 32 experts above 993
// against 976), so they have it in calls of more than 4,096 rows (fp16) or 32,768 (bf16). Up to there
// one accumulator's bias is a nineteenth of the type's unit roundoff at most: over operands of one
// sign, where it is largest, 2.5e-5 and 2.1e-4 (6.4e-9 a row). An fp32 weight gradient of segments
// that are short on average, or from saved rows (whose decoding warps need the registers), takes 16
// stages and adds the parts of the few segments that are longer in memory, by TMA. A 16-bit one from
// saved rows, in calls of more rows than that, takes 64 stages (2.5e-5) and adds the parts of a longer
// segment up in TMEM: one accumulator holds the sum, so that the MMAs wait while a part is added to
// it.
//
// Measured on GB300: product of 24,576 rows over 256 experts, 4096 x 7168, 2,328 us (6.7 TB/s, the
// measured copy rate); over 32 experts of 768 rows 791 us (1,825 TFLOP/s in a burst; 1,550 in a
// long run, where the power cap holds the clock at 1.41 GHz); its input gradient 779 us; its
// weight gradient 848 us, of one expert's 24,576 rows 730 us (1,977 TFLOP/s); from saved rows, uneven
// load, 1,044 us. Bound by memory below about 200 rows per expert, above by the tensor cores, the
// weight gradient also by shared memory (operands in and out leave little room for the tile on
// its way out), the saved rows by decoding.
//
// Roles: warp 0 TMA, warp 1 MMA issue and TMEM, warp 2 segment tails (weight grad) or codes
// (saved rows), warps 4-11 epilogue, warps 12 on decode (saved rows). Every mbarrier wait is
// bounded: on timeout the kernel raises FTMOE_ERR_WAIT_TIMEOUT, stops its roles, waits for its own
// loads and MMAs, frees its TMEM and returns.
#include <cuda.h>

#include "common.cuh"
#include "elem16.cuh"
#include "internal.h"
#include "ptx.cuh"

namespace ftmoe {

namespace tc16 {

// kWeightGradT: the weight gradient with the operands' roles exchanged (A = x, B = dy), stored
// transposed like the product: fp32 outputs and long segments, see the epilogue
// kWeightGradSavedLong: kWeightGradSaved for segments that are long on average
enum Mode { kProduct = 0, kInputGrad = 1, kWeightGrad = 2, kWeightGradSaved = 3, kWeightGradT = 4, kWeightGradSavedLong = 5 };

constexpr int kBK = 64;                   // elements of l per stage: one 128-byte swizzle atom
constexpr int kM = 256, kN = 256;         // of the pair
constexpr int kTile = 128 * kBK * 2;      // 16 KiB: this CTA's half of A, and of B at most
constexpr int kRaw = 128 * kBK;           // saved rows: 8 KiB of codes
constexpr int kOutBuf = 8192;             // an output box: 32 columns of c (16 of fp32) by 128 of m
constexpr int kOutBufs = 3;               // boxes in flight for each half of the epilogue
constexpr int kEpiWarps = 8, kTeamWarps = 4;
constexpr int kMaxExperts = 1024;  // segment bounds and unit counts live in shared memory

__host__ __device__ constexpr bool is_wgrad(int mode) { return mode >= kWeightGrad; }
// whether an accumulator is a tile of the output as it lies in memory
__host__ __device__ constexpr bool by_rows(int mode) { return is_wgrad(mode) && mode != kWeightGradT; }
__host__ __device__ constexpr bool is_saved(int mode) { return mode == kWeightGradSaved || mode == kWeightGradSavedLong; }
constexpr int kSquareRows = 4096;         // weight grad: see the order of units
// 32 KiB a stage, the output boxes, and the ring of codes. Five stages: with four a weight
// gradient of 24,576 rows, 4096 x 7168, takes 863 us instead of 715.
__host__ __device__ constexpr int stages(int mode) { return mode == kWeightGradSaved ? 4 : 5; }
// Saved rows: teams of decoding warps and code slots, as many of one as of the other: a team meets
// its slot in every one of its phases. (Waiting by parity, it could take a phase that another team
// has yet to see for its own.) Long segments: a fifth stage and a fourth team for one of the two
// box buffers of each pair of epilogue warps. Measured (64 experts, 2048 x 4096, fp32, us), short
// and long: 128 rows each 366, 394; 300 rows 448, 449; 500 rows 566, 520; 1,500 rows 1416, 1223.
__host__ __device__ constexpr int teams(int mode) { return !is_saved(mode) ? 0 : mode == kWeightGradSaved ? 3 : 4; }
__host__ __device__ constexpr int row_bufs(int mode) { return mode == kWeightGradSavedLong ? 1 : 2; }
// Weight grad: boxes of 64 rows of 128 bytes for each pair of epilogue warps. A TMA
// instruction costs the loads' engine about 100 clocks whatever it moves: with boxes of 16 rows 24,576
// rows over 32 experts took 904 us.
constexpr int kRowBuf = 64 * 128;
__host__ __device__ constexpr int out_bytes(int mode) { return by_rows(mode) ? 4 * row_bufs(mode) * kRowBuf : 2 * kOutBufs * kOutBuf; }
__host__ __device__ constexpr int smem_bytes(int mode) {
  return stages(mode) * 2 * kTile + out_bytes(mode) + teams(mode) * kRaw;
}
__host__ __device__ constexpr int threads(int mode) { return 32 * (4 + kEpiWarps + kTeamWarps * teams(mode)); }

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
  int tma_out;               // whether maps.o describes the output
  int chunk;                 // stages that one accumulator adds up (see "Long sums")
};

// A stage's four MMAs (16 of l each) and the commit that frees its slot, issued by the lane with
// lead != 0 of a converged warp: with the whole warp in the issue loop the descriptors stay in
// uniform registers, and with predicates instead of branches nothing stands between the MMAs.
// (The loop is what bounds the kernel where it is longer than the MMAs it issues. Measured on
// GB300 without any loads, clocks a stage: run by lane 0 alone, which moves every descriptor
// over, 830; whole warp, a branch in front of each MMA, 900; predicates, 590; one block, 460; no
// vote on the waits, 410.) acc: whether the first MMA adds to the accumulator; left: rows of l that count, the
// MMAs past them are off (kTail).
template <bool kTail>
__device__ __forceinline__ void mma_stage(uint32_t d, const uint64_t (&a)[4], const uint64_t (&b)[4], uint32_t idesc,
                                          uint32_t acc, int left, uint32_t lead, uint32_t empty_bar) {
  if constexpr (kTail) {
    asm volatile(
        "{\n .reg .pred p, q, q1, q2, q3;\n setp.ne.b32 p, %10, 0;\n setp.ne.b32 q, %12, 0;\n"
        " setp.gt.and.s32 q1, %11, 16, q;\n setp.gt.and.s32 q2, %11, 32, q;\n setp.gt.and.s32 q3, %11, 48, q;\n"
        " @q tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %5, %9, p;\n"
        " setp.eq.b32 p, 0, 0;\n"
        " @q1 tcgen05.mma.cta_group::2.kind::f16 [%0], %2, %6, %9, p;\n"
        " @q2 tcgen05.mma.cta_group::2.kind::f16 [%0], %3, %7, %9, p;\n"
        " @q3 tcgen05.mma.cta_group::2.kind::f16 [%0], %4, %8, %9, p;\n"
        " @q tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%13], %14;\n}" ::"r"(d),
        "l"(a[0]), "l"(a[1]), "l"(a[2]), "l"(a[3]), "l"(b[0]), "l"(b[1]), "l"(b[2]), "l"(b[3]), "r"(idesc), "r"(acc),
        "r"(left), "r"(lead), "r"(empty_bar), "h"((uint16_t)0x3)
        : "memory");
  } else {
    asm volatile(
        "{\n .reg .pred p, q;\n setp.ne.b32 p, %10, 0;\n setp.ne.b32 q, %11, 0;\n"
        " @q tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %5, %9, p;\n"
        " setp.eq.b32 p, 0, 0;\n"
        " @q tcgen05.mma.cta_group::2.kind::f16 [%0], %2, %6, %9, p;\n"
        " @q tcgen05.mma.cta_group::2.kind::f16 [%0], %3, %7, %9, p;\n"
        " @q tcgen05.mma.cta_group::2.kind::f16 [%0], %4, %8, %9, p;\n"
        " @q tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%12], %13;\n}" ::"r"(d),
        "l"(a[0]), "l"(a[1]), "l"(a[2]), "l"(a[3]), "l"(b[0]), "l"(b[1]), "l"(b[2]), "l"(b[3]), "r"(idesc), "r"(acc),
        "r"(lead), "r"(empty_bar), "h"((uint16_t)0x3)
        : "memory");
  }
}
__device__ __forceinline__ void commit_pair_lead(uint32_t bar, uint32_t lead) {
  asm volatile(
      "{\n .reg .pred q;\n setp.ne.b32 q, %2, 0;\n"
      " @q tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;\n}" ::"r"(
          bar),
      "h"((uint16_t)0x3), "r"(lead)
      : "memory");
}
__device__ __forceinline__ uint32_t elect_one() {
  uint32_t r;
  asm volatile("{\n .reg .pred q;\n elect.sync _|q, 0xffffffff;\n selp.u32 %0, 1, 0, q;\n}" : "=r"(r));
  return r;
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

// Handing operand tiles that ordinary stores have touched (decoded codes, zeroed lines) to the
// pair's MMA issuer: every writing thread fences its stores into the async proxy, which waits
// until they are performed in this SM's shared memory, the warp converges, and one lane arrives
// on the first CTA's barrier. Each SM's tensor core reads its operands from its own shared
// memory, so nothing has to become visible in the other SM but the arrival, and the arrival
// needs no cluster-scope release. That release waits for global memory: with it the decode of
// 24,576 rows over 32 experts, 4096 x 7168, took 2,007 us instead of 1,342.
__device__ __forceinline__ void fence_async_shared() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }
__device__ __forceinline__ void hand_over(uint64_t* full, int lane) {
  fence_async_shared();
  __syncwarp();
  if (lane == 0) mbar_arrive_cluster(mapa_shared(smem_u32(full), 0));
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

__device__ __forceinline__ void tma_store_3d(const CUtensorMap* map, uint32_t src, int x, int y, int z) {
  asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.bulk_group [%0, {%2, %3, %4}], [%1];" ::"l"(
                   reinterpret_cast<uint64_t>(map)),
               "r"(src), "r"(x), "r"(y), "r"(z)
               : "memory");
}
// fp32 boxes added to memory, each element once (an fp32 sum rounded to nearest)
__device__ __forceinline__ void tma_add_3d(const CUtensorMap* map, uint32_t src, int x, int y, int z) {
  asm volatile("cp.reduce.async.bulk.tensor.3d.global.shared::cta.add.bulk_group [%0, {%2, %3, %4}], [%1];" ::"l"(
                   reinterpret_cast<uint64_t>(map)),
               "r"(src), "r"(x), "r"(y), "r"(z)
               : "memory");
}

// 32 columns d[0..31] of this lane's m into out[j * ld + m], j < cols, m < m_dim, or (`add`) added
// to it in fp32 and rounded once. 16-bit types: neighbouring lanes trade every second column, so that each stores two adjacent m of one column
// as one word (where `words` says that rows keep 4-byte alignment).
template <typename Elem>
__device__ __forceinline__ void store_columns(typename Elem::T* out, int64_t ld, const float (&d)[32], int cols, int m,
                                              int m_dim, int lane, bool words, bool add) {
  using T = typename Elem::T;
  if (sizeof(T) == 2 && words && !add) {
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
#pragma unroll
    for (int j0 = 0; j0 < 32; j0 += 8) {
      float old[8] = {};
      if (add) {
#pragma unroll
        for (int j = 0; j < 8; ++j) old[j] = j0 + j < cols ? Elem::get(o[(j0 + j) * ld]) : 0.0f;
      }
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (j0 + j < cols) o[(j0 + j) * ld] = Elem::put(add ? old[j] + d[j0 + j] : d[j0 + j]);
    }
  }
}

// d[0 .. cols - 1] (32 at most) along a row, added to what is there (in fp32, rounded once) or in its place
template <typename Elem>
__device__ __forceinline__ void store_row(typename Elem::T* o, const float (&d)[32], int cols, bool add) {
  const bool vec = (uintptr_t)o % 16 == 0;
#pragma unroll
  for (int j0 = 0; j0 < 32; j0 += 8) {
    const int n = cols - j0;
    if (n <= 0) break;
    float v[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = d[j0 + j];
    if (add) {
      float old[8];
      raw_get8<Elem>(raw_load8<Elem>(o + j0, vec, n), old);
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] += old[j];
    }
    elem_store8<Elem>(o + j0, vec, n, v);
  }
}

// Tensor maps: A, the output, and B (K-major: boxes of 16, 32, .. 128 rows, half of a column tile's
// width each, since what a wider box brings along costs as much as what is used; else one map).
struct Maps {
  CUtensorMap a, o, b[8];
};

// Register splits (setmaxnreg). Sums in registers: 384 threads launch with 168 each; the control
// warpgroup keeps 80, the two epilogue warpgroups take 208. From saved rows 768 (long
// segments: 896) threads launch with 80 (72): control keeps 56, the epilogue takes 96, the decoding
// warpgroups, a team each, keep 72 (64).
template <int MODE, bool kSum>
struct Regs {
  static constexpr bool kSplit = kSum || is_saved(MODE);
  static constexpr int kCtl = is_saved(MODE) ? 56 : 80, kEpi = is_saved(MODE) ? 96 : 208, kDec = MODE == kWeightGradSavedLong ? 64 : 72;
  static constexpr int kNeeded = 128 * kCtl + 256 * kEpi + 128 * teams(MODE) * kDec;
};
constexpr int kSumStages = 8, kSumStages16 = 32, kAddStages = 16, kHoldStages = 64, kNoChunk = 0x3fffffff;
// The accumulator in turn: its index, the phase of its barriers, and, after the last one, the phase
// of its last use. They alternate; with kHold a unit may go on with the one that it has.
template <bool kHold>
struct Turn {
  uint32_t n = 0;
  __device__ __forceinline__ uint32_t at() const { return n & 1; }
  __device__ __forceinline__ uint32_t phase() const { return (n >> 1) & 1; }
  __device__ __forceinline__ void next(bool) { ++n; }
  __device__ __forceinline__ bool used(uint32_t b) const { return b < n; }
  __device__ __forceinline__ uint32_t last(uint32_t b) const { return ((n - 1 - ((n - 1 - b) & 1)) >> 1) & 1; }
};
template <>
struct Turn<true> {
  uint32_t b = 0, odd = 0, any = 0;  // bit i: uses of accumulator i mod 2, whether it was used
  __device__ __forceinline__ uint32_t at() const { return b; }
  __device__ __forceinline__ uint32_t phase() const { return odd >> b & 1; }
  __device__ __forceinline__ void next(bool stay) {
    odd ^= 1u << b;
    any |= 1u << b;
    if (!stay) b ^= 1;
  }
  __device__ __forceinline__ bool used(uint32_t i) const { return any >> i & 1; }
  __device__ __forceinline__ uint32_t last(uint32_t i) const { return (odd >> i & 1) ^ 1; }
};
// rows of a call up to which a 16-bit weight gradient stays in one accumulator
constexpr int64_t plain_rows(int32_t out_dtype) { return out_dtype == FTMOE_OUT_FP16 ? 4096 : 32768; }

template <int MODE, bool kSum>
__global__ void __launch_bounds__(threads(MODE), 1)
    tc_matmul16_kernel(const __grid_constant__ Maps maps, Params p) {
  constexpr bool kWG = is_wgrad(MODE), kSaved = is_saved(MODE), kRows = by_rows(MODE);
  constexpr bool kHold = kSum && kSaved, kInRegs = kSum && !kSaved;  // where long sums are added up
  constexpr int kTeams = teams(MODE), kRawSlots = kTeams > 0 ? kTeams : 1, kRowBufs = row_bufs(MODE);
  constexpr int S = stages(MODE), kStage = 2 * kTile;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* tiles = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
  uint8_t* outbuf = tiles + (size_t)S * kStage;  // [2 halves of the epilogue][kOutBufs], or [warp pairs][2], boxes
  uint8_t* raws = outbuf + out_bytes(MODE);      // saved rows: [kRawSlots] codes
  // product and input grad: [E + 1] segment offsets, cut to [0, rows]; [E + 1] units before expert e
  int* seg = reinterpret_cast<int*>(raws);
  int* cum = seg + p.E + 1;
  __shared__ __align__(8) uint64_t full[S], empty[S], lfull[S], tfull[2], tempty[2];
  __shared__ __align__(8) uint64_t rfull[kRawSlots], rempty[kRawSlots];  // saved rows: codes landed, codes taken
  __shared__ uint32_t s_tmem;
  __shared__ volatile int s_abort;

  const int warp = __shfl_sync(0xffffffffu, (int)(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;
  const uint32_t crank = cluster_rank();
  const int MB = (p.m_dim + kM - 1) / kM;
  const int CB = kWG ? (p.c_dim + kN - 1) / kN : 0;

  if (threadIdx.x < (kWG ? 3 : 10))  // the descriptors are fetched while the rest is set up
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&maps) + threadIdx.x * sizeof(CUtensorMap)) : "memory");
  if (threadIdx.x == 0) {
    s_abort = 0;
    for (int i = 0; i < S; ++i) {
      // weight grad: two arrivals of the first CTA's producer, or (a segment's last stage) one
      // of each CTA's tail warp; saved rows: the decoding warps of both CTAs and the first
      // CTA's producer
      mbar_init(smem_u32(&full[i]), kSaved ? 2 * kTeamWarps + 1 : kWG ? 2 : 1);
      mbar_init(smem_u32(&empty[i]), 1);
      mbar_init(smem_u32(&lfull[i]), 1);
    }
    for (int i = 0; i < kRawSlots; ++i) {
      mbar_init(smem_u32(&rfull[i]), 1);
      mbar_init(smem_u32(&rempty[i]), kTeamWarps);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_u32(&tfull[i]), 1);
      mbar_init(smem_u32(&tempty[i]), 2 * kEpiWarps);
    }
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&s_tmem)), "r"(512));
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;");
  }
  // everything so far overlaps the end of the previous kernel, whose results are complete from here on
  pdl_wait();
  pdl_trigger();
  auto cut = [&](int v) { return v < 0 ? 0 : v > p.rows ? (int)p.rows : v; };
  if constexpr (!kWG)
    for (int e = threadIdx.x; e <= p.E; e += blockDim.x) seg[e] = cut(__ldg(p.offsets + e));
  // (weight grad: one expert has many units in a row, its offsets stay in L1)
  auto bounds = [&](int e, int& lo, int& hi) {
    lo = kWG ? cut(__ldg(p.offsets + e)) : seg[e];
    hi = max(lo, kWG ? cut(__ldg(p.offsets + e + 1)) : seg[e + 1]);
  };

  __syncthreads();
  if constexpr (!kWG) {
    if (warp == 0) {
      // (64-bit, and cut off at the largest int: overlapping segments can count rows many times)
      long long run = 0;
      for (int base = 0; base < p.E; base += 32) {
        const int e = base + lane;
        long long u = 0;
        if (e < p.E) {
          int lo, hi;
          bounds(e, lo, hi);
          u = (long long)((hi - lo + kN - 1) / kN) * MB;
        }
        long long inc = u;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const long long t = __shfl_up_sync(0xffffffffu, inc, o);
          if (lane >= o) inc += t;
        }
        if (e < p.E) cum[e] = (int)min(run + inc - u, (long long)0x7fffffff);
        run += __shfl_sync(0xffffffffu, inc, 31);
      }
      if (lane == 0) cum[p.E] = (int)min(run, (long long)0x7fffffff);
    }
  }
  fence_before();
  cluster_sync();  // both CTAs' barriers are initialised before either reports to the other
  fence_after();
  const uint32_t tmem_base = s_tmem;
  const int u_end = kWG ? p.E * MB * CB : cum[p.E];
  const int u_begin = (int)cluster_id_x(), u_step = (int)cluster_count_x();

  auto decode = [&](int u, Unit& t) {
    if constexpr (kWG) {
      // Units of one expert adjacent: they read the same rows.
      t.e = u / (MB * CB);
      int lo, hi;
      bounds(t.e, lo, hi);
      t.l0 = lo;
      t.len = hi - lo;
      int local = u - t.e * MB * CB;
      if (t.len > kSquareRows) {
        // bound by what it reads: eight blocks of m at a time, m innermost, so that the pairs at
        // work cover a near square: 8 + 10 tiles of 7,168 columns, not 3 + 28
        const int group = local / (8 * CB), width = min(8, MB - 8 * group);
        local -= group * 8 * CB;
        t.m0 = (8 * group + local % width) * kM;
        t.c0 = local / width * kN;
      } else {
        // whole rows of dw at a time (32 experts of 768 rows: 849 us, in squares 875; one of
        // 24,576 rows: 755 us, in squares 706)
        t.m0 = local / CB * kM;
        t.c0 = local % CB * kN;
      }
      t.cols = min(kN, p.c_dim - t.c0);
    } else {
      int a = 0, b = p.E - 1;
      while (a < b) {  // the last expert whose units begin at or before u
        const int mid = (a + b + 1) >> 1;
        if (cum[mid] <= u) a = mid; else b = mid - 1;
      }
      t.e = a;
      int lo, hi;
      bounds(a, lo, hi);
      const int nt = (hi - lo + kN - 1) / kN, local = u - cum[a];
      const int per = ((hi - lo + nt - 1) / nt + 31) & ~31;
      t.m0 = local / nt * kM;
      t.c0 = lo + local % nt * per;
      t.cols = min(per, hi - t.c0);
      t.l0 = 0;
      t.len = p.l_dim;
    }
    // (saved rows: each CTA's half starts on a 32-wide scale group)
    t.n = kSaved ? (t.cols + 63) & ~63 : (t.cols + 31) & ~31;
  };
  // A unit whose parts all go through one accumulator while the other holds their sum. The MMAs leave
  // the other alone until the last part, and with it the sum, has been read: the unit after begins
  // with the first one again.
  auto hold = [&](const Unit& t) { return kHold && (t.len + kBK - 1) / kBK > p.chunk; };

  if (warp < 4) {
  using R = Regs<MODE, kSum>;
  if constexpr (R::kSplit) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(R::kCtl));
  if (warp == 0) {
    // ------------------------------- TMA producer -------------------------------
    if (lane == 0) {
      uint32_t it = 0, tails = 0, tail_ph = 0;  // bit st: slot st's last use was a tail; uses of lfull[st], mod 2
      for (int64_t u = u_begin; u < u_end && !s_abort; u += u_step) {
        Unit t;
        decode((int)u, t);
        const int half = t.n >> 1;  // of c in each CTA
        const int steps = (t.len + kBK - 1) / kBK;
        const int cb = t.c0 + (int)crank * half, ma = t.m0 + (int)crank * 128;
        const CUtensorMap* mb = &maps.b[kWG ? 0 : half / 16 - 1];
        const uint32_t bytes_b = kWG ? (half > 64 ? kTile : kTile / 2) : (uint32_t)half * 128;
        const uint32_t bytes = kTile + (kSaved ? 0 : bytes_b);
        for (int s = 0; s < steps; ++s, ++it) {
          const int st = it % S;
          if (!mbar_wait(smem_u32(&empty[st]), ((it / S) & 1) ^ 1, &s_abort)) break;
          const uint32_t ta = smem_u32(tiles + (size_t)st * kStage), tb = ta + kTile;
          const bool tail = kWG && t.len - s * kBK < kBK;
          // a tail lands on this CTA's own barrier, everything else on the first CTA's
          const uint32_t bar = tail ? smem_u32(&lfull[st]) : mapa_shared(smem_u32(&full[st]), 0);
          tails = tail ? tails | (1u << st) : tails & ~(1u << st);
          if (tail) {
            mbar_expect_tx(bar, bytes);
            tail_ph ^= 1u << st;
            if (kSaved && crank == 0) mbar_arrive(smem_u32(&full[st]));
          } else if (crank == 0) {
            mbar_expect_tx(smem_u32(&full[st]), 2 * bytes);
            if (kWG && !kSaved) mbar_arrive(smem_u32(&full[st]));
          }
          if constexpr (kWG) {
            const int l = t.l0 + s * kBK;
            tma_pair_2d(ta, &maps.a, bar, ma, l);
            tma_pair_2d(ta + kTile / 2, &maps.a, bar, ma + 64, l);
            if constexpr (!kSaved) {
              tma_pair_2d(tb, mb, bar, cb, l);
              if (half > 64) tma_pair_2d(tb + kTile / 2, mb, bar, cb + 64, l);
            }
          } else {
            if constexpr (MODE == kProduct) {
              tma_pair_3d(ta, &maps.a, bar, s * kBK, ma, t.e);
            } else {
              tma_pair_3d(ta, &maps.a, bar, ma, s * kBK, t.e);
              tma_pair_3d(ta + kTile / 2, &maps.a, bar, ma + 64, s * kBK, t.e);
            }
            tma_pair_2d(tb, mb, bar, s * kBK, cb);
          }
        }
      }
      // Loads still in flight after an abort (bounded): tails land on this CTA's barriers, the
      // rest on the first CTA's, which the second outlives no longer than the closing cluster
      // barrier.
      for (int st = 0; st < S && (uint32_t)st < it; ++st) {
        const uint32_t last = it - 1 - ((it - 1 - st) % S);
        const bool on_local = tails >> st & 1;
        if (!on_local && crank != 0) continue;
        const uint32_t bar = on_local ? smem_u32(&lfull[st]) : smem_u32(&full[st]);
        const uint32_t ph = on_local ? (tail_ph >> st & 1) ^ 1 : (last / S) & 1;
        // (saved rows: a full barrier whose decoders have left never completes; a millisecond is
        // ample for the copies themselves)
        const unsigned long long limit = kSaved && s_abort ? 1000000ull : kTimeoutNs;
        const unsigned long long t0 = globaltimer();
        while (!mbar_try_wait(bar, ph) && globaltimer() - t0 < limit) {
        }
      }
    }
  } else if (warp == 1) {
    // -------------------------------- MMA issuer --------------------------------
    // The whole warp runs the loop, one elected lane issues. Nothing in it needs the warp together
    // (a vote on each wait cost 50 clocks a stage): after a wait that ran out the lanes leave one by
    // one, as each sees the abort flag.
    if (crank == 0) {
      const uint32_t lead = elect_one();
      Turn<kHold> acc;
      uint32_t st = 0, ph = 0;  // the ring's slot and its phase
      // low words of the operands' descriptors for slot 0; a slot and 16 of l further on
      const uint64_t a0 = MODE == kProduct ? smem_desc_sw128(smem_u32(tiles)) : smem_desc_mn_sw128(smem_u32(tiles));
      const uint64_t b0 = kWG ? smem_desc_mn_sw128(smem_u32(tiles) + kTile) : smem_desc_sw128(smem_u32(tiles) + kTile);
      constexpr uint32_t kSlot = kStage >> 4, kStepA = (MODE == kProduct ? 32 : 2048) >> 4, kStepB = (kWG ? 2048 : 32) >> 4;
      const uint32_t full0 = smem_u32(&full[0]), empty0 = smem_u32(&empty[0]);
      bool ok = true;
      for (int64_t u = u_begin; u < u_end && ok; u += u_step) {
        Unit t;
        decode((int)u, t);
        const uint32_t idesc = (1u << 4) | ((uint32_t)p.bf16 << 7) | ((uint32_t)p.bf16 << 10) |
                               (MODE == kProduct ? 0u : 1u << 15) | (kWG ? 1u << 16 : 0u) |
                               ((uint32_t)(t.n >> 3) << 17) | ((uint32_t)(kM >> 4) << 24);
        int left = t.len, part = 0;
        const bool stay = hold(t);
        uint32_t d = 0;
        while (left > 0) {
          if (part == 0) {  // a free accumulator
            ok = mbar_wait(smem_u32(&tempty[acc.at()]), acc.phase() ^ 1, &s_abort);
            if (!ok) break;
            d = tmem_base + acc.at() * kN;
          }
          const uint32_t bar = full0 + 8 * st;
          ok = kWG ? wait_cluster(bar, ph, &s_abort) : mbar_wait(bar, ph, &s_abort);
          if (!ok) break;
          fence_after();
          uint64_t da[4], db[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            da[j] = a0 + st * kSlot + j * kStepA;
            db[j] = b0 + st * kSlot + j * kStepB;
          }
          mma_stage<kWG>(d, da, db, idesc, (uint32_t)part, left, lead, empty0 + 8 * st);
          left -= kBK;
          if (++st == S) {
            st = 0;
            ph ^= 1;
          }
          if (++part == p.chunk || left <= 0) {
            commit_pair_lead(smem_u32(&tfull[acc.at()]), lead);
            acc.next(stay);
            part = 0;
          }
        }
      }
      // MMAs still running write TMEM: wait (bounded) for the last commit of each accumulator
      for (uint32_t b = 0; b < 2 && acc.used(b); ++b) {
        const unsigned long long t0 = globaltimer();
        while (!mbar_try_wait(smem_u32(&tfull[b]), acc.last(b)) && globaltimer() - t0 < kTimeoutNs) {
        }
      }
    }
  } else if (kWG && !kSaved && warp == 2) {
    // ------------------------- tails of segments -------------------------
    uint32_t it = 0, ph = 0;
    bool ok = true;
    for (int64_t u = u_begin; u < u_end && ok; u += u_step) {
      Unit t;
      decode((int)u, t);
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
        hand_over(&full[st], lane);
      }
      it += steps;
    }
  } else if (kSaved && warp == 2) {
    // ------------------------ saved rows: codes ------------------------
    if (lane == 0) {
      uint32_t it = 0;
      for (int64_t u = u_begin; u < u_end && !s_abort; u += u_step) {
        Unit t;
        decode((int)u, t);
        const int steps = (t.len + kBK - 1) / kBK, cb = t.c0 + (int)crank * (t.n >> 1);
        for (int s = 0; s < steps; ++s, ++it) {
          const int r = it % kRawSlots;
          if (!mbar_wait(smem_u32(&rempty[r]), ((it / kRawSlots) & 1) ^ 1, &s_abort)) break;
          mbar_expect_tx(smem_u32(&rfull[r]), kRaw);
          tma_pair_2d(smem_u32(raws + r * kRaw), &maps.b[0], smem_u32(&rfull[r]), cb, t.l0 + s * kBK);
        }
      }
      for (int r = 0; r < kRawSlots && (uint32_t)r < it; ++r) {  // in flight after an abort
        const uint32_t last = it - 1 - ((it - 1 - r) % kRawSlots);
        const unsigned long long t0 = globaltimer();
        while (!mbar_try_wait(smem_u32(&rfull[r]), (last / kRawSlots) & 1) && globaltimer() - t0 < kTimeoutNs) {
        }
      }
    }
  }
  } else if (warp < 4 + kEpiWarps) {
    // --------------------------------- epilogue ---------------------------------
    using R = Regs<MODE, kSum>;
    if constexpr (R::kSplit) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(R::kEpi));
    // Two groups of four warps take runs of 32 columns in turn. A run goes through shared memory
    // and leaves by TMA. Transposed (product, input grad, fp32 weight grad): boxes of 128 m by 32 c
    // (16 of fp32), 256 or 512 contiguous bytes a row, one for the four warps of a group; a run
    // that ends inside the tile of an expert's rows is stored from registers. By rows (weight
    // grad): boxes of 64 rows of 128 bytes, one for a pair of warps. By rows a lane writes 16
    // bytes to shared memory at a time, transposed 2 or 4; transposed, memory is written in longer
    // rows. Measured on the weight gradient of 64 experts, 2048 x 4096, transposed and by rows, us:
    // bf16, 20 rows each 297, 250; 128 rows 308, 252; 700 rows 460, 473; fp32, 20 rows 355, 371;
    // 128 rows 403, 423; 700 rows 600, 639. So 16-bit gradients of segments of up to 512 rows on
    // average go by rows, others and fp32 ones transposed.
    // (From registers, 64 bytes a row and warp, bf16 at 128 rows took 477.) An unaligned output and
    // a 16-bit accumulation are stored from registers.
    const int ew = warp - 4, quarter = warp & 3, half = ew >> 2;
    const bool leader = quarter == 0 && lane == 0;
    Turn<kHold> acc;
    uint32_t box = 0;  // output boxes so far
    const bool words = p.ld_out % 2 == 0 && p.out_expert % 2 == 0 && reinterpret_cast<uintptr_t>(p.out) % 4 == 0;
    const bool f32 = p.out_dtype == FTMOE_OUT_FP32;
    const bool tma_out = p.tma_out && (!p.accumulate || p.out_dtype == FTMOE_OUT_FP32);
    for (int64_t u = u_begin; u < u_end; u += u_step) {
      Unit t;
      decode((int)u, t);
      const bool none = kWG && t.len == 0;  // an expert without rows: zeros, or nothing to add
      if (none && p.accumulate) continue;
      const int mc = t.m0 + (int)crank * 128, ml = 32 * quarter + lane, m = mc + ml;
      const int64_t first = (int64_t)t.e * p.out_expert + (int64_t)t.c0 * p.ld_out;
      // 32 columns from c on, transposed: written, or (`add`) added to what memory holds
      auto emit_transposed = [&](int c, const float (&d)[32], bool add) {
        const int cols = t.cols - c;
        if (tma_out && (kWG || cols >= 32)) {  // (a weight gradient's edge is clipped by its tensor map)
          const int per = f32 ? 16 : 32;
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            if (h == 1 && per == 32) break;
            // free: the barrier of the box before this one followed the leader's wait for the
            // store that last used this buffer
            uint8_t* ob = outbuf + (kOutBufs * half + box % kOutBufs) * kOutBuf;
            if (f32) {
#pragma unroll
              for (int j = 0; j < 16; ++j) reinterpret_cast<float*>(ob)[j * 128 + ml] = d[16 * h + j];
            } else if (p.out_dtype == FTMOE_OUT_BF16) {
#pragma unroll
              for (int j = 0; j < 32; j += 2) {
                const uint32_t w = pack2<ElemBf16>(d[j], d[j + 1]);
                reinterpret_cast<uint16_t*>(ob)[j * 128 + ml] = (uint16_t)w;
                reinterpret_cast<uint16_t*>(ob)[(j + 1) * 128 + ml] = (uint16_t)(w >> 16);
              }
            } else {
#pragma unroll
              for (int j = 0; j < 32; j += 2) {
                const uint32_t w = pack2<ElemF16>(d[j], d[j + 1]);
                reinterpret_cast<uint16_t*>(ob)[j * 128 + ml] = (uint16_t)w;
                reinterpret_cast<uint16_t*>(ob)[(j + 1) * 128 + ml] = (uint16_t)(w >> 16);
              }
            }
            fence_async_shared();
            // all stores but the latest have read their buffers, the next box's among them
            if (leader) asm volatile("cp.async.bulk.wait_group.read %0;" ::"n"(kOutBufs - 2) : "memory");
            named_bar(1 + half, 128);
            if (leader) {
              const int y = t.c0 + c + 16 * h;
              if (mc < p.m_dim && (!kWG || y < p.c_dim)) {
                if (add)
                  tma_add_3d(&maps.o, smem_u32(ob), mc, y, kWG ? t.e : 0);
                else
                  tma_store_3d(&maps.o, smem_u32(ob), mc, y, kWG ? t.e : 0);
              }
              asm volatile("cp.async.bulk.commit_group;" ::: "memory");
            }
            ++box;
          }
        } else {
          const int64_t o = first + (int64_t)c * p.ld_out;
          if (f32)
            store_columns<ElemF32>(static_cast<float*>(p.out) + o, p.ld_out, d, cols, m, p.m_dim, lane, words, add);
          else if (p.out_dtype == FTMOE_OUT_BF16)
            store_columns<ElemBf16>(static_cast<uint16_t*>(p.out) + o, p.ld_out, d, cols, m, p.m_dim, lane, words, add);
          else
            store_columns<ElemF16>(static_cast<uint16_t*>(p.out) + o, p.ld_out, d, cols, m, p.m_dim, lane, words, add);
        }
      };
      // Weight grad: 32 columns from c on of this warp's 32 rows (lane: row), added to what memory
      // holds or in place of it. A pair of warps fills a box of 64 rows of 128 bytes; 16-bit calls
      // come in twos, an even one fills the rows' first halves, an odd one the second and sends.
      auto emit_rows = [&](int c, const float (&d)[32], bool add) {
        if (tma_out) {  // (edges are clipped by the tensor map)
          const int pair = 2 * half + (quarter >> 1);
          const bool sender = (quarter & 1) == 0 && lane == 0;
          uint8_t* ob = outbuf + (kRowBufs * pair + (int)(box % kRowBufs)) * kRowBuf;
          const bool first_half = !f32 && (c & 32) == 0, sends = !first_half || c + 32 >= t.cols;
          if (f32 || first_half) {
            // the store that last used this buffer has read it
            if (sender) asm volatile("cp.async.bulk.wait_group.read %0;" ::"n"(kRowBufs - 1) : "memory");
            named_bar(3 + pair, 64);
          }
          const uint32_t row = smem_u32(ob) + (32 * (quarter & 1) + lane) * 128;
          if (f32) {
#pragma unroll
            for (int j = 0; j < 8; ++j)
              st_shared_16(row + ((j ^ (lane & 7)) << 4), __float_as_uint(d[4 * j]), __float_as_uint(d[4 * j + 1]),
                           __float_as_uint(d[4 * j + 2]), __float_as_uint(d[4 * j + 3]));
          } else {
            const int j0 = first_half ? 0 : 4;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              uint32_t w[4];
#pragma unroll
              for (int i = 0; i < 4; ++i)
                w[i] = p.out_dtype == FTMOE_OUT_BF16 ? pack2<ElemBf16>(d[8 * j + 2 * i], d[8 * j + 2 * i + 1])
                                                     : pack2<ElemF16>(d[8 * j + 2 * i], d[8 * j + 2 * i + 1]);
              st_shared_16(row + (((j0 + j) ^ (lane & 7)) << 4), w[0], w[1], w[2], w[3]);
            }
          }
          if (sends) {
            fence_async_shared();
            named_bar(3 + pair, 64);
            if (sender) {
              const int x = t.c0 + (f32 ? c : c & ~32), y = mc + 64 * (quarter >> 1);
              if (y < p.m_dim) {
                if (add)
                  tma_add_3d(&maps.o, smem_u32(ob), x, y, t.e);
                else
                  tma_store_3d(&maps.o, smem_u32(ob), x, y, t.e);
              }
              asm volatile("cp.async.bulk.commit_group;" ::: "memory");
            }
            ++box;
          }
        } else if (m < p.m_dim) {
          const int64_t o = (int64_t)t.e * p.out_expert + (int64_t)m * p.ld_out + t.c0 + c;
          const int cols = t.cols - c;
          if (f32)
            store_row<ElemF32>(static_cast<float*>(p.out) + o, d, cols, add);
          else if (p.out_dtype == FTMOE_OUT_BF16)
            store_row<ElemBf16>(static_cast<uint16_t*>(p.out) + o, d, cols, add);
          else
            store_row<ElemF16>(static_cast<uint16_t*>(p.out) + o, d, cols, add);
        }
      };
      auto emit = [&](int c, const float (&d)[32], bool add) {
        if constexpr (kRows)
          emit_rows(c, d, add);
        else
          emit_transposed(c, d, add);
      };
      // the first column of this half's i-th run of 32 (by rows: runs in pairs)
      auto column = [&](int i) { return kRows ? 64 * half + 128 * (i >> 1) + 32 * (i & 1) : 32 * half + 64 * i; };
      auto wait_acc = [&]() {
        const int got = mbar_wait(smem_u32(&tfull[acc.at()]), acc.phase(), &s_abort) ? 1 : 0;
        // the group's warps share barriers in emit: they leave together
        const bool left = named_bar_or(1 + half, 128, got == 0);
        fence_after();
        return !left;
      };
      auto release_acc = [&]() {  // this warp's last read of the accumulator: it goes back to the MMAs
        fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_cluster(mapa_shared(smem_u32(&tempty[acc.at()]), 0));
      };
      const uint32_t lanes = tmem_base + ((uint32_t)(32 * quarter) << 16);
      const int parts = none ? 1 : ((t.len + kBK - 1) / kBK + p.chunk - 1) / p.chunk;
      if constexpr (kInRegs) {
        float sum[4][32];
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int j = 0; j < 32; ++j) sum[i][j] = 0.0f;
        bool ok = true;
        for (int q = 0; q < parts && !none; ++q, acc.next(false)) {
          ok = wait_acc();
          if (!ok) break;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int c = column(i);
            if (c < t.cols) {
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                float d[16];
                tmem_ld<16>(lanes + acc.at() * kN + c + 16 * h, d);
                tmem_ld_wait();
#pragma unroll
                for (int j = 0; j < 16; ++j) sum[i][16 * h + j] += d[j];
              }
            }
          }
          release_acc();
        }
        if (!ok) break;
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (column(i) < t.cols) emit(column(i), sum[i], p.accumulate != 0);
      } else {
        const bool stay = hold(t);
        bool ok = true;
        for (int q = 0; q < parts; ++q) {
          if (!none) {
            ok = wait_acc();
            if (!ok) break;
          }
          // a part is added to what the parts before it have left in memory
          if (!kHold && q > 0 && lane == 0) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
          bool held = !none;
          for (int i = 0; i < 4; ++i) {
            const int c = column(i);
            if (c >= t.cols) break;
            float d[32];
            if (none) {
#pragma unroll
              for (int j = 0; j < 32; ++j) d[j] = 0.0f;
            } else {
              tmem_ld<32>(lanes + acc.at() * kN + c, d);
              tmem_ld_wait();
              if constexpr (kHold) {
                const uint32_t sum = lanes + (acc.at() ^ 1) * kN + c;
                if (q > 0) {
#pragma unroll
                  for (int h = 0; h < 2; ++h) {
                    float v[16];
                    tmem_ld<16>(sum + 16 * h, v);
                    tmem_ld_wait();
#pragma unroll
                    for (int j = 0; j < 16; ++j) d[16 * h + j] += v[j];
                  }
                }
                if (q < parts - 1) {
                  uint32_t w[32];
#pragma unroll
                  for (int j = 0; j < 32; ++j) w[j] = __float_as_uint(d[j]);
                  tmem_st16(sum, w);
                  tmem_st16(sum + 16, w + 16);
                  tmem_st_wait();
                }
              }
              if (i == 3 || column(i + 1) >= t.cols) {
                release_acc();
                held = false;
              }
              if (kHold && q < parts - 1) continue;
            }
            emit(c, d, p.accumulate != 0 || (!kHold && q > 0));
          }
          if (held) release_acc();  // no column of this unit was this warp's
          if (!none) acc.next(stay);
        }
        if (!ok) break;
      }
    }
    // (their shared memory has been read; the writes complete with the kernel)
    if (lane == 0) asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
  } else if constexpr (kSaved) {
    // ------------------------ saved rows: decode ------------------------
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(Regs<MODE, kSum>::kDec));
    // Teams of four warps take stages in turn, so that some decode while others wait for
    // codes, for a free operand slot or for their stores to be visible. Thread (warp dw of the
    // team, lane): lines r0 + 16 v of the stage's 64, r0 = 8 dw + lane % 8, and the 32-wide group
    // lane / 8 of their 128 codes. Eight lanes with consecutive lines touch eight different
    // 16-byte columns of the swizzled lines, reading and writing.
    const int dw = (warp - 4 - kEpiWarps) % kTeamWarps, team = (warp - 4 - kEpiWarps) / kTeamWarps;
    const int r0 = 8 * dw + (lane & 7), grp = lane >> 3;
    constexpr int kLines = 64 / (8 * kTeamWarps);
    const int kg = p.c_dim / kMxBlock;
    uint32_t it = 0, tph = 0;  // tph, bit st: uses of lfull[st], mod 2 (every team counts them all)
    bool ok = true;
    for (int64_t u = u_begin; u < u_end && ok; u += u_step) {
      Unit t;
      decode((int)u, t);
      const int steps = (t.len + kBK - 1) / kBK;
      const int g = (t.c0 + (int)crank * (t.n >> 1)) / kMxBlock + grp;
      // scale bytes, fetched one of the team's stages ahead of their codes
      uint32_t next = 0;
      auto fetch = [&](int s) {
        next = 0;
#pragma unroll
        for (int v = 0; v < kLines; ++v) {
          const int l = s * kBK + r0 + 8 * kTeamWarps * v;
          const uint32_t b = g < kg && l < t.len ? (uint32_t)__ldg(p.x_scales + (int64_t)(t.l0 + l) * kg + g) : 0u;
          next |= b << (8 * v);
        }
      };
      int s = (int)((team + kTeams - it % kTeams) % kTeams);
      fetch(s);
      const bool ragged = t.len % kBK != 0;
      for (; s < steps; s += kTeams) {
        const uint32_t i = it + s, scales = next;
        const int st = i % S, raw_slot = i % kRawSlots;
        fetch(s + kTeams);
        const bool tail = ragged && s == steps - 1;
        const int left = t.len - s * kBK;
        ok = mbar_wait(smem_u32(&rfull[raw_slot]), (i / kRawSlots) & 1, &s_abort);
        // the operand slot is free (its last MMAs have read it)
        ok = ok && mbar_wait(smem_u32(&empty[st]), ((i / S) & 1) ^ 1, &s_abort);
        // and dy's rows of a last stage are in place, to be cut off below
        if (tail) ok = ok && mbar_wait(smem_u32(&lfull[st]), tph >> st & 1, &s_abort);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        const uint32_t ta = smem_u32(tiles + (size_t)st * kStage), tb = ta + kTile, raw = smem_u32(raws + raw_slot * kRaw);
        // (the element type is chosen outside the loops)
        auto lines = [&](auto elem) {
          using Elem = decltype(elem);
#pragma unroll 2
          for (int v = 0; v < kLines; ++v) {
            const int r = r0 + 8 * kTeamWarps * v;
            const bool live = r < left;
            const float sc = e8m0_to_f((uint8_t)(scales >> (8 * v)));
            // columns 32 grp + 16 h .. + 15: two 16-byte columns of the line in box grp / 2
            const uint32_t line = tb + (grp >> 1) * (kTile / 2) + r * 128;
            uint4 c[2];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              c[h] = ld_shared_16(raw + r * 128 + (((2 * grp + h) ^ (r & 7)) << 4));
              if (!live) c[h] = make_uint4(0u, 0u, 0u, 0u);  // (a code past the segment may be NaN)
            }
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const uint32_t cw[4] = {c[h].x, c[h].y, c[h].z, c[h].w};
              uint32_t o[8];
#pragma unroll
              for (int k = 0; k < 8; ++k) {
                const uint32_t two = (cw[k >> 1] >> (16 * (k & 1))) & 0xffffu;
                const __half2_raw hr = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)two, __NV_E4M3);
                const float2 f = __half22float2(__half2(hr));
                float lo, hi;
                (F32Pair(f.x, f.y) * F32Pair(sc)).get(lo, hi);
                o[k] = pack2<Elem>(lo, hi);
              }
              const int col = (grp & 1) * 4 + 2 * h;
              st_shared_16(line + ((col ^ (r & 7)) << 4), o[0], o[1], o[2], o[3]);
              st_shared_16(line + (((col + 1) ^ (r & 7)) << 4), o[4], o[5], o[6], o[7]);
            }
          }
        };
        if (p.bf16)
          lines(ElemBf16{});
        else
          lines(ElemF16{});
        if (tail) {
#pragma unroll
          for (int v = 0; v < kLines; ++v) {
            const int r = r0 + 8 * kTeamWarps * v;
            if (r < left) continue;
            // dy's line past the segment's end: this thread's quarter of both 64-column boxes
            const uint32_t line = ta + r * 128;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const int chunk = grp * 4 + k;
              st_shared_16(line + (chunk >> 3) * (kTile / 2) + ((chunk & 7) << 4), 0, 0, 0, 0);
            }
          }
        }
        hand_over(&full[st], lane);
        if (lane == 0) mbar_arrive(smem_u32(&rempty[raw_slot]));
      }
      if (ragged) tph ^= 1u << ((it + steps - 1) % S);
      it += steps;
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

static bool encode(CUtensorMap* map, const void* base, CUtensorMapDataType type, int rank, const uint64_t* dims,
                   const uint64_t* strides, const uint32_t* box, CUtensorMapSwizzle swizzle) {
  EncodeTiledFn enc = encode_fn();
  if (!enc) return false;
  cuuint64_t d[3], st[2];
  cuuint32_t b[3], es[3] = {1, 1, 1};
  for (int i = 0; i < rank; ++i) d[i] = dims[i], b[i] = box[i];
  for (int i = 0; i + 1 < rank; ++i) st[i] = strides[i];
  return enc(map, type, (cuuint32_t)rank, const_cast<void*>(base), d, st, b, es, CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// operand tiles of 2-byte elements
static bool encode16(CUtensorMap* map, const void* base, int rank, const uint64_t* dims, const uint64_t* strides,
                     const uint32_t* box) {
  return encode(map, base, CU_TENSOR_MAP_DATA_TYPE_UINT16, rank, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B);
}

// Output boxes of `cols` elements by `rows` rows; false (and an unused map) where rows of memory do
// not start on 16-byte boundaries, or do not end on one: a TMA store cut off inside 16 bytes writes
// all of them (measured: seven bf16 past rows of 33).
static bool encode_out(CUtensorMap* map, void* base, int32_t dtype, uint64_t width, uint64_t height, uint64_t E, int64_t ld,
                       int64_t expert, uint32_t cols, uint32_t rows, CUtensorMapSwizzle swizzle) {
  const bool f32 = dtype == FTMOE_OUT_FP32;
  const int64_t b = f32 ? 4 : 2;
  if ((uintptr_t)base % 16 != 0 || ld * b % 16 != 0 || (E > 1 && expert * b % 16 != 0) || width * b % 16 != 0) return false;
  const uint64_t dims[3] = {width, height, E}, st[2] = {(uint64_t)(ld * b), (uint64_t)(E > 1 ? expert * b : ld * b)};
  const uint32_t box[3] = {cols, rows, 1};
  return encode(map, base, f32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_UINT16, 3, dims, st, box, swizzle);
}

template <int MODE, bool kSum>
static cudaError_t launch(const Maps& maps, const Params& p, cudaStream_t st, int* unsupported) {
  const size_t smem = 1024 + (size_t)smem_bytes(MODE) + (is_wgrad(MODE) ? 0 : ((size_t)p.E + 1) * 8);
  int dev = 0;
  cudaGetDevice(&dev);
  // per device: CTA pairs that can be resident at once, with the largest shared memory this
  // kernel asks for (one CTA per SM either way)
  static int pairs[64] = {};
  int np = dev >= 0 && dev < 64 ? pairs[dev] : 0;
  if (np == 0) {
    const size_t most = 1024 + (size_t)smem_bytes(MODE) + (is_wgrad(MODE) ? 0 : (size_t)(kMaxExperts + 1) * 8);
    const cudaError_t e =
        cudaFuncSetAttribute(tc_matmul16_kernel<MODE, kSum>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)most);
    if (e != cudaSuccess) return e;
    np = max_active_clusters(tc_matmul16_kernel<MODE, kSum>, dim3(threads(MODE)), most, 2, 2 * (sm_count() / 2));
    if (np > sm_count() / 2) np = sm_count() / 2;
    if constexpr (Regs<MODE, kSum>::kSplit) {
      // the register split has to fit what the block is launched with
      cudaFuncAttributes fa;
      const cudaError_t ea = cudaFuncGetAttributes(&fa, tc_matmul16_kernel<MODE, kSum>);
      if (ea != cudaSuccess) return ea;
      if (fa.numRegs * threads(MODE) < Regs<MODE, kSum>::kNeeded) np = 0;
    }
    if (dev >= 0 && dev < 64) pairs[dev] = np;
  }
  if (np < 1) {
    *unsupported = 1;
    return cudaSuccess;
  }
  const OverlapLaunch overlap;
  return launch_kernel_cluster(tc_matmul16_kernel<MODE, kSum>, dim3(2 * np), dim3(threads(MODE)), smem, st, true, 2, maps, p);
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
  Maps maps;
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
    if (!encode16(&maps.a, w.w, 3, wd, ws, wb)) return cudaSuccess;
    const uint64_t ad[2] = {(uint64_t)l, R}, as[1] = {2 * (uint64_t)a.ld_a};
    const int widest = (int)(R < 256 ? cdiv(a.rows, 32) : 8);  // no column tile is wider than all rows
    for (int i = 0; i < 8; ++i) {
      const uint32_t ab[2] = {64, 16u * (i + 1)};
      if (i < widest ? !encode16(&maps.b[i], a.a, 2, ad, as, ab) : (maps.b[i] = maps.b[0], false)) return cudaSuccess;
    }
    p.out = a.out;
    p.ld_out = a.ld_out;
    p.m_dim = (int)m;
    p.l_dim = (int)l;
    p.out_dtype = a.out_dtype;
    p.tma_out = encode_out(&maps.o, a.out, a.out_dtype, (uint64_t)m, R, 1, a.ld_out, 0, 128,
                           a.out_dtype == FTMOE_OUT_FP32 ? 16 : 32, CU_TENSOR_MAP_SWIZZLE_NONE);
    if (!p.tma_out) maps.o = maps.a;
    *unsupported = 0;
    p.chunk = a.out_dtype == FTMOE_OUT_FP32 ? kSumStages : kSumStages16;
    if (l > p.chunk * kBK)
      return a.input_grad ? launch<kInputGrad, true>(maps, p, st, unsupported) : launch<kProduct, true>(maps, p, st, unsupported);
    return a.input_grad ? launch<kInputGrad, false>(maps, p, st, unsupported) : launch<kProduct, false>(maps, p, st, unsupported);
  }
  if (!tma16(a.a, a.ld_a) || E * cdiv(w.n, kM) * cdiv(w.k, kN) > 0x7fffffff) return cudaSuccess;
  // see the epilogue: by rows for 16-bit outputs of segments that are short on average
  const bool f32 = w.dtype == FTMOE_OUT_FP32, long_segments = a.rows > E * kSumStages * kBK;
  const bool transposed = !a.x_scales && (f32 || long_segments);
  CUtensorMap &mdy = transposed ? maps.b[0] : maps.a, &mx = transposed ? maps.a : maps.b[0];
  const uint64_t dd[2] = {(uint64_t)w.n, R}, ds[1] = {2 * (uint64_t)a.ld_a};
  const uint32_t box[2] = {64, 64};
  if (!encode16(&mdy, a.a, 2, dd, ds, box)) return cudaSuccess;
  const uint64_t xd[2] = {(uint64_t)w.k, R};
  if (a.x_scales) {
    if ((uintptr_t)a.x % 16 != 0 || a.ld_x % 16 != 0) return cudaSuccess;
    const uint64_t xs[1] = {(uint64_t)a.ld_x};
    const uint32_t xb[2] = {128, 64};
    if (!encode_u8_tmap(&mx, a.x, 2, xd, xs, xb)) return cudaSuccess;
  } else {
    if (!tma16(a.x, a.ld_x)) return cudaSuccess;
    const uint64_t xs[1] = {2 * (uint64_t)a.ld_x};
    if (!encode16(&mx, a.x, 2, xd, xs, box)) return cudaSuccess;
  }
  for (int i = 1; i < 8; ++i) maps.b[i] = maps.b[0];
  p.x_scales = a.x_scales;
  p.out = w.w;
  p.ld_out = w.ld;
  p.out_expert = w.expert_stride;
  p.m_dim = (int)(transposed ? w.k : w.n);
  p.c_dim = (int)(transposed ? w.n : w.k);
  p.out_dtype = w.dtype;
  p.accumulate = a.accumulate;
  p.tma_out = encode_out(&maps.o, w.w, w.dtype, (uint64_t)w.k, (uint64_t)w.n, (uint64_t)E, w.ld, w.expert_stride,
                         transposed ? 128 : f32 ? 32 : 64, !transposed ? 64 : f32 ? 16 : 32,
                         transposed ? CU_TENSOR_MAP_SWIZZLE_NONE : CU_TENSOR_MAP_SWIZZLE_128B);
  if (!p.tma_out) maps.o = maps.a;
  *unsupported = 0;
  p.chunk = f32 ? kAddStages : kNoChunk;
  if (a.x_scales) {
    const bool many = a.rows > E * 256;  // rows per expert
    if (!f32 && a.rows > plain_rows(w.dtype)) {
      p.chunk = kHoldStages;
      return many ? launch<kWeightGradSavedLong, true>(maps, p, st, unsupported)
                  : launch<kWeightGradSaved, true>(maps, p, st, unsupported);
    }
    return many ? launch<kWeightGradSavedLong, false>(maps, p, st, unsupported)
                : launch<kWeightGradSaved, false>(maps, p, st, unsupported);
  }
  // fp32 and short on average: the few segments that are long are added in memory, the rest need
  // neither that nor registers for a sum. 16 bits: see "Long sums".
  if (f32 ? long_segments : a.rows > plain_rows(w.dtype)) {
    p.chunk = f32 ? kSumStages : kSumStages16;
    return transposed ? launch<kWeightGradT, true>(maps, p, st, unsupported) : launch<kWeightGrad, true>(maps, p, st, unsupported);
  }
  return transposed ? launch<kWeightGradT, false>(maps, p, st, unsupported) : launch<kWeightGrad, false>(maps, p, st, unsupported);
}

FTMOE_DEFINE_ERR_READER(read_err_tc_matmul16)

}  // namespace ftmoe
