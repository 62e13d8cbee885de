// E4M3 products with an f32 scale for each block of 128 on CTA pairs (include/mok.h: mok_fp8_matmul,
// mok_fp8_weight_grad):
//   product       out[r][n] = sum_b xs[b][r] ws[e][n / 128][b] (x_b w_b^T)[r][n]     over the rows r of group e
//   weight grad   out[e][n][h] = sum_b ds[b][n] xs[b][h] (dy_b x_b^T)[n][h]        over the 128-row blocks b of group e
// Both are out[col][row] = sum_b s_b (A_b B_b^T) with A's rows the MMA's M (256 a pair tile, 128 a CTA: weights' rows, or
// h) and B's rows its N (a multiple of 16 up to 256: the group's rows, or n), so that a group of few rows pads to 16 only.
//
// The scales are arbitrary f32 numbers and change with each 128 of K, so a block's sum cannot stay in the tensor
// cores: tcgen05.mma.kind::f8f6f4 forms it (four K = 32 steps) in one of two TMEM accumulators of 256 columns, and eight epilogue
// warps add it, scaled, to their f32 sums in registers (128 a thread) while the next block's MMAs run into the other.  They
// read TMEM as 16 lanes x 256 bits: a lane then has two columns of each 8, so that it needs a quarter of the columns' scales, and
// four rows of each column.  With A's rows mixed on the way into shared memory (a five-dimensional tensor map: TMEM lane
// 8 k + u holds row 4 u + k) these four are neighbours in out, stored together.  Tiles of at most 128 (64) columns put two
// (four) blocks into an accumulator and hand them over together.
// What bounds it: few rows a group, DRAM (32 rows on 25 of 64 experts of 7,168 x 2,048 64 us, 5.7 TB/s; 16,384 rows of 128
// experts of 4,096 x 7,168 705 us, 5.7 TB/s).  Many, the epilogue: a block of 256 columns takes its warps about 1,150 cycles
// against 520 of MMAs (8,192^3 534 us, 2.06 PFLOP/s; the MMAs alone 246 us, with their loads 338).
//
// Roles of both CTAs of a pair: warp 0 TMA producer, warp 1 MMA issuer (even CTA), warp 2 the scales, warps 4 to 11 epilogue
// (warp w reads TMEM lane quarter w % 4; the two warps of a quarter take alternate 32-column pieces).  The scales' warp
// reads four blocks' scales at a time, multiplies the two where one is the same for a whole 128-row tile (product; see f8_apart) and puts
// them into a ring in shared memory, in the order in which the epilogue's lanes take them.  All waits and loops are a whole
// warp's, one elected thread issues: addresses and descriptors then stay in uniform registers.  Barriers: full[s] in the even
// CTA (one arrival with both CTAs' bytes), empty[s] and pfull[a] in both (multicast commits), pempty[a] in the even CTA (16
// arrivals), sfull[q] and sempty[q] in each CTA.  Tiles (group, weight tile m, chunk c of the group's rows; c fastest, then
// m) are dealt to the pairs round-robin; where there are few, up to four pairs of a cluster share a tile along K and add
// their sums in order.  Every output element is summed over its blocks in order, so results do not depend on the deal.
// Every wait is bounded.
#include <cuda_bf16.h>

#include <algorithm>
#include <type_traits>

#include "fp8.cuh"
#include "fp8_plan.h"
#include "ptx.cuh"
#include "tmap.cuh"

namespace mok {
namespace {

struct Fp8GemmArgs {
  int E;
  int nkb;                // product: blocks along K
  int NM;                 // A rows of a group: weights' rows, or H
  int NB;                 // weight grad: B rows (n)
  int MT;                 // pair tiles along A's rows
  int nmax;               // columns of a chunk at most (a multiple of 16 up to 256)
  int64_t R;
  int64_t blocks;         // weight grad: 128-row blocks that the operands have
  const int32_t* offsets; // [E+1] or null: one group of R rows
  const float* a_scale;   // product: [E][NM / 128][nkb]; weight grad: [blocks][NM]
  const float* b_scale;   // product: [nkb][b_ld]; weight grad: [blocks][NB]
  int64_t b_ld;
  void* out;
  int64_t ld;             // elements between out's rows
  int mixed;              // TMEM lane 8 k + u of a quarter holds A's row 4 u + k, else the rows are in order
  int packed;             // host: which kernel
  int splits;             // pairs of a cluster, each with its share of a tile's blocks
  uint32_t magic_per, magic_nc;  // f8_divide: tiles of a group and of a column (weight grad), or MT
  int wide_out;           // mixed, and out's rows take four neighbours at once
  int* status;
};

constexpr int F8_STAGES = 6;
constexpr int F8_SLOTS = 3;
constexpr int F8_GROUP = 4;  // K blocks whose scales share a slot
constexpr int F8_A_BYTES = 128 * 128;
constexpr int F8_B_BYTES = 128 * 128;
constexpr int F8_STAGE = F8_A_BYTES + F8_B_BYTES;
// Words of a block in a slot: the columns' scales, and the lanes' (weight grad) or (product) which columns meet the weights'
// scale apart (a bit for each), that scale, and whether there may be any.
constexpr int F8_SLOT_BLOCK = 256 + 128;
constexpr int F8_APART = 256, F8_APART_SCALE = 264, F8_APART_ANY = 265;
constexpr int F8_SLOT = F8_GROUP * F8_SLOT_BLOCK * 4;
constexpr int F8_EPI_WARPS = 8;
constexpr int F8_THREADS = 32 * (4 + F8_EPI_WARPS);
// Registers of a thread: 168 at launch (384 threads of them are the register file); the epilogue's 128 f32 sums
// need more, and the scales' warp of the weight gradient too: 128 x 72 + 256 x 216 = 128 x 88 + 256 x 208 = 384 x 168.
template <bool WGRAD>
struct F8Regs {
  static constexpr int FEW = WGRAD ? 88 : 72, EPI = WGRAD ? 208 : 216;
  static_assert(128 * FEW + 256 * EPI <= F8_THREADS * 168, "register split");
};
constexpr int F8_SMEM_BARS = 512;
constexpr size_t f8_smem(int E) {
  return 1024 + size_t(F8_STAGES) * F8_STAGE + size_t(F8_SLOTS) * F8_SLOT + F8_SMEM_BARS + size_t(3) * (E + 1) * 4;
}
static_assert(f8_smem(FP8_MAX_E) <= 232448, "shared memory");

struct Fp8Tile {
  int e, m;
  int col0, cols, n;  // B's first row, how many there are, padded to the MMA's N
  int kb0, nkb;       // first block of K, number of blocks
};

// g / d by a product with ceil(2^32 / d), which is at most one too much for g below 2^31.
__device__ __forceinline__ int f8_divide(int g, int d, uint32_t magic) {
  if (d == 1) return g;
  const int q = (int)__umulhi((uint32_t)g, magic);
  return q - (q * (int64_t)d > g);
}

// Tile g, by all lanes of a warp together.  s_at / s_cnt (addresses in shared memory): product: first row and rows of
// each group, s_first: chunks before it; weight grad: first block and blocks.  The product's group is the last whose first
// tile is not behind g: 32 entries are looked at at once, first every 32nd.
template <bool WGRAD, bool SPLIT>
__device__ __forceinline__ Fp8Tile f8_tile(int g, int split, const Fp8GemmArgs& a, uint32_t s_at, uint32_t s_cnt,
                                           uint32_t s_first) {
  Fp8Tile t;
  int nc, c, rows;
  if (WGRAD) {
    nc = (a.NB + a.nmax - 1) / a.nmax;
    t.e = f8_divide(g, nc * a.MT, a.magic_per);
    const int l = g - t.e * nc * a.MT;
    t.m = f8_divide(l, nc, a.magic_nc);
    c = l - t.m * nc;
    rows = a.NB;
    t.kb0 = lds1i(s_at + 4 * t.e);
    t.nkb = lds1i(s_cnt + 4 * t.e);
    t.col0 = 0;
  } else {
    const int chunk = f8_divide(g, a.MT, a.magic_per);  // this tile's place among chunks, groups without rows left out
    const int lane = threadIdx.x & 31;
    int lo = 0;
    if (a.E > 32) lo = 32 * (__popc(__ballot_sync(0xffffffffu, lds1i(s_first + 4 * min(32 * lane, a.E)) <= chunk && 32 * lane < a.E)) - 1);
    const int at = lo + lane;
    lo += __popc(__ballot_sync(0xffffffffu, at < a.E && lds1i(s_first + 4 * min(at, a.E)) <= chunk)) - 1;
    t.e = lo;
    const int before = lds1i(s_first + 4 * lo);
    nc = lds1i(s_first + 4 * lo + 4) - before;
    const int l = g - before * a.MT;
    t.m = nc == 1 ? l : l / nc;
    c = l - t.m * nc;
    rows = lds1i(s_cnt + 4 * lo);
    t.kb0 = 0;
    t.nkb = a.nkb;
    t.col0 = lds1i(s_at + 4 * lo);
  }
  if (SPLIT) {
    const int lo = t.nkb * split / a.splits;
    t.kb0 += lo;
    t.nkb = t.nkb * (split + 1) / a.splits - lo;
  }
  const int each = nc == 1 ? rows : ((rows + nc - 1) / nc + 15) & ~15;  // equal chunks
  t.col0 += c * each;
  t.cols = max(0, min(each, rows - c * each));
  t.n = max(16, (t.cols + 15) & ~15);
  return t;
}

// A bounded wait by all lanes of a warp together.  The timer is read only once a wait has gone on for a while: reading
// it takes longer than most waits here do.
__device__ __forceinline__ bool f8_wait(uint32_t bar, uint32_t parity, volatile int* abort_flag, int* status, int site) {
  if (mbar_try_wait(bar, parity)) return true;
  uint64_t t0 = 0;
  uint32_t spins = 0;
#pragma unroll 1
  while (!mbar_try_wait(bar, parity)) {
    if ((++spins & 63u) == 0) {
      if (*abort_flag) return false;
      const uint64_t now = global_timer_ns();
      if (t0 == 0) {
        t0 = now;
      } else if (now - t0 > kWaitLimitNs) {
        *abort_flag = 1;
        report_status(status, MOK_DEV_TIMEOUT, site);
        return false;
      }
    }
  }
  return true;
}

// 32-column pieces of the epilogue warp that has most of them (two warps take turns).
__device__ __forceinline__ int np_of(int n) { return (((n + 31) >> 5) + 1) >> 1; }

// Blocks of K whose sums share an accumulator of 256 columns: narrow tiles hand over several at once, since handing
// over costs the epilogue as much as 128 columns do.
__device__ __forceinline__ int f8_blocks_at_once(int n) { return n <= 64 ? 4 : n <= 128 ? 2 : 1; }

// Where column c (of 32) has its scale: the four columns 8 g + 2 t, + 1 of two neighbouring g that a lane (t = lane % 4) holds
// follow each other.
__device__ __forceinline__ int f8_scale_at(int c) { return (c >> 4) * 16 + ((c >> 1) & 3) * 4 + ((c >> 3) & 1) * 2 + (c & 1); }

// The two scales of a product go to the epilogue as one factor, unless that is no normal f32: it would lose bits that the block's sum
// may still bring back, or be infinite beside a sum of 0.  Such a column keeps its row's scale, and its sums are
// multiplied with the weights' one first ("apart"; to f32's precision for scales from 2^-119 on), which the epilogue does in TMEM before
// it takes them (8,192^3 with all columns apart 1,340 us).  Scales of 0, and the quantisers'
// least one, which stands for zeros (masked tokens' gradients, weights that are off), are left out: what little is lost there
// stays below 2^-125 a block.  At least F8_NORMALS for scales that meet apart.
constexpr uint32_t F8_NORMALS = 0x7f000000u;
__device__ __forceinline__ bool f8_zeros(float scale) { return scale == 0.0f || scale == FP8_LEAST_SCALE; }
__device__ __forceinline__ uint32_t f8_apart(float row, float weights) {
  return f8_zeros(row) || f8_zeros(weights) ? 0 : (__float_as_uint(row * weights) & 0x7fffffffu) - 0x00800000u;
}

__device__ __forceinline__ void f8_put4(float* p, float4 v) { *reinterpret_cast<float4*>(p) = v; }
__device__ __forceinline__ void f8_put4(__nv_bfloat16* p, float4 v) {
  __nv_bfloat162 a = __floats2bfloat162_rn(v.x, v.y), b = __floats2bfloat162_rn(v.z, v.w);
  *reinterpret_cast<uint2*>(p) = make_uint2(*reinterpret_cast<uint32_t*>(&a), *reinterpret_cast<uint32_t*>(&b));
}

__device__ __forceinline__ void f8_put(float* p, float v) { *p = v; }
__device__ __forceinline__ void f8_put(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }

// tmA: A's rows, [groups][NM][K] bytes, boxes of 128 bytes x 128 rows; tmB: B's rows, boxes of 128 bytes x 32 rows.
// PACKED: wide tiles form two sums in one instruction (launch chooses).
template <bool WGRAD, bool SPLIT, bool PACKED, typename OUT>
__global__ void __launch_bounds__(F8_THREADS, 1)
    fp8_gemm_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                    const __grid_constant__ CUtensorMap tmB64, const __grid_constant__ CUtensorMap tmB32,
                    const Fp8GemmArgs args) {
  constexpr int STAGES = F8_STAGES, SLOTS = F8_SLOTS;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t slots0 = smem_u32(smem) + STAGES * F8_STAGE;
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + STAGES * F8_STAGE + SLOTS * F8_SLOT);
  // bars: full, empty [STAGES], pfull, pempty [2], sfull, sempty [SLOTS], drain; the TMEM address; the abort flag
  constexpr int NBARS = 2 * STAGES + 4 + 2 * SLOTS + 1;
  static_assert(NBARS * 8 + 8 <= F8_SMEM_BARS, "barriers");
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + NBARS);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  int* s_at = reinterpret_cast<int*>(reinterpret_cast<uint8_t*>(bars) + F8_SMEM_BARS);
  int* s_cnt = s_at + (args.E + 1);
  int* s_first = s_cnt + (args.E + 1);
  const uint32_t at0 = smem_u32(s_at);

  const int warp = __reduce_max_sync(0xffffffffu, (int)threadIdx.x >> 5);  // uniform, and known to be
  const int lane = threadIdx.x & 31;
  const uint32_t cta = cluster_ctarank(), rank = cta & 1;  // rank 0 issues its pair's MMAs
  const int split = SPLIT ? (int)(cta >> 1) : 0;
  const int pair = SPLIT ? (int)blockIdx.x / (2 * args.splits) : (int)blockIdx.x >> 1;  // with splits: the cluster
  const int npairs = SPLIT ? (int)gridDim.x / (2 * args.splits) : (int)gridDim.x >> 1;
  const uint16_t both = (uint16_t)(3u << (cta & ~1u));
  const uint32_t bars0 = smem_u32(bars);
  auto full_bar = [&](int s) { return bars0 + 8u * s; };
  auto empty_bar = [&](int s) { return bars0 + 8u * (STAGES + s); };
  auto pfull_bar = [&](int a) { return bars0 + 8u * (2 * STAGES + a); };
  auto pempty_bar = [&](int a) { return bars0 + 8u * (2 * STAGES + 2 + a); };
  auto sfull_bar = [&](int q) { return bars0 + 8u * (2 * STAGES + 4 + q); };
  auto sempty_bar = [&](int q) { return bars0 + 8u * (2 * STAGES + 4 + SLOTS + q); };
  const uint32_t drain_bar = bars0 + 8u * (2 * STAGES + 4 + 2 * SLOTS);

  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(full_bar(s), 1);
      mbar_init(empty_bar(s), 1);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(pfull_bar(a), 1);
      mbar_init(pempty_bar(a), 2 * F8_EPI_WARPS);
    }
    for (int q = 0; q < SLOTS; ++q) {
      mbar_init(sfull_bar(q), 1);
      mbar_init(sempty_bar(q), F8_EPI_WARPS);
    }
    mbar_init(drain_bar, 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc_pair(smem_u32(tmem_slot), 512);
    tmem_relinquish_pair();
  }
  if (warp == 0) {
    // the groups' rows and the chunks (weight grad: 128-row blocks) before each: a scan, 32 groups at a time.  A group
    // starts no earlier than those before it end, whatever the table says: the chunks are then at most as many as the
    // host counted.
    int before = 0, row = 0;
    for (int e0 = 0; e0 < args.E; e0 += 32) {
      const int e = e0 + lane;
      int lo = 0, cnt = 0;
      if (e < args.E) {
        if (args.offsets == nullptr) {
          cnt = (int)args.R;
        } else {
          lo = fp8_offset(args.offsets[e], 0, args.R);
          cnt = fp8_offset(args.offsets[e + 1], lo, args.R);  // the end, for now
        }
      }
      int end = max(row, cnt);
#pragma unroll
      for (int s = 1; s < 32; s <<= 1) end = max(end, __shfl_up_sync(0xffffffffu, end, s));
      int start = __shfl_up_sync(0xffffffffu, end, 1);
      if (lane == 0) start = row;
      lo = max(lo, start);
      cnt = max(0, cnt - lo);
      row = __shfl_sync(0xffffffffu, end, 31);
      const int mine = WGRAD ? (cnt + 127) >> 7 : (cnt + args.nmax - 1) / args.nmax;
      int sum = mine;
#pragma unroll
      for (int s = 1; s < 32; s <<= 1) {
        const int o = __shfl_up_sync(0xffffffffu, sum, s);
        if (lane >= s) sum += o;
      }
      const int first = before + sum - mine;
      if (e < args.E) {
        if (WGRAD) {  // a wrong table may count more blocks than there are
          s_at[e] = min(first, (int)args.blocks);
          s_cnt[e] = min(first + mine, (int)args.blocks) - s_at[e];
        } else {
          s_at[e] = lo;
          s_cnt[e] = cnt;
          s_first[e] = first;
        }
      }
      before += __shfl_sync(0xffffffffu, sum, 31);
    }
    if (lane == 0) s_first[args.E] = before;
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();  // both CTAs' barriers are initialised before either signals the other's
  tc_fence_after();
  const uint32_t tmem_base = __reduce_or_sync(0xffffffffu, *tmem_slot);
  const int total = WGRAD ? args.E * args.MT * ((args.NB + args.nmax - 1) / args.nmax) : s_first[args.E] * args.MT;

  bool met = false;  // has been at the two meetings of a split tile's pairs
  if (warp < 4) {
    reg_dec<F8Regs<WGRAD>::FEW>();
    if (warp == 0) {
      // ------------------------------------------------------------------ TMA producer (both CTAs)
      const bool leader = elect_one();
      if (leader) {
        tma_prefetch_desc(&tmA);
        tma_prefetch_desc(&tmB);
      }
      const uint64_t pol_a = l2_policy_evict_normal();
      const uint64_t pol_once = l2_policy_evict_first();
      const uint64_t pol_b = l2_policy_evict_last();  // read by every tile along A's rows
      const uint32_t full0_cl = mapa_shared(full_bar(0), cta & ~1u);
      const uint32_t smem0 = smem_u32(smem);
      int stage = 0, issued = 0;
      uint32_t phase = 0;
      bool ok = true;
      for (int g = pair; g < total && ok; g += npairs) {
        const Fp8Tile t = f8_tile<WGRAD, SPLIT>(g, split, args, at0, at0 + 4 * (args.E + 1), at0 + 8 * (args.E + 1));
        const int half = t.n >> 1;
        // the CTA's rows of B in the fewest boxes of 128, 64 and 32 rows
        const int b128 = half > 96, b64 = !b128 && half > 32, b32 = !b128 && (half <= 32 || half > 64);
        const uint32_t pair_tx = 2u * (F8_A_BYTES + (b128 * 128 + b64 * 64 + b32 * 32) * 128);
        const uint64_t pa = !WGRAD && t.n == 16 ? pol_once : pol_a;
        const int a_row = t.m * 256 + 128 * (int)rank;
        const int b_row = t.col0 + (int)rank * half;
        for (int kb = 0; kb < t.nkb; ++kb) {
          ok = __all_sync(0xffffffffu,
                          f8_wait(empty_bar(stage), phase ^ 1, abort_flag, args.status, SITE_GEMM_PRODUCER_EMPTY));
          if (!ok) break;
          if (leader) {
            const uint32_t fb = full0_cl + 8u * stage;
            const uint32_t sa = smem0 + stage * F8_STAGE;
            const uint32_t sb = sa + F8_A_BYTES;
            if (rank == 0) mbar_arrive_expect_tx(full_bar(stage), pair_tx);
            const int k0 = (t.kb0 + kb) * 128;
            if (args.mixed) tma_load_5d_pair(sa, &tmA, fb, k0, 0, 0, a_row >> 5, WGRAD ? 0 : t.e, pa);
            else tma_load_3d_pair(sa, &tmA, fb, k0, a_row, WGRAD ? 0 : t.e, pa);
            if (b128) tma_load_2d_pair(sb, &tmB, fb, k0, b_row, pol_b);
            if (b64) tma_load_2d_pair(sb, &tmB64, fb, k0, b_row, pol_b);
            if (b32) tma_load_2d_pair(sb + b64 * 64 * 128, &tmB32, fb, k0, b_row + b64 * 64, pol_b);
          }
          __syncwarp();
          ++issued;
          if (++stage == STAGES) {
            stage = 0;
            phase ^= 1;
          }
        }
      }
      if (!ok) {
        if (rank == 0) {
          // Aborted: wait for the stages that were armed, so that no copy is still landing when the pair exits.
          const int outstanding = min(issued, STAGES);
          int s = stage;
          uint32_t ph = phase;
          for (int i = 0; i < outstanding; ++i) {
            if (--s < 0) {
              s = STAGES - 1;
              ph ^= 1;
            }
            volatile int no_abort = 0;
            f8_wait(full_bar(s), ph, &no_abort, args.status, SITE_GEMM_DRAIN);
          }
        } else {
          // the peer cannot observe its own copies: give those in flight time to land
          const uint64_t t0 = global_timer_ns();
          while (global_timer_ns() - t0 < 100000ull) __nanosleep(1000);
        }
      }
    } else if (warp == 1) {
      // ------------------------------------------------------------------ MMA issuer (even CTA)
      // The whole warp goes through the loop, one thread issues: the descriptors then stay in uniform registers.
      if (rank == 0) {
        const bool leader = elect_one();
        const uint64_t adesc0 = smem_desc_sw128(smem_u32(smem), 16, 1024);
        const uint64_t bdesc0 = smem_desc_sw128(smem_u32(smem) + F8_A_BYTES, 16, 1024);
        int stage = 0, acc = 0;
        uint32_t phase = 0, acc_phase = 0;
        bool ok = true, any = false;
        for (int g = pair; g < total && ok; g += npairs) {
          const Fp8Tile t = f8_tile<WGRAD, SPLIT>(g, split, args, at0, at0 + 4 * (args.E + 1), at0 + 8 * (args.E + 1));
          const uint32_t idesc = idesc_e4m3_f32(256, t.n);
          const int per = f8_blocks_at_once(t.n), width = 256 / per;
          for (int kb = 0; kb < t.nkb; ++kb) {
            const int sub = kb & (per - 1);
            const bool last = sub == per - 1 || kb == t.nkb - 1;
            ok = f8_wait(full_bar(stage), phase, abort_flag, args.status, SITE_GEMM_MMA_FULL) &&
                 (sub != 0 || f8_wait(pempty_bar(acc), acc_phase ^ 1, abort_flag, args.status, SITE_GEMM_MMA_TMEM_EMPTY));
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
            tc_fence_after();
            const uint64_t off = (uint64_t)(stage * (F8_STAGE >> 4));
            if (leader) {
#pragma unroll
              for (int k4 = 0; k4 < 4; ++k4)
                umma_f8_pair(tmem_base + acc * 256 + sub * width, adesc0 + off + 2 * k4, bdesc0 + off + 2 * k4, idesc, k4 != 0 ? 1u : 0u);
              umma_commit_pair(empty_bar(stage), both);
              if (last) umma_commit_pair(pfull_bar(acc), both);
            }
            __syncwarp();
            any = true;
            if (++stage == STAGES) {
              stage = 0;
              phase ^= 1;
            }
            if (last) {
              acc ^= 1;
              if (acc == 0) acc_phase ^= 1;
            }
          }
        }
        if (any) {
          if (leader) umma_commit_pair(drain_bar, (uint16_t)(1u << cta));
          volatile int no_abort = 0;
          f8_wait(drain_bar, 0, &no_abort, args.status, SITE_GEMM_DRAIN);
        }
        __syncwarp();
      }
    } else if (warp == 2) {
      // ------------------------------------------------------------------ scales (both CTAs, each its own ring)
      int q = 0;
      uint32_t q_phase = 0;
      bool ok = true;
      for (int g = pair; g < total && ok; g += npairs) {
        const Fp8Tile t = f8_tile<WGRAD, SPLIT>(g, split, args, at0, at0 + 4 * (args.E + 1), at0 + 8 * (args.E + 1));
        const int a_row = t.m * 256 + 128 * (int)rank;
        auto weights_scale = [&](int64_t kb) {  // product: of the CTA's 128 rows
          const int tiles = (args.NM + 127) >> 7;
          return a_row < args.NM ? __ldg(args.a_scale + ((int64_t)t.e * tiles + (a_row >> 7)) * args.nkb + kb) : 0.0f;
        };
        auto rows_scale = [&](int64_t kb, int c) {
          return c < t.cols ? __ldg(args.b_scale + kb * args.b_ld + t.col0 + c) : 0.0f;
        };
        for (int kb0 = 0; kb0 < t.nkb; kb0 += F8_GROUP) {
          float b[F8_GROUP][8], a4[F8_GROUP][4];
  #pragma unroll
          for (int j = 0; j < F8_GROUP; ++j) {
            const int64_t kb = t.kb0 + min(kb0 + j, t.nkb - 1);
            if (WGRAD) {
  #pragma unroll
              for (int i = 0; i < 4; ++i) {
                const int r = a_row + i * 32 + lane;
                a4[j][i] = r < args.NM ? __ldg(args.a_scale + kb * args.NM + r) : 0.0f;
              }
            } else {
              a4[j][0] = weights_scale(kb);
            }
  #pragma unroll
            for (int i = 0; i < 8; ++i) {
              b[j][i] = rows_scale(kb, i * 32 + lane);
            }
          }
          bool apart = false;  // of any column
          if (!WGRAD) {
            uint32_t worst = 0;
  #pragma unroll
            for (int j = 0; j < F8_GROUP; ++j)
  #pragma unroll
              for (int i = 0; i < 8; ++i) worst = max(worst, f8_apart(b[j][i], a4[j][0]));
            apart = __any_sync(0xffffffffu, worst >= F8_NORMALS);
          }
          ok = __all_sync(0xffffffffu, f8_wait(sempty_bar(q), q_phase ^ 1, abort_flag, args.status, SITE_FP8_SCALES));
          if (!ok) break;
#pragma unroll
          for (int j = 0; j < F8_GROUP; ++j) {
            const uint32_t s = slots0 + q * F8_SLOT + j * (F8_SLOT_BLOCK * 4);
#pragma unroll
            for (int i = 0; i < 8; ++i)
              if (i * 32 < t.n) sts1(s + 4 * (i * 32 + f8_scale_at(lane)), WGRAD ? b[j][i] : b[j][i] * a4[j][0]);
            if (WGRAD) {
#pragma unroll
              for (int i = 0; i < 4; ++i) sts1(s + 4 * (256 + i * 32 + lane), a4[j][i]);
            }
          }
          if (!WGRAD) {
            const uint32_t s = slots0 + q * F8_SLOT;
            if (lane < F8_GROUP) sts1(s + lane * (F8_SLOT_BLOCK * 4) + 4 * F8_APART_ANY, __uint_as_float(apart));
            if (apart) {  // rare: the scales are read again, which costs no registers
#pragma unroll 1
              for (int j = 0; j < F8_GROUP; ++j) {
                const int64_t kb = t.kb0 + min(kb0 + j, t.nkb - 1);
                const float w = weights_scale(kb);
                const uint32_t to = s + j * (F8_SLOT_BLOCK * 4);
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                  const float r = rows_scale(kb, i * 32 + lane);
                  const bool mine = f8_apart(r, w) >= F8_NORMALS;
                  const uint32_t bits = __ballot_sync(0xffffffffu, mine);
                  if (mine) sts1(to + 4 * (i * 32 + f8_scale_at(lane)), r);
                  if (lane == 0) sts1(to + 4 * (F8_APART + i), __uint_as_float(bits));
                }
                if (lane == 0) sts1(to + 4 * F8_APART_SCALE, w);
              }
            }
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(sfull_bar(q));
          if (++q == SLOTS) {
            q = 0;
            q_phase ^= 1;
          }
        }
      }
    }
  } else {
    reg_inc<F8Regs<WGRAD>::EPI>();
    // ------------------------------------------------------------------ epilogue (both CTAs)
    const int quarter = warp & 3;
    const int side = (warp - 4) >> 2;  // 32-column pieces 2 i + side are this warp's
    const uint32_t pempty0_cl = mapa_shared(pempty_bar(0), cta & ~1u);
    const uint32_t tlane = __reduce_or_sync(0xffffffffu, tmem_base + (uint32_t(quarter * 32) << 16) + side * 32);
    const uint32_t lane_slot = side * 128 + 16 * (lane & 3), lane_rows = 4 * (256 + quarter * 32 + (lane >> 2) * (args.mixed ? 4 : 1)), row_step = args.mixed ? 4 : 32;
    const bool leader = elect_one();
    int acc = 0, q = 0;
    uint32_t acc_phase = 0, q_phase = 0;
    bool ok = true;
    // ready: the next accumulator and the slot of its scales have been seen complete, without columns apart.  Where they have not,
    // they are waited for, and `apart` is read again with the slot.
    bool ready = false, apart = false;
    for (int g = pair; g < total && ok; g += npairs) {
      const Fp8Tile t = f8_tile<WGRAD, SPLIT>(g, split, args, at0, at0 + 4 * (args.E + 1), at0 + 8 * (args.E + 1));
      // sum[s]: piece s / 2, TMEM lanes 16 (s % 2) of the quarter: [g][row lane / 4, + 8], columns 2 t, 2 t + 1 of group g
      float sum[8][4][2][2];
#pragma unroll
      for (int i = 0; i < 8; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          sum[i][j >> 1][j & 1][0] = sum[i][j >> 1][j & 1][1] = 0.0f;
        }
      // G blocks at once, of which this warp has NP pieces each
      auto run = [&](auto pieces, auto at_once) {
        constexpr int NP = decltype(pieces)::value, G = decltype(at_once)::value, S = 2 * NP;
        for (int kb = 0; kb < t.nkb; kb += G) {
          const uint32_t s0 = slots0 + q * F8_SLOT + (kb & (F8_GROUP - 1)) * (F8_SLOT_BLOCK * 4);
          const int blocks = min(G, t.nkb - kb);
          if (!ready) {
            if ((kb & (F8_GROUP - 1)) == 0) {
              ok = __all_sync(0xffffffffu, f8_wait(sfull_bar(q), q_phase, abort_flag, args.status, SITE_FP8_SCALES));
              if (!WGRAD) apart = __any_sync(0xffffffffu, lds1i(s0 + 4 * F8_APART_ANY));
            }
            ok = __all_sync(0xffffffffu,
                            f8_wait(pfull_bar(acc), acc_phase, abort_flag, args.status, SITE_GEMM_EPI_TMEM_FULL) && ok);
            if (!WGRAD && apart && ok) {  // the weights' scale onto the sums of columns that meet it apart, in place
              tc_fence_after();
#pragma unroll 1
              for (int i = 0; i < blocks * S; ++i) {
                const int g8 = i / S, p = i - g8 * S;
                const uint32_t s = s0 + g8 * (F8_SLOT_BLOCK * 4);
                const uint32_t at = tlane + acc * 256 + g8 * (256 / G) + (p >> 1) * 64 + (p & 1) * (16u << 16);
                const uint32_t bits = (uint32_t)lds1i(s + 4 * (F8_APART + 2 * (p >> 1) + side)) >> (2 * (lane & 3));
                const float ws = lds1(s + 4 * F8_APART_SCALE);
                uint32_t v[16];
                tmem_ld_16x256b_x4(at, v);
                tmem_wait_ld();
#pragma unroll
                for (int j = 0; j < 16; ++j)
                  if (bits >> (8 * (j >> 2) + (j & 1)) & 1) v[j] = __float_as_uint(__uint_as_float(v[j]) * ws);
                tmem_st_16x256b_x4(at, v);
                tmem_wait_st();
              }
            }
          }
          if (!ok) break;
          tc_fence_after();
#pragma unroll
          for (int g8 = 0; g8 < G; ++g8) {
            if (G == 1 || g8 < blocks) {
              const bool final = G == 1 || g8 == blocks - 1;
              const uint32_t s = s0 + g8 * (F8_SLOT_BLOCK * 4);
              const uint32_t tacc = tlane + acc * 256 + g8 * (256 / G);
              const uint32_t sl = s + lane_slot;
              float sa[4];
              if (WGRAD) {
#pragma unroll
                for (int i = 0; i < 4; ++i) sa[i] = lds1(s + lane_rows + row_step * i);
              }
              uint32_t v[2][16];
              float4 f[2];
              if (S > 0) {
                tmem_ld_16x256b_x4(tacc, v[0]);
                f[0] = lds4(sl);
                f[1] = lds4(sl + 64);
                tmem_wait_ld();
              }
              auto done = [&]() {  // the accumulator is in registers
                tc_fence_before();
                bool next = mbar_test_wait(pfull_bar(acc ^ 1), acc_phase ^ (uint32_t)acc);
                __syncwarp();
                if (leader) mbar_arrive_cluster_relaxed(pempty0_cl + 8u * acc);
                if ((kb & (F8_GROUP - 1)) + G >= F8_GROUP || kb + G >= t.nkb) {
                  const int q1 = q + 1 == SLOTS ? 0 : q + 1;
                  next = mbar_test_wait(sfull_bar(q1), q_phase ^ (uint32_t)(q1 == 0)) && next;
                  if (!WGRAD) apart = lds1i(slots0 + q1 * F8_SLOT + 4 * F8_APART_ANY) != 0;
                }
                ready = __all_sync(0xffffffffu, next && (WGRAD || !apart));
              };
              if (S == 0 && final) done();
#pragma unroll
              for (int p = 0; p < S; ++p) {
                if (p + 1 < S)
                  tmem_ld_16x256b_x4(tacc + ((p + 1) >> 1) * 64 + ((p + 1) & 1) * (16u << 16), v[(p + 1) & 1]);
                else if (final)
                  done();
                const float c[4][2] = {{f[0].x, f[0].y}, {f[0].z, f[0].w}, {f[1].x, f[1].y}, {f[1].z, f[1].w}};
                if ((p & 1) && p + 1 < S) {
                  f[0] = lds4(sl + ((p + 1) >> 1) * 256);
                  f[1] = lds4(sl + ((p + 1) >> 1) * 256 + 64);
                }
#pragma unroll
                for (int j = 0; j < 4; ++j)
#pragma unroll
                  for (int r = 0; r < 2; ++r) {
                    float2 x = make_float2(__uint_as_float(v[p & 1][4 * j + 2 * r]), __uint_as_float(v[p & 1][4 * j + 2 * r + 1]));
                    float (&to)[2] = sum[p][j][r];
                    float2 by = make_float2(c[j][0], c[j][1]);
                    if (WGRAD) {  // dy's scales first: x may hold a mask's lowest value, a sum of 448^2 times whose scale is infinite
                      x = __fmul2_rn(x, by);
                      by.x = by.y = sa[2 * (p & 1) + r];
                    }
                    if (PACKED && G == 1) {
                      const float2 z = __ffma2_rn(x, by, make_float2(to[0], to[1]));
                      to[0] = z.x;
                      to[1] = z.y;
                    } else {
                      to[0] = fmaf(x.x, by.x, to[0]);
                      to[1] = fmaf(x.y, by.y, to[1]);
                    }
                  }
                if (p + 1 < S) tmem_wait_ld();
              }
            }
          }
          if ((kb & (F8_GROUP - 1)) + G >= F8_GROUP || kb + G >= t.nkb) {
            __syncwarp();
            if (leader) mbar_arrive(sempty_bar(q));
            if (++q == SLOTS) {
              q = 0;
              q_phase ^= 1;
            }
          }
          acc ^= 1;
          if (acc == 0) acc_phase ^= 1;
        }
      };
      using one = std::integral_constant<int, 1>;
      using two = std::integral_constant<int, 2>;
      using three = std::integral_constant<int, 3>;
      using four = std::integral_constant<int, 4>;
      const int pieces = (t.n + 31) >> 5;
      if (pieces > 6 + side) run(four{}, one{});
      else if (pieces > 4) run(three{}, one{});
      else if (pieces > 2) run(two{}, two{});
      else run(one{}, four{});
      if (!ok) break;
      if (SPLIT) {
        // One tile a cluster: the other pairs' sums come into the stages of the first one's CTAs, which nothing uses any more
        // once all have met, and are added in the splits' order.
        cluster_sync();
        const uint32_t to = mapa_shared(smem_u32(smem), rank) + 4u * (threadIdx.x - 128);
        const int regs = 32 * np_of(t.n);  // of this warp's side or the wider one
        if (split > 0) {
#pragma unroll
          for (int i = 0; i < 8; ++i)
            if ((i >> 1) < np_of(t.n))
#pragma unroll
              for (int j = 0; j < 16; ++j)
                st_shared_cluster_u32(to + 1024u * (uint32_t)((split - 1) * regs + 16 * i + j),
                                      __float_as_uint(sum[i][j >> 2][j >> 1 & 1][j & 1]));
        }
        cluster_sync();
        met = true;
        if (split > 0) break;
        const uint32_t from = smem_u32(smem) + 4u * (threadIdx.x - 128);
#pragma unroll 1
        for (int p = 1; p < args.splits; ++p) {
#pragma unroll
          for (int i = 0; i < 8; ++i)
            if ((i >> 1) < np_of(t.n))
#pragma unroll
              for (int j = 0; j < 16; ++j)
                sum[i][j >> 2][j >> 1 & 1][j & 1] += lds1(from + 1024u * (uint32_t)((p - 1) * regs + 16 * i + j));
        }
      }
      // out[column][row]: of a column a lane has four rows, neighbours where the rows are mixed
      const int u = lane >> 2;
      const int j0 = t.m * 256 + 128 * (int)rank + 32 * quarter + (args.mixed ? 4 * u : u);
      const int jstep = args.mixed ? 1 : 8;
      const int left = t.cols - side * 32 - 2 * (lane & 3);  // of the columns from this lane's first on
      OUT* o = static_cast<OUT*>(args.out) +
               ((WGRAD ? (int64_t)t.e * args.NB + t.col0 : (int64_t)t.col0) + side * 32 + 2 * (lane & 3)) * args.ld + j0;
      const int64_t ld = args.ld;
      auto columns = [&](auto&& store) {  // store(o, four rows of a column)
#pragma unroll
        for (int i = 0; i < 4; ++i, o += 32 * ld)
#pragma unroll
          for (int g8 = 0; g8 < 4; ++g8, o += 8 * ld)
#pragma unroll
            for (int h = 0; h < 2; ++h)
              store(o + h * ld, 64 * i + 8 * g8 + h < left,
                    make_float4(sum[2 * i][g8][0][h], sum[2 * i][g8][1][h], sum[2 * i + 1][g8][0][h], sum[2 * i + 1][g8][1][h]));
      };
      if (args.wide_out && t.cols == 256 && j0 < args.NM) {
        columns([&](OUT* p, bool, float4 v) { f8_put4(p, v); });
      } else if (args.wide_out) {
        if (j0 < args.NM) columns([&](OUT* p, bool in, float4 v) {
          if (in) f8_put4(p, v);
        });
      } else {
        columns([&](OUT* p, bool in, float4 v) {
          if (in) {
            if (j0 < args.NM) f8_put(p, v.x);
            if (j0 + jstep < args.NM) f8_put(p + jstep, v.y);
            if (j0 + 2 * jstep < args.NM) f8_put(p + 2 * jstep, v.z);
            if (j0 + 3 * jstep < args.NM) f8_put(p + 3 * jstep, v.w);
          }
        });
      }
    }
  }

  if (SPLIT && !met) {  // the roles that joined no sums, and pairs without a tile
    cluster_sync();
    cluster_sync();
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();  // neither CTA leaves while the pair's MMAs or signals may still touch it
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_pair(tmem_base, 512);
  }
}

// E4M3 rows [groups][rows][K], `ld` bytes apart, in boxes of 128 bytes x box_rows; bytes behind K and rows behind
// `rows` read as zero.
bool tmap_e4m3_rows(CUtensorMap* m, const void* base, int64_t K, int64_t rows, int64_t groups, int64_t ld, uint32_t box_rows,
                    bool grouped) {
  const uint64_t dims[3] = {(uint64_t)K, (uint64_t)rows, (uint64_t)groups};
  const uint64_t strides[2] = {(uint64_t)ld, (uint64_t)(ld * rows)};
  const uint32_t box[3] = {128, box_rows, 1};
  return make_tmap(m, base, grouped ? 3 : 2, dims, strides, box, CU_TENSOR_MAP_DATA_TYPE_UINT8);
}

// A's rows in boxes of 128.  Mixed: of each 32 rows, box row 8 k + u is row 4 u + k, by a map with dimensions u (4 rows
// apart) and k (one row apart).
bool tmap_a(CUtensorMap* m, const void* base, int64_t K, int64_t rows, int64_t groups, int64_t ld, bool mixed) {
  if (!mixed) return tmap_e4m3_rows(m, base, K, rows, groups, ld, 128, true);
  const uint64_t dims[5] = {(uint64_t)K, 8, 4, (uint64_t)rows / 32, (uint64_t)groups};
  const uint64_t strides[4] = {(uint64_t)(4 * ld), (uint64_t)ld, (uint64_t)(32 * ld), (uint64_t)(ld * rows)};
  const uint32_t box[5] = {128, 8, 4, 4, 1};
  return make_tmap(m, base, 5, dims, strides, box, CU_TENSOR_MAP_DATA_TYPE_UINT8);
}

// B's rows in boxes of 128, 64 and 32
bool tmap_boxes(CUtensorMap (&m)[3], const void* base, int64_t K, int64_t rows, int64_t ld) {
  for (int i = 0; i < 3; ++i)
    if (!tmap_e4m3_rows(&m[i], base, K, rows, 1, ld, 128u >> i, false)) return false;
  return true;
}

bool f8_wide(const void* out, int64_t ld, int64_t width, bool bf16) {
  return ld % 4 == 0 && width % 4 == 0 && (reinterpret_cast<uintptr_t>(out) & (bf16 ? 7u : 15u)) == 0;
}

uint32_t f8_magic(int64_t d) { return d == 1 ? 0 : (uint32_t)(((int64_t(1) << 32) + d - 1) / d); }

// The counts of Fp8Clusters for the current device; with the first question, each kernel is allowed its shared memory.
template <bool WGRAD, typename OUT>
cudaError_t f8_clusters(int (&clusters)[2]) {
  static Fp8Clusters known;
  int dev = 0;
  const cudaError_t err = cudaGetDevice(&dev);
  if (err != cudaSuccess) return err;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  return known.get<cudaError_t>(dev, clusters, [](int (&counts)[2]) {
    auto kern = fp8_gemm_kernel<WGRAD, true, false, OUT>;
    for (auto each : {kern, fp8_gemm_kernel<WGRAD, false, false, OUT>, fp8_gemm_kernel<WGRAD, false, true, OUT>}) {
      const cudaError_t err = cudaFuncSetAttribute(each, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)f8_smem(FP8_MAX_E));
      if (err != cudaSuccess) return err;
    }
    for (int i = 0; i < 2; ++i) {
      cudaLaunchConfig_t cfg{};
      cudaLaunchAttribute attr[1];
      attr[0].id = cudaLaunchAttributeClusterDimension;
      attr[0].val.clusterDim.x = 4u << i;
      attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
      cfg.blockDim = dim3(F8_THREADS, 1, 1);
      cfg.gridDim = dim3(128u << i, 1, 1);
      cfg.dynamicSmemBytes = f8_smem(FP8_MAX_E);
      cfg.attrs = attr;
      cfg.numAttrs = 1;
      const cudaError_t err = cudaOccupancyMaxActiveClusters(&counts[i], kern, &cfg);
      if (err != cudaSuccess) return err;
    }
    return cudaSuccess;
  });
}

template <bool WGRAD, typename OUT>
cudaError_t launch(const CUtensorMap& ta, const CUtensorMap (&tb)[3], const Fp8GemmArgs& args, int64_t tiles, int n_sm,
                   cudaStream_t st) {
  auto kern = args.splits > 1 ? fp8_gemm_kernel<WGRAD, true, false, OUT>
              : args.packed   ? fp8_gemm_kernel<WGRAD, false, true, OUT>
                              : fp8_gemm_kernel<WGRAD, false, false, OUT>;
  cudaLaunchConfig_t cfg{};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2 * args.splits;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.blockDim = dim3(F8_THREADS, 1, 1);
  cfg.dynamicSmemBytes = f8_smem(args.E);
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  // with splits every tile has its cluster
  cfg.gridDim = dim3((unsigned)(2 * args.splits * (args.splits > 1 ? tiles : std::min<int64_t>(tiles, std::max(1, n_sm / 2)))), 1, 1);
  const cudaError_t err = cudaLaunchKernelEx(&cfg, kern, ta, tb[0], tb[1], tb[2], args);
  return err != cudaSuccess ? err : cudaGetLastError();
}

}  // namespace

cudaError_t launch_fp8_matmul(const Fp8MatmulArgs& a, bool bf16_out, int n_sm, cudaStream_t st) {
  Fp8GemmArgs g = {};
  g.E = a.E;
  g.nkb = (int)((a.K + 127) / 128);
  g.NM = (int)a.N;
  g.MT = (int)((a.N + 255) / 256);
  g.R = a.R;
  g.offsets = a.offsets;
  g.a_scale = a.w_scale;
  g.b_scale = a.x_scale;
  g.b_ld = a.x_scale_stride;
  g.out = a.out;
  g.ld = a.out_stride;
  g.mixed = a.N % 32 == 0;
  g.wide_out = g.mixed && f8_wide(a.out, a.out_stride, a.N, bf16_out);
  g.status = a.status;
  const int64_t groups = std::min<int64_t>(a.E, a.R);  // that can have rows
  int clusters[2];
  const cudaError_t err = bf16_out ? f8_clusters<false, __nv_bfloat16>(clusters) : f8_clusters<false, float>(clusters);
  if (err != cudaSuccess) return err;
  const Fp8Plan plan = f8_plan(a.E, g.MT, n_sm, g.nkb, groups, (a.R + groups - 1) / groups, a.E == 1, clusters, F8_STAGES * F8_STAGE);
  g.nmax = plan.nmax;
  g.splits = plan.splits;
  int64_t tiles = plan.tiles;
  if (a.E > 1) tiles = ((a.R + g.nmax - 1) / g.nmax + a.E) * g.MT;  // at most, whatever the groups' sizes
  if (tiles > INT32_MAX) return cudaErrorInvalidValue;
  g.magic_per = f8_magic(g.MT);
  // 8,192 x 8,192 x 8,192 554 -> 534 us with two sums an instruction, 256 rows a group 186 -> 182; 16,384 rows of 128 groups 711 both
  g.packed = a.R >= 192 * groups;
  CUtensorMap ta, tb[3];
  if (!tmap_a(&ta, a.w, a.K, a.N, a.E, a.w_stride, g.mixed) ||
      !tmap_boxes(tb, a.x, a.K, a.R, a.x_stride))
    return cudaErrorInvalidValue;
  return bf16_out ? launch<false, __nv_bfloat16>(ta, tb, g, tiles, n_sm, st) : launch<false, float>(ta, tb, g, tiles, n_sm, st);
}

cudaError_t launch_fp8_weight_grad(const Fp8WeightGradArgs& a, bool bf16_out, int n_sm, cudaStream_t st) {
  Fp8GemmArgs g = {};
  g.E = a.E;
  g.NM = (int)a.H;
  g.NB = (int)a.N;
  g.MT = (int)((a.H + 255) / 256);
  g.R = a.R;
  g.blocks = a.R / 128 + a.E;
  g.offsets = a.offsets;
  g.a_scale = a.x_scale;
  g.b_scale = a.dy_scale;
  g.b_ld = a.N;
  g.out = a.out;
  g.ld = a.H;
  g.mixed = a.H % 32 == 0;
  g.wide_out = g.mixed && f8_wide(a.out, a.H, a.H, bf16_out);
  g.status = a.status;
  int clusters[2];
  const cudaError_t err = bf16_out ? f8_clusters<true, __nv_bfloat16>(clusters) : f8_clusters<true, float>(clusters);
  if (err != cudaSuccess) return err;
  const Fp8Plan plan = f8_plan(a.E, g.MT, n_sm, (a.R / 128 + a.E - 1) / a.E, a.E, a.N, true, clusters, F8_STAGES * F8_STAGE);
  g.nmax = plan.nmax;
  g.splits = plan.splits;
  const int64_t tiles = plan.tiles;
  if (tiles > INT32_MAX) return cudaErrorInvalidValue;
  const int64_t nc = (a.N + g.nmax - 1) / g.nmax;
  g.magic_per = f8_magic(nc * g.MT);
  g.magic_nc = f8_magic(nc);
  // 1,024 rows a group 1,254 -> 1,231 us with two sums an instruction, 512 1,647 -> 1,624, but 256 2,153 -> 2,266 and 128 (one block)
  // 760 -> 853: the sums' pairs cost the stores moves
  g.packed = a.R >= 384 * (int64_t)a.E;
  CUtensorMap ta, tb[3];
  const int64_t P = 128 * g.blocks;
  if (!tmap_a(&ta, a.x, P, a.H, 1, a.x_stride, g.mixed) ||
      !tmap_boxes(tb, a.dy, P, a.N, a.dy_stride))
    return cudaErrorInvalidValue;
  return bf16_out ? launch<true, __nv_bfloat16>(ta, tb, g, tiles, n_sm, st) : launch<true, float>(ta, tb, g, tiles, n_sm, st);
}

}  // namespace mok
