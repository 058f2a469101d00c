// lin_tc.cu - the causal linear memory on the tensor cores: bf16 tensors.
//
// One job (linear.h) over 128-row chunks, in four products a chunk, all with
// fp32 accumulators in TMEM:
//
//   S  = X Y^T                         (rows x rows)
//   O1 = P Z,  P = bf16(S decayed and masked), from TMEM
//   O2 = X bf16(W)                     W: the state before the chunk
//   dW = (Y1 + Y2 + ..)^T Z            Y1 + Y2 + .. = Y decayed to the chunk's end
//
// out = alpha (O1 + factor O2), and W = lambda^n W + dW is carried in fp32 in
// registers.  P and the W of the read are rounded to bf16 once (2^-8 of a
// term, as the tensors themselves); the decayed Y that enters the carried
// state is kept in two or three bf16 parts (16 or 24 bits), because a state is
// read by every later token.
//
// A chunk reads three tiles and writes one (128 KB at head_dim 128: 3.0 us of a
// 148th of the HBM rate, 5500 cycles at 1.85 GHz) against 2560 cycles of
// products; TMA keeps the next chunk's tiles in flight in a ring of slots.
// Measured: 7000 cycles at 128 columns, 4700 at 64 (241920 x 4 x 128: 210 us; the
// scan and the parts of the ranges, 91 us, beside).  Bound by shared memory, 85 %
// of its cycles at 128 columns, and by the issue of the warps' instructions,
// 0.54-0.56 a cycle.  A memory that spans the whole sequence (log_decay -1e-5)
// takes 262 us and 165: no chunk falls out of the parts, and every chunk of the
// CTAs that end a head has a third part.
//
// Roles (28 warps): warp 0 TMA, warps 1-2 issue the products, warps 4-19 decay
// (P in TMEM, then Y: its first part in place, the others beside), warps 20-27
// write the output rows and carry W (a thread owns half a row of W).  TMEM is
// full: S | O1 | O2 | dW, 128 columns each; P overwrites S's columns in place.
// Two warps issue, P Z and the next chunk's scores in turn, X W and dW in turn:
// W of this chunk is published while P Z and the scores run, Y decayed while
// all three do, and the next P made during dW.  (S and dW twice, which 64
// columns have room for, made a chunk longer: 277 us instead of 211 at 8 x 10000
// x 16 x 64.)
//
// Products of 128 x 128 x 16 from shared memory take all its bandwidth (8 KB in
// 64 cycles), so that every other access lengthens the chunk: arrivals are one
// a warp, output rows leave by TMA, and the decayed Y has a third part only
// where the state is handed out (two: states 2.4e-6 off, which the bf16 read
// of W does not see; three: 4e-7 and less, as fp32 sums are).
//
// The roles' loops run at once and share an instruction cache of about 32 KB:
// loops over halves and rows stay rolled and waits are short.  The products are
// unrolled all the same: their operands are then made in uniform registers (5-8
// % of the call).
//
// head_dim 32 takes the 64-column form: TMA fills the upper columns with
// zeros, so that DRAM traffic stays that of 32.
#include <algorithm>

#include "lin_common.cuh"
#include "pdl.cuh"
#include "sm100.cuh"
#include "tma_encode.h"

namespace vdn {
namespace {

constexpr int kChunk = kLinTcChunk;

template <int D>
struct TcLayout {
  static constexpr int kTile = kChunk * D * 2;
  static constexpr int kSlots = D == 128 ? 5 : 9;
  static constexpr int kLo = kSlots * kTile;                 // second and third part of 64 rows of the decayed Y
  static constexpr int kW = kLo + kTile;                     // bf16(W), [z box of 64][y][64]
  static constexpr int kZero = kW + D * D * 2;               // D = 64: the upper half of a 128-row A operand, one K step
  static constexpr int kTab = kZero + (D == 64 ? 2048 : 0);  // lambda^0..31 of a piece's head between zeros, two in turn
  static constexpr int kStage = D == 128 ? kW : kTab + 1024;  // its rows on their way out: W's tile (see there), or 8 x 2 KB
  static constexpr int kBar = D == 128 ? kTab + 2 * 384 : kStage + 8 * 2048;
  static constexpr int kRange = kBar + 288;  // the CTA's range: its first chunk and the next range's
  static constexpr int kBytes = kRange + 16 + 1024;
};
static_assert(TcLayout<128>::kBytes <= 232448 && TcLayout<64>::kBytes <= 232448, "shared memory of an SM");

// barriers: kFull + slot, kEmpty + slot, then one of each (a phase a chunk)
enum { kFull = 0, kEmpty = 9, kSFull = 18, kPReady, kYReady, kYFree, kYReady2, kOFull, kOFree, kDwFull, kWReady, kDone, kNumBars };

constexpr int kDecay = 512, kOut = 256;  // threads of the decay warps, and of the output warps
constexpr int kTcThreads = 128 + kDecay + kOut;
constexpr uint32_t kCtlRegs = 56, kDecayRegs = 48, kOutRegs = 128, kTcRegs = 72;
static_assert(128 * kCtlRegs + kDecay * kDecayRegs + kOut * kOutRegs <= kTcThreads * kTcRegs, "registers of a CTA");

constexpr uint32_t kColS = 0, kColO1 = 128, kColO2 = 256, kColDw = 384;

__device__ __forceinline__ void tma_load_4d(void* dst, const CUtensorMap* map, uint64_t* bar, int x, int h, int n, int b) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5, %6}], [%2];" ::"r"(
          smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(x), "r"(h), "r"(n), "r"(b)
      : "memory");
}

// A value the compiler takes for a new one: it stays in a register and is not read again from the parameters.
__device__ __forceinline__ uint32_t fresh(uint32_t v) {
  asm volatile("" : "+r"(v));
  return v;
}

// A tensor's map with its multipliers in registers (a read of the parameters at each load is a miss in their cache).
struct MapRef {
  const CUtensorMap* map;
  uint32_t mh, mb;
  __device__ __forceinline__ MapRef(const LinMap& m) : map(&m.map), mh(fresh(m.mh)), mb(fresh(m.mb)) {
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(map)) : "memory");
  }
};

template <int D>
__device__ __forceinline__ void load_tile(uint8_t* dst, const MapRef& m, uint64_t* bar, int h, int row, int b) {
  mbar_expect_tx(bar, kChunk * D * 2);
#pragma unroll
  for (int bx = 0; bx < D / 64; ++bx) tma_load_4d(dst + bx * kChunk * 128, m.map, bar, bx * 64, h * (int)m.mh, row, b * (int)m.mb);
}

// What the first wait of a CTA that ran out leaves in shared memory (a call at each wait would cost its callers registers).
struct WaitRecord {
  int given_up, bar, parity, warp;
  long long ns;
};

static_assert(kNumBars * 8 + 8 + sizeof(WaitRecord) <= 272, "barrier block");

// A probe may suspend the warp until the phase completes, so that a wait seldom probes twice.
constexpr uint32_t kSuspendNs = 100000;
// mbar_wait in few instructions (see the head of the file): the same bound in global time, read at every probe.
__device__ __forceinline__ bool try_wait_long(uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred P;\n\t"
      "mbarrier.try_wait.parity.shared::cta.b64 P, [%1], %2, %3;\n\t"
      "selp.b32 %0, 1, 0, P;\n\t}"
      : "=r"(ok)
      : "r"(smem_u32(bar)), "r"(parity), "r"(kSuspendNs)
      : "memory");
  return ok != 0;
}
__device__ __forceinline__ bool lin_wait(uint64_t* bar, uint32_t parity, WaitRecord* rec, long long limit_ns = kWaitNs) {
  long long t0 = 0;
  while (!try_wait_long(bar, parity)) {
    if (*reinterpret_cast<volatile int*>(&rec->given_up)) return false;
    const long long t = global_ns();
    if (t0 == 0) {
      t0 = t;
    } else if (t - t0 > limit_ns) {
      if (atomicExch(&rec->given_up, 1) == 0) {
        rec->bar = (int)smem_u32(rec) - (int)smem_u32(bar);
        rec->parity = (int)parity;
        rec->warp = (int)warp_id();
        rec->ns = t - t0;
      }
      return false;
    }
  }
  return true;
}

// After the CTA's last barrier: the status word and the timeout record (sm100.cuh), of a CTA that gave up.
__device__ __forceinline__ void report(const WaitRecord& w, int* status, int* r, int kernel) {
  if (!w.given_up) return;
  if (status) atomicExch(status, kStatusTimeout);
  if (!r || atomicAdd(r + kRecTimeouts, 1) != 0) return;
  r[kRecKernel] = kernel;
  r[kRecBlock] = (int)blockIdx.x;
  r[kRecWarp] = w.warp;
  r[kRecBarOff] = w.bar;
  r[kRecParity] = w.parity;
  r[kRecNs] = (int)(w.ns & 0xffffffffll);
  r[kRecNs + 1] = (int)(w.ns >> 32);
  r[kRecSm] = sm_id();
}

// A place in a ring of kSlots with the phase of its barriers.
template <int kSlots>
struct Ring {
  int slot;
  uint32_t phase;
  __device__ __forceinline__ Ring(int at = 0) : slot(at), phase(0) {}
  __device__ __forceinline__ void advance(int n) {
    slot += n;
    if (slot >= kSlots) {
      slot -= kSlots;
      phase ^= 1;
    }
  }
};

// One arrival for the warp, after what all its lanes did before (arrivals of 32 lanes are 32 turns of shared memory).
__device__ __forceinline__ void arrive_warp(uint64_t* bar) {
  __syncwarp();
  if (lane_id() == 0) mbar_arrive(bar);
}

// Weight of row r of a chunk with n real rows, `more` rows before the place it is decayed to.  Rows from n on, which are
// zeros, have a real row's weight: with decays above 1 a larger one could be infinite.
__device__ __forceinline__ float row_weight(float l2, int r, int n, int reverse, int more) {
  return lin_pow(l2, more + (reverse ? min(r + 1, n) : max(n - 1 - r, 0)));
}

constexpr int kHalf = kChunk / 2;  // rows whose second and third parts are held at a time

__device__ __forceinline__ uint64_t bf16x2_to_f32x2(uint32_t u) { return f32x2_pack(bf16_lo(u), bf16_hi(u)); }
__device__ __forceinline__ uint32_t f32x2_to_bf16x2(uint64_t v) {
  float a, b;
  f32x2_unpack(v, a, b);
  return pack_bf16x2(a, b);
}

// Decays rows row0 .. row0 + 63 of a tile of Y (128-byte rows, boxes of 64 columns) by 512 threads, of which each has one
// row, w its weight: the first part in place, the second and, if `third`, the third into `parts` (64 rows each, the same
// layout).  Rows from n on (padding, whatever it holds) become zeros.
template <int D>
__device__ __forceinline__ void decay_half(uint8_t* tile, uint8_t* parts, int row0, int tid, float w, int n, bool third) {
  constexpr int kThreads = 512, kPart = kHalf * D * 2, kUnits = kPart / 16 / kThreads;
  static_assert(kThreads / 8 == kHalf, "a thread's units lie in one row");
  const uint64_t w2 = f32x2_pack(w, w);
#pragma unroll
  for (int i = 0; i < kUnits; ++i) {
    const int off = (tid + i * kThreads) * 16;                                              // in a part
    uint8_t* y = tile + off / (kHalf * 128) * (kChunk * 128) + row0 * 128 + off % (kHalf * 128);  // in the tile
    uint4 v = *reinterpret_cast<const uint4*>(y);
    if (row0 + tid / 8 >= n) v = make_uint4(0, 0, 0, 0);
    const uint32_t x[4] = {v.x, v.y, v.z, v.w};
    uint32_t u[4];
    uint64_t f[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      f[e] = f32x2_mul(bf16x2_to_f32x2(x[e]), w2);
      u[e] = f32x2_to_bf16x2(f[e]);
      f[e] = f32x2_sub(f[e], bf16x2_to_f32x2(u[e]));
    }
    *reinterpret_cast<uint4*>(y) = make_uint4(u[0], u[1], u[2], u[3]);
#pragma unroll
    for (int e = 0; e < 4; ++e) u[e] = f32x2_to_bf16x2(f[e]);
    *reinterpret_cast<uint4*>(parts + off) = make_uint4(u[0], u[1], u[2], u[3]);
    if (third) {
#pragma unroll
      for (int e = 0; e < 4; ++e) u[e] = f32x2_to_bf16x2(f32x2_sub(f[e], bf16x2_to_f32x2(u[e])));
      *reinterpret_cast<uint4*>(parts + kPart + off) = make_uint4(u[0], u[1], u[2], u[3]);
    }
  }
}

// Rows from n on of a tile become zeros.
template <int D, int kThreads>
__device__ __forceinline__ void clear_rows(uint8_t* z, int tid, int n) {
#pragma unroll
  for (int i = 0; i < kChunk * D / 8 / kThreads; ++i) {
    const int idx = tid + i * kThreads;
    if (idx / 8 % kChunk >= n) *reinterpret_cast<uint4*>(z + idx * 16) = make_uint4(0, 0, 0, 0);
  }
}

// acc = A B over the columns of K-major A (128-byte rows, boxes of 64 columns); B K-major likewise, or MN-major from its
// first row on
template <int D, bool kBMn>
__device__ __forceinline__ void mma_columns(uint32_t acc, uint32_t a, uint32_t b, uint32_t idesc) {
  const uint64_t da = smem_desc(a, 16, 1024, kLayoutSw128);
  const uint64_t db = kBMn ? smem_desc(b, D * 128, 1024, kLayoutSw128) : smem_desc(b, 16, 1024, kLayoutSw128);
#pragma unroll
  for (int kk = 0; kk < D / 16; ++kk) {
    const uint64_t step = (kk >> 2) * (kChunk * 8) + (kk & 3) * 2;
    mma_ss(acc, da + step, db + (kBMn ? (uint64_t)kk * 128 : step), idesc, kk > 0);
  }
}

// dW (+)= Yk^T Z over 64 rows of a chunk, Yk one part of Y from its first row on, boxes of 64 columns `a_stride` apart, z at
// its first row (D = 64: rows 64-127 of the transposed operand are the zero block, which stays where it is from one 16-row
// step to the next)
template <int D>
__device__ __forceinline__ void mma_part(uint32_t acc, uint32_t a, uint32_t a_stride, uint32_t zero, uint32_t z, uint32_t go) {
  constexpr uint32_t idesc = idesc_bf16_f32(128, D, 1, 1);
  constexpr uint64_t step = D == 64 ? 128ull - (128ull << 16) : 128ull;
  const uint64_t dz = smem_desc(z, kChunk * 128, 1024, kLayoutSw128);
  const uint64_t da = smem_desc(a, D == 64 ? zero - a : a_stride, 1024, kLayoutSw128);
#pragma unroll
  for (int kk = 0; kk < kHalf / 16; ++kk) mma_ss(acc, da + kk * step, dz + kk * 128, idesc, kk || go);
}
// The parts behind the first, as decay_half leaves them, and the first.  An accumulator cuts what it adds at its own last
// bit, and in one direction: the small parts come before the first one, and an accumulator has one chunk.
template <int D>
__device__ __forceinline__ void mma_small(uint32_t acc, uint32_t parts, uint32_t zero, uint32_t z, uint32_t go, int n_parts) {
  if (n_parts == 3) mma_part<D>(acc, parts + kHalf * D * 2, kHalf * 128, zero, z, go);
  mma_part<D>(acc, parts, kHalf * 128, zero, z, n_parts == 3 || go);
}
template <int D>
__device__ __forceinline__ void mma_first(uint32_t acc, uint32_t y, uint32_t zero, uint32_t z) {
  mma_part<D>(acc, y, kChunk * 128, zero, z, 1);
}

// Stores a box of shared memory through a tensor map; this thread's stores have read their memory after store_wait.
__device__ __forceinline__ void tma_store_4d(const CUtensorMap* map, const void* src, int x, int h, int n, int b) {
  asm volatile("cp.async.bulk.tensor.4d.global.shared::cta.bulk_group [%0, {%2, %3, %4, %5}], [%1];" ::"l"(
                   reinterpret_cast<uint64_t>(map)),
               "r"(smem_u32(src)), "r"(x), "r"(h), "r"(n), "r"(b)
               : "memory");
  asm volatile("cp.async.bulk.commit_group;" ::: "memory");
}
__device__ __forceinline__ void store_wait() { asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory"); }

}  // namespace

namespace {

// Whether the third part of the decayed Y counts in a state that is handed out (or on): in chunks whose weight there,
// `rows` rows later, is above 2^-4 (without decay the first part is Y itself).  What is left out is below 2^-16 of a term,
// and 2^-20 of terms of weight one.
__device__ __forceinline__ bool third_part(float l2, int rows) { return l2 != 0.f && l2 * (float)rows > -4.f; }

}  // namespace

// kSplit: of a plan with equal parts.  Whole heads have a kernel of their own: the ranges' ends come from the parameters
// there, and with them in other registers the 64-column walk took 6 % longer (gradients at 8 x 8000 x 4 x 64: 177 us and 166).
template <int D, bool kSplit>
__global__ void __launch_bounds__(kTcThreads, 1) lin_out_tc(const __grid_constant__ LinTcMaps maps,
                                                            const __grid_constant__ LinOutParams p) {
  using L = TcLayout<D>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + L::kBar);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + L::kBar + kNumBars * 8);
  WaitRecord* ab = reinterpret_cast<WaitRecord*>(smem + L::kBar + kNumBars * 8 + 8);
  volatile int* parts_of = reinterpret_cast<int*>(smem + L::kBar + 272);  // of a chunk, two in turn
  const LinPlan& pl = p.pl;
  const LinJob& jb = p.job[blockIdx.x % p.n_jobs];
  const int range = blockIdx.x / p.n_jobs, rev = jb.reverse;
  long long* range_at = reinterpret_cast<long long*>(smem + L::kRange);
  const uint32_t warp = warp_id(), lane = lane_id();

  if (threadIdx.x == 0) {
    for (int s = 0; s < L::kSlots; ++s) {
      mbar_init(&bars[kFull + s], 1);
      mbar_init(&bars[kEmpty + s], 2);  // both issuing warps
    }
    mbar_init(&bars[kSFull], 1);
    mbar_init(&bars[kPReady], kDecay / 32);
    mbar_init(&bars[kYReady], kDecay / 32);
    mbar_init(&bars[kYFree], 1);
    mbar_init(&bars[kYReady2], kDecay / 32);
    mbar_init(&bars[kOFull], 2);
    mbar_init(&bars[kOFree], kOut / 32);
    mbar_init(&bars[kDwFull], 1);
    mbar_init(&bars[kWReady], kOut / 32);
    mbar_init(&bars[kDone], 2);
    ab->given_up = 0;
    fence_mbar_init();
  }
  if (kSplit && warp == 2) {
    const LinCuts cuts(pl, p.lengths, p.B, p.H, p.N, rev);
    const long long t0 = cuts.start(range), t1 = cuts.start(range + 1);
    if (lane == 0) range_at[0] = t0, range_at[1] = t1;
  }
  if (D == 64)
    for (int i = threadIdx.x; i < 2048 / 16; i += kTcThreads)
      reinterpret_cast<uint4*>(smem + L::kZero)[i] = make_uint4(0, 0, 0, 0);
  fence_proxy_async_smem();
  if (warp == 1) {
    tmem_alloc(tmem_slot, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  // (uniform registers)
  const long long t_begin = kSplit ? __shfl_sync(0xffffffffu, range_at[0], 0) : pl.start(range),
                  t_end = kSplit ? __shfl_sync(0xffffffffu, range_at[1], 0) : pl.start(range + 1);

  if (warp < 4) {
    regs_dec<kCtlRegs>();
    if (warp == 0 && lane == 0) {
      // ------------------------------------------------------------ loads: X, Y, Z of each chunk
      int i = 0;
      bool ok = true;
      Ring<L::kSlots> ring;
      const MapRef mx(maps.m[jb.mx]), my(maps.m[jb.my]), mz(maps.m[jb.mz]);
      for (long long t = t_begin; t < t_end && ok;) {
        const LinPiece pc(t, t_end, pl);
        t += pc.u1 - pc.u0;
        const int b = pc.bh / p.H, h = pc.bh % p.H;
        int ua, ub;
        lin_real(pc.u0, pc.u1, lin_length(p.lengths, b, p.N), pl, rev, ua, ub);
        for (int u = ua; u < ub && ok; ++u) {
          const int row = (rev ? pl.nc - 1 - u : u) * kChunk;
#pragma unroll
          for (int k = 0; k < 3; ++k, ++i, ring.advance(1)) {
            const MapRef& m = k == 0 ? mx : k == 1 ? my : mz;
            if (!lin_wait(&bars[kEmpty + ring.slot], ring.phase ^ 1, ab)) {
              ok = false;
              break;
            }
            load_tile<D>(smem + ring.slot * L::kTile, m, &bars[kFull + ring.slot], h, row, b);
          }
        }
      }
      if (!ok)
        for (int k = (i > L::kSlots ? i - L::kSlots : 0); k < i; ++k)
          mbar_drain(&bars[kFull + k % L::kSlots], (k / L::kSlots) & 1);
    } else if (warp == 1 || warp == 2) {
      // ------------------------------------------------------------ products
      // Warp 1: scores and P Z; warp 2: X W and dW, so that one's waits pass while the other's products run.  The whole warp
      // goes through the loop and one lane issues: operands of warp-uniform code are made in uniform registers, which a
      // product takes.
      int total = 0;
      for (long long t = t_begin; t < t_end;) {
        const LinPiece pc(t, t_end, pl);
        t += pc.u1 - pc.u0;
        int ua, ub;
        lin_real(pc.u0, pc.u1, lin_length(p.lengths, pc.bh / p.H, p.N), pl, rev, ua, ub);
        total += ub - ua;
      }
      constexpr uint32_t id_s = idesc_bf16_f32(128, kChunk, 0, 0), id_o = idesc_bf16_f32(128, D, 0, 1);
      const uint32_t base = smem_u32(smem);
      using R = Ring<L::kSlots>;
      R x(0), y(1), z(2);  // the chunk's tiles
      auto tile = [&](const R& t) { return base + t.slot * L::kTile; };
      auto wait = [&](uint64_t* bar, uint32_t ph, long long limit = kWaitNs) {
        const bool got = __all_sync(0xffffffffu, lin_wait(bar, ph, ab, limit));
        tc_fence_after();
        return got;
      };
      auto loaded = [&](const R& t) { return wait(&bars[kFull + t.slot], t.phase); };
      if (warp == 1) {
        // failure-path test: wait, with a short limit, for a phase that only this warp's own commit completes
        bool ok = !(p.inject_timeout && blockIdx.x == 0 && !wait(&bars[kSFull], 0, 10000000ll));
        for (int c = -1; c < total && ok; ++c) {
          const uint32_t ph = c & 1;
          if (c >= 0) {
            if (!loaded(z) || !wait(&bars[kPReady], ph)) break;
            if (c > 0 && !wait(&bars[kOFree], ph ^ 1)) break;
            if (elect_one()) {
              const uint64_t dz = smem_desc(tile(z), kChunk * 128, 1024, kLayoutSw128);
#pragma unroll
              for (int kk = 0; kk < kChunk / 16; ++kk)
                mma_ts(tmem + kColO1, tmem + kColS + (kk >> 1) * 32 + (kk & 1) * 8, dz + kk * 128, id_o, kk > 0);
              mma_commit(&bars[kOFull]);
              mma_commit(&bars[kEmpty + z.slot]);
            }
            __syncwarp();
            z.advance(3);
          }
          if (c + 1 == total) break;
          if (!loaded(x) || !loaded(y)) break;
          if (elect_one()) {
            mma_columns<D, false>(tmem + kColS, tile(x), tile(y), id_s);
            mma_commit(&bars[kSFull]);
            mma_commit(&bars[kEmpty + x.slot]);
            mma_commit(&bars[kEmpty + y.slot]);
          }
          __syncwarp();
          x.advance(3);
          y.advance(3);
        }
      } else {
        for (int c = 0; c < total; ++c, x.advance(3), y.advance(3), z.advance(3)) {
          const uint32_t ph = c & 1;
          if (!loaded(x) || !wait(&bars[kWReady], ph)) break;
          if (c > 0 && !wait(&bars[kOFree], ph ^ 1)) break;
          if (elect_one()) {
            mma_columns<D, true>(tmem + kColO2, tile(x), base + L::kW, id_o);
            mma_commit(&bars[kOFull]);
            mma_commit(&bars[kEmpty + x.slot]);
          }
          __syncwarp();
          const uint32_t ty = tile(y), tz = tile(z);
          if (!loaded(z) || !wait(&bars[kYReady], ph)) break;
          const int n_parts = parts_of[ph];  // as the decay warps have decided
          if (n_parts == 3) {
            if (elect_one()) {
              mma_small<D>(tmem + kColDw, base + L::kLo, base + L::kZero, tz, 0, 3);
              mma_first<D>(tmem + kColDw, ty, base + L::kZero, tz);
              mma_commit(&bars[kYFree]);
            }
            __syncwarp();
          }
          if (!wait(&bars[kYReady2], ph)) break;
          if (elect_one()) {
            if (n_parts == 2) mma_small<D>(tmem + kColDw, base + L::kLo, base + L::kZero, tz, 0, 2);
            mma_small<D>(tmem + kColDw, base + L::kLo + (n_parts == 2 ? kHalf * D * 2 : 0), base + L::kZero,
                         tz + kHalf * 128, 1, n_parts);
            if (n_parts == 2) {
              mma_first<D>(tmem + kColDw, ty, base + L::kZero, tz);
              mma_commit(&bars[kYFree]);
            }
            mma_first<D>(tmem + kColDw, ty + kHalf * 128, base + L::kZero, tz + kHalf * 128);
            mma_commit(&bars[kEmpty + y.slot]);
            mma_commit(&bars[kEmpty + z.slot]);
            mma_commit(&bars[kDwFull]);
          }
          __syncwarp();
        }
      }
      // every product of this warp completes before TMEM is released
      if (elect_one()) mma_commit(&bars[kDone]);
      __syncwarp();
    }
  } else if (warp < 4 + kDecay / 32) {
    // ------------------------------------------------------------ decays
    regs_dec<kDecayRegs>();
    const int tid = threadIdx.x - 128, q = warp & 3, block = (warp - 4) >> 2;  // rows 32 q .., columns 32 block .. of P
    const uint32_t s_lane = tmem_addr(tmem + kColS, q * 32, block * 32);
    const int away = rev ? block - q : q - block;  // blocks between P's columns and its rows' own; < 0: masked
    int c = 0, table = 0;
    Ring<L::kSlots> ry(1), rz(2);
    bool ok = true;
    for (long long t = t_begin; t < t_end && ok;) {
      const LinPiece pc(t, t_end, pl);
      t += pc.u1 - pc.u0;
      const int b = pc.bh / p.H, h = pc.bh % p.H, len = lin_length(p.lengths, b, p.N);
      int ua, ub;
      lin_real(pc.u0, pc.u1, len, pl, rev, ua, ub);
      if (ua == ub) continue;
      const float l2 = lin_log2_decay(p.log_decay[h]);
      // Every warp writes the same table.  One that is ahead fills the other: it has passed a chunk of this piece, which
      // takes all warps, before it comes to the next but one.
      float* pw = reinterpret_cast<float*>(smem + L::kTab) + (table ^= 96) + 32;
      pw[lane] = lin_pow(l2, rev ? lane : 31 - lane);
      pw[(int)lane - 32] = pw[lane + 32] = 0.f;
      __syncwarp();
      const bool final_piece = jb.final_out && pc.u1 == pl.nc;
      // of this thread's rows of Y in a whole chunk
      const float whole0 = row_weight(l2, tid / 8, kChunk, rev, 0), whole1 = row_weight(l2, kHalf + tid / 8, kChunk, rev, 0);
      // decay of row i, column j of a block before the diagonal: near * pw[j], both powers non-negative
      const float near = away > 0 ? lin_pow(l2, rev ? 32 * away - (int)lane : 32 * away - 31 + (int)lane) : 1.f;
      for (int u = ua; u < ub; ++u, ++c, ry.advance(3), rz.advance(3)) {
        const int row0 = (rev ? pl.nc - 1 - u : u) * kChunk, n = min(len - row0, kChunk);
        const uint32_t ph = c & 1;
        uint8_t *y = smem + ry.slot * L::kTile, *parts = smem + L::kLo;
        const bool third = final_piece && third_part(l2, lin_rows(u + 1, ub, len, pl, rev));
        if (tid == 0) parts_of[ph] = third ? 3 : 2;
        bool got = lin_wait(&bars[kSFull], ph, ab);
        if (got && n < kChunk) got = lin_wait(&bars[kFull + rz.slot], rz.phase, ab);
        if (__any_sync(0xffffffffu, !got)) { ok = false; break; }
        tc_fence_after();
#pragma unroll 1
        for (int hb = 0; hb < 2; ++hb) {  // 16 columns at a time
          uint32_t out[8];
          if (away < 0) {
#pragma unroll
            for (int e = 0; e < 8; ++e) out[e] = 0;
          } else {
            uint32_t s[16];
            tmem_ld16(s_lane + hb * 16, s);
            if (away > 0) {
              ulonglong2 f[4];
#pragma unroll
              for (int e = 0; e < 4; ++e) f[e] = reinterpret_cast<const ulonglong2*>(pw + hb * 16)[e];
              const uint64_t near2 = f32x2_pack(near, near);
              tmem_wait_ld();
#pragma unroll
              for (int e = 0; e < 8; ++e) {
                const uint64_t v = f32x2_pack(__uint_as_float(s[2 * e]), __uint_as_float(s[2 * e + 1]));
                out[e] = f32x2_to_bf16x2(f32x2_mul(f32x2_mul(v, near2), e & 1 ? f[e >> 1].y : f[e >> 1].x));
              }
            } else {
              // the row's powers lie from a place of its own on; masked scores go whatever they are
              const float* f = pw + hb * 16 + (rev ? -(int)lane : 31 - (int)lane);
              const uint32_t keep = (rev ? 0xFFFFFFFFu << lane : 0xFFFFFFFFu >> (31 - lane)) >> (hb * 16);
              float w[16];
#pragma unroll
              for (int e = 0; e < 16; ++e) w[e] = f[e];
              tmem_wait_ld();
#pragma unroll
              for (int e = 0; e < 16; ++e) w[e] = keep >> e & 1 ? __uint_as_float(s[e]) * w[e] : 0.f;
#pragma unroll
              for (int e = 0; e < 8; ++e) out[e] = pack_bf16x2(w[2 * e], w[2 * e + 1]);
            }
            if (n < kChunk) {
              const int cols = q * 32 + (int)lane < n ? n - block * 32 - hb * 16 : 0;  // real columns
#pragma unroll
              for (int e = 0; e < 8; ++e)
                out[e] = 2 * e + 1 < cols ? out[e] : 2 * e < cols ? out[e] & 0xFFFFu : 0u;
            }
          }
          tmem_st8(s_lane + hb * 8, out);
        }
        if (n < kChunk) {
          clear_rows<D, kDecay>(smem + rz.slot * L::kTile, tid, n);
          fence_proxy_async_smem();
        }
        tmem_wait_st();
        tc_fence_before();
        arrive_warp(&bars[kPReady]);
        // the parts' tile is free once the state product that read it is done; three parts of 64 rows fill it
        if (c > 0 && __any_sync(0xffffffffu, !lin_wait(&bars[kDwFull], ph ^ 1, ab))) { ok = false; break; }
#pragma unroll 1
        for (int a = 0; a < 2; ++a) {
          if (a == 1 && third && __any_sync(0xffffffffu, !lin_wait(&bars[kYFree], ph, ab))) { ok = false; break; }
          const float w = n == kChunk ? (a ? whole1 : whole0) : row_weight(l2, a * kHalf + tid / 8, n, rev, 0);
          decay_half<D>(y, parts + (third ? 0 : a * kHalf * D * 2), a * kHalf, tid, w, n, third);
          fence_proxy_async_smem();
          arrive_warp(&bars[a ? kYReady2 : kYReady]);
        }
        if (!ok) break;
      }
    }
  } else {
    // ------------------------------------------------------------ output rows, state
    regs_inc<kOutRegs>();
    const int q = warp & 3, half = (warp - 4 - kDecay / 32) >> 2;
    constexpr int kCols = D / 2;  // columns of a thread, of its output row and of its state row
    const int r = q * 32 + lane, z0 = half * kCols, d = D == 128 ? 128 : p.d;
    const bool owner = r < D;     // has a row of W
    __nv_bfloat16* out_base = static_cast<__nv_bfloat16*>(jb.o.p);
    // The warp's 32 rows x kCols columns leave through 4 KB (2 KB) of shared memory and TMA: a thread has a row, and 32
    // rows' pieces in one store instruction take it 32 turns.  At D = 128 that memory is the part of W's tile that this
    // warp itself publishes: W has been read when O is complete, and is not written before the store has read.
    uint8_t* stage = smem + L::kStage + (D == 128 ? half * D * 128 + q * 4096 : (half * 4 + q) * 2048);
    const MapRef om(maps.m[jb.mo]);
    const float alpha = __uint_as_float(fresh(__float_as_uint(p.alpha)));
    const uint32_t N = fresh(p.N);
    uint64_t W[kCols / 2];  // pairs of columns
    auto staged = [&] {  // this warp's last store has read its rows
      if (lane == 0) store_wait();
      __syncwarp();
    };
    auto publish = [&] {  // bf16(W) for the read
      if (D == 128) staged();
      if (owner) {
        uint8_t* row = smem + L::kW + (z0 >> 6) * D * 128 + r * 128;
#pragma unroll
        for (int e = 0; e < kCols / 8; ++e) {
          const int unit = ((z0 & 63) >> 3) + e;
          *reinterpret_cast<uint4*>(row + ((unit ^ (r & 7)) << 4)) =
              make_uint4(f32x2_to_bf16x2(W[4 * e]), f32x2_to_bf16x2(W[4 * e + 1]), f32x2_to_bf16x2(W[4 * e + 2]),
                         f32x2_to_bf16x2(W[4 * e + 3]));
        }
      }
      fence_proxy_async_smem();
      arrive_warp(&bars[kWReady]);
    };
    int c = 0;
    bool ok = true, waited = false;  // for the scan: the other warps need the call's inputs only
    for (long long t = t_begin; t < t_end && ok;) {
      const LinPiece pc(t, t_end, pl);
      t += pc.u1 - pc.u0;
      const int b = pc.bh / p.H, h = pc.bh % p.H, len = lin_length(p.lengths, b, p.N);
      int ua, ub;
      lin_real(pc.u0, pc.u1, len, pl, rev, ua, ub);
      const float log_decay = p.log_decay[h], l2 = lin_log2_decay(log_decay);
      __nv_bfloat16* o = out_base + b * jb.o.sb + h * jb.o.sh;
      // chunks behind the sequence
#pragma unroll 1
      for (int u = pc.u0; u < pc.u1; ++u) {
        const int row0 = (rev ? pl.nc - 1 - u : u) * kChunk, lg = D == 128 ? 4 : d == 64 ? 3 : 2;  // 2^lg units in a row
        const int units = min(kChunk, p.N - row0) << lg;
        if (row0 < len) continue;
#pragma unroll 1
        for (int i = threadIdx.x - 128 - kDecay; i < units; i += kOut)
          *reinterpret_cast<uint4*>(o + (long long)(row0 + (i >> lg)) * jb.o.sn + (i & ((1 << lg) - 1)) * 8) =
              make_uint4(0, 0, 0, 0);
      }
      // the state before the piece
      if (!waited) pdl_wait();
      waited = true;
      const float* src = nullptr;
      float mul = 1.f;
      if (pc.u0 > 0) {
        src = jb.s_in + (long long)range * d * d;
      } else if (jb.s_head && pc.u1 < pl.nc) {
        src = jb.s_head + (long long)range * d * d;
      } else if (jb.init) {
        src = jb.init + b * jb.init_stride + (long long)h * d * d;
        mul = jb.init_mul;
      }
      const bool mine = owner && r < d && z0 < d;
#pragma unroll
      for (int e = 0; e < kCols / 2; ++e) W[e] = 0;
      if (src && mine) {
#pragma unroll
        for (int e = 0; e < kCols; e += 4) {
          if (jb.transposed) {
#pragma unroll
            for (int k = 0; k < 4; k += 2)
              W[(e + k) / 2] = f32x2_pack(mul * src[(z0 + e + k) * d + r], mul * src[(z0 + e + k + 1) * d + r]);
          } else {
            const float4 a = *reinterpret_cast<const float4*>(src + r * d + z0 + e);
            W[e / 2] = f32x2_pack(mul * a.x, mul * a.y);
            W[e / 2 + 1] = f32x2_pack(mul * a.z, mul * a.w);
          }
        }
      }
      const float f_whole = alpha * lin_pow(l2, rev ? kChunk - 1 - r : r + 1);
      LinFactors g_whole(log_decay, kChunk);
      if (ua < ub) publish();
      for (int u = ua; u < ub; ++u, ++c) {
        const int row0 = (rev ? pl.nc - 1 - u : u) * kChunk, n = min(len - row0, kChunk);
        const uint32_t ph = c & 1;
        if (__any_sync(0xffffffffu, !lin_wait(&bars[kOFull], ph, ab))) { ok = false; break; }
        tc_fence_after();
        const float f = n == kChunk ? f_whole : alpha * lin_pow(l2, rev ? max(n - 1 - r, 0) : r + 1);
        const uint64_t f2 = f32x2_pack(f, f), a2 = f32x2_pack(alpha, alpha);
        if (D == 64) staged();
#pragma unroll 1
        for (int e = 0; e < kCols; e += 16) {
          uint32_t w[8];
#pragma unroll
          for (int g = 0; g < 2; ++g) {
            uint32_t o1[8], o2[8];
            tmem_ld8(tmem_addr(tmem + kColO1, q * 32, z0 + e + 8 * g), o1);
            tmem_ld8(tmem_addr(tmem + kColO2, q * 32, z0 + e + 8 * g), o2);
            tmem_wait_ld();
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const uint64_t x1 = f32x2_pack(__uint_as_float(o1[2 * k]), __uint_as_float(o1[2 * k + 1]));
              const uint64_t x2 = f32x2_pack(__uint_as_float(o2[2 * k]), __uint_as_float(o2[2 * k + 1]));
              float v0, v1;
              f32x2_unpack(f32x2_fma(f2, x2, f32x2_mul(a2, x1)), v0, v1);
              w[4 * g + k] = r < n ? pack_bf16x2(v0, v1) : 0u;
            }
          }
          const int unit = e / 8;
          if (D == 128) {
            *reinterpret_cast<uint4*>(stage + lane * 128 + ((unit ^ (lane & 7)) << 4)) = make_uint4(w[0], w[1], w[2], w[3]);
            *reinterpret_cast<uint4*>(stage + lane * 128 + (((unit + 1) ^ (lane & 7)) << 4)) = make_uint4(w[4], w[5], w[6], w[7]);
          } else {
            const int turn = (lane >> 1) & 3;
            *reinterpret_cast<uint4*>(stage + lane * 64 + ((unit ^ turn) << 4)) = make_uint4(w[0], w[1], w[2], w[3]);
            *reinterpret_cast<uint4*>(stage + lane * 64 + (((unit + 1) ^ turn) << 4)) = make_uint4(w[4], w[5], w[6], w[7]);
          }
        }
        tc_fence_before();
        fence_proxy_async_smem();
        arrive_warp(&bars[kOFree]);
        if (lane == 0 && row0 + q * 32 < (int)N && z0 < d)
          tma_store_4d(om.map, stage, z0, h * (int)om.mh, row0 + q * 32, b * (int)om.mb);
        if (__any_sync(0xffffffffu, !lin_wait(&bars[kDwFull], ph, ab))) { ok = false; break; }
        tc_fence_after();
        const float g = n == kChunk ? g_whole.next() : lin_pow(l2, n);
        const uint64_t g2 = f32x2_pack(g, g);
        if (q * 32 < D) {
#pragma unroll
          for (int e = 0; e < kCols; e += 16) {
            uint32_t x[16];
            tmem_ld16(tmem_addr(tmem + kColDw, q * 32, z0 + e), x);
            tmem_wait_ld();
#pragma unroll
            for (int k = 0; k < 16; k += 2)
              W[(e + k) / 2] = f32x2_fma(g2, W[(e + k) / 2], f32x2_pack(__uint_as_float(x[k]), __uint_as_float(x[k + 1])));
          }
        }
        tc_fence_before();
        if (u + 1 < ub) publish();
      }
      if (ok && pc.u1 == pl.nc && jb.final_out && mine) {
        float* dst = jb.final_out + b * jb.final_stride + (long long)h * d * d;
#pragma unroll
        for (int e = 0; e < kCols; e += 4) {
          float v[4];
          f32x2_unpack(W[e / 2], v[0], v[1]);
          f32x2_unpack(W[e / 2 + 1], v[2], v[3]);
          if (jb.transposed) {
#pragma unroll
            for (int k = 0; k < 4; ++k) dst[(z0 + e + k) * d + r] = jb.final_mul * v[k];
          } else {
            *reinterpret_cast<float4*>(dst + r * d + z0 + e) =
                make_float4(jb.final_mul * v[0], jb.final_mul * v[1], jb.final_mul * v[2], jb.final_mul * v[3]);
          }
        }
      }
    }
    staged();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (threadIdx.x == 0) report(*ab, p.status, p.record, 20);
  if (warp == 1) {
    mbar_drain(&bars[kDone], 0);
    tmem_dealloc(tmem, 512);
  }
}

// ------------------------------------------------------------------ the ranges' own states

namespace {

constexpr int kStMost = kLinMaxSub;  // pieces of a CTA: those of kLinSms ranges, shared by as many CTAs

template <int D>
struct StLayout {
  static constexpr int kTile = kChunk * D * 2;
  static constexpr int kSlots = D == 128 ? 5 : 8;
  static constexpr int kLo = kSlots * kTile;  // two tiles of parts
  // Second part of half `a` of chunk c: in one of the tiles, in turn; with a third part behind it, in tile a.
  static __device__ __forceinline__ int parts(int c, int a, bool third) {
    return third ? kLo + a * kTile : kLo + (c & 1) * kTile + a * kHalf * D * 2;
  }
  static constexpr int kZero = kLo + 2 * kTile;
  static constexpr int kBar = kZero + (D == 64 ? 2048 : 0);
  static constexpr int kPieces = kBar + 288;  // the CTA's pieces
  static constexpr int kBytes = kPieces + kStMost * 48 + 1024;
};
static_assert(StLayout<128>::kBytes <= 232448 && StLayout<64>::kBytes <= 232448, "shared memory of an SM");
enum { sFull = 0, sEmpty = 8, sReady = 16, sLoFree = 18, sAccFull = 20, sAccFree = 22, sDone = 24, sNumBars };
static_assert(sNumBars * 8 + 8 + sizeof(WaitRecord) <= 272, "barrier block");
constexpr int kStThreads = kTcThreads;  // roles as above: decay warps 4-19, warps 20-27 add up
constexpr uint32_t kStDecayRegs = 56, kStOutRegs = 112;
static_assert(128 * kCtlRegs + kDecay * kStDecayRegs + kOut * kStOutRegs <= kStThreads * kTcRegs, "registers of a CTA");

// One of the pieces that a CTA of the ranges' states goes through.
struct StPiece {
  const LinWalk* wk;
  int slot, h, b, len, rev, u0, u1, end;  // slot: its place among the walk's parts
  float l2;
  __device__ __forceinline__ StPiece(int i, const LinStateParams& p) {
    const LinPlan& pl = p.pl;
    wk = &p.walk[i % p.n_walks];
    slot = i / p.n_walks;
    const int range = slot / pl.sub;
    rev = wk->reverse;
    const LinCuts cuts(pl, p.lengths, p.B, p.H, p.N, rev);
    const long long t0 = cuts.start(range), t1 = cuts.start(range + 1);
    const int bh = (int)((t1 - 1) / pl.nc);
    b = bh / p.H, h = bh % p.H;
    len = lin_length(p.lengths, b, p.N);
    l2 = lin_log2_decay(p.log_decay[h]);
    const long long head0 = (long long)bh * pl.nc;
    const LinStretch st =
        lin_piece_of(lin_stretch((int)(max(t0, head0) - head0), (int)(t1 - head0), len, l2, pl, rev), slot % pl.sub, pl);
    u0 = st.u0, u1 = st.u1, end = st.end;
  }
};
static_assert(sizeof(StPiece) == 48, "room in shared memory");

}  // namespace

// part = sum over a range's stretch (linear.h) of the rows' w y^T z, w the decay to the stretch's end, in pieces.  A chunk
// whose decay to there is below fp32's range adds nothing and is not read: a head that forgets within some hundred tokens
// costs a few chunks, whatever the range.  A CTA goes through pieces gridDim apart, so that heads share the SMs evenly;
// loads run ahead into the next piece.  A chunk's products have one of two accumulators in turn, which warps 20-27 read out
// and add up in registers, where sums round to nearest: one accumulator over a whole piece cuts its sum at every step and
// was up to 4e-5 off after 80 chunks (without a decay 3e-5).  Two tiles a chunk (64 KB at head_dim 128).
template <int D>
__global__ void __launch_bounds__(kStThreads, 1) lin_states_tc(const __grid_constant__ LinTcMaps maps,
                                                               const __grid_constant__ LinStateParams p) {
  using L = StLayout<D>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + L::kBar);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + L::kBar + sNumBars * 8);
  WaitRecord* ab = reinterpret_cast<WaitRecord*>(smem + L::kBar + sNumBars * 8 + 8);
  const LinPlan& pl = p.pl;
  // the CTA's pieces, gridDim apart
  StPiece* pieces = reinterpret_cast<StPiece*>(smem + L::kPieces);
  const int n_pieces = (p.n_walks * pl.grid * pl.sub - blockIdx.x + gridDim.x - 1) / gridDim.x;
  pdl_release();
  const uint32_t warp = warp_id(), lane = lane_id();

  if (threadIdx.x == 0) {
    for (int s = 0; s < L::kSlots; ++s) {
      mbar_init(&bars[sFull + s], 1);
      mbar_init(&bars[sEmpty + s], 1);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(&bars[sReady + a], kDecay / 32);
      mbar_init(&bars[sLoFree + a], 1);
      mbar_init(&bars[sAccFull + a], 1);
      mbar_init(&bars[sAccFree + a], kOut / 32);
    }
    mbar_init(&bars[sDone], 1);
    ab->given_up = 0;
    fence_mbar_init();
  }
  if (warp == 2)
    for (int k = 0; k < n_pieces; ++k) {
      const StPiece pc(blockIdx.x + k * gridDim.x, p);
      if (lane == 0) pieces[k] = pc;
    }
  if (D == 64)
    for (int i = threadIdx.x; i < 2048 / 16; i += kStThreads)
      reinterpret_cast<uint4*>(smem + L::kZero)[i] = make_uint4(0, 0, 0, 0);
  fence_proxy_async_smem();
  if (warp == 1) {
    tmem_alloc(tmem_slot, 256);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  if (warp < 4) {
    regs_dec<kCtlRegs>();
    if (warp == 0 && lane == 0) {
      int i = 0;
      bool ok = true;
      for (int k = 0; k < n_pieces && ok; ++k) {
        const StPiece& pc = pieces[k];
        if (pc.u0 == pc.u1) continue;
        const MapRef my(maps.m[pc.wk->my]), mz(maps.m[pc.wk->mz]);
        for (int u = pc.u0; u < pc.u1 && ok; ++u) {
          const int row = (pc.rev ? pl.nc - 1 - u : u) * kChunk;
#pragma unroll
          for (int j = 0; j < 2; ++j, ++i) {
            const int s = i % L::kSlots;
            if (!lin_wait(&bars[sEmpty + s], ((i / L::kSlots) & 1) ^ 1, ab)) {
              ok = false;
              break;
            }
            load_tile<D>(smem + s * L::kTile, j ? mz : my, &bars[sFull + s], pc.h, row, pc.b);
          }
        }
      }
      if (!ok)
        for (int k = (i > L::kSlots ? i - L::kSlots : 0); k < i; ++k)
          mbar_drain(&bars[sFull + k % L::kSlots], (k / L::kSlots) & 1);
    } else if (warp == 1) {
      const uint32_t base = smem_u32(smem);
      auto wait = [&](uint64_t* bar, uint32_t ph) {
        const bool got = __all_sync(0xffffffffu, lin_wait(bar, ph, ab));
        tc_fence_after();
        return got;
      };
      bool ok = true;
      int c = 0;  // chunks
      for (int k = 0; k < n_pieces && ok; ++k) {
        const StPiece& pc = pieces[k];
        for (int u = pc.u0; u < pc.u1 && ok; ++u, ++c) {
          const int ty = 2 * c, tz = ty + 1, buf = c & 1;
          const uint32_t acc = tmem + buf * 128;
          const int n_parts = third_part(pc.l2, lin_rows(u + 1, pc.end, pc.len, pl, pc.rev)) ? 3 : 2;
          if (c > 1 && !(ok = wait(&bars[sAccFree + buf], ((c >> 1) & 1) ^ 1))) break;
          if (!(ok = wait(&bars[sFull + tz % L::kSlots], (tz / L::kSlots) & 1))) break;
          if (!(ok = wait(&bars[sReady + buf], (c >> 1) & 1))) break;
          const uint32_t y = base + ty % L::kSlots * L::kTile, z = base + tz % L::kSlots * L::kTile;
          if (elect_one()) {
#pragma unroll 1
            for (int a = 0; a < 2; ++a)
              mma_small<D>(acc, base + L::parts(c, a, n_parts == 3), base + L::kZero, z + a * kHalf * 128, a, n_parts);
#pragma unroll 1
            for (int a = 0; a < 2; ++a)
              mma_first<D>(acc, y + a * kHalf * 128, base + L::kZero, z + a * kHalf * 128);
            mma_commit(&bars[sEmpty + ty % L::kSlots]);
            mma_commit(&bars[sEmpty + tz % L::kSlots]);
            mma_commit(&bars[sLoFree + buf]);
            mma_commit(&bars[sAccFull + buf]);
          }
          __syncwarp();
        }
      }
      if (elect_one()) mma_commit(&bars[sDone]);
      __syncwarp();
    }
  } else if (warp < 4 + kDecay / 32) {
    regs_dec<kStDecayRegs>();
    const int tid = threadIdx.x - 128;
    bool ok = true;
    int c = 0;
    bool both = false;  // the chunk before takes both tiles of parts
    for (int k = 0; k < n_pieces && ok; ++k) {
      const StPiece& pc = pieces[k];
      for (int u = pc.u0; u < pc.u1; ++u, ++c) {
        const int row0 = (pc.rev ? pl.nc - 1 - u : u) * kChunk, n = min(pc.len - row0, kChunk);
        const int ty = 2 * c, tz = ty + 1, more = lin_rows(u + 1, pc.end, pc.len, pl, pc.rev);
        bool got = lin_wait(&bars[sFull + ty % L::kSlots], (ty / L::kSlots) & 1, ab);
        if (got && n < kChunk) got = lin_wait(&bars[sFull + tz % L::kSlots], (tz / L::kSlots) & 1, ab);
        if (__any_sync(0xffffffffu, !got)) { ok = false; break; }
        // the tiles of parts that this chunk takes are free: the products of the chunk before, or of the one before that
        const bool third = third_part(pc.l2, more);
        const int after = c - (third || both ? 1 : 2);
        if (after >= 0 && __any_sync(0xffffffffu, !lin_wait(&bars[sLoFree + (after & 1)], (after >> 1) & 1, ab))) {
          ok = false;
          break;
        }
        both = third;
        if (n < kChunk) clear_rows<D, kDecay>(smem + tz % L::kSlots * L::kTile, tid, n);
#pragma unroll 1
        for (int a = 0; a < 2; ++a)
          decay_half<D>(smem + ty % L::kSlots * L::kTile, smem + L::parts(c, a, third), a * kHalf, tid,
                        row_weight(pc.l2, a * kHalf + tid / 8, n, pc.rev, more), n, third);
        fence_proxy_async_smem();
        arrive_warp(&bars[sReady + (c & 1)]);
      }
    }
  } else {
    // sums of the chunks' products: a thread has half a row
    regs_inc<kStOutRegs>();
    const int q = warp & 3, half = (warp - 4 - kDecay / 32) >> 2;
    constexpr int kCols = D / 2;
    const int r = q * 32 + lane, z0 = half * kCols, d = D == 128 ? 128 : p.d;
    uint64_t W[kCols / 2];  // pairs of columns
    bool ok = true;
    int c = 0;
    for (int k = 0; k < n_pieces && ok; ++k) {
      const StPiece& pc = pieces[k];
      if (pc.u0 == pc.u1) continue;
#pragma unroll
      for (int e = 0; e < kCols / 2; ++e) W[e] = 0;
      for (int u = pc.u0; u < pc.u1; ++u, ++c) {
        const int buf = c & 1;
        if (__any_sync(0xffffffffu, !lin_wait(&bars[sAccFull + buf], (c >> 1) & 1, ab))) { ok = false; break; }
        tc_fence_after();
        if (q * 32 < D) {
#pragma unroll
          for (int e = 0; e < kCols; e += 16) {
            uint32_t x[16];
            tmem_ld16(tmem_addr(tmem + buf * 128, q * 32, z0 + e), x);
            tmem_wait_ld();
#pragma unroll
            for (int i = 0; i < 16; i += 2)
              W[(e + i) / 2] = f32x2_add(W[(e + i) / 2], f32x2_pack(__uint_as_float(x[i]), __uint_as_float(x[i + 1])));
          }
        }
        tc_fence_before();
        arrive_warp(&bars[sAccFree + buf]);
      }
      if (ok && r < d && z0 < d) {
        float* dst = pc.wk->parts + (long long)pc.slot * d * d + (long long)r * d + z0;
#pragma unroll
        for (int e = 0; e < kCols; e += 4) {
          float v[4];
          f32x2_unpack(W[e / 2], v[0], v[1]);
          f32x2_unpack(W[e / 2 + 1], v[2], v[3]);
          *reinterpret_cast<float4*>(dst + e) = make_float4(v[0], v[1], v[2], v[3]);
        }
      }
      __syncwarp();
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (threadIdx.x == 0) report(*ab, p.status, p.record, 21);
  if (warp == 1) {
    mbar_drain(&bars[sDone], 0);
    tmem_dealloc(tmem, 256);
  }
}

namespace {

template <int D, bool kSplit>
cudaError_t out_tc(const LinTcMaps& m, const LinOutParams& p, cudaStream_t st) {
  static std::atomic<unsigned long long> done{0};
  // the warps' register shares are drawn from what the CTA was launched with
  const cudaError_t e = lin_prepare((const void*)lin_out_tc<D, kSplit>, TcLayout<D>::kBytes, kTcRegs, done);
  if (e != cudaSuccess) return e;
  if (kSplit) return launch_after(lin_out_tc<D, kSplit>, p.n_jobs * p.pl.grid, kTcThreads, TcLayout<D>::kBytes, st, m, p);
  lin_out_tc<D, kSplit><<<p.n_jobs * p.pl.grid, kTcThreads, TcLayout<D>::kBytes, st>>>(m, p);
  return cudaGetLastError();
}

template <int D>
cudaError_t states_tc(const LinTcMaps& m, const LinStateParams& p, cudaStream_t st) {
  static std::atomic<unsigned long long> done{0};
  const cudaError_t e = lin_prepare((const void*)lin_states_tc<D>, StLayout<D>::kBytes, kTcRegs, done);
  if (e != cudaSuccess) return e;
  const int pieces = p.n_walks * p.pl.grid * p.pl.sub;
  if (pieces > kStMost * kLinSms) return cudaErrorInvalidValue;  // no plan has more
  lin_states_tc<D><<<std::min(kLinSms, pieces), kStThreads, StLayout<D>::kBytes, st>>>(m, p);
  return cudaGetLastError();
}

}  // namespace

cudaError_t lin_prepare(const void* kernel, int smem_bytes, int min_regs, std::atomic<unsigned long long>& done) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const unsigned long long bit = dev < 64 ? 1ull << dev : 0ull;
  if (done.load(std::memory_order_acquire) & bit) return cudaSuccess;
  cudaFuncAttributes a;
  if ((e = cudaFuncGetAttributes(&a, kernel)) != cudaSuccess) return e;
  if (a.numRegs < min_regs) return cudaErrorInvalidConfiguration;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem_bytes);
  if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_release);
  return e;
}

cudaError_t launch_lin_out_tc(const LinTcMaps& m, const LinOutParams& p, cudaStream_t st) {
  if (p.pl.split) return p.d == 128 ? out_tc<128, true>(m, p, st) : out_tc<64, true>(m, p, st);
  return p.d == 128 ? out_tc<128, false>(m, p, st) : out_tc<64, false>(m, p, st);
}

cudaError_t launch_lin_states_tc(const LinTcMaps& m, const LinStateParams& p, cudaStream_t st) {
  return p.d == 128 ? states_tc<128>(m, p, st) : states_tc<64>(m, p, st);
}

// [B, N, H, d] view: dimensions (d, H, N, B), box 64 x 1 x 128 x 1, 128-byte swizzle, zeros out of bounds.  A dimension
// of one entry, or broadcast (stride 0), becomes one entry with coordinate 0.
// For an output: the box of one output warp, 32 rows of 64 columns (head_dim 128) or of 32 with the 64-byte swizzle.
bool make_lin_map(LinMap* m, const LinView& v, int B, int N, int H, int d, bool output) {
  EncodeTiledFn fn = encode_fn();
  if (!fn) return false;
  m->mh = H > 1 && v.sh != 0;
  m->mb = B > 1 && v.sb != 0;
  const cuuint64_t dims[4] = {(cuuint64_t)d, (cuuint64_t)(m->mh ? H : 1), (cuuint64_t)N, (cuuint64_t)(m->mb ? B : 1)};
  const cuuint64_t strides[3] = {(cuuint64_t)(m->mh ? v.sh * 2 : 16), (cuuint64_t)(N > 1 ? v.sn * 2 : 16),
                                 (cuuint64_t)(m->mb ? v.sb * 2 : 16)};
  const bool half_box = output && d != 128;
  const cuuint32_t box[4] = {half_box ? 32u : 64u, 1, output ? 32u : kChunk, 1}, estr[4] = {1, 1, 1, 1};
  return fn(&m->map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, v.p, dims, strides, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, half_box ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace vdn
