// Attention kernel over 4-bit cache rows (packed384) (sm_103a).
//
// The same function, plan, pieces and transposed products as the kernel of
// the other row formats (qsfm_attention.cu):
//   S^T[j, h]  = sum_d K~[j, d] Q[h, d]      (M = 128 rows, N = 64 heads, K = 512)
//   O^T[d, h] += sum_j V~[j, d] P[h, j]      (M = 128 d per chunk, N = 64, K = 128 rows)
// with K~ = V~ = code * scale * 2^(exponent - 127): two, four and one
// significant bits, so a dequantised element is exact in bf16 and both
// operands of the score product are the inputs' own values.
//
// What differs is the division of labour: the softmax warps never wait for a
// load, and as much of the codes' conversion as registers hold is off the chain.
//   warps 0-7    softmax and epilogue: warp w reads tensor-memory lanes
//                32 (w % 4) .. + 31 and heads 32 (w / 4) .. + 31;
//   warps 8-15   producers: thread (row r, half h) converts and stores d-block
//                2c + h of chunk c of its row: 32-byte loads, so a warp's load
//                touches whole sectors, and a row's 16-byte units land in the
//                eight bank groups of the swizzle. Two chunks are converted to
//                registers ahead of PV freeing their places, so that only
//                their stores follow;
//   warp 16      MMA issue;
//   warp 17      resolver: walks the CTA's pieces (work units, or parts of one)
//                and publishes them and their tiles' rows in two rings, so that
//                no other warp waits for a length or an index (18 and 19 only
//                complete the warpgroup).
// Chain per tile: PV(n) frees chunk pairs -> stores of tile n + 1 -> QK^T(n + 1)
// chunk by chunk -> softmax(n + 1) -> PV(n + 1). A unit's output is read, scaled
// and written after the next unit's first P is on its way: O^T takes four of
// seven blocks of tensor memory, the next unit's the following four (modulo
// seven), so its PV waits only for the first chunk to be read. The next unit's q
// is requested as soon as the last score product of the unit has completed.
//
// What bounds it, per tile of 128 rows x 64 heads: the 64 MMAs read 6 KB of shared
// memory each, 48 cycles at 128 B / cycle (48.8 measured, issued back to back, and the
// same beside busy warps), where the tensor pipe alone would take 32; K~ takes 1024
// cycles to store and the codes some 2000 issue cycles to convert (28 elements / cycle /
// SM: the conversion to f16 pairs, to fp32, one packed product, one to bf16). The chain
// above runs them partly in turn: about 7100 cycles per tile, 3.6 us. Measured on 152
// SMs: prefill in chunks (128 heads, 640 rows per token) 590 us, 683 TFLOP/s; windows of
// 128 rows for 8192 tokens 285 us, 3.8 TB/s of q, output and cache (a unit's output
// takes the softmax warps some 5000 of 9000 cycles: their issue slots and the shared
// memory are the MMAs' and producers' as well, and all roles' loops together are more
// code than the instruction caches next to the schedulers hold: every variant with more
// of it ran slower, whatever it saved); 128 requests of 2 tokens x 640 rows 47 us; 64 of
// 1 token on up to 1152 rows 36 us, both with the plan (3 us), and 10 us of them start
// and end.
#include <atomic>

#include "qsfm_attention_common.cuh"

namespace qsfm {
namespace {

constexpr int kSmWarps = 8;                  // softmax / epilogue
constexpr int kSmThreads = kSmWarps * 32;
constexpr int kPrWarps = 8;                  // producers
constexpr int kMmaWarp = kSmWarps + kPrWarps;
constexpr int kResolverWarp = kMmaWarp + 1;
constexpr int kThreads = (kMmaWarp + 4) * 32;
// Registers per thread: 96 at launch (five warps on an SM sub-partition), then
// 96 for the softmax warps, 112 for the producers, 64 for the last warpgroup.
constexpr int kLaunchRegs = 96, kPrRegs = 112, kLastRegs = 64;
static_assert(kSmThreads * kLaunchRegs + kPrWarps * 32 * kPrRegs + 128 * kLastRegs <= kThreads * kLaunchRegs,
              "register split");
constexpr int kHPT = 32;                     // heads per softmax thread
constexpr int kBarSm = 1;                    // named barriers: the softmax warps, the start
constexpr int kBarSetup = 2;
constexpr int kRowB = QSFM_PACKED384_ROW_BYTES;
constexpr int kTileRing = 4;                 // tiles, and pieces, that the resolver may be ahead

// shared memory map (byte offsets from a 1024-aligned base)
constexpr uint32_t kSlabBytes = kTileRows * 128;              // 128 rows x 64 d (bf16): 16 KB
constexpr uint32_t kSK = 0;                                   // K~ tile: 8 slabs
constexpr uint32_t kSQ = kSK + 8 * kSlabBytes;                // Q: 8 d-blocks x 64 heads x 128 B
constexpr uint32_t kSP = kSQ + 8 * 64 * 128;                  // P: 128 rows x 64 heads (bf16)
constexpr uint32_t kSRows = kSP + kTileRows * 128;            // [ring][128] i32 physical rows
constexpr uint32_t kSTile = kSRows + kTileRing * kTileRows * 4;  // [ring] i32: what the slot holds
constexpr uint32_t kSPiece = kSTile + kTileRing * 4;          // [ring] pieces, then two being handed over
constexpr uint32_t kSValid = kSPiece + (kTileRing + 2) * 16;  // [128] i32: row of the tile valid
constexpr uint32_t kSRed = kSValid + kTileRows * 4;           // [4][64] f32 per-quadrant partials
constexpr uint32_t kSMUsed = kSRed + 1024;                    // [64] f32
constexpr uint32_t kSAlpha = kSMUsed + 256;                   // [64] f32
constexpr uint32_t kSInv = kSAlpha + 256;                     // [2][64] f32: by the unit's parity
constexpr uint32_t kSSink = kSInv + 512;                      // [128] f32: the heads' sinks, log2 units
constexpr uint32_t kSAny = kSSink + 512;                      // [4] i32: a row of the quadrant valid
constexpr uint32_t kSBar = kSAny + 16;                        // mbarriers, tmem base, flags
constexpr uint32_t kSmemBytes = kSBar + 384;
static_assert(kSValid % 16 == 0 && kSAny % 16 == 0 && kSBar % 16 == 0, "alignment");
constexpr uint32_t kSmemAlloc = kSmemBytes + 1024;
static_assert(kSmemAlloc <= 232448, "more than the 227 KB a CTA may use");

// mbarrier slots
constexpr int kBarQFull = 0;
constexpr int kBarFull = 1;        // [chunk]: stored (one arrive per producer warp)
constexpr int kBarFree = 5;        // [chunk pair]: PV of chunks 2i, 2i + 1 completed (commit)
constexpr int kBarSFull = 7;       // S^T of the tile complete (commit)
constexpr int kBarPFull = 8;       // P of the tile written (one arrive per softmax warp)
constexpr int kBarOFree = 9;       // chunk 0 of O^T read by the epilogue (one arrive per softmax warp)
constexpr int kBarDrain = 10;      // every MMA of the CTA completed (commit)

constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kTmemS = 0;
// O^T of the CTA's i-th piece with tiles: chunk c in columns 64 .. 127 of block
// (4 i + c) mod 7 behind S^T
__device__ __forceinline__ uint32_t o_column(uint32_t piece, int c) { return 64 + 64 * ((4 * piece + uint32_t(c)) % 7); }
constexpr float kGuessLog2 = 60.0f;  // below a guessed maximum
constexpr uint32_t kIdescQK = make_idesc_bf16(128, 64, /*a_mn=*/0, /*b_mn=*/0);
constexpr uint32_t kIdescPV = make_idesc_bf16(128, 64, /*a_mn=*/1, /*b_mn=*/1);

// What the resolver says of a ring slot (a KV tile): its pool, and its place in
// the piece; or the end.
constexpr int kTileEnd = -1, kTileCmp = 1, kTileFirst = 2, kTileLast = 4;
// A piece: tiles of a work unit (none: a unit without rows), all or a part of
// them; unit -1: the end.
struct __align__(16) Piece {
  int unit, tiles, whole, unused;  // 16 bytes, copied at once
};

struct Smem {
  static constexpr int kRing = kTileRing;
  static constexpr int kBarRowsFull = 11;                // [ring slot]
  static constexpr int kBarRowsEmpty = 11 + kRing;       // [ring slot]: one arrive per producer warp and the MMA warp
  static constexpr int kBarPieceFull = 11 + 2 * kRing;   // [ring slot]
  static constexpr int kBarPieceEmpty = 11 + 3 * kRing;  // [ring slot]
  static constexpr int kNumBars = 11 + 4 * kRing;
  uint32_t base;
  uint8_t* ptr;
  __device__ float* f(uint32_t off) const { return reinterpret_cast<float*>(ptr + off); }
  __device__ int* ring_rows() const { return reinterpret_cast<int*>(ptr + kSRows); }
  __device__ int* tiles() const { return reinterpret_cast<int*>(ptr + kSTile); }
  __device__ Piece* pieces() const { return reinterpret_cast<Piece*>(ptr + kSPiece); }
  __device__ int* valid() const { return reinterpret_cast<int*>(ptr + kSValid); }
  __device__ int* any() const { return reinterpret_cast<int*>(ptr + kSAny); }
  __device__ uint64_t* bar(int i) const { return reinterpret_cast<uint64_t*>(ptr + kSBar) + i; }
  __device__ uint32_t* tmem_slot() const { return reinterpret_cast<uint32_t*>(ptr + kSBar + 352); }
  __device__ volatile int* abort_flag() const { return reinterpret_cast<volatile int*>(ptr + kSBar + 360); }
};
static_assert(Smem::kNumBars * 8 <= 352, "barriers overlap the tmem slot");

template <int kRegs>
__device__ __forceinline__ void more_registers() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegs));
}
template <int kRegs>
__device__ __forceinline__ void fewer_registers() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegs));
}

// Bounded waits as wait_or_abort(), but suspended in hardware: try_wait gets a
// time to stay blocked (20 us), so a waiting warp takes no issue slots from the
// producers, and no sleep delays it once the phase completes. All lanes of a
// warp wait together.
constexpr uint32_t kSuspendNs = 20000;
__device__ __forceinline__ bool mbar_suspend(uint32_t addr, uint32_t parity) {
  uint32_t done;
  asm volatile(
      "{\n .reg .pred p;\n"
      " mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n"
      " selp.u32 %0, 1, 0, p;\n}"
      : "=r"(done)
      : "r"(addr), "r"(parity), "r"(kSuspendNs)
      : "memory");
  return done != 0;
}
__device__ __forceinline__ uint32_t globaltimer_lo() {  // wraps after 4.3 s, past the limit of a wait
  uint32_t t;
  asm volatile("mov.u32 %0, %globaltimer_lo;" : "=r"(t));
  return t;
}
__device__ __forceinline__ bool wait_fast(const Smem& sm, int bar, uint32_t parity, int* fault) {
  const uint32_t addr = smem_u32(sm.bar(bar));
  if (mbar_suspend(addr, parity)) return true;
  const uint32_t start = globaltimer_lo();
  while (!mbar_suspend(addr, parity)) {
    if (*sm.abort_flag()) return false;
    if (globaltimer_lo() - start > uint32_t(kTimeoutNs)) {
      *sm.abort_flag() = 1;
      atomicOr(fault, QSFM_FAULT_TIMEOUT);
      return false;
    }
  }
  return true;
}
__device__ __forceinline__ bool warp_wait_fast(const Smem& sm, int bar, uint32_t parity, int* fault) {
  const bool ok = wait_fast(sm, bar, parity, fault);
  return __all_sync(0xffffffffu, ok);  // the lanes of a warp never split on a timeout
}

// Waits for the tensor-memory loads into v (the registers pass through the
// statement, so nothing that uses them moves above it).
__device__ __forceinline__ void tmem_ld_wait_for(float (&v)[32]) {
  tmem_ld_wait();
#pragma unroll
  for (int i = 0; i < 32; ++i) asm volatile("" : "+f"(v[i]));
}

// ------------------------------------------------------------- MMA issue
// The whole warp runs the issue loop and one elected lane (always the same one)
// issues: descriptors and addresses are then provably the same in every lane and
// stay in uniform registers. A loop on one lane alone takes 60 to 100 cycles per
// MMA (each operand is moved to a uniform register in issue slots that the
// producers' conversions contend for); this one the 48 that the operands take to be
// read from shared memory (128 x 16 + 64 x 16 bf16 at 128 B / cycle).
// Descriptors of 128-byte-swizzled operands in 8-row groups of 1 KB.
constexpr uint32_t kDescHigh = (1024u >> 4) | (1u << 14) | (2u << 29);  // group stride, version, swizzle
__device__ __forceinline__ uint32_t desc_low(uint32_t saddr, uint32_t lbo) {
  return ((saddr >> 4) & 0x3FFFu) | ((lbo >> 4) << 16);
}
// a, b: low words of the operands' descriptors; the high words are all alike.
template <uint32_t kAOff, uint32_t kBOff, uint32_t kIdesc>
__device__ __forceinline__ void mma_elected(uint32_t d, uint32_t a, uint32_t b, uint32_t accumulate) {
  asm volatile(
      "{\n .reg .pred p, e;\n .reg .b32 x, y;\n .reg .b64 a, b;\n add.u32 x, %1, %6;\n add.u32 y, %2, %7;\n"
      " mov.b64 a, {x, %5};\n mov.b64 b, {y, %5};\n"
      " setp.ne.b32 p, %4, 0;\n elect.sync _|e, 0xffffffff;\n"
      " mov.b32 x, %3;\n @e tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, x, p;\n}" ::"r"(d),
      "r"(a), "r"(b), "n"(kIdesc), "r"(accumulate), "n"(kDescHigh), "n"(kAOff), "n"(kBOff)
      : "memory");
}
__device__ __forceinline__ void commit_elected(uint64_t* bar) {
  asm volatile(
      "{\n .reg .pred e;\n elect.sync _|e, 0xffffffff;\n"
      " @e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n}" ::"r"(smem_u32(bar))
      : "memory");
}

// QK^T of chunk c (d-blocks 2c, 2c + 1), k-step s of d-block db: A (K~,
// K-major) at + db * 16 KB + s * 32 B, B (Q, K-major) at + db * 8 KB + s * 32 B.
template <int kI = 0>
__device__ __forceinline__ void qk_chunk(uint32_t d, uint32_t a, uint32_t b, uint32_t acc0) {
  constexpr uint32_t db = kI / 4, st = kI % 4;
  mma_elected<((db * kSlabBytes + st * 32) >> 4), ((db * 8192 + st * 32) >> 4), kIdescQK>(d, a, b, kI == 0 ? acc0 : 1u);
  if constexpr (kI < 7) qk_chunk<kI + 1>(d, a, b, acc0);
}

// PV of head-dim chunk c, k-step s: A (V~^T, MN-major: 64-d atoms 16 KB apart,
// 8-row groups 1 KB apart) at + c * 32 KB + s * 2 KB, B (P^T, MN-major) at
// + s * 2 KB; accumulates into 64 columns of O^T.
template <int kI = 0>
__device__ __forceinline__ void pv_chunk(uint32_t d, uint32_t a, uint32_t b, uint32_t acc0) {
  mma_elected<((kI * 2048) >> 4), ((kI * 2048) >> 4), kIdescPV>(d, a, b, kI == 0 ? acc0 : 1u);
  if constexpr (kI < 7) pv_chunk<kI + 1>(d, a, b, acc0);
}

// What tile n's ring slot holds, once published; kTileEnd after an abort.
__device__ __forceinline__ int read_tile(const Smem& sm, uint32_t n, int* fault) {
  const uint32_t slot = n % Smem::kRing;
  return wait_fast(sm, Smem::kBarRowsFull + slot, (n / Smem::kRing) & 1, fault) ? sm.tiles()[slot] : kTileEnd;
}
__device__ __forceinline__ void tile_done(const Smem& sm, uint32_t n) {
  mbar_arrive(sm.bar(Smem::kBarRowsEmpty + n % Smem::kRing));
}

// Tile n of the CTA's sequence: every per-tile barrier completes once per
// tile, so a wait for tile n uses phase parity n & 1.
__device__ void mma_role(const Smem& sm, uint32_t tmem_any, int* fault) {
  const uint32_t qa = desc_low(sm.base + kSK, 16);
  const uint32_t qb = desc_low(sm.base + kSQ, 16);
  const uint32_t pa = desc_low(sm.base + kSK, kSlabBytes);
  const uint32_t pb = desc_low(sm.base + kSP, 16);
  const uint32_t tmem = __shfl_sync(0xffffffffu, tmem_any, 0);  // the same in every lane, to the compiler too
  uint32_t piece = 0;
#pragma unroll 1
  for (uint32_t n = 0;; ++n) {
    const int tile = __shfl_sync(0xffffffffu, read_tile(sm, n, fault), 0);
    if (tile == kTileEnd) return;
    if ((threadIdx.x & 31) == 0) tile_done(sm, n);
    __syncwarp();
    const bool first = tile & kTileFirst;
    const uint32_t par = n & 1;
    if (first && !warp_wait_fast(sm, kBarQFull, piece & 1, fault)) return;
#pragma unroll 1
    for (uint32_t c = 0; c < 4; ++c) {
      if (!warp_wait_fast(sm, kBarFull + c, par, fault)) return;
      tc_fence_after();
      qk_chunk(tmem + kTmemS, qa + c * (2 * kSlabBytes >> 4), qb + c * (2 * 8192 >> 4), c != 0 ? 1u : 0u);
    }
    commit_elected(sm.bar(kBarSFull));
    // P(n) written (so S^T(n) has been read; and the piece before the last has
    // been read out, which these warps did before)
    if (!warp_wait_fast(sm, kBarPFull, par, fault)) return;
    tc_fence_after();
    const uint32_t acc0 = first ? 0u : 1u;
#pragma unroll 1
    for (uint32_t c = 0; c < 4; ++c) {
      if (c == 3 && first && piece > 0) {
        // chunk 3 takes the place of the last piece's chunk 0
        if (!warp_wait_fast(sm, kBarOFree, (piece - 1) & 1, fault)) return;
        tc_fence_after();
      }
      pv_chunk(tmem + o_column(piece, c), pa + c * (2 * kSlabBytes >> 4), pb, acc0);
      if (c & 1) commit_elected(sm.bar(kBarFree + (c >> 1)));
    }
    if (tile & kTileLast) ++piece;
  }
}

// ------------------------------------------------------------- resolver
// Walks the pieces of the CTA's range: each piece goes to the ring of pieces,
// each tile's 128 physical rows (-1 = masked) to the ring of tiles; both end
// with a mark.
__device__ void resolver_role(const qsfm_params& p, const Smem& sm, Range rg, int T, int* fault) {
  const int lane = threadIdx.x & 31;
  int* rows = sm.ring_rows();
  PieceIter pieces(&p, rg, T);
  uint32_t n = 0, m = 0;  // next tile, next piece
  auto put_piece = [&](int unit, int tiles, int whole) -> bool {
    const uint32_t slot = m % Smem::kRing;
    if (!warp_wait_or_abort(sm, Smem::kBarPieceEmpty + slot, ((m / Smem::kRing) & 1) ^ 1, fault)) return false;
    if (lane == 0) {
      sm.pieces()[slot] = Piece{unit, tiles, whole, 0};
      mbar_arrive(sm.bar(Smem::kBarPieceFull + slot));
    }
    ++m;
    return true;
  };
  auto wait_tile = [&]() {
    return warp_wait_or_abort(sm, Smem::kBarRowsEmpty + n % Smem::kRing, ((n / Smem::kRing) & 1) ^ 1, fault);
  };
  auto put_tile = [&](int what) {
    if (lane == 0) sm.tiles()[n % Smem::kRing] = what;
    __syncwarp();
    if (lane == 0) mbar_arrive(sm.bar(Smem::kBarRowsFull + n % Smem::kRing));
    ++n;
  };
  int unit, lo, hi;
  TokenGeom g;
  while (pieces.next(unit, g, lo, hi)) {
    if (!put_piece(unit, max(hi - lo, 0), lo == 0 && hi == g.n_tiles ? 1 : 0)) return;
    if (lo >= hi) continue;
    // the next token's index list goes to L2 while this one is resolved (q does
    // not: what every CTA fetches ahead would drive out what the others did)
    if (p.cmp_sparse_indices != nullptr && g.tok + 1 < (T >> unit_shift(p))) {
      const uint8_t* ix = reinterpret_cast<const uint8_t*>(p.cmp_sparse_indices + (size_t)(g.tok + 1) * p.k2);
      for (int off = 128 * lane; off < 4 * p.k2; off += 32 * 128) prefetch_l2(ix + off);
    }
    for (int k0 = lo; k0 < hi; ++k0) {
      if (!wait_tile()) return;
      const int k[1] = {k0};
      const bool live[1] = {true};
      int lg[1][4], pr[1][4];
      bool cmp[1];
      resolve_tile_rows<1>(p, g, k, live, lane, fault, lg, pr, cmp);
#pragma unroll
      for (int u = 0; u < 4; ++u) rows[(n % Smem::kRing) * kTileRows + lane + 32 * u] = pr[0][u];
      put_tile((cmp[0] ? kTileCmp : 0) | (k0 == lo ? kTileFirst : 0) | (k0 == hi - 1 ? kTileLast : 0));
    }
  }
  if (put_piece(-1, 0, 0) && wait_tile()) put_tile(kTileEnd);
}

// ------------------------------------------------------------- producers
// 32 bytes (32-byte aligned), read once.
struct Raw8 {
  uint32_t w[8];
};
__device__ __forceinline__ Raw8 ldg_stream_v8(const void* ptr) {
  Raw8 r;
  asm volatile("ld.global.nc.L1::no_allocate.v8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
               : "=r"(r.w[0]), "=r"(r.w[1]), "=r"(r.w[2]), "=r"(r.w[3]), "=r"(r.w[4]), "=r"(r.w[5]), "=r"(r.w[6]),
                 "=r"(r.w[7])
               : "l"(ptr));
  return r;
}

// 64 codes with four scales (word ws) to 64 bf16.
__device__ __forceinline__ void convert64(const Raw8& codes, uint32_t ws, uint32_t exponent, uint32_t (&out)[32]) {
  const float power = e8m0_value(exponent & 0xFFu);
#pragma unroll
  for (int g = 0; g < 4; ++g) {
    const float s = scale_e4m3(ws, g, power);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint32_t w = codes.w[2 * g + i];
      const uint2 x = dequant4_e2m1(w, s), y = dequant4_e2m1(w >> 16, s);
      out[8 * g + 4 * i] = x.x;
      out[8 * g + 4 * i + 1] = x.y;
      out[8 * g + 4 * i + 2] = y.x;
      out[8 * g + 4 * i + 3] = y.y;
    }
  }
}

// d-block 2c + half of row r, every chunk c. The block of chunk 0, half 0 is the
// bf16 rope: loaded as it is stored.
__device__ void producer_role(const qsfm_params& p, const Smem& sm, int* fault) {
  const int tid = int(threadIdx.x) - kSmThreads, lane = tid & 31;
  const int half = tid >> 7, r = tid & 127;
  const bool rope = half == 0;
  const int* rows = sm.ring_rows();
  const uint32_t rowb = sm.base + kSK + uint32_t(half) * kSlabBytes + uint32_t(r) * 128;
  const uint32_t sw = uint32_t(r & 7);
  uint32_t ca[32], cb[32];  // the two converted blocks
  Raw8 ra, rb;              // codes of the blocks to convert next
  uint32_t s0 = 0, s1 = 0, s2 = 0, s3 = 0, ex = 0;  // scale words of the four blocks, the row's exponent

  auto take_rows = [&](uint32_t n, const uint8_t*& row, bool& v) -> bool {
    const int tile = read_tile(sm, n, fault);
    const int pr = rows[(n % Smem::kRing) * kTileRows + r];
    // uniform even where a wait ran out for some lanes
    if (__any_sync(0xffffffffu, tile == kTileEnd)) return false;
    if (lane == 0) tile_done(sm, n);
    v = pr >= 0;
    row = static_cast<const uint8_t*>(tile & kTileCmp ? p.cmp_kv : p.ori_kv) + size_t(v ? pr : 0) * kRowB;
    return true;
  };
  // Codes of chunk c's block: bytes 96 + 64 c + 32 half (none for the rope
  // block). A masked row's codes are read all the same (row 0 of the pool) and
  // times a scale of zero.
  auto load_codes = [&](int c, const uint8_t* row) { return ldg_stream_v8(row + 96 + 64 * c + 32 * half); };
  auto load_scales = [&](const uint8_t* row, bool v) {
    const Raw8 q = ldg_stream_v8(row + 352);
    s0 = v ? q.w[0] : 0u;
    s1 = v ? (half ? q.w[2] : q.w[1]) : 0u;
    s2 = v ? (half ? q.w[4] : q.w[3]) : 0u;
    s3 = v ? (half ? q.w[6] : q.w[5]) : 0u;
    ex = v ? q.w[7] : 0u;
  };
  auto load_rope = [&](const uint8_t* row, bool v) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const Raw8 q = ldg_stream_v8(row + 32 * i);
#pragma unroll
      for (int k = 0; k < 8; ++k) ca[8 * i + k] = v ? q.w[k] : 0u;
    }
  };
  auto store = [&](int c, const uint32_t (&conv)[32]) {  // into chunk c's place, published
    const uint32_t at = rowb + uint32_t(2 * c) * kSlabBytes;
#pragma unroll
    for (int i = 0; i < 8; ++i)
      sts_v4(at + ((uint32_t(i) ^ sw) << 4), make_uint4(conv[4 * i], conv[4 * i + 1], conv[4 * i + 2], conv[4 * i + 3]));
    fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) mbar_arrive(sm.bar(kBarFull + c));
  };

  const uint8_t* row;
  bool v;
  if (!take_rows(0, row, v)) return;
  load_scales(row, v);
  if (!rope) ra = load_codes(0, row);
  rb = load_codes(1, row);
#pragma unroll 1
  for (uint32_t n = 0;; ++n) {
    // chunk 0 is converted at once, chunk 1 behind the last tile's P (its
    // conversion would take the softmax's issue slots)
    if (rope) load_rope(row, v);
    else convert64(ra, s0, ex, ca);
    ra = load_codes(2, row);
    if (n > 0 && !warp_wait_fast(sm, kBarPFull, (n - 1) & 1, fault)) return;
    convert64(rb, s1, ex, cb);
    rb = load_codes(3, row);
    if (n > 0 && !warp_wait_fast(sm, kBarFree, (n - 1) & 1, fault)) return;
    if (rope) {
      // the tile's valid flags: the softmax has read the last tile's (its P was
      // written) and reads these after chunk 0 is published
      sm.valid()[r] = v ? 1 : 0;
      const bool any = __any_sync(0xffffffffu, v);
      if (lane == 0) sm.any()[r >> 5] = any ? 1 : 0;
    }
    store(0, ca);
    store(1, cb);
    convert64(ra, s2, ex, ca);
    if (n > 0 && !warp_wait_fast(sm, kBarFree + 1, (n - 1) & 1, fault)) return;
    store(2, ca);
    convert64(rb, s3, ex, cb);
    store(3, cb);
    // the next tile: its loads after the last store (stores queue behind loads
    // in the load/store unit)
    if (!take_rows(n + 1, row, v)) return;
    load_scales(row, v);
    if (!rope) ra = load_codes(0, row);
    rb = load_codes(1, row);
  }
}

// ------------------------------------------------------------- softmax, epilogue
__device__ void softmax_role(const qsfm_params& p, const Smem& sm, int first_unit, uint32_t tmem, const Workspace& ws,
                             int c_idx, const CUtensorMap* qmap, int* fault) {
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int qd = warp & 3;            // tensor-memory lane quadrant
  const int h0 = kHPT * (warp >> 2);  // first of this warp's heads
  const int r = 32 * qd + lane;       // tile row of this thread
  const uint32_t lane_base = uint32_t(32 * qd) << 16;
  const uint32_t s_addr = tmem + kTmemS + h0 + lane_base;
  const uint32_t prow_addr = sm.base + kSP + uint32_t(r) * 128;
  float* m_used = sm.f(kSMUsed);
  float* alpha = sm.f(kSAlpha);
  float* inv = sm.f(kSInv);
  float* red = sm.f(kSRed);
  const float qk_scale = p.softmax_scale * kLog2e;

  // q of a unit by TMA (thread 0)
  auto load_q = [&](int unit) {
    mbar_arrive_expect_tx(sm.bar(kBarQFull), kHeads * kDim * 2);
#pragma unroll
    for (int db = 0; db < 8; ++db)
      tma_load_2d(sm.base + kSQ + db * 8192, qmap, db * 64, unit * 64, sm.bar(kBarQFull));
  };

  // The next piece from the resolver, by thread 0, handed to the other warps
  // through shared memory at the next barrier (so that all of them go the same
  // way, whatever an abort does to the ring).
  uint32_t taken = 0;
  auto fetch_piece = [&](uint32_t place) {
    const uint32_t slot = taken % Smem::kRing;
    Piece q = {-1, 0, 0, 0};
    if (wait_fast(sm, Smem::kBarPieceFull + slot, (taken / Smem::kRing) & 1, fault)) {
      q = sm.pieces()[slot];
      mbar_arrive(sm.bar(Smem::kBarPieceEmpty + slot));
      ++taken;
    }
    sm.pieces()[Smem::kRing + place] = q;
    return q;
  };
  float* sinks = sm.f(kSSink);
  if (tid < p.n1) sinks[tid] = p.sinks != nullptr ? __ldg(p.sinks + tid) * kLog2e : -INFINITY;
  if (tid < 64) m_used[tid] = 0.f;  // the first unit's guess
  uint32_t handed = 0;
  if (tid == 0) {
    const Piece q = fetch_piece(0);
    if (q.tiles > 0) load_q(q.unit);
  }
  named_sync(kBarSm, kSmThreads);
  Piece cur = sm.pieces()[Smem::kRing];
  named_sync(kBarSm, kSmThreads);

  // The output of the piece before: O^T in tensor memory, its 1 / den in inv.
  struct Out {
    int unit, whole, slot;  // unit -1: none; slot -1: not written
    uint32_t piece, tile;   // among the pieces with tiles; the piece's last tile
  };
  // Reads, scales and writes it: thread (lane d of a chunk) has one element of
  // each of its 32 heads. bf16 outputs are 64 contiguous bytes per head and warp
  // in 2-byte stores: no exchange between lanes, nothing to wait for, few
  // instructions. Windows for 8192 tokens: 295 us; with 16-byte stores of what
  // stmatrix turns in shared memory 303 us, with 8-byte stores of what lanes
  // exchange 331 us.
  auto write_out = [&](const Out& o) {
    // Free[1] of its last tile: every PV product is complete. (Free[0] may be a
    // phase ahead: the next piece's PV has begun.)
    warp_wait_fast(sm, kBarFree + 1, o.tile & 1, fault);
    tc_fence_after();
    const float* iv = inv + 64 * (o.piece & 1) + h0;
    const int d0 = 32 * qd + lane;
    __nv_bfloat16* out = static_cast<__nv_bfloat16*>(p.attn_out) + (size_t(o.unit) * 64 + h0) * kDim + d0;
    float* part = ws.out + (size_t(o.slot < 0 ? 0 : o.slot) * 64 + h0) * kDim + d0;
#pragma unroll 1
    for (int c = 0; c < 4; ++c) {
      float x[kHPT];
      tmem_load(tmem + o_column(o.piece, c) + h0 + lane_base, x);
      tmem_ld_wait_for(x);
      if (c == 0) {  // the next piece's last chunk may overwrite it
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(sm.bar(kBarOFree));
      }
      if (o.whole) {
#pragma unroll
        for (int i = 0; i < kHPT; i += 4) {
          const float4 v4 = *reinterpret_cast<const float4*>(iv + i);
          const uint32_t a = pack_bf16(x[i] * v4.x, x[i + 1] * v4.y), b = pack_bf16(x[i + 2] * v4.z, x[i + 3] * v4.w);
          uint16_t* at = reinterpret_cast<uint16_t*>(out + 128 * c) + size_t(i) * kDim;
          at[0] = uint16_t(a);
          at[kDim] = uint16_t(a >> 16);
          at[2 * kDim] = uint16_t(b);
          at[3 * kDim] = uint16_t(b >> 16);
        }
      } else if (o.slot >= 0) {
#pragma unroll
        for (int i = 0; i < kHPT; ++i) part[128 * c + size_t(i) * kDim] = x[i] * iv[i];
      }
    }
    tc_fence_before();  // before this warp's next arrival at a barrier the MMA thread waits on
  };

  uint32_t n = 0, live = 0;  // tiles, pieces with tiles so far
  Out pending = {-1, 0, -1, 0, 0};
#pragma unroll 1
  while (cur.unit >= 0) {
    const int t = cur.unit;
    const bool whole = cur.whole, any = cur.tiles > 0;
    const int slot = (t == first_unit) ? 2 * c_idx : 2 * c_idx + 1;
    const bool writable = whole || slot < ws.slots;  // split pieces need the workspace
    if (!writable && tid == 0) atomicOr(fault, QSFM_FAULT_METADATA);
    // Lane i of the warp keeps the running sum of P for head h0 + i over this
    // warp's 32 rows: each tile's P is folded in with a lane reduction once P
    // is published (one register instead of kHPT).
    float l_sum = 0.f;
    // The first tile takes the last unit's maxima (0 at first) as a guess: any reference is
    // right that leaves no t above 8 (P stays in range) and none of the first
    // rows' below -60 (P and its sum keep their precision; bf16 has the range
    // of fp32). Where the guess fails the vote sends the tile down the slow
    // path. `seen`: a tile with a valid row has set or confirmed the maxima. So on
    // which side P is rounded depends on the units before: a call repeats its bits,
    // a token in another batch may differ in its last ones.
    bool seen = false;
#pragma unroll 1
    for (int k = 0; k < cur.tiles; ++k, ++n) {
      const uint32_t par = n & 1;
      // After an abort the waits fall through at once; the warps keep running
      // the same named-barrier sequence so that none of them blocks.
      warp_wait_fast(sm, kBarFull + 0, par, fault);  // the tile's valid flags
      const bool v = sm.valid()[r] != 0;
      const int4 quadrants = *reinterpret_cast<const int4*>(sm.any());
      // The next piece, and its q as soon as this one's last score product has
      // completed. Not earlier: at the start the resolver is still at the first
      // piece's tiles, and the softmax of the first would wait for the last.
      Piece next = {-1, 0, 0, 0};
      if (k == cur.tiles - 1 && tid == 0) next = fetch_piece(handed ^ 1u);
      warp_wait_fast(sm, kBarSFull, par, fault);
      if (next.tiles > 0 && !*sm.abort_flag()) load_q(next.unit);
      tc_fence_after();
      float x[kHPT];
      tmem_load(s_addr, x);
      tmem_ld_wait_for(x);
      // Fast path: t = score * scale - m (log2 units), P = 2^t computed before
      // the vote; valid only if no t exceeds 8 anywhere in the tile.
      float tmax = -INFINITY, tmin = INFINITY;
#pragma unroll
      for (int i = 0; i < kHPT; i += 4) {
        const float4 m4 = *reinterpret_cast<const float4*>(m_used + h0 + i);
        const float t0 = v ? fmaf(x[i], qk_scale, -m4.x) : -INFINITY;
        const float t1 = v ? fmaf(x[i + 1], qk_scale, -m4.y) : -INFINITY;
        const float t2 = v ? fmaf(x[i + 2], qk_scale, -m4.z) : -INFINITY;
        const float t3 = v ? fmaf(x[i + 3], qk_scale, -m4.w) : -INFINITY;
        tmax = fmaxf(tmax, fmaxf(fmaxf(t0, t1), fmaxf(t2, t3)));
        if (!seen) tmin = fminf(tmin, fminf(fminf(t0, t1), fminf(t2, t3)));
        x[i] = ex2_approx(t0);
        x[i + 1] = ex2_approx(t1);
        x[i + 2] = ex2_approx(t2);
        x[i + 3] = ex2_approx(t3);
      }
      // also true against a maximum of -inf (t = inf)
      const bool move = named_sync_or(kBarSm, kSmThreads, tmax > kRescaleLog2 || (v && !seen && tmin < -kGuessLog2));
      float lscale = 1.f;  // 0 after a moved max: the running sums take alpha first
      if (move) {
        // Slow path: the scores again, the tile max per head over its 128
        // rows, the new running max, then O^T and the row sums rescaled.
        tmem_load(s_addr, x);
        tmem_ld_wait_for(x);
#pragma unroll
        for (int i = 0; i < kHPT; ++i) x[i] = v ? __fmul_rn(x[i], qk_scale) : -INFINITY;
        const float mx = reduce_lanes<true>(x);  // head h0 + lane, this quadrant's rows
        red[qd * 64 + h0 + lane] = mx;
        named_sync(kBarSm, kSmThreads);
        if (tid < 64) {
          const float mt = fmaxf(fmaxf(red[tid], red[64 + tid]), fmaxf(red[128 + tid], red[192 + tid]));
          const float mu = m_used[tid];
          float a = 1.f;
          if (!seen) {
            // Nothing is accumulated yet. Of scores that are all -inf the guess must not
            // stay: a later score far below it would be lost. Any other is far above this.
            m_used[tid] = mt > -INFINITY ? mt : -3e38f;
          } else if (mt > -INFINITY && (mu == -INFINITY || mt > mu + kRescaleLog2)) {
            a = (mu == -INFINITY) ? 0.f : exp2f(mu - mt);
            m_used[tid] = mt;
          }
          alpha[tid] = a;
        }
        named_sync(kBarSm, kSmThreads);
        if (seen) {
          // O^T at this thread's lane, its heads, every chunk. The PV products
          // of the earlier tiles have completed: S^T(n) was committed after
          // them.
#pragma unroll 1
          for (int c = 0; c < 4; ++c) {
            float o[kHPT];
            const uint32_t addr = tmem + o_column(live, c) + h0 + lane_base;
            tmem_load(addr, o);
            tmem_ld_wait_for(o);
#pragma unroll
            for (int i = 0; i < kHPT; ++i) o[i] *= alpha[h0 + i];
            tmem_store(addr, o);
          }
          tmem_st_wait();
        }
        tmem_load(s_addr, x);
        tmem_ld_wait_for(x);
#pragma unroll
        for (int i = 0; i < kHPT; ++i) {
          const float m = m_used[h0 + i];
          const float mz = m == -INFINITY ? 0.f : m;
          // the product rounded as for the maximum: of a huge score, what a fused
          // multiply-add keeps of the product's rounding would overflow 2^t
          x[i] = ex2_approx(v ? __fsub_rn(__fmul_rn(x[i], qk_scale), mz) : -INFINITY);
        }
        lscale = 0.f;
      }
      // P into the P buffer as [128 rows][64 heads] bf16 with the 128-B
      // swizzle (the MN-major B operand of PV): this thread's row, its
      // 16-byte units of 8 heads. bf16 because both operands of a product have one
      // type, and V~ in f16 would need its range followed. It costs accuracy: the
      // root-mean-square error of the output is 2.2e-3 of its own instead of the
      // 1.65e-3 of its rounding to bf16 alone.
#pragma unroll
      for (int vv = 0; vv < kHPT / 8; ++vv) {
        const uint32_t u = uint32_t((h0 >> 3) + vv);
        const uint4 pk = make_uint4(pack_bf16(x[8 * vv + 0], x[8 * vv + 1]), pack_bf16(x[8 * vv + 2], x[8 * vv + 3]),
                                    pack_bf16(x[8 * vv + 4], x[8 * vv + 5]), pack_bf16(x[8 * vv + 6], x[8 * vv + 7]));
        sts_v4(prow_addr + ((u ^ uint32_t(r & 7)) << 4), pk);
      }
      fence_proxy_async_smem();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(sm.bar(kBarPFull));
      {
        // running sums += this tile's P, folded over the warp's rows (after
        // P is published: off the PV path); a moved max rescales them first
        const float tile_sum = reduce_lanes<false>(x);
        if (lscale == 0.f) l_sum *= alpha[h0 + lane];
        l_sum += tile_sum;
      }
      seen = seen || (quadrants.x | quadrants.y | quadrants.z | quadrants.w) != 0;
      if (k == 0 && pending.unit >= 0) {
        write_out(pending);
        pending.unit = -1;
      }
    }
    // ---------------- the piece's sums, lse and 1 / den; the next piece
    if (any) {
      red[qd * 64 + h0 + lane] = l_sum;
    } else if (tid == 0) {
      const Piece next = fetch_piece(handed ^ 1u);
      if (next.tiles > 0 && !*sm.abort_flag()) load_q(next.unit);
    }
    // One barrier of all softmax warps. red, m_used and inv are used again behind
    // the next one (the first tile's vote, or a piece's without tiles); of the
    // two places of the handed piece, this one behind the next but one.
    const bool stop = named_sync_or(kBarSm, kSmThreads, *sm.abort_flag());  // the same for all
    handed ^= 1u;
    cur = sm.pieces()[Smem::kRing + handed];
    if (tid >= kSmThreads - 64 && writable) {
      const int h = tid - (kSmThreads - 64);
      const float lt = any ? (red[h] + red[64 + h]) + (red[128 + h] + red[192 + h]) : 0.f;
      const float mu = m_used[h];
      const bool none = lt == 0.f;  // no row (a sum of NaN is not none: it shows in the output and lse)
      const float lse2 = none ? -INFINITY : mu + log2f(lt);
      float den = lt;
      if (whole) {
        const float sink2 = sinks[unit_head0(p, t) + h];  // -inf without sinks
        if (!none) den += exp2f(sink2 - mu);
        if (p.return_lse) p.softmax_lse[size_t(t) * 64 + h] = lse2 * kLn2;
      } else {
        ws.lse[size_t(slot) * 64 + h] = lse2 * kLn2;
      }
      inv[64 * (live & 1) + h] = none ? 0.f : 1.f / den;
    }
    if (any) {
      pending = Out{t, whole, writable ? slot : -1, live, n - 1};
      ++live;
    } else if (writable) {  // no rows: zeros
      const uint4 z = make_uint4(0, 0, 0, 0);
      uint4* zeros = whole ? reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p.attn_out) + size_t(t) * 64 * kDim)
                           : reinterpret_cast<uint4*>(ws.out + size_t(slot) * 64 * kDim);
      for (int i = tid; i < 64 * kDim * (whole ? 2 : 4) / 16; i += kSmThreads) zeros[i] = z;
    }
    if (stop) return;
  }
  named_sync(kBarSm, kSmThreads);  // the last piece's inv
  if (pending.unit >= 0 && !*sm.abort_flag()) write_out(pending);
}

__global__ void __launch_bounds__(kThreads, 1)
    attention4_kernel(const qsfm_params p, const int T, const Workspace ws, int* fault,
                      const __grid_constant__ CUtensorMap qmap) {
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw_addr = smem_u32(smem_raw);
  Smem sm;
  sm.base = (raw_addr + 1023u) & ~1023u;
  sm.ptr = smem_raw + (sm.base - raw_addr);

  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
  if (warp == 0) warm_first_token(p, T, blockIdx.x, gridDim.x, tid);
  if (tid == 0) {
    mbar_init(sm.bar(kBarQFull), 1);
    for (int i = 0; i < 4; ++i) mbar_init(sm.bar(kBarFull + i), kPrWarps);
    for (int i = 0; i < 2; ++i) mbar_init(sm.bar(kBarFree + i), 1);
    mbar_init(sm.bar(kBarSFull), 1);
    mbar_init(sm.bar(kBarPFull), kSmWarps);
    mbar_init(sm.bar(kBarOFree), kSmWarps);
    for (int i = 0; i < Smem::kRing; ++i) {
      mbar_init(sm.bar(Smem::kBarRowsFull + i), 1);
      mbar_init(sm.bar(Smem::kBarRowsEmpty + i), kPrWarps + 1);
      mbar_init(sm.bar(Smem::kBarPieceFull + i), 1);
      mbar_init(sm.bar(Smem::kBarPieceEmpty + i), 1);
    }
    mbar_init(sm.bar(kBarDrain), 1);
    *sm.abort_flag() = 0;
    fence_mbar_init();
  }
  __syncthreads();
  grid_dependency_wait();    // the plan (and every input) is written by now
  grid_launch_dependents();  // the combine kernel may take SMs as CTAs finish
  const int* meta = p.metadata;
  const int c = blockIdx.x;
  // read at once: c is below QSFM_MAX_CTAS, so its range lies in the buffer whatever the header says
  const int magic = meta[0], G = meta[1], planned = meta[2];
  const Range rg{meta[kMetaHeader + 2 * c], meta[kMetaHeader + 2 * c + 1],
                 meta[kMetaHeader + 2 * c + 2], meta[kMetaHeader + 2 * c + 3]};
  if (magic != kMetaMagic || planned != T || G < 0 || G > int(gridDim.x) || G > QSFM_MAX_CTAS) {
    if (tid == 0 && blockIdx.x == 0) atomicOr(fault, QSFM_FAULT_METADATA);
    return;
  }
  if (c >= G) return;
  if (rg.t0 < 0 || rg.t1 > T || rg.t0 > rg.t1 || rg.k0 < 0 || rg.k1 < 0 ||
      (rg.t1 == T && rg.k1 != 0)) {
    if (tid == 0) atomicOr(fault, QSFM_FAULT_METADATA);
    return;
  }
  if (rg.t0 == rg.t1 && rg.k0 == rg.k1) return;

  // The resolver does not wait for tensor memory: it reads its first lengths.
  if (warp == kMmaWarp) tmem_alloc(sm.tmem_slot(), kTmemCols);
  tc_fence_before();
  if (warp != kResolverWarp) named_sync(kBarSetup, kThreads - 32);
  tc_fence_after();
  const uint32_t tmem = *sm.tmem_slot();

  if (warp < kSmWarps) {
    softmax_role(p, sm, rg.t0, tmem, ws, c, &qmap, fault);
  } else if (warp < kMmaWarp) {
    more_registers<kPrRegs>();
    producer_role(p, sm, fault);
  } else {
    fewer_registers<kLastRegs>();
    if (warp == kMmaWarp) {
      mma_role(sm, tmem, fault);
      // every MMA issued above has completed before tensor memory is freed
      // (after an abort some may still be in flight)
      commit_elected(sm.bar(kBarDrain));
      warp_wait_fast(sm, kBarDrain, 0, fault);
    } else if (warp == kResolverWarp) {
      resolver_role(p, sm, rg, T, fault);
    }
  }

  // After an abort a copy of q may still be on its way into this CTA's shared
  // memory: give it a millisecond, far more than it takes.
  if (tid == 0 && *sm.abort_flag())
    for (int i = 0; i < 1000; ++i) __nanosleep(1000);

  // Roles run on single lanes (the MMA issue): each warp's lanes meet before
  // the barrier (a barrier reached by part of a warp counts the whole warp).
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (warp == kMmaWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
}

}  // namespace

cudaError_t launch_attention4(const qsfm_params& p, int num_tokens, int num_ctas, const Workspace& ws, int* fault,
                              cudaStream_t s) {
  // The register split takes from what the launch gives: with fewer registers per
  // thread than it counts on, the producers would wait for theirs forever.
  static std::atomic<bool> enough{false};
  if (!enough.load(std::memory_order_relaxed)) {
    cudaFuncAttributes a;
    const cudaError_t q = cudaFuncGetAttributes(&a, attention4_kernel);
    if (q != cudaSuccess) return q;
    if (a.numRegs < kLaunchRegs) return cudaErrorInvalidConfiguration;
    enough.store(true, std::memory_order_relaxed);
  }
  cudaError_t e = cudaFuncSetAttribute(attention4_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemAlloc);
  if (e != cudaSuccess) return e;
  CUtensorMap qmap;
  e = make_q_map(p.q, num_tokens, &qmap);
  if (e != cudaSuccess) return e;
  return launch_after_predecessor(attention4_kernel, dim3(num_ctas), dim3(kThreads), kSmemAlloc, s, p, num_tokens,
                                  ws, fault, qmap);
}

}  // namespace qsfm
