// int8 products over dense rows or expert windows on the 5th-generation
// tensor cores (tcgen05 kind::i8): exact int32 sums, scaled in fp32 and rounded
// once, y[r, n] = (sum_k x[r, k] w[n, k]) ws[n] xs[r], or silu(gate) * up of two
// such products.
//
// The weights are the MMA's A operand (M = 128 channels a CTA) and the rows its
// N operand, so a few rows cost few columns. A unit of work is (expert, channel
// tile, chunk of up to kRows rows, the expert's chunks being alike); a persistent grid takes the units in a
// fixed order, which every warp derives by itself from the windows. With an up
// projection a CTA's 128 A rows are 64 gate and 64 up channels, and the
// epilogue brings the two halves of tensor memory together through shared
// memory: the main loop is the same as without.
//
// Per CTA (320 threads): warp 0 streams K slabs of 128 bytes into a ring of
// stages with TMA, warp 1 issues the MMAs into tensor memory, warps
// 2-9 read finished ones back, scale and store. Four forms:
//   kOne    chunks of 64 rows, one CTA: a decode batch reads every weight once,
//           and the many small stages keep the loads in flight that HBM needs
//   kSplit  the same with a unit's K slabs split over the CTAs of a cluster,
//           where there are fewer units than SMs: each CTA writes its int32
//           sums of a row into the shared memory of the CTA that owns the row
//           (row mod cluster size), which adds and stores them (integers: the
//           order changes nothing)
//   kPair   chunks of 256 rows, or up to 288 where that saves one, a CTA pair
//           (M = 256 over two SMs, each holding half of the rows): for many rows
//           an expert, where the tensor cores and the L2's delivery of operands
//           bound it. The 512 columns of tensor memory are a ring: a unit takes
//           as many as it has rows, and the next one starts when enough of the
//           last but one's are read, 32 at a time.
//   kPair128  the same with chunks of up to 128 rows, whose eight smaller stages
//           keep more loads in flight
// Measured from a cold start: 8192 x 4096 x 7168 141 us, 3.4 POP/s (kPair, 87 % of
// the tensor pipe; 173 us at the power cap); gate/up of 32 experts, 2 x 2048 x
// 7168, with 128 rows 148 us = 6.2 TB/s (kOne; 31.45 of the 32 experts have rows on
// average), with 8192 rows 205 us (kPair, 5.1 TB/s and 2.35 POP/s at once).
// Every wait is bounded: on expiry the kernel latches MOE_ERR_TIMEOUT, drains
// its copies and MMAs, frees tensor memory and exits.
#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstring>
#include <type_traits>

#include "ffn_common.cuh"
#include "gemm_i8.cuh"

namespace moe {
namespace {

using ffn::kABytes;
using ffn::kMaxDynSmem;
using ffn::kSlab;
using ffn::wait_bar;

constexpr int kThreads = 320;      // warps: 0 TMA, 1 MMA, 2-9 epilogue (two sets of four)
constexpr int kEpiThreads = 256;
constexpr int kMaxExperts = 1024;
constexpr int kBand = 8;           // chunks that share each channel tile in turn (unit order)

enum : int { kOne, kSplit, kPair, kPair128 };

template <int kForm, bool kUp>
struct Form {
  static constexpr bool kPaired = kForm >= kPair;
  static constexpr int kG = kPaired ? 2 : 1;                  // CTAs of one MMA
  static constexpr int kFull = kForm == kPair ? 256 : kPaired ? 128 : 64;   // rows of a chunk: MMA columns
  static constexpr int kRows = kForm == kPair ? 288 : kFull;  // and of the largest
  static constexpr int kBRows = kRows / kG;                   // of them in this CTA's shared memory
  static constexpr int kCh = kUp ? 64 : 128;                  // channels a CTA
  static constexpr int kStage = kABytes + kBRows * kSlab;
  // kSplit: [CTA][rows owned][128 A rows] int32, the sums of this CTA's rows; else with up
  // [set][gate, up][8 rows][64 channels] int32
  static constexpr int kXchg = kForm == kSplit ? kRows * 128 * 4 : kUp ? 2 * 2 * 8 * 64 * 4 : 0;
  static constexpr int kXs = 2 * kRows * 4;                   // row scales, two units
  static constexpr int kTab = (kMaxExperts + 1) * 4 + 12;
  static constexpr int kCtl = 512;
  static constexpr int kStages = (kMaxDynSmem - 1024 - kXchg - kXs - kTab - kCtl) / kStage;
  static constexpr int kOffXchg = kStages * kStage;
  static constexpr int kOffXs = kOffXchg + kXchg;
  static constexpr int kOffTab = kOffXs + kXs;
  static constexpr int kOffCtl = (kOffTab + kTab + 15) / 16 * 16;
  static constexpr int kSmem = kOffCtl + kCtl + 1024;         // and alignment slack
  static constexpr uint32_t kTmemCols = 2 * kFull;            // pairs: the ring; else two accumulators
  static constexpr int kGran = 32;                            // columns given back at a time
  static_assert(kSmem <= kMaxDynSmem && (2 * kStages + 7 + (int)kTmemCols / kGran) * 8 <= kCtl - 32, "shared memory");
  static_assert(!kPaired || kStages >= 6, "stages of a pair");
};

struct Params {
  CUtensorMap tm_w, tm_wu;   // [experts * N, K], boxes of 128 (64 with up) channels
  CUtensorMap tm_x[4];       // [M, K], boxes of 16, 32, 64 and 128 rows
  const float* xs;
  const float* ws;
  const float* wus;
  RowWindows win;
  void* y;
  Header* hdr;
  int64_t M, N;
  int nk;        // K slabs
  int tiles;     // channel tiles of one expert
  int wide;      // kPair: chunks of more than kFull rows may be taken
};

// One unit: chunk `chunk` of expert e's rows, channel tile `tile`.
struct Unit {
  int e, tile, rows;
  int64_t row;   // first row
};

template <int kForm, bool kUp, typename O>
__global__ void __launch_bounds__(kThreads, 1) gemm_i8_kernel(const __grid_constant__ Params p) {
  using F = Form<kForm, kUp>;
  constexpr int kG = F::kG;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
  uint8_t* ctl = smem + F::kOffCtl;
  uint64_t* full = reinterpret_cast<uint64_t*>(ctl);      // [kStages] CTA 0: all halves landed
  uint64_t* empty = full + F::kStages;                    // [kStages] each CTA: the stage's MMAs are done
  uint64_t* acc_full = empty + F::kStages;                // [2] each CTA: an accumulator is complete
  uint64_t* acc_empty = acc_full + 2;                     // [2] CTA 0: all epilogue warps have read it
  uint64_t* drain = acc_empty + 2;
  uint64_t* part_full = drain + 1;                        // kSplit: all CTAs' sums of this one's rows are here
  uint64_t* part_free = part_full + 1;                    // kSplit: all CTAs have read what they got
  uint64_t* col_free = part_free + 1;                     // pairs, CTA 0: both CTAs have read these 32 columns
  volatile int* abort_flag = reinterpret_cast<volatile int*>(ctl + F::kCtl - 32);
  volatile int* epi_ok = abort_flag + 1;                  // [2]
  volatile int* part_ok = epi_ok + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(ctl + F::kCtl - 16);
  int* tab = reinterpret_cast<int*>(smem + F::kOffTab);   // [experts + 1] first chunk of each expert

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = F::kPaired ? ptx::cluster_ctarank() : 0u;   // CTA of the MMA
  const uint32_t part = kForm == kSplit ? ptx::cluster_ctarank() : 0u;  // share of K
  const uint32_t parts = kForm == kSplit ? ptx::cluster_nctarank() : 1u;
  const int team = kForm == kSplit ? (int)parts : kG;                   // CTAs of a worker
  const int worker = blockIdx.x / team, workers = gridDim.x / team;
  const int k_first = (int)(part * (uint32_t)p.nk / parts), k_end = (int)((part + 1) * (uint32_t)p.nk / parts);
  const int E = p.win.experts;

  if (threadIdx.x == 0) {
    for (int s = 0; s < F::kStages; ++s) {
      ptx::mbar_init(full + s, 1);
      ptx::mbar_init(empty + s, 1);
    }
    for (int s = 0; s < 2; ++s) {
      ptx::mbar_init(acc_full + s, 1);
      ptx::mbar_init(acc_empty + s, 8 * kG);
    }
    ptx::mbar_init(drain, 1);
    ptx::mbar_init(part_full, 8 * parts);
    ptx::mbar_init(part_free, 8 * parts);
    if constexpr (F::kPaired)
      for (int g = 0; g < (int)F::kTmemCols / F::kGran; ++g) ptx::mbar_init(col_free + g, 8);   // a set's warps, two CTAs
    *abort_flag = 0;
    ptx::fence_mbar_init();
  }
  if (warp == 1) {
    if constexpr (kG == 2) {
      ptx::tmem_alloc_pair(tmem_slot, F::kTmemCols);
      ptx::tmem_relinquish_pair();
    } else {
      ptx::tmem_alloc(tmem_slot, F::kTmemCols);
      ptx::tmem_relinquish();
    }
  }
  // MMA columns for that many rows
  auto columns = [](int rows) { return (rows + 16 * kG - 1) / (16 * kG) * (16 * kG); };
  // Chunks of a window. A unit's time goes like its columns + 72 (measured, per
  // channel tile of K = 7168: 160 columns 20 us, 256 29 us), so that chunks of
  // more than kFull rows are taken where that saves 3 %: 270 rows are one chunk
  // of 288 columns, not 160 and 128.
  auto chunks = [&](int rows) {
    const int c = (rows + F::kFull - 1) / F::kFull, d = (rows + F::kRows - 1) / F::kRows;
    if (kForm != kPair || !p.wide || d >= c) return c;
    auto cost = [&](int n) { return (int64_t)n * (72 + columns((rows + n - 1) / n)); };
    return cost(d) * 33 < cost(c) * 32 ? d : c;
  };
  if (warp == 2)   // first chunk of every expert
    window_prefix(p.win, p.M, (p.M + F::kFull - 1) / F::kFull + E, chunks, tab);
  ptx::tc_fence_before();
  if constexpr (kForm != kOne) ptx::cluster_sync();   // every CTA's barriers and tensor memory exist
  else __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const int units = tab[E] * p.tiles;   // below 2^31 (checked by the ABI)

  auto remote = [&](const void* q, uint32_t r) { return ptx::mapa_shared(ptx::smem_u32(q), r); };

  // Unit u. Within an expert: bands of kBand chunks, in a band channel tile by
  // channel tile, so that the workers of one moment share few rows and few
  // channels in L2.
  auto unit = [&](int u) -> Unit {
    const uint32_t nt = (uint32_t)p.tiles;
    int lo = 0, hi = E - 1;   // the last expert whose first unit is <= u (empty ones never are)
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if ((uint32_t)tab[mid] * nt <= (uint32_t)u) lo = mid;
      else hi = mid - 1;
    }
    const int nc = tab[lo + 1] - tab[lo];
    const uint32_t v = (uint32_t)u - (uint32_t)tab[lo] * nt;
    const uint32_t band = v / (kBand * nt), w = v - band * kBand * nt;
    const int left = nc - (int)band * kBand;
    const uint32_t bh = (uint32_t)(left < kBand ? left : kBand);
    Unit r;
    r.e = lo;
    r.tile = (int)(w / bh);
    const int chunk = (int)(band * kBand + w - (uint32_t)r.tile * bh);
    int64_t row0;
    // an expert's chunks are of one size, so that the units that follow one
    // another cost alike
    const int rows = window_rows(p.win, lo, p.M, &row0);
    const int each = columns((int)(((uint32_t)rows + (uint32_t)nc - 1u) / (uint32_t)nc));
    const int left_rows = rows - chunk * each;
    r.rows = left_rows < each ? left_rows : each;
    r.row = row0 + (int64_t)chunk * each;
    return r;
  };
  // Pairs: of n columns from `at` on, those of the first MMA: up to the ring's
  // end, and 256 at most. A second one takes the rest (288 or fewer are left
  // with 256 or fewer).
  auto first_columns = [](int at, int n) {
    if (!F::kPaired) return n;
    const int to_end = (int)F::kTmemCols - at;
    return n < to_end ? (n < 256 ? n : 256) : (to_end < 256 ? to_end : 256);
  };

  if (warp == 0) {
    // ---------------------------------------------------------------- TMA producer (both CTAs)
    if (lane == 0) {
      ptx::prefetch_tmap(&p.tm_w);
      for (int b = 0; b < 4; ++b) ptx::prefetch_tmap(&p.tm_x[b]);
      if (kUp) ptx::prefetch_tmap(&p.tm_wu);
    }
    uint32_t stage = 0, phase = 0;
    uint32_t armed = 0, armed_parity = 0;
    const uint64_t pol = ptx::policy_evict_first();   // kOne, kSplit: weights are read once
    bool ok = true;
    int at = 0;   // pairs: the unit's first column
    for (int u = worker; ok && u < units; u += workers) {
      const Unit j = unit(u);
      const int cols = columns(j.rows), c1 = first_columns(at, cols);
      at = (at + cols) % (int)F::kTmemCols;
      const int n = cols / kG;                                  // rows this CTA loads
      const int n1 = c1 / kG, n2 = n - n1;                      // its halves of the two MMAs' columns
      const int wrow = (int)(j.e * p.N + (int64_t)j.tile * (kG * F::kCh) + rank * F::kCh);
      const int xrow = (int)(j.row + rank * n1), xrow2 = (int)(j.row + c1 + rank * n2);
      for (int k = k_first; k < k_end; ++k) {
        int good = 1;
        if (lane == 0) good = wait_bar(empty + stage, phase ^ 1u, abort_flag, p.hdr, 0x48000000u | stage);
        if (!__shfl_sync(0xffffffffu, good, 0)) { ok = false; break; }
        __syncwarp();
        uint8_t* st = smem + stage * F::kStage;
        if (ptx::elect_one()) {
          if (rank == 0) ptx::mbar_arrive_expect_tx(full + stage, (uint32_t)(kG * (kABytes + n * kSlab)));
          const int kx = k * kSlab;
          uint8_t* sx = st + kABytes;
          // rows in the fewest boxes, each map at a fixed parameter address
          auto rows = [&](int m, int to, int from, auto load) {
            int r = 0;
            if (F::kBRows >= 128 && m & 128) { load(&p.tm_x[3], to, from); r = 128; }
            if (m & 64) { load(&p.tm_x[2], to + r, from + r); r += 64; }
            if (m & 32) { load(&p.tm_x[1], to + r, from + r); r += 32; }
            if (m & 16) load(&p.tm_x[0], to + r, from + r);
          };
          if constexpr (kG == 2) {
            const uint32_t fb = remote(full + stage, 0);
            ptx::tma_load_2d_pair(st, &p.tm_w, fb, kx, wrow);
            if (kUp) ptx::tma_load_2d_pair(st + 64 * kSlab, &p.tm_wu, fb, kx, wrow);
            auto load = [&](const CUtensorMap* m, int to, int from) {
              ptx::tma_load_2d_pair(sx + to * kSlab, m, fb, kx, from);
            };
            rows(n1, 0, xrow, load);
            if (n2) rows(n2, n1, xrow2, load);
          } else {
            uint64_t* fb = full + stage;
            ptx::tma_load_2d_hint(st, &p.tm_w, fb, kx, wrow, pol);
            if (kUp) ptx::tma_load_2d_hint(st + 64 * kSlab, &p.tm_wu, fb, kx, wrow, pol);
            rows(n, 0, xrow, [&](const CUtensorMap* m, int to, int from) {
              ptx::tma_load_2d(sx + to * kSlab, m, fb, kx, from);
            });
          }
        }
        __syncwarp();
        armed |= 1u << stage;
        armed_parity = (armed_parity & ~(1u << stage)) | (phase << stage);
        if (++stage == (uint32_t)F::kStages) { stage = 0; phase ^= 1u; }
      }
    }
    // drain (CTA 0): every load counted on its barriers has landed
    if (rank == 0 && lane == 0) {
      for (int s = 0; s < F::kStages; ++s) {
        if (!((armed >> s) & 1u)) continue;
        const unsigned long long t0 = globaltimer();
        while (!ptx::mbar_try_wait(full + s, (armed_parity >> s) & 1u))
          if (globaltimer() - t0 > kWaitBudgetNs) break;
      }
    }
    __syncwarp();
  } else if (warp == 1) {
    // ---------------------------------------------------------------- MMA issuer (CTA 0)
    if (rank == 0) {
      uint32_t stage = 0, phase = 0, i = 0;
      uint32_t uses = 0;   // pairs: bit g: parity of the uses of columns 32 g ..
      int at = 0;
      bool ok = true;
      for (int u = worker; ok && u < units; u += workers, ++i) {
        const uint32_t slot = i & 1u, use = (i >> 1) & 1u;
        const int cols = columns(unit(u).rows), c1 = first_columns(at, cols);
        int good = 1;
        if (lane == 0) good = wait_bar(acc_empty + slot, use ^ 1u, abort_flag, p.hdr, 0x58000000u | slot);
        if constexpr (F::kPaired) {   // and the unit's columns are free, lane by lane
          constexpr int kGrans = (int)F::kTmemCols / F::kGran;
          const int g = (at / F::kGran + lane) % kGrans;
          const bool mine = lane < cols / F::kGran;
          if (mine && good) good = wait_bar(col_free + g, ((uses >> g) & 1u) ^ 1u, abort_flag, p.hdr, 0x59000000u);
          uses ^= __reduce_or_sync(0xffffffffu, mine ? 1u << g : 0u);
        }
        if (!__all_sync(0xffffffffu, good)) break;
        ptx::tc_fence_after();
        const uint32_t d = tmem + (F::kPaired ? (uint32_t)at : slot * F::kRows);
        const uint32_t d2 = tmem + (uint32_t)((at + c1) % (int)F::kTmemCols);   // pairs: of the second MMA
        const uint32_t idesc = ptx::idesc_i8(128 * kG, c1), idesc2 = ptx::idesc_i8(128 * kG, cols - c1);
        const uint64_t b2_off = (uint64_t)(c1 / kG * kSlab) >> 4;
        const bool two = c1 < cols;
        at = (at + cols) % (int)F::kTmemCols;
        for (int k = k_first; k < k_end; ++k) {
          if (lane == 0) good = wait_bar(full + stage, phase, abort_flag, p.hdr, 0x68000000u | stage);
          if (!__shfl_sync(0xffffffffu, good, 0)) { ok = false; break; }
          ptx::tc_fence_after();
          uint8_t* st = smem + stage * F::kStage;
          const uint64_t a = ptx::desc_kmajor_sw128(st), b = ptx::desc_kmajor_sw128(st + kABytes);
          if (ptx::elect_one()) {
#pragma unroll
            for (int kk = 0; kk < 4; ++kk) {   // 32 bytes of K per MMA
              if constexpr (kG == 2) ptx::mma_i8_pair(d, a + 2 * kk, b + 2 * kk, idesc, k > k_first || kk ? 1u : 0u);
              else ptx::mma_i8(d, a + 2 * kk, b + 2 * kk, idesc, k > k_first || kk ? 1u : 0u);
            }
            if (F::kPaired && two) {
#pragma unroll
              for (int kk = 0; kk < 4; ++kk)
                ptx::mma_i8_pair(d2, a + 2 * kk, b + b2_off + 2 * kk, idesc2, k > k_first || kk ? 1u : 0u);
            }
            if constexpr (kG == 2) {
              ptx::mma_commit_pair(remote(empty + stage, 0));
              ptx::mma_commit_pair(remote(empty + stage, 1));
            } else {
              ptx::mma_commit(empty + stage);
            }
          }
          __syncwarp();
          if (++stage == (uint32_t)F::kStages) { stage = 0; phase ^= 1u; }
        }
        if (!ok) break;
        if (ptx::elect_one()) {
          if constexpr (kG == 2) {
            ptx::mma_commit_pair(remote(acc_full + slot, 0));
            ptx::mma_commit_pair(remote(acc_full + slot, 1));
          } else {
            ptx::mma_commit(acc_full + slot);
          }
        }
        __syncwarp();
      }
      if (ptx::elect_one()) {   // every MMA issued is complete
        if constexpr (kG == 2) ptx::mma_commit_pair(remote(drain, 0));
        else ptx::mma_commit(drain);
        const unsigned long long t0 = globaltimer();
        while (!ptx::mbar_try_wait(drain, 0))
          if (globaltimer() - t0 > kWaitBudgetNs) break;
      }
      __syncwarp();
    }
  } else {
    // ---------------------------------------------------------------- epilogue
    // Warp w reads tensor-memory lanes 32 (w % 4) .. + 31 (A rows); set s takes
    // the 32-column batches s, s + 2, ...
    const int q = warp & 3, et = threadIdx.x - 64, set = et >> 7;
    const int arow = q * 32 + lane;
    const int ch = kUp ? arow & 63 : arow;           // channel of the CTA's tile
    int* xg = reinterpret_cast<int*>(smem + F::kOffXchg) + set * 2 * 8 * 64;   // [8][64]
    int* xu = xg + 8 * 64;
    float* xs_all = reinterpret_cast<float*>(smem + F::kOffXs);
    // kSplit: this CTA's sums to the owners of their rows, then its own rows
    auto split_epilogue = [&](const Unit& j, uint32_t slot, uint32_t use, uint32_t turn) -> bool {
      int* sums = reinterpret_cast<int*>(smem + F::kOffXchg);
      const int shift = __ffs(parts) - 1, owned = F::kRows >> shift;   // parts is a power of two
      // a thread's channel when it stores, fetched while the sums are made
      const int n = et % F::kCh;
      const int64_t nn = (int64_t)j.tile * F::kCh + n;
      const bool real = nn < p.N;
      const float sw = real ? __ldg(p.ws + j.e * p.N + nn) : 0.f;
      const float su = kUp && real ? __ldg(p.wus + j.e * p.N + nn) : 0.f;
      float* xs = xs_all + slot * F::kRows;
      if (et < j.rows) xs[et] = __ldg(p.xs + j.row + et);
      if (et == 0)
        epi_ok[slot] = wait_bar(acc_full + slot, use, abort_flag, p.hdr, 0x78000000u | slot) &&
                       wait_bar<true>(part_free, turn ^ 1u, abort_flag, p.hdr, 0x79000000u);
      ptx::named_barrier(1, kEpiThreads);
      if (!epi_ok[slot]) return false;
      while (!ptx::mbar_try_wait(acc_full + slot, use)) {}   // both completed: return at once
      while (!ptx::mbar_try_wait_cluster(part_free, turn ^ 1u)) {}
      ptx::tc_fence_after();
      for (int c0 = 32 * set; c0 < j.rows; c0 += 64) {
        uint32_t v[32];
        ptx::tmem_ld_x32(tmem + slot * F::kRows + ((uint32_t)(q * 32) << 16) + c0, v);
        ptx::tmem_wait_ld();
        int* mine = sums + (part * owned + (c0 >> shift)) * 128 + arow;
        auto push = [&](auto count) {   // column c to owner c mod kParts
          constexpr int kParts = decltype(count)::value;
          uint32_t at[kParts];
#pragma unroll
          for (int r = 0; r < kParts; ++r) at[r] = remote(mine, r);
#pragma unroll
          for (int c = 0; c < 32; ++c)
            if (c0 + c < j.rows) ptx::st_cluster_u32(at[c % kParts] + c / kParts * 512, v[c]);
        };
        if (parts == 2) push(std::integral_constant<int, 2>());
        else push(std::integral_constant<int, 4>());
      }
      ptx::tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        ptx::mbar_arrive(acc_empty + slot);
        for (uint32_t r = 0; r < parts; ++r) ptx::mbar_arrive_cluster(remote(part_full, r));
      }
      if (et == 0) *part_ok = wait_bar<true>(part_full, turn, abort_flag, p.hdr, 0x7a000000u);
      ptx::named_barrier(1, kEpiThreads);
      if (!*part_ok) return false;
      while (!ptx::mbar_try_wait_cluster(part_full, turn)) {}   // completed: returns at once
      if (real) {
        for (int o = et / F::kCh; (o << shift) + (int)part < j.rows; o += kEpiThreads / F::kCh) {
          const int c = (o << shift) + (int)part;
          int a = 0, b = 0;
          for (uint32_t r = 0; r < parts; ++r) {
            a += sums[(r * owned + o) * 128 + n];
            if (kUp) b += sums[(r * owned + o) * 128 + 64 + n];
          }
          float f = (float)a * sw * xs[c];
          if (kUp) f = i8::swiglu<O>(f, (float)b * su * xs[c]);
          i8::put(reinterpret_cast<O*>(p.y) + (j.row + c) * p.N + nn, f);
        }
      }
      __syncwarp();
      if (lane == 0)
        for (uint32_t r = 0; r < parts; ++r) ptx::mbar_arrive_cluster(remote(part_free, r));
      return true;
    };
    uint32_t i = 0;
    int at = 0;   // pairs: the unit's first column
    for (int u = worker; u < units; u += workers, ++i) {
      const Unit j = unit(u);
      const uint32_t slot = i & 1u, use = (i >> 1) & 1u;
      if constexpr (kForm == kSplit) {
        if (!split_epilogue(j, slot, use, i & 1u)) break;
        continue;
      }
      float* xs = xs_all + slot * F::kRows;
      const int64_t n0 = (int64_t)j.tile * (kG * F::kCh) + rank * F::kCh + ch;
      const bool real = n0 < p.N;
      const float sw = real ? __ldg(p.ws + j.e * p.N + n0) : 0.f;
      const float su = kUp && real ? __ldg(p.wus + j.e * p.N + n0) : 0.f;
      for (int r = et; r < j.rows; r += kEpiThreads) xs[r] = __ldg(p.xs + j.row + r);
      // one thread waits and tells the others, so that all leave together
      if (et == 0) epi_ok[slot] = wait_bar(acc_full + slot, use, abort_flag, p.hdr, 0x78000000u | slot);
      ptx::named_barrier(1, kEpiThreads);
      if (!epi_ok[slot]) break;
      while (!ptx::mbar_try_wait(acc_full + slot, use)) {}   // completed: returns at once
      ptx::tc_fence_after();
      const uint32_t lanes = tmem + ((uint32_t)(q * 32) << 16);
      const int d = F::kPaired ? at : (int)slot * F::kRows;
      at = (at + columns(j.rows)) % (int)F::kTmemCols;
      const int64_t tile0 = n0 - ch;   // the CTA's first channel
      // bf16: two lanes exchange half of their rows, so that each stores two
      // neighbouring channels at once
      const bool pairs = sizeof(O) == 2 && (p.N & 1) == 0 && tile0 + F::kCh <= p.N;
      O* y = reinterpret_cast<O*>(p.y) + j.row * p.N + n0;
      // rows c .. c + 15 of this thread's channel
      auto store16 = [&](int c, const float (&f)[16]) {
        if (pairs && c + 16 <= j.rows) {
          const bool odd = lane & 1;
          O* q = y + (int64_t)(c + (odd ? 1 : 0)) * p.N - (odd ? 1 : 0);
#pragma unroll
          for (int i = 0; i < 16; i += 2) {
            const float got = __shfl_xor_sync(0xffffffffu, odd ? f[i] : f[i + 1], 1);
            const __nv_bfloat162 two = __floats2bfloat162_rn(odd ? got : f[i], odd ? f[i + 1] : got);
            *reinterpret_cast<__nv_bfloat162*>(q) = two;
            q += 2 * p.N;
          }
        } else if (real) {
          O* q = y + (int64_t)c * p.N;
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            if (c + i < j.rows) i8::put(q, f[i]);
            q += p.N;
          }
        }
      };
      for (int c0 = 32 * set; c0 < j.rows; c0 += 64) {
        uint32_t v[32];
        const int col = F::kPaired ? (d + c0) % (int)F::kTmemCols : d + c0;
        ptx::tmem_ld_x32(lanes + (uint32_t)col, v);
        ptx::tmem_wait_ld();
        if constexpr (F::kPaired) {   // the columns are in registers: give them back
          ptx::tc_fence_before();
          __syncwarp();
          if (lane == 0) {
            if (rank == 0) ptx::mbar_arrive(col_free + col / F::kGran);
            else ptx::mbar_arrive_remote(remote(col_free + col / F::kGran, 0));
          }
        }
        float f[16];
        if constexpr (!kUp) {
#pragma unroll
          for (int h = 0; h < 32; h += 16) {
            if (c0 + h >= j.rows) break;
#pragma unroll
            for (int c = 0; c < 16; c += 4) {
              const float4 s = *reinterpret_cast<const float4*>(xs + c0 + h + c);
              f[c] = (float)(int)v[h + c] * sw * s.x;
              f[c + 1] = (float)(int)v[h + c + 1] * sw * s.y;
              f[c + 2] = (float)(int)v[h + c + 2] * sw * s.z;
              f[c + 3] = (float)(int)v[h + c + 3] * sw * s.w;
            }
            store16(c0 + h, f);
          }
        } else {
          // gate warps finish the batch's first 16 columns, up warps the last; eight
          // at a time change hands
          const bool gate = q < 2;
          const int first = c0 + (gate ? 0 : 16);
#pragma unroll
          for (int h = 0; h < 16; h += 8) {
#pragma unroll
            for (int c = 0; c < 8; ++c) {
              if (gate) xg[c * 64 + ch] = (int)v[16 + h + c];
              else xu[c * 64 + ch] = (int)v[h + c];
            }
            ptx::named_barrier(2 + set, 128);
            if (first + h < j.rows) {
              const int* other = gate ? xu : xg;
              float g[8], u[8];
#pragma unroll
              for (int c = 0; c < 8; c += 4) {
                const float4 s4 = *reinterpret_cast<const float4*>(xs + first + h + c);
                const float s[4] = {s4.x, s4.y, s4.z, s4.w};
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                  const int own = (int)(gate ? v[h + c + i] : v[16 + h + c + i]), far = other[(c + i) * 64 + ch];
                  g[c + i] = (float)(gate ? own : far) * sw * s[i];
                  u[c + i] = (float)(gate ? far : own) * su * s[i];
                }
              }
              i8::swiglu<O>(g, u, f + h);
            }
            ptx::named_barrier(2 + set, 128);
          }
          if (first < j.rows) store16(first, f);
        }
      }
      ptx::tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        if (rank == 0) ptx::mbar_arrive(acc_empty + slot);
        else ptx::mbar_arrive_remote(remote(acc_empty + slot, 0));
      }
    }
  }
  // every role is done in every CTA before tensor memory is freed and one exits
  ptx::tc_fence_before();
  if constexpr (kForm != kOne) ptx::cluster_sync();
  else __syncthreads();
  if (warp == 1) {
    ptx::tc_fence_after();
    if constexpr (kG == 2) ptx::tmem_dealloc_pair(tmem, F::kTmemCols);
    else ptx::tmem_dealloc(tmem, F::kTmemCols);
  }
}

// ---- host side ------------------------------------------------------------

// team: CTAs of a worker (the cluster), 1, 2 or 4
template <int kForm, bool kUp, typename O>
cudaError_t launch(const GemmI8Args& a, int team, bool wide) {
  using F = Form<kForm, kUp>;
  constexpr int kMaxDevices = 64;
  static std::atomic<bool> prepared[kMaxDevices];   // the kernel's shared memory is allowed on this device
  int dev = 0;
  cudaError_t err = cudaGetDevice(&dev);
  if (err != cudaSuccess) return err;
  if (dev < 0 || dev >= kMaxDevices) return cudaErrorInvalidDevice;
  if (!prepared[dev].load(std::memory_order_acquire)) {
    if ((err = cudaFuncSetAttribute(gemm_i8_kernel<kForm, kUp, O>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                    F::kSmem)) != cudaSuccess)
      return err;
    prepared[dev].store(true, std::memory_order_release);
  }

  Params p;
  memset(&p, 0, sizeof(p));
  const int64_t N = a.d.N, K = a.d.K, E = a.d.experts;
  if (!ffn::make_tmap(&p.tm_w, a.w, ffn::kElU8, K, E * N, kSlab, F::kCh) ||
      (kUp && !ffn::make_tmap(&p.tm_wu, a.wu, ffn::kElU8, K, E * N, kSlab, F::kCh)))
    return cudaErrorInvalidValue;
  for (int b = 0; b < 4; ++b)
    if (!ffn::make_tmap(&p.tm_x[b], a.x, ffn::kElU8, K, a.d.M, kSlab, 16 << b)) return cudaErrorInvalidValue;
  p.xs = a.xs;
  p.ws = a.ws;
  p.wus = a.wus;
  p.win = a.win;
  p.y = a.y;
  p.hdr = a.hdr;
  p.M = a.d.M;
  p.N = N;
  p.nk = (int)ceil_div(K, kSlab);
  p.tiles = (int)ceil_div(N, F::kG * F::kCh);
  p.wide = wide ? 1 : 0;

  cudaLaunchConfig_t cfg;
  memset(&cfg, 0, sizeof(cfg));
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)team;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  const int fit = std::max(1, a.num_sms / team);
  cfg.gridDim = dim3((unsigned)(team * fit), 1, 1);
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.dynamicSmemBytes = F::kSmem;
  cfg.stream = a.stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  // no more workers than the most units there can be, and where that does not
  // settle it, no more than are resident at once: of the SMs of this stream (a green
  // context may have few), so it is asked each time
  const int64_t most = (ceil_div(a.d.M, F::kFull) + (a.win.offsets ? E : 0)) * p.tiles;
  int workers = fit;
  if (most > fit) {
    if (cudaOccupancyMaxActiveClusters(&workers, gemm_i8_kernel<kForm, kUp, O>, &cfg) != cudaSuccess || workers < 1)
      workers = fit;
    (void)cudaGetLastError();   // a failed query is not the launch's error
  }
  cfg.gridDim.x = (unsigned)(team * std::min<int64_t>(std::min(workers, fit), most));
  return cudaLaunchKernelEx(&cfg, gemm_i8_kernel<kForm, kUp, O>, p);
}

template <int kForm>
cudaError_t launch_form(const GemmI8Args& a, int team, bool wide = false) {
  const bool f32 = a.d.out_dtype == MOE_F32;
  if (a.wu) return f32 ? launch<kForm, true, float>(a, team, wide) : launch<kForm, true, __nv_bfloat16>(a, team, wide);
  return f32 ? launch<kForm, false, float>(a, team, wide) : launch<kForm, false, __nv_bfloat16>(a, team, wide);
}

}  // namespace

cudaError_t launch_gemm_i8(const GemmI8Args& a) {
  // A few dense rows without tensor cores: integer dot products keep up with the
  // weights while rows x matrices are few, or the weights are soon read.
  // Measured against the forms here, weights in L2 / from HBM, us: 7168 x 2048, one
  // row 3.3 / 4.5 against 8.4 / 8.9, eight 5.7 / 6.9 against 8.4 / 9.0; 4096 x 7168,
  // one 4.4 / 7.6 against 10.7 / 12.3, eight 9.3 / 13.9 against 10.9 / 12.4; 8192 x
  // 8192, four 9.9 / 14.0 against 15.7 / 17.6, eight 17.1 / 19.2 against 15.4 / 18.0;
  // with up 2048 x 7168, four 6.4 / 9.0 against 11.2 / 12.4; 4096 x 7168, two 11.7 /
  // 13.8 against 13.8 / 16.4, four 17.3 / 18.4 against 13.7 / 16.3
  const int64_t mats = a.wu ? 2 : 1, sums = a.d.M * mats, weights = mats * a.d.N * a.d.K;
  if (!a.win.offsets && a.d.M <= kFewRows && a.d.M * a.d.K <= kFewBytes &&
      (sums <= 4 || weights <= (sums <= 8 ? 32 : 16) * (int64_t)(1 << 20)))
    return launch_gemm_i8_few(a);
  const int64_t fill = a.d.fill > 0 && a.d.fill < a.d.M ? a.d.fill : a.d.M, E = a.d.experts;
  const int64_t nk = ceil_div(a.d.K, kSlab), ch = a.wu ? 64 : 128;
  // units to expect: experts with rows, each of its share, and in windows of what
  // few exceed where every token picks its experts at random
  const int64_t used = std::min(E, fill), even = ceil_div(fill, used);
  const int64_t share = a.win.offsets ? even + (int64_t)(2.0 * std::sqrt((double)even)) : even;
  const int64_t pairs = used * ceil_div(share, 256) * ceil_div(a.d.N, 2 * ch);
  const int64_t ones = used * ceil_div(share, 64) * ceil_div(a.d.N, ch);
  // A pair takes 0.36 us a slab (a full chunk), a CTA 0.24 us: compare the
  // rounds of units. Measured, pairs / single CTAs: 200 x 4096 x 7168 28 / 18 us;
  // 32 experts of gate/up 2048 x 7168, 64 rows each 180 / 164 us, 128 rows 186 / 234.
  // Chunks of 128 / 256 rows: 96 rows each 174 / 184 us, about 128 each 211 / 188
  // (half of the experts then have two). Chunks of more than 256 where two rounds
  // of units are full anyway.
  if (a.num_sms >= 2 && 3 * ceil_div(pairs, a.num_sms / 2) <= 2 * ceil_div(ones, a.num_sms))
    return share <= 128 ? launch_form<kPair128>(a, 2) : launch_form<kPair>(a, 2, pairs >= a.num_sms);
  // A CTA takes 0.24 us a slab; sharing K over 2 or 4 costs 2 to 4 us. Measured,
  // 1 / 2 / 4 CTAs: one row, 4096 x 7168 17.2 / 12.3 / 9.9 us, 64 rows 18.0 /
  // 15.1 / 12.0; 7168 x 2048 7.6 / 7.6 us, 64 rows 8.2 / 10.2
  int team = 1;
  while (team < 4 && ones * 2 * team <= a.num_sms && nk >= 24 * team) team *= 2;
  return team > 1 ? launch_form<kSplit>(a, team) : launch_form<kOne>(a, 1);
}

}  // namespace moe
