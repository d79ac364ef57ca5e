// kvq_batch.cu - attention of many query rows over cached sequences (cross attention, prefill of
// ragged batches), and the attention weight each cached token receives from them.
//
// x = scale q.k over the tokens a row sees; lse = log sum exp x; out = sum exp(x - lse) v;
// mass[t] = sum over rows exp(x[t] - lse).
#include <cuda_runtime.h>
#include <math.h>

#include <algorithm>
#include <atomic>
#include <type_traits>

#include "kvq_codes.cuh"
#include "kvq_internal.h"
#include "kvq_tc.cuh"

using namespace kvq;

namespace {

constexpr unsigned FULL = 0xffffffffu;
constexpr int MAXE = 32;  // entries per launch (kernel arguments of 4 KB)
constexpr float LOG2E = 1.4426950408889634f;
constexpr float LN2 = 0.6931471805599453f;

// One entry: nq query tokens from row token q0 on, over the first n rows of stream `slot`.
struct BEntry {
  int32_t slot, nq;
  int32_t out;      // position in the call's list (mass rows)
  int64_t n, q0;
  int32_t nblk;     // blocks of query tokens
  int32_t nsplit;   // splits of the key tiles
  int32_t cps;      // key tiles per split
  int32_t cta0;     // first CTA
  int64_t part0;    // first partial record (nsplit > 1)
  int32_t mgroup;   // weights: groups of key pairs per KV head,
  int32_t mpairs;   // pairs of key tiles in each,
  int32_t mqs, mqc; // splits of the query tiles, tiles in each
  int32_t mtb;      // query tokens per tile (as even as the number of tiles allows)
  int64_t mpart0;   // first partial sum (mqs > 1): [split][head][n rounded up to 4]
};

// 16-bit rows: row t of (slot, head, side) at ((slot * hkv + head) * sides + side) * cap + t; K is
// side 0, V the last; a rebuilt cache has the keys' remainders in between.
struct Source {
  const uint16_t *base;
  int64_t cap;
  int32_t slots;
  int32_t f16;    // element type: F16, else BF16
  int32_t sides;  // 2 or 3
};

struct BArgs {
  int32_t ne, hkv, G, causal, io_f16;
  float qscale;  // softmax scale * log2(e)
  Source src;
  uint16_t *out;
  float *lse;
  const float *mass_in;
  float *mass_out;
  int64_t mass_ld;
  float decay;
  float *part;
  int32_t *status;
  BEntry e[MAXE];
};

// ---- attention ------------------------------------------------------------------------------------
//
// One CTA per (entry, KV head, block of query tokens, split of the key tiles).  A tile of 128 rows
// holds the G query heads of floor(128 / G) tokens (row = token * G + head), so one K/V tile serves
// all of them; a block is two such tiles, or one when the entry has no more rows.
//  - a load warp fetches 128-token K and V tiles (32 KB each) with TMA into a ring of stages;
//  - one thread issues S = Q.K^T (M = N = 128, SS) and O += P.V (P from tensor memory, V as the
//    MN-major operand straight from the rows), S, P and O in tensor memory: 512 columns;
//  - two softmax groups of eight warps: group t owns query tile t, or, in a block of one tile, the key
//    tiles j = t mod 2 (`halves`, joined in shared memory at the end).  A row of a group belongs to two
//    threads, 64 of the tile's tokens each (one thread per row left the warps waiting on their own
//    instructions: 810 us for a causal 8k prompt of 40 heads).  While one group works on its scores
//    the tensor core runs the other's products; a half of P is handed over as soon as it is written.
//  - the running maximum moves only when a score passes it by 2^8 (the weights stay below 2^8, O is
//    rescaled in tensor memory then), so most tiles need no correction and the two threads of a row
//    only agree, by one barrier with an OR, that none is due.
// Weights are rounded to the 16-bit type of the product (V's), the sum l is of the unrounded ones.  F16 weights
// are 2^7 times as large (below 2^15): what falls under the normal range there is off by 2^-32 of the row's
// largest weight at most, not 2^-25, which many faint tokens would add up (l and the results are scaled back).
// Entries whose rows fill no more than one tile, which latency or HBM bounds, multiply the weights' remainders
// too and are as exact as their output's type, whatever else is in the call (replays, rounded weights and then
// these, BF16, 8 KV heads: one row over 4096 tokens 15.3 and 16.4 us, 16 384: 23.3 and 24.5, 65 536: 53.8 and
// 53.6, 131 072: 93.3 and 93.4; 400 calls in a row, which the power limit slows: 65 536: 53.2 and 53.8, 131 072:
// 95 and 101).  With two tiles they cost 6 % and more (causal 8k prompt 613 us for 577).
// Bound, many rows: the chain scores -> maximum -> exponentials -> weights of a tile against the other
// group's products (causal 8k prompt of 40 heads, F16: 581 us, 1183 TFLOP/s in replays with pauses, 660 to 690
// in a stream of calls, which the power limit slows; tensor pipe 53 %, exponentials 48 %).  Bound, one row:
// HBM (65 536 tokens, 268 MB: 50 us + the join, 4.9 TB/s).
constexpr int BT = 128;            // rows of a query tile, tokens of a key tile
constexpr int NSOFT = 16;          // softmax warps
constexpr int W_MMA = 16, W_LOAD = 17;
// 16 of softmax, one that issues the products, one that loads; 96 registers a thread either way
// (register splits between the warpgroups measured the same)
constexpr int NT = 576;
constexpr int TILE = BT * D * 2;   // bytes of a tile
constexpr int HALF = TILE / 2;     // 64 channels of it
constexpr int MAXST = 6;           // stages
constexpr float TAU = 8.f;         // lazy maximum, log2 units
constexpr float LIFT = 7.f;        // of F16 weights, log2 units
constexpr int PREC = 4 + D;        // floats of a partial record: m, l, -, -, acc
constexpr int MAXSPL = 64;
constexpr int EXG = BT * 129 + 2 * BT;  // floats a group leaves in the stages at the end (rows padded to 129)
static_assert(2 * EXG * 4 <= 5 * TILE, "two groups' rows fit the stages");
// which of eight score pairs are exponentiated on the FMA pipe: one (causal 8k prompt of 40 heads, replayed in
// turn: 596 us; none 603)
constexpr int EMU = 0x10;

struct Ctl {
  uint64_t full[MAXST], empty[MAXST], tmp, q_full;
  uint64_t s_full[2], p_full[4], o_full;  // p_full: [group][half]
  uint32_t tmem;
  int32_t abort;
  float row[2][2][BT];  // [group][half][row]: maxima, then sums
  // what the end of the kernel needs of the launch, so that no register holds it across the tiles
  int64_t q0, part0;
  int32_t tok0, tok1, head, sp, nsplit, halves, nt;
};
constexpr int OFF_CTL = 7 * TILE;  // two or one query tiles and five or six stages
constexpr int ATTN_SMEM = OFF_CTL + (int)sizeof(Ctl);
static_assert(ATTN_SMEM <= 232448, "shared memory per CTA");

// The visible tokens of query token i of an entry.
__device__ __forceinline__ int64_t limit_of(const BArgs &A, const BEntry &e, int i) {
  return A.causal ? e.n - e.nq + 1 + i : e.n;
}

// A position in a ring of n stages: the stage and the parity of its current round.
struct Ring {
  int at = 0;
  uint32_t phase = 0;
  __device__ __forceinline__ void next(int n) {
    if (++at == n) {
      at = 0;
      phase ^= 1u;
    }
  }
};

// The entry of this CTA.
__device__ __forceinline__ const BEntry &entry_of(const BArgs &A) {
  int ei = 0;
  while (ei + 1 < A.ne && A.e[ei + 1].cta0 <= (int)blockIdx.x) ++ei;
  return A.e[ei];
}

// LO: the keys have remainders (a rebuilt cache).  ONE: the query rows of the entry fill no more than one tile.
template <bool F16, bool LO, bool ONE>
__device__ __forceinline__ void attend(const CUtensorMap &map, const CUtensorMap &qmap, const BArgs &A) {
  extern __shared__ __align__(1024) uint8_t S[];
  const uint32_t base = tc::smem_u32(S);
  if (base & 1023u) {  // the swizzled tiles need it; no launch gives anything else
    if (threadIdx.x == 0) atomicOr(A.status, kStatusWait);
    return;
  }
  Ctl &C = *reinterpret_cast<Ctl *>(S + OFF_CTL);
  const int tid = threadIdx.x, lane = tid & 31, warp = __shfl_sync(FULL, tid >> 5, 0);
  if (warp == W_LOAD && lane == 0) {
    tc::prefetch_map(&qmap);
    tc::prefetch_map(&map);
  }
  if (warp == W_MMA) tc::tmem_alloc(tc::smem_u32(&C.tmem), 512);
  const BEntry &e = entry_of(A);
  const int G = A.G, hq = A.hkv * G, TB = BT / G;
  const int local = blockIdx.x - e.cta0;
  const int sp = local % e.nsplit, head = local / e.nsplit % A.hkv;
  const int blk = e.nblk - 1 - local / e.nsplit / A.hkv;  // the last (causal: longest) first
  const int tok0 = blk * 2 * TB, tok1 = min(e.nq, tok0 + 2 * TB);
  const bool halves = ONE || tok1 - tok0 <= TB;
  const int ntile = halves ? 1 : 2;  // query tiles
  const int64_t lim_max = limit_of(A, e, tok1 - 1);
  const int kt = (int)((lim_max + BT - 1) / BT);
  const int j0 = sp * e.cps, nt = max(0, min(e.cps, kt - j0));
  const int nst = halves ? 6 : 5;
  const uint32_t stage0 = base + ntile * TILE;
  constexpr bool lo = LO;
  constexpr int sides = LO ? 3 : 2;
  const uint32_t cb = tc::smem_u32(&C);
  const uint32_t b_full = cb + (uint32_t)offsetof(Ctl, full), b_empty = cb + (uint32_t)offsetof(Ctl, empty);
  const uint32_t b_s = cb + (uint32_t)offsetof(Ctl, s_full), b_p = cb + (uint32_t)offsetof(Ctl, p_full);
  const uint32_t b_o = cb + (uint32_t)offsetof(Ctl, o_full), b_tmp = cb + (uint32_t)offsetof(Ctl, tmp);
  const uint32_t b_q = cb + (uint32_t)offsetof(Ctl, q_full);
  volatile int32_t *abort = &C.abort;
  const int z0 = (e.slot * A.hkv + head) * sides, zv = z0 + sides - 1;

  if (warp == W_LOAD && lane == 0) {
    for (int i = 0; i < MAXST; ++i) {
      tc::mbar_init(b_full + 8 * i, 1);
      tc::mbar_init(b_empty + 8 * i, 1);
    }
    for (int i = 0; i < 2; ++i) tc::mbar_init(b_s + 8 * i, 1);
    for (int i = 0; i < 4; ++i) tc::mbar_init(b_p + 8 * i, 4);
    tc::mbar_init(b_o, 1);
    tc::mbar_init(b_tmp, 1);
    tc::mbar_init(b_q, 1);
    C.abort = 0;
    tc::fence_mbar_init();
    // (what rebuilt the rows and converted the queries is through: everything else of this CTA comes
    // behind this thread, at the barrier below)
    if (LO) asm volatile("griddepcontrol.wait;\n\tfence.proxy.async.global;" ::: "memory");
    // the query tiles and the first keys are on their way while the rest is set up.  A tile takes
    // whatever rows follow an entry's last one too: rows do not mix, and those are never written out
    // (a CTA without key tiles asks for nothing: its zeros pass through the same shared memory)
    if (nt > 0) {
      tc::mbar_expect(b_q, ntile * 2 * TB * G * 128);
      for (int t = 0; t < ntile; ++t)
        for (int h = 0; h < 2; ++h)
          tc::tma_load4(base + t * TILE + h * HALF, &qmap, 64 * h, 0, head, (int)(e.q0 + tok0 + t * TB), b_q);
      tc::mbar_expect(b_full, TILE);
      tc::tma_load3(stage0, &map, 0, j0 * BT, z0, b_full);
      tc::tma_load3(stage0 + HALF, &map, 64, j0 * BT, z0, b_full);
    }
  }
  if (tid == 0) {
    C.q0 = e.q0, C.part0 = e.part0;
    C.tok0 = tok0, C.tok1 = tok1, C.head = head, C.sp = sp, C.nsplit = e.nsplit, C.halves = halves, C.nt = nt;
  }
  tc::fence_before();
  __syncthreads();
  tc::fence_after();
  const uint32_t tm = __shfl_sync(FULL, C.tmem, 0);
  asm volatile("griddepcontrol.launch_dependents;");  // (a join, which waits for this grid's end)

  if (warp >= NSOFT) {
    if (warp == W_LOAD) {
      // ---- K and V tiles in the order they are used: two tiles K0 V0 K1 V1 ..; halves K0 K1 V0 K2 V1 ..
      int n_issued = 0;
      Ring g;
      auto load = [&](int j, int z, bool value) {
        if (n_issued >= nst) tc::mbar_wait(b_empty + 8 * g.at, g.phase ^ 1u, abort, A.status);
        const uint32_t dst = stage0 + g.at * TILE, b_st = b_full + 8 * g.at;
        const int64_t t0 = (int64_t)(j0 + j) * BT;
        const int valid = (int)min((int64_t)BT, e.n - t0);
        // rows past the sequence's end may hold anything: their keys are masked, their values would
        // turn a weight of 0 into NaN, so they are zeroed before the tile is handed over
        const bool patch = value && valid < BT;
        const uint32_t bar = patch ? b_tmp : b_st;
        if (lane == 0 && n_issued > 0) {  // (the first tile has been asked for above)
          tc::mbar_expect(bar, TILE);
          tc::tma_load3(dst, &map, 0, (int)t0, z, bar);
          tc::tma_load3(dst + HALF, &map, 64, (int)t0, z, bar);
        }
        if (patch) {  // (the last tile of the sequence: once per CTA)
          tc::mbar_wait(b_tmp, 0, abort, A.status, false);
          uint8_t *p = S + (dst - base);
          for (int u = lane; u < (BT - valid) * 16; u += 32)
            *reinterpret_cast<uint4 *>(p + (u & 1) * HALF + (valid + (u >> 4)) * 128 + ((u >> 1) & 7) * 16) =
                make_uint4(0u, 0u, 0u, 0u);
          tc::fence_async_smem();
          tc::mbar_arrive_warp(b_st);
        }
        __syncwarp();
        ++n_issued;
        g.next(nst);
      };
      auto keys = [&](int j) {
        load(j, z0, false);
        if (lo) load(j, z0 + 1, false);
      };
      if (nt > 0) keys(0);
#pragma unroll 1
      for (int j = 0; j < nt; ++j) {
        if (halves && j + 1 < nt) keys(j + 1);
        load(j, zv, true);
        if (!halves && j + 1 < nt) keys(j + 1);
      }
      // no copy is in flight when the CTA ends (its pipeline may have been given up)
      for (int i = max(0, n_issued - nst); i < n_issued; ++i)
        tc::mbar_wait(b_full + 8 * (i % nst), (i / nst) & 1, abort, A.status, false);
      if (nt > 0) tc::mbar_wait(b_q, 0, abort, A.status, false);
    } else if (warp == W_MMA && nt > 0) {
      // ---- products: the whole warp waits (its values stay in uniform registers), one lane issues
      constexpr uint32_t idS = tc::idesc(F16, BT, BT, 0), idO = tc::idesc(F16, BT, D, 1);
      const uint64_t dq = tc::desc_sw128(base, 0), dk = tc::desc_sw128(stage0, 0), dv = tc::desc_sw128(stage0, HALF);
      const bool leader = tc::elect_one();
      Ring g;
      auto take = [&]() -> uint32_t {
        const uint32_t st = g.at;
        tc::mbar_wait(b_full + 8 * st, g.phase, abort, A.status);
        g.next(nst);
        return st;
      };
      auto qk = [&](int t, int qtile, uint32_t st, uint32_t acc) {
        const uint64_t q = dq + (uint64_t)(qtile * (TILE >> 4)), k = dk + (uint64_t)(st * (TILE >> 4));
        if (leader) {
#pragma unroll
          for (int s = 0; s < D / 16; ++s) {
            const uint64_t o = (uint64_t)((s & 3) * 2 + (s >> 2) * (HALF >> 4));  // 32 bytes along the channels
            tc::mma_ss(tm + BT * t, q + o, k + o, idS, s == 0 ? acc : 1u);
          }
        }
      };
      // the j-th weights of group t, half by half as they are written: 16 tokens are 8 columns of P
      // and two groups of 8 rows of V
      auto pv = [&](int t, uint32_t ph, uint32_t st, uint32_t acc) {
        const uint64_t v = dv + (uint64_t)(st * (TILE >> 4));
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          tc::mbar_wait(b_p + 8 * (2 * t + h), ph, abort, A.status);
          tc::fence_after();
          if (leader) {
#pragma unroll
            for (int s = 0; s < 4; ++s)
              tc::mma_ts(tm + 2 * BT + D * t, tm + BT * t + 64 * h + 8 * s, v + (uint64_t)((4 * h + s) * (2048 >> 4)), idO,
                         h == 0 && s == 0 ? acc : 1u);
            if (ONE) {
#pragma unroll
              for (int s = 0; s < 4; ++s)
                tc::mma_ts(tm + 2 * BT + D * t, tm + BT * t + 64 * h + 32 + 8 * s,
                           v + (uint64_t)((4 * h + s) * (2048 >> 4)), idO, 1u);
            }
          }
        }
      };
      auto done = [&](uint32_t bar) {
        if (leader) tc::commit(bar);
      };
      tc::mbar_wait(b_q, 0, abort, A.status);
      if (!halves) {
        {
          const uint32_t k = take(), l = lo ? take() : 0;
          tc::fence_after();
#pragma unroll
          for (int t = 0; t < 2; ++t) {
            qk(t, t, k, 0u);
            if (lo) qk(t, t, l, 1u);
            done(b_s + 8 * t);
          }
          done(b_empty + 8 * k);
          if (lo) done(b_empty + 8 * l);
        }
#pragma unroll 1
        for (int j = 0; j < nt; ++j) {
          const bool more = j + 1 < nt;
          const uint32_t v = take();
          uint32_t k = 0, l = 0;
          if (more) {
            k = take();
            if (lo) l = take();
          }
#pragma unroll
          for (int t = 0; t < 2; ++t) {
            pv(t, j & 1, v, j > 0);
            if (more) {
              qk(t, t, k, 0u);
              if (lo) qk(t, t, l, 1u);
              done(b_s + 8 * t);
            }
          }
          done(b_empty + 8 * v);
          if (more) {
            done(b_empty + 8 * k);
            if (lo) done(b_empty + 8 * l);
          }
        }
      } else {
        auto keys = [&](int j) {
          const uint32_t k = take(), l = lo ? take() : 0;
          tc::fence_after();
          qk(j & 1, 0, k, 0u);
          if (lo) qk(j & 1, 0, l, 1u);
          done(b_s + 8 * (j & 1));
          done(b_empty + 8 * k);
          if (lo) done(b_empty + 8 * l);
        };
        // S and P of a group share columns: the scores of tile j + 2 follow the product of tile j
        keys(0);
        if (nt > 1) keys(1);
#pragma unroll 1
        for (int j = 0; j < nt; ++j) {
          const uint32_t v = take();
          pv(j & 1, (j >> 1) & 1, v, j >= 2);
          done(b_empty + 8 * v);
          if (j + 2 < nt) keys(j + 2);
        }
      }
      done(b_o);
      tc::mbar_wait(b_o, 0, abort, A.status, false);
    }
  } else {
    // ---- softmax: row r of query tile t (halves: of the one tile), tokens 64 h .. 64 h + 63 of a tile
    const int t = warp >> 3, h = (warp >> 2) & 1, r = tid & 127;
    const uint32_t lanes = (uint32_t)(32 * (warp & 3)) << 16;
    const uint32_t tS = tm + lanes + BT * t + 64 * h, tO = tm + lanes + 2 * BT + D * t + 64 * h;
    const int pair = 1 + 4 * t + (warp & 3);  // barrier of the two warps that share these rows
    // (rows that hold no query see everything, a mask for them would hold up their warp on every tile, and
    // never move the maximum: the products of what lies behind the queries in shared memory are anything)
    const bool live = r < TB * G;
    const int row_tok = tok0 + (halves ? 0 : t * TB) + r / G;
    // visible tokens from this thread's half of the group's first tile on; tiles of the group
    int left = (int)(live && row_tok < tok1 ? limit_of(A, e, row_tok) : e.n) - (j0 + (halves ? t : 0)) * BT - 64 * h;
    const int count = halves ? (nt + 1 - t) >> 1 : nt, stride = halves ? 2 * BT : BT;
    float m = -INFINITY, l = 0.f;
#pragma unroll 1
    for (int u = 0; u < count; ++u, left -= stride) {
      tc::mbar_wait(b_s + 8 * t, u & 1, abort, A.status);
      tc::fence_after();
      float s[64], mx[4];
#pragma unroll
      for (int v = 0; v < 4; ++v) mx[v] = -INFINITY;
      // the first 32 are searched for their maximum while the others are read
      tc::tmem_ld32(tS, s);
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        tc::tmem_wait_ld();
        if (c == 0) tc::tmem_ld32(tS + 32, s + 32);
        if (left < 64) {
#pragma unroll
          for (int v = 0; v < 32; ++v)
            if (32 * c + v >= left) s[32 * c + v] = -INFINITY;
        }
#pragma unroll
        for (int v = 0; v < 32; v += 8) {
#pragma unroll
          for (int k = 0; k < 4; ++k) mx[k] = fmaxf(fmaxf(mx[k], s[32 * c + v + k]), s[32 * c + v + 4 + k]);
        }
      }
      float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * A.qscale;
      if (!live) top = -INFINITY;
      if (tc::bar_any(pair, 64, top > m + TAU)) {
        // a row's first scores, or some far above the maximum in use: both threads take the new one
        C.row[t][h][r] = top;
        tc::bar_sync(pair, 64);
        const float both = fmaxf(top, C.row[t][h ^ 1][r]);
        float alpha = 1.f;
        if (both > m + TAU) {
          alpha = tc::ex2(m - both);  // (m = -inf, nothing summed yet: 0)
          m = both;
          l *= alpha;
        }
        if (u > 0 && __any_sync(FULL, alpha != 1.f)) {
#pragma unroll 1
          for (int c = 0; c < 64; c += 16) {  // (the scores are held meanwhile: few registers are left)
            uint32_t o[16];
            tc::tmem_ld16(tO + c, o);
            tc::tmem_wait_ld();
#pragma unroll
            for (int v = 0; v < 16; ++v) o[v] = __float_as_uint(__uint_as_float(o[v]) * alpha);
            tc::tmem_st16(tO + c, o);
          }
          tc::tmem_wait_st();
          tc::fence_before();
        }
        // (a half of P lets the product add to every channel: both halves are rescaled by then)
        tc::bar_sync(pair, 64);
        tc::fence_after();
      }
      const float sub = m == -INFINITY ? 0.f : (F16 ? LIFT - m : -m);
      const tc::f2 sc = tc::pack2(A.qscale, A.qscale), ms = tc::pack2(sub, sub);
      tc::f2 sum[4] = {0ull, 0ull, 0ull, 0ull};
      // P over the scores this thread has read; with ONE the weights' remainders behind it
      if constexpr (ONE) {
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          uint32_t hi[8], lo16[8];
#pragma unroll
          for (int v = 0; v < 8; ++v) {
            float x0, x1;
            const int at = 16 * c + 2 * v;
            tc::unpack2(tc::fma2(tc::pack2(s[at], s[at + 1]), sc, ms), x0, x1);
            x0 = tc::ex2(x0);
            x1 = tc::ex2(x1);
            sum[v & 3] = tc::add2(sum[v & 3], tc::pack2(x0, x1));
            hi[v] = tc::round2<F16>(x0, x1);
            const float2 f = tc::widen2<F16>(hi[v]);
            lo16[v] = tc::round2<F16>(x0 - f.x, x1 - f.y);
          }
          tc::tmem_st8(tS + 8 * c, hi);
          tc::tmem_st8(tS + 32 + 8 * c, lo16);
        }
      } else {
        uint32_t w[32];
#pragma unroll
        for (int v = 0; v < 32; ++v) {
          float x0, x1;
          const tc::f2 x = tc::fma2(tc::pack2(s[2 * v], s[2 * v + 1]), sc, ms);
          if ((EMU >> (v & 7)) & 1) {
            tc::ex2_fma<false>(x, x0, x1);
          } else {
            tc::unpack2(x, x0, x1);
            x0 = tc::ex2(x0);
            x1 = tc::ex2(x1);
          }
          sum[v & 3] = tc::add2(sum[v & 3], tc::pack2(x0, x1));
          w[v] = tc::round2<F16>(x0, x1);
        }
        tc::tmem_st32(tS, w);
      }
      tc::tmem_wait_st();
      tc::fence_before();
      tc::mbar_arrive_warp(b_p + 8 * (2 * t + h));
      float l0, l1;
      tc::unpack2(tc::add2(tc::add2(sum[0], sum[1]), tc::add2(sum[2], sum[3])), l0, l1);
      l += l0 + l1;
    }
    // ---- the result: m, l of the row, 64 channels of the accumulator
    C.row[t][h][r] = l;
    tc::bar_sync(pair, 64);
    constexpr float back = F16 ? 1.f / (1 << (int)LIFT) : 1.f;
    l = (C.row[t][0][r] + C.row[t][1][r]) * back;
    const int tiles = C.nt;
    if (tiles > 0) {
      tc::mbar_wait(b_o, 0, abort, A.status);
      tc::fence_after();
    }
    // halves: group 1 leaves its own in the stages (all consumed), group 0 joins the two
    const bool one = ONE || C.halves, join = one && tiles > 1, split = C.nsplit > 1;
    float *ex = reinterpret_cast<float *>(S + (one ? 1 : 2) * TILE);  // [128 rows][129], then m and l
    if (join && t == 1) {
#pragma unroll 1
      for (int c = 0; c < 2; ++c) {
        float o[32];
        tc::tmem_ld32(tO + 32 * c, o);
        tc::tmem_wait_ld();
#pragma unroll
        for (int v = 0; v < 32; ++v) ex[r * 129 + 64 * h + 32 * c + v] = o[v];
      }
      if (h == 0) {
        ex[128 * 129 + 2 * r] = m;
        ex[128 * 129 + 2 * r + 1] = l;
      }
    }
    if (join) tc::bar_sync(9, 32 * NSOFT);
    if (!(one && t == 1)) {
      float f0 = 1.f, f1 = 0.f;
      if (join) {
        const float m1 = ex[128 * 129 + 2 * r], l1 = ex[128 * 129 + 2 * r + 1];
        const float mn = fmaxf(m, m1);
        f0 = m == -INFINITY ? 0.f : tc::ex2(m - mn);
        f1 = m1 == -INFINITY ? 0.f : tc::ex2(m1 - mn);
        m = mn;
        l = l * f0 + l1 * f1;
      }
      // a split's rows in fp32, behind what the other group left; otherwise through the query tile (no
      // product reads it any more), in its layout
      const float inv = split ? back : (l > 0.f ? back / l : (l == l ? 0.f : l));
      float *part = ex + (one ? 1 : t) * EXG;
      uint8_t *qt = S + t * TILE;
#pragma unroll 1
      for (int c = 0; c < 2; ++c) {
        float o[32];
        if (tiles > 0) {
          tc::tmem_ld32(tO + 32 * c, o);
          tc::tmem_wait_ld();
        } else {
#pragma unroll
          for (int v = 0; v < 32; ++v) o[v] = 0.f;
        }
        const int ch = 64 * h + 32 * c;
        if (join) {
#pragma unroll
          for (int v = 0; v < 32; ++v) o[v] = o[v] * f0 + ex[r * 129 + ch + v] * f1;
        }
        if (split) {
#pragma unroll
          for (int v = 0; v < 32; ++v) part[r * 129 + ch + v] = o[v] * inv;
        } else {
          uint8_t *dst = qt + h * HALF + r * 128;
#pragma unroll
          for (int v = 0; v < 4; ++v) {
            uint32_t w[4];
#pragma unroll
            for (int k = 0; k < 4; ++k)
              w[k] = A.io_f16 ? tc::round2<true>(o[8 * v + 2 * k] * inv, o[8 * v + 2 * k + 1] * inv)
                              : tc::round2<false>(o[8 * v + 2 * k] * inv, o[8 * v + 2 * k + 1] * inv);
            *reinterpret_cast<uint4 *>(dst + (((4 * c + v) ^ (r & 7)) << 4)) = make_uint4(w[0], w[1], w[2], w[3]);
          }
        }
      }
      // whole rows to memory, 512 or 256 bytes at once
      tc::bar_sync(10 + t, 256);
      const int first = C.tok0 + (one ? 0 : t * TB), rows = min(TB, C.tok1 - first) * G;  // (below 0: none)
      const int head0 = C.head * G, ns = C.nsplit;
      if (split) {
        float *rec0 = A.part + (C.part0 + (int64_t)C.sp) * PREC;
        for (int rr = (tid & 255) >> 5; rr < rows; rr += 8) {
          const float *v = part + rr * 129 + 4 * lane;
          *reinterpret_cast<float4 *>(rec0 + ((int64_t)(first + rr / G) * hq + head0 + rr % G) * ns * PREC + 4 + 4 * lane) =
              make_float4(v[0], v[1], v[2], v[3]);
        }
        if (h == 0 && r < rows) {
          float *rec = rec0 + ((int64_t)(first + r / G) * hq + head0 + r % G) * ns * PREC;
          rec[0] = m;
          rec[1] = l;
        }
      } else {
        for (int p = tid & 255; p < rows * 16; p += 256) {
          const int rr = p >> 4, c = p & 15;
          const int64_t at = (C.q0 + first + rr / G) * hq + head0 + rr % G;
          *reinterpret_cast<uint4 *>(A.out + at * D + 8 * c) =
              *reinterpret_cast<const uint4 *>(qt + (c >> 3) * HALF + rr * 128 + (((c & 7) ^ (rr & 7)) << 4));
        }
        if (A.lse && h == 0 && r < rows)
          A.lse[(C.q0 + first + r / G) * hq + head0 + r % G] = l == 0.f ? -INFINITY : (m + log2f(l)) * LN2;
      }
    }
  }
  tc::fence_before();
  __syncthreads();
  tc::fence_after();
  if (warp == W_MMA) tc::tmem_free(tm, 512);
}

// A launch of entries of one tile of rows (ONE), of more (MORE), or of both (ANY), whose CTAs take either body
// (31 entries of one row and one of 512 over 4096 tokens: 163 us, with the choice inside one body 168, all
// weights rounded 151; 7 of one row and one of 2048 over 8192: 371, 408, 367).
enum Rows { ONE, MORE, ANY };
template <bool F16, bool LO, Rows ROWS>
__global__ void __launch_bounds__(NT, 1) k_attn(const __grid_constant__ CUtensorMap map,
                                                const __grid_constant__ CUtensorMap qmap,
                                                const __grid_constant__ BArgs A) {
  if (ROWS == ONE || (ROWS == ANY && entry_of(A).nq <= BT / A.G))
    attend<F16, LO, true>(map, qmap, A);
  else
    attend<F16, LO, false>(map, qmap, A);
}

// Joins the splits of a row (log-sum-exp, in split order): a block per (query token, query head), a
// thread per channel, all splits' loads in flight.  Set up behind the attention, waiting only for it.
__global__ void __launch_bounds__(D) k_attn_join(const __grid_constant__ BArgs A) {
  __shared__ float weight[MAXSPL];
  __shared__ float total[2];
  const int tid = threadIdx.x, hq = A.hkv * A.G;
  int64_t it = blockIdx.x;
  int ei = 0;
  for (;; ++ei) {
    const int64_t c = A.e[ei].nsplit > 1 ? (int64_t)A.e[ei].nq * hq : 0;
    if (it < c) break;
    it -= c;
  }
  const int ns = A.e[ei].nsplit;
  const float *rec = A.part + (A.e[ei].part0 + it * ns) * PREC;
  const int64_t row = A.e[ei].q0 * hq + it;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (tid < 32) {
    float m[2], l[2], M = -INFINITY;
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int k = tid + 32 * u;
      m[u] = k < ns ? rec[(int64_t)k * PREC] : -INFINITY;
      l[u] = k < ns ? rec[(int64_t)k * PREC + 1] : 0.f;
      M = fmaxf(M, m[u]);
    }
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) M = fmaxf(M, __shfl_xor_sync(FULL, M, o));
    float L = 0.f;
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const float f = m[u] == -INFINITY ? 0.f : tc::ex2(m[u] - M);
      weight[tid + 32 * u] = f;
      L = fmaf(f, l[u], L);
    }
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) L += __shfl_xor_sync(FULL, L, o);
    if (tid == 0) {
      total[0] = L;
      if (A.lse) A.lse[row] = L == 0.f ? -INFINITY : (M + log2f(L)) * LN2;
    }
  }
  float v[16], a = 0.f;
  for (int k0 = 0; k0 < ns; k0 += 16) {
#pragma unroll
    for (int u = 0; u < 16; ++u) v[u] = k0 + u < ns ? rec[(int64_t)(k0 + u) * PREC + 4 + tid] : 0.f;
    if (k0 == 0) __syncthreads();
#pragma unroll
    for (int u = 0; u < 16; ++u)
      if (k0 + u < ns) a = fmaf(weight[k0 + u], v[u], a);
  }
  const float L = total[0], o = a * (L > 0.f ? 1.f / L : (L == L ? 0.f : L));
  A.out[row * D + tid] = A.io_f16 ? __half_as_ushort(__float2half_rn(o)) : __bfloat16_as_ushort(__float2bfloat16_rn(o));
}

// ---- attention weights ------------------------------------------------------------------------------
//
// mass[t] = sum over query rows r of 2^(x[t, r] - lse2[r]): with the lse given, one product and one
// exponential per (token, row), no second pass.  The product is taken the other way round, S^T = K.Q^T
// (tokens are the MMA's rows), so that a sum stays in its thread (two per token, half of the columns
// each): no shuffles, no atomics, the order of the sum fixed by the tiles.
//
// One CTA per (entry, KV head, group of key-tile pairs, split of the query tiles): the two key tiles of
// a pair belong to the two groups of eight warps and share each query tile.  Up to three query tiles
// stay in shared memory while the keys stream past (a window of queries: each key is read once, HBM
// bound); more of them stream for each pair (a prompt: bound by the exponentials, 16 a cycle and SM).
// Query tiles come by TMA as [token][head] rows of 64 channels, the tokens spread evenly over the
// tiles; only the columns that hold queries are exponentiated, in steps of 8.
// 32 queries over 65 536 tokens: 45 us (134 MB; exponentials and products take turns); every query of
// prompts of 4096 and 512 tokens: 150 us (exponential unit 64 % busy).
constexpr int NKS = 4, NQS = 3;  // key and query stages
constexpr int OFF_MCTL = (NKS + NQS) * TILE;

struct MCtl {
  uint64_t k_full[NKS], k_empty[NKS], q_full[NQS], q_empty[NQS], s_full[4], s_empty[4], last;
  uint64_t h_full[8], h_free[8];    // half sums of a warp's 32 keys: written, read
  alignas(16) float nlse[NQS][BT];  // -lse * log2(e) of the tile's rows
  float half[2][BT];                // sums of the second half of the columns
  uint32_t tmem;
  int32_t abort;
};
constexpr int MASS_SMEM = OFF_MCTL + (int)sizeof(MCtl);

// which of four groups of columns have half of theirs exponentiated on the FMA pipe: one (weights of a
// 4k prompt: 149 us; none 152)
constexpr int MEMU = 0x1;
static_assert(MASS_SMEM <= 232448, "shared memory per CTA");

template <bool F16>
__global__ void __launch_bounds__(NT, 1) k_mass(const __grid_constant__ CUtensorMap kmap,
                                                const __grid_constant__ CUtensorMap qmap,
                                                const __grid_constant__ BArgs A) {
  extern __shared__ __align__(1024) uint8_t S[];
  const uint32_t base = tc::smem_u32(S);
  if (base & 1023u) {  // the swizzled tiles need it; no launch gives anything else
    if (threadIdx.x == 0) atomicOr(A.status, kStatusWait);
    return;
  }
  MCtl &C = *reinterpret_cast<MCtl *>(S + OFF_MCTL);
  const int tid = threadIdx.x, lane = tid & 31, warp = __shfl_sync(FULL, tid >> 5, 0);
  const BEntry &e = entry_of(A);
  const int G = A.G, hq = A.hkv * G, TB = e.mtb, box = BT / G;  // tokens of a tile, of a copy
  const int local = blockIdx.x - e.cta0;
  const int qs = local % e.mqs, head = local / e.mqs % A.hkv;
  const int grp = local / e.mqs / A.hkv;  // the first keys (causal: seen by most queries) first
  const int npair = (int)((e.n + 2 * BT - 1) / (2 * BT));
  const int p0 = grp * e.mpairs, p1 = min(npair, p0 + e.mpairs);
  const int nqt = (e.nq + TB - 1) / TB;  // tiles of query tokens
  const int qb = min(nqt, (qs + 1) * e.mqc);
  // first query tile of this split that sees any key of pair p
  auto first_tile = [&](int p) -> int {
    const int64_t i = (int64_t)p * 2 * BT - (e.n - e.nq);
    return max(qs * e.mqc, A.causal && i > 0 ? (int)(i / TB) : 0);
  };
  const int f0 = first_tile(p0);
  if (f0 >= qb && e.mqs > 1) return;  // no query of the split sees the group (the join leaves it out)
  const bool resident = qb - f0 <= NQS;
  const bool lo = A.src.sides == 3;
  const uint32_t q0s = base + NKS * TILE;
  const uint32_t cb = tc::smem_u32(&C);
  const uint32_t b_kf = cb + (uint32_t)offsetof(MCtl, k_full), b_ke = cb + (uint32_t)offsetof(MCtl, k_empty);
  const uint32_t b_qf = cb + (uint32_t)offsetof(MCtl, q_full), b_qe = cb + (uint32_t)offsetof(MCtl, q_empty);
  const uint32_t b_sf = cb + (uint32_t)offsetof(MCtl, s_full), b_se = cb + (uint32_t)offsetof(MCtl, s_empty);
  const uint32_t b_hf = cb + (uint32_t)offsetof(MCtl, h_full), b_he = cb + (uint32_t)offsetof(MCtl, h_free);
  const uint32_t b_last = cb + (uint32_t)offsetof(MCtl, last);
  volatile int32_t *abort = &C.abort;

  if (warp == W_LOAD && lane == 0) {
    for (int i = 0; i < NKS; ++i) {
      tc::mbar_init(b_kf + 8 * i, 1);
      tc::mbar_init(b_ke + 8 * i, 1);
    }
    for (int i = 0; i < NQS; ++i) {
      tc::mbar_init(b_qf + 8 * i, 2);           // the copy, and the lse values
      tc::mbar_init(b_qe + 8 * i, 1 + NSOFT);   // the products, and the softmax warps
    }
    for (int i = 0; i < 4; ++i) {
      tc::mbar_init(b_sf + 8 * i, 1);
      tc::mbar_init(b_se + 8 * i, 8);
    }
    for (int i = 0; i < 8; ++i) {
      tc::mbar_init(b_hf + 8 * i, 1);
      tc::mbar_init(b_he + 8 * i, 1);
    }
    tc::mbar_init(b_last, 1);
    C.abort = 0;
    tc::fence_mbar_init();
  }
  if (warp == W_MMA) tc::tmem_alloc(cb + (uint32_t)offsetof(MCtl, tmem), 512);
  tc::fence_before();
  __syncthreads();
  tc::fence_after();
  const uint32_t tm = __shfl_sync(FULL, C.tmem, 0);
  asm volatile("griddepcontrol.launch_dependents;");  // (a join, which waits for this grid's end)
  const int z0 = (e.slot * A.hkv + head) * A.src.sides;

  if (warp == W_LOAD) {
    int kc = 0, qc = 0;
    auto load_k = [&](int64_t t0, int z) {
      const int st = kc % NKS;
      if (kc >= NKS) tc::mbar_wait(b_ke + 8 * st, (kc / NKS - 1) & 1, abort, A.status);
      if (lane == 0) {
        tc::mbar_expect(b_kf + 8 * st, TILE);
        tc::tma_load3(base + st * TILE, &kmap, 0, (int)t0, z, b_kf + 8 * st);
        tc::tma_load3(base + st * TILE + HALF, &kmap, 64, (int)t0, z, b_kf + 8 * st);
      }
      __syncwarp();
      ++kc;
    };
    // the lse of a tile's columns, four per lane, fetched a tile ahead of their use
    int off[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) off[k] = (lane + 32 * k) / G * hq + (lane + 32 * k) % G;
    auto fetch = [&](int a, float (&v)[4]) {
      const int nc = a < qb ? min(TB, e.nq - a * TB) * G : 0;
      const float *src = A.lse + (e.q0 + (int64_t)a * TB) * hq + head * G;
#pragma unroll
      for (int k = 0; k < 4; ++k) v[k] = lane + 32 * k < nc ? __ldg(src + off[k]) : -INFINITY;
    };
    float ahead[4];
    auto load_q = [&](int a, bool first) {
      const int st = qc % NQS;
      if (first) fetch(a, ahead);
      if (qc >= NQS) tc::mbar_wait(b_qe + 8 * st, (qc / NQS - 1) & 1, abort, A.status);
      // the copy also brings the rows behind the tile's last: their columns are never added up
      if (lane == 0) {
        tc::mbar_expect(b_qf + 8 * st, 2 * box * G * 128);
        tc::tma_load4(q0s + st * TILE, &qmap, 0, 0, head, (int)(e.q0 + a * TB), b_qf + 8 * st);
        tc::tma_load4(q0s + st * TILE + HALF, &qmap, 64, 0, head, (int)(e.q0 + a * TB), b_qf + 8 * st);
      }
#pragma unroll
      for (int k = 0; k < 4; ++k)
        C.nlse[st][lane + 32 * k] = ahead[k] == -INFINITY ? -INFINITY : -ahead[k] * LOG2E;
      tc::mbar_arrive_warp(b_qf + 8 * st);
      fetch(a + 1, ahead);
      ++qc;
    };
#pragma unroll 1
    for (int p = p0; p < p1; ++p) {
      const int f = first_tile(p);
      if (f >= qb) break;  // (the keys behind see fewer queries still)
      const int64_t key0 = (int64_t)p * 2 * BT;
      for (int t = 0; t < 2 && key0 + t * BT < e.n; ++t) {
        load_k(key0 + t * BT, z0);
        if (lo) load_k(key0 + t * BT, z0 + 1);
      }
      if (!resident || p == p0)
        for (int a = f; a < qb; ++a) load_q(a, a == f);
    }
    for (int i = max(0, kc - NKS); i < kc; ++i)
      tc::mbar_wait(b_kf + 8 * (i % NKS), (i / NKS) & 1, abort, A.status, false);
    for (int i = max(0, qc - NQS); i < qc; ++i)
      tc::mbar_wait(b_qf + 8 * (i % NQS), (i / NQS) & 1, abort, A.status, false);
  } else if (warp == W_MMA) {
    const uint64_t dk = tc::desc_sw128(base, 0), dq = tc::desc_sw128(q0s, 0);
    const bool leader = tc::elect_one();
    Ring gk, gq;
    uint32_t used[2] = {0, 0};  // score buffers filled, per key tile of the pair
#pragma unroll 1
    for (int p = p0; p < p1; ++p) {
      const int f = first_tile(p);
      if (f >= qb) break;
      const int nk = (int64_t)p * 2 * BT + BT < e.n ? 2 : 1;
      uint32_t ks[4];  // the pair's stages
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        if (u >= nk * (lo ? 2 : 1)) break;
        ks[u] = gk.at;
        tc::mbar_wait(b_kf + 8 * gk.at, gk.phase, abort, A.status);
        gk.next(NKS);
      }
#pragma unroll 1
      for (int a = f; a < qb; ++a) {
        const uint32_t st = resident ? a - f0 : gq.at;
        tc::mbar_wait(b_qf + 8 * st, resident ? 0u : gq.phase, abort, A.status);
        if (!resident) gq.next(NQS);
        const uint64_t q = dq + (uint64_t)(st * (TILE >> 4));
        // (as many columns as the tile's queries need, in steps of 16)
        const uint32_t idS = tc::idesc(F16, BT, (min(TB, e.nq - a * TB) * G + 15) / 16 * 16, 0);
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          if (t >= nk) break;
          const uint32_t b = 2 * t + (used[t] & 1);
          if (used[t] >= 2) tc::mbar_wait(b_se + 8 * b, (used[t] / 2 - 1) & 1, abort, A.status);
          ++used[t];
          tc::fence_after();
          auto product = [&](uint32_t kst, uint32_t acc) {
            const uint64_t k = dk + (uint64_t)(kst * (TILE >> 4));
#pragma unroll
            for (int s = 0; s < D / 16; ++s) {
              const uint64_t o = (uint64_t)((s & 3) * 2 + (s >> 2) * (HALF >> 4));
              tc::mma_ss(tm + BT * b, k + o, q + o, idS, s == 0 ? acc : 1u);
            }
          };
          if (leader) {
            product(lo ? ks[2 * t] : ks[t], 0u);
            if (lo) product(ks[2 * t + 1], 1u);
            tc::commit(b_sf + 8 * b);
          }
        }
        if (!resident && leader) tc::commit(b_qe + 8 * st);
      }
      if (leader) {
#pragma unroll
        for (int u = 0; u < 4; ++u)
          if (u < nk * (lo ? 2 : 1)) tc::commit(b_ke + 8 * ks[u]);
      }
    }
    if (leader) tc::commit(b_last);
    tc::mbar_wait(b_last, 0, abort, A.status, false);
  } else if (warp < NSOFT) {
    // key r of the pair's tile t, the query columns 64 h .. 64 h + 63 of each tile
    const int t = warp >> 3, h = (warp >> 2) & 1, r = tid & 127;
    const uint32_t lanes = (uint32_t)(32 * (warp & 3)) << 16;
    const tc::f2 sc2 = tc::pack2(A.qscale, A.qscale);
    const int n = (int)e.n, nq = e.nq, past = n - nq;  // (fewer than 2^31 tokens)
    const bool causal = A.causal;
    uint32_t sc = 0;
    Ring g;
#pragma unroll 1
    for (int p = p0; p < p1; ++p) {
      const int f = first_tile(p);
      const int tile0 = p * 2 * BT + t * BT, key = tile0 + r;
      float total = 0.f, rest = 0.f;  // the sum over query tiles and what its additions rounded off
#pragma unroll 1
      for (int a = f; a < qb; ++a) {
        const int st = resident ? a - f0 : g.at;
        tc::mbar_wait(b_qf + 8 * st, resident ? 0u : g.phase, abort, A.status);
        if (!resident) g.next(NQS);
        if (tile0 < n) {
          // the tile's columns in two halves of a multiple of 8; this thread's are [0, ncol) of its half,
          // those below c0 are queries in front of the token (causal)
          const int tok = a * TB, nc = min(TB, nq - tok) * G, hc = (nc + 15) / 16 * 8;
          const int ncol = h ? nc - hc : min(hc, nc);
          const bool diag = causal && tile0 + BT - 1 - past > tok;
          const int c0 = diag ? min(max(key - past - tok, 0), BT) * G - h * hc : 0;
          const uint32_t b = 2 * t + (sc & 1), tS = tm + lanes + BT * b + h * hc;
          const float4 *nl = reinterpret_cast<const float4 *>(&C.nlse[st][h * hc]);
          tc::mbar_wait(b_sf + 8 * b, (sc >> 1) & 1, abort, A.status);
          ++sc;
          tc::fence_after();
          tc::f2 sum[4] = {0ull, 0ull, 0ull, 0ull};
          float s[64];
          auto mask = [&](int from, int to) {
#pragma unroll
            for (int c = 0; c < 64; ++c)
              if (c >= from && c < to && (c < c0 || c >= ncol)) s[c] = -INFINITY;
          };
          auto add = [&](int c, tc::f2 xa, tc::f2 xb) {  // columns 4 c .. 4 c + 3
            float x0, x1, x2, x3;
            if ((MEMU >> (c & 3)) & 1) {
              tc::ex2_fma<true>(xa, x0, x1);
            } else {
              tc::unpack2(xa, x0, x1);
              x0 = tc::ex2(x0);
              x1 = tc::ex2(x1);
            }
            tc::unpack2(xb, x2, x3);
            sum[2 * (c & 1)] = tc::add2(sum[2 * (c & 1)], tc::pack2(x0, x1));
            sum[2 * (c & 1) + 1] = tc::add2(sum[2 * (c & 1) + 1], tc::pack2(tc::ex2(x2), tc::ex2(x3)));
          };
          // n columns from group `from` of four on: tiles on the diagonal are masked behind the subtraction,
          // since the lse of a row that does not see the token may be NaN
          auto exps = [&](auto masked, int from, int n) {
            if constexpr (decltype(masked)::value) {
#pragma unroll
              for (int u = 0; u < n; ++u) {
                const int c = from + u;
                const float4 n4 = nl[c];
                tc::unpack2(tc::fma2(tc::pack2(s[4 * c], s[4 * c + 1]), sc2, tc::pack2(n4.x, n4.y)), s[4 * c], s[4 * c + 1]);
                tc::unpack2(tc::fma2(tc::pack2(s[4 * c + 2], s[4 * c + 3]), sc2, tc::pack2(n4.z, n4.w)), s[4 * c + 2],
                            s[4 * c + 3]);
              }
              mask(4 * from, 4 * (from + n));
#pragma unroll
              for (int u = 0; u < n; ++u) {
                const int c = from + u;
                add(c, tc::pack2(s[4 * c], s[4 * c + 1]), tc::pack2(s[4 * c + 2], s[4 * c + 3]));
              }
            } else {
#pragma unroll
              for (int u = 0; u < n; ++u) {
                const int c = from + u;
                const float4 n4 = nl[c];
                add(c, tc::fma2(tc::pack2(s[4 * c], s[4 * c + 1]), sc2, tc::pack2(n4.x, n4.y)),
                    tc::fma2(tc::pack2(s[4 * c + 2], s[4 * c + 3]), sc2, tc::pack2(n4.z, n4.w)));
              }
            }
          };
          auto tile = [&](auto masked) {
            constexpr bool late = decltype(masked)::value;
            tc::tmem_ld32(tS, s);
            tc::tmem_wait_ld();
            if (ncol > 32) tc::tmem_ld32(tS + 32, s + 32);
            if (!late && ncol < 32) mask(0, 32);
            exps(masked, 0, 8);
            if (ncol > 32) tc::tmem_wait_ld();
            tc::fence_before();
            tc::mbar_arrive_warp(b_se + 8 * b);
            // the second 32: all of them when nearly full, else in steps of 8
            if (!late) {
              if (ncol > 56)
                mask(56, 64);
            }
            if (ncol > 56) {
              exps(masked, 8, 8);
            } else {
#pragma unroll
              for (int c = 8; c < 14; c += 2) {
                if (4 * c >= ncol) break;
                if (!late && 4 * c + 8 > ncol) mask(4 * c, 4 * c + 8);
                exps(masked, c, 2);
              }
            }
          };
          if (__builtin_expect(!diag, 1))
            tile(std::false_type{});
          else
            tile(std::true_type{});
          float v0, v1;
          tc::unpack2(tc::add2(tc::add2(sum[0], sum[1]), tc::add2(sum[2], sum[3])), v0, v1);
          const float v = v0 + v1, w = total + v, d = w - total;
          rest += (total - (w - d)) + (v - d);
          total = w;
        }
        if (!resident) tc::mbar_arrive_warp(b_qe + 8 * st);
      }
      // the second half hands its sum over and goes on, the first one writes
      if (total != INFINITY) total += rest;  // (of an infinite sum the rest is NaN)
      const uint32_t hb = 8 * (4 * t + (warp & 3));
      if (h == 1) {
        if (p > p0) tc::mbar_wait(b_he + hb, (p - p0 - 1) & 1, abort, A.status);
        C.half[t][r] = total;
        tc::mbar_arrive_warp(b_hf + hb);
      } else {
        tc::mbar_wait(b_hf + hb, (p - p0) & 1, abort, A.status);
        const float v = total + C.half[t][r];
        tc::mbar_arrive_warp(b_he + hb);
        if (key < n) {
          if (e.mqs > 1) {
            A.part[e.mpart0 + ((int64_t)qs * A.hkv + head) * ((e.n + 3) & ~3ll) + key] = v;
          } else {
            const int64_t at = ((int64_t)e.out * A.hkv + head) * A.mass_ld + key;
            A.mass_out[at] = A.decay != 0.f ? A.decay * A.mass_in[at] + v : v;
          }
        }
      }
    }
  }
  tc::fence_before();
  __syncthreads();
  tc::fence_after();
  if (warp == W_MMA) tc::tmem_free(tm, 512);
}

// Adds the splits of the query tiles, in order: one thread per (token, KV head).
__global__ void __launch_bounds__(256) k_mass_join(const __grid_constant__ BArgs A, int64_t items) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  int64_t it = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (it >= items) return;
  int ei = 0;
  for (;; ++ei) {
    const int64_t c = A.e[ei].mqs > 1 ? A.e[ei].n * A.hkv : 0;
    if (it < c) break;
    it -= c;
  }
  const BEntry &e = A.e[ei];
  const int64_t head = it / e.n, t = it % e.n, ld = (e.n + 3) & ~3ll;
  // splits of which no query sees the group of t hold nothing
  const int64_t i = t / (2 * BT) / e.mpairs * e.mpairs * 2 * BT - (e.n - e.nq);
  float v = 0.f;
  for (int k = A.causal && i > 0 ? (int)(i / e.mtb) / e.mqc : 0; k < e.mqs; ++k)
    v += A.part[e.mpart0 + (k * A.hkv + head) * ld + t];
  const int64_t at = ((int64_t)e.out * A.hkv + head) * A.mass_ld + t;
  A.mass_out[at] = A.decay != 0.f ? A.decay * A.mass_in[at] + v : v;
}

// ---- quantized caches: values rebuilt in the original basis as F16 rows --------------------------
// A warp takes four tokens of a (slot, head, side); a token belongs to eight lanes, 16 channels each
// (lane part p: channels 4 p + 32 j + (0..3), j = 0..3: one 32-bit word of the stored planes per
// block).  Keys are kept as an F16 high part and the F16 remainder (22 bits: a score is an exponent, and
// the log-sum-exp and the weights are fp32 results); values, whose result is rounded to 16 bits, as one F16.  Bound: the stores
// (9217 tokens of 8 heads, q8_0, K and V in one launch: 18 us for 57 MB written, 20 MB read).
// The blocks behind the slots' turn BF16 queries into F16 rows for the products (exact in the F16 range).
constexpr int MAXR = 128;  // slots per launch
struct Rebuild {
  int32_t n, which;  // slots; side (2: K and V, by blockIdx.y)
  int64_t cap;
  int32_t first;     // slot of entry 0
  int32_t blocks;    // those of the slots
  const uint4 *q;    // BF16 queries to convert, nq pieces of 8, or none
  uint4 *q16;
  int64_t nq;
  struct {
    int32_t seq, n, Q, block0;
  } s[MAXR];
};
constexpr int RT = 32;  // tokens of a block (8 warps of 4)

template <int FAM, int BITS>
__global__ void __launch_bounds__(256) k_rebuild(LayerView L, const __grid_constant__ Rebuild R, uint16_t *dst) {
  constexpr int WL = plane_lo(BITS), WH = plane_hi(BITS);
  const int lane = threadIdx.x & 31, part = lane & 7;
  asm volatile("griddepcontrol.launch_dependents;");  // (the attention, which waits for this grid's end)
  if ((int)blockIdx.x >= R.blocks) {
    const int64_t at = (int64_t)((int)blockIdx.x - R.blocks) * 256 + threadIdx.x;
    if (blockIdx.y == 0 && at < R.nq) R.q16[at] = bf16x8_to_ring(R.q[at], 1);
    return;
  }
  int i = 0;
  while (i + 1 < R.n && R.s[i + 1].block0 <= (int)blockIdx.x) ++i;
  const int per = (R.s[i].n + RT - 1) / RT, local = blockIdx.x - R.s[i].block0;
  const int head = local / per, p = local % per * RT + (threadIdx.x >> 5) * 4 + (lane >> 3);
  const int seq = R.s[i].seq, which = R.which == 2 ? (int)blockIdx.y : R.which;
  const bool on = p < R.s[i].n;
  float v[16];  // channel 4 part + 32 j + k at 4 j + k
  if (!on || p >= R.s[i].Q) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      uint2 w = make_uint2(0u, 0u);
      if (on) w = *reinterpret_cast<const uint2 *>(ring_row(L, seq, head, which, p) + 32 * j + 4 * part);
      const float2 a = ring2f(w.x, L.tail_f16), b = ring2f(w.y, L.tail_f16);
      v[4 * j] = a.x, v[4 * j + 1] = a.y, v[4 * j + 2] = b.x, v[4 * j + 3] = b.y;
    }
  } else {
    const SubLayout lay = sub_layout(FAM, BITS);
    const uint8_t *sub = subpage_ptr(L, seq, p / GROUP, head, which);
    const int tip = p % GROUP;
    const uint2 d2 = *reinterpret_cast<const uint2 *>(sub + lay.d + 8 * tip);
    const float2 d01 = __half22float2(*reinterpret_cast<const __half2 *>(&d2.x)),
                 d23 = __half22float2(*reinterpret_cast<const __half2 *>(&d2.y));
    const float d[4] = {d01.x, d01.y, d23.x, d23.y};
    float m[4] = {0.f, 0.f, 0.f, 0.f}, t = 1.f;
    if (FAM == FAM_ASYM) {
      const uint2 m2 = *reinterpret_cast<const uint2 *>(sub + lay.m + 8 * tip);
      const float2 m01 = __half22float2(*reinterpret_cast<const __half2 *>(&m2.x)),
                   m23 = __half22float2(*reinterpret_cast<const __half2 *>(&m2.y));
      m[0] = m01.x, m[1] = m01.y, m[2] = m23.x, m[3] = m23.y;
    }
    if (FAM == FAM_KVARN) t = __half2float(reinterpret_cast<const __half *>(sub + lay.t)[tip]);
    uint32_t f[16];
    if (which == 0) {
      // channels 32 j + 4 part + k: byte k of word (part / F, j) of each plane, field part % F
      constexpr int FL = 8 / WL, FH = WH ? 8 / (WH ? WH : 1) : 1;
      const uint8_t *tok = sub + tip * 16 * BITS;
      const uint4 lo = *reinterpret_cast<const uint4 *>(tok + 16 * (part / FL));
      uint4 hi = make_uint4(0u, 0u, 0u, 0u);
      if (WH) hi = *reinterpret_cast<const uint4 *>(tok + 16 * WL + 16 * (part / FH));
      const uint32_t wl[4] = {lo.x, lo.y, lo.z, lo.w}, wh[4] = {hi.x, hi.y, hi.z, hi.w};
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          uint32_t x = (wl[j] >> (8 * k + (part % FL) * WL)) & ((1u << WL) - 1u);
          if (WH) x |= ((wh[j] >> (8 * k + (part % FH) * WH)) & ((1u << WH) - 1u)) << WL;
          f[4 * j + k] = x;
        }
    } else {
      // channel e = 4 part + k of block j: byte (token of the quad) of word e / F, field e % F
      const uint8_t *quad = sub + (tip >> 2) * 64 * BITS;
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int k = 0; k < 4; ++k) f[4 * j + k] = v_field<BITS>(quad, tip & 3, 32 * j + 4 * part + k);
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      float c[4] = {1.f, 1.f, 1.f, 1.f};
      if (FAM == FAM_KVARN) {
        const uint2 c2 = *reinterpret_cast<const uint2 *>(sub + lay.c + 2 * (32 * j + 4 * part));
        const float2 c01 = __half22float2(*reinterpret_cast<const __half2 *>(&c2.x)),
                     c23 = __half22float2(*reinterpret_cast<const __half2 *>(&c2.y));
        c[0] = c01.x, c[1] = c01.y, c[2] = c23.x, c[3] = c23.y;
      }
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        float x = (float)code_value<FAM, BITS>(f[4 * j + k]) * d[j];
        if (FAM == FAM_ASYM) x += m[j];
        if (FAM == FAM_KVARN) x = x * t * c[k];
        v[4 * j + k] = x;
      }
    }
  }
  if (FAM == FAM_KVARN) {
    // H.x.kappa of the quantized rows: stages 1 and 2 inside a word, 4 .. 16 over the eight lanes, 32
    // and 64 over the blocks.  (Tail rows of a warp take part in the exchange and keep their own.)
    float y[16];
#pragma unroll
    for (int q = 0; q < 16; ++q) y[q] = v[q];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      float *z = y + 4 * j;
      const float a = z[0] + z[1], b = z[0] - z[1], c = z[2] + z[3], d = z[2] - z[3];
      z[0] = a + c, z[2] = a - c, z[1] = b + d, z[3] = b - d;
    }
#pragma unroll
    for (int o = 1; o <= 4; o <<= 1) {
#pragma unroll
      for (int q = 0; q < 16; ++q) {
        const float other = __shfl_xor_sync(FULL, y[q], o);
        y[q] = (lane & o) ? other - y[q] : y[q] + other;
      }
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float a = y[k] + y[4 + k], b = y[k] - y[4 + k], c = y[8 + k] + y[12 + k], d = y[8 + k] - y[12 + k];
      y[k] = a + c, y[8 + k] = a - c, y[4 + k] = b + d, y[12 + k] = b - d;
    }
    if (p < R.s[i].Q) {
#pragma unroll
      for (int q = 0; q < 16; ++q) v[q] = y[q] * kKappa();
    }
  }
  if (!on) return;
  uint16_t *row = dst + ((((int64_t)(R.first + i) * L.hkv + head) * 3 + 2 * which) * R.cap + p) * D + 4 * part;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const __half2 h[2] = {__floats2half2_rn(v[4 * j], v[4 * j + 1]), __floats2half2_rn(v[4 * j + 2], v[4 * j + 3])};
    *reinterpret_cast<uint2 *>(row + 32 * j) = *reinterpret_cast<const uint2 *>(h);
    if (which == 0) {
      const float2 a = __half22float2(h[0]), b = __half22float2(h[1]);
      const __half2 q[2] = {__floats2half2_rn(v[4 * j] - a.x, v[4 * j + 1] - a.y),
                            __floats2half2_rn(v[4 * j + 2] - b.x, v[4 * j + 3] - b.y)};
      *reinterpret_cast<uint2 *>(row + R.cap * D + 32 * j) = *reinterpret_cast<const uint2 *>(q);
    }
  }
}

cudaError_t rebuild(int fam, int bits, const LayerView &L, const Rebuild &R, unsigned blocks, uint16_t *dst,
                    cudaStream_t st) {
#define KVQ_RB(F, B) \
  if (fam == F && bits == B) { k_rebuild<F, B><<<dim3(blocks, R.which == 2 ? 2 : 1), 256, 0, st>>>(L, R, dst); return cudaGetLastError(); }
  KVQ_RB(FAM_SYM, 2) KVQ_RB(FAM_SYM, 3) KVQ_RB(FAM_SYM, 4) KVQ_RB(FAM_SYM, 5) KVQ_RB(FAM_SYM, 6) KVQ_RB(FAM_SYM, 8)
  KVQ_RB(FAM_ASYM, 2) KVQ_RB(FAM_ASYM, 3) KVQ_RB(FAM_ASYM, 4) KVQ_RB(FAM_ASYM, 5) KVQ_RB(FAM_ASYM, 6)
  KVQ_RB(FAM_KVARN, 2) KVQ_RB(FAM_KVARN, 3) KVQ_RB(FAM_KVARN, 4) KVQ_RB(FAM_KVARN, 5) KVQ_RB(FAM_KVARN, 6)
  KVQ_RB(FAM_KVARN, 8)
#undef KVQ_RB
  return cudaErrorInvalidValue;
}

// ---- host side ----------------------------------------------------------------------------------

constexpr size_t align256(size_t x) { return (x + 255) / 256 * 256; }

// What a call covers: its entries and the sequences to rebuild.
struct Plan {
  std::vector<BEntry> e;
  std::vector<int> slot_seq;  // quantized cache: the sequence behind each rebuilt slot
  int64_t cap = 0;            // rows per rebuilt stream
  int64_t rows = 0;           // query tokens in all
  size_t rebuilt_bytes = 0, part_bytes = 0, q16_bytes = 0, bytes = 0;
};

// Blocks and key splits of up to MAXE entries: without splits when there is a block for every SM, or
// no context is longer than four key tiles (one row over 512 tokens: 12.4 us for about 10.4, but the
// host issues one launch less, 4 to 5 us); otherwise the fewest key tiles per CTA that one wave holds, down to one: the join, set
// up behind the attention, costs less than a tile (one row over 1024 / 2048 / 4096 tokens: 10.3 / 10.3 /
// 12.4 us with splits of one tile and more, 13.1 / 13.9 / 14.3 us with at least four).
void plan_attn(BEntry *e, int ne, int hkv, int G, int sms, int64_t *records) {
  const int TB = BT / G;
  int64_t blocks = 0, most = 1;
  for (int i = 0; i < ne; ++i) {
    e[i].nblk = (int)(((int64_t)e[i].nq + 2 * TB - 1) / (2 * TB));
    blocks += (int64_t)e[i].nblk * hkv;
    if (e[i].nblk) most = std::max(most, (e[i].n + BT - 1) / BT);
  }
  auto ctas = [&](int64_t cps) {
    int64_t n = 0;
    for (int i = 0; i < ne; ++i) n += e[i].nblk * (int64_t)hkv * std::max<int64_t>(1, ((e[i].n + BT - 1) / BT + cps - 1) / cps);
    return n;
  };
  int64_t cps = most;
  if (blocks < sms && most > 4) {
    int64_t lo = (most + MAXSPL - 1) / MAXSPL, hi = std::max(most, lo);
    while (lo < hi) {
      const int64_t mid = (lo + hi) / 2;
      if (ctas(mid) <= sms) hi = mid; else lo = mid + 1;
    }
    cps = lo;
  }
  for (int i = 0; i < ne; ++i) {
    const int64_t kt = (e[i].n + BT - 1) / BT;
    e[i].nsplit = (int)std::max<int64_t>(1, (kt + cps - 1) / cps);
    // as even as the count allows
    e[i].cps = (int)std::max<int64_t>(1, (kt + e[i].nsplit - 1) / e[i].nsplit);
    if (e[i].nsplit > 1) {
      e[i].part0 = *records;
      *records += (int64_t)e[i].nq * hkv * G * e[i].nsplit;
    }
  }
}

// Groups of key pairs and splits of the query tiles.  Up to three query tiles: they stay in shared
// memory, and one wave of CTAs streams the keys.  More: items of about a sixth of an SM's share, so
// that the causal ones even out (4k prompt: a third 156 us, a fifth 150, an eighth 151, a twelfth 162).
void plan_mass(BEntry *e, int ne, int hkv, int G, int sms, int64_t *floats) {
  const int TB = BT / G;
  int64_t units = 0, most = 1;
  bool heavy = false;
  for (int i = 0; i < ne; ++i) {
    const int64_t np = (e[i].n + 2 * BT - 1) / (2 * BT), qt = ((int64_t)e[i].nq + TB - 1) / TB;
    units += hkv * np * std::max<int64_t>(1, qt);
    most = std::max(most, np);
    heavy |= qt > NQS;
  }
  const int64_t target = std::min<int64_t>(64, std::max<int64_t>(8, units / (6 * sms)));
  int64_t lo = 1, hi = most;
  while (lo < hi) {
    const int64_t mid = (lo + hi) / 2;
    int64_t n = 0;
    for (int i = 0; i < ne; ++i) n += hkv * (((e[i].n + 2 * BT - 1) / (2 * BT) + mid - 1) / mid);
    if (n <= sms) hi = mid; else lo = mid + 1;
  }
  for (int i = 0; i < ne; ++i) {
    const int64_t np = (e[i].n + 2 * BT - 1) / (2 * BT), qt = std::max<int64_t>(1, ((int64_t)e[i].nq + TB - 1) / TB);
    e[i].mtb = (int)std::max<int64_t>(1, (e[i].nq + qt - 1) / qt);
    e[i].mqs = heavy ? (int)((qt + target - 1) / target) : 1;
    e[i].mqc = (int)((qt + e[i].mqs - 1) / e[i].mqs);
    e[i].mpairs = (int)(heavy ? std::max<int64_t>(1, std::min(np, target / qt)) : lo);
    e[i].mgroup = (int)((np + e[i].mpairs - 1) / e[i].mpairs);
    if (e[i].mqs > 1) {
      e[i].mpart0 = *floats;
      *floats += (int64_t)e[i].mqs * hkv * ((e[i].n + 3) & ~3ll);
    }
  }
}

int make_plan(const kvq_cache *c, int layer, int n_seqs, const int32_t *seq_ids, const int32_t *n_q, int n_q_heads,
              int causal, Plan *P) {
  if (!c || layer < 0 || layer >= c->p.n_layers || n_seqs < 0 || n_q_heads < 1) return KVQ_E_INVAL;
  if (n_q_heads % c->p.n_kv_heads) return KVQ_E_INVAL;
  const int G = n_q_heads / c->p.n_kv_heads, hkv = c->p.n_kv_heads;
  if (G > MAX_G) return KVQ_E_UNSUPPORTED;
  if (n_seqs > 0 && (!seq_ids || !n_q)) return KVQ_E_INVAL;
  const bool quant = c->fam_k != FAM_BF16;
  std::vector<int> slot(quant ? c->p.n_seqs : 0, -1);
  P->e.reserve(n_seqs);
  for (int i = 0; i < n_seqs; ++i) {
    const int s = seq_ids[i];
    if (s < 0 || s >= c->p.n_seqs || n_q[i] < 0) return KVQ_E_INVAL;
    const int64_t n = c->len[(size_t)layer * c->p.n_seqs + s];
    if (n > INT32_MAX - 256) return KVQ_E_UNSUPPORTED;
    if (causal && n_q[i] > n) return KVQ_E_INVAL;
    BEntry e{};
    e.slot = s;
    e.nq = n_q[i];
    e.out = i;
    e.n = n;
    e.q0 = P->rows;
    P->rows += n_q[i];
    if (quant) {
      if (slot[s] < 0 && n > 0) {
        slot[s] = (int)P->slot_seq.size();
        P->slot_seq.push_back(s);
        P->cap = std::max(P->cap, n);
      }
      e.slot = std::max(slot[s], 0);
    }
    P->e.push_back(e);
  }
  if (P->rows > INT32_MAX) return KVQ_E_UNSUPPORTED;
  // the longest first: their CTAs are the ones to start early
  std::stable_sort(P->e.begin(), P->e.end(), [](const BEntry &a, const BEntry &b) { return a.n > b.n; });
  P->rebuilt_bytes = align256((size_t)P->slot_seq.size() * hkv * 3 * P->cap * (2 * D));
  for (size_t base = 0; base < P->e.size(); base += MAXE) {
    int64_t records = 0, floats = 0;
    const int ne = (int)std::min<size_t>(MAXE, P->e.size() - base);
    plan_attn(&P->e[base], ne, hkv, G, c->num_sms, &records);
    plan_mass(&P->e[base], ne, hkv, G, c->num_sms, &floats);
    P->part_bytes = std::max({P->part_bytes, align256(sizeof(float) * PREC * (size_t)records),
                              align256(sizeof(float) * (size_t)floats)});
  }
  if (quant && !c->p.tail_f16) P->q16_bytes = align256((size_t)P->rows * n_q_heads * 2 * D);
  P->bytes = P->rebuilt_bytes + P->part_bytes + P->q16_bytes;
  return KVQ_OK;
}

// Where a call's F16 queries go.
uint4 *q16_rows(const Plan &P, void *workspace) {
  return reinterpret_cast<uint4 *>(static_cast<uint8_t *>(workspace) + P.rebuilt_bytes + P.part_bytes);
}

// Rebuilds what a quantized cache needs and names the source of the rows.
// Queries to convert go along with the first launch (a launch of their own costs the host 4 us); without a
// sequence to rebuild nothing reads them.
int make_source(const kvq_cache *c, int layer, const Plan &P, bool values, const void *q, int n_q_heads,
                void *workspace, cudaStream_t st, Source *s) {
  const LayerView L = layer_view(c, layer);
  if (c->fam_k == FAM_BF16) {
    *s = Source{reinterpret_cast<const uint16_t *>(L.ring), L.ring_cap, c->p.n_seqs, L.tail_f16, 2};
    return KVQ_OK;
  }
  uint16_t *dst = static_cast<uint16_t *>(workspace);
  *s = Source{dst, std::max<int64_t>(P.cap, 1), std::max(1, (int)P.slot_seq.size()), 1, 3};
  for (size_t base = 0; base < P.slot_seq.size(); base += MAXR) {
    Rebuild R{};
    R.n = (int)std::min<size_t>(MAXR, P.slot_seq.size() - base);
    R.cap = P.cap;
    R.first = (int)base;
    int64_t blocks = 0;
    for (int i = 0; i < R.n; ++i) {
      const int seq = P.slot_seq[base + i];
      const int64_t n = c->len[(size_t)layer * c->p.n_seqs + seq];
      R.s[i] = {seq, (int32_t)n, (int32_t)quantized_len(c, n), (int32_t)blocks};
      blocks += (n + RT - 1) / RT * c->p.n_kv_heads;
      if (blocks > INT32_MAX) return KVQ_E_UNSUPPORTED;
    }
    R.blocks = (int32_t)blocks;
    if (base == 0 && P.q16_bytes) {
      R.q = static_cast<const uint4 *>(q);
      R.q16 = q16_rows(P, workspace);
      R.nq = P.rows * n_q_heads * (D / 8);
    }
    const bool both = values && c->p.type_k == c->p.type_v;
    for (int which = 0; which < (values && !both ? 2 : 1); ++which) {
      R.which = both ? 2 : which;
      const int64_t grid = blocks + (R.nq + 255) / 256;
      if (grid > INT32_MAX) return KVQ_E_UNSUPPORTED;
      if (rebuild(which ? c->fam_v : c->fam_k, which ? c->bits_v : c->bits_k, L, R, (unsigned)grid, dst, st) !=
          cudaSuccess)
        return KVQ_E_CUDA;
      note_launches(1);
      R.nq = 0;
    }
  }
  return KVQ_OK;
}

// cuTensorMapEncodeTiled, looked up in the driver once (the library links no driver stub)
typedef CUresult (*EncodeFn)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                             const cuuint64_t *, const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave,
                             CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
EncodeFn encoder() {
  static std::atomic<EncodeFn> fn{nullptr};
  EncodeFn f = fn.load(std::memory_order_acquire);
  if (!f) {
    void *p = nullptr;
    cudaDriverEntryPointQueryResult r;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &r) != cudaSuccess ||
        r != cudaDriverEntryPointSuccess)
      return nullptr;
    f = reinterpret_cast<EncodeFn>(p);
    fn.store(f, std::memory_order_release);
  }
  return f;
}

// rows of 128 16-bit channels, boxes of 64 channels x 128 rows of one stream
int map_rows(const Source &s, int hkv, CUtensorMap *map) {
  const EncodeFn f = encoder();
  if (!f) return KVQ_E_CUDA;
  const cuuint64_t dims[3] = {D, (cuuint64_t)s.cap, (cuuint64_t)s.slots * hkv * s.sides};
  const cuuint64_t strides[2] = {2 * D, (cuuint64_t)s.cap * 2 * D};
  const cuuint32_t box[3] = {64, BT, 1}, one[3] = {1, 1, 1};
  return f(map, s.f16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3,
           const_cast<uint16_t *>(s.base), dims, strides, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
           CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
           CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS
             ? KVQ_OK
             : KVQ_E_CUDA;
}

// query rows as [token][KV head][G][128], boxes of 64 channels x the G heads x as many tokens as fill a tile
int map_queries(const void *q, int f16, int hkv, int G, int64_t rows, CUtensorMap *map) {
  const EncodeFn f = encoder();
  if (!f) return KVQ_E_CUDA;
  const cuuint64_t dims[4] = {D, (cuuint64_t)G, (cuuint64_t)hkv, (cuuint64_t)rows};
  const cuuint64_t strides[3] = {2 * D, (cuuint64_t)G * 2 * D, (cuuint64_t)hkv * G * 2 * D};
  const cuuint32_t box[4] = {64, (cuuint32_t)G, 1, (cuuint32_t)(BT / G)}, one[4] = {1, 1, 1, 1};
  return f(map, f16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void *>(q),
           dims, strides, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
           CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS
             ? KVQ_OK
             : KVQ_E_CUDA;
}

// The query rows as the kernels read them: the converted ones where a BF16 tail meets F16 products.
int make_queries(const Plan &P, const void *q, int f16, int hkv, int n_q_heads, void *workspace, CUtensorMap *map) {
  return map_queries(P.q16_bytes ? q16_rows(P, workspace) : q, f16, hkv, n_q_heads / hkv, P.rows, map);
}

// The dynamic shared memory of a kernel, allowed once per device.
template <typename K>
bool allow_smem(K kernel, int bytes, std::atomic<uint64_t> &done) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return false;
  const uint64_t bit = 1ull << (dev & 63);
  if (dev < 64 && (done.load(std::memory_order_relaxed) & bit)) return true;
  if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) != cudaSuccess) return false;
  if (dev < 64) done.fetch_or(bit, std::memory_order_relaxed);
  return true;
}

// Launches a kernel that waits itself (griddepcontrol.wait) for the one in front of it.
template <typename... P, typename... Q>
bool launch_behind(void (*kernel)(P...), unsigned grid, unsigned block, size_t smem, cudaStream_t st,
                   const Q &...args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(block);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute la[1];
  la[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  la[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = la;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...) == cudaSuccess;
}

bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

template <bool F16, bool LO, Rows ROWS>
int run_attn(const CUtensorMap &map, const CUtensorMap &qmap, const BArgs &A, unsigned ctas, cudaStream_t st) {
  static std::atomic<uint64_t> done{0};
  if (!allow_smem(k_attn<F16, LO, ROWS>, ATTN_SMEM, done)) return KVQ_E_CUDA;
  if (LO) {  // set up behind the rebuild (64 rows over 4096 q8_0 tokens: 62.8 -> 59.4 us)
    if (!launch_behind(k_attn<F16, LO, ROWS>, ctas, NT, ATTN_SMEM, st, map, qmap, A)) return KVQ_E_CUDA;
  } else {
    k_attn<F16, LO, ROWS><<<ctas, NT, ATTN_SMEM, st>>>(map, qmap, A);
    if (cudaGetLastError() != cudaSuccess) return KVQ_E_CUDA;
  }
  note_launches(1);
  return KVQ_OK;
}

// by whether some entries have no more than one tile of query rows, and some more
template <bool F16, bool LO>
auto pick_attn(bool one, bool more) {
  return !more ? run_attn<F16, LO, ONE> : (one ? run_attn<F16, LO, ANY> : run_attn<F16, LO, MORE>);
}

template <bool F16>
int run_mass(const CUtensorMap &kmap, const CUtensorMap &qmap, const BArgs &A, unsigned ctas, cudaStream_t st) {
  static std::atomic<uint64_t> done{0};
  if (!allow_smem(k_mass<F16>, MASS_SMEM, done)) return KVQ_E_CUDA;
  k_mass<F16><<<ctas, NT, MASS_SMEM, st>>>(kmap, qmap, A);
  if (cudaGetLastError() != cudaSuccess) return KVQ_E_CUDA;
  note_launches(1);
  return KVQ_OK;
}

}  // namespace

extern "C" int kvq_batch_workspace_bytes(const kvq_cache *c, int32_t layer, int32_t n_seqs, const int32_t *seq_ids,
                                         const int32_t *n_q, int32_t n_q_heads, size_t *bytes) try {
  if (!bytes) return KVQ_E_INVAL;
  Plan P;
  if (const int rc = make_plan(c, layer, n_seqs, seq_ids, n_q, n_q_heads, 0, &P)) return rc;
  *bytes = P.bytes;
  return KVQ_OK;
} catch (...) {
  return KVQ_E_INVAL;  // host memory for the call's lists ran out
}

extern "C" int kvq_batch_attn(kvq_cache *c, int32_t layer, int32_t n_seqs, const int32_t *seq_ids,
                              const int32_t *n_q, int32_t n_q_heads, int32_t causal, const void *q,
                              float softmax_scale, void *out, float *lse, void *workspace, size_t ws_bytes,
                              kvq_stream_t stream) try {
  if (causal != 0 && causal != 1) return KVQ_E_INVAL;
  Plan P;
  if (const int rc = make_plan(c, layer, n_seqs, seq_ids, n_q, n_q_heads, causal, &P)) return rc;
  if (P.rows == 0) return KVQ_OK;
  if (!q || !out || (!workspace && P.bytes > 0)) return KVQ_E_INVAL;
  if (!aligned16(q) || !aligned16(out) || !aligned16(lse) || !aligned16(workspace)) return KVQ_E_ALIGN;
  const uint64_t row_bytes = (uint64_t)P.rows * n_q_heads * D * 2;
  const uint64_t lse_bytes = (uint64_t)P.rows * n_q_heads * sizeof(float);
  if (overlap(q, row_bytes, out, row_bytes) || overlap(lse, lse_bytes, q, row_bytes) ||
      overlap(lse, lse_bytes, out, row_bytes))
    return KVQ_E_INVAL;
  if (ws_bytes < P.bytes) return KVQ_E_SIZE;
  if (const int rc = check_device(c)) return rc;
  const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  BArgs A{};
  if (const int rc = make_source(c, layer, P, true, q, n_q_heads, workspace, st, &A.src)) return rc;
  CUtensorMap map, qmap;
  if (const int rc = map_rows(A.src, c->p.n_kv_heads, &map)) return rc;
  if (const int rc = make_queries(P, q, A.src.f16, c->p.n_kv_heads, n_q_heads, workspace, &qmap)) return rc;
  A.hkv = c->p.n_kv_heads;
  A.G = n_q_heads / c->p.n_kv_heads;
  A.causal = causal;
  A.io_f16 = c->p.tail_f16;
  A.qscale = (softmax_scale > 0.f ? softmax_scale : 1.0f / sqrtf((float)D)) * LOG2E;
  A.out = static_cast<uint16_t *>(out);
  A.lse = lse;
  A.part = reinterpret_cast<float *>(static_cast<uint8_t *>(workspace) + P.rebuilt_bytes);
  A.status = reinterpret_cast<int32_t *>(c->base + c->off_status);
  for (size_t base = 0; base < P.e.size(); base += MAXE) {
    const int ne = (int)std::min<size_t>(MAXE, P.e.size() - base);
    int64_t ctas = 0, joins = 0;
    bool one = false, more = false;
    A.ne = 0;
    for (int i = 0; i < ne; ++i) {
      BEntry e = P.e[base + i];
      if (e.nq == 0) continue;
      (e.nq <= BT / A.G ? one : more) = true;
      e.cta0 = (int)ctas;
      ctas += (int64_t)e.nblk * A.hkv * e.nsplit;
      if (e.nsplit > 1) joins += (int64_t)e.nq * n_q_heads;
      A.e[A.ne++] = e;
    }
    if (ctas == 0) continue;
    if (ctas > INT32_MAX) return KVQ_E_UNSUPPORTED;
    const auto run = A.src.sides == 3 ? pick_attn<true, true>(one, more)
                                      : (A.src.f16 ? pick_attn<true, false>(one, more) : pick_attn<false, false>(one, more));
    if (const int rc = run(map, qmap, A, (unsigned)ctas, st)) return rc;
    if (joins == 0) continue;
    if (joins > INT32_MAX) return KVQ_E_UNSUPPORTED;
    if (!launch_behind(k_attn_join, (unsigned)joins, D, 0, st, A)) return KVQ_E_CUDA;
    note_launches(1);
  }
  return KVQ_OK;
} catch (...) {
  return KVQ_E_INVAL;
}

extern "C" int kvq_attn_mass(kvq_cache *c, int32_t layer, int32_t n_seqs, const int32_t *seq_ids, const int32_t *n_q,
                             int32_t n_q_heads, int32_t causal, const void *q, float softmax_scale, const float *lse,
                             float decay, const float *mass_in, float *mass_out, int64_t mass_ld, void *workspace,
                             size_t ws_bytes, kvq_stream_t stream) try {
  if (causal != 0 && causal != 1) return KVQ_E_INVAL;
  if (!(decay >= 0.f && decay <= 1.f)) return KVQ_E_INVAL;
  Plan P;
  if (const int rc = make_plan(c, layer, n_seqs, seq_ids, n_q, n_q_heads, causal, &P)) return rc;
  int64_t most = 0;
  for (const BEntry &e : P.e) most = std::max(most, e.n);
  if (most == 0) return KVQ_OK;
  if (!mass_out || (decay != 0.f && !mass_in) || (P.rows > 0 && (!q || !lse)) || (!workspace && P.bytes > 0))
    return KVQ_E_INVAL;
  const int64_t mass_rows = (int64_t)n_seqs * c->p.n_kv_heads;
  if (mass_ld < most || mass_ld > INT64_MAX / 8 / mass_rows) return KVQ_E_INVAL;
  const uint64_t mass_bytes = (uint64_t)(mass_rows * mass_ld) * sizeof(float);
  if (decay != 0.f && mass_in != mass_out && overlap(mass_in, mass_bytes, mass_out, mass_bytes)) return KVQ_E_INVAL;
  const uint64_t row_values = (uint64_t)P.rows * n_q_heads;
  if (overlap(mass_out, mass_bytes, lse, row_values * sizeof(float)) || overlap(mass_out, mass_bytes, q, row_values * D * 2))
    return KVQ_E_INVAL;
  if (!aligned16(q) || !aligned16(lse) || !aligned16(mass_in) || !aligned16(mass_out) || !aligned16(workspace))
    return KVQ_E_ALIGN;
  if (ws_bytes < P.bytes) return KVQ_E_SIZE;
  if (const int rc = check_device(c)) return rc;
  const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  BArgs A{};
  if (const int rc = make_source(c, layer, P, false, q, n_q_heads, workspace, st, &A.src)) return rc;
  A.hkv = c->p.n_kv_heads;
  A.G = n_q_heads / c->p.n_kv_heads;
  A.causal = causal;
  A.io_f16 = c->p.tail_f16;
  A.qscale = (softmax_scale > 0.f ? softmax_scale : 1.0f / sqrtf((float)D)) * LOG2E;
  A.lse = const_cast<float *>(lse);
  A.mass_in = mass_in;
  A.mass_out = mass_out;
  A.mass_ld = mass_ld;
  A.decay = decay;
  A.part = reinterpret_cast<float *>(static_cast<uint8_t *>(workspace) + P.rebuilt_bytes);
  A.status = reinterpret_cast<int32_t *>(c->base + c->off_status);
  CUtensorMap kmap, qmap{};
  if (const int rc = map_rows(A.src, A.hkv, &kmap)) return rc;
  if (P.rows > 0)
    if (const int rc = make_queries(P, q, A.src.f16, A.hkv, n_q_heads, workspace, &qmap)) return rc;
  for (size_t base = 0; base < P.e.size(); base += MAXE) {
    const int ne = (int)std::min<size_t>(MAXE, P.e.size() - base);
    int64_t ctas = 0, joins = 0;
    A.ne = 0;
    for (int i = 0; i < ne; ++i) {
      BEntry e = P.e[base + i];
      if (e.n == 0) continue;
      e.cta0 = (int)ctas;
      ctas += (int64_t)e.mgroup * A.hkv * e.mqs;
      if (e.mqs > 1) joins += e.n * A.hkv;
      A.e[A.ne++] = e;
    }
    if (ctas == 0) continue;
    if (ctas > INT32_MAX) return KVQ_E_UNSUPPORTED;
    if (const int rc = A.src.f16 ? run_mass<true>(kmap, qmap, A, (unsigned)ctas, st)
                                 : run_mass<false>(kmap, qmap, A, (unsigned)ctas, st))
      return rc;
    if (joins == 0) continue;
    if (!launch_behind(k_mass_join, (unsigned)((joins + 255) / 256), 256, 0, st, A, joins)) return KVQ_E_CUDA;
    note_launches(1);
  }
  return KVQ_OK;
} catch (...) {
  return KVQ_E_INVAL;
}
