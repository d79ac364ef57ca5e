// kvq_batch.cu - attention of many query rows over cached sequences (cross attention, prefill of
// ragged batches), and the attention weight each cached token receives from them.
//
// x = scale q.k over the tokens a row sees; lse = log sum exp x; out = sum exp(x - lse) v;
// mass[t] = sum over rows exp(x[t] - lse).
#include <cuda_runtime.h>
#include <math.h>

#include <algorithm>

#include "kvq_codes.cuh"
#include "kvq_internal.h"

using namespace kvq;

namespace {

constexpr unsigned FULL = 0xffffffffu;
constexpr int MAXE = 64;  // entries per launch
constexpr float LOG2E = 1.4426950408889634f;

// One entry: nq query tokens from row token q0 on, over the first n rows of stream `slot`.
struct BEntry {
  int32_t slot, seq, nq;
  int32_t out;  // position in the call's list (mass rows)
  int64_t n, q0;
};

// 16-bit K and V rows: row t of (slot, head, which) at ((slot * hkv + head) * 2 + which) * cap + t
struct Source {
  const uint16_t *base;
  int64_t cap;
  int32_t f16;  // element type: F16, else BF16
};

struct BArgs {
  int32_t ne, hkv, G, causal, io_f16;
  float qscale;  // softmax scale * log2(e)
  Source src;
  const uint16_t *q;
  uint16_t *out;
  float *lse;
  const float *mass_in;
  float *mass_out;
  int64_t mass_ld;
  float decay;
  BEntry e[MAXE];
};

__device__ __forceinline__ const uint16_t *kv_row(const BArgs &A, int slot, int head, int which, int64_t t) {
  return A.src.base + ((((int64_t)slot * A.hkv + head) * 2 + which) * A.src.cap + t) * D;
}

__device__ __forceinline__ void load4(const uint16_t *p, int f16, float (&x)[4]) {
  const uint2 v = *reinterpret_cast<const uint2 *>(p);
  const float2 a = ring2f(v.x, f16), b = ring2f(v.y, f16);
  x[0] = a.x, x[1] = a.y, x[2] = b.x, x[3] = b.y;
}
__device__ __forceinline__ float dot4(const float (&a)[4], const float (&b)[4]) {
  float s = a[0] * b[0] + a[1] * b[1] + a[2] * b[2] + a[3] * b[3];
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) s += __shfl_xor_sync(FULL, s, o);
  return s;
}

// One warp per (query token, query head).
__global__ void __launch_bounds__(256) k_attn_rows(const __grid_constant__ BArgs A, int64_t items) {
  const int lane = threadIdx.x & 31, hq = A.hkv * A.G;
  int64_t it = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
  if (it >= items) return;
  int ei = 0;
  while (it >= (int64_t)A.e[ei].nq * hq) it -= (int64_t)A.e[ei++].nq * hq;
  const BEntry &e = A.e[ei];
  const int i = (int)(it / hq), h = (int)(it % hq), head = h / A.G;
  const int64_t row = (e.q0 + i) * hq + h;
  const int64_t lim = A.causal ? e.n - e.nq + 1 + i : e.n;
  float q[4], k[4], v[4], o[4] = {0.f, 0.f, 0.f, 0.f}, m = -INFINITY, l = 0.f;
  load4(A.q + row * D + 4 * lane, A.io_f16, q);
  for (int64_t t = 0; t < lim; ++t) {
    load4(kv_row(A, e.slot, head, 0, t) + 4 * lane, A.src.f16, k);
    load4(kv_row(A, e.slot, head, 1, t) + 4 * lane, A.src.f16, v);
    const float x = dot4(q, k) * A.qscale, mn = fmaxf(m, x);
    const float a = exp2f(m - mn), p = exp2f(x - mn);
    m = mn;
    l = l * a + p;
#pragma unroll
    for (int j = 0; j < 4; ++j) o[j] = o[j] * a + p * v[j];
  }
  const float inv = lim > 0 ? 1.f / l : 0.f;
  uint2 w;
  __nv_bfloat162 b[2] = {__floats2bfloat162_rn(o[0] * inv, o[1] * inv), __floats2bfloat162_rn(o[2] * inv, o[3] * inv)};
  __half2 f[2] = {__floats2half2_rn(o[0] * inv, o[1] * inv), __floats2half2_rn(o[2] * inv, o[3] * inv)};
  w = A.io_f16 ? *reinterpret_cast<const uint2 *>(f) : *reinterpret_cast<const uint2 *>(b);
  *reinterpret_cast<uint2 *>(A.out + row * D + 4 * lane) = w;
  if (A.lse && lane == 0) A.lse[row] = lim > 0 ? (m + log2f(l)) / LOG2E : -INFINITY;
}

// One warp per (token, KV head): the sum over the entry's query rows, in their order.
__global__ void __launch_bounds__(256) k_mass_rows(const __grid_constant__ BArgs A, int64_t items) {
  const int lane = threadIdx.x & 31, hq = A.hkv * A.G;
  int64_t it = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
  if (it >= items) return;
  int ei = 0;
  while (it >= A.e[ei].n * A.hkv) it -= A.e[ei++].n * A.hkv;
  const BEntry &e = A.e[ei];
  const int head = (int)(it / e.n);
  const int64_t t = it % e.n;
  float q[4], k[4], sum = 0.f;
  load4(kv_row(A, e.slot, head, 0, t) + 4 * lane, A.src.f16, k);
  const int64_t i0 = A.causal ? max((int64_t)0, t - (e.n - e.nq)) : 0;
  for (int64_t r = i0 * A.G; r < (int64_t)e.nq * A.G; ++r) {
    const int64_t row = (e.q0 + r / A.G) * hq + head * A.G + r % A.G;
    load4(A.q + row * D + 4 * lane, A.io_f16, q);
    const float l = A.lse[row];
    const float x = dot4(q, k) * A.qscale;
    if (l != -INFINITY) sum += exp2f(x - l * LOG2E);
  }
  if (lane == 0) {
    const int64_t at = ((int64_t)e.out * A.hkv + head) * A.mass_ld + t;
    A.mass_out[at] = A.decay != 0.f ? A.decay * A.mass_in[at] + sum : sum;
  }
}

// ---- quantized caches: one side's values rebuilt in the original basis as F16 rows --------------
// One warp per (token, head); lane holds channels 4 lane .. 4 lane + 3.  F16 keeps 11 significant
// bits of a value of at most 8 + 11; the rounding (at most 2^-12 of the value) is the only one
// before the products.
struct Rebuild {
  int32_t seq, slot, which;
  int64_t n, Q;
};

template <int FAM, int BITS>
__global__ void __launch_bounds__(256) k_rebuild(LayerView L, Rebuild R, uint16_t *dst, int64_t cap) {
  const int lane = threadIdx.x & 31;
  const int64_t it = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
  if (it >= R.n * L.hkv) return;
  const int head = (int)(it / R.n);
  const int64_t p = it % R.n;
  float v[4];
  if (p >= R.Q) {
    load4(reinterpret_cast<const uint16_t *>(ring_row(L, R.seq, head, R.which, p)) + 4 * lane, L.tail_f16, v);
  } else {
    const SubLayout lay = sub_layout(FAM, BITS);
    const uint8_t *sub = subpage_ptr(L, R.seq, p / GROUP, head, R.which);
    const int tip = (int)(p % GROUP);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int ch = 4 * lane + e, blk = ch >> 5;
      const uint32_t f = R.which == 0 ? k_field<BITS>(sub + tip * 16 * BITS, ch)
                                      : v_field<BITS>(sub + (tip >> 2) * 64 * BITS, tip & 3, ch);
      float x = (float)code_value<FAM, BITS>(f) * __half2float(reinterpret_cast<const __half *>(sub + lay.d)[tip * 4 + blk]);
      if (FAM == FAM_ASYM) x += __half2float(reinterpret_cast<const __half *>(sub + lay.m)[tip * 4 + blk]);
      if (FAM == FAM_KVARN) {
        x *= __half2float(reinterpret_cast<const __half *>(sub + lay.t)[tip]);
        x *= __half2float(reinterpret_cast<const __half *>(sub + lay.c)[ch]);
      }
      v[e] = x;
    }
    if (FAM == FAM_KVARN) {
      // H.x.kappa: stages 1, 2 inside the lane, 4 .. 64 across lanes
      float a = v[0] + v[1], b = v[0] - v[1], c = v[2] + v[3], d = v[2] - v[3];
      v[0] = a + c, v[2] = a - c, v[1] = b + d, v[3] = b - d;
#pragma unroll
      for (int o = 1; o <= 16; o <<= 1) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float other = __shfl_xor_sync(FULL, v[e], o);
          v[e] = (lane & o) ? other - v[e] : v[e] + other;
        }
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] *= kKappa();
    }
  }
  const __half2 h[2] = {__floats2half2_rn(v[0], v[1]), __floats2half2_rn(v[2], v[3])};
  *reinterpret_cast<uint2 *>(dst + ((((int64_t)R.slot * L.hkv + head) * 2 + R.which) * cap + p) * D + 4 * lane) =
      *reinterpret_cast<const uint2 *>(h);
}

cudaError_t rebuild(int fam, int bits, const LayerView &L, const Rebuild &R, uint16_t *dst, int64_t cap,
                    cudaStream_t st) {
  const unsigned grid = (unsigned)((R.n * L.hkv + 7) / 8);
#define KVQ_RB(F, B) \
  if (fam == F && bits == B) { k_rebuild<F, B><<<grid, 256, 0, st>>>(L, R, dst, cap); return cudaGetLastError(); }
  KVQ_RB(FAM_SYM, 2) KVQ_RB(FAM_SYM, 3) KVQ_RB(FAM_SYM, 4) KVQ_RB(FAM_SYM, 5) KVQ_RB(FAM_SYM, 6) KVQ_RB(FAM_SYM, 8)
  KVQ_RB(FAM_ASYM, 2) KVQ_RB(FAM_ASYM, 3) KVQ_RB(FAM_ASYM, 4) KVQ_RB(FAM_ASYM, 5) KVQ_RB(FAM_ASYM, 6)
  KVQ_RB(FAM_KVARN, 2) KVQ_RB(FAM_KVARN, 3) KVQ_RB(FAM_KVARN, 4) KVQ_RB(FAM_KVARN, 5) KVQ_RB(FAM_KVARN, 6)
  KVQ_RB(FAM_KVARN, 8)
#undef KVQ_RB
  return cudaErrorInvalidValue;
}

// ---- host side ----------------------------------------------------------------------------------

// What a call covers: its entries (those with query tokens), the sequences to rebuild.
struct Plan {
  std::vector<BEntry> e;
  std::vector<int> slot_seq;  // quantized cache: the sequence behind each rebuilt slot
  int64_t cap = 0;            // rows per rebuilt stream
  int64_t rows = 0;           // query tokens in all
  size_t rebuilt_bytes = 0, bytes = 0;
};

int make_plan(const kvq_cache *c, int layer, int n_seqs, const int32_t *seq_ids, const int32_t *n_q, int n_q_heads,
              int causal, Plan *P) {
  if (!c || layer < 0 || layer >= c->p.n_layers || n_seqs < 0 || n_q_heads < 1) return KVQ_E_INVAL;
  if (n_q_heads % c->p.n_kv_heads) return KVQ_E_INVAL;
  if (n_q_heads / c->p.n_kv_heads > MAX_G) return KVQ_E_UNSUPPORTED;
  if (n_seqs > 0 && (!seq_ids || !n_q)) return KVQ_E_INVAL;
  const bool quant = c->fam_k != FAM_BF16;
  std::vector<int> slot(quant ? c->p.n_seqs : 0, -1);
  for (int i = 0; i < n_seqs; ++i) {
    const int s = seq_ids[i];
    if (s < 0 || s >= c->p.n_seqs || n_q[i] < 0) return KVQ_E_INVAL;
    const int64_t n = c->len[(size_t)layer * c->p.n_seqs + s];
    if (n > INT32_MAX - 256) return KVQ_E_UNSUPPORTED;
    if (causal && n_q[i] > n) return KVQ_E_INVAL;
    BEntry e{};
    e.seq = s;
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
  P->rebuilt_bytes = (size_t)P->slot_seq.size() * c->p.n_kv_heads * 2 * P->cap * (2 * D);
  P->bytes = P->rebuilt_bytes;
  return KVQ_OK;
}

// Rebuilds what a quantized cache needs and names the source of the rows.
int make_source(const kvq_cache *c, int layer, const Plan &P, bool values, void *workspace, cudaStream_t st,
                Source *s) {
  const LayerView L = layer_view(c, layer);
  if (c->fam_k == FAM_BF16) {
    *s = Source{reinterpret_cast<const uint16_t *>(L.ring), L.ring_cap, L.tail_f16};
    return KVQ_OK;
  }
  uint16_t *dst = static_cast<uint16_t *>(workspace);
  *s = Source{dst, P.cap, 1};
  for (size_t i = 0; i < P.slot_seq.size(); ++i) {
    const int64_t n = c->len[(size_t)layer * c->p.n_seqs + P.slot_seq[i]];
    for (int which = 0; which < (values ? 2 : 1); ++which) {
      const Rebuild R{P.slot_seq[i], (int)i, which, n, quantized_len(c, n)};
      if (rebuild(which ? c->fam_v : c->fam_k, which ? c->bits_v : c->bits_k, L, R, dst, P.cap, st) != cudaSuccess)
        return KVQ_E_CUDA;
      note_launches(1);
    }
  }
  return KVQ_OK;
}

bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

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
  if (ws_bytes < P.bytes) return KVQ_E_SIZE;
  if (const int rc = check_device(c)) return rc;
  const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  BArgs A{};
  if (const int rc = make_source(c, layer, P, true, workspace, st, &A.src)) return rc;
  A.hkv = c->p.n_kv_heads;
  A.G = n_q_heads / c->p.n_kv_heads;
  A.causal = causal;
  A.io_f16 = c->p.tail_f16;
  A.qscale = (softmax_scale > 0.f ? softmax_scale : 1.0f / sqrtf((float)D)) * LOG2E;
  A.q = static_cast<const uint16_t *>(q);
  A.out = static_cast<uint16_t *>(out);
  A.lse = lse;
  for (size_t base = 0; base < P.e.size(); base += MAXE) {
    A.ne = (int)std::min<size_t>(MAXE, P.e.size() - base);
    int64_t items = 0;
    for (int i = 0; i < A.ne; ++i) {
      A.e[i] = P.e[base + i];
      items += (int64_t)A.e[i].nq * n_q_heads;
    }
    if (items == 0) continue;
    k_attn_rows<<<(unsigned)((items + 7) / 8), 256, 0, st>>>(A, items);
    if (cudaGetLastError() != cudaSuccess) return KVQ_E_CUDA;
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
  if (mass_ld < most) return KVQ_E_INVAL;
  if (!aligned16(q) || !aligned16(lse) || !aligned16(mass_in) || !aligned16(mass_out) || !aligned16(workspace))
    return KVQ_E_ALIGN;
  if (ws_bytes < P.bytes) return KVQ_E_SIZE;
  if (const int rc = check_device(c)) return rc;
  const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  BArgs A{};
  if (const int rc = make_source(c, layer, P, false, workspace, st, &A.src)) return rc;
  A.hkv = c->p.n_kv_heads;
  A.G = n_q_heads / c->p.n_kv_heads;
  A.causal = causal;
  A.io_f16 = c->p.tail_f16;
  A.qscale = (softmax_scale > 0.f ? softmax_scale : 1.0f / sqrtf((float)D)) * LOG2E;
  A.q = static_cast<const uint16_t *>(q);
  A.lse = const_cast<float *>(lse);
  A.mass_in = mass_in;
  A.mass_out = mass_out;
  A.mass_ld = mass_ld;
  A.decay = decay;
  for (size_t base = 0; base < P.e.size(); base += MAXE) {
    A.ne = (int)std::min<size_t>(MAXE, P.e.size() - base);
    int64_t items = 0;
    for (int i = 0; i < A.ne; ++i) {
      A.e[i] = P.e[base + i];
      items += A.e[i].n * A.hkv;
    }
    if (items == 0) continue;
    k_mass_rows<<<(unsigned)((items + 7) / 8), 256, 0, st>>>(A, items);
    if (cudaGetLastError() != cudaSuccess) return KVQ_E_CUDA;
    note_launches(1);
  }
  return KVQ_OK;
} catch (...) {
  return KVQ_E_INVAL;
}
