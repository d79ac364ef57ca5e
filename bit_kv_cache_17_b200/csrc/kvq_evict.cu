// kvq_evict.cu - cuts sequences down to the tokens with the most accumulated attention weight.
//
// Selection: per (sequence, KV head) the first `sink`, the last `recent` and the largest weights in
// between, ties to the lower index.  The weights map to 32-bit keys that order like them; a radix
// select finds the key T of the last token to keep, and a scan in index order emits every key above
// T and the first of those equal to it.  No atomics decide an order: the result is a function of
// the input alone.
// Compaction: the kept rows of K and V are copied to the destination's ring in order (a BF16
// destination), or to the workspace and appended from there (a quantized one).
#include <cuda_runtime.h>

#include <algorithm>

#include "kvq_internal.h"

using namespace kvq;

namespace {

constexpr unsigned FULL = 0xffffffffu;
constexpr int MAXE = 64;   // entries per launch
constexpr int NT = 1024;   // selection threads

struct EvictSeq {
  int32_t src, dst, n, count;
  int64_t row0;  // first staged row (quantized destination)
};

struct EvictArgs {
  int32_t hkv, budget, sink, recent, nseq, entry0;
  int64_t mass_ld, out_ld;
  const float *mass;
  float *mass_out;
  int32_t *kept;
  EvictSeq s[MAXE];
};

// 32-bit keys in the order of the weights: NaN above all, -0 equal to +0
__device__ __forceinline__ uint32_t key_of(float x) {
  uint32_t u = __float_as_uint(x);
  if ((u & 0x7fffffffu) > 0x7f800000u) return 0xffffffffu;
  if (u == 0x80000000u) u = 0u;
  return u ^ ((u >> 31) ? 0xffffffffu : 0x80000000u);
}

// inclusive sums of two 16-bit-packed counts over the block's threads; total in *all
__device__ __forceinline__ uint64_t block_scan(uint64_t v, uint64_t *warp_sums, uint64_t *all) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  uint64_t x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint64_t y = __shfl_up_sync(FULL, x, o);
    if (lane >= o) x += y;
  }
  __syncthreads();
  if (lane == 31) warp_sums[warp] = x;
  __syncthreads();
  uint64_t before = 0, total = 0;
  for (int w = 0; w < NT / 32; ++w) {
    if (w < warp) before += warp_sums[w];
    total += warp_sums[w];
  }
  *all = total;
  return x + before;
}

__global__ void __launch_bounds__(NT) k_select(const __grid_constant__ EvictArgs A) {
  __shared__ uint32_t hist[256];
  __shared__ uint64_t warp_sums[NT / 32];
  __shared__ uint32_t s_prefix, s_need;
  const int e = blockIdx.x / A.hkv, head = blockIdx.x % A.hkv, tid = threadIdx.x;
  const EvictSeq &s = A.s[e];
  const int64_t row = (int64_t)(A.entry0 + e) * A.hkv + head;
  const float *mass = A.mass + row * A.mass_ld;
  int32_t *kept = A.kept + row * A.budget;
  float *out = A.mass_out ? A.mass_out + row * A.out_ld : nullptr;
  // places behind the kept tokens
  for (int i = s.count + tid; i < A.budget; i += NT) kept[i] = -1;
  if (out)
    for (int64_t i = s.count + tid; i < A.out_ld; i += NT) out[i] = 0.f;
  const int lo = min(A.sink, s.n), hi = max(lo, s.n - A.recent);
  const bool cut = s.n > A.budget;
  uint32_t T = 0, need = 0;  // keys above T are kept, and the first `need` equal to it
  if (cut) {
    uint32_t prefix = 0, mask = 0;
    need = (uint32_t)(A.budget - A.sink - A.recent);
    if (need > 0) {
      for (int sh = 24; sh >= 0; sh -= 8) {
        if (tid < 256) hist[tid] = 0;
        __syncthreads();
        for (int i = lo + tid; i < hi; i += NT) {
          const uint32_t k = key_of(mass[i]);
          if ((k & mask) == prefix) atomicAdd(&hist[(k >> sh) & 255u], 1u);
        }
        __syncthreads();
        if (tid == 0) {
          uint32_t left = need;
          int d = 255;
          while (d > 0 && hist[d] < left) left -= hist[d--];
          s_prefix = prefix | ((uint32_t)d << sh);
          s_need = left;
        }
        __syncthreads();
        prefix = s_prefix;
        need = s_need;
        mask |= 255u << sh;
        __syncthreads();
      }
      T = prefix;
    } else {
      T = 0xffffffffu;
    }
  }
  // emit in index order: high half counts the kept, low half those equal to T
  uint64_t base = 0;
  for (int i0 = 0; i0 < s.n; i0 += NT) {
    const int i = i0 + tid;
    bool safe = false, eq = false, above = false;
    if (i < s.n) {
      safe = !cut || i < lo || i >= hi;
      if (!safe) {
        const uint32_t k = key_of(mass[i]);
        above = k > T;
        eq = k == T;
      }
    }
    uint64_t all;
    const uint64_t v = ((uint64_t)(safe || above) << 32) | (uint64_t)eq;
    const uint64_t x = base + block_scan(v, warp_sums, &all) - v;
    const uint32_t eqs = (uint32_t)x;
    const bool take = safe || above || (eq && eqs < need);
    if (take) {
      const uint32_t at = (uint32_t)(x >> 32) + min(eqs, need);
      kept[at] = i;
      if (out) out[at] = mass[i];
    }
    base += all;
  }
}

// One warp per (kept token, head): the K row in lanes 0..15, the V row in lanes 16..31.
// stage_k / stage_v: [row][hkv][128] BF16 for a destination that is appended to; otherwise the rows
// go to the destination's ring.
__global__ void __launch_bounds__(256) k_gather(LayerView S, LayerView T, const __grid_constant__ EvictArgs A,
                                                int64_t items, uint4 *stage_k, uint4 *stage_v) {
  const int lane = threadIdx.x & 31, which = lane >> 4, part = lane & 15;
  int64_t it = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
  if (it >= items) return;
  int e = 0;
  while (it >= (int64_t)A.s[e].count * A.hkv) it -= (int64_t)A.s[e++].count * A.hkv;
  const EvictSeq &s = A.s[e];
  const int head = (int)(it / s.count), i = (int)(it % s.count);
  const int from = A.kept[((int64_t)(A.entry0 + e) * A.hkv + head) * A.budget + i];
  uint4 v = reinterpret_cast<const uint4 *>(ring_row(S, s.src, head, which, from))[part];
  const bool staged = stage_k != nullptr;
  if (staged ? S.tail_f16 : S.tail_f16 != T.tail_f16) {
    if (S.tail_f16) {  // F16 rows hold BF16 inputs rounded to F16: back to BF16 is exact
      uint32_t *w = reinterpret_cast<uint32_t *>(&v);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float2 f = ring2f(w[j], 1);
        const __nv_bfloat162 b = __floats2bfloat162_rn(f.x, f.y);
        w[j] = *reinterpret_cast<const uint32_t *>(&b);
      }
    } else {
      v = bf16x8_to_ring(v, 1);
    }
  }
  if (staged)
    (which ? stage_v : stage_k)[((s.row0 + i) * A.hkv + head) * (D / 8) + part] = v;
  else
    reinterpret_cast<uint4 *>(ring_row(T, s.dst, head, which, i))[part] = v;
}

constexpr size_t align256(size_t x) { return (x + 255) / 256 * 256; }
size_t kept_bytes(const kvq_cache *c, int n_seqs, int budget) {
  return align256(sizeof(int32_t) * (size_t)n_seqs * c->p.n_kv_heads * budget);
}
size_t staged_bytes(const kvq_cache *c, int64_t rows) { return align256((size_t)rows * c->p.n_kv_heads * 2 * D); }

}  // namespace

extern "C" int kvq_evict_workspace_bytes(const kvq_cache *src, const kvq_cache *dst, int32_t n_seqs, int32_t budget,
                                         size_t *bytes) {
  if (!src || !dst || !bytes || n_seqs < 0 || budget < 0) return KVQ_E_INVAL;
  size_t b = kept_bytes(src, n_seqs, budget);
  if (dst->fam_k != FAM_BF16) b += 2 * staged_bytes(src, (int64_t)n_seqs * budget);
  *bytes = b;
  return KVQ_OK;
}

extern "C" int kvq_evict(kvq_cache *src, int32_t src_layer, kvq_cache *dst, int32_t dst_layer, int32_t n_seqs,
                         const int32_t *src_ids, const int32_t *dst_ids, const float *mass, int64_t mass_ld,
                         int32_t budget, int32_t sink, int32_t recent, int32_t *kept, float *mass_out,
                         int64_t mass_out_ld, void *workspace, size_t ws_bytes, kvq_stream_t stream) try {
  if (!src || !dst || n_seqs < 0 || budget < 0 || sink < 0 || recent < 0) return KVQ_E_INVAL;
  if (src_layer < 0 || src_layer >= src->p.n_layers || dst_layer < 0 || dst_layer >= dst->p.n_layers)
    return KVQ_E_INVAL;
  if ((int64_t)sink + recent > budget) return KVQ_E_INVAL;
  if (src->fam_k != FAM_BF16) return KVQ_E_UNSUPPORTED;
  if (src->p.n_kv_heads != dst->p.n_kv_heads) return KVQ_E_UNSUPPORTED;
  if (src->device != dst->device) return KVQ_E_INVAL;
  if (n_seqs == 0) return KVQ_OK;
  if (!src_ids || !dst_ids || !mass || !workspace) return KVQ_E_INVAL;
  if (mass_out && mass_out_ld < budget) return KVQ_E_INVAL;
  std::vector<char> seen(dst->p.n_seqs, 0);
  std::vector<EvictSeq> seqs;
  int64_t rows = 0, most = 0;
  for (int i = 0; i < n_seqs; ++i) {
    const int a = src_ids[i], b = dst_ids[i];
    if (a < 0 || a >= src->p.n_seqs || b < 0 || b >= dst->p.n_seqs || seen[b]) return KVQ_E_INVAL;
    seen[b] = 1;
    const int64_t n = src->len[(size_t)src_layer * src->p.n_seqs + a];
    if (n > INT32_MAX) return KVQ_E_UNSUPPORTED;
    const int64_t count = std::min<int64_t>(n, budget);
    if (count > dst->p.max_ctx) return KVQ_E_CAPACITY;
    seqs.push_back({a, b, (int32_t)n, (int32_t)count, rows});
    rows += count;
    most = std::max(most, n);
  }
  if (src == dst && src_layer == dst_layer)
    for (int i = 0; i < n_seqs; ++i)
      if (seen[src_ids[i]]) return KVQ_E_INVAL;
  if (mass_ld < most) return KVQ_E_INVAL;
  if (((uintptr_t)mass | (uintptr_t)kept | (uintptr_t)mass_out | (uintptr_t)workspace) & 15u) return KVQ_E_ALIGN;
  const bool staged = dst->fam_k != FAM_BF16;
  size_t need;
  if (const int rc = kvq_evict_workspace_bytes(src, dst, n_seqs, budget, &need)) return rc;
  if (ws_bytes < need) return KVQ_E_SIZE;
  if (const int rc = check_device(src)) return rc;

  const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const LayerView S = layer_view(src, src_layer), T = layer_view(dst, dst_layer);
  const int hkv = src->p.n_kv_heads;
  uint8_t *ws = static_cast<uint8_t *>(workspace);
  uint4 *stage_k = nullptr, *stage_v = nullptr;
  if (staged) {
    stage_k = reinterpret_cast<uint4 *>(ws + kept_bytes(src, n_seqs, budget));
    stage_v = stage_k + staged_bytes(src, (int64_t)n_seqs * budget) / sizeof(uint4);
  }
  for (int base = 0; base < n_seqs; base += MAXE) {
    EvictArgs A{};
    A.nseq = std::min(MAXE, n_seqs - base);
    A.entry0 = base;
    A.hkv = hkv;
    A.budget = budget;
    A.sink = sink;
    A.recent = recent;
    A.mass = mass;
    A.mass_ld = mass_ld;
    A.mass_out = mass_out;
    A.out_ld = mass_out_ld;
    A.kept = kept ? kept : reinterpret_cast<int32_t *>(ws);
    int64_t items = 0;
    for (int i = 0; i < A.nseq; ++i) {
      A.s[i] = seqs[base + i];
      items += (int64_t)A.s[i].count * hkv;
    }
    k_select<<<(unsigned)(A.nseq * hkv), NT, 0, st>>>(A);
    if (cudaGetLastError() != cudaSuccess) return KVQ_E_CUDA;
    note_launches(1);
    if (items == 0) continue;
    k_gather<<<(unsigned)((items + 7) / 8), 256, 0, st>>>(S, T, A, items, stage_k, stage_v);
    if (cudaGetLastError() != cudaSuccess) return KVQ_E_CUDA;
    note_launches(1);
  }
  if (staged) {
    std::vector<AppendSeq> app;
    for (const EvictSeq &s : seqs)
      if (s.count > 0) app.push_back({s.dst, s.count, 0, s.row0});
    if (!app.empty())
      if (const int rc = launch_append(dst, dst_layer, app, stage_k, stage_v, st)) return rc;
  }
  for (const EvictSeq &s : seqs) dst->len[(size_t)dst_layer * dst->p.n_seqs + s.dst] = s.count;
  return KVQ_OK;
} catch (...) {
  return KVQ_E_INVAL;  // host memory for the call's lists ran out
}
