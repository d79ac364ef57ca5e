// kvq_evict.cu - cuts sequences down to the tokens with the most accumulated attention weight.
//
// Selection: per (sequence, KV head) the first `sink`, the last `recent` and the largest weights in
// between, ties to the lower index.  The weights map to 32-bit keys that order like them; a radix
// select (digits of 11, 11 and 10 bits) finds the key T of the last token to keep, and a scan in index
// order emits every key above T and the first of those equal to it.  No atomics decide an order: the
// result is a function of the input alone.
// A cluster of up to 8 CTAs takes a row: each keeps the keys of a contiguous segment in shared memory
// (one read of the weights), the histograms and counts are added up through distributed shared memory.
// Bound: instructions and the latency of the five visits to a segment, not the 4 bytes a token
// (128 rows of up to 32 768: 28 us; 8 rows of 2048: 8.5 us).
// Compaction: the kept rows of K and V are copied to the destination's ring in order (a BF16
// destination), or to the workspace and appended from there (a quantized one).  Bound: HBM; a warp has
// eight rows of K and V in flight (one row: 167 us for 16 x 4096 tokens of 8 heads; eight: 95 us, 5.6 TB/s).
#include <cooperative_groups.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>

#include "kvq_internal.h"

using namespace kvq;

namespace {

constexpr unsigned FULL = 0xffffffffu;
constexpr int MAXE = 64;    // entries per launch
constexpr int NT = 512;     // selection threads
constexpr int MAXC = 8;     // CTAs of a cluster
constexpr int SEG = 51200;  // tokens of a segment that shared memory holds (longer ones are read again)

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

constexpr int NWARP = NT / 32, BINS = 2048;

struct SelectShared {
  alignas(16) uint32_t hist[2][BINS];  // alternating: the cluster may still read one while the next is filled
  uint32_t warp_sums[NWARP];
  uint32_t above[NWARP], equal[NWARP];  // of each warp's part of the segment
  uint32_t all_above, all_equal;
  uint32_t digit, need;
};

// CACHED: shared memory holds the segment's keys; otherwise they are made from the weights each time
template <bool CACHED>
__global__ void __launch_bounds__(NT) k_select(const __grid_constant__ EvictArgs A) {
  namespace cg = cooperative_groups;
  extern __shared__ __align__(16) uint32_t keys[];
  __shared__ SelectShared H;
  cg::cluster_group cl = cg::this_cluster();
  const int rank = (int)cl.block_rank(), size = (int)cl.num_blocks();
  asm volatile("griddepcontrol.launch_dependents;");
  const int it = blockIdx.x / size, e = it / A.hkv, head = it % A.hkv;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const EvictSeq &s = A.s[e];
  const int64_t r = (int64_t)(A.entry0 + e) * A.hkv + head;
  int32_t *kept = A.kept + r * A.budget;
  float *out = A.mass_out ? A.mass_out + r * A.out_ld : nullptr;
  // places behind the kept tokens
  for (int i = s.count + rank * NT + tid; i < A.budget; i += size * NT) kept[i] = -1;
  if (out)
    for (int64_t i = s.count + rank * NT + tid; i < A.out_ld; i += size * NT) out[i] = 0.f;
  // this CTA's tokens [i0, i0 + n), those of them that compete [c0, c1)
  const int per = (s.n + size - 1) / size, i0 = min(s.n, rank * per), n = min(s.n - i0, per);
  const bool cut = s.n > A.budget;
  const int lo = min(A.sink, s.n), hi = max(lo, s.n - A.recent);
  const int c0 = min(max(lo - i0, 0), n), c1 = min(max(hi - i0, c0), n);
  const float *mass = A.mass + r * A.mass_ld + i0;
  auto key = [&](int i) { return CACHED ? keys[i] : key_of(mass[i]); };
  for (int b = tid; b < 2 * BINS; b += NT) H.hist[0][b] = 0;  // (both)
  __syncthreads();
  const bool select = cut && A.budget > A.sink + A.recent;  // (uniform over the cluster)
  // one addition for all lanes that hold lane 0's key (many weights may be equal, most often 0)
  auto add = [&](uint32_t *hist, uint32_t k, uint32_t digit, bool in) {
    const uint32_t k0 = __shfl_sync(FULL, k, 0), same = __ballot_sync(FULL, in && k == k0);
    if (in && k != k0) atomicAdd(&hist[digit], 1u);
    if (lane == 0 && same) atomicAdd(&hist[digit], (uint32_t)__popc(same));
  };
#pragma unroll 1
  for (int i = tid; i - tid < n; i += 4 * NT) {
    float x[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) x[u] = i + u * NT < n ? __ldg(mass + i + u * NT) : 0.f;
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int at = i + u * NT;
      const uint32_t k = key_of(x[u]);
      if (CACHED && at < n) keys[at] = k;
      if (select) add(H.hist[0], k, k >> 21, at >= c0 && at < c1);
    }
  }
  uint32_t T = 0xffffffffu, need = 0;  // keys above T are kept, and the first `need` equal to it
  if (select) {
    need = (uint32_t)(A.budget - A.sink - A.recent);
    uint32_t prefix = 0;
#pragma unroll 1
    for (int pass = 0; pass < 3; ++pass) {
      const int sh = pass == 0 ? 21 : (pass == 1 ? 10 : 0), bits = pass == 2 ? 10 : 11;
      uint32_t *hist = H.hist[pass & 1];
      if (pass > 0) {
        const uint32_t want = prefix >> (sh + bits);
#pragma unroll 4
        for (int i = c0 + tid; i < c1; i += NT) {
          const uint32_t k = key(i);
          if (k >> (sh + bits) == want) atomicAdd(&hist[(k >> sh) & ((1u << bits) - 1u)], 1u);
        }
      }
      cl.sync();
      if (pass == 1)  // (the first histogram has been read by all: it takes the last digit)
        for (int b = tid; b < BINS; b += NT) H.hist[0][b] = 0;
      // the cluster's histogram, four digits a thread, largest first, and where `need` falls in it
      uint32_t v[4] = {0, 0, 0, 0};
      const int top = (1 << bits) - 1 - 4 * tid;
      if (top >= 0) {
#pragma unroll
        for (int c = 0; c < MAXC; ++c) {
          if (c >= size) break;
          const uint4 q = *reinterpret_cast<const uint4 *>(cl.map_shared_rank(hist, c) + (top - 3));
          v[0] += q.w, v[1] += q.z, v[2] += q.y, v[3] += q.x;
        }
      }
      const uint32_t sum = v[0] + v[1] + v[2] + v[3];
      uint32_t x = sum;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const uint32_t y = __shfl_up_sync(FULL, x, o);
        if (lane >= o) x += y;
      }
      if (lane == 31) H.warp_sums[warp] = x;
      __syncthreads();
      uint32_t before = x - sum;
#pragma unroll
      for (int w = 0; w < NWARP; ++w) before += w < warp ? H.warp_sums[w] : 0u;
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        if (before < need && need <= before + v[u]) {
          H.digit = (uint32_t)(top - u);
          H.need = need - before;
        }
        before += v[u];
      }
      __syncthreads();
      prefix |= H.digit << sh;
      need = H.need;
    }
    T = prefix;
  }
  __syncthreads();
  // a contiguous part of the segment per warp: what it holds above T (or keeps whatever happens) and
  // equal to T, then the same again with the places known
  const int part = ((n + NWARP - 1) / NWARP + 31) / 32 * 32, w0 = min(n, warp * part), w1 = min(n, w0 + part);
  auto classes = [&](int i, uint32_t &above, uint32_t &equal) {
    const bool in = i < w1, free = in && (!cut || i < c0 || i >= c1);
    const uint32_t k = in && cut ? key(i) : 0u;
    above = __ballot_sync(FULL, free || (in && cut && k > T));
    equal = __ballot_sync(FULL, in && cut && !free && k == T);
  };
  uint32_t na = 0, ne = 0;
#pragma unroll 2
  for (int i = w0; i < w1; i += 32) {
    uint32_t above, equal;
    classes(i + lane, above, equal);
    na += __popc(above);
    ne += __popc(equal);
  }
  if (lane == 0) {
    H.above[warp] = na;
    H.equal[warp] = ne;
  }
  __syncthreads();
  if (warp == 0) {
    uint32_t a = lane < NWARP ? H.above[lane] : 0u, q = lane < NWARP ? H.equal[lane] : 0u;
    a = __reduce_add_sync(FULL, a);
    q = __reduce_add_sync(FULL, q);
    if (lane == 0) {
      H.all_above = a;
      H.all_equal = q;
    }
  }
  cl.sync();
  na = ne = 0;
  for (int c = 0; c < rank; ++c) {
    na += *cl.map_shared_rank(&H.all_above, c);
    ne += *cl.map_shared_rank(&H.all_equal, c);
  }
  for (int w = 0; w < warp; ++w) {
    na += H.above[w];
    ne += H.equal[w];
  }
#pragma unroll 2
  for (int i = w0; i < w1; i += 32) {
    uint32_t above, equal;
    classes(i + lane, above, equal);
    const uint32_t below = (1u << lane) - 1u, ties = ne + __popc(equal & below);
    if ((above >> lane & 1u) || ((equal >> lane & 1u) && ties < need)) {
      const uint32_t at = na + __popc(above & below) + min(ties, need);
      kept[at] = i0 + i + lane;
    }
    na += __popc(above);
    ne += __popc(equal);
  }
  cl.sync();  // (no CTA's shared memory goes while another reads it)
}

// Eight kept tokens of a head per warp, their weights and rows: K in lanes 0..15, V in lanes 16..31.
// stage_k / stage_v: [row][hkv][128] BF16 for a destination that is appended to; otherwise the rows
// go to the destination's ring.  (Rows of a BF16 cache never wrap.)
constexpr int GR = 8;
__global__ void __launch_bounds__(256) k_gather(LayerView S, LayerView T, const __grid_constant__ EvictArgs A,
                                                int64_t groups, uint4 *stage_k, uint4 *stage_v) {
  asm volatile("griddepcontrol.wait;" ::: "memory");  // the indices
  const int lane = threadIdx.x & 31, which = lane >> 4, part = lane & 15;
  int64_t it = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
  if (it >= groups) return;
  int e = 0;
  for (;; ++e) {
    const int64_t c = (int64_t)((A.s[e].count + GR - 1) / GR) * A.hkv;
    if (it < c) break;
    it -= c;
  }
  const EvictSeq &s = A.s[e];
  const int per = (s.count + GR - 1) / GR;
  const int head = (int)(it / per), first = (int)(it % per) * GR, rows = min(GR, s.count - first);
  const int32_t *kept = A.kept + ((int64_t)(A.entry0 + e) * A.hkv + head) * A.budget + first;
  const int idx = lane < rows ? kept[lane] : 0;
  if (A.mass_out && lane < rows) {
    const int64_t r = (int64_t)(A.entry0 + e) * A.hkv + head;
    A.mass_out[r * A.out_ld + first + lane] = __ldg(A.mass + r * A.mass_ld + idx);
  }
  const uint4 *src = reinterpret_cast<const uint4 *>(
      S.ring + (((int64_t)s.src * S.hkv + head) * 2 + which) * S.ring_cap * (2 * D)) + part;
  uint4 v[GR];
#pragma unroll
  for (int j = 0; j < GR; ++j) {
    const int64_t from = __shfl_sync(FULL, idx, j);
    if (j < rows) v[j] = __ldcs(src + from * (2 * D / 16));
  }
  const bool staged = stage_k != nullptr;
  if (staged ? S.tail_f16 : S.tail_f16 != T.tail_f16) {
#pragma unroll
    for (int j = 0; j < GR; ++j) {
      if (S.tail_f16) {  // F16 rows hold BF16 inputs rounded to F16: back to BF16 is exact
        uint32_t *w = reinterpret_cast<uint32_t *>(&v[j]);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const float2 f = ring2f(w[k], 1);
          const __nv_bfloat162 b = __floats2bfloat162_rn(f.x, f.y);
          w[k] = *reinterpret_cast<const uint32_t *>(&b);
        }
      } else {
        v[j] = bf16x8_to_ring(v[j], 1);
      }
    }
  }
  uint4 *dst;
  int64_t ld;
  if (staged) {
    dst = (which ? stage_v : stage_k) + ((s.row0 + first) * A.hkv + head) * (D / 8) + part;
    ld = (int64_t)A.hkv * (D / 8);
  } else {
    dst = reinterpret_cast<uint4 *>(
              T.ring + ((((int64_t)s.dst * T.hkv + head) * 2 + which) * T.ring_cap + first) * (2 * D)) + part;
    ld = 2 * D / 16;
  }
#pragma unroll
  for (int j = 0; j < GR; ++j)
    if (j < rows) __stcs(dst + j * ld, v[j]);
}

constexpr size_t align256(size_t x) { return (x + 255) / 256 * 256; }
size_t kept_bytes(const kvq_cache *c, int n_seqs, int budget) {
  return align256(sizeof(int32_t) * (size_t)n_seqs * c->p.n_kv_heads * budget);
}
size_t staged_bytes(const kvq_cache *c, int64_t rows) { return align256((size_t)rows * c->p.n_kv_heads * 2 * D); }

template <bool CACHED>
bool launch_select(const EvictArgs &A, unsigned rows, unsigned size, size_t smem, cudaStream_t st) {
  static std::atomic<uint64_t> done{0};  // devices on which the shared memory has been allowed
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return false;
  if (dev >= 64 || !(done.load(std::memory_order_relaxed) >> dev & 1)) {
    if (cudaFuncSetAttribute(k_select<CACHED>, cudaFuncAttributeMaxDynamicSharedMemorySize, SEG * 4) != cudaSuccess)
      return false;
    if (dev < 64) done.fetch_or(1ull << dev, std::memory_order_relaxed);
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(rows * size);
  cfg.blockDim = dim3(NT);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute la[1];
  la[0].id = cudaLaunchAttributeClusterDimension;
  la[0].val.clusterDim.x = size;
  la[0].val.clusterDim.y = la[0].val.clusterDim.z = 1;
  cfg.attrs = la;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, k_select<CACHED>, A) == cudaSuccess;
}

// set up behind the selection, waiting only for its results
bool launch_gather(const LayerView &S, const LayerView &T, const EvictArgs &A, int64_t groups, uint4 *stage_k,
                   uint4 *stage_v, cudaStream_t st) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((groups + 7) / 8));
  cfg.blockDim = dim3(256);
  cfg.stream = st;
  cudaLaunchAttribute la[1];
  la[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  la[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = la;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, k_gather, S, T, A, groups, stage_k, stage_v) == cudaSuccess;
}

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
  if (!src_ids || !dst_ids || !mass) return KVQ_E_INVAL;
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
  const int64_t head_rows = (int64_t)n_seqs * src->p.n_kv_heads, most_ld = INT64_MAX / 8 / head_rows;
  if (mass_ld < most || mass_ld > most_ld || (mass_out && mass_out_ld > most_ld)) return KVQ_E_INVAL;
  const auto bytes = [&](int64_t ld) { return (uint64_t)(head_rows * ld) * sizeof(float); };
  if (overlap(mass, bytes(mass_ld), kept, bytes(budget)) ||
      overlap(mass, bytes(mass_ld), mass_out, bytes(mass_out_ld)) ||
      overlap(kept, bytes(budget), mass_out, bytes(mass_out_ld)))
    return KVQ_E_INVAL;
  if (((uintptr_t)mass | (uintptr_t)kept | (uintptr_t)mass_out | (uintptr_t)workspace) & 15u) return KVQ_E_ALIGN;
  // the indices go to `kept` where the caller wants them, else in front of the staged rows
  const bool staged = dst->fam_k != FAM_BF16;
  const size_t for_kept = kept ? 0 : kept_bytes(src, n_seqs, budget);
  const size_t need = for_kept + (staged ? 2 * staged_bytes(src, (int64_t)n_seqs * budget) : 0);
  if (need > 0 && !workspace) return KVQ_E_INVAL;
  if (ws_bytes < need) return KVQ_E_SIZE;
  if (const int rc = check_device(src)) return rc;

  const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const LayerView S = layer_view(src, src_layer), T = layer_view(dst, dst_layer);
  const int hkv = src->p.n_kv_heads;
  uint8_t *ws = static_cast<uint8_t *>(workspace);
  uint4 *stage_k = nullptr, *stage_v = nullptr;
  if (staged) {
    stage_k = reinterpret_cast<uint4 *>(ws + for_kept);
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
    int64_t groups = 0, longest = 0;
    for (int i = 0; i < A.nseq; ++i) {
      A.s[i] = seqs[base + i];
      groups += (int64_t)((A.s[i].count + GR - 1) / GR) * hkv;
      longest = std::max<int64_t>(longest, A.s[i].n);
    }
    // a CTA for every 2048 tokens, up to a cluster of 8, as long as the rows leave two places an SM for
    // them (128 rows of 32 768: one CTA a row 83 us, two 56, four 59, in an earlier form), or while
    // shared memory holds no more
    unsigned size = 1;
    while (size < MAXC && longest > 2048 * (int64_t)size &&
           (A.nseq * hkv * 2 * (int)size <= 2 * src->num_sms || longest > SEG * (int64_t)size))
      size *= 2;
    const int64_t seg = (longest + size - 1) / size;
    const unsigned nrows = (unsigned)(A.nseq * hkv);
    if (!(seg <= SEG ? launch_select<true>(A, nrows, size, sizeof(uint32_t) * (size_t)seg, st)
                     : launch_select<false>(A, nrows, size, 0, st)))
      return KVQ_E_CUDA;
    note_launches(1);
    if (groups == 0) continue;
    if (!launch_gather(S, T, A, groups, stage_k, stage_v, st)) return KVQ_E_CUDA;
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
