// kvq_rope.cu - rotary positions with several axes, for query and key rows in one launch.
//
// The cache takes rotated rows; this is the step before it.  Channel pair i of a head turns by
// angle = pos[axis(i)] * f_i.  The angle is formed and reduced to one turn in 64 bits (a position
// of 10^7 leaves fp32 no correct digit of the fast pairs), then sin and cos are fp32; a rotation
// is two fp32 multiplies and adds per pair and one rounding to the output type.
//
// Bound: HBM (each row read once, written once).  A block takes TT tokens: its threads first fill
// a table of TT x 64 (cos, sin) in shared memory (64-bit work shared by all heads of a token), then
// stream the rows, one thread per unit of 16 channels (8 pairs), in 16-byte pieces.
#include <cuda_runtime.h>
#include <math.h>

#include "kvq_internal.h"

using namespace kvq;

namespace {

constexpr int NT = 256;

struct RopeArgs {
  double f[64];     // f_i / pi: half turns per position step
  uint8_t axis[64];
  const int32_t *pos;
  int64_t pos_ld, n;
  const void *q, *k;
  void *qo, *ko;
  int64_t q_ld, qo_ld, k_ld, ko_ld;
  int32_t hq, hk, half, adjacent, tt;
  float sign;       // -1: turn back
};

template <int T>
struct Elem;
template <>
struct Elem<KVQ_DT_F32> {
  using type = float;
  static __device__ __forceinline__ float up(float x) { return x; }
  static __device__ __forceinline__ float down(float x) { return x; }
};
template <>
struct Elem<KVQ_DT_BF16> {
  using type = __nv_bfloat16;
  static __device__ __forceinline__ float up(__nv_bfloat16 x) { return __bfloat162float(x); }
  static __device__ __forceinline__ __nv_bfloat16 down(float x) { return __float2bfloat16_rn(x); }
};
template <>
struct Elem<KVQ_DT_F16> {
  using type = __half;
  static __device__ __forceinline__ float up(__half x) { return __half2float(x); }
  static __device__ __forceinline__ __half down(float x) { return __float2half_rn(x); }
};

// 8 consecutive elements (16-byte aligned) as fp32, and back
template <int T>
__device__ __forceinline__ void load8(const typename Elem<T>::type *p, float (&x)[8]) {
  using E = typename Elem<T>::type;
  if constexpr (T == KVQ_DT_F32) {
    const float4 a = reinterpret_cast<const float4 *>(p)[0], b = reinterpret_cast<const float4 *>(p)[1];
    x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w, x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
  } else {
    const uint4 v = *reinterpret_cast<const uint4 *>(p);
    const E *e = reinterpret_cast<const E *>(&v);
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = Elem<T>::up(e[i]);
  }
}
template <int T>
__device__ __forceinline__ void store8(typename Elem<T>::type *p, const float (&x)[8]) {
  using E = typename Elem<T>::type;
  if constexpr (T == KVQ_DT_F32) {
    reinterpret_cast<float4 *>(p)[0] = make_float4(x[0], x[1], x[2], x[3]);
    reinterpret_cast<float4 *>(p)[1] = make_float4(x[4], x[5], x[6], x[7]);
  } else {
    uint4 v;
    E *e = reinterpret_cast<E *>(&v);
#pragma unroll
    for (int i = 0; i < 8; ++i) e[i] = Elem<T>::down(x[i]);
    *reinterpret_cast<uint4 *>(p) = v;
  }
}

// One unit u (0..7) of a head: 8 pairs of 16 channels.  VEC (rot_dim a multiple of 16): whole
// 16-byte pieces; the units behind the rotating ones carry the channels that pass through.
// Otherwise pairs straddle the pieces and are moved one by one.
template <int TI, int TO, bool VEC>
__device__ __forceinline__ void turn_unit(const typename Elem<TI>::type *x, typename Elem<TO>::type *y, int u,
                                          int half, int adjacent, const float2 *cs) {
  if constexpr (VEC) {
    const int rot = 2 * half;
    int ca, cb;
    if (adjacent) {
      ca = 16 * u, cb = ca + 8;
    } else if (8 * u < half) {
      ca = 8 * u, cb = half + 8 * u;
    } else {
      ca = rot + 16 * (u - half / 8), cb = ca + 8;
    }
    if (TI == TO && 8 * u >= half) {  // channels that pass through keep their bits (NaN payloads too)
      constexpr int V = sizeof(typename Elem<TI>::type) / 2;
      uint4 w[2 * V];
#pragma unroll
      for (int j = 0; j < V; ++j) {
        w[j] = reinterpret_cast<const uint4 *>(x + ca)[j];
        w[V + j] = reinterpret_cast<const uint4 *>(x + cb)[j];
      }
#pragma unroll
      for (int j = 0; j < V; ++j) {
        reinterpret_cast<uint4 *>(y + ca)[j] = w[j];
        reinterpret_cast<uint4 *>(y + cb)[j] = w[V + j];
      }
      return;
    }
    float a[8], b[8];
    load8<TI>(x + ca, a);
    load8<TI>(x + cb, b);
    if (8 * u >= half) {
      // converted only
    } else if (adjacent) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float2 t = cs[8 * u + j], v = cs[8 * u + 4 + j];
        const float p = a[2 * j], r = a[2 * j + 1], m = b[2 * j], n = b[2 * j + 1];
        a[2 * j] = p * t.x - r * t.y;
        a[2 * j + 1] = r * t.x + p * t.y;
        b[2 * j] = m * v.x - n * v.y;
        b[2 * j + 1] = n * v.x + m * v.y;
      }
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float2 t = cs[8 * u + j];
        const float p = a[j], r = b[j];
        a[j] = p * t.x - r * t.y;
        b[j] = r * t.x + p * t.y;
      }
    }
    store8<TO>(y + ca, a);
    store8<TO>(y + cb, b);
  } else {
#pragma unroll 1
    for (int j = 0; j < 8; ++j) {
      const int i = 8 * u + j;
      const bool on = i < half;
      const int ca = adjacent ? 2 * i : (on ? i : i + half), cb = adjacent ? ca + 1 : (on ? i + half : ca + 64 - half);
      if (TI == TO && !on) {
        const typename Elem<TI>::type xa = x[ca], xb = x[cb];
        reinterpret_cast<typename Elem<TI>::type *>(y)[ca] = xa;
        reinterpret_cast<typename Elem<TI>::type *>(y)[cb] = xb;
        continue;
      }
      const float p = Elem<TI>::up(x[ca]), r = Elem<TI>::up(x[cb]);
      const float2 t = on ? cs[i] : make_float2(1.f, 0.f);
      y[ca] = Elem<TO>::down(on ? p * t.x - r * t.y : p);
      y[cb] = Elem<TO>::down(on ? r * t.x + p * t.y : r);
    }
  }
}

template <int TQI, int TQO, bool VEC>
__global__ void __launch_bounds__(NT) k_rope(const __grid_constant__ RopeArgs A) {
  extern __shared__ float2 cs[];  // [tt][64]
  const int tid = threadIdx.x;
  const int64_t t0 = (int64_t)blockIdx.x * A.tt;
  const int nt = (int)min((int64_t)A.tt, A.n - t0);
  for (int e = tid; e < nt * 64; e += NT) {
    const int i = e & 63;
    if (i >= A.half) continue;
    // half turns, reduced to [-1, 1]: exact after the one 64-bit product
    const double a = (double)A.pos[A.axis[i] * A.pos_ld + t0 + (e >> 6)] * A.f[i];
    float s, c;
    sincospif((float)(a - 2.0 * rint(0.5 * a)), &s, &c);
    cs[e] = make_float2(c, A.sign * s);
  }
  __syncthreads();
  const int units = 8 * (A.hq + A.hk);
  using EI = typename Elem<TQI>::type;
  using EO = typename Elem<TQO>::type;
  for (int e = tid; e < nt * units; e += NT) {
    const int tl = e / units, r = e - tl * units, h = r >> 3, u = r & 7;
    const int64_t t = t0 + tl;
    if (h < A.hq)
      turn_unit<TQI, TQO, VEC>(static_cast<const EI *>(A.q) + t * A.q_ld + h * D,
                               static_cast<EO *>(A.qo) + t * A.qo_ld + h * D, u, A.half, A.adjacent, cs + 64 * tl);
    else
      turn_unit<KVQ_DT_BF16, KVQ_DT_BF16, VEC>(
          static_cast<const __nv_bfloat16 *>(A.k) + t * A.k_ld + (h - A.hq) * D,
          static_cast<__nv_bfloat16 *>(A.ko) + t * A.ko_ld + (h - A.hq) * D, u, A.half, A.adjacent, cs + 64 * tl);
  }
}

int elem_bytes(int t) { return t == KVQ_DT_F32 ? 4 : 2; }

// one tensor's arguments: in and out rows of `heads` heads
int check_rows(int64_t n, int heads, const void *x, int ti, int64_t ld, const void *y, int to, int64_t ldo) {
  if (heads == 0) return KVQ_OK;
  if (!x || !y) return KVQ_E_INVAL;
  if (ld < (int64_t)heads * D || ldo < (int64_t)heads * D) return KVQ_E_INVAL;
  const int64_t most = INT64_MAX / 8 / (n + 1);
  if (ld > most || ldo > most) return KVQ_E_INVAL;
  if (((uintptr_t)x | (uintptr_t)y) & 15u) return KVQ_E_ALIGN;
  if ((ld * elem_bytes(ti)) % 16 || (ldo * elem_bytes(to)) % 16) return KVQ_E_ALIGN;
  if (x == y && ti == to && ld == ldo) return KVQ_OK;
  const uintptr_t x0 = (uintptr_t)x, x1 = x0 + ((n - 1) * ld + heads * D) * elem_bytes(ti);
  const uintptr_t y0 = (uintptr_t)y, y1 = y0 + ((n - 1) * ldo + heads * D) * elem_bytes(to);
  return x0 < y1 && y0 < x1 ? KVQ_E_INVAL : KVQ_OK;
}

template <bool VEC>
cudaError_t run(int qi, int qo, unsigned grid, size_t smem, cudaStream_t st, const RopeArgs &A) {
#define KVQ_ROPE(I, O)                                    \
  if (qi == I && qo == O) {                               \
    k_rope<I, O, VEC><<<grid, NT, smem, st>>>(A);         \
    return cudaGetLastError();                            \
  }
  KVQ_ROPE(KVQ_DT_F32, KVQ_DT_F32) KVQ_ROPE(KVQ_DT_F32, KVQ_DT_BF16) KVQ_ROPE(KVQ_DT_F32, KVQ_DT_F16)
  KVQ_ROPE(KVQ_DT_BF16, KVQ_DT_F32) KVQ_ROPE(KVQ_DT_BF16, KVQ_DT_BF16) KVQ_ROPE(KVQ_DT_BF16, KVQ_DT_F16)
  KVQ_ROPE(KVQ_DT_F16, KVQ_DT_F32) KVQ_ROPE(KVQ_DT_F16, KVQ_DT_BF16) KVQ_ROPE(KVQ_DT_F16, KVQ_DT_F16)
#undef KVQ_ROPE
  return cudaErrorInvalidValue;
}

}  // namespace

extern "C" void kvq_rope_default_params(kvq_rope_params *p) {
  if (!p) return;
  *p = kvq_rope_params{};
  p->rot_dim = D;
  p->n_axes = 1;
  p->sections[0] = D / 2;
  p->theta = 10000.0;
}

extern "C" int kvq_rope(const kvq_rope_params *p, const double *inv_freq, int64_t n_tokens, const int32_t *pos,
                        int64_t pos_ld, int32_t n_q_heads, const void *q, int32_t q_type, int64_t q_ld, void *q_out,
                        int32_t q_out_type, int64_t q_out_ld, int32_t n_k_heads, const void *k, int64_t k_ld,
                        void *k_out, int64_t k_out_ld, kvq_stream_t stream) {
  if (!p || n_tokens < 0 || n_q_heads < 0 || n_k_heads < 0) return KVQ_E_INVAL;
  if (p->rot_dim < 2 || p->rot_dim > D || (p->rot_dim & 1) || p->n_axes < 1 || p->n_axes > 4) return KVQ_E_INVAL;
  if ((p->turns | p->adjacent | p->inverse) & ~1) return KVQ_E_INVAL;
  if (!inv_freq && !(p->theta > 0.0 && isfinite(p->theta))) return KVQ_E_INVAL;
  const int half = p->rot_dim / 2;
  int64_t pairs = 0;
  for (int a = 0; a < p->n_axes; ++a) {
    if (p->sections[a] < 0) return KVQ_E_INVAL;
    pairs += p->sections[a];
  }
  if (pairs != half) return KVQ_E_INVAL;
  if (n_q_heads > 0 && (q_type < 0 || q_type > KVQ_DT_F16 || q_out_type < 0 || q_out_type > KVQ_DT_F16))
    return KVQ_E_UNSUPPORTED;
  if (n_tokens > INT32_MAX || n_q_heads > 65536 || n_k_heads > 65536) return KVQ_E_INVAL;
  if (n_tokens == 0 || n_q_heads + n_k_heads == 0) return KVQ_OK;
  if (!pos || pos_ld < n_tokens || pos_ld > INT64_MAX / 32) return KVQ_E_INVAL;
  if ((uintptr_t)pos & 3u) return KVQ_E_ALIGN;
  int rc = check_rows(n_tokens, n_q_heads, q, q_type, q_ld, q_out, q_out_type, q_out_ld);
  if (rc == KVQ_OK) rc = check_rows(n_tokens, n_k_heads, k, KVQ_DT_BF16, k_ld, k_out, KVQ_DT_BF16, k_out_ld);
  if (rc) return rc;

  RopeArgs A{};
  int left[4] = {0, 0, 0, 0}, a = 0;
  for (int j = 0; j < p->n_axes; ++j) left[j] = p->sections[j];
  for (int i = 0; i < half; ++i) {
    while (left[a] == 0) a = (a + 1) % p->n_axes;
    A.axis[i] = (uint8_t)a;
    --left[a];
    if (p->turns) a = (a + 1) % p->n_axes;
    A.f[i] = (inv_freq ? inv_freq[i] : pow(p->theta, -2.0 * i / p->rot_dim)) / M_PI;
  }
  A.pos = pos;
  A.pos_ld = pos_ld;
  A.n = n_tokens;
  A.q = q, A.qo = q_out, A.q_ld = q_ld, A.qo_ld = q_out_ld, A.hq = n_q_heads;
  A.k = k, A.ko = k_out, A.k_ld = k_ld, A.ko_ld = k_out_ld, A.hk = n_k_heads;
  A.half = half;
  A.adjacent = p->adjacent;
  A.sign = p->inverse ? -1.f : 1.f;
  // few tokens: a block each (latency); many: four to a block, whose 256 angles are one per thread
  A.tt = n_tokens >= 4096 ? 4 : 1;
  const unsigned grid = (unsigned)((n_tokens + A.tt - 1) / A.tt);
  const size_t smem = sizeof(float2) * 64 * A.tt;
  const bool vec = p->rot_dim % 16 == 0;
  const int qi = n_q_heads ? q_type : KVQ_DT_BF16, qo = n_q_heads ? q_out_type : KVQ_DT_BF16;
  const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const cudaError_t e = vec ? run<true>(qi, qo, grid, smem, st, A) : run<false>(qi, qo, grid, smem, st, A);
  if (e != cudaSuccess) return KVQ_E_CUDA;
  note_launches(1);
  return KVQ_OK;
}
