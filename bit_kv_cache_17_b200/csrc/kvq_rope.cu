// kvq_rope.cu - rotary positions with several axes, for query and key rows in one launch.
//
// The cache takes rotated rows; this is the step before it.  Channel pair i of a head turns by
// angle = pos[axis(i)] * f_i.  The angle is formed and reduced to one turn in 64 bits (a position
// of 10^7 leaves fp32 no correct digit of the fast pairs), then sin and cos are fp32; a rotation
// is two fp32 multiplies and adds per pair and one rounding to the output type.
//
// Bound: HBM (each row read once, written once).  A block takes tt tokens: its threads fill a table
// of tt x 64 (cos, sin) in shared memory (64-bit work shared by all heads of a token), then stream the
// rows in pieces of 16 bytes, two to a thread and step, asked for before the table is made.
#include <cuda_runtime.h>
#include <math.h>

#include <algorithm>
#include <utility>

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

// A unit of a head: two pieces of E elements, 16 bytes each as they are read (E = 4 for fp32, 8 for
// the 16-bit types), a head being 64 / E units.  Consecutive lanes take consecutive pieces.
template <int T>
constexpr int E_OF = T == KVQ_DT_F32 ? 4 : 8;

// Where the two pieces of unit u lie: pairs E u .. of the halves (E u, half + E u); adjacent pairs: the
// pieces u of each half of the head; behind the rotating ones, pieces of the channels that pass through.
template <int E>
__device__ __forceinline__ void places(int u, int half, int adjacent, int &a, int &b) {
  if (adjacent) {
    a = E * u;
    b = 64 + E * u;
  } else if (E * u < half) {
    a = E * u;
    b = half + E * u;
  } else {
    a = 2 * half + (E * u - half);
    b = a + (64 - half);
  }
}

// elements 2 i and 2 i + 1 of a piece, as fp32; and back
template <int T>
__device__ __forceinline__ float2 get2(const uint4 &w, int i) {
  if constexpr (T == KVQ_DT_F32) return i ? make_float2(__uint_as_float(w.z), __uint_as_float(w.w))
                                          : make_float2(__uint_as_float(w.x), __uint_as_float(w.y));
  return ring2f(i == 0 ? w.x : (i == 1 ? w.y : (i == 2 ? w.z : w.w)), T == KVQ_DT_F16);
}
template <int T>
__device__ __forceinline__ uint32_t round_pair(float x, float y) {
  if constexpr (T == KVQ_DT_F16) {
    const __half2 h = __floats2half2_rn(x, y);
    return *reinterpret_cast<const uint32_t *>(&h);
  }
  const __nv_bfloat162 h = __floats2bfloat162_rn(x, y);
  return *reinterpret_cast<const uint32_t *>(&h);
}
// N consecutive fp32 values to a piece of type T
template <int T, int N>
__device__ __forceinline__ void put(typename Elem<T>::type *y, const float (&x)[N]) {
  if constexpr (T == KVQ_DT_F32) {
#pragma unroll
    for (int i = 0; i < N; i += 4) *reinterpret_cast<float4 *>(y + i) = make_float4(x[i], x[i + 1], x[i + 2], x[i + 3]);
  } else if constexpr (N == 4) {
    *reinterpret_cast<uint2 *>(y) = make_uint2(round_pair<T>(x[0], x[1]), round_pair<T>(x[2], x[3]));
  } else {
    *reinterpret_cast<uint4 *>(y) = make_uint4(round_pair<T>(x[0], x[1]), round_pair<T>(x[2], x[3]),
                                               round_pair<T>(x[4], x[5]), round_pair<T>(x[6], x[7]));
  }
}

// The angles of one token: the cosine of pair p at float cos_at(p), its sine 64 floats behind, in an
// order in which the lanes of a head read 128 consecutive bytes at once (pair by pair they met in four
// banks: 88 us for 16384 tokens of 48 heads in BF16).
__device__ __forceinline__ int cos_at(int pair) { return 32 * ((pair >> 2) & 1) + 4 * (pair >> 3) + (pair & 3); }
constexpr int TAB = 128;  // floats per token

// Rotates the unit (wa, wb) whose pieces lie at channels a and b and stores it.  Channels that pass
// through keep their bits where the types agree (NaN payloads too).
template <int TI, int TO>
__device__ __forceinline__ void turn(const uint4 &wa, const uint4 &wb, typename Elem<TO>::type *y, int a, int b,
                                     int half, int adjacent, const float *cs) {
  constexpr int E = E_OF<TI>;
  float xa[E], xb[E];
#pragma unroll
  for (int i = 0; i < E / 2; ++i) {
    const float2 p = get2<TI>(wa, i), r = get2<TI>(wb, i);
    xa[2 * i] = p.x, xa[2 * i + 1] = p.y, xb[2 * i] = r.x, xb[2 * i + 1] = r.y;
  }
  if (adjacent) {
    auto piece = [&](float (&x)[E], int at, const uint4 &w) {
      if (at >= 2 * half) {
        if constexpr (TI == TO)
          *reinterpret_cast<uint4 *>(y + at) = w;
        else
          put<TO, E>(y + at, x);
        return;
      }
#pragma unroll
      for (int i = 0; i < E / 2; ++i) {
        const float c = cs[cos_at(at / 2) + i], s = cs[64 + cos_at(at / 2) + i];
        const float p = x[2 * i], r = x[2 * i + 1];
        x[2 * i] = p * c - r * s;
        x[2 * i + 1] = r * c + p * s;
      }
      put<TO, E>(y + at, x);
    };
    piece(xa, a, wa);
    piece(xb, b, wb);
    return;
  }
  if (a >= 2 * half) {
    if constexpr (TI == TO) {
      *reinterpret_cast<uint4 *>(y + a) = wa;
      *reinterpret_cast<uint4 *>(y + b) = wb;
    } else {
      put<TO, E>(y + a, xa);
      put<TO, E>(y + b, xb);
    }
    return;
  }
#pragma unroll
  for (int g = 0; g < E / 4; ++g) {
    const float4 c4 = *reinterpret_cast<const float4 *>(cs + cos_at(a + 4 * g));
    const float4 s4 = *reinterpret_cast<const float4 *>(cs + 64 + cos_at(a + 4 * g));
    const float c[4] = {c4.x, c4.y, c4.z, c4.w}, s[4] = {s4.x, s4.y, s4.z, s4.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float p = xa[4 * g + j], r = xb[4 * g + j];
      xa[4 * g + j] = p * c[j] - r * s[j];
      xb[4 * g + j] = r * c[j] + p * s[j];
    }
  }
  put<TO, E>(y + a, xa);
  put<TO, E>(y + b, xb);
}

// rot_dim no multiple of 16: pairs straddle the pieces and are moved one by one
template <int TI, int TO>
__device__ __forceinline__ void turn_pairs(const typename Elem<TI>::type *x, typename Elem<TO>::type *y, int u,
                                           int half, int adjacent, const float *cs) {
#pragma unroll 1
  for (int j = 0; j < 8; ++j) {
    const int i = 8 * u + j;
    const bool on = i < half;
    const int ca = adjacent ? 2 * i : (on ? i : i + half), cb = adjacent ? ca + 1 : (on ? i + half : ca + 64 - half);
    if constexpr (TI == TO) {
      if (!on) {
        const typename Elem<TI>::type xa = x[ca], xb = x[cb];
        y[ca] = xa;
        y[cb] = xb;
        continue;
      }
    }
    const float p = Elem<TI>::up(x[ca]), r = Elem<TI>::up(x[cb]);
    const float2 t = on ? make_float2(cs[cos_at(i)], cs[64 + cos_at(i)]) : make_float2(1.f, 0.f);
    y[ca] = Elem<TO>::down(on ? p * t.x - r * t.y : p);
    y[cb] = Elem<TO>::down(on ? r * t.x + p * t.y : r);
  }
}

// units in flight per thread
constexpr int UNITS = 3;

template <int TQI, int TQO, bool VEC>
__global__ void __launch_bounds__(NT) k_rope(const __grid_constant__ RopeArgs A) {
  extern __shared__ __align__(16) float tables[];  // [2][tt][TAB]
  using EI = typename Elem<TQI>::type;
  using EO = typename Elem<TQO>::type;
  constexpr int KT = KVQ_DT_BF16;
  const int tid = threadIdx.x;
  constexpr int EQ = E_OF<TQI>, PQ = 64 / EQ;  // units of a q head; a k head has 8
  const int nq = PQ * A.hq, units = VEC ? nq + 8 * A.hk : 8 * (A.hq + A.hk);
  // this thread's pair, the same for every token: its frequency and axis are read once per block
  const int pair = tid & 63;
  const double freq = pair < A.half ? A.f[pair] : 0.0;
  const int32_t *pos = A.pos + (pair < A.half ? A.axis[pair] : 0) * A.pos_ld;
  int odd = 0;
#pragma unroll 1
  for (int64_t t0 = (int64_t)blockIdx.x * A.tt; t0 < A.n; t0 += (int64_t)gridDim.x * A.tt, odd ^= 1) {
    const int nt = (int)min((int64_t)A.tt, A.n - t0), all = nt * units;
    float *cs = tables + odd * A.tt * TAB;  // (the other one may still be in use)
    auto table = [&]() {
      for (int j = tid >> 6; j < nt; j += NT / 64) {
        // half turns, reduced to [-1, 1]: exact after the one 64-bit product
        const double a = (double)pos[t0 + j] * freq;
        float s, c;
        sincospif((float)(a - 2.0 * rint(0.5 * a)), &s, &c);
        cs[TAB * j + cos_at(pair)] = c;
        cs[TAB * j + 64 + cos_at(pair)] = A.sign * s;
      }
      __syncthreads();
    };
    if constexpr (VEC) {
      // U units a thread, all on their way before the table is made (one round: tt is chosen so)
      constexpr int U = UNITS;
      bool made = false;
#pragma unroll 1
      for (int e0 = 0; e0 < all; e0 += U * NT) {
        uint4 wa[U], wb[U];
        int tl[U], at[U], a[U], b[U];
#pragma unroll
        for (int j = 0; j < U; ++j) {
          const int e = e0 + j * NT + tid;
          if (e >= all) break;
          tl[j] = e / units;
          at[j] = e - tl[j] * units;
          if (at[j] < nq) {
            places<EQ>(at[j] % PQ, A.half, A.adjacent, a[j], b[j]);
            const EI *p = static_cast<const EI *>(A.q) + (t0 + tl[j]) * A.q_ld + at[j] / PQ * D;
            wa[j] = *reinterpret_cast<const uint4 *>(p + a[j]);
            wb[j] = *reinterpret_cast<const uint4 *>(p + b[j]);
          } else {
            const int k = at[j] - nq;
            places<8>(k & 7, A.half, A.adjacent, a[j], b[j]);
            const __nv_bfloat16 *p = static_cast<const __nv_bfloat16 *>(A.k) + (t0 + tl[j]) * A.k_ld + (k >> 3) * D;
            wa[j] = *reinterpret_cast<const uint4 *>(p + a[j]);
            wb[j] = *reinterpret_cast<const uint4 *>(p + b[j]);
          }
        }
        if (!made) table();
        made = true;
#pragma unroll
        for (int j = 0; j < U; ++j) {
          if (e0 + j * NT + tid >= all) break;
          const float *c = cs + TAB * tl[j];
          if (at[j] < nq)
            turn<TQI, TQO>(wa[j], wb[j], static_cast<EO *>(A.qo) + (t0 + tl[j]) * A.qo_ld + at[j] / PQ * D, a[j], b[j],
                           A.half, A.adjacent, c);
          else
            turn<KT, KT>(wa[j], wb[j],
                         static_cast<__nv_bfloat16 *>(A.ko) + (t0 + tl[j]) * A.ko_ld + ((at[j] - nq) >> 3) * D, a[j],
                         b[j], A.half, A.adjacent, c);
        }
      }
    } else {
      table();
      for (int e = tid; e < all; e += NT) {
        const int tl = e / units, r = e - tl * units, h = r >> 3, u = r & 7;
        const int64_t t = t0 + tl;
        if (h < A.hq)
          turn_pairs<TQI, TQO>(static_cast<const EI *>(A.q) + t * A.q_ld + h * D,
                               static_cast<EO *>(A.qo) + t * A.qo_ld + h * D, u, A.half, A.adjacent, cs + TAB * tl);
        else
          turn_pairs<KT, KT>(static_cast<const __nv_bfloat16 *>(A.k) + t * A.k_ld + (h - A.hq) * D,
                             static_cast<__nv_bfloat16 *>(A.ko) + t * A.ko_ld + (h - A.hq) * D, u, A.half, A.adjacent,
                             cs + TAB * tl);
      }
    }
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

// Rows of one tensor: n of `width` bytes, `stride` apart (at least the width).
struct Rows {
  uintptr_t at;
  uint64_t width, stride;
};

// Whether n rows of a and n of b share a byte.  Of one stride (slices of a packed row) they may interleave:
// what counts then is where b lies within a's row.
bool rows_overlap(int64_t n, Rows a, Rows b) {
  if (b.at < a.at) std::swap(a, b);
  const uint64_t apart = b.at - a.at;
  if (apart >= (uint64_t)(n - 1) * a.stride + a.width) return false;
  if (n == 1 || a.stride != b.stride) return true;
  const uint64_t within = apart % a.stride;
  return within < a.width || a.stride - within < b.width;
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
  if (!pos || (pos_ld != 0 && pos_ld < n_tokens) || pos_ld > INT64_MAX / 32) return KVQ_E_INVAL;
  if ((uintptr_t)pos & 3u) return KVQ_E_ALIGN;
  int rc = check_rows(n_tokens, n_q_heads, q, q_type, q_ld, q_out, q_out_type, q_out_ld);
  if (rc == KVQ_OK) rc = check_rows(n_tokens, n_k_heads, k, KVQ_DT_BF16, k_ld, k_out, KVQ_DT_BF16, k_out_ld);
  if (rc) return rc;
  // an output over another tensor's rows, or over the positions: other blocks still read (or write) those
  const auto rows = [](const void *x, int heads, int type, int64_t ld) {
    return Rows{(uintptr_t)x, (uint64_t)heads * D * elem_bytes(type), (uint64_t)ld * elem_bytes(type)};
  };
  const Rows rq = rows(q, n_q_heads, q_type, q_ld), rqo = rows(q_out, n_q_heads, q_out_type, q_out_ld);
  const Rows rk = rows(k, n_k_heads, KVQ_DT_BF16, k_ld), rko = rows(k_out, n_k_heads, KVQ_DT_BF16, k_out_ld);
  if (n_q_heads && n_k_heads &&
      (rows_overlap(n_tokens, rqo, rk) || rows_overlap(n_tokens, rko, rq) || rows_overlap(n_tokens, rqo, rko)))
    return KVQ_E_INVAL;
  const uint64_t pos_bytes = (uint64_t)((p->n_axes - 1) * pos_ld + n_tokens) * sizeof(int32_t);
  const auto over_pos = [&](const Rows &r) {
    return overlap(pos, pos_bytes, (const void *)r.at, (uint64_t)(n_tokens - 1) * r.stride + r.width);
  };
  if ((n_q_heads && over_pos(rqo)) || (n_k_heads && over_pos(rko))) return KVQ_E_INVAL;

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
  // a block takes the tokens whose units its threads hold at once (fewer tokens than blocks: one each) and
  // stays for more: a thread reads its frequency once, six blocks an SM (16384 tokens of 48 heads, BF16:
  // 70 us; eight blocks of four units a thread 74, a block for every group of tokens 78)
  const int64_t units = (n_q_heads && q_type == KVQ_DT_F32 ? 16ll : 8ll) * n_q_heads + 8ll * n_k_heads, held = UNITS * NT;
  A.tt = (int)std::max<int64_t>(1, std::min<int64_t>({held / units, n_tokens / (4 * 148), 32}));
  const unsigned grid = (unsigned)std::min<int64_t>((n_tokens + A.tt - 1) / A.tt, 148 * 6);
  const size_t smem = sizeof(float) * 2 * TAB * A.tt;
  const bool vec = p->rot_dim % 16 == 0;
  const int qi = n_q_heads ? q_type : KVQ_DT_BF16, qo = n_q_heads ? q_out_type : KVQ_DT_BF16;
  const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const cudaError_t e = vec ? run<true>(qi, qo, grid, smem, st, A) : run<false>(qi, qo, grid, smem, st, A);
  if (e != cudaSuccess) return KVQ_E_CUDA;
  note_launches(1);
  return KVQ_OK;
}
