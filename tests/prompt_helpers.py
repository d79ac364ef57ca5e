"""References in 64 bits for the operators around a prompt's cache (rope, batch attention, attention
weights, eviction), and the error bounds their results are held to.

Bounds count roundings: half a step is eps / 2 of the type, relative to the value (fp32 2^-24, F16
2^-11, BF16 2^-8)."""
import math

import numpy as np

D = 128
U32, U16, UB16 = 2.0 ** -24, 2.0 ** -11, 2.0 ** -8


def torch():
    import torch as t

    return t


def half_step(dtype):
    return torch().finfo(dtype).eps / 2


def kv(seed, lens, hkv, scale=1.0):
    """BF16 K and V rows [sum(lens), hkv, 128] with two large key channels."""
    t = torch()
    g = t.Generator().manual_seed(seed)
    n = sum(lens)
    k = t.randn(n, hkv, D, generator=g)
    k[..., 7] *= 5.0
    k[..., 63] *= 5.0
    v = t.randn(n, hkv, D, generator=g)
    return (k * scale).bfloat16().cuda(), v.bfloat16().cuda()


def queries(seed, rows, hq, dtype):
    t = torch()
    g = t.Generator().manual_seed(1000 + seed)
    # BF16 values, which F16 holds too
    return t.randn(rows, hq, D, generator=g).bfloat16().to(dtype).cuda()


def cache(type_, lens, hkv, k, v, tail=0, tail_f16=0, type_v=None, n_layers=1, layer=0, max_ctx=None):
    from bit_kv_cache_17_b200.kvq import KVCache

    c = KVCache(n_layers=n_layers, n_seqs=len(lens), n_kv_heads=hkv, max_ctx=max_ctx or max(max(lens), 1), type_k=type_,
                type_v=type_v or type_, tail=tail, tail_f16=tail_f16)
    # what no token has written yet holds NaN patterns
    if type_ == "bf16":
        c.rows16(layer).fill_(math.nan)
    else:
        c.storage[: c.locate(2, 0, 0, 0, 0, 0)[0]].fill_(255)
    c.append(layer, list(range(len(lens))), lens, k, v)
    return c


def cached(c, layer, seq):
    """The values a sequence holds, [n, hkv, 128] fp64, K and V."""
    n = c.seq_len(layer, seq)
    if n == 0:
        z = torch().zeros(0, c.params.n_kv_heads, D, dtype=torch().float64, device="cuda")
        return z, z
    return tuple(c.dequant(layer, seq, w, 0, n).double() for w in (0, 1))


def attention(q, k, v, causal, scale=None):
    """q [m, hq, 128], k / v [n, hkv, 128] fp64 -> x, seen [hq, m, n]; out, its absolute sum, lse,
    and per row the largest sum of |q k| scale."""
    t = torch()
    m, hq, n = q.shape[0], q.shape[1], k.shape[0]
    g = hq // k.shape[1]
    scale = D ** -0.5 if scale is None else scale
    q, kk, vv = q.double(), k.repeat_interleave(g, 1), v.repeat_interleave(g, 1)
    x = t.einsum("mhd,nhd->hmn", q, kk) * scale
    spread = t.einsum("mhd,nhd->hmn", q.abs(), kk.abs()).amax(-1).T * scale if n else t.zeros(m, hq, device=q.device)
    seen = t.ones(m, n, dtype=t.bool, device=q.device)
    if causal:
        seen = t.arange(n, device=q.device)[None] < n - m + 1 + t.arange(m, device=q.device)[:, None]
    x = x.masked_fill(~seen, -math.inf)
    lse = t.logsumexp(x, -1) if n else t.full((hq, m), -math.inf, dtype=t.float64, device=q.device)
    p = t.where(lse[..., None] == -math.inf, 0.0, t.exp(x - t.where(lse == -math.inf, 0.0, lse)[..., None]))
    out = t.einsum("hmn,nhd->mhd", p, vv)
    mag = t.einsum("hmn,nhd->mhd", p, vv.abs())
    return x, out, mag, lse.T, spread


def score_error(spread, u_key=0.0):
    """Bound of a score's error per row: 128 products and sums in fp32 (the tensor core may truncate:
    a whole step each), the scale's multiply, and the rounding of the cached values if there is one."""
    return spread * (2 * 130 * U32 + u_key)


def check_attention(out, lse, ref, n, u_weight, quantized=False):
    """u_weight: half a step of the weights' 16-bit type."""
    t = torch()
    _, want, mag, want_lse, spread = ref
    e = score_error(spread, U16 if quantized else 0.0)[..., None]
    # exp of a score off by e, twice (weight and sum); the weight's rounding; the value's rounding when
    # rebuilt; fp32 sums over n tokens; F16 weights below its normal range are off by up to 2^-25 each
    rel = 2 * e + u_weight + (U16 if quantized else 0.0) + (n + 8) * 2 * U32
    vmax = mag.abs().amax() if mag.numel() else 0.0
    tol = rel * mag + half_step(out.dtype) * (want.abs() + rel * mag) + n * 2.0 ** -25 * 16 * vmax + 2.0 ** -25
    err = (out.double() - want).abs()
    assert bool((err <= tol).all()), (float((err - tol).max()), float(err.max()))
    if lse is not None:
        inf = want_lse == -math.inf
        assert t.equal(inf, lse == -math.inf)
        d = (lse.double() - want_lse)[~inf].abs()
        bound = (e[..., 0] + 4 * U32 * want_lse.abs() + (n + 8) * 2 * U32)[~inf]
        assert bool((d <= bound).all()), float((d - bound).max())


def evict_ref(mass, n, budget, sink, recent):
    """Kept indices of one (sequence, head): numpy, 64-bit keys."""
    if n <= budget:
        return np.arange(n)
    mid = np.arange(sink, n - recent)
    w = mass[mid].astype(np.float64)
    w = np.where(np.isnan(w), np.inf, w)
    nan = np.isnan(mass[mid])
    order = np.lexsort((mid, -w, ~nan))  # NaN first, then by weight, then by index
    take = mid[order[: budget - sink - recent]]
    return np.sort(np.concatenate([np.arange(sink), take, np.arange(n - recent, n)]))
