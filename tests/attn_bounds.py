"""Bounds of batch attention that see a single wrong tile: values that mark the 128-token tile they belong
to, and tolerances without slack.

Value rows of tile j are zero but for channel j mod 128, which is 1 + (token mod 5) / 4: every sum is one of
non-negative terms, so a bound relative to the terms is one relative to the result."""
import prompt_helpers as P

TILE = 128


def marked_values(n, hkv):
    """[n, hkv, 128] BF16 (exact in F16 too)"""
    t = P.torch()
    i = t.arange(n)
    v = t.zeros(n, hkv, P.D)
    v[i, :, i // TILE % P.D] = (1 + (i % 5) / 4)[:, None]
    return v.bfloat16()


def check(out, lse, ref, n, u_weight, f16_weights, quantized=False):
    """ref: P.attention's.  u_weight: half a step of the weights as the product takes them (of their
    remainders, where it takes those too).  f16_weights: weights are F16, the largest of a row 2^7 or more:
    below the normal range each is off by up to 2^-25 / 2^7 of the largest."""
    t = P.torch()
    _, want, mag, want_lse, spread = ref
    e = P.score_error(spread, P.U16 if quantized else 0.0)[..., None]
    # a weight and the sum of the weights off by the score's error each, the weight's and (rebuilt) the
    # value's rounding, a step of fp32 for every addition and a few for exp and the division
    rel = 2 * e + u_weight + (P.U16 if quantized else 0.0) + (n + 16) * 2 * P.U32
    faint = n * 2.0 ** -32 * 2.0 if f16_weights else 0.0  # (values are below 2)
    tol = rel * mag + faint
    tol = tol + P.half_step(out.dtype) * (want.abs() + tol) + (2.0 ** -25 if out.dtype == t.float16 else 0.0)
    err = (out.double() - want).abs()
    assert bool((err <= tol).all()), (float((err - tol).max()), float(err.max()))
    if lse is not None:
        d = (lse.double() - want_lse).abs()
        bound = e[..., 0] + 4 * P.U32 * want_lse.abs() + (n + 16) * 2 * P.U32
        assert bool((d <= bound).all()), float((d - bound).max())


def weight_step(m, G, f16):
    """Half a step of an entry's weights: with their remainders where its query rows fill no more than one tile."""
    u = P.U16 if f16 else P.UB16
    return u * u if m <= TILE // G else u


def inputs(seed, n, m, hkv, G):
    """queries [m, hkv G, 128] and keys [n, hkv, 128], BF16, on the host"""
    t = P.torch()
    g = t.Generator().manual_seed(seed)
    return t.randn(m, hkv * G, P.D, generator=g).bfloat16(), (t.randn(n, hkv, P.D, generator=g)).bfloat16()


def rounded(ref, dtype):
    """The exact result as the call would return it."""
    return ref[1].to(dtype), ref[3].float()
