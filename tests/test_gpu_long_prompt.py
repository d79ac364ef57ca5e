"""The operators as a long multimodal prompt uses them: rotate, append, attend in chunks, weigh the
tokens, keep those that matter in a quantized cache, decode on; and decoder rows that attend to an
encoder's states."""
import pytest

import prompt_helpers as P
from bit_kv_cache_17_b200 import kvq

pytestmark = pytest.mark.gpu


def test_prompt_to_decode():
    t = P.torch()
    hkv, G, n, chunk, budget, tail = 2, 4, 1500, 600, 700, 128
    hq = hkv * G
    g = t.Generator().manual_seed(0)
    q, k, v = (t.randn(n + 1, h, 128, generator=g).bfloat16().cuda() for h in (hq, hkv, hkv))
    i = t.arange(n + 1)
    pos = t.stack([i // 256, i % 256 // 16, i % 16]).int().cuda()
    rope = kvq.Rope((24, 20, 20), theta=1e6, turns=True)
    stage = kvq.KVCache(n_kv_heads=hkv, max_ctx=n, type_k="bf16", type_v="bf16", tail=0)
    mass = t.zeros(1, hkv, n, device="cuda")
    qr, kr = rope.apply(pos, q, k)
    outs = []
    for a in range(0, n, chunk):
        b = min(n, a + chunk)
        # chunk by chunk as a serving loop does
        qc, kc = rope.apply(pos[:, a:b].contiguous(), q[a:b], k[a:b])
        assert t.equal(qc, qr[a:b]) and t.equal(kc, kr[a:b])
        stage.append(0, [0], [b - a], kc, v[a:b])
        out, lse = stage.batch_attn(0, [0], [b - a], qc, causal=True, return_lse=True)
        stage.attn_mass(0, [0], [b - a], qc, lse, causal=True, decay=1.0, mass_in=mass, mass_out=mass)
        outs.append(out)
    # the chunks give what the whole prompt gives, and the weights of all its rows
    ref = P.attention(qr[:n], kr[:n].double(), v[:n].double(), True)
    P.check_attention(t.cat(outs), None, ref, n, P.UB16)
    total = mass.double().sum(-1)
    assert bool(((total - n * G).abs() <= 1e-4 * n * G).all())
    dec = kvq.KVCache(n_kv_heads=hkv, max_ctx=1024, type_k="q8_0", type_v="q8_0", tail=tail)
    kept, mass2 = stage.evict(dec, 0, 0, [0], [0], mass, budget, sink=4, recent=tail)
    assert dec.seq_len(0, 0) == budget
    # one decode step on the cut cache, at the position after the prompt
    q1, k1 = rope.apply(pos[:, n:].contiguous(), q[n:], k[n:], q_dtype=t.float32)
    got = dec.append_decode(0, [0], [1], k1, v[n:], q1)
    kk, vv = (dec.dequant(0, 0, w, 0, budget + 1).double() for w in (0, 1))
    for h in range(hkv):
        at = kept[0, h].long()
        # stored in 8 bits: half a step of a block's scale, absmax / 127
        d = (kk[:budget, h] - kr[at, h].double()).abs()
        assert bool((d <= kr[at, h].double().abs().amax(-1, keepdim=True) / 127 * 0.502).all())
        x = t.einsum("gd,nd->gn", q1[0, h * G:(h + 1) * G].double(), kk[:, h]) * 128 ** -0.5
        want = t.softmax(x, -1) @ vv[:, h]
        rel = (got[0, h * G:(h + 1) * G].double() - want).norm() / want.norm()
        assert rel <= 1e-3  # the decode's own bound
    assert dec.status() == 0 and stage.status() == 0


def test_decoder_over_encoder_states():
    """Two requests with two beams each attend, token by token, to their encoder's states: one cache,
    written once."""
    t = P.torch()
    lens, hkv, G = [210, 90], 2, 2
    k, v = P.kv(1, lens, hkv)
    enc = P.cache("bf16", lens, hkv, k, v, tail_f16=1)
    beams = [0, 0, 1, 1]
    for step in range(3):
        q = P.queries(step, 4, hkv * G, t.float16)
        out = enc.batch_attn(0, beams, [1] * 4, q)
        for i, s in enumerate(beams):
            ref = P.attention(q[i:i + 1], *P.cached(enc, 0, s), False)
            P.check_attention(out[i:i + 1], None, ref, lens[s], P.U16)
