"""The fp64 attention oracle against central differences and closed cases (CPU), and
the host side of the attention operators: refusals, workspace sizes, frequencies."""
import math

import numpy as np
import pytest

from oracle import attention as O


def _diff(f, x, d, h=1e-6):
    return (f(x + h * d) - f(x - h * d)) / (2 * h)


@pytest.mark.parametrize("n,m,causal", [(5, 7, True), (7, 5, True), (4, 6, False), (1, 1, True)])
def test_attention_gradients_are_the_differences(n, m, causal):
    r = np.random.default_rng(n * 10 + m)
    D, scale = 6, 0.4
    q, k, v = (r.standard_normal((c, D)) for c in (n, m, m))
    do = r.standard_normal((n, D))
    p = O.attention(q, k, v, scale, causal)[2]
    dq, dk, dv, _ = O.attention_backward(do, q, k, v, p, scale)

    def loss(q, k, v):
        return float((O.attention(q, k, v, scale, causal)[0] * do).sum())

    for x, g, f in ((q, dq, lambda t: loss(t, k, v)), (k, dk, lambda t: loss(q, t, v)),
                    (v, dv, lambda t: loss(q, k, t))):
        d = r.standard_normal(x.shape)
        assert abs(_diff(f, x, d) - (g * d).sum()) < 1e-6


def test_rows_without_a_key_are_zero():
    r = np.random.default_rng(0)
    q, k, v = r.standard_normal((5, 4)), r.standard_normal((3, 4)), r.standard_normal((3, 4))
    out, lse, p = O.attention(q, k, v, 1.0, True)
    assert (out[:2] == 0).all() and np.isneginf(lse[:2]).all() and (p[:2] == 0).all()
    assert np.allclose(out[2], v[0]) and np.allclose(p[2:].sum(-1), 1)


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("rot", [0, 4, 8])
def test_norm_rope_gradients_are_the_differences(interleaved, rot):
    r = np.random.default_rng(rot)
    T, H, D = 3, 2, 8
    x, g, w = r.standard_normal((T, H, D)), r.standard_normal((T, H, D)), r.standard_normal(D)
    ang = r.standard_normal((T, rot // 2))
    c, s = np.cos(ang), np.sin(ang)
    dx, dw = O.norm_rope_backward(g, x, w, 1e-3, c, s, interleaved)

    def loss(x, w):
        return float((O.norm_rope(x, w, 1e-3, c, s, interleaved) * g).sum())

    d, e = r.standard_normal(x.shape), r.standard_normal(D)
    assert abs(_diff(lambda t: loss(t, w), x, d) - (dx * d).sum()) < 1e-6
    assert abs(_diff(lambda t: loss(x, t), w, e) - (dw * e).sum()) < 1e-6


def test_rotation_turns_with_the_position():
    """q at p against k at p' depends on p - p' alone, in both layouts."""
    r = np.random.default_rng(3)
    q, k = r.standard_normal((1, 1, 8)), r.standard_normal((1, 1, 8))
    inv = 10.0 ** -np.arange(4)

    def at(x, p, il):
        a = (p * inv)[None]
        return O.rotate(x, np.cos(a), np.sin(a), il)

    for il in (False, True):
        a = (at(q, 5, il) * at(k, 2, il)).sum()
        b = (at(q, 105, il) * at(k, 102, il)).sum()
        assert abs(a - b) < 1e-12 and abs(a - (q * k).sum()) > 1e-3


# ------------------------------------------------------------------ host side
@pytest.fixture(scope="module")
def B():
    from token_dispatch_grouped_gb300 import build
    build.build()
    from token_dispatch_grouped_gb300 import binding
    return binding


FAKE = 1 << 20   # an aligned address that no refused call reads


def _heads(B, ts, hs, at=FAKE):
    return B.MoeHeads(at, ts, hs)


def _norm_rope(B, a=(4, 2, 64), T=3, q=None, k=None, wq=FAKE, wk=FAKE, eps=1e-6, pos=FAKE,
               rope=(FAKE, 10, 64, 0), q_out=None, k_out=None):
    Hq, Hkv, D = a
    q, q_out = (q or _heads(B, Hq * D, D), q_out or _heads(B, Hq * D, D))
    k, k_out = (k or _heads(B, Hkv * D, D), k_out or _heads(B, Hkv * D, D))
    return B.LIB.moe_norm_rope(B.MoeAttnShape(*a), T, q, k, wq, wk, eps, pos, B.MoeRope(*rope),
                               q_out, k_out, None)


def test_norm_rope_refusals(B):
    bad, shape, mis = B.MOE_ERR_INVALID_ARG, B.MOE_ERR_UNSUPPORTED_SHAPE, B.MOE_ERR_MISALIGNED
    assert _norm_rope(B, a=(0, 2, 64)) == bad
    assert _norm_rope(B, a=(5, 2, 64)) == shape
    assert _norm_rope(B, a=(130, 2, 64)) == shape           # 65 query heads on a key head
    assert _norm_rope(B, a=(4, 2, 60)) == shape
    assert _norm_rope(B, a=(4, 2, 136)) == shape
    assert _norm_rope(B, T=-1) == bad
    assert _norm_rope(B, T=(1 << 24) + 1) == shape
    assert _norm_rope(B, wk=None) == bad                    # one norm weight alone
    assert _norm_rope(B, eps=float("nan")) == bad
    assert _norm_rope(B, eps=-1.0) == bad
    assert _norm_rope(B, wq=FAKE + 4) == mis
    assert _norm_rope(B, pos=None) == bad
    assert _norm_rope(B, rope=(None, 10, 64, 0)) == bad
    assert _norm_rope(B, rope=(FAKE, 0, 64, 0)) == bad
    assert _norm_rope(B, rope=(FAKE, 10, 66, 0)) == bad
    assert _norm_rope(B, rope=(FAKE, 10, 63, 0)) == bad
    assert _norm_rope(B, rope=(FAKE, 10, 64, 2)) == bad
    assert _norm_rope(B, rope=(FAKE + 4, 10, 64, 0)) == mis
    assert _norm_rope(B, q=_heads(B, 256, 64, FAKE + 2)) == mis
    assert _norm_rope(B, q=_heads(B, 0, 64)) == bad         # broadcast tokens
    assert _norm_rope(B, q=_heads(B, 256, 0)) == bad        # broadcast heads
    assert _norm_rope(B, q=_heads(B, 260, 64)) == mis       # stride not of 16 bytes
    assert _norm_rope(B, q_out=_heads(B, 128, 64)) == bad   # an output over itself
    assert _norm_rope(B, q=B.MoeHeads(None, 256, 64)) == bad
    assert _norm_rope(B, T=0) == B.MOE_OK


def _packed(B, n=2, Tq=10, Tk=10, mq=8, mk=8, causal=1, cu=FAKE):
    return B.MoePacked(n, Tq, Tk, mq, mk, causal, cu, cu)


def test_attention_refusals(B):
    bad, shape, mis = B.MOE_ERR_INVALID_ARG, B.MOE_ERR_UNSUPPORTED_SHAPE, B.MOE_ERR_MISALIGNED
    a = B.MoeAttnShape(4, 2, 64)
    q, k = _heads(B, 256, 64), _heads(B, 128, 64)

    def fwd(a=a, s=None, scale=0.125, q=q, k=k, v=k, out=q, lse=FAKE):
        return B.LIB.moe_attention_forward(a, s or _packed(B), scale, q, k, v, out, lse, None)

    assert fwd(a=B.MoeAttnShape(4, 3, 64)) == shape
    assert fwd(s=_packed(B, n=-1)) == bad
    assert fwd(s=_packed(B, n=70000)) == shape
    assert fwd(s=_packed(B, causal=2)) == bad
    assert fwd(s=_packed(B, cu=None)) == bad
    assert fwd(s=_packed(B, Tk=-5)) == bad
    assert fwd(scale=0.0) == bad and fwd(scale=float("inf")) == bad and fwd(scale=-1.0) == bad
    assert fwd(lse=None) == bad and fwd(lse=FAKE + 4) == mis
    assert fwd(v=_heads(B, 128, 64, FAKE + 8)) == mis
    assert fwd(out=_heads(B, 64, 64)) == bad
    assert fwd(s=_packed(B, Tq=0)) == B.MOE_OK and fwd(s=_packed(B, n=0)) == B.MOE_OK

    def bwd(ws=FAKE, size=1 << 20, dk=k, lse=FAKE):
        return B.LIB.moe_attention_backward(a, _packed(B), 0.125, q, q, k, k, q, lse, q, dk, k, ws,
                                            size, None)

    need = B.moe_attention_backward_workspace_size(a, _packed(B))
    assert need >= 10 * 4 * 4
    assert bwd(size=need - 1) == B.MOE_ERR_WORKSPACE_TOO_SMALL
    assert bwd(ws=None) == bad and bwd(lse=None) == bad and bwd(ws=FAKE + 8) == mis
    assert bwd(dk=_heads(B, 64, 64)) == bad


def test_cache_refusals(B):
    bad, shape, mis = B.MOE_ERR_INVALID_ARG, B.MOE_ERR_UNSUPPORTED_SHAPE, B.MOE_ERR_MISALIGNED
    a = B.MoeAttnShape(4, 2, 64)
    q, k = _heads(B, 256, 64), _heads(B, 128, 64)
    rope = B.MoeRope(FAKE, 10, 64, 0)

    def app(cache, slots=FAKE, T=3):
        return B.LIB.moe_kv_append(a, T, q, k, k, FAKE, FAKE, 1e-6, FAKE, rope, slots, q, cache,
                                   None)

    def cache(k=FAKE, v=FAKE, pages=5, size=16):
        return B.MoeKvCache(k, v, pages, size)

    assert app(cache(k=None)) == bad and app(cache(v=FAKE + 8)) == mis
    assert app(cache(pages=0)) == bad
    for size in (4, 24, 512):
        assert app(cache(size=size)) == shape
    assert app(cache(pages=1 << 23, size=256)) == shape      # 2^32 rows
    assert app(cache(), slots=None) == bad and app(cache(), slots=FAKE + 4) == mis
    assert app(cache(), T=0) == B.MOE_OK

    def dec(batch=2, n=1, max_kv=60, scale=0.125, table=FAKE, stride=4, lens=FAKE, ws=FAKE,
            size=1 << 24, c=None):
        return B.LIB.moe_attention_decode(a, batch, n, max_kv, scale, q, c or cache(), table,
                                          stride, lens, q, ws, size, None)

    assert dec(batch=-1) == bad and dec(n=0) == bad and dec(max_kv=-1) == bad
    assert dec(max_kv=65) == bad                             # four pages of 16 a sequence
    assert dec(table=None) == bad and dec(lens=None) == bad and dec(scale=0.0) == bad
    assert dec(batch=1 << 20, n=32) == shape
    assert dec(c=cache(size=12)) == shape
    assert dec(batch=0) == B.MOE_OK
    need = B.moe_attention_decode_workspace_size(a, 2, 1, 60)
    if need:
        assert dec(size=need - 1) == B.MOE_ERR_WORKSPACE_TOO_SMALL and dec(ws=None) == bad


def test_frequencies():
    from token_dispatch_grouped_gb300.attention import rope_inv_freq
    f, s = rope_inv_freq(64)
    assert s == 1.0 and f[0] == 1.0 and abs(float(f[16]) - 0.01) < 1e-15
    g, _ = rope_inv_freq(64, scaling="linear", factor=4.0)
    assert np.allclose(g, f / 4)
    g, _ = rope_inv_freq(64, scaling="ntk", factor=4.0)
    assert g[0] == f[0] and abs(float(g[-1] / f[-1]) - 0.25) < 1e-12
    g, s = rope_inv_freq(64, scaling="yarn", factor=4.0, original=2048)
    assert abs(s - (0.1 * math.log(4) + 1)) < 1e-15
    assert np.allclose(g[:8], f[:8]) and np.allclose(g[-4:], f[-4:] / 4)
    assert ((g <= f) & (g >= f / 4)).all()
    with pytest.raises(ValueError):
        rope_inv_freq(64, scaling="other")
    with pytest.raises(ValueError):
        rope_inv_freq(63)


def test_integers_off_their_alignment_are_refused(B):
    """int32 arrays are read as words: an address that is no multiple of 4 is refused on
    the host, before any launch."""
    mis, a = B.MOE_ERR_MISALIGNED, B.MoeAttnShape(4, 2, 64)
    q, k = _heads(B, 256, 64), _heads(B, 128, 64)
    rope, cache = B.MoeRope(FAKE, 10, 64, 0), B.MoeKvCache(FAKE, FAKE, 5, 16)
    for off in (1, 2, 3):
        at = FAKE + off
        assert _norm_rope(B, pos=at) == mis
        assert B.LIB.moe_norm_rope_backward(a, 3, q, k, q, k, FAKE, FAKE, 1e-6, at, rope, q, k,
                                            FAKE, FAKE, FAKE, 1 << 24, None) == mis
        assert B.LIB.moe_kv_append(a, 3, q, k, k, FAKE, FAKE, 1e-6, at, rope, FAKE, q, cache,
                                   None) == mis
        for s in (B.MoePacked(2, 10, 10, 8, 8, 1, at, FAKE), B.MoePacked(2, 10, 10, 8, 8, 1, FAKE, at)):
            assert B.LIB.moe_attention_forward(a, s, 0.125, q, k, k, q, FAKE, None) == mis
            assert B.LIB.moe_attention_backward(a, s, 0.125, q, q, k, k, q, FAKE, q, k, k, FAKE,
                                                1 << 20, None) == mis
        for table, lens in ((at, FAKE), (FAKE, at)):
            assert B.LIB.moe_attention_decode(a, 2, 1, 60, 0.125, q, cache, table, 4, lens, q, FAKE,
                                              1 << 24, None) == mis
