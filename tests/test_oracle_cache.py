"""The oracle of the small cache against torch and by its properties, and what the entry points
refuse on the host: no call here reaches a GPU."""
import numpy as np
import pytest
import torch

from oracle import cache as C

FAKE = 1 << 20   # a pointer that no refused call follows


@pytest.fixture(scope="module")
def B():
    from token_dispatch_grouped_gb300 import build
    build.build()
    from token_dispatch_grouped_gb300 import binding
    return binding


def test_e4m3_is_the_format_of_torch():
    every = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double()
    fine = every[every.isfinite()].numpy()
    assert np.array_equal(C.e4m3(fine), fine) and fine.max() == C.TOP
    x = np.sort(fine)
    x = np.concatenate([x, (x[1:] + x[:-1]) / 2, np.random.default_rng(0).uniform(-448, 448, 5000),
                        np.random.default_rng(1).uniform(-0.02, 0.02, 5000)]).astype(np.float32)
    assert np.array_equal(C.e4m3(x), torch.from_numpy(x).to(torch.float8_e4m3fn).double().numpy())
    assert (np.abs(C.e4m3(x) - x) <= C.half_step(x.astype(np.float64), 1.0)).all()


def test_scale_of_a_page():
    assert C.power(448.0) == 1 and C.power(448.1) == 2 and C.power(224.0) == 0.5
    assert C.power(0.0) == 2.0 ** -100 and C.power(3e38) == 2.0 ** 120
    assert C.finite_top(np.array([1.0, -np.inf, np.nan, -3.0])) == 3.0


def test_a_grown_scale_rounds_normal_values_once():
    """Rows that move to a scale 2^k times larger are what a first write with it gives, but
    for values below its normal range, which may be a half step off."""
    x = np.random.default_rng(2).standard_normal((64, 16)) * 300
    page, one = C.append8(np.zeros((80, 16)), 0.0, 0, x)
    page, s = C.append8(page, one, 64, np.full((1, 16), 448.0 * 8 * one))
    want = C.e4m3(x / s)
    assert s == 8 * one
    big = np.abs(x / s) >= 2.0 ** -6
    assert np.array_equal(page[:64][big], want[big]) and big.mean() > 0.9
    assert np.abs(page[:64] - want).max() <= 2.0 ** -9


def test_kept_tokens():
    w = np.array([5, 1, 5, np.nan, 5, 0, 9, 2, 2], dtype=np.float32)
    assert list(C.kept(w, 4, 2)) == [0, 6, 7, 8]
    assert list(C.kept(w, 5, 2)) == [0, 2, 6, 7, 8]
    assert list(C.kept(w, 9, 2)) == list(range(9)) and list(C.kept(w, 3, 3)) == [6, 7, 8]
    assert list(C.kept(np.array([np.nan, -np.inf, np.nan]), 2, 0)) == [0, 1]


def _heads(B, ts, hs, at=FAKE):
    return B.MoeHeads(at, ts, hs)


def test_append8_refusals(B):
    bad, shape, mis = B.MOE_ERR_INVALID_ARG, B.MOE_ERR_UNSUPPORTED_SHAPE, B.MOE_ERR_MISALIGNED
    q, k = _heads(B, 256, 64), _heads(B, 128, 64)

    def cache(k=FAKE, v=FAKE, ks=FAKE, vs=FAKE, pages=5, size=16):
        return B.MoeKv8Cache(k, v, ks, vs, pages, size)

    def app(a=B.MoeAttnShape(4, 2, 64), batch=2, T=3, max_kv=60, c=None, cu=FAKE, table=FAKE,
            stride=4, lens=FAKE, k=k, q_out=q, w=FAKE, pos=FAKE):
        rope = B.MoeRope(FAKE, 10, 64, 0)
        return B.LIB.moe_kv8_append(a, batch, T, max_kv, q, k, k, w, FAKE, 1e-6, pos, rope, cu,
                                    table, stride, lens, q_out, c or cache(), None)

    assert app(a=B.MoeAttnShape(4, 2, 56)) == shape          # rows of 16 bytes
    assert app(a=B.MoeAttnShape(4, 3, 64)) == shape
    assert app(batch=-1) == bad and app(max_kv=-1) == bad and app(T=-1) == bad
    assert app(batch=70000) == shape and app(max_kv=(1 << 30) + 1) == shape
    assert app(c=cache(ks=None)) == bad and app(c=cache(vs=FAKE + 2)) == mis
    assert app(c=cache(k=FAKE + 8)) == mis and app(c=cache(size=24)) == shape
    assert app(cu=None) == bad and app(table=None) == bad and app(lens=None) == bad
    assert app(cu=FAKE + 1) == mis and app(table=FAKE + 2) == mis and app(lens=FAKE + 3) == mis
    assert app(max_kv=65) == bad and app(stride=-1) == bad   # four pages of 16 a sequence
    assert app(k=_heads(B, 0, 64)) == bad and app(q_out=_heads(B, 64, 64)) == bad
    assert app(w=None) == bad and app(pos=None) == bad
    assert app(T=0) == B.MOE_OK
    for same in (cache(), cache(v=FAKE + 4096), cache(vs=FAKE + 4096)):   # one array for both
        assert app(c=same) == bad


def test_decode_refusals(B):
    bad, shape, mis = B.MOE_ERR_INVALID_ARG, B.MOE_ERR_UNSUPPORTED_SHAPE, B.MOE_ERR_MISALIGNED
    a, q = B.MoeAttnShape(4, 2, 64), _heads(B, 256, 64)
    full = B.MoeKvCache(FAKE, FAKE, 5, 16)
    small = B.MoeKv8Cache(FAKE, FAKE, FAKE, FAKE, 5, 16)

    def dec(eight, a=a, batch=2, n=1, max_kv=60, scale=0.125, table=FAKE, stride=4, lens=FAKE,
            weights=FAKE, fresh=0, ws=FAKE, size=1 << 24, c=None):
        f, c = (B.LIB.moe_attention_decode8, c or small) if eight else \
            (B.LIB.moe_attention_decode_weights, c or full)
        return f(a, batch, n, max_kv, scale, q, c, table, stride, lens, weights, fresh, q, ws, size,
                 None)

    for e in (True, False):
        assert dec(e, batch=-1) == bad and dec(e, n=0) == bad and dec(e, max_kv=-1) == bad
        assert dec(e, max_kv=65) == bad and dec(e, scale=-1.0) == bad and dec(e, fresh=2) == bad
        assert dec(e, table=None) == bad and dec(e, lens=None) == bad and dec(e, lens=FAKE + 2) == mis
        assert dec(e, weights=FAKE + 8) == mis and dec(e, batch=1 << 20, n=32) == shape
        assert dec(e, batch=0) == B.MOE_OK
        need = B.moe_attention_decode8_workspace_size(a, 2, 1, 60, 1) if e else \
            B.moe_attention_decode_weights_workspace_size(a, 2, 1, 60)
        assert need >= 2 * 4 * 64 * 4                        # the scores of 8 rows
        assert dec(e, size=need - 1) == B.MOE_ERR_WORKSPACE_TOO_SMALL and dec(e, ws=None) == bad
    assert dec(False, weights=None) == bad
    assert dec(True, a=B.MoeAttnShape(4, 2, 40)) == shape
    assert dec(True, c=B.MoeKv8Cache(FAKE, FAKE, FAKE, None, 5, 16)) == bad
    assert B.moe_attention_decode8_workspace_size(B.MoeAttnShape(4, 2, 40), 2, 1, 60, 1) == 0


def test_evict_refusals(B):
    bad, shape, mis = B.MOE_ERR_INVALID_ARG, B.MOE_ERR_UNSUPPORTED_SHAPE, B.MOE_ERR_MISALIGNED

    def ev(eight, a=B.MoeAttnShape(4, 2, 64), batch=2, max_kv=60, keep=20, recent=4, weights=FAKE,
           table=FAKE, stride=4, lens=FAKE, goal=FAKE, goal_stride=2, new=FAKE, kept=FAKE, size=16):
        if eight:
            f, c = B.LIB.moe_kv8_evict, B.MoeKv8Cache(FAKE, FAKE, FAKE, FAKE, 5, size)
        else:
            f, c = B.LIB.moe_kv_evict, B.MoeKvCache(FAKE, FAKE, 5, size)
        return f(a, batch, max_kv, keep, recent, c, weights, table, stride, lens, goal,
                 goal_stride, new, kept, None)

    for e in (True, False):
        assert ev(e, batch=-1) == bad and ev(e, keep=0) == bad and ev(e, recent=-1) == bad
        assert ev(e, recent=21) == bad and ev(e, max_kv=-1) == bad and ev(e, max_kv=65) == bad
        assert ev(e, goal_stride=1) == bad and ev(e, max_kv=(1 << 30) + 1) == shape
        for name in ("weights", "table", "lens", "goal", "new", "kept"):
            assert ev(e, **{name: None}) == bad, name
            assert ev(e, **{name: FAKE + 2}) == mis, name
        assert ev(e, weights=FAKE + 8) == mis and ev(e, size=20) == shape
        assert ev(e, batch=0) == B.MOE_OK
    assert ev(True, a=B.MoeAttnShape(4, 2, 24)) == shape


def test_wrong_tensors_are_refused(B):
    """What the class refuses before it calls: tensors on the CPU among them."""
    from token_dispatch_grouped_gb300.attention import Attention
    att = Attention(4, 2, 64, device="cpu")
    k8 = torch.zeros(5, 2, 16, 64).to(torch.float8_e4m3fn)
    k16, s = torch.zeros(5, 2, 16, 64, dtype=torch.bfloat16), torch.zeros(5, 2)
    q, t = torch.zeros(2, 4, 64, dtype=torch.bfloat16), torch.zeros(2, 4, dtype=torch.int32)
    n = torch.ones(2, dtype=torch.int32)
    w = torch.zeros(5, 2, 16)
    for call in (lambda: att.decode8(q, k8, k8, s, s, t, n, 60),
                 lambda: att.decode8(q, k16, k16, s, s, t, n, 60),
                 lambda: att.decode(q, k16, k16, t, n, 60, weights=w),
                 lambda: att.append8(q, q[:, :2], q[:, :2], None, None, n, n, t, n, k8, k8, s, s),
                 lambda: att.evict(k16, k16, w, t, n, 60, 8, 2, t),
                 lambda: att.evict(k8, k8, w, t, n, 60, 8, 2, t, k_scales=s),
                 lambda: att.evict(k8, k8, w, t, n, 60, 8, 9, t, k_scales=s, v_scales=s)):
        with pytest.raises(B.MoeError):
            call()
