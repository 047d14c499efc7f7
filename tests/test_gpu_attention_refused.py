"""One refused row, sequence or page beside good ones: the others keep every bit, in the call
that meets it and in calls that find the status already set."""
import pytest
import torch

from test_gpu_attention import (attention_data, clean_status, norm_rope_data,  # noqa: F401
                                offsets, paged, rnd)

pytestmark = pytest.mark.gpu


def test_one_bad_position_leaves_the_other_rows():
    """norm_rope and its gradient over many waves of CTAs: every other row is what it is
    without the bad one, and the weights' gradients are the sums without it."""
    from token_dispatch_grouped_gb300 import binding as B
    T, Hq, Hkv, D = 60000, 4, 2, 64
    att, qkv, (wq, wk), _, pos, _ = norm_rope_data((T, Hq, Hkv, D, D, "half", True), 41)
    q, k = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv]
    gq, gk = rnd((T, Hq, D), 42).cuda(), rnd((T, Hkv, D), 43).cuda()
    want = att.norm_rope(q, k, wq, wk, pos)
    at, keep = 1, torch.arange(T, device="cuda") != 1
    # a row whose upstream gradient is zero adds nothing to the weights' gradients
    zq, zk = gq.clone(), gk.clone()
    zq[at], zk[at] = 0, 0
    want_g = att.norm_rope_backward(zq, zk, q, k, wq, wk, pos)
    bad = pos.clone()
    bad[at] = 500
    for _ in range(2):                      # the second call finds the status already set
        got = att.norm_rope(q, k, wq, wk, bad, q_out=torch.zeros_like(gq),
                            k_out=torch.zeros_like(gk))
        for a, b in zip(got, want):
            assert torch.equal(a[keep], b[keep])
        got = att.norm_rope_backward(gq, gk, q, k, wq, wk, bad, dq=torch.zeros_like(gq),
                                     dk=torch.zeros_like(gk))
        for a, b in zip(got[:2], want_g[:2]):
            assert torch.equal(a[keep], b[keep])
        for a, b in zip(got[2:], want_g[2:]):
            assert torch.equal(a, b)
    assert B.moe_get_error() == B.MOE_ERR_BAD_INDEX


@pytest.mark.parametrize("wrong", ["long", "past"])
def test_one_bad_sequence_leaves_the_others(wrong):
    from token_dispatch_grouped_gb300 import binding as B
    att, lq, lk, q, k, v, do = attention_data(([700, 300, 500, 90], None, 4, 2, 64, True), 45)
    n = 1500 if wrong == "past" else 700     # rows of the good sequences
    T = sum(lq) - (0 if wrong == "long" else 90)
    q, k, v, do = (x[:T] for x in (q, k, v, do))
    good = offsets(lq[:3] if wrong == "past" else lq)
    out, lse = att.forward(q, k, v, good, 700)
    grads = att.backward(do, q, k, v, out, lse, good, 700)
    # the last sequence passes the arrays, or the first is longer than stated
    bad, longest = (offsets(lq), 700) if wrong == "past" else (good, 500)
    rows = slice(0, n) if wrong == "past" else slice(700, T)
    for _ in range(2):
        o, l = (torch.zeros_like(x) for x in (out, lse))
        att.forward(q, k, v, bad, longest, out=o, lse=l)
        assert torch.equal(o[rows], out[rows]) and torch.equal(l[rows], lse[rows])
        g = att.backward(do, q, k, v, out, lse, bad, longest,
                         **{m: torch.zeros_like(x) for m, x in zip(("dq", "dk", "dv"), grads)})
        for a, b in zip(g, grads):
            assert torch.equal(a[rows], b[rows])
    assert B.moe_get_error() == B.MOE_ERR_BAD_INDEX


@pytest.mark.parametrize("wrong", ["page", "length"])
def test_one_bad_page_leaves_the_other_sequences(wrong):
    """Sequences long enough that their tokens are split and joined."""
    from token_dispatch_grouped_gb300 import binding as B
    from token_dispatch_grouped_gb300.attention import Attention
    att, lens, page = Attention(8, 2, 64), [1500, 900, 3, 0, 1200], 16
    k, v = rnd((sum(lens), 2, 64), 51), rnd((sum(lens), 2, 64), 52)
    q = rnd((len(lens), 8, 64), 53).cuda()
    kp, vp, table, _ = paged(k, v, lens, page)
    kv = torch.tensor(lens, dtype=torch.int32, device="cuda")
    assert B.moe_attention_decode_workspace_size(att.a, len(lens), 1, 1500) > 0   # split
    want = att.decode(q, kp, vp, table, kv, 1500)
    table, kv = table.clone(), kv.clone()
    if wrong == "page":
        table[1, 50] = kp.shape[0]
    else:
        kv[1] = 1501
    keep = [0, 2, 3, 4]
    for _ in range(2):
        got = att.decode(q, kp, vp, table, kv, 1500, out=torch.full_like(want, 7))
        assert torch.equal(got[keep], want[keep])
    assert B.moe_get_error() == B.MOE_ERR_BAD_INDEX
