"""Stated bounds of the sequences' lengths: any value that is no smaller than the longest."""
import pytest
import torch

from test_gpu_attention import attention_data, clean_status, offsets  # noqa: F401

pytestmark = pytest.mark.gpu
MOST = 2 ** 31 - 1


@pytest.mark.parametrize("max_q,max_k", [(MOST, MOST), (MOST, 300), (200, MOST), (1 << 20, 1 << 24)])
@pytest.mark.parametrize("D", [64, 128])
def test_large_bounds_change_nothing(max_q, max_k, D):
    att, lq, lk, q, k, v, do = attention_data(([200, 0, 33], [300, 5, 33], 6, 2, D, True), 71)
    cq, ck = offsets(lq), offsets(lk)
    out, lse = att.forward(q, k, v, cq, 200, ck, 300)
    want = (out, lse) + att.backward(do, q, k, v, out, lse, cq, 200, ck, 300)
    out, lse = att.forward(q, k, v, cq, max_q, ck, max_k, out=torch.zeros_like(q))
    got = (out, lse) + att.backward(do, q, k, v, out, lse, cq, max_q, ck, max_k,
                                    dq=torch.zeros_like(q), dk=torch.zeros_like(k),
                                    dv=torch.zeros_like(v))
    for a, b in zip(got, want):
        assert torch.equal(a, b)


def test_bounds_of_zero():
    """Empty sequences only: nothing is done. A sequence that is longer is reported."""
    from token_dispatch_grouped_gb300 import binding as B
    att, lq, lk, q, k, v, do = attention_data(([20, 30], None, 4, 2, 64, True), 73)
    lse = torch.zeros(50, 4, device="cuda")
    for cu, status in ((torch.zeros(3, dtype=torch.int32, device="cuda"), B.MOE_OK),
                       (offsets(lq), B.MOE_ERR_BAD_INDEX)):
        out, _ = att.forward(q, k, v, cu, 0, out=torch.full_like(q, 7))
        assert B.moe_get_error() == status and (out == 7).all()
        g = att.backward(do, q, k, v, q, lse, cu, 0,
                         **{n: torch.full_like(x, 7) for n, x in (("dq", q), ("dk", k), ("dv", v))})
        assert B.moe_get_error() == status and all((x == 7).all() for x in g)
