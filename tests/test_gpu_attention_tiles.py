"""The attention forward, bit for bit, whatever stands in the rows of a tile that belong to
no item: queries of the next sequence, or shared memory that no load wrote."""
import pytest
import torch

from test_gpu_attention import attention_data, clean_status, offsets  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("causal", [False, True])
def test_forward_of_a_sequence_does_not_depend_on_the_next(causal):
    """The last tile of a sequence also holds queries of the next one. However large their
    scores are, the bits of the first sequence stay."""
    case = ([37, 60], [1024, 1024], 4, 1, 64, causal)   # rows 0 to 147, the first 20 of a warp
    att, lq, lk, q, k, v, _ = attention_data(case, 31)
    cq, ck = offsets(lq), offsets(lk)
    want = [x[:37].clone() for x in att.forward(q, k, v, cq, 60, ck, 1024, causal=causal)]
    for factor in (30.0, 100.0, 300.0):
        loud = q.clone()
        loud[37:] *= factor
        got = att.forward(loud, k, v, cq, 60, ck, 1024, causal=causal)
        for a, b in zip(got, want):
            assert torch.equal(a[:37], b), factor


@pytest.mark.parametrize("G", [3, 5])
def test_forward_does_not_depend_on_earlier_kernels(G):
    """Where G does not divide 128 a tile's last rows are not loaded and hold what an
    earlier kernel left in shared memory."""
    att, lq, lk, q, k, v, _ = attention_data(([700], [1500], G, 1, 128, False), 33)
    cq, ck = offsets(lq), offsets(lk)
    # items that fill every row of both tiles, on every SM
    other, _, _, q2, k2, v2, _ = attention_data(([64] * 400, None, 4, 1, 128, False), 34)
    c2 = offsets([64] * 400)
    got = []
    for factor in (0.0, 1.0, 30.0, 300.0):
        other.forward(q2 * factor, k2, v2, c2, 64)
        got.append(att.forward(q, k, v, cq, 700, ck, 1500, causal=False))
    for out, lse in got[1:]:
        assert torch.equal(out, got[0][0]) and torch.equal(lse, got[0][1])
