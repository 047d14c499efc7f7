"""Packed attention beyond one wave of key tiles, and its backward at large scores, against
the fp64 oracle."""
import numpy as np
import pytest
import torch

from oracle import attention as O
from test_gpu_attention import (attention_data, check_all, clean_status, f64,  # noqa: F401
                                offsets, reference, within)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("case", [
    ([2500, 1], None, 2, 1, 128, True), ([1, 1300], [5000, 1290], 4, 2, 64, True),
    ([1100, 3], [2049, 1], 3, 1, 96, False), ([2100], None, 5, 1, 64, True)])
def test_sequences_of_thousands_of_tokens(case):
    causal = case[5]
    att, lq, lk, q, k, v, do = attention_data(case, 81)
    cq, ck, mq, mk = offsets(lq), offsets(lk), max(lq), max(lk)
    out, lse = att.forward(q, k, v, cq, mq, ck, mk, causal=causal)
    grads = att.backward(do, q, k, v, out, lse, cq, mq, ck, mk, causal=causal)
    check_all(out, lse, grads, *reference(att, lq, lk, q, k, v, do, causal))


@pytest.mark.parametrize("case", [([90], None, 4, 2, 64, True), ([400], None, 4, 2, 64, True),
                                  ([300, 41], [20, 400], 6, 2, 80, True)])
def test_gradients_at_large_scores(case):
    """Scores of some hundreds, rows whose maximum comes late. A score's fp32 error of
    s 2^-20 is a relative error d of its weight, which reaches dv as it is, dS with dS, and
    delta twice (through the weight and the sum) with the magnitudes it adds."""
    causal = case[5]
    att, lq, lk, q, k, v, do = attention_data(case, 83, std=12.0)
    k[sum(lk) * 3 // 4:] *= 2
    cq, ck, mq, mk = offsets(lq), offsets(lk), max(lq), max(lk)
    out, lse = att.forward(q, k, v, cq, mq, ck, mk, causal=causal)
    got = att.backward(do, q, k, v, out, lse, cq, mq, ck, mk, causal=causal)
    r, b = reference(att, lq, lk, q, k, v, do, causal)
    nq, nk, nv, nd = (f64(x) for x in (q, k, v, do))
    d = np.abs(nq).sum(-1).max() * np.abs(nk).max() * att.scale * 2.0 ** -20
    G, a0, b0 = att.Hq // att.Hkv, 0, 0
    for n, m in zip(lq, lk):
        a, c = slice(a0, a0 + n), slice(b0, b0 + m)
        a0, b0 = a0 + n, b0 + m
        for h in range(att.Hq):
            g = h // G
            p = O.attention(nq[a, h], nk[c, g], nv[c, g], att.scale, causal)[2]
            ds = O.attention_backward(nd[a, h], nq[a, h], nk[c, g], nv[c, g], p, att.scale)[3]
            add = (np.abs(nd[a, h]) * (p @ np.abs(nv[c, g]))).sum(-1, keepdims=True)
            e = d * np.abs(ds) + 2 * d * p * add
            b["out"][a, h] += 2 * d * p @ np.abs(nv[c, g])
            b["dq"][a, h] += att.scale * e @ np.abs(nk[c, g])
            b["dk"][c, g] += att.scale * e.T @ np.abs(nq[a, h])
            b["dv"][c, g] += d * p.T @ np.abs(nd[a, h])
    within(out, r["out"], b["out"], "out")
    for n, x in zip(("dq", "dk", "dv"), got):
        within(x, r[n], b[n], n)
