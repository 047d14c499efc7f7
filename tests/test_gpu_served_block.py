"""The served path goes through the whole block: paged attention, then the MoE layer."""
import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu


def test_a_served_token_goes_through_the_layer():
    """One new token of each of two sequences after an empty and a cached context: x1 plus
    the experts' weighted sum in fp32 from the served routing."""
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples",
                        "decoder_block.py")
    spec = importlib.util.spec_from_file_location("decoder_block", path)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    b = m.Block(d=256, Hq=4, Hkv=2, D=64, E=4, K=2, h=128, positions=64, seed=3)
    g = torch.Generator(device="cuda").manual_seed(4)
    kp = torch.randn(4, 2, 16, 64, generator=g, device="cuda").bfloat16()
    vp = torch.randn(4, 2, 16, 64, generator=g, device="cuda").bfloat16()
    table = torch.tensor([[0, 1], [2, 3]], dtype=torch.int32, device="cuda")
    x = torch.randn(2, 256, generator=g, device="cuda").bfloat16()
    pos = torch.tensor([0, 20], dtype=torch.int32, device="cuda")
    slots = torch.tensor([0, 3 * 16 + 4], dtype=torch.int64, device="cuda")
    out, x1, ids = b.serve(b.moe(2), x, pos, slots, kp, vp, table, pos + 1, 32)
    b.att.check_error()
    z = x1.float()
    p = (z @ b.Wg.T).softmax(-1)
    want = []
    for t in range(2):
        chosen = ids[t].long()
        assert set(chosen.tolist()) == set(p[t].topk(2).indices.tolist())
        w = p[t, chosen] / p[t, chosen].sum()
        y = sum(wi * ((torch.nn.functional.silu(z[t] @ b.W1[e].float().T) * (z[t] @ b.W3[e].float().T))
                      @ b.W2[e].float().T) for wi, e in zip(w, chosen.tolist()))
        want.append(z[t] + y)
    want = torch.stack(want)
    assert float((out.float() - want).norm() / want.norm()) < 1e-2
