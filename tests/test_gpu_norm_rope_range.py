"""norm_rope's gradient over the range of magnitudes that bf16 and its fp32 squares hold."""
import numpy as np
import pytest
import torch

from oracle import attention as O
from test_gpu_attention import clean_status, f64, rnd, within  # noqa: F401

pytestmark = pytest.mark.gpu


def test_norm_rope_gradient_of_small_and_large_heads():
    """Heads of magnitudes whose cubed norm leaves the range of fp32, where the gradient
    itself is well inside it."""
    for std, eps in ((2.0 ** -50, 0.0), (2.0 ** 50, 1e-6)):
        T, H, D = 40, 2, 64
        from token_dispatch_grouped_gb300.attention import Attention
        att = Attention(H, H, D, eps=eps)
        q, k = rnd((T, H, D), 61, std).cuda(), rnd((T, H, D), 62, std).cuda()
        gq, gk = rnd((T, H, D), 63).cuda(), rnd((T, H, D), 64).cuda()
        w = 1 + 0.2 * torch.randn(D, generator=torch.Generator().manual_seed(1))
        zero = np.zeros((T, 0))
        got = att.norm_rope_backward(gq, gk, q, k, w.cuda(), w.cuda(), None)
        for i, (x, g) in enumerate(((q, gq), (k, gk))):
            x, g, n = f64(x), f64(g), f64(w)
            dx, dw = O.norm_rope_backward(g, x, n, eps, zero, zero, False)
            r = 1 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
            mag = r * (np.abs(g * n) + np.abs(x * r) * np.abs(g * n * x * r).mean(-1, keepdims=True))
            within(got[i], dx, O.U * np.abs(dx) + 2.0 ** -16 * mag.max(-1, keepdims=True), "dx")
            within(got[2 + i], dw, 2.0 ** -16 * np.abs(g * x * r).sum((0, 1)), "dw")
