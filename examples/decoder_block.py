"""One decoder block around the MoE layer: trained on a packed batch, then served token by
token from a paged cache.

    python examples/decoder_block.py

A block is x1 = x + attention(x), x2 = x1 + moe(x1). The projections are plain matrix
products; everything between them runs in the library: norm and rotary positions of the
heads, attention over the packed sequences (and its backward), and the MoE layer. Serving
appends each new token's keys and values to pages, attends over them and runs the layer on
the result; its outputs are compared with the packed forward's.
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))


class Block:
    """Weights of the block, random: d wide, Hq query heads on Hkv key/value heads of D
    values, E experts of width h, K of them per token."""

    def __init__(self, d=1024, Hq=8, Hkv=2, D=128, E=8, K=2, h=512, positions=4096, seed=0):
        from token_dispatch_grouped_gb300.attention import Attention, rope_inv_freq, rope_table
        g = torch.Generator(device="cuda").manual_seed(seed)

        def rand(*shape, std):
            return torch.randn(*shape, generator=g, device="cuda") * std

        self.d, self.Hq, self.Hkv, self.D, self.E, self.K, self.h = d, Hq, Hkv, D, E, K, h
        self.Wqkv = rand((Hq + 2 * Hkv) * D, d, std=d ** -0.5).bfloat16()
        self.Wo = rand(d, Hq * D, std=(Hq * D) ** -0.5).bfloat16()
        self.wq, self.wk = 1 + rand(D, std=0.1), 1 + rand(D, std=0.1)
        self.Wg = rand(E, d, std=d ** -0.5)
        self.W1 = rand(E, h, d, std=d ** -0.5).bfloat16()
        self.W3 = rand(E, h, d, std=d ** -0.5).bfloat16()
        self.W2 = rand(E, d, h, std=h ** -0.5).bfloat16()
        inv, scale = rope_inv_freq(D, scaling="yarn", factor=4.0, original=positions // 4)
        self.att = Attention(Hq, Hkv, D, rope_table=rope_table(positions, inv, scale))

    def heads(self, x):
        """Queries, keys and values of the fused projection, in place."""
        y = (x @ self.Wqkv.T).view(-1, self.Hq + 2 * self.Hkv, self.D)
        return y, y[:, :self.Hq], y[:, self.Hq:self.Hq + self.Hkv], y[:, self.Hq + self.Hkv:]

    def moe(self, T):
        from token_dispatch_grouped_gb300.layer import MoELayer
        return MoELayer(T, self.d, self.E, self.K, self.h)

    def experts(self, layer, x1):
        """moe(x1) and what its backward takes: the routing, its index and H."""
        r = layer.route(x1, self.Wg)
        dp = layer.dispatch(r.ids)
        y, H = layer.forward(x1, self.W1, self.W3, self.W2, r, dp)
        return y, r, dp, H

    # --------------------------------------------------------------- training
    def step(self, x, dy, cu, longest, positions):
        """Output and gradients of one training step on a packed batch [T, d]."""
        a, T = self.att, x.shape[0]
        qkv, q, k, v = self.heads(x)
        qr, kr = a.norm_rope(q, k, self.wq, self.wk, positions)
        o, lse = a.forward(qr, kr, v, cu, longest)
        x1 = x + o.view(T, -1) @ self.Wo.T
        layer = self.moe(T)
        y, r, dp, H = self.experts(layer, x1)

        g = layer.backward(dy, x1, self.Wg, self.W1, self.W3, self.W2, r, dp, H)
        dx1 = dy + g["dx"]
        dWo = dx1.T @ o.view(T, -1)
        do = (dx1 @ self.Wo).view(T, self.Hq, self.D)
        dqkv = torch.empty_like(qkv)     # the gradients land in the fused projection's layout
        dq, dk, _ = a.backward(do, qr, kr, v, o, lse, cu, longest, dv=dqkv[:, self.Hq + self.Hkv:])
        _, _, dwq, dwk = a.norm_rope_backward(dq, dk, q, k, self.wq, self.wk, positions,
                                              dq=dqkv[:, :self.Hq],
                                              dk=dqkv[:, self.Hq:self.Hq + self.Hkv])
        dqkv = dqkv.view(T, -1)
        grads = dict(g, dx=dx1 + dqkv @ self.Wqkv, dWqkv=dqkv.T @ x, dWo=dWo, dwq=dwq, dwk=dwk)
        a.check_error()
        return x1 + y, grads

    # ---------------------------------------------------------------- serving
    def attend_new(self, x, positions, slots, k_pages, v_pages, block_table, kv_lens, max_kv):
        """x1 of the newest token of every sequence."""
        _, q, k, v = self.heads(x)
        q = self.att.append(q, k, v, self.wq, self.wk, positions, slots, k_pages, v_pages)
        o = self.att.decode(q, k_pages, v_pages, block_table, kv_lens, max_kv)
        return x + o.view(x.shape[0], -1) @ self.Wo.T

    def serve(self, layer, x, *cache):
        """The block's output for the newest token of every sequence, with x1 and the
        experts. layer: of as many tokens, kept by the caller."""
        x1 = self.attend_new(x, *cache)
        y, r, _, _ = self.experts(layer, x1)
        return x1 + y, x1, r.ids


def main():
    b = Block()
    lens = [300, 37, 512]
    T, n = sum(lens), len(lens)
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(T, b.d, generator=g, device="cuda").bfloat16()
    dy = torch.randn(T, b.d, generator=g, device="cuda").bfloat16()
    at = [sum(lens[:i]) for i in range(n + 1)]
    cu = torch.tensor(at, dtype=torch.int32, device="cuda")
    pos = torch.cat([torch.arange(m, dtype=torch.int32, device="cuda") for m in lens])
    y, grads = b.step(x, dy, cu, max(lens), pos)
    print("trained one step:", {k: tuple(t.shape) for k, t in grads.items() if t is not None})
    assert all(bool(torch.isfinite(t.float()).all()) for t in grads.values() if t is not None)

    # the packed forward's x1 and experts, to compare the served tokens with
    _, q, k, v = b.heads(x)
    qr, kr = b.att.norm_rope(q, k, b.wq, b.wk, pos)
    x1 = x + b.att.forward(qr, kr, v, cu, max(lens))[0].view(T, -1) @ b.Wo.T
    ids = b.moe(T).route(x1, b.Wg).ids

    # serve the last `new` tokens of every sequence: the prompt enters the pages at once
    page, new = 64, 5
    need = [-(-m // page) for m in lens]
    table = torch.zeros(n, max(need), dtype=torch.int32, device="cuda")
    order = torch.randperm(sum(need), generator=g, device="cuda").to(torch.int32)
    for i, m in enumerate(need):
        table[i, :m] = order[sum(need[:i]):sum(need[:i]) + m]
    k_pages = torch.zeros(sum(need), b.Hkv, page, b.D, dtype=torch.bfloat16, device="cuda")
    v_pages = torch.zeros_like(k_pages)

    def slots(seq, tok):
        return table[seq, tok // page].long() * page + tok % page

    seq = torch.cat([torch.full((m,), i, device="cuda") for i, m in enumerate(lens)])
    last = torch.tensor(lens, device="cuda")[seq]
    prompt = pos < last - new
    _, q, k, v = b.heads(x)
    slot = torch.where(prompt, slots(seq, pos.long()), -1)   # -1: not stored
    b.att.append(q, k, v, b.wq, b.wk, pos, slot, k_pages, v_pages)
    worst, same, layer = 0.0, 0, b.moe(n)

    def off(got, ref):
        return float((got.float() - ref.float()).norm() / ref.float().norm())

    for i in range(new):
        p = torch.tensor(lens, device="cuda") - new + i
        rows = cu[:-1].long() + p
        got, got1, to = b.serve(layer, x[rows], p.to(torch.int32),
                                slots(torch.arange(n, device="cuda"), p), k_pages, v_pages,
                                table, (p + 1).to(torch.int32), max(lens))
        worst = max(worst, off(got1, x1[rows]))
        # (experts whose scores are closer than x1's rounding may change places)
        for j in (to.sort(1)[0] == ids[rows].sort(1)[0]).all(1).nonzero().flatten().tolist():
            worst, same = max(worst, off(got[j], y[rows[j]])), same + 1
    b.att.check_error()
    print(f"served {new} tokens of {n} sequences through the block: relative difference to the "
          f"packed forward {worst:.1e}, the same experts for {same} of {new * n}")
    assert worst < 1e-2 and same >= 0.8 * new * n
    return worst


if __name__ == "__main__":
    main()
