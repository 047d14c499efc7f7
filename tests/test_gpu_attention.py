"""The attention operators against the fp64 oracle, with elementwise bounds (derived in
oracle/attention.py: what bf16 operands and results allow), over packed batches with
empty and odd sequences, grouped heads, strides, masks that leave a row nothing,
non-finite values that must not spread, and device-side refusals."""
import numpy as np
import pytest
import torch

from oracle import attention as O

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def clean_status():
    from token_dispatch_grouped_gb300 import binding as B
    B.moe_get_error()
    yield
    assert B.moe_get_error() == B.MOE_OK


def rnd(shape, seed, std=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=g) * std).to(torch.bfloat16)


def f64(t):
    return t.detach().cpu().double().numpy()


def offsets(lens):
    return torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32, device="cuda")


def within(got, ref, bound, what):
    got = f64(got)
    assert got.shape == ref.shape, what
    off = np.abs(got - ref) - bound
    assert np.isfinite(got).all(), what
    assert (off <= 0).all(), (what, np.unravel_index(off.argmax(), off.shape), off.max())


# ------------------------------------------------------------------ norm and rotation
def table_of(positions, dims, base=10000.0):
    from token_dispatch_grouped_gb300.attention import rope_inv_freq, rope_table
    return rope_table(positions, rope_inv_freq(dims, base)[0])


def test_rope_table_keeps_late_positions():
    from token_dispatch_grouped_gb300.attention import rope_inv_freq, rope_table
    inv, _ = rope_inv_freq(64)
    t = f64(rope_table(200_000, inv, 1.25))
    p = np.array([0, 1, 77, 131071, 199_999])
    ang = p[:, None] * inv.numpy()[None]
    ref = 1.25 * np.stack([np.cos(ang), np.sin(ang)], -1)
    assert np.abs(t[p] - ref).max() <= 1.25 * 2.0 ** -23


NR = [  # T, Hq, Hkv, D, rot, layout, norm
    (1, 1, 1, 8, 8, "half", True), (3, 4, 2, 64, 64, "half", True),
    (17, 8, 8, 64, 32, "interleaved", True), (5, 6, 2, 96, 96, "half", True),
    (33, 5, 1, 80, 40, "half", True), (33, 5, 1, 80, 80, "interleaved", True),
    (7, 3, 3, 128, 128, "half", False), (7, 3, 1, 40, 0, "half", True),
    (130, 32, 8, 128, 128, "half", True), (900, 4, 4, 16, 6, "half", True),
    (9, 12, 4, 120, 2, "interleaved", False), (6000, 2, 1, 128, 64, "half", True),
    (20001, 2, 2, 16, 16, "half", True), (19999, 3, 1, 24, 8, "interleaved", True)]


def norm_rope_data(case, seed=0, fused=True):
    T, Hq, Hkv, D, rot, layout, norm = case
    from token_dispatch_grouped_gb300.attention import Attention
    qkv = rnd((T, Hq + 2 * Hkv, D), seed).cuda()
    g = torch.Generator().manual_seed(seed + 9)
    w = [1 + 0.2 * torch.randn(D, generator=g) for _ in range(2)]
    pos = torch.randint(0, 500, (T,), generator=g, dtype=torch.int32)
    table = table_of(500, rot) if rot else None
    att = Attention(Hq, Hkv, D, eps=1e-5, rope_table=table, rope_layout=layout)
    cs = f64(table)[pos.numpy()] if rot else np.zeros((T, 0, 2))
    return att, qkv, [x.cuda() if norm else None for x in w], \
        [f64(x) if norm else None for x in w], pos.cuda(), cs


@pytest.mark.parametrize("case", NR)
def test_norm_rope(case):
    T, Hq, Hkv, D, rot, layout, norm = case
    att, qkv, (wq, wk), (nq, nk), pos, cs = norm_rope_data(case)
    q, k = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv]          # views with the fused stride
    outs = att.norm_rope(q, k, wq, wk, pos)
    for x, w, o in ((q, nq, outs[0]), (k, nk, outs[1])):
        ref = O.norm_rope(f64(x), w, 1e-5, cs[..., 0], cs[..., 1], layout == "interleaved")
        top = np.abs(ref).max(-1, keepdims=True)
        within(o, ref, O.U * np.abs(ref) + 2.0 ** -16 * top, "norm_rope")
    # in place, head-major outputs: the same bits
    hm = torch.empty(Hq, T, D, dtype=torch.bfloat16, device="cuda").transpose(0, 1)
    x = qkv.clone()
    att.norm_rope(x[:, :Hq], x[:, Hq:Hq + Hkv], wq, wk, pos, q_out=hm, k_out=x[:, Hq:Hq + Hkv])
    assert torch.equal(hm, outs[0]) and torch.equal(x[:, Hq:Hq + Hkv], outs[1])
    assert torch.equal(x[:, Hq + Hkv:], qkv[:, Hq + Hkv:]) and torch.equal(x[:, :Hq], q)


@pytest.mark.parametrize("case", NR)
def test_norm_rope_backward(case):
    T, Hq, Hkv, D, rot, layout, norm = case
    att, qkv, (wq, wk), (nq, nk), pos, cs = norm_rope_data(case, 3)
    q, k = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv]
    gq, gk = rnd((T, Hq, D), 50).cuda(), rnd((T, Hkv, D), 51).cuda()
    got = att.norm_rope_backward(gq, gk, q, k, wq, wk, pos)
    again = att.norm_rope_backward(gq, gk, q, k, wq, wk, pos)
    il = layout == "interleaved"
    for i, (x, g, w) in enumerate(((q, gq, nq), (k, gk, nk))):
        x, g = f64(x), f64(g)
        dx, dw = O.norm_rope_backward(g, x, w, 1e-5, cs[..., 0], cs[..., 1], il)
        dy = O.rotate(g, cs[..., 0], -cs[..., 1], il)
        if norm:
            r = 1 / np.sqrt((x * x).mean(-1, keepdims=True) + 1e-5)
            n = x * r
            mag = r * (np.abs(dy * w) + np.abs(n) * np.abs(dy * w * n).mean(-1, keepdims=True))
        else:
            mag = np.abs(dy)
        top = mag.max(-1, keepdims=True)
        within(got[i], dx, O.U * np.abs(dx) + 2.0 ** -16 * top, "dx")
        if norm:
            within(got[2 + i], dw, 2.0 ** -18 * np.abs(dy * n).sum((0, 1)) + 2.0 ** -16 *
                   np.abs(n).max() * np.abs(dy).max() * 1e-2, "dw")
        else:
            assert got[2 + i] is None
    for a, b in zip(got, again):
        assert a is None or torch.equal(a, b)


def test_norm_rope_no_tokens_and_bad_positions():
    from token_dispatch_grouped_gb300 import binding as B
    att, qkv, (wq, wk), _, pos, _ = norm_rope_data((4, 4, 2, 64, 64, "half", True))
    e = qkv[:0]
    dq, dk, dwq, dwk = att.norm_rope_backward(e[:, :4], e[:, 4:6], e[:, :4], e[:, 4:6], wq, wk,
                                              pos[:0])
    assert dq.shape == (0, 4, 64) and (dwq == 0).all() and (dwk == 0).all()
    good = att.norm_rope(qkv[:, :4], qkv[:, 4:6], wq, wk, pos)
    for wrong in (-1, 500):
        bad = pos.clone()
        bad[2] = wrong
        o = [torch.full_like(x, 7) for x in good]
        att.norm_rope(qkv[:, :4], qkv[:, 4:6], wq, wk, bad, q_out=o[0], k_out=o[1])
        assert B.moe_get_error() == B.MOE_ERR_BAD_INDEX
        assert (o[0][2] == 7).all() and (o[1][2] == 7).all()   # left out


# ------------------------------------------------------------------ packed attention
AT = [  # lens_q, lens_k, Hq, Hkv, D, causal
    ([1], [1], 1, 1, 64, True), ([1], [1], 1, 1, 8, False),
    ([5, 0, 130, 1], None, 4, 2, 64, True), ([5, 0, 130, 1], None, 4, 2, 64, False),
    ([127, 128, 129], None, 2, 1, 128, True), ([257], None, 3, 1, 96, True),
    ([300, 41], [20, 400], 6, 2, 80, True), ([64, 10], [0, 7], 4, 4, 128, True),
    ([64, 10], [0, 7], 4, 4, 128, False), ([33, 70], [300, 5], 8, 1, 40, False),
    ([513], None, 5, 1, 128, True), ([200, 100], None, 16, 1, 64, True),
    ([90], [1000], 10, 2, 128, True), ([700], None, 2, 2, 64, False),
    ([3, 2], [200, 131], 64, 1, 24, True), ([1024], None, 4, 1, 128, True),
    # more items of work than SMs, and more sequences than one warp holds
    ([(7 * i) % 41 for i in range(70)], None, 8, 4, 64, True),
    ([(11 * i) % 150 for i in range(33)], [(13 * i) % 160 for i in range(33)], 6, 6, 40, True),
    ([(5 * i) % 140 + 1 for i in range(32)], [(17 * i) % 300 for i in range(32)], 9, 3, 72, False),
    ([600, 20, 900, 1, 300], None, 16, 4, 128, True)]


def attention_data(case, seed=0, std=1.0):
    lq, lk, Hq, Hkv, D, causal = case
    lk = lq if lk is None else lk
    from token_dispatch_grouped_gb300.attention import Attention
    q, do = rnd((sum(lq), Hq, D), seed, std), rnd((sum(lq), Hq, D), seed + 1)
    k, v = rnd((sum(lk), Hkv, D), seed + 2, std), rnd((sum(lk), Hkv, D), seed + 3)
    return Attention(Hq, Hkv, D), lq, lk, *(x.cuda() for x in (q, k, v, do))


def reference(att, lq, lk, q, k, v, do, causal):
    """Oracle results and bounds of out, lse, dq, dk, dv."""
    G, sc = att.Hq // att.Hkv, att.scale
    q, k, v, do = (f64(x) for x in (q, k, v, do))
    r = {n: np.zeros_like(x) for n, x in (("out", q), ("dq", q), ("dk", k), ("dv", v))}
    r["lse"] = np.full(q.shape[:2], -np.inf)
    b = {n: np.zeros_like(x) for n, x in r.items()}
    a0 = b0 = 0
    for n, m in zip(lq, lk):
        a, c = slice(a0, a0 + n), slice(b0, b0 + m)
        a0, b0 = a0 + n, b0 + m
        for h in range(att.Hq if n and m else 0):
            g = h // G
            out, lse, p = O.attention(q[a, h], k[c, g], v[c, g], sc, causal)
            dq, dk, dv, ds = O.attention_backward(do[a, h], q[a, h], k[c, g], v[c, g], p, sc)
            ob = O.forward_bound(out, v[c, g], p)
            bq, bk, bv = O.backward_bounds(do[a, h], q[a, h], k[c, g], v[c, g], p, ds, out, ob,
                                           dq, dk, dv, sc)
            r["out"][a, h], r["lse"][a, h], r["dq"][a, h] = out, lse, dq
            r["dk"][c, g] += dk
            r["dv"][c, g] += dv
            b["out"][a, h], b["dq"][a, h] = ob, bq
            b["dk"][c, g] += bk
            b["dv"][c, g] += bv
    for n in ("dk", "dv"):
        b[n] += O.U * np.abs(r[n]) + 1e-30
    return r, b


def check_all(out, lse, grads, r, b):
    within(out, r["out"], b["out"], "out")
    fin = np.isfinite(r["lse"])
    got = f64(lse)
    assert np.array_equal(np.isneginf(got), ~fin)
    assert (np.abs(got[fin] - r["lse"][fin]) <= 2.0 ** -16 * (1 + np.abs(r["lse"][fin]))).all()
    for n, g in zip(("dq", "dk", "dv"), grads):
        within(g, r[n], b[n], n)


@pytest.mark.parametrize("case", AT)
def test_attention(case):
    causal = case[5]
    att, lq, lk, q, k, v, do = attention_data(case)
    cq, ck, mq, mk = offsets(lq), offsets(lk), max(lq), max(lk)
    out, lse = att.forward(q, k, v, cq, mq, ck, mk, causal=causal)
    grads = att.backward(do, q, k, v, out, lse, cq, mq, ck, mk, causal=causal)
    check_all(out, lse, grads, *reference(att, lq, lk, q, k, v, do, causal))
    out2, lse2 = att.forward(q, k, v, cq, mq, ck, mk, causal=causal)
    assert torch.equal(out, out2) and torch.equal(lse, lse2)
    for a, c in zip(grads, att.backward(do, q, k, v, out, lse, cq, mq, ck, mk, causal=causal)):
        assert torch.equal(a, c)


def test_attention_large_scores():
    """Scores of some hundreds: weights of 0 and 1, one row's maximum late in the row."""
    case = ([400], None, 4, 2, 64, True)
    att, lq, lk, q, k, v, do = attention_data(case, 5, std=12.0)
    k[300:] *= 2
    cq = offsets(lq)
    out, lse = att.forward(q, k, v, cq, 400)
    r, b = reference(att, lq, lk, q, k, v, do, True)
    # a score of magnitude s carries an fp32 error of s * 2^-20 into its weight
    s = np.abs(f64(q)).sum(-1).max() * np.abs(f64(k)).max() * att.scale * 2.0 ** -20
    within(out, r["out"], b["out"] + s * np.abs(f64(v)).max(), "out")
    assert np.allclose(f64(lse), r["lse"], rtol=2.0 ** -16, atol=s)


def test_strided_views_and_another_stream():
    """q, k, v as views of one fused array, head-major outputs, gradients into one fused
    array, on a side stream: the bits of the dense call."""
    case = ([150, 77], None, 6, 2, 64, True)
    att, lq, lk, q, k, v, do = attention_data(case, 7)
    T, cq = sum(lq), offsets(lq)
    out, lse = att.forward(q, k, v, cq, 150)
    dense = att.backward(do, q, k, v, out, lse, cq, 150)
    fused = torch.cat([q, k, v], 1).contiguous()
    dfused = torch.zeros_like(fused)
    hm = torch.zeros(6, T, 64, dtype=torch.bfloat16, device="cuda").transpose(0, 1)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        qs, ks, vs = fused[:, :6], fused[:, 6:8], fused[:, 8:]
        out2, lse2 = att.forward(qs, ks, vs, cq, 150, out=hm)
        att.backward(do.transpose(0, 1).contiguous().transpose(0, 1), qs, ks, vs, out2, lse2, cq,
                     150, dq=dfused[:, :6], dk=dfused[:, 6:8], dv=dfused[:, 8:])
    side.synchronize()
    assert torch.equal(out2, out) and torch.equal(lse, lse2)
    for a, c in zip((dfused[:, :6], dfused[:, 6:8], dfused[:, 8:]), dense):
        assert torch.equal(a, c)


def test_non_finite_values_stay_in_their_sequence():
    """NaN and infinities in one sequence and in rows of no sequence leave every bit of
    the other sequences as it was; rows of no sequence are not written."""
    for lens in ([40, 50, 60], [130, 10, 200]):
        T, pad = sum(lens), 37
        att, lq, lk, q, k, v, do = attention_data((lens + [pad], None, 4, 2, 64, True), 9)
        cq = offsets(lens)
        out, lse = att.forward(q, k, v, cq, max(lens), out=torch.zeros_like(q),
                               lse=torch.zeros(T + pad, 4, device="cuda"))
        g = att.backward(do, q, k, v, out, lse, cq, max(lens), dq=torch.zeros_like(q),
                         dk=torch.zeros_like(k), dv=torch.zeros_like(v))
        a, b = lens[0], lens[0] + lens[1]
        clean = [x.clone() for x in (q, k, v, do)]
        for x in (q, k, v, do):
            x[a:b:3] = float("nan")
            x[a + 1:b:3] = float("inf")
            x[T:] = float("nan")
        out2, lse2 = att.forward(q, k, v, cq, max(lens), out=torch.zeros_like(q),
                                 lse=torch.zeros(T + pad, 4, device="cuda"))
        g2 = att.backward(do, q, k, v, out2, lse2, cq, max(lens), dq=torch.zeros_like(q),
                          dk=torch.zeros_like(k), dv=torch.zeros_like(v))
        for x, y in zip((out, lse) + g, (out2, lse2) + g2):
            assert torch.equal(x[:a], y[:a]) and torch.equal(x[b:], y[b:])
            assert (y[T:] == 0).all()
        del clean


def test_calls_back_to_back_give_the_same_bits():
    """Hundreds of forward and backward passes in a row, without a wait between them: no
    bounded wait runs out and the last results are the first ones."""
    case = ([700, 64, 333], None, 12, 4, 128, True)
    att, lq, lk, q, k, v, do = attention_data(case, 17)
    cq = offsets(lq)
    out, lse = att.forward(q, k, v, cq, 700)
    grads = att.backward(do, q, k, v, out, lse, cq, 700)
    first = [x.clone() for x in (out, lse) + grads]
    for _ in range(400):
        att.forward(q, k, v, cq, 700, out=out, lse=lse)
        att.backward(do, q, k, v, out, lse, cq, 700, dq=grads[0], dk=grads[1], dv=grads[2])
    for a, b in zip(first, (out, lse) + grads):
        assert torch.equal(a, b)


def test_gradient_is_the_difference():
    """The gradients along random directions against fp64 central differences."""
    case = ([37, 21], [37, 30], 4, 2, 32, True)
    att, lq, lk, q, k, v, do = attention_data(case, 11)
    cq, ck = offsets(lq), offsets(lk)
    out, lse = att.forward(q, k, v, cq, 37, ck, 37)
    grads = [f64(g) for g in att.backward(do, q, k, v, out, lse, cq, 37, ck, 37)]
    r, b = reference(att, lq, lk, q, k, v, do, True)
    x = [f64(t) for t in (q, k, v)]
    rng = np.random.default_rng(1)

    def loss(q, k, v):
        s, a0, b0 = 0.0, 0, 0
        for n, m in zip(lq, lk):
            for h in range(4):
                o = O.attention(q[a0:a0 + n, h], k[b0:b0 + m, h // 2], v[b0:b0 + m, h // 2],
                                att.scale, True)[0]
                s += float((o * f64(do)[a0:a0 + n, h]).sum())
            a0, b0 = a0 + n, b0 + m
        return s

    for i, n in enumerate(("dq", "dk", "dv")):
        d = rng.standard_normal(x[i].shape)
        hi, lo = list(x), list(x)
        hi[i], lo[i] = x[i] + 1e-5 * d, x[i] - 1e-5 * d
        diff = (loss(*hi) - loss(*lo)) / 2e-5
        assert abs(diff - (grads[i] * d).sum()) <= (b[n] * np.abs(d)).sum() + 1e-5


def test_sequences_refused_on_the_device():
    from token_dispatch_grouped_gb300 import binding as B
    att, lq, lk, q, k, v, do = attention_data(([20, 30], None, 4, 2, 64, True), 13)
    good = offsets(lq)
    for cu, mq in (([0, 20, 51], 31), ([0, 30, 20], 30), ([-4, 20, 50], 30), ([0, 20, 50], 29)):
        c = torch.tensor(cu, dtype=torch.int32, device="cuda")
        out, lse = att.forward(q, k, v, c, mq, good, 30)
        assert B.moe_get_error() == B.MOE_ERR_BAD_INDEX, cu
        out, lse = att.forward(q, k, v, good, 30)
        att.backward(do, q, k, v, out, lse, good, 30, c, mq)
        assert B.moe_get_error() == B.MOE_ERR_BAD_INDEX, cu


# ------------------------------------------------------------------ paged cache
DC = [  # kv_lens, n, Hq, Hkv, D, page
    ([1], 1, 1, 1, 64, 16), ([1, 16, 17, 64, 65], 1, 8, 2, 128, 16),
    ([700, 3, 1500], 1, 32, 8, 128, 64), ([129, 0, 255], 1, 4, 4, 64, 128),
    ([40, 2, 300], 4, 6, 2, 96, 8), ([4000], 1, 5, 1, 80, 256), ([9000, 100], 1, 16, 1, 128, 32),
    ([513, 512, 511], 3, 64, 1, 40, 64), ([2, 1], 4, 3, 3, 8, 16), ([6000], 20, 4, 1, 64, 16)]


def paged(k, v, lens, page, seed=0, fill=float("nan")):
    """Pages in a shuffled order; everything outside the lengths holds `fill`."""
    Hkv, D = k.shape[1:]
    need = [-(-n // page) for n in lens]
    N, wide = sum(need) + 2, max(max(need), 1)
    order = np.random.default_rng(seed).permutation(N)
    kp = torch.full((N, Hkv, page, D), fill, dtype=torch.bfloat16)
    vp = kp.clone()
    table = np.full((len(lens), wide), 2 ** 30, dtype=np.int32)  # past the pages: not read
    slots, at, t = [], 0, 0
    for b, n in enumerate(lens):
        table[b, :need[b]] = order[at:at + need[b]]
        at += need[b]
        s = table[b, np.arange(n) // page].astype(np.int64) * page + np.arange(n) % page
        kp[s // page, :, s % page] = k[t:t + n].cpu()
        vp[s // page, :, s % page] = v[t:t + n].cpu()
        slots.append(s)
        t += n
    return kp.cuda(), vp.cuda(), torch.from_numpy(table).cuda(), np.concatenate(slots)


@pytest.mark.parametrize("case", DC)
def test_decode(case):
    lens, n, Hq, Hkv, D, page = case
    from token_dispatch_grouped_gb300.attention import Attention
    att, G = Attention(Hq, Hkv, D), Hq // Hkv
    k, v = rnd((sum(lens), Hkv, D), 1), rnd((sum(lens), Hkv, D), 2)
    q = rnd((len(lens) * n, Hq, D), 3).cuda()
    kp, vp, table, _ = paged(k, v, lens, page)
    kv = torch.tensor(lens, dtype=torch.int32, device="cuda")
    out = att.decode(q, kp, vp, table, kv, max(lens))
    assert torch.equal(out, att.decode(q, kp, vp, table, kv, max(lens)))
    ref, bound = np.zeros(q.shape), np.zeros(q.shape)
    at = 0
    for b, m in enumerate(lens):
        rows = slice(b * n, b * n + n)
        kb, vb = f64(k)[at:at + m], f64(v)[at:at + m]
        at += m
        for h in range(Hq if m else 0):
            o, _, p = O.attention(f64(q)[rows, h], kb[:, h // G], vb[:, h // G], att.scale, True)
            ref[rows, h], bound[rows, h] = o, O.forward_bound(o, vb[:, h // G], p)
    within(out, ref, bound, "decode")
    # a larger stated bound and a head-major output change nothing but the split
    hm = torch.zeros(Hq, len(lens) * n, D, dtype=torch.bfloat16, device="cuda").transpose(0, 1)
    if max(lens) < table.shape[1] * page:
        att.decode(q, kp, vp, table, kv, table.shape[1] * page, out=hm)
        within(hm, ref, bound, "decode, larger bound")


def test_decode_refused_on_the_device():
    from token_dispatch_grouped_gb300 import binding as B
    from token_dispatch_grouped_gb300.attention import Attention
    att = Attention(4, 2, 64)
    k = rnd((80, 2, 64), 1)
    q = rnd((2, 4, 64), 3).cuda()
    kp, vp, table, _ = paged(k, k, [50, 30], 16)
    good = torch.tensor([50, 30], dtype=torch.int32, device="cuda")
    for lens in ([50, -1], [51, 30]):
        att.decode(q, kp, vp, table, torch.tensor(lens, dtype=torch.int32, device="cuda"), 50)
        assert B.moe_get_error() == B.MOE_ERR_BAD_INDEX
    for page in (-1, kp.shape[0]):
        t = table.clone()
        t[1, 1] = page
        out = att.decode(q, kp, vp, t, good, 50)
        assert B.moe_get_error() == B.MOE_ERR_BAD_INDEX
        assert torch.equal(out[0], att.decode(q, kp, vp, table, good, 50)[0])


@pytest.mark.parametrize("case", [(9, 4, 2, 64, 64, "half", True), (40, 8, 8, 128, 64,
                                  "interleaved", True), (21, 5, 1, 80, 40, "half", False)])
def test_append(case):
    T, Hq, Hkv, D, rot, layout, norm = case
    from token_dispatch_grouped_gb300 import binding as B
    att, qkv, (wq, wk), _, pos, _ = norm_rope_data(case, 21)
    q, k, v = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
    qo, ko = att.norm_rope(q, k, wq, wk, pos)
    kp = torch.full((6, Hkv, 16, D), 5.0, dtype=torch.bfloat16, device="cuda")
    vp = kp.clone()
    slots = torch.randperm(96, generator=torch.Generator().manual_seed(1))[:T]
    slots[3] = -1                                        # not stored
    want_k, want_v = kp.clone(), vp.clone()
    for t, s in enumerate(slots.tolist()):
        if s >= 0:
            want_k[s // 16, :, s % 16], want_v[s // 16, :, s % 16] = ko[t], v[t]
    assert torch.equal(att.append(q, k, v, wq, wk, pos, slots.cuda(), kp, vp), qo)
    assert torch.equal(kp, want_k) and torch.equal(vp, want_v)
    slots[1] = 96                                        # past the cache: left out, reported
    att.append(q, k, v, wq, wk, pos, slots.cuda(), kp, vp)
    assert B.moe_get_error() == B.MOE_ERR_BAD_INDEX
    assert torch.equal(kp, want_k) and torch.equal(vp, want_v)


def test_wrong_tensors_are_refused():
    from token_dispatch_grouped_gb300 import binding as B
    att, lq, lk, q, k, v, do = attention_data(([8], None, 4, 2, 64, True))
    cq = offsets(lq)
    for bad in (q.float(), q[:, :3], q.cpu(), q.transpose(1, 2)):
        with pytest.raises(B.MoeError):
            att.forward(bad, k, v, cq, 8)
    with pytest.raises(B.MoeError):
        att.forward(q, k, v[:4], cq, 8)
    with pytest.raises(B.MoeError):
        att.forward(q, k[:1].expand(8, 2, 64), v, cq, 8)   # a broadcast input
    with pytest.raises(B.MoeError):
        att.forward(q, k, v, cq.long(), 8)
    with pytest.raises(B.MoeError):
        att.decode(q, v[None].contiguous(), v[None].contiguous(), cq[None], cq[:1], 8)


def test_decoder_block_example():
    """The example runs: one training step, then served tokens that agree with it."""
    import importlib.util
    import os
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples",
                        "decoder_block.py")
    spec = importlib.util.spec_from_file_location("decoder_block", path)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    assert m.main() < 1e-2


@pytest.mark.parametrize("case", NR)
def test_norm_rope_backward_in_place(case):
    """dq and dk over the gradients they come from, in one fused array: the same bits,
    and the values between them stay."""
    T, Hq, Hkv, D, rot, layout, norm = case
    att, qkv, (wq, wk), _, pos, _ = norm_rope_data(case, 3)
    q, k = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv]
    g = rnd(tuple(qkv.shape), 52).cuda()
    kept = g.clone()
    want = att.norm_rope_backward(kept[:, :Hq], kept[:, Hq:Hq + Hkv], q, k, wq, wk, pos)
    got = att.norm_rope_backward(g[:, :Hq], g[:, Hq:Hq + Hkv], q, k, wq, wk, pos, dq=g[:, :Hq],
                                 dk=g[:, Hq:Hq + Hkv])
    for x, y in zip(want, got):
        assert x is None or torch.equal(x, y)
    assert torch.equal(g[:, Hq + Hkv:], kept[:, Hq + Hkv:])


def test_served_tokens_from_a_graph():
    """append and decode captured once and replayed with other lengths, pages and tokens:
    the bits of the plain calls."""
    from token_dispatch_grouped_gb300.attention import Attention
    Hq, Hkv, D, page = 8, 2, 64, 16
    att = Attention(Hq, Hkv, D, rope_table=table_of(256, D))
    w = torch.ones(D, device="cuda")
    kp = rnd((24, Hkv, page, D), 5).cuda()
    vp = rnd((24, Hkv, page, D), 6).cuda()
    table = torch.arange(24, dtype=torch.int32, device="cuda").view(3, 8)
    qkv = torch.zeros(3, Hq + 2 * Hkv, D, dtype=torch.bfloat16, device="cuda")
    kv = torch.ones(3, dtype=torch.int32, device="cuda")
    pos = torch.zeros(3, dtype=torch.int32, device="cuda")
    slots = torch.zeros(3, dtype=torch.int64, device="cuda")

    def step(kp, vp):
        q, k, v = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
        return att.decode(att.append(q, k, v, w, w, pos, slots, kp, vp), kp, vp, table, kv, 128)

    def fill(i):
        lens = torch.tensor([1 + 40 * i, 17 + i, 128 - i], dtype=torch.int32)
        qkv.copy_(rnd(tuple(qkv.shape), 70 + i))
        kv.copy_(lens)
        pos.copy_(lens - 1)
        at = (lens - 1).long()
        slots.copy_(table.cpu().long()[torch.arange(3), at // page] * page + at % page)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    fill(0)
    with torch.cuda.stream(side):
        step(kp.clone(), vp.clone())
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step(kp, vp)
    for i in (1, 2, 0):
        fill(i)
        ck, cv = kp.clone(), vp.clone()
        graph.replay()
        want = step(ck, cv)
        assert torch.equal(out, want) and torch.equal(kp, ck) and torch.equal(vp, cv)
