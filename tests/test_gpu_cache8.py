"""The 8-bit cache on the GPU against the fp64 oracle: append8 (scales and values to the bit,
keys within half a step), decode8, and the sums of softmax weights over both caches."""
import numpy as np
import pytest
import torch

from oracle import attention as O
from oracle import cache as C
from test_gpu_attention import (clean_status, f64, norm_rope_data, offsets, paged, rnd,  # noqa: F401
                                within)

pytestmark = pytest.mark.gpu

E4M3 = torch.float8_e4m3fn


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def table_for(need, extra=2, seed=0):
    """(pages in a shuffled order [B, most], how many there are)."""
    N = sum(need) + extra
    order = np.random.default_rng(seed).permutation(N)
    t, at = np.full((len(need), max(max(need), 1)), 2 ** 30, dtype=np.int32), 0
    for b, n in enumerate(need):
        t[b, :n] = order[at:at + n]
        at += n
    return torch.from_numpy(t).cuda(), N


def raw(t):
    return t.view(torch.uint8)


# ------------------------------------------------------------------------ append8
AP = [  # new tokens of each call's sequences, Hq, Hkv, D, rot, layout, norm, page
    ([[1]], 1, 1, 16, 16, "half", True, 8),
    ([[5, 0, 40], [1, 1, 1], [30, 3, 0]], 4, 2, 64, 64, "half", True, 16),
    ([[64, 65, 63, 1], [1, 2, 64, 130]], 8, 8, 128, 64, "interleaved", True, 64),
    ([[300], [1], [1], [257]], 6, 2, 96, 96, "half", True, 256),
    ([[7] * 40, [1] * 40, [9] * 40], 3, 1, 48, 40, "half", True, 8),
    ([[100, 20], [3, 0]], 5, 1, 80, 0, "half", False, 32),
    ([[33, 90], [40, 1]], 4, 4, 112, 12, "interleaved", True, 128)]


@pytest.mark.parametrize("case", AP)
@pytest.mark.parametrize("loud", [1.0, 40.0, 0.01])
def test_append8(case, loud):
    """Calls one after the other, each `loud` times the last one: pages go on, begin and grow."""
    calls, Hq, Hkv, D, rot, layout, norm, P = case
    nb = len(calls[0])
    total = [sum(c[b] for c in calls) for b in range(nb)]
    table, N = table_for([-(-n // P) for n in total])
    g = torch.Generator().manual_seed(5)
    kp, vp = ((torch.randn(N, Hkv, P, D, generator=g) * 50).to(E4M3).cuda() for _ in range(2))
    ks, vs = (torch.full((N, Hkv), 3.0, device="cuda") for _ in range(2))  # of what was there before
    had = [0] * nb
    for i, new in enumerate(calls):
        T = sum(new)
        shape = (T, Hq, Hkv, D, rot, layout, norm)
        att, qkv, (wq, wk), (nq, nk), pos, cs = norm_rope_data(shape, 7 + i)
        if norm:      # the norm takes the keys' size away: it is in the weights then
            wk, nk = wk * loud ** i, nk * loud ** i
            wk, nk = wk.float(), f64(wk.float())
            qkv[:, Hq + Hkv:] *= loud ** i
        else:
            qkv *= loud ** i
        q, k, v = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
        before = [f64(x.float()) for x in (kp, vp, ks, vs)]
        lens = [a + b for a, b in zip(had, new)]
        out = att.append8(q, k, v, wq, wk, pos, offsets(new), table, ints(lens), kp, vp, ks, vs)
        want, _ = att.norm_rope(q, k, wq, wk, pos)
        assert torch.equal(out, want)
        y = O.norm_rope(f64(k), nk if norm else None, 1e-5, cs[..., 0], cs[..., 1],
                        layout == "interleaved")
        off = 2.0 ** -16 * np.abs(y).max(-1, keepdims=True)  # of the keys before they are rounded
        got = [f64(x.float()) for x in (kp, vp, ks, vs)]
        touched, row = np.zeros((N, P), bool), 0
        for b in range(nb):
            t = had[b]
            while t < lens[b]:
                p, o = int(table[b, t // P]), t % P
                n = min(P - o, lens[b] - t)
                touched[p, :o + n] = True
                for h in range(Hkv):
                    page, s = C.append8(before[1][p, h], before[3][p, h], o, f64(v)[row:row + n, h])
                    assert got[3][p, h] == s
                    assert np.array_equal(got[1][p, h, :o + n], page[:o + n])
                    x = y[row:row + n, h]
                    page, s = C.append8(before[0][p, h], before[2][p, h], o, x)
                    top = C.finite_top(x)
                    if o == 0 or s > before[2][p, h]:   # no other scale within the rows' error
                        assert C.power(top * (1 + 2.0 ** -15)) == C.power(top * (1 - 2.0 ** -15))
                    assert got[2][p, h] == s
                    assert np.array_equal(got[0][p, h, :o], page[:o])
                    new_rows = got[0][p, h, o:o + n] * s
                    bound = C.half_step(np.abs(x) + off[row:row + n, h], s) + off[row:row + n, h]
                    assert (np.abs(new_rows - x) <= bound).all()
                t, row = t + n, row + n
        for a, b in zip(got[:2], before[:2]):            # nothing else moves
            assert np.array_equal(a.transpose(0, 2, 1, 3)[~touched], b.transpose(0, 2, 1, 3)[~touched])
        for a, b in zip(got[2:], before[2:]):
            assert np.array_equal(a[~touched.any(1)], b[~touched.any(1)])
        had = lens


def cache8(N, Hkv, P, D, scale=1.0):
    k = torch.zeros(N, Hkv, P, D, device="cuda").to(E4M3)
    s = torch.full((N, Hkv), scale, device="cuda")
    return k, k.clone(), s, s.clone()


def test_append8_rows_that_are_not_finite():
    """They become NaN; the page's scale and its other values are what they are without them."""
    from token_dispatch_grouped_gb300.attention import Attention
    att = Attention(2, 2, 32)
    x = rnd((20, 2, 32), 1).cuda()
    clean, bad = x.clone(), x.clone()
    for t, h, d, v in ((3, 0, 5, float("inf")), (4, 1, 0, float("-inf")), (17, 1, 31, float("nan"))):
        bad[t, h, d], clean[t, h, d] = v, 0
    out = []
    for y in (clean, bad):
        c = cache8(3, 2, 16, 32)
        att.append8(x, y, y, None, None, None, offsets([20]), ints([[2, 0]]), ints([20]), *c)
        out.append(c)
    for a, b in zip(out[0], out[1]):
        a, b = a.float(), b.float()
        assert torch.equal(a, torch.where(b.isnan(), 0.0, b))
    assert [int(c.float().isnan().sum()) for c in out[1][:2]] == [3, 3]
    assert out[1][0].float()[2, 0, 3, 5].isnan() and out[1][0].float()[0, 1, 1, 31].isnan()


def test_append8_rows_of_no_sequence_and_strides():
    """Rows outside cu_new are not stored; head-major inputs give the same bits; no sequence at
    all leaves the cache alone, and the queries are formed all the same."""
    shape = (50, 4, 2, 64, 64, "half", True)
    att, qkv, (wq, wk), _, pos, _ = norm_rope_data(shape, 3)
    q, k, v = qkv[:, :4], qkv[:, 4:6], qkv[:, 6:]
    table = ints([[1, 2], [3, 4]])
    a, b = cache8(6, 2, 16, 64), cache8(6, 2, 16, 64)
    cu = ints([3, 10, 40])
    out = att.append8(q, k, v, wq, wk, pos, cu, table, ints([9, 32]), *a)
    r = slice(3, 40)
    want = att.append8(q[r], k[r], v[r], wq, wk, pos[r], offsets([7, 30]), table, ints([9, 32]), *b)
    assert torch.equal(out[r], want)
    for x, y in zip(a, b):
        assert torch.equal(x.float(), y.float())
    hm = [x.transpose(0, 1).contiguous().transpose(0, 1) for x in (q, k, v)]
    c = cache8(6, 2, 16, 64)
    assert torch.equal(out, att.append8(*hm, wq, wk, pos, cu, table, ints([9, 32]), *c))
    for x, y in zip(a, c):
        assert torch.equal(x.float(), y.float())
    none = table[:0]
    assert torch.equal(out, att.append8(q, k, v, wq, wk, pos, ints([0]), none, ints([]), *c, max_kv=0))
    for x, y in zip(a, c):
        assert torch.equal(x.float(), y.float())


@pytest.mark.parametrize("wrong", ["page", "long", "short", "position"])
def test_append8_one_bad_sequence_leaves_the_others(wrong):
    from token_dispatch_grouped_gb300 import binding as B
    shape = (60, 4, 2, 64, 64, "half", True)
    att, qkv, (wq, wk), _, pos, _ = norm_rope_data(shape, 4)
    q, k, v = qkv[:, :4], qkv[:, 4:6], qkv[:, 6:]
    new, lens, table = [20, 15, 25], [30, 15, 25], ints([[0, 1, 2], [3, 4, 5], [6, 7, 8]])
    good, bad = cache8(9, 2, 16, 64, 0.01), cache8(9, 2, 16, 64, 0.01)
    out = att.append8(q, k, v, wq, wk, pos, offsets(new), table, ints(lens), *good, max_kv=40)
    t, n, p = table.clone(), list(lens), pos.clone()
    if wrong == "page":
        t[0, 1] = 9
    elif wrong == "long":
        n[0] = 41
    elif wrong == "short":
        n[0] = 19
    else:
        p[2] = 500
    for _ in range(2):                       # the second call finds the status already set
        got = att.append8(q, k, v, wq, wk, p, offsets(new), t, ints(n), *bad, max_kv=40)
        keep = torch.arange(60, device="cuda") != (2 if wrong == "position" else -1)
        assert torch.equal(got[keep], out[keep])
        for a, b in zip(good, bad):
            assert torch.equal(a[3:].float(), b[3:].float())
    assert B.moe_get_error() == B.MOE_ERR_BAD_INDEX


def test_append8_bad_offsets_are_reported():
    from token_dispatch_grouped_gb300 import binding as B
    shape = (60, 4, 2, 64, 64, "half", True)
    att, qkv, (wq, wk), _, pos, _ = norm_rope_data(shape, 4)
    q, k, v = qkv[:, :4], qkv[:, 4:6], qkv[:, 6:]
    table = ints([[0, 1, 2, 3], [4, 5, 6, 7]])
    want = att.norm_rope(q, k, wq, wk, pos)[0]
    for cu in ([0, 20, 61], [0, 30, 20], [-4, 20, 50]):
        out = att.append8(q, k, v, wq, wk, pos, ints(cu), table, ints([40, 40]),
                          *cache8(8, 2, 16, 64))
        assert B.moe_get_error() == B.MOE_ERR_BAD_INDEX and torch.equal(out, want)


# ------------------------------------------------------------------------ decode
DC = [  # kv_lens, n, Hq, Hkv, D, page
    ([1], 1, 1, 1, 64, 16), ([1, 16, 17, 64, 65], 1, 8, 2, 128, 16),
    ([700, 3, 1500], 1, 32, 8, 128, 64), ([129, 0, 255], 1, 4, 4, 64, 128),
    ([40, 2, 300], 4, 6, 2, 96, 8), ([4000], 1, 5, 1, 80, 256), ([9000, 100], 1, 16, 1, 128, 32),
    ([513, 512, 511], 3, 64, 1, 48, 64), ([2, 1], 4, 3, 3, 16, 16), ([6000], 20, 4, 1, 64, 16)]


def decode_data(case, bits, seed=0, scale=lambda g, s: torch.exp2(torch.randint(
        -9, -5, s, generator=g).float())):
    """Pages of random values (NaN outside the lengths), what they stand for, and weights."""
    lens, n, Hq, Hkv, D, P = case
    k, v = rnd((sum(lens), Hkv, D), seed + 1), rnd((sum(lens), Hkv, D), seed + 2)
    q = rnd((len(lens) * n, Hq, D), seed + 3).cuda()
    g = torch.Generator().manual_seed(seed + 4)
    if bits == 16:
        kp, vp, table, _ = paged(k, v, lens, P)
        pages, kv = (kp, vp), [f64(k), f64(v)]
    else:
        k8, v8 = ((x.float() * 64).clamp(-448, 448).to(E4M3) for x in (k, v))
        kp, vp, table, _ = paged(k8.bfloat16(), v8.bfloat16(), lens, P)
        kp, vp = kp.to(E4M3), vp.to(E4M3)
        ks, vs = (scale(g, (kp.shape[0], Hkv)) for _ in range(2))
        kv = []
        for x, s in ((k8, ks), (v8, vs)):
            page = torch.cat([table[b, torch.arange(m) // P].cpu().long()
                              for b, m in enumerate(lens)]) if sum(lens) else torch.zeros(0).long()
            kv.append(x.double().numpy() * s.double().numpy()[page][..., None])
        pages = (kp, vp, ks.cuda(), vs.cuda())
    w = torch.rand(kp.shape[0], Hkv, P, generator=g).cuda()
    return q, pages, kv, table, ints(lens), w


def decode_of(att, pages, q, table, kv_lens, most, **kw):
    f = att.decode if len(pages) == 2 else att.decode8
    return f(q, *pages, table, kv_lens, most, **kw)


def reference(case, q, kv, scale):
    """out, its bound, and per sequence the weights [Hkv, tokens] that the call adds."""
    lens, n, Hq, Hkv, D, P = case
    G = Hq // Hkv
    ref, bound, add, at = np.zeros(q.shape), np.zeros(q.shape), [], 0
    for b, m in enumerate(lens):
        rows = slice(b * n, b * n + n)
        kb, vb = (x[at:at + m] for x in kv)
        at += m
        add.append(np.zeros((Hkv, m)))
        for h in range(Hq if m else 0):
            o, _, p = O.attention(f64(q)[rows, h], kb[:, h // G], vb[:, h // G], scale, True)
            ref[rows, h], bound[rows, h] = o, O.forward_bound(o, vb[:, h // G], p)
            add[b][h // G] += p.sum(0)
    return ref, bound, add


@pytest.mark.parametrize("bits", [8, 16])
@pytest.mark.parametrize("case", DC)
def test_decode_with_weights(case, bits):
    lens, n, Hq, Hkv, D, P = case
    from token_dispatch_grouped_gb300.attention import Attention
    att = Attention(Hq, Hkv, D)
    q, pages, kv, table, kv_lens, w = decode_data(case, bits)
    out = decode_of(att, pages, q, table, kv_lens, max(lens))
    assert torch.equal(out, decode_of(att, pages, q, table, kv_lens, max(lens)))
    ref, bound, add = reference(case, q, kv, att.scale)
    within(out, ref, bound, "decode")
    if max(lens) < table.shape[1] * P:   # a larger stated bound, a head-major output
        hm = torch.zeros(Hq, len(lens) * n, D, dtype=torch.bfloat16, device="cuda").transpose(0, 1)
        decode_of(att, pages, q, table, kv_lens, table.shape[1] * P, out=hm)
        within(hm, ref, bound, "decode, larger bound")
    for fresh in (False, True):
        got = w.clone()
        assert torch.equal(out, decode_of(att, pages, q, table, kv_lens, max(lens), weights=got,
                                          fresh=fresh))
        want = f64(w).copy()
        slack = np.zeros_like(want)
        for b, m in enumerate(lens):
            t = np.arange(m)
            page, off = table.cpu().numpy()[b, t // P], t % P
            had = want[page, :, off].T
            had = np.where((t >= m - n) | fresh, 0.0, had)
            want[page, :, off] = (had + add[b]).T
            # F: scores and exponentials in fp32; one rounding of the sum, and of its terms
            slack[page, :, off] = (O.F * add[b] + 2.0 ** -22 * (had + add[b])).T
        assert (np.abs(f64(got) - want) <= slack).all()


@pytest.mark.parametrize("scales", ["odd", "zero", "wide"])
def test_decode8_scales(scales):
    """Scales that are no powers of two, of empty pages (zero), and far apart."""
    from token_dispatch_grouped_gb300.attention import Attention
    case = ([700, 90], 2, 8, 2, 64, 16)

    def scale(g, s):
        if scales == "odd":
            return 0.001 + 0.01 * torch.rand(s, generator=g)
        e = torch.exp2(torch.randint(-9, -5, s, generator=g).float())
        if scales == "zero":
            return e * (torch.rand(s, generator=g) < 0.5)
        return torch.exp2(torch.randint(-40, -6, s, generator=g).float())

    att = Attention(8, 2, 64)
    q, pages, kv, table, kv_lens, _ = decode_data(case, 8, 3, scale)
    out = decode_of(att, pages, q, table, kv_lens, 700)
    ref, bound, _ = reference(case, q, kv, att.scale)
    within(out, ref, bound, scales)


def test_decode8_many_small_weights_beside_a_large_one():
    """40,000 tokens of a weight of about 2^-30 beside one of 1: their share, which fp16 alone
    would lose, stays (it is 4e-5 of the sum; V is 448 where they are and 2^-9 at the one)."""
    from token_dispatch_grouped_gb300.attention import Attention
    L, D, P = 40000, 64, 64
    att = Attention(1, 1, D, scale=1.0)
    k = torch.zeros(L, 1, D)
    k[0] = 1.0
    v = torch.full((L, 1, D), 448.0)
    v[0] = 2.0 ** -9
    q = torch.full((1, 1, D), 30 * np.log(2) / D).bfloat16()
    kp, vp, table, _ = paged(k.bfloat16(), v.bfloat16(), [L], P)
    one = torch.ones(kp.shape[0], 1, device="cuda")
    out = att.decode8(q.cuda(), kp.to(E4M3), vp.to(E4M3), one, one, table, ints([L]), L)
    o, _, p = O.attention(f64(q)[:, 0], f64(k)[:, 0], f64(v)[:, 0], 1.0, False)
    assert p[0, 1] < 2.0 ** -28 and o[0, 0] > 4 * 2.0 ** -9
    within(out[:, 0], o, O.forward_bound(o, f64(v)[:, 0], p), "small weights")


@pytest.mark.parametrize("size", [1e-30, 1e30])
def test_decode8_queries_of_any_size(size):
    from token_dispatch_grouped_gb300.attention import Attention
    case = ([300], 1, 4, 2, 128, 64)
    q, pages, kv, table, kv_lens, _ = decode_data(case, 8, 5)
    q = (q.float() * size).bfloat16()
    att = Attention(4, 2, 128, scale=128 ** -0.5 / size)
    out = decode_of(att, pages, q, table, kv_lens, 300)
    ref, bound, _ = reference(case, q, kv, att.scale)
    within(out, ref, bound, "size")


@pytest.mark.parametrize("bits", [8, 16])
@pytest.mark.parametrize("wrong", ["page", "length"])
def test_one_bad_sequence_leaves_the_others(wrong, bits):
    from token_dispatch_grouped_gb300 import binding as B
    from token_dispatch_grouped_gb300.attention import Attention
    case = ([1500, 900, 3, 0, 1200], 1, 8, 2, 64, 16)
    att = Attention(8, 2, 64)
    q, pages, _, table, kv, w = decode_data(case, bits)
    good, bad = w.clone(), w.clone()
    want = decode_of(att, pages, q, table, kv, 1500, weights=good)
    mine = table.cpu().numpy()[1, :-(-900 // 16)]
    table, kv = table.clone(), kv.clone()
    if wrong == "page":
        table[1, 50] = pages[0].shape[0]
    else:
        kv[1] = 1501
    keep = [0, 2, 3, 4]
    others = np.setdiff1d(np.arange(w.shape[0]), mine)
    got = decode_of(att, pages, q, table, kv, 1500, out=torch.full_like(want, 7), weights=bad)
    assert torch.equal(got[keep], want[keep])
    assert torch.equal(bad[others], good[others])
    assert B.moe_get_error() == B.MOE_ERR_BAD_INDEX


def test_a_value_that_is_not_finite_stays_in_its_sequence():
    from token_dispatch_grouped_gb300.attention import Attention
    case = ([200, 150, 70], 1, 4, 2, 64, 16)
    att = Attention(4, 2, 64)
    q, pages, _, table, kv, w = decode_data(case, 8)
    a, b = w.clone(), w.clone()
    want = decode_of(att, pages, q, table, kv, 200, weights=a)
    page = int(table[1, 3])
    raw(pages[0])[page, :, 2, 5] = 0x7f      # NaN
    got = decode_of(att, pages, q, table, kv, 200, weights=b)
    assert torch.equal(got[[0, 2]], want[[0, 2]]) and got[1].isnan().all()
    others = [p for p in range(w.shape[0]) if p not in table.cpu().numpy()[1, :-(-150 // 16)]]
    assert torch.equal(a[others], b[others])


@pytest.mark.parametrize("bits", [8, 16])
@pytest.mark.parametrize("seqs", [3, 400])
def test_no_cached_token_at_all(seqs, bits):
    """A stated bound of 0: zeros, weights untouched, and no workspace to write to."""
    from token_dispatch_grouped_gb300.attention import Attention
    att, table = Attention(4, 2, 64), torch.zeros(seqs, 1, dtype=torch.int32, device="cuda")
    k, _, s, _ = cache8(2, 2, 16, 64)
    pages = (k, k, s, s) if bits == 8 else (k.bfloat16(), k.bfloat16())
    w = torch.rand(2, 2, 16, device="cuda")
    before, q = w.clone(), rnd((seqs, 4, 64), 1).cuda()
    out = decode_of(att, pages, q, table, ints([0] * seqs), 0, weights=w,
                    out=torch.full_like(q, 3))
    assert bool((out == 0).all()) and torch.equal(w, before)


MANY = [  # sequences, longest, n, Hq, Hkv, D, page: parts for more CTAs than the GPU holds
    (64, 900, 1, 8, 8, 64, 64), (40, 1500, 3, 8, 2, 128, 16), (300, 300, 1, 16, 2, 96, 8),
    (1100, 200, 1, 2, 1, 64, 64)]


@pytest.mark.parametrize("case", MANY)
def test_decode8_many_parts(case):
    """Uneven sequences, empty ones among them, whose parts the CTAs take in turn; then one of
    them with a length out of range: the others keep every bit, in a replayed graph too."""
    seqs, longest, n, Hq, Hkv, D, P = case
    from token_dispatch_grouped_gb300 import binding as B
    from token_dispatch_grouped_gb300.attention import Attention
    r = np.random.default_rng(seqs)
    lens = [int(x) for x in r.integers(0, longest, seqs)]
    lens[3], lens[5], lens[-1] = 0, longest, 1
    att, full = Attention(Hq, Hkv, D), (lens, n, Hq, Hkv, D, P)
    q, pages, kv, table, kv_lens, w = decode_data(full, 8)
    got = w.clone()
    out = decode_of(att, pages, q, table, kv_lens, longest, weights=got)
    assert torch.equal(out, decode_of(att, pages, q, table, kv_lens, longest))
    ref, bound, add = reference(full, q, kv, att.scale)
    within(out, ref, bound, "many parts")
    for b in (0, 5, seqs // 2, seqs - 1):
        t = np.arange(lens[b])
        page, off = table.cpu().numpy()[b, t // P], t % P
        had = np.where(t >= lens[b] - n, 0.0, f64(w)[page, :, off].T)
        want = (had + add[b]).T
        assert (np.abs(f64(got)[page, :, off] - want) <= (O.F * add[b] + 2.0 ** -22 * want.T).T).all()
    args = (q, table, kv_lens, longest)
    decode_of(att, pages, *args)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        again = decode_of(att, pages, *args)
    for _ in range(3):
        again.zero_()
        graph.replay()
        assert torch.equal(again, out)
    kv_lens[5] = longest + 1
    graph.replay()
    assert B.moe_get_error() == B.MOE_ERR_BAD_INDEX
    rows = torch.arange(seqs * n, device="cuda") // n != 5
    assert torch.equal(again[rows], out[rows])
