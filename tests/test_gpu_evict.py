"""Eviction on the GPU, whole numbers and moved rows to the bit, and the small cache as a server
uses it: a prompt, votes on its tokens, eviction, more tokens."""
import numpy as np
import pytest
import torch

from oracle import attention as O
from oracle import cache as C
from test_gpu_attention import clean_status, f64, norm_rope_data, offsets, within  # noqa: F401
from test_gpu_cache8 import E4M3, cache8, ints, raw, table_for

pytestmark = pytest.mark.gpu

EV = [  # lens, keep, recent, Hkv, D, page, bits
    ([1], 1, 0, 1, 8, 8, 16), ([5, 0, 9, 8], 8, 3, 2, 64, 8, 16), ([5, 0, 9, 8], 8, 3, 2, 64, 8, 8),
    ([300, 77, 1000], 128, 20, 2, 96, 16, 8), ([300, 77, 1000], 128, 128, 2, 96, 64, 16),
    ([700], 333, 0, 3, 128, 256, 8), ([40] * 30, 13, 1, 1, 16, 32, 8),
    ([2500, 1024, 1025], 1024, 100, 1, 40, 16, 16), ([60000, 20], 20001, 2000, 2, 32, 64, 8),
    ([100, 50], 200, 10, 2, 64, 16, 8), ([70, 64], 1, 1, 2, 64, 64, 16)]
KINDS = ["spread", "ties", "odd"]


def evict_data(case, kind):
    lens, keep, recent, Hkv, D, P, bits = case
    g = torch.Generator().manual_seed(9)
    need = [-(-n // P) for n in lens]
    goal = [-(-min(n, keep) // P) for n in lens]
    both, N = table_for(need + goal)
    table, new = both[:len(lens), :max(max(need), 1)], both[len(lens):, :max(max(goal), 1)]
    x = torch.randn(2, N, Hkv, P, D, generator=g)
    if bits == 8:
        kp, vp = ((y * 60).to(E4M3).cuda() for y in x)
        e = torch.randint(-9, -5, (2, N, Hkv), generator=g)
        scales = tuple(torch.exp2(y.float()).cuda() for y in e)
    else:
        kp, vp = (y.bfloat16().cuda() for y in x)
        scales = ()
    w = torch.exp(2 * torch.randn(N, Hkv, P, generator=g))
    if kind == "ties":
        w = (w * 2).round() / 2
    if kind == "odd":
        pick = torch.randint(0, 12, w.shape, generator=g)
        for i, v in enumerate((float("nan"), float("inf"), -0.0, 0.0, -1.0, float("-inf"))):
            w[pick == i] = v
    return kp, vp, scales, w.cuda(), table, new


def evict_of(att, d, lens, most, keep, recent, **kw):
    kp, vp, scales, w, table, new = d
    if scales:
        kw.update(k_scales=scales[0], v_scales=scales[1])
    return att.evict(kp, vp, w, table, lens, most, keep, recent, new, **kw)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("case", EV)
def test_evict(case, kind):
    from token_dispatch_grouped_gb300.attention import Attention
    lens, keep, recent, Hkv, D, P, bits = case
    att = Attention(Hkv, Hkv, D)
    d = evict_data(case, kind)
    kp, vp, scales, w, table, new = d
    before = [x.float().cpu().numpy() for x in (kp, vp, w) + scales]
    new_lens, kept = evict_of(att, d, ints(lens), max(lens), keep, recent)
    assert new_lens.tolist() == [min(n, keep) for n in lens]
    want = [x.copy() for x in before]
    tab, goal = table.cpu().numpy(), new.cpu().numpy()
    kept = kept.cpu().numpy()
    for b, n in enumerate(lens):
        t = np.arange(n)
        for h in range(Hkv):
            ws = before[2][tab[b, t // P], h, t % P]
            pick = C.kept(ws, keep, recent)
            m = len(pick)
            assert np.array_equal(kept[b, h, :m], pick) and (kept[b, h, m:] == -1).all()
            src, so, i = tab[b, pick // P], pick % P, np.arange(m)
            dst, do = goal[b, i // P], i % P
            want[2][dst, h, do] = before[2][src, h, so]
            for x in range(2):
                rows = before[x][src, h, so].astype(np.float64)
                if bits == 8:
                    old = before[3 + x][src, h].astype(np.float64)
                    top = np.array([old[j:j + P].max() for j in range(0, m, P)])
                    want[3 + x][goal[b, :len(top)], h] = top
                    rows = C.e4m3(rows * (old / top[i // P])[:, None])
                want[x][dst, h, do] = rows
    for x, y in zip((kp, vp, w) + scales, want):
        assert np.array_equal(x.float().cpu().numpy(), y, equal_nan=True)


def test_lengths_in_place_and_a_larger_bound():
    from token_dispatch_grouped_gb300.attention import Attention
    case = ([300, 77, 1000], 128, 20, 2, 96, 16, 8)
    lens, keep, recent, Hkv, D, P, bits = case
    att = Attention(Hkv, Hkv, D)
    a, b = evict_data(case, "spread"), evict_data(case, "spread")
    new, kept = evict_of(att, a, ints(lens), 1000, keep, recent)
    n = ints(lens)
    got, again = evict_of(att, b, n, b[4].shape[1] * P, keep, recent, new_lens=n)
    assert got is n and torch.equal(n, new) and torch.equal(kept, again)
    for x, y in zip(a[:2] + a[2], b[:2] + b[2]):
        assert torch.equal(x.float(), y.float())


@pytest.mark.parametrize("wrong", ["page", "goal", "length"])
def test_one_bad_sequence_leaves_the_others(wrong):
    from token_dispatch_grouped_gb300 import binding as B
    from token_dispatch_grouped_gb300.attention import Attention
    case = ([300, 500, 400], 128, 20, 2, 64, 16, 8)
    lens, keep, recent, Hkv, D, P, bits = case
    att = Attention(Hkv, Hkv, D)
    a, b = evict_data(case, "spread"), evict_data(case, "spread")
    new, kept = evict_of(att, a, ints(lens), 500, keep, recent)
    n, d = list(lens), list(b)
    d[4], d[5] = d[4].clone(), d[5].clone()
    if wrong == "page":
        d[4][1, 31] = -1                    # of the newest tokens
    elif wrong == "goal":
        d[5][1, 3] = d[0].shape[0]
    else:
        n[1] = 501
    got, places = evict_of(att, d, ints(n), 500, keep, recent)
    keepers = [0, 2]
    assert torch.equal(got[keepers], new[keepers]) and torch.equal(places[keepers], kept[keepers])
    pages = a[5][keepers].flatten().long()
    for x, y in zip(a[:2] + a[2] + a[3:4], d[:2] + list(d[2]) + d[3:4]):
        assert torch.equal(x[pages].float(), y[pages].float())
    assert B.moe_get_error() == B.MOE_ERR_BAD_INDEX


def test_shared_pages_are_only_read():
    """Two sequences on the same pages (a shared prompt), cut into pages of their own."""
    from token_dispatch_grouped_gb300.attention import Attention
    att = Attention(2, 2, 64)
    d = list(evict_data(([300, 300], 100, 10, 2, 64, 16, 8), "spread"))
    d[4][1] = d[4][0]
    old = [x[d[4][0].long()].float() for x in (d[0], d[1], d[3])]
    _, kept = evict_of(att, d, ints([300, 300]), 300, 100, 10)
    assert torch.equal(kept[0], kept[1])
    for x in (d[0], d[1], d[3]):
        a, b = (x[p.long()].float() for p in d[5])
        valid = torch.arange(7 * 16, device="cuda").view(7, 1, 16) < 100
        valid = valid if x.dim() == 3 else valid[..., None]
        assert torch.equal(a * valid, b * valid)
    for x, y in zip((d[0], d[1], d[3]), old):
        assert torch.equal(x[d[4][0].long()].float(), y)


# ------------------------------------------------------------------- as a server runs it
class Small:
    """Three sequences on a small cache; `step` appends and decodes, `cut` evicts."""

    def __init__(self, Hq=8, Hkv=2, D=64, P=16, most=256, seed=1):
        from token_dispatch_grouped_gb300.attention import Attention, rope_inv_freq, rope_table
        self.att = Attention(Hq, Hkv, D, rope_table=rope_table(1000, rope_inv_freq(D)[0]))
        self.Hq, self.Hkv, self.D, self.P = Hq, Hkv, D, P
        g = torch.Generator().manual_seed(seed)
        self.w = [(1 + 0.1 * torch.randn(D, generator=g)).cuda() for _ in range(2)]
        wide = most // P
        order = torch.randperm(6 * wide, generator=g).to(torch.int32).cuda()
        self.tables = order.view(2, 3, wide)
        self.cache = cache8(6 * wide, Hkv, P, D)
        self.weights = torch.zeros(6 * wide, Hkv, P, device="cuda")
        self.most, self.now = most, 0

    def step(self, qkv, new, lens, pos, window, fresh):
        """Appends new[b] tokens of each sequence; the last `window` attend."""
        Hq, Hkv = self.Hq, self.Hkv
        q = self.att.append8(qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:], *self.w, pos,
                             offsets(new), self.tables[self.now], lens, *self.cache)
        last = torch.cat([torch.arange(sum(new[:b + 1]) - window, sum(new[:b + 1]))
                          for b in range(3)]).cuda()
        return q[last], self.att.decode8(q[last], *self.cache, self.tables[self.now], lens,
                                         self.most, weights=self.weights, fresh=fresh)

    def cut(self, lens, keep, recent):
        k, v, ks, vs = self.cache
        _, kept = self.att.evict(k, v, self.weights, self.tables[self.now], lens, self.most, keep,
                                 recent, self.tables[1 - self.now], k_scales=ks, v_scales=vs,
                                 new_lens=lens)
        self.now = 1 - self.now
        return kept

    def tokens(self, b, n):
        """Keys, values and weights of sequence b as the cache stands for them."""
        t = np.arange(n)
        page, off = self.tables[self.now][b].cpu().numpy()[t // self.P], t % self.P
        k, v, ks, vs = (f64(x.float()) for x in self.cache)
        return (k[page, :, off] * ks[page][..., None], v[page, :, off] * vs[page][..., None],
                f64(self.weights)[page, :, off])


def test_prompt_votes_eviction_and_more_tokens():
    s = Small()
    prompt, keep, recent, lens = [200, 90, 31], 64, 16, None
    total = [p + 12 for p in prompt]
    g = torch.Generator().manual_seed(3)
    lens = ints(prompt)
    n = list(prompt)
    pos = torch.cat([torch.arange(p) for p in prompt]).to(torch.int32).cuda()
    data = torch.randn(sum(prompt), 12, 64, generator=g).bfloat16().cuda()
    G = 4

    def check(q, out, window, before, fresh):
        ref, bound = np.zeros(q.shape), np.zeros(q.shape)
        for b in range(3):
            k, v, w = s.tokens(b, n[b])
            add = np.zeros((n[b], 2))
            for h in range(8):
                rows = slice(b * window, (b + 1) * window)
                o, _, p = O.attention(f64(q)[rows, h], k[:, h // G], v[:, h // G], s.att.scale, True)
                ref[rows, h], bound[rows, h] = o, O.forward_bound(o, v[:, h // G], p)
                add[:, h // G] += p.sum(0)
            had = np.zeros_like(add)
            if not fresh:
                m = min(len(before[b]), n[b] - window)
                had[:m] = before[b][:m]
            assert (np.abs(w - had - add) <= O.F * add + 2.0 ** -22 * (had + add)).all()
        within(out, ref, bound, "served")

    q, out = s.step(data, prompt, lens, pos, 8, True)
    check(q, out, 8, None, True)
    for turn in range(2):
        old = [s.tokens(b, n[b]) for b in range(3)]
        kept = s.cut(lens, keep, recent).cpu().numpy()
        for b in range(3):
            m = min(n[b], keep)
            k, v, w = s.tokens(b, m)
            for h in range(2):
                pick = C.kept(old[b][2][:, h].astype(np.float32), keep, recent)
                assert np.array_equal(kept[b, h, :m], pick)
                assert np.array_equal(w[:, h], old[b][2][pick, h])
                for x, y in ((k, old[b][0]), (v, old[b][1])):
                    top = np.abs(y[pick, h]).max()   # moved values: below the normal range only
                    assert np.abs(x[:, h] - y[pick, h]).max() <= top * 2.0 ** -8 * 2.0 ** -9
            n[b] = m
        assert lens.tolist() == n
        for i in range(6):
            data = torch.randn(3, 12, 64, generator=g).bfloat16().cuda()
            before = [s.tokens(b, n[b])[2] for b in range(3)]
            lens += 1
            n = [x + 1 for x in n]
            pos = ints([p + 6 * turn + i for p in prompt])
            q, out = s.step(data, [1, 1, 1], lens, pos, 1, False)
            check(q, out, 1, before, False)
    assert max(n) <= max(total)


def test_a_replayed_graph_serves_as_the_calls_do():
    """append8, decode8 with weights and an eviction captured on a side stream and replayed with
    other tokens, lengths and weights."""
    a, b = Small(seed=2), Small(seed=2)
    g = torch.Generator().manual_seed(4)
    first = torch.randn(150, 12, 64, generator=g).bfloat16().cuda()
    pos = torch.cat([torch.arange(50)] * 3).to(torch.int32).cuda()
    for s in (a, b):
        s.step(first, [50] * 3, ints([50] * 3), pos, 4, True)
    qkv, p, lens = torch.zeros(3, 12, 64).bfloat16().cuda(), ints([50] * 3), ints([51] * 3)
    keep_lens = ints([0] * 3)
    kept = torch.zeros(3, 2, 32, dtype=torch.int32, device="cuda")
    cu = offsets([1, 1, 1])
    k, v, ks, vs = a.cache

    def calls():
        q = a.att.append8(qkv[:, :8], qkv[:, 8:10], qkv[:, 10:], *a.w, p, cu, a.tables[0], lens,
                          *a.cache)
        out = a.att.decode8(q, *a.cache, a.tables[0], lens, a.most, weights=a.weights)
        a.att.evict(k, v, a.weights, a.tables[0], lens, a.most, 32, 8, a.tables[1], k_scales=ks,
                    v_scales=vs, kept=kept, new_lens=keep_lens)
        return out

    saved = [x.clone() for x in a.cache + (a.weights,)]
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        calls()
    torch.cuda.current_stream().wait_stream(stream)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = calls()
    for x, y in zip(a.cache + (a.weights,), saved):
        x.copy_(y)
    for i in range(5):
        new = torch.randn(3, 12, 64, generator=g).bfloat16().cuda()
        qkv.copy_(new)
        p.fill_(50 + i)
        lens.fill_(51 + i)
        graph.replay()
        q, want = b.step(new, [1, 1, 1], ints([51 + i] * 3), ints([50 + i] * 3), 1, False)
        assert torch.equal(out, want) and torch.equal(a.weights[a.tables[0].long()],
                                                      b.weights[b.tables[0].long()])
        n = ints([51 + i] * 3)
        kb, vb, ksb, vsb = b.cache
        _, places = b.att.evict(kb, vb, b.weights, b.tables[0], n, b.most, 32, 8, b.tables[1],
                                k_scales=ksb, v_scales=vsb, new_lens=n)
        assert torch.equal(kept, places) and torch.equal(keep_lens, n)
        for x, y in zip(a.cache, b.cache):
            assert torch.equal(raw(x) if x.dtype == E4M3 else x, raw(y) if y.dtype == E4M3 else y)


def test_calls_of_two_streams_do_not_disturb_each_other():
    """An Attention each, on the same pages for reading: the same bits as one after the other."""
    s = Small(seed=6)
    g = torch.Generator().manual_seed(8)
    first = torch.randn(600, 12, 64, generator=g).bfloat16().cuda()
    pos = torch.cat([torch.arange(200)] * 3).to(torch.int32).cuda()
    s.step(first, [200] * 3, ints([200] * 3), pos, 4, True)
    from token_dispatch_grouped_gb300.attention import Attention
    q = torch.randn(3, 8, 64, generator=g).bfloat16().cuda()
    lens = ints([200, 150, 20])
    atts = [Attention(8, 2, 64) for _ in range(2)]
    ws = [s.weights.clone() for _ in range(3)]
    want = atts[0].decode8(q, *s.cache, s.tables[0], lens, 256, weights=ws[2])
    torch.cuda.synchronize()
    outs, streams = [], [torch.cuda.Stream() for _ in range(2)]
    for att, w, st in zip(atts, ws, streams):
        with torch.cuda.stream(st):
            for _ in range(3):
                w.copy_(s.weights)
                out = att.decode8(q, *s.cache, s.tables[0], lens, 256, weights=w)
            outs.append(out)
    torch.cuda.synchronize()
    for out, w in zip(outs, ws):
        assert torch.equal(out, want) and torch.equal(w, ws[2])
