"""The operators of a small paged cache (8 bits a value, fewer tokens), as a program that
serves a decoder block calls them, and what each has to compute.

    append8         norm_rope of new tokens whose keys and values go into pages of e4m3
                    values with one power-of-two scale for each page and head
    decode8         attention of each sequence's newest tokens over those pages; `kept`:
                    every cached token's softmax weights are added up beside it
    decode_weights  the same sums over a bf16 cache
    evict           the heaviest and the newest tokens of every sequence and head go into
                    other pages, of bf16 or e4m3

`own` chooses the side: False computes the plain form (elementary torch operations in
32 bits, rounded once at the end), True makes the framework's calls. Pages of 8 bits come
back as the e4m3 values that they hold, with their scales beside them.
"""
import math
import random

import torch

own = False

EPS = 1e-6
BASE = 10000.0
TOP = 448.0              # the largest e4m3 value
E4M3 = torch.float8_e4m3fn


# ------------------------------------------------------------------ the cases
def listed():
    return [
        # One new token of each of eight sequences: latency.
        dict(name="append8 8x32/8x128", op="append8", tokens=8, seqs=8, Hq=32, Hkv=8, D=128,
             rot=128, layout="half", page=64, context=1500),
        # A prompt of 4096 tokens in three sequences that enters the cache.
        dict(name="append8 4096x32/8x128", op="append8", tokens=4096, seqs=3, Hq=32, Hkv=8, D=128,
             rot=128, layout="half", page=64, context=0),
        # A short odd batch that goes on in started pages, half of each head rotated.
        dict(name="append8 333x6/2x96", op="append8", tokens=333, seqs=4, Hq=6, Hkv=2, D=96,
             rot=48, layout="interleaved", page=16, context=77),
        # The next token of one sequence: latency.
        dict(name="decode8 1x1500", op="decode8", seqs=1, newest=1, longest=1500, Hq=32, Hkv=8,
             D=128, page=64, kept=False, fresh=False),
        # The next token of 64 sequences of up to 32768 tokens: the cache read once.
        dict(name="decode8 64x32768", op="decode8", seqs=64, newest=1, longest=32768, Hq=32, Hkv=8,
             D=128, page=64, kept=False, fresh=False),
        # The same step where the cache will be thinned out: weights added up.
        dict(name="decode8 64x32768 kept", op="decode8", seqs=64, newest=1, longest=32768, Hq=32,
             Hkv=8, D=128, page=64, kept=True, fresh=False),
        # The last 16 tokens of three prompts vote on what is kept of them, odd heads.
        dict(name="decode8 3x16x5000 fresh", op="decode8", seqs=3, newest=16, longest=5000, Hq=10,
             Hkv=2, D=80, page=16, kept=True, fresh=True),
        # The next token of one sequence, weights added up: latency.
        dict(name="decode_weights 1x1500", op="decode_weights", seqs=1, newest=1, longest=1500,
             Hq=32, Hkv=8, D=128, page=64, kept=True, fresh=False),
        # A serving batch on a bf16 cache.
        dict(name="decode_weights 32x8192", op="decode_weights", seqs=32, newest=1, longest=8192,
             Hq=32, Hkv=8, D=128, page=64, kept=True, fresh=False),
        # One long prompt cut to a quarter before it is served.
        dict(name="evict 1x32768", op="evict", seqs=1, longest=32768, keep=8192, recent=1024, Hq=32,
             Hkv=8, D=128, page=64, bits=16),
        # A short odd batch.
        dict(name="evict 5x777", op="evict", seqs=5, longest=777, keep=301, recent=33, Hq=6, Hkv=2,
             D=96, page=16, bits=8),
        # A serving batch on an 8-bit cache cut to a quarter.
        dict(name="evict 64x16384", op="evict", seqs=64, longest=16384, keep=4096, recent=256,
             Hq=32, Hkv=8, D=128, page=64, bits=8),
    ]


def _log(rng, lo, hi):
    """A whole number between lo and hi, spread over its logarithm."""
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    """One more case of the ranges above, of no more work than the largest of its kind."""
    most = {}
    for c in listed():
        w = work(c)
        a, b = most.get(c["op"], (0, 0))
        most[c["op"]] = max(a, w["flops"]), max(b, w["bytes"])
    while True:
        c = _drawn(rng)
        w = work(c)
        if w["flops"] <= most[c["op"]][0] and 0 < w["bytes"] <= most[c["op"]][1]:
            return c


def _drawn(rng):
    op = rng.choice(["append8", "decode8", "decode8", "decode_weights", "evict"])
    D = rng.choice([16, 48, 64, 64, 80, 96, 128, 128, 128])
    Hkv = rng.choice([1, 2, 4, 8])
    c = dict(op=op, Hq=Hkv * rng.choice([1, 2, 3, 4, 4, 5, 8]), Hkv=Hkv, D=D,
             page=rng.choice([8, 16, 64, 128]))
    if op == "append8":
        c["tokens"] = _log(rng, 1, 4096)
        c["seqs"] = min(c["tokens"], _log(rng, 1, 32))
        return dict(c, rot=rng.choice([D, D, D // 2 // 8 * 8]),
                    context=rng.choice([0, rng.randint(1, 1500)]),
                    layout=rng.choice(["half", "interleaved"]))
    c["seqs"] = _log(rng, 1, 64)
    if op == "evict":
        c.update(longest=_log(rng, 1, 32768), bits=rng.choice([8, 16]))
        keep = max(1, round(c["longest"] * rng.uniform(0.05, 1.1)))
        return dict(c, keep=keep, recent=rng.choice([0, keep, rng.randint(0, keep)]))
    newest = rng.choice([1, 1, 1, 2, 4, 16])
    kept = op == "decode_weights" or rng.random() < 0.5
    return dict(c, newest=newest, longest=_log(rng, 1, 32768 if op == "decode8" else 8192),
                kept=kept, fresh=kept and rng.random() < 0.3)


def _new_lengths(c):
    """(new tokens, cached tokens before them) of the sequences of an append8 case."""
    r = random.Random(c["tokens"] * 131 + c["seqs"])
    T, B = c["tokens"], c["seqs"]
    cuts = sorted(r.sample(range(1, T), B - 1)) if B > 1 else []
    at = [0] + cuts + [T]
    return [b - a for a, b in zip(at, at[1:])], [r.randint(c["context"] // 2, c["context"])
                                                for _ in range(B)]


def _kv_lengths(c):
    """Cached tokens of the sequences, the longest among them."""
    r = random.Random(c["longest"] * 131 + c["seqs"])
    lens = [max(1, round(c["longest"] * r.random())) for _ in range(c["seqs"])]
    lens[r.randrange(len(lens))] = c["longest"]
    return lens


# ------------------------------------------------------------------ the inputs
def _table(pages, order, dev):
    """[B, most pages] of consecutive pages in `order`, zeros past a sequence's."""
    wide, at = max(pages), 0
    first = []
    for n in pages:
        first.append(at)
        at += n
    col = torch.arange(wide, device=dev)[None]
    first, n = (torch.tensor(x, device=dev)[:, None] for x in (first, pages))
    t = torch.where(col < n, order[(first + col).clamp(max=order.numel() - 1)], 0)
    return t.to(torch.int32).contiguous()


def prepare(c, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    dev = "cuda"
    Hq, Hkv, D, P = c["Hq"], c["Hkv"], c["D"], c["page"]

    def normal(*shape):
        return torch.randn(*shape, generator=g, device=dev, dtype=torch.bfloat16)

    def ints(v):
        return torch.tensor(v, dtype=torch.int32, device=dev)

    def pages_of(n, bits):
        """A cache that has been written: values of about 1."""
        s = {}
        for x in ("k", "v"):
            p = normal(n, Hkv, P, D)
            if bits == 8:
                e = torch.randint(-8, -5, (n, Hkv), generator=g, device=dev)
                s[x + "_scales"] = torch.exp2(e.float())
                p = (p * 64).clamp_(-TOP, TOP).to(E4M3)
            s[x + "_pages"] = p
        return s

    s = dict(c)
    if c["op"] == "append8":
        new, before = _new_lengths(c)
        lens = [a + b for a, b in zip(new, before)]
        pages = [-(-n // P) for n in lens]
        N, T = sum(pages) + 2, c["tokens"]
        most = max(lens)
        inv = BASE ** (-torch.arange(0, c["rot"], 2, dtype=torch.float64, device=dev) / c["rot"])
        angle = torch.arange(most, dtype=torch.float64, device=dev)[:, None] * inv[None]
        s.update(pages_of(N, 8), qkv=normal(T, (Hq + 2 * Hkv) * D),
                 positions=torch.cat([torch.arange(b, b + n, device=dev, dtype=torch.int32)
                                      for n, b in zip(new, before)]),
                 rope_table=torch.stack([angle.cos(), angle.sin()], -1).float().contiguous(),
                 wq=1 + 0.1 * torch.randn(D, generator=g, device=dev),
                 wk=1 + 0.1 * torch.randn(D, generator=g, device=dev),
                 cu_new=ints([sum(new[:i]) for i in range(len(new) + 1)]), kv_lens=ints(lens),
                 block_table=_table(pages, torch.randperm(N, generator=g, device=dev), dev))
        return s
    lens = _kv_lengths(c)
    pages = [-(-n // P) for n in lens]
    s.update(kv_lens=ints(lens), max_kv=max(lens))
    if c["op"] == "evict":
        goal = [-(-min(n, c["keep"]) // P) for n in lens]
        N = sum(pages) + sum(goal) + 2
        order = torch.randperm(N, generator=g, device=dev)
        s.update(block_table=_table(pages, order, dev),
                 new_table=_table(goal, order[sum(pages):], dev), **pages_of(N, c["bits"]))
    else:
        N = sum(pages) + 3
        s.update(block_table=_table(pages, torch.randperm(N, generator=g, device=dev), dev),
                 q=normal(c["seqs"] * c["newest"], Hq, D),
                 **pages_of(N, 8 if c["op"] == "decode8" else 16))
    if c["op"] == "evict" or c["kept"]:
        # sums of softmax weights over some steps: a few tokens have most of them
        s["weights"] = torch.randn(N, Hkv, P, generator=g, device=dev).mul_(2).exp_().mul_(
            4 / c["longest"])
    return s


# ------------------------------------------------------------------ one pass
def run(s):
    return _own(s) if own else _PLAIN[s["op"]](s)


def _split(s):
    """Queries, keys and values of the fused projection, in place."""
    Hq, Hkv, D = s["Hq"], s["Hkv"], s["D"]
    x = s["qkv"].view(-1, Hq + 2 * Hkv, D)
    return x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:]


def _own(s):
    a = s.get("handle")
    if a is None:                        # kept from then on, as a program keeps its layer
        from token_dispatch_grouped_gb300.attention import Attention
        a = s["handle"] = Attention(s["Hq"], s["Hkv"], s["D"], eps=EPS,
                                    rope_table=s.get("rope_table"),
                                    rope_layout=s.get("layout", "half"))
    op = s["op"]
    if op == "append8":
        q, k, v = _split(s)
        out = a.append8(q, k, v, s["wq"], s["wk"], s["positions"], s["cu_new"], s["block_table"],
                        s["kv_lens"], s["k_pages"], s["v_pages"], s["k_scales"], s["v_scales"])
        return out, s["k_pages"], s["v_pages"], s["k_scales"], s["v_scales"]
    if op == "evict":
        lens, kept = a.evict(s["k_pages"], s["v_pages"], s["weights"], s["block_table"],
                             s["kv_lens"], s["max_kv"], s["keep"], s["recent"], s["new_table"],
                             k_scales=s.get("k_scales"), v_scales=s.get("v_scales"))
        return (lens, kept) + _cache_of(s)
    if op == "decode8":
        out = a.decode8(s["q"], s["k_pages"], s["v_pages"], s["k_scales"], s["v_scales"],
                        s["block_table"], s["kv_lens"], s["max_kv"], weights=s.get("weights"),
                        fresh=s["fresh"])
    else:
        out = a.decode(s["q"], s["k_pages"], s["v_pages"], s["block_table"], s["kv_lens"],
                       s["max_kv"], weights=s["weights"], fresh=s["fresh"])
    return (out, s["weights"]) if s["kept"] else out


def _cache_of(s):
    names = ["k_pages", "v_pages", "weights"]
    if s["bits"] == 8:
        names += ["k_scales", "v_scales"]
    return tuple(s[n] for n in names)


# ------------------------------------------------------------------ the plain forms
def _norm_rope_of(x, w, s):
    """Normed and rotated heads in 32 bits."""
    x = x.float()
    y = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * w
    r, half = s["rot"], s["rot"] // 2
    t = s["rope_table"][s["positions"].long()][:, None]
    cos, sin = t[..., 0], t[..., 1]
    if s["layout"] == "half":
        a, b = y[..., :half], y[..., half:r]
    else:
        a, b = y[..., 0:r:2], y[..., 1:r:2]
    a, b = a * cos - b * sin, b * cos + a * sin
    ab = torch.cat([a, b], -1) if s["layout"] == "half" else torch.stack([a, b], -1).flatten(-2)
    return torch.cat([ab, y[..., r:]], -1)


def _power(a):
    """The smallest power of two p with a <= 448 p (2^-100 at least)."""
    m, e = torch.frexp(a)                # a = m 2^e, m in [1/2, 1); 448 = 7/8 2^9
    e = torch.where(a > 0, e - 9 + (m > 0.875).to(e.dtype), -100).clamp(-100, 120)
    return ((e.to(torch.int32) + 127) << 23).view(torch.float32)


def _plain_append8(s):
    q, k, v = _split(s)
    P, T, Hkv = s["page"], q.shape[0], s["Hkv"]
    cu, lens = s["cu_new"].long(), s["kv_lens"].long()
    row = torch.arange(T, device=q.device)
    b = torch.searchsorted(cu, row, right=True) - 1
    tok = lens[b] - cu[b + 1] + row      # its place in the sequence
    page, at = s["block_table"].long()[b, tok // P], tok % P
    N = s["k_pages"].shape[0]
    # the first new row of every page that the call writes
    first = torch.full((N,), P, device=q.device).scatter_reduce_(0, page, at, "amin")
    written = first < P
    for x, name in ((_norm_rope_of(k, s["wk"], s), "k"), (v.float(), "v")):
        pages, scales = s[name + "_pages"], s[name + "_scales"]
        top = torch.zeros(N, Hkv, device=q.device).scatter_reduce_(
            0, page[:, None].expand(T, Hkv), x.abs().amax(-1), "amax")
        new = _power(top)
        new = torch.where((first > 0)[:, None], torch.maximum(new, scales), new)
        change = written & (first > 0)
        old = pages[change].float() * (scales / new)[change][:, :, None, None]
        keep = (torch.arange(P, device=q.device) < first[change][:, None])[:, None, :, None]
        pages[change] = torch.where(keep, old, pages[change].float()).to(E4M3)
        pages[page, :, at] = (x / new[page][:, :, None]).to(E4M3)
        scales.copy_(torch.where(written[:, None], new, scales))
    return (_norm_rope_of(q, s["wq"], s).bfloat16(), s["k_pages"], s["v_pages"], s["k_scales"],
            s["v_scales"])


def _cached(s, name, L):
    """[B, Hkv, L, ...] in 32 bits from pages [N, Hkv, P, ...]."""
    at, x = s["block_table"].long(), s[name + "_pages"]
    y = x[at].float()                    # [B, pages, Hkv, P, D]
    if name + "_scales" in s:
        y *= s[name + "_scales"][at][..., None, None]
    B, n, H, P, D = y.shape
    return y.transpose(1, 2).reshape(B, H, n * P, D)[:, :, :L]


def _plain_decode(s):
    Hq, Hkv, D, n, P = s["Hq"], s["Hkv"], s["D"], s["newest"], s["page"]
    B, G, L = s["seqs"], Hq // Hkv, s["max_kv"]
    q = s["q"].float().view(B, n, Hkv, G, D).permute(0, 2, 3, 1, 4).reshape(B, Hkv, G * n, D)
    lens = s["kv_lens"].long()[:, None, None]
    i, j = torch.arange(n, device=q.device)[:, None], torch.arange(L, device=q.device)
    seen = (j <= i + lens - n) & (j < lens)          # [B, n, L]
    x = (q @ _cached(s, "k", L).transpose(2, 3)).mul_(D ** -0.5).view(B, Hkv, G, n, L)
    x.masked_fill_(~seen[:, None, None], -math.inf)
    m = x.amax(-1, keepdim=True)
    p = x.sub_(m.masked_fill(m == -math.inf, 0)).exp_()
    p /= p.sum(-1, keepdim=True).clamp_min(1e-38)
    out = p.view(B, Hkv, G * n, L) @ _cached(s, "v", L)
    out = out.view(B, Hkv, G, n, D).permute(0, 3, 1, 2, 4).reshape(B * n, Hq, D).bfloat16()
    if not s["kept"]:
        return out
    w, at = s["weights"], s["block_table"].long()
    add = p.sum((2, 3))                              # [B, Hkv, L]
    b, t = ((j < lens[:, 0])).nonzero(as_tuple=True)
    page, off = at[b, t // P], t % P
    had = w[page, :, off]
    if s["fresh"]:
        had = torch.zeros_like(had)
    had = torch.where((t >= s["kv_lens"][b] - n)[:, None], torch.zeros_like(had), had)
    w[page, :, off] = had + add[b, :, t]
    return out, w


def _plain_evict(s):
    P, L, keep, recent = s["page"], s["max_kv"], s["keep"], s["recent"]
    at, lens, N = s["block_table"].long(), s["kv_lens"].long(), s["weights"].shape[0]
    B, Hkv, dev = s["seqs"], s["Hkv"], at.device
    w = s["weights"][at].transpose(1, 2).reshape(B, Hkv, -1)[:, :, :L]
    j, n = torch.arange(L, device=dev), lens[:, None, None]
    w = w.masked_fill((j >= n - recent) | (n <= keep), math.inf).masked_fill(j >= n, -math.inf)
    kept = torch.sort(w, dim=-1, descending=True, stable=True)[1][:, :, :keep]
    new = torch.clamp(lens, max=keep)
    most = kept.shape[2]                 # min(keep, L)
    real = torch.arange(most, device=dev) < new[:, None, None]
    kept = torch.where(real, kept, L).sort(-1)[0]
    out = torch.full((B, Hkv, keep), -1, dtype=torch.int32, device=dev)
    out[:, :, :most] = torch.where(real, kept, -1).int()
    # (sequence, head, place) of every kept token, its page and the one it goes to
    b, h, i = real.expand(B, Hkv, most).nonzero(as_tuple=True)
    t = kept[b, h, i]
    page, off = at[b, t // P], t % P
    goal, to = s["new_table"].long()[b, i // P], i % P
    for name in ("k", "v"):
        pages = s[name + "_pages"]
        x = pages[page, h, off]
        if s["bits"] == 8:
            scales = s[name + "_scales"]
            old = scales[page, h]
            scale = torch.zeros(N * Hkv, device=dev).scatter_reduce_(0, goal * Hkv + h, old, "amax")
            scale = scale.view(N, Hkv)
            x = (x.float() * (old / scale[goal, h])[:, None]).to(E4M3)
            scales.copy_(torch.where(scale > 0, scale, scales))
        pages[goal, h, to] = x
    s["weights"][goal, h, to] = s["weights"][page, h, off]
    return (new.int(), out) + _cache_of(s)


_PLAIN = dict(append8=_plain_append8, decode8=_plain_decode, decode_weights=_plain_decode,
              evict=_plain_evict)


# ------------------------------------------------------------------ the exact results
def _exact_append8(c, s):
    """The pages' values come unrounded, in units of their scale."""
    new, before = _new_lengths(c)
    q, k, v = (t.double() for t in _split(s))
    r, h, P = c["rot"], c["rot"] // 2, c["page"]
    inv = BASE ** (-torch.arange(0, r, 2, dtype=torch.float64, device="cuda") / r)
    angle = s["positions"].double()[:, None] * inv
    z = torch.complex(angle.cos().float().double(), angle.sin().float().double())[:, None]
    i = torch.arange(h, device="cuda")
    a, b = (i, i + h) if c["layout"] == "half" else (2 * i, 2 * i + 1)

    def turned(x, w):
        y = x / (x.pow(2).sum(-1, keepdim=True) / x.shape[-1] + EPS).sqrt() * w.double()
        u = torch.complex(y[..., a], y[..., b]) * z
        y[..., a], y[..., b] = u.real, u.imag
        return y

    got = [turned(q, s["wq"])]
    table = s["block_table"].tolist()
    scales = []
    for x, name in ((turned(k, s["wk"]), "k"), (v, "v")):
        pages, scale = s[name + "_pages"].double(), s[name + "_scales"].double()
        row = 0
        for n, m, line in zip(new, before, table):
            t = m
            while t < m + n:             # page by page
                g, o = line[t // P], t % P
                e = min(P - o, m + n - t)
                part = x[row:row + e].transpose(0, 1)        # [Hkv, e, D]
                top = part.abs().amax((1, 2)) / TOP
                m2, e2 = torch.frexp(top)                # powers of two are 1/2 2^e2
                want = torch.ldexp(torch.ones_like(top), e2 - (m2 == 0.5).to(e2.dtype))
                if o > 0:
                    want = torch.maximum(want, scale[g])
                    pages[g, :, :o] *= (scale[g] / want)[:, None, None]
                pages[g, :, o:o + e] = part / want[:, None, None]
                scale[g] = want
                t, row = t + e, row + e
        got.append(pages)
        scales.append(scale)
    return (*got, *scales)


def _exact_decode(c, s):
    Hq, Hkv, D, n, P = c["Hq"], c["Hkv"], c["D"], c["newest"], c["page"]
    G = Hq // Hkv
    out = torch.zeros(c["seqs"], n, Hq, D, dtype=torch.float64, device="cuda")
    w = s["weights"].double() if c["kept"] else None
    q = s["q"].double().view_as(out)
    for b, m in enumerate(_kv_lengths(c)):
        used = s["block_table"][b, :-(-m // P)].long()
        kv = []
        for x in ("k", "v"):
            y = s[x + "_pages"][used].double()
            if c["op"] == "decode8":
                y = y * s[x + "_scales"][used].double()[:, :, None, None]
            kv.append(y.transpose(0, 1).reshape(Hkv, -1, D)[:, :m])
        add = torch.zeros(Hkv, used.numel() * P, dtype=torch.float64, device="cuda")
        for h in range(Hq):
            x = (q[b, :, h] @ kv[0][h // G].T) / math.sqrt(D)
            x += torch.full_like(x, -math.inf).triu(m - n + 1)
            p = torch.softmax(x, -1).nan_to_num(0.0)   # rows that see nothing: none of it
            out[b, :, h] = p @ kv[1][h // G]
            add[h // G, :m] += p.sum(0)
        if c["kept"]:
            had = w[used].transpose(0, 1).reshape(Hkv, -1).clone()
            had[:, 0 if c["fresh"] else max(0, m - n):m] = 0
            w[used] = (had + add).view(Hkv, -1, P).transpose(0, 1)
    out = out.view(-1, Hq, D)
    return (out, w) if c["kept"] else out


def _exact_evict(c, s):
    """The 8-bit pages' values come unrounded, in units of their scale."""
    P, Hkv, keep, recent = c["page"], c["Hkv"], c["keep"], c["recent"]
    lens = _kv_lengths(c)
    names = _cache_of(s)
    pages = [x.double() for x in names[:2]]
    weights = s["weights"]
    moved = weights.double()
    scales = [x.double() for x in names[3:]]
    kept = torch.full((len(lens), Hkv, keep), -1, dtype=torch.int32, device="cuda")
    for b, m in enumerate(lens):
        used, n = s["block_table"][b, :-(-m // P)].long(), min(m, keep)
        w = weights[used].transpose(0, 1).reshape(Hkv, -1)[:, :m].double()
        pick = torch.ones(Hkv, m, dtype=torch.bool, device="cuda")
        if m > keep:
            pick[:, :m - recent] = False
            if keep > recent:            # the heaviest of the others: above the last one's
                old = w[:, :m - recent]  # weight, and the first that have just that
                last = old.sort(-1)[0][:, recent - keep][:, None]
                more, same = old > last, old == last
                room = keep - recent - more.sum(-1, keepdim=True)
                pick[:, :m - recent] = more | (same & (same.cumsum(-1) <= room))
        t = pick.nonzero()[:, 1].view(Hkv, n)
        kept[b, :, :n] = t.int()
        h = torch.arange(Hkv, device="cuda")[:, None]
        page, off = used[t // P], t % P
        i = torch.arange(n, device="cuda")
        goal = s["new_table"][b].long()[i // P]
        moved[goal, h, i % P] = weights.double()[page, h, off]
        for x, (all_, src) in enumerate(zip(pages, names[:2])):
            y = src[page, h, off].double()
            if scales:
                old = names[3 + x].double()[page, h]           # [Hkv, n]
                pad = torch.zeros(Hkv, -(-n // P) * P, dtype=torch.float64, device="cuda")
                pad[:, :n] = old
                top = pad.view(Hkv, -1, P).amax(-1)
                scales[x][s["new_table"][b, :top.shape[1]].long()] = top.T
                y = y * (old / top[:, i // P])[..., None]
            all_[goal, h, i % P] = y
    new = torch.tensor([min(m, keep) for m in lens], dtype=torch.int32, device="cuda")
    return (new, kept, *pages, moved, *scales)


def exact(c, seed):
    s = prepare(c, seed)
    if c["op"] == "append8":
        return _exact_append8(c, s)
    return _exact_evict(c, s) if c["op"] == "evict" else _exact_decode(c, s)


# ------------------------------------------------------------------ the least work
def work(c):
    """Bytes (each input read once, each output written once) and flops of one pass."""
    Hq, Hkv, D, P = c["Hq"], c["Hkv"], c["D"], c["page"]
    if c["op"] == "append8":
        T = c["tokens"]
        new, before = _new_lengths(c)
        pages = sum(-(-(n + m) // P) - m // P for n, m in zip(new, before))
        table = 4 * c["rot"] * len({p for n, m in zip(new, before) for p in range(m, m + n)})
        return {"bytes": 2 * T * (Hq + 2 * Hkv) * D + 2 * T * Hq * D + 2 * T * Hkv * D + 4 * T
                + table + 8 * D + pages * (8 * Hkv + 4) + 8 * c["seqs"] + 4,
                "flops": T * (9 * (Hq + Hkv) + 3 * Hkv) * D}
    lens = _kv_lengths(c)
    pages = sum(-(-n // P) for n in lens)
    if c["op"] == "evict":
        new = [min(n, c["keep"]) for n in lens]
        goal = sum(-(-n // P) for n in new)
        size = c["bits"] // 8
        cut = sum(n for n in lens if n > c["keep"])
        whole = sum(n for n in lens if n <= c["keep"])
        data = sum(new) * Hkv * (4 * D * size + 4 + 4)         # rows twice, weight and index out
        data += 4 * Hkv * (cut + whole) + 4 * (pages + goal + 2 * len(lens))
        if size == 1:
            data += 8 * Hkv * (pages + goal)
        return {"bytes": data, "flops": Hkv * cut}
    rows = c["seqs"] * c["newest"]
    size = 1 if c["op"] == "decode8" else 2
    data = sum(lens) * Hkv * D * 2 * size + rows * Hq * D * 4 + 4 * (pages + len(lens))
    if size == 1:
        data += 8 * Hkv * pages
    seen = sum(max(0, n - i) for n in lens for i in range(c["newest"]))
    flops = 4 * D * Hq * seen
    if c["kept"]:
        data += (4 if c["fresh"] else 8) * Hkv * sum(lens)
        flops += Hq * seen
    return {"bytes": data, "flops": flops}
