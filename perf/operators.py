"""The attention operators beside the MoE layer, as a program that trains or serves
a decoder block calls them, and what each has to compute.

    norm_rope       RMS norm of every query and key head, then the rotary positions
    norm_rope_grad  its backward: dq, dk and the gradients of the two norm weights
    attention       softmax attention over packed sequences (causal or full, grouped
                    heads), out and the log-sum-exp of every row
    attention_step  that forward and its backward: out, lse, dq, dk, dv
    append          norm_rope of new tokens whose keys and values go into a paged cache
    decode          attention of each sequence's newest tokens over its paged cache

`own` chooses the side: False computes the plain form (elementary torch operations in
32 bits, rounded once at the end), True makes the framework's calls.
"""
import math
import random

import torch

own = False

EPS = 1e-6
BASE = 10000.0


# ------------------------------------------------------------------ the cases
def listed():
    return [
        # One step's tokens of the 32-head, d = 4096 layer, T = 4096, queries and keys
        # read in place from the fused projection.
        dict(name="norm_rope 4096x32/8x128", op="norm_rope", tokens=4096, seqs=3, Hq=32, Hkv=8,
             D=128, rot=128, layout="half"),
        # The d = 512 layer's 32 sequences of 2048 tokens: narrow heads, half of each
        # head rotated, interleaved pairs.
        dict(name="norm_rope 65536x8/8x64", op="norm_rope", tokens=65536, seqs=32, Hq=8, Hkv=8,
             D=64, rot=32, layout="interleaved"),
        # A short odd batch, where the launches count.
        dict(name="norm_rope_grad 333x6/2x96", op="norm_rope_grad", tokens=333, seqs=4, Hq=6,
             Hkv=2, D=96, rot=96, layout="half"),
        # The d = 2048 layer's batch of 16384 tokens.
        dict(name="norm_rope_grad 16384x16/4x128", op="norm_rope_grad", tokens=16384, seqs=5,
             Hq=16, Hkv=4, D=128, rot=128, layout="half"),
        # A ragged packed batch of T = 4096 tokens.
        dict(name="attention 4096x32/8x128", op="attention", tokens=4096, seqs=5, Hq=32, Hkv=8,
             D=128, causal=True, context=0),
        # One long sequence of 16384 tokens.
        dict(name="attention 16384x16/4x128", op="attention", tokens=16384, seqs=1, Hq=16, Hkv=4,
             D=128, causal=True, context=0),
        # A short odd batch in training, one head group of three.
        dict(name="attention_step 777x6/2x96", op="attention_step", tokens=777, seqs=4, Hq=6,
             Hkv=2, D=96, causal=True, context=0),
        # Long sequences in training.
        dict(name="attention_step 8192x32/8x128", op="attention_step", tokens=8192, seqs=1, Hq=32,
             Hkv=8, D=128, causal=True, context=0),
        # One new token of each of eight sequences.
        dict(name="append 8x32/8x128", op="append", tokens=8, seqs=8, Hq=32, Hkv=8, D=128, rot=128,
             layout="half", page=64, context=1500),
        # A prompt of 4096 tokens in three sequences that enters the cache.
        dict(name="append 4096x32/8x128", op="append", tokens=4096, seqs=3, Hq=32, Hkv=8, D=128,
             rot=128, layout="half", page=64, context=0),
        # The next token of one sequence: latency.
        dict(name="decode 1x1500", op="decode", seqs=1, newest=1, longest=1500, Hq=32, Hkv=8, D=128,
             page=64),
        # The next token of 64 sequences of up to 32768 tokens: the cache read once.
        dict(name="decode 64x32768", op="decode", seqs=64, newest=1, longest=32768, Hq=32, Hkv=8,
             D=128, page=64),
    ]


def _log(rng, lo, hi):
    """A whole number between lo and hi, spread over its logarithm."""
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    """One more case of the ranges above, of no more work than the largest of its kind."""
    most = {}
    for c in listed():
        w = work(c)
        most[c["op"]] = max(most.get(c["op"], (0, 0)), (w["flops"], w["bytes"]))
    while True:
        c = _drawn(rng)
        w = work(c)
        if 0 < w["flops"] <= most[c["op"]][0] and w["bytes"] <= most[c["op"]][1] and _fits(c):
            return c


def _drawn(rng):
    op = rng.choice(["norm_rope", "norm_rope_grad", "attention", "attention_step", "append",
                     "decode"])
    D = rng.choice([64, 64, 80, 96, 128, 128, 128])
    Hkv = rng.choice([1, 2, 4, 8])
    c = dict(op=op, Hq=Hkv * rng.choice([1, 2, 3, 4, 4, 5, 8]), Hkv=Hkv, D=D)
    if op == "decode":
        return dict(c, seqs=_log(rng, 1, 64), newest=rng.choice([1, 1, 1, 2, 4]),
                    longest=_log(rng, 1, 32768), page=rng.choice([16, 64, 128]))
    c["tokens"] = _log(rng, 1, {"append": 4096, "attention": 16384, "attention_step": 8192}.get(
        op, 65536))
    c["seqs"] = min(c["tokens"], _log(rng, 1, 32))
    if op in ("attention", "attention_step"):
        return dict(c, causal=rng.random() < 0.75,
                    context=rng.choice([0, 0, 0, rng.randint(1, 1500), -rng.randint(1, 40)]))
    c.update(rot=rng.choice([D, D, D // 2 // 8 * 8]), layout=rng.choice(["half", "interleaved"]))
    if op == "append":
        c.update(page=rng.choice([16, 64, 128]), context=rng.choice([0, rng.randint(1, 3000)]))
    return c


def _fits(c):
    """Whether the plain form's padded score matrices fit the card."""
    if c["op"] not in ("attention", "attention_step"):
        return True
    lq, lk = _lengths(c)
    return len(lq) * max(lq) * max(lk) * c["Hq"] <= (
        8192 * 8192 * 32 if c["op"] == "attention_step" else 16384 * 16384 * 16)


def _lengths(c):
    """Query and key lengths of the packed sequences: a function of the case alone."""
    r = random.Random(c["tokens"] * 131 + c["seqs"])
    cuts = sorted(r.sample(range(1, c["tokens"]), c["seqs"] - 1)) if c["seqs"] > 1 else []
    if c["op"] == "append" and c["tokens"] == c["seqs"]:
        cuts = list(range(1, c["tokens"]))
    at = [0] + cuts + [c["tokens"]]
    lq = [b - a for a, b in zip(at, at[1:])]
    return lq, [max(0, n + c.get("context", 0)) for n in lq]


def _kv_lengths(c):
    """Cached tokens of the sequences of a decode case, the longest among them."""
    r = random.Random(c["longest"] * 131 + c["seqs"])
    lens = [max(1, round(c["longest"] * r.random())) for _ in range(c["seqs"])]
    lens[r.randrange(len(lens))] = c["longest"]
    return lens


def _pairs(c):
    """Visible (query, key) pairs of a packed batch, for one head."""
    if not c["causal"]:
        return sum(a * b for a, b in zip(*_lengths(c)))
    n = 0
    for a, b in zip(*_lengths(c)):
        first = max(0, a - b)            # queries before it see no key
        n += sum((i + b - a + 1 for i in (first, a - 1))) * (a - first) // 2 if a > first else 0
    return n


# ------------------------------------------------------------------ the inputs
def prepare(c, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    dev = "cuda"

    def normal(*shape):
        return torch.randn(*shape, generator=g, device=dev, dtype=torch.bfloat16)

    def ints(v):
        return torch.tensor(v, dtype=torch.int32, device=dev)

    Hq, Hkv, D = c["Hq"], c["Hkv"], c["D"]
    s = dict(c)
    if c["op"] == "decode":
        lens = _kv_lengths(c)
        pages = [-(-n // c["page"]) for n in lens]
        N, wide = sum(pages) + 3, max(pages)
        order = torch.randperm(N, generator=g, device=dev).to(torch.int32)
        at = torch.arange(wide, device=dev)[None]
        first = ints([sum(pages[:i]) for i in range(len(pages))])[:, None]
        table = torch.where(at < ints(pages)[:, None], order[(first + at).clamp(max=N - 1)], 0)
        s.update(q=normal(c["seqs"] * c["newest"], Hq, D), k_pages=normal(N, Hkv, c["page"], D),
                 v_pages=normal(N, Hkv, c["page"], D), block_table=table.to(torch.int32).contiguous(),
                 kv_lens=ints(lens), max_kv=max(lens))
        return s
    T = c["tokens"]
    lq, lk = _lengths(c)
    if c["op"] in ("attention", "attention_step"):
        at = lambda v: [sum(v[:i]) for i in range(len(v) + 1)]  # noqa: E731
        s.update(q=normal(T, Hq, D), k=normal(sum(lk), Hkv, D), v=normal(sum(lk), Hkv, D),
                 cu_q=ints(at(lq)), cu_k=ints(at(lk)), max_q=max(lq), max_k=max(lk))
        if c["op"] == "attention_step":
            s["dout"] = normal(T, Hq, D)
        return s
    start = [n - m if m >= n else 0 for n, m in zip(lk, lq)] if c["op"] == "append" else [0] * len(lq)
    positions = torch.cat([torch.arange(a, a + n, device=dev, dtype=torch.int32)
                           for a, n in zip(start, lq)])
    most = max(a + n for a, n in zip(start, lq))
    inv = BASE ** (-torch.arange(0, c["rot"], 2, dtype=torch.float64, device=dev) / c["rot"])
    angle = torch.arange(most, dtype=torch.float64, device=dev)[:, None] * inv[None]
    s.update(qkv=normal(T, (Hq + 2 * Hkv) * D), positions=positions,
             rope_table=torch.stack([angle.cos(), angle.sin()], -1).float().contiguous(),
             wq=1 + 0.1 * torch.randn(D, generator=g, device=dev),
             wk=1 + 0.1 * torch.randn(D, generator=g, device=dev))
    if c["op"] == "norm_rope_grad":
        s.update(dq_out=normal(T, Hq, D), dk_out=normal(T, Hkv, D))
    if c["op"] == "append":
        P = c["page"]
        pages = [-(-(a + n) // P) for a, n in zip(start, lq)]
        N = sum(pages) + 2
        order = torch.randperm(N, generator=g, device=dev)
        first = torch.cat([torch.full((n,), sum(pages[:i]), device=dev, dtype=torch.int64)
                           for i, n in enumerate(lq)])
        s.update(k_pages=normal(N, Hkv, P, D), v_pages=normal(N, Hkv, P, D),
                 slots=order[first + positions.long() // P] * P + positions.long() % P)
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
    if op == "norm_rope":
        q, k, _ = _split(s)
        return a.norm_rope(q, k, s["wq"], s["wk"], s["positions"])
    if op == "norm_rope_grad":
        q, k, _ = _split(s)
        return a.norm_rope_backward(s["dq_out"], s["dk_out"], q, k, s["wq"], s["wk"],
                                    s["positions"])
    if op == "append":
        q, k, v = _split(s)
        out = a.append(q, k, v, s["wq"], s["wk"], s["positions"], s["slots"], s["k_pages"],
                       s["v_pages"])
        return out, s["k_pages"], s["v_pages"]
    if op == "decode":
        return a.decode(s["q"], s["k_pages"], s["v_pages"], s["block_table"], s["kv_lens"],
                        s["max_kv"])
    out, lse = a.forward(s["q"], s["k"], s["v"], s["cu_q"], s["max_q"], s["cu_k"], s["max_k"],
                         causal=s["causal"])
    if op == "attention":
        return out, lse
    return (out, lse) + a.backward(s["dout"], s["q"], s["k"], s["v"], out, lse, s["cu_q"],
                                   s["max_q"], s["cu_k"], s["max_k"], causal=s["causal"])


# ------------------------------------------------------------------ the plain forms
def _pairs_of(x, rot, layout):
    """The rotated pairs (a, b) of the first `rot` values, and the rest."""
    if layout == "half":
        return x[..., :rot // 2], x[..., rot // 2:rot], x[..., rot:]
    return x[..., 0:rot:2], x[..., 1:rot:2], x[..., rot:]


def _joined(a, b, rest, layout):
    ab = torch.cat([a, b], -1) if layout == "half" else torch.stack([a, b], -1).flatten(-2)
    return torch.cat([ab, rest], -1)


def _cos_sin(s):
    t = s["rope_table"][s["positions"].long()][:, None]
    return t[..., 0], t[..., 1]


def _norm_rope_of(x, w, s):
    x = x.float()
    y = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * w
    a, b, rest = _pairs_of(y, s["rot"], s["layout"])
    cos, sin = _cos_sin(s)
    return _joined(a * cos - b * sin, b * cos + a * sin, rest, s["layout"]).bfloat16()


def _plain_norm_rope(s):
    q, k, _ = _split(s)
    return _norm_rope_of(q, s["wq"], s), _norm_rope_of(k, s["wk"], s)


def _norm_rope_grad_of(dout, x, w, s):
    a, b, rest = _pairs_of(dout.float(), s["rot"], s["layout"])
    cos, sin = _cos_sin(s)
    dy = _joined(a * cos + b * sin, b * cos - a * sin, rest, s["layout"])
    x = x.float()
    r = torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS)
    n = x * r
    dn = dy * w
    return (r * (dn - n * (dn * n).mean(-1, keepdim=True))).bfloat16(), (dy * n).sum((0, 1))


def _plain_norm_rope_grad(s):
    q, k, _ = _split(s)
    dq, dwq = _norm_rope_grad_of(s["dq_out"], q, s["wq"], s)
    dk, dwk = _norm_rope_grad_of(s["dk_out"], k, s["wk"], s)
    return dq, dk, dwq, dwk


def _plain_append(s):
    q, k, v = _split(s)
    page, at = s["slots"] // s["page"], s["slots"] % s["page"]
    s["k_pages"][page, :, at] = _norm_rope_of(k, s["wk"], s)
    s["v_pages"][page, :, at] = v
    return _norm_rope_of(q, s["wq"], s), s["k_pages"], s["v_pages"]


def _padded(x, cu, longest):
    """Packed rows as [B, longest, ...] in 32 bits, zeros past each length."""
    at = torch.arange(longest, device=x.device)
    n = (cu[1:] - cu[:-1])[:, None]
    x = x[(cu[:-1, None] + at).clamp(max=x.shape[0] - 1).long()].float()
    return x * (at < n)[(...,) + (None,) * (x.dim() - 2)]


def _packed(x, cu, T):
    """The packed rows [T, ...] of [B, longest, ...]."""
    t = torch.arange(T, device=x.device, dtype=cu.dtype)
    b = torch.searchsorted(cu, t, right=True) - 1
    return x[b, (t - cu[b]).long()]


def _softmax_of(x, mask):
    """(weights, log-sum-exp) of the last axis; a row without a value has weights 0."""
    x.masked_fill_(~mask, -math.inf)
    m = x.amax(-1, keepdim=True)
    m0 = m.masked_fill(m == -math.inf, 0)
    p = x.sub_(m0).exp_()
    l = p.sum(-1, keepdim=True)
    lse = (m0 + l.log()).squeeze(-1)
    return p.div_(l.clamp_min(1e-38)), lse


def _plain_forward(s):
    Hq, Hkv, D = s["Hq"], s["Hkv"], s["D"]
    cu_q, cu_k, Lq, Lk = s["cu_q"], s["cu_k"], s["max_q"], s["max_k"]
    B, G, T = cu_q.numel() - 1, Hq // Hkv, s["q"].shape[0]
    if Lk == 0:
        return (torch.zeros_like(s["q"]),
                torch.full((T, Hq), -math.inf, device=s["q"].device)), None
    q = _padded(s["q"], cu_q, Lq).view(B, Lq, Hkv, G, D).permute(0, 2, 3, 1, 4)
    q = q.reshape(B, Hkv, G * Lq, D)
    k = _padded(s["k"], cu_k, Lk).transpose(1, 2)
    v = _padded(s["v"], cu_k, Lk).transpose(1, 2)
    lq, lk = (cu_q[1:] - cu_q[:-1])[:, None, None], (cu_k[1:] - cu_k[:-1])[:, None, None]
    i, j = torch.arange(Lq, device=q.device)[:, None], torch.arange(Lk, device=q.device)
    mask = j < lk
    if s["causal"]:
        mask = mask & (j <= i + lk - lq)
    mask = mask.expand(B, Lq, Lk)[:, None, None]
    x = (q @ k.transpose(2, 3)).mul_(D ** -0.5).view(B, Hkv, G, Lq, Lk)
    p, lse = _softmax_of(x, mask)
    p = p.view(B, Hkv, G * Lq, Lk)
    out = p @ v

    def back(y):                         # [B, Hkv, G*Lq, ...] to packed [T, Hq, ...]
        y = y.reshape(B, Hkv, G, Lq, -1).permute(0, 3, 1, 2, 4).reshape(B, Lq, Hq, -1)
        return _packed(y, cu_q, T)

    return (back(out).bfloat16(), back(lse)[..., 0].contiguous()), (q, k, v, p, out, back)


def _plain_attention(s):
    return _plain_forward(s)[0]


def _plain_attention_step(s):
    (out, lse), kept = _plain_forward(s)
    if kept is None:
        return out, lse, torch.zeros_like(s["q"]), torch.zeros_like(s["k"]), torch.zeros_like(s["v"])
    q, k, v, p, o, back = kept
    B, Hkv, rows, D = q.shape
    G = s["Hq"] // Hkv
    do = _padded(s["dout"], s["cu_q"], s["max_q"]).view(B, -1, Hkv, G, D).permute(0, 2, 3, 1, 4)
    do = do.reshape(B, Hkv, rows, D)
    dv = p.transpose(2, 3) @ do
    ds = (do @ v.transpose(2, 3)).sub_((do * o).sum(-1, keepdim=True)).mul_(p).mul_(D ** -0.5)
    dq, dk = ds @ k, ds.transpose(2, 3) @ q
    Tk = s["k"].shape[0]
    return (out, lse, back(dq).bfloat16(), _packed(dk.transpose(1, 2), s["cu_k"], Tk).bfloat16(),
            _packed(dv.transpose(1, 2), s["cu_k"], Tk).bfloat16())


def _plain_decode(s):
    Hq, Hkv, D, n = s["Hq"], s["Hkv"], s["D"], s["newest"]
    B, G, L = s["seqs"], Hq // Hkv, s["max_kv"]
    at = s["block_table"].long()

    def cached(pages):                   # [B, Hkv, L, D]
        return pages[at].permute(0, 2, 1, 3, 4).reshape(B, Hkv, -1, D)[:, :, :L].float()

    q = s["q"].float().view(B, n, Hkv, G, D).permute(0, 2, 3, 1, 4).reshape(B, Hkv, G * n, D)
    lens = s["kv_lens"][:, None, None]
    i, j = torch.arange(n, device=q.device)[:, None], torch.arange(L, device=q.device)
    mask = (j <= i + lens - n).expand(B, n, L)[:, None, None]
    x = (q @ cached(s["k_pages"]).transpose(2, 3)).mul_(D ** -0.5).view(B, Hkv, G, n, L)
    p, _ = _softmax_of(x, mask)
    out = p.view(B, Hkv, G * n, L) @ cached(s["v_pages"])
    return out.view(B, Hkv, G, n, D).permute(0, 3, 1, 2, 4).reshape(B * n, Hq, D).bfloat16()


_PLAIN = dict(norm_rope=_plain_norm_rope, norm_rope_grad=_plain_norm_rope_grad,
              attention=_plain_attention, attention_step=_plain_attention_step,
              append=_plain_append, decode=_plain_decode)


# ------------------------------------------------------------------ the exact results
def _exact_rotation(c, positions):
    """[T, rot/2] complex rotations, from the 32-bit table that both sides are given."""
    inv = BASE ** (-torch.arange(0, c["rot"], 2, dtype=torch.float64, device="cuda") / c["rot"])
    angle = positions.double()[:, None] * inv
    return torch.complex(angle.cos().float().double(), angle.sin().float().double())


def _exact_rotate(x, z, c):
    """x [T, H, D] in 64 bits with its pairs multiplied by z [T, rot/2]."""
    r, h = c["rot"], c["rot"] // 2
    i = torch.arange(h, device=x.device)
    a, b = (i, i + h) if c["layout"] == "half" else (2 * i, 2 * i + 1)
    w = torch.complex(x[..., a], x[..., b]) * z[:, None]
    y = x.clone()
    y[..., a], y[..., b] = w.real, w.imag
    return y


def _exact_norm(x, w):
    return x / (x.pow(2).sum(-1, keepdim=True) / x.shape[-1] + EPS).sqrt() * w


def _exact_attention(q, k, v, scale, causal):
    """out, lse and weights of one head: q [n, D], k, v [m, D], in 64 bits."""
    x = scale * (q @ k.T)
    if causal:
        x += torch.full_like(x, -math.inf).triu(k.shape[0] - q.shape[0] + 1)
    lse = torch.logsumexp(x, -1)
    p = torch.exp(x - lse.clamp_min(-1e300)[:, None]) if k.shape[0] else x
    return p @ v, lse, p


def exact(c, seed):
    s = prepare(c, seed)
    Hq, Hkv, D, G = c["Hq"], c["Hkv"], c["D"], c["Hq"] // c["Hkv"]
    if c["op"] == "decode":
        out = torch.zeros(c["seqs"], c["newest"], Hq, D, dtype=torch.float64, device="cuda")
        q = s["q"].double().view_as(out)
        for b, n in enumerate(_kv_lengths(c)):
            used = s["block_table"][b, :-(-n // c["page"])].long()
            k, v = (s[x][used].double().transpose(0, 1).reshape(Hkv, -1, D)[:, :n]
                    for x in ("k_pages", "v_pages"))
            for h in range(Hq):
                out[b, :, h] = _exact_attention(q[b, :, h], k[h // G], v[h // G], D ** -0.5,
                                                True)[0]
        return out.view(-1, Hq, D)
    if c["op"] in ("attention", "attention_step"):
        q, k, v = s["q"].double(), s["k"].double(), s["v"].double()
        out, dq, dk, dv = (torch.zeros_like(t) for t in (q, q, k, v))
        lse = torch.full(q.shape[:2], -math.inf, dtype=torch.float64, device="cuda")
        a0 = b0 = 0
        for n, m in zip(*_lengths(c)):
            a, b = slice(a0, a0 + n), slice(b0, b0 + m)
            a0, b0 = a0 + n, b0 + m
            for h in range(Hq if n and m else 0):
                g = h // G
                o, l, p = _exact_attention(q[a, h], k[b, g], v[b, g], D ** -0.5, c["causal"])
                out[a, h], lse[a, h] = o, l
                if c["op"] == "attention_step":
                    do = s["dout"][a, h].double()
                    dp = do @ v[b, g].T
                    ds = p * (dp - (p * dp).sum(-1, keepdim=True)) * D ** -0.5
                    dv[b, g] += p.T @ do
                    dq[a, h] = ds @ k[b, g]
                    dk[b, g] += ds.T @ q[a, h]
        return (out, lse) if c["op"] == "attention" else (out, lse, dq, dk, dv)
    z = _exact_rotation(c, s["positions"])
    q, k, v = (t.double() for t in _split(s))
    wq, wk = s["wq"].double(), s["wk"].double()
    if c["op"] == "norm_rope_grad":
        got = []
        for x, w, d in ((q, wq, s["dq_out"]), (k, wk, s["dk_out"])):
            dy = _exact_rotate(d.double(), z.conj(), c)
            ms = x.pow(2).mean(-1, keepdim=True) + EPS
            dx = dy * w / ms.sqrt() - x * (dy * w * x).mean(-1, keepdim=True) / ms ** 1.5
            got.append((dx, (dy * x / ms.sqrt()).flatten(0, 1).sum(0)))
        return got[0][0], got[1][0], got[0][1], got[1][1]
    q = _exact_rotate(_exact_norm(q, wq), z, c)
    k = _exact_rotate(_exact_norm(k, wk), z, c)
    if c["op"] == "norm_rope":
        return q, k
    k_pages, v_pages = s["k_pages"].double(), s["v_pages"].double()
    for pages, x in ((k_pages, k), (v_pages, v)):
        for h in range(Hkv):
            pages[:, h][s["slots"] // c["page"], s["slots"] % c["page"]] = x[:, h]
    return q, k_pages, v_pages


# ------------------------------------------------------------------ the least work
def work(c):
    """Bytes (each input read once, each output written once) and flops of one pass."""
    Hq, Hkv, D = c["Hq"], c["Hkv"], c["D"]
    if c["op"] == "decode":
        lens, rows = _kv_lengths(c), c["seqs"] * c["newest"]
        cached = sum(lens) * Hkv * D * 4
        pages = sum(-(-n // c["page"]) for n in lens)
        seen = sum(max(0, n - i) for n in lens for i in range(c["newest"]))
        return {"bytes": cached + rows * Hq * D * 4 + 4 * (pages + len(lens)),
                "flops": 4 * D * Hq * seen}
    T = c["tokens"]
    if c["op"] in ("attention", "attention_step"):
        Tk = sum(_lengths(c)[1])
        data = 2 * D * (2 * T * Hq + 2 * Tk * Hkv) + 4 * T * Hq + 8 * (c["seqs"] + 1)
        flops = 4 * D * Hq * _pairs(c)
        if c["op"] == "attention":
            return {"bytes": data, "flops": flops}
        return {"bytes": 2 * D * (4 * T * Hq + 4 * Tk * Hkv) + 4 * T * Hq + 8 * (c["seqs"] + 1),
                "flops": flops * 7 // 2}
    rows = T * (Hq + Hkv) * D
    # the table's rows that some position reads, once each
    table = 4 * c["rot"] * (T if c["op"] == "append" and c["tokens"] == c["seqs"]
                            else max(_lengths(c)[0]))
    if c["op"] == "norm_rope":
        return {"bytes": 4 * rows + 4 * T + table + 8 * D, "flops": 9 * rows}
    if c["op"] == "norm_rope_grad":
        return {"bytes": 6 * rows + 4 * T + table + 16 * D, "flops": 17 * rows}
    return {"bytes": 4 * rows + 4 * T * Hkv * D + 12 * T + table + 8 * D, "flops": 9 * rows}
