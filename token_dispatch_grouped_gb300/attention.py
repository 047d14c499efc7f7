"""Buffer management around the attention operators of the C ABI
(include/moe_attention.h): checks that the tensors are what the call takes,
allocates outputs and workspaces with torch and calls the entry points. Every step
runs in the CUDA library."""
from __future__ import annotations

import math

import torch

from . import binding as B


def rope_inv_freq(dims: int, base: float = 10000.0, scaling: str | None = None,
                  factor: float = 1.0, original: int = 4096, slow: float = 1.0,
                  fast: float = 32.0) -> tuple[torch.Tensor, float]:
    """(frequencies [dims / 2] fp64, scale of the table) of the rotary positions.

    theta_i = base^(-2 i / dims), i < dims / 2. For contexts `factor` times as long
    as the `original` one:
      "linear"  theta_i / factor (interpolated positions);
      "ntk"     base * factor^(dims / (dims - 2)): the fastest pair keeps its
                frequency, the slowest is interpolated;
      "yarn"    pairs that turn more than `fast` times within the original context
                keep theta_i, those that turn less than `slow` times are
                interpolated, with a linear ramp between, and the table (so both
                query and key) is scaled by 0.1 ln(factor) + 1.
    """
    if dims < 0 or dims % 2:
        raise ValueError("dims is even and not negative")
    i = torch.arange(0, dims, 2, dtype=torch.float64)
    if scaling == "ntk" and dims > 2:
        base = base * factor ** (dims / (dims - 2))
    theta = base ** (-i / max(dims, 1))
    if scaling in (None, "ntk"):
        return theta, 1.0
    if scaling == "linear":
        return theta / factor, 1.0
    if scaling == "yarn":
        turns = original * theta / (2 * math.pi)
        keep = ((turns - slow) / (fast - slow)).clamp(0, 1)
        return theta * keep + theta / factor * (1 - keep), \
            0.1 * math.log(factor) + 1.0 if factor > 1 else 1.0
    raise ValueError(f"scaling {scaling!r}: None, 'linear', 'ntk' or 'yarn'")


def rope_table(positions: int, inv_freq: torch.Tensor, scale: float = 1.0,
               device="cuda") -> torch.Tensor:
    """(cos, sin) of every position: fp32 [positions, dims / 2, 2]."""
    inv = inv_freq.to(device=device, dtype=torch.float64).contiguous()
    out = torch.empty(positions, inv.numel(), 2, dtype=torch.float32, device=device)
    B.moe_rope_table(positions, 2 * inv.numel(), inv, scale, out)
    return out


class Attention:
    """The attention of a decoder block: Hq query heads on Hkv key/value heads of D
    values, on a CUDA device. Tensors of heads are bf16 [tokens, heads, D] with
    dense values; their token and head strides are free (multiples of 8), so views
    of a fused projection are taken as they are.

    eps: of the RMS norm of the heads. rope_table: from rope_table() (None: no
    rotation); rope_layout "half" or "interleaved". scale: of the scores, by
    default D^-1/2. The workspace is kept and grows to the largest call."""

    def __init__(self, Hq: int, Hkv: int, D: int, device="cuda", eps: float = 1e-6,
                 rope_table: torch.Tensor | None = None, rope_layout: str = "half",
                 scale: float | None = None):
        self.a = B.MoeAttnShape(Hq, Hkv, D)
        self.Hq, self.Hkv, self.D = Hq, Hkv, D
        self.device = torch.device(device)
        self.eps = eps
        self.scale = D ** -0.5 if scale is None else scale
        self.table = rope_table  # kept alive: the views below point into it
        if rope_table is None:
            self.rope = B.MoeRope(None, 0, 0, 0)
        else:
            if rope_table.dtype != torch.float32 or not rope_table.is_contiguous() or \
                    rope_table.dim() != 3 or rope_table.shape[2] != 2 or not rope_table.is_cuda:
                raise B.MoeError(B.MOE_ERR_INVALID_ARG, "Attention: rope_table")
            self.rope = B.MoeRope(rope_table.data_ptr(), rope_table.shape[0],
                                  2 * rope_table.shape[1], B.ROPE_LAYOUTS[rope_layout])
        self._ws = None

    # ---------------------------------------------------------------- checks
    def _heads(self, t, T: int, H: int, where: str):
        if t.dtype != torch.bfloat16 or t.dim() != 3 or t.shape[0] != T or t.shape[1] != H or \
                t.shape[2] != self.D or (t.stride(2) != 1 and self.D > 1 and T > 0) or \
                not t.is_cuda:
            raise B.MoeError(B.MOE_ERR_INVALID_ARG, where)
        return t

    def _ints(self, t, n: int, where: str, dtype=torch.int32):
        if t.dtype != dtype or t.numel() != n or not t.is_contiguous() or not t.is_cuda:
            raise B.MoeError(B.MOE_ERR_INVALID_ARG, where)
        return t

    def _norm(self, wq, wk, where: str):
        for w in (wq, wk):
            if w is not None and (w.dtype != torch.float32 or w.numel() != self.D or
                                  not w.is_contiguous() or not w.is_cuda):
                raise B.MoeError(B.MOE_ERR_INVALID_ARG, where)

    def _out(self, T: int, H: int) -> torch.Tensor:
        return torch.empty(T, H, self.D, dtype=torch.bfloat16, device=self.device)

    def _workspace(self, nbytes: int):
        if nbytes == 0:
            return None
        if self._ws is None or self._ws.numel() < nbytes:
            self._ws = torch.empty(nbytes, dtype=torch.uint8, device=self.device)
        return self._ws

    # ------------------------------------------------------- norm and positions
    def norm_rope(self, q, k, wq, wk, positions, q_out=None, k_out=None):
        """Normed (unless wq is None) and rotated (unless without a table) heads."""
        T, where = q.shape[0], "norm_rope"
        self._heads(q, T, self.Hq, where)
        self._heads(k, T, self.Hkv, where)
        self._norm(wq, wk, where)
        if self.table is not None:
            self._ints(positions, T, where)
        q_out = self._out(T, self.Hq) if q_out is None else self._heads(q_out, T, self.Hq, where)
        k_out = self._out(T, self.Hkv) if k_out is None else self._heads(k_out, T, self.Hkv, where)
        B.moe_norm_rope(self.a, T, q, k, wq, wk, self.eps, positions, self.rope, q_out, k_out)
        return q_out, k_out

    def norm_rope_backward(self, dq_out, dk_out, q, k, wq, wk, positions, dq=None, dk=None):
        """dq, dk, dwq, dwk (the last two None without a norm)."""
        T, where = q.shape[0], "norm_rope_backward"
        for x in (dq_out, q):
            self._heads(x, T, self.Hq, where)
        for x in (dk_out, k):
            self._heads(x, T, self.Hkv, where)
        self._norm(wq, wk, where)
        if self.table is not None:
            self._ints(positions, T, where)
        dq = self._out(T, self.Hq) if dq is None else self._heads(dq, T, self.Hq, where)
        dk = self._out(T, self.Hkv) if dk is None else self._heads(dk, T, self.Hkv, where)
        dwq = dwk = ws = None
        if wq is not None:
            dw = torch.empty(2, self.D, dtype=torch.float32, device=self.device)
            dwq, dwk = dw[0], dw[1]
            ws = self._workspace(B.moe_norm_rope_workspace_size(self.a, T))
        B.moe_norm_rope_backward(self.a, T, dq_out, dk_out, q, k, wq, wk, self.eps, positions,
                                 self.rope, dq, dk, dwq, dwk, ws)
        return dq, dk, dwq, dwk

    # ------------------------------------------------------------ packed batches
    def _packed(self, q, k, cu_q, max_q, cu_k, max_k, causal, where):
        self._ints(cu_q, cu_q.numel(), where)
        self._ints(cu_k, cu_q.numel(), where)
        return B.MoePacked(cu_q.numel() - 1, q.shape[0], k.shape[0], max_q, max_k, int(causal),
                           cu_q.data_ptr(), cu_k.data_ptr())

    def forward(self, q, k, v, cu_q, max_q, cu_k=None, max_k=None, causal=True, out=None,
                lse=None):
        """out [Tq, Hq, D] and lse [Tq, Hq] of the sequences between the offsets cu_q
        and cu_k (int32, on the device; cu_k = None: those of the queries). max_q and
        max_k bound their lengths."""
        where = "attention_forward"
        cu_k, max_k = (cu_q, max_q) if cu_k is None else (cu_k, max_k)
        Tq, Tk = q.shape[0], k.shape[0]
        self._heads(q, Tq, self.Hq, where)
        self._heads(k, Tk, self.Hkv, where)
        self._heads(v, Tk, self.Hkv, where)
        out = self._out(Tq, self.Hq) if out is None else self._heads(out, Tq, self.Hq, where)
        if lse is None:
            lse = torch.empty(Tq, self.Hq, dtype=torch.float32, device=self.device)
        else:
            self._ints(lse, Tq * self.Hq, where, torch.float32)
        s = self._packed(q, k, cu_q, max_q, cu_k, max_k, causal, where)
        B.moe_attention_forward(self.a, s, self.scale, q, k, v, out, lse)
        return out, lse

    def backward(self, dout, q, k, v, out, lse, cu_q, max_q, cu_k=None, max_k=None, causal=True,
                 dq=None, dk=None, dv=None):
        """dq, dk, dv of forward()."""
        where = "attention_backward"
        cu_k, max_k = (cu_q, max_q) if cu_k is None else (cu_k, max_k)
        Tq, Tk = q.shape[0], k.shape[0]
        for x in (dout, q, out):
            self._heads(x, Tq, self.Hq, where)
        for x in (k, v):
            self._heads(x, Tk, self.Hkv, where)
        self._ints(lse, Tq * self.Hq, where, torch.float32)
        dq = self._out(Tq, self.Hq) if dq is None else self._heads(dq, Tq, self.Hq, where)
        dk = self._out(Tk, self.Hkv) if dk is None else self._heads(dk, Tk, self.Hkv, where)
        dv = self._out(Tk, self.Hkv) if dv is None else self._heads(dv, Tk, self.Hkv, where)
        s = self._packed(q, k, cu_q, max_q, cu_k, max_k, causal, where)
        ws = self._workspace(B.moe_attention_backward_workspace_size(self.a, s))
        B.moe_attention_backward(self.a, s, self.scale, dout, q, k, v, out, lse, dq, dk, dv, ws)
        return dq, dk, dv

    # --------------------------------------------------------------- paged cache
    def _cache(self, k_pages, v_pages, where):
        for x in (k_pages, v_pages):
            if x.dtype != torch.bfloat16 or x.dim() != 4 or x.shape != k_pages.shape or \
                    x.shape[1] != self.Hkv or x.shape[3] != self.D or not x.is_contiguous() or \
                    not x.is_cuda:
                raise B.MoeError(B.MOE_ERR_INVALID_ARG, where)
        return B.MoeKvCache(k_pages.data_ptr(), v_pages.data_ptr(), k_pages.shape[0],
                            k_pages.shape[2])

    def append(self, q, k, v, wq, wk, positions, slots, k_pages, v_pages, q_out=None):
        """norm_rope of new tokens; keys and values go to slots (int64) of the pages
        [pages, Hkv, page_size, D], the queries are returned."""
        T, where = q.shape[0], "append"
        self._heads(q, T, self.Hq, where)
        self._heads(k, T, self.Hkv, where)
        self._heads(v, T, self.Hkv, where)
        self._norm(wq, wk, where)
        if self.table is not None:
            self._ints(positions, T, where)
        self._ints(slots, T, where, torch.int64)
        cache = self._cache(k_pages, v_pages, where)
        q_out = self._out(T, self.Hq) if q_out is None else self._heads(q_out, T, self.Hq, where)
        B.moe_kv_append(self.a, T, q, k, v, wq, wk, self.eps, positions, self.rope, slots, q_out,
                        cache)
        return q_out

    def decode(self, q, k_pages, v_pages, block_table, kv_lens, max_kv, out=None):
        """Attention of the newest q.shape[0] / B tokens of B sequences, whose cached
        lengths (those tokens included) are kv_lens, at most max_kv."""
        T, nb, where = q.shape[0], kv_lens.numel(), "decode"
        self._heads(q, T, self.Hq, where)
        self._ints(kv_lens, nb, where)
        if T == 0 and nb == 0:
            return self._out(0, self.Hq) if out is None else out
        if nb == 0 or T % nb or T < nb or block_table.dtype != torch.int32 or \
                block_table.dim() != 2 or block_table.shape[0] != nb or \
                block_table.stride(1) != 1 or not block_table.is_cuda or \
                (nb > 1 and block_table.stride(0) < block_table.shape[1]):
            raise B.MoeError(B.MOE_ERR_INVALID_ARG, where)
        cache = self._cache(k_pages, v_pages, where)
        if max_kv > block_table.shape[1] * k_pages.shape[2]:
            raise B.MoeError(B.MOE_ERR_INVALID_ARG, where)
        out = self._out(T, self.Hq) if out is None else self._heads(out, T, self.Hq, where)
        n = T // nb
        ws = self._workspace(B.moe_attention_decode_workspace_size(self.a, nb, n, max_kv))
        stride = block_table.stride(0) if nb > 1 else block_table.shape[1]
        B.moe_attention_decode(self.a, nb, n, max_kv, self.scale, q, cache, block_table, stride,
                               kv_lens, out, ws)
        return out

    def check_error(self) -> None:
        rc = B.moe_get_error()
        if rc != B.MOE_OK:
            raise B.MoeError(rc, "device")
