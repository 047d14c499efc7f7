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
    values, on the current CUDA device. Tensors of heads are bf16 [tokens, heads, D] with
    dense values; their token and head strides are free (multiples of 8), so views
    of a fused projection are taken as they are.

    eps: of the RMS norm of the heads. rope_table: from rope_table() (None: no
    rotation); rope_layout "half" or "interleaved". scale: of the scores, by
    default D^-1/2. Calls run on the current stream. The workspace is kept, grows to the
    largest call and is shared by all of them: use one Attention per stream. Workspaces that
    were outgrown are kept too, as a captured CUDA graph goes on using the one that its calls
    were given: a graph holds as long as its Attention does."""

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
        self._ws = []  # the last one is in use

    # ---------------------------------------------------------------- checks
    def _heads(self, t, T: int, H: int, where: str) -> B.MoeHeads:
        """The view of t, a bf16 tensor [T, H, D] with dense values on the device."""
        if t.dtype is not torch.bfloat16 or t.shape != (T, H, self.D) or not t.is_cuda:
            raise B.MoeError(B.MOE_ERR_INVALID_ARG, where)
        ts, hs, vs = t.stride()
        if vs != 1 and T > 0:
            raise B.MoeError(B.MOE_ERR_INVALID_ARG, where)
        return B.MoeHeads(t.data_ptr(), ts, hs)

    def _ints(self, t, n: int, where: str, dtype=torch.int32) -> int:
        if t.dtype is not dtype or t.numel() != n or not t.is_contiguous() or not t.is_cuda:
            raise B.MoeError(B.MOE_ERR_INVALID_ARG, where)
        return t.data_ptr()

    def _norm(self, w, where: str) -> int | None:
        return None if w is None else self._ints(w, self.D, where, torch.float32)

    def _positions(self, positions, T: int, where: str) -> int | None:
        return None if self.table is None else self._ints(positions, T, where)

    def _out(self, T: int, H: int) -> torch.Tensor:
        return torch.empty(T, H, self.D, dtype=torch.bfloat16, device=self.device)

    def _workspace(self, nbytes: int):
        if nbytes == 0:
            return None
        if not self._ws or self._ws[-1].numel() < nbytes:
            # at least twice the last one: those kept for graphs stay smaller together
            # than the one in use
            least = 2 * self._ws[-1].numel() if self._ws else 0
            self._ws.append(torch.empty(max(nbytes, least), dtype=torch.uint8,
                                        device=self.device))
        return self._ws[-1]

    # ------------------------------------------------------- norm and positions
    def norm_rope(self, q, k, wq, wk, positions, q_out=None, k_out=None):
        """Normed (unless wq is None) and rotated (unless without a table) heads."""
        T, where = q.shape[0], "norm_rope"
        if q_out is None:
            q_out = self._out(T, self.Hq)
        if k_out is None:
            k_out = self._out(T, self.Hkv)
        B.moe_norm_rope(self.a, T, self._heads(q, T, self.Hq, where),
                        self._heads(k, T, self.Hkv, where), self._norm(wq, where),
                        self._norm(wk, where), self.eps, self._positions(positions, T, where),
                        self.rope, self._heads(q_out, T, self.Hq, where),
                        self._heads(k_out, T, self.Hkv, where))
        return q_out, k_out

    def norm_rope_backward(self, dq_out, dk_out, q, k, wq, wk, positions, dq=None, dk=None):
        """dq, dk, dwq, dwk (the last two None without a norm)."""
        T, where = q.shape[0], "norm_rope_backward"
        Hq, Hkv = self.Hq, self.Hkv
        if dq is None:
            dq = self._out(T, Hq)
        if dk is None:
            dk = self._out(T, Hkv)
        dwq = dwk = ws = None
        if wq is not None:
            dwq = torch.empty(self.D, dtype=torch.float32, device=self.device)
            dwk = torch.empty(self.D, dtype=torch.float32, device=self.device)
            ws = self._workspace(B.moe_norm_rope_workspace_size(self.a, T))
        B.moe_norm_rope_backward(self.a, T, self._heads(dq_out, T, Hq, where),
                                 self._heads(dk_out, T, Hkv, where),
                                 self._heads(q, T, Hq, where), self._heads(k, T, Hkv, where),
                                 self._norm(wq, where), self._norm(wk, where), self.eps,
                                 self._positions(positions, T, where), self.rope,
                                 self._heads(dq, T, Hq, where), self._heads(dk, T, Hkv, where),
                                 dwq, dwk, ws)
        return dq, dk, dwq, dwk

    # ------------------------------------------------------------ packed batches
    def _packed(self, Tq, Tk, cu_q, max_q, cu_k, max_k, causal, where):
        n = cu_q.numel()
        q = self._ints(cu_q, n, where)
        k = q if cu_k is None else self._ints(cu_k, n, where)
        return B.MoePacked(n - 1, Tq, Tk, max_q, max_q if cu_k is None else max_k, bool(causal), q,
                           k)

    def forward(self, q, k, v, cu_q, max_q, cu_k=None, max_k=None, causal=True, out=None,
                lse=None):
        """out [Tq, Hq, D] and lse [Tq, Hq] of the sequences between the offsets cu_q
        and cu_k (int32, on the device; cu_k = None: those of the queries). max_q and
        max_k bound their lengths. Rows of no sequence are not written."""
        Tq, Tk, Hq, Hkv, where = q.shape[0], k.shape[0], self.Hq, self.Hkv, "attention_forward"
        if out is None:
            out = self._out(Tq, Hq)
        if lse is None:
            lse = torch.empty(Tq, Hq, dtype=torch.float32, device=self.device)
        B.moe_attention_forward(self.a,
                                self._packed(Tq, Tk, cu_q, max_q, cu_k, max_k, causal, where),
                                self.scale, self._heads(q, Tq, Hq, where),
                                self._heads(k, Tk, Hkv, where), self._heads(v, Tk, Hkv, where),
                                self._heads(out, Tq, Hq, where),
                                self._ints(lse, Tq * Hq, where, torch.float32))
        return out, lse

    def backward(self, dout, q, k, v, out, lse, cu_q, max_q, cu_k=None, max_k=None, causal=True,
                 dq=None, dk=None, dv=None):
        """dq, dk, dv of forward(), at the rows that belong to a sequence."""
        Tq, Tk, Hq, Hkv, where = q.shape[0], k.shape[0], self.Hq, self.Hkv, "attention_backward"
        if dq is None:
            dq = self._out(Tq, Hq)
        if dk is None:
            dk = self._out(Tk, Hkv)
        if dv is None:
            dv = self._out(Tk, Hkv)
        s = self._packed(Tq, Tk, cu_q, max_q, cu_k, max_k, causal, where)
        B.moe_attention_backward(self.a, s, self.scale, self._heads(dout, Tq, Hq, where),
                                 self._heads(q, Tq, Hq, where), self._heads(k, Tk, Hkv, where),
                                 self._heads(v, Tk, Hkv, where), self._heads(out, Tq, Hq, where),
                                 self._ints(lse, Tq * Hq, where, torch.float32),
                                 self._heads(dq, Tq, Hq, where), self._heads(dk, Tk, Hkv, where),
                                 self._heads(dv, Tk, Hkv, where),
                                 self._workspace(
                                     B.moe_attention_backward_workspace_size(self.a, s)))
        return dq, dk, dv

    # --------------------------------------------------------------- paged cache
    def _cache(self, k_pages, v_pages, where):
        shape = k_pages.shape
        for x in (k_pages, v_pages):
            if x.dtype is not torch.bfloat16 or x.dim() != 4 or x.shape != shape or \
                    not x.is_contiguous() or not x.is_cuda:
                raise B.MoeError(B.MOE_ERR_INVALID_ARG, where)
        pages, heads, size, values = shape
        if heads != self.Hkv or values != self.D:
            raise B.MoeError(B.MOE_ERR_INVALID_ARG, where)
        return B.MoeKvCache(k_pages.data_ptr(), v_pages.data_ptr(), pages, size)

    def append(self, q, k, v, wq, wk, positions, slots, k_pages, v_pages, q_out=None):
        """norm_rope of new tokens; keys and values go to slots (int64) of the pages
        [pages, Hkv, page_size, D], the queries are returned."""
        T, where = q.shape[0], "append"
        if q_out is None:
            q_out = self._out(T, self.Hq)
        B.moe_kv_append(self.a, T, self._heads(q, T, self.Hq, where),
                        self._heads(k, T, self.Hkv, where), self._heads(v, T, self.Hkv, where),
                        self._norm(wq, where), self._norm(wk, where), self.eps,
                        self._positions(positions, T, where), self.rope,
                        self._ints(slots, T, where, torch.int64),
                        self._heads(q_out, T, self.Hq, where),
                        self._cache(k_pages, v_pages, where))
        return q_out

    def decode(self, q, k_pages, v_pages, block_table, kv_lens, max_kv, out=None):
        """Attention of the newest q.shape[0] / B tokens of B sequences, whose cached
        lengths (those tokens included) are kv_lens, at most max_kv. block_table
        [B, pages of a sequence] int32."""
        T, nb, where = q.shape[0], kv_lens.numel(), "decode"
        if out is None:
            out = self._out(T, self.Hq)
        if T == 0 and nb == 0:
            return out
        if nb == 0 or T % nb or T < nb or block_table.dtype is not torch.int32 or \
                block_table.dim() != 2 or not block_table.is_cuda:
            raise B.MoeError(B.MOE_ERR_INVALID_ARG, where)
        rows, wide = block_table.shape
        stride = block_table.stride()
        cache = self._cache(k_pages, v_pages, where)
        if rows != nb or (wide > 1 and stride[1] != 1) or (nb > 1 and stride[0] < wide) or \
                max_kv > wide * cache.page_size:
            raise B.MoeError(B.MOE_ERR_INVALID_ARG, where)
        n = T // nb
        ws = self._workspace(B.moe_attention_decode_workspace_size(self.a, nb, n, max_kv))
        B.moe_attention_decode(self.a, nb, n, max_kv, self.scale,
                               self._heads(q, T, self.Hq, where), cache, block_table.data_ptr(),
                               stride[0] if nb > 1 else wide, self._ints(kv_lens, nb, where),
                               self._heads(out, T, self.Hq, where), ws)
        return out

    def check_error(self) -> None:
        """Waits for the device and raises what it has reported since the last check. After a
        bad index (MOE_ERR_BAD_INDEX) the other rows and sequences hold."""
        rc = B.moe_get_error()
        if rc != B.MOE_OK:
            raise B.MoeError(rc, "device")
