"""The workspace of an Attention, which captured CUDA graphs go on using."""
import weakref

import pytest
import torch


def test_outgrown_workspaces_stay_allocated():
    """A larger call takes a larger workspace; the one that an earlier call was given stays
    allocated as long as the object, and all that are kept stay within twice the need."""
    from token_dispatch_grouped_gb300 import build
    build.build()
    from token_dispatch_grouped_gb300.attention import Attention
    att = Attention(4, 2, 64, device="cpu")
    assert att._workspace(0) is None
    first = att._workspace(1000)
    assert att._workspace(1000) is first and att._workspace(10) is first
    kept = [weakref.ref(first)]
    del first
    for n in (1001, 1500, 2500, 5000, 70000):
        w = att._workspace(n)
        assert w.numel() >= n and w.data_ptr() % 16 == 0
        if kept[-1]() is not w:
            kept.append(weakref.ref(w))
        del w
    assert all(r() is not None for r in kept)
    assert sum(r().numel() for r in kept[:-1]) < kept[-1]().numel() <= 2 * 70000
    del att
    assert all(r() is None for r in kept)


@pytest.mark.gpu
def test_a_graph_keeps_its_workspace():
    """decode captured for two batch sizes in ascending order with tokens split over CTAs,
    then larger calls and new tensors: replays give the plain call's bits and write nowhere
    else."""
    from token_dispatch_grouped_gb300 import binding as B
    from token_dispatch_grouped_gb300.attention import Attention
    from test_gpu_attention import offsets, paged, rnd
    B.moe_get_error()
    att, other, page, most = Attention(8, 2, 64), Attention(8, 2, 64), 16, 1600
    graphs = []
    for seqs in (2, 5):
        lens = [1500 - 70 * i for i in range(seqs)]
        k, v = rnd((sum(lens), 2, 64), 1), rnd((sum(lens), 2, 64), 2)
        kp, vp, table, _ = paged(k, v, lens, page, fill=0.0)
        wide = torch.zeros(seqs, most // page, dtype=torch.int32, device="cuda")
        wide[:, :table.shape[1]] = table.clamp(max=kp.shape[0] - 1)
        kv = torch.tensor(lens, dtype=torch.int32, device="cuda")
        q = rnd((seqs, 8, 64), 3).cuda()
        assert B.moe_attention_decode_workspace_size(att.a, seqs, 1, most) > 0
        args = (q, kp, vp, wide, kv, most)
        att.decode(*args)                  # the workspace comes from this stream's memory
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = att.decode(*args)
        graphs.append((graph, out, args))
    # a larger call of another kind, then tensors that fill what the allocator has free
    q, k = rnd((3000, 8, 64), 5).cuda(), rnd((3000, 2, 64), 6).cuda()
    cu = offsets([3000])
    o, lse = att.forward(q, k, k, cu, 3000)
    att.backward(q, q, k, k, o, lse, cu, 3000)
    guards = [torch.full((n,), 0x5a, dtype=torch.uint8, device="cuda")
              for n in [w.numel() for w in att._ws] * 8 + [1 << 16] * 32 + [1 << 20] * 8]
    for graph, out, args in graphs:
        args[0].copy_(rnd(tuple(args[0].shape), 9))
        graph.replay()
        assert torch.equal(out, other.decode(*args))
    assert all(bool((g == 0x5a).all()) for g in guards)
    assert B.moe_get_error() == B.MOE_OK
