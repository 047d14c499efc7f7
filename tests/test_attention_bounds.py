"""Host side of the cache's bounds (CPU): more cached tokens than 32-bit arithmetic holds."""


def test_more_cached_tokens_than_supported_are_refused():
    from token_dispatch_grouped_gb300 import build
    build.build()
    from token_dispatch_grouped_gb300 import binding as B
    a, at = B.MoeAttnShape(4, 2, 64), 1 << 20   # an aligned address that no refused call reads
    q = B.MoeHeads(at, 256, 64)
    cache = B.MoeKvCache(at, at, 5, 16)
    for most in ((1 << 30) + 1, (1 << 31) - 1):
        assert B.LIB.moe_attention_decode(a, 2, 1, most, 0.125, q, cache, at, (1 << 31) - 1, at, q,
                                          at, 1 << 40, None) == B.MOE_ERR_UNSUPPORTED_SHAPE
        assert B.moe_attention_decode_workspace_size(a, 2, 1, most) == 0
    assert B.moe_attention_decode_workspace_size(a, 2, 1, 1 << 30) > 0
