"""The C ABI and the Python wrappers of the decode of shared prompts, the products with adapters and
the router by scores, on the CPU: bad arguments are refused with a status code (or an exception)
before anything touches the GPU."""
import ctypes

import pytest
import torch

SA_OK, SA_ERR_NULL, SA_ERR_SHAPE, SA_ERR_UNSUPPORTED, SA_ERR_ALIGNMENT = 0, 1, 2, 3, 7
FAKE = ctypes.c_void_p(0x10000)       # aligned, never dereferenced: rejected first
EIGHT, TWO, ODD = ctypes.c_void_p(0x10008), ctypes.c_void_p(0x10002), ctypes.c_void_p(0x10001)
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def lib():
    from attention_softmax_sinks_gb300 import _build
    import attention_softmax_sinks_gb300 as sa
    _build.build()
    return sa.load_library()


def _shared(lib, **kw):
    a = dict(q=FAKE, k=FAKE, v=FAKE, table=FAKE, lens=FAKE, sinks=FAKE, offsets=FAKE, pages=FAKE, batch=4, groups=2,
             hq=64, hkv=8, dim=64, page=16, max_pages=40, num_pages=100, max_shared=20, scale=0.125, ss=3, so=2,
             po=FAKE, pl=FAKE, out=FAKE, lse=FAKE)
    assert not kw.keys() - a.keys()
    a.update(kw)
    return lib.sink_attn_decode_shared(*a.values(), None)


@pytest.mark.parametrize("kw,status", [
    (dict(batch=-1), SA_ERR_SHAPE), (dict(batch=65536), SA_ERR_SHAPE), (dict(groups=0), SA_ERR_SHAPE),
    (dict(groups=-3), SA_ERR_SHAPE), (dict(groups=65536), SA_ERR_SHAPE), (dict(max_pages=0), SA_ERR_SHAPE),
    (dict(num_pages=0), SA_ERR_SHAPE), (dict(max_shared=-1), SA_ERR_SHAPE), (dict(max_shared=41), SA_ERR_SHAPE),
    (dict(max_pages=2 ** 26 + 1), SA_ERR_SHAPE), (dict(hq=0), SA_ERR_SHAPE), (dict(hkv=0), SA_ERR_SHAPE),
    (dict(hq=65), SA_ERR_SHAPE), (dict(hq=17, hkv=1), SA_ERR_UNSUPPORTED), (dict(dim=128), SA_ERR_UNSUPPORTED),
    (dict(page=32), SA_ERR_UNSUPPORTED), (dict(scale=NAN), SA_ERR_SHAPE), (dict(scale=INF), SA_ERR_SHAPE),
    (dict(ss=0), SA_ERR_SHAPE), (dict(ss=-1, so=1), SA_ERR_SHAPE), (dict(so=0), SA_ERR_SHAPE), (dict(ss=0, so=0), SA_ERR_SHAPE),
    (dict(ss=0, so=1, po=None, pl=None, q=None), SA_ERR_NULL), (dict(ss=0, so=1, po=None, pl=None, out=EIGHT), SA_ERR_ALIGNMENT), (dict(ss=255), SA_ERR_SHAPE),
    (dict(ss=2 ** 31 - 1, so=2 ** 31 - 1), SA_ERR_SHAPE),
    (dict(num_pages=2 ** 24, hkv=8), SA_ERR_SHAPE),                   # rows of the cache beyond 32 bits
    (dict(num_pages=2 ** 24 - 1, hkv=8, q=None), SA_ERR_NULL),        # just within them
    (dict(batch=65535, hq=65536, hkv=65536 // 16, num_pages=1), SA_ERR_SHAPE),
    (dict(batch=65535, hq=1024, hkv=1024, max_pages=2 ** 20, max_shared=2 ** 20, num_pages=1), SA_ERR_SHAPE),
    *((dict([(p, None)]), SA_ERR_NULL) for p in ("q", "k", "v", "table", "lens", "sinks", "offsets", "pages", "po", "pl", "out")),
    *((dict([(p, EIGHT)]), SA_ERR_ALIGNMENT) for p in ("q", "k", "v", "po", "out")),
    *((dict([(p, TWO)]), SA_ERR_ALIGNMENT) for p in ("table", "lens", "sinks", "offsets", "pages", "pl", "lse")),
    (dict(batch=0), SA_OK),
    (dict(batch=0, q=None, table=None, lens=None, offsets=None, pages=None, po=None, pl=None, out=None, lse=None), SA_OK),
])
def test_decode_of_shared_prompts_rejects(lib, kw, status):
    assert _shared(lib, **kw) == status


def test_splits_of_shared_prompts():
    import attention_softmax_sinks_gb300 as sa
    f = sa.sink_attn_decode_shared_splits
    for batch in (1, 2, 7, 64, 500, 65535):
        for groups in (1, 3, 64, 65535):
            for hq, hkv in ((1, 1), (64, 8), (40, 8), (16, 1), (128, 128)):
                for shared in (0, 1, 7, 128, 4096, 2 ** 26):
                    for own in (0, 1, 100, 4096):
                        s, o = f(batch, groups, hq, hkv, shared, shared + max(own, 1 if shared == 0 else 0))
                        assert (s, o) == (0, 1) or 2 <= s <= 40 and o in (1, 2, 4, 8)
                        # memory of the partial results beyond what one slot of each kind takes
                        assert batch * hq * 260 * (s - 2) <= 96 << 20
    for bad in ((0, 1, 64, 8, 4, 8), (4, 0, 64, 8, 4, 8), (4, 1, 8, 64, 4, 8), (4, 1, 64, 0, 4, 8), (4, 1, 64, 8, -1, 8),
                (4, 1, 64, 8, 0, 0), (-1, -1, -1, -1, -1, -1)):
        assert f(*bad) == (1, 1)
    assert f(64, 1, 64, 8, 2048, 2112) == f(64, 1, 64, 8, 2048, 2112, 152)
    assert f(4, 1, 64, 8, 16, 20) == (0, 1) and f(64, 1, 64, 8, 2048, 2112)[0] > 0


def test_splits_go_by_the_prompts_and_not_by_the_tables_width():
    import attention_softmax_sinks_gb300 as sa
    f = sa.sink_attn_decode_shared_splits
    for batch in (1, 4, 16, 37, 64, 512):
        for groups in (1, 5, 8):
            for hq, hkv in ((64, 8), (40, 8), (28, 4), (16, 1)):
                for shared in (1, 16, 128, 501, 2048):
                    tight = f(batch, groups, hq, hkv, shared, shared + 96)
                    for width in (shared + 100, 4096, 8192, 65536):
                        wide = f(batch, groups, hq, hkv, shared, width)
                        assert wide[0] == tight[0] and wide[1] >= tight[1]
                    # few of their own: SMs are moved between the parts, a slot or two with them
                    assert (f(batch, groups, hq, hkv, shared, shared + 4)[0] == 0) == (tight[0] == 0)
    assert f(4, 1, 64, 8, 128, 8192) == (0, 1)


def _lora(lib, **kw):
    a = dict(x=FAKE, w=FAKE, bias=FAKE, a=FAKE, b=FAKE, scale=FAKE, idx=FAKE, m=5, n=640, k=256, rank=16, adapters=3,
             ws=FAKE, out=FAKE)
    assert not kw.keys() - a.keys()
    a.update(kw)
    return lib.lora_linear_bias(*a.values(), None)


@pytest.mark.parametrize("kw,status", [
    (dict(m=-1), SA_ERR_SHAPE), (dict(n=0), SA_ERR_SHAPE), (dict(k=0), SA_ERR_SHAPE), (dict(n=-8), SA_ERR_SHAPE),
    (dict(n=2 ** 30 + 8), SA_ERR_SHAPE), (dict(k=2 ** 30 + 8), SA_ERR_SHAPE), (dict(rank=0), SA_ERR_SHAPE),
    (dict(rank=-8), SA_ERR_SHAPE), (dict(adapters=0), SA_ERR_SHAPE), (dict(adapters=1025), SA_ERR_SHAPE),
    (dict(n=641), SA_ERR_UNSUPPORTED), (dict(n=644), SA_ERR_UNSUPPORTED), (dict(k=252), SA_ERR_UNSUPPORTED),
    (dict(rank=12), SA_ERR_UNSUPPORTED), (dict(rank=136), SA_ERR_UNSUPPORTED),
    (dict(m=2 ** 23 - 127), SA_ERR_SHAPE),                          # more row blocks than a grid has
    (dict(m=2 ** 22, n=2 ** 20), SA_ERR_SHAPE),                     # more tiles than are counted
    (dict(adapters=1024, rank=128, k=2 ** 30, n=8), SA_ERR_SHAPE),
    *((dict([(p, None)]), SA_ERR_NULL) for p in ("x", "w", "a", "b", "idx", "ws", "out")),
    *((dict([(p, EIGHT)]), SA_ERR_ALIGNMENT) for p in ("x", "w", "a", "b", "ws", "out")),
    (dict(bias=ODD), SA_ERR_ALIGNMENT), (dict(scale=TWO), SA_ERR_ALIGNMENT), (dict(idx=TWO), SA_ERR_ALIGNMENT),
    (dict(m=0), SA_OK), (dict(m=0, x=None, w=None, a=None, b=None, idx=None, ws=None, out=None), SA_OK),
])
def test_product_with_adapters_rejects(lib, kw, status):
    assert _lora(lib, **kw) == status


def test_workspace_of_the_product_with_adapters():
    import attention_softmax_sinks_gb300 as sa
    assert sa.lora_workspace_bytes(1, 4096, 16) == 256
    assert sa.lora_workspace_bytes(2 ** 23 - 128, 8, 128) == 16 * 128 * (2 ** 23 - 128)
    for bad in ((0, 64, 16), (-1, 64, 16), (4, 0, 16), (4, 64, 0), (4, 64, 136)):
        assert sa.lora_workspace_bytes(*bad) == 0
    with pytest.raises(ValueError):
        sa.lora_workspace_bytes(2 ** 31, 64, 16)


def _scores(lib, **kw):
    a = dict(logits=FAKE, fp32=1, t=5, e=64, k=4, sigmoid=1, bias=FAKE, groups=8, top_groups=4, renorm=1, scale=2.5,
             idx=FAKE, w=FAKE, counts=None)
    assert not kw.keys() - a.keys()
    a.update(kw)
    return lib.moe_router_scores(*a.values(), None)


@pytest.mark.parametrize("kw,status", [
    (dict(t=-1), SA_ERR_SHAPE), (dict(e=0), SA_ERR_SHAPE), (dict(e=257, groups=1, top_groups=1), SA_ERR_SHAPE),
    (dict(groups=0), SA_ERR_SHAPE), (dict(groups=33, e=66), SA_ERR_SHAPE), (dict(groups=7), SA_ERR_SHAPE),
    (dict(top_groups=0), SA_ERR_SHAPE), (dict(top_groups=9), SA_ERR_SHAPE), (dict(k=0), SA_ERR_SHAPE),
    (dict(k=9), SA_ERR_SHAPE), (dict(k=5, e=32, groups=32, top_groups=4), SA_ERR_SHAPE),  # fewer experts than that are left
    (dict(scale=NAN), SA_ERR_SHAPE), (dict(scale=-INF), SA_ERR_SHAPE), (dict(t=2 ** 40), SA_ERR_SHAPE),
    (dict(logits=None), SA_ERR_NULL), (dict(idx=None), SA_ERR_NULL), (dict(w=None), SA_ERR_NULL),
    (dict(logits=TWO), SA_ERR_ALIGNMENT), (dict(logits=ODD, fp32=0), SA_ERR_ALIGNMENT), (dict(bias=TWO), SA_ERR_ALIGNMENT),
    (dict(idx=TWO), SA_ERR_ALIGNMENT), (dict(w=ODD), SA_ERR_ALIGNMENT), (dict(counts=TWO), SA_ERR_ALIGNMENT),
    (dict(t=0), SA_OK), (dict(t=0, logits=None, idx=None, w=None), SA_OK),
])
def test_router_by_scores_rejects(lib, kw, status):
    assert _scores(lib, **kw) == status


def test_wrappers_refuse_what_is_not_a_cuda_tensor_of_the_right_kind():
    import attention_softmax_sinks_gb300 as sa
    q, kv = torch.zeros(2, 8, 64, dtype=torch.bfloat16), torch.zeros(4, 1, 16, 64, dtype=torch.bfloat16)
    table, ints, sinks = torch.zeros(2, 2, dtype=torch.int32), torch.zeros(2, dtype=torch.int32), torch.zeros(8)
    x, w = torch.zeros(4, 64, dtype=torch.bfloat16), torch.zeros(32, 64, dtype=torch.bfloat16)
    a, b = torch.zeros(3, 16, 64, dtype=torch.bfloat16), torch.zeros(3, 32, 16, dtype=torch.bfloat16)
    idx = torch.zeros(4, dtype=torch.int32)
    calls = [lambda: sa.sink_attn_decode_shared(q, kv, kv, table, ints, sinks, ints, ints[:1], 1, 0.125),
             lambda: sa.sink_attn_decode_shared(None, kv, kv, table, ints, sinks, ints, ints[:1], 1, 0.125),
             lambda: sa.sink_attn_decode_shared(q, kv, kv, table, ints, sinks, None, ints[:1], 1, 0.125),
             lambda: sa.lora_linear_bias(x, w, a, b, idx), lambda: sa.lora_linear_bias(x, w, a, None, idx),
             lambda: sa.lora_linear_bias(x, w, a, b, None), lambda: sa.lora_linear_bias(x.half(), w, a, b, idx),
             lambda: sa.moe_router_scores(x, 2), lambda: sa.moe_router_scores(None, 2),
             lambda: sa.moe_router_scores(x.double(), 2), lambda: sa.moe_router_scores(x, 2, bias=x)]
    for call in calls:
        with pytest.raises((TypeError, ValueError)):
            call()
    for call in (lambda: sa.sink_attn_decode_shared(q[0], kv, kv, table, ints, sinks, ints, ints[:1], 1, 0.125),
                 lambda: sa.lora_linear_bias(x, w[0], a, b, idx), lambda: sa.moe_router_scores(x[0], 2),
                 lambda: sa.moe_router_scores(x, 2, score="relu")):
        with pytest.raises(ValueError):
            call()
