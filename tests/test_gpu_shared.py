"""Decode of a batch that shares prompts, against attention in 64 bits over each whole sequence.

Tolerances.  P is rounded to bf16 before it is multiplied with V and the result once more at the
end; each rounding is off by at most half a step, 2^-8 of the value.  With A = sum_j p_j |v_j| the
output is therefore within 2^-8 (A + |out|), plus 2^-13 A for the fp32 scores: 64 products and
their sum are off by at most 64 * 2^-24 sum |q k| sm_scale < 2^-13.5 for the inputs here, and
exp2 and the sums add some 2^-20.  lse: the same 2^-13, and 2^-22 |lse|."""
import pytest
import torch

pytestmark = pytest.mark.gpu
PAGE, DIM, SCALE = 16, 64, 0.125
NAN, INF = float("nan"), float("inf")


def make(groups, own, hq, hkv, seed=0, spare=3, extra_width=2, sink_std=1.0):
    """groups: (sequences, shared pages) per group; own: tokens of each sequence behind them.
    Pages that no sequence uses, and what lies behind a sequence's last token, hold NaN."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    n_seq = sum(n for n, _ in groups)
    assert len(own) == n_seq
    starts, lens, rows, used = [0], [], [], 0
    for n, pages in groups:
        common = list(range(used, used + pages))
        used += pages
        for _ in range(n):
            mine = (own[len(lens)] + PAGE - 1) // PAGE
            rows.append(common + list(range(used, used + mine)))
            used += mine
            lens.append(pages * PAGE + own[len(lens)])
        starts.append(starts[-1] + n)
    num_pages = max(used, 1) + spare
    place = torch.randperm(num_pages, generator=g, device="cuda").to(torch.int32)
    width = max([len(r) for r in rows] + [1]) + extra_width
    table = torch.full((n_seq, width), -1, dtype=torch.int32, device="cuda")
    for b, r in enumerate(rows):
        if r:
            table[b, : len(r)] = place[torch.tensor(r, device="cuda")]

    def normal(*shape):
        return torch.randn(*shape, generator=g, device="cuda").to(torch.bfloat16)

    k, v = normal(num_pages, hkv, PAGE, DIM), normal(num_pages, hkv, PAGE, DIM)
    for x in (k, v):
        x[place[used:].long()] = NAN
        for b, n in enumerate(lens):
            if n % PAGE:
                x[table[b, n // PAGE].long(), :, n % PAGE :] = NAN
    ints = lambda values: torch.tensor(values, dtype=torch.int32, device="cuda")
    return dict(q=normal(n_seq, hq, DIM), paged_k=k, paged_v=v, page_table=table, kv_lens=ints(lens),
                sinks=sink_std * torch.randn(hq, generator=g, device="cuda"), group_offsets=ints(starts),
                shared_pages=ints([p for _, p in groups]), max_shared_pages=max([p for _, p in groups]), sm_scale=SCALE)


def reference(a):
    """out, lse and A = sum p |v| in 64 bits, sequence by sequence."""
    q = a["q"].double()
    n_seq, hq, _ = q.shape
    hkv = a["paged_k"].shape[1]
    out, lse, mag = torch.zeros_like(q), torch.zeros(n_seq, hq, dtype=torch.float64, device="cuda"), torch.zeros_like(q)
    for b, n in enumerate(a["kv_lens"].tolist()):
        ids = a["page_table"][b, : (n + PAGE - 1) // PAGE].long()
        k = a["paged_k"][ids].double().transpose(0, 1).reshape(hkv, -1, DIM)[:, :n].repeat_interleave(hq // hkv, 0)
        v = a["paged_v"][ids].double().transpose(0, 1).reshape(hkv, -1, DIM)[:, :n].repeat_interleave(hq // hkv, 0)
        x = torch.cat([(k @ q[b, :, :, None]).squeeze(2) * a["sm_scale"], a["sinks"].double()[:, None]], 1)
        lse[b] = torch.logsumexp(x, 1)
        p = torch.exp(x - torch.where(lse[b].isinf(), 0.0, lse[b])[:, None])[:, None, :n]
        out[b], mag[b] = (p @ v).squeeze(1), (p @ v.abs()).squeeze(1)
    return out, lse, mag


def check(a, out, lse):
    ro, rl, mag = reference(a)
    bound = 2.0 ** -8 * (ro.abs() + mag) + 2.0 ** -13 * mag + 1e-30
    err = (out.double() - ro).abs()
    assert bool((err <= bound).all()), f"out: worst error / bound {(err / bound).max().item()}"
    same = lse.double() == rl  # infinities
    err = torch.where(same, 0.0, (lse.double() - rl).abs())
    assert bool((err <= 2.0 ** -13 + 2.0 ** -22 * rl.abs()).all()), f"lse: worst error {err.max().item()}"


def call(a, **kw):
    import attention_softmax_sinks_gb300 as sa
    sa.sink_attn_device_status(True)
    out, lse = sa.sink_attn_decode_shared(**a, **kw)
    torch.cuda.synchronize()
    assert sa.sink_attn_device_status(True) == 0
    return out, lse


CASES = {
    "one sequence, one page": ([(1, 1)], [1], 64, 8, None),
    "one token, nothing shared": ([(1, 0)], [1], 8, 8, None),
    "own part empty": ([(3, 2)], [0, 0, 5], 8, 1, (2, 1)),
    "nothing shared anywhere": ([(5, 0)], [1, 16, 17, 100, 33], 16, 2, (3, 2)),
    "prompt ends inside a tile": ([(4, 13)], [1, 2, 30, 31], 64, 8, (2, 1)),
    "one tile of keys": ([(4, 8)], [7, 300, 1, 16], 64, 8, (1, 2)),
    "more slots than tiles": ([(2, 9)], [5, 50], 64, 8, (24, 4)),
    "two row tiles, odd group of 5": ([(37, 40)], [(i * 13) % 50 + 1 for i in range(37)], 40, 8, (3, 1)),
    "group of 7, rows end inside a tile": ([(19, 24)], [3 + i for i in range(19)], 28, 4, None),
    "group of 16": ([(17, 33)], [1 + 9 * i for i in range(17)], 64, 4, (2, 2)),
    "no grouped heads": ([(130, 17)], [1 + i % 40 for i in range(130)], 4, 4, None),
    "several row pairs": ([(70, 30)], [1 + (i * 31) % 90 for i in range(70)], 64, 8, (2, 1)),
    "groups of all kinds": ([(1, 5), (0, 3), (20, 60), (3, 0), (0, 0), (40, 1), (1, 129)],
                            [1 + (i * 17) % 70 for i in range(65)], 64, 8, None),
    "long prompt": ([(9, 700)], [1 + i for i in range(9)], 64, 8, None),
    "long own parts": ([(3, 20)], [4000, 1, 2500], 64, 8, None),
    "one slot, more units than SMs": ([(40, 9), (300, 3), (1, 33), (30, 1)], [1 + i % 19 for i in range(371)], 64, 8, (1, 1)),
    "two slots, uneven groups": ([(40, 90), (3, 300), (60, 7)], [1 + i % 35 for i in range(103)], 64, 8, (2, 1)),
    "long own parts, few SMs for the shared": ([(60, 130)], [900 + i for i in range(60)], 64, 8, None),
    "most slots": ([(2, 300)], [2000, 10], 16, 8, (200, 56)),
}


@pytest.mark.parametrize("name", CASES)
def test_shared_decode(name):
    groups, own, hq, hkv, splits = CASES[name]
    a = make(groups, own, hq, hkv, seed=len(name))
    for s in {splits, (5, 2), (0, 1)}:  # .. and every sequence by itself
        check(a, *call(a, splits=s))


def test_many_groups():
    # more groups than a CTA's threads look at in one go, some of them empty
    groups = [(i % 3, i % 4) for i in range(900)]
    n = sum(g for g, _ in groups)
    a = make(groups, [1 + i % 20 for i in range(n)], 8, 2)
    for splits in (None, (3, 1), (0, 1)):
        check(a, *call(a, splits=splits))


def test_agrees_with_plain_decode():
    import attention_softmax_sinks_gb300 as sa
    a = make([(6, 50), (3, 10)], [1 + 40 * i for i in range(9)], 64, 8)
    for x in (a["paged_k"], a["paged_v"]):
        x.copy_(torch.nan_to_num(x))
    out, lse = call(a, splits=(6, 2))
    o, l = sa.sink_attn_decode(a["q"], a["paged_k"], a["paged_v"], a["page_table"], a["kv_lens"], a["sinks"], SCALE)
    mag = reference(a)[2]
    assert bool(((out.float() - o.float()).abs() <= 2 * (2.0 ** -8 * (o.float().abs() + mag) + 2.0 ** -13 * mag)).all())
    assert bool(((lse - l).abs() <= 2.0 ** -12).all())


@pytest.mark.parametrize("splits", [(2, 1), (0, 1)])
@pytest.mark.parametrize("sink", [-INF, -1e30, 80.0, INF])
def test_sinks_at_the_extremes(sink, splits):
    a = make([(3, 9)], [1, 0, 20], 16, 2)
    a["sinks"].fill_(sink)
    a["sinks"][0] = 0.5
    out, lse = call(a, splits=splits)
    if sink == INF:  # the sink takes all the weight
        assert bool((out[:, 1:] == 0).all()) and bool((lse[:, 1:] == INF).all())
        a["sinks"][1:] = 0.5
        ro, rl, mag = reference(a)
        assert bool(((out[:, :1] - ro[:, :1]).abs() <= 2.0 ** -7 * mag[:, :1] + 2.0 ** -8 * ro[:, :1].abs()).all())
    else:
        check(a, out, lse)


@pytest.mark.parametrize("splits", [(2, 1), (0, 1)])
def test_no_keys_and_no_sink(splits):
    a = make([(2, 0)], [0, 3], 8, 1)
    a["sinks"].fill_(-INF)
    out, lse = call(a, splits=splits)
    assert bool((out[0] == 0).all()) and bool((lse[0] == -INF).all())
    check({**a, "q": a["q"][1:], "page_table": a["page_table"][1:], "kv_lens": a["kv_lens"][1:]}, out[1:], lse[1:])


def test_scores_far_apart():
    # keys of very different size: the running maximum grows in several steps, both ways
    for flip in (False, True):
        a = make([(5, 64)], [40] * 5, 64, 8)
        size = torch.linspace(0.05, 6.0, a["paged_k"].shape[0], device="cuda")
        order = a["page_table"][0, :64].long()
        size = size.flip(0) if flip else size
        k = a["paged_k"].float()
        k[order] = k[order] * size[:64].reshape(-1, 1, 1, 1)
        a["paged_k"] = k.to(torch.bfloat16)
        out, lse = call(a, splits=(6, 1))
        ro, rl, mag = reference(a)
        # scores of size up to 6 * 64 * 0.125 * ...: their fp32 error is 6 times that of unit keys
        assert bool(((out - ro).abs() <= 2.0 ** -8 * (ro.abs() + mag) + 2.0 ** -10 * mag).all())
        assert bool(((lse - rl).abs() <= 2.0 ** -10).all())


def test_outputs_workspace_and_stream():
    import attention_softmax_sinks_gb300 as sa
    a = make([(4, 10), (2, 3)], [1, 20, 3, 40, 5, 6], 64, 8)
    want = call(a, splits=(2, 2))
    ws = (torch.full((6, 4, 64, DIM), NAN, device="cuda"), torch.full((6, 4, 64), NAN, device="cuda"))
    out = torch.full((8, 64, DIM), 7.0, dtype=torch.bfloat16, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = sa.sink_attn_decode_shared(**a, splits=(2, 2), workspace=ws, out=out[:6], return_lse=False, stream=s)
    s.synchronize()
    assert got[1] is None and torch.equal(got[0], want[0]) and bool((out[6:] == 7).all())


def test_repeated_calls_and_graph_replay():
    import attention_softmax_sinks_gb300 as sa
    a = make([(30, 40), (11, 7)], [1 + (i * 7) % 60 for i in range(41)], 64, 8)
    want = call(a)
    for _ in range(5):
        got = call(a)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        sa.sink_attn_decode_shared(**a)
    s.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out, lse = sa.sink_attn_decode_shared(**a)
    other = torch.Generator(device="cuda").manual_seed(5)
    for name in ("q", "paged_k", "paged_v"):
        a[name].copy_(torch.randn(a[name].shape, generator=other, device="cuda"))
    a["kv_lens"][30:] -= 2 * (a["kv_lens"][30:] > 7 * PAGE + 2)  # shorter own parts, same pages
    for _ in range(3):
        g.replay()
    torch.cuda.synchronize()
    assert sa.sink_attn_device_status(True) == 0
    check(a, out, lse)


@pytest.mark.parametrize("splits", [(3, 1), (0, 1)])
def test_device_side_reports(splits):
    import attention_softmax_sinks_gb300 as sa
    SA_ERR_BOUNDS = 5

    def status(**change):
        a = make([(3, 4), (2, 2)], [1, 20, 3, 40, 5], 16, 2)
        for x in (a["paged_k"], a["paged_v"]):
            x.copy_(torch.nan_to_num(x))
        for name, f in change.items():
            f(a[name])
        sa.sink_attn_decode_shared(**a, splits=splits)
        torch.cuda.synchronize()
        return sa.sink_attn_device_status(True)

    assert status() == 0
    assert status(group_offsets=lambda t: t.copy_(torch.tensor([0, 3, 4], device="cuda"))) == SA_ERR_BOUNDS
    assert status(group_offsets=lambda t: t.copy_(torch.tensor([1, 3, 5], device="cuda"))) == SA_ERR_BOUNDS
    assert status(group_offsets=lambda t: t.copy_(torch.tensor([0, 9, 5], device="cuda"))) == SA_ERR_BOUNDS
    assert status(group_offsets=lambda t: t.copy_(torch.tensor([0, -3, 5], device="cuda"))) == SA_ERR_BOUNDS
    assert status(shared_pages=lambda t: t.fill_(5)) == SA_ERR_BOUNDS   # above max_shared_pages
    assert status(shared_pages=lambda t: t.fill_(-1)) == SA_ERR_BOUNDS
    assert status(kv_lens=lambda t: t[1:2].fill_(10)) == SA_ERR_BOUNDS  # shorter than its prompt
    assert status(kv_lens=lambda t: t.fill_(1 << 30)) == SA_ERR_BOUNDS
    assert status(page_table=lambda t: t[0, 1:2].fill_(10 ** 6)) == SA_ERR_BOUNDS  # a shared page
    assert status(page_table=lambda t: t[1, 5:6].fill_(-7)) == SA_ERR_BOUNDS      # an own one
    assert status() == 0


@pytest.mark.parametrize("splits", [(3, 1), (0, 1)])
def test_shorter_than_its_prompt(splits):
    import attention_softmax_sinks_gb300 as sa
    a = make([(3, 4)], [5, 6, 7], 16, 2)
    a["kv_lens"][1] = 20
    out, lse = sa.sink_attn_decode_shared(**a, splits=splits)
    torch.cuda.synchronize()
    assert sa.sink_attn_device_status(True) == 5
    for b in (0, 2):  # the others are not touched by it
        one = {**a, **{n: a[n][b : b + 1] for n in ("q", "page_table", "kv_lens")}}
        check(one, out[b : b + 1], lse[b : b + 1])


def test_by_itself_in_a_graph_and_on_a_stream():
    import attention_softmax_sinks_gb300 as sa
    a = make([(4, 10), (2, 3)], [1, 20, 3, 40, 5, 6], 64, 8)
    assert sa.sink_attn_decode_shared_splits(6, 2, 64, 8, 10, a["page_table"].shape[1]) == (0, 1)
    want = call(a)
    out = torch.full((8, 64, DIM), 7.0, dtype=torch.bfloat16, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = sa.sink_attn_decode_shared(**a, out=out[:6], return_lse=False, stream=s)
    s.synchronize()
    assert got[1] is None and torch.equal(got[0], want[0]) and bool((out[6:] == 7).all())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        o, l = sa.sink_attn_decode_shared(**a)
    a["q"].copy_(a["q"].flip(0))
    g.replay()
    torch.cuda.synchronize()
    check(a, o, l)
    with pytest.raises(ValueError):
        sa.sink_attn_decode_shared(**a, splits=(0, 2))


@pytest.mark.parametrize("groups", [[(5, 61)], [(24, 100)], [(3, 40), (30, 9)], [(2, 300), (1, 7), (2, 130)], [(1, 3)], [(9, 8), (9, 8)]])
@pytest.mark.parametrize("hq,hkv", [(64, 8), (8, 1), (6, 6)])
def test_any_number_of_slots(groups, hq, hkv):
    # units whose parts end with a run and across runs, tiles of keys in turn and not, with slots
    # that nothing goes into: whatever the workspace held before
    n = sum(c for c, _ in groups)
    a = make(groups, [1 + 13 * i % 50 for i in range(n)], hq, hkv, seed=hq)
    for slots in (1, 2, 3, 4, 5, 6, 7, 8, 11, 14, 15, 20, 39, 64):
        ws = (torch.full((n, slots + 1, hq, DIM), NAN, device="cuda"), torch.full((n, slots + 1, hq), NAN, device="cuda"))
        check(a, *call(a, splits=(slots, 1), workspace=ws))


@pytest.mark.parametrize("splits", [(3, 2), (1, 1), (6, 1), (0, 1)])
@pytest.mark.parametrize("place", ["query", "shared key", "own key", "shared value", "own value", "only key"])
@pytest.mark.parametrize("sink", [0.5, -INF])
def test_what_is_not_finite_shows(splits, place, sink):
    # as in sink_attn_decode: whatever a head attends to is in its result, in every plan
    import attention_softmax_sinks_gb300 as sa
    a = make([(4, 20), (2, 3), (1, 0)], [1, 20, 1, 40, 5, 60, 30], 16, 2)
    for x in (a["paged_k"], a["paged_v"]):
        x.copy_(torch.nan_to_num(x))
    a["sinks"].fill_(sink)
    table, hit = a["page_table"], torch.zeros(7, 16, dtype=torch.bool, device="cuda")
    if place == "query":
        a["q"][2, 11, 5] = NAN
        a["q"][6, 1, 7] = NAN
        hit[2, 11] = hit[6, 1] = True
    elif place == "shared key":
        a["paged_k"][table[0, 17].long(), 1, 3, 9] = NAN
        hit[:4, 8:] = True
    elif place == "own key":  # the second of a sequence's own pages, the only token of another's
        a["paged_k"][table[1, 21].long(), 0, 2, 0] = NAN
        a["paged_k"][table[2, 20].long(), 0, 0, 0] = NAN
        hit[1:3, :8] = True
    elif place == "shared value":
        a["paged_v"][table[4, 1].long(), 0, 15, :] = NAN
        hit[4:6, :8] = True
    elif place == "own value":
        a["paged_v"][table[6, 0].long(), 1, 0, :] = INF
        hit[6, 8:] = True
    else:  # every shared key
        a["paged_k"][table[4, :3].long()] = NAN
        hit[4:6] = True
    sa.sink_attn_device_status(True)
    out, lse = sa.sink_attn_decode_shared(**a, splits=splits)
    o, l = sa.sink_attn_decode(a["q"], a["paged_k"], a["paged_v"], table, a["kv_lens"], a["sinks"], SCALE)
    torch.cuda.synchronize()
    assert sa.sink_attn_device_status(True) == 0
    assert torch.equal(~torch.isfinite(out).all(2), hit) and torch.equal(~torch.isfinite(out).any(2), hit)
    if not (place == "query" and sink == -INF):  # (nothing but that there: no weight at all)
        assert torch.equal(torch.isfinite(out), torch.isfinite(o)) and torch.equal(torch.isfinite(lse), torch.isfinite(l))
    ro, _, mag = reference({**a, "q": torch.where(hit[:, :, None], 0.0, a["q"])})
    good = ~hit
    bound = 2.0 ** -8 * (ro.abs() + mag) + 2.0 ** -13 * mag + 1e-30
    assert bool(((out.double() - ro).abs() <= bound)[good].all())


@pytest.mark.parametrize("splits", [(3, 2), (1, 1), (0, 1)])
def test_a_value_without_weight_that_is_infinite(splits):
    # a slot whose weight vanishes beside another's is multiplied all the same
    import attention_softmax_sinks_gb300 as sa
    a = make([(2, 20)], [5, 3], 8, 1)
    for x in (a["paged_k"], a["paged_v"]):
        x.copy_(torch.nan_to_num(x))
    a["q"].fill_(1.0)
    table = a["page_table"]
    a["paged_k"][table[:, 20].long()] = 40.0   # own scores 320
    a["paged_k"][table[0, :20].long()] = 0.0   # shared ones 0
    a["paged_v"][table[0, 3].long(), 0, 2, 8:] = INF
    out, _ = sa.sink_attn_decode_shared(**a, splits=splits)
    o, _ = sa.sink_attn_decode(a["q"], a["paged_k"], a["paged_v"], table, a["kv_lens"], a["sinks"], SCALE)
    assert not bool(torch.isfinite(out[:, :, 8:]).any()) and bool(torch.isfinite(out[:, :, :8]).all())
    assert torch.equal(torch.isfinite(out), torch.isfinite(o))


@pytest.mark.parametrize("own", [1, 4])
def test_nothing_shared_and_one_slot(own):
    for groups in ([(5, 0)], [(2, 0), (0, 0), (3, 0)]):
        a = make(groups, [1, 16, 17, 100, 33], 16, 2)
        check(a, *call(a, splits=(1, own)))
        check(a, *call({**a, "max_shared_pages": 3}, splits=(1, own)))


@pytest.mark.parametrize("splits", [(3, 1), (1, 1), (0, 1)])
@pytest.mark.parametrize("times", [2, 40, 4000])
def test_offsets_that_go_back(splits, times):
    # every second group is the whole batch, within its own bounds: reported, and not worked through
    import attention_softmax_sinks_gb300 as sa
    a = make([(9, 4)], [1 + i for i in range(9)], 16, 2)
    want = call(a, splits=splits)
    offsets = torch.tensor([0, 9], device="cuda", dtype=torch.int32).repeat(times)
    bad = {**a, "group_offsets": offsets, "shared_pages": torch.full((2 * times - 1,), 4, device="cuda", dtype=torch.int32)}
    sa.sink_attn_decode_shared(**bad, splits=splits)
    torch.cuda.synchronize()
    assert sa.sink_attn_device_status(True) == 5
    got = call(a, splits=splits)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("groups", [[(4, 128)], [(30, 200), (1, 0), (9, 77)], [(5, 3)]])
def test_a_table_as_wide_as_the_context(groups):
    # captured once, replayed with other lengths
    import attention_softmax_sinks_gb300 as sa
    n = sum(c for c, _ in groups)
    a = make(groups, [40 + 11 * i % 60 for i in range(n)], 64, 8, extra_width=8000)
    check(a, *call(a))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out, lse = sa.sink_attn_decode_shared(**a)
    for less in (20, 3, 15):
        a["kv_lens"] -= less
        a["q"].copy_(a["q"].flip(1))
        g.replay()
        torch.cuda.synchronize()
        assert sa.sink_attn_device_status(True) == 0
        check(a, out, lse)
