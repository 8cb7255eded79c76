"""GPU tests of the attention path where values, masks and work sharing meet:
value scales far apart, scores beyond fp32's whole numbers, windows on the
shared line, two launches a call under streams, graphs and programmatic
launches.  The bound of a result is its own here: it counts only what a right
kernel may lose on the tokens that the query sees."""
import math

import pytest
import torch

import attn_ref as ref

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f16": torch.float16}


@pytest.fixture(scope="module")
def rn():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from residual_add_rmsnorm_vec_gb300 import build

    build.build()
    import residual_add_rmsnorm_vec_gb300 as p

    torch.cuda.set_device(0)
    p.rmsattn_read_status(clear=True)
    yield p
    assert p.rmsattn_read_status() == 0


def rand(shape, seed, dtype=torch.float32):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed)).to(dtype)


def make_cache(rn, t):
    return rn.KVCache(t["k"], t["v"], t["k_scale"], t["v_scale"])


def widened(table, tokens, page):
    """The table with bad pages behind it, up to `tokens` tokens a row."""
    wide = torch.full((table.shape[0], tokens // page), -1, dtype=torch.int32, device=table.device)
    wide[:, :table.shape[1]] = table
    return wide


def workspace(rn, q, Hk, table, page, window=0, sinks=0):
    """Bytes of workspace of a call: 0 where clusters take the rows."""
    B, n, Hq, D = q.shape
    return rn.load_attn().rmsattn_kv_attention_workspace(B, n, Hq, Hk, D, table.shape[1] * page, window, sinks)


def attend(q, t, table, lengths, scale, window=0, sinks=0, more=0.0):
    """(out, bound) in fp64, [B, n, Hq, D].

    With u = 2^-24: a score is D products of exact factors in fp32 sums (2 u a
    term where a tensor-core sum truncates) and four roundings of its own size;
    a weight has that, exp2's 2 ulp, and a rounding to fp16: half a step (2^-11
    of it), or, below fp16's normal range, at most 2^-33 of the row's largest
    weight and at most itself; its sums take a rounding for every 16 tokens and
    the joins.  more: a relative error of every term beside these."""
    B, n, Hq, D = q.shape
    Hk, page = t["k"].shape[1:3]
    G = Hq // Hk
    out = torch.zeros((B, n, Hq, D), dtype=torch.float64, device=q.device)
    bound = torch.zeros_like(out)
    for b, L in enumerate(lengths.tolist()):
        for i in range(n):
            pos = L - n + i
            j = torch.arange(max(0, pos + 1), device=q.device)
            if window:
                j = j[(j > pos - window) | (j < sinks)]
            if not j.numel():
                continue
            pg, at = table[b].long()[j // page], j % page
            for h in range(Hk):
                k = ref.e4m3(t["k"][pg, h, at]) * t["k_scale"][pg, h, at // 16].double()[:, None]
                v = ref.e4m3(t["v"][pg, h, at]) * t["v_scale"][pg, h, at // 16].double()[:, None]
                qq = q[b, i, h * G:(h + 1) * G].double()
                s = qq @ k.T * scale
                p = torch.softmax(s, -1)
                ds = float((qq.abs() @ k.abs().T).max()) * abs(scale) * (2 * D + 8) * ref.U + float(s.abs().max()) * 4 * ref.U
                rel = 2.0 ** -11 + 2 * (ds + 4 * ref.U) + (2 * j.numel() / 16 + 64) * 2 * ref.U + more
                lost = torch.minimum(p, 2.0 ** -33 * p.amax(-1, keepdim=True)) @ v.abs()
                heads = slice(h * G, (h + 1) * G)
                out[b, i, heads] = p @ v
                bound[b, i, heads] = rel * (p @ v.abs()) + lost
    half = ref.HALF[q.dtype]
    return out, bound + half * (out.abs() + bound) + ref.TINY[q.dtype]


def within(got, want, bound):
    off = (got.double() - want).abs()
    assert bool((off <= bound).all()), f"{float((off / bound).nan_to_num(9e9).max())} of the bound"


# ---------------------------------------------------------------- value scales

HOW = {"rows": 0, "line": 40000}  # tokens of a table's row; 0: as the sequence needs


def case(D, L, n, dtype="bf16", page=16, Hk=2, Hq=8, how="rows"):
    pages = -(-L // page)
    t = ref.random_cache(pages, Hk, page, D, 5, "cuda", spread=False)
    table = torch.randperm(pages, generator=torch.Generator().manual_seed(2)).to(torch.int32)[None].cuda()
    q = rand((1, n, Hq, D), 3, DT[dtype]).cuda()
    lens = torch.tensor([L], dtype=torch.int32, device="cuda")
    return t, table, widened(table, HOW[how], page) if HOW[how] else table, q, lens


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("how", HOW)
@pytest.mark.parametrize("bits", [20, 26, 32, 40])
@pytest.mark.parametrize("below", [30.0, 400.0])
def test_a_large_value_scale_of_no_weight_coarsens_nothing(rn, D, how, bits, below):
    # one block of 16 tokens: values 2^bits times the rest's, scores `below` (nats) under them
    t, table, given, q, lens = case(D, 700, 1, how=how)
    q[..., 0] = 8.0
    first = int(table[0, 3])
    t["k"][:, :, :, 0] = 0
    t["k"][first, :, :, 0] = 0xF8  # -256
    t["k_scale"][first] = below * math.sqrt(D) / (8 * 256)
    t["k"][first, :, :, 1:] = 0
    t["v_scale"][first] *= 2.0 ** bits
    assert (workspace(rn, q, 2, given, 16) > 0) == (how == "line")
    got = rn.kv_cache_attention(q, make_cache(rn, t), given, lens)
    within(got, *attend(q, t, table, lens, 1 / math.sqrt(D)))


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("bits", [26, 34])
def test_a_large_value_scale_seen_by_another_query_alone(rn, D, bits):
    # the window of the first drafted query reaches one token, with a large value scale, that the
    # window of the second does not
    n, L, window = 2, 420, 420 - 2 + 1 - 47  # reaches from token 47, the last of its block
    t, table, given, q, lens = case(D, L, n)
    t["v_scale"][int(table[0, 2])] *= 2.0 ** bits
    got = rn.kv_cache_attention(q, make_cache(rn, t), given, lens, window=window)
    want, bound = attend(q, t, table, lens, 1 / math.sqrt(D), window)
    within(got[:, 1], want[:, 1], bound[:, 1])
    within(got, want, bound)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("n", [1, 3])
@pytest.mark.parametrize("low,high", [(-20, 20), (-126, -100), (60, 90)])
def test_value_scales_of_any_size(rn, D, n, low, high):
    t, table, given, q, lens = case(D, 333, n)
    e = torch.randint(low, high + 1, t["v_scale"].shape, generator=torch.Generator().manual_seed(1))
    part = torch.rand(e.shape, generator=torch.Generator().manual_seed(4))
    t["v_scale"] = (torch.exp2(e.double()).float() * (1 + part)).cuda()
    got = rn.kv_cache_attention(q, make_cache(rn, t), given, lens)
    # scales below 2^-118 lose up to 8 of their 24 bits on their way into the sum
    within(got, *attend(q, t, table, lens, 1 / math.sqrt(D), more=2.0 ** -16 if low < -118 else 0.0))


# ---------------------------------------------------------------- scores

@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("n", [1, 3])
@pytest.mark.parametrize("how", HOW)
@pytest.mark.parametrize("top", [1e7, 3e9, -3e9, 1e15, 1e30])
def test_scores_beyond_whole_numbers_of_fp32(rn, D, n, how, top):
    # Scores that fp32 holds to hundreds and more: the largest must still weigh 1.  The 16 tokens of a
    # block have equal scores, the blocks' lie at least 0.05 of their size apart: a mean of 16 values.
    L = 160
    t, table, given, q, lens = case(D, L + n - 1, n, how=how)
    q[...] = 1.0 / 3
    t["k"][...] = 0x39  # 1.125
    t["k_scale"][...] = 1e-9  # of the drafted tokens behind the first query's position
    order = [(7 * i) % 10 for i in range(10)]  # up and down
    for i in range(10):
        t["k_scale"][int(table[0, i])] = 1.0 + 0.137 * order[i]
    scale = top / (float(q[0, 0, 0, 0]) * 1.125 * D)
    got = rn.kv_cache_attention(q, make_cache(rn, t), given, lens, scale=scale)
    page = int(table[0, order.index(9 if top > 0 else 0)])
    v = ref.e4m3(t["v"][page]) * t["v_scale"][page].double()[:, :, None]  # [Hk, 16, D]
    want = v.mean(1).repeat_interleave(4, 0)
    # weights of 1 are exact; a sum of 16 terms (2 u a term), a multiply-add, the joins and a division: 64 u
    bound = v.abs().mean(1).repeat_interleave(4, 0) * 64 * ref.U
    bound = bound + ref.HALF[q.dtype] * (want.abs() + bound)
    within(got[0, 0], want, bound)
    if top > 0:
        within(got[0], want.expand(n, -1, -1), bound.expand(n, -1, -1))
    assert bool(torch.isfinite(got).all())


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("how", HOW)
@pytest.mark.parametrize("code", [0x38, 0xB8, 0])  # 1, -1, 0: the keys where the query is infinite
@pytest.mark.parametrize("value", [math.inf, -math.inf])
def test_an_infinite_query_gives_nan(rn, D, dtype, how, code, value):
    # scores of +inf, -inf or NaN alone: a softmax of any of them is NaN, where a token is seen
    n, L = 3, 2
    t, table, given, q, lens = case(D, 40, n, dtype, how=how)
    lens[0] = L  # the first of the three queries sees nothing
    q[0, :, 5, 7] = value
    t["k"][..., 7] = code
    got = rn.kv_cache_attention(q, make_cache(rn, t), given, lens)
    assert bool(got[0, 1:, 5].isnan().all()) and bool((got[0, 0] == 0).all())
    want, bound = attend(q.nan_to_num(0, 0, 0), t, table, lens, 1 / math.sqrt(D))
    rest = [h for h in range(8) if h != 5]
    within(got[:, :, rest], want[:, :, rest], bound[:, :, rest])


# ---------------------------------------------------------------- handles

def test_a_cache_whose_tensors_were_given_other_memory(rn):
    # the next calls read and write where the tensors lie now; the old memory stays as it is
    t, table, _, q, lens = case(64, 30, 1)
    cache = make_cache(rn, t)
    rn.kv_cache_attention(q, cache, table, lens)
    old = {name: x.detach() for name, x in t.items()}  # keeps the memory
    was = {name: x.clone() for name, x in old.items()}
    for name, x in t.items():
        x.data = torch.empty_like(x).copy_(x)
    k, v = rand((1, 2, 64), 1, torch.bfloat16).cuda(), rand((1, 2, 64), 2, torch.bfloat16).cuda()
    rn.kv_cache_append_(cache, k, v, table, lens)
    for name in t:
        assert torch.equal(old[name], was[name])
    for side, x in (("k", k), ("v", v)):
        ref.check_append(was, t, x, side, table.cpu(), lens.cpu(), None)
    within(rn.kv_cache_attention(q, cache, table, lens + 1), *attend(q, t, table, lens + 1, 0.125))
    t["v"].untyped_storage().resize_(0)  # given back
    with pytest.raises(ValueError):
        rn.kv_cache_attention(q, cache, table, lens)
    with pytest.raises(ValueError):
        rn.kv_cache_append_(cache, k, v, table, lens)
    table = rn.rope_table(64)
    x, pos = rand((1, 64), 1).cuda(), torch.ones(1, dtype=torch.int32, device="cuda")
    rn.qk_norm_rope(x, None, pos, table, head_dim=64)
    table.axis.data = table.axis.long()
    with pytest.raises(TypeError):
        rn.qk_norm_rope(x, None, pos, table, head_dim=64)


# ---------------------------------------------------------------- windows

@pytest.mark.parametrize("window", [2**29 - 1, 2**29, 2**31, 2**62, 2**63 - 257, 2**63 - 256, 2**63 - 1])
@pytest.mark.parametrize("sinks", [0, 5, 2**62, 2**63 - 1])
def test_a_window_wider_than_any_row_is_planned_as_none(rn, window, sinks):
    # a row of 131072 tokens belongs on the shared line, whose workspace it needs
    q = torch.empty((1, 1, 32, 128), dtype=torch.bfloat16)
    table = torch.empty((1, 2048), dtype=torch.int32)
    none = workspace(rn, q, 8, table, 64)
    assert none > 0 and workspace(rn, q, 8, table, 64, window, sinks) == none


def test_a_window_of_the_largest_integer(rn):
    t, table, given, q, lens = case(128, 300, 2, how="line")
    want = rn.kv_cache_attention(q, make_cache(rn, t), given, lens)
    got = rn.kv_cache_attention(q, make_cache(rn, t), given, lens, window=2**63 - 1)
    assert torch.equal(got, want)
    within(got, *attend(q, t, table, lens, 1 / math.sqrt(128)))


# the shared line's steps skip from the sinks to the window; rows are cut by the shares' borders on
# both sides of that gap, and joined
ON_THE_LINE = [
    # lengths, n, Hq, Hk, D, page, dtype, window, sinks
    ([26000, 21000, 24017], 1, 8, 2, 128, 64, "bf16", 20000, 5),
    ([26000, 700, 24017, 0], 3, 8, 2, 128, 16, "f16", 20000, 40),
    ([30000, 19999, 20001], 2, 32, 4, 128, 48, "bf16", 20000, 0),
    ([22003], 5, 8, 1, 128, 64, "bf16", 18000, 1000),
    ([14000, 9000, 10016], 1, 8, 2, 256, 32, "bf16", 9000, 20),
    ([20011, 25000], 3, 8, 1, 256, 64, "f16", 18000, 17),
    ([5000, 4096, 7001, 300, 4100, 6011, 1, 5555] * 8, 1, 8, 4, 64, 64, "f16", 4096, 4),
    ([5000, 4096, 7001, 300, 4100, 6011, 0, 5555] * 8, 3, 8, 4, 64, 16, "bf16", 4096, 33),
    ([5000, 4096, 7001, 3000] * 24, 1, 4, 4, 128, 16, "bf16", 3000, 100),
]


def shared_pages(lengths, Hk, D, page, seed=3):
    """Sequences that read the same few pages in orders of their own."""
    pool, width = 90, -(-max(lengths) // page)
    t = ref.random_cache(pool, Hk, page, D, 7, "cuda", spread=False)
    g = torch.Generator().manual_seed(seed)
    return t, torch.randint(0, pool, (len(lengths), width), generator=g, dtype=torch.int32).cuda()


@pytest.mark.parametrize("lengths,n,Hq,Hk,D,page,dtype,window,sinks", ON_THE_LINE)
def test_windows_on_the_shared_line(rn, lengths, n, Hq, Hk, D, page, dtype, window, sinks):
    t, table = shared_pages(lengths, Hk, D, page)
    lens = torch.tensor(lengths, dtype=torch.int32, device="cuda")
    q = rand((len(lengths), n, Hq, D), 3, DT[dtype]).cuda()
    assert workspace(rn, q, Hk, table, page, window, sinks) > 0
    got = rn.kv_cache_attention(q, make_cache(rn, t), table, lens, window=window, sinks=sinks)
    within(got, *attend(q, t, table, lens, 1 / math.sqrt(D), window, sinks))


@pytest.mark.parametrize("D,n", [(64, 1), (64, 3), (128, 1), (128, 3), (256, 2)])
def test_masked_places_on_the_shared_line_hold_anything(rn, D, n):
    # NaN codes, and NaN or infinite scales, between the sinks and the window and behind the length
    page, Hk, Hq, L, sinks = 16, 2, 8, 40011, 21
    window = 33000 if D == 64 else 20000
    pages = -(-L // page) + 1
    t = ref.random_cache(pages, Hk, page, D, 7, "cuda", spread=False)
    table = torch.randperm(pages, generator=torch.Generator().manual_seed(1)).to(torch.int32)[None].cuda()
    lens = torch.tensor([L], dtype=torch.int32, device="cuda")
    q = rand((1, n, Hq, D), 3, torch.bfloat16).cuda()
    want, bound = attend(q, t, table, lens, 1 / math.sqrt(D), window, sinks)
    j = torch.arange(pages * page, device="cuda")
    hidden = (j >= L) | ((j < L - n + 1 - window) & (j >= sinks))
    pg, at = table[0].long()[j // page], j % page
    t["k"][pg[hidden], :, at[hidden]] = 0x7F
    t["v"][pg[hidden], :, at[hidden]] = 0xFF
    blocks = hidden.view(-1, 16).all(1).nonzero()[:, 0]
    t["k_scale"][table[0].long()[blocks]] = math.nan
    t["v_scale"][table[0].long()[blocks]] = math.inf
    assert workspace(rn, q, Hk, table, page, window, sinks) > 0
    got = rn.kv_cache_attention(q, make_cache(rn, t), table, lens, window=window, sinks=sinks)
    within(got, want, bound)


@pytest.mark.parametrize("B,tokens,window,line", [(2, 128, 0, False), (1, 131072, 0, True), (1, 131072, 60, False),
                                                  (3, 40000, 20000, True), (2, 40000, 0, True)])
def test_which_calls_take_the_line(rn, B, tokens, window, line):
    # so that the tests of either way of sharing the work stay tests of that way
    q, table = torch.empty((B, 1, 8, 128), dtype=torch.bfloat16), torch.empty((B, tokens // 16), dtype=torch.int32)
    assert (workspace(rn, q, 2, table, 16, window, 3 if window else 0) > 0) == line


# ---------------------------------------------------------------- two launches a call

def test_calls_with_workspaces_on_two_streams_at_once(rn):
    # each stream's calls have parts and cuts of their own, although the pool hands out freed memory
    t, table = shared_pages([5400, 4000], 2, 128, 16)
    table = widened(table, 40000, 16)
    cache, lens = make_cache(rn, t), torch.tensor([5400, 4000], dtype=torch.int32, device="cuda")
    qs = [rand((2, 8, 128), i, torch.bfloat16).cuda() for i in range(12)]
    assert workspace(rn, qs[0][:, None], 2, table, 16) > 0
    alone = [rn.kv_cache_attention(q, cache, table, lens) for q in qs]
    for q, a in zip(qs[:2], alone):
        within(a[:, None], *attend(q[:, None], t, table, lens, 1 / math.sqrt(128)))
    streams = [torch.cuda.Stream() for _ in range(4)]
    torch.cuda.synchronize()
    for _ in range(5):
        for s in streams:  # all start behind a pause, and then run side by side
            with torch.cuda.stream(s):
                torch.cuda._sleep(1_000_000)
        got = [rn.kv_cache_attention(q, cache, table, lens, stream=streams[i % 4]) for i, q in enumerate(qs)]
        torch.cuda.synchronize()
        for a, b in zip(got, alone):
            assert torch.equal(a, b)


def step(rn, s, row, pdl):
    """Rotary QK norm, append, attention over the cache."""
    B, n, Hq, Hk, D = s["B"], s["n"], 8, 2, 128
    q, k, v = row.split([Hq * D, Hk * D, Hk * D], 1)
    q, k = rn.qk_norm_rope(q, k, s["pos"], s["rope"], s["w"], s["w"], head_dim=D, eps=1e-6, pdl=pdl)
    rn.kv_cache_append_(s["cache"], k, v, s["table"], s["before"], s["cu"], pdl=pdl)
    o = rn.kv_cache_attention(q.view(B, n, Hq, D), s["cache"], s["table"], s["after"], window=s["window"], sinks=4,
                              pdl=pdl)
    return q, o


def state(rn, n, lengths, window):
    """Sequences whose tables hold 40000 tokens: the attention makes two launches."""
    B, page = len(lengths), 16
    used = -(-(max(lengths) + 40) // page)
    s = dict(B=B, n=n, window=window, rope=rn.rope_table(128), w=rand((128,), 1, torch.bfloat16).cuda())
    s["t"] = ref.random_cache(B * used, 2, page, 128, 7, "cuda", spread=False)
    order = torch.randperm(B * used, generator=torch.Generator().manual_seed(2)).to(torch.int32).cuda()
    s["table"], s["cache"] = widened(order.view(B, used), 40000, page), make_cache(rn, s["t"])
    s["before"] = torch.tensor(lengths, dtype=torch.int32, device="cuda")
    s["after"], s["pos"] = s["before"] + n, s["before"].repeat_interleave(n)
    s["cu"] = torch.arange(0, B * n + 1, n, dtype=torch.int32, device="cuda")
    q = torch.empty((B, n, 8, 128), dtype=torch.bfloat16)
    assert workspace(rn, q, 2, s["table"], page, window, 4) > 0
    return s


@pytest.mark.parametrize("n", [1, 4])
@pytest.mark.parametrize("window", [0, 20000])
@pytest.mark.parametrize("pdl", [False, True])
def test_steps_with_two_launches(rn, n, window, pdl):
    # one call right behind the other: what the launches hand on is there, and workspaces are not mixed up
    s = state(rn, n, [9000, 0, 2047] if not window else [30000, 100, 23000], window)
    e = state(rn, n, [9000, 0, 2047] if not window else [30000, 100, 23000], window)
    rows = [rand((s["B"] * n, 12 * 128), i, torch.bfloat16).cuda() for i in range(6)]
    torch.cuda.synchronize()
    got = []
    for row in rows:
        got.append(step(rn, s, row, pdl))
        for name in ("before", "after", "pos"):
            s[name] = s[name] + n
    for row, (q, o) in zip(rows, got):
        q2, o2 = step(rn, e, row, False)
        torch.cuda.synchronize()
        assert torch.equal(q, q2) and torch.equal(o, o2)
        for name in ("before", "after", "pos"):
            e[name] = e[name] + n
    for name in s["t"]:
        assert torch.equal(s["t"][name], e["t"][name])
    within(o2, *attend(q2.view(s["B"], n, 8, 128), e["t"], e["table"], e["after"] - n, 1 / math.sqrt(128), window,
                       4 if window else 0))


@pytest.mark.parametrize("pdl", [False, True])
def test_two_launches_captured_and_replayed_as_lengths_change(rn, pdl):
    s, e = state(rn, 1, [4000, 0, 2047], 0), state(rn, 1, [4000, 0, 2047], 0)
    row = rand((3, 12 * 128), 3, torch.bfloat16).cuda()
    warm = state(rn, 1, [4000, 0, 2047], 0)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(rn, warm, row, pdl)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        q, o = step(rn, s, row, pdl)
    for i in range(20):
        row.copy_(rand(row.shape, 10 + i, torch.bfloat16))
        graph.replay()
        q2, o2 = step(rn, e, row, False)
        assert torch.equal(q, q2) and torch.equal(o, o2), i
        for x in (s, e):
            for name in ("before", "after", "pos"):
                x[name] += 1 if i < 15 else -300  # and shorter again
            x["before"].clamp_(min=0)
            x["after"].copy_(x["before"] + 1)
            x["pos"].clamp_(min=0)
    for name in s["t"]:
        assert torch.equal(s["t"][name], e["t"][name])


def test_calls_are_ordered_behind_the_stream_they_name(rn):
    # inputs that arrive late on that stream, while the current one is idle: a launch on the current
    # stream would read what was there before
    D, s = 64, torch.cuda.Stream()
    t, table, given, q, lens = case(D, 500, 1, how="line")
    cache, late = make_cache(rn, t), {name: torch.zeros_like(x) for name, x in t.items()}
    into = make_cache(rn, late)
    rope, pos = rn.rope_table(D), torch.full((1,), 3, dtype=torch.int32, device="cuda")
    kv = rand((1, 2, D), 4, torch.bfloat16).cuda()
    x, y, z = torch.zeros_like(q), torch.zeros_like(kv), torch.zeros_like(q)
    old = lens - 1
    want_q, _ = rn.qk_norm_rope(q.view(1, -1), None, pos, rope, head_dim=D)
    want_o = rn.kv_cache_attention(q, cache, given, lens)
    after = {name: a.clone() for name, a in t.items()}
    rn.kv_cache_append_(make_cache(rn, after), kv, kv, table, old)
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        torch.cuda._sleep(200_000_000)  # some 100 ms
        for a, b in ((x, q), (y, kv), (z, q)):
            a.copy_(b)
        for name in t:
            late[name].copy_(t[name])
    got_q, _ = rn.qk_norm_rope(x.view(1, -1), None, pos, rope, head_dim=D, stream=s)
    got_o = rn.kv_cache_attention(z, into, given, lens, stream=s)
    rn.kv_cache_append_(into, y, y, table, old, stream=s)
    assert not s.query()  # the calls came before their inputs
    torch.cuda.synchronize()
    assert torch.equal(got_q, want_q) and torch.equal(got_o, want_o)
    for name in t:
        assert torch.equal(late[name], after[name])
