"""GPU tests of the operators around the attention in a serving step:
kv_pages_step_, kv_cache_prefix_attention and fused_block_norms against plain
references (tests/step_ref.py, tests/attn_ref.py), and a run of them together."""
import math
import random

import pytest
import torch

import attn_ref as ref
import step_ref
from test_gpu_attn import DT, layers_cache, make_cache, rand, within

pytestmark = pytest.mark.gpu


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


def i32(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


# ---------------------------------------------------------------- pages


def pages_state(rng, B, page, width, spare, done=0.2, absent=0.1, shared=0, new=1, most=None):
    """A pool of pages, the sequences' tables of it, their lengths and what they get."""
    n = B * width + spare
    order = rng.sample(range(n), n)
    prefix, order = order[:shared], order[shared:]
    lengths, more, table, keep = [], [], [], []
    for s in range(B):
        L = rng.randint(0, (most or width) * page)
        if L < shared * page:
            L = shared * page
        own = -(-L // page)
        take = max(0, own - shared)
        table.append(prefix[:min(shared, own)] + order[:take] + [-1] * (width - own))
        order = order[take:]
        table[-1] = (table[-1] + [-1] * width)[:width]  # (a pool that ran out leaves rows short)
        kind = rng.random()
        more.append(-1 if kind < done else rng.choice([0, new, rng.randint(0, 2 * new)]))
        lengths.append(-1 if kind > 1 - absent else L)
        keep.append(shared)
    free = order + [-1] * (n - len(order))
    return free, len(order), table, lengths, more, keep


def check_pages(rn, free, n_free, table, lengths, new, shared, page, T, **kw):
    f, t = i32(free), i32(table).reshape(len(lengths), len(table[0]) if table else 3)
    was = [i32([n_free]), i32(lengths), i32(new), None if shared is None else i32(shared)]
    args = [None if w is None else w.clone() for w in was]
    step = rn.kv_pages_step_(f, args[0], t, *args[1:], page_size=page, n_rows=T, **kw)
    torch.cuda.synchronize()
    want, wt, wf = step_ref.pages_step(free, n_free, table, lengths, new, shared, page, T)
    for name, got, w in zip(step._fields, step, want):
        assert got.tolist() == w, name
    assert t.tolist() == wt and f.tolist() == wf
    for a, w in zip(args, was):
        assert a is None or torch.equal(a, w)
    again = rn.kv_pages_step_(f, args[0], t, *args[1:], page_size=page, n_rows=T, **kw)
    for a, b in zip(step, again):
        assert torch.equal(a, b)
    assert t.tolist() == wt and f.tolist() == wf
    return step


@pytest.mark.parametrize("B,page,width,new,shared", [
    (1, 16, 3, 1, 0), (1, 48, 4, 100, 0), (2, 16, 8, 7, 2), (7, 16, 5, 1, 0), (31, 32, 6, 20, 1), (33, 16, 9, 1, 3),
    (128, 64, 4, 1, 0), (129, 16, 7, 3, 0), (300, 16, 20, 40, 4), (513, 128, 3, 1, 0), (1024, 16, 12, 9, 0),
    (2047, 16, 6, 2, 1), (2048, 16, 5, 1, 0), (2049, 16, 5, 1, 0), (5000, 16, 6, 3, 2),
])
@pytest.mark.parametrize("poor", [False, True])
def test_pages(rn, B, page, width, new, shared, poor):
    rng = random.Random(B * 7 + new)
    free, n_free, table, lengths, more, keep = pages_state(rng, B, page, width, 5, new=new, shared=shared)
    if poor:
        n_free = min(n_free, B // 3)
        free = free[:n_free] + [-1] * (len(free) - n_free)
    T = sum(m for m, L in zip(more, lengths) if m > 0 and L >= 0) + rng.randint(0, 9)
    check_pages(rn, free, n_free, table, lengths, more, keep if shared or B % 2 else None, page, T)


def test_pages_of_no_sequences(rn):
    step = check_pages(rn, [2, 0, 1], 3, [], [], [], None, 16, 7)
    assert step.slots.tolist() == [-1] * 7
    check_pages(rn, [], 0, [[], []], [0, 0], [0, 1], None, 16, 1)


def test_pages_that_a_finished_sequence_returns_are_taken_in_the_same_step(rn):
    # two free pages, three come back, four are taken: both lists are met
    step = check_pages(rn, [6, 5] + [-1] * 6, 2, [[0, 1, 2, -1], [3, -1, -1, -1], [-1] * 4], [40, 16, 0], [-1, 33, 16],
                       None, 16, 60)
    assert step.n_free.tolist() == [1]


@pytest.mark.parametrize("lengths,new,T", [
    ([16, 16, 16], [1, 40, 1], 42),      # the second outruns its row: the third goes on
    ([2 ** 31 - 1, 5, 0], [1, 1, 1], 3),  # 31 bits
    ([10, 20, 30], [5, 5, 5], 12),       # rows for two
    ([10, 20, 30], [2 ** 31 - 1] * 3, 12),
    ([-5, 20, -1], [3, -1, -1], 4),
])
def test_pages_left_out(rn, lengths, new, T):
    check_pages(rn, [9, 8, 7, 6] + [-1] * 6, 4, [[0, 1], [2, 3], [4, 5]], lengths, new, None, 16, T)


def test_pages_kept_by_a_finished_sequence(rn):
    for shared in ([0, 2], [5, 9], [-3, 1]):
        check_pages(rn, [7] + [-1] * 7, 1, [[0, 1, 2], [0, 1, 3]], [48, 40], [-1, -1], shared, 16, 0)


def test_pages_bad_entries_are_reported(rn):
    check_pages(rn, [9, 0, 77, -1], 3, [[1, -1]], [10], [10], None, 16, 10)  # the page that is taken
    assert rn.rmsattn_read_status(clear=True) == rn.RMSATTN_BAD_PAGE
    check_pages(rn, [0, 1, 2], 3, [[5, -1]], [10], [3], None, 16, 3)  # the page that it holds
    assert rn.rmsattn_read_status(clear=True) == rn.RMSATTN_BAD_PAGE
    check_pages(rn, [0, 1, 2], 9, [[1, 2]], [32], [-1], None, 16, 0)  # more free pages than there are
    assert rn.rmsattn_read_status(clear=True) == rn.RMSATTN_BAD_PAGE


def test_pages_in_a_strided_table(rn):
    wide = torch.full((3, 11), -7, dtype=torch.int32, device="cuda")
    table = wide[:, 2:6]
    free, n_free = rn.kv_free_pages(12)
    rn.kv_pages_step_(free, n_free, table, i32([0, 0, 0]), i32([20, 64, 1]), page_size=16, n_rows=85)
    assert table.tolist() == [[0, 1, -7, -7], [2, 3, 4, 5], [6, -7, -7, -7]]
    assert (wide[:, :2] == -7).all() and (wide[:, 6:] == -7).all()


def test_pages_through_a_graph_and_streams(rn):
    """A server's steps: captured once, replayed with other lengths."""
    B, page, width, T = 5, 16, 6, 40
    free, n_free = rn.kv_free_pages(B * width)
    table = torch.full((B, width), -1, dtype=torch.int32, device="cuda")
    lengths, new = i32([0] * B), i32([0] * B)
    s = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    state = [free.tolist(), B * width, table.tolist(), [0] * B]
    with torch.cuda.graph(graph, stream=s):
        step = rn.kv_pages_step_(free, n_free, table, lengths, new, page_size=page, n_rows=T)
        lengths.copy_(step.after)
        n_free.copy_(step.n_free)
    rng = random.Random(3)
    for _ in range(30):
        more = [rng.choice([-1, 0, 1, 1, 1, 9, 17]) for _ in range(B)]
        new.copy_(i32(more))
        graph.replay()
        torch.cuda.synchronize()
        want, state[2], state[0] = step_ref.pages_step(state[0], state[1], state[2], state[3], more, None, page, T)
        for got, w in zip(step, want):
            assert got.tolist() == w
        assert table.tolist() == state[2] and free.tolist() == state[0]
        state[1], state[3] = want[6][0], want[5]
    # a stream of the call's own
    other = torch.cuda.Stream()
    torch.cuda.synchronize()
    new.copy_(i32([1] * B))
    other.wait_stream(torch.cuda.current_stream())
    got = rn.kv_pages_step_(free, n_free, table, lengths, new, page_size=page, n_rows=T, stream=other)
    other.synchronize()
    want, _, _ = step_ref.pages_step(state[0], state[1], state[2], state[3], [1] * B, None, page, T)
    assert [g.tolist() for g in got] == want


def test_pages_chained_by_programmatic_launches(rn):
    free, n_free = rn.kv_free_pages(64)
    table = torch.full((4, 16), -1, dtype=torch.int32, device="cuda")
    lengths = i32([0, 3, 0, 16])
    new = i32([1, 5, 2, 1])
    state = [free.tolist(), 64, table.tolist(), lengths.tolist()]
    step = None
    for _ in range(12):
        step = rn.kv_pages_step_(free, n_free, table, lengths, new, page_size=16, n_rows=9, pdl=True)
        lengths, n_free = step.after, step.n_free
        want, state[2], state[0] = step_ref.pages_step(state[0], state[1], state[2], state[3], new.tolist(), None, 16, 9)
        state[1], state[3] = want[6][0], want[5]
    assert [g.tolist() for g in step] == want and table.tolist() == state[2]


# ---------------------------------------------------------------- norms

NORMS = [
    # T, H, dtype, stream, gate, fp8, offset
    (1, 1, "bf16", "same", "none", False, 0.0), (3, 8, "bf16", "same", "layer", False, 0.0),
    (2, 64, "f32", "same", "token", False, 1.0), (5, 100, "f16", "same", "sequence", True, 0.0),
    (4, 4096, "bf16", "same", "none", False, 0.0), (3, 4104, "bf16", "f32", "layer", False, 1.0),
    (2, 8192, "f16", "f32", "token", True, 0.0), (3, 8200, "bf16", "same", "sequence", True, 1.0),
    (2, 16384, "bf16", "same", "layer", False, 0.0), (2, 16384, "f32", "same", "token", True, 0.0),
    (2, 16392, "bf16", "same", "none", True, 0.0), (1, 20001, "f16", "f32", "sequence", False, 0.5),
    (7, 2045, "f16", "f32", "token", False, 1.0), (3, 8191, "bf16", "same", "layer", True, 0.0),
    (2, 8193, "bf16", "same", "token", False, 0.0), (300, 257, "f32", "same", "none", False, 0.0),
    (1000, 512, "bf16", "f32", "sequence", True, 0.0), (6, 40, "f16", "same", "none", True, 0.0),
    (2, 33000, "f32", "same", "layer", True, 0.0), (3, 5120, "bf16", "same", "sequence", True, 0.0),
]


def norms_inputs(T, H, dtype, stream, gate, offset, seed=1):
    dt = DT[dtype]
    x = rand((T, H), seed, dt, 3.0).cuda()
    r = rand((T, H), seed + 1, torch.float32 if stream == "f32" else dt, 2.0).cuda()
    pw, w = ((1 - offset + 0.1 * rand((H,), seed + k)).to(dt).cuda() for k in (2, 3))
    g = index = None
    if gate == "layer":
        g = rand((H,), seed + 4, dt).cuda()
    elif gate == "token":
        g = rand((T, H), seed + 4, dt).cuda()
    elif gate == "sequence":
        g = rand((3, H), seed + 4, dt).cuda()
        index = torch.randint(0, 3, (T,), generator=torch.Generator().manual_seed(seed)).to(torch.int32).cuda()
    return x, r, pw, w, g, index


def check_norms(done, x, r, pw, w, g, index, fp8, alpha, offset, eps=1e-6):
    y, h, scale = done
    cpu = [None if t is None else t.cpu() for t in (x, r, pw, w, g, index)]
    want, bound, of = step_ref.norms(*cpu, eps, alpha, offset)
    within(h, want, bound, "residual")
    wy, by, err = of(h.cpu())
    if fp8:
        step_ref.check_codes(y.cpu(), scale.cpu(), wy, err)
    else:
        assert scale is None
        within(y, wy, by, "out")


@pytest.mark.parametrize("T,H,dtype,stream,gate,fp8,offset", NORMS)
def test_norms(rn, T, H, dtype, stream, gate, fp8, offset):
    x, r, pw, w, g, index = norms_inputs(T, H, dtype, stream, gate, offset)
    done = rn.fused_block_norms(x, r, pw, w, eps=1e-6, gate=g, gate_index=index, residual_scale=0.75,
                                weight_offset=offset, out_dtype="fp8" if fp8 else None)
    check_norms(done, x, r, pw, w, g, index, fp8, 0.75, offset)


@pytest.mark.parametrize("H", [63, 64, 4096])
def test_norms_without_weights_in_place_and_zero_rows(rn, H):
    x, r, _, _, _, _ = norms_inputs(5, H, "bf16", "same", "none", 0.0)
    x[1] = 0
    r[2] = 0
    x[3] = 0
    r[3] = 0
    keep = x.clone(), r.clone()
    y, h, _ = rn.fused_block_norms(x, r, eps=1e-6, residual_scale=-1.0, out=x, residual_out=r)
    assert y is x and h is r
    check_norms((y, h, None), *keep, None, None, None, None, False, -1.0, 0.0)
    assert float(y[3].abs().max()) == 0
    q, h, s = rn.fused_block_norms(*keep, eps=1e-6, residual_scale=-1.0, out_dtype="fp8")
    assert int(q[3].max()) == 0 and float(s[3]) == 0
    check_norms((q, h, s), *keep, None, None, None, None, True, -1.0, 0.0)


@pytest.mark.parametrize("off", [1, 3, 4, 8])
@pytest.mark.parametrize("H", [96, 4096])
def test_norms_of_rows_at_any_alignment(rn, off, H):
    T = 4
    x, r, pw, w, g, _ = norms_inputs(T, H, "bf16", "same", "token", 0.0)

    def moved(t):
        room = torch.zeros(t.numel() + off, dtype=t.dtype, device="cuda")
        room[off:] = t.flatten()
        return room[off:].reshape(t.shape)

    out, ro = moved(torch.zeros_like(x)), moved(torch.zeros_like(x))
    args = [moved(t) for t in (x, r, pw, w, g)]
    rn.fused_block_norms(*args[:4], eps=1e-6, gate=args[4], out=out, residual_out=ro)
    check_norms((out, ro, None), x, r, pw, w, g, None, False, 1.0, 0.0)


def test_norms_strided_gates_and_rows_left_out(rn):
    T, H = 9, 256
    x, r, pw, w, _, _ = norms_inputs(T, H, "bf16", "same", "none", 0.0)
    wide = rand((4, 3 * H), 9, torch.bfloat16).cuda()
    gate = wide[:, H:2 * H]
    index = i32([0, 3, -1, 1, 2, -1, 0, -7, 3])
    out, ro = torch.full_like(x, 7.0), torch.full_like(r, 5.0)
    rn.fused_block_norms(x, r, pw, w, eps=1e-6, gate=gate, gate_index=index, out=out, residual_out=ro)
    on = (index >= 0).cpu()
    assert (out[~on] == 7).all() and (ro[~on] == 5).all()
    check_norms((out[on], ro[on], None), x[on], r[on], pw, w, gate, index[on], False, 1.0, 0.0)
    index[1] = 4  # no such row: left out, and told
    out.fill_(7.0)
    rn.fused_block_norms(x, r, pw, w, eps=1e-6, gate=gate, gate_index=index, out=out, residual_out=ro)
    torch.cuda.synchronize()
    assert rn.rmsattn_read_status(clear=True) == rn.RMSATTN_BAD_PAGE
    assert (out[1] == 7).all() and not (out[0] == 7).all()


def test_norms_refuse_wrong_tensors(rn):
    x, r, pw, w, g, index = norms_inputs(4, 64, "bf16", "same", "sequence", 0.0)
    bad = [dict(residual=r.half()), dict(post_weight=pw.float()), dict(weight=w[:32]), dict(gate=g), dict(gate=g.float()),
           dict(gate=g, gate_index=index.long()), dict(gate=g, gate_index=index[:2]), dict(gate_index=index),
           dict(gate=g[:, :32]), dict(out=x.float()), dict(out_scale=torch.zeros(4, device="cuda")),
           dict(gate=g[:1].expand(4, 64)), dict(x=x.t()), dict(residual=r.cpu()), dict(eps=-1.0), dict(eps=math.nan),
           dict(residual_scale=math.inf), dict(out=torch.zeros_like(x).t().contiguous().t())]
    for change in bad:
        a = dict(x=x, residual=r, post_weight=pw, weight=w, eps=1e-6)
        a.update(change)
        with pytest.raises((ValueError, TypeError, rn.RmsnError)):
            rn.fused_block_norms(**a)


def test_norms_chained_streams_and_graph(rn):
    T, H = 40, 2048
    x, r, pw, w, g, _ = norms_inputs(T, H, "bf16", "same", "token", 0.0)

    def chain(pdl):
        a, b = x, r
        for _ in range(6):
            a, b, _ = rn.fused_block_norms(a, b, pw, w, eps=1e-6, gate=g, residual_scale=0.5, pdl=pdl)
        return a, b

    want = chain(False)
    for got in (chain(True), chain(False)):
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = chain(True)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    y, h, _ = rn.fused_block_norms(x, r, pw, w, eps=1e-6, gate=g, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    check_norms((y, h, None), x, r, pw, w, g, None, False, 1.0, 0.0)


# ---------------------------------------------------------------- shared prefix


def prefix_state(groups, own, Hk, page, D, seed=7, spread=False, n=1):
    """Cache, table, lengths: groups of (sequences, shared tokens); own: tokens of
    each sequence behind the shared pages."""
    B = sum(g[0] for g in groups)
    rng = random.Random(seed)
    width = max(-(-g[1] // page) for g in groups) + -(-max(own) // page) + 1
    pages = B * width + 3
    t = ref.random_cache(pages, Hk, page, D, seed, "cuda", spread=spread)
    order = rng.sample(range(pages), pages)
    table, lengths = [], []
    for count, shared in groups:
        first = [order.pop() for _ in range(shared // page)]
        for _ in range(count):
            s = len(lengths)
            mine = -(-(shared + own[s]) // page) - len(first)
            row = first + [order.pop() for _ in range(mine)]
            table.append(row + [rng.randrange(pages)] * (width - len(row)))
            lengths.append(shared + own[s])
    cu = [0]
    for count, _ in groups:
        cu.append(cu[-1] + count)
    return t, i32(table), i32(lengths), i32([g[1] for g in groups]), i32(cu)


def owns(groups, n, seed=3, most=70):
    rng = random.Random(seed)
    return [rng.randint(n, most) for _ in range(sum(g[0] for g in groups))]


PREFIX = [
    # groups of (sequences, shared tokens), n, Hq, Hk, D, page, dtype
    ([(2, 16)], 1, 4, 1, 64, 16, "bf16"), ([(3, 128)], 1, 8, 2, 128, 32, "bf16"), ([(5, 160)], 1, 4, 4, 128, 16, "f16"),
    ([(4, 64)], 1, 16, 2, 256, 64, "bf16"), ([(2, 272)], 1, 3, 1, 256, 16, "f16"), ([(33, 256)], 1, 8, 2, 128, 64, "bf16"),
    ([(40, 400)], 1, 28, 4, 64, 16, "f16"), ([(70, 1040)], 1, 16, 2, 128, 16, "bf16"), ([(17, 512)], 2, 16, 1, 128, 64, "f16"),
    ([(9, 96)], 5, 14, 2, 64, 48, "bf16"), ([(3, 2048)], 32, 4, 2, 128, 16, "bf16"), ([(6, 700 // 16 * 16)], 3, 10, 1, 256, 16, "f16"),
    ([(2, 0), (3, 48), (1, 64), (4, 16)], 1, 8, 2, 128, 16, "bf16"), ([(1, 128)], 1, 4, 2, 64, 16, "bf16"),
    ([(5, 320), (7, 640), (3, 16), (6, 1600)], 2, 8, 4, 64, 16, "f16"), ([(2, 32)] * 30, 1, 4, 2, 128, 16, "bf16"),
    ([(20, 512), (30, 1536)], 1, 32, 8, 128, 64, "bf16"), ([(13, 4096), (2, 192)], 1, 8, 1, 256, 32, "bf16"),
    ([(65, 8192)], 1, 16, 4, 128, 128, "bf16"), ([(300, 64)], 1, 8, 2, 64, 32, "bf16"), ([(4, 20000 // 16 * 16)], 1, 4, 1, 64, 16, "f16"),
]


def run_prefix(rn, q, t, table, lengths, P, cu, n, **kw):
    return rn.kv_cache_prefix_attention(q if n > 1 else q[:, 0], make_cache(rn, t), table, lengths, P, cu,
                                        **kw).reshape(q.shape)


@pytest.mark.parametrize("groups,n,Hq,Hk,D,page,dtype", PREFIX)
def test_prefix(rn, groups, n, Hq, Hk, D, page, dtype):
    t, table, lengths, P, cu = prefix_state(groups, owns(groups, n), Hk, page, D, n=n)
    q = rand((lengths.shape[0], n, Hq, D), 3, DT[dtype]).cuda()
    want, bound = ref.attend(q, t, table, lengths, 1 / math.sqrt(D), 0, 0)
    within(run_prefix(rn, q, t, table, lengths, P, cu, n), want, bound)
    if len(groups) == 1:
        within(run_prefix(rn, q, t, table, lengths, P, None, n), want, bound)


@pytest.mark.parametrize("D", [64, 128, 256])
def test_prefix_of_any_length_within_the_shared_pages(rn, D):
    # lengths off the blocks, beyond what all share (nobody sees all of it), negative and huge ones
    groups, Hk, page = [(6, 512)], 2, 64
    t, table, lengths, _, _ = prefix_state(groups, owns(groups, 1), Hk, page, D)
    q = rand((6, 1, 8, D), 3, torch.bfloat16).cuda()
    want, bound = ref.attend(q, t, table, lengths, 1 / math.sqrt(D), 0, 0)
    for p in (0, 1, 15, 16, 17, 100, 127, 128, 129, 333, 511, 512, -1, -2 ** 31, 2 ** 31 - 1):
        within(run_prefix(rn, q, t, table, lengths, i32([p]), None, 1), want, bound, str(p))


@pytest.mark.parametrize("n", [1, 3])
def test_prefix_sequences_that_do_not_share(rn, n):
    # empty and absent rows, short ones that end within the prefix, one with a single own token
    groups, Hk, page, D = [(12, 320)], 2, 16, 128
    t, table, lengths, P, cu = prefix_state(groups, owns(groups, n), Hk, page, D)
    q = rand((12, n, 8, D), 3, torch.float16).cuda()
    for s, L in ((0, 0), (1, 100), (3, -4), (4, 320 + n - 1), (5, 320 + n - 2), (6, 320), (7, 1), (11, 0)):
        lengths[s] = L
    want, bound = ref.attend(q, t, table, lengths, 1 / math.sqrt(D), 0, 0)
    got = run_prefix(rn, q, t, table, lengths, P, cu, n)
    within(got, want, bound)
    assert float(got[0].abs().max()) == 0 and float(got[3].abs().max()) == 0
    # a group's first sequence is finished and its row names other pages
    table[0] = table[0].roll(5)
    within(run_prefix(rn, q, t, table, lengths, P, cu, n), want, bound)


def test_prefix_groups_out_of_order_share_nothing(rn):
    groups, Hk, page, D = [(6, 128)], 2, 16, 64
    t, table, lengths, _, _ = prefix_state(groups, owns(groups, 1), Hk, page, D)
    q = rand((6, 1, 4, D), 3, torch.bfloat16).cuda()
    want, bound = ref.attend(q, t, table, lengths, 1 / math.sqrt(D), 0, 0)
    for cu in ([0, 4, 2, 6], [-1, 3, 6, 6], [0, 3, 6, 7], [6, 3, 0, 0]):
        within(run_prefix(rn, q, t, table, lengths, i32([128, 128, 128]), i32(cu), 1), want, bound, str(cu))
        assert rn.rmsattn_read_status(clear=True) == rn.RMSATTN_BAD_PAGE
    # groups that leave sequences out, and none at all
    for P, cu in (([64, 128], [1, 3, 5]), ([64], [6, 6]), ([], [0])):
        within(run_prefix(rn, q, t, table, lengths, i32(P), i32(cu), 1), want, bound, str(cu))


@pytest.mark.parametrize("D,dtype,qscale", [(64, "bf16", 1.0), (128, "f16", 30.0), (256, "bf16", 1e-3),
                                            (128, "bf16", 1e6), (128, "bf16", 1e-20), (64, "f16", 0.01)])
def test_prefix_scales_over_many_binades(rn, D, dtype, qscale):
    groups, Hk, page = [(9, 768), (3, 256)], 2, 32
    t, table, lengths, P, cu = prefix_state(groups, owns(groups, 1), Hk, page, D, spread=True)
    q = (rand((12, 1, 8, D), 3) * qscale).to(DT[dtype]).cuda()
    scale = 0.3 / math.sqrt(D) / qscale
    want, bound = ref.attend(q, t, table, lengths, float(torch.tensor(scale, dtype=torch.float32)), 0, 0)
    within(run_prefix(rn, q, t, table, lengths, P, cu, 1, scale=scale), want, bound)


@pytest.mark.parametrize("D", [64, 128, 256])
def test_prefix_value_scales_of_any_ratio(rn, D):
    # block after block 2^40 apart, up and down, zeros among them; the tokens of the small ones alone weigh
    groups, Hk, page, n = [(4, 512)], 1, 16, 1
    t, table, lengths, P, cu = prefix_state(groups, owns(groups, 1, most=16), Hk, page, D)
    q = rand((4, n, 4, D), 3, torch.float16).cuda()
    rows = table[0, :512 // page].long()
    for i, r in enumerate(rows.tolist()):
        t["v_scale"][r] = (1.0, 2.0 ** -40, 0.0, 3e30, 2.0 ** -100, 2.0 ** -20, 1.7e-3, 2.0 ** -126)[i * 5 % 8]
        if i % 8 not in (1, 4):
            t["k"][r] = 0
            t["v"][r] = 0  # their values are 0 whatever the scale
    for s in range(4):
        for r in table[s, 512 // page:].tolist():
            t["v_scale"][r] = 2.0 ** -30
    want, bound = ref.attend(q, t, table, lengths, 0.1, 0, 0)
    # (the bound's part for weights below fp16's range goes with the largest scale; none is that small here)
    p = 2.0 ** -8 * want.abs().amax(-1, keepdim=True) + 1e-30
    assert float(want.abs().max()) > 0
    got = run_prefix(rn, q, t, table, lengths, P, cu, n, scale=0.1).double()
    within(got, want, torch.minimum(bound, p + ref.TINY[torch.float16]))


def test_prefix_one_strong_token_among_many(rn):
    # a first token 20 above the rest: the others' small weights still add up
    P, D = 20000, 64
    t = ref.random_cache(P // 16 + 2, 1, 16, D, 7, "cuda", spread=False)
    table = torch.arange(P // 16, dtype=torch.int32, device="cuda").repeat(2, 1)
    table = torch.cat([table, i32([[P // 16], [P // 16 + 1]])], 1)
    t["k"].zero_()
    t["k"][0, 0, 0] = 0x38
    t["k_scale"].fill_(1.0)
    t["v"].fill_(0x38)
    t["v"][0, 0, 0] = 0
    t["v_scale"].fill_(1.0)
    q = torch.full((2, 1, 1, D), 16.0 / D, dtype=torch.float16, device="cuda")
    lens = i32([P + 1, P + 5])
    got = run_prefix(rn, q, t, table, lens, i32([P]), None, 1, scale=1.0)
    within(got, *ref.attend(q, t, table, lens, 1.0, 0, 0))
    assert float(got[0, 0, 0, 0]) > 1e-3


@pytest.mark.parametrize("D", [64, 128, 256])
def test_prefix_what_is_behind_it_has_no_influence(rn, D):
    # the prefix ends within a page and a tile; what lies behind in the first sequence's row, and behind the
    # sequences' ends, is NaN for the others
    Hk, page, P = 2, 64, 144
    t = ref.random_cache(20, Hk, page, D, 7, "cuda", spread=False)
    table = i32([[0, 1, 2, 3, 4], [0, 1, 5, 6, 7], [0, 1, 8, 9, 10]])
    lengths = i32([300, 193, 250])
    q = rand((3, 1, 8, D), 3, torch.bfloat16).cuda()
    table[1:, 2] = i32([5, 8])
    t["k"][5], t["v"][5], t["k"][8], t["v"][8] = t["k"][2], t["v"][2], t["k"][2], t["v"][2]
    for x in ("k_scale", "v_scale"):
        t[x][5] = t[x][8] = t[x][2]
    want, bound = ref.attend(q, t, table, lengths, 1 / math.sqrt(D), 0, 0)
    for s, L in enumerate(lengths.tolist()):
        for j in range(L, 5 * page):
            pg = int(table[s, j // page])
            t["k"][pg, :, j % page] = 0x7F
            t["v"][pg, :, j % page] = 0xFF
        for blk in range(-(-L // 16), 5 * page // 16):
            t["k_scale"][int(table[s, blk * 16 // page]), :, blk % (page // 16)] = math.nan
            t["v_scale"][int(table[s, blk * 16 // page]), :, blk % (page // 16)] = math.inf
    for shared in (P, 128, 130, 16):
        within(run_prefix(rn, q, t, table, lengths, i32([shared]), None, 1), want, bound, str(shared))


@pytest.mark.parametrize("D", [64, 128, 256])
def test_prefix_nan_and_infinite_values_reach_who_sees_them(rn, D):
    groups, Hk, page = [(5, 256), (3, 64)], 2, 16
    t, table, lengths, P, cu = prefix_state(groups, owns(groups, 1), Hk, page, D)
    q = rand((8, 1, 8, D), 3, torch.bfloat16).cuda()
    want, bound = ref.attend(q, t, table, lengths, 1 / math.sqrt(D), 0, 0)
    # an infinite and a NaN query: their rows alone
    q2 = q.clone()
    q2[1, 0, 2, 3], q2[6, 0, 5, 0], q2[2, 0, 7, 1] = math.inf, math.nan, -math.inf
    got = run_prefix(rn, q2, t, table, lengths, P, cu, 1)
    bad = torch.zeros_like(got, dtype=torch.bool)
    bad[1, 0, 2], bad[6, 0, 5], bad[2, 0, 7] = True, True, True
    assert torch.equal(got.isnan(), bad)
    within(got[~bad], want[~bad], bound[~bad])
    # a NaN value of the first group's prefix: that dim of all of its sequences' heads
    t["v"][int(table[0, 3]), 1, 5, 7] = 0x7F
    got = run_prefix(rn, q, t, table, lengths, P, cu, 1)
    bad = torch.zeros_like(got, dtype=torch.bool)
    bad[:5, 0, 4:, 7] = True
    assert torch.equal(got.isnan(), bad)
    within(got[~bad], want[~bad], bound[~bad])
    # a NaN key: all dims
    t["k"][int(table[0, 9]), 0, 2, 1] = 0xFF
    got = run_prefix(rn, q, t, table, lengths, P, cu, 1)
    bad[:5, 0, :4] = True
    assert torch.equal(got.isnan(), bad)


def test_prefix_bad_pages_are_left_out(rn):
    D, page = 128, 16
    t = ref.random_cache(12, 2, page, D, 7, "cuda", spread=False)
    first = [3, -1, 99, 2, 12]
    table = i32([first + [0, 1, -1], first + [4, 5, 6], first + [7, 8, 9]])
    lengths = i32([100, 128, 90])
    q = rand((3, 1, 4, D), 3, torch.bfloat16).cuda()
    got = run_prefix(rn, q, t, table, lengths, i32([80]), None, 1)
    assert rn.rmsattn_read_status(clear=True) == rn.RMSATTN_BAD_PAGE
    within(got, *ref.attend(q, t, table, lengths, 1 / math.sqrt(D), 0, 0))
    # a cache of no pages, a table of no columns
    empty = {x: t[x][:0] for x in t}
    got = run_prefix(rn, q, empty, table, lengths, i32([80]), None, 1)
    assert rn.rmsattn_read_status(clear=True) == rn.RMSATTN_BAD_PAGE and float(got.abs().max()) == 0
    got = run_prefix(rn, q, t, table[:, :0], i32([0, 0, 0]), i32([80]), None, 1)
    assert float(got.abs().max()) == 0


def test_prefix_strides_scales_and_signs(rn):
    groups, Hk, page, D, n = [(7, 192)], 2, 16, 64, 2
    _, _, t = layers_cache(rn, 80, Hk, page, D)
    _, table, lengths, P, cu = prefix_state(groups, owns(groups, n, most=40), Hk, page, D)
    table %= 80
    own = torch.arange(12, 80, dtype=torch.int32, device="cuda")[:7 * (table.shape[1] - 12)].reshape(7, -1)
    table = torch.cat([torch.arange(12, dtype=torch.int32, device="cuda").repeat(7, 1), own], 1)
    wide = rand((7, n, 3, 8 * D), 3, torch.bfloat16).cuda()
    q = wide[:, :, 1].unflatten(2, (8, D))
    room = torch.full((7, n, 2, 8 * D), 3.0, dtype=torch.bfloat16, device="cuda")
    out = room[:, :, 1].unflatten(2, (8, D))
    for scale in (-0.2, 0.0, 0.125):
        got = rn.kv_cache_prefix_attention(q, make_cache(rn, t), table, lengths, P, cu, scale=scale, out=out)
        assert got is out
        within(out, *ref.attend(q, t, table, lengths, float(torch.tensor(scale)), 0, 0))
    assert (room[:, :, 0] == 3).all()


def test_prefix_repeats_streams_and_graphs(rn):
    groups, Hk, page, D = [(20, 1024), (9, 320)], 2, 16, 128
    t, table, lengths, P, cu = prefix_state(groups, owns(groups, 1), Hk, page, D)
    cache = make_cache(rn, t)
    qs = [rand((29, 8, D), i, torch.bfloat16).cuda() for i in range(6)]

    def call(q, **kw):
        return rn.kv_cache_prefix_attention(q, cache, table, lengths, P, cu, **kw)

    want = [call(q) for q in qs]
    within(want[0][:, None], *ref.attend(qs[0][:, None], t, table, lengths, 1 / math.sqrt(D), 0, 0))
    for q, w in zip(qs, want):
        assert torch.equal(call(q), w)
        assert torch.equal(call(q, pdl=True), w)
    streams = [torch.cuda.Stream() for _ in range(3)]
    torch.cuda.synchronize()
    for _ in range(4):
        got = [call(q, stream=streams[i % 3]) for i, q in enumerate(qs)]
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    # two graphs of the same call, replayed in turn, with other queries and lengths than when captured
    live, outs, graphs = qs[0].clone(), [], []
    for _ in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append(call(live, pdl=True))
        graphs.append(graph)
    keep = lengths.clone()
    for i, q in enumerate(qs):
        live.copy_(q)
        lengths.copy_(keep - i % 2)
        for graph, out in zip(graphs, outs):
            graph.replay()
            if i % 2 == 0:
                assert torch.equal(out, want[i])
            else:
                assert torch.equal(out, call(q))
    lengths.copy_(keep)


def test_prefix_refuses_wrong_tensors(rn):
    groups, Hk, page, D = [(3, 64)], 2, 16, 64
    t, table, lengths, P, cu = prefix_state(groups, owns(groups, 1), Hk, page, D)
    q = rand((3, 4, D), 3, torch.bfloat16).cuda()
    for change in (dict(q=q.float()), dict(q=q[:, :3]), dict(q=q.cpu()), dict(prefix_lengths=P.long()),
                   dict(prefix_lengths=P.repeat(2)), dict(groups=cu.long()), dict(groups=cu[:1]), dict(groups=cu.cpu()),
                   dict(lengths=lengths[:2]), dict(block_table=table.long()), dict(out=q.half()), dict(scale=math.nan),
                   dict(prefix_lengths=P.cpu())):
        a = dict(q=q, cache=make_cache(rn, t), block_table=table, lengths=lengths, prefix_lengths=P, groups=cu)
        a.update(change)
        with pytest.raises((ValueError, TypeError, rn.RmsnError)):
            rn.kv_cache_prefix_attention(**a)


# ---------------------------------------------------------------- together


def test_a_serving_step(rn):
    """Two prompts that share their first pages, then decode steps: plan, rotary
    positions, append, attention with the shared prefix, norms with a gate row for
    each sequence; one sequence ends and another takes its place."""
    B, Hq, Hk, D, page, width, H = 4, 8, 2, 64, 16, 12, 8 * 64
    cache = rn.KVCache.empty(B * width, Hk, page, D)
    for x in (cache.k, cache.v, cache.k_scale, cache.v_scale):
        x.zero_()
    rope = rn.rope_table(D)
    free, n_free = rn.kv_free_pages(B * width)
    table = torch.full((B, width), -1, dtype=torch.int32, device="cuda")
    gate, w = rand((B, H), 1, torch.bfloat16).cuda(), (1 + 0.1 * rand((H,), 2)).bfloat16().cuda()
    lengths = i32([0] * B)
    shared = i32([0] * B)
    # the system prompt: two pages, by the first sequence, then named by all
    T = 32
    step = rn.kv_pages_step_(free, n_free, table, lengths, i32([T, 0, 0, 0]), shared, page_size=page, n_rows=T)
    kv = rand((T, 2, Hk, D), 4, torch.bfloat16).cuda()
    _, k = rn.qk_norm_rope(None, kv[:, 0], step.positions, rope, head_dim=D, eps=1e-6)
    rn.kv_cache_append_(cache, k, kv[:, 1], table, step.before, step.cu_seqlens)
    table[1:, :2] = table[0, :2]
    lengths, n_free, shared = i32([T] * B), step.n_free, i32([2] * B)
    prefix = i32([T])
    seen = 0
    plans = [[5, 1, 9, 3], [1, 1, 1, 1], [1, -1, 1, 1], [1, 20, 1, 1], [1, 1, 1, 1]]
    for i, new in enumerate(plans):
        T = 40
        step = rn.kv_pages_step_(free, n_free, table, lengths, i32(new), shared, page_size=page, n_rows=T)
        row = rand((T, (Hq + 2 * Hk) * D), 10 + i, torch.bfloat16).cuda()
        q, k = rn.qk_norm_rope(row[:, :Hq * D], row[:, Hq * D:(Hq + Hk) * D], step.positions, rope, head_dim=D, eps=1e-6)
        rn.kv_cache_append_(cache, k, row[:, (Hq + Hk) * D:], table, step.before, step.cu_seqlens)
        # the last row of each sequence asks
        last = (step.cu_seqlens[1:] - 1).long().clamp(min=0)
        ask = q[last].view(B, Hq, D)
        o = rn.kv_cache_prefix_attention(ask, cache, table, step.after, prefix)
        t = {"k": cache.k, "v": cache.v, "k_scale": cache.k_scale, "v_scale": cache.v_scale}
        want, bound = ref.attend(ask[:, None], t, table, step.after, 1 / math.sqrt(D), 0, 0)
        within(o[:, None], want, bound)
        x, r = rand((T, H), 20 + i, torch.bfloat16).cuda(), rand((T, H), 30 + i, torch.bfloat16).cuda()
        y, h = torch.full_like(x, 7.0), torch.full_like(r, 7.0)
        rn.fused_block_norms(x, r, w, w, eps=1e-6, gate=gate, gate_index=step.rows, out=y, residual_out=h)
        on = step.rows >= 0
        assert int(on.sum()) == sum(max(a, 0) for a in new) and (y[~on] == 7).all()
        check_norms((y[on], h[on], None), x[on], r[on], w, w, gate, step.rows[on], False, 1.0, 0.0)
        # every row's slot holds its value
        for tk in torch.nonzero(on)[:, 0].tolist()[::7]:
            slot = int(step.slots[tk])
            code = cache.v[slot // page, :, slot % page].view(torch.float8_e4m3fn).float()
            v = code * cache.v_scale[slot // page, :, slot % page // 16][:, None]
            was = row[tk, (Hq + Hk) * D:].view(Hk, D).float()
            # a code's half step, or half of 2^-9 of the scale (at most the largest of 16 rows over 448)
            assert bool(((v - was).abs() <= was.abs() * 2.0 ** -3 + 8 * 2.0 ** -9).all())
        lengths, n_free = step.after, step.n_free
        seen += int(on.sum())
        if new[1] < 0:  # the next one begins behind the same prompt
            assert int(lengths[1]) == 0
            lengths[1] = 32
    assert seen == sum(max(a, 0) for p in plans for a in p)
    assert int(n_free) == B * width - 2 - sum(-(-int(L) // page) - 2 for L in lengths)


# ---------------------------------------------------------------- drawn cases


@pytest.mark.parametrize("seed", range(24))
def test_prefix_drawn(rn, seed):
    rng = random.Random(1000 + seed)
    D, Hk, n = rng.choice([64, 128, 256]), rng.choice([1, 2, 3]), rng.choice([1, 1, 2, 5])
    G, page = rng.choice([1, 3, 4, 8]), rng.choice([16, 32, 48, 128])
    groups = [(rng.randint(1, rng.choice([2, 9, 40])), rng.randint(0, rng.choice([6, 40])) * page)
              for _ in range(rng.choice([1, 1, 2, 5]))]
    t, table, lengths, P, cu = prefix_state(groups, owns(groups, n, seed, rng.choice([n + 1, 60, 300])), Hk, page, D,
                                            seed=seed, spread=rng.random() < 0.3, n=n)
    for s in range(lengths.shape[0]):
        if rng.random() < 0.1:
            lengths[s] = rng.choice([0, -1, 1, int(lengths[s]) // 2])
    dt = rng.choice([torch.bfloat16, torch.float16])
    q = rand((lengths.shape[0], n, Hk * G, D), seed, dt).cuda()
    if rng.random() < 0.3:  # lengths that are shorter than what is shared in earnest
        P = (P.double() * rng.random()).to(torch.int32)
    want, bound = ref.attend(q, t, table, lengths, float(torch.tensor(0.09)), 0, 0)
    within(run_prefix(rn, q, t, table, lengths, P, cu, n, scale=0.09), want, bound)


@pytest.mark.parametrize("seed", range(24))
def test_norms_drawn(rn, seed):
    rng = random.Random(2000 + seed)
    T, H = rng.choice([1, 3, 50, 700]), rng.choice([rng.randint(1, 300), rng.randint(300, 5000), 8 * rng.randint(1, 2100)])
    dtype, gate, offset = rng.choice(["bf16", "f16", "f32"]), rng.choice(["none", "layer", "token", "sequence"]), rng.choice([0.0, 1.0])
    stream, fp8 = ("same" if dtype == "f32" else rng.choice(["same", "f32"])), rng.random() < 0.4
    x, r, pw, w, g, index = norms_inputs(T, H, dtype, stream, gate, offset, seed)
    if rng.random() < 0.2:
        pw = None
    if rng.random() < 0.2:
        w = None
    if gate == "sequence" and rng.random() < 0.5:  # rows of a wider tensor, off the grid
        wide = torch.zeros((3, 2 * H + 1), dtype=g.dtype, device="cuda")
        wide[:, 1:H + 1] = g
        g = wide[:, 1:H + 1]
    done = rn.fused_block_norms(x, r, pw, w, eps=1e-5, gate=g, gate_index=index, residual_scale=-0.5, weight_offset=offset,
                                out_dtype="fp8" if fp8 else None)
    check_norms(done, x, r, pw, w, g, index, fp8, -0.5, offset, 1e-5)


@pytest.mark.parametrize("seed", range(24))
def test_pages_drawn(rn, seed):
    rng = random.Random(3000 + seed)
    B, page, width = rng.randint(1, rng.choice([5, 60, 900])), rng.choice([16, 48, 256]), rng.randint(1, 20)
    free, n_free, table, lengths, more, keep = pages_state(rng, B, page, width, rng.randint(0, 4), done=rng.choice([0.0, 0.3]),
                                                           shared=rng.choice([0, 0, 1]), new=rng.choice([1, 30]),
                                                           most=rng.randint(1, width + 1))
    n_free = min(n_free, rng.choice([n_free, B // 2, 0]))
    rows = sum(m for m, L in zip(more, lengths) if m > 0 and L >= 0)
    step = check_pages(rn, free, n_free, table, lengths, more, keep, page, max(0, rows + rng.choice([0, 0, 3, -2])))
    # a pool that ran out leaves entries of -1 inside of the sequences
    bad = any(p < 0 for s, m in enumerate(more) if m < 0 <= lengths[s] for p in table[s][keep[s]:-(-lengths[s] // page)])
    bad = bad or any(row >= 0 and slot < 0 and step.before[row] >= 0 for row, slot in zip(step.rows.tolist(), step.slots.tolist()))
    assert rn.rmsattn_read_status(clear=True) == (rn.RMSATTN_BAD_PAGE if bad else 0)


def test_a_window_of_no_rows_and_one_column(rn):
    # the smallest of everything: one head, one sequence of a group of one, one token
    t = ref.random_cache(2, 1, 16, 64, 7, "cuda", spread=False)
    q = rand((1, 1, 1, 64), 3, torch.bfloat16).cuda()
    table, lengths = i32([[1]]), i32([1])
    for P in (0, 1, 16):
        within(run_prefix(rn, q, t, table, lengths, i32([P]), None, 1), *ref.attend(q, t, table, lengths, 0.125, 0, 0))
    empty = rn.kv_cache_prefix_attention(q[:0, 0], make_cache(rn, t), table[:0], lengths[:0], i32([16]))
    assert tuple(empty.shape) == (0, 1, 64)


# ---------------------------------------------------------------- far and empty


def test_prefix_pages_past_32_bits(rn):
    # the same pages at the begin of a cache and behind 2^32 bytes of it
    Hk, page, D, groups = 8, 64, 128, [(9, 640), (3, 128)]
    t, table, lengths, P, cu = prefix_state(groups, owns(groups, 1), Hk, page, D)
    n, size = t["k"].shape[0], Hk * page * D
    far = 2 ** 32 // size + 5
    big = {}
    for name, v in t.items():
        big[name] = torch.empty((far + n,) + v.shape[1:], dtype=v.dtype, device="cuda")
        big[name][far:] = v
    q = rand((12, 1, 32, D), 3, torch.bfloat16).cuda()
    got = run_prefix(rn, q, big, table + far, lengths, P, cu, 1)
    within(got, *ref.attend(q, t, table, lengths, 1 / math.sqrt(D), 0, 0))
    assert torch.equal(got, run_prefix(rn, q, t, table, lengths, P, cu, 1))


def test_prefix_of_no_groups(rn):
    t, table, lengths, _, _ = prefix_state([(5, 64)], owns([(5, 64)], 1), 2, 16, 64)
    q = rand((5, 1, 4, 64), 3, torch.bfloat16).cuda()
    got = run_prefix(rn, q, t, table, lengths, i32([]), i32([0]), 1)
    within(got, *ref.attend(q, t, table, lengths, 0.125, 0, 0))


def test_pages_slots_past_32_bits(rn):
    page, n = 65536, 40000
    free, n_free = rn.kv_free_pages(n)
    free = free.flip(0).contiguous()  # the last page first
    table = torch.full((3, 4), -1, dtype=torch.int32, device="cuda")
    step = rn.kv_pages_step_(free, n_free, table, i32([0, 0, 0]), i32([70000, 5, 1]), page_size=page, n_rows=70010)
    assert table[:, 0].tolist() == [n - 1, n - 3, n - 4] and int(table[0, 1]) == n - 2
    want = [(n - 1) * page + i for i in range(page)] + [(n - 2) * page + i for i in range(70000 - page)]
    want += [(n - 3) * page + i for i in range(5)] + [(n - 4) * page] + [-1] * 4
    assert step.slots.tolist() == want and step.n_free.tolist() == [n - 4]


@pytest.mark.parametrize("H", [8192, 8191])
def test_norms_of_elements_past_31_bits(rn, H):
    T = 2 ** 31 // H + 3
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn((T, H), generator=g, device="cuda", dtype=torch.bfloat16)
    gate = torch.randn((T, H), generator=g, device="cuda", dtype=torch.bfloat16)
    y, h, _ = rn.fused_block_norms(x, x, eps=1e-6, gate=gate, residual_scale=0.5)
    rows = slice(T - 4, T)
    check_norms((y[rows], h[rows], None), x[rows], x[rows], None, None, gate[rows], None, False, 0.5, 0.0)
    check_norms((y[:2], h[:2], None), x[:2], x[:2], None, None, gate[:2], None, False, 0.5, 0.0)


def test_prefix_of_more_groups_than_a_block_has_threads(rn):
    groups = [(2, 32 * (g % 3)) for g in range(700)]
    t, table, lengths, P, cu = prefix_state(groups, owns(groups, 1, most=20), 1, 16, 64)
    q = rand((1400, 1, 2, 64), 3, torch.bfloat16).cuda()
    within(run_prefix(rn, q, t, table, lengths, P, cu, 1), *ref.attend(q, t, table, lengths, 0.125, 0, 0))
