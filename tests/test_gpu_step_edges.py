"""GPU tests of the serving step's operators at their edges: empty batches, rows and
sequences that are left out, shared memory between arguments, many small groups."""
import math

import pytest
import torch
from torch.utils._python_dispatch import TorchDispatchMode

import attn_ref as ref
import step_ref
from test_gpu_attn import DT, make_cache, rand, within
from test_gpu_step import i32, norms_inputs, owns, prefix_state, rn, run_prefix  # noqa: F401  (rn: a fixture)

pytestmark = pytest.mark.gpu


# ---------------------------------------------------------------- norms


@pytest.mark.parametrize("eps", [1e-6, 1])  # (a whole number: the way that is not marshalled natively)
@pytest.mark.parametrize("out_dtype", [None, "fp8"])
@pytest.mark.parametrize("gate", ["none", "layer", "token", "sequence"])
def test_norms_of_no_tokens(rn, eps, out_dtype, gate):  # noqa: F811
    H = 64
    x, r, pw, w, _, _ = norms_inputs(0, H, "bf16", "same", "none", 0.0)
    g = {"none": None, "layer": torch.ones(H), "token": torch.ones(0, H), "sequence": torch.ones(3, H)}[gate]
    out, ro, scale = rn.fused_block_norms(x, r, pw, w, eps=eps, gate=None if g is None else g.bfloat16().cuda(),
                                          gate_index=i32([]) if gate == "sequence" else None, out_dtype=out_dtype)
    assert out.shape == (0, H) and ro.shape == (0, H) and (scale is None if out_dtype is None else scale.shape == (0,))


@pytest.mark.parametrize("eps", [1e-6, 1])
def test_norms_of_no_gates(rn, eps):  # noqa: F811
    # no sequence has a gate row: every token is left out, and one that names a row is told
    x, r, pw, w, _, _ = norms_inputs(5, 64, "bf16", "same", "none", 0.0)
    none = torch.ones(0, 64, dtype=torch.bfloat16, device="cuda")
    out, ro = torch.full_like(x, 7.0), torch.full_like(r, 5.0)
    for index, status in (([-1] * 5, 0), ([-1, -3, 0, -1, -1], rn.RMSATTN_BAD_PAGE)):
        rn.fused_block_norms(x, r, pw, w, eps=eps, gate=none, gate_index=i32(index), out=out, residual_out=ro)
        torch.cuda.synchronize()
        assert rn.rmsattn_read_status(clear=True) == status
        assert (out == 7).all() and (ro == 5).all()


@pytest.mark.parametrize("eps", [1e-6, 1])
@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("H,stream", [(64, "same"), (257, "f32"), (4096, "same"), (20000, "f32")])
def test_norms_rows_left_out_of_new_outputs_are_zeros(rn, eps, fp8, H, stream):  # noqa: F811
    T = 7
    x, r, pw, w, g, _ = norms_inputs(T, H, "bf16", stream, "sequence", 0.0)
    index = i32([0, -1, 2, -1, -5, 1, -1])
    off = (index < 0).cpu()
    kw = dict(eps=eps, gate=g, gate_index=index, out_dtype="fp8" if fp8 else None)
    size = T * H * (1 if fp8 else 2)

    def dirty():  # what the allocator hands out next is not zeros
        junk = [torch.full((n,), 0x7F, dtype=torch.uint8, device="cuda")
                for n in (size, T * H * r.element_size(), 4 * T) for _ in range(8)]
        del junk

    full = rn.fused_block_norms(x, r, pw, w, **{**kw, "gate_index": index.clamp(min=0)})
    dirty()
    out, ro, scale = rn.fused_block_norms(x, r, pw, w, **kw)
    assert not out[off].any() and not ro[off].any() and (scale is None or not scale[off].any())
    for a, b in zip((out, ro, scale), full):
        assert a is None or torch.equal(a[~off], b[~off])
    # a given output keeps its rows, beside new ones
    mine = torch.full_like(ro, 5.0)
    out, ro, scale = rn.fused_block_norms(x, r, pw, w, residual_out=mine, **kw)
    assert (mine[off] == 5).all() and not out[off].any() and torch.equal(mine[~off], full[1][~off])
    if fp8:
        mine = torch.full((T,), 3.0, device="cuda")
        out, ro, scale = rn.fused_block_norms(x, r, pw, w, out_scale=mine, **kw)
        assert (mine[off] == 3).all() and not out[off].any() and not ro[off].any()


# ---------------------------------------------------------------- shared prefix


@pytest.mark.parametrize("D", [64, 128, 256])
def test_prefix_follows_tables_scales_and_queries_written_just_before(rn, D):  # noqa: F811
    # the shared part does not wait for the launch before it: what the stream wrote up to the call
    # (table, scales, codes, queries, lengths) is read, never what lay there at the call before
    groups, Hk, page = [(12, 640), (9, 320)], 2, 16
    t, table, lengths, P, cu = prefix_state(groups, owns(groups, 1), Hk, page, D)
    B, pages = lengths.shape[0], t["k"].shape[0]
    states = []
    for i in range(6):
        order = torch.randperm(pages, generator=torch.Generator().manual_seed(i)).cuda()
        back = torch.argsort(order)  # the same tokens in other pages, under other scales
        moved = {n: v[order].contiguous() for n, v in t.items()}
        moved["k_scale"] *= 0.5 + 0.1 * i
        moved["v_scale"] *= 2.0 ** (i - 3)
        states.append((rand((B, 8, D), i, torch.bfloat16).cuda(), moved, back[table.long()].to(torch.int32), lengths - i % 3))
    live = [states[0][0].clone(), {n: v.clone() for n, v in t.items()}, table.clone(), lengths.clone()]
    cache = make_cache(rn, live[1])

    def one(state):
        live[0].copy_(state[0])
        for n, v in state[1].items():
            live[1][n].copy_(v)
        live[2].copy_(state[2])
        live[3].copy_(state[3])
        return rn.kv_cache_prefix_attention(live[0], cache, live[2], live[3], P, cu, pdl=True)

    want = [rn.kv_cache_prefix_attention(q, make_cache(rn, c), tab, lens, P, cu) for q, c, tab, lens in states]
    assert len({w.float().sum().item() for w in want}) == len(want)
    one(states[0])
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = [one(s) for s in states]
    for _ in range(5):
        for o in outs:
            o.zero_()
        graph.replay()
        assert all(torch.equal(o, w) for o, w in zip(outs, want))
    assert all(torch.equal(one(s), w) for s, w in zip(states, want))


# ---------------------------------------------------------------- pages


def test_pages_of_lengths_between_the_tables_rows(rn):  # noqa: F811
    # one buffer: three rows of two entries, five apart, and the lengths in the gap behind the first row
    room = torch.zeros(16, dtype=torch.int32, device="cuda")
    table, lengths = room[:15].view(3, 5)[:, :2], room[2:5]
    table.fill_(-1)
    lengths.copy_(i32([0, 0, 0]))
    free, n_free = rn.kv_free_pages(6)
    for page in (16, 48):
        step = rn.kv_pages_step_(free, n_free, table, lengths, i32([20, -1, page]), page_size=page, n_rows=96)
        assert step.after.tolist() == [20, 0, page] and lengths.tolist() == [0, 0, 0]
    # ... but not in a row
    with pytest.raises(rn.RmsnError):
        rn.kv_pages_step_(free, n_free, table, room[1:4], i32([1, 1, 1]), page_size=16, n_rows=96)
    with pytest.raises(rn.RmsnError):
        rn.kv_pages_step_(free, n_free, table, free[:3], i32([1, 1, 1]), page_size=16, n_rows=96)
    with pytest.raises(rn.RmsnError):
        rn.kv_pages_step_(free, free[5:], table, lengths, i32([1, 1, 1]), page_size=16, n_rows=96)


@pytest.mark.parametrize("H", [256, 251, 20000])
def test_norms_outputs_on_inputs_row_for_row(rn, H):  # noqa: F811
    x, r, pw, w, g, _ = norms_inputs(9, H, "bf16", "same", "token", 0.0)
    want = rn.fused_block_norms(x, r, pw, w, eps=1e-6, gate=g)[:2]
    for out, ro in (("x", "r"), ("r", "x"), ("g", "r"), ("x", "g"), (None, "x"), ("r", None)):
        t = dict(x=x.clone(), r=r.clone(), g=g.clone())
        got = rn.fused_block_norms(t["x"], t["r"], pw, w, eps=1e-6, gate=t["g"], out=t.get(out), residual_out=t.get(ro))
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    # bytes of codes on x's rows are another row's
    codes = x.view(torch.uint8).flatten()[:9 * H].view(9, H)
    with pytest.raises(rn.RmsnError):
        rn.fused_block_norms(x, r, pw, w, eps=1e-6, out_dtype="fp8", out=codes)
    with pytest.raises(rn.RmsnError):
        rn.fused_block_norms(x, r, pw, w, eps=1e-6, gate=g, gate_index=i32([0] * 9), out=g)


@pytest.mark.parametrize("pdl", [False, 0])  # (a number: the way that is not marshalled natively)
def test_pages_of_lazy_copies(rn, pdl):  # noqa: F811
    # a copy that shares its memory until it is written to gets its own then
    free, n_free = rn.kv_free_pages(8)
    table, lengths = i32([[0, 1], [2, -1]]), i32([32, 5])
    n_free.fill_(5)
    copies = [torch._lazy_clone(t) for t in (free, table)]
    step = rn.kv_pages_step_(copies[0], n_free, copies[1], lengths, i32([-1, 20]), page_size=16, n_rows=20, pdl=pdl)
    assert free.tolist() == list(range(7, -1, -1)) and table.tolist() == [[0, 1], [2, -1]]
    assert copies[1].tolist() == [[0, 1], [2, 1]] and copies[0].tolist() == [7, 6, 5, 4, 3, 0, 1, 0]
    assert step.n_free.tolist() == [6]


# ---------------------------------------------------------------- the native binding


class Seen(TorchDispatchMode):
    """What a mode sees being made."""

    def __init__(self):
        super().__init__()
        self.made = []

    def __torch_dispatch__(self, func, types, args=(), kwargs=None):
        out = func(*args, **(kwargs or {}))
        if func is torch.ops.aten.empty.memory_format:
            self.made.append((tuple(out.shape), out.dtype, out.data_ptr()))
        return out


@pytest.mark.parametrize("eps", [1e-6, 1])
def test_dispatch_modes_see_the_results(rn, eps):  # noqa: F811
    groups, Hk, page, D = [(4, 64)], 2, 16, 64
    t, table, lengths, P, cu = prefix_state(groups, owns(groups, 1), Hk, page, D)
    cache = make_cache(rn, t)
    q, k = rand((4, 4, D), 1, torch.bfloat16).cuda(), rand((4, Hk, D), 2, torch.bfloat16).cuda()
    x, r, pw, w, _, _ = norms_inputs(3, 64, "bf16", "f32", "none", 0.0)
    free, n_free = rn.kv_free_pages(8)
    rope = rn.rope_table(D)
    positions = i32([0, 1, 2, 3])
    scale = None if eps != 1 else 1
    calls = [
        lambda: rn.qk_norm_rope(q, k, positions, rope, head_dim=D, eps=eps),
        lambda: [rn.kv_cache_attention(q, cache, table, lengths, scale=scale)],
        lambda: [rn.kv_cache_prefix_attention(q, cache, table, lengths, P, cu, scale=scale)],
        lambda: rn.fused_block_norms(x, r, pw, w, eps=eps, out_dtype="fp8"),
        lambda: rn.kv_pages_step_(free, n_free, i32([[-1, -1]]), i32([0]), i32([3]), page_size=16, n_rows=4),
    ]
    for call in calls:
        with Seen() as seen:
            made = call()
        for m in made:
            assert (tuple(m.shape), m.dtype, m.data_ptr()) in seen.made
        free, n_free = rn.kv_free_pages(8)
        for a, b in zip(made, call()):
            assert torch.equal(a, b)
        free, n_free = rn.kv_free_pages(8)


def test_prefix_workspace_goes_by_rows_not_by_groups(rn):  # noqa: F811
    size = rn.load_attn().rmsattn_kv_prefix_attention_workspace
    for B, n, Hq, Hk, D in ((4096, 1, 32, 8, 128), (4096, 1, 16, 2, 256), (3000, 2, 64, 8, 64)):
        one, pairs = size(B, n, Hq, Hk, D, 4096, 1), size(B, n, Hq, Hk, D, 4096, B // 2)
        rows = B * n * Hq
        assert one < rows * (8 * D + 16) + 2 ** 28
        # a group more: 32 bytes, and what fills its rows up to eights for each key head
        assert pairs < one + B // 2 * (32 + 7 * Hk * (D + 2) * 4) + 2 ** 20


@pytest.mark.parametrize("groups,n,Hq,Hk,D,page,dtype", [
    ([(2, 32)] * 90 + [(3, 64)] * 5 + [(1, 48)] * 3, 1, 32, 8, 128, 16, "bf16"),
    ([(65, 256), (2, 48), (33, 128), (7, 64), (129, 32), (2, 16)], 1, 16, 4, 128, 16, "f16"),
    ([(70, 512), (3, 64), (64, 192), (2, 48)], 1, 32, 8, 64, 16, "bf16"), ([(21, 512), (3, 64), (2, 48)] * 3, 3, 12, 4, 64, 16, "f16"),
    ([(2, 64), (40, 320), (2, 32), (17, 320)], 1, 14, 2, 256, 16, "bf16"), ([(2, 3200)] * 4, 1, 5, 1, 128, 32, "bf16"),
    ([(600, 64), (2, 32)], 1, 9, 3, 64, 32, "bf16"), ([(300, 16)], 2, 7, 1, 128, 16, "bf16"),
])
def test_prefix_groups_of_any_size_side_by_side(rn, groups, n, Hq, Hk, D, page, dtype):  # noqa: F811
    t, table, lengths, P, cu = prefix_state(groups, owns(groups, n, most=40), Hk, page, D, n=n)
    q = rand((lengths.shape[0], n, Hq, D), 3, DT[dtype]).cuda()
    want, bound = ref.attend(q, t, table, lengths, 1 / math.sqrt(D), 0, 0)
    within(run_prefix(rn, q, t, table, lengths, P, cu, n), want, bound)


@pytest.mark.parametrize("H", [64, 251, 4096, 20000])
@pytest.mark.parametrize("stream", ["same", "f32"])
def test_norms_codes_of_rows_near_zero(rn, H, stream):  # noqa: F811
    # rows whose 448 / max|y| lies outside fp32's range: y = h / sqrt(eps), for h^2 is far below eps
    T, eps = 8, 1e-6
    x = torch.zeros(T, H, dtype=torch.bfloat16)
    g = torch.Generator().manual_seed(5)
    whole = torch.randint(-64, 65, (T, H), generator=g).float()
    whole[:, 0] = 64
    whole[:, 1] = 0
    size = [2.0 ** -133, 2.0 ** -136, 2.0 ** -130, 1.0, 0.0, 2.0 ** -127, 2.0 ** -124, 2.0 ** -100]  # (bf16 ends at 2^-133)
    if stream == "same":
        size[1] = 2.0 ** -132
    r = (whole * torch.tensor(size)[:, None]).to(torch.float32 if stream == "f32" else torch.bfloat16)
    y, h, scale = rn.fused_block_norms(x.cuda(), r.cuda(), eps=eps, out_dtype="fp8")
    assert torch.equal(h.cpu(), r)
    _, _, of = step_ref.norms(x, r, None, None, None, None, eps, 1.0, 0.0)
    want, _, err = of(r)
    # (y is rounded twice, to 2^-149 at the least; the scale once)
    normal = (scale > 2.0 ** -126).cpu()
    step_ref.check_codes(y.cpu()[normal], scale.cpu()[normal], want[normal], err[normal] + 2.0 ** -148)
    assert bool(((scale.cpu().double() - want.abs().amax(-1) / 448).abs() <= (err.amax(-1) + 2.0 ** -140) / 448 + 2.0 ** -149).all())
    codes = y.cpu().view(torch.float8_e4m3fn).double()
    assert bool(codes.isfinite().all()) and not codes[4].any() and (codes[:, 1] == 0).all()
    live = [i for i, s in enumerate(size) if s]
    q = want[live] * 448 / want[live].abs().amax(-1, keepdim=True)
    # half a step of the code, and y's roundings over the row's largest (2^-117 at the least)
    assert bool(((codes[live] - q).abs() <= ref.half_step(q) * (1 + 2.0 ** -20) + 448 * (2.0 ** -30 + 2.0 ** -18)).all())
