"""GPU tests of the attention path: qk_norm_rope, kv_cache_append_ and
kv_cache_attention against 64-bit references (tests/attn_ref.py), at the
sizes, masks, strides and values where they can go wrong."""
import math
import os
import subprocess
import sys

import pytest
import torch

import attn_ref as ref
import oracle
import parity

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


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


def rand(shape, seed, dtype=torch.float32, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (scale * torch.randn(shape, generator=g)).to(dtype)


def within(got, want, bound, what=""):
    got = got.double().cpu()
    off = (got - want.cpu()).abs()
    assert bool((off <= bound.cpu()).all()), f"{what}: {float((off / bound.cpu()).nan_to_num(9e9).max())} of the bound"


# ---------------------------------------------------------------- rope

ROPE = [
    # T, Hq, Hk, D, sections, dtype
    (1, 32, 8, 128, [64], "bf16"), (7, 4, 2, 64, [8, 12, 12], "bf16"), (1, 1, 1, 16, [8], "bf16"),
    (3, 2, 0, 128, [10, 0, 20], "f16"), (5, 0, 3, 256, [128], "bf16"), (33, 5, 1, 96, [16, 16, 16], "f16"),
    (9, 3, 2, 80, [5, 7, 8], "bf16"), (4, 2, 1, 512, [100, 56], "bf16"), (5, 2, 2, 128, [20, 20, 24], "f32"),
    (6, 1, 1, 20, [3, 2], "f32"), (2, 2, 1, 17, [4], "bf16"), (3, 1, 2, 1, [], "f32"), (4, 2, 2, 64, [], "f16"),
    (2, 1, 1, 1000, [7, 9], "f16"), (300, 6, 2, 128, [16, 24, 24], "bf16"), (2, 40, 40, 128, [32], "bf16"),
    (1, 64, 8, 256, [32, 32], "f32"),
]


@pytest.mark.parametrize("T,Hq,Hk,D,sections,dtype", ROPE)
@pytest.mark.parametrize("norm,woff,weights", [(True, 0.0, True), (True, 1.0, True), (True, 0.0, False),
                                               (False, 0.0, False)])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("form", ["own", "fused", "place"])
def test_rope(rn, T, Hq, Hk, D, sections, dtype, norm, woff, weights, interleaved, form):
    dt = DT[dtype]
    table = rn.rope_table(2 * sum(sections), sections=sections or None, device="cuda")
    row = rand((T, (Hq + 2 * Hk) * D), 11 * T + D, dt, 2.0)
    q, k = row[:, :Hq * D], row[:, Hq * D:(Hq + Hk) * D]
    wq, wk = (rand((D,), s, dt, 0.3) for s in (1, 2))
    if not weights:
        wq = wk = None
    g = torch.Generator().manual_seed(T)
    pos = torch.randint(0, 1 << 20, (table.n_axes, T), generator=g)
    pos = pos.to(torch.int64 if D % 3 else torch.int32)
    eps = 1e-5 if norm else None
    full = row.cuda()
    gq, gk = full[:, :Hq * D], full[:, Hq * D:(Hq + Hk) * D]
    if form == "own":
        gq, gk = gq.reshape(T, Hq, D).contiguous(), gk.reshape(T, Hk, D).contiguous()
    if not Hq:
        gq = None
    if not Hk:
        gk = None
    kw = dict(q_out=gq, k_out=gk) if form == "place" else {}
    oq, ok = rn.qk_norm_rope(gq, gk, pos.cuda(), table, None if wq is None else wq.cuda(),
                             None if wk is None else wk.cuda(), head_dim=D, eps=eps, weight_offset=woff,
                             interleaved=interleaved, **kw)
    for x, w, o, H in ((q, wq, oq, Hq), (k, wk, ok, Hk)):
        if H:
            want, bound = ref.rope(x, w, table, pos, D, eps, woff, interleaved)
            within(o.reshape(T, H * D), want, bound, f"H {H}")
    if form == "place":  # the value heads stay, and the results lie in the row
        assert torch.equal(full[:, (Hq + Hk) * D:].cpu(), row[:, (Hq + Hk) * D:])
    elif form == "fused":
        assert torch.equal(full.cpu(), row)


@pytest.mark.parametrize("bits,top", [(32, 2**31 - 1), (64, 2**53 + 12345), (64, 2**63 - 1)])
def test_rope_far_and_negative_positions(rn, bits, top):
    D = 64
    pos = torch.tensor([[top, -top, 1 - top, top - 7, 0, -1]], dtype=torch.int32 if bits == 32 else torch.int64)
    x = rand((6, 2 * D), 5)
    table = rn.rope_table(D, device="cuda")
    out, _ = rn.qk_norm_rope(x.cuda(), None, pos[0].cuda(), table, head_dim=D)
    within(out, *ref.rope(x, None, table, pos, D, None, 0.0, False))


@pytest.mark.parametrize("T", [1, 5])
def test_rope_one_row_of_positions_for_all_axes(rn, T):
    table = rn.rope_table(64, sections=[8, 12, 12])
    x = rand((T, 4 * 64), 1, torch.bfloat16).cuda()
    pos = torch.arange(3, 3 + T, dtype=torch.int32, device="cuda")
    got, _ = rn.qk_norm_rope(x, None, pos.expand(3, T), table, head_dim=64, eps=1e-6)
    want, _ = rn.qk_norm_rope(x, None, pos.expand(3, T).contiguous(), table, head_dim=64, eps=1e-6)
    assert torch.equal(got, want)


def test_rope_axis_order_and_pair_tables(rn):
    # pairs handed to the axes in turn, with frequencies of the caller's own
    D, T = 32, 5
    axis = [p % 3 for p in range(D // 2)]
    table = rn.rope_table(D, axis=axis, inv_freq=[(-1) ** p * 3.0 / (p + 1) for p in range(D // 2)], device="cuda")
    pos = torch.arange(3 * T, dtype=torch.int32).reshape(3, T) * 17 - 20
    x = rand((T, 3 * D), 8, torch.bfloat16)
    wide = torch.zeros((3, T + 9), dtype=torch.int32, device="cuda")
    wide[:, :T] = pos
    out, _ = rn.qk_norm_rope(x.cuda(), None, wide[:, :T], table, head_dim=D, interleaved=True)
    within(out, *ref.rope(x, None, table, pos, D, None, 0.0, True))


@pytest.mark.parametrize("off,pad", [(1, 0), (3, 5), (8, 8), (0, 3)])
def test_rope_unaligned_views(rn, off, pad):
    T, H, D = 6, 3, 64
    flat = torch.zeros(T * (H * D + pad) + off + 8, dtype=torch.bfloat16, device="cuda")
    q = flat[off:off + T * (H * D + pad)].reshape(T, H * D + pad)[:, :H * D]
    x = rand((T, H * D), 4, torch.bfloat16)
    q.copy_(x)
    table = rn.rope_table(D, device="cuda")
    pos = torch.arange(T, dtype=torch.int32)
    w = rand((D,), 3, torch.bfloat16)
    out, _ = rn.qk_norm_rope(q, None, pos.cuda(), table, w.cuda(), head_dim=D, eps=1e-6)
    within(out, *ref.rope(x, w, table, pos[None], D, 1e-6, 0.0, False))


def test_rope_special_values(rn):
    # zero heads with eps 0 give NaN as 0 * inf does; infinities and NaN stay in their pair without the norm
    D = 64
    x = torch.zeros((4, D))
    x[0, 3] = math.inf
    x[1, 5] = math.nan
    x[2] = 1e-30
    table = rn.rope_table(D, device="cuda")
    pos = torch.tensor([1, 2, 3, 4], dtype=torch.int32, device="cuda")
    out, _ = rn.qk_norm_rope(x.cuda(), None, pos, table, head_dim=D)
    bad = ~torch.isfinite(out.cpu())
    want = torch.zeros((4, D), dtype=torch.bool)
    want[0, [3, 35]] = want[1, [5, 37]] = True
    assert torch.equal(bad, want)
    out, _ = rn.qk_norm_rope(x.cuda(), None, pos, table, head_dim=D, eps=1e-6)
    assert bool(out[0].isnan().any()) and bool(out[1].isnan().all()) and bool((out[3] == 0).all())


def test_rope_equals_qk_norm_where_nothing_turns(rn):
    T, Hq, Hk, D = 37, 4, 2, 128
    x = rand((T, (Hq + Hk) * D), 9, torch.bfloat16).cuda()
    wq, wk = rand((D,), 1, torch.bfloat16).cuda(), rand((D,), 2, torch.bfloat16).cuda()
    table = rn.rope_table(D, device="cuda")
    oq, ok = rn.qk_norm_rope(x[:, :Hq * D], x[:, Hq * D:], torch.zeros(T, dtype=torch.int32, device="cuda"), table,
                             wq, wk, head_dim=D, eps=1e-6)
    y = x.clone()
    rn.qk_norm_(y[:, :Hq * D], y[:, Hq * D:], wq, wk, head_dim=D, eps=1e-6)
    step = (torch.cat([oq, ok], 1).float() - y.float()).abs() / y.float().abs().clamp(min=1e-30)
    assert float(step.max()) <= 2.0 ** -7  # one bf16 step: the two order their products differently


# ---------------------------------------------------------------- append

def make_cache(rn, tensors):
    return rn.KVCache(tensors["k"], tensors["v"], tensors["k_scale"], tensors["v_scale"])


def copy_of(t):
    return {k: v.clone() for k, v in t.items()}


APPEND = [
    # lengths, new, H, D, page, dtype
    ([0], [1], 1, 64, 16, "bf16"), ([15, 16, 17, 31], [1, 1, 1, 1], 2, 128, 16, "bf16"),
    ([0, 5, 16, 40], [3, 30, 16, 1], 2, 64, 32, "f16"), ([7, 0, 100], [0, 77, 28], 1, 256, 64, "bf16"),
    ([1, 2, 3, 14], [15, 14, 13, 2], 3, 128, 16, "f32"), ([33], [200], 8, 128, 64, "bf16"),
    ([0, -1, 8, -5, 9], [4, 6, 8, 0, 7], 2, 64, 16, "bf16"), ([12], [600], 2, 256, 128, "f32"),
    ([0] * 40, [1] * 40, 1, 64, 16, "f16"), ([3, 50], [16, 17], 5, 128, 48, "bf16"),
    ([0] * 70, [0, 33] * 35, 2, 64, 16, "bf16"),
]


@pytest.mark.parametrize("lengths,new,H,D,page,dtype", APPEND)
@pytest.mark.parametrize("fused", [True, False])
def test_append(rn, lengths, new, H, D, page, dtype, fused):
    B, T = len(lengths), sum(new)
    most = max(max(l, 0) + n for l, n in zip(lengths, new))
    width = -(-most // page)
    pages = B * width + 3
    before = ref.random_cache(pages, H, page, D, T, "cuda")
    after = copy_of(before)
    table = ref.tables(B, width, pages, 3, "cuda")
    x = rand((T, 2 * H * D + 16), 5 + T) * torch.exp2(2 * rand((T, 1), 6))
    x = x.to(DT[dtype]).cuda()
    k, v = x[:, :H * D], x[:, H * D:2 * H * D]
    if not fused:
        k, v = k.reshape(T, H, D).contiguous(), v.reshape(T, H, D).contiguous()
    cu = torch.tensor([0] + list(torch.tensor(new).cumsum(0)), dtype=torch.int32)
    lens = torch.tensor(lengths, dtype=torch.int32)
    got = rn.kv_cache_append_(make_cache(rn, after), k, v, table, lens.cuda(), cu.cuda())
    assert got.k is after["k"]
    for side, y in (("k", k), ("v", v)):
        ref.check_append(before, after, y.reshape(T, H, D), side, table.cpu(), lens, cu)
    # the same append again finds every scale grown: nothing changes
    again = copy_of(after)
    rn.kv_cache_append_(make_cache(rn, again), k, v, table, lens.cuda(), cu.cuda())
    for name in after:
        assert torch.equal(again[name], after[name]), name


@pytest.mark.parametrize("D,dtype", [(64, "bf16"), (128, "f16"), (256, "bf16"), (128, "f32")])
def test_append_one_token_at_a_time(rn, D, dtype):
    # a decode loop over two block borders, without cu_seqlens; scales grow and shrink
    B, H, page = 3, 2, 16
    t = ref.random_cache(B * 3, H, page, D, 1, "cuda")
    table = ref.tables(B, 3, B * 3, 2, "cuda")
    cache = make_cache(rn, t)
    for step in range(35):
        x = (rand((B, 2 * H * D), step) * 2.0 ** ((step * 7) % 11 - 5)).to(DT[dtype]).cuda()
        lens = torch.tensor([step, step + 3, -1 if step % 5 == 0 else step + 9], dtype=torch.int32)
        before = copy_of(t)
        k, v = x[:, :H * D].reshape(B, H, D), x[:, H * D:]
        rn.kv_cache_append_(cache, k, v, table, lens.cuda())
        for side, y in (("k", k), ("v", v.reshape(B, H, D))):
            ref.check_append(before, t, y, side, table.cpu(), lens, None)


def test_append_special_values(rn):
    H, D, page = 1, 64, 16
    t = ref.random_cache(4, H, page, D, 1, "cuda")
    table = torch.tensor([[2, 0], [1, 3]], dtype=torch.int32, device="cuda")
    x = torch.zeros((12, H, D))
    x[1, 0, 3], x[1, 0, 4] = math.nan, -math.nan
    x[2, 0, 5], x[2, 0, 6], x[2, 0, 7] = math.inf, -math.inf, 1.0
    x[3, 0, 0] = 1e-44  # below every scale
    x[6:] = 3e-39  # a block of subnormals alone
    y = x.clone()
    y[2] = 0  # v without infinities: a NaN does not set a scale
    lens, cu = torch.tensor([14, 3], dtype=torch.int32), torch.tensor([0, 6, 12], dtype=torch.int32)
    before = copy_of(t)
    rn.kv_cache_append_(make_cache(rn, t), x.cuda(), y.cuda(), table, lens.cuda(), cu.cuda())
    ref.check_append(before, t, x, "k", table.cpu(), lens, cu)
    ref.check_append(before, t, y, "v", table.cpu(), lens, cu)
    assert bool(torch.isfinite(t["k_scale"]).all())


def test_append_zero_block_then_values(rn):
    t = ref.random_cache(1, 1, 16, 64, 1, "cuda")
    cache = make_cache(rn, t)
    table = torch.zeros((1, 1), dtype=torch.int32, device="cuda")
    zero = torch.zeros((1, 1, 64), device="cuda")
    rn.kv_cache_append_(cache, zero, zero, table, torch.tensor([0], dtype=torch.int32, device="cuda"))
    assert float(t["k_scale"][0, 0, 0]) == 0 and not bool(t["k"][0, 0, 0].any())
    x = rand((1, 1, 64), 3).cuda()
    before = copy_of(t)
    lens = torch.tensor([1], dtype=torch.int32)
    rn.kv_cache_append_(cache, x, x, table, lens.cuda())
    ref.check_append(before, t, x, "k", table.cpu(), lens, None)


def test_append_bad_pages_and_tokens_past_the_table(rn):
    H, D, page = 2, 64, 16
    before = ref.random_cache(3, H, page, D, 1, "cuda")
    t = copy_of(before)
    table = torch.tensor([[0, 7], [-1, 1], [2, 2]], dtype=torch.int32, device="cuda")
    lens, cu = torch.tensor([10, 12, 30], dtype=torch.int32), torch.tensor([0, 20, 30, 45], dtype=torch.int32)
    x = rand((45, H, D), 2).cuda()
    rn.kv_cache_append_(make_cache(rn, t), x, x, table, lens.cuda(), cu.cuda())
    assert rn.rmsattn_read_status(clear=True) == rn.RMSATTN_BAD_PAGE
    for side in ("k", "v"):
        ref.check_append(before, t, x, side, table.cpu(), lens, cu)


@pytest.mark.parametrize("off", [1, 4])
def test_append_unaligned_views(rn, off):
    T, H, D = 19, 2, 128
    x = torch.zeros(T * (2 * H * D + 3) + 8, dtype=torch.bfloat16, device="cuda")
    row = x[off:off + T * (2 * H * D + 3)].reshape(T, 2 * H * D + 3)
    row.copy_(rand(row.shape, 1))
    k, v = row[:, :H * D], row[:, H * D:2 * H * D]
    before = ref.random_cache(4, H, 16, D, 1, "cuda")
    t = copy_of(before)
    table = ref.tables(1, 3, 4, 1, "cuda")
    lens, cu = torch.tensor([6], dtype=torch.int32), torch.tensor([0, T], dtype=torch.int32)
    rn.kv_cache_append_(make_cache(rn, t), k, v, table, lens.cuda(), cu.cuda())
    for side, y in (("k", k), ("v", v)):
        ref.check_append(before, t, y.reshape(T, H, D), side, table.cpu(), lens, cu)


def layers_cache(rn, pages, H, page, D, device="cuda"):
    """Layer 1 of a cache whose layers lie side by side in each page."""
    codes = torch.randint(0, 100, (pages, 3, 2, H, page, D), dtype=torch.uint8, device=device)
    scale = torch.rand((pages, 3, 2, H, page // 16), device=device)
    t = {"k": codes[:, 1, 0], "v": codes[:, 1, 1], "k_scale": scale[:, 1, 0], "v_scale": scale[:, 1, 1]}
    return codes, scale, t


def test_append_and_attention_in_a_strided_cache(rn):
    H, D, page, T = 2, 64, 16, 50
    codes, scale, t = layers_cache(rn, 6, H, page, D)
    whole = codes.clone(), scale.clone()
    before = copy_of(t)
    table = ref.tables(1, 4, 6, 1, "cuda")
    x = rand((T, 2, H, D), 1, torch.bfloat16).cuda()
    lens, cu = torch.tensor([0], dtype=torch.int32), torch.tensor([0, T], dtype=torch.int32)
    cache = make_cache(rn, t)
    rn.kv_cache_append_(cache, x[:, 0], x[:, 1], table, lens.cuda(), cu.cuda())
    for i, side in enumerate(("k", "v")):
        ref.check_append(before, t, x[:, i], side, table.cpu(), lens, cu)
    for layer in (0, 2):
        assert torch.equal(codes[:, layer], whole[0][:, layer]) and torch.equal(scale[:, layer], whole[1][:, layer])
    q = rand((1, 4, D), 2, torch.bfloat16).cuda()
    lens = torch.tensor([T], dtype=torch.int32, device="cuda")
    got = rn.kv_cache_attention(q, cache, table, lens)
    within(got, *[y[:, 0] for y in ref.attend(q[:, None], t, table, lens, 0.125, 0, 0)])


# ---------------------------------------------------------------- attention

ATTEND = [
    # lengths, n, Hq, Hk, D, page, dtype, window, sinks
    ([1], 1, 1, 1, 64, 16, "bf16", 0, 0), ([1, 2, 15, 16, 17, 33], 1, 4, 2, 128, 16, "bf16", 0, 0),
    ([100, 7, 0, 64], 1, 8, 2, 64, 32, "f16", 0, 0), ([300], 1, 16, 1, 256, 64, "bf16", 0, 0),
    ([1000, 513], 1, 32, 8, 128, 64, "bf16", 0, 0), ([70, 5], 4, 8, 2, 128, 16, "bf16", 0, 0),
    ([40, 3, 8], 5, 7, 1, 64, 16, "f16", 0, 0), ([90], 32, 4, 4, 64, 16, "bf16", 0, 0),
    ([200, 31], 3, 24, 2, 128, 48, "f16", 0, 0), ([130, 9], 2, 12, 1, 256, 16, "bf16", 0, 0),
    ([500, 20], 1, 8, 4, 128, 16, "bf16", 64, 4), ([500, 100], 3, 8, 4, 128, 16, "bf16", 33, 5),
    ([257], 1, 4, 1, 64, 64, "f16", 1, 0), ([257], 4, 4, 1, 64, 64, "f16", 16, 20),
    ([400], 1, 8, 2, 256, 32, "bf16", 100, 1), ([64, 65], 1, 2, 1, 64, 16, "bf16", 64, 0),
    ([333], 2, 64, 1, 64, 16, "f16", 0, 0), ([100], 1, 2, 2, 128, 16, "bf16", 7, 300),
    ([5000, 17, 2100], 1, 8, 2, 128, 64, "bf16", 0, 0), ([3, 2, 1], 8, 2, 1, 128, 16, "bf16", 0, 0),
    ([900], 7, 40, 2, 256, 16, "f16", 200, 3), ([12000], 1, 4, 1, 64, 128, "bf16", 0, 0),
    ([40] * 50, 1, 4, 2, 64, 16, "bf16", 0, 0), ([2000] * 3, 1, 20, 4, 128, 16, "f16", 1000, 17),
]


def spread_out(table, how, Hk):
    """(table, repeats) for the ways that the work is shared out: "rows", short
    tables, a row to a cluster; "line", tables wide enough for long rows, few
    rows; "many", the same with more rows than a block's warps could each have
    eight of (the same sequences over and over)."""
    if how == "rows":
        return table, 1
    page_room = 40000 // 16
    wide = torch.full((table.shape[0], page_room), -1, dtype=torch.int32, device=table.device)
    wide[:, :table.shape[1]] = table
    if how == "line":
        return wide, 1
    times = -(-400 // (table.shape[0] * Hk))
    return wide.repeat(times, 1), times


@pytest.mark.parametrize("lengths,n,Hq,Hk,D,page,dtype,window,sinks", ATTEND)
@pytest.mark.parametrize("how", ["rows", "line", "many"])
def test_attention(rn, lengths, n, Hq, Hk, D, page, dtype, window, sinks, how):
    B = len(lengths)
    width = -(-max(lengths) // page) + 1
    pages = B * width + 2
    t = ref.random_cache(pages, Hk, page, D, 7, "cuda", spread=False)
    table = ref.tables(B, width, pages, 1, "cuda")
    lens = torch.tensor(lengths, dtype=torch.int32, device="cuda")
    q = rand((B, n, Hq, D), 3, DT[dtype]).cuda()
    want, bound = ref.attend(q, t, table, lens, 1 / math.sqrt(D), window, sinks)
    table, times = spread_out(table, how, Hk)
    big = q.repeat(times, 1, 1, 1)
    got = rn.kv_cache_attention(big if n > 1 else big[:, 0], make_cache(rn, t), table, lens.repeat(times),
                                window=window, sinks=sinks)
    within(got.reshape(times, *q.shape), want[None], bound[None])


@pytest.mark.parametrize("D,dtype,qscale", [(64, "bf16", 1.0), (128, "f16", 30.0), (256, "bf16", 1e-3),
                                            (128, "bf16", 1e6), (128, "bf16", 1e-20)])
def test_attention_scales_over_many_binades(rn, D, dtype, qscale):
    # block scales from 2^-8 to 2^8 times the usual: peaked rows, value sums of mixed size; queries
    # outside fp16's range are scaled back by `scale`
    lens = torch.tensor([777, 300], dtype=torch.int32, device="cuda")
    t = ref.random_cache(60, 2, 32, D, 7, "cuda")
    table = ref.tables(2, 25, 60, 1, "cuda")
    q = (rand((2, 1, 8, D), 3) * qscale).to(DT[dtype]).cuda()
    scale = 0.3 / math.sqrt(D) / qscale
    got = rn.kv_cache_attention(q[:, 0], make_cache(rn, t), table, lens, scale=scale)
    want, bound = ref.attend(q, t, table, lens, float(torch.tensor(scale, dtype=torch.float32)), 0, 0)
    within(got[:, None], want, bound)


def test_attention_one_strong_token_among_many(rn):
    # a first token 20 above the rest: the others' small weights still add up
    L, D = 20000, 64
    t = ref.random_cache(L // 16, 1, 16, D, 7, "cuda", spread=False)
    table = torch.arange(L // 16, dtype=torch.int32, device="cuda")[None]
    t["k"].zero_()
    t["k"][0, 0, 0] = 0x38  # 1.0
    t["k_scale"].fill_(1.0)
    t["v"].fill_(0x38)
    t["v"][0, 0, 0] = 0
    t["v_scale"].fill_(1.0)
    q = torch.full((1, 1, 1, D), 16.0 / D, dtype=torch.float16, device="cuda")
    lens = torch.tensor([L], dtype=torch.int32, device="cuda")
    got = rn.kv_cache_attention(q[:, 0], make_cache(rn, t), table, lens, scale=1.0)
    within(got[:, None], *ref.attend(q, t, table, lens, 1.0, 0, 0))
    assert float(got[0, 0, 0]) > 1e-3


@pytest.mark.parametrize("n", [1, 3])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("window,sinks", [(0, 0), (40, 3)])
@pytest.mark.parametrize("how", ["rows", "line", "many"])
def test_attention_masked_places_hold_anything(rn, n, D, window, sinks, how):
    # NaN codes and NaN, infinite or huge scales in every place that a query must not see
    L, page, Hk, Hq = 150, 16, 2, 8
    t = ref.random_cache(14, Hk, page, D, 7, "cuda", spread=False)
    table = ref.tables(1, 12, 14, 1, "cuda")
    lens = torch.tensor([L], dtype=torch.int32, device="cuda")
    q = rand((1, n, Hq, D), 3, torch.bfloat16).cuda()
    want, bound = ref.attend(q, t, table, lens, 1 / math.sqrt(D), window, sinks)
    row = table[0].tolist()
    for j in range(12 * page):
        low = L - n + 1 - window if window else 0  # first token that any query's window reaches
        if j >= L or (window and j < low and j >= sinks):
            t["k"][row[j // page], :, j % page] = 0x7F
            t["v"][row[j // page], :, j % page] = 0xFF
    for blk in range(12):
        unseen = all(j >= L or (window and j < L - n + 1 - window and j >= sinks)
                     for j in range(16 * blk, 16 * blk + 16))
        if unseen:
            t["k_scale"][row[blk]] = (math.nan, math.inf, 1e38)[blk % 3]
            t["v_scale"][row[blk]] = (math.inf, math.nan, 1e38)[blk % 3]
    table, times = spread_out(table, how, Hk)
    got = rn.kv_cache_attention(q.repeat(times, 1, 1, 1), make_cache(rn, t), table, lens.repeat(times),
                                window=window, sinks=sinks)
    within(got.reshape(times, *q.shape), want[None], bound[None])


@pytest.mark.parametrize("D", [64, 128, 256])
def test_attention_nan_reaches_the_queries_that_see_it(rn, D):
    # a NaN value of the last drafted token: the queries before it must not notice
    L, n = 50, 3
    t = ref.random_cache(4, 1, 16, D, 7, "cuda", spread=False)
    table = ref.tables(1, 4, 4, 1, "cuda")
    lens = torch.tensor([L], dtype=torch.int32, device="cuda")
    q = rand((1, n, 4, D), 3, torch.bfloat16).cuda()
    want, bound = ref.attend(q, t, table, lens, 1 / math.sqrt(D), 0, 0)
    t["v"][int(table[0, 3]), 0, L - 1 - 48, 5] = 0x7F
    got = rn.kv_cache_attention(q, make_cache(rn, t), table, lens)
    bad = got.isnan()
    assert bool(bad[0, n - 1, :, 5].all()) and int(bad.sum()) == 4
    ok = torch.ones_like(bad)
    ok[0, n - 1, :, 5] = False
    within(got[ok], want[ok], bound[ok])
    # and of a key: the query that sees it has no weights at all
    t["v"][int(table[0, 3]), 0, L - 1 - 48, 5] = 0
    t["k"][int(table[0, 3]), 0, L - 1 - 48, 7] = 0x7F
    got = rn.kv_cache_attention(q, make_cache(rn, t), table, lens)
    assert bool(got[0, n - 1].isnan().all()) and not bool(got[0, :n - 1].isnan().any())
    within(got[0, 0], want[0, 0], bound[0, 0])


def test_attention_bad_pages_are_left_out(rn):
    D = 128
    t = ref.random_cache(6, 2, 16, D, 7, "cuda", spread=False)
    table = torch.tensor([[3, -1, 6, 2], [1, 0, 4, 5], [-7, 99, 6, 6]], dtype=torch.int32, device="cuda")
    lens = torch.tensor([60, 200, 30], dtype=torch.int32, device="cuda")
    q = rand((3, 1, 4, D), 3, torch.bfloat16).cuda()
    got = rn.kv_cache_attention(q, make_cache(rn, t), table, lens)
    assert rn.rmsattn_read_status(clear=True) == rn.RMSATTN_BAD_PAGE
    within(got, *ref.attend(q, t, table, lens, 1 / math.sqrt(D), 0, 0))
    assert bool((got[2] == 0).all())


def test_attention_empty_batch_and_rows(rn):
    D = 64
    t = ref.random_cache(2, 1, 16, D, 7, "cuda")
    q = rand((3, 2, D), 3, torch.bfloat16).cuda()
    lens = torch.tensor([0, -4, 0], dtype=torch.int32, device="cuda")
    table = torch.full((3, 2), -1, dtype=torch.int32, device="cuda")
    assert bool((rn.kv_cache_attention(q, make_cache(rn, t), table, lens) == 0).all())
    none = rn.kv_cache_attention(q, make_cache(rn, t), table[:, :0], lens)  # no pages at all
    assert bool((none == 0).all())
    got = rn.kv_cache_attention(q[:0], make_cache(rn, t), table[:0], lens[:0])
    assert got.shape == (0, 2, D)


@pytest.mark.parametrize("n", [1, 2])
def test_attention_strided_queries_and_out(rn, n):
    B, Hq, Hk, D = 3, 4, 2, 64
    t = ref.random_cache(12, Hk, 16, D, 7, "cuda", spread=False)
    table = ref.tables(B, 4, 12, 1, "cuda")
    wide = torch.zeros((B, 9), dtype=torch.int32, device="cuda")
    wide[:, 2:6] = table
    lens = torch.tensor([60, 33, 7], dtype=torch.int32, device="cuda")
    row = rand((B * n, (Hq + 2 * Hk) * D), 3, torch.bfloat16).cuda()
    q = row[:, :Hq * D].unflatten(1, (Hq, D)).unflatten(0, (B, n))
    big = torch.full((B * n, Hq * D + 24), 7.0, dtype=torch.bfloat16, device="cuda")
    out = big[:, 8:8 + Hq * D].unflatten(1, (Hq, D)).unflatten(0, (B, n))
    if n == 1:
        q, out = q[:, 0], out[:, 0]
    got = rn.kv_cache_attention(q, make_cache(rn, t), wide[:, 2:6], lens, out=out)
    assert got is out
    want, bound = ref.attend(q.reshape(B, n, Hq, D), t, table, lens, 0.125, 0, 0)
    within(got.reshape(want.shape), want, bound)
    assert bool((big[:, :8] == 7).all()) and bool((big[:, 8 + Hq * D:] == 7).all())


@pytest.mark.parametrize("how", ["rows", "line", "many"])
def test_attention_gives_the_same_bits_every_time(rn, how):
    t = ref.random_cache(400, 2, 32, 128, 7, "cuda", spread=False)
    table, times = spread_out(ref.tables(3, 130, 400, 1, "cuda"), how, 2)
    lens = torch.tensor([4100, 1000, 3], dtype=torch.int32, device="cuda").repeat(times)
    q = rand((3, 8, 128), 3, torch.bfloat16).cuda().repeat(times, 1, 1)
    first = rn.kv_cache_attention(q, make_cache(rn, t), table, lens)
    for _ in range(5):
        assert torch.equal(rn.kv_cache_attention(q, make_cache(rn, t), table, lens), first)


def test_attention_offsets_past_32_bits(rn):
    # pages beyond 4 GB of codes
    H, D, page = 8, 256, 1024
    pages = (1 << 32) // (H * D * page) + 4
    codes = torch.zeros((pages, H, page, D), dtype=torch.uint8, device="cuda")
    t = {"k": codes, "v": codes, "k_scale": torch.ones((pages, H, page // 16), device="cuda"),
         "v_scale": torch.ones((pages, H, page // 16), device="cuda")}
    table = torch.tensor([[pages - 1, 0]], dtype=torch.int32, device="cuda")
    x = rand((30, H, D), 1, torch.bfloat16).cuda()
    lens, cu = torch.tensor([1010], dtype=torch.int32), torch.tensor([0, 30], dtype=torch.int32)
    cache = make_cache(rn, t)
    rn.kv_cache_append_(cache, x, x, table, lens.cuda(), cu.cuda())
    small = {k: v[[pages - 1, 0]].clone() for k, v in t.items()}
    zero = {"k": torch.zeros_like(small["k"]), "k_scale": torch.ones_like(small["k_scale"])}
    ref.check_append(zero, small, x, "k", torch.tensor([[0, 1]]), lens, cu)
    q = rand((1, 1, 8, D), 3, torch.bfloat16).cuda()
    total = torch.tensor([1040], dtype=torch.int32, device="cuda")
    got = rn.kv_cache_attention(q, cache, table, total, window=60)
    want, bound = ref.attend(q, small, torch.tensor([[0, 1]], dtype=torch.int32, device="cuda"), total,
                             1 / 16, 60, 0)
    within(got, want, bound)
    del codes, t, cache


@pytest.mark.parametrize("scale", [-0.3, 0.0, 1e-30])
@pytest.mark.parametrize("how", ["rows", "line"])
def test_attention_scale_of_any_sign(rn, scale, how):
    t = ref.random_cache(30, 2, 16, 128, 7, "cuda", spread=False)
    table = ref.tables(2, 14, 30, 1, "cuda")
    lens = torch.tensor([200, 37], dtype=torch.int32, device="cuda")
    q = rand((2, 2, 8, 128), 3, torch.bfloat16).cuda()
    want, bound = ref.attend(q, t, table, lens, float(torch.tensor(scale, dtype=torch.float32)), 0, 0)
    got = rn.kv_cache_attention(q, make_cache(rn, t), spread_out(table, how, 2)[0], lens, scale=scale)
    within(got, want, bound)


def test_attention_infinite_and_nan_queries_stay_in_their_row(rn):
    t = ref.random_cache(12, 1, 16, 64, 7, "cuda", spread=False)
    table = ref.tables(1, 12, 12, 1, "cuda")
    lens = torch.tensor([180], dtype=torch.int32, device="cuda")
    q = rand((1, 1, 8, 64), 3, torch.bfloat16).cuda()
    want, bound = ref.attend(q, t, table, lens, 0.125, 0, 0)
    q[0, 0, 2, 5], q[0, 0, 6, 7] = math.nan, math.inf
    got = rn.kv_cache_attention(q, make_cache(rn, t), table, lens)
    rest = [0, 1, 3, 4, 5, 7]
    assert bool(got[0, 0, [2, 6]].isnan().all())
    within(got[0, 0, rest], want[0, 0, rest], bound[0, 0, rest])


def test_attention_many_columns(rn):
    # 16 query heads a key head x 32 query tokens: 512 columns of a row
    t = ref.random_cache(10, 1, 16, 64, 7, "cuda", spread=False)
    table = ref.tables(1, 10, 10, 1, "cuda")
    lens = torch.tensor([150], dtype=torch.int32, device="cuda")
    q = rand((1, 32, 16, 64), 3, torch.bfloat16).cuda()
    got = rn.kv_cache_attention(q, make_cache(rn, t), table, lens, window=100, sinks=2)
    within(got, *ref.attend(q, t, table, lens, 0.125, 100, 2))


def test_attention_largest_page_and_no_pages(rn):
    t = ref.random_cache(1, 2, 65536, 64, 7, "cuda", spread=False)
    table = torch.zeros((1, 1), dtype=torch.int32, device="cuda")
    lens = torch.tensor([65500], dtype=torch.int32, device="cuda")
    q = rand((1, 1, 4, 64), 3, torch.bfloat16).cuda()
    got = rn.kv_cache_attention(q, make_cache(rn, t), table, lens, window=300, sinks=20)
    within(got, *ref.attend(q, t, table, lens, 0.125, 300, 20))
    none = rn.KVCache.empty(0, 2, 16, 64)
    assert bool((rn.kv_cache_attention(q, none, table, lens * 0) == 0).all())
    assert bool((rn.kv_cache_attention(q, none, table, lens * 0 + 5) == 0).all())
    assert rn.rmsattn_read_status(clear=True) == rn.RMSATTN_BAD_PAGE


def test_refused_calls_raise(rn):
    t = ref.random_cache(2, 1, 16, 64, 7, "cuda")
    cache = make_cache(rn, t)
    table = torch.zeros((1, 1), dtype=torch.int32, device="cuda")
    lens = torch.ones(1, dtype=torch.int32, device="cuda")
    flat = torch.zeros(4 * 64 + 8, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(rn.RmsnError) as e:  # not on a 16-byte boundary
        rn.kv_cache_attention(flat[1:257].view(1, 4, 64), cache, table, lens)
    assert e.value.status == rn.RMSN_EALIGN
    with pytest.raises(rn.RmsnError) as e:
        rn.kv_cache_attention(flat[:256].view(1, 4, 64), cache, table, lens, scale=math.inf)
    assert e.value.status == rn.RMSN_EINVAL
    with pytest.raises(rn.RmsnError) as e:  # one token on all rows
        rn.kv_cache_append_(cache, flat[:64].expand(3, 64), flat[:64].expand(3, 64), table.repeat(3, 1),
                            lens.repeat(3))
    assert e.value.status == rn.RMSN_EINVAL
    with pytest.raises(ValueError):
        rn.kv_cache_attention(flat[:256].view(1, 4, 64), cache, table.cpu(), lens)
    with pytest.raises(ValueError):
        rn.kv_cache_append_(cache, flat[:64].view(1, 64).cpu(), flat[:64].view(1, 64), table, lens)
    with pytest.raises(ValueError):
        rn.qk_norm_rope(flat[:256].view(4, 64), None, torch.zeros(4, dtype=torch.int32), rn.rope_table(64), head_dim=64)


# ---------------------------------------------------------------- the path together

def layer(rn, s, row, weight, residual, pdl=False):
    """One decode or drafted step of a layer's attention: qkv row in, normed
    hidden state out."""
    B, n, Hq, Hk, D = s["B"], s["n"], s["Hq"], s["Hk"], s["D"]
    q, k, v = row.split([Hq * D, Hk * D, Hk * D], 1)
    q, k = rn.qk_norm_rope(q, k, s["pos"], s["rope"], s["wq"], s["wk"], head_dim=D, eps=1e-6, pdl=pdl)
    rn.kv_cache_append_(s["cache"], k, v, s["table"], s["before"], s["cu"], pdl=pdl)
    o = rn.kv_cache_attention(q.view(B, n, Hq, D), s["cache"], s["table"], s["after"], window=s["window"],
                              sinks=s["sinks"], pdl=pdl)
    return rn.fused_add_rmsnorm(o.view(B * n, Hq * D), residual, weight, eps=1e-6, pdl=pdl)[:2]


def layer_state(rn, n, seed=1):
    B, Hq, Hk, D, page = 3, 8, 2, 128, 16
    g = torch.Generator().manual_seed(seed)
    s = dict(B=B, n=n, Hq=Hq, Hk=Hk, D=D, window=60, sinks=3)
    s["rope"] = rn.rope_table(D, sections=[16, 24, 24], device="cuda")
    before = torch.tensor([100, 0, 47], dtype=torch.int32)
    s["before"], s["after"] = before.cuda(), (before + n).cuda()
    s["cu"] = torch.arange(0, B * n + 1, n, dtype=torch.int32).cuda()
    s["pos"] = torch.randint(0, 500, (3, B * n), generator=g).to(torch.int32).cuda()
    s["wq"], s["wk"] = (rand((D,), i, torch.bfloat16).cuda() for i in (1, 2))
    s["t"] = ref.random_cache(30, Hk, page, D, 7, "cuda", spread=False)
    s["table"] = ref.tables(B, 8, 30, 1, "cuda")
    s["cache"] = make_cache(rn, s["t"])
    return s


@pytest.mark.parametrize("n", [1, 4])
@pytest.mark.parametrize("pdl", [False, True])
def test_the_path_of_a_layer(rn, n, pdl):
    s = layer_state(rn, n)
    T, Hq, Hk, D = s["B"] * n, s["Hq"], s["Hk"], s["D"]
    row = rand((T, (Hq + 2 * Hk) * D), 3, torch.bfloat16)
    weight, residual = rand((Hq * D,), 4, torch.bfloat16).cuda(), rand((T, Hq * D), 5, torch.bfloat16).cuda()
    before = copy_of(s["t"])
    y, res = layer(rn, s, row.cuda(), weight, residual, pdl)
    # each step against its own definition, on what the step before gave
    q, k, v = row.split([Hq * D, Hk * D, Hk * D], 1)
    rq, rk = rn.qk_norm_rope(q.cuda(), k.cuda(), s["pos"], s["rope"], s["wq"], s["wk"], head_dim=D, eps=1e-6)
    within(rq, *ref.rope(q, s["wq"].cpu(), s["rope"], s["pos"].cpu(), D, 1e-6, 0.0, False))
    within(rk, *ref.rope(k, s["wk"].cpu(), s["rope"], s["pos"].cpu(), D, 1e-6, 0.0, False))
    for side, x in (("k", rk), ("v", v)):
        ref.check_append(before, s["t"], x.reshape(T, Hk, D), side, s["table"].cpu(), s["before"].cpu(), s["cu"].cpu())
    qn = rq.view(s["B"], n, Hq, D)
    want, bound = ref.attend(qn, s["t"], s["table"], s["after"], 1 / math.sqrt(D), s["window"], s["sinks"])
    o = rn.kv_cache_attention(qn, s["cache"], s["table"], s["after"], window=s["window"], sinks=s["sinks"])
    within(o, want, bound)
    o2 = o.reshape(T, Hq * D)
    r = oracle.rmsnorm(o2.cpu(), residual.cpu(), weight.cpu(), None, eps=1e-6, in_dtype="bf16", out_dtype="bf16")
    assert torch.equal(res, o2 + residual)
    d = parity.ordered16(y.cpu().view(torch.int16).numpy().view("uint16")) - parity.ordered16(r["out"])
    assert abs(d).max() <= parity.BF16_ULP


def test_the_path_captured_and_replayed_on_new_inputs(rn):
    # one graph, replayed as lengths and rows change in place; eager calls in between
    n = 1
    s, e = layer_state(rn, n), layer_state(rn, n)
    T, Hq, Hk, D = s["B"] * n, s["Hq"], s["Hk"], s["D"]
    weight, residual = rand((Hq * D,), 4, torch.bfloat16).cuda(), rand((T, Hq * D), 5, torch.bfloat16).cuda()
    row = rand((T, (Hq + 2 * Hk) * D), 3, torch.bfloat16).cuda()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    warm = layer_state(rn, n)
    with torch.cuda.stream(side):
        layer(rn, warm, row, weight, residual)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y, res = layer(rn, s, row, weight, residual)
    for step in range(20):
        row.copy_(rand(row.shape, 10 + step, torch.bfloat16))
        graph.replay()
        y2, res2 = layer(rn, e, row, weight, residual)
        assert torch.equal(y, y2) and torch.equal(res, res2), step
        for x in (s, e):
            x["before"] += 1
            x["after"] += 1
            x["pos"] += 1
    for name in s["t"]:
        assert torch.equal(s["t"][name], e["t"][name])


def test_calls_on_two_streams_at_once(rn):
    # each stream with its own queries over one cache: workspaces and outputs do not meet
    t = ref.random_cache(700, 2, 16, 128, 7, "cuda", spread=False)
    cache = make_cache(rn, t)
    table = ref.tables(2, 340, 700, 1, "cuda")
    lens = torch.tensor([5400, 4000], dtype=torch.int32, device="cuda")
    qs = [rand((2, 8, 128), i, torch.bfloat16).cuda() for i in range(8)]
    want = [rn.kv_cache_attention(q, cache, table, lens) for q in qs]
    streams = [torch.cuda.Stream() for _ in range(4)]
    torch.cuda.synchronize()
    for _ in range(5):
        got = [rn.kv_cache_attention(q, cache, table, lens, stream=streams[i % 4]) for i, q in enumerate(qs)]
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b)


def test_stream_of_another_call_is_used(rn):
    # the call's work is ordered behind the given stream's, not the current one's
    D = 64
    s = torch.cuda.Stream()
    x = torch.zeros((64, 4 * D), dtype=torch.bfloat16, device="cuda")
    table = rn.rope_table(D, device="cuda")
    pos = torch.arange(64, dtype=torch.int32, device="cuda")
    want = rand((64, 4 * D), 2, torch.bfloat16)
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        for _ in range(50):
            x.copy_(want.cuda())
    out, _ = rn.qk_norm_rope(x, None, pos, table, head_dim=D, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    within(out, *ref.rope(want, None, table, pos.cpu()[None], D, None, 0.0, False))


@pytest.mark.parametrize("past", [2**62, 2**64, 2**64 + 5])
def test_attention_masks_wider_than_any_integer(rn, past):
    t = ref.random_cache(16, 2, 16, 64, 3, "cuda")
    cache, table = make_cache(rn, t), ref.tables(2, 8, 16, 4, "cuda")
    lens = torch.tensor([100, 7], dtype=torch.int32, device="cuda")
    q = rand((2, 4, 64), 5, torch.bfloat16).cuda()
    want = rn.kv_cache_attention(q, cache, table, lens)
    assert torch.equal(rn.kv_cache_attention(q, cache, table, lens, window=past), want)
    assert torch.equal(rn.kv_cache_attention(q, cache, table, lens, window=9, sinks=past), want)


FIRST = """
import torch
import residual_add_rmsnorm_vec_gb300 as rn
B, Hq, Hk, D, pages = 3, 8, 2, 128, {pages}
x = torch.randn((B, (Hq + 2 * Hk) * D), device="cuda").to(torch.bfloat16)
pos = torch.arange(B, dtype=torch.int32, device="cuda")
cache = rn.KVCache.empty(B * pages, Hk, 16, D)
for t in (cache.k, cache.v, cache.k_scale, cache.v_scale):
    t.zero_()
table = torch.arange(B * pages, dtype=torch.int32, device="cuda").view(B, pages)
before = torch.zeros(B, dtype=torch.int32, device="cuda")
rope = rn.rope_table(D)
def step():
    q, k, v = x.split([Hq * D, Hk * D, Hk * D], 1)
    q, k = rn.qk_norm_rope(q, k, pos, rope, head_dim=D, eps=1e-6)
    rn.kv_cache_append_(cache, k, v, table, before)
    return rn.kv_cache_attention(q.view(B, Hq, D), cache, table, before + 1)
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    got = step()
graph.replay()
torch.cuda.synchronize()
assert torch.equal(got, step())
v = x[:, (Hq + Hk) * D:].view(B, Hk, 1, D).expand(B, Hk, Hq // Hk, D).reshape(B, Hq, D).float()
# one token seen: its value, rounded to E4M3 (2^-4, or half of 2^-9 of the scale) and bf16 (2^-8); products below 2^-9
assert ((got.float() - v).abs() <= v.abs() * (2.0 ** -4 + 2.0 ** -7) + v.abs().amax() * 2.0 ** -18).all()
"""


@pytest.mark.parametrize("pages", [4, 4096])
def test_the_first_call_of_a_process_may_be_captured(rn, pages):
    # clusters (4 pages) and the line with its workspace (4096)
    r = subprocess.run([sys.executable, "-c", FIRST.format(pages=pages)], capture_output=True, text=True,
                       timeout=300, cwd=os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
    assert r.returncode == 0, r.stderr[-2000:]
