"""CPU checks of the operators around the attention in a serving step: refusals of
bad arguments before anything is launched.  No call here reaches a kernel."""
import ctypes
import math

import pytest
import torch

from test_attn_binding import BF16, CACHE_BAD, F32, cache_struct, rn  # noqa: F401  (rn: a fixture)

F16, R32, FP8, PDL = 2, 0x200, 0x8000, 0x80
OK, EINVAL, EALIGN, EUNSUPPORTED = 0, -1, -2, -3


@pytest.mark.parametrize("kw,status", [
    (dict(flags=1), EINVAL), (dict(pages=-1), EINVAL), (dict(pages=1 << 31), EINVAL), (dict(B=-1), EINVAL),
    (dict(B=(1 << 24) + 1), EINVAL), (dict(T=-1), EINVAL), (dict(T=(1 << 29) + 1), EINVAL), (dict(page=0), EINVAL),
    (dict(page=24), EINVAL), (dict(page=65552), EINVAL), (dict(ts=1), EINVAL), (dict(width=-1), EINVAL),
    (dict(width=1 << 26, ts=1 << 26), EINVAL), (dict(table=None), EINVAL), (dict(free=None), EINVAL),
    (dict(n_free=None), EINVAL), (dict(lengths=None), EINVAL), (dict(new=None), EINVAL), (dict(cu=None), EINVAL),
    (dict(pos=None), EINVAL), (dict(slots=None), EINVAL), (dict(rows=None), EINVAL), (dict(before=None), EINVAL),
    (dict(after=None), EINVAL), (dict(out=None), EINVAL), (dict(out=32), EINVAL), (dict(after=80), EINVAL),
    (dict(before=80), EINVAL), (dict(before=96), EINVAL), (dict(after=96), EINVAL),
    (dict(B=5000, ws=None), EINVAL), (dict(B=5000, ws=16, wsb=60000), EINVAL),
    (dict(free=18), EALIGN), (dict(lengths=18), EALIGN), (dict(shared=18), EALIGN), (dict(pos=20), EALIGN),
    (dict(slots=24), EALIGN), (dict(rows=8), EALIGN), (dict(B=5000, ws=8, wsb=1 << 20), EALIGN),
])
def test_pages_refusals(rn, kw, status):  # noqa: F811
    a = dict(free=16, pages=8, n_free=32, table=64, ts=2, width=2, lengths=80, new=96, shared=None, B=3, page=16, T=4,
             cu=112, pos=128, slots=144, rows=160, before=176, after=192, out=208, ws=None, wsb=0, flags=0)
    a.update(kw)
    assert rn.load_attn().rmsattn_pages_step(*a.values(), None) == status


@pytest.mark.parametrize("n,want", [(-1, EINVAL), ((1 << 24) + 1, EINVAL), (0, 0), (2048, 0), (2049, (4 + 3 * 2050) * 4)])
def test_pages_workspace(rn, n, want):  # noqa: F811
    assert rn.load_attn().rmsattn_pages_workspace(n) == want


@pytest.mark.parametrize("kw,status", [
    (dict(flags=3), EINVAL), (dict(flags=BF16 | 4), EINVAL), (dict(flags=F32 | R32), EINVAL), (dict(T=-1), EINVAL),
    (dict(H=0), EINVAL), (dict(H=(1 << 24) + 1), EINVAL), (dict(T=1 << 31), EINVAL), (dict(eps=-1.0), EINVAL),
    (dict(eps=math.nan), EINVAL), (dict(alpha=math.inf), EINVAL), (dict(off=math.nan), EINVAL),
    (dict(gs=64), EINVAL), (dict(n_gates=1), EINVAL), (dict(index=16), EINVAL),
    (dict(gate=16, gs=63, n_gates=4), EINVAL), (dict(gate=16, gs=-64, n_gates=4), EINVAL),
    (dict(gate=16, gs=64, n_gates=3), EINVAL), (dict(gate=16, gs=0, n_gates=4), EINVAL),
    (dict(gate=16, gs=64, n_gates=-1, index=16), EINVAL), (dict(gate=16, gs=64, n_gates=1 << 60, index=16), EINVAL),
    (dict(scale=16), EINVAL), (dict(flags=BF16 | FP8), EINVAL), (dict(x=None), EINVAL), (dict(residual=None), EINVAL),
    (dict(out=None), EINVAL), (dict(ro=None), EINVAL), (dict(x=17), EALIGN), (dict(ro=17), EALIGN),
    (dict(flags=BF16 | R32, residual=18), EALIGN), (dict(flags=BF16 | FP8, scale=18), EALIGN),
    (dict(gate=17, n_gates=1), EALIGN), (dict(gate=16, gs=64, n_gates=9, index=18), EALIGN), (dict(w=17), EALIGN),
    (dict(T=0, x=None, residual=None, out=None, ro=None), OK),
])
def test_norms_refusals(rn, kw, status):  # noqa: F811
    a = dict(x=16, residual=16, post=16, w=16, gate=None, gs=0, index=None, n_gates=0, out=16, ro=16, scale=None,
             T=4, H=64, eps=1e-6, alpha=1.0, off=0.0, flags=BF16)
    a.update(kw)
    assert rn.load_attn().rmsattn_block_norms(*a.values(), None) == status


@pytest.mark.parametrize("kw,status", CACHE_BAD + [
    (dict(flags=F32), EUNSUPPORTED), (dict(flags=3), EINVAL), (dict(flags=BF16 | 8), EINVAL), (dict(n=0), EINVAL),
    (dict(n=33), EINVAL), (dict(hq=3), EINVAL), (dict(B=-1), EINVAL), (dict(groups=-1), EINVAL),
    (dict(groups=(1 << 24) + 1), EINVAL), (dict(cu=None), EINVAL), (dict(scale=math.nan), EINVAL),
    (dict(qs=255), EINVAL), (dict(os=252), EINVAL), (dict(ts=1), EINVAL), (dict(q=None), EINVAL),
    (dict(out=None), EINVAL), (dict(lengths=None), EINVAL), (dict(prefix=None), EINVAL), (dict(ws=None), EINVAL),
    (dict(q=24), EALIGN), (dict(out=8), EALIGN), (dict(lengths=18), EALIGN), (dict(prefix=18), EALIGN),
    (dict(cu=18), EALIGN), (dict(ws=16), EALIGN), (dict(B=0, q=None, out=None, ws=None), OK),
])
def test_prefix_refusals(rn, kw, status):  # noqa: F811
    a = dict(q=16, cache=None, table=16, ts=2, width=2, lengths=16, prefix=16, cu=16, groups=2, out=16, qs=256, os=256,
             B=3, n=1, hq=4, scale=0.125, ws=32, wsb=1 << 40, flags=BF16)
    c = {k: kw[k] for k in kw if k not in a}
    a.update({k: kw[k] for k in kw if k in a})
    a["cache"] = ctypes.byref(cache_struct(rn, **c))
    assert rn.load_attn().rmsattn_kv_prefix_attention(*a.values(), None) == status


@pytest.mark.parametrize("sizes,status", [
    ((3, 0, 4, 2, 64, 64, 1), EINVAL), ((3, 33, 4, 2, 64, 64, 1), EINVAL), ((-1, 1, 4, 2, 64, 64, 1), EINVAL),
    ((3, 1, 5, 2, 64, 64, 1), EINVAL), ((3, 1, 4, 2, 96, 64, 1), EUNSUPPORTED), ((3, 1, 4, 2, 64, -1, 1), EINVAL),
    ((3, 1, 4, 2, 64, 1 << 40, 1), EINVAL), ((3, 1, 4, 2, 64, 64, -1), EINVAL), ((0, 1, 4, 2, 64, 64, 1), 0),
])
def test_prefix_workspace_refusals(rn, sizes, status):  # noqa: F811
    assert rn.load_attn().rmsattn_kv_prefix_attention_workspace(*sizes) == status


# ---------------------------------------------------------------- tensors


def ints(*shape):
    return torch.zeros(shape, dtype=torch.int32)


@pytest.mark.parametrize("change", [
    dict(free_pages=ints(2, 4)), dict(free_pages=ints(8).long()), dict(n_free=ints(2)), dict(block_table=ints(4, 2)),
    dict(block_table=ints(3, 2).long()), dict(block_table=ints(3)), dict(lengths=ints(2)), dict(lengths=ints(1, 3)),
    dict(new_tokens=ints(3).float()), dict(shared_pages=ints(4)), dict(page_size=8), dict(page_size=40), dict(n_rows=-1), dict(n_rows=(1 << 29) + 1),
    dict(lengths=ints(6)[::2]), dict(block_table=ints(2, 3).t()),
    dict(),  # all of it right, but on the CPU
])
def test_pages_tensors_refused(rn, change):  # noqa: F811
    a = dict(free_pages=ints(8), n_free=ints(1), block_table=ints(3, 2), lengths=ints(3), new_tokens=ints(3),
             shared_pages=None, page_size=16, n_rows=4)
    a.update(change)
    with pytest.raises((ValueError, TypeError)):
        rn.kv_pages_step_(**a)


def test_free_pages(rn):  # noqa: F811
    free, n = rn.kv_free_pages(4, device="cpu")
    assert free.tolist() == [3, 2, 1, 0] and n.tolist() == [4]
    with pytest.raises(ValueError):
        rn.kv_free_pages(-1, device="cpu")


B16 = torch.bfloat16


@pytest.mark.parametrize("change", [
    dict(x=torch.zeros(4)), dict(x=torch.zeros(4, 8, dtype=torch.int32)), dict(residual=None), dict(out_dtype="fp4"),
    dict(out_dtype="f32"), dict(),
])
def test_norms_tensors_refused(rn, change):  # noqa: F811
    a = dict(x=torch.zeros(4, 8, dtype=B16), residual=torch.zeros(4, 8, dtype=B16), eps=1e-6)
    a.update(change)
    with pytest.raises((ValueError, TypeError)):
        rn.fused_block_norms(**a)


@pytest.mark.parametrize("change", [
    dict(q=torch.zeros(3, 256, dtype=B16)), dict(q=torch.zeros(3, 3, 64, dtype=B16)), dict(q=torch.zeros(3, 4, 64)),
    dict(q=torch.zeros(3, 33, 4, 64, dtype=B16)), dict(lengths=ints(2)), dict(block_table=ints(2, 2)),
    dict(prefix_lengths=ints(1, 1)), dict(prefix_lengths=ints(2)), dict(groups=ints(3)), dict(),
])
def test_prefix_tensors_refused(rn, change):  # noqa: F811
    cache = rn.KVCache.empty(4, 2, 16, 64, device="cpu")
    a = dict(q=torch.zeros(3, 4, 64, dtype=B16), cache=cache, block_table=ints(3, 2), lengths=ints(3),
             prefix_lengths=ints(1))
    a.update(change)
    with pytest.raises((ValueError, TypeError)):
        rn.kv_cache_prefix_attention(**a)


def test_norms_outputs_lie_apart(rn):  # noqa: F811
    for flags, out, ro in ((BF16, 32, 32), (F32, 32, 32), (BF16 | FP8, 64, 64)):
        assert rn.load_attn().rmsattn_block_norms(
            32, 64, None, None, None, 0, None, 0, out, ro, 16 if flags & FP8 else None, 4, 64, 1e-6, 1.0, 0.0, flags,
            None) == EINVAL


def test_status_bits(rn):  # noqa: F811
    assert (rn.RMSATTN_WAIT_RAN_OUT, rn.RMSATTN_BAD_PAGE) == (1, 4)


def test_prefix_of_more_columns_than_are_counted(rn):  # noqa: F811
    # sequences x query tokens x heads of a key head past 31 bits
    lib = rn.load_attn()
    assert lib.rmsattn_kv_prefix_attention_workspace(1 << 24, 32, 4, 1, 64, 64, 1) == EUNSUPPORTED
