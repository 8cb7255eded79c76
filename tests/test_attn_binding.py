"""CPU checks of the attention-path library and its binding: exported symbols,
refusals of bad arguments before anything is launched, and the rotary table.
No call here reaches a kernel."""
import ctypes
import math
import os
import re
import subprocess

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def rn():
    from residual_add_rmsnorm_vec_gb300 import build

    build.build()
    import residual_add_rmsnorm_vec_gb300 as p

    return p


def declared():
    src = open(os.path.join(ROOT, "include", "rmsnorm_attn.h")).read()
    src = re.sub(r"/\*.*?\*/", "", src, flags=re.S)
    return sorted(set(re.findall(r"^\s*\w+\s*\*?\s*(rmsattn_\w+)\s*\(", src, re.M)))


def test_library_exports_what_the_header_declares(rn):
    out = subprocess.run(["nm", "-D", "--defined-only", rn.attn_library_path()], capture_output=True,
                         text=True, check=True).stdout
    ours = [l.split()[-1] for l in out.splitlines() if " T " in l]
    assert sorted(s for s in ours if not s.startswith("_")) == declared()
    assert sorted(rn.EXPORTED_ATTN) == declared()


# ---------------------------------------------------------------- C ABI

BF16, F32, F16 = 1, 0, 2
NORM, INTER, I64 = 0x1000, 0x2000, 0x4000


def rope_call(rn, **kw):
    a = dict(q=16, k=16, qw=None, kw=None, qo=32, ko=32, pos=16, ps=4, turns=16, axis=16, T=4, hq=2, hk=1,
             D=64, R=64, axes=1, qs=128, ks=64, qos=128, kos=64, eps=1e-6, woff=0.0, flags=BF16)
    a.update(kw)
    return rn.load_attn().rmsattn_qk_rope_fwd(*a.values(), None)


@pytest.mark.parametrize("kw,status", [
    (dict(flags=3), -1), (dict(flags=BF16 | 4), -1), (dict(flags=BF16 | 0x8000), -1),
    (dict(T=-1), -1), (dict(D=0, R=0), -1), (dict(D=4098, qs=8196, ks=4098, qos=8196, kos=4098), -1),
    (dict(R=63), -1), (dict(R=66), -1), (dict(R=-2), -1), (dict(axes=0), -1), (dict(axes=65), -1),
    (dict(hq=-1), -1), (dict(qs=127), -1), (dict(kos=63), -1), (dict(eps=-1.0), -1),
    (dict(eps=math.nan), -1), (dict(woff=math.inf), -1), (dict(axes=2, ps=3), -1),
    (dict(q=None), -1), (dict(ko=None), -1), (dict(pos=None), -1), (dict(turns=None), -1),
    (dict(axis=None), -1), (dict(q=17), -2), (dict(qw=17, flags=BF16 | NORM), -2), (dict(pos=18), -2),
    (dict(pos=20, flags=BF16 | I64), -2), (dict(turns=20), -2), (dict(flags=F32, ko=18), -2),
    (dict(T=1 << 60), -1),
    (dict(T=0, q=None, k=None, pos=None), 0), (dict(hq=0, hk=0, q=None), 0),
])
def test_rope_refusals(rn, kw, status):
    assert rope_call(rn, **kw) == status


def cache_struct(rn, **kw):
    a = dict(k=16, v=16, k_scale=16, v_scale=16, n_pages=4, page_stride=2 * 32 * 64, scale_stride=4,
             n_kv_heads=2, page_size=32, head_dim=64, reserved=0)
    a.update(kw)
    from residual_add_rmsnorm_vec_gb300._attn_lib import RmsattnCache
    return RmsattnCache(*a.values())


CACHE_BAD = [
    (dict(reserved=1), -1), (dict(n_pages=-1), -1), (dict(n_kv_heads=0), -1), (dict(page_size=24), -1),
    (dict(page_size=0), -1), (dict(page_size=65552), -1), (dict(head_dim=96), -3),
    (dict(page_stride=4095), -1), (dict(page_stride=4104), -1), (dict(scale_stride=3), -1),
    (dict(k=None), -1), (dict(v_scale=None), -1), (dict(scale_stride=1 << 30), -3), (dict(k=8), -2), (dict(k_scale=18), -2),
]


@pytest.mark.parametrize("kw,status", CACHE_BAD + [
    (dict(flags=4 | BF16), -1), (dict(flags=3), -1), (dict(T=-1), -1), (dict(ks=127), -1),
    (dict(vs=0), -1), (dict(cu=None, T=5), -1), (dict(ts=1), -1), (dict(table=None), -1),
    (dict(lengths=None), -1), (dict(kp=None), -1), (dict(kp=17), -2), (dict(lengths=18), -2),
    (dict(cu=18), -2), (dict(width=1 << 26, ts=1 << 26), -1), (dict(T=0, kp=None, vp=None), 0),
    (dict(B=0, T=0, lengths=None), 0),
])
def test_append_refusals(rn, kw, status):
    a = dict(kp=16, vp=16, ks=128, vs=128, table=16, ts=2, width=2, lengths=16, cu=16, T=4, B=3, flags=BF16)
    c = {k: kw[k] for k in kw if k not in a}
    a.update({k: kw[k] for k in kw if k in a})
    assert rn.load_attn().rmsattn_kv_append(ctypes.byref(cache_struct(rn, **c)), *a.values(), None) == status


@pytest.mark.parametrize("kw,status", CACHE_BAD + [
    (dict(flags=F32), -3), (dict(flags=3), -1), (dict(flags=BF16 | 8), -1), (dict(n=0), -1), (dict(n=33), -1),
    (dict(hq=3), -1), (dict(hq=0), -1), (dict(B=-1), -1), (dict(scale=math.nan), -1),
    (dict(scale=math.inf), -1), (dict(window=-1), -1), (dict(sinks=-1), -1), (dict(qs=255), -1),
    (dict(qs=260), -1), (dict(os=252), -1), (dict(ts=1), -1), (dict(q=None), -1), (dict(out=None), -1),
    (dict(lengths=None), -1), (dict(q=24), -2), (dict(out=8), -2), (dict(lengths=18), -2),
    (dict(B=0, q=None, out=None), 0),
])
def test_attention_refusals(rn, kw, status):
    a = dict(q=16, cache=None, table=16, ts=2, width=2, lengths=16, out=16, qs=256, os=256, B=3, n=1, hq=4,
             scale=0.125, window=0, sinks=0, ws=16, wsb=1 << 40, flags=BF16)
    c = {k: kw[k] for k in kw if k not in a}
    a.update({k: kw[k] for k in kw if k in a})
    a["cache"] = ctypes.byref(cache_struct(rn, **c))
    assert rn.load_attn().rmsattn_kv_attention(*a.values(), None) == status


def test_null_cache_refused(rn):
    lib = rn.load_attn()
    assert lib.rmsattn_kv_append(None, 16, 16, 128, 128, 16, 2, 2, 16, 16, 4, 3, BF16, None) == -1
    assert lib.rmsattn_kv_attention(16, None, 16, 2, 2, 16, 16, 256, 256, 3, 1, 4, 0.1, 0, 0, 16, 1 << 40,
                                    BF16, None) == -1


@pytest.mark.parametrize("sizes,status", [
    ((3, 0, 4, 2, 64, 64, 0, 0), -1), ((3, 33, 4, 2, 64, 64, 0, 0), -1), ((-1, 1, 4, 2, 64, 64, 0, 0), -1),
    ((3, 1, 5, 2, 64, 64, 0, 0), -1), ((3, 1, 4, 0, 64, 64, 0, 0), -1), ((3, 1, 4, 2, 96, 64, 0, 0), -3),
    ((3, 1, 4, 2, 64, -1, 0, 0), -1), ((3, 1, 4, 2, 64, 1 << 40, 0, 0), -1), ((0, 1, 4, 2, 64, 64, 0, 0), 0),
    ((3, 1, 4, 2, 64, 64, -1, 0), -1), ((3, 1, 4, 2, 64, 64, 0, -1), -1),
])
def test_workspace_refusals(rn, sizes, status):
    assert rn.load_attn().rmsattn_kv_attention_workspace(*sizes) == status


# ---------------------------------------------------------------- tensor level

def test_rope_table(rn):
    t = rn.rope_table(8, base=100.0, sections=[1, 2, 1], device="cpu")
    assert (t.rot_dim, t.n_axes, t.axis.tolist()) == (8, 3, [0, 1, 1, 2])
    for p, b in enumerate(t.turns.tolist()):
        assert abs((b % 2**64) / 2.0**64 * 2 * math.pi - 100.0 ** (-p / 4)) < 2.0 ** -52
    t = rn.rope_table(4, inv_freq=[-0.5, 7.0], axis=[1, 0], device="cpu")
    assert t.n_axes == 2
    f = [(b % 2**64) / 2.0**64 * 2 * math.pi for b in t.turns.tolist()]
    assert abs(f[0] - (2 * math.pi - 0.5)) < 1e-15 and abs(f[1] - (7.0 - 2 * math.pi)) < 1e-15
    assert rn.rope_table(0, device="cpu").rot_dim == 0
    for bad in (dict(rot_dim=7), dict(rot_dim=-2), dict(rot_dim=8, sections=[1, 2]),
                dict(rot_dim=8, sections=[5, -1]), dict(rot_dim=8, axis=[0, 0, 0]),
                dict(rot_dim=8, axis=[0, 0, 0, -1]), dict(rot_dim=8, inv_freq=[1.0]),
                dict(rot_dim=4, inv_freq=[1.0, math.inf]), dict(rot_dim=4, base=0.0),
                dict(rot_dim=4, sections=[2], axis=[0, 0])):
        with pytest.raises(ValueError):
            rn.rope_table(device="cpu", **bad)


def z(*shape, dtype=torch.bfloat16):
    return torch.zeros(shape, dtype=dtype)


@pytest.mark.parametrize("kw,err", [
    (dict(q=z(4, 100)), ValueError), (dict(q=z(4, 2, 32)), ValueError), (dict(q=z(256, 4).t()), ValueError),
    (dict(q=z(4)), ValueError), (dict(k=z(3, 64)), ValueError), (dict(k=z(4, 64, dtype=torch.float32)), ValueError),
    (dict(q=z(4, 128, dtype=torch.int32), k=None), TypeError), (dict(positions=z(5, dtype=torch.int32)), ValueError),
    (dict(positions=z(2, 4, dtype=torch.int32)), ValueError), (dict(positions=z(4)), TypeError),
    (dict(positions=z(8, dtype=torch.int32)[::2]), ValueError), (dict(rot=128), ValueError),
    (dict(head_dim=0), ValueError), (dict(), ValueError),  # host tensors
])
def test_rope_arguments(rn, kw, err):
    a = dict(q=z(4, 128), k=z(4, 64), positions=z(4, dtype=torch.int32), head_dim=64, rot=64)
    a.update(kw)
    table = rn.rope_table(a.pop("rot"), device="cpu")
    with pytest.raises(err):
        rn.qk_norm_rope(a.pop("q"), a.pop("k"), a.pop("positions"), table, **a)


def host_cache(rn, **kw):
    a = dict(k=z(4, 2, 32, 64, dtype=torch.uint8), v=z(4, 2, 32, 64, dtype=torch.uint8),
             k_scale=z(4, 2, 2, dtype=torch.float32), v_scale=z(4, 2, 2, dtype=torch.float32))
    a.update(kw)
    return rn.KVCache(**a)


@pytest.mark.parametrize("kw,err", [
    (dict(k=z(2, 32, 64, dtype=torch.uint8)), ValueError), (dict(v=z(3, 2, 32, 64, dtype=torch.uint8)), ValueError),
    (dict(k=z(4, 2, 32, 64, dtype=torch.int16)), TypeError), (dict(k_scale=z(4, 2, 1, dtype=torch.float32)), ValueError),
    (dict(v_scale=z(4, 2, 2)), TypeError), (dict(k=z(4, 2, 24, 64, dtype=torch.uint8)), ValueError),
    (dict(k=z(4, 32, 2, 64, dtype=torch.uint8).transpose(1, 2)), ValueError),
    (dict(v=z(4, 4, 32, 64, dtype=torch.uint8)[:, :2]), ValueError),  # another page stride than k
])
def test_cache_arguments(rn, kw, err):
    with pytest.raises(err):
        host_cache(rn, **kw)
    assert host_cache(rn).page_size == 32


@pytest.mark.parametrize("heads,dim", [(0, 64), (2, 0), (0, 0)])
def test_cache_without_heads_or_dims_refused(rn, heads, dim):
    # nothing divides by either once a cache exists
    codes, scales = z(4, heads, 32, dim, dtype=torch.uint8), z(4, heads, 2, dtype=torch.float32)
    with pytest.raises(ValueError, match="heads"):
        rn.KVCache(codes, codes.clone(), scales, scales.clone())
    with pytest.raises(ValueError, match="heads"):
        rn.KVCache.empty(4, heads, 32, dim, device="cpu")


I32 = torch.int32


@pytest.mark.parametrize("kw,err", [
    (dict(k=z(5, 1, 64)), ValueError), (dict(k=z(5, 3, 64)), ValueError), (dict(v=z(4, 2, 64)), ValueError),
    (dict(v=z(5, 2, 64, dtype=torch.float16)), ValueError), (dict(k=z(5, 2, 32)), ValueError),
    (dict(k=z(5, 2, 64, dtype=torch.float64), v=z(5, 2, 64, dtype=torch.float64)), TypeError),
    (dict(lengths=z(3, dtype=torch.int64)), TypeError), (dict(block_table=z(2, 2, dtype=I32)), ValueError),
    (dict(block_table=z(2, 3, dtype=I32).t()), ValueError), (dict(cu_seqlens=z(3, dtype=I32)), ValueError),
    (dict(cu_seqlens=z(4, dtype=torch.int64)), TypeError), (dict(cu_seqlens=None), ValueError),
    (dict(lengths=z(1, 3, dtype=I32)), ValueError), (dict(), ValueError),  # host tensors
])
def test_append_arguments(rn, kw, err):
    a = dict(k=z(5, 2, 64), v=z(5, 2, 64), block_table=z(3, 2, dtype=I32), lengths=z(3, dtype=I32),
             cu_seqlens=z(4, dtype=I32))
    a.update(kw)
    with pytest.raises(err):
        rn.kv_cache_append_(host_cache(rn), **a)


@pytest.mark.parametrize("kw,err", [
    (dict(q=z(3, 4 * 64)), ValueError), (dict(q=z(3, 3, 64)), ValueError), (dict(q=z(3, 4, 128)), ValueError),
    (dict(q=z(3, 33, 4, 64)), ValueError), (dict(q=z(3, 4, 64, dtype=torch.float32)), TypeError),
    (dict(window=-1), ValueError), (dict(sinks=-1), ValueError), (dict(lengths=z(2, dtype=I32)), ValueError),
    (dict(block_table=z(3, 2, dtype=torch.int64)), TypeError), (dict(), ValueError),  # host tensors
])
def test_attention_arguments(rn, kw, err):
    a = dict(q=z(3, 4, 64), block_table=z(3, 2, dtype=I32), lengths=z(3, dtype=I32))
    a.update(kw)
    with pytest.raises(err):
        rn.kv_cache_attention(a.pop("q"), host_cache(rn), **a)
