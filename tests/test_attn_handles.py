"""CPU tests of what a KVCache and a RopeTable keep beside their tensors: it
cannot fall out of step with them."""
import copy
import pickle

import pytest
import torch


@pytest.fixture(scope="module")
def rn():
    from residual_add_rmsnorm_vec_gb300 import build

    build.build()
    import residual_add_rmsnorm_vec_gb300 as p

    return p


def tensors(pages=4):
    return [torch.zeros((pages, 2, 32, 64), dtype=torch.uint8), torch.zeros((pages, 2, 32, 64), dtype=torch.uint8),
            torch.zeros((pages, 2, 2)), torch.zeros((pages, 2, 2))]


def described(cache):
    """Addresses and strides that the C ABI is given."""
    cache._current()
    c = cache._c
    return (c.k, c.v, c.k_scale, c.v_scale), c.page_stride, c.scale_stride


@pytest.mark.parametrize("name", ["k", "v", "k_scale", "v_scale", "n_pages", "n_kv_heads", "page_size", "head_dim",
                                  "device", "index"])
def test_a_cache_keeps_the_tensors_that_it_describes(rn, name):
    # the addresses were those of the first tensors: another one in their place left the old address
    # behind, of memory that may be freed
    cache = rn.KVCache(*tensors())
    was = getattr(cache, name)
    with pytest.raises(AttributeError):
        setattr(cache, name, tensors()[0])
    with pytest.raises(AttributeError):
        delattr(cache, name)
    assert getattr(cache, name) is was


@pytest.mark.parametrize("name", ["turns", "axis", "rot_dim", "n_axes", "index"])
def test_a_rope_table_keeps_its_tensors(rn, name):
    table = rn.rope_table(64, sections=[8, 12, 12], device="cpu")
    was = getattr(table, name)
    with pytest.raises(AttributeError):
        setattr(table, name, torch.zeros(1, dtype=torch.int32))
    assert getattr(table, name) is was


@pytest.mark.parametrize("i", range(4))
@pytest.mark.parametrize("how", ["data", "set", "storage"])
def test_a_tensor_given_other_memory_is_found_again(rn, i, how):
    t = tensors()
    cache = rn.KVCache(*t)
    old = t[i].data_ptr()
    keep = t[i].detach().clone()  # neither address is handed out again meanwhile
    other = torch.zeros_like(keep)
    if how == "data":
        t[i].data = other
    elif how == "set":
        t[i].set_(other)
    else:
        t[i].untyped_storage().resize_(1 << 24)
    assert t[i].data_ptr() != old
    assert described(cache)[0] == tuple(x.data_ptr() for x in t)


def test_a_tensor_that_changed_its_form_is_refused(rn):
    for change in (lambda t: t[0].set_(torch.zeros((3, 2, 32, 64), dtype=torch.uint8)),
                   lambda t: setattr(t[2], "data", torch.zeros((4, 2, 2), dtype=torch.float64)),
                   lambda t: t[1].untyped_storage().resize_(0),
                   lambda t: t[3].set_(torch.zeros((4, 2, 4))[:, :, ::2])):
        t = tensors()
        cache = rn.KVCache(*t)
        change(t)
        with pytest.raises((ValueError, TypeError)):
            cache._current()
    # all four alike, but fewer pages than the cache was made for
    t = tensors()
    cache = rn.KVCache(*t)
    for x, y in zip(t, tensors(3)):
        x.set_(y)
    with pytest.raises(ValueError):
        cache._current()


def test_a_tensor_larger_than_its_storage_is_refused(rn):
    t = tensors()
    t[0].untyped_storage().resize_(100)
    with pytest.raises(ValueError):
        rn.KVCache(*t)


def test_a_rope_table_whose_tensor_changed_is_refused(rn):
    for name, other in (("turns", torch.zeros(31, dtype=torch.int64)), ("axis", torch.zeros(32, dtype=torch.int64))):
        table = rn.rope_table(64, device="cpu")
        getattr(table, name).data = other
        with pytest.raises((ValueError, TypeError)):
            table._pointers()


def test_copies(rn):
    cache = rn.KVCache(*tensors())
    near = copy.copy(cache)
    assert near.k is cache.k and described(near) == described(cache)
    far = pickle.loads(pickle.dumps(cache))
    assert far.k.data_ptr() != cache.k.data_ptr() and described(far)[0][0] == far.k.data_ptr()
    table = rn.rope_table(64, sections=[8, 12, 12], device="cpu")
    far = copy.deepcopy(table)
    assert torch.equal(far.turns, table.turns) and far.n_axes == 3


def test_a_subclass_has_attributes_of_its_own(rn):
    class Named(rn.KVCache):
        def __init__(self, *tensors):
            super().__init__(*tensors)
            self.name = "layer 3"

    cache = Named(*tensors())
    cache.name = "layer 4"
    del cache.name
    with pytest.raises(AttributeError):
        cache.k = cache.v
    with pytest.raises(AttributeError):
        rn.KVCache(*tensors()).name = "a slot that is not there"
    assert type(copy.copy(cache)) is Named
