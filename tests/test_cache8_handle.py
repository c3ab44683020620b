"""A KvCache8 stands for the tensors that it holds: copies have their own, and tensors whose memory has been
exchanged are refused (no compute calls here)."""
import copy
import ctypes
import io

import pytest

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def sa2():
    from block_sparse_attention_sa2_gb300 import build_lib
    if not build_lib.up_to_date():
        build_lib.build()
    import block_sparse_attention_sa2_gb300 as m
    return m


def pointers(c):
    """The four device pointers of the sa2_cache8 that calls are made with."""
    return list((ctypes.c_uint64 * 4).from_buffer_copy(c._struct[:32]))


def tensors(c):
    return [x.data_ptr() for x in (c.k, c.v, c.k_scale, c.v_scale)]


def filled(sa2):
    c = sa2.KvCache8.empty(2, 3, 130, 64, "cpu")
    for i, x in enumerate((c.k, c.v)):
        x.view(torch.uint8).fill_(i + 1)
    c.k_scale.fill_(1), c.v_scale.fill_(2)
    return c


def saved(c):
    f = io.BytesIO()
    torch.save(c, f)
    f.seek(0)
    return torch.load(f, weights_only=False)


@pytest.mark.parametrize("how", [copy.deepcopy, saved])
def test_a_copy_has_its_own_memory(sa2, how):
    c = filled(sa2)
    d = how(c)
    assert pointers(c) == tensors(c) and pointers(d) == tensors(d)
    assert not set(pointers(c)) & set(pointers(d))
    assert d.shape == c.shape and torch.equal(d.k.view(torch.uint8), c.k.view(torch.uint8))
    assert torch.equal(d.v_scale, c.v_scale)


def test_a_shallow_copy_is_the_same_cache(sa2):
    c = filled(sa2)
    d = copy.copy(c)
    assert d.k is c.k and d.v_scale is c.v_scale and pointers(d) == pointers(c) == tensors(c)


def test_a_copy_is_of_the_same_class(sa2):
    class Named(sa2.KvCache8):
        pass

    c = filled(sa2)
    n = Named(c.k, c.v, c.k_scale, c.v_scale)
    assert type(copy.deepcopy(n)) is Named and type(copy.copy(n)) is Named


def test_a_copy_is_made_after_tensors_moved(sa2):
    c = filled(sa2)
    c.k.data = c.k.clone()
    d = copy.copy(c)
    assert pointers(d) == tensors(c) and pointers(c) != tensors(c)


@pytest.mark.parametrize("name", ["k", "v", "k_scale", "v_scale"])
def test_moved_tensors_are_refused(sa2, name):
    c = filled(sa2)
    x = getattr(c, name)
    kept = x.data.clone()  # noqa: F841  (the old memory is still in use: the new one lies elsewhere)
    x.data = x.data.clone()
    q = torch.zeros((2, 3, 4, 64), dtype=torch.bfloat16)
    i = torch.zeros(2, dtype=torch.int32)
    for call in (lambda: sa2.cache8_append(c, q, q, i), lambda: sa2.cache8_read(c, i, 3), lambda: sa2.cache8_attn(q, c, i)):
        with pytest.raises(ValueError, match="moved"):
            call()
