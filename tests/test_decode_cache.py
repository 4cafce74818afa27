"""Caches whose arrays changed since they were made, on the CPU: stand-ins for CUDA
tensors, and a launch failure armed, so that a call that were passed on would come
back as KQError and launch nothing."""
import ctypes

import pytest

torch = pytest.importorskip("torch")

import hadamard_rotated_activation_b200 as kq
from hadamard_rotated_activation_b200 import build as kqbuild
from test_decode_call import BF, F16, F32, I8, I32, U8, P, Tensor


class Array(Tensor):
    """What KVCacheInt4 and the checks that name an error ask besides."""

    is_cuda = True

    def dim(self):
        return len(self.shape)

    def numel(self):
        return self.shape.numel()


@pytest.fixture()
def armed():
    """The library with device 0 current and every launch failing."""
    kqbuild.build()
    L = kq.lib()
    entries = [ctypes.cast(f, ctypes.c_void_p).value
               for f in (L.kq_gemv, L.kq_attn_decode_int4_kv, L.kq_kv_copy_pages)]
    kq._native().init(BF, F32, F16, U8, I8, I32, lambda index: 0, lambda: 0, *entries)
    L.kq_diag_fail_next_launch(701)
    yield
    L.kq_diag_fail_next_launch(0)
    kq._call = None
    kq._native()


def _cache(layers=0):
    lead = (layers, 64) if layers else (64,)
    return kq.KVCacheInt4(Array(U8, *lead, 128), Array(F16, *lead, 2), Array(F16, *lead, 2))


def _attn(k, v):
    kq.kq_attn_decode_int4_kv(Array(BF, 2, 4, 128), k, v, None, None, Array(I32, 2, 4), 16,
                              Array(I32, 2), 0.1, Array(BF, 2, 4, 128, ptr=2 * P),
                              Array(U8, 1 << 26), stream=0)


def _copy(k, v):
    kq.kq_kv_copy_pages(Array(I32, 2, 2), 16, k, v, stream=0)


CHANGES = [("codes", dict(shape=(16, 128))), ("codes", dict(shape=(64, 64))),
           ("codes", dict(shape=(64 * 128,))), ("codes", dict(shape=(1, 64, 128))),
           ("codes", dict(shape=(0, 128))), ("codes", dict(dtype=I8)), ("codes", dict(_at=1)),
           ("codes", dict(_at=-1)), ("codes", dict(_contiguous=False)),
           ("scales", dict(shape=(16, 2))), ("scales", dict(dtype=BF)),
           ("zeros", dict(shape=(64, 1))), ("zeros", dict(_contiguous=False))]


def _change(cache, name, change):
    for key, value in change.items():
        setattr(getattr(cache, name), key, torch.Size(value) if key == "shape" else value)


@pytest.mark.parametrize("name,change", CHANGES)
@pytest.mark.parametrize("which", [0, 1])
@pytest.mark.parametrize("call", [_attn, _copy])
def test_changed_arrays_are_refused(armed, call, which, name, change):
    caches = _cache(), _cache()
    with pytest.raises(kq.KQError):          # passed on
        call(*caches)
    kq.lib().kq_diag_fail_next_launch(701)
    _change(caches[which], name, change)
    with pytest.raises(ValueError):
        call(*caches)
    with pytest.raises(ValueError):          # with nothing native in between
        kq._call = type("None_", (), dict(attn=lambda *a: None, copy=lambda *a: None))
        call(*caches)


@pytest.mark.parametrize("change", [dict(shape=(2, 64, 128)), dict(shape=(3 * 64, 128)),
                                    dict(shape=(3, 16, 128))])
def test_changed_arrays_of_layers(armed, change):
    caches = _cache(3), _cache(3)
    with pytest.raises(kq.KQError):
        _copy(*caches)
    kq.lib().kq_diag_fail_next_launch(701)
    _change(caches[1], "codes", change)
    with pytest.raises(ValueError):
        _copy(*caches)
    with pytest.raises((ValueError, TypeError)):
        caches[1].layer(0)


def test_arrays_that_moved_are_followed(armed):
    """Other memory of the same shape, type and place is the cache's from then on."""
    caches = _cache(), _cache()
    caches[0].codes._ptr = 8 * P
    with pytest.raises(kq.KQError) as e:
        _attn(*caches)
    assert e.value.status == kq.KQ_ERR_CUDA
    caches[0].codes._ptr = 8 * P + 8
    with pytest.raises(kq.KQError) as e:
        _attn(*caches)
    assert e.value.status == kq.KQ_ERR_MISALIGNED
