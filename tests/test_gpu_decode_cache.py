"""GPU: caches whose arrays were resized, set or given other data since they were
made are refused before anything is launched."""
import pytest

torch = pytest.importorskip("torch")

import hadamard_rotated_activation_b200 as kq

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    kq.lib()


def _calls(k, v):
    q = torch.ones((2, 4, 128), dtype=torch.bfloat16, device="cuda")
    table = torch.tensor([[0, 3], [2, -1]], dtype=torch.int32, device="cuda")
    lens = torch.tensor([30, 9], dtype=torch.int32, device="cuda")
    pairs = torch.tensor([[0, 1]], dtype=torch.int32, device="cuda")
    out, ws = torch.empty_like(q), kq.empty_attn_workspace(2, 4, 2)
    return (lambda: kq.kq_attn_decode_int4_kv(q, k, v, None, None, table, 16, lens, 0.1, out, ws),
            lambda: kq.kq_kv_copy_pages(pairs, 16, k, v), lambda: kq.kq_kv_copy_pages(pairs, 16, k))


@pytest.mark.parametrize("name", ["codes", "scales", "zeros"])
@pytest.mark.parametrize("change", [
    lambda t: t.resize_(4, t.shape[1]), lambda t: t.set_(t[:4].clone()), lambda t: t.t_(),
    lambda t: setattr(t, "data", t[:4].clone()), lambda t: setattr(t, "data", t.view(-1).clone()),
    lambda t: t.unsqueeze_(0), lambda t: setattr(t, "data", t.cpu())],
    ids=["resize", "set", "transpose", "data", "flat", "unsqueeze", "host"])
def test_changed_arrays_are_refused(name, change):
    k, v = (kq.empty_kv_cache(64, 256) for _ in range(2))
    for c in (k, v):
        for a in (c.codes, c.scales, c.zeros):
            a.zero_()
    attn, both, one = _calls(k, v)
    for call in (attn, both, one):
        call()
    change(getattr(k, name))
    for call in (attn, both, one):
        with pytest.raises(ValueError):
            call()
    torch.cuda.synchronize()


def test_other_data_of_the_same_shape_is_the_caches():
    k, v = (kq.empty_kv_cache(64, 256) for _ in range(2))
    for c in (k, v):
        for a in (c.codes, c.scales, c.zeros):
            a.zero_()
    other = torch.arange(64, dtype=torch.uint8, device="cuda").view(64, 1).repeat(1, 128)
    k.codes.data = other
    _calls(k, v)[1]()
    assert k.codes.data_ptr() == other.data_ptr()
    assert torch.equal(other[16:32], other[:16]) and not torch.equal(other[32:48], other[:16])
