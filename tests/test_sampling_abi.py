"""The sampler's handle and the 8-bit matrices' calls on the host (no GPU): what they accept
and refuse, the workspace's size; and the 64-bit references of the GPU tests against
closed forms."""
import math

import numpy as np
import pytest

import block8_reference as b8
import sampling_reference as ref
import exact_tensor_network_gb300 as tn
from exact_tensor_network_gb300 import build as tnbuild

INF, NAN = math.inf, math.nan


@pytest.fixture(scope="module", autouse=True)
def _built():
    tnbuild.build()


# ---- the sampler -------------------------------------------------------------

@pytest.mark.parametrize("args, status", [
    ((4, 10, 1, 1.0), tn.TN_EINVAL),
    ((-1, 10, 1, 1.0), tn.TN_EINVAL),
    ((1, 0, 1, 1.0), tn.TN_EINVAL),
    ((1, 10, 0, 1.0), tn.TN_EINVAL),
    ((1, 10, 1, 0.0), tn.TN_EINVAL),
    ((1, 10, 1, -1.0), tn.TN_EINVAL),
    ((1, 10, 1, NAN), tn.TN_EINVAL),
    ((1, 10, 1, INF), tn.TN_EINVAL),
    ((1, 1 << 31, 1, 1.0), tn.TN_EOVERFLOW),
    ((1, 1 << 30, 1 << 40, 1.0), tn.TN_EOVERFLOW),
])
def test_sampler_create_refuses(args, status):
    with pytest.raises(tn.TNError) as e:
        tn.tn_sampler_create(*args)
    assert e.value.status == status and tn.tn_sampler_last_error() in str(e.value)


def test_sampler_workspace_grows_with_rows():
    for type_ in range(4):
        for cols in (1, 64, 5000, 131072, 1 << 24):
            sizes = []
            for rows in (1, 7, 100, 700, 20000):
                h = tn.tn_sampler_create(type_, cols, rows, 1.0)
                sizes.append(tn.tn_sampler_workspace_bytes(h))
                tn.tn_sampler_destroy(h)
            assert sizes == sorted(sizes) and sizes[0] >= 256


def test_sampler_calls_without_workspace_or_arguments():
    h = tn.tn_sampler_create(tn.TN_TYPE_F32, 16, 2, 1.0)
    good = tn.tn_rows(4096, 2, 16, 1, None, 0, 0)
    try:
        def draw(rows, u=4096, wide=0, draws=1, ids=4096, logp=4096, kept=4096):
            with pytest.raises(tn.TNError) as e:
                tn.tn_sampler_draw(h, rows, None, u, wide, draws, ids, logp, kept)
            return e.value.status
        assert draw(good) == tn.TN_ENOMEM and "workspace" in tn.tn_sampler_last_error(h)
        for rows in (tn.tn_rows(4098, 2, 16, 1, None, 0, 0), tn.tn_rows(4096, 3, 16, 1, None, 0, 0),
                     tn.tn_rows(None, 1, 16, 1, None, 0, 0), tn.tn_rows(4096, 2, -16, 1, None, 0, 0),
                     tn.tn_rows(4096, 2, 16, 0, None, 0, 0), tn.tn_rows(4096, 2, 16, 1, 4096, -1, 1),
                     tn.tn_rows(4096, -1, 16, 1, None, 0, 0)):
            assert draw(rows) == tn.TN_EINVAL
        for bad in ({"u": None}, {"ids": None}, {"logp": None}, {"kept": None}, {"draws": -1}, {"u": 4098},
                    {"u": 4100, "wide": 1}):
            assert draw(good, **bad) == tn.TN_EINVAL
        assert draw(good, draws=1 << 62) == tn.TN_EOVERFLOW
        assert draw(good, draws=0, u=None, ids=None, logp=None) == tn.TN_ENOMEM
        for ptr, size, status in ((None, 1 << 20, tn.TN_EINVAL), (4097, 1 << 20, tn.TN_EINVAL),
                                  (4096, 16, tn.TN_ENOMEM)):
            with pytest.raises(tn.TNError) as e:
                tn.tn_sampler_set_workspace(h, ptr, size)
            assert e.value.status == status
        tn.tn_sampler_check(h)      # nothing bound: nothing to report
        L = tn.lib()
        assert L.tn_sampler_draw(None, None, None, None, 0, 1, None, None, None, None) == tn.TN_EINVAL
        assert L.tn_sampler_draw(h, None, None, None, 0, 1, None, None, None, None) == tn.TN_EINVAL
        assert L.tn_sampler_check(None) == tn.TN_EINVAL
        assert L.tn_sampler_create(1, 1, 1, 1.0, None) == tn.TN_EINVAL
        assert L.tn_sampler_workspace_bytes(h, None) == tn.TN_EINVAL
        L.tn_sampler_destroy(None)
    finally:
        tn.tn_sampler_destroy(h)


def test_sampler_refuses_host_tensors():
    import torch
    op = tn.Sampler(16, torch.float32, max_rows=2)
    with pytest.raises(ValueError):
        op.sample(torch.zeros(2, 16), torch.zeros(2))
    with pytest.raises(ValueError):
        op.sample(torch.zeros(2, 15), torch.zeros(2))
    with pytest.raises(ValueError):
        tn.Sampler(16, torch.float64)


class _Tensor:
    """What a call looks at before it launches anything, on any device."""

    def __init__(self, device, shape=(2, 16)):
        import torch
        self.device, self.shape, self.dtype, self.is_cuda = torch.device(device), shape, torch.float32, True

    def stride(self):
        return (self.shape[1], 1)

    def dim(self):
        return len(self.shape)

    def data_ptr(self):
        return 4096

    def is_conj(self):
        return False

    is_neg = is_conj


@pytest.mark.parametrize("bound, current, rows", [(0, 0, 1), (0, 1, 1), (0, 1, 0), (None, 0, 1)])
def test_rows_of_another_device_are_refused(bound, current, rows, monkeypatch):
    """On the host, before anything is bound or launched: a kernel would run on the current device with
    another one's addresses."""
    import torch
    op = tn.Sampler(16, torch.float32, max_rows=2)
    monkeypatch.setattr(op, "_L", None)
    monkeypatch.setattr(op, "_current_device", lambda: current)
    monkeypatch.setattr(op, "bind_workspace", lambda device=None: pytest.fail("workspace bound"))
    if bound is not None:
        op._ws, op._index = object(), bound
    with pytest.raises(ValueError, match="cuda"):
        op.sample(_Tensor(f"cuda:{rows}"), _Tensor(f"cuda:{rows}", (2,)))
    op._ws = None


def test_matrices_of_another_device_are_refused(monkeypatch):
    import torch
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0, raising=False)
    for call in (lambda x: tn.quantize8(x), lambda x: tn.linear8(x, None), lambda x: tn.linear8_grad(x, x, None)):
        with pytest.raises(ValueError, match="not the current device"):
            call(_Tensor("cuda:1"))


def test_sampler_reference_closed_forms():
    z = np.log(np.array([1, 2, 4, 1], np.float64)).astype(np.float32)
    assert list(ref.left(z, None, 1.0)) == [0, 1, 2, 3]
    assert list(ref.left(z, None, 1.0, top_k=2)) == [1, 2] and list(ref.left(z, None, 1.0, top_k=3)) == [0, 1, 2]
    assert list(ref.left(z, None, 1.0, top_p=0.5)) == [2] and list(ref.left(z, None, 1.0, top_p=0.51)) == [1, 2]
    assert list(ref.left(z, None, 1.0, min_p=0.3)) == [1, 2]
    assert list(ref.left(z, None, 1.0, temperature=0.0)) == [2]
    assert list(ref.left(z, np.array([1, 1, 0, 0]), 1.0, temperature=0.0)) == [1]
    assert ref.left(z, np.zeros(4), 1.0) == "empty" and ref.left(z * NAN, None, 1.0) == "undefined"
    e = ref.left(z, None, 1.0)
    for u, i in ((0.0, 0), (0.124, 0), (0.126, 1), (0.374, 1), (0.376, 2), (0.874, 2), (0.876, 3)):
        got, logp = ref.draw(e, u)
        assert got == i and abs(logp - math.log([1, 2, 4, 1][i] / 8)) < 1e-6
    w = np.array([0.6, 0.8j, 0.0], np.complex64)
    e = ref.left(w, None, 1.0)
    assert list(e) == [0, 1] and ref.draw(e, 0.35)[0] == 0 and ref.draw(e, 0.37)[0] == 1


# ---- 8-bit matrices ------------------------------------------------------------

def _blocks(rows=4, cols=256, codes=4096, scales=4096, row_stride=256, scale_stride=1, scale_block=4, tall=1, powers=1):
    return tn.tn_block8(codes, scales, rows, cols, row_stride, scale_stride, scale_block, tall, powers)


BAD_BLOCKS = [dict(rows=-1), dict(cols=-1), dict(tall=2), dict(tall=0), dict(row_stride=255), dict(row_stride=248),
              dict(scale_stride=0), dict(scale_block=0), dict(scale_stride=-1), dict(codes=None), dict(scales=None),
              dict(codes=4104), dict(scales=4098)]


@pytest.mark.parametrize("bad", BAD_BLOCKS, ids=str)
def test_matrices_that_are_refused(bad):
    x = tn.tn_matrix(4096, tn.TN_TYPE_BF16, bad.get("rows", 4), bad.get("cols", 256), 256, 1)
    for call in (lambda: tn.tn_block8_quantize(x, _blocks(**bad), None),
                 lambda: tn.tn_block8_product(_blocks(**bad), _blocks(), 4096, tn.TN_TYPE_F32, 4),
                 lambda: tn.tn_block8_product(_blocks(), _blocks(**bad), 4096, tn.TN_TYPE_F32, 4)):
        with pytest.raises(tn.TNError) as e:
            call()
        assert e.value.status == tn.TN_EINVAL and tn.tn_block8_last_error()


def test_calls_that_are_refused():
    def refused(status, f, *a):
        with pytest.raises(tn.TNError) as e:
            f(*a)
        assert e.value.status == status
    q, p, E = tn.tn_block8_quantize, tn.tn_block8_product, tn.TN_EINVAL
    x = tn.tn_matrix(4096, tn.TN_TYPE_BF16, 4, 256, 256, 1)
    wide = _blocks(256, 4, row_stride=16, scale_block=256)
    refused(E, q, x, None, None)
    refused(E, q, x, _blocks(5), None)                              # another shape
    refused(E, q, x, None, _blocks())                               # not the transposed one
    refused(E, q, x, _blocks(tall=128), wide)                       # two kinds of blocks
    refused(E, q, tn.tn_matrix(4096, tn.TN_TYPE_C64, 4, 256, 256, 1), _blocks(), None)
    refused(E, q, tn.tn_matrix(4097, tn.TN_TYPE_BF16, 4, 256, 256, 1), _blocks(), None)
    refused(E, q, tn.tn_matrix(None, tn.TN_TYPE_BF16, 4, 256, 256, 1), _blocks(), None)
    refused(E, q, tn.tn_matrix(4096, tn.TN_TYPE_BF16, 4, 256, -1, 1), _blocks(), None)
    big = 1 << 31
    refused(tn.TN_EOVERFLOW, q, tn.tn_matrix(4096, tn.TN_TYPE_BF16, big, 1, 1, 1), _blocks(big, 1, row_stride=16), None)
    refused(tn.TN_EOVERFLOW, p, _blocks(big), _blocks(), 4096, tn.TN_TYPE_F32, 4)
    refused(E, p, _blocks(), _blocks(cols=128), 4096, tn.TN_TYPE_F32, 4)
    refused(E, p, _blocks(), _blocks(), 4096, tn.TN_TYPE_C64, 4)
    refused(E, p, _blocks(), _blocks(), 4096, tn.TN_TYPE_F32, 3)    # rows of the output would overlap
    refused(E, p, _blocks(), _blocks(), None, tn.TN_TYPE_F32, 4)
    refused(E, p, _blocks(), _blocks(), 4098, tn.TN_TYPE_F32, 4)
    L = tn.lib()
    assert L.tn_block8_quantize(None, None, None, None) == E
    assert L.tn_block8_product(None, None, None, 1, 0, None) == E
    # nothing to do is not an error, and nothing is launched
    p(_blocks(0), _blocks(), 0, tn.TN_TYPE_F32, 4)
    q(tn.tn_matrix(0, tn.TN_TYPE_BF16, 0, 256, 256, 1), _blocks(0), None)
    q(tn.tn_matrix(0, tn.TN_TYPE_BF16, 4, 0, 1, 1), _blocks(4, 0, row_stride=0), None)


def test_host_tensors_are_refused():
    import torch
    x = torch.zeros(4, 256)
    b = tn.Blocks8(torch.zeros(4, 256, dtype=torch.float8_e4m3fn), torch.ones(4, 2))
    for call in (lambda: tn.quantize8(x), lambda: tn.linear8(x, b), lambda: tn.linear8_grad(x, x, b),
                 lambda: tn.product8(b, b), lambda: tn.quantize8(x, layout="other")):
        with pytest.raises(ValueError):
            call()
    assert torch.equal(b.values(), torch.zeros(4, 256))


def test_block_reference_closed_forms():
    import torch
    x = torch.tensor([[448.0, 1.0, -0.3], [449.0, 0.0, 2.0 ** -9], [0.0, 0.0, 0.0], [1.0, INF, 0.0], [1.0, NAN, 2.0]])
    codes, scales = b8.quantize(x, False)
    assert scales[:3, 0].tolist() == [1.0, 2.0, 1.0] and scales[3:].isnan().all()
    assert codes.tolist() == [[448.0, 1.0, -0.3125], [224.0, 0.0, 0.0], [0.0] * 3, [0.0] * 3, [0.0] * 3]
    # ties to even: halfway between 16 and 18, 18 and 20, and among the smallest
    assert b8.e4m3(torch.tensor([17.0, 19.0, 2.0 ** -10, 3 * 2.0 ** -10])).tolist() == [16.0, 20.0, 0.0, 2.0 ** -8]
    v = b8.e4m3(torch.linspace(-448, 448, 1001)).float()
    assert torch.equal(v.to(torch.float8_e4m3fn).float(), v)
