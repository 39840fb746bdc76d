"""The outcome operators' handle on the host (no GPU): what creation accepts
and refuses, the workspace's size, errors of calls that never reach the GPU;
and the 64-bit reference of the GPU tests against closed forms."""
import ctypes

import numpy as np
import pytest

import exact_tensor_network_gb300 as tn
from exact_tensor_network_gb300 import build as tnbuild
from outcome_reference import INF, Row


@pytest.fixture(scope="module", autouse=True)
def _built():
    tnbuild.build()


@pytest.mark.parametrize("args, status", [
    ((4, 10, 1, 0, 1.0), tn.TN_EINVAL),
    ((-1, 10, 1, 0, 1.0), tn.TN_EINVAL),
    ((1, 0, 1, 0, 1.0), tn.TN_EINVAL),
    ((1, 10, 0, 0, 1.0), tn.TN_EINVAL),
    ((1, 10, 1, -1, 1.0), tn.TN_EINVAL),
    ((1, 10, 1, 129, 1.0), tn.TN_EINVAL),
    ((1, 10, 1, 0, 0.0), tn.TN_EINVAL),
    ((1, 10, 1, 0, -1.0), tn.TN_EINVAL),
    ((1, 10, 1, 0, float("nan")), tn.TN_EINVAL),
    ((1, 10, 1, 0, INF), tn.TN_EINVAL),
    ((1, 1 << 41, 1, 0, 1.0), tn.TN_EOVERFLOW),
    ((1, 10, 1 << 31, 0, 1.0), tn.TN_EOVERFLOW),
    ((1, 1 << 40, 1 << 20, 0, 1.0), tn.TN_EOVERFLOW),
])
def test_create_refuses(args, status):
    with pytest.raises(tn.TNError) as e:
        tn.tn_outcomes_create(*args)
    assert e.value.status == status and str(e.value)


def test_workspace_is_enough_for_fewer_rows():
    """Fewer rows are cut into more segments: the workspace of a handle
    covers them."""
    for type_ in range(4):
        for cols in (1, 64, 5000, 131072, 1 << 24):
            sizes = []
            for rows in (1, 7, 100, 700, 20000):
                h = tn.tn_outcomes_create(type_, cols, rows, 20, 1.0)
                sizes.append(tn.tn_outcomes_workspace_bytes(h))
                tn.tn_outcomes_destroy(h)
            assert sizes == sorted(sizes) and sizes[0] >= 256


def test_calls_without_workspace_or_arguments():
    h = tn.tn_outcomes_create(tn.TN_TYPE_F32, 16, 2, 4, 1.0)
    try:
        r = tn.tn_rows(4096, 2, 16, 1, None, 0, 0)
        with pytest.raises(tn.TNError) as e:
            tn.tn_outcomes_score(h, r, None, 0, None, 4096, 4096, 0, None, None)
        assert e.value.status == tn.TN_ENOMEM and "workspace" in str(e.value)
        for rows in (tn.tn_rows(4098, 2, 16, 1, None, 0, 0), tn.tn_rows(4096, 3, 16, 1, None, 0, 0),
                     tn.tn_rows(None, 1, 16, 1, None, 0, 0), tn.tn_rows(4096, 2, -16, 1, None, 0, 0),
                     tn.tn_rows(4096, 2, 16, 0, None, 0, 0), tn.tn_rows(4096, 2, 16, 1, 4096, -1, 1)):
            with pytest.raises(tn.TNError) as e:
                tn.tn_outcomes_score(h, rows, None, 0, None, 4096, 4096, 0, None, None)
            assert e.value.status == tn.TN_EINVAL
        for ptr, size, status in ((None, 1 << 20, tn.TN_EINVAL), (4097, 1 << 20, tn.TN_EINVAL),
                                  (4096, 16, tn.TN_ENOMEM)):
            with pytest.raises(tn.TNError) as e:
                tn.tn_outcomes_set_workspace(h, ptr, size)
            assert e.value.status == status
        tn.tn_outcomes_check(h)      # nothing bound: nothing to report
        L = tn.lib()
        assert L.tn_outcomes_score(None, None, None, 0, None, None, None, 0, None, None, None) == tn.TN_EINVAL
        assert L.tn_outcomes_check(None) == tn.TN_EINVAL
        assert L.tn_outcomes_create(1, 1, 1, 0, 1.0, None) == tn.TN_EINVAL
        assert L.tn_outcomes_workspace_bytes(h, None) == tn.TN_EINVAL
        L.tn_outcomes_destroy(None)
    finally:
        tn.tn_outcomes_destroy(h)


def test_reference_closed_forms():
    """Uniform row, two-level row, Born rule, empty and invalid rows."""
    r = Row(np.zeros(8, np.float32), None, 3.0)
    assert np.isclose(r.logz, np.log(8)) and np.isclose(r.entropy, np.log(8))
    assert r.top(3)[0].tolist() == [0, 1, 2]
    r = Row(np.array([0.6, 0.8j], np.complex64), None, 1.0)
    assert np.allclose(r.logp([0, 1]), np.log([0.36, 0.64]), atol=1e-6) and abs(r.logz) < 1e-6
    r = Row(np.ones(4, np.float32), np.zeros(4), 1.0)
    assert r.logz == -INF and r.entropy == 0 and r.top(2)[0].tolist() == [-1, -1]
    assert r.distill([0], [1.0]) == 0
    assert np.isnan(Row(np.array([0, np.nan], np.float32), None, 1.0).logz)
    # KL of a teacher equal to the row is zero, and so is its gradient
    z = np.array([0.3, -1.0, 2.0], np.float32)
    r = Row(z, None, 1.0)
    assert abs(r.distill([0, 1, 2], z.astype(np.float64))) < 1e-12
    assert np.abs(r.distill_grad([0, 1, 2], z.astype(np.float64), 1.0)[0]).max() < 1e-12


class _Tensor:
    """What a call looks at before it launches anything, on any device."""

    def __init__(self, device, shape=(2, 16)):
        import torch
        self.device, self.shape, self.dtype, self.is_cuda = torch.device(device), shape, torch.float32, True

    def dim(self):
        return len(self.shape)

    def stride(self):
        return (self.shape[1], 1)

    def data_ptr(self):
        return 4096

    def is_conj(self):
        return False

    is_neg = is_conj


class _NoLaunch:
    def __getattr__(self, name):
        raise AssertionError(f"{name} was reached")


@pytest.mark.parametrize("bound, current, rows", [
    (0, 0, 1),      # rows of another device than the workspace, and not current
    (0, 1, 1),      # current, but the workspace is elsewhere
    (0, 1, 0),      # with the workspace, but not current
    (None, 0, 1),   # not current, nothing bound yet
])
def test_rows_of_another_device_are_refused(bound, current, rows, monkeypatch):
    """On the host, before anything is bound or launched: a kernel would run on
    the current device with another one's addresses."""
    import torch
    op = tn.Outcomes(16, torch.float32, max_rows=2)
    monkeypatch.setattr(op, "_L", _NoLaunch())
    monkeypatch.setattr(op, "_current_device", lambda: current, raising=False)
    monkeypatch.setattr(op, "bind_workspace", lambda device=None: pytest.fail("workspace bound"))
    if bound is not None:
        op._ws, op._index = object(), bound
    x = _Tensor(f"cuda:{rows}")
    for call in (lambda: op.score(x), lambda: op.score_grad(x, None, None, None, None),
                 lambda: op.distill(x, None, None), lambda: op.distill_grad(x, None, None, None, None),
                 lambda: op.distill_step(x, None, None, None)):
        with pytest.raises(ValueError, match="device|workspace"):
            call()


def test_stream_of_another_device_is_refused(monkeypatch):
    import torch
    op = tn.Outcomes(16, torch.float32, max_rows=2)
    monkeypatch.setattr(op, "_L", _NoLaunch())
    monkeypatch.setattr(op, "_current_device", lambda: 0, raising=False)
    op._ws, op._index = object(), 0

    class Stream:
        cuda_stream, device = 1, torch.device("cuda", 1)

    with pytest.raises(ValueError, match="stream"):
        op.score(_Tensor("cuda:0"), stream=Stream())
