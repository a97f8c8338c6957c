"""What the torch helpers of the grouped operators tell the library about a
view: a recorder takes the library's place, so nothing runs on a device."""
import pytest
import torch

import dense_gemm_08_gb300 as lib


@pytest.fixture
def calls(monkeypatch):
    """Calls of the C entry points as (name, arguments); the tensors stay on the CPU."""
    made = []

    class Recorder:
        def __getattr__(self, name):
            def call(*args):
                made.append((name, args))
                return lib.GEMM_OK
            return call

    monkeypatch.setattr(lib, "library", Recorder)
    monkeypatch.setattr(lib, "_on_device", lambda device: None)
    monkeypatch.setattr(lib, "_stream_of", lambda stream: 0)
    return made


def wgrad(groups, M, N, **kwargs):
    A, B = torch.zeros(6, M), torch.zeros(6, N)
    return lib.gemm_grouped_wgrad(A, B, torch.zeros(groups + 1, dtype=torch.int32), **kwargs)


def test_one_row_gradients_in_a_column_are_refused(calls):
    # shape 2 x 1 x 4, strides 12, 1, 3: a row's values lie three apart
    apart = torch.zeros(2, 4, 3)[:, :, :1].transpose(1, 2)
    assert apart.shape == (2, 1, 4) and apart.stride() == (12, 1, 3)
    with pytest.raises(ValueError, match="out"):
        wgrad(2, 1, 4, out=apart)
    with pytest.raises(ValueError, match="C"):
        wgrad(2, 1, 4, beta=1.0, C=apart)
    assert not calls


@pytest.mark.parametrize("shape,strides,ld,stride", [
    ((2, 1, 4), (12, 1, 1), 4, 12),    # one row: its pitch says nothing
    ((2, 1, 4), (12, 50, 1), 50, 12),
    ((2, 3, 1), (12, 4, 1), 4, 12),
    ((2, 3, 1), (12, 4, 7), 4, 12),    # one column: neither does its distance
    ((2, 3, 1), (12, 1, 3), 1, 12),
    ((2, 3, 4), (12, 4, 1), 4, 12),
    ((2, 3, 4), (4, 8, 1), 8, 4),      # rows of the matrices in turn
    ((1, 3, 4), (12, 4, 1), 4, 0)])
def test_gradient_views(calls, shape, strides, ld, stride):
    t = torch.zeros(200).as_strided(shape, strides)
    wgrad(*shape, beta=1.0, C=t, out=t)
    (name, a), = calls
    assert name == "gemm_grouped_wgrad_f32"
    assert a[14:16] == (max(ld, shape[2]), stride) and a[17:19] == (max(ld, shape[2]), stride)


@pytest.mark.parametrize("strides", [(12, 4, 2), (12, 1, 3), (12, 3, 1)])
def test_gradient_views_refused(calls, strides):
    # columns apart, column-major, rows that overlap
    t = torch.zeros(200).as_strided((2, 3, 4), strides)
    with pytest.raises(ValueError):
        wgrad(2, 3, 4, out=t)
    assert not calls
