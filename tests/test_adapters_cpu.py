"""Host-side refusals of the adapter and optimiser calls: every one is answered before a device is touched."""
import ctypes as C

import numpy as np
import pytest


@pytest.fixture(scope="module")
def dp():
    import dictionary_compressed_linear_b200 as m
    from dictionary_compressed_linear_b200 import build
    build.build()
    return m


def _status(f):
    with pytest.raises(Exception) as e:
        f()
    return e.value.status


@pytest.mark.parametrize("args,status", [
    ((0, 64, 8, 1, 1), -2), ((48, 64, 8, 1, 1), -2), ((64, 0, 8, 1, 1), -2), ((64, -3, 8, 1, 1), -2),
    ((64, 64, 0, 1, 1), -5), ((64, 64, 129, 1, 1), -5), ((64, 64, 8, 0, 1), -5), ((64, 64, 8, 1025, 1), -5),
    ((64, 64, 8, 1, 0), -5), ((64, 64, 8, 1, (1 << 20) + 1), -5)])
def test_pool_limits(dp, args, status):
    assert _status(lambda: dp.dictproj_adapters_create(*args)) == status


@pytest.mark.parametrize("args", [(0, 1), ((1 << 20) + 1, 1), (1, 0), (1, 1025)])
def test_plan_limits(dp, args):
    assert _status(lambda: dp.dictproj_rows_create(*args)) == -5


def test_null_handles_and_arrays(dp):
    L = dp.lib()
    assert L.dictproj_adapters_create(64, 64, 8, 1, 1, None) == -1
    assert L.dictproj_rows_create(1, 1, None) == -1
    assert L.dictproj_adapters_set(None, 0, 0, 1.0, None, None, None) == -1
    assert L.dictproj_adapters_slot(None, 0, None, None, None) == -1
    assert L.dictproj_rows_set(None, None, 1, None) == -1
    assert L.dictproj_adapter_forward(None, None, 16, None, 16, None) == -1
    assert L.dictproj_adapter_forward(None, None, None, None, None, None) == -1
    assert L.dictproj_forward_adapters(16, None, None, None, None, 16, None) == -1
    assert L.dictproj_adapter_backward(None, None, 16, 16, None, 16, None, None, 0, None) == -1
    assert L.dictproj_adapter_backward(None, None, 16, 16, None, None, None, None, 0, None) == -1  # no output
    assert L.dictproj_adapter_backward(None, None, 16, 16, None, None, 16, None, 0, None) == -1  # dA without dB
    assert L.dictproj_group_reserve_backward(None, 1) == -1
    assert L.dictproj_backward_input(16, 1, None, None, 16, None) == -1
    assert L.dictproj_adamw_create(None, 1, 32, None) == -1
    assert L.dictproj_adamw_step(None, 1, 0.1, 0.9, 0.99, 1e-8, 0.0, 1.0, None) == -1
    for free in (L.dictproj_free_adapters, L.dictproj_free_rows, L.dictproj_free_adamw):
        free(None)


def _tensor(**kw):
    return {"p": 64, "g": 64, "m": 64, "v": 64, "n": 5, **kw}


@pytest.mark.parametrize("tensors,bits,status", [
    ([], 32, -5), ([_tensor()], 16, -5), ([_tensor(n=-1)], 32, -5), ([_tensor(n=1 << 32)], 32, -5),
    ([_tensor(p=0)], 32, -1), ([_tensor(g=0)], 32, -1), ([_tensor(m=0)], 8, -1), ([_tensor()], 8, -1),
    ([_tensor(), _tensor(v=66)], 32, -3), ([_tensor(copy=65)], 32, -3), ([_tensor(p=62)], 32, -3),
    ([_tensor(m_scale=64, v_scale=66)], 8, -3), ([_tensor(n=(1 << 32) - 1)] * 1025, 32, -5)])
def test_optimiser_tables(dp, tensors, bits, status):
    assert _status(lambda: dp.dictproj_adamw_create(tensors, bits)) == status


def _apart(at, **kw):
    return {"p": at, "g": at + 64, "m": at + 128, "v": at + 192, "n": 16, **kw}


@pytest.mark.parametrize("tensors,bits", [
    ([_apart(4096), _apart(4096)], 32), ([_apart(4096, g=4096)], 32), ([_apart(4096), _apart(8192, copy=4156)], 32),
    ([_apart(4096, n=17)], 32), ([_apart(4096), _apart(8192, g=4096 + 128)], 32), ([_apart(4096, n=1 << 20), _apart(8192, n=0), _apart(1 << 25)], 32),
    ([_apart(4096, m_scale=4096 + 132, v_scale=1024)], 8)])
def test_an_optimiser_writes_an_array_once(dp, tensors, bits):
    assert _status(lambda: dp.dictproj_adamw_create(tensors, bits)) == -5


@pytest.mark.parametrize("tensors,bits", [
    ([_apart(4096), _apart(4352)], 32), ([_apart(4096, g=1024), _apart(4352, g=1024), _apart(8192, g=1028)], 32),
    ([_apart(4096, n=0), _apart(4096)], 32), ([_apart(4096, m_scale=1024, v_scale=1028), _apart(4352, m_scale=1032, v_scale=1036)], 8)])
def test_neighbours_and_shared_gradients_do_not_overlap(dp, tensors, bits):
    # past the checks of the list there is no device to keep it on
    import torch
    if not torch.cuda.is_available():
        assert _status(lambda: dp.dictproj_adamw_create(tensors, bits)) not in (0, -5)


def test_the_reference_step_is_adamw():
    # the tests' fp32 restatement against the textbook form in fp64
    from adapter_reference import adamw
    rng = np.random.default_rng(5)
    n, step, lr, b1, b2, eps, wd = 1000, 7, 1e-2, 0.9, 0.99, 1e-8, 0.1
    t = {"p": rng.standard_normal(n), "g": rng.standard_normal(n), "m": rng.standard_normal(n), "v": rng.random(n)}
    t = {k: v.astype(np.float32) for k, v in t.items()}
    got = adamw(t, step, lr, b1, b2, eps, wd, 0.25, 32)
    p, g, m, v = (t[k].astype(np.float64) for k in "pgmv")
    g = 0.25 * g
    m, v = b1 * m + (1 - b1) * g, b2 * v + (1 - b2) * g * g
    want = p - lr * wd * p - lr * (m / (1 - b1 ** step)) / (np.sqrt(v / (1 - b2 ** step)) + eps)
    # a dozen roundings of 2^-24, on terms no larger than |p| + lr |m / r| each
    assert np.all(np.abs(got["p"] - want) <= 12 * 2.0 ** -24 * (np.abs(p) + lr * 40 * np.abs(m / np.sqrt(v))))


@pytest.mark.parametrize("step", [1, 2, 1000])
def test_the_dither_is_spread_evenly(step):
    from adapter_reference import dither
    d = dither(1 << 16, step) / 2.0 ** 20
    # mean and variance of a uniform variable, four standard errors of 2^16 draws
    assert abs(d.mean() - 0.5) < 4 * (1 / 12) ** 0.5 / 256
    assert abs(d.var() - 1 / 12) < 4 * (1 / 180) ** 0.5 / 256
    assert abs(np.corrcoef(d[:-1], d[1:])[0, 1]) < 4 / 256
