"""moe_combine_bwd with a workgroup a token (65536 16-byte units of token rows or
more): whole, repeated and ragged batches of routes, for each number of units a
thread holds. Batches are of 8, 4 and 2 routes with 1, 2 and 4 units a thread
(rows of up to 1024, 2048 and 4096 units)."""
import pytest

from .test_gpu_sort import Maps, _check_all

pytestmark = pytest.mark.gpu


def _units(H, dt):
    return H * (2 if dt == "bf16" else 4) // 16


def _run(T, K, H, dt, padding):
    assert T * _units(H, dt) >= 65536, "a workgroup a route"
    m = Maps(T, K, 40, 16, padding=padding)
    _check_all(m, H, dt)
    _check_all(m, H, dt, pad=8, seed=2, inplace=True)


@pytest.mark.parametrize("padding", [0.0, 0.2])
@pytest.mark.parametrize("dt,T,H", [("bf16", 600, 1024), ("f32", 520, 512), ("bf16", 66, 8192)])
@pytest.mark.parametrize("K", [1, 7, 8, 9, 17, 32])
def test_batches_of_8(K, dt, T, H, padding):
    """1 unit a thread, workgroups of 2 and of 16 waves: less than a batch, one, one
    and a route, two and a route, four."""
    assert _units(H, dt) <= 1024
    _run(T, K, H, dt, padding)


@pytest.mark.parametrize("dt,T,H", [("bf16", 64, 8200), ("f32", 40, 8184)])
@pytest.mark.parametrize("K", [3, 4, 5, 9])
def test_batches_of_4(K, dt, T, H):
    assert 1024 < _units(H, dt) <= 2048
    _run(T, K, H, dt, 0.1)


@pytest.mark.parametrize("T,H", [(32, 8200), (16, 16384)])
@pytest.mark.parametrize("K", [1, 2, 3, 5])
def test_batches_of_2(K, T, H):
    assert 2048 < _units(H, "f32") <= 4096
    _run(T, K, H, "f32", 0.1)
