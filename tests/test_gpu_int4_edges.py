"""Attention over INT4 pages where roundings, masks and integer ranges meet their ends."""
import pytest
import torch

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():          # collected on CPU-only hosts, never run there
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

import __graft_entry__  # noqa: E402

__graft_entry__.build()

import paged_kv_cache_221_gb300 as pa  # noqa: E402
from bounded_cases import Case  # noqa: E402
from gpu_util import to_dev  # noqa: E402


@pytest.fixture(autouse=True)
def no_device_error():
    yield
    assert pa.get_device_error() == 0, "device error word was set"


def attend(c, **kw):
    return pa.attention_int4(to_dev(c.q), to_dev(c.k), to_dev(c.v), to_dev(c.k_scale),
                             to_dev(c.v_scale), to_dev(c.tables), to_dev(c.lens),
                             int(c.lens.max()), c.scale, **kw)


# ------------------------------------------------------------------------------- windows
@pytest.mark.parametrize("T", [1, 2, 5, 16])
@pytest.mark.parametrize("psize", [0, 32])
@pytest.mark.parametrize("window", [2 ** 31 - 1, 2 ** 31 - 40, 1 << 30])
def test_window_up_to_the_largest(window, psize, T):
    """A window past every context is no window, up to the largest integer."""
    c = Case(T, [T, 17 + T, 96 + T, 97, 300], 4, 2, 64, T=T)
    plain = attend(c, partition_size=psize)
    assert torch.isfinite(plain.float()).all()
    assert torch.equal(attend(c, window_size=window, partition_size=psize), plain)
