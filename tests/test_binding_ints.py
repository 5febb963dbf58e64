"""Python integers past 32 bits are not cut to their low bits on the way to the library."""
import pytest
import torch

import __graft_entry__

__graft_entry__.build()

import paged_kv_cache_221_gb300 as pa  # noqa: E402


def test_prompt_workspace_of_large_sizes():
    args = (20, 2, 4, 4, 4096, 64, 128)
    assert pa.prompt_workspace_size(*args, 2 ** 32 + 5) == pa.prompt_workspace_size(*args)
    assert pa.prompt_workspace_size(*args, 5) < pa.prompt_workspace_size(*args)
    assert pa.prompt_workspace_size(2 ** 32 + 20, 2, 4, 4, 4096, 64, 128) > \
        pa.prompt_workspace_size(2 ** 30, 2, 4, 4, 4096, 64, 128)
    assert pa.prompt_workspace_size(20, 2, 4, 4, 4096, 64, 2 ** 32 + 128) == 0


@pytest.mark.gpu
def test_calls_of_large_sizes():
    from prompt_cases import Prompts
    c = Prompts(1, [40, 3], [100, 7], 4, 2, 64)

    def attend(**kw):
        return pa.prompt_attention(c.q, c.k, c.v, c.tables, c.ctx, c.starts,
                                   kw.pop("most", c.most), **kw)
    want = attend()
    assert torch.equal(attend(window_size=2 ** 32 + 5), want)
    for kw in (dict(window_size=-2 ** 32 + 5), dict(most=2 ** 32 + c.most),
               dict(partition_size=2 ** 32 + 128)):
        with pytest.raises(pa.PagedAttnError):
            attend(**kw)
    state = [torch.full((1, 4), -1, dtype=torch.int32, device="cuda"),
             torch.zeros(1, dtype=torch.int32, device="cuda"),
             torch.zeros(8, dtype=torch.int32, device="cuda")]
    with pytest.raises(ValueError):
        pa.extend_sequences(*state, torch.ones(1, dtype=torch.int32, device="cuda"), 2 ** 32 + 1)
    assert pa.get_device_error() == 0
