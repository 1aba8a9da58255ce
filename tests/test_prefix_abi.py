"""Shared-prefix calls refuse bad arguments on the host, before anything reaches the GPU."""
import ctypes as C
import types

import pytest
import torch

from block_diffusion_drafter_fc_gb300 import dflash as D
from test_cache_abi import _binding


def test_null_handle():
    L, b = D.LIB, C.c_size_t()
    assert L.dflash_prefix_plan(None, 1, None, 1, 16, 16, None) == -1
    assert L.dflash_prefix_workspace_size(None, 1, C.byref(b)) == -1
    assert L.dflash_prefix_attend(None, 0, 1, None, 16, 1, 1, None, 0, 1, 16, 16, 256, 16, 64, 16, 64, None, None) == -1


def test_binding_refuses_wrong_tensors():
    c = _binding()
    c.prefix_workspace = lambda rows: 1000
    x = torch.zeros(3, 8, 64, dtype=torch.bfloat16)
    i = torch.zeros(3, dtype=torch.int32)
    start, bounds, plan = (torch.tensor(v, dtype=torch.int32) for v in ([0, 1, 3], [0, 2], [0, 0, 0]))
    work = torch.zeros(1000, dtype=torch.uint8)
    s = types.SimpleNamespace(cuda_stream=0)

    def attend(**kw):
        a = dict(q=x, out=torch.empty_like(x), group_start=bounds, plan=plan, work=work, row_start=start)
        a.update(kw)
        c.dflash_prefix_attend(0, a.pop("row_start"), 3, a.pop("q"), a.pop("out"), a.pop("group_start"), a.pop("plan"),
                               a.pop("work"), stream=s, **a)

    with pytest.raises(D.DFlashError, match="invalid argument"):   # no handle: what the binding lets through
        attend()
    for kw in (dict(out=x[:2]), dict(plan=plan[:2]), dict(plan=plan.long()), dict(work=work[:-1]), dict(work=work[::2]),
               dict(group_start=bounds.long()), dict(mask=torch.zeros(2, 1, dtype=torch.int32)),
               dict(mask=torch.zeros(3, 0, dtype=torch.int32)), dict(lse=torch.zeros(3, 8, dtype=torch.float64)),
               dict(seqs=i[:1]), dict(q=x.float())):
        with pytest.raises(D.DFlashError) as e:
            attend(**kw)
        assert "invalid argument" not in str(e.value), kw
    with pytest.raises(D.DFlashError, match="n_seq"):
        c.dflash_prefix_plan(torch.zeros(5, dtype=torch.int32), plan, stream=s)
    with pytest.raises(D.DFlashError):
        c.dflash_prefix_plan(bounds, plan.long(), stream=s)
    c.device_index = 0
    for call in (attend, lambda: c.dflash_prefix_plan(bounds, plan, stream=s)):
        with pytest.raises(D.DFlashError, match="device"):
            call()
