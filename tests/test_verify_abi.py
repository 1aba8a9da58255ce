"""Sampling calls refuse bad arguments on the host, before anything reaches the GPU."""
import types

import pytest
import torch

from block_diffusion_drafter_fc_gb300 import dflash as D
from test_cache_abi import _binding


def test_null_handle():
    L = D.LIB
    assert L.dflash_sample(None, 1, 4, 16, 4, 0, 1, None, None, 16, 4, 16, None) == -1
    assert L.dflash_tree_verify(None, 1, 16, 1, 16, 16, 4, 16, 4, 0, None, None, 0, 0, 0, None, None, 16, 16, 4, 16, 1, 16, 16,
                                None) == -1


def test_binding_refuses_wrong_tensors():
    c = _binding()
    s = types.SimpleNamespace(cuda_stream=0)
    x, e = torch.zeros(3, 10), torch.ones(3, 10)
    i = torch.zeros(3, dtype=torch.int32)
    start, path = torch.tensor([0, 3], dtype=torch.int32), torch.zeros(1, 4, dtype=torch.int32)
    n = torch.zeros(1, dtype=torch.int32)

    def sample(logits=x, noise=e, tokens=i, **kw):
        c.dflash_sample(logits, noise, tokens, stream=s, **kw)

    def verify(**kw):
        a = dict(row_start=start, parents=i, tokens=i, target=x, uniform=torch.zeros(3), noise=e[:1], path=path, n_path=n, id_last=n)
        a.update(kw)
        names = ("row_start", "parents", "tokens", "target", "uniform", "noise", "path", "n_path", "id_last")
        first = [a.pop(k) for k in names]
        c.dflash_tree_verify(*first, stream=s, **a)

    for call in (sample, verify):
        with pytest.raises(D.DFlashError, match="invalid argument"):   # no handle: what the binding lets through
            call()
    for kw in (dict(logits=x.double()), dict(logits=x.half()), dict(logits=x[0]), dict(logits=x.t()), dict(noise=e.bfloat16()),
               dict(noise=e[:2]), dict(noise=e[:, :9]), dict(tokens=i.long()), dict(rows=i[:2]), dict(rows=i.long()),
               dict(temperature=torch.ones(2)), dict(temperature=torch.ones(3).double())):
        with pytest.raises(D.DFlashError) as err:
            sample(**kw)
        assert "invalid argument" not in str(err.value), kw
    for kw in (dict(target=x[:2]), dict(target=x.double()), dict(noise=e[:0]), dict(noise=e[:1, :9]), dict(uniform=torch.zeros(2)),
               dict(uniform=None), dict(uniform=torch.zeros(3).double()), dict(path=path[0]), dict(tokens=i[:2]), dict(n_path=n.long()),
               dict(draft=x[:2]), dict(draft=x[:, :9], draft_row=i), dict(draft_row=i), dict(draft_temperature=torch.ones(3)),
               dict(draft=x, draft_row=i[:2]), dict(draft=x, draft_temperature=torch.ones(2)), dict(temperature=torch.ones(2))):
        with pytest.raises(D.DFlashError) as err:
            verify(**kw)
        assert "invalid argument" not in str(err.value), kw
    c.device_index = 0
    for call in (sample, verify):
        with pytest.raises(D.DFlashError, match="device"):
            call()
