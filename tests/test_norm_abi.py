"""Norm and rotation calls refuse bad arguments on the host, before anything reaches the GPU."""
import pytest
import torch

from block_diffusion_drafter_fc_gb300 import dflash as D
from test_cache_abi import _binding


def test_null_handle():
    L = D.LIB
    assert L.dflash_norm_rope(None, 1, 16, 1e-6, 16, 64, 16, 16, 64, None, 0, None, None, 0, None) == -1
    assert L.dflash_norm_rope_grad(None, 1, 16, 1e-6, 16, 64, 16, 16, 64, 16, 64, 16, None, 0, None, None, 0, None, 0, None,
                                   None) == -1
    assert L.dflash_norm_append(None, 0, 1, None, 16, 1, None, 1e-6, None, 0, None, None, 0, 16, 64, 16, 16, 64, None) == -1


def test_binding_refuses_wrong_tensors():
    c = _binding()
    q, k = torch.zeros(3, 8, 64, dtype=torch.bfloat16), torch.zeros(3, 2, 64, dtype=torch.bfloat16)
    w, pos, start = torch.ones(64, dtype=torch.bfloat16), torch.zeros(3, dtype=torch.int32), torch.tensor([0, 3], dtype=torch.int32)
    dw = torch.zeros(64)
    with pytest.raises(D.DFlashError, match="neither"):
        c.dflash_norm_rope(pos)
    with pytest.raises(D.DFlashError, match="neither"):
        c.dflash_norm_rope_grad(pos)
    for kw in (dict(q=q, q_norm=w), dict(q=q, q_out=q), dict(q=q, q_norm=w.float(), q_out=q), dict(q=q, q_norm=w[:32], q_out=q),
               dict(q=q, q_norm=torch.ones(128, dtype=torch.bfloat16)[::2], q_out=q), dict(q=k, q_norm=w, q_out=k),
               dict(q=q, q_norm=w, q_out=q[:2]), dict(q=q, q_norm=w, q_out=q, k=k[:2], k_norm=w, k_out=k[:2]),
               dict(q=q.float(), q_norm=w, q_out=q), dict(k=k, k_norm=w, k_out=k, q_norm=w)):
        with pytest.raises(D.DFlashError):
            c.dflash_norm_rope(pos, **kw)
    with pytest.raises(D.DFlashError):
        c.dflash_norm_rope(pos[:2], q=q, q_norm=w, q_out=q)
    with pytest.raises(D.DFlashError):
        c.dflash_norm_rope(pos.long(), q=q, q_norm=w, q_out=q)
    good = dict(q=q, q_norm=w, dq_out=q, dq=q, dq_norm=dw)
    for kw in (dict(dq_norm=None), dict(dq_norm=dw.double()), dict(dq_norm=dw[:32]), dict(dq_out=None), dict(dq=k),
               dict(dk_norm=dw), dict(q_norm=None)):
        with pytest.raises(D.DFlashError):
            c.dflash_norm_rope_grad(pos, **{**good, **kw})
    for kw in (dict(q=q), dict(q=q, q_out=q), dict(q=q, q_norm=w), dict(q_norm=w)):
        with pytest.raises(D.DFlashError):
            c.dflash_norm_append(0, start, k, k, w, **kw)
    with pytest.raises(D.DFlashError):
        c.dflash_norm_append(0, start, k, k, w.float())
    with pytest.raises(D.DFlashError):
        c.dflash_norm_append(0, start, k, k[:2], w)
    for call in (lambda: c.dflash_norm_rope(pos, q=q, q_norm=w, q_out=q), lambda: c.dflash_norm_rope_grad(pos, **good),
                 lambda: c.dflash_norm_append(0, start, k, k, w)):
        c.device_index = -1
        with pytest.raises(D.DFlashError, match="invalid argument"):   # no handle
            call_with_null_stream(c, call)
        c.device_index = 0
        with pytest.raises(D.DFlashError, match="device"):
            call()


def call_with_null_stream(c, call):
    c._on = lambda stream: 0
    try:
        call()
    finally:
        del c._on
