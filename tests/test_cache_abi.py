"""Cache calls refuse bad arguments on the host, before anything reaches the GPU."""
import ctypes as C
import types

import pytest
import torch

from block_diffusion_drafter_fc_gb300 import dflash as D

GOOD = dict(n_layer=2, n_head=8, n_head_kv=2, head_dim=64, page_size=16, n_pages=40, max_seq=4, max_pages=9)


def _size(**kw):
    cfg = D.CacheConfig(**{**GOOD, **kw})
    a, b, s = C.c_size_t(), C.c_size_t(), C.c_size_t()
    return D.LIB.dflash_cache_workspace_size(C.byref(D.make_cache_config(cfg)), C.byref(a), C.byref(b), C.byref(s))


def test_struct_layout_matches_header():
    assert C.sizeof(D.dflash_cache_config) == 80
    assert D.dflash_cache_config.rope_theta.offset == 72


def test_workspace_sizes():
    page, state, scratch = D.cache_workspace_size(D.make_cache_config(D.CacheConfig(**GOOD)))
    assert page == 40 * 2 * 2 * 2 * 16 * 64 * 2
    assert state == 256 + 256 + 256      # 144, 16 and 160 bytes
    assert scratch > 0 and scratch % 256 == 0
    big = D.make_cache_config(D.CacheConfig(**{**GOOD, "n_pages": 30000, "n_layer": 64, "n_head_kv": 8, "head_dim": 128,
                                              "page_size": 64}))
    assert D.cache_workspace_size(big)[0] == 30000 * 64 * 2 * 8 * 64 * 128 * 2   # past 32 bits


@pytest.mark.parametrize("want,kw", [
    (0, {}), (0, {"dtype": "f32"}), (0, {"rotary_dim": 0}), (0, {"rotary_dim": 56}), (0, {"n_head": 2}),
    (-1, {"n_layer": 0}), (-1, {"n_pages": 0}), (-1, {"max_pages": 0}), (-1, {"rotary_dim": -8}),
    (-1, {"rope_theta": 1.0}), (-1, {"rope_factor": 0.5}), (-1, {"attn_scale": float("nan")}),
    (-1, {"rope_scaling": "yarn"}), (0, {"rope_scaling": "yarn", "rope_orig_positions": 4096}),
    (-1, {"rope_scaling": "yarn", "rope_orig_positions": 4096, "rope_beta_fast": 0.5}),
    (-1, {"rope_mscale": -1.0}), (-1, {"attn_scale": -0.5}), (0, {"rotary_dim": 0, "rope_theta": 0.0}),
    (-2, {"dtype": "fp8"}), (-2, {"n_head": 7}), (-2, {"head_dim": 96}), (-2, {"head_dim": 256}),
    (-2, {"page_size": 8}), (-2, {"page_size": 48}), (-2, {"page_size": 512}), (-2, {"rotary_dim": 72}),
    (-2, {"rotary_dim": 12}), (-2, {"max_seq": 4097}), (-2, {"max_pages": 1 << 28}),
    (-2, {"n_pages": 1 << 30}),
], ids=str)
def test_config_validation(want, kw):
    assert _size(**kw) == want


def test_bad_enums():
    c = D.make_cache_config(D.CacheConfig(**GOOD))
    a, b, s = C.c_size_t(), C.c_size_t(), C.c_size_t()
    for name, v in (("dtype", 4), ("dtype", -1), ("rope_layout", 2), ("rope_scaling", 4)):
        was = getattr(c, name)
        setattr(c, name, v)
        assert D.LIB.dflash_cache_workspace_size(C.byref(c), C.byref(a), C.byref(b), C.byref(s)) == -1
        setattr(c, name, was)
    assert D.LIB.dflash_cache_workspace_size(C.byref(c), None, C.byref(b), C.byref(s)) == -1


def test_null_handle_and_areas():
    c = D.make_cache_config(D.CacheConfig(**GOOD))
    h, L = C.c_void_p(), D.LIB
    assert L.dflash_cache_create(None, 256, 256, 256, C.byref(h)) == -1
    assert L.dflash_cache_create(C.byref(c), None, 256, 256, C.byref(h)) == -1
    assert L.dflash_cache_create(C.byref(c), 256, 264, 256, C.byref(h)) == -1      # not 256-byte aligned
    assert L.dflash_rope(None, 1, 1, 16, 64, 16, 16, 64, 0, None) == -1
    assert L.dflash_cache_append(None, 0, 1, None, 16, 1, None, None, 0, None, 0, 16, 64, 16, 64, None) == -1
    assert L.dflash_tree_mask(None, 1, 16, 1, 16, 16, 1, None, None) == -1
    assert L.dflash_tree_attend(None, 0, 1, None, 16, 1, 1, None, 0, 16, 64, 16, 64, None, None) == -1
    assert L.dflash_tree_accept(None, 1, 16, 1, 16, 16, 16, 16, 1, 16, 16, None) == -1
    assert L.dflash_cache_commit(None, 1, None, None, 0, 16, None) == -1
    assert L.dflash_cache_reserve(None, 1, None, 16, None) == -1
    assert L.dflash_cache_fork(None, 1, 16, 16, None) == -1
    assert L.dflash_cache_trim(None, 1, None, 16, None) == -1
    v = C.c_uint32()
    assert L.dflash_cache_read_status(None, C.byref(v), None) == -1
    assert L.dflash_cache_last_error(None) == b""
    L.dflash_cache_destroy(None)


def _binding():
    """A PagedCache without a handle: the binding's own checks come first."""
    c = object.__new__(D.PagedCache)
    c.cfg, c.dtype, c.h = D.CacheConfig(**GOOD), torch.bfloat16, None
    return c


def test_binding_refuses_wrong_tensors():
    c = _binding()
    x = torch.zeros(3, 8, 64, dtype=torch.bfloat16)
    pos = torch.zeros(3, dtype=torch.int32)
    for bad in (x.float(), x[..., :32], x[0], x.transpose(0, 1)):
        with pytest.raises(D.DFlashError):
            c.dflash_rope(bad, pos, torch.empty_like(bad))
    with pytest.raises(D.DFlashError):
        c.dflash_rope(x, pos.long(), x)
    with pytest.raises(D.DFlashError):
        c.dflash_rope(x, pos[:2], x)
    with pytest.raises(D.DFlashError):
        c.dflash_rope(x, pos, x[:2])
    start = torch.tensor([0, 3], dtype=torch.int32)
    kv = torch.zeros(3, 2, 64, dtype=torch.bfloat16)
    with pytest.raises(D.DFlashError):
        c.dflash_cache_append(0, start, kv, kv[:2])
    with pytest.raises(D.DFlashError):
        c.dflash_cache_append(0, start, kv, kv, q=x)
    with pytest.raises(D.DFlashError):
        c.dflash_cache_append(0, start, x, x)              # key rows have n_head_kv heads
    with pytest.raises(D.DFlashError):
        c.dflash_tree_attend(0, start, 3, x, x[:2])
    with pytest.raises(D.DFlashError):
        c.dflash_tree_attend(0, start, 3, x, torch.empty_like(x), mask=torch.zeros(2, 1, dtype=torch.int32))
    with pytest.raises(D.DFlashError):
        c.dflash_tree_attend(0, start, 3, x, torch.empty_like(x), lse=torch.zeros(3, 8, dtype=torch.float64))
    with pytest.raises(D.DFlashError):
        c.dflash_cache_commit(torch.zeros(2, 3, dtype=torch.int32), torch.zeros(3, dtype=torch.int32))
    with pytest.raises(D.DFlashError):
        c.dflash_cache_trim(torch.zeros(3, dtype=torch.int32), seqs=torch.zeros(2, dtype=torch.int32))
    with pytest.raises(D.DFlashError, match="invalid argument"):
        c.dflash_rope(x, pos, x, stream=types.SimpleNamespace(cuda_stream=0))   # no handle


def test_binding_refuses_streams_of_another_device():
    c = _binding()
    x, i = torch.zeros(3, 8, 64, dtype=torch.bfloat16), torch.zeros(3, dtype=torch.int32)
    with pytest.raises(D.DFlashError, match="device 1"):
        c.dflash_rope(x, i, x, stream=types.SimpleNamespace(cuda_stream=16, device_index=1))


def test_binding_refuses_masks_and_paths_without_columns():
    """An empty tensor has no address, which to the library means a chain, or no path at all."""
    c = _binding()
    x = torch.zeros(3, 8, 64, dtype=torch.bfloat16)
    start = torch.tensor([0, 3], dtype=torch.int32)
    with pytest.raises(D.DFlashError, match="words"):
        c.dflash_tree_attend(0, start, 3, x, torch.empty_like(x), mask=torch.zeros(3, 0, dtype=torch.int32))
    with pytest.raises(D.DFlashError, match="max_path"):
        c.dflash_cache_commit(torch.zeros(2, 0, dtype=torch.int32), torch.zeros(2, dtype=torch.int32))


def test_binding_refuses_tensors_of_another_device():
    c = _binding()
    c.device_index = 0
    x = torch.zeros(3, 8, 64, dtype=torch.bfloat16)
    kv = torch.zeros(3, 2, 64, dtype=torch.bfloat16)
    i = torch.zeros(3, dtype=torch.int32)
    start = torch.tensor([0, 3], dtype=torch.int32)
    calls = [lambda: c.dflash_rope(x, i, x), lambda: c.dflash_cache_append(0, start, kv, kv),
             lambda: c.dflash_tree_mask(start, i, torch.zeros(3, 1, dtype=torch.int32)),
             lambda: c.dflash_tree_attend(0, start, 3, x, torch.empty_like(x)),
             lambda: c.dflash_tree_accept(start, i, i, i, i.view(1, 3), i[:1], i[:1]),
             lambda: c.dflash_cache_commit(i[None], i[:1]), lambda: c.dflash_cache_reserve(i),
             lambda: c.dflash_cache_fork(i, i), lambda: c.dflash_cache_trim(i)]
    for call in calls:
        with pytest.raises(D.DFlashError, match="device"):
            call()


def test_most_slots_of_a_sequence():
    """Slot numbers of a whole tile of slots stay below 2^31."""
    assert _size(max_pages=(1 << 27) - 64) == 0        # pages of 16 slots
    assert _size(max_pages=(1 << 27) - 63) == -2
