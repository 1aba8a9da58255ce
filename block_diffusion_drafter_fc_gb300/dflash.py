"""ctypes binding of libdflash (include/dflash.h): argument marshalling only.

Every step of the drafter runs in the library's CUDA kernels.  torch is used
for device memory (the ring, the scratch area, inputs and outputs) and for the
current stream.  Importing this module loads the library; a missing or
unloadable library raises immediately - there is no fallback path.
"""
from __future__ import annotations

import ctypes as C
import dataclasses
import pathlib
import re
from typing import Dict, List, Optional

import torch

BLOCK = 16          # rows of one noise block (anchor + 15 masks)

PKG = pathlib.Path(__file__).resolve().parent
LIB_PATH = PKG / "libdflash.so"
HEADER = PKG.parent / "include" / "dflash.h"

DTYPE = {"f32": 0, "bf16": 1, "fp8": 2, "fp4": 3}
MAX_LAYERS = 16
PROF_N = 12
PROF_CLASSES = ("embed", "qkv", "attention", "attn_merge", "o_proj", "gate_up", "down", "lm_head",
                "encode", "inject", "accept", "chain")
STATUS = {0: "ok", -1: "invalid argument", -2: "unsupported", -3: "too many rows",
          -4: "sequence out of range", -5: "CUDA error", -6: "not captured", -7: "device status"}


class dflash_config(C.Structure):
    _fields_ = [(n, C.c_int32) for n in (
        "n_layer", "n_embd", "n_head", "n_head_kv", "head_dim", "n_ff", "window", "n_vocab",
        "n_target_layers", "target_embd", "max_seq", "max_inject", "mask_token_id",
        "weight_dtype", "dense_dtype", "ring_dtype")] + [
        ("eps", C.c_float), ("reserved0", C.c_int32), ("rope_theta", C.c_double)]


_LAYER_PTRS = ("attn_norm", "wq", "wk", "wv", "wo", "q_norm", "k_norm", "ffn_norm", "gate", "up",
               "down")
_LAYER_SCALES = ("wq_scale", "wk_scale", "wv_scale", "wo_scale", "gate_scale", "up_scale",
                 "down_scale")


class dflash_layer_weights(C.Structure):
    _fields_ = [(n, C.c_void_p) for n in _LAYER_PTRS + _LAYER_SCALES]


class dflash_weights(C.Structure):
    _fields_ = [(n, C.c_void_p) for n in ("tok_embd", "lm_head", "lm_head_scale", "fc",
                                           "hidden_norm", "out_norm")] + [
        ("layers", dflash_layer_weights * MAX_LAYERS)]


class dflash_cache_config(C.Structure):
    _fields_ = [(n, C.c_int32) for n in (
        "n_layer", "n_head", "n_head_kv", "head_dim", "page_size", "n_pages", "max_seq",
        "max_pages", "dtype", "rope_layout", "rotary_dim", "rope_scaling",
        "rope_orig_positions")] + [(n, C.c_float) for n in (
            "rope_factor", "rope_beta_fast", "rope_beta_slow", "rope_mscale", "attn_scale")] + [
        ("rope_theta", C.c_double)]


class DFlashError(RuntimeError):
    pass


def _load() -> C.CDLL:
    if not LIB_PATH.exists():
        raise DFlashError(f"{LIB_PATH} is missing: build it with block_diffusion_drafter_fc_gb300.build")
    lib = C.CDLL(str(LIB_PATH))
    vp, i32, i64, f32, szp = C.c_void_p, C.c_int32, C.c_int64, C.c_float, C.POINTER(C.c_size_t)
    sig = {
        "dflash_workspace_size": (C.c_int, [C.POINTER(dflash_config), szp, szp]),
        "dflash_create": (C.c_int, [C.POINTER(dflash_config), C.POINTER(dflash_weights), vp, vp,
                                    C.POINTER(vp)]),
        "dflash_destroy": (None, [vp]),
        "dflash_encode": (C.c_int, [vp, vp, i32, vp, vp]),
        "dflash_inject": (C.c_int, [vp, i32, vp, vp, i32, vp]),
        "dflash_step": (C.c_int, [vp, i32, vp, vp, vp, vp, vp]),
        "dflash_accept": (C.c_int, [vp, i32, vp, vp, vp, vp]),
        "dflash_capture": (C.c_int, [vp, i32, vp, vp, vp, vp, vp, vp, vp]),
        "dflash_replay": (C.c_int, [vp, vp]),
        "dflash_replay_loop": (C.c_int, [vp, vp]),
        "dflash_graph_nodes": (C.c_int, [vp, i32, C.POINTER(i32), C.POINTER(i32), C.POINTER(i32)]),
        "dflash_profile_stamps": (C.c_int, [vp, i32, C.POINTER(i32), C.POINTER(C.c_double),
                                            C.POINTER(C.c_double), C.POINTER(i32), vp]),
        "dflash_encode_noalloc": (C.c_int, [C.POINTER(dflash_config), vp, vp, vp, i32, vp, vp]),
        "dflash_advance": (C.c_int, [vp, i32, vp, vp, vp, vp, vp, vp, vp]),
        "dflash_set_block_width": (C.c_int, [vp, i32]),
        "dflash_set_chain": (C.c_int, [vp, i32]),
        "dflash_attention_kernel": (C.c_int, [vp, i32]),
        "dflash_capture_loop": (C.c_int, [vp, i32, vp, vp, vp, vp, vp, vp, vp, vp]),
        "dflash_step_host": (C.c_int, [vp, i32, vp, vp, vp, vp, vp]),
        "dflash_ring_reset": (C.c_int, [vp, i32, vp]),
        "dflash_read_status": (C.c_int, [vp, C.POINTER(C.c_uint32), vp]),
        "dflash_profile_enable": (C.c_int, [vp, C.c_int]),
        "dflash_profile_read": (C.c_int, [vp, C.POINTER(C.c_double), C.POINTER(C.c_int32)]),
        "dflash_status_string": (C.c_char_p, [C.c_int]),
        "dflash_last_error": (C.c_char_p, [vp]),
        "dflash_cache_workspace_size": (C.c_int, [C.POINTER(dflash_cache_config), szp, szp, szp]),
        "dflash_cache_create": (C.c_int, [C.POINTER(dflash_cache_config), vp, vp, vp,
                                          C.POINTER(vp)]),
        "dflash_cache_destroy": (None, [vp]),
        "dflash_rope": (C.c_int, [vp, i32, i32, vp, i64, vp, vp, i64, i32, vp]),
        "dflash_cache_append": (C.c_int, [vp, i32, i32, vp, vp, i32, vp, vp, i64, vp, i64, vp, i64,
                                          vp, i64, vp]),
        "dflash_norm_append": (C.c_int, [vp, i32, i32, vp, vp, i32, vp, f32, vp, i64, vp, vp, i64, vp, i64,
                                         vp, vp, i64, vp]),
        "dflash_norm_rope": (C.c_int, [vp, i32, vp, f32, vp, i64, vp, vp, i64, vp, i64, vp, vp, i64, vp]),
        "dflash_norm_rope_grad": (C.c_int, [vp, i32, vp, f32, vp, i64, vp, vp, i64, vp, i64, vp,
                                            vp, i64, vp, vp, i64, vp, i64, vp, vp]),
        "dflash_tree_mask": (C.c_int, [vp, i32, vp, i32, vp, vp, i32, vp, vp]),
        "dflash_tree_attend": (C.c_int, [vp, i32, i32, vp, vp, i32, i32, vp, i32, vp, i64, vp, i64,
                                         vp, vp]),
        "dflash_prefix_plan": (C.c_int, [vp, i32, vp, i32, vp, vp, vp]),
        "dflash_prefix_workspace_size": (C.c_int, [vp, i32, szp]),
        "dflash_prefix_attend": (C.c_int, [vp, i32, i32, vp, vp, i32, i32, vp, i32, i32, vp, vp, vp, vp, i64, vp, i64,
                                           vp, vp]),
        "dflash_tree_accept": (C.c_int, [vp, i32, vp, i32, vp, vp, vp, vp, i32, vp, vp, vp]),
        "dflash_sample": (C.c_int, [vp, i32, i32, vp, i64, i32, i32, vp, vp, vp, i64, vp, vp]),
        "dflash_tree_verify": (C.c_int, [vp, i32, vp, i32, vp, vp, i32, vp, i64, i32, vp, vp, i64, i32, i32, vp, vp, vp, vp,
                                         i64, vp, i32, vp, vp, vp]),
        "dflash_cache_commit": (C.c_int, [vp, i32, vp, vp, i32, vp, vp]),
        "dflash_cache_reserve": (C.c_int, [vp, i32, vp, vp, vp]),
        "dflash_cache_fork": (C.c_int, [vp, i32, vp, vp, vp]),
        "dflash_cache_trim": (C.c_int, [vp, i32, vp, vp, vp]),
        "dflash_cache_read_status": (C.c_int, [vp, C.POINTER(C.c_uint32), vp]),
        "dflash_cache_last_error": (C.c_char_p, [vp]),
    }
    for name, (res, args) in sig.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    return lib


LIB = _load()


def header_symbols() -> List[str]:
    """Every function the public header declares."""
    text = HEADER.read_text()
    return sorted(set(re.findall(r"^\s*DFLASH_API\s+(?:const\s+)?\w+\s*\*?\s*(dflash_\w+)\s*\(", text, re.M)))


def _check(rc: int, h: Optional[int] = None, what: str = "") -> None:
    if rc != 0:
        msg = LIB.dflash_status_string(rc).decode()
        if h:
            extra = LIB.dflash_last_error(h).decode()
            if extra:
                msg += f" ({extra})"
        raise DFlashError(f"{what}: {msg} [{rc}]")


def _ptr(t: Optional[torch.Tensor]) -> Optional[int]:
    return None if t is None else t.data_ptr()


def _stream(stream=None) -> int:
    s = stream if stream is not None else torch.cuda.current_stream()
    return s.cuda_stream


def make_config(cfg, max_seq: Optional[int] = None,
                max_inject: Optional[int] = None) -> dflash_config:
    """dflash_config from any object with the drafter's geometry attributes
    (n_layer, n_embd, n_head, n_head_kv, head_dim, n_ff, window, n_vocab,
    n_target_layers, d_t, n_seq, mask_token_id, weight_dtype, dense_dtype,
    ring_dtype as "f32" | "bf16" | "fp8" | "fp4", eps, rope_theta)."""
    c = dflash_config()
    c.n_layer, c.n_embd, c.n_head, c.n_head_kv = cfg.n_layer, cfg.n_embd, cfg.n_head, cfg.n_head_kv
    c.head_dim, c.n_ff, c.window, c.n_vocab = cfg.head_dim, cfg.n_ff, cfg.window, cfg.n_vocab
    c.n_target_layers, c.target_embd = cfg.n_target_layers, cfg.d_t
    c.max_seq = max_seq if max_seq is not None else cfg.n_seq
    c.max_inject = max_inject if max_inject is not None else cfg.window
    c.mask_token_id = cfg.mask_token_id
    c.weight_dtype, c.dense_dtype = DTYPE[cfg.weight_dtype], DTYPE[cfg.dense_dtype]
    c.ring_dtype = DTYPE[cfg.ring_dtype]
    c.eps, c.rope_theta = cfg.eps, cfg.rope_theta
    return c


def workspace_size(c: dflash_config):
    rb, sb = C.c_size_t(), C.c_size_t()
    _check(LIB.dflash_workspace_size(C.byref(c), C.byref(rb), C.byref(sb)), what="workspace_size")
    return rb.value, sb.value


class Drafter:
    """A libdflash handle over the caller's device weights.

    `cfg` is any object with the geometry attributes make_config reads;
    `dev_weights` maps "tok_embd", "lm_head", "fc", "hidden_norm", "out_norm"
    and "l{i}.{attn_norm, wq, wk, wv, wo, q_norm, k_norm, ffn_norm, gate, up,
    down}" to DeviceWeight(data, scale) pairs of device tensors in the stored
    layout the header describes.  The ring and scratch areas are torch uint8
    tensors owned by this object; the weights stay the caller's (kept
    referenced here)."""

    def __init__(self, cfg, dev_weights: Dict[str, "DeviceWeight"],
                 max_seq: Optional[int] = None, max_inject: Optional[int] = None,
                 device: str = "cuda"):
        self.cfg = cfg
        self.c = make_config(cfg, max_seq, max_inject)
        self.ring_bytes, self.scratch_bytes = workspace_size(self.c)
        self.ring_mem = torch.empty(self.ring_bytes + 256, dtype=torch.uint8, device=device)
        self.scratch = torch.empty(self.scratch_bytes + 256, dtype=torch.uint8, device=device)
        self.dev_weights = dev_weights
        w = dflash_weights()
        for n in ("tok_embd", "lm_head", "fc", "hidden_norm", "out_norm"):
            setattr(w, n, dev_weights[n].data.data_ptr())
        if dev_weights["lm_head"].scale is not None:
            w.lm_head_scale = dev_weights["lm_head"].scale.data_ptr()
        for i in range(cfg.n_layer):
            lw = w.layers[i]
            for n in _LAYER_PTRS:
                setattr(lw, n, dev_weights[f"l{i}.{n}"].data.data_ptr())
            for n in ("wq", "wk", "wv", "wo", "gate", "up", "down"):
                sc = dev_weights[f"l{i}.{n}"].scale
                if sc is not None:
                    setattr(lw, n + "_scale", sc.data_ptr())
        self.w = w
        h = C.c_void_p()
        _check(LIB.dflash_create(C.byref(self.c), C.byref(w), self._aligned(self.ring_mem),
                                 self._aligned(self.scratch), C.byref(h)), what="create")
        self.h = h.value

    @staticmethod
    def _aligned(t: torch.Tensor) -> int:
        p = t.data_ptr()
        return (p + 255) // 256 * 256

    def close(self):
        if getattr(self, "h", None):
            LIB.dflash_destroy(self.h)
            self.h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    # ---- views of caller-visible state
    def ring_views(self):
        """(K, V, ring_pos) as torch views: K/V [max_seq][L][Hkv][W][hd]."""
        cfg, ms = self.cfg, self.c.max_seq
        el = 2 if cfg.ring_dtype == "bf16" else 4
        kv_bytes = cfg.n_layer * 2 * cfg.n_head_kv * cfg.window * cfg.head_dim * el
        base = self._aligned(self.ring_mem) - self.ring_mem.data_ptr()
        raw = self.ring_mem[base:base + kv_bytes * ms]
        dt = torch.bfloat16 if cfg.ring_dtype == "bf16" else torch.float32
        kv = raw.view(dt).view(ms, cfg.n_layer, 2, cfg.n_head_kv, cfg.window, cfg.head_dim)
        pos_off = base + (kv_bytes * ms + 255) // 256 * 256
        pos = self.ring_mem[pos_off:pos_off + 4 * ms * cfg.window].view(torch.int32).view(ms, cfg.window)
        return kv[:, :, 0], kv[:, :, 1], pos

    # ---- C-ABI calls (same names)
    def dflash_encode(self, feats: torch.Tensor, H_t: torch.Tensor, stream=None):
        _check(LIB.dflash_encode(self.h, _ptr(feats), feats.shape[0], _ptr(H_t), _stream(stream)),
               self.h, "encode")

    def dflash_inject(self, seq: int, H_t: torch.Tensor, pos: torch.Tensor, stream=None):
        _check(LIB.dflash_inject(self.h, seq, _ptr(H_t), _ptr(pos), pos.shape[0], _stream(stream)),
               self.h, "inject")

    def dflash_step(self, id_last, n_past, logits, drafts, stream=None):
        _check(LIB.dflash_step(self.h, id_last.shape[0], _ptr(id_last), _ptr(n_past), _ptr(logits),
                               _ptr(drafts), _stream(stream)), self.h, "step")

    def dflash_accept(self, drafts, targets, n_ok, stream=None):
        _check(LIB.dflash_accept(self.h, drafts.shape[0], _ptr(drafts), _ptr(targets), _ptr(n_ok),
                                 _stream(stream)), self.h, "accept")

    def dflash_capture(self, id_last, n_past, logits, drafts, targets=None, n_ok=None, stream=None):
        _check(LIB.dflash_capture(self.h, id_last.shape[0], _ptr(id_last), _ptr(n_past),
                                  _ptr(logits), _ptr(drafts), _ptr(targets), _ptr(n_ok),
                                  _stream(stream)), self.h, "capture")

    def dflash_replay(self, stream=None):
        _check(LIB.dflash_replay(self.h, _stream(stream)), self.h, "replay")

    def dflash_replay_loop(self, stream=None):
        _check(LIB.dflash_replay_loop(self.h, _stream(stream)), self.h, "replay_loop")

    def dflash_graph_nodes(self, loop: bool = False):
        """(kernel nodes, memory alloc/free nodes, other nodes) of the captured graph."""
        k, m, o = C.c_int32(), C.c_int32(), C.c_int32()
        _check(LIB.dflash_graph_nodes(self.h, int(loop), C.byref(k), C.byref(m), C.byref(o)),
               self.h, "graph_nodes")
        return k.value, m.value, o.value

    def dflash_set_chain(self, enable: bool):
        _check(LIB.dflash_set_chain(self.h, int(bool(enable))), self.h, "set_chain")

    def dflash_attention_kernel(self, n_seq: int) -> int:
        """Attention kernel of a step of n_seq sequences: 0 split, 1 clusters, 2 stream-K."""
        rc = LIB.dflash_attention_kernel(self.h, int(n_seq))
        _check(min(rc, 0), self.h, "attention_kernel")
        return rc

    def dflash_set_block_width(self, width: int):
        _check(LIB.dflash_set_block_width(self.h, int(width)), self.h, "set_block_width")

    def dflash_advance(self, drafts, targets, feats, id_last, n_past, n_ok, stream=None):
        _check(LIB.dflash_advance(self.h, drafts.shape[0], _ptr(drafts), _ptr(targets), _ptr(feats),
                                  _ptr(id_last), _ptr(n_past), _ptr(n_ok), _stream(stream)),
               self.h, "advance")

    def dflash_capture_loop(self, targets, feats, id_last, n_past, n_ok, logits, drafts, stream=None):
        _check(LIB.dflash_capture_loop(self.h, targets.shape[0], _ptr(targets), _ptr(feats),
                                       _ptr(id_last), _ptr(n_past), _ptr(n_ok), _ptr(logits),
                                       _ptr(drafts), _stream(stream)), self.h, "capture_loop")

    def dflash_step_host(self, id_last: torch.Tensor, n_past: torch.Tensor, drafts: torch.Tensor,
                         logits: Optional[torch.Tensor] = None, stream=None):
        _check(LIB.dflash_step_host(self.h, id_last.shape[0], _ptr(id_last), _ptr(n_past),
                                    _ptr(logits), _ptr(drafts), _stream(stream)), self.h, "step_host")

    def dflash_ring_reset(self, seq: int, stream=None):
        _check(LIB.dflash_ring_reset(self.h, seq, _stream(stream)), self.h, "ring_reset")

    def dflash_read_status(self, stream=None) -> int:
        v = C.c_uint32()
        rc = LIB.dflash_read_status(self.h, C.byref(v), _stream(stream))
        if rc not in (0, -7):
            _check(rc, self.h, "read_status")
        return v.value

    def dflash_profile_enable(self, enable: bool = True):
        _check(LIB.dflash_profile_enable(self.h, int(enable)), self.h, "profile_enable")

    def dflash_profile_read(self):
        ms = (C.c_double * PROF_N)()
        n = (C.c_int32 * PROF_N)()
        _check(LIB.dflash_profile_read(self.h, ms, n), self.h, "profile_read")
        return {PROF_CLASSES[i]: (ms[i], n[i]) for i in range(PROF_N)}

    def dflash_profile_stamps(self, stream=None, max_launches: int = 128):
        """[(class name, start_us, end_us)] of the last recorded step's launches."""
        cls = (C.c_int32 * max_launches)()
        t0 = (C.c_double * max_launches)()
        t1 = (C.c_double * max_launches)()
        n = C.c_int32()
        _check(LIB.dflash_profile_stamps(self.h, max_launches, cls, t0, t1, C.byref(n),
                                         _stream(stream)), self.h, "profile_stamps")
        return [(PROF_CLASSES[cls[i]], t0[i], t1[i]) for i in range(n.value)]


class DeviceWeight:
    """One weight tensor on the device in its stored layout, and its per-row f32
    scales (FP8 / FP4 projections; None otherwise)."""

    def __init__(self, data: torch.Tensor, scale: Optional[torch.Tensor]):
        self.data, self.scale = data, scale


# ---------------------------------------------------------------------------
# the target model's side: paged cache, tree attention, rotary positions

MAX_TREE = 1024       # most nodes of a tree with a mask
_INT32, _raw_stream = torch.int32, getattr(torch._C, "_cuda_getCurrentRawStream", None)
_LOGITS = {torch.float32: DTYPE["f32"], torch.bfloat16: DTYPE["bf16"]}
ROPE_LAYOUT = {"half": 0, "interleaved": 1}
ROPE_SCALING = {"none": 0, "linear": 1, "ntk": 2, "yarn": 3}


@dataclasses.dataclass(frozen=True)
class CacheConfig:
    """Geometry of a PagedCache (include/dflash.h, dflash_cache_config).  dtype: "f32" |
    "bf16"; rotary_dim None: the whole head."""

    n_layer: int
    n_head: int
    n_head_kv: int
    head_dim: int
    page_size: int
    n_pages: int
    max_seq: int
    max_pages: int
    dtype: str = "bf16"
    rope_layout: str = "half"       # half | interleaved
    rotary_dim: Optional[int] = None
    rope_theta: float = 1e6
    rope_scaling: str = "none"      # none | linear | ntk | yarn
    rope_factor: float = 1.0
    rope_orig_positions: int = 0
    rope_beta_fast: float = 32.0
    rope_beta_slow: float = 1.0
    rope_mscale: float = 0.0
    attn_scale: float = 0.0


def make_cache_config(cfg) -> dflash_cache_config:
    """dflash_cache_config from any object with CacheConfig's attributes."""
    c = dflash_cache_config()
    for n in ("n_layer", "n_head", "n_head_kv", "head_dim", "page_size", "n_pages", "max_seq",
              "max_pages", "rope_orig_positions", "rope_factor", "rope_beta_fast",
              "rope_beta_slow", "rope_mscale", "attn_scale", "rope_theta"):
        setattr(c, n, getattr(cfg, n))
    c.dtype = DTYPE[cfg.dtype]
    c.rope_layout, c.rope_scaling = ROPE_LAYOUT[cfg.rope_layout], ROPE_SCALING[cfg.rope_scaling]
    c.rotary_dim = cfg.head_dim if cfg.rotary_dim is None else cfg.rotary_dim
    return c


def cache_workspace_size(c: dflash_cache_config):
    """(page bytes, state bytes, scratch bytes) of a cache handle."""
    a, b, s = C.c_size_t(), C.c_size_t(), C.c_size_t()
    _check(LIB.dflash_cache_workspace_size(C.byref(c), C.byref(a), C.byref(b), C.byref(s)),
           what="cache_workspace_size")
    return a.value, b.value, s.value


class PagedCache:
    """A libdflash cache handle.  Pages, state and scratch are torch areas owned by
    this object; `pages` [n_pages][n_layer][2][n_head_kv][page_size][head_dim], `table`
    [max_seq][max_pages], `length` [max_seq] and `refs` [n_pages] are views of them.

    Tensors of rows are [T][heads][head_dim] with any row stride of a multiple of 16
    bytes (a slice of a fused projection's rows will do); row_start is int32 [n_seq + 1],
    seqs int32 [n_seq] or None for sequences 0.., all on the cache's device.

    A call runs on `stream`, or torch's current one.  The cache's own memory may be dropped
    with work in flight on any of them; a caller's tensors are the caller's to keep."""

    device_index = -1     # before the handle: the host's
    _areas = ()
    _streams = frozenset()   # those of the calls so far

    def __init__(self, cfg, device: str = "cuda"):
        self.cfg = cfg
        self.c = make_cache_config(cfg)
        pb, stb, scb = cache_workspace_size(self.c)
        self.page_mem = torch.empty(pb + 256, dtype=torch.uint8, device=device)
        self.state_mem = torch.empty(stb + 256, dtype=torch.uint8, device=device)
        self.scratch = torch.empty(scb + 256, dtype=torch.uint8, device=device)
        h = C.c_void_p()
        _check(LIB.dflash_cache_create(C.byref(self.c), Drafter._aligned(self.page_mem),
                                       Drafter._aligned(self.state_mem),
                                       Drafter._aligned(self.scratch), C.byref(h)),
               what="cache_create")
        self.h = h.value
        self.device_index = self.page_mem.device.index
        self._areas = (self.page_mem, self.state_mem, self.scratch)
        self.dtype = torch.bfloat16 if cfg.dtype == "bf16" else torch.float32

        def view(mem, off, shape, dt):
            n = dt.itemsize
            for d in shape:
                n *= d
            off += Drafter._aligned(mem) - mem.data_ptr()
            return mem[off:off + n].view(dt).view(shape)

        up = lambda x: (x + 255) // 256 * 256  # noqa: E731
        self.pages = view(self.page_mem, 0, (cfg.n_pages, cfg.n_layer, 2, cfg.n_head_kv,
                                             cfg.page_size, cfg.head_dim), self.dtype)
        self.table = view(self.state_mem, 0, (cfg.max_seq, cfg.max_pages), torch.int32)
        off = up(4 * cfg.max_seq * cfg.max_pages)
        self.length = view(self.state_mem, off, (cfg.max_seq,), torch.int32)
        self.refs = view(self.state_mem, off + up(4 * cfg.max_seq), (cfg.n_pages,), torch.int32)

    def close(self):
        if getattr(self, "h", None):
            LIB.dflash_cache_destroy(self.h)
            self.h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def _ok(self, rc: int, what: str) -> None:
        if rc != 0:
            extra = LIB.dflash_cache_last_error(self.h).decode() if self.h else ""
            msg = LIB.dflash_status_string(rc).decode() + (f" ({extra})" if extra else "")
            raise DFlashError(f"{what}: {msg} [{rc}]")

    def _rows(self, t: torch.Tensor, what: str, heads: Optional[int] = None):
        """(rows, row stride) of a [T][heads][head_dim] operand."""
        shape, stride = t.shape, t.stride()
        hd = self.cfg.head_dim
        if t.dtype is not self.dtype or len(shape) != 3 or shape[2] != hd or (
                heads is not None and shape[1] != heads):
            raise DFlashError(f"{what}: {tuple(shape)} {t.dtype} is not [T][{heads or 'heads'}]"
                              f"[{hd}] {self.dtype}")
        if shape[0] and (stride[2] != 1 or (stride[1] != hd and shape[1] > 1)):
            raise DFlashError(f"{what}: a row's heads have to be contiguous")
        if t.get_device() != self.device_index:
            raise DFlashError(f"{what}: a tensor on {t.device}, not on the cache's device")
        return shape[0], stride[0] if shape[0] > 1 else shape[1] * hd

    def _int(self, what: str, t, n: int) -> int:
        """Address of a contiguous int32 tensor of at least n values (None: null)."""
        if t is None:
            return 0
        if (t.dtype is _INT32 and t.get_device() == self.device_index and t.numel() >= n
                and t.is_contiguous()):
            return t.data_ptr()
        if t.get_device() != self.device_index:
            raise DFlashError(f"{what}: an index array on {t.device}, not on the cache's device")
        raise DFlashError(f"{what}: index arrays are contiguous int32 of the call's size")

    def _on(self, stream) -> int:
        """The stream's handle (None: torch's current one of the cache's device)."""
        h = _raw_stream(self.device_index) if stream is None else stream.cuda_stream
        if h not in self._streams:
            if h and getattr(stream, "device_index", self.device_index) != self.device_index:
                raise DFlashError(f"a stream of device {stream.device_index}, not of the cache's")
            # freed areas are handed out again only once this stream is done with them
            self._streams |= {h}
            for area in self._areas:
                area.record_stream(torch.cuda.ExternalStream(h, device=area.device))
        return h

    # ---- C-ABI calls (same names)
    def dflash_rope(self, x, pos, out, backward: bool = False, stream=None):
        T, xs = self._rows(x, "rope")
        n = x.shape[1]
        rows, os_ = self._rows(out, "rope", n)
        if rows != T:
            raise DFlashError("rope: x and out have different rows")
        self._ok(LIB.dflash_rope(self.h, T, n, x.data_ptr(), xs, self._int("rope", pos, T), out.data_ptr(), os_,
                                 backward, self._on(stream)), "rope")

    def dflash_cache_append(self, layer: int, row_start, k, v, depth=None, q=None, q_out=None,
                            seqs=None, stream=None):
        cfg, n = self.cfg, row_start.shape[0] - 1
        T, ks = self._rows(k, "append", cfg.n_head_kv)
        rows, vs = self._rows(v, "append", cfg.n_head_kv)
        qs = qos = qp = qop = 0
        if (q is None) != (q_out is None):
            raise DFlashError("append: q and q_out go together")
        same = rows == T
        if q is not None:
            rows, qs = self._rows(q, "append", cfg.n_head)
            rows_out, qos = self._rows(q_out, "append", cfg.n_head)
            same = same and rows == T and rows_out == T
            qp, qop = q.data_ptr(), q_out.data_ptr()
        if not same:
            raise DFlashError("append: operands have different rows")
        self._ok(LIB.dflash_cache_append(
            self.h, layer, n, self._int("append", seqs, n), self._int("append", row_start, 1), T,
            self._int("append", depth, T), qp, qs, qop, qos, k.data_ptr(), ks, v.data_ptr(), vs,
            self._on(stream)), "append")

    def _norm(self, what: str, w) -> int:
        """Address of a head's norm weights."""
        if (w.dtype is self.dtype and w.get_device() == self.device_index and w.dim() == 1
                and w.shape[0] == self.cfg.head_dim and w.is_contiguous()):
            return w.data_ptr()
        if w.get_device() != self.device_index:
            raise DFlashError(f"{what}: norm weights on {w.device}, not on the cache's device")
        raise DFlashError(f"{what}: norm weights are contiguous [{self.cfg.head_dim}] {self.dtype}")

    def dflash_norm_append(self, layer: int, row_start, k, v, k_norm, depth=None, q=None, q_out=None,
                           q_norm=None, eps: float = 1e-6, seqs=None, stream=None):
        cfg, n = self.cfg, row_start.shape[0] - 1
        T, ks = self._rows(k, "norm_append", cfg.n_head_kv)
        rows, vs = self._rows(v, "norm_append", cfg.n_head_kv)
        qs = qos = qp = qop = qn = 0
        if (q is None) != (q_out is None) or (q is None) != (q_norm is None):
            raise DFlashError("norm_append: q, q_norm and q_out go together")
        same = rows == T
        if q is not None:
            rows, qs = self._rows(q, "norm_append", cfg.n_head)
            rows_out, qos = self._rows(q_out, "norm_append", cfg.n_head)
            same = same and rows == T and rows_out == T
            qp, qop, qn = q.data_ptr(), q_out.data_ptr(), self._norm("norm_append", q_norm)
        if not same:
            raise DFlashError("norm_append: operands have different rows")
        i = self._int
        self._ok(LIB.dflash_norm_append(
            self.h, layer, n, i("norm_append", seqs, n), i("norm_append", row_start, 1), T, i("norm_append", depth, T),
            eps, qp, qs, qn, qop, qos, k.data_ptr(), ks, self._norm("norm_append", k_norm), v.data_ptr(), vs,
            self._on(stream)), "norm_append")

    def _pair(self, what: str, T: int, heads: int, x, w, out):
        """(address, stride) of x, address of its weights, (address, stride) of out; all None: nulls."""
        if x is None or w is None or out is None:
            if x is None and w is None and out is None:
                return 0, 0, 0, 0, 0
            raise DFlashError(f"{what}: a part's tensors go together")
        rows, xs = self._rows(x, what, heads)
        rows_out, os_ = self._rows(out, what, heads)
        if rows != T or rows_out != T:
            raise DFlashError(f"{what}: operands have different rows")
        return x.data_ptr(), xs, self._norm(what, w), out.data_ptr(), os_

    def dflash_norm_rope(self, pos, q=None, q_norm=None, q_out=None, k=None, k_norm=None, k_out=None,
                         eps: float = 1e-6, stream=None):
        x = k if q is None else q
        if x is None:
            raise DFlashError("norm_rope: neither q nor k")
        T = x.shape[0]
        self._ok(LIB.dflash_norm_rope(
            self.h, T, self._int("norm_rope", pos, T), eps, *self._pair("norm_rope", T, self.cfg.n_head, q, q_norm, q_out),
            *self._pair("norm_rope", T, self.cfg.n_head_kv, k, k_norm, k_out), self._on(stream)), "norm_rope")

    def _grad(self, T: int, heads: int, x, w, dout, dx, dw):
        """_pair's, with the gradients of the result and of the weights."""
        if dout is None or dw is None:
            if all(t is None for t in (x, w, dout, dx, dw)):
                return 0, 0, 0, 0, 0, 0, 0, 0
            raise DFlashError("norm_rope_grad: a part's tensors go together")
        rows, ds = self._rows(dout, "norm_rope_grad", heads)
        if rows != T:
            raise DFlashError("norm_rope_grad: operands have different rows")
        p, xs, wp, dp, dxs = self._pair("norm_rope_grad", T, heads, x, w, dx)
        if not p and x is None:
            raise DFlashError("norm_rope_grad: a part's tensors go together")
        if (dw.dtype is not torch.float32 or dw.dim() != 1 or dw.shape[0] != self.cfg.head_dim or not dw.is_contiguous()
                or dw.get_device() != self.device_index):
            raise DFlashError("norm_rope_grad: gradients of norm weights are contiguous f32 [head_dim] on the cache's device")
        return p, xs, wp, dout.data_ptr(), ds, dp, dxs, dw.data_ptr()

    def dflash_norm_rope_grad(self, pos, q=None, q_norm=None, dq_out=None, dq=None, dq_norm=None, k=None,
                              k_norm=None, dk_out=None, dk=None, dk_norm=None, eps: float = 1e-6, stream=None):
        x = k if q is None else q
        if x is None:
            raise DFlashError("norm_rope_grad: neither q nor k")
        T = x.shape[0]
        self._ok(LIB.dflash_norm_rope_grad(
            self.h, T, self._int("norm_rope_grad", pos, T), eps,
            *self._grad(T, self.cfg.n_head, q, q_norm, dq_out, dq, dq_norm),
            *self._grad(T, self.cfg.n_head_kv, k, k_norm, dk_out, dk, dk_norm), self._on(stream)), "norm_rope_grad")

    def dflash_tree_mask(self, row_start, parents, mask, depth=None, stream=None):
        T, shape = parents.shape[0], mask.shape
        if len(shape) != 2 or shape[0] != T:
            raise DFlashError("tree_mask: mask is int32 [T][words]")
        i = self._int
        self._ok(LIB.dflash_tree_mask(
            self.h, row_start.shape[0] - 1, i("tree_mask", row_start, 1), T, i("tree_mask", parents, T),
            i("tree_mask", mask, T), shape[1], i("tree_mask", depth, T), self._on(stream)), "tree_mask")

    def _attend_rows(self, what: str, q, out, mask, lse):
        """(rows, q's and out's strides, mask words, lse's address) of an attention call."""
        hq = self.cfg.n_head
        T, qs = self._rows(q, what, hq)
        rows, os_ = self._rows(out, what, hq)
        words = lp = 0
        if mask is not None:
            if mask.dim() != 2 or mask.shape[0] != T or T and not mask.shape[1]:   # (no words: a null address, a chain)
                raise DFlashError(f"{what}: mask is int32 [T][words]")
            words = mask.shape[1]
        if rows != T:
            raise DFlashError(f"{what}: q and out have different rows")
        if lse is not None:
            if (lse.dtype is not torch.float32 or not lse.is_contiguous() or lse.numel() != T * hq
                    or lse.get_device() != self.device_index):
                raise DFlashError(f"{what}: lse is contiguous f32 [T][n_head] on the cache's device")
            lp = lse.data_ptr()
        return T, qs, os_, words, lp

    def dflash_tree_attend(self, layer: int, row_start, max_tree: int, q, out, mask=None, lse=None,
                           seqs=None, stream=None):
        n, i = row_start.shape[0] - 1, self._int
        T, qs, os_, words, lp = self._attend_rows("tree_attend", q, out, mask, lse)
        self._ok(LIB.dflash_tree_attend(
            self.h, layer, n, i("tree_attend", seqs, n), i("tree_attend", row_start, 1), T, max_tree,
            i("tree_attend", mask, 0), words, q.data_ptr(), qs, out.data_ptr(), os_, lp, self._on(stream)),
            "tree_attend")

    def dflash_prefix_plan(self, group_start, plan, seqs=None, stream=None):
        """plan int32 [n_seq + n_group], written."""
        g, i = group_start.shape[0] - 1, self._int
        n = plan.shape[0] - g
        if n < 0:
            raise DFlashError("prefix_plan: plan is int32 [n_seq + n_group]")
        self._ok(LIB.dflash_prefix_plan(self.h, n, i("prefix_plan", seqs, n), g, i("prefix_plan", group_start, 1),
                                        i("prefix_plan", plan, n + g), self._on(stream)), "prefix_plan")

    def prefix_workspace(self, rows: int) -> int:
        """Bytes of dflash_prefix_attend's work area."""
        b = C.c_size_t()
        self._ok(LIB.dflash_prefix_workspace_size(self.h, rows, C.byref(b)), "prefix_workspace")
        return b.value

    def dflash_prefix_attend(self, layer: int, row_start, max_tree: int, q, out, group_start, plan, work,
                             mask=None, lse=None, seqs=None, stream=None):
        """work: a tensor of prefix_workspace(rows) bytes."""
        n, g, i = row_start.shape[0] - 1, group_start.shape[0] - 1, self._int
        T, qs, os_, words, lp = self._attend_rows("prefix_attend", q, out, mask, lse)
        if plan.shape[0] != n + g:
            raise DFlashError("prefix_attend: plan is int32 [n_seq + n_group]")
        if work.get_device() != self.device_index:
            raise DFlashError(f"prefix_attend: work on {work.device}, not on the cache's device")
        if not work.is_contiguous() or work.numel() * work.element_size() < self.prefix_workspace(T):
            raise DFlashError(f"prefix_attend: work is contiguous, of prefix_workspace({T}) bytes")
        self._ok(LIB.dflash_prefix_attend(
            self.h, layer, n, i("prefix_attend", seqs, n), i("prefix_attend", row_start, 1), T, max_tree,
            i("prefix_attend", mask, 0), words, g, i("prefix_attend", group_start, 1), i("prefix_attend", plan, n + g),
            work.data_ptr(), q.data_ptr(), qs, out.data_ptr(), os_, lp, self._on(stream)), "prefix_attend")

    def dflash_tree_accept(self, row_start, parents, tokens, targets, path, n_path, id_last,
                           stream=None):
        n, T, shape, i = row_start.shape[0] - 1, parents.shape[0], path.shape, self._int
        if len(shape) != 2 or shape[0] != n:
            raise DFlashError("tree_accept: path is int32 [n_seq][max_path]")
        self._ok(LIB.dflash_tree_accept(
            self.h, n, i("tree_accept", row_start, 1), T, i("tree_accept", parents, T),
            i("tree_accept", tokens, T), i("tree_accept", targets, T), i("tree_accept", path, 0), shape[1],
            i("tree_accept", n_path, n), i("tree_accept", id_last, n), self._on(stream)), "tree_accept")

    def _logits(self, what: str, t):
        """(address, row stride, dtype code, rows, tokens) of logits [rows][n_vocab]."""
        code, shape = _LOGITS.get(t.dtype), t.shape
        if code is None or len(shape) != 2 or (t.stride(1) != 1 and shape[1] > 1):
            raise DFlashError(f"{what}: logits are f32 or bf16 [rows][n_vocab], a row's contiguous")
        if t.get_device() != self.device_index:
            raise DFlashError(f"{what}: logits on {t.device}, not on the cache's device")
        rows, vocab = shape
        return t.data_ptr(), t.stride(0) if rows > 1 else vocab, code, rows, vocab

    def _floats(self, what: str, t, n: int) -> int:
        """Address of a contiguous f32 tensor of at least n values (None: null)."""
        if t is None:
            return 0
        if t.dtype is not torch.float32 or not t.is_contiguous() or t.numel() < n:
            raise DFlashError(f"{what}: temperatures and uniform numbers are contiguous f32 of the call's size")
        if t.get_device() != self.device_index:
            raise DFlashError(f"{what}: a tensor on {t.device}, not on the cache's device")
        return t.data_ptr()

    def _noise(self, what: str, t, rows: int, vocab: int):
        p, stride, code, n, v = self._logits(what, t)
        if code != DTYPE["f32"] or n < rows or v != vocab:
            raise DFlashError(f"{what}: noise is f32 [{rows}][{vocab}]")
        return p, stride

    def dflash_sample(self, logits, noise, tokens, rows=None, temperature=None, stream=None):
        """tokens int32 [T]; rows int32 [T] or None: row t of logits for tokens[t]."""
        T, i = tokens.shape[0], self._int
        p, stride, code, n, vocab = self._logits("sample", logits)
        e, es = self._noise("sample", noise, T, vocab)
        self._ok(LIB.dflash_sample(self.h, T, vocab, p, stride, code, n, i("sample", rows, T),
                                   self._floats("sample", temperature, T), e, es, i("sample", tokens, T), self._on(stream)),
                 "sample")

    def dflash_tree_verify(self, row_start, parents, tokens, target, uniform, noise, path, n_path, id_last,
                           draft=None, draft_row=None, temperature=None, draft_temperature=None, stream=None):
        n, T, shape, i, f = row_start.shape[0] - 1, parents.shape[0], path.shape, self._int, self._floats
        if len(shape) != 2 or shape[0] != n:
            raise DFlashError("tree_verify: path is int32 [n_seq][max_path]")
        p, stride, code, rows, vocab = self._logits("tree_verify", target)
        if rows != T:
            raise DFlashError("tree_verify: target has a row of logits for every node")
        e, es = self._noise("tree_verify", noise, n, vocab)
        d, ds, dc, nd = 0, 0, 0, 0
        if draft is not None and not T:
            draft = draft_row = draft_temperature = None
        if draft is not None:
            d, ds, dc, nd, dv = self._logits("tree_verify", draft)
            if dv != vocab or (nd < T if draft_row is None else T and not nd):
                raise DFlashError("tree_verify: draft is [n_draft][n_vocab], a row for every node without draft_row")
        elif draft_row is not None or draft_temperature is not None:
            raise DFlashError("tree_verify: draft_row and draft_temperature go with draft")
        if uniform is None:
            raise DFlashError("tree_verify: a uniform number for every node")
        self._ok(LIB.dflash_tree_verify(
            self.h, n, i("tree_verify", row_start, 1), T, i("tree_verify", parents, T), i("tree_verify", tokens, T), vocab,
            p, stride, code, f("tree_verify", temperature, T), d, ds, dc, nd, i("tree_verify", draft_row, T),
            f("tree_verify", draft_temperature, nd), f("tree_verify", uniform, T), e, es, i("tree_verify", path, 0), shape[1],
            i("tree_verify", n_path, n), i("tree_verify", id_last, n), self._on(stream)), "tree_verify")

    def dflash_cache_commit(self, path, n_path, seqs=None, stream=None):
        """path int32 [n_seq][max_path], or None: the first n_path nodes stay in place."""
        n, i, most = n_path.shape[0], self._int, 0
        if path is not None:
            if path.dim() != 2 or path.shape[0] != n or n and not path.shape[1]:   # (a null address: no path)
                raise DFlashError("commit: path is int32 [n_seq][max_path]")
            most = path.shape[1]
        self._ok(LIB.dflash_cache_commit(self.h, n, i("commit", seqs, n), i("commit", path, 0), most,
                                         i("commit", n_path, n), self._on(stream)), "commit")

    def dflash_cache_reserve(self, count, seqs=None, stream=None):
        n, i = count.shape[0], self._int
        self._ok(LIB.dflash_cache_reserve(self.h, n, i("reserve", seqs, n), i("reserve", count, n),
                                          self._on(stream)), "reserve")

    def dflash_cache_fork(self, src, dst, stream=None):
        n, i = src.shape[0], self._int
        self._ok(LIB.dflash_cache_fork(self.h, n, i("fork", src, n), i("fork", dst, n), self._on(stream)),
                 "fork")

    def dflash_cache_trim(self, new_len, seqs=None, stream=None):
        n, i = new_len.shape[0], self._int
        self._ok(LIB.dflash_cache_trim(self.h, n, i("trim", seqs, n), i("trim", new_len, n),
                                       self._on(stream)), "trim")

    def dflash_cache_read_status(self, stream=None) -> int:
        v = C.c_uint32()
        rc = LIB.dflash_cache_read_status(self.h, C.byref(v), self._on(stream))
        if rc not in (0, -7):
            self._ok(rc, "cache_read_status")
        return v.value
