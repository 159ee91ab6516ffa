"""Python binding of the B200 block-sparse FlexAttention library (libflexattn.so).

Argument marshalling only: every step of the computation runs in the CUDA kernels
behind the C ABI of ``include/flexattn.h``.  PyTorch provides device memory and
streams.  There is no CPU fallback: importing this module without the built
library raises.

    bm = create_block_mask("and", [("causal",)], B=1, H=1, q_len=S, kv_len=S)
    o, lse = flex_attention(q, k, v, bm, score_mod=("alibi", slopes))

Around a paged cache: paged_append (new keys and values, rotary positions on the way),
flex_decode_paged (a few query tokens per sequence, each sequence with its own length),
flex_decode_shared (a batch that shares a long prefix), and rope_apply / rope_autograd.

Mask leaves: ("causal",), ("sliding", W), ("document",), ("prefix", P), combined
by "and" / "or" ("Concepts": mask_mod, Composing masks).  Score mods: None,
("alibi", slopes[Hq] fp32), ("softcap", cap), ("bias", bias[B, Hq, Sq, Skv] bf16),
("bias_softcap", bias, cap) ("Concepts": score_mod; attention-gym issue "Dynamic
Bias Tensor"; paper review sec. 2.1).
"""

from __future__ import annotations

import contextlib
import ctypes
import functools
import inspect
import os
from typing import Optional, Sequence, Tuple

import torch
from torch.autograd.function import once_differentiable

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libflexattn.so")

FA_OK, FA_ERR_INVALID_ARG, FA_ERR_UNSUPPORTED, FA_ERR_CUDA, FA_ERR_TIMEOUT, FA_ERR_BAD_BLOCKMASK = range(6)
BLOCK_SIZE = 128
MAX_LEAVES = 4
LEAF = {"causal": 0, "sliding": 1, "document": 2, "prefix": 3}
OP = {"and": 0, "or": 1}
ROPE_SCALING = {"linear": 1, "base": 2, "bands": 3, "yarn": 4}
SCORE = {"none": 0, "alibi": 1, "softcap": 2, "bias": 3, "bias_softcap": 4}

EXPORTS = ("fa_status_string", "fa_block_mask_shape", "fa_create_block_mask", "fa_create_block_mask_unsplit",
           "fa_workspace_size", "fa_backward_workspace_size", "fa_backward", "fa_forward_paged",
           "fa_decode_workspace_size", "fa_decode",
           "fa_forward", "fa_get_device_status", "fa_set_watchdog_ms", "fa_set_selftest_stall",
           "fa_forward_static_scratch", "fa_rope_frequencies", "fa_rope_apply", "fa_paged_append",
           "fa_decode_paged_workspace_size", "fa_decode_paged", "fa_decode_shared_workspace_size",
           "fa_decode_shared")


class FlexAttnError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        super().__init__(f"{what}: {status_string(status)}")


class MaskDesc(ctypes.Structure):
    _fields_ = [("n_leaves", ctypes.c_int32), ("op", ctypes.c_int32),
                ("kind", ctypes.c_int32 * MAX_LEAVES), ("param", ctypes.c_int64 * MAX_LEAVES),
                ("doc_ids", ctypes.c_void_p), ("doc_stride", ctypes.c_int64), ("doc_len", ctypes.c_int64),
                ("q_offset", ctypes.c_int64)]


class BlockMaskDesc(ctypes.Structure):
    _fields_ = [("kv_num_blocks", ctypes.c_void_p), ("kv_indices", ctypes.c_void_p),
                ("full_kv_num_blocks", ctypes.c_void_p), ("full_kv_indices", ctypes.c_void_p),
                ("B", ctypes.c_int32), ("H", ctypes.c_int32), ("nq", ctypes.c_int32), ("nkv", ctypes.c_int32),
                ("block_size", ctypes.c_int32), ("has_full", ctypes.c_int32),
                ("q_len", ctypes.c_int64), ("kv_len", ctypes.c_int64), ("mask", MaskDesc),
                ("q_num_blocks", ctypes.c_void_p), ("q_indices", ctypes.c_void_p),
                ("full_q_num_blocks", ctypes.c_void_p), ("full_q_indices", ctypes.c_void_p)]


class TensorDesc(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("dims", ctypes.c_int64 * 4), ("strides", ctypes.c_int64 * 4)]


class ScoreModDesc(ctypes.Structure):
    _fields_ = [("kind", ctypes.c_int32), ("softcap", ctypes.c_float), ("alibi_slopes", ctypes.c_void_p),
                ("bias", ctypes.c_void_p), ("bias_strides", ctypes.c_int64 * 4)]


class RopeDesc(ctypes.Structure):
    _fields_ = [("inv_freq", ctypes.c_void_p), ("rotary_dim", ctypes.c_int32), ("interleaved", ctypes.c_int32),
                ("amplitude", ctypes.c_float)]


class RopeScalingDesc(ctypes.Structure):
    _fields_ = [("kind", ctypes.c_int32), ("factor", ctypes.c_double), ("original_len", ctypes.c_double),
                ("rot_lo", ctypes.c_double), ("rot_hi", ctypes.c_double)]


def _load():
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"{LIB_PATH} is missing: build it with `python block_sparse_attention_48_b200/build.py`")
    lib = ctypes.CDLL(LIB_PATH)
    vp, i64 = ctypes.c_void_p, ctypes.c_int64
    lib.fa_status_string.argtypes = [ctypes.c_int]
    lib.fa_status_string.restype = ctypes.c_char_p
    lib.fa_block_mask_shape.argtypes = [i64, i64, ctypes.c_int, ctypes.POINTER(ctypes.c_int32),
                                        ctypes.POINTER(ctypes.c_int32)]
    lib.fa_create_block_mask.argtypes = [ctypes.POINTER(MaskDesc), ctypes.c_int, ctypes.c_int, i64, i64,
                                         ctypes.c_int, ctypes.POINTER(BlockMaskDesc), vp]
    lib.fa_create_block_mask_unsplit.argtypes = lib.fa_create_block_mask.argtypes
    lib.fa_workspace_size.argtypes = []
    lib.fa_workspace_size.restype = ctypes.c_size_t
    lib.fa_forward.argtypes = [ctypes.POINTER(TensorDesc)] * 3 + [
        ctypes.POINTER(BlockMaskDesc), ctypes.POINTER(ScoreModDesc), ctypes.c_float,
        ctypes.POINTER(TensorDesc), vp, vp, ctypes.c_size_t, vp]
    lib.fa_backward_workspace_size.argtypes = [i64, i64, i64, i64]
    lib.fa_backward_workspace_size.restype = ctypes.c_size_t
    lib.fa_backward.argtypes = [ctypes.POINTER(TensorDesc)] * 5 + [
        vp, ctypes.POINTER(BlockMaskDesc), ctypes.POINTER(ScoreModDesc), ctypes.c_float] + \
        [ctypes.POINTER(TensorDesc)] * 3 + [vp, ctypes.c_size_t, vp]
    lib.fa_forward_paged.argtypes = [ctypes.POINTER(TensorDesc)] * 3 + [vp, i64] + [
        ctypes.POINTER(BlockMaskDesc), ctypes.POINTER(ScoreModDesc), ctypes.c_float,
        ctypes.POINTER(TensorDesc), vp, vp, ctypes.c_size_t, vp]
    lib.fa_decode_workspace_size.argtypes = [i64] * 6
    lib.fa_decode_workspace_size.restype = ctypes.c_size_t
    lib.fa_decode.argtypes = lib.fa_forward.argtypes
    lib.fa_get_device_status.argtypes = [vp, vp]
    lib.fa_set_watchdog_ms.argtypes = [ctypes.c_int]
    lib.fa_set_selftest_stall.argtypes = [ctypes.c_int]
    lib.fa_forward_static_scratch.argtypes = [ctypes.POINTER(TensorDesc)] * 3 + [
        ctypes.POINTER(BlockMaskDesc), ctypes.POINTER(ScoreModDesc), ctypes.c_float,
        ctypes.POINTER(TensorDesc), vp, vp]
    td, ci, sz, f32 = ctypes.POINTER(TensorDesc), ctypes.c_int, ctypes.c_size_t, ctypes.c_float
    rope, score = ctypes.POINTER(RopeDesc), ctypes.POINTER(ScoreModDesc)
    lib.fa_rope_frequencies.argtypes = [ci, ctypes.c_double, ctypes.POINTER(RopeScalingDesc),
                                        ctypes.POINTER(ctypes.c_double), ctypes.POINTER(f32)]
    lib.fa_rope_apply.argtypes = [td, td, rope, vp, i64, i64, ci, td, td, vp]
    lib.fa_paged_append.argtypes = [td, td, td, rope, vp, vp, vp, i64, i64, td, td, td, vp, sz, vp]
    lib.fa_decode_paged_workspace_size.argtypes = [i64] * 5
    lib.fa_decode_paged_workspace_size.restype = sz
    lib.fa_decode_paged.argtypes = [td, td, td, vp, i64, i64, vp, i64, score, f32, td, vp, vp, sz, vp]
    lib.fa_decode_shared_workspace_size.argtypes = [i64] * 6
    lib.fa_decode_shared_workspace_size.restype = sz
    lib.fa_decode_shared.argtypes = lib.fa_decode_paged.argtypes
    return lib


_lib = _load()
if not os.path.exists(os.path.join(_HERE, "_binding.so")):
    raise ImportError("_binding.so is missing: build it with `python block_sparse_attention_48_b200/build.py`")
try:
    from . import _binding  # noqa: E402  (the serving calls' binding; needs torch loaded)
except ImportError as e:
    raise ImportError("_binding.so does not load, as after a change of torch or Python: build it again with "
                      "`python block_sparse_attention_48_b200/build.py`") from e
if _binding.torch_version != torch.__version__:
    raise ImportError(f"_binding.so was built against torch {_binding.torch_version}, this is {torch.__version__}: build "
                      "it again with `python block_sparse_attention_48_b200/build.py`")

_binding.bind(*[ctypes.cast(getattr(_lib, name), ctypes.c_void_p).value for name in
                ("fa_rope_apply", "fa_paged_append", "fa_decode_paged", "fa_decode_shared",
                 "fa_decode_paged_workspace_size", "fa_decode_shared_workspace_size", "fa_workspace_size")])


def library() -> ctypes.CDLL:
    return _lib


def status_string(status: int) -> str:
    return _lib.fa_status_string(int(status)).decode()


def _check(rc: int, what: str):
    if rc != FA_OK:
        raise FlexAttnError(rc, what)


def _stream_ptr(stream: Optional[torch.cuda.Stream]) -> ctypes.c_void_p:
    s = stream if stream is not None else torch.cuda.current_stream()
    return ctypes.c_void_p(s.cuda_stream)


def mask_desc(op: str, leaves: Sequence[tuple], doc_ids: Optional[torch.Tensor] = None,
              q_offset: int = 0) -> MaskDesc:
    if len(leaves) > MAX_LEAVES:
        raise ValueError("at most 4 mask leaves")
    m = MaskDesc()
    m.q_offset = int(q_offset)
    m.n_leaves = len(leaves)
    m.op = OP[op]
    for i, leaf in enumerate(leaves):
        m.kind[i] = LEAF[leaf[0]]
        m.param[i] = int(leaf[1]) if len(leaf) > 1 else 0
    if doc_ids is not None:
        if doc_ids.dim() == 1:
            doc_ids = doc_ids.unsqueeze(0)
        m.doc_ids = doc_ids.data_ptr()
        m.doc_stride = doc_ids.stride(0) if doc_ids.shape[0] > 1 else 0
        m.doc_len = doc_ids.shape[1]
    return m


TRANSPOSED = ("q_num_blocks", "q_indices", "full_q_num_blocks", "full_q_indices")


class BlockMask:
    """Device BlockMask: kv_num_blocks [B,H,nq], kv_indices [B,H,nq,nkv] (partial
    blocks) and full_kv_num_blocks / full_kv_indices (full blocks), int32 on the GPU;
    with transposed=True also q_num_blocks [B,H,nkv], q_indices [B,H,nkv,nq] and the
    full_q_* pair (the view the backward pass walks)."""

    def __init__(self, desc: BlockMaskDesc, tensors: dict, keep: list):
        self.desc = desc
        self.kv_num_blocks = tensors["kv_num_blocks"]
        self.kv_indices = tensors["kv_indices"]
        self.full_kv_num_blocks = tensors["full_kv_num_blocks"]
        self.full_kv_indices = tensors["full_kv_indices"]
        self.transposed = {k: tensors[k] for k in TRANSPOSED if k in tensors}
        self._keep = keep

    @property
    def shape(self) -> Tuple[int, int, int, int]:
        return (self.desc.B, self.desc.H, self.desc.nq, self.desc.nkv)

    def to_cpu(self) -> dict:
        return {"kv_num_blocks": self.kv_num_blocks.cpu().numpy(), "kv_indices": self.kv_indices.cpu().numpy(),
                "full_kv_num_blocks": self.full_kv_num_blocks.cpu().numpy(),
                "full_kv_indices": self.full_kv_indices.cpu().numpy()}

    def transposed_to_cpu(self) -> dict:
        return {k: t.cpu().numpy() for k, t in self.transposed.items()}

    def sparsity(self) -> float:
        """Share of empty blocks ("Concepts", Inspecting a BlockMask)."""
        B, H, nq, nkv = self.shape
        total = B * H * nq * nkv
        if total == 0:
            return 0.0
        used = int(self.kv_num_blocks.sum().item() + self.full_kv_num_blocks.sum().item())
        return 1.0 - used / total


def create_block_mask(op: str, leaves: Sequence[tuple], B: int, H: int, q_len: int, kv_len: int,
                      doc_ids: Optional[torch.Tensor] = None, device=None,
                      stream: Optional[torch.cuda.Stream] = None, split_full: bool = True,
                      transposed: bool = False, q_offset: int = 0) -> BlockMask:
    """create_block_mask(mask_mod, B, H, Q_LEN, KV_LEN) on the GPU (fa_create_block_mask).
    split_full=False builds the BlockMask without the full / partial split
    (fa_create_block_mask_unsplit): every non-empty tile is masked per element.
    transposed=True also builds the q_* view the backward pass needs.  q_offset:
    position of query row 0 (decoding after a cache of q_offset keys)."""
    device = torch.device(device) if device is not None else torch.device("cuda", torch.cuda.current_device())
    nq, nkv = ctypes.c_int32(), ctypes.c_int32()
    _check(_lib.fa_block_mask_shape(q_len, kv_len, BLOCK_SIZE, ctypes.byref(nq), ctypes.byref(nkv)),
           "fa_block_mask_shape")
    nq, nkv = nq.value, nkv.value
    keep = []
    if doc_ids is not None:
        # rows padded to a multiple of 4 ids (16 bytes): the kernels read ids in 16-byte vectors
        ids = doc_ids.to(device=device, dtype=torch.int32)
        ids = ids.unsqueeze(0) if ids.dim() == 1 else ids
        L = ids.shape[1]
        buf = torch.zeros((ids.shape[0], (L + 3) // 4 * 4), dtype=torch.int32, device=device)
        buf[:, :L] = ids
        doc_ids = buf[:, :L]
        keep.append(buf)
    t = {"kv_num_blocks": torch.empty((B, H, nq), dtype=torch.int32, device=device),
         "kv_indices": torch.empty((B, H, nq, nkv), dtype=torch.int32, device=device),
         "full_kv_num_blocks": torch.empty((B, H, nq), dtype=torch.int32, device=device),
         "full_kv_indices": torch.empty((B, H, nq, nkv), dtype=torch.int32, device=device)}
    d = BlockMaskDesc()
    d.kv_num_blocks = t["kv_num_blocks"].data_ptr()
    d.kv_indices = t["kv_indices"].data_ptr()
    d.full_kv_num_blocks = t["full_kv_num_blocks"].data_ptr()
    d.full_kv_indices = t["full_kv_indices"].data_ptr()
    if transposed:
        for name, shape in (("q_num_blocks", (B, H, nkv)), ("q_indices", (B, H, nkv, nq)),
                            ("full_q_num_blocks", (B, H, nkv)), ("full_q_indices", (B, H, nkv, nq))):
            t[name] = torch.empty(shape, dtype=torch.int32, device=device)
            setattr(d, name, t[name].data_ptr() if t[name].numel() else None)
    m = mask_desc(op, leaves, doc_ids, q_offset)
    with torch.cuda.device(device):
        fn = _lib.fa_create_block_mask if split_full else _lib.fa_create_block_mask_unsplit
        _check(fn(ctypes.byref(m), B, H, q_len, kv_len, BLOCK_SIZE, ctypes.byref(d), _stream_ptr(stream)),
               "fa_create_block_mask" if split_full else "fa_create_block_mask_unsplit")
    return BlockMask(d, t, keep)


def _expanded(t: torch.Tensor) -> bool:
    """True if a dimension of size > 1 has stride 0 (an expand()ed broadcast)."""
    return any(t.stride(i) == 0 and t.shape[i] > 1 for i in range(t.dim()))


def tensor_desc(t: torch.Tensor) -> TensorDesc:
    if t.dtype != torch.bfloat16 or t.dim() != 4 or not t.is_cuda:
        raise TypeError("expected a 4-D bf16 CUDA tensor [B, H, S, D]")
    if _expanded(t):
        raise TypeError("expanded (stride-0) dimensions of size > 1 are not accepted; materialise the tensor")
    d = TensorDesc()
    d.data = t.data_ptr()
    for i in range(4):
        d.dims[i] = t.shape[i]
        d.strides[i] = t.stride(i)
    return d


_workspaces = {}


def workspace(device: torch.device) -> torch.Tensor:
    """The per-device workspace (status word) used by default; zero-filled."""
    key = device.index if device.index is not None else torch.cuda.current_device()
    ws = _workspaces.get(key)
    if ws is None:
        ws = torch.zeros((int(_lib.fa_workspace_size()),), dtype=torch.uint8, device=device)
        _workspaces[key] = ws
    return ws


_decode_workspaces = {}


def decode_workspace(device: torch.device, need: int = 0) -> torch.Tensor:
    """The per-device workspace flex_decode uses by default: zero-filled when it is
    (re)allocated, at least `need` bytes; every fa_decode call leaves it ready for
    the next.  Calls that use it run one after another (one stream)."""
    key = device.index if device.index is not None else torch.cuda.current_device()
    ws = _decode_workspaces.get(key)
    if ws is None or ws.numel() < need:
        ws = torch.zeros((max(need, 256),), dtype=torch.uint8, device=device)
        _decode_workspaces[key] = ws
    return ws


def score_mod_desc(score_mod) -> Tuple[ScoreModDesc, list]:
    sm = ScoreModDesc()
    keep = []
    if score_mod is None or score_mod[0] == "none":
        sm.kind = SCORE["none"]
    elif score_mod[0] == "alibi":
        slopes = score_mod[1]
        if not (slopes.is_cuda and slopes.dtype == torch.float32 and slopes.is_contiguous()):
            raise TypeError("ALiBi slopes: contiguous fp32 CUDA tensor [Hq]")
        sm.kind = SCORE["alibi"]
        sm.alibi_slopes = slopes.data_ptr()
        keep.append(slopes)
    elif score_mod[0] == "softcap":
        sm.kind = SCORE["softcap"]
        sm.softcap = float(score_mod[1])
    elif score_mod[0] in ("bias", "bias_softcap"):
        b = score_mod[1]
        if not (b.is_cuda and b.dtype == torch.bfloat16 and b.dim() == 4):
            raise TypeError("bias: bf16 CUDA tensor [B, Hq, Sq, Skv]")
        # stride 0 over batch or heads is passed through (the kernel broadcasts it)
        if b.stride(3) != 1 or any(b.stride(i) % 8 for i in range(3)) or b.data_ptr() % 16 or \
                (b.stride(2) == 0 and b.shape[2] > 1):
            # TMA needs 16-byte row strides: copy into rows padded to 8 elements
            kl = b.shape[3]
            pad = torch.zeros(b.shape[:3] + ((kl + 7) // 8 * 8,), dtype=b.dtype, device=b.device)
            pad[..., :kl] = b
            b = pad[..., :kl]
        sm.kind = SCORE[score_mod[0]]
        if score_mod[0] == "bias_softcap":
            sm.softcap = float(score_mod[2])
        sm.bias = b.data_ptr()
        for i in range(4):
            sm.bias_strides[i] = b.stride(i)
        keep.append(b)
    else:
        raise ValueError(f"unknown score_mod {score_mod[0]!r}")
    return sm, keep


def flex_attention(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, block_mask: BlockMask,
                   score_mod=None, scale: Optional[float] = None, return_lse: bool = True,
                   out: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None,
                   ws: Optional[torch.Tensor] = None,
                   stream: Optional[torch.cuda.Stream] = None):
    """flex_attention(q, k, v, block_mask, score_mod) -> (out, lse) through fa_forward.

    q [B,Hq,Sq,D], k/v [B,Hkv,Skv,D] bf16 CUDA tensors (D contiguous).  Returns
    out [B,Hq,Sq,D] bf16 and lse [B,Hq,Sq] fp32 (natural log), or out alone."""
    # inputs expanded over a dimension (stride 0) are materialised: the kernels
    # address tiles by coordinates
    q, k, v = (t.contiguous() if _expanded(t) else t for t in (q, k, v))
    B, Hq, Sq, D = q.shape
    if out is None:
        out = torch.empty((B, Hq, Sq, D), dtype=torch.bfloat16, device=q.device)
    if return_lse and lse is None:
        lse = torch.empty((B, Hq, Sq), dtype=torch.float32, device=q.device)
    if lse is not None and not (lse.is_contiguous() and lse.dtype == torch.float32 and lse.shape == (B, Hq, Sq)):
        raise TypeError("lse: contiguous fp32 [B, Hq, Sq]")
    sm, keep = score_mod_desc(score_mod)
    ws = ws if ws is not None else workspace(q.device)
    qd, kd, vd, od = tensor_desc(q), tensor_desc(k), tensor_desc(v), tensor_desc(out)
    with torch.cuda.device(q.device):
        rc = _lib.fa_forward(ctypes.byref(qd), ctypes.byref(kd), ctypes.byref(vd), ctypes.byref(block_mask.desc),
                             ctypes.byref(sm), ctypes.c_float(scale if scale is not None else 0.0),
                             ctypes.byref(od), ctypes.c_void_p(lse.data_ptr() if lse is not None else 0),
                             ctypes.c_void_p(ws.data_ptr()), ctypes.c_size_t(ws.numel()), _stream_ptr(stream))
    _check(rc, "fa_forward")
    return (out, lse) if return_lse else out


def flex_decode(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, block_mask: BlockMask, score_mod=None,
                scale: Optional[float] = None, out: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None,
                ws: Optional[torch.Tensor] = None, stream: Optional[torch.cuda.Stream] = None):
    """FlexDecoding (fa_decode): a few query tokens (G * q_len <= 16 per kv head)
    against a long cache, split along KV and merged.  Build the BlockMask with
    q_offset = the position of the first query token."""
    B, Hq, Sq, D = q.shape
    out = out if out is not None else torch.empty((B, Hq, Sq, D), dtype=torch.bfloat16, device=q.device)
    lse = lse if lse is not None else torch.empty((B, Hq, Sq), dtype=torch.float32, device=q.device)
    need = int(_lib.fa_decode_workspace_size(B, Hq, k.shape[1], Sq, k.shape[2], D))
    if ws is None:
        ws = decode_workspace(q.device, need)
    elif ws.numel() < need:
        raise FlexAttnError(f"fa_decode: workspace of {ws.numel()} bytes, {need} needed")
    sm, keep = score_mod_desc(score_mod)
    qd, kd, vd, od = tensor_desc(q), tensor_desc(k), tensor_desc(v), tensor_desc(out)
    with torch.cuda.device(q.device):
        rc = _lib.fa_decode(ctypes.byref(qd), ctypes.byref(kd), ctypes.byref(vd), ctypes.byref(block_mask.desc),
                            ctypes.byref(sm), ctypes.c_float(scale if scale is not None else 0.0), ctypes.byref(od),
                            ctypes.c_void_p(lse.data_ptr()), ctypes.c_void_p(ws.data_ptr()),
                            ctypes.c_size_t(ws.numel()), _stream_ptr(stream))
    _check(rc, "fa_decode")
    return out, lse


def flex_attention_paged(q: torch.Tensor, k_pages: torch.Tensor, v_pages: torch.Tensor, page_table: torch.Tensor,
                         block_mask: BlockMask, score_mod=None, scale: Optional[float] = None,
                         out: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None,
                         ws: Optional[torch.Tensor] = None, stream: Optional[torch.cuda.Stream] = None):
    """flex_attention over a paged KV cache (fa_forward_paged): k_pages / v_pages
    [num_pages, Hkv, 128, D] bf16, page_table int32 [B, >= nkv] mapping logical kv
    block kb of batch b to a page; the BlockMask is over logical positions."""
    B, Hq, Sq, D = q.shape
    if not (page_table.is_cuda and page_table.dtype == torch.int32 and page_table.dim() == 2
            and page_table.stride(1) == 1):
        raise TypeError("page_table: int32 CUDA tensor [B, pages per sequence], rows contiguous")
    out = out if out is not None else torch.empty((B, Hq, Sq, D), dtype=torch.bfloat16, device=q.device)
    lse = lse if lse is not None else torch.empty((B, Hq, Sq), dtype=torch.float32, device=q.device)
    sm, keep = score_mod_desc(score_mod)
    ws = ws if ws is not None else workspace(q.device)
    qd, kd, vd, od = tensor_desc(q), tensor_desc(k_pages), tensor_desc(v_pages), tensor_desc(out)
    with torch.cuda.device(q.device):
        rc = _lib.fa_forward_paged(ctypes.byref(qd), ctypes.byref(kd), ctypes.byref(vd),
                                   ctypes.c_void_p(page_table.data_ptr()), page_table.stride(0),
                                   ctypes.byref(block_mask.desc), ctypes.byref(sm),
                                   ctypes.c_float(scale if scale is not None else 0.0), ctypes.byref(od),
                                   ctypes.c_void_p(lse.data_ptr()), ctypes.c_void_p(ws.data_ptr()),
                                   ctypes.c_size_t(ws.numel()), _stream_ptr(stream))
    _check(rc, "fa_forward_paged")
    return out, lse


def flex_attention_backward(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, out: torch.Tensor,
                            lse: torch.Tensor, grad_out: torch.Tensor, block_mask: BlockMask, score_mod=None,
                            scale: Optional[float] = None, dq: Optional[torch.Tensor] = None,
                            dk: Optional[torch.Tensor] = None, dv: Optional[torch.Tensor] = None,
                            ws: Optional[torch.Tensor] = None, stream: Optional[torch.cuda.Stream] = None):
    """Gradients (dq, dk, dv) of flex_attention through fa_backward, given the
    forward's out and lse and the upstream gradient.  block_mask must have been
    built with transposed=True.  ws, if given, is a uint8 device buffer of at least
    fa_backward_workspace_size bytes; its first word holds the device status."""
    q, k, v = (t.contiguous() if _expanded(t) else t for t in (q, k, v))
    grad_out = grad_out.contiguous() if _expanded(grad_out) else grad_out
    B, Hq, Sq, D = q.shape
    if not block_mask.transposed:
        raise ValueError("the backward pass needs a BlockMask built with transposed=True")
    if not (lse.is_contiguous() and lse.dtype == torch.float32 and lse.shape == (B, Hq, Sq)):
        raise TypeError("lse: contiguous fp32 [B, Hq, Sq]")
    dq = dq if dq is not None else torch.empty_like(q)
    dk = dk if dk is not None else torch.empty_like(k)
    dv = dv if dv is not None else torch.empty_like(v)
    need = int(_lib.fa_backward_workspace_size(B, Hq, Sq, D))
    if ws is None:
        # the prologue writes every row of the workspace it reads; only the status
        # word at its start needs a defined value
        with torch.cuda.stream(stream) if stream is not None else contextlib.nullcontext():
            ws = torch.empty((need,), dtype=torch.uint8, device=q.device)
            ws[:256].zero_()
    sm, keep = score_mod_desc(score_mod)
    descs = [tensor_desc(t) for t in (q, k, v, out, grad_out, dq, dk, dv)]
    with torch.cuda.device(q.device):
        rc = _lib.fa_backward(*[ctypes.byref(d) for d in descs[:5]], ctypes.c_void_p(lse.data_ptr()),
                              ctypes.byref(block_mask.desc), ctypes.byref(sm),
                              ctypes.c_float(scale if scale is not None else 0.0),
                              *[ctypes.byref(d) for d in descs[5:]], ctypes.c_void_p(ws.data_ptr()),
                              ctypes.c_size_t(ws.numel()), _stream_ptr(stream))
    _check(rc, "fa_backward")
    return dq, dk, dv


class FlexAttentionFunction(torch.autograd.Function):
    """flex_attention as a torch autograd function: forward through fa_forward,
    backward through fa_backward (the BlockMask must carry its transposed view)."""

    @staticmethod
    def forward(ctx, q, k, v, block_mask, score_mod, scale):
        out, lse = flex_attention(q, k, v, block_mask, score_mod=score_mod, scale=scale)
        ctx.save_for_backward(q, k, v, out, lse)
        ctx.block_mask, ctx.score_mod, ctx.scale = block_mask, score_mod, scale
        ctx.mark_non_differentiable(lse)
        return out, lse

    @staticmethod
    def backward(ctx, grad_out, grad_lse):
        q, k, v, out, lse = ctx.saved_tensors
        dq, dk, dv = flex_attention_backward(q, k, v, out, lse, grad_out.contiguous(), ctx.block_mask,
                                             score_mod=ctx.score_mod, scale=ctx.scale)
        return dq, dk, dv, None, None, None


def flex_attention_autograd(q, k, v, block_mask: BlockMask, score_mod=None, scale: Optional[float] = None):
    """Differentiable flex_attention: returns (out, lse); out.backward() runs fa_backward."""
    return FlexAttentionFunction.apply(q, k, v, block_mask, score_mod, scale)


# ------------------------------------------------------------------ rotary positions, paged cache

def _on_stream(fn):
    """Adds stream= to fn: the CUDA stream to run on (its own tensors are allocated for it)."""
    first = next(iter(inspect.signature(fn).parameters))

    @functools.wraps(fn)
    def call(*args, stream: Optional[torch.cuda.Stream] = None, **kw):
        if stream is None:
            return fn(*args, **kw)
        tensor = args[0] if args else kw.get(first)
        if not isinstance(tensor, torch.Tensor):
            raise TypeError(f"{fn.__name__}: {first}: expected a tensor, got {type(tensor).__name__}")
        if tensor.device != stream.device:
            raise ValueError(f"{fn.__name__}: the stream is on {stream.device}, the tensors on {tensor.device}")
        with torch.cuda.stream(stream):
            return fn(*args, **kw)
    return call


def paged_workspace(device: torch.device, need: int = 0) -> torch.Tensor:
    """The workspace paged_append, flex_decode_paged and flex_decode_shared use by
    default: one per device and stream, its first 16 KB (the status word and counters)
    zeroed when allocated; a larger one, at least twice as large, takes over its
    predecessor's status word and replaces it.  While a CUDA graph is captured each call
    gets a workspace of the graph's own instead (pass ws= to read the status of captured
    calls), of which every replay zeroes the same 16 KB.  A capture that torch.cuda.graph
    or CUDAGraph does not make has no memory of its own: pass ws= there."""
    return _binding.workspace(device.index if device.index is not None else torch.cuda.current_device(), need)


def _score(score_mod) -> tuple:
    """(kind, slopes, softcap) of a score_mod for _binding.decode."""
    if score_mod is None:
        return 0, None, 0.0
    kind = score_mod[0]
    if kind not in SCORE:
        raise ValueError(f"unknown score_mod {kind!r}")
    return SCORE[kind], score_mod[1] if kind == "alibi" else None, score_mod[1] if kind == "softcap" else 0.0


def rope_frequencies(rotary_dim: int, base: float = 10000.0, scaling: Optional[tuple] = None,
                     device=None) -> Tuple[torch.Tensor, float]:
    """Frequencies of rotary positions (fa_rope_frequencies): (inv_freq fp64
    [rotary_dim / 2] on the device, amplitude).  scaling: None, ("linear", factor),
    ("base", factor), ("bands", factor, original_len, rot_lo, rot_hi) or ("yarn", factor,
    original_len, rot_lo, rot_hi) with rot_lo < rot_hi in turns over original_len."""
    sc = None
    if scaling is not None:
        if scaling[0] not in ROPE_SCALING:
            raise ValueError(f"unknown rope scaling {scaling[0]!r}")
        if len(scaling) != (2 if scaling[0] in ("linear", "base") else 5):
            raise ValueError(f"rope scaling {scaling[0]!r}: wrong number of parameters")
        sc = RopeScalingDesc(ROPE_SCALING[scaling[0]], *[float(x) for x in scaling[1:]])
    host = (ctypes.c_double * max(1, rotary_dim // 2))()
    amplitude = ctypes.c_float()
    _check(_lib.fa_rope_frequencies(rotary_dim, base, ctypes.byref(sc) if sc is not None else None, host,
                                    ctypes.byref(amplitude)), "fa_rope_frequencies")
    inv_freq = torch.tensor(list(host), dtype=torch.float64)
    return inv_freq.to(device if device is not None else "cuda"), amplitude.value


@_on_stream
def rope_apply(q: torch.Tensor, k: Optional[torch.Tensor], inv_freq: torch.Tensor,
               positions: Optional[torch.Tensor] = None, interleaved: bool = False, amplitude: float = 1.0,
               inverse: bool = False, offset: int = 0, out: Optional[tuple] = None):
    """Rotary positions on q [B,Hq,S,D] and k [B,Hk,S,D] (or None) through fa_rope_apply:
    returns (q_out, k_out).  inv_freq: fp64 [rotary_dim / 2] (rope_frequencies), the
    first rotary_dim elements of a head are turned.  positions: int32 [B,S] or [S] (None:
    offset + s).  inverse=True turns the other way, which takes the gradients of the
    outputs to those of q and k.  out: (q_out, k_out), which may be (q, k).  stream=:
    the CUDA stream to run on."""
    q_out, k_out = out if out is not None else (None, None)
    r = _binding.rope_apply(q, k, inv_freq, positions, interleaved, amplitude, inverse, offset, q_out, k_out)
    return r if r.__class__ is tuple else _check(r, "fa_rope_apply")


class RopeFunction(torch.autograd.Function):
    """rope_apply as a torch autograd function (no gradient for the frequencies)."""

    @staticmethod
    def forward(ctx, q, k, inv_freq, positions, interleaved, amplitude, offset):
        ctx.save_for_backward(inv_freq, positions)
        ctx.opts = dict(interleaved=interleaved, amplitude=amplitude, offset=offset)
        out = rope_apply(q, k, inv_freq, positions=positions, **ctx.opts)
        return out if k is not None else out[0]

    @staticmethod
    @once_differentiable
    def backward(ctx, grad_q, grad_k=None):
        inv_freq, positions = ctx.saved_tensors
        gq, gk = rope_apply(grad_q, grad_k, inv_freq, positions=positions, inverse=True, **ctx.opts)
        return gq, gk, None, None, None, None, None


def rope_autograd(q, k, inv_freq, positions=None, interleaved: bool = False, amplitude: float = 1.0, offset: int = 0):
    """Differentiable rope_apply: returns (q_out, k_out)."""
    out = RopeFunction.apply(q, k, inv_freq, positions, interleaved, amplitude, offset)
    return out if k is not None else (out, None)


@_on_stream
def paged_append(k: torch.Tensor, v: torch.Tensor, k_pages: torch.Tensor, v_pages: torch.Tensor,
                 page_table: torch.Tensor, cache_lens: torch.Tensor, new_lens: Optional[torch.Tensor] = None,
                 q: Optional[torch.Tensor] = None, q_out: Optional[torch.Tensor] = None,
                 inv_freq: Optional[torch.Tensor] = None, interleaved: bool = False, amplitude: float = 1.0,
                 ws: Optional[torch.Tensor] = None):
    """Append k, v [B,Hkv,S,D] to a paged cache (fa_paged_append): token s of sequence b
    goes to position cache_lens[b] + s, rotated there when inv_freq is given (k, and q
    [B,Hq,S,D] into q_out), if s < new_lens[b] (None: all).  k_pages / v_pages
    [num_pages,Hkv,128,D] are written in place; page_table int32 [B, pages],
    cache_lens / new_lens int32 [B] are not changed.  Returns q_out (None without q;
    rows past new_lens are left as they were, zero in a q_out made here).  Bad lengths
    and pages: device_status(ws)."""
    r = _binding.paged_append(k, v, k_pages, v_pages, page_table, cache_lens, new_lens, q, q_out, inv_freq, interleaved,
                              amplitude, ws)
    return _check(r, "fa_paged_append") if r.__class__ is int else r


@_on_stream
def flex_decode_paged(q: torch.Tensor, k_pages: torch.Tensor, v_pages: torch.Tensor, page_table: torch.Tensor,
                      seq_lens: torch.Tensor, window: Optional[int] = None, score_mod=None,
                      scale: Optional[float] = None, out: Optional[torch.Tensor] = None,
                      lse: Optional[torch.Tensor] = None, ws: Optional[torch.Tensor] = None):
    """FlexDecoding over a paged cache (fa_decode_paged): q [B,Hq,q_len,D], at most 16
    query rows per kv head ((Hq / Hkv) * q_len), k_pages / v_pages [num_pages,Hkv,128,D],
    page_table int32 [B, pages], seq_lens int32 [B] (each sequence's keys, the new tokens'
    included).  Query token i of sequence b sits at position seq_lens[b] - q_len + i and
    attends the keys at or before it, with window= also at or after it - window.
    score_mod: None, ("alibi", slopes) or ("softcap", cap).  Returns (out, lse)."""
    if window is not None and window < 0:
        raise ValueError("flex_decode_paged: window must not be negative")
    r = _binding.decode(False, q, k_pages, v_pages, page_table, seq_lens, -1 if window is None else window,
                        *_score(score_mod), 0.0 if scale is None else scale, out, lse, ws)
    return r if r.__class__ is tuple else _check(r, "fa_decode_paged")


@_on_stream
def flex_decode_shared(q: torch.Tensor, k_pages: torch.Tensor, v_pages: torch.Tensor, page_table: torch.Tensor,
                       seq_lens: torch.Tensor, prefix_len: int, score_mod=None, scale: Optional[float] = None,
                       out: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None,
                       ws: Optional[torch.Tensor] = None):
    """flex_decode_paged for sequences that share their first prefix_len keys (a multiple
    of 128: the first prefix_len / 128 entries of every row of page_table are the same
    pages), which are taken once for the whole batch (fa_decode_shared).  They are read from
    row 0, whatever sequence 0's length; a sequence that ends in the prefix is taken from its
    own row."""
    r = _binding.decode(True, q, k_pages, v_pages, page_table, seq_lens, prefix_len, *_score(score_mod),
                        0.0 if scale is None else scale, out, lse, ws)
    return r if r.__class__ is tuple else _check(r, "fa_decode_shared")


def device_status(ws: Optional[torch.Tensor] = None, device=None, stream=None) -> int:
    """Synchronise and return (and clear) the device status of earlier forward calls."""
    device = torch.device(device) if device is not None else torch.device("cuda", torch.cuda.current_device())
    ws = ws if ws is not None else workspace(device)
    return int(_lib.fa_get_device_status(ctypes.c_void_p(ws.data_ptr()), _stream_ptr(stream)))


def set_watchdog_ms(ms: int):
    _check(_lib.fa_set_watchdog_ms(int(ms)), "fa_set_watchdog_ms")


def set_selftest_stall(on: bool):
    """Watchdog self-test: while on, every forward launch stalls its producer
    until the watchdog limit runs out and reports FA_ERR_TIMEOUT."""
    _check(_lib.fa_set_selftest_stall(1 if on else 0), "fa_set_selftest_stall")
